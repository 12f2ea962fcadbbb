"""Plain definitions of the operators around the verify step (test infrastructure only): rotary
positions with several axes, acceptance from given probabilities and random numbers, and the pages
of a paged cache.  numpy and Python integers; no code of the CUDA library.
"""
from __future__ import annotations

import itertools

import numpy as np

PAGE = 16
BAD_ENTRY, EXHAUSTED, BAD_REQUEST, BAD_COUNT = 1, 8, 16, 32


# ------------------------------------------------------------------ rotary positions


def _inverse_two_pi(bits):
    """floor(2^bits / (2 pi)), pi by Machin's formula in integers."""
    work = bits + 32

    def arctan_inverse(x):
        term = (1 << work) // x
        total, k, sign = term, 1, -1
        while term:
            term //= x * x
            k += 2
            total += sign * (term // k)
            sign = -sign
        return total

    pi = 4 * (4 * arctan_inverse(5) - arctan_inverse(239))
    return (1 << (bits + work)) // (2 * pi)


_BITS = 256
_TURN = _inverse_two_pi(_BITS)


def angle(position: int, inv_freq: float) -> float:
    """position * inv_freq modulo 2 pi, in [-pi, pi): exact integers up to the last rounding."""
    num, den = float(inv_freq).as_integer_ratio()
    turns = (int(position) * num * _TURN // den) % (1 << _BITS)
    if turns >= 1 << (_BITS - 1):
        turns -= 1 << _BITS
    return turns / (1 << _BITS) * 2.0 * np.pi


def rope(x, positions, inv_freq, axis, adjacent=False, scale=1.0, inverse=False):
    """x [B, T, H, D] -> the rotated tensor in binary64; positions [axes, B, T]."""
    y = np.array(x, np.float64)
    P = len(inv_freq)
    B, T = y.shape[:2]
    for b, t, i in itertools.product(range(B), range(T), range(P)):
        a = angle(positions[axis[i]][b][t], inv_freq[i])
        c, s = np.cos(a), -np.sin(a) if inverse else np.sin(a)
        m, n = (2 * i, 2 * i + 1) if adjacent else (i, i + P)
        u, v = y[b, t, :, m].copy(), y[b, t, :, n].copy()
        y[b, t, :, m] = scale * (u * c - v * s)
        y[b, t, :, n] = scale * (v * c + u * s)
    return y


# ------------------------------------------------------------------ acceptance


def fixed54(p):
    """Probabilities as multiples of 2^-54, Python integers: NaN and negative 0, above one 1."""
    p = np.asarray(p, np.float64)
    p = np.where(np.isnan(p), 0.0, np.clip(p, 0.0, 1.0))
    return [int(v) for v in np.rint(p * 2.0 ** 54).astype(np.uint64)]


def accept_probs(p, drafts, u_accept, u_emit, q=None, lens=None):
    """(out_tokens [B, T + 1], num_accepted [B]) of p [B, T + 1, V], drafts [B, T], uniforms
    u_accept [B, T] and u_emit [B], q [B, T, V] or None, lens [B] or None."""
    p = np.asarray(p, np.float64)
    B, T1, V = p.shape
    T = T1 - 1
    out, nacc = np.full((B, T1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        count = T if lens is None else min(max(int(lens[b]), 0), T)
        n = 0
        while n < count:
            d = int(drafts[b][n])
            if not 0 <= d < V:
                break
            q_d = 1.0 if q is None else float(q[b][n][d])
            if not float(u_accept[b][n]) * q_d < p[b, n, d]:
                break
            out[b, n] = d
            n += 1
        nacc[b] = n
        full = fixed54(p[b, n])
        weights = full
        if n < count:
            if q is None:
                weights = [0 if i == int(drafts[b][n]) else w for i, w in enumerate(full)]
            else:
                weights = [max(0, w - v) for w, v in zip(full, fixed54(q[b][n]))]
            if not any(weights):
                weights = full
        total = sum(weights)
        if total == 0:
            continue
        u = float(u_emit[b])
        u = min(u, 1.0 - 2.0 ** -24) if u > 0 else 0.0
        num, den = u.as_integer_ratio()
        for i, s in enumerate(itertools.accumulate(weights)):
            if s * den > num * total:
                out[b, n] = i
                break
    return out, nacc


# ------------------------------------------------------------------ pages


def blocks(n):
    return -(-n // PAGE)


class Pages:
    """A page pool on the host, its calls carried out one entry after the other."""

    def __init__(self, num_pages, num_seqs, stride, buffers=()):
        self.table = np.full((num_seqs, stride), -1, np.int64)
        self.lens = np.zeros(num_seqs, np.int64)
        self.ref = np.zeros(num_pages, np.int64)
        self.stack = np.arange(num_pages - 1, -1, -1)
        self.num_free = num_pages
        self.flags = 0
        self.buffers = [np.array(b) for b in buffers]

    def _push(self, pages):
        for page in sorted(pages):
            self.stack[self.num_free] = page
            self.num_free += 1

    def _take(self):
        self.num_free -= 1
        page = int(self.stack[self.num_free])
        self.ref[page] = 1
        return page

    def _copy(self, pairs):
        for x in self.buffers:
            for src, dst in pairs:
                x[dst] = x[src]

    def resize(self, new_lens, kept=None):
        B, stride = self.table.shape
        new = [int(n) for n in new_lens]
        cut = [int(n) for n in (self.lens if kept is None else kept)]
        for b in range(B):
            if new[b] > PAGE * stride or (new[b] >= 0 and not 0 <= cut[b] <= self.lens[b]):
                self.flags |= BAD_REQUEST
                new[b] = -1
            cut[b] = min(cut[b], new[b])
        gone = []
        for b in range(B):
            if 0 <= cut[b] < self.lens[b]:
                for j in range(blocks(cut[b]), blocks(int(self.lens[b]))):
                    page = int(self.table[b, j])
                    self.table[b, j] = -1
                    self.ref[page] -= 1
                    if self.ref[page] == 0:
                        gone.append(page)
                self.lens[b] = cut[b]
        self._push(gone)
        # what a sequence needs goes by the counts before any sequence has grown
        plan = []
        for b in range(B):
            if new[b] > self.lens[b]:
                L = int(self.lens[b])
                own = L % PAGE != 0 and self.ref[self.table[b, L // PAGE]] > 1
                plan.append((b, own, blocks(new[b]) - blocks(L) + int(own)))
        pairs, left, short = [], [], False
        for b, own, need in plan:
            short = short or need > self.num_free
            if need and short:
                self.flags |= EXHAUSTED
                continue
            L = int(self.lens[b])
            if own:
                page = self._take()
                pairs.append((int(self.table[b, L // PAGE]), page))
                left.append(int(self.table[b, L // PAGE]))
                self.table[b, L // PAGE] = page
            for j in range(blocks(L), blocks(new[b])):
                self.table[b, j] = self._take()
            self.lens[b] = new[b]
        gone = []
        for page in left:
            self.ref[page] -= 1
            if self.ref[page] == 0:
                gone.append(page)
        self._push(gone)
        self._copy(pairs)

    def fork(self, parents, children, lens=None, share=True):
        B = len(self.lens)
        before, taken, pairs, short = self.lens.copy(), set(), [], False
        for f, (p, c) in enumerate(zip(parents, children)):
            p, c = int(p), int(c)
            first = c not in taken
            taken.add(c)
            n = -1
            if 0 <= p < B and 0 <= c < B and before[c] == 0 and first:
                n = int(before[p]) if lens is None else int(lens[f])
                if not 0 <= n <= before[p]:
                    n = -1
            if n < 0:
                self.flags |= BAD_REQUEST
                continue
            full = n // PAGE if share else 0
            need = blocks(n) - full
            short = short or need > self.num_free
            if need and short:
                self.flags |= EXHAUSTED
                continue
            for j in range(full):
                self.table[c, j] = self.table[p, j]
                self.ref[self.table[p, j]] += 1
            for j in range(full, blocks(n)):
                page = self._take()
                pairs.append((int(self.table[p, j]), page))
                self.table[c, j] = page
            self.lens[c] = n
        self._copy(pairs)

    def compact(self):
        P = len(self.ref)
        held = [p for p in range(P) if self.ref[p] > 0]
        n = len(held)
        places = [p for p in range(n) if self.ref[p] == 0]
        pairs = list(zip([p for p in held if p >= n], places))
        to = dict(pairs)
        for b in range(len(self.lens)):
            for j in range(blocks(int(self.lens[b]))):
                self.table[b, j] = to.get(int(self.table[b, j]), int(self.table[b, j]))
        for src, dst in pairs:
            self.ref[dst], self.ref[src] = self.ref[src], 0
        self._copy(pairs)
        self.num_free = P - n
        self.stack[:P - n] = np.arange(P - 1, n - 1, -1)

    def check(self):
        """Counts, lists and tables say the same."""
        count = np.zeros_like(self.ref)
        for b in range(len(self.lens)):
            for j in range(blocks(int(self.lens[b]))):
                count[self.table[b, j]] += 1
        assert np.array_equal(count, self.ref)
        free = sorted(self.stack[:self.num_free])
        assert free == [p for p in range(len(self.ref)) if self.ref[p] == 0]
