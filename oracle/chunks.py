"""Plain definitions of the operators of a prompt worked in chunks (test infrastructure only): attention of
ragged chunks over a paged cache, the weight that cached tokens gather, eviction by it, and log
probabilities.  numpy in 64 bits; no code of the CUDA library.
"""
from __future__ import annotations

import numpy as np

PAGE = 16
BAD_ENTRY, BAD_REQUEST = 1, 16


def e4m3(codes):
    """OCP e4m3 bytes as numbers: 1 sign, 4 exponent (bias 7), 3 mantissa bits; 0x7F and 0xFF are NaN, no infinities."""
    c = np.asarray(codes, np.uint8).astype(np.int64)
    e, m = (c >> 3) & 15, c & 7
    x = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    x = np.where((c & 127) == 127, np.nan, x)
    return np.where(c & 128, -x, x)


def decode(pages, kv_dtype):
    """Codes of a cache [.., row] as numbers [.., D]; a bf16 cache comes as its 16-bit patterns."""
    if kv_dtype == "bf16":
        return (np.asarray(pages).view(np.uint16).astype(np.uint32) << 16).view(np.float32).astype(np.float64)
    if kv_dtype == "fp8_e4m3":
        return e4m3(np.asarray(pages).view(np.uint8))
    if kv_dtype == "int8":
        return np.asarray(pages).view(np.int8).astype(np.float64)
    bits = {"int4": 4, "int2": 2}[kv_dtype]
    b = np.asarray(pages).view(np.uint8).astype(np.int64)
    x = np.stack([(b >> at) & ((1 << bits) - 1) for at in range(0, 8, bits)], -1).reshape(*b.shape[:-1], -1)
    return np.where(x >= 1 << (bits - 1), x - (1 << bits), x).astype(np.float64)


def rows(pages, scale, table, L, g, kv_dtype, num_pages):
    """(keys or values [L, D] of kv head g, which of them there are): entries outside the pool are absent."""
    at = np.asarray(table)[np.arange(L) // PAGE]
    there = (at >= 0) & (at < num_pages)
    at = np.where(there, at, 0)
    x = decode(pages[at, np.arange(L) % PAGE, g], kv_dtype)
    if scale is not None:
        x = x * np.asarray(scale, np.float64)[at, np.arange(L) % PAGE, g][:, None]
    return x, there


def scores(q, keys, there, L, n):
    """[n, L] scaled scores of one head's n new tokens, -inf where a key is not seen."""
    with np.errstate(invalid="ignore", over="ignore"):
        x = np.asarray(q, np.float64) @ np.where(there[:, None], keys, 0.0).T / np.sqrt(q.shape[-1])
    seen = there[None, :] & (np.arange(L)[None, :] <= (np.arange(n) + L - n)[:, None])
    return np.where(seen, x, -np.inf), seen


def chunk(q, k_pages, v_pages, k_scale, v_scale, table, chunk_lens, seq_lens, kv_dtype, num_kv_heads):
    """q [N, Hq, D] -> (out, lse, (size, small), reach), the last two for error bounds: size [N, Hq, D] is sum p |V|; small the
    sum of |V| times (the largest value scale over the key's) over the keys whose probability, relative to the likeliest
    key's, times their value scale, relative to the largest, is below 2^-8; reach what the scores are made of, sum |q||k| /
    sqrt(D) at most."""
    N, Hq, D = q.shape
    G = Hq // num_kv_heads
    out, lse = np.zeros((N, Hq, D)), np.full((N, Hq), -np.inf)
    size, small, reach = np.zeros((N, Hq, D)), np.zeros((N, Hq, D)), np.zeros((N, Hq))
    at = 0
    for b, (n, L) in enumerate(zip(chunk_lens, seq_lens)):
        for g in range(num_kv_heads if n else 0):
            K, there = rows(k_pages, k_scale, table[b], L, g, kv_dtype, k_pages.shape[0])
            V, _ = rows(v_pages, v_scale, table[b], L, g, kv_dtype, k_pages.shape[0])
            at_v = np.where(there, np.asarray(table[b])[np.arange(L) // PAGE], 0)
            sv = np.ones(L) if v_scale is None else np.asarray(v_scale, np.float64)[at_v, np.arange(L) % PAGE, g]
            for h in range(g * G, g * G + G):
                x, seen = scores(q[at:at + n, h], K, there, L, n)
                for t in range(n):  # keys that are not seen have no part, whatever they hold
                    s = seen[t]
                    if not s.any():
                        continue
                    y = x[t, s]
                    m = y.max()
                    p = np.exp(y - m)
                    least = p * sv[s] < 2.0 ** -8 * sv[s].max()
                    if least.any():
                        with np.errstate(invalid="ignore", divide="ignore"):
                            small[at + t, h] = (np.abs(V[s][least]) * (sv[s].max() / sv[s][least])[:, None]).sum(0)
                    lse[at + t, h] = m + np.log(p.sum())
                    p /= p.sum()
                    with np.errstate(invalid="ignore"):
                        out[at + t, h] = p @ V[s]
                        size[at + t, h] = p @ np.abs(V[s])
                        reach[at + t, h] = (np.abs(q[at + t, h]) @ np.abs(K[s]).T).max() / np.sqrt(D)
        at += n
    return out, lse, (size, small), reach


def chunk_weights(q, k_pages, k_scale, table, chunk_lens, seq_lens, kv_dtype, num_kv_heads, lse, old):
    """weights [B, Hkv, slots]: old ones added to at the tokens that were cached before (None: set), set at the new ones;
    and the largest sum |q||k| / sqrt(D) that went into each."""
    B, Hkv = len(chunk_lens), num_kv_heads
    G = q.shape[1] // Hkv
    w = np.zeros((B, Hkv, max(seq_lens))) if old is None else np.array(old, np.float64)
    at = 0
    for b, (n, L) in enumerate(zip(chunk_lens, seq_lens)):
        for g in range(Hkv if n else 0):
            K, there = rows(k_pages, k_scale, table[b], L, g, kv_dtype, k_pages.shape[0])
            total = np.zeros(L)
            for h in range(g * G, g * G + G):
                x, seen = scores(q[at:at + n, h], K, there, L, n)
                z = np.asarray(lse[at:at + n, h], np.float64)[:, None]
                with np.errstate(invalid="ignore", over="ignore"):
                    total += np.where(seen & ~np.isneginf(z), np.exp(x - z), 0.0).sum(0)
            keep = L - n if old is not None else 0
            w[b, g, :keep] += total[:keep]
            w[b, g, keep:L] = total[keep:]
        at += n
    return w


def evict(buffers, table, seq_lens, weights, keep, slot_pos=None, num_sinks=0, recent_from=None, ref_count=None,
          num_pages=None):
    """Changes buffers (each [pages, 16, Hkv, ..]), weights and slot_pos in place, one token after the other; returns (new
    lengths, flags)."""
    B, Hkv, slots = weights.shape
    new, flags = np.array(seq_lens).copy(), 0
    for b in range(B):
        L, want = int(seq_lens[b]), int(keep[b])
        if L < 0 or L > slots or L > table.shape[1] * PAGE:
            flags |= BAD_REQUEST
            continue
        if want < 0 or want >= L:
            continue
        used = table[b, :(L + PAGE - 1) // PAGE]
        bad = (used < 0) | (used >= num_pages)
        wrong = BAD_ENTRY if bad.any() else 0
        if ref_count is not None and (ref_count[used[~bad]] > 1).any():
            wrong |= BAD_REQUEST
        if wrong:
            flags |= wrong
            continue
        new[b] = want
        for g in range(Hkv):
            def rank(j):
                pos = j if slot_pos is None else slot_pos[b, g, j]
                if pos < num_sinks or (recent_from is not None and pos >= recent_from[b]):
                    return (2, 0.0)
                w = float(weights[b, g, j])
                return (0, 0.0) if np.isnan(w) else (1, w)
            order = sorted(range(L), key=lambda j: (rank(j), -j), reverse=True)
            kept = set(order[:want])
            holes = [j for j in range(want) if j not in kept]
            for src, dst in zip(sorted(j for j in kept if j >= want), holes):
                for x in buffers:
                    x[used[dst // PAGE], dst % PAGE, g] = x[used[src // PAGE], src % PAGE, g]
                weights[b, g, dst] = weights[b, g, src]
                if slot_pos is not None:
                    slot_pos[b, g, dst] = slot_pos[b, g, src]
    return new, flags


def logprobs(x, tokens, top):
    """Row by row in 64 bits: (logprobs, ranks, entropy, top tokens, top logprobs, (Z', S) for error bounds)."""
    x = np.asarray(x, np.float64)
    N, V = x.shape
    lp, ent = np.full(N, -np.inf), np.zeros(N)
    ranks, tt, tl = np.full(N, -1, np.int64), np.zeros((N, top), np.int64), np.zeros((N, top))
    parts = np.zeros((N, 2))
    for n in range(N):
        r = x[n]
        order = sorted(range(V), key=lambda i: (np.isnan(r[i]), 0.0 if np.isnan(r[i]) else -r[i], i))
        tt[n] = order[:top]
        t = int(tokens[n])
        known = 0 <= t < V
        if known:
            ranks[n] = order.index(t)
        if np.isnan(r).any() or np.isposinf(r).any():
            ent[n], tl[n] = np.nan, np.nan
            lp[n] = np.nan if known else -np.inf
            continue
        m = r.max()
        if np.isneginf(m):
            tl[n] = -np.inf
            continue
        d = r - m
        e = np.exp(d)
        e[order[0]] = 0.0
        Z = e.sum()
        S = (e[e > 0] * d[e > 0]).sum()
        l = d - np.log1p(Z)
        parts[n] = Z, S
        tl[n] = l[tt[n]]
        if known:
            lp[n] = l[t]
        ent[n] = np.log1p(Z) - S / (1 + Z)
    return lp, ranks, ent, tt, tl, parts
