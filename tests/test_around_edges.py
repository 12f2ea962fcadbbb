"""Edges of the operators around the verify step on the CPU: sequences that are cut back into pages that a fork shares,
frequencies above one, inputs that require a gradient, head counts and strides at their limits."""
import ctypes
from fractions import Fraction

import numpy as np
import pytest

from oracle import around
import speculative_decoding_verify_causal_gb300 as va
from speculative_decoding_verify_causal_gb300 import build as vbuild

from test_around_oracle import _heads, _pool, _rope


@pytest.fixture(scope="module", autouse=True)
def built():
    vbuild.build()


# ------------------------------------------------------------------ pages


class Tokens:
    """What each sequence of a pool should read: its tokens, written through the table as they come."""

    def __init__(self, pool):
        self.pool, self.seqs, self.next = pool, [[] for _ in pool.lens], 1

    def write(self, b, kept):
        """The block of sequence b, tokens kept .. its length - 1, as an append writes it."""
        self.seqs[b] = self.seqs[b][:kept]
        for at in range(kept, int(self.pool.lens[b])):
            self.seqs[b].append(self.next)
            self.pool.buffers[0][self.pool.table[b, at // 16], at % 16] = self.next
            self.next += 1

    def check(self):
        for b, tokens in enumerate(self.seqs):
            n = int(self.pool.lens[b])
            assert [self.pool.buffers[0][self.pool.table[b, i // 16], i % 16] for i in range(n)] == tokens[:n], b


@pytest.mark.parametrize("kept,new", [([20, 20], [36, 36]), ([20, 27], [36, 31]), ([3, 32], [19, 48]), ([16, 17], [32, 32]),
                                      ([31, 0], [32, 16]), ([20, 20], [30, 32])])
def test_a_fork_made_before_the_drafts_were_decided_keeps_its_tokens(kept, new):
    """32 tokens, the last 16 of them drafts, are forked with their full pages shared; then both sequences keep what was
    accepted and write their next blocks."""
    pool = around.Pages(16, 2, 4, [np.zeros((16, 16), np.int64)])
    tokens = Tokens(pool)
    pool.resize([32, 0])
    tokens.write(0, 0)
    pool.fork([0], [1])
    tokens.seqs[1] = list(tokens.seqs[0])
    pool.resize(new, kept=kept)
    pool.check()
    for b in (0, 1):
        tokens.write(b, kept[b])
    tokens.check()
    assert pool.flags == 0 and pool.lens.tolist() == new


@pytest.mark.parametrize("seed", range(6))
def test_resize_with_kept_lengths_is_two_calls(seed):
    rng = np.random.default_rng(seed)
    make = lambda: around.Pages(40, 5, 8, [np.arange(40 * 4).reshape(40, 4)])  # noqa: E731
    a, b = make(), make()
    for _ in range(60):
        if rng.random() < 0.3:
            args = rng.integers(0, 5, 2), rng.integers(0, 5, 2)
            a.fork(*args)
            b.fork(*args)
        kept = rng.integers(0, a.lens + 1)
        new = np.where(rng.random(5) < 0.2, -1, np.minimum(kept + rng.integers(-10, 30, 5), 128).clip(0))
        a.resize(new, kept=kept)
        b.resize(np.where(new < 0, -1, np.minimum(kept, new)))
        b.resize(new)
        a.check()
        for x, y in zip((a.table, a.lens, a.ref, a.stack[:a.num_free], a.buffers[0], a.flags),
                        (b.table, b.lens, b.ref, b.stack[:b.num_free], b.buffers[0], b.flags)):
            assert np.array_equal(x, y)


def test_resize_refuses_kept_lengths_that_are_not_there():
    pool = around.Pages(8, 4, 4)
    pool.resize([20, 20, 20, 0])
    pool.resize([30, 30, -1, 5], kept=[21, -1, 99, 0])
    assert pool.flags == around.BAD_REQUEST and pool.lens.tolist() == [20, 20, 20, 5]


def test_resize_ex_refusals():
    lib, s = va.library(), _pool()
    ref = ctypes.byref(s)
    assert lib.verify_attn_pages_resize_ex(None, None, 4096, None) == -1
    assert lib.verify_attn_pages_resize_ex(ref, None, None, None) == -1
    assert lib.verify_attn_pages_resize_ex(ref, 4096, None, None) == -1
    assert lib.verify_attn_pages_resize_ex(ref, 4098, 4096, None) == -1
    assert lib.verify_attn_pages_resize_ex(ref, 4096, 4098, None) == -1


# ------------------------------------------------------------------ rotary


def test_rope_spec_rounds_the_part_of_a_turn_correctly():
    """turn[i] is inv_freq / (2 pi) to half a unit of 2^-64, whatever the frequency: at the largest position that is 2^-34
    of a turn."""
    rng = np.random.default_rng(1)
    freq = [2.0 ** 20, -(2.0 ** 20), 3.0e4, 1024.0, 129.0, 7.5, 1.0, 0.37, -0.25, 1e-3, 3e-30, 0.0, 2.0 ** -66, 1e-18]
    freq += list(2.0 ** rng.uniform(-30, 20, 100) * rng.choice([-1, 1], 100))
    spec = va.verify_attn_rope_spec(2 * len(freq), inv_freq=freq)
    for i, f in enumerate(freq):
        exact = Fraction(f) * Fraction(around._TURN, 2 ** around._BITS) * 2 ** 64
        err = (Fraction(spec._struct.turn[i]) - exact) % 2 ** 64
        assert min(err, 2 ** 64 - err) <= Fraction(1, 2) + Fraction(1, 2 ** 20), f


def test_calls_that_would_lose_a_gradient_are_refused():
    """Before anything else is looked at; without grad mode or on detached tensors the call goes on (to the next refusal
    here, which is that there is no GPU)."""
    torch = pytest.importorskip("torch")
    rope = va.verify_attn_rope_spec(16)
    pos = torch.zeros(1, 1, 2, dtype=torch.int32)
    x, w = torch.zeros(1, 2, 3, 16), torch.zeros(1, 2, 3, 16, requires_grad=True)
    for kw in (dict(q=w), dict(q=x, k=w), dict(q=w, q_out=w), dict(q=x, q_out=w), dict(q=x, k=x, k_out=w), dict(q=w * 2)):
        with pytest.raises(ValueError, match="gradient"):
            va.verify_attn_rope(rope, pos, **kw)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            va.verify_attn_rope(rope, pos, **kw)
    with pytest.raises(ValueError, match="CUDA"):
        va.verify_attn_rope(rope, pos, w.detach())
    for q, k, v in ((w, x, x), (x, w, x), (x, x, w), (None, w, x)):
        with pytest.raises(ValueError, match="gradient"):
            va.verify_attn_rope_append(rope, pos, q, k, v, x, x, x, x, pos, pos, "int8")
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            va.verify_attn_rope_append(rope, pos, q, k, v, x, x, x, x, pos, pos, "int8")


@pytest.mark.parametrize("change", [
    dict(k=_heads(4096, 2 ** 40, 2 ** 38, 16, 2 ** 31 - 1), k_out=_heads(8192, 2 ** 40, 2 ** 38, 16, 2 ** 31 - 1)),
    dict(q=_heads(4096, 2 ** 24, 2 ** 22, 16, 65535), q_out=_heads(8192, 2 ** 24, 2 ** 22, 16, 65535),
         k=_heads(4096), k_out=_heads(8192)),
    # outputs whose elements lie on one another, with extents past 63 bits
    dict(B=5, T=3, q_out=_heads(8192, seq=2 ** 61, token=2 ** 62, head=16)),
    dict(T=2, B=2 ** 20, q_out=_heads(8192, seq=2 ** 44, token=2 ** 63 - 1, head=16)),
])
def test_rope_refuses_counts_and_extents_that_wrap(change):
    """More than 65,535 heads in sum: their sum once wrapped and ended the process with a division by zero."""
    assert _rope(**change) == -1
