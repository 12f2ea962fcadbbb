"""Pins of the plain definitions of the operators around the verify step, and the refusals of their
entry points (all on the CPU: a refused call touches no device)."""
import ctypes

import numpy as np
import pytest

from oracle import around
import speculative_decoding_verify_causal_gb300 as va
from speculative_decoding_verify_causal_gb300 import build as vbuild


@pytest.fixture(scope="module", autouse=True)
def built():
    vbuild.build()


# ------------------------------------------------------------------ rotary


def test_angle_is_the_product_modulo_a_turn():
    assert around.angle(0, 0.37) == 0.0
    assert abs(around.angle(5, 0.25) - 1.25) < 1e-15
    for pos, f in ((7, 0.9), (-12, 0.31), (1000, 0.125)):
        assert abs(np.exp(1j * around.angle(pos, f)) - np.exp(1j * pos * f)) < 1e-12
    # a far position: 2^31 - 1 radians, where binary64's own product is still exact
    far = 2 ** 31 - 1
    assert abs(around.angle(far, 1.0) - float(np.angle(np.exp(1j * np.longdouble(far))))) < 1e-6


@pytest.mark.parametrize("adjacent", [False, True])
def test_rope_is_a_rotation_and_its_inverse_undoes_it(adjacent):
    rng = np.random.default_rng(1)
    x = rng.standard_normal((2, 3, 2, 12))
    pos = rng.integers(-50, 50, (2, 2, 3))
    f, axis = [1.0, 0.3, 0.01, 0.5], [0, 1, 1, 0]
    y = around.rope(x, pos, f, axis, adjacent)
    assert np.allclose(y[..., 8:], x[..., 8:], atol=0)
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose(around.rope(y, pos, f, axis, adjacent, inverse=True), x, atol=1e-14)
    # pairs as complex numbers
    a, b = (x[..., 0:8:2], x[..., 1:8:2]) if adjacent else (x[..., :4], x[..., 4:8])
    turn = np.stack([pos[axis[i]] * f[i] for i in range(4)], -1)[:, :, None, :]
    z = (a + 1j * b) * np.exp(1j * turn)
    got = (y[..., 0:8:2], y[..., 1:8:2]) if adjacent else (y[..., :4], y[..., 4:8])
    assert np.allclose(z.real, got[0], atol=1e-12) and np.allclose(z.imag, got[1], atol=1e-12)


def test_scores_of_rotated_heads_depend_on_the_distance_alone():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 1, 16))
    f, axis = list(10000.0 ** (-np.arange(8) / 8)), [0] * 8
    at = lambda p, x: around.rope(x, [[[p]]], f, axis)  # noqa: E731
    near = (at(7, q) * at(3, k)).sum()
    assert abs(near - (at(100007, q) * at(100003, k)).sum()) < 1e-9


def test_rope_spec_turns_and_sections():
    r = va.verify_attn_rope_spec(16, base=100.0, sections=[2, 3, 3], layout="dealt")
    assert r.axis == [0, 1, 2, 0, 1, 2, 1, 2] and r.num_axes == 3 and r.num_pairs == 8
    assert va.verify_attn_rope_spec(16, sections=[2, 3, 3]).axis == [0, 0, 1, 1, 1, 2, 2, 2]
    freq = [1.0, 0.5, 1e-3, -0.25, 3.0e-30, 0.0, 1048576.0, 7.5]
    r = va.verify_attn_rope_spec(16, inv_freq=freq)
    for i, f in enumerate(freq):
        num, den = f.as_integer_ratio()
        exact = num * around._TURN * 2 ** 64 // den / 2 ** around._BITS
        got = r._struct.turn[i]
        want = num * around._TURN // (den << (around._BITS - 64)) % 2 ** 64
        # inv_freq / 2 pi as a multiple of 2^-64: 1/(2 pi) is cut at 2^-67 of its own size
        err = (got - want + 2 ** 63) % 2 ** 64 - 2 ** 63
        assert abs(err) <= 1 + abs(exact) * 2.0 ** -64, (f, err)


@pytest.mark.parametrize("kw", [
    dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=258), dict(rotary_dim=8, inv_freq=[1.0] * 3),
    dict(rotary_dim=8, sections=[1, 2]), dict(rotary_dim=8, sections=[1, 1, 1, 1, 0]),
    dict(rotary_dim=8, sections=[5, -1]), dict(rotary_dim=8, layout="mixed"), dict(rotary_dim=8, pairing="thirds"),
])
def test_rope_spec_refusals(kw):
    with pytest.raises(ValueError):
        va.verify_attn_rope_spec(**kw)


@pytest.mark.parametrize("freq,scale", [([1.0, float("nan")], 1.0), ([1.0, float("inf")], 1.0), ([2.0 ** 21, 1.0], 1.0),
                                        ([1.0, 1.0], float("inf"))])
def test_rope_spec_refuses_numbers_out_of_range(freq, scale):
    with pytest.raises(va.VerifyAttnError):
        va.verify_attn_rope_spec(4, inv_freq=freq, scale=scale)


def _heads(data=4096, seq=64, token=64, head=16, n=2):
    return va._Heads(data, seq, token, head, n)


def _rope(**change):
    """Status of a verify_attn_rope call whose pointers are never followed: it is refused."""
    a = dict(rope=va.verify_attn_rope_spec(16)._struct, type=0, B=2, T=3, D=16, q=_heads(), q_out=_heads(8192), k=None,
             k_out=None, pos=va._Positions(4096, 0, 1, 1))
    a.update(change)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return va.library().verify_attn_rope(ref(a["rope"]), ref(a["pos"]), a["type"], a["B"], a["T"], a["D"], ref(a["q"]),
                                         ref(a["q_out"]), ref(a["k"]), ref(a["k_out"]), 0, None)


@pytest.mark.parametrize("change,status", [
    (dict(rope=None), -1), (dict(pos=None), -1), (dict(q=None), -1), (dict(q_out=None), -1), (dict(type=3), -2),
    (dict(type=-1), -2), (dict(B=-1), -1), (dict(T=-1), -1), (dict(D=14), -1), (dict(D=1026), -1),
    (dict(k=_heads()), -1), (dict(k_out=_heads()), -1), (dict(q=_heads(n=3)), -1), (dict(q=_heads(n=0), q_out=_heads(n=0)), -1),
    (dict(q=_heads(data=0)), -1), (dict(q=_heads(data=4097)), -1), (dict(q=_heads(data=4098), type=2), -1),
    (dict(pos=va._Positions(0, 0, 1, 1)), -1), (dict(pos=va._Positions(4098, 0, 1, 1)), -1),
    (dict(q_out=_heads(8192, head=8)), -1),     # heads of the output overlap
    (dict(q_out=_heads(8192, seq=0)), -1),      # sequences of the output lie on one another
    (dict(q_out=_heads(8192, token=24)), -1),   # tokens overlap the heads before them
    (dict(q_out=_heads(4096, token=32, seq=96)), -1),   # in place with other strides
    (dict(q=_heads(token=-64)), -1),
    (dict(B=2 ** 20, T=2 ** 20), -1), (dict(B=2 ** 14, T=2 ** 14, q=_heads(4098), q_out=_heads(8194)), -1),  # too many
    (dict(B=0), 0), (dict(T=0), 0),             # nothing to do
])
def test_rope_refusals(change, status):
    assert _rope(**change) == status


def test_rope_refuses_a_description_that_was_never_filled():
    assert _rope(rope=va._Rope()) == -1
    bad = va.verify_attn_rope_spec(16)._struct
    bad.axis[3] = 1  # of one axis
    assert _rope(rope=bad) == -1


def _append(**change):
    a = dict(rope=va.verify_attn_rope_spec(change.pop("rotary", 32))._struct, pos=None, B=1, T=2, D=64, q=_heads(4096, 256, 128, 64), q_out=8192,
             k=_heads(4096, 256, 128, 64), v=_heads(4096, 256, 128, 64), dtype=2, k_pages=4096, v_pages=4096, k_scale=4096,
             v_scale=4096, table=4096, stride=4, lens=4096, pages=8, flags=None)
    a.update(change)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return va.library().verify_attn_rope_append(
        ref(a["rope"]), ref(a["pos"]), a["B"], a["T"], a["D"], ref(a["q"]), a["q_out"], ref(a["k"]), ref(a["v"]),
        a["dtype"], a["k_pages"], a["v_pages"], a["k_scale"], a["v_scale"], a["table"], a["stride"], a["lens"], a["pages"],
        a["flags"], None)


@pytest.mark.parametrize("change,status", [
    (dict(rope=None), -1), (dict(q=None), -1), (dict(q_out=None), -1), (dict(k=None), -1), (dict(v=None), -1),
    (dict(k_pages=None), -1), (dict(v_pages=None), -1), (dict(k_scale=None), -1), (dict(v_scale=None), -1),
    (dict(table=None), -1), (dict(lens=None), -1), (dict(B=0), -1), (dict(T=0), -1), (dict(stride=0), -1),
    (dict(pages=-1), -1), (dict(D=96), -2), (dict(dtype=5), -2), (dict(dtype=-1), -2),
    (dict(rotary=128), -1),   # wider than the head
    (dict(q=_heads(8192, 512, 256, 64), q_out=8192), -1),   # in place where q does not lie as q_out does
    (dict(v=_heads(4096, 256, 128, 64, n=1)), -1), (dict(q=_heads(4096, 256, 128, 64, n=0)), -1),
    (dict(k=_heads(4104, 256, 128, 64)), -1), (dict(v=_heads(4096, 256, 132, 64)), -1), (dict(q_out=8200), -1),
    (dict(k_pages=4104), -1), (dict(table=4098), -1), (dict(flags=4098), -1), (dict(pos=va._Positions(0, 0, 0, 1)), -1),
])
def test_rope_append_refusals(change, status):
    assert _append(**change) == status


# ------------------------------------------------------------------ acceptance


def test_accept_probs_samples_the_target_whatever_the_proposal():
    """The first emitted or accepted token is distributed as p_0 for a model's and a point mass's
    proposals: over a grid of the given numbers the shares are p_0 to the grid's width."""
    p0 = np.array([0.5, 0.2, 0.2, 0.1, 0.0])
    q0 = np.array([0.1, 0.6, 0.1, 0.1, 0.1])
    n = 50
    grid = (np.arange(n) + 0.5) / n
    u, v = [g.reshape(-1).astype(np.float32) for g in np.meshgrid(grid, grid)]
    B = u.size
    p = np.tile(np.stack([p0, p0])[None], (B, 1, 1)).astype(np.float32)
    share = np.zeros(5)
    for d in range(5):  # the draft is d with probability q0[d]
        q = np.tile(q0[None, None], (B, 1, 1)).astype(np.float32)
        out, _ = around.accept_probs(p, np.full((B, 1), d), u[:, None], v, q)
        share += q0[d] * np.bincount(out[:, 0], minlength=5) / B
    assert np.abs(share - p0).max() < 2.0 / n
    out, acc = around.accept_probs(p, np.full((B, 1), 2), u[:, None], v)  # point mass on 2
    assert np.abs(np.bincount(out[:, 0], minlength=5) / B - p0).max() < 2.0 / n
    assert abs(acc.mean() - 0.2) < 1.0 / n


def test_accept_probs_decisions_by_hand():
    p = np.array([[[0.25, 0.75, 0, 0], [0, 0.5, 0, 0.5], [0, 0, 1, 0]]], np.float32)
    one = lambda d, ua, ue, **kw: [x.tolist() for x in around.accept_probs(p, [d], [ua], [ue], **kw)]  # noqa: E731
    assert one([1, 3], [0.7, 0.4], 0.3) == [[[1, 3, 2]], [2]]
    assert one([1, 3], [0.75, 0.4], 0.0) == [[[0, -1, -1]], [0]]           # u = p(d): rejected; the rest is 0
    assert one([1, 3], [0.7, 0.5], 0.99) == [[[1, 1, -1]], [1]]
    assert one([1, 9], [0.7, 0.0], 0.5) == [[[1, 3, -1]], [1]]             # no such token: nothing is taken away
    assert one([1, 3], [0.7, 0.4], 0.3, lens=[1]) == [[[1, 1, -1]], [1]]   # two drafts, one counts
    assert one([2, 3], [0.0, 0.4], 1.0, lens=[-4]) == [[[1, -1, -1]], [0]]
    q = np.array([[[0.25, 0.75, 0, 0], [0.5, 0.5, 0, 0]]], np.float32)
    assert one([1, 0], [0.99, 0.5], 0.2, q=q) == [[[1, 3, -1]], [1]]       # p - q leaves 3 alone
    same = np.array([[[0.25, 0.75, 0, 0], [0, 0.5, 0, 0.5]]], np.float32)
    assert one([2, 0], [0.5, 0.5], 0.9, q=same) == [[[1, -1, -1]], [0]]    # p = q: p itself
    dead = np.zeros((1, 2, 3), np.float32)
    assert around.accept_probs(dead, [[1]], [[0.5]], [0.5])[0].tolist() == [[-1, -1]]


def _accept(**change):
    a = dict(p=va._Rows(4096, 8, 4), q=None, type=2, drafts=4096, lens=None, ua=4096, ue=4096, B=1, T=1, V=4, out=4096, n=4096)
    a.update(change)
    ref = lambda x: None if x is None else ctypes.byref(x)  # noqa: E731
    return va.library().verify_attn_accept_probs(ref(a["p"]), ref(a["q"]), a["type"], a["drafts"], a["lens"], a["ua"],
                                                 a["ue"], a["B"], a["T"], a["V"], a["out"], a["n"], None)


@pytest.mark.parametrize("change,status", [
    (dict(p=None), -1), (dict(p=va._Rows(0, 8, 4)), -1), (dict(p=va._Rows(4098, 8, 4)), -1), (dict(p=va._Rows(4096, -8, 4)), -1),
    (dict(q=va._Rows(4098, 4, 4)), -1), (dict(q=va._Rows(4096, 4, -4)), -1), (dict(type=3), -2), (dict(drafts=None), -1),
    (dict(ua=None), -1), (dict(ue=None), -1), (dict(out=None), -1), (dict(n=None), -1), (dict(B=0), -1), (dict(B=65536), -1),
    (dict(T=-1), -1), (dict(T=65536), -1), (dict(V=0), -1), (dict(V=2 ** 30 + 1), -1), (dict(drafts=4097), -1), (dict(lens=4098), -1), (dict(out=4099), -1),
])
def test_accept_probs_refusals(change, status):
    assert _accept(**change) == status


# ------------------------------------------------------------------ pages


def random_step(rng, pool, grow=40):
    """One call on `pool` as (name, arguments), some of them ones that are refused."""
    B, stride = pool.table.shape
    op = rng.choice(["resize", "resize", "resize", "fork", "fork", "compact"])
    if op == "resize":
        new = pool.lens + rng.integers(-grow, grow + 1, B)
        new = np.where(rng.random(B) < 0.1, 0, np.maximum(new, 0))
        new = np.minimum(new, around.PAGE * stride)
        new = np.where(rng.random(B) < 0.1, -1, new)
        new = np.where(rng.random(B) < 0.02, around.PAGE * stride + 1, new)
        return "resize", (new.astype(np.int32),)
    if op == "compact":
        return "compact", ()
    F = int(rng.integers(1, 5))
    parents, children = rng.integers(0, B, F), rng.integers(0, B, F)
    if rng.random() < 0.1:
        children[0] = B + 3
    if rng.random() < 0.1:
        parents[0] = -1
    empty = np.flatnonzero(pool.lens == 0)
    if len(empty):
        children[-1] = rng.choice(empty)
    lens = None
    if rng.random() < 0.4:
        lens = np.array([rng.integers(0, max(1, pool.lens[p] + 1)) if 0 <= p < B else 3 for p in parents], np.int32)
        if rng.random() < 0.1:
            lens[0] = 10 ** 6
    return "fork", (parents.astype(np.int32), children.astype(np.int32), lens, bool(rng.random() < 0.6))


@pytest.mark.parametrize("seed", range(8))
def test_pages_oracle_keeps_its_books_and_every_sequences_tokens(seed):
    """Each cell of the cache holds the token it was written for: writing through the table after
    each call, no sequence ever reads another one's tokens."""
    rng = np.random.default_rng(seed)
    P, B, stride = 60, 7, 12
    pool = around.Pages(P, B, stride, [np.zeros((P, around.PAGE), np.int64)])
    tokens = [[] for _ in range(B)]
    fresh = itertools_count()
    for _ in range(120):
        name, args = random_step(rng, pool)
        before = pool.lens.copy()
        getattr(pool, name)(*args)
        pool.check()
        if name == "fork":
            parents, children, lens, _ = args
            for f in range(len(parents)):
                c = children[f]
                if 0 <= c < B and before[c] == 0 and pool.lens[c] > 0 and not tokens[c]:
                    tokens[c] = tokens[parents[f]][:int(pool.lens[c])]
        for b in range(B):
            tokens[b] = tokens[b][:int(pool.lens[b])]
            while len(tokens[b]) < pool.lens[b]:
                at = len(tokens[b])
                tokens[b].append(next(fresh))
                pool.buffers[0][pool.table[b, at // 16], at % 16] = tokens[b][-1]
            got = [pool.buffers[0][pool.table[b, i // 16], i % 16] for i in range(int(pool.lens[b]))]
            assert got == tokens[b]


def itertools_count():
    n = 0
    while True:
        n += 1
        yield n


def _pool(**change):
    a = dict(block_table=4096, seq_lens=4096, ref_count=4096, free_list=4096, num_free=4096, flags=None,
             block_table_stride=4, num_seqs=2, num_pages=8, num_buffers=1, page=(4096, 64), workspace=4096)
    a.update(change)
    page = a.pop("page")
    array = (va._PageBuffer * 1)(va._PageBuffer(*page))
    s = va._PagePool(*[a[n] for n in ("block_table", "seq_lens", "ref_count", "free_list", "num_free", "flags",
                                      "block_table_stride", "num_seqs", "num_pages", "num_buffers")], array, a["workspace"])
    s._keep = array
    return s


@pytest.mark.parametrize("change", [
    dict(block_table=None), dict(seq_lens=None), dict(ref_count=None), dict(free_list=None), dict(num_free=None),
    dict(workspace=None), dict(workspace=4104), dict(block_table=4098), dict(flags=4097), dict(block_table_stride=0),
    dict(num_seqs=0), dict(num_seqs=8193), dict(num_pages=0), dict(num_pages=2 ** 22 + 1), dict(block_table_stride=2 ** 30), dict(num_seqs=4096, block_table_stride=2 ** 18 + 1),
    dict(num_buffers=-1), dict(page=(0, 64)), dict(page=(4104, 64)), dict(page=(4096, 24)), dict(page=(4096, 0)),
])
def test_page_pool_refusals(change):
    lib, s = va.library(), _pool(**change)
    ref = ctypes.byref(s)
    assert lib.verify_attn_pages_resize(ref, 4096, None) == -1
    assert lib.verify_attn_pages_fork(ref, 4096, 4096, None, 1, 1, None) == -1
    assert lib.verify_attn_pages_compact(ref, None) == -1


def test_page_call_refusals():
    lib, s = va.library(), _pool()
    ref = ctypes.byref(s)
    assert lib.verify_attn_pages_resize(ref, None, None) == -1
    assert lib.verify_attn_pages_resize(ref, 4098, None) == -1
    assert lib.verify_attn_pages_resize(None, 4096, None) == -1
    for args in ((None, 4096, None, 1), (4096, None, None, 1), (4098, 4096, None, 1), (4096, 4096, 4098, 1),
                 (4096, 4096, None, -1), (4096, 4096, None, 8193)):
        assert lib.verify_attn_pages_fork(ref, *args, 1, None) == -1, args
    assert lib.verify_attn_pages_fork(ref, None, None, None, 0, 1, None) == 0  # no forks: nothing is launched


def test_page_workspace_size():
    lib = va.library()
    assert lib.verify_attn_pages_workspace_bytes(0, 8) == 0 and lib.verify_attn_pages_workspace_bytes(8, 0) == 0
    assert lib.verify_attn_pages_workspace_bytes(8193, 8) == 0
    small, large = lib.verify_attn_pages_workspace_bytes(4, 100), lib.verify_attn_pages_workspace_bytes(4, 200)
    assert 0 < small < large and small % 16 == 0


# ------------------------------------------------------------------ the binding's own checks


def test_binding_refuses_tensors_that_are_not_on_a_gpu():
    torch = pytest.importorskip("torch")
    rope = va.verify_attn_rope_spec(16)
    x = torch.zeros(1, 2, 3, 16)
    with pytest.raises(ValueError):
        va.verify_attn_rope(rope, torch.zeros(1, 1, 2, dtype=torch.int32), x)
    with pytest.raises(ValueError):
        va.verify_attn_rope(rope, torch.zeros(1, 1, 2, dtype=torch.int32), x.double())
    with pytest.raises(ValueError):
        va.verify_attn_accept_probs(torch.zeros(1, 2, 4), torch.zeros(1, 1, dtype=torch.int32), torch.zeros(1, 1), torch.zeros(1))
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        va.PagePool(i(2, 3), i(2), i(8), i(8), i(1), [torch.zeros(8, 4)])
