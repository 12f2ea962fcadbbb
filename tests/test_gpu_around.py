"""GPU parity of the operators around the verify step against their plain definitions: rotary
positions (alone and with the append), acceptance from given probabilities, the page pool, and a run
of them together with verify attention.

Tolerances.  A rotated element is s (a c - b d) in binary32.  Its cosine and sine are off by at most
4 x 2^-24 (the remainder of the angle is rounded once, 2^-24 of at most pi / 4; sincospif is within
two ulps of a value of at most 1; the scale is one more rounding), and the two products and the sum
add three roundings of at most 2^-24 each of a term: 7 x 2^-24 s (|a| + |b|) bounds it.  A 16-bit
output adds half a step, eps / 2 of the value.  Codes are decided in binary32 on both sides and are
equal.  Everything else here is whole numbers and copies: equal."""
import ctypes

import numpy as np
import pytest

import oracle
from oracle import around

from parity import compare
from test_around_oracle import random_step

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    from speculative_decoding_verify_causal_gb300 import build
    build.build()


@pytest.fixture(scope="module")
def va():
    import speculative_decoding_verify_causal_gb300 as va
    return va


def cuda(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t if dtype is None else t.to(dtype)).cuda()


def normal(seed, *shape, dtype=torch.float32):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


# ------------------------------------------------------------------ rotary


def rope_bound(x, P, adjacent, scale, dtype, ref):
    """Per element: 7 x 2^-24 scale (|a| + |b|), 0 for the elements that are copied, and half a step."""
    x = np.abs(x.astype(np.float64))
    size = np.zeros_like(x)
    if adjacent:
        pair = x[..., 0:2 * P:2] + x[..., 1:2 * P:2]
        size[..., 0:2 * P:2] = size[..., 1:2 * P:2] = pair
    else:
        pair = x[..., :P] + x[..., P:2 * P]
        size[..., :P] = size[..., P:2 * P] = pair
    half = 0.0 if dtype == torch.float32 else torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 0.0  # half a step of fp16's subnormals
    return 7 * U32 * abs(scale) * size * (1 + half) + half * np.abs(ref) + tiny


ROPE_CASES = [  # B, T, Hq, Hk, D, rotary_dim, sections, layout, pairing
    (1, 1, 1, 0, 2, 2, None, "blocked", "half"),
    (1, 1, 24, 4, 256, 256, [32, 48, 48], "dealt", "half"),
    (2, 7, 4, 1, 64, 64, None, "blocked", "half"),
    (1, 5, 3, 3, 80, 80, [20, 20], "blocked", "adjacent"),
    (3, 11, 2, 1, 72, 36, [6, 6, 6], "dealt", "half"),
    (2, 3, 5, 2, 96, 30, [5, 5, 5], "blocked", "adjacent"),
    (1, 17, 7, 7, 65, 34, [9, 0, 8], "dealt", "half"),
    (2, 33, 2, 2, 128, 128, [16, 24, 24], "blocked", "half"),
    (1, 2, 3, 1, 515, 256, [128], "blocked", "adjacent"),
    (1, 130, 2, 1, 24, 24, [3, 3, 3, 3], "dealt", "half"),
    (2, 9, 19, 3, 72, 72, [18, 18], "blocked", "half"),       # 8-byte vectors of 16-bit types
    (1, 9, 19, 3, 88, 40, None, "blocked", "half"),           # an odd number of vectors past the pairs
    (1, 9, 19, 3, 90, 36, None, "blocked", "adjacent"),
]


@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "-".join(map(str, c[:6])))
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("inverse", [False, True])
def test_rope(va, case, dtype, inverse):
    B, T, Hq, Hk, D, R, sections, layout, pairing = case
    spec = va.verify_attn_rope_spec(R, sections=sections, layout=layout, pairing=pairing, scale=1.25)
    freq = 1.0e6 ** (-np.arange(R // 2, dtype=np.float64) / (R // 2))
    rng = np.random.default_rng(B * 1000 + T * 10 + D)
    pos = rng.integers(-5, 300000, (spec.num_axes, B, T)).astype(np.int32)
    pos[0, 0, 0] = 0
    pos[-1, -1, -1] = 2 ** 31 - 1 if T > 1 else -(2 ** 31)
    q = normal(1, B, T, Hq, D, dtype=dtype)
    k = normal(2, B, T, Hk, D, dtype=dtype) if Hk else None
    before = q.clone()
    got_q, got_k = va.verify_attn_rope(spec, cuda(pos), q, k, inverse=inverse)
    torch.cuda.synchronize()
    assert torch.equal(q, before) and got_q.is_contiguous()
    for x, y in ((q, got_q), (k, got_k)):
        if x is None:
            assert y is None
            continue
        xs = x.double().cpu().numpy()
        ref = around.rope(xs, pos.tolist(), freq, spec.axis, pairing == "adjacent", 1.25, inverse)
        err = np.abs(y.double().cpu().numpy() - ref)
        bound = rope_bound(xs, R // 2, pairing == "adjacent", 1.25, dtype, ref)
        assert (err <= bound).all(), (err - bound).max()
        assert torch.equal(y[..., R:], x[..., R:])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("D,R", [(128, 128), (80, 40), (66, 34)])
def test_rope_takes_tensors_as_they_lie(va, dtype, D, R):
    """Slices of a fused projection, [B, H, T, D], a padded head, an odd offset, positions shared over the batch, in
    place, and outputs into slices: all the same values as the contiguous call."""
    B, T, Hq, Hk = 2, 9, 4, 2
    spec = va.verify_attn_rope_spec(R, sections=[R // 2 - 3, 3])
    pos = cuda(np.random.default_rng(3).integers(0, 5000, (2, 1, T)).astype(np.int32)).expand(2, B, T)
    q, k = normal(3, B, T, Hq, D, dtype=dtype), normal(4, B, T, Hk, D, dtype=dtype)
    want_q, want_k = va.verify_attn_rope(spec, pos.contiguous(), q, k)

    def same(a, b):
        got = va.verify_attn_rope(spec, pos, a, b)
        assert torch.equal(got[0], want_q) and torch.equal(got[1], want_k)

    fused = torch.zeros(B, T, Hq + 2 * Hk, D, dtype=dtype, device="cuda")
    fused[:, :, :Hq], fused[:, :, Hq:Hq + Hk] = q, k
    same(fused[:, :, :Hq], fused[:, :, Hq:Hq + Hk])
    same(q.transpose(1, 2).contiguous().transpose(1, 2), k.transpose(0, 1).contiguous().transpose(0, 1))
    wide = torch.zeros(B, T, Hq, D + 5, dtype=dtype, device="cuda")
    wide[..., 3:3 + D] = q
    same(wide[..., 3:3 + D], k)
    flat = torch.zeros(q.numel() + 1, dtype=dtype, device="cuda")
    flat[1:] = q.reshape(-1)
    same(flat[1:].view_as(q), k)
    # in place, in the projection itself: v and the gaps stay
    work = fused.clone()
    va.verify_attn_rope(spec, pos, work[:, :, :Hq], work[:, :, Hq:Hq + Hk], q_out=work[:, :, :Hq],
                        k_out=work[:, :, Hq:Hq + Hk])
    assert torch.equal(work[:, :, :Hq], want_q) and torch.equal(work[:, :, Hq:Hq + Hk], want_k)
    assert torch.equal(work[:, :, Hq + Hk:], fused[:, :, Hq + Hk:])
    out = torch.full_like(wide, 7.0)
    va.verify_attn_rope(spec, pos, q, q_out=out[..., 3:3 + D])
    assert torch.equal(out[..., 3:3 + D], want_q)
    assert (out[..., :3] == 7).all() and (out[..., 3 + D:] == 7).all()


def test_rope_gradient_by_differences_and_by_the_formula(va):
    """The rotation is linear, so <w, rope(x + h e) - rope(x)> / h is the gradient's component for any h: it is
    compared with the inverse call on w.  h = 1; both sides are sums of at most two terms of size about 1 with 7 x 2^-24
    each, and the difference of two outputs of size up to 4 adds 2 x 4 x 7 x 2^-24: 100 x 2^-24 covers them."""
    spec = va.verify_attn_rope_spec(24, sections=[5, 7], layout="dealt", pairing="adjacent", scale=0.75)
    B, T, H, D = 2, 3, 2, 30
    pos = cuda(np.random.default_rng(5).integers(0, 90000, (2, B, T)).astype(np.int32))
    x, w = normal(6, B, T, H, D), normal(7, B, T, H, D)
    grad, _ = va.verify_attn_rope(spec, pos, w, inverse=True)
    y, _ = va.verify_attn_rope(spec, pos, x)
    rng = np.random.default_rng(8)
    for _ in range(40):
        at = tuple(int(rng.integers(0, n)) for n in x.shape)
        moved = x.clone()
        moved[at] += 1.0
        z, _ = va.verify_attn_rope(spec, pos, moved)
        slope = float((w.double() * (z.double() - y.double())).sum())
        assert abs(slope - float(grad[at])) <= 100 * U32 * (1 + abs(slope)), at
    # <w, R x> = <R^T w, x> over everything
    left, right = float((w.double() * y.double()).sum()), float((grad.double() * x.double()).sum())
    assert abs(left - right) <= 14 * U32 * 0.75 * 4 * x.numel()


def test_rope_nothing_to_do_and_special_values(va):
    spec = va.verify_attn_rope_spec(4)
    empty = torch.zeros(0, 3, 2, 4, device="cuda")
    assert va.verify_attn_rope(spec, torch.zeros(1, 0, 3, dtype=torch.int32, device="cuda"), empty)[0].shape == (0, 3, 2, 4)
    assert va.verify_attn_rope(spec, torch.zeros(1, 2, 0, dtype=torch.int32, device="cuda"),
                               torch.zeros(2, 0, 2, 4, device="cuda"))[0].numel() == 0
    x = torch.tensor([float("inf"), 1.0, float("nan"), -2.0, float("-inf")], device="cuda").view(1, 1, 1, 5)
    y, _ = va.verify_attn_rope(spec, torch.zeros(1, 1, 1, dtype=torch.int32, device="cuda"), x)
    y = y.reshape(-1)
    assert y[1] == 1 and y[3] == -2 and y[4] == float("-inf")  # a pair's NaN and the copied element stay where they are
    with pytest.raises(ValueError):
        va.verify_attn_rope(spec, torch.zeros(2, 1, 1, dtype=torch.int32, device="cuda"), x)
    with pytest.raises(ValueError):
        va.verify_attn_rope(spec, torch.zeros(1, 1, 1, dtype=torch.int64, device="cuda"), x)
    with pytest.raises(va.VerifyAttnError):  # an output that lies on itself
        va.verify_attn_rope(spec, torch.zeros(1, 1, 2, dtype=torch.int32, device="cuda"), torch.zeros(1, 2, 1, 4, device="cuda"),
                            q_out=torch.zeros(1, 1, 1, 4, device="cuda").expand(1, 2, 1, 4))


def test_rope_strides_past_32_bits(va):
    """Two sequences more than 2^31 elements apart in one 4.3 GB tensor."""
    far = 2 ** 31 + 64
    base = torch.empty(far + 4096, dtype=torch.bfloat16, device="cuda")
    x = base.as_strided((2, 3, 2, 64), (far, 128, 64, 1))
    x.copy_(normal(9, 2, 3, 2, 64, dtype=torch.bfloat16))
    spec = va.verify_attn_rope_spec(64)
    pos = cuda(np.arange(6, dtype=np.int32).reshape(1, 2, 3) * 1000)
    want, _ = va.verify_attn_rope(spec, pos, x.contiguous())
    va.verify_attn_rope(spec, pos, x, q_out=x)
    assert torch.equal(x, want)


# ------------------------------------------------------------------ rotary and append


def cache_case(seed, lens, T, Hkv, D, kv_dtype, extra_pages=3):
    """(page array, scale array or None, block table, lens, pages used) of a cache with arbitrary contents."""
    rng = np.random.default_rng(seed)
    need = [max(1, -(-L // 16)) for L in lens]
    P = sum(need) + extra_pages
    order = rng.permutation(P).astype(np.int32)
    bt, at = np.zeros((len(lens), max(need)), np.int32), 0
    for b, n in enumerate(need):
        bt[b, :n] = order[at:at + n]
        at += n
    width = {"bf16": D, "fp8_e4m3": D, "int8": D, "int4": D // 2, "int2": D // 4}[kv_dtype]
    if kv_dtype == "bf16":
        pages = rng.integers(0, 0x3F80, (P, 16, Hkv, width)).astype(np.uint16)
    else:
        pages = rng.integers(0, 120, (P, 16, Hkv, width)).astype(np.int8 if kv_dtype == "int8" else np.uint8)
    scale = None if kv_dtype == "bf16" else rng.random((P, 16, Hkv)).astype(np.float32)
    return pages, scale, bt, np.array(lens, np.int32), P


def bits16(t):
    return t.contiguous().view(torch.int16).cpu().numpy().view(np.uint16)


def run_append(va, spec, pos, q, k, v, pages, scale, bt, lens, kv_dtype, num_pages=0, **kw):
    dev = lambda a: cuda(a.view(np.int16) if a.dtype == np.uint16 else a)  # noqa: E731
    kp, vp = dev(pages), dev(pages)
    ks, vs = (None, None) if scale is None else (cuda(scale), cuda(scale))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    if kv_dtype == "bf16":
        kp, vp = kp.view(torch.bfloat16), vp.view(torch.bfloat16)
    out = va.verify_attn_rope_append(spec, pos, q, k, v, kp, vp, ks, vs, cuda(bt), cuda(lens), kv_dtype,
                                     num_pages=num_pages, flags=flags, **kw)
    torch.cuda.synchronize()
    raw = [(bits16(x) if kv_dtype == "bf16" else x.cpu().numpy()) for x in (kp, vp)]
    return out, raw, [None if x is None else x.cpu().numpy() for x in (ks, vs)], int(flags.item())


def expected_cache(rows, pages, scale, bt, lens, kv_dtype, num_pages):
    """The append's rule in binary32 on rows [B, T, Hkv, D] (float32), through torch's own casts."""
    pages, scale = pages.copy(), None if scale is None else scale.copy()
    B, T = rows.shape[:2]
    for b in range(B):
        for t in range(T):
            at = int(lens[b]) - T + t
            if at < 0 or at // 16 >= bt.shape[1] or not 0 <= bt[b, at // 16] < num_pages:
                continue
            page, slot = bt[b, at // 16], at % 16
            x = rows[b, t]
            if kv_dtype == "bf16":
                pages[page, slot] = torch.from_numpy(x).to(torch.bfloat16).view(torch.int16).numpy().view(np.uint16)
                continue
            qmax = np.float32({"fp8_e4m3": 448, "int8": 127, "int4": 7, "int2": 1}[kv_dtype])
            a = np.abs(x).max(-1)
            s = np.where(a > 0, a / qmax, np.float32(1)).astype(np.float32)
            y = (x / s[:, None]).astype(np.float32)
            if kv_dtype == "fp8_e4m3":
                codes = torch.from_numpy(np.clip(y, -448, 448)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
            else:
                codes = np.clip(np.rint(y), -qmax, qmax).astype(np.int8)
                if kv_dtype != "int8":
                    from speculative_decoding_verify_causal_gb300 import workloads as wl
                    codes = wl.pack_codes(codes, wl.KV_ELEM_BITS[kv_dtype])
            pages[page, slot], scale[page, slot] = codes, s
    return pages, scale


APPEND_CASES = [  # lens, T, Hq, Hkv, D, rotary_dim, pairing
    ([1], 1, 1, 1, 64, 64, "half"),
    ([20, 5, 33], 5, 4, 1, 64, 16, "adjacent"),
    ([25016], 16, 24, 4, 256, 64, "half"),
    ([100, 16], 16, 6, 2, 128, 128, "half"),
    ([70, 300, 16, 17], 7, 8, 8, 256, 256, "adjacent"),
    ([40] * 80, 5, 32, 8, 128, 96, "half"),              # three passes a warp
    ([400, 500, 600], 200, 24, 4, 256, 34, "adjacent"),  # four, and pairs that end inside a lane
    ([400, 500, 600], 200, 5, 2, 256, 22, "half"),       # two, and halves that start inside a lane
    ([33, 40], 9, 3, 1, 64, 6, "half"),
    ([500] * 9, 50, 33, 7, 64, 62, "half"),
]


@pytest.mark.parametrize("case", APPEND_CASES, ids=lambda c: f"B{len(c[0])}-T{c[1]}-{c[2]}-{c[3]}-{c[4]}-{c[5]}{c[6][0]}")
@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3", "int8", "int4", "int2"])
def test_rope_append(va, case, kv_dtype):
    """q and the cache are what the rotary alone gives in fp32 and the append's rule makes of it, bit for bit."""
    lens, T, Hq, Hkv, D, R, pairing = case
    B = len(lens)
    pages, scale, bt, lens, P = cache_case(T + D, lens, T, Hkv, D, kv_dtype)
    spec = va.verify_attn_rope_spec(R, sections=[R // 2 - 2, 1, 1] if R > 8 else None, pairing=pairing)
    pos = cuda(np.random.default_rng(1).integers(0, 250000, (spec.num_axes, B, T)).astype(np.int32))
    qkv = normal(11, B, T, Hq + 2 * Hkv, D, dtype=torch.bfloat16)
    q, k, v = qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]
    out, (kp, vp), (ks, vs), flags = run_append(va, spec, pos, q, k, v, pages, scale, bt, lens, kv_dtype)
    assert flags == 0
    turned_q, turned_k = va.verify_attn_rope(spec, pos, q.float(), k.float())
    assert torch.equal(out, turned_q.to(torch.bfloat16))
    for rows, got, got_scale in ((turned_k, kp, ks), (v.float(), vp, vs)):
        want, want_scale = expected_cache(rows.cpu().numpy(), pages, scale, bt, lens, kv_dtype, P)
        assert np.array_equal(got, want)
        if scale is not None:
            assert np.array_equal(got_scale.view(np.uint32), want_scale.view(np.uint32))


@pytest.mark.parametrize("kv_dtype", ["bf16", "fp8_e4m3", "int8", "int4", "int2"])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_rope_append_at_position_zero_is_the_append(va, kv_dtype, D):
    """Bit for bit, 2,000 rows of every size: ties, tiny and subnormal rows, huge ones, zeros, and rows of one value among
    them, where a quotient that is not rounded as a division would show."""
    B, T, Hkv = 3, 334, 2
    pages, scale, bt, lens, P = cache_case(5, [400, 340, 334], T, Hkv, D, kv_dtype)
    rng = np.random.default_rng(D)

    def rows(seed):
        x = normal(seed, B, T, Hkv, D).cpu().numpy().astype(np.float64)
        x *= 2.0 ** rng.integers(-120, 100, (B, T, Hkv, 1))
        x[0, 0], x[0, 1, 0], x[0, 2, 1] = 0.0, 2.5, 1e-40
        x[0, 3] = np.linspace(-1, 1, D)
        x[0, 4] = np.arange(D) - D // 2
        x[0, 5, 0] = 3e38 * np.sign(x[0, 5, 0])
        x[0, 6] = np.where(np.arange(D) % 7 == 0, 1.0, 2.0 ** -rng.integers(0, 30, D))
        x[1, :200] = rng.integers(-448, 449, (200, Hkv, D)) / 2  # halves of codes: ties where the scale is a power of two
        x[1, :200, :, 0] = 2.0 ** rng.integers(6, 9, (200, Hkv)) * rng.choice([1.75, 1.984375, 1.0])
        return torch.from_numpy(np.clip(x, -3e38, 3e38).astype(np.float32)).to(torch.bfloat16).cuda()

    k, v = rows(12), rows(13)
    spec = va.verify_attn_rope_spec(D)
    zero = torch.zeros(1, B, T, dtype=torch.int32, device="cuda")
    out, (kp, vp), (ks, vs), _ = run_append(va, spec, zero, None, k, v, pages, scale, bt, lens, kv_dtype)
    assert out is None
    rk, rv, rks, rvs, _ = oracle.kv_append(bits16(k), bits16(v), pages, pages, scale, scale, bt, lens, kv_dtype)
    assert np.array_equal(kp, rk) and np.array_equal(vp, rv)
    if scale is not None:
        assert np.array_equal(ks, rks) and np.array_equal(vs, rvs)


def test_rope_append_takes_the_place_in_the_sequence_without_positions(va):
    B, T, Hq, Hkv, D = 2, 6, 4, 2, 64
    pages, scale, bt, lens, P = cache_case(6, [30, 6], T, Hkv, D, "int8")
    q, k, v = (normal(14 + i, B, T, h, D, dtype=torch.bfloat16) for i, h in enumerate((Hq, Hkv, Hkv)))
    spec = va.verify_attn_rope_spec(D, sections=[20, 6, 6])
    place = (lens[:, None] - T + np.arange(T)).astype(np.int32)
    a = run_append(va, spec, None, q, k, v, pages, scale, bt, lens, "int8")
    b = run_append(va, spec, cuda(np.stack([place] * 3)), q, k, v, pages, scale, bt, lens, "int8")
    assert torch.equal(a[0], b[0]) and all(np.array_equal(x, y) for x, y in zip(a[1] + a[2], b[1] + b[2]))
    work = q.clone()  # q in place
    got, *_ = run_append(va, spec, None, work, k, v, pages, scale, bt, lens, "int8", q_out=work)
    assert got is work and torch.equal(work, a[0])


def test_rope_append_skips_and_flags_rows_without_a_page(va):
    """A padded slot (length 0), a length below T, a block past the table's row and a page outside the pool: those rows
    are left out, q is rotated for all."""
    T, Hq, Hkv, D = 4, 2, 1, 64
    pages, scale, bt, lens, P = cache_case(7, [40, 40, 40, 40, 40], T, Hkv, D, "int8", extra_pages=8)
    lens[1], lens[2] = 0, 2
    lens[3] = bt.shape[1] * 16 + 2           # two of its rows in the table, two past it
    small = P - 4
    used = set(bt.reshape(-1).tolist())
    spare = [p for p in range(small, P) if p not in used]
    bt[4, (lens[4] - 1) // 16] = spare[0] if spare else P - 1  # allocated, but not in a pool of `small` pages
    q, k, v = (normal(20 + i, 5, T, h, D, dtype=torch.bfloat16) for i, h in enumerate((Hq, Hkv, Hkv)))
    spec = va.verify_attn_rope_spec(D)
    pos = cuda(np.arange(20, dtype=np.int32).reshape(1, 5, T))
    out, (kp, vp), (ks, vs), flags = run_append(va, spec, pos, q, k, v, pages, scale, bt, lens, "int8", num_pages=small)
    assert flags == 1
    tq, tk = va.verify_attn_rope(spec, pos, q.float(), k.float())
    assert torch.equal(out, tq.to(torch.bfloat16))
    for rows, got, got_scale in ((tk, kp, ks), (v.float(), vp, vs)):
        want, want_scale = expected_cache(rows.cpu().numpy(), pages, scale, bt, lens, "int8", small)
        assert np.array_equal(got, want) and np.array_equal(got_scale, want_scale)


def test_rope_append_into_a_cache_past_4_gb(va):
    Hkv, D, T = 4, 256, 3
    P = 300_000  # 16 KB each: 4.9 GB of codes
    kp = torch.zeros(P, 16, Hkv, D, dtype=torch.int8, device="cuda")
    vp = torch.zeros_like(kp)
    ks = torch.zeros(P, 16, Hkv, device="cuda")
    vs = torch.zeros_like(ks)
    bt = torch.tensor([[P - 1, P - 2]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([18], dtype=torch.int32, device="cuda")
    k, v = normal(30, 1, T, Hkv, D, dtype=torch.bfloat16), normal(31, 1, T, Hkv, D, dtype=torch.bfloat16)
    spec = va.verify_attn_rope_spec(D)
    va.verify_attn_rope_append(spec, None, None, k, v, kp, vp, ks, vs, bt, lens, "int8")
    assert (vp[P - 1, 15].abs().amax(-1) == 127).all() and (vp[P - 2, :2].abs().amax(-1) == 127).all()
    assert int((vs > 0).sum()) == T * Hkv and int((ks > 0).sum()) == T * Hkv
    got = vp[P - 1, 15].float() * vs[P - 1, 15].unsqueeze(-1)
    assert ((got - v[0, 0].float()).abs() <= 0.5001 * vs[P - 1, 15].unsqueeze(-1)).all()


def test_rope_append_argument_errors(va):
    pages, scale, bt, lens, P = cache_case(8, [20], 2, 2, 64, "int8")
    k = normal(1, 1, 2, 2, 64, dtype=torch.bfloat16)
    spec = va.verify_attn_rope_spec(64)
    good = dict(positions=None, q=None, k_new=k, v_new=k, k_pages=cuda(pages), v_pages=cuda(pages), k_scale=cuda(scale),
                v_scale=cuda(scale), block_table=cuda(bt), seq_lens=cuda(lens), kv_dtype="int8")
    va.verify_attn_rope_append(spec, **good)
    for change in (dict(v_new=k[:, :1]), dict(k_scale=None), dict(k_pages=cuda(pages)[:, :8]), dict(num_pages=P + 1),
                   dict(k_new=k.float()), dict(q=k[0]), dict(block_table=cuda(bt).long()), dict(v_scale=cuda(scale)[:1]),
                   dict(positions=torch.zeros(2, 1, 2, dtype=torch.int32, device="cuda")), dict(seq_lens=cuda(lens)[:0])):
        with pytest.raises(ValueError):
            va.verify_attn_rope_append(spec, **{**good, **change})
    with pytest.raises(va.VerifyAttnError):  # heads whose rows start off 16 bytes
        odd = torch.zeros(1, 2, 2, 68, dtype=torch.bfloat16, device="cuda")[..., 2:66]
        va.verify_attn_rope_append(spec, **{**good, "k_new": odd, "v_new": odd})


# ------------------------------------------------------------------ acceptance


def probs(seed, B, T, V, dtype, model, spread=3.0, top=0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(B, T + 1, V, generator=g) * spread
    if top:
        kth = z.topk(min(top, V), -1).values[..., -1:]
        z = z.masked_fill(z < kth, float("-inf"))
    p = torch.softmax(z, -1).to(dtype)
    q = torch.softmax(z[:, :T] + torch.randn(B, T, V, generator=g), -1).to(dtype) if model else None
    d = (q if model else p[:, :T]).float().flatten(0, 1)
    d = torch.multinomial(d + 1e-30, 1, generator=g).view(B, T).int() if T else torch.zeros(B, 0, dtype=torch.int32)
    return p, q, d, torch.rand(B, T, generator=g), torch.rand(B, generator=g)


def check_accept(va, p, q, d, ua, ue, lens=None, stored=None):
    dev = lambda t: None if t is None else t.cuda()  # noqa: E731
    ref_out, ref_n = around.accept_probs(p.double().numpy(), d.tolist(), ua.tolist(), ue.tolist(),
                                         None if q is None else q.double().numpy(), None if lens is None else lens.tolist())
    ps, qs = stored or (dev(p), dev(q))
    out, n = va.verify_attn_accept_probs(ps, dev(d), dev(ua), dev(ue), draft_probs=qs, draft_lens=dev(lens))
    assert np.array_equal(n.cpu().numpy(), ref_n)
    assert np.array_equal(out.cpu().numpy(), ref_out)
    return ref_out, ref_n


ACCEPT_CASES = [(B, T, V, dtype) for B, T, V in ((1, 0, 5), (1, 1, 1), (3, 2, 7), (2, 5, 1000), (5, 3, 32003), (1, 16, 151936),
                                                 (40, 4, 50257), (310, 1, 64))
                for dtype in (torch.float32, torch.bfloat16, torch.float16)
                if B * V <= 10 ** 6 or dtype != torch.float16]


@pytest.mark.parametrize("B,T,V,dtype", ACCEPT_CASES)
@pytest.mark.parametrize("model", [False, True])
def test_accept_probs(va, B, T, V, dtype, model):
    p, q, d, ua, ue = probs(B + T + V, B, T, V, dtype, model and T > 0)
    out, n = check_accept(va, p, q, d, ua, ue)
    if B * T > 20:
        assert 0 < n.sum() < B * T  # acceptances and rejections both occur


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("top", [0, 20])
def test_accept_probs_truncated_rows_ragged_counts_and_strides(va, dtype, top):
    B, T, V = 9, 4, 3001
    p, q, d, ua, ue = probs(7, B, T, V, dtype, True, top=top)
    lens = torch.tensor([0, 1, 2, 3, 4, 5, -1, 100, 2], dtype=torch.int32)
    check_accept(va, p, q, d, ua, ue, lens)
    # rows of a padded vocabulary (aligned and not), and positions before sequences
    for pad in (1, 5, 7):
        wide_p = torch.rand(B, T + 1, V + pad).to(dtype).cuda()
        wide_q = torch.rand(T, B, V + pad).to(dtype).cuda().transpose(0, 1)
        wide_p[..., :V], wide_q[..., :V] = p.cuda(), q.cuda()
        check_accept(va, p, q, d, ua, ue, lens, stored=(wide_p[..., :V], wide_q[..., :V]))


def test_accept_probs_borders(va):
    """Rows where the sums are exact and the threshold lies on a border, empty residuals, rows without weight,
    out-of-range numbers and tokens, NaN."""
    nan, inf = float("nan"), float("inf")
    V = 70
    rows = []

    def case(p0, p1, draft, ua, ue, q0=None):
        rows.append((p0, p1, draft, ua, ue, q0))

    half = [0.0] * V
    half[3] = half[60] = 0.5
    last = [0.0] * V
    last[V - 1] = 1.0
    flat = [1.0 / 64] * 64 + [0.0] * 6
    zero = [0.0] * V
    for ue in (0.0, 0.25, 0.5, 0.75, 1.0 - 2.0 ** -24, 1.0, 2.0, -1.0, nan):
        case(half, flat, 3, 0.5, ue)        # rejected: u = p(d)
        case(half, flat, 3, 0.4999, ue)     # accepted, then the flat row
        case(last, last, 5, 0.0, ue)
    case(half, flat, 3, 0.9, 0.3, half)     # p = q: the residual is empty, p itself
    case(zero, flat, 3, 0.0, 0.3)           # nothing to draw from
    case(zero, flat, 3, 0.0, 0.3, half)
    case(half, flat, -1, 0.0, 0.9)          # no such token
    case(half, flat, V, 0.0, 0.9, half)
    case(half, flat, 3, nan, 0.2)           # no comparison with NaN holds
    odd = [nan, -0.5, inf, 2.0, 1e-45, 2.0 ** -54, 2.0 ** -55, -inf, -0.0] + [0.0] * (V - 9)
    for ue in (0.0, 0.49, 0.5, 0.51, 0.9999):
        case(odd, odd, 0, 0.1, ue)          # draft 0 has p = NaN: rejected
        case(odd, odd, 2, 0.1, ue)          # p = inf: accepted
        case(odd, odd, 8, 0.1, ue, odd)
    tiny = [0.0] * V
    tiny[10], tiny[20], tiny[30], tiny[40] = 2.0 ** -53, 2.0 ** -54, 2.0 ** -55, 1.5 * 2.0 ** -54
    for ue in (0.0, 0.39, 0.41, 0.59, 0.61, 0.99):
        case(tiny, tiny, 20, 0.5, ue)
    edge = [2.0 ** -10, 2.0 ** -10 - 2.0 ** -34, 2.0 ** -11, 3.0 * 2.0 ** -33, 2.0 ** -32 + 2.0 ** -55] + [0.0] * (V - 5)
    for ue in (0.0, 0.3, 0.399999, 0.4, 0.7999, 0.8, 0.999999):  # around the steps in which the numbers are read
        case(edge, edge, 60, 0.5, ue)
        case(edge, edge, 60, 0.5, ue, [x / 2 for x in edge])
    for model in (False, True):
        some = [r for r in rows if (r[5] is not None) == model]
        p = torch.tensor([[r[0], r[1]] for r in some], dtype=torch.float32)
        q = torch.tensor([[r[5]] for r in some], dtype=torch.float32) if model else None
        d = torch.tensor([[r[2]] for r in some], dtype=torch.int32)
        check_accept(va, p, q, d, torch.tensor([[r[3]] for r in some]), torch.tensor([r[4] for r in some]))


def test_accept_probs_is_the_target_distribution(va):
    """A grid of given numbers through the kernel: the shares of the first token are p_0 (to the grid's width)."""
    n, V = 64, 12
    p0 = torch.softmax(torch.randn(V, generator=torch.Generator().manual_seed(1)), 0)
    q0 = torch.softmax(torch.randn(V, generator=torch.Generator().manual_seed(2)), 0)
    grid = (torch.arange(n) + 0.5) / n
    u, v = [g.reshape(-1).cuda() for g in torch.meshgrid(grid, grid, indexing="ij")]
    share = torch.zeros(V, dtype=torch.float64)
    B = n * n
    p = p0.cuda().expand(B, 2, V)
    q = q0.cuda().expand(B, 1, V)
    for d in range(V):
        out, _ = va.verify_attn_accept_probs(p, torch.full((B, 1), d, dtype=torch.int32, device="cuda"), u[:, None].contiguous(),
                                             v, draft_probs=q)
        share += float(q0[d]) * torch.bincount(out[:, 0].cpu().long(), minlength=V).double() / B
    assert (share - p0.double()).abs().max() < 2.0 / n


def test_accept_probs_rows_past_32_bits(va):
    """Sequences more than 2^31 elements apart in one tensor."""
    V, far = 500, 2 ** 31 + 16
    p, _, d, ua, ue = probs(3, 2, 2, V, torch.bfloat16, False)
    base = torch.empty(far + 3 * V, dtype=torch.bfloat16, device="cuda")
    ps = base.as_strided((2, 3, V), (far, V, 1))
    ps.copy_(p)
    check_accept(va, p, None, d, ua, ue, stored=(ps, None))


def test_accept_probs_argument_errors(va):
    p, q, d, ua, ue = (None if t is None else t.cuda() for t in probs(1, 2, 3, 50, torch.float32, True))
    va.verify_attn_accept_probs(p, d, ua, ue, draft_probs=q)
    for change in (dict(target_probs=p[0]), dict(target_probs=p.double()), dict(draft_tokens=d.long()), dict(u_accept=ua[:, :2]),
                   dict(u_emit=ue[:1]), dict(draft_probs=q[:, :2]), dict(draft_probs=q.half()), dict(draft_lens=d[0, :1].contiguous()),
                   dict(out_tokens=d), dict(target_probs=p.transpose(1, 2).contiguous().transpose(1, 2)),
                   dict(draft_tokens=d.cpu())):
        with pytest.raises(ValueError):
            va.verify_attn_accept_probs(**{**dict(target_probs=p, draft_tokens=d, u_accept=ua, u_emit=ue, draft_probs=q), **change})


# ------------------------------------------------------------------ pages


def gpu_pool(va, pool, extra=()):
    """A PagePool with the state of an around.Pages and its buffers (and more)."""
    i32 = lambda a: cuda(np.asarray(a, np.int32))  # noqa: E731
    return va.PagePool(i32(pool.table), i32(pool.lens), i32(pool.ref), i32(pool.stack), i32([pool.num_free]),
                       [cuda(b) for b in pool.buffers] + list(extra))


def check_pool(dev, pool):
    torch.cuda.synchronize()
    assert np.array_equal(dev.seq_lens.cpu().numpy(), pool.lens)
    assert np.array_equal(dev.ref_count.cpu().numpy(), pool.ref)
    assert int(dev.num_free.item()) == pool.num_free
    assert np.array_equal(dev.free_list.cpu().numpy(), pool.stack)
    assert np.array_equal(dev.block_table.cpu().numpy(), pool.table)
    assert int(dev.flags.item()) == pool.flags
    for x, y in zip(dev.buffers, pool.buffers):
        assert np.array_equal(x.cpu().numpy(), y)


def apply(va, dev, pool, name, args):
    getattr(pool, name)(*args)
    if name == "resize":
        va.verify_attn_pages_resize(dev, cuda(args[0]))
    elif name == "compact":
        va.verify_attn_pages_compact(dev)
    else:
        parents, children, lens, share = args
        va.verify_attn_pages_fork(dev, cuda(parents), cuda(children), None if lens is None else cuda(lens), share)


def make_buffers(rng, P):
    """A K, V and scale buffer of odd sizes (256 B, 2,048 + 16 B and 48 B a page)."""
    return [rng.integers(0, 255, (P, 256)).astype(np.uint8), rng.integers(0, 255, (P, 2064)).astype(np.uint8),
            rng.random((P, 12)).astype(np.float32)]


@pytest.mark.parametrize("P,B,stride,steps,grow", [(60, 7, 12, 150, 40), (9, 3, 6, 60, 30), (1, 1, 1, 10, 16),
                                                   (5000, 300, 40, 12, 300), (40000, 50, 3000, 8, 9000)])
def test_pages_random_calls(va, P, B, stride, steps, grow):
    """Every table, count, list and page after each of a run of random calls, refused ones among them."""
    rng = np.random.default_rng(P + B)
    pool = around.Pages(P, B, stride, make_buffers(rng, P))
    dev = gpu_pool(va, pool)
    for _ in range(steps):
        name, args = random_step(rng, pool, grow)
        apply(va, dev, pool, name, args)
        check_pool(dev, pool)
        pool.check()
        if pool.flags:
            assert va.verify_attn_pages_flags(dev) == pool.flags
            pool.flags = 0


def test_pages_create_takes_the_lowest_page_first(va):
    kp = torch.zeros(50, 16, 2, 64, dtype=torch.int8, device="cuda")
    pool = va.PagePool.create(50, 4, 10, [kp])
    va.verify_attn_pages_resize(pool, cuda(np.array([33, 0, 16, 1], np.int32)))
    assert pool.block_table[0, :4].tolist() == [0, 1, 2, -1] and pool.block_table[2, 0] == 3 and pool.block_table[3, 0] == 4
    assert pool.num_free.item() == 45 and va.verify_attn_pages_flags(pool) == 0


def test_pages_at_the_limits(va):
    """The most sequences, forks and pages that a call takes."""
    P, B, stride = 2 ** 22, 8192, 40
    rng = np.random.default_rng(6)
    pool = around.Pages(P, B, stride, [rng.integers(0, 255, (P, 16)).astype(np.uint8)])
    pool.stack = rng.permutation(P)
    dev = gpu_pool(va, pool)
    lens = rng.integers(0, 640, B)
    lens[B // 2:] = 0
    order = rng.permutation(B // 2)
    for name, args in (("resize", (lens.astype(np.int32),)),
                       ("fork", (order.astype(np.int32), (B // 2 + order).astype(np.int32), None, True)),
                       ("fork", (np.arange(B, dtype=np.int32), np.arange(B, dtype=np.int32)[::-1].copy(), None, False)),
                       ("resize", (np.where(rng.random(B) < 0.5, lens // 2, 640).astype(np.int32),)), ("compact", ())):
        apply(va, dev, pool, name, args)
        check_pool(dev, pool)


def test_pages_all_of_a_long_sequence_at_once(va):
    """A 262,144-token sequence taken, shared, copied, freed and the rest compacted, on the wide path."""
    P, B, stride = 40000, 3, 16400
    rng = np.random.default_rng(4)
    pool = around.Pages(P, B, stride, [rng.integers(0, 255, (P, 16)).astype(np.uint8)])
    dev = gpu_pool(va, pool)
    child = (np.array([0], np.int32), np.array([1], np.int32), None)
    for name, args in (("resize", (np.array([262144, 0, 100], np.int32),)), ("fork", child + (True,)),
                       ("resize", (np.array([262150, -1, 0], np.int32),)), ("resize", (np.array([5, -1, -1], np.int32),)),
                       ("fork", (np.array([1], np.int32), np.array([2], np.int32), np.array([200001], np.int32), False)),
                       ("resize", (np.array([-1, 0, -1], np.int32),)), ("compact", ())):
        apply(va, dev, pool, name, args)
        check_pool(dev, pool)
        pool.check()


def test_pages_sequences_cut_back_into_a_shared_page_get_their_own(va):
    rng = np.random.default_rng(5)
    pool = around.Pages(12, 3, 4, [rng.integers(0, 255, (12, 64)).astype(np.uint8)])
    dev = gpu_pool(va, pool)
    both = np.array([0, 0], np.int32), np.array([1, 2], np.int32)
    for name, args in (("resize", (np.array([48, 0, 0], np.int32),)), ("fork", both + (None, True)),
                       ("resize", (np.array([40, 40, 33], np.int32),)),      # all three into page 2, shared
                       ("resize", (np.array([48, 41, 34], np.int32),))):     # three copies; the old page is given back
        apply(va, dev, pool, name, args)
        check_pool(dev, pool)
        pool.check()
    assert pool.ref.max() == 3 and len({int(pool.table[b, 2]) for b in range(3)}) == 3
    apply(va, dev, pool, "resize", (np.array([64, 49, 49], np.int32),))
    check_pool(dev, pool)


def test_pages_exhausted_pool_serves_in_order(va):
    pool = around.Pages(5, 4, 8, [np.zeros((5, 16), np.uint8)])
    dev = gpu_pool(va, pool)
    for new in ([20, 48, 10, 0], [-1, 16, 16, 3], [0, 80, 1, 32], [0, 0, 0, 0], [100, 0, 0, 0]):
        apply(va, dev, pool, "resize", (np.array(new, np.int32),))
        check_pool(dev, pool)
        pool.check()
    assert pool.flags == around.EXHAUSTED


def test_pages_bad_tables_are_flagged_and_skipped(va):
    """Entries outside the pool, counts that are too low, a list that is too long: flagged, and nothing outside is read
    or written (the tensors around the pool's stay as they are)."""
    P, B, stride = 8, 2, 3
    room = torch.full((1000,), 77, dtype=torch.int32, device="cuda")
    cut = lambda at, n: room[at:at + n]  # noqa: E731
    table, lens, ref, stack, left, flags = cut(100, 6).view(2, 3), cut(200, 2), cut(300, 8), cut(400, 8), cut(500, 1), cut(600, 1)

    def state(t, ln, r, s, n):
        for x, v in ((table, t), (lens, ln), (ref, r), (stack, s), (left, n), (flags, [0])):
            x.copy_(torch.tensor(v, dtype=torch.int32).view(x.shape))

    data = torch.arange(P * 16, dtype=torch.int32, device="cuda").view(P, 16)
    before = data.clone()
    pool = va.PagePool(table, lens, ref, stack, left, [data], flags=flags)
    new = lambda *v: cuda(np.array(v, np.int32))  # noqa: E731
    ok_stack = [0, 1, 2, 3, 4, 5, 6, 7]
    state([5, 99, -7, -1, -1, -1], [40, 0], [0, 0, 0, 0, 0, 1, 0, 0], ok_stack, [5])
    va.verify_attn_pages_resize(pool, new(3, 0))      # drops 99 and -7
    assert flags.item() == va.VA_PAGES_BAD_ENTRY and left.item() == 5 and table[0].tolist() == [5, -1, -1]
    state([5, 6, 7, -1, -1, -1], [48, 0], [0] * 8, ok_stack, [5])
    va.verify_attn_pages_resize(pool, new(0, 0))      # nobody holds them
    assert flags.item() == va.VA_PAGES_BAD_COUNT and left.item() == 5 and ref.tolist() == [0] * 8
    state([5, 6, 7, -1, -1, -1], [48, 0], [0, 0, 0, 0, 0, 1, 1, 1], ok_stack, [8])
    va.verify_attn_pages_resize(pool, new(0, 0))      # a full list gets three more
    assert flags.item() & va.VA_PAGES_BAD_COUNT and left.item() == 8
    state([-1] * 6, [0, 0], [0] * 8, ok_stack, [1000])
    va.verify_attn_pages_resize(pool, new(16, -1))    # a count of free pages outside the pool
    assert flags.item() == va.VA_PAGES_BAD_COUNT and left.item() == 7 and table[0, 0] == 7
    state([-1] * 6, [0, 0], [0] * 8, [0, 1, 2, 3, 4, 5, 6, 800], [8])
    va.verify_attn_pages_resize(pool, new(32, -1))    # a list entry outside the pool
    assert flags.item() == va.VA_PAGES_BAD_ENTRY and table[0].tolist() == [-1, 6, -1]
    state([-1] * 6, [-5, 10 ** 6], [0] * 8, ok_stack, [8])
    va.verify_attn_pages_resize(pool, new(16, 16))    # lengths that no table holds
    assert flags.item() == va.VA_PAGES_BAD_REQUEST and lens.tolist() == [-5, 10 ** 6] and left.item() == 8
    state([9, -3, 2, -1, -1, -1], [40, 0], [0, 0, 1, 0, 0, 0, 0, 0], ok_stack, [8])
    va.verify_attn_pages_fork(pool, new(0), new(1))
    assert flags.item() == va.VA_PAGES_BAD_ENTRY and table[1].tolist() == [-1, -1, 7]
    assert torch.equal(data[7], before[2])
    data.copy_(before)
    state([9, -3, 6, 4, -1, -1], [40, 16], [0, 0, 0, 0, 0, 0, 1, 0], ok_stack, [3])
    va.verify_attn_pages_compact(pool)                # 9, -3 outside, 4 held by nobody, 3 free pages of 7
    assert flags.item() == va.VA_PAGES_BAD_ENTRY | va.VA_PAGES_BAD_COUNT
    assert table.tolist() == [[9, -3, 0], [4, -1, -1]] and ref.tolist() == [1] + [0] * 7 and left.item() == 7
    assert torch.equal(data[0], before[6])
    torch.cuda.synchronize()
    mine = torch.zeros(1000, dtype=torch.bool)
    for at, n in ((100, 6), (200, 2), (300, 8), (400, 8), (500, 1), (600, 1)):
        mine[at:at + n] = True
    assert (room.cpu()[~mine] == 77).all()


def test_pages_copies_past_4_gb(va):
    P = 300_000
    data = torch.zeros(P, 16384, dtype=torch.uint8, device="cuda")
    data[P - 1] = torch.arange(16384, device="cuda") % 251
    data[P - 2] = 9
    pool = va.PagePool.create(P, 3, 4, [data])
    pool.free_list.copy_(torch.arange(P, dtype=torch.int32, device="cuda"))  # the highest page first
    va.verify_attn_pages_resize(pool, cuda(np.array([32, 0, 0], np.int32)))
    assert pool.block_table[0, :2].tolist() == [P - 1, P - 2]
    va.verify_attn_pages_fork(pool, cuda(np.array([0], np.int32)), cuda(np.array([1], np.int32)), share=False)
    assert torch.equal(data[P - 3], data[P - 1]) and (data[P - 4] == 9).all()
    va.verify_attn_pages_compact(pool)
    assert sorted(pool.block_table[:2, :2].reshape(-1).tolist()) == [0, 1, 2, 3]
    assert (data[0] == 9).all() and torch.equal(data[1], data[P - 3]) and va.verify_attn_pages_flags(pool) == 0


def test_pages_many_buffers(va):
    """More buffers than one launch takes."""
    P, n = 20, 150
    buffers = [torch.randint(0, 100, (P, 8 + 4 * (i % 3)), dtype=torch.int32, device="cuda") for i in range(n)]
    want = [b.clone() for b in buffers]
    pool = va.PagePool.create(P, 2, 4, buffers)
    va.verify_attn_pages_resize(pool, cuda(np.array([20, 0], np.int32)))
    va.verify_attn_pages_fork(pool, cuda(np.array([0], np.int32)), cuda(np.array([1], np.int32)))
    assert pool.block_table[1, :2].tolist() == [0, 2]
    for b, w in zip(buffers, want):
        w[2] = w[1]
        assert torch.equal(b, w)
    va.verify_attn_pages_resize(pool, cuda(np.array([0, -1], np.int32)))
    va.verify_attn_pages_compact(pool)  # pages 0 and 2, shared and copied, become 0 and 1
    assert pool.block_table[1, :2].tolist() == [0, 1] and pool.num_free.item() == P - 2
    for b, w in zip(buffers, want):
        w[1] = w[2]
        assert torch.equal(b, w)
    bare = va.PagePool.create(P, 2, 4, [])
    va.verify_attn_pages_resize(bare, cuda(np.array([20, 40], np.int32)))
    assert bare.num_free.item() == P - 5
    va.verify_attn_pages_resize(bare, cuda(np.array([0, 40], np.int32)))
    va.verify_attn_pages_compact(bare)
    assert bare.block_table[1, :3].tolist() == [2, 0, 1] and bare.ref_count.tolist() == [1] * 3 + [0] * (P - 3)


def test_page_pool_argument_errors(va):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    good = [i32(2, 3), i32(2), i32(8), i32(8), i32(1), [torch.zeros(8, 4, device="cuda")]]
    pool = va.PagePool(*good)
    for at, bad in ((0, i32(6)), (1, i32(3)), (2, i32(8).long()), (3, i32(7)), (4, i32(2)), (5, [torch.zeros(7, 4, device="cuda")]),
                    (5, [torch.zeros(4, 8, device="cuda").t()]), (5, [torch.zeros(8, 4)])):
        with pytest.raises(ValueError):
            va.PagePool(*[bad if i == at else x for i, x in enumerate(good)])
    with pytest.raises(ValueError):
        va.PagePool.create(0, 2, 3, [torch.zeros(0, 4, device="cuda")])
    with pytest.raises(ValueError):
        va.verify_attn_pages_resize(pool, i32(3))
    with pytest.raises(ValueError):
        va.verify_attn_pages_fork(pool, i32(2), i32(3))
    with pytest.raises(ValueError):
        va.verify_attn_pages_fork(pool, i32(2), i32(2), lens=i32(1))
    odd = va.PagePool(*good[:5], [torch.zeros(8, 3, device="cuda")])  # 12 bytes a page
    with pytest.raises(va.VerifyAttnError):
        va.verify_attn_pages_compact(odd)


# ------------------------------------------------------------------ streams, graphs, together


class Step:
    """One request's verify step through the entry points, on buffers that stay."""

    def __init__(self, va, kv_dtype="int8", T=5, Hq=8, Hkv=2, D=64, B=3, V=700, seed=0):
        self.va, self.kv, self.T, self.B, self.V = va, kv_dtype, T, B, V
        P, self.stride = 64, 12
        self.spec = va.verify_attn_rope_spec(D, sections=[D // 2 - 8, 4, 4], layout="dealt")
        make = lambda *s, **k: torch.zeros(*s, device="cuda", **k)  # noqa: E731
        kind = torch.bfloat16 if kv_dtype == "bf16" else torch.int8
        self.kp, self.vp = make(P, 16, Hkv, D, dtype=kind), make(P, 16, Hkv, D, dtype=kind)
        self.ks, self.vs = make(P, 16, Hkv), make(P, 16, Hkv)
        self.pool = va.PagePool.create(P, B, self.stride, [self.kp, self.vp, self.ks, self.vs])
        self.qkv = normal(seed + 1, B, T, Hq + 2 * Hkv, D, dtype=torch.bfloat16)
        self.q, self.k, self.v = self.qkv.split([Hq, Hkv, Hkv], 2)
        self.q_out = make(B, T, Hq, D, dtype=torch.bfloat16)
        p, q, d, ua, ue = probs(seed, B, T, V, torch.float32, True)
        self.given = [t.cuda() for t in (p, d, ua, ue, q)]
        self.tokens, self.accepted = make(B, T + 1, dtype=torch.int32), make(B, dtype=torch.int32)
        self.new, self.kept = make(B, dtype=torch.int32), make(B, dtype=torch.int32)

    def run(self, stream=None):
        """Grow by T, rotate and append, decide, cut back to what was accepted."""
        va = self.va
        torch.add(self.pool.seq_lens, self.T, out=self.new)
        va.verify_attn_pages_resize(self.pool, self.new, stream=stream)
        va.verify_attn_rope_append(self.spec, None, self.q, self.k, self.v, self.kp, self.vp, self.ks, self.vs,
                                   self.pool.block_table, self.pool.seq_lens, self.kv, q_out=self.q_out, stream=stream)
        p, d, ua, ue, q = self.given
        va.verify_attn_accept_probs(p, d, ua, ue, draft_probs=q, out_tokens=self.tokens, num_accepted=self.accepted, stream=stream)
        torch.add(self.pool.seq_lens, self.accepted, out=self.kept)
        self.kept -= self.T
        va.verify_attn_pages_resize(self.pool, self.kept, stream=stream)

    def state(self):
        torch.cuda.synchronize()
        p = self.pool
        return [t.clone() for t in (p.block_table, p.seq_lens, p.ref_count, p.num_free, p.flags, self.kp, self.vp, self.ks,
                                    self.vs, self.q_out, self.tokens, self.accepted)]


def test_steps_on_a_side_stream_and_captured_are_the_eager_ones(va):
    """Three steps eagerly; on a side stream; and as two graphs over one pool (one workspace), replayed in order."""
    eager, side, graph = Step(va), Step(va), Step(va)
    for _ in range(3):
        eager.run()
    want = eager.state()
    assert want[1].sum() > 0 and want[4].item() == 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(3):
            side.run()
    for a, b in zip(side.state(), want):
        assert torch.equal(a, b)
    explicit = Step(va)
    s2 = torch.cuda.Stream()
    s2.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        with torch.cuda.stream(s2):  # torch's own additions there too; the calls are told the raw handle
            explicit.run(stream=s2.cuda_stream)
    for a, b in zip(explicit.state(), want):
        assert torch.equal(a, b)
    default = Step(va)
    for _ in range(3):
        default.run(stream=0)  # the raw handle of the default stream
    for a, b in zip(default.state(), want):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    first, second = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(first):
        graph.run()
    with torch.cuda.graph(second):
        graph.run()
        graph.run()
    assert graph.pool.seq_lens.sum().item() == 0  # captured, not run
    first.replay()
    second.replay()
    for a, b in zip(graph.state(), want):
        assert torch.equal(a, b)


def test_two_steps_at_once_on_two_streams(va):
    """Pools of their own on streams of their own: nothing is shared."""
    steps = [Step(va, seed=s) for s in (0, 1)]
    alone = [Step(va, seed=s) for s in (0, 1)]
    for st in alone:
        for _ in range(10):
            st.run()
    want = [st.state() for st in alone]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for st, s in zip(steps, streams):
            with torch.cuda.stream(s):
                st.run()
    for st, w in zip(steps, want):
        for a, b in zip(st.state(), w):
            assert torch.equal(a, b)


def test_outputs_made_on_a_given_stream_belong_to_it(va):
    """Without outputs given, the call makes them on the stream it runs on: work that is still queued on the current
    stream cannot share their memory."""
    spec = va.verify_attn_rope_spec(128)
    q = normal(1, 1, 4096, 8, 128, dtype=torch.bfloat16)
    pos = torch.arange(4096, dtype=torch.int32, device="cuda").view(1, 1, -1)
    want, _ = va.verify_attn_rope(spec, pos, q)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = []
    for _ in range(20):
        scratch = torch.empty_like(q)
        scratch.fill_(3.0)
        del scratch  # its memory may be handed out again on this stream, whose fill may not have run yet
        got.append(va.verify_attn_rope(spec, pos, q, stream=s)[0])
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.parametrize("kv_dtype", ["int8", "bf16"])
def test_a_run_of_all_of_them_with_verify_attention(va, kv_dtype):
    """Steps with forks and compaction between: attention over the pool's own table equals the plain definition over a
    cache that is read back, and moving pages does not change a bit of it."""
    step = Step(va, kv_dtype, B=4)
    T, B, D, Hq, Hkv = step.T, step.B, 64, 8, 2
    pool = step.pool

    def attention():
        lens = pool.seq_lens.tolist()
        act = [b for b in range(B) if lens[b] >= T]
        plan = va.verify_attn_plan([lens[b] for b in act], T, Hq, Hkv, D, kv_dtype, block_table_stride=step.stride,
                                   num_pages=pool.num_pages)
        table, sl = pool.block_table[act].contiguous(), pool.seq_lens[act].contiguous()
        q = step.q_out[act].contiguous()
        out, lse = torch.empty_like(q), torch.empty(len(act), T, Hq, device="cuda")
        va.verify_attn_with_plan(plan, q, step.kp, step.vp, step.ks, step.vs, table, sl, T, out, lse)
        torch.cuda.synchronize()
        assert va.verify_attn_plan_device_flags(plan) == 0
        plan.destroy()
        raw = (lambda t: bits16(t)) if kv_dtype == "bf16" else (lambda t: t.cpu().numpy())
        w = dict(q=bits16(q), k_pages=raw(step.kp), v_pages=raw(step.vp), k_scale=None if kv_dtype == "bf16" else step.ks.cpu().numpy(),
                 v_scale=None if kv_dtype == "bf16" else step.vs.cpu().numpy(), block_table=table.cpu().numpy(),
                 seq_lens=sl.cpu().numpy(), T=T, Hq=Hq, Hkv=Hkv, D=D, kv_dtype=kv_dtype, B=len(act), num_pages=pool.num_pages)
        ref_out, ref_lse = oracle.verify_attn(w)
        compare(out.float().cpu().numpy(), lse.cpu().numpy(), ref_out, ref_lse, "attention over the pool")
        return out, lse

    i32 = lambda *v: cuda(np.array(v, np.int32))  # noqa: E731
    va.verify_attn_pages_resize(pool, i32(40, 21, 0, 0))
    va.verify_attn_pages_fork(pool, i32(0), i32(2))
    for _ in range(2):
        step.run()
    va.verify_attn_pages_resize(pool, (pool.seq_lens + T * (pool.seq_lens > 0)).int())
    va.verify_attn_rope_append(step.spec, None, step.q, step.k, step.v, step.kp, step.vp, step.ks, step.vs, pool.block_table,
                               pool.seq_lens, kv_dtype, q_out=step.q_out)
    attention()
    va.verify_attn_pages_resize(pool, i32(-1, 0, -1, -1))     # one request leaves
    va.verify_attn_pages_fork(pool, i32(2), i32(1), share=False)
    second = attention()
    va.verify_attn_pages_compact(pool)
    third = attention()
    assert torch.equal(third[0], second[0]) and torch.equal(third[1], second[1])
    assert va.verify_attn_pages_flags(pool) == 0
    held = pool.block_table[pool.block_table >= 0]
    assert int(held.max()) < pool.num_pages - pool.num_free.item()


def test_a_refused_call_leaves_its_outputs_alone(va):
    """A refused call leaves its outputs alone and the context usable."""
    p, _, d, ua, ue = (None if t is None else t.cuda() for t in probs(1, 1, 1, 16, torch.float32, False))
    out = torch.full((1, 2), 5, dtype=torch.int32, device="cuda")
    n = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    rows = va._Rows(p.data_ptr(), 32, 16)
    lib = va.library()
    P = ctypes.c_void_p
    rc = lib.verify_attn_accept_probs(ctypes.byref(rows), None, 7, P(d.data_ptr()), None, P(ua.data_ptr()), P(ue.data_ptr()), 1,
                                      1, 16, P(out.data_ptr()), P(n.data_ptr()), None)
    assert rc == -2 and out.tolist() == [[5, 5]] and n.item() == 5
    va.verify_attn_accept_probs(p, d, ua, ue, out_tokens=out, num_accepted=n)
    assert n.item() in (0, 1)
