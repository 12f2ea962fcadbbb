"""GPU parity of the operators of a prompt worked in chunks against their definitions in 64 bits: attention of
ragged chunks, the weights that cached tokens gather, eviction, log probabilities, and a run of them
together.

Tolerances.  A score is a sum of D exact products in binary32, off by at most D 2^-23 of what it is made
of, sum |q_d| |K_d| / sqrt(D) =: reach (a multiplication by the key's scale and one by the softmax's scale are
two roundings more, within the same bound for D >= 64); exp2's argument is rounded once more and exp2 is good
to 2^-22.  So a probability is off by e := 2 D 2^-23 reach + 2^-20 of itself (once in the numerator, once in the
sum).  It is rounded to half a step of the values' tile's type, h = 2^-8 (bf16 cache) or 2^-11 (fp16, codes), which
moves the output by at most h sum p |V|.  fp16 has a smallest step: half of it is 2^-25, in units in which the
largest value scale of a tile of keys is at least 2^-6 (and the likeliest key's p is 1), and it takes the place of
h P where P < 2^-14, so at most where p vs < 2^-8 of the likeliest key's p and the largest vs: 2^-19 |V| (largest vs) /
vs of each such key.  The output's own rounding is 2^-8 of it.  Binary32 sums of exponentials
over a few thousand keys: 2^-14 (at most 2^10 additions in a row).  log-sum-exp: D 2^-23 reach + 2^-14 for the sum's
error + 2^-22 of its size.  Gathered weights: e + 2^-14, and a rounding of lse's product, 2^-22 (1 + |lse|).
Log probabilities: derived at the test.  Everything else is whole numbers and copies: equal."""
import threading

import numpy as np
import pytest

from oracle import chunks

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

KINDS = ["bf16", "fp8_e4m3", "int8", "int4", "int2"]


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


def make_pool(seed, P, Hkv, D, kv, std=1.0):
    """(pages, scales) of one pool of random rows."""
    x = normal(seed, P, 16, Hkv, D) * std
    if kv == "bf16":
        return x.bfloat16(), None
    top = x.abs().amax(-1)
    most = {"fp8_e4m3": 448.0, "int8": 127.0, "int4": 7.0, "int2": 1.0}[kv]
    scale = torch.where(top > 0, top / most, torch.ones_like(top))
    y = x / scale.unsqueeze(-1)
    if kv == "fp8_e4m3":
        return y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale
    y = y.round().clamp(-most, most).to(torch.int8)
    if kv == "int8":
        return y, scale
    w = 4 if kv == "int4" else 2
    y = (y.view(torch.uint8) & ((1 << w) - 1)).view(P, 16, Hkv, D * w // 8, 8 // w)
    packed = torch.zeros_like(y[..., 0])
    for i in range(8 // w):
        packed |= y[..., i] << (i * w)
    return packed, scale


class Batch:
    """A batch of chunks over a pool in mixed order, and the definition's view of it."""

    def __init__(self, new, lens, Hq, Hkv, D, kv, seed=0, k_std=1.0, v_std=1.0, extra=3):
        self.new, self.lens, self.Hq, self.Hkv, self.D, self.kv = list(new), list(lens), Hq, Hkv, D, kv
        blocks = [(n + 15) // 16 for n in lens]
        P = sum(blocks) + extra
        order = np.random.default_rng(seed).permutation(P).astype(np.int32)
        table = np.full((len(lens), max(max(blocks), 1) + 1), -5, np.int32)  # entries past a sequence are not looked at
        at = 0
        for b, n in enumerate(blocks):
            table[b, :n] = order[at:at + n]
            at += n
        self.table, self.bt, self.P = table, cuda(table), P
        self.kp, self.ks = make_pool(seed + 1, P, Hkv, D, kv, k_std)
        self.vp, self.vs = make_pool(seed + 2, P, Hkv, D, kv, v_std)
        self.N = sum(new)
        self.q = normal(seed + 3, self.N, Hq, D, dtype=torch.bfloat16)

    def host(self):
        """Pages, scales as numpy."""
        def of(t):
            return None if t is None else (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy()
        return of(self.kp), of(self.vp), of(self.ks), of(self.vs)

    def plan(self, va, **kw):
        return va.verify_attn_chunk_plan(self.new, self.lens, self.Hq, self.Hkv, self.D, self.kv, **kw)

    def run(self, va, plan, q=None, **kw):
        return va.verify_attn_chunk(plan, self.q if q is None else q, self.kp, self.vp, self.ks, self.vs, self.bt, **kw)

    def weigh(self, va, plan, lse, w, **kw):
        return va.verify_attn_chunk_weights(plan, self.q, self.kp, self.ks, self.bt, lse, w, **kw)

    def want(self):
        kp, vp, ks, vs = self.host()
        return chunks.chunk(self.q.double().cpu().numpy(), kp, vp, ks, vs, self.table, self.new, self.lens, self.kv, self.Hkv)

    def check(self, out, lse):
        ref, ref_lse, size, reach = self.want()
        check_rows(self.kv, self.D, out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, ref_lse, size, reach)


def check_rows(kv, D, out, lse, ref, ref_lse, sizes, reach):
    size, small = sizes
    half = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
    e = (2 * D * 2.0 ** -23 * reach + 2.0 ** -20 + 2.0 ** -14)[..., None]
    assert np.array_equal(np.isfinite(out), np.isfinite(ref))
    with np.errstate(invalid="ignore"):
        bound = (half + e) * size + (0 if kv == "bf16" else 2.0 ** -19 * small) + 2.0 ** -8 * np.abs(ref) * (1 + half + e)
        bad = np.abs(out - ref) > bound + 1e-38
    assert not bad[np.isfinite(ref)].any(), (np.abs(out - ref)[bad].max(), bound[bad].min(), np.argwhere(bad)[:5])
    assert np.array_equal(np.isneginf(lse), np.isneginf(ref_lse))
    ok = np.isfinite(ref_lse)
    assert (np.abs(lse[ok] - ref_lse[ok]) <= D * 2.0 ** -23 * reach[ok] + 2.0 ** -14 + 2.0 ** -22 * np.abs(ref_lse[ok])).all()


# ------------------------------------------------------------------ chunk attention

SHAPES = [  # new, lens, Hq, Hkv
    ([1], [1], 1, 1),
    ([1], [17], 4, 4),
    ([16], [16], 4, 1),
    ([127, 0, 1], [130, 40, 129], 3, 1),
    ([33, 64, 5], [33, 200, 1000], 8, 2),
    ([65, 2], [300, 2], 12, 2),          # 126 of a tile's 128 rows
    ([20], [2500], 7, 1),                # few rows: keys split
    ([3, 1], [140, 4000], 40, 1),        # three tokens a tile
    ([5], [77], 128, 1),                 # one token a tile
    ([260], [260], 1, 1),                # two tiles of rows of one head, the second nearly empty
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}of{s[1]}-{s[2]}q{s[3]}")
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv", KINDS)
def test_chunk(va, shape, D, kv):
    b = Batch(*shape, D, kv, seed=len(shape[0]) + D)
    plan = b.plan(va)
    out, lse = b.run(va, plan)
    b.check(out, lse)
    assert va.verify_attn_chunk_plan_device_flags(plan) == 0


@pytest.mark.parametrize("shape,sms", [(([100], [1500], 6, 1), 2), (([40], [2500], 12, 2), 16)], ids=["whole", "split"])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv", KINDS)
def test_chunk_and_weights_of_many_tiles_of_keys(va, kv, D, shape, sms):
    """Every ring of the kernel is gone through several times: an odd number of stages between its two producers once let
    one of them pass a barrier two phases ahead, and a slot was once given back before its loads were done."""
    b = Batch(*shape, D, kv, seed=D + 7)
    plan = b.plan(va, num_sms=sms)
    out, lse = b.run(va, plan)
    b.check(out, lse)
    w = torch.zeros(len(b.new), b.Hkv, max(b.lens), device="cuda")
    check_weights(b, b.weigh(va, plan, lse, w), lse, None)
    assert va.verify_attn_chunk_plan_device_flags(plan) == 0


def test_weights_of_many_tiles_of_rows(va):
    for D, kv in ((64, "bf16"), (128, "fp8_e4m3"), (256, "int8"), (256, "bf16")):
        b = Batch([700, 30], [800, 300], 16, 1, D, kv, seed=D)
        plan = b.plan(va)
        _, lse = b.run(va, plan)
        old = normal(2, 2, 1, 800).abs()
        w = old.clone()
        check_weights(b, b.weigh(va, plan, lse, w), lse, old)
        assert va.verify_attn_chunk_plan_device_flags(plan) == 0


@pytest.mark.parametrize("kv", ["bf16", "int8", "int4"])
@pytest.mark.parametrize("k_std,v_std", [(3.0, 1e-4), (0.05, 40.0), (1e-3, 1e4), (30.0, 1e-30)])
def test_chunk_rows_of_any_size(va, kv, k_std, v_std):
    b = Batch([40, 3], [200, 900], 8, 2, 128, kv, seed=5, k_std=k_std, v_std=v_std)
    plan = b.plan(va)
    b.check(*b.run(va, plan))


@pytest.mark.parametrize("kv", ["bf16", "fp8_e4m3"])
@pytest.mark.parametrize("D", [64, 256])
def test_chunk_takes_q_as_it_lies(va, kv, D):
    """A slice of a fused projection, heads outside tokens, padded rows; rows behind the last token stay."""
    b = Batch([30, 9], [80, 400], 6, 2, D, kv, seed=7)
    plan = b.plan(va)
    want, want_lse = b.run(va, plan)
    fused = normal(8, b.N, 6 + 4, D, dtype=torch.bfloat16)
    fused[:, 2:8] = b.q
    outside = torch.empty(6, b.N, D, dtype=torch.bfloat16, device="cuda").copy_(b.q.transpose(0, 1)).transpose(0, 1)
    wide = torch.full((b.N, 6, D + 24), 9.0, dtype=torch.bfloat16, device="cuda")[..., 8:D + 8].copy_(b.q)
    more = torch.full((b.N + 5, 6, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    more[:b.N] = b.q
    for q in (fused[:, 2:8], outside, wide, more):
        out = torch.full((q.shape[0], 6, D), 7.0, dtype=torch.bfloat16, device="cuda")
        lse = torch.full((q.shape[0], 6), 7.0, device="cuda")
        b.run(va, plan, q=q, out=out, lse=lse)
        assert torch.equal(out[:b.N], want) and torch.equal(lse[:b.N], want_lse)
        assert (out[b.N:] == 7).all() and (lse[b.N:] == 7).all()
    one = Batch([1], [40], 1, 1, D, kv, seed=9)  # strides that nothing is reached by may be anything
    p1 = one.plan(va)
    want = one.run(va, p1)[0]
    assert torch.equal(one.run(va, p1, q=torch.as_strided(one.q, (1, 1, D), (1, 1, 1)))[0], want)


def test_chunk_of_the_same_length_is_verify_attention(va):
    """The verify step's own path, for a batch that both take."""
    for kv in ("int8", "bf16"):
        T, lens = 16, [500, 40, 16]
        b = Batch([T] * 3, lens, 8, 2, 128, kv, seed=11)
        out, lse = b.run(va, b.plan(va))
        stride = b.bt.shape[1]
        vplan = va.verify_attn_plan(lens, T, 8, 2, 128, kv, block_table_stride=stride)
        vout, vlse = torch.empty_like(b.q), torch.empty(b.N, 8, device="cuda")
        va.verify_attn_with_plan(vplan, b.q, b.kp, b.vp, b.ks, b.vs, b.bt, cuda(np.array(lens, np.int32)), T, vout, vlse)
        ref, ref_lse, size, reach = b.want()
        for o, l in ((out, lse), (vout, vlse)):
            check_rows(kv, 128, o.double().cpu().numpy(), l.double().cpu().numpy(), ref, ref_lse, size, reach)


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
def test_keys_that_a_token_does_not_see_do_not_touch_it(va, kv, D):
    """Not finite values, keys and scales in the chunk's later tokens, behind the last token, and in other pages."""
    new, lens = [70, 40], [131, 500]
    b = Batch(new, lens, 4, 1, D, kv, seed=13)
    plan = b.plan(va)
    clean, clean_lse = b.run(va, plan)
    bad = float("nan"), float("inf"), float("-inf")
    first = {0: 45, 1: 3}  # tokens from these on hold what the ones before must not feel
    for s in range(2):
        for j in range(lens[s] - new[s] + first[s], ((lens[s] + 15) // 16) * 16):
            page, slot = b.table[s, j // 16], j % 16
            x = bad[j % 3]
            if kv == "bf16":
                b.kp[page, slot, 0, j % D] = x
                b.vp[page, slot, 0, (7 * j) % D] = x
                b.vp[page, slot, 0, (7 * j + 9) % D] = x
            else:
                if kv == "fp8_e4m3":
                    b.vp[page, slot, 0, (7 * j) % D] = 0x7F
                    b.kp[page, slot, 0, j % D] = 0xFF
                b.ks[page, slot, 0] = x
                b.vs[page, slot, 0] = x
    free = np.setdiff1d(np.arange(b.P), np.concatenate([b.table[s, :(lens[s] + 15) // 16] for s in range(2)]))
    b.kp[torch.from_numpy(free).cuda()] = float("nan") if kv == "bf16" else -1 if kv == "int8" else 255
    out, lse = b.run(va, plan)
    at = 0
    for s in range(2):
        upto = at + first[s]
        assert torch.equal(out[at:upto], clean[at:upto]) and torch.equal(lse[at:upto], clean_lse[at:upto])
        assert not torch.isfinite(out[upto:at + new[s]].float()).all(-1).any()  # those who see them do feel them
        at += new[s]


def test_values_that_are_not_finite_reach_exactly_the_rows_that_see_them(va):
    """Element by element, in unsplit and split items."""
    for new, lens, Hq in (([50], [50], 2), ([30], [3000], 1), ([4], [4000], 2)):
        b = Batch(new, lens, Hq, 1, 64, "bf16", seed=17)
        n, L = new[0], lens[0]
        plan = b.plan(va)
        for j, d, x in ((L - 1, 5, float("inf")), (L - n // 2, 9, float("nan")), (L - n + 1, 60, float("-inf")), (L - 1, 60, float("inf"))):
            b.vp[b.table[0, j // 16], j % 16, 0, d] = x
        out, lse = b.run(va, plan)
        ref = b.want()[0]
        got = out.double().cpu().numpy()
        assert np.array_equal(np.isnan(got), np.isnan(ref)) and np.array_equal(np.isposinf(got), np.isposinf(ref))
        assert np.array_equal(np.isneginf(got), np.isneginf(ref)) and torch.isfinite(lse).all()


def test_chunk_without_any_token_and_rows_without_any_key(va):
    b = Batch([0, 0], [0, 30], 4, 2, 64, "int8", seed=1)
    plan = b.plan(va)
    out, lse = torch.full((3, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda"), torch.full((3, 4), 5.0, device="cuda")
    b.run(va, plan, q=torch.zeros_like(out), out=out, lse=lse)
    assert (out == 5).all() and (lse == 5).all() and plan.info()["num_items"] == 0
    for kv in KINDS:  # pages outside the pool are skipped; a row without any other key is empty
        for D in (64, 256):
            b = Batch([20, 3], [20, 700], 4, 2, D, kv, seed=2)
            b.table[0, :2] = b.P, -1
            b.table[1, 3], b.table[1, 20] = 10 ** 6, -2 ** 31
            b.bt = cuda(b.table)
            plan = b.plan(va)
            out, lse = b.run(va, plan)
            assert (out[:20] == 0).all() and torch.isneginf(lse[:20]).all()
            b.check(out, lse)
            assert va.verify_attn_chunk_plan_device_flags(plan) == 1 and va.verify_attn_chunk_plan_device_flags(plan) == 0
            w = torch.full((2, 2, 700), 3.0, device="cuda")
            b.weigh(va, plan, lse, w, accumulate=False)
            assert (w[0, :, :20] == 0).all() and (w[0, :, 20:] == 3).all() and torch.isfinite(w).all()
            assert (w[1, :, 48:64] == 0).all() and (w[1, :, 320:336] == 0).all() and (w[1, :, :48] > 0).all()
            assert va.verify_attn_chunk_plan_device_flags(plan) == 1


def test_chunk_over_a_cache_past_4_gb(va):
    Hkv, D, P = 8, 256, 70_000
    kp, vp = (torch.zeros(P, 16, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    small = Batch([20], [50], 16, Hkv, D, "bf16", seed=21, extra=0)
    far = np.array([[P - 1, P - 40000, P - 2, P - 65000]], np.int32)
    for j in range(4):
        kp[far[0, j]], vp[far[0, j]] = small.kp[small.table[0, j]], small.vp[small.table[0, j]]
    plan = small.plan(va)
    want = small.run(va, plan)
    got = va.verify_attn_chunk(plan, small.q, kp, vp, None, None, cuda(far))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    w = [torch.zeros(1, Hkv, 64, device="cuda") for _ in range(2)]
    va.verify_attn_chunk_weights(plan, small.q, kp, None, cuda(far), want[1], w[0])
    small.weigh(va, plan, want[1], w[1])
    assert torch.equal(w[0], w[1]) and w[0].sum() > 0


def test_chunk_argument_errors(va):
    b = Batch([5, 6], [50, 60], 8, 2, 64, "int8", seed=3)
    plan = b.plan(va)
    out, lse = b.run(va, plan)
    good = dict(q=b.q, k_pages=b.kp, v_pages=b.vp, k_scale=b.ks, v_scale=b.vs, block_table=b.bt, out=out, lse=lse)
    for change in (dict(q=b.q[:10]), dict(q=b.q.float()), dict(q=b.q[:, :4]), dict(q=b.q.cpu()), dict(q=b.q[..., ::2]),
                   dict(k_pages=b.kp.view(torch.uint8)), dict(k_pages=b.kp[:, :8]), dict(v_pages=b.vp[:-1]), dict(k_scale=None),
                   dict(v_scale=b.vs[:-1]), dict(block_table=b.bt[:1]), dict(block_table=b.bt.long()), dict(num_pages=b.P + 1),
                   dict(out=out[:10]), dict(out=out.float()), dict(lse=lse[:, :4]), dict(lse=lse.double()),
                   dict(q=b.q.clone().requires_grad_())):
        with pytest.raises(ValueError):
            va.verify_attn_chunk(plan, **dict(good, **change))
    odd = torch.zeros(11 * 8 * 68 + 8, dtype=torch.bfloat16, device="cuda")
    for change in (dict(q=torch.as_strided(odd, (11, 8, 64), (8 * 68, 68, 1))), dict(q=odd[4:4 + 11 * 512].view(11, 8, 64)),
                   dict(q=b.q[:1].expand(11, 8, 64)), dict(block_table=b.bt[:, :3].contiguous()),
                   dict(out=odd[4:4 + 11 * 512].view(11, 8, 64))):
        with pytest.raises(va.VerifyAttnError) as e:
            va.verify_attn_chunk(plan, **dict(good, **change))
        assert e.value.status == -1
    w = torch.zeros(2, 2, 60, device="cuda")
    pos = torch.zeros(11, dtype=torch.int32, device="cuda")
    good = dict(q=b.q, k_pages=b.kp, k_scale=b.ks, block_table=b.bt, lse=lse, weights=w)
    for change in (dict(weights=w[..., :59]), dict(weights=w.double()), dict(weights=w[:1]), dict(lse=lse[:5]),
                   dict(slot_pos=w.int()), dict(slot_pos=w.int(), positions=pos[:5]),
                   dict(slot_pos=torch.zeros(2, 2, 61, dtype=torch.int32, device="cuda"), positions=pos), dict(slot_pos=w, positions=pos),
                   dict(weights=w.transpose(1, 2).contiguous().transpose(1, 2)), dict(num_pages=b.P + 1)):
        with pytest.raises(ValueError):
            va.verify_attn_chunk_weights(plan, **dict(good, **change))
    for on_one_another in (w[:1].expand(2, 2, 60), w[:, :1].expand(2, 2, 60), torch.as_strided(w, (2, 2, 60), (59, 120, 1))):
        with pytest.raises(va.VerifyAttnError):
            va.verify_attn_chunk_weights(plan, **dict(good, weights=on_one_another))
    heads_first = torch.zeros(2, 2, 60, device="cuda").transpose(0, 1)  # and what does not
    va.verify_attn_chunk_weights(plan, **dict(good, weights=heads_first))


# ------------------------------------------------------------------ gathered weights


def check_weights(b, got, lse, old):
    kp, _, ks, _ = b.host()
    ref = chunks.chunk_weights(b.q.double().cpu().numpy(), kp, ks, b.table, b.new, b.lens, b.kv, b.Hkv, lse.cpu().numpy(),
                               None if old is None else old.cpu().numpy())
    got = got.double().cpu().numpy()
    reach = b.want()[3]
    e = 2 * b.D * 2.0 ** -23 * reach.max() + 2.0 ** -20 + 2.0 ** -14 + 2.0 ** -22 * (1 + np.abs(lse.cpu().numpy()).max())
    for s, (n, L) in enumerate(zip(b.new, b.lens)):
        if n:
            x, y = got[s, :, :L], ref[s, :, :L]
            assert (np.abs(x - y) <= e * np.abs(y) + 1e-38).all(), (np.abs(x - y) / np.abs(y)).max()


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: f"{s[0]}of{s[1]}-{s[2]}q{s[3]}")
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv", KINDS)
def test_chunk_weights(va, shape, D, kv):
    b = Batch(*shape, D, kv, seed=len(shape[0]) + D)
    plan = b.plan(va)
    _, lse = b.run(va, plan)
    B, most = len(b.new), max(b.lens)
    for add in (False, True):
        room = normal(1, B, b.Hkv + 1, most + 9).abs()  # strides wider than the shape
        w = room[:, 1:, 3:most + 6]
        before = room.clone()
        old = w.clone()
        assert b.weigh(va, plan, lse, w, accumulate=add) is w
        check_weights(b, w, lse, old if add else None)
        for s, (n, L) in enumerate(zip(b.new, b.lens)):  # what lies behind the sequences is as it was
            assert torch.equal(w[s, :, L if n else 0:], old[s, :, L if n else 0:])
        w.copy_(old)
        assert torch.equal(room, before)


def test_chunk_weights_keep_the_new_tokens_positions(va):
    b = Batch([7, 0, 20], [40, 16, 20], 4, 2, 64, "int8", seed=4)
    plan = b.plan(va)
    _, lse = b.run(va, plan)
    w = torch.zeros(3, 2, 50, device="cuda")
    pos = torch.full((3, 2, 50), -7, dtype=torch.int32, device="cuda")
    positions = torch.arange(100, 100 + b.N, dtype=torch.int32, device="cuda")
    b.weigh(va, plan, lse, w, slot_pos=pos, positions=positions)
    want = torch.full((3, 2, 50), -7, dtype=torch.int32)
    want[0, :, 33:40] = torch.arange(100, 107, dtype=torch.int32)
    want[2, :, :20] = torch.arange(107, 127, dtype=torch.int32)
    assert torch.equal(pos.cpu(), want)


def test_chunk_weights_shared_by_a_cluster_are_the_same_every_time(va):
    """One long chunk over few keys: CTAs share a block of keys, and their sums are added in one order."""
    b = Batch([3000], [3000], 16, 1, 128, "bf16", seed=6)
    plan = b.plan(va)
    _, lse = b.run(va, plan)
    w = torch.zeros(1, 1, 3000, device="cuda")
    first = b.weigh(va, plan, lse, w).clone()
    assert abs(first.double().sum().item() - 3000 * 16) < 3000 * 16 * 2.0 ** -13
    for _ in range(5):
        w.zero_()
        assert torch.equal(b.weigh(va, plan, lse, w), first)


# ------------------------------------------------------------------ eviction


def evict_both(va, B, Hkv, D, kv, lens, keep, slots, seed, ties=False, pos=True, sinks=0, recent=None, ref=None, mutate=None):
    rng = np.random.default_rng(seed)
    blocks = [(n + 15) // 16 for n in lens]
    P = sum(blocks) + 2
    table = np.full((B, max(blocks) + 1), -1, np.int32)
    order = rng.permutation(P).astype(np.int32)
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    if mutate:
        mutate(table)
    kp, ks = make_pool(seed, P, Hkv, D, kv)
    vp, vs = make_pool(seed + 1, P, Hkv, D, kv)
    w = rng.choice([0.0, -0.0, 0.25, 1.0, np.nan, np.inf, -np.inf, -3.0], (B, Hkv, slots)) if ties else rng.exponential(1.0, (B, Hkv, slots))
    w = w.astype(np.float32)
    sp = np.stack([[rng.permutation(slots) for _ in range(Hkv)] for _ in range(B)]).astype(np.int32) if pos else None
    lens, keep = np.array(lens, np.int32), np.array(keep, np.int32)
    gpu = [kp, vp, ks, vs]
    host = [None if t is None else (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy().copy() for t in gpu]
    wd, pd, flags = cuda(w), None if sp is None else cuda(sp), torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = lambda x: None if x is None else cuda(np.asarray(x, np.int32))  # noqa: E731
    got = va.verify_attn_evict(kp, vp, ks, vs, i32(table), i32(lens), wd, i32(keep), kv, slot_pos=pd, num_sinks=sinks,
                               recent_from=i32(recent), ref_count=i32(None if ref is None else ref(table, P)), flags=flags)
    new, f = chunks.evict([x for x in host if x is not None], table, lens, w, keep, sp, sinks, recent,
                          None if ref is None else ref(table, P), P)
    assert got.tolist() == new.tolist() and flags.item() == f
    for x, y in zip(gpu, host):
        if x is not None:
            x = x.view(torch.int16) if x.dtype == torch.bfloat16 else x
            assert np.array_equal(x.cpu().numpy(), y)
    assert np.array_equal(wd.cpu().numpy(), w, equal_nan=True) and (sp is None or np.array_equal(pd.cpu().numpy(), sp))
    return got, flags


@pytest.mark.parametrize("kv", KINDS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ties", [False, True])
def test_evict(va, kv, D, ties):
    evict_both(va, 5, 3, D, kv, [100, 33, 1, 17, 64], [50, 32, 0, 40, -1], 130, 1, ties=ties, sinks=4, recent=[80, 10, 0, 3, 9])


@pytest.mark.parametrize("L,keep", [(1, 0), (2, 1), (16, 15), (17, 16), (513, 512), (2000, 1), (2000, 1999), (5000, 2500),
                                    (9000, 100), (40_000, 20_000), (40_001, 39_990)])
@pytest.mark.parametrize("ties", [False, True])
def test_evict_lengths(va, L, keep, ties):
    evict_both(va, 1, 2, 64, "int8", [L], [keep], L, L + keep, ties=ties, pos=False, sinks=2, recent=[L - 3])


def test_evict_more_slots_than_shared_memory_holds(va):
    evict_both(va, 1, 1, 64, "int2", [400_000], [150_000], 400_003, 11, sinks=3)
    evict_both(va, 1, 1, 64, "int2", [400_000], [399_000], 400_000, 12, ties=True)


def test_evict_more_protected_than_kept_all_equal_and_nothing_to_do(va):
    evict_both(va, 2, 2, 64, "bf16", [90, 70], [20, 30], 90, 3, sinks=200)                # everything is protected
    evict_both(va, 2, 2, 64, "bf16", [90, 70], [20, 30], 90, 4, recent=[-5, 0])
    evict_both(va, 3, 2, 64, "int4", [90, 70, 16], [90, 71, 10 ** 9], 90, 5)              # nothing goes
    evict_both(va, 3, 2, 64, "int4", [90, 70, 16], [0, 0, 0], 90, 6, ties=True)           # everything goes


def test_evict_refuses_what_it_must_not_move(va):
    def shared(table, P):
        ref = np.ones(P, np.int32)
        ref[table[1, 2]] = 2
        return ref
    got, flags = evict_both(va, 3, 2, 64, "int8", [90, 70, 40], [20, 30, 10], 96, 7, ref=shared)
    assert got.tolist() == [20, 70, 10] and flags.item() == va.VA_PAGES_BAD_REQUEST

    def broken(table):
        table[0, 3], table[2, 1] = 10 ** 6, -4
    got, flags = evict_both(va, 3, 2, 64, "int8", [90, 70, 40], [20, 30, 10], 96, 8, mutate=broken)
    assert got.tolist() == [90, 30, 40] and flags.item() == va.VA_PAGES_BAD_ENTRY
    # lengths that there are no weights or no table entries for
    kp, ks = make_pool(1, 4, 1, 64, "int8")
    before = kp.clone()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    flags = i32(0)
    got = va.verify_attn_evict(kp, kp.clone(), ks, ks.clone(), i32(0, 1, 2, 3).view(2, 2), i32(31, 33), torch.zeros(2, 1, 30, device="cuda"),
                               i32(4, 4), "int8", flags=flags)
    assert got.tolist() == [31, 33] and flags.item() == va.VA_PAGES_BAD_REQUEST and torch.equal(kp, before)


def test_evict_argument_errors(va):
    kp, ks = make_pool(1, 4, 2, 64, "int8")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    w = torch.zeros(2, 2, 32, device="cuda")
    good = dict(k_pages=kp, v_pages=kp.clone(), k_scale=ks, v_scale=ks.clone(), block_table=i32(0, 1, 2, 3).view(2, 2), seq_lens=i32(32, 20),
                weights=w, keep_lens=i32(4, 4), kv_dtype="int8")
    for change in (dict(k_pages=kp.float()), dict(v_pages=kp[:3]), dict(k_scale=None), dict(v_scale=ks[:3]), dict(seq_lens=i32(32)),
                   dict(block_table=i32(0, 1, 2)), dict(weights=w[:, :1]), dict(weights=w.half()), dict(keep_lens=i32(4)),
                   dict(slot_pos=w), dict(slot_pos=torch.zeros(2, 2, 33, dtype=torch.int32, device="cuda")), dict(recent_from=i32(1)),
                   dict(ref_count=i32(1, 1)), dict(new_lens=i32(1)), dict(flags=w), dict(num_pages=5)):
        with pytest.raises(ValueError):
            va.verify_attn_evict(**dict(good, **change))
    with pytest.raises(va.VerifyAttnError):
        va.verify_attn_evict(**dict(good, num_sinks=-1))


# ------------------------------------------------------------------ log probabilities


def check_logprobs(va, z, t, top):
    """Z' is a sum of V terms exp(d), each off by 2^-22 and 2^-23 |d| of itself (|d| <= 104, then it is 0), added at most
    2^10 in a row: 2^-13 of itself.  log1p and the subtractions: 2^-22 of their results and of x - M.  What is below
    binary32's smallest normal number, 2^-126, may be 0: a term exp(d) below it has |d| exp(d) < 2^-126 * 88 (x exp(-x)
    falls from there on), so V < 2^19 of them are worth less than 2^-126 * 2^7 * 2^19 = 2^-100."""
    got = va.verify_attn_logprobs(z, t, top)
    lp, ranks, ent, tt, tl, parts = chunks.logprobs(z.float().cpu().numpy(), t.cpu().numpy(), top)
    assert got[1].tolist() == ranks.tolist()
    assert np.array_equal(got[3].cpu().numpy(), tt)
    Z, S = parts[:, 0], parts[:, 1]
    moved = 2.0 ** -13 * Z / (1 + Z)

    def close(x, y, more):
        x = x.double().cpu().numpy()
        assert np.array_equal(np.isnan(x), np.isnan(y)) and np.array_equal(np.isneginf(x), np.isneginf(y))
        ok = np.isfinite(y)
        with np.errstate(invalid="ignore"):
            bad = np.abs(x - y) > more + 2.0 ** -100
        assert not bad[ok].any(), (np.abs(x - y)[ok & bad].max())
    with np.errstate(invalid="ignore"):
        close(got[0], lp, moved + 2.0 ** -21 * np.abs(lp))
        close(got[2], ent, moved + 2.0 ** -13 * (np.abs(S) + Z) / (1 + Z) + 2.0 ** -21 * np.abs(ent))
        close(got[4], tl, moved[:, None] + 2.0 ** -21 * np.abs(tl))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N,V,top", [(1, 1, 1), (3, 2, 2), (2, 31, 31), (5, 500, 32), (2, 4097, 5), (17, 9000, 20), (300, 1031, 3),
                                     (1, 40_000, 32), (4, 33_333, 1), (400, 12_000, 0)])
def test_logprobs(va, dtype, N, V, top):
    z = (normal(N + V, N, V) * 3).to(dtype)
    t = torch.randint(0, V, (N,), generator=torch.Generator().manual_seed(V), dtype=torch.int32).cuda()
    z[0, t[0].item()] += 30  # a likely one
    check_logprobs(va, z, t, top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("offset,pad", [(1, 3), (3, 0), (0, 5), (7, 64)])
def test_logprobs_rows_as_they_lie(va, dtype, offset, pad):
    N, V = 6, 5003
    room = (normal(3, N * (V + pad) + 16) * 3).to(dtype)
    z = torch.as_strided(room, (N, V), (V + pad, 1), offset)
    check_logprobs(va, z, torch.arange(N, dtype=torch.int32, device="cuda") * 1000, 20)
    same = torch.as_strided(room, (N, V), (0, 1), offset)  # one row for all tokens
    check_logprobs(va, same, torch.arange(N, dtype=torch.int32, device="cuda") * 1000, 2)


@pytest.mark.parametrize("N", [1, 400])
def test_logprobs_special_rows(va, N):
    V, K = 20_000, 20
    inf, nan = float("inf"), float("nan")
    base = normal(9, V) * 2
    rows = [torch.full((V,), -inf), torch.zeros(V), base.cpu().clone(), torch.arange(V).flip(0).float() * 1e-3,
            torch.arange(V).float() * 1e-3, base.cpu().clone(), base.cpu().clone(), torch.full((V,), torch.finfo(torch.float32).min),
            base.cpu().clone(), torch.full((V,), nan), base.cpu().clone(), torch.where(torch.arange(V) % 2 == 0, 0.0, -0.0)]
    rows[2][5:] = -inf
    rows[5][77] = nan
    rows[6][9] = inf
    rows[8][:] = -1e30
    rows[8][19_999] = 3.0
    rows[10][::2] = -inf
    rows[10][19_997] = nan
    for i, row in enumerate(rows):
        z = row.cuda().expand(N, V).contiguous() if N > 1 else row[None].cuda()
        for token in (3, 78, V - 1, -1, V):
            t = torch.full((1,), token, dtype=torch.int32).cuda()
            if N == 1:
                check_logprobs(va, z, t, K)
            elif token == 78:  # the same row in a batch of many
                one = va.verify_attn_logprobs(z[:1], t, K)
                many = va.verify_attn_logprobs(z, t.expand(N).contiguous(), K)
                assert torch.equal(many[1], one[1].expand(N)) and torch.equal(many[3], one[3].expand(N, K)), i
                assert torch.allclose(many[0], one[0].expand(N), rtol=1e-5, atol=1e-5, equal_nan=True)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_logprobs_of_more_rows_than_ctas_and_of_several_chunks(va, dtype):
    N, V = 1000, 17_003
    z = (normal(5, N, V) * 3).to(dtype)
    t = torch.randint(-1, V + 1, (N,), generator=torch.Generator().manual_seed(6), dtype=torch.int32).cuda()
    got = va.verify_attn_logprobs(z, t, 3)
    some = list(range(0, N, 97)) + [N - 1]
    check_logprobs(va, z[some].contiguous(), t[some].contiguous(), 3)
    one = [va.verify_attn_logprobs(z[i:i + 1], t[i:i + 1], 3) for i in range(N)]  # by a cluster each
    for k in (1, 3):
        assert torch.equal(got[k], torch.cat([x[k] for x in one]))
    for k in (0, 2, 4):  # each within 2^-13 Z' / (1 + Z') + 2^-21 |x|, the entropy 2^-13 (|S| + Z') / (1 + Z'), |S| < 16 Z'
        x, y = got[k], torch.cat([x[k] for x in one])
        assert torch.equal(x.isinf(), y.isinf())
        assert ((x - y).nan_to_num(0.0).abs() <= 2.0 ** -12 * (17 if k == 2 else 1) + 2.0 ** -20 * y.nan_to_num(0, 0, 0).abs()).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("N", [1, 500])
def test_logprobs_of_large_and_masked_values(va, dtype, N):
    """Around the size from which a row is taken entry by entry, with parts of a row on either side of it."""
    V = 20_000
    base = normal(8, V).cpu() * 2
    low = torch.finfo(dtype).min
    rows = [base + x for x in (4090.0, 4100.0, -4090.0, -4100.0, 20_000.0, -20_000.0, 60_000.0, -60_000.0)] + [base * 500, base * 8000]
    if dtype != torch.float16:
        rows += [base + 1e30, base - 1e30, base * 1e30, base * 1e37]
    for at, x in ((0, -5000.0), (9_000, -17_000.0), (15_000, low), (19_000, -float("inf"))):
        masked = torch.full((V,), x)
        masked[at:at + 300] = base[:300]
        rows.append(masked)
        part = base.clone()
        part[at:at + 4000] = x
        rows.append(part)
        last = torch.full((V,), x)
        last[V - 2] = -4000.0
        rows.append(last)
    for row in rows:
        z = row.to(dtype)[None].cuda()
        for token in (1, 9_050, V - 2):
            t = torch.full((1,), token, dtype=torch.int32).cuda()
            check_logprobs(va, z, t, 20)
            if N > 1 and token == 1:  # and by one CTA a row
                one = va.verify_attn_logprobs(z, t, 20)
                many = va.verify_attn_logprobs(z.expand(N, V), t.expand(N).contiguous(), 20)
                assert torch.equal(many[1], one[1].expand(N)) and torch.equal(many[3], one[3].expand(N, 20))
                for k in (0, 2, 4):
                    assert torch.allclose(many[k], one[k].expand(many[k].shape), rtol=2.0 ** -12, atol=2.0 ** -9, equal_nan=True)


@pytest.mark.parametrize("dtype,n", [(torch.float32, 4), (torch.bfloat16, 8), (torch.float16, 8)])
def test_logprobs_alternatives_among_many_equal_entries(va, dtype, n):
    """Ties with the threshold past every list: masks but for a few entries, and entries above it that one lane of each warp
    has, more than the list holds, and NaN at a row's start."""
    V, K = 60_000, 20
    i = torch.arange(V)
    rows = [torch.zeros(V), torch.full((V,), -float("inf")), torch.full((V,), torch.finfo(dtype).min),
            torch.where(i // n % 32 == 0, 1.0 + (i * 7919 % V) / V, 0.0), torch.zeros(V)]
    for row, at in ((0, 59_999), (1, 30_000), (2, 700)):
        rows[row][at], rows[row][at // 2] = 2.0, 3.0
    rows[4][:3000] = float("nan")
    rows[4][40_000] = 1.0
    for row in rows:
        z = row.to(dtype)[None].cuda()
        t = torch.full((1,), 40_000, dtype=torch.int32).cuda()
        check_logprobs(va, z, t, K)
        many = va.verify_attn_logprobs(z.expand(300, V), t.expand(300).contiguous(), K)  # one CTA a row
        one = va.verify_attn_logprobs(z, t, K)
        assert torch.equal(many[3], one[3].expand(300, K)) and torch.equal(many[1], one[1].expand(300))


def test_logprobs_past_32_bits_and_argument_errors(va):
    N, V = 9, 300_000_000
    z = torch.zeros(N, V, dtype=torch.bfloat16, device="cuda")
    z[:, -1] = 20
    z[8, 5] = 30
    lp, rk, en, tt, _ = va.verify_attn_logprobs(z, torch.full((N,), V - 1, dtype=torch.int32, device="cuda"), 2)
    assert rk.tolist() == [0] * 8 + [1] and tt.tolist() == [[V - 1, 0]] * 8 + [[5, V - 1]]
    want = -np.log1p((V - 1) * np.exp(-20.0))
    assert abs(lp[0].item() - want) < 2.0 ** -10 * abs(want)  # 2^18 additions in a row at most, by 2^-24, and the terms' 2^-17
    del z
    z = torch.zeros(3, 50, device="cuda")
    t = torch.zeros(3, dtype=torch.int32, device="cuda")
    for args in ((z.double(), t), (z.t(), t), (z[0], t), (z, t[:2]), (z, t.long()), (z, t, 33), (z, t, -1), (z[:, :4], t, 5),
                 (z.clone().requires_grad_(), t)):
        with pytest.raises(ValueError):
            va.verify_attn_logprobs(*args)
    empty = va.verify_attn_logprobs(z[:0], t[:0], 5)
    assert [tuple(x.shape) for x in empty] == [(0,), (0,), (0,), (0, 5), (0, 5)]


# ------------------------------------------------------------------ streams, graphs, together


class Step:
    """Chunks, their weights, a cut and log probabilities, on buffers that stay."""

    def __init__(self, va, kv="int8", seed=0):
        self.va = va
        self.b = Batch([30, 1, 64], [300, 90, 64], 8, 2, 128, kv, seed=seed)
        self.plan = self.b.plan(va)
        self.out, self.lse = torch.zeros_like(self.b.q), torch.zeros(self.b.N, 8, device="cuda")
        self.w = normal(seed + 9, 3, 2, 300).abs()
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
        self.lens, self.keep, self.new_lens = i32(300, 90, 64), i32(100, 50, 60), i32(0, 0, 0)
        self.z = normal(seed + 10, self.b.N, 3001)
        self.t = torch.arange(self.b.N, dtype=torch.int32, device="cuda")
        self.lp = None

    def run(self, stream=None):
        b = self.b
        b.run(self.va, self.plan, out=self.out, lse=self.lse, stream=stream)
        b.weigh(self.va, self.plan, self.lse, self.w, stream=stream)
        self.lp = self.va.verify_attn_logprobs(self.z, self.t, 5, stream=stream)
        self.va.verify_attn_evict(b.kp, b.vp, b.ks, b.vs, b.bt, self.lens, self.w, self.keep, b.kv, new_lens=self.new_lens,
                                  num_sinks=2, stream=stream)

    def state(self):
        torch.cuda.synchronize()
        b = self.b
        return [x.clone() for x in (self.out, self.lse, self.w, self.new_lens, b.kp, b.vp, *self.lp)]


@pytest.mark.parametrize("kv", ["int8", "bf16"])
def test_calls_on_a_side_stream_and_captured_are_the_eager_ones(va, kv):
    eager, side, raw, graph = (Step(va, kv) for _ in range(4))
    for _ in range(3):
        eager.run()
    want = eager.state()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        side.run(stream=s)
        raw.run(stream=s.cuda_stream)
    for step in (side, raw):
        for x, y in zip(step.state(), want):
            assert torch.equal(x, y)
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]  # two of them over one plan, one after the other
    for g in graphs:
        with torch.cuda.graph(g):
            graph.run()
    for i in range(3):
        graphs[i % 2].replay()
    for x, y in zip(graph.state()[:6], want[:6]):
        assert torch.equal(x, y)


def test_two_batches_at_once_on_two_streams_and_from_fresh_threads(va):
    steps = [Step(va, "int8", seed=40), Step(va, "bf16", seed=41)]
    alone = []
    for kv, seed in (("int8", 40), ("bf16", 41)):
        x = Step(va, kv, seed=seed)
        for _ in range(4):
            x.run()
        alone.append(x.state())
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    errors = []

    def work(step, stream):
        try:
            for _ in range(4):
                step.run(stream=stream)
        except Exception as e:  # pragma: no cover
            errors.append(e)
    threads = [threading.Thread(target=work, args=x) for x in zip(steps, streams)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    for step, want in zip(steps, alone):
        for x, y in zip(step.state(), want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("kv", ["int8", "bf16"])
def test_a_prompt_in_chunks(va, kv):
    """A prompt of 90 tokens in three chunks beside a request that adds one token a step: pages, rotary append,
    attention, weights; then both are cut, pages go back, and a verify block runs over what is left."""
    Hq, Hkv, D, P = 8, 2, 64, 40
    pools = [make_pool(i, P, Hkv, D, kv) for i in range(2)]
    (kp, ks), (vp, vs) = pools
    buffers = [x for p in pools for x in p if x is not None]
    pool = va.PagePool.create(P, 2, 10, buffers)
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    rope = va.verify_attn_rope_spec(D)
    w = torch.zeros(2, Hkv, 160, device="cuda")
    pos = torch.zeros(2, Hkv, 160, dtype=torch.int32, device="cuda")
    lens, seen = [0, 0], [0, 0]

    def add(new, seed, check=True):
        """new tokens of both requests through one layer."""
        for b in range(2):
            lens[b] += new[b]
        va.verify_attn_pages_resize(pool, i32(*lens))
        x = normal(seed, sum(new), Hq + 2 * Hkv, D, dtype=torch.bfloat16)
        q = torch.empty(sum(new), Hq, D, dtype=torch.bfloat16, device="cuda")
        positions = torch.cat([torch.arange(seen[b], seen[b] + new[b], dtype=torch.int32) for b in range(2)]).cuda()
        at = 0
        for b in range(2):  # chunks of different lengths: one append each
            part = x[None, at:at + new[b]]
            q[at:at + new[b]] = va.verify_attn_rope_append(
                rope, positions[None, None, at:at + new[b]], part[:, :, :Hq], part[:, :, Hq:Hq + Hkv], part[:, :, Hq + Hkv:], kp, vp,
                ks, vs, pool.block_table[b:b + 1], pool.seq_lens[b:b + 1], kv)[0]
            at += new[b]
            seen[b] += new[b]
        batch = Batch.__new__(Batch)
        batch.new, batch.lens, batch.Hq, batch.Hkv, batch.D, batch.kv, batch.N = new, list(lens), Hq, Hkv, D, kv, sum(new)
        batch.kp, batch.vp, batch.ks, batch.vs, batch.q, batch.bt = kp, vp, ks, vs, q, pool.block_table
        batch.table = pool.block_table.cpu().numpy()
        plan = batch.plan(va)
        out, lse = batch.run(va, plan)
        batch.check(out, lse)
        old = w.clone()
        batch.weigh(va, plan, lse, w, slot_pos=pos, positions=positions)
        check_weights(batch, w, lse, old)
        assert va.verify_attn_chunk_plan_device_flags(plan) == 0
        return out
    add([31, 20], 1)
    add([40, 1], 2)
    out = add([19, 1], 3)
    assert lens == [90, 22] and pos[0, 0, :90].tolist() == list(range(90))
    logits = (out.flatten(1).float() @ normal(5, Hq * D, 700)).bfloat16()
    check_logprobs(va, logits, torch.arange(20, dtype=torch.int32, device="cuda"), 5)
    # cut both to what they may hold, in a layer whose heads choose for themselves
    table = pool.block_table.cpu().numpy()
    bits = lambda t: (t.view(torch.int16) if t.dtype == torch.bfloat16 else t).cpu().numpy().copy()  # noqa: E731
    host, hw, hp = [bits(x) for x in buffers], w.cpu().numpy().copy(), pos.cpu().numpy().copy()
    new_lens = va.verify_attn_evict(kp, vp, ks, vs, pool.block_table, pool.seq_lens, w, i32(40, 40), kv, slot_pos=pos, num_sinks=2,
                                    recent_from=i32(80, 0), ref_count=pool.ref_count, flags=pool.flags)
    want, _ = chunks.evict(host, table, [90, 22], hw, [40, 40], hp, 2, [80, 0], pool.ref_count.cpu().numpy(), P)
    assert new_lens.tolist() == want.tolist() == [40, 22]
    for x, y in zip(buffers, host):
        assert np.array_equal(bits(x), y)
    assert np.array_equal(w.cpu().numpy(), hw) and np.array_equal(pos.cpu().numpy(), hp)
    assert set(range(80, 90)) | {0, 1} <= set(hp[0, 1, :40].tolist())  # protected
    free = pool.num_free.item()
    va.verify_attn_pages_resize(pool, new_lens)
    assert pool.num_free.item() == free + 3 and va.verify_attn_pages_flags(pool) == 0
    lens[:] = [40, 22]
    add([5, 5], 6)  # a block over the cut cache, positions going on
    assert seen == [95, 27] and pos[0, 1, 40:45].tolist() == list(range(90, 95))
    # and the verify step's own attention over the same cache
    T, q = 5, normal(8, 10, Hq, D, dtype=torch.bfloat16)
    vplan = va.verify_attn_plan([45, 27], T, Hq, Hkv, D, kv, block_table_stride=10, num_pages=P)
    vout, vlse = torch.empty_like(q), torch.empty(10, Hq, device="cuda")
    va.verify_attn_with_plan(vplan, q, kp, vp, ks, vs, pool.block_table, pool.seq_lens, T, vout, vlse)
    cplan = va.verify_attn_chunk_plan([T, T], [45, 27], Hq, Hkv, D, kv)
    out, lse = va.verify_attn_chunk(cplan, q, kp, vp, ks, vs, pool.block_table)
    assert (out.float() - vout.float()).abs().max() < 2.0 ** -6 * out.float().abs().max() and (lse - vlse).abs().max() < 1e-4
