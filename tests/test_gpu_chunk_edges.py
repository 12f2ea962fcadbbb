"""GPU: ends of the ranges of the operators of a prompt worked in chunks.  Definitions, tolerances and helpers are those of
``test_gpu_chunk``."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_chunk import Batch, check_rows, cuda, normal  # noqa: E402

MOST = {"fp8_e4m3": 448.0, "int8": 127.0, "int4": 7.0, "int2": 1.0}


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


def cells(b, s, first=0, last=None):
    """Pages and slots of the keys [first, last) of sequence s."""
    j = torch.arange(first, b.lens[s] if last is None else last)
    return torch.from_numpy(b.table)[s][j // 16].long().cuda(), (j % 16).cuda()


def ones(b, pages, at):
    """The largest code in an element or all of a row."""
    code = {"fp8_e4m3": 0x7E, "int8": 127, "int4": 7, "int2": 1}[b.kv]
    if at is not None:
        pages[(*at, slice(None), 0)] = code  # of the packed types the first element of the row's first byte
    return {"int4": 0x77, "int2": 0x55}.get(b.kv, code)


def score_of_keys(b, s, first, value):
    """Keys of sequence s from `first` on: zero but for element 0, whose product with q (also zero but there) makes the
    softmax's exponent, in powers of two, `value` at q[0] = sqrt(D); the keys before them: all zero."""
    b.kp[cells(b, s)] = 0
    b.ks[cells(b, s)] = 1.0
    ones(b, b.kp, cells(b, s, first))
    b.ks[cells(b, s, first)] = value * np.log(2.0) / MOST[b.kv]
    b.q.zero_()
    b.q[..., 0] = b.D ** 0.5


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8", "int4", "int2"])
def test_chunk_sums_of_the_smallest_value_scales(va, kv, D):
    """Value scales near 2^-118 with scores just under the step at which the running maximum moves: probabilities of nearly
    2^8 against it, times the largest power of two that the scales are brought up by."""
    b = Batch([20, 3], [700, 250], 8, 2, D, kv, seed=31, v_std=2.0 ** -118 * MOST[kv] / 3)
    for s in range(2):
        score_of_keys(b, s, 80, 7.75)
    plan = b.plan(va, num_sms=1)  # keys not split: the first tile sets the maximum
    assert plan.info()["num_split_groups"] == 0
    out, lse = b.run(va, plan)
    assert (out != 0).any(-1).all()
    b.check(out, lse)


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8", "int4", "int2"])
@pytest.mark.parametrize("scale", [2.0 ** 79, 2.0 ** 85, 2.0 ** 103])
def test_chunk_of_the_largest_value_scales(va, kv, scale):
    for D in (64, 256):
        b = Batch([20, 3], [700, 250], 8, 2, D, kv, seed=35, v_std=scale * MOST[kv] / 4)
        for s in range(2):
            score_of_keys(b, s, 80, 7.75)
        b.check(*b.run(va, b.plan(va, num_sms=1)))


def verify(va, b, path="mma"):
    """The verify step on a batch whose chunks are of one length: (out, lse)."""
    plan = va.verify_attn_plan(b.lens, b.new[0], b.Hq, b.Hkv, b.D, b.kv, num_sms=1, path=path, block_table_stride=b.bt.shape[1])
    out, lse = torch.empty_like(b.q), torch.empty(b.N, b.Hq, device="cuda")
    va.verify_attn_with_plan(plan, b.q, b.kp, b.vp, b.ks, b.vs, b.bt, cuda(np.array(b.lens, np.int32)), b.new[0], out, lse)
    return out, lse


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8", "int4", "int2"])
def test_verify_sums_of_the_smallest_value_scales(va, kv, D):
    b = Batch([16, 16], [700, 250], 8, 2, D, kv, seed=32, v_std=2.0 ** -118 * MOST[kv] / 3)
    for s in range(2):
        score_of_keys(b, s, 80, 7.75)
    ref, ref_lse, size, reach = b.want()
    out, lse = verify(va, b)
    check_rows(kv, D, out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, ref_lse, size, reach)


def values_of_two_sizes(kv, D, where, large, step, seed):
    """Values of `large` but for the keys of `where`, which have value scales of 2^-118 and scores larger by `step` powers of
    two."""
    b = Batch([16], [4200], 4, 1, D, kv, seed=seed)
    score_of_keys(b, 0, 4200, 0.0)
    b.vp[:] = ones(b, b.vp, None)
    b.vs[:] = large / MOST[kv]
    at = cells(b, 0, *where)
    b.vs[at] = 2.0 ** -118
    if step:
        ones(b, b.kp, at)
        b.ks[at] = step * np.log(2.0) / MOST[kv]
    return b


# Nearly 4,000 keys make a sum of as many times the codes; then come more than a tile of either kernel's tiny values, which
# are next to nothing beside the others (0), or all that counts (250), or not of fp16's reach from them (60: a key of a
# probability of 2^-60 has no part, however large its value; the bound's second part).
SIZES = [((3840, 4000), (3840, 4200), (0, 160), (3840, 4160), (0, 320)), [0.0, 60.0, 250.0], [1.0, 2.0 ** 20]]


def check_two_sizes(b, out, lse, where, step, tile):
    """The bound's second part is for keys whose products are small beside the largest value scale of their own tile of
    keys.  Where a tile has one value scale (both ends of the tiny values at tiles' ends), those are keys of p < 2^-8 of the
    likeliest only: of the steps 0 and 250 there are none, or such ones as are worth 2^-250 of the others.  So there the
    bound has its first part alone."""
    ref, ref_lse, (size, small), reach = b.want()
    one_scale = all(end % tile == 0 or end == b.lens[0] for end in where)
    check_rows(b.kv, b.D, out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, ref_lse,
               (size, 0 * small if one_scale and step != 60 else small), reach)


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8", "int4", "int2"])
@pytest.mark.parametrize("step", SIZES[1])
@pytest.mark.parametrize("large", SIZES[2])
def test_chunk_tiles_of_tiny_values_among_ordinary_ones(va, kv, step, large):
    for D in (64, 256):
        for where in SIZES[0]:
            b = values_of_two_sizes(kv, D, where, large, step, 33)
            check_two_sizes(b, *b.run(va, b.plan(va, num_sms=1)), where, step, 80)


@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8", "int4", "int2"])
@pytest.mark.parametrize("step", SIZES[1])
@pytest.mark.parametrize("large", SIZES[2])
def test_verify_tiles_of_tiny_values_among_ordinary_ones(va, kv, step, large):
    for D in (64, 256):
        for where in SIZES[0]:
            b = values_of_two_sizes(kv, D, where, large, step, 34)
            check_two_sizes(b, *verify(va, b), where, step, 64)

def with_loads_withheld(rank, where):
    """The library with log probabilities in which the CTAs of one rank of a cluster get the first chunk of their first row only:
    their next wait runs out after 5 ms."""
    from speculative_decoding_verify_causal_gb300 import build
    src, obj, out = os.path.join(build.CSRC, "va_logprobs.cu"), str(where / f"l{rank}.o"), str(where / f"l{rank}.so")
    subprocess.run([build._nvcc(), *build.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", f"-DVA_LOGPROBS_WITHHELD={rank}",
                    "-DVA_LOGPROBS_WAIT_NS=5000000ull", "-I", build.INCLUDE, "-I", build.CSRC, "-c", src, "-o", obj], check=True)
    others = [os.path.join(build.BUILD_DIR, f) for f in os.listdir(build.BUILD_DIR)
              if f.endswith(".o") and f != "va_logprobs.cu.o"]
    subprocess.run([build._nvcc(), *build.ARCH, "-shared", "-cudart", "static", "-o", out, obj, *others], check=True)
    call = ctypes.CDLL(out).verify_attn_logprobs
    P, I = ctypes.c_void_p, ctypes.c_int
    call.argtypes, call.restype = [P, ctypes.c_int64, I, P, I, I, I, P, P, P, P, P, P], I
    return call


@pytest.mark.parametrize("rank", [0, 1, 7])
def test_logprobs_of_a_wait_that_ran_out(va, rank, tmp_path):
    """NaN, whichever CTA of a row's cluster it was; and in all further rows of the CTA."""
    call = with_loads_withheld(rank, tmp_path)
    for N, V in ((3, 70_000), (2, 9_000), (1000, 6_000)):  # clusters of 8 and 2; two rows and more a CTA
        x = normal(40, N, V)
        tokens = torch.arange(N, dtype=torch.int32, device="cuda")
        want = va.verify_attn_logprobs(x, tokens, 3)
        got = [torch.empty_like(t) for t in want]
        p = [t.data_ptr() for t in got]
        rc = call(x.data_ptr(), V, va.VA_FLOAT_FP32, tokens.data_ptr(), N, V, 3, *p, torch.cuda.current_stream().cuda_stream)
        torch.cuda.synchronize()
        assert rc == 0
        hit = rank < {3: 8, 2: 2, 1000: 1}[N]
        for i in (0, 2, 4):
            if hit:
                assert torch.isnan(got[i]).all(), (N, V, i)
            else:
                assert torch.equal(got[i], want[i]), (N, V, i)


@pytest.mark.parametrize("which", ["chunk", "verify"])
def test_a_plan_is_on_the_device_when_it_is_returned(va, which):
    """Nothing of it is under way on the legacy stream, which a side stream's first call does not wait for; on an idle
    and on a full GPU."""
    side, busy = torch.cuda.Stream(), normal(50, 4096, 4096)
    legacy = torch.cuda.default_stream()
    lib, code = va.library(), va.KV_DTYPE_CODES["int8"]
    for B, full in [(1, 0), (4, 0), (64, 0), (1, 4), (64, 4)] * 20:
        new, host = np.ones(B, np.int32), np.full(B, 3000, np.int32)
        with torch.cuda.stream(side):
            for _ in range(full):
                busy @ busy
        plan = ctypes.c_void_p()
        if which == "chunk":
            rc = lib.verify_attn_chunk_plan(new.ctypes.data, host.ctypes.data, B, 8, 8, 64, code, 0, ctypes.byref(plan))
        else:
            rc = lib.verify_attn_plan_ex(host.ctypes.data, B, 1, 8, 8, 64, code, 0, None, ctypes.byref(plan))
        done = legacy.query()
        assert rc == 0
        (lib.verify_attn_chunk_plan_destroy if which == "chunk" else lib.verify_attn_plan_destroy)(plan)
        assert done
    torch.cuda.synchronize()


@pytest.mark.parametrize("kv", ["bf16", "int8"])
def test_a_batch_without_new_tokens(va, kv):
    """Tensors without rows, which have no address; the outputs that the call makes."""
    b = Batch([0, 0, 0], [0, 30, 17], 4, 2, 64, kv, seed=51)
    plan = b.plan(va)
    assert b.q.shape == (0, 4, 64)
    out, lse = b.run(va, plan)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    w = torch.full((3, 2, 30), 2.0, device="cuda")
    pos = torch.full((3, 2, 30), 7, dtype=torch.int32, device="cuda")
    b.weigh(va, plan, lse, w, slot_pos=pos, positions=torch.empty(0, dtype=torch.int32, device="cuda"))
    b.weigh(va, plan, lse, torch.empty(3, 2, 0, device="cuda"))
    assert (w == 2).all() and (pos == 7).all() and va.verify_attn_chunk_plan_device_flags(plan) == 0


def test_evict_of_no_slots(va):
    """Sequences of no tokens, whose weights have no address; one that says otherwise is flagged."""
    kp, vp = (torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    lens, keep = cuda(np.array([0, 0, 5], np.int32)), cuda(np.array([0, 3, 2], np.int32))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    new = va.verify_attn_evict(kp, vp, None, None, table, lens, torch.empty(3, 2, 0, device="cuda"), keep, "bf16", flags=flags)
    assert new.tolist() == [0, 0, 5] and flags.item() == va.VA_PAGES_BAD_REQUEST
    assert (kp == 0).all() and (vp == 0).all()
