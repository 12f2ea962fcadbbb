"""GPU: ends of the ranges of the operators of a prompt worked in chunks.  Definitions, tolerances and helpers are those of
``test_gpu_chunk``."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_chunk import Batch, check_rows, cuda  # noqa: E402

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


def score_of_key(b, s, first, value):
    """Keys of sequence s from `first` on: zero but for element 0, whose product with q (also zero but there) makes the
    softmax's exponent, in powers of two, `value` at q[0] = sqrt(D); the keys before them: all zero."""
    most = MOST[b.kv]
    code = most if b.kv == "fp8_e4m3" else int(most)
    for j in range(b.lens[s]):
        page, slot = b.table[s, j // 16], j % 16
        b.kp[page, slot] = 0
        b.ks[page, slot] = 1.0
        if j >= first:
            if b.kv == "fp8_e4m3":
                b.kp.view(torch.float8_e4m3fn)[page, slot, :, 0] = code
            else:
                b.kp[page, slot, :, 0] = code  # of the packed types the low bits of the first byte
            b.ks[page, slot] = value * np.log(2.0) / code
    b.q.zero_()
    b.q[..., 0] = b.D ** 0.5


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv", ["fp8_e4m3", "int8", "int4", "int2"])
def test_chunk_sums_of_the_smallest_value_scales(va, kv, D):
    """Value scales near 2^-118 with scores just under the step at which the running maximum moves: probabilities of nearly
    2^8 against it, times the largest power of two that the scales are brought up by."""
    b = Batch([20, 3], [700, 250], 8, 2, D, kv, seed=31, v_std=2.0 ** -118 * MOST[kv] / 3)
    for s in range(2):
        score_of_key(b, s, 80, 7.75)
    plan = b.plan(va, num_sms=1)  # keys not split: the first tile sets the maximum
    assert plan.info()["num_split_groups"] == 0
    out, lse = b.run(va, plan)
    assert (out != 0).any(-1).all()
    b.check(out, lse)


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
        score_of_key(b, s, 80, 7.75)
    ref, ref_lse, size, reach = b.want()
    out, lse = verify(va, b)
    check_rows(kv, D, out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, ref_lse, size, reach)
