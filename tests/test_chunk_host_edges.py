"""Host: refusals and empty calls of the operators of a prompt worked in chunks, beside those of ``test_chunk_host``."""
import numpy as np
import pytest

import speculative_decoding_verify_causal_gb300 as va
from speculative_decoding_verify_causal_gb300 import build as vbuild

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    vbuild.build()


def test_outputs_and_moved_tensors_that_require_a_gradient_are_refused():
    x, w = torch.zeros(2, 8), torch.zeros(2, 8, requires_grad=True)
    t = torch.zeros(2, dtype=torch.int32)
    plan = va.ChunkPlan(None, (1, 8, 2, 64, 2, 2, 2), 0)
    calls = [lambda y: va.verify_attn_evict(y, x, x, x, t, t, x, t, "int8"), lambda y: va.verify_attn_evict(x, y, x, x, t, t, x, t, "int8"),
             lambda y: va.verify_attn_evict(x, x, y, x, t, t, x, t, "int8"), lambda y: va.verify_attn_evict(x, x, x, y, t, t, x, t, "int8"),
             lambda y: va.verify_attn_evict(x, x, x, x, t, t, y, t, "int8"),
             lambda y: va.verify_attn_chunk(plan, x, x, x, x, x, t, lse=y)]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call(w)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call(w)


def test_evict_workspace_of_more_slots_than_a_call_takes():
    size = va.library().verify_attn_evict_workspace_bytes
    assert size(1, 1, 2 ** 30) >= 2 ** 32 + 4 and size(1, 1, 2 ** 30 + 1) == size(1, 1, 2 ** 31 - 1) == 0


class Cuda(torch.Tensor):
    """A tensor that says it is on the current GPU: for checks that come before any address is used."""
    is_cuda = True
    device = torch.device("cuda", 0)

    def get_device(self):
        return 0


def on_gpu(*shape, dtype=torch.float32):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Cuda)


@pytest.mark.parametrize("wrong", [None, [0, 1], 3.0, torch.zeros(2)])
def test_arguments_that_are_no_gpu_tensors_are_refused_by_name(wrong):
    plan = va.ChunkPlan(None, (1, 8, 2, 64, 2, 2, 2), 0)
    i32 = torch.int32
    good = dict(plan=plan, q=on_gpu(2, 8, 64, dtype=torch.bfloat16), k_pages=on_gpu(3, 16, 2, 64, dtype=torch.int8), k_scale=on_gpu(3, 16, 2),
                block_table=on_gpu(1, 2, dtype=i32), lse=on_gpu(2, 8), weights=on_gpu(1, 2, 5), slot_pos=on_gpu(1, 2, 5, dtype=i32),
                positions=on_gpu(2, dtype=i32))
    for name in ("q", "k_pages", "k_scale", "block_table", "lse", "weights", "slot_pos", "positions"):
        if name == "slot_pos" and wrong is None:
            continue
        with pytest.raises(ValueError, match=name):
            va.verify_attn_chunk_weights(**dict(good, **{name: wrong}))
    pages, lens = good["k_pages"], on_gpu(1, dtype=i32)
    good = dict(k_pages=pages, v_pages=pages, k_scale=good["k_scale"], v_scale=good["k_scale"], block_table=good["block_table"],
                seq_lens=lens, weights=good["weights"], keep_lens=lens, kv_dtype="int8")
    for name in ("k_pages", "v_pages", "k_scale", "v_scale", "block_table", "seq_lens", "weights", "keep_lens"):
        with pytest.raises(ValueError, match=name):
            va.verify_attn_evict(**dict(good, **{name: wrong}))
    with pytest.raises(ValueError, match="tokens"):
        va.verify_attn_logprobs(on_gpu(2, 9), wrong)


def test_numbers_past_32_bits_are_refused_not_cut():
    """2^32 + 5 is 5 in its low 32 bits."""
    for far in (torch.tensor([2 ** 32 + 5]), [2 ** 32 + 5], torch.tensor([-2 ** 32 + 5])):
        for new, lens in ((far, [100]), ([5], far)):
            with pytest.raises((ValueError, OverflowError)):
                va.verify_attn_chunk_plan_describe(new, lens, 8, 2, 64, "int8", 152)
            with pytest.raises((ValueError, OverflowError)):
                va.verify_attn_chunk_plan(new, lens, 8, 2, 64, "int8")
        with pytest.raises((ValueError, OverflowError)):
            va.verify_attn_plan_describe(far, 4, 8, 2, 64, "int8", 152)
    assert va.verify_attn_chunk_plan_describe(torch.tensor([5]), torch.tensor([100]), 8, 2, 64, "int8", 152)[0]["num_tokens"] == 5
    pages, lens = on_gpu(3, 16, 2, 64, dtype=torch.bfloat16), on_gpu(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="num_sinks"):
        va.verify_attn_evict(pages, pages, None, None, on_gpu(1, 2, dtype=torch.int32), lens, on_gpu(1, 2, 5), lens, "bf16",
                             num_sinks=2 ** 32)


def test_a_block_table_of_another_width_than_the_plan_is_refused():
    """The kernels step through the table by the plan's stride: rows of another width are read from the wrong places."""
    bf, i32 = torch.bfloat16, torch.int32
    q, pages, lens = on_gpu(2, 4, 8, 64, dtype=bf), on_gpu(9, 16, 2, 64, dtype=bf), on_gpu(2, dtype=i32)
    plan = va.Plan(None, np.array([40, 100], np.int32), 4, 0)
    assert plan.block_table_stride == 7
    assert va.Plan(None, np.array([40, 100], np.int32), 4, 0, 12).block_table_stride == 12
    for table in (on_gpu(2, 8, dtype=i32), on_gpu(2, 6, dtype=i32), on_gpu(1, 7, dtype=i32)):
        with pytest.raises(ValueError, match="block_table.*7"):
            va.verify_attn_with_plan(plan, q, pages, pages, None, None, table, lens, 4, q)
        with pytest.raises(ValueError, match="block_table.*7"):
            va.verify_attn_noalloc([40, 100], 4, 8, 2, 64, "bf16", q, pages, pages, None, None, table, lens, q)
        with pytest.raises(ValueError, match="block_table.*9"):
            va.verify_attn_noalloc([40, 100], 4, 8, 2, 64, "bf16", q, pages, pages, None, None, table, lens, q, block_table_stride=9)
    one = va.Plan(None, np.array([40], np.int32), 4, 0)  # one sequence: a wider row is read no further than it has to be
    with pytest.raises(ValueError, match="block_table.*3"):
        va.verify_attn_with_plan(one, q[:1], pages, pages, None, None, on_gpu(1, 2, dtype=i32), lens, 4, q)
    for table in (on_gpu(1, 8, dtype=i32), on_gpu(1, 3, dtype=i32), on_gpu(5, dtype=i32)):
        with pytest.raises(va.VerifyAttnError):  # no handle: past the check
            va.verify_attn_with_plan(one, q[:1], pages, pages, None, None, table, lens, 4, q, stream=0)
