"""Host: refusals and empty calls of the operators of a prompt worked in chunks, beside those of ``test_chunk_host``."""
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
