"""Calls on a stream that is not the current one: what a call allocates belongs to the stream it runs on."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


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


@pytest.mark.parametrize("raw", [False, True])
def test_acceptance_and_lookup_on_another_stream(va, raw):
    """Calls that wait behind other work on a side stream, while the current stream takes and fills memory of the sizes
    that they use: their workspace and outputs are not among it."""
    B, T, V = 64, 7, 4000
    g = torch.Generator().manual_seed(1)
    logits = torch.randn(B, T + 1, V, generator=g).cuda() * 3
    drafts = logits[:, :T].argmax(-1).int()
    drafts[::3, 4] = 5
    tau = torch.full((B,), 0.8, device="cuda")
    history = torch.randint(0, 6, (B, 600), generator=g, dtype=torch.int32).cuda()
    lens = torch.full((B,), 600, dtype=torch.int32, device="cuda")
    calls = (lambda s: va.verify_attn_accept(logits, drafts, tau, 17, stream=s),
             lambda s: va.verify_attn_lookup_draft(history, lens, 16, min_match=2, stream=s))
    want = [call(None) for call in calls]
    torch.cuda.synchronize()
    need = int(va.library().verify_attn_accept_workspace_bytes(B, T))
    big = torch.empty(2 ** 31, dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for call, expect in zip(calls, want):
        for _ in range(4):
            with torch.cuda.stream(side):
                for _ in range(6):
                    big.fill_(1)
            got = call(side.cuda_stream if raw else side)
            for n in (need, 4 * B, 4 * B * (T + 1), 64 * B):
                torch.zeros(n, dtype=torch.uint8, device="cuda")
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, expect))
