"""Calls on a stream that is not the current one: what a call allocates belongs to the stream it runs on.  Calls from host
threads that have called nothing else."""
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


@pytest.mark.parametrize("kv_dtype", ["int8", "fp8_e4m3"])
def test_attention_of_several_host_threads(va, kv_dtype):
    """Plans used by host threads that have called nothing of CUDA before, on streams of their own: every call is launched,
    and the results are those of one thread."""
    import threading
    from speculative_decoding_verify_causal_gb300 import workloads as wl
    jobs = []
    for i, Hkv in enumerate((1, 8, 1, 8)):
        w = wl.make_workload(i, [300, 77], 4, 4 * Hkv, Hkv, 256, kv_dtype)
        d = wl.to_device(w)
        plan = va.verify_attn_plan(w["seq_lens"], 4, 4 * Hkv, Hkv, 256, kv_dtype, path="mma", num_pages=w["num_pages"],
                                   block_table_stride=d["block_table"].shape[1])
        out, lse = torch.empty_like(d["q"]), torch.empty(2, 4, 4 * Hkv, device="cuda")
        rest = [d[n] for n in ("q", "k_pages", "v_pages", "k_scale", "v_scale", "block_table", "seq_lens")]
        va.verify_attn_with_plan(plan, *rest, 4, out, lse)
        torch.cuda.synchronize()
        jobs.append((plan, rest, out, lse, out.clone(), lse.clone(), torch.cuda.Stream()))
        out.zero_()
    torch.cuda.synchronize()
    call = va.library().verify_attn_with_plan
    codes, start = [set() for _ in jobs], threading.Barrier(len(jobs))

    def work(i):
        plan, rest, out, lse, _, _, stream = jobs[i]
        args = plan.handle, *(t.data_ptr() for t in rest), 4, out.data_ptr(), lse.data_ptr(), stream.cuda_stream
        start.wait()
        codes[i] = {call(*args) for _ in range(500)}

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(jobs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}] * len(jobs)
    for plan, _, out, lse, want_out, want_lse, _ in jobs:
        assert torch.equal(out, want_out) and torch.equal(lse, want_lse)
        plan.destroy()
