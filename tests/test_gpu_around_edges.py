"""Edges of the operators around the verify step on the GPU: forks whose sequences are cut back before they write,
host threads at once, a pool dropped early, the signs of zeros, frequencies above one,
gradients, q in place,
sizes past 32 bits, lengths past the block table."""
import numpy as np
import pytest

from oracle import around

from test_gpu_around import bits16, cache_case, check_pool, cuda, expected_cache, gpu_pool, normal, rope_bound, run_append

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


def i32(*v):
    return cuda(np.array(v, np.int32))


# ------------------------------------------------------------------ pages


@pytest.mark.parametrize("kept", [[20, 20], [20, 27], [3, 32], [16, 17], [31, 0]])
@pytest.mark.parametrize("calls", [1, 2])
def test_a_fork_made_before_the_drafts_were_decided_keeps_its_tokens(va, kept, calls):
    """32 tokens, 16 of them drafts, forked with their full pages shared; both sequences keep what was accepted, take
    pages for their next block and append it.  Each reads its own tokens afterwards."""
    T, Hkv, D = 16, 1, 64
    pages = torch.zeros(16, 16, Hkv, D, dtype=torch.bfloat16, device="cuda")
    values = torch.zeros_like(pages)
    pool = va.PagePool.create(16, 2, 4, [pages, values])
    spec = va.verify_attn_rope_spec(D)

    def append(seed):
        """T rows before each sequence's end, whole numbers: v is stored as it is."""
        v = torch.randint(1, 200, (2, T, Hkv, D), generator=torch.Generator().manual_seed(seed)).bfloat16().cuda()
        va.verify_attn_rope_append(spec, None, None, v, v, pages, values, None, None, pool.block_table, pool.seq_lens, "bf16")
        return v

    def read(b):
        n = int(pool.seq_lens[b])
        return torch.cat([values[p] for p in pool.block_table[b, :-(-n // 16)].tolist()])[:n]

    va.verify_attn_pages_resize(pool, i32(16, 0))
    first = append(1)[0]
    va.verify_attn_pages_resize(pool, i32(32, 0))
    second = append(2)[0]
    va.verify_attn_pages_fork(pool, i32(0), i32(1))
    old = torch.cat([first, second])
    assert torch.equal(read(0), old) and torch.equal(read(1), old)
    new = [n + T for n in kept]
    if calls == 1:
        va.verify_attn_pages_resize(pool, i32(*new), kept_lens=i32(*kept))
    else:
        va.verify_attn_pages_resize(pool, i32(*kept))
        va.verify_attn_pages_resize(pool, i32(*new))
    for b in (0, 1):
        assert torch.equal(read(b)[:kept[b]], old[:kept[b]])
    block = append(3)
    for b in (0, 1):
        assert torch.equal(read(b), torch.cat([old[:kept[b]], block[b]])), b
    assert va.verify_attn_pages_flags(pool) == 0


@pytest.mark.parametrize("seed,P,B,stride", [(0, 60, 7, 12), (1, 500, 45, 8), (2, 3000, 300, 20), (3, 40, 9, 6)])
def test_resize_with_kept_lengths(va, seed, P, B, stride):
    """Random steps, refused ones and exhausted lists among them, against the sequential definition after each."""
    rng = np.random.default_rng(seed)
    pool = around.Pages(P, B, stride, [rng.integers(0, 255, (P, 32)).astype(np.uint8)])
    pool.stack = rng.permutation(P)
    dev = gpu_pool(va, pool)
    for _ in range(40):
        if rng.random() < 0.4:
            n = max(1, B // 6)
            args = [rng.integers(0, B, n).astype(np.int32) for _ in range(2)]
            pool.fork(*args)
            va.verify_attn_pages_fork(dev, *map(cuda, args))
            check_pool(dev, pool)
        kept = rng.integers(0, pool.lens + 1)
        kept = np.where(rng.random(B) < 0.05, rng.choice([-1, 10 ** 6], B), kept).astype(np.int32)
        new = np.minimum(np.maximum(kept, 0) + rng.integers(-8, 40, B), 16 * stride).clip(0)
        new = np.where(rng.random(B) < 0.15, -1, new).astype(np.int32)
        pool.resize(new, kept=kept)
        va.verify_attn_pages_resize(dev, cuda(new), kept_lens=cuda(kept))
        check_pool(dev, pool)
        pool.check()


def test_resize_kept_lengths_argument_errors(va):
    pool = va.PagePool.create(8, 2, 3, [])
    for bad in (i32(1), i32(1, 2).long(), torch.zeros(2, dtype=torch.int32)):
        with pytest.raises(ValueError):
            va.verify_attn_pages_resize(pool, i32(1, 2), kept_lens=bad)


def test_page_calls_of_several_host_threads(va):
    """Pools whose bookkeeping wants shared memory past the default, in two different amounts, each used by a host thread
    and on a stream of its own, as fast as they can: no call changes what a call of another thread may ask for."""
    import threading
    pools = [va.PagePool.create(P, B, 2, []) for B, P in 2 * ((8192, 20000), (2700, 64))]
    streams = [torch.cuda.Stream() for _ in pools]
    lens = [torch.ones(pool.num_seqs, dtype=torch.int32, device="cuda") for pool in pools]
    for x in lens:
        x[50:] = 0
    torch.cuda.synchronize()
    resize = va.library().verify_attn_pages_resize
    codes, start = [set() for _ in pools], threading.Barrier(len(pools))

    def work(i):
        args = pools[i]._ref, lens[i].data_ptr(), streams[i].cuda_stream
        start.wait()
        codes[i] = {resize(*args) for _ in range(4000)}

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(pools))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert codes == [{0}] * len(pools)
    for pool, want in zip(pools, lens):
        assert torch.equal(pool.seq_lens, want) and pool.num_free.item() == pool.num_pages - 50
        assert va.verify_attn_pages_flags(pool) == 0


@pytest.mark.parametrize("given", [False, True])
def test_a_dropped_pool_keeps_its_memory_until_its_calls_are_done(va, given):
    """A pool dropped while its calls are queued on another stream: none of its tensors' memory is handed out before they
    have run (the tensors here are too large to share a block with anything else)."""
    big = torch.empty(2 ** 32, dtype=torch.uint8, device="cuda")
    pages = torch.zeros(2 ** 20, 64, dtype=torch.uint8, device="cuda")
    pool = va.PagePool.create(2 ** 20, 8, 2 ** 18, [pages])
    sizes = [(t.data_ptr(), t.numel() * t.element_size()) for t in (pool.workspace, pool.block_table, pool.ref_count,
                                                                    pool.free_list, pages)]
    new = i32(100, 2 ** 20, 0, 0, 0, 0, 0, 0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        for _ in range(60):  # some 30 ms before the pool's calls
            big.fill_(1)
        if not given:
            va.verify_attn_pages_resize(pool, new)
    if given:
        va.verify_attn_pages_resize(pool, new, stream=side)
    del pool, pages
    taken = [torch.empty(n, dtype=torch.uint8, device="cuda") for _, n in sizes for _ in range(2)]
    waiting = not side.query()
    reused = {t.data_ptr() for t in taken} & {at for at, _ in sizes}
    torch.cuda.synchronize()
    assert waiting and not reused


# ------------------------------------------------------------------ rotary and append


@pytest.mark.parametrize("kv_dtype", ["fp8_e4m3", "int8", "int4", "int2", "bf16"])
@pytest.mark.parametrize("D,R,pairing", [(64, 64, "half"), (128, 96, "half"), (256, 34, "adjacent"), (128, 22, "half")])
def test_rope_append_keeps_the_signs_of_zeros(va, kv_dtype, D, R, pairing):
    """Negative zeros, rows of them, and negative numbers too small for their row's scale: v is stored byte for byte as
    verify_attn_kv_append stores it, k as the append's rule makes it of the rotated rows."""
    B, T, Hkv = 2, 40, 2
    pages, scale, bt, lens, P = cache_case(3, [47, 40], T, Hkv, D, kv_dtype)

    def rows(seed):
        x = normal(seed, B, T, Hkv, D)
        kind = torch.randint(0, 5, x.shape, generator=torch.Generator().manual_seed(seed + 1)).cuda()
        x = torch.where(kind == 0, torch.full_like(x, -0.0), x)
        x = torch.where(kind == 1, -1e-6 * x.abs(), x)
        x = torch.where(kind == 2, torch.full_like(x, -1e-38), x)
        x[0, :4] = -0.0
        x[1, 5:9] = x[1, 5:9].sign() * 0.0
        return x.bfloat16()

    k, v = rows(40), rows(42)
    spec = va.verify_attn_rope_spec(R, pairing=pairing)
    pos = cuda((np.arange(B * T, dtype=np.int32) // 30).reshape(1, B, T))
    _, (kp, vp), (ks, vs), _ = run_append(va, spec, pos, None, k, v, pages, scale, bt, lens, kv_dtype)
    dev = cuda(pages.view(np.int16) if kv_dtype == "bf16" else pages)
    other, s1, s2 = dev.clone(), None if scale is None else cuda(scale), None if scale is None else cuda(scale)
    va.verify_attn_kv_append(v, v, dev, other, s1, s2, cuda(bt), cuda(lens), T, kv_dtype)
    assert np.array_equal(vp, bits16(dev) if kv_dtype == "bf16" else dev.cpu().numpy())
    _, turned = va.verify_attn_rope(spec, pos, k.float(), k.float())
    want, _ = expected_cache(turned.cpu().numpy(), pages, scale, bt, lens, kv_dtype, P)
    assert np.array_equal(kp, want)
    if kv_dtype == "fp8_e4m3":
        assert (vp == 0x80).sum() > 1000 and (kp == 0x80).sum() > 100


def test_rope_inside_an_autograd_function_and_refused_outside(va):
    """The way that the refusal names: forward and inverse calls in a Function.  The gradient of sum(w y) is the transposed
    map of w, within the bound of a rotated element; it also goes through a broadcast input, whose gradients add up (3
    heads: three elements and two additions)."""
    spec = va.verify_attn_rope_spec(16, sections=[3, 5])
    pos = cuda(np.random.default_rng(2).integers(0, 9000, (2, 2, 5)).astype(np.int32))

    class Rotate(torch.autograd.Function):
        @staticmethod
        def forward(ctx, q, k):
            return va.verify_attn_rope(spec, pos, q, k)

        @staticmethod
        def backward(ctx, dq, dk):
            return va.verify_attn_rope(spec, pos, dq, dk, inverse=True)

    q, one = normal(1, 2, 5, 4, 20).requires_grad_(), normal(2, 2, 5, 1, 20).requires_grad_()
    wq, wk = normal(3, 2, 5, 4, 20), normal(4, 2, 5, 3, 20)
    y, z = Rotate.apply(q, one.expand(2, 5, 3, 20))
    ((y * wq).sum() + (z * wk).sum()).backward()
    freq = 1.0e6 ** (-np.arange(8) / 8)
    for got, w, heads in ((q.grad, wq, 1), (one.grad, wk, 3)):
        ws = w.double().cpu().numpy()
        want = around.rope(ws, pos.tolist(), freq, spec.axis, inverse=True)
        bound = rope_bound(ws, 8, False, 1.0, torch.float32, want)
        if heads > 1:
            bound = bound.sum(2, keepdims=True) + 2 * 2.0 ** -24 * np.abs(want).sum(2, keepdims=True) * (1 + 1e-6)
            want = want.sum(2, keepdims=True)
        assert (np.abs(got.double().cpu().numpy() - want) <= bound).all()
    with pytest.raises(ValueError, match="gradient"):
        va.verify_attn_rope(spec, pos, q)
    with torch.no_grad():
        va.verify_attn_rope(spec, pos, q)
    assert torch.equal(va.verify_attn_rope(spec, pos, q.detach())[0], y.detach())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_rope_at_frequencies_above_one(va, dtype):
    """Frequencies up to 2^20 at the ends of int32: within the bound of every other angle."""
    freq = [2.0 ** 20, 3.0e4, 1024.0, 7.5, 1.0, -65536.5, 1e-3, 129.0]
    spec = va.verify_attn_rope_spec(16, inv_freq=freq)
    pos = np.array([2 ** 31 - 1, -(2 ** 31), 2 ** 30 + 7, 123456789, -1, 1], np.int32).reshape(1, 1, -1)
    x = normal(50, 1, 6, 3, 16, dtype=dtype)
    got, _ = va.verify_attn_rope(spec, cuda(pos), x)
    xs = x.double().cpu().numpy()
    ref = around.rope(xs, pos.tolist(), freq, [0] * 8)
    err = np.abs(got.double().cpu().numpy() - ref)
    assert (err <= rope_bound(xs, 8, False, 1.0, dtype, ref)).all(), err.max()


@pytest.mark.parametrize("kv_dtype", ["int8", "bf16"])
@pytest.mark.parametrize("D,R,pairing", [(64, 22, "half"), (256, 34, "half"), (128, 128, "adjacent"), (256, 34, "adjacent"),
                                         (128, 96, "half")])
def test_rope_append_in_place(va, kv_dtype, D, R, pairing):
    """q as its own output, halves that begin inside a vector and adjacent pairs among them; k and v as [B, H, T, D] and
    as one head for all."""
    B, T, Hq, Hkv = 3, 70, 5, 2
    pages, scale, bt, lens, P = cache_case(9, [70, 100, 81], T, Hkv, D, kv_dtype)
    q, k, v = (normal(60 + i, B, T, h, D, dtype=torch.bfloat16) for i, h in enumerate((Hq, Hkv, Hkv)))
    spec = va.verify_attn_rope_spec(R, pairing=pairing)
    want = run_append(va, spec, None, q, k, v, pages, scale, bt, lens, kv_dtype)
    work = q.clone()
    lie = lambda x: x.transpose(1, 2).contiguous().transpose(1, 2)  # noqa: E731
    got = run_append(va, spec, None, work, lie(k), lie(v), pages, scale, bt, lens, kv_dtype, q_out=work)
    assert got[0] is work and torch.equal(work, want[0])
    assert all(np.array_equal(a, b) for a, b in zip(got[1] + got[2], want[1] + want[2]))
    one = k[:, :, :1].expand(B, T, Hkv, D)
    a = run_append(va, spec, None, None, one, one, pages, scale, bt, lens, kv_dtype)
    b = run_append(va, spec, None, None, one.contiguous(), one.contiguous(), pages, scale, bt, lens, kv_dtype)
    assert all(np.array_equal(x, y) for x, y in zip(a[1] + a[2], b[1] + b[2]))


def test_sizes_past_32_bits_are_refused(va):
    """Sizes whose low 32 bits alone would be a small call (tensors of one element here, broadcast)."""
    far = 2 ** 32 + 3
    big = lambda *s, dtype=torch.bfloat16: torch.zeros((), dtype=dtype, device="cuda").expand(*s)  # noqa: E731
    head = torch.zeros(1, 1, 1, 64, dtype=torch.bfloat16, device="cuda")
    spec = va.verify_attn_rope_spec(64)
    pos = big(1, 1, far, dtype=torch.int32)
    with pytest.raises(ValueError, match="32 bits"):
        va.verify_attn_rope(spec, pos, head.expand(1, far, 1, 64))
    with pytest.raises(ValueError, match="32 bits"):
        va.verify_attn_rope(spec, i32(0).view(1, 1, 1), head, head.expand(1, 1, far, 64))
    with pytest.raises(ValueError, match="32 bits"):
        va.verify_attn_rope_append(spec, None, None, head.expand(1, far, 1, 64), head.expand(1, far, 1, 64), head, head, None,
                                   None, i32(0).view(1, 1), i32(far % 2 ** 31), "bf16")
    for shape in ((1, 2, far), (1, far, 4), (far, 1, 4)):
        with pytest.raises(ValueError, match="32 bits"):
            va.verify_attn_accept_probs(big(*shape), i32(0).view(1, 1), torch.zeros(1, 1, device="cuda"), torch.zeros(1, device="cuda"))
    with pytest.raises(ValueError, match="32 bits"):
        va.PagePool(big(1, far, dtype=torch.int32), i32(0), i32(0), i32(0), i32(1), [])
    with pytest.raises(ValueError, match="32 bits"):
        va.PagePool(i32(0).view(1, 1), i32(0), big(far, dtype=torch.int32), big(far, dtype=torch.int32), i32(1), [])
    with pytest.raises(ValueError, match="32 bits"):
        va.verify_attn_accept(big(1, 2, far, dtype=torch.float32), i32(0).view(1, 1), torch.zeros(1, device="cuda"), 1)
    with pytest.raises(ValueError, match="32 bits"):
        va.verify_attn_lookup_draft(big(1, far, dtype=torch.int32), i32(5), 4)
    with pytest.raises(ValueError, match="32 bits"):
        va.verify_attn_kv_append(head, head, head, head, None, None, big(1, far, dtype=torch.int32), i32(1), 1, "bf16")


@pytest.mark.parametrize("kv_dtype", ["int8", "bf16"])
@pytest.mark.parametrize("num_pages", [0, 8])
def test_append_rows_without_a_page_are_skipped_and_flagged(va, kv_dtype, num_pages):
    """A device length past what the table's row holds, whose rows do not go by the next row's entries, and an entry of -1,
    as a page pool's table has it where nothing is held; with and without the count of pages."""
    T, Hkv, D = 4, 2, 64
    kind = torch.bfloat16 if kv_dtype == "bf16" else torch.int8
    kp, vp = (torch.zeros(8, 16, Hkv, D, dtype=kind, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros(8, 16, Hkv, device="cuda") for _ in range(2))
    flags = i32(0)
    x = normal(1, 2, T, Hkv, D, dtype=torch.bfloat16)
    table = i32(0, 1, 2, 3, 4, 5).view(2, 3)[:, :2].contiguous()  # rows of two blocks: 0 1, 3 4
    va.verify_attn_kv_append(x, x, kp, vp, ks, vs, table, i32(34, 10), T, kv_dtype, num_pages=num_pages, flags=flags)
    torch.cuda.synchronize()
    assert flags.item() == 1
    written = (vp.float().abs().amax((2, 3)) > 0).nonzero().tolist()
    assert written == [[1, 14], [1, 15], [3, 6], [3, 7], [3, 8], [3, 9]]
    flags.zero_()
    va.verify_attn_kv_append(x, x, kp, vp, ks, vs, i32(-1, 5, 6, -1).view(2, 2), i32(18, 18), T, kv_dtype, num_pages=num_pages,
                             flags=flags)
    torch.cuda.synchronize()
    assert flags.item() == 1
    written = (vp[4:].float().abs().amax((2, 3)) > 0).nonzero().tolist()
    assert written == [[1, 0], [1, 1], [2, 14], [2, 15]]
