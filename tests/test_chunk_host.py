"""The operators of a prompt worked in chunks, without a GPU: their plain definitions against statements
that do not share them, the plan of a batch, and every refusal that is taken before the GPU is touched."""
import ctypes

import numpy as np
import pytest

import speculative_decoding_verify_causal_gb300 as va
from oracle import chunks
from speculative_decoding_verify_causal_gb300 import build as vbuild

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module", autouse=True)
def built():
    vbuild.build()


def bits(x):
    return torch.from_numpy(np.ascontiguousarray(x)).bfloat16().view(torch.int16).numpy()


# ------------------------------------------------------------------ the definitions


def test_chunk_is_masked_softmax_attention():
    rng = np.random.default_rng(0)
    n, L, Hq, Hkv, D, P = 7, 45, 4, 2, 64, 5
    K, V = rng.standard_normal((2, P, 16, Hkv, D)).astype(np.float32)
    q = rng.standard_normal((n, Hq, D))
    table = rng.permutation(P)[None, :3].astype(np.int32)
    out, lse, _, _ = chunks.chunk(q, bits(K), bits(V), None, None, table, [n], [L], "bf16", Hkv)
    k, v = (torch.from_numpy(chunks.decode(bits(x), "bf16"))[table[0].astype(np.int64)].flatten(0, 1)[:L] for x in (K, V))
    k, v = (x.transpose(0, 1).repeat_interleave(Hq // Hkv, 0) for x in (k, v))
    mask = torch.arange(L)[None] <= (torch.arange(n) + L - n)[:, None]
    want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q).transpose(0, 1), k, v, attn_mask=mask)
    assert np.abs(out - want.transpose(0, 1).numpy()).max() < 1e-12
    x = torch.from_numpy(q).transpose(0, 1) @ k.transpose(1, 2) / 8.0
    want = torch.logsumexp(x.masked_fill(~mask, -np.inf), -1).T.numpy()
    assert np.abs(lse - want).max() < 1e-12


def test_each_token_gives_one_unit_of_weight():
    rng = np.random.default_rng(1)
    new, lens, Hq, Hkv, D, P = [3, 0, 5], [20, 9, 5], 6, 2, 64, 6
    K, V = rng.standard_normal((2, P, 16, Hkv, D)).astype(np.float32)
    q = rng.standard_normal((8, Hq, D))
    table = rng.permutation(P).reshape(3, 2).astype(np.int32)
    _, lse, _, _ = chunks.chunk(q, bits(K), bits(V), None, None, table, new, lens, "bf16", Hkv)
    w = chunks.chunk_weights(q, bits(K), None, table, new, lens, "bf16", Hkv, lse, None)
    assert np.abs(w.sum(-1) - np.array([9, 0, 15])[:, None]).max() < 1e-12 and (w[0, :, 20:] == 0).all()
    old = rng.random(w.shape)
    more = chunks.chunk_weights(q, bits(K), None, table, new, lens, "bf16", Hkv, lse, old)
    assert np.abs(more[0, :, :17] - old[0, :, :17] - w[0, :, :17]).max() < 1e-12
    assert np.abs(more[0, :, 17:20] - w[0, :, 17:20]).max() < 1e-12 and (more[1] == old[1]).all()


def test_decoders_against_torch():
    every = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(every).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(chunks.e4m3(every), want, equal_nan=True)
    assert np.array_equal(chunks.decode(every, "int8"), every.view(np.int8))
    field = np.unpackbits(every[:, None], axis=1, bitorder="little")
    for kv, w in (("int4", 4), ("int2", 2)):
        f = field.reshape(256, 8 // w, w).astype(np.int64)
        value = (f * 2 ** np.arange(w)).sum(-1)
        value -= f[..., -1] << w
        assert np.array_equal(chunks.decode(every[:, None], kv), value)


@pytest.mark.parametrize("seed", range(8))
def test_evict_keeps_the_heaviest(seed):
    rng = np.random.default_rng(seed)
    B, Hkv, P = 3, 2, 12
    table = rng.permutation(P).reshape(B, 4).astype(np.int32)
    lens = rng.integers(1, 65, B)
    keep = rng.integers(0, 70, B)
    w = rng.choice([0.0, 0.5, 1.0, 2.0, np.nan], (B, Hkv, 64))
    pos = np.stack([[rng.permutation(64) for _ in range(Hkv)] for _ in range(B)]).astype(np.int32)
    data = rng.integers(0, 1 << 30, (P, 16, Hkv, 3))
    before, w0, p0 = data.copy(), w.copy(), pos.copy()
    new, flags = chunks.evict([data], table, lens, w, keep, pos, 4, lens - 5, num_pages=P)
    assert flags == 0 and np.array_equal(new, np.minimum(lens, keep))
    for b in range(B):
        at = lambda x, j, g: x[table[b, j // 16], j % 16, g].tolist()  # noqa: E731
        for g in range(Hkv):
            L, k = lens[b], int(new[b])
            safe = (p0[b, g, :L] < 4) | (p0[b, g, :L] >= lens[b] - 5)
            value = np.where(safe, np.inf, np.nan_to_num(w0[b, g, :L], nan=-np.inf))
            want = np.lexsort((np.arange(L), -value))[:k]
            held = {j for j in range(L) for i in range(k) if at(data, i, g) == at(before, j, g)}
            assert held == set(want.tolist())
            for i in range(k):  # weights and positions came along, and what could stay did
                j = next(j for j in range(L) if at(data, i, g) == at(before, j, g))
                assert np.array_equal([w[b, g, i]], [w0[b, g, j]], equal_nan=True) and pos[b, g, i] == p0[b, g, j]
                assert j == i or (j >= k and i not in want)


def test_logprobs_definition():
    rng = np.random.default_rng(2)
    x = rng.standard_normal((5, 300)) * 3
    x[1, 7] = 40.0
    x[2] = -np.inf
    x[3, 10:] = -np.inf
    t = np.array([3, 7, 0, 299, -1])
    lp, ranks, ent, tt, tl, _ = chunks.logprobs(x, t, 4)
    z = torch.log_softmax(torch.from_numpy(x), -1).numpy()
    for n in (0, 1, 3):
        assert lp[n] == pytest.approx(z[n, t[n]], rel=1e-12) and np.allclose(tl[n], z[n, tt[n]], rtol=1e-9)
        p = np.exp(z[n])
        assert ent[n] == pytest.approx(-(p[p > 0] * z[n][p > 0]).sum(), rel=1e-9)
    assert -1e-12 < lp[1] < 0 and ranks.tolist()[1:] == [0, 0, 299, -1]
    assert lp[2] == -np.inf and ent[2] == 0 and (tl[2] == -np.inf).all() and tt[2].tolist() == [0, 1, 2, 3]
    assert lp[4] == -np.inf


# ------------------------------------------------------------------ the plan


@pytest.mark.parametrize("seed", range(40))
def test_plan_covers_every_token_and_key_once(seed):
    rng = np.random.default_rng(seed)
    B = int(rng.integers(1, 20))
    Hkv, G, D = int(rng.choice([1, 2, 4, 8])), int(rng.choice([1, 3, 4, 6, 7, 8, 16, 128])), int(rng.choice([64, 128, 256]))
    new = rng.integers(0, int(rng.choice([2, 50, 2000])), B)
    lens = new + rng.integers(0, int(rng.choice([1, 300, 40000])), B)
    info, items = va.verify_attn_chunk_plan_describe(new, lens, Hkv * G, Hkv, D, "int8", num_sms=int(rng.choice([8, 152])))
    assert info["num_tokens"] == new.sum() and info["num_items"] == len(items)
    live = new > 0
    assert info["max_blocks"] == (max((lens[live] + 15) // 16) if live.any() else 0)
    starts = np.concatenate([[0], np.cumsum(new)])
    tpt = 128 // G
    seen = {}
    for b, h, q0, nt, k0, k1 in items.tolist():
        t = q0 - starts[b]
        assert 0 <= t and t + nt <= new[b] and 1 <= nt <= tpt * (1 if D == 256 else 2) and k0 % 16 == 0 and k0 < k1
        seen.setdefault((b, h, t, nt), []).append((k0, k1))
    for b in range(B):
        for h in range(Hkv):
            spans = sorted((t, nt) for bb, hh, t, nt in seen if (bb, hh) == (b, h))
            assert sum(nt for _, nt in spans) == new[b] and all(t + n == u for (t, n), (u, _) in zip(spans, spans[1:]))
    for (b, h, t, nt), ranges in seen.items():
        ranges.sort()
        # up to the last key that one of its tokens sees
        assert ranges[0][0] == 0 and ranges[-1][1] == lens[b] - new[b] + t + nt
        assert all(x[1] == y[0] for x, y in zip(ranges, ranges[1:]))


@pytest.mark.parametrize("kw,status", [
    (dict(chunk_lens=[5], seq_lens=[4]), -1), (dict(chunk_lens=[-1], seq_lens=[4]), -1),
    (dict(chunk_lens=[], seq_lens=[]), -1), (dict(num_q_heads=5), -1), (dict(num_q_heads=0), -1), (dict(num_kv_heads=0), -1),
    (dict(seq_lens=[2 ** 30 + 1]), -1), (dict(chunk_lens=[2 ** 30] * 2, seq_lens=[2 ** 30] * 2), -1), (dict(num_sms=0), -1),
    (dict(head_dim=96), -2), (dict(kv_dtype=7), -2), (dict(num_q_heads=258, num_kv_heads=2), -2),
])
def test_plan_refusals(kw, status):
    args = dict(dict(chunk_lens=[4], seq_lens=[9], num_q_heads=8, num_kv_heads=2, head_dim=64, kv_dtype="int8", num_sms=152), **kw)
    with pytest.raises(va.VerifyAttnError) as e:
        va.verify_attn_chunk_plan_describe(**args)
    assert e.value.status == status
    if "num_sms" not in kw:
        with pytest.raises(va.VerifyAttnError) as e:  # before a device is asked for
            va.verify_attn_chunk_plan(**args)
        assert e.value.status == status
    with pytest.raises(ValueError):
        va.verify_attn_chunk_plan_describe([1, 2], [3], 8, 2, 64, "int8", 152)


def test_calls_without_a_plan():
    lib = va.library()
    heads = va._Heads(4096, 0, 512, 64, 8)
    assert lib.verify_attn_chunk(None, heads, 4096, 4096, None, None, 4096, 1, 1, 4096, None, None) == -4
    assert lib.verify_attn_chunk_weights(None, heads, 4096, None, 4096, 1, 1, 4096, 4096, 1, 1, 0, None, None, None) == -4
    lib.verify_attn_chunk_plan_destroy(None)
    assert lib.verify_attn_chunk_plan_get_info(None, ctypes.byref(va.ChunkPlanInfo())) == -1


# ------------------------------------------------------------------ refusals


EVICT = dict(k_pages=4096, v_pages=4096, k_scale=4096, v_scale=4096, kv_dtype=2, block_table=4096, block_table_stride=4,
             seq_lens=4096, num_seqs=2, num_kv_heads=2, head_dim=64, num_pages=8, weights=4096, slot_pos=None, stride_seq=128,
             stride_head=64, num_slots=64, keep_lens=4096, num_sinks=0, recent_from=None, ref_count=None, new_lens=8192,
             workspace=4096, flags=None, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(head_dim=96), -2), (dict(kv_dtype=9), -2), (dict(num_seqs=0), -1), (dict(num_seqs=40000), -1),
    (dict(num_kv_heads=0), -1), (dict(num_slots=-1), -1), (dict(num_slots=2 ** 30 + 2), -1), (dict(num_sinks=-1), -1),
    (dict(block_table_stride=-1), -1), (dict(num_pages=-1), -1), (dict(stride_seq=-1), -1), (dict(stride_head=-1), -1),
    # rows of weights on one another, with extents past 63 bits too; new lengths over what other heads still read
    (dict(stride_seq=0), -1), (dict(stride_head=0), -1), (dict(stride_head=63), -1), (dict(stride_seq=127), -1),
    (dict(stride_seq=64, stride_head=127), -1), (dict(stride_seq=2 ** 62, stride_head=2 ** 62), -1),
    (dict(new_lens=4096), -1), (dict(new_lens=4100), -1), (dict(new_lens=4092), -1), (dict(recent_from=8188), -1),
    *[(dict([(n, None)]), -1) for n in ("k_pages", "v_pages", "k_scale", "v_scale", "block_table", "seq_lens", "weights",
                                        "keep_lens", "new_lens", "workspace")],
    *[(dict([(n, 4104)]), -1) for n in ("k_pages", "v_pages", "workspace")],
    *[(dict([(n, 4098)]), -1) for n in ("k_scale", "v_scale", "block_table", "seq_lens", "weights", "slot_pos", "keep_lens",
                                        "recent_from", "ref_count", "new_lens", "flags")],
])
def test_evict_refusals(change, status):
    assert va.library().verify_attn_evict(*dict(EVICT, **change).values()) == status


def test_evict_workspace_size():
    size = va.library().verify_attn_evict_workspace_bytes
    assert size(2, 4, 1000) >= 8 * (4 + 500 * 8) and size(1, 1, 0) > 0
    assert size(0, 1, 9) == size(1, 0, 9) == size(1, 1, -1) == size(65536, 1, 9) == 0


LOGPROBS = dict(logits=4096, stride=100, type=0, tokens=4096, num_rows=3, vocab=100, num_top=5, logprobs=4096, ranks=4096,
                entropy=4096, top_tokens=4096, top_logprobs=4096, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(type=3), -2), (dict(num_rows=-1), -1), (dict(num_rows=2 ** 27 + 1), -1), (dict(vocab=0), -1),
    (dict(vocab=2 ** 30 + 1), -1), (dict(num_top=-1), -1), (dict(num_top=33), -1), (dict(num_top=5, vocab=4), -1),
    (dict(logits=None), -1), (dict(tokens=None), -1), (dict(top_tokens=None), -1), (dict(top_logprobs=None), -1),
    (dict(logits=4097), -1), (dict(logits=4098, type=2), -1),
    *[(dict([(n, 4098)]), -1) for n in ("tokens", "logprobs", "ranks", "entropy", "top_tokens", "top_logprobs")],
    (dict(num_rows=0), 0),
])
def test_logprobs_refusals(change, status):
    assert va.library().verify_attn_logprobs(*dict(LOGPROBS, **change).values()) == status


def test_calls_that_would_lose_a_gradient_or_have_no_gpu_tensors_are_refused():
    x, w = torch.zeros(2, 8), torch.zeros(2, 8, requires_grad=True)
    t = torch.zeros(2, dtype=torch.int32)
    plan = va.ChunkPlan(None, (1, 8, 2, 64, 2, 2, 2), 0)
    q = torch.zeros(2, 8, 64, dtype=torch.bfloat16)
    calls = [lambda y: va.verify_attn_logprobs(y, t), lambda y: va.verify_attn_chunk(plan, y, x, x, x, x, t),
             lambda y: va.verify_attn_chunk(plan, q, x, x, x, y, t),
             lambda y: va.verify_attn_chunk_weights(plan, q, x, x, t, y, x),
             lambda y: va.verify_attn_chunk_weights(plan, q, x, x, t, x, y)]
    for call in calls:
        with pytest.raises(ValueError, match="gradient"):
            call(w)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call(w)
    with pytest.raises(ValueError, match="CUDA"):
        va.verify_attn_evict(x, x, x, x, t, t, x, t, "int8")
