"""The operators around a verify step, as they are measured: rotary positions with several axes
(alone, and fused with the KV append), acceptance of drafted tokens from given probabilities and
random numbers, and the care of a paged cache (resize, fork, compact).

``run`` computes each operator in its plain form, elementary torch operations, or, where ``own``
is true, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
E4M3_MAX = 448.0
FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FLOAT_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
# bytes of one cached element; the packed 4-bit cache holds two to a byte
CACHE_BYTES = {"bf16": 2.0, "int8": 1.0, "fp8_e4m3": 1.0, "int4": 0.5}


# ---------------------------------------------------------------------------------------------
# the cases


def listed():
    return [
        # a video prompt through an attention layer: q and k are slices of one fused projection
        {"name": "rope_video_prompt", "op": "rope", "batch": 1, "tokens": 32768, "q_heads": 32, "k_heads": 8,
         "head_dim": 128, "rotary_dim": 128, "axes": 3, "pairing": "half", "layout": "dealt", "dtype": "bf16",
         "inverse": False, "fused": True},
        # gradients of an image tower's q and k in fp32: 37 x 37 patches and one more, head_dim 80
        {"name": "rope_patch_gradient", "op": "rope", "batch": 3, "tokens": 1370, "q_heads": 16, "k_heads": 16,
         "head_dim": 80, "rotary_dim": 80, "axes": 2, "pairing": "adjacent", "layout": "blocked", "dtype": "fp32",
         "inverse": True, "fused": False},
        # the 16-token verify block of the 25k-token lookup workload, a quarter of each head rotated
        {"name": "append_verify_block", "op": "append", "batch": 1, "tokens": 16, "context": 25000, "q_heads": 24,
         "kv_heads": 4, "head_dim": 256, "rotary_dim": 64, "axes": 3, "pairing": "half", "layout": "dealt",
         "kv": "fp8_e4m3"},
        # one chunk of prefill for eight requests, bf16 cache, every position one axis
        {"name": "append_prefill_chunk", "op": "append", "batch": 8, "tokens": 1024, "context": 2048, "q_heads": 32,
         "kv_heads": 8, "head_dim": 128, "rotary_dim": 128, "axes": 1, "pairing": "half", "layout": "blocked",
         "kv": "bf16"},
        # lookup drafts (point-mass proposals) of one request over the full vocabulary
        {"name": "accept_lookup_drafts", "op": "accept", "batch": 1, "drafts": 16, "vocab": 151936, "model": False,
         "dtype": "fp32", "top_k": 0, "ragged": False},
        # a batch with a drafting model, so that a rejection reads two rows, and ragged draft counts
        {"name": "accept_model_drafts", "op": "accept", "batch": 64, "drafts": 5, "vocab": 151936, "model": True,
         "dtype": "fp32", "top_k": 0, "ragged": True},
        # eight samples of one 25k-token prompt: full pages shared, the last one copied
        {"name": "fork_samples", "op": "fork", "share": True, "parents": 1, "each": 8, "tokens": 25013, "layers": 2,
         "kv_heads": 4, "head_dim": 256, "kv": "int8"},
        # sixteen sequences copied whole, in four layers
        {"name": "fork_copies", "op": "fork", "share": False, "parents": 16, "each": 1, "tokens": 4090, "layers": 4,
         "kv_heads": 4, "head_dim": 256, "kv": "int8"},
        # between two verify steps of a small batch: rejected drafts give pages back, the next block takes them
        {"name": "resize_between_steps", "op": "resize", "seqs": 16, "tokens": 4500, "drafts": 16, "churn": False,
         "layers": 1, "kv_heads": 4, "head_dim": 256, "kv": "int8"},
        # a large batch with a quarter of its requests leaving and as many prompts coming in
        {"name": "resize_churn", "op": "resize", "seqs": 256, "tokens": 8000, "drafts": 5, "churn": True, "layers": 1,
         "kv_heads": 1, "head_dim": 64, "kv": "int8"},
        # a small pool, half empty
        {"name": "compact_small", "op": "compact", "pages": 700, "seqs": 5, "live": 0.5, "layers": 1, "kv_heads": 1,
         "head_dim": 64, "kv": "bf16"},
        # a pool of 131k tokens in two layers that many requests have left
        {"name": "compact_pool", "op": "compact", "pages": 8192, "seqs": 37, "live": 0.45, "layers": 2, "kv_heads": 4,
         "head_dim": 256, "kv": "int8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "accept", "fork", "resize", "compact"])
    if op == "rope":
        q_heads, k_heads = rng.choice([(4, 1), (8, 8), (16, 16), (28, 4), (32, 8), (7, 7)])
        head_dim = rng.choice([64, 72, 80, 96, 128, 256])
        rotary = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4 * 2 - 2])
        dtype = rng.choice(["bf16", "fp16", "fp32"])
        top = int(32768 * 40 * 128 / ((q_heads + k_heads) * head_dim * FLOAT_BYTES[dtype] / 2))
        total = _log(rng, 1, min(top, 60000))
        batch = rng.choice([1, 1, 2, 3]) if total >= 3 else 1
        return {"op": op, "batch": batch, "tokens": max(1, total // batch), "q_heads": q_heads, "k_heads": k_heads,
                "head_dim": head_dim, "rotary_dim": rotary, "axes": rng.choice([1, 2, 3]),
                "pairing": rng.choice(["half", "adjacent"]), "layout": rng.choice(["blocked", "dealt"]),
                "dtype": dtype, "inverse": rng.random() < 0.4, "fused": rng.random() < 0.5}
    if op == "append":
        q_heads, kv_heads = rng.choice([(4, 1), (24, 4), (32, 8), (8, 8)])
        head_dim = rng.choice([64, 128, 256])
        total = _log(rng, 1, 8192 * 40 * 128 // ((q_heads + 2 * kv_heads) * head_dim))
        batch = min(total, _log(rng, 1, 64))
        return {"op": op, "batch": batch, "tokens": max(1, total // batch), "context": _log(rng, 1, 65536 // batch),
                "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
                "rotary_dim": rng.choice([head_dim, head_dim // 2, head_dim // 4]), "axes": rng.choice([1, 3]),
                "pairing": rng.choice(["half", "adjacent"]), "layout": rng.choice(["blocked", "dealt"]),
                "kv": rng.choice(["bf16", "fp8_e4m3"])}
    if op == "accept":
        vocab = rng.choice([1000, 32000, 50257, 128256, 151936, 200019])
        return {"op": op, "batch": _log(rng, 1, max(2, 64 * 151936 // max(vocab, 151936))), "drafts": rng.randint(1, 8),
                "vocab": vocab, "model": rng.random() < 0.5, "dtype": rng.choice(["fp32", "bf16", "fp16"]),
                "top_k": rng.choice([0, 0, 50]), "ragged": rng.random() < 0.5}
    shape = {"layers": rng.choice([1, 2, 3]), "kv_heads": rng.choice([1, 4, 8]), "head_dim": rng.choice([64, 128, 256]),
             "kv": rng.choice(["bf16", "int8", "int4"])}
    page_bytes = _page_bytes(shape)
    if op == "fork":
        share = rng.random() < 0.5
        parents = _log(rng, 1, 16)
        each = rng.randint(1, 8) if share else 1
        most = 16 * 256 * 4 * 2 * PAGE * 4 * 260
        tokens = _log(rng, 17, max(40, min(30000, most // (parents * page_bytes) * PAGE)))
        return {"op": op, "share": share, "parents": parents, "each": each, "tokens": tokens, **shape}
    if op == "resize":
        return {"op": op, "seqs": _log(rng, 1, 256), "tokens": _log(rng, 40, 8000), "drafts": rng.choice([5, 8, 16]),
                "churn": rng.random() < 0.5, "layers": 1, "kv_heads": 1, "head_dim": 64, "kv": rng.choice(["int8", "bf16"])}
    most = 8192 * 2 * 2 * PAGE * 4 * 260
    pages = _log(rng, 40, min(60000, most // page_bytes))
    return {"op": op, "pages": pages, "seqs": min(pages // 8, _log(rng, 1, 64)), "live": round(rng.uniform(0.2, 0.9), 3),
            **shape}


# ---------------------------------------------------------------------------------------------
# inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _sections(case):
    """Pairs of each axis: a quarter of them the first axis's where there are three, else even shares."""
    pairs, axes = case["rotary_dim"] // 2, case["axes"]
    if axes == 1:
        return [pairs]
    first = pairs // 4 if axes == 3 else pairs // 2
    rest = pairs - first
    return [first, rest] if axes == 2 else [first, rest - rest // 2, rest // 2]


def _axis_of_pair(sections, layout):
    """The axis whose position turns each pair: the sections one after the other, or dealt round to
    the axes that still have pairs left."""
    if layout == "blocked":
        return [a for a, n in enumerate(sections) for _ in range(n)]
    left, out = list(sections), []
    while any(left):
        for a in range(len(left)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _positions(case, start):
    """int32 [axes, B, T]: the text's running position, or a frame, row and column of each token."""
    B, T, A = case["batch"], case["tokens"], case["axes"]
    t = torch.arange(T, dtype=torch.int64)[None, :].expand(B, T) + start[:, None]
    if A == 1:
        pos = t[None]
    else:
        w = max(1, int(math.sqrt(min(T, 4096))))
        grid = torch.arange(T, dtype=torch.int64)[None, :].expand(B, T)
        parts = [start[:, None] + grid // (w * w), start[:, None] + grid // w % w, start[:, None] + grid % w]
        pos = torch.stack(parts[3 - A:] if A < 3 else parts)
    return pos.to(torch.int32).contiguous().cuda()


def _rotary(case):
    pairs = case["rotary_dim"] // 2
    inv_freq = np.array([1.0e6 ** (-i / pairs) for i in range(pairs)], np.float64)
    axis = _axis_of_pair(_sections(case), case["layout"])
    s = {"inv_freq": torch.from_numpy(inv_freq).cuda(), "axis": torch.tensor(axis, dtype=torch.int64).cuda()}
    if own:  # the description of the rotation that a user's program keeps
        import speculative_decoding_verify_causal_gb300 as va
        s["rope"] = va.verify_attn_rope_spec(case["rotary_dim"], inv_freq=inv_freq, sections=_sections(case),
                                             layout=case["layout"], pairing=case["pairing"])
    return s


def _prepare_rope(case, seed):
    g = _generator(seed)
    B, T, Hq, Hk, D = (case[k] for k in ("batch", "tokens", "q_heads", "k_heads", "head_dim"))
    dt = FLOATS[case["dtype"]]
    s = _rotary(case)
    if case["fused"]:  # q, k and v side by side in one projection's output
        x = _normal(g, B, T, Hq + 2 * Hk, D, dtype=dt)
        s["q"], s["k"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hk]
    else:
        s["q"], s["k"] = _normal(g, B, T, Hq, D, dtype=dt), _normal(g, B, T, Hk, D, dtype=dt)
    start = torch.randint(0, 200000, (B,), generator=torch.Generator().manual_seed(int(seed)))
    s["positions"] = _positions(case, start)
    s["q_out"] = torch.empty(B, T, Hq, D, dtype=dt, device="cuda")
    s["k_out"] = torch.empty(B, T, Hk, D, dtype=dt, device="cuda")
    return s


def _context_lens(case):
    """Lengths of a batch's contexts, the T new tokens not counted: the same for every seed."""
    rng = np.random.default_rng([case["batch"], case["context"], case["tokens"]])
    c = case["context"]
    return rng.integers(max(0, c // 2), c + 1, case["batch"]) if case["batch"] > 1 else np.array([c])


def _prepare_append(case, seed):
    g = _generator(seed)
    B, T, Hq, Hk, D = (case[k] for k in ("batch", "tokens", "q_heads", "kv_heads", "head_dim"))
    s = _rotary(case)
    x = _normal(g, B, T, Hq + 2 * Hk, D, dtype=torch.bfloat16)
    s["q"], s["k"], s["v"] = x[:, :, :Hq], x[:, :, Hq:Hq + Hk], x[:, :, Hq + Hk:]
    lens = _context_lens(case) + T
    blocks = -(-lens // PAGE)
    P = int(blocks.sum())
    order = np.random.default_rng(seed).permutation(P).astype(np.int32)
    table, at = np.zeros((B, int(blocks.max())), np.int32), 0
    for b in range(B):
        table[b, :blocks[b]] = order[at:at + blocks[b]]
        at += blocks[b]
    s["block_table"] = torch.from_numpy(table).cuda()
    s["seq_lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    s["positions"] = _positions(case, torch.from_numpy(lens - T))
    if case["kv"] == "bf16":
        s["k_pages"], s["v_pages"] = (_normal(g, P, PAGE, Hk, D, dtype=torch.bfloat16) for _ in range(2))
        s["k_scale"] = s["v_scale"] = None
    else:
        s["k_pages"], s["v_pages"] = (_normal(g, P, PAGE, Hk, D).mul_(100).clamp_(-448, 448).to(torch.float8_e4m3fn)
                                      .view(torch.uint8) for _ in range(2))
        s["k_scale"], s["v_scale"] = (torch.rand(P, PAGE, Hk, generator=g, device="cuda") * 0.01 for _ in range(2))
    s["q_out"] = torch.empty(B, T, Hq, D, dtype=torch.bfloat16, device="cuda")
    s["kv"] = case["kv"]
    s["num_pages"] = P
    return s


def _prepare_accept(case, seed):
    g = _generator(seed)
    B, T, V = case["batch"], case["drafts"], case["vocab"]
    dt = FLOATS[case["dtype"]]
    z = _normal(g, B, T + 1, V) * 3
    if case["top_k"]:
        kth = z.topk(min(case["top_k"], V), dim=-1).values[..., -1:]
        z = z.masked_fill(z < kth, -math.inf)
    s = {"p": torch.softmax(z, -1).to(dt), "q": None, "lens": None}
    w = z[:, :T]
    if case["model"]:
        w = w + _normal(g, B, T, V)
        s["q"] = torch.softmax(w, -1).to(dt)
    # a draft is what its proposal would sample: the Gumbel race of its logits, cooled for lookup drafts
    noise = -torch.log(-torch.log(torch.rand(B, T, V, generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)))
    s["drafts"] = (w * (1.0 if case["model"] else 4.0) + noise).argmax(-1).to(torch.int32)
    if case["ragged"]:
        s["lens"] = torch.randint(0, T + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    s["u_accept"] = torch.rand(B, T, generator=g, device="cuda")
    s["u_emit"] = torch.rand(B, generator=g, device="cuda")
    s["tokens"] = torch.empty(B, T + 1, dtype=torch.int32, device="cuda")
    s["accepted"] = torch.empty(B, dtype=torch.int32, device="cuda")
    return s


def _page_bytes(case):
    """Bytes of one page in all of a cache's buffers: K and V of every layer, scales with them."""
    rows = PAGE * case["kv_heads"]
    per = rows * int(case["head_dim"] * CACHE_BYTES[case["kv"]]) + (0 if case["kv"] == "bf16" else rows * 4)
    return 2 * per * case["layers"]


def _lens_of(case):
    """(lengths now, wanted lengths, (parent, child) pairs, pages, stride) of a pages case: the same for every seed."""
    op = case["op"]
    if op == "fork":
        rng = np.random.default_rng([case["parents"], case["tokens"], case["each"]])
        n, c = case["parents"], case["tokens"]
        lens = rng.integers(max(1, c * 3 // 4), c + 1, n) if n > 1 else np.array([c])
        pairs = [(p, n + p * case["each"] + i) for p in range(n) for i in range(case["each"])]
        now = np.concatenate([lens, np.zeros(len(pairs), np.int64)])
        blocks = -(-lens // PAGE)
        need = len(pairs) if case["share"] else int(blocks.sum()) * case["each"]
        return now, now, pairs, int(blocks.sum()) + need + 5, int(blocks.max()) + 2
    if op == "resize":
        B, c, T = case["seqs"], case["tokens"], case["drafts"]
        rng = np.random.default_rng([B, c, T])
        now = rng.integers(max(1, c // 8), c + 1, B)
        new = np.maximum(now + rng.integers(-T, T + 2, B), 0)
        if case["churn"]:
            kind = rng.integers(0, 4, B)
            new = np.where(kind == 0, 0, new)
            now = np.where(kind == 1, 0, now)
            new = np.where(kind == 1, rng.integers(max(1, c // 8), c + 1, B), new)
        most = np.maximum(now, new)
        return now, new, [], int((-(-most // PAGE)).sum()) + B + 5, int(-(-int(most.max()) // PAGE)) + 1
    P, B = case["pages"], case["seqs"]
    rng = np.random.default_rng([P, B])
    share = rng.dirichlet(np.full(B, 3.0)) * (P * case["live"] - B)
    blocks = np.maximum(1, share.astype(np.int64) + 1)
    now = blocks * PAGE - rng.integers(0, PAGE, B)
    return now, now, [], P, int(blocks.max()) + 1


def _prepare_pages(case, seed):
    g = _generator(seed)
    rng = np.random.default_rng(seed)
    now, new, pairs, P, stride = _lens_of(case)
    B = len(now)
    order = rng.permutation(P).astype(np.int32)
    table, ref, at = np.full((B, stride), -1, np.int32), np.zeros(P, np.int32), 0
    for b in range(B):
        n, first = -(-int(now[b]) // PAGE), 0
        if case["op"] == "resize" and b % 8 == 3 and n and now[b - 1]:
            # a sample that shares its prompt with the one before it, in some the last page too
            first = min(n, -(-int(now[b - 1]) // PAGE))
            table[b, :first] = table[b - 1, :first]
        table[b, first:n] = order[at:at + n - first]
        at += n - first
        np.add.at(ref, table[b, :n], 1)
    free = np.sort(order[at:])[::-1]
    stack = np.zeros(P, np.int32)
    stack[:len(free)] = free
    meta = np.concatenate([table.reshape(-1), now.astype(np.int32), ref, stack, np.array([len(free), 0], np.int32)])
    s = {"pristine": torch.from_numpy(meta.astype(np.int32)).cuda(), "op": case["op"]}
    s["meta"] = s["pristine"].clone()
    cuts = np.cumsum([0, B * stride, B, P, P, 1, 1])
    parts = [s["meta"][cuts[i]:cuts[i + 1]] for i in range(6)]
    s["block_table"], s["seq_lens"], s["ref_count"], s["free_list"], s["num_free"], s["flags"] = \
        parts[0].view(B, stride), *parts[1:]
    s["new_lens"] = torch.from_numpy(new.astype(np.int32)).cuda()
    s["share"] = case.get("share", True)
    if pairs:
        mixed = rng.permutation(len(pairs))
        both = np.array(pairs, np.int32)[mixed]
        s["parents"], s["children"] = torch.from_numpy(both[:, 0].copy()).cuda(), torch.from_numpy(both[:, 1].copy()).cuda()
    s["buffers"] = []
    row = int(case["head_dim"] * CACHE_BYTES[case["kv"]])
    for _ in range(2 * case["layers"]):
        s["buffers"].append(torch.randint(-128, 128, (P, PAGE, case["kv_heads"], row), generator=g, device="cuda",
                                          dtype=torch.int8))
    if case["kv"] != "bf16":
        for _ in range(2 * case["layers"]):
            s["buffers"].append(torch.rand(P, PAGE, case["kv_heads"], generator=g, device="cuda"))
    if own:  # the handle of the cache that a user's program keeps
        import speculative_decoding_verify_causal_gb300 as va
        s["pool"] = va.PagePool(s["block_table"], s["seq_lens"], s["ref_count"], s["free_list"], s["num_free"],
                                s["buffers"], flags=s["flags"])
    return s


def prepare(case, seed):
    if case["op"] == "rope":
        s = _prepare_rope(case, seed)
    elif case["op"] == "append":
        s = _prepare_append(case, seed)
    elif case["op"] == "accept":
        s = _prepare_accept(case, seed)
    else:
        s = _prepare_pages(case, seed)
    s["case"] = dict(case)
    return s


# ---------------------------------------------------------------------------------------------
# the plain forms


def _turn(s, x, inverse):
    """The rotation of x [B, T, H, D] by its positions, in 32 bits; angles in 64, since a position
    in the hundreds of thousands leaves 32 bits few for its fraction of a turn."""
    case = s["case"]
    at = s["positions"].index_select(0, s["axis"]).permute(1, 2, 0).double() * s["inv_freq"]
    cos, sin = at.cos().float().unsqueeze(2), at.sin().float().unsqueeze(2)
    if inverse:
        sin = -sin
    r = case["rotary_dim"]
    x = x.float()
    if case["pairing"] == "half":
        a, b = x[..., :r // 2], x[..., r // 2:r]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    else:
        a, b = x[..., 0:r:2], x[..., 1:r:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    return torch.cat([turned, x[..., r:]], -1)


def _plain_rope(s):
    dt = s["q"].dtype
    inverse = s["case"]["inverse"]
    return {"q": _turn(s, s["q"], inverse).to(dt), "k": _turn(s, s["k"], inverse).to(dt)}


def _store(s, rows, pages, scale, page, slot):
    if s["kv"] == "bf16":
        pages[page, slot] = rows.to(torch.bfloat16)
        return
    top = rows.abs().amax(-1)
    by = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    codes = (rows / by.unsqueeze(-1)).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    pages[page, slot] = codes.view(torch.uint8)
    scale[page, slot] = by


def _plain_append(s):
    T = s["case"]["tokens"]
    at = (s["seq_lens"].long() - T).unsqueeze(1) + torch.arange(T, device="cuda")
    page = s["block_table"].long().gather(1, at // PAGE)
    _store(s, _turn(s, s["k"], False), s["k_pages"], s["k_scale"], page, at % PAGE)
    _store(s, s["v"].float(), s["v_pages"], s["v_scale"], page, at % PAGE)
    return _append_outputs(s, _turn(s, s["q"], False).to(torch.bfloat16))


def _append_outputs(s, q):
    """The rotated q and the cache: codes as the e4m3 values they are, and their scales."""
    kind = torch.bfloat16 if s["kv"] == "bf16" else torch.float8_e4m3fn
    return {"q": q, "k_pages": s["k_pages"].view(kind), "v_pages": s["v_pages"].view(kind), "k_scale": s["k_scale"],
            "v_scale": s["v_scale"]}


def _plain_accept(s):
    p, q, d = s["p"], s["q"], s["drafts"].long()
    B, T = d.shape
    seqs = torch.arange(B, device="cuda")
    lens = torch.full((B,), T, device="cuda") if s["lens"] is None else s["lens"].long()
    pd = p[:, :T].gather(2, d.unsqueeze(2)).squeeze(2).double()
    qd = torch.ones_like(pd) if q is None else q.gather(2, d.unsqueeze(2)).squeeze(2).double()
    good = (s["u_accept"].double() * qd < pd) & (torch.arange(T, device="cuda") < lens.unsqueeze(1))
    n = good.long().cumprod(1).sum(1)
    rejected = n < lens
    at = n.clamp(max=T - 1)
    row = p[seqs, n].double()
    if q is None:  # a point mass takes its token's probability and no other
        left = row.scatter(1, d.gather(1, at.unsqueeze(1)), 0.0)
    else:
        left = (row - q[seqs, at].double()).clamp(min=0)
    use = rejected & (left.sum(1) > 0)
    weights = torch.where(use.unsqueeze(1), left, row)
    sums = weights.cumsum(1)
    token = (sums <= s["u_emit"].double().unsqueeze(1) * sums[:, -1:]).sum(1).clamp(max=p.shape[2] - 1)
    place = torch.arange(T + 1, device="cuda")
    padded = torch.cat([d, d[:, :1]], 1)
    out = torch.where(place < n.unsqueeze(1), padded, torch.where(place == n.unsqueeze(1), token.unsqueeze(1), -1))
    return {"tokens": out.to(torch.int32), "accepted": n.to(torch.int32)}


def _pages_outputs(s):
    return {"block_table": s["block_table"], "seq_lens": s["seq_lens"], "ref_count": s["ref_count"],
            "free_list": s["free_list"], "num_free": s["num_free"], "flags": s["flags"], "buffers": s["buffers"]}


def _copy_pages(s, src, dst):
    for x in s["buffers"]:
        x[dst] = x[src]


def _plain_fork(s):
    table, lens, ref, stack, left = s["block_table"], s["seq_lens"], s["ref_count"], s["free_list"], s["num_free"]
    parent, child = s["parents"].long(), s["children"].long()
    j = torch.arange(table.shape[1], device="cuda")
    L = lens[parent].long()
    full, blocks = L // PAGE, (L + PAGE - 1) // PAGE
    rows = table[parent]
    held = j < blocks.unsqueeze(1)
    shared = j < full.unsqueeze(1) if s["share"] else torch.zeros_like(held)
    fresh = held & ~shared
    ref.index_add_(0, rows[shared].long(), torch.ones_like(rows[shared]))
    src = rows[fresh].long()
    k = torch.arange(src.numel(), device="cuda")
    dst = stack[left.long() - 1 - k].long()
    rows = torch.where(held, rows, torch.full_like(rows, -1))
    rows[fresh] = dst.to(torch.int32)
    ref[dst] = 1
    left -= src.numel()
    table[child] = rows
    lens[child] = L.to(torch.int32)
    _copy_pages(s, src, dst)
    return _pages_outputs(s)


def _release(s, pages):
    """Drops a reference of each page in the list; the pages that nobody holds any more go onto the
    stack in ascending order."""
    ref, stack, left = s["ref_count"], s["free_list"], s["num_free"]
    ref.index_add_(0, pages, torch.full_like(pages, -1, dtype=torch.int32))
    touched = torch.zeros_like(ref, dtype=torch.bool)
    touched[pages] = True
    gone = (touched & (ref == 0)).nonzero().squeeze(1)
    stack[left.long() + torch.arange(gone.numel(), device="cuda")] = gone.to(torch.int32)
    left += gone.numel()


def _plain_resize(s):
    table, lens, ref, stack, left = s["block_table"], s["seq_lens"], s["ref_count"], s["free_list"], s["num_free"]
    L, N = lens.long(), s["new_lens"].long()
    j = torch.arange(table.shape[1], device="cuda")
    old, new = ((L + PAGE - 1) // PAGE).unsqueeze(1), ((N + PAGE - 1) // PAGE).unsqueeze(1)
    drop = (j >= new) & (j < old)
    _release(s, table[drop].long())
    table[drop] = -1
    # a growing sequence that shares its partly filled last page gets a copy of its own
    last = table.gather(1, (L // PAGE).clamp(max=table.shape[1] - 1).unsqueeze(1)).squeeze(1).clamp(min=0).long()
    own_copy = (N > L) & (L % PAGE != 0) & (ref[last] > 1)
    need = (new - old).squeeze(1).clamp(min=0) + own_copy
    fits = (N <= L) | (need == 0) | (need.cumsum(0) <= left.long())
    own_copy &= fits
    take = ((j >= old) & (j < new) | own_copy.unsqueeze(1) & (j == (L // PAGE).unsqueeze(1))) & fits.unsqueeze(1)
    count = int(take.sum())
    got = stack[left.long() - 1 - torch.arange(count, device="cuda")]
    left -= count
    table[take] = got
    ref[got.long()] = 1
    src = last[own_copy]
    dst = table.gather(1, (L // PAGE).clamp(max=table.shape[1] - 1).unsqueeze(1)).squeeze(1)[own_copy].long()
    _release(s, src)
    lens.copy_(torch.where(fits, N, L))
    _copy_pages(s, src, dst)
    return _pages_outputs(s)


def _plain_compact(s):
    table, lens, ref, stack, left = s["block_table"], s["seq_lens"], s["ref_count"], s["free_list"], s["num_free"]
    P = ref.numel()
    live = ref > 0
    n = int(live.sum())
    src = live[n:].nonzero().squeeze(1) + n
    dst = (~live[:n]).nonzero().squeeze(1)
    to = torch.arange(P, device="cuda", dtype=torch.int32)
    to[src] = dst.to(torch.int32)
    held = torch.arange(table.shape[1], device="cuda") < ((lens.long() + PAGE - 1) // PAGE).unsqueeze(1)
    table[held] = to[table[held].long()]
    ref[dst] = ref[src]
    ref[src] = 0
    stack[:P - n] = torch.arange(P - 1, n - 1, -1, device="cuda", dtype=torch.int32)
    left.fill_(P - n)
    _copy_pages(s, src, dst)
    return _pages_outputs(s)


# ---------------------------------------------------------------------------------------------
# one pass


def run(state):
    s, op = state, state["case"]["op"]
    if op in ("fork", "resize", "compact"):
        s["meta"].copy_(s["pristine"])  # the table as it was before the call, for the next pass
    if not own:
        return {"rope": _plain_rope, "append": _plain_append, "accept": _plain_accept, "fork": _plain_fork,
                "resize": _plain_resize, "compact": _plain_compact}[op](s)
    import speculative_decoding_verify_causal_gb300 as va
    if op == "rope":
        q, k = va.verify_attn_rope(s["rope"], s["positions"], s["q"], s["k"], q_out=s["q_out"], k_out=s["k_out"],
                                   inverse=s["case"]["inverse"])
        return {"q": q, "k": k}
    if op == "append":
        q = va.verify_attn_rope_append(s["rope"], s["positions"], s["q"], s["k"], s["v"], s["k_pages"], s["v_pages"],
                                       s["k_scale"], s["v_scale"], s["block_table"], s["seq_lens"], s["kv"],
                                       q_out=s["q_out"], num_pages=s["num_pages"])
        return _append_outputs(s, q)
    if op == "accept":
        tokens, accepted = va.verify_attn_accept_probs(s["p"], s["drafts"], s["u_accept"], s["u_emit"],
                                                       draft_probs=s["q"], draft_lens=s["lens"],
                                                       out_tokens=s["tokens"], num_accepted=s["accepted"])
        return {"tokens": tokens, "accepted": accepted}
    if op == "fork":
        va.verify_attn_pages_fork(s["pool"], s["parents"], s["children"], share=s["share"])
    elif op == "resize":
        va.verify_attn_pages_resize(s["pool"], s["new_lens"])
    else:
        va.verify_attn_pages_compact(s["pool"])
    return _pages_outputs(s)


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without


def work(case):
    op = case["op"]
    if op == "rope":
        n = case["batch"] * case["tokens"]
        heads = case["q_heads"] + case["k_heads"]
        return {"bytes": n * (2 * heads * case["head_dim"] * FLOAT_BYTES[case["dtype"]] + 4 * case["axes"]),
                "flops": 6 * n * heads * (case["rotary_dim"] // 2)}
    if op == "append":
        n, D, Hk = case["batch"] * case["tokens"], case["head_dim"], case["kv_heads"]
        cell = int(D * CACHE_BYTES[case["kv"]]) + (0 if case["kv"] == "bf16" else 4)
        return {"bytes": n * (4 * case["q_heads"] * D + 2 * Hk * (2 * D + cell) + 4 * case["axes"] + 8),
                "flops": 6 * n * (case["q_heads"] + Hk) * (case["rotary_dim"] // 2)}
    if op == "accept":
        # one row of the target; where a model drafts, its row too at the sequences that reject
        rows = case["batch"] * (1.5 if case["model"] else 1.0)
        return {"bytes": rows * case["vocab"] * FLOAT_BYTES[case["dtype"]] + case["batch"] * case["drafts"] * 16,
                "flops": rows * case["vocab"]}
    now, new, pairs, P, stride = _lens_of(case)
    blocks = -(-now // PAGE)
    if op == "fork":
        held = int(sum(blocks[p] for p, _ in pairs))
        copied = len(pairs) if case["share"] else held
        return {"bytes": 2 * copied * _page_bytes(case) + 16 * held, "flops": 0}
    if op == "resize":
        moved = int(np.abs(-(-new // PAGE) - blocks).sum())
        return {"bytes": 16 * moved + 12 * len(now), "flops": 0}
    holes = int(blocks.sum()) * (1 - int(blocks.sum()) / P)  # of that many free places below the live count
    return {"bytes": 2 * holes * _page_bytes(case) + 12 * P + 8 * int(blocks.sum()), "flops": 0}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_turn(s, x, inverse=False):
    """Every pair as a complex number times exp(+- i angle)."""
    case, r = s["case"], s["case"]["rotary_dim"]
    pos = s["positions"].double()
    turns = torch.stack([pos[int(a)] * f for a, f in zip(s["axis"].tolist(), s["inv_freq"].tolist())], -1)
    by = torch.polar(torch.ones_like(turns), -turns if inverse else turns).unsqueeze(2)
    y = x.double().clone()
    if case["pairing"] == "half":
        z = torch.complex(y[..., :r // 2].contiguous(), y[..., r // 2:r].contiguous()) * by
        y[..., :r // 2], y[..., r // 2:r] = z.real, z.imag
    else:
        z = torch.complex(y[..., 0:r:2].contiguous(), y[..., 1:r:2].contiguous()) * by
        y[..., 0:r:2], y[..., 1:r:2] = z.real, z.imag
    return y


def _exact_append(s):
    T, B = s["case"]["tokens"], s["case"]["batch"]
    kind = torch.bfloat16 if s["kv"] == "bf16" else torch.float8_e4m3fn
    out = {"q": _exact_turn(s, s["q"])}
    lens, table = s["seq_lens"].tolist(), s["block_table"].cpu().numpy()
    at = np.array([np.arange(n - T, n) for n in lens])
    page = torch.from_numpy(np.array([table[b][at[b] // PAGE] for b in range(B)]).astype(np.int64)).cuda()
    slot = torch.from_numpy(at % PAGE).cuda()
    for name, rows in (("k", _exact_turn(s, s["k"])), ("v", s["v"].double())):
        cells = s[name + "_pages"].view(kind).double()
        if s["kv"] == "bf16":
            cells[page, slot] = rows
            out[name + "_scale"] = None
        else:
            by = rows.abs().amax(-1) / E4M3_MAX
            by = torch.where(by > 0, by, torch.ones_like(by))
            cells[page, slot] = rows / by.unsqueeze(-1)
            scale = s[name + "_scale"].double()
            scale[page, slot] = by
            out[name + "_scale"] = scale
        out[name + "_pages"] = cells
    return out


def _exact_accept(s):
    """Sequence by sequence, the decisions in the order in which they are taken."""
    p, d = s["p"].double().cpu().numpy(), s["drafts"].tolist()
    q = None if s["q"] is None else s["q"].double().cpu().numpy()
    u, v = s["u_accept"].double().tolist(), s["u_emit"].double().tolist()
    B, T = len(d), len(d[0])
    tokens, accepted = np.full((B, T + 1), -1, np.int32), np.zeros(B, np.int32)
    for b in range(B):
        count = T if s["lens"] is None else int(s["lens"][b])
        n = 0
        while n < count and u[b][n] * (1.0 if q is None else q[b, n, d[b][n]]) < p[b, n, d[b][n]]:
            tokens[b, n] = d[b][n]
            n += 1
        w = p[b, n]
        if n < count:
            without = np.zeros_like(w)
            if q is None:
                without[d[b][n]] = 1.0
            r = np.maximum(w - (without if q is None else q[b, n]), 0.0)
            w = r if r.sum() > 0 else w
        sums = np.cumsum(w)
        tokens[b, n] = min(int(np.searchsorted(sums, v[b] * sums[-1], side="right")), len(w) - 1)
        accepted[b] = n
    return {"tokens": tokens, "accepted": accepted}


def exact(case, seed):
    if case["op"] not in ("rope", "append", "accept"):
        return None  # pages are moved and counted: nothing is rounded
    s = prepare(case, seed)
    if case["op"] == "rope":
        return {"q": _exact_turn(s, s["q"], case["inverse"]), "k": _exact_turn(s, s["k"], case["inverse"])}
    return _exact_append(s) if case["op"] == "append" else _exact_accept(s)
