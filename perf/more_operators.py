"""Operators of a prompt that is worked in chunks, as they are measured: attention of ragged chunks of
new tokens over a paged cache, the attention weight that each cached token has gathered, eviction
from the cache by that weight, and log probabilities of given tokens with their place, the entropy and the
top alternatives.

``run`` computes each operator in its plain form, elementary torch operations, or, where ``own``
is true, through the package's entry points.
"""
import math

import numpy as np
import torch

own = False

PAGE = 16
FLOATS = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FLOAT_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
# bytes of one cached element; the packed caches hold two or four to a byte
CACHE_BYTES = {"bf16": 2.0, "int8": 1.0, "fp8_e4m3": 1.0, "int4": 0.5, "int2": 0.25}
CODE_MAX = {"int8": 127, "int4": 7, "int2": 1}


# ---------------------------------------------------------------------------------------------
# the cases


def listed():
    return [
        # a whole prompt in one chunk: nothing is cached before it
        {"name": "chunk_prompt", "op": "chunk", "seqs": 1, "new": 8192, "cached": 0, "singles": 0.0, "q_heads": 32,
         "kv_heads": 8, "head_dim": 128, "kv": "bf16", "fused": True},
        # the last 2,000 tokens of the 25k-token document over the tokens before them, 8-bit cache
        {"name": "chunk_document", "op": "chunk", "seqs": 1, "new": 2000, "cached": 23000, "singles": 0.0,
         "q_heads": 24, "kv_heads": 4, "head_dim": 256, "kv": "int8", "fused": False},
        # one step of a mixed batch: three quarters of the requests add one token, the others a chunk of their prompt
        {"name": "chunk_mixed", "op": "chunk", "seqs": 48, "new": 700, "cached": 6000, "singles": 0.75, "q_heads": 32,
         "kv_heads": 8, "head_dim": 128, "kv": "fp8_e4m3", "fused": True},
        # the short question behind a 1.5k-token context: latency
        {"name": "chunk_question", "op": "chunk", "seqs": 1, "new": 45, "cached": 1500, "singles": 0.0, "q_heads": 24,
         "kv_heads": 4, "head_dim": 256, "kv": "fp8_e4m3", "fused": False},
        # weights that a prompt's own tokens gather, before its cache is cut
        {"name": "weights_prompt", "op": "weights", "seqs": 1, "new": 8192, "cached": 0, "singles": 0.0, "q_heads": 32,
         "kv_heads": 8, "head_dim": 128, "kv": "bf16", "fused": True, "add": False},
        # a chunk adds to the weights of the 25k-token document
        {"name": "weights_document", "op": "weights", "seqs": 1, "new": 500, "cached": 24500, "singles": 0.0,
         "q_heads": 24, "kv_heads": 4, "head_dim": 256, "kv": "int8", "fused": False, "add": True},
        # a verify block of eight requests adds to the weights of caches held at 2,048 tokens
        {"name": "weights_blocks", "op": "weights", "seqs": 8, "new": 16, "cached": 2048, "singles": 0.0, "q_heads": 24,
         "kv_heads": 4, "head_dim": 256, "kv": "fp8_e4m3", "fused": False, "add": True},
        # after a verify block, 16 requests go back to the 2,048 tokens that each may hold
        {"name": "evict_step", "op": "evict", "seqs": 16, "tokens": 2064, "keep": 2048, "sinks": 4, "recent": 64,
         "ragged": False, "kv_heads": 8, "head_dim": 128, "kv": "bf16"},
        # four 25k-token documents are cut to a sixth
        {"name": "evict_document", "op": "evict", "seqs": 4, "tokens": 25000, "keep": 4096, "sinks": 4, "recent": 256,
         "ragged": True, "kv_heads": 4, "head_dim": 256, "kv": "int8"},
        # the tokens of one verify block with twenty alternatives each
        {"name": "logprobs_block", "op": "logprobs", "rows": 17, "vocab": 151936, "top": 20, "dtype": "fp32", "pad": 0},
        # one emitted token of each of 256 requests with five alternatives, rows of a padded vocabulary
        {"name": "logprobs_batch", "op": "logprobs", "rows": 256, "vocab": 151936, "top": 5, "dtype": "bf16", "pad": 64},
        # the log probabilities of a prompt's tokens
        {"name": "logprobs_prompt", "op": "logprobs", "rows": 2048, "vocab": 151936, "top": 1, "dtype": "bf16", "pad": 0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["chunk", "chunk", "weights", "evict", "logprobs"])
    if op in ("chunk", "weights"):
        q_heads, kv_heads = rng.choice([(4, 1), (24, 4), (32, 8), (8, 8), (28, 4), (16, 1), (40, 8)])
        head_dim = rng.choice([64, 128, 256])
        seqs = _log(rng, 1, 48)
        kv = rng.choice(["bf16", "fp8_e4m3", "int8", "int4", "int2"])
        held = int(150e6 / (seqs * kv_heads * head_dim * CACHE_BYTES[kv]))
        cached = rng.choice([0, _log(rng, 1, min(30000, held))])
        # scores of one pass: no more than those of the whole prompt
        most = 8192 * 8192 * 32 * 128 // (2 * q_heads * head_dim * seqs)
        top = int(math.sqrt(most + cached * cached / 4.0) - cached / 2.0)
        new = _log(rng, 1, max(2, min(top, 8192, held)))
        case = {"op": op, "seqs": seqs, "new": new, "cached": cached, "singles": rng.choice([0.0, 0.0, 0.5]),
                "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
                "kv": kv, "fused": rng.random() < 0.5}
        if op == "weights":
            case["add"] = rng.random() < 0.5
        return case
    if op == "evict":
        kv_heads, head_dim = rng.choice([1, 4, 8, 5]), rng.choice([64, 128, 256])
        kv = rng.choice(["bf16", "fp8_e4m3", "int8"])
        seqs = _log(rng, 1, 32)
        row = kv_heads * head_dim * CACHE_BYTES[kv]
        tokens = _log(rng, 20, max(40, min(40000, int(4 * 25000 * 4 * 256 / (row * seqs)))))
        return {"op": op, "seqs": seqs, "tokens": tokens, "keep": max(1, int(tokens * rng.choice([0.1, 0.5, 0.9, 0.99, 1.1]))),
                "sinks": rng.choice([0, 4]), "recent": rng.choice([0, 16, 200]), "ragged": rng.random() < 0.5,
                "kv_heads": kv_heads, "head_dim": head_dim, "kv": kv}
    vocab = rng.choice([1000, 32000, 50257, 128256, 151936, 200019])
    dtype = rng.choice(["bf16", "fp16", "fp32"])
    top = 2048 * 151936 * 2 // (vocab * FLOAT_BYTES[dtype])
    return {"op": op, "rows": _log(rng, 1, min(top, 5000)), "vocab": vocab, "top": rng.choice([0, 1, 5, 20, 32]),
            "dtype": dtype, "pad": rng.choice([0, 0, 64, 3])}


# ---------------------------------------------------------------------------------------------
# inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 17)
    return g


def _normal(g, *shape, dtype=torch.float32):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _lens(case):
    """(new tokens, cached tokens with the new ones) of each sequence: the same for every seed."""
    B, n, c = case["seqs"], case["new"], case["cached"]
    if B == 1:
        return np.array([n]), np.array([n + c])
    rng = np.random.default_rng([B, n, c])
    new = rng.integers(max(1, n // 2), n + 1, B)
    new = np.where(rng.random(B) < case["singles"], 1, new)
    return new, new + rng.integers(c // 2, c + 1, B)


def _table(lens, seed):
    """A block table whose pages lie in a pool in random order, and the pool's size."""
    blocks = -(-lens // PAGE)
    P = int(blocks.sum())
    order = np.random.default_rng(seed).permutation(P).astype(np.int32)
    table, at = np.zeros((len(lens), int(blocks.max())), np.int32), 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.from_numpy(table).cuda(), P


def _cells(g, P, case):
    """One pool of cached rows with their scales, quantised by each row's largest magnitude."""
    Hk, D, kv = case["kv_heads"], case["head_dim"], case["kv"]
    x = _normal(g, P, PAGE, Hk, D)
    if kv == "bf16":
        return x.to(torch.bfloat16), None
    top = x.abs().amax(-1)
    if kv == "fp8_e4m3":
        scale = top / 448.0
        return (x / scale.unsqueeze(-1)).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), scale
    scale = top / CODE_MAX[kv]
    code = (x / scale.unsqueeze(-1)).round_().clamp_(-CODE_MAX[kv], CODE_MAX[kv]).to(torch.int8)
    if kv == "int8":
        return code, scale
    per = 2 if kv == "int4" else 4
    bits, code = 8 // per, code.view(torch.uint8).view(P, PAGE, Hk, D // per, per)
    packed = torch.zeros(P, PAGE, Hk, D // per, dtype=torch.uint8, device="cuda")
    for i in range(per):
        packed |= (code[..., i] & ((1 << bits) - 1)) << (i * bits)
    return packed, scale


def _prepare_chunk(case, seed):
    g = _generator(seed)
    new, lens = _lens(case)
    Hq, Hk, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    N = int(new.sum())
    s = {"new": new, "lens": lens, "kv": case["kv"]}
    s["block_table"], P = _table(lens, seed)
    s["k_pages"], s["k_scale"] = _cells(g, P, case)
    if case["op"] == "chunk":
        s["v_pages"], s["v_scale"] = _cells(g, P, case)
    if case["fused"]:  # q, k and v side by side in one projection's output
        s["q"] = _normal(g, N, Hq + 2 * Hk, D, dtype=torch.bfloat16)[:, :Hq]
    else:
        s["q"] = _normal(g, N, Hq, D, dtype=torch.bfloat16)
    if case["op"] == "chunk":
        s["out"] = torch.empty(N, Hq, D, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.empty(N, Hq, device="cuda")
    else:
        s["lse"] = torch.cat([_scores(s, case, b)[1] for b in range(len(new))])
        s["pristine"] = torch.rand(len(new), Hk, int(lens.max()), generator=g, device="cuda") * 4
        s["weights"] = s["pristine"].clone()
    if own:  # the plan of the batch that a user's program keeps
        import speculative_decoding_verify_causal_gb300 as va
        s["plan"] = va.verify_attn_chunk_plan(new, lens, Hq, Hk, D, case["kv"])
    return s


def _evict_lens(case):
    """Cached tokens of each sequence: the same for every seed."""
    B, n = case["seqs"], case["tokens"]
    return np.random.default_rng([B, n]).integers(max(1, n * 3 // 4), n + 1, B) if case["ragged"] else np.full(B, n)


def _prepare_evict(case, seed):
    g = _generator(seed)
    lens = _evict_lens(case)
    B = len(lens)
    s = {"kv": case["kv"]}
    s["block_table"], P = _table(lens, seed)
    s["k_pages"], s["k_scale"] = _cells(g, P, case)
    s["v_pages"], s["v_scale"] = _cells(g, P, case)
    s["seq_lens"] = torch.from_numpy(lens.astype(np.int32)).cuda()
    s["keep"] = torch.from_numpy(np.minimum(case["keep"], lens + 3).astype(np.int32)).cuda()
    shape = (B, case["kv_heads"], int(lens.max()))
    # weights of attention: most tokens have gathered next to nothing, a few very much
    w = torch.exp(_normal(g, *shape) * 2 - 3)
    # a cache that was cut before: its tokens' positions in mixed order
    place = torch.rand(*shape, generator=g, device="cuda")
    place += 2 * (torch.arange(shape[2], device="cuda") >= s["seq_lens"].view(B, 1, 1))
    order = place.argsort(-1)
    s["pristine"] = w
    s["pristine_pos"] = order.to(torch.int32)
    s["weights"], s["slot_pos"] = w.clone(), s["pristine_pos"].clone()
    s["recent_from"] = torch.from_numpy((lens - case["recent"]).astype(np.int32)).cuda()
    s["new_lens"] = torch.empty(B, dtype=torch.int32, device="cuda")
    return s


def _prepare_logprobs(case, seed):
    g = _generator(seed)
    N, V, dt = case["rows"], case["vocab"], FLOATS[case["dtype"]]
    z = torch.empty(N, V + case["pad"], dtype=dt, device="cuda")
    # one token of each row stands out, in some rows by so much that the others hardly count
    three = torch.randint(0, V, (N, 3), generator=g, device="cuda")
    lift = torch.rand(N, 1, generator=g, device="cuda") * 30
    for i in range(0, N, 256):  # by pieces: no more than needed is held in 32 bits
        x = _normal(g, *z[i:i + 256].shape) * 2.5
        z[i:i + 256] = x.scatter_add_(1, three[i:i + 256, :1], lift[i:i + 256]).to(dt)
    s = {"logits": z[:, :V]}
    # a token is mostly a likely one: of three, the one with the largest logit
    best = s["logits"].gather(1, three).float().argmax(1, keepdim=True)
    s["tokens"] = three.gather(1, best).squeeze(1).to(torch.int32)
    s["top"] = case["top"]
    return s


def prepare(case, seed):
    if case["op"] in ("chunk", "weights"):
        s = _prepare_chunk(case, seed)
    elif case["op"] == "evict":
        s = _prepare_evict(case, seed)
    else:
        s = _prepare_logprobs(case, seed)
    s["case"] = dict(case)
    return s


# ---------------------------------------------------------------------------------------------
# the plain forms


def _decoded(cells, scale, kv, to):
    """Cached rows as numbers."""
    if kv == "bf16":
        return cells.to(to)
    if kv == "fp8_e4m3":
        x = cells.view(torch.float8_e4m3fn).to(to)
    elif kv == "int8":
        x = cells.to(to)
    else:
        bits = 4 if kv == "int4" else 2
        parts = [(cells >> at) & ((1 << bits) - 1) for at in range(0, 8, bits)]
        x = torch.stack(parts, -1).flatten(-2).to(to)
        x = torch.where(x >= 1 << (bits - 1), x - (1 << bits), x)
    return x * scale.to(to).unsqueeze(-1)


def _rows_of(s, name, b):
    """The cached rows of sequence b, [kv heads, tokens, D], in 32 bits."""
    n = int(s["lens"][b])
    pages = s["block_table"][b, :-(-n // PAGE)].long()
    scale = s[name + "_scale"]
    x = _decoded(s[name + "_pages"][pages], None if scale is None else scale[pages], s["kv"], torch.float32)
    return x.flatten(0, 1)[:n].transpose(0, 1).contiguous()


def _scores(s, case, b):
    """(scores with the causal mask [kv heads, new * group, tokens], log-sum-exp [new, heads]) of sequence b."""
    n, L = int(s["new"][b]), int(s["lens"][b])
    at = int(s["new"][:b].sum())
    Hq, Hk, D = case["q_heads"], case["kv_heads"], case["head_dim"]
    q = s["q"][at:at + n].float().view(n, Hk, Hq // Hk, D).permute(1, 0, 2, 3).reshape(Hk, -1, D)
    x = torch.bmm(q, _rows_of(s, "k", b).transpose(1, 2))
    x *= 1.0 / math.sqrt(D)
    token = torch.arange(n, device="cuda").repeat_interleave(Hq // Hk)
    hidden = torch.arange(L, device="cuda") > (token + (L - n)).unsqueeze(1)
    x.masked_fill_(hidden, -math.inf)
    m = x.amax(-1, keepdim=True)
    lse = (m + (x - m).exp_().sum(-1, keepdim=True).log()).squeeze(-1)
    return x, lse.view(Hk, n, Hq // Hk).permute(1, 0, 2).reshape(n, Hq)


def _packed(x, case):
    """[new, heads] as [kv heads, new * group, 1]."""
    n, Hk = x.shape[0], case["kv_heads"]
    return x.view(n, Hk, -1).permute(1, 0, 2).reshape(Hk, -1, 1)


def _plain_chunk(s):
    case, out, lse = s["case"], [], []
    for b in range(len(s["new"])):
        x, z = _scores(s, case, b)
        p = (x - _packed(z, case)).exp_()
        o = torch.bmm(p, _rows_of(s, "v", b))
        n, Hk = int(s["new"][b]), case["kv_heads"]
        out.append(o.view(Hk, n, -1, case["head_dim"]).permute(1, 0, 2, 3).reshape(n, -1, case["head_dim"]))
        lse.append(z)
    return {"out": torch.cat(out).to(torch.bfloat16), "lse": torch.cat(lse)}


def _plain_weights(s):
    case = s["case"]
    at = 0
    for b in range(len(s["new"])):
        n, L = int(s["new"][b]), int(s["lens"][b])
        x, _ = _scores(s, case, b)
        gathered = (x - _packed(s["lse"][at:at + n], case)).exp_().sum(1)
        if case["add"]:
            gathered[:, :L - n] += s["weights"][b, :, :L - n]
        s["weights"][b, :, :L] = gathered
        at += n
    return {"weights": s["weights"]}


def _evict_outputs(s, new_lens):
    cells = {"fp8_e4m3": torch.float8_e4m3fn}.get(s["kv"])
    view = (lambda x: x) if cells is None else (lambda x: x.view(cells))
    return {"k_pages": view(s["k_pages"]), "v_pages": view(s["v_pages"]), "k_scale": s["k_scale"],
            "v_scale": s["v_scale"], "weights": s["weights"], "slot_pos": s["slot_pos"], "new_lens": new_lens}


def _plain_evict(s):
    case = s["case"]
    B, Hk, stride = s["weights"].shape
    slot = torch.arange(stride, device="cuda")
    L, keep = s["seq_lens"].long().view(B, 1, 1), s["keep"].long().view(B, 1, 1)
    pos = s["slot_pos"]
    safe = (pos < case["sinks"]) | (pos >= s["recent_from"].view(B, 1, 1))
    order = torch.where(safe, math.inf, s["weights"])
    order = torch.where(slot < L, order, -math.inf)
    first = torch.sort(order, dim=-1, descending=True, stable=True).indices
    kept = torch.zeros_like(safe).scatter_(-1, first, (slot < keep).expand(B, Hk, stride).contiguous()) & (slot < L)
    # the k-th kept slot from keep on goes to the k-th slot below it that is not kept
    mover, hole = kept & (slot >= keep), ~kept & (slot < keep) & (slot < L)
    b, g, src = mover.nonzero(as_tuple=True)
    dst = hole.nonzero(as_tuple=True)[2]
    table = s["block_table"].long()
    at = (table[b, src // PAGE], src % PAGE, g)
    to = (table[b, dst // PAGE], dst % PAGE, g)
    for x in (s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"]):
        if x is not None:
            x[to] = x[at]
    for x in (s["weights"], s["slot_pos"]):
        x[b, g, dst] = x[b, g, src]
    return _evict_outputs(s, torch.minimum(s["seq_lens"], s["keep"]))


def _plain_logprobs(s):
    K = s["top"]
    parts = []
    for i in range(0, s["logits"].shape[0], 256):  # by pieces: the sort takes memory
        z = s["logits"][i:i + 256].float()
        t = s["tokens"][i:i + 256].long().unsqueeze(1)
        m = z.amax(1, keepdim=True)
        x = z - m
        e = x.exp()
        total = e.sum(1, keepdim=True, dtype=torch.float64)  # a likely token's log is what the sum has above 1
        log = total.log()
        mine = z.gather(1, t)
        index = torch.arange(z.shape[1], device="cuda")
        rank = ((z > mine) | ((z == mine) & (index < t))).sum(1)
        entropy = log - (e * x).sum(1, keepdim=True, dtype=torch.float64) / total
        top = torch.sort(z, dim=1, descending=True, stable=True)
        parts.append({"logprobs": ((mine - m).double() - log).squeeze(1).float(), "ranks": rank.to(torch.int32),
                      "entropy": entropy.squeeze(1).float(), "top_tokens": top.indices[:, :K].to(torch.int32),
                      "top_logprobs": ((top.values[:, :K] - m).double() - log).float()})
    return {name: torch.cat([p[name] for p in parts]) for name in parts[0]}


# ---------------------------------------------------------------------------------------------
# one pass


def run(state):
    s, op = state, state["case"]["op"]
    if op == "evict":  # the weights and positions as they were before the call, for the next pass
        s["weights"].copy_(s["pristine"])
        s["slot_pos"].copy_(s["pristine_pos"])
    elif op == "weights" and s["case"]["add"]:
        s["weights"].copy_(s["pristine"])
    if not own:
        return {"chunk": _plain_chunk, "weights": _plain_weights, "evict": _plain_evict,
                "logprobs": _plain_logprobs}[op](s)
    import speculative_decoding_verify_causal_gb300 as va
    if op == "chunk":
        out, lse = va.verify_attn_chunk(s["plan"], s["q"], s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"],
                                        s["block_table"], out=s["out"], lse=s["lse"])
        return {"out": out, "lse": lse}
    if op == "weights":
        va.verify_attn_chunk_weights(s["plan"], s["q"], s["k_pages"], s["k_scale"], s["block_table"], s["lse"],
                                     s["weights"], accumulate=s["case"]["add"])
        return {"weights": s["weights"]}
    if op == "evict":
        new_lens = va.verify_attn_evict(s["k_pages"], s["v_pages"], s["k_scale"], s["v_scale"], s["block_table"],
                                        s["seq_lens"], s["weights"], s["keep"], s["kv"], slot_pos=s["slot_pos"],
                                        num_sinks=s["case"]["sinks"], recent_from=s["recent_from"],
                                        new_lens=s["new_lens"])
        return _evict_outputs(s, new_lens)
    logprobs, ranks, entropy, top_tokens, top_logprobs = va.verify_attn_logprobs(s["logits"], s["tokens"],
                                                                                 num_top=s["top"])
    return {"logprobs": logprobs, "ranks": ranks, "entropy": entropy, "top_tokens": top_tokens,
            "top_logprobs": top_logprobs}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without


def _row_bytes(case):
    """Bytes of one cached row of one kv head, its scale with it."""
    return int(case["head_dim"] * CACHE_BYTES[case["kv"]]) + (0 if case["kv"] == "bf16" else 4)


def work(case):
    op = case["op"]
    if op in ("chunk", "weights"):
        new, lens = _lens(case)
        pairs = int((new * (lens - new) + new * (new + 1) // 2).sum())
        N, cached, Hq, D = int(new.sum()), int(lens.sum()), case["q_heads"], case["head_dim"]
        rows = cached * case["kv_heads"]
        if op == "chunk":
            return {"bytes": N * Hq * (4 * D + 4) + 2 * rows * _row_bytes(case), "flops": 4 * pairs * Hq * D}
        return {"bytes": N * Hq * (2 * D + 4) + rows * (_row_bytes(case) + (8 if case["add"] else 4)),
                "flops": 2 * pairs * Hq * D}
    if op == "evict":
        lens = _evict_lens(case)
        keep = np.minimum(case["keep"], lens)
        moved = keep * (lens - keep) / lens  # of the kept tokens, the share that lies behind the first keep
        return {"bytes": int(case["kv_heads"] * (8 * lens.sum() + moved.sum() * 2 * (2 * _row_bytes(case) + 8))), "flops": 0}
    n = case["rows"] * case["vocab"]
    return {"bytes": n * FLOAT_BYTES[case["dtype"]] + case["rows"] * (16 + 8 * case["top"]), "flops": 4 * n}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits


def _exact_attention(s, case, b, at):
    """Sequence b head by head: (weights [new, tokens], log-sum-exp [new]) of every query head, in order."""
    n, L, D = int(s["new"][b]), int(s["lens"][b]), case["head_dim"]
    G = case["q_heads"] // case["kv_heads"]
    where = torch.arange(L, device="cuda")
    page, slot = s["block_table"][b].long()[where // PAGE], where % PAGE
    seen = where <= (torch.arange(n, device="cuda") + L - n)[:, None]
    for h in range(case["q_heads"]):
        scale = None if s["k_scale"] is None else s["k_scale"][page, slot, h // G]
        keys = _decoded(s["k_pages"][page, slot, h // G], scale, s["kv"], torch.float64)
        x = s["q"][at:at + n, h].double() @ keys.T / math.sqrt(D)
        lse = torch.logsumexp(torch.where(seen, x, -math.inf), -1)
        yield h, torch.where(seen, (x - lse[:, None]).exp(), 0.0), lse, x, seen, (page, slot)


def _exact_chunk(s, case):
    new = s["new"]
    N, Hq, D = int(new.sum()), case["q_heads"], case["head_dim"]
    G = Hq // case["kv_heads"]
    out = torch.empty(N, Hq, D, dtype=torch.float64, device="cuda")
    lses = torch.empty(N, Hq, dtype=torch.float64, device="cuda")
    at = 0
    for b in range(len(new)):
        n = int(new[b])
        for h, p, lse, _, _, (page, slot) in _exact_attention(s, case, b, at):
            scale = None if s["v_scale"] is None else s["v_scale"][page, slot, h // G]
            out[at:at + n, h] = p @ _decoded(s["v_pages"][page, slot, h // G], scale, s["kv"], torch.float64)
            lses[at:at + n, h] = lse
        at += n
    return {"out": out, "lse": lses}


def _exact_weights(s, case):
    w = s["pristine"].double()
    G, at = case["q_heads"] // case["kv_heads"], 0
    for b in range(len(s["new"])):
        n, L = int(s["new"][b]), int(s["lens"][b])
        w[b, :, (L - n if case["add"] else 0):L] = 0.0
        for h, _, _, x, seen, _ in _exact_attention(s, case, b, at):
            given = s["lse"][at:at + n, h].double()[:, None]
            w[b, h // G, :L] += torch.where(seen, (x - given).exp(), 0.0).sum(0)
        at += n
    return {"weights": w}


def _exact_logprobs(s, case):
    z, K = s["logits"], case["top"]
    out = {k: [] for k in ("logprobs", "ranks", "entropy", "top_tokens", "top_logprobs")}
    index = torch.arange(z.shape[1], device="cuda")
    for i in range(0, z.shape[0], 128):
        x = z[i:i + 128].double()
        t = s["tokens"][i:i + 128].long()[:, None]
        high = x.amax(1, keepdim=True)
        x = x - high
        rest = x.exp()
        rest[torch.arange(x.shape[0], device="cuda"), x.argmax(1)] = 0.0  # all but one of the largest
        rest = rest.sum(1, keepdim=True)
        lp = x - torch.log1p(rest)
        bits = (z[i:i + 128].float() + 0.0).view(torch.int32).long()
        key = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits) * (1 << 32) + (z.shape[1] - 1 - index)
        out["logprobs"].append(lp.gather(1, t).squeeze(1))
        out["ranks"].append((key > key.gather(1, t)).sum(1).to(torch.int32))
        out["entropy"].append(-(lp.exp() * lp).sum(1))
        best = key.topk(K, 1).indices
        out["top_tokens"].append(best.to(torch.int32))
        out["top_logprobs"].append(lp.gather(1, best))
    return {k: torch.cat(v) for k, v in out.items()}


def exact(case, seed):
    if case["op"] == "evict":
        return None  # tokens are ordered and moved: nothing is rounded
    s = prepare(case, seed)
    if case["op"] == "chunk":
        return _exact_chunk(s, case)
    return _exact_weights(s, case) if case["op"] == "weights" else _exact_logprobs(s, case)
