"""Cases, plain forms and exact values of three serving operators over the paged KV cache:

  plan    block tables, slots, start locations and positions of a step, built on the GPU from the
          requests' lengths (ops.build_step)
  rotary  rotary positions with several axes on q and k, and the slot scatter of k and v
          (ops.rotary_reshape_and_cache, ops.rotary_reshape_and_cache_fp8)
  window  attention with a sliding window and sink tokens over the paged cache, decode rows and
          prompt chunks (ops.paged_attention_window, ops.paged_attention_window_fp8)

`run` computes a case in its plain form (elementary torch operations) where `own` is false, and by
the framework's operators where it is true.  Both take what `prepare` gives.
"""
import math
import random

import numpy as np
import torch

own = False

PAGE = 16       # tokens of a page of the 8-bit cache
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------- cases
def listed():
    heads = {"n_q": 32, "n_kv": 8, "d": 128, "block": 16}
    return [
        # a decode step of 64 running requests: the smallest call, all latency
        {"name": "plan_decode_64", "op": "plan", "decodes": 64, "ctx_lo": 128, "ctx_hi": 4096,
         "chunks": 0, "chunk_lo": 0, "chunk_hi": 0, "chunk_ctx": 0, "block": 16, "axes": 1,
         "pad": 0},
        # 256 running requests, a quarter of them with prompt slices, image positions (three
        # axes), token arrays padded to a captured graph's maximum
        {"name": "plan_prompts_256", "op": "plan", "decodes": 191, "ctx_lo": 64, "ctx_hi": 8192,
         "chunks": 65, "chunk_lo": 64, "chunk_hi": 512, "chunk_ctx": 7680, "block": 16, "axes": 3,
         "pad": 1024},
        # four decode tokens of a small model, plain text positions
        {"name": "rotary_tiny_4", "op": "rotary", "tokens": 4, "pad": 0, "n_q": 4, "n_kv": 2,
         "d": 64, "rot": 64, "axes": 1, "cycle": False, "interleaved": False, "packed": False,
         "cache": "bf16", "block": 16, "far": 4096},
        # a decode step of 64 requests, q, k and v as slices of one projection's output
        {"name": "rotary_decode_64", "op": "rotary", "tokens": 64, "pad": 0, **heads, "rot": 128,
         "axes": 3, "cycle": False, "interleaved": False, "packed": True, "cache": "bf16",
         "far": 32768},
        # a full step under a 2048-token budget, padded tail, frequencies dealt to the axes in turn
        {"name": "rotary_step_2048", "op": "rotary", "tokens": 2048, "pad": 37, **heads,
         "rot": 128, "axes": 3, "cycle": True, "interleaved": False, "packed": True,
         "cache": "bf16", "far": 32768},
        # a long image or video prompt into the 8-bit cache, an odd token count
        {"name": "rotary_prompt_8191_fp8", "op": "rotary", "tokens": 8191, "pad": 0, **heads,
         "rot": 128, "axes": 3, "cycle": False, "interleaved": False, "packed": True,
         "cache": "fp8", "far": 131072},
        # half of each head rotated, neighbouring elements paired, 32-token blocks
        {"name": "rotary_partial_4099", "op": "rotary", "tokens": 4099, "pad": 0, "n_q": 16,
         "n_kv": 4, "d": 64, "rot": 32, "axes": 2, "cycle": False, "interleaved": True,
         "packed": False, "cache": "bf16", "block": 32, "far": 1 << 20},
        # four short requests of a small model, a window shorter than most of them
        {"name": "window_tiny_4", "op": "window", "decodes": 4, "ctx_lo": 5, "ctx_hi": 48,
         "chunks": 0, "chunk_lo": 0, "chunk_hi": 0, "chunk_ctx": 0, "n_q": 4, "n_kv": 2, "d": 64,
         "block": 16, "window": 20, "sinks": 4, "cache": "bf16"},
        # a decode step of 64 requests of mixed lengths
        {"name": "window_decode_64", "op": "window", "decodes": 64, "ctx_lo": 128, "ctx_hi": 4096,
         "chunks": 0, "chunk_lo": 0, "chunk_hi": 0, "chunk_ctx": 0, **heads, "window": 1024,
         "sinks": 4, "cache": "bf16"},
        # long contexts in the 8-bit cache: eight decodes at 32768 tokens beside two slices
        {"name": "window_long_fp8", "op": "window", "decodes": 8, "ctx_lo": 32767,
         "ctx_hi": 32767, "chunks": 2, "chunk_lo": 509, "chunk_hi": 512, "chunk_ctx": 16384,
         **heads, "window": 4096, "sinks": 64, "cache": "fp8"},
        # a mixed step: 128 decodes beside one 512-token slice
        {"name": "window_mixed_640", "op": "window", "decodes": 128, "ctx_lo": 256,
         "ctx_hi": 2048, "chunks": 1, "chunk_lo": 512, "chunk_hi": 512, "chunk_ctx": 3584,
         **heads, "window": 1024, "sinks": 4, "cache": "bf16"},
        # a long prompt in one call, as an offline run has it
        {"name": "window_prompt_8192", "op": "window", "decodes": 0, "ctx_lo": 0, "ctx_hi": 0,
         "chunks": 1, "chunk_lo": 8192, "chunk_hi": 8192, "chunk_ctx": 4096, **heads,
         "window": 4096, "sinks": 4, "cache": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm, odd ones as likely as even."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50.0)


def draw(rng):
    most = max(_cost(c) for c in listed())
    while True:
        op = rng.choice(["plan", "rotary", "rotary", "window", "window", "window"])
        block = rng.choice([16, 16, 32])
        if op == "plan":
            case = {"op": op, "decodes": _spread(rng, 1, 700), "ctx_lo": _spread(rng, 1, 512),
                    "ctx_hi": _spread(rng, 512, 32768), "chunks": rng.choice([0, 1, 2, 7, 33, 64]),
                    "chunk_lo": _spread(rng, 2, 256), "chunk_hi": _spread(rng, 256, 2048),
                    "chunk_ctx": rng.choice([0, 1, 511, 4096, _spread(rng, 1, 16384)]),
                    "block": block, "axes": rng.choice([1, 2, 3, 4]),
                    "pad": rng.choice([0, 1, _spread(rng, 1, 4096)])}
            return case
        n_kv, group, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        cache = rng.choice(["bf16", "fp8"])
        heads = {"n_q": n_kv * group, "n_kv": n_kv, "d": d, "block": block, "cache": cache}
        if op == "rotary":
            case = {"op": op, "tokens": _spread(rng, 1, 16384), "pad": rng.choice([0, 0, 3, 33]),
                    **heads, "rot": rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d]),
                    "axes": rng.choice([1, 2, 3, 4]), "cycle": rng.random() < 0.5,
                    "interleaved": rng.random() < 0.5, "packed": rng.random() < 0.5,
                    "far": rng.choice([4096, 32768, 131072, 1 << 20])}
        else:
            kind = rng.choice(["decode", "chunk", "mixed"])
            decodes = 0 if kind == "chunk" else _spread(rng, 1, 300)
            chunks = 0 if kind == "decode" else rng.choice([1, 1, 2, 5])
            lo, hi = sorted((_spread(rng, 1, 16384), _spread(rng, 1, 16384)))
            clo, chi = sorted((_spread(rng, 2, 2048), _spread(rng, 2, 2048)))
            case = {"op": op, "decodes": decodes, "ctx_lo": lo, "ctx_hi": hi, "chunks": chunks,
                    "chunk_lo": clo if chunks else 0, "chunk_hi": chi if chunks else 0,
                    "chunk_ctx": rng.choice([0, 1, 777, _spread(rng, 1, 16384)]) if chunks else 0,
                    **heads, "window": _spread(rng, 1, 8192),
                    "sinks": rng.choice([0, 1, 4, 16, 100])}
        if _cost(case) <= most:
            return case


def _even(lo, hi, n):
    """n whole numbers from lo to hi at even distances."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _lengths(case):
    """(tokens in the cache, new tokens) of each request, decodes first.  For the attention a
    request's new tokens are in the cache already; for the plan they are about to be."""
    new = _even(case["chunk_lo"], case["chunk_hi"], case["chunks"])
    ctx = _even(case["ctx_lo"], case["ctx_hi"], case["decodes"])
    return (ctx + _even(case["chunk_ctx"] // 2, case["chunk_ctx"], case["chunks"]),
            [1] * case["decodes"] + new)


def _blocks(n, block):
    return -(-n // block)


# ----------------------------------------------------------------------------------- inputs
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _quantised(x, block):
    """Rows x [slots, n_kv, d] as an 8-bit cache: pages of 16 rows' codes, then their scales."""
    slots, n_kv, d = x.shape
    x = x.float()
    top = x.abs().amax(-1)
    scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
    codes = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
    pages = torch.cat([codes.view(slots // PAGE, -1),
                       scale.view(slots // PAGE, -1).contiguous().view(torch.uint8)], 1)
    return pages.view(slots // block, block // PAGE, -1)


def _codes_scales(cache, n_kv, d):
    """Views of an 8-bit cache: codes [blocks, pages, 16 n_kv d] and scales [.., 16 n_kv]."""
    n = PAGE * n_kv * d
    return cache[:, :, :n].view(torch.float8_e4m3fn), cache[:, :, n:].view(torch.float32)


def prepare(case, seed):
    op = case["op"]
    rng = random.Random(seed)
    g = _generator(seed)
    s = {"case": dict(case)}
    if op == "plan":
        ctx, new = _lengths(case)
        order = list(range(len(ctx)))
        rng.shuffle(order)
        ctx, new = [ctx[i] for i in order], [new[i] for i in order]
        block = case["block"]
        total = [_blocks(c + n, block) for c, n in zip(ctx, new)]
        pool = sum(total) + 64
        width = max(total)
        ids = np.random.default_rng(seed).permutation(pool).astype(np.int32)
        tables = np.full((len(ctx), width), -1, np.int32)
        at = 0
        for i, c in enumerate(ctx):
            n = _blocks(c, block)
            tables[i, :n] = ids[at:at + n]
            at += n
        free = np.full(pool, -1, np.int32)
        free[:pool - at] = ids[at:]
        offsets = [rng.randint(-min(c, 600), 0) for c in ctx]  # text after images counts less
        s.update(context_lens=_int32(ctx), new_lens=_int32(new), offsets=_int32(offsets),
                 tables=torch.from_numpy(tables).cuda(), free=torch.from_numpy(free).cuda(),
                 count=_int32([pool - at]), count_out=_int32([0]), pool=pool,
                 tokens=sum(new) + case["pad"])
        return s
    n_q, n_kv, d, block = case["n_q"], case["n_kv"], case["d"], case["block"]
    if op == "rotary":
        T, rot, axes = case["tokens"], case["rot"], case["axes"]
        wide = (n_q + 2 * n_kv) * d
        if case["packed"]:
            qkv = torch.randn(T, wide, device="cuda", dtype=torch.bfloat16, generator=g)
            parts = qkv.split([n_q * d, n_kv * d, n_kv * d], 1)
        else:
            parts = [torch.randn(T, n * d, device="cuda", dtype=torch.bfloat16, generator=g)
                     for n in (n_q, n_kv, n_kv)]
        s["q"], s["k"], s["v"] = (p.view(T, -1, d) for p in parts)
        first = torch.randint(0, case["far"], (1,), device="cuda", generator=g, dtype=torch.int32)
        steps = torch.arange(T, device="cuda", dtype=torch.int32)
        rows = [(first + steps) % case["far"]]
        rows += [torch.randint(0, case["far"], (T,), device="cuda", generator=g,
                               dtype=torch.int32) for _ in range(axes - 1)]
        s["positions"] = torch.stack(rows)
        i = torch.arange(rot // 2, dtype=torch.float64)
        s["inv_freq"] = (10000.0 ** (-2.0 * i / rot)).cuda()
        if case["cycle"]:
            of = [j % axes for j in range(rot // 2)]
        else:
            of = [j * axes // (rot // 2) for j in range(rot // 2)]
        s["axes"] = _int32(of)
        blocks = _blocks(T, block) + 3
        slots = torch.randperm(blocks * block, device="cuda", generator=g)[:T].to(torch.int32)
        if case["pad"]:
            slots[max(0, T - case["pad"]):] = -1
        s["slots"] = slots
        if case["cache"] == "bf16":
            shape, kind = (blocks, block, n_kv, d), torch.bfloat16
        else:
            shape, kind = (blocks, block // PAGE, PAGE * n_kv * (d + 4)), torch.uint8
        s["k_cache"] = torch.zeros(shape, dtype=kind, device="cuda")
        s["v_cache"] = torch.zeros(shape, dtype=kind, device="cuda")
        s["q_out"] = torch.empty(T, n_q, d, dtype=torch.bfloat16, device="cuda")
        return s
    # window: the blocks that no row of a request sees any more have been handed on
    ctx, new = _lengths(case)
    order = list(range(len(ctx)))
    rng.shuffle(order)
    ctx, new = [ctx[i] for i in order], [new[i] for i in order]
    lens = [c + n for c, n in zip(ctx, new)]
    width = max(_blocks(n, block) for n in lens)
    live = np.zeros((len(lens), width), bool)
    for i, (c, n) in enumerate(zip(ctx, lens)):
        live[i, :min(_blocks(case["sinks"], block), _blocks(n, block))] = True
        live[i, max(0, c - case["window"] + 1) // block:_blocks(n, block)] = True
    blocks = int(live.sum()) + 5
    ids = np.random.default_rng(seed).permutation(blocks).astype(np.int32)
    tables = np.full(live.shape, -1, np.int32)
    tables[live] = ids[:int(live.sum())]
    starts = np.concatenate([[0], np.cumsum(new)])
    s["tables"] = torch.from_numpy(tables).cuda()
    s["seq_lens"], s["starts"] = _int32(lens), _int32(starts.tolist())
    s["is_chunk"] = [n > 1 for n in new]
    s["max_q_len"], s["max_seq_len"] = max(new), max(lens)
    s["min_q_len"] = min(new)
    s["scale"] = 1.0 / math.sqrt(d)
    T = sum(new)
    s["q"] = torch.randn(T, n_q, d, device="cuda", dtype=torch.bfloat16, generator=g)
    rows = [torch.randn(blocks * block, n_kv, d, device="cuda", dtype=torch.bfloat16,
                        generator=g) for _ in range(2)]
    if case["cache"] == "bf16":
        s["k_cache"], s["v_cache"] = (r.view(blocks, block, n_kv, d) for r in rows)
    else:
        s["k_cache"], s["v_cache"] = (_quantised(r, block) for r in rows)
    s["out"] = torch.empty_like(s["q"])
    if own:  # the scratch buffer that a serving loop holds for all its calls
        from paged_kv_cache_174_gb300 import ops
        s["workspace"] = ops.alloc_workspace(len(lens), T, n_q, n_kv, d, s["max_q_len"],
                                             s["max_seq_len"], "cuda")
    return s


# -------------------------------------------------------------------------------------- run
def run(state):
    case = state["case"]
    if own:
        return {"plan": _own_plan, "rotary": _own_rotary, "window": _own_window}[case["op"]](state)
    return {"plan": _plain_plan, "rotary": _plain_rotary,
            "window": _plain_window}[case["op"]](state)


def _own_plan(s):
    from paged_kv_cache_174_gb300 import ops
    lens, starts, slots, positions = ops.build_step(
        s["context_lens"], s["new_lens"], s["tables"], s["free"], s["count"],
        block_size=s["case"]["block"], num_tokens=s["tokens"], num_axes=s["case"]["axes"],
        position_offsets=s["offsets"], free_count_out=s["count_out"])
    return {"tables": s["tables"], "count": s["count_out"], "lens": lens, "starts": starts,
            "slots": slots, "positions": positions}


def _plain_plan(s):
    block, axes, T = s["case"]["block"], s["case"]["axes"], s["tokens"]
    ctx, new = s["context_lens"].long(), s["new_lens"].long()
    first = (ctx + block - 1) // block
    need = (ctx + new + block - 1) // block - first
    ends_b, ends_t = need.cumsum(0), new.cumsum(0)
    served = (ends_b <= s["count"]) & (ends_t <= T)
    new, need = new * served, need * served
    ends_b, ends_t = need.cumsum(0), new.cumsum(0)
    column = torch.arange(s["tables"].shape[1], device=ctx.device)
    nth = (ends_b - need)[:, None] + column - first[:, None]
    fresh = (column >= first[:, None]) & (column < (first + need)[:, None])
    popped = s["free"][(s["count"] - 1 - nth).clamp(0, s["free"].numel() - 1)]
    tables = torch.where(fresh, popped, s["tables"])
    token = torch.arange(T, device=ctx.device)
    owner = torch.searchsorted(ends_t, token, right=True)
    real = owner < ctx.numel()
    owner = owner.clamp(max=ctx.numel() - 1)
    pos = ctx[owner] + token - (ends_t - new)[owner]
    slots = tables[owner, (pos // block).clamp(max=tables.shape[1] - 1)] * block + pos % block
    slots = torch.where(real, slots, -1).int()
    positions = torch.where(real, pos + s["offsets"][owner], 0).int().expand(axes, T).contiguous()
    starts = torch.cat([ends_t.new_zeros(1), ends_t]).int()
    count = (s["count"] - need.sum()).int()
    return {"tables": tables, "count": count, "lens": (ctx + new).int(), "starts": starts,
            "slots": slots, "positions": positions}


def _written(s):
    """The caches as run() returns them: bf16 rows, or codes and scales."""
    case = s["case"]
    if case["cache"] == "bf16":
        return {"k": s["k_cache"], "v": s["v_cache"]}
    k, ks = _codes_scales(s["k_cache"], case["n_kv"], case["d"])
    v, vs = _codes_scales(s["v_cache"], case["n_kv"], case["d"])
    return {"k": k, "k_scale": ks, "v": v, "v_scale": vs}


def _own_rotary(s):
    from paged_kv_cache_174_gb300 import ops
    case = s["case"]
    call = ops.rotary_reshape_and_cache if case["cache"] == "bf16" else \
        ops.rotary_reshape_and_cache_fp8
    q = call(s["q"], s["k"], s["v"], s["positions"], s["inv_freq"], s["k_cache"], s["v_cache"],
             s["slots"], axes=s["axes"], interleaved=case["interleaved"], q_out=s["q_out"])
    return {"q": q, **_written(s)}


def _plain_rotated(x, cos, sin, rot, interleaved):
    x = x.float()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rotary(s):
    case = s["case"]
    rot, n_kv, d, block = case["rot"], case["n_kv"], case["d"], case["block"]
    angle = s["positions"][s["axes"].long()].t().double() * s["inv_freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    q = _plain_rotated(s["q"], cos, sin, rot, case["interleaved"]).bfloat16()
    k = _plain_rotated(s["k"], cos, sin, rot, case["interleaved"])
    v = s["v"].float()
    blocks = s["k_cache"].shape[0]
    # one row more than the pool has: where the tokens without a slot go
    slot = torch.where(s["slots"] >= 0, s["slots"].long(), blocks * block)
    if case["cache"] == "bf16":
        def put(cache, rows):
            whole = torch.cat([cache.view(-1, n_kv, d), cache.new_zeros(1, n_kv, d)])
            whole[slot] = rows.bfloat16()
            cache.copy_(whole[:-1].view_as(cache))
    else:
        def put(cache, rows):
            codes, scales = _codes_scales(cache, n_kv, d)
            top = rows.abs().amax(-1)
            scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
            code = (rows / scale[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
            whole = torch.cat([codes.view(torch.uint8).reshape(-1, n_kv, d),
                               cache.new_zeros(1, n_kv, d)])
            whole[slot] = code.to(torch.float8_e4m3fn).view(torch.uint8)
            codes.view(torch.uint8).copy_(whole[:-1].view(codes.shape))
            whole = torch.cat([scales.reshape(-1, n_kv), scales.new_zeros(1, n_kv)])
            whole[slot] = scale
            scales.copy_(whole[:-1].view(scales.shape))
    put(s["k_cache"], k)
    put(s["v_cache"], v)
    return {"q": q, **_written(s)}


def _own_window(s):
    from paged_kv_cache_174_gb300 import ops
    case = s["case"]
    call = ops.paged_attention_window if case["cache"] == "bf16" else \
        ops.paged_attention_window_fp8
    return call(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["seq_lens"], s["starts"],
                s["scale"], window=case["window"], num_sinks=case["sinks"],
                min_q_len=s["min_q_len"], max_q_len=s["max_q_len"],
                max_seq_len=s["max_seq_len"], out=s["out"], workspace=s["workspace"])


def _plain_rows(cache, slot, case):
    """Rows of the cache at these slots, in 32 bits."""
    n_kv, d = case["n_kv"], case["d"]
    if case["cache"] == "bf16":
        return cache.view(-1, n_kv, d)[slot].float()
    codes, scales = _codes_scales(cache, n_kv, d)
    code = codes.view(torch.uint8).reshape(-1, n_kv, d)[slot].view(torch.float8_e4m3fn).float()
    return code * scales.reshape(-1, n_kv)[slot][..., None]


def _plain_group(s, which, most, out):
    """The rows of the requests `which`, each with at most `most` of them, into out [T + 1, ...]."""
    case = s["case"]
    n_kv, d, block, W, N = (case[x] for x in ("n_kv", "d", "block", "window", "sinks"))
    which = torch.tensor(which, device="cuda")
    R, T = which.numel(), s["q"].shape[0]
    length = s["seq_lens"][which].long()[:, None]
    begin = s["starts"][which].long()[:, None]
    rows = s["starts"][which + 1].long()[:, None] - begin
    first = (length - rows - W + 1).clamp(min=N)
    span = min(W - 1 + most, s["max_seq_len"])
    key = torch.cat([torch.arange(N, device="cuda").expand(R, N),
                     first + torch.arange(span, device="cuda")], 1)
    there = key < length
    column = (key // block).clamp(max=s["tables"].shape[1] - 1)
    slot = s["tables"][which].gather(1, column).long().clamp(min=0) * block + key % block
    K = _plain_rows(s["k_cache"], slot, case)
    V = _plain_rows(s["v_cache"], slot, case)
    i = torch.arange(most, device="cuda")
    pos = length - rows + i
    token = torch.where(i < rows, begin + i, T)
    q = s["q"][token.clamp(max=T - 1)].float().view(R, most, n_kv, -1, d)
    score = torch.einsum("rmgcd,rkgd->rgcmk", q, K).mul_(s["scale"])
    gap = pos[:, :, None] - key[:, None, :]
    seen = there[:, None, :] & (gap >= 0) & ((gap < W) | (key < N)[:, None, :])
    score.masked_fill_(~seen[:, None, None], -math.inf)
    score.sub_(score.amax(-1, keepdim=True)).exp_()
    total = score.sum(-1)
    o = torch.einsum("rgcmk,rkgd->rmgcd", score, V)
    o = o / total.permute(0, 3, 1, 2)[..., None]
    out[token] = o.reshape(R, most, -1, d).to(out.dtype)


def _plain_window(s):
    out = s["q"].new_zeros((s["q"].shape[0] + 1,) + s["q"].shape[1:])
    one = [i for i, c in enumerate(s["is_chunk"]) if not c]
    many = [i for i, c in enumerate(s["is_chunk"]) if c]
    if one:
        _plain_group(s, one, 1, out)
    if many:
        _plain_group(s, many, s["max_q_len"], out)
    return out[:-1]


# ------------------------------------------------------------------------------------- work
def work(case):
    if case["op"] == "plan":
        ctx, new = _lengths(case)
        S, T, block = len(ctx), sum(new) + case["pad"], case["block"]
        fresh = sum(_blocks(c + n, block) - _blocks(c, block) for c, n in zip(ctx, new))
        partial = sum(c % block > 0 for c in ctx)
        read = 4 * (3 * S + partial + fresh + 1)
        return {"bytes": read + 4 * (fresh + 2 * S + 2 + T * (1 + case["axes"])), "flops": 0}
    n_q, n_kv, d = case["n_q"], case["n_kv"], case["d"]
    row = 2 * d if case["cache"] == "bf16" else d + 4
    if case["op"] == "rotary":
        T = case["tokens"]
        kept = max(0, T - case["pad"])
        data = T * (2 * n_q + n_kv) * d * 2 + kept * n_kv * (d * 2 + 2 * row)
        return {"bytes": data + 4 * T * (1 + case["axes"]) + 6 * case["rot"],
                "flops": 3 * case["rot"] * T * (n_q + n_kv)}
    ctx, new = _lengths(case)
    W, N = case["window"], case["sinks"]
    keys = pairs = 0
    for c, n in zip(ctx, new):
        keys += (c + n) - max(0, c - W + 1) + min(N, max(0, c - W + 1))
        p = np.arange(c, c + n)
        out_of_window = np.maximum(0, p - W + 1)
        pairs += int((p + 1 - out_of_window + np.minimum(N, out_of_window)).sum())
    T = sum(new)
    return {"bytes": 2 * keys * n_kv * row + 2 * T * n_q * d * 2 + 8 * len(ctx)
            + 4 * _blocks(keys, case["block"]),
            "flops": 4 * d * n_q * pairs}


# ------------------------------------------------------------------------------------ exact
def _e4m3(x):
    """The nearest E4M3 values of x (64 bits), ties to the even code."""
    size = x.abs().clamp(min=2.0 ** -6)
    step = torch.exp2(torch.floor(torch.log2(size)) - 3)
    return (torch.round(x / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def exact(case, seed):
    s = prepare(case, seed)
    return {"plan": _exact_plan, "rotary": _exact_rotary, "window": _exact_window}[case["op"]](s)


def _exact_plan(s):
    block, T, axes = s["case"]["block"], s["tokens"], s["case"]["axes"]
    ctx, new, off = (s[x].tolist() for x in ("context_lens", "new_lens", "offsets"))
    tables = s["tables"].cpu().numpy().copy()
    free = s["free"].tolist()[:int(s["count"])]
    slots, positions = np.full(T, -1, np.int32), np.zeros((axes, T), np.int32)
    starts, lens, t, open_ = [0], [], 0, True
    for i, (c, n) in enumerate(zip(ctx, new)):
        fresh = _blocks(c + n, block) - _blocks(c, block)
        open_ = open_ and fresh <= len(free) and t + n <= T
        if open_:
            for j in range(fresh):
                tables[i, _blocks(c, block) + j] = free.pop()
            for p in range(c, c + n):
                slots[t] = tables[i, p // block] * block + p % block
                positions[:, t] = p + off[i]
                t += 1
        starts.append(t)
        lens.append(c + n if open_ else c)
    return {"tables": tables, "count": np.array([len(free)], np.int32),
            "lens": np.array(lens, np.int32), "starts": np.array(starts, np.int32),
            "slots": slots, "positions": positions}


def _exact_rotary(s):
    case = s["case"]
    rot, n_kv, d, block, half = case["rot"], case["n_kv"], case["d"], case["block"], \
        case["rot"] // 2
    theta = torch.stack([s["positions"][a].double() * f
                         for a, f in zip(s["axes"].tolist(), s["inv_freq"])], 1)
    turn = torch.complex(theta.cos(), theta.sin())[:, None, :]
    lo = torch.arange(half, device="cuda")
    one, two = (2 * lo, 2 * lo + 1) if case["interleaved"] else (lo, lo + half)

    def turned(x):
        y = x.double().clone()
        z = torch.complex(y[..., one], y[..., two]) * turn
        y[..., one], y[..., two] = z.real, z.imag
        return y
    blocks = s["k_cache"].shape[0]
    at = torch.nonzero(s["slots"] >= 0)[:, 0]
    slot = s["slots"][at].long()
    found = {"q": turned(s["q"])}
    for name, rows in (("k", turned(s["k"])), ("v", s["v"].double())):
        rows = rows[at]
        if case["cache"] == "bf16":
            whole = torch.zeros(blocks * block, n_kv, d, dtype=torch.float64, device="cuda")
            whole[slot] = rows
            found[name] = whole.view(blocks, block, n_kv, d)
            continue
        scale = rows.abs().amax(-1) / E4M3_MAX
        scale[scale == 0] = 1.0
        codes = torch.zeros(blocks * block, n_kv, d, dtype=torch.float64, device="cuda")
        codes[slot] = _e4m3(rows / scale[..., None])
        scales = torch.zeros(blocks * block, n_kv, dtype=torch.float64, device="cuda")
        scales[slot] = scale
        found[name] = codes.view(blocks, block // PAGE, -1)
        found[name + "_scale"] = scales.view(blocks, block // PAGE, -1)
    return found


def _exact_window(s):
    case = s["case"]
    n_q, n_kv, d, block, W, N = (case[x] for x in ("n_q", "n_kv", "d", "block", "window",
                                                   "sinks"))
    if case["cache"] == "bf16":
        K, V = (s[x].view(-1, n_kv, d) for x in ("k_cache", "v_cache"))
        value = lambda rows, slot, h: rows[slot, h].double()  # noqa: E731
    else:
        K, V = (tuple(x.reshape(-1, n_kv, w) for x, w in zip(_codes_scales(s[c], n_kv, d),
                                                             (d, 1)))
                for c in ("k_cache", "v_cache"))
        value = lambda rows, slot, h: (rows[0].view(torch.uint8)[slot, h]  # noqa: E731
                                       .view(torch.float8_e4m3fn).double()
                                       * rows[1][slot, h].double())
    lens, starts = s["seq_lens"].tolist(), s["starts"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for r, L in enumerate(lens):
        t0, t1 = starts[r], starts[r + 1]
        p = torch.arange(L - (t1 - t0), L, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")
        j = j[(j < N) | (j > L - (t1 - t0) - W)]
        masked = (j > p) | ((p - j >= W) & (j >= N))
        slot = s["tables"][r][j // block].long() * block + j % block
        for h in range(n_kv):
            k, v = value(K, slot, h), value(V, slot, h)
            for head in range(h * (n_q // n_kv), (h + 1) * (n_q // n_kv)):
                a = s["q"][t0:t1, head].double() @ k.t() * s["scale"]
                a[masked] = -math.inf
                out[t0:t1, head] = torch.softmax(a, -1) @ v
    return out
