"""Cases, plain forms and exact values of operators for long contexts over the paged KV cache,
which read less of it (blocks chosen for each query) or hold less of it (tokens evicted):

  summary  bounds of each block's keys, kept up to date step by step (ops.summarize_blocks,
           ops.summarize_blocks_fp8)
  select   the blocks that a query's heads attend to, by a score from the bounds
           (ops.select_blocks)
  blocks   attention over the chosen blocks (ops.paged_attention_blocks,
           ops.paged_attention_blocks_fp8)
  weights  attention that adds up the weight each cached token gets (ops.paged_attention_weights,
           ops.paged_attention_weights_fp8)
  evict    the tokens of least weight dropped, the cache compacted, blocks returned
           (ops.evict_tokens, ops.evict_tokens_fp8)

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
MOST_TOKENS = 600_000  # cached tokens of a drawn case


# ------------------------------------------------------------------------------------- cases
def listed():
    heads = {"n_q": 32, "n_kv": 8, "d": 128, "block": 16}
    return [
        # after the slot scatter of a decode step: 64 running requests, one block each
        {"name": "summary_decode_64", "op": "summary", "seqs": 64, "len_lo": 128, "len_hi": 4096,
         "rows": 1, "whole": False, **heads, "cache": "bf16"},
        # the bounds of whole 8-bit caches, as after an eviction or a swap in
        {"name": "summary_whole_fp8", "op": "summary", "seqs": 16, "len_lo": 1024,
         "len_hi": 8191, "rows": 1, "whole": True, **heads, "cache": "fp8"},
        # a decode step of 64 requests of mixed lengths, at most 512 tokens each
        {"name": "select_decode_64", "op": "select", "seqs": 64, "len_lo": 128, "len_hi": 4096,
         "rows": 1, **heads, "selected": 32, "sinks": 1, "recent": 2},
        # eight requests of long contexts, 2048 tokens each
        {"name": "select_long_8", "op": "select", "seqs": 8, "len_lo": 98304, "len_hi": 131071,
         "rows": 1, **heads, "selected": 128, "sinks": 1, "recent": 4},
        # four short requests of a small model: the smallest call, all latency
        {"name": "blocks_tiny_4", "op": "blocks", "seqs": 4, "len_lo": 5, "len_hi": 300,
         "rows": 1, "n_q": 4, "n_kv": 2, "d": 64, "block": 16, "cache": "bf16", "selected": 8},
        # a decode step of 64 requests at 8192 tokens, 2048 of them read
        {"name": "blocks_decode_64", "op": "blocks", "seqs": 64, "len_lo": 4096, "len_hi": 8192,
         "rows": 1, **heads, "cache": "bf16", "selected": 128},
        # four drafted tokens of each of 16 requests, 8-bit cache in 32-token blocks
        {"name": "blocks_drafted_fp8", "op": "blocks", "seqs": 16, "len_lo": 16384,
         "len_hi": 32767, "rows": 4, "n_q": 32, "n_kv": 4, "d": 128, "block": 32, "cache": "fp8",
         "selected": 64},
        # a decode step of 64 requests of mixed lengths
        {"name": "weights_decode_64", "op": "weights", "decodes": 64, "ctx_lo": 128,
         "ctx_hi": 4096, "chunks": 0, "chunk_lo": 0, "chunk_hi": 0, "chunk_ctx": 0, **heads,
         "cache": "bf16"},
        # long contexts in the 8-bit cache: eight decodes beside a prompt slice
        {"name": "weights_long_fp8", "op": "weights", "decodes": 8, "ctx_lo": 16384,
         "ctx_hi": 32767, "chunks": 1, "chunk_lo": 509, "chunk_hi": 509, "chunk_ctx": 4096,
         **heads, "cache": "fp8"},
        # a prompt in one call, as an offline run has it
        {"name": "weights_prompt_4096", "op": "weights", "decodes": 0, "ctx_lo": 0, "ctx_hi": 0,
         "chunks": 1, "chunk_lo": 4096, "chunk_hi": 4096, "chunk_ctx": 0, **heads,
         "cache": "bf16"},
        # 64 requests that ran past 2048 tokens, some of them not yet
        {"name": "evict_decode_64", "op": "evict", "seqs": 64, "len_lo": 1900, "len_hi": 2304,
         "budget": 2048, "sinks": 4, "recent": 256, **heads, "cache": "bf16"},
        # long prompts cut down to an eighth, 8-bit cache
        {"name": "evict_long_fp8", "op": "evict", "seqs": 8, "len_lo": 16384, "len_hi": 32767,
         "budget": 4096, "sinks": 16, "recent": 1024, **heads, "cache": "fp8"},
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
        op = rng.choice(["summary", "select", "blocks", "blocks", "weights", "weights", "evict"])
        n_kv, group, d = rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
        heads = {"n_q": n_kv * group, "n_kv": n_kv, "d": d, "block": rng.choice([16, 16, 32])}
        cache = {"cache": rng.choice(["bf16", "fp8"])}
        seqs = _spread(rng, 1, 256)
        lo, hi = sorted((_spread(rng, 1, 32768), _spread(rng, 1, 32768)))
        rows = rng.choice([1, 1, 1, 2, 5, 8, _spread(rng, 2, 200)])
        if op == "summary":
            case = {"op": op, "seqs": seqs, "len_lo": max(lo, rows), "len_hi": max(hi, rows),
                    "rows": rows, "whole": rng.random() < 0.3, **heads, **cache}
        elif op == "select":
            lo, hi = lo * rng.choice([1, 1, 4]), hi * 4
            sinks, recent = rng.choice([0, 1, 3]), rng.choice([1, 2, 7])
            case = {"op": op, "seqs": seqs, "len_lo": max(lo, rows), "len_hi": max(hi, rows),
                    "rows": rows, **heads, "selected": sinks + recent + _spread(rng, 2, 300),
                    "sinks": sinks, "recent": recent}
            if _blocks(hi, case["block"]) < case["selected"] + 16:  # little to choose
                continue
        elif op == "blocks":
            case = {"op": op, "seqs": seqs, "len_lo": max(lo, rows), "len_hi": max(hi, rows),
                    "rows": rows, **heads, **cache, "selected": _spread(rng, 1, 300)}
        elif op == "weights":
            kind = rng.choice(["decode", "chunk", "mixed"])
            chunks = 0 if kind == "decode" else rng.choice([1, 1, 2, 5])
            clo, chi = sorted((_spread(rng, 2, 4096), _spread(rng, 2, 4096)))
            case = {"op": op, "decodes": 0 if kind == "chunk" else seqs, "ctx_lo": lo,
                    "ctx_hi": hi, "chunks": chunks, "chunk_lo": clo if chunks else 0,
                    "chunk_hi": chi if chunks else 0,
                    "chunk_ctx": rng.choice([0, 1, 777, _spread(rng, 1, 16384)]) if chunks else 0,
                    **heads, **cache}
        else:
            sinks, recent = rng.choice([0, 1, 4, 33]), rng.choice([0, 1, 32, _spread(rng, 1, 700)])
            case = {"op": op, "seqs": seqs, "len_lo": lo, "len_hi": hi,
                    "budget": sinks + recent + _spread(rng, 1, 4096) - 1, "sinks": sinks,
                    "recent": recent, **heads, **cache}
        tokens = sum(_lengths(case)[0])
        if _cost(case) <= most and tokens <= MOST_TOKENS * (8 if op == "select" else 1):
            return case


def _even(lo, hi, n):
    """n whole numbers from lo to hi at even distances."""
    return [lo + (hi - lo) * i // max(1, n - 1) for i in range(n)]


def _lengths(case):
    """(tokens in the cache, new ones among them) of each request."""
    if case["op"] != "weights":
        lens = _even(case["len_lo"], case["len_hi"], case["seqs"])
        return lens, [case.get("rows", 1)] * len(lens)
    new = _even(case["chunk_lo"], case["chunk_hi"], case["chunks"])
    held = _even(case["chunk_ctx"] // 2, case["chunk_ctx"], case["chunks"])
    return (_even(case["ctx_lo"], case["ctx_hi"], case["decodes"])
            + [c + n for c, n in zip(held, new)], [1] * case["decodes"] + new)


def _blocks(n, block):
    return -(-n // block)


# ----------------------------------------------------------------------------------- inputs
def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _quantised(x, block):
    """Rows x [slots, n_kv, d] as an 8-bit cache: pages of 16 rows' codes, then their scales."""
    slots, n_kv, d = x.shape
    pages = []
    for part in x.split(1 << 16):
        part = part.float()
        top = part.abs().amax(-1)
        scale = torch.where(top > 0, top / E4M3_MAX, torch.ones_like(top))
        codes = (part / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
        n = part.shape[0] // PAGE
        pages.append(torch.cat([codes.view(n, -1), scale.view(n, -1).view(torch.uint8)], 1))
    return torch.cat(pages).view(slots // block, block // PAGE, -1)


def _codes_scales(cache, n_kv, d):
    """Views of an 8-bit cache: codes [blocks, pages, 16 n_kv d] and scales [.., 16 n_kv]."""
    n = PAGE * n_kv * d
    return cache[:, :, :n].view(torch.float8_e4m3fn), cache[:, :, n:].view(torch.float32)


def prepare(case, seed):
    op = case["op"]
    rng = random.Random(seed)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    n_kv, d, block = case["n_kv"], case["d"], case["block"]
    lens, new = _lengths(case)
    order = list(range(len(lens)))
    rng.shuffle(order)
    lens, new = [lens[i] for i in order], [new[i] for i in order]
    held = [_blocks(n, block) for n in lens]
    width, blocks = max(held), sum(held) + 5
    ids = np.random.default_rng(seed).permutation(blocks).astype(np.int32)
    tables = np.full((len(lens), width), -1, np.int32)
    at = 0
    for i, n in enumerate(held):
        tables[i, :n] = ids[at:at + n]
        at += n
    T = sum(new)
    s = {"case": dict(case), "tables": torch.from_numpy(tables).cuda(), "lens": _int32(lens),
         "starts": _int32(np.concatenate([[0], np.cumsum(new)]).tolist()), "tokens": T,
         "max_q_len": max(new), "min_q_len": min(new), "max_seq_len": max(lens),
         "host_lens": lens, "host_new": new, "scale": 1.0 / math.sqrt(d)}

    def randn(*shape):
        return torch.randn(shape, device="cuda", dtype=torch.bfloat16, generator=g)
    if op in ("select", "blocks", "weights"):
        s["q"] = randn(T, case["n_q"], d)
    if op == "select":
        # what blocks of normal keys come to: bounds about two standard deviations out
        low = torch.randint(24, 96, (2, blocks, n_kv, d), device="cuda", generator=g)
        s["bounds"] = torch.stack([low[0], -low[1]], 2).to(torch.int8)
        s["bound_scales"] = torch.exp2(torch.randint(-7, -3, (blocks, n_kv), device="cuda",
                                                     generator=g).float())
        s["selected"] = torch.empty(T, n_kv, case["selected"], dtype=torch.int32, device="cuda")
        return s
    # keys that drift from block to block, as neighbouring tokens are alike
    rows = [randn(blocks * block, n_kv, d) for _ in range(2)]
    rows[0].view(blocks, block, n_kv, d).add_(randn(blocks, 1, n_kv, d), alpha=0.5)
    if op == "summary":
        del rows[1]
    caches = [r.view(blocks, block, n_kv, d) if case["cache"] == "bf16" else _quantised(r, block)
              for r in rows]
    s["k_cache"] = caches[0]
    if op == "summary":
        s["bounds"] = torch.zeros(blocks, n_kv, 2, d, dtype=torch.int8, device="cuda")
        s["bound_scales"] = torch.zeros(blocks, n_kv, device="cuda")
        return s
    s["v_cache"] = caches[1]
    if op == "blocks":
        # the row's own block and others at random, in order; -1 where there are fewer
        p = torch.cat([torch.arange(n - r, n) for n, r in zip(lens, new)]).cuda()
        last = (p // block)[:, None, None]
        column = torch.arange(max(width, case["selected"]), device="cuda")
        chance = torch.rand(T, n_kv, column.numel(), device="cuda", generator=g)
        chance = chance.masked_fill(column == last, 2.0).masked_fill(column > last, -1.0)
        top, pick = chance.topk(case["selected"], -1)
        pick = pick.masked_fill(top < 0, 1 << 30).sort(-1).values
        s["selected"] = pick.masked_fill(pick == 1 << 30, -1).int()
    elif op == "weights":
        s["weights"] = torch.rand(len(lens), n_kv, width * block, device="cuda", generator=g)
        if own:  # the scratch buffer that a serving loop holds for all its calls
            from paged_kv_cache_174_gb300 import ops
            s["workspace"] = ops.alloc_weights_workspace(len(lens), T, case["n_q"], n_kv, d,
                                                         s["max_q_len"], s["max_seq_len"], "cuda")
    else:
        # few tokens hold most of the weight
        s["weights"] = torch.randn(len(lens), n_kv, width * block, device="cuda",
                                   generator=g).mul_(2).exp_()
        s["budgets"] = _int32([case["budget"]] * len(lens))
        free = np.full(blocks, -1, np.int32)
        free[:blocks - at] = ids[at:]
        s["free"] = torch.from_numpy(free).cuda()
        s["count"], s["count_out"] = _int32([blocks - at]), _int32([0])
        s["lens_out"] = _int32([0] * len(lens))
    if op != "evict":
        s["out"] = torch.empty_like(s["q"])
    return s


# -------------------------------------------------------------------------------------- run
def run(state):
    op = state["case"]["op"]
    return (_OWN if own else _PLAIN)[op](state)


def _own_summary(s):
    from paged_kv_cache_174_gb300 import ops
    case = s["case"]
    call = ops.summarize_blocks if case["cache"] == "bf16" else ops.summarize_blocks_fp8
    call(s["k_cache"], s["tables"], s["lens"], None if case["whole"] else s["starts"],
         s["bounds"], s["bound_scales"], num_tokens=s["tokens"])
    return {"bounds": s["bounds"], "scales": s["bound_scales"]}


def _own_select(s):
    from paged_kv_cache_174_gb300 import ops
    case = s["case"]
    return ops.select_blocks(
        s["q"], s["bounds"], s["bound_scales"], s["tables"], s["lens"], s["starts"],
        num_selected=case["selected"], num_sinks=case["sinks"], num_recent=case["recent"],
        block_size=case["block"], max_seq_len=s["max_seq_len"], out=s["selected"])


def _own_blocks(s):
    from paged_kv_cache_174_gb300 import ops
    call = ops.paged_attention_blocks if s["case"]["cache"] == "bf16" else \
        ops.paged_attention_blocks_fp8
    return call(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["starts"],
                s["scale"], s["selected"], out=s["out"])


def _own_weights(s):
    from paged_kv_cache_174_gb300 import ops
    call = ops.paged_attention_weights if s["case"]["cache"] == "bf16" else \
        ops.paged_attention_weights_fp8
    out = call(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["starts"],
               s["scale"], s["weights"], min_q_len=s["min_q_len"], max_q_len=s["max_q_len"],
               max_seq_len=s["max_seq_len"], out=s["out"], workspace=s["workspace"])
    return {"out": out, "weights": s["weights"]}


def _caches(s):
    """The caches as run() returns them: bf16 rows, or codes and scales."""
    case = s["case"]
    if case["cache"] == "bf16":
        return {"k": s["k_cache"], "v": s["v_cache"]}
    k, ks = _codes_scales(s["k_cache"], case["n_kv"], case["d"])
    v, vs = _codes_scales(s["v_cache"], case["n_kv"], case["d"])
    return {"k": k, "k_scale": ks, "v": v, "v_scale": vs}


def _own_evict(s):
    from paged_kv_cache_174_gb300 import ops
    case = s["case"]
    call = ops.evict_tokens if case["cache"] == "bf16" else ops.evict_tokens_fp8
    lens = call(s["k_cache"], s["v_cache"], s["weights"], s["tables"], s["lens"], s["budgets"],
                s["free"], s["count"], num_sinks=case["sinks"], num_recent=case["recent"],
                max_seq_len=s["max_seq_len"], seq_lens_out=s["lens_out"],
                free_count_out=s["count_out"])
    return {**_caches(s), "weights": s["weights"], "lens": lens, "free": s["free"],
            "count": s["count_out"]}


_OWN = {"summary": _own_summary, "select": _own_select, "blocks": _own_blocks,
        "weights": _own_weights, "evict": _own_evict}


def _plain_rows(cache, slot, case):
    """Rows of the cache at these slots, all kv heads, in 32 bits."""
    n_kv, d = case["n_kv"], case["d"]
    if case["cache"] == "bf16":
        return cache.view(-1, n_kv, d)[slot].float()
    codes, scales = _codes_scales(cache, n_kv, d)
    code = codes.view(torch.uint8).reshape(-1, n_kv, d)[slot].view(torch.float8_e4m3fn).float()
    return code * scales.reshape(-1, n_kv)[slot][..., None]


def _power(top, most):
    """The least power of two p with top <= most p (1 for 0)."""
    m, x = torch.frexp(top)
    e = x - 7 + (m * 128 > most).int()
    return torch.where(top > 0, torch.ldexp(torch.ones_like(top), e.clamp(min=-126)), 1.0)


def _plain_summary(s):
    case = s["case"]
    block, blocks = case["block"], s["bounds"].shape[0]
    length = s["lens"].long()[:, None]
    if case["whole"]:
        first, most = torch.zeros_like(length), s["tables"].shape[1]
    else:
        first = (length - s["starts"].diff()[:, None]) // block
        most = min(s["tables"].shape[1], (case["rows"] + block - 2) // block + 1)
    column = first + torch.arange(most, device="cuda")
    there = column * block < length
    table = s["tables"].gather(1, column.clamp(max=s["tables"].shape[1] - 1)).long()
    table = torch.where(there, table, blocks)
    step = max(1, (1 << 28) // (table.shape[1] * block * case["n_kv"] * case["d"]))
    bounds = torch.cat([s["bounds"], s["bounds"][:1]])
    scales = torch.cat([s["bound_scales"], s["bound_scales"][:1]])
    for part, col, n in zip(table.split(step), column.split(step), length.split(step)):
        i = torch.arange(block, device="cuda")
        K = _plain_rows(s["k_cache"], (part.clamp(max=blocks - 1)[..., None] * block + i), case)
        K = torch.nan_to_num(K)
        out = (col[..., None] * block + i >= n[..., None])[..., None, None]
        hi = K.masked_fill(out, -math.inf).amax(2)
        lo = K.masked_fill_(out, math.inf).amin(2)
        p = _power(torch.maximum(hi.abs(), lo.abs()).amax(-1), 127)
        hi, lo = (hi / p[..., None]).ceil(), (lo / p[..., None]).floor()
        bounds[part] = torch.stack([hi, lo], -2).nan_to_num().to(torch.int8)
        scales[part] = p
    s["bounds"].copy_(bounds[:-1])
    s["bound_scales"].copy_(scales[:-1])
    return {"bounds": s["bounds"], "scales": s["bound_scales"]}


def _plain_tokens(s):
    """(request, position) of each new token."""
    token = torch.arange(s["tokens"], device="cuda")
    request = torch.searchsorted(s["starts"][1:].long(), token, right=True)
    return request, s["lens"].long()[request] - s["starts"].long()[request + 1] + token


def _plain_select(s):
    case = s["case"]
    n_kv, d, K, block = case["n_kv"], case["d"], case["selected"], case["block"]
    request, p = _plain_tokens(s)
    width = s["tables"].shape[1]
    column = torch.arange(width, device="cuda")
    out = s["selected"]
    step = max(1, (1 << 29) // (width * n_kv * d))
    for t in range(0, s["tokens"], step):
        to = min(s["tokens"], t + step)
        table = s["tables"][request[t:to]].long().clamp(min=0)
        q = s["q"][t:to].float().view(to - t, n_kv, -1, d)
        pq = _power(q.abs().amax(-1), 127)
        q = (q / pq[..., None]).round()
        bound = s["bounds"][table]
        score = torch.einsum("thgd,tchd->thgc", q.clamp(min=0), bound[..., 0, :].float())
        score += torch.einsum("thgd,tchd->thgc", q.clamp(max=0), bound[..., 1, :].float())
        score = score * pq[..., None] * s["bound_scales"][table].transpose(1, 2)[:, :, None]
        score = score.amax(2)
        last = (p[t:to] // block)[:, None, None]
        forced = (column < case["sinks"]) | (column > last - case["recent"])
        score.masked_fill_(forced, math.inf).masked_fill_(column > last, -math.inf)
        order = score.sort(dim=-1, descending=True, stable=True).indices[..., :K]
        order = order.masked_fill(order > last, width).sort(-1).values
        order = order.masked_fill(order == width, -1)
        out[t:to, :, :min(K, width)] = order.int()
        out[t:to, :, min(K, width):] = -1
    return out


def _plain_blocks(s):
    case = s["case"]
    n_kv, d, block = case["n_kv"], case["d"], case["block"]
    request, p = _plain_tokens(s)
    out, i = s["out"], torch.arange(block, device="cuda")
    head = torch.arange(n_kv, device="cuda")[:, None]
    step = max(1, (1 << 27) // (case["selected"] * block * n_kv * d))
    for t in range(0, s["tokens"], step):
        to = min(s["tokens"], t + step)
        pick = s["selected"][t:to].long()
        table = s["tables"][request[t:to]].long()[:, None].expand(-1, n_kv, -1)
        base = table.gather(2, pick.clamp(min=0))
        key = (pick[..., None] * block + i).flatten(2)
        slot = (base[..., None] * block + i).flatten(2).clamp(min=0)
        if case["cache"] == "bf16":
            K, V = (c.view(-1, n_kv, d)[slot, head].float()
                    for c in (s["k_cache"], s["v_cache"]))
        else:
            K, V = ((codes.view(torch.uint8).reshape(-1, n_kv, d)[slot, head]
                     .view(torch.float8_e4m3fn).float()
                     * scales.reshape(-1, n_kv)[slot, head][..., None])
                    for codes, scales in (_codes_scales(c, n_kv, d)
                                          for c in (s["k_cache"], s["v_cache"])))
        q = s["q"][t:to].float().view(to - t, n_kv, -1, d)
        score = torch.einsum("thgd,thkd->thgk", q, K).mul_(s["scale"])
        seen = (key >= 0) & (key <= p[t:to, None, None])
        score.masked_fill_(~seen[:, :, None], -math.inf)
        score.sub_(score.amax(-1, keepdim=True)).exp_()
        o = torch.einsum("thgk,thkd->thgd", score, V) / score.sum(-1)[..., None]
        out[t:to] = o.reshape(to - t, -1, d).to(out.dtype)
    return out


def _plain_weights(s):
    case = s["case"]
    n_kv, d, block = case["n_kv"], case["d"], case["block"]
    out, weights = s["out"], s["weights"]

    def attend(which, length, rows):
        """These requests, of at most `length` tokens and `rows` new ones each."""
        which = torch.tensor(which, device="cuda")
        L, n = s["lens"][which].long()[:, None], s["starts"].diff()[which].long()[:, None]
        key = torch.arange(length, device="cuda")
        slot = s["tables"][which].long().clamp(min=0)[:, key // block] * block + key % block
        K, V = (_plain_rows(s[c], slot, case) for c in ("k_cache", "v_cache"))
        i = torch.arange(rows, device="cuda")
        token = s["starts"][which].long()[:, None] + i
        real = i < n
        q = s["q"][token.clamp(max=s["tokens"] - 1)].float().view(*token.shape, n_kv, -1, d)
        unseen = (key > (L - n + i)[..., None])[:, None]
        put = token[real]
        for h in range(n_kv):
            score = torch.einsum("rmgd,rkd->rgmk", q[:, :, h], K[:, :, h]).mul_(s["scale"])
            score.masked_fill_(unseen, -math.inf)
            score.sub_(score.amax(-1, keepdim=True)).exp_()
            score /= score.sum(-1, keepdim=True)
            score.masked_fill_(~real[:, None, :, None], 0)
            o = torch.einsum("rgmk,rkd->rmgd", score, V[:, :, h])
            G = o.shape[2]
            out[put, h * G:(h + 1) * G] = o[real].to(out.dtype)
            old = weights[which, h, :length].masked_fill(key >= L - n, 0)
            total = torch.where(key < L, old + score.sum((1, 2)), weights[which, h, :length])
            weights[which, h, :length] = total
    one = sorted((n, i) for i, (n, r) in enumerate(zip(s["host_lens"], s["host_new"])) if r == 1)
    while one:
        n = one[-1][0]
        fit = max(1, (1 << 28) // (n * n_kv * d))
        attend([i for _, i in one[-fit:]], n, 1)
        one = one[:-fit]
    for i, (n, r) in enumerate(zip(s["host_lens"], s["host_new"])):
        if r > 1:
            attend([i], n, r)
    return {"out": out, "weights": weights}


def _plain_evict(s):
    case = s["case"]
    n_kv, d, block = case["n_kv"], case["d"], case["block"]
    L, budget = s["lens"].long(), s["budgets"].long()
    S = L.numel()
    over = L > budget
    kept = torch.minimum(L, budget)
    most, span = min(case["budget"], s["max_seq_len"]), s["max_seq_len"]
    j = torch.arange(span, device="cuda")
    forced = (j < case["sinks"]) | (j >= L[:, None] - case["recent"]) | ~over[:, None]
    rank = s["weights"][:, :, :span].masked_fill(forced[:, None], math.inf)
    rank.masked_fill_((j >= L[:, None])[:, None], -math.inf)
    source = rank.sort(dim=-1, descending=True, stable=True).indices[..., :most]
    i = torch.arange(most, device="cuda")
    source = source.masked_fill((i >= kept[:, None])[:, None], 1 << 30).sort(-1).values
    moves = ((source != 1 << 30) & (source != i))
    source = torch.where(moves, source, i)
    request = torch.arange(S, device="cuda")[:, None, None]
    head = torch.arange(n_kv, device="cuda")[:, None]

    def slot(x):
        return s["tables"][request, x // block].long().clamp(min=0) * block + x % block
    s["weights"][:, :, :most] = s["weights"].gather(2, source)
    # one slot more than the pool has: where the tokens that stay go
    slots = s["k_cache"].shape[0] * block
    to = torch.where(moves, slot(i.expand_as(source)), slots)
    frm = slot(source)
    for cache in (s["k_cache"], s["v_cache"]):
        if case["cache"] == "bf16":
            parts = [(cache, d)]
        else:
            codes, scales = _codes_scales(cache, n_kv, d)
            parts = [(codes.view(torch.uint8), d), (scales, 1)]
        for part, w in parts:
            flat = part.reshape(-1, n_kv, w)
            whole = torch.cat([flat, flat[:1]])
            whole[to, head] = flat[frm, head]
            part.copy_(whole[:-1].view(part.shape))
    first, last = (kept + block - 1) // block, (L + block - 1) // block
    ends = (last - first).cumsum(0)
    column = torch.arange(s["tables"].shape[1], device="cuda")
    gone = (column >= first[:, None]) & (column < last[:, None])
    place = s["count"].long() + (ends - last)[:, None] + column
    whole = torch.cat([s["free"], s["free"][:1]])
    whole[torch.where(gone, place, s["free"].numel())] = s["tables"]
    s["free"].copy_(whole[:-1])
    s["count_out"].copy_(s["count"] + ends[-1:])
    s["lens_out"].copy_(kept)
    return {**_caches(s), "weights": s["weights"], "lens": s["lens_out"], "free": s["free"],
            "count": s["count_out"]}


_PLAIN = {"summary": _plain_summary, "select": _plain_select, "blocks": _plain_blocks,
          "weights": _plain_weights, "evict": _plain_evict}


# ------------------------------------------------------------------------------------- work
def work(case):
    n_kv, d, block, op = case["n_kv"], case["d"], case["block"], case["op"]
    lens, new = _lengths(case)
    S, T = len(lens), sum(new)
    bound = n_kv * (2 * d + 4)  # of a block
    if op == "select":
        seen = sum((p // block + 1) for n, r in zip(lens, new) for p in (n - 1,))
        scored = sum(_blocks(p + 1, block) for n, r in zip(lens, new)
                     for p in range(n - r, n))
        return {"bytes": seen * (bound + 4) + T * case["n_q"] * d * 2
                + T * n_kv * case["selected"] * 4 + 8 * S,
                "flops": 4 * d * case["n_q"] * scored}
    row = 2 * d if case["cache"] == "bf16" else d + 4
    if op == "summary":
        from_ = [0 if case["whole"] else (n - r) // block for n, r in zip(lens, new)]
        rows = sum(n - f * block for n, f in zip(lens, from_))
        blocks = sum(_blocks(n, block) - f for n, f in zip(lens, from_))
        return {"bytes": rows * n_kv * row + blocks * (bound + 4) + 8 * S,
                "flops": 2 * rows * n_kv * d}
    n_q = case["n_q"]
    if op == "blocks":
        keys = sum(min(case["selected"] * block - (block - 1 - p % block), p + 1)
                   for n, r in zip(lens, new) for p in range(n - r, n))
        entries = sum(min(case["selected"], p // block + 1)
                      for n, r in zip(lens, new) for p in range(n - r, n))
        return {"bytes": 2 * keys * n_kv * row + 2 * T * n_q * d * 2
                + 4 * T * n_kv * case["selected"] + 4 * entries + 8 * S,
                "flops": 4 * d * n_q * keys}
    keys = sum(lens)
    if op == "weights":
        pairs = sum(r * n - r * (r - 1) // 2 for n, r in zip(lens, new))
        more = sum(r * n - r * (r - 1) // 2 for n, r in zip(lens, new) if r > 1)
        return {"bytes": 2 * keys * n_kv * row + 8 * keys * n_kv + 2 * T * n_q * d * 2
                + 4 * _blocks(keys, block) + 8 * S,
                "flops": 4 * d * n_q * pairs + 2 * d * n_q * more}
    # of the tokens between sinks and recent ones an even share is taken to go
    budget, sinks = case["budget"], case["sinks"]
    moved = sum(budget - sinks for n in lens if n > budget)
    over = sum(n for n in lens if n > budget)
    freed = sum(_blocks(n, block) - _blocks(min(n, budget), block) for n in lens)
    return {"bytes": 4 * n_kv * over + moved * n_kv * (4 * row + 4) + 8 * freed + 12 * S,
            "flops": 0}


# ------------------------------------------------------------------------------------ exact
def exact(case, seed):
    lens, new = _lengths(case)
    if case["op"] in ("select", "blocks"):  # a loop over tokens and heads
        long = sum(new) * case["n_kv"] > 40_000
    else:
        long = case["op"] == "weights" and \
            4 * case["d"] * case["n_q"] * sum(n * r for n, r in zip(lens, new)) > 3e12
    return None if long else _EXACT[case["op"]](prepare(case, seed))


def _exact_value(s, name):
    """A function (slots, kv head) -> rows of a cache in 64 bits."""
    case = s["case"]
    n_kv, d = case["n_kv"], case["d"]
    if case["cache"] == "bf16":
        rows = s[name].view(-1, n_kv, d)
        return lambda slot, h: rows[slot, h].double()
    codes, scales = _codes_scales(s[name], n_kv, d)
    codes = codes.view(torch.uint8).reshape(-1, n_kv, d)
    scales = scales.reshape(-1, n_kv, 1)
    return lambda slot, h: (codes[slot, h].view(torch.float8_e4m3fn).double()
                            * scales[slot, h].double())


def _exact_exponent(top):
    """The least e with top <= 127 * 2^e, found from above."""
    e = torch.full_like(top, 130.0)
    while True:
        lower = (top <= 127 * torch.exp2(e - 1)) & (top > 0) & (e > -126)
        if not lower.any():
            return torch.where(top > 0, e, 0.0)
        e = e - lower.double()


def _exact_summary(s):
    case = s["case"]
    n_kv, block = case["n_kv"], case["block"]
    key = _exact_value(s, "k_cache")
    codes, scales = s["bounds"].double(), s["bound_scales"].double()
    jobs, tops, his, los = [], [], [], []
    tables = s["tables"].tolist()
    for r, (n, new) in enumerate(zip(s["host_lens"], s["host_new"])):
        for b in range(0 if case["whole"] else (n - new) // block, _blocks(n, block)):
            jobs.append((tables[r][b], min(block, n - b * block)))
    # (blocks with as many tokens together)
    for rows in sorted({m for _, m in jobs}):
        ids = torch.tensor([b for b, m in jobs if m == rows], device="cuda")
        for h in range(n_kv):
            K = key(ids[:, None] * block + torch.arange(rows, device="cuda"), h).float().double()
            hi, lo = K.max(1).values, K.min(1).values
            e = _exact_exponent(torch.maximum(hi.abs(), lo.abs()).max(-1).values)
            unit = torch.exp2(e)
            scales[ids, h] = unit
            codes[ids, h, 0] = torch.ceil(hi / unit[:, None])
            codes[ids, h, 1] = torch.floor(lo / unit[:, None])
    return {"bounds": codes, "scales": scales}


def _exact_select(s):
    case = s["case"]
    n_kv, G, d, block, K = case["n_kv"], case["n_q"] // case["n_kv"], case["d"], case["block"], \
        case["selected"]
    found = np.full((s["tokens"], n_kv, K), -1, np.int32)
    q_all = s["q"].double().view(-1, n_kv, G, d)
    unit_q = torch.exp2(_exact_exponent(q_all.abs().amax(-1)))
    q_all = torch.round(q_all / unit_q[..., None])
    t = 0
    for r, (n, new) in enumerate(zip(s["host_lens"], s["host_new"])):
        ids = s["tables"][r, :_blocks(n, block)].long()
        bound, unit = s["bounds"][ids].double(), s["bound_scales"][ids].double()
        for p in range(n - new, n):
            last = p // block
            best = None
            for g in range(G):
                each = torch.maximum(q_all[t, :, g] * bound[:last + 1, :, 0],
                                     q_all[t, :, g] * bound[:last + 1, :, 1]).sum(-1)
                each = each * unit_q[t, :, g] * unit[:last + 1]
                best = each if best is None else torch.maximum(best, each)
            best, b = best.cpu().numpy(), np.arange(last + 1)
            keep = (b < case["sinks"]) | (b > last - case["recent"])
            rest = b[~keep]
            for h in range(n_kv):
                top = rest[np.argsort(-best[rest, h], kind="stable")][:K - int(keep.sum())]
                chosen = np.sort(np.concatenate([b[keep], top]))
                found[t, h, :len(chosen)] = chosen
            t += 1
    return found


def _exact_blocks(s):
    case = s["case"]
    n_kv, G, block = case["n_kv"], case["n_q"] // case["n_kv"], case["block"]
    key, value = _exact_value(s, "k_cache"), _exact_value(s, "v_cache")
    picks, tables = s["selected"].cpu().numpy(), s["tables"].cpu().numpy()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    i, t = np.arange(block), 0
    for r, (n, new) in enumerate(zip(s["host_lens"], s["host_new"])):
        for p in range(n - new, n):
            for h in range(n_kv):
                b = picks[t, h][picks[t, h] >= 0]
                j = (b[:, None] * block + i).ravel()
                slot = (tables[r][b][:, None].astype(np.int64) * block + i).ravel()[j <= p]
                slot = torch.from_numpy(slot).cuda()
                a = s["q"][t, h * G:(h + 1) * G].double() @ key(slot, h).t() * s["scale"]
                out[t, h * G:(h + 1) * G] = torch.softmax(a, -1) @ value(slot, h)
            t += 1
    return out


def _exact_weights(s):
    case = s["case"]
    n_kv, G, block = case["n_kv"], case["n_q"] // case["n_kv"], case["block"]
    key, value = _exact_value(s, "k_cache"), _exact_value(s, "v_cache")
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    weights, t = s["weights"].double(), 0
    for r, (n, new) in enumerate(zip(s["host_lens"], s["host_new"])):
        j = torch.arange(n, device="cuda")
        slot = s["tables"][r][j // block].long() * block + j % block
        hidden = j > torch.arange(n - new, n, device="cuda")[:, None]
        weights[r, :, n - new:n] = 0
        for h in range(n_kv):
            k, v = key(slot, h), value(slot, h)
            for head in range(h * G, (h + 1) * G):
                a = s["q"][t:t + new, head].double() @ k.t() * s["scale"]
                a = torch.softmax(a.masked_fill_(hidden, -math.inf), -1)
                weights[r, h, :n] += a.sum(0)
                out[t:t + new, head] = a @ v
        t += new
    return {"out": out, "weights": weights}


def _exact_evict(s):
    case = s["case"]
    n_kv, d, block = case["n_kv"], case["d"], case["block"]
    weights = s["weights"].cpu().numpy().copy()
    tables, free = s["tables"].cpu().numpy(), s["free"].cpu().numpy().copy()
    count, lens, i = int(s["count"]), [], np.arange
    if case["cache"] == "bf16":
        parts = [s[c].view(-1, n_kv, d) for c in ("k_cache", "v_cache")]
    else:
        pairs = [_codes_scales(s[c], n_kv, d) for c in ("k_cache", "v_cache")]
        parts = [x for codes, scales in pairs
                 for x in (codes.view(torch.uint8).reshape(-1, n_kv, d),
                           scales.reshape(-1, n_kv, 1))]
    to, frm, heads = [], [], []
    for r, (n, budget) in enumerate(zip(s["host_lens"], s["budgets"].tolist())):
        lens.append(min(n, budget))
        if n <= budget:
            continue
        slot = tables[r, i(n) // block].astype(np.int64) * block + i(n) % block
        middle = i(case["sinks"], n - case["recent"])
        for h in range(n_kv):
            w = weights[r, h]
            best = middle[np.argsort(-w[middle], kind="stable")]
            best = best[:budget - case["sinks"] - case["recent"]]
            keep = np.concatenate([i(case["sinks"]), np.sort(best), i(n - case["recent"], n)])
            to.append(slot[:budget])
            frm.append(slot[keep])
            heads.append(np.full(budget, h))
            w[:budget] = w[keep]
        for b in range(_blocks(budget, block), _blocks(n, block)):
            free[count] = tables[r, b]
            count += 1
    if to:
        to, frm, heads = (torch.from_numpy(np.concatenate(x)).cuda() for x in (to, frm, heads))
        for x in parts:
            x[to, heads] = x[frm, heads]
    names = ["k", "v"] if case["cache"] == "bf16" else ["k", "k_scale", "v", "v_scale"]
    found = {}
    for name, x, y in zip(names, parts, _caches(s).values()):
        x = x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x
        found[name] = x.reshape(y.shape)
    return {**found, "weights": weights, "lens": np.array(lens, np.int32), "free": free,
            "count": np.array([count], np.int32)}


_EXACT = {"summary": _exact_summary, "select": _exact_select, "blocks": _exact_blocks,
          "weights": _exact_weights, "evict": _exact_evict}
