"""Plain 64-bit definitions of the operators for long contexts, for the tests: bounds
of blocks, the choice of blocks, attention over chosen blocks, accumulated weights,
eviction.  They share no code with the library.  Also the inputs the tests share."""
import numpy as np
import torch

HALF_BF16 = 2.0 ** -8   # half a step, relative to the value
EPS = 2.0 ** -24        # of fp32
FP32_MAX = float(np.finfo(np.float32).max)


# ------------------------------------------------------------------ definitions
def power(top):
    """The least power of two p >= 2^-126 with top <= 127 p (1 for 0)."""
    if top == 0:
        return 1.0
    p = 2.0 ** -126
    while top > 127 * p:
        p *= 2
    return p


def bounds_of(K):
    """K [rows, d] float64 of one block and kv head: (codes [2, d], scale)."""
    K = np.nan_to_num(K, nan=0.0, posinf=FP32_MAX, neginf=-FP32_MAX)
    hi, lo = K.max(0), K.min(0)
    p = power(max(np.abs(hi).max(), np.abs(lo).max()))
    return np.stack([np.ceil(hi / p), np.floor(lo / p)]), p


def bounds(codes, scales, K, tables, lens, starts, block):
    """codes [blocks, n_kv, 2, d] and scales [blocks, n_kv] after the call; K [slots,
    n_kv, d] float64; starts None: every block."""
    codes, scales = codes.copy(), scales.copy()
    for s, n in enumerate(lens):
        new = n if starts is None else int(starts[s + 1] - starts[s])
        if new == 0:
            continue
        for c in range((n - new) // block, -(-n // block)):
            at = int(tables[s][c]) * block
            for h in range(K.shape[1]):
                rows = K[at:at + min(block, n - c * block), h]
                codes[tables[s][c], h], scales[tables[s][c], h] = bounds_of(rows)
    return codes, scales


def token_rows(lens, starts):
    """(token, request, position) of every row of a request."""
    for s, n in enumerate(lens):
        a, b = int(starts[s]), int(starts[s + 1])
        for t in range(a, b):
            yield t, s, n - (b - t)


def choose(q, codes, scales, tables, lens, starts, block, n_sel, sinks, recent, out):
    """out [T, n_kv, n_sel] after the call.  q [T, n_q, d] float64."""
    out = out.copy()
    n_kv = codes.shape[1]
    G = q.shape[1] // n_kv
    for t, s, p in token_rows(lens, starts):
        last = p // block
        ids = np.asarray(tables[s][:last + 1])
        for h in range(n_kv):
            best = np.full(last + 1, -np.inf)
            for g in range(h * G, (h + 1) * G):
                pq = power(np.abs(q[t, g]).max())
                x = np.rint(q[t, g] / pq)
                each = (x * np.where(x > 0, codes[ids, h, 0], codes[ids, h, 1])).sum(-1)
                best = np.maximum(best, each * pq * scales[ids, h])
            c = np.arange(last + 1)
            keep = (c < sinks) | (c > last - recent)
            rest = c[~keep]
            rest = rest[np.argsort(-best[rest], kind="stable")][:max(0, n_sel - int(keep.sum()))]
            chosen = np.sort(np.concatenate([c[keep], rest]))[:n_sel]
            out[t, h] = -1
            out[t, h, :len(chosen)] = chosen
    return out


def _attend(q, K, V, scale):
    """(out [G, d], weights [G, n], size of the error bound's terms) of one kv head."""
    x = q @ K.T * scale
    w = np.exp(x - x.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    S = (np.abs(q) @ np.abs(K).T * abs(scale)).max(-1)
    top = np.abs(q).max(-1) * (np.abs(K).sum(-1) * abs(scale)).max()
    return w @ V, w, w @ np.abs(V), S, top


def blocks_attention(q, K, V, tables, lens, starts, scale, block, selected):
    """(out, A, E): the output (NaN rows: of no request), the weighted mean of |v| and
    the relative error that a weight may have."""
    n_kv = K.shape[1]
    G = q.shape[1] // n_kv
    out, A = np.full(q.shape, np.nan), np.zeros(q.shape)
    E = np.zeros(q.shape[:2])
    for t, s, p in token_rows(lens, starts):
        for h in range(n_kv):
            hs = slice(h * G, (h + 1) * G)
            e = selected[t, h][selected[t, h] >= 0].astype(np.int64)
            j = (e[:, None] * block + np.arange(block)).ravel()
            slot = (np.asarray(tables[s], np.int64)[e][:, None] * block +
                    np.arange(block)).ravel()[j <= p]
            if len(slot) == 0:
                out[t, hs] = 0
                continue
            out[t, hs], _, A[t, hs], S, top = _attend(q[t, hs], K[slot, h], V[slot, h], scale)
            E[t, hs] = weight_error(q.shape[2], S, top, len(slot))
    return out, A, E


def weight_error(d, S, top, n):
    """Relative error of a softmax weight: the score's (a sum of d exact products in
    fp32, at most a step of S each; the 8-bit cache's q in f16, at most half of f16's
    smallest step, 2^-25, of twice q's largest element times the keys; the factors
    log2(e) and scale, 2^-22 of S), for the weight and for the sum; the exponential
    2^-21; the sum of n terms."""
    return 2 * (2 * d * EPS * S + 2.0 ** -24 * top + 2.0 ** -22 * S) + 2.0 ** -20 + n * EPS


def assert_blocks_close(got, ref, what=""):
    """The output is rounded to bf16; a relative error e of the weights moves a weighted
    mean by e (A + |out|); a weight enters P V as two bf16 (2^-16 of it is lost), and
    P V sums in fp32 (2^-12 covers 2^11 keys' steps of it)."""
    out, A, E = ref
    rows = ~np.isnan(out[:, 0, 0])
    assert np.isfinite(got[rows]).all(), f"{what}: non-finite outputs"
    e = E[..., None] + 2.0 ** -16 + 2.0 ** -12
    tol = HALF_BF16 * np.abs(out) * 1.01 + e * (A + np.abs(out)) + 1e-7
    off = (np.abs(got - out) / tol)[rows]
    worst = float(off.max()) if off.size else 0.0
    assert worst <= 1.0, f"{what}: an output is {worst:.2f} times its tolerance off"


def weights_attention(q, K, V, tables, lens, starts, scale, block, weights):
    """(out, A, E, weights, tolerance of the weights)."""
    n_kv = K.shape[1]
    G = q.shape[1] // n_kv
    out, A = np.full(q.shape, np.nan), np.zeros(q.shape)
    E = np.zeros(q.shape[:2])
    weights, tol = weights.astype(np.float64), np.zeros(weights.shape)
    for s, n in enumerate(lens):
        a, b = int(starts[s]), int(starts[s + 1])
        if a == b:
            continue
        j = np.arange(n)
        slot = np.asarray(tables[s], np.int64)[j // block] * block + j % block
        weights[s, :, n - (b - a):n] = 0
        for h in range(n_kv):
            hs = slice(h * G, (h + 1) * G)
            k, v = torch.from_numpy(K[slot, h]), torch.from_numpy(V[slot, h])
            x = torch.from_numpy(q[a:b, hs]).transpose(0, 1)
            hidden = torch.from_numpy(j[None] > np.arange(n - (b - a), n)[:, None])
            score = (x @ k.t() * scale).masked_fill(hidden, -float("inf"))
            w = torch.softmax(score, -1)
            S = (x.abs() @ k.abs().t() * abs(scale)).masked_fill(hidden, 0.0).amax(-1)
            top = x.abs().amax(-1) * (k.abs().sum(-1).max() * abs(scale))
            e = weight_error(q.shape[2], S, top, n)
            out[a:b, hs] = (w @ v).transpose(0, 1).numpy()
            A[a:b, hs] = (w @ v.abs()).transpose(0, 1).numpy()
            E[a:b, hs] = e.transpose(0, 1).numpy()
            weights[s, h, :n] += w.sum((0, 1)).numpy()
            # every weight's own error, the sum over rows and heads, the addition
            tol[s, h, :n] = (w * e[..., None]).sum((0, 1)).numpy() + \
                EPS * ((b - a) * G + 2) * weights[s, h, :n]
    return out, A, E, weights, tol


def evict(parts, weights, tables, lens, budgets, free, count, sinks, recent, block):
    """Moves rows of `parts` (arrays [slots, n_kv, ...]) and weights in place; returns
    (lens, free, count, gone)."""
    free, lens, gone = list(free), list(lens), []
    for s, n in enumerate(lens):
        B = int(budgets[s])
        gone.append(0)
        if n <= B or B < sinks + recent:
            continue
        j = np.arange(n)
        slot = np.asarray(tables[s], np.int64)[j // block] * block + j % block
        for h in range(weights.shape[1]):
            w = weights[s, h]
            order = sorted(range(sinks, n - recent),
                           key=lambda i: (0 if np.isnan(w[i]) else 1,
                                          0 if np.isnan(w[i]) else -float(w[i]), i))
            keep = np.array(list(range(sinks)) + sorted(order[:B - sinks - recent]) +
                            list(range(n - recent, n)), np.int64)
            for x in parts:
                x[slot[:B], h] = x[slot[keep], h]
            w[:B] = w[keep]
        for c in range(-(-B // block), -(-n // block)):
            free[count] = int(tables[s][c])
            count += 1
        gone[s], lens[s] = n - B, B
    return lens, free, count, gone


# ----------------------------------------------------------------------- inputs
class Cache:
    """Requests of these (cached, new) lengths over a cache of random rows, every slot
    that no request holds poisoned with NaN."""

    def __init__(self, requests, n_kv, d, block, fp8, seed, pad=0, spread=1.0):
        from paged_kv_cache_174_gb300 import ops
        rng = np.random.default_rng(seed)
        self.block, self.n_kv, self.d, self.fp8 = block, n_kv, d, fp8
        self.lens = [c + n for c, n in requests]
        new = [n for _, n in requests]
        self.starts = np.concatenate([[0], np.cumsum(new)]).astype(np.int64)
        self.tokens = int(self.starts[-1]) + pad
        held = [-(-n // block) for n in self.lens]
        self.blocks = sum(held) + 3
        ids = rng.permutation(self.blocks)
        self.tables = np.full((len(requests), max(held + [1]) + 1), -1, np.int32)
        live = np.zeros(self.blocks * block, bool)
        at = 0
        for s, n in enumerate(held):
            self.tables[s, :n] = ids[at:at + n]
            at += n
            j = np.arange(self.lens[s])
            live[self.tables[s][j // block].astype(np.int64) * block + j % block] = True
        self.spare = ids[at:]
        g = torch.Generator().manual_seed(seed)
        rows = [torch.randn(self.blocks * block, n_kv, d, generator=g) * spread for _ in range(2)]
        dead = torch.from_numpy(~live)
        if fp8:
            self.device, self.values = [], []
            for x in rows:
                scale = x.abs().amax(-1) / 448.0
                codes = (x / scale[..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
                codes[dead], scale[dead] = 0x7f, float("nan")
                cache = torch.empty(self.blocks, block // 16, ops.fp8_page_bytes(n_kv, d),
                                    dtype=torch.uint8)
                c, f = ops.fp8_cache_views(cache, n_kv, d)
                c.copy_(codes.view(c.shape))
                f.copy_(scale.view(f.shape))
                self.device.append(cache.cuda())
                self.values.append((codes.view(torch.float8_e4m3fn).float() * scale[..., None])
                                   .double().numpy())
        else:
            for x in rows:
                x[dead] = float("nan")
            self.device = [x.bfloat16().view(self.blocks, block, n_kv, d).cuda() for x in rows]
            self.values = [x.bfloat16().double().numpy() for x in rows]
        self.k, self.v = self.device
        self.K, self.V = self.values

    def step(self):
        """(block_tables, seq_lens, query_start_loc) on the GPU."""
        i32 = torch.int32
        return (torch.from_numpy(self.tables).cuda(),
                torch.tensor(self.lens, dtype=i32, device="cuda"),
                torch.tensor(self.starts, dtype=i32, device="cuda"))

    def queries(self, n_q, seed, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        q = (torch.randn(self.tokens, n_q, self.d, generator=g) * spread).bfloat16()
        return q.cuda(), q.double().numpy()

    def parts(self):
        """The caches' rows as arrays [slots, n_kv, ...], as they are held."""
        from paged_kv_cache_174_gb300 import ops
        out = []
        for x in (self.k, self.v):
            if self.fp8:
                c, f = ops.fp8_cache_views(x.cpu(), self.n_kv, self.d)
                out += [c.reshape(-1, self.n_kv, self.d).numpy().copy(),
                        f.reshape(-1, self.n_kv).view(torch.int32).numpy().copy()]
            else:
                out.append(x.cpu().view(torch.int16).view(-1, self.n_kv, self.d).numpy().copy())
        return out
