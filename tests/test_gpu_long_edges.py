"""The operators for long contexts at the ends of their inputs' ranges, on the GPU: scores
past fp32, bounds never written, table entries that name no block, requests longer than what
is held in shared memory, caches of several layers."""
import numpy as np
import pytest
import torch

import long_reference as R
from paged_kv_cache_174_gb300 import ops

pytestmark = pytest.mark.gpu


class Bounds:
    """Requests of these lengths (new tokens: 1 each) with codes and scales and no keys."""

    def __init__(self, lens, n_kv, d, seed, block=16):
        rng = np.random.default_rng(seed)
        self.lens, self.n_kv, self.d, self.block = list(lens), n_kv, d, block
        self.tokens = len(lens)
        self.starts = np.arange(len(lens) + 1)
        held = [-(-n // block) for n in lens]
        self.blocks = sum(held) + 2
        ids = rng.permutation(self.blocks)
        self.tables = np.full((len(lens), max(held)), -1, np.int32)
        at = 0
        for s, n in enumerate(held):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        self.codes = torch.from_numpy(
            rng.integers(-127, 128, (self.blocks, n_kv, 2, d))).to(torch.int8).cuda()
        self.scales = torch.ones(self.blocks, n_kv, device="cuda")

    def choose(self, q, n_sel, sinks, recent, guard=3):
        """(chosen, the rows before and behind them)."""
        i32 = dict(dtype=torch.int32, device="cuda")
        rows = torch.full((self.tokens + 2 * guard, self.n_kv, n_sel), -9, **i32)
        out = rows[guard:guard + self.tokens]
        ops.select_blocks(q, self.codes, self.scales, torch.from_numpy(self.tables).cuda(),
                          torch.tensor(self.lens, **i32), torch.tensor(self.starts, **i32),
                          num_selected=n_sel, num_sinks=sinks, num_recent=recent,
                          block_size=self.block, max_seq_len=max(self.lens), out=out)
        ops.check_device_errors()
        return out.cpu().numpy(), torch.cat([rows[:guard], rows[guard + self.tokens:]])


@pytest.mark.parametrize("scores", ["nan scales", "past fp32 by no scale"])
@pytest.mark.parametrize("lens", [[640, 300, 4096], [16000, 640], [40000, 17000, 300]])
def test_scores_of_no_number_stay_in_their_row(lens, scores):
    """Blocks whose bounds hold anything: as many as asked for are chosen, no more."""
    b = Bounds(lens, 2, 128, seed=1)
    q = torch.ones(len(lens), 16, 128, dtype=torch.bfloat16, device="cuda")
    if scores == "nan scales":
        b.scales.fill_(float("nan"))
    else:
        q.fill_(2.0 ** 115)  # (each sum is past fp32 and then multiplied by a scale of 0)
        b.codes.fill_(127)
        b.scales.zero_()
    for n_sel, sinks, recent in ((5, 1, 2), (3, 1, 2), (16, 0, 1)):
        got, guard = b.choose(q, n_sel, sinks, recent)
        assert (guard == -9).all()
        assert (np.diff(got, axis=-1) > 0).all() and (got >= 0).all()
        assert (got[..., -1] < -(-np.array(lens)[:, None] // 16)).all()


@pytest.mark.parametrize("n_kv,G,d", [(2, 8, 128), (1, 1, 64), (4, 2, 128)])
@pytest.mark.parametrize("lens", [[640, 300, 4096], [16000, 640, 90], [40000, 17000, 300]])
def test_scores_outside_fp32_keep_their_order(lens, n_kv, G, d):
    """Queries and keys of any finite size: the integer sums and the powers of two decide,
    whether or not their product is an fp32 number."""
    b = Bounds(lens, n_kv, d, seed=G)
    rng = np.random.default_rng(7)
    cases = [(1e38, 2.0 ** rng.integers(-3, 4, b.scales.shape)),     # past the largest
             (3e38, 2.0 ** rng.integers(100, 123, b.scales.shape)),
             (1e-37, 2.0 ** rng.integers(-126, -100, b.scales.shape)),  # below the smallest
             (1e-39, 2.0 ** rng.integers(-126, 123, b.scales.shape)),
             (1.0, np.where(rng.random(b.scales.shape) < 0.5, 0.0, 2.0 ** -126)),
             (2e38, np.where(rng.random(b.scales.shape) < 0.9, 0.0, 64.0))]
    g = torch.Generator().manual_seed(1)
    for size, scales in cases:
        q = (torch.rand(len(lens), n_kv * G, d, generator=g) * 2 - 1) * size
        q[0, ::2] *= 2.0 ** -20  # (heads of other sizes in a group)
        q = q.bfloat16().cuda()
        b.scales = torch.from_numpy(scales).float().cuda()
        got, guard = b.choose(q, 17, 1, 2)
        want = R.choose(q.cpu().double().numpy(), b.codes.cpu().double().numpy(), scales,
                        b.tables, b.lens, b.starts, b.block, 17, 1, 2, np.zeros_like(got))
        assert np.array_equal(got, want), size
        assert (guard == -9).all()


@pytest.mark.parametrize("in_place", [False, True])
def test_entries_that_name_no_block_are_not_handed_out(in_place):
    """Evicted from a table with bad entries: flagged, the blocks of the others returned in
    order, and the next step gets blocks without a flag."""
    requests, n, budget, pushed = 300, 200, 40, 2
    c = R.Cache([(n, 0)] * requests, 1, 64, 16, False, seed=1)
    rng = np.random.default_rng(1)
    for s, col in zip(rng.integers(0, requests, 40), rng.integers(3, 13, 40)):
        c.tables[s, col] = rng.choice([-1, c.blocks, 2 ** 31 - 1, -2 ** 31])
    c.tables[7, 3:13] = -1
    entries = c.tables[:, 3:13].ravel()
    good = entries[(entries >= 0) & (entries < c.blocks)]
    assert len(good) < entries.size - 20 and entries.size > 2048
    i32 = dict(dtype=torch.int32, device="cuda")
    tables, lens, _ = c.step()
    free, count = torch.full((c.blocks,), -5, **i32), torch.tensor([pushed], **i32)
    free[:pushed] = torch.from_numpy(c.spare[:pushed]).int()
    out = None if in_place else torch.empty_like(lens)
    w = torch.rand(requests, 1, n, device="cuda")
    left = ops.evict_tokens(c.k, c.v, w, tables, lens, torch.full((requests,), budget, **i32), free,
                            count, num_sinks=budget // 2, num_recent=budget // 2, max_seq_len=n,
                            seq_lens_out=out)
    with pytest.raises(ops.PagedAttnError, match="out of range"):
        ops.check_device_errors()
    assert left.tolist() == [budget] * requests and count.tolist() == [pushed + len(good)]
    want = np.full(c.blocks, -5)
    want[:pushed], want[pushed:pushed + len(good)] = c.spare[:pushed], good
    assert np.array_equal(free.cpu().numpy(), want)
    ops.build_step(left, torch.full((requests,), 16, **i32), tables, free, count, block_size=16,
                   num_tokens=16 * requests)
    ops.check_device_errors()


@pytest.mark.parametrize("fp8", [False, True])
def test_a_row_that_stays_keeps_its_weight(fp8):
    """Rows from or to an entry that names no block do not move, and neither do their weights;
    all others do."""
    c = R.Cache([(300, 0), (90, 0), (2000, 0)], 2, 64, 16, fp8, seed=2)
    tables = c.tables.copy()
    tables[0, 3], tables[0, 9], tables[1, 1], tables[2, 90] = c.blocks, -1, c.blocks + 7, -2
    w = torch.rand(3, 2, 2003, generator=torch.Generator().manual_seed(2))
    budgets, sinks, recent = [150, 60, 1800], 3, 20
    want_rows, want_w = c.parts(), w.numpy().copy()
    for s, (n, B) in enumerate(zip(c.lens, budgets)):
        bad = (tables[s] < 0) | (tables[s] >= c.blocks)
        slot = c.tables[s][np.arange(n) // 16].astype(np.int64) * 16 + np.arange(n) % 16
        for h in range(2):
            middle = sinks + np.argsort(-w[s, h, sinks:n - recent].numpy(), kind="stable")
            keep = np.sort(np.concatenate([np.arange(sinks), middle[:B - sinks - recent],
                                           np.arange(n - recent, n)]))
            to = np.arange(B)
            move = ~bad[keep // 16] & ~bad[to // 16]
            to, keep = to[move], keep[move]
            for x, y in zip(want_rows, c.parts()):
                x[slot[to], h] = y[slot[keep], h]
            want_w[s, h, to] = w[s, h, keep].numpy()
    i32 = dict(dtype=torch.int32, device="cuda")
    wd = w.cuda()
    call = ops.evict_tokens_fp8 if fp8 else ops.evict_tokens
    call(c.k, c.v, wd, torch.from_numpy(tables).cuda(), c.step()[1], torch.tensor(budgets, **i32),
         torch.zeros(c.blocks, **i32), torch.zeros(1, **i32), num_sinks=sinks, num_recent=recent,
         max_seq_len=2000)
    with pytest.raises(ops.PagedAttnError, match="out of range"):
        ops.check_device_errors()
    assert np.array_equal(wd.cpu().numpy(), want_w)
    for got, want in zip(c.parts(), want_rows):
        assert np.array_equal(got, want)


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_every_layer_of_a_model_is_cut(fp8, captured):
    """Layers share tables, lengths, offsets and free list: scratch lengths and counts for
    all calls but the last.  Every layer keeps its own tokens, and the books are kept once."""
    c = R.Cache([(300, 0), (90, 0), (700, 0), (40, 0)], 2, 64, 16, fp8, seed=3)
    budgets, sinks, recent, pushed = [100, 60, 333, 50], 3, 20, 1
    caches = [(c.k, c.v), (c.v.clone(), c.k.clone()), (c.k.flip(0), c.v.flip(0))]
    g = torch.Generator().manual_seed(3)
    weights = [torch.rand(4, 2, 703, generator=g) for _ in caches]
    i32 = dict(dtype=torch.int32, device="cuda")
    tables, lens, _ = c.step()
    free, count = torch.full((c.blocks,), -5, **i32), torch.tensor([pushed], **i32)
    offsets, budgets_d = torch.arange(4, **i32), torch.tensor(budgets, **i32)
    want, start = [], free.tolist()
    for (k, v), w in zip(caches, weights):
        c.k, c.v = k, v
        rows, w64 = c.parts(), w.numpy().copy()
        books = R.evict(rows, w64, c.tables, c.lens, budgets, start, pushed, sinks, recent, 16)
        want.append((rows, w64))
    on_gpu = [w.cuda() for w in weights]
    call = ops.evict_tokens_fp8 if fp8 else ops.evict_tokens

    def every_layer():
        scratch = torch.empty_like(lens), torch.empty_like(count)
        for i, ((k, v), w) in enumerate(zip(caches, on_gpu)):
            last = i + 1 == len(caches)
            call(k, v, w, tables, lens, budgets_d, free, count, num_sinks=sinks,
                 num_recent=recent, max_seq_len=700, seq_lens_out=None if last else scratch[0],
                 free_count_out=None if last else scratch[1],
                 position_offsets=offsets if last else None)

    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            every_layer()
        graph.replay()
    else:
        every_layer()
    ops.check_device_errors()
    for (k, v), w, (rows, w64) in zip(caches, on_gpu, want):
        c.k, c.v = k, v
        for got, expected in zip(c.parts(), rows):
            assert np.array_equal(got, expected)
        assert np.array_equal(w.cpu().numpy(), w64)
    assert lens.tolist() == books[0] and free.tolist() == books[1]
    assert count.tolist() == [books[2]]
    assert (offsets.cpu() - torch.arange(4)).tolist() == books[3]


# ------------------------------------------------ longer than what shared memory holds
STAGED = (196624 - 16) * 32 // (32 * 4 + 8)  # about: bits, prefix counts and weights of a request


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("lens,budgets,most", [
    ([46_000, 300], [20_000, 200], 46_000),        # the weights held in shared memory ...
    ([46_800, 300], [20_000, 200], 46_800),        # ... and read from memory in each pass
    ([200_001, 60_000, 47_000], [150_000, 33, 46_999], 200_001),
    ([70_000, 9_000], [4_000, 8_000], 524_288),    # the longest that a call may say
])
def test_requests_past_the_weights_held(lens, budgets, most, fp8):
    assert min(abs(n - STAGED) for n in (46_000, 46_800)) < 600 and 46_000 < STAGED < 46_800
    c = R.Cache([(n, 0) for n in lens], 1, 64, 16, fp8, seed=5)
    width = -(-most // 16)
    tables = np.full((len(lens), width), -1, np.int32)
    tables[:, :c.tables.shape[1]] = c.tables[:, :width]
    g = torch.Generator().manual_seed(5)
    w = (torch.randn(len(lens), 1, max(lens), generator=g) * 2).exp()
    w[0, 0, 1000:1500] = 0.25  # ties across words and windows
    full = torch.zeros(len(lens), 1, most)
    full[..., :max(lens)] = w
    sinks, recent, pushed = 5, 17, 2
    i32 = dict(dtype=torch.int32, device="cuda")
    free, count = torch.full((c.blocks,), -1, **i32), torch.tensor([pushed], **i32)
    rows, w64 = c.parts(), full.numpy().copy()
    books = R.evict(rows, w64, c.tables, c.lens, budgets, free.tolist(), pushed, sinks, recent, 16)
    wd, seq = full.cuda(), c.step()[1]
    call = ops.evict_tokens_fp8 if fp8 else ops.evict_tokens
    call(c.k, c.v, wd, torch.from_numpy(tables).cuda(), seq, torch.tensor(budgets, **i32), free,
         count, num_sinks=sinks, num_recent=recent, max_seq_len=most)
    ops.check_device_errors()
    assert seq.tolist() == books[0] and free.tolist() == books[1] and count.tolist() == [books[2]]
    assert np.array_equal(wd.cpu().numpy().view(np.int32), w64.view(np.int32))
    for got, want in zip(c.parts(), rows):
        assert np.array_equal(got, want)


# --------------------------------------------- weights whose scores are computed again
KEPT_BYTES, MOST_CTAS = 44 * 1024, 16


@pytest.mark.parametrize("n_kv,G,d,block,fp8", [
    (1, 8, 64, 16, True), (1, 8, 128, 16, True), (2, 8, 128, 32, True), (1, 4, 128, 16, True),
    (1, 2, 64, 32, True), (1, 8, 128, 32, False), (1, 4, 64, 16, False), (1, 1, 128, 16, False),
    (1, 1, 64, 16, True),
])
def test_scores_past_those_kept(n_kv, G, d, block, fp8):
    """A context whose scores do not fit beside the pages even over the largest cluster: those
    of its last pages are computed again from K, and the new token is among them."""
    kept = KEPT_BYTES // (16 * G * 4)                # pages of a CTA whose scores stay
    n = MOST_CTAS * (kept + 70) * 16 - 5
    share = -(-(-(-n // 16)) // MOST_CTAS)
    assert share >= kept + 70
    c = R.Cache([(n - 1, 1), (29, 1), (n // 2, 1)], n_kv, d, block, fp8, seed=G, pad=1)
    q, q64 = c.queries(n_kv * G, 1)
    tables, lens, starts = c.step()
    before = torch.rand(3, n_kv, n + 3, generator=torch.Generator().manual_seed(G))
    for s, m in enumerate(c.lens):
        before[s, :, m - 1] = float("nan")           # (the new token's entry starts from 0)
    w = before.cuda()
    call = ops.paged_attention_weights_fp8 if fp8 else ops.paged_attention_weights
    out = call(q, c.k, c.v, tables, lens, starts, d ** -0.5, w, max_q_len=1, max_seq_len=n)
    ops.check_device_errors()
    o64, A, E, w64, tol = R.weights_attention(q64, c.K, c.V, c.tables, c.lens, c.starts, d ** -0.5,
                                              block, before.numpy())
    got = w.double().cpu().numpy()
    for s, m in enumerate(c.lens):
        assert (np.abs(got[s, :, :m] - w64[s, :, :m]) <= tol[s, :, :m] + 1e-30).all()
        assert torch.equal(w[s, :, m:].cpu(), before[s, :, m:])
    rows = slice(0, 3)
    R.assert_blocks_close(out.double().cpu().numpy()[rows], (o64[rows], A[rows], E[rows]))
