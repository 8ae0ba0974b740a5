"""The operators for long contexts run together as a serving loop runs them: step inputs,
rotary positions with the slot scatter, bounds of the new blocks, the choice of blocks and
attention over them or attention with accumulated weights, eviction down to a budget, and
the evicted blocks handed out again.  Every step is checked against the plain 64-bit
definitions; a captured step is replayed against the same steps launched one by one."""
import math

import numpy as np
import pytest
import torch

import long_reference as R
import step_reference as S
from paged_kv_cache_174_gb300 import ops

pytestmark = pytest.mark.gpu

BS, NQ, NKV, D = 16, 8, 2, 64
SELECTED, SINK_BLOCKS, RECENT_BLOCKS = 5, 1, 2


class Loop:
    def __init__(self, requests, fp8, pool=90, width=40, seed=0):
        self.S, self.fp8 = requests, fp8
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.inv_freq = 10000.0 ** (-np.arange(D // 2) * 2.0 / D)
        self.freq_d = torch.from_numpy(self.inv_freq).cuda()
        self.free = rng.permutation(pool).astype(np.int32)
        self.count = pool
        self.tables = np.full((requests, width), -1, np.int32)
        self.lens = np.zeros(requests, np.int64)
        self.offsets = np.zeros(requests, np.int64)
        i32 = dict(dtype=torch.int32, device="cuda")
        self.tables_d = torch.from_numpy(self.tables).cuda()
        self.free_d = torch.from_numpy(self.free).cuda()
        self.count_d = torch.tensor([pool], **i32)
        self.lens_d, self.offsets_d = torch.zeros(requests, **i32), torch.zeros(requests, **i32)
        if fp8:
            self.kc, self.vc = ops.empty_fp8_cache(pool, BS, NKV, D)
        else:
            self.kc = torch.full((pool, BS, NKV, D), float("nan"), dtype=torch.bfloat16,
                                 device="cuda")
            self.vc = self.kc.clone()
        self.codes_d, self.scales_d = ops.alloc_bounds(pool, NKV, D)
        self.codes, self.scales = (x.cpu().double().numpy() for x in (self.codes_d, self.scales_d))
        self.weights = torch.full((requests, NKV, width * BS), float("nan"), device="cuda")
        self.scale = 1.0 / math.sqrt(D)

    def qkv(self, T):
        return torch.randn(T, (NQ + 2 * NKV) * D, device="cuda", dtype=torch.bfloat16,
                           generator=self.gen)

    def op(self, name):
        return getattr(ops, name + "_fp8" if self.fp8 else name)

    def rows(self, cache):
        if not self.fp8:
            return cache.cpu().double().numpy().reshape(-1, NKV, D)
        codes, scales = ops.fp8_cache_views(cache, NKV, D)
        value = codes.view(torch.float8_e4m3fn).float() * scales[..., None]
        return value.cpu().double().numpy().reshape(-1, NKV, D)

    def parts(self):
        out = []
        for x in (self.kc, self.vc):
            if self.fp8:
                c, f = ops.fp8_cache_views(x, NKV, D)
                out += [c.cpu().numpy().reshape(-1, NKV, D).copy(),
                        f.cpu().view(torch.int32).numpy().reshape(-1, NKV).copy()]
            else:
                out.append(x.cpu().view(torch.int16).numpy().reshape(-1, NKV, D).copy())
        return out

    # ------------------------------------------------ on the device; no read of its memory
    def scatter(self, new_d, T, qkv):
        lens, starts, slots, pos = ops.build_step(
            self.lens_d, new_d, self.tables_d, self.free_d, self.count_d, block_size=BS,
            num_tokens=T, position_offsets=self.offsets_d, seq_lens=self.lens_d)
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([NQ * D, NKV * D, NKV * D], 1))
        q = self.op("rotary_reshape_and_cache")(q, k, v, pos, self.freq_d, self.kc, self.vc, slots)
        self.op("summarize_blocks")(self.kc, self.tables_d, lens, starts, self.codes_d,
                                    self.scales_d, num_tokens=T)
        return starts, slots, pos, q

    def attend_weights(self, q, starts, max_q_len, max_seq_len, workspace=None, **kw):
        return self.op("paged_attention_weights")(
            q, self.kc, self.vc, self.tables_d, self.lens_d, starts, self.scale, self.weights,
            max_q_len=max_q_len, max_seq_len=max_seq_len, workspace=workspace, **kw)

    def attend_blocks(self, q, starts, max_seq_len, **kw):
        chosen = ops.select_blocks(q, self.codes_d, self.scales_d, self.tables_d, self.lens_d,
                                   starts, num_selected=SELECTED, num_sinks=SINK_BLOCKS,
                                   num_recent=RECENT_BLOCKS, block_size=BS,
                                   max_seq_len=max_seq_len)
        return chosen, self.op("paged_attention_blocks")(
            q, self.kc, self.vc, self.tables_d, self.lens_d, starts, self.scale, chosen, **kw)

    def cut(self, budgets_d, max_seq_len):
        lens = self.op("evict_tokens")(
            self.kc, self.vc, self.weights, self.tables_d, self.lens_d, budgets_d, self.free_d,
            self.count_d, num_sinks=2, num_recent=9, max_seq_len=max_seq_len,
            position_offsets=self.offsets_d)
        assert lens is self.lens_d
        self.op("summarize_blocks")(self.kc, self.tables_d, lens, None, self.codes_d,
                                    self.scales_d)

    # ------------------------------------------------------------------ checked
    def step(self, new, pad, chosen_only):
        new = np.asarray(new)
        T = int(new.sum()) + pad
        starts, slots, pos, q = self.scatter(
            torch.tensor(new, dtype=torch.int32, device="cuda"), T, self.qkv(T))
        tables, lens, w_starts, w_slots, w_pos, count, flagged = S.build_step(
            self.lens, new, self.tables, self.free, self.count, BS, T, 1, self.offsets)
        assert not flagged
        for got, want in ((self.tables_d, tables), (self.lens_d, lens), (starts, w_starts),
                          (slots, w_slots), (pos, w_pos), (self.count_d, [count])):
            assert np.array_equal(got.cpu().numpy(), want)
        self.tables, self.lens, self.count = tables, lens.astype(np.int64), count
        K, V = self.rows(self.kc), self.rows(self.vc)
        self.check_bounds(K, w_starts)
        q64 = q.cpu().double().numpy()
        most, before = int(self.lens.max()), self.weights.cpu().numpy()
        args = (tables, list(lens), w_starts)
        n = int(new.sum())
        if chosen_only:
            chosen, out = self.attend_blocks(q, starts, most)
            got = chosen.cpu().numpy()
            want = R.choose(q64, self.codes, self.scales, *args, BS, SELECTED, SINK_BLOCKS,
                            RECENT_BLOCKS, got)
            assert np.array_equal(got, want)
            ref = R.blocks_attention(q64, K, V, *args, self.scale, BS, got)
            R.assert_blocks_close(out.cpu().double().numpy(), ref)
            self.new_weights_start_from_zero(new)
        else:
            out = self.attend_weights(q, starts, int(new.max()), most).cpu().double().numpy()
            o64, A, E, w64, tol = R.weights_attention(q64, K, V, *args, self.scale, BS, before)
            w = self.weights.cpu().double().numpy()
            for s in np.flatnonzero(new):
                at = (s, slice(None), slice(0, int(lens[s])))
                assert (np.abs(w[at] - w64[at]) <= tol[at] + 1e-30).all()
            size = E[:n] / (4 * D * R.EPS)  # (an upper bound of the scores' terms)
            S.assert_window_close(out[:n], (o64[:n], A[:n], size), self.fp8)
        ops.check_device_errors()

    def new_weights_start_from_zero(self, new):
        """Tokens that only chosen blocks were attended with have no weight of their own."""
        for s, n in enumerate(self.lens):
            self.weights[s, :, int(n) - int(new[s]):int(n)] = 0

    def check_bounds(self, K, starts):
        self.codes, self.scales = R.bounds(self.codes, self.scales, K, self.tables, self.lens,
                                           starts, BS)
        assert np.array_equal(self.codes_d.cpu().double().numpy(), self.codes)
        assert np.array_equal(self.scales_d.cpu().double().numpy(), self.scales)

    def evict(self, budgets):
        parts, w = self.parts(), self.weights.cpu().numpy()
        most = int(self.lens.max())
        lens, free, count, gone = R.evict(parts, w, self.tables, self.lens, budgets, self.free,
                                          self.count, 2, 9, BS)
        self.cut(torch.tensor(budgets, dtype=torch.int32, device="cuda"), most)
        ops.check_device_errors()
        self.lens, self.count = np.asarray(lens, np.int64), count
        self.free, self.offsets = np.asarray(free, np.int32), self.offsets + gone
        for got, want in ((self.lens_d, self.lens), (self.free_d, self.free),
                          (self.count_d, [count]), (self.offsets_d, self.offsets),
                          (self.weights.view(torch.int32), w.view(np.int32))):
            assert np.array_equal(got.cpu().numpy(), want)
        for got, want in zip(self.parts(), parts):
            assert np.array_equal(got, want)
        self.check_bounds(self.rows(self.kc), None)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_serving_loop(fp8):
    """Prompts in chunks, then decodes over chosen blocks or all, cut down to budgets every
    few steps: a pool too small for the whole sequences, the positions go on."""
    loop = Loop(5, fp8, pool=64)
    rng = np.random.default_rng(2)
    left = np.array([300, 17, 1, 129, 400])  # prompt tokens still to come
    for step in range(28):
        new = np.where(left > 0, np.minimum(left, rng.integers(1, 70, 5)), 1)
        new[rng.random(5) < 0.1] = 0
        if not new.any():
            new[0] = 1
        loop.step(new, int(rng.integers(0, 5)), chosen_only=step % 3 == 2)
        left = np.maximum(0, left - new)
        if step % 4 == 3:
            loop.evict(rng.integers(60, 150, 5))
    positions = loop.lens + loop.offsets
    assert positions.max() > 400 and positions.sum() > 64 * BS * 0.8
    assert (loop.offsets > 0).sum() >= 3


def decode(loop, new_d, T, qkv, budgets_d):
    """A decode step with everything in it."""
    starts, _, _, q = loop.scatter(new_d, T, qkv)
    whole = loop.attend_weights(q, starts, 1, 200)
    chosen, out = loop.attend_blocks(q, starts, 200)
    loop.cut(budgets_d, 200)
    return whole, chosen, out


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


STATE = ("tables_d", "count_d", "lens_d", "offsets_d", "free_d", "codes_d", "scales_d", "kc", "vc")


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_captured_decode_steps(fp8):
    """Captured once and replayed, with eviction: the same bits as the steps launched one by
    one on another stream."""
    loops = [Loop(6, fp8, seed=3) for _ in range(2)]
    for l in loops:
        l.step([33, 16, 2, 70, 15, 64], 0, False)
    eager, captured = loops
    T = 8  # two padded rows
    ones = torch.ones(6, dtype=torch.int32, device="cuda")
    budgets = torch.tensor([40, 30, 12, 75, 100, 60], dtype=torch.int32, device="cuda")
    qkv = captured.qkv(T)
    eager.qkv(T)  # the generators stay alike
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = decode(captured, ones, T, qkv, budgets)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    for _ in range(40):
        with torch.cuda.stream(other):
            x = eager.qkv(T)
            want = decode(eager, ones, T, x, budgets)
        torch.cuda.current_stream().wait_stream(other)
        qkv.copy_(x)
        graph.replay()
        for g, w in zip(got, want):
            assert same(g[:6], w[:6])
        for name in STATE:
            assert same(getattr(captured, name), getattr(eager, name)), name
        for s, n in enumerate(eager.lens_d.tolist()):
            assert same(captured.weights[s, :, :n], eager.weights[s, :, :n])
    ops.check_device_errors()
    assert captured.lens_d.tolist() == [40, 30, 12, 75, 55, 60]


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_two_graphs_with_one_workspace(fp8):
    """Two captured calls of different steps share their workspace, replayed in turn."""
    loops = [Loop(3, fp8, seed=s) for s in (5, 6)]
    steps = ([1, 70, 33], [130, 1, 0])
    work = ops.alloc_weights_workspace(3, 140, NQ, NKV, D, 130, 400)
    graphs, outs, inputs, wants = [], [], [], []
    for loop, new in zip(loops, steps):
        loop.step([40, 100, 7], 0, False)
        T = sum(new)
        starts, _, _, q = loop.scatter(torch.tensor(new, dtype=torch.int32, device="cuda"), T,
                                       loop.qkv(T))
        start = loop.weights.clone()
        wants.append((loop.attend_weights(q, starts, max(new), 400), loop.weights.clone()))
        loop.weights.copy_(start)
        work.fill_(0xff)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(loop.attend_weights(q, starts, max(new), 400, work))
        graphs.append(graph)
        inputs.append((start, q, starts))  # (a graph holds addresses, not tensors)
    for _ in range(3):
        for graph, loop, (start, *_) in zip(graphs, loops, inputs):
            loop.weights.copy_(start)
            graph.replay()
        for loop, out, (want, w) in zip(loops, outs, wants):
            assert same(out, want)
            for s, n in enumerate(loop.lens_d.tolist()):
                assert same(loop.weights[s, :, :n], w[s, :, :n])
    ops.check_device_errors()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_two_steps_at_once(fp8):
    """Steps of two sets of requests on two streams, not ordered against each other."""
    loops, wants, inputs = [Loop(4, fp8, seed=s) for s in (8, 9)], [], []
    new = [90, 1, 30, 64]
    for loop in loops:
        loop.step([100, 47, 200, 3], 0, False)
        T = sum(new)
        starts, _, _, q = loop.scatter(torch.tensor(new, dtype=torch.int32, device="cuda"), T,
                                       loop.qkv(T))
        start = loop.weights.clone()
        wants.append([loop.attend_weights(q, starts, 90, 400), loop.weights.clone(),
                      *loop.attend_blocks(q, starts, 400)])
        inputs.append((q, starts, start))
    streams = [torch.cuda.Stream() for _ in loops]
    torch.cuda.synchronize()
    for _ in range(5):
        gots = []
        for loop, stream, (q, starts, start) in zip(loops, streams, inputs):
            with torch.cuda.stream(stream):
                loop.weights.copy_(start)
                gots.append([loop.attend_weights(q, starts, 90, 400), loop.weights,
                             *loop.attend_blocks(q, starts, 400)])
        torch.cuda.synchronize()
        for loop, got, want in zip(loops, gots, wants):
            for i in (0, 2, 3):
                assert same(got[i], want[i])
            for s, n in enumerate(loop.lens_d.tolist()):
                assert same(got[1][s, :, :n], want[1][s, :, :n])
    ops.check_device_errors()


def test_requests_of_nothing():
    """No requests, no tokens, and requests without a token or a cached one."""
    loop = Loop(2, False)
    empty = torch.zeros(0, NQ, D, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    for requests in (0, 2):
        tables, lens = loop.tables_d[:requests], loop.lens_d[:requests]
        starts = torch.zeros(requests + 1, **i32)
        before = {name: getattr(loop, name).clone() for name in STATE}
        ops.summarize_blocks(loop.kc, tables, lens, starts, loop.codes_d, loop.scales_d,
                             num_tokens=0)
        ops.summarize_blocks(loop.kc, tables, lens, None, loop.codes_d, loop.scales_d)
        chosen = ops.select_blocks(empty, loop.codes_d, loop.scales_d, tables, lens, starts,
                                   num_selected=3, block_size=BS, max_seq_len=1)
        assert chosen.shape == (0, NKV, 3)
        out = ops.paged_attention_blocks(empty, loop.kc, loop.vc, tables, lens, starts, 1.0,
                                         chosen)
        assert out.shape == empty.shape
        out = ops.paged_attention_weights(empty, loop.kc, loop.vc, tables, lens, starts, 1.0,
                                          loop.weights[:requests], max_q_len=1, max_seq_len=1)
        assert out.shape == empty.shape
        ops.evict_tokens(loop.kc, loop.vc, loop.weights[:requests], tables, lens,
                         torch.zeros(requests, **i32), loop.free_d, loop.count_d, max_seq_len=1)
        ops.check_device_errors()
        for name in STATE:
            assert same(getattr(loop, name), before[name]), name


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_pages_behind_32_bits_of_bytes(fp8):
    """The same requests at the far end of a cache of more than 2^32 bytes (8-bit codes: 2^31):
    the same bits."""
    n_kv, d, blocks = 8, 128, 140_000
    c = R.Cache([(300, 1), (40, 70), (1000, 1), (0, 33)], n_kv, d, BS, fp8, seed=4)
    tables, lens, starts = c.step()
    q, _ = c.queries(4 * n_kv, 4)
    far = blocks - c.blocks
    i32 = dict(dtype=torch.int32, device="cuda")

    def suffixed(name):
        return getattr(ops, name + "_fp8" if fp8 else name)

    def everything(k, v, first, pool):
        tables_ = torch.where(tables >= 0, tables + first, tables)
        codes, scales = ops.alloc_bounds(pool, n_kv, d)
        suffixed("summarize_blocks")(k, tables_, lens, None, codes, scales)
        chosen = ops.select_blocks(q, codes, scales, tables_, lens, starts, num_selected=6,
                                   block_size=BS, max_seq_len=1001)
        out = suffixed("paged_attention_blocks")(q, k, v, tables_, lens, starts, 0.1, chosen)
        w = torch.zeros(4, n_kv, 1001, device="cuda")
        whole = suffixed("paged_attention_weights")(q, k, v, tables_, lens, starts, 0.1, w,
                                                    max_q_len=70, max_seq_len=1001)
        free, count = torch.zeros(pool, **i32), torch.zeros(1, **i32)
        left = suffixed("evict_tokens")(k, v, w, tables_, lens, lens // 2, free, count,
                                        num_sinks=2, num_recent=3, max_seq_len=1001,
                                        seq_lens_out=torch.empty_like(lens))
        n = int(count)
        return [codes[first:first + c.blocks], scales[first:first + c.blocks], chosen, out, w,
                whole, left, count, free[:n] - first, k[first:first + c.blocks],
                v[first:first + c.blocks]]

    big = [torch.empty(blocks, *x.shape[1:], dtype=x.dtype, device="cuda") for x in (c.k, c.v)]
    for x, y in zip(big, (c.k, c.v)):
        x[far:] = y
    near = everything(c.k, c.v, 0, c.blocks)
    for got, want in zip(everything(*big, far, blocks), near):
        assert same(got, want)
    ops.check_device_errors()
    assert big[0].numel() * big[0].element_size() > (2 ** 31 if fp8 else 2 ** 32)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_bounds_far_above_the_lengths(fp8):
    """Maxima as a captured step has them, far above any length: the same choice and the
    same tokens kept, and weights to their tolerance."""
    n_kv, d = 2, 64
    c = R.Cache([(300, 1), (15, 1), (1000, 1), (40, 70), (0, 33), (7, 0)], n_kv, d, BS, fp8, seed=6)
    width = 8192
    wide = np.full((len(c.lens), width), -1, np.int32)
    wide[:, :c.tables.shape[1]] = c.tables
    c.tables = wide
    tables, lens, starts = c.step()
    q, q64 = c.queries(4 * n_kv, 6)
    codes, scales = ops.alloc_bounds(c.blocks, n_kv, d)
    name = (lambda n: n + "_fp8") if fp8 else (lambda n: n)
    getattr(ops, name("summarize_blocks"))(c.k, tables, lens, None, codes, scales)
    chosen = [ops.select_blocks(q, codes, scales, tables, lens, starts, num_selected=6,
                                block_size=BS, max_seq_len=most, out=torch.full(
                                    (c.tokens, n_kv, 6), -7, dtype=torch.int32, device="cuda"))
              for most in (1001, width * BS, 49152 * BS)]
    assert same(chosen[0], chosen[1]) and same(chosen[0], chosen[2])
    w = torch.zeros(len(c.lens), n_kv, width * BS, device="cuda")
    out = getattr(ops, name("paged_attention_weights"))(
        q, c.k, c.v, tables, lens, starts, 0.1, w, max_q_len=2048, max_seq_len=width * BS)
    ops.check_device_errors()
    o64, A, E, w64, tol = R.weights_attention(q64, c.K, c.V, c.tables, c.lens, c.starts, 0.1, BS,
                                              np.zeros((len(c.lens), n_kv, 1001)))
    got = w.double().cpu().numpy()
    assert (np.abs(got[..., :1001] - w64) <= tol + 1e-30).all() and not got[..., 1001:].any()
    S.assert_window_close(out.cpu().double().numpy(), (o64, A, E / (4 * d * R.EPS)), fp8)
    budgets, i32 = lens // 2, dict(dtype=torch.int32, device="cuda")
    kept = []
    for most in (1001, width * BS):
        k, v, weights = c.k.clone(), c.v.clone(), w.clone()
        free, count = torch.zeros(c.blocks, **i32), torch.zeros(1, **i32)
        left = getattr(ops, name("evict_tokens"))(
            k, v, weights, tables, lens, budgets, free, count, max_seq_len=most,
            seq_lens_out=torch.empty_like(lens))
        kept.append((k, v, weights, left, free, count))
    ops.check_device_errors()
    assert kept[0][3].tolist() == budgets.tolist()
    for a, b in zip(*kept):
        assert same(a, b)
