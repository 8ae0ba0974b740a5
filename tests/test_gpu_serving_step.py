"""The operators around a step run together as a serving loop runs them: step
inputs from lengths, rotary positions with the slot scatter, sliding-window
attention, blocks behind the window handed back to the free list.  Every step
is checked against the plain 64-bit definitions; a captured decode step is
replayed against the same steps launched one by one."""
import math

import numpy as np
import pytest
import torch

import step_reference as R
from paged_kv_cache_174_gb300 import ops

pytestmark = pytest.mark.gpu

BS, NQ, NKV, D, AXES = 16, 8, 2, 64, 3


class Loop:
    def __init__(self, S, window, sinks, fp8, pool=90, width=40, seed=0):
        self.S, self.window, self.sinks, self.fp8 = S, window, sinks, fp8
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.inv_freq = 10000.0 ** (-np.arange(D // 2) * 2.0 / D)
        self.axes = rng.integers(0, AXES, D // 2).astype(np.int32)
        self.freq_d = torch.from_numpy(self.inv_freq).cuda()
        self.axes_d = torch.from_numpy(self.axes).cuda()
        self.free = rng.permutation(pool).astype(np.int32)
        self.count = pool
        self.tables = np.full((S, width), -1, np.int32)
        self.lens = np.zeros(S, np.int64)
        self.tables_d = torch.from_numpy(self.tables).cuda()
        self.free_d = torch.from_numpy(self.free).cuda()
        self.count_d = torch.tensor([pool], dtype=torch.int32, device="cuda")
        self.lens_d = torch.zeros(S, dtype=torch.int32, device="cuda")
        if fp8:
            self.kc, self.vc = ops.empty_fp8_cache(pool, BS, NKV, D)
        else:
            self.kc = torch.full((pool, BS, NKV, D), float("nan"), dtype=torch.bfloat16,
                                 device="cuda")
            self.vc = self.kc.clone()
        self.scale = 1.0 / math.sqrt(D)

    def rows(self, cache):
        if not self.fp8:
            return cache.cpu().double().numpy().reshape(-1, NKV, D)
        codes, scales = ops.fp8_cache_views(cache, NKV, D)
        value = codes.view(torch.float8_e4m3fn).float().cpu().double().numpy()
        return value.reshape(-1, NKV, D) * scales.cpu().double().numpy().reshape(-1, NKV, 1)

    def layer(self, new_d, T, max_q_len, qkv, max_seq_len, **bufs):
        """One step on the device; nothing here reads device memory."""
        lens, starts, slots, pos = ops.build_step(
            self.lens_d, new_d, self.tables_d, self.free_d, self.count_d, block_size=BS,
            num_tokens=T, num_axes=AXES, seq_lens=self.lens_d, **bufs)
        q, k, v = (x.unflatten(1, (-1, D)) for x in qkv.split([NQ * D, NKV * D, NKV * D], 1))
        rotary = ops.rotary_reshape_and_cache_fp8 if self.fp8 else ops.rotary_reshape_and_cache
        q = rotary(q, k, v, pos, self.freq_d, self.kc, self.vc, slots, axes=self.axes_d)
        attend = ops.paged_attention_window_fp8 if self.fp8 else ops.paged_attention_window
        out = attend(q, self.kc, self.vc, self.tables_d, lens, starts, self.scale,
                     window=self.window, num_sinks=self.sinks, max_q_len=max_q_len,
                     max_seq_len=max_seq_len)
        return starts, slots, pos, q, out

    def qkv(self, T):
        return torch.randn(T, (NQ + 2 * NKV) * D, device="cuda", dtype=torch.bfloat16,
                           generator=self.gen)

    def step(self, new, pad=0):
        new = np.asarray(new)
        T = int(new.sum()) + pad
        qkv = self.qkv(T)
        starts, slots, pos, q, out = self.layer(
            torch.tensor(new, dtype=torch.int32, device="cuda"), T, int(new.max()), qkv,
            int((self.lens + new).max()))
        ops.check_device_errors()
        tables, lens, w_starts, w_slots, w_pos, count, flagged = R.build_step(
            self.lens, new, self.tables, self.free, self.count, BS, T, AXES)
        assert not flagged
        for got, want in ((self.tables_d, tables), (self.lens_d, lens), (starts, w_starts),
                          (slots, w_slots), (pos, w_pos), (self.count_d, [count])):
            assert np.array_equal(got.cpu().numpy(), want)
        x = qkv.cpu().double().numpy()
        xq, xk, xv = (x[:, a:b].reshape(T, -1, D) for a, b in
                      ((0, NQ * D), (NQ * D, (NQ + NKV) * D), ((NQ + NKV) * D, None)))
        n = int(new.sum())
        # eager T may hold padded rows: their queries are turned by position 0
        q64 = q.cpu().double().numpy()
        want, size = R.rotate(xq, w_pos, self.inv_freq, self.axes, False)
        assert (np.abs(q64 - want) <= R.HALF_BF16 * np.abs(want) + 2.0 ** -20 * size).all()
        K, V = self.rows(self.kc), self.rows(self.vc)
        want, size = R.rotate(xk, w_pos, self.inv_freq, self.axes, False)
        got = K[w_slots[:n]]
        # half a step of the stored type: bf16, or a code (2^-4, and 2^-10 in
        # units of the scale at the bottom)
        half = 2.0 ** -4 if self.fp8 else R.HALF_BF16
        low = 2.0 ** -10 * np.abs(want).max(-1, keepdims=True) / 448 if self.fp8 else 0.0
        tol = (half * np.abs(want) + low) * (1 + 2.0 ** -8) + 2.0 ** -16 * size
        assert (np.abs(got - want[:n]) <= tol[:n]).all()
        ref = R.window_attention(q64, K, V, tables, lens, w_starts, self.scale, self.window,
                                 self.sinks, BS)
        R.assert_window_close(out.cpu().double().numpy(), ref, self.fp8)
        self.tables, self.lens, self.count = tables, lens.astype(np.int64), count

    def release(self):
        """Hand back the blocks that no later row sees, on both sides."""
        for s in range(self.S):
            first = max(0, int(self.lens[s]) - self.window + 1) // BS
            for j in range(-(-self.sinks // BS), first):
                b = int(self.tables[s, j])
                if b < 0:
                    continue
                self.free[self.count] = b
                self.count += 1
                self.tables[s, j] = -1
        self.tables_d.copy_(torch.from_numpy(self.tables))
        self.free_d.copy_(torch.from_numpy(self.free))
        self.count_d.fill_(self.count)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_serving_loop(fp8):
    """Prompts in chunks, then decodes, over a pool too small for the whole
    sequences: only the sinks and the window are held."""
    loop = Loop(5, window=70, sinks=4, fp8=fp8, pool=64)
    rng = np.random.default_rng(1)
    left = np.array([300, 17, 1, 129, 550])  # prompt tokens still to come
    for step in range(24):
        new = np.where(left > 0, np.minimum(left, rng.integers(1, 90, 5)), 1)
        new[rng.random(5) < 0.1] = 0
        if not new.any():
            new[0] = 1
        loop.step(new, pad=int(rng.integers(0, 5)))
        left = np.maximum(0, left - new)
        loop.release()
    assert int(loop.lens.max()) > 400
    assert loop.lens.sum() > 64 * BS * 0.8


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_captured_decode_steps(fp8):
    """A decode step captured once and replayed: lengths, tables and the free
    list go on by themselves; the same bits as the steps launched one by one."""
    loops = [Loop(6, window=40, sinks=2, fp8=fp8, seed=3) for _ in range(2)]
    for l in loops:
        l.step([33, 16, 2, 70, 15, 64])
    eager, cap = loops
    T = 8  # two padded rows
    ones = torch.ones(6, dtype=torch.int32, device="cuda")
    qkv = cap.qkv(T)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = cap.layer(ones, T, 1, qkv, 200)
    eager.qkv(T)  # the generators stay alike
    for _ in range(40):
        x = eager.qkv(T)
        qkv.copy_(x)
        graph.replay()
        want = eager.layer(ones, T, 1, x, 200)
        for g, w in zip(got[:4], want[:4]):
            assert torch.equal(g, w)
        assert torch.equal(got[4][:6].view(torch.int16), want[4][:6].view(torch.int16))
        for name in ("tables_d", "count_d", "lens_d"):
            assert torch.equal(getattr(cap, name), getattr(eager, name))
    ops.check_device_errors()


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_captured_after_copies_and_other_streams(fp8):
    """A captured step whose inputs come by copies on its own stream and by
    kernels on another that it joins: replayed, it gives what it gave eagerly."""
    a, b = Loop(5, window=50, sinks=3, fp8=fp8, seed=7), Loop(5, window=50, sinks=3, fp8=fp8, seed=7)
    for l in (a, b):
        l.step([20, 1, 300, 16, 47])
    new = torch.tensor([1, 3, 70, 0, 2], dtype=torch.int32, device="cuda")
    T = 76
    source = a.qkv(T)
    want = a.layer(new, T, 70, source, 400)[-1]
    held, into, half = torch.empty_like(new), torch.empty_like(source), source * 0.5
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    start = [x.clone() for x in (b.lens_d, b.tables_d, b.count_d, b.kc, b.vc)]
    with torch.cuda.graph(graph):
        held.copy_(new)
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            torch.add(half, half, out=into)
        for x, y in zip((b.lens_d, b.tables_d, b.count_d, b.kc, b.vc), start):
            x.copy_(y)
        here.wait_stream(side)
        got = b.layer(held, T, 70, into, 400)[-1]
    for _ in range(3):
        got.zero_()
        graph.replay()
        ops.check_device_errors()
        assert torch.equal(got.view(torch.int16), want.view(torch.int16))
        assert torch.equal(b.lens_d, a.lens_d) and torch.equal(b.count_d, a.count_d)
