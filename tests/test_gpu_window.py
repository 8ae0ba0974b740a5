"""Sliding-window attention on the GPU against the 64-bit definition, over both
caches: decode rows, chunks and mixtures, windows and sinks around page and
tile edges, blocks outside every view freed and poisoned, workspaces with and
without room for key pieces, streams and graphs."""
import math

import numpy as np
import pytest
import torch

import step_reference as R
from paged_kv_cache_174_gb300 import ops

pytestmark = pytest.mark.gpu


class Batch:
    """Requests with a paged cache on the host (64 bits) and the device; every
    slot that no row of its request sees holds NaN, every table entry of a block
    without a visible key an id that is out of range."""

    def __init__(self, seed, lens, q_lens, nq, nkv, d, window, sinks, bs=16, fp8=False,
                 scale=None, spread=1.0, tail=0):
        rng = np.random.default_rng(seed)
        self.lens, self.q_lens, self.fp8 = np.array(lens, np.int32), list(q_lens), fp8
        self.window, self.sinks, self.bs = window, sinks, bs
        self.scale = 1.0 / math.sqrt(d) if scale is None else scale
        S, width = len(lens), max(1, -(-max(lens) // bs))
        self.starts = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        T = int(self.starts[-1]) + tail
        seen = np.zeros((S, width * bs), bool)
        for s, (L, n) in enumerate(zip(lens, q_lens)):
            if n:
                j = np.arange(L)
                seen[s, :L] = (j < sinks) | (j > L - n - window)
        held = seen.reshape(S, width, bs).any(-1)
        nb = int(held.sum()) + 3
        ids = rng.permutation(nb)
        self.tables = np.full((S, width), -1, np.int32)
        self.tables[held] = ids[:int(held.sum())]
        self.tables[~held] = rng.choice([-1, nb, 2 ** 31 - 1], int((~held).sum()))
        live = np.zeros((nb, bs), bool)
        live[self.tables[held]] = seen.reshape(S, width, bs)[held]
        live = live.reshape(-1)

        def bf16(shape, s=1.0):
            return torch.from_numpy(rng.standard_normal(shape).astype(np.float32) * s).bfloat16()
        q, K, V = bf16((T, nq, d)), bf16((nb * bs, nkv, d), spread), bf16((nb * bs, nkv, d))
        self.q = q.cuda()
        self.q64 = q.double().numpy()
        if fp8:
            kc, vc = ops.empty_fp8_cache(nb, bs, nkv, d)
            slots = torch.arange(nb * bs, dtype=torch.int32, device="cuda")
            ops.reshape_and_cache_fp8(K.cuda(), V.cuda(), kc, vc, slots)
            rows = []
            for c in (kc, vc):
                codes, scales = ops.fp8_cache_views(c, nkv, d)
                value = codes.view(torch.float8_e4m3fn).float().cpu().double().numpy()
                rows.append(value.reshape(-1, nkv, d)
                            * scales.cpu().double().numpy().reshape(-1, nkv)[..., None])
                dead = torch.from_numpy(~live).cuda().view(codes.shape[:3])
                codes[dead] = 0x7F
                scales[dead] = float("nan")
            self.K, self.V = rows
            self.kc, self.vc = kc, vc
        else:
            K[torch.from_numpy(~live)] = float("nan")
            V[torch.from_numpy(~live)] = float("nan")
            self.K, self.V = K.double().numpy(), V.double().numpy()
            self.kc, self.vc = (x.cuda().view(nb, bs, nkv, d) for x in (K, V))
        self.dt = torch.from_numpy(self.tables).cuda()
        self.dl = torch.from_numpy(self.lens).cuda()
        self.ds = torch.from_numpy(self.starts).cuda()

    def run(self, **kw):
        call = ops.paged_attention_window_fp8 if self.fp8 else ops.paged_attention_window
        kw.setdefault("max_q_len", max(self.q_lens))
        kw.setdefault("max_seq_len", int(self.lens.max()))
        return call(self.q, self.kc, self.vc, self.dt, self.dl, self.ds, self.scale,
                    window=self.window, num_sinks=self.sinks, **kw)

    def reference(self):
        return R.window_attention(self.q64, self.K, self.V, self.tables, self.lens, self.starts,
                                  self.scale, self.window, self.sinks, self.bs)

    def check(self, what="", **kw):
        out = torch.full_like(self.q, 3.0)
        self.run(out=out, **kw)
        ops.check_device_errors()
        ref = self.reference()
        got = out.cpu().double().numpy()
        R.assert_window_close(got, ref, self.fp8, what)
        free = np.isnan(ref[0][:, 0, 0])
        assert (got[free] == 3.0).all(), "rows of no request were written"
        return out


BOTH = pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])


@BOTH
@pytest.mark.parametrize("window,sinks", [
    (1, 0), (1, 1), (2, 0), (15, 4), (16, 0), (16, 16), (17, 3), (33, 17), (100, 0), (128, 4),
    (129, 130), (1000, 1), (5000, 0), (7, 5000),
])
def test_decode_windows(window, sinks, fp8):
    lens = [1, 2, 5, 15, 16, 17, 31, 32, 33, 48, 100, 127, 128, 129, 300, 700]
    Batch(1, lens, [1] * len(lens), 8, 2, 64, window, sinks, fp8=fp8).check()


@BOTH
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [1, 2, 4, 8])
@pytest.mark.parametrize("nkv", [1, 2, 4, 8])
def test_shapes(nkv, group, d, fp8):
    """Every head layout: decode rows beside chunks, 16- and 32-token blocks."""
    bs = 16 if (nkv * group) % 2 else 32
    lens, q_lens = [333, 90, 513, 40, 7, 260], [1, 1, 70, 40, 0, 1]
    Batch(nkv * group, lens, q_lens, nkv * group, nkv, d, 75, 5, bs=bs, fp8=fp8).check()


@BOTH
@pytest.mark.parametrize("window,sinks", [
    (1, 0), (2, 1), (16, 0), (31, 4), (100, 17), (128, 0), (129, 128), (200, 4), (256, 129),
    (640, 300), (9000, 0),
])
@pytest.mark.parametrize("lens,q_lens", [
    ([2], [2]), ([300], [300]), ([700, 33], [37, 2]), ([1000, 129, 128], [128, 129, 1]),
    ([1500], [513]),
])
def test_chunks(lens, q_lens, window, sinks, fp8):
    Batch(2, lens, q_lens, 8, 2, 128, window, sinks, fp8=fp8).check()


@BOTH
@pytest.mark.parametrize("window,sinks", [(40, 4), (150, 0), (129, 140), (2000, 3)])
@pytest.mark.parametrize("group,d", [(1, 64), (1, 128), (2, 128), (4, 64), (4, 128), (8, 64),
                                     (8, 128)])
def test_many_query_tiles(group, d, window, sinks, fp8):
    """Calls with more query tiles than SMs (pairs of tiles), requests of odd
    numbers of tiles, one row, a row more than a tile and a row less among them."""
    tm = 128 // group
    q_lens = [tm, 5 * tm, 1, 2, tm + 1, 2 * tm - 1, 2 * tm, 2 * tm + 1, 6 * tm, 3 * tm + 5]
    lens = [n + x for n, x in zip(q_lens, (0, 700, 300, 0, 33, 128, 1000, 15, 64, 0))]
    Batch(20 + group, lens, q_lens, 8 * group, 8, d, window, sinks, fp8=fp8).check()


@BOTH
@pytest.mark.parametrize("seed", range(24))
def test_random(seed, fp8):
    rng = np.random.default_rng(500 + seed)
    d, g, nkv, bs = (int(rng.choice(x)) for x in ([64, 128], [1, 2, 4, 8], [1, 2, 4, 8],
                                                  [16, 32]))
    S = int(rng.integers(1, 12))
    lens = [int(math.exp(rng.uniform(0, math.log(2500)))) for _ in range(S)]
    q_lens = []
    for L in lens:
        kind = rng.random()
        q_lens.append(1 if kind < 0.5 else 0 if kind < 0.55 else
                      int(rng.integers(1, min(L, 300) + 1)))
    if not any(q_lens):
        q_lens[0] = 1
    window = int(math.exp(rng.uniform(0, math.log(1500))))
    sinks = int(rng.choice([0, 0, 1, 4, 16, 20, 150]))
    Batch(600 + seed, lens, q_lens, g * nkv, nkv, d, window, sinks, bs=bs, fp8=fp8,
          tail=int(rng.integers(0, 4))).check(f"lens {lens} q {q_lens} w {window} n {sinks}")


@BOTH
@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scales(scale, fp8):
    Batch(3, [200, 500], [1, 60], 4, 1, 64, 90, 4, fp8=fp8, scale=scale).check()


@BOTH
def test_few_rows_over_long_contexts(fp8):
    """One request: the window's pages are split over the whole device."""
    Batch(4, [40000], [1], 8, 8, 128, 20000, 64, fp8=fp8).check()
    Batch(5, [20000], [3], 8, 1, 64, 9000, 64, fp8=fp8).check()


@BOTH
def test_many_requests(fp8):
    """More requests than the kernels' shared-memory lists and scans hold."""
    n = 1100
    lens = [17 + i % 40 for i in range(n)]
    Batch(6, lens, [1] * n, 2, 1, 64, 20, 2, fp8=fp8).check()
    Batch(7, lens, [2 + i % 3 for i in range(n)], 2, 1, 64, 20, 2, fp8=fp8).check()
    Batch(7, lens, [2 + i % 16 for i in range(n)], 8, 1, 64, 20, 2, fp8=fp8).check()


@BOTH
def test_window_that_hides_nothing_is_paged_attention(fp8):
    b = Batch(8, [300, 40, 90], [1, 40, 20], 8, 2, 64, 300, 0, fp8=fp8)
    plain = ops.paged_attention_fp8 if fp8 else ops.paged_attention
    want = plain(b.q, b.kc, b.vc, b.dt, b.dl, b.ds, b.scale, max_q_len=40, max_seq_len=300)
    for window, sinks in ((300, 0), (2 ** 31 - 1, 2 ** 31 - 1), (5, 300)):
        b.window, b.sinks = window, sinks
        assert torch.equal(b.run().view(torch.int16), want.view(torch.int16))


@BOTH
def test_same_bits_for_any_block_ids_and_every_run(fp8):
    """A row's result depends on neither the ids of its blocks nor the run."""
    a = Batch(9, [900, 300], [1, 130], 8, 2, 128, 200, 4, fp8=fp8)
    first = a.run().clone()
    for _ in range(3):
        assert torch.equal(a.run().view(torch.int16), first.view(torch.int16))
    nb = a.kc.shape[0]
    perm = torch.randperm(nb, device="cuda")
    back = torch.argsort(perm)
    a.kc, a.vc = a.kc[perm].contiguous(), a.vc[perm].contiguous()
    t = a.dt.long()
    inside = (t >= 0) & (t < nb)
    a.dt = torch.where(inside, back[t.clamp(0, nb - 1)], t).int()
    assert torch.equal(a.run().view(torch.int16), first.view(torch.int16))


@BOTH
def test_workspace_without_room_for_key_pieces(fp8):
    b = Batch(10, [4000], [64], 4, 1, 64, 3000, 4, fp8=fp8)
    whole = b.check()
    small = ops.alloc_workspace(1, 64, 4, 1, 64, 1, 4000)  # a decode-only call's
    out = b.run(workspace=small)
    ops.check_device_errors()
    R.assert_window_close(out.cpu().double().numpy(), b.reference(), fp8)
    assert whole.shape == out.shape
    with pytest.raises(ops.PagedAttnError) as e:
        b.run(workspace=small[:1024])
    assert e.value.code == 6


@BOTH
def test_chunks_only_calls(fp8):
    b = Batch(11, [500, 90], [70, 30], 8, 2, 64, 60, 4, fp8=fp8)
    want = b.check()
    assert torch.equal(b.check(min_q_len=2).view(torch.int16), want.view(torch.int16))
    one = Batch(12, [500, 90], [70, 1], 8, 2, 64, 60, 4, fp8=fp8)
    out = torch.full_like(one.q, 3.0)
    one.run(out=out, min_q_len=2)  # a promise broken: flagged, the row not written
    with pytest.raises(ops.PagedAttnError) as e:
        ops.check_device_errors()
    assert e.value.code == 4
    assert (out[70] == 3.0).all()


@BOTH
@pytest.mark.parametrize("q_len", [1, 40])
def test_lengths_and_ids_out_of_range_are_flagged(q_len, fp8):
    def flagged(b, **kw):
        out = torch.full_like(b.q, 3.0)
        b.run(out=out, **kw)
        with pytest.raises(ops.PagedAttnError) as e:
            ops.check_device_errors()
        assert e.value.code == 4
        return out
    b = Batch(13, [300, 200], [q_len, q_len], 4, 2, 64, 50, 4, fp8=fp8)
    good = b.run()
    out = flagged(b, max_seq_len=250)  # the first request is longer: not written
    assert (out[:q_len] == 3.0).all()
    assert torch.equal(out[q_len:].view(torch.int16), good[q_len:].view(torch.int16))
    b.dl[1] = 64 * 16
    out = flagged(b)  # the second is longer than its table
    assert (out[q_len:] == 3.0).all()
    assert torch.equal(out[:q_len].view(torch.int16), good[:q_len].view(torch.int16))
    b.dl[1] = 200
    for column in (0, 299 // 16):  # a sink's block, and the last of the window
        keep = int(b.dt[0, column])
        for bad in (-1, b.kc.shape[0], 2 ** 31 - 1):
            b.dt[0, column] = bad
            out = flagged(b)
            assert torch.equal(out[q_len:].view(torch.int16), good[q_len:].view(torch.int16))
        b.dt[0, column] = keep
    assert torch.equal(b.run().view(torch.int16), good.view(torch.int16))
    ops.check_device_errors()


@BOTH
def test_infinite_keys_of_one_request_stay_there(fp8):
    if fp8:
        pytest.skip("the 8-bit cache holds no infinities")
    b = Batch(14, [200, 210, 64], [1, 50, 64], 4, 2, 64, 60, 4)
    good = b.run()
    slot = int(b.dt[0, 190 // 16]) * 16 + 190 % 16
    b.kc.view(-1, 2, 64)[slot] = float("inf")
    out = b.run()
    assert torch.equal(out[1:].view(torch.int16), good[1:].view(torch.int16))


@BOTH
def test_streams_and_graphs(fp8):
    """Two calls on two streams at once, each with its workspace, and captured
    calls that share one workspace replayed in turn."""
    a = Batch(15, [900, 70], [1, 70], 8, 2, 128, 100, 4, fp8=fp8)
    b = Batch(16, [3000] * 20, [1] * 20, 8, 2, 128, 700, 4, fp8=fp8)
    want = a.run().clone(), b.run().clone()
    side = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in side:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        got = [x.run(stream=s) for x, s in zip((a, b), (side[0], side[1].cuda_stream))]
    for s in side:
        s.synchronize()
    for g, w in zip(got, want):
        assert torch.equal(g.view(torch.int16), w.view(torch.int16))
    size = max(ops.workspace_size(2, 71, 8, 2, 128, 70, 900),
               ops.workspace_size(20, 20, 8, 2, 128, 1, 3000))
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    outs, graphs = [], []
    for x in (a, b):
        out = torch.zeros_like(x.q)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            x.run(out=out, workspace=ws)
        outs.append(out)
        graphs.append(g)
    for _ in range(3):
        for o in outs:
            o.zero_()
        for g in graphs + graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o.view(torch.int16), w.view(torch.int16))
    ops.check_device_errors()


def test_refusals():
    b = Batch(17, [40, 30], [1, 5], 4, 2, 64, 20, 0)
    for bad in (dict(max_seq_len=1000), dict(max_q_len=50, max_seq_len=40), dict(min_q_len=9)):
        with pytest.raises(ops.PagedAttnError):
            b.run(**bad)
    for window, sinks in ((0, 0), (-1, 0), (5, -1)):
        b.window, b.sinks = window, sinks
        with pytest.raises(ops.PagedAttnError):
            b.run()
    b.window, b.sinks = 20, 0
    with pytest.raises(ValueError):
        b.run(out=b.q[:3].contiguous())
    with pytest.raises(ValueError):
        b.run(workspace=torch.empty(1 << 20, dtype=torch.uint8))
    keep = b.dt
    b.dt = keep[:1]
    with pytest.raises(ValueError):
        b.run()
    b.dt = keep.long()
    with pytest.raises(TypeError):
        b.run()


@BOTH
def test_either_way_into_the_library(fp8):
    """The extension module's calls and the binding's own checks (taken for a
    given stream, other number types, a workspace to allocate, a tensor
    subclass) give the same bits."""
    b = Batch(18, [300, 90, 513], [1, 40, 70], 8, 2, 64, 75, 5, fp8=fp8)
    ws = ops.alloc_workspace(3, 111, 8, 2, 64, 70, 513)
    want = b.run(workspace=ws)
    here = torch.cuda.current_stream()
    for kw in (dict(workspace=ws, stream=here), dict(), dict(workspace=ws, max_q_len=np.int64(70)),
               dict(workspace=torch.nn.Parameter(ws, requires_grad=False))):
        assert torch.equal(b.run(**kw).view(torch.int16), want.view(torch.int16))
    assert b.run(workspace=ws, out=want) is want
    ops.check_device_errors()


@pytest.mark.parametrize("form", ["single tiles", "pairs of tiles", "no window"])
@pytest.mark.parametrize("top", [2.4e-4, 1e-3, 1e-2, 4e4, "mixed"])
def test_row_maxima_of_the_8_bit_cache(top, form):
    """Decode rows and chunk rows of one call over cached rows whose maxima lie far
    from 1, or at 1.2e-4 to 1 within one page."""
    window, sinks = (9000, 0) if form == "no window" else (6, 1)
    if form == "pairs of tiles":
        lens, q_lens, heads = [513, 90, 2, 1100, 60], [513, 1, 2, 400, 40], (32, 8, 128)
    else:
        lens, q_lens, heads = [90, 60, 200], [1, 40, 70], (8, 2, 64)
    d = heads[2]
    rng = np.random.default_rng(31)
    b = Batch(30, lens, q_lens, *heads, window, sinks, fp8=True)
    for cache, rows in ((b.kc, b.K), (b.vc, b.V)):
        scales = ops.fp8_cache_views(cache, heads[1], d)[1]
        old = scales.cpu().numpy()
        if top == "mixed":
            new = np.exp2(rng.uniform(math.log2(1.2e-4), 0, old.shape))
        else:  # keys past 1 would make scores that nothing but their largest is seen of
            new = (min(top, 1.0) if cache is b.kc else top) * rng.uniform(0.5, 1, old.shape)
        new = np.where(np.isnan(old), old, new / 448).astype(np.float32)
        scales.copy_(torch.from_numpy(new).cuda())
        rows *= (new.astype(np.float64) / old).reshape(rows.shape[0], heads[1])[..., None]
    b.scale = 1.0 / (math.sqrt(d) * (min(top, 1.0) if top != "mixed" else 1.0))
    got = b.run().cpu().double().numpy()
    ops.check_device_errors()
    out, A, S = b.reference()
    assert np.isfinite(got).all()
    # beside the relative errors: a key or value below f16's normal range is right
    # to 2^-25, which a score takes once for each |q_i|; and a decode row's weight
    # times value scale times 2^9 is, which each key's code, at most 448, takes
    one = np.repeat(np.array(q_lens) == 1, q_lens)[:, None, None]
    keys = max(lens) if form == "no window" else window + sinks
    e = 2.0 ** -25 * b.scale * np.abs(b.q64).sum(-1, keepdims=True)
    tol = R.window_tolerance(out, A, S, True) + e * (A + np.abs(out)) + 1.01 * 2.0 ** -25 \
        + one * keys * 2.0 ** -25 * 448 / 512
    assert (np.abs(got - out) <= tol).all(), float((np.abs(got - out) / tol).max())


@BOTH
@pytest.mark.parametrize("q_lens", [[1] * 150 + [700] + [1] * 50, [4] * 256],
                         ids=["a chunk in pairs of tiles beside decodes", "short requests"])
def test_decodes_and_short_requests_beside_query_tiles(q_lens, fp8):
    lens = [n + (37 * i) % 200 for i, n in enumerate(q_lens)]
    Batch(32, lens, q_lens, 32, 8, 128, 90, 4, fp8=fp8).check()
