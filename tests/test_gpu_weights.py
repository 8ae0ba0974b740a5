"""Attention with accumulated weights on the GPU, against its plain definition in 64 bits."""
import numpy as np
import pytest
import torch

import long_reference as R
import step_reference as S
from paged_kv_cache_174_gb300 import ops

pytestmark = pytest.mark.gpu

DECODES = [(0, 1), (15, 1), (16, 1), (0, 0), (70, 1), (199, 1), (1000, 1), (47, 1)]


def run(c, n_q, scale, seed=0, q=None, old=None, min_q_len=0, workspace=True):
    bt, sl, qsl = c.step()
    qd, q64 = c.queries(n_q, seed) if q is None else (q, q.cpu().double().numpy())
    new = np.diff(c.starts)
    length = max(c.lens) + 5
    g = torch.Generator().manual_seed(seed)
    w = torch.rand(len(c.lens), c.n_kv, length, generator=g) if old is None else old.cpu()
    for s, n in enumerate(c.lens):  # new tokens' entries hold anything before the call
        w[s, :, n - int(new[s]):n] = float("nan")
    wd = w.cuda()
    out = torch.full(qd.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    call = ops.paged_attention_weights_fp8 if c.fp8 else ops.paged_attention_weights
    assert call(qd, c.k, c.v, bt, sl, qsl, scale, wd, max_q_len=int(new.max()),
                max_seq_len=max(c.lens), min_q_len=min_q_len, out=out) is out
    ops.check_device_errors()
    ref = R.weights_attention(q64, c.K, c.V, c.tables, c.lens, c.starts, scale, c.block,
                              w.numpy())
    return out, wd, w, ref


def check(c, got, what=""):
    out, wd, before, (o64, A, E, w64, tol) = got
    new = np.diff(c.starts)
    w = wd.double().cpu().numpy()
    for s, n in enumerate(c.lens):
        if new[s] == 0:
            assert torch.equal(wd[s].cpu(), before[s]), what  # left as they were
            continue
        off = np.abs(w[s, :, :n] - w64[s, :, :n])
        assert np.isfinite(w[s, :, :n]).all(), what
        assert (off <= tol[s, :, :n] + 1e-30).all(), \
            f"{what}: request {s} (length {n}): {(off / (tol[s, :, :n] + 1e-30)).max():.2f} times"
        assert torch.equal(wd[s, :, n:].cpu(), before[s, :, n:]), what
    o = out.double().cpu().numpy()
    rows = ~np.isnan(o64[:, 0, 0])
    assert (o[~rows] == 7.0).all(), what
    chunk = np.zeros(c.tokens, bool)
    for s in range(len(c.lens)):
        if new[s] > 1:
            chunk[c.starts[s]:c.starts[s + 1]] = True
    one = rows & ~chunk
    R.assert_blocks_close(o[one], (o64[one], A[one], E[one]), what)
    if chunk.any():  # the prefill kernel's outputs, to its tolerance
        size = E[chunk] / (4 * c.d * R.EPS)  # (an upper bound of the scores' terms)
        S.assert_window_close(o[chunk], (o64[chunk], A[chunk], size), c.fp8, what)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_kv,G,d,block", [(1, 1, 64, 16), (2, 2, 128, 16), (4, 4, 64, 32),
                                            (8, 4, 128, 16), (1, 8, 128, 32), (2, 8, 64, 16)])
def test_decode(n_kv, G, d, block, fp8):
    c = R.Cache(DECODES, n_kv, d, block, fp8, seed=G + d, pad=3)
    check(c, run(c, n_kv * G, 1 / d ** 0.5), "decode")


@pytest.mark.parametrize("n_kv,G,d,fp8", [(1, 8, 64, False), (1, 4, 128, True),
                                          (2, 8, 128, False)])
def test_long_decode_beyond_the_kept_scores(n_kv, G, d, fp8):
    """Contexts whose scores do not fit in shared memory: the rest are computed again."""
    c = R.Cache([(40_000, 1), (5, 1)], n_kv, d, 16, fp8, seed=1)
    check(c, run(c, n_kv * G, 1 / d ** 0.5), "long decode")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_kv,G,d,block", [(1, 1, 64, 16), (2, 2, 128, 16), (4, 4, 64, 32),
                                            (8, 4, 128, 16), (1, 8, 128, 32), (2, 8, 64, 16)])
def test_chunks(n_kv, G, d, block, fp8):
    c = R.Cache([(0, 2), (100, 37), (0, 130), (515, 64), (0, 0), (129, 300)], n_kv, d, block, fp8,
                seed=G + d, pad=1)
    check(c, run(c, n_kv * G, 1 / d ** 0.5), "chunks")
    c = R.Cache([(0, 257)], n_kv, d, block, fp8, seed=G)
    check(c, run(c, n_kv * G, 1 / d ** 0.5, min_q_len=2), "a prompt")


@pytest.mark.parametrize("fp8", [False, True])
def test_mixed_step(fp8):
    c = R.Cache(DECODES + [(700, 129), (33, 2)] + DECODES, 2, 128, 16, fp8, seed=2, pad=2)
    check(c, run(c, 8, 0.088), "mixed")


@pytest.mark.parametrize("fp8", [False, True])
def test_few_rows_over_a_long_context(fp8):
    """The keys of a row cut into pieces."""
    c = R.Cache([(6000, 3), (2500, 17)], 1, 128, 16, fp8, seed=3)
    check(c, run(c, 4, 0.088), "pieces")


@pytest.mark.parametrize("fp8", [False, True])
def test_many_query_tiles(fp8):
    """Query tiles of a key tile shared by a cluster, units in several rounds."""
    c = R.Cache([(0, 1500), (1000, 700)], 4, 64, 16, fp8, seed=4)
    check(c, run(c, 32, 0.125), "tiles")


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("requests,n_kv,G,d", [
    ([(0, 1500)], 1, 8, 64),              # clusters of four take a key tile's query tiles
    ([(1100, 1000)], 2, 2, 128),          # of four, a row's keys, and a key tile's query tiles
    ([(1100 + s, 2) for s in range(60)], 2, 4, 64),   # ... in several rounds
    ([(1100 + 9 * s, 2 + s % 3) for s in range(45)] + [(30, 1)], 4, 1, 128),
])
def test_clusters(requests, n_kv, G, d, fp8):
    c = R.Cache(requests, n_kv, d, 16, fp8, seed=8)
    check(c, run(c, n_kv * G, 1 / d ** 0.5), "clusters")


def test_more_chunk_requests_than_a_launch_lists():
    c = R.Cache([(s % 5, 2 + s % 2) for s in range(1100)], 1, 64, 16, False, seed=5)
    check(c, run(c, 1, 0.125), "many requests")


def test_weights_add_up_over_steps():
    """Row sums: each step spreads n_q / n_kv per kv head and row."""
    c = R.Cache([(64, 1), (0, 40)], 2, 64, 16, False, seed=6)
    out, w, _, _ = run(c, 4, 0.125, old=torch.zeros(2, 2, 70))
    assert torch.allclose(w[0].sum(-1).cpu(), torch.full((2,), 2.0), rtol=1e-5)
    assert torch.allclose(w[1].sum(-1).cpu(), torch.full((2,), 80.0), rtol=1e-5)


def test_large_scores_and_other_scales():
    c = R.Cache([(300, 1), (90, 50)], 2, 128, 16, False, seed=7, spread=3.0)
    q, _ = c.queries(8, 2, spread=4.0)
    for scale in (1.0, -0.5, 0.0, 1e-3):
        check(c, run(c, 8, scale, q=q), f"scale {scale}")


def test_the_same_call_gives_the_same_bits():
    c = R.Cache(DECODES + [(700, 129)], 2, 128, 16, False, seed=8)
    a, b = run(c, 8, 0.088), run(c, 8, 0.088)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1].isnan(), b[1].isnan())
    assert torch.equal(a[1].nan_to_num(), b[1].nan_to_num())


def test_requests_beyond_the_bounds_are_flagged():
    c = R.Cache([(30, 1), (20, 3)], 1, 64, 16, False, seed=9)
    bt, sl, qsl = c.step()
    q, _ = c.queries(1, 0)
    w = torch.zeros(2, 1, 64, device="cuda")
    for maxq, maxl, minq in ((1, 40, 0), (3, 25, 0), (3, 40, 2)):
        ops.paged_attention_weights(q, c.k, c.v, bt, sl, qsl, 0.1, w, max_q_len=maxq,
                                    max_seq_len=maxl, min_q_len=minq)
        with pytest.raises(ops.PagedAttnError, match="out of range"):
            ops.check_device_errors()


def test_workspace_and_shapes():
    c = R.Cache([(30, 1), (20, 3)], 1, 64, 16, False, seed=10)
    bt, sl, qsl = c.step()
    q, _ = c.queries(1, 0)
    w = torch.zeros(2, 1, 64, device="cuda")
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    kw = dict(max_q_len=3, max_seq_len=40)
    with pytest.raises(ops.PagedAttnError, match="WORKSPACE"):
        ops.paged_attention_weights(q, c.k, c.v, bt, sl, qsl, 0.1, w, workspace=small, **kw)
    with pytest.raises(ops.PagedAttnError, match="weights_len"):
        ops.paged_attention_weights(q, c.k, c.v, bt, sl, qsl, 0.1, w[:, :, :39].contiguous(), **kw)
    with pytest.raises(ValueError, match="weights"):
        ops.paged_attention_weights(q, c.k, c.v, bt, sl, qsl, 0.1, w[:1], **kw)
    with pytest.raises(ValueError, match="contiguous"):
        ops.paged_attention_weights(q, c.k, c.v, bt, sl, qsl, 0.1, w[:, :, :50], **kw)
    # one buffer for every call within its sizes
    big = ops.alloc_weights_workspace(4, 4096, 32, 8, 128, 4096, 8192).numel()
    for T in (1, 7, 300, 4096):
        assert ops.alloc_weights_workspace(4, T, 32, 8, 128, min(T, 100), 8000).numel() <= big
