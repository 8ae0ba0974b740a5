"""Bounds of blocks, the choice of blocks and the attention over chosen blocks on the
GPU, against the plain definitions in 64 bits."""
import numpy as np
import pytest
import torch

import long_reference as R
from paged_kv_cache_174_gb300 import ops

pytestmark = pytest.mark.gpu

REQUESTS = [(0, 1), (15, 1), (16, 1), (0, 0), (31, 3), (70, 1), (0, 37), (200, 17), (47, 1)]


def run_bounds(c, starts=True, fill=77):
    bt, sl, qsl = c.step()
    codes = torch.full((c.blocks, c.n_kv, 2, c.d), fill, dtype=torch.int8, device="cuda")
    scales = torch.full((c.blocks, c.n_kv), -3.0, device="cuda")
    call = ops.summarize_blocks_fp8 if c.fp8 else ops.summarize_blocks
    before = codes.cpu().double().numpy(), scales.cpu().double().numpy()
    call(c.k, bt, sl, qsl if starts else None, codes, scales, num_tokens=c.tokens)
    ops.check_device_errors()
    want = R.bounds(*before, c.K, c.tables, c.lens, c.starts if starts else None, c.block)
    return codes, scales, want


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_kv,d,block", [(1, 64, 16), (8, 128, 16), (2, 128, 32), (4, 64, 32)])
@pytest.mark.parametrize("starts", [True, False])
def test_bounds(n_kv, d, block, fp8, starts):
    c = R.Cache(REQUESTS, n_kv, d, block, fp8, seed=n_kv + d)
    codes, scales, (want_c, want_s) = run_bounds(c, starts)
    assert np.array_equal(codes.cpu().double().numpy(), want_c)
    assert np.array_equal(scales.cpu().double().numpy(), want_s)


def test_bounds_of_values_at_the_borders():
    c = R.Cache([(0, 16), (0, 9), (0, 16), (0, 5), (0, 16)], 1, 64, 16, False, seed=3)
    rows = [c.tables[s][0] * 16 for s in range(5)]
    c.K[rows[0]:rows[0] + 16] = 0                       # all zero
    c.K[rows[1]:rows[1] + 9] = 1e-39                    # below the smallest scale
    c.K[rows[2] + 3, 0, 5] = np.nan                     # counts as 0
    c.K[rows[2]:rows[2] + 16, 0, 7] = np.nan            # nothing but NaN in a channel
    c.K[rows[3], 0, :3] = [np.inf, -np.inf, 127.0]
    c.K[rows[4]:rows[4] + 16] = -127.0
    c.K[rows[4], 0, 0] = 127.5
    c.k = torch.from_numpy(c.K).bfloat16().view(c.k.shape).cuda()
    c.K = c.k.cpu().double().view(-1, 1, 64).numpy()
    codes, scales, (want_c, want_s) = run_bounds(c)
    assert np.array_equal(codes.cpu().double().numpy(), want_c)
    assert np.array_equal(scales.cpu().double().numpy(), want_s)


def test_bounds_with_more_places_than_a_warp_of_requests():
    c = R.Cache([(5 * s % 50, s % 3) for s in range(100)], 2, 64, 16, False, seed=4, pad=3)
    codes, scales, (want_c, want_s) = run_bounds(c)
    assert np.array_equal(codes.cpu().double().numpy(), want_c)
    assert np.array_equal(scales.cpu().double().numpy(), want_s)


def run_choice(c, n_q, n_sel, sinks, recent, codes=None, scales=None, q=None, seed=0):
    bt, sl, qsl = c.step()
    if codes is None:
        codes, scales, _ = run_bounds(c, starts=False)
    qd, q64 = c.queries(n_q, seed) if q is None else (q, q.cpu().double().numpy())
    out = torch.full((c.tokens, c.n_kv, n_sel), -9, dtype=torch.int32, device="cuda")
    got = ops.select_blocks(qd, codes, scales, bt, sl, qsl, num_selected=n_sel, num_sinks=sinks,
                            num_recent=recent, block_size=c.block,
                            max_seq_len=max(c.lens + [0]), out=out)
    ops.check_device_errors()
    assert got is out
    want = R.choose(q64, codes.cpu().double().numpy(), scales.cpu().double().numpy(), c.tables,
                    c.lens, c.starts, c.block, n_sel, sinks, recent,
                    np.full(out.shape, -9, np.int64))
    return got, want


@pytest.mark.parametrize("n_kv,G,d,block", [(1, 1, 64, 16), (2, 2, 128, 16), (4, 4, 64, 32),
                                            (8, 4, 128, 16), (1, 8, 128, 32), (2, 8, 64, 16),
                                            (8, 1, 128, 16), (2, 4, 128, 16), (1, 2, 64, 16)])
@pytest.mark.parametrize("n_sel,sinks,recent", [(4, 1, 1), (3, 0, 3), (9, 2, 2), (1, 0, 1)])
def test_choice(n_kv, G, d, block, n_sel, sinks, recent):
    c = R.Cache(REQUESTS + [(700, 2)], n_kv, d, block, False, seed=G, pad=2)
    got, want = run_choice(c, n_kv * G, n_sel, sinks, recent)
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("n_kv,G,d", [(1, 4, 128), (2, 1, 64), (8, 8, 128)])
def test_choice_over_a_cluster(n_kv, G, d):
    """A few long contexts: several CTAs share a (token, kv head)'s blocks."""
    lens = [(40_000, 1), (21_503, 2), (300, 1)]
    blocks = sum(-(-(a + b) // 16) for a, b in lens) + 2
    rng = np.random.default_rng(G)
    c = R.Cache([(0, 0)], n_kv, d, 16, False, seed=0)
    c.lens = [a + b for a, b in lens]
    c.starts = np.array([0, 1, 3, 4])
    c.tokens, c.blocks = 4, blocks
    ids = rng.permutation(blocks)
    c.tables = np.full((3, 2501), -1, np.int32)
    at = 0
    for s, n in enumerate(c.lens):
        m = -(-n // 16)
        c.tables[s, :m] = ids[at:at + m]
        at += m
    codes = torch.from_numpy(rng.integers(-127, 128, (blocks, n_kv, 2, d))).to(torch.int8).cuda()
    scales = torch.from_numpy(2.0 ** rng.integers(-4, 1, (blocks, n_kv))).float().cuda()
    for n_sel in (100, 1500):
        got, want = run_choice(c, n_kv * G, n_sel, 2, 3, codes, scales)
        assert np.array_equal(got.cpu().numpy(), want)


def test_ties_go_to_the_lowest_block():
    c = R.Cache([(160 * 16, 1), (900, 1)], 2, 64, 16, False, seed=0)
    codes = torch.full((c.blocks, 2, 2, 64), 5, dtype=torch.int8, device="cuda")
    scales = torch.ones(c.blocks, 2, device="cuda")
    codes[c.tables[0][70], 0] = 6  # one block above the tie, one head
    q = torch.ones(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    got, want = run_choice(c, 4, 20, 1, 1, codes, scales, q)
    assert np.array_equal(got.cpu().numpy(), want)
    assert got[0, 1].tolist() == list(range(19)) + [160]
    assert got[0, 0].tolist() == list(range(18)) + [70, 160]
    # a query of zeros, and of one huge element: ties everywhere, scores near fp32's end
    q[0] = 0
    q[1, :, 3] = -3e38
    got, want = run_choice(c, 4, 20, 0, 2, codes, scales, q)
    assert np.array_equal(got.cpu().numpy(), want)


def run_blocks(c, n_q, selected, scale, seed=0, q=None):
    bt, sl, qsl = c.step()
    qd, q64 = c.queries(n_q, seed) if q is None else (q, q.cpu().double().numpy())
    call = ops.paged_attention_blocks_fp8 if c.fp8 else ops.paged_attention_blocks
    out = torch.full(qd.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    sel = torch.from_numpy(np.ascontiguousarray(selected, np.int32)).cuda()
    assert call(qd, c.k, c.v, bt, sl, qsl, scale, sel, out=out) is out
    ref = R.blocks_attention(q64, c.K, c.V, c.tables, c.lens, c.starts, scale, c.block, selected)
    return out.double().cpu().numpy(), ref


def random_choice(c, n, seed, order=True):
    rng = np.random.default_rng(seed)
    sel = np.full((c.tokens, c.n_kv, n), -1, np.int64)
    for t, s, p in R.token_rows(c.lens, c.starts):
        for h in range(c.n_kv):
            some = rng.permutation(p // c.block + 1)[:n]
            sel[t, h, :len(some)] = np.sort(some) if order else some
    return sel


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_kv,G,d,block", [(1, 1, 64, 16), (2, 2, 128, 16), (4, 4, 64, 32),
                                            (8, 4, 128, 16), (1, 8, 128, 32), (2, 8, 64, 16)])
def test_attention_over_chosen_blocks(n_kv, G, d, block, fp8):
    c = R.Cache(REQUESTS + [(700, 2)], n_kv, d, block, fp8, seed=G + d, pad=2)
    for n, order in ((1, True), (5, False), (40, True)):
        got, ref = run_blocks(c, n_kv * G, random_choice(c, n, n, order), 1 / d ** 0.5)
        R.assert_blocks_close(got, ref, f"{n} blocks")
        assert (got[np.isnan(ref[0])] == 7.0).all()  # rows of no request
    ops.check_device_errors()


@pytest.mark.parametrize("fp8", [False, True])
def test_long_lists_over_a_cluster(fp8):
    c = R.Cache([(9000, 1), (3000, 3)], 1, 128, 16, fp8, seed=5)
    for n in (33, 150, 600):
        got, ref = run_blocks(c, 4, random_choice(c, n, n), 0.09)
        R.assert_blocks_close(got, ref, f"{n} blocks")
    ops.check_device_errors()


@pytest.mark.parametrize("fp8", [False, True])
def test_lists_with_gaps_repeats_and_nothing(fp8):
    c = R.Cache([(100, 1), (200, 2), (15, 1)], 2, 64, 16, fp8, seed=6)
    sel = np.full((4, 2, 6), -1, np.int64)
    sel[0, 0] = [-1, 3, -5, 3, 0, -1]    # gaps, and a block twice
    sel[1, 0] = [12, -1, -1, -1, -1, 7]  # its own block (partly ahead of it) and another
    sel[1, 1, 2] = 12
    sel[2, 0, 0] = 0
    sel[3, 1, 5] = 0                     # (the other lists hold nothing: rows of zeros)
    got, ref = run_blocks(c, 8, sel, 0.125)
    R.assert_blocks_close(got, ref)
    assert (got[0, 4:] == 0).all() and (got[3, :4] == 0).all() and (got[2, 4:] == 0).all()
    ops.check_device_errors()


def test_large_scores_and_other_scales():
    c = R.Cache([(300, 1), (90, 1)], 2, 128, 16, False, seed=7, spread=6.0)
    sel = random_choice(c, 9, 1)
    q, _ = c.queries(8, 2, spread=8.0)
    for scale in (1.0, -1.0, 0.0, 1e-3):  # at 1, scores past +-1000
        got, ref = run_blocks(c, 8, sel, scale, q=q)
        R.assert_blocks_close(got, ref, f"scale {scale}")
    q *= 1e-30
    got, ref = run_blocks(c, 8, sel, 1.0, q=q)
    R.assert_blocks_close(got, ref, "tiny q")
    c8 = R.Cache([(300, 1), (90, 1)], 2, 128, 16, True, seed=7)
    for factor in (1e-30, 1e30):
        q8, _ = c8.queries(8, 2)
        q8 *= factor
        got, ref = run_blocks(c8, 8, sel, 0.1 / factor, q=q8)
        R.assert_blocks_close(got, ref, f"8-bit, q times {factor}")
    ops.check_device_errors()


def test_entries_out_of_range_are_flagged_and_passed_over():
    c = R.Cache([(100, 1)], 1, 64, 16, False, seed=8)
    sel = np.full((1, 1, 4), -1, np.int64)
    sel[0, 0] = [2, 7, 5, -1]  # block 7 lies past the token's own
    bt, sl, qsl = c.step()
    q, q64 = c.queries(2, 0)
    out = ops.paged_attention_blocks(q, c.k, c.v, bt, sl, qsl, 0.1,
                                     torch.from_numpy(sel).int().cuda())
    with pytest.raises(ops.PagedAttnError, match="out of range"):
        ops.check_device_errors()
    sel[0, 0, 1] = -1
    R.assert_blocks_close(out.double().cpu().numpy(), R.blocks_attention(
        q64, c.K, c.V, c.tables, c.lens, c.starts, 0.1, 16, sel))
    bt[0, 5] = c.blocks  # a table entry past the pool
    out = ops.paged_attention_blocks(q, c.k, c.v, bt, sl, qsl, 0.1,
                                     torch.from_numpy(sel).int().cuda())
    with pytest.raises(ops.PagedAttnError, match="out of range"):
        ops.check_device_errors()
    sel[0, 0, 2] = -1
    R.assert_blocks_close(out.double().cpu().numpy(), R.blocks_attention(
        q64, c.K, c.V, c.tables, c.lens, c.starts, 0.1, 16, sel))


def test_lengths_out_of_range_are_flagged():
    c = R.Cache([(40, 1), (20, 1)], 1, 64, 16, False, seed=9)
    bt, sl, qsl = c.step()
    codes, scales = ops.alloc_bounds(c.blocks, 1, 64)
    q, _ = c.queries(1, 0)
    bad = sl.clone()
    bad[0] = 10 ** 6
    calls = [lambda: ops.summarize_blocks(c.k, bt, bad, qsl, codes, scales, num_tokens=2),
             lambda: ops.summarize_blocks(c.k, bt, bad, None, codes, scales),
             lambda: ops.select_blocks(q, codes, scales, bt, bad, qsl, num_selected=2,
                                       block_size=16, max_seq_len=64),
             lambda: ops.paged_attention_blocks(q, c.k, c.v, bt, bad, qsl, 0.1, torch.zeros(
                 2, 1, 1, dtype=torch.int32, device="cuda"))]
    for call in calls:
        call()
        with pytest.raises(ops.PagedAttnError, match="out of range"):
            ops.check_device_errors()


def test_both_ways_into_the_library_agree():
    """The extension module and, on another stream, ctypes."""
    c = R.Cache(REQUESTS, 2, 64, 16, False, seed=10)
    bt, sl, qsl = c.step()
    q, _ = c.queries(8, 0)
    codes, scales = ops.alloc_bounds(c.blocks, 2, 64)
    codes2, scales2 = ops.alloc_bounds(c.blocks, 2, 64)
    other = torch.cuda.Stream()
    other.wait_stream(torch.cuda.current_stream())
    most = max(c.lens)
    res = []
    for stream, (b, s) in ((None, (codes, scales)), (other, (codes2, scales2))):
        ops.summarize_blocks(c.k, bt, sl, qsl, b, s, num_tokens=c.tokens, stream=stream)
        sel = ops.select_blocks(q, b, s, bt, sl, qsl, num_selected=3, block_size=16,
                                max_seq_len=most, stream=stream)
        res.append((sel, ops.paged_attention_blocks(q, c.k, c.v, bt, sl, qsl, 0.1, sel,
                                                    stream=stream)))
    torch.cuda.synchronize()
    assert torch.equal(codes, codes2) and torch.equal(scales, scales2)
    assert torch.equal(res[0][0], res[1][0]) and torch.equal(res[0][1], res[1][1])
    with pytest.raises(ValueError, match="num_selected"):
        ops.select_blocks(q, codes, scales, bt, sl, qsl, num_selected=0, block_size=16,
                          max_seq_len=most)
    with pytest.raises(ValueError, match="selected"):
        ops.paged_attention_blocks(q[:-1], c.k, c.v, bt, sl, qsl, 0.1, res[0][0])
    with pytest.raises(ValueError, match="blocks"):
        ops.summarize_blocks(c.k[:-1].contiguous(), bt, sl, qsl, codes, scales, num_tokens=3)
