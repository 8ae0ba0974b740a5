"""Eviction by accumulated weight on the GPU, against its plain definition: what is
kept and moved is equal bit for bit."""
import numpy as np
import pytest
import torch

import long_reference as R
from paged_kv_cache_174_gb300 import ops

pytestmark = pytest.mark.gpu


def bits(w):
    return w.view(torch.int32).cpu().numpy()


def run(c, w, budgets, sinks, recent, in_place=False, offsets=True, pushed=2):
    bt, sl, _ = c.step()
    i32 = torch.int32
    free = torch.full((c.blocks,), -1, dtype=i32, device="cuda")
    free[:pushed] = torch.from_numpy(c.spare[:pushed]).int()
    count = torch.tensor([pushed], dtype=i32, device="cuda")
    off = torch.arange(len(c.lens), dtype=i32, device="cuda") if offsets else None
    b = torch.tensor(budgets, dtype=i32, device="cuda")
    wd = w.clone().cuda()
    before = c.parts()
    w64 = w.clone().numpy()
    lens, free64, n, gone = R.evict(before, w64, c.tables, c.lens, budgets,
                                    free.tolist(), pushed, sinks, recent, c.block)
    call = ops.evict_tokens_fp8 if c.fp8 else ops.evict_tokens
    lens_out = None if in_place else torch.full_like(sl, -7)
    count_out = None if in_place else torch.full_like(count, -7)
    got = call(c.k, c.v, wd, bt, sl, b, free, count, num_sinks=sinks, num_recent=recent,
               max_seq_len=max(c.lens), seq_lens_out=lens_out, free_count_out=count_out,
               position_offsets=off)
    assert got is (sl if in_place else lens_out)
    assert got.tolist() == lens
    assert (count if in_place else count_out).tolist() == [n]
    if not in_place:
        assert sl.tolist() == c.lens and count.tolist() == [pushed]
    assert free.tolist() == free64
    if offsets:
        assert (off.cpu() - torch.arange(len(lens))).tolist() == gone
    assert np.array_equal(bits(wd), w64.view(np.int32))
    for x, y in zip(c.parts(), before):
        assert np.array_equal(x, y)
    assert np.array_equal(bt.cpu().numpy(), c.tables)


def random_weights(c, seed, extra=3):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(len(c.lens), c.n_kv, max(c.lens) + extra, generator=g) * 2).exp()


LENS = [1, 40, 41, 47, 48, 49, 64, 200, 333, 0, 1500]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("n_kv,d,block", [(1, 64, 16), (8, 128, 16), (2, 128, 32), (4, 64, 32),
                                          (2, 64, 16)])
@pytest.mark.parametrize("sinks,recent", [(0, 0), (4, 17), (1, 39)])
def test_evict(n_kv, d, block, fp8, sinks, recent):
    c = R.Cache([(n, 0) for n in LENS], n_kv, d, block, fp8, seed=n_kv)
    run(c, random_weights(c, 1), [40] * len(LENS), sinks, recent)
    ops.check_device_errors()


@pytest.mark.parametrize("fp8", [False, True])
def test_budgets_of_each_request(fp8):
    c = R.Cache([(300, 0)] * 5, 2, 128, 16, fp8, seed=2)
    run(c, random_weights(c, 2), [12, 299, 300, 10 ** 9, 160], 5, 7, in_place=True)
    ops.check_device_errors()


@pytest.mark.parametrize("requests", [1, 9, 40])
@pytest.mark.parametrize("fp8", [False, True])
def test_ranges_of_rows(requests, fp8):
    """Few (request, kv head) pairs: a row's bytes are moved by several CTAs."""
    c = R.Cache([(700 - s, 0) for s in range(requests)], 8, 128, 16, fp8, seed=3)
    run(c, random_weights(c, 3), [333] * requests, 3, 50)
    ops.check_device_errors()


def test_ties_and_special_weights():
    c = R.Cache([(200, 0)] * 4, 2, 64, 16, False, seed=4)
    w = torch.ones(4, 2, 203)
    w[1] = torch.randint(0, 4, (2, 203)).float()
    w[2, 0, 10:60] = float("nan")
    w[2, 1, 60:90] = float("inf")
    w[2, 1, 100:150] = -float("inf")
    w[3] = -torch.rand(2, 203)
    w[3, 0, ::2], w[3, 0, 1::2] = 0.0, -0.0   # equal weights
    run(c, w, [90, 90, 90, 90], 2, 20)
    c = R.Cache([(200, 0)] * 4, 2, 64, 16, False, seed=4)
    run(c, w, [22, 23, 30, 199], 2, 20)       # nothing, and one, to choose
    ops.check_device_errors()


@pytest.mark.parametrize("fp8", [False, True])
def test_long_requests(fp8):
    """Weights that are read from memory in each pass, and those that are held."""
    c = R.Cache([(30_000, 0), (9_000, 0)], 1, 64, 16, fp8, seed=5)
    run(c, random_weights(c, 5), [4_000, 8_999], 16, 512)
    c = R.Cache([(9_000, 0), (1_000, 0)], 1, 64, 16, fp8, seed=5)
    run(c, random_weights(c, 5), [4_000, 512], 16, 496)
    ops.check_device_errors()


def test_more_requests_than_a_block_of_threads():
    c = R.Cache([(20 + s % 30, 0) for s in range(600)], 1, 64, 16, False, seed=6)
    for in_place in (False, True):
        run(c, random_weights(c, 6), [25] * 600, 1, 2, in_place=in_place)
        c = R.Cache([(20 + s % 30, 0) for s in range(600)], 1, 64, 16, False, seed=6)
    ops.check_device_errors()


def test_nothing_to_evict():
    c = R.Cache([(50, 0), (3, 0)], 1, 64, 16, False, seed=7)
    run(c, random_weights(c, 7), [50, 50], 0, 0, in_place=True)
    ops.check_device_errors()


def call_with(c, w, budgets=(30, 30), lens=None, tables=None, count=1, **kw):
    bt, sl, _ = c.step()
    i32 = torch.int32
    free = torch.full((c.blocks,), -1, dtype=i32, device="cuda")
    count = torch.tensor([count], dtype=i32, device="cuda")
    sl = sl if lens is None else torch.tensor(lens, dtype=i32, device="cuda")
    bt = bt if tables is None else torch.from_numpy(tables).cuda()
    out = ops.evict_tokens(c.k, c.v, w, bt, sl, torch.tensor(budgets, dtype=i32, device="cuda"),
                           free, count, max_seq_len=kw.pop("max_seq_len", max(c.lens)), **kw)
    return out, free, count


def test_what_is_out_of_range_is_flagged():
    c = R.Cache([(100, 0), (90, 0)], 1, 64, 16, False, seed=8)
    w = random_weights(c, 8).cuda()
    flagged = lambda: pytest.raises(ops.PagedAttnError, match="out of range")  # noqa: E731
    # a budget below what has to stay: its request is left alone
    out, _, _ = call_with(c, w, (5, 30), num_sinks=4, num_recent=4)
    with flagged():
        ops.check_device_errors()
    assert out.tolist() == [100, 30]
    c = R.Cache([(100, 0), (90, 0)], 1, 64, 16, False, seed=8)
    out, _, _ = call_with(c, w, lens=[10 ** 6, 90])
    with flagged():
        ops.check_device_errors()
    assert out.tolist() == [10 ** 6, 30]
    # a free list without room, and a count out of range
    c = R.Cache([(100, 0), (90, 0)], 1, 64, 16, False, seed=8)
    _, free, count = call_with(c, w, count=c.blocks - 2)
    with flagged():
        ops.check_device_errors()
    assert count.tolist() == [c.blocks]
    c = R.Cache([(100, 0), (90, 0)], 1, 64, 16, False, seed=8)
    _, free, count = call_with(c, w, count=-4)
    with flagged():
        ops.check_device_errors()
    assert count.tolist() == [-4] and (free == -1).all()
    # a table entry that names no block: rows of other blocks still move
    c = R.Cache([(100, 0), (90, 0)], 1, 64, 16, False, seed=8)
    tables = c.tables.copy()
    tables[0, 5] = c.blocks + 3
    call_with(c, w, tables=tables)
    with flagged():
        ops.check_device_errors()


def test_refusals():
    c = R.Cache([(100, 0), (90, 0)], 1, 64, 16, False, seed=9)
    w = random_weights(c, 9).cuda()
    with pytest.raises(ops.PagedAttnError, match="weights_len"):
        call_with(c, w[:, :, :99].contiguous())
    with pytest.raises(ops.PagedAttnError, match="num_sinks"):
        call_with(c, w, num_sinks=-1)
    with pytest.raises(ValueError, match="weights"):
        call_with(c, w[:1])
    with pytest.raises(ValueError, match="budgets"):
        call_with(c, w, budgets=(30,))
    with pytest.raises(ops.PagedAttnError, match="max_seq_len"):
        big = torch.zeros(2, 1, 524289, device="cuda")
        call_with(c, big, max_seq_len=524289)
    ops.check_device_errors()
