"""pa_build_step on the GPU against the plain definition: every output whole,
over block sizes, axes, lengths from none to long, exhausted pools and rows,
invalid requests, in-place use, streams and graph replays."""
import numpy as np
import pytest
import torch

import step_reference as R
from paged_kv_cache_174_gb300 import ops

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _case(seed, S, ctx_hi, new_hi, block_size, zero=0.2, spare=5, width=None):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, ctx_hi + 1, S)
    new = rng.integers(0, new_hi + 1, S) * (rng.random(S) >= zero)
    held = -(-ctx // block_size)
    total = -(-(ctx + new) // block_size)
    width = width or max(1, int(total.max(initial=1)))
    pool = int(total.sum()) + spare
    ids = rng.permutation(pool).astype(np.int32)
    tables = np.full((S, width), -7, np.int32)  # what the call must leave alone
    at = 0
    for s in range(S):
        tables[s, :held[s]] = ids[at:at + held[s]]
        at += held[s]
    free = np.full(pool, -1, np.int32)
    free[:pool - at] = ids[at:]
    offsets = rng.integers(-50, 50, S)
    return ctx, new, tables, free, pool - at, offsets


def _run(ctx, new, tables, free, count, offsets, block_size, T, axes, **kw):
    t = _i32(tables)
    c = _i32([count])
    lens, starts, slots, pos = ops.build_step(
        _i32(ctx), _i32(new), t, _i32(free), c, block_size=block_size, num_tokens=T,
        num_axes=axes, position_offsets=None if offsets is None else _i32(offsets), **kw)
    return [x.cpu().numpy() for x in (t, lens, starts, slots, pos)] + [int(c)]


def _compare(got, want):
    for g, w, name in zip(got, want, ("tables", "seq_lens", "starts", "slots", "positions",
                                      "count")):
        assert np.array_equal(g, w), name


def _errors(flagged):
    if flagged:
        with pytest.raises(ops.PagedAttnError) as e:
            ops.check_device_errors()
        assert e.value.code == 4
    else:
        ops.check_device_errors()


@pytest.mark.parametrize("S,ctx_hi,new_hi,bs,axes,pad,offsets", [
    (1, 0, 1, 16, 1, 0, False), (1, 5000, 513, 16, 3, 7, True), (64, 4096, 1, 16, 1, 0, False),
    (63, 300, 40, 32, 2, 100, True), (129, 2048, 300, 16, 3, 0, True), (7, 40, 9, 1, 1, 3, False),
    (1025, 100, 3, 16, 4, 1, True), (3000, 50, 2, 48, 1, 0, False), (5, 70000, 9000, 16, 1, 0, True),
])
def test_against_definition(S, ctx_hi, new_hi, bs, axes, pad, offsets):
    ctx, new, tables, free, count, off = _case(S + new_hi, S, ctx_hi, new_hi, bs)
    off = off if offsets else None
    T = int(new.sum()) + pad
    want = R.build_step(ctx, new, tables, free, count, bs, T, axes, off)
    got = _run(ctx, new, tables, free, count, off, bs, T, axes)
    _errors(want[-1])
    assert not want[-1]
    _compare(got, want)


def test_no_requests_and_no_rows():
    for S, T in ((0, 5), (0, 0), (3, 0)):
        ctx, new, tables, free, count, off = _case(1, S, 20, 0, 16, width=4)
        want = R.build_step(ctx, new, tables, free, count, 16, T, 2, off)
        got = _run(ctx, new, tables, free, count, off, 16, T, 2)
        ops.check_device_errors()
        _compare(got, want)


@pytest.mark.parametrize("short", ["blocks", "rows", "blocks to none"])
@pytest.mark.parametrize("S", [5, 40, 1500])
def test_requests_past_what_fits_are_not_served(S, short):
    ctx, new, tables, free, count, off = _case(3, S, 100, 30, 16, zero=0.1, spare=0)
    T = int(new.sum())
    if short == "rows":
        T = T // 2
    else:
        count = count // 2 if short == "blocks" else 0
    want = R.build_step(ctx, new, tables, free, count, 16, T, 1, off)
    assert want[-1]
    got = _run(ctx, new, tables, free, count, off, 16, T, 1)
    _errors(True)
    _compare(got, want)


@pytest.mark.parametrize("change", ["negative context", "negative new", "past the table",
                                    "negative count", "count past the pool", "free id",
                                    "held id", "sums past 32 bits"])
def test_values_out_of_range_are_flagged(change):
    ctx, new, tables, free, count, off = _case(4, 9, 100, 30, 16, zero=0.0)
    ctx, new = ctx.copy(), new.copy() + 1
    T = int(new.sum())
    if change == "negative context":
        ctx[3] = -1
    elif change == "negative new":
        new[0] = -4
    elif change == "past the table":
        new[5] = tables.shape[1] * 16 + 1 - ctx[5]
    elif change == "negative count":
        count = -1
    elif change == "count past the pool":
        count = len(free) + 1
    elif change == "free id":
        free[count - 2] = len(free)
    elif change == "held id":
        ctx[2], tables[2, 0] = 5, -3
    else:
        new[1:] = 2 ** 31 - 1
    want = R.build_step(ctx, new, tables, free, count, 16, T, 1, off)
    assert want[-1]
    got = _run(ctx, new, tables, free, count, off, 16, T, 1)
    _errors(True)
    _compare(got, want)


def test_in_place_steps_replayed_from_a_graph():
    """seq_lens written over context_lens and free_count in place: each replay
    is the next step."""
    ctx, _, tables, free, count, _ = _case(5, 33, 60, 0, 16, spare=200, width=20)
    lens, new, t = _i32(ctx), _i32(np.ones(33)), _i32(tables)
    f, c = _i32(free), _i32([count])
    out = [torch.empty(34, dtype=torch.int32, device="cuda"),
           torch.empty(40, dtype=torch.int32, device="cuda"),
           torch.empty(1, 40, dtype=torch.int32, device="cuda")]

    def call():
        ops.build_step(lens, new, t, f, c, block_size=16, num_tokens=40, seq_lens=lens,
                       query_start_loc=out[0], slot_mapping=out[1], positions=out[2])
    state = [x.clone() for x in (lens, t, c)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()  # before the capture: the library looks up its device state once
    torch.cuda.current_stream().wait_stream(side)
    for x, y in zip((lens, t, c), state):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for _ in range(40):
        graph.replay()
        tables, ctx, starts, slots, pos, count, flagged = R.build_step(
            ctx, np.ones(33, int), tables, free, count, 16, 40)
        assert not flagged
        _compare([t.cpu().numpy(), lens.cpu().numpy()] + [x.cpu().numpy() for x in out]
                 + [int(c)], (tables, ctx, starts, slots, pos, count))
    ops.check_device_errors()


def test_given_stream():
    ctx, new, tables, free, count, off = _case(6, 20, 100, 30, 16)
    T = int(new.sum())
    want = R.build_step(ctx, new, tables, free, count, 16, T, 1, off)
    s = torch.cuda.Stream()
    args = [_i32(ctx), _i32(new), _i32(tables), _i32(free), _i32([count])]
    o = _i32(off)
    s.wait_stream(torch.cuda.current_stream())
    for handle in (s, s.cuda_stream):
        args[2].copy_(_i32(tables))
        args[4].fill_(count)
        s.wait_stream(torch.cuda.current_stream())
        got = ops.build_step(*args, block_size=16, num_tokens=T, position_offsets=o,
                             stream=handle)
        s.synchronize()
        _compare([args[2].cpu().numpy()] + [x.cpu().numpy() for x in got] + [int(args[4])], want)
    ops.check_device_errors()


def test_refusals():
    a = [_i32([1, 2]), _i32([1, 1]), _i32([[0], [1]]), _i32([2, 3, 4]), _i32([2])]
    kw = dict(block_size=16, num_tokens=2)
    for bad in (dict(num_tokens=-1), dict(num_axes=-1), dict(seq_lens=_i32([1])),
                dict(slot_mapping=_i32([1, 2, 3])), dict(position_offsets=_i32([1])),
                dict(free_count_out=_i32([1, 2]))):
        with pytest.raises(ValueError):
            ops.build_step(*a, **{**kw, **bad})
    for bad in (dict(block_size=0), dict(num_axes=5)):
        with pytest.raises(ops.PagedAttnError):
            ops.build_step(*a, **{**kw, **bad})
    with pytest.raises(ValueError):
        ops.build_step(a[0], _i32([1]), *a[2:], **kw)
    with pytest.raises(ValueError):
        ops.build_step(*a[:4], _i32([1, 2]), **kw)


def test_either_way_into_the_library():
    """The extension module's call and the binding's own checks (taken for a
    given stream, other number types) write the same values."""
    ctx, new, tables, free, count, off = _case(7, 20, 100, 30, 16)
    T = int(new.sum()) + 3
    want = R.build_step(ctx, new, tables, free, count, 16, T, 2, off)
    for kw in (dict(), dict(stream=torch.cuda.current_stream())):
        for num in (int, np.int64):
            _compare(_run(ctx, new, tables, free, count, off, num(16), num(T), num(2), **kw), want)
    ops.check_device_errors()


@pytest.mark.parametrize("given", [(), (0,), (1, 3), (0, 1, 2, 3)])
def test_outputs_made_by_the_call_are_apart(given):
    """Whichever outputs the caller passes, the others are contiguous tensors
    that writing to one, and dropping the rest, leaves as they are."""
    ctx, new, tables, free, count, offsets = _case(4, 7, 90, 30, 16)
    T, axes = int(new.sum()) + 3, 3
    want = R.build_step(ctx, new, tables, free, count, 16, T, axes, offsets)
    names = ("seq_lens", "query_start_loc", "slot_mapping", "positions")
    shapes = ((7,), (8,), (T,), (axes, T))
    for mode in (torch.no_grad, torch.inference_mode):
        with mode():
            mine = {names[i]: torch.full(shapes[i], -9, dtype=torch.int32, device="cuda")
                    for i in given}
            args = (_i32(ctx), _i32(new), _i32(tables), _i32(free), _i32([count]))
            out = ops.build_step(*args, block_size=16, num_tokens=T, num_axes=axes,
                                 position_offsets=_i32(offsets), **mine)
            ops.check_device_errors()
            for i, x in enumerate(out):
                assert x.is_contiguous() and x.dtype is torch.int32 and tuple(x.shape) == shapes[i]
                assert (x is mine[names[i]]) if i in given else x.data_ptr() % 16 == 0
            for i, x in enumerate(out):
                kept = [y.clone() for y in out]
                x.fill_(-5)
                for j, y in enumerate(out):
                    assert j == i or torch.equal(y, kept[j])
                x.copy_(kept[i])
            last = out[3]
            rest = [x.cpu().numpy() for x in out[:3]]
            del out, mine, x, y
            torch.empty(1 << 16, dtype=torch.int32, device="cuda").fill_(77)
            for got, w in zip(rest + [last.cpu().numpy()], want[1:5]):
                assert np.array_equal(got, w)


@pytest.mark.parametrize("S", [4051, 4052, 4095, 4096, 16384])
@pytest.mark.parametrize("pad", [0, 20000])
def test_as_many_requests_as_the_call_takes(S, pad):
    """Past a block's 48 KB of shared memory, its fixed part counted: 12 bytes a
    request beside it reach them at 4052 requests."""
    ctx, new, tables, free, count, off = _case(S, S, 60, 1, 16, zero=0.9)
    T = int(new.sum()) + pad
    want = R.build_step(ctx, new, tables, free, count, 16, T, 1, off)
    got = _run(ctx, new, tables, free, count, off, 16, T, 1)
    _errors(want[-1])
    assert not want[-1]
    _compare(got, want)
