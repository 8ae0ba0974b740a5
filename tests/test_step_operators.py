"""The operators around a step on the CPU: their plain definitions against
independent statements, and every refusal that needs no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import step_reference as R
from paged_kv_cache_174_gb300 import build as pkg_build
from paged_kv_cache_174_gb300 import ops
from paged_kv_cache_174_gb300.host.allocator import BlockAllocator


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return ops.lib()


def _status(code):
    return ops.STATUS_NAMES[code]


# ------------------------------------------------------------- the definitions
def test_build_step_hands_out_blocks_as_the_host_allocator_does():
    alloc = BlockAllocator(20, 16)
    free = list(range(19, -1, -1))  # the top of the list is its end
    tables = np.full((2, 4), -1, np.int32)
    held = [[alloc.allocate() for _ in range(2)], [alloc.allocate()]]
    for s, blocks in enumerate(held):
        tables[s, :len(blocks)] = blocks
    t, lens, starts, slots, pos, count, flagged = R.build_step(
        [20, 16], [30, 1], tables, free, 17, 16, 40)
    want = [[alloc.allocate() for _ in range(2)], [alloc.allocate()]]
    assert not flagged and count == alloc.free_count
    assert t[0].tolist() == held[0] + want[0] and t[1, :2].tolist() == held[1] + want[1]
    assert lens.tolist() == [50, 17] and starts.tolist() == [0, 30, 31]
    assert slots[0] == held[0][1] * 16 + 4 and slots[30] == want[1][0] * 16
    assert (slots[31:] == -1).all() and pos[0, :31].tolist() == list(range(20, 50)) + [16]


def test_rotation_keeps_length_and_relative_angle():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 1, 64))
    f = 10000.0 ** (-np.arange(32) / 32.0)
    for inter in (False, True):
        a, _ = R.rotate(x, [5, 5], f, None, inter)
        b, _ = R.rotate(x, [105, 105], f, None, inter)
        assert np.allclose((a * a).sum(-1), (x * x).sum(-1))
        # the product of two rotated rows depends on their distance alone
        c, _ = R.rotate(x, [5, 9], f, None, inter)
        d, _ = R.rotate(x, [1005, 1009], f, None, inter)
        assert np.allclose((c[0] * c[1]).sum(), (d[0] * d[1]).sum())


def test_wide_window_is_plain_causal_attention():
    rng = np.random.default_rng(1)
    q, K, V = (rng.standard_normal(s) for s in ((5, 4, 64), (48, 2, 64), (48, 2, 64)))
    tables, lens, starts = np.array([[1, 2, 0]]), [37], [0, 5]
    out, A, S = R.window_attention(q, K, V, tables, lens, starts, 0.125, 99, 0, 16)
    slot = tables[0][np.arange(37) // 16] * 16 + np.arange(37) % 16
    for r in range(5):
        n = 33 + r
        for h in range(4):
            s = K[slot[:n], h // 2] @ q[r, h] * 0.125
            w = np.exp(s - s.max())
            assert np.allclose(out[r, h], (w / w.sum()) @ V[slot[:n], h // 2])
    one, _, _ = R.window_attention(q, K, V, tables, lens, starts, 0.125, 1, 0, 16)
    assert np.allclose(one[4, 1], V[slot[36], 0])  # a window of one is the row's own value


# ---------------------------------------------------------------- the refusals
def test_build_step_refusals(lib):
    vp = 4096  # never read: every call here is refused before a launch
    names = ["context_lens", "new_lens", "position_offsets", "num_seqs", "num_tokens",
             "num_axes", "block_tables", "max_blocks", "block_size", "free_blocks", "free_count",
             "free_count_out", "num_blocks", "seq_lens", "query_start_loc", "slot_mapping",
             "positions"]
    good = dict(zip(names, [vp, vp, None, 4, 8, 1, vp, 4, 16, vp, vp, vp, 64, vp, vp, vp, vp]))

    def call(**kw):
        a = {**good, **kw}
        return _status(lib.pa_build_step(*[a[n] for n in names], None))
    for bad in (dict(num_seqs=-1), dict(num_tokens=-1), dict(num_axes=-1), dict(max_blocks=-1),
                dict(block_size=0), dict(num_blocks=0), dict(context_lens=None),
                dict(new_lens=None), dict(block_tables=None), dict(free_blocks=None),
                dict(free_count=None), dict(free_count_out=None), dict(seq_lens=None),
                dict(query_start_loc=None), dict(slot_mapping=None), dict(positions=None),
                dict(positions=4098), dict(context_lens=4097), dict(position_offsets=4099)):
        assert call(**bad) == "PA_ERR_INVALID_ARG", bad
    for bad in (dict(num_axes=5), dict(num_seqs=16385), dict(num_blocks=1 << 28),
                dict(max_blocks=1 << 28)):
        assert call(**bad) == "PA_ERR_UNSUPPORTED", bad


ROTARY = ["q", "q_stride", "k", "k_stride", "v", "v_stride", "num_tokens", "positions",
          "positions_stride", "num_axes", "inv_freq", "axes", "rotary_dim", "interleaved",
          "q_out", "k_cache", "v_cache", "num_blocks", "block_size", "num_q_heads",
          "num_kv_heads", "head_dim", "slot_mapping"]


@pytest.mark.parametrize("form", ["pa_rotary_reshape_and_cache",
                                  "pa_rotary_reshape_and_cache_fp8"])
def test_rotary_refusals(lib, form):
    vp = 4096
    good = dict(zip(ROTARY, [vp, 256, vp, 128, vp, 128, 3, vp, 3, 2, vp, vp, 64, 0, 8192, vp, vp,
                             8, 16, 4, 2, 64, vp]))

    def call(**kw):
        a = {**good, **kw}
        return _status(getattr(lib, form)(*[a[n] for n in ROTARY], None))
    assert call(num_tokens=0) == "PA_OK"
    for bad in (dict(num_tokens=-1), dict(num_q_heads=0), dict(rotary_dim=-16),
                dict(rotary_dim=80), dict(num_axes=0), dict(q=None), dict(k=None), dict(v=None),
                dict(q_out=None), dict(k_cache=None), dict(v_cache=None),
                dict(slot_mapping=None), dict(positions=None), dict(inv_freq=None),
                dict(q=4104), dict(v_cache=4104), dict(positions=4098), dict(inv_freq=4100),
                dict(axes=4098), dict(q_stride=252), dict(q_stride=248), dict(v_stride=120),
                dict(positions_stride=2), dict(q_out=vp, q_stride=512), dict(num_blocks=0)):
        assert call(**bad) == "PA_ERR_INVALID_ARG", bad
    for bad in (dict(head_dim=96, q_stride=384, k_stride=192, v_stride=192),
                dict(rotary_dim=40), dict(num_axes=5)):
        assert call(**bad) == "PA_ERR_UNSUPPORTED", bad
    if form.endswith("fp8"):
        assert call(block_size=24) == "PA_ERR_UNSUPPORTED"


WINDOW = ["q", "k", "v", "nb", "bs", "nq", "nkv", "d", "bt", "maxb", "sl", "qsl", "S", "T",
          "minq", "maxq", "maxl", "window", "sinks", "scale", "out", "ws", "wsb"]


@pytest.mark.parametrize("form", ["pa_paged_attention_window", "pa_paged_attention_window_fp8"])
def test_window_refusals(lib, form):
    good = dict(zip(WINDOW, [None, None, None, 32, 16, 4, 2, 64, None, 4, None, None, 4, 4, 0, 1,
                             48, 16, 4, 0.125, None, None, 0]))

    def call(**kw):
        a = {**good, **kw}
        a["scale"] = ctypes.c_float(a["scale"])
        return _status(getattr(lib, form)(*[a[n] for n in WINDOW], None))
    assert call(S=0) == "PA_OK" and call(T=0) == "PA_OK"
    assert call(window=1 << 30, sinks=0, S=0) == "PA_OK"
    for bad in (dict(window=0), dict(window=-5), dict(sinks=-1), dict(), dict(minq=3, maxq=2),
                dict(maxq=50), dict(scale=math.nan), dict(S=-1), dict(nq=5)):
        assert call(**bad) == "PA_ERR_INVALID_ARG", bad
    for bad in (dict(bs=64), dict(d=96), dict(nq=48), dict(nb=1 << 27)):
        assert call(**bad) == "PA_ERR_UNSUPPORTED", bad


def test_extension_module_leaves_what_is_not_plain(lib):
    """It answers None, and the binding's own checks decide."""
    m = ops._load_binding()
    assert m.build_step() is None and m.rotary(1, 2) is None and m.window() is None
    i32 = torch.zeros(4, dtype=torch.int32)
    assert m.build_step(i32, i32, i32.view(2, 2), i32, i32[:1], *[None] * 6, 16, 4, 1) is None
    assert m.rotary(False, *[i32] * 9, False, None) is None
    assert m.rotary(False, *[3] * 9, False, None) is None
    assert m.window(False, *[i32] * 6, 0.5, 1, 0, 0, 1, 4, None, i32) is None
    assert m.window(False, *[None] * 6, 0.5, 1, 0, 0, 1, 4, None, None) is None


def test_binding_refuses_cpu_tensors_and_wrong_types(lib):
    i32 = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.build_step(i32, i32, torch.zeros(4, 4, dtype=torch.int32), i32, i32[:1],
                       block_size=16, num_tokens=4)
    with pytest.raises(TypeError):
        ops.build_step(i32.long(), i32, torch.zeros(4, 4, dtype=torch.int32), i32, i32[:1],
                       block_size=16, num_tokens=4)
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    f = torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        ops.rotary_reshape_and_cache(x, x, x, i32, f, cache, cache, i32)
    with pytest.raises(TypeError):
        ops.rotary_reshape_and_cache(x.float(), x, x, i32, f, cache, cache, i32)
    with pytest.raises(ValueError, match="CUDA"):
        ops.paged_attention_window(x, cache, cache, i32.view(2, 2), i32[:2], i32[:3], 0.125,
                                   window=4, max_q_len=2, max_seq_len=4)


@pytest.mark.parametrize("past", [2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1, 2 ** 63 + 1])
def test_numbers_past_int32_are_refused(lib, past):
    """ctypes passes the lower 32 bits of a number: a window of 2 ** 32 + 5 would be
    a window of 5."""
    i32 = torch.zeros(4, dtype=torch.int32)
    for name in ("block_size", "num_tokens", "num_axes"):
        with pytest.raises(ValueError, match=f"{name}.*int32"):
            ops.build_step(i32, i32, torch.zeros(4, 4, dtype=torch.int32), i32, i32[:1],
                           **{"block_size": 16, "num_tokens": 4, "num_axes": 1, name: past})
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    cache = torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    for call in (ops.paged_attention_window, ops.paged_attention_window_fp8):
        for name in ("window", "num_sinks", "min_q_len", "max_q_len", "max_seq_len"):
            with pytest.raises(ValueError, match=f"{name}.*int32"):
                call(x, cache, cache, i32.view(2, 2), i32[:2], i32[:3], 0.125,
                     **{"window": 4, "max_q_len": 2, "max_seq_len": 4, name: past})
