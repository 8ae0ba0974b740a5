"""The operators for long contexts on the CPU: their plain definitions against
independent statements, and every refusal that needs no GPU."""
import ctypes
import math

import numpy as np
import pytest
import torch

import long_reference as R
from paged_kv_cache_174_gb300 import build as pkg_build
from paged_kv_cache_174_gb300 import ops


@pytest.fixture(scope="module")
def lib():
    pkg_build.build()
    return ops.lib()


def _status(code):
    return ops.STATUS_NAMES[code]


# ------------------------------------------------------------- the definitions
def test_bounds_hold_every_key_and_the_score_every_product():
    rng = np.random.default_rng(0)
    K = rng.standard_normal((16, 64)) * np.exp(rng.standard_normal(64))
    codes, p = R.bounds_of(K)
    assert (codes[0] * p >= K.max(0)).all() and (codes[1] * p <= K.min(0)).all()
    assert np.abs(codes).max() <= 127 and np.abs(codes).max() >= 64
    assert (codes[0] * p - K.max(0) < p).all()
    q = np.rint(rng.standard_normal(64) * 40)
    assert np.maximum(q * codes[0], q * codes[1]).sum() * p >= (K @ q).max()
    x = np.clip(q, 0, None) @ codes[0] + np.clip(q, None, 0) @ codes[1]  # the kernel's form
    assert x == np.maximum(q * codes[0], q * codes[1]).sum()
    # the largest sum: 256 products of 127 by 127 are exact in fp32
    assert 256 * 127 * 127 < 2 ** 24


def test_power_of_two_rule_at_its_borders():
    for top in (127.0, 127.00001, 1.0, 126.9, 63.5, 63.6, 2.0 ** -140, R.FP32_MAX):
        p = R.power(top)
        assert top <= 127 * p and (top > 127 * p / 2 or p == 2.0 ** -126)
    assert R.power(0.0) == 1.0


def test_choosing_every_block_is_plain_attention():
    rng = np.random.default_rng(1)
    q, K, V = (rng.standard_normal(s) for s in ((3, 4, 64), (64, 2, 64), (64, 2, 64)))
    tables, lens, starts = np.array([[2, 0, 3]]), [37], [0, 3]
    sel = np.tile(np.arange(3), (3, 2, 1))
    out, _, _ = R.blocks_attention(q, K, V, tables, lens, starts, 0.1, 16, sel)
    w0 = np.zeros((1, 2, 48))
    out2, _, _, w, _ = R.weights_attention(q, K, V, tables, lens, starts, 0.1, 16, w0)
    assert np.allclose(out, out2)
    # each row spreads a weight of one over what it sees, each head of the group
    assert np.allclose(w.sum(-1), 3 * 2) and (w[0, :, 37:] == 0).all()
    codes, scales = np.zeros((4, 2, 2, 64)), np.ones((4, 2))
    codes, scales = R.bounds(codes, scales, K, tables, lens, None, 16)
    chosen = R.choose(q, codes, scales, tables, lens, starts, 16, 5, 1, 1,
                      np.zeros((3, 2, 5), np.int64))
    assert (chosen == [0, 1, 2, -1, -1]).all()


def test_eviction_keeps_the_heaviest_in_order():
    w = np.array([[[5, 1, 3, 3, 9, 3, 0, 2.0]]], np.float32)
    rows = np.arange(8)[:, None]
    lens, free, count, gone = R.evict([rows], w, np.array([[0]]), [8], [5], [7, -1], 1, 1, 1, 8)
    assert rows[:5, 0].tolist() == [0, 2, 3, 4, 7] and w[0, 0, :5].tolist() == [5, 3, 3, 9, 2]
    assert (lens, count, gone) == ([5], 1, [3])


# ---------------------------------------------------------------- the refusals
VP = 4096  # never read: every call here is refused before a launch, or does nothing

SUMMARIZE = ["k", "nb", "bs", "nkv", "d", "bt", "maxb", "sl", "qsl", "S", "T", "bounds", "scales"]


@pytest.mark.parametrize("form", ["pa_summarize_blocks", "pa_summarize_blocks_fp8"])
def test_summarize_refusals(lib, form):
    good = dict(zip(SUMMARIZE, [VP, 8, 16, 2, 64, VP, 4, VP, VP, 3, 5, VP, VP]))

    def call(**kw):
        a = {**good, **kw}
        return _status(getattr(lib, form)(*[a[n] for n in SUMMARIZE], None))
    assert call(S=0) == call(T=0) == call(qsl=None, maxb=0) == "PA_OK"
    for bad in (dict(nb=0), dict(bs=-16), dict(nkv=0), dict(d=0), dict(S=-1), dict(T=-1),
                dict(maxb=-1), dict(k=None), dict(bt=None), dict(sl=None), dict(bounds=None),
                dict(scales=None), dict(k=VP + 8), dict(bounds=VP + 8), dict(scales=VP + 2),
                dict(qsl=VP + 1)):
        assert call(**bad) == "PA_ERR_INVALID_ARG", bad
    for bad in (dict(bs=64), dict(bs=8), dict(d=96), dict(nkv=3), dict(nb=1 << 28),
                dict(maxb=1 << 28), dict(qsl=None, S=1 << 20, maxb=1 << 10)):
        assert call(**bad) == "PA_ERR_UNSUPPORTED", bad


SELECT = ["q", "bounds", "scales", "nb", "bs", "nq", "nkv", "d", "bt", "maxb", "sl", "qsl", "S",
          "T", "maxl", "n", "sinks", "recent", "out"]


def test_select_refusals(lib):
    good = dict(zip(SELECT, [VP, VP, VP, 8, 16, 4, 2, 64, VP, 4, VP, VP, 3, 5, 64, 3, 1, 1, VP]))

    def call(**kw):
        a = {**good, **kw}
        return _status(lib.pa_select_blocks(*[a[n] for n in SELECT], None))
    assert call(S=0) == call(T=0) == "PA_OK"
    for bad in (dict(sinks=-1), dict(recent=0), dict(n=1), dict(n=0), dict(sinks=2, recent=2),
                dict(sinks=2 ** 31 - 1, recent=2 ** 31 - 1), dict(nq=5), dict(nq=0),
                dict(maxl=-1), dict(T=-1), dict(q=None), dict(bounds=None), dict(scales=None),
                dict(bt=None), dict(sl=None), dict(qsl=None), dict(out=None), dict(q=VP + 8),
                dict(bounds=VP + 4), dict(out=VP + 2)):
        assert call(**bad) == "PA_ERR_INVALID_ARG", bad
    for bad in (dict(bs=64), dict(d=96), dict(nq=32), dict(nkv=16, nq=16), dict(T=1 << 28),
                dict(maxl=49153 * 16)):
        assert call(**bad) == "PA_ERR_UNSUPPORTED", bad
    assert call(maxl=49152 * 16, T=0) == "PA_OK"


BLOCKS = ["q", "k", "v", "nb", "bs", "nq", "nkv", "d", "bt", "maxb", "sl", "qsl", "S", "T",
          "scale", "sel", "n", "out"]


@pytest.mark.parametrize("form", ["pa_paged_attention_blocks", "pa_paged_attention_blocks_fp8"])
def test_blocks_refusals(lib, form):
    good = dict(zip(BLOCKS, [VP, VP, VP, 8, 16, 4, 2, 64, VP, 4, VP, VP, 3, 5, 0.125, VP, 3, VP]))

    def call(**kw):
        a = {**good, **kw}
        a["scale"] = ctypes.c_float(a["scale"])
        return _status(getattr(lib, form)(*[a[n] for n in BLOCKS], None))
    assert call(S=0) == call(T=0) == "PA_OK"
    for bad in (dict(n=0), dict(n=-3), dict(scale=math.nan), dict(nq=5), dict(S=-1),
                dict(q=None), dict(k=None), dict(v=None), dict(bt=None), dict(sl=None),
                dict(qsl=None), dict(sel=None), dict(out=None), dict(q=VP + 8), dict(v=VP + 8),
                dict(out=VP + 8), dict(sel=VP + 2)):
        assert call(**bad) == "PA_ERR_INVALID_ARG", bad
    for bad in (dict(bs=64), dict(d=96), dict(nq=32), dict(nb=1 << 27), dict(n=1 << 22),
                dict(T=1 << 28)):
        assert call(**bad) == "PA_ERR_UNSUPPORTED", bad


WEIGHTS = ["q", "k", "v", "nb", "bs", "nq", "nkv", "d", "bt", "maxb", "sl", "qsl", "S", "T",
           "minq", "maxq", "maxl", "scale", "w", "wlen", "out", "ws", "wsb"]


@pytest.mark.parametrize("form", ["pa_paged_attention_weights", "pa_paged_attention_weights_fp8"])
def test_weights_refusals(lib, form):
    good = dict(zip(WEIGHTS, [VP, VP, VP, 8, 16, 4, 2, 64, VP, 4, VP, VP, 3, 5, 0, 2, 64, 0.125,
                              VP, 64, VP, VP, 1 << 20]))

    def call(**kw):
        a = {**good, **kw}
        a["scale"] = ctypes.c_float(a["scale"])
        return _status(getattr(lib, form)(*[a[n] for n in WEIGHTS], None))
    assert call(S=0) == call(T=0) == "PA_OK"
    for bad in (dict(wlen=63), dict(maxl=65), dict(maxq=65), dict(minq=3), dict(maxq=-1),
                dict(wlen=-1), dict(scale=math.nan), dict(nq=5), dict(T=-1), dict(q=None),
                dict(k=None), dict(v=None), dict(bt=None), dict(sl=None), dict(qsl=None),
                dict(w=None), dict(out=None), dict(q=VP + 8), dict(w=VP + 2), dict(k=VP + 8)):
        assert call(**bad) == "PA_ERR_INVALID_ARG", bad
    for bad in (dict(bs=64), dict(d=96), dict(nq=32), dict(nb=1 << 27), dict(S=1 << 27)):
        assert call(**bad) == "PA_ERR_UNSUPPORTED", bad
    assert lib.pa_weights_workspace_size(3, 5, 5, 2, 64, 2, 64) == 0
    assert lib.pa_weights_workspace_size(3, 5, 4, 2, 96, 2, 64) == 0
    assert lib.pa_weights_workspace_size(-1, 5, 4, 2, 64, 2, 64) == 0


EVICT = ["k", "v", "w", "wlen", "nb", "bs", "nkv", "d", "bt", "maxb", "sl", "budgets", "S",
         "maxl", "sinks", "recent", "free", "count", "sl_out", "count_out", "offsets"]


@pytest.mark.parametrize("form", ["pa_evict_tokens", "pa_evict_tokens_fp8"])
def test_evict_refusals(lib, form):
    good = dict(zip(EVICT, [VP, VP, VP, 64, 8, 16, 2, 64, VP, 4, VP, VP, 3, 64, 1, 2, VP, VP, VP,
                            VP, None]))

    def call(**kw):
        a = {**good, **kw}
        return _status(getattr(lib, form)(*[a[n] for n in EVICT], None))
    for bad in (dict(sinks=-1), dict(recent=-1), dict(sinks=2 ** 31 - 1, recent=1), dict(wlen=63),
                dict(maxl=-1), dict(wlen=-1), dict(S=-1), dict(k=None), dict(v=None),
                dict(w=None), dict(bt=None), dict(sl=None), dict(budgets=None), dict(free=None),
                dict(count=None), dict(sl_out=None), dict(count_out=None), dict(k=VP + 8),
                dict(w=VP + 1), dict(offsets=VP + 2), dict(nb=0)):
        assert call(**bad) == "PA_ERR_INVALID_ARG", bad
    for bad in (dict(bs=64), dict(d=96), dict(nkv=3), dict(maxl=524289, wlen=524289),
                dict(S=1 << 27), dict(nb=1 << 28)):
        assert call(**bad) == "PA_ERR_UNSUPPORTED", bad


def test_extension_module_leaves_what_is_not_plain(lib):
    """It answers None, and the binding's own checks decide."""
    m = ops._load_binding()
    i32 = torch.zeros(4, dtype=torch.int32)
    assert m.summarize() is None and m.select_blocks(1) is None and m.blocks() is None
    assert m.weights() is None and m.evict(1, 2) is None
    for x in (i32, 3, None):
        assert m.summarize(False, *[x] * 6, 4) is None
        assert m.select_blocks(*[x] * 6, 1, 0, 1, 16, 64, None) is None
        assert m.blocks(False, *[x] * 6, 0.5, x, None) is None
        assert m.weights(False, *[x] * 6, 0.5, x, 0, 1, 4, None, None) is None
        assert m.evict(False, *[x] * 8, 0, 0, 64, None, None, None) is None


def test_binding_refuses_cpu_tensors_and_wrong_types(lib):
    bf, i32, f32 = torch.bfloat16, torch.int32, torch.float32
    k = torch.zeros(4, 16, 2, 64, dtype=bf)
    q = torch.zeros(3, 4, 64, dtype=bf)
    bt, sl, qsl = torch.zeros(2, 3, dtype=i32), torch.zeros(2, dtype=i32), torch.zeros(3, dtype=i32)
    bounds, scales = ops.alloc_bounds(4, 2, 64, device="cpu")
    assert bounds.shape == (4, 2, 2, 64) and scales.shape == (4, 2)
    w, sel = torch.zeros(2, 2, 48), torch.zeros(3, 2, 2, dtype=i32)
    calls = [
        lambda **kw: ops.summarize_blocks(*kw.get("a", (k, bt, sl, qsl, bounds, scales)),
                                          num_tokens=3),
        lambda **kw: ops.select_blocks(*kw.get("a", (q, bounds, scales, bt, sl, qsl)),
                                       num_selected=2, block_size=16, max_seq_len=48),
        lambda **kw: ops.paged_attention_blocks(*kw.get("a", (q, k, k, bt, sl, qsl)), 0.1, sel),
        lambda **kw: ops.paged_attention_weights(*kw.get("a", (q, k, k, bt, sl, qsl)), 0.1, w,
                                                 max_q_len=1, max_seq_len=48),
        lambda **kw: ops.evict_tokens(*kw.get("a", (k, k, w, bt, sl, sl)), torch.zeros(
            4, dtype=i32), torch.zeros(1, dtype=i32), max_seq_len=48)]
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call()
        with pytest.raises(TypeError, match="bfloat16"):
            call(a=(k.float(), bt, sl, qsl, bounds, scales))
    for name in ("summarize_blocks_fp8", "paged_attention_blocks_fp8",
                 "paged_attention_weights_fp8", "evict_tokens_fp8"):
        with pytest.raises((TypeError, ValueError)):
            a = {"summarize_blocks_fp8": ((k, bt, sl, qsl, bounds, scales), {}),
                 "paged_attention_blocks_fp8": ((q, k, k, bt, sl, qsl, 0.1, sel), {}),
                 "paged_attention_weights_fp8": ((q, k, k, bt, sl, qsl, 0.1, w),
                                                 dict(max_q_len=1, max_seq_len=48)),
                 "evict_tokens_fp8": ((k, k, w, bt, sl, sl, sl, sl), dict(max_seq_len=48))}[name]
            getattr(ops, name)(*a[0], **a[1])


@pytest.mark.parametrize("call", [ops.summarize_blocks, ops.summarize_blocks_fp8])
def test_a_steps_bounds_need_its_number_of_tokens(lib, call):
    """Left out beside query_start_loc it is an error, not a call that does nothing."""
    k = torch.zeros(4, 1, ops.fp8_page_bytes(2, 64), dtype=torch.uint8) \
        if call is ops.summarize_blocks_fp8 else torch.zeros(4, 16, 2, 64, dtype=torch.bfloat16)
    bt, sl, qsl = torch.zeros(2, 3, dtype=torch.int32), *(
        torch.zeros(n, dtype=torch.int32) for n in (2, 3))
    bounds, scales = ops.alloc_bounds(4, 2, 64, device="cpu")
    with pytest.raises(ValueError, match="num_tokens"):
        call(k, bt, sl, qsl, bounds, scales)
    for n in (0, 3):  # given: on to the check of the tensors
        with pytest.raises(ValueError, match="CUDA"):
            call(k, bt, sl, qsl, bounds, scales, num_tokens=n)
    with pytest.raises(ValueError, match="CUDA"):
        call(k, bt, sl, None, bounds, scales)
