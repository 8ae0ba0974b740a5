"""Rotary positions with the slot scatter on the GPU against 64-bit rotation:
both caches, several axes, pairings, partial rotation, far and negative
positions, strided inputs, skipped slots, in-place use."""
from fractions import Fraction

import numpy as np
import pytest
import torch

import step_reference as R
from paged_kv_cache_174_gb300 import ops

pytestmark = pytest.mark.gpu


def _inputs(seed, T, nq, nkv, d, rot, axes, far, packed=False, bs=16, skip=0.2, scale=1.0):
    rng = np.random.default_rng(seed)
    g = torch.Generator().manual_seed(seed)
    widths = [nq * d, nkv * d, nkv * d]
    if packed:
        qkv = (torch.randn(T, sum(widths) + 8, generator=g) * scale).bfloat16().cuda()
        parts = qkv[:, 8:].split(widths, 1)
    else:
        parts = [(torch.randn(T, w, generator=g) * scale).bfloat16().cuda() for w in widths]
    q, k, v = (p.unflatten(1, (-1, d)) for p in parts)
    pos = torch.from_numpy(rng.integers(-far // 4, far, (axes, T)).astype(np.int32)).cuda()
    freq = 10000.0 ** (-np.arange(rot // 2) * 2.0 / max(1, rot))
    of = rng.integers(0, axes, rot // 2).astype(np.int32)
    nb = -(-T // bs) + 2
    slots = rng.permutation(nb * bs)[:T].astype(np.int32)
    slots[rng.random(T) < skip] = -rng.integers(1, 9)
    return q, k, v, pos, freq, of, slots, nb


def _f64(t):
    return t.detach().cpu().double().numpy()


def _check_bf16(got, ref, size, what):
    y, tol = ref, R.HALF_BF16 * np.abs(ref) + 2.0 ** -20 * size
    off = np.abs(got - y)
    # cos and sin of an angle right to 2^-24 of a turn, two fp32 products and
    # a sum: 2^-20 of |x1| + |x2|; then one rounding to bf16
    assert (off <= tol).all(), f"{what}: {float((off - tol).max()):.3e} past the tolerance"
    assert np.array_equal(got[size == 0], y[size == 0]), f"{what}: passed-through elements"


CASES = [
    # T, n_q, n_kv, d, rot, axes, interleaved, far, packed, block size
    (1, 4, 2, 64, 64, 1, False, 4096, False, 16),
    (3, 8, 1, 128, 128, 3, False, 1 << 20, True, 16),
    (65, 32, 8, 128, 128, 3, False, 32768, True, 16),
    (130, 16, 2, 64, 32, 2, True, 1 << 20, False, 32),
    (77, 6, 3, 128, 96, 4, True, 2 ** 31 - 1, True, 16),
    (257, 5, 5, 64, 48, 3, False, 2 ** 31 - 1, False, 32),
    (31, 1, 1, 128, 16, 1, False, 100, True, 48),
    (9, 8, 8, 64, 0, 1, False, 100, False, 16),
    (601, 32, 8, 128, 128, 3, False, 1 << 20, True, 16),
    (703, 5, 1, 64, 64, 2, True, 9999, False, 16),
    (1, 64, 8, 128, 64, 2, True, 9999, True, 32),
]


@pytest.mark.parametrize("T,nq,nkv,d,rot,axes,inter,far,packed,bs", CASES)
def test_bf16(T, nq, nkv, d, rot, axes, inter, far, packed, bs):
    q, k, v, pos, freq, of, slots, nb = _inputs(T, T, nq, nkv, d, rot, axes, far, packed, bs)
    kc = torch.full((nb, bs, nkv, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vc = torch.full_like(kc, 9.0)
    before = [x.clone() for x in (q, k, v)]
    out = ops.rotary_reshape_and_cache(
        q, k, v, pos, torch.from_numpy(freq).cuda(), kc, vc, torch.from_numpy(slots).cuda(),
        axes=torch.from_numpy(of).cuda() if axes > 1 else None, interleaved=inter)
    ops.check_device_errors()
    for x, y in zip((q, k, v), before):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))  # inputs only read
    P, ax = pos.cpu().numpy(), of if axes > 1 else None
    ref, size = R.rotate(_f64(q), P, freq, ax, inter)
    _check_bf16(_f64(out), ref, size, "q")
    kref, ksize = R.rotate(_f64(k), P, freq, ax, inter)
    at = np.nonzero(slots >= 0)[0]
    rows = _f64(kc).reshape(-1, nkv, d)
    _check_bf16(rows[slots[at]], kref[at], ksize[at], "k")
    vrows = _f64(vc).reshape(-1, nkv, d)
    assert np.array_equal(vrows[slots[at]], _f64(v)[at])
    rest = np.setdiff1d(np.arange(nb * bs), slots[at])
    assert (rows[rest] == 7.0).all() and (vrows[rest] == 9.0).all()


@pytest.mark.parametrize("T,nq,nkv,d,rot,axes,inter,far,packed,bs", CASES)
def test_fp8(T, nq, nkv, d, rot, axes, inter, far, packed, bs):
    q, k, v, pos, freq, of, slots, nb = _inputs(T, T, nq, nkv, d, rot, axes, far, packed, bs,
                                                scale=3.0)
    k[0].zero_()  # an all-zero row
    kc, vc = ops.empty_fp8_cache(nb, bs, nkv, d)
    kw, vw = ops.empty_fp8_cache(nb, bs, nkv, d)
    dslots = torch.from_numpy(slots).cuda()
    out = ops.rotary_reshape_and_cache_fp8(
        q, k, v, pos, torch.from_numpy(freq).cuda(), kc, vc, dslots,
        axes=torch.from_numpy(of).cuda() if axes > 1 else None, interleaved=inter)
    # values are stored as the plain scatter stores them
    ops.reshape_and_cache_fp8(k.contiguous(), v.contiguous(), kw, vw, dslots)
    ops.check_device_errors()
    assert torch.equal(vc, vw)
    P, ax = pos.cpu().numpy(), of if axes > 1 else None
    ref, size = R.rotate(_f64(q), P, freq, ax, inter)
    _check_bf16(_f64(out), ref, size, "q")
    codes, scales = ops.fp8_cache_views(kc, nkv, d)
    value = _f64(codes.view(torch.float8_e4m3fn)).reshape(-1, nkv, d)
    scale = _f64(scales).reshape(-1, nkv)
    at = np.nonzero(slots >= 0)[0]
    kref, ksize = R.rotate(_f64(k), P, freq, ax, inter)
    kref, ksize = kref[at], ksize[at]
    top = np.abs(kref).max(-1)
    want = np.where(top > 0, top / 448.0, 1.0)
    got = scale[slots[at]]
    # the row's maximum is off by 2^-20 of a pair's |x1| + |x2| at most, which
    # is at most sqrt(2) times a rotated pair's length, itself at most sqrt(2)
    # times the maximum when the pair is the largest: 2^-18 covers it
    assert (np.abs(got - want) <= 2.0 ** -18 * want).all()
    mid = value[slots[at]] * got[..., None]
    # half a step of a code: 2^-4 of the value, or 2^-10 in units of the scale
    # among the subnormals
    tol = np.maximum(2.0 ** -4 * np.abs(kref), 2.0 ** -10 * want[..., None]) * (1 + 2.0 ** -10) \
        + 2.0 ** -17 * top[..., None] + 1e-30
    assert (np.abs(mid - kref) <= tol).all()
    rest = np.setdiff1d(np.arange(nb * bs), slots[at])
    assert (value[rest] == 0).all() and (scale[rest] == 0).all()


def test_in_place_queries_and_given_stream():
    q, k, v, pos, freq, of, slots, nb = _inputs(5, 40, 8, 2, 128, 128, 3, 9999)
    f, a, s = torch.from_numpy(freq).cuda(), torch.from_numpy(of).cuda(), \
        torch.from_numpy(slots).cuda()
    kc = torch.zeros(nb, 16, 2, 128, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    want = ops.rotary_reshape_and_cache(q, k, v, pos, f, kc, vc, s, axes=a)
    kc2, vc2, q2 = torch.zeros_like(kc), torch.zeros_like(kc), q.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.rotary_reshape_and_cache(q2, k, v, pos, f, kc2, vc2, s, axes=a, q_out=q2,
                                       stream=side)
    side.synchronize()
    ops.check_device_errors()
    assert got is q2
    for x, y in ((want, q2), (kc, kc2), (vc, vc2)):
        assert torch.equal(x.view(torch.int16), y.view(torch.int16))
    # one axis of positions as [T], and as rows of a wider (padded) array
    one = ops.rotary_reshape_and_cache(q, k, v, pos[1].contiguous(), f, kc, vc, s)
    wide = torch.zeros(3, 64, dtype=torch.int32, device="cuda")
    wide[0, :40] = pos[1]
    two = ops.rotary_reshape_and_cache(q, k, v, wide[:, :40], f, kc, vc, s)
    assert torch.equal(one.view(torch.int16), two.view(torch.int16))


def test_values_out_of_range_are_flagged():
    q, k, v, pos, freq, of, slots, nb = _inputs(6, 8, 4, 2, 64, 64, 2, 999, skip=0.0)
    kc = torch.zeros(nb, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    f, a, s = torch.from_numpy(freq).cuda(), torch.from_numpy(of).cuda(), \
        torch.from_numpy(slots).cuda()

    def flagged(f=f, a=a, s=s):
        out = ops.rotary_reshape_and_cache(q, k, v, pos, f, kc, vc, s, axes=a)
        with pytest.raises(ops.PagedAttnError) as e:
            ops.check_device_errors()
        assert e.value.code == 4
        return out
    bad = s.clone()
    bad[3] = nb * 16
    flagged(s=bad)
    assert (kc.view(-1, 2, 64)[s[3].item()] == 0).all()  # the token was skipped
    for value in (float("inf"), float("nan"), 2.0 ** 31):
        g = f.clone()
        g[1] = value
        out = flagged(f=g)  # the frequency counts as 0: its pair is unturned
        assert torch.equal(out[:, :, 1].view(torch.int16), q[:, :, 1].view(torch.int16))
    for value in (-1, 2):
        b = a.clone()
        b[0] = value
        flagged(a=b)
    ops.rotary_reshape_and_cache(q, k, v, pos, f, kc, vc, s, axes=a)
    ops.check_device_errors()


def test_not_a_number_stays_in_its_pair():
    q, k, v, pos, freq, of, slots, nb = _inputs(7, 5, 4, 2, 64, 64, 1, 999, skip=0.0)
    q[2, 1, 3] = float("nan")
    k[1, 0, 5] = float("inf")
    kc = torch.zeros(nb, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    out = ops.rotary_reshape_and_cache(q, k, v, pos, torch.from_numpy(freq).cuda(), kc,
                                       torch.zeros_like(kc), torch.from_numpy(slots).cuda())
    bad = torch.zeros(5, 4, 64, dtype=torch.bool, device="cuda")
    bad[2, 1, 3] = bad[2, 1, 35] = True
    assert torch.equal(~torch.isfinite(out), bad)
    rows = torch.isfinite(kc.view(-1, 2, 64)[torch.from_numpy(slots).long().cuda()])
    bad = torch.zeros(5, 2, 64, dtype=torch.bool, device="cuda")
    bad[1, 0, 5] = bad[1, 0, 37] = True
    assert torch.equal(~rows, bad)


def test_refusals():
    q, k, v, pos, freq, of, slots, nb = _inputs(8, 6, 4, 2, 64, 64, 2, 999)
    kc = torch.zeros(nb, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    f, a, s = torch.from_numpy(freq).cuda(), torch.from_numpy(of).cuda(), \
        torch.from_numpy(slots).cuda()
    good = dict(q=q, k=k, v=v, positions=pos, inv_freq=f, k_cache=kc, v_cache=kc.clone(),
                slot_mapping=s, axes=a)
    for bad in (dict(k=k[:5]), dict(v=v[:, :1]), dict(q=q.transpose(0, 1)),
                dict(slot_mapping=s[:5]), dict(positions=pos[:, :5]), dict(axes=a[:3]),
                dict(v_cache=kc[:1]), dict(q_out=q[:5].contiguous()),
                dict(k=k.repeat(1, 1, 2)[..., :64]), dict(positions=pos.t()),
                dict(positions=pos[0].expand(2, 6)), dict(q=q.cpu())):
        with pytest.raises(ValueError):
            ops.rotary_reshape_and_cache(**{**good, **bad})
    for bad in (dict(inv_freq=f.float()), dict(positions=pos.long()), dict(q=q.float()),
                dict(axes=a.long())):
        with pytest.raises(TypeError):
            ops.rotary_reshape_and_cache(**{**good, **bad})
    with pytest.raises(ops.PagedAttnError):  # 24 rotated elements
        ops.rotary_reshape_and_cache(**{**good, "inv_freq": f[:12].contiguous(),
                                        "axes": a[:12].contiguous()})


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_either_way_into_the_library(fp8):
    """The extension module's call and the binding's own checks (taken for a
    given stream and for a tensor subclass) write the same bits."""
    q, k, v, pos, freq, of, slots, nb = _inputs(9, 50, 8, 2, 64, 64, 3, 9999, packed=True)
    f, a, s = torch.from_numpy(freq).cuda(), torch.from_numpy(of).cuda(), \
        torch.from_numpy(slots).cuda()
    call = ops.rotary_reshape_and_cache_fp8 if fp8 else ops.rotary_reshape_and_cache
    seen = []
    for kw in (dict(), dict(stream=torch.cuda.current_stream()),
               dict(axes=torch.nn.Parameter(a, requires_grad=False))):
        kc, vc = ops.empty_fp8_cache(nb, 16, 2, 64) if fp8 else \
            (torch.zeros(nb, 16, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        out = call(q, k, v, pos, f, kc, vc, s, **{"axes": a, **kw})
        seen.append([x.view(torch.uint8) for x in (out, kc, vc)])
    for other in seen[1:]:
        assert all(torch.equal(x, y) for x, y in zip(seen[0], other))
    ops.check_device_errors()


def test_quotients_are_those_of_the_plain_scatter():
    """Values whose row maxima cover fp32's range, elements down to nothing:
    every code as the plain 8-bit scatter's division gives it."""
    g = torch.Generator().manual_seed(11)
    T, nkv, d = 2048, 2, 128
    x = torch.randn(T, nkv, d, generator=g)
    x = x * torch.exp2(torch.randint(-126, 120, (T, nkv, 1), generator=g).float())
    x = x * torch.exp2(-torch.randint(0, 30, (T, nkv, d), generator=g).float())
    v = x.bfloat16().cuda()
    q = torch.zeros(T, 2, d, dtype=torch.bfloat16, device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    pos = torch.zeros(T, dtype=torch.int32, device="cuda")  # no turn: keys as they are
    f = torch.ones(d // 2, dtype=torch.float64, device="cuda")
    a, b = ops.empty_fp8_cache(T // 16, 16, nkv, d)
    c, e = ops.empty_fp8_cache(T // 16, 16, nkv, d)
    ops.rotary_reshape_and_cache_fp8(q, v, v, pos, f, a, b, slots)
    ops.reshape_and_cache_fp8(v, v, c, e, slots)
    ops.check_device_errors()
    assert torch.equal(b, e)
    # a key turned by no angle is x2 * 1 + x1 * 0, which is +0 for x2 = -0 and
    # x1 >= 0: zeros are compared as numbers
    a, c = (ops.fp8_cache_views(x, nkv, d) for x in (a, c))
    assert torch.equal(a[1], c[1])
    assert torch.equal(torch.where(a[0] == 0x80, 0, a[0]), torch.where(c[0] == 0x80, 0, c[0]))


@pytest.mark.parametrize("d", [64, 128])
def test_zeros_and_non_finite_values_as_the_plain_scatter(d):
    """Signed zeros, infinities and NaN among the values, and among keys that no
    rotation touches: the plain 8-bit scatter's bytes."""
    g = torch.Generator().manual_seed(5)
    T, nkv = 333, 3
    x = torch.randn(T, nkv, d, generator=g)
    pick = torch.rand(T, nkv, d, generator=g)
    x[pick < 0.3] = 0.0
    x[pick < 0.15] = -0.0
    x[5, 0], x[6, 1] = -0.0, 0.0  # rows of zeros alone
    x[100:200][pick[100:200] > 0.99] = float("nan")
    x[200:300][pick[200:300] > 0.99] = -float("inf")
    x = x.bfloat16().cuda()
    q = torch.zeros(T, 3, d, dtype=torch.bfloat16, device="cuda")
    slots = torch.randperm(352, generator=g)[:T].int().cuda()
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    a, b = ops.empty_fp8_cache(22, 16, nkv, d)
    c, e = ops.empty_fp8_cache(22, 16, nkv, d)
    ops.rotary_reshape_and_cache_fp8(
        q, x, x, pos, torch.ones(0, dtype=torch.float64, device="cuda"), a, b, slots)
    ops.reshape_and_cache_fp8(x, x, c, e, slots)
    ops.check_device_errors()
    assert torch.equal(a, c) and torch.equal(b, e)


def _two_pi():
    """2 pi as a fraction, to 300 bits (Machin's formula)."""
    def arctan_of_inverse(n, one):
        term = total = one // n
        k, sign = 3, -1
        while term:
            term //= n * n
            total += sign * (term // k)
            k, sign = k + 2, -sign
        return total
    one = 1 << 320
    return Fraction(8 * (4 * arctan_of_inverse(5, one) - arctan_of_inverse(239, one)), one)


@pytest.mark.parametrize("fp8", [False, True], ids=["bf16", "fp8"])
def test_any_frequency_at_any_position(fp8):
    """Frequencies of both signs up to the largest, at positions up to both ends of
    int32: (1, 0) turned is (cos, sin) of an angle that whole fractions reduce."""
    freqs = [1.0, 0.37, 3.7, -3.7, 4.1, 10000.1, -7777.7, 1e6 + 0.1, -1e8 - 0.3, 3e8 + 0.7,
             2.0 ** 30 + 0.3, -(2.0 ** 30) - 0.9, 2.0 ** 31 - 0.7, -(2.0 ** 31) + 0.4,
             2.0 ** -40, -1e-300]
    positions = [0, 1, -1, 77, 2 ** 31 - 1, -2 ** 31, 2 ** 30 + 12345, -2 ** 30 - 7, 123456789,
                 1999999973]
    d, T = 64, len(positions)
    f = np.array(freqs * 2)
    tau = _two_pi()
    theta = np.empty((T, d // 2))
    for t, p in enumerate(positions):
        for i, x in enumerate(f):
            turns = p * Fraction(float(x)) / tau
            turns -= round(turns)
            theta[t, i] = float(turns * tau)
    q = torch.zeros(T, 1, d, dtype=torch.bfloat16, device="cuda")
    q[..., :d // 2] = 1.0
    slots = torch.arange(T, dtype=torch.int32, device="cuda")
    pos = torch.tensor(positions, dtype=torch.int32, device="cuda")
    if fp8:
        kc, vc = ops.empty_fp8_cache(1, 16, 1, d)
        call = ops.rotary_reshape_and_cache_fp8
    else:
        kc, vc = (torch.zeros(1, 16, 1, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        call = ops.rotary_reshape_and_cache
    out = call(q, q, q, pos, torch.from_numpy(f).cuda(), kc, vc, slots)
    ops.check_device_errors()
    ref = np.concatenate([np.cos(theta), np.sin(theta)], -1)[:, None]
    size = np.ones_like(ref)
    _check_bf16(_f64(out), ref, size, "q")
    if fp8:
        codes, scales = ops.fp8_cache_views(kc, 1, d)
        got = _f64(codes.view(torch.float8_e4m3fn)).reshape(16, 1, d)[:T] \
            * _f64(scales).reshape(16, 1)[:T, :, None]
        # half a step of a code (a subnormal one: 2^-10 of the scale, which is at
        # most 1 / 448), and as above for the turn
        tol = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 / 448) * (1 + 2.0 ** -10) + 2.0 ** -17
        assert (np.abs(got - ref) <= tol).all()
    else:
        _check_bf16(_f64(kc).reshape(16, 1, d)[:T], ref, size, "k")
