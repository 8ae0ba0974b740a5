"""Plain 64-bit definitions of the operators around a step, for the tests:
block tables and slots from lengths, rotary positions, attention with a
sliding window.  They share no code with the library and no code with the
oracle."""
import numpy as np
import torch

HALF_BF16 = 2.0 ** -8    # half a step, relative to the value
HALF_F16 = 2.0 ** -11


def build_step(context, new, tables, free, count, block_size, num_tokens, num_axes=1,
               offsets=None):
    """What pa_build_step defines, with lists.  Returns (tables, seq_lens,
    starts, slots, positions, count, flagged)."""
    tables = np.array(tables, np.int32)
    num_blocks, width = len(free), tables.shape[1]
    flagged = not 0 <= count <= num_blocks
    stack = [] if flagged else list(free[:count])
    slots = np.full(num_tokens, -1, np.int32)
    positions = np.zeros((num_axes, num_tokens), np.int32)
    starts, lens, row, serving, taken = [0], [], 0, True, 0
    for s, (c, n) in enumerate(zip(context, new)):
        valid = c >= 0 and n >= 0 and c + n <= width * block_size
        if not valid:
            flagged = True
        need = -(-(c + n) // block_size) - (-(-c // block_size)) if valid else 0
        if valid and (not serving or need > len(stack) or row + n > num_tokens):
            serving, flagged = False, True
        if valid and serving:
            for k in range(need):
                b = stack.pop()
                taken += 1
                if not 0 <= b < num_blocks:
                    b, flagged = -1, True
                tables[s, -(-c // block_size) + k] = b
            for p in range(c, c + n):
                b = int(tables[s, p // block_size])
                if 0 <= b < num_blocks:
                    slots[row] = b * block_size + p % block_size
                else:
                    flagged = True
                positions[:, row] = p + (offsets[s] if offsets is not None else 0)
                row += 1
            lens.append(c + n)
        else:
            lens.append(c)
        starts.append(row)
    return (tables, np.array(lens, np.int32), np.array(starts, np.int32), slots, positions,
            count - taken, flagged)


def rotate(x, positions, inv_freq, axes, interleaved):
    """x [T, heads, d] float64 turned; also |x1| + |x2| of each element's pair
    (0 for elements passed through).  Angles modulo a turn in exact rational
    steps: the position is split so that no product loses bits."""
    T = x.shape[0]
    half = len(inv_freq)
    y, size = x.copy(), np.zeros_like(x)
    if half == 0 or T == 0:
        return y, size
    pos = np.asarray(positions, np.int64).reshape(-1, T)
    theta = np.empty((T, half))
    for i in range(half):
        p = pos[axes[i] if axes is not None else 0]
        # a position below 2^31 times a frequency: high and low halves apart,
        # each reduced by whole turns before they are added
        hi, lo = (p >> 16).astype(np.float64) * 65536.0, (p & 0xffff).astype(np.float64)
        f = np.longdouble(inv_freq[i])
        tau = 2 * np.longdouble("3.14159265358979323846264338327950288")
        theta[:, i] = np.float64(np.fmod(hi * f, tau) + np.fmod(lo * f, tau))
    c, s = np.cos(theta)[:, None], np.sin(theta)[:, None]
    i = np.arange(half)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
    x1, x2 = x[..., a], x[..., b]
    y[..., a], y[..., b] = x1 * c - x2 * s, x2 * c + x1 * s
    size[..., a] = size[..., b] = np.abs(x1) + np.abs(x2)
    return y, size


def window_attention(q, K, V, tables, seq_lens, starts, scale, window, sinks, block_size):
    """Attention of the requests' rows in 64 bits.  q [T, n_q, d]; K, V [slots,
    n_kv, d] float64 (numpy).  Returns (out, A, S): the output, the weighted
    mean of |v| per element and the largest scale * sum |q_i k_i| per head row
    (the sizes the tolerances below are made of).  Rows of no request: NaN."""
    T, nq, d = q.shape
    nkv = K.shape[1]
    G = nq // nkv
    out = np.full((T, nq, d), np.nan)
    A, S = np.zeros((T, nq, d)), np.zeros((T, nq))
    for s in range(len(seq_lens)):
        t0, t1, L = int(starts[s]), int(starts[s + 1]), int(seq_lens[s])
        if t1 == t0:
            continue
        p = np.arange(L - (t1 - t0), L)[:, None]
        j = np.arange(L)
        seen = (j <= p) & ((p - j < window) | (j < sinks))
        j = j[seen.any(0)]
        seen = seen[:, j]
        slot = tables[s][j // block_size].astype(np.int64) * block_size + j % block_size
        for g in range(nkv):
            k, v = torch.from_numpy(K[slot, g]), torch.from_numpy(V[slot, g])
            x = torch.from_numpy(q[t0:t1, g * G:(g + 1) * G]).transpose(0, 1)
            hidden = torch.from_numpy(~seen)
            score = (x @ k.t() * scale).masked_fill(hidden, -float("inf"))
            size = (x.abs() @ k.abs().t() * abs(scale)).masked_fill(hidden, 0.0)
            w = torch.softmax(score, -1)
            out[t0:t1, g * G:(g + 1) * G] = (w @ v).transpose(0, 1).numpy()
            A[t0:t1, g * G:(g + 1) * G] = (w @ v.abs()).transpose(0, 1).numpy()
            S[t0:t1, g * G:(g + 1) * G] = size.amax(-1).transpose(0, 1).numpy()
    return out, A, S


def window_tolerance(out, A, S, fp8):
    """Largest error an output element may have.  The output is rounded to bf16
    (half a step of |out|).  A relative error e of the weights moves a weighted
    mean by at most e (A + |out|).  bf16 cache: weights rounded to bf16, and
    scores summed in fp32 (head_dim products: 128 * 2^-24 of S).  8-bit cache:
    q and (twice) k rounded to f16, so scores are off by 3 half steps of S, as
    is the weight; the weight and (twice) v rounded to f16.  2^-12 covers the
    exponential, the sums and the rescaling in fp32."""
    S = S[..., None]
    if fp8:
        e = 3 * HALF_F16 * S + 3 * HALF_F16 + 2.0 ** -12
    else:
        e = HALF_BF16 + 128 * 2.0 ** -24 * S + 2.0 ** -12
    return HALF_BF16 * np.abs(out) * 1.01 + e * (A + np.abs(out)) + 1e-7


def assert_window_close(got, ref, fp8, what=""):
    out, A, S = ref
    rows = ~np.isnan(out[:, 0, 0])
    assert np.isfinite(got[rows]).all(), f"{what}: non-finite outputs"
    off = np.abs(got - out)[rows]
    tol = window_tolerance(out, A, S, fp8)[rows]
    worst = float((off / tol).max()) if off.size else 0.0
    assert worst <= 1.0, f"{what}: an output is {worst:.2f} times its tolerance off"
