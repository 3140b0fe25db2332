"""Oracle for AdamW with 8-bit moments and for the gradient norm (test infrastructure only).

A moment is held as e4m3 codes (sign, 4 exponent bits of bias 7, 3 mantissa bits; 0x7f and 0xff NaN) with one
e8m0 exponent byte e, standing for 2^(e - 127), for each 32 elements of a tensor.  The AdamW formulas are those of
adamw.py (the deep-dive page's AdamW, with the decoupled decay); the moments' new values are float32 with one IEEE
rounding per operation, the weights are computed from them in float64, and the moments are then coded:

    e     the smallest byte, 17 at least, with |x| 2^(127-e) <= 448 for all x of the block
    y     x 2^(127-e); for exp_avg_sq, where its block holds a value above zero, 2^-9 at least
    code  the e4m3 value next below |y| or the one next above: above if the distance to the lower one in units
          of the gap between the two, plus u, is 1 or more; u is a multiple of 2^-20 below 1 that a hash gives for
          (seed, step, element)

A block that holds a value which is not finite is NaN throughout (e = 255).
"""

import math

import numpy as np

from .adamw import adamw_scalars_f32

BLOCK = 32
_M = 0xFFFFFFFF


def e4m3_values():
    """The 256 values of e4m3 as float64, from the definition of its fields."""
    out = np.empty(256)
    for c in range(256):
        s, e, m = c >> 7, (c >> 3) & 15, c & 7
        v = math.ldexp(1 + m / 8, e - 7) if e else math.ldexp(m / 8, -6)
        out[c] = math.nan if c & 0x7F == 0x7F else (-v if s else v)
    return out


def moment_values(codes, scale):
    """float64 values of a moment from its code bytes and exponent bytes."""
    s = np.array([math.nan if e == 255 else math.ldexp(1.0, int(e) - 127) for e in range(256)])[scale]
    return e4m3_values()[codes] * np.repeat(s, BLOCK)[:codes.size]


def mix32(x):
    """The 32-bit mixing function, on numpy uint64 arrays or ints holding 32-bit values."""
    x = np.asarray(x, dtype=np.uint64) & np.uint64(_M)
    x = x ^ (x >> np.uint64(16))
    x = (x * np.uint64(0x6A09E667)) & np.uint64(_M)
    x = x ^ (x >> np.uint64(15))
    x = (x * np.uint64(0xBB67AE85)) & np.uint64(_M)
    return x ^ (x >> np.uint64(16))


def dither(index, seed, step, turn):
    """u of the elements `index` (int64 array): multiples of 2^-20 below 1; turn: 0 for exp_avg, 16 for exp_avg_sq."""
    key = 0
    for word in (step >> 32, step & _M, seed >> 32, seed & _M):
        key = int(mix32(word ^ key))
    index = np.asarray(index, dtype=np.uint64)
    q, j = index >> np.uint64(2), index & np.uint64(3)
    high = ((q >> np.uint64(32)) * np.uint64(0x9E3779B9)) & np.uint64(_M)
    h = mix32((q & np.uint64(_M)) ^ np.uint64(key) ^ high)
    t = (np.uint64(8) * j + np.uint64(turn)) & np.uint64(31)
    r = ((h << t) | (h >> (np.uint64(32) - t))) & np.uint64(_M)
    return (r >> np.uint64(12)).astype(np.float64) / 2 ** 20


def quantise(x, floor, index, seed, step, turn):
    """(codes, scale) of float32 values x, elements `index` of their tensor (starting at a multiple of 32)."""
    x = np.asarray(x, dtype=np.float32)
    n = x.size
    nb = -(-n // BLOCK)
    pad = np.zeros(nb * BLOCK)
    pad[:n] = x
    blocks = pad.reshape(nb, BLOCK)
    finite = np.isfinite(blocks).all(axis=1)
    largest = np.abs(np.where(np.isfinite(blocks), blocks, 0.0)).max(axis=1)
    e = np.empty(nb, dtype=np.int64)
    for k, a in enumerate(largest):
        mant, exp = math.frexp(a) if a > 0 else (0.0, -1000)   # a = mant 2^exp, mant in [1/2, 1)
        # a 2^(127-e) <= 448 = 0.875 2^9
        e[k] = max(17, 127 + exp - 9 + (1 if mant > 0.875 else 0))
    with np.errstate(invalid="ignore"):
        y = np.ldexp(blocks, (127 - e)[:, None].astype(np.int32))
    if floor:
        y = np.where((largest > 0)[:, None], np.maximum(y, 2.0 ** -9), y)
    y = np.where(finite[:, None], y, 0.0).reshape(-1)[:n]
    grid = e4m3_values()[:127]                                  # 0 .. 448, increasing
    low = np.searchsorted(grid, np.abs(y), side="right") - 1
    high = np.minimum(low + 1, 126)
    gap = np.where(high > low, grid[high] - grid[low], 1.0)
    up = (np.abs(y) - grid[low]) / gap + dither(index, seed, step, turn) >= 1
    codes = np.where(up, high, low).astype(np.uint8)
    codes = np.where(np.signbit(y), codes | 0x80, codes).astype(np.uint8)
    bad = np.repeat(~finite, BLOCK)[:n]
    codes[bad] = 0x7F
    e[~finite] = 255
    return codes, e.astype(np.uint8)


def adamw8_step(p, g, state, lr, beta1, beta2, eps, weight_decay, step, seed=0, factor=None):
    """One step: p, g float32 values, state (m codes, m scale, v codes, v scale) uint8.  Returns (p_new in float64,
    before rounding to the weights' type, the size of the update in float64, new state)."""
    k = adamw_scalars_f32(lr, beta1, beta2, eps, weight_decay, step)
    g = np.asarray(g, dtype=np.float32)
    if factor is not None:
        g = np.float32(factor) * g
    m = moment_values(state[0], state[1]).astype(np.float32)
    v = moment_values(state[2], state[3]).astype(np.float32)
    m1 = (k["beta1"] * m) + (k["one_minus_beta1"] * g)
    v1 = (k["beta2"] * v) + ((k["one_minus_beta2"] * g) * g)
    m64, v64 = m1.astype(np.float64), v1.astype(np.float64)
    v_hat = v64 / (1 - beta2 ** step)
    v_hat = np.where(np.isinf(v_hat.astype(np.float32)), np.inf, v_hat)  # as the quotient in float32, in both steps
    update = lr * (m64 / (1 - beta1 ** step)) / (np.sqrt(v_hat) + eps)
    p_new = (1 - lr * weight_decay) * np.asarray(p, dtype=np.float64) - update
    index = np.arange(g.size)
    mc, me = quantise(m1, False, index, seed, step, 0)
    vc, ve = quantise(v1, True, index, seed, step, 16)
    return p_new, update, (mc, me, vc, ve)


def grad_norm(grads, max_norm):
    """(norm, factor) of arrays of gradients: the norm in float64 with exactly rounded sums, the factor float32."""
    flat = [np.asarray(g, dtype=np.float64).ravel() for g in grads]
    if not all(np.isfinite(a).all() for a in flat):
        bad = np.concatenate([a[~np.isfinite(a)] for a in flat])
        return (math.nan if np.isnan(bad).any() else math.inf), np.float32(math.nan)
    norm = math.sqrt(math.fsum(x for a in flat for x in (a * a).tolist()))
    return norm, np.float32(max_norm / norm if norm > max_norm else 1.0)
