"""MXFP4 and the operators on it in numpy float64, written from the definitions in include/tmoe.h."""
import numpy as np

MAGS = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
BORDERS = (MAGS[1:] + MAGS[:-1]) / 2


def quantize(x):
    """(element codes [..., K], scale bytes [..., K / 32]) of float64 x."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    amax = np.abs(b).max(-1)
    e = np.full(amax.shape, -127)
    m, ex = np.frexp(amax)                              # amax = m 2^ex, m in [0.5, 1); 6 = 0.75 * 2^3
    e = np.where(amax > 0, np.maximum(ex - 3 + (m > 0.75), -127), e)
    v = np.ldexp(np.abs(b), -e[..., None])
    code = np.searchsorted(BORDERS, v, side="left")     # a value on a border takes the lower code ...
    on = np.isin(v, BORDERS[1::2])                      # ... unless the upper one is even
    code = code + on + 8 * np.signbit(b)
    code = np.where(bad[..., None], 0, code)
    return code.reshape(x.shape).astype(np.uint8), np.where(bad, 255, e + 127).astype(np.uint8)


def pack(code):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).astype(np.uint8)


def unpack(codes):
    return np.stack([codes & 15, codes >> 4], -1).reshape(*codes.shape[:-1], -1)


def values(code, scales):
    v = MAGS[code & 7] * np.where(code & 8, -1.0, 1.0)
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (v.reshape(*v.shape[:-1], -1, 32) * s[..., None]).reshape(v.shape)


def rounded(x):
    return values(*quantize(x))


def random_operand(rng, rows, K, scale=1.0):
    """(packed codes, scales, float64 values) of normal rows."""
    code, s = quantize(rng.normal(size=(rows, K)) * scale)
    return pack(code), s, values(code, s)


U = 2.0 ** -24


def product_slack(K):
    """Relative to sum |x w|: each 128-deep step rounds its sum and its addition to the accumulator (a step of
    2^-23 each if the unit truncates), and up to 16 partial sums of a split K are added."""
    return (4 * ((K + 127) // 128) + 32) * U


def layer(x, ids, w, w1, w2, y_half):
    """Reference y and a bound of what fp32 sums may change: [T][H] each.

    x float64 [T][H] (exact bf16 values); w1 [E][2I][H], w2 [E][H][I] float64 values. A sum that is off by d
    moves h = silu(g) u by dh; where h / 2^e lies within dh / 2^e of a border of the codes, or the block's
    largest value within dh of a border of the scale, the quantised value may be its neighbour."""
    T, k = ids.shape
    E, two_i, H = w1.shape
    I = two_i // 2
    xq = rounded(x)
    y, slack = np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        t, j = np.nonzero(ids == e)
        if not len(t):
            continue
        a = xq[t]
        z = a @ w1[e].T
        dz = product_slack(H) * (np.abs(a) @ np.abs(w1[e]).T)
        g, u, dg, du = z[:, :I], z[:, I:], dz[:, :I], dz[:, I:]
        sig = 1.0 / (1.0 + np.exp(-g))
        silu = g * sig
        h = silu * u
        # |silu'| <= 1.1; the fp32 exp, sum, division and product add at most 8 half steps and |g| of them in exp
        dh = 1.1 * dg * (np.abs(u) + du) + np.abs(silu) * du + (10 + np.abs(g)) * U * np.abs(h)
        code, s = quantize(h)
        b = values(code, s)
        scale = np.ldexp(1.0, s.astype(np.int64) - 127)
        v = (np.abs(h).reshape(len(t), -1, 32) / scale[..., None])
        dv = dh.reshape(v.shape) / scale[..., None]
        near = np.abs(v[..., None] - BORDERS).min(-1) <= dv
        step = np.where(near, np.where(v < 2, 0.5, np.where(v < 4, 1.0, 2.0)), 0.0)
        top, dtop = v.max(-1), dv.max(-1)
        # the scale may double (top near 6) or halve (top near 3): every value may move a coarse half step
        edge = (np.abs(top - 6) <= dtop) | (np.abs(top - 3) <= dtop)
        step = np.where(edge[..., None], 2.0, step)
        db = (step * scale[..., None]).reshape(b.shape)
        o = b @ w2[e].T
        do = db @ np.abs(w2[e]).T + product_slack(I) * (np.abs(b) @ np.abs(w2[e]).T)
        ww = w[t, j][:, None]
        np.add.at(y, t, ww * o)
        np.add.at(slack, t, np.abs(ww) * (do + (k + 2) * U * np.abs(o)))
    return y, slack * 1.01 + y_half * np.abs(y) + 1e-30
