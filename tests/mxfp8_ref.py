"""float64 references of MXFP8 quantisation, the RMS norm and the products grouped by expert, and what fp32 may round."""
import numpy as np

U = 2.0 ** -24                                    # half a step of fp32, relative


def decode(codes):
    """Values of E4M3 bytes (0x7f and 0xff: NaN)."""
    c = codes.astype(np.int64)
    ex, man = (c >> 3) & 15, (c & 7).astype(np.float64)
    v = np.where(ex == 0, np.ldexp(man, -9), np.ldexp(8 + man, ex - 10))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


POSITIVE = decode(np.arange(127))                 # ascending


def scale_exponent(amax):
    """The smallest e >= -127 with amax / 2^e <= 448 (amax finite)."""
    m, x = np.frexp(amax)                         # amax = m 2^x, m in [0.5, 1); 448 = 0.875 * 2^9
    return np.where(amax > 0, np.maximum(x - 9 + (m > 0.875), -127), -127)


def quantize(x):
    """(codes, scale bytes) of float64 x [..., K]; the nearest of all E4M3 values, ties to the even code."""
    b = x.reshape(*x.shape[:-1], -1, 32)
    bad = ~np.isfinite(b).all(-1)
    amax = np.where(bad, 0.0, np.abs(np.where(np.isfinite(b), b, 0.0)).max(-1))
    e = scale_exponent(amax)
    m = np.abs(np.where(bad[..., None], 0.0, b)) * np.ldexp(1.0, -e)[..., None]
    up = np.clip(np.searchsorted(POSITIVE, m), 1, 126)          # POSITIVE[up - 1] < m <= POSITIVE[up]
    lo, hi = m - POSITIVE[up - 1], POSITIVE[up] - m
    code = np.where((hi < lo) | ((hi == lo) & (up % 2 == 0)), up, up - 1).astype(np.uint8)
    code = np.where(np.signbit(np.where(bad[..., None], 0.0, b)), code | 128, code).astype(np.uint8)
    return code.reshape(x.shape), np.where(bad, 255, e + 127).astype(np.uint8)


def values(codes, scales):
    s = np.where(scales == 255, np.nan, np.ldexp(1.0, scales.astype(np.int64) - 127))
    return (decode(codes).reshape(*codes.shape[:-1], -1, 32) * s[..., None]).reshape(codes.shape)


def norm(h, g, eps):
    """(y, unit values, r) of float64 rows."""
    r = 1.0 / np.sqrt((h * h).mean(-1, keepdims=True) + eps)
    return h * r * g, h * r, r


# What fp32 rounds in r: a sum of positive squares through at most 16 additions in a lane, 6 across the wavefront and 16
# across wavefronts (38 with the squares themselves), halved by the root, then the mean, eps, the root and the reciprocal.
NORM_R = 19 + 4


def norm_bound(y, half, tiny):
    """r's error and the two products, then the one rounding to the output type."""
    return (half + (NORM_R + 3) * U) * np.abs(y) * 1.001 + tiny


def norm_grad(h, g, eps, dy, dh):
    _, u, r = norm(h, g, eps)
    d = dy * g
    c = (d * u).mean(-1, keepdims=True)
    return r * (d - u * c) + (0.0 if dh is None else dh), (dy * u).sum(0)


def norm_grad_bounds(h, g, eps, dy, dh, half_x, tiny_x, half_g, tiny_g):
    """u = h r is off by NORM_R + 1 units, c by those, the products and 38 additions of |d u|; dx by c's and u's share, its own
    four roundings and r's. dg sums dy u over the rows: at most 1 + T / 256 of them in a lane, 8 across a
    workgroup's rows, then n / 64 + 6 partial sums with n <= 2048."""
    dx, dg = norm_grad(h, g, eps, dy, dh)
    _, u, r = norm(h, g, eps)
    d = dy * g
    a = np.abs(d * u).mean(-1, keepdims=True)
    ex = r * (np.abs(u) * a * (2 * NORM_R + 50) + np.abs(d) * (NORM_R + 6)) * U + (0 if dh is None else np.abs(dh) * U)
    eg = np.abs(dy * u).sum(0) * (NORM_R + 2 + 1 + len(h) / 256 + 8 + 2048 / 64 + 6) * U
    return half_x * np.abs(dx) + 1.01 * ex + tiny_x, half_g * np.abs(dg) + 1.01 * eg + tiny_g


def product_bound(abs_sum, depth, ref, half, tiny):
    """fp32 sums of exact products: at most depth additions, each rounding (or cutting) at most a whole step of a partial sum
    that is at most abs_sum, plus the one rounding to the output type."""
    return half * np.abs(ref) + 2 * U * (depth + 4) * abs_sum * 1.001 + tiny


def grouped(x, w, off):
    """(y, sums of magnitudes) of x [R][K], w [E][N][K]; zeros outside every group."""
    y, s = np.zeros((len(x), w.shape[1])), np.zeros((len(x), w.shape[1]))
    for e in range(len(w)):
        a, b = off[e], off[e + 1]
        y[a:b], s[a:b] = x[a:b] @ w[e].T, np.abs(x[a:b]) @ np.abs(w[e]).T
    return y, s


def grouped_grad_w(dy, x, off):
    E = len(off) - 1
    d, s = np.zeros((E, dy.shape[1], x.shape[1])), np.zeros((E, dy.shape[1], x.shape[1]))
    for e in range(E):
        a, b = off[e], off[e + 1]
        d[e], s[e] = dy[a:b].T @ x[a:b], np.abs(dy[a:b]).T @ np.abs(x[a:b])
    return d, s


def powers(codes, scales):
    """2^exponent of MXFP8 values, as their products are aligned by the matrix unit: at least E4M3's lowest, 0 for zeros."""
    ex = np.maximum((codes.astype(np.int64) >> 3) & 15, 1) - 7
    p = np.where((codes & 127) == 0, 0.0, np.ldexp(1.0, ex))
    return (p.reshape(*codes.shape[:-1], -1, 32) * np.ldexp(1.0, scales.astype(np.int64) - 127)[..., None]).reshape(codes.shape)


def cut_bound(pa, pb):
    """What the 8-bit matrix unit may cut: it adds 16 neighbouring products at a time, each short of at most 2^-13 of the
    largest of their powers of two (that power is at most the largest product, so 16 products lose at most 16 * 2^-13 of
    it). pa [R][K], pb [N][K] powers; the sum over the groups of 16 * 2^-13 * their largest power: [R][N]."""
    total = np.zeros((len(pa), len(pb)))
    for g in range(0, pa.shape[1], 16):
        top = np.zeros_like(total)
        for k in range(g, g + 16):
            np.maximum(top, np.outer(pa[:, k], pb[:, k]), out=top)
        total += top
    return total * 2.0 ** -9
