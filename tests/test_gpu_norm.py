"""RMS norm, its MXFP8 form and its gradients against float64 (mxfp8_ref.py), within what fp32 sums may round; MXFP8
quantisation bit for bit."""
import numpy as np
import pytest
import torch

import mxfp8_ref as M
from gpu_cases import say

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-37, torch.bfloat16: 1e-37, torch.float16: 2.0 ** -25}   # half a step below the normal numbers


def _norm():
    from trellis_quantized_moe_tmoe_amd import norm
    return norm


def _mx():
    from trellis_quantized_moe_tmoe_amd import mxfp8
    return mxfp8


def _np(t):
    return t.double().cpu().numpy()


def _rows(T, H, dtype, seed, pad=0):
    """[T, H] values on the GPU, rows H + pad apart."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H + pad, generator=g)
    x = torch.where(torch.rand(x.shape, generator=g) < 0.01, x * 20, x)
    return x.to(dtype).cuda()[:, :H]


def _weight(H, dtype, seed):
    return (1 + 0.2 * torch.randn(H, generator=torch.Generator().manual_seed(seed))).to(dtype).cuda()


SHAPES = [(1, 1), (1, 7), (3, 8), (5, 31), (2, 255), (9, 256), (4, 257), (7, 511), (3, 512), (5, 1000), (33, 1024), (2, 2047),
          (6, 2048), (3, 2049), (2, 4095), (2, 4097), (3, 8192), (2, 10001), (1, 16384), (2, 16383), (1111, 264)]


def _check(T, H, dtype, wdtype, residual, dh, pad=0, seed=1):
    say(f"[case] norm {T}x{H} {dtype} weight {wdtype} residual {residual} dh {dh} pad {pad}")
    norm = _norm()
    x, w = _rows(T, H, dtype, seed, pad), _weight(H, wdtype, seed + 1)
    res = _rows(T, H, dtype, seed + 2, 2 * pad) if residual else None
    y, h, rstd = norm.rms_norm(x, w, res, eps=1e-5)
    want_h = x if res is None else (x.float() + res.float()).to(dtype)
    assert h is x if res is None else torch.equal(h, want_h)
    assert y.shape == (T, H) and y.dtype == dtype and y.is_contiguous() and rstd.dtype == torch.float32
    hn, g = _np(want_h), _np(w)
    ref, u, r = M.norm(hn, g, 1e-5)
    assert np.all(np.abs(_np(rstd) - r[:, 0]) <= M.NORM_R * 1.001 * M.U * r[:, 0])
    assert np.all(np.abs(_np(y) - ref) <= M.norm_bound(ref, HALF[dtype], TINY[dtype]))
    dy = _rows(T, H, dtype, seed + 3).contiguous()
    gh = _rows(T, H, dtype, seed + 4).contiguous() if dh else None
    dx, dg = norm.backward(h, w, rstd, dy, gh)
    assert dx.dtype == dtype and dg.dtype == wdtype and dg.shape == (H,)
    args = (hn, g, 1e-5, _np(dy), None if gh is None else _np(gh))
    wx, wg = M.norm_grad(*args)
    bx, bg = M.norm_grad_bounds(*args, HALF[dtype], TINY[dtype], HALF[wdtype], TINY[wdtype])
    assert np.all(np.abs(_np(dx) - wx) <= bx)
    assert np.all(np.abs(_np(dg) - wg) <= bg)


@pytest.mark.parametrize("T,H", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_norm_and_gradients(T, H, dtype):
    _check(T, H, dtype, dtype, residual=True, dh=True)


@pytest.mark.parametrize("dtype,wdtype", [(torch.bfloat16, torch.float32), (torch.float16, torch.float32)])
@pytest.mark.parametrize("residual,dh", [(False, False), (True, False), (False, True)])
def test_fp32_weight_without_residual_or_outer_gradient(dtype, wdtype, residual, dh):
    for T, H in ((17, 96), (3, 1001), (5, 4096)):
        _check(T, H, dtype, wdtype, residual, dh)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_strided_rows_at_any_element(dtype):
    for T, H, pad in ((9, 333, 5), (6, 1024, 3), (4, 2560, 1)):
        _check(T, H, dtype, dtype, residual=True, dh=True, pad=pad)
    norm = _norm()
    base = _rows(5, 700, dtype, 3)
    x, w = base[:, 13:653], _weight(641, dtype, 4)[1:]          # rows and weight start at an odd element
    y, _, _ = norm.rms_norm(x, w)
    assert torch.equal(y, norm.rms_norm(x.contiguous(), w.clone())[0])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_gradients_at_odd_addresses(dtype):
    """h strided, dy and dh contiguous but one and three elements behind an aligned address."""
    norm = _norm()
    for T, H in ((9, 256), (5, 1000), (3, 4096)):
        h, w = _rows(T, H, dtype, 1, pad=7), _weight(H, dtype, 2)
        dy, dh = (torch.empty(T * H + k, dtype=dtype, device="cuda")[k:].view(T, H).copy_(_rows(T, H, dtype, 3 + k)) for k in (1, 3))
        _, _, rstd = norm.rms_norm(h, w)
        a = norm.backward(h, w, rstd, dy, dh)
        b = norm.backward(h.contiguous(), w, rstd, dy.clone(), dh.clone())
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_rows_beyond_32_bits_of_bytes():
    """x, h and y of more than 4 GiB: the last rows are the same rows alone."""
    norm = _norm()
    T, H = 270001, 8192
    x = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
    x.zero_()
    x[-5:] = _rows(5, H, torch.bfloat16, 1)
    x[0] = _rows(1, H, torch.bfloat16, 2)
    w = _weight(H, torch.bfloat16, 3)
    y, h, rstd = norm.rms_norm(x, w, x)
    a, b, c = norm.rms_norm(x[-5:], w, x[-5:])
    assert torch.equal(y[-5:], a) and torch.equal(h[-5:], b) and torch.equal(rstd[-5:], c) and torch.all(y[1] == 0)
    codes, scales, _ = norm.rms_norm_mxfp8(x, w)
    assert torch.equal(codes[-5:], norm.rms_norm_mxfp8(x[-5:], w)[0])
    q, s = _mx().quantize(x)
    assert torch.equal(q[-5:], _mx().quantize(x[-5:].contiguous())[0]) and torch.equal(s[-5:], _mx().quantize(x[-5:].contiguous())[1])
    del y, codes, scales, q, s
    dx, dg = norm.backward(h, w, rstd, h)
    want = norm.backward(torch.cat([h[:1], h[-5:]]), w, torch.cat([rstd[:1], rstd[-5:]]), torch.cat([h[:1], h[-5:]]))
    assert torch.equal(dx[-5:], want[0][1:])
    # rows of zeros add nothing to dweight; the six others are summed in another order
    assert bool(((dg.double() - want[1].double()).abs() <= 2.0 ** -7 * want[1].double().abs()).all())


@pytest.mark.parametrize("T", [3000, 5003])
def test_many_rows(T):
    _check(T, 96, torch.bfloat16, torch.bfloat16, residual=True, dh=True)
    _check(T, 2056, torch.bfloat16, torch.float32, residual=True, dh=True)


def test_no_rows_and_one():
    norm = _norm()
    w = _weight(64, torch.bfloat16, 1)
    x = torch.zeros(0, 64, dtype=torch.bfloat16, device="cuda")
    y, h, rstd = norm.rms_norm(x, w, x)
    assert y.shape == (0, 64) and h.shape == (0, 64) and rstd.shape == (0,)
    dx, dg = norm.backward(h, w, rstd, y)
    assert dx.shape == (0, 64) and torch.equal(dg, torch.zeros_like(w))
    codes, scales, _ = norm.rms_norm_mxfp8(x, w)
    assert codes.shape == (0, 64) and scales.shape == (0, 2)


def test_zeros_infinities_and_large_rows():
    norm = _norm()
    w = torch.ones(64, device="cuda")
    x = torch.ones(6, 64, device="cuda")
    x[0] = 0.0
    x[1, 5] = float("inf")
    x[2, 5] = float("nan")
    x[3] = 1e30                                  # its squares pass fp32
    x[4] = 1e-30
    y, _, rstd = norm.rms_norm(x, w, eps=1e-6)
    assert torch.all(y[0] == 0) and torch.isnan(y[1, 5]) and torch.all(y[1, :5] == 0) and torch.isnan(y[2]).all()
    assert torch.all(y[3] == 0) and torch.allclose(y[4], x[4] * 1e3) and torch.allclose(y[5], x[5], atol=1e-6)
    codes, scales, _ = norm.rms_norm_mxfp8(x, w)
    assert torch.all(scales[2] == 255) and scales[1, 0] == 255 and scales[1, 1] == 0 and torch.all(codes[2] == 0)
    assert torch.all(scales[5] == 119) and torch.all(codes[5] == 0x78)   # 1 = 256 * 2^-8


@pytest.mark.parametrize("T,H", [(1, 32), (5, 96), (16, 1024), (3, 2080), (7, 2560), (2, 8192), (1, 16384), (300, 160)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("residual", [False, True])
def test_norm_in_mxfp8(T, H, dtype, residual):
    say(f"[case] norm mxfp8 {T}x{H} {dtype} residual {residual}")
    norm = _norm()
    x, w = _rows(T, H, dtype, 5, pad=3), _weight(H, dtype, 6)
    res = _rows(T, H, dtype, 7) if residual else None
    codes, scales, h = norm.rms_norm_mxfp8(x, w, res, eps=1e-5)
    want_h = x if res is None else (x.float() + res.float()).to(dtype)
    assert h is x if res is None else torch.equal(h, want_h)
    ref = M.norm(_np(want_h), _np(w), 1e-5)[0]
    eps = (M.NORM_R + 3) * 1.001 * M.U
    amax = np.abs(ref).reshape(T, -1, 32).max(-1)
    s = scales.cpu().numpy()
    assert np.all((s >= M.scale_exponent(amax * (1 - eps)) + 127) & (s <= M.scale_exponent(amax * (1 + eps)) + 127))
    v = M.values(codes.cpu().numpy(), s)
    scale = np.repeat(np.ldexp(1.0, s.astype(np.int64) - 127), 32, -1).reshape(T, H)
    # half a step of E4M3: 2^-4 of the value, 2^-10 of the scale below the normal numbers; and y's own error
    assert np.all(np.abs(v - ref) <= np.maximum(np.abs(ref) * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 1e-5) + eps * np.abs(ref))
    # the same bits as quantising the fp32 norm of the same rows
    y = norm.rms_norm(want_h.float(), w.float(), eps=1e-5)[0]
    if dtype == torch.float32:
        c2, s2 = _mx().quantize(y)
        assert torch.equal(c2, codes) and torch.equal(s2, scales)


def test_autograd():
    norm = _norm()
    T, H = 37, 200
    for dtype in (torch.float32, torch.bfloat16):
        for with_res in (False, True):
            x, w = _rows(T, H, dtype, 1).clone().requires_grad_(), _weight(H, dtype, 2).requires_grad_()
            res = _rows(T, H, dtype, 3).clone().requires_grad_() if with_res else None
            y, h, rstd = norm.rms_norm(x, w, res)
            assert y.requires_grad and h.requires_grad and not rstd.requires_grad
            a, b = _rows(T, H, dtype, 4).contiguous(), _rows(T, H, dtype, 5).contiguous()
            torch.autograd.backward([y, h], [a, b])
            with torch.no_grad():
                _, hh, rr = norm.rms_norm(x, w, res)
                if with_res:
                    dx, dg = norm.backward(hh, w, rr, a, b)
                else:                             # h is x: its gradient is added outside
                    dx, dg = norm.backward(hh, w, rr, a)
                    dx = dx + b
            assert torch.equal(x.grad, dx) and torch.equal(w.grad, dg)
            if with_res:
                assert torch.equal(res.grad, dx) and res.grad.data_ptr() != x.grad.data_ptr()
    # h alone, an expanded gradient, one input only, and the same tensor twice
    x, w = _rows(T, H, torch.float32, 1).clone().requires_grad_(), _weight(H, torch.float32, 2)
    r = _rows(T, H, torch.float32, 3)
    norm.rms_norm(x, w, r)[1].sum().backward()
    assert torch.equal(x.grad, torch.ones_like(x))
    x.grad = None
    norm.rms_norm(x, w, r)[0].sum().backward()
    with torch.no_grad():
        _, h, rstd = norm.rms_norm(x, w, r)
    assert torch.equal(x.grad, norm.backward(h, w, rstd, torch.ones_like(h))[0])
    x.grad = None
    norm.rms_norm(x, w, x)[1].sum().backward()
    assert torch.equal(x.grad, torch.full_like(x, 2.0))


def test_gradient_against_differences():
    """Central differences of the float64 formula, at the kernel's own inputs."""
    norm = _norm()
    T, H = 3, 40
    x, w, r = _rows(T, H, torch.float32, 1).clone(), _weight(H, torch.float32, 2), _rows(T, H, torch.float32, 3).clone()
    dy, dh = _rows(T, H, torch.float32, 4).contiguous(), _rows(T, H, torch.float32, 5).contiguous()
    _, h, rstd = norm.rms_norm(x, w, r, eps=1e-3)
    dx, dg = norm.backward(h, w, rstd, dy, dh)
    hn, g = _np(h), _np(w)
    f = lambda h, g: (M.norm(h, g, 1e-3)[0] * _np(dy) + h * _np(dh)).sum()  # noqa: E731
    for i, j in ((0, 0), (1, 17), (2, 39)):
        e = np.zeros_like(hn)
        e[i, j] = 1e-5
        # differences: 1e-10 of the third derivative and the sum's rounding / 2e-5; fp32: a few hundred units of 2^-24
        assert abs((f(hn + e, g) - f(hn - e, g)) / 2e-5 - float(dx[i, j])) < 1e-4
    for j in (0, 17, 39):
        e = np.zeros(H)
        e[j] = 1e-5
        assert abs((f(hn, g + e) - f(hn, g - e)) / 2e-5 - float(dg[j])) < 1e-4


def test_repeatable_other_stream_and_graph():
    norm = _norm()
    T, H = 700, 1032
    x, w, r = _rows(T, H, torch.bfloat16, 1).clone(), _weight(H, torch.bfloat16, 2), _rows(T, H, torch.bfloat16, 3).clone()
    dy = _rows(T, H, torch.bfloat16, 4).contiguous()

    def step():
        y, h, rstd = norm.rms_norm(x, w, r)
        return (y, h, *norm.backward(h, w, rstd, dy, h))
    a = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in range(4):
        x.copy_(_rows(T, H, torch.bfloat16, 50 + seed))
        g.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        assert all(torch.equal(p, q) for p, q in zip(got, step()))


# ---------------------------------------------------------------- MXFP8 quantisation

def _check_codes(x):
    codes, scales = _mx().quantize(x.cuda())
    want, s = M.quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), want)
    v = M.values(want, s)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        got = _mx().dequantize(codes, scales, dt)
        assert got.dtype == dt
        ref = torch.from_numpy(v).to(torch.float32).to(dt)
        assert torch.equal(got.cpu().nan_to_num(7.0, 8.0, 9.0), ref.nan_to_num(7.0, 8.0, 9.0))


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (17, 1024), (1000, 160), (2, 8192), (5, 4128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_quantize_bit_for_bit(rows, cols, dtype):
    say(f"[case] mxfp8 quantize {rows}x{cols} {dtype}")
    rng = np.random.default_rng(rows + cols)
    x = rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, 1)) * 3)
    x[rng.random((rows, cols)) < 0.02] *= 30
    x[rng.random((rows, cols)) < 0.1] = 0.0
    _check_codes(torch.from_numpy(x).to(dtype))


def test_quantize_borders_and_extremes():
    mid = (M.POSITIVE[1:] + M.POSITIVE[:-1]) / 2
    vals = np.concatenate([mid, M.POSITIVE]).astype(np.float32)
    near = np.concatenate([vals, np.nextafter(vals, np.float32(999)), np.nextafter(vals, np.float32(-999))])
    near = np.concatenate([near, -near]).astype(np.float64)
    rows = []
    for e in (-127, -126, -125, -100, -1, 0, 1, 60, 118, 119):
        for top in (448.0, 300.0, 225.0, 224.00002):
            for part in range(0, len(near), 31):
                b = np.zeros(32)
                p = np.clip(near[part:part + 31], -top, top)
                b[:len(p)] = p
                b[31] = top
                rows.append(np.ldexp(b, e))
    x = torch.from_numpy(np.array(rows)).to(torch.float32)
    assert torch.isfinite(x).all()
    _check_codes(x)
    odd = torch.zeros(8, 64)
    odd[0, 3], odd[1, 40], odd[2, 5] = float("inf"), float("nan"), -float("inf")
    odd[3] = -0.0
    odd[4, :32] = torch.finfo(torch.float32).max
    odd[5, 7] = 2.0 ** -149
    odd[6, 1], odd[6, 33] = torch.finfo(torch.float32).tiny, -torch.finfo(torch.float32).tiny
    odd[7] = torch.arange(64) - 31.5
    _check_codes(odd)


def test_dequantize_every_code_and_scale():
    codes = np.tile(np.arange(256, dtype=np.uint8), (256, 1))
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 8, 1)
    v = M.values(codes, scales)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        got = _mx().dequantize(torch.from_numpy(codes).cuda(), torch.from_numpy(scales).cuda(), dt).cpu()
        with np.errstate(over="ignore"):
            ref = torch.from_numpy(v.astype(np.float32)).to(dt)
        assert torch.equal(got.nan_to_num(7.0, 8.0, 9.0), ref.nan_to_num(7.0, 8.0, 9.0))


def test_quantize_leading_dimensions_and_no_rows():
    x = torch.randn(2, 3, 64)
    codes, scales = _mx().quantize(x.cuda())
    assert codes.shape == (2, 3, 64) and scales.shape == (2, 3, 2)
    assert np.array_equal(codes.cpu().numpy(), M.quantize(x.double().numpy())[0])
    codes, scales = _mx().quantize(torch.zeros(0, 64, device="cuda"))
    assert codes.shape == (0, 64) and _mx().dequantize(codes, scales).shape == (0, 64)


@pytest.mark.parametrize("T,H,dtype,wdtype,residual,pad", [(17003, 1001, torch.float32, torch.float32, True, 1),
                                                          (4110, 8200, torch.bfloat16, torch.float32, True, 0),
                                                          (350007, 257, torch.float16, torch.float16, True, 3)])
def test_more_bytes_than_the_caches_hold(T, H, dtype, wdtype, residual, pad):
    """Forward and backward beyond 256 MiB, with rows at any element."""
    assert T * H * dtype.itemsize * 4 > 256 << 20
    _check(T, H, dtype, wdtype, residual, residual, pad)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_mxfp8_of_more_bytes_than_the_caches_hold(dtype):
    """The same codes, scales and values as of parts that the caches hold."""
    say(f"[case] mxfp8 beyond the caches {dtype}")
    norm, mx = _norm(), _mx()
    H = 2080
    T = (256 << 20) // (H * (dtype.itemsize + 1)) + 3
    x, w = _rows(T, H, dtype, 7), _weight(H, dtype, 8)
    half = T // 2
    q, s = mx.quantize(x)
    v = mx.dequantize(q, s, dtype)
    y = norm.rms_norm_mxfp8(x, w, x)
    for a, b in ((0, half), (half, half + 1000), (T - 1000, T)):
        part = x[a:b].contiguous()
        pq, ps = mx.quantize(part)
        assert torch.equal(q[a:b], pq) and torch.equal(s[a:b], ps)
        assert torch.equal(v[a:b], mx.dequantize(pq, ps, dtype))
        small = part[:1000]
        for got, want in zip(y, norm.rms_norm_mxfp8(small, w, small)):
            assert torch.equal(got[a:a + 1000], want)


@pytest.mark.parametrize("T,H", [(3, 40), (5, 1000), (2, 2049), (3, 4096), (2, 16384)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("eps", [0.0, 1e-40, 1e-33])
def test_rows_whose_squares_are_too_small_for_fp32(T, H, dtype, eps):
    """Squares below fp32's smallest numbers, beside no eps or one that is as small: the formula's values all the same."""
    norm, eps = _norm(), float(np.float32(eps))
    w = _weight(H, dtype, 2)
    dy = _rows(T, H, dtype, 3).contiguous()
    for p in (-45, -50, -63, -75, -90, -120):     # the root mean square; r = 2^-p at most
        say(f"[case] norm {T}x{H} {dtype} eps {eps} of values near 2^{p}")
        x = (_rows(T, H, torch.float32, 1).double() * 2.0 ** p).to(dtype)
        x[0, 0] = 0.0
        y, h, rstd = norm.rms_norm(x, w, eps=eps)
        hn, g = _np(x), _np(w)
        ref, u, r = M.norm(hn, g, eps)
        assert np.all(np.abs(_np(rstd) - r[:, 0]) <= M.NORM_R * 1.001 * M.U * r[:, 0])
        assert np.all(np.abs(_np(y) - ref) <= M.norm_bound(ref, HALF[dtype], TINY[dtype]))
        if H % 32 == 0 and dtype == torch.float32:
            assert torch.equal(torch.cat(norm.rms_norm_mxfp8(x, w, eps=eps)[:2], 1), torch.cat(_mx().quantize(y), 1))
        if abs(p) > 100:                          # dx of order dy / 2^p passes the types' range
            continue
        dx, dg = norm.backward(h, w, rstd, dy)
        args = (hn, g, eps, _np(dy), None)
        wx, wg = M.norm_grad(*args)
        bx, bg = M.norm_grad_bounds(*args, HALF[dtype], TINY[dtype], HALF[dtype], TINY[dtype])
        assert np.all(np.abs(_np(dx) - wx) <= bx)
        assert np.all(np.abs(_np(dg) - wg) <= bg)


def test_rows_whose_rstd_passes_fp32():
    """A root mean square below 2^-128: y is the formula's, r is infinite. Rows of zeros without eps: 0 / 0."""
    norm = _norm()
    x = _rows(3, 72, torch.float32, 1) * 2.0 ** -100 * 2.0 ** -35
    x[1] = 0.0
    w = _weight(72, torch.float32, 2)
    y, _, rstd = norm.rms_norm(x, w, eps=0.0)
    keep = [0, 2]
    ref = M.norm(_np(x)[keep], _np(w), 0.0)[0]
    assert np.all(np.abs(_np(y)[keep] - ref) <= M.norm_bound(ref, HALF[torch.float32], TINY[torch.float32]))
    assert torch.isinf(rstd).all() and torch.isnan(y[1]).all()
    x = torch.zeros(2, 72, dtype=torch.float16, device="cuda")
    assert torch.isnan(norm.rms_norm(x, w, eps=0.0)[0]).all() and torch.all(norm.rms_norm(x, w)[0] == 0)


def test_a_weight_that_changes_before_its_own_gradient():
    """dg does not read the weight: where it alone is trained it may be written before the backward; where dx is wanted it may not."""
    norm = _norm()
    x, r, dy = (_rows(9, 200, torch.float32, s).contiguous() for s in (1, 2, 3))
    for res in (None, r):
        w = _weight(200, torch.float32, 4).requires_grad_()
        out = norm.rms_norm(x, w, res)
        with torch.no_grad():
            h, rstd = norm.rms_norm(x, w, res)[1:]
            want = norm.backward(h, w, rstd, dy)[1]
            w.zero_()
        out[0].backward(dy)
        assert torch.equal(w.grad, want)
        w = _weight(200, torch.float32, 4).requires_grad_()
        for tracked in ("x", "residual") if res is not None else ("x",):
            a = dict(x=x, residual=res)
            a[tracked] = a[tracked].clone().requires_grad_()
            y = norm.rms_norm(weight=w, **a)[0]
            with torch.no_grad():
                w.mul_(2)
            with pytest.raises(RuntimeError, match="inplace"):
                y.backward(dy)


def test_h_is_tracked_where_what_it_is_the_sum_of_is():
    """h = x + residual does not depend on the weight: with that alone tracked nothing flows through h."""
    norm = _norm()
    x, r, dy = (_rows(9, 64, torch.float32, s).contiguous() for s in (1, 2, 3))
    w = _weight(64, torch.float32, 4).requires_grad_()
    y, h, rstd = norm.rms_norm(x, w, r)
    assert y.requires_grad and not h.requires_grad and not rstd.requires_grad and torch.equal(h, x + r)
    norm.rms_norm_mxfp8(h, w.detach())            # not refused
    y.backward(dy)
    assert torch.equal(w.grad, norm.backward(h, w.detach(), rstd, dy)[1])
    for a, b in ((x.clone().requires_grad_(), r), (x, r.clone().requires_grad_())):
        assert norm.rms_norm(a, w, b)[1].requires_grad and norm.rms_norm(a, w.detach(), b)[1].requires_grad
