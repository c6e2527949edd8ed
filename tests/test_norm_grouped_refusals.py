"""RMS norm, MXFP8 and grouped-product calls that are refused on the host, before any launch; and the float64 references
against values worked by hand."""
import ctypes

import numpy as np
import pytest
import torch
from torch.autograd import forward_ad

import mxfp8_ref as M

FAKE = 1 << 20                                    # never dereferenced: the checks return first


@pytest.fixture(scope="module")
def N():
    from trellis_quantized_moe_tmoe_amd import native
    return native


def _norm_cfg(N, **kw):
    d = dict(hidden=64, dtype=1, weight_dtype=1, eps=1e-6)
    d.update(kw)
    return ctypes.byref(N.NormConfig(*[d[n] for n, _ in N.NormConfig._fields_]))


BAD_NORM = [(dict(hidden=0), 1), (dict(hidden=-8), 1), (dict(dtype=3), 1), (dict(weight_dtype=2), 1),
            (dict(weight_dtype=-1), 1), (dict(eps=-1e-6), 1), (dict(eps=float("nan")), 1), (dict(eps=float("inf")), 1),
            (dict(hidden=16385), 2)]


@pytest.mark.parametrize("kw,status", BAD_NORM)
def test_norm_configuration(N, kw, status):
    need, c = ctypes.c_size_t(), _norm_cfg(N, **kw)
    assert N.lib.tmoe_rms_norm(c, FAKE, 64, None, 0, FAKE, 4, FAKE, None, FAKE, None) == status
    assert N.lib.tmoe_rms_norm_mxfp8(c, FAKE, 64, None, 0, FAKE, 4, FAKE, FAKE, None, None) == status
    assert N.lib.tmoe_rms_norm_backward_scratch(c, 4, ctypes.byref(need)) == status
    assert N.lib.tmoe_rms_norm_backward(c, FAKE, 64, FAKE, FAKE, FAKE, None, 4, FAKE, FAKE, FAKE, 1 << 30, None) == status


def test_norm_arguments(N):
    def call(x=FAKE, xs=64, res=FAKE, rs=64, w=FAKE, T=4, y=FAKE, h=FAKE, rstd=FAKE, **kw):
        return N.lib.tmoe_rms_norm(_norm_cfg(N, **kw), x, xs, res, rs, w, T, y, h, rstd, None)
    assert N.lib.tmoe_rms_norm(None, FAKE, 64, None, 0, FAKE, 4, FAKE, None, None, None) == 1
    assert call(T=0) == 0 and call(T=-1) == 1 and call(T=(1 << 22) + 1) == 2
    assert call(x=0) == 1 and call(w=0) == 1 and call(y=0) == 1 and call(h=0) == 1 and call(res=0) == 1
    assert call(xs=63) == 1 and call(rs=63) == 1 and call(xs=(1 << 32) + 1) == 1
    assert call(x=FAKE + 1) == 5 and call(res=FAKE + 1) == 5 and call(h=FAKE + 1) == 5 and call(y=FAKE + 1) == 5
    assert call(w=FAKE + 1) == 5 and call(rstd=FAKE + 2) == 5 and call(w=FAKE + 2, weight_dtype=0) == 5

    def mx(x=FAKE, res=None, h=None, codes=FAKE, scales=FAKE, T=4, **kw):
        return N.lib.tmoe_rms_norm_mxfp8(_norm_cfg(N, **kw), x, 64, res, 64, FAKE, T, codes, scales, h, None)
    assert mx(T=0) == 0 and mx(hidden=48) == 2 and mx(codes=0) == 1 and mx(scales=0) == 1 and mx(codes=FAKE + 8) == 5
    assert mx(res=FAKE) == 1 and mx(h=FAKE) == 1


def test_norm_backward_arguments(N):
    need = ctypes.c_size_t()
    assert N.lib.tmoe_rms_norm_backward_scratch(_norm_cfg(N), 0, ctypes.byref(need)) == 0 and need.value == 0
    assert N.lib.tmoe_rms_norm_backward_scratch(_norm_cfg(N), 7, None) == 1
    assert N.lib.tmoe_rms_norm_backward_scratch(_norm_cfg(N), -1, ctypes.byref(need)) == 1
    assert N.lib.tmoe_rms_norm_backward_scratch(_norm_cfg(N), 7, ctypes.byref(need)) == 0 and need.value >= 4 * 64

    def call(h=FAKE, hs=64, w=FAKE, rstd=FAKE, dy=FAKE, dh=FAKE, T=7, dx=FAKE, dw=FAKE, scratch=FAKE, size=need.value):
        return N.lib.tmoe_rms_norm_backward(_norm_cfg(N), h, hs, w, rstd, dy, dh, T, dx, dw, scratch, size, None)
    assert call(T=-1) == 1 and call(h=0) == 1 and call(w=0) == 1 and call(rstd=0) == 1 and call(dy=0) == 1
    assert call(dx=0) == 1 and call(dw=0) == 1 and call(hs=63) == 1
    assert call(scratch=0) == 3 and call(scratch=FAKE + 8) == 3 and call(size=need.value - 1) == 3
    assert call(h=FAKE + 1) == 5 and call(dy=FAKE + 1) == 5 and call(dh=FAKE + 1) == 5 and call(dx=FAKE + 1) == 5
    assert call(dw=FAKE + 1) == 5 and call(w=FAKE + 1) == 5 and call(rstd=FAKE + 2) == 5


def test_mxfp8_arguments(N):
    for fn, order in ((N.lib.tmoe_mxfp8_quantize, 0), (N.lib.tmoe_mxfp8_dequantize, 1)):
        def call(x=FAKE, dtype=0, rows=4, cols=64, codes=FAKE, scales=FAKE):
            if order == 0:
                return fn(x, dtype, rows, cols, codes, scales, None)
            return fn(codes, scales, rows, cols, dtype, x, None)
        assert call(rows=0) == 0
        assert call(rows=-1) == 1 and call(cols=0) == 1 and call(dtype=3) == 1
        assert call(cols=48) == 2 and call(rows=1 << 40) == 2
        assert call(x=0) == 1 and call(codes=0) == 1 and call(scales=0) == 1
        assert call(x=FAKE + 8) == 5 and call(codes=FAKE + 4) == 5


def _grouped_cfg(N, **kw):
    d = dict(num_experts=4, in_features=64, out_features=32, dtype=1, out_dtype=1, offsets_dtype=0)
    d.update(kw)
    return ctypes.byref(N.GroupedConfig(*[d[n] for n, _ in N.GroupedConfig._fields_]))


@pytest.mark.parametrize("kw,status", [
    (dict(num_experts=0), 1), (dict(num_experts=513), 2), (dict(in_features=0), 1), (dict(in_features=68), 2),
    (dict(in_features=65544), 2), (dict(out_features=0), 1), (dict(out_features=36), 2), (dict(out_features=65544), 2),
    (dict(dtype=0), 1), (dict(dtype=3), 1), (dict(out_dtype=2), 1), (dict(out_dtype=3), 1), (dict(offsets_dtype=2), 1)])
def test_grouped_configuration(N, kw, status):
    for fn in (N.lib.tmoe_grouped_linear, N.lib.tmoe_grouped_grad_x, N.lib.tmoe_grouped_grad_w):
        assert fn(_grouped_cfg(N, **kw), FAKE, FAKE, FAKE, 4, FAKE, None) == status
    if "dtype" not in kw:
        assert N.lib.tmoe_grouped_linear_mxfp8(_grouped_cfg(N, **kw), FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, None) == status


def test_grouped_arguments(N):
    for fn in (N.lib.tmoe_grouped_linear, N.lib.tmoe_grouped_grad_x, N.lib.tmoe_grouped_grad_w):
        def call(r=FAKE, c=FAKE, off=FAKE, R=4, y=FAKE, **kw):
            return fn(_grouped_cfg(N, **kw), r, c, off, R, y, None)
        assert fn(None, FAKE, FAKE, FAKE, 4, FAKE, None) == 1
        assert call(R=-1) == 1 and call(R=(1 << 26) + 1) == 2
        assert call(r=0) == 1 and call(c=0) == 1 and call(off=0) == 1 and call(y=0) == 1
        assert call(r=FAKE + 8) == 5 and call(c=FAKE + 8) == 5 and call(y=FAKE + 8) == 5 and call(off=FAKE + 2) == 5
        assert call(off=FAKE + 4, offsets_dtype=1) == 5
    for fn in (N.lib.tmoe_grouped_linear, N.lib.tmoe_grouped_grad_x):
        assert fn(_grouped_cfg(N), 0, 0, 0, 0, 0, None) == 0
    # more tiles than a launch has workgroups
    wide = dict(num_experts=512, in_features=65536, out_features=65536)
    assert N.lib.tmoe_grouped_grad_w(_grouped_cfg(N, **wide), FAKE, FAKE, FAKE, 4, FAKE, None) == 2
    assert N.lib.tmoe_grouped_linear(_grouped_cfg(N, **wide), FAKE, FAKE, FAKE, 1 << 26, FAKE, None) == 2

    def mx(xq=FAKE, xs=FAKE, wq=FAKE, ws=FAKE, off=FAKE, R=4, y=FAKE, **kw):
        return N.lib.tmoe_grouped_linear_mxfp8(_grouped_cfg(N, **kw), xq, xs, wq, ws, off, R, y, None)
    assert mx(R=0) == 0 and mx(R=-1) == 1 and mx(in_features=72) == 2 and mx(out_dtype=2) == 1
    for name in ("xq", "xs", "wq", "ws", "off", "y"):
        assert mx(**{name: 0}) == 1
    assert mx(xq=FAKE + 8) == 5 and mx(wq=FAKE + 8) == 5 and mx(y=FAKE + 8) == 5


def test_bindings_refuse_what_does_not_fit():
    from trellis_quantized_moe_tmoe_amd import grouped, mxfp8, norm
    z = torch.zeros
    bf = torch.bfloat16
    x, w, off = z(6, 64, dtype=bf), z(3, 32, 64, dtype=bf), z(4, dtype=torch.int32)
    dy, g = z(6, 32, dtype=bf), z(64, dtype=bf)
    u8 = lambda *s: z(*s, dtype=torch.uint8)  # noqa: E731
    tracked = z(6, 64, dtype=bf, requires_grad=True)
    for bad, msg in [
            (lambda: norm.rms_norm(x[0], g), "2-D"), (lambda: norm.rms_norm(x.double(), g), "dtype"),
            (lambda: norm.rms_norm(x.t(), z(6, dtype=bf)), "adjacent"), (lambda: norm.rms_norm(x, g[:32]), "weight: shape"),
            (lambda: norm.rms_norm(x[:1].expand(6, 64), g), "overlap"),
            (lambda: norm.rms_norm(x, g.half()), "weight: dtype"), (lambda: norm.rms_norm(x, g, x.float()), "residual: dtype"),
            (lambda: norm.rms_norm(x, g, x[:5]), "residual: shape"), (lambda: norm.rms_norm(x, g), "GPU device"),
            (lambda: norm.rms_norm_mxfp8(tracked, g), "requires a gradient"),
            (lambda: norm.rms_norm_mxfp8(x, g), "GPU device"),
            (lambda: norm.backward(x, g, z(6), x), "GPU device"),
            (lambda: mxfp8.quantize(z(4, 64)), "GPU device"), (lambda: mxfp8.quantize(z(4, 48)), "multiple of 32"),
            (lambda: mxfp8.quantize(z(4, 0)), "multiple of 32"), (lambda: mxfp8.quantize(z(64, 4).t()), "contiguous"),
            (lambda: mxfp8.quantize(z(4, 64, dtype=torch.float64)), "dtype"),
            (lambda: mxfp8.quantize(tracked * 2), "requires a gradient"),
            (lambda: mxfp8.dequantize(u8(4, 64), u8(4, 1)), "scales: shape"),
            (lambda: mxfp8.dequantize(u8(4, 64), u8(4, 2), torch.int8), "dtype"),
            (lambda: mxfp8.dequantize(u8(4, 64), u8(4, 2)), "GPU device"),
            (lambda: grouped.linear(x[0], w, off), "2 dimensions"), (lambda: grouped.linear(x, w[0], off), "3 dimensions"),
            (lambda: grouped.linear(x.float(), w, off), "dtype"), (lambda: grouped.linear(x.half(), w, off), "w: dtype"),
            (lambda: grouped.linear(x[:, ::2], w, off), "contiguous"), (lambda: grouped.linear(x[:, :32].contiguous(), w, off), "rows of 64"),
            (lambda: grouped.linear(x, w, off[:3]), "expected E"), (lambda: grouped.linear(x, w, off.float()), "offsets"),
            (lambda: grouped.linear(x, w, z(8, dtype=torch.int32)[::2]), "contiguous"),
            (lambda: grouped.linear(x, w, off, torch.float16), "out_dtype"), (lambda: grouped.linear(x, w, off), "GPU device"),
            (lambda: grouped.grad_x(x, w, off), "32 rows"), (lambda: grouped.grad_x(dy, w, off), "GPU device"),
            (lambda: grouped.grad_w(dy[:5], x, off), "6 rows"), (lambda: grouped.grad_w(dy.half(), x, off), "dy: dtype"),
            (lambda: grouped.grad_w(dy, x, off[:1]), "expected E"), (lambda: grouped.grad_w(dy, x, off), "GPU device"),
            (lambda: mxfp8.grouped_linear(u8(6, 64), u8(6, 2), u8(3, 32, 32), u8(3, 32, 1), off), "rows of 32"),
            (lambda: mxfp8.grouped_linear(u8(6, 64), u8(6, 2), u8(3, 32, 64), u8(3, 32, 1), off), "w scales: shape"),
            (lambda: mxfp8.grouped_linear(u8(6, 64), u8(6, 2), u8(3, 32, 64), u8(3, 32, 2), off, torch.float16), "out_dtype"),
            (lambda: mxfp8.grouped_linear(u8(6, 64), u8(6, 2), u8(3, 32, 64), u8(3, 32, 2), off), "GPU device")]:
        with pytest.raises(ValueError, match=msg):
            bad()


def test_configurations_are_refused_before_outputs_are_allocated(N):
    from trellis_quantized_moe_tmoe_amd import norm
    with pytest.raises(N.TmoeError, match="INVALID_ARG"):
        norm._config(64, torch.bfloat16, torch.bfloat16, -1.0)
    with pytest.raises(N.TmoeError, match="UNSUPPORTED"):
        norm._config(1 << 20, torch.bfloat16, torch.bfloat16, 1e-6)


def test_forward_mode_tangents_are_refused():
    from trellis_quantized_moe_tmoe_amd import grouped, mxfp8, norm
    with forward_ad.dual_level():
        x = forward_ad.make_dual(torch.zeros(4, 64), torch.ones(4, 64))
        b = forward_ad.make_dual(torch.zeros(4, 64).bfloat16(), torch.ones(4, 64).bfloat16())
        off = torch.zeros(2, dtype=torch.int32)
        for call in (lambda: norm.rms_norm(x, torch.ones(64)), lambda: norm.rms_norm_mxfp8(x, torch.ones(64)),
                     lambda: norm.backward(x, torch.ones(64), torch.ones(4), x), lambda: mxfp8.quantize(x),
                     lambda: grouped.linear(b, torch.zeros(1, 8, 64).bfloat16(), off),
                     lambda: grouped.grad_x(b, torch.zeros(1, 64, 8).bfloat16(), off),
                     lambda: grouped.grad_w(b, b.detach(), off)):
            with pytest.raises(ValueError, match="forward-mode"):
                call()


def test_reference_by_hand():
    assert list(M.decode(np.array([0, 1, 7, 8, 0x38, 0x7E, 0xB8], np.uint8))) == [0, 2 ** -9, 7 * 2 ** -9, 2 ** -6, 1, 448, -1]
    x = np.zeros((1, 32))
    x[0, :6] = [448, 1, -17, 18.5, 19, 0.0009]     # spacing 2 between 16 and 32, 2^-9 at the bottom
    c, s = M.quantize(x)
    assert s[0, 0] == 127 and list(M.values(c, s)[0, :6]) == [448, 1, -16, 18, 20, 0]
    x[0, 0] = 449
    assert M.quantize(x)[1][0, 0] == 128
    t = torch.arange(-460, 460, 0.37, dtype=torch.float64)
    t = t[: len(t) // 32 * 32].clamp(-448, 448)
    t[::32] = 448.0
    want = t.to(torch.float32).to(torch.float8_e4m3fn).to(torch.float64).numpy()
    c, s = M.quantize(t.to(torch.float32).double().numpy().reshape(-1, 32))
    assert np.array_equal(M.values(c, s).ravel(), want)
    y, u, r = M.norm(np.array([[3.0, -4.0]]), np.array([1.0, 2.0]), 0.0)
    assert np.allclose(r, 1 / np.sqrt(12.5)) and np.allclose(y, [[3 / np.sqrt(12.5), -8 / np.sqrt(12.5)]])
    rng = np.random.default_rng(0)
    h, g, dy, dh = rng.normal(size=(3, 5)), rng.normal(size=5), rng.normal(size=(3, 5)), rng.normal(size=(3, 5))
    dx, dg = M.norm_grad(h, g, 0.1, dy, dh)
    f = lambda h, g: (M.norm(h, g, 0.1)[0] * dy + h * dh).sum()  # noqa: E731
    for i in range(3):
        for j in range(5):
            e = np.zeros_like(h)
            e[i, j] = 1e-5
            assert abs((f(h + e, g) - f(h - e, g)) / 2e-5 - dx[i, j]) < 1e-7
    for j in range(5):
        e = np.zeros(5)
        e[j] = 1e-5
        assert abs((f(h, g + e) - f(h, g - e)) / 2e-5 - dg[j]) < 1e-7
    y, _ = M.grouped(np.eye(3), np.arange(8.0).reshape(2, 2, 2)[:, :, [0, 1, 1]], [1, 1, 3])
    assert np.array_equal(y, [[0, 0], [5, 7], [5, 7]])


def test_norm_rows_that_a_launch_has_threads_for(N):
    """A row of 16384 values takes 1024 threads, and a launch has fewer than 2^32."""
    c, need = _norm_cfg(N, hidden=16384), ctypes.c_size_t()
    T = 1 << 22
    assert N.lib.tmoe_rms_norm(c, FAKE, 16384, None, 0, FAKE, T, FAKE, None, FAKE, None) == 2
    assert N.lib.tmoe_rms_norm_mxfp8(c, FAKE, 16384, None, 0, FAKE, T, FAKE, FAKE, None, None) == 2
    assert N.lib.tmoe_rms_norm_backward_scratch(c, T, ctypes.byref(need)) == 2
    assert N.lib.tmoe_rms_norm_backward_scratch(c, T - 1, ctypes.byref(need)) == 0


def test_quantising_a_leaf_that_wants_a_gradient():
    """Only a parameter may be quantised as it is: any other tensor's gradient would get lost without a word."""
    from trellis_quantized_moe_tmoe_amd import mxfp8
    x = torch.zeros(4, 64, requires_grad=True)    # an input that the caller differentiates: a leaf
    with pytest.raises(ValueError, match="x: requires a gradient"):
        mxfp8.quantize(x)
    for fine in (lambda: mxfp8.quantize(torch.nn.Parameter(torch.zeros(4, 64))), lambda: mxfp8.quantize(x.detach())):
        with pytest.raises(ValueError, match="GPU device"):
            fine()
    with torch.no_grad(), pytest.raises(ValueError, match="GPU device"):
        mxfp8.quantize(x)
    p = torch.nn.Parameter(torch.zeros(4, 64))
    with forward_ad.dual_level(), torch.no_grad(), pytest.raises(ValueError, match="forward-mode"):
        mxfp8.quantize(forward_ad.make_dual(p, torch.ones(4, 64)))


def test_grouped_configurations_are_refused_before_outputs_are_allocated(N):
    from trellis_quantized_moe_tmoe_amd import grouped
    for sizes in ((513, 64, 32), (4, 68, 32), (4, 64, 36), (4, 65544, 32), (4, 64, 65544)):
        with pytest.raises(N.TmoeError, match="UNSUPPORTED"):
            grouped._config(*sizes, torch.bfloat16, torch.bfloat16, torch.int32)
    with pytest.raises(N.TmoeError, match="INVALID_ARG"):
        grouped._config(4, 64, 0, torch.bfloat16, torch.bfloat16, torch.int32)
    grouped._config(4, 64, 32, torch.bfloat16, torch.float32, torch.int64)
