"""MXFP4 calls that are refused on the host, before any launch; and the float64 reference against values
worked by hand."""
import ctypes

import numpy as np
import pytest
import torch

import mxfp4_ref as M

FAKE = 1 << 20                                    # never dereferenced: the checks return first


@pytest.fixture(scope="module")
def N():
    from trellis_quantized_moe_tmoe_amd import native
    return native


def test_quantize_arguments(N):
    for fn, order in ((N.lib.tmoe_mxfp4_quantize, 0), (N.lib.tmoe_mxfp4_dequantize, 1)):
        def call(x=FAKE, dtype=0, rows=4, cols=64, codes=FAKE, scales=FAKE):
            if order == 0:
                return fn(x, dtype, rows, cols, codes, scales, None)
            return fn(codes, scales, rows, cols, dtype, x, None)
        assert call(rows=0) == 0
        assert call(rows=-1) == 1 and call(cols=0) == 1 and call(dtype=3) == 1
        assert call(cols=48) == 2 and call(rows=1 << 40) == 2
        assert call(x=0) == 1 and call(codes=0) == 1 and call(scales=0) == 1
        assert call(x=FAKE + 8) == 5 and call(codes=FAKE + 4) == 5


def test_linear_arguments(N):
    def call(xq=FAKE, xs=FAKE, T=4, wq=FAKE, ws=FAKE, K=64, n=10, dtype=0, y=FAKE):
        return N.lib.tmoe_linear_mxfp4(xq, xs, T, wq, ws, K, n, dtype, y, None)
    assert call(T=0) == 0
    assert call(T=-1) == 1 and call(K=0) == 1 and call(n=0) == 1 and call(dtype=2) == 1
    assert call(K=48) == 2 and call(K=65568) == 2 and call(n=65537) == 2 and call(T=(1 << 20) + 1) == 2
    assert call(xq=0) == 1 and call(xs=0) == 1 and call(wq=0) == 1 and call(ws=0) == 1 and call(y=0) == 1
    assert call(xq=FAKE + 8) == 5 and call(wq=FAKE + 4) == 5 and call(y=FAKE + 2) == 5


def _cfg(N, **kw):
    d = dict(hidden=1024, inter=512, num_experts=8, top_k=2, max_tokens=16, ids_dtype=1, y_dtype=0)
    d.update(kw)
    return N.Mxfp4Config(*[d[n] for n, _ in N.Mxfp4Config._fields_])


@pytest.mark.parametrize("kw,status", [
    (dict(), 0), (dict(hidden=32, inter=32), 0), (dict(hidden=2560, inter=320), 0), (dict(hidden=0), 1),
    (dict(hidden=48), 2), (dict(hidden=8224), 2), (dict(inter=16), 2), (dict(num_experts=513), 2), (dict(top_k=33), 2),
    (dict(num_experts=0), 1), (dict(top_k=0), 1), (dict(max_tokens=0), 1), (dict(max_tokens=1 << 22), 2),
    (dict(ids_dtype=2), 1), (dict(y_dtype=2), 1)])
def test_plan_is_checked(N, kw, status):
    h, sb = ctypes.c_void_p(), ctypes.c_size_t()
    assert N.lib.tmoe_mxfp4_plan(ctypes.byref(_cfg(N, **kw)), ctypes.byref(h), ctypes.byref(sb)) == status
    if status == 0:
        assert sb.value > 0 and N.lib.tmoe_mxfp4_plan_destroy(h) == 0
    else:
        assert not h.value


def test_forward_arguments(N):
    h, sb = ctypes.c_void_p(), ctypes.c_size_t()
    assert N.lib.tmoe_mxfp4_plan(None, ctypes.byref(h), None) == 1 and N.lib.tmoe_mxfp4_plan_destroy(None) == 1
    assert N.lib.tmoe_mxfp4_plan(ctypes.byref(_cfg(N)), ctypes.byref(h), ctypes.byref(sb)) == 0
    w = N.Mxfp4Weights(*([FAKE] * 4))

    def call(**o):
        return N.lib.tmoe_forward_mxfp4(o.get("plan", h), o.get("x", FAKE), o.get("ids", FAKE), o.get("w", FAKE),
                                        o.get("T", 4), ctypes.byref(o.get("wt", w)), o.get("y", FAKE),
                                        o.get("scratch", FAKE), o.get("bytes", sb.value), None)
    assert call(T=0) == 0 and call(T=17) == 4 and call(T=-1) == 1 and call(plan=None) == 1
    assert call(bytes=sb.value - 1) == 3 and call(scratch=FAKE + 8) == 3 and call(scratch=0) == 3
    assert call(x=0) == 1 and call(ids=0) == 1 and call(w=0) == 1 and call(y=0) == 1
    assert call(x=FAKE + 2) == 5 and call(ids=FAKE + 4) == 5 and call(w=FAKE + 2) == 5 and call(y=FAKE + 8) == 5
    for i in range(4):
        assert call(wt=N.Mxfp4Weights(*[0 if j == i else FAKE for j in range(4)])) == 1
    assert call(wt=N.Mxfp4Weights(FAKE + 8, FAKE, FAKE, FAKE)) == 5
    assert call(wt=N.Mxfp4Weights(FAKE, FAKE, FAKE + 4, FAKE)) == 5
    N.lib.tmoe_mxfp4_plan_destroy(h)


def test_binding_refuses_what_does_not_fit():
    from trellis_quantized_moe_tmoe_amd import mxfp4
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    xq, xs, wq, ws = u8(4, 32), u8(4, 2), u8(6, 32), u8(6, 2)
    plan = mxfp4.ExpertPlan(64, 32, 4, 2, 8)
    wt = mxfp4.ExpertWeights(u8(4, 64, 32), u8(4, 64, 2), u8(4, 64, 16), u8(4, 64, 1))
    a = dict(x=torch.zeros(3, 64, dtype=torch.bfloat16), ids=torch.zeros(3, 2, dtype=torch.int64), w=torch.zeros(3, 2),
             weights=wt, scratch=u8(plan.scratch_bytes))
    short = mxfp4.ExpertWeights(wt.w1, wt.s1[:, :, :1], wt.w2, wt.s2)
    for bad, msg in [(lambda: mxfp4.quantize(torch.zeros(4, 64)), "GPU device"),
                     (lambda: mxfp4.quantize(torch.zeros(4, 48)), "multiple of 32"),
                     (lambda: mxfp4.quantize(torch.zeros(4, 0)), "multiple of 32"),
                     (lambda: mxfp4.quantize(torch.zeros(64, 4).t()), "contiguous"),
                     (lambda: mxfp4.quantize(torch.zeros(4, 64, dtype=torch.float64)), "dtype"),
                     (lambda: mxfp4.dequantize(xq, ws), "scales: shape"),
                     (lambda: mxfp4.dequantize(xq, xs, torch.int8), "dtype"),
                     (lambda: mxfp4.dequantize(xq, xs), "GPU device"),
                     (lambda: mxfp4.linear(xq, xs, u8(6, 16), u8(6, 1)), "rows of 32"),
                     (lambda: mxfp4.linear(xq[0], xs[0], wq, ws), "2 dimensions"),
                     (lambda: mxfp4.linear(xq, xs, wq, ws, torch.float16), "out_dtype"),
                     (lambda: mxfp4.linear(xq, xs, wq, ws, y=torch.zeros(4, 5)), "y: shape"),
                     (lambda: mxfp4.linear(xq, xs, wq, ws), "GPU device"),
                     (lambda: mxfp4.ExpertPlan(64, 32, 4, 2, 8, ids_dtype=torch.int16), "ids_dtype"),
                     (lambda: mxfp4.ExpertPlan(64, 32, 4, 2, 8, out_dtype=torch.float16), "out_dtype"),
                     (lambda: plan.forward(**{**a, "x": torch.zeros(9, 64, dtype=torch.bfloat16)}), "at most"),
                     (lambda: plan.forward(**{**a, "ids": a["ids"].int()}), "ids: dtype"),
                     (lambda: plan.forward(**{**a, "w": a["w"][:2]}), "w: shape"),
                     (lambda: plan.forward(**{**a, "weights": short}), "s1: shape"),
                     (lambda: plan.forward(**{**a, "scratch": a["scratch"][:-1]}), "scratch"),
                     (lambda: plan.forward(**a, y=torch.zeros(3, 64, dtype=torch.bfloat16)), "y: dtype"),
                     (lambda: plan.forward(**a), "GPU device")]:
        with pytest.raises(ValueError, match=msg):
            bad()


def test_a_refused_call_leaves_its_output_as_it_was():
    """Autograd is told that y is written only by a call that writes it."""
    from trellis_quantized_moe_tmoe_amd import mxfp4
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    plan = mxfp4.ExpertPlan(64, 32, 4, 2, 8)
    wt = mxfp4.ExpertWeights(u8(4, 64, 32), u8(4, 64, 2), u8(4, 64, 16), u8(4, 64, 1))
    y = torch.zeros(3, 64)
    with pytest.raises(ValueError, match="GPU device"):
        plan.forward(torch.zeros(3, 64, dtype=torch.bfloat16), torch.zeros(3, 2, dtype=torch.int64), torch.zeros(3, 2), wt,
                     u8(plan.scratch_bytes), y=y)
    with pytest.raises(ValueError, match="GPU device"):
        mxfp4.linear(u8(3, 32), u8(3, 2), u8(64, 32), u8(64, 2), y=y)
    assert y._version == 0


def test_gradients_are_refused_not_lost():
    """The calls read addresses and have no backward: a tensor that wants a gradient, in either mode, is refused unless
    gradients are off; the bf16 activations and the router's weights of a training step among them."""
    from torch.autograd import forward_ad
    from trellis_quantized_moe_tmoe_amd import mxfp4
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8)  # noqa: E731
    plan = mxfp4.ExpertPlan(64, 32, 4, 2, 8)
    a = dict(x=torch.zeros(3, 64, dtype=torch.bfloat16), ids=torch.zeros(3, 2, dtype=torch.int64), w=torch.zeros(3, 2),
             weights=mxfp4.ExpertWeights(u8(4, 64, 32), u8(4, 64, 2), u8(4, 64, 16), u8(4, 64, 1)),
             scratch=u8(plan.scratch_bytes), y=torch.zeros(3, 64))
    logits = torch.zeros(3, 4, requires_grad=True)
    calls = [lambda f: mxfp4.quantize(f(torch.zeros(4, 64)) * 1.0),    # an activation: something lies behind it
             lambda f: mxfp4.linear(u8(4, 32), u8(4, 2), u8(6, 32), u8(6, 2), y=f(torch.zeros(4, 6)))]
    calls += [lambda f, n=n: plan.forward(**{**a, n: f(a[n])}) for n in ("x", "w", "y")]
    leaf = lambda t: t.clone().requires_grad_()  # noqa: E731
    for call in calls:
        with pytest.raises(ValueError, match="requires a gradient"):
            call(leaf)
        with torch.no_grad(), pytest.raises(ValueError, match="GPU device"):
            call(leaf)
        with forward_ad.dual_level(), torch.no_grad(), pytest.raises(ValueError, match="forward-mode"):
            call(lambda t: forward_ad.make_dual(t, torch.ones_like(t)))
    with pytest.raises(ValueError, match="GPU device"):                # a parameter, as a program loads it
        mxfp4.quantize(torch.nn.Parameter(torch.zeros(4, 64)))
    with pytest.raises(ValueError, match="w: requires a gradient"):
        plan.forward(**{**a, "w": torch.softmax(logits, 1)[:, :2].contiguous()})


def test_reference_by_hand():
    x = np.zeros(64)
    x[:8] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0]
    x[32:36] = [-7.0, 0.5, -0.5, 12.0]
    code, s = M.quantize(x)
    assert s.tolist() == [127, 128]                     # 6 fits at 2^0, 12 at 2^1
    assert code[:8].tolist() == [0, 2, 2, 4, 4, 6, 6, 7]
    assert code[32:36].tolist() == [14, 0, 8, 7]        # -3.5 -> -4 (even), +-0.25 -> +-0, 6
    assert M.values(code, s)[32:36].tolist() == [-8.0, 0.0, -0.0, 12.0]
    assert M.quantize(np.full(32, np.nextafter(6.0, 7.0)))[1].tolist() == [128]
    assert M.quantize(np.full(32, 2.0 ** -126))[1].tolist() == [0]
    bad = np.ones(32)
    bad[7] = np.inf
    assert M.quantize(bad)[1].tolist() == [255] and not M.quantize(bad)[0].any()
    assert np.array_equal(M.unpack(M.pack(code)), code)


def test_sizes_past_what_a_launch_or_an_argument_holds():
    """A plan of more than 2^33 input values (the weighted sum's threads), and sizes that lose their high bits in a
    32-bit argument: 2^32 + 64 must not pass for 64."""
    from trellis_quantized_moe_tmoe_amd import mxfp4, native
    h = ctypes.c_void_p()
    for T, H, want in [(1 << 20, 8192, 0), ((1 << 20) + 1, 8192, 2), (1 << 22, 2048, 0), (1 << 22, 2080, 2)]:
        cfg = native.Mxfp4Config(H, 32, 4, 1, T, native.IDS_I32, native.F32)
        assert native.lib.tmoe_mxfp4_plan(ctypes.byref(cfg), ctypes.byref(h), None) == want
        if want == 0:
            native.lib.tmoe_mxfp4_plan_destroy(h)
    big = 2 ** 32 + 64
    m = lambda *s: torch.empty(*s, dtype=torch.uint8, device="meta")  # noqa: E731
    for bad in [lambda: mxfp4.quantize(torch.empty(1, big, device="meta")),
                lambda: mxfp4.dequantize(m(1, big // 2), m(1, big // 32)),
                lambda: mxfp4.linear(m(big, 32), m(big, 2), m(6, 32), m(6, 2)),
                lambda: mxfp4.linear(m(6, 32), m(6, 2), m(big, 32), m(big, 2)),
                lambda: mxfp4.ExpertPlan(big, 32, 4, 2, 8), lambda: mxfp4.ExpertPlan(64, 32, 4, 2, big)]:
        with pytest.raises(ValueError, match="out of range"):
            bad()
