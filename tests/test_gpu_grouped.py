"""The products grouped by expert and their gradients, bf16, fp16 and MXFP8, against float64 (mxfp8_ref.py) within what
fp32 sums of exact products may round."""
import ctypes

import numpy as np
import pytest
import torch

import mxfp8_ref as M
from gpu_cases import say

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 1e-37, torch.bfloat16: 1e-37, torch.float16: 2.0 ** -25}


def _g():
    from trellis_quantized_moe_tmoe_amd import grouped
    return grouped


def _mx():
    from trellis_quantized_moe_tmoe_amd import mxfp8
    return mxfp8


def _np(t):
    return t.double().cpu().numpy()


def _close(got, ref, s, depth, cut=0.0):
    depth = np.asarray(depth, np.float64)
    bound = M.product_bound(s, depth, ref, HALF[got.dtype], TINY[got.dtype]) + cut * (1 + HALF[got.dtype])
    off = np.abs(_np(got) - ref)
    assert np.all(off <= bound), (float(off.max()), np.argwhere(~(off <= bound))[:4].tolist())


def _offsets(sizes, front=0, back=0):
    off = front + np.concatenate([[0], np.cumsum(sizes)])
    return off, int(off[-1] + back)


class Case:
    """Rows outside every group hold NaN: nothing of them may reach a result."""

    def __init__(self, sizes, K, N, dtype, front=0, back=0, ids=torch.int32, seed=0):
        self.off, self.R = _offsets(sizes, front, back)
        say(f"[case] grouped {sizes if len(sizes) < 12 else len(sizes)} front {front} back {back} K={K} N={N} {dtype}")
        g = torch.Generator().manual_seed(seed + K + 7 * N)
        E = len(sizes)
        self.x, self.dy = torch.randn(self.R, K, generator=g).to(dtype), torch.randn(self.R, N, generator=g).to(dtype)
        self.w = (torch.randn(E, N, K, generator=g) / K ** 0.5).to(dtype)
        self.out = np.r_[0:front, self.off[-1]:self.R]
        self.x[self.out] = float("nan")
        self.dy[self.out] = float("nan")
        self.offsets = torch.tensor(self.off, dtype=ids).cuda()
        self.K, self.N = K, N
        self.cx, self.cdy, self.cw = self.x.cuda(), self.dy.cuda(), self.w.cuda()
        self.nx, self.ndy, self.nw = (np.nan_to_num(_np(t)) for t in (self.x, self.dy, self.w))

    def linear(self, out_dtype=None):
        y = _g().linear(self.cx, self.cw, self.offsets, out_dtype)
        assert y.shape == (self.R, self.N) and y.dtype == (out_dtype or self.x.dtype)
        _close(y, *M.grouped(self.nx, self.nw, self.off), self.K)
        assert torch.all(y[self.out] == 0)

    def grad_x(self, out_dtype=None):
        d = _g().grad_x(self.cdy, self.cw, self.offsets, out_dtype)
        assert d.shape == (self.R, self.K) and d.dtype == (out_dtype or self.x.dtype)
        _close(d, *M.grouped(self.ndy, self.nw.transpose(0, 2, 1), self.off), self.N)
        assert torch.all(d[self.out] == 0)

    def grad_w(self, out_dtype=None):
        d = _g().grad_w(self.cdy, self.cx, self.offsets, out_dtype)
        assert d.shape == self.w.shape and d.dtype == (out_dtype or self.x.dtype)
        _close(d, *M.grouped_grad_w(self.ndy, self.nx, self.off), np.diff(self.off)[:, None, None])
        assert torch.all(d[np.diff(self.off) == 0] == 0)

    def all(self, out_dtype=None):
        self.linear(out_dtype)
        self.grad_x(out_dtype)
        self.grad_w(out_dtype)


FEW = [([1], 8, 8, 0, 0), ([0, 1, 0, 2], 64, 24, 0, 0), ([3, 0, 15, 16, 17, 0, 1, 0], 72, 136, 2, 3),
       ([16, 0, 0, 33], 136, 128, 0, 1), ([1] * 40, 1024, 264, 0, 0), ([0] * 30 + [32, 31, 65], 264, 1000, 5, 0),
       ([0, 0, 0], 128, 64, 1, 2), ([2, 5], 2560, 640, 0, 0)]
MID = [([17], 8, 8, 0, 0), ([127, 128, 129, 0, 1], 64, 128, 3, 130), ([300, 31], 72, 136, 0, 0), ([63, 64, 65, 66], 200, 8, 129, 0),
       ([500], 1000, 264, 0, 7), ([33, 257, 0, 96], 256, 392, 1, 1), ([200, 1, 90], 520, 1032, 0, 0)]
BIG = [([1024], 64, 256, 0, 0), ([1030], 136, 264, 3, 0), ([2100, 7], 72, 520, 0, 300), ([1, 0, 3500], 328, 136, 0, 0)]


@pytest.mark.parametrize("sizes,K,N,front,back", FEW + MID + BIG)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_product_and_gradients(sizes, K, N, front, back, dtype):
    Case(sizes, K, N, dtype, front, back).all()


@pytest.mark.parametrize("sizes,K,N,front,back", [FEW[2], FEW[5], MID[1], MID[4], BIG[1]])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_fp32_results_and_64_bit_offsets(sizes, K, N, front, back, dtype):
    Case(sizes, K, N, dtype, front, back, ids=torch.int64).all(torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_256_x_256_tiles(dtype):
    """Rows and outputs large enough for the largest tiles: odd depths, short last tiles, rows outside, both output types."""
    for out in (None, torch.float32):
        Case([700, 0, 341], 200, 10008, dtype, 3, 300).linear(out)
        Case([513], 8, 16392, dtype).linear(out)
        Case([700, 0, 341], 10008, 136, dtype, 3, 300).grad_x(out)
        Case([513], 16392, 72, dtype).grad_x(out)
        Case([700, 331], 2312, 2568, dtype, 5, 9).grad_w(out)
        Case([1100, 0, 37, 950], 1800, 1544, dtype).grad_w(out)


def test_popular_experts_first():
    """grad_w takes experts with more than three times the average first: none, one, as many as there can be, and the last one."""
    for sizes in ([40] * 9, [1200] + [0] * 30, [0] * 40 + [1500], [300, 0, 0, 0] * 8 + [1], [0, 0, 0, 900, 4, 4, 4, 700] * 3,
                  [33] * 65 + [3000] + [20] * 70):
        Case(sizes, 136, 72, torch.bfloat16, 1, 1).grad_w()


def test_many_experts():
    rng = np.random.default_rng(1)
    for E, top in ((511, 3), (512, 60), (300, 9)):
        Case(list(rng.integers(0, top, E)), 64, 40, torch.bfloat16, 1, 2).all()


def test_no_rows():
    g = _g()
    for R in (0, 5):
        x, w = torch.ones(R, 64, device="cuda").half(), torch.ones(3, 16, 64, device="cuda").half()
        off = torch.zeros(4, dtype=torch.int32, device="cuda")
        dy = torch.ones(R, 16, device="cuda").half()
        assert torch.equal(g.linear(x, w, off), torch.zeros(R, 16, device="cuda").half())
        assert torch.equal(g.grad_x(dy, w, off), torch.zeros_like(x)) and torch.equal(g.grad_w(dy, x, off), torch.zeros_like(w))


def test_infinities_stay_in_their_rows():
    c = Case([40, 30], 72, 24, torch.bfloat16)
    c.cx[3, 5] = float("inf")
    c.cx[50, 71] = float("nan")
    c.cw[0, 7, 11] = -float("inf")
    y = _np(_g().linear(c.cx, c.cw, c.offsets))
    ref = M.grouped(_np(c.cx), _np(c.cw), c.off)[0]
    assert np.array_equal(np.isfinite(y), np.isfinite(ref))
    clean = np.isfinite(ref)
    assert np.abs(y - ref)[clean].max() < 0.05


def test_offsets_outside_the_rows_stay_inside_the_arrays():
    """Offsets past the rows are cut at the last one, negative ones at the first."""
    g = _g()
    c = Case([30, 34], 64, 16, torch.bfloat16)
    bad = torch.tensor([-5, 30, 900], dtype=torch.int32, device="cuda")
    assert torch.equal(g.linear(c.cx, c.cw, bad), g.linear(c.cx, c.cw, c.offsets))
    assert torch.equal(g.grad_w(c.cdy, c.cx, bad), g.grad_w(c.cdy, c.cx, c.offsets))


def test_nothing_behind_the_outputs_is_written():
    from trellis_quantized_moe_tmoe_amd import native as n
    c = Case([5, 40, 0, 12], 72, 40, torch.bfloat16, 1, 2)
    cfg = ctypes.byref(n.GroupedConfig(4, 72, 40, n.BF16, n.BF16, n.IDS_I32))
    for fn, r, cc, shape in ((n.lib.tmoe_grouped_linear, c.cx, c.cw, (c.R, 40)), (n.lib.tmoe_grouped_grad_x, c.cdy, c.cw, (c.R, 72)),
                             (n.lib.tmoe_grouped_grad_w, c.cdy, c.cx, (4, 40, 72))):
        size = int(np.prod(shape))
        buf = torch.full((size + 4096,), 77.0, dtype=torch.bfloat16, device="cuda")
        assert fn(cfg, r.data_ptr(), cc.data_ptr(), c.offsets.data_ptr(), c.R, buf.data_ptr(), torch.cuda.current_stream().cuda_stream) == 0
        torch.cuda.synchronize()
        assert torch.all(buf[size:] == 77.0) and torch.isfinite(buf[:size]).all()


@pytest.mark.parametrize("E", [2, 200])
def test_rows_beyond_32_bits_of_bytes(E):
    """x of more than 4 GiB (rows far behind) and the last expert's weights far behind."""
    g = _g()
    R, K, N = 700001, 4096, 16
    x = torch.empty(R, K, dtype=torch.bfloat16, device="cuda")
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    last = 300
    x[-last:] = torch.randn(last, K, generator=gen, device="cuda").bfloat16()
    x[:last] = 1.0
    w[-1] = (torch.randn(N, K, generator=gen, device="cuda") / 64).bfloat16()
    off = torch.full((E + 1,), R - last, dtype=torch.int64, device="cuda")
    off[-1] = R
    y = g.linear(x, w, off)
    ref = x[-last:].double() @ w[-1].double().t()
    s = x[-last:].double().abs() @ w[-1].double().abs().t()
    _close(y[-last:], _np(ref), _np(s), K)
    assert torch.all(y[:-last] == 0)
    dw = g.grad_w(y, x, off)
    ref = y[-last:].double().t() @ x[-last:].double()
    s = y[-last:].double().abs().t() @ x[-last:].double().abs()
    _close(dw[-1], _np(ref), _np(s), last)
    assert torch.all(dw[:-1] == 0)
    dx = g.grad_x(y, w, off)
    ref, s = y[-last:].double() @ w[-1].double(), y[-last:].double().abs() @ w[-1].double().abs()
    _close(dx[-last:], _np(ref), _np(s), N)
    assert torch.all(dx[: R - last].view(torch.int16).amax() == 0)


def test_weights_beyond_32_bits_of_bytes():
    """w and dw of more than 4 GiB: only the last expert has rows, only its weights are read."""
    g = _g()
    E, N, K, R = 270, 2048, 4096, 9
    w = torch.empty(E, N, K, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(1)
    w[-1] = (torch.randn(N, K, generator=gen, device="cuda") / 64).bfloat16()
    w[:-1].fill_(float("nan"))
    x = torch.randn(R, K, generator=gen, device="cuda").bfloat16()
    off = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    off[-1] = R
    y = g.linear(x, w, off)
    _close(y, _np(x.double() @ w[-1].double().t()), _np(x.double().abs() @ w[-1].double().abs().t()), K)
    dx = g.grad_x(y, w, off)
    _close(dx, _np(y.double() @ w[-1].double()), _np(y.double().abs() @ w[-1].double().abs()), N)
    del w
    dw = g.grad_w(y, x, off)
    _close(dw[-1], _np(y.double().t() @ x.double()), _np(y.double().abs().t() @ x.double().abs()), R)
    assert int(dw[:-1].view(torch.int16).count_nonzero()) == 0


def test_autograd():
    g = _g()
    for dtype, out in ((torch.bfloat16, None), (torch.float16, torch.float32)):
        c = Case([20, 0, 45], 64, 24, dtype)
        x, w = c.cx.clone().requires_grad_(), c.cw.clone().requires_grad_()
        y = g.linear(x, w, c.offsets, out)
        y.backward(c.cdy.to(y.dtype))
        assert torch.equal(x.grad, g.grad_x(c.cdy, c.cw, c.offsets)) and torch.equal(w.grad, g.grad_w(c.cdy, c.cx, c.offsets))
        x.grad = None
        g.linear(x, c.cw, c.offsets, out).sum().backward()           # an expanded gradient, the weights not tracked
        assert torch.equal(x.grad, g.grad_x(torch.ones_like(c.cdy), c.cw, c.offsets))
        w.grad = None
        g.linear(c.cx, w, c.offsets, out).backward(c.cdy.to(y.dtype).t().contiguous().t())   # a transposed one
        assert torch.equal(w.grad, g.grad_w(c.cdy, c.cx, c.offsets))


def test_gradients_against_differences():
    """Central differences of sum(y * dy) along random directions: y is linear in x and in w, so they are exact up to y's
    own rounding to fp32 (2^-24 relative, and its sums')."""
    g = _g()
    c = Case([9, 0, 30], 64, 32, torch.float16)
    d = torch.randn(c.x.shape, generator=torch.Generator().manual_seed(5)).half().cuda()
    dw = torch.randn(c.w.shape, generator=torch.Generator().manual_seed(6)).half().cuda()
    f = lambda x, w: (g.linear(x, w, c.offsets, torch.float32).double() * c.cdy.double()).sum()  # noqa: E731
    for got, plus, minus, along in (
            (g.grad_x(c.cdy, c.cw, c.offsets, torch.float32), (c.cx + d, c.cw), (c.cx - d, c.cw), (c.cx + d).double() - (c.cx - d).double()),
            (g.grad_w(c.cdy, c.cx, c.offsets, torch.float32), (c.cx, c.cw + dw), (c.cx, c.cw - dw), (c.cw + dw).double() - (c.cw - dw).double())):
        want = (got.double() * along).sum()
        assert abs(float(f(*plus) - f(*minus) - want)) <= 1e-4 * float((got.double() * along).abs().sum())


def test_saved_operands_that_change():
    """A backward that saved x, w or the offsets does not run on values written since."""
    g = _g()
    c = Case([9, 3], 64, 16, torch.bfloat16)
    for which in range(3):
        x, w, off = c.cx.clone().requires_grad_(), c.cw.clone().requires_grad_(), c.offsets.clone()
        y = g.linear(x, w, off)
        with torch.no_grad():
            (x, w, off)[which].zero_()
        with pytest.raises(RuntimeError, match="inplace"):
            y.sum().backward()


def test_two_streams_at_once():
    g = _g()
    a, b = Case([100, 30], 520, 392, torch.bfloat16), Case([7, 0, 200], 136, 1032, torch.float16)
    want = [g.linear(c.cx, c.cw, c.offsets) for c in (a, b)] + [g.grad_w(c.cdy, c.cx, c.offsets) for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(5):
        for c, s in zip((a, b), streams):
            with torch.cuda.stream(s):
                got.append((c, g.linear(c.cx, c.cw, c.offsets), g.grad_w(c.cdy, c.cx, c.offsets)))
    torch.cuda.synchronize()
    for c, y, dw in got:
        i = 0 if c is a else 1
        assert torch.equal(y.nan_to_num(), want[i].nan_to_num()) and torch.equal(dw, want[2 + i])


def test_repeatable_other_stream_and_graph():
    g = _g()
    rng = np.random.default_rng(3)
    c = Case(list(rng.integers(0, 90, 24)), 264, 200, torch.bfloat16, 2, 3)

    def step():
        return g.linear(c.cx, c.cw, c.offsets), g.grad_x(c.cdy, c.cw, c.offsets), g.grad_w(c.cdy, c.cx, c.offsets)
    a = step()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(4):                        # other rows and other groups
        c.cx.copy_(torch.randn(c.x.shape, generator=torch.Generator().manual_seed(seed)).bfloat16())
        c.cdy.copy_(torch.randn(c.dy.shape, generator=torch.Generator().manual_seed(seed + 9)).bfloat16())
        cut = np.sort(rng.integers(0, c.R + 1, len(c.off)))
        c.offsets.copy_(torch.tensor(cut, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


# ---------------------------------------------------------------- MXFP8 operands

@pytest.mark.parametrize("sizes,N,front,back", [(s, n, f, b) for s, _, n, f, b in FEW + MID + BIG])
@pytest.mark.parametrize("K", [32, 128, 160, 640])
def test_mxfp8(sizes, N, front, back, K):
    off, R = _offsets(sizes, front, back)
    say(f"[case] grouped mxfp8 {sizes if len(sizes) < 12 else len(sizes)} front {front} back {back} K={K} N={N}")
    rng = np.random.default_rng(K + N)
    E = len(sizes)
    x = rng.normal(size=(R, K)) * np.exp(rng.normal(size=(R, 1)))
    w = rng.normal(size=(E, N, K)) / np.sqrt(K) * np.exp(rng.normal(size=(E, N, 1)))
    (xq, xs), (wq, ws) = M.quantize(x), M.quantize(w)
    vx, vw = M.values(xq, xs), M.values(wq, ws)
    out = np.r_[0:front, off[-1]:R]
    xs[out] = 255                                # NaN outside the groups
    gpu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    ref, s = M.grouped(vx, vw, off)
    cut, px, pw = np.zeros((R, N)), M.powers(xq, np.minimum(xs, 254)), M.powers(wq, ws)
    for e in range(E):
        cut[off[e]:off[e + 1]] = M.cut_bound(px[off[e]:off[e + 1]], pw[e])
    for dt in (torch.bfloat16, torch.float32):
        y = _mx().grouped_linear(gpu(xq), gpu(xs), gpu(wq), gpu(ws), gpu(off), dt)
        assert y.shape == (R, N) and y.dtype == dt
        _close(y, ref, s, K, cut)
        assert torch.all(y[out] == 0)


def test_mxfp8_256_x_256_tiles():
    off, R = _offsets([1100, 0, 700], 3, 9)
    for K, N in ((4096, 8200), (4224, 7944), (512, 10008)):
        gen = torch.Generator(device="cuda").manual_seed(K)
        (xq, xs), (wq, ws) = (_mx().quantize(torch.randn(*s, generator=gen, device="cuda")) for s in ((R, K), (3, N, K)))
        y = _mx().grouped_linear(xq, xs, wq, ws, torch.from_numpy(off).cuda(), torch.float32)
        x, w = _mx().dequantize(xq, xs).double(), _mx().dequantize(wq, ws).double()
        px, pw = (torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -40)))) for t in (x, w))
        for e in (0, 2):
            a, b = int(off[e]), int(off[e + 1])
            ref, s = x[a:b] @ w[e].t(), x[a:b].abs() @ w[e].abs().t()
            # the cut of 16 products is at most 2^-9 of their largest, which is at most the sum of all (mxfp8_ref.cut_bound)
            bound = 2 * M.U * (K + 4) * s + 2.0 ** -9 * (px[a:b] @ pw[e].t())
            assert bool(((y[a:b].double() - ref).abs() <= bound).all())
        assert torch.all(y[:3] == 0) and torch.all(y[-9:] == 0)


@pytest.mark.parametrize("sizes,K,N", [([1, 0, 40], 32, 24), ([30, 2, 70], 96, 136), ([500], 1088, 264), ([2000, 9], 640, 72), ([1040], 640, 10008), ([540], 4224, 16392)])
def test_mxfp8_products_of_one_size_are_exact(sizes, K, N):
    """Values 1, 2 and 3 times a power of two by blocks: nothing is cut and every sum fits fp32, so every product counts."""
    off, R = _offsets(sizes)
    rng = np.random.default_rng(K)
    E = len(sizes)

    def draw(*shape):
        codes = rng.choice(np.array([0x38, 0x40, 0x44, 0xB8, 0xC0, 0xC4, 0], np.uint8), size=shape)
        return codes, (127 + rng.integers(0, 3, size=(*shape[:-1], shape[-1] // 32))).astype(np.uint8)
    (xq, xs), (wq, ws) = draw(R, K), draw(E, N, K)
    gpu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    y = _mx().grouped_linear(gpu(xq), gpu(xs), gpu(wq), gpu(ws), gpu(off), torch.float32)
    assert np.array_equal(_np(y), M.grouped(M.values(xq, xs), M.values(wq, ws), off)[0])


def test_mxfp8_scales_of_infinity_and_odd_addresses():
    off, R = _offsets([40, 5])
    rng = np.random.default_rng(4)
    (xq, xs), (wq, ws) = M.quantize(rng.normal(size=(R, 256))), M.quantize(rng.normal(size=(2, 24, 256)))
    gpu = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
    y = _mx().grouped_linear(gpu(xq), gpu(xs), gpu(wq), gpu(ws), gpu(off), torch.float32)
    # scales that start at an odd byte take the byte loads: the same values
    ox, ow = torch.zeros(xs.size + 1, dtype=torch.uint8, device="cuda"), torch.zeros(ws.size + 3, dtype=torch.uint8, device="cuda")
    ox[1:], ow[3:] = gpu(xs).flatten(), gpu(ws).flatten()
    z = _mx().grouped_linear(gpu(xq), ox[1:].view(xs.shape), gpu(wq), ow[3:].view(ws.shape), gpu(off), torch.float32)
    assert torch.equal(y, z)
    xs[7, 3], ws[1, 5, 0] = 255, 255
    y = _np(_mx().grouped_linear(gpu(xq), gpu(xs), gpu(wq), gpu(ws), gpu(off), torch.float32))
    want = np.zeros((R, 24), bool)
    want[7] = want[40:, 5] = True
    assert np.array_equal(np.isnan(y), want)


# ---------------------------------------------------------------- as they are used together

def _route(ids, E):
    flat = ids.flatten() + 1
    return torch.sort(flat, stable=True).indices, torch.bincount(flat, minlength=E + 1).cumsum(0)


def test_a_trained_layer():
    """norm -> router -> grouped products -> weighted sum, and its gradients, against the same layer in float64."""
    from trellis_quantized_moe_tmoe_amd import norm, router
    T, H, I, E, k = 61, 64, 48, 7, 2
    gen = torch.Generator().manual_seed(11)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    p = dict(x=rnd(T, H), res=rnd(T, H), g=1 + 0.1 * rnd(H), wr=rnd(E, H) / 8, w1=rnd(E, 2 * I, H) / 8, w2=rnd(E, H, I) / 7)
    p = {n: (t.half().float() if n != "wr" else t) for n, t in p.items()}
    mask = torch.arange(T) % 13 != 5
    dy = rnd(T, H).half()

    def layer(own, d):
        if own:
            n, h, _ = norm.rms_norm(d["x"].half(), d["g"].half(), d["res"].half())
            ids, w, _ = router.topk(n.float() @ d["wr"].t(), k, token_mask=mask.cuda())
            route, off = _route(ids, E)
            z = _g().linear(n[route // k], d["w1"].half(), off)
            a = torch.nn.functional.silu(z[:, :I].float()) * z[:, I:].float()
            v = _g().linear(a.half(), d["w2"].half(), off)
            out = torch.zeros(T, H, device="cuda").index_add_(0, route // k, v.float() * w.flatten()[route, None])
            return (h.float() + out) * dy.cuda().float(), ids
        h = d["x"] + d["res"]
        n = h / torch.sqrt((h * h).mean(-1, keepdim=True) + 1e-6) * d["g"]
        l = n @ d["wr"].t()
        w, i = l.topk(k, dim=1)
        w = torch.softmax(w, 1) * mask[:, None]
        out = torch.zeros_like(h)
        for e in range(E):
            z = n @ d["w1"][e].t()
            v = (torch.nn.functional.silu(z[:, :I]) * z[:, I:]) @ d["w2"][e].t()
            out = out + (w * (i == e)).sum(1, keepdim=True) * v
        return (h + out) * dy.double(), i

    a = {n: t.cuda().requires_grad_() for n, t in p.items()}
    b = {n: t.double().requires_grad_() for n, t in p.items()}
    ya, ia = layer(True, a)
    yb, ib = layer(False, b)
    assert torch.equal(ia.cpu()[mask], ib[mask]) and torch.all(ia[~mask.cuda()] == -1)
    ya.sum().backward()
    yb.sum().backward()
    # fp16 roundings of the values between the operators (at most 8 on a path, 2^-11 each) on sums of at most H values
    # of either sign: within 2 % of the largest gradient
    assert float((ya.double().cpu() - yb).abs().max()) <= 0.02 * float(yb.abs().max())
    for n in p:
        assert float((a[n].grad.double().cpu() - b[n].grad).abs().max()) <= 0.02 * float(b[n].grad.abs().max()), n


def test_a_served_layer_in_8_bits():
    """norm in MXFP8 -> grouped product: what the same rows give through quantize, at every batch size from one token."""
    from trellis_quantized_moe_tmoe_amd import norm
    H, N, E = 128, 72, 5
    gen = torch.Generator().manual_seed(2)
    w = torch.randn(E, N, H, generator=gen).bfloat16().cuda()
    wq, ws = _mx().quantize(w)
    g = torch.ones(H, dtype=torch.bfloat16, device="cuda")
    full = torch.randn(500, H, generator=gen).bfloat16().cuda()
    for T in (1, 3, 40, 500):
        ids = torch.randint(0, E, (T,), generator=gen)
        route, off = _route(ids, E)
        route, off = route.cuda(), off.cuda()
        codes, scales, _ = norm.rms_norm_mxfp8(full[:T][route], g)
        y = _mx().grouped_linear(codes, scales, wq, ws, off)
        xq, xs, nq, ns, o = (t.cpu().numpy() for t in (codes, scales, wq, ws, off))
        cut = np.concatenate([M.cut_bound(M.powers(xq, xs)[o[e]:o[e + 1]], M.powers(nq, ns)[e]) for e in range(E)])
        _close(y, *M.grouped(M.values(xq, xs), M.values(nq, ns), o), H, cut)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes,K,N", [([7 * i % 37 for i in range(64)], 264, 520), ([7 * i % 37 for i in range(64)], 1000, 136),
                                       ([11 * i % 199 for i in range(32)], 72, 1032), ([11 * i % 199 for i in range(32)], 1160, 40),
                                       ([300, 0] + [150] * 38, 72, 1800), ([300, 0] + [150] * 38, 1800, 72)])
def test_weights_that_are_read_once(sizes, K, N, dtype):
    """Many experts of about one row tile each: 32, 128 and 256 rows."""
    Case(sizes, K, N, dtype, 3, 40).all()
    Case(sizes, K, N, dtype, 0, 0).linear(torch.float32)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_weight_gradients_of_few_rows_beyond_the_caches(dtype):
    """Few rows an expert, and more bytes of dw than the memory-side cache holds."""
    say(f"[case] grad_w beyond the caches {dtype}")
    E, N, K = 130, 1032, 1024
    off, R = _offsets([0, 5] * (E // 2 - 1) + [3, 70], 2, 1)
    gen = torch.Generator(device="cuda").manual_seed(5)
    x, dy = (torch.randn(R, n, generator=gen, device="cuda").to(dtype) for n in (K, N))
    offsets = torch.tensor(off, dtype=torch.int32).cuda()
    assert E * N * K * 2 > 256 << 20
    dw = _g().grad_w(dy, x, offsets)
    for e in (1, 65, E - 2, E - 1):
        a, b = dy[off[e]:off[e + 1]].double().t(), x[off[e]:off[e + 1]].double()
        _close(dw[e], _np(a @ b), _np(a.abs() @ b.abs()), off[e + 1] - off[e])
    assert torch.all(dw[0:E - 2:2] == 0)


def _spread_sizes(E, sizes, rest):
    """E groups: `sizes` by index, `rest` in the others."""
    return [sizes.get(e, rest) for e in range(E)]


# sizes, how many of the experts have more than three times the average, K, N
POPULAR = [([65] * 9, 0, 136, 72),
           ([2700] + [0] * 40, 1, 136, 72),
           ([0] * 40 + [2700], 1, 136, 72),
           (_spread_sizes(33, {e: 220 for e in range(0, 30, 3)}, 0), 10, 136, 72),         # as many as there can be: (E - 1) / 3
           (_spread_sizes(33, {e: 220 for e in range(23, 33)}, 0), 10, 40, 264),
           (_spread_sizes(136, {63: 2100, 64: 2107, 130: 2200}, 20), 3, 136, 72),          # on both sides of 64, and in the third 64
           (_spread_sizes(512, {0: 5000, 447: 5003, 448: 4999, 450: 5000, 511: 5001}, 16), 5, 72, 136),
           (_spread_sizes(200, {e: 350 for e in range(130, 196)}, 0), 66, 8, 24),          # as many as there can be, behind the second 64
           ([100, 0, 2400, 60, 30], 1, 1544, 1800),                                        # 256 x 256 tiles
           ([1700, 10, 0, 1750, 20, 100, 30], 2, 1544, 1800)]


@pytest.mark.parametrize("sizes,popular,K,N", POPULAR)
def test_popular_experts_come_first_and_are_all_written(sizes, popular, K, N):
    """grad_w looks popular experts up from 64 rows an expert on; every value of a result that held NaN is written."""
    from trellis_quantized_moe_tmoe_amd import native as n
    c = Case(sizes, K, N, torch.bfloat16)
    E, R = len(sizes), c.R
    assert R >= 64 * E and sum(s * E > 3 * R for s in sizes) == popular <= (E - 1) // 3
    if K > 1024:
        assert R >= 512 * E and -(-K // 256) * -(-N // 256) * E >= 192
    dw = torch.full((E, N, K), float("nan"), dtype=torch.bfloat16, device="cuda")
    cfg = ctypes.byref(n.GroupedConfig(E, K, N, n.BF16, n.BF16, n.IDS_I32))
    assert n.lib.tmoe_grouped_grad_w(cfg, c.cdy.data_ptr(), c.cx.data_ptr(), c.offsets.data_ptr(), R, dw.data_ptr(),
                                     torch.cuda.current_stream().cuda_stream) == 0
    _close(dw, *M.grouped_grad_w(c.ndy, c.nx, c.off), np.diff(c.off)[:, None, None])
    assert torch.all(dw[np.diff(c.off) == 0] == 0)


def test_operands_that_no_gradient_reads_are_not_saved():
    """dx reads w and dW reads x: with one operand tracked the other's gradient is nobody's, so the tracked one may change, or go."""
    g = _g()
    c = Case([9, 0, 30], 64, 32, torch.bfloat16)
    other = torch.randn(c.x.shape, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    x = c.cx.clone().requires_grad_()             # frozen experts
    y = g.linear(x, c.cw, c.offsets)
    with torch.no_grad():
        x.copy_(other)
    y.backward(c.cdy)
    assert torch.equal(x.grad, g.grad_x(c.cdy, c.cw, c.offsets))
    w = c.cw.clone().requires_grad_()             # an input that nothing lies behind
    y = g.linear(c.cx, w, c.offsets)
    with torch.no_grad():
        w.zero_()
    y.backward(c.cdy)
    assert torch.equal(w.grad, g.grad_w(c.cdy, c.cx, c.offsets))
    # what is read is still guarded
    for x, w, change in ((c.cx.clone().requires_grad_(), c.cw.clone(), 1), (c.cx.clone(), c.cw.clone().requires_grad_(), 0),
                         (c.cx.clone().requires_grad_(), c.cw.clone(), 2), (c.cx.clone(), c.cw.clone().requires_grad_(), 2)):
        off = c.offsets.clone()
        y = g.linear(x, w, off)
        with torch.no_grad():
            (x, w, off)[change].zero_()
        with pytest.raises(RuntimeError, match="inplace"):
            y.backward(c.cdy)
    # and its memory is given back
    leaf, off = torch.zeros(1 << 20, 16, dtype=torch.bfloat16, device="cuda", requires_grad=True), torch.tensor([0, 1 << 20], device="cuda")
    w = torch.ones(1, 8, 16, dtype=torch.bfloat16, device="cuda")
    x = leaf + 1
    y = g.linear(x, w, off)
    before = torch.cuda.memory_allocated()
    del x
    assert torch.cuda.memory_allocated() <= before - (32 << 20)
    y.sum().backward()
    assert torch.all(leaf.grad == 8)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_a_gradient_that_arrives_at_an_odd_address(dtype):
    """The gradient of a concatenation is a part of a larger one: contiguous, but not aligned to the products' 16 bytes."""
    g = _g()
    c = Case([20, 0, 45], 64, 24, dtype)
    for lead in (1, 3, 4):
        x, w = c.cx.clone().requires_grad_(), c.cw.clone().requires_grad_()
        y = g.linear(x, w, c.offsets)
        head = torch.zeros(lead, dtype=dtype, device="cuda")
        torch.cat([head, y.flatten()]).backward(torch.cat([head, c.cdy.flatten()]))
        assert torch.equal(x.grad, g.grad_x(c.cdy, c.cw, c.offsets)) and torch.equal(w.grad, g.grad_w(c.cdy, c.cx, c.offsets))


def test_sizes_are_refused_before_outputs_are_allocated():
    """Outputs that no card holds: the library's refusal, not the allocator's."""
    from trellis_quantized_moe_tmoe_amd.native import TmoeError
    z = lambda *s: torch.zeros(*s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    u8 = lambda *s: torch.zeros(*s, dtype=torch.uint8, device="cuda")  # noqa: E731
    off, R = torch.zeros(2, dtype=torch.int32, device="cuda"), 1 << 22
    for call in (lambda: _g().linear(z(R, 8), z(1, 65544, 8), off), lambda: _g().grad_x(z(R, 8), z(1, 8, 65544), off),
                 lambda: _g().grad_w(z(4, 65544), z(4, 65544), torch.zeros(513, dtype=torch.int32, device="cuda")),
                 lambda: _mx().grouped_linear(u8(R, 32), u8(R, 1), u8(1, 65544, 32), u8(1, 65544, 1), off)):
        with pytest.raises(TmoeError, match="UNSUPPORTED"):
            call()
