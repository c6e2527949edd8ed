"""MXFP4 kernels against the float64 reference (mxfp4_ref.py): codes, scales and values bit for bit, products
within what fp32 sums may round (mxfp4_ref.product_slack), the layer within its reference's own bound."""
import numpy as np
import pytest
import torch

import mxfp4_ref as M
from gpu_cases import say

pytestmark = pytest.mark.gpu

HALF = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def _mx():
    from trellis_quantized_moe_tmoe_amd import mxfp4
    return mxfp4


def _gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _check_codes(x):
    """x: a CPU tensor. Codes, scales and values of the kernels against the reference."""
    codes, scales = _mx().quantize(x.cuda())
    want, s = M.quantize(x.double().numpy())
    assert np.array_equal(scales.cpu().numpy(), s)
    assert np.array_equal(codes.cpu().numpy(), M.pack(want))
    v = M.values(want, s)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        got = _mx().dequantize(codes, scales, dt)
        assert got.dtype == dt
        ref = torch.from_numpy(v).to(torch.float32).to(dt)
        assert torch.equal(got.cpu().nan_to_num(7.0, 8.0, 9.0), ref.nan_to_num(7.0, 8.0, 9.0))


@pytest.mark.parametrize("rows,cols", [(1, 32), (3, 96), (17, 1024), (1000, 160), (2, 8192), (5, 4128)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_quantize_bit_for_bit(rows, cols, dtype):
    say(f"[case] quantize {rows}x{cols} {dtype}")
    rng = np.random.default_rng(rows + cols)
    x = rng.normal(size=(rows, cols)) * np.exp(rng.normal(size=(rows, 1)) * 3)
    x[rng.random((rows, cols)) < 0.02] *= 30
    x[rng.random((rows, cols)) < 0.1] = 0.0
    _check_codes(torch.from_numpy(x).to(dtype))


def test_quantize_borders_and_extremes():
    vals = np.concatenate([M.BORDERS, M.MAGS])
    near = np.concatenate([vals, np.nextafter(vals.astype(np.float32), np.float32(9)),
                           np.nextafter(vals.astype(np.float32), np.float32(-9))])
    near = np.concatenate([near, -near]).astype(np.float32)
    rows = []
    for e in (-140, -127, -126, -125, -100, -1, 0, 1, 60, 124, 125):
        for top in (6.0, 4.5, 3.1, 6.0000005):
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
    scales = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    v = M.values(M.unpack(codes), scales)
    for dt in (torch.float32, torch.bfloat16, torch.float16):
        got = _mx().dequantize(_gpu(codes), _gpu(scales), dt).cpu()
        with np.errstate(over="ignore"):
            ref = torch.from_numpy(v.astype(np.float32)).to(dt)
        assert torch.equal(got.nan_to_num(7.0, 8.0, 9.0), ref.nan_to_num(7.0, 8.0, 9.0))


def test_quantize_leading_dimensions_and_no_rows():
    x = torch.randn(2, 3, 64)
    codes, scales = _mx().quantize(x.cuda())
    assert codes.shape == (2, 3, 32) and scales.shape == (2, 3, 2)
    assert np.array_equal(codes.cpu().numpy(), M.pack(M.quantize(x.double().numpy())[0]))
    codes, scales = _mx().quantize(torch.zeros(0, 64, device="cuda"))
    assert codes.shape == (0, 32) and _mx().dequantize(codes, scales).shape == (0, 64)


LINEAR = [(1, 32, 1), (1, 4096, 64), (2, 64, 3), (15, 96, 17), (16, 128, 63), (17, 160, 64), (31, 2560, 65), (33, 416, 300),
          (64, 512, 257), (65, 1024, 128), (130, 288, 320), (200, 4128, 100), (513, 320, 1111), (300, 1024, 512)]


@pytest.mark.parametrize("T,K,N", LINEAR)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear(T, K, N, dtype):
    say(f"[case] linear T={T} K={K} N={N} {dtype}")
    rng = np.random.default_rng(T * 7 + K + N)
    xq, xs, x = M.random_operand(rng, T, K)
    wq, ws, w = M.random_operand(rng, N, K, 0.05)
    y = torch.full((T, N), float("nan"), dtype=dtype, device="cuda")
    got = _mx().linear(_gpu(xq), _gpu(xs), _gpu(wq), _gpu(ws), out_dtype=dtype, y=y)
    assert got is y
    ref = x @ w.T
    bound = M.product_slack(K) * (np.abs(x) @ np.abs(w).T)
    err = np.abs(y.double().cpu().numpy() - ref)
    assert np.all(err <= bound + HALF[dtype] * (np.abs(ref) + bound)), float((err / (bound + 1e-30)).max())


@pytest.mark.parametrize("T,K,N", [(2000, 160, 2100), (2049, 544, 1800), (1793, 640, 2305), (2048, 512, 2048),
                                   (1900, 1152, 2100), (4100, 96, 1030), (2048, 2080, 2048)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_linear_many_rows_and_columns(T, K, N, dtype):
    test_linear(T, K, N, dtype)


def test_linear_unaligned_scales():
    """Scales of a K that is a multiple of 128, but not at a 4-byte address."""
    rng = np.random.default_rng(3)
    T, K, N = 2048, 640, 2048
    xq, xs, x = M.random_operand(rng, T, K)
    wq, ws, w = M.random_operand(rng, N, K)
    odd = torch.empty(T * K // 32 + 1, dtype=torch.uint8, device="cuda")
    odd[1:] = _gpu(xs).flatten()
    y = _mx().linear(_gpu(xq), odd[1:].view(T, K // 32), _gpu(wq), _gpu(ws)).cpu().numpy()
    assert np.all(np.abs(y - x @ w.T) <= M.product_slack(K) * (np.abs(x) @ np.abs(w).T))


@pytest.mark.parametrize("T", [1, 16, 40, 300, 2300])
def test_linear_operand_layout_is_exact(T):
    """Small whole numbers times powers of two: every sum is exact, so a value in a wrong place shows."""
    rng = np.random.default_rng(T)
    K, N = 288, 96 if T < 1000 else 2000
    code = rng.integers(0, 16, size=(T, K)).astype(np.uint8)
    xs = rng.integers(124, 131, size=(T, K // 32)).astype(np.uint8)
    wcode = rng.integers(0, 16, size=(N, K)).astype(np.uint8)
    ws = rng.integers(125, 130, size=(N, K // 32)).astype(np.uint8)
    y = _mx().linear(_gpu(M.pack(code)), _gpu(xs), _gpu(M.pack(wcode)), _gpu(ws))
    assert np.array_equal(y.double().cpu().numpy(), M.values(code, xs) @ M.values(wcode, ws).T)


def test_linear_nan_scales_and_extreme_scales():
    rng = np.random.default_rng(1)
    xq, xs, x = M.random_operand(rng, 20, 256)
    wq, ws, w = M.random_operand(rng, 40, 256)
    xs[3, 5], ws[7, 0] = 255, 255
    y = _mx().linear(_gpu(xq), _gpu(xs), _gpu(wq), _gpu(ws)).cpu().numpy()
    nan = np.zeros((20, 40), bool)
    nan[3], nan[:, 7] = True, True
    assert np.array_equal(np.isnan(y), nan)
    code = np.full((1, 32), 7, np.uint8)                # 32 * 36 * 2^-127 * 2^126 and the largest finite pair
    for a, b in ((0, 253), (254, 0), (1, 252)):
        y = _mx().linear(_gpu(M.pack(code)), _gpu(np.array([[a]], np.uint8)), _gpu(M.pack(code)),
                         _gpu(np.array([[b]], np.uint8)))
        assert float(y) == 32 * 36 * 2.0 ** (a + b - 254)


def test_linear_no_tokens_and_neighbours_untouched():
    mx = _mx()
    wq, ws, _ = M.random_operand(np.random.default_rng(0), 30, 64)
    y = mx.linear(torch.empty(0, 32, dtype=torch.uint8, device="cuda"), torch.empty(0, 2, dtype=torch.uint8, device="cuda"),
                  _gpu(wq), _gpu(ws))
    assert y.shape == (0, 30)
    for T in (3, 70):
        xq, xs, _ = M.random_operand(np.random.default_rng(T), T, 64)
        whole = torch.full((T + 2, 30 * 2), 5.0, device="cuda")
        flat = whole.view(-1)[60:60 + T * 30].view(T, 30)       # 240 bytes in: 16-byte aligned
        mx.linear(_gpu(xq), _gpu(xs), _gpu(wq), _gpu(ws), y=flat)
        assert torch.all(whole.view(-1)[:60] == 5.0) and torch.all(whole.view(-1)[60 + T * 30:] == 5.0)


# ---------------------------------------------------------------- the expert layer

class Layer:
    def __init__(self, T, H, I, E, k, seed=0, ids_dtype=torch.int64, out_dtype=torch.float32, skew=False, drop=0.0,
                 max_tokens=None):
        mx = _mx()
        rng = np.random.default_rng(seed + T + H + I + E + k)
        self.w1q, self.s1, w1 = M.random_operand(rng, E * 2 * I, H, 1 / np.sqrt(H))
        self.w2q, self.s2, w2 = M.random_operand(rng, E * H, I, 1 / np.sqrt(I))
        self.w1, self.w2 = w1.reshape(E, 2 * I, H), w2.reshape(E, H, I)
        self.weights = mx.ExpertWeights(_gpu(self.w1q.reshape(E, 2 * I, -1)), _gpu(self.s1.reshape(E, 2 * I, -1)),
                                        _gpu(self.w2q.reshape(E, H, -1)), _gpu(self.s2.reshape(E, H, -1)))
        self.x = torch.from_numpy(rng.normal(size=(T, H)) * 1.5).to(torch.bfloat16)
        p = rng.gumbel(size=(T, E)) - (2.0 * np.log(np.arange(E) + 1) if skew else 0.0)
        ids = np.argsort(-p, axis=1)[:, :k].astype(np.int64)
        if drop:
            out = rng.random((T, k))
            ids[out < drop] = -1
            ids[out > 1 - drop / 2] = E + 3
        self.ids, self.w = ids, np.abs(rng.normal(size=(T, k))).astype(np.float32)
        self.plan = mx.ExpertPlan(H, I, E, k, max_tokens or T, ids_dtype=ids_dtype, out_dtype=out_dtype)
        self.scratch = self.plan.alloc_scratch()
        self.scratch.fill_(0xFF)                        # nothing is read before it is written
        self.dx, self.dids, self.dw = self.x.cuda(), _gpu(ids).to(ids_dtype), _gpu(self.w)

    def run(self, y=None):
        return self.plan.forward(self.dx, self.dids, self.dw, self.weights, self.scratch, y=y)

    def check(self, y):
        ref, bound = M.layer(self.x.double().numpy(), self.ids, self.w.astype(np.float64), self.w1, self.w2,
                             HALF[self.plan.out_dtype])
        err = np.abs(y.double().cpu().numpy() - ref)
        say(f"[result] max error {err.max():.2e} of max {np.abs(ref).max():.2e}")
        assert np.all(err <= bound), float((err / bound).max())
        # the bound is no licence: over all values the difference stays far below one code's step
        assert np.linalg.norm(err) <= 1e-2 * np.linalg.norm(ref) + 1e-30


@pytest.mark.parametrize("T,H,I,E,k", [(1, 64, 32, 4, 2), (1, 1024, 512, 96, 8), (4, 256, 128, 8, 2), (3, 96, 160, 5, 3),
                                       (16, 1024, 512, 32, 8), (16, 2560, 320, 16, 10), (50, 32, 96, 1, 1),
                                       (150, 288, 224, 6, 4), (300, 512, 256, 8, 8), (700, 128, 64, 3, 2)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_layer(T, H, I, E, k, dtype):
    say(f"[case] MXFP4 layer T={T} H={H} I={I} E={E} k={k} {dtype}")
    c = Layer(T, H, I, E, k, out_dtype=dtype, ids_dtype=torch.int32 if T % 2 else torch.int64)
    y = torch.full((T, H), float("nan"), dtype=dtype, device="cuda")
    c.run(y)
    c.check(y)


@pytest.mark.parametrize("T,H,I,E,k", [(40, 160, 96, 64, 8), (35, 1056, 64, 70, 8), (60, 64, 1088, 40, 6),   # 16-row tiles
                                       (300, 672, 96, 4, 2), (200, 96, 640, 5, 2), (130, 512, 544, 3, 2),
                                       (8, 64, 32, 40, 32), (90, 64, 64, 33, 32)])
def test_layer_other_forms(T, H, I, E, k):
    """Routes between the layer's forms, rows of 17 to 34 blocks, the largest top-k."""
    say(f"[case] MXFP4 layer T={T} H={H} I={I} E={E} k={k}")
    c = Layer(T, H, I, E, k, drop=0.1)
    y = torch.full((T, H), float("nan"), device="cuda")
    c.run(y)
    c.check(y)


@pytest.mark.parametrize("T,k", [(20, 3), (85, 3), (256, 1)])
def test_layer_few_routes_one_expert_dropped_and_repeated(T, k):
    """Up to 256 routes without a route map: many routes of one expert, ids outside, the same id twice."""
    c = Layer(T, 128, 96, 60, k, ids_dtype=torch.int32)
    c.ids[:] = 7
    c.ids[3] = -1
    c.ids[T // 2:T // 2 + 4, 0] = 60
    c.ids[-1] = 2 ** 31 - 1
    c.ids[1, 0] = 59
    c.dids = _gpu(c.ids).to(torch.int32)
    c.dw[3] = float("inf")
    y = torch.full((T, 128), float("nan"), device="cuda")
    c.run(y)
    assert torch.all(y[3] == 0) and torch.all(y[-1] == 0)
    c.check(y)


@pytest.mark.parametrize("T,E", [(12, 40), (60, 70), (200, 6)])
def test_layer_a_token_with_an_infinity_stays_alone(T, E):
    c = Layer(T, 96, 64, E, 4)
    good = c.run().clone()
    c.dx[5, 40], c.dx[9, 3] = float("inf"), float("nan")
    y = c.run()
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[5] = bad[9] = True
    assert torch.isnan(y[bad]).all() and torch.equal(y[~bad], good[~bad])


def test_layer_uneven_routes_and_dropped_ids():
    c = Layer(260, 256, 128, 40, 6, skew=True, drop=0.2, max_tokens=300)
    c.ids[7] = -1                                       # a token without any expert
    c.dids = _gpu(c.ids)
    c.dw[7] = float("nan")                              # a dropped route's weight is not used
    y = torch.full((260, 256), float("nan"), device="cuda")
    c.run(y)
    assert torch.all(y[7] == 0)
    c.check(y)


def test_layer_every_token_to_one_expert_and_the_same_id_twice():
    c = Layer(200, 128, 96, 7, 3)
    c.ids[:] = 5
    c.dids = _gpu(c.ids)
    c.check(c.run())


def test_layer_large_batch_many_routes():
    """More than 4096 routes: the route map's two-launch form."""
    c = Layer(1500, 64, 64, 12, 4, skew=True)
    c.check(c.run())


@pytest.mark.parametrize("T,H,I,E,k,skew", [(500, 640, 2048, 10, 4, False), (1300, 1152, 2080, 6, 1, False),
                                            (900, 1024, 1536, 12, 3, True)])
def test_layer_more_tiles_than_workgroups(T, H, I, E, k, skew):
    """The first product's workgroups take several tiles each: rows of whole and of part groups of scales, an odd
    number of groups, top-1, a last column block that is not full, dropped routes; and the same bits again."""
    say(f"[case] MXFP4 layer T={T} H={H} I={I} E={E} k={k} skew={skew}")
    c = Layer(T, H, I, E, k, skew=skew, drop=0.2 if skew else 0.0)
    y = torch.full((T, H), float("nan"), device="cuda")
    c.run(y)
    c.check(y)
    assert torch.equal(c.run(), y)


def test_layer_zero_tokens_and_smaller_batches():
    c = Layer(40, 128, 64, 6, 2, max_tokens=64)
    y = torch.full((0, 128), 1.0, device="cuda")
    assert c.plan.forward(c.dx[:0], c.dids[:0], c.dw[:0], c.weights, c.scratch, y=y) is y
    full = c.run()
    part = c.plan.forward(c.dx[:5], c.dids[:5], c.dw[:5], c.weights, c.scratch)
    c.check(full)
    ref, bound = M.layer(c.x[:5].double().numpy(), c.ids[:5], c.w[:5].astype(np.float64), c.w1, c.w2, 2.0 ** -24)
    assert np.all(np.abs(part.double().cpu().numpy() - ref) <= bound)


def test_layer_repeatable_other_stream_and_graph():
    c = Layer(64, 256, 128, 16, 4, out_dtype=torch.bfloat16)
    a = c.run().clone()
    c.scratch.fill_(0x7F)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = c.run()
    torch.cuda.synchronize()
    assert torch.equal(a, b)
    y = torch.empty_like(a)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(y)
    for seed in range(4):
        torch.manual_seed(seed)
        c.dx.copy_(torch.randn(64, 256).to(torch.bfloat16).cuda())
        c.dids.copy_(torch.rand(64, 16).argsort(1)[:, :4].cuda())
        g.replay()
        torch.cuda.synchronize()
        got = y.clone()
        assert torch.equal(got, c.run())


def test_router_quantisation_and_layer_together():
    """A model step: logits -> ids, weights, balance loss -> expert layer; weights quantised by the kernel."""
    from trellis_quantized_moe_tmoe_amd import router
    mx = _mx()
    T, H, I, E, k = 33, 128, 64, 8, 2
    rng = np.random.default_rng(9)
    w1 = (rng.normal(size=(E, 2 * I, H)) / np.sqrt(H)).astype(np.float32)
    w2 = (rng.normal(size=(E, H, I)) / np.sqrt(I)).astype(np.float32)
    wr = rng.normal(size=(E, H)).astype(np.float32)
    x = torch.from_numpy(rng.normal(size=(T, H))).to(torch.bfloat16)
    gx = x.cuda()
    # the router's own projection in MXFP4, in fp32 out
    xq, xs = mx.quantize(gx)
    logits = mx.linear(xq, xs, *mx.quantize(_gpu(wr)))
    mask = torch.arange(T) % 11 != 4
    ids, w, lse = router.topk(logits, k, token_mask=mask.cuda())
    loss, counts, slope = router.balance_loss(logits, lse, ids, 0.01)
    plan = mx.ExpertPlan(H, I, E, k, T)
    y = plan.forward(gx, ids, w, mx.ExpertWeights(*mx.quantize(_gpu(w1)), *mx.quantize(_gpu(w2))), plan.alloc_scratch())
    xv = x.double().numpy()
    want_logits = M.rounded(xv) @ M.rounded(wr.astype(np.float64)).T
    assert np.abs(logits.double().cpu().numpy() - want_logits).max() <= 1e-4
    i = ids.cpu().numpy()
    assert np.all(i[~mask.numpy()] == -1) and int(counts.sum()) == int(mask.sum()) * k
    top = np.argsort(-logits.double().cpu().numpy(), axis=1, kind="stable")[:, :k]
    assert np.array_equal(i[mask.numpy()], top[mask.numpy()])
    ref, bound = M.layer(xv, i, w.double().cpu().numpy(), M.rounded(w1.astype(np.float64)),
                         M.rounded(w2.astype(np.float64)), 2.0 ** -24)
    assert np.all(np.abs(y.double().cpu().numpy() - ref) <= bound)
    assert torch.all(y[~mask.cuda()] == 0) and torch.isfinite(loss)
    d = router.backward(logits, lse, ids, w=w, dw=torch.ones_like(w), slope=slope, dloss=torch.ones((), device="cuda"))
    assert torch.isfinite(d).all() and torch.all(d[~mask.cuda()] == 0)


def test_weights_of_a_tracked_router():
    """topk's weights carry a gradient that the layer cannot pass on: refused; the same call without gradients runs."""
    from trellis_quantized_moe_tmoe_amd import router
    mx = _mx()
    T, H, I, E, k = 5, 64, 32, 4, 2
    g = torch.Generator().manual_seed(3)
    weights = mx.ExpertWeights(*mx.quantize(torch.randn(E, 2 * I, H, generator=g).cuda()),
                               *mx.quantize(torch.randn(E, H, I, generator=g).cuda()))
    x = torch.randn(T, H, generator=g).to(torch.bfloat16).cuda()
    logits = torch.randn(T, E, generator=g).cuda().requires_grad_()
    plan = mx.ExpertPlan(H, I, E, k, T)
    scratch = plan.alloc_scratch()
    ids, w, lse = router.topk(logits, k)
    with pytest.raises(ValueError, match="w: requires a gradient"):
        plan.forward(x, ids, w, weights, scratch)
    y = plan.forward(x, ids, w.detach(), weights, scratch)
    with torch.no_grad():
        assert torch.equal(plan.forward(x, ids, w, weights, scratch), y)


def test_an_output_that_a_backward_still_needs():
    """y is written in place: a gradient that saved it before must fail, as after torch's own in-place operations,
    not be computed from the new values."""
    mx = _mx()
    g = torch.Generator().manual_seed(4)
    xq, xs = mx.quantize(torch.randn(3, 64, generator=g).cuda())
    wq, ws = mx.quantize(torch.randn(5, 64, generator=g).cuda())
    plan = mx.ExpertPlan(64, 32, 4, 2, 3)
    weights = mx.ExpertWeights(*mx.quantize(torch.randn(4, 64, 64, generator=g).cuda()),
                               *mx.quantize(torch.randn(4, 64, 32, generator=g).cuda()))
    x = torch.randn(3, 64, generator=g).to(torch.bfloat16).cuda()
    ids, w, scratch = torch.zeros(3, 2, dtype=torch.int64, device="cuda"), torch.ones(3, 2, device="cuda"), plan.alloc_scratch()
    for y, call in [(torch.empty(3, 5, device="cuda"), lambda y: mx.linear(xq, xs, wq, ws, y=y)),
                    (torch.empty(3, 64, device="cuda"), lambda y: plan.forward(x, ids, w, weights, scratch, y=y))]:
        gate = torch.ones((), device="cuda", requires_grad=True)
        out = (call(y) * gate).sum()
        out.backward()
        assert torch.equal(gate.grad, y.sum())
        out = (call(y) * gate).sum()
        call(y)
        with pytest.raises(RuntimeError, match="inplace"):
            out.backward()
        with torch.inference_mode():
            kept = torch.empty_like(y)
            assert call(kept) is kept and torch.equal(kept, y)
