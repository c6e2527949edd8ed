"""Router kernels against the float64 reference (router_ref.py).

Tolerances, with u = 2^-24 (half a step of fp32) and R the largest distance of an available logit from
its row's largest: l - m is off by R u, exp of it by R u + 2 u relative, the sum of E <= 512 positive
terms (8 in a lane, 6 exchanges) by 14 u more, the division by u: a weight is off by at most
(2 R + 20) u relative. Gradients are sums of products of such weights; each term's factor is stated
at its check. Outputs in 16 bits add half a step of their type."""
import numpy as np
import pytest
import torch

import router_ref as R
from gpu_cases import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.float32: U, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -140, torch.bfloat16: 2.0 ** -130, torch.float16: 2.0 ** -25}   # below the normal numbers


def _logits(T, E, dtype, seed, unavailable=0.05, mask_p=0.0, nan_masked=True):
    rng = np.random.default_rng(seed)
    l = torch.from_numpy(rng.normal(size=(T, E)) * 2.0).to(torch.float32).to(dtype)
    l[torch.from_numpy(rng.random((T, E)) < unavailable)] = -np.inf
    mask = None
    if mask_p:
        mask = torch.from_numpy(rng.random(T) >= mask_p)
        if nan_masked:
            l[~mask] = np.nan
    return l, mask


def _np(l):
    return l.detach().double().cpu().numpy()


def _spread(l64):
    fin = np.isfinite(l64)
    top = np.where(fin, l64, -np.inf).max(1, initial=-np.inf)
    low = np.where(fin, l64, np.inf).min(1, initial=np.inf)
    d = (top - low)[np.isfinite(top - low)]
    return float(d.max()) if d.size else 0.0


def _valid(l64, mask):
    return (R.masked(l64, mask) > -np.inf).any(1)


SHAPES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (16, 96, 8), (7, 64, 32), (33, 65, 10), (5, 128, 1), (130, 256, 8),
          (9, 257, 16), (4, 512, 32), (1025, 96, 8)]


@pytest.mark.parametrize("T,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("renormalize", [True, False])
def test_topk_and_its_gradient(T, E, k, dtype, renormalize):
    from trellis_quantized_moe_tmoe_amd import router
    say(f"[case] router T={T} E={E} k={k} {dtype} renormalize={renormalize}")
    l, mask = _logits(T, E, dtype, 100 * T + E + k, mask_p=0.2 if T > 2 else 0.0)
    l64, m64 = _np(l), None if mask is None else mask.numpy()
    want_ids, want_w, want_lse = R.topk(l64, k, renormalize, m64)
    ids_dtype = torch.int32 if T % 2 else torch.int64
    gl = l.cuda()
    ids, w, lse = router.topk(gl, k, renormalize=renormalize, token_mask=None if mask is None else mask.cuda(),
                              ids_dtype=ids_dtype)
    assert ids.dtype == ids_dtype and w.dtype == lse.dtype == torch.float32
    assert np.array_equal(ids.cpu().numpy(), want_ids)
    r = _spread(R.masked(l64, m64))
    tol = (2 * r + 20) * U
    assert np.all(np.abs(_np(w) - want_w) <= tol * want_w)
    got = _np(lse)
    assert np.array_equal(np.isinf(got), np.isinf(want_lse))
    fin = np.isfinite(want_lse)
    # the relative error of s is an absolute one of its logarithm; log and the sum round once each
    assert np.all(np.abs(got[fin] - want_lse[fin]) <= (r + 20 + 2 * np.abs(want_lse[fin]) + 2 * np.log(E + 1)) * U)

    dw = np.random.default_rng(T).normal(size=(T, k)).astype(np.float32)
    gdw = torch.from_numpy(dw).cuda()
    if m64 is not None:
        gdw[~mask.cuda()] = float("nan")              # a masked row's gradient may hold anything
    d = router.backward(gl, lse, ids, w=w, dw=gdw, renormalize=renormalize)
    assert d.dtype == dtype and d.shape == (T, E)
    lm = R.masked(l64, m64)
    want = R.topk_grad(lm, want_ids, want_w, dw.astype(np.float64), renormalize)
    p = R.softmax_rows(lm)[0]
    wide = np.zeros_like(lm)
    t, j = np.nonzero(want_ids >= 0)
    wide[t, want_ids[t, j]] = want_w[t, j]
    # |dl| terms: w dw and w (or p) times the sum over k terms; each factor carries tol, sums k + 8 roundings
    big = np.abs(dw).max(1, keepdims=True)
    bound = (wide + (0 if renormalize else p)) * big * (2 * tol + (k + 10) * U) * 2
    assert np.all(np.abs(_np(d) - want) <= bound + HALF[dtype] * np.abs(want) + TINY[dtype])


@pytest.mark.parametrize("T,E,k", [(1, 4, 2), (6, 96, 8), (257, 65, 3), (2051, 256, 8), (5000, 512, 16), (9000, 3, 1),
                                   (4097, 1, 1)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_balance_loss_and_its_gradient(T, E, k, dtype):
    from trellis_quantized_moe_tmoe_amd import router
    say(f"[case] balance T={T} E={E} k={k} {dtype}")
    l, mask = _logits(T, E, dtype, 7 * T + E, mask_p=0.25 if T > 4 else 0.0)
    l64, m64 = _np(l), None if mask is None else mask.numpy()
    gl = l.cuda()
    ids, w, lse = router.topk(gl, k, token_mask=None if mask is None else mask.cuda())
    loss, counts, slope = router.balance_loss(gl, lse, ids, 0.5)
    valid = _valid(l64, m64)
    want, c, want_slope, p = R.balance(l64, valid, ids.cpu().numpy(), 0.5)
    assert loss.shape == () and counts.dtype == torch.int32
    assert np.array_equal(counts.cpu().numpy(), c)
    assert np.all(np.abs(_np(slope) - want_slope) <= 2 * U * np.abs(want_slope))
    tol = (2 * _spread(R.masked(l64, m64)) + 20) * U
    rows = T // 2048 + 8                              # rows one wavefront adds up, and four wavefronts
    assert abs(float(loss) - want) <= (tol + rows * U + 4 * U) * abs(want)

    scale = np.float32(0.75 * T * E)                  # a loss scale that keeps fp16 gradients normal
    d = router.backward(gl, lse, ids, slope=slope, dloss=torch.tensor(scale, device="cuda"))
    g = R.balance_grad(p, want_slope, float(scale))
    bound = float(scale) * p * (want_slope + (p * want_slope).sum(1, keepdims=True)) * (2 * tol + 24 * U)
    assert np.all(np.abs(_np(d) - g) <= bound + HALF[dtype] * np.abs(g) + TINY[dtype])

    # both parts in one pass: their sum, rounded once
    dw = np.random.default_rng(E).normal(size=(T, k)).astype(np.float32)
    both = router.backward(gl, lse, ids, w=w, dw=torch.from_numpy(dw).cuda(), slope=slope,
                           dloss=torch.tensor(scale, device="cuda"))
    lm = R.masked(l64, m64)
    rid, rw, _ = R.topk(l64, k, True, m64)
    total = g + R.topk_grad(lm, rid, rw, dw.astype(np.float64), True)
    wide = np.zeros_like(lm)
    t, j = np.nonzero(rid >= 0)
    wide[t, rid[t, j]] = rw[t, j]
    bound = bound + wide * np.abs(dw).max(1, keepdims=True) * (2 * tol + (k + 10) * U) * 2 + 2 * U * np.abs(total)
    assert np.all(np.abs(_np(both) - total) <= bound + HALF[dtype] * np.abs(total) + TINY[dtype])


def test_gradients_against_differences():
    """Central differences of the float64 loss, h = 1e-4: truncation below h^2 times the third derivative
    (under 10 here), cancellation below 1e-16 / h."""
    from trellis_quantized_moe_tmoe_amd import router
    l, _ = _logits(3, 7, torch.float32, 5, unavailable=0.0)
    l64, k, h = _np(l), 3, 1e-4
    dw = np.random.default_rng(1).normal(size=(3, k)).astype(np.float32)
    for renormalize in (True, False):
        ids, w, lse = router.topk(l.cuda(), k, renormalize=renormalize)
        loss, _, slope = router.balance_loss(l.cuda(), lse, ids, 1.0)
        d = _np(router.backward(l.cuda(), lse, ids, w=w, dw=torch.from_numpy(dw).cuda(), renormalize=renormalize,
                                slope=slope, dloss=torch.tensor(0.5, device="cuda")))
        i = ids.cpu().numpy()

        def f(x):
            return R.topk_loss(x, i, dw.astype(np.float64), renormalize) + \
                0.5 * R.balance(x, np.ones(3, bool), i, 1.0)[0]
        for t in range(3):
            for e in range(7):
                up, dn = l64.copy(), l64.copy()
                up[t, e] += h
                dn[t, e] -= h
                assert abs((f(up) - f(dn)) / (2 * h) - d[t, e]) <= 10 * h * h + 1e-11 + 200 * U


def test_ties_zeros_and_lowest_values():
    from trellis_quantized_moe_tmoe_amd import router
    l = torch.zeros(2, 200)
    l[0, ::2] = -0.0                                  # equal to +0: the lowest experts win
    l[1] = torch.finfo(torch.float32).min
    l[1, 150] = l[1, 70] = 1.0
    ids, w, lse = router.topk(l.cuda(), 4)
    assert ids.tolist() == [[0, 1, 2, 3], [70, 150, 0, 1]]
    assert w.tolist() == [[0.25] * 4, [0.5, 0.5, 0.0, 0.0]]
    assert abs(float(lse[0]) - np.log(200.0)) < 1e-6 and abs(float(lse[1]) - 1 - np.log(2.0)) < 1e-6
    low = torch.full((1, 64), torch.finfo(torch.float16).min, dtype=torch.float16)
    ids, w, lse = router.topk(low.cuda(), 2, renormalize=False)
    assert ids.tolist() == [[0, 1]] and w.tolist() == [[1 / 64] * 2] and torch.isfinite(lse).all()


def test_rows_with_few_or_no_experts():
    from trellis_quantized_moe_tmoe_amd import router
    l = torch.full((3, 100), -float("inf"))
    l[1, 42] = -3.0
    l[2, 99], l[2, 0] = 5.0, 4.0
    ids, w, lse = router.topk(l.cuda(), 4, ids_dtype=torch.int32)
    assert ids.tolist() == [[-1] * 4, [42, -1, -1, -1], [99, 0, -1, -1]]
    assert w[0].tolist() == [0.0] * 4 and w[1].tolist() == [1.0, 0.0, 0.0, 0.0]
    assert lse[0] == -float("inf") and abs(float(lse[1]) + 3.0) < 1e-6
    loss, counts, slope = router.balance_loss(l.cuda(), lse, ids, 2.0)
    want, c, _, _ = R.balance(_np(l), np.array([False, True, True]), ids.cpu().numpy(), 2.0)
    assert abs(float(loss) - want) <= 1e-6 * want and np.array_equal(counts.cpu().numpy(), c)
    d = router.backward(l.cuda(), lse, ids, slope=slope, dloss=torch.ones((), device="cuda"))
    assert torch.isfinite(d).all() and torch.all(d[0] == 0)


def test_nan_and_infinity_in_a_row_that_counts():
    from trellis_quantized_moe_tmoe_amd import router
    l = torch.zeros(3, 10)
    l[0, 3], l[1, 4] = float("nan"), float("inf")
    ids, w, lse = router.topk(l.cuda(), 2)
    assert ids.tolist() == [[0, 1], [4, 0], [0, 1]]
    assert torch.isnan(w[:2]).all() and torch.isnan(lse[:2]).all()
    assert w[2].tolist() == [0.5, 0.5]
    mask = torch.tensor([False, False, True])
    ids, w, lse = router.topk(l.cuda(), 2, token_mask=mask.cuda())
    assert ids.tolist() == [[-1, -1], [-1, -1], [0, 1]] and w[:2].abs().sum() == 0
    loss, counts, slope = router.balance_loss(l.cuda(), lse, ids)
    assert torch.isfinite(loss) and counts.sum() == 2
    d = router.backward(l.cuda(), lse, ids, w=w, dw=torch.full_like(w, 2.0), renormalize=False, slope=slope,
                        dloss=torch.ones((), device="cuda"))
    assert torch.isfinite(d).all() and torch.all(d[:2] == 0)


@pytest.mark.parametrize("T,E,k", [(6, 10, 2), (300, 65, 3), (2051, 256, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_balance_loss_leaves_out_rows_whose_lse_is_nan(T, E, k, dtype):
    """Rows with a NaN or +inf logit that no mask takes out: lse is NaN, which is not > -inf. They add nothing to n and
    P and get no gradient; their ids are counted like all others. Tolerances as for the healthy batch."""
    from trellis_quantized_moe_tmoe_amd import router
    say(f"[case] balance with NaN rows T={T} E={E} k={k} {dtype}")
    l, _ = _logits(T, E, dtype, 13 * T + E)
    l[1, E // 2], l[3, E - 1], l[4] = float("nan"), float("inf"), -float("inf")
    l[5::97, 0] = float("nan")
    l64, gl = _np(l), l.cuda()
    ids, w, lse = router.topk(gl, k)
    bad = np.isnan(l64).any(1) | np.isposinf(l64).any(1)
    assert np.array_equal(torch.isnan(lse).cpu().numpy(), bad)
    valid = ~bad & (l64 > -np.inf).any(1)
    assert valid.any() and not valid[4]
    healthy = np.where(valid[:, None], l64, 0.0)
    loss, counts, slope = router.balance_loss(gl, lse, ids, 0.5)
    want, c, want_slope, p = R.balance(healthy, valid, ids.cpu().numpy(), 0.5)
    assert c.sum() == (ids >= 0).sum() and np.array_equal(counts.cpu().numpy(), c)
    assert np.all(np.abs(_np(slope) - want_slope) <= 2 * U * np.abs(want_slope))
    tol = (2 * _spread(healthy) + 20) * U
    assert abs(float(loss) - want) <= (tol + (T // 2048 + 8) * U + 4 * U) * abs(want)

    scale = np.float32(0.75 * T * E)
    dloss = torch.tensor(scale, device="cuda")
    d = router.backward(gl, lse, ids, slope=slope, dloss=dloss)
    g = R.balance_grad(p, want_slope, float(scale))
    bound = float(scale) * p * (want_slope + (p * want_slope).sum(1, keepdims=True)) * (2 * tol + 24 * U)
    assert np.all(np.abs(_np(d) - g) <= bound + HALF[dtype] * np.abs(g) + TINY[dtype])
    assert not d[torch.from_numpy(~valid).cuda()].any()
    # beside the weights' gradient, which is NaN where such a row's weights are: the selected logits, or all of them
    both = router.backward(gl, lse, ids, w=w, dw=torch.ones_like(w), slope=slope, dloss=dloss)
    alone = router.backward(gl, lse, ids, w=w, dw=torch.ones_like(w))
    assert torch.equal(torch.isnan(both), torch.isnan(alone)) and torch.isnan(both).any(1).cpu().numpy().sum() == bad.sum()
    soft = router.backward(gl, lse, ids, w=w, dw=torch.ones_like(w), renormalize=False, slope=slope, dloss=dloss)
    assert np.array_equal(torch.isnan(soft).all(1).cpu().numpy(), bad)
    assert np.array_equal(torch.isnan(soft).any(1).cpu().numpy(), bad)


def test_strided_rows_and_large_logits():
    from trellis_quantized_moe_tmoe_amd import router
    wide = torch.full((6, 100), float("nan"), device="cuda")
    l, _ = _logits(6, 33, torch.float32, 3, unavailable=0.0)
    l = l + 5000.0                                    # exp(l - lse) would lose 3 digits here
    wide[:, 17:50] = l.cuda()
    part = wide[:, 17:50]
    for renormalize in (True, False):
        ids, w, lse = router.topk(part, 3, renormalize=renormalize)
        rid, rw, _ = R.topk(_np(l), 3, renormalize)
        assert np.array_equal(ids.cpu().numpy(), rid)
        assert np.all(np.abs(_np(w) - rw) <= (2 * _spread(_np(l)) + 20) * U * rw)
    d = router.backward(part, lse, ids, w=w, dw=torch.ones_like(w), renormalize=False)
    want = R.topk_grad(_np(l), rid, rw, np.ones_like(rw), False)
    assert d.is_contiguous() and np.all(np.abs(_np(d) - want) <= 200 * U)


def test_no_tokens():
    from trellis_quantized_moe_tmoe_amd import router
    l = torch.empty(0, 16, device="cuda")
    ids, w, lse = router.topk(l, 2)
    assert ids.shape == (0, 2) and lse.shape == (0,)
    loss, counts, slope = router.balance_loss(l, lse, ids)
    assert float(loss) == 0.0 and counts.tolist() == [0] * 16 and slope.tolist() == [0.0] * 16
    assert router.backward(l, lse, ids, w=w, dw=w).shape == (0, 16)


def test_autograd_equals_the_explicit_gradient():
    from trellis_quantized_moe_tmoe_amd import router
    l, mask = _logits(40, 96, torch.bfloat16, 11, mask_p=0.2)
    gl = l.cuda().requires_grad_()
    ids, w, lse = router.topk(gl, 8, token_mask=mask.cuda())
    assert w.requires_grad and not ids.requires_grad and not lse.requires_grad
    loss, counts, slope = router.balance_loss(gl, lse, ids, 0.1)
    w.sum().backward(retain_graph=True)               # an expanded (stride 0) gradient
    assert torch.equal(gl.grad, router.backward(gl.detach(), lse, ids, w=w.detach(), dw=torch.ones_like(w)))
    gl.grad = None
    (3.0 * loss).backward()
    assert torch.equal(gl.grad, router.backward(gl.detach(), lse, ids, slope=slope,
                                                dloss=torch.full((), 3.0, device="cuda")))
    with torch.no_grad():
        assert not router.topk(gl, 8)[1].requires_grad


def test_repeatable_and_on_another_stream():
    from trellis_quantized_moe_tmoe_amd import router
    l, mask = _logits(3000, 256, torch.float32, 21, mask_p=0.1)
    l, mask = l.cuda(), mask.cuda()

    def all_of():
        ids, w, lse = router.topk(l, 8, token_mask=mask)
        loss, counts, slope = router.balance_loss(l, lse, ids)
        return ids, w, lse, loss, counts, slope, router.backward(l, lse, ids, w=w, dw=w.clone(), slope=slope, dloss=loss)
    a = all_of()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = all_of()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    for x, y in zip(a, b):
        assert torch.equal(x.view(torch.int32) if x.dtype == torch.float32 else x,
                           y.view(torch.int32) if y.dtype == torch.float32 else y)


def test_captured_graph_replays():
    from trellis_quantized_moe_tmoe_amd import router
    l, _ = _logits(512, 96, torch.float32, 31)
    buf = l.cuda()
    dw = torch.randn(512, 8, device="cuda")

    def step():
        ids, w, lse = router.topk(buf, 8)
        loss, counts, slope = router.balance_loss(buf, lse, ids)
        return ids, w, loss, counts, router.backward(buf, lse, ids, w=w, dw=dw, slope=slope, dloss=loss)
    step()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    for seed in (31, 32, 33, 34):
        buf.copy_(_logits(512, 96, torch.float32, seed)[0].cuda())
        g.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in out]
        want = step()
        torch.cuda.synchronize()
        for x, y in zip(got, want):
            assert torch.equal(x, y)


def test_routes_feed_the_layer():
    """Top-k ids and weights straight into the layer: rows left out give zeros, the others what the same
    ids and weights give from outside."""
    from gpu_cases import Case
    from trellis_quantized_moe_tmoe_amd import router
    c = Case("tiny", 16)
    l, _ = _logits(16, c.inp.experts, torch.float32, 3, unavailable=0.0)
    mask = torch.ones(16, dtype=torch.bool)
    mask[5] = mask[11] = False
    ids, w, lse = router.topk(l.cuda(), c.inp.top_k, token_mask=mask.cuda())
    y = c.plan.forward(c.x, ids, w, c.weights, c.scratch)
    rid, rw, _ = R.topk(_np(l), c.inp.top_k, True, mask.numpy())
    ref = c.plan.forward(c.x, torch.from_numpy(rid).cuda(), torch.from_numpy(rw.astype(np.float32)).cuda(), c.weights,
                         c.scratch)
    assert torch.all(y[~mask.cuda()] == 0)
    assert float((y - ref).abs().max()) <= 1e-5 * float(ref.abs().max())
