"""Router calls that are refused on the host, before any launch; and its float64 reference checked by hand."""
import ctypes

import numpy as np
import pytest
import torch

import router_ref as R

FAKE = 1 << 20                                    # never dereferenced: the checks return first


@pytest.fixture(scope="module")
def N():
    from trellis_quantized_moe_tmoe_amd import native
    return native


def _cfg(N, **kw):
    d = dict(num_experts=96, top_k=8, logits_dtype=0, ids_dtype=1, renormalize=1)
    d.update(kw)
    return N.RouterConfig(*[d[n] for n, _ in N.RouterConfig._fields_])


def _topk(N, cfg=None, **o):
    cfg = cfg or _cfg(N)
    return N.lib.tmoe_router_topk(ctypes.byref(cfg), o.get("logits", FAKE), o.get("stride", 96), o.get("mask", None),
                                  o.get("T", 4), o.get("ids", FAKE), o.get("w", FAKE), o.get("lse", FAKE), None)


@pytest.mark.parametrize("kw,status", [
    (dict(num_experts=0), 1), (dict(top_k=0), 1), (dict(top_k=97), 2), (dict(num_experts=7), 1), (dict(num_experts=513), 2),
    (dict(top_k=33), 2), (dict(logits_dtype=3), 1), (dict(logits_dtype=-1), 1), (dict(ids_dtype=2), 1),
    (dict(renormalize=2), 1)])
def test_config_is_checked(N, kw, status):
    cfg = _cfg(N, **kw)
    assert _topk(N, cfg, T=0) == status
    need = ctypes.c_size_t()
    assert N.lib.tmoe_balance_loss_scratch(ctypes.byref(cfg), 4, ctypes.byref(need)) == status


def test_topk_arguments(N):
    assert _topk(N, T=0) == 0
    assert _topk(N, T=-1) == 1
    assert _topk(N, T=(1 << 24) + 1) == 2
    assert _topk(N, logits=0) == 1 and _topk(N, ids=0) == 1 and _topk(N, w=0) == 1 and _topk(N, lse=0) == 1
    assert _topk(N, stride=95) == 1
    assert _topk(N, logits=FAKE + 2) == 5 and _topk(N, ids=FAKE + 4) == 5 and _topk(N, w=FAKE + 2) == 5
    assert _topk(N, _cfg(N, logits_dtype=1), logits=FAKE + 1) == 5
    assert N.lib.tmoe_router_topk(None, FAKE, 96, None, 4, FAKE, FAKE, FAKE, None) == 1


def test_balance_loss_arguments(N):
    cfg, need = _cfg(N), ctypes.c_size_t()
    assert N.lib.tmoe_balance_loss_scratch(ctypes.byref(cfg), 100, ctypes.byref(need)) == 0 and need.value > 0
    assert N.lib.tmoe_balance_loss_scratch(ctypes.byref(cfg), -1, ctypes.byref(need)) == 1
    assert N.lib.tmoe_balance_loss_scratch(ctypes.byref(cfg), 100, None) == 1
    assert N.lib.tmoe_balance_loss_scratch(ctypes.byref(cfg), 100, ctypes.byref(need)) == 0

    def call(**o):
        return N.lib.tmoe_balance_loss(ctypes.byref(cfg), o.get("logits", FAKE), 96, o.get("lse", FAKE),
                                       o.get("ids", FAKE), o.get("T", 100), o.get("coefficient", 0.01),
                                       o.get("loss", FAKE), o.get("counts", FAKE), o.get("slope", FAKE),
                                       o.get("scratch", FAKE), o.get("bytes", need.value), None)
    assert call(bytes=need.value - 1) == 3 and call(scratch=FAKE + 8) == 3 and call(scratch=0) == 3
    assert call(coefficient=float("nan")) == 1 and call(coefficient=float("inf")) == 1
    assert call(loss=0) == 1 and call(counts=0) == 1 and call(slope=0) == 1 and call(lse=0) == 1
    assert call(T=-1) == 1 and call(logits=0) == 1 and call(ids=0) == 1
    assert call(lse=FAKE + 1) == 5 and call(counts=FAKE + 2) == 5


def test_backward_arguments(N):
    cfg = _cfg(N)

    def call(**o):
        return N.lib.tmoe_router_backward(ctypes.byref(cfg), o.get("logits", FAKE), o.get("stride", 96),
                                          o.get("lse", FAKE), o.get("ids", FAKE), o.get("w", FAKE), o.get("dw", FAKE),
                                          o.get("slope", FAKE), o.get("dloss", FAKE), o.get("T", 4),
                                          o.get("dlogits", FAKE), None)
    assert call(T=0) == 0
    assert call(w=0) == 1 and call(dw=0) == 1 and call(slope=0) == 1 and call(dloss=0) == 1
    assert call(w=0, dw=0, slope=0, dloss=0) == 1 and call(w=0, dw=0, slope=0, dloss=0, T=0) == 1
    assert call(lse=0) == 1 and call(dlogits=0) == 1 and call(stride=1) == 1
    assert call(dlogits=FAKE + 2) == 5 and call(dw=FAKE + 1) == 5


def test_binding_refuses_what_does_not_fit():
    from trellis_quantized_moe_tmoe_amd import router
    l = torch.zeros(4, 16)
    ids, w, lse = torch.zeros(4, 2, dtype=torch.int64), torch.zeros(4, 2), torch.zeros(4)
    for bad, msg in [(lambda: router.topk(l, 2), "GPU device"), (lambda: router.topk(l[0], 2), "2-D"),
                     (lambda: router.topk(l.double(), 2), "dtype"), (lambda: router.topk(l.t(), 2), "adjacent"),
                     (lambda: router.topk(l[:1].expand(4, 16), 2), "overlap"),
                     (lambda: router.topk(l, 2, ids_dtype=torch.int16), "ids: dtype"),
                     (lambda: router.topk(l, 2, token_mask=torch.ones(3, dtype=torch.bool)), "token_mask: shape"),
                     (lambda: router.topk(l, 2, token_mask=torch.ones(4)), "token_mask: dtype"),
                     (lambda: router.balance_loss(l, lse[:3], ids), "lse: shape"),
                     (lambda: router.balance_loss(l, lse, ids[:3]), "ids: shape"),
                     (lambda: router.balance_loss(l, lse, ids.float()), "ids: dtype"),
                     (lambda: router.balance_loss(l, lse, ids), "GPU device"),
                     (lambda: router.backward(l, lse, ids), "give w and dw"),
                     (lambda: router.backward(l, lse, ids, w=w), "give w and dw"),
                     (lambda: router.backward(l, lse, ids, w=w, dw=w[:, :1]), "dw: shape"),
                     (lambda: router.backward(l, lse, ids, w=w, dw=torch.zeros(2, 4).t()), "dw: must be contiguous"),
                     (lambda: router.backward(l, lse, ids, slope=torch.zeros(15), dloss=torch.ones(())), "slope: shape"),
                     (lambda: router.backward(l, lse, ids, slope=torch.zeros(16), dloss=torch.ones(2)), "dloss"),
                     (lambda: router.backward(l, lse, ids, w=w, dw=w), "GPU device")]:
        with pytest.raises(ValueError, match=msg):
            bad()


def test_reference_by_hand():
    l = np.array([[0.0, np.log(2.0), np.log(2.0), -np.inf], [-np.inf] * 4])
    ids, w, lse = R.topk(l, 3, True)
    assert ids.tolist() == [[1, 2, 0], [-1, -1, -1]]
    assert np.allclose(w, [[0.4, 0.4, 0.2], [0, 0, 0]]) and np.isclose(lse[0], np.log(5.0)) and lse[1] == -np.inf
    # a uniform router has loss = coefficient
    ids = np.arange(16).reshape(4, 4) % 8
    loss, c, _, _ = R.balance(np.zeros((4, 8)), np.ones(4, bool), ids, 0.25)
    assert c.tolist() == [2] * 8 and np.isclose(loss, 0.25)


def test_configurations_are_refused_before_the_outputs_are_allocated(monkeypatch):
    """A top_k that no configuration allows must come back as the library's refusal, not as what the allocator says of
    outputs [T, top_k]: negative sizes, or more memory than there is."""
    from trellis_quantized_moe_tmoe_amd import native, router
    l, made = torch.zeros(4, 16), []
    monkeypatch.setattr(router, "_one_gpu", lambda *t: True)         # as if on a GPU: no call below gets as far
    monkeypatch.setattr(torch, "empty", lambda *a, **k: made.append(a) or pytest.fail("allocated"))
    mask = torch.ones(4, dtype=torch.bool)
    for top_k, name in [(-1, "INVALID_ARG"), (0, "INVALID_ARG"), (17, "INVALID_ARG"), (33, "UNSUPPORTED"),
                        (2 ** 30, "UNSUPPORTED"), (-2 ** 30, "INVALID_ARG")]:
        with pytest.raises(native.TmoeError, match=name):
            router.topk(l, top_k, token_mask=mask)
    with pytest.raises(native.TmoeError, match="UNSUPPORTED"):
        router.topk(torch.zeros(2, 513), 2, token_mask=mask[:2])
    assert not made


def test_forward_mode_derivatives_are_refused():
    """A dual tensor has requires_grad False: its tangent must not get lost without a word, without gradients either."""
    from torch.autograd import forward_ad
    from trellis_quantized_moe_tmoe_amd import router
    l, lse, ids = torch.zeros(4, 16), torch.zeros(4), torch.zeros(4, 2, dtype=torch.int64)
    w, slope, one = torch.zeros(4, 2), torch.zeros(16), torch.ones(())
    with forward_ad.dual_level(), torch.no_grad():
        d = lambda t: forward_ad.make_dual(t, torch.ones_like(t))  # noqa: E731
        assert not d(l).requires_grad
        for bad in [lambda: router.topk(d(l), 2), lambda: router.balance_loss(d(l), lse, ids),
                    lambda: router.balance_loss(l, d(lse), ids), lambda: router.backward(d(l), lse, ids, w=w, dw=w),
                    lambda: router.backward(l, d(lse), ids, w=w, dw=w), lambda: router.backward(l, lse, ids, w=d(w), dw=w),
                    lambda: router.backward(l, lse, ids, w=w, dw=d(w)),
                    lambda: router.backward(l, lse, ids, slope=d(slope), dloss=one),
                    lambda: router.backward(l, lse, ids, slope=slope, dloss=d(one))]:
            with pytest.raises(ValueError, match="forward-mode"):
                bad()
        with pytest.raises(ValueError, match="GPU device"):      # beside a dual, other tensors go on as they did
            router.topk(l, 2)


def test_sizes_past_32_bits():
    """2^32 + 5 rows or experts must not pass for 5."""
    from trellis_quantized_moe_tmoe_amd import router
    big = 2 ** 32 + 5
    for l, k in [(torch.empty(big, 8, device="meta"), 2), (torch.empty(8, big, device="meta"), 2),
                 (torch.empty(8, 8, device="meta"), 2 ** 32 + 2)]:
        with pytest.raises(ValueError, match="out of range"):
            router.topk(l, k)
