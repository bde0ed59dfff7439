"""CPU checks of the scored router, the dense product and the gate's gradients: the C ABI's
refusals (nothing is enqueued), the binding's checks, and the fp64 reference against differences."""
import ctypes

import numpy as np
import pytest
import torch

import sparse_mixture_experts_topk_amd as moe
from oracle import operators as ref
from sparse_mixture_experts_topk_amd import _lib

A = 0x10000                 # an aligned address that no refused call reads
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def shape(**kw):
    base = dict(T=16, d_model=256, d_ff=256, n_experts=64, top_k=6)
    base.update(kw)
    return moe.make_shape(**base)


def status(fn, *args):
    return getattr(_lib.load(), fn)(*[ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in args])


# ---- routers ----

@pytest.mark.parametrize("router,want", [
    (dict(score=2), INVALID), (dict(score=-1), INVALID),
    (dict(n_groups=0), INVALID), (dict(n_groups=5, topk_groups=5), INVALID),       # 64 % 5
    (dict(n_groups=65), INVALID), (dict(n_groups=8, topk_groups=9), INVALID),
    (dict(n_groups=8, topk_groups=0), INVALID), (dict(group_top=0), INVALID), (dict(group_top=3), INVALID),
    (dict(n_groups=64, topk_groups=8, group_top=2), INVALID),                       # groups of one expert
    (dict(n_groups=16, topk_groups=1), INVALID),                                    # 4 experts for top-6
    (dict(renormalize=2), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
])
def test_router_refusals(router, want):
    r = moe.make_router(**router)
    assert status("moe_route_scored", shape(), r, A, None, A, A, None, None, None) == want
    assert status("moe_route_scored_backward", shape(), r, A, A, A, None, A, None) == want


def test_router_refuses_many_groups_pointers_and_shapes():
    r = moe.make_router()
    wide = moe.make_router(n_groups=128, topk_groups=64)
    assert status("moe_route_scored", shape(n_experts=128), wide, A, None, A, A, None, None, None) == UNSUPPORTED
    assert status("moe_route_scored", shape(n_experts=257), r, A, None, A, A, None, None, None) == UNSUPPORTED
    ok = (A, None, A, A, None, None)
    for i in (0, 2, 3):                                   # required
        bad = list(ok)
        bad[i] = None
        assert status("moe_route_scored", shape(), r, *bad, None) == INVALID
    for i in range(6):                                    # 16-byte alignment
        bad = list(ok)
        bad[i] = A + 4
        assert status("moe_route_scored", shape(), r, *bad, None) == INVALID
    ok = (A, A, A, None, A)
    for i in range(5):
        bad = list(ok)
        bad[i] = A + 8
        assert status("moe_route_scored_backward", shape(), r, *bad, None) == INVALID
        if i != 3:
            bad[i] = None
            assert status("moe_route_scored_backward", shape(), r, *bad, None) == INVALID
    assert _lib.load().moe_route_scored(ctypes.byref(shape()), None, *([A] * 6), None) == INVALID
    # no tokens: nothing to do, pointers not looked at
    assert status("moe_route_scored", shape(T=0), r, None, None, None, None, None, None, None) == 0
    assert status("moe_route_scored_backward", shape(T=0), r, None, None, None, None, None, None) == 0


def test_combine_backward_refusals():
    ok = [A, A, A, A, A, A]                               # dy y_perm slot_to_row weights dy_perm dweights
    fn = "moe_combine_backward"
    for i in (0, 2, 3):
        bad = list(ok)
        bad[i] = None
        assert status(fn, shape(), *bad, None) == INVALID
    for i in range(6):
        bad = list(ok)
        bad[i] = A + 2
        assert status(fn, shape(), *bad, None) == INVALID
    assert status(fn, shape(), A, A, A, A, None, None, None) == INVALID       # no output
    assert status(fn, shape(), A, None, A, A, A, A, None) == INVALID          # dweights need y_perm
    assert status(fn, shape(T=0), None, None, None, None, A, None, None) == 0
    assert status(fn, shape(d_model=100), *ok, None) == UNSUPPORTED


# ---- dense product ----

@pytest.mark.parametrize("kw,want", [
    (dict(), 0), (dict(M=0), 0), (dict(M=-1), INVALID), (dict(M=(1 << 24) + 1), INVALID), (dict(N=0), INVALID),
    (dict(K=0), INVALID), (dict(N=12), UNSUPPORTED), (dict(K=100), UNSUPPORTED), (dict(N=(1 << 18) + 8), UNSUPPORTED),
    (dict(K=(1 << 18) + 8), UNSUPPORTED), (dict(dtype="f32"), UNSUPPORTED), (dict(dtype="f32", y_dtype="f32"), 0), (dict(dtype="fp8_e4m3"), UNSUPPORTED),
    (dict(dtype=9), INVALID), (dict(y_dtype="mxfp4"), UNSUPPORTED), (dict(y_dtype=-1), INVALID),
    (dict(act=5), INVALID), (dict(act=-1), INVALID),
])
def test_linear_descriptor(kw, want):
    lin = moe.make_linear(**{**dict(M=7, N=64, K=128), **kw})
    n = ctypes.c_size_t(0)
    for call in (moe.MOE_CALL_LINEAR, moe.MOE_CALL_LINEAR_BACKWARD):
        assert _lib.load().moe_linear_workspace_bytes(ctypes.byref(lin), call, ctypes.byref(n)) == want
    if want:
        assert status("moe_linear", lin, A, A, None, None, A, None, A, 1 << 40, None) == want
        assert status("moe_linear_backward", lin, A, A, A, A, A, A, None, A, 1 << 40, None) == want


def test_linear_pointer_and_workspace_refusals():
    lin = moe.make_linear(300, 512, 256, act="silu")
    big = 1 << 40
    ok = [A, A, A, A, A, A]                               # x w bias residual y pre
    for i in (0, 1, 4):
        bad = list(ok)
        bad[i] = None
        assert status("moe_linear", lin, *bad, A, big, None) == INVALID
    for i in range(6):
        bad = list(ok)
        bad[i] = A + 8
        assert status("moe_linear", lin, *bad, A, big, None) == INVALID
    need = moe.moe_linear_workspace_bytes(lin, moe.MOE_CALL_LINEAR)
    if need:
        assert status("moe_linear", lin, *ok, A, need - 1, None) == WORKSPACE
        assert status("moe_linear", lin, *ok, None, need, None) == WORKSPACE
        assert status("moe_linear", lin, *ok, A + 8, need, None) == WORKSPACE
    back = [A] * 7                                        # dy pre x w dx dw dbias
    for missing in ((0,), (1,), (2,), (3,), (4, 5, 6)):
        bad = [None if i in missing else A for i in range(7)]
        assert status("moe_linear_backward", lin, *bad, A, big, None) == INVALID
    for i in range(7):
        bad = list(back)
        bad[i] = A + 4
        assert status("moe_linear_backward", lin, *bad, A, big, None) == INVALID
    need = moe.moe_linear_workspace_bytes(lin, moe.MOE_CALL_LINEAR_BACKWARD)
    assert need > 0
    assert status("moe_linear_backward", lin, *back, A, need - 1, None) == WORKSPACE
    assert status("moe_linear_backward", lin, *back, None, need, None) == WORKSPACE
    assert status("moe_linear", moe.make_linear(0, 64, 64), None, None, None, None, None, None, None, 0, None) == 0
    n = ctypes.c_size_t(0)
    assert _lib.load().moe_linear_workspace_bytes(ctypes.byref(lin), moe.MOE_CALL_FORWARD, ctypes.byref(n)) == INVALID
    assert _lib.load().moe_linear_workspace_bytes(ctypes.byref(lin), moe.MOE_CALL_LINEAR, None) == INVALID
    s = shape()
    assert _lib.load().moe_workspace_bytes(ctypes.byref(s), moe.MOE_CALL_LINEAR, ctypes.byref(n)) == INVALID


def test_forward_routed_refusals():
    s = shape(n_experts=8, top_k=2)
    fn = "moe_forward_routed"
    ok = [A, A, A, None, A, A, A, None, None, None, A, None, None, A, 1 << 40]
    for i in (0, 1, 2, 4, 5, 6, 10):
        bad = list(ok)
        bad[i] = None
        assert status(fn, s, *bad, None) == INVALID
    assert status(fn, s, *ok[:13], None, 0, None) == WORKSPACE
    assert status(fn, s, *ok[:13], A, moe.moe_workspace_bytes(s, moe.MOE_CALL_FORWARD) - 1, None) == WORKSPACE
    capped = shape(n_experts=8, top_k=2, capacity=4, overflow="next_best")
    assert status(fn, capped, *ok, None) == INVALID       # the fallback round needs next_ids


def test_binding_refuses_wrong_tensors():
    lin = moe.make_linear(4, 64, 64)
    host = torch.empty(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device memory"):
        moe.moe_linear(lin, host, A, None, None, A)
    with pytest.raises(moe.MoEError, match="INVALID_ARG"):
        moe.moe_linear(lin, None, A, None, None, A)


# ---- the reference against differences and known values ----

ROUTERS = [dict(kind="softmax", renormalize=True), dict(kind="softmax", renormalize=False),
           dict(kind="sigmoid", renormalize=True), dict(kind="sigmoid", renormalize=False)]


@pytest.mark.parametrize("r", ROUTERS)
def test_reference_route_gradient_is_the_difference_quotient(r):
    rng = np.random.default_rng(5)
    T, E, k, scale = 3, 12, 4, 1.7
    x = rng.normal(size=(T, E))
    g, D = rng.normal(size=(T, k)), rng.normal(size=(T, E))
    ids = ref.route_scored(x, None, k, scale=scale, **r)[0]

    def loss(z):
        s = ref.scores(z, r["kind"])
        w = np.take_along_axis(s, ids, 1)
        if r["renormalize"]:
            w = w / w.sum(1, keepdims=True)
        return float((g * w * scale).sum() + (D * s).sum())

    grad = ref.route_scored_backward(x, ids, g, D, scale=scale, **r)
    h = 1e-6
    for t in range(T):
        for e in range(E):
            p, m = x.copy(), x.copy()
            p[t, e] += h
            m[t, e] -= h
            assert abs((loss(p) - loss(m)) / (2 * h) - grad[t, e]) < 1e-8


@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_reference_linear_gradient_is_the_difference_quotient(act):
    rng = np.random.default_rng(6)
    M, N, K, h = 3, 8, 8, 1e-6
    x, w, b, dy = (rng.normal(size=s) for s in ((M, K), (N, K), (N,), (M, N)))
    pre = ref.linear(x, w, b, None, act)[1]
    dx, dw, db, _ = ref.linear_backward(dy, pre, x, w, act)

    def loss(x_, w_, b_):
        return float((ref.linear(x_, w_, b_, None, act)[0] * dy).sum())

    for a, grad, at in ((x, dx, 0), (w, dw, 1), (b, db, 2)):
        for i in np.ndindex(*a.shape):
            p, m = a.copy(), a.copy()
            p[i] += h
            m[i] -= h
            args_p, args_m = [x, w, b], [x, w, b]
            args_p[at], args_m[at] = p, m
            assert abs((loss(*args_p) - loss(*args_m)) / (2 * h) - grad[i]) < 1e-7


def test_reference_combine_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(7)
    T, k, d = 4, 2, 8
    s2r = np.array([3, 0, 1, -1, 2, 4, -1, -1, 5, 6, 7, 8])       # shared rows last
    w, y, dy = rng.normal(size=(T, k)), rng.normal(size=(9, d)), rng.normal(size=(T, d))

    def loss(w_, y_):
        out = np.zeros((T, d))
        for t in range(T):
            for j in range(k):
                if s2r[t * k + j] >= 0:
                    out[t] += w_[t, j] * y_[s2r[t * k + j]]
            out[t] += y_[s2r[T * k + t]]
        return float((out * dy).sum())

    rows, dw = ref.combine_backward(dy, y, s2r, w, k, 1)
    h = 1e-6
    for a, at in ((w, 0), (y, 1)):
        for i in np.ndindex(*a.shape):
            p, m = a.copy(), a.copy()
            p[i] += h
            m[i] -= h
            q = (loss(p, y) - loss(m, y) if at == 0 else loss(w, p) - loss(w, m)) / (2 * h)
            assert abs(q - (dw[i] if at == 0 else rows[i[0]][i[1]])) < 1e-7


def test_reference_route_reproduces_the_worked_example():
    # the pages' router scores: experts 0 and 2 (0-based) with weights 0.6682 / 0.3318
    x = np.array([[2.1, 0.3, 1.4, -0.5, 0.0, 0.9, -1.2, 0.2]])
    ids, w, _, nxt = ref.route_scored(x, None, 2)
    assert list(ids[0]) == [0, 2] and list(nxt[0]) == [5, 1]
    assert np.allclose(w[0], [0.6682, 0.3318], atol=5e-5)


def test_reference_groups_bias_and_ties():
    x = np.array([[3.0, 0.0, 2.0, 2.0, 2.0, 2.0, 0.0, 0.0]])
    # groups of two: sums 3, 4, 4, 0 -> groups 1 and 2 (by score sums), ties to the lower index
    ids, _, _, nxt = ref.route_scored(x, np.zeros(8), 2, "sigmoid", 4, 2, 2)
    assert list(ids[0]) == [2, 3] and list(nxt[0]) == [4, 5]
    # one-expert rule: the group of the 3.0 comes first
    ids, _, _, nxt = ref.route_scored(x, None, 3, "softmax", 4, 2, 1)
    assert list(ids[0]) == [0, 2, 3] and list(nxt[0]) == [1, -1]
    bias = np.array([-np.inf, 0, 0, 0, 0, 0, 5.0, 0])
    ids, w, s, _ = ref.route_scored(x, bias, 2, "sigmoid")
    assert list(ids[0]) == [6, 2] and np.allclose(w[0].sum(), 1.0) and w[0, 0] < w[0, 1]
