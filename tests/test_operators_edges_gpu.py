"""GPU checks of the scored router and the dense product at their edges: NaN and infinite logits, groups
whose choices cancel, expert counts that are no multiple of 8, activations of fp32 operands over their
whole range, every tile shape of the forward product.

Tolerances count half steps (see test_operators_gpu); what a test needs beyond that is derived in it."""
import math
import pathlib
import re

import numpy as np
import pytest
import torch

import sparse_mixture_experts_topk_amd as moe
import test_operators_gpu as base
from oracle import operators as ref
from sparse_mixture_experts_topk_amd import runner, synthetic
from test_operators_gpu import BF16, DEV, F32, Out, close, cuda, f64, gen, normal, say

pytestmark = pytest.mark.gpu


# ---- logits that are no numbers ----

def unclean_logits(T, E, values):
    """Rows with every third, one, all but two and all logits replaced by each of `values` in turn."""
    x = normal(gen(101), T, E)
    for i, v in enumerate(values):
        x[4 * i, ::3] = v
        x[4 * i + 1, 5 + i] = v
        x[4 * i + 2, 2:] = v
        x[4 * i + 3] = v
    return x


def check_as(x, counts_as, k, kind, groups, bias, renorm):
    """Ids, weights, scores and both gradients of x are those of `counts_as` (fp64 reference)."""
    T, E = x.shape
    say(f"unclean {kind} groups={groups} bias={None if bias is None else float(bias.abs().max())} renorm={renorm}")
    n, kept, top = groups
    s, r = moe.make_shape(T, 64, 64, E, k), moe.make_router(kind, n, kept, top, renorm, 1.5)
    ids, w, sc = Out(T, k, dtype=torch.int32, fill=-77), Out(T, k), Out(T, E)
    nx = Out(T, 2, dtype=torch.int32, fill=-77)
    moe.moe_route_scored(s, r, cuda(x), cuda(bias), ids.t, w.t, sc.t, nx.t)
    g, D, dl = normal(gen(102), T, k), normal(gen(103), T, E), Out(T, E)
    moe.moe_route_scored_backward(s, r, cuda(x), ids.t, cuda(g), cuda(D), dl.t)
    torch.cuda.synchronize()
    want = ref.route_scored(f64(counts_as), f64(bias), k, kind, n, kept, top, renorm, 1.5)
    assert np.array_equal(ids.np(), want[0]), "ids"
    assert np.array_equal(nx.np(), want[3]), "next ids"
    # logits of N(0, 1), span below 10: exp's argument up to that many half steps, some ten roundings, the sum
    tol = 2 * F32 * (10 + 24)
    close(w.np(), want[1], tol * want[1] + 1e-37, "weights")
    close(sc.np(), want[2], tol * want[2] + 1e-37, "scores")
    wdl = ref.route_scored_backward(f64(counts_as), want[0], f64(g), f64(D), kind, renorm, 1.5)
    size = 1.5 * np.abs(f64(g)).max(1, keepdims=True) * (2 if renorm else 1) + np.abs(f64(D)).max(1, keepdims=True)
    close(dl.np(), wdl, 2 * tol * size, "dlogits")


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 4, 2), (8, 3, 1)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_nan_logit_counts_as_minus_infinity(kind, groups, renorm):
    T, E, k = 8, 40, 8
    x = unclean_logits(T, E, [float("nan")])
    x[4] = x[0]
    x[4, 1] = -float("inf")                                  # beside a masked one: equal, the lower index first
    as_masked = torch.where(torch.isnan(x), -float("inf"), x)
    favoured = torch.zeros(E)
    favoured[5], favoured[6] = 0.75, 0.25                    # 5 and 6: NaN in some of the rows
    for bias in (None, torch.zeros(E), normal(gen(104), E, std=0.05), favoured):
        check_as(x, as_masked, k, kind, groups, bias, renorm)


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("spread", [1e-4, 0.01, 1.0])
@pytest.mark.parametrize("size", [(33.0,), (0.5, 33.0, 1000.0)])
def test_route_groups_whose_choices_cancel_are_ordered_as_in_fp64(kind, spread, size):
    """Groups of two experts with biases +B and -B: each choice is rounded by B, their sum is far below it."""
    T, E, k, n, kept = 32768, 64, 8, 32, 12
    say(f"cancelling groups {kind} spread={spread} biases={size}")
    g = torch.Generator(device=DEV).manual_seed(18)
    x = torch.randn(T, E, device=DEV, generator=g) * spread
    b = torch.tensor([size[i % len(size)] for i in range(n)], device=DEV)
    b = torch.stack((b, -b), 1).flatten().contiguous()
    ids, w = Out(T, k, dtype=torch.int32, fill=-77), Out(T, k)
    moe.moe_route_scored(moe.make_shape(T, 64, 64, E, k), moe.make_router(kind, n, kept, 2), x, b, ids.t, w.t)
    z = x.double()
    c = (torch.sigmoid(z) if kind == "sigmoid" else torch.softmax(z, 1)) + b.double()
    of_group = c.view(T, n, 2).sum(2)
    best = of_group.sort(dim=1, descending=True, stable=True).indices[:, :kept]
    mask = torch.zeros(T, n, dtype=torch.bool, device=DEV).scatter_(1, best, True)
    c = torch.where(mask.repeat_interleave(2, 1), c, -float("inf"))
    want = c.sort(dim=1, descending=True, stable=True).indices[:, :k]
    off = (ids.t.long() != want).any(1)
    assert not off.any(), f"{int(off.sum())} of {T} tokens"


@pytest.mark.parametrize("kind", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups", [(1, 1, 1), (8, 4, 2), (8, 3, 1)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_infinite_logit_counts_as_the_largest_number(kind, groups, renorm):
    T, E, k = 12, 40, 8
    x = unclean_logits(T, E, [float("inf")])
    x[4] = x[0]
    x[4, 1], x[4, 2] = -float("inf"), float("nan")
    x[5, 3] = torch.finfo(torch.float32).max
    counts_as = torch.nan_to_num(x, nan=-float("inf"), posinf=torch.finfo(torch.float32).max, neginf=-float("inf"))
    for bias in (None, torch.zeros(E), normal(gen(104), E, std=0.05)):
        check_as(x, counts_as, k, kind, groups, bias, renorm)


# ---- nothing to do ----

def test_gradients_of_no_rows_through_the_binding():
    """Outputs of no elements, alone: nothing is written and nothing is refused."""
    say("no rows")
    e = torch.empty(0, 64, device=DEV, dtype=torch.bfloat16)
    w = torch.zeros(72, 64, device=DEV, dtype=torch.bfloat16)
    moe.moe_linear_backward(moe.make_linear(0, 72, 64), e, None, e, w, e, None, None)
    f, i = torch.empty(0, 2, device=DEV), torch.empty(0, device=DEV, dtype=torch.int32)
    moe.moe_combine_backward(moe.make_shape(0, 64, 64, 8, 2), e, f, i, f, e, None)
    moe.moe_combine_backward(moe.make_shape(0, 64, 64, 8, 2), e, f, i, f, None, f)
    torch.cuda.synchronize()


def test_route_looks_at_tokens_experts_and_k_alone():
    x, b = cuda(normal(gen(106), 50, 256)), cuda(normal(gen(107), 256, std=0.05))
    say("route with shapes of other types and widths")
    r, outs = moe.make_router("sigmoid", 8, 4, 2), []
    for kw in (dict(), dict(act_dtype="f32", w_dtype="f32"), dict(w_dtype="mxfp4", capacity=3), dict(d_model=100)):
        s = moe.make_shape(50, **{**dict(d_model=64, d_ff=64, n_experts=256, top_k=8), **kw})
        ids, w, dl = Out(50, 8, dtype=torch.int32, fill=-77), Out(50, 8), Out(50, 256)
        moe.moe_route_scored(s, r, x, b, ids.t, w.t)
        moe.moe_route_scored_backward(s, r, x, ids.t, w.t, None, dl.t)
        torch.cuda.synchronize()
        outs.append((ids.np(), w.np(), dl.np()))
    for o in outs[1:]:
        assert all(np.array_equal(g, want) for g, want in zip(o, outs[0]))


@pytest.mark.parametrize("kw", [dict(E=60), dict(T=5, E=12, k=3, shared=0), dict(T=33, E=100, k=6),
                                dict(T=50, E=12, k=2, shared=0, act_dtype="f32", w_dtype="f32")])
def test_scored_layer_of_expert_counts_that_are_no_multiple_of_8(kw):
    base.test_scored_layer_and_its_gate_gradient(kw)


def test_gate_gradient_of_12_experts_on_a_stream_of_its_own():
    cfg, inp, balance = base.layer(T=700, E=12, k=3)
    say("gate gradient of 12 experts on another stream")
    di = runner.DeviceInputs.from_host(inp)
    router, dy = moe.make_router(**base.ROUTER), cuda(normal(gen(105), 700, cfg.d_model, dtype=torch.bfloat16))
    st = runner.staged(di, router=router, balance_bias=cuda(balance))
    want = runner.gate_backward(di, st, router, dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    for stream in (side, side.cuda_stream):
        got = runner.gate_backward(di, st, router, dy, stream=stream)
        side.synchronize()
        for name in ("dx", "dw_gate", "dbias", "dlogits"):
            assert torch.equal(got[name], want[name]), name


def test_readme_example_of_the_scored_layer_runs():
    readme = pathlib.Path(__file__).resolve().parent.parent / "README.md"
    if not readme.exists():
        pytest.skip("a copy of the tree without its documents")
    code = [b for b in re.findall(r"```python\n(.*?)```", readme.read_text(), re.S) if "make_router" in b]
    say("the README's example")
    names = {"torch": torch, "moe": moe, "runner": runner, "synthetic": synthetic}
    exec(compile(code[0], "README.md", "exec"), names)
    torch.cuda.synchronize()
    assert len(code) == 1 and torch.equal(names["out"].y, names["st"]["y"])
    assert all(bool(torch.isfinite(names["grads"][n]).all()) for n in ("dx", "dw_gate", "dlogits"))
    assert bool(torch.isfinite(names["y"]).all())


def fp32_activation(act, span, out_dtype="f32", dtype="f32"):
    """(p, act(p), act'(p)) of 32768 values over +-span, the identity as weights: pre-activations are exact."""
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    p = torch.linspace(-span, span, 4096 * 8).to(dt).view(4096, 8)
    lin = moe.make_linear(4096, 8, 8, dtype=dtype, y_dtype=out_dtype, act=act)
    eye = cuda(torch.eye(8, dtype=dt))
    y = Out(4096, 8)
    moe.moe_linear(lin, cuda(p), eye, None, None, y.t, None, runner._bytes(moe.moe_linear_workspace_bytes(lin), DEV))
    if dtype != "f32":
        torch.cuda.synchronize()
        return f64(p), y.np(), None
    dx, dy = Out(4096, 8), torch.ones(4096, 8, device=DEV)
    moe.moe_linear_backward(lin, dy, cuda(p), None, eye, dx.t, None, None,
                            runner._bytes(moe.moe_linear_workspace_bytes(lin, moe.MOE_CALL_LINEAR_BACKWARD), DEV))
    torch.cuda.synchronize()
    return f64(p), y.np(), dx.np()


def sigmoid_pair(z):
    """sigmoid(z), 1 - sigmoid(z) in fp64."""
    e = np.exp(-np.abs(z))
    return np.where(z < 0, e, 1.0) / (1.0 + e), np.where(z < 0, 1.0, e) / (1.0 + e)


# sigmoid from e^-|z|: e to 3 half steps (exp2 to 1 ulp, one rounding), 1 + e one more, the reciprocal to 1 ulp,
# one product: 3 / (1 + e) + 1 + 2 + 1 <= 7 relative, 1 - sigmoid likewise
SIGMOID = 7 * F32


def test_silu_of_fp32_operands_over_the_whole_range():
    p, y, dx = fp32_activation("silu", 86.0)
    s, below = sigmoid_pair(p)
    close(y, p * s, 1.05 * (SIGMOID + F32) * np.abs(p * s) + 2.0 ** -120, "silu")
    slope = s * (1 + p * below)
    # s, the rounding of 1 + p below, the product; below inside the bracket
    close(dx, slope, 1.05 * ((SIGMOID + 2 * F32) * np.abs(slope) + SIGMOID * s * np.abs(p) * below) + 2.0 ** -120, "slope")


def test_gelu_tanh_of_fp32_operands_over_the_whole_range():
    p, y, dx = fp32_activation("gelu_tanh", 10.0)
    a, b = 2 * math.sqrt(2 / math.pi), 0.044715
    s, below = sigmoid_pair(a * (p + b * p ** 3))
    close(y, p * s, 1.05 * (SIGMOID + F32) * np.abs(p * s) + 2.0 ** -120, "gelu_tanh")
    inner = np.abs(p) * s * below * a * (1 + 3 * b * p * p)
    # both factors, four products, a and 3 b p^2 with two roundings and a constant's: 7 + 7 + 4 + 1 + 4
    tol = 23 * F32 * inner + SIGMOID * s + F32 * np.abs(s + np.sign(p) * inner)
    close(dx, s + np.sign(p) * inner, 1.05 * tol + 2.0 ** -120, "slope")


def test_gelu_of_fp32_operands_over_the_whole_range():
    p, y, dx = fp32_activation("gelu", 13.0)
    tail = np.array([0.5 * math.erfc(abs(t) / math.sqrt(2)) for t in p.ravel()]).reshape(p.shape)
    cdf, phi = np.where(p < 0, tail, 1 - tail), np.exp(-0.5 * p * p) / math.sqrt(2 * math.pi)
    # the tail's polynomial with a reciprocal to 1 ulp 6.4e-7, e^(-p^2/2) 3 half steps, their product one
    e_tail = (6.4e-7 + 4 * F32) * tail
    e_cdf = e_tail + np.where(p < 0, 0.0, F32 * cdf)
    close(y, p * cdf, 1.05 * (np.abs(p) * e_cdf + F32 * np.abs(p) * cdf) + 2.0 ** -120, "gelu")
    slope = cdf + p * phi
    close(dx, slope, 1.05 * (e_cdf + 4.5 * F32 * np.abs(p) * phi + F32 * np.abs(slope)) + 2.0 ** -120, "slope")


@pytest.mark.parametrize("act,span", [("silu", 86.0), ("gelu", 13.0), ("gelu_tanh", 10.0)])
def test_activation_tails_of_bf16_operands(act, span):
    """fp32 outputs of bf16 operands: exact to a few half steps of the value and of exp's argument."""
    p, y, _ = fp32_activation(act, span, dtype="bf16")
    want = ref.activation(p, act)[0]
    if act == "gelu":                                        # (1 + erf cancels in the reference)
        want = p * np.array([0.5 * math.erfc(-t / math.sqrt(2)) for t in p.ravel()]).reshape(p.shape)
    if act == "gelu_tanh":                                   # (1 + tanh too)
        z = 2 * math.sqrt(2 / math.pi) * (p + 0.044715 * p ** 3)
        want = p * sigmoid_pair(z)[0]
    # the argument's roundings: |p| by its product with log2 e; p^2 / 2 by two products; 2 u by seven of its terms
    arg = {"silu": 1.25 * np.abs(p), "gelu": 2.5 * p * p / 2,
           "gelu_tanh": 8 * 2 * math.sqrt(2 / math.pi) * np.abs(p + 0.044715 * p ** 3)}[act]
    close(y, want, 1.05 * (6.4e-7 + (9 + arg) * F32) * np.abs(want) + 2.0 ** -120, act)


@pytest.mark.parametrize("dims", [(33, 4096, 4096), (64, 4096, 4096), (65, 4096, 4096), (129, 4096, 4096), (16, 256, 4096)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_linear_repeats_bit_for_bit(dims, dtype):
    """Whatever the workspace held before."""
    M, N, K = dims
    say(f"repeated {dtype} M={M} N={N} K={K}")
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x, w = base.device_normal(1, M, K, dtype=dt), base.device_normal(2, N, K, std=K ** -0.5, dtype=dt)
    lin = moe.make_linear(M, N, K, dtype=dtype, y_dtype="f32")
    ws = runner._bytes(moe.moe_linear_workspace_bytes(lin), DEV)
    outs = []
    for fill in (0xFF, 0, 77):
        if ws is not None:
            ws.fill_(fill)
        y = torch.empty(M, N, device=DEV)
        moe.moe_linear(lin, x, w, None, None, y, None, ws)
        outs.append(y)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# each tile shape of the forward product: taken whole in part of a round, whole over several rounds,
# cut along the contraction and joined, with and without full rounds before
@pytest.mark.parametrize("dims", [(40, 256, 72), (40, 256, 2056), (1900, 1032, 72), (1100, 1000, 4104), (2500, 1544, 2056),
                                  (256, 4096, 4096), (2500, 1544, 72), (512, 14336, 4096), (700, 4096, 8200),
                                  (384, 4096, 14336), (2049, 4096, 4104), (2049, 4096, 72), (2500, 4096, 8200),
                                  (4097, 4096, 4104), (8192, 14336, 4096)])
def test_linear_in_every_tile_shape(dims):
    """Against 64-bit products on the device: bare with fp32 output, and with bias, silu, residual and pre."""
    M, N, K = dims
    say(f"linear tiles M={M} N={N} K={K}")
    x, w = base.device_normal(1, M, K), base.device_normal(2, N, K, std=K ** -0.5)
    b, r = base.device_normal(3, N, dtype=torch.float32), base.device_normal(4, M, N)
    x64, wt64 = x.double(), w.double().t().contiguous()
    want = x64 @ wt64
    dot = (K + 4) * 2.0 ** -23 * (x64.abs() @ wt64.abs() + b.double().abs())

    def inside(got, want, tol, what):
        off = (got.double() - want).abs() - tol
        assert not torch.isnan(got).any() and off.max() <= 0, f"{what}: {float(off.max())} past the tolerance"

    for out in ("f32", "bf16"):
        whole = out == "bf16"
        lin = moe.make_linear(M, N, K, y_dtype=out, act="silu" if whole else "none")
        n = moe.moe_linear_workspace_bytes(lin)
        ws = Out(n, dtype=torch.uint8, fill=77) if n else None
        if ws:
            ws.t.fill_(0xFF)
        y = Out(M, N, dtype=torch.bfloat16 if whole else torch.float32)
        p = Out(M, N, dtype=torch.bfloat16)
        moe.moe_linear(lin, x, w, b if whole else None, r if whole else None, y.t, p.t if whole else None,
                       ws.t if ws else None)
        torch.cuda.synchronize()
        for o in (y, p, ws):
            assert o is None or bool((o.flat[o.n:] == o.fill).all()), "written past the end"
        if whole:
            want += b.double()
            inside(p.t, want, (dot + BF16 * want.abs()) * (1 + BF16), "pre")
            value = want * torch.sigmoid(want) + r.double()
            tol = 1.13 * dot + 2.0 ** -19 * (1 + want.abs()) + BF16 * value.abs() + 2 * F32 * r.double().abs()
            inside(y.t, value, tol * (1 + BF16), "y")
        else:
            inside(y.t, want, dot + 2 * F32 * want.abs(), "y")
