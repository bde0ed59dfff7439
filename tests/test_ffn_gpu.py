"""GPU parity of the gated feed-forward block, its gradients, the permutation's gradient and clipping with the
fp64 reference, through the public entry points.

Tolerances.  h(t) is half a step of a type, relative to the value: bf16 2^-8, fp32 2^-24.  A dot product of n
terms on the matrix cores, whose adder may truncate, is held to (n + 4) 2^-23 sum |a b| (fp32 operands: their
products round too, (n + 4) 2^-22); each activation and its slope to 2^-19 (1 + |p|).  An activation's slope is
under 1.2 and its second derivative under 1.6, so a pre-activation that is off by e moves the value by 1.2 e.
Errors pass through the later products with the absolute values of what they meet, and each stored value adds
its half step."""
import math
import sys

import numpy as np
import pytest
import torch

import sparse_mixture_experts_topk_amd as moe
from oracle import ffn as ref
from oracle.operators import activation
from sparse_mixture_experts_topk_amd import runner, synthetic

pytestmark = pytest.mark.gpu

BF16, F32 = 2.0 ** -8, 2.0 ** -24
DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]
GUARD = 32      # elements behind an output that must stay as they were


def say(msg):
    print(f"\n[case] {msg}", flush=True)
    sys.stdout.flush()


def gen(seed):
    return torch.Generator().manual_seed(seed)


def normal(g, *shape, std=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g) * std).to(dtype)


def f64(t):
    return None if t is None else t.detach().cpu().double().numpy()


def cuda(t):
    return None if t is None else t.to(DEV)


class Out:
    """A device output with a guard behind it."""

    def __init__(self, *shape, dtype=torch.float32, fill=-7.0):
        n = int(np.prod(shape))
        self.flat = torch.full((n + GUARD,), fill, dtype=dtype, device=DEV)
        self.fill, self.n = fill, n
        self.t = self.flat[:n].view(*shape)

    def np(self):
        guard = self.flat[self.n:].cpu().float().numpy()
        assert (guard == self.fill).all(), "written past the end"
        return f64(self.t)


def close(got, want, tol, what):
    assert got.shape == want.shape
    if got.size == 0:
        return
    assert np.isfinite(got).all(), f"{what}: not finite"
    off = np.abs(got - want) - tol
    at = np.unravel_index(off.argmax(), off.shape)
    assert off.max() <= 0, f"{what}{at}: {got[at]} against {want[at]}, allowed {np.broadcast_to(tol, got.shape)[at]}"


def workspace(n):
    """One with a guard, full of NaN: contents need no initialisation."""
    ws = Out(n, dtype=torch.uint8, fill=77) if n else None
    if ws:
        ws.t.fill_(0xFF)
    return ws


def steps(dtype):
    return (BF16, 2.0 ** -23) if dtype == "bf16" else (F32, 2.0 ** -22)


# ---- groups ----

def even(M, G):
    return [M * e // G for e in range(G + 1)]


def uneven(M, G, seed, behind=0, before=0):
    """Offsets with empty groups; `before` and `behind` rows of no group."""
    w = torch.rand(G, generator=gen(seed)) ** 3
    w[torch.rand(G, generator=gen(seed + 1)) < 0.25] = 0
    if w.sum() == 0:
        w[0] = 1
    c = torch.cumsum(w / w.sum(), 0) * (M - behind - before)
    return [before] + [before + int(v) for v in c[:-1].round()] + [M - behind]


def off(offsets):
    return None if offsets is None else torch.tensor(offsets, dtype=torch.int32, device=DEV)


def outside(M, offsets):
    inside = np.zeros(M, dtype=bool)
    if offsets is None:
        inside[:] = True
    else:
        inside[offsets[0]:offsets[-1]] = True
    return ~inside


# M, d_model, d_ff, groups, offsets: one row, widths of less than a tile, odd tails of rows, of terms and of
# channels, several tiles, groups that are empty, of one row, and of all rows
SHAPES = [
    (1, 8, 8, 1, None), (1, 512, 264, 1, None), (2, 64, 1032, 1, None), (3, 72, 40, 1, None), (17, 136, 4104, 1, None),
    (31, 2056, 128, 1, None), (32, 256, 256, 1, None), (33, 128, 264, 1, None), (64, 64, 64, 1, None),
    (129, 200, 520, 1, None), (257, 520, 136, 1, None), (300, 1032, 520, 1, None), (700, 264, 1288, 1, [0, 700]),
    (64, 72, 136, 8, even(64, 8)), (5, 64, 64, 8, [0, 0, 1, 1, 1, 3, 3, 5, 5]), (130, 128, 200, 3, [0, 0, 130, 130]),
    (300, 136, 264, 5, uneven(300, 5, 1, behind=7)), (300, 264, 136, 9, uneven(300, 9, 2, behind=3, before=5)),
    (1000, 72, 72, 60, uneven(1000, 60, 3)), (77, 64, 136, 257, uneven(77, 257, 4)), (16, 136, 72, 64, [0] * 64 + [16]),
    (40, 64, 64, 4, [40] * 5), (900, 520, 392, 2, [0, 643, 900]), (1500, 192, 328, 4, [0, 256, 512, 1283, 1500]),
]


def gate_up_case(M, d, F, G, offsets, act="silu", dtype="bf16", keep=True, std=1.0, seed=0):
    say(f"gate/up {dtype} M={M} d={d} F={F} G={G} {act} keep={keep} seed={seed}")
    g = gen(seed + M + d + F + G)
    dt, (step, per) = DT[dtype], steps(dtype)
    x = normal(g, M, d, dtype=dt)
    w1, w3 = (normal(g, G, F, d, std=std * d ** -0.5, dtype=dt) for _ in range(2))
    away = outside(M, offsets)
    x[torch.from_numpy(away)] = float("nan")             # rows of no group are not read
    f = moe.make_ffn(M, d, F, G, dtype, act)
    ws = workspace(moe.moe_ffn_workspace_bytes(f, moe.MOE_CALL_FFN_GATE_UP))
    h = Out(M, F, dtype=dt)
    p1, p3 = (Out(M, F, dtype=dt) if keep else None for _ in range(2))
    moe.moe_ffn_gate_up(f, cuda(x), off(offsets), cuda(w1), cuda(w3), h.t, p1.t if keep else None, p3.t if keep else None,
                        ws.t if ws else None)
    torch.cuda.synchronize()
    got = {"h": h.np()}
    if keep:
        got.update(g=p1.np(), u=p3.np())
    if ws:
        ws.np()
    for name, v in got.items():
        assert (v[away] == -7.0).all(), f"{name}: rows of no group"
    for e, a, b in ref.spans(offsets, G, M):
        xs, a1, a3 = f64(x[a:b]), f64(w1[e]), f64(w3[e])
        wh, wg, wu = ref.gate_up(xs, a1, a3, act)
        eg, eu = ((d + 4) * per * (np.abs(xs) @ np.abs(q).T) for q in (a1, a3))
        av = np.abs(activation(wg, act)[0])
        ea = 1.2 * eg + (0.0 if act in ("none", "relu") else 2.0 ** -19 * (1 + np.abs(wg)))
        tol = av * eu + np.abs(wu) * ea + ea * eu + 4 * F32 * np.abs(wh)
        close(got["h"][a:b], wh, tol * (1 + step) + step * np.abs(wh), f"h of group {e}")
        if keep:
            close(got["g"][a:b], wg, eg * (1 + step) + step * np.abs(wg), f"g of group {e}")
            close(got["u"][a:b], wu, eu * (1 + step) + step * np.abs(wu), f"u of group {e}")
    return got


@pytest.mark.parametrize("case", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gate_up(case, dtype):
    gate_up_case(*case, dtype=dtype)
    gate_up_case(*case, dtype=dtype, act="gelu_tanh", keep=False, seed=1)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_gate_up_activations(act, dtype):
    for std in (0.1, 3.0):
        gate_up_case(5, 72, 136, 1, None, act, dtype, std=std)
        gate_up_case(300, 264, 200, 3, [0, 100, 100, 300], act, dtype, std=std)


def backward_case(M, d, F, G, offsets, act="silu", dtype="bf16", outputs="dx dw13 dw2", std=1.0, seed=0):
    say(f"backward {dtype} M={M} d={d} F={F} G={G} {act} [{outputs}] seed={seed}")
    outputs = outputs.split()
    g = gen(seed + M + d + F + G)
    dt, (step, per) = DT[dtype], steps(dtype)
    x, dy = normal(g, M, d, dtype=dt), normal(g, M, d, dtype=dt)
    p, q = normal(g, M, F, std=std, dtype=dt), normal(g, M, F, dtype=dt)
    h = (torch.from_numpy(activation(f64(p), act)[0]) * q.double()).to(dt)
    w1, w3 = (normal(g, G, F, d, std=F ** -0.5, dtype=dt) for _ in range(2))
    w2 = normal(g, G, d, F, std=d ** -0.5, dtype=dt)
    away = outside(M, offsets)
    for t in (x, dy, p, q, h):
        t[torch.from_numpy(away)] = float("nan")
    f = moe.make_ffn(M, d, F, G, dtype, act)
    ws = workspace(moe.moe_ffn_workspace_bytes(f, moe.MOE_CALL_FFN_BACKWARD))
    dx, dw1, dw3, dw2 = Out(M, d, dtype=dt), Out(G, F, d, dtype=dt), Out(G, F, d, dtype=dt), Out(G, d, F, dtype=dt)
    has = {n: n in outputs for n in ("dx", "dw13", "dw2")}
    inner = has["dx"] or has["dw13"]
    moe.moe_ffn_backward(
        f, cuda(dy), off(offsets), cuda(x) if has["dw13"] else None, cuda(p) if inner else None,
        cuda(q) if inner else None, cuda(h) if has["dw2"] else None, cuda(w1) if has["dx"] else None,
        cuda(w3) if has["dx"] else None, cuda(w2) if inner else None, dx.t if has["dx"] else None,
        dw1.t if has["dw13"] else None, dw3.t if has["dw13"] else None, dw2.t if has["dw2"] else None, ws.t)
    torch.cuda.synchronize()
    ws.np()
    got = {"dx": dx.np(), "dw1": dw1.np(), "dw3": dw3.np(), "dw2": dw2.np()}
    for n, v in got.items():
        if not has["dw13" if n in ("dw1", "dw3") else n]:
            assert (v == -7.0).all(), f"{n} was not asked for"
    if has["dx"]:
        assert (got["dx"][away] == -7.0).all(), "rows of no group"
    full = {e: (a, b) for e, a, b in ref.spans(offsets, G, M)}
    for e in range(G):
        if e not in full:
            for n in ("dw1", "dw3") if has["dw13"] else ():
                assert (got[n][e] == 0).all(), n
            if has["dw2"]:
                assert (got["dw2"][e] == 0).all()
            continue
        a, b = full[e]
        ys, xs, ps, qs, hs = (f64(t[a:b]) for t in (dy, x, p, q, h))
        a1, a3, a2 = f64(w1[e]), f64(w3[e]), f64(w2[e])
        r = ref.backward(ys, xs, ps, qs, hs, a1, a3, a2, act)
        n = b - a
        if has["dw2"]:
            tol = (n + 4) * per * (np.abs(ys).T @ np.abs(hs))
            close(got["dw2"][e], r["dw2"], tol * (1 + step) + step * np.abs(r["dw2"]), f"dw2 of group {e}")
        if not inner:
            continue
        edh = (d + 4) * per * (np.abs(ys) @ np.abs(a2))
        value, slope = (np.abs(v) for v in activation(ps, act))
        ea = 0.0 if act in ("none", "relu") else 2.0 ** -19 * (1 + np.abs(ps))
        adh = np.abs(r["dh"])
        edg = np.abs(qs) * (slope * edh + (adh + edh) * ea) + 4 * F32 * np.abs(r["dg"])
        edu = value * edh + (adh + edh) * ea + 4 * F32 * np.abs(r["du"])
        edg, edu = edg * (1 + step) + step * np.abs(r["dg"]), edu * (1 + step) + step * np.abs(r["du"])
        adg, adu = np.abs(r["dg"]) + edg, np.abs(r["du"]) + edu
        if has["dx"]:
            w = np.abs(a1), np.abs(a3)
            tol = edg @ w[0] + edu @ w[1] + (2 * F + 4) * per * (adg @ w[0] + adu @ w[1])
            close(got["dx"][a:b], r["dx"], tol * (1 + step) + step * np.abs(r["dx"]), f"dx of group {e}")
        if has["dw13"]:
            for name, err, size in (("dw1", edg, adg), ("dw3", edu, adu)):
                tol = err.T @ np.abs(xs) + (n + 4) * per * (size.T @ np.abs(xs))
                close(got[name][e], r[name], tol * (1 + step) + step * np.abs(r[name]), f"{name} of group {e}")
    return got


@pytest.mark.parametrize("case", SHAPES)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward(case, dtype):
    backward_case(*case, dtype=dtype)


@pytest.mark.parametrize("outputs", ["dx", "dw13", "dw2", "dx dw13", "dx dw2", "dw13 dw2"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_outputs_one_by_one(outputs, dtype):
    for case in ((70, 136, 264, 1, None), (300, 136, 264, 5, uneven(300, 5, 1, behind=7))):
        got = backward_case(*case, dtype=dtype, outputs=outputs)
        assert got is not None


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_backward_activations(act, dtype):
    for std in (0.1, 3.0):
        backward_case(5, 72, 136, 1, None, act, dtype, std=std)
        backward_case(300, 264, 200, 3, [0, 100, 100, 300], act, dtype, std=std)


def test_backward_of_no_rows_is_zero():
    f = moe.make_ffn(0, 64, 72, 3)
    dw1, dw3 = Out(3, 72, 64, dtype=torch.bfloat16), Out(3, 72, 64, dtype=torch.bfloat16)
    dw2 = Out(3, 64, 72, dtype=torch.bfloat16)
    moe.moe_ffn_backward(f, None, None, None, None, None, None, None, None, None, None, dw1.t, dw3.t, dw2.t)
    torch.cuda.synchronize()
    assert all((o.np() == 0).all() for o in (dw1, dw3, dw2))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_groups_do_not_see_each_other(dtype):
    """A group of NaN rows, or of NaN weights, between others: theirs are as without it."""
    dt = DT[dtype]
    M, d, F, G, offsets = 330, 136, 200, 3, [0, 101, 230, 330]
    g = gen(90)
    t = dict(x=normal(g, M, d, dtype=dt), dy=normal(g, M, d, dtype=dt), w1=normal(g, G, F, d, std=0.1, dtype=dt),
             w3=normal(g, G, F, d, std=0.1, dtype=dt), w2=normal(g, G, d, F, std=0.1, dtype=dt))
    f = moe.make_ffn(M, d, F, G, dtype)

    def run(t):
        t = {n: cuda(v) for n, v in t.items()}
        e = lambda *s: torch.zeros(*s, dtype=dt, device=DEV)          # noqa: E731
        o = dict(h=e(M, F), p1=e(M, F), p3=e(M, F), dx=e(M, d), dw1=e(G, F, d), dw3=e(G, F, d), dw2=e(G, d, F))
        n = max(moe.moe_ffn_workspace_bytes(f, c) for c in (moe.MOE_CALL_FFN_GATE_UP, moe.MOE_CALL_FFN_BACKWARD))
        ws = runner._bytes(n, DEV)
        moe.moe_ffn_gate_up(f, t["x"], off(offsets), t["w1"], t["w3"], o["h"], o["p1"], o["p3"], ws)
        moe.moe_ffn_backward(f, t["dy"], off(offsets), t["x"], o["p1"], o["p3"], o["h"], t["w1"], t["w3"], t["w2"],
                             o["dx"], o["dw1"], o["dw3"], o["dw2"], ws)
        torch.cuda.synchronize()
        return o

    clean = run(t)
    for spoil in (("x", slice(101, 230)), ("dy", slice(101, 230)), ("w1", 1), ("w2", 1), ("w3", 1)):
        bad = {n: v.clone() for n, v in t.items()}
        bad[spoil[0]][spoil[1]] = float("nan")
        o = run(bad)
        for n in ("h", "p1", "p3", "dx"):
            assert torch.equal(o[n][:101], clean[n][:101]) and torch.equal(o[n][230:], clean[n][230:]), (spoil, n)
        for n in ("dw1", "dw3", "dw2"):
            assert torch.equal(o[n][0], clean[n][0]) and torch.equal(o[n][2], clean[n][2]), (spoil, n)
        assert torch.isnan(o["dx"][101:230]).all()


def test_gate_up_keeps_nan_and_infinities_in_their_rows():
    for M in (3, 200):
        x, w = torch.ones(M, 64, dtype=torch.bfloat16), torch.ones(1, 72, 64, dtype=torch.bfloat16)
        x[2, 5] = float("nan")
        x[0, 1] = float("inf")
        f = moe.make_ffn(M, 64, 72)
        h = Out(M, 72, dtype=torch.bfloat16)
        ws = runner._bytes(moe.moe_ffn_workspace_bytes(f), DEV)
        moe.moe_ffn_gate_up(f, cuda(x), None, cuda(w), cuda(w), h.t, None, None, ws)
        torch.cuda.synchronize()
        assert torch.isnan(h.t[2]).all() and torch.isinf(h.t[0]).all()
        assert torch.isfinite(h.t[1]).all() and torch.isfinite(h.t[3:]).all()


def test_offsets_out_of_range_are_bounded():
    """Offsets that no permutation writes stay inside the buffers."""
    M, d, F = 100, 64, 72
    g = gen(91)
    x, w = normal(g, M, d, dtype=torch.bfloat16), normal(g, 3, F, d, std=0.1, dtype=torch.bfloat16)
    f = moe.make_ffn(M, d, F, 3)
    ws = runner._bytes(moe.moe_ffn_workspace_bytes(f), DEV)
    for given, read in (([-50, 40, 30, 70], [0, 40, 40, 70]), ([10, 20, 1 << 30, 50], [10, 20, 100, 100]),
                        ([200, 300, 400, 500], [100] * 4)):
        a, b = Out(M, F, dtype=torch.bfloat16), Out(M, F, dtype=torch.bfloat16)
        moe.moe_ffn_gate_up(f, cuda(x), off(given), cuda(w), cuda(w), a.t, None, None, ws)
        moe.moe_ffn_gate_up(f, cuda(x), off(read), cuda(w), cuda(w), b.t, None, None, ws)
        torch.cuda.synchronize()
        assert np.array_equal(a.np(), b.np())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_group_with_bounds(dtype):
    """Given bounds of the one group: few rows (streamed) and more, none at all."""
    for M, offsets in ((20, [4, 15]), (20, [0, 0]), (20, [20, 20]), (32, [0, 32]), (200, [7, 180]), (200, [100, 100]),
                       (1, [0, 1]), (1, [1, 1])):
        gate_up_case(M, 136, 264, 1, offsets, dtype=dtype)
        backward_case(M, 136, 264, 1, offsets, dtype=dtype)


@pytest.mark.parametrize("d,F", [(1 << 18, 8), (8, 1 << 18)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_the_widest_channels(d, F, dtype):
    for M, G, offsets in ((5, 1, None), (40, 2, [0, 3, 40])):
        gate_up_case(M, d, F, G, offsets, dtype=dtype)
        backward_case(M, d, F, G, offsets, dtype=dtype)


@pytest.mark.parametrize("dims", [(33, 4096, 512, 1), (500, 392, 264, 4), (3000, 264, 136, 2), (90, 104, 1008, 200), (7, 512, 64, 1)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_repeats_bit_for_bit(dims, dtype):
    a, b = (gate_up_case(*dims, off_list, dtype=dtype) for off_list in [uneven(dims[0], dims[3], 5)] * 2)
    assert all(np.array_equal(a[n], b[n]) for n in a)
    a, b = (backward_case(*dims, off_list, dtype=dtype) for off_list in [uneven(dims[0], dims[3], 5)] * 2)
    assert all(np.array_equal(a[n], b[n]) for n in a)


# ---- gradient of the permutation ----

def rows_of(T, k, S, drop, seed):
    g = gen(seed)
    kept = torch.rand(T * k, generator=g) >= drop
    row = torch.full((T * k,), -1, dtype=torch.int64)
    row[kept] = torch.randperm(int(kept.sum()), generator=g)
    if S:
        row = torch.cat((row, int(kept.sum()) + torch.arange(T)))
    return row.to(torch.int32)


@pytest.mark.parametrize("T,d,k,S", [(1, 64, 1, 0), (1, 4096, 2, 0), (7, 128, 2, 1), (61, 4096, 2, 0), (33, 192, 8, 1),
                                     (50, 64, 5, 0), (19, 320, 3, 1), (23, 704, 4, 0), (9, 1216, 6, 1), (5, 2112, 7, 0)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("drop", [0.0, 0.4, 1.0])
def test_permute_backward(T, d, k, S, dtype, drop):
    g = gen(T + d + k)
    dt = DT[dtype]
    s2r = rows_of(T, k, S, drop, T + d)
    dxp = normal(g, T * (k + S), d, dtype=dt)
    dxp[int(s2r.max()) + 1:] = float("nan") if drop else 0.0         # rows no slot points to; row 0 may be one
    add = normal(g, T, d, dtype=dt)
    s = moe.make_shape(T, d, 64, 8, k, act_dtype=dtype, w_dtype=dtype, n_shared=S)
    for a in (None, add):
        say(f"permute backward {dtype} T={T} d={d} k={k} S={S} drop={drop} addend={a is not None}")
        o = Out(T, d, dtype=dt)
        moe.moe_permute_backward(s, cuda(dxp), cuda(s2r), cuda(a), o.t)
        torch.cuda.synchronize()
        want, size = ref.permute_backward(f64(dxp), s2r.numpy(), f64(a), T, k, S)
        step = steps(dtype)[0]
        close(o.np(), want, (k + S) * F32 * size * (1 + step) + step * np.abs(want), "dx")
    mine = cuda(add).clone()
    moe.moe_permute_backward(s, cuda(dxp), cuda(s2r), mine, mine)    # onto the addend
    torch.cuda.synchronize()
    assert torch.equal(mine, o.t)


# ---- norm and clipping ----

def clip_case(grads, max_norm, in_place=False, outs=None):
    """grads: device tensors."""
    say(f"clip {[(tuple(t.shape), str(t.dtype)[6:], t.data_ptr() % 16) for t in grads[:8]]} x{len(grads)} to {max_norm}")
    src = [f64(t) for t in grads]
    total, n, want = ref.clip(src, max_norm)
    lst = moe.make_tensors(grads)
    ws = workspace(moe.moe_grad_norm_workspace_bytes(lst))
    S, N = Out(1, dtype=torch.float64), Out(1)
    moe.moe_grad_norm(lst, S.t, N.t, ws.t if ws else None)
    if in_place:
        out = grads
    else:
        out = [torch.full_like(t, -7.0) for t in grads] if outs is None else outs
    moe.moe_grad_clip(lst, None if in_place else out, S.t, max_norm)
    torch.cuda.synchronize()
    if ws:
        ws.np()
    # fp64 sums of up to 2^30 terms
    close(S.np(), np.array([total]), 2.0 ** -23 * 2.0 ** -20 * total, "sum of squares")
    close(N.np(), np.array([n]), F32 * n * 1.001 + 1e-45, "norm")
    for i, (o, w) in enumerate(zip(out, want)):
        step = BF16 if o.dtype is torch.bfloat16 else F32
        tiny = 2.0 ** -133 if o.dtype is torch.bfloat16 else 2.0 ** -149     # steps below the normal range
        # (bf16 values pass fp32 on the way: its half step beside theirs)
        close(f64(o), w, (step + 2 * F32) * np.abs(w) + tiny, f"tensor {i}")
    return out


def grads_of(seed, *spec):
    g = gen(seed)
    return [cuda(normal(g, n, std=0.01 * (i % 3 + 1), dtype=DT[dt])) for i, (n, dt) in enumerate(spec)]


LISTS = [
    [(1, "f32")], [(1, "bf16")], [(7, "bf16"), (9, "f32")], [(8, "bf16"), (4, "f32"), (16384, "bf16"), (16383, "bf16")],
    [(16385, "bf16"), (8193, "f32"), (0, "f32"), (3, "bf16")], [(100003, "f32"), (700001, "bf16"), (5, "f32")],
    [(4096 * 17, "bf16")] * 3, [(1 + 13 * i, "bf16" if i % 2 else "f32") for i in range(301)],
    [(0, "f32"), (0, "bf16")],
]


@pytest.mark.parametrize("spec", LISTS)
@pytest.mark.parametrize("in_place", [False, True])
def test_clip(spec, in_place):
    n = math.sqrt(sum(n * (0.01 * (i % 3 + 1)) ** 2 for i, (n, _) in enumerate(spec)))
    for share in (0.3, 2.0, 0.0):
        clip_case(grads_of(100, *spec), n * share, in_place)


def test_clip_of_tensors_that_begin_anywhere():
    """Slices of one buffer, on and off 16-byte boundaries, their neighbours left as they were."""
    for dt, size in ((torch.bfloat16, 2), (torch.float32, 4)):
        for start in range(0, 16 // size):
            for n in (1, 2, 3, 7, 8, 9, 15, 16, 17, 100, 20011):
                base = cuda(normal(gen(start + n), n + 64, std=0.1, dtype=dt))
                keep = base.clone()
                view = base[start:start + n]
                clip_case([view], 0.05, in_place=True)
                assert torch.equal(base[:start], keep[:start]) and torch.equal(base[start + n:], keep[start + n:])
                for shift in (start, (start + 1) % (16 // size)):        # an output of equal, of other alignment
                    out = torch.full((n + 64,), -7.0, dtype=dt, device=DEV)
                    clip_case([keep[start:start + n]], 0.05, outs=[out[shift:shift + n]])
                    assert (out[:shift] == -7).all() and (out[shift + n:] == -7).all()


def test_clip_extremes():
    big, small = torch.full((1000,), 1e30, device=DEV), torch.full((1000,), 1e-30, device=DEV)
    clip_case([big.clone(), small.clone()], 1.0)
    clip_case([small.clone()], 1e-32)
    clip_case([big.to(torch.bfloat16), small.to(torch.bfloat16)], 1e3)
    clip_case([torch.zeros(100, device=DEV)], 0.0)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_a_norm_that_is_not_finite_scales_nothing(bad):
    a, b = cuda(normal(gen(1), 5000)), cuda(normal(gen(2), 77, dtype=torch.bfloat16))
    a[4321] = bad
    want = [a.clone(), b.clone()]
    S, N = torch.zeros(1, dtype=torch.float64, device=DEV), torch.zeros(1, device=DEV)
    lst = moe.make_tensors([a, b])
    outs = [torch.empty_like(a), torch.empty_like(b)]
    moe.moe_grad_norm(lst, S, N, runner._bytes(moe.moe_grad_norm_workspace_bytes(lst), DEV))
    moe.moe_grad_clip(lst, outs, S, 0.5)
    moe.moe_grad_clip(lst, None, S, 0.5)
    torch.cuda.synchronize()
    assert (torch.isnan if bad != bad else torch.isinf)(N).all()
    for got in (outs, [a, b]):
        for o, w in zip(got, want):
            assert torch.equal(o.nan_to_num(9.0, 8.0, 7.0), w.nan_to_num(9.0, 8.0, 7.0))


def test_clip_within_the_bound_changes_no_bit():
    g = grads_of(3, (1000, "bf16"), (1001, "f32"))
    out = clip_case(g, 1e6)
    assert all(torch.equal(a, b) for a, b in zip(g, out))


def test_norm_of_no_tensors():
    S, N = Out(1, dtype=torch.float64), Out(1)
    moe.moe_grad_norm([], S.t, N.t, None)
    moe.moe_grad_clip([], None, S.t, 1.0)
    torch.cuda.synchronize()
    assert S.np()[0] == 0 and N.np()[0] == 0


def test_binding_refuses_lists_of_other_lengths():
    a = torch.zeros(4, device=DEV)
    S = torch.zeros(1, dtype=torch.float64, device=DEV)
    with pytest.raises(ValueError, match="1 tensors, 2 outputs"):
        moe.moe_grad_clip([a], [a, a.clone()], S, 1.0)
    with pytest.raises(moe.MoEError, match="INVALID_ARG"):
        moe.moe_grad_clip([a, a], None, S, 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        moe.make_tensors([torch.zeros(4, 4, device=DEV).t()])


# ---- streams, graphs, calls side by side ----

def training_setup(M, d, F, G, seed):
    g = gen(seed)
    bf = torch.bfloat16
    f = moe.make_ffn(M, d, F, G)
    e = lambda *s, dt=bf: torch.zeros(*s, dtype=dt, device=DEV)       # noqa: E731
    t = dict(x=cuda(normal(g, M, d, dtype=bf)), dy=cuda(normal(g, M, d, dtype=bf)),
             w1=cuda(normal(g, G, F, d, std=0.05, dtype=bf)), w3=cuda(normal(g, G, F, d, std=0.05, dtype=bf)),
             w2=cuda(normal(g, G, d, F, std=0.05, dtype=bf)), off=off(uneven(M, G, seed)),
             h=e(M, F), p1=e(M, F), p3=e(M, F), dx=e(M, d), dw1=e(G, F, d), dw3=e(G, F, d), dw2=e(G, d, F),
             S=e(1, dt=torch.float64), N=e(1, dt=torch.float32))
    lst = moe.make_tensors([t["dw1"], t["dw3"], t["dw2"]])
    ws = [runner._bytes(n, DEV) for n in (moe.moe_ffn_workspace_bytes(f, moe.MOE_CALL_FFN_GATE_UP),
                                          moe.moe_ffn_workspace_bytes(f, moe.MOE_CALL_FFN_BACKWARD),
                                          moe.moe_grad_norm_workspace_bytes(lst))]

    def run(stream=None):
        moe.moe_ffn_gate_up(f, t["x"], t["off"], t["w1"], t["w3"], t["h"], t["p1"], t["p3"], ws[0], stream)
        moe.moe_ffn_backward(f, t["dy"], t["off"], t["x"], t["p1"], t["p3"], t["h"], t["w1"], t["w3"], t["w2"], t["dx"],
                             t["dw1"], t["dw3"], t["dw2"], ws[1], stream)
        moe.moe_grad_norm(lst, t["S"], t["N"], ws[2], stream)
        moe.moe_grad_clip(lst, None, t["S"], 0.5, stream)
    return t, run


RESULTS = ("h", "p1", "p3", "dx", "dw1", "dw3", "dw2", "S", "N")


@pytest.mark.parametrize("dims", [(16, 256, 512, 1), (500, 392, 264, 4)])
def test_training_calls_captured_and_replayed(dims):
    t, run = training_setup(*dims, seed=50)
    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=torch.cuda.Stream()):
        run()
    for i in range(3):
        t["x"].normal_()
        t["dy"].normal_()
        t["off"].copy_(off(uneven(dims[0], dims[3], 60 + i)))
        for n in RESULTS:
            t[n].zero_()
        run()
        torch.cuda.synchronize()
        want = [t[n].clone() for n in RESULTS]
        for n in RESULTS:
            t[n].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(t[n], w) for n, w in zip(RESULTS, want)), f"replay {i}"


def test_training_calls_on_two_streams_at_once():
    a, run_a = training_setup(700, 512, 264, 5, seed=60)
    b, run_b = training_setup(16, 1024, 2048, 1, seed=61)
    run_a()
    run_b()
    torch.cuda.synchronize()
    want = [a[n].clone() for n in RESULTS] + [b[n].clone() for n in RESULTS]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(4):
        run_a(s1)
        run_b(s2)
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip([a[n] for n in RESULTS] + [b[n] for n in RESULTS], want))


# ---- together, as used: a training pass of the layer ----

def layer(T=96, E=8, k=2, shared=0, **kw):
    cfg = synthetic.MoEConfig(name="train", T=T, d_model=128, d_ff=192, n_experts=E, top_k=k, n_shared=shared,
                              wg_std=128 ** -0.5, w13_std=0.08, w2_std=0.08, seed=12, **kw)
    inp = synthetic.make_inputs(cfg)
    inp.router_bias = normal(gen(70), E, std=0.3)
    return cfg, inp


F32S = dict(act_dtype="f32", w_dtype="f32")
LAYERS = [dict(), dict(shared=1, E=32, k=4), dict(T=1), dict(T=700), dict(capacity=20), dict(capacity=0), dict(capacity=0, shared=1), dict(E=12, k=3),
          dict(T=200, capacity=40, overflow="next_best"), dict(T=64, **F32S), dict(T=90, shared=1, k=3, **F32S)]


def autograd_layer(cfg, inp, st, dy):
    """The layer's gradients by autograd in fp64 on the CPU, for the rows that `st` grouped."""
    E, k, S, T = cfg.n_experts, cfg.top_k, cfg.n_shared, cfg.T
    leaf = {n: getattr(inp, n).double().clone().requires_grad_() for n in ("x", "w_gate", "router_bias", "w1", "w3", "w2")}
    logits = leaf["x"] @ leaf["w_gate"].t() + leaf["router_bias"]
    ids, row = st["topk_ids"].cpu().long(), st["slot_to_row"].cpu().long()
    ends = st["expert_offsets"].cpu().long()
    weights = torch.softmax(torch.gather(logits, 1, ids), 1)
    y = torch.zeros(T, cfg.d_model, dtype=torch.float64)
    for j in range(k + S):
        r = row[: T * k].view(T, k)[:, j] if j < k else row[T * k:]
        t = torch.nonzero(r >= 0).flatten()
        e = torch.searchsorted(ends, r[t], right=True) - 1
        w = weights[t, j][:, None] if j < k else torch.ones(len(t), 1, dtype=torch.float64)
        x = leaf["x"][t]
        h = torch.nn.functional.silu((leaf["w1"][e] @ x[:, :, None])[:, :, 0]) * (leaf["w3"][e] @ x[:, :, None])[:, :, 0]
        y = y.index_add(0, t, w * (leaf["w2"][e] @ h[:, :, None])[:, :, 0])
    (y * dy.double()).sum().backward()
    return {"dx": leaf["x"].grad, "dw_gate": leaf["w_gate"].grad, "dbias": leaf["router_bias"].grad,
            "dw1": leaf["w1"].grad, "dw3": leaf["w3"].grad, "dw2": leaf["w2"].grad}


@pytest.mark.parametrize("kw", LAYERS)
def test_layer_backward(kw):
    """Against autograd in fp64.  A gradient passes some six roundings to the operands' type on its way (h, y's
    rows' gradient, dg or du, g and u, dx_perm, its own), each half a step of a term at most and of either sign:
    relative to the whole, 6 half steps; fp32 the same with its sums' steps."""
    cfg, inp = layer(**kw)
    say(f"layer {kw}")
    di = runner.DeviceInputs.from_host(inp)
    dy = normal(gen(73), cfg.T, cfg.d_model, dtype=DT[cfg.act_dtype])
    st = runner.staged(di, keep=True)
    got = runner.layer_backward(di, st, cuda(dy))
    torch.cuda.synchronize()
    want = autograd_layer(cfg, inp, st, dy)
    tol = 6 * BF16 if cfg.act_dtype == "bf16" else 6 * F32 * 32
    for n, w in want.items():
        err = torch.linalg.vector_norm(got[n].cpu().double() - w) / torch.linalg.vector_norm(w).clamp(min=1e-30)
        assert err <= tol, (n, float(err))
    # the kept pass has the same y as the layer's own kernels to their roundings
    y = runner.staged(di)["y"].float()
    torch.cuda.synchronize()
    assert torch.linalg.vector_norm(st["y"].float() - y) <= 2 * BF16 * torch.linalg.vector_norm(y)


def test_layer_backward_with_a_scored_router_and_clipping():
    cfg, inp = layer(E=32, k=4, shared=1)
    di = runner.DeviceInputs.from_host(inp)
    router = moe.make_router("sigmoid", 4, 2, 2, True, 2.5)
    st = runner.staged(di, router=router, keep=True)
    dy = cuda(normal(gen(74), cfg.T, cfg.d_model, dtype=torch.bfloat16))
    o = runner.layer_backward(di, st, dy, router)
    alone = runner.gate_backward(di, st, router, dy)
    grads = [o[n] for n in ("dw_gate", "dbias", "dw1", "dw3", "dw2")]
    want = ref.clip([f64(t) for t in grads], 0.1)
    norm = runner.clip_gradients(grads, 0.1)
    torch.cuda.synchronize()
    assert torch.equal(o["dweights"], alone["dweights"]) and torch.equal(o["dlogits"], alone["dlogits"])
    assert abs(norm.item() - want[1]) <= 2 * F32 * want[1] and want[1] > 0.1
    for t, w in zip(grads, want[2]):
        step = BF16 if t.dtype is torch.bfloat16 else F32
        close(f64(t), w, (step + 2 * F32) * np.abs(w) + 1e-38, "clipped")
    assert runner.clip_gradients([], 1.0).item() == 0


def test_layer_gradient_is_the_difference_quotient():
    """fp32: along random directions of each weight, sum(y dy) changes by <gradient, direction>."""
    cfg, inp = layer(T=24, **F32S)
    di = runner.DeviceInputs.from_host(inp)
    dy = cuda(normal(gen(75), cfg.T, cfg.d_model))
    st = runner.staged(di, keep=True)
    o = runner.layer_backward(di, st, dy)

    def loss(**kw):
        s = runner.staged(__import__("dataclasses").replace(di, **kw), keep=True)
        assert torch.equal(s["topk_ids"], st["topk_ids"])
        return (s["y"].double() * dy.double()).sum().item()

    for name, grad in (("w1", "dw1"), ("w3", "dw3"), ("w2", "dw2"), ("x", "dx"), ("w_gate", "dw_gate")):
        base = getattr(di, name)
        g = torch.Generator(device=DEV).manual_seed(5)
        v = torch.empty_like(base).normal_(generator=g)
        eps = 2.0 ** -9 * (base.double().norm() / v.double().norm()).item()
        got = (loss(**{name: base + eps * v}) - loss(**{name: base - eps * v})) / (2 * eps)
        want = (o[grad].double() * v.double()).sum().item()
        # the third derivative's part, (2^-9)^2 of the function's size along v, and 2^9 times fp32's rounding of y
        size = o[grad].double().norm().item() * v.double().norm().item()
        assert abs(got - want) <= 0.01 * size, (name, got, want, size)


def test_layer_backward_refuses_quantised_experts():
    cfg = synthetic.MoEConfig(name="q", T=16, d_model=128, d_ff=128, w_dtype="fp8_e4m3")
    di = runner.DeviceInputs.from_host(synthetic.make_inputs(cfg))
    with pytest.raises(ValueError, match="no backward pass"):
        runner.staged(di, keep=True)


def test_layer_backward_on_a_stream_of_its_own():
    cfg, inp = layer(T=300, shared=1, E=12, k=3)
    di = runner.DeviceInputs.from_host(inp)
    dy = cuda(normal(gen(76), cfg.T, cfg.d_model, dtype=torch.bfloat16))
    st = runner.staged(di, keep=True)
    want = runner.layer_backward(di, st, dy)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    st2 = runner.staged(di, side, keep=True)
    got = runner.layer_backward(di, st2, dy, stream=side)
    norm = runner.clip_gradients([got["dw1"].clone()], 1.0, stream=side)
    side.synchronize()
    torch.cuda.synchronize()
    for n in ("dx", "dw_gate", "dbias", "dw1", "dw3", "dw2"):
        assert torch.equal(got[n], want[n]), n
    assert norm.item() > 0


# ---- sizes whose offsets pass 32 bits ----

def device_normal(seed, *shape, std=1.0, dtype=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(*shape, device=DEV, dtype=dtype).normal_(0, std, generator=g)


@pytest.mark.parametrize("d,F", [(8, 1032), (1032, 8)])
def test_ffn_of_more_than_2_31_elements(d, F):
    M = (1 << 21) + 77
    say(f"block M={M} d={d} F={F}")
    bf = torch.bfloat16
    cut = M - 1000
    offsets = off([0, cut, M])
    x, dy = device_normal(1, M, d), device_normal(2, M, d, std=0.01)
    w1, w3, w2 = device_normal(3, 2, F, d, std=0.1), device_normal(4, 2, F, d, std=0.1), device_normal(5, 2, d, F, std=0.1)
    f = moe.make_ffn(M, d, F, 2)
    e = lambda *s: torch.empty(*s, dtype=bf, device=DEV)              # noqa: E731
    h, p1, p3, dx, dw1, dw3, dw2 = e(M, F), e(M, F), e(M, F), e(M, d), e(2, F, d), e(2, F, d), e(2, d, F)
    ws = runner._bytes(max(moe.moe_ffn_workspace_bytes(f, c) for c in (moe.MOE_CALL_FFN_GATE_UP, moe.MOE_CALL_FFN_BACKWARD)), DEV)
    moe.moe_ffn_gate_up(f, x, offsets, w1, w3, h, p1, p3, ws)
    moe.moe_ffn_backward(f, dy, offsets, x, p1, p3, h, w1, w3, w2, dx, dw1, dw3, dw2, ws)
    torch.cuda.synchronize()
    for at in (0, cut - 50, M - 100):
        rows = slice(at, at + 100)
        for i, r in enumerate(range(at, at + 100)):
            if i % 25 and r not in (cut - 1, cut):
                continue
            k = 0 if r < cut else 1
            wh, wg, wu = ref.gate_up(f64(x[r:r + 1]), f64(w1[k]), f64(w3[k]), "silu")
            assert np.abs(f64(h[r]) - wh).max() <= 4 * BF16 * np.abs(wh).max() + 1e-3, r
            b = ref.backward(f64(dy[r:r + 1]), f64(x[r:r + 1]), f64(p1[r:r + 1]), f64(p3[r:r + 1]), f64(h[r:r + 1]),
                             f64(w1[k]), f64(w3[k]), f64(w2[k]), "silu")
            assert np.abs(f64(dx[r]) - b["dx"]).max() <= 4 * BF16 * np.abs(b["dx"]).max() + 1e-5, r
        assert torch.isfinite(h[rows]).all()
    # the last group's weight gradients, over its thousand rows
    b = ref.backward(*(f64(t[cut:]) for t in (dy, x, p1, p3, h)), f64(w1[1]), f64(w3[1]), f64(w2[1]), "silu")
    for got, want in ((dw1, b["dw1"]), (dw3, b["dw3"]), (dw2, b["dw2"])):
        assert np.abs(f64(got[1]) - want).max() <= 4 * BF16 * np.abs(want).max()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_block_of_the_most_rows(dtype):
    M, d, F, G = 1 << 24, 8, 8, 257
    say(f"block {dtype} M={M} d={d} F={F} G={G}")
    offsets = [M // 300 * e for e in range(G)] + [M - 1]
    x = device_normal(1, M, d, dtype=DT[dtype])
    w1, w3 = device_normal(2, G, F, d, dtype=DT[dtype]), device_normal(3, G, F, d, dtype=DT[dtype])
    f = moe.make_ffn(M, d, F, G, dtype)
    h = torch.full((M, F), -7.0, dtype=DT[dtype], device=DEV)
    moe.moe_ffn_gate_up(f, x, off(offsets), w1, w3, h, None, None, runner._bytes(moe.moe_ffn_workspace_bytes(f), DEV))
    torch.cuda.synchronize()
    assert (h[-1] == -7).all()
    for e in (0, 1, 100, 255, 256):
        for r in (offsets[e], offsets[e] + 1000, offsets[e + 1] - 1):
            want = ref.gate_up(f64(x[r:r + 1]), f64(w1[e]), f64(w3[e]), "silu")[0]
            assert np.abs(f64(h[r]) - want).max() <= 2 * steps(dtype)[0] * np.abs(want).max() + 1e-4, (e, r)


def test_permute_backward_of_the_most_tokens():
    T, d = 1 << 24, 64
    say(f"permute backward T={T} d={d}")
    dxp, add = device_normal(1, T * 2, d), device_normal(2, T, d)
    rows = torch.arange(2 * T - 1, -1, -1, dtype=torch.int32, device=DEV)     # last row first
    dx = torch.empty(T, d, dtype=torch.bfloat16, device=DEV)
    moe.moe_permute_backward(moe.make_shape(T, d, 64, 16, 2), dxp, rows, add, dx)
    torch.cuda.synchronize()
    for at in (0, (1 << 23) - 50, T - 100):
        tok = torch.arange(at, at + 100, device=DEV)
        want = add[tok].double() + dxp[2 * T - 1 - 2 * tok].double() + dxp[2 * T - 2 - 2 * tok].double()
        close(f64(dx[at:at + 100]), f64(want), BF16 * 1.001 * np.abs(f64(want)) + 1e-5, "dx")


def test_clip_of_a_tensor_of_more_than_2_31_elements():
    n = (1 << 31) + 12345
    say(f"clip n={n}")
    a = device_normal(1, n, std=0.01)
    S, N = torch.zeros(1, dtype=torch.float64, device=DEV), torch.zeros(1, device=DEV)
    lst = moe.make_tensors([a])
    want = sum((a[i:i + (1 << 28)].double() ** 2).sum().item() for i in range(0, n, 1 << 28))
    tail, head = a[-1000:].clone(), a[:1000].clone()
    moe.moe_grad_norm(lst, S, N, runner._bytes(moe.moe_grad_norm_workspace_bytes(lst), DEV))
    moe.moe_grad_clip(lst, None, S, 1.0)
    torch.cuda.synchronize()
    assert abs(S.item() - want) <= 1e-9 * want and want > 1
    for got, was in ((a[-1000:], tail), (a[:1000], head)):
        w = f64(was) / math.sqrt(want)
        close(f64(got), w, BF16 * 1.001 * np.abs(w), "scaled")


# ---- every tile shape and schedule, whole, against fp64 products on the device ----

def large_case(M, d, F, G, offsets, act="silu", dtype="bf16"):
    """Sizes at which the plans differ: tiles of each shape, cut and whole, groups' ends apart.  Relative to the
    Frobenius norm, each output is off by its own half step and those of its operands (dg, du: from dh and an
    activation of some ten fp32 roundings), and by the roundings of its sums: after m of n independent terms a sum
    has sqrt(m / n) of its final size, so n additions, each rounding by half a step of fp32 (products alike), leave
    2 n of these half steps at most; n counts the terms of every sum on the way."""
    say(f"large {dtype} M={M} d={d} F={F} G={G}")
    dt = DT[dtype]
    x, dy = device_normal(1, M, d, dtype=dt), device_normal(2, M, d, dtype=dt)
    w1, w3 = (device_normal(3 + i, G, F, d, std=d ** -0.5, dtype=dt) for i in range(2))
    w2 = device_normal(5, G, d, F, std=F ** -0.5, dtype=dt)
    f = moe.make_ffn(M, d, F, G, dtype, act)
    ws = [workspace(moe.moe_ffn_workspace_bytes(f, c)) for c in (moe.MOE_CALL_FFN_GATE_UP, moe.MOE_CALL_FFN_BACKWARD)]
    h, p1, p3 = (torch.full((M + 1, F), -7.0, dtype=dt, device=DEV) for _ in range(3))
    dx = torch.full((M + 1, d), -7.0, dtype=dt, device=DEV)
    dw1, dw3, dw2 = torch.full((G + 1, F, d), -7.0, dtype=dt, device=DEV), torch.full((G + 1, F, d), -7.0, dtype=dt, device=DEV), \
        torch.full((G + 1, d, F), -7.0, dtype=dt, device=DEV)
    o = off(offsets)
    moe.moe_ffn_gate_up(f, x, o, w1, w3, h, p1, p3, ws[0].t if ws[0] else None)
    moe.moe_ffn_backward(f, dy, o, x, p1, p3, h, w1, w3, w2, dx, dw1, dw3, dw2, ws[1].t)
    torch.cuda.synchronize()
    for w in ws:
        if w:
            w.np()
    for t in (h, p1, p3, dx, dw1, dw3, dw2):
        assert (t[-1] == -7).all(), "written past the end"
    away = torch.from_numpy(outside(M, offsets)).to(DEV)
    for t in (h, p1, p3, dx):
        assert (t[:M][away] == -7).all(), "rows of no group"
    step = steps(dtype)[0]

    def near(got, want, halves, n, what):
        tol = halves * step + (2 * n + 10) * F32
        err = torch.linalg.vector_norm(got.double() - want) / torch.linalg.vector_norm(want).clamp(min=1e-30)
        assert err <= tol, (what, float(err) / step)
        big = (got.double() - want).abs().amax() / want.abs().amax()       # no element far off
        assert big <= 4 * tol, (what, float(big) / step)

    with_rows = {e: (a, b) for e, a, b in ref.spans(offsets, G, M)}

    def check_gradients(outputs):
        for e in range(G):
            if e not in with_rows:
                assert not any(t[e].any() for n, ts in (("dw13", (dw1, dw3)), ("dw2", (dw2,))) if n in outputs for t in ts)
                continue
            a, b = with_rows[e]
            xs, ys, a1, a3, a2 = x[a:b].double(), dy[a:b].double(), w1[e].double(), w3[e].double(), w2[e].double()
            g, u, hs = p1[a:b].double(), p3[a:b].double(), h[a:b].double()
            sg = torch.sigmoid(g)
            if "dw2" in outputs:
                near(dw2[e], ys.t().contiguous() @ hs, 1.0, b - a, f"dw2 {e}")
            if outputs == "dw2":
                continue
            dh = ys @ a2
            dg, du = dh * u * (sg + g * sg * (1 - sg)), dh * g * sg
            if "dx" in outputs:
                near(dx[a:b], dg @ a1 + du @ a3, 2.0, d + 2 * F, f"dx {e}")
            if "dw13" in outputs:
                near(dw1[e], dg.t().contiguous() @ xs, 2.0, d + b - a, f"dw1 {e}")
                near(dw3[e], du.t().contiguous() @ xs, 2.0, d + b - a, f"dw3 {e}")

    for e, (a, b) in with_rows.items():
        xs = x[a:b].double()
        g, u = xs @ w1[e].double().t().contiguous(), xs @ w3[e].double().t().contiguous()
        near(h[a:b], g * torch.sigmoid(g) * u, 1.0, d, f"h {e}")
        near(p1[a:b], g, 1.0, d, f"g {e}")
        near(p3[a:b], u, 1.0, d, f"u {e}")
    check_gradients("dx dw13 dw2")
    for outputs in ("dx", "dw13", "dw2"):                    # alone: launches of their own
        for t in (dx, dw1, dw3, dw2):
            t.fill_(-7.0)
        ws[1].t.fill_(0xFF)
        has = [outputs == n for n in ("dx", "dw13", "dw2")]
        moe.moe_ffn_backward(f, dy, o, x, p1, p3, h, w1, w3, w2, dx if has[0] else None, dw1 if has[1] else None,
                             dw3 if has[1] else None, dw2 if has[2] else None, ws[1].t)
        torch.cuda.synchronize()
        ws[1].np()
        check_gradients(outputs)
        for t, there in ((dx, has[0]), (dw1, has[1]), (dw3, has[1]), (dw2, has[2])):
            assert (t[-1] == -7).all() and (there or (t == -7).all()), "written past the end, or not asked for"


@pytest.mark.parametrize("case", [
    # many rounds of large tiles: groups that end in a few rows of one, in many, at its border, groups of one row, of none
    (4500, 256, 8192, 3, [0, 1152, 2944, 4500]), (5000, 136, 8200, 6, [0, 1, 1, 1537, 3202, 3330, 4990]),
    (3000, 264, 12296, 4, [5, 5, 1100, 1229, 2995]), (2048, 4096, 8192, 2, [0, 1025, 2048]),
    # one group: whole and cut tiles of every shape
    (4096, 4096, 1024, 1, None), (2000, 2048, 2048, 1, None), (1024, 1024, 2048, 1, None), (300, 4096, 4096, 1, None),
    (700, 512, 512, 1, [0, 690]), (96, 2048, 1024, 1, None), (33, 8192, 264, 1, None), (40, 264, 8192, 1, None),
    (16, 8192, 64, 1, None), (32, 1024, 14336, 1, None), (24, 4096, 2048, 1, [3, 24]), (4, 512, 512, 1, None),
    (12, 2048, 512, 1, None), (8192, 512, 256, 1, None), (2500, 136, 72, 1, None),
    (8192, 2048, 1024, 1, None), (6000, 1024, 1024, 1, None), (16000, 512, 512, 1, None), (5000, 136, 264, 1, [1, 4999]),
    (1100, 4096, 2048, 1, None), (520, 2048, 4096, 1, None), (2100, 1024, 4096, 1, None), (2048, 4096, 4352, 1, None),
    (1792, 4352, 8192, 1, None),
    # several: few rounds, cut
    (600, 2048, 512, 4, [0, 100, 300, 301, 600]), (1500, 1024, 2048, 8, [0, 100, 300, 600, 900, 900, 1100, 1480, 1500]),
    (900, 4096, 264, 2, [0, 450, 900]), (8000, 64, 64, 32, [250 * i for i in range(33)]),
    # few weight tiles over long contractions, cut: groups of all rows, of few, of none
    (7080, 1352, 280, 2, [0, 3200, 7080]), (6000, 72, 136, 3, [0, 5990, 5990, 6000]), (5000, 520, 264, 5, [7, 7, 2000, 2001, 4000, 4900]),
    (2, 216, 248, 256, [0] * 100 + [1] * 100 + [2] * 57), (40, 64, 136, 257, [0] * 3 + [7] * 200 + [20] * 50 + [40] * 5),
])
def test_block_in_every_tile_shape(case):
    large_case(*case)


@pytest.mark.parametrize("case", [(700, 1024, 512, 1, None), (64, 4096, 512, 1, None), (3000, 256, 1024, 3, [0, 1000, 1001, 2990]),
                                  (20, 2048, 64, 2, [0, 11, 20]), (2048, 512, 1024, 1, None), (2048, 2048, 512, 1, None),
                                  (2048, 512, 2048, 1, None)])
def test_block_in_fp32_in_every_schedule(case):
    large_case(*case, dtype="f32")
