"""The feed-forward block's gradients, clipping and the runner's training pass at their edges: roundings, long sums,
norms that leave fp32, lists whose memory moves."""
import dataclasses
import math
import random
import sys

import numpy as np
import pytest
import torch

import sparse_mixture_experts_topk_amd as moe
from differences import SHARE, STEP, slope_along
from oracle import ffn as ref
from sparse_mixture_experts_topk_amd import runner, synthetic

pytestmark = pytest.mark.gpu

DEV = "cuda"
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def say(msg):
    print(f"\n[case] {msg}", flush=True)
    sys.stdout.flush()


# ---- clipping: one rounding ----

def bf16_nearest(v):
    """The bf16 value nearest to each fp64 value, the even one in the middle; in fp64, whose steps hold every distance here."""
    bits = np.abs(v).astype(np.float32)
    bits = np.where(bits.astype(np.float64) > np.abs(v), np.nextafter(bits, np.float32(0)), bits).view(np.uint32)
    low = (bits >> 16).astype(np.uint64)                    # the bf16 at or below |v|
    value = [(((low + i) << 16).astype(np.uint32)).view(np.float32).astype(np.float64) for i in (0, 1)]
    down, up = np.abs(v) - value[0], value[1] - np.abs(v)
    take = np.where(down == up, low & 1, up < down).astype(bool)
    return np.copysign(np.where(take, value[1], value[0]), v)


def clip_by(values, scale, offset, in_place):
    """Clips the bf16 values (placed `offset` elements behind a 16-byte boundary) by a scale below 1."""
    host = torch.from_numpy(values).to(torch.bfloat16)
    base = torch.zeros(offset + len(values) + 16, dtype=torch.bfloat16, device=DEV)
    t = base[offset:offset + len(values)]
    t.copy_(host)
    total = torch.tensor([1.0 / (scale * scale)], dtype=torch.float64, device=DEV)
    out = t if in_place else torch.empty(len(values), dtype=torch.bfloat16, device=DEV)
    moe.moe_grad_clip([t], None if in_place else [out], total, 1.0)
    torch.cuda.synchronize()
    want = host.double().numpy() * (1.0 / np.sqrt(total.cpu().numpy()[0]))
    return out.cpu().double().numpy(), bf16_nearest(want)


@pytest.mark.parametrize("offset,in_place", [(0, False), (0, True), (3, True), (5, False)])
@pytest.mark.parametrize("scale", [
    # powers of two times these lie 2^-30 from the middle between two bf16 values: above one whose even
    # neighbour is below, below one whose even neighbour is above; on the middle itself; and any
    0.5 * (1 + 2.0 ** -8 + 2.0 ** -30), 0.5 * (1 + 3 * 2.0 ** -8 - 2.0 ** -30), 0.5 * (1 + 2.0 ** -8), 0.3, 0.0371,
])
def test_clipped_bf16_is_rounded_once(scale, offset, in_place):
    say(f"clip rounding scale={scale!r} offset={offset} in place={in_place}")
    every = np.arange(1 << 16, dtype=np.uint32)              # each finite bf16 value, the subnormal ones too
    every = (every << 16).view(np.float32)
    every = every[np.isfinite(every)].astype(np.float64)
    got, want = clip_by(every, scale, offset, in_place)
    assert np.array_equal(got, want), [(every[i], got[i], want[i]) for i in np.nonzero(got != want)[0][:4]]


# ---- clipping: norms at the end of fp32 ----

@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("values,clipped", [
    ([3e38, 3e38, 3e38, -3e38], False),                 # the sum is finite in fp64, the norm, 6e38, not in fp32
    ([2e38, 2e38, 1e38, -1e38], True),                  # 3.16e38: finite
    ([3.38e38, 0.0], True), ([math.inf, 1.0], False), ([math.nan, 2.0], False),
])
def test_a_norm_that_is_not_finite_in_fp32_scales_nothing(values, clipped, dtype):
    say(f"clip at the end of fp32 {dtype} {values}")
    t = torch.tensor(values, dtype=torch.float64).to(DT[dtype]).to(DEV)
    was = t.clone()
    _, norm, want = ref.clip([was.cpu().double().numpy()], 5.0)
    got = runner.clip_gradients([t], 5.0)
    torch.cuda.synchronize()
    assert math.isfinite(got.item()) == clipped
    if not clipped:
        assert torch.equal(t.view(torch.uint8), was.view(torch.uint8)) and not norm <= torch.finfo(torch.float32).max
        return
    assert abs(got.item() - norm) <= 2.0 ** -23 * norm
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    assert (np.abs(t.cpu().double().numpy() - want[0]) <= step * 1.001 * np.abs(want[0])).all()


@pytest.mark.parametrize("on_stream", [False, True])
def test_the_norm_of_no_gradients_is_on_the_device(on_stream):
    for grads in ([], [torch.empty(0, device=DEV)]):
        norm = runner.clip_gradients(grads, 1.0, torch.cuda.Stream() if on_stream else None)
        torch.cuda.synchronize()
        assert norm.device.type == "cuda" and norm.shape == (1,) and norm.dtype is torch.float32 and norm.item() == 0


# ---- lists whose tensors' memory moves ----

@pytest.mark.parametrize("in_place", [True, False])
def test_a_list_follows_its_tensors(in_place):
    """Gradients that get other memory between steps (bucketed ones, say): the new values are read and scaled, the
    old memory is left alone."""
    sizes, g = (1000, 3, 4097), torch.Generator().manual_seed(31)
    fresh = lambda: [torch.randn(n, generator=g).to(dt).to(DEV)                                   # noqa: E731
                     for n, dt in zip(sizes, (torch.float32, torch.bfloat16, torch.bfloat16))]
    grads, outs = fresh(), fresh()
    lst, to = moe.make_tensors(grads), None if in_place else moe.make_tensors(outs)
    total, norm = torch.zeros(1, dtype=torch.float64, device=DEV), torch.zeros(1, device=DEV)
    ws = torch.empty(moe.moe_grad_norm_workspace_bytes(lst), dtype=torch.uint8, device=DEV)
    old, left = None, None
    for step in range(3):
        if step:
            old = [t.data for t in grads]
            left = [t.clone() for t in old]
            for t, v in zip(grads, fresh()):
                t.data = v
            outs[1].data = torch.zeros_like(outs[1])
        _, n, want = ref.clip([t.cpu().double().numpy() for t in grads], 2.0)
        moe.moe_grad_norm(lst, total, norm, ws)
        moe.moe_grad_clip(lst, to, total, 2.0)
        torch.cuda.synchronize()
        assert abs(norm.item() - n) <= 2.0 ** -22 * n
        for t, w in zip(grads if in_place else outs, want):
            step_of = 2.0 ** -8 if t.dtype is torch.bfloat16 else 2.0 ** -24
            assert (np.abs(t.cpu().double().numpy() - w) <= 1.001 * step_of * np.abs(w)).all()
        if old is not None:
            assert all(torch.equal(a, b) for a, b in zip(old, left))


@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("count", [3, 1500, 9000])
def test_clip_of_many_neighbours(count, in_place):
    """Tensors that touch one another in memory, in any order, overlap nowhere: accepted and scaled, each once."""
    say(f"clip of {count} neighbours in place={in_place}")
    rng = random.Random(count)
    sizes = [rng.randint(0, 9) for _ in range(count)]
    src = torch.randn(sum(sizes), generator=torch.Generator().manual_seed(count)).to(DEV)
    dst = torch.zeros_like(src)
    pairs = list(zip(src.split(sizes), (src if in_place else dst).split(sizes)))
    rng.shuffle(pairs)
    total = torch.full((1,), 4.0, dtype=torch.float64, device=DEV)
    want = src * 0.5
    moe.moe_grad_clip([a for a, _ in pairs], None if in_place else [b for _, b in pairs], total, 1.0)
    torch.cuda.synchronize()
    assert torch.equal(src if in_place else dst, want)


# ---- weight gradients over many rows ----

def device_values(seed, *shape, std=1.0, dtype=torch.float32, positive=False):
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = torch.empty(*shape, device=DEV, dtype=dtype).normal_(0, std, generator=g)
    return t.abs_() if positive else t


def weight_gradients(M, d, F, offsets, dtype, positive):
    """Every group's dw1, dw3, dw2 (no activation: dg = dh u, du = dh g) and fp64 sums of the same products."""
    G, dt = len(offsets) - 1, DT[dtype]
    say(f"weight gradients {dtype} M={M} d={d} F={F} G={G} positive={positive}")
    val = lambda seed, *s, std=1.0: device_values(seed, *s, std=std, dtype=dt, positive=positive)      # noqa: E731
    x, dy, p1, p3, h = val(1, M, d), val(2, M, d, std=0.01), val(3, M, F), val(4, M, F), val(5, M, F)
    w2 = val(6, G, d, F, std=F ** -0.5)
    f = moe.make_ffn(M, d, F, G, dtype, "none")
    dw1, dw3, dw2 = (torch.full(s, -7.0, dtype=dt, device=DEV) for s in ((G, F, d), (G, F, d), (G, d, F)))
    ws = runner._bytes(moe.moe_ffn_workspace_bytes(f, moe.MOE_CALL_FFN_BACKWARD), DEV)
    moe.moe_ffn_backward(f, dy, torch.tensor(offsets, dtype=torch.int32, device=DEV), x, p1, p3, h, None, None, w2, None,
                         dw1, dw3, dw2, ws)
    torch.cuda.synchronize()
    for e in range(G):
        a, b = offsets[e], offsets[e + 1]
        if a == b:
            assert not (dw1[e].any() or dw3[e].any() or dw2[e].any()), e
            continue
        want = [torch.zeros(s, dtype=torch.float64, device=DEV) for s in ((F, d), (F, d), (d, F))]
        for r in range(a, b, 1 << 18):
            rows = slice(r, min(b, r + (1 << 18)))
            ys, xs = dy[rows].double(), x[rows].double()
            dh = ys @ w2[e].double()
            want[0] += (dh * p3[rows].double()).t().contiguous() @ xs
            want[1] += (dh * p1[rows].double()).t().contiguous() @ xs
            want[2] += ys.t().contiguous() @ h[rows].double()
        for got, w, what in zip((dw1[e], dw3[e], dw2[e]), want, ("dw1", "dw3", "dw2")):
            yield e, b - a, what, got.double(), w


@pytest.mark.parametrize("M,d,F,offsets", [
    ((1 << 20) + 5, 64, 64, [0, (1 << 20) + 2] + [(1 << 20) + 5] * 256),           # all rows but three in one of many groups
    (1 << 24, 64, 64, [0, (1 << 24) - 7] + [1 << 24] * 256),
    ((1 << 20) + 77, 136, 72, [0, (1 << 20) + 77]), (1 << 24, 64, 64, [0, (1 << 24)]),
    ((1 << 17) + 3, 1032, 2048, [0, 70000, 70001, (1 << 17) + 3]), (40000, 4096, 1024, [0, 40000]),
])
def test_fp32_weight_gradients_over_many_rows_of_one_sign(M, d, F, offsets):
    """An addition rounds by half a step (2^-24) of the sum so far at most.  m terms of one sign: on average of half
    the sum, so m / 2 half steps of it.  Terms are added up to 2^15 in a row, or 2^12 where there are more; then N chains
    are (up to 64 runs of them, and they among themselves); dg and du are off by the additions of their d terms, every
    product by a half step: the bound of an element.  The roundings are independent, uniform within the half step and, as
    long as a step of the sum stays far below a term, of either sign: a chain's standard deviation is sqrt(m / 9) of
    its half steps, and the whole is within twice that, relative to the Frobenius norm."""
    for e, n, what, got, want in weight_gradients(M, d, F, offsets, "f32", True):
        m, N = min(n, 1 << 15), n / (1 << 12) + 64
        worst = ((got - want).abs() / want.abs()).amax().item()
        whole = (torch.linalg.vector_norm(got - want) / torch.linalg.vector_norm(want)).item()
        print(f"{e} {what} n={n}: worst {worst:.3e} whole {whole:.3e}")
        assert worst <= (m / 2 + N / 2 + d / 2 + 8) * 2.0 ** -24, (e, what, worst)
        assert whole <= 2 * (math.sqrt(m / 9) + math.sqrt(N / 9) + math.sqrt(d / 9) + 4) * 2.0 ** -24, (e, what, whole)


@pytest.mark.parametrize("positive", [True, False])
@pytest.mark.parametrize("M,d,F,offsets", [
    ((1 << 21) + 77, 8, 1032, [0, (1 << 21) - 923, (1 << 21) + 77]), ((1 << 21) + 77, 1032, 8, [0, (1 << 21) - 923, (1 << 21) + 77]),
    ((1 << 21) + 77, 136, 200, [5, (1 << 21) + 77]), ((1 << 20) + 9, 64, 64, [0, 0, (1 << 20) + 2] + [(1 << 20) + 9] * 254),
])
def test_bf16_weight_gradients_over_many_rows(M, d, F, offsets, positive):
    """Off by their own half step (2^-8) and, dg and du, by one of each term's; by the roundings of fp32 sums, of 32
    terms an instruction, which may round four times: n / 8 additions.  Of one sign: half steps of half the sum.  Of
    either sign the sum grows as the square root of its terms: relative to the Frobenius norm n / 8 additions leave
    sqrt(n / 8 / 2) half steps if they are independent, doubled."""
    for e, n, what, got, want in weight_gradients(M, d, F, offsets, "bf16", positive):
        own = 2.0 ** -8 * (1 if what == "dw2" else 2)
        whole = (torch.linalg.vector_norm(got - want) / torch.linalg.vector_norm(want)).item()
        print(f"{e} {what} n={n}: whole {whole:.3e}")
        assert whole <= own + (2 * math.sqrt(n / 16) + d / 2) * 2.0 ** -24, (e, what, whole)
        if positive:
            worst = ((got - want).abs() / want.abs()).amax().item()
            assert worst <= own * 1.01 + (n / 16 + d / 2) * 2.0 ** -24, (e, what, worst)


@pytest.mark.parametrize("M,d,F", [(4097, 512, 20000), (8192, 1024, 16392), (300, 72, 20000)])
def test_fp32_input_gradient_over_many_channels_of_one_sign(M, d, F):
    """dx sums 2 F terms: bounds as for the weight gradients, with n = 2 F."""
    say(f"input gradient M={M} d={d} F={F}")
    val = lambda seed, *s, std=1.0: device_values(seed, *s, std=std, positive=True)      # noqa: E731
    dy, p1, p3 = val(1, M, d, std=0.01), val(2, M, F), val(3, M, F)
    w1, w3, w2 = val(4, F, d), val(5, F, d), val(6, d, F)
    f = moe.make_ffn(M, d, F, 1, "f32", "none")
    dx = torch.full((M + 1, d), -7.0, device=DEV)
    ws = runner._bytes(moe.moe_ffn_workspace_bytes(f, moe.MOE_CALL_FFN_BACKWARD), DEV)
    moe.moe_ffn_backward(f, dy, None, None, p1, p3, None, w1, w3, w2, dx, None, None, None, ws)
    torch.cuda.synchronize()
    assert (dx[M] == -7).all()
    dh = dy.double() @ w2.double()
    want = (dh * p3.double()) @ w1.double() + (dh * p1.double()) @ w3.double()
    got, n = dx[:M].double(), 2 * F
    m, N = min(n, 1 << 15), n / (1 << 12) + 64
    worst = ((got - want).abs() / want.abs()).amax().item()
    whole = (torch.linalg.vector_norm(got - want) / torch.linalg.vector_norm(want)).item()
    print(f"worst {worst:.3e} whole {whole:.3e}")
    assert worst <= (m / 2 + N / 2 + d / 2 + 8) * 2.0 ** -24
    assert whole <= 2 * (math.sqrt(m / 9) + math.sqrt(N / 9) + math.sqrt(d / 9) + 4) * 2.0 ** -24


# ---- the whole layer's gradients against differences along themselves ----

@pytest.mark.parametrize("kw", [dict(), dict(n_shared=1, top_k=3), dict(T=40, capacity=9)])
def test_layer_gradients_against_differences_along_themselves(kw):
    cfg = synthetic.MoEConfig(**{**dict(name="slopes", T=24, d_model=128, d_ff=192, n_experts=8, act_dtype="f32", w_dtype="f32",
                                        wg_std=128 ** -0.5, w13_std=0.08, w2_std=0.08, seed=12), **kw})
    say(f"differences {kw}")
    inp = synthetic.make_inputs(cfg)
    inp.router_bias = 0.3 * torch.randn(cfg.n_experts, generator=torch.Generator().manual_seed(70))
    di = runner.DeviceInputs.from_host(inp)
    dy = torch.randn(cfg.T, cfg.d_model, generator=torch.Generator().manual_seed(75)).to(DEV)
    st = runner.staged(di, keep=True)
    o = runner.layer_backward(di, st, dy)

    def loss(name, value):
        s = runner.staged(dataclasses.replace(di, **{name: value.float()}), keep=True)
        assert torch.equal(s["slot_to_row"], st["slot_to_row"]), "the step changes the choice of experts"
        return (s["y"].double() * dy.double()).sum().item()

    for name, grad in (("w1", "dw1"), ("w3", "dw3"), ("w2", "dw2"), ("x", "dx"), ("w_gate", "dw_gate"), ("router_bias", "dbias")):
        # Where logits move no token may choose other experts: shorter steps, which y's roundings allow: independent ones
        # of 2^-21 in the n = T d elements leave 2^-21 |y| |dy| / sqrt(n) in the loss, sqrt(n) > 2^5; over 2^-13 |base|
        # |grad| that is 2^-13 of the ratio.
        step = STEP if name in ("w1", "w3", "w2") else 2.0 ** -13
        got, want = slope_along(lambda v, n=name: loss(n, v), getattr(di, name).double(), o[grad].double(), step)
        print(f"{name}: {got:.6e} {want:.6e} {abs(got - want) / want:.2e}")
        assert abs(got - want) <= SHARE * want, name
