"""CPU checks of the gated feed-forward block, its gradients, the permutation's gradient and clipping: the C
ABI's refusals (nothing is enqueued), the binding's checks, and the fp64 reference against differences."""
import ctypes
import math

import numpy as np
import pytest
import torch

import sparse_mixture_experts_topk_amd as moe
from oracle import ffn as ref
from sparse_mixture_experts_topk_amd import _lib

A = 0x10000                 # an aligned address that no refused call reads
BIG = 1 << 50
INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 3


def status(fn, *args):
    return getattr(_lib.load(), fn)(*[ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in args])


GATE = [A] * 7              # x offsets w1 w3 h pre1 pre3
BACK = [A] * 13             # dy offsets x pre1 pre3 h w1 w3 w2 dx dw1 dw3 dw2


@pytest.mark.parametrize("kw,want", [
    (dict(), 0), (dict(M=-1), INVALID), (dict(M=(1 << 24) + 1), INVALID), (dict(d_model=0), INVALID),
    (dict(d_ff=-8), INVALID), (dict(groups=0), INVALID), (dict(groups=258), UNSUPPORTED), (dict(groups=257), 0),
    (dict(d_model=12), UNSUPPORTED), (dict(d_ff=100), UNSUPPORTED), (dict(d_model=(1 << 18) + 8), UNSUPPORTED),
    (dict(d_ff=(1 << 18) + 8), UNSUPPORTED), (dict(dtype="f32"), 0), (dict(dtype="fp8_e4m3"), UNSUPPORTED),
    (dict(dtype="mxfp4"), UNSUPPORTED), (dict(dtype=4), INVALID), (dict(dtype=-1), INVALID), (dict(act=5), INVALID),
    (dict(act=-1), INVALID), (dict(M=1 << 24, d_model=1 << 13), UNSUPPORTED),
    (dict(groups=2, d_model=1 << 18, d_ff=1 << 18), UNSUPPORTED),
])
def test_ffn_descriptor(kw, want):
    f = moe.make_ffn(**{**dict(M=7, d_model=64, d_ff=128, groups=3), **kw})
    n = ctypes.c_size_t(0)
    for call in (moe.MOE_CALL_FFN_GATE_UP, moe.MOE_CALL_FFN_BACKWARD):
        assert _lib.load().moe_ffn_workspace_bytes(ctypes.byref(f), call, ctypes.byref(n)) == want
    if want:
        assert status("moe_ffn_gate_up", f, *GATE, A, BIG, None) == want
        assert status("moe_ffn_backward", f, *BACK, A, BIG, None) == want


def test_ffn_pointer_and_workspace_refusals():
    f = moe.make_ffn(300, 256, 512, 4)
    for i in (0, 1, 2, 3, 4, 5, 6):                       # offsets too, with several groups; one of pre1, pre3
        bad = list(GATE)
        bad[i] = None
        assert status("moe_ffn_gate_up", f, *bad, A, BIG, None) == INVALID, i
    for i in range(7):
        bad = list(GATE)
        bad[i] = A + 8
        assert status("moe_ffn_gate_up", f, *bad, A, BIG, None) == INVALID, i
    need = moe.moe_ffn_workspace_bytes(f, moe.MOE_CALL_FFN_GATE_UP)
    if need:
        for ws in ((A, need - 1), (None, need), (A + 8, need)):
            assert status("moe_ffn_gate_up", f, *GATE, *ws, None) == WORKSPACE
    # each input that an asked-for output needs; one of dw1, dw3; no output
    for missing in ((0,), (1,), (2,), (3,), (4,), (5,), (6,), (7,), (8,), (10,), (11,), (9, 10, 11, 12)):
        bad = [None if i in missing else A for i in range(13)]
        assert status("moe_ffn_backward", f, *bad, A, BIG, None) == INVALID, missing
    for i in range(13):
        bad = list(BACK)
        bad[i] = A + 4
        assert status("moe_ffn_backward", f, *bad, A, BIG, None) == INVALID, i
    need = moe.moe_ffn_workspace_bytes(f, moe.MOE_CALL_FFN_BACKWARD)
    assert need > 0
    for ws in ((A, need - 1), (None, need), (A + 8, need)):
        assert status("moe_ffn_backward", f, *BACK, *ws, None) == WORKSPACE
    n = ctypes.c_size_t(0)
    assert _lib.load().moe_ffn_workspace_bytes(ctypes.byref(f), moe.MOE_CALL_LINEAR, ctypes.byref(n)) == INVALID
    assert _lib.load().moe_ffn_workspace_bytes(ctypes.byref(f), moe.MOE_CALL_FFN_GATE_UP, None) == INVALID
    assert _lib.load().moe_ffn_workspace_bytes(None, moe.MOE_CALL_FFN_GATE_UP, ctypes.byref(n)) == INVALID
    none = moe.make_ffn(0, 64, 64)
    assert status("moe_ffn_gate_up", none, *[None] * 7, None, 0, None) == 0
    assert moe.moe_ffn_workspace_bytes(none, moe.MOE_CALL_FFN_BACKWARD) == 0


def test_permute_backward_refusals():
    s = moe.make_shape(16, 256, 256, 8, 2)
    ok = [A, A, A, A]                                     # dx_perm slot_to_row addend dx
    for i in (0, 1, 3):
        bad = list(ok)
        bad[i] = None
        assert status("moe_permute_backward", s, *bad, None) == INVALID
    for i in range(4):
        bad = list(ok)
        bad[i] = A + 2
        assert status("moe_permute_backward", s, *bad, None) == INVALID
    assert status("moe_permute_backward", moe.make_shape(0, 256, 256, 8, 2), *[None] * 4, None) == 0
    assert status("moe_permute_backward", moe.make_shape(16, 100, 256, 8, 2), *ok, None) == UNSUPPORTED


def tensors(*entries):
    return (_lib.MoeTensor * max(1, len(entries)))(*entries)


def norm(list_, count, total=A, out=A, ws=A, n=BIG):
    return _lib.load().moe_grad_norm(list_, count, total, out, ws, n, None)


def clip(list_, outs, count, total=A, bound=1.0):
    return _lib.load().moe_grad_clip(list_, outs, count, total, bound, None)


@pytest.mark.parametrize("entry,want", [
    ((None, 5, moe.MOE_F32), INVALID), ((A, -1, moe.MOE_F32), INVALID), ((A, (1 << 40) + 1, moe.MOE_F32), INVALID),
    ((A + 2, 5, moe.MOE_F32), INVALID), ((A + 1, 5, moe.MOE_BF16), INVALID), ((A, 5, 7), INVALID), ((A, 5, -1), INVALID),
    ((A, 5, moe.MOE_FP8_E4M3), UNSUPPORTED), ((A, 5, moe.MOE_MXFP4), UNSUPPORTED),
])
def test_tensor_list_refusals(entry, want):
    n = ctypes.c_size_t(0)
    good = (A, 4, moe.MOE_F32)
    lists = tensors(good, entry)
    assert _lib.load().moe_grad_norm_workspace_bytes(lists, 2, ctypes.byref(n)) == want
    assert norm(lists, 2) == want
    assert clip(lists, None, 2) == want
    assert clip(tensors(good, (A + 64, max(entry[1], 0), moe.MOE_F32)), lists, 2) in (want, INVALID)


def test_list_argument_refusals():
    good = tensors((A, 4, moe.MOE_F32))
    assert norm(None, 1) == INVALID and norm(good, -1) == INVALID and norm(good, (1 << 16) + 1) == INVALID
    assert norm(good, 1, total=None) == INVALID and norm(good, 1, total=A + 8) == INVALID
    assert norm(good, 1, out=A + 4) == INVALID
    assert norm(good, 1, ws=None) == WORKSPACE and norm(good, 1, n=7) == WORKSPACE and norm(good, 1, ws=A + 8) == WORKSPACE
    n = ctypes.c_size_t(0)
    assert _lib.load().moe_grad_norm_workspace_bytes(good, 1, None) == INVALID
    assert _lib.load().moe_grad_norm_workspace_bytes(tensors((None, 0, moe.MOE_BF16)), 1, ctypes.byref(n)) == 0
    assert n.value == 0
    for bound in (-1.0, math.nan, -math.inf):
        assert clip(good, None, 1, bound=bound) == INVALID
    assert clip(good, None, 1, total=None) == INVALID


def test_clip_refuses_overlapping_outputs():
    f32, bf16 = moe.MOE_F32, moe.MOE_BF16
    # in place: twice the same tensor, two that share an element
    assert clip(tensors((A, 8, f32), (A, 8, f32)), None, 2) == INVALID
    assert clip(tensors((A, 8, f32), (A + 28, 8, f32)), None, 2) == INVALID
    assert clip(tensors((A + 30, 8, bf16), (A, 16, bf16), (A + 256, 8, f32)), None, 3) == INVALID
    # out of place: an output on another's input, on another output, shifted on its own input
    a, b = (A, 8, f32), (A + 32, 8, f32)
    assert clip(tensors(a, b), tensors(b, (A + 64, 8, f32)), 2) == INVALID
    assert clip(tensors(a, b), tensors((A + 64, 8, f32), (A + 92, 8, f32)), 2) == INVALID
    assert clip(tensors(a), tensors((A + 4, 8, f32)), 1) == INVALID
    assert clip(tensors((A, 100, f32), (A + 40, 2, f32), (A + 1024, 8, f32)), tensors((A + 2048, 100, f32), (A + 4096, 2, f32), (A + 384, 8, f32)), 3) == INVALID
    # outputs of another size or type
    assert clip(tensors(a), tensors((A + 64, 7, f32)), 1) == INVALID
    assert clip(tensors(a), tensors((A + 64, 8, bf16)), 1) == INVALID


def test_binding_refuses_wrong_tensors():
    f = moe.make_ffn(4, 64, 64)
    host = torch.empty(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device memory"):
        moe.moe_ffn_gate_up(f, host, None, A, A, A)
    with pytest.raises(moe.MoEError, match="INVALID_ARG"):
        moe.moe_ffn_gate_up(f, None, None, A, A, A)
    with pytest.raises(ValueError, match="float32 or torch.bfloat16"):
        moe.make_tensors([torch.empty(3, dtype=torch.float16)])
    with pytest.raises(ValueError, match="device memory"):
        moe.make_tensors([torch.empty(3)])


# ---- the reference against differences ----

@pytest.mark.parametrize("act", ["none", "relu", "silu", "gelu", "gelu_tanh"])
def test_reference_block_gradient_is_the_difference_quotient(act):
    rng = np.random.default_rng(8)
    M, d, f, h = 3, 4, 5, 1e-6
    x, w1, w3, w2, dy = (rng.normal(size=s) for s in ((M, d), (f, d), (f, d), (d, f), (M, d)))
    hid, g, u = ref.gate_up(x, w1, w3, act)
    grads = ref.backward(dy, x, g, u, hid, w1, w3, w2, act)

    def loss(x_, w1_, w3_, w2_):
        return float(((ref.gate_up(x_, w1_, w3_, act)[0] @ w2_.T) * dy).sum())

    args = [x, w1, w3, w2]
    for at, name in enumerate(("dx", "dw1", "dw3", "dw2")):
        for i in np.ndindex(*args[at].shape):
            p, m = [a.copy() for a in args], [a.copy() for a in args]
            p[at][i] += h
            m[at][i] -= h
            assert abs((loss(*p) - loss(*m)) / (2 * h) - grads[name][i]) < 1e-7


def test_reference_permute_gradient_is_the_difference_quotient():
    rng = np.random.default_rng(9)
    T, k, d = 4, 2, 3
    s2r = np.array([3, 0, 1, -1, 2, 4, -1, -1, 5, 6, 7, 8])       # shared rows last
    x, g = rng.normal(size=(T, d)), rng.normal(size=(9, d))

    def loss(x_):                                                 # each row holds its token's x
        out = 0.0
        for s, r in enumerate(s2r):
            if r >= 0:
                out += float(g[r] @ x_[s // k if s < T * k else s - T * k])
        return out

    dx, _ = ref.permute_backward(g, s2r, None, T, k, 1)
    for i in np.ndindex(T, d):
        p, m = x.copy(), x.copy()
        p[i] += 1e-6
        m[i] -= 1e-6
        assert abs((loss(p) - loss(m)) / 2e-6 - dx[i]) < 1e-7
    add = rng.normal(size=(T, d))
    assert np.allclose(ref.permute_backward(g, s2r, add, T, k, 1)[0], dx + add)


def test_reference_clip():
    g = [np.array([3.0, 0.0]), np.array([[4.0]])]
    total, n, out = ref.clip(g, 1.0)
    assert total == 25.0 and n == 5.0 and np.allclose(out[0], [0.6, 0]) and np.allclose(out[1], [[0.8]])
    assert ref.clip(g, 6.0)[2][1][0, 0] == 4.0
