"""CPU checks of lists of tensors, of clipping's refusals and of the difference test at their edges."""
import ctypes
import os
import random
import re
import shutil
import subprocess

import numpy as np
import pytest
import torch

import sparse_mixture_experts_topk_amd as moe
from differences import SHARE, STEP, slope_along
from oracle import ffn as ref
from sparse_mixture_experts_topk_amd import _lib


# ---- lists whose tensors' memory moves ----

class Tensor:
    """As much of a device tensor as a list looks at."""

    def __init__(self, address, n, dtype=torch.float32):
        self.address, self.n, self.dtype = address, n, dtype

    def data_ptr(self):
        return self.address

    def numel(self):
        return self.n

    def is_contiguous(self):
        return True

    def get_device(self):
        return None                   # as the device of a list without torch tensors

    def detach(self):
        return Tensor(self.address, self.n, self.dtype)


class Calls:
    """The library, with the lists' calls written down instead of made."""

    def __init__(self):
        self.lists = []

    def take(self, array, count):
        self.lists.append([(array[i].data, array[i].n, array[i].dtype) for i in range(count)])

    def moe_grad_norm_workspace_bytes(self, array, count, out):
        self.take(array, count)
        return 0

    def moe_grad_norm(self, array, count, *rest):
        self.take(array, count)
        return 0

    def moe_grad_clip(self, array, outs, count, *rest):
        self.take(array, count)
        if outs is not None:
            self.take(outs, count)
        return 0


def test_calls_look_up_where_a_lists_tensors_are(monkeypatch):
    calls = Calls()
    monkeypatch.setattr(_lib, "load", lambda: calls)
    a, b, o = Tensor(0x1000, 4), Tensor(0x2000, 6, torch.bfloat16), [Tensor(0x5000, 4), Tensor(0x6000, 6, torch.bfloat16)]
    lst, outs = moe.make_tensors([a, b]), moe.make_tensors(o)
    total = 0x100
    for step in range(3):
        if step:
            a.address, o[1].address = 0x1000 + 0x40 * step, 0x6000 + 0x40 * step
            b.address, b.n, b.dtype = 0x2000 + 0x40 * step, 6 + step, torch.float32
            o[1].n, o[1].dtype = b.n, b.dtype
        now = [(a.address, 4, moe.MOE_F32), (b.address, b.n, moe.MOE_F32 if step else moe.MOE_BF16)]
        there = [(0x5000, 4, moe.MOE_F32), (o[1].address, o[1].n, now[1][2])]
        moe.moe_grad_norm_workspace_bytes(lst)
        moe.moe_grad_norm(lst, total, None, None)
        moe.moe_grad_clip(lst, None, total, 1.0)
        moe.moe_grad_clip(lst, outs, total, 1.0)
        assert calls.lists == [now, now, now, now, there], step
        calls.lists.clear()


def test_a_list_whose_tensor_became_another_type_is_refused_until_it_is_mended(monkeypatch):
    calls = Calls()
    monkeypatch.setattr(_lib, "load", lambda: calls)
    a = Tensor(0x1000, 4)
    lst = moe.make_tensors([a])
    a.address, a.dtype = 0x2000, torch.float16
    for _ in range(2):
        with pytest.raises(ValueError, match="float32 or torch.bfloat16"):
            moe.moe_grad_norm(lst, 0x100)
    a.address, a.dtype = 0x1000, torch.float32
    moe.moe_grad_norm(lst, 0x100)
    assert calls.lists == [[(0x1000, 4, moe.MOE_F32)]]


# ---- clipping's refusals ----

INVALID = 1
TOTAL = 1 << 44                 # an aligned address that no refused call reads


def tensors(entries):
    return (_lib.MoeTensor * len(entries))(*[(a, n, t) for a, n, t in entries])


def clip(ins, outs, total=TOTAL):
    """Refused calls only: an accepted one would read its tensors."""
    return _lib.load().moe_grad_clip(tensors(ins), None if outs is None else tensors(outs), len(ins),
                                     ctypes.c_void_p(total), ctypes.c_float(1.0), None)


def lists(count, seed, in_place):
    """Tensors of 1 to 16 fp32 or bf16 elements in slots of 64 bytes, in any order: none overlap."""
    rng = random.Random(seed)
    slots = list(range(2 * count))
    rng.shuffle(slots)
    ins = [(0x100000 + 64 * slots[i], rng.randint(1, 16), rng.choice((moe.MOE_F32, moe.MOE_BF16))) for i in range(count)]
    outs = None if in_place else [(0x100000 + 64 * slots[count + i], n, t) for i, (_, n, t) in enumerate(ins)]
    return rng, ins, outs


@pytest.mark.parametrize("count", [2, 40, 1023, 2048, 4100, 20000])
@pytest.mark.parametrize("in_place", [True, False])
def test_clip_refuses_one_overlap_among_many_tensors(count, in_place):
    for seed in range(6):
        rng, ins, outs = lists(count, seed, in_place)
        i, j = rng.sample(range(count), 2)
        if in_place:                                        # the last element of i is the first of j
            a, n, t = ins[j]
            ins[i] = (a, n, t) if seed % 2 else (a - 4 * ins[i][1] + 4, ins[i][1], moe.MOE_F32)
        elif seed % 2:                                      # an output on another's input
            outs[i] = (ins[j][0], *ins[i][1:])
        else:                                               # on another output's last element
            a, n, t = outs[j]
            outs[i] = (a + (n - 1) * (4 if t == moe.MOE_F32 else 2) // 4 * 4, *ins[i][1:])
        assert clip(ins, outs) == INVALID, (seed, i, j)


@pytest.mark.parametrize("at", [0x1000, 0x1010, 0x1020])
def test_clip_refuses_a_sum_that_an_output_would_overwrite(at):
    """Every workgroup reads the sum while others already write."""
    f32, bf16 = moe.MOE_F32, moe.MOE_BF16
    before = (0x1ff0, 4, f32)
    for mine in ((0x1000, 9, f32), (0x1000, 17, bf16), (0x0ffe, 18, bf16)):     # up to 0x1024, 0x1022, 0x1022
        assert clip([before, mine], None, total=at) == INVALID
        assert clip([before, (0x4000, *mine[1:])], [(0x5000, *before[1:]), mine], total=at) == INVALID


def test_the_library_asks_for_no_host_memory():
    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("no nm here")
    _lib.load()
    names = subprocess.run([nm, "-D", "--undefined-only", _lib.LIB_PATH], capture_output=True, text=True, check=True).stdout.split()
    asks = [n for n in names if n.split("@")[0] in ("malloc", "calloc", "realloc", "aligned_alloc", "posix_memalign")
            or n.startswith(("_Znw", "_Zna"))]              # operator new, new[]
    assert not asks, asks


def test_the_permutations_gradient_promises_nothing_about_addend_and_dx():
    """The two may be the same memory, so the kernel's declaration keeps __restrict__ off both."""
    source = os.path.join(os.path.dirname(_lib.LIB_PATH), "csrc", "permute_backward.hip")
    with open(source) as f:
        declared = re.search(r"void permute_backward_kernel\(([^)]*)\)", f.read()).group(1)
    args = {a.split()[-1]: a for a in declared.split(",")}
    assert "__restrict__" in args["dx_perm"]
    assert "__restrict__" not in args["addend"] and "__restrict__" not in args["dx"]


# ---- differences along the gradient: the reference's gradients pass, planted mistakes do not ----

@pytest.mark.parametrize("mistake", [None, "sign", "other", "swapped", "no slope"])
def test_differences_along_the_gradient_tell_mistakes(mistake):
    rng = np.random.default_rng(21)
    M, d, f = 24, 40, 56
    w = {"x": rng.normal(size=(M, d)), "w1": rng.normal(size=(f, d)) * d ** -0.5, "w3": rng.normal(size=(f, d)) * d ** -0.5,
         "w2": rng.normal(size=(d, f)) * f ** -0.5}
    dy = rng.normal(size=(M, d))

    def loss(**kw):
        a = {**w, **kw}
        return float(((ref.gate_up(a["x"], a["w1"], a["w3"], "silu")[0] @ a["w2"].T) * dy).sum())

    h, g, u = ref.gate_up(w["x"], w["w1"], w["w3"], "silu")
    grads = ref.backward(dy, w["x"], g, u, h, w["w1"], w["w3"], w["w2"], "silu")
    none = ref.backward(dy, w["x"], g, u, h, w["w1"], w["w3"], w["w2"], "none")
    for name in w:
        grad = grads["d" + name]
        if mistake == "sign":
            grad = -grad
        elif mistake == "other":
            grad = rng.permutation(grad.ravel()).reshape(grad.shape)
        elif mistake == "swapped":
            if name not in ("w1", "w3"):
                continue
            grad = grads["dw3" if name == "w1" else "dw1"]
        elif mistake == "no slope":                       # the activation taken for the identity
            if name == "w2":
                continue
            grad = none["d" + name]
        got, want = slope_along(lambda v, n=name: loss(**{n: v}), w[name], grad, STEP)
        assert (abs(got - want) <= SHARE * want) == (mistake is None), (name, got, want)
