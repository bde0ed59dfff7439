"""CPU checks of lists of tensors and of clipping's refusals at their edges."""
import pytest
import torch

import sparse_mixture_experts_topk_amd as moe
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
