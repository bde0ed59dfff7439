"""CPU checks of the operators' calls at their edges: no tokens, shapes that only routing looks at, what the
documents show."""
import ctypes

import pytest

import sparse_mixture_experts_topk_amd as moe
from sparse_mixture_experts_topk_amd import _lib

A = 0x10000                 # an aligned address that no refused call reads
INVALID, UNSUPPORTED = 1, 2


def status(fn, *args):
    return getattr(_lib.load(), fn)(*[ctypes.byref(x) if isinstance(x, ctypes.Structure) else x for x in args])


def test_no_rows_with_outputs_of_no_elements():
    """A tensor without elements has no address: an output of no rows comes as NULL."""
    empty = moe.make_shape(0, 256, 256, 64, 6)
    assert status("moe_combine_backward", empty, *[None] * 6, None) == 0
    for kw in (dict(), dict(act="silu"), dict(dtype="f32", y_dtype="f32")):
        lin = moe.make_linear(0, 64, 128, **kw)
        assert status("moe_linear_backward", lin, *[None] * 7, None, 0, None) == 0
        assert status("moe_linear", lin, *[None] * 6, None, 0, None) == 0
    # with rows an output is needed
    assert status("moe_combine_backward", moe.make_shape(1, 256, 256, 64, 6), A, A, A, A, None, None, None) == INVALID
    assert status("moe_linear_backward", moe.make_linear(1, 64, 128), A, A, A, A, None, None, None, A, 1 << 40, None) == INVALID
    # and what is given still has to be aligned
    assert status("moe_linear_backward", moe.make_linear(0, 64, 128), *[None] * 5, A + 4, None, None, 0, None) == INVALID
