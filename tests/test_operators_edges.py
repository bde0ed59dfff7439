"""CPU checks of the operators' calls at their edges: no tokens, shapes that only routing looks at, what the
documents show, the constants of the sources."""
import ast
import ctypes
import inspect
import math
import pathlib
import re
import types

import numpy as np
import pytest
import torch

import sparse_mixture_experts_topk_amd as moe
from sparse_mixture_experts_topk_amd import _lib, runner

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


def test_routing_looks_at_tokens_experts_and_k_alone():
    """Routing from given logits has no use for the layer's widths and types, nor for the limits they bring."""
    r = moe.make_router("sigmoid", 8, 4, 2)
    forward = lambda s: status("moe_route_scored", s, r, *[None] * 6, None)              # noqa: E731
    backward = lambda s: status("moe_route_scored_backward", s, r, *[None] * 5, None)    # noqa: E731
    for call in (forward, backward):
        # more experts than the fp32 router takes, more rows than MXFP4 experts do, widths of no kernel
        for kw in (dict(act_dtype="f32", w_dtype="f32"), dict(w_dtype="mxfp4"), dict(w_dtype="fp8_e4m3"),
                   dict(d_model=100, d_ff=0), dict(overflow="next_best", capacity=4, top_k=6)):
            s = moe.make_shape(0, **{**dict(d_model=320, d_ff=64, n_experts=256, top_k=8), **kw})
            assert call(s) == 0, kw
            s.T = 1
            assert call(s) == INVALID, kw                   # missing pointers
        for kw, want in ((dict(T=-1), INVALID), (dict(T=(1 << 24) + 1), INVALID), (dict(top_k=0), INVALID),
                         (dict(n_experts=1), INVALID), (dict(n_experts=8, top_k=9), INVALID),
                         (dict(top_k=9), UNSUPPORTED), (dict(n_experts=264), UNSUPPORTED)):
            s = moe.make_shape(**{**dict(T=0, d_model=256, d_ff=256, n_experts=256, top_k=8), **kw})
            assert call(s) == want, kw


def test_calls_in_the_readme_fit_their_signatures():
    """Names that the README's Python gives to arguments are those of the parameters, in their order."""
    root = pathlib.Path(__file__).resolve().parent.parent
    blocks = re.findall(r"```python\n(.*?)```", (root / "README.md").read_text(), re.S)
    calls = 0
    for node in (n for b in blocks for n in ast.walk(ast.parse(b)) if isinstance(n, ast.Call)):
        f = node.func
        owner = {"moe": moe, "runner": runner}.get(getattr(getattr(f, "value", None), "id", None))
        if owner is None:
            continue
        calls += 1
        sig = inspect.signature(getattr(owner, f.attr))
        bound = sig.bind(*node.args, **{k.arg: k.value for k in node.keywords})
        for name, value in bound.arguments.items():
            if isinstance(value, ast.Name) and value.id in sig.parameters:
                assert value.id == name, f"{f.attr}: {value.id} in the place of {name}"
    assert calls >= 8


def test_gelu_tail_polynomial_is_as_near_as_its_comment_says():
    """The coefficients of the source against erfc, in 64 bits over the stated range."""
    root = pathlib.Path(moe.__file__).resolve().parent
    src = (root / "csrc" / "linear_epilogue.hpp").read_text()
    q0 = re.search(r"float q = ([-0-9.]+)f;", src)
    coeffs = [float(q0.group(1))] + [float(v) for v in re.findall(r"q = fmaf\(q, t, ([-0-9.]+)f\);", src)]
    scale = np.float64(np.float32(re.search(r"fmaf\(([0-9.]+)f, fabsf\(p\), 1\.0f\)", src).group(1)))
    bound = float(re.search(r"these coefficients: relative error ([-0-9.e]+);", src).group(1))
    assert len(coeffs) == 9
    u = np.linspace(0.0, 13.6, 20001)
    want = np.array([0.5 * math.erfc(v / math.sqrt(2)) * math.exp(0.5 * v * v) for v in u])
    t, q = 1.0 / (scale * u + 1.0), 0.0
    for c in coeffs:
        q = q * t + np.float64(np.float32(c))
    err = np.abs(q * t / want - 1.0).max()
    assert 0.9 * bound < err < bound, err


@pytest.mark.parametrize("name", ["scored_routing", "gate_backward", "forward", "staged"])
def test_sequences_run_on_their_inputs_device(name, monkeypatch):
    """With another device current, the calls (some take the current device's stream) are made on the inputs' one."""
    entered = []

    class Entered:
        def __init__(self, device):
            self.device = torch.device(device)

        def __enter__(self):
            entered.append(self.device.index)
            raise InterruptedError                     # nothing of the sequence itself runs here

        def __exit__(self, *exc):
            return False

    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch.cuda, "device", Entered)
    di = types.SimpleNamespace(x=types.SimpleNamespace(device=torch.device("cuda", 1)))
    with pytest.raises(InterruptedError):
        getattr(runner, name)(di)
    assert entered == [1]
