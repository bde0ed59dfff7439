"""Device buffers and call sequences around the C ABI (allocation and marshalling only).

``DeviceInputs`` moves a synthetic.MoEInputs to the GPU; ``forward`` runs the
fused ``moe_forward``; ``staged`` runs the five boundary calls one after the
other and returns every intermediate, so each step can be checked on its own.
Given a ``MoeRouter``, both route by ``scored_routing`` (``moe_linear`` for the
logits, ``moe_route_scored`` for the choice) instead of the library's top-k
softmax router, and ``gate_backward`` takes the gradient at y of such a staged
pass back to x and the router's weights (the experts' weights held fixed).
``layer_backward`` takes it back through the whole layer, the experts' weights
included, from a pass that kept what it needs (``staged(..., keep=True)``), and
``clip_gradients`` scales gradients to a bound of their norm.
"""
from __future__ import annotations

import contextlib
import dataclasses
import functools
from typing import Optional

import torch

from . import (make_ffn, make_linear, make_router, make_tensors, moe_combine, moe_combine_backward,
               moe_expert_gemm_down, moe_expert_gemm_gate_up, moe_ffn_backward, moe_ffn_gate_up,
               moe_ffn_workspace_bytes, moe_forward, moe_forward_routed, moe_grad_clip, moe_grad_norm,
               moe_grad_norm_workspace_bytes, moe_linear, moe_linear_backward,
               moe_linear_workspace_bytes, moe_permute, moe_permute_backward, moe_route_scored,
               moe_route_scored_backward, moe_route_topk, moe_workspace_bytes, shape_of,
               MOE_CALL_DOWN, MOE_CALL_FFN_BACKWARD, MOE_CALL_FFN_GATE_UP, MOE_CALL_FORWARD,
               MOE_CALL_LINEAR, MOE_CALL_LINEAR_BACKWARD, MOE_CALL_ROUTE)


def _dev(t: Optional[torch.Tensor], device) -> Optional[torch.Tensor]:
    if t is None:
        return None
    if t.dtype == torch.float8_e4m3fn:
        t = t.view(torch.uint8)
    return t.to(device).contiguous()


@dataclasses.dataclass
class DeviceInputs:
    cfg: object
    x: torch.Tensor
    w_gate: torch.Tensor
    router_bias: Optional[torch.Tensor]
    w1: torch.Tensor
    w3: torch.Tensor
    w2: torch.Tensor
    w1_scale: Optional[torch.Tensor]
    w3_scale: Optional[torch.Tensor]
    w2_scale: Optional[torch.Tensor]

    @classmethod
    def from_host(cls, inp, device="cuda"):
        return cls(inp.cfg, *(_dev(getattr(inp, f), device) for f in
                              ("x", "w_gate", "router_bias", "w1", "w3", "w2", "w1_scale",
                               "w3_scale", "w2_scale")))

    def with_weights(self, w1, w3, w2):
        return dataclasses.replace(self, w1=w1, w3=w3, w2=w2)


def _act_dtype(cfg):
    return torch.float32 if cfg.act_dtype == "f32" else torch.bfloat16


def _perm_dtype(cfg):
    if cfg.w_dtype == "fp8_e4m3":
        return torch.uint8
    return _act_dtype(cfg)


@dataclasses.dataclass
class ForwardBuffers:
    y: torch.Tensor
    topk_ids: torch.Tensor
    topk_weights: torch.Tensor
    expert_counts: torch.Tensor
    drop_mask: torch.Tensor
    logits: torch.Tensor
    workspace: torch.Tensor
    routing: Optional[dict] = None        # scored_routing's buffers: as long-lived as the others


def alloc_forward(cfg, device="cuda", with_outputs=True) -> ForwardBuffers:
    T, d, E, k = cfg.T, cfg.d_model, cfg.n_experts, cfg.top_k
    shape = shape_of(cfg)
    ws = torch.empty(max(1, moe_workspace_bytes(shape, MOE_CALL_FORWARD)), dtype=torch.uint8,
                     device=device)
    y = torch.empty(T, d, dtype=_act_dtype(cfg), device=device)
    if not with_outputs:
        return ForwardBuffers(y, None, None, None, None, None, ws)
    return ForwardBuffers(y, torch.empty(T, k, dtype=torch.int32, device=device),
                          torch.empty(T, k, dtype=torch.float32, device=device),
                          torch.empty(E + cfg.n_shared, dtype=torch.int32, device=device),
                          torch.empty(T * k, dtype=torch.uint8, device=device),
                          torch.empty(T, E, dtype=torch.float32, device=device), ws)


def _bytes(n: int, device) -> Optional[torch.Tensor]:
    return torch.empty(n, dtype=torch.uint8, device=device) if n else None


def _on(stream, device):
    """The context in which torch's own operations go to ``stream`` (None: where they go anyway)."""
    if stream is None:
        return contextlib.nullcontext()
    return torch.cuda.stream(stream if hasattr(stream, "cuda_stream")
                             else torch.cuda.ExternalStream(int(stream), device=device))


def _on_its_device(f):
    """The calls of a sequence go to the device that its inputs are on, whichever is current."""
    @functools.wraps(f)
    def run(di, *args, **kw):
        dev = di.x.device
        if dev.index is None or dev.index == torch.cuda.current_device():
            return f(di, *args, **kw)
        with torch.cuda.device(dev):
            return f(di, *args, **kw)
    return run


@_on_its_device
def scored_routing(di: DeviceInputs, router, balance_bias=None, stream=None, out: Optional[dict] = None,
                   scores: bool = False) -> dict:
    """logits = x . w_gate^T (+ router_bias) in fp32, then moe_route_scored: the buffers of both
    (``out`` holds ones to use: logits, topk_ids, topk_weights, next_ids, scores, linear_ws).
    moe_linear has widths of multiples of 8: the logits of other expert counts are those that
    moe_route_topk writes, and its choice is written over."""
    cfg, dev = di.cfg, di.x.device
    T, E, k = cfg.T, cfg.n_experts, cfg.top_k
    o = {} if out is None else out
    for name, shape, dtype in (("topk_ids", (T, k), torch.int32), ("topk_weights", (T, k), torch.float32),
                               ("logits", (T, E), torch.float32), ("next_ids", (T, 2), torch.int32),
                               ("scores", (T, E) if scores else None, torch.float32)):
        if o.get(name) is None:
            o[name] = None if shape is None else torch.empty(*shape, dtype=dtype, device=dev)
    if E % 8 == 0:
        lin = make_linear(T, E, cfg.d_model, dtype=cfg.act_dtype, y_dtype="f32")
        if o.get("linear_ws") is None:
            o["linear_ws"] = _bytes(moe_linear_workspace_bytes(lin, MOE_CALL_LINEAR), dev)
        moe_linear(lin, di.x, di.w_gate, di.router_bias, None, o["logits"], None, o["linear_ws"], stream)
    else:
        moe_route_topk(shape_of(cfg), di.x, di.w_gate, di.router_bias, o["topk_ids"], o["topk_weights"], o["logits"],
                       None, None, stream)
    moe_route_scored(shape_of(cfg), router, o["logits"], balance_bias, o["topk_ids"], o["topk_weights"],
                     o["scores"], o["next_ids"], stream)
    return o


@_on_its_device
def gate_backward(di: DeviceInputs, st: dict, router, dy: torch.Tensor, dscores=None, stream=None) -> dict:
    """Gradients of the gate from the gradient ``dy`` at y: ``st`` is the result of ``staged`` with
    the same router.  dy_perm is the gradient at the experts' rows (layer_backward takes it on
    through the experts); dx and dw_gate, dbias are those of the router's product alone (the path
    through the gate weights)."""
    cfg, dev = di.cfg, di.x.device
    T, d, E, k = cfg.T, cfg.d_model, cfg.n_experts, cfg.top_k
    W = (E + 7) // 8 * 8          # moe_linear_backward has widths of multiples of 8: zero rows behind the experts'
    act, shape = _act_dtype(cfg), shape_of(cfg)
    dw = torch.empty(W, d, dtype=act, device=dev)
    db = torch.empty(W, device=dev) if di.router_bias is not None else None
    o = {"dy_perm": torch.empty(T * (k + cfg.n_shared), d, dtype=act, device=dev),
         "dweights": torch.empty(T, k, device=dev), "dlogits": torch.empty(T, E, device=dev),
         "dx": torch.empty(T, d, dtype=act, device=dev), "dw_gate": dw[:E],
         "dbias": None if db is None else db[:E]}
    moe_combine_backward(shape, dy, st["y_perm"], st["slot_to_row"], st["topk_weights"], o["dy_perm"],
                         o["dweights"], stream)
    moe_route_scored_backward(shape, router, st["logits"], st["topk_ids"], o["dweights"], dscores,
                              o["dlogits"], stream)
    dlogits, w_gate = o["dlogits"], di.w_gate
    if W != E:
        o["padded"] = dlogits, w_gate = torch.empty(T, W, device=dev), torch.empty(W, d, dtype=act, device=dev)
        with _on(stream, dev):
            dlogits[:, :E].copy_(o["dlogits"])
            dlogits[:, E:].zero_()
            w_gate[:E].copy_(di.w_gate)
            w_gate[E:].zero_()
    lin = make_linear(T, W, d, dtype=cfg.act_dtype, y_dtype="f32")
    o["ws"] = _bytes(moe_linear_workspace_bytes(lin, MOE_CALL_LINEAR_BACKWARD), dev)
    moe_linear_backward(lin, dlogits, None, di.x, w_gate, o["dx"], dw, db, o["ws"], stream)
    return o


def _ffn_of(cfg):
    """The experts' block as moe_ffn_gate_up and moe_ffn_backward have it: a group per expert."""
    if cfg.w_dtype != cfg.act_dtype:
        raise ValueError(f"{cfg.w_dtype} experts have no backward pass: bf16 or fp32 weights do")
    return make_ffn(cfg.T * (cfg.top_k + cfg.n_shared), cfg.d_model, cfg.d_ff, cfg.n_experts + cfg.n_shared,
                    cfg.act_dtype, "silu")


@_on_its_device
def layer_backward(di: DeviceInputs, st: dict, dy: torch.Tensor, router=None, dscores=None, stream=None) -> dict:
    """Gradients of the whole layer from the gradient ``dy`` at y: ``st`` is the result of
    ``staged(..., keep=True)`` with the same router (None: the library's own, a softmax over the kept
    logits).  dx, dw_gate, dbias (with a router bias), dw1, dw3, dw2, beside what gate_backward gives.  Between the
    calls the gradients at the experts' rows (dy_perm, dx_perm) and the router's part of dx are in the activations' type."""
    cfg, dev = di.cfg, di.x.device
    ffn = _ffn_of(cfg)
    o = gate_backward(di, st, make_router() if router is None else router, dy, dscores, stream)
    o["dx_perm"] = torch.empty_like(st["x_perm"])
    for n in ("w1", "w3", "w2"):
        o["d" + n] = torch.empty_like(getattr(di, n))
    o["ffn_ws"] = _bytes(moe_ffn_workspace_bytes(ffn, MOE_CALL_FFN_BACKWARD), dev)
    moe_ffn_backward(ffn, o["dy_perm"], st["expert_offsets"], st["x_perm"], st["pre1"], st["pre3"], st["h"], di.w1,
                     di.w3, di.w2, o["dx_perm"], o["dw1"], o["dw3"], o["dw2"], o["ffn_ws"], stream)
    moe_permute_backward(shape_of(cfg), o["dx_perm"], st["slot_to_row"], o["dx"], o["dx"], stream)
    return o


def clip_gradients(grads, max_norm: float, stream=None) -> torch.Tensor:
    """Scales the tensors ``grads`` in place to a norm of at most ``max_norm`` (not where the norm is not
    finite); returns the norm they had, [1] fp32 on their device (on the current one for no tensors)."""
    t = make_tensors(grads)
    dev = torch.cuda.current_device() if t.device is None else t.device
    with torch.cuda.device(dev), _on(stream, dev):
        total, norm = torch.empty(1, dtype=torch.float64, device=dev), torch.empty(1, device=dev)
        ws = _bytes(moe_grad_norm_workspace_bytes(t), dev)
        moe_grad_norm(t, total, norm, ws, stream)
        moe_grad_clip(t, None, total, max_norm, stream)
    return norm


@_on_its_device
def forward(di: DeviceInputs, buf: Optional[ForwardBuffers] = None, stream=None, router=None,
            balance_bias=None) -> ForwardBuffers:
    cfg = di.cfg
    if buf is None:
        buf = alloc_forward(cfg, di.x.device)
    if router is not None:
        if buf.routing is None:
            buf.routing = {"topk_ids": buf.topk_ids, "topk_weights": buf.topk_weights, "logits": buf.logits}
        r = scored_routing(di, router, balance_bias, stream, buf.routing)
        moe_forward_routed(shape_of(cfg), di.x, r["topk_ids"], r["topk_weights"], r["next_ids"], di.w1, di.w3,
                           di.w2, di.w1_scale, di.w3_scale, di.w2_scale, buf.y, buf.expert_counts,
                           buf.drop_mask, buf.workspace, stream)
        return buf
    moe_forward(shape_of(cfg), di.x, di.w_gate, di.router_bias, di.w1, di.w3, di.w2, di.w1_scale,
                di.w3_scale, di.w2_scale, buf.y, buf.topk_ids, buf.topk_weights,
                buf.expert_counts, buf.drop_mask, buf.logits, buf.workspace, stream)
    return buf


@_on_its_device
def staged(di: DeviceInputs, stream=None, router=None, balance_bias=None, keep: bool = False) -> dict:
    """The five boundary calls in sequence (with a router: scored_routing in place of
    moe_route_topk); returns every intermediate buffer.  ``keep``: for layer_backward, the
    experts' pre-activations too, by moe_ffn_gate_up (bf16 or fp32 experts, up to 2^24 slots of all tokens)."""
    cfg = di.cfg
    dev = di.x.device
    T, d, F, E, k, S = cfg.T, cfg.d_model, cfg.d_ff, cfg.n_experts, cfg.top_k, cfg.n_shared
    A = T * k                  # routed slots
    R = T * (k + S)            # slots incl. the shared expert = most rows
    shape = shape_of(cfg)
    fp8 = cfg.w_dtype == "fp8_e4m3"
    o = {}
    if router is not None:
        scored_routing(di, router, balance_bias, stream, o, scores=True)
    else:
        o["topk_ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
        o["topk_weights"] = torch.empty(T, k, dtype=torch.float32, device=dev)
        o["logits"] = torch.empty(T, E, dtype=torch.float32, device=dev)
        o["next_ids"] = torch.empty(T, 2, dtype=torch.int32, device=dev)
        route_ws = moe_workspace_bytes(shape, MOE_CALL_ROUTE)   # used when no logits buffer is passed
        o["route_ws"] = _bytes(route_ws, dev)
        moe_route_topk(shape, di.x, di.w_gate, di.router_bias, o["topk_ids"], o["topk_weights"],
                       o["logits"], o["next_ids"], None, stream)
    o["expert_counts"] = torch.empty(E + S, dtype=torch.int32, device=dev)
    o["expert_offsets"] = torch.empty(E + S + 1, dtype=torch.int32, device=dev)
    o["perm_src"] = torch.full((R,), -7, dtype=torch.int32, device=dev)
    o["slot_to_row"] = torch.empty(R, dtype=torch.int32, device=dev)
    o["drop_mask"] = torch.empty(A, dtype=torch.uint8, device=dev)
    o["x_perm"] = torch.empty(R, d, dtype=_perm_dtype(cfg), device=dev)
    o["x_perm_scale"] = torch.empty(R, d // 32, dtype=torch.uint8, device=dev) if fp8 else None
    moe_permute(shape, o["topk_ids"], o["topk_weights"], o["next_ids"], di.x, o["expert_counts"],
                o["expert_offsets"], o["perm_src"], o["slot_to_row"], o["drop_mask"], o["x_perm"],
                o["x_perm_scale"], None, stream)
    o["h"] = torch.empty(R, F, dtype=_perm_dtype(cfg), device=dev)
    o["h_scale"] = torch.empty(R, F // 32, dtype=torch.uint8, device=dev) if fp8 else None
    if keep:
        ffn = _ffn_of(cfg)
        o["pre1"], o["pre3"] = (torch.empty(R, F, dtype=_act_dtype(cfg), device=dev) for _ in range(2))
        o["ffn_ws"] = _bytes(moe_ffn_workspace_bytes(ffn, MOE_CALL_FFN_GATE_UP), dev)
        moe_ffn_gate_up(ffn, o["x_perm"], o["expert_offsets"], di.w1, di.w3, o["h"], o["pre1"], o["pre3"],
                        o["ffn_ws"], stream)
    else:
        moe_expert_gemm_gate_up(shape, o["x_perm"], o["x_perm_scale"], o["expert_offsets"], di.w1,
                                di.w3, di.w1_scale, di.w3_scale, o["h"], o["h_scale"], None, stream)
    o["y_perm"] = torch.empty(R, d, dtype=torch.float32, device=dev)
    down_ws = moe_workspace_bytes(shape, MOE_CALL_DOWN)
    o["down_ws"] = torch.empty(down_ws, dtype=torch.uint8, device=dev) if down_ws else None
    moe_expert_gemm_down(shape, o["h"], o["h_scale"], o["expert_offsets"], di.w2, di.w2_scale,
                         o["y_perm"], o["down_ws"], stream)
    o["y"] = torch.empty(T, d, dtype=_act_dtype(cfg), device=dev)
    moe_combine(shape, o["y_perm"], o["slot_to_row"], o["topk_weights"], o["y"], stream)
    return o
