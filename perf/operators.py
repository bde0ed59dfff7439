"""Measured cases of the routing and dense-product operators.

``run`` makes one pass through an operator: with ``own`` unset in its plain form
(elementary torch operations in 32 or 64 bits), with ``own`` set through the
package's entry points.

  linear            y = act(x W^T + b) + residual
  linear_backward   dx, dW, db of it from dy and the saved pre-activation
  route             scored top-k routing from logits (softmax or sigmoid scores,
                    balance bias, expert groups, renormalised weights)
  route_backward    gradient of the gate weights (and of the scores) at the logits
  combine_backward  gradient of the gate-weighted combine at the expert rows and
                    at the gate weights
"""
import math

import torch

own = False

D_MODEL, D_FF = 4096, 14336        # the layer's widths; fine-grained experts: 2048
FINE_E, FINE_K = 256, 8


def listed():
    return [
        # one token through a dense feed-forward product while decoding: reads the weights once
        {"name": "linear 1 token", "op": "linear", "M": 1, "N": D_FF, "K": D_MODEL, "act": "silu",
         "bias": True, "residual": False, "save_pre": False, "out": "bf16"},
        # the router's product of a decode batch, fp32 logits: latency alone
        {"name": "linear router 16 tokens", "op": "linear", "M": 16, "N": FINE_E, "K": D_MODEL,
         "act": "none", "bias": True, "residual": False, "save_pre": False, "out": "f32"},
        # a chunk of a prompt of odd length, the product back to the model width with its residual
        {"name": "linear 509 tokens", "op": "linear", "M": 509, "N": D_MODEL, "K": 2048,
         "act": "none", "bias": False, "residual": True, "save_pre": False, "out": "bf16"},
        # a prefill or training batch through a dense feed-forward product, pre-activation kept
        {"name": "linear 8192 tokens", "op": "linear", "M": 8192, "N": D_FF, "K": D_MODEL,
         "act": "silu", "bias": True, "residual": False, "save_pre": True, "out": "bf16"},
        # gradient of the router's product over a training batch of odd length
        {"name": "linear back router", "op": "linear_backward", "M": 4099, "N": FINE_E, "K": D_MODEL,
         "act": "none", "bias": True, "out": "f32"},
        # gradient of a dense feed-forward product over a training batch
        {"name": "linear back 8192 tokens", "op": "linear_backward", "M": 8192, "N": D_FF, "K": D_MODEL,
         "act": "gelu_tanh", "bias": True, "out": "bf16"},
        # routing of a decode batch to many small experts in groups: latency alone
        {"name": "route 16 tokens", "op": "route", "T": 16, "E": FINE_E, "k": FINE_K, "score": "sigmoid",
         "n_groups": 8, "topk_groups": 4, "group_top": 2, "renormalize": True, "scale": 2.5,
         "bias": True, "scores": False},
        # routing of a long prompt
        {"name": "route 16384 tokens", "op": "route", "T": 16384, "E": FINE_E, "k": FINE_K, "score": "sigmoid",
         "n_groups": 8, "topk_groups": 4, "group_top": 2, "renormalize": True, "scale": 2.5,
         "bias": True, "scores": False},
        # gradient at the logits of few experts, with a balance loss's gradient at the scores
        {"name": "route back 1021 tokens", "op": "route_backward", "T": 1021, "E": 8, "k": 2,
         "score": "softmax", "renormalize": False, "scale": 1.0, "dscores": True},
        # gradient at the logits of many experts over a training batch
        {"name": "route back 16384 tokens", "op": "route_backward", "T": 16384, "E": FINE_E, "k": FINE_K,
         "score": "sigmoid", "renormalize": True, "scale": 2.5, "dscores": False},
        # gradient of the combine: a small batch over few experts with a capacity
        {"name": "combine back 61 tokens", "op": "combine_backward", "T": 61, "d": D_MODEL, "E": 8, "k": 2,
         "shared": 0, "dropped": 0.1},
        # gradient of the combine: a training batch over many experts and the shared one
        {"name": "combine back 8192 tokens", "op": "combine_backward", "T": 8192, "d": D_MODEL, "E": FINE_E,
         "k": FINE_K, "shared": 1, "dropped": 0.0},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_backward", "linear_backward", "route", "route",
                     "route_backward", "combine_backward"))
    if op in ("linear", "linear_backward"):
        while True:
            M, N, K = _log_int(rng, 1, 8192), _log_int(rng, 64, D_FF, 8), _log_int(rng, 64, D_FF, 8)
            if M * N * K <= 8192 * D_FF * D_MODEL and M * (N + K) <= 8192 * (D_FF + D_MODEL):
                break
        out = rng.choice(("bf16", "bf16", "f32"))
        act = rng.choice(("none", "relu", "silu", "gelu", "gelu_tanh"))
        case = {"op": op, "M": M, "N": N, "K": K, "act": act, "bias": rng.random() < 0.6, "out": out}
        if op == "linear":
            case.update(residual=rng.random() < 0.4, save_pre=act != "none" and rng.random() < 0.4)
        return case
    if op == "combine_backward":
        E = rng.choice((8, 16, 60, 64, 160, 256))
        return {"op": op, "T": _log_int(rng, 1, 8192), "d": _log_int(rng, 128, D_MODEL, 64), "E": E,
                "k": rng.choice((1, 2, 4, 6, 8)), "shared": rng.choice((0, 1)),
                "dropped": rng.choice((0.0, 0.05, 0.3))}
    groups, kept, top, E, k = rng.choice(((1, 1, 1, 8, 2), (1, 1, 1, 16, 2), (1, 1, 1, 60, 4), (1, 1, 1, 64, 6),
                                          (1, 1, 1, 128, 8), (1, 1, 1, 256, 8), (4, 2, 1, 64, 6),
                                          (8, 3, 1, 160, 6), (8, 4, 2, 256, 8), (16, 5, 2, 128, 7)))
    case = {"op": op, "T": _log_int(rng, 1, 16384), "E": E, "k": k, "score": rng.choice(("softmax", "sigmoid")),
            "renormalize": rng.random() < 0.7, "scale": rng.choice((1.0, 2.5))}
    if op == "route":
        case.update(n_groups=groups, topk_groups=kept, group_top=top, bias=rng.random() < 0.6,
                    scores=rng.random() < 0.3)
    else:
        case["dscores"] = rng.random() < 0.5
    return case


def _n_dropped(case):
    return int(case["T"] * case["k"] * case["dropped"])


# ---- inputs ----

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(*shape, device=dev).normal_(0, std, generator=g).to(dtype)

    op = case["op"]
    s = {"case": case}
    bf16 = torch.bfloat16
    if op in ("linear", "linear_backward"):
        M, N, K = case["M"], case["N"], case["K"]
        out = torch.float32 if case["out"] == "f32" else bf16
        s["x"] = normal(M, K, dtype=bf16)
        s["w"] = normal(N, K, std=K ** -0.5, dtype=bf16)
        s["b"] = normal(N, std=0.5) if case["bias"] else None
        if op == "linear":
            s["res"] = normal(M, N, dtype=out) if case["residual"] else None
            s["y"] = torch.empty(M, N, dtype=out, device=dev)
            s["pre"] = torch.empty(M, N, dtype=bf16, device=dev) if case["save_pre"] else None
        else:
            s["dy"] = normal(M, N, std=0.01, dtype=out)
            s["pre"] = normal(M, N, std=1.1, dtype=bf16) if case["act"] != "none" else None
            s["dx"] = torch.empty(M, K, dtype=bf16, device=dev)
            s["dw"] = torch.empty(N, K, dtype=bf16, device=dev)
            s["db"] = torch.empty(N, device=dev) if case["bias"] else None
        return s
    T, E, k = case["T"], case["E"], case["k"]
    if op in ("route", "route_backward"):
        s["logits"] = normal(T, E)
        s["ids"] = torch.empty(T, k, dtype=torch.int32, device=dev)
        s["weights"] = torch.empty(T, k, device=dev)
        if op == "route":
            std = 0.05 if case["score"] == "sigmoid" else 0.2 / E
            s["bias"] = normal(E, std=std) if case["bias"] else None
            s["scores"] = torch.empty(T, E, device=dev) if case["scores"] else None
        else:
            s["ids"] = torch.topk(s["logits"], k, dim=1).indices.to(torch.int32)
            s["dweights"] = normal(T, k, std=0.1)
            s["dscores"] = normal(E, std=0.01).expand(T, E).contiguous() if case["dscores"] else None
            s["dlogits"] = torch.empty(T, E, device=dev)
        return s
    d, S = case["d"], case["shared"]
    # rows grouped by expert in token order, some slots dropped, the shared expert's rows last
    ids = torch.rand(T, E, device=dev, generator=g).topk(k, dim=1).indices.flatten()
    drop = torch.zeros(T * k, dtype=torch.bool, device=dev)
    drop[torch.randperm(T * k, device=dev, generator=g)[: _n_dropped(case)]] = True
    order = torch.sort(torch.where(drop, E, ids), stable=True).indices
    row = torch.empty(T * k, dtype=torch.int64, device=dev)
    row[order] = torch.arange(T * k, device=dev)
    kept = T * k - _n_dropped(case)
    row = torch.where(drop, -1, row)
    if S:
        row = torch.cat((row, kept + torch.arange(T, device=dev)))
    s["slot_to_row"] = row.to(torch.int32)
    s["rows"] = kept + S * T
    R = T * (k + S)
    s["y_perm"] = normal(R, d)
    s["dy"] = normal(T, d, std=0.01, dtype=bf16)
    s["weights"] = torch.softmax(normal(T, k), dim=1)
    s["dy_perm"] = torch.empty(R, d, dtype=bf16, device=dev)
    s["dweights"] = torch.empty(T, k, device=dev)
    return s


# ---- plain forms ----

def _act(p, act):
    if act == "relu":
        return torch.clamp(p, min=0)
    if act == "silu":
        return p / (1 + torch.exp(-p))
    if act == "gelu":
        return 0.5 * p * (1 + torch.erf(p * 0.5 ** 0.5))
    if act == "gelu_tanh":
        return 0.5 * p * (1 + torch.tanh((2 / math.pi) ** 0.5 * (p + 0.044715 * p * p * p)))
    return p


def _act_grad(p, act):
    if act == "relu":
        return (p > 0).to(p.dtype)
    if act == "silu":
        sg = 1 / (1 + torch.exp(-p))
        return sg * (1 + p * (1 - sg))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(p * 0.5 ** 0.5)) + p * torch.exp(-0.5 * p * p) * (2 * math.pi) ** -0.5
    c = (2 / math.pi) ** 0.5
    t = torch.tanh(c * (p + 0.044715 * p * p * p))
    return 0.5 * (1 + t) + 0.5 * p * (1 - t * t) * c * (1 + 3 * 0.044715 * p * p)


def _plain_linear(s):
    case = s["case"]
    p = s["x"].float() @ s["w"].float().t()
    if s["b"] is not None:
        p = p + s["b"]
    y = _act(p, case["act"])
    if s["res"] is not None:
        y = y + s["res"].float()
    out = {"y": y.to(s["y"].dtype)}
    if s["pre"] is not None:
        out["pre"] = p.to(torch.bfloat16)
    return out


def _plain_linear_backward(s):
    d = s["dy"].float()
    if s["pre"] is not None:
        d = d * _act_grad(s["pre"].float(), s["case"]["act"])
    out = {"dx": (d @ s["w"].float()).to(torch.bfloat16), "dw": (d.t() @ s["x"].float()).to(torch.bfloat16)}
    if s["b"] is not None:
        out["db"] = d.double().sum(0).float()
    return out


def _scores(logits, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-logits))
    e = torch.exp(logits - logits.max(1, keepdim=True).values)
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    case = s["case"]
    T, E, k, G = case["T"], case["E"], case["k"], case["n_groups"]
    # 64 bits: choices next to a border must not depend on the rounding of the scores
    score = _scores(s["logits"].double(), case["score"])
    choice = score if s["bias"] is None else score + s["bias"].double()
    if G > 1:
        in_group = torch.sort(choice.view(T, G, E // G), dim=2, descending=True).values
        of_group = in_group[:, :, : case["group_top"]].sum(2)
        best = torch.sort(of_group, dim=1, descending=True, stable=True).indices[:, : case["topk_groups"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=choice.device).scatter_(1, best, True)
        choice = torch.where(open_.repeat_interleave(E // G, dim=1), choice, -math.inf)
    ids = torch.sort(choice, dim=1, descending=True, stable=True).indices[:, :k]
    w = score.gather(1, ids)
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    out = {"ids": ids.to(torch.int32), "weights": (w * case["scale"]).float()}
    if case["scores"]:
        out["scores"] = score.float()
    return out


def _plain_route_backward(s):
    case = s["case"]
    score = _scores(s["logits"], case["score"])
    ids = s["ids"].long()
    ds = torch.zeros_like(score) if s["dscores"] is None else s["dscores"].clone()
    g = s["dweights"] * case["scale"]
    if case["renormalize"]:
        kept = score.gather(1, ids)
        total = kept.sum(1, keepdim=True)
        g = (g - (g * kept).sum(1, keepdim=True) / total) / total
    ds.scatter_add_(1, ids, g)
    if case["score"] == "sigmoid":
        return {"dlogits": ds * score * (1 - score)}
    return {"dlogits": score * (ds - (ds * score).sum(1, keepdim=True))}


def _plain_combine_backward(s):
    case = s["case"]
    T, k, S = case["T"], case["k"], case["shared"]
    row = s["slot_to_row"].long()
    w = s["weights"].flatten()
    token = torch.arange(T * k, device=row.device) // k
    if S:
        w = torch.cat((w, torch.ones(T, device=row.device)))
        token = torch.cat((token, torch.arange(T, device=row.device)))
    slot = torch.nonzero(row >= 0).flatten()
    at = row[slot]
    dy_rows = s["dy"].float()[token[slot]]
    dy_perm = torch.empty(s["rows"], case["d"], dtype=torch.bfloat16, device=row.device)
    dy_perm[at] = (dy_rows * w[slot, None]).to(torch.bfloat16)
    # 64 bits: a row's gradient may be small next to the terms that it sums
    dots = torch.zeros(row.numel(), device=row.device)
    dots[slot] = (dy_rows.double() * s["y_perm"][at]).sum(1).float()
    return {"dy_perm": dy_perm, "dweights": dots[: T * k].view(T, k)}


_PLAIN = {"linear": _plain_linear, "linear_backward": _plain_linear_backward, "route": _plain_route,
          "route_backward": _plain_route_backward, "combine_backward": _plain_combine_backward}


# ---- the package's calls ----

def _handles(s):
    """The descriptors and the workspace that a program makes once and keeps."""
    import sparse_mixture_experts_topk_amd as moe
    case = s["case"]
    h = {"moe": moe, "ws": None}
    if case["op"] in ("linear", "linear_backward"):
        h["lin"] = moe.make_linear(case["M"], case["N"], case["K"], y_dtype=case["out"], act=case["act"])
        call = moe.MOE_CALL_LINEAR if case["op"] == "linear" else moe.MOE_CALL_LINEAR_BACKWARD
        n = moe.moe_linear_workspace_bytes(h["lin"], call)
        h["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
        return h
    h["shape"] = moe.make_shape(case["T"], case.get("d", D_MODEL), D_FF, case["E"], case["k"],
                                n_shared=case.get("shared", 0))
    if case["op"] != "combine_backward":
        h["router"] = moe.make_router(case["score"], case.get("n_groups", 1), case.get("topk_groups", 1),
                                      case.get("group_top", 1), case["renormalize"], case["scale"])
    return h


def _own(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    h = s["handles"]
    moe, op = h["moe"], s["case"]["op"]
    if op == "linear":
        moe.moe_linear(h["lin"], s["x"], s["w"], s["b"], s["res"], s["y"], s["pre"], h["ws"])
        return {"y": s["y"]} if s["pre"] is None else {"y": s["y"], "pre": s["pre"]}
    if op == "linear_backward":
        moe.moe_linear_backward(h["lin"], s["dy"], s["pre"], s["x"], s["w"], s["dx"], s["dw"], s["db"], h["ws"])
        out = {"dx": s["dx"], "dw": s["dw"]}
        return out if s["db"] is None else {**out, "db": s["db"]}
    if op == "route":
        moe.moe_route_scored(h["shape"], h["router"], s["logits"], s["bias"], s["ids"], s["weights"], s["scores"])
        out = {"ids": s["ids"], "weights": s["weights"]}
        return out if s["scores"] is None else {**out, "scores": s["scores"]}
    if op == "route_backward":
        moe.moe_route_scored_backward(h["shape"], h["router"], s["logits"], s["ids"], s["dweights"], s["dscores"],
                                      s["dlogits"])
        return {"dlogits": s["dlogits"]}
    moe.moe_combine_backward(h["shape"], s["dy"], s["y_perm"], s["slot_to_row"], s["weights"], s["dy_perm"],
                             s["dweights"])
    return {"dy_perm": s["dy_perm"][: s["rows"]], "dweights": s["dweights"]}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ----

def work(case):
    op = case["op"]
    if op in ("linear", "linear_backward"):
        M, N, K = case["M"], case["N"], case["K"]
        ob = 4 if case["out"] == "f32" else 2
        b = 4 * N if case["bias"] else 0
        if op == "linear":
            nbytes = 2 * M * K + 2 * N * K + b + M * N * (ob * (2 if case["residual"] else 1)
                                                          + (2 if case["save_pre"] else 0))
            return {"bytes": nbytes, "flops": 2 * M * N * K}
        nbytes = M * N * (ob + (2 if case["act"] != "none" else 0)) + 4 * (M * K + N * K) + b
        return {"bytes": nbytes, "flops": 4 * M * N * K}
    T, E, k = case["T"], case["E"], case["k"]
    if op == "route":
        return {"bytes": 4 * T * E * (2 if case["scores"] else 1) + 8 * T * k + (4 * E if case["bias"] else 0),
                "flops": 8 * T * E}
    if op == "route_backward":
        return {"bytes": 4 * T * E * (3 if case["dscores"] else 2) + 8 * T * k, "flops": 8 * T * E}
    d, S = case["d"], case["shared"]
    slots = T * k - _n_dropped(case)
    return {"bytes": 2 * T * d + slots * d * 4 + (slots + S * T) * d * 2 + 4 * T * (3 * k + S), "flops": 3 * slots * d}


# ---- the definitions in 64 bits ----

def _phi(p, act):
    """(act(p), act'(p)) in 64 bits."""
    one = torch.ones_like(p)
    if act == "none":
        return p, one
    if act == "relu":
        return torch.where(p > 0, p, torch.zeros_like(p)), torch.where(p > 0, one, torch.zeros_like(p))
    if act == "silu":
        sg = torch.special.expit(p)
        return p * sg, sg + p * sg * torch.special.expit(-p)
    if act == "gelu":
        cdf = torch.special.ndtr(p)
        return p * cdf, cdf + p * torch.exp(-p.square() / 2) / math.sqrt(2 * math.pi)
    a = math.sqrt(8 / math.pi)                    # 1 + tanh(u / 2) = 2 / (1 + e^-u)
    sg = torch.special.expit(a * (p + 0.044715 * p ** 3))
    return p * sg, sg + p * sg * (1 - sg) * a * (1 + 0.134145 * p.square())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        p = torch.matmul(s["x"].double(), s["w"].double().t().contiguous())
        if s["b"] is not None:
            p += s["b"].double()
        y = _phi(p, case["act"])[0]
        if s["res"] is not None:
            y = y + s["res"].double()
        return {"y": y} if s["pre"] is None else {"y": y, "pre": p}
    if op == "linear_backward":
        d = s["dy"].double()
        if s["pre"] is not None:
            d = d * _phi(s["pre"].double(), case["act"])[1]
        out = {"dx": torch.matmul(d, s["w"].double()), "dw": torch.matmul(d.t().contiguous(), s["x"].double())}
        return out if s["db"] is None else {**out, "db": d.sum(0)}
    if op == "combine_backward":
        T, k, S, d = case["T"], case["k"], case["shared"], case["d"]
        row = s["slot_to_row"].long()
        dy = s["dy"].double()
        dy_perm = torch.zeros(s["rows"], d, dtype=torch.float64, device=dy.device)
        dw = torch.zeros(T, k, dtype=torch.float64, device=dy.device)
        for j in range(k + S):
            at = row[: T * k].view(T, k)[:, j] if j < k else row[T * k:]
            t = torch.nonzero(at >= 0).flatten()
            if j < k:
                dy_perm[at[t]] = dy[t] * s["weights"][t, j, None].double()
                dw[t, j] = torch.linalg.vecdot(dy[t], s["y_perm"][at[t]].double())
            else:
                dy_perm[at[t]] = dy[t]
        return {"dy_perm": dy_perm, "dweights": dw}
    x = s["logits"].double()
    p = torch.special.expit(x) if case["score"] == "sigmoid" else torch.softmax(x, 1)
    if op == "route":
        T, E, k, G = case["T"], case["E"], case["k"], case["n_groups"]
        c = (p if s["bias"] is None else p + s["bias"].double()).view(T, G, E // G)
        top = c.topk(case["group_top"], dim=2).values.sum(2)
        shut = torch.ones(T, G, 1, dtype=torch.bool, device=x.device)
        shut.scatter_(1, top.topk(case["topk_groups"], dim=1).indices[:, :, None], False)
        ids = c.masked_fill(shut, -math.inf).view(T, E).topk(k, dim=1).indices
        w = torch.take_along_dim(p, ids, 1)
        if case["renormalize"]:
            w = w / w.sum(1, keepdim=True)
        out = {"ids": None, "weights": w * case["scale"]}
        return {**out, "scores": p} if case["scores"] else out
    # the gradient by the chain rule through ln s: d ln s / d logit is (1 - s) or (I - s)
    ids = s["ids"].long()
    kept = torch.zeros_like(p).scatter_(1, ids, 1.0)
    w = p * kept
    if case["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    g = torch.zeros_like(p).scatter_(1, ids, s["dweights"].double()) * case["scale"]
    at_log = w * g
    if case["renormalize"]:
        at_log = at_log - w * (w * g).sum(1, keepdim=True)
    if s["dscores"] is not None:
        at_log = at_log + s["dscores"].double() * p
    if case["score"] == "sigmoid":
        return {"dlogits": at_log * torch.special.expit(-x)}
    return {"dlogits": at_log - p * at_log.sum(1, keepdim=True)}
