"""Measured cases of the operators that train the feed-forward blocks.

``run`` makes one pass through an operator: with ``own`` unset in its plain form
(elementary torch operations in 32 or 64 bits), with ``own`` set through the
package's entry points.

  gate_up           h = act(x w1^T) * (x w3^T), rows grouped by expert or dense,
                    the two pre-activations kept or not
  backward          dx, dw1, dw3, dw2 of y = h w2^T from dy and what was kept
  permute_backward  gradient at the tokens from the gradient at the experts' rows
  clip              the norm over a list of gradients, and the list scaled to it
"""
import math

import torch

own = False

D_MODEL, D_FF = 4096, 14336        # the layer's widths; fine-grained experts: 2048
FINE_E, FINE_K, FINE_FF = 256, 8, 2048


def listed():
    return [
        # one token through a dense gated block while decoding: reads both weights once
        {"name": "gate up 1 token", "op": "gate_up", "rows": 1, "groups": 1, "d": D_MODEL, "f": D_FF,
         "dtype": "bf16", "act": "silu", "keep": False, "behind": 0},
        # a chunk of a prompt of odd length through a shared expert, activations kept
        {"name": "gate up 509 tokens", "op": "gate_up", "rows": 509, "groups": 1, "d": D_MODEL, "f": FINE_FF,
         "dtype": "bf16", "act": "gelu_tanh", "keep": True, "behind": 0},
        # a training batch of 4096 tokens, two experts of eight each, activations kept
        {"name": "gate up 8 experts", "op": "gate_up", "rows": 8192, "groups": 8, "d": D_MODEL, "f": D_FF,
         "dtype": "bf16", "act": "silu", "keep": True, "behind": 0},
        # a short batch over many small experts, a tenth of the slots dropped: a few rows each
        {"name": "gate up 256 experts", "op": "gate_up", "rows": 7351, "groups": FINE_E, "d": D_MODEL, "f": FINE_FF,
         "dtype": "bf16", "act": "silu", "keep": True, "behind": 817},
        # gradients of a small layer in fp32
        {"name": "back fp32", "op": "backward", "rows": 128, "groups": 8, "d": 128, "f": 256,
         "dtype": "f32", "act": "silu", "behind": 0},
        # gradients of a shared expert over a short batch of odd length
        {"name": "back 509 tokens", "op": "backward", "rows": 509, "groups": 1, "d": D_MODEL, "f": FINE_FF,
         "dtype": "bf16", "act": "gelu_tanh", "behind": 0},
        # gradients of the experts over a training batch of 4096 tokens
        {"name": "back 8 experts", "op": "backward", "rows": 8192, "groups": 8, "d": D_MODEL, "f": D_FF,
         "dtype": "bf16", "act": "silu", "behind": 0},
        # gradients of many small experts: a few rows each
        {"name": "back 256 experts", "op": "backward", "rows": 7351, "groups": FINE_E, "d": D_MODEL, "f": FINE_FF,
         "dtype": "bf16", "act": "silu", "behind": 817},
        # gradient of the grouping: a small batch over few experts with a capacity
        {"name": "permute back 61 tokens", "op": "permute_backward", "T": 61, "d": D_MODEL, "k": 2, "shared": 0,
         "dropped": 0.1, "addend": False, "dtype": "bf16"},
        # a training batch over many experts and the shared one, added to the gate's gradient
        {"name": "permute back 8192 tokens", "op": "permute_backward", "T": 8192, "d": D_MODEL, "k": FINE_K,
         "shared": 1, "dropped": 0.0, "addend": True, "dtype": "bf16"},
        # the gradients of a gate and a small dense layer
        {"name": "clip gate", "op": "clip", "sizes": "1048576 256 262144 520 1", "dtypes": "bf16 f32 bf16 f32 f32",
         "norm_to": 0.3},
        # the gradients of a layer's eight experts and its gate
        {"name": "clip 8 experts", "op": "clip", "sizes": "469762048 469762048 469762048 32768 8",
         "dtypes": "bf16 bf16 bf16 bf16 f32", "norm_to": 0.3},
    ]


def _log_int(rng, lo, hi, step=1):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))
    return max(lo, min(hi, int(v) // step * step))


def draw(rng):
    op = rng.choice(("gate_up", "gate_up", "backward", "backward", "permute_backward", "clip"))
    if op in ("gate_up", "backward"):
        dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
        most = 8192 * D_FF * D_MODEL // (16 if dtype == "f32" else 1)
        while True:
            rows, groups = _log_int(rng, 1, 8192), rng.choice((1, 1, 1, 2, 8, 9, 60, 64, 128, 256, 257))
            d, f = _log_int(rng, 64, D_MODEL, 8), _log_int(rng, 64, D_FF, 8)
            # products, weights and activations no larger than those of the largest listed case
            if rows * d * f <= most and groups * d * f <= 8 * D_FF * D_MODEL and rows * (d + f) <= 8192 * (D_FF + D_MODEL):
                break
        case = {"op": op, "rows": rows, "groups": groups, "d": d, "f": f, "dtype": dtype,
                "act": rng.choice(("silu", "silu", "gelu", "gelu_tanh", "relu", "none")),
                "behind": rng.choice((0, 0, 1, 37)) if groups > 1 else 0}
        if op == "gate_up":
            case["keep"] = rng.random() < 0.6
        return case
    if op == "permute_backward":
        return {"op": op, "T": _log_int(rng, 1, 8192), "d": _log_int(rng, 64, D_MODEL, 64), "k": rng.choice((1, 2, 4, 6, 8)),
                "shared": rng.choice((0, 1)), "dropped": rng.choice((0.0, 0.05, 0.3)), "addend": rng.random() < 0.5,
                "dtype": rng.choice(("bf16", "bf16", "f32"))}
    count = rng.choice((1, 2, 5, 12, 40, 300))
    most = 400_000_000 // count
    return {"op": op, "sizes": " ".join(str(_log_int(rng, 1, most)) for _ in range(count)),
            "dtypes": " ".join(rng.choice(("bf16", "bf16", "f32")) for _ in range(count)),
            "norm_to": rng.choice((0.01, 0.3, 0.9, 2.0))}


def _n_dropped(case):
    return int(case["T"] * case["k"] * case["dropped"])


_DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _tensors(case):
    return [(int(n), _DT[t]) for n, t in zip(case["sizes"].split(), case["dtypes"].split())]


# ---- inputs ----

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dev = "cuda"

    def normal(*shape, std=1.0, dtype=torch.float32):
        return torch.empty(*shape, device=dev, dtype=dtype).normal_(0, std, generator=g)

    op = case["op"]
    s = {"case": case}
    if op in ("gate_up", "backward"):
        R, G, d, f, dt = case["rows"], case["groups"], case["d"], case["f"], _DT[case["dtype"]]
        M = R + case["behind"]                          # rows of the buffers; those behind the last group hold nothing
        # uneven groups, some of them empty where there are few rows
        load = torch.softmax(normal(G, std=0.5), 0)
        of = torch.multinomial(load, R, replacement=True, generator=g)
        counts = torch.bincount(of, minlength=G)
        s["offsets"] = torch.cat((torch.zeros(1, dtype=torch.int64, device=dev), counts.cumsum(0))).to(torch.int32)
        s["x"] = normal(M, d, dtype=dt)
        s["w1"] = normal(G, f, d, std=d ** -0.5, dtype=dt)
        s["w3"] = normal(G, f, d, std=d ** -0.5, dtype=dt)
        if op == "gate_up":
            s["h"] = torch.zeros(M, f, dtype=dt, device=dev)
            s["pre1"], s["pre3"] = (torch.zeros(M, f, dtype=dt, device=dev) if case["keep"] else None for _ in range(2))
        else:
            s["w2"] = normal(G, d, f, std=f ** -0.5, dtype=dt)
            s["pre1"], s["pre3"] = (normal(M, f, dtype=dt) for _ in range(2))
            s["h"] = (_act(s["pre1"].float(), case["act"]) * s["pre3"].float()).to(dt)
            s["dy"] = normal(M, d, std=0.01, dtype=dt)
            s["dx"] = torch.zeros(M, d, dtype=dt, device=dev)
            s["dw1"], s["dw3"] = (torch.empty(G, f, d, dtype=dt, device=dev) for _ in range(2))
            s["dw2"] = torch.empty(G, d, f, dtype=dt, device=dev)
        return s
    if op == "permute_backward":
        T, d, k, S, dt = case["T"], case["d"], case["k"], case["shared"], _DT[case["dtype"]]
        drop = torch.zeros(T * k, dtype=torch.bool, device=dev)
        drop[torch.randperm(T * k, device=dev, generator=g)[: _n_dropped(case)]] = True
        # kept slots in the order of some grouping by expert, the shared expert's rows last
        order = torch.argsort(torch.where(drop, 2.0, torch.rand(T * k, device=dev, generator=g)))
        row = torch.empty(T * k, dtype=torch.int64, device=dev)
        row[order] = torch.arange(T * k, device=dev)
        kept = T * k - _n_dropped(case)
        row = torch.where(drop, -1, row)
        if S:
            row = torch.cat((row, kept + torch.arange(T, device=dev)))
        s["slot_to_row"] = row.to(torch.int32)
        s["dx_perm"] = normal(T * (k + S), d, std=0.01, dtype=dt)
        s["addend"] = normal(T, d, std=0.01, dtype=dt) if case["addend"] else None
        s["dx"] = torch.empty(T, d, dtype=dt, device=dev)
        return s
    sizes = _tensors(case)
    s["grads"] = [normal(n, std=0.01 * (1 + i % 3), dtype=dt) for i, (n, dt) in enumerate(sizes)]
    s["outs"] = [torch.empty_like(t) for t in s["grads"]]
    # a bound at the given share of the norm that such gradients have
    s["max_norm"] = case["norm_to"] * math.sqrt(sum(n * (0.01 * (1 + i % 3)) ** 2 for i, (n, _) in enumerate(sizes)))
    s["sum"] = torch.empty(1, dtype=torch.float64, device=dev)
    s["norm"] = torch.empty(1, device=dev)
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
    if act == "none":
        return torch.ones_like(p)
    c = (2 / math.pi) ** 0.5
    t = torch.tanh(c * (p + 0.044715 * p * p * p))
    return 0.5 * (1 + t) + 0.5 * p * (1 - t * t) * c * (1 + 3 * 0.044715 * p * p)


def _spans(s):
    """(group, first row, end) of the groups that have rows."""
    o = s["offsets"].tolist()
    return [(e, o[e], o[e + 1]) for e in range(len(o) - 1) if o[e + 1] > o[e]]


def _plain_gate_up(s):
    case = s["case"]
    names = ("h", "pre1", "pre3") if case["keep"] else ("h",)
    out = {n: torch.empty(case["rows"], case["f"], dtype=s["x"].dtype, device=s["x"].device) for n in names}
    for e, a, b in _spans(s):
        x = s["x"][a:b].float()
        p, q = x @ s["w1"][e].float().t(), x @ s["w3"][e].float().t()
        out["h"][a:b] = (_act(p, case["act"]) * q).to(out["h"].dtype)
        if case["keep"]:
            out["pre1"][a:b], out["pre3"][a:b] = p.to(s["x"].dtype), q.to(s["x"].dtype)
    return out


def _plain_backward(s):
    case = s["case"]
    dt = s["x"].dtype
    out = {"dx": torch.empty(case["rows"], case["d"], dtype=dt, device=s["x"].device)}
    for n in ("w1", "w3", "w2"):
        out["d" + n] = torch.zeros_like(s[n])
    for e, a, b in _spans(s):
        dy, p, q = s["dy"][a:b].float(), s["pre1"][a:b].float(), s["pre3"][a:b].float()
        x = s["x"][a:b].float()
        dh = dy @ s["w2"][e].float()
        dp, dq = dh * q * _act_grad(p, case["act"]), dh * _act(p, case["act"])
        out["dx"][a:b] = (dp @ s["w1"][e].float() + dq @ s["w3"][e].float()).to(dt)
        out["dw1"][e] = (dp.t() @ x).to(dt)
        out["dw3"][e] = (dq.t() @ x).to(dt)
        out["dw2"][e] = (dy.t() @ s["h"][a:b].float()).to(dt)
    return out


def _plain_permute_backward(s):
    case = s["case"]
    T, k, S = case["T"], case["k"], case["shared"]
    row = s["slot_to_row"].long()
    rows = torch.where((row >= 0)[:, None], s["dx_perm"][row.clamp(min=0)].float(), 0.0)     # of every slot
    dx = rows[: T * k].view(T, k, -1).sum(1)
    if S:
        dx = dx + rows[T * k:]
    if s["addend"] is not None:
        dx = dx + s["addend"].float()
    return {"dx": dx.to(s["dx"].dtype)}


def _plain_clip(s):
    # 64 bits: a long sum
    total = sum((t.double() * t.double()).sum() for t in s["grads"])
    norm = torch.sqrt(total)
    scale = torch.clamp(s["max_norm"] / norm, max=1.0).float()
    return {"norm": norm.float().view(1), "grads": [(t.float() * scale).to(t.dtype) for t in s["grads"]]}


_PLAIN = {"gate_up": _plain_gate_up, "backward": _plain_backward, "permute_backward": _plain_permute_backward,
          "clip": _plain_clip}


# ---- the package's calls ----

def _handles(s):
    """The descriptors and the workspace that a program makes once and keeps."""
    import sparse_mixture_experts_topk_amd as moe
    case = s["case"]
    h = {"moe": moe, "ws": None}
    n = 0
    if case["op"] in ("gate_up", "backward"):
        h["ffn"] = moe.make_ffn(case["rows"] + case["behind"], case["d"], case["f"], case["groups"], case["dtype"], case["act"])
        h["offsets"] = s["offsets"] if case["groups"] > 1 else None
        n = moe.moe_ffn_workspace_bytes(h["ffn"], moe.MOE_CALL_FFN_GATE_UP if case["op"] == "gate_up"
                                        else moe.MOE_CALL_FFN_BACKWARD)
    elif case["op"] == "permute_backward":
        h["shape"] = moe.make_shape(case["T"], case["d"], D_FF, 8, case["k"], act_dtype=case["dtype"],
                                    w_dtype=case["dtype"], n_shared=case["shared"])
    else:
        h["grads"], h["outs"] = moe.make_tensors(s["grads"]), moe.make_tensors(s["outs"])
        n = moe.moe_grad_norm_workspace_bytes(h["grads"])
    h["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda") if n else None
    return h


def _own(s):
    if "handles" not in s:
        s["handles"] = _handles(s)
    h = s["handles"]
    moe, case = h["moe"], s["case"]
    op = case["op"]
    if op == "gate_up":
        moe.moe_ffn_gate_up(h["ffn"], s["x"], h["offsets"], s["w1"], s["w3"], s["h"], s["pre1"], s["pre3"], h["ws"])
        return {n: s[n][: case["rows"]] for n in (("h", "pre1", "pre3") if case["keep"] else ("h",))}
    if op == "backward":
        moe.moe_ffn_backward(h["ffn"], s["dy"], h["offsets"], s["x"], s["pre1"], s["pre3"], s["h"], s["w1"], s["w3"],
                             s["w2"], s["dx"], s["dw1"], s["dw3"], s["dw2"], h["ws"])
        return {"dx": s["dx"][: case["rows"]], "dw1": s["dw1"], "dw3": s["dw3"], "dw2": s["dw2"]}
    if op == "permute_backward":
        moe.moe_permute_backward(h["shape"], s["dx_perm"], s["slot_to_row"], s["addend"], s["dx"])
        return {"dx": s["dx"]}
    moe.moe_grad_norm(h["grads"], s["sum"], s["norm"], h["ws"])
    moe.moe_grad_clip(h["grads"], h["outs"], s["sum"], s["max_norm"])
    return {"norm": s["norm"], "grads": s["outs"]}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- what a pass cannot do without ----

def work(case):
    op = case["op"]
    if op in ("gate_up", "backward"):
        R, G, d, f, b = case["rows"], case["groups"], case["d"], case["f"], 4 if case["dtype"] == "f32" else 2
        read = min(G, R) * d * f                        # one weight of every group that can have rows
        if op == "gate_up":
            return {"bytes": b * (R * d + 2 * read + R * f * (3 if case["keep"] else 1)), "flops": 4 * R * d * f}
        return {"bytes": b * (R * (3 * d + 3 * f) + 3 * read + 3 * G * d * f), "flops": 12 * R * d * f}
    if op == "permute_backward":
        T, k, S, d, b = case["T"], case["k"], case["shared"], case["d"], 4 if case["dtype"] == "f32" else 2
        rows = T * (k + S) - _n_dropped(case)
        return {"bytes": b * d * (rows + T * (2 if case["addend"] else 1)) + 4 * T * (k + S), "flops": rows * d}
    sizes = _tensors(case)
    return {"bytes": sum(2 * n * dt.itemsize for n, dt in sizes), "flops": 3 * sum(n for n, _ in sizes)}


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


def _exact_group(s, e, a, b):
    """The outputs of one group's rows [a, b)."""
    case = s["case"]
    x, w1, w3 = s["x"][a:b].double(), s["w1"][e].double(), s["w3"][e].double()
    if case["op"] == "gate_up":
        p, q = torch.matmul(x, w1.t().contiguous()), torch.matmul(x, w3.t().contiguous())
        return {"h": _phi(p, case["act"])[0] * q, "pre1": p, "pre3": q}
    dy, w2 = s["dy"][a:b].double(), s["w2"][e].double()
    value, slope = _phi(s["pre1"][a:b].double(), case["act"])
    dh = torch.matmul(dy, w2)
    both = torch.cat((dh * slope * s["pre3"][a:b].double(), dh * value), 1)         # at [g u] = x [w1; w3]^T
    dw = torch.matmul(both.t().contiguous(), x)
    return {"dx": torch.matmul(both, torch.cat((w1, w3), 0)), "dw1": dw[: case["f"]], "dw3": dw[case["f"]:],
            "dw2": torch.matmul(dy.t().contiguous(), s["h"][a:b].double())}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gate_up", "backward"):
        R, G, d, f = case["rows"], case["groups"], case["d"], case["f"]
        out = {"h": (R, f), "pre1": (R, f), "pre3": (R, f)} if op == "gate_up" else \
              {"dx": (R, d), "dw1": (G, f, d), "dw3": (G, f, d), "dw2": (G, d, f)}
        if op == "gate_up" and not case["keep"]:
            out = {"h": (R, f)}
        out = {n: torch.zeros(*shape, dtype=torch.float64, device="cuda") for n, shape in out.items()}
        ends = s["offsets"].long().cpu()
        for e in range(G):
            a, b = int(ends[e]), int(ends[e + 1])
            if a == b:
                continue
            part = _exact_group(s, e, a, b)
            for n in out:
                if n.startswith("dw"):
                    out[n][e] = part[n]
                else:
                    out[n][a:b] = part[n]
        return out
    if op == "permute_backward":
        T, k, S = case["T"], case["k"], case["shared"]
        dx = torch.zeros(T, case["d"], dtype=torch.float64, device="cuda")
        if s["addend"] is not None:
            dx += s["addend"]
        rows = s["dx_perm"].double()
        at = s["slot_to_row"].long()
        for j in range(k + S):
            r = at[: T * k].view(T, k)[:, j] if j < k else at[T * k:]
            dx += torch.where((r >= 0)[:, None], rows[r.clamp(min=0)], 0.0)
        return {"dx": dx}
    norm = math.sqrt(math.fsum(float(torch.linalg.vector_norm(t, dtype=torch.float64)) ** 2 for t in s["grads"]))
    factor = s["max_norm"] / norm if norm > s["max_norm"] else 1.0
    return {"norm": torch.tensor([norm], dtype=torch.float64, device="cuda"),
            "grads": [t.double() * factor for t in s["grads"]]}
