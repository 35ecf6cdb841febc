"""Cases of the operators around the experts' products, in plain torch and through the library.

unpermute: expert rows back to their tokens with the routing weights applied, and the gradients of
    that (rows, weights, router logits) and of the gather that sorted the tokens by expert.
norm: layer norm forward and backward, and rms_norm's backward, with the weight's gradient.
linear: a product with bias, activation and residual in its epilogue, and its gradients.
"""
import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6
ACTS = ("none", "relu", "silu", "gelu", "gelu_tanh")


# ------------------------------------------------------------------ cases --

def _rows(name, way, T, H, E, k, y, stream, res, drop, logits=False):
    """way: "return" (weighted sum back to the tokens), "return grad" or "gather grad".  y: type of
    the expert rows; stream: type of the token rows.  res: a residual (or the gradient that arrives
    past the block) is added.  drop: share of pairs over their expert's capacity.  logits: the
    gradient goes on to the router's logits."""
    return {"name": name, "op": "rows", "way": way, "T": T, "H": H, "E": E, "k": k, "y": y,
            "stream": stream, "res": res, "drop": drop, "logits": logits}


def _norm(name, way, T, H, x, dy, w, bias, res):
    """way: "layer" (forward), "layer grad" or "rms grad".  x: type of the rows (and of dx), dy: type of
    the forward's output and of its gradient.  w: type of the weights.  res: the gradient of the
    residual stream is added to dx."""
    return {"name": name, "op": "norm", "way": way, "T": T, "H": H, "x": x, "dy": dy, "w": w,
            "bias": bias, "res": res}


def _linear(name, way, M, N, K, act, bias, res, out):
    """way: "forward", "forward pre" (the values before the activation are kept for the backward pass)
    or "grad".  res: "none", "bf16" or "fp32" residual.  out: type of the output; of the weight's
    gradient with "grad"."""
    return {"name": name, "op": "linear", "way": way, "M": M, "N": N, "K": K, "act": act, "bias": bias,
            "res": res, "out": out}


def listed():
    return [
        # one user decoding: eight expert rows and the shared expert's
        _rows("return one token", "return", 1, 4096, 64, 8, "bf16", "bf16", True, 0.0),
        # a training batch: the expert rows are most of the bytes
        _rows("return batch", "return", 4096, 4096, 64, 8, "bf16", "bf16", True, 0.0),
        # its gradient, down to the router's logits
        _rows("return gradient", "return grad", 4096, 4096, 64, 8, "bf16", "bf16", False, 0.0, True),
        # a ragged batch with an expert capacity, fp32 token gradients
        _rows("gather gradient dropped", "gather grad", 1999, 2944, 256, 6, "bf16", "fp32", True, 0.1),
        # a decode batch in front of an attention block
        _norm("layer norm decode", "layer", 16, 4096, "bf16", "bf16", "bf16", True, False),
        # a training batch of a wide model
        _norm("layer norm batch", "layer", 8192, 7168, "bf16", "bf16", "bf16", True, False),
        # its backward pass: rows, weights, bias, residual gradient
        _norm("layer norm gradient", "layer grad", 8192, 7168, "bf16", "bf16", "bf16", True, True),
        # the block's own norm on an fp32 residual stream, a ragged batch
        _norm("rms norm gradient", "rms grad", 2047, 5120, "fp32", "bf16", "bf16", False, False),
        # one user decoding: an output projection, its weights read once
        _linear("linear one token", "forward", 1, 4096, 4096, "none", False, "bf16", "bf16"),
        # a decode batch through a shared expert's projection, odd row count
        _linear("linear decode", "forward", 61, 7168, 2048, "none", True, "fp32", "fp32"),
        # a training batch into a dense layer, the values before the activation kept
        _linear("linear batch", "forward pre", 4096, 12288, 4096, "gelu_tanh", True, "none", "bf16"),
        # the backward pass of such a layer
        _linear("linear gradient", "grad", 4096, 12288, 4096, "silu", True, "none", "bf16"),
    ]


def _spread(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return min(hi, max(lo, int(v / step + 0.5) * step))


def draw(rng):
    op = rng.choice(["rows", "norm", "linear"])
    types = ["bf16", "bf16", "fp32"]
    if op == "rows":
        way = rng.choice(["return", "return grad", "gather grad"])
        E = _spread(rng, 8, 256, 1)
        k = rng.choice([1, 2, 4, 6, 8])
        T, H = _spread(rng, 1, 8192, 1), _spread(rng, 256, 8192, 8)
        y, stream = rng.choice(types), rng.choice(types)
        while T * H * (2 * k + 1) * (2 if y == "fp32" or stream == "fp32" else 1) > 4096 * 4096 * 17:
            T = (T + 1) // 2
        c = _rows("", way, T, H, E, k, y, stream, way != "return grad" and rng.random() < 0.5,
                  rng.choice([0.0, 0.0, 0.1, 0.5]), way == "return grad" and rng.random() < 0.5)
    elif op == "norm":
        way = rng.choice(["layer", "layer grad", "rms grad"])
        T, H = _spread(rng, 1, 16384, 1), _spread(rng, 128, 8192, 8)
        x, dy = rng.choice(types), rng.choice(types)
        while T * H * (2 if x == "fp32" or dy == "fp32" else 1) > 8192 * 7168:
            T = (T + 1) // 2
        c = _norm("", way, T, H, x, dy, "bf16" if way == "rms grad" else rng.choice(types),
                  way != "rms grad" and rng.random() < 0.7, way != "layer" and rng.random() < 0.5)
    else:
        way = rng.choice(["forward", "forward", "forward pre", "grad"])
        M = _spread(rng, 1 if way == "forward" else 16, 8192, 1)
        N, K = _spread(rng, 256, 12288, 8), _spread(rng, 256, 12288, 8)
        while M * N * K > 4096 * 12288 * 4096:
            M = (M + 1) // 2
        act = rng.choice(ACTS) if way != "forward pre" else rng.choice(ACTS[1:])
        c = _linear("", way, M, N, K, act, rng.random() < 0.6,
                    rng.choice(["none", "bf16", "fp32"]) if way == "forward" else "none",
                    "bf16" if way == "forward pre" or (way == "grad" and act != "none") else rng.choice(types))
    del c["name"]
    return c


def _size(t):
    return 4 if t == "fp32" else 2


def work(case):
    c = case
    if c["op"] == "rows":
        T, H, k = c["T"], c["H"], c["k"]
        live = T * k * (1.0 - c["drop"])
        rows, token = live * H * _size(c["y"]), T * H * _size(c["stream"])
        if c["way"] == "return grad":
            b = 2 * rows + token + 4 * T * k * 3 + ((4 * T * k + 4 * T * c["E"]) if c["logits"] else 0)
            return {"bytes": float(b), "flops": 3.0 * live * H}
        b = rows + token * (2 if c["res"] else 1) + 4 * T * k * (2 if c["way"] == "return" else 1)
        return {"bytes": float(b), "flops": (2.0 if c["way"] == "return" else 1.0) * live * H}
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        sx, sd = _size(c["x"]), _size(c["dy"])
        nw = 2 if c["bias"] else 1
        if c["way"] == "layer":
            return {"bytes": float(T * H * (sx + sd) + nw * H * _size(c["w"]) + 8 * T), "flops": 8.0 * T * H}
        b = T * H * (2 * sx + sd + (sx if c["res"] else 0)) + H * _size(c["w"]) + 4 * nw * H
        b += 8 * T if c["way"] == "layer grad" else 0
        return {"bytes": float(b), "flops": 14.0 * T * H}
    M, N, K = c["M"], c["N"], c["K"]
    if c["way"] == "grad":
        b = 2 * (2 * M * K + N * K + M * N * (1 if c["act"] == "none" else 2)) + N * K * _size(c["out"])
        b += 4 * N if c["bias"] else 0
        return {"bytes": float(b), "flops": 4.0 * M * N * K}
    b = 2 * (M * K + N * K) + M * N * _size(c["out"]) + (2 * N if c["bias"] else 0)
    b += {"none": 0, "bf16": 2 * M * N, "fp32": 4 * M * N}[c["res"]]
    b += 2 * M * N if c["way"] == "forward pre" else 0
    return {"bytes": float(b), "flops": 2.0 * M * N * K}


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 6151 + 29)


def _type(t):
    return torch.float32 if t == "fp32" else torch.bfloat16


def _randn(g, *shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).add_(mean).to(dtype)


def _stream(g, T, H, dtype):
    """A residual stream: some channels much larger than the rest, rows off centre."""
    chan = _randn(g, H, std=0.6, dtype=torch.float32).exp_()
    off = _randn(g, T, 1, std=0.2, mean=0.3, dtype=torch.float32)
    return (_randn(g, T, H, dtype=torch.float32) * chan + off).to(dtype)


def prepare(case, seed):
    g = _gen(seed)
    return {"rows": _prepare_rows, "norm": _prepare_norm, "linear": _prepare_linear}[case["op"]](case, g)


def _prepare_rows(c, g):
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    yt, st = _type(c["y"]), _type(c["stream"])
    s = {"case": c}
    z = _randn(g, T, E, std=1.5, dtype=torch.float32)
    top = z.sort(1, descending=True)
    s["ids"] = top.indices[:, :k].to(torch.int32).contiguous()
    p = torch.exp(top.values[:, :k] - top.values[:, :1])
    s["w"] = (p / p.sum(1, keepdim=True)).contiguous()
    # rows in expert order, then token order; pairs over the capacity have none
    key = s["ids"].reshape(-1).long()
    kept = torch.rand((T * k,), generator=g, device=DEV) >= c["drop"]
    order = torch.where(kept, key, torch.full_like(key, E)).argsort(stable=True)
    row = torch.empty(T * k, dtype=torch.int64, device=DEV)
    row[order] = torch.arange(T * k, device=DEV)
    s["row"] = torch.where(kept, row, torch.full_like(row, -1)).to(torch.int32)
    s["y"] = _randn(g, T * k, H, std=0.3, dtype=yt)
    s["res"] = _stream(g, T, H, st) if c["res"] else None
    s["dout"] = _randn(g, T, H, std=0.05, dtype=st) if c["way"] == "return grad" else None
    return s


def _prepare_norm(c, g):
    T, H = c["T"], c["H"]
    xt, dt, wt = _type(c["x"]), _type(c["dy"]), _type(c["w"])
    s = {"case": c, "x": _stream(g, T, H, xt), "w": _randn(g, H, std=0.1, mean=1.0, dtype=wt)}
    s["b"] = _randn(g, H, std=0.1, dtype=wt) if c["bias"] else None
    s["dy"] = s["res"] = s["mean"] = s["rstd"] = None
    if c["way"] != "layer":
        s["dy"] = _randn(g, T, H, std=0.05, dtype=dt)
        s["res"] = _randn(g, T, H, std=0.05, dtype=xt) if c["res"] else None
    if c["way"] == "layer grad":  # what the forward pass kept
        x = s["x"].double()
        m = x.mean(1)
        s["mean"] = m.float()
        s["rstd"] = (1 / ((x - m[:, None]).square().mean(1) + EPS).sqrt()).float()
    return s


def _prepare_linear(c, g):
    M, N, K = c["M"], c["N"], c["K"]
    s = {"case": c, "x": _randn(g, M, K), "w": _randn(g, N, K, std=K ** -0.5)}
    s["b"] = _randn(g, N, std=0.1) if c["bias"] else None
    s["res"] = None if c["res"] == "none" else _stream(g, M, N, _type(c["res"]))
    s["dout"] = s["pre"] = None
    if c["way"] == "grad":
        s["dout"] = _randn(g, M, N, std=0.05)
        s["pre"] = None if c["act"] == "none" else _randn(g, M, N)
    return s


# -------------------------------------------------------------- plain form --

def _plain_rows(s):
    c = s["case"]
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    row = s["row"].long()
    live = row >= 0
    at = row.clamp(min=0)
    y = torch.where(live[:, None], s["y"][at].float(), torch.zeros((), device=DEV)).view(T, k, H)
    if c["way"] == "return grad":
        d = s["dout"].float()
        dy = torch.zeros_like(s["y"])
        pair = (s["w"][:, :, None] * d[:, None, :]).view(T * k, H)
        dy[row[live]] = pair[live].to(dy.dtype)
        dw = (y * d[:, None, :]).sum(2)
        r = {"dy": dy, "dw": dw}
        if c["logits"]:
            v = s["w"] * (dw - (s["w"] * dw).sum(1, keepdim=True))
            r["dlogits"] = torch.zeros((T, E), device=DEV).scatter_(1, s["ids"].long(), v)
        return r
    f = (y * s["w"][:, :, None]).sum(1) if c["way"] == "return" else y.sum(1)
    if s["res"] is not None:
        f = f + s["res"].float()
    return {"out": f.to(_type(c["stream"]))}


def _plain_norm(s):
    c = s["case"]
    x, w = s["x"].float(), s["w"].float()
    if c["way"] == "layer":
        m = x.mean(1, keepdim=True)
        v = x - m
        r = 1 / (v.square().mean(1, keepdim=True) + EPS).sqrt()
        y = v * r * w
        if s["b"] is not None:
            y = y + s["b"].float()
        return {"y": y.to(_type(c["dy"])), "mean": m[:, 0], "rstd": r[:, 0]}
    dy = s["dy"].float()
    if c["way"] == "layer grad":
        xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
        g = dy * w
        dx = s["rstd"][:, None] * (g - g.mean(1, keepdim=True) - xh * (g * xh).mean(1, keepdim=True))
    else:
        r = 1 / (x.square().mean(1, keepdim=True) + EPS).sqrt()
        xh = x * r
        g = dy * w
        dx = r * (g - xh * (g * xh).mean(1, keepdim=True))
    if s["res"] is not None:
        dx = dx + s["res"].float()
    out = {"dx": dx.to(s["x"].dtype), "dw": (dy * xh).sum(0, dtype=torch.float64).float()}
    if s["b"] is not None:
        out["db"] = dy.sum(0, dtype=torch.float64).float()
    return out


def _act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    a = math.sqrt(2 / math.pi)
    t = torch.tanh(a * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * a * (1 + 3 * 0.044715 * z * z)


def _plain_linear(s):
    c = s["case"]
    x, w = s["x"].float(), s["w"].float()
    if c["way"] == "grad":
        d = s["dout"].float()
        if c["act"] != "none":
            d = d * _act_slope(s["pre"].float(), c["act"])
        r = {"dx": (d @ w).to(torch.bfloat16), "dw": (d.t() @ x).to(_type(c["out"]))}
        if s["b"] is not None:
            r["db"] = d.sum(0, dtype=torch.float64).float()
        return r
    z = x @ w.t()
    if s["b"] is not None:
        z = z + s["b"].float()
    f = _act(z, c["act"])
    if s["res"] is not None:
        f = f + s["res"].float()
    r = {"out": f.to(_type(c["out"]))}
    if c["way"] == "forward pre":
        r["pre"] = z.to(torch.bfloat16)
    return r


# ------------------------------------------------------------- the library --

def _plan_rows(s):
    """Buffers that a program keeps over its steps; rows of dy that no pair owns stay zero."""
    import moe_expert_ffn_rms_gb300 as M
    c = s["case"]
    p = {"M": M}
    if c["way"] == "return grad":
        p["dy"] = torch.zeros_like(s["y"])
        p["dw"] = torch.empty((c["T"], c["k"]), device=DEV)
        if c["logits"]:
            p["dlogits"] = torch.empty((c["T"], c["E"]), device=DEV)
    else:
        p["out"] = torch.empty((c["T"], c["H"]), dtype=_type(c["stream"]), device=DEV)
    return p


def _own_rows(s):
    if "plan" not in s:
        s["plan"] = _plan_rows(s)
    p, c = s["plan"], s["case"]
    T, k = c["T"], c["k"]
    if c["way"] == "return":
        p["M"].moe_unpermute(s["y"], s["row"], p["out"], T, k, topk_w=s["w"], residual=s["res"])
    elif c["way"] == "gather grad":
        p["M"].moe_permute_backward(s["y"], s["row"], p["out"], T, k, dres=s["res"])
    else:
        p["M"].moe_unpermute_backward(s["dout"], s["y"], s["row"], s["w"], T, k, dy=p["dy"], dw=p["dw"],
                                      ids=s["ids"] if c["logits"] else None, dlogits=p.get("dlogits"))
    return {n: p[n] for n in ("out", "dy", "dw", "dlogits") if n in p}


def _plan_norm(s):
    import moe_expert_ffn_rms_gb300 as M
    c = s["case"]
    T, H = c["T"], c["H"]
    p = {"M": M}
    if c["way"] == "layer":
        p["y"] = torch.empty((T, H), dtype=_type(c["dy"]), device=DEV)
        p["mean"], p["rstd"] = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    else:
        p["ws"] = M.alloc_workspace(M.moe_norm_backward_workspace_size(T, H), DEV)
        p["dx"], p["dw"] = torch.empty_like(s["x"]), torch.empty(H, device=DEV)
        if c["bias"]:
            p["db"] = torch.empty(H, device=DEV)
    return p


def _own_norm(s):
    if "plan" not in s:
        s["plan"] = _plan_norm(s)
    p, c = s["plan"], s["case"]
    if c["way"] == "layer":
        p["M"].moe_layernorm(s["x"], s["w"], EPS, p["y"], b=s["b"], mean=p["mean"], rstd=p["rstd"])
    elif c["way"] == "layer grad":
        p["M"].moe_layernorm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"], p["dx"], p["dw"], p["ws"],
                                      db=p.get("db"), dres=s["res"])
    else:
        p["M"].moe_rmsnorm_backward(s["dy"], s["x"], s["w"], EPS, p["dx"], p["dw"], p["ws"], dres=s["res"])
    return {n: p[n] for n in ("y", "mean", "rstd", "dx", "dw", "db") if n in p}


def _plan_linear(s):
    import moe_expert_ffn_rms_gb300 as M
    c = s["case"]
    n, m, k = c["N"], c["M"], c["K"]
    p = {"M": M, "act": getattr(M, "ACT_" + c["act"].upper())}
    if c["way"] == "grad":
        p["ws"] = M.alloc_workspace(M.moe_linear_backward_workspace_size(m, n, k), DEV)
        p["dx"] = torch.empty_like(s["x"])
        p["dw"] = torch.empty((n, k), dtype=_type(c["out"]), device=DEV)
        if c["bias"]:
            p["db"] = torch.empty(n, device=DEV)
    else:
        p["out"] = torch.empty((m, n), dtype=_type(c["out"]), device=DEV)
        if c["way"] == "forward pre":
            p["pre"] = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    return p


def _own_linear(s):
    if "plan" not in s:
        s["plan"] = _plan_linear(s)
    p, c = s["plan"], s["case"]
    if c["way"] == "grad":
        p["M"].moe_linear_backward(s["dout"], s["x"], s["w"], p["ws"], dx=p["dx"], dw=p["dw"], db=p.get("db"),
                                   pre=s["pre"], act=p["act"])
    else:
        p["M"].moe_linear(s["x"], s["w"], p["out"], bias=s["b"], residual=s["res"], act=p["act"],
                          pre=p.get("pre"))
    return {n: p[n] for n in ("out", "pre", "dx", "dw", "db") if n in p}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"rows": _own_rows, "norm": _own_norm, "linear": _own_linear}[op](state)
    return {"rows": _plain_rows, "norm": _plain_norm, "linear": _plain_linear}[op](state)


# ------------------------------------------------------------- definition --

def exact(case, seed):
    s = prepare(case, seed)
    return {"rows": _exact_rows, "norm": _exact_norm, "linear": _exact_linear}[case["op"]](case, s)


def _exact_rows(c, s):
    """Row by row of the expert order: the pairs that own a row, found from the row's side."""
    T, H, E, k = c["T"], c["H"], c["E"], c["k"]
    row = s["row"].cpu().tolist()
    owner = sorted((r, p) for p, r in enumerate(row) if r >= 0)
    r_ix = torch.tensor([r for r, _ in owner], dtype=torch.int64, device=DEV)
    p_ix = torch.tensor([p for _, p in owner], dtype=torch.int64, device=DEV)
    token = torch.div(p_ix, k, rounding_mode="floor")
    w = s["w"].double().view(-1)[p_ix]
    y = s["y"].double()[r_ix]
    if c["way"] == "return grad":
        d = s["dout"].double()[token]
        dy = torch.zeros((T * k, H), dtype=torch.float64, device=DEV)
        dy[r_ix] = d * w[:, None]
        dw = torch.zeros(T * k, dtype=torch.float64, device=DEV)
        dw[p_ix] = torch.einsum("rh,rh->r", d, y)
        r = {"dy": dy, "dw": dw.view(T, k)}
        if c["logits"]:
            # the Jacobian of the softmax over the selected logits, token by token
            ws = s["w"].double()
            jac = torch.diag_embed(ws) - ws[:, :, None] * ws[:, None, :]
            part = torch.einsum("tij,tj->ti", jac, r["dw"])
            full = torch.zeros((T, E), dtype=torch.float64, device=DEV)
            for j in range(k):
                full[torch.arange(T, device=DEV), s["ids"][:, j].long()] += part[:, j]
            r["dlogits"] = full
        return r
    out = torch.zeros((T, H), dtype=torch.float64, device=DEV) if s["res"] is None else s["res"].double()
    out.index_add_(0, token, y * w[:, None] if c["way"] == "return" else y)
    return {"out": out}


def _exact_norm(c, s):
    x = s["x"].double().requires_grad_()
    w = s["w"].double().requires_grad_()
    b = torch.zeros_like(w) if s["b"] is None else s["b"].double()
    b = b.detach().requires_grad_()
    if c["way"] == "rms grad":
        y = x * torch.rsqrt(torch.mean(x * x, 1, keepdim=True) + EPS) * w
    else:
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        y = (x - mean) * torch.rsqrt(var + EPS) * w + b
    if c["way"] == "layer":
        return {"y": y.detach(), "mean": mean.detach()[:, 0], "rstd": torch.rsqrt(var + EPS).detach()[:, 0]}
    leaves = [x, w] + ([b] if c["way"] == "layer grad" else [])
    grads = torch.autograd.grad(y, leaves, s["dy"].double())
    r = {"dx": grads[0] if s["res"] is None else grads[0] + s["res"].double(), "dw": grads[1]}
    if c["bias"]:
        r["db"] = grads[2]
    return r


def _exact_linear(c, s):
    F = torch.nn.functional
    f = {"none": lambda z: z, "relu": F.relu, "silu": F.silu, "gelu": F.gelu,
         "gelu_tanh": lambda z: F.gelu(z, approximate="tanh")}[c["act"]]
    x, w = s["x"].double(), s["w"].double()
    if c["way"] == "grad":
        d = s["dout"].double()
        if s["pre"] is not None:
            z = s["pre"].double().requires_grad_()
            d = torch.autograd.grad(f(z), z, d)[0]
        r = {"dx": torch.matmul(d, w), "dw": torch.matmul(x.t(), d).t()}
        if c["bias"]:
            r["db"] = torch.einsum("mn->n", d)
        return r
    z = torch.einsum("mk,nk->mn", x, w)
    if s["b"] is not None:
        z = z + s["b"].double()
    r = {"out": f(z) if s["res"] is None else s["res"].double() + f(z)}
    if c["way"] == "forward pre":
        r["pre"] = z
    return r
