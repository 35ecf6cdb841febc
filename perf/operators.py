"""Cases of two operators around a mixture-of-experts block, in plain torch and through the library.

moe_layer_forward: the whole block for one to eight tokens -- rms_norm, router, top-k, the experts'
    gated FFN, the weighted sum and (with a tail) what follows it.
moe_combine_norm: what follows a block for any number of tokens -- the sum of a token's expert rows,
    a norm after the block, the gate and residual scale, the residual, and the next block's norm
    with its E4M3 quantisation.

With f the block's output, the tail is
    h = residual + scale * gate * rms_norm(f; post_w)        (a missing part drops out)
    x_hat = rms_norm(h; next_w),  xq = e4m3(x_hat / s),  s = max|x_hat| / 448 per token or per 128.
"""
import torch

own = False

DEV = "cuda"
EPS = 1e-6


# ------------------------------------------------------------------ cases --

def _layer(name, T, H, E, k, I, fmt, routing, tail):
    """fmt: weights "bf16", "fp8" (a scale per output channel) or "block" (a scale per 128 x 128).
    routing: "router" (learned, in the call), "bias" (the same with a skewing bias), "logits" (given
    logits) or "ids" (given experts and weights).  tail: "none", "residual", "sandwich" (residual,
    norm after, next norm) or "gated" (sandwich with a gate per channel and a residual scale)."""
    return {"name": name, "op": "layer", "T": T, "H": H, "E": E, "k": k, "I": I, "fmt": fmt,
            "routing": routing, "tail": tail}


def _norm(name, T, H, k, y, order, stream, post, gate, nxt):
    """y: type of the expert rows; order: "pair" ((token, slot) rows) or "expert" (rows through
    row_of_pair).  stream: type of the residual.  gate: "none", "channel", "token" or "rows" (one
    row per request).  nxt: "none", "bf16", "e4m3" (per token) or "e4m3g" (per 128 columns)."""
    return {"name": name, "op": "norm", "T": T, "H": H, "k": k, "y": y, "order": order,
            "stream": stream, "post": post, "gate": gate, "next": nxt}


def listed():
    return [
        # the smoke-sized model: launch and hand-over latency is all there is
        _layer("layer tiny", 4, 256, 8, 2, 512, "bf16", "router", "none"),
        # one user decoding: eight experts of 38 MB each, read once
        _layer("layer one token", 1, 4096, 64, 8, 1536, "bf16", "router", "sandwich"),
        # the largest batch of the operator, logits from the host program; about 42 of 64 experts
        _layer("layer eight tokens", 8, 4096, 64, 8, 1536, "bf16", "logits", "residual"),
        # a wide model with skewed routing and a gated residual
        _layer("layer wide skewed", 2, 7168, 64, 8, 2048, "bf16", "bias", "gated"),
        # FP8 weights, routing decided elsewhere (the fused-experts call)
        _layer("layer fp8 routed", 1, 4096, 64, 8, 1536, "fp8", "ids", "none"),
        # block-wise FP8 weights, a few users at once
        _layer("layer fp8 block", 4, 4096, 64, 8, 1536, "block", "router", "sandwich"),
        # one token after its eight experts: latency
        _norm("norm one token", 1, 4096, 8, "bf16", "pair", "bf16", True, "none", "bf16"),
        # a decode batch on an fp32 residual stream, one gate row per request
        _norm("norm decode gated", 64, 7168, 8, "bf16", "pair", "fp32", True, "rows", "bf16"),
        # a prefill batch: the eight expert rows of each token are most of the bytes
        _norm("norm prefill", 4096, 4096, 8, "bf16", "pair", "bf16", True, "none", "bf16"),
        # after an attention block (one row per token), FP8 input of the next projection
        _norm("norm dense e4m3", 2047, 5120, 1, "bf16", "pair", "fp32", False, "token", "e4m3"),
        # fp32 rows in expert order, as the FC2 step writes them; group-quantised next input
        _norm("norm expert order", 333, 2944, 4, "fp32", "expert", "bf16", True, "channel", "e4m3g"),
    ]


def _spread(rng, lo, hi, step):
    """A multiple of `step` in [lo, hi], spread over the logarithm."""
    v = lo * (hi / lo) ** rng.random()
    return min(hi, max(lo, int(v / step + 0.5) * step))


def draw(rng):
    if rng.random() < 0.5:
        fmt = rng.choice(["bf16", "bf16", "fp8", "block"])
        T = rng.randint(1, 8)
        H = _spread(rng, 256, 7168, 256 if fmt == "block" else 64)
        I = _spread(rng, 128, 2048, 128 if fmt == "block" else 64)
        E = _spread(rng, 4, 256, 1)
        k = rng.randint(1, min(8, E))
        while E * H * I > 64 * 4096 * 1536:  # weights within those of the listed models
            E = max(k, E // 2)
            if E == k:
                I = max(128, I // 256 * 128)
        c = _layer("", T, H, E, k, I, fmt, rng.choice(["router", "router", "bias", "logits", "ids"]),
                   rng.choice(["none", "residual", "sandwich", "gated"]))
    else:
        H = _spread(rng, 256, 8192, 8)
        nxt = rng.choice(["none", "bf16", "bf16", "e4m3", "e4m3g"])
        if nxt != "none":
            H = H // 128 * 128 if nxt == "e4m3g" else H // 16 * 16
        k = rng.choice([1, 2, 4, 6, 8])
        T = _spread(rng, 1, 4096, 1)
        while T * H * (k + 3) > 4096 * 4096 * 11:
            T //= 2
        c = _norm("", T, H, k, rng.choice(["bf16", "fp32"]) if T <= 2048 else "bf16",
                  rng.choice(["pair", "expert"]), rng.choice(["bf16", "fp32"]),
                  rng.random() < 0.7, rng.choice(["none", "channel", "token", "rows"]), nxt)
    del c["name"]
    return c


def _distinct(E, k, T):
    return min(E, T * k, E * (1.0 - (1.0 - k / E) ** T))


def work(case):
    c = case
    T, H = c["T"], c["H"]
    if c["op"] == "layer":
        E, k, I = c["E"], c["k"], c["I"]
        n = _distinct(E, k, T)
        b = n * 3 * H * I * (2 if c["fmt"] == "bf16" else 1)
        if c["fmt"] == "fp8":
            b += n * (2 * I + H) * 4
        if c["fmt"] == "block":
            b += n * 3 * H * I // (128 * 128) * 4
        b += {"router": 4 * H * E, "bias": 4 * H * E + 4 * E, "logits": 4 * T * E,
              "ids": 8 * T * k}[c["routing"]]
        b += 2 * H + 2 * 2 * T * H + 8 * T * k
        if c["tail"] in ("sandwich", "gated"):
            b += 4 * H + 2 * T * H
        if c["tail"] == "gated":
            b += 2 * H
        f = 6.0 * T * k * H * I + (2.0 * T * H * E if c["routing"] in ("router", "bias") else 0)
        return {"bytes": float(b), "flops": f}
    k = c["k"]
    st = 4 if c["stream"] == "fp32" else 2
    b = T * H * k * (2 if c["y"] == "bf16" else 4) + 2 * T * H * st
    b += 4 * T * k if c["order"] == "expert" else 0
    b += 2 * H if c["post"] else 0
    b += {"none": 0, "channel": 2 * H, "token": 4 * T, "rows": 4 * T + 2 * H * _requests(T)}[c["gate"]]
    b += {"none": 0, "bf16": 2 * T * H + 2 * H, "e4m3": T * H + 4 * T + 2 * H,
          "e4m3g": T * H + T * H // 128 * 4 + 2 * H}[c["next"]]
    return {"bytes": float(b), "flops": float(T * H * (k + 12))}


def _requests(T):
    return max(1, min(16, T // 4))


# ----------------------------------------------------------------- inputs --

def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed) * 7919 + 11)


def _randn(g, *shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).add_(mean).to(dtype)


def _fp8_rows(w):
    """Codes and one scale per row: scale = max|row| / 448."""
    s = w.abs().amax(-1).float() / 448
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (w.float() / s[..., None]).clamp_(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s


def _fp8_blocks(w):
    """Codes and one scale per 128 x 128 tile of the last two axes."""
    n, k = w.shape[-2:]
    t = w.view(*w.shape[:-2], n // 128, 128, k // 128, 128)
    s = t.abs().amax((-3, -1)).float() / 448
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (t.float() / s[..., :, None, :, None]).clamp_(-448, 448).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(w.shape), s


def prepare(case, seed):
    return _prepare_layer(case, seed) if case["op"] == "layer" else _prepare_norm(case, seed)


def _prepare_layer(c, seed):
    g = _gen(seed)
    T, H, E, k, I = c["T"], c["H"], c["E"], c["k"], c["I"]
    s = {"case": c, "norm_w": _randn(g, H, std=0.1, mean=1.0)}
    s["w13"] = _randn(g, E, 2 * I, H, std=H ** -0.5)
    s["w2"] = _randn(g, E, H, I, std=I ** -0.5)
    s["w13_scale"] = s["w2_scale"] = None
    if c["fmt"] != "bf16":
        q = _fp8_rows if c["fmt"] == "fp8" else _fp8_blocks
        s["w13"], s["w13_scale"] = q(s["w13"])
        s["w2"], s["w2_scale"] = q(s["w2"])
    for n in ("router_w", "bias", "logits", "ids", "tw"):
        s[n] = None
    # a residual stream: some channels much larger than the rest
    chan = _randn(g, H, std=0.6, dtype=torch.float32).exp_()
    x = (_randn(g, 8 * T, H, dtype=torch.float32) * chan).to(torch.bfloat16)
    if c["routing"] in ("router", "bias"):
        s["router_w"] = _randn(g, H, E, std=2.0 * H ** -0.5, dtype=torch.float32)
        if c["routing"] == "bias":
            p = 1.0 / (1 + torch.arange(E, device=DEV, dtype=torch.float32)) ** 1.2
            p = p[torch.randperm(E, generator=g, device=DEV)].log()
            s["bias"] = (p - p.mean()) / p.std(correction=0).clamp_min(1e-6)
        # tokens whose k + 1 best experts are apart by more than any rounding
        xd = x.double()
        xd = xd / (xd.square().mean(1, keepdim=True) + EPS).sqrt() * s["norm_w"].double()
        z = xd @ s["router_w"].double()
        z = z if s["bias"] is None else z + s["bias"].double()
        top = z.sort(1, descending=True).values[:, :min(k + 1, E)]
        near = ((top[:, :-1] - top[:, 1:]) < 1e-4).any(1)
        x = x[near.to(torch.int32).argsort(dim=0, stable=True)]
    s["x"] = x[:T].contiguous()
    if c["routing"] == "logits":
        s["logits"] = _randn(g, T, E, std=1.5, dtype=torch.float32)
    if c["routing"] == "ids":
        s["ids"] = torch.rand((T, E), generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
        s["tw"] = torch.rand((T, k), generator=g, device=DEV).add_(0.05)
        s["tw"] /= s["tw"].sum(1, keepdim=True)
    for n in ("post_w", "gate", "next_w"):
        s[n] = None
    if c["tail"] in ("sandwich", "gated"):
        s["post_w"] = _randn(g, H, std=0.1, mean=0.5)
        s["next_w"] = _randn(g, H, std=0.1, mean=1.0)
    if c["tail"] == "gated":
        s["gate"] = _randn(g, H, std=0.5, mean=0.5)
    s["scale"] = 0.7 if c["tail"] == "gated" else 1.0
    return s


def _prepare_norm(c, seed):
    g = _gen(seed)
    T, H, k = c["T"], c["H"], c["k"]
    yt = torch.bfloat16 if c["y"] == "bf16" else torch.float32
    st = torch.bfloat16 if c["stream"] == "bf16" else torch.float32
    chan = _randn(g, H, std=0.6, dtype=torch.float32).exp_()
    s = {"case": c, "y": _randn(g, T * k, H, std=0.3, dtype=yt),
         "residual": (_randn(g, T, H, dtype=torch.float32) * chan).to(st)}
    s["row_of_pair"] = None
    if c["order"] == "expert":
        s["row_of_pair"] = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32)
    s["post_w"] = _randn(g, H, std=0.1, mean=0.5) if c["post"] else None
    s["gate"] = s["gate_row"] = None
    if c["gate"] == "channel":
        s["gate"] = _randn(g, H, std=0.5, mean=0.5)
    if c["gate"] == "token":
        s["gate"] = torch.sigmoid(_randn(g, T, 1, dtype=torch.float32))
    if c["gate"] == "rows":
        n = _requests(T)
        s["gate"] = _randn(g, n, H, std=0.5, mean=0.5)
        s["gate_row"] = torch.randint(0, n, (T,), generator=g, device=DEV).sort().values.to(torch.int32)
    s["scale"] = 0.7 if c["gate"] != "none" else 1.0
    s["next_w"] = _randn(g, H, std=0.1, mean=1.0) if c["next"] != "none" else None
    return s


# -------------------------------------------------------------- plain form --

def _rms(v, w):
    return v / (v.square().mean(-1, keepdim=True) + EPS).sqrt() * w.float()


def _dequant(q, scale, fmt):
    """Gathered weights [.., N, K] and their gathered scales in 32 bits."""
    if fmt == "bf16":
        return q.float()
    w = q.view(torch.float8_e4m3fn).float()
    if fmt == "fp8":
        return w * scale[..., None]
    return w * scale.repeat_interleave(128, -2).repeat_interleave(128, -1)


def _gated_ffn(v, ids, tw, s):
    """sum_j tw_j (silu(v Wg^T) * (v Wu^T)) W2^T over the token's experts, weights gathered."""
    c = s["case"]
    I = c["I"]
    ix = ids.long()
    w13 = _dequant(s["w13"][ix], None if s["w13_scale"] is None else s["w13_scale"][ix], c["fmt"])
    u = torch.matmul(w13, v[:, None, :, None]).squeeze(-1)
    del w13
    a = u[..., :I] / (1 + torch.exp(-u[..., :I])) * u[..., I:]
    w2 = _dequant(s["w2"][ix], None if s["w2_scale"] is None else s["w2_scale"][ix], c["fmt"])
    y = torch.matmul(w2, a[..., None]).squeeze(-1)
    return (y * tw[..., None]).sum(1)


def _tail(f, s, residual, gate, st):
    """h and x_hat (or None) in 32 bits."""
    if s["post_w"] is not None:
        f = _rms(f, s["post_w"])
    if gate is not None:
        f = f * gate.float()
    h = f * s["scale"]
    if residual is not None:
        h = h + residual.float()
    return h, None if s["next_w"] is None else _rms(h, s["next_w"])


def _e4m3(v, group):
    """E4M3 values of v / s and s = max|v| / 448 per row (group 0) or per `group` columns."""
    t = v.view(v.shape[0], -1, group) if group else v[:, None, :]
    sc = t.abs().amax(-1) / 448
    sc = torch.where(sc > 0, sc, torch.ones_like(sc))
    q = (t / sc[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(v.shape)
    return q, sc if group else sc[:, 0]


def _plain_layer(s):
    c = s["case"]
    k = c["k"]
    v = _rms(s["x"].float(), s["norm_w"])
    ids, tw = s["ids"], s["tw"]
    if ids is None:
        # the selection compares values that may be near each other: 64 bits
        z = s["logits"].double() if s["logits"] is not None else \
            (_rms(s["x"].double(), s["norm_w"].double()) @ s["router_w"].double())
        if s["bias"] is not None:
            z = z + s["bias"].double()
        z, ids = z.sort(dim=1, descending=True, stable=True)
        e = torch.exp(z[:, :k] - z[:, :1])
        ids, tw = ids[:, :k].to(torch.int32), (e / e.sum(1, keepdim=True)).float()
    f = _gated_ffn(v, ids, tw, s)
    if c["tail"] == "none":
        return {"out": f.to(torch.bfloat16), "ids": ids, "tw": tw}
    h, xh = _tail(f, s, s["x"], s["gate"], torch.bfloat16)
    r = {"out": h.to(torch.bfloat16), "ids": ids, "tw": tw}
    if xh is not None:
        r["xhat"] = xh.to(torch.bfloat16)
    return r


def _plain_norm(s):
    c = s["case"]
    T, H, k = c["T"], c["H"], c["k"]
    y = s["y"] if s["row_of_pair"] is None else s["y"][s["row_of_pair"].long()]
    f = y.view(T, k, H).float().sum(1)
    gate = s["gate"] if s["gate_row"] is None else s["gate"][s["gate_row"].long()]
    h, xh = _tail(f, s, s["residual"], gate, None)
    r = {"out": h.to(s["residual"].dtype)}
    if c["next"] == "bf16":
        r["xhat"] = xh.to(torch.bfloat16)
    elif c["next"] != "none":
        r["xq"], r["xscale"] = _e4m3(xh, 128 if c["next"] == "e4m3g" else 0)
    return r


# ------------------------------------------------------------- the library --

def _plan_layer(s):
    """Buffers and descriptors a decoding program makes once."""
    import moe_expert_ffn_rms_gb300 as M
    c = s["case"]
    T, H, E, k, I = c["T"], c["H"], c["E"], c["k"], c["I"]
    shape = M.make_shape(T, H, E, I, k, EPS, fp8={"bf16": False, "fp8": True, "block": "block"}[c["fmt"]])
    p = {"M": M, "shape": shape,
         "ws": M.alloc_workspace(M.moe_layer_workspace_size(shape), DEV),
         "out": torch.empty((T, H), dtype=torch.bfloat16, device=DEV),
         "ids": s["ids"], "tw": s["tw"], "xhat": None, "tail": None, "ids_out": None, "tw_out": None}
    if s["ids"] is None:
        p["ids_out"] = p["ids"] = torch.empty((T, k), dtype=torch.int32, device=DEV)
        p["tw_out"] = p["tw"] = torch.empty((T, k), dtype=torch.float32, device=DEV)
    if s["next_w"] is not None:
        p["xhat"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    if c["tail"] != "none":
        p["tail"] = M.make_block_tail(residual=s["x"], post_w=s["post_w"], post_eps=EPS, gate=s["gate"],
                                      scale=s["scale"], next_w=s["next_w"], next_eps=EPS, xhat=p["xhat"])
    return p


def _own_layer(s):
    if "plan" not in s:
        s["plan"] = _plan_layer(s)
    p = s["plan"]
    p["M"].moe_layer_forward(p["shape"], s["x"], s["norm_w"], s["w13"], s["w2"], p["out"], p["ws"],
                             router_w=s["router_w"], router_logits=s["logits"], router_bias=s["bias"],
                             topk_ids=s["ids"], topk_w=s["tw"], w13_scale=s["w13_scale"],
                             w2_scale=s["w2_scale"], tail=p["tail"], topk_ids_out=p["ids_out"],
                             topk_w_out=p["tw_out"])
    r = {"out": p["out"], "ids": p["ids"], "tw": p["tw"]}
    if p["xhat"] is not None:
        r["xhat"] = p["xhat"]
    return r


def _plan_norm(s):
    import moe_expert_ffn_rms_gb300 as M
    c = s["case"]
    T, H = c["T"], c["H"]
    p = {"M": M, "out": torch.empty_like(s["residual"])}
    if c["next"] == "bf16":
        p["xhat"] = torch.empty((T, H), dtype=torch.bfloat16, device=DEV)
    elif c["next"] != "none":
        p["xq"] = torch.empty((T, H), dtype=torch.float8_e4m3fn, device=DEV)
        p["xscale"] = torch.empty((T, H // 128) if c["next"] == "e4m3g" else (T,), device=DEV)
    p["tail"] = M.make_block_tail(residual=s["residual"], post_w=s["post_w"], post_eps=EPS, gate=s["gate"],
                                  gate_row=s["gate_row"], scale=s["scale"], next_w=s["next_w"],
                                  next_eps=EPS, xhat=p.get("xhat"), xq=p.get("xq"),
                                  xscale=p.get("xscale"))
    return p


def _own_norm(s):
    if "plan" not in s:
        s["plan"] = _plan_norm(s)
    p, c = s["plan"], s["case"]
    p["M"].moe_combine_norm(s["y"], p["out"], c["T"], c["k"], p["tail"], row_of_pair=s["row_of_pair"],
                            pair_order=c["order"] == "pair")
    return {n: p[n] for n in ("out", "xhat", "xq", "xscale") if n in p}


def run(state):
    if own:
        return _own_layer(state) if state["case"]["op"] == "layer" else _own_norm(state)
    return _plain_layer(state) if state["case"]["op"] == "layer" else _plain_norm(state)


# ------------------------------------------------------------- definition --

def _norm64(row, w):
    r = torch.sqrt((row * row).sum() / row.numel() + EPS)
    return row / r * w.double()


def _weights64(s, name, e):
    """One expert's matrix in 64 bits."""
    q, sc, fmt = s[name][e], s[name + "_scale"], s["case"]["fmt"]
    if fmt == "bf16":
        return q.double()
    w = q.view(torch.float8_e4m3fn).double()
    n, k = w.shape
    if fmt == "fp8":
        return w * sc[e].double().view(n, 1)
    return (w.view(n // 128, 128, k // 128, 128) * sc[e].double().view(n // 128, 1, k // 128, 1)).view(n, k)


def _tail64(f, s, t, residual, gate):
    if s["post_w"] is not None:
        f = _norm64(f, s["post_w"])
    if gate is not None:
        f = gate.double() * f
    h = s["scale"] * f + residual[t].double()
    return h, None if s["next_w"] is None else _norm64(h, s["next_w"])


def exact(case, seed):
    c, s = case, prepare(case, seed)
    T, H, k = c["T"], c["H"], c["k"]
    if c["op"] == "layer":
        I = c["I"]
        f = torch.zeros((T, H), dtype=torch.float64, device=DEV)
        v = [_norm64(s["x"][t].double(), s["norm_w"]) for t in range(T)]
        picks = {}
        ids_all, tw_all = [], []
        for t in range(T):
            if s["ids"] is not None:
                ids, tw = s["ids"][t].tolist(), s["tw"][t].double()
            else:
                z = s["logits"][t].double() if s["logits"] is not None else v[t] @ s["router_w"].double()
                z = (z if s["bias"] is None else z + s["bias"].double()).cpu()
                ids = sorted(range(c["E"]), key=lambda e: (-float(z[e]), e))[:k]
                tw = torch.softmax(z[ids], 0).to(DEV)
            ids_all.append(ids)
            tw_all.append(tw)
            for j, e in enumerate(ids):
                picks.setdefault(e, []).append((t, tw[j]))
        for e, users in picks.items():
            w13, w2 = _weights64(s, "w13", e), _weights64(s, "w2", e)
            for t, w in users:
                u = w13 @ v[t]
                f[t] += w * (w2 @ (u[:I] * torch.sigmoid(u[:I]) * u[I:]))
        r = {"ids": torch.tensor(ids_all, dtype=torch.int32), "tw": torch.stack(tw_all)}
        if c["tail"] == "none":
            r["out"] = f
            return r
        rows = [_tail64(f[t], s, t, s["x"], s["gate"]) for t in range(T)]
        r["out"] = torch.stack([a for a, _ in rows])
        if s["next_w"] is not None:
            r["xhat"] = torch.stack([b for _, b in rows])
        return r
    hs, xs = [], []
    at = torch.arange(T * k).view(T, k) if s["row_of_pair"] is None else s["row_of_pair"].cpu().view(T, k)
    gr = None if s["gate_row"] is None else s["gate_row"].tolist()
    for t in range(T):
        f = s["y"][at[t].tolist()].double().sum(0)
        g = s["gate"]
        if c["gate"] == "token":
            g = g[t]
        elif c["gate"] == "rows":
            g = g[gr[t]]
        h, x = _tail64(f, s, t, s["residual"], g)
        hs.append(h)
        xs.append(x)
    r = {"out": torch.stack(hs)}
    if c["next"] == "bf16":
        r["xhat"] = torch.stack(xs)
    elif c["next"] != "none":
        x = torch.stack(xs)
        t = x.view(T, -1, 128 if c["next"] == "e4m3g" else H)
        sc = t.abs().amax(-1) / 448
        # the quantised values have no value of their own in 64 bits but the nearest code's
        r["xscale"] = sc if c["next"] == "e4m3g" else sc[:, 0]
        r["xq"] = None
    return r
