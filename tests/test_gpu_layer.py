"""moe_layer_forward on the GPU against the block's formulas in 64 bits.

The tolerances count roundings (u = 2^-24, half a step of fp32):
  products   activations enter as hi + lo bf16 terms: hi is half a bf16 step
             (2^-8) off, lo half a step of that (2^-16 of the value); the fp16
             terms beside E4M3 weights are nearer.  A product of two 16-bit terms
             is exact in fp32
  sums       one MMA adds 16 products to the accumulator; its internal sums are
             taken to be good to 2^-22 of the magnitudes; each of 8 warps adds
             at most 2 K / (16 * 8) MMAs one after the other, then the 8 warps
             are added
  r          28 u (as in test_gpu_block_tail)
  silu(g) u  |silu'| <= 1.1; exp, divide and products within 8 u
  logits     a warp adds at most 8 ceil(H / 2048) rows (a chunk is at most
             ceil(H / 2048) units of 128 rows over 16 warps), then the 16 warps
             and the 16 chunks are added
  weights    the relative error of exp(z - z_max) is twice the logits' error
and the tail adds what test_gpu_block_tail counts."""
import pytest
import torch

from tests.test_gpu_block_tail import (RNORM, U, check_outputs, codes_by_definition, exact_weights, randn,
                                       tail_reference)

pytestmark = pytest.mark.gpu
DEV = "cuda"
EPS = 1e-6


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_ffn_rms_gb300 as M
    return M


def quantize(w, fmt):
    """Codes and scales (bf16 weights pass through)."""
    if fmt == "bf16":
        return w, None
    if fmt == "fp8":
        s = (w.abs().amax(-1).float() / 448).clamp_min(1e-12)
        q = w.float() / s[..., None]
    else:
        n, k = w.shape[-2:]
        t = w.view(*w.shape[:-2], n // 128, 128, k // 128, 128)
        s = (t.abs().amax((-3, -1)).float() / 448).clamp_min(1e-12)
        q = (t.float() / s[..., :, None, :, None]).view(w.shape)
    return q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8), s.contiguous()


def weights64(d, name, e):
    q, s = d[name][e], d[name + "_scale"]
    if s is None:
        return q.double()
    w = q.view(torch.float8_e4m3fn).double()
    if d["fmt"] == "fp8":
        return w * s[e].double()[:, None]
    return w * s[e].double().repeat_interleave(128, 0).repeat_interleave(128, 1)


def make(T, H, E, k, I, fmt="bf16", routing="router", tail="none", seed=0, gate=None, nxt="bf16",
         res=torch.bfloat16):
    g = torch.Generator(device=DEV).manual_seed(seed)
    d = dict(T=T, H=H, E=E, k=k, I=I, fmt=fmt, tail=tail, norm_w=randn(g, H, std=0.2, mean=1.0))
    d["w13"], d["w13_scale"] = quantize(randn(g, E, 2 * I, H, std=H ** -0.5), fmt)
    d["w2"], d["w2_scale"] = quantize(randn(g, E, H, I, std=I ** -0.5), fmt)
    x = randn(g, 16 * T + 16, H, std=1.5)
    d["router_w"] = d["logits"] = d["bias"] = d["ids"] = d["tw"] = None
    if routing in ("router", "bias"):
        d["router_w"] = randn(g, H, E, std=2.0 * H ** -0.5, dtype=torch.float32)
        d["bias"] = randn(g, E, dtype=torch.float32) if routing == "bias" else None
        # tokens whose choice and order of experts no rounding can change
        z = logits64(d, x)
        top = z.sort(dim=1, descending=True).values[:, :min(k + 1, E)]
        far = ~((top[:, :-1] - top[:, 1:]) < 1e-3).any(1)
        assert int(far.sum()) >= T
        x = x[far]
    elif routing == "logits":
        d["logits"] = randn(g, T, E, std=1.5, dtype=torch.float32)
    else:
        d["ids"] = torch.rand((T, E), generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
        d["tw"] = torch.rand((T, k), generator=g, device=DEV) + 0.05
    d["x"] = x[:T].contiguous()
    # the tail's entries, as tests/test_gpu_block_tail.py names them
    d.update(residual=None, post_w=None, gate=None, gate_row=None, next_w=None, scale=1.0, post_eps=EPS,
             next_eps=1e-5, next="none")
    if tail != "none":
        d["residual"] = d["x"] if res == torch.bfloat16 else randn(g, T, H, dtype=res)
        if tail == "full":
            d.update(post_w=randn(g, H, std=0.2, mean=0.5), next_w=randn(g, H, std=0.2, mean=1.0), next=nxt,
                     scale=0.7)
            if gate == "channel":
                d["gate"] = randn(g, H)
            elif gate == "token":
                d["gate"] = randn(g, T, 1, dtype=torch.float32)
            elif gate == "rows":
                d["gate"] = randn(g, 3, H)
                d["gate_row"] = torch.randint(0, 3, (T,), generator=g, device=DEV, dtype=torch.int32)
    return d


def xhat64(d, x):
    v = x.double()
    return v / (v.square().mean(1, keepdim=True) + EPS).sqrt() * d["norm_w"].double()


def logits64(d, x):
    z = xhat64(d, x) @ d["router_w"].double()
    return z if d["bias"] is None else z + d["bias"].double()


def plan(M, d):
    T, H, E, k, I = d["T"], d["H"], d["E"], d["k"], d["I"]
    shape = M.make_shape(T, H, E, I, k, EPS, fp8={"bf16": False, "fp8": True, "block": "block"}[d["fmt"]])
    ws = M.alloc_workspace(M.moe_layer_workspace_size(shape), DEV)
    ws.fill_(255)  # nothing in it is assumed
    return shape, ws


def call(M, d, p=None, stream=None, out=None):
    T, H, k = d["T"], d["H"], d["k"]
    shape, ws = p or plan(M, d)
    nan = float("nan")
    dt = d["residual"].dtype if d["residual"] is not None else torch.bfloat16
    o = {"out": torch.full((T, H), nan, device=DEV, dtype=dt) if out is None else out}
    tail = None
    if d["tail"] != "none":
        if d["next"] in ("bf16", "both"):
            o["xhat"] = torch.full((T, H), nan, device=DEV, dtype=torch.bfloat16)
        if d["next"] in ("e4m3", "both"):
            o["xq"] = torch.full((T, H), 0x7f, device=DEV, dtype=torch.uint8)
            o["xscale"] = torch.full((T,), nan, device=DEV)
        if d["next"] == "e4m3g":
            o["xq"] = torch.full((T, H), 0x7f, device=DEV, dtype=torch.uint8)
            o["xscale"] = torch.full((T, H // 128), nan, device=DEV)
        tail = M.make_block_tail(residual=d["residual"], post_w=d["post_w"], post_eps=d["post_eps"],
                                 gate=d["gate"], gate_row=d["gate_row"], scale=d["scale"],
                                 next_w=d["next_w"], next_eps=d["next_eps"], xhat=o.get("xhat"),
                                 xq=o.get("xq"), xscale=o.get("xscale"))
    ids = torch.full((T, k), -7, dtype=torch.int32, device=DEV)
    tw = torch.full((T, k), nan, dtype=torch.float32, device=DEV)
    M.moe_layer_forward(shape, d["x"], d["norm_w"], d["w13"], d["w2"], o["out"], ws,
                        router_w=d["router_w"], router_logits=d["logits"], router_bias=d["bias"],
                        topk_ids=d["ids"], topk_w=d["tw"], w13_scale=d["w13_scale"],
                        w2_scale=d["w2_scale"], tail=tail, topk_ids_out=ids, topk_w_out=tw, stream=stream)
    return o, ids, tw


def routing64(d):
    """ids, weights and the relative error fp32 logits leave in the weights."""
    if d["ids"] is not None:
        return d["ids"].tolist(), d["tw"].double(), torch.zeros((d["T"], 1), device=DEV, dtype=torch.float64)
    k = d["k"]
    if d["logits"] is not None:
        z, dz = d["logits"].double(), 0.0 * d["logits"].double()
    else:
        z = logits64(d, d["x"])
        mag = xhat64(d, d["x"]).abs() @ d["router_w"].double().abs()
        dz = mag * (8 * -(-d["H"] // 2048) + 16 + 16 + RNORM + 4) * U + 2 * U * z.abs()
    zs, ids = z.sort(dim=1, descending=True, stable=True)
    w = torch.softmax(zs[:, :k], 1)
    return ids[:, :k].tolist(), w, 2 * dz.amax(1, keepdim=True) + 2 * U * zs[:, :k].abs().amax(1, keepdim=True) + 16 * U


def block64(d, skip=()):
    """f and the absolute error its arithmetic may leave; ids and weights."""
    T, H, E, k, I = d["T"], d["H"], d["E"], d["k"], d["I"]
    ids, w, dw = routing64(d)
    v = xhat64(d, d["x"])
    split = 2.0 ** -16
    acc1 = (H / 64 + 16) * 2.0 ** -22
    f = torch.zeros((T, H), dtype=torch.float64, device=DEV)
    df = torch.zeros_like(f)
    users = {}
    for t in range(T):
        for j, e in enumerate(ids[t]):
            if 0 <= e < E and t not in skip:
                users.setdefault(e, []).append((t, j))
    acc2 = (max(1, len(users)) * I / 64 + 16) * 2.0 ** -22
    for e, us in users.items():
        w13, w2 = weights64(d, "w13", e), weights64(d, "w2", e)
        for t, j in us:
            h = w13 @ v[t]
            dh = (w13.abs() @ v[t].abs()) * (split + acc1 + (RNORM + 6) * U)
            ga, up, dg, du = h[:I], h[I:], dh[:I], dh[I:]
            s = ga * torch.sigmoid(ga)
            a = s * up
            da = 1.1 * dg * (up.abs() + du) + s.abs() * du + 8 * U * a.abs()
            f[t] += w[t, j] * (w2 @ a)
            df[t] += w[t, j].abs() * (w2.abs() @ (da + a.abs() * (split + acc2 + 8 * U)))
            df[t] += w[t, j].abs() * dw[t].max() * (w2 @ a).abs()
    return f, df, ids, w, dw


def check(d, res, skip=()):
    o, ids, tw = res
    f, df, ids64, w, dw = block64(d, skip)
    rows = [t for t in range(d["T"]) if t not in skip]
    if d["ids"] is None:
        assert [ids.tolist()[t] for t in rows] == [ids64[t] for t in rows]
        assert ((tw.double() - w).abs() <= (dw + 4 * U) * w)[rows].all()
    h, dh, x, dx = tail_reference(d, f, df) if d["tail"] != "none" else (f, df, None, None)
    if not skip:
        check_outputs(d, o, h, dh, x, dx)
    else:
        half = torch.finfo(o["out"].dtype).eps / 2
        assert ((o["out"].double() - h).abs() <= dh + half * (h.abs() + dh))[rows].all()


SHAPES = [  # T, H, E, k, I
    (1, 64, 1, 1, 64), (1, 256, 8, 2, 512), (4, 256, 8, 2, 512), (8, 192, 3, 3, 192), (3, 320, 5, 4, 128),
    (5, 1024, 16, 8, 192), (8, 512, 256, 8, 128), (2, 4096, 8, 2, 256), (7, 7168, 4, 1, 64),
    (6, 128, 64, 8, 1536), (8, 2048, 33, 5, 320), (1, 16384, 2, 2, 64), (8, 448, 200, 6, 448)]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_shapes(M, shape, fmt):
    d = make(*shape, fmt=fmt, tail="none", seed=sum(shape))
    check(d, call(M, d))
    assert M.device_status() == 0


@pytest.mark.parametrize("shape", [(1, 256, 4, 2, 128), (8, 512, 16, 4, 384), (3, 1280, 8, 8, 640),
                                   (2, 8192, 3, 2, 128)], ids=lambda s: "x".join(map(str, s)))
def test_block_scales(M, shape):
    d = make(*shape, fmt="block", tail="residual", seed=3)
    check(d, call(M, d))


@pytest.mark.parametrize("routing", ["router", "bias", "logits", "ids"])
@pytest.mark.parametrize("tail", ["none", "residual", "full"])
@pytest.mark.parametrize("T", [1, 2, 5, 8])
def test_routing_and_tails(M, routing, tail, T):
    d = make(T, 384, 12, 3, 192, routing=routing, tail=tail, seed=T)
    check(d, call(M, d))


@pytest.mark.parametrize("nxt", ["bf16", "e4m3", "e4m3g", "both"])
@pytest.mark.parametrize("gate", [None, "channel", "token", "rows"])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_tail_outputs(M, nxt, gate, res):
    for T, H in ((3, 640), (8, 1280)):
        d = make(T, H, 6, 2, 128, tail="full", gate=gate, nxt=nxt, res=res, seed=T)
        check(d, call(M, d))


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("T,H", [(2, 16384), (8, 12352), (3, 12288), (5, 64)])
def test_tail_of_long_and_short_rows(M, fmt, T, H):
    """Rows that the tail keeps in shared memory with all their inputs, and longer ones."""
    for gate, nxt in (("channel", "both"), ("rows", "bf16")):
        d = make(T, H, 4, 2, 64, fmt=fmt, tail="full", gate=gate, nxt=nxt, res=torch.float32, seed=H)
        check(d, call(M, d))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "block"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8])
def test_every_batch(M, fmt, T):
    """Each kernel instance (tokens per MMA column set, routing width), rows that do not fill the
    CTAs' slices evenly, experts from one to many."""
    for H, E, k, I in ((1280, 40, 6, 640), (256, 2, 1, 128), (2304, 16, 4, 256)):
        d = make(T, H, E, k, I, fmt=fmt, tail="full", seed=T)
        check(d, call(M, d))
    assert M.device_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_magnitudes(M, fmt):
    """Columns and tokens of very different size share MMAs; tiny and huge weights of the norm."""
    d = make(4, 512, 6, 2, 256, fmt=fmt, routing="ids", seed=12)
    d["x"] *= torch.logspace(-6, 6, 4, device=DEV)[:, None].to(torch.bfloat16)
    d["norm_w"] *= torch.logspace(-3, 3, 512, device=DEV).to(torch.bfloat16)
    d["tw"] *= torch.logspace(-4, 0, 4, device=DEV)[:, None]
    check(d, call(M, d))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "block"])
@pytest.mark.parametrize("T", [1, 8])
def test_model_sized(M, fmt, T):
    d = make(T, 4096, 24, 8, 1536, fmt=fmt, tail="full", seed=9)
    check(d, call(M, d))
    assert M.device_status() == 0


def test_all_tokens_on_one_expert_and_none_in_common(M):
    d = make(8, 512, 64, 8, 256, routing="ids", seed=1)
    d["ids"][:] = torch.arange(8, device=DEV, dtype=torch.int32) + 5
    check(d, call(M, d))
    d["ids"][:] = torch.arange(64, device=DEV, dtype=torch.int32).view(8, 8)
    check(d, call(M, d))


def test_ids_out_of_range_given_twice_and_empty(M):
    M.device_status(clear=True)
    d = make(4, 256, 8, 2, 128, routing="ids", tail="residual", seed=2)
    d["ids"][1, 0] = 8
    d["ids"][2, 1] = -1
    d["ids"][3] = torch.tensor([2 ** 31 - 1, -2 ** 31], device=DEV)  # no expert at all: f = 0
    o = call(M, d)
    check(d, o)
    assert torch.equal(o[0]["out"][3], d["x"][3])
    assert M.device_status(clear=True) == 1
    d["ids"].fill_(-1)  # nothing to do for anyone
    o = call(M, d)
    assert torch.equal(o[0]["out"], d["x"]) and M.device_status(clear=True) == 1
    d = make(3, 256, 8, 3, 128, routing="ids", seed=2)
    d["ids"][1] = 4  # the same expert three times: its weights add up
    check(d, call(M, d))
    assert M.device_status(clear=True) == 0


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_non_finite_values_stay_in_their_token(M, fmt):
    d = make(4, 256, 12, 2, 128, fmt=fmt, routing="ids", tail="full", nxt="both", seed=4)
    d["ids"].copy_(torch.tensor([[0, 1], [2, 3], [0, 4], [5, 1]], dtype=torch.int32))
    d["x"][1, 3] = float("nan")
    o = call(M, d)
    assert torch.isnan(o[0]["out"][1]).all()
    check(d, o, skip=(1,))
    d["x"][1, 3] = float("inf")
    o = call(M, d)
    assert torch.isnan(o[0]["out"][1]).any() and not torch.isfinite(o[0]["out"][1]).all()
    check(d, o, skip=(1,))
    # weights that are not finite, in an expert of token 0 and of an expert nobody uses
    d = make(4, 256, 12, 2, 128, fmt=fmt, routing="ids", seed=4)
    d["ids"].copy_(torch.tensor([[0, 1], [2, 3], [6, 4], [5, 1]], dtype=torch.int32))
    for e in (0, 9):
        d["w13"][e, 5] = float("inf") if fmt == "bf16" else 0x7f  # (E4M3 has NaN only)
        d["w2"][e, 7] = float("nan") if fmt == "bf16" else 0xff
    o = call(M, d)
    assert torch.isnan(o[0]["out"][0, 7])
    check(d, o, skip=(0,))
    # NaN and infinite logits rank as moe_route_topk ranks them
    d = make(3, 256, 8, 2, 128, routing="logits", seed=5)
    d["logits"][0, 3] = float("nan")
    d["logits"][1] = float("-inf")
    d["logits"][2, 6] = float("-inf")
    o = call(M, d)
    ids, tw = (torch.empty((3, 2), dtype=t, device=DEV) for t in (torch.int32, torch.float32))
    M.moe_route_topk(3, 256, 8, 2, ids, tw, logits_in=d["logits"])
    assert torch.equal(o[1], ids) and torch.equal(o[2], tw)
    assert (o[0]["out"][1] == 0).all() and torch.isfinite(o[0]["out"].float()).all()


def test_ties_take_the_lower_expert(M):
    d = make(2, 256, 40, 4, 128, routing="logits", seed=6)
    d["logits"].zero_()
    d["logits"][1, 35] = d["logits"][1, 33] = 1.0
    _, ids, tw = call(M, d)
    assert ids.tolist() == [[0, 1, 2, 3], [33, 35, 0, 1]]
    assert (tw[0] == 0.25).all()


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "block"])
def test_repeats_bit_for_bit(M, fmt):
    d = make(8, 1024, 32, 8, 512, fmt=fmt, tail="full", nxt="both", seed=7)
    p = plan(M, d)
    first = call(M, d, p)
    for _ in range(20):
        o = call(M, d, p)
        for n in first[0]:
            assert torch.equal(o[0][n], first[0][n]), n


def test_rows_behind_the_last_and_inputs_stay(M):
    d = make(3, 256, 8, 2, 128, tail="residual", seed=8)
    x = d["x"].clone()
    big = torch.full((8, 256), 7.0, device=DEV, dtype=torch.bfloat16)
    call(M, d, out=big[:3])
    assert (big[3:] == 7.0).all() and torch.equal(d["x"], x)
    want = big[:3].clone()
    d2 = dict(d, residual=d["x"].clone())
    d2["residual"] = d2["x"] = d["x"].clone()
    o = call(M, d2, out=d2["x"])  # the residual stream updated in place
    assert torch.equal(o[0]["out"], want)


def test_no_tokens(M):
    n = M.lib.moe_launch_count()
    s = M.make_shape(0, 256, 8, 128, 2)
    e = torch.empty((0, 256), dtype=torch.bfloat16, device=DEV)
    w = torch.ones(256, dtype=torch.bfloat16, device=DEV)
    M.moe_layer_forward(s, e, w, torch.empty((8, 256, 256), dtype=torch.bfloat16, device=DEV),
                        torch.empty((8, 256, 128), dtype=torch.bfloat16, device=DEV), e,
                        M.alloc_workspace(256, DEV))
    assert M.lib.moe_launch_count() == n


def test_launches(M):
    d = make(4, 256, 8, 2, 512, tail="full", seed=1)
    p = plan(M, d)
    n = M.lib.moe_launch_count()
    call(M, d, p)
    assert M.lib.moe_launch_count() == n + 2


@pytest.mark.parametrize("n,fmt", [(2, "bf16"), (3, "fp8"), (8, "bf16")])
def test_streams_at_once(M, n, fmt):
    ds = [make(8 - i % 3, 1024, 16, 4, 512, fmt=fmt, tail="full", nxt="both", seed=30 + i) for i in range(n)]
    ps = [plan(M, d) for d in ds]
    want = [call(M, d, p) for d, p in zip(ds, ps)]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in ds]
    for _ in range(20):
        got = []
        for d, p, s in zip(ds, ps, ss):
            with torch.cuda.stream(s):
                got.append(call(M, d, p))
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            for n in w[0]:
                assert torch.equal(w[0][n], o[0][n]), n
    assert M.device_status() == 0


def test_without_dependent_launch(M, monkeypatch):
    # (the switch is read once per process: a process of its own)
    import os
    import subprocess
    import sys
    code = ("import tests.test_gpu_layer as t, moe_expert_ffn_rms_gb300 as M\n"
            "d = t.make(4, 512, 16, 4, 256, tail='full', nxt='both', seed=1)\n"
            "t.check(d, t.call(M, d))\nprint('fine')")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, env=dict(os.environ, MOE_PDL="0"),
                       capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
def test_graphs_sharing_a_workspace(M, fmt):
    d = make(2, 512, 16, 4, 256, fmt=fmt, tail="full", seed=40)
    d2 = dict(d, x=d["x"].flip(0).contiguous())
    d2["residual"] = d2["x"]
    p = plan(M, d)
    want, want2 = call(M, d, p), call(M, d2, p)
    torch.cuda.synchronize()
    graphs, outs = [], []
    for dd in (d, d2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(M, dd, p))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for w, o in zip((want, want2), outs):
        for n in w[0]:
            assert torch.equal(w[0][n], o[0][n]), n


def test_near_the_forward(M):
    """The separate-launch forward rounds x_hat and the intermediate to bf16: equal to within that."""
    import workloads
    inp = workloads.make_inputs("c1_tiny", DEV)
    T, H, E, k, I = inp["T"], inp["H"], inp["E"], inp["k"], inp["I"]
    shape = M.make_shape(T, H, E, I, k, inp["eps"])
    ref = torch.empty_like(inp["x"])
    M.moe_ffn_forward(shape, inp["x"], inp["norm_w"], inp["w13"], inp["w2"], ref,
                      M.alloc_workspace(M.moe_ffn_workspace_size(shape), DEV), router_w=inp["router_w"])
    out = torch.empty_like(ref)
    M.moe_layer_forward(shape, inp["x"], inp["norm_w"], inp["w13"], inp["w2"], out,
                        M.alloc_workspace(M.moe_layer_workspace_size(shape), DEV), router_w=inp["router_w"])
    rms = ref.float().square().mean(1, keepdim=True).sqrt()
    assert ((out.float() - ref.float()).abs() <= 2e-2 * torch.maximum(ref.float().abs(), rms)).all()


def test_two_layers_in_a_row(M):
    """As a decoding program uses it: the first layer's tail writes the second one's residual stream,
    and an attention-like block between them goes through moe_combine_norm."""
    a = make(3, 512, 8, 2, 256, tail="residual", seed=50)
    b = make(3, 512, 8, 2, 256, tail="full", seed=51)
    oa = call(M, a)
    mid = randn(torch.Generator(device=DEV).manual_seed(5), 3, 512)
    stream = torch.empty_like(oa[0]["out"])
    t = M.make_block_tail(residual=oa[0]["out"])
    M.moe_combine_norm(mid, stream, 3, 1, t)
    b["x"] = b["residual"] = stream
    ob = call(M, b)
    torch.cuda.synchronize()
    check(a, oa)
    assert torch.equal(stream, (oa[0]["out"].float() + mid.float()).to(torch.bfloat16))
    check(b, ob)


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "block"])
def test_calls_after_one_another_on_one_workspace(M, fmt):
    """Each call's input is the output of the one before it, all in one workspace and one pair of
    buffers: eagerly with a synchronisation after each call, without any, and in a graph."""
    d = make(3, 768, 16, 4, 256, fmt=fmt, tail="full", nxt="bf16", seed=60)
    p = plan(M, d)
    n = 24

    def run(sync):
        a, b, outs = d["x"].clone(), torch.empty_like(d["x"]), []
        for _ in range(n):
            call(M, dict(d, x=a, residual=a), p, out=b)
            if sync:
                torch.cuda.synchronize()
            outs.append(b.clone())
            a, b = b, a
        return outs

    want = run(True)
    got = run(False)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        replayed = run(False)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for w, o, r in zip(want, got, replayed):
        assert torch.equal(w, o) and torch.equal(w, r)
    assert M.device_status() == 0


def test_output_over_the_input(M):
    """out = x (= residual): the block's update in place; and without a tail."""
    for tail in ("full", "none"):
        d = make(5, 512, 8, 2, 256, tail=tail, seed=61)
        want = call(M, d)[0]["out"]
        x = d["x"].clone()
        e = dict(d, x=x, residual=x if tail == "full" else None)
        call(M, e, out=x)
        assert torch.equal(x, want)


@pytest.mark.parametrize("T,H,E", [(8, 16384, 256), (8, 14336, 96), (4, 16384, 40)])
def test_router_of_the_longest_rows(M, T, H, E):
    d = make(T, H, E, 4, 64, tail="none", seed=62)
    check(d, call(M, d))


def test_host_threads_at_once(M):
    """Layers of different sizes from several host threads, each with a stream and a workspace of its own."""
    import threading
    cases = [make(T, H, 8, 2, 128, fmt=fmt, tail="residual", seed=80 + T)
             for T, H, fmt in [(8, 16384, "bf16"), (8, 12800, "bf16"), (2, 512, "fp8"), (6, 1024, "fp8")]]
    plans = [plan(M, d) for d in cases]
    want = [call(M, d, p)[0]["out"] for d, p in zip(cases, plans)]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(100):
                    o = call(M, cases[i], plans[i])[0]["out"]
                s.synchronize()
            assert torch.equal(o, want[i])
        except Exception as e:  # noqa: BLE001 (reported below, from the main thread)
            errors.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("E", [5, 31, 32, 33, 64, 65, 100, 128, 129, 200, 256])
def test_choice_among_equal_and_special_logits(M, E):
    """Larger logits first, equal ones (-0 and 0 among them) by the lower expert, NaN as -inf."""
    g = torch.Generator().manual_seed(E)
    k, T = min(8, E), 8
    d = make(T, 128, E, k, 64, routing="logits", seed=7)
    z = torch.randint(-2, 3, (T, E), generator=g).float() * 0.5
    z[z == 0] = torch.where(torch.rand((T, E), generator=g) < 0.5, 0.0, -0.0)[z == 0]
    z[1, torch.rand((E,), generator=g) < 0.7] = float("nan")
    z[2, torch.rand((E,), generator=g) < 0.7] = float("-inf")
    z[3] = 1.0
    z[4] = float("-inf")
    z[5] = float("nan")
    z[6] = torch.linspace(3e38, -3e38, E)  # (its step is beyond fp32: infinities, too)
    z[7] = torch.randn((E,), generator=g) * 1e-40
    d["logits"] = z.to(DEV)
    _, ids, tw = call(M, d)
    key = z.double().masked_fill(z.isnan(), float("-inf")) + 0.0
    want = key.sort(dim=1, descending=True, stable=True).indices[:, :k]
    assert ids.tolist() == want.tolist()
    top = key.gather(1, want)
    w = torch.softmax(top, 1)
    w[top[:, 0] == float("-inf")] = 0.0  # nothing but -inf (a weight beside +inf is NaN, as in any softmax)
    # exp, the sum and the divide: within 16 u of the weight (differences of fp32 logits are exact to u)
    tol = (16 + 2 * (top - top[:, :1]).abs().nan_to_num(0, 0, 0).clamp_max(100)) * U * w + 2.0 ** -126
    tw = tw.cpu().double()
    assert (((tw - w).abs() <= tol) | (tw.isnan() & w.isnan())).all()


@pytest.mark.parametrize("routing", ["router", "bias", "logits"])
@pytest.mark.parametrize("T,E", [(1, 65), (5, 96), (4, 128), (3, 129), (2, 200), (2, 256), (1, 256)])
def test_many_experts_of_few_tokens(M, T, E, routing):
    """The logits are added by all warps there, and by the token's own warp in a call with more tokens:
    both against the definition, and the same choice and weights."""
    d = make(8, 320, E, 8, 64, routing=routing, seed=E + T)
    whole = call(M, d)
    check(d, whole)
    few = dict(d, T=T, x=d["x"][:T].contiguous(), logits=None if d["logits"] is None else d["logits"][:T].contiguous())
    got = call(M, few)
    check(few, got)
    assert torch.equal(got[1], whole[1][:T]) and torch.equal(got[2], whole[2][:T])
    if routing == "logits":  # special ones, through this path as well
        few["logits"][0, ::2] = float("nan")
        few["logits"][0, 1] = float("-inf")
        few["logits"][T - 1, 3:] = 0.25
        whole = call(M, dict(d, logits=torch.cat([few["logits"], d["logits"][T:]])))
        got = call(M, few)
        assert torch.equal(got[1], whole[1][:T]) and torch.equal(got[2], whole[2][:T])


@pytest.mark.parametrize("spread", [20, 40])
@pytest.mark.parametrize("fmt", ["fp8", "block"])
@pytest.mark.parametrize("T", [1, 3, 4, 5, 8])
def test_spread_of_the_intermediate(M, T, fmt, spread):
    """Some of 128 intermediate columns 2^spread times the others: output rows whose W2 codes are 0 there
    come from the others alone.  (Values are held to 2^-38 of the largest of their 128 columns; at 2^20 that
    is below the 2^-16 that the tolerance counts, so there only the large column's own codes are 0 in some
    rows, at 2^40 those of its 128 columns.)"""
    I = 512
    d = make(T, 512, 6, 2, I, fmt=fmt, routing="ids", tail="residual", res=torch.float32, seed=90 + T)
    d["residual"].zero_()  # out = f in fp32
    if fmt == "fp8":
        large = slice(130, 131)
        d["w13_scale"][:, I + 130] *= 2.0 ** spread
    else:
        large = slice(128, 256)
        d["w13_scale"][:, (I + 128) // 128] *= 2.0 ** spread
    d["w2"][:, :, large] = 0x38  # 1.0
    d["w2"][:, ::3, 128:256] = 0
    if spread == 20:
        d["w2"][:, 1::3, large] = 0
    check(d, call(M, d))


@pytest.mark.parametrize("fmt", ["bf16", "fp8", "block"])
@pytest.mark.parametrize("T", [1, 4, 7])
def test_spread_of_the_input(M, T, fmt):
    """A column of x 2^30 times the others and weights of 0 beside it: intermediate columns of 2^-60 beside
    some of 2^8, and output rows that only the small ones reach."""
    H, I = 512, 384
    d = make(T, H, 6, 2, I, fmt=fmt, routing="ids", tail="residual", res=torch.float32, seed=95 + T)
    d["residual"].zero_()
    d["x"][:, 200] *= 2.0 ** 30
    for first in (0, I):  # gate and up rows of the first 128 intermediate columns
        d["w13"][:, first:first + 128, 128:256] = 0
    d["w2"][:, ::3, 128:] = 0
    res = call(M, d)
    check(d, res)
    assert 0 < res[0]["out"][:, ::3].abs().max() < 2.0 ** -40


@pytest.mark.parametrize("nxt,H", [("e4m3", 1024), ("e4m3g", 12288), ("e4m3g", 16384)])
def test_codes_are_those_of_the_quotient(M, nxt, H):
    """W2 of 0 and rows of +-1: x_hat is +-next_w exactly (as in test_gpu_block_tail), codes bit for bit."""
    for w in exact_weights(H, "group" if nxt == "e4m3g" else "row"):
        d = make(3, H, 2, 1, 64, routing="logits", tail="full", nxt=nxt, seed=5)
        d["w2"].zero_()
        d["residual"] = torch.where(d["x"] > 0, 1.0, -1.0).to(torch.bfloat16)
        d["next_w"], d["next_eps"] = w, 0.0
        o = call(M, d)[0]
        q, s = codes_by_definition(d["residual"].float() * w.float(), 128 if nxt == "e4m3g" else H)
        assert torch.equal(o["xscale"].cpu().view(s.shape), s) and torch.equal(o["xq"].cpu(), q)


@pytest.mark.parametrize("nxt", ["e4m3", "e4m3g"])
def test_scale_of_rows_that_vanish(M, nxt):
    d = make(3, 512, 2, 1, 64, routing="logits", tail="full", nxt=nxt, res=torch.float32, seed=5)
    d["w2"].zero_()
    d["residual"].zero_()
    d["residual"][:, ::2] = 2.0 ** -10
    d["next_w"] = torch.full((512,), 1, dtype=torch.int16, device=DEV).view(torch.bfloat16)  # 2^-133
    d["next_eps"] = 1.0
    o = call(M, d)[0]
    assert (o["xscale"] == 1).all() and (o["xq"] & 0x7f == 0).all()


@pytest.mark.parametrize("fmt,value", [("bf16", float("inf")), ("bf16", float("-inf")), ("bf16", float("nan")),
                                       ("fp8", 0x7f), ("fp8", 0xff), ("block", 0x7f)])
def test_one_weight_that_is_not_finite(M, fmt, value):
    """In W13 it takes the whole row of the tokens that use the expert, in W2 (without a tail) its own
    output column of them; other tokens keep theirs."""
    d = make(4, 256, 12, 2, 128, fmt=fmt, routing="ids", seed=4)
    d["ids"].copy_(torch.tensor([[0, 1], [2, 3], [6, 4], [5, 1]], dtype=torch.int32))
    f, df, *_ = block64(d)
    tol = df + 2.0 ** -8 * (f.abs() + df)
    for name, at in (("w13", (0, 5, 3)), ("w13", (0, 128 + 9, 200)), ("w2", (0, 7, 3))):
        w = d[name].clone()
        w[at] = value
        out = call(M, dict(d, **{name: w}))[0]["out"].double()
        good = torch.ones_like(out, dtype=torch.bool)
        if name == "w13":
            good[0] = False
            assert torch.isnan(out[0]).all()
        else:
            good[0, 7] = False
            assert not torch.isfinite(out[0, 7])
        assert ((out - f).abs() <= tol)[good].all()
