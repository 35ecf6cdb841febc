"""moe_combine_norm on the GPU against the tail's formulas in 64 bits.

The tolerances count roundings.  With u = 2^-24 (half a step of fp32) and
S = sum_j |y_j|:
  f       k - 1 additions                           |df| <= k u S
  r       a sum of H squares: at most 32 terms per thread, then two 5-step
          trees, one divide, one add, one square root, one reciprocal; half
          of the relative error of the sum reaches r
                                                    (24 + 4) u, plus |df|'s share
  g       f * r * w: two products
  h       scale * gate * g + residual: two products and one fma
  x_hat   as g, from h
and each output adds half a step of its own type."""
import itertools

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
RNORM = 28.0  # roundings (in u) of 1 / sqrt(mean of squares + eps)


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_ffn_rms_gb300 as M
    return M


@pytest.fixture(params=["auto", "row", "stream"])
def form(request, monkeypatch):
    """The launcher's own choice, and both kernels wherever their rows fit."""
    if request.param != "auto":
        monkeypatch.setenv("MOE_CN_STREAM", "1" if request.param == "stream" else "0")
    return request.param


def randn(g, *shape, std=1.0, mean=0.0, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).add_(mean).to(dtype)


def make(T, H, k, y=torch.bfloat16, order="pair", res=torch.bfloat16, post=True, gate="none",
         nxt="none", drop=0.0, seed=0, scale=0.7):
    g = torch.Generator(device=DEV).manual_seed(seed)
    d = dict(T=T, H=H, k=k, scale=scale, post_eps=1e-5, next_eps=1e-6)
    d["y"] = randn(g, T * k, H, std=0.3, dtype=y)
    d["pair_order"] = order != "expert"
    d["row_of_pair"] = None
    if order == "expert":
        d["row_of_pair"] = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32)
    elif order == "pair_idx":
        d["row_of_pair"] = torch.arange(T * k, device=DEV, dtype=torch.int32)
    if drop:
        d["row_of_pair"][torch.rand((T * k,), generator=g, device=DEV) < drop] = -1
    d["residual"] = randn(g, T, H, std=2.0, dtype=res) if res is not None else None
    d["post_w"] = randn(g, H, std=0.2, mean=0.6) if post else None
    d["gate"] = d["gate_row"] = None
    if gate == "channel":
        d["gate"] = randn(g, H)
    elif gate == "channel_f32":
        d["gate"] = randn(g, H, dtype=torch.float32)
    elif gate == "token":
        d["gate"] = randn(g, T, 1)
    elif gate == "token_f32":
        d["gate"] = randn(g, T, 1, dtype=torch.float32)
    elif gate == "full":
        d["gate"] = randn(g, T, H)
    elif gate == "rows":
        d["gate"] = randn(g, 5, H)
        d["gate_row"] = torch.randint(0, 5, (T,), generator=g, device=DEV, dtype=torch.int32)
    elif gate == "row_scalars":
        d["gate"] = randn(g, 5, 1, dtype=torch.float32)
        d["gate_row"] = torch.randint(0, 5, (T,), generator=g, device=DEV, dtype=torch.int32)
    d["next_w"] = randn(g, H, std=0.2, mean=1.0) if nxt != "none" else None
    d["next"] = nxt
    return d


def call(M, d, out=None, stream=None, inplace=False):
    T, H = d["T"], d["H"]
    nan = float("nan")
    if out is None:
        dt = d["residual"].dtype if d["residual"] is not None else torch.bfloat16
        out = torch.full((T, H), nan, device=DEV, dtype=dt)
    o = {"out": d["residual"] if inplace else out}
    n = d["next"]
    if n in ("bf16", "both"):
        o["xhat"] = torch.full((T, H), nan, device=DEV, dtype=torch.bfloat16)
    if n in ("e4m3", "both"):
        o["xq"] = torch.full((T, H), 0x7f, device=DEV, dtype=torch.uint8)
        o["xscale"] = torch.full((T,), nan, device=DEV)
    if n == "e4m3g":
        o["xq"] = torch.full((T, H), 0x7f, device=DEV, dtype=torch.uint8)
        o["xscale"] = torch.full((T, H // 128), nan, device=DEV)
    tail = M.make_block_tail(residual=d["residual"], post_w=d["post_w"], post_eps=d["post_eps"],
                             gate=d["gate"], gate_row=d["gate_row"], scale=d["scale"],
                             next_w=d["next_w"], next_eps=d["next_eps"], xhat=o.get("xhat"),
                             xq=o.get("xq"), xscale=o.get("xscale"))
    M.moe_combine_norm(d["y"], o["out"], T, d["k"], tail, row_of_pair=d["row_of_pair"],
                       pair_order=d["pair_order"], stream=stream)
    return o


def reference(d):
    """h, x_hat (64 bits) and the absolute error fp32 arithmetic may leave in each."""
    T, H, k = d["T"], d["H"], d["k"]
    y = d["y"].double()
    if d["row_of_pair"] is not None:
        ok = (d["row_of_pair"] >= 0)
        if not d["pair_order"]:
            y = y[d["row_of_pair"].clamp_min(0).long()]
        y = torch.where(ok[:, None], y, torch.zeros_like(y))
    y = y.view(T, k, H)
    f, df = y.sum(1), k * U * y.abs().sum(1)
    return tail_reference(d, f, df)


def norm_reference(v, dv, w, eps):
    ms = v.square().mean(1, keepdim=True) + eps
    r = 1 / ms.sqrt()
    # a relative error of the norm of v reaches r at most once
    share = dv.square().mean(1, keepdim=True).sqrt() * r
    g = v * r * w.double()
    return g, g.abs() * (RNORM * U + share + 2 * U) + dv * r * w.double().abs()


def tail_reference(d, f, df):
    T, H = f.shape
    if d["post_w"] is not None:
        f, df = norm_reference(f, df, d["post_w"], d["post_eps"])
    factor = torch.full((T, 1), d["scale"], device=DEV, dtype=torch.float64)
    factor = torch.tensor(d["scale"], dtype=torch.float32).double().item() + torch.zeros_like(factor)
    if d["gate"] is not None:
        gt = d["gate"].double()
        gt = gt[None].expand(T, -1) if gt.dim() == 1 else gt
        if d["gate_row"] is not None:
            gt = gt[d["gate_row"].long()]
        factor = factor * gt
    h = factor * f
    dh = factor.abs() * df + 3 * U * h.abs()
    if d["residual"] is not None:
        h = h + d["residual"].double()
        dh = dh + U * h.abs()
    if d["next_w"] is None:
        return h, dh, None, None
    x, dx = norm_reference(h, dh, d["next_w"], d["next_eps"])
    return h, dh, x, dx


def e4m3_values(q):
    return q.view(torch.float8_e4m3fn).double()


def assert_within(got, want, tol, what):
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    bad = (got - want).abs() > tol
    if bad.any():
        i = torch.nonzero(bad)[0].tolist()
        raise AssertionError(f"{what}: {int(bad.sum())} values off, first at {i}: got {got[tuple(i)]}, "
                             f"want {want[tuple(i)]} +- {tol[tuple(i)]}")


def check(d, o):
    h, dh, x, dx = reference(d)
    check_outputs(d, o, h, dh, x, dx)


def check_outputs(d, o, h, dh, x, dx):
    half = torch.finfo(o["out"].dtype).eps / 2
    assert_within(o["out"], h, dh + half * (h.abs() + dh), "out")
    if "xhat" in o:
        assert_within(o["xhat"], x, dx + 2.0 ** -8 * (x.abs() + dx), "xhat")
    if "xq" in o:
        T, H = h.shape
        n = 128 if d["next"] == "e4m3g" else H
        am = x.abs().view(T, -1, n).amax(-1)
        dam = dx.view(T, -1, n).amax(-1)
        s = am / 448
        got_s = o["xscale"].double().view(T, -1)
        zero = am == 0
        assert (got_s[zero] == 1).all()
        assert_within(got_s[~zero], s[~zero], (dam / 448 + U * s)[~zero], "xscale")
        sw = got_s.repeat_interleave(n, 1)
        # a code is half a step (2^-4 of the value, or 2^-10 below the normals) of x_hat / s
        tol = dx + 2.0 ** -4 * (x.abs() + dx) * (1 + 4 * U) + 2.0 ** -10 * sw
        assert_within(e4m3_values(o["xq"]) * sw, x, tol, "xq")


SIZES = [(1, 8), (3, 24), (5, 64), (2, 1000), (7, 2048), (4, 4096), (3, 7168), (2, 8200), (1, 16392),
         (2, 32768), (600, 264), (513, 4096), (640, 8192), (170, 16384), (1300, 7168)]


@pytest.mark.parametrize("T,H", SIZES)
@pytest.mark.parametrize("k", [1, 8])
def test_sizes(M, form, T, H, k):
    d = make(T, H, k, nxt="both", gate="channel", seed=T + H)
    check(d, call(M, d))


@pytest.mark.parametrize("y,order,res", list(itertools.product(
    [torch.bfloat16, torch.float32], ["pair", "pair_idx", "expert"],
    [None, torch.bfloat16, torch.float32])))
def test_types_and_orders(M, form, y, order, res):
    for T, H, k in ((6, 512, 4), (530, 1032, 3)):
        d = make(T, H, k, y=y, order=order, res=res, nxt="bf16", drop=0.0, seed=k)
        check(d, call(M, d))


@pytest.mark.parametrize("gate", ["none", "channel", "channel_f32", "token", "token_f32", "full", "rows",
                                  "row_scalars"])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("nxt", ["none", "bf16", "e4m3", "e4m3g", "both"])
def test_gates_and_outputs(M, form, gate, post, nxt):
    for T, H, k in ((1, 128, 1), (9, 640, 2), (515, 384, 1)):
        d = make(T, H, k, post=post, gate=gate, nxt=nxt, seed=T)
        check(d, call(M, d))


@pytest.mark.parametrize("order", ["pair_idx", "expert"])
def test_skipped_pairs(M, form, order):
    d = make(40, 256, 4, order=order, drop=0.5, nxt="bf16", seed=3)
    d["row_of_pair"][8:12] = -1  # token 2 has no row at all: f = 0, out = residual
    o = call(M, d)
    check(d, o)
    assert torch.equal(o["out"][2], d["residual"][2])


def test_empty_rows_and_zero_input(M, form):
    d = make(4, 256, 2, order="pair_idx", res=None, nxt="e4m3", seed=4)
    d["row_of_pair"].fill_(-1)  # f = 0 everywhere and no residual: h = 0
    o = call(M, d)
    assert (o["out"] == 0).all() and (o["xq"] & 0x7f == 0).all() and (o["xscale"] == 1).all()
    d = make(4, 256, 2, res=None, nxt="e4m3g", seed=4)
    d["y"].zero_()
    o = call(M, d)
    assert (o["out"] == 0).all() and (o["xq"] & 0x7f == 0).all() and (o["xscale"] == 1).all()


def test_non_finite_rows_stay_in_their_token(M, form):
    d = make(6, 512, 2, nxt="both", gate="rows", seed=5)
    clean = call(M, d)
    d["y"][4] = float("nan")       # token 2
    d["residual"][4, 7] = float("inf")  # token 4
    o = call(M, d)
    for t in (0, 1, 3, 5):
        for n in o:
            assert torch.equal(o[n][t], clean[n][t]), (n, t)
    assert torch.isnan(o["out"][2]).all() and torch.isnan(o["xhat"][2]).all()
    assert torch.isinf(o["out"][4, 7])


def test_bad_indices_are_flagged_and_skipped(M, form):
    M.device_status(clear=True)
    d = make(8, 256, 2, order="expert", gate="rows", nxt="bf16", seed=6)
    want = dict(d, row_of_pair=d["row_of_pair"].clone())
    d["row_of_pair"][5] = 16
    d["row_of_pair"][9] = 2 ** 31 - 1
    want["row_of_pair"][5] = want["row_of_pair"][9] = -1
    o = call(M, d)
    check(want, o)
    assert M.device_status(clear=True) == 1
    d = make(8, 256, 2, gate="rows", nxt="bf16", seed=6)
    d["gate_row"][3] = 5
    d["gate_row"][6] = -1
    o = call(M, d)
    assert M.device_status(clear=True) == 1
    assert torch.equal(o["out"][3], d["residual"][3]) and torch.equal(o["out"][6], d["residual"][6])
    keep = [0, 1, 2, 4, 5, 7]
    d["gate_row"][3] = d["gate_row"][6] = 0
    o2 = call(M, d)
    assert torch.equal(o["out"][keep], o2["out"][keep])
    assert M.device_status(clear=True) == 0


def test_in_place_and_rows_behind_the_last(M, form):
    d = make(5, 512, 2, nxt="bf16", seed=7)
    want = call(M, d)
    keep = d["residual"].clone()
    d2 = dict(d, residual=d["residual"].clone())
    got = call(M, d2, inplace=True)
    assert torch.equal(got["out"], want["out"]) and torch.equal(got["xhat"], want["xhat"])
    assert torch.equal(d["residual"], keep)
    big = torch.full((8, 512), 7.0, device=DEV, dtype=torch.bfloat16)
    call(M, d, out=big[:5])
    assert torch.equal(big[:5], want["out"]) and (big[5:] == 7.0).all()


def test_no_tokens(M):
    d = make(1, 256, 2, nxt="bf16")
    n = M.lib.moe_launch_count()
    tail = M.make_block_tail(post_w=d["post_w"], scale=1.0)
    M.moe_combine_norm(d["y"][:0], d["y"][:0], 0, 2, tail)
    assert M.lib.moe_launch_count() == n


def test_equals_combine_and_rmsnorm(M):
    """Without a norm after the block it is moe_combine, + residual, moe_rmsnorm."""
    d = make(33, 1024, 8, order="pair_idx", post=False, res=None, nxt="bf16", scale=1.0, seed=8)
    o = call(M, d)
    ref = torch.empty((33, 1024), dtype=torch.bfloat16, device=DEV)
    M.moe_combine(d["y"], d["row_of_pair"], 33, 8, ref, pair_order=True)
    assert torch.equal(o["out"], ref)  # the same sum in the same order, rounded once


def test_streams_and_graph(M):
    ds = [make(64, 1024, 4, nxt="both", gate="channel", seed=20 + i) for i in range(2)]
    want = [call(M, d) for d in ds]
    torch.cuda.synchronize()
    ss = [torch.cuda.Stream() for _ in ds]
    got = [None, None]
    for _ in range(3):  # two streams at once
        for i, d in enumerate(ds):
            with torch.cuda.stream(ss[i]):
                got[i] = call(M, d)
    torch.cuda.synchronize()
    for w, o in zip(want, got):
        for n in w:
            assert torch.equal(w[n], o[n]), n
    # captured once, replayed on changed inputs
    g = torch.cuda.CUDAGraph()
    d = dict(ds[0], y=ds[0]["y"].clone())
    with torch.cuda.graph(g):
        o = call(M, d)
    d["y"].copy_(ds[1]["y"])
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    w = call(M, dict(ds[0], y=ds[1]["y"]))
    for n in w:
        assert torch.equal(w[n], o[n]), n


def test_after_the_grouped_ffn(M):
    """As a program uses it: the FFN step's rows, then the tail, then the next rms_norm's input."""
    import workloads
    inp = workloads.make_inputs("c1_tiny", DEV)
    T, H, E, k, I = inp["T"], inp["H"], inp["E"], inp["k"], inp["I"]
    shape = M.make_shape(T, H, E, I, k, inp["eps"])
    xh = torch.empty_like(inp["x"])
    M.moe_rmsnorm(inp["x"], inp["norm_w"], inp["eps"], xh)
    ids = torch.empty((T, k), dtype=torch.int32, device=DEV)
    tw = torch.empty((T, k), dtype=torch.float32, device=DEV)
    wsr = M.alloc_workspace(M.moe_route_workspace_size(T, H, E), DEV)
    M.moe_route_topk(T, H, E, k, ids, tw, xhat=xh, router_w=inp["router_w"], workspace=wsr)
    off = torch.empty((E + 1,), dtype=torch.int32, device=DEV)
    src, rop = (torch.empty((T * k,), dtype=torch.int32, device=DEV) for _ in range(2))
    xp = torch.empty((T * k, H), dtype=torch.bfloat16, device=DEV)
    M.moe_permute(ids, T, E, k, off, src, rop, xhat=xh, xp=xp, row_bytes=2 * H)
    act = torch.empty((T * k, I), dtype=torch.bfloat16, device=DEV)
    y = torch.empty((T * k, H), dtype=torch.float32, device=DEV)
    M.moe_grouped_gemm(shape, M.GEMM_FC1_SILU, xp, inp["w13"], off, act)
    M.moe_grouped_gemm(shape, M.GEMM_FC2, act, inp["w2"], off, y, row_src=src, topk_w=tw)
    g = torch.Generator(device=DEV).manual_seed(1)
    d = dict(T=T, H=H, k=k, y=y, pair_order=False, row_of_pair=rop, residual=inp["x"],
             post_w=randn(g, H, std=0.1, mean=0.5), gate=None, gate_row=None, scale=1.0,
             post_eps=1e-6, next_eps=1e-6, next_w=inp["norm_w"], next="both")
    check(d, call(M, d))


def test_host_threads_at_once(M):
    """Calls of different sizes from several host threads, each on a stream of its own."""
    import threading
    cases = [make(T, H, k, nxt="bf16", res=None, seed=70 + i)
             for i, (T, H, k) in enumerate([(400, 2048, 8), (600, 512, 2), (300, 4096, 8), (900, 256, 1)])]
    want = [call(M, d) for d in cases]
    torch.cuda.synchronize()
    errors = []

    def work(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for _ in range(200):
                    o = call(M, cases[i])
                s.synchronize()
            for n in want[i]:
                assert torch.equal(want[i][n], o[n]), n
        except Exception as e:  # noqa: BLE001 (reported below, from the main thread)
            errors.append(e)

    ts = [threading.Thread(target=work, args=(i,)) for i in range(len(cases))]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not errors, errors


@pytest.mark.parametrize("H,T,k", [(4096, 70000, 8), (32768, 70000, 1)])
def test_offsets_beyond_32_bits(M, H, T, k):
    """More elements than 32 bits count; the rows that are checked lie at the ends and beside 2^31 elements."""
    g = torch.Generator(device=DEV).manual_seed(9)
    base = randn(g, 4096, H, std=0.3)
    y = base.repeat(-(-T * k // 4096), 1)[:T * k]
    assert y.numel() > 2 ** 31
    d = dict(T=T, H=H, k=k, scale=0.7, post_eps=1e-5, next_eps=1e-6, y=y, pair_order=True, row_of_pair=None,
             residual=None, post_w=randn(g, H, std=0.2, mean=0.6), gate=None, gate_row=None,
             next_w=randn(g, H, std=0.2, mean=1.0), next="bf16")
    o = call(M, d)
    at = 2 ** 31 // (H * k)  # the token that holds element 2^31 of y
    rows = torch.tensor([0, 1, at - 1, at, at + 1, T // 2, T - 2, T - 1], device=DEV)
    part = dict(d, T=len(rows), y=y.view(T, k, H)[rows].reshape(-1, H))
    check(part, {n: v[rows] for n, v in o.items()})


@pytest.mark.parametrize("T,H,k,y,res", [
    (400, 12288, 1, torch.bfloat16, torch.bfloat16), (330, 12288, 3, torch.bfloat16, torch.float32),
    (400, 9000, 8, torch.bfloat16, torch.bfloat16), (310, 15872, 8, torch.bfloat16, torch.bfloat16),
    (700, 5000, 2, torch.bfloat16, torch.bfloat16), (700, 5000, 8, torch.bfloat16, torch.bfloat16),
    (320, 7936, 8, torch.float32, torch.float32), (500, 7944, 4, torch.bfloat16, None),
    (900, 5120, 2, torch.float32, torch.bfloat16), (640, 8192, 1, torch.bfloat16, torch.float32),
    (330, 16384, 2, torch.bfloat16, torch.bfloat16), (320, 8200, 1, torch.float32, torch.bfloat16)])
@pytest.mark.parametrize("gate,post,nxt", [("none", True, "both"), ("rows", True, "bf16"),
                                           ("channel", False, "both"), ("token", True, "none")])
def test_long_rows_of_many_tokens(M, T, H, k, y, res, gate, post, nxt):
    """Several tokens per CTA in every width of the streaming form, with whole and split tokens."""
    d = make(T, H, k, y=y, order="pair_idx", res=res, post=post, gate=gate, nxt=nxt, drop=0.2, seed=T + H + k)
    o = call(M, d)
    check(d, o)
    again = call(M, d)
    for n in o:
        assert torch.equal(o[n], again[n]), n
    assert M.device_status() == 0


def exact_weights(H, form):
    """Norm weights in bf16 whose quotients by max / 448 lie beside ties of E4M3: every mantissa under a
    maximum of every mantissa (a group's, or the row's own)."""
    mant = 1.0 + torch.arange(128) / 128.0
    j = torch.arange(H)
    w = mant[j % 128] * 2.0 ** -(1 + (j // 128 + j) % 20)  # (codes below the normals and 0 among them)
    if form == "group":
        w[::128] = mant[(torch.arange(H // 128)) % 128]
        return [w.to(torch.bfloat16).to(DEV)]
    rows = []
    for i in (0, 10, 24, 38, 68, 76, 80, 120, 127):  # where a product by the reciprocal differs, and others
        v = w.clone()
        v[5] = mant[i]
        rows.append(v.to(torch.bfloat16).to(DEV))
    return rows


def codes_by_definition(x, n):
    """Codes and scales of x (fp32, on the CPU): IEEE divisions, one scale per n columns."""
    t = x.float().cpu().view(x.shape[0], -1, n)
    s = t.abs().amax(-1) / 448
    s = torch.where(s > 0, s, torch.ones_like(s))
    q = (t / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return q.view(x.shape), s


@pytest.mark.parametrize("T", [3, 400])
@pytest.mark.parametrize("nxt,H", [("e4m3", 1024), ("e4m3", 5120), ("e4m3g", 16384)])
def test_codes_are_those_of_the_quotient(M, form, nxt, H, T):
    """Rows of +-1 (their norm is 1 without eps), so x_hat is +-next_w exactly: codes bit for bit."""
    for w in exact_weights(H, "group" if nxt == "e4m3g" else "row"):
        d = make(T, H, 1, post=False, nxt=nxt, seed=3)
        d["y"].zero_()
        d["residual"] = torch.where(d["residual"] > 0, 1.0, -1.0).to(torch.bfloat16)
        d["next_w"], d["next_eps"] = w, 0.0
        o = call(M, d)
        x = (d["residual"].float() * w.float()).to(torch.bfloat16)
        q, s = codes_by_definition(x, 128 if nxt == "e4m3g" else H)
        assert torch.equal(o["xscale"].cpu().view(s.shape), s)
        assert torch.equal(o["xq"].cpu(), q)
        if nxt == "e4m3":  # and those of the library's own quantisation
            q2, s2 = torch.empty_like(o["xq"]), torch.empty_like(o["xscale"])
            M.moe_quantize_fp8_rows(x, q2, s2)
            assert torch.equal(o["xq"], q2) and torch.equal(o["xscale"], s2)


@pytest.mark.parametrize("nxt", ["e4m3", "e4m3g"])
@pytest.mark.parametrize("T", [3, 400])
def test_scale_of_rows_that_vanish(M, form, nxt, T):
    """x_hat of 2^-143 (64 steps of the smallest fp32): its 448th part is 0, the scale 1, the codes 0."""
    d = make(T, 512, 1, post=False, nxt=nxt, res=torch.float32, seed=3)
    d["y"].zero_()
    d["residual"].zero_()
    d["residual"][:, ::2] = 2.0 ** -10
    d["next_w"] = torch.full((512,), 1, dtype=torch.int16, device=DEV).view(torch.bfloat16)  # 2^-133
    d["next_eps"] = 1.0
    o = call(M, d)
    assert (o["xscale"] == 1).all() and (o["xq"] & 0x7f == 0).all()


@pytest.mark.parametrize("T", [33, 700])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_equals_combine_residual_and_rmsnorm(M, form, T, res):
    """Integers whose sums and squares are exact in every step: out is moe_combine + residual and x_hat the
    stand-alone moe_rmsnorm of it, bit for bit."""
    d = make(T, 1024, 8, order="pair_idx", post=False, res=res, nxt="bf16", scale=1.0, seed=8)
    g = torch.Generator(device=DEV).manual_seed(8)
    d["y"] = torch.randint(-4, 5, d["y"].shape, generator=g, device=DEV).to(torch.bfloat16)
    d["residual"] = torch.randint(-64, 65, (T, 1024), generator=g, device=DEV).to(res)
    d["next_eps"] = 2.0 ** -20
    o = call(M, d)
    f = torch.empty((T, 1024), dtype=torch.bfloat16, device=DEV)
    M.moe_combine(d["y"], d["row_of_pair"], T, 8, f, pair_order=True)
    h = f.float() + d["residual"].float()
    assert torch.equal(o["out"].float(), h)
    x = torch.empty_like(f)
    M.moe_rmsnorm(h.to(torch.bfloat16), d["next_w"], d["next_eps"], x)
    assert torch.equal(o["xhat"], x)
