"""moe_linear and moe_linear_backward on the GPU against their formulas in 64 bits.

The tolerances: products of bf16 values are exact in fp32, and their sums are truncated additions in the
tensor cores, at most 2^-23 of the running sum each, 16 products at a time:
  sum of n products  e = 2^-23 (n / 16 + 4) sum |terms|   (fp32 results add at most 768 of them so, and the
                     sums of those rounded to nearest: 2^-23 (n / 768 + 52) sum |terms|)
  bias, residual     one rounding of 2^-24 each
  activation         |slope| e (|slope| <= 1.13), and 2^-20 |z| (1 + |z|) of its own: the fast exponential's argument
                     is rounded (2^-24 |u|) and the result is off by 2^-21
  dpre               2^-20 (1 + |z|)^2 |dout| (the same, with z sigma'), and half a step of bf16 where it enters a
                     product
and each output adds half a step of its own type."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32
ACTS = ["NONE", "RELU", "SILU", "GELU", "GELU_TANH"]


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_ffn_rms_gb300 as M
    M.check_device()
    M.device_status()
    return M


@pytest.fixture(params=["auto", "pair", "split"])
def form(request, monkeypatch):
    """The launcher's own choice, and both kernels everywhere."""
    if request.param != "auto":
        monkeypatch.setenv("MOE_LINEAR_FORM", request.param)
    return request.param


def step(t, v):
    return v * (torch.finfo(t).eps / 2)


def gen(seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def rn(*s, std=1.0, dtype=BF):
        return torch.randn(s, generator=g, device=DEV).mul_(std).to(dtype)
    return rn


def act64(z, act):
    if act == "RELU":
        return z.clamp(min=0)
    if act == "SILU":
        return z * torch.sigmoid(z)
    if act == "GELU":
        return z * 0.5 * torch.erfc(-z / math.sqrt(2))
    if act == "GELU_TANH":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z


def sum_err(n, size, f32):
    return (2 * U) * ((n / 768 + 52) if f32 and n > 768 else (n / 16 + 4)) * size


def forward(M, m, n, k, act="NONE", bias=None, res=None, out=BF, pre=False, seed=0, inplace=False):
    rn = gen(seed + m + 3 * n + 7 * k)
    x, w = rn(m, k), rn(n, k, std=k ** -0.5)
    b = None if bias is None else rn(n, std=0.5, dtype=bias)
    r = None if res is None else rn(m, n, std=2.0, dtype=res)
    o = torch.full((m, n), float("nan"), device=DEV, dtype=out)
    p = torch.full((m, n), float("nan"), device=DEV, dtype=BF) if pre else None
    if inplace:
        o.copy_(r)
        rr = o
    else:
        rr = r
    M.moe_linear(x, w, o, bias=b, residual=rr, act=getattr(M, "ACT_" + act), pre=p)
    xd, wd = x.double(), w.double()
    z = xd @ wd.t()
    e = sum_err(k, xd.abs() @ wd.abs().t(), out == F32)
    if b is not None:
        z = z + b.double()
        e = e + U * z.abs()
    if pre:
        assert ((p.double() - z).abs() <= e + step(BF, z.abs() + e)).all()
    f = act64(z, act)
    if act != "NONE":
        e = 1.13 * e + 2.0 ** -20 * z.abs() * (1 + z.abs())
    if r is not None:
        f = f + r.double()
        e = e + U * f.abs()
    tol = e + step(out, f.abs() + e)
    bad = (o.double() - f).abs() > tol
    assert not bad.any(), (int(bad.sum()), bad.nonzero()[:4].tolist())
    assert M.device_status() == 0
    return o


SHAPES = [(1, 8, 8), (1, 128, 64), (1, 4096, 4096), (1, 1032, 12296), (2, 136, 200), (4, 5128, 520), (3, 256, 1000), (16, 512, 256), (17, 1032, 72),
          (33, 264, 4104), (61, 7168, 2048), (64, 128, 512), (65, 384, 320), (100, 1544, 2944), (128, 256, 128),
          (129, 2056, 136), (255, 520, 1032), (256, 4096, 512), (257, 776, 264), (333, 2944, 1000),
          (512, 512, 8192), (1000, 4104, 1536), (2047, 2048, 520), (4096, 1288, 264), (2500, 5128, 1024)]


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_forward_shapes(M, m, n, k, form):
    forward(M, m, n, k)
    forward(M, m, n, k, act="SILU", bias=BF, res=F32, out=F32)
    forward(M, m, n, k, bias=F32, res=BF, out=BF, inplace=True)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(5, 264, 136), (300, 1032, 520), (2100, 2312, 200)])
def test_forward_epilogues(M, m, n, k, act, form):
    for bias in (None, BF, F32):
        for res in (None, BF, F32):
            for out in (BF, F32):
                forward(M, m, n, k, act=act, bias=bias, res=res, out=out, pre=act != "NONE",
                        inplace=res is not None and res == out)


@pytest.mark.parametrize("m", [1, 300, 1100])
def test_long_sums_keep_fp32(M, m, form):
    """fp32 outputs of long sums: against 64 bits, relative to the whole output."""
    n, k = 512, 16384
    rn = gen(m)
    x, w = rn(m, k), rn(n, k)
    out = torch.empty((m, n), device=DEV)
    M.moe_linear(x, w, out)
    ref = x.double() @ w.double().t()
    # sums of 768 terms truncated (0.9e-6 of their size), 22 of them added: as a random walk no more than that
    assert (out.double() - ref).norm() <= 2e-6 * ref.norm()


def slope64(z, act):
    z = z.clone().requires_grad_()
    return torch.autograd.grad(act64(z, act).sum(), z)[0].detach()


def backward(M, m, n, k, act="NONE", dout=BF, dw=BF, which="dx dw db", seed=0):
    rn = gen(seed + m + 3 * n + 7 * k)
    x, w, d = rn(m, k), rn(n, k, std=k ** -0.5), rn(m, n, std=0.1, dtype=dout)
    pre = None if act == "NONE" else rn(m, n, std=2.0)
    o = {"dx": torch.full((m, k), float("nan"), device=DEV, dtype=BF),
         "dw": torch.full((n, k), float("nan"), device=DEV, dtype=dw),
         "db": torch.full((n,), float("nan"), device=DEV)}
    o = {a: t for a, t in o.items() if a in which}
    ws = M.alloc_workspace(M.moe_linear_backward_workspace_size(m, n, k))
    ws.fill_(255)
    M.moe_linear_backward(d, x, w, ws, pre=pre, act=getattr(M, "ACT_" + act), **o)
    g, e = d.double(), torch.zeros((), device=DEV, dtype=torch.float64)
    if act != "NONE":
        z = pre.double()
        g = g * (slope64(z, act) if act != "RELU" else (z > 0).double())
        e = 2.0 ** -20 * (1 + z.abs()) ** 2 * d.double().abs()
    if "db" in o:
        s = g.abs().sum(0)
        rows = m / 128 + 300
        tol = (e * torch.ones_like(g)).sum(0) + rows * U * s
        assert ((o["db"].double() - g.sum(0)).abs() <= tol + U * s).all()
    if act != "NONE" or dout == F32:
        e = e + step(BF, g.abs() + e)
    e = e * torch.ones_like(g)
    for name, a, b, ea in (("dx", g, w.double(), e), ("dw", g.t(), x.double(), e.t())):
        if name not in o:
            continue
        ref = a @ b
        size = a.abs() @ b.abs()
        tol = ea @ b.abs() + sum_err(a.shape[1], size, o[name].dtype == F32)
        tol = tol + step(o[name].dtype, ref.abs() + tol)
        bad = (o[name].double() - ref).abs() > tol
        assert not bad.any(), (name, int(bad.sum()), bad.nonzero()[:4].tolist())
    assert M.device_status() == 0
    return o


@pytest.mark.parametrize("m,n,k", SHAPES)
def test_backward_shapes(M, m, n, k, form):
    backward(M, m, n, k, dw=F32)
    backward(M, m, n, k, act="GELU_TANH")
    one = backward(M, m, n, k, dout=F32, dw=F32)
    for name in ("dx", "dw", "db"):  # each alone has the same bits
        alone = backward(M, m, n, k, dout=F32, dw=F32, which=name)
        assert torch.equal(alone[name], one[name])


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("m,n,k", [(40, 264, 136), (700, 1032, 520), (4096, 256, 256)])
def test_backward_activations(M, m, n, k, act, form):
    for dout in (BF, F32):
        for dw in (BF, F32):
            backward(M, m, n, k, act=act, dout=dout, dw=dw)


# few tiles and a long K (clusters of up to sixteen, tiles narrower than the rows), in each product
LONG = [(1, 64, 16384), (16, 128, 16392), (25, 456, 4024), (64, 256, 8192), (100, 72, 5000), (128, 256, 256),
        (200, 136, 12288), (512, 1024, 1024), (700, 264, 2056)]


@pytest.mark.parametrize("m,n,k", LONG)
def test_few_tiles_and_long_sums(M, m, n, k, form):
    forward(M, m, n, k, act="GELU", bias=F32, res=BF, pre=True)
    forward(M, m, n, k, out=F32)
    backward(M, m, k, n, which="dx")
    backward(M, max(k, 16), n, max(m // 8 * 8, 8), which="dw")
    backward(M, max(k, 16), n, max(m // 8 * 8, 8), dw=F32, which="dw")


@pytest.mark.parametrize("act", ["SILU", "GELU", "GELU_TANH"])
def test_backward_against_differences(M, act):
    """Gradients against central differences of the forward in 64 bits at the kept bf16 values."""
    m, n, k = 12, 24, 16
    rn = gen(1)
    x, w, b, d = rn(m, k), rn(n, k, std=0.3), rn(n, std=0.3, dtype=F32), rn(m, n, dtype=F32)
    out, pre = torch.empty((m, n), device=DEV), torch.empty((m, n), device=DEV, dtype=BF)
    a = getattr(M, "ACT_" + act)
    M.moe_linear(x, w, out, bias=b, act=a, pre=pre)
    dx, dw, db = torch.empty_like(x), torch.empty((n, k), device=DEV), torch.empty(n, device=DEV)
    M.moe_linear_backward(d, x, w, M.alloc_workspace(M.moe_linear_backward_workspace_size(m, n, k)), dx=dx, dw=dw,
                          db=db, pre=pre, act=a)
    vx, vw, vb = (rn(*t.shape, dtype=F32).double() for t in (x, w, b))

    def loss(h):
        z = (x.double() + h * vx) @ (w.double() + h * vw).t() + b.double() + h * vb
        return (act64(z, act) * d.double()).sum()

    h = 1e-4
    num = (loss(h) - loss(-h)) / (2 * h)
    parts = [dx.double() * vx, dw.double() * vw, db.double() * vb]
    # bf16 pre (half a step of |z| times the slope's slope, below 1), bf16 dpre, bf16 dx
    z = x.double() @ w.double().t() + b.double()
    dz = (vx @ w.double().t() + x.double() @ vw.t() + vb).abs()
    tol = (d.double().abs() * dz * (2.0 ** -8 * (1 + z.abs()))).sum() + 2.0 ** -8 * parts[0].abs().sum() + 1e-6
    assert abs(num - sum(p.sum() for p in parts)) <= tol


def test_special_values_stay_where_they_belong(M, form):
    """A NaN or an infinity in a row of x (a column of the output's transpose) reaches that row alone, values outside
    the matrices never count, and each activation keeps its limits."""
    m, n, k = 70, 200, 72
    rn = gen(2)
    x, w = rn(m, k), rn(n, k, std=0.1)
    clean = torch.empty((m, n), device=DEV, dtype=BF)
    M.moe_linear(x, w, clean)
    y = x.clone()
    y[5, 3] = float("nan")
    out = torch.empty_like(clean)
    M.moe_linear(y, w, out)
    assert torch.isnan(out[5]).all()
    keep = torch.arange(m, device=DEV) != 5
    assert torch.equal(out[keep], clean[keep])
    # the operands as the inner part of buffers full of NaN
    big = torch.full((m * k + 64,), float("nan"), device=DEV, dtype=BF)
    xs = big[:m * k].view(m, k)
    xs.copy_(x)
    M.moe_linear(xs, w, out)
    assert torch.equal(out, clean)
    # saturated activations: exp overflows, z^3 leaves the exponent's range
    z = torch.tensor([-3e38, -1e30, -200.0, -100.0, -20.0, 0.0, 20.0, 100.0, 1e30, 3e38, 0.0, 0.0, 0.0, 0.0, 0.0, 0.0],
                     device=DEV)
    one, zero = torch.zeros((1, 8), device=DEV, dtype=BF), torch.zeros((16, 8), device=DEV, dtype=BF)
    for act in ACTS[1:]:
        a = getattr(M, "ACT_" + act)
        f = torch.empty((1, 16), device=DEV)
        M.moe_linear(one, zero, f, bias=z, act=a)
        want = torch.where(z > 0, z, torch.zeros_like(z))
        assert ((f[0] - want).abs() <= 1e-6 * (1 + z.abs())).all(), act
        db = torch.empty(16, device=DEV)
        M.moe_linear_backward(torch.ones((1, 16), device=DEV), one, zero,
                              M.alloc_workspace(M.moe_linear_backward_workspace_size(1, 16, 8)), db=db,
                              pre=z.to(BF)[None], act=a)
        want = torch.where(z > 0, 1.0, 0.0)
        ok = (db - want).abs() <= 1e-6
        assert ok[z.abs() >= 20].all(), (act, db)


@pytest.mark.parametrize("act", ["SILU", "GELU", "GELU_TANH"])
def test_activations_keep_their_relative_precision(M, act):
    """Over the whole range, the lower tail included, z given exactly by the bias.  An exponent of size u has three
    roundings (3 U u relative in the result); the factors around it, 1 / (1 + .) and a polynomial within 1.3e-7,
    have less than 16 more.  Results below 2^-126 may be 0."""
    n = 4096
    z = torch.linspace(-13.0, 13.0, n, device=DEV).to(BF)
    zd = z.double()
    one, zero = torch.zeros((1, 8), device=DEV, dtype=BF), torch.zeros((n, 8), device=DEV, dtype=BF)
    a = getattr(M, "ACT_" + act)
    f, db = torch.empty((1, n), device=DEV), torch.empty(n, device=DEV)
    M.moe_linear(one, zero, f, bias=z.float(), act=a)
    M.moe_linear_backward(torch.ones((1, n), device=DEV), one, zero,
                          M.alloc_workspace(M.moe_linear_backward_workspace_size(1, n, 8)), db=db, pre=z[None], act=a)
    c = 2 * math.sqrt(2 / math.pi)
    if act == "SILU":
        u, gate = zd.abs(), torch.sigmoid(zd)
        parts = gate, zd * gate * torch.sigmoid(-zd)
        loss = (zd * gate).abs()
    elif act == "GELU":
        u, gate = zd * zd / 2, 0.5 * torch.erfc(-zd / math.sqrt(2))
        parts = gate, zd * torch.exp(-u) / math.sqrt(2 * math.pi)
        loss = 0 * zd
    else:
        u = (c * (zd + 0.044715 * zd ** 3)).abs()
        gate, rise = torch.sigmoid(u * zd.sign()), zd * c * (1 + 3 * 0.044715 * zd * zd)
        parts = gate, rise * gate * torch.sigmoid(-u * zd.sign())
        loss = (rise * gate).abs()
    rel, least = U * (16 + 3 * u), 2.0 ** -126 * (1 + zd.abs() ** 3)
    want = zd * gate
    assert ((f[0].double() - want).abs() <= rel * want.abs() + least).all()
    # the slope: its two terms' errors, and that of 1 - gate, two roundings of 1, times what stands before it
    size = parts[0] + parts[1].abs()
    assert ((db.double() - parts[0] - parts[1]).abs() <= 2 * rel * size + 2 * U * loss + least).all()


def test_streams_graphs_shared_workspace_and_empty_batches(M, form):
    m, n, k = 130, 1032, 520
    rn = gen(4)
    x, w, b, d = rn(m, k), rn(n, k, std=0.05), rn(n), rn(m, n)
    ws = M.alloc_workspace(M.moe_linear_backward_workspace_size(m, n, k))

    def bufs():
        return (torch.zeros((m, n), device=DEV, dtype=BF), torch.zeros((m, n), device=DEV, dtype=BF),
                torch.zeros((m, k), device=DEV, dtype=BF), torch.zeros((n, k), device=DEV),
                torch.zeros(n, device=DEV))

    def run(o, ws=ws, stream=None):
        M.moe_linear(x, w, o[0], bias=b, act=M.ACT_SILU, pre=o[1], stream=stream)
        M.moe_linear_backward(d, x, w, ws, dx=o[2], dw=o[3], db=o[4], pre=o[1], act=M.ACT_SILU, stream=stream)

    ref = bufs()
    run(ref)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    many = [(bufs(), torch.empty_like(ws)) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, (o, wk) in zip(streams, many):
            run(o, wk, s)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    graphs = []
    with torch.cuda.stream(s):
        for _ in range(2):
            o = bufs()
            run(o)
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                run(o)
            for t in o:
                t.zero_()
            graphs.append((g, o))
        for g, _ in graphs * 2:
            g.replay()
    torch.cuda.synchronize()
    for o in [o for o, _ in many] + [o for _, o in graphs]:
        assert all(torch.equal(p, q) for p, q in zip(o, ref))
    e = torch.empty((0, k), device=DEV, dtype=BF)
    M.moe_linear(e, w, torch.empty((0, n), device=DEV, dtype=BF))
    ref[3].fill_(7)
    ref[4].fill_(7)
    M.moe_linear_backward(torch.empty((0, n), device=DEV, dtype=BF), e, w, ws, dw=ref[3], db=ref[4])
    assert (ref[3] == 0).all() and (ref[4] == 0).all()
    assert M.device_status() == 0


def test_offsets_beyond_32_bits(M):
    """An output of more than 2^31 elements: the last rows hold what the first do."""
    m, n, k = 270000, 8200, 64
    x = torch.empty((m, k), device=DEV, dtype=BF)
    x.view(-1, 1000, k)[:] = gen(6)(1000, k)
    w = gen(7)(n, k, std=0.1)
    out = torch.empty((m, n), device=DEV, dtype=BF)
    M.moe_linear(x, w, out)
    o = out.view(-1, 1000, n)
    assert torch.equal(o[-1], o[0]) and torch.equal(o[137], o[0])
    ref = x[:1000].double() @ w.double().t()
    assert ((o[0].double() - ref).abs() <= step(BF, ref.abs()) + 1e-5).all()
