"""moe_layernorm and the backward passes of layer norm and rms_norm on the GPU against their formulas in 64
bits.

The tolerances count roundings, u = 2^-24 (half a step of fp32).  A sum over a row adds at most 32 values in
a chain per thread and 10 steps over the CTA, and is divided once: R = 44 u of the sum of magnitudes.
  mean   em = R sum |x| / H
  rstd   relative: half of (R + 4 u), of the sum of squares and its square root, + (em / sigma)^2 + 2 u
  y      |v r w| (er + 3 u) + em r |w| + u |y|
  dx     r (3 u (|g| + |c0| + |xh c1|) + e0 + |xh| e1), with e0, e1 R of the means' magnitudes (+ 3 u for
         the terms of e1); rms_norm: its r is computed, so er of all of it
  dw     a chain over the rows of a CTA (at most one in 64 of them), at most 320 partial sums, 3 u per term
and each output adds half a step of its own type."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
R = 44 * U
BF, F32 = torch.bfloat16, torch.float32
EPS = 1e-5


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_ffn_rms_gb300 as M
    M.check_device()
    M.device_status()
    return M


def make(T, H, x=BF, dy=BF, w=BF, bias=True, res=True, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 17 * T + H)

    def rn(*s, std=1.0, mean=0.0, dtype=BF):
        return torch.randn(s, generator=g, device=DEV).mul_(std).add_(mean).to(dtype)

    return dict(T=T, H=H, x=(rn(T, H, dtype=F32) * rn(H, std=0.6, dtype=F32).exp() + rn(T, 1, mean=2.0, dtype=F32)).to(x),
                dy=rn(T, H, std=0.1, dtype=dy), w=rn(H, std=0.2, mean=1.0, dtype=w),
                b=rn(H, std=0.2, dtype=w) if bias else None, res=rn(T, H, std=0.1, dtype=x) if res else None)


def step(t, v):
    return v * (torch.finfo(t).eps / 2)


def stats(x):
    m = x.mean(1, keepdim=True)
    v = x - m
    var = v.square().mean(1, keepdim=True)
    return m, v, var, 1 / (var + EPS).sqrt()


SHAPES = [(1, 8), (2, 16), (3, 24), (1, 4096), (5, 264), (33, 2944), (257, 256), (64, 2056), (300, 5120),
          (90, 7168), (4, 8200), (7, 16384), (1000, 1024), (700, 40)]
TYPES = [(BF, BF, BF), (F32, BF, F32), (BF, F32, BF), (F32, F32, F32)]


@pytest.mark.parametrize("x,y,w", TYPES)
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(M, T, H, x, y, w):
    for bias in (True, False):
        d = make(T, H, x, y, w, bias)
        out = torch.full((T, H), float("nan"), device=DEV, dtype=y)
        mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
        M.moe_layernorm(d["x"], d["w"], EPS, out, b=d["b"], mean=mean, rstd=rstd)
        xd, wd = d["x"].double(), d["w"].double()
        m, v, var, r = stats(xd)
        em = R * xd.abs().mean(1, keepdim=True)
        er = 0.5 * (R + 4 * U + em * em / (var + EPS)) + 2 * U
        ref = v * r * wd + (0 if d["b"] is None else d["b"].double())
        tol = (v * r * wd).abs() * (er + 3 * U) + em * r * wd.abs() + U * ref.abs()
        tol = tol + step(y, ref.abs() + tol)
        assert ((out.double() - ref).abs() <= tol).all()
        assert ((mean.double() - m[:, 0]).abs() <= em[:, 0] + U * m[:, 0].abs()).all()
        assert ((rstd.double() - r[:, 0]).abs() <= ((er + U) * r)[:, 0]).all()
        again = torch.empty_like(out)
        M.moe_layernorm(d["x"], d["w"], EPS, again, b=d["b"])
        assert torch.equal(again, out)
        if x == y:  # in place
            M.moe_layernorm(d["x"], d["w"], EPS, d["x"], b=d["b"])
            assert torch.equal(d["x"], out)


def reference(d, rms):
    """dx, dw, db in 64 bits and what fp32 arithmetic may leave in each; the statistics in fp32."""
    x, dy, w = d["x"].double(), d["dy"].double(), d["w"].double()
    T, H = d["T"], d["H"]
    if rms:
        r = 1 / (x.square().mean(1, keepdim=True) + EPS).sqrt()
        mean = rstd = None
        xh, er = x * r, 0.5 * (R + 4 * U) + 2 * U
    else:
        m, _, _, r = stats(x)
        mean, rstd = m[:, 0].float(), r[:, 0].float()
        r = rstd.double()[:, None]
        xh, er = (x - mean.double()[:, None]) * r, 0.0
    g = dy * w
    c0 = torch.zeros_like(r) if rms else g.mean(1, keepdim=True)
    c1 = (g * xh).mean(1, keepdim=True)
    core = g - c0 - xh * c1
    dx = r * core
    e0 = 0.0 if rms else (R + U) * g.abs().mean(1, keepdim=True)
    e1 = (R + (3 + 2) * U + er) * (g * xh).abs().mean(1, keepdim=True)
    tol = r * (3 * U * (g.abs() + c0.abs() + (xh * c1).abs()) + e0 + xh.abs() * e1 + er * (xh * c1).abs())
    tol = tol + (er + 2 * U) * dx.abs()
    if d["res"] is not None:
        dx = dx + d["res"].double()
        tol = tol + U * dx.abs()
    tol = tol + step(d["x"].dtype, dx.abs() + tol)
    n = (T + 63) // 64 + min(T, 320) + 3
    dw, db = (dy * xh).sum(0), dy.sum(0)
    tw = (n * U + er) * (dy * xh).abs().sum(0) + U * dw.abs()
    tb = n * U * dy.abs().sum(0) + U * db.abs()
    return mean, rstd, (dx, tol), (dw, tw), (db, tb)


def grads(M, d, rms, mean, rstd, dx=None, ws=None, stream=None, db=True):
    T, H = d["T"], d["H"]
    dx = torch.full_like(d["x"], float("nan")) if dx is None else dx
    dw = torch.full((H,), float("nan"), device=DEV)
    if ws is None:
        ws = M.alloc_workspace(M.moe_norm_backward_workspace_size(T, H))
        ws.fill_(255)  # NaN patterns: nothing in it has to be initialised
    if rms:
        M.moe_rmsnorm_backward(d["dy"], d["x"], d["w"], EPS, dx, dw, ws, dres=d["res"], stream=stream)
        return dx, dw, None
    db = torch.full((H,), float("nan"), device=DEV) if db else None
    M.moe_layernorm_backward(d["dy"], d["x"], d["w"], mean, rstd, dx, dw, ws, db=db, dres=d["res"], stream=stream)
    return dx, dw, db


def near(got, want):
    return ((got.double() - want[0]).abs() <= want[1]).all()


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("x,dy,w", TYPES)
@pytest.mark.parametrize("T,H", SHAPES)
def test_backward(M, T, H, x, dy, w, rms):
    for res in (True, False):
        d = make(T, H, x, dy, w, res=res)
        mean, rstd, rx, rw, rb = reference(d, rms)
        dx, dw, db = grads(M, d, rms, mean, rstd)
        assert near(dx, rx) and near(dw, rw)
        if not rms:
            assert near(db, rb)
            _, dw2, _ = grads(M, d, rms, mean, rstd, db=False)
            assert torch.equal(dw2, dw)
        # dx over dres, over dy, over x: each alone
        if res:
            e = dict(d, res=d["res"].clone())
            assert torch.equal(grads(M, e, rms, mean, rstd, dx=e["res"])[0], dx)
        if x == dy:
            e = dict(d, dy=d["dy"].clone())
            got = grads(M, e, rms, mean, rstd, dx=e["dy"])
            assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
        e = dict(d, x=d["x"].clone())
        got = grads(M, e, rms, mean, rstd, dx=e["x"])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    assert M.device_status() == 0


@pytest.mark.parametrize("T,H", [(5000, 512), (16384, 256), (3001, 4096)])
def test_many_rows(M, T, H):
    for rms in (False, True):
        d = make(T, H)
        mean, rstd, rx, rw, rb = reference(d, rms)
        dx, dw, db = grads(M, d, rms, mean, rstd)
        assert near(dx, rx) and near(dw, rw) and (rms or near(db, rb))


@pytest.mark.parametrize("rms", [False, True])
def test_backward_against_differences(M, rms):
    T, H = 6, 48
    d = make(T, H, F32, F32, F32, res=False)
    mean, rstd, *_ = reference(d, rms)
    dx, dw, db = grads(M, d, rms, mean, rstd)
    g = torch.Generator(device=DEV).manual_seed(3)

    def loss(x, w, b):
        if rms:
            y = x / (x.square().mean(1, keepdim=True) + EPS).sqrt() * w
        else:
            _, v, _, r = stats(x)
            y = v * r * w + b
        return (y * d["dy"].double()).sum()

    x, w, b = (d[n].double() for n in ("x", "w", "b"))
    vx, vw, vb = (torch.randn(t.shape, generator=g, device=DEV, dtype=torch.float64) for t in (x, w, b))
    h = 1e-4
    num = (loss(x + h * vx, w + h * vw, b + h * vb) - loss(x - h * vx, w - h * vw, b - h * vb)) / (2 * h)
    parts = [(dx.double() * vx), (dw.double() * vw)] + ([] if rms else [(db.double() * vb)])
    ana, size = sum(p.sum() for p in parts), sum(p.abs().sum() for p in parts)
    # fp32 results, and the difference's own h^2 times third derivatives (rows of unit size and more: below 10)
    assert abs(num - ana) <= (200 * U + 10 * h * h) * size


def test_rows_without_spread_and_special_values(M):
    """Rows of one value (variance 0), of zeros, of large offsets; a NaN or an infinity stays in its row."""
    H = 512
    x = torch.zeros((6, H), device=DEV)
    x[1] = 3.0
    x[2] = 1e4 + torch.arange(H, device=DEV) / H
    x[3] = torch.arange(H, device=DEV)
    x[4, 7] = float("nan")
    x[5, 9] = float("inf")
    w, b = torch.ones(H, device=DEV), torch.full((H,), 0.25, device=DEV)
    y, mean, rstd = torch.empty_like(x), torch.empty(6, device=DEV), torch.empty(6, device=DEV)
    M.moe_layernorm(x, w, EPS, y, b=b, mean=mean, rstd=rstd)
    assert (y[:2] == 0.25).all()
    m, v, var, r = stats(x[:4].double())
    em = R * x[:4].double().abs().mean(1, keepdim=True)
    tol = (v * r).abs() * (R + 6 * U + em * em / (var + EPS)) + em * r + 2 * U
    assert ((y[:4].double() - v * r - 0.25).abs() <= tol).all()
    assert torch.isnan(y[4:]).all()
    # eps = 0 with rows that have a spread
    M.moe_layernorm(x[2:4].contiguous(), w, 0.0, y[:2])
    assert torch.isfinite(y[:2]).all()
    dy = torch.ones_like(x)
    dx, dw, db, ws = torch.empty_like(x), torch.empty(H, device=DEV), torch.empty(H, device=DEV), M.alloc_workspace(
        M.moe_norm_backward_workspace_size(6, H))
    M.moe_layernorm_backward(dy, x, w, mean, rstd, dx, dw, ws, db=db)
    assert torch.isfinite(dx[:4]).all() and (db == 6).all()


def test_streams_graphs_shared_workspace_and_empty_batches(M):
    T, H = 500, 2944
    d = make(T, H)
    mean, rstd, *_ = reference(d, False)
    ref = grads(M, d, False, mean, rstd)
    ws = M.alloc_workspace(M.moe_norm_backward_workspace_size(T, H))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    outs = []
    with torch.cuda.stream(s):
        graphs = []
        for _ in range(2):  # two graphs with one workspace, replayed one after the other
            dx, dw, db = torch.empty_like(d["x"]), torch.empty(H, device=DEV), torch.empty(H, device=DEV)
            M.moe_layernorm_backward(d["dy"], d["x"], d["w"], mean, rstd, dx, dw, ws, db=db, dres=d["res"])
            s.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=s):
                M.moe_layernorm_backward(d["dy"], d["x"], d["w"], mean, rstd, dx, dw, ws, db=db, dres=d["res"])
            for t in (dx, dw, db):
                t.zero_()
            graphs.append(g)
            outs.append((dx, dw, db))
        for g in graphs * 2:
            g.replay()
    torch.cuda.synchronize()
    for o in outs:
        assert all(torch.equal(a, b) for a, b in zip(o, ref))
    e = torch.empty((0, H), device=DEV, dtype=BF)
    none = torch.empty(0, device=DEV)
    M.moe_layernorm(e, d["w"], EPS, e.clone())
    dw, db = torch.full((H,), 7.0, device=DEV), torch.full((H,), 7.0, device=DEV)
    M.moe_layernorm_backward(e, e, d["w"], none, none, e.clone(), dw, ws, db=db)
    assert (dw == 0).all() and (db == 0).all()
    dw.fill_(7.0)
    M.moe_rmsnorm_backward(e, e, d["w"], EPS, e.clone(), dw, ws)
    assert (dw == 0).all()


def test_rows_beyond_32_bit_offsets(M):
    T, H = 140000, 16384
    x = torch.empty((T, H), device=DEV, dtype=BF)
    x[:] = torch.arange(H, device=DEV).remainder(7).to(BF)
    y = torch.empty_like(x)
    w = torch.ones(H, device=DEV, dtype=BF)
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    M.moe_layernorm(x, w, EPS, y, mean=mean, rstd=rstd)
    assert torch.equal(y, y[:1].expand(T, -1)) and (mean == mean[0]).all()
    dx, dw = torch.empty_like(x), torch.empty(H, device=DEV)
    M.moe_rmsnorm_backward(y, x, w, EPS, dx, dw, M.alloc_workspace(M.moe_norm_backward_workspace_size(T, H)))
    assert torch.equal(dx, dx[:1].expand(T, -1)) and torch.isfinite(dw).all()
