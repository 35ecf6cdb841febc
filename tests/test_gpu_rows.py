"""moe_unpermute, moe_unpermute_backward and moe_permute_backward on the GPU against their formulas in 64
bits.

The tolerances count roundings, u = 2^-24 (half a step of fp32):
  out      one fma per expert row: (k + 1) u (|residual| + sum |w y|)
  dy       one product
  dw       H products added by at most 128 in a chain per thread, 5 steps within a warp, at most 32 over
           the warps: 168 u sum |dout y|
  dlogits  s = sum w dw over k terms, then a difference and a product: w (e_dw + sum w e_dw) and
           (k + 3) u w (|dw| + sum |w dw|)
and each output adds half a step of its own type."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
U = 2.0 ** -24
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_ffn_rms_gb300 as M
    M.check_device()
    M.device_status()
    return M


def randn(g, *shape, std=1.0, dtype=BF):
    return torch.randn(shape, generator=g, device=DEV).mul_(std).to(dtype)


def make(T, H, k, E=16, y=BF, stream=BF, res=True, drop=0.0, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + 31 * T + H)
    d = dict(T=T, H=H, k=k, E=E)
    d["ids"] = torch.rand((T, E), generator=g, device=DEV).argsort(1)[:, :k].to(torch.int32).contiguous()
    w = torch.rand((T, k), generator=g, device=DEV) + 0.05
    d["w"] = (w / w.sum(1, keepdim=True)).contiguous()
    row = torch.randperm(T * k, generator=g, device=DEV).to(torch.int32)
    if drop:
        row[torch.rand((T * k,), generator=g, device=DEV) < drop] = -1
        row[:k] = -1  # a token of which nothing is left
    d["row"] = row
    d["y"] = randn(g, T * k, H, std=0.3, dtype=y)
    d["res"] = randn(g, T, H, std=2.0, dtype=stream) if res else None
    d["dout"] = randn(g, T, H, std=0.05, dtype=stream)
    # rows without a pair are never looked at
    free = torch.ones(T * k, dtype=torch.bool, device=DEV)
    free[row[row >= 0].long()] = False
    d["y"][free] = float("nan")
    d["free"] = free
    return d


def step(t, v):
    """Half a step of type t at magnitude v."""
    return v * (torch.finfo(t).eps / 2)


def gathered(d):
    live = d["row"] >= 0
    y = d["y"].double()[d["row"].long().clamp(min=0)]
    return torch.where(live[:, None], y, torch.zeros_like(y)).view(d["T"], d["k"], d["H"]), live.view(d["T"], d["k"])


def check_sum(d, out, w):
    y, _ = gathered(d)
    y = y if w is None else y * w.double()[:, :, None]
    res = d["res"].double() if d["res"] is not None else torch.zeros((), device=DEV, dtype=torch.float64)
    ref = res + y.sum(1)
    tol = (d["k"] + 1) * U * (res.abs() + y.abs().sum(1))
    tol = tol + step(out.dtype, ref.abs() + tol)
    assert ((out.double() - ref).abs() <= tol).all()


SHAPES = [(1, 8, 1), (1, 4096, 8), (3, 24, 2), (7, 264, 3), (33, 2944, 6), (257, 256, 8), (65, 2056, 5),
          (130, 7168, 4), (5, 32768, 8), (1000, 512, 7), (900, 264, 3), (640, 96, 8)]
TYPES = [(BF, BF), (BF, F32), (F32, BF), (F32, F32)]


@pytest.mark.parametrize("y,stream", TYPES)
@pytest.mark.parametrize("T,H,k", SHAPES)
def test_return_and_gather_gradient(M, T, H, k, y, stream):
    for drop, res in ((0.0, True), (0.3, False), (0.3, True)):
        d = make(T, H, k, y=y, stream=stream, res=res, drop=drop)
        out = torch.full((T, H), float("nan"), device=DEV, dtype=stream)
        M.moe_unpermute(d["y"], d["row"], out, T, k, topk_w=d["w"], residual=d["res"])
        check_sum(d, out, d["w"])
        out.fill_(float("nan"))
        M.moe_permute_backward(d["y"], d["row"], out, T, k, dres=d["res"])
        check_sum(d, out, None)
        if res:  # in place over the residual
            M.moe_unpermute(d["y"], d["row"], d["res"], T, k, topk_w=d["w"], residual=d["res"])
            ref = torch.empty_like(out)
            d2 = make(T, H, k, y=y, stream=stream, res=res, drop=drop)
            M.moe_unpermute(d2["y"], d2["row"], ref, T, k, topk_w=d2["w"], residual=d2["res"])
            assert torch.equal(d["res"], ref)
    assert M.device_status() == 0


def check_grad(d, dy, dw, dlogits, before):
    T, k, H = d["T"], d["k"], d["H"]
    y, live = gathered(d)
    do, w = d["dout"].double(), d["w"].double()
    if dy is not None:
        ref = (w[:, :, None] * do[:, None]).view(T * k, H)
        got = dy.double()[d["row"].long().clamp(min=0)]
        tol = U * ref.abs()
        tol = tol + step(dy.dtype, ref.abs() + tol)
        ok = (got - ref).abs() <= tol
        assert ok[live.view(-1)].all()
        assert torch.equal(dy[d["free"]].view(torch.int8), before[d["free"]].view(torch.int8))
    rw = (do[:, None] * y).sum(2)
    ew = 168 * U * (do[:, None] * y).abs().sum(2)
    if dw is not None:
        assert ((dw.double() - rw).abs() <= ew + U * rw.abs()).all()
        assert (dw[~live] == 0).all()
    if dlogits is not None:
        s = (w * rw).sum(1, keepdim=True)
        es = (w * ew).sum(1, keepdim=True)
        v = w * (rw - s)
        tol = w * (ew + es) + (k + 3) * U * w * (rw.abs() + (w * rw).abs().sum(1, keepdim=True))
        at = d["ids"].long()
        ref = torch.zeros((T, d["E"]), dtype=torch.float64, device=DEV).scatter_(1, at, v)
        tol = torch.zeros_like(ref).scatter_(1, at, tol)
        assert ((dlogits.double() - ref).abs() <= tol).all()


@pytest.mark.parametrize("y,stream", TYPES)
@pytest.mark.parametrize("T,H,k", SHAPES)
def test_return_gradient(M, T, H, k, y, stream):
    for drop, E in ((0.0, 256), (0.3, 8)):
        d = make(T, H, k, E=E, y=y, stream=stream, drop=drop)
        dy = torch.full_like(d["y"], float("nan"))
        before = dy.clone()
        dw = torch.full((T, k), float("nan"), device=DEV)
        dl = torch.full((T, E), float("nan"), device=DEV)
        M.moe_unpermute_backward(d["dout"], d["y"], d["row"], d["w"], T, k, dy=dy, dw=dw, ids=d["ids"], dlogits=dl)
        check_grad(d, dy, dw, dl, before)
        # each output by itself has the same bits
        one = torch.full_like(dy, float("nan"))
        M.moe_unpermute_backward(d["dout"], None, d["row"], d["w"], T, k, dy=one)
        assert torch.equal(one.view(torch.int8), dy.view(torch.int8))
        two, three = torch.empty_like(dw), torch.empty_like(dl)
        M.moe_unpermute_backward(d["dout"], d["y"], d["row"], d["w"], T, k, dw=two)
        M.moe_unpermute_backward(d["dout"], d["y"], d["row"], d["w"], T, k, ids=d["ids"], dlogits=three)
        assert torch.equal(two, dw) and torch.equal(three, dl)
        # dy over y
        M.moe_unpermute_backward(d["dout"], d["y"], d["row"], d["w"], T, k, dy=d["y"], dw=two)
        assert torch.equal(two, dw)
        keep = ~d["free"]
        assert torch.equal(d["y"][keep], dy[keep])
    assert M.device_status() == 0


def test_return_gradient_against_differences(M):
    """<gradients, direction> against central differences of the forward in 64 bits."""
    T, H, k, E = 9, 64, 4, 12
    d = make(T, H, k, E=E, y=F32, stream=F32, drop=0.2)
    g = torch.Generator(device=DEV).manual_seed(5)
    z = torch.randn((T, E), generator=g, device=DEV, dtype=torch.float64)
    at = d["ids"].long()
    d["w"] = torch.softmax(z.gather(1, at), 1).float()
    dy, dw, dl = torch.zeros_like(d["y"]), torch.empty((T, k), device=DEV), torch.empty((T, E), device=DEV)
    M.moe_unpermute_backward(d["dout"], d["y"], d["row"], d["w"], T, k, dy=dy, dw=dw, ids=d["ids"], dlogits=dl)
    y, live = gathered(d)

    def loss(y, z):
        w = torch.softmax(z.gather(1, at), 1)
        return ((y * w[:, :, None]).sum(1) * d["dout"].double()).sum()

    vy = torch.randn(y.shape, generator=g, device=DEV, dtype=torch.float64) * live[:, :, None]
    vz = torch.randn(z.shape, generator=g, device=DEV, dtype=torch.float64)
    h = 1e-4
    num = (loss(y + h * vy, z + h * vz) - loss(y - h * vy, z - h * vz)) / (2 * h)
    gy = dy.double()[d["row"].long().clamp(min=0)].view(T, k, H)
    ana = (gy * vy).sum() + (dl.double() * vz).sum()
    scale = (gy * vy).abs().sum() + (dl.double() * vz).abs().sum()
    # fp32 results (200 u) and the difference's own error (h^2 times third derivatives of a softmax, below 1)
    assert abs(num - ana) <= (200 * U + h * h) * scale


def test_rows_out_of_range_are_flagged_and_left_out(M):
    T, H, k = 4, 256, 2
    d = make(T, H, k)
    bad = d["row"].clone()
    bad[3] = T * k
    bad[5] = 2 ** 31 - 1
    good = d["row"].clone()
    good[3] = good[5] = -1
    out, ref = torch.empty((T, H), device=DEV, dtype=BF), torch.empty((T, H), device=DEV, dtype=BF)
    M.device_status()
    M.moe_unpermute(d["y"], bad, out, T, k, topk_w=d["w"])
    assert M.device_status() == 1
    M.moe_unpermute(d["y"], good, ref, T, k, topk_w=d["w"])
    assert M.device_status() == 0 and torch.equal(out, ref)
    dw, dl = torch.empty((T, k), device=DEV), torch.empty((T, 16), device=DEV)
    ids = d["ids"].clone()
    ids[0, 0], ids[1, 1] = -1, 16
    M.moe_unpermute_backward(d["dout"], d["y"], good, d["w"], T, k, dw=dw, ids=ids, dlogits=dl)
    assert M.device_status() == 1
    assert torch.isfinite(dl).all() and int((dl[0] != 0).sum()) <= 1
    # an expert given twice for a token counts with both
    ids = d["ids"].clone()
    ids[2, 1] = ids[2, 0]
    M.moe_unpermute_backward(d["dout"], d["y"], good, d["w"], T, k, dw=dw, ids=ids, dlogits=dl)
    s = (d["w"][2] * dw[2]).sum()
    v = (d["w"][2] * (dw[2] - s)).sum()
    assert abs(dl[2, ids[2, 0].long()] - v) <= 8 * U * (d["w"][2] * (dw[2].abs() + s.abs())).sum()
    assert M.device_status() == 0


def test_offsets_beyond_32_bits(M):
    """Rows whose byte and element offsets do not fit 32 bits."""
    T, H, k = 33000, 8192, 8
    row = torch.arange(T * k - 1, -1, -1, device=DEV, dtype=torch.int32)
    y = torch.empty((T * k, H), device=DEV, dtype=BF)
    y.copy_((torch.arange(T * k, device=DEV) % 251).to(BF)[:, None].expand(-1, H))
    out = torch.empty((T, H), device=DEV, dtype=BF)
    M.moe_permute_backward(y, row, out, T, k)
    ref = y[:, 0].float().flip(0).view(T, k).sum(1).to(BF)
    assert torch.equal(out, ref[:, None].expand(-1, H))
    w = torch.ones((T, k), device=DEV)
    dy = torch.zeros_like(y)
    M.moe_unpermute_backward(out, None, row, w, T, k, dy=dy)
    assert torch.equal(dy.view(T, k, H).flip(0), out[:, None].expand(-1, k, -1))


def test_streams_graphs_and_empty_batches(M):
    T, H, k = 96, 2944, 6
    d = make(T, H, k, drop=0.1)
    ref = torch.empty((T, H), device=DEV, dtype=BF)
    rdy, rdw = torch.zeros_like(d["y"]), torch.empty((T, k), device=DEV)

    def run(out, dy, dw, stream=None):
        M.moe_unpermute(d["y"], d["row"], out, T, k, topk_w=d["w"], residual=d["res"], stream=stream)
        M.moe_unpermute_backward(out, d["y"], d["row"], d["w"], T, k, dy=dy, dw=dw, stream=stream)
        M.moe_permute_backward(dy, d["row"], out, T, k, stream=stream)

    run(ref, rdy, rdw)
    torch.cuda.synchronize()
    bufs = [(torch.zeros_like(ref), torch.zeros_like(rdy), torch.zeros_like(rdw)) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, b in zip(streams, bufs):
        run(*b, stream=s)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        run(*bufs[2])
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            run(*bufs[2])
    for b in bufs[2]:
        b.zero_()
    torch.cuda.synchronize()
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    for out, dy, dw in bufs:
        assert torch.equal(out, ref) and torch.equal(dw, rdw)
        assert torch.equal(dy.view(torch.int16), rdy.view(torch.int16))
    e = torch.empty((0, H), device=DEV, dtype=BF)
    none = torch.empty(0, device=DEV, dtype=torch.int32)
    M.moe_unpermute(e, none, e.clone(), 0, k)
    M.moe_permute_backward(e, none, e.clone(), 0, k)
    M.moe_unpermute_backward(e, e, none, torch.empty((0, k), device=DEV), 0, k, dy=e.clone())
    with pytest.raises(ValueError):
        M.moe_unpermute(d["y"], d["row"], ref.cpu(), T, k)
    with pytest.raises(ValueError):
        M.moe_unpermute(d["y"], d["row"][:-1], ref, T, k)
