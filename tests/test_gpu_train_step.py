"""A training step of a block from the operators together: layer norm, router, sort by expert, a linear layer with an
activation per expert, weighted return with residual, then every gradient back to the inputs, against
torch.autograd in 64 bits.

Tolerance: each tensor between two operators is rounded to bf16 (half a step: 2^-8 of its magnitude), and no path from
an input to a result has more than eight of them (x_hat, kept values, y, out; dy, dpre, dxp, dx_hat); fp32 sums are far
below.  The roundings are independent of the values' signs, so the norm of a result's error is at most 8 x 2^-8 of the
norm of the result."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF = torch.bfloat16
TOL = 8 * 2.0 ** -8


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_ffn_rms_gb300 as M
    M.check_device()
    M.device_status()
    return M


class Block:
    def __init__(self, M, T, H, E, k, norm, drop, seed=0):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def rn(*s, std=1.0, mean=0.0, dtype=BF):
            return torch.randn(s, generator=g, device=DEV).mul_(std).add_(mean).to(dtype)

        self.M, self.T, self.H, self.E, self.k, self.norm = M, T, H, E, k, norm
        self.x, self.g = rn(T, H, mean=0.5), rn(T, H, std=0.1)
        self.w, self.b = rn(H, std=0.1, mean=1.0), rn(H, std=0.1)
        self.wr = rn(H, E, std=H ** -0.5, dtype=torch.float32)
        self.we, self.be = rn(E, H, H, std=H ** -0.5), rn(E, H, std=0.2)
        self.keep = torch.rand((T * k,), generator=g, device=DEV) >= drop
        e = lambda *s, dtype=torch.float32: torch.empty(s, device=DEV, dtype=dtype)  # noqa: E731
        self.mean, self.rstd = e(T), e(T)
        self.xhat, self.out, self.dxhat, self.dx = (e(T, H, dtype=BF) for _ in range(4))
        self.ids, self.tw = e(T, k, dtype=torch.int32), e(T, k)
        self.off, self.src, self.row = e(E + 1, dtype=torch.int32), e(T * k, dtype=torch.int32), e(T * k, dtype=torch.int32)
        self.xp, self.pre, self.y, self.dy, self.dxp = (torch.zeros((T * k, H), device=DEV, dtype=BF) for _ in range(5))
        self.dtw, self.dl = e(T, k), e(T, E)
        self.dw, self.db, self.dwe, self.dbe = e(H), e(H), e(E, H, H), e(E, H)
        self.dwr = e(H, E)
        self.ws_route = M.alloc_workspace(max(256, M.moe_route_workspace_size(T, H, E)))
        self.ws_perm = M.alloc_workspace(max(256, M.moe_permute_workspace_size(T, E, k)))
        self.ws_norm = M.alloc_workspace(M.moe_norm_backward_workspace_size(T, H))
        self.ws_lin = M.alloc_workspace(M.moe_linear_backward_workspace_size(T * k, H, H))

    def route(self):
        M = self.M
        if self.norm == "layer":
            M.moe_layernorm(self.x, self.w, 1e-5, self.xhat, b=self.b, mean=self.mean, rstd=self.rstd)
        else:
            M.moe_rmsnorm(self.x, self.w, 1e-5, self.xhat)
        M.moe_route_topk(self.T, self.H, self.E, self.k, self.ids, self.tw, xhat=self.xhat, router_w=self.wr,
                         workspace=self.ws_route)
        M.moe_permute(self.ids, self.T, self.E, self.k, self.off, self.src, self.row, xhat=self.xhat, xp=self.xp,
                      row_bytes=2 * self.H, workspace=self.ws_perm)

    def step(self, off):
        """The step behind the routing; off: the experts' segments on the host."""
        M, T, k, E = self.M, self.T, self.k, self.E
        self.row.copy_(torch.where(self.keep, self.row, torch.full_like(self.row, -1)))
        seg = [slice(off[e], off[e + 1]) for e in range(E)]
        for e in range(E):
            M.moe_linear(self.xp[seg[e]], self.we[e], self.y[seg[e]], bias=self.be[e], act=M.ACT_SILU,
                         pre=self.pre[seg[e]])
        M.moe_unpermute(self.y, self.row, self.out, T, k, topk_w=self.tw, residual=self.x)
        # backward: the loss is <out, g>; rows of dropped pairs have no gradient
        self.dy.zero_()
        M.moe_unpermute_backward(self.g, self.y, self.row, self.tw, T, k, dy=self.dy, dw=self.dtw, ids=self.ids,
                                 dlogits=self.dl)
        for e in range(E):
            M.moe_linear_backward(self.dy[seg[e]], self.xp[seg[e]], self.we[e], self.ws_lin, dx=self.dxp[seg[e]],
                                  dw=self.dwe[e], db=self.dbe[e], pre=self.pre[seg[e]], act=M.ACT_SILU)
        router = (self.dl @ self.wr.t()).to(BF)
        M.moe_permute_backward(self.dxp, self.row, self.dxhat, T, k, dres=router)
        torch.matmul(self.xhat.float().t(), self.dl, out=self.dwr)
        if self.norm == "layer":
            M.moe_layernorm_backward(self.dxhat, self.x, self.w, self.mean, self.rstd, self.dx, self.dw, self.ws_norm,
                                     db=self.db, dres=self.g)
        else:
            M.moe_rmsnorm_backward(self.dxhat, self.x, self.w, 1e-5, self.dx, self.dw, self.ws_norm, dres=self.g)

    def results(self):
        r = {n: getattr(self, n) for n in ("out", "dx", "dw", "dwe", "dbe", "dwr")}
        return r if self.norm == "rms" else dict(r, db=self.db)

    def reference(self):
        d = lambda t: t.double().detach().requires_grad_()  # noqa: E731
        x, w, b, wr, we, be = d(self.x), d(self.w), d(self.b), d(self.wr), d(self.we), d(self.be)
        if self.norm == "layer":
            h = torch.nn.functional.layer_norm(x, (self.H,), w, b, 1e-5)
        else:
            h = x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5) * w
        ids = self.ids.long()
        tw = torch.softmax((h @ wr).gather(1, ids), 1)
        z = torch.einsum("th,tkoh->tko", h, we[ids]) + be[ids]
        y = torch.nn.functional.silu(z) * self.keep.view(self.T, self.k, 1).double()
        out = x + (tw[:, :, None] * y).sum(1)
        leaves = {"dx": x, "dw": w, "dwe": we, "dbe": be, "dwr": wr}
        if self.norm == "layer":
            leaves["db"] = b
        grads = torch.autograd.grad((out * self.g.double()).sum(), list(leaves.values()))
        return dict(zip(leaves, grads), out=out.detach())


@pytest.mark.parametrize("norm,T,H,E,k,drop", [("layer", 37, 256, 5, 2, 0.0), ("rms", 130, 576, 8, 3, 0.2),
                                               ("layer", 600, 320, 4, 4, 0.1), ("rms", 1, 64, 3, 1, 0.0)])
def test_training_step(M, norm, T, H, E, k, drop):
    b = Block(M, T, H, E, k, norm, drop)
    b.route()
    off = b.off.tolist()
    b.step(off)
    assert M.device_status() == 0
    ref, got = b.reference(), b.results()
    for n, r in ref.items():
        err, size = (got[n].double() - r).norm(), r.norm()
        assert err <= TOL * size, (n, float(err / size))


def test_training_step_captured(M):
    """The step in a graph, replayed on other inputs, has the bits of the eager step."""
    b = Block(M, 96, 256, 4, 2, "layer", 0.1)
    b.route()
    off = b.off.tolist()
    kept = b.row.clone()
    b.step(off)
    want = {n: t.clone() for n, t in b.results().items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.row.copy_(kept)
        b.step(off)
        s.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            b.step(off)
        b.row.copy_(kept)
        for t in b.results().values():
            t.zero_()
        g.replay()
        s.synchronize()
        for n, t in b.results().items():
            assert torch.equal(t, want[n]), n
        b.g.mul_(2)  # a power of two: every gradient doubles exactly
        b.row.copy_(kept)
        g.replay()
        s.synchronize()
        for n in ("dx", "dwe", "dwr", "dw"):
            assert torch.equal(b.results()[n], 2 * want[n]), n
    assert M.device_status() == 0
