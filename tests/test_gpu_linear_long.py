"""Long sums with bf16 results: a bf16 output of moe_linear, and dx and dW in bf16, over up to 2^23 terms.

All terms are positive, so that what the tensor cores cut off adds up.  With spread, rows and columns have scales of their
own, so that the results lie anywhere between two steps of bf16; without, all results of 2^20 terms lie within half a percent
of one value, less than a step, and are rounded to the same one or two: their roundings are no independent ones, and
only the bound on every value says something.  An addition of 16 products truncates at most 2^-23 of the running
sum, 16384 terms are added so at most, and the sums of those (or of 4096 terms, in longer parts) are rounded to nearest:
  every value  2^-23 (16384 / 16 + 4) of the sum, 2^-24 for each of 2^20 / 4096 = 256 sums (2^23 terms are 2048 of
               them in one pair of CTAs: rounded to nearest, they come to much less than 256 in one direction), and half a step
  their mean   6.1e-9 a term, measured for the truncation of one sign (1e-4 at 16384), and that of N roundings, each
               within 2^-8 and independent of the others: six standard deviations, 6 * 2^-8 / sqrt(3 N)"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


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
    if request.param != "auto":
        monkeypatch.setenv("MOE_LINEAR_FORM", request.param)
    return request.param


def positive(seed, *shape, scaled=None):
    """|normal| values, each row (scaled = 0) or column (1) with a scale of its own between 1 and 4."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    t = torch.randn(shape, generator=g, device=DEV).abs_()
    if scaled is not None:
        s = (2 * torch.rand(shape[scaled], generator=g, device=DEV)).exp2_()
        t.mul_(s[:, None] if scaled == 0 else s)
    return t.to(BF)


def product64(a, b):
    """a^T b over the rows, in 64 bits, a part of the rows at a time."""
    out = torch.zeros((a.shape[1], b.shape[1]), device=DEV, dtype=torch.float64)
    for i in range(0, a.shape[0], 1 << 18):
        out += a[i:i + (1 << 18)].double().t() @ b[i:i + (1 << 18)].double()
    return out


def close(got, ref, spread):
    err = got.double() - ref
    tol = (2.0 ** -23 * (16384 / 16 + 4) + 2.0 ** -24 * 256) * ref
    tol = tol + (ref + tol) * (torch.finfo(got.dtype).eps / 2)
    assert (err.abs() <= tol).all(), float((err / ref).abs().max())
    if not spread:
        return
    bias = float((err / ref).mean())
    assert abs(bias) <= 1e-4 + 6 * 2.0 ** -8 / math.sqrt(3 * err.numel()), bias


@pytest.mark.parametrize("spread", [True, False])
@pytest.mark.parametrize("m,n,k", [(1 << 20, 264, 520), (1 << 23, 64, 72), ((1 << 20) + 77, 2056, 1288),
                                   (16384, 264, 520), (16385, 2056, 2312)])
def test_weight_gradient(M, m, n, k, form, spread):
    by = 1 if spread else None
    x, d, w = positive(1, m, k, scaled=by), positive(2, m, n, scaled=by), positive(3, n, k)
    dw = torch.full((n, k), float("nan"), device=DEV, dtype=BF)
    M.moe_linear_backward(d, x, w, M.alloc_workspace(M.moe_linear_backward_workspace_size(m, n, k)), dw=dw)
    close(dw, product64(d, x), spread)
    assert M.device_status() == 0


@pytest.mark.parametrize("spread", [True, False])
@pytest.mark.parametrize("m,n,k", [(300, 520, 1 << 20), (1, 136, 1 << 20), (7, 40, 1 << 20), (2048, 2312, 69640)])
def test_forward(M, m, n, k, form, spread):
    x, w = positive(4, m, k, scaled=0 if spread else None), positive(5, n, k, scaled=0 if spread else None)
    out = torch.full((m, n), float("nan"), device=DEV, dtype=BF)
    M.moe_linear(x, w, out)
    ref = product64(x.t().contiguous(), w.t().contiguous())
    close(out, ref, spread)
    # the epilogue behind it: bias, activation, the values before it, residual
    b, r = positive(6, n), positive(7, m, n, scaled=0 if spread else None)
    pre, o = torch.full_like(out, float("nan")), r.clone()
    M.moe_linear(x, w, o, bias=b, residual=o, act=M.ACT_SILU, pre=pre)
    z = ref + b.double()
    close(pre, z, spread)
    # silu of more than 60 is its argument (exp(-60) is less than 2^-80 of it)
    assert float(z.min()) > 60
    close(o, z + r.double(), spread)
    assert M.device_status() == 0


@pytest.mark.parametrize("spread", [True, False])
@pytest.mark.parametrize("m,n,k", [(300, 1 << 20, 264), (33, 1 << 20, 72), (2048, 69640, 2312)])
def test_input_gradient(M, m, n, k, form, spread):
    d, w, x = positive(8, m, n, scaled=0 if spread else None), positive(9, n, k, scaled=1 if spread else None), positive(10, m, k)
    dx = torch.full((m, k), float("nan"), device=DEV, dtype=BF)
    M.moe_linear_backward(d, x, w, M.alloc_workspace(M.moe_linear_backward_workspace_size(m, n, k)), dx=dx)
    close(dx, product64(d.t().contiguous(), w), spread)
    assert M.device_status() == 0
