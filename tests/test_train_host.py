"""Refusals of the operators around the experts on the host: nothing is enqueued, and no CUDA call is made
before the checks."""
import pytest
import torch

FAKE = 1 << 20  # 16-byte aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_ffn_rms_gb300 as M
    return M


def refused(M, name, args, kw, code):
    n = M.lib.moe_launch_count()
    assert getattr(M.lib, name)(*dict(args, **kw).values()) == code, kw
    assert M.last_error()
    assert M.lib.moe_launch_count() == n


ROWS = [(dict(T=-1), 2), (dict(k=0), 2), (dict(k=9), 2), (dict(H=0), 2), (dict(H=252), 2), (dict(H=32776), 2),
        (dict(T=1 << 22, k=8), 2)]


@pytest.mark.parametrize("kw,code", ROWS + [
    (dict(y=None), 1), (dict(row=None), 1), (dict(out=None), 1), (dict(y=FAKE + 8), 1), (dict(row=FAKE + 2), 1),
    (dict(w=FAKE + 2), 1), (dict(res=FAKE + 4), 1), (dict(out=FAKE + 8), 1), (dict(res_f32=1), 1)])
def test_unpermute(M, kw, code):
    args = dict(y=FAKE, y_bf16=1, row=FAKE, w=FAKE, T=4, k=2, H=256, res=FAKE, res_f32=0, out=FAKE, out_f32=0, st=None)
    refused(M, "moe_unpermute", args, kw, code)
    if "w" not in kw:
        del args["w"]
        refused(M, "moe_permute_backward", args, kw, code)


@pytest.mark.parametrize("kw,code", ROWS + [
    (dict(dout=None), 1), (dict(y=None), 1), (dict(row=None), 1), (dict(w=None), 1), (dict(ids=None), 1),
    (dict(dy=None, dw=None, dl=None), 1), (dict(dout=FAKE + 8), 1), (dict(y=FAKE + 8), 1), (dict(dy=FAKE + 8), 1),
    (dict(row=FAKE + 2), 1), (dict(w=FAKE + 2), 1), (dict(ids=FAKE + 2), 1), (dict(dw=FAKE + 2), 1),
    (dict(dl=FAKE + 2), 1), (dict(E=0), 2), (dict(E=257), 2)])
def test_unpermute_backward(M, kw, code):
    args = dict(dout=FAKE, dout_f32=0, y=FAKE, y_bf16=1, row=FAKE, w=FAKE, ids=FAKE, T=4, k=2, H=256, E=8, dy=FAKE,
                dw=FAKE, dl=FAKE, st=None)
    refused(M, "moe_unpermute_backward", args, kw, code)


NORM = [(dict(T=-1), 2), (dict(H=0), 2), (dict(H=252), 2), (dict(H=16392), 2), (dict(x=None), 1), (dict(w=None), 1),
        (dict(x=FAKE + 8), 1), (dict(w=FAKE + 8), 1)]


@pytest.mark.parametrize("kw,code", NORM + [
    (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1), (dict(y=None), 1), (dict(mean=None), 1), (dict(rstd=None), 1),
    (dict(b=FAKE + 8), 1), (dict(y=FAKE + 8), 1), (dict(mean=FAKE + 2), 1), (dict(rstd=FAKE + 2), 1),
    (dict(y_f32=1), 1)])
def test_layernorm(M, kw, code):
    args = dict(x=FAKE, x_f32=0, w=FAKE, b=FAKE, w_f32=0, T=4, H=256, eps=1e-6, y=FAKE, y_f32=0, mean=FAKE, rstd=FAKE,
                st=None)
    refused(M, "moe_layernorm", args, kw, code)


GRAD = NORM + [(dict(dy=None), 1), (dict(dx=None), 1), (dict(dw=None), 1), (dict(dy=FAKE + 8), 1),
               (dict(dx=FAKE + 8), 1), (dict(dres=FAKE + 8), 1), (dict(dw=FAKE + 2), 1), (dict(ws=None), 4),
               (dict(ws=FAKE + 16), 1), (dict(wsb=100), 4), (dict(dy_f32=1), 1)]


@pytest.mark.parametrize("kw,code", GRAD + [(dict(mean=None), 1), (dict(rstd=None), 1), (dict(db=FAKE + 2), 1),
                                            (dict(mean=FAKE + 2), 1)])
def test_layernorm_backward(M, kw, code):
    args = dict(dy=FAKE, dy_f32=0, x=FAKE, x_f32=0, w=FAKE, w_f32=0, mean=FAKE, rstd=FAKE, dres=FAKE, T=4, H=256,
                dx=FAKE, dw=FAKE, db=FAKE, ws=FAKE, wsb=1 << 30, st=None)
    refused(M, "moe_layernorm_backward", args, kw, code)


@pytest.mark.parametrize("kw,code", GRAD + [(dict(eps=-1.0), 1), (dict(eps=float("nan")), 1)])
def test_rmsnorm_backward(M, kw, code):
    args = dict(dy=FAKE, dy_f32=0, x=FAKE, x_f32=0, w=FAKE, w_f32=0, eps=1e-6, dres=FAKE, T=4, H=256, dx=FAKE, dw=FAKE,
                ws=FAKE, wsb=1 << 30, st=None)
    refused(M, "moe_rmsnorm_backward", args, kw, code)


def test_norm_workspace_size(M):
    assert M.moe_norm_backward_workspace_size(0, 256) > 0
    assert M.moe_norm_backward_workspace_size(1 << 20, 16384) >= 2 * 16384 * 4
    for T, H in ((-1, 256), (4, 0), (4, 252), (4, 16392)):
        with pytest.raises(M.MoeError):
            M.moe_norm_backward_workspace_size(T, H)


def test_binding_refuses_host_tensors_and_wrong_types(M):
    bf = torch.bfloat16
    y, x, w = torch.zeros((8, 256), dtype=bf), torch.zeros((4, 256), dtype=bf), torch.ones(256, dtype=bf)
    row = torch.zeros(8, dtype=torch.int32)
    f = torch.zeros(256)
    for call in (lambda: M.moe_unpermute(y, row, x, 4, 2), lambda: M.moe_permute_backward(y, row, x, 4, 2),
                 lambda: M.moe_unpermute_backward(x, y, row, torch.zeros(4, 2), 4, 2, dy=y),
                 lambda: M.moe_layernorm(x, w, 1e-6, x),
                 lambda: M.moe_layernorm_backward(x, x, w, f[:4], f[:4], x, f, y.view(torch.uint8)),
                 lambda: M.moe_rmsnorm_backward(x, x, w, 1e-6, x, f, y.view(torch.uint8))):
        with pytest.raises(ValueError):
            call()


LINEAR = [(dict(M=-1), 2), (dict(M=(1 << 23) + 1), 2), (dict(N=0), 2), (dict(N=100), 2), (dict(K=0), 2),
          (dict(K=60), 2), (dict(K=(1 << 20) + 8), 2), (dict(act=-1), 1), (dict(act=5), 1), (dict(x=None), 1),
          (dict(w=None), 1), (dict(x=FAKE + 8), 1), (dict(w=FAKE + 8), 1), (dict(pre=FAKE + 8), 1)]


@pytest.mark.parametrize("kw,code", LINEAR + [
    (dict(out=None), 1), (dict(out=FAKE + 8), 1), (dict(bias=FAKE + 8), 1), (dict(res=FAKE + 8), 1),
    (dict(res=FAKE, res_f32=1), 1)])
def test_linear(M, kw, code):
    args = dict(x=FAKE, w=FAKE, bias=FAKE, bias_f32=0, res=FAKE, res_f32=0, M=4, N=256, K=128, act=2, pre=FAKE + 4096,
                out=FAKE, out_f32=0, st=None)
    refused(M, "moe_linear", args, kw, code)


@pytest.mark.parametrize("kw,code", LINEAR + [
    (dict(dout=None), 1), (dict(pre=None), 1), (dict(dx=None, dw=None, db=None), 1), (dict(dx=FAKE + 8), 1),
    (dict(dw=FAKE + 8), 1), (dict(db=FAKE + 2), 1), (dict(dout=FAKE + 8), 1), (dict(ws=None), 4),
    (dict(ws=FAKE + 16), 1), (dict(wsb=1000), 4)])
def test_linear_backward(M, kw, code):
    args = dict(dout=FAKE, dout_f32=0, pre=FAKE, x=FAKE, w=FAKE, M=4, N=256, K=128, act=2, dx=FAKE, dw=FAKE, dw_f32=0,
                db=FAKE, ws=FAKE, wsb=1 << 30, st=None)
    refused(M, "moe_linear_backward", args, kw, code)


def test_linear_workspace_size_and_binding(M):
    assert M.moe_linear_backward_workspace_size(0, 8, 8) > 0
    assert M.moe_linear_backward_workspace_size(100, 256, 8) >= 100 * 256 * 2
    for m, n, k in ((-1, 8, 8), (1, 4, 8), (1, 8, 4)):
        with pytest.raises(M.MoeError):
            M.moe_linear_backward_workspace_size(m, n, k)
    x, w = torch.zeros((4, 64), dtype=torch.bfloat16), torch.zeros((8, 64), dtype=torch.bfloat16)
    for call in (lambda: M.moe_linear(x, w, torch.zeros((4, 8))),
                 lambda: M.moe_linear_backward(torch.zeros((4, 8)), x, w, w.view(torch.uint8), dx=x)):
        with pytest.raises(ValueError):
            call()
