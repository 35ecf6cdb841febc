"""The norm kernels over more rows than one round of CTAs takes, against their formulas in 64 bits: stages that are sent
for again (rows of 520 columns and more, in both types of every operand), warps that take several rows (short rows), CTAs
that add several rows' dw (rows above 8192 columns), and offsets beyond 32 bits.  Inputs, references and tolerances are
those of test_gpu_norm.py."""
import pytest
import torch

from tests.test_gpu_norm import BF, DEV, EPS, F32, R, TYPES, U, M, grads, make, near, reference, stats, step  # noqa: F401

pytestmark = pytest.mark.gpu


def check_forward(d, out, mean, rstd):
    wd = d["w"].double()
    for i in range(0, out.shape[0], 4096):  # (a part of the rows at a time: the 64-bit copies are large)
        rows = slice(i, i + 4096)
        xd = d["x"][rows].double()
        m, v, var, r = stats(xd)
        em = R * xd.abs().mean(1, keepdim=True)
        er = 0.5 * (R + 4 * U + em * em / (var + EPS)) + 2 * U
        ref = v * r * wd + (0 if d["b"] is None else d["b"].double())
        tol = (v * r * wd).abs() * (er + 3 * U) + em * r * wd.abs() + U * ref.abs()
        tol = tol + step(out.dtype, ref.abs() + tol)
        bad = (out[rows].double() - ref).abs() > tol
        assert not bad.any(), (i, int(bad.sum()), bad.nonzero()[:4].tolist())
        assert ((mean[rows].double() - m[:, 0]).abs() <= em[:, 0] + U * m[:, 0].abs()).all()
        assert ((rstd[rows].double() - r[:, 0]).abs() <= ((er + U) * r)[:, 0]).all()


@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("x,y,w", TYPES + [(BF, BF, F32), (F32, F32, BF)])
@pytest.mark.parametrize("T,H", [(25001, 40), (20001, 256), (12000, 512), (6000, 520), (7001, 960), (5000, 4096),
                                 (1999, 8192), (1500, 16384)])
def test_forward(M, T, H, x, y, w, bias):  # noqa: F811
    d = make(T, H, x, y, w, bias, res=False)
    out = torch.full((T, H), float("nan"), device=DEV, dtype=y)
    mean, rstd = torch.full((T,), float("nan"), device=DEV), torch.full((T,), float("nan"), device=DEV)
    M.moe_layernorm(d["x"], d["w"], EPS, out, b=d["b"], mean=mean, rstd=rstd)
    check_forward(d, out, mean, rstd)
    if x == y:  # in place
        M.moe_layernorm(d["x"], d["w"], EPS, d["x"], b=d["b"])
        assert torch.equal(d["x"], out)
    assert M.device_status() == 0


@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("res", [True, False])
@pytest.mark.parametrize("x,dy,w", TYPES + [(BF, BF, F32), (F32, F32, BF)])
@pytest.mark.parametrize("T,H", [(16384, 40), (9000, 256), (5000, 264), (4001, 1024), (3001, 4096), (1500, 8192),
                                 (1000, 8200), (700, 16384)])
def test_backward(M, T, H, x, dy, w, res, rms):  # noqa: F811
    d = make(T, H, x, dy, w, res=res)
    mean, rstd, rx, rw, rb = reference(d, rms)
    dx, dw, db = grads(M, d, rms, mean, rstd)
    assert near(dx, rx) and near(dw, rw) and (rms or near(db, rb))
    # dx over what it is made from
    if x == dy:
        e = dict(d, dy=d["dy"].clone())
        got = grads(M, e, rms, mean, rstd, dx=e["dy"])
        assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    e = dict(d, x=d["x"].clone())
    got = grads(M, e, rms, mean, rstd, dx=e["x"])
    assert torch.equal(got[0], dx) and torch.equal(got[1], dw)
    assert M.device_status() == 0


def test_rows_beyond_32_bit_offsets(M):  # noqa: F811
    """Equal rows: the first against its formula, the others equal to it, and dw and db as many times one row's."""
    T, H = 140000, 16384
    one = make(1, H, bias=True, res=False)
    d = dict(one, T=T, x=one["x"].expand(T, -1).contiguous(), dy=one["dy"].expand(T, -1).contiguous())
    y = torch.empty_like(d["x"])
    mean, rstd = torch.empty(T, device=DEV), torch.empty(T, device=DEV)
    M.moe_layernorm(d["x"], d["w"], EPS, y, b=d["b"], mean=mean, rstd=rstd)
    check_forward(one, y[:1], mean[:1], rstd[:1])
    assert torch.equal(y, y[:1].expand(T, -1)) and (mean == mean[0]).all() and (rstd == rstd[0]).all()
    del y
    n = (T + 63) // 64 + 320 + 3
    for rms in (False, True):
        m1, r1, rx, rw, rb = reference(one, rms)
        mean, rstd = (None, None) if rms else (m1.expand(T).contiguous(), r1.expand(T).contiguous())
        dx, dw, db = grads(M, d, rms, mean, rstd)
        assert near(dx[:1], rx) and torch.equal(dx, dx[:1].expand(T, -1))
        for got, (ref, tol) in ((dw, rw), (db, rb)):
            if got is not None:
                assert ((got.double() - T * ref).abs() <= T * (tol + n * U * ref.abs())).all()
        del dx
    assert M.device_status() == 0
