"""Refusals of moe_combine_norm and of the block tail on the host: nothing is
enqueued, and no CUDA call is made before the checks."""
import ctypes

import pytest
import torch

FAKE = 1 << 20  # 16-byte aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_ffn_rms_gb300 as M
    return M


def tail(M, **kw):
    s = M.MoeBlockTail()
    s.scale, s.post_eps, s.next_eps = 1.0, 1e-6, 1e-6
    for n, v in kw.items():
        setattr(s, n, v)
    return s


def rc(M, s, y=FAKE, y_bf16=1, pair=1, rop=None, T=4, k=2, H=256, out=FAKE):
    return M.lib.moe_combine_norm(y, y_bf16, pair, rop, T, k, H, None if s is None else ctypes.byref(s),
                                  out, 0, None)


@pytest.mark.parametrize("kw,code", [
    (dict(y=None), 1), (dict(out=None), 1), (dict(pair=0), 1), (dict(y=FAKE + 8), 1),
    (dict(out=FAKE + 8), 1), (dict(rop=FAKE + 2), 1), (dict(H=252), 2), (dict(H=0), 2),
    (dict(H=32776), 2), (dict(k=0), 2), (dict(k=9), 2), (dict(T=-1), 2), (dict(T=1 << 23, k=8), 2)])
def test_call_refusals(M, kw, code):
    n = M.lib.moe_launch_count()
    assert rc(M, tail(M), **kw) == code
    assert M.last_error()
    assert M.lib.moe_launch_count() == n


@pytest.mark.parametrize("kw,code", [
    (dict(residual=FAKE + 8), 1), (dict(post_w=FAKE + 2), 1), (dict(post_eps=-1.0), 1),
    (dict(next_eps=float("nan")), 1), (dict(next_w=FAKE), 1), (dict(xhat=FAKE), 1),
    (dict(next_w=FAKE, xhat=FAKE + 8), 1), (dict(next_w=FAKE, xq=FAKE), 1),
    (dict(next_w=FAKE, xhat=FAKE, xscale=FAKE), 1),
    (dict(next_w=FAKE, xq=FAKE, xscale=FAKE + 2), 1),
    (dict(next_w=FAKE, xq=FAKE, xscale=FAKE, q_group=64), 1),
    (dict(gate=FAKE, gate_cols=128, gate_rows=1), 1), (dict(gate=FAKE, gate_cols=256, gate_rows=0), 1),
    (dict(gate=FAKE, gate_cols=256, gate_rows=3), 1), (dict(gate=FAKE + 8, gate_cols=256, gate_rows=1), 1),
    (dict(gate=FAKE + 2, gate_cols=1, gate_rows=4, gate_f32=1), 1), (dict(gate_row=FAKE), 1)])
def test_tail_refusals(M, kw, code):
    assert rc(M, tail(M, **kw)) == code
    assert M.last_error()


def test_group_scales_need_whole_groups(M):
    s = tail(M, next_w=FAKE, xq=FAKE, xscale=FAKE, q_group=128)
    assert rc(M, s, H=264) == 2
    assert rc(M, None) == 1


def test_binding_refusals(M):
    bf = torch.bfloat16
    x, w = torch.zeros((4, 256), dtype=bf), torch.ones(256, dtype=bf)
    bad = [dict(residual=x.half()), dict(residual=x[0]), dict(residual=x[:, ::2]),
           dict(residual=x, post_w=w[:128]), dict(residual=x, post_w=w.float()),
           dict(residual=x, gate=torch.zeros((3, 256))), dict(residual=x, gate=torch.zeros((4, 2))),
           dict(residual=x, gate=torch.zeros(2, 2, 2)),
           dict(residual=x, gate=w, gate_row=torch.zeros(3, dtype=torch.int32)),
           dict(residual=x, gate_row=torch.zeros(4, dtype=torch.int32)),
           dict(residual=x, gate=w, gate_row=torch.zeros(4, dtype=torch.int64)),
           dict(residual=x, next_w=w, xhat=torch.zeros((5, 256), dtype=bf)),
           dict(residual=x, next_w=w, xq=torch.zeros((4, 256))),
           dict(residual=x, next_w=w, xq=torch.zeros((4, 256), dtype=torch.uint8),
                xscale=torch.zeros(4, 3))]
    for kw in bad:
        with pytest.raises(ValueError):
            M.make_block_tail(**kw)
    t = M.make_block_tail(residual=x, post_w=w, gate=w.float(), scale=0.5)
    assert (t.T, t.H) == (4, 256) and t.struct.gate_cols == 256 and t.struct.gate_rows == 1
    assert t.struct.gate_f32 == 1 and t.struct.residual_f32 == 0
    t = M.make_block_tail(gate=torch.zeros((6, 1)), post_w=w)
    assert t.T == 6 and t.struct.gate_cols == 1
    with pytest.raises(ValueError):  # host tensors are refused before any launch
        M.moe_combine_norm(torch.zeros((8, 256), dtype=bf), x, 4, 2, t)


def test_codes_from_products_on_both_sides_of_the_quotient():
    """The rule of the E4M3 codes in block_tail.cuh, in fp32 on the CPU: where the products with 2^-21 less and
    2^-21 more than the rounded reciprocal have one code, it is the code of the IEEE quotient; elsewhere the
    kernel divides.  Values beside every middle between two codes, over scales of every mantissa and size."""
    g = torch.Generator().manual_seed(1)
    grid = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    mid = (grid[1:] + grid[:-1]) / 2

    def codes(q):
        return q.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)

    divided = 0
    for e in (-99, -60, -20, -9, 0, 40, 110):
        s = (1 + torch.rand((20000, 1), generator=g)) * 2.0 ** e
        v = mid * s
        v = torch.stack([v, *(v.view(torch.int32).add(d).view(torch.float32) for d in (-3, -2, -1, 1, 2, 3, 40, -40))])
        inv = 1 / s
        lo, hi = codes(v * (inv * (1 - 2.0 ** -21))), codes(v * (inv * (1 + 2.0 ** -21)))
        same = lo == hi
        assert torch.equal(lo[same], codes(v / s)[same])
        divided += int((~same).sum())
    assert divided > 0
    w = torch.randn((1000, 4096), generator=g)  # ordinary rows hardly ever divide
    s = w.abs().amax(1, keepdim=True) / 448
    lo, hi = (codes(w * (1 / s * f)) for f in (1 - 2.0 ** -21, 1 + 2.0 ** -21))
    assert (lo != hi).float().mean() < 5e-5
