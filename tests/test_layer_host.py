"""Refusals of moe_layer_forward on the host: nothing is enqueued, and no CUDA
call is made before the checks."""
import ctypes

import pytest
import torch

FAKE = 1 << 20  # 256-byte aligned non-null address; never dereferenced


@pytest.fixture(scope="module")
def M():
    import __graft_entry__
    __graft_entry__.build()
    import moe_expert_ffn_rms_gb300 as M
    return M


def rc(M, shape, **kw):
    a = dict(x=FAKE, norm_w=FAKE, router_w=FAKE, logits=None, bias=None, ids=None, tw=None, w13=FAKE, w2=FAKE,
             s13=None, s2=None, tail=None, out=FAKE, f32=0, ids_out=None, tw_out=None, ws=FAKE, wsb=1 << 40)
    a.update(kw)
    n = M.lib.moe_launch_count()
    r = M.lib.moe_layer_forward(
        ctypes.byref(shape), a["x"], a["norm_w"], a["router_w"], a["logits"], a["bias"], a["ids"], a["tw"],
        a["w13"], a["w2"], a["s13"], a["s2"], a["tail"], a["out"], a["f32"], a["ids_out"], a["tw_out"],
        a["ws"], a["wsb"], None)
    assert M.lib.moe_launch_count() == n
    if r:
        assert M.last_error()
    return r


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), 1), (dict(norm_w=None), 1), (dict(w13=None), 1), (dict(w2=None), 1), (dict(out=None), 1),
    (dict(ws=None), 1), (dict(router_w=None), 1), (dict(logits=FAKE), 1), (dict(ids=FAKE, tw=FAKE), 1),
    (dict(router_w=None, ids=FAKE), 1), (dict(router_w=None, ids=FAKE, tw=FAKE, bias=FAKE), 1),
    (dict(tw=FAKE), 1), (dict(x=FAKE + 8), 1), (dict(w13=FAKE + 8), 1), (dict(out=FAKE + 2), 1),
    (dict(router_w=FAKE + 2), 1), (dict(bias=FAKE + 1), 1), (dict(ids_out=FAKE + 2), 1),
    (dict(tw_out=FAKE + 3), 1), (dict(ws=FAKE + 128), 1), (dict(wsb=1000), 4), (dict(f32=1), 1)])
def test_call_refusals(M, kw, code):
    assert rc(M, M.make_shape(4, 256, 8, 512, 2), **kw) == code


def test_shape_refusals(M):
    bad = [M.make_shape(9, 256, 8, 512, 2), M.make_shape(4, 16448, 8, 512, 2),
           M.make_shape(4, 256, 8, 512, 2, nvfp4=True), M.make_shape(4, 200, 8, 512, 2),
           M.make_shape(4, 256, 8, 500, 2), M.make_shape(4, 256, 300, 512, 2),
           M.make_shape(4, 256, 8, 512, 9), M.make_shape(4, 384, 8, 512, 2, fp8="block")]
    for s in bad:
        assert rc(M, s) == 2
        assert M.lib.moe_layer_workspace_size(ctypes.byref(s)) == 0
        with pytest.raises(M.MoeError):
            M.moe_layer_workspace_size(s)
    assert rc(M, M.make_shape(-1, 256, 8, 512, 2)) == 1
    assert rc(M, M.make_shape(0, 256, 8, 512, 2), x=None, out=None, ws=None) == 0


def test_fp8_needs_scales(M):
    for fp8 in (True, "block"):
        s = M.make_shape(4, 256, 8, 512, 2, fp8=fp8)
        assert rc(M, s) == 1
        assert rc(M, s, s13=FAKE) == 1
        assert rc(M, s, s13=FAKE + 4, s2=FAKE) == 1


def test_tail_is_checked(M):
    t = M.MoeBlockTail()
    t.next_w = FAKE  # without xhat or xq
    assert rc(M, M.make_shape(4, 256, 8, 512, 2), tail=ctypes.byref(t)) == 1
    t = M.MoeBlockTail()
    t.gate, t.gate_cols, t.gate_rows = FAKE, 256, 3  # three rows for four tokens, no index
    assert rc(M, M.make_shape(4, 256, 8, 512, 2), tail=ctypes.byref(t)) == 1


def test_workspace_size(M):
    s = M.make_shape(8, 4096, 64, 1536, 8)
    n = M.moe_layer_workspace_size(s)
    assert n % 256 == 0
    # x_hat and the intermediate in two bf16 terms, partial logits, f
    assert n >= 8 * 4096 * 4 + 64 * 1536 * 4 + 16 * 8 * 64 * 4 + 8 * 4096 * 4


def test_binding_refusals(M):
    s = M.make_shape(4, 256, 8, 512, 2)
    x = torch.zeros((4, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError):  # host tensors are refused before any launch
        M.moe_layer_forward(s, x, x[0], x, x, x, torch.empty(1 << 20, dtype=torch.uint8))


def test_workspace_bytes_never_exceed_the_tensor(M):
    """Views that end before their first 256-byte boundary, expanded and strided ones."""
    whole = torch.empty(4096, dtype=torch.uint8)
    start = -whole.data_ptr() % 256
    assert M._ws_bytes(whole) == 4096 - start
    assert M._ws_bytes(whole[start + 1:start + 41]) == 0
    assert M._ws_bytes(whole[start:start + 1].expand(1 << 20)) == 1
    assert M._ws_bytes(whole[start:start + 2000:2]) == 1000
    assert M._ws_bytes(whole[start:start]) == 0
    # a call with such a view is refused, before any CUDA call
    bf = torch.bfloat16
    T, H, E, I, k = 2, 256, 4, 128, 2
    x, w, out = torch.zeros((T, H), dtype=bf), torch.zeros(H, dtype=bf), torch.zeros((T, H), dtype=bf)
    w13, w2 = torch.zeros((E, 2 * I, H), dtype=bf), torch.zeros((E, H, I), dtype=bf)
    wr = torch.zeros((H, E))
    s = M.make_shape(T, H, E, I, k)
    for ws in (whole[start + 1:start + 41], whole[start:start + 1].expand(1 << 30)):
        with pytest.raises(M.MoeError) as e:
            M.moe_ffn_forward(s, x, w, w13, w2, out, ws, router_w=wr, stream=0)
        assert e.value.name == "MOE_ERR_WORKSPACE_TOO_SMALL"
        rc = M.lib.moe_layer_forward(ctypes.byref(s), 1 << 20, 1 << 20, 1 << 20, None, None, None, None, 1 << 20,
                                     1 << 20, None, None, None, 1 << 20, 0, None, None, M._ws_ptr(ws),
                                     M._ws_bytes(ws), None)
        assert rc == 4
