"""Python binding of libmoeffn.so -- the MoE expert FFN forward on a GB300.

Argument marshalling only: every step runs in the library's CUDA kernels.
Functions take torch tensors (device memory) and enqueue work on the current
torch CUDA stream unless a stream is given.  They have the same names as the
C entry points in include/moe_ffn.h.

Importing the package loads the library; if it has not been built
(``python -m moe_expert_ffn_rms_gb300.build`` or ``__graft_entry__.build()``)
the import fails with an ImportError -- there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libmoeffn.so")

if not os.path.exists(LIB_PATH):
    raise ImportError(f"{LIB_PATH} is not built; run moe_expert_ffn_rms_gb300.build.build()")

lib = ctypes.CDLL(LIB_PATH)

MOE_OK = 0
STATUS_NAMES = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE",
                3: "MOE_ERR_UNSUPPORTED_DEVICE", 4: "MOE_ERR_WORKSPACE_TOO_SMALL",
                5: "MOE_ERR_CUDA", 6: "MOE_ERR_TIMEOUT"}
W_BF16, W_FP8_E4M3, W_NVFP4, W_FP8_BLOCK = 0, 1, 2, 3
ACT_NONE, ACT_RELU, ACT_SILU, ACT_GELU, ACT_GELU_TANH = 0, 1, 2, 3, 4
GEMM_FC1_RAW, GEMM_FC1_SILU, GEMM_FC2, GEMM_FC2_BF16 = 0, 1, 2, 3
ENGINE_AUTO, ENGINE_DECODE, ENGINE_PREFILL = 0, 1, 2


class MoeShape(ctypes.Structure):
    _fields_ = [("T", ctypes.c_int32), ("H", ctypes.c_int32), ("E", ctypes.c_int32),
                ("I", ctypes.c_int32), ("top_k", ctypes.c_int32), ("eps", ctypes.c_float),
                ("wdtype", ctypes.c_int32), ("engine", ctypes.c_int32)]


class MoeBlockTail(ctypes.Structure):
    _fields_ = [("residual", ctypes.c_void_p), ("post_w", ctypes.c_void_p),
                ("gate", ctypes.c_void_p), ("gate_row", ctypes.c_void_p),
                ("next_w", ctypes.c_void_p), ("xhat", ctypes.c_void_p), ("xq", ctypes.c_void_p),
                ("xscale", ctypes.c_void_p), ("post_eps", ctypes.c_float),
                ("next_eps", ctypes.c_float), ("scale", ctypes.c_float),
                ("residual_f32", ctypes.c_int32), ("gate_f32", ctypes.c_int32),
                ("gate_cols", ctypes.c_int32), ("gate_rows", ctypes.c_int32),
                ("q_group", ctypes.c_int32)]


class MoeError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status
        self.name = STATUS_NAMES.get(status, str(status))


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_SZ = ctypes.c_size_t

_SIGS = {
    "moe_abi_version": (_I32, []),
    "moe_launch_count": (ctypes.c_int64, []),
    "moe_last_error": (ctypes.c_char_p, []),
    "moe_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "moe_check_device": (ctypes.c_int, []),
    "moe_device_status": (ctypes.c_int, [ctypes.POINTER(_I32), _I32]),
    "moe_selftest_wait_timeout": (ctypes.c_int, [ctypes.c_int64, _P]),
    "moe_ffn_workspace_size": (_SZ, [ctypes.POINTER(MoeShape)]),
    "moe_ffn_forward": (ctypes.c_int, [ctypes.POINTER(MoeShape), _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                       _P, _P, _P, _P, _SZ, _P]),
    "moe_ffn_forward_routed": (ctypes.c_int, [ctypes.POINTER(MoeShape), _P, _P, _P, _P, _P, _P, _P,
                                              _P, _P, _P, _SZ, _P]),
    "moe_ffn_forward_static_ws": (ctypes.c_int, [ctypes.POINTER(MoeShape), _P, _P, _P, _P, _P, _P,
                                                 _P, _P, _P, _P, _P, _P, _P]),
    "moe_rmsnorm": (ctypes.c_int, [_P, _P, _I32, _I32, ctypes.c_float, _P, _P, _P, _P]),
    "moe_route_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "moe_route_topk": (ctypes.c_int, [_P, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _SZ,
                                      _P]),
    "moe_permute_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "moe_permute": (ctypes.c_int, [_P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _I32, _P, _P, _P, _SZ,
                                   _P]),
    "moe_grouped_gemm": (ctypes.c_int, [ctypes.POINTER(MoeShape), _I32, _P, _P, _P, _P, _P, _P, _P,
                                        _P, _P]),
    "moe_grouped_ffn_workspace_size": (_SZ, [ctypes.POINTER(MoeShape)]),
    "moe_grouped_ffn": (ctypes.c_int, [ctypes.POINTER(MoeShape), _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                       _P, _P, _P, _SZ, _P]),
    "moe_silu_and_mul": (ctypes.c_int, [_P, _I32, _I32, _P, _P]),
    "moe_combine": (ctypes.c_int, [_P, _I32, _I32, _P, _I32, _I32, _I32, _P, _P]),
    "moe_layer_workspace_size": (_SZ, [ctypes.POINTER(MoeShape)]),
    "moe_layer_forward": (ctypes.c_int, [ctypes.POINTER(MoeShape), _P, _P, _P, _P, _P, _P, _P, _P, _P,
                                         _P, _P, ctypes.POINTER(MoeBlockTail), _P, _I32, _P, _P, _P,
                                         _SZ, _P]),
    "moe_combine_norm": (ctypes.c_int, [_P, _I32, _I32, _P, _I32, _I32, _I32,
                                        ctypes.POINTER(MoeBlockTail), _P, _I32, _P]),
    "moe_quantize_fp8_rows": (ctypes.c_int, [_P, ctypes.c_int64, _I32, _P, _P, _P]),
    "moe_ffn_forward_nvfp4": (ctypes.c_int, [ctypes.POINTER(MoeShape), _P, _P, _P, _P, _P, _P, _P, _P,
                                             _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_quantize_nvfp4": (ctypes.c_int, [_P, _I32, _I32, _I32, _P, _P, _P, _P]),
    "moe_grouped_ffn_nvfp4": (ctypes.c_int, [ctypes.POINTER(MoeShape), _P, _P, _P, _P, _P, _P, _P, _P,
                                             _P, _P, _P, _P, _P, _SZ, _P]),
    "moe_quantize_fp8_blocks": (ctypes.c_int, [_P, _I32, _I32, _I32, _P, _P, _P]),
    "moe_unpermute": (ctypes.c_int, [_P, _I32, _P, _P, _I32, _I32, _I32, _P, _I32, _P, _I32, _P]),
    "moe_unpermute_backward": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _P, _P, _I32, _I32, _I32, _I32, _P,
                                              _P, _P, _P]),
    "moe_permute_backward": (ctypes.c_int, [_P, _I32, _P, _I32, _I32, _I32, _P, _I32, _P, _I32, _P]),
    "moe_layernorm": (ctypes.c_int, [_P, _I32, _P, _P, _I32, _I32, _I32, ctypes.c_float, _P, _I32, _P, _P,
                                     _P]),
    "moe_norm_backward_workspace_size": (_SZ, [_I32, _I32]),
    "moe_layernorm_backward": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _I32, _P, _P, _P, _I32, _I32, _P, _P,
                                              _P, _P, _SZ, _P]),
    "moe_rmsnorm_backward": (ctypes.c_int, [_P, _I32, _P, _I32, _P, _I32, ctypes.c_float, _P, _I32, _I32,
                                            _P, _P, _P, _SZ, _P]),
    "moe_linear": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _I32, _I32, _I32, _I32, _P, _P, _I32, _P]),
    "moe_linear_backward_workspace_size": (_SZ, [_I32, _I32, _I32]),
    "moe_linear_backward": (ctypes.c_int, [_P, _I32, _P, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _I32, _P, _P,
                                           _SZ, _P]),
}
for _name, (_res, _args) in _SIGS.items():
    _f = getattr(lib, _name)
    _f.restype = _res
    _f.argtypes = _args

EXPORTED = tuple(_SIGS)


def last_error() -> str:
    return lib.moe_last_error().decode()


def _check(rc: int):
    if rc != MOE_OK:
        raise MoeError(rc, last_error() or STATUS_NAMES.get(rc, str(rc)))


def _ptr(t):
    if t is None:
        return None
    if isinstance(t, int):
        return t
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


# The current stream's handle.  torch.cuda.current_stream() builds a Stream
# object (about 3 us of a 10 us call); the raw query is used where torch has it.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream):
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        return torch.cuda.current_stream().cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def make_shape(T, H, E, I, top_k, eps=1e-6, fp8=False, engine=ENGINE_AUTO, nvfp4=False) -> MoeShape:
    """fp8: False (bf16), True (per-channel E4M3) or "block" (block-wise E4M3)."""
    wd = W_NVFP4 if nvfp4 else (W_FP8_BLOCK if fp8 == "block" else (W_FP8_E4M3 if fp8 else W_BF16))
    return MoeShape(T, H, E, I, top_k, eps, wd, engine)


def abi_version() -> int:
    return lib.moe_abi_version()


def check_device():
    _check(lib.moe_check_device())


def device_status(clear: bool = True) -> int:
    v = _I32(0)
    _check(lib.moe_device_status(ctypes.byref(v), 1 if clear else 0))
    return v.value


def moe_selftest_wait_timeout(limit_cycles: int, stream=None):
    _check(lib.moe_selftest_wait_timeout(limit_cycles, _stream(stream)))


def moe_ffn_workspace_size(shape: MoeShape) -> int:
    n = lib.moe_ffn_workspace_size(ctypes.byref(shape))
    if n == 0:
        raise MoeError(1, last_error())
    return n


def alloc_workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Device workspace (torch owns the memory; 256-byte aligned)."""
    return torch.empty(nbytes + 256, dtype=torch.uint8, device=device)


def _ws_ptr(ws: torch.Tensor) -> int:
    p = ws.data_ptr()
    return (p + 255) & ~255


def _ws_bytes(ws: torch.Tensor) -> int:
    """Bytes from the aligned start on that surely belong to ws: none of a view that ends before
    it, and no more of an expanded one than its storage holds."""
    n = ws.numel()
    if not ws.is_contiguous():
        n = min(n, 1 + sum((size - 1) * stride for size, stride in zip(ws.shape, ws.stride())))
    return max(0, n - (_ws_ptr(ws) - ws.data_ptr()))


def moe_ffn_forward(shape: MoeShape, x, norm_w, w13, w2, out, workspace, router_w=None,
                    router_logits=None, router_bias=None, w13_scale=None, w2_scale=None,
                    topk_ids_out=None, topk_w_out=None, stream=None):
    _check(lib.moe_ffn_forward(ctypes.byref(shape), _ptr(x), _ptr(norm_w), _ptr(router_w),
                               _ptr(router_logits), _ptr(router_bias), _ptr(w13), _ptr(w2),
                               _ptr(w13_scale), _ptr(w2_scale), _ptr(out), _ptr(topk_ids_out),
                               _ptr(topk_w_out), _ws_ptr(workspace), _ws_bytes(workspace),
                               _stream(stream)))
    return out


def moe_ffn_forward_static_ws(shape: MoeShape, x, norm_w, w13, w2, out, router_w=None,
                              router_logits=None, router_bias=None, w13_scale=None,
                              w2_scale=None, topk_ids_out=None, topk_w_out=None, stream=None):
    """moe_ffn_forward with the library's fixed 32 MiB device scratch instead
    of a caller workspace (for callers that cannot allocate device memory)."""
    _check(lib.moe_ffn_forward_static_ws(ctypes.byref(shape), _ptr(x), _ptr(norm_w), _ptr(router_w),
                                         _ptr(router_logits), _ptr(router_bias), _ptr(w13),
                                         _ptr(w2), _ptr(w13_scale), _ptr(w2_scale), _ptr(out),
                                         _ptr(topk_ids_out), _ptr(topk_w_out), _stream(stream)))
    return out


def moe_ffn_forward_routed(shape: MoeShape, x, norm_w, topk_ids, topk_w, w13, w2, out, workspace,
                           w13_scale=None, w2_scale=None, stream=None):
    _check(lib.moe_ffn_forward_routed(ctypes.byref(shape), _ptr(x), _ptr(norm_w), _ptr(topk_ids),
                                      _ptr(topk_w), _ptr(w13), _ptr(w2), _ptr(w13_scale),
                                      _ptr(w2_scale), _ptr(out), _ws_ptr(workspace),
                                      _ws_bytes(workspace), _stream(stream)))
    return out


def moe_rmsnorm(x, w, eps, y, yq=None, yscale=None, stream=None):
    T, H = x.shape
    _check(lib.moe_rmsnorm(_ptr(x), _ptr(w), T, H, eps, _ptr(y), _ptr(yq), _ptr(yscale),
                           _stream(stream)))
    return y


def moe_route_workspace_size(T, H, E) -> int:
    return lib.moe_route_workspace_size(T, H, E)


def moe_route_topk(T, H, E, k, ids, weights, xhat=None, router_w=None, router_bias=None,
                   logits_in=None, logits_out=None, workspace=None, stream=None):
    wsp = _ws_ptr(workspace) if workspace is not None else None
    wsb = _ws_bytes(workspace) if workspace is not None else 0
    _check(lib.moe_route_topk(_ptr(xhat), _ptr(router_w), _ptr(router_bias), _ptr(logits_in), T, H,
                              E, k, _ptr(ids), _ptr(weights), _ptr(logits_out), wsp, wsb,
                              _stream(stream)))


def moe_permute_workspace_size(T, E, k) -> int:
    return lib.moe_permute_workspace_size(T, E, k)


def moe_permute(ids, T, E, k, offsets, row_src, row_of_pair, xhat=None, xp=None, row_bytes=0,
                xscale=None, xp_scale=None, workspace=None, stream=None):
    wsp = _ws_ptr(workspace) if workspace is not None else None
    wsb = _ws_bytes(workspace) if workspace is not None else 0
    _check(lib.moe_permute(_ptr(ids), T, E, k, _ptr(offsets), _ptr(row_src), _ptr(row_of_pair),
                           _ptr(xhat), _ptr(xp), row_bytes, _ptr(xscale), _ptr(xp_scale), wsp,
                           wsb, _stream(stream)))


def moe_grouped_gemm(shape: MoeShape, mode, a, w, offsets, c, a_scale=None, w_scale=None,
                     row_src=None, topk_w=None, stream=None):
    _check(lib.moe_grouped_gemm(ctypes.byref(shape), mode, _ptr(a), _ptr(a_scale), _ptr(w),
                                _ptr(w_scale), _ptr(offsets), _ptr(row_src), _ptr(topk_w), _ptr(c),
                                _stream(stream)))
    return c


def moe_grouped_ffn_workspace_size(shape: MoeShape) -> int:
    return lib.moe_grouped_ffn_workspace_size(ctypes.byref(shape))


def moe_grouped_ffn(shape: MoeShape, xp, w13, w2, offsets, row_src, topk_w, act, y, workspace,
                    xp_scale=None, w13_scale=None, w2_scale=None, stream=None):
    _check(lib.moe_grouped_ffn(ctypes.byref(shape), _ptr(xp), _ptr(xp_scale), _ptr(w13),
                               _ptr(w13_scale), _ptr(w2), _ptr(w2_scale), _ptr(offsets),
                               _ptr(row_src), _ptr(topk_w), _ptr(act), _ptr(y), _ws_ptr(workspace),
                               _ws_bytes(workspace), _stream(stream)))
    return y


def moe_silu_and_mul(h, a, stream=None):
    R, I2 = h.shape
    _check(lib.moe_silu_and_mul(_ptr(h), R, I2 // 2, _ptr(a), _stream(stream)))
    return a


def moe_combine(y, row_of_pair, T, k, out, pair_order=False, stream=None):
    H = y.shape[1]
    y_bf16 = 1 if y.dtype == torch.bfloat16 else 0
    _check(lib.moe_combine(_ptr(y), y_bf16, 1 if pair_order else 0, _ptr(row_of_pair), T, k, H,
                           _ptr(out), _stream(stream)))
    return out


def moe_ffn_forward_nvfp4(shape: MoeShape, x, norm_w, w13, w13_sb, w13_sg, w2, w2_sb, w2_sg, out,
                          workspace, router_w=None, router_logits=None, router_bias=None,
                          topk_ids_out=None, topk_w_out=None, stream=None):
    """The forward with NVFP4 expert weights (codes, E4M3 block scales, fp32
    matrix scales from moe_quantize_nvfp4) and bf16 activations."""
    _check(lib.moe_ffn_forward_nvfp4(ctypes.byref(shape), _ptr(x), _ptr(norm_w), _ptr(router_w),
                                     _ptr(router_logits), _ptr(router_bias), _ptr(w13), _ptr(w13_sb),
                                     _ptr(w13_sg), _ptr(w2), _ptr(w2_sb), _ptr(w2_sg), _ptr(out),
                                     _ptr(topk_ids_out), _ptr(topk_w_out), _ws_ptr(workspace),
                                     _ws_bytes(workspace), _stream(stream)))
    return out


def moe_grouped_ffn_nvfp4(shape: MoeShape, xp, w13, w13_sb, w13_sg, w2, w2_sb, w2_sg, offsets,
                          row_src, topk_w, act, y, workspace, stream=None):
    """The NVFP4 FFN step: xp fp16 [R, H] -> act fp16 [R, I] -> y bf16 [R, H]."""
    _check(lib.moe_grouped_ffn_nvfp4(ctypes.byref(shape), _ptr(xp), _ptr(w13), _ptr(w13_sb),
                                     _ptr(w13_sg), _ptr(w2), _ptr(w2_sb), _ptr(w2_sg), _ptr(offsets),
                                     _ptr(row_src), _ptr(topk_w), _ptr(act), _ptr(y),
                                     _ws_ptr(workspace), _ws_bytes(workspace), _stream(stream)))


def moe_quantize_nvfp4(w, q, sb, sg, stream=None):
    """NVFP4 quantisation of w bf16 [M, N, K] (or [N, K]) into q uint8
    [.., N, K/2], sb uint8 [.., N, K/16], sg fp32 [M]."""
    K = w.shape[-1]
    N = w.shape[-2]
    M = w.numel() // (N * K) if w.numel() else 0
    _check(lib.moe_quantize_nvfp4(_ptr(w), M, N, K, _ptr(q), _ptr(sb), _ptr(sg), _stream(stream)))


def _check_tensor(t, name, shape, dtypes, device):
    """Raises ValueError unless t is a contiguous tensor of this shape, one of
    these types, on this device."""
    if t.dtype not in dtypes:
        raise ValueError(f"{name}: dtype {t.dtype}, need {' or '.join(map(str, dtypes))}")
    if t.shape != shape:
        raise ValueError(f"{name}: shape {tuple(t.shape)}, need {tuple(shape)}")
    if t.device != device:
        raise ValueError(f"{name}: on {t.device}, need {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: tensors must be contiguous")


_BF16 = (torch.bfloat16,)
_FLOATS = (torch.bfloat16, torch.float32)
_I32S = (torch.int32,)
_F32S = (torch.float32,)


class BlockTail:
    """A moe_block_tail and the tensors it points to (kept alive by it).  T is
    None while none of them fixes the number of tokens."""

    def __init__(self, struct, tensors, T, H, device, rows):
        self.struct = struct
        self.ref = ctypes.byref(struct)
        self.tensors = tensors
        self.T, self.H, self.device, self.rows = T, H, device, rows


def make_block_tail(residual=None, post_w=None, post_eps=1e-6, gate=None, gate_row=None, scale=1.0,
                    next_w=None, next_eps=1e-6, xhat=None, xq=None, xscale=None) -> BlockTail:
    """What follows a block (moe_block_tail in include/moe_ffn.h):
    h = residual + scale * gate * rms_norm(f; post_w); x_hat = rms_norm(h; next_w).

    residual bf16 / fp32 [T, H]; post_w, next_w bf16 [H]; gate bf16 / fp32: [H]
    (one factor per column), [T, 1] (one per token), [T, H], or [G, H] / [G, 1]
    with gate_row int32 [T]; xhat bf16 [T, H], xq uint8 or float8_e4m3fn [T, H]
    with xscale fp32 [T] (a scale per token) or [T, H/128] (per 128 columns).

    The result can be used for any number of calls; it holds pointers to the
    tensors it was made from."""
    ts = {n: t for n, t in (("residual", residual), ("post_w", post_w), ("gate", gate),
                            ("gate_row", gate_row), ("next_w", next_w), ("xhat", xhat), ("xq", xq),
                            ("xscale", xscale)) if t is not None}
    T = H = device = None
    for n in ("residual", "xhat", "xq"):
        if n in ts:
            if ts[n].dim() != 2:
                raise ValueError(f"{n}: must be [T, H]")
            T, H = ts[n].shape
            break
    for n in ("post_w", "next_w"):
        if H is None and n in ts:
            H = ts[n].numel()
    if gate is not None and gate.dim() not in (1, 2):
        raise ValueError("gate: must be [H] or [rows, H or 1]")
    if H is None and gate is not None and gate.shape[-1] != 1:
        H = gate.shape[-1]
    if T is None and gate_row is not None:
        T = gate_row.numel()
    for t in ts.values():
        device = t.device
        break
    s = MoeBlockTail()
    s.post_eps, s.next_eps, s.scale = post_eps, next_eps, scale
    rows = 1
    if residual is not None:
        _check_tensor(residual, "residual", (T, H), _FLOATS, device)
        s.residual_f32 = residual.dtype == torch.float32
    for n in ("post_w", "next_w"):
        if n in ts:
            _check_tensor(ts[n], n, (H,), _BF16, device)
    if gate is not None:
        g = gate if gate.dim() == 2 else gate[None]
        rows, cols = g.shape
        if cols != 1 and cols != H:
            raise ValueError(f"gate: {cols} columns, need 1 or {H}")
        _check_tensor(gate, "gate", gate.shape, _FLOATS, device)
        s.gate_rows, s.gate_cols, s.gate_f32 = rows, cols, gate.dtype == torch.float32
        if gate_row is None and rows != 1:
            if T is None:
                T = rows
            elif rows != T:
                raise ValueError(f"gate: {rows} rows without gate_row, need 1 or {T}")
    if gate_row is not None:
        if gate is None:
            raise ValueError("gate_row: needs gate")
        _check_tensor(gate_row, "gate_row", (T,), _I32S, device)
    if xhat is not None:
        _check_tensor(xhat, "xhat", (T, H), _BF16, device)
    if xq is not None:
        _check_tensor(xq, "xq", (T, H), (torch.uint8, torch.float8_e4m3fn), device)
    if xscale is not None:
        if xscale.dim() == 2:
            s.q_group = 128
            _check_tensor(xscale, "xscale", (T, (H or 0) // 128), _F32S, device)
        else:
            _check_tensor(xscale, "xscale", (T,), _F32S, device)
    for n, t in ts.items():
        setattr(s, n, t.data_ptr())
    return BlockTail(s, tuple(ts.values()), T, H, device, rows)


def _check_current(device):
    if device.type != "cuda":
        raise ValueError(f"tensors must be on a CUDA device, not {device}")
    if device.index != torch.cuda.current_device():
        raise ValueError(f"tensors are on {device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _check_tail(tail, T, H, device):
    if tail.T is not None and tail.T != T:
        raise ValueError(f"tail: made for {tail.T} tokens, need {T}")
    if tail.H is not None and tail.H != H:
        raise ValueError(f"tail: made for H={tail.H}, need {H}")
    if tail.device is not None and tail.device != device:
        raise ValueError(f"tail: tensors on {tail.device}, need {device}")


def moe_combine_norm(y, out, T, k, tail: BlockTail, row_of_pair=None, pair_order=True, stream=None):
    """Sum of each token's k expert rows and what follows the block, in one
    pass.  y bf16 / fp32 [T*k, H], out bf16 / fp32 [T, H]; rows in (token, slot)
    order, or (pair_order=False) at row_of_pair int32 [T*k]."""
    H = y.shape[-1]
    device = y.device
    _check_current(device)
    _check_tensor(y, "y", (T * k, H), _FLOATS, device)
    _check_tensor(out, "out", (T, H), _FLOATS, device)
    if row_of_pair is not None:
        if row_of_pair.numel() != T * k:
            raise ValueError(f"row_of_pair: {row_of_pair.numel()} entries, need {T * k}")
        _check_tensor(row_of_pair, "row_of_pair", row_of_pair.shape, _I32S, device)
    _check_tail(tail, T, H, device)
    _check(lib.moe_combine_norm(y.data_ptr(), y.dtype == torch.bfloat16, 1 if pair_order else 0,
                                None if row_of_pair is None else row_of_pair.data_ptr(), T, k, H,
                                tail.ref, out.data_ptr(), out.dtype == torch.float32,
                                _stream(stream)))
    return out


def moe_layer_workspace_size(shape: MoeShape) -> int:
    n = lib.moe_layer_workspace_size(ctypes.byref(shape))
    if n == 0:
        raise MoeError(2, last_error())
    return n


def _opt(t, name, shape, dtypes, device):
    if t is None:
        return None
    _check_tensor(t, name, shape, dtypes, device)
    return t.data_ptr()


_CODES = (torch.uint8, torch.float8_e4m3fn)


def moe_layer_forward(shape: MoeShape, x, norm_w, w13, w2, out, workspace, router_w=None,
                      router_logits=None, router_bias=None, topk_ids=None, topk_w=None,
                      w13_scale=None, w2_scale=None, tail: BlockTail = None, topk_ids_out=None,
                      topk_w_out=None, stream=None):
    """The whole MoE block for 1..8 tokens in two launches: norm, router (or
    given logits, or given topk_ids / topk_w), experts, weighted sum, and with a
    tail (make_block_tail) what follows the block.  Tensors as in
    moe_ffn_forward; out bf16 [T, H], or the type of the residual stream (bf16 /
    fp32) with a tail; workspace of moe_layer_workspace_size(shape) bytes."""
    T, H, E, I, k, wd = shape.T, shape.H, shape.E, shape.I, shape.top_k, shape.wdtype
    device = x.device
    _check_current(device)
    wt = _BF16 if wd == W_BF16 else _CODES
    if wd == W_FP8_BLOCK:
        s13, s2 = (E, 2 * I // 128, H // 128), (E, H // 128, I // 128)
    else:
        s13, s2 = (E, 2 * I), (E, H)
    _check_tensor(x, "x", (T, H), _BF16, device)
    _check_tensor(norm_w, "norm_w", (H,), _BF16, device)
    _check_tensor(w13, "w13", (E, 2 * I, H), wt, device)
    _check_tensor(w2, "w2", (E, H, I), wt, device)
    _check_tensor(out, "out", (T, H), _BF16 if tail is None else _FLOATS, device)
    if workspace.device != device:
        raise ValueError(f"workspace: on {workspace.device}, need {device}")
    if tail is not None:
        _check_tail(tail, T, H, device)
    _check(lib.moe_layer_forward(
        ctypes.byref(shape), x.data_ptr(), norm_w.data_ptr(),
        _opt(router_w, "router_w", (H, E), _F32S, device),
        _opt(router_logits, "router_logits", (T, E), _F32S, device),
        _opt(router_bias, "router_bias", (E,), _F32S, device),
        _opt(topk_ids, "topk_ids", (T, k), _I32S, device), _opt(topk_w, "topk_w", (T, k), _F32S, device),
        w13.data_ptr(), w2.data_ptr(), _opt(w13_scale, "w13_scale", s13, _F32S, device),
        _opt(w2_scale, "w2_scale", s2, _F32S, device), None if tail is None else tail.ref,
        out.data_ptr(), out.dtype == torch.float32,
        _opt(topk_ids_out, "topk_ids_out", (T, k), _I32S, device),
        _opt(topk_w_out, "topk_w_out", (T, k), _F32S, device), _ws_ptr(workspace),
        _ws_bytes(workspace), _stream(stream)))
    return out


def moe_quantize_fp8_rows(x, q, scale, stream=None):
    cols = x.shape[-1]
    rows = x.numel() // cols
    _check(lib.moe_quantize_fp8_rows(_ptr(x), rows, cols, _ptr(q), _ptr(scale), _stream(stream)))
    return q, scale


def moe_quantize_fp8_blocks(x, q, scale, block_rows, stream=None):
    """Block-wise E4M3 quantisation of x bf16 [..., K] viewed as [N, K]:
    q uint8 [N, K], scale fp32 [N / block_rows, K / 128] (block_rows 1 or 128)."""
    K = x.shape[-1]
    N = x.numel() // K if x.numel() else 0
    _check(lib.moe_quantize_fp8_blocks(_ptr(x), N, K, block_rows, _ptr(q), _ptr(scale),
                                       _stream(stream)))
    return q, scale


# --------------------------------------------- around the experts, and training --

# The checks of these calls cost as much host time as a small call's kernel takes, so each
# tensor's are one expression that also ends in its pointer.

_cur_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


_INT32 = 0x7fffffff


def _fits(*sizes):
    """ValueError unless each fits the int32 of the C entry points; ctypes would cut it off without a word.  (The calls
    below look at the sizes' bits together first: an or of two or three costs a tenth of this.)"""
    for v in sizes:
        if not -_INT32 <= v <= _INT32:
            raise ValueError(f"size {v}: does not fit an int32")


def _arg(t, name, shape, dtypes, index):
    """Pointer of a checked tensor on CUDA device `index`."""
    if t.dtype in dtypes and t.shape == shape and t.get_device() == index and t.is_contiguous():
        return t.data_ptr()
    _check_tensor(t, name, shape, dtypes, torch.device("cuda", index))
    return t.data_ptr()


def _queue(t, stream):
    """Device index of t and the call's stream; ValueError unless t is on the current device."""
    index = t.get_device()
    if index < 0 or index != _cur_device():
        _check_current(t.device)
    if stream is None and _raw_stream is not None:
        return index, _raw_stream(index)
    return index, _stream(stream)


def _ws(workspace, index):
    if workspace.get_device() != index:
        raise ValueError(f"workspace: on {workspace.device}, need cuda:{index}")
    if not workspace.is_contiguous():
        return _ws_ptr(workspace), _ws_bytes(workspace)
    p = workspace.data_ptr()
    q = (p + 255) & ~255
    return q, max(0, workspace.numel() - (q - p))


def _pairs(row_of_pair, n, index):
    if row_of_pair.numel() != n:
        raise ValueError(f"row_of_pair: {row_of_pair.numel()} entries, need {n}")
    return _arg(row_of_pair, "row_of_pair", row_of_pair.shape, _I32S, index)


def moe_unpermute(y, row_of_pair, out, T, k, topk_w=None, residual=None, stream=None):
    """out = residual + each token's expert rows times their routing weights.  y bf16 / fp32
    [T*k, H] in expert order, row_of_pair int32 [T*k] of moe_permute (negative: dropped), topk_w
    fp32 [T, k] (None: all 1), residual and out bf16 / fp32 [T, H]; residual may be out."""
    H = y.shape[-1]
    if T | k | H > _INT32:
        _fits(T, k, H)
    index, st = _queue(y, stream)
    _check(lib.moe_unpermute(
        _arg(y, "y", (T * k, H), _FLOATS, index), y.dtype == torch.bfloat16, _pairs(row_of_pair, T * k, index),
        None if topk_w is None else _arg(topk_w, "topk_w", (T, k), _F32S, index), T, k, H,
        None if residual is None else _arg(residual, "residual", (T, H), _FLOATS, index),
        residual is not None and residual.dtype == torch.float32, _arg(out, "out", (T, H), _FLOATS, index),
        out.dtype == torch.float32, st))
    return out


def moe_unpermute_backward(dout, y, row_of_pair, topk_w, T, k, dy=None, dw=None, ids=None, dlogits=None,
                           stream=None):
    """Gradients of moe_unpermute from dout bf16 / fp32 [T, H]: dy [T*k, H] (y's type, bf16 or fp32
    without y; rows that no pair owns are left as they were), dw fp32 [T, k], and with ids int32 [T, k] the
    router's dlogits fp32 [T, E].  y is needed for dw and dlogits; dy may be y."""
    H = dout.shape[-1]
    yt = y if y is not None else dy
    if dy is not None and y is not None and dy.dtype != y.dtype:
        raise ValueError(f"dy: dtype {dy.dtype}, need {y.dtype}")
    if dlogits is not None and dlogits.dim() != 2:
        raise ValueError("dlogits: must be [T, E]")
    E = 0 if dlogits is None else dlogits.shape[1]
    if T | k | H | E > _INT32:
        _fits(T, k, H, E)
    index, st = _queue(dout, stream)
    _check(lib.moe_unpermute_backward(
        _arg(dout, "dout", (T, H), _FLOATS, index), dout.dtype == torch.float32,
        None if y is None else _arg(y, "y", (T * k, H), _FLOATS, index), yt is None or yt.dtype == torch.bfloat16,
        _pairs(row_of_pair, T * k, index), _arg(topk_w, "topk_w", (T, k), _F32S, index),
        None if ids is None else _arg(ids, "ids", (T, k), _I32S, index), T, k, H, E,
        None if dy is None else _arg(dy, "dy", (T * k, H), _FLOATS, index),
        None if dw is None else _arg(dw, "dw", (T, k), _F32S, index),
        None if dlogits is None else _arg(dlogits, "dlogits", (T, E), _F32S, index), st))


def moe_permute_backward(dxp, row_of_pair, dx, T, k, dres=None, stream=None):
    """Gradient of moe_permute's gather: dx = dres + the sum of each token's rows of dxp (bf16 / fp32
    [T*k, H], expert order).  dres and dx bf16 / fp32 [T, H]; dres may be dx."""
    H = dxp.shape[-1]
    if T | k | H > _INT32:
        _fits(T, k, H)
    index, st = _queue(dxp, stream)
    _check(lib.moe_permute_backward(
        _arg(dxp, "dxp", (T * k, H), _FLOATS, index), dxp.dtype == torch.bfloat16,
        _pairs(row_of_pair, T * k, index), T, k, H,
        None if dres is None else _arg(dres, "dres", (T, H), _FLOATS, index),
        dres is not None and dres.dtype == torch.float32, _arg(dx, "dx", (T, H), _FLOATS, index),
        dx.dtype == torch.float32, st))
    return dx


def moe_layernorm(x, w, eps, y, b=None, mean=None, rstd=None, stream=None):
    """y = (x - mean) * rstd * w + b over the rows of x bf16 / fp32 [T, H]; w, b bf16 / fp32 [H] of one
    type; y bf16 / fp32 [T, H]; mean, rstd fp32 [T] for the backward pass."""
    shape = x.shape
    T, H = shape
    if T | H > _INT32:
        _fits(T, H)
    index, st = _queue(x, stream)
    wt = w.dtype
    _check(lib.moe_layernorm(
        _arg(x, "x", shape, _FLOATS, index), x.dtype == torch.float32, _arg(w, "w", (H,), _FLOATS, index),
        None if b is None else _arg(b, "b", (H,), (wt,), index), wt == torch.float32, T, H, eps,
        _arg(y, "y", shape, _FLOATS, index), y.dtype == torch.float32,
        None if mean is None else _arg(mean, "mean", (T,), _F32S, index),
        None if rstd is None else _arg(rstd, "rstd", (T,), _F32S, index), st))
    return y


def moe_norm_backward_workspace_size(T, H) -> int:
    _fits(T, H)
    n = lib.moe_norm_backward_workspace_size(T, H)
    if n == 0:
        raise MoeError(2, last_error())
    return n


def moe_layernorm_backward(dy, x, w, mean, rstd, dx, dw, workspace, db=None, dres=None, stream=None):
    """Gradients of moe_layernorm: dx [T, H] of x's type (plus dres, of the same type), dw and db fp32
    [H]; mean and rstd of the forward call, workspace of moe_norm_backward_workspace_size(T, H) bytes.
    dx may be x, dres, or dy of the same type."""
    shape, xt = x.shape, (x.dtype,)
    T, H = shape
    if T | H > _INT32:
        _fits(T, H)
    index, st = _queue(x, stream)
    _check(lib.moe_layernorm_backward(
        _arg(dy, "dy", shape, _FLOATS, index), dy.dtype == torch.float32, _arg(x, "x", shape, _FLOATS, index),
        x.dtype == torch.float32, _arg(w, "w", (H,), _FLOATS, index), w.dtype == torch.float32,
        _arg(mean, "mean", (T,), _F32S, index), _arg(rstd, "rstd", (T,), _F32S, index),
        None if dres is None else _arg(dres, "dres", shape, xt, index), T, H, _arg(dx, "dx", shape, xt, index),
        _arg(dw, "dw", (H,), _F32S, index), None if db is None else _arg(db, "db", (H,), _F32S, index),
        *_ws(workspace, index), st))
    return dx


def moe_rmsnorm_backward(dy, x, w, eps, dx, dw, workspace, dres=None, stream=None):
    """Gradients of moe_rmsnorm: dx [T, H] of x's type (plus dres), dw fp32 [H]; the rest as
    moe_layernorm_backward."""
    shape, xt = x.shape, (x.dtype,)
    T, H = shape
    if T | H > _INT32:
        _fits(T, H)
    index, st = _queue(x, stream)
    _check(lib.moe_rmsnorm_backward(
        _arg(dy, "dy", shape, _FLOATS, index), dy.dtype == torch.float32, _arg(x, "x", shape, _FLOATS, index),
        x.dtype == torch.float32, _arg(w, "w", (H,), _FLOATS, index), w.dtype == torch.float32, eps,
        None if dres is None else _arg(dres, "dres", shape, xt, index), T, H, _arg(dx, "dx", shape, xt, index),
        _arg(dw, "dw", (H,), _F32S, index), *_ws(workspace, index), st))
    return dx


def moe_linear(x, w, out, bias=None, residual=None, act=ACT_NONE, pre=None, stream=None):
    """out = residual + act(x w^T + bias).  x bf16 [M, K], w bf16 [N, K], bias bf16 / fp32 [N], residual
    and out bf16 / fp32 [M, N] (residual may be out), act one of the ACT_ constants; pre bf16 [M, N]
    receives the values before the activation."""
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w: must be [M, K] and [N, K]")
    (m, k), n = x.shape, w.shape[0]
    if m | n | k | act > _INT32:
        _fits(m, n, k, act)
    index, st = _queue(x, stream)
    _check(lib.moe_linear(
        _arg(x, "x", (m, k), _BF16, index), _arg(w, "w", (n, k), _BF16, index),
        None if bias is None else _arg(bias, "bias", (n,), _FLOATS, index),
        bias is not None and bias.dtype == torch.float32,
        None if residual is None else _arg(residual, "residual", (m, n), _FLOATS, index),
        residual is not None and residual.dtype == torch.float32, m, n, k, act,
        None if pre is None else _arg(pre, "pre", (m, n), _BF16, index),
        _arg(out, "out", (m, n), _FLOATS, index), out.dtype == torch.float32, st))
    return out


def moe_linear_backward_workspace_size(M, N, K) -> int:
    _fits(M, N, K)
    n = lib.moe_linear_backward_workspace_size(M, N, K)
    if n == 0:
        raise MoeError(2, last_error())
    return n


def moe_linear_backward(dout, x, w, workspace, dx=None, dw=None, db=None, pre=None, act=ACT_NONE, stream=None):
    """Gradients of moe_linear from dout bf16 / fp32 [M, N]: dx bf16 [M, K], dw bf16 / fp32 [N, K], db fp32
    [N], each where it is given; pre of the forward call with an activation; workspace of
    moe_linear_backward_workspace_size(M, N, K) bytes."""
    if x.dim() != 2 or w.dim() != 2:
        raise ValueError("x and w: must be [M, K] and [N, K]")
    (m, k), n = x.shape, w.shape[0]
    if m | n | k | act > _INT32:
        _fits(m, n, k, act)
    index, st = _queue(dout, stream)
    _check(lib.moe_linear_backward(
        _arg(dout, "dout", (m, n), _FLOATS, index), dout.dtype == torch.float32,
        None if pre is None else _arg(pre, "pre", (m, n), _BF16, index), _arg(x, "x", (m, k), _BF16, index),
        _arg(w, "w", (n, k), _BF16, index), m, n, k, act,
        None if dx is None else _arg(dx, "dx", (m, k), _BF16, index),
        None if dw is None else _arg(dw, "dw", (n, k), _FLOATS, index),
        dw is not None and dw.dtype == torch.float32, None if db is None else _arg(db, "db", (n,), _F32S, index),
        *_ws(workspace, index), st))
