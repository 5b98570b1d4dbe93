"""Python binding for libwq: the W8A8 dynamic-quant linear and the FP8 per-token-group
quant with packed UE8M0 scales, hand-written for MI355X (gfx950).

Argument marshalling only: every step runs in the HIP kernels behind the C ABI in
``include/wq.h``; PyTorch supplies device memory and the current stream.  There is no
fallback: if libwq.so is missing or the device is not gfx950, calls raise.

The functions carry the C names:
  wq_dynamic_quant(x, ...)                -> (x_q int8 [M,K], x_scale f32 [M])
  wq_group_quant_fp8_ue8m0(x)             -> (x_q uint8 [T,G,D], x_s int32 view [T,G,PH], storage [G,PH,TA])
  wq_quant_matmul(a, a_scale, b, b_scale) -> y bf16 [M,N]   (INT8 dense / segments, FP8 groups)
  wq_fused_quant_matmul(x, w, w_scale)    -> y bf16 [M,N]
  wq_moe_sort(ids, E)                     -> (perm, row_token, offsets)
  wq_group_quant_mxfp4(x)                 -> (x_q uint8 [T,G,D/2], x_s int32 view [T,G,PH], storage [G,PH,TA])
  wq_group_dequant_mxfp4(x_q, storage)    -> bf16 [T,G,D]
  wq_kv_append(cache, k, v, ...)             quantises rows into a paged 8-bit cache (KvCache)
  wq_kv_attention(cache, q, ...)          -> bf16 [T, heads, D] (and lse)
"""

from __future__ import annotations

import ctypes
import os
from typing import NamedTuple

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libwq.so")

WQ_OK = 0
WQ_IN_BF16, WQ_IN_F32 = 1, 2
WQ_PAYLOAD_INT8, WQ_PAYLOAD_FP8_E4M3, WQ_PAYLOAD_MXFP8 = 1, 2, 3
WQ_PAYLOAD_MXFP4, WQ_PAYLOAD_MXFP8_W4 = 4, 5
WQ_KV_E4M3, WQ_KV_INT8 = 1, 2
WQ_EPI_BF16, WQ_EPI_SWIGLU_F32 = 1, 2
WQ_LAYOUT_PLAIN, WQ_LAYOUT_FRAGMENT = 0, 1

_c_void_p = ctypes.c_void_p
_i64 = ctypes.c_int64


class WqError(RuntimeError):
    def __init__(self, fn: str, status: int):
        super().__init__(f"{fn} failed: status {status} ({lib().wq_status_str(status).decode()})")
        self.status = status


class MatmulDesc(ctypes.Structure):
    _fields_ = [
        ("payload", ctypes.c_int32), ("epilogue", ctypes.c_int32),
        ("M", _i64), ("N", _i64), ("K", _i64), ("batch", _i64),
        ("seg_offsets", _c_void_p),
        ("a", _c_void_p), ("lda", _i64), ("a_batch_stride", _i64),
        ("a_scale", _c_void_p), ("a_scale_tokens", _i64),
        ("b", _c_void_p), ("b_batch_stride", _i64),
        ("b_scale", _c_void_p),
        ("y", _c_void_p), ("ldy", _i64), ("y_batch_stride", _i64),
        ("acc_out", _c_void_p),
        ("b_layout", ctypes.c_int32),
        ("expected_rows", _i64),
    ]


class KvCacheDesc(ctypes.Structure):
    _fields_ = [
        ("code", ctypes.c_int32),
        ("pages", _i64), ("heads", _i64), ("page_tokens", _i64), ("head_dim", _i64),
        ("k", _c_void_p), ("v", _c_void_p), ("k_scale", _c_void_p), ("v_scale", _c_void_p),
        ("table", _c_void_p), ("table_stride", _i64), ("max_pages", _i64),
    ]


EXPORTS = {
    "wq_status_str": (ctypes.c_char_p, [ctypes.c_int]),
    "wq_abi_version": (ctypes.c_int, []),
    "wq_workspace_bytes": (ctypes.c_size_t, []),
    "wq_ctx_create": (ctypes.c_int, [ctypes.c_int, _c_void_p, ctypes.c_size_t, ctypes.POINTER(_c_void_p)]),
    "wq_ctx_destroy": (None, [_c_void_p]),
    "wq_ctx_set_split": (ctypes.c_int, [_c_void_p, ctypes.c_int]),
    "wq_ctx_set_fused_shape": (ctypes.c_int, [_c_void_p, ctypes.c_int, ctypes.c_int]),
    "wq_dynamic_quant": (ctypes.c_int, [_c_void_p, _c_void_p, ctypes.c_int, _i64, _i64, _i64, _c_void_p,
                                        ctypes.c_float, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "wq_group_quant_fp8_ue8m0": (ctypes.c_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p,
                                                _c_void_p]),
    "wq_quant_matmul": (ctypes.c_int, [_c_void_p, ctypes.POINTER(MatmulDesc), _c_void_p]),
    "wq_fused_quant_matmul": (ctypes.c_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _i64,
                                             _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "wq_moe_sort": (ctypes.c_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p, _c_void_p,
                                   _c_void_p]),
    "wq_fused_path": (ctypes.c_int, [_c_void_p, _i64, _i64, _i64]),
    "wq_group_quant_mxfp8": (ctypes.c_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p,
                                            _c_void_p]),
    "wq_group_quant_mxfp4": (ctypes.c_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p,
                                            _c_void_p]),
    "wq_group_dequant_mxfp4": (ctypes.c_int, [_c_void_p, _c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p,
                                              _c_void_p]),
    "wq_kv_append": (ctypes.c_int, [_c_void_p, ctypes.POINTER(KvCacheDesc), _c_void_p, _i64, _c_void_p, _i64, _i64,
                                    _i64, _c_void_p, _c_void_p, _c_void_p]),
    "wq_kv_attention": (ctypes.c_int, [_c_void_p, ctypes.POINTER(KvCacheDesc), _c_void_p, _i64, _i64, _i64, _i64,
                                       _c_void_p, _c_void_p, ctypes.c_float, ctypes.c_int, _c_void_p, _i64,
                                       _c_void_p, _c_void_p, ctypes.c_size_t, _c_void_p]),
    "wq_kv_attention_workspace_bytes": (_i64, [_c_void_p, ctypes.POINTER(KvCacheDesc), _i64, _i64, _i64]),
    "wq_kv_attention_path": (ctypes.c_int, [_c_void_p, ctypes.POINTER(KvCacheDesc), _i64, _i64, _i64]),
    "wq_mx4_path": (ctypes.c_int, [_c_void_p, _i64, _i64, _i64, _i64]),
    "wq_pack_weight_i8": (ctypes.c_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p]),
    "wq_fused_quant_matmul_packed": (ctypes.c_int, [_c_void_p, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p,
                                                    _i64, _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p,
                                                    _c_void_p]),
    "wq_fused_quant_matmul_static": (ctypes.c_int, [ctypes.c_int, _c_void_p, _i64, _i64, _i64, _c_void_p, _c_void_p,
                                                    _i64, _c_void_p, _i64, _c_void_p, _c_void_p, _c_void_p,
                                                    _c_void_p]),
}

_LIB = None


def lib() -> ctypes.CDLL:
    """Load libwq.so (built by fp8_dynamic_quant_amd.build); raise if it is missing."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run `python -m fp8_dynamic_quant_amd.build` first")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in EXPORTS.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        _LIB = L
    return _LIB


class Context:
    """One libwq context per device; owns its zero-initialised workspace tensor."""

    def __init__(self, device: torch.device):
        L = lib()
        self.device = device
        self.workspace = torch.zeros(int(L.wq_workspace_bytes()), dtype=torch.uint8, device=device)
        h = _c_void_p()
        st = L.wq_ctx_create(device.index, self.workspace.data_ptr(), self.workspace.numel(), ctypes.byref(h))
        if st != WQ_OK:
            raise WqError("wq_ctx_create", st)
        self.handle = h

    def __del__(self):
        try:
            if self.handle:
                lib().wq_ctx_destroy(self.handle)
        except Exception:
            pass


_CTX: dict[int, Context] = {}


def set_split(device, n: int) -> None:
    """Force the K-split factor of later calls on `device` (0 = automatic)."""
    _check("wq_ctx_set_split", lib().wq_ctx_set_split(context(device).handle, int(n)))


def set_fused_shape(device, rows_per_wg: int, cols_per_wg: int) -> None:
    """Force the one-launch fused kernel's rows and columns per workgroup on `device` (0 = automatic)."""
    _check("wq_ctx_set_fused_shape",
           lib().wq_ctx_set_fused_shape(context(device).handle, int(rows_per_wg), int(cols_per_wg)))


def context(device) -> Context:
    device = torch.device(device)
    if device.type != "cuda":
        raise RuntimeError("libwq runs on the GPU only; got a tensor on " + str(device))
    idx = device.index if device.index is not None else torch.cuda.current_device()
    if idx not in _CTX:
        _CTX[idx] = Context(torch.device("cuda", idx))
    return _CTX[idx]


def _stream(device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _on(fn, first, *others):
    """(context handle, raw current stream) of the device that all the tensors are on.  The calls
    that decode steps make take this way: the public stream object costs 2 us, these lookups 0.2."""
    idx = first.get_device()
    for t in others:
        if t.get_device() != idx:
            raise ValueError(f"{fn}: tensors on {first.device} and {t.device}")
    ctx = _CTX.get(idx)
    if ctx is None:
        ctx = context(first.device)
    return ctx.handle, torch._C._cuda_getCurrentRawStream(idx)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _check(fn, st):
    if st != WQ_OK:
        raise WqError(fn, st)


# ------------------------------------------------------------------------------------


def wq_dynamic_quant(x: torch.Tensor, rms_gamma: torch.Tensor | None = None, rms_eps: float = 1e-6,
                     row_index: torch.Tensor | None = None, x_q: torch.Tensor | None = None,
                     x_scale: torch.Tensor | None = None):
    """Per-token INT8 quant of x [*, K] (bf16 or f32, unit stride along K).  With
    row_index, output row r reads input row row_index[r]; with rms_gamma an RMSNorm runs
    first.  Returns (x_q int8 [M, K], x_scale f32 [M])."""
    if x.dim() != 2 or x.stride(1) != 1:
        raise ValueError("x must be 2-D with unit stride along K")
    if x.dtype not in (torch.bfloat16, torch.float32):
        raise ValueError("x must be bf16 or f32")
    M = row_index.numel() if row_index is not None else x.shape[0]
    K = x.shape[1]
    ctx = context(x.device)
    if x_q is None:
        x_q = torch.empty((M, K), dtype=torch.int8, device=x.device)
    if x_scale is None:
        x_scale = torch.empty((M,), dtype=torch.float32, device=x.device)
    st = lib().wq_dynamic_quant(ctx.handle, _ptr(x), WQ_IN_F32 if x.dtype == torch.float32 else WQ_IN_BF16, M, K,
                                x.stride(0), _ptr(rms_gamma), float(rms_eps), _ptr(row_index), _ptr(x_q),
                                _ptr(x_scale), _stream(x.device))
    _check("wq_dynamic_quant", st)
    return x_q, x_scale


def packed_scale_dims(T: int, D: int, group: int = 128):
    HG = D // group
    return HG, (HG + 3) // 4, (T + 3) // 4 * 4


def wq_group_quant_fp8_ue8m0(x: torch.Tensor, x_q: torch.Tensor | None = None, storage: torch.Tensor | None = None,
                             group: int = 128):
    """x bf16 [T, G, D] contiguous -> (x_q uint8 [T, G, D] E4M3FN codes,
    x_s int32 logical view [T, G, PH] with strides (1, PH*TA, TA), storage [G, PH, TA]).
    x_q / storage may be passed in (contiguous, those shapes) instead of allocated.
    group=32: the MX-like 32-element blocks (wq_group_quant_mxfp8)."""
    if x.dim() != 3 or not x.is_contiguous() or x.dtype != torch.bfloat16:
        raise ValueError("x must be a contiguous bf16 [T, G, D] tensor")
    if group not in (128, 32):
        raise ValueError("group must be 128 or 32")
    T, G, D = x.shape
    _, PH, TA = packed_scale_dims(T, D, group)
    ctx = context(x.device)
    if x_q is None:
        x_q = torch.empty((T, G, D), dtype=torch.uint8, device=x.device)
    if storage is None:
        storage = torch.empty((G, PH, TA), dtype=torch.int32, device=x.device)
    if tuple(x_q.shape) != (T, G, D) or not x_q.is_contiguous() or tuple(storage.shape) != (G, PH, TA) \
            or not storage.is_contiguous() or storage.dtype != torch.int32:
        raise ValueError("x_q must be uint8 [T, G, D] and storage int32 [G, PH, TA], both contiguous")
    if x.numel() > 0:
        fn = "wq_group_quant_fp8_ue8m0" if group == 128 else "wq_group_quant_mxfp8"
        st = getattr(lib(), fn)(ctx.handle, _ptr(x), T, G, D, _ptr(x_q), _ptr(storage), _stream(x.device))
        _check(fn, st)
    x_s = storage.transpose(-1, -2)[:, :T, :].transpose(0, 1)
    return x_q, x_s, storage


def wq_group_quant_mxfp4(x: torch.Tensor, x_q: torch.Tensor | None = None, storage: torch.Tensor | None = None):
    """x bf16 [T, G, D] contiguous, D % 32 == 0 -> (x_q uint8 [T, G, D/2], two E2M1 codes to a
    byte, x_s int32 logical view [T, G, PH], storage [G, PH, TA]), one UE8M0 scale for 32
    elements.  Weights [N, K] are cast as x = w[:, None, :]."""
    if x.dim() != 3 or not x.is_contiguous() or x.dtype != torch.bfloat16:
        raise ValueError("x must be a contiguous bf16 [T, G, D] tensor")
    T, G, D = x.shape
    if D % 32:
        raise ValueError("D must be a multiple of 32")
    PH, TA = (D + 127) // 128, (T + 3) // 4 * 4
    if x_q is None:
        x_q = x.new_empty((T, G, D // 2), dtype=torch.uint8)
    elif x_q.shape != (T, G, D // 2) or x_q.dtype != torch.uint8 or not x_q.is_contiguous():
        raise ValueError("x_q must be contiguous uint8 [T, G, D/2]")
    if storage is None:
        storage = x.new_empty((G, PH, TA), dtype=torch.int32)
    elif storage.shape != (G, PH, TA) or storage.dtype != torch.int32 or not storage.is_contiguous():
        raise ValueError("storage must be contiguous int32 [G, PH, TA]")
    h, stream = _on("wq_group_quant_mxfp4", x, x_q, storage)
    st = lib().wq_group_quant_mxfp4(h, x.data_ptr(), T, G, D, x_q.data_ptr(), storage.data_ptr(), stream)
    if st:
        _check("wq_group_quant_mxfp4", st)
    return x_q, storage.as_strided((T, G, PH), (1, PH * TA, TA)), storage


def wq_group_dequant_mxfp4(x_q: torch.Tensor, storage: torch.Tensor, y: torch.Tensor | None = None):
    """The values of wq_group_quant_mxfp4's codes: bf16 [T, G, D], exact."""
    if x_q.dim() != 3 or x_q.dtype != torch.uint8 or not x_q.is_contiguous():
        raise ValueError("x_q must be a contiguous uint8 [T, G, D/2] tensor")
    T, G, D = x_q.shape[0], x_q.shape[1], 2 * x_q.shape[2]
    if D % 32:
        raise ValueError("D must be a multiple of 32")
    if storage.shape != (G, (D + 127) // 128, (T + 3) // 4 * 4) or storage.dtype != torch.int32 \
            or not storage.is_contiguous():
        raise ValueError("storage must be contiguous int32 [G, PH, TA]")
    if y is None:
        y = x_q.new_empty((T, G, D), dtype=torch.bfloat16)
    elif y.shape != (T, G, D) or y.dtype != torch.bfloat16 or not y.is_contiguous():
        raise ValueError("y must be contiguous bf16 [T, G, D]")
    h, stream = _on("wq_group_dequant_mxfp4", x_q, storage, y)
    st = lib().wq_group_dequant_mxfp4(h, x_q.data_ptr(), storage.data_ptr(), T, G, D, y.data_ptr(), stream)
    if st:
        _check("wq_group_dequant_mxfp4", st)
    return y


def _mx4_matmul(a, a_scale, b, b_scale, G, y):
    if a.dim() != 3 or b.dim() != 3 or a_scale.dim() != 3 or b_scale.dim() != 3 or a.dtype != torch.uint8 \
            or b.dtype != torch.uint8 or a_scale.dtype != torch.int32 or b_scale.dtype != torch.int32:
        raise ValueError("a must be uint8 [M, G, K/2] or [M, G, K], b uint8 [G, N, K/2], their scales int32 storages")
    M, Ga, row = a.shape
    Gb, N, half = b.shape
    K = 2 * half
    TA = a_scale.shape[2]
    if Ga != G or Gb != G or (row != half and row != K):
        raise ValueError("a and b must hold fp8_groups groups of K/2 bytes (E2M1 pairs) or, a, K bytes (E4M3)")
    sa, sb = a.stride(), b.stride()
    if sa[2] != 1 or sb[2] != 1 or (N > 1 and sb[1] != half):
        raise ValueError("a's and b's rows must be dense, b's consecutive")
    kt = (K + 127) // 128
    if a_scale.shape != (G, kt, TA) or TA < (M + 3) // 4 * 4 or not a_scale.is_contiguous() or b_scale.shape != (G, kt, N) \
            or not b_scale.is_contiguous():
        raise ValueError("a_scale must be contiguous [G, K/128, align4(M) or more] and b_scale [G, K/128, N]")
    if y is None:
        y = a.new_empty((M, G, N), dtype=torch.bfloat16)
        sy = (G * N, N)
    else:
        if y.shape != (M, G, N) or y.dtype != torch.bfloat16 or y.stride(2) != 1:
            raise ValueError("y must be bf16 [M, G, N] with unit stride along N")
        sy = y.stride()
    h, stream = _on("wq_quant_matmul", a, a_scale, b, b_scale, y)
    # a stride of an axis of length one says nothing: the descriptor takes the dense one
    d = MatmulDesc(WQ_PAYLOAD_MXFP8_W4 if row == K else WQ_PAYLOAD_MXFP4, WQ_EPI_BF16, M, N, K, G, None, a.data_ptr(),
                   sa[0] if M > 1 else row, sa[1] if G > 1 else 0, a_scale.data_ptr(), TA, b.data_ptr(),
                   sb[0] if G > 1 else 0, b_scale.data_ptr(), y.data_ptr(), sy[0] if M > 1 else N,
                   sy[1] if G > 1 else 0, None, WQ_LAYOUT_PLAIN, 0)
    st = lib().wq_quant_matmul(h, ctypes.byref(d), stream)
    if st:
        _check("wq_quant_matmul", st)
    return y


def wq_quant_matmul(a, a_scale, b, b_scale, *, y=None, acc_out=None, seg_offsets=None,
                    epilogue=WQ_EPI_BF16, fp8_groups=None, a_scale_tokens=0, b_fragment=False, n=None,
                    mx=False, mx4=False, expected_rows=0):
    """INT8: a int8 [M, K] (row stride a.stride(0)), a_scale f32 [M], b int8 [N, K] (or
    [E, N, K] with seg_offsets int64 [E+1]), b_scale f32 [N] (or [E, N]) -> y.
    FP8 (fp8_groups=G): a uint8 [M, G, K], a_scale = packed storage [G, PH, TA],
    b uint8 [G, N, K], b_scale f32 [G, N/128, K/128] -> y bf16 [M, G, N].
    mx (with fp8_groups): the MX-like 32-element blocks: a_scale = storage of
    wq_group_quant_mxfp8 [G, K/128, TA], b_scale = UE8M0 bytes uint8 [G, N, K/32].
    mx4 (with fp8_groups): 4-bit weights, b uint8 [G, N, K/2] and b_scale int32 [G, K/128, N]
    as wq_group_quant_mxfp4 casts each group's w[:, None, :]; a uint8 [M, G, K/2] of
    wq_group_quant_mxfp4 or [M, G, K] of wq_group_quant_fp8_ue8m0(group=32), a_scale its storage.
    b_fragment: INT8 weights cast by wq_pack_weight_i8: expert weights [E, N, K] (same shape
    and strides) with seg_offsets, or a dense [N, K] cast (flat N*K bytes; give n = N) at
    M < 256 (K % 512 == 0, K <= 4096).
    expected_rows: with seg_offsets, the rows per expert the caller expects (a kernel-choice
    hint; the same bytes for every value)."""
    if mx4:
        if fp8_groups is None or acc_out is not None or seg_offsets is not None or epilogue != WQ_EPI_BF16 or b_fragment:
            raise ValueError("mx4 takes fp8_groups, and no acc_out, segments, SwiGLU epilogue or fragment order")
        if mx or (a_scale_tokens and a_scale_tokens != a_scale.shape[-1]) or (n is not None and n != b.shape[-2]):
            raise ValueError("mx4 is not mx, and takes a_scale_tokens and n from the operands' shapes")
        return _mx4_matmul(a, a_scale, b, b_scale, fp8_groups, y)
    d = MatmulDesc()
    d.b_layout = WQ_LAYOUT_FRAGMENT if b_fragment else WQ_LAYOUT_PLAIN
    d.expected_rows = expected_rows
    dev = a.device
    if fp8_groups is not None:
        G = fp8_groups
        M, Ga, K = a.shape
        N = b.shape[1]
        if y is None:
            y = torch.empty((M, G, N), dtype=torch.bfloat16, device=dev)
        d.payload, d.epilogue = (WQ_PAYLOAD_MXFP8 if mx else WQ_PAYLOAD_FP8_E4M3), WQ_EPI_BF16
        d.M, d.N, d.K, d.batch = M, N, K, G
        d.a, d.lda, d.a_batch_stride = _ptr(a), a.stride(0), a.stride(1)
        d.a_scale, d.a_scale_tokens = _ptr(a_scale), a_scale.shape[2]
        d.b, d.b_batch_stride, d.b_scale = _ptr(b), b.stride(0), _ptr(b_scale)
        d.y, d.ldy, d.y_batch_stride = _ptr(y), y.stride(0), y.stride(1)
    else:
        M, K = a.shape
        if b.dim() == 1:
            if not b_fragment or n is None:
                raise ValueError("a flat b is a fragment-order cast: pass b_fragment=True and n")
            N = n
        else:
            N = b.shape[-2]
        batch = b.shape[0] if b.dim() == 3 else 1
        ncols = N // 2 if epilogue == WQ_EPI_SWIGLU_F32 else N
        if y is None:
            y = torch.empty((M, ncols), dtype=torch.float32 if epilogue == WQ_EPI_SWIGLU_F32 else torch.bfloat16,
                            device=dev)
        d.payload, d.epilogue = WQ_PAYLOAD_INT8, epilogue
        d.M, d.N, d.K, d.batch = M, N, K, batch
        d.seg_offsets = _ptr(seg_offsets)
        d.a, d.lda, d.a_scale = _ptr(a), a.stride(0), _ptr(a_scale)
        d.b, d.b_batch_stride, d.b_scale = _ptr(b), (b.stride(0) if b.dim() == 3 else 0), _ptr(b_scale)
        d.y, d.ldy = _ptr(y), y.stride(0)
        d.acc_out = _ptr(acc_out)
    ctx = context(dev)
    _check("wq_quant_matmul", lib().wq_quant_matmul(ctx.handle, ctypes.byref(d), _stream(dev)))
    return y


class KvCache(NamedTuple):
    """A paged 8-bit cache (wq.h): codes uint8 (E4M3) or int8, k [pages, heads, page_tokens, D]
    and v [pages, heads, D, page_tokens], and their UE8M0 bytes [pages, heads]."""

    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor


def kv_cache(pages: int, heads: int, page_tokens: int, head_dim: int, *, dtype=torch.uint8, device="cuda") -> KvCache:
    """A zeroed cache: dtype torch.uint8 for E4M3 codes, torch.int8 for int8."""
    return KvCache(torch.zeros((pages, heads, page_tokens, head_dim), dtype=dtype, device=device),
                   torch.zeros((pages, heads, head_dim, page_tokens), dtype=dtype, device=device),
                   torch.zeros((pages, heads), dtype=torch.uint8, device=device),
                   torch.zeros((pages, heads), dtype=torch.uint8, device=device))


def _kv_desc(cache, offsets, lens, table):
    k, v, ks, vs = cache
    if k.dim() != 4 or (k.dtype != torch.uint8 and k.dtype != torch.int8) or v.dtype != k.dtype:
        raise ValueError("a cache's codes are uint8 (E4M3) or int8, k [pages, heads, page_tokens, D]")
    pages, heads, page_tokens, D = k.shape
    if v.shape != (pages, heads, D, page_tokens) or ks.shape != (pages, heads) or vs.shape != (pages, heads) \
            or ks.dtype != torch.uint8 or vs.dtype != torch.uint8:
        raise ValueError("a cache has v [pages, heads, D, page_tokens] and uint8 k_scale, v_scale [pages, heads]")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError("a cache's tensors must be contiguous")
    if offsets.dtype != torch.int64 or lens.dtype != torch.int32 or table.dtype != torch.int32:
        raise ValueError("offsets are int64, lens and table int32")
    B = lens.numel()
    if lens.dim() != 1 or offsets.shape != (B + 1,) or table.dim() != 2 or not offsets.is_contiguous() \
            or not lens.is_contiguous():
        raise ValueError("offsets must be [B + 1], lens [B] and table [B, pages of a sequence]")
    Bt, width = table.shape
    ts = table.stride()
    if Bt != B or (width > 1 and ts[1] != 1):
        raise ValueError("table must be [B, pages of a sequence] with dense rows")
    return KvCacheDesc(WQ_KV_INT8 if k.dtype == torch.int8 else WQ_KV_E4M3, pages, heads, page_tokens, D, k.data_ptr(),
                       v.data_ptr(), ks.data_ptr(), vs.data_ptr(), table.data_ptr(), ts[0] if B > 1 else width, width), B


def _kv_rows(name, x, heads, D):
    """Row stride of bf16 rows [T, heads, D] whose last two axes are dense."""
    if x.dim() != 3 or x.dtype != torch.bfloat16 or x.shape[1] != heads or x.shape[2] != D:
        raise ValueError(f"{name} must be bf16 [T, {heads}, {D}]")
    s = x.stride()
    if x.shape[0] and (s[2] != 1 or (heads > 1 and s[1] != D)):
        raise ValueError(f"{name} must have dense rows")
    return s[0] if x.shape[0] > 1 else heads * D


def wq_kv_append(cache: KvCache, k: torch.Tensor, v: torch.Tensor, offsets, lens, table) -> None:
    """Quantise the rows k, v bf16 [T, heads, D] into the cache, in place.  offsets int64
    [B + 1]: rows of each sequence; lens int32 [B]: its tokens, these rows among them; table
    int32 [B, pages of a sequence]."""
    d, B = _kv_desc(cache, offsets, lens, table)
    ldk, ldv = _kv_rows("k", k, d.heads, d.head_dim), _kv_rows("v", v, d.heads, d.head_dim)
    T = k.shape[0]
    if v.shape[0] != T:
        raise ValueError("k and v must have the same number of rows")
    h, stream = _on("wq_kv_append", k, v, *cache, offsets, lens, table)
    st = lib().wq_kv_append(h, ctypes.byref(d), k.data_ptr(), ldk, v.data_ptr(), ldv, T, B, offsets.data_ptr(),
                            lens.data_ptr(), stream)
    if st:
        _check("wq_kv_append", st)


def wq_kv_attention(cache: KvCache, q: torch.Tensor, offsets, lens, table, *, scale=None, causal=True, out=None,
                    lse=None, return_lse=False):
    """Attention of the rows q bf16 [T, q_heads, D] over the cache (offsets, lens and table as
    in wq_kv_append, the newest rows last) -> bf16 [T, q_heads, D], and the f32 log-sum-exp
    [T, q_heads] with return_lse or lse=.  scale: 1 / sqrt(D) by default."""
    d, B = _kv_desc(cache, offsets, lens, table)
    if q.dim() != 3:
        raise ValueError("q must be bf16 [T, q_heads, D]")
    T, heads, D = q.shape
    ldq = _kv_rows("q", q, heads, d.head_dim)
    if out is None:
        out, ldo = q.new_empty((T, heads, D)), heads * D
    else:
        if out.dim() != 3 or out.shape[0] != T:
            raise ValueError("out must have q's shape")
        ldo = _kv_rows("out", out, heads, D)
    if lse is not None:
        if lse.shape != (T, heads) or lse.dtype != torch.float32 or not lse.is_contiguous():
            raise ValueError("lse must be contiguous f32 [T, q_heads]")
    elif return_lse:
        lse = q.new_empty((T, heads), dtype=torch.float32)
    h, stream = _on("wq_kv_attention", q, *cache, offsets, lens, table, out, *(() if lse is None else (lse,)))
    by = ctypes.byref(d)
    need = lib().wq_kv_attention_workspace_bytes(h, by, T, heads, B)
    if need < 0:
        _check("wq_kv_attention", -need)
    # from torch's allocator, call by call: calls on several streams and captured graphs share nothing
    ws = q.new_empty(need, dtype=torch.uint8) if need else None
    st = lib().wq_kv_attention(h, by, q.data_ptr(), ldq, T, heads, B, offsets.data_ptr(), lens.data_ptr(),
                               D ** -0.5 if scale is None else scale, causal, out.data_ptr(), ldo, _ptr(lse), _ptr(ws),
                               need, stream)
    if st:
        _check("wq_kv_attention", st)
    return (out, lse) if lse is not None else out


def wq_kv_attention_path(cache: KvCache, T: int, q_heads: int, table) -> int:
    """Which kernels wq_kv_attention takes for T rows of q_heads heads (the numbers stand in wq.h)."""
    pages, heads, page_tokens, D = cache.k.shape
    d = KvCacheDesc(WQ_KV_E4M3, pages, heads, page_tokens, D, None, None, None, None, None, table.shape[1], table.shape[1])
    r = lib().wq_kv_attention_path(context(cache.k.device).handle, ctypes.byref(d), T, q_heads, table.shape[0])
    if r < 0:
        _check("wq_kv_attention_path", -r)
    return r


def wq_mx4_path(M: int, N: int, K: int, groups: int = 1, device=None) -> int:
    """Which kernel a product on 4-bit weights takes (the numbers stand in wq.h)."""
    r = lib().wq_mx4_path(context(device if device is not None else "cuda").handle, M, N, K, groups)
    if r < 0:
        _check("wq_mx4_path", -r)
    return r


def wq_fused_quant_matmul(x, w, w_scale, *, y=None, x_q_out=None, x_scale_out=None, acc_out=None):
    """x bf16 [M, K], w int8 [N, K], w_scale f32 [N] -> y bf16 [M, N] in one launch."""
    if x.dim() != 2 or x.stride(1) != 1 or x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16 [M, K] with unit stride along K")
    M, K = x.shape
    N = w.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    ctx = context(x.device)
    st = lib().wq_fused_quant_matmul(ctx.handle, _ptr(x), M, K, x.stride(0), _ptr(w), _ptr(w_scale), N, _ptr(y),
                                     y.stride(0), _ptr(x_q_out), _ptr(x_scale_out), _ptr(acc_out),
                                     _stream(x.device))
    _check("wq_fused_quant_matmul", st)
    return y


def wq_fused_quant_matmul_static(x, w, w_scale, *, y=None, x_q_out=None, x_scale_out=None, acc_out=None):
    """wq_fused_quant_matmul through the allocation-free entry point (no context, the library's
    static staging buffer); y is allocated here unless given."""
    if x.dim() != 2 or x.stride(1) != 1 or x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16 [M, K] with unit stride along K")
    M, K = x.shape
    N = w.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    idx = x.device.index if x.device.index is not None else torch.cuda.current_device()
    st = lib().wq_fused_quant_matmul_static(idx, _ptr(x), M, K, x.stride(0), _ptr(w), _ptr(w_scale), N, _ptr(y),
                                            y.stride(0), _ptr(x_q_out), _ptr(x_scale_out), _ptr(acc_out),
                                            _stream(x.device))
    _check("wq_fused_quant_matmul_static", st)
    return y


def wq_pack_weight_i8(w, wp=None):
    """int8 w [N, K] (unit stride along K) -> the same bytes in fragment order (wq.h), as a
    flat int8 tensor of N*K bytes for wq_fused_quant_matmul_packed.  For expert weights
    [E, N, K] (contiguous) each expert is cast in place of its own [N, K] block: the result
    has w's shape, for wq_quant_matmul(..., seg_offsets=..., b_fragment=True)."""
    if w.dim() == 3:
        if not w.is_contiguous() or w.dtype != torch.int8:
            raise ValueError("expert weights must be contiguous int8 [E, N, K]")
        out = torch.empty_like(w) if wp is None else wp
        for e in range(w.shape[0]):
            wq_pack_weight_i8(w[e], out[e].view(-1))
        return out
    if w.dim() != 2 or w.stride(1) != 1 or w.dtype != torch.int8:
        raise ValueError("w must be int8 [N, K] with unit stride along K")
    N, K = w.shape
    if wp is None:
        wp = torch.empty((N * K,), dtype=torch.int8, device=w.device)
    ctx = context(w.device)
    _check("wq_pack_weight_i8", lib().wq_pack_weight_i8(ctx.handle, _ptr(w), N, K, w.stride(0), _ptr(wp),
                                                         _stream(w.device)))
    return wp


def wq_fused_quant_matmul_packed(x, wp, w_scale, N, *, y=None, x_q_out=None, x_scale_out=None, acc_out=None):
    """x bf16 [M, K], wp from wq_pack_weight_i8 (N*K bytes), w_scale f32 [N] -> y bf16 [M, N]."""
    if x.dim() != 2 or x.stride(1) != 1 or x.dtype != torch.bfloat16:
        raise ValueError("x must be bf16 [M, K] with unit stride along K")
    M, K = x.shape
    if wp.numel() != N * K:
        raise ValueError("wp must hold N*K bytes")
    if y is None:
        y = torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    ctx = context(x.device)
    st = lib().wq_fused_quant_matmul_packed(ctx.handle, _ptr(x), M, K, x.stride(0), _ptr(wp), _ptr(w_scale), N,
                                            _ptr(y), y.stride(0), _ptr(x_q_out), _ptr(x_scale_out), _ptr(acc_out),
                                            _stream(x.device))
    _check("wq_fused_quant_matmul_packed", st)
    return y


FUSED_PATHS = {0: "quant kernel + GEMM (two launches)", 1: "one launch: dot4 GEMV", 2: "one launch: 8-wave MFMA"}


def wq_fused_path(M: int, K: int, N: int, device=None) -> int:
    """Launch sequence wq_fused_quant_matmul takes for these sizes (see FUSED_PATHS)."""
    ctx = context(device or torch.device("cuda", torch.cuda.current_device()))
    r = lib().wq_fused_path(ctx.handle, M, K, N)
    if r < 0:
        _check("wq_fused_path", -r)
    return r


def wq_moe_sort(ids: torch.Tensor, num_experts: int):
    """ids int32 [T, topk] -> (perm int32 [T*topk], row_token int32 [T*topk], offsets int64 [E+1])."""
    T, topk = ids.shape
    dev = ids.device
    perm = torch.empty(T * topk, dtype=torch.int32, device=dev)
    row_token = torch.empty(T * topk, dtype=torch.int32, device=dev)
    offsets = torch.empty(num_experts + 1, dtype=torch.int64, device=dev)
    ctx = context(dev)
    st = lib().wq_moe_sort(ctx.handle, _ptr(ids.contiguous()), T, topk, num_experts, _ptr(perm), _ptr(row_token),
                           _ptr(offsets), _stream(dev))
    _check("wq_moe_sort", st)
    return perm, row_token, offsets
