"""GB300-native block-scaled MoE top-k expert layer (A8W4 / A4W4).

A thin ctypes binding over ``libmoe_topk.so`` (the C ABI declared in
``include/moe_topk.h``).  Every function here only marshals torch tensors to
device pointers and sizes and raises on a non-zero status; every step of the
layer runs in the library's CUDA kernels.  There is no fallback: if the
library is missing the functions raise.
"""
from __future__ import annotations

import ctypes
import os

import torch

__all__ = [
    "MoeError", "MOE_ACT_MXFP8", "MOE_ACT_MXFP4", "MOE_SCHEDULE_AUTO", "MOE_SCHEDULE_CHAIN", "MOE_SCHEDULE_FUSED",
    "MOE_SCHEDULE_CHAIN_BF16_H", "MOE_SCHEDULE_CHAIN_SINGLE_CTA", "MOE_SCHEDULE_CHAIN_FP8_Y2", "lib", "moe_status_string", "moe_workspace_bytes",
    "moe_get_workspace_layout", "moe_topk_route", "moe_sort_by_expert", "moe_sort_by_expert_noalloc",
    "moe_quantize_mx", "moe_a8w4_forward",
    "moe_a4w4_forward", "moe_forward_ex", "moe_a8w4_forward_prequant", "moe_a4w4_forward_prequant", "moe_prepack_scales", "moe_a8w4_forward_prepacked", "moe_a4w4_forward_prepacked",
    "moe_read_device_status", "moe_forward_launch_count", "moe_forward_launch_count_ex", "moe_forward_launch_count_cfg",
    "moe_forward_split_gemms", "moe_profile_forward",
    "workspace_views",
    "MOE_DTYPE_BF16", "MOE_DTYPE_F16", "MOE_DTYPE_F32", "MOE_DTYPE_U8", "moe_permute", "moe_permute_backward",
    "moe_unpermute", "moe_unpermute_backward", "moe_topk_route_backward", "moe_quantize_fp8_block",
    "moe_permute_quantize_fp8_block", "moe_gemm_fp8_block_workspace_bytes", "moe_gemm_fp8_block",
    "moe_gemm_fp8_block_dgrad",
    "MOE_GATE_UP_INTERLEAVED", "MOE_GATE_UP_STACKED", "moe_rms_norm", "moe_rms_norm_quantize_fp8_block",
    "moe_rms_norm_quantize_mx", "moe_rms_norm_backward_workspace_bytes", "moe_rms_norm_backward",
    "moe_swiglu_backward", "moe_gemm_fp8_block_swiglu",
]

MOE_ACT_MXFP8 = 0
MOE_ACT_MXFP4 = 1
MOE_SCHEDULE_AUTO = 0   # the library's choice for the shape and T
MOE_SCHEDULE_CHAIN = 1  # kernel chain, one CTA per 128 x 256 GEMM tile over the whole K
MOE_SCHEDULE_FUSED = 2  # T <= 64: the whole layer in one persistent kernel
MOE_SCHEDULE_CHAIN_BF16_H = 3  # kernel chain, GEMM1 writes bf16 h, a separate kernel requantises
MOE_SCHEDULE_CHAIN_SINGLE_CTA = 4  # kernel chain with single-CTA GEMM tiles only (no pair split)
MOE_SCHEDULE_CHAIN_FP8_Y2 = 5  # kernel chain, GEMM2 rows travel as weighted E4M3 + E8M0 scales
MOE_DTYPE_BF16 = 0
MOE_DTYPE_F16 = 1
MOE_DTYPE_F32 = 2
MOE_DTYPE_U8 = 3  # moe_permute only: rows of bytes
MOE_GATE_UP_INTERLEAVED = 0  # rows (columns of the products) 2j gate, 2j + 1 up
MOE_GATE_UP_STACKED = 1      # [0, I) gate, [I, 2I) up
_DTYPES = {torch.bfloat16: MOE_DTYPE_BF16, torch.float16: MOE_DTYPE_F16, torch.float32: MOE_DTYPE_F32,
           torch.uint8: MOE_DTYPE_U8}
LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libmoe_topk.so")

STATUS_NAMES = {
    0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED_SHAPE", 3: "MOE_ERR_UNSUPPORTED_DEVICE",
    4: "MOE_ERR_WORKSPACE_TOO_SMALL", 5: "MOE_ERR_CUDA", 6: "MOE_ERR_DEVICE_TIMEOUT", 7: "MOE_ERR_MISALIGNED",
}


class MoeError(RuntimeError):
    def __init__(self, status: int, where: str):
        super().__init__(f"{where}: {STATUS_NAMES.get(status, status)}")
        self.status = status


class WorkspaceLayout(ctypes.Structure):
    _fields_ = [(n, ctypes.c_size_t) for n in (
        "status", "sync", "topk_ids", "topk_w", "counts", "offsets", "padded_offsets", "mtile_base", "chunk_hist",
        "sorted_pair", "inv", "inv_padded", "xq", "xs", "a2", "a2s", "y2", "sf_rot", "part", "y2f", "total")] + [
        ("rows_cap", ctypes.c_int64), ("nchunk", ctypes.c_int64)]


class ForwardArgs(ctypes.Structure):
    _fields_ = [("act_fmt", ctypes.c_int), ("prequantized", ctypes.c_int), ("weight_scales_prepacked", ctypes.c_int),
                ("x", ctypes.c_void_p), ("x_scale", ctypes.c_void_p), ("gate_logits", ctypes.c_void_p),
                ("w1", ctypes.c_void_p), ("w1_scale", ctypes.c_void_p), ("w2", ctypes.c_void_p),
                ("w2_scale", ctypes.c_void_p), ("out", ctypes.c_void_p), ("T", ctypes.c_int64), ("H", ctypes.c_int),
                ("I", ctypes.c_int), ("E", ctypes.c_int), ("k", ctypes.c_int), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t), ("stream", ctypes.c_void_p), ("schedule", ctypes.c_int)]


_lib = None


def lib():
    """Load libmoe_topk.so (built in-tree by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"{LIB_PATH} is missing: build it with __graft_entry__.build() "
                           "(there is no non-CUDA fallback)")
    L = ctypes.CDLL(LIB_PATH)
    P, i64, i32, sz = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
    L.moe_status_string.restype = ctypes.c_char_p
    L.moe_status_string.argtypes = [i32]
    L.moe_get_workspace_layout.restype = i32
    L.moe_get_workspace_layout.argtypes = [i64, i32, i32, i32, i32, i32, ctypes.POINTER(WorkspaceLayout)]
    L.moe_workspace_bytes.restype = sz
    L.moe_workspace_bytes.argtypes = [i64, i32, i32, i32, i32, i32]
    L.moe_topk_route.restype = i32
    L.moe_topk_route.argtypes = [P, i64, i32, i32, P, P, P]
    L.moe_sort_by_expert.restype = i32
    L.moe_sort_by_expert.argtypes = [P, i64, i32, i32, P, P, P, P, P, sz, P]
    L.moe_quantize_mx.restype = i32
    L.moe_quantize_mx.argtypes = [P, i64, i32, i32, P, P, P]
    for name in ("moe_a8w4_forward", "moe_a4w4_forward", "moe_a8w4_forward_prepacked",
                 "moe_a4w4_forward_prepacked"):
        f = getattr(L, name)
        f.restype = i32
        f.argtypes = [P, P, P, P, P, P, P, i64, i32, i32, i32, i32, P, sz, P]
    L.moe_read_device_status.restype = i32
    L.moe_read_device_status.argtypes = [P, P, ctypes.POINTER(ctypes.c_int)]
    L.moe_forward_launch_count.restype = i32
    L.moe_forward_launch_count.argtypes = [i64, i32, i32]
    L.moe_forward_launch_count_ex.restype = i32
    L.moe_forward_launch_count_ex.argtypes = [i64, i32, i32, i32]
    L.moe_forward_launch_count_cfg.restype = i32
    L.moe_forward_launch_count_cfg.argtypes = [i64, i32, i32, i32, i32, i32, i32, i32]
    L.moe_forward_split_gemms.restype = i32
    L.moe_forward_split_gemms.argtypes = [i64, i32, i32, i32, i32, i32, i32, i32]
    L.moe_profile_forward.restype = i32
    L.moe_profile_forward.argtypes = [i32, P, P, P, P, P, P, P, i64, i32, i32, i32, i32, P, sz, P, i32, i32,
                                      ctypes.POINTER(ctypes.c_float)]
    for name in ("moe_a8w4_forward_prequant", "moe_a4w4_forward_prequant"):
        f = getattr(L, name)
        f.restype = i32
        f.argtypes = [P, P, P, P, P, P, P, P, i64, i32, i32, i32, i32, P, sz, P]
    L.moe_forward_ex.restype = i32
    L.moe_forward_ex.argtypes = [ctypes.POINTER(ForwardArgs)]
    L.moe_prepack_scales.restype = i32
    L.moe_prepack_scales.argtypes = [P, i64, i32, P, P]
    L.moe_permute.argtypes = [P, i64, i32, P, i64, i32, i32, P, i64, i64, P]
    L.moe_permute_backward.argtypes = [P, i64, i64, i32, P, i64, i32, i32, P, i64, P]
    L.moe_unpermute.argtypes = [P, i64, i64, i32, P, P, i64, i32, i32, P, i64, P]
    L.moe_unpermute_backward.argtypes = [P, i64, P, i64, i64, i32, P, P, i64, i32, i32, P, i64, P, P]
    L.moe_topk_route_backward.argtypes = [P, P, P, i64, i32, i32, P, P]
    L.moe_quantize_fp8_block.argtypes = [P, i64, i32, i64, i32, i32, P, P, P]
    L.moe_permute_quantize_fp8_block.argtypes = [P, i64, i32, P, i64, i32, i32, P, P, i64, P]
    f32 = ctypes.c_float
    rows_in, rows_out = [P, i64, P, i64, i32, P, i32, f32, i64, i32], [P, i64, P, i64, P, P]
    L.moe_rms_norm.argtypes = rows_in + rows_out
    L.moe_rms_norm_quantize_fp8_block.argtypes = rows_in + [P, P] + rows_out
    L.moe_rms_norm_quantize_mx.argtypes = rows_in + [i32, P, P] + rows_out
    L.moe_rms_norm_backward_workspace_bytes.argtypes = [i64, i32]
    L.moe_rms_norm_backward_workspace_bytes.restype = sz
    L.moe_rms_norm_backward.argtypes = [P, i64, P, i64, P, i64, i32, P, i32, P, i64, i32, P, i64, P, P, sz, P]
    L.moe_swiglu_backward.argtypes = [P, i64, P, i64, i32, i32, i64, i32, P, i64, P, P, P]
    L.moe_gemm_fp8_block_swiglu.argtypes = [P, P, P, P, i32, P, i64, i32, i32, i32, P, P, i32, P, P, P, sz, P]
    L.moe_gemm_fp8_block_workspace_bytes.argtypes = [i64, i32, i32, i32]
    L.moe_gemm_fp8_block_workspace_bytes.restype = sz
    for name in ("moe_gemm_fp8_block", "moe_gemm_fp8_block_dgrad"):
        getattr(L, name).argtypes = [P, P, P, P, P, i64, i32, i32, i32, P, i32, P, sz, P]
    _lib = L
    return L


def _check(status: int, where: str):
    if status != 0:
        raise MoeError(status, where)


def _stream(stream):
    """The stream's handle; None: the current stream (torch.cuda.current_stream() builds a Stream
    object, 3 us a call; the raw handle costs 0.1)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _p(t):
    return ctypes.c_void_p(t.data_ptr())


def moe_status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def moe_get_workspace_layout(T, H, I, E, k, fmt=MOE_ACT_MXFP8) -> WorkspaceLayout:
    lay = WorkspaceLayout()
    _check(lib().moe_get_workspace_layout(int(T), int(H), int(I), int(E), int(k), int(fmt), ctypes.byref(lay)),
           "moe_get_workspace_layout")
    return lay


def moe_workspace_bytes(T, H, I, E, k, fmt=MOE_ACT_MXFP8) -> int:
    return int(lib().moe_workspace_bytes(int(T), int(H), int(I), int(E), int(k), int(fmt)))


def moe_forward_launch_count(T, H, I) -> int:
    return int(lib().moe_forward_launch_count(int(T), int(H), int(I)))


def moe_forward_launch_count_ex(T, H, I, schedule) -> int:
    return int(lib().moe_forward_launch_count_ex(int(T), int(H), int(I), int(schedule)))


def moe_forward_launch_count_cfg(T, H, I, E, k, fmt, schedule, prepacked_scales) -> int:
    return int(lib().moe_forward_launch_count_cfg(int(T), int(H), int(I), int(E), int(k), int(fmt), int(schedule),
                                                  int(bool(prepacked_scales))))


def moe_forward_split_gemms(T, H, I, E, k, fmt, schedule, prepacked_scales) -> int:
    return int(lib().moe_forward_split_gemms(int(T), int(H), int(I), int(E), int(k), int(fmt), int(schedule),
                                             int(bool(prepacked_scales))))


def moe_topk_route(gate_logits, k, topk_ids, topk_w, stream=None):
    """gate_logits fp32 [T, E] -> topk_ids int32 [T, k], topk_w fp32 [T, k] (outputs given)."""
    T, E = gate_logits.shape
    _check(lib().moe_topk_route(_p(gate_logits), T, E, int(k), _p(topk_ids), _p(topk_w), _stream(stream)),
           "moe_topk_route")


def moe_sort_by_expert(topk_ids, E, counts, offsets, sorted_pair, inv, workspace, stream=None):
    T, k = topk_ids.shape
    _check(lib().moe_sort_by_expert(_p(topk_ids), T, int(E), k, _p(counts), _p(offsets), _p(sorted_pair), _p(inv),
                                    _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream)),
           "moe_sort_by_expert")


def moe_sort_by_expert_noalloc(topk_ids, E, counts, offsets, sorted_pair, inv, stream=None):
    """moe_sort_by_expert for callers that cannot provide scratch memory: the library uses
    its own fixed 4 MiB device array instead of a workspace (see include/moe_topk.h)."""
    f = lib().moe_sort_by_expert_noalloc
    f.restype = ctypes.c_int
    f.argtypes = [ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p,
                  ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p]
    T, k = topk_ids.shape
    _check(f(_p(topk_ids), T, int(E), k, _p(counts), _p(offsets), _p(sorted_pair), _p(inv), _stream(stream)),
           "moe_sort_by_expert_noalloc")


def moe_quantize_mx(x, fmt, codes, scales, stream=None):
    rows, K = x.shape
    _check(lib().moe_quantize_mx(_p(x), rows, K, int(fmt), _p(codes), _p(scales), _stream(stream)),
           "moe_quantize_mx")


def _forward(name, x, gate_logits, w1, w1_scale, w2, w2_scale, out, E, k, workspace, stream):
    T, H = x.shape
    I = w2.shape[-1] * 2
    f = getattr(lib(), name)
    _check(f(_p(x), _p(gate_logits), _p(w1), _p(w1_scale), _p(w2), _p(w2_scale), _p(out), T, H, I, int(E), int(k),
             _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream)), name)


def moe_a8w4_forward(x, gate_logits, w1, w1_scale, w2, w2_scale, out, E, k, workspace, stream=None):
    """x bf16 [T, H], gate_logits fp32 [T, E], w1 u8 [E, 2I, H/2], w1_scale u8 [E, 2I, H/32],
    w2 u8 [E, H, I/2], w2_scale u8 [E, H, I/32] -> out bf16 [T, H]."""
    _forward("moe_a8w4_forward", x, gate_logits, w1, w1_scale, w2, w2_scale, out, E, k, workspace, stream)


def moe_a4w4_forward(x, gate_logits, w1, w1_scale, w2, w2_scale, out, E, k, workspace, stream=None):
    _forward("moe_a4w4_forward", x, gate_logits, w1, w1_scale, w2, w2_scale, out, E, k, workspace, stream)


def _forward_prequant(name, xq, xq_scale, gate_logits, w1, w1_scale, w2, w2_scale, out, E, k, workspace, stream):
    T, H = out.shape
    I = w2.shape[-1] * 2
    f = getattr(lib(), name)
    _check(f(_p(xq), _p(xq_scale), _p(gate_logits), _p(w1), _p(w1_scale), _p(w2), _p(w2_scale), _p(out), T, H, I,
             int(E), int(k), _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream)), name)


def moe_a8w4_forward_prequant(xq, xq_scale, gate_logits, w1, w1_scale, w2, w2_scale, out, E, k, workspace,
                              stream=None):
    """The A8W4 layer from prequantised activations: xq u8 [T, H] E4M3, xq_scale u8 [T, H/32]."""
    _forward_prequant("moe_a8w4_forward_prequant", xq, xq_scale, gate_logits, w1, w1_scale, w2, w2_scale, out, E, k,
                      workspace, stream)


def moe_a4w4_forward_prequant(xq, xq_scale, gate_logits, w1, w1_scale, w2, w2_scale, out, E, k, workspace,
                              stream=None):
    """The A4W4 layer from prequantised activations: xq u8 [T, H/2] E2M1, xq_scale u8 [T, H/32]."""
    _forward_prequant("moe_a4w4_forward_prequant", xq, xq_scale, gate_logits, w1, w1_scale, w2, w2_scale, out, E, k,
                      workspace, stream)


def moe_forward_ex(x, gate_logits, w1, w1_scale, w2, w2_scale, out, E, k, workspace, act_fmt=MOE_ACT_MXFP8,
                   x_scale=None, weight_scales_prepacked=False, stream=None, schedule=MOE_SCHEDULE_AUTO):
    """Any forward variant: bf16 x (x_scale None) or prequantised codes + scales; canonical or
    prepacked weight scales; the schedule (MOE_SCHEDULE_*)."""
    T, H = out.shape
    a = ForwardArgs(act_fmt=int(act_fmt), prequantized=int(x_scale is not None),
                    weight_scales_prepacked=int(bool(weight_scales_prepacked)), x=x.data_ptr(),
                    x_scale=None if x_scale is None else x_scale.data_ptr(), gate_logits=gate_logits.data_ptr(),
                    w1=w1.data_ptr(), w1_scale=w1_scale.data_ptr(), w2=w2.data_ptr(), w2_scale=w2_scale.data_ptr(),
                    out=out.data_ptr(), T=T, H=H, I=w2.shape[-1] * 2, E=int(E), k=int(k),
                    workspace=workspace.data_ptr(), workspace_bytes=workspace.numel() * workspace.element_size(),
                    stream=_stream(stream), schedule=int(schedule))
    _check(lib().moe_forward_ex(ctypes.byref(a)), "moe_forward_ex")


def moe_prepack_scales(scales, tiled, stream=None):
    """E8M0 scales [..., rows, K/32] (any leading dims) -> 128x4 tile layout into ``tiled`` (same bytes)."""
    K = scales.shape[-1] * 32
    rows = scales.numel() // (K // 32)
    _check(lib().moe_prepack_scales(_p(scales), rows, K, _p(tiled), _stream(stream)), "moe_prepack_scales")


def moe_a8w4_forward_prepacked(x, gate_logits, w1, w1_scale_tiled, w2, w2_scale_tiled, out, E, k, workspace,
                               stream=None):
    """moe_a8w4_forward with both weight-scale tensors prepacked by moe_prepack_scales."""
    _forward("moe_a8w4_forward_prepacked", x, gate_logits, w1, w1_scale_tiled, w2, w2_scale_tiled, out, E, k,
             workspace, stream)


def moe_a4w4_forward_prepacked(x, gate_logits, w1, w1_scale_tiled, w2, w2_scale_tiled, out, E, k, workspace,
                               stream=None):
    _forward("moe_a4w4_forward_prepacked", x, gate_logits, w1, w1_scale_tiled, w2, w2_scale_tiled, out, E, k,
             workspace, stream)


KERNEL_NAMES = ("route", "scan", "scatter", "quant", "gemm1", "gemm2", "combine")
KERNEL_NAMES_SMALL = ("route_sort", "quant", "gemm1", "gemm2", "combine")  # kernel chain, T <= 64
KERNEL_NAMES_FUSED = ("decode",)  # fused schedule
KERNEL_NAMES_BF16_H = ("route", "scan", "scatter", "quant", "gemm1", "requant", "gemm2", "combine")
KERNEL_NAMES_BF16_H_SMALL = ("route_sort", "quant", "gemm1", "requant", "gemm2", "combine")


def moe_profile_forward(fmt, x, gate_logits, w1, w1_scale, w2, w2_scale, out, E, k, workspace, stream=None,
                        prepacked_scales=False, schedule=MOE_SCHEDULE_AUTO):
    """One forward with a CUDA event between kernels; returns {kernel name: microseconds}."""
    T, H = x.shape
    I = w2.shape[-1] * 2
    n = moe_forward_launch_count_cfg(T, H, I, E, k, fmt, schedule, prepacked_scales)
    split = moe_forward_split_gemms(T, H, I, E, k, fmt, schedule, prepacked_scales)
    us = (ctypes.c_float * max(n, 1))()
    _check(lib().moe_profile_forward(int(fmt), _p(x), _p(gate_logits), _p(w1), _p(w1_scale), _p(w2), _p(w2_scale),
                                     _p(out), T, H, I, int(E), int(k), _p(workspace),
                                     workspace.numel() * workspace.element_size(), _stream(stream),
                                     int(bool(prepacked_scales)), int(schedule), us),
           "moe_profile_forward")
    n_base = n - bin(max(split, 0)).count("1")
    if schedule == MOE_SCHEDULE_CHAIN_BF16_H:
        names = KERNEL_NAMES_BF16_H if n_base == len(KERNEL_NAMES_BF16_H) else KERNEL_NAMES_BF16_H_SMALL
    else:
        names = {len(KERNEL_NAMES): KERNEL_NAMES, len(KERNEL_NAMES_SMALL): KERNEL_NAMES_SMALL,
                 1: KERNEL_NAMES_FUSED}[n_base]
    # a split GEMM: its pair kernel, then its tail pass
    expand = {"gemm1": ("gemm1_pairs", "gemm1_tails") if split & 1 else ("gemm1",),
              "gemm2": ("gemm2_pairs", "gemm2_tails") if split & 2 else ("gemm2",)}
    names = [m for nm in names for m in expand.get(nm, (nm,))]
    assert len(names) == n
    return {names[i]: float(us[i]) for i in range(n)}


def moe_read_device_status(workspace, stream=None) -> int:
    st = ctypes.c_int(0)
    _check(lib().moe_read_device_status(_p(workspace), _stream(stream), ctypes.byref(st)), "moe_read_device_status")
    return int(st.value)


def workspace_views(workspace, T, H, I, E, k, fmt=MOE_ACT_MXFP8):
    """Typed views of the forward's intermediates inside a uint8 workspace tensor."""
    L = moe_get_workspace_layout(T, H, I, E, k, fmt)
    R = T * k
    hb = H if fmt == MOE_ACT_MXFP8 else H // 2
    ib = I if fmt == MOE_ACT_MXFP8 else I // 2
    rc = L.rows_cap

    def v(off, n, dtype):
        nbytes = n * torch.empty((), dtype=dtype).element_size()
        return workspace[off:off + nbytes].view(dtype)

    return dict(
        layout=L,
        topk_ids=v(L.topk_ids, R, torch.int32).view(T, k), topk_w=v(L.topk_w, R, torch.float32).view(T, k),
        counts=v(L.counts, E, torch.int32), offsets=v(L.offsets, E + 1, torch.int64),
        padded_offsets=v(L.padded_offsets, E + 1, torch.int64), mtile_base=v(L.mtile_base, E + 1, torch.int32),
        sorted_pair=v(L.sorted_pair, R, torch.int32), inv=v(L.inv, R, torch.int32),
        inv_padded=v(L.inv_padded, R, torch.int32), xq=v(L.xq, rc * hb, torch.uint8).view(rc, hb),
        xs=v(L.xs, rc * H // 32, torch.uint8), a2=v(L.a2, rc * ib, torch.uint8).view(rc, ib),
        a2s=v(L.a2s, rc * I // 32, torch.uint8), y2=v(L.y2, rc * H, torch.bfloat16).view(rc, H),
        status=v(L.status, 8, torch.int32))


# ---------------------------------------------------------------- expert rows and FP8 experts
# The C entry points see only pointers, so these bindings check what a pointer cannot tell: element
# types, shapes, strides and the device (MOE_ERR_INVALID_ARG naming the tensor): all tensors of a call on
# one GPU, which is the current one, whose stream the kernel runs on.  A decode step is a few
# microseconds on the GPU, so each binding makes one plain test of everything first; only when it fails
# do the _want / _matrix / _table checks run, which say what is wrong.  ``dev`` is the device of the call's
# first tensor (-1: the host).
_F32, _I32, _I64, _U8 = torch.float32, torch.int32, torch.int64, torch.uint8


def _want(ok: bool, where: str, what: str):
    if not ok:
        raise MoeError(1, f"{where}: {what}")


def _place(t, dev, where, name):
    d = t.get_device()
    _want(d >= 0, where, f"{name} must be on the GPU")
    _want(d == dev, where, f"{name} is on cuda:{d}, expected cuda:{dev}")


def _matrix(t, dev, where, name, shape, dtypes=None):
    """A row-major matrix on the GPU with unit column stride; None in ``shape``: any size."""
    _want(t is not None and t.dim() == 2, where, f"{name} must be a matrix")
    _want(all(n is None or n == m for n, m in zip(shape, t.shape)), where,
          f"{name} has shape {list(t.shape)}, expected {list(shape)}")
    _want(t.stride(1) == 1 or t.shape[1] <= 1, where, f"{name} must have unit column stride")
    _want(dtypes is None or t.dtype in dtypes, where, f"{name} has the unsupported type {t.dtype}")
    _place(t, dev, where, name)


def _table(t, dev, dtype, shape, where, name):
    _want(t is not None and t.dtype == dtype, where, f"{name} must be {dtype}")
    _want(len(t.shape) == len(shape) and all(n is None or n == m for n, m in zip(shape, t.shape)), where,
          f"{name} has shape {list(t.shape)}, expected {list(shape)}")
    _want(t.is_contiguous(), where, f"{name} must be contiguous")
    _place(t, dev, where, name)


_ROWS = {d: c for d, c in _DTYPES.items() if d is not torch.uint8}


def _fixed(t, dev, dtype):
    return t.dtype is dtype and t.get_device() == dev and t.is_contiguous()


def _row_stride(t, dev, shape):
    """Elements between rows, or 0 unless the matrix plainly has unit column stride and is on that GPU."""
    st = t.stride()
    if len(shape) != 2 or st[1] != 1 or dev < 0 or t.get_device() != dev:
        return 0
    return st[0] if shape[0] > 1 else max(st[0], shape[1])


def _stride(t):
    """Elements between rows of a matrix; overlapping rows are left for the library to refuse."""
    return t.stride(0) if t.shape[0] > 1 else max(t.stride(0), t.shape[1])


def _current_device():
    return torch._C._cuda_getDevice()


def _launch_stream(stream, dev, where):
    """The stream's handle, for a kernel over tensors of device ``dev``."""
    now = _current_device()
    if now != dev:
        raise MoeError(1, f"{where}: the tensors are on cuda:{dev}, the current device is cuda:{now}")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else _stream(stream)


def moe_permute(x, inv, rows, stream=None):
    """rows[inv[t, j]] = x[t]: x [T, H], inv int32 [T, k] (outside [0, R): dropped) -> rows [R, H]."""
    fn = "moe_permute"
    dt, sx, si, sr, dev = x.dtype, x.shape, inv.shape, rows.shape, inv.get_device()
    tx, tr = _row_stride(x, dev, sx), _row_stride(rows, dev, sr)
    if not (tx and tr and dt in _DTYPES and rows.dtype is dt and _fixed(inv, dev, _I32) and len(si) == 2 and
            si[0] == sx[0] and sr[1] == sx[1]):
        _table(inv, dev, _I32, (None, None), fn, "inv")
        _matrix(x, dev, fn, "x", (si[0], None), _DTYPES)
        _matrix(rows, dev, fn, "rows", (None, sx[1]), (dt,))
        tx, tr = _stride(x), _stride(rows)
    _check(lib().moe_permute(x.data_ptr(), tx, _DTYPES[dt], inv.data_ptr(), sx[0], sx[1], si[1], rows.data_ptr(), tr,
                             sr[0], _launch_stream(stream, dev, fn)), fn)


def moe_permute_backward(d_rows, inv, d_x, stream=None):
    """Gradient of moe_permute: d_x[t] = sum_j d_rows[inv[t, j]]."""
    fn = "moe_permute_backward"
    dt, sr, si, sx, dev = d_rows.dtype, d_rows.shape, inv.shape, d_x.shape, inv.get_device()
    tr, tx = _row_stride(d_rows, dev, sr), _row_stride(d_x, dev, sx)
    if not (tr and tx and dt in _ROWS and d_x.dtype is dt and _fixed(inv, dev, _I32) and len(si) == 2 and
            si[0] == sx[0] and sr[1] == sx[1]):
        _table(inv, dev, _I32, (None, None), fn, "inv")
        _matrix(d_rows, dev, fn, "d_rows", (None, None), _ROWS)
        _matrix(d_x, dev, fn, "d_x", (si[0], sr[1]), (dt,))
        tr, tx = _stride(d_rows), _stride(d_x)
    _check(lib().moe_permute_backward(d_rows.data_ptr(), tr, sr[0], _DTYPES[dt], inv.data_ptr(), sx[0], sx[1], si[1],
                                      d_x.data_ptr(), tx, _launch_stream(stream, dev, fn)), fn)


def moe_unpermute(rows, inv, topk_w, out, stream=None):
    """out[t] = sum_j topk_w[t, j] rows[inv[t, j]]: rows [R, H], topk_w fp32 [T, k] -> out [T, H]."""
    fn = "moe_unpermute"
    dt, sr, si, so, dev = rows.dtype, rows.shape, inv.shape, out.shape, inv.get_device()
    tr, to = _row_stride(rows, dev, sr), _row_stride(out, dev, so)
    if not (tr and to and dt in _ROWS and out.dtype is dt and _fixed(inv, dev, _I32) and len(si) == 2 and
            topk_w is not None and _fixed(topk_w, dev, _F32) and topk_w.shape == si and si[0] == so[0] and
            sr[1] == so[1]):
        _table(inv, dev, _I32, (None, None), fn, "inv")
        _matrix(rows, dev, fn, "rows", (None, None), _ROWS)
        _matrix(out, dev, fn, "out", (si[0], sr[1]), (dt,))
        _table(topk_w, dev, _F32, si, fn, "topk_w")
        tr, to = _stride(rows), _stride(out)
    _check(lib().moe_unpermute(rows.data_ptr(), tr, sr[0], _DTYPES[dt], inv.data_ptr(), topk_w.data_ptr(), so[0],
                               so[1], si[1], out.data_ptr(), to, _launch_stream(stream, dev, fn)), fn)


def moe_unpermute_backward(d_out, rows, inv, topk_w, d_rows, d_topk_w, stream=None):
    """Gradients of moe_unpermute: d_rows[inv[t, j]] = topk_w[t, j] d_out[t] and d_topk_w[t, j] =
    <d_out[t], rows[inv[t, j]]>.  Either result may be None; rows may be None without d_topk_w."""
    fn = "moe_unpermute_backward"
    dt, so, si, dev = d_out.dtype, d_out.shape, inv.shape, inv.get_device()
    to = _row_stride(d_out, dev, so)
    if not (to and dt in _ROWS and _fixed(inv, dev, _I32) and len(si) == 2 and si[0] == so[0] and
            topk_w is not None and _fixed(topk_w, dev, _F32) and topk_w.shape == si):
        _table(inv, dev, _I32, (None, None), fn, "inv")
        _matrix(d_out, dev, fn, "d_out", (si[0], None), _ROWS)
        _table(topk_w, dev, _F32, si, fn, "topk_w")
        to = _stride(d_out)
    R = rp = tr = dp = td = 0
    wp = None
    if d_rows is not None:
        sd = d_rows.shape
        td = _row_stride(d_rows, dev, sd)
        if not (td and d_rows.dtype is dt and sd[1] == so[1]):
            _matrix(d_rows, dev, fn, "d_rows", (None, so[1]), (dt,))
            td = _stride(d_rows)
        R, dp = sd[0], d_rows.data_ptr()
    if d_topk_w is not None:
        _want(rows is not None, fn, "d_topk_w needs rows")
        sr = rows.shape
        tr = _row_stride(rows, dev, sr)
        if not (tr and rows.dtype is dt and sr[1] == so[1] and (d_rows is None or sr[0] == R) and
                _fixed(d_topk_w, dev, _F32) and d_topk_w.shape == si):
            _matrix(rows, dev, fn, "rows", (None if d_rows is None else R, so[1]), (dt,))
            _table(d_topk_w, dev, _F32, si, fn, "d_topk_w")
            tr = _stride(rows)
        R, rp, wp = sr[0], rows.data_ptr(), d_topk_w.data_ptr()
    _check(lib().moe_unpermute_backward(d_out.data_ptr(), to, rp, tr, R, _DTYPES[dt], inv.data_ptr(),
                                        topk_w.data_ptr(), so[0], so[1], si[1], dp, td, wp,
                                        _launch_stream(stream, dev, fn)), fn)


def moe_topk_route_backward(topk_ids, topk_w, d_topk_w, d_logits, stream=None):
    """Gradient of moe_topk_route's weights: ids int32, topk_w and d_topk_w fp32 [T, k] -> d_logits fp32 [T, E]."""
    fn = "moe_topk_route_backward"
    si, sl, dev = topk_ids.shape, d_logits.shape, topk_ids.get_device()
    if not (dev >= 0 and _fixed(topk_ids, dev, _I32) and _fixed(topk_w, dev, _F32) and
            _fixed(d_topk_w, dev, _F32) and _fixed(d_logits, dev, _F32) and len(si) == 2 and len(sl) == 2 and
            topk_w.shape == si and d_topk_w.shape == si and si[0] == sl[0]):
        _table(topk_ids, dev, _I32, (None, None), fn, "topk_ids")
        _table(topk_w, dev, _F32, si, fn, "topk_w")
        _table(d_topk_w, dev, _F32, si, fn, "d_topk_w")
        _table(d_logits, dev, _F32, (si[0], None), fn, "d_logits")
    _check(lib().moe_topk_route_backward(topk_ids.data_ptr(), topk_w.data_ptr(), d_topk_w.data_ptr(), sl[0], sl[1],
                                         si[1], d_logits.data_ptr(), _launch_stream(stream, dev, fn)), fn)


def moe_quantize_fp8_block(x, codes, scales, block_rows=1, stream=None):
    """x [rows, K] -> E4M3 codes u8 [rows, K] and fp32 scales [ceil(rows / block_rows), ceil(K / 128)],
    block_rows = 1 or 128."""
    fn = "moe_quantize_fp8_block"
    _want(block_rows == 1 or block_rows == 128, fn, "block_rows must be 1 or 128")
    dt, sx, dev = x.dtype, x.shape, x.get_device()
    tx = _row_stride(x, dev, sx)
    if not (tx and dt in _ROWS and _fixed(codes, dev, _U8) and codes.shape == sx and _fixed(scales, dev, _F32) and
            scales.shape == ((sx[0] + block_rows - 1) // block_rows, (sx[1] + 127) // 128)):
        _matrix(x, dev, fn, "x", (None, None), _ROWS)
        _table(codes, dev, _U8, sx, fn, "codes")
        _table(scales, dev, _F32, (-(-sx[0] // block_rows), -(-sx[1] // 128)), fn, "scales")
        tx = _stride(x)
    _check(lib().moe_quantize_fp8_block(x.data_ptr(), tx, _DTYPES[dt], sx[0], sx[1], block_rows, codes.data_ptr(),
                                        scales.data_ptr(), _launch_stream(stream, dev, fn)), fn)


def moe_permute_quantize_fp8_block(x, inv, codes, scales, stream=None):
    """moe_permute and moe_quantize_fp8_block in one pass: codes u8 [R, K], scales fp32 [R, ceil(K / 128)]."""
    fn = "moe_permute_quantize_fp8_block"
    dt, sx, si, sc, dev = x.dtype, x.shape, inv.shape, codes.shape, inv.get_device()
    tx = _row_stride(x, dev, sx)
    if not (tx and dt in _ROWS and _fixed(inv, dev, _I32) and len(si) == 2 and si[0] == sx[0] and
            _fixed(codes, dev, _U8) and len(sc) == 2 and sc[1] == sx[1] and _fixed(scales, dev, _F32) and
            scales.shape == (sc[0], (sx[1] + 127) // 128)):
        _table(inv, dev, _I32, (None, None), fn, "inv")
        _matrix(x, dev, fn, "x", (si[0], None), _ROWS)
        _table(codes, dev, _U8, (None, sx[1]), fn, "codes")
        _table(scales, dev, _F32, (sc[0], (sx[1] + 127) // 128), fn, "scales")
        tx = _stride(x)
    _check(lib().moe_permute_quantize_fp8_block(x.data_ptr(), tx, _DTYPES[dt], inv.data_ptr(), sx[0], sx[1], si[1],
                                                codes.data_ptr(), scales.data_ptr(), sc[0],
                                                _launch_stream(stream, dev, fn)), fn)


def moe_gemm_fp8_block_workspace_bytes(M, N, K, E) -> int:
    return int(lib().moe_gemm_fp8_block_workspace_bytes(int(M), int(N), int(K), int(E)))


def _gemm_block(fn, dgrad, x, x_scale, w, w_scale, out, workspace, offsets, stream):
    dev, sx, dt = w.get_device(), x.shape, out.dtype
    if len(w.shape) != 3:
        _table(w, dev, _U8, (None, None, None), fn, "w")
    E, N, K = w.shape
    if not sx:
        _want(False, fn, "the codes have shape []")
    M = sx[0]
    inner, outer = (N, K) if dgrad else (K, N)
    if not (dev >= 0 and _fixed(w, dev, _U8) and _fixed(x, dev, _U8) and _fixed(x_scale, dev, _F32) and
            _fixed(w_scale, dev, _F32) and dt in _ROWS and _fixed(out, dev, dt) and
            workspace.get_device() == dev and sx == (M, inner) and out.shape == (M, outer) and
            x_scale.shape == (M, (inner + 127) // 128) and
            w_scale.shape == (E, (N + 127) // 128, (K + 127) // 128) and
            (offsets is None or _fixed(offsets, dev, _I64) and offsets.shape == (E + 1,))):
        _table(w, dev, _U8, (None, None, None), fn, "w")
        _table(w_scale, dev, _F32, (E, (N + 127) // 128, (K + 127) // 128), fn, "w_scale")
        _table(x, dev, _U8, (M, inner), fn, "the codes")
        _table(x_scale, dev, _F32, (M, (inner + 127) // 128), fn, "the codes' scales")
        _want(dt in _ROWS, fn, "the output must be bf16, f16 or f32")
        _table(out, dev, dt, (M, outer), fn, "the output")
        if offsets is not None:
            _table(offsets, dev, _I64, (E + 1,), fn, "offsets")
        _place(workspace, dev, fn, "the workspace")
    L = lib()
    _check((L.moe_gemm_fp8_block_dgrad if dgrad else L.moe_gemm_fp8_block)(
        x.data_ptr(), x_scale.data_ptr(), w.data_ptr(), w_scale.data_ptr(),
        None if offsets is None else offsets.data_ptr(), M, N, K, E, out.data_ptr(), _DTYPES[dt], workspace.data_ptr(),
        workspace.nbytes, _launch_stream(stream, dev, fn)), fn)


def moe_gemm_fp8_block(x, x_scale, w, w_scale, out, workspace, offsets=None, stream=None):
    """FP8 product with block scales: x u8 [M, K], x_scale fp32 [M, ceil(K/128)], w u8 [E, N, K], w_scale fp32
    [E, ceil(N/128), ceil(K/128)], offsets int64 [E + 1] (None: E = 1, all rows) -> out [M, N]."""
    _gemm_block("moe_gemm_fp8_block", False, x, x_scale, w, w_scale, out, workspace, offsets, stream)


def moe_gemm_fp8_block_dgrad(dy, dy_scale, w, w_scale, dx, workspace, offsets=None, stream=None):
    """Gradient of moe_gemm_fp8_block with respect to x: dy u8 [M, N], dy_scale fp32 [M, ceil(N/128)] -> dx [M, K]."""
    _gemm_block("moe_gemm_fp8_block_dgrad", True, dy, dy_scale, w, w_scale, dx, workspace, offsets, stream)


# ---------------------------------------------------------------- norms and gated blocks

def _rows_at(t, shape, dt, dev, where, name):
    """Pointer and row stride of a matrix of that shape and type; (None, 0) without one."""
    if t is None:
        return None, 0
    if t.dtype is dt and t.get_device() == dev and t.is_contiguous() and t.shape == shape:
        return t.data_ptr(), shape[1]
    _matrix(t, dev, where, name, shape, (dt,))
    return t.data_ptr(), _stride(t)


def _flat_at(t, shape, dt, dev, where, name):
    """Pointer of a contiguous tensor of that shape and type; None without one."""
    if t is None:
        return None
    if not (t.dtype is dt and t.get_device() == dev and t.is_contiguous() and t.shape == shape):
        _table(t, dev, dt, shape, where, name)
    return t.data_ptr()


def _norm_rows(fn, x, weight):
    """What a norm's rows and weight have to be: (shape, type, device, row stride, the weight's type)."""
    _want(weight is not None, fn, "weight is needed")
    sx, dt, dev, wt = x.shape, x.dtype, x.get_device(), weight.dtype
    if (dev >= 0 and len(sx) == 2 and dt in _ROWS and x.is_contiguous() and (wt is dt or wt is _F32) and
            weight.get_device() == dev and weight.is_contiguous() and weight.shape == sx[1:]):
        return sx, dt, dev, sx[1], wt
    _matrix(x, dev, fn, "x", (None, None), _ROWS)
    _want(wt in (dt, _F32), fn, f"weight has the unsupported type {wt}")
    _table(weight, dev, wt, (sx[1],), fn, "weight")
    return sx, dt, dev, _stride(x), wt


def _rms_norm(fn, call, x, weight, eps, fmt, codes, scales, out, residual, residual_out, rstd, stream):
    """``fmt``: None (values), -1 (FP8 block codes), or an MX format."""
    sx, dt, dev, tx, wt = _norm_rows(fn, x, weight)
    rp = op = sp = tp = None
    tr = to = ts = 0
    if residual is not None:
        rp, tr = _rows_at(residual, sx, dt, dev, fn, "residual")
    if out is not None:
        op, to = _rows_at(out, sx, dt, dev, fn, "out")
    if residual_out is not None:
        sp, ts = _rows_at(residual_out, sx, dt, dev, fn, "residual_out")
    if rstd is not None:
        tp = _flat_at(rstd, sx[:1], _F32, dev, fn, "rstd")
    T, H = sx
    xp, wp, d, w, stream = x.data_ptr(), weight.data_ptr(), _DTYPES[dt], _DTYPES[wt], _launch_stream(stream, dev, fn)
    if fmt is None:
        status = call(xp, tx, rp, tr, d, wp, w, eps, T, H, op, to, sp, ts, tp, stream)
    elif fmt < 0:
        status = call(xp, tx, rp, tr, d, wp, w, eps, T, H, codes, scales, op, to, sp, ts, tp, stream)
    else:
        status = call(xp, tx, rp, tr, d, wp, w, eps, T, H, fmt, codes, scales, op, to, sp, ts, tp, stream)
    if status:
        _check(status, fn)


def moe_rms_norm(x, weight, eps, out, residual=None, residual_out=None, rstd=None, stream=None):
    """out = weight * s / sqrt(mean(s^2) + eps) with s = x + residual: x, residual, out, residual_out (s) [T, H],
    weight [H] of x's type or fp32, rstd fp32 [T] (1 / sqrt(...), for the gradient)."""
    fn = "moe_rms_norm"
    _want(out is not None, fn, "out must be a matrix")
    _rms_norm(fn, lib().moe_rms_norm, x, weight, eps, None, None, None, out, residual, residual_out, rstd, stream)


def moe_rms_norm_quantize_fp8_block(x, weight, eps, codes, scales, out=None, residual=None, residual_out=None,
                                    rstd=None, stream=None):
    """moe_rms_norm with its result as E4M3 codes u8 [T, H] and fp32 scales [T, ceil(H / 128)], and in out too."""
    fn = "moe_rms_norm_quantize_fp8_block"
    _want(codes is not None and scales is not None, fn, "codes and scales are needed")
    sx, dev = x.shape, x.get_device()
    if len(sx) != 2 or dev < 0:
        _matrix(x, dev, fn, "x", (None, None), _ROWS)
    cp = _flat_at(codes, sx, _U8, dev, fn, "codes")
    sp = _flat_at(scales, (sx[0], (sx[1] + 127) // 128), _F32, dev, fn, "scales")
    _rms_norm(fn, lib().moe_rms_norm_quantize_fp8_block, x, weight, eps, -1, cp, sp, out, residual, residual_out, rstd,
              stream)


def moe_rms_norm_quantize_mx(x, weight, eps, fmt, codes, scales, out=None, residual=None, residual_out=None, rstd=None,
                             stream=None):
    """moe_rms_norm with its result as MX codes (fmt MOE_ACT_MXFP8: u8 [T, H], MOE_ACT_MXFP4: u8 [T, H / 2]) and E8M0
    scales u8 [T, H / 32], as the *_forward_prequant calls read them, and in out too."""
    fn = "moe_rms_norm_quantize_mx"
    _want(codes is not None and scales is not None, fn, "codes and scales are needed")
    _want(fmt in (MOE_ACT_MXFP8, MOE_ACT_MXFP4), fn, "fmt must be MOE_ACT_MXFP8 or MOE_ACT_MXFP4")
    sx, dev = x.shape, x.get_device()
    if len(sx) != 2 or dev < 0:
        _matrix(x, dev, fn, "x", (None, None), _ROWS)
    T, H = sx
    _want(H % 32 == 0, fn, "the rows' width must be a multiple of 32")
    cp = _flat_at(codes, (T, H if fmt == MOE_ACT_MXFP8 else H // 2), _U8, dev, fn, "codes")
    sp = _flat_at(scales, (T, H // 32), _U8, dev, fn, "scales")
    _rms_norm(fn, lib().moe_rms_norm_quantize_mx, x, weight, eps, fmt, cp, sp, out, residual, residual_out, rstd, stream)


def moe_rms_norm_backward_workspace_bytes(T, H) -> int:
    return int(lib().moe_rms_norm_backward_workspace_bytes(int(T), int(H)))


def moe_rms_norm_backward(dy, x, weight, rstd, dx, d_weight=None, workspace=None, d_residual=None, stream=None):
    """Gradients of moe_rms_norm from its sum x (residual_out) [T, H] and rstd fp32 [T]: dx [T, H], of x and residual
    alike, with d_residual [T, H] (what reaches residual_out from elsewhere) added; d_weight fp32 [H], which needs the
    workspace."""
    fn = "moe_rms_norm_backward"
    sx, dt, dev, tx, wt = _norm_rows(fn, x, weight)
    _want(dy is not None and dx is not None and rstd is not None, fn, "dy, rstd and dx are needed")
    yp, ty = _rows_at(dy, sx, dt, dev, fn, "dy")
    dp, td = _rows_at(dx, sx, dt, dev, fn, "dx")
    rp, tr = _rows_at(d_residual, sx, dt, dev, fn, "d_residual")
    sp = _flat_at(rstd, sx[:1], _F32, dev, fn, "rstd")
    wp = _flat_at(d_weight, sx[1:], _F32, dev, fn, "d_weight")
    space = size = None
    if wp is not None:
        _want(workspace is not None, fn, "d_weight needs the workspace")
        _place(workspace, dev, fn, "the workspace")
        space, size = workspace.data_ptr(), workspace.nbytes
    _check(lib().moe_rms_norm_backward(yp, ty, x.data_ptr(), tx, rp, tr, _DTYPES[dt], weight.data_ptr(), _DTYPES[wt],
                                       sp, sx[0], sx[1], dp, td, wp, space, size or 0,
                                       _launch_stream(stream, dev, fn)), fn)


def moe_swiglu_backward(gate_up, d_h, d_gate_up=None, codes=None, scales=None, layout=MOE_GATE_UP_INTERLEAVED,
                        stream=None):
    """Gradient of h = silu(gate) * up: gate_up [R, 2I] (columns as ``layout`` says), d_h [R, I] -> d_gate_up [R, 2I],
    or E4M3 codes u8 [R, 2I] with fp32 scales [R, ceil(2I / 128)], or both."""
    fn = "moe_swiglu_backward"
    _want(layout in (MOE_GATE_UP_INTERLEAVED, MOE_GATE_UP_STACKED), fn, "unknown layout")
    _want(d_gate_up is not None or codes is not None, fn, "d_gate_up or codes are needed")
    _want((codes is None) == (scales is None), fn, "codes and scales come together")
    sh, dt, dev = d_h.shape, d_h.dtype, d_h.get_device()
    if dev >= 0 and dt in _ROWS and len(sh) == 2 and d_h.is_contiguous():
        th = sh[1]
    else:
        _matrix(d_h, dev, fn, "d_h", (None, None), _ROWS)
        th = _stride(d_h)
    wide = (sh[0], 2 * sh[1])
    _want(gate_up is not None, fn, "gate_up must be a matrix")
    gp, tg = _rows_at(gate_up, wide, dt, dev, fn, "gate_up")
    dp, td = _rows_at(d_gate_up, wide, dt, dev, fn, "d_gate_up")
    cp = _flat_at(codes, wide, _U8, dev, fn, "codes")
    sp = _flat_at(scales, (sh[0], (wide[1] + 127) // 128), _F32, dev, fn, "scales")
    _check(lib().moe_swiglu_backward(gp, tg, d_h.data_ptr(), th, _DTYPES[dt], layout, sh[0], sh[1], dp, td, cp, sp,
                                     _launch_stream(stream, dev, fn)), fn)


def moe_gemm_fp8_block_swiglu(x, x_scale, w, w_scale, workspace, out=None, codes=None, scales=None, gate_up=None,
                              layout=MOE_GATE_UP_INTERLEAVED, offsets=None, stream=None):
    """h = silu(gate) * up of the products of x u8 [M, K], x_scale fp32 [M, ceil(K/128)] with w u8 [E, 2I, K] (gate and
    up rows as ``layout`` says), w_scale fp32 [E, ceil(2I/128), ceil(K/128)], rows grouped by offsets int64 [E + 1]
    (None: E = 1, all rows) -> out [M, I], or E4M3 codes u8 [M, I] with fp32 scales [M, ceil(I/128)], or both; the
    products themselves to gate_up [M, 2I] of out's type."""
    fn = "moe_gemm_fp8_block_swiglu"
    _want(layout in (MOE_GATE_UP_INTERLEAVED, MOE_GATE_UP_STACKED), fn, "unknown layout")
    _want(out is not None or codes is not None, fn, "out or codes are needed")
    _want((codes is None) == (scales is None), fn, "codes and scales come together")
    dev, sw, sx = w.get_device(), w.shape, x.shape
    if not (len(sw) == 3 and sw[1] % 2 == 0 and dev >= 0 and w.dtype is _U8 and w.is_contiguous()):
        _table(w, dev, _U8, (None, None, None), fn, "w")
        _want(sw[1] % 2 == 0, fn, f"w has {sw[1]} rows, gate and up make an even number")
    E, N, K = sw
    if not (len(sx) == 2 and sx[1] == K and x.dtype is _U8 and x.get_device() == dev and x.is_contiguous()):
        _table(x, dev, _U8, (None, K), fn, "x")
    blocks = (K + 127) // 128
    xp = _flat_at(x_scale, (sx[0], blocks), _F32, dev, fn, "x_scale")
    wp = _flat_at(w_scale, (E, (N + 127) // 128, blocks), _F32, dev, fn, "w_scale")
    _want(xp is not None and wp is not None, fn, "x_scale and w_scale are needed")
    if workspace.get_device() != dev:
        _place(workspace, dev, fn, "the workspace")
    M, I = sx[0], N // 2
    dt = out.dtype if out is not None else gate_up.dtype if gate_up is not None else torch.bfloat16
    _want(dt in _ROWS, fn, "out and gate_up must be bf16, f16 or f32")
    op = gp = cp = sp = rp = None
    if out is not None:
        op = _flat_at(out, (M, I), dt, dev, fn, "out")
    if gate_up is not None:
        gp = _flat_at(gate_up, (M, N), dt, dev, fn, "gate_up")
    if codes is not None:
        cp = _flat_at(codes, (M, I), _U8, dev, fn, "codes")
        sp = _flat_at(scales, (M, (I + 127) // 128), _F32, dev, fn, "scales")
    if offsets is not None:
        rp = _flat_at(offsets, (E + 1,), _I64, dev, fn, "offsets")
    status = lib().moe_gemm_fp8_block_swiglu(x.data_ptr(), xp, w.data_ptr(), wp, layout, rp, M, I, K, E, op, gp,
                                             _DTYPES[dt], cp, sp, workspace.data_ptr(), workspace.nbytes,
                                             _launch_stream(stream, dev, fn))
    if status:
        _check(status, fn)
