"""ctypes binding of libmoe.so: the same entry points as include/moe.h.

Argument marshalling only -- every step runs in the library's CUDA kernels.
Torch is used for device memory and the current stream.  If the shared
library is missing the import of this module fails loudly, and so does every
call of a dense operator without _marshal.so, their compiled marshalling;
there is no fallback path.
"""
from __future__ import annotations

import ctypes
import os

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "libmoe.so")

# status codes (include/moe.h)
MOE_OK = 0
MOE_ERR_INVALID_ARG = 1
MOE_ERR_UNSUPPORTED = 2
MOE_ERR_ALIGNMENT = 3
MOE_ERR_WORKSPACE = 4
MOE_ERR_CUDA = 5
MOE_ERR_NOT_INITIALIZED = 6
MOE_ERR_BAD_EXPERT = 16
MOE_ERR_BAD_OFFSETS = 17
MOE_ERR_DEVICE_TIMEOUT = 18
MOE_ERR_CAPACITY = 19

MOE_SCORE_SOFTMAX, MOE_SCORE_SIGMOID = 0, 1
MOE_QUANT_ROWWISE, MOE_QUANT_COLWISE_GROUPED, MOE_QUANT_COLWISE_GLU = 0, 1, 2
MOE_QUANT_COLWISE_BATCHED, MOE_QUANT_COLWISE_BATCHED_GLU = 3, 4
MOE_GEMM_FWD, MOE_GEMM_DGRAD, MOE_GEMM_WGRAD = 0, 1, 2
MOE_EPI_NONE, MOE_EPI_SWIGLU, MOE_EPI_SWIGLU_BWD, MOE_EPI_NONE_F32 = 0, 1, 2, 3
MOE_B_GNK, MOE_B_NGK, MOE_B_SF_TILE224 = 0, 1, 2
MOE_SF_ATOMS, MOE_SF_TILE224, MOE_SF_CANONICAL, MOE_SF_TILE224_AND_ATOMS = 0, 1, 2, 3
MOE_TYPE_BF16, MOE_TYPE_F32 = 0, 1
MOE_ACT_NONE, MOE_ACT_RELU, MOE_ACT_GELU, MOE_ACT_SILU = range(4)
MOE_DENSE_FWD, MOE_DENSE_GATED, MOE_DENSE_DGRAD, MOE_DENSE_WGRAD, MOE_DENSE_BACKWARD = range(5)
MOE_GEMM_KERNEL_AUTO, MOE_GEMM_KERNEL_1SM, MOE_GEMM_KERNEL_1SM_N128 = 0, 1, 2
MOE_GEMM_KERNEL_PAIR, MOE_GEMM_KERNEL_PAIR_N128 = 3, 4
(MOE_OP_ROUTE_TOPK, MOE_OP_PERMUTE, MOE_OP_GROUP_QUANTIZE, MOE_OP_GATHER_QUANTIZE, MOE_OP_GROUPED_GEMM,
 MOE_OP_UNPERMUTE_COMBINE, MOE_OP_COMBINE_BWD, MOE_OP_ROUTE_BWD) = range(8)

EXPORTS = [
    "moe_abi_version", "moe_status_string", "moe_init", "moe_row_capacity",
    "moe_route_workspace_size", "moe_permute_workspace_size", "moe_route_topk",
    "moe_permute", "mxfp8_group_quantize", "grouped_gemm_mxfp8",
    "moe_unpermute_combine", "moe_combine_bwd", "moe_route_bwd", "moe_route_topk_noalloc",
    "mxfp8_gather_quantize", "grouped_gemm_mxfp8_swiglu_quant", "mxfp8_swiglu_bwd_quantize",
    "gemm_bf16_nt", "moe_transpose_bf16", "moe_unpermute_combine_add", "moe_route_append_shared",
    "moe_route_drop_shared", "nvfp4_sf_bytes", "nvfp4_quantize", "grouped_gemm_nvfp4", "nvfp4_quantize_cols",
    "moe_selftest_bounded_wait", "moe_workspace_size", "mxfp8_scale_layout", "grouped_gemm_mxfp8_ex",
    "grouped_gemm_mxfp8_swiglu_quant_ex", "grouped_gemm_nvfp4_ex", "moe_hbm_fill", "mxfp8_gather_quantize_ex",
    "mxfp8_swiglu_bwd_quantize_ex", "mxfp8_group_quantize_ex",
    "rmsnorm_residual_fwd", "rmsnorm_bwd_workspace_size", "rmsnorm_residual_bwd",
    "adamw_plan_bytes", "adamw_plan_encode", "adamw_step",
    "linear_fwd", "linear_bwd_workspace_size", "linear_bwd", "gated_ffn_fwd", "gated_ffn_bwd",
    "moe_selftest_dense_plan",
]

_vp, _i32, _i64, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_size_t
_f32 = ctypes.c_float


class GemmOpts(ctypes.Structure):
    """moe_gemm_opts_t (include/moe.h): per-call grouped-GEMM kernel choice."""
    _fields_ = [("kernel", ctypes.c_int), ("band", ctypes.c_int), ("register_stores", ctypes.c_int),
                ("wgrad_rows_lo", ctypes.c_int), ("wgrad_rows_hi", ctypes.c_int)]


class DensePlan(ctypes.Structure):
    """moe_dense_plan_t (include/moe.h)."""
    _fields_ = [(k, ctypes.c_int) for k in ("few_rows", "tile_cols", "parts", "swap_bytes", "box_at", "box_bytes",
                                           "few_parts")]


class AdamWTensor(ctypes.Structure):
    """moe_adamw_tensor_t (include/moe.h)."""
    _fields_ = [("p", _vp), ("g", _vp), ("m", _vp), ("v", _vp), ("m_scale", _vp), ("v_scale", _vp), ("copy", _vp),
                ("n", _i64), ("rng_base", _i64), ("weight_decay", _f32)]


class AdamWOpts(ctypes.Structure):
    """moe_adamw_opts_t (include/moe.h)."""
    _fields_ = [("lr", ctypes.c_double), ("beta1", ctypes.c_double), ("beta2", ctypes.c_double),
                ("eps", ctypes.c_double), ("step", _i64), ("step_dev", _vp), ("lr_dev", _vp), ("grad_scale", _vp),
                ("seed", ctypes.c_uint32)]


_GEMM_KERNELS = {"auto": MOE_GEMM_KERNEL_AUTO, "1sm": MOE_GEMM_KERNEL_1SM, "1sm_n128": MOE_GEMM_KERNEL_1SM_N128,
                 "pair": MOE_GEMM_KERNEL_PAIR, "pair_n128": MOE_GEMM_KERNEL_PAIR_N128}


def gemm_opts(kernel="auto", band=0, register_stores=False, wgrad_rows=(0, 0)):
    """A GemmOpts for the opts= argument of the grouped-GEMM wrappers;
    kernel is one of "auto", "1sm", "1sm_n128", "pair", "pair_n128" (or the
    MOE_GEMM_KERNEL_* value); wgrad_rows = (lo, hi): WGRAD computes only the
    groups with lo <= rows and (hi == 0 or rows < hi)."""
    k = _GEMM_KERNELS[kernel] if isinstance(kernel, str) else int(kernel)
    lo, hi = wgrad_rows
    return GemmOpts(k, int(band), int(bool(register_stores)), int(lo), int(hi))


_SIGS = {
    "moe_abi_version": (_i32, []),
    "moe_status_string": (ctypes.c_char_p, [_i32]),
    "moe_init": (_i32, [_i32]),
    "moe_row_capacity": (_i64, [_i32, _i32, _i32]),
    "moe_route_workspace_size": (_sz, [_i32, _i32]),
    "moe_permute_workspace_size": (_sz, [_i32, _i32]),
    "moe_route_topk": (_i32, [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "moe_permute": (_i32, [_vp, _i32, _i32, _i32, _i32, _vp, _i64, _vp, _vp, _vp, _vp, _vp, _sz, _vp, _vp]),
    "mxfp8_group_quantize": (_i32, [_vp, _i64, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _vp]),
    "mxfp8_group_quantize_ex": (_i32, [_vp, _i64, _i32, _i32, _vp, _i32, _vp, _vp, _vp, _i32, _vp, _vp]),
    "mxfp8_gather_quantize": (_i32, [_vp, _i64, _i32, _i32, _vp, _vp, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp,
                                     _vp]),
    "gemm_bf16_nt": (_i32, [_vp, _vp, _i64, _i32, _i64, _vp, _vp, _vp]),
    "moe_route_append_shared": (_i32, [_vp, _vp, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moe_route_drop_shared": (_i32, [_vp, _i32, _i32, _i32, _vp, _vp]),
    "moe_transpose_bf16": (_i32, [_vp, _i32, _i64, _i64, _vp, _vp]),
    "moe_unpermute_combine_add": (_i32, [_vp, _vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp]),
    "mxfp8_swiglu_bwd_quantize": (_i32, [_vp, _vp, _i32, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "grouped_gemm_mxfp8_swiglu_quant": (_i32, [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i64, _i32, _i64, _vp, _vp, _vp,
                                               _vp, _vp, _vp, _vp, _vp]),
    "grouped_gemm_mxfp8": (_i32, [_i32, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i64, _i32, _i64, _i32, _vp, _vp,
                                  _vp, _vp, _vp]),
    "moe_unpermute_combine": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moe_combine_bwd": (_i32, [_vp, _vp, _vp, _vp, _vp, _vp, _i32, _i32, _i32, _i32, _i64, _vp, _vp, _vp, _vp]),
    "moe_route_bwd": (_i32, [_vp, _vp, _vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp]),
    "moe_route_topk_noalloc": (_i32, [_vp, _i32, _i32, _i32, _i32, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "nvfp4_sf_bytes": (_i64, [_i64, _i32]),
    "moe_selftest_bounded_wait": (_i32, [ctypes.c_uint64, _vp, _vp, _vp]),
    "nvfp4_quantize": (_i32, [_vp, _i64, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "nvfp4_quantize_cols": (_i32, [_vp, _i64, _i32, _vp, _i32, _vp, _vp, _vp, _vp, _vp, _vp]),
    "grouped_gemm_nvfp4": (_i32, [_i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i64, _i32, _vp, _vp,
                                  _vp]),
    "moe_workspace_size": (_sz, [_i32, _i32, _i32, _i32, _i32, _i32]),
    "mxfp8_scale_layout": (_i32, [_vp, _i64, _i32, _i32, _vp, _vp]),
    "grouped_gemm_mxfp8_ex": (_i32, [_i32, _vp, _vp, _vp, _vp, _i32, _vp, _i32, _i64, _i32, _i64, _i32, _vp, _vp,
                                     _vp, _vp, _vp, _vp]),
    "grouped_gemm_mxfp8_swiglu_quant_ex": (_i32, [_vp, _vp, _vp, _vp, _i32, _vp, _i32, _i64, _i32, _i64, _vp, _vp,
                                                  _vp, _vp, _vp, _vp, _vp, _vp, _vp]),
    "grouped_gemm_nvfp4_ex": (_i32, [_i32, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _i32, _i64, _i32, _vp,
                                     _vp, _vp, _vp]),
    "moe_hbm_fill": (_i32, [_vp, _sz, ctypes.c_uint32, _i32, _vp]),
    "mxfp8_gather_quantize_ex": (_i32, [_vp, _i64, _i32, _i32, _vp, _vp, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _i32,
                                        _vp, _vp]),
    "mxfp8_swiglu_bwd_quantize_ex": (_i32, [_vp, _vp, _i32, _vp, _i32, _i64, _vp, _vp, _vp, _vp, _vp, _i32, _vp,
                                            _vp]),
    "rmsnorm_residual_fwd": (_i32, [_vp, _i32, _i64, _vp, _i32, _i64, _vp, _i32, _f32, _i64, _i32, _vp, _i64, _vp,
                                    _i32, _i64, _vp, _vp, _vp, _i32, _vp]),
    "rmsnorm_bwd_workspace_size": (_sz, [_i64, _i32]),
    "rmsnorm_residual_bwd": (_i32, [_vp, _i32, _i64, _vp, _i32, _i64, _vp, _i32, _vp, _vp, _i64, _i64, _i32, _vp,
                                    _i64, _vp, _vp, _sz, _vp]),
    "linear_fwd": (_i32, [_vp, _i64, _vp, _i64, _vp, _i32, _vp, _i64, _i64, _i32, _i64, _vp, _i64, _vp, _i64, _vp,
                          _vp]),
    "linear_bwd_workspace_size": (_sz, [_i64, _i32]),
    "linear_bwd": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _i64, _i32, _i64, _vp, _i64, _vp, _i32,
                          _i64, _vp, _vp, _sz, _vp, _vp]),
    "gated_ffn_fwd": (_i32, [_vp, _i64, _vp, _i64, _i32, _i64, _i32, _i64, _vp, _i64, _vp, _i64, _vp, _vp]),
    "gated_ffn_bwd": (_i32, [_vp, _i64, _vp, _i64, _vp, _i64, _vp, _i64, _i32, _i64, _i32, _i64, _vp, _i64, _vp,
                             _i64, _vp, _i32, _i64, _vp, _vp]),
    "moe_selftest_dense_plan": (_i32, [_i32, _i64, _i64, _i64, _vp, ctypes.POINTER(DensePlan)]),
    "adamw_plan_bytes": (_sz, [_i32]),
    "adamw_plan_encode": (_i32, [_vp, _i32, _i32, _i32, _i32, _vp, ctypes.POINTER(_i64)]),
    "adamw_step": (_i32, [_vp, _i32, _i64, _i32, _i32, _i32, _vp, _vp]),
}


class MoEError(RuntimeError):
    def __init__(self, fn, status):
        self.status = status
        super().__init__(f"{fn} failed: status {status} ({status_string(status)})")


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"libmoe.so not found at {LIB_PATH}; build it with grouped_gemm_top_gb300.build.build()")
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in _SIGS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


class _NoMarshal:
    """In _marshal's place where it was not built: the dense operators say so,
    everything else works."""

    def __init__(self, why):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"{name} needs _marshal.so: run grouped_gemm_top_gb300.build with a C compiler and "
                          f"Python's headers ({self._why})")


try:
    from . import _marshal  # noqa: E402  (links libmoe.so, loaded above)
except ImportError as e:
    _marshal = _NoMarshal(e)


def status_string(status: int) -> str:
    return lib.moe_status_string(int(status)).decode()


def _check(fn, status):
    if status != MOE_OK:
        raise MoEError(fn, status)


def _p(t):
    """Device pointer of a tensor (or None for NULL)."""
    if t is None:
        return None
    return ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


# ------------------------------------------------------------ entry points --

def moe_abi_version() -> int:
    return lib.moe_abi_version()


def moe_init(device: int = 0) -> None:
    _check("moe_init", lib.moe_init(int(device)))


def moe_row_capacity(T: int, E: int, k: int) -> int:
    return int(lib.moe_row_capacity(T, E, k))


def moe_route_workspace_size(T: int, E: int) -> int:
    return int(lib.moe_route_workspace_size(T, E))


def moe_permute_workspace_size(T: int, E: int) -> int:
    return int(lib.moe_permute_workspace_size(T, E))


def moe_workspace_size(op: int, T: int, d: int, E: int, k: int, f: int) -> int:
    """Workspace bytes of call `op` (MOE_OP_*); -1 for an unknown op or bad sizes."""
    v = int(lib.moe_workspace_size(int(op), int(T), int(d), int(E), int(k), int(f)))
    return -1 if v == ctypes.c_size_t(-1).value else v


def mxfp8_scale_layout(src, rows, cols, to_canonical=True, dst=None, stream=None):
    """Scales of a [rows, cols] matrix quantized along cols: atom layout ->
    canonical [rows, cols/32] (to_canonical) or back.  See include/moe.h."""
    dst = dst if dst is not None else _empty((rows * (cols // 32),), torch.uint8, src)
    _check("mxfp8_scale_layout", lib.mxfp8_scale_layout(_p(src), int(rows), int(cols), int(bool(to_canonical)),
                                                        _p(dst), _stream(stream)))
    return dst


def moe_hbm_fill(dst, value=0, method=0, stream=None):
    """Write the 32-bit value over all of dst's bytes (write-only stream)."""
    nbytes = dst.numel() * dst.element_size()
    _check("moe_hbm_fill", lib.moe_hbm_fill(_p(dst), nbytes, ctypes.c_uint32(int(value) & 0xFFFFFFFF).value,
                                            int(method), _stream(stream)))


def _empty(shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device)


def moe_route_topk(logits, k, score=MOE_SCORE_SOFTMAX, normalize=True, topk_idx=None, topk_w=None,
                   counts=None, offsets=None, ws=None, err=None, stream=None):
    T, E = logits.shape
    topk_idx = topk_idx if topk_idx is not None else _empty((T, k), torch.int32, logits)
    topk_w = topk_w if topk_w is not None else _empty((T, k), torch.float32, logits)
    counts = counts if counts is not None else _empty((E,), torch.int32, logits)
    offsets = offsets if offsets is not None else _empty((E + 1,), torch.int32, logits)
    ws = ws if ws is not None else _empty((moe_route_workspace_size(T, E),), torch.uint8, logits)
    _check("moe_route_topk", lib.moe_route_topk(_p(logits), T, E, k, int(score), int(bool(normalize)),
                                                _p(topk_idx), _p(topk_w), _p(counts), _p(offsets), _p(ws),
                                                ws.numel(), _p(err), _stream(stream)))
    return topk_idx, topk_w, counts, offsets


def moe_permute(x, topk_idx, E, row_cap=None, gofs=None, slot_of=None, row_id=None, x_perm=None,
                want_x_perm=True, ws=None, err=None, stream=None):
    T, k = topk_idx.shape
    d = x.shape[1] if x is not None else 0
    row_cap = row_cap if row_cap is not None else moe_row_capacity(T, E, k)
    like = topk_idx
    gofs = gofs if gofs is not None else _empty((E + 1,), torch.int32, like)
    slot_of = slot_of if slot_of is not None else _empty((T, k), torch.int32, like)
    row_id = row_id if row_id is not None else _empty((row_cap,), torch.int32, like)
    if want_x_perm and x_perm is None:
        x_perm = _empty((row_cap, d), torch.bfloat16, like)
    ws = ws if ws is not None else _empty((moe_permute_workspace_size(T, E),), torch.uint8, like)
    _check("moe_permute", lib.moe_permute(_p(x), T, d, E, k, _p(topk_idx), row_cap, _p(gofs), _p(slot_of),
                                          _p(row_id), _p(x_perm) if want_x_perm else None, _p(ws), ws.numel(),
                                          _p(err), _stream(stream)))
    return gofs, slot_of, row_id, x_perm


def sf_bytes(rows: int, cols: int) -> int:
    """Bytes of the scale array of a [rows, cols] matrix quantized along cols."""
    return rows * (cols // 32)


def sf_bytes_tile224(rows: int, cols: int) -> int:
    """Bytes of the tile-224 scale layout of a [rows, cols] matrix quantized
    along cols (include/moe.h): (cols / 128) k-blocks of ceil(rows / 224)
    tiles of 1024 bytes."""
    return (cols // 128) * ((rows + 223) // 224) * 1024


def col_sf_bytes(layout: int, rows: int, cols: int) -> int:
    """Bytes of the columnwise scales of a [rows, cols] quantization (the
    transposed [cols, rows] matrix) in moe_sf_layout_t `layout`; for
    MOE_SF_TILE224_AND_ATOMS the atom layout starts at
    sf_bytes_tile224(cols, rows)."""
    if layout == MOE_SF_TILE224:
        return sf_bytes_tile224(cols, rows)
    if layout == MOE_SF_TILE224_AND_ATOMS:
        return sf_bytes_tile224(cols, rows) + sf_bytes(rows, cols)
    return sf_bytes(rows, cols)


def mxfp8_group_quantize(x, axis=MOE_QUANT_ROWWISE, gofs=None, G=0, codes=None, scales=None, err=None,
                         stream=None):
    """See include/moe.h.  Returns (codes, scales) with the scales in the
    atom layout."""
    rows, cols = x.shape
    if axis == MOE_QUANT_ROWWISE:
        codes = codes if codes is not None else _empty((rows, cols), torch.uint8, x)
    elif axis in (MOE_QUANT_COLWISE_BATCHED, MOE_QUANT_COLWISE_BATCHED_GLU):
        codes = codes if codes is not None else _empty((G, cols, rows // G), torch.uint8, x)
    else:
        codes = codes if codes is not None else _empty((cols, rows), torch.uint8, x)
    scales = scales if scales is not None else _empty((sf_bytes(rows, cols),), torch.uint8, x)
    _check("mxfp8_group_quantize", lib.mxfp8_group_quantize(_p(x), rows, cols, int(axis), _p(gofs), int(G),
                                                            _p(codes), _p(scales), _p(err), _stream(stream)))
    return codes, scales


def mxfp8_group_quantize_ex(x, axis=MOE_QUANT_ROWWISE, gofs=None, G=0, scale_layout=MOE_SF_CANONICAL,
                            want_padded_offsets=True, codes=None, scales=None, padded_offsets=None, err=None,
                            stream=None):
    """mxfp8_group_quantize with the scale layout chosen (MOE_SF_ATOMS or
    MOE_SF_CANONICAL, row-major [R, C / 32] of the output matrix) and the
    padded group offsets written out.  Returns (codes, scales,
    padded_offsets or None)."""
    rows, cols = x.shape
    if axis == MOE_QUANT_ROWWISE:
        codes = codes if codes is not None else _empty((rows, cols), torch.uint8, x)
    elif axis in (MOE_QUANT_COLWISE_BATCHED, MOE_QUANT_COLWISE_BATCHED_GLU):
        codes = codes if codes is not None else _empty((G, cols, rows // G), torch.uint8, x)
    else:
        codes = codes if codes is not None else _empty((cols, rows), torch.uint8, x)
    scales = scales if scales is not None else _empty((sf_bytes(rows, cols),), torch.uint8, x)
    if padded_offsets is None and want_padded_offsets:
        padded_offsets = _empty((int(G) + 1,), torch.int32, x)
    _check("mxfp8_group_quantize_ex",
           lib.mxfp8_group_quantize_ex(_p(x), rows, cols, int(axis), _p(gofs), int(G), _p(codes), _p(scales),
                                       _p(padded_offsets), int(scale_layout), _p(err), _stream(stream)))
    return codes, scales, padded_offsets


def mxfp8_gather_quantize(src, gofs, G, rows, row_id=None, k=1, row_w=None, rowwise=True, colwise=True,
                          codes_row=None, scales_row=None, codes_col=None, scales_col=None, err=None, stream=None,
                          col_sf_layout=MOE_SF_ATOMS):
    """Rowwise and/or group-aware columnwise MXFP8 codes of the permuted
    matrix whose row s is src[row_id[s] // k] (times row_w[row_id[s]]), or
    src[s] without row_id.  See include/moe.h (a given codes_row must be
    32-byte aligned, as fresh torch allocations are).  col_sf_layout
    MOE_SF_TILE224 writes the columnwise scales in the tile-224 layout,
    MOE_SF_TILE224_AND_ATOMS that and the atom layout after it
    (mxfp8_gather_quantize_ex).  Returns (codes_row, scales_row, codes_col,
    scales_col), None for an axis not asked for."""
    cols = src.shape[1]
    if rowwise:
        codes_row = codes_row if codes_row is not None else _empty((rows, cols), torch.uint8, src)
        scales_row = scales_row if scales_row is not None else _empty((sf_bytes(rows, cols),), torch.uint8, src)
    else:
        codes_row = scales_row = None
    if colwise:
        codes_col = codes_col if codes_col is not None else _empty((cols, rows), torch.uint8, src)
        nsc = col_sf_bytes(col_sf_layout, rows, cols)
        scales_col = scales_col if scales_col is not None else torch.zeros((nsc,), dtype=torch.uint8,
                                                                           device=src.device)
    else:
        codes_col = scales_col = None
    args = (_p(src), src.shape[0], cols, int(k), _p(row_id), _p(row_w), _p(gofs), int(G), int(rows), _p(codes_row),
            _p(scales_row), _p(codes_col), _p(scales_col))
    if col_sf_layout == MOE_SF_ATOMS:
        _check("mxfp8_gather_quantize", lib.mxfp8_gather_quantize(*args, _p(err), _stream(stream)))
    else:
        _check("mxfp8_gather_quantize_ex", lib.mxfp8_gather_quantize_ex(*args, int(col_sf_layout), _p(err),
                                                                        _stream(stream)))
    return codes_row, scales_row, codes_col, scales_col


def grouped_gemm_mxfp8(mode, a, a_sf, b, b_sf, b_layout, gofs, G, M, N, K, epilogue=MOE_EPI_NONE,
                       epi_aux=None, d=None, d2=None, err=None, stream=None, opts=None):
    """See include/moe.h.  Allocates d (and d2 for SwiGLU) when not given.
    opts: a GemmOpts (gemm_opts()) selects grouped_gemm_mxfp8_ex."""
    if d is None:
        if mode == MOE_GEMM_WGRAD:
            d = _empty((G, M, N), torch.bfloat16, a)
        elif epilogue == MOE_EPI_SWIGLU_BWD:
            d = _empty((M, 2 * N), torch.bfloat16, a)
        elif epilogue == MOE_EPI_NONE_F32:
            d = _empty((M, N), torch.float32, a)
        else:
            d = _empty((M, N), torch.bfloat16, a)
    if epilogue == MOE_EPI_SWIGLU and d2 is None:
        d2 = _empty((M, N // 2), torch.bfloat16, a)
    args = (int(mode), _p(a), _p(a_sf), _p(b), _p(b_sf), int(b_layout), _p(gofs), int(G), int(M), int(N), int(K),
            int(epilogue), _p(epi_aux), _p(d), _p(d2))
    if opts is None:
        _check("grouped_gemm_mxfp8", lib.grouped_gemm_mxfp8(*args, _p(err), _stream(stream)))
    else:
        _check("grouped_gemm_mxfp8_ex", lib.grouped_gemm_mxfp8_ex(*args, ctypes.byref(opts), _p(err),
                                                                  _stream(stream)))
    return (d, d2) if epilogue == MOE_EPI_SWIGLU else d


def mxfp8_swiglu_bwd_quantize(dH, a_pre, gofs, G, dA=None, want_dA=False, codes_row=None, scales_row=None,
                              codes_col=None, scales_col=None, err=None, stream=None, col_sf_layout=MOE_SF_ATOMS):
    """MXFP8 (both axes) of dA = SwiGLU-backward(a_pre, dH); dA itself in bf16
    only if want_dA or dA is given.  See include/moe.h.  Returns (dA or None,
    codes_row, scales_row, codes_col, scales_col)."""
    rows, f = dH.shape
    if dA is None and want_dA:
        dA = _empty((rows, 2 * f), torch.bfloat16, dH)
    codes_row = codes_row if codes_row is not None else _empty((rows, 2 * f), torch.uint8, dH)
    scales_row = scales_row if scales_row is not None else _empty((sf_bytes(rows, 2 * f),), torch.uint8, dH)
    codes_col = codes_col if codes_col is not None else _empty((2 * f, rows), torch.uint8, dH)
    nsc = col_sf_bytes(col_sf_layout, rows, 2 * f)
    scales_col = scales_col if scales_col is not None else torch.zeros((nsc,), dtype=torch.uint8, device=dH.device)
    args = (_p(dH), _p(a_pre), int(f), _p(gofs), int(G), int(rows), _p(dA), _p(codes_row), _p(scales_row),
            _p(codes_col), _p(scales_col))
    if col_sf_layout == MOE_SF_ATOMS:
        _check("mxfp8_swiglu_bwd_quantize", lib.mxfp8_swiglu_bwd_quantize(*args, _p(err), _stream(stream)))
    else:
        _check("mxfp8_swiglu_bwd_quantize_ex",
               lib.mxfp8_swiglu_bwd_quantize_ex(*args, int(col_sf_layout), _p(err), _stream(stream)))
    return dA, codes_row, scales_row, codes_col, scales_col


def grouped_gemm_mxfp8_swiglu_quant(a, a_sf, b, b_sf, b_layout, gofs, G, M, N, K, a_pre=None, h=None, want_h=False,
                                    h_codes_row=None, h_scales_row=None, h_codes_col=None, h_scales_col=None,
                                    err=None, stream=None, opts=None):
    """Up/gate GEMM with the SwiGLU epilogue writing a_pre [M, N] and the
    MXFP8 codes of h on both axes (h bf16 [M, N/2] only if want_h or h is
    given).  See include/moe.h.  Returns (a_pre, h or None, codes_row,
    scales_row, codes_col, scales_col)."""
    f = N // 2
    a_pre = a_pre if a_pre is not None else _empty((M, N), torch.bfloat16, a)
    if h is None and want_h:
        h = _empty((M, f), torch.bfloat16, a)
    h_codes_row = h_codes_row if h_codes_row is not None else _empty((M, f), torch.uint8, a)
    h_scales_row = h_scales_row if h_scales_row is not None else _empty((sf_bytes(M, f),), torch.uint8, a)
    h_codes_col = h_codes_col if h_codes_col is not None else _empty((f, M), torch.uint8, a)
    h_scales_col = h_scales_col if h_scales_col is not None else _empty((sf_bytes(M, f),), torch.uint8, a)
    args = (_p(a), _p(a_sf), _p(b), _p(b_sf), int(b_layout), _p(gofs), int(G), int(M), int(N), int(K), _p(a_pre),
            _p(h), _p(h_codes_row), _p(h_scales_row), _p(h_codes_col), _p(h_scales_col))
    if opts is None:
        _check("grouped_gemm_mxfp8_swiglu_quant",
               lib.grouped_gemm_mxfp8_swiglu_quant(*args, _p(err), _stream(stream)))
    else:
        _check("grouped_gemm_mxfp8_swiglu_quant_ex",
               lib.grouped_gemm_mxfp8_swiglu_quant_ex(*args, ctypes.byref(opts), _p(err), _stream(stream)))
    return a_pre, h, h_codes_row, h_scales_row, h_codes_col, h_scales_col


def moe_route_append_shared(topk_idx, topk_w, E, n_shared, idx_out=None, w_out=None, stream=None):
    """[T, k+S] choices: the routed ones, then the S shared experts E.. with weight 1."""
    T, k = topk_idx.shape
    idx_out = idx_out if idx_out is not None else _empty((T, k + n_shared), torch.int32, topk_idx)
    w_out = w_out if w_out is not None else _empty((T, k + n_shared), torch.float32, topk_idx)
    _check("moe_route_append_shared", lib.moe_route_append_shared(_p(topk_idx), _p(topk_w), T, k, int(E),
                                                                  int(n_shared), _p(idx_out), _p(w_out),
                                                                  _stream(stream)))
    return idx_out, w_out


def moe_route_drop_shared(dw_all, k, dw=None, stream=None):
    T, k2 = dw_all.shape
    dw = dw if dw is not None else _empty((T, k), torch.float32, dw_all)
    _check("moe_route_drop_shared", lib.moe_route_drop_shared(_p(dw_all), T, int(k), int(k2 - k), _p(dw),
                                                              _stream(stream)))
    return dw


def gemm_bf16_nt(a, b, d=None, err=None, stream=None):
    """d [M, N] fp32 = a [M, K] @ b [N, K]^T (bf16 operands).  See include/moe.h."""
    M, K = a.shape
    N = b.shape[0]
    d = d if d is not None else _empty((M, N), torch.float32, a)
    _check("gemm_bf16_nt", lib.gemm_bf16_nt(_p(a), _p(b), int(M), int(N), int(K), _p(d), _p(err), _stream(stream)))
    return d


def moe_transpose_bf16(src, dst=None, stream=None):
    """dst [cols, rows] bf16 = src [rows, cols]^T (src bf16 or fp32)."""
    rows, cols = src.shape
    dst = dst if dst is not None else _empty((cols, rows), torch.bfloat16, src)
    _check("moe_transpose_bf16", lib.moe_transpose_bf16(_p(src), int(src.dtype == torch.float32), int(rows),
                                                        int(cols), _p(dst), _stream(stream)))
    return dst


def moe_unpermute_combine_add(y_perm, slot_of, topk_w, addend, out=None, err=None, stream=None):
    T, k = slot_of.shape
    d = y_perm.shape[1]
    out = out if out is not None else _empty((T, d), torch.bfloat16, y_perm)
    _check("moe_unpermute_combine_add", lib.moe_unpermute_combine_add(_p(y_perm), _p(slot_of), _p(topk_w),
                                                                      _p(addend), T, d, k, _p(out), _p(err),
                                                                      _stream(stream)))
    return out


def moe_unpermute_combine(y_perm, slot_of, topk_w, out=None, err=None, stream=None):
    T, k = slot_of.shape
    d = y_perm.shape[1]
    out = out if out is not None else _empty((T, d), torch.bfloat16, y_perm)
    _check("moe_unpermute_combine", lib.moe_unpermute_combine(_p(y_perm), _p(slot_of), _p(topk_w), T, d, k,
                                                              _p(out), _p(err), _stream(stream)))
    return out


def moe_combine_bwd(dout, y_perm, slot_of, topk_w, row_id, gofs, E, dy_perm=None, dw=None, err=None, stream=None,
                    want_dy=True):
    """dy_perm (unless want_dy is False: then dw only, dy_perm is None) and dw."""
    T, k = slot_of.shape
    d = dout.shape[1]
    row_cap = row_id.shape[0] if row_id is not None else 0
    if want_dy:
        dy_perm = dy_perm if dy_perm is not None else _empty((row_cap, d), torch.bfloat16, dout)
    else:
        dy_perm = None
        row_cap = max(row_cap, 1)
    dw = dw if dw is not None else _empty((T, k), torch.float32, dout)
    _check("moe_combine_bwd", lib.moe_combine_bwd(_p(dout), _p(y_perm), _p(slot_of), _p(topk_w), _p(row_id),
                                                  _p(gofs), T, d, k, E, row_cap, _p(dy_perm), _p(dw), _p(err),
                                                  _stream(stream)))
    return dy_perm, dw


def moe_route_bwd(logits, topk_idx, dw, score=MOE_SCORE_SOFTMAX, normalize=True, dlogits=None, err=None,
                  stream=None):
    T, E = logits.shape
    k = topk_idx.shape[1]
    dlogits = dlogits if dlogits is not None else _empty((T, E), torch.float32, logits)
    _check("moe_route_bwd", lib.moe_route_bwd(_p(logits), _p(topk_idx), _p(dw), T, E, k, int(score),
                                              int(bool(normalize)), _p(dlogits), _p(err), _stream(stream)))
    return dlogits


def moe_route_topk_noalloc(logits, k, score=MOE_SCORE_SOFTMAX, normalize=True, topk_idx=None, topk_w=None,
                           counts=None, offsets=None, err=None, stream=None):
    """moe_route_topk for callers that cannot allocate device scratch: the
    library uses a fixed internal array instead of a workspace (limit
    ceil(T/128) * E <= 262144; calls must not overlap on the GPU).  The
    output tensors are allocated here only when not passed in."""
    T, E = logits.shape
    topk_idx = topk_idx if topk_idx is not None else _empty((T, k), torch.int32, logits)
    topk_w = topk_w if topk_w is not None else _empty((T, k), torch.float32, logits)
    counts = counts if counts is not None else _empty((E,), torch.int32, logits)
    offsets = offsets if offsets is not None else _empty((E + 1,), torch.int32, logits)
    _check("moe_route_topk_noalloc", lib.moe_route_topk_noalloc(_p(logits), T, E, k, int(score),
                                                                int(bool(normalize)), _p(topk_idx), _p(topk_w),
                                                                _p(counts), _p(offsets), _p(err), _stream(stream)))
    return topk_idx, topk_w, counts, offsets


def nvfp4_sf_bytes(rows: int, cols: int) -> int:
    return int(lib.nvfp4_sf_bytes(int(rows), int(cols)))


def nvfp4_quantize(x, codes=None, scales=None, tensor_scale=None, amax_ws=None, err=None, stream=None):
    """Two-level NVFP4 of bf16 x [rows, cols] (rows % 128, cols % 256).  See
    include/moe.h.  Returns (codes [rows, cols/2] u8, scales u8, tensor_scale
    float32 [1])."""
    rows, cols = x.shape
    codes = codes if codes is not None else _empty((rows, cols // 2), torch.uint8, x)
    scales = scales if scales is not None else _empty((max(nvfp4_sf_bytes(rows, cols), 0),), torch.uint8, x)
    tensor_scale = tensor_scale if tensor_scale is not None else _empty((1,), torch.float32, x)
    amax_ws = amax_ws if amax_ws is not None else _empty((1,), torch.int32, x)
    _check("nvfp4_quantize", lib.nvfp4_quantize(_p(x), int(rows), int(cols), _p(codes), _p(scales),
                                                _p(tensor_scale), _p(amax_ws), _p(err), _stream(stream)))
    return codes, scales, tensor_scale


def nvfp4_quantize_cols(x, gofs, G, codes_t=None, scales_t=None, tensor_scale=None, amax_ws=None, err=None,
                        stream=None):
    """Group-aware columnwise NVFP4 of bf16 x [rows, cols] (rows % 256, cols %
    128; groups at multiples of 128 rows).  See include/moe.h.  Returns
    (codes_t [cols, rows/2] u8, scales_t u8, tensor_scale float32 [1])."""
    rows, cols = x.shape
    codes_t = codes_t if codes_t is not None else _empty((cols, rows // 2), torch.uint8, x)
    scales_t = scales_t if scales_t is not None else _empty((max(nvfp4_sf_bytes(cols, rows), 0),), torch.uint8, x)
    tensor_scale = tensor_scale if tensor_scale is not None else _empty((1,), torch.float32, x)
    amax_ws = amax_ws if amax_ws is not None else _empty((1,), torch.int32, x)
    _check("nvfp4_quantize_cols", lib.nvfp4_quantize_cols(_p(x), int(rows), int(cols), _p(gofs), int(G),
                                                          _p(codes_t), _p(scales_t), _p(tensor_scale),
                                                          _p(amax_ws), _p(err), _stream(stream)))
    return codes_t, scales_t, tensor_scale


def grouped_gemm_nvfp4(mode, a, a_sf, a_scale, b, b_sf, b_scale, gofs, G, M, N, K, epilogue=MOE_EPI_NONE, d=None,
                       err=None, stream=None, opts=None):
    """See include/moe.h.  Allocates d when not given."""
    if d is None:
        shape = (G, M, N) if mode == MOE_GEMM_WGRAD else (M, N)
        d = _empty(shape, torch.float32 if epilogue == MOE_EPI_NONE_F32 else torch.bfloat16, a)
    args = (int(mode), _p(a), _p(a_sf), _p(a_scale), _p(b), _p(b_sf), _p(b_scale), _p(gofs), int(G), int(M), int(N),
            int(K), int(epilogue), _p(d))
    if opts is None:
        _check("grouped_gemm_nvfp4", lib.grouped_gemm_nvfp4(*args, _p(err), _stream(stream)))
    else:
        _check("grouped_gemm_nvfp4_ex", lib.grouped_gemm_nvfp4_ex(*args, ctypes.byref(opts), _p(err),
                                                                  _stream(stream)))
    return d


def moe_selftest_bounded_wait(timeout_ns, err, completed, stream=None):
    """A bounded wait on an mbarrier that nothing arrives at (include/moe.h)."""
    _check("moe_selftest_bounded_wait", lib.moe_selftest_bounded_wait(int(timeout_ns), _p(err), _p(completed),
                                                                      _stream(stream)))



# ------------------------------------------------------ dense operators ----
# These take any strided rows (unit stride inside a row) on the current
# device; a tensor that does not fit the call is refused with
# MOE_ERR_INVALID_ARG before anything is launched.  They also serve steps of a
# few microseconds, so tensors are read and checked in compiled code
# (csrc/marshal.c); what is left here is defaults and allocation.

_TYPES = {torch.bfloat16: MOE_TYPE_BF16, torch.float32: MOE_TYPE_F32}
_ACTS = {"none": MOE_ACT_NONE, "relu": MOE_ACT_RELU, "gelu": MOE_ACT_GELU, "silu": MOE_ACT_SILU}
if not isinstance(_marshal, _NoMarshal):
    _marshal.setup(torch.bfloat16, torch.float32, torch.uint8, torch.float8_e4m3fn, torch.int32,
                   torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream)


def _need(fn, ok):
    if not ok:
        raise MoEError(fn, MOE_ERR_INVALID_ARG)


def _act(fn, act):
    a = _ACTS.get(act, act)
    _need(fn, isinstance(a, int))
    return a


def _new(shape, dtype, like, stream):
    """An uninitialised tensor that belongs to the stream it is used on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _new_rows(m, n, dtype, like, stream):
    """An uninitialised [m, n] whose rows start at multiples of 16 bytes."""
    t = _new((m, (n + 7) // 8 * 8), dtype, like, stream)
    return t if n % 8 == 0 else t[:, :n]


def _size(fn, *matrices):
    """(rows, columns) of the first one; all have to be matrices."""
    for t in matrices:
        _need(fn, isinstance(t, torch.Tensor) and t.dim() == 2)
    return matrices[0].shape


def rmsnorm_residual_fwd(x, w, residual=None, eps=1e-6, y=None, r=None, rstd=None, codes=None, scales=None,
                         want_y=True, want_r=True, want_codes=False, sf_layout=MOE_SF_ATOMS, y_dtype=torch.bfloat16,
                         stream=None):
    """r = x + residual, y = r / sqrt(mean r^2 + eps) * w, and y's MXFP8
    codes and scales.  See include/moe.h.  Outputs that are wanted and not
    given are allocated, their rows at multiples of 16 bytes, as the linear
    layers take them; r is only written when there is a residual, or given.
    Returns (y, r, rstd, codes, scales), None for what is not produced."""
    fn = "rmsnorm_residual_fwd"
    if rstd is None or (y is None and want_y) or (want_codes and codes is None) or (
            r is None and want_r and residual is not None):
        M, N = _size(fn, x)
        if rstd is None:
            rstd = _new((M,), torch.float32, x, stream)
        if y is None and want_y:
            y = _new_rows(M, N, y_dtype, x, stream)
        if r is None and want_r and residual is not None:
            r = _new_rows(M, N, residual.dtype, x, stream)
        if want_codes and codes is None:
            rows = (M + 127) // 128 * 128 if sf_layout == MOE_SF_ATOMS else M
            codes = _new((rows, N), torch.uint8, x, stream)
            scales = _new((rows * (N // 32),), torch.uint8, x, stream) if scales is None else scales
    st = _marshal.rmsnorm_residual_fwd(x, w, residual, eps, y, r, rstd, codes, scales, sf_layout, stream)
    if st:
        raise MoEError(fn, st)
    return y, r, rstd, codes, scales


def rmsnorm_bwd_workspace_size(M: int, N: int) -> int:
    v = int(lib.rmsnorm_bwd_workspace_size(int(M), int(N)))
    return -1 if v == ctypes.c_size_t(-1).value else v


def rmsnorm_residual_bwd(dy, r, w, rstd, dres=None, want_dw=True, dx=None, dw=None, ws=None, stream=None):
    """Gradients of rmsnorm_residual_fwd: dx (of x and of the residual; + dres)
    and dw (fp32).  See include/moe.h.  Returns (dx, dw)."""
    fn = "rmsnorm_residual_bwd"
    if dx is None or (want_dw and dw is None) or (ws is None and (want_dw or dw is not None)):
        M, N = _size(fn, r)
        if dx is None:
            dx = _new_rows(M, N, r.dtype, r, stream)
        if want_dw and dw is None:
            dw = _new((N,), torch.float32, r, stream)
        if dw is not None and ws is None:
            ws = _new((max(rmsnorm_bwd_workspace_size(M, N), 0),), torch.uint8, r, stream)
    st = _marshal.rmsnorm_residual_bwd(dy, r, w, rstd, dres, dx, dw, ws, stream)
    if st:
        raise MoEError(fn, st)
    return dx, dw


def linear_fwd(x, w, bias=None, act="none", residual=None, y=None, z=None, want_z=False, err=None, stream=None):
    """z = x w + bias, y = act(z) + residual (bf16; act "none", "relu", "gelu"
    or "silu").  See include/moe.h.  Rows of every matrix start at multiples
    of 16 bytes.  Returns y, or (y, z) when z is asked for."""
    fn = "linear_fwd"
    if y is None or (want_z and z is None):
        M, N = _size(fn, x, w)[0], w.shape[1]
        y = y if y is not None else _new_rows(M, N, torch.bfloat16, x, stream)
        z = z if z is not None or not want_z else _new_rows(M, N, torch.bfloat16, x, stream)
    st = _marshal.linear_fwd(x, w, bias, _act(fn, act), residual, y, z, err, stream)
    if st:
        raise MoEError(fn, st)
    return y if z is None else (y, z)


def linear_bwd_workspace_size(M: int, N: int) -> int:
    v = int(lib.linear_bwd_workspace_size(int(M), int(N)))
    return -1 if v == ctypes.c_size_t(-1).value else v


def linear_bwd(dy, x, w, z=None, act="none", want_dx=True, want_dw=True, want_dbias=False, dx=None, dw=None,
               dbias=None, dw_dtype=torch.bfloat16, ws=None, err=None, stream=None):
    """Gradients of linear_fwd: dx, dw (bfloat16 or float32) and dbias
    (float32), those that are wanted or given.  See include/moe.h.  Returns
    (dx, dw, dbias)."""
    fn = "linear_bwd"
    act = _act(fn, act)
    need_ws = ws is None and (want_dbias or dbias is not None or act != MOE_ACT_NONE)
    if need_ws or (want_dx and dx is None) or (want_dw and dw is None) or (want_dbias and dbias is None):
        (M, N), K = _size(fn, dy, x), x.shape[1]
        if want_dx and dx is None:
            dx = _new_rows(M, K, torch.bfloat16, x, stream)
        if want_dw and dw is None:
            dw = _new_rows(K, N, dw_dtype, x, stream)
        if want_dbias and dbias is None:
            dbias = _new((N,), torch.float32, x, stream)
        if need_ws:
            ws = _new((max(linear_bwd_workspace_size(M, N), 0),), torch.uint8, x, stream)
    st = _marshal.linear_bwd(dy, x, w, z, act, dx, dw, dbias, ws, err, stream)
    if st:
        raise MoEError(fn, st)
    return dx, dw, dbias


def gated_ffn_fwd(x, w1, act="silu", h=None, a=None, want_a=False, err=None, stream=None):
    """[gate | up] = x w1, h = act(gate) * up in one kernel (bf16).  See
    include/moe.h.  Returns h, or (h, a) when a = [gate | up] is asked for."""
    fn = "gated_ffn_fwd"
    if h is None or (want_a and a is None):
        M, f2 = _size(fn, x, w1)[0], w1.shape[1]
        h = h if h is not None else _new_rows(M, f2 // 2, torch.bfloat16, x, stream)
        a = a if a is not None or not want_a else _new_rows(M, f2, torch.bfloat16, x, stream)
    st = _marshal.gated_ffn_fwd(x, w1, _act(fn, act), h, a, err, stream)
    if st:
        raise MoEError(fn, st)
    return h if a is None else (h, a)


def gated_ffn_bwd(dh, a, x, w1, act="silu", want_dx=True, want_dw=True, dx=None, dw1=None, da=None,
                  dw_dtype=torch.bfloat16, err=None, stream=None):
    """Gradients of gated_ffn_fwd from the kept a: dx and dw1 (bfloat16 or
    float32); da [M, 2f] is written on the way (may be a itself).  See
    include/moe.h.  Returns (dx, dw1)."""
    fn = "gated_ffn_bwd"
    if da is None or (want_dx and dx is None) or (want_dw and dw1 is None):
        (M, f), d = _size(fn, dh, x), x.shape[1]
        da = da if da is not None else _new_rows(M, 2 * f, torch.bfloat16, x, stream)
        dx = dx if dx is not None or not want_dx else _new_rows(M, d, torch.bfloat16, x, stream)
        dw1 = dw1 if dw1 is not None or not want_dw else _new_rows(d, 2 * f, dw_dtype, x, stream)
    st = _marshal.gated_ffn_bwd(dh, a, x, w1, _act(fn, act), da, dx, dw1, err, stream)
    if st:
        raise MoEError(fn, st)
    return dx, dw1


def moe_selftest_dense_plan(product, M, N, K, clusters=None) -> DensePlan:
    """How the product D[M, N] of depth K (MOE_DENSE_*) is launched.  See
    include/moe.h."""
    plan = DensePlan()
    slots = None if clusters is None else (ctypes.c_int * 4)(*clusters)
    _check("moe_selftest_dense_plan", lib.moe_selftest_dense_plan(int(product), int(M), int(N), int(K), slots,
                                                                  ctypes.byref(plan)))
    return plan


class AdamWPlan:
    """The device table of one AdamW step over a list of tensors (adamw_plan)
    and the references that keep the tensors alive."""

    def __init__(self, table, tensors, tiles, p_type, g_type, state_bits, kept):
        self.table, self.kept = table, kept
        self.args = (table.data_ptr(), table.get_device(), tensors, tiles, p_type, g_type, state_bits)


def adamw_plan(params, grads, ms, vs, m_scales=None, v_scales=None, copies=None, weight_decay=0.0, rng_base=None,
               stream=None):
    """Builds the table that adamw_step runs over (include/moe.h).  Lists of
    contiguous tensors of equal sizes: params, grads (each list of one dtype,
    float32 or bfloat16), first and second moments (float32; or 8 bits:
    uint8 / float8_e4m3fn with m_scales and v_scales, float32 of ceil(n/256)),
    optional bfloat16 copies of the params.  weight_decay: one number, or one
    per tensor.  rng_base: first counter of each tensor's rounding (8 bits;
    multiples of 256), by default one tensor after the other."""
    fn = "adamw_plan_encode"
    dev = torch._C._cuda_getDevice()

    def address(t, n, *dtypes):
        _need(fn, t.dtype in dtypes and t.numel() == n and t.get_device() == dev and t.is_contiguous())
        return t.data_ptr()

    n = len(params)
    _need(fn, n >= 1 and len(grads) == len(ms) == len(vs) == n)
    bits = 32 if ms[0].dtype == torch.float32 else 8
    _need(fn, (bits == 8) == (m_scales is not None) == (v_scales is not None))
    state = (torch.float32,) if bits == 32 else (torch.uint8, torch.float8_e4m3fn)
    pt, gt = params[0].dtype, grads[0].dtype
    _need(fn, pt in _TYPES and gt in _TYPES)
    for opt in (m_scales, v_scales, copies, rng_base):
        _need(fn, opt is None or len(opt) == n)
    wd = [float(weight_decay)] * n if isinstance(weight_decay, (int, float)) else [float(v) for v in weight_decay]
    _need(fn, len(wd) == n)
    arr = (AdamWTensor * n)()
    counter = 0
    for i in range(n):
        e, k = arr[i], params[i].numel()
        e.p, e.g = address(params[i], k, pt), address(grads[i], k, gt)
        e.m, e.v = address(ms[i], k, *state), address(vs[i], k, *state)
        if bits == 8:
            e.m_scale = address(m_scales[i], (k + 255) // 256, torch.float32)
            e.v_scale = address(v_scales[i], (k + 255) // 256, torch.float32)
        if copies is not None:
            e.copy = address(copies[i], k, torch.bfloat16)
        e.n, e.weight_decay = k, wd[i]
        e.rng_base = counter if rng_base is None else int(rng_base[i])
        counter += (k + 255) // 256 * 256
    size = int(lib.adamw_plan_bytes(n))
    host = torch.zeros((size + 7) // 8, dtype=torch.int64)
    tiles = _i64(0)
    _check(fn, lib.adamw_plan_encode(ctypes.cast(arr, _vp), n, _TYPES[pt], _TYPES[gt], bits, host.data_ptr(),
                                     ctypes.byref(tiles)))
    table = _new(host.shape, torch.int64, params[0], stream)
    with torch.cuda.stream(stream if stream is not None else torch.cuda.current_stream()):
        table.copy_(host)
    return AdamWPlan(table, n, tiles.value, _TYPES[pt], _TYPES[gt], bits,
                     (params, grads, ms, vs, m_scales, v_scales, copies))


def adamw_step(plan, lr, betas=(0.9, 0.999), eps=1e-8, step=1, grad_scale=None, seed=0, stream=None):
    """One AdamW step over a plan's tensors, in place.  step: the number of
    this step (from 1), or an int32 device tensor with the steps taken so far,
    which the call counts up.  lr: a number or a float32 device tensor.
    grad_scale: float32 device tensor, a factor of every gradient; when it is
    not finite the call changes nothing.  seed: of the 8-bit rounding."""
    st = _marshal.adamw_step(*plan.args, lr, betas[0], betas[1], eps, step, grad_scale, seed, stream)
    if st:
        raise MoEError("adamw_step", st)
