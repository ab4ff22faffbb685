"""MI355X (gfx950) NVFP4 W4A4 MoE hot path: a thin Python binding over libnvfp4moe.so.

Every function here marshals arguments into the C ABI declared in
``include/nvfp4moe.h`` and calls it on the current HIP stream; all arithmetic
runs in the library's HIP kernels.  PyTorch supplies device memory and the
stream only.  If the library has not been built, calls raise
``LibraryNotBuilt`` - there is no fallback implementation.

Tensor conventions: bf16 data may be passed as ``torch.bfloat16`` or as
2-byte integer tensors holding the bits; NVFP4 codes and scales are
``torch.uint8``; row scales, GEMM outputs and router weights ``torch.float32``;
routing ids, offsets and identity maps ``torch.int32``.  FP8 codes are ``torch.uint8`` or
``torch.float8_e4m3fn``.
"""
from __future__ import annotations

import ctypes
import math
import os
from array import array
from operator import attrgetter, is_

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
_LIB = None

W_KN = 0
W_NK = 1
W_ROWMAJOR = 0   # NVFP4 weights [E, N, K/2] / [E, N, K/16]
W_KTILED = 1     # NVFP4 weights [E, K/64, N, 32] / [E, K/64, N, 4]
OUT_F32 = 0      # grouped GEMM output dtypes
OUT_BF16 = 1
OP_QUANTIZE_PERMUTE, OP_QUANTIZE_ROWS, OP_GROUPED_GEMM, OP_SWIGLU_QUANTIZE = 0, 1, 2, 3
OP_UNPERMUTE_COMBINE, OP_BF16_GROUPED_GEMM, OP_SWIGLU_BACKWARD, OP_GROUPED_GEMM_SWIGLU = 4, 5, 6, 7


class LibraryNotBuilt(RuntimeError):
    pass


class NVFP4Error(RuntimeError):
    def __init__(self, fn: str, status: int, text: str):
        super().__init__(f"{fn} failed with status {status}: {text}")
        self.status = status


def library_path() -> str:
    return os.path.join(_PKG, "libnvfp4moe.so")


_c = ctypes
_P = _c.c_void_p
_I64 = _c.c_int64
_I32 = _c.c_int32

# C signatures, in the order of include/nvfp4moe.h
SIGNATURES = {
    "nvfp4moe_status_string": ([_I32], _c.c_char_p),
    "nvfp4moe_abi_version": ([], _c.c_int),
    "nvfp4moe_permute_workspace_size": ([_I64, _I32, _I32], _c.c_size_t),
    "nvfp4moe_workspace_size": ([_I32, _I64, _I32, _I32, _I64, _I64], _c.c_size_t),
    "nvfp4moe_bscale_index": ([_I64, _I64, _I64, _I64], _I64),
    "nvfp4moe_code_index": ([_I64, _I64, _I64, _I64], _I64),
    "nvfp4_quantize_rows": ([_P, _I64, _I64, _P, _P, _P, _P], _c.c_int),
    "nvfp4_quantize_permute": ([_P, _I64, _I64, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P,
                                _c.c_size_t, _P, _P], _c.c_int),
    "nvfp4_quantize_permute_noalloc": ([_P, _I64, _I64, _P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P, _P],
                                       _c.c_int),
    "nvfp4_quantize_rows_tiled": ([_P, _I64, _I64, _I64, _P, _P, _P, _P], _c.c_int),
    "nvfp4_grouped_gemm": ([_P, _P, _P, _P, _I32, _I64, _P, _P, _P, _I64, _I64, _I32, _P, _I32, _P],
                           _c.c_int),
    "nvfp4_grouped_gemm_swiglu": ([_P, _P, _P, _P, _I32, _I64, _P, _P, _P, _I64, _I64, _P, _P, _P, _P, _P,
                                   _c.c_size_t, _P], _c.c_int),
    "nvfp4_quantize_rows_f32": ([_P, _I64, _I64, _P, _I32, _P, _P, _P, _P], _c.c_int),
    "nvfp4moe_token_blocks": ([_P, _I32, _P, _P], _c.c_int),
    "nvfp4_quantize_tokens": ([_P, _I32, _I64, _I64, _P, _I32, _P, _P, _I32, _I64, _I32, _P, _P, _P, _P],
                              _c.c_int),
    "nvfp4_grouped_gemm_wgrad": ([_P, _P, _P, _P, _P, _P, _P, _I32, _I64, _I64, _I64, _P, _I32, _P], _c.c_int),
    "swiglu_quantize": ([_P, _I64, _I64, _P, _I32, _P, _P, _P, _P, _P, _P, _P], _c.c_int),
    "unpermute_combine": ([_P, _I64, _I32, _I64, _P, _P, _P, _P], _c.c_int),
    "permute_gather_bf16": ([_P, _I64, _I64, _I32, _P, _I32, _P, _P, _P], _c.c_int),
    "bf16_grouped_gemm": ([_P, _P, _I32, _I64, _P, _I32, _I64, _I64, _P, _P], _c.c_int),
    "bf16_grouped_gemm_gather": ([_P, _I64, _P, _I32, _P, _I32, _I64, _P, _I32, _I64, _I64, _P, _P],
                                 _c.c_int),
    "swiglu_backward": ([_P, _P, _I64, _I64, _P, _I32, _P, _P, _P, _P], _c.c_int),
    "bf16_transpose": ([_P, _I64, _I64, _I64, _P, _P], _c.c_int),
    "fp8_quantize_rows": ([_P, _I32, _I64, _I64, _P, _I32, _P, _P, _P], _c.c_int),
    "fp8_quantize_weights": ([_P, _I64, _I64, _I64, _P, _P, _P, _P, _P], _c.c_int),
    "fp8_swiglu_quantize": ([_P, _I32, _I64, _I64, _P, _I32, _P, _P, _P, _P, _P, _P], _c.c_int),
    "fp8_grouped_gemm": ([_P, _P, _P, _I32, _I64, _P, _P, _I64, _I64, _P, _I32, _P], _c.c_int),
    "fp8_grouped_gemm_gather": ([_P, _P, _I64, _P, _I32, _P, _I32, _I64, _P, _P, _I64, _I64, _P, _I32, _P],
                                _c.c_int),
    "bf16_grouped_gemm_wgrad": ([_P, _I64, _I32, _P, _I64, _I32, _P, _P, _I32, _I64, _I64, _I64, _P, _I32, _P],
                                _c.c_int),
    "moe_router_topk": ([_P, _I32, _I64, _I32, _I32, _I32, _P, _P, _P], _c.c_int),
    "moe_router_topk_backward": ([_P, _I32, _P, _P, _P, _I64, _I32, _I32, _I32, _P, _P], _c.c_int),
    "moe_permute_workspace_size": ([_I64, _I32, _I32], _c.c_size_t),
    "moe_permute": ([_P, _I32, _I64, _I64, _P, _I32, _I32, _P, _P, _P, _P, _P, _c.c_size_t, _P, _P], _c.c_int),
    "moe_combine": ([_P, _I32, _I64, _I32, _I64, _P, _P, _P, _I32, _P], _c.c_int),
    "moe_combine_backward": ([_P, _I32, _P, _I32, _I64, _I32, _I64, _P, _P, _P, _P, _P], _c.c_int),
    "swiglu_backward_weights": ([_P, _P, _I64, _I64, _P, _I32, _P, _P, _P, _P, _P, _P], _c.c_int),
    "moe_grad_workspace_size": ([_I32], _c.c_size_t),
    "moe_grad_norm": ([_P, _P, _P, _I32, _P, _P, _c.c_size_t, _P], _c.c_int),
    "moe_grad_clip": ([_P, _P, _P, _P, _I32, _c.c_double, _P, _P, _c.c_size_t, _P], _c.c_int),
    "nvfp4moe_mfma_ceiling": ([_I64, _P, _P], _c.c_int),
}


def load_library():
    """Load libnvfp4moe.so (cached).  Raises LibraryNotBuilt if it is missing."""
    global _LIB
    if _LIB is not None:
        return _LIB
    path = library_path()
    if not os.path.exists(path):
        raise LibraryNotBuilt(
            f"{path} is missing: build it with `python -m precision_moe_gemm_amd.build`")
    lib = ctypes.CDLL(path)
    for name, (args, res) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = res
    _LIB = lib
    return lib


def status_string(status: int) -> str:
    return load_library().nvfp4moe_status_string(status).decode()


def _check(fn: str, status: int):
    if status != 0:
        raise NVFP4Error(fn, status, status_string(status))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream():
    return torch.cuda.current_stream().cuda_stream


def _req(t, name, dtypes, ndim=None, numel=None):
    """Check a tensor argument; `numel`: the elements the library reads or writes
    through it (the C-ABI sees only the pointer, so a smaller buffer is refused here)."""
    if t is None:
        return
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name}: dtype {t.dtype} not in {dtypes}")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a device tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if ndim is not None and t.dim() != ndim:
        raise ValueError(f"{name} must have {ndim} dims, got {t.dim()}")
    if numel is not None and t.numel() < numel:
        raise ValueError(f"{name} holds {t.numel()} elements, needs {numel}")


_BF16 = (torch.bfloat16, torch.int16, torch.uint16)
_U8 = (torch.uint8,)
_F32 = (torch.float32,)
_I32T = (torch.int32,)


def _empty(shape, dtype, like):
    return torch.empty(shape, dtype=dtype, device=like.device)


# ---------------------------------------------------------------------- entry points
def nvfp4_quantize_rows(x, codes=None, bscales=None, rscales=None):
    """x bf16 [rows, K] -> (codes u8 [rows, K/2], bscales u8 [rows, K/16], rscales f32 [rows])."""
    _req(x, "x", _BF16, 2)
    rows, K = x.shape
    codes = _empty((rows, K // 2), torch.uint8, x) if codes is None else codes
    bscales = _empty((rows, K // 16), torch.uint8, x) if bscales is None else bscales
    rscales = _empty((rows,), torch.float32, x) if rscales is None else rscales
    _req(codes, "codes", _U8, numel=rows * (K // 2)); _req(bscales, "bscales", _U8, numel=rows * (K // 16))
    _req(rscales, "rscales", _F32, numel=rows)
    _check("nvfp4_quantize_rows", load_library().nvfp4_quantize_rows(
        _ptr(x), rows, K, _ptr(codes), _ptr(bscales), _ptr(rscales), _stream()))
    return codes, bscales, rscales


def nvfp4_quantize_rows_tiled(x, group_rows: int, codes=None, bscales=None, rscales=None):
    """x bf16 [rows, K] -> the K-tiled NVFP4 layout of groups of `group_rows` rows:
    (codes u8 [rows/G, K/64, G, 32], bscales u8 [rows/G, K/64, G, 4], rscales f32 [rows])."""
    _req(x, "x", _BF16, 2)
    rows, K = x.shape
    G = int(group_rows)
    if G <= 0 or rows % G or K % 64:
        raise ValueError("need rows % group_rows == 0 and K % 64 == 0")
    codes = _empty((rows // G, K // 64, G, 32), torch.uint8, x) if codes is None else codes
    bscales = _empty((rows // G, K // 64, G, 4), torch.uint8, x) if bscales is None else bscales
    rscales = _empty((rows,), torch.float32, x) if rscales is None else rscales
    _req(codes, "codes", _U8, numel=rows * (K // 2)); _req(bscales, "bscales", _U8, numel=rows * (K // 16))
    _req(rscales, "rscales", _F32, numel=rows)
    _check("nvfp4_quantize_rows_tiled", load_library().nvfp4_quantize_rows_tiled(
        _ptr(x), rows, K, G, _ptr(codes), _ptr(bscales), _ptr(rscales), _stream()))
    return codes, bscales, rscales


def permute_workspace_size(T: int, k: int, E: int) -> int:
    return int(load_library().nvfp4moe_permute_workspace_size(T, k, E))


def workspace_size(op: int, T: int = 0, E: int = 0, k: int = 0, R_max: int = 0, N: int = 0) -> int:
    """Device workspace bytes of an operation (OP_*); only OP_QUANTIZE_PERMUTE needs any."""
    return int(load_library().nvfp4moe_workspace_size(op, T, E, k, R_max, N))


def bscale_index(r: int, kb: int, K: int, group_rows: int = 0) -> int:
    """Byte offset of block kb of row r: row-major (group_rows 0) or K-tiled groups."""
    return int(load_library().nvfp4moe_bscale_index(r, kb, K, group_rows))


def code_index(r: int, i: int, K: int, group_rows: int = 0) -> int:
    """Byte offset of the byte holding element i of row r (low nibble for even i)."""
    return int(load_library().nvfp4moe_code_index(r, i, K, group_rows))


def nvfp4_quantize_permute(x, topk_ids, E: int, workspace=None, dev_err=None, out=None):
    """Route + permute + quantise.  Returns dict with codes, bscales, rscales,
    expert_offsets [E+1], row_to_tk [T*k], tk_to_row [T*k]."""
    _req(x, "x", _BF16, 2)
    _req(topk_ids, "topk_ids", _I32T, 2)
    T, H = x.shape
    k = topk_ids.shape[1]
    if topk_ids.shape[0] != T:
        raise ValueError("topk_ids must have one row per token")
    R = T * k
    o = out or {}
    shapes = {"codes": ((R, H // 2), torch.uint8), "bscales": ((R, H // 16), torch.uint8),
              "rscales": ((R,), torch.float32), "expert_offsets": ((E + 1,), torch.int32),
              "row_to_tk": ((R,), torch.int32), "tk_to_row": ((R,), torch.int32)}
    res = {n: o[n] if n in o else _empty(shp, dt, x) for n, (shp, dt) in shapes.items()}
    ws_bytes = permute_workspace_size(T, k, E)
    if ws_bytes == 0:
        raise ValueError("invalid routing shape")
    if workspace is None:
        workspace = _empty((max(ws_bytes, 256),), torch.uint8, x)
    for name, (shp, _) in shapes.items():
        _req(res[name], name, _U8 if name in ("codes", "bscales") else _F32 if name == "rscales" else _I32T,
             numel=math.prod(shp))
    _req(workspace, "workspace", _U8)
    _req(dev_err, "dev_err", _I32T, numel=1)
    _check("nvfp4_quantize_permute", load_library().nvfp4_quantize_permute(
        _ptr(x), T, H, _ptr(topk_ids), k, E, _ptr(res["codes"]), _ptr(res["bscales"]),
        _ptr(res["rscales"]), _ptr(res["expert_offsets"]), _ptr(res["row_to_tk"]),
        _ptr(res["tk_to_row"]), _ptr(workspace), workspace.numel(), _ptr(dev_err), _stream()))
    return res


NOALLOC_MAX_ENTRIES = 1 << 20
_QP_OUTPUTS = ("codes", "bscales", "rscales", "expert_offsets", "row_to_tk", "tk_to_row")


def nvfp4_quantize_permute_noalloc(x, topk_ids, E: int, out, dev_err=None):
    """nvfp4_quantize_permute without a workspace and without any allocation: the
    library's fixed device scratch serves T*k <= NOALLOC_MAX_ENTRIES entries.  Every
    output must be given in `out` (same names and sizes as nvfp4_quantize_permute's
    result); returns `out`.  Calls on one device that overlap in time race."""
    _req(x, "x", _BF16, 2)
    _req(topk_ids, "topk_ids", _I32T, 2)
    T, H = x.shape
    k = topk_ids.shape[1]
    if topk_ids.shape[0] != T:
        raise ValueError("topk_ids must have one row per token")
    missing = [n for n in _QP_OUTPUTS if n not in out]
    if missing:
        raise ValueError(f"the allocation-free call needs every output given: missing {missing}")
    R = T * k
    need = {"codes": (R * (H // 2), _U8), "bscales": (R * (H // 16), _U8), "rscales": (R, _F32),
            "expert_offsets": (E + 1, _I32T), "row_to_tk": (R, _I32T), "tk_to_row": (R, _I32T)}
    for name, (n, dt) in need.items():
        _req(out[name], name, dt, numel=n)
    _req(dev_err, "dev_err", _I32T, numel=1)
    _check("nvfp4_quantize_permute_noalloc", load_library().nvfp4_quantize_permute_noalloc(
        _ptr(x), T, H, _ptr(topk_ids), k, E, _ptr(out["codes"]), _ptr(out["bscales"]),
        _ptr(out["rscales"]), _ptr(out["expert_offsets"]), _ptr(out["row_to_tk"]),
        _ptr(out["tk_to_row"]), _ptr(dev_err), _stream()))
    return out


def nvfp4_grouped_gemm(a_codes, a_bscales, a_rscales, expert_offsets, w_codes, w_bscales,
                       w_rscales, c=None, out_dtype=None):
    """C[r] = A[r] W_e^T over expert-grouped rows.  Returns C [R_cap, N], float32
    (default) or bfloat16 (out_dtype=torch.bfloat16, or a bf16 `c`).
    W in either layout: row-major codes [E, N, K/2] (bscales [E, N, K/16]) or
    K-tiled codes [E, K/64, N, 32] (bscales [E, K/64, N, 4]); w_rscales [E, N]."""
    for t, n, d in ((a_codes, "a_codes", _U8), (a_bscales, "a_bscales", _U8),
                    (a_rscales, "a_rscales", _F32), (expert_offsets, "expert_offsets", _I32T),
                    (w_codes, "w_codes", _U8), (w_bscales, "w_bscales", _U8),
                    (w_rscales, "w_rscales", _F32)):
        _req(t, n, d)
    R_cap = a_codes.shape[0]
    K = a_codes.shape[1] * 2
    E = expert_offsets.numel() - 1
    if w_codes.dim() == 4:
        layout, N = W_KTILED, w_codes.shape[2]
        ok = tuple(w_codes.shape) == (E, K // 64, N, 32) and tuple(w_bscales.shape) == (E, K // 64, N, 4)
    else:
        layout, N = W_ROWMAJOR, w_codes.shape[1]
        ok = (w_codes.dim() == 3 and w_codes.shape[0] == E and w_codes.shape[2] * 2 == K
              and w_bscales.numel() >= E * N * (K // 16))
    if not ok:
        raise ValueError("w_codes/w_bscales shapes do not match E, K and a known layout")
    _req(a_bscales, "a_bscales", _U8, numel=R_cap * (K // 16))
    _req(a_rscales, "a_rscales", _F32, numel=R_cap)
    _req(w_rscales, "w_rscales", _F32, numel=E * N)
    if out_dtype is None:
        out_dtype = torch.float32 if c is None or c.dtype == torch.float32 else torch.bfloat16
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    c = _empty((R_cap, N), out_dtype, a_codes) if c is None else c
    _req(c, "c", _F32 if out_dtype == torch.float32 else _BF16, numel=R_cap * N)
    _check("nvfp4_grouped_gemm", load_library().nvfp4_grouped_gemm(
        _ptr(a_codes), _ptr(a_bscales), _ptr(a_rscales), _ptr(expert_offsets), E, R_cap,
        _ptr(w_codes), _ptr(w_bscales), _ptr(w_rscales), N, K, layout, _ptr(c),
        OUT_F32 if out_dtype == torch.float32 else OUT_BF16, _stream()))
    return c


def nvfp4_grouped_gemm_swiglu(a_codes, a_bscales, a_rscales, expert_offsets, w_codes, w_bscales,
                              w_rscales, topk_w=None, row_to_tk=None, h=None, gu=None, want_gu=False,
                              workspace=None):
    """gate_up GEMM with the weighted SwiGLU in its epilogue.  W K-tiled
    (codes [E, K/64, 2I, 32], bscales [E, K/64, 2I, 4], rscales [E, 2I]).
    Returns (h f32 [R_cap, I], gu f32 [R_cap, 2I] or None)."""
    for t, n, d in ((a_codes, "a_codes", _U8), (a_bscales, "a_bscales", _U8),
                    (a_rscales, "a_rscales", _F32), (expert_offsets, "expert_offsets", _I32T),
                    (w_codes, "w_codes", _U8), (w_bscales, "w_bscales", _U8),
                    (w_rscales, "w_rscales", _F32), (topk_w, "topk_w", _F32), (row_to_tk, "row_to_tk", _I32T)):
        _req(t, n, d)
    R_cap = a_codes.shape[0]
    K = a_codes.shape[1] * 2
    E = expert_offsets.numel() - 1
    if w_codes.dim() != 4 or w_codes.shape[0] != E or w_codes.shape[1] != K // 64 or w_codes.shape[2] % 2:
        raise ValueError("w_codes must be K-tiled [E, K/64, 2I, 32]")
    N = w_codes.shape[2]
    I = N // 2
    if tuple(w_bscales.shape) != (E, K // 64, N, 4):
        raise ValueError("w_bscales must be K-tiled [E, K/64, 2I, 4]")
    _req(a_bscales, "a_bscales", _U8, numel=R_cap * (K // 16))
    _req(a_rscales, "a_rscales", _F32, numel=R_cap)
    _req(w_rscales, "w_rscales", _F32, numel=E * N)
    if topk_w is not None:
        if row_to_tk is None:
            raise ValueError("topk_w needs row_to_tk")
        _req(topk_w, "topk_w", _F32, numel=R_cap)
        _req(row_to_tk, "row_to_tk", _I32T, numel=R_cap)
        ws_bytes = workspace_size(OP_GROUPED_GEMM_SWIGLU, R_max=R_cap)
        workspace = _empty((ws_bytes,), torch.uint8, a_codes) if workspace is None else workspace
        _req(workspace, "workspace", _U8, numel=ws_bytes)
    h = _empty((R_cap, I), torch.float32, a_codes) if h is None else h
    _req(h, "h", _F32, numel=R_cap * I)
    if want_gu and gu is None:
        gu = _empty((R_cap, N), torch.float32, a_codes)
    _req(gu, "gu", _F32, numel=R_cap * N)
    _check("nvfp4_grouped_gemm_swiglu", load_library().nvfp4_grouped_gemm_swiglu(
        _ptr(a_codes), _ptr(a_bscales), _ptr(a_rscales), _ptr(expert_offsets), E, R_cap, _ptr(w_codes),
        _ptr(w_bscales), _ptr(w_rscales), I, K, _ptr(topk_w), _ptr(row_to_tk), _ptr(h), _ptr(gu),
        _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream()))
    return h, gu


def nvfp4_quantize_rows_f32(x, expert_offsets=None, codes=None, bscales=None, rscales=None):
    """FP32 rows [rows, K] -> NVFP4 (codes, bscales, rscales); with expert_offsets only
    the routed rows [0, offsets[E]) are written."""
    _req(x, "x", _F32, 2)
    _req(expert_offsets, "expert_offsets", _I32T)
    rows, K = x.shape
    E = 0 if expert_offsets is None else expert_offsets.numel() - 1
    codes = _empty((rows, K // 2), torch.uint8, x) if codes is None else codes
    bscales = _empty((rows, K // 16), torch.uint8, x) if bscales is None else bscales
    rscales = _empty((rows,), torch.float32, x) if rscales is None else rscales
    _req(codes, "codes", _U8, numel=rows * (K // 2)); _req(bscales, "bscales", _U8, numel=rows * (K // 16))
    _req(rscales, "rscales", _F32, numel=rows)
    _check("nvfp4_quantize_rows_f32", load_library().nvfp4_quantize_rows_f32(
        _ptr(x), rows, K, _ptr(expert_offsets), E, _ptr(codes), _ptr(bscales), _ptr(rscales), _stream()))
    return codes, bscales, rscales


def token_blocks(expert_offsets, kofs=None):
    """kofs [E+1] int32: the first 64-token step of each expert's slab along K."""
    _req(expert_offsets, "expert_offsets", _I32T)
    E = expert_offsets.numel() - 1
    kofs = _empty((E + 1,), torch.int32, expert_offsets) if kofs is None else kofs
    _req(kofs, "kofs", _I32T, numel=E + 1)
    _check("nvfp4moe_token_blocks", load_library().nvfp4moe_token_blocks(
        _ptr(expert_offsets), E, _ptr(kofs), _stream()))
    return kofs


def token_capacity(R: int, E: int) -> int:
    """K positions that always hold every expert's padded slab."""
    return 64 * (-(-R // 64) + E)


def nvfp4_quantize_tokens(x, expert_offsets, kofs, Kp: int, layout: int = W_ROWMAJOR, row_to_tk=None, k: int = 1,
                          out=None):
    """Quantise along tokens, per expert: x [rows, C] (bf16 or f32; token order with
    row_to_tk/k, else expert-grouped rows).  Returns (codes, bscales, rscales [E, C]):
    row-major codes [C, Kp/2] / bscales [C, Kp/16], or K-tiled [Kp/64, C, 32] / [Kp/64, C, 4]."""
    _req(x, "x", _BF16 + _F32, 2)
    _req(expert_offsets, "expert_offsets", _I32T)
    _req(row_to_tk, "row_to_tk", _I32T)
    E = expert_offsets.numel() - 1
    _req(kofs, "kofs", _I32T, numel=E + 1)
    rows, C = x.shape
    if row_to_tk is None and rows < 1:
        raise ValueError("x has no rows")
    o = out or {}
    shp_c = (C, Kp // 2) if layout == W_ROWMAJOR else (Kp // 64, C, 32)
    shp_b = (C, Kp // 16) if layout == W_ROWMAJOR else (Kp // 64, C, 4)
    codes = o["codes"] if "codes" in o else _empty(shp_c, torch.uint8, x)
    bsc = o["bscales"] if "bscales" in o else _empty(shp_b, torch.uint8, x)
    rsc = o["rscales"] if "rscales" in o else _empty((E, C), torch.float32, x)
    _req(codes, "codes", _U8, numel=C * Kp // 2); _req(bsc, "bscales", _U8, numel=C * Kp // 16)
    _req(rsc, "rscales", _F32, numel=E * C)
    dt = 1 if x.dtype == torch.float32 else 0
    _check("nvfp4_quantize_tokens", load_library().nvfp4_quantize_tokens(
        _ptr(x), dt, rows, C, _ptr(row_to_tk), k, _ptr(expert_offsets), _ptr(kofs), E, Kp, layout,
        _ptr(codes), _ptr(bsc), _ptr(rsc), _stream()))
    return codes, bsc, rsc


def nvfp4_grouped_gemm_wgrad(a, w, kofs, c=None, out_dtype=None):
    """dW [E, M, N] = per expert dequant(A_e) dequant(W_e)^T over its token slab,
    float32 (default) or bfloat16 (out_dtype=torch.bfloat16, or a bf16 `c`).
    a: row-major (codes [M, Kp/2], bscales [M, Kp/16], rscales [E, M]);
    w: K-tiled (codes [Kp/64, N, 32], bscales [Kp/64, N, 4], rscales [E, N])."""
    ac, ab, ar = a
    wc, wb, wr = w
    for t, n, d in ((ac, "a_codes", _U8), (ab, "a_bscales", _U8), (ar, "a_rscales", _F32),
                    (wc, "w_codes", _U8), (wb, "w_bscales", _U8), (wr, "w_rscales", _F32), (kofs, "kofs", _I32T)):
        _req(t, n, d)
    M, half = ac.shape
    Kp = half * 2
    E = kofs.numel() - 1
    if wc.dim() != 3 or wc.shape[0] != Kp // 64 or wc.shape[2] != 32:
        raise ValueError("w codes must be K-tiled [Kp/64, N, 32] over the same Kp")
    N = wc.shape[1]
    _req(ab, "a_bscales", _U8, numel=M * Kp // 16); _req(ar, "a_rscales", _F32, numel=E * M)
    _req(wb, "w_bscales", _U8, numel=N * Kp // 16); _req(wr, "w_rscales", _F32, numel=E * N)
    if out_dtype is None:
        out_dtype = torch.float32 if c is None or c.dtype == torch.float32 else torch.bfloat16
    if out_dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    c = _empty((E, M, N), out_dtype, ac) if c is None else c
    _req(c, "c", _F32 if out_dtype == torch.float32 else _BF16, numel=E * M * N)
    _check("nvfp4_grouped_gemm_wgrad", load_library().nvfp4_grouped_gemm_wgrad(
        _ptr(ac), _ptr(ab), _ptr(ar), _ptr(wc), _ptr(wb), _ptr(wr), _ptr(kofs), E, M, N, Kp, _ptr(c),
        OUT_F32 if out_dtype == torch.float32 else OUT_BF16, _stream()))
    return c


def swiglu_quantize(gu, expert_offsets, topk_w=None, row_to_tk=None, h_out=False, out=None):
    """Weighted SwiGLU + NVFP4 quantise of routed rows.  Returns (codes, bscales, rscales, h or None)."""
    _req(gu, "gu", _F32, 2)
    _req(expert_offsets, "expert_offsets", _I32T)
    _req(topk_w, "topk_w", _F32)
    _req(row_to_tk, "row_to_tk", _I32T)
    R_cap, I2 = gu.shape
    I = I2 // 2
    E = expert_offsets.numel() - 1
    # the kernel reads topk_w[row_to_tk[r]], and row_to_tk holds entries below R_cap
    _req(topk_w, "topk_w", _F32, numel=R_cap)
    o = out or {}
    codes = o["codes"] if "codes" in o else _empty((R_cap, I // 2), torch.uint8, gu)
    bsc = o["bscales"] if "bscales" in o else _empty((R_cap, I // 16), torch.uint8, gu)
    rsc = o["rscales"] if "rscales" in o else _empty((R_cap,), torch.float32, gu)
    h = (o["h"] if "h" in o else _empty((R_cap, I), torch.float32, gu)) if h_out else None
    _req(codes, "codes", _U8, numel=R_cap * (I // 2)); _req(bsc, "bscales", _U8, numel=R_cap * (I // 16))
    _req(rsc, "rscales", _F32, numel=R_cap); _req(h, "h", _F32, numel=R_cap * I)
    _req(row_to_tk, "row_to_tk", _I32T, numel=R_cap)
    _check("swiglu_quantize", load_library().swiglu_quantize(
        _ptr(gu), R_cap, I, _ptr(expert_offsets), E, _ptr(topk_w), _ptr(row_to_tk),
        _ptr(codes), _ptr(bsc), _ptr(rsc), _ptr(h), _stream()))
    return codes, bsc, rsc, h


def unpermute_combine(d, tk_to_row, k: int, topk_w=None, y=None):
    """y[t] = bf16(sum over slots of w * d[row(t, slot)]).  Returns y as torch.bfloat16 [T, H]."""
    _req(d, "d", _F32, 2)
    _req(tk_to_row, "tk_to_row", _I32T)
    _req(topk_w, "topk_w", _F32)
    if k < 1 or tk_to_row.numel() % k:
        raise ValueError("tk_to_row must hold T * k entries")
    T = tk_to_row.numel() // k
    H = d.shape[1]
    # tk_to_row names rows below T * k (the routed rows of nvfp4_quantize_permute)
    _req(d, "d", _F32, numel=T * k * H)
    _req(topk_w, "topk_w", _F32, numel=T * k)
    y = _empty((T, H), torch.bfloat16, d) if y is None else y
    _req(y, "y", _BF16, numel=T * H)
    _check("unpermute_combine", load_library().unpermute_combine(
        _ptr(d), T, k, H, _ptr(tk_to_row), _ptr(topk_w), _ptr(y), _stream()))
    return y


def permute_gather_bf16(x, expert_offsets, row_to_tk, k: int, out=None):
    _req(x, "x", _BF16, 2)
    _req(expert_offsets, "expert_offsets", _I32T)
    _req(row_to_tk, "row_to_tk", _I32T)
    T, H = x.shape
    E = expert_offsets.numel() - 1
    _req(row_to_tk, "row_to_tk", _I32T, numel=T * k)
    out = _empty((T * k, H), torch.bfloat16, x) if out is None else out
    _req(out, "out", _BF16, numel=T * k * H)
    _check("permute_gather_bf16", load_library().permute_gather_bf16(
        _ptr(x), T, H, k, _ptr(expert_offsets), E, _ptr(row_to_tk), _ptr(out), _stream()))
    return out


def bf16_transpose(x, out=None):
    """out[b] = x[b].T for bf16 x [B, rows, cols] (weight preparation).  Returns [B, cols, rows]."""
    _req(x, "x", _BF16, 3)
    B, rows, cols = x.shape
    out = _empty((B, cols, rows), torch.bfloat16, x) if out is None else out
    _req(out, "out", _BF16, numel=B * rows * cols)
    _check("bf16_transpose", load_library().bf16_transpose(_ptr(x), B, rows, cols, _ptr(out), _stream()))
    return out


def bf16_grouped_gemm(a, expert_offsets, w, w_layout: int = W_KN, c=None):
    """c[r] = a[r] @ W_e with W [E, K, N] (W_KN) or [E, N, K] (W_NK).  Returns f32 [R_cap, N]."""
    _req(a, "a", _BF16, 2)
    _req(expert_offsets, "expert_offsets", _I32T)
    _req(w, "w", _BF16, 3)
    R_cap, K = a.shape
    E = expert_offsets.numel() - 1
    N = w.shape[2] if w_layout == W_KN else w.shape[1]
    kw = w.shape[1] if w_layout == W_KN else w.shape[2]
    if kw != K or w.shape[0] != E:
        raise ValueError("weight shape does not match a / expert_offsets")
    c = _empty((R_cap, N), torch.float32, a) if c is None else c
    _req(c, "c", _F32, numel=R_cap * N)
    _check("bf16_grouped_gemm", load_library().bf16_grouped_gemm(
        _ptr(a), _ptr(expert_offsets), E, R_cap, _ptr(w), w_layout, N, K, _ptr(c), _stream()))
    return c


def bf16_grouped_gemm_gather(a, row_to_tk, k: int, expert_offsets, w, w_layout: int = W_KN, c=None):
    """c[r] = a[row_to_tk[r] // k] @ W_e: the grouped GEMM over token rows gathered in its loads.

    a bf16 [T, K]; row_to_tk int32 [R_cap].  Returns f32 [R_cap, N]."""
    _req(a, "a", _BF16, 2)
    _req(row_to_tk, "row_to_tk", _I32T)
    _req(expert_offsets, "expert_offsets", _I32T)
    _req(w, "w", _BF16, 3)
    T, K = a.shape
    R_cap = row_to_tk.numel()
    E = expert_offsets.numel() - 1
    N = w.shape[2] if w_layout == W_KN else w.shape[1]
    kw = w.shape[1] if w_layout == W_KN else w.shape[2]
    if kw != K or w.shape[0] != E:
        raise ValueError("weight shape does not match a / expert_offsets")
    c = _empty((R_cap, N), torch.float32, a) if c is None else c
    _req(c, "c", _F32, numel=R_cap * N)
    _check("bf16_grouped_gemm_gather", load_library().bf16_grouped_gemm_gather(
        _ptr(a), T, _ptr(row_to_tk), k, _ptr(expert_offsets), E, R_cap, _ptr(w), w_layout, N, K,
        _ptr(c), _stream()))
    return c


def swiglu_backward(gu, dh, expert_offsets, topk_w=None, row_to_tk=None, dgu=None):
    _req(gu, "gu", _F32, 2)
    _req(dh, "dh", _F32, 2)
    _req(expert_offsets, "expert_offsets", _I32T)
    _req(topk_w, "topk_w", _F32)
    _req(row_to_tk, "row_to_tk", _I32T)
    R_cap, I2 = gu.shape
    E = expert_offsets.numel() - 1
    _req(dh, "dh", _F32, numel=R_cap * (I2 // 2))
    _req(topk_w, "topk_w", _F32, numel=R_cap)
    _req(row_to_tk, "row_to_tk", _I32T, numel=R_cap)
    dgu = _empty((R_cap, I2), torch.bfloat16, gu) if dgu is None else dgu
    _req(dgu, "dgu", _BF16, numel=R_cap * I2)
    _check("swiglu_backward", load_library().swiglu_backward(
        _ptr(gu), _ptr(dh), R_cap, I2 // 2, _ptr(expert_offsets), E, _ptr(topk_w),
        _ptr(row_to_tk), _ptr(dgu), _stream()))
    return dgu


# ---------------------------------------------------------------------- FP8, 128 elements a scale
FP8_BLOCK = 128
_FP8 = (torch.uint8, torch.float8_e4m3fn)
_BF16_F32 = _BF16 + _F32
_OUT_DTYPES = {torch.float32: (OUT_F32, _F32), torch.bfloat16: (OUT_BF16, _BF16)}


def _call(name, dev, *args):
    """The entry point on device `dev` (an index) and that device's current stream.

    Small calls are bound by the host, so this asks torch for the raw stream
    (torch.cuda.current_stream builds an object around it first)."""
    fn = getattr(_LIB or load_library(), name)
    if dev == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(dev))
    if status:
        _check(name, status)


def _arg(t, name, dtypes, dev, ndim=None, numel=None):
    """_req of a tensor that must be there, and that it lies on device `dev`."""
    # one test that all is well (small calls are bound by the host), then the ones that say what is not
    if (isinstance(t, torch.Tensor) and t.dtype in dtypes and t.get_device() == dev and t.is_contiguous()
            and (ndim is None or t.dim() == ndim) and (numel is None or t.numel() >= numel) and dev >= 0):
        return
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    _req(t, name, dtypes, ndim, numel)
    raise ValueError(f"{name} is on {t.device}, expected cuda:{dev}")


def _head(t, name, dtypes, ndim):
    """_req of the argument whose device the call runs on; returns that device's index."""
    if t is None:
        raise TypeError(f"{name} must be a torch.Tensor")
    _req(t, name, dtypes, ndim)
    return t.get_device()


def _give(t, name, shape, dtype, dtypes, like, dev):
    """An output: the caller's tensor, checked, or a new one."""
    if t is None:
        return like.new_empty(shape, dtype=dtype)
    _arg(t, name, dtypes, dev, numel=math.prod(shape))
    return t


def _out_dtype(c, out_dtype):
    """(torch dtype, accepted dtypes, dtype code) of an FP32 / BF16 product's output."""
    if out_dtype is None:
        out_dtype = torch.float32 if c is None or c.dtype == torch.float32 else torch.bfloat16
    if out_dtype not in _OUT_DTYPES:
        raise TypeError("out_dtype must be torch.float32 or torch.bfloat16")
    code, dtypes = _OUT_DTYPES[out_dtype]
    return out_dtype, dtypes, code


def _blocks(n):
    return -(-n // FP8_BLOCK)


def fp8_quantize_rows(x, expert_offsets=None, codes=None, scales=None):
    """x bf16 or f32 [rows, K] -> (codes u8 [rows, K], scales f32 [ceil(K/128), rows]);
    with expert_offsets only the routed rows [0, offsets[E]) are written."""
    dev = _head(x, "x", _BF16_F32, 2)
    rows, K = x.shape
    E = 0
    if expert_offsets is not None:
        _arg(expert_offsets, "expert_offsets", _I32T, dev)
        E = expert_offsets.numel() - 1
    codes = _give(codes, "codes", (rows, K), torch.uint8, _FP8, x, dev)
    scales = _give(scales, "scales", (_blocks(K), rows), torch.float32, _F32, x, dev)
    _call("fp8_quantize_rows", dev, x.data_ptr(), x.dtype == torch.float32, rows, K, _ptr(expert_offsets), E,
          codes.data_ptr(), scales.data_ptr())
    return codes, scales


def fp8_quantize_weights(w, transposed: bool = False, out=None):
    """w bf16 [E, N, K] -> (codes u8 [E, N, K], scales f32 [E, ceil(N/128), ceil(K/128)]) by
    128 x 128 blocks; with `transposed` also the same blocks of the transposed matrices,
    (codes_t u8 [E, K, N], scales_t f32 [E, ceil(K/128), ceil(N/128)]), for the input gradient."""
    dev = _head(w, "w", _BF16, 3)
    E, N, K = w.shape
    nb, kb = _blocks(N), _blocks(K)
    o = out or {}
    res = (_give(o.get("codes"), "codes", (E, N, K), torch.uint8, _FP8, w, dev),
           _give(o.get("scales"), "scales", (E, nb, kb), torch.float32, _F32, w, dev))
    if transposed:
        res += (_give(o.get("codes_t"), "codes_t", (E, K, N), torch.uint8, _FP8, w, dev),
                _give(o.get("scales_t"), "scales_t", (E, kb, nb), torch.float32, _F32, w, dev))
    _call("fp8_quantize_weights", dev, w.data_ptr(), E, N, K, *[t.data_ptr() for t in res], *[None] * (4 - len(res)))
    return res


def fp8_swiglu_quantize(gu, expert_offsets, topk_w=None, row_to_tk=None, h_out=False, out=None):
    """Weighted SwiGLU of gu bf16 or f32 [R_cap, 2I] + FP8 quantise of the routed rows.
    Returns (codes u8 [R_cap, I], scales f32 [ceil(I/128), R_cap], h bf16 [R_cap, I] or None)."""
    dev = _head(gu, "gu", _BF16_F32, 2)
    _arg(expert_offsets, "expert_offsets", _I32T, dev)
    R_cap, I2 = gu.shape
    if I2 % 2:
        raise ValueError("gu must have 2 I columns")
    I = I2 // 2
    if topk_w is not None:
        if row_to_tk is None:
            raise ValueError("topk_w needs row_to_tk")
        _arg(topk_w, "topk_w", _F32, dev, numel=R_cap)
        _arg(row_to_tk, "row_to_tk", _I32T, dev, numel=R_cap)
    o = out or {}
    codes = _give(o.get("codes"), "codes", (R_cap, I), torch.uint8, _FP8, gu, dev)
    scales = _give(o.get("scales"), "scales", (_blocks(I), R_cap), torch.float32, _F32, gu, dev)
    h = _give(o.get("h"), "h", (R_cap, I), torch.bfloat16, _BF16, gu, dev) if h_out else None
    _call("fp8_swiglu_quantize", dev, gu.data_ptr(), gu.dtype == torch.float32, R_cap, I, _ptr(expert_offsets),
          expert_offsets.numel() - 1, _ptr(topk_w), _ptr(row_to_tk), codes.data_ptr(), scales.data_ptr(), _ptr(h))
    return codes, scales, h


def _fp8_operands(a_codes, a_scales, expert_offsets, w_codes, w_scales):
    dev = _head(a_codes, "a_codes", _FP8, 2)
    _arg(w_codes, "w_codes", _FP8, dev, 3)
    _arg(expert_offsets, "expert_offsets", _I32T, dev)
    rows, K = a_codes.shape
    E, N, kw = w_codes.shape
    if kw != K or E != expert_offsets.numel() - 1:
        raise ValueError("w_codes must be [E, N, K] for a_codes [rows, K] and expert_offsets [E + 1]")
    _arg(a_scales, "a_scales", _F32, dev)
    _arg(w_scales, "w_scales", _F32, dev)
    kb = _blocks(K)
    if tuple(a_scales.shape) != (kb, rows):
        raise ValueError(f"a_scales must be [ceil(K/128), rows] = {(kb, rows)}, got {tuple(a_scales.shape)}")
    if tuple(w_scales.shape) != (E, _blocks(N), kb):
        raise ValueError(f"w_scales must be [E, ceil(N/128), ceil(K/128)] = {(E, _blocks(N), kb)}, "
                         f"got {tuple(w_scales.shape)}")
    return dev, rows, K, E, N


def fp8_grouped_gemm(a_codes, a_scales, expert_offsets, w_codes, w_scales, c=None, out_dtype=None):
    """c[r] = dequant(A)[r] @ dequant(W_e).T over expert-grouped rows.  A: codes [R_cap, K], scales
    [ceil(K/128), R_cap]; W: codes [E, N, K], scales [E, ceil(N/128), ceil(K/128)].
    Returns [R_cap, N], float32 (default) or bfloat16 (out_dtype=torch.bfloat16, or a bf16 `c`)."""
    dev, rows, K, E, N = _fp8_operands(a_codes, a_scales, expert_offsets, w_codes, w_scales)
    dt, dtypes, code = _out_dtype(c, out_dtype)
    c = _give(c, "c", (rows, N), dt, dtypes, a_codes, dev)
    _call("fp8_grouped_gemm", dev, a_codes.data_ptr(), a_scales.data_ptr(), expert_offsets.data_ptr(), E, rows,
          w_codes.data_ptr(), w_scales.data_ptr(), N, K, c.data_ptr(), code)
    return c


def fp8_grouped_gemm_gather(a_codes, a_scales, row_to_tk, k: int, expert_offsets, w_codes, w_scales, c=None,
                            out_dtype=None):
    """fp8_grouped_gemm whose left operand is in token order: routed row r reads row
    row_to_tk[r] // k of A (codes [T, K], scales [ceil(K/128), T]).  Returns [R_cap, N]
    for row_to_tk of R_cap entries."""
    dev, T, K, E, N = _fp8_operands(a_codes, a_scales, expert_offsets, w_codes, w_scales)
    _arg(row_to_tk, "row_to_tk", _I32T, dev)
    R_cap = row_to_tk.numel()
    dt, dtypes, code = _out_dtype(c, out_dtype)
    c = _give(c, "c", (R_cap, N), dt, dtypes, a_codes, dev)
    _call("fp8_grouped_gemm_gather", dev, a_codes.data_ptr(), a_scales.data_ptr(), T, row_to_tk.data_ptr(), k,
          expert_offsets.data_ptr(), E, R_cap, w_codes.data_ptr(), w_scales.data_ptr(), N, K, c.data_ptr(), code)
    return c


def bf16_grouped_gemm_wgrad(g, x, expert_offsets, row_to_tk=None, k: int = 1, gather=None, c=None, out_dtype=None):
    """dW [E, M, N] = per expert g_e.T @ x_e over its rows (zeros for an expert without rows),
    float32 (default) or bfloat16.  g bf16 [rows, M], x bf16 [rows, N], in the expert-grouped
    order, or with gather="g" / "x" / "both" in token order: routed row r is row
    row_to_tk[r] // k of that operand."""
    if gather is None and (row_to_tk is not None or k != 1):
        raise ValueError('row_to_tk and k need gather="g", "x" or "both"')
    dev = _head(g, "g", _BF16, 2)
    _arg(x, "x", _BF16, dev, 2)
    _arg(expert_offsets, "expert_offsets", _I32T, dev)
    g_rows, M = g.shape
    x_rows, N = x.shape
    g_k = x_k = 0
    if gather is None:
        if g_rows != x_rows:
            raise ValueError("g and x must have the same rows")
        R_cap = g_rows
    else:
        if gather not in ("g", "x", "both"):
            raise ValueError('gather must be None, "g", "x" or "both"')
        if row_to_tk is None or k < 1:
            raise ValueError("gather needs row_to_tk and k >= 1")
        _arg(row_to_tk, "row_to_tk", _I32T, dev)
        R_cap = row_to_tk.numel()
        if gather != "x":
            g_k = k
        if gather != "g":
            x_k = k
        if gather != "both":
            rows = x_rows if g_k else g_rows
            if rows < R_cap:
                raise ValueError(f"the expert-grouped operand has {rows} rows, row_to_tk {R_cap} entries")
    E = expert_offsets.numel() - 1
    dt, dtypes, code = _out_dtype(c, out_dtype)
    c = _give(c, "c", (E, M, N), dt, dtypes, g, dev)
    _call("bf16_grouped_gemm_wgrad", dev, g.data_ptr(), g_rows, g_k, x.data_ptr(), x_rows, x_k,
          _ptr(row_to_tk) if gather else None, expert_offsets.data_ptr(), E, R_cap, M, N, c.data_ptr(), code)
    return c


# ---------------------------------------------------------------------- router, token sort, gradients
def moe_router_topk(logits, k: int, renorm: bool = True, ids=None, weights=None):
    """The k largest logits of each token (bf16 or f32 [T, E]; ties: the lower expert first) ->
    (topk_ids i32 [T, k], topk_w f32 [T, k]): their softmax over the k, or over all E (renorm=False)."""
    dev = _head(logits, "logits", _BF16_F32, 2)
    T, E = logits.shape
    ids = _give(ids, "ids", (T, k), torch.int32, _I32T, logits, dev)
    weights = _give(weights, "weights", (T, k), torch.float32, _F32, logits, dev)
    _call("moe_router_topk", dev, logits.data_ptr(), logits.dtype == torch.float32, T, E, k, bool(renorm),
          ids.data_ptr(), weights.data_ptr())
    return ids, weights


def moe_router_topk_backward(dweights, ids, weights, logits, renorm: bool = True, dlogits=None):
    """The gradient of moe_router_topk's logits [T, E] from that of its weights: dlogits [T, E] of the
    logits' type.  ids and weights are moe_router_topk's [T, k]; with renorm the logits are not read."""
    dev = _head(logits, "logits", _BF16_F32, 2)
    _arg(ids, "ids", _I32T, dev, 2)
    T, E = logits.shape
    k = ids.shape[1]
    if ids.shape[0] != T:
        raise ValueError("ids must have one row per token")
    _arg(weights, "weights", _F32, dev, numel=T * k)
    _arg(dweights, "dweights", _F32, dev, numel=T * k)
    dlogits = _give(dlogits, "dlogits", (T, E), logits.dtype, (logits.dtype,), logits, dev)
    _call("moe_router_topk_backward", dev, logits.data_ptr(), logits.dtype == torch.float32, ids.data_ptr(),
          weights.data_ptr(), dweights.data_ptr(), T, E, k, bool(renorm), dlogits.data_ptr())
    return dlogits


def moe_permute_workspace_size(T: int, k: int, E: int) -> int:
    """Device workspace bytes of moe_permute: 0 for short routing lists."""
    return int(load_library().moe_permute_workspace_size(T, k, E))


def moe_permute(x, topk_ids, E: int, workspace=None, dev_err=None, out=None):
    """Route + permute without quantising.  x bf16 or f32 [T, H], or None for the maps alone.  Returns dict
    with rows [T*k, H] (x's type; not with x None), expert_offsets [E+1], row_to_tk [T*k], tk_to_row [T*k].
    What lies in rows and row_to_tk at or behind expert_offsets[E] is not written: as it was in `out`, else
    uninitialised."""
    dev = _head(topk_ids, "topk_ids", _I32T, 2)
    T, k = topk_ids.shape
    R, H = T * k, 0
    shapes = {}
    if x is not None:
        _arg(x, "x", _BF16_F32, dev, 2)
        if x.shape[0] != T:
            raise ValueError("topk_ids must have one row per token")
        H = x.shape[1]
        shapes["rows"] = ((R, H), x.dtype, (x.dtype,))
    shapes |= {"expert_offsets": ((E + 1,), torch.int32, _I32T), "row_to_tk": ((R,), torch.int32, _I32T),
               "tk_to_row": ((R,), torch.int32, _I32T)}
    o = out or {}
    res = {n: _give(o.get(n), n, shp, dt, dts, topk_ids, dev) for n, (shp, dt, dts) in shapes.items()}
    if workspace is None:
        need = load_library().moe_permute_workspace_size(T, k, E)
        workspace = _empty((need,), torch.uint8, topk_ids) if need else None
    else:
        _arg(workspace, "workspace", _U8, dev)
    if dev_err is not None:
        _arg(dev_err, "dev_err", _I32T, dev, numel=1)
    _call("moe_permute", dev, _ptr(x), x is not None and x.dtype == torch.float32, T, H, topk_ids.data_ptr(), k, E,
          _ptr(res.get("rows")), res["expert_offsets"].data_ptr(), res["row_to_tk"].data_ptr(),
          res["tk_to_row"].data_ptr(), _ptr(workspace), 0 if workspace is None else workspace.numel(), _ptr(dev_err))
    return res


def _entries(tk_to_row, k, dev):
    """Tokens of a map of T * k entries."""
    _arg(tk_to_row, "tk_to_row", _I32T, dev)
    if k < 1 or tk_to_row.numel() % k:
        raise ValueError("tk_to_row must hold T * k entries")
    return tk_to_row.numel() // k


def moe_combine(d, tk_to_row, k: int, topk_w=None, y=None, out_dtype=None):
    """y[t] = sum over slots of w * d[row(t, slot)]; d bf16 or f32 [T*k, H].  Returns y [T, H], bfloat16
    (default) or float32 (out_dtype=torch.float32, or an f32 `y`).  Without weights: moe_permute's gradient."""
    dev = _head(d, "d", _BF16_F32, 2)
    T = _entries(tk_to_row, k, dev)
    rows, H = d.shape
    if rows < T * k:
        raise ValueError(f"d holds {rows} rows, needs {T * k}")
    if topk_w is not None:
        _arg(topk_w, "topk_w", _F32, dev, numel=T * k)
    if out_dtype is None and y is None:
        out_dtype = torch.bfloat16
    dt, dtypes, code = _out_dtype(y, out_dtype)
    y = _give(y, "y", (T, H), dt, dtypes, d, dev)
    _call("moe_combine", dev, d.data_ptr(), d.dtype == torch.float32, T, k, H, tk_to_row.data_ptr(), _ptr(topk_w),
          y.data_ptr(), code == OUT_F32)
    return y


def moe_combine_backward(dy, d, tk_to_row, k: int, topk_w=None, dd=None, dw=None, want_dd: bool = True):
    """The gradient of moe_combine: (dd [T*k, H], dw f32 [T, k]) from dy [T, H], both bf16 or f32.  dd has
    d's type; with d None only dd is computed, of dy's type (or the given dd's); want_dd=False: only dw."""
    dev = _head(dy, "dy", _BF16_F32, 2)
    T, H = dy.shape
    if _entries(tk_to_row, k, dev) != T:
        raise ValueError("tk_to_row must hold T * k entries for dy [T, H]")
    if d is not None:
        _arg(d, "d", _BF16_F32, dev, 2, numel=T * k * H)
        if d.shape[1] != H:
            raise ValueError("d and dy must have the same row length")
        dw = _give(dw, "dw", (T, k), torch.float32, _F32, dy, dev)
        dt = d.dtype
    else:
        if dw is not None or not want_dd:
            raise ValueError("dw needs d")
        dt = dy.dtype if dd is None else dd.dtype
    if topk_w is not None:
        _arg(topk_w, "topk_w", _F32, dev, numel=T * k)
    dd = _give(dd, "dd", (T * k, H), dt, _F32 if dt == torch.float32 else _BF16, dy, dev) if want_dd else None
    _call("moe_combine_backward", dev, dy.data_ptr(), dy.dtype == torch.float32, _ptr(d), dt == torch.float32, T, k, H,
          tk_to_row.data_ptr(), _ptr(topk_w), _ptr(dd), _ptr(dw))
    return dd, dw


def swiglu_backward_weights(gu, dh, expert_offsets, topk_w, row_to_tk, tk_to_row, dgu=None, dw=None):
    """swiglu_backward with the gradient of the router weights too: (dgu bf16 [R_cap, 2I], dw f32 of
    topk_w's shape; entries without a row have 0)."""
    dev = _head(gu, "gu", _F32, 2)
    _arg(expert_offsets, "expert_offsets", _I32T, dev)
    R_cap, I2 = gu.shape
    if I2 % 2:
        raise ValueError("gu must have 2 I columns")
    _arg(dh, "dh", _F32, dev, 2, numel=R_cap * (I2 // 2))
    _arg(topk_w, "topk_w", _F32, dev)
    if topk_w.numel() != R_cap:
        raise ValueError(f"topk_w holds {topk_w.numel()} weights for {R_cap} rows")
    _arg(row_to_tk, "row_to_tk", _I32T, dev, numel=R_cap)
    _arg(tk_to_row, "tk_to_row", _I32T, dev, numel=R_cap)
    dgu = _give(dgu, "dgu", (R_cap, I2), torch.bfloat16, _BF16, gu, dev)
    dw = _give(dw, "dw", tuple(topk_w.shape), torch.float32, _F32, gu, dev)
    _call("swiglu_backward_weights", dev, gu.data_ptr(), dh.data_ptr(), R_cap, I2 // 2, expert_offsets.data_ptr(),
          expert_offsets.numel() - 1, topk_w.data_ptr(), row_to_tk.data_ptr(), tk_to_row.data_ptr(), dgu.data_ptr(),
          dw.data_ptr())
    return dgu, dw


def grad_workspace_size(n: int) -> int:
    """Device workspace bytes of grad_norm and grad_clip for n tensors."""
    return int(load_library().moe_grad_workspace_size(n))


_DTYPE = attrgetter("dtype")
_GRAD_TYPES = {torch.float32: 1, **dict.fromkeys(_BF16, 0)}


def _grads(grads, what, dev):
    """The tensors' addresses, types and sizes as C arrays (to be kept during the call), and their device."""
    # models hold hundreds of tensors, so the checks run over the whole list; the loop names the one that fails
    if grads and all(isinstance(t, torch.Tensor) for t in grads):
        where = set(map(torch.Tensor.get_device, grads))
        types = list(map(_GRAD_TYPES.get, map(_DTYPE, grads)))
        at = where.pop()
        if not where and at >= 0 and dev in (None, at) and None not in types and all(map(torch.Tensor.is_contiguous, grads)):
            return array("Q", map(torch.Tensor.data_ptr, grads)), array("i", types), array("q", map(torch.Tensor.numel, grads)), at
    for j, t in enumerate(grads):
        if dev is None:
            dev = _head(t, f"{what}[0]", _BF16_F32, None)
        _arg(t, f"{what}[{j}]", _BF16_F32, dev)
    return array("Q"), array("i"), array("q"), dev


def _grad_buffers(n, norm, workspace, dev):
    """The device, norm and workspace of a call on n tensors of device `dev` (None: no tensors)."""
    if dev is None:
        dev = torch.cuda.current_device() if norm is None else _head(norm, "norm", _F32, None)
    where = torch.device("cuda", dev)
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=where)
    else:
        _arg(norm, "norm", _F32, dev, numel=1)
    if workspace is None:
        workspace = torch.empty(grad_workspace_size(n) or 256, dtype=torch.uint8, device=where)
    else:
        _arg(workspace, "workspace", _U8, dev)
    return dev, norm, workspace


def grad_norm(grads, norm=None, workspace=None):
    """sqrt of the sum of squares over all elements of the tensors (bf16 or f32, any shapes and alignment):
    a float32 device tensor [1]."""
    grads = list(grads)
    ptrs, types, sizes, dev = _grads(grads, "grads", None)
    dev, norm, workspace = _grad_buffers(len(grads), norm, workspace, dev)
    _call("moe_grad_norm", dev, *(a.buffer_info()[0] for a in (ptrs, types, sizes)), len(grads), norm.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return norm


def grad_clip(grads, max_norm: float, out=None, norm=None, workspace=None):
    """Scale the tensors by min(1, max_norm / (norm + 1e-6)), norm as grad_norm's: (norm f32 [1], out).
    `out`: tensors of the same sizes and types; `out=grads` clips in place; None: new ones.
    max_norm=inf: the norm alone (a factor of 1 whatever the norm).  Outputs that lie towards a 16-byte
    boundary as their tensors do are faster; new ones start at one, views into a flat buffer may not."""
    grads = list(grads)
    ptrs, types, sizes, dev = _grads(grads, "grads", None)
    out = [torch.empty_like(t) for t in grads] if out is None else list(out)
    if len(out) != len(grads):
        raise ValueError(f"{len(out)} outputs for {len(grads)} tensors")
    outs = ptrs
    if not all(map(is_, out, grads)):
        outs, otypes, osizes, _ = _grads(out, "out", dev)
        if otypes != types or osizes != sizes:
            raise ValueError("out must have the sizes and types of grads")
    dev, norm, workspace = _grad_buffers(len(grads), norm, workspace, dev)
    _call("moe_grad_clip", dev, *(a.buffer_info()[0] for a in (ptrs, outs, types, sizes)), len(grads), max_norm,
          norm.data_ptr(), workspace.data_ptr(), workspace.numel())
    return norm, out


def mfma_ceiling(iters: int, sink=None):
    """Launch the FP16 MFMA-only measurement kernel on the current stream.

    Returns (sink, flops issued).  Timing is the caller's."""
    if sink is None:
        sink = torch.empty(256 * 512, dtype=torch.float32, device="cuda")
    _req(sink, "sink", _F32, numel=256 * 512)
    _check("nvfp4moe_mfma_ceiling", load_library().nvfp4moe_mfma_ceiling(iters, _ptr(sink), _stream()))
    return sink, 256 * 8 * iters * 8 * 32768
