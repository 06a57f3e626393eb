"""Quantized MoE expert layer for AMD Instinct MI355X (gfx950).

Python binding of the C ABI in include/pmn.h (libpmn.so, built by ``build.py``). The functions
below have the ABI's names and only marshal arguments: they allocate outputs with torch on the
current device, pass raw pointers and torch's current HIP stream, and check the status code.
Every step of the computation runs in the library's HIP kernels; if the library is not built
the import fails.
"""
from __future__ import annotations

import ctypes as C
import os
from dataclasses import dataclass, fields
from typing import List, Optional, Union

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpmn.so")

P, I64, I32, U32, U64, SZ = C.c_void_p, C.c_int64, C.c_int, C.c_uint32, C.c_uint64, C.c_size_t
F32, F64 = C.c_float, C.c_double

_SIGS = {
    "pmn_strerror": (C.c_char_p, [I32]),
    "pmn_version": (I32, []),
    "pmn_padded_bound": (I64, [I64, I32]),
    "nvfp4_quantize": (I32, [P, I64, I64, I32, I64, P, P, P, P, P]),
    "nvfp4_quantize_ws_size": (SZ, []),
    "nvfp4_quantize_ws": (I32, [P, I64, I64, I32, I64, P, P, P, P, P, SZ, P]),
    "nvfp4_quantize_weights_bwd": (I32, [P, I64, I64, I64, P, P, P, P, P, U64, U32, P, SZ, P]),
    "requant_transpose_sr_mxfp8": (I32, [P, P, P, I64, I64, I64, P, I64, P, I32, I32, U64, U32, P, P, I64, P, P]),
    "mxfp8_quantize": (I32, [P, I64, I64, I32, P, I32, I32, U64, U32, P, P, I64, P, P]),
    "rht32_s2f6_quantize": (I32, [P, I32, I64, I64, U32, P, P, P]),
    "moe_grouped_gemm_fwd": (I32, [P, P, P, I64, I64, P, P, P, P, I64, P, I32, I64, I64, I64, I32, U32, P, P, P, P]),
    "moe_grouped_gemm_bwd_workspace_size": (SZ, [I64, I32, I64, I64, I32]),
    "moe_grouped_gemm_bwd": (I32, [P, P, P, P, I64, I64, P, P, P, P, I64, P, I32, I64, I64, I64, I32, I32, U64,
                                   U32, U32, U32, P, P, P, SZ, P]),
    "moe_grouped_gemm_bwd_swiglu": (I32, [P, P, P, P, P, I64, I64, P, P, P, P, I64, P, I32, I64, I64, I64, I32, U64,
                                          U32, U32, P, P, P, SZ, P]),
    "moe_grouped_gemm_fwd_mxfp8_workspace_size": (SZ, [I64, I32, I64, I64]),
    "moe_grouped_gemm_fwd_mxfp8": (I32, [P, I64, P, P, P, I32, I64, I64, I64, I32, U32, P, P, P, P, SZ, P]),
    "swiglu_bwd": (I32, [P, P, I64, I64, P, P]),
    "moe_route_topk": (I32, [P, I64, I32, I32, P, P, P, P, P, P]),
    "moe_combine_s2f6": (I32, [P, P, I64, I64, U32, P, P, I64, I32, P, P]),
    "pmn_check_indices": (I32, [P, I32, I64, P, I64, I64, P, P]),
    "pmn_noalloc_scratch_bytes": (SZ, []),
    "moe_grouped_gemm_bwd_noalloc": (I32, [P, P, P, P, I64, I64, P, P, P, P, I64, P, I32, I64, I64, I64, I32, I32,
                                           U64, U32, U32, U32, P, P, P]),
    "rmsnorm_residual_fwd": (I32, [P, P, I32, P, F32, I64, I64, P, P, P, P, P, P]),
    "rmsnorm_residual_bwd_workspace_size": (SZ, [I64, I64]),
    "rmsnorm_residual_bwd": (I32, [P, I32, P, I32, P, P, P, I64, I64, P, P, P, SZ, P]),
    "swiglu_ffn_fwd_workspace_size": (SZ, [I64, I64, I64]),
    "swiglu_ffn_fwd": (I32, [P, P, P, P, I64, I64, I64, P, P, P, SZ, P]),
    "swiglu_ffn_bwd_workspace_size": (SZ, [I64, I64, I64]),
    "swiglu_ffn_bwd": (I32, [P, P, P, P, P, I64, I64, I64, I32, P, P, P, I32, P, SZ, P]),
    "adamw_table_size": (SZ, [P, I32]),
    "adamw_table_build": (I32, [P, I32, I32, P, SZ, P]),
    "adamw_step": (I32, [P, I64, I32, F64, F64, F64, F64, I64, P, P, P, U64, U32, P]),
    "moe_grouped_gemm_fwd_bf16": (I32, [P, I64, P, P, P, I32, I64, I64, I64, I32, P, P, P]),
    "moe_grouped_gemm_bwd_bf16_workspace_size": (SZ, [I64, I32, I64, I64, I32, I32]),
    "moe_grouped_gemm_bwd_bf16": (I32, [P, P, I64, P, P, P, I32, I64, I64, I64, I32, P, P, I32, P, I32, P, SZ, P]),
    "moe_gemv_nvfp4_workspace_size": (SZ, [I64, I32, I64, I32]),
    "moe_gemv_nvfp4": (I32, [P, I32, P, P, P, I64, P, P, P, I64, I32, I32, I64, I64, I32, P, P, SZ, P]),
    "moe_combine_rows_fwd": (I32, [P, I32, I64, I64, P, P, P, I64, I32, P, I32, P]),
    "moe_combine_rows_bwd": (I32, [P, I32, P, I32, I64, I64, P, P, I64, I32, P, P, P]),
    "moe_rows_zero_unnamed": (I32, [P, I32, I64, I64, P, I64, I32, P]),
    # measurement kernels (include/pmn_probe.h)
    "pmn_probe_stream": (I32, [P, P, I64, I32, I32, I32, I32, P]),
    "pmn_probe_mfma_sink_floats": (SZ, [I32, I32]),
    "pmn_probe_mfma": (I32, [I32, I32, I32, I32, P, P, P]),
    "pmn_probe_recip_check": (I32, [U32, U32, P, P]),
}

ABI_FUNCTIONS = tuple(n for n in _SIGS if not n.startswith("pmn_"))


def _load():
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"{LIB_PATH} is not built: run `python -c 'import __graft_entry__ as g; g.build()'`")
    lib = C.CDLL(LIB_PATH)
    for name, (res, args) in _SIGS.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    return lib


_lib = _load()

# ---- constants of include/pmn.h -------------------------------------------------------------
NVFP4_WEIGHT, NVFP4_ACT, NVFP4_WEIGHT_2D = 0, 1, 2
TARGET_E4M3, TARGET_E2M1 = 0, 1
ROWWISE, COLWISE = 0, 1
RNE, SR = 0, 1
DTYPE_BF16, DTYPE_F32 = 0, 1
EPI_F32, EPI_BF16, EPI_SWIGLU, EPI_RHT32_S2F6 = 0, 1, 2, 3
BWD_DGRAD, BWD_WGRAD, BWD_FP4, BWD_W_PREPARED = 1, 2, 4, 8


CHECK_OFFSETS_START, CHECK_OFFSETS_END, CHECK_OFFSETS_ORDER, CHECK_OFFSETS_RANGE, CHECK_GATHER_RANGE = 1, 2, 4, 8, 16
_CHECK_RULES = ((CHECK_OFFSETS_START, "offsets[0] != 0"), (CHECK_OFFSETS_END, "offsets[G] != M"),
                (CHECK_OFFSETS_ORDER, "offsets decrease"), (CHECK_OFFSETS_RANGE, "an offset outside [0, M]"),
                (CHECK_GATHER_RANGE, "a gather index outside the gathered matrix"))

# PMN_CHECK_INDICES=1 in the environment: every grouped call first checks its device index arrays
# with pmn_check_indices (one small launch and a synchronization) and refuses bad ones
CHECK_INDICES = os.environ.get("PMN_CHECK_INDICES", "") not in ("", "0")


class PmnError(RuntimeError):
    pass


def _check(st: int, what: str):
    if st != 0:
        raise PmnError(f"{what}: {_lib.pmn_strerror(st).decode()} (status {st})")


def _ptr(t: Optional[torch.Tensor]):
    if t is None:
        return None
    if not t.is_cuda:
        raise PmnError("tensor must be on the GPU")
    if not t.is_contiguous():
        raise PmnError("tensor must be contiguous")
    return t.data_ptr()


def _stream():
    return torch.cuda.current_stream().cuda_stream


# ---- argument checks of the binding: the C ABI takes sizes as integers and cannot see the
# tensors, so tensors whose shape or dtype disagrees with those integers are refused here
def _need(cond: bool, what: str):
    if not cond:
        raise PmnError(what)


def _tensor(t: Optional[torch.Tensor], shape, dtype, name: str):
    if t is None or t.dtype != dtype or t.shape != shape:
        raise PmnError(f"{name} must be {dtype} of shape {tuple(shape)}"
                       + ("" if t is None else f", got {t.dtype} of shape {tuple(t.shape)}"))


def _index(t: Optional[torch.Tensor], n: int, dtype, name: str):
    if t is not None:
        _need(t.dtype == dtype and t.numel() == n, f"{name} must hold {n} values of {dtype}")


def _nvfp4(q: "NVFP4", name: str):
    _need(q.codes.dtype == torch.uint8 and q.codes.dim() == 2, f"{name}.codes must be uint8 [rows, cols/2]")
    R, C = q.rows, q.cols
    _tensor(q.scales, (R, C // 16), torch.uint8, f"{name}.scales")
    _need(q.rows_per_outer >= 1 and q.outer.dtype == torch.float32 and q.outer.numel() * q.rows_per_outer >= R,
          f"{name}.outer must be fp32 with one value per {q.rows_per_outer} rows")


def check_indices(offsets: Optional[torch.Tensor] = None, M: int = 0, gather: Optional[torch.Tensor] = None,
                  src_rows: int = 0) -> int:
    """pmn_check_indices: the mask of CHECK_* rules that the device arrays offsets [G+1] (int64)
    and gather (int32, indexing a matrix of src_rows rows) break, 0 if none. Synchronizes."""
    _need(offsets is not None or gather is not None, "check_indices needs offsets or gather")
    _need(offsets is None or (offsets.dtype == torch.int64 and offsets.numel() >= 2), "offsets must be int64 [G+1]")
    _need(gather is None or gather.dtype == torch.int32, "gather must be int32")
    dev = (offsets if offsets is not None else gather).device
    res = torch.empty(1, dtype=torch.int32, device=dev)
    G = offsets.numel() - 1 if offsets is not None else 0
    n = gather.numel() if gather is not None else 0
    _check(_lib.pmn_check_indices(_ptr(offsets), G, M, _ptr(gather), n, src_rows, _ptr(res), _stream()),
           "pmn_check_indices")
    return int(res.item()) & 0xFFFFFFFF


def _debug_indices(what: str, offsets, M: int, gather=None, src_rows: int = 0):
    if not CHECK_INDICES or (offsets is None and gather is None):
        return
    bad = check_indices(offsets, M, gather, src_rows)
    if bad:
        raise PmnError(f"{what}: the device index arrays break the contract: "
                       + ", ".join(t for b, t in _CHECK_RULES if bad & b))


def version() -> int:
    return _lib.pmn_version()


def padded_bound(M: int, G: int) -> int:
    return _lib.pmn_padded_bound(M, G)


@dataclass
class NVFP4:
    """An NVFP4 matrix [rows x cols]: codes u8 [rows, cols/2], scales u8 (E4M3) [rows, cols/16],
    outer fp32 [rows / rows_per_outer]."""
    codes: torch.Tensor
    scales: torch.Tensor
    outer: torch.Tensor
    rows_per_outer: int

    @property
    def rows(self) -> int:
        return self.codes.shape[0]

    @property
    def cols(self) -> int:
        return self.codes.shape[1] * 2


def nvfp4_quantize_ws_size() -> int:
    return _lib.nvfp4_quantize_ws_size()


def nvfp4_quantize(x: torch.Tensor, mode: int = NVFP4_ACT, rows_per_outer: int = 1,
                   outer_in: Optional[torch.Tensor] = None, out: Optional[NVFP4] = None,
                   workspace: Optional[torch.Tensor] = None) -> NVFP4:
    """NVFP4 of x; `out` (optional) supplies the output tensors to write into. With `workspace`
    (uint8, at least nvfp4_quantize_ws_size() bytes) the call goes through nvfp4_quantize_ws: the
    same outputs, weights taken in one read of x."""
    _need(x.dtype == torch.bfloat16 and x.dim() == 2, "x must be bf16 [rows, cols]")
    R, Cc = x.shape
    dev = x.device
    n_outer = max(R // max(rows_per_outer, 1), 0)
    if out is None:
        codes = torch.empty((R, Cc // 2), dtype=torch.uint8, device=dev)
        scales = torch.empty((R, Cc // 16), dtype=torch.uint8, device=dev)
        outer = torch.empty((n_outer,), dtype=torch.float32, device=dev)
    else:
        codes, scales, outer = out.codes, out.scales, out.outer
        _tensor(codes, (R, Cc // 2), torch.uint8, "out.codes")
        _tensor(scales, (R, Cc // 16), torch.uint8, "out.scales")
        _tensor(outer, (n_outer,), torch.float32, "out.outer")
    if workspace is None:
        _check(_lib.nvfp4_quantize(_ptr(x), R, Cc, mode, rows_per_outer, _ptr(outer_in), _ptr(codes),
                                   _ptr(scales), _ptr(outer), _stream()), "nvfp4_quantize")
    else:
        _need(workspace.dtype == torch.uint8, "workspace must be uint8")
        _check(_lib.nvfp4_quantize_ws(_ptr(x), R, Cc, mode, rows_per_outer, _ptr(outer_in), _ptr(codes),
                                      _ptr(scales), _ptr(outer), _ptr(workspace), workspace.numel(), _stream()),
               "nvfp4_quantize_ws")
    return NVFP4(codes, scales, outer, rows_per_outer)


@dataclass
class WeightsBwd:
    """Weights quantized for both passes (nvfp4_quantize_weights_bwd): q, the NVFP4 matrix for
    the forward, and the backward's W^T operand, wt u8 [cols, rows] (E4M3 codes, blocked layout)
    with wte u8 [rows/32, cols] (E8M0), drawn with (seed, rng_stream). The backward calls take it
    in place of the NVFP4 weights."""
    q: NVFP4
    wt: torch.Tensor
    wte: torch.Tensor
    seed: int
    rng_stream: int


def nvfp4_quantize_weights_bwd(w: torch.Tensor, rows_per_outer: int, seed: int = 0, rng_stream: int = 2,
                               workspace: Optional[torch.Tensor] = None) -> WeightsBwd:
    """nvfp4_quantize_weights_bwd: w bf16 [rows, cols] (rows % 64 == 0) in weight mode with one
    outer scale per rows_per_outer rows, and its W^T operand for the backward's dgrad."""
    _need(w.dtype == torch.bfloat16 and w.dim() == 2, "w must be bf16 [rows, cols]")
    R, Cc = w.shape
    dev = w.device
    if workspace is None:
        workspace = torch.empty((nvfp4_quantize_ws_size(),), dtype=torch.uint8, device=dev)
    _need(workspace.dtype == torch.uint8, "workspace must be uint8")
    codes = torch.empty((R, Cc // 2), dtype=torch.uint8, device=dev)
    scales = torch.empty((R, Cc // 16), dtype=torch.uint8, device=dev)
    outer = torch.empty((R // max(rows_per_outer, 1),), dtype=torch.float32, device=dev)
    wt = torch.empty((Cc, R), dtype=torch.uint8, device=dev)
    wte = torch.empty((R // 32, Cc), dtype=torch.uint8, device=dev)
    _check(_lib.nvfp4_quantize_weights_bwd(_ptr(w), R, Cc, rows_per_outer, _ptr(codes), _ptr(scales), _ptr(outer),
                                           _ptr(wt), _ptr(wte), seed, rng_stream, _ptr(workspace),
                                           workspace.numel(), _stream()), "nvfp4_quantize_weights_bwd")
    return WeightsBwd(NVFP4(codes, scales, outer, rows_per_outer), wt, wte, seed, rng_stream)


def _bwd_weights(wq, G: int, N: int, K: int):
    """(codes, scales, outer, rows_per_outer, extra flags) of the backward's weight operand: the
    NVFP4 weights, or a WeightsBwd's prepared W^T (PMN_BWD_W_PREPARED)."""
    if isinstance(wq, WeightsBwd):
        _need(wq.q.cols == K and wq.q.rows == G * N, f"wq must be [G*N, K] = [{G * N}, {K}]")
        _tensor(wq.wt, (K, G * N), torch.uint8, "wq.wt")
        _tensor(wq.wte, (G * N // 32, K), torch.uint8, "wq.wte")
        return _ptr(wq.wt), _ptr(wq.wte), None, 1, BWD_W_PREPARED
    _nvfp4(wq, "wq")
    _need(wq.cols == K and wq.rows == G * N, f"wq must be [G*N, K] = [{G * N}, {K}], got [{wq.rows}, {wq.cols}]")
    return _ptr(wq.codes), _ptr(wq.scales), _ptr(wq.outer), wq.rows_per_outer, 0


def requant_transpose_sr_mxfp8(q: NVFP4, gather: Optional[torch.Tensor] = None,
                               offsets: Optional[torch.Tensor] = None, M: Optional[int] = None,
                               target: int = TARGET_E4M3, seed: int = 0, rng_stream: int = 0,
                               ld: Optional[int] = None, want_padded_offsets: bool = False,
                               out: Optional[torch.Tensor] = None, out_e8m0: Optional[torch.Tensor] = None):
    """Returns (out [cols, ld] u8, out_e8m0 [cols, ld/32] u8, padded_offsets or None); columns
    past the padded total are not written."""
    if M is None:
        M = gather.numel() if gather is not None else q.rows
    G = 0 if offsets is None else offsets.numel() - 1
    if ld is None:
        ld = padded_bound(M, G)
    dev = q.codes.device
    _nvfp4(q, "q")
    _index(gather, M, torch.int32, "gather")
    _index(offsets, G + 1, torch.int64, "offsets")
    _debug_indices("requant_transpose_sr_mxfp8", offsets, M, gather, q.rows)
    out = torch.empty((q.cols, ld), dtype=torch.uint8, device=dev) if out is None else out
    oe = torch.empty((q.cols, ld // 32), dtype=torch.uint8, device=dev) if out_e8m0 is None else out_e8m0
    _tensor(out, (q.cols, ld), torch.uint8, "out")
    _tensor(oe, (q.cols, ld // 32), torch.uint8, "out_e8m0")
    po = torch.zeros((max(G, 1) + 1,), dtype=torch.int64, device=dev) if want_padded_offsets else None
    _check(_lib.requant_transpose_sr_mxfp8(_ptr(q.codes), _ptr(q.scales), _ptr(q.outer), q.rows, q.cols,
                                           q.rows_per_outer, _ptr(gather), M, _ptr(offsets), G, target, seed,
                                           rng_stream, _ptr(out), _ptr(oe), ld, _ptr(po), _stream()),
           "requant_transpose_sr_mxfp8")
    return out, oe, po


def mxfp8_quantize(x: torch.Tensor, layout: int = ROWWISE, offsets: Optional[torch.Tensor] = None,
                   rounding: int = RNE, seed: int = 0, rng_stream: int = 0, ld: Optional[int] = None,
                   want_padded_offsets: bool = False):
    _need(x.dtype == torch.bfloat16 and x.dim() == 2, "x must be bf16 [M, N]")
    M, N = x.shape
    dev = x.device
    G = 0 if offsets is None else offsets.numel() - 1
    _index(offsets, G + 1, torch.int64, "offsets")
    _debug_indices("mxfp8_quantize", offsets, M)
    po = None
    if layout == ROWWISE:
        out = torch.empty((M, N), dtype=torch.uint8, device=dev)
        oe = torch.empty((M, N // 32), dtype=torch.uint8, device=dev)
        ld = N
    else:
        if ld is None:
            ld = padded_bound(M, G)
        out = torch.empty((N, ld), dtype=torch.uint8, device=dev)
        oe = torch.empty((N, ld // 32), dtype=torch.uint8, device=dev)
        po = torch.zeros((max(G, 1) + 1,), dtype=torch.int64, device=dev) if want_padded_offsets else None
    _check(_lib.mxfp8_quantize(_ptr(x), M, N, layout, _ptr(offsets), G, rounding, seed, rng_stream, _ptr(out),
                               _ptr(oe), ld, _ptr(po), _stream()), "mxfp8_quantize")
    return out, oe, po


def rht32_s2f6_quantize(x: torch.Tensor, sign_mask: int):
    _need(x.dim() == 2 and x.dtype in (torch.bfloat16, torch.float32), "x must be bf16 or fp32 [rows, cols]")
    R, Cc = x.shape
    codes = torch.empty((R, Cc), dtype=torch.int8, device=x.device)
    e = torch.empty((R, Cc // 32), dtype=torch.uint8, device=x.device)
    _check(_lib.rht32_s2f6_quantize(_ptr(x), DTYPE_F32 if x.dtype == torch.float32 else DTYPE_BF16, R, Cc,
                                    sign_mask & 0xFFFFFFFF, _ptr(codes), _ptr(e), _stream()), "rht32_s2f6_quantize")
    return codes, e


def moe_grouped_gemm_fwd(xq: NVFP4, wq: NVFP4, offsets: torch.Tensor, M: int, N: int,
                         epilogue: int = EPI_F32, gather: Optional[torch.Tensor] = None,
                         rht_sign_mask: int = 0, save_h13: bool = False, out=None, out_e8m0=None,
                         out_aux=None):
    """Y = grouped NVFP4 product; returns the epilogue's outputs (see include/pmn.h)."""
    K = xq.cols
    G = offsets.numel() - 1
    dev = xq.codes.device
    _nvfp4(xq, "xq")
    _nvfp4(wq, "wq")
    _need(wq.cols == K and wq.rows == G * N, f"wq must be [G*N, K] = [{G * N}, {K}], got [{wq.rows}, {wq.cols}]")
    _index(offsets, G + 1, torch.int64, "offsets")
    _index(gather, M, torch.int32, "gather")
    _debug_indices("moe_grouped_gemm_fwd", offsets, M, gather, xq.rows)
    if out is None:
        if epilogue == EPI_F32:
            out = torch.empty((M, N), dtype=torch.float32, device=dev)
        elif epilogue == EPI_BF16:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        elif epilogue == EPI_SWIGLU:
            out = torch.empty((M, N // 2), dtype=torch.bfloat16, device=dev)
        else:
            out = torch.empty((M, N), dtype=torch.int8, device=dev)
    if epilogue == EPI_RHT32_S2F6 and out_e8m0 is None:
        out_e8m0 = torch.empty((M, N // 32), dtype=torch.uint8, device=dev)
    if epilogue == EPI_SWIGLU and save_h13 and out_aux is None:
        out_aux = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _epilogue_outputs(epilogue, M, N, out, out_e8m0, out_aux)
    _check(_lib.moe_grouped_gemm_fwd(_ptr(xq.codes), _ptr(xq.scales), _ptr(xq.outer), xq.rows, xq.rows_per_outer,
                                     _ptr(gather), _ptr(wq.codes), _ptr(wq.scales), _ptr(wq.outer),
                                     wq.rows_per_outer, _ptr(offsets), G, M, N, K, epilogue,
                                     rht_sign_mask & 0xFFFFFFFF, _ptr(out), _ptr(out_e8m0), _ptr(out_aux), _stream()),
           "moe_grouped_gemm_fwd")
    if epilogue == EPI_RHT32_S2F6:
        return out, out_e8m0
    if epilogue == EPI_SWIGLU:
        return out, out_aux
    return out


def _epilogue_outputs(epilogue: int, M: int, N: int, out, out_e8m0, out_aux):
    shape, dtype = {EPI_F32: ((M, N), torch.float32), EPI_BF16: ((M, N), torch.bfloat16),
                    EPI_SWIGLU: ((M, N // 2), torch.bfloat16)}.get(epilogue, ((M, N), torch.int8))
    _tensor(out, shape, dtype, "out")
    if epilogue == EPI_RHT32_S2F6:
        _tensor(out_e8m0, (M, N // 32), torch.uint8, "out_e8m0")
    if epilogue == EPI_SWIGLU and out_aux is not None:
        _tensor(out_aux, (M, N), torch.bfloat16, "out_aux")


def moe_grouped_gemm_bwd_workspace_size(M: int, G: int, N: int, K: int, flags: int) -> int:
    return _lib.moe_grouped_gemm_bwd_workspace_size(M, G, N, K, flags)


def moe_grouped_gemm_fwd_mxfp8(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, M: int, N: int,
                               epilogue: int = EPI_F32, gather: Optional[torch.Tensor] = None,
                               rht_sign_mask: int = 0, save_h13: bool = False, workspace=None, out=None,
                               out_e8m0=None, out_aux=None):
    """MXFP8 forward (row-wise RNE quantization of x and w inside the call); returns the
    epilogue's outputs as moe_grouped_gemm_fwd does."""
    K = x.shape[1]
    G = offsets.numel() - 1
    dev = w.device
    _need(x.dtype == torch.bfloat16 and x.dim() == 2, "x must be bf16 [rows, K]")
    _tensor(w, (G * N, K), torch.bfloat16, "w")
    _index(offsets, G + 1, torch.int64, "offsets")
    _index(gather, M, torch.int32, "gather")
    _debug_indices("moe_grouped_gemm_fwd_mxfp8", offsets, M, gather, x.shape[0])
    if workspace is None:
        workspace = torch.empty((_lib.moe_grouped_gemm_fwd_mxfp8_workspace_size(M, G, N, K),), dtype=torch.uint8,
                                device=dev)
    if out is None:
        if epilogue == EPI_F32:
            out = torch.empty((M, N), dtype=torch.float32, device=dev)
        elif epilogue == EPI_BF16:
            out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
        elif epilogue == EPI_SWIGLU:
            out = torch.empty((M, N // 2), dtype=torch.bfloat16, device=dev)
        else:
            out = torch.empty((M, N), dtype=torch.int8, device=dev)
    if epilogue == EPI_RHT32_S2F6 and out_e8m0 is None:
        out_e8m0 = torch.empty((M, N // 32), dtype=torch.uint8, device=dev)
    if epilogue == EPI_SWIGLU and save_h13 and out_aux is None:
        out_aux = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _epilogue_outputs(epilogue, M, N, out, out_e8m0, out_aux)
    _need(workspace.dtype == torch.uint8 and workspace.dim() == 1, "workspace must be a 1-D uint8 tensor")
    _check(_lib.moe_grouped_gemm_fwd_mxfp8(_ptr(x), x.shape[0], _ptr(gather), _ptr(w), _ptr(offsets), G, M, N, K,
                                           epilogue, rht_sign_mask & 0xFFFFFFFF, _ptr(out), _ptr(out_e8m0),
                                           _ptr(out_aux), _ptr(workspace), workspace.numel(), _stream()),
           "moe_grouped_gemm_fwd_mxfp8")
    if epilogue == EPI_RHT32_S2F6:
        return out, out_e8m0
    if epilogue == EPI_SWIGLU:
        return out, out_aux
    return out


def moe_grouped_gemm_bwd(dy: torch.Tensor, xq: NVFP4, wq, offsets: torch.Tensor, M: int, N: int,
                         flags: int = BWD_DGRAD | BWD_WGRAD, gather: Optional[torch.Tensor] = None,
                         dy_rounding: int = RNE, seed: int = 0, rng_stream_a: int = 1, rng_stream_b: int = 2,
                         rng_stream_dy: int = 3, workspace: Optional[torch.Tensor] = None, da=None, db=None):
    """wq: the NVFP4 weights [G*N, K], or a WeightsBwd (its prepared W^T, PMN_BWD_W_PREPARED).
    Returns (da [M, K] fp32 or None, db [G*N, K] fp32 or None, workspace)."""
    K = xq.cols
    G = offsets.numel() - 1
    dev = dy.device
    _tensor(dy, (M, N), torch.bfloat16, "dy")
    _nvfp4(xq, "xq")
    bc, bs, bo, brpo, wflag = _bwd_weights(wq, G, N, K)
    flags |= wflag
    _index(offsets, G + 1, torch.int64, "offsets")
    _index(gather, M, torch.int32, "gather")
    _debug_indices("moe_grouped_gemm_bwd", offsets, M, gather, xq.rows)
    ws_bytes = moe_grouped_gemm_bwd_workspace_size(M, G, N, K, flags)
    if workspace is None:
        workspace = torch.empty((ws_bytes,), dtype=torch.uint8, device=dev)
    if da is None and flags & BWD_DGRAD:
        da = torch.empty((M, K), dtype=torch.float32, device=dev)
    if db is None and flags & BWD_WGRAD:
        db = torch.empty((G * N, K), dtype=torch.float32, device=dev)
    if flags & BWD_DGRAD:
        _tensor(da, (M, K), torch.float32, "da")
    if flags & BWD_WGRAD:
        _tensor(db, (G * N, K), torch.float32, "db")
    _need(workspace.dtype == torch.uint8 and workspace.dim() == 1, "workspace must be a 1-D uint8 tensor")
    _check(_lib.moe_grouped_gemm_bwd(_ptr(dy), _ptr(xq.codes), _ptr(xq.scales), _ptr(xq.outer), xq.rows,
                                     xq.rows_per_outer, _ptr(gather), bc, bs, bo, brpo, _ptr(offsets), G, M, N, K,
                                     flags, dy_rounding, seed,
                                     rng_stream_a, rng_stream_b, rng_stream_dy, _ptr(da), _ptr(db),
                                     _ptr(workspace), workspace.numel(), _stream()), "moe_grouped_gemm_bwd")
    return da, db, workspace


def moe_grouped_gemm_bwd_swiglu(da_act: torch.Tensor, h13: torch.Tensor, xq: NVFP4, wq,
                                offsets: torch.Tensor, M: int, N: int, gather: Optional[torch.Tensor] = None,
                                seed: int = 0, rng_stream_a: int = 1, rng_stream_b: int = 2,
                                workspace: Optional[torch.Tensor] = None, dx=None, dw=None):
    """The w1||w3 backward with the SwiGLU backward folded into dY's quantization: the results of
    swiglu_bwd(da_act, h13) followed by moe_grouped_gemm_bwd(..., both gradients, RNE).
    Returns (dx [M, K] fp32, dw [G*N, K] fp32, workspace)."""
    K = xq.cols
    G = offsets.numel() - 1
    dev = h13.device
    _tensor(da_act, (M, N // 2), torch.float32, "da_act")
    _tensor(h13, (M, N), torch.bfloat16, "h13")
    _nvfp4(xq, "xq")
    bc, bs, bo, brpo, wflag = _bwd_weights(wq, G, N, K)
    _index(offsets, G + 1, torch.int64, "offsets")
    _index(gather, M, torch.int32, "gather")
    _debug_indices("moe_grouped_gemm_bwd_swiglu", offsets, M, gather, xq.rows)
    ws_bytes = moe_grouped_gemm_bwd_workspace_size(M, G, N, K, BWD_DGRAD | BWD_WGRAD)
    if workspace is None:
        workspace = torch.empty((ws_bytes,), dtype=torch.uint8, device=dev)
    dx = torch.empty((M, K), dtype=torch.float32, device=dev) if dx is None else dx
    dw = torch.empty((G * N, K), dtype=torch.float32, device=dev) if dw is None else dw
    _tensor(dx, (M, K), torch.float32, "dx")
    _tensor(dw, (G * N, K), torch.float32, "dw")
    _need(workspace.dtype == torch.uint8 and workspace.dim() == 1, "workspace must be a 1-D uint8 tensor")
    _check(_lib.moe_grouped_gemm_bwd_swiglu(_ptr(da_act), _ptr(h13), _ptr(xq.codes), _ptr(xq.scales), _ptr(xq.outer),
                                            xq.rows, xq.rows_per_outer, _ptr(gather), bc, bs, bo, brpo,
                                            _ptr(offsets), G, M, N, K, wflag, seed, rng_stream_a, rng_stream_b,
                                            _ptr(dx), _ptr(dw),
                                            _ptr(workspace), workspace.numel(), _stream()),
           "moe_grouped_gemm_bwd_swiglu")
    return dx, dw, workspace


def moe_grouped_gemm_bwd_noalloc(dy: torch.Tensor, xq: "NVFP4", wq, offsets: torch.Tensor, M: int, N: int,
                                 flags: int = BWD_DGRAD | BWD_WGRAD, gather: Optional[torch.Tensor] = None,
                                 dy_rounding: int = RNE, seed: int = 0, rng_stream_a: int = 1, rng_stream_b: int = 2,
                                 rng_stream_dy: int = 3, da=None, db=None):
    """moe_grouped_gemm_bwd with the library's static scratch as its workspace (no workspace
    argument; the C call allocates nothing). Returns (da or None, db or None)."""
    K = xq.cols
    G = offsets.numel() - 1
    dev = dy.device
    _tensor(dy, (M, N), torch.bfloat16, "dy")
    _nvfp4(xq, "xq")
    bc, bs, bo, brpo, wflag = _bwd_weights(wq, G, N, K)
    flags |= wflag
    _index(offsets, G + 1, torch.int64, "offsets")
    _index(gather, M, torch.int32, "gather")
    _debug_indices("moe_grouped_gemm_bwd_noalloc", offsets, M, gather, xq.rows)
    if da is None and flags & BWD_DGRAD:
        da = torch.empty((M, K), dtype=torch.float32, device=dev)
    if db is None and flags & BWD_WGRAD:
        db = torch.empty((G * N, K), dtype=torch.float32, device=dev)
    if flags & BWD_DGRAD:
        _tensor(da, (M, K), torch.float32, "da")
    if flags & BWD_WGRAD:
        _tensor(db, (G * N, K), torch.float32, "db")
    _check(_lib.moe_grouped_gemm_bwd_noalloc(_ptr(dy), _ptr(xq.codes), _ptr(xq.scales), _ptr(xq.outer), xq.rows,
                                             xq.rows_per_outer, _ptr(gather), bc, bs, bo, brpo, _ptr(offsets), G, M,
                                             N, K, flags,
                                             dy_rounding, seed, rng_stream_a, rng_stream_b, rng_stream_dy, _ptr(da),
                                             _ptr(db), _stream()), "moe_grouped_gemm_bwd_noalloc")
    return da, db


def bwd_workspace_views(workspace: torch.Tensor, M: int, G: int, N: int, K: int, fp4: bool = False):
    """Views of the backward workspace parts, in the order include/pmn.h documents them: groups
    padded to U = 64 slots (E4M3) or 128 (FP4: E2M1 codes packed two per byte, rows of half the
    bytes) and the code parts (dq at padded slot rows, wt, dt, xt) in the blocked layout, viewed
    here as raw bytes of the matrix's shape."""
    U = 128 if fp4 else 64
    Pb = (M + U - 1) // U * U + U * G
    h = 2 if fp4 else 1
    Nk = (N + U - 1) // U * U   # dgrad's contraction: N rounded up to a whole stage (64 E4M3 / 128 E2M1 values)
    sizes = [("dq", Pb * Nk // h, (Pb, Nk // h)), ("de", N // 32 * Pb, (N // 32, Pb)),
             ("wt", K * G * Nk // h, (K, G * Nk // h)), ("wte", K * G * Nk // 32, (G * Nk // 32, K)),
             ("dt", N * Pb // h, (N, Pb // h)), ("dte", N * Pb // 32, (Pb // 32, N)),
             ("xt", K * Pb // h, (K, Pb // h)), ("xte", K * Pb // 32, (Pb // 32, K)), ("po", (G + 1) * 8, None),
             ("woff", (G + 1) * 8, None)]
    off, views = 0, {}
    for name, nbytes, shape in sizes:
        used = nbytes if shape is None else shape[0] * shape[1]
        part = workspace[off:off + used]
        views[name] = part.view(torch.int64) if shape is None else part.view(*shape)
        off += (nbytes + 255) // 256 * 256
    return views


def swiglu_bwd(da: torch.Tensor, h13: torch.Tensor) -> torch.Tensor:
    _need(da.dtype == torch.float32 and da.dim() == 2, "da must be fp32 [M, F]")
    M, F = da.shape
    _tensor(h13, (M, 2 * F), torch.bfloat16, "h13")
    out = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=da.device)
    _check(_lib.swiglu_bwd(_ptr(da), _ptr(h13), M, F, _ptr(out), _stream()), "swiglu_bwd")
    return out


def moe_route_topk(logits: torch.Tensor, k: int):
    """Returns dict(ids, gates, offsets, gather, slot_of) on the device."""
    _need(logits.dtype == torch.float32 and logits.dim() == 2, "logits must be fp32 [T, E]")
    T, E = logits.shape
    dev = logits.device
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    gates = torch.empty((T, k), dtype=torch.float32, device=dev)
    offsets = torch.empty((E + 1,), dtype=torch.int64, device=dev)
    gather = torch.empty((T * k,), dtype=torch.int32, device=dev)
    slot_of = torch.empty((T * k,), dtype=torch.int32, device=dev)
    _check(_lib.moe_route_topk(_ptr(logits), T, E, k, _ptr(ids), _ptr(gates), _ptr(offsets), _ptr(gather),
                               _ptr(slot_of), _stream()), "moe_route_topk")
    return dict(ids=ids, gates=gates, offsets=offsets, gather=gather, slot_of=slot_of)


def moe_combine_s2f6(codes: torch.Tensor, e8m0: torch.Tensor, sign_mask: int, slot_of: torch.Tensor,
                     gates: torch.Tensor, out=None):
    """Receiver side of the combine: bf16 [T x H], row t = sum_j gates[t, j] * decode(codes[slot_of[t, j]])."""
    _need(codes.dtype == torch.int8 and codes.dim() == 2, "codes must be int8 [M, H]")
    M, H = codes.shape
    _tensor(e8m0, (M, H // 32), torch.uint8, "e8m0")
    _need(gates.dtype == torch.float32 and gates.dim() == 2, "gates must be fp32 [T, k]")
    T, k = gates.shape
    _index(slot_of, T * k, torch.int32, "slot_of")
    _need(slot_of is not None, "slot_of is required")
    if out is None:
        out = torch.empty((T, H), dtype=torch.bfloat16, device=codes.device)
    _tensor(out, (T, H), torch.bfloat16, "out")
    _check(_lib.moe_combine_s2f6(_ptr(codes), _ptr(e8m0), M, H, sign_mask & 0xFFFFFFFF, _ptr(slot_of), _ptr(gates),
                                 T, k, _ptr(out), _stream()), "moe_combine_s2f6")
    return out


# ---- around the routed experts: the norm, the shared expert and the weight update -----------

def _dtype_code(t: torch.Tensor, name: str) -> int:
    _need(t.dtype in (torch.bfloat16, torch.float32), f"{name} must be bf16 or fp32")
    return DTYPE_F32 if t.dtype == torch.float32 else DTYPE_BF16


def _device_ptr(t: Optional[torch.Tensor], dev: int, name: str):
    """Pointer of a contiguous tensor on device dev (None for None)."""
    if t is None:
        return None
    at = t.get_device()
    if at != dev:
        raise PmnError(f"{name} must be on the GPU" if at < 0 else f"{name} is on cuda:{at}, the call is for cuda:{dev}")
    if not t.is_contiguous():
        raise PmnError(f"{name} must be contiguous")
    return t.data_ptr()


def _device_of(t: torch.Tensor, name: str) -> int:
    """The device of t, which must be the current one: the call goes to its current stream."""
    dev = t.get_device()
    if dev < 0:
        raise PmnError(f"{name} must be on the GPU")
    current = torch.cuda.current_device()
    if dev != current:
        raise PmnError(f"{name} is on cuda:{dev}, the current device is cuda:{current}")
    return dev


def _raw_stream(dev: int) -> int:
    return torch._C._cuda_getCurrentRawStream(dev)   # current_stream(dev).cuda_stream without its objects


def _workspace(workspace: Optional[torch.Tensor], nbytes: int, device) -> torch.Tensor:
    if workspace is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    _need(workspace.dtype == torch.uint8 and workspace.dim() == 1, "workspace must be a 1-D uint8 tensor")
    return workspace


@dataclass
class RmsNorm:
    """Outputs of rmsnorm_residual_fwd; what was not asked for is None. y bf16; codes u8 (E4M3)
    [rows, cols] with e8m0 u8 [rows, cols/32]; z the residual stream after the addition (None without
    a residual); rstd fp32 [rows]."""
    y: Optional[torch.Tensor]
    codes: Optional[torch.Tensor]
    e8m0: Optional[torch.Tensor]
    z: Optional[torch.Tensor]
    rstd: Optional[torch.Tensor]


def rmsnorm_residual_fwd(x: torch.Tensor, gamma: torch.Tensor, eps: float = 1e-6,
                         residual: Optional[torch.Tensor] = None, want_y: bool = True, want_mxfp8: bool = False,
                         want_rstd: bool = False, z_out: Optional[torch.Tensor] = None) -> RmsNorm:
    """RMS norm of x (+ residual), bf16 [rows, cols]; residual bf16 or fp32, z_out (optional, it may be
    residual itself) receives the sum. want_y: the bf16 output; want_mxfp8: the row-wise MXFP8 output;
    want_rstd: what the backward needs."""
    _need(x.dtype == torch.bfloat16 and x.dim() == 2, "x must be bf16 [rows, cols]")
    shape = x.shape
    R, Cc = shape
    _tensor(gamma, (Cc,), torch.float32, "gamma")
    _need(want_y or want_mxfp8, "want_y or want_mxfp8 must be set")
    _need(not want_mxfp8 or Cc % 32 == 0, "MXFP8 output needs cols to be a multiple of 32")
    rcode = DTYPE_BF16
    if residual is not None:
        rcode = _dtype_code(residual, "residual")
        _tensor(residual, shape, residual.dtype, "residual")
        if z_out is not None:
            _tensor(z_out, shape, residual.dtype, "z_out")
    else:
        _need(z_out is None, "z_out needs a residual")
    at = _device_of(x, "x")
    dev = x.device
    if residual is not None and z_out is None:
        z_out = torch.empty_like(residual)
    y = torch.empty_like(x) if want_y else None
    codes = torch.empty(shape, dtype=torch.uint8, device=dev) if want_mxfp8 else None
    e8m0 = torch.empty((R, Cc // 32), dtype=torch.uint8, device=dev) if want_mxfp8 else None
    rstd = torch.empty(R, dtype=torch.float32, device=dev) if want_rstd else None
    _check(_lib.rmsnorm_residual_fwd(
        _device_ptr(x, at, "x"), _device_ptr(residual, at, "residual"), rcode, _device_ptr(gamma, at, "gamma"), eps, R,
        Cc, _device_ptr(z_out, at, "z_out"), _device_ptr(y, at, "y"), _device_ptr(codes, at, "codes"),
        _device_ptr(e8m0, at, "e8m0"), _device_ptr(rstd, at, "rstd"), _raw_stream(at)), "rmsnorm_residual_fwd")
    return RmsNorm(y, codes, e8m0, z_out, rstd)


def rmsnorm_residual_bwd(dy: torch.Tensor, z: torch.Tensor, gamma: torch.Tensor, rstd: torch.Tensor,
                         dres: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
                         dz: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None):
    """Backward of rmsnorm_residual_fwd: z its residual stream (x where there was no residual), dres the
    gradient that reaches z along the stream; dz (it may be dres itself) and dgamma (the gradient of an
    AdamWTensor, for one) may be given. Returns (dz [rows, cols] of z's type, dgamma fp32 [cols])."""
    _need(z.dim() == 2, "z must be [rows, cols]")
    R, Cc = z.shape
    zcode, dcode = _dtype_code(z, "z"), _dtype_code(dy, "dy")
    _tensor(dy, (R, Cc), dy.dtype, "dy")
    _tensor(gamma, (Cc,), torch.float32, "gamma")
    _tensor(rstd, (R,), torch.float32, "rstd")
    if dres is not None:
        _tensor(dres, (R, Cc), z.dtype, "dres")
    if dz is not None:
        _tensor(dz, (R, Cc), z.dtype, "dz")
    if dgamma is not None:
        _tensor(dgamma, (Cc,), torch.float32, "dgamma")
    at = _device_of(z, "z")
    dz = torch.empty_like(z) if dz is None else dz
    workspace = _workspace(workspace, _lib.rmsnorm_residual_bwd_workspace_size(R, Cc), z.device)
    dgamma = torch.empty_like(gamma) if dgamma is None else dgamma
    _check(_lib.rmsnorm_residual_bwd(
        _device_ptr(dy, at, "dy"), dcode, _device_ptr(z, at, "z"), zcode, _device_ptr(gamma, at, "gamma"),
        _device_ptr(rstd, at, "rstd"), _device_ptr(dres, at, "dres"), R, Cc, _device_ptr(dz, at, "dz"),
        _device_ptr(dgamma, at, "dgamma"), _device_ptr(workspace, at, "workspace"), workspace.numel(),
        _raw_stream(at)), "rmsnorm_residual_bwd")
    return dz, dgamma


def swiglu_ffn_fwd_workspace_size(M: int, H: int, F: int) -> int:
    return _lib.swiglu_ffn_fwd_workspace_size(M, H, F)


def swiglu_ffn_bwd_workspace_size(M: int, H: int, F: int) -> int:
    return _lib.swiglu_ffn_bwd_workspace_size(M, H, F)


def _ffn_weights(w13: torch.Tensor, w2: torch.Tensor, H: int) -> int:
    _need(w2.dim() == 2 and w2.shape[0] == H, f"w2 must be bf16 [{H}, F]")
    F = w2.shape[1]
    _tensor(w2, (H, F), torch.bfloat16, "w2")
    _tensor(w13, (2 * F, H), torch.bfloat16, "w13")
    return F


def swiglu_ffn_fwd(x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, add: Optional[torch.Tensor] = None,
                   save_h13: bool = False, workspace: Optional[torch.Tensor] = None,
                   out: Optional[torch.Tensor] = None):
    """The dense gated block y = (silu(x w1^T) * (x w3^T)) w2^T (+ add), bf16: x [M, H], w13 [2F, H] (w1
    over w3), w2 [H, F]; out may be add itself. Returns (y, h13 [M, 2F] for the backward or None)."""
    _need(x.dtype == torch.bfloat16 and x.dim() == 2, "x must be bf16 [M, H]")
    M, H = x.shape
    F = _ffn_weights(w13, w2, H)
    if add is not None:
        _tensor(add, (M, H), torch.bfloat16, "add")
    if out is not None:
        _tensor(out, (M, H), torch.bfloat16, "out")
    at = _device_of(x, "x")
    workspace = _workspace(workspace, _lib.swiglu_ffn_fwd_workspace_size(M, H, F), x.device)
    out = torch.empty_like(x) if out is None else out
    h13 = torch.empty((M, 2 * F), dtype=torch.bfloat16, device=x.device) if save_h13 else None
    _check(_lib.swiglu_ffn_fwd(
        _device_ptr(x, at, "x"), _device_ptr(w13, at, "w13"), _device_ptr(w2, at, "w2"), _device_ptr(add, at, "add"), M,
        H, F, _device_ptr(h13, at, "h13"), _device_ptr(out, at, "out"), _device_ptr(workspace, at, "workspace"),
        workspace.numel(), _raw_stream(at)), "swiglu_ffn_fwd")
    return out, h13


def swiglu_ffn_bwd(dy: torch.Tensor, x: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, h13: torch.Tensor,
                   flags: int = BWD_DGRAD | BWD_WGRAD, dw_dtype: torch.dtype = torch.float32,
                   workspace: Optional[torch.Tensor] = None, dw13: Optional[torch.Tensor] = None,
                   dw2: Optional[torch.Tensor] = None):
    """Backward of swiglu_ffn_fwd from its saved h13 (the gradient of add is dy). Returns (dx bf16 [M, H]
    or None, dw13 [2F, H] and dw2 [H, F] of dw_dtype or None), as flags asks."""
    _need(dy.dtype == torch.bfloat16 and dy.dim() == 2, "dy must be bf16 [M, H]")
    M, H = dy.shape
    F = _ffn_weights(w13, w2, H)
    _tensor(x, (M, H), torch.bfloat16, "x")
    _tensor(h13, (M, 2 * F), torch.bfloat16, "h13")
    _need(dw_dtype in (torch.bfloat16, torch.float32), "dw_dtype must be bf16 or fp32")
    wgrad = bool(flags & BWD_WGRAD)
    _need(wgrad or (dw13 is None and dw2 is None), "dw13 and dw2 need BWD_WGRAD")
    if dw13 is not None:
        _tensor(dw13, (2 * F, H), dw_dtype, "dw13")
    if dw2 is not None:
        _tensor(dw2, (H, F), dw_dtype, "dw2")
    at = _device_of(dy, "dy")
    dev = dy.device
    workspace = _workspace(workspace, _lib.swiglu_ffn_bwd_workspace_size(M, H, F), dev)
    dx = torch.empty_like(x) if flags & BWD_DGRAD else None
    if wgrad:
        dw13 = torch.empty((2 * F, H), dtype=dw_dtype, device=dev) if dw13 is None else dw13
        dw2 = torch.empty((H, F), dtype=dw_dtype, device=dev) if dw2 is None else dw2
    _check(_lib.swiglu_ffn_bwd(
        _device_ptr(dy, at, "dy"), _device_ptr(x, at, "x"), _device_ptr(w13, at, "w13"), _device_ptr(w2, at, "w2"),
        _device_ptr(h13, at, "h13"), M, H, F, flags, _device_ptr(dx, at, "dx"), _device_ptr(dw13, at, "dw13"),
        _device_ptr(dw2, at, "dw2"), DTYPE_F32 if dw_dtype == torch.float32 else DTYPE_BF16,
        _device_ptr(workspace, at, "workspace"), workspace.numel(), _raw_stream(at)), "swiglu_ffn_bwd")
    return dx, dw13, dw2


# ---- the expert layer on unquantized activations --------------------------------------------

def _group_args(w: torch.Tensor, offsets: torch.Tensor, M: int, N: int, gather, what: str, src_rows: Optional[int]):
    """(G, K) of bf16 weights [G*N, K]."""
    _need(offsets is not None and offsets.dtype == torch.int64 and offsets.dim() == 1 and offsets.numel() >= 2,
          "offsets must be int64 [G+1]")
    G = offsets.numel() - 1
    if w.dtype != torch.bfloat16 or w.dim() != 2 or w.shape[0] != G * N:
        raise PmnError(f"w must be bf16 [G*N, K] with {G * N} rows")
    _index(gather, M, torch.int32, "gather")
    if src_rows is None:   # no rows that gather would name
        _debug_indices(what, offsets, M)
    else:
        _debug_indices(what, offsets, M, gather, src_rows)
    return G, w.shape[1]


def moe_grouped_gemm_fwd_bf16(x: torch.Tensor, w: torch.Tensor, offsets: torch.Tensor, M: int, N: int,
                              epilogue: int = EPI_BF16, gather: Optional[torch.Tensor] = None, save_h13: bool = False,
                              out: Optional[torch.Tensor] = None, out_aux: Optional[torch.Tensor] = None):
    """Grouped product of bf16 x [rows, K] with bf16 w [G*N, K]: Y [M, N] (EPI_F32, EPI_BF16), or with
    EPI_SWIGLU (silu(h1) * h3 [M, N/2], h1 | h3 [M, N] or None), as moe_grouped_gemm_fwd returns them."""
    _need(x.dtype == torch.bfloat16 and x.dim() == 2, "x must be bf16 [rows, K]")
    _need(epilogue in (EPI_F32, EPI_BF16, EPI_SWIGLU), "epilogue must be EPI_F32, EPI_BF16 or EPI_SWIGLU")
    G, K = _group_args(w, offsets, M, N, gather, "moe_grouped_gemm_fwd_bf16", x.shape[0])
    if x.shape[1] != K:
        raise PmnError(f"x must have {K} columns")
    at = _device_of(w, "w")
    dev = w.device
    swiglu = epilogue == EPI_SWIGLU
    if out is None:
        out = torch.empty((M, N // 2 if swiglu else N), dtype=torch.float32 if epilogue == EPI_F32 else torch.bfloat16,
                          device=dev)
    if swiglu and save_h13 and out_aux is None:
        out_aux = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    _epilogue_outputs(epilogue, M, N, out, None, out_aux)
    _check(_lib.moe_grouped_gemm_fwd_bf16(
        _device_ptr(x, at, "x"), x.shape[0], _device_ptr(gather, at, "gather"), _device_ptr(w, at, "w"),
        _device_ptr(offsets, at, "offsets"), G, M, N, K, epilogue, _device_ptr(out, at, "out"),
        _device_ptr(out_aux, at, "out_aux") if swiglu else None, _raw_stream(at)), "moe_grouped_gemm_fwd_bf16")
    return (out, out_aux) if swiglu else out


def moe_grouped_gemm_bwd_bf16_workspace_size(M: int, G: int, N: int, K: int, flags: int, from_h13: bool) -> int:
    return _lib.moe_grouped_gemm_bwd_bf16_workspace_size(M, G, N, K, flags, int(from_h13))


def moe_grouped_gemm_bwd_bf16(dy: torch.Tensor, x: Optional[torch.Tensor], w: torch.Tensor, offsets: torch.Tensor,
                              M: int, N: int, flags: int = BWD_DGRAD | BWD_WGRAD,
                              gather: Optional[torch.Tensor] = None, h13: Optional[torch.Tensor] = None,
                              da_dtype: torch.dtype = torch.bfloat16, db_dtype: torch.dtype = torch.float32,
                              workspace: Optional[torch.Tensor] = None, da: Optional[torch.Tensor] = None,
                              db: Optional[torch.Tensor] = None):
    """Backward of moe_grouped_gemm_fwd_bf16. Returns (da [M, K] or None, db [G*N, K] or None), as flags asks.
    h13 [M, 2K]: the gradient goes on through the SwiGLU that made the product's input, and da is dh13
    [M, 2K]; x may then be None (its values are taken from h13)."""
    _tensor(dy, (M, N), torch.bfloat16, "dy")
    dgrad, wgrad = bool(flags & BWD_DGRAD), bool(flags & BWD_WGRAD)
    for name, dt in (("da_dtype", da_dtype), ("db_dtype", db_dtype)):
        if dt not in (torch.bfloat16, torch.float32):
            raise PmnError(f"{name} must be bf16 or fp32")
    _need(dgrad or da is None, "da needs BWD_DGRAD")
    _need(wgrad or db is None, "db needs BWD_WGRAD")
    _need(x is not None or not wgrad or h13 is not None, "the weight gradient needs x or h13")
    G, K = _group_args(w, offsets, M, N, gather, "moe_grouped_gemm_bwd_bf16", None if x is None else x.shape[0])
    if x is not None:
        if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != K:
            raise PmnError(f"x must be bf16 [rows, {K}]")
    if h13 is not None:
        _tensor(h13, (M, 2 * K), torch.bfloat16, "h13")
        _need(gather is None and dgrad and da_dtype == torch.bfloat16, "h13 goes with BWD_DGRAD, a bf16 da and no gather")
    at = _device_of(dy, "dy")
    dev = dy.device
    width = K if h13 is None else 2 * K
    if da is not None:
        _tensor(da, (M, width), da_dtype, "da")
    elif dgrad:
        da = torch.empty((M, width), dtype=da_dtype, device=dev)
    if db is not None:
        _tensor(db, (G * N, K), db_dtype, "db")
    elif wgrad:
        db = torch.empty((G * N, K), dtype=db_dtype, device=dev)
    need = _lib.moe_grouped_gemm_bwd_bf16_workspace_size(M, G, N, K, flags, x is None and h13 is not None)
    workspace = _workspace(workspace, need, dev) if need or workspace is not None else None
    _check(_lib.moe_grouped_gemm_bwd_bf16(
        _device_ptr(dy, at, "dy"), _device_ptr(x, at, "x"), 0 if x is None else x.shape[0],
        _device_ptr(gather, at, "gather"), _device_ptr(w, at, "w"), _device_ptr(offsets, at, "offsets"), G, M, N, K, flags,
        _device_ptr(h13, at, "h13"), _device_ptr(da, at, "da"), DTYPE_F32 if da_dtype == torch.float32 else DTYPE_BF16,
        _device_ptr(db, at, "db"), DTYPE_F32 if db_dtype == torch.float32 else DTYPE_BF16,
        _device_ptr(workspace, at, "workspace"), 0 if workspace is None else workspace.numel(), _raw_stream(at)),
        "moe_grouped_gemm_bwd_bf16")
    return da, db


def moe_gemv_nvfp4_workspace_size(T: int, k: int, N: int, summed: bool) -> int:
    return _lib.moe_gemv_nvfp4_workspace_size(T, k, N, int(summed))


def moe_gemv_nvfp4(x: torch.Tensor, wq: NVFP4, N: int, ids: Optional[torch.Tensor] = None, epilogue: int = EPI_BF16,
                   gates: Optional[torch.Tensor] = None, add: Optional[torch.Tensor] = None,
                   workspace: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """A few tokens' bf16 activations times NVFP4 weights wq [G*N, K]. x [T, K], or [T, k, K] with a row for
    each of a token's experts; ids int32 [T, k] names them (None: G = 1, a dense product). Without gates
    y [T, k, N] (without ids [T, N]) in fp32 or bf16, or with EPI_SWIGLU silu(h1) * h3 [T, k, N/2] in bf16; with
    gates fp32 [T, k] their sum over k (+ add bf16 [T, N]), [T, N]."""
    _need(x.dtype == torch.bfloat16 and x.dim() in (2, 3), "x must be bf16 [T, K] or [T, k, K]")
    _need(epilogue in (EPI_F32, EPI_BF16, EPI_SWIGLU), "epilogue must be EPI_F32, EPI_BF16 or EPI_SWIGLU")
    _nvfp4(wq, "wq")
    T, K = x.shape[0], x.shape[-1]
    if wq.cols != K:
        raise PmnError(f"wq must have {K} columns")
    R = wq.rows
    if N <= 0 or R % N != 0 or R == 0:
        raise PmnError(f"wq must have a multiple of {N} rows")
    G, k = R // N, 1
    if ids is not None:
        if ids.dtype != torch.int32 or ids.dim() != 2 or ids.shape[0] != T:
            raise PmnError(f"ids must be int32 [{T}, k]")
        k = ids.shape[1]
    else:
        if G != 1:
            raise PmnError(f"without ids wq must have {N} rows")
    if x.dim() == 3 and x.shape[1] != k:
        raise PmnError(f"x must have {k} rows a token")
    if gates is not None:
        _tensor(gates, (T, k), torch.float32, "gates")
        _need(epilogue != EPI_SWIGLU, "gates do not go with EPI_SWIGLU")
    if add is not None:
        _need(gates is not None, "add needs gates")
        _tensor(add, (T, N), torch.bfloat16, "add")
    at = _device_of(x, "x")
    dev = x.device
    width = N // 2 if epilogue == EPI_SWIGLU else N
    shape = (T, width) if gates is not None or ids is None else (T, k, width)
    dtype = torch.float32 if epilogue == EPI_F32 else torch.bfloat16
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=dev)
    else:
        _tensor(out, shape, dtype, "out")
    if gates is not None:
        need = _lib.moe_gemv_nvfp4_workspace_size(T, k, N, 1)
        workspace = _workspace(workspace, need, dev) if need or workspace is not None else None
    _check(_lib.moe_gemv_nvfp4(
        _device_ptr(x, at, "x"), int(x.dim() == 3), _device_ptr(wq.codes, at, "wq.codes"),
        _device_ptr(wq.scales, at, "wq.scales"), _device_ptr(wq.outer, at, "wq.outer"), wq.rows_per_outer,
        _device_ptr(ids, at, "ids"), _device_ptr(gates, at, "gates"), _device_ptr(add, at, "add"), T, k, G, N, K, epilogue,
        _device_ptr(out, at, "out"), _device_ptr(workspace, at, "workspace"),
        0 if workspace is None else workspace.numel(), _raw_stream(at)), "moe_gemv_nvfp4")
    return out


def _rows_args(y: torch.Tensor, slot_of: torch.Tensor, gates: Optional[torch.Tensor]):
    """(M, H, T, k) of y [M, H] and slot_of [T, k], or [T*k] as moe_route_topk gives it, beside gates [T, k]."""
    _need(y.dim() == 2, "y must be [M, H]")
    shape = slot_of.shape
    if slot_of.dim() == 1 and gates is not None and gates.dim() == 2:
        shape = gates.shape
    _need(slot_of.dtype == torch.int32 and len(shape) == 2 and slot_of.numel() == shape[0] * shape[1],
          "slot_of must be int32 [T, k] (or [T*k] with gates)")
    if gates is not None:
        _tensor(gates, shape, torch.float32, "gates")
    return (*y.shape, *shape)


def moe_combine_rows_fwd(y: torch.Tensor, slot_of: torch.Tensor, gates: Optional[torch.Tensor] = None,
                         add: Optional[torch.Tensor] = None, out_dtype: torch.dtype = torch.bfloat16,
                         out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Row t = sum_j gates[t, j] * y[slot_of[t, j]] (+ add[t]): y bf16 or fp32 [M, H], gates None: ones, add
    bf16 [T, H] (it may be out). A slot outside [0, M) adds nothing."""
    ycode = _dtype_code(y, "y")
    M, H, T, k = _rows_args(y, slot_of, gates)
    if add is not None:
        _tensor(add, (T, H), torch.bfloat16, "add")
    _need(out_dtype in (torch.bfloat16, torch.float32), "out_dtype must be bf16 or fp32")
    at = _device_of(slot_of, "slot_of")
    if out is None:
        out = torch.empty((T, H), dtype=out_dtype, device=y.device)
    else:
        _tensor(out, (T, H), out_dtype, "out")
    _check(_lib.moe_combine_rows_fwd(
        _device_ptr(y, at, "y"), ycode, M, H, _device_ptr(slot_of, at, "slot_of"), _device_ptr(gates, at, "gates"),
        _device_ptr(add, at, "add"), T, k, _device_ptr(out, at, "out"),
        DTYPE_F32 if out_dtype == torch.float32 else DTYPE_BF16, _raw_stream(at)), "moe_combine_rows_fwd")
    return out


# A new dy's rows that no pair names: found among the pairs (0.08 us for 1024 of them) from this many bytes a row and in
# all, else all rows get zeros beforehand. (Zeros / found, with the gradient, us: 16384 tokens of 8 rows of 4096 bf16
# 622 / 480, of 512 68 / 62, of 256 38 / 40; 501 of 4 rows of 4096 14.5 / 16.)
_FOUND_ROW_BYTES, _FOUND_BYTES = 1024, 32 << 20


def moe_combine_rows_bwd(dout: torch.Tensor, y: torch.Tensor, slot_of: torch.Tensor,
                         gates: Optional[torch.Tensor] = None, want_dy: bool = True, want_dgates: bool = True,
                         dy: Optional[torch.Tensor] = None):
    """Gradients of moe_combine_rows_fwd from dout [T, H] (bf16 or fp32): (dy [M, H] of y's type or None, dgates
    fp32 [T, k] or None). No slot may be named twice. Rows of a given dy that no pair names are left as they
    are; without one they are zeros. (CHECK_INDICES refuses a slot that is named twice, and of M == T * k rows of a
    new dy one that no pair names, as a lost slot.)"""
    ycode, dcode = _dtype_code(y, "y"), _dtype_code(dout, "dout")
    M, H, T, k = _rows_args(y, slot_of, gates)
    _tensor(dout, (T, H), dout.dtype, "dout")
    _need(want_dy or dy is None, "dy needs want_dy")
    _need(want_dy or want_dgates, "want_dy or want_dgates must be set")
    if dy is not None:
        _tensor(dy, (M, H), y.dtype, "dy")
    at = _device_of(slot_of, "slot_of")
    if CHECK_INDICES and want_dy:
        inside = slot_of[(slot_of >= 0) & (slot_of < M)]
        _need(inside.unique().numel() == inside.numel(), "moe_combine_rows_bwd: a slot is named twice")
        _need(dy is not None or M != T * k or inside.numel() == M, "moe_combine_rows_bwd: a row of the new dy is no pair's")
    rest = False
    if want_dy and dy is None:
        rest = H * y.element_size() >= _FOUND_ROW_BYTES and M * H * y.element_size() >= _FOUND_BYTES
        dy = torch.empty_like(y) if rest else torch.zeros_like(y)
    dgates = torch.empty((T, k), dtype=torch.float32, device=y.device) if want_dgates else None
    _check(_lib.moe_combine_rows_bwd(
        _device_ptr(dout, at, "dout"), dcode, _device_ptr(y, at, "y"), ycode, M, H, _device_ptr(slot_of, at, "slot_of"),
        _device_ptr(gates, at, "gates"), T, k, _device_ptr(dy, at, "dy"), _device_ptr(dgates, at, "dgates"),
        _raw_stream(at)), "moe_combine_rows_bwd")
    if rest:
        moe_rows_zero_unnamed(dy, slot_of.view(T, k))
    return dy, dgates


def moe_rows_zero_unnamed(x: torch.Tensor, slot_of: torch.Tensor) -> torch.Tensor:
    """Zeros to the rows of x [M, H] (bf16 or fp32) that no slot of slot_of int32 [T, k] names, in place; returns x."""
    xcode = _dtype_code(x, "x")
    M, H, T, k = _rows_args(x, slot_of, None)
    at = _device_of(slot_of, "slot_of")
    _check(_lib.moe_rows_zero_unnamed(_device_ptr(x, at, "x"), xcode, M, H, _device_ptr(slot_of, at, "slot_of"), T, k,
                                      _raw_stream(at)), "moe_rows_zero_unnamed")
    return x


@dataclass
class AdamWTensor:
    """One tensor of an AdamWPlan: param fp32 and grad (bf16 or fp32) of n values, copy (optional) its
    bf16 copy; moments m and v fp32, or u8 with m_e8m0 and v_e8m0 u8 [ceil(n / 32)]. Updated in place."""
    param: torch.Tensor
    grad: torch.Tensor
    m: torch.Tensor
    v: torch.Tensor
    copy: Optional[torch.Tensor] = None
    m_e8m0: Optional[torch.Tensor] = None
    v_e8m0: Optional[torch.Tensor] = None
    weight_decay: float = 0.0

    _replaced = 0   # fields set anew, over all instances: plans look at theirs again where it has grown

    def __setattr__(self, name, value):
        if name in self.__dict__:
            AdamWTensor._replaced += 1
        object.__setattr__(self, name, value)

    @staticmethod
    def new(param: torch.Tensor, grad: torch.Tensor, state_bits: int = 32, copy: Optional[torch.Tensor] = None,
            weight_decay: float = 0.0) -> "AdamWTensor":
        """With zero moments."""
        _need(state_bits in (8, 32), "state_bits must be 8 or 32")
        n, dev = param.numel(), param.device
        dt = torch.uint8 if state_bits == 8 else torch.float32
        e8 = [torch.zeros(((n + 31) // 32,), dtype=torch.uint8, device=dev) if state_bits == 8 else None for _ in "mv"]
        return AdamWTensor(param, grad, torch.zeros((n,), dtype=dt, device=dev),
                           torch.zeros((n,), dtype=dt, device=dev), copy, e8[0], e8[1], weight_decay)


class _AdamWEntry(C.Structure):
    _fields_ = [("param", P), ("grad", P), ("copy", P), ("m", P), ("v", P), ("m_e8m0", P), ("v_e8m0", P),
                ("n", I64), ("weight_decay", F32), ("grad_dtype", I32)]


class AdamWPlan:
    """A list of tensors to be updated together, as a table on their device, built once and kept for
    every step. All of one state width; no tensor twice. The table holds addresses: the plan keeps the
    tensors that it was built of, gradients are written into theirs, and a field of an AdamWTensor that is
    set anew needs another plan (steps of this one are refused)."""

    def __init__(self, tensors: List[AdamWTensor]):
        self.tensors = list(tensors)
        self._built_of = [(t, [(f.name, getattr(t, f.name)) for f in fields(t)]) for t in self.tensors]
        self._replaced = AdamWTensor._replaced
        _need(len(self.tensors) > 0, "an AdamWPlan needs at least one tensor")
        dev = self.tensors[0].param.device
        self.state_bits = 8 if self.tensors[0].m.dtype == torch.uint8 else 32
        sdt = torch.uint8 if self.state_bits == 8 else torch.float32
        at = dev.index if dev.type == "cuda" else -1
        entries = (_AdamWEntry * len(self.tensors))()
        spans = []
        for i, t in enumerate(self.tensors):
            n = t.param.numel()
            nb = (n + 31) // 32
            ptr = {}
            for what, dt, k in (("param", torch.float32, n), ("grad", None, n), ("m", sdt, n), ("v", sdt, n),
                                ("copy", torch.bfloat16, n), ("m_e8m0", torch.uint8, nb), ("v_e8m0", torch.uint8, nb)):
                v = getattr(t, what)
                if what in ("m_e8m0", "v_e8m0") and self.state_bits == 32:
                    _need(v is None, f"tensors[{i}].{what} belongs to states in 8 bits")
                    continue
                if what == "copy" and v is None:
                    continue
                if what == "grad":
                    gcode = _dtype_code(v, f"tensors[{i}].grad")
                    dt = v.dtype
                if v is None or v.dtype != dt or v.numel() != k:
                    raise PmnError(f"tensors[{i}].{what} must hold {k} values of {dt}")
                if v.get_device() != at:
                    raise PmnError(f"tensors[{i}].{what} must be on {dev}")
                if not v.is_contiguous():
                    raise PmnError(f"tensors[{i}].{what} must be contiguous")
                p = ptr[what] = v.data_ptr()
                if k:
                    spans.append((p, p + k * v.element_size(), what != "grad", i, what))
            entries[i] = _AdamWEntry(ptr["param"], ptr["grad"], ptr.get("copy"), ptr["m"], ptr["v"], ptr.get("m_e8m0"),
                                     ptr.get("v_e8m0"), n, t.weight_decay, gcode)
        # buffers that are written overlap no other; gradients may share memory among themselves
        spans.sort()
        end, owner, wend, wowner = 0, None, 0, None
        for lo, hi, written, i, what in spans:
            if lo < (end if written else wend):
                j, other = owner if written else wowner
                raise PmnError(f"tensors[{i}].{what} overlaps tensors[{j}].{other}")
            if hi > end:
                end, owner = hi, (i, what)
            if written and hi > wend:
                wend, wowner = hi, (i, what)
        _need(at >= 0, "the tensors must be on the GPU")
        size = _lib.adamw_table_size(entries, len(entries))
        host = torch.empty(((size + 7) // 8,), dtype=torch.int64)
        chunks = C.c_int64(0)
        _check(_lib.adamw_table_build(entries, len(entries), self.state_bits, host.data_ptr(), host.numel() * 8,
                                      C.byref(chunks)), "adamw_table_build")
        self.chunks = chunks.value
        self.table = host.to(dev)
        self._stream = _raw_stream(at)   # whose memory the table is

    def _check_tensors(self):
        for i, (t, built_of) in enumerate(self._built_of):
            for what, v in built_of:
                now = getattr(t, what)
                _need(now is v or (what == "weight_decay" and now == v),
                      f"tensors[{i}].{what} is not what the plan was built of")
        self._replaced = AdamWTensor._replaced


def adamw_step(plan: AdamWPlan, lr: Union[float, torch.Tensor], step: Union[int, torch.Tensor], beta1: float = 0.9,
               beta2: float = 0.95, eps: float = 1e-8, grad_scale: Optional[torch.Tensor] = None, seed: int = 0,
               rng_stream: int = 0) -> None:
    """One AdamW step over the plan's tensors, in place. step counts from 1. lr (fp32), step (int64) and
    grad_scale (fp32) may be device tensors of one value, read when the step runs: a captured graph
    that is replayed needs the step there, and changes it between its replays."""
    dev = {}
    for name, v, dt in (("lr", lr, torch.float32), ("step", step, torch.int64), ("grad_scale", grad_scale, torch.float32)):
        if isinstance(v, torch.Tensor):
            _need(v.dtype == dt and v.numel() == 1, f"{name} must be one value of {dt}")
            dev[name] = v
    _need(grad_scale is None or "grad_scale" in dev, "grad_scale must be a device tensor")
    if plan._replaced != AdamWTensor._replaced:
        plan._check_tensors()
    at = _device_of(plan.table, "the plan")
    stream = _raw_stream(at)
    if stream != plan._stream:
        # a plan dropped while this step is still to run must not give its table's memory away
        plan.table.record_stream(torch.cuda.current_stream())
    _check(_lib.adamw_step(
        _device_ptr(plan.table, at, "the plan"), plan.chunks, plan.state_bits, 0.0 if "lr" in dev else lr, beta1, beta2,
        eps, 1 if "step" in dev else step, _device_ptr(dev.get("lr"), at, "lr"), _device_ptr(dev.get("step"), at, "step"),
        _device_ptr(dev.get("grad_scale"), at, "grad_scale"), seed, rng_stream & 0xFFFFFFFF, stream), "adamw_step")


# ---- measurement kernels of include/pmn_probe.h ---------------------------------------------

PROBE_MFMA_KINDS = {0: "v_mfma_f32_32x32x16_f16", 1: "v_mfma_f32_16x16x32_f16",
                    2: "v_mfma_scale_f32_32x32x64_f8f6f4 (E4M3)", 3: "v_mfma_scale_f32_16x16x128_f8f6f4 (E4M3)",
                    4: "v_mfma_scale_f32_32x32x64_f8f6f4 (E2M1)",
                    5: "v_mfma_f32_32x32x16_f16 + FP4 dequantization", 6: "v_mfma_f32_16x16x32_f16 + FP4 dequantization"}


def probe_stream(src: Optional[torch.Tensor], dst: Optional[torch.Tensor], units: int, read_kb: int, write_kb: int,
                 grid: int = 8192, hints: int = 3):
    """Stream `units` units of read_kb KB read from src and write_kb KB written to dst (hints: bit 0
    nontemporal loads, bit 1 nontemporal stores)."""
    if read_kb:
        _need(src is not None and src.numel() * src.element_size() >= units * read_kb * 1024, "src too small")
    if write_kb:
        _need(dst is not None and dst.numel() * dst.element_size() >= units * write_kb * 1024, "dst too small")
    _check(_lib.pmn_probe_stream(_ptr(src) if read_kb else None, _ptr(dst) if write_kb else None, units, read_kb,
                                 write_kb, grid, hints, _stream()), "pmn_probe_stream")


def probe_mfma(kind: int, waves_per_simd: int, workgroups: int, iters: int, sink: torch.Tensor) -> float:
    """Launch the MFMA throughput probe; returns the launch's FLOPs (time it on the current stream)."""
    n = _lib.pmn_probe_mfma_sink_floats(waves_per_simd, workgroups)
    _need(sink.dtype == torch.float32 and sink.numel() >= n, f"sink must hold {n} floats")
    fl = C.c_double(0.0)
    _check(_lib.pmn_probe_mfma(kind, waves_per_simd, workgroups, iters, _ptr(sink), C.byref(fl), _stream()),
           "pmn_probe_mfma")
    return fl.value


def probe_recip_check(first_bits: int, last_bits: int) -> int:
    """Number of fp32 values with bit patterns in [first_bits, last_bits] whose division-free
    reciprocal (the activation quantizer's) differs from the IEEE quotient 1/d."""
    count = torch.zeros(1, dtype=torch.int64, device=torch.device("cuda", torch.cuda.current_device()))
    _check(_lib.pmn_probe_recip_check(first_bits, last_bits, _ptr(count), _stream()), "pmn_probe_recip_check")
    return int(count.item())
