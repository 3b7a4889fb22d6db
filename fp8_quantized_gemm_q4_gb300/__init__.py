"""Block-scaled FP4 / FP8 GEMM for GB300 (sm_103a): Python binding.

Thin ctypes binding of the C ABI in ``include/bsgemm.h``: it marshals torch
tensors (device memory, the current stream) into the library's entry points
and allocates outputs with torch.  Every step of the computation runs in the
library's CUDA kernels; there is no fallback.  If ``libbsgemm.so`` has not
been built, ``load()`` raises.

    Y = (Q(X) Q(W)^T) (.) scale + L(X) + b
    ("Warp-specialised W4A4 kernel on the newest GPU architecture", section 1)
"""
from __future__ import annotations

import ctypes
import os
import struct
import threading
from typing import NamedTuple

import torch

from ._build import LIB as _LIB_PATH

__all__ = [
    "load", "sf_bytes", "sf_offset", "q4_quantize", "tensor_amax", "q4_quantize_two_level", "fp4_gather_rows", "fp8_gather_rows", "q8_quantize", "gemm_fp4", "gemm_fp8", "gemm_fp8_multi", "gemm_fp4_multi",
    "grouped_gemm_fp4", "grouped_gemm_fp4_swiglu_q4", "grouped_gemm_fp8", "moe_router_topk", "moe_dispatch", "moe_finalize", "moe_combine", "moe_rows_bound", "kv_plan", "kv_release", "kv_append", "kv_positions", "kv_append_rotary", "kv_gather", "kv_attention", "kv_attention_workspace", "matvec_fp4", "lora_add", "rotary_angles", "KVCache", "KVCacheFP4", "device_status",
    "clear_device_status", "BSError", "EPI_STORE", "EPI_SWIGLU", "EPI_COMBINE", "EPI_ROWS", "kernel_options",
    "current_kernel_options", "FP4_ONE_CTA", "FP4_PAIR",
]

BS_OK, BS_ERR_INVALID, BS_ERR_ALIGN, BS_ERR_UNSUPPORTED, BS_ERR_CUDA, BS_ERR_TIMEOUT, BS_ERR_OFFSETS, BS_ERR_PAGES = range(8)
DTYPE_F32, DTYPE_BF16 = 0, 1
FMT_FP4, FMT_FP8 = 0, 1
EPI_STORE, EPI_SWIGLU, EPI_COMBINE, EPI_ROWS = 0, 1, 2, 3
Q8_TOKEN, Q8_BLOCK, Q8_ROW = 1, 128, 3


class BSError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(f"bsgemm status {status}: {msg}")
        self.status = status


class GemmArgs(ctypes.Structure):
    _fields_ = [
        ("fmt", ctypes.c_int), ("a", ctypes.c_void_p), ("sfa", ctypes.c_void_p), ("b", ctypes.c_void_p),
        ("sfb", ctypes.c_void_p), ("M", ctypes.c_int64), ("N", ctypes.c_int64), ("K", ctypes.c_int64),
        ("alpha", ctypes.c_float), ("col_scale", ctypes.c_void_p), ("lora_t", ctypes.c_void_p),
        ("lora_b_t", ctypes.c_void_p), ("r", ctypes.c_int), ("bias", ctypes.c_void_p), ("out", ctypes.c_void_p),
        ("out_dtype", ctypes.c_int), ("ldo", ctypes.c_int64), ("num_sms", ctypes.c_int),
        ("n_chunk_blocks", ctypes.c_int), ("fp4_kernel", ctypes.c_int), ("fp4_stage_k", ctypes.c_int),
        ("fp4_small_experts", ctypes.c_int), ("fp4_half_tail", ctypes.c_int), ("fp8_stream_k", ctypes.c_int),
        ("fp8_scaling", ctypes.c_int), ("wait_timeout_us", ctypes.c_int), ("weights_ready", ctypes.c_int), ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t), ("a_tensor_scale", ctypes.c_void_p), ("b_tensor_scale", ctypes.c_void_p),
        ("fp4_decode", ctypes.c_int),
    ]


# bs_kv_append_args and bs_kv_attention_args, packed in native layout: building
# a ctypes.Structure of as many fields takes three times as long.
_KV_PLAN_ARGS = struct.Struct("PPiPqiPPiiqPPPP")
_FP4_MATVEC_ARGS = struct.Struct("PqiPPqqfPPPiq")
_KV_APPEND_ARGS = struct.Struct("PPiqiiqqqqPPPPPqi4x")
_KV_ATTENTION_ARGS = struct.Struct("PqqPqqPPPPPqiPqiPPiqiiiifiPN")
_KV_APPEND_ROTARY_ARGS = struct.Struct("PqqPqqPPiiiiqqqqqPPPqiiiiPPPPq")
_KV_GATHER_ARGS = struct.Struct("PqiiPPqqqqiiPPPPq")
_LORA_ARGS = struct.Struct("PqPPPPPPqPqiiqqqii")


# Per-call kernel choices of bs_gemm_args (0 = the library's default), see
# include/bsgemm.h.  Every GEMM call of this binding fills them from the
# options active on the calling thread: the defaults, or those of an enclosing
# ``with kernel_options(...)`` block.
_CHOICES = ("fp4_kernel", "fp4_stage_k", "fp4_small_experts", "fp4_half_tail", "fp4_decode", "fp8_stream_k",
            "wait_timeout_us")
FP4_ONE_CTA, FP4_PAIR = 1, 2
_tls = threading.local()


def current_kernel_options() -> dict:
    return dict(getattr(_tls, "opts", {}))


class kernel_options:
    """Context manager: GEMM calls made on this thread inside the block pass
    these kernel choices in their bs_gemm_args (unnamed fields keep the value
    of any enclosing block, else 0 = default)."""

    def __init__(self, **choices):
        bad = set(choices) - set(_CHOICES)
        if bad:
            raise TypeError(f"unknown kernel choices {sorted(bad)}")
        self.choices = {k: int(v) for k, v in choices.items()}

    def __enter__(self):
        self.saved = getattr(_tls, "opts", {})
        _tls.opts = {**self.saved, **self.choices}
        return self

    def __exit__(self, *exc):
        _tls.opts = self.saved
        return False


_lib = None
_lock = threading.Lock()


def load(path: str | None = None):
    """Load libbsgemm.so (built by ``__graft_entry__.build()``); raise if absent."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or os.environ.get("BSGEMM_LIB") or _LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(f"CUDA library not built: {p} is missing (run __graft_entry__.build())")
        lib = ctypes.CDLL(p)
        P, I64, I, F, SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
        lib.bs_sf_bytes.restype = SZ
        lib.bs_sf_bytes.argtypes = [I64, I64]
        lib.bs_sf_offset.restype = I64
        lib.bs_sf_offset.argtypes = [I64, I64, I64]
        lib.q4_quantize.restype = I
        lib.q4_quantize.argtypes = [P, I, I64, I64, I64, P, P, P, P, I, P, P]
        lib.bs_tensor_amax.restype = I
        lib.bs_tensor_amax.argtypes = [P, I, I64, I64, I64, P, P]
        lib.q4_quantize_two_level.restype = I
        lib.q4_quantize_two_level.argtypes = [P, I, I64, I64, I64, P, P, P, P, P]
        lib.bs_fp4_gather_rows.restype = I
        lib.bs_fp4_gather_rows.argtypes = [P, P, I64, I64, P, I64, P, P, P]
        lib.bs_fp8_gather_rows.restype = I
        lib.bs_fp8_gather_rows.argtypes = [P, P, I64, I64, P, I64, P, P, P]
        lib.q8_quantize.restype = I
        lib.q8_quantize.argtypes = [P, I, I64, I64, I64, I, P, P, P]
        lib.bs_gemm.restype = I
        lib.bs_gemm.argtypes = [ctypes.POINTER(GemmArgs), P]
        lib.bs_gemm_workspace_bytes.restype = SZ
        lib.bs_gemm_workspace_bytes.argtypes = [ctypes.POINTER(GemmArgs)]
        lib.bs_gemm_multi.restype = I
        lib.bs_gemm_multi.argtypes = [ctypes.POINTER(GemmArgs), I, P, P, P, P]
        lib.bs_gemm_multi_workspace_bytes.restype = SZ
        lib.bs_gemm_multi_workspace_bytes.argtypes = [ctypes.POINTER(GemmArgs), I]
        lib.bs_grouped_gemm.restype = I
        lib.bs_grouped_gemm.argtypes = [ctypes.POINTER(GemmArgs), I, P, P, I, P, P, P, I64, P]
        lib.bs_moe_rows_bound.restype = I64
        lib.bs_grouped_gemm_swiglu_q4.restype = I
        lib.bs_grouped_gemm_swiglu_q4.argtypes = [ctypes.POINTER(GemmArgs), I, P, P, P, P, P]
        lib.bs_moe_rows_bound.argtypes = [I64, I, I]
        lib.bs_moe_dispatch_workspace_bytes.restype = SZ
        lib.bs_moe_dispatch_workspace_bytes.argtypes = [I64, I, I]
        lib.bs_moe_router_topk.restype = I
        lib.bs_moe_router_topk.argtypes = [P, I64, I, I, P, P, P]
        lib.bs_moe_dispatch.restype = I
        lib.bs_moe_dispatch.argtypes = [P, P, I64, I, I, P, P, P, P, P, P, SZ, P]
        lib.bs_moe_dispatch_noalloc.restype = I
        lib.bs_moe_dispatch_noalloc.argtypes = [P, P, I64, I, I, P, P, P, P, P, P]
        lib.bs_moe_finalize.restype = I
        lib.bs_moe_finalize.argtypes = [P, P, I64, P]
        lib.bs_moe_combine.restype = I
        lib.bs_moe_combine.argtypes = [P, I64, P, I64, I64, I, I64, P, P, I64, P]
        lib.bs_kv_plan.restype = I
        lib.bs_kv_plan.argtypes = [ctypes.c_char_p, P]   # the packed structs
        lib.bs_kv_release.restype = I
        lib.bs_kv_release.argtypes = [P, P, I, P, I64, I, P, P, I, I, P]
        lib.bs_kv_append.restype = I
        lib.bs_kv_append.argtypes = [ctypes.c_char_p, P]
        lib.bs_kv_attention_workspace_bytes.restype = SZ
        lib.bs_kv_attention_workspace_bytes.argtypes = [ctypes.c_char_p]
        lib.bs_kv_attention.restype = I
        lib.bs_kv_attention.argtypes = [ctypes.c_char_p, P]
        lib.bs_kv_positions.restype = I
        lib.bs_kv_positions.argtypes = [P, P, I, I64, P, P]
        lib.bs_kv_attention_fp4.restype = I
        lib.bs_kv_attention_fp4.argtypes = [ctypes.c_char_p, P, P, P]
        lib.bs_kv_append_rotary.restype = I
        lib.bs_kv_append_rotary.argtypes = [ctypes.c_char_p, P]
        lib.bs_kv_gather.restype = I
        lib.bs_kv_gather.argtypes = [ctypes.c_char_p, P]
        lib.bs_lora_add.restype = I
        lib.bs_lora_add.argtypes = [ctypes.c_char_p, P]
        lib.bs_fp4_matvec.restype = I
        lib.bs_fp4_matvec.argtypes = [ctypes.c_char_p, P]
        lib.bs_get_device_status.restype = I
        lib.bs_get_device_status.argtypes = [ctypes.POINTER(I)]
        lib.bs_clear_device_status.restype = I
        lib.bs_clear_device_status.argtypes = []
        lib.bs_status_string.restype = ctypes.c_char_p
        lib.bs_status_string.argtypes = [I]
        lib.bs_last_error.restype = ctypes.c_char_p
        lib.bs_last_error.argtypes = []
        _lib = lib
        return lib


def _check(status: int):
    if status:
        lib = load()
        raise BSError(status, lib.bs_last_error().decode(errors="replace") or
                      lib.bs_status_string(status).decode())


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)   # neither name is public
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _stream(stream=None):
    """The cudaStream_t handle of ``stream``, or of the current stream of the
    current device.  The raw handle is asked for directly where torch has it:
    building the torch.cuda.Stream object around it takes 2.9 us of a 3.1 us launch."""
    if stream is not None:
        return stream.cuda_stream
    if _raw_stream is None:
        return torch.cuda.current_stream().cuda_stream
    return _raw_stream(_device())


def _empty(shape, dtype, device, stream):
    """A new tensor of the stream that the call goes to: memory of another stream's may still be in use there."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _dt(t: torch.Tensor) -> int:
    if t.dtype == torch.float32:
        return DTYPE_F32
    if t.dtype == torch.bfloat16:
        return DTYPE_BF16
    raise TypeError(f"unsupported dtype {t.dtype}")


def sf_bytes(rows: int, K: int) -> int:
    """Bytes of the MMA-layout scale tensor of an [rows, K] FP4 operand."""
    return int(load().bs_sf_bytes(rows, K))


def sf_offset(row: int, group: int, K: int) -> int:
    return int(load().bs_sf_offset(row, group, K))


def q4_quantize(x: torch.Tensor, gather: torch.Tensor | None = None, rows: int | None = None,
                lora_a_t: torch.Tensor | None = None, out=None, stream=None):
    """FP4 E2M1 group-16 quantization.  Returns (codes [M, K/2] u8, sf u8 [sf_bytes],
    lora_t bf16 [M, 64] or None).  With ``gather``, output row i is x[gather[i]]
    (negative: zero row) and M = len(gather) (or ``rows``)."""
    assert x.is_cuda and x.dim() == 2 and x.stride(1) == 1
    M = int(rows if rows is not None else (gather.numel() if gather is not None else x.shape[0]))
    K = x.shape[1]
    if out is None:
        codes = _empty((M, K // 2), torch.uint8, x.device, stream)
        sf = _empty(sf_bytes(M, K), torch.uint8, x.device, stream)
        lt = _empty((M, 64), torch.bfloat16, x.device, stream) if lora_a_t is not None else None
    else:
        codes, sf, lt = out
    _check(load().q4_quantize(_ptr(x), _dt(x), M, K, x.stride(0), _ptr(gather), _ptr(codes), _ptr(sf),
                              _ptr(lora_a_t), 32 if lora_a_t is not None else 0, _ptr(lt), _stream(stream)))
    return codes, sf, lt


def tensor_amax(x: torch.Tensor, out=None, stream=None):
    """max |x| over the whole [M, K] tensor, as a device fp32 tensor [1]."""
    amax = out if out is not None else _empty(1, torch.float32, x.device, stream)
    _check(load().bs_tensor_amax(_ptr(x), _dt(x), x.shape[0], x.shape[1], x.stride(0), _ptr(amax), _stream(stream)))
    return amax


def q4_quantize_two_level(x: torch.Tensor, amax=None, out=None, stream=None):
    """Two-level FP4: power-of-two tensor scale above the e4m3 group scales.
    Returns (codes [M, K/2], sf, tensor_scale device fp32 [1]); ``amax``
    (device fp32 [1]) defaults to tensor_amax(x)."""
    assert x.is_cuda and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    if amax is None:
        amax = tensor_amax(x, stream=stream)
    if out is None:
        out = (_empty((M, K // 2), torch.uint8, x.device, stream),
               _empty(sf_bytes(M, K), torch.uint8, x.device, stream),
               _empty(1, torch.float32, x.device, stream))
    codes, sf, ts = out
    _check(load().q4_quantize_two_level(_ptr(x), _dt(x), M, K, x.stride(0), _ptr(amax), _ptr(codes), _ptr(sf),
                                        _ptr(ts), _stream(stream)))
    return codes, sf, ts


def fp4_gather_rows(codes, sf, K: int, gather, out=None, stream=None):
    """Rows gather[i] of an FP4 matrix (codes + MMA-layout scales); -1 -> zero row."""
    rows_out = gather.numel()
    if out is None:
        out = (_empty((rows_out, K // 2), torch.uint8, codes.device, stream),
               _empty(sf_bytes(rows_out, K), torch.uint8, codes.device, stream))
    _check(load().bs_fp4_gather_rows(_ptr(codes), _ptr(sf), codes.shape[0], K, _ptr(gather), rows_out,
                                     _ptr(out[0]), _ptr(out[1]), _stream(stream)))
    return out


def fp8_gather_rows(codes, scales, gather, out=None, stream=None):
    """Rows gather[i] of an FP8 matrix (codes [rows, K] + TOKEN-mode scales
    [K/128, rows]); -1 -> zero row with zero scales."""
    rows_in, K = codes.shape
    rows_out = gather.numel()
    if out is None:
        out = (_empty((rows_out, K), torch.uint8, codes.device, stream),
               _empty((K // 128, rows_out), torch.float32, codes.device, stream))
    _check(load().bs_fp8_gather_rows(_ptr(codes), _ptr(scales), rows_in, K, _ptr(gather), rows_out,
                                     _ptr(out[0]), _ptr(out[1]), _stream(stream)))
    return out


def q8_quantize(x: torch.Tensor, mode: int = Q8_TOKEN, out=None, stream=None):
    """FP8 e4m3 quantization.  TOKEN mode: scales fp32 [K/128, M]; BLOCK mode:
    scales fp32 [ceil(M/128), K/128]; ROW mode (W8A8): scales fp32 [M]."""
    assert x.is_cuda and x.dim() == 2 and x.stride(1) == 1
    M, K = x.shape
    if out is None:
        codes = _empty((M, K), torch.uint8, x.device, stream)
        shape = {Q8_TOKEN: (K // 128, M), Q8_BLOCK: ((M + 127) // 128, K // 128), Q8_ROW: (M,)}[mode]
        scales = _empty(shape, torch.float32, x.device, stream)
    else:
        codes, scales = out
    _check(load().q8_quantize(_ptr(x), _dt(x), M, K, x.stride(0), mode, _ptr(codes), _ptr(scales),
                              _stream(stream)))
    return codes, scales


def _args(fmt, a, sfa, b, sfb, M, N, K, out, alpha=1.0, col_scale=None, lora_t=None, lora_b_t=None,
          bias=None, num_sms=0):
    g = GemmArgs()
    g.fmt = fmt
    g.a, g.sfa, g.b, g.sfb = a.data_ptr(), sfa.data_ptr(), b.data_ptr(), sfb.data_ptr()
    g.M, g.N, g.K = M, N, K
    g.alpha = alpha
    g.col_scale = None if col_scale is None else col_scale.data_ptr()
    g.lora_t = None if lora_t is None else lora_t.data_ptr()
    g.lora_b_t = None if lora_b_t is None else lora_b_t.data_ptr()
    g.r = 32 if lora_t is not None else 0
    g.bias = None if bias is None else bias.data_ptr()
    if out is not None:
        g.out = out.data_ptr()
        g.out_dtype = _dt(out)
        g.ldo = out.stride(0)
    g.num_sms = num_sms
    for k, v in getattr(_tls, "opts", {}).items():
        setattr(g, k, v)
    return g


def gemm_fp4(a, sfa, b, sfb, K: int, out_dtype=torch.bfloat16, alpha: float = 1.0, col_scale=None,
             lora_t=None, lora_b_t=None, bias=None, out=None, num_sms: int = 0, a_tensor_scale=None,
             b_tensor_scale=None, weights_ready: bool = False, stream=None):
    """Dense block-scaled FP4 GEMM: Y[M, N] from A codes [M, K/2] and B codes [N, K/2]
    (two-level operands: their device tensor scales from q4_quantize_two_level)."""
    M, N = a.shape[0], b.shape[0]
    if out is None:
        out = _empty((M, N), out_dtype, a.device, stream)
    g = _args(FMT_FP4, a, sfa, b, sfb, M, N, K, out, alpha, col_scale, lora_t, lora_b_t, bias, num_sms)
    g.a_tensor_scale = None if a_tensor_scale is None else a_tensor_scale.data_ptr()
    g.b_tensor_scale = None if b_tensor_scale is None else b_tensor_scale.data_ptr()
    g.weights_ready = 1 if weights_ready else 0
    lib = load()
    nbytes = int(lib.bs_gemm_workspace_bytes(ctypes.byref(g)))
    if nbytes:   # the decode kernel (M <= 32): stream-K scratch
        s = stream if stream is not None else torch.cuda.current_stream(a.device)
        ws = _workspace(a.device, s, nbytes)
        g.workspace, g.workspace_bytes = ws.data_ptr(), ws.numel()
    _check(load().bs_gemm(ctypes.byref(g), _stream(stream)))
    return out


# Workspaces of calls that bring none of their own (stream-K GEMMs, attention), one
# per (device, stream): calls on one stream run in order, so they may share it;
# the library leaves it zeroed where the next call reads it.  A CUDA graph keeps
# the address that it was captured with, so a buffer that a larger one replaces
# stays; sizes at least double, which bounds what all of them take by twice the last.
# Graphs captured on one stream share its buffer and must not overlap.
_workspaces: dict = {}
_outgrown: list = []


def _workspace(device, stream, nbytes: int):
    return _workspace_of(device, stream.cuda_stream, nbytes)


def _workspace_of(device, handle: int, nbytes: int):
    key = (device.index, handle)
    ws = _workspaces.get(key)
    if ws is None or ws.numel() < nbytes:
        # allocated and zeroed on the stream that uses it
        s = torch.cuda.current_stream(device)
        if s.cuda_stream != handle:
            s = torch.cuda.ExternalStream(handle, device=device)
        size = max(nbytes, 256, 2 * ws.numel() if ws is not None else 0)
        with torch.cuda.stream(s):
            new = torch.zeros(size, dtype=torch.uint8, device=device)
            if torch.cuda.is_current_stream_capturing():
                # the graph's own memory, zeroed when the graph runs and not
                # before: for this call alone
                return new
        if ws is not None:
            _outgrown.append(ws)
        _workspaces[key] = ws = new
    return ws


def gemm_fp8(a, sa, b, sb, out_dtype=torch.bfloat16, out=None, num_sms: int = 0, weights_ready: bool = False,
             rowwise: bool = False, stream=None):
    """Dense FP8 GEMM with 1x128 A scales [K/128, M] and 128x128 B scales.
    ``weights_ready``: the kernel just before this call on the stream does not
    write ``b`` / ``sb``, so the weight loads may start before it finishes."""
    M, K = a.shape
    N = b.shape[0]
    if out is None:
        out = _empty((M, N), out_dtype, a.device, stream)
    g = _args(FMT_FP8, a, sa, b, sb, M, N, K, out, num_sms=num_sms)
    g.weights_ready = 1 if weights_ready else 0
    g.fp8_scaling = 2 if rowwise else 0   # W8A8: sa [M] per token, sb [N] per channel
    lib = load()
    nbytes = int(lib.bs_gemm_workspace_bytes(ctypes.byref(g)))
    if nbytes:
        s = stream if stream is not None else torch.cuda.current_stream(a.device)
        ws = _workspace(a.device, s, nbytes)
        g.workspace, g.workspace_bytes = ws.data_ptr(), ws.numel()
    _check(lib.bs_gemm(ctypes.byref(g), _stream(stream)))
    return out


def _gemm_multi(fmt, a, sa, weights, M, N, K, out_dtype, outs, num_sms, weights_ready, alpha=1.0,
                a_tensor_scale=None, stream=None):
    G = len(weights)
    if G == 0:
        raise ValueError("bs_gemm_multi needs at least one weight set")
    if outs is not None and len(outs) != G:
        raise ValueError(f"{len(outs)} outputs for {G} weight sets")
    if outs is None:
        outs = [_empty((M, N), out_dtype, a.device, stream) for _ in range(G)]
    b0, sb0 = weights[0]
    g = _args(fmt, a, sa, b0, sb0, M, N, K, outs[0], alpha=alpha, num_sms=num_sms)
    g.weights_ready = 1 if weights_ready else 0
    g.a_tensor_scale = None if a_tensor_scale is None else a_tensor_scale.data_ptr()
    arr = ctypes.c_void_p * max(G, 1)
    bp = arr(*[w[0].data_ptr() for w in weights])
    sp = arr(*[w[1].data_ptr() for w in weights])
    op = arr(*[o.data_ptr() for o in outs])
    lib = load()
    nbytes = int(lib.bs_gemm_multi_workspace_bytes(ctypes.byref(g), G))
    if nbytes:
        s = stream if stream is not None else torch.cuda.current_stream(a.device)
        ws = _workspace(a.device, s, nbytes)
        g.workspace, g.workspace_bytes = ws.data_ptr(), ws.numel()
    _check(lib.bs_gemm_multi(ctypes.byref(g), G, bp, sp, op, _stream(stream)))
    return outs


def gemm_fp8_multi(a, sa, weights, out_dtype=torch.bfloat16, outs=None, num_sms: int = 0,
                   weights_ready: bool = False, stream=None):
    """G block-scaled FP8 GEMMs that share the tokens ``a`` [M, K] (M <= 32,
    TOKEN-mode scales ``sa``) in one launch: ``weights`` is a list of (codes
    [N, K], BLOCK-mode scales) pairs, one per product; returns the G outputs
    [M, N] (or fills ``outs``)."""
    M, K = a.shape
    N = weights[0][0].shape[0] if weights else 0
    return _gemm_multi(FMT_FP8, a, sa, weights, M, N, K, out_dtype, outs, num_sms, weights_ready, stream=stream)


def gemm_fp4_multi(a, sfa, weights, K: int, out_dtype=torch.bfloat16, outs=None, alpha: float = 1.0,
                   a_tensor_scale=None, num_sms: int = 0, weights_ready: bool = False, stream=None):
    """G FP4 decode GEMMs that share the tokens ``a`` (codes [M, K/2], M <= 32,
    scales ``sfa``) in one launch: ``weights`` is a list of (codes [N, K/2],
    scales) pairs from q4_quantize; returns the G outputs [M, N]."""
    M = a.shape[0]
    N = weights[0][0].shape[0] if weights else 0
    return _gemm_multi(FMT_FP4, a, sfa, weights, M, N, K, out_dtype, outs, num_sms, weights_ready, alpha=alpha,
                       a_tensor_scale=a_tensor_scale, stream=stream)


def grouped_gemm_fp4(a, sfa, b, sfb, K: int, N: int, E: int, offsets, counts, epilogue: int, out=None,
                     token_of=None, weight_of=None, out32=None, num_sms: int = 0, n_chunk_blocks: int = 0,
                     stream=None):
    """FP4 GEMM grouped over experts (rows of ``a`` grouped by ``offsets``/``counts``)."""
    M = a.shape[0]
    g = _args(FMT_FP4, a, sfa, b, sfb, M, N, K, out, num_sms=num_sms)
    g.n_chunk_blocks = n_chunk_blocks
    ld32 = 0 if out32 is None else out32.stride(0)
    _check(load().bs_grouped_gemm(ctypes.byref(g), E, _ptr(offsets), _ptr(counts), epilogue, _ptr(token_of),
                                  _ptr(weight_of), _ptr(out32), ld32, _stream(stream)))
    return out


def grouped_gemm_fp8(a, sfa, b, sfb, N: int, E: int, offsets, counts, epilogue: int, out=None, weight_of=None,
                     num_sms: int = 0, stream=None):
    """FP8 GEMM grouped over experts: ``a`` e4m3 [M, K] with TOKEN-mode scales
    ``sfa`` [K/128, M] (rows grouped by ``offsets``/``counts``), ``b`` the
    stacked expert weights [E*Nw, K] with 128x128 block scales ``sfb``.
    Epilogues EPI_STORE, EPI_SWIGLU (bf16 h) and EPI_ROWS (fp32, weight_of)."""
    M, K = a.shape
    if out is None:
        dt = torch.float32 if epilogue == EPI_ROWS else torch.bfloat16
        out = _empty((M, N), dt, a.device, stream)
    g = _args(FMT_FP8, a, sfa, b, sfb, M, N, K, out, num_sms=num_sms)
    _check(load().bs_grouped_gemm(ctypes.byref(g), E, _ptr(offsets), _ptr(counts), epilogue, None,
                                  _ptr(weight_of), None, 0, _stream(stream)))
    return out


def grouped_gemm_fp4_swiglu_q4(a, sfa, b, sfb, K: int, N: int, E: int, offsets, counts, h_codes=None, h_sf=None,
                               num_sms: int = 0, n_chunk_blocks: int = 0, stream=None):
    """Grouped gate/up GEMM with h = bf16(silu(g) * u) quantized to FP4 in the
    epilogue: returns (h_codes uint8 [M, N/2], h_sf scale bytes), as
    q4_quantize would write them for the segment rows."""
    M = a.shape[0]
    if h_codes is None:
        h_codes = _empty((M, N // 2), torch.uint8, a.device, stream)
    if h_sf is None:
        h_sf = _empty(sf_bytes(M, N), torch.uint8, a.device, stream)
    g = _args(FMT_FP4, a, sfa, b, sfb, M, N, K, None, num_sms=num_sms)
    g.n_chunk_blocks = n_chunk_blocks
    _check(load().bs_grouped_gemm_swiglu_q4(ctypes.byref(g), E, _ptr(offsets), _ptr(counts), _ptr(h_codes),
                                            _ptr(h_sf), _stream(stream)))
    return h_codes, h_sf


def moe_rows_bound(T: int, k: int, E: int) -> int:
    return int(load().bs_moe_rows_bound(T, k, E))


def moe_router_topk(logits, k: int, out=None, stream=None):
    """Top-k routing from fp32 router logits [T, E]: (topk_ids int32 [T, k] in
    descending order of logit, ties to the lower id; topk_w fp32 [T, k], the
    softmax of the chosen logits)."""
    T, E = logits.shape
    if out is None:
        out = (_empty((T, k), torch.int32, logits.device, stream),
               _empty((T, k), torch.float32, logits.device, stream))
    _check(load().bs_moe_router_topk(_ptr(logits), T, E, k, _ptr(out[0]), _ptr(out[1]), _stream(stream)))
    return out


def moe_dispatch(topk_ids, topk_w, E: int, out=None, workspace=None, stream=None):
    """Group (token, slot) pairs by expert.  Returns dict(counts, offsets,
    pair_of_row, token_of, weight_of) of device tensors (rows = moe_rows_bound)."""
    lib = load()
    T, k = topk_ids.shape
    dev = topk_ids.device
    rows = moe_rows_bound(T, k, E)
    if out is None:
        out = dict(counts=_empty(E, torch.int32, dev, stream),
                   offsets=_empty(E + 1, torch.int32, dev, stream),
                   pair_of_row=_empty(rows, torch.int32, dev, stream),
                   token_of=_empty(rows, torch.int32, dev, stream),
                   weight_of=_empty(rows, torch.float32, dev, stream))
    wsb = int(lib.bs_moe_dispatch_workspace_bytes(T, k, E))
    if workspace is None:
        workspace = _empty(max(wsb, 16), torch.uint8, dev, stream)
    _check(lib.bs_moe_dispatch(_ptr(topk_ids), _ptr(topk_w), T, k, E, _ptr(out["counts"]), _ptr(out["offsets"]),
                               _ptr(out["pair_of_row"]), _ptr(out["token_of"]), _ptr(out["weight_of"]),
                               _ptr(workspace), workspace.numel(), _stream(stream)))
    return out


def moe_finalize(out32, out_bf16, stream=None):
    _check(load().bs_moe_finalize(_ptr(out32), _ptr(out_bf16), out32.numel(), _stream(stream)))
    return out_bf16


def moe_combine(rows, pair_of_row, T: int, k: int, out=None, row_of_pair=None, stream=None):
    """out[t] = bf16(sum_j rows[row of pair t*k + j]) (fp32 sum in slot order);
    ``rows`` fp32 [n_rows, H] from a grouped GEMM with EPI_ROWS."""
    n_rows, H = rows.shape
    if out is None:
        out = _empty((T, H), torch.bfloat16, rows.device, stream)
    if row_of_pair is None:
        row_of_pair = _empty(max(T * k, 1), torch.int32, rows.device, stream)
    _check(load().bs_moe_combine(_ptr(rows), rows.stride(0), _ptr(pair_of_row), n_rows, T, k, H, _ptr(row_of_pair),
                                 _ptr(out), out.stride(0), _stream(stream)))
    return out


class KVCache(NamedTuple):
    """One layer's 8-bit paged cache: e4m3 codes uint8 [pages, Hkv, page_size,
    D] and fp32 scales [pages, Hkv] of keys and values."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @classmethod
    def empty(cls, num_pages: int, Hkv: int, page_size: int, D: int, device="cuda") -> "KVCache":
        shape = (num_pages, Hkv, page_size, D)
        return cls(torch.zeros(shape, dtype=torch.uint8, device=device),
                   torch.zeros(shape, dtype=torch.uint8, device=device),
                   torch.ones(shape[:2], dtype=torch.float32, device=device),
                   torch.ones(shape[:2], dtype=torch.float32, device=device))


class KVCacheFP4(NamedTuple):
    """One layer's 4-bit paged cache: E2M1 codes uint8 [pages, Hkv, page_size,
    D / 2] (two a byte) and e4m3 scales uint8 [pages, Hkv, page_size, D / 16] of
    keys and values."""
    k: torch.Tensor
    v: torch.Tensor
    k_scale: torch.Tensor
    v_scale: torch.Tensor

    @classmethod
    def empty(cls, num_pages: int, Hkv: int, page_size: int, D: int, device="cuda") -> "KVCacheFP4":
        shape = (num_pages, Hkv, page_size)
        return cls(*(torch.zeros((*shape, n), dtype=torch.uint8, device=device)
                     for n in (D // 2, D // 2, D // 16, D // 16)))


# Short names, identities instead of comparisons, one attribute read each: these
# calls launch kernels of a few microseconds, and their checks cost as much as
# the launch if they are written at leisure.
_F32, _BF16, _I32, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.uint8


def _check_kv_cache(cache):
    """(k, v, k_scale, v_scale, shape) of a KVCache (or such a tuple), checked
    for type and layout."""
    k, v, ks, vs = cache
    shape = k.shape
    if len(shape) != 4 or v.shape != shape or ks.shape != shape[:2] or vs.shape != shape[:2]:
        raise ValueError("a KV cache is codes [pages, Hkv, page_size, D] and scales [pages, Hkv], twice")
    if k.dtype is not _U8 or v.dtype is not _U8 or ks.dtype is not _F32 or vs.dtype is not _F32:
        raise TypeError("KV cache codes are uint8 (e4m3), scales float32")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError("KV cache buffers must be contiguous")
    return k, v, ks, vs, shape


def _check_kv_cache_fp4(cache):
    """(k, v, k_scale, v_scale, shape with D) of a KVCacheFP4, checked for type and layout."""
    k, v, ks, vs = cache
    shape, groups = k.shape, ks.shape
    if len(shape) != 4 or v.shape != shape or vs.shape != groups or groups != (*shape[:3], shape[3] // 8):
        raise ValueError("a 4-bit KV cache is codes [pages, Hkv, page_size, D / 2] and scales [.., D / 16], twice")
    if k.dtype is not _U8 or v.dtype is not _U8 or ks.dtype is not _U8 or vs.dtype is not _U8:
        raise TypeError("4-bit KV cache codes and scales are uint8 (E2M1 pairs, e4m3)")
    if not (k.is_contiguous() and v.is_contiguous() and ks.is_contiguous() and vs.is_contiguous()):
        raise ValueError("KV cache buffers must be contiguous")
    return k, v, ks, vs, (shape[0], shape[1], shape[2], 2 * shape[3])


def _not_on_gpu(name):
    """The calls hand addresses to kernels on the current GPU's stream: a tensor elsewhere is refused before that."""
    raise ValueError(f"{name}: every tensor is on the current GPU")


def _ints(name, *tensors):
    for t in tensors:
        if t.dtype is not _I32 or not t.is_contiguous():
            raise TypeError(f"{name}: lengths, tables and slots are contiguous int32 tensors")


def _check_table(name, table, B):
    """(row stride, width) of a block table of B requests."""
    shape, stride = table.shape, table.stride()
    if table.dtype is not _I32 or len(shape) != 2 or stride[1] != 1:
        raise TypeError(f"{name}: block_table is an int32 [B, max_pages] tensor with contiguous rows")
    if shape[0] != B:
        raise ValueError(f"{name}: block_table has {shape[0]} rows for {B} requests")
    return stride[0], shape[1]


def kv_plan(seq_lens, new_lens, block_table, free_pages, n_free, page_size: int, total_new: int, out=None,
            stream=None):
    """Block tables and slots of a step, from the requests' lengths (device
    int32): request b takes the pages that its new tokens need from the end of
    ``free_pages[:n_free]``; ``block_table`` [B, max_pages] is updated in place.
    Returns (cu_new [B + 1], kv_lens [B], slots [total_new], n_free [1])."""
    B = seq_lens.numel()
    if out is None:
        dev = seq_lens.device
        out = (_empty(B + 1, _I32, dev, stream), _empty(B, _I32, dev, stream), _empty(total_new, _I32, dev, stream),
               _empty(1, _I32, dev, stream))
    cu, kv, slots, left = out
    _ints("kv_plan", seq_lens, new_lens, free_pages, n_free, cu, kv, slots, left)
    if new_lens.numel() != B:
        raise ValueError("kv_plan: seq_lens and new_lens differ in the number of requests")
    ld, width = _check_table("kv_plan", block_table, B)
    if cu.numel() < B + 1 or kv.numel() < B or slots.numel() < total_new or left.numel() < 1:
        raise ValueError("kv_plan: outputs are [B + 1], [B], [total_new] and [1]")
    if n_free.numel() != 1:
        raise ValueError("kv_plan: n_free is an int32 tensor of one element")
    here = seq_lens.get_device()
    if (here < 0 or new_lens.get_device() != here or block_table.get_device() != here or free_pages.get_device() != here
            or n_free.get_device() != here or cu.get_device() != here or kv.get_device() != here
            or slots.get_device() != here or left.get_device() != here or here != _device()):
        _not_on_gpu("kv_plan")
    a = _KV_PLAN_ARGS.pack(seq_lens.data_ptr(), new_lens.data_ptr(), B, block_table.data_ptr(), ld, width,
                           free_pages.data_ptr(), n_free.data_ptr(), free_pages.numel(), page_size, total_new,
                           cu.data_ptr(), kv.data_ptr(), slots.data_ptr(), left.data_ptr())
    _check((_lib or load()).bs_kv_plan(a, _stream(stream)))
    return out


def kv_release(lens, done, block_table, free_pages, n_free, page_size: int, stream=None):
    """Give the pages of the requests with ``done[b] != 0`` (``lens[b]`` cached
    tokens) back to the free list, in place."""
    _ints("kv_release", lens, done, free_pages, n_free)
    B = lens.numel()
    if done.numel() != B:
        raise ValueError("kv_release: lens and done differ in the number of requests")
    if n_free.numel() != 1:
        raise ValueError("kv_release: n_free is an int32 tensor of one element")
    ld, width = _check_table("kv_release", block_table, B)
    here = lens.get_device()
    if (here < 0 or done.get_device() != here or block_table.get_device() != here or free_pages.get_device() != here
            or n_free.get_device() != here or here != _device()):
        _not_on_gpu("kv_release")
    _check((_lib or load()).bs_kv_release(
        lens.data_ptr(), done.data_ptr(), B, block_table.data_ptr(), ld, width, free_pages.data_ptr(),
        n_free.data_ptr(), free_pages.numel(), page_size, _stream(stream)))


def kv_append(k, v, slots, cache, stream=None):
    """Quantize new keys and values [T, Hkv, D] (fp32 or bf16, any token and
    head strides) into their slots of the cache (KVCache or KVCacheFP4), in place."""
    if type(cache) is KVCacheFP4:
        kv_append_rotary(None, k, v, slots, None, None, cache, stream=stream)
        return
    kc, vc, ks, vs, (pages, Hkv, page, D) = _check_kv_cache(cache)
    shape = k.shape
    T = slots.numel()
    if shape != (T, Hkv, D) or v.shape != shape:
        raise ValueError(f"kv_append: k and v are [{T}, {Hkv}, {D}] for these slots and this cache")
    (kt, kh, kd), (vt, vh, vd) = k.stride(), v.stride()
    dt = k.dtype
    if kd != 1 or vd != 1 or v.dtype is not dt:
        raise ValueError("kv_append: k and v have one type and contiguous rows of D")
    if dt is not _BF16 and dt is not _F32:
        raise TypeError(f"unsupported dtype {dt}")
    if slots.dtype is not _I32 or not slots.is_contiguous():
        raise TypeError("kv_append: slots is a contiguous int32 tensor")
    here = k.get_device()
    if (here < 0 or v.get_device() != here or slots.get_device() != here or kc.get_device() != here
            or vc.get_device() != here or ks.get_device() != here or vs.get_device() != here or here != _device()):
        _not_on_gpu("kv_append")
    a = _KV_APPEND_ARGS.pack(k.data_ptr(), v.data_ptr(), DTYPE_BF16 if dt is _BF16 else DTYPE_F32, T, Hkv, D, kt, kh,
                             vt, vh, slots.data_ptr(), kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                             pages, page)
    _check((_lib or load()).bs_kv_append(a, _stream(stream)))


def rotary_angles(max_positions: int, rotary_dim: int, base: float = 10000.0, device="cuda"):
    """The table that kv_append_rotary reads: cos, then sin, of position *
    base^(-2 i / rotary_dim), i < rotary_dim / 2, in fp32 (computed in 64 bits)."""
    f = base ** (-torch.arange(0, rotary_dim, 2, dtype=torch.float64, device=device) / rotary_dim)
    a = torch.arange(max_positions, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def kv_positions(seq_lens, cu_new, total_new: int, out=None, stream=None):
    """The place of each new token in its request, int32 [total_new]: seq_lens[b] + i for
    row cu_new[b] + i (both as kv_plan takes and gives them), 0 behind the last request."""
    B = seq_lens.numel()
    if out is None:
        out = _empty((total_new,), _I32, seq_lens.device, stream)
    _ints("kv_positions", seq_lens, cu_new, out)
    if cu_new.numel() != B + 1 or out.numel() != total_new:
        raise ValueError("kv_positions: cu_new is [B + 1], out [total_new]")
    here = seq_lens.get_device()
    if here < 0 or cu_new.get_device() != here or out.get_device() != here or here != _device():
        _not_on_gpu("kv_positions")
    _check((_lib or load()).bs_kv_positions(seq_lens.data_ptr(), cu_new.data_ptr(), B, total_new, out.data_ptr(),
                                            _stream(stream)))
    return out


def kv_append_rotary(q, k, v, slots, positions, angles, cache, q_out=None, interleaved: bool = False, stream=None):
    """New keys and values [T, Hkv, D] into their slots of the cache (KVCache or
    KVCacheFP4), in place, and new queries [T, Hq, D] to bf16, queries and keys
    rotated by the angles (fp32 [max_positions, R], see rotary_angles) of their
    positions (int32 [T]): pairs i, i + R / 2, or 2 i, 2 i + 1 if ``interleaved``.
    ``q`` None: keys and values only; ``angles`` None: no rotation.  ``q_out`` may be
    ``q`` (bf16).  Rows with a negative slot are skipped.  Returns q_out."""
    fp4 = type(cache) is KVCacheFP4
    kc, vc, ks, vs, (pages, Hkv, page, D) = _check_kv_cache_fp4(cache) if fp4 else _check_kv_cache(cache)
    T = slots.numel()
    dt = k.dtype
    if k.shape != (T, Hkv, D) or v.shape != k.shape:
        raise ValueError(f"kv_append_rotary: k and v are [{T}, {Hkv}, {D}] for these slots and this cache")
    if dt is not _BF16 and dt is not _F32:
        raise TypeError(f"unsupported dtype {dt}")
    (kt, kh, kd), (vt, vh, vd) = k.stride(), v.stride()
    if kd != 1 or vd != 1 or v.dtype is not dt:
        raise ValueError("kv_append_rotary: q, k and v have one type and contiguous rows of D")
    if slots.dtype is not _I32 or not slots.is_contiguous():
        raise TypeError("kv_append_rotary: slots is a contiguous int32 tensor")
    here = k.get_device()
    elsewhere = (here < 0 or v.get_device() != here or slots.get_device() != here or kc.get_device() != here
                 or vc.get_device() != here or ks.get_device() != here or vs.get_device() != here)
    if q is None:
        if q_out is not None:
            raise ValueError("kv_append_rotary: q_out without q")
        q_ptr = qt = qh = out_ptr = ot = oh = Hq = 0
    else:
        shape = q.shape
        if q_out is None:
            q_out = _empty(shape, _BF16, q.device, stream)
        if len(shape) != 3 or shape[0] != T or shape[2] != D or q_out.shape != shape:
            raise ValueError(f"kv_append_rotary: q and q_out are [{T}, Hq, {D}]")
        Hq = shape[1]
        (qt, qh, qd), (ot, oh, od) = q.stride(), q_out.stride()
        if qd != 1 or od != 1 or q.dtype is not dt:
            raise ValueError("kv_append_rotary: q, k and v have one type and contiguous rows of D")
        if q_out.dtype is not _BF16:
            raise TypeError("kv_append_rotary: q_out is bfloat16")
        q_ptr, out_ptr = q.data_ptr(), q_out.data_ptr()
        elsewhere = elsewhere or q.get_device() != here or q_out.get_device() != here
    if angles is None:
        at_ptr = angles_ptr = rows = R = 0
    else:
        if angles.dtype is not _F32 or angles.dim() != 2 or not angles.is_contiguous():
            raise TypeError("kv_append_rotary: angles is a contiguous float32 [max_positions, R] tensor")
        if positions is None or positions.dtype is not _I32 or positions.numel() != T or not positions.is_contiguous():
            raise TypeError(f"kv_append_rotary: positions is a contiguous int32 tensor of {T}")
        rows, R = angles.shape
        at_ptr, angles_ptr = positions.data_ptr(), angles.data_ptr()
        elsewhere = elsewhere or positions.get_device() != here or angles.get_device() != here
    if elsewhere or here != _device():
        _not_on_gpu("kv_append_rotary")
    a = _KV_APPEND_ROTARY_ARGS.pack(q_ptr, qt, qh, out_ptr, ot, oh, k.data_ptr(), v.data_ptr(),
                                    DTYPE_BF16 if dt is _BF16 else DTYPE_F32, Hq, Hkv, D, T, kt, kh, vt, vh,
                                    slots.data_ptr(), at_ptr, angles_ptr, rows, R, 1 if interleaved else 0,
                                    FMT_FP4 if fp4 else FMT_FP8, page, kc.data_ptr(), vc.data_ptr(), ks.data_ptr(),
                                    vs.data_ptr(), pages)
    status = (_lib or load()).bs_kv_append_rotary(a, _stream(stream))
    if status:
        _check(status)
    return q_out


def kv_gather(cache, slots, out=None, stream=None):
    """The rows of the cache (KVCache or KVCacheFP4) at these slots as bf16: (k, v),
    [T, Hkv, D] each.  Rows of negative slots are left as they were (whatever a new
    tensor holds, without ``out``)."""
    fp4 = type(cache) is KVCacheFP4
    kc, vc, ks, vs, (pages, Hkv, page, D) = _check_kv_cache_fp4(cache) if fp4 else _check_kv_cache(cache)
    if slots.dtype is not _I32 or not slots.is_contiguous():
        raise TypeError("kv_gather: slots is a contiguous int32 tensor")
    shape = (slots.numel(), Hkv, D)
    if out is None:
        out = (_empty(shape, _BF16, kc.device, stream), _empty(shape, _BF16, kc.device, stream))
    k, v = out
    (kt, kh, kd), (vt, vh, vd) = k.stride(), v.stride()
    if k.shape != shape or v.shape != shape or kd != 1 or vd != 1:
        raise ValueError(f"kv_gather: k and v are {list(shape)} with contiguous rows of D")
    if k.dtype is not _BF16 or v.dtype is not _BF16:
        raise TypeError("kv_gather: k and v are bfloat16")
    here = slots.get_device()
    if (here < 0 or here != _device() or kc.get_device() != here or vc.get_device() != here or ks.get_device() != here
            or vs.get_device() != here or k.get_device() != here or v.get_device() != here):
        _not_on_gpu("kv_gather")
    a = _KV_GATHER_ARGS.pack(slots.data_ptr(), shape[0], Hkv, D, k.data_ptr(), v.data_ptr(), kt, kh, vt, vh,
                             FMT_FP4 if fp4 else FMT_FP8, page, kc.data_ptr(), vc.data_ptr(), ks.data_ptr(),
                             vs.data_ptr(), pages)
    _check((_lib or load()).bs_kv_gather(a, _stream(stream)))
    return k, v


_kv_workspace_sizes: dict = {}   # (device, D) -> bytes


def _kv_workspace_bytes(lib, dev: int, D: int) -> int:
    """Workspace of any kv_attention call of heads of D on this device: the
    library's answer for a long call, no bound known, which is its largest.  0,
    which is not kept, where the library has no answer (and refuses the call)."""
    nbytes = _kv_workspace_sizes.get((dev, D))
    if nbytes is None:
        a = _KV_ATTENTION_ARGS.pack(*(0,) * 19, 1 << 20, 1, 1, D, *(0,) * 5)   # T, Hq, Hkv, D
        nbytes = int(lib.bs_kv_attention_workspace_bytes(a))
        if nbytes:
            _kv_workspace_sizes[(dev, D)] = nbytes
    return nbytes


def kv_attention_workspace(D: int, device=None):
    """A zeroed workspace for kv_attention calls with heads of D that run one
    after the other, whatever their lengths."""
    device = torch.device("cuda" if device is None else device)
    with torch.cuda.device(device):
        nbytes = _kv_workspace_bytes(_lib or load(), torch.cuda.current_device(), D)
    if not nbytes:
        raise ValueError(f"kv_attention_workspace: no kernel for heads of {D}")
    return torch.zeros(nbytes, dtype=torch.uint8, device=device)


def kv_attention(q, cache, block_table, cu_q, kv_lens, max_q_len: int, softmax_scale: float | None = None, out=None,
                 lse=None, stream=None, workspace=None):
    """Causal attention of new tokens q bf16 [T, Hq, D] over the cache, KVCache or
    KVCacheFP4 (their own keys and values appended first).  ``lse`` (fp32 [T, Hq], natural
    log) is filled if given.  ``workspace`` from kv_attention_workspace, or the
    stream's own if None.  Returns out bf16 [T, Hq, D]."""
    fp4 = type(cache) is KVCacheFP4
    kc, vc, ks, vs, (pages, Hkv, page, D) = _check_kv_cache_fp4(cache) if fp4 else _check_kv_cache(cache)
    shape = q.shape
    if out is None:
        out = _empty(shape, _BF16, q.device, stream)
    if q.dtype is not _BF16 or out.dtype is not _BF16:
        raise TypeError("kv_attention: q and out are bfloat16")
    if len(shape) != 3 or shape[2] != D or out.shape != shape:
        raise ValueError(f"kv_attention: q and out are [T, Hq, {D}]")
    T, Hq, _ = shape
    (qt, qh, qd), (ot, oh, od) = q.stride(), out.stride()
    if qd != 1 or od != 1:
        raise ValueError("kv_attention: rows of q and out are contiguous")
    B = kv_lens.numel()
    ld, width = _check_table("kv_attention", block_table, B)
    if cu_q.numel() != B + 1:
        raise ValueError("kv_attention: cu_q is [B + 1] and kv_lens [B]")
    if cu_q.dtype is not _I32 or kv_lens.dtype is not _I32 or not cu_q.is_contiguous() or not kv_lens.is_contiguous():
        raise TypeError("kv_attention: cu_q and kv_lens are contiguous int32 tensors")
    here = q.get_device()
    if lse is None:
        lse_ptr = 0
    else:
        if lse.dtype is not _F32 or lse.shape != (T, Hq) or not lse.is_contiguous():
            raise ValueError("kv_attention: lse is a contiguous float32 [T, Hq] tensor")
        if here < 0 or lse.get_device() != here:
            _not_on_gpu("kv_attention")
        lse_ptr = lse.data_ptr()
    if workspace is not None:
        if workspace.dtype is not _U8 or not workspace.is_contiguous():
            raise TypeError("kv_attention: workspace is a contiguous uint8 tensor of kv_attention_workspace")
        if here < 0 or workspace.get_device() != here:
            _not_on_gpu("kv_attention")
    if (here < 0 or out.get_device() != here or kc.get_device() != here or vc.get_device() != here
            or ks.get_device() != here or vs.get_device() != here or block_table.get_device() != here
            or cu_q.get_device() != here or kv_lens.get_device() != here or here != _device()):
        _not_on_gpu("kv_attention")
    handle = _stream(stream)
    opts = getattr(_tls, "opts", None)
    args = (q.data_ptr(), qt, qh, out.data_ptr(), ot, oh, lse_ptr, kc.data_ptr(), vc.data_ptr(), ks.data_ptr(),
            vs.data_ptr(), pages, page, block_table.data_ptr(), ld, width, cu_q.data_ptr(), kv_lens.data_ptr(), B, T,
            Hq, Hkv, D, max_q_len, D ** -0.5 if softmax_scale is None else softmax_scale,
            opts.get("wait_timeout_us", 0) if opts else 0)
    lib = _lib or load()
    if workspace is not None:
        ws, nbytes = workspace, workspace.numel()
    else:
        nbytes = _kv_workspace_bytes(lib, here, D)
        ws = _workspaces.get((here, handle))
        if ws is None or ws.numel() < nbytes:
            ws = _workspace_of(q.device, handle, nbytes)
    packed = _KV_ATTENTION_ARGS.pack(*args, ws.data_ptr(), nbytes)
    if fp4:
        _check(lib.bs_kv_attention_fp4(packed, ks.data_ptr(), vs.data_ptr(), handle))
    else:
        _check(lib.bs_kv_attention(packed, handle))
    return out


def matvec_fp4(x, codes, sf, out_dtype=torch.bfloat16, alpha: float = 1.0, bias=None, tensor_scale=None, out=None,
               stream=None):
    """x [M <= 16, K] bf16 times FP4 weights (codes [N, K/2] and MMA-layout
    scales from q4_quantize, with ``tensor_scale`` of q4_quantize_two_level):
    Y = alpha tensor_scale x W^T + bias, x left unquantized."""
    (M, K), (N, half) = x.shape, codes.shape
    ldx, one = x.stride()
    if x.dtype is not _BF16 or one != 1:
        raise TypeError("matvec_fp4: x is a bfloat16 [M, K] tensor with contiguous rows")
    if codes.dtype is not _U8 or half * 2 != K or not codes.is_contiguous():
        raise ValueError(f"matvec_fp4: codes are contiguous uint8 [N, {K // 2}]")
    if sf.dtype is not _U8 or sf.numel() < (N + 127) // 128 * 128 * (K // 16) or not sf.is_contiguous():
        raise ValueError("matvec_fp4: sf are the uint8 scales of [N, K], bs_sf_bytes(N, K) of them, contiguous")
    if bias is not None and (bias.dtype is not _BF16 or bias.numel() != N or not bias.is_contiguous()):
        raise ValueError("matvec_fp4: bias is a contiguous bfloat16 [N] tensor")
    if tensor_scale is not None and (tensor_scale.dtype is not _F32 or tensor_scale.numel() != 1):
        raise TypeError("matvec_fp4: tensor_scale is a float32 tensor of one element")
    if out is None:
        out = _empty((M, N), out_dtype, x.device, stream)
    ldo, one = out.stride()
    if out.shape != (M, N) or one != 1:
        raise ValueError(f"matvec_fp4: out is [{M}, {N}] with contiguous rows")
    here = x.get_device()
    if (here < 0 or codes.get_device() != here or sf.get_device() != here or out.get_device() != here
            or (bias is not None and bias.get_device() != here)
            or (tensor_scale is not None and tensor_scale.get_device() != here) or here != _device()):
        _not_on_gpu("matvec_fp4")
    if M <= 1:
        ldx, ldo = K, N   # the stride of a single row means nothing
    a = _FP4_MATVEC_ARGS.pack(x.data_ptr(), ldx, M, codes.data_ptr(), sf.data_ptr(), N, K, alpha,
                              0 if tensor_scale is None else tensor_scale.data_ptr(),
                              0 if bias is None else bias.data_ptr(), out.data_ptr(), _dt(out), ldo)
    _check((_lib or load()).bs_fp4_matvec(a, _stream(stream)))
    return out


def lora_add(x, y, a, b, cu_rows, which, scales=None, out=None, stream=None):
    """y + scale x A^T B^T with the low-rank adapter of each request, beside a
    projection y [T, N] (bf16 or fp32) of x bf16 [T, K] that all share.  ``a`` bf16
    [adapters, r, K], ``b`` bf16 [adapters, N, r], ``scales`` fp32 [adapters] or None
    (1); request b has the rows cu_rows[b] .. cu_rows[b + 1] - 1 (int32 [B + 1], as
    kv_plan gives them) and the adapter which[b] (int32 [B]; negative: none).  ``out``
    may be ``y``; rows from cu_rows[B] on are not written.  Returns out."""
    if x.dim() != 2 or y.dim() != 2 or a.dim() != 3 or b.dim() != 3:
        raise ValueError("lora_add: x [T, K], y [T, N], a [adapters, r, K], b [adapters, N, r]")
    (T, K), N, (n, r, _) = x.shape, y.shape[1], a.shape
    if out is None:
        out = _empty(y.shape, y.dtype, y.device, stream)
    if y.shape[0] != T or a.shape[2] != K or b.shape != (n, N, r) or out.shape != y.shape:
        raise ValueError("lora_add: x [T, K], y and out [T, N], a [adapters, r, K], b [adapters, N, r]")
    if x.dtype is not _BF16 or a.dtype is not _BF16 or b.dtype is not _BF16:
        raise TypeError("lora_add: x, a and b are bfloat16")
    if out.dtype is not y.dtype:
        raise TypeError("lora_add: y and out have one type")
    (ldx, x1), (ldy, y1), (ldo, o1) = x.stride(), y.stride(), out.stride()
    if x1 != 1 or y1 != 1 or o1 != 1 or not a.is_contiguous() or not b.is_contiguous():
        raise ValueError("lora_add: rows of x, y and out, and all of a and b, are contiguous")
    _ints("lora_add", cu_rows, which)
    B = which.numel()
    if cu_rows.numel() != B + 1:
        raise ValueError("lora_add: cu_rows is [B + 1] and which [B]")
    if scales is not None and (scales.dtype is not _F32 or scales.numel() != n or not scales.is_contiguous()):
        raise TypeError(f"lora_add: scales is a contiguous float32 tensor of {n}")
    here = x.get_device()
    if (here < 0 or y.get_device() != here or a.get_device() != here or b.get_device() != here or out.get_device() != here
            or cu_rows.get_device() != here or which.get_device() != here
            or (scales is not None and scales.get_device() != here) or here != _device()):
        _not_on_gpu("lora_add")
    packed = _LORA_ARGS.pack(x.data_ptr(), ldx, a.data_ptr(), b.data_ptr(), 0 if scales is None else scales.data_ptr(),
                             cu_rows.data_ptr(), which.data_ptr(), y.data_ptr(), ldy, out.data_ptr(), ldo, _dt(y), B, T,
                             K, N, r, n)
    status = (_lib or load()).bs_lora_add(packed, _stream(stream))
    if status:
        _check(status)
    return out


def device_status() -> tuple[int, int]:
    d = ctypes.c_int(0)
    s = load().bs_get_device_status(ctypes.byref(d))
    return int(s), int(d.value)


def clear_device_status():
    _check(load().bs_clear_device_status())
