"""ctypes binding of libaggemm.so: argument marshalling only.

Every step of the operation runs in the library's HIP kernels; this module
turns torch tensors into device pointers and sizes, passes the current
stream, and raises on a non-zero status.  The library must have been built
(``python communication_gemm_amd/build.py``); importing this module without
it fails loudly, there is no fallback.
"""
from __future__ import annotations

import ctypes
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libaggemm.so")

(AGG_OK, AGG_E_INVALID, AGG_E_UNSUPPORTED, AGG_E_NOMEM, AGG_E_HIP, AGG_E_TIMEOUT,
 AGG_E_TOO_LARGE) = range(7)
NOALLOC_MAX_BYTES = 64 << 20   # AGG_NOALLOC_MAX_BYTES
MODE_PIPELINED, MODE_COMPUTE_ONLY, MODE_SEQUENTIAL, MODE_COPY_ONLY = range(4)
SCHEME_COUNTERS, SCHEME_BARRIER = range(2)
LINKS_PARALLEL, LINKS_SERIAL = range(2)
PRODUCER_KERNEL, PRODUCER_SDMA, PRODUCER_SEPARATE, PRODUCER_FUSED = range(4)
MAX_SHARDS = 64
TYPE_F16, TYPE_BF16, TYPE_FP8, TYPE_F32 = 0, 2, 3, 4   # enum agg_type
SCALE_BLOCK = 128
MX_BLOCK = 32          # columns that one E8M0 scale covers
MAX_EXPERTS = 4096     # of a sort


class AggError(RuntimeError):
    """A non-zero status from the library."""

    def __init__(self, status: int, what: str):
        self.status = status
        super().__init__(f"{what}: {status_string(status)} (status {status})")


class Options(ctypes.Structure):
    """Mirror of ``struct agg_options`` in include/aggemm.h."""

    _fields_ = [
        ("struct_size", ctypes.c_uint32),
        ("local_shard", ctypes.c_int),
        ("send_order", ctypes.POINTER(ctypes.c_int)),
        ("mode", ctypes.c_int),
        ("link_gbps", ctypes.c_double),
        ("link_model", ctypes.c_int),
        ("producer_wgs", ctypes.c_int),
        ("consumer_wgs", ctypes.c_int),
        ("tile", ctypes.c_int),
        ("acc_out", ctypes.c_void_p),
        ("workspace", ctypes.c_void_p),
        ("workspace_bytes", ctypes.c_size_t),
        ("timeout_ms", ctypes.c_double),
        ("debug_drop_chunk", ctypes.c_int),
        ("consumer_events", ctypes.c_void_p * 2),
        ("workspace_stages", ctypes.c_int),
        ("scheme", ctypes.c_int),
        ("pvalue", ctypes.c_int),
        ("trace", ctypes.c_void_p),
        ("producer_piece_bytes", ctypes.c_int64),
        ("k_splits", ctypes.c_int),
        ("debug_delay_us", ctypes.c_double),
        ("debug_delay_seed", ctypes.c_uint32),
        ("producer", ctypes.c_int),
        ("producer_cus", ctypes.c_int),
        ("k_block", ctypes.c_int64),
    ]


class PlanInfo(ctypes.Structure):
    """Mirror of ``struct agg_plan_info``."""

    _fields_ = [
        ("shard_rows", ctypes.c_int64),
        ("chunk_rows", ctypes.c_int),
        ("chunks_per_source", ctypes.c_int),
        ("tile_m", ctypes.c_int),
        ("tile_n", ctypes.c_int),
        ("m_tiles_per_shard", ctypes.c_int),
        ("n_tiles", ctypes.c_int),
        ("total_tiles", ctypes.c_int64),
        ("total_chunks", ctypes.c_int64),
        ("consumer_wgs", ctypes.c_int),
        ("producer_wgs", ctypes.c_int),
        ("tile_id", ctypes.c_int),
        ("trace_words", ctypes.c_int64),
        ("workspace_stages", ctypes.c_int),
        ("workspace_bytes", ctypes.c_int64),
        ("k_splits", ctypes.c_int),
        ("k_blocks", ctypes.c_int),
        ("k_block", ctypes.c_int64),
        ("producer_fused", ctypes.c_int),
    ]


def _sig(spec):
    """argtypes from letters: p(ointer), l (int64), i(nt), z (size_t), f(loat)."""
    kinds = {"p": ctypes.c_void_p, "l": ctypes.c_int64, "i": ctypes.c_int, "z": ctypes.c_size_t,
             "f": ctypes.c_float}
    return [kinds[c] for c in spec.replace(" ", "")]


EXPORTS = {
    # name: (restype, argtypes)
    "ag_gemm_options_init": (None, [ctypes.POINTER(Options)]),
    "ag_gemm_f16": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                   ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]),
    "ag_gemm_f16_ex": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                      ctypes.POINTER(Options)]),
    "ag_gemm_f16_noalloc": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                           ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                           ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                           ctypes.POINTER(Options)]),
    "ag_gemm_bf16": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                    ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                    ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]),
    "ag_gemm_bf16_ex": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                       ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                       ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                       ctypes.POINTER(Options)]),
    "ag_gemm_fp8": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                   ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                   ctypes.c_int64, ctypes.c_int, ctypes.c_void_p]),
    "ag_gemm_fp8_ex": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                      ctypes.c_void_p, ctypes.c_int64, ctypes.c_int64,
                                      ctypes.c_int64, ctypes.c_int, ctypes.c_void_p,
                                      ctypes.POINTER(Options)]),
    "ag_gemm_i8_dequant": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                          ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                          ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                          ctypes.c_int, ctypes.c_void_p]),
    "ag_gemm_i8_dequant_ex": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_int, ctypes.c_void_p,
                                             ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p,
                                             ctypes.c_int64, ctypes.c_int64, ctypes.c_int64,
                                             ctypes.c_int, ctypes.c_void_p,
                                             ctypes.POINTER(Options)]),
    "ag_gemm_pick_chunk_rows": (ctypes.c_int, [ctypes.c_int64]),
    "ag_gemm_workspace_bytes": (ctypes.c_size_t, [ctypes.c_int, ctypes.c_int64,
                                                  ctypes.c_int64, ctypes.c_int]),
    "ag_gemm_workspace_reset": (ctypes.c_int, [ctypes.c_void_p, ctypes.c_size_t,
                                               ctypes.c_void_p]),
    "ag_gemm_check": (ctypes.c_int, [ctypes.c_void_p]),
    "ag_gemm_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "ag_gemm_release": (None, []),
    "ag_gemm_plan": (ctypes.c_int, [ctypes.c_int, ctypes.c_int, ctypes.c_int64,
                                    ctypes.c_int64, ctypes.c_int64, ctypes.c_int,
                                    ctypes.POINTER(Options), ctypes.c_int,
                                    ctypes.POINTER(PlanInfo), ctypes.c_void_p,
                                    ctypes.c_void_p]),
    "ag_gemm_grouped": (ctypes.c_int, _sig("i pl pll i pi pl i lll p")),
    "ag_gemm_grouped_wgrad": (ctypes.c_int, _sig("i pl pl pi pll i lll p")),
    "ag_gemm_fp8_block": (ctypes.c_int, _sig("pl pl pl pl pl i lll p")),
    "ag_gemm_grouped_fp8_block": (ctypes.c_int, _sig("pl pl pll pll pi pl i lll p")),
    "ag_gemm_quant_fp8_block": (ctypes.c_int, _sig("i pl pl pl i ll p")),
    "ag_gemm_expert_sort_workspace_bytes": (ctypes.c_size_t, _sig("lii")),
    "ag_gemm_expert_sort": (ctypes.c_int, _sig("pil lii pp pz p")),
    "ag_gemm_expert_dispatch": (ctypes.c_int, _sig("i pl pi pll ll p")),
    "ag_gemm_expert_combine": (ctypes.c_int, _sig("i pll pi pl pli ll p")),
    "ag_gemm_expert_combine_grad": (ctypes.c_int, _sig("i pl pll pi pl pl pl ll p")),
    "ag_gemm_rmsnorm": (ctypes.c_int, _sig("i pl pl p pl pl pl pl pf ll p")),
    "ag_gemm_rmsnorm_grad_workspace_bytes": (ctypes.c_size_t, _sig("ll")),
    "ag_gemm_rmsnorm_grad": (ctypes.c_int, _sig("i pl pl pp pl pl pi pz ll p")),
    "ag_gemm_quant_mxfp4": (ctypes.c_int, _sig("i pl pl pl ll p")),
    "ag_gemm_dequant_mxfp4": (ctypes.c_int, _sig("pl pl pli ll p")),
    "ag_gemm_mxfp4": (ctypes.c_int, _sig("pl pl pl pl pl i lll p")),
    "ag_gemm_grouped_mxfp4": (ctypes.c_int, _sig("pl pl pll pll pi pl i lll p")),
}


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(
            f"{LIB_PATH} is missing: build it with "
            "`python communication_gemm_amd/build.py` (hipcc, gfx950)")
    # torch first: it brings its own HIP runtime, and the library must bind
    # to that one.  Loaded the other way round, the process ends up with the
    # system runtime under torch, and torch's first device allocation fails.
    import torch  # noqa: F401
    lib = ctypes.CDLL(LIB_PATH)
    for name, (res, args) in EXPORTS.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


lib = _load()


def status_string(status: int) -> str:
    return lib.ag_gemm_status_string(int(status)).decode()


def _raise(status: int, what: str):
    if status:
        raise AggError(status, what)


class Prepared:
    """One call with its arguments marshalled once: each call of this object
    only crosses the C ABI (tight loops pay no Python-side checks).  It runs on
    the stream it was prepared for: the one given, or the one current at the
    time.  (The expert products, prepared without a stream, follow the current
    one.)  It keeps the ctypes arguments and the options alive; the caller
    keeps the tensors alive."""

    __slots__ = ("_fn", "_args", "_what", "_keep")

    def __init__(self, fn, args, what, keep):
        self._fn = fn
        self._args = tuple(args)
        self._what = what
        self._keep = keep

    def __call__(self):
        rc = self._fn(*self._args)
        if rc:
            raise AggError(rc, self._what)


def _invoke(plain, ex, args, opts, what, prepare):
    """Call (or, with prepare=True, return a Prepared call of) the plain or
    the _ex entry point with marshalled arguments."""
    fn = plain if opts is None else ex
    full = tuple(args) if opts is None else tuple(args) + (ctypes.byref(opts),)
    if prepare:
        return Prepared(fn, full, what, (args, opts))
    _raise(fn(*full), what)


def options(**kw) -> Options:
    """An agg_options with the library's defaults, then ``kw`` applied.

    ``send_order`` may be a sequence of ints; ``consumer_events`` a pair of
    torch.cuda.Event objects; ``acc_out``/``workspace`` torch tensors.
    """
    o = Options()
    lib.ag_gemm_options_init(ctypes.byref(o))
    keep = []
    for k, v in kw.items():
        if v is None:
            continue
        if k == "send_order":
            arr = (ctypes.c_int * len(v))(*[int(x) for x in v])
            keep.append(arr)
            o.send_order = ctypes.cast(arr, ctypes.POINTER(ctypes.c_int))
        elif k == "consumer_events":
            o.consumer_events[0] = ctypes.c_void_p(v[0].cuda_event)
            o.consumer_events[1] = ctypes.c_void_p(v[1].cuda_event)
        elif k in ("acc_out", "workspace", "trace"):
            if hasattr(v, "data_ptr"):
                if not v.is_cuda or not v.is_contiguous():
                    raise ValueError(f"{k} must be a contiguous CUDA tensor")
                _on_current_device(v)
            setattr(o, k, v.data_ptr() if hasattr(v, "data_ptr") else int(v))
            if k == "workspace" and hasattr(v, "numel"):
                o.workspace_bytes = v.numel() * v.element_size()
            if k == "trace" and hasattr(v, "numel"):
                o._trace_words = v.numel() * v.element_size() // 8
        else:
            setattr(o, k, v)
    o._keep = keep   # keep ctypes arrays alive with the struct
    return o


def _check_trace(kind, n_shards, M, K, N, chunk_rows, opts):
    """A trace tensor must hold the call's plan's trace_words: the library
    takes a bare pointer and writes that many words."""
    words = getattr(opts, "_trace_words", None) if opts is not None else None
    if words is None:
        return
    import torch
    cus = torch.cuda.get_device_properties(torch.cuda.current_device()).multi_processor_count
    need = plan(kind, n_shards, M, K, N, chunk_rows, opts, num_cus=cus)[0].trace_words
    if words < need:
        raise ValueError(f"trace holds {words} words; this call's plan needs {need}")


def _stream_handle(stream):
    import torch
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream))


def _on_current_device(*tensors):
    """Every tensor lives on the current device (the library launches there
    and takes the pointers as that device's)."""
    import torch
    cur = torch.cuda.current_device()
    for t in tensors:
        if t is not None and t.device.index != cur:
            raise ValueError(f"tensor on {t.device}, but the current device is cuda:{cur}")


def _shard_ptrs(shards, dtype, K):
    import torch
    if not shards:
        raise ValueError("need at least one shard")
    if len(shards) > MAX_SHARDS:
        raise ValueError(f"at most {MAX_SHARDS} shards")
    S = shards[0].shape[0]
    for t in shards:
        if t.dtype != dtype or not t.is_cuda or not t.is_contiguous() or t.dim() != 2:
            raise ValueError(f"shards must be contiguous 2-D {dtype} CUDA tensors")
        if tuple(t.shape) != (S, K):
            raise ValueError("all shards must be S x K")
    _on_current_device(*shards)
    return (ctypes.c_void_p * len(shards))(*[t.data_ptr() for t in shards]), S


def _check_out(C, shape, dtype):
    if C.dtype != dtype or not C.is_cuda or not C.is_contiguous() or tuple(C.shape) != shape:
        raise ValueError(f"output must be a contiguous {dtype} CUDA tensor of shape {shape}")
    _on_current_device(C)


def _check_vec(v, n, dtype, what):
    """A contiguous (n,) vector of `dtype` on the current device: a strided
    view would be read as if it were contiguous."""
    if v.dtype != dtype or tuple(v.shape) != (n,) or not v.is_cuda or not v.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} CUDA tensor of shape ({n},)")
    _on_current_device(v)


def ag_gemm_f16(shards, B, C, chunk_rows: int = 0, stream=None, opts: Options | None = None,
                prepare: bool = False):
    """C[M, N] (fp32) = concat(shards)[M, K] (fp16) x B[K, N] (fp16).

    With prepare=True nothing runs: the call is returned as a Prepared
    object (arguments checked and marshalled once) to be called later."""
    import torch
    if B.dtype != torch.float16 or not B.is_cuda or not B.is_contiguous() or B.dim() != 2:
        raise ValueError("B must be a contiguous 2-D fp16 CUDA tensor")
    K, N = B.shape
    _on_current_device(B)
    table, S = _shard_ptrs(shards, torch.float16, K)
    M = S * len(shards)
    _check_out(C, (M, N), torch.float32)
    _check_trace("f16", len(shards), M, K, N, int(chunk_rows), opts)
    st = _stream_handle(stream)
    r = _invoke(lib.ag_gemm_f16, lib.ag_gemm_f16_ex,
                (table, len(shards), B.data_ptr(), C.data_ptr(), M, K, N, int(chunk_rows), st),
                opts, "ag_gemm_f16", prepare)
    return r if prepare else C


def ag_gemm_f16_noalloc(shards, B, C, chunk_rows: int = 0, stream=None,
                        opts: Options | None = None, prepare: bool = False):
    """ag_gemm_f16 through the allocation-free entry point: the library's
    fixed per-GPU scratch array is the workspace (opts.workspace must be
    unset); AggError with AGG_E_TOO_LARGE if the call needs more than
    NOALLOC_MAX_BYTES of it."""
    import torch
    if B.dtype != torch.float16 or not B.is_cuda or not B.is_contiguous() or B.dim() != 2:
        raise ValueError("B must be a contiguous 2-D fp16 CUDA tensor")
    K, N = B.shape
    _on_current_device(B)
    table, S = _shard_ptrs(shards, torch.float16, K)
    M = S * len(shards)
    _check_out(C, (M, N), torch.float32)
    _check_trace("f16", len(shards), M, K, N, int(chunk_rows), opts)
    st = _stream_handle(stream)
    args = (table, len(shards), B.data_ptr(), C.data_ptr(), M, K, N, int(chunk_rows), st,
            ctypes.byref(opts) if opts is not None else None)
    if prepare:
        return Prepared(lib.ag_gemm_f16_noalloc, args, "ag_gemm_f16_noalloc", (table, opts))
    _raise(lib.ag_gemm_f16_noalloc(*args), "ag_gemm_f16_noalloc")
    return C


def ag_gemm_bf16(shards, B, C, chunk_rows: int = 0, stream=None, opts: Options | None = None,
                 prepare: bool = False):
    """C[M, N] (fp32) = concat(shards)[M, K] (bf16) x B[K, N] (bf16)."""
    import torch
    if B.dtype != torch.bfloat16 or not B.is_cuda or not B.is_contiguous() or B.dim() != 2:
        raise ValueError("B must be a contiguous 2-D bf16 CUDA tensor")
    K, N = B.shape
    _on_current_device(B)
    table, S = _shard_ptrs(shards, torch.bfloat16, K)
    M = S * len(shards)
    _check_out(C, (M, N), torch.float32)
    _check_trace("bf16", len(shards), M, K, N, int(chunk_rows), opts)
    st = _stream_handle(stream)
    r = _invoke(lib.ag_gemm_bf16, lib.ag_gemm_bf16_ex,
                (table, len(shards), B.data_ptr(), C.data_ptr(), M, K, N, int(chunk_rows), st),
                opts, "ag_gemm_bf16", prepare)
    return r if prepare else C


def _fp8_dtypes():
    import torch
    return (torch.uint8, torch.float8_e4m3fn)


def ag_gemm_fp8(shards, B, C, chunk_rows: int = 0, stream=None, opts: Options | None = None,
                prepare: bool = False):
    """C[M, N] (fp32) = concat(shards)[M, K] (fp8 E4M3) x B[K, N] (fp8 E4M3).

    Shards and B are torch.float8_e4m3fn tensors, or uint8 tensors holding
    E4M3 bit patterns (all of one dtype)."""
    import torch
    dt = B.dtype
    if dt not in _fp8_dtypes() or not B.is_cuda or not B.is_contiguous() or B.dim() != 2:
        raise ValueError("B must be a contiguous 2-D float8_e4m3fn (or uint8) CUDA tensor")
    K, N = B.shape
    _on_current_device(B)
    table, S = _shard_ptrs(shards, dt, K)
    M = S * len(shards)
    _check_out(C, (M, N), torch.float32)
    _check_trace("fp8", len(shards), M, K, N, int(chunk_rows), opts)
    st = _stream_handle(stream)
    r = _invoke(lib.ag_gemm_fp8, lib.ag_gemm_fp8_ex,
                (table, len(shards), B.data_ptr(), C.data_ptr(), M, K, N, int(chunk_rows), st),
                opts, "ag_gemm_fp8", prepare)
    return r if prepare else C


def ag_gemm_i8_dequant(shards, B, bias, scale, C, chunk_rows: int = 0, stream=None,
                       opts: Options | None = None, prepare: bool = False):
    """C[M, N] (fp16) = fp16(fp32(concat(shards) x B + bias) * scale)."""
    import torch
    if B.dtype != torch.int8 or not B.is_cuda or not B.is_contiguous() or B.dim() != 2:
        raise ValueError("B must be a contiguous 2-D int8 CUDA tensor")
    K, N = B.shape
    _on_current_device(B)
    table, S = _shard_ptrs(shards, torch.int8, K)
    M = S * len(shards)
    _check_vec(bias, N, torch.int32, "bias")
    _check_vec(scale, N, torch.float32, "scale")
    _check_out(C, (M, N), torch.float16)
    _check_trace("i8", len(shards), M, K, N, int(chunk_rows), opts)
    st = _stream_handle(stream)
    r = _invoke(lib.ag_gemm_i8_dequant, lib.ag_gemm_i8_dequant_ex,
                (table, len(shards), B.data_ptr(), bias.data_ptr(), scale.data_ptr(),
                 C.data_ptr(), M, K, N, int(chunk_rows), st),
                opts, "ag_gemm_i8_dequant", prepare)
    return r if prepare else C


# ---- products of rows grouped by expert ----------------------------------
#
# A small call's kernel takes a few microseconds, and so do its checks here:
# they are written to cost little where they pass.

import torch  # noqa: E402  (after the library's own order of loading, see _load)

_CODES = {torch.float16: TYPE_F16, torch.bfloat16: TYPE_BF16, torch.float32: TYPE_F32,
          torch.float8_e4m3fn: TYPE_FP8, torch.uint8: TYPE_FP8}
_IN16 = (TYPE_F16, TYPE_BF16)
_OUT = (TYPE_F16, TYPE_BF16, TYPE_F32)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _type_of(t, allowed, what):
    code = _CODES.get(t.dtype)
    if code not in allowed:
        raise ValueError(f"{what} cannot be {t.dtype}")
    return code


def _device():
    """The current device; -2, which no tensor is on, where there is none."""
    return _get_device() if torch.cuda.is_initialized() else -2


def _stream(stream, dev):
    if stream is None and _raw_stream is not None and dev >= 0:
        return _raw_stream(dev)
    return _stream_handle(stream)


def _refuse(t, shape, what):
    if not t.is_cuda or tuple(t.shape) != shape:
        raise ValueError(f"{what} must be a CUDA tensor of shape {shape}")
    _on_current_device(t)
    raise ValueError(f"{what} must have unit column stride and rows that do not overlap")


def _matrix(t, m, n, dev, what):
    """Row stride of a CUDA matrix [m, n] with unit column stride on device dev
    (n for a single row, whose own stride says nothing)."""
    if t.shape != (m, n) or t.get_device() != dev:
        _refuse(t, (m, n), what)
    if t.is_contiguous():
        return n
    ld, unit = t.stride()
    if (unit != 1 and n > 1) or (ld < n and m > 1):
        _refuse(t, (m, n), what)
    return ld if m > 1 else n


def _matrices(t, e, m, n, dev, what):
    """Row and matrix strides of a stack [e, m, n] of such matrices."""
    if t.shape != (e, m, n) or t.get_device() != dev:
        _refuse(t, (e, m, n), what)
    step, ld, unit = t.stride()
    if (unit != 1 and n > 1) or (ld < n and m > 1):
        _refuse(t, (e, m, n), what)
    return (ld if m > 1 else n), (step if e > 1 else 0)


def _check_offsets(offsets, groups, dev):
    if (offsets.dtype != torch.int32 or offsets.shape != (groups + 1,) or
            offsets.get_device() != dev or not offsets.is_contiguous()):
        raise ValueError(f"offsets must be a contiguous int32 CUDA tensor of {groups + 1} values "
                         "on the current device")


class _Following(Prepared):
    """A prepared call that runs on whichever stream of its device is current
    when it is called."""

    __slots__ = ("_dev",)

    def __init__(self, fn, args, what, dev):
        super().__init__(fn, args, what, args)
        self._dev = dev

    def __call__(self):
        rc = self._fn(*self._args, _stream(None, self._dev))
        if rc:
            raise AggError(rc, self._what)


def _call(fn, args, stream, dev, what, out, prepare):
    """fn(*args, stream), or the prepared call: on `stream`, or without one on
    the stream that is current when it is called."""
    if prepare:
        if stream is None:
            return _Following(fn, args, what, dev)
        args = (*args, _stream(stream, dev))
        return Prepared(fn, args, what, args)
    rc = fn(*args, _stream(stream, dev))
    if rc:
        raise AggError(rc, what)
    return out


def ag_gemm_grouped(x, w, offsets, y, trans_w: bool = False, stream=None, prepare: bool = False):
    """y[T, N] = x[T, K] (fp16 or bf16) times each row's group's weights.

    Group e holds rows offsets[e] .. offsets[e + 1]; w is [E, K, N], or with
    trans_w [E, N, K].  y has x's type or fp32.  Rows of no group are not
    written.  Matrices may have any row and group stride."""
    typ = _type_of(x, _IN16, "x")
    out = _type_of(y, (typ, TYPE_F32), "y")
    if w.dim() != 3 or w.dtype != x.dtype or x.dim() != 2:
        raise ValueError("x must be [T, K] and w [E, K, N] (or [E, N, K]) of one type")
    dev = _device()
    T, K = x.shape
    E, N = w.shape[0], w.shape[1 if trans_w else 2]
    ldx = _matrix(x, T, K, dev, "x")
    ldw, w_stride = _matrices(w, E, N, K, dev, "w") if trans_w else _matrices(w, E, K, N, dev, "w")
    ldy = _matrix(y, T, N, dev, "y")
    _check_offsets(offsets, E, dev)
    args = (typ, x.data_ptr(), ldx, w.data_ptr(), ldw, w_stride, 1 if trans_w else 0,
            offsets.data_ptr(), E, y.data_ptr(), ldy, out, T, K, N)
    return _call(lib.ag_gemm_grouped, args, stream, dev, "ag_gemm_grouped", y, prepare)


def ag_gemm_grouped_wgrad(x, dy, offsets, dw, stream=None, prepare: bool = False):
    """dw[E, K, N] = x[rows of e]^T dy[rows of e] for every group (zeros for
    an empty one); x [T, K] and dy [T, N] fp16 or bf16, dw their type or fp32."""
    typ = _type_of(x, _IN16, "x")
    out = _type_of(dw, (typ, TYPE_F32), "dw")
    if x.dim() != 2 or dy.dim() != 2 or dw.dim() != 3 or dy.dtype != x.dtype:
        raise ValueError("x must be [T, K], dy [T, N] of one type and dw [E, K, N]")
    dev = _device()
    (T, K), N, E = x.shape, dy.shape[1], dw.shape[0]
    ldx, lddy = _matrix(x, T, K, dev, "x"), _matrix(dy, T, N, dev, "dy")
    lddw, dw_stride = _matrices(dw, E, K, N, dev, "dw")
    _check_offsets(offsets, E, dev)
    args = (typ, x.data_ptr(), ldx, dy.data_ptr(), lddy, offsets.data_ptr(), E, dw.data_ptr(),
            lddw, dw_stride, out, T, K, N)
    return _call(lib.ag_gemm_grouped_wgrad, args, stream, dev, "ag_gemm_grouped_wgrad", dw, prepare)


def _fp8_operands(a, a_scale, b, b_scale, c, dev):
    _type_of(a, (TYPE_FP8,), "a")
    _type_of(b, (TYPE_FP8,), "b")
    out = _type_of(c, _OUT, "c")
    if a.dim() != 2 or a_scale.dtype != torch.float32 or b_scale.dtype != torch.float32:
        raise ValueError("a must be [M, K] and the scales fp32")
    M, K = a.shape
    N = b.shape[-2]
    kb, nb = -(-K // SCALE_BLOCK), -(-N // SCALE_BLOCK)
    return (out, M, K, N, kb, nb, _matrix(a, M, K, dev, "a"),
            _matrix(a_scale, M, kb, dev, "a_scale"), _matrix(c, M, N, dev, "c"))


def ag_gemm_fp8_block(a, a_scale, b, b_scale, c, stream=None, prepare: bool = False):
    """c[M, N] = (a * a_scale) (b * b_scale)^T: a [M, K] and b [N, K] E4M3
    (float8_e4m3fn, or uint8 bit patterns), a_scale fp32 [M, ceil(K / 128)],
    b_scale fp32 [ceil(N / 128), ceil(K / 128)], c fp16, bf16 or fp32."""
    if b.dim() != 2:
        raise ValueError("b must be [N, K]")
    dev = _device()
    out, M, K, N, kb, nb, lda, ldas, ldc = _fp8_operands(a, a_scale, b, b_scale, c, dev)
    ldb, ldbs = _matrix(b, N, K, dev, "b"), _matrix(b_scale, nb, kb, dev, "b_scale")
    args = (a.data_ptr(), lda, a_scale.data_ptr(), ldas, b.data_ptr(), ldb, b_scale.data_ptr(),
            ldbs, c.data_ptr(), ldc, out, M, K, N)
    return _call(lib.ag_gemm_fp8_block, args, stream, dev, "ag_gemm_fp8_block", c, prepare)


def ag_gemm_grouped_fp8_block(a, a_scale, b, b_scale, offsets, c, stream=None,
                              prepare: bool = False):
    """ag_gemm_fp8_block with b [E, N, K] and b_scale [E, ceil(N / 128),
    ceil(K / 128)] chosen by each row's group (see ag_gemm_grouped)."""
    if b.dim() != 3 or b_scale.dim() != 3:
        raise ValueError("b must be [E, N, K] and b_scale one matrix for each")
    dev = _device()
    out, M, K, N, kb, nb, lda, ldas, ldc = _fp8_operands(a, a_scale, b, b_scale, c, dev)
    E = b.shape[0]
    ldb, b_step = _matrices(b, E, N, K, dev, "b")
    ldbs, bs_step = _matrices(b_scale, E, nb, kb, dev, "b_scale")
    _check_offsets(offsets, E, dev)
    args = (a.data_ptr(), lda, a_scale.data_ptr(), ldas, b.data_ptr(), ldb, b_step,
            b_scale.data_ptr(), ldbs, bs_step, offsets.data_ptr(), E, c.data_ptr(), ldc, out, M, K,
            N)
    return _call(lib.ag_gemm_grouped_fp8_block, args, stream, dev, "ag_gemm_grouped_fp8_block", c, prepare)


def ag_gemm_quant_fp8_block(x, q, scale, block_rows: int = 1, stream=None, prepare: bool = False):
    """E4M3 codes q [M, K] and fp32 scales of x [M, K] (fp16, bf16 or fp32):
    blocks of 1 x 128 (block_rows 1) or 128 x 128 (block_rows 128)."""
    typ = _type_of(x, _OUT, "x")
    _type_of(q, (TYPE_FP8,), "q")
    if x.dim() != 2 or scale.dtype != torch.float32 or block_rows not in (1, SCALE_BLOCK):
        raise ValueError("x must be [M, K], scale fp32 and block_rows 1 or 128")
    dev = _device()
    M, K = x.shape
    ldx, ldq = _matrix(x, M, K, dev, "x"), _matrix(q, M, K, dev, "q")
    lds = _matrix(scale, -(-M // block_rows), -(-K // SCALE_BLOCK), dev, "scale")
    args = (typ, x.data_ptr(), ldx, q.data_ptr(), ldq, scale.data_ptr(), lds, block_rows, M, K)
    return _call(lib.ag_gemm_quant_fp8_block, args, stream, dev, "ag_gemm_quant_fp8_block", (q, scale), prepare)


# ---- around the products: sorting by expert and back, norm ----------------

_ROWS = (TYPE_F16, TYPE_BF16, TYPE_F32)
_BYTES = (torch.uint8, getattr(torch, "float4_e2m1fn_x2", torch.uint8))
_EXPONENTS = (torch.uint8, getattr(torch, "float8_e8m0fnu", torch.uint8))


def _same(t, like, what):
    if t.dtype != like.dtype:
        raise ValueError(f"{what} must be {like.dtype}, not {t.dtype}")


def _dense(t, shape, dtype, dev, what):
    """The address of a contiguous CUDA tensor."""
    if t.dtype != dtype or t.shape != shape or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"{what} must be a contiguous {dtype} CUDA tensor of shape {tuple(shape)} "
                         "on the current device")
    return t.data_ptr()


def _workspace(t, need, dev):
    """Address and bytes of a workspace that a call needs `need` bytes of."""
    if not need:
        return None, 0
    if t is None or t.get_device() != dev or not t.is_contiguous():
        raise ValueError(f"the workspace must be a contiguous CUDA tensor of {need} bytes on the "
                         "current device")
    return t.data_ptr(), t.numel() * t.element_size()


def _optional(t, m, n, dev, what):
    """Address and row stride of a matrix that may be absent."""
    return (None, n) if t is None else (t.data_ptr(), _matrix(t, m, n, dev, what))


def expert_sort_workspace_bytes(tokens: int, top: int, experts: int) -> int:
    """Bytes of workspace that ag_gemm_expert_sort needs for these sizes."""
    return lib.ag_gemm_expert_sort_workspace_bytes(int(tokens), int(top), int(experts))


def ag_gemm_expert_sort(ids, experts: int, offsets, place, workspace=None, stream=None,
                        prepare: bool = False):
    """offsets (int32 [experts + 1]) and place (int32 [T, top]) of ids [T, top]
    (int32 or int64): a stable sort by expert; ids outside [0, experts) get no
    place (-1).  workspace: expert_sort_workspace_bytes() bytes where that is
    not zero."""
    if ids.dim() != 2 or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be [T, top], int32 or int64")
    dev = _device()
    T, top = ids.shape
    ldi = _matrix(ids, T, top, dev, "ids")
    _check_offsets(offsets, experts, dev)
    at = _dense(place, ids.shape, torch.int32, dev, "place")
    ws, size = _workspace(workspace, lib.ag_gemm_expert_sort_workspace_bytes(T, top, experts), dev)
    args = (ids.data_ptr(), ids.element_size(), ldi, T, top, experts, offsets.data_ptr(), at, ws, size)
    return _call(lib.ag_gemm_expert_sort, args, stream, dev, "ag_gemm_expert_sort", (offsets, place), prepare)


def ag_gemm_expert_dispatch(x, place, xs, stream=None, prepare: bool = False):
    """xs[place[t, j]] = x[t]: x [T, K] and xs [rows, K] of one type (fp16, bf16,
    fp32, or codes of one byte), place int32 [T, top].  Rows that no place names
    are not written."""
    typ = _type_of(x, (*_ROWS, TYPE_FP8), "x")
    if x.dim() != 2 or xs.dim() != 2 or place.dim() != 2:
        raise ValueError("x must be [T, K], place [T, top] and xs [rows, K]")
    _same(xs, x, "xs")
    dev = _device()
    (T, K), top, rows = x.shape, place.shape[1], xs.shape[0]
    ldx, ldxs = _matrix(x, T, K, dev, "x"), _matrix(xs, rows, K, dev, "xs")
    at = _dense(place, (T, top), torch.int32, dev, "place")
    args = (typ, x.data_ptr(), ldx, at, top, xs.data_ptr(), ldxs, rows, T, K)
    return _call(lib.ag_gemm_expert_dispatch, args, stream, dev, "ag_gemm_expert_dispatch", xs, prepare)


def ag_gemm_expert_combine(h, place, weights, y, stream=None, prepare: bool = False):
    """y[t] = sum over j of weights[t, j] * h[place[t, j]]: h [rows, K] fp16, bf16
    or fp32, weights fp32 [T, top] or None (ones), y [T, K] of h's type or fp32."""
    typ = _type_of(h, _ROWS, "h")
    out = _type_of(y, (typ, TYPE_F32), "y")
    if h.dim() != 2 or y.dim() != 2 or place.dim() != 2:
        raise ValueError("h must be [rows, K], place [T, top] and y [T, K]")
    if weights is not None and weights.dtype != torch.float32:
        raise ValueError("weights must be fp32")
    dev = _device()
    (rows, K), (T, top) = h.shape, place.shape
    ldh, ldy = _matrix(h, rows, K, dev, "h"), _matrix(y, T, K, dev, "y")
    at = _dense(place, (T, top), torch.int32, dev, "place")
    w, ldw = _optional(weights, T, top, dev, "weights")
    args = (typ, h.data_ptr(), ldh, rows, at, top, w, ldw, y.data_ptr(), ldy, out, T, K)
    return _call(lib.ag_gemm_expert_combine, args, stream, dev, "ag_gemm_expert_combine", y, prepare)


def ag_gemm_expert_combine_grad(dy, h, place, weights, dh=None, dweights=None, stream=None,
                                prepare: bool = False):
    """dh[place[t, j]] = weights[t, j] * dy[t] and dweights[t, j] = <dy[t],
    h[place[t, j]]> (either may be None): dy [T, K], h and dh [rows, K] of one
    type, weights and dweights fp32 [T, top].  Rows of dh that no place names
    are not written."""
    typ = _type_of(dy, _ROWS, "dy")
    if dh is None and dweights is None:
        raise ValueError("one of dh and dweights is wanted")
    if dy.dim() != 2 or h.dim() != 2 or place.dim() != 2:
        raise ValueError("dy must be [T, K], h [rows, K] and place [T, top]")
    _same(h, dy, "h")
    if dh is not None:
        _same(dh, dy, "dh")
    if weights.dtype != torch.float32 or (dweights is not None and dweights.dtype != torch.float32):
        raise ValueError("weights and dweights must be fp32")
    dev = _device()
    (rows, K), (T, top) = h.shape, place.shape
    lddy, ldh = _matrix(dy, T, K, dev, "dy"), _matrix(h, rows, K, dev, "h")
    at = _dense(place, (T, top), torch.int32, dev, "place")
    ldw = _matrix(weights, T, top, dev, "weights")
    to, lddh = _optional(dh, rows, K, dev, "dh")
    dw, lddw = _optional(dweights, T, top, dev, "dweights")
    args = (typ, dy.data_ptr(), lddy, h.data_ptr(), ldh, rows, at, top, weights.data_ptr(), ldw, to, lddh, dw,
            lddw, T, K)
    return _call(lib.ag_gemm_expert_combine_grad, args, stream, dev, "ag_gemm_expert_combine_grad",
                 (dh, dweights), prepare)


def ag_gemm_rmsnorm(x, weight=None, y=None, q=None, scale=None, residual=None, h=None, rstd=None,
                    eps: float = 1e-6, stream=None, prepare: bool = False):
    """h = x + residual (rounded); y = h / sqrt(mean(h^2) + eps) * weight.

    x, residual, h and y [T, K] and weight [K] of one type (fp16, bf16 or
    fp32); q E4M3 [T, K] with scale fp32 [T, ceil(K / 128)] are y's codes; rstd
    fp32 [T].  Only what is given is written (y or q at least); h may be x or
    the residual itself."""
    typ = _type_of(x, _ROWS, "x")
    if x.dim() != 2 or (y is None and q is None) or (q is None) != (scale is None):
        raise ValueError("x must be [T, K], and y, or q and its scale, are wanted")
    for t, what in ((residual, "residual"), (weight, "weight"), (h, "h"), (y, "y")):
        if t is not None:
            _same(t, x, what)
    dev = _device()
    T, K = x.shape
    ldx = _matrix(x, T, K, dev, "x")
    res, ldr = _optional(residual, T, K, dev, "residual")
    w = None if weight is None else _dense(weight, (K,), x.dtype, dev, "weight")
    hp, ldh = _optional(h, T, K, dev, "h")
    yp, ldy = _optional(y, T, K, dev, "y")
    qp, ldq, sp, lds = None, K, None, 1
    if q is not None:
        _type_of(q, (TYPE_FP8,), "q")
        if scale.dtype != torch.float32:
            raise ValueError("scale must be fp32")
        qp, ldq = q.data_ptr(), _matrix(q, T, K, dev, "q")
        sp, lds = scale.data_ptr(), _matrix(scale, T, -(-K // SCALE_BLOCK), dev, "scale")
    rs = None if rstd is None else _dense(rstd, (T,), torch.float32, dev, "rstd")
    args = (typ, x.data_ptr(), ldx, res, ldr, w, hp, ldh, yp, ldy, qp, ldq, sp, lds, rs, eps, T, K)
    return _call(lib.ag_gemm_rmsnorm, args, stream, dev, "ag_gemm_rmsnorm", y if q is None else (q, scale),
                 prepare)


def rmsnorm_grad_workspace_bytes(rows: int, k: int) -> int:
    """Bytes of workspace that the weight's gradient needs for these sizes."""
    return lib.ag_gemm_rmsnorm_grad_workspace_bytes(int(rows), int(k))


def ag_gemm_rmsnorm_grad(dy, h, weight, rstd, dx, dweight=None, workspace=None, dh=None, stream=None,
                         prepare: bool = False):
    """dx of ag_gemm_rmsnorm (x's gradient and the residual's) from dy and, added
    to it, the gradient dh of h: all [T, K] of one type, weight [K] of it or
    None, rstd fp32 [T].  dweight [K] of that type or fp32 needs a workspace of
    rmsnorm_grad_workspace_bytes() bytes."""
    typ = _type_of(dy, _ROWS, "dy")
    if dy.dim() != 2:
        raise ValueError("dy must be [T, K]")
    for t, what in ((h, "h"), (weight, "weight"), (dh, "dh"), (dx, "dx")):
        if t is not None:
            _same(t, dy, what)
    dev = _device()
    T, K = dy.shape
    lddy, ldh, lddx = (_matrix(t, T, K, dev, n) for t, n in ((dy, "dy"), (h, "h"), (dx, "dx")))
    w = None if weight is None else _dense(weight, (K,), dy.dtype, dev, "weight")
    rs = _dense(rstd, (T,), torch.float32, dev, "rstd")
    dhp, lddh = _optional(dh, T, K, dev, "dh")
    dw = ws = None
    dw_type, size = typ, 0
    if dweight is not None:
        dw_type = _type_of(dweight, (typ, TYPE_F32), "dweight")
        dw = _dense(dweight, (K,), dweight.dtype, dev, "dweight")
        ws, size = _workspace(workspace, lib.ag_gemm_rmsnorm_grad_workspace_bytes(T, K), dev)
    args = (typ, dy.data_ptr(), lddy, h.data_ptr(), ldh, w, rs, dhp, lddh, dx.data_ptr(), lddx, dw, dw_type, ws,
            size, T, K)
    return _call(lib.ag_gemm_rmsnorm_grad, args, stream, dev, "ag_gemm_rmsnorm_grad", (dx, dweight), prepare)


# ---- microscaled 4-bit values ---------------------------------------------


def _codes(q, scale, what):
    """Checks the types of E2M1 codes (two a byte) and E8M0 scales."""
    if q.dtype not in _BYTES or scale.dtype not in _EXPONENTS:
        raise ValueError(f"{what} must be uint8 or float4_e2m1fn_x2 and its scales uint8 or float8_e8m0fnu")


def _mx_matrix(t, q, scale, what):
    """Type code and sizes of the matrix t [M, K] whose codes and scales are q
    and scale, and the addresses and row strides of the three."""
    typ = _type_of(t, _ROWS, what)
    _codes(q, scale, "q")
    shape = t.shape
    if len(shape) != 2 or shape[1] & 1:
        raise ValueError(f"{what} must be [M, K] with K even")
    dev = _device()
    M, K = shape
    return (typ, M, K, dev, (t.data_ptr(), _matrix(t, M, K, dev, what)),
            (q.data_ptr(), _matrix(q, M, K // 2, dev, "q"), scale.data_ptr(),
             _matrix(scale, M, -(-K // MX_BLOCK), dev, "scale")))


def ag_gemm_quant_mxfp4(x, q, scale, stream=None, prepare: bool = False):
    """E2M1 codes q [M, K / 2] (two a byte, the even column in the low half;
    uint8 or float4_e2m1fn_x2) and E8M0 scales [M, ceil(K / 32)] (uint8 or
    float8_e8m0fnu) of x [M, K] (fp16, bf16 or fp32, K even)."""
    typ, M, K, dev, matrix, codes = _mx_matrix(x, q, scale, "x")
    return _call(lib.ag_gemm_quant_mxfp4, (typ, *matrix, *codes, M, K), stream, dev, "ag_gemm_quant_mxfp4",
                 (q, scale), prepare)


def ag_gemm_dequant_mxfp4(q, scale, y, stream=None, prepare: bool = False):
    """y [M, K] (fp16, bf16 or fp32) = the values of codes q and their scales."""
    typ, M, K, dev, matrix, codes = _mx_matrix(y, q, scale, "y")
    return _call(lib.ag_gemm_dequant_mxfp4, (*codes, *matrix, typ, M, K), stream, dev, "ag_gemm_dequant_mxfp4", y,
                 prepare)


def _mx_operands(a, a_scale, b, b_scale, c, dev):
    out = _type_of(c, _OUT, "c")
    _codes(a, a_scale, "a")
    _codes(b, b_scale, "b")
    if a.dim() != 2:
        raise ValueError("a must be [M, K / 2]")
    (M, half), N = a.shape, b.shape[-2]
    K = 2 * half
    kb = -(-K // MX_BLOCK)
    return (out, M, K, N, kb, _matrix(a, M, half, dev, "a"), _matrix(a_scale, M, kb, dev, "a_scale"),
            _matrix(c, M, N, dev, "c"))


def ag_gemm_mxfp4(a, a_scale, b, b_scale, c, stream=None, prepare: bool = False):
    """c[M, N] = a b^T of E2M1 codes a [M, K / 2] and b [N, K / 2] with E8M0
    scales [M, ceil(K / 32)] and [N, ceil(K / 32)] (see ag_gemm_quant_mxfp4); c
    fp16, bf16 or fp32."""
    if b.dim() != 2:
        raise ValueError("b must be [N, K / 2]")
    dev = _device()
    out, M, K, N, kb, lda, ldas, ldc = _mx_operands(a, a_scale, b, b_scale, c, dev)
    ldb, ldbs = _matrix(b, N, K // 2, dev, "b"), _matrix(b_scale, N, kb, dev, "b_scale")
    args = (a.data_ptr(), lda, a_scale.data_ptr(), ldas, b.data_ptr(), ldb, b_scale.data_ptr(), ldbs, c.data_ptr(),
            ldc, out, M, K, N)
    return _call(lib.ag_gemm_mxfp4, args, stream, dev, "ag_gemm_mxfp4", c, prepare)


def ag_gemm_grouped_mxfp4(a, a_scale, b, b_scale, offsets, c, stream=None, prepare: bool = False):
    """ag_gemm_mxfp4 with b [E, N, K / 2] and b_scale [E, N, ceil(K / 32)] chosen
    by each row's group (see ag_gemm_grouped)."""
    if b.dim() != 3 or b_scale.dim() != 3:
        raise ValueError("b must be [E, N, K / 2] and b_scale one matrix for each")
    dev = _device()
    out, M, K, N, kb, lda, ldas, ldc = _mx_operands(a, a_scale, b, b_scale, c, dev)
    E = b.shape[0]
    ldb, b_step = _matrices(b, E, N, K // 2, dev, "b")
    ldbs, bs_step = _matrices(b_scale, E, N, kb, dev, "b_scale")
    _check_offsets(offsets, E, dev)
    args = (a.data_ptr(), lda, a_scale.data_ptr(), ldas, b.data_ptr(), ldb, b_step, b_scale.data_ptr(), ldbs,
            bs_step, offsets.data_ptr(), E, c.data_ptr(), ldc, out, M, K, N)
    return _call(lib.ag_gemm_grouped_mxfp4, args, stream, dev, "ag_gemm_grouped_mxfp4", c, prepare)


def pick_chunk_rows(shard_rows: int) -> int:
    return lib.ag_gemm_pick_chunk_rows(int(shard_rows))


def workspace_bytes(n_shards: int, M: int, K: int, elt_bytes: int) -> int:
    return lib.ag_gemm_workspace_bytes(int(n_shards), int(M), int(K), int(elt_bytes))


def workspace_reset(ws, stream=None):
    rc = lib.ag_gemm_workspace_reset(ctypes.c_void_p(ws.data_ptr()),
                                     ws.numel() * ws.element_size(), _stream_handle(stream))
    _raise(rc, "ag_gemm_workspace_reset")


def check(stream=None) -> int:
    """Synchronise and return the status of the calls since the last check."""
    return lib.ag_gemm_check(_stream_handle(stream))


def release():
    lib.ag_gemm_release()


def plan(kind: str, n_shards: int, M: int, K: int, N: int, chunk_rows: int = 0,
         opts: Options | None = None, num_cus: int = 256, orders: bool = False):
    """Host-only schedule query: (PlanInfo, tile_order or None, chunk_order or None)."""
    import numpy as np
    info = PlanInfo()
    k = {"f16": 0, "i8": 1, "bf16": 2, "fp8": 3}[kind]
    o = ctypes.byref(opts) if opts is not None else None
    rc = lib.ag_gemm_plan(k, n_shards, M, K, N, chunk_rows, o, num_cus, ctypes.byref(info),
                          None, None)
    _raise(rc, "ag_gemm_plan")
    if not orders:
        return info, None, None
    tiles = np.zeros((info.total_tiles, 4), np.int32)
    chunks = np.zeros((max(info.total_chunks, 0), 2), np.int32)
    rc = lib.ag_gemm_plan(k, n_shards, M, K, N, chunk_rows, o, num_cus, ctypes.byref(info),
                          tiles.ctypes.data, chunks.ctypes.data if chunks.size else None)
    _raise(rc, "ag_gemm_plan")
    return info, tiles, chunks
