"""ctypes binding of the C ABI declared in ``include/pda.h``.

Argument marshalling only: tensors become device pointers and sizes, and
every step of the computation runs in the library's CUDA kernels. The shared
library ``libpda.so`` is built in-tree (``paged_kv_decode_pda_gb300.build``);
if it is missing the first call raises ``PdaError`` -- there is no fallback.
"""

from __future__ import annotations

import ctypes
import os
import threading

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libpda.so")

PDA_OK = 0
PDA_ERR_INVALID_ARG = 1
PDA_ERR_UNSUPPORTED = 2
PDA_ERR_WORKSPACE = 3
PDA_ERR_CUDA = 4
PDA_ERR_DEVICE_TIMEOUT = 5
PDA_ERR_NOALLOC_CAPACITY = 6

PDA_ROPE_PLAIN, PDA_ROPE_LINEAR, PDA_ROPE_BASE, PDA_ROPE_RAMP, PDA_ROPE_BANDS = range(5)


class _RopeHeads(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("src_token", ctypes.c_longlong),
                ("src_head", ctypes.c_longlong), ("dst_token", ctypes.c_longlong), ("dst_head", ctypes.c_longlong),
                ("num_heads", ctypes.c_int)]


class _TokenRows(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("token", ctypes.c_longlong), ("head", ctypes.c_longlong)]


class _PageTable(ctypes.Structure):
    _fields_ = [("ref_counts", ctypes.c_void_p), ("block_tables", ctypes.c_void_p), ("seq_lens", ctypes.c_void_p),
                ("num_blocks", ctypes.c_longlong), ("num_rows", ctypes.c_int), ("max_blocks", ctypes.c_int),
                ("block_size", ctypes.c_int)]


class _PageArray(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("bytes_per_block", ctypes.c_longlong)]


# Functions (name -> (restype, argtypes)) the header declares.
_P, _I, _F, _D = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_double
SIGNATURES = {
    "pda_decode": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _F, _F, _P]),
    "pda_status_string": (ctypes.c_char_p, [_I]),
    "pda_choose_splits": (_I, [_I, _I, _I, _I, _I, _I]),
    "pda_plan_splits": (_I, [_I, _I, _I, _I, _I]),
    "pda_plan_kernel": (_I, [_I, _I, _I, _I, _I]),
    "pda_plan_launches": (_I, [_I, _I, _I, _I, _I]),
    "pda_plan_slot_scales": (_I, [_I, _I, _I, _I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "pda_tail_pieces": (_I, [_I, _I, _I, _I, ctypes.POINTER(_I), _I]),
    "pda_choose_kernel": (_I, [_I, _I, _I, _I, _I, _I, _I, ctypes.POINTER(_I), ctypes.POINTER(_I)]),
    "pda_set_split_override": (None, [_I]),
    "pda_set_tail_split": (None, [_I]),
    "pda_set_tma_gather": (None, [_I]),
    "pda_set_block_check": (None, [ctypes.c_longlong]),
    "pda_reserve": (_I, [_I, _I, _I, _I, _I, _P]),
    "pda_release": (_I, []),
    "pda_workspace_info": (_I, [_P, ctypes.POINTER(ctypes.c_longlong), ctypes.POINTER(_I)]),
    "pda_query_device_status": (_I, [_P, ctypes.POINTER(ctypes.c_int)]),
    "pda_set_profile_events": (None, [_P, _P]),
    "pda_test_bounded_wait": (_I, [_I, _P]),
    "pda_reshape_and_cache": (_I, [_P, _P, _P, _P, _P, _I, _I, _I, _I, ctypes.c_longlong, _F, _F, _I, _P]),
    "pda_decode_slot_scales": (_I, [_P, _P, _P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _P]),
    "pda_decode_noalloc": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _F, _F, _P]),
    "pda_decode_host": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, ctypes.c_longlong, _F, _F, _F, _P]),
    "pda_decode_ex": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I, _F, _F, _F, _I, _P, _I, _F, _P]),
    "pda_decode_strided": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, _I, _I, _I] + [ctypes.c_longlong] * 7
                           + [_F, _F, _F, _P]),
    "pda_rope": (_I, [_P, _P, _P, _I, _I, _P, _I, _I, _F, _P]),
    "pda_rope_and_cache": (_I, [_P, _P, _P, _P, _P, _I, _I, _P, _I, _I, _F, _P, _P, _I, ctypes.c_longlong, _F, _F, _I,
                                _P]),
    "pda_rope_frequencies": (_I, [_P, _P, _I, _D, _I, _D, _D, _D, _D]),
    "pda_extend": (_I, [_P] * 7 + [_I] * 7 + [_F, _F, _F, _I, _I, _P, _I, _F, _P]),
    "pda_reserve_extend": (_I, [_I, _I, _I, _I, _I, _I, _P]),
    "pda_copy_pages": (_I, [_P, _I, _P, _P, _I, ctypes.c_longlong, _P]),
    "pda_grow_pages": (_I, [_P, _P, _P, _I, _P]),
    "pda_fork_pages": (_I, [_P, _P, _P, _I, _P, _I, _P]),
    "pda_free_pages": (_I, [_P, _P, _I, _P]),
    "pda_compact_pages": (_I, [_P, _P, _I, _P, _P]),
    "pda_reshape_and_cache_slot_scales": (_I, [_P] * 7 + [_I, _I, _I, _I, ctypes.c_longlong, _F, _P]),
    "pda_reshape_and_cache_fp4": (_I, [_P] * 4 + [_I, _I, _I, _I, ctypes.c_longlong, _F, _F, _P]),
    "pda_gather_cache": (_I, [_P] * 7 + [_I] * 6 + [ctypes.c_longlong, _F, _F, _I, _P]),
    "pda_gather_cache_slot_scales": (_I, [_P] * 9 + [_I] * 6 + [ctypes.c_longlong, _P]),
    "pda_gather_cache_fp4": (_I, [_P] * 6 + [_I] * 6 + [ctypes.c_longlong, _F, _F, _P]),
    "pda_decode_fp4": (_I, [_P] * 5 + [_I] * 6 + [ctypes.c_longlong, _F, _F, _F, _I, _P, _I, _F, _P]),
    "pda_reserve_fp4": (_I, [_P]),
    "pda_reserve_pages": (_I, [ctypes.c_longlong, _I, _I, _P]),
}

PDA_OUT_BF16 = 0
PDA_OUT_E4M3 = 1
PDA_KV_NATIVE = 0
PDA_KV_SHUFFLED_V = 1

_lock = threading.RLock()
_lib = None


class PdaError(RuntimeError):
    def __init__(self, status: int, what: str = ""):
        self.status = status
        super().__init__("%s: %s (status %d)" % (what or "pda", status_string(status), status))


def load(path: str | None = None):
    """Load libpda.so (once) and bind every declared entry point."""
    global _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise PdaError(PDA_ERR_CUDA, "libpda.so not built at %s (run paged_kv_decode_pda_gb300.build.build())" % p)
        lib = ctypes.CDLL(p)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        if path is None:
            _lib = lib
        return lib


def status_string(status: int) -> str:
    if _lib is None:
        return _STATUS_TEXT.get(int(status), "unknown status")
    return _lib.pda_status_string(int(status)).decode()


_STATUS_TEXT = {PDA_OK: "ok", PDA_ERR_INVALID_ARG: "invalid argument", PDA_ERR_UNSUPPORTED: "unsupported configuration",
                PDA_ERR_WORKSPACE: "workspace must grow during stream capture", PDA_ERR_CUDA: "CUDA runtime error",
                PDA_ERR_DEVICE_TIMEOUT: "a kernel gave up on a bounded wait",
                PDA_ERR_NOALLOC_CAPACITY: "the call needs more split scratch than the static buffer holds"}


def _check(status: int, what: str):
    if status != PDA_OK:
        raise PdaError(status, what)


def _stream_ptr(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    if isinstance(stream, torch.cuda.Stream):
        return int(stream.cuda_stream)
    return int(stream)


def decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
           seq_lens: torch.Tensor, scale: float, k_scale: float, v_scale: float, *,
           out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """Decode attention over a paged fp8 cache (``pda_decode``).

    q ``[S, H, 128]`` bf16; k_cache ``[NB, Hk, 8, bs, 16]`` and v_cache
    ``[NB, Hk, 128, bs]`` float8_e4m3fn (or uint8 bytes); block_tables
    ``[S, MB]`` int32; seq_lens ``[S]`` int32; all contiguous on one CUDA
    device. Returns ``out`` (allocated like q when not given).
    """
    lib = load()
    _check_decode_args(q, k_cache, v_cache, block_tables, seq_lens)
    out = _out_like(q, out)
    S, H, D = q.shape
    NB, Hk, D16, bs, sixteen = k_cache.shape
    st = lib.pda_decode(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                        block_tables.data_ptr(), seq_lens.data_ptr(), S, H, Hk, D, bs,
                        int(block_tables.shape[1]), float(scale), float(k_scale), float(v_scale),
                        _stream_ptr(stream))
    _check(st, "pda_decode")
    return out


def _out_like(q, out):
    if out is None:
        return torch.empty_like(q)
    if out.shape != q.shape or out.dtype != torch.bfloat16 or not out.is_contiguous() or not out.is_cuda:
        raise PdaError(PDA_ERR_INVALID_ARG, "decode: out")
    return out


def _check_decode_args(q, k_cache, v_cache, block_tables, seq_lens, v_shuffled=False):
    if (q.dim() != 3 or k_cache.dim() != 5 or v_cache.dim() != (5 if v_shuffled else 4) or block_tables.dim() != 2
            or seq_lens.dim() != 1):
        raise PdaError(PDA_ERR_INVALID_ARG, "decode: tensor ranks")
    if q.dtype != torch.bfloat16 or block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise PdaError(PDA_ERR_INVALID_ARG, "decode: dtypes (q bf16, tables/seq_lens int32)")
    for t in (k_cache, v_cache):
        if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise PdaError(PDA_ERR_INVALID_ARG, "decode: cache dtype must be float8_e4m3fn")
    ts = [q, k_cache, v_cache, block_tables, seq_lens]
    if not all(t.is_cuda and t.is_contiguous() for t in ts):
        raise PdaError(PDA_ERR_INVALID_ARG, "decode: tensors must be contiguous CUDA tensors")
    S, H, D = q.shape
    NB, Hk, D16, bs, sixteen = k_cache.shape
    v_want = (NB, Hk, bs // 16, D, 16) if v_shuffled else (NB, Hk, D, bs)
    if (sixteen != 16 or D16 * 16 != D or tuple(v_cache.shape) != v_want
            or block_tables.shape[0] != S or seq_lens.shape[0] != S):
        raise PdaError(PDA_ERR_INVALID_ARG, "decode: shapes")


def decode_slot_scales(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                       v_scales: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float, *,
                       out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``pda_decode_slot_scales``: decode with per-slot fp32 scale tables ``[NB, Hk, bs]``."""
    lib = load()
    _check_decode_args(q, k_cache, v_cache, block_tables, seq_lens)
    NB, Hk, _, bs, _ = k_cache.shape
    for t in (k_scales, v_scales):
        if t.dtype != torch.float32 or tuple(t.shape) != (NB, Hk, bs) or not t.is_cuda or not t.is_contiguous():
            raise PdaError(PDA_ERR_INVALID_ARG, "decode_slot_scales: scale tables must be fp32 [NB, Hk, bs]")
    out = _out_like(q, out)
    S, H, D = q.shape
    st = lib.pda_decode_slot_scales(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                    k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(),
                                    seq_lens.data_ptr(), S, H, Hk, D, bs, int(block_tables.shape[1]), float(scale),
                                    _stream_ptr(stream))
    _check(st, "pda_decode_slot_scales")
    return out


def decode_ex(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
              seq_lens: torch.Tensor, scale: float, k_scale: float, v_scale: float, *, sinks=None,
              output_scale: float | None = None, v_shuffled: bool = False, out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor:
    """``pda_decode_ex``: decode with optional per-head sinks (fp32 ``[H]``),
    e4m3 output ``E4M3(o / output_scale)`` when ``output_scale`` is given, and
    the shuffled V layout ``[NB, Hk, bs/16, 128, 16]`` when ``v_shuffled``."""
    lib = load()
    _check_decode_args(q, k_cache, v_cache, block_tables, seq_lens, v_shuffled)
    S, H, D = q.shape
    NB, Hk, _, bs, _ = k_cache.shape
    if sinks is not None and (sinks.dtype != torch.float32 or tuple(sinks.shape) != (H,) or not sinks.is_cuda):
        raise PdaError(PDA_ERR_INVALID_ARG, "decode_ex: sinks must be a CUDA float32 [num_heads] tensor")
    fp8 = output_scale is not None
    want = torch.float8_e4m3fn if fp8 else torch.bfloat16
    if out is None:
        out = torch.empty(q.shape, dtype=want, device=q.device)
    elif out.shape != q.shape or out.dtype not in ((want, torch.uint8) if fp8 else (want,)) or not out.is_contiguous():
        raise PdaError(PDA_ERR_INVALID_ARG, "decode_ex: out")
    st = lib.pda_decode_ex(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                           block_tables.data_ptr(), seq_lens.data_ptr(), S, H, Hk, D, bs, int(block_tables.shape[1]),
                           float(scale), float(k_scale), float(v_scale),
                           PDA_KV_SHUFFLED_V if v_shuffled else PDA_KV_NATIVE,
                           sinks.data_ptr() if sinks is not None else None,
                           PDA_OUT_E4M3 if fp8 else PDA_OUT_BF16, float(output_scale) if fp8 else 1.0,
                           _stream_ptr(stream))
    _check(st, "pda_decode_ex")
    return out


def decode_strided(q: torch.Tensor, k_rows_base: int, v_rows_base: int, block_tables: torch.Tensor,
                   seq_lens: torch.Tensor, scale: float, k_scale: float, v_scale: float, *, num_kv_heads: int,
                   block_size: int, num_blocks: int, k_strides, v_strides, out: torch.Tensor | None = None,
                   stream=None) -> torch.Tensor:
    """``pda_decode_strided``: decode on a token-major fp8 cache.

    ``k_rows_base`` / ``v_rows_base`` are device addresses of the (block 0,
    token 0, head 0) rows; ``k_strides`` / ``v_strides`` are byte strides
    (block, token, kv head); every row holds 128 contiguous e4m3 bytes.
    """
    lib = load()
    if q.dim() != 3 or q.dtype != torch.bfloat16 or not q.is_cuda or not q.is_contiguous():
        raise PdaError(PDA_ERR_INVALID_ARG, "decode_strided: q")
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise PdaError(PDA_ERR_INVALID_ARG, "decode_strided: tables / seq_lens dtype")
    out = _out_like(q, out)
    S, H, D = q.shape
    kb, kt, kh = (int(x) for x in k_strides)
    vb, vt, vh = (int(x) for x in v_strides)
    st = lib.pda_decode_strided(out.data_ptr(), q.data_ptr(), int(k_rows_base), int(v_rows_base),
                                block_tables.data_ptr(), seq_lens.data_ptr(), S, H, int(num_kv_heads), D,
                                int(block_size), int(block_tables.shape[1]), int(num_blocks), kb, kt, kh, vb, vt, vh,
                                float(scale), float(k_scale), float(v_scale), _stream_ptr(stream))
    _check(st, "pda_decode_strided")
    return out


def decode_noalloc(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                   seq_lens: torch.Tensor, scale: float, k_scale: float, v_scale: float, *, out: torch.Tensor,
                   stream=None) -> torch.Tensor:
    """``pda_decode_noalloc``: ``decode`` without any device allocation.

    The output buffer must be given (nothing is allocated here either); the
    library keeps split partials in its fixed 16 MiB device array.
    """
    lib = load()
    _check_decode_args(q, k_cache, v_cache, block_tables, seq_lens)
    if out is None:
        raise PdaError(PDA_ERR_INVALID_ARG, "decode_noalloc: out must be given")
    out = _out_like(q, out)
    S, H, D = q.shape
    NB, Hk, _, bs, _ = k_cache.shape
    st = lib.pda_decode_noalloc(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                block_tables.data_ptr(), seq_lens.data_ptr(), S, H, Hk, D, bs,
                                int(block_tables.shape[1]), float(scale), float(k_scale), float(v_scale),
                                _stream_ptr(stream))
    _check(st, "pda_decode_noalloc")
    return out


def decode_host(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
                seq_lens: torch.Tensor, scale: float, k_scale: float, v_scale: float, *, out: torch.Tensor,
                stream=None) -> torch.Tensor:
    """``pda_decode_host``: ``decode`` on CPU tensors (pinned for asynchronous copies).

    Shapes and dtypes as ``decode``; every tensor, ``out`` included, is a
    contiguous CPU tensor. The call enqueues the copies in, the decode and
    the copy out on ``stream`` and returns: synchronise the stream before
    reading ``out``, and keep the inputs unchanged until then.
    """
    lib = load()
    if (q.dim() != 3 or k_cache.dim() != 5 or v_cache.dim() != 4 or block_tables.dim() != 2
            or seq_lens.dim() != 1):
        raise PdaError(PDA_ERR_INVALID_ARG, "decode_host: tensor ranks")
    if q.dtype != torch.bfloat16 or block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise PdaError(PDA_ERR_INVALID_ARG, "decode_host: dtypes (q bf16, tables/seq_lens int32)")
    if any(t.dtype not in (torch.float8_e4m3fn, torch.uint8) for t in (k_cache, v_cache)):
        raise PdaError(PDA_ERR_INVALID_ARG, "decode_host: cache dtype must be float8_e4m3fn")
    if out is None or out.shape != q.shape or out.dtype != torch.bfloat16:
        raise PdaError(PDA_ERR_INVALID_ARG, "decode_host: out must be given, shaped and typed like q")
    ts = [out, q, k_cache, v_cache, block_tables, seq_lens]
    if any(t.is_cuda or not t.is_contiguous() for t in ts):
        raise PdaError(PDA_ERR_INVALID_ARG, "decode_host: tensors must be contiguous CPU tensors")
    S, H, D = q.shape
    NB, Hk, D16, bs, sixteen = k_cache.shape
    if (sixteen != 16 or D16 * 16 != D or tuple(v_cache.shape) != (NB, Hk, D, bs) or block_tables.shape[0] != S
            or seq_lens.shape[0] != S):
        raise PdaError(PDA_ERR_INVALID_ARG, "decode_host: shapes")
    st = lib.pda_decode_host(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                             block_tables.data_ptr(), seq_lens.data_ptr(), S, H, Hk, D, bs,
                             int(block_tables.shape[1]), NB, float(scale), float(k_scale), float(v_scale),
                             _stream_ptr(stream))
    _check(st, "pda_decode_host")
    return out


def decode_raw(out_ptr: int, q_ptr: int, k_ptr: int, v_ptr: int, tables_ptr: int, lens_ptr: int, num_seqs: int,
               num_heads: int, num_kv_heads: int, head_size: int, block_size: int, max_num_blocks_per_seq: int,
               scale: float, k_scale: float, v_scale: float, stream_ptr: int = 0) -> int:
    """``pda_decode`` on raw device addresses; returns the status code."""
    return load().pda_decode(out_ptr, q_ptr, k_ptr, v_ptr, tables_ptr, lens_ptr, num_seqs, num_heads,
                             num_kv_heads, head_size, block_size, max_num_blocks_per_seq, float(scale),
                             float(k_scale), float(v_scale), stream_ptr)


def choose_splits(num_seqs, num_kv_heads, max_num_blocks_per_seq, block_size, sm_count, ctas_per_sm) -> int:
    return load().pda_choose_splits(num_seqs, num_kv_heads, max_num_blocks_per_seq, block_size, sm_count,
                                    ctas_per_sm)


def plan_splits(num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq, block_size) -> int:
    n = load().pda_plan_splits(num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq, block_size)
    if n < 1:
        raise PdaError(PDA_ERR_CUDA, "pda_plan_splits")
    return n


PDA_KERNEL_PER_UNIT, PDA_KERNEL_PER_UNIT_DENSE, PDA_KERNEL_PERSISTENT = 0, 1, 2
KERNEL_NAMES = {PDA_KERNEL_PER_UNIT: "per-unit (3 CTAs/SM)", PDA_KERNEL_PER_UNIT_DENSE: "per-unit dense (4 CTAs/SM)",
                PDA_KERNEL_PERSISTENT: "persistent"}


def plan_kernel(num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq, block_size) -> int:
    """The decode kernel instance (PDA_KERNEL_*) pda_decode would launch for these sizes."""
    k = load().pda_plan_kernel(num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq, block_size)
    if k < 0:
        raise PdaError(PDA_ERR_CUDA, "pda_plan_kernel")
    return k


def choose_kernel(num_seqs, num_kv_heads, max_num_blocks_per_seq, block_size, sm_count, ctas_per_sm,
                  ctas_per_sm_dense) -> tuple[int, int, int]:
    """The planner's pure choice: (PDA_KERNEL_* instance, split count, launches per call)."""
    ns, nl = ctypes.c_int(0), ctypes.c_int(0)
    k = load().pda_choose_kernel(num_seqs, num_kv_heads, max_num_blocks_per_seq, block_size, sm_count, ctas_per_sm,
                                 ctas_per_sm_dense, ctypes.byref(ns), ctypes.byref(nl))
    if k < 0:
        raise PdaError(PDA_ERR_INVALID_ARG, "pda_choose_kernel")
    return k, ns.value, nl.value


def plan_launches(num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq, block_size) -> int:
    """Kernels one pda_decode call launches for these sizes."""
    n = load().pda_plan_launches(num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq, block_size)
    if n < 0:
        raise PdaError(PDA_ERR_CUDA, "pda_plan_launches")
    return n


def plan_slot_scales(num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq, block_size) -> tuple[int, int, int]:
    """The plan of a pda_decode_slot_scales call: (PDA_KERNEL_* instance, split count, launches per call)."""
    k, ns, nl = ctypes.c_int(0), ctypes.c_int(0), ctypes.c_int(0)
    if load().pda_plan_slot_scales(num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq, block_size,
                                   ctypes.byref(k), ctypes.byref(ns), ctypes.byref(nl)) != 0:
        raise PdaError(PDA_ERR_CUDA, "pda_plan_slot_scales")
    return k.value, ns.value, nl.value


def tail_pieces(pages: int, tail_units: int, ctas: int, block_size: int) -> list[int]:
    """``pda_tail_pieces``: the piece sizes (pages) a tail unit of ``pages`` pages is cut into."""
    buf = (_I * 8)()
    n = load().pda_tail_pieces(pages, tail_units, ctas, block_size, buf, 8)
    if n < 0:
        raise PdaError(PDA_ERR_INVALID_ARG, "pda_tail_pieces")
    return [buf[i] for i in range(n)]


def set_split_override(n: int) -> None:
    load().pda_set_split_override(int(n))


def set_tail_split(enable: bool) -> None:
    """``pda_set_tail_split``: tail pieces of the persistent kernel on (default) or off."""
    load().pda_set_tail_split(1 if enable else 0)


def set_tma_gather(enable: bool) -> None:
    """``pda_set_tma_gather``: four-row TMA gathers of pages and scale rows on (default) or off."""
    load().pda_set_tma_gather(1 if enable else 0)


def set_block_check(num_blocks: int) -> None:
    """``pda_set_block_check``: check decode block ids against [0, num_blocks) on the device (0 = off)."""
    load().pda_set_block_check(int(num_blocks))


def reserve(num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq, block_size, stream=None) -> None:
    _check(load().pda_reserve(num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq, block_size,
                              _stream_ptr(stream)), "pda_reserve")


def release() -> None:
    _check(load().pda_release(), "pda_release")


def workspace_info(stream=None) -> tuple[int, int]:
    """``pda_workspace_info``: (current bytes, retired buffers kept alive) of
    the current device's workspace for ``stream``."""
    lib = load()
    nbytes, retired = ctypes.c_longlong(0), _I(0)
    _check(lib.pda_workspace_info(_stream_ptr(stream), ctypes.byref(nbytes), ctypes.byref(retired)),
           "pda_workspace_info")
    return int(nbytes.value), int(retired.value)


def query_device_status(stream=None) -> int:
    code = ctypes.c_int(0)
    st = load().pda_query_device_status(_stream_ptr(stream), ctypes.byref(code))
    if st not in (PDA_OK, PDA_ERR_DEVICE_TIMEOUT):
        raise PdaError(st, "pda_query_device_status")
    return int(code.value)


def set_profile_events(before, after) -> None:
    """Record two torch.cuda.Event around the decode kernel (None, None: off)."""
    if before is None or after is None:
        load().pda_set_profile_events(None, None)
    else:
        for e in (before, after):
            if int(e.cuda_event) == 0:   # torch creates the event on its first record
                e.record()
        load().pda_set_profile_events(int(before.cuda_event), int(after.cuda_event))


def bounded_wait_check(timeout_us: int, stream=None) -> None:
    _check(load().pda_test_bounded_wait(int(timeout_us), _stream_ptr(stream)), "pda_test_bounded_wait")


def reshape_and_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      slot_mapping: torch.Tensor, k_scale: float, v_scale: float, *, v_shuffled: bool = False,
                      stream=None) -> None:
    """Quantise and scatter new tokens into the paged fp8 cache (``pda_reshape_and_cache``).

    key / value ``[T, Hk, 128]`` bf16; slot_mapping ``[T]`` int64 (negative =
    skip); caches as for ``decode`` (written in place).
    """
    lib = load()
    if key.dim() != 3 or value.shape != key.shape or key.dtype != torch.bfloat16 or value.dtype != torch.bfloat16:
        raise PdaError(PDA_ERR_INVALID_ARG, "reshape_and_cache: key/value")
    if slot_mapping.dtype != torch.int64 or slot_mapping.shape != (key.shape[0],):
        raise PdaError(PDA_ERR_INVALID_ARG, "reshape_and_cache: slot_mapping")
    for t in (k_cache, v_cache):
        if t.dtype not in (torch.float8_e4m3fn, torch.uint8):
            raise PdaError(PDA_ERR_INVALID_ARG, "reshape_and_cache: cache dtype")
    ts = [key, value, k_cache, v_cache, slot_mapping]
    if not all(t.is_cuda and t.is_contiguous() for t in ts):
        raise PdaError(PDA_ERR_INVALID_ARG, "reshape_and_cache: tensors must be contiguous CUDA tensors")
    T, Hk, D = key.shape
    NB, Hk2, D16, bs, sixteen = k_cache.shape
    v_want = (NB, Hk, bs // 16, D, 16) if v_shuffled else (NB, Hk, D, bs)
    if Hk2 != Hk or D16 * 16 != D or sixteen != 16 or tuple(v_cache.shape) != v_want:
        raise PdaError(PDA_ERR_INVALID_ARG, "reshape_and_cache: shapes")
    _check(lib.pda_reshape_and_cache(key.data_ptr(), value.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                     slot_mapping.data_ptr(), T, Hk, D, bs, NB, float(k_scale), float(v_scale),
                                     PDA_KV_SHUFFLED_V if v_shuffled else PDA_KV_NATIVE, _stream_ptr(stream)),
           "pda_reshape_and_cache")


def _refuse(what: str):
    raise PdaError(PDA_ERR_INVALID_ARG, what)


def _on_device(what: str, tensors) -> int:
    """Every tensor must lie on the current CUDA device, whose streams the calls use; returns its index."""
    dev = tensors[0].get_device()
    for t in tensors:
        if t.get_device() != dev:
            _refuse(what + ": tensors must be on one CUDA device")
    if dev < 0 or dev != _device():
        _refuse(what + ": tensors must be on the current CUDA device")
    return dev


def _stream_on(stream, dev: int) -> int:
    """The raw handle of ``stream``, or of the current stream of device ``dev``."""
    return _raw_stream(dev) if stream is None else _stream_ptr(stream)


# ---------------------------------------------------------------- rotary

def rope_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: int = PDA_ROPE_PLAIN, factor: float = 1.0,
                     original_length: float = 0.0, low: float | None = None,
                     high: float | None = None) -> tuple[torch.Tensor, float]:
    """``pda_rope_frequencies``: (inv_freq float64 ``[rot_dim/2]`` on the CPU, magnitude).

    ``scaling`` is one of ``PDA_ROPE_*``; ``low`` / ``high`` default to 1 and
    32 (RAMP) or 1 and 4 (BANDS).
    """
    if int(rot_dim) <= 0:
        raise PdaError(PDA_ERR_INVALID_ARG, "rope_frequencies: rot_dim")
    f = torch.empty(int(rot_dim) // 2, dtype=torch.float64)
    mag = _D(1.0)
    lo = 1.0 if low is None else float(low)
    hi = (4.0 if scaling == PDA_ROPE_BANDS else 32.0) if high is None else float(high)
    _check(load().pda_rope_frequencies(f.data_ptr(), ctypes.addressof(mag), int(rot_dim), float(base), int(scaling),
                                       float(factor), float(original_length), lo, hi), "pda_rope_frequencies")
    return f, mag.value


def _rope_refuse(what, heads, positions, inv_freq):
    """Says what is wrong with a call whose quick checks failed."""
    for x in heads:
        if x.dtype != torch.bfloat16 or x.dim() != 3:
            _refuse(what + ": heads must be bf16 [T, heads, 128]")
        if x.stride(2) != 1:
            _refuse(what + ": the 128 dims of a head must be contiguous")
    if positions.dtype != torch.int64 or positions.dim() != 1 or not positions.is_contiguous():
        _refuse(what + ": positions must be contiguous int64 [T]")
    if inv_freq.dtype != torch.float64 or inv_freq.dim() != 1 or inv_freq.is_cuda or not inv_freq.is_contiguous():
        _refuse(what + ": inv_freq must be a contiguous CPU float64 [rot_dim/2]")
    _refuse(what + ": tokens, head sizes, shapes or devices do not agree (all on the current CUDA device)")


_BF16, _I64, _I32, _F64 = torch.bfloat16, torch.int64, torch.int32, torch.float64
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)   # absent in builds without CUDA


def rope(q: torch.Tensor, k: torch.Tensor | None, positions: torch.Tensor, inv_freq: torch.Tensor, *,
         magnitude: float = 1.0, interleaved: bool = False, q_out: torch.Tensor | None = None,
         k_out: torch.Tensor | None = None, stream=None):
    """``pda_rope``: rotary positions of q ``[T, H, 128]`` and k ``[T, Hk, 128]`` (bf16; any token and head strides).

    positions ``[T]`` int64; inv_freq float64 ``[rot_dim/2]`` on the CPU
    (``rope_frequencies``). k may be None. Returns (q_out, k_out), allocated
    contiguous when not given; ``q_out=q`` rotates in place.
    """
    lib = _lib or load()
    # One condition: a decode step spends more time in these checks than on the GPU.
    heads = [q] if k is None else [q, k]
    dev = q.get_device()
    if not (positions.dtype is _I64 and positions.dim() == 1 and positions.is_contiguous()
            and positions.get_device() == dev and inv_freq.dtype is _F64 and inv_freq.dim() == 1
            and inv_freq.get_device() == -1 and inv_freq.is_contiguous() and q.dim() == 3):
        _rope_refuse("rope", heads, positions, inv_freq)
    T, D, done = positions.shape[0], q.shape[2], []
    for x, out in zip(heads, (q_out, k_out)):
        if x.dim() != 3 or x.dtype is not _BF16 or x.get_device() != dev:
            _rope_refuse("rope", heads, positions, inv_freq)
        n, h, d = x.shape
        s0, s1, s2 = x.stride()
        if out is None:
            out = torch.empty((n, h, d), dtype=_BF16, device=x.device)
            o0, o1, o2 = h * d, d, 1
        elif out.shape != x.shape or out.dtype is not _BF16 or out.get_device() != dev:
            _refuse("rope: out must be bf16, shaped like its input, on its device")
        else:
            o0, o1, o2 = out.stride()
        if n != T or d != D or ((s2 != 1 or o2 != 1) and n * h):
            _rope_refuse("rope", heads + [out], positions, inv_freq)
        done.append(out)
        done.append(_RopeHeads(x.data_ptr(), out.data_ptr(), s0, s1, o0, o1, h))
    if dev != _device():
        _rope_refuse("rope", heads, positions, inv_freq)
    st = lib.pda_rope(ctypes.addressof(done[1]), None if k is None else ctypes.addressof(done[3]),
                      positions.data_ptr(), T, D, inv_freq.data_ptr(), 2 * inv_freq.shape[0], 1 if interleaved else 0,
                      magnitude, _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        raise PdaError(st, "pda_rope")
    return done[0], None if k is None else done[2]


def rope_and_cache(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, positions: torch.Tensor,
                   slot_mapping: torch.Tensor, inv_freq: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                   k_scale: float, v_scale: float, *, magnitude: float = 1.0, interleaved: bool = False,
                   v_shuffled: bool = False, q_out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``pda_rope_and_cache``: rotate q and k, and write the rotated k and v into the paged fp8 cache.

    q ``[T, H, 128]``, k and v ``[T, Hk, 128]`` bf16 with any token and head
    strides; slot_mapping and the caches as for ``reshape_and_cache``. Returns
    the rotated queries (``q_out``, allocated contiguous when not given).
    """
    lib = _lib or load()
    what = "rope_and_cache"
    dev = q.get_device()
    if not (positions.dtype is _I64 and positions.dim() == 1 and positions.is_contiguous()
            and positions.get_device() == dev and inv_freq.dtype is _F64 and inv_freq.dim() == 1
            and inv_freq.get_device() == -1 and inv_freq.is_contiguous() and q.dim() == 3 and k.dim() == 3
            and v.dim() == 3 and q.dtype is _BF16 and k.dtype is _BF16 and v.dtype is _BF16):
        _rope_refuse(what, (q, k, v), positions, inv_freq)
    T, H, D = q.shape
    Hk = k.shape[1]
    q0, q1, q2 = q.stride()
    k0, k1, k2 = k.stride()
    v0, v1, v2 = v.stride()
    if (k.shape != (T, Hk, D) or v.shape != (T, Hk, D) or positions.shape[0] != T
            or ((q2 != 1 or k2 != 1 or v2 != 1) and T) or k.get_device() != dev or v.get_device() != dev
            or dev != _device()):
        _rope_refuse(what, (q, k, v), positions, inv_freq)
    if (slot_mapping.dtype is not _I64 or slot_mapping.shape != (T,) or not slot_mapping.is_contiguous()
            or slot_mapping.get_device() != dev):
        _refuse(what + ": slot_mapping must be contiguous int64 [T] on q's device")
    for t in (k_cache, v_cache):
        if t.dtype not in _CACHE_TYPES or not t.is_contiguous() or t.get_device() != dev:
            _refuse(what + ": caches must be contiguous float8_e4m3fn on q's device")
    if k_cache.dim() != 5:
        _refuse(what + ": shapes")
    NB, Hk2, D16, bs, sixteen = k_cache.shape
    if Hk2 != Hk or D16 * 16 != D or sixteen != 16 \
            or v_cache.shape != ((NB, Hk, bs // 16, D, 16) if v_shuffled else (NB, Hk, D, bs)):
        _refuse(what + ": shapes")
    if q_out is None:
        q_out = torch.empty((T, H, D), dtype=_BF16, device=q.device)
        o0, o1, o2 = H * D, D, 1
    else:
        o0, o1, o2 = q_out.stride() if q_out.dim() == 3 else (0, 0, 0)
        if q_out.shape != q.shape or q_out.dtype is not _BF16 or q_out.get_device() != dev or (o2 != 1 and T):
            _refuse(what + ": q_out must be bf16 and shaped like q, heads contiguous, on its device")
    hq = _RopeHeads(q.data_ptr(), q_out.data_ptr(), q0, q1, o0, o1, H)
    hk = _RopeHeads(k.data_ptr(), None, k0, k1, 0, 0, Hk)
    hv = _RopeHeads(v.data_ptr(), None, v0, v1, 0, 0, Hk)
    st = lib.pda_rope_and_cache(ctypes.addressof(hq), ctypes.addressof(hk), ctypes.addressof(hv),
                                positions.data_ptr(), slot_mapping.data_ptr(), T, D, inv_freq.data_ptr(),
                                2 * inv_freq.shape[0], 1 if interleaved else 0, magnitude, k_cache.data_ptr(),
                                v_cache.data_ptr(), bs, NB, k_scale, v_scale,
                                PDA_KV_SHUFFLED_V if v_shuffled else PDA_KV_NATIVE,
                                _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        raise PdaError(st, "pda_rope_and_cache")
    return q_out


_CACHE_TYPES = (torch.float8_e4m3fn, torch.uint8)


# ------------------------------------------------- attention of new tokens

def extend(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor,
           seq_lens: torch.Tensor, query_starts: torch.Tensor, scale: float, k_scale: float, v_scale: float, *,
           window: int = 0, sinks: torch.Tensor | None = None, output_scale: float | None = None,
           v_shuffled: bool = False, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``pda_extend``: causal attention of each sequence's new tokens over its pages.

    q ``[T, H, 128]`` bf16, the new tokens packed; query_starts ``[S + 1]``
    int32; seq_lens ``[S]`` int32 counts the new tokens too. ``window`` > 0
    limits a token to the last ``window`` tokens. sinks, output_scale and
    v_shuffled as for ``decode_ex``. Rows of no sequence are left as they are
    in ``out`` (uninitialised when ``out`` is not given).
    """
    lib = _lib or load()
    if q.dim() != 3 or k_cache.dim() != 5 or block_tables.dim() != 2:
        _refuse("extend: tensor ranks")
    T, H, D = q.shape
    NB, Hk, D16, bs, sixteen = k_cache.shape
    S, MB = block_tables.shape
    i32 = torch.int32
    if q.dtype != torch.bfloat16 or block_tables.dtype != i32 or seq_lens.dtype != i32 or query_starts.dtype != i32:
        _refuse("extend: dtypes (q bf16, tables / seq_lens / query_starts int32)")
    f8 = (torch.float8_e4m3fn, torch.uint8)
    if k_cache.dtype not in f8 or v_cache.dtype not in f8:
        _refuse("extend: cache dtype must be float8_e4m3fn")
    if (sixteen != 16 or D16 * 16 != D
            or v_cache.shape != ((NB, Hk, bs // 16, D, 16) if v_shuffled else (NB, Hk, D, bs))
            or seq_lens.shape != (S,) or query_starts.shape != (S + 1,)):
        _refuse("extend: shapes")
    fp8 = output_scale is not None
    want = torch.float8_e4m3fn if fp8 else torch.bfloat16
    if out is None:
        out = torch.empty((T, H, D), dtype=want, device=q.device)
    elif out.shape != q.shape or out.dtype not in ((want, torch.uint8) if fp8 else (want,)):
        _refuse("extend: out")
    ts = (q, k_cache, v_cache, block_tables, seq_lens, query_starts, out)
    if sinks is not None:
        if sinks.dtype != torch.float32 or sinks.shape != (H,):
            _refuse("extend: sinks must be a float32 [num_heads] tensor")
        ts += (sinks,)
    for t in ts:
        if not t.is_contiguous():
            _refuse("extend: tensors must be contiguous")
    dev = _on_device("extend", ts)
    _check(lib.pda_extend(out.data_ptr(), q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                          block_tables.data_ptr(), seq_lens.data_ptr(), query_starts.data_ptr(), T, S, H, Hk, D, bs,
                          MB, scale, k_scale, v_scale, window, PDA_KV_SHUFFLED_V if v_shuffled else PDA_KV_NATIVE,
                          None if sinks is None else sinks.data_ptr(), PDA_OUT_E4M3 if fp8 else PDA_OUT_BF16,
                          output_scale if fp8 else 1.0, _stream_on(stream, dev)), "pda_extend")
    return out


def reserve_extend(num_tokens, num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq, block_size,
                   stream=None) -> None:
    """``pda_reserve_extend``: size the workspace for ``extend`` calls up to these sizes (before a stream capture)."""
    _check(load().pda_reserve_extend(num_tokens, num_seqs, num_heads, num_kv_heads, max_num_blocks_per_seq,
                                     block_size, _stream_ptr(stream)), "pda_reserve_extend")


# ----------------------------------------------------------------- pages

def _page_table(what, ref_counts, block_tables, seq_lens, block_size, *lists):
    """(ctypes pda_page_table, device index) of the checked state and request lists."""
    dev = ref_counts.get_device()
    S, MB = block_tables.shape if block_tables.dim() == 2 else (-1, -1)
    if ref_counts.dim() != 1 or seq_lens.shape != (S,):
        _refuse(what + ": shapes (ref_counts [NB], block_tables [S, MB], seq_lens [S])")
    for t in (ref_counts, block_tables, seq_lens, *lists):
        if t.dtype is not _I32 or not t.is_contiguous() or t.get_device() != dev:
            _refuse(what + ": tables, counts, lengths and lists must be contiguous int32 on one CUDA device")
    if lists and (lists[0].dim() != 1 or lists[-1].shape != lists[0].shape):
        _refuse(what + ": request lists must be vectors of one length")
    if dev < 0 or dev != _device():
        _refuse(what + ": tensors must be on the current CUDA device")
    return _PageTable(ref_counts.data_ptr(), block_tables.data_ptr(), seq_lens.data_ptr(), ref_counts.shape[0], S, MB,
                      block_size), dev


_page_array_types = {}     # ctypes array types by length (making one takes longer than filling it)


def _page_arrays(what, caches, num_blocks, dev):
    """(ctypes array of pda_page_array, count) of tensors ``[num_blocks, ...]`` on device ``dev``."""
    n = len(caches)
    kind = _page_array_types.get(n)
    if kind is None:
        kind = _page_array_types[n] = _PageArray * n
    if not num_blocks:
        return kind(), 0
    flat = []
    for t in caches:
        if t.dim() == 0 or t.shape[0] != num_blocks or not t.is_contiguous() or t.get_device() != dev:
            _refuse(what + ": caches must be contiguous [num_blocks, ...] tensors on the current device")
        flat.append((t.data_ptr(), t.nbytes // num_blocks))
    return kind(*flat), n


def copy_pages(caches, src: torch.Tensor, dst: torch.Tensor, *, stream=None) -> None:
    """``pda_copy_pages``: copy pages ``src[i]`` to ``dst[i]`` in every cache tensor ``[num_blocks, ...]``."""
    lib = _lib or load()
    if src.dtype != torch.int32 or dst.dtype != torch.int32 or src.dim() != 1 or src.shape != dst.shape \
            or not src.is_contiguous() or not dst.is_contiguous():
        _refuse("copy_pages: src and dst must be contiguous int32 vectors of one length")
    dev = _on_device("copy_pages", (src, dst))
    NB = caches[0].shape[0] if len(caches) and caches[0].dim() else 0
    arr, n = _page_arrays("copy_pages", caches, NB, dev)
    _check(lib.pda_copy_pages(ctypes.addressof(arr), n, src.data_ptr(), dst.data_ptr(), src.shape[0], NB,
                              _stream_on(stream, dev)), "pda_copy_pages")


def grow_pages(ref_counts: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, rows: torch.Tensor,
               add: torch.Tensor, block_size: int, *, stream=None) -> None:
    """``pda_grow_pages``: row ``rows[i]`` takes ``add[i]`` more tokens, with fresh pages where it needs them."""
    tab, dev = _page_table("grow_pages", ref_counts, block_tables, seq_lens, block_size, rows, add)
    st = (_lib or load()).pda_grow_pages(ctypes.addressof(tab), rows.data_ptr(), add.data_ptr(), rows.shape[0],
                                         _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        raise PdaError(st, "pda_grow_pages")


def fork_pages(ref_counts: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, parents: torch.Tensor,
               children: torch.Tensor, block_size: int, caches=(), *, stream=None) -> None:
    """``pda_fork_pages``: empty row ``children[i]`` becomes a copy of row ``parents[i]``.

    Full pages are shared; a partly filled last page is copied to a fresh one
    in every tensor of ``caches`` (``[num_blocks, ...]`` each).
    """
    tab, dev = _page_table("fork_pages", ref_counts, block_tables, seq_lens, block_size, parents, children)
    arr, n = _page_arrays("fork_pages", caches, tab.num_blocks, dev)
    st = (_lib or load()).pda_fork_pages(ctypes.addressof(tab), parents.data_ptr(), children.data_ptr(),
                                         parents.shape[0], ctypes.addressof(arr), n,
                                         _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        raise PdaError(st, "pda_fork_pages")


def free_pages(ref_counts: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, rows: torch.Tensor,
               block_size: int, *, stream=None) -> None:
    """``pda_free_pages``: rows become empty and give their pages up."""
    tab, dev = _page_table("free_pages", ref_counts, block_tables, seq_lens, block_size, rows)
    st = (_lib or load()).pda_free_pages(ctypes.addressof(tab), rows.data_ptr(), rows.shape[0],
                                         _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        raise PdaError(st, "pda_free_pages")


def compact_pages(ref_counts: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, block_size: int,
                  caches=(), *, new_ids: torch.Tensor | None = None, stream=None) -> None:
    """``pda_compact_pages``: move the held pages to the lowest ids, in every cache, count and table entry.

    ``new_ids`` (int32 ``[num_blocks]``) receives every page's id after the call.
    """
    lib = _lib or load()
    tab, dev = _page_table("compact_pages", ref_counts, block_tables, seq_lens, block_size)
    arr, n = _page_arrays("compact_pages", caches, ref_counts.shape[0], dev)
    if new_ids is not None and (new_ids.shape != ref_counts.shape or new_ids.dtype is not _I32
                                or not new_ids.is_contiguous() or new_ids.get_device() != dev):
        _refuse("compact_pages: new_ids must be contiguous int32 [num_blocks] on the tables' device")
    _check(lib.pda_compact_pages(ctypes.addressof(tab), ctypes.addressof(arr), n,
                                 None if new_ids is None else new_ids.data_ptr(), _stream_on(stream, dev)),
           "pda_compact_pages")


def reserve_pages(num_blocks: int, num_rows: int, max_requests: int, stream=None) -> None:
    """``pda_reserve_pages``: size the page calls' workspace (before a stream capture)."""
    _check(load().pda_reserve_pages(int(num_blocks), int(num_rows), int(max_requests), _stream_ptr(stream)),
           "pda_reserve_pages")


# ------------------------------------------------- caches in fewer bits

FP4_TOKEN_BYTES = 144     # K and V of one (token, kv head): codes and group scales


def fp4_cache_shape(num_blocks: int, num_kv_heads: int, block_size: int) -> tuple[int, int, int]:
    """Shape of the uint8 tensor of a 4-bit cache (layout: ``include/pda.h``)."""
    return num_blocks, num_kv_heads, FP4_TOKEN_BYTES * block_size


_U8, _F32 = torch.uint8, torch.float32


def _say_why(what, checks):
    """Raises with the first of the (holds, message) checks that fails: the quick checks of a call did."""
    for holds, message in checks:
        if not holds():
            _refuse(what + ": " + message)
    _refuse(what + ": tensors must be on the current CUDA device")


def _write_refuse(what, key, value, slot_mapping, cache_checks):
    _say_why(what, [
        (lambda: key.dim() == 3 and value.shape == key.shape and key.dtype is _BF16 and value.dtype is _BF16,
         "key and value must be bf16 [T, Hk, 128] of one shape"),
        (lambda: key.numel() == 0 or (key.stride(2) == 1 and value.stride(2) == 1),
         "the 128 dims of a row must be contiguous"),
        (lambda: slot_mapping.dtype is _I64 and slot_mapping.shape == key.shape[:1] and slot_mapping.is_contiguous(),
         "slot_mapping must be contiguous int64 [T]")] + cache_checks)


def _e4m3_checks(k_cache, v_cache, v_shuffled=False, heads=None):
    def shapes():
        if k_cache.dim() != 5:
            return False
        NB, Hk, D16, bs, sixteen = k_cache.shape
        want = (NB, Hk, bs // 16, 128, 16) if v_shuffled else (NB, Hk, 128, bs)
        return D16 == 8 and sixteen == 16 and v_cache.shape == want and heads in (None, Hk)

    return [(lambda: k_cache.dtype in _CACHE_TYPES and v_cache.dtype in _CACHE_TYPES and k_cache.is_contiguous()
             and v_cache.is_contiguous(), "caches must be contiguous float8_e4m3fn"), (shapes, "shapes of the caches")]


def _scale_checks(k_scales, v_scales, k_cache):
    return [(lambda: all(t.dtype is _F32 and t.is_contiguous() and t.shape == (k_cache.shape[0], k_cache.shape[1],
                                                                               k_cache.shape[3])
                         for t in (k_scales, v_scales)), "scale tables must be contiguous float32 [NB, Hk, bs]")]


def _fp4_checks(kv_cache, heads=None):
    return [(lambda: kv_cache.dim() == 3 and kv_cache.dtype is _U8 and kv_cache.is_contiguous() and kv_cache.shape[2] > 0
             and kv_cache.shape[2] % FP4_TOKEN_BYTES == 0 and heads in (None, kv_cache.shape[1]),
             "kv_cache must be contiguous uint8 [NB, Hk, 144 * bs]")]


def reshape_and_cache_slot_scales(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                                  k_scales: torch.Tensor, v_scales: torch.Tensor, slot_mapping: torch.Tensor, *,
                                  min_scale: float = 2.0 ** -20, stream=None) -> None:
    """``pda_reshape_and_cache_slot_scales``: write new tokens as e4m3, each row with a scale of its own.

    key / value ``[T, Hk, 128]`` bf16 with any token and head strides; the
    caches (native layout) and ``slot_mapping`` as for ``reshape_and_cache``;
    k_scales / v_scales float32 ``[NB, Hk, bs]``, as ``decode_slot_scales``
    reads them. A scale is the row's amax / 448, at least ``min_scale``.
    """
    what = "reshape_and_cache_slot_scales"
    lib = _lib or load()
    # One condition, as in rope: a decode step spends more time in these checks than on the GPU.
    dev = key.get_device()
    ks, cs = key.shape, k_cache.shape
    if not (len(ks) == 3 and len(cs) == 5 and value.shape == ks and key.dtype is _BF16 and value.dtype is _BF16
            and slot_mapping.dtype is _I64 and slot_mapping.shape == ks[:1] and slot_mapping.is_contiguous()
            and k_cache.dtype in _CACHE_TYPES and v_cache.dtype in _CACHE_TYPES and k_cache.is_contiguous()
            and v_cache.is_contiguous() and cs[1] == ks[1] and cs[2] == 8 and cs[4] == 16
            and v_cache.shape == (cs[0], cs[1], 128, cs[3]) and k_scales.dtype is _F32 and v_scales.dtype is _F32
            and k_scales.shape == (cs[0], cs[1], cs[3]) and v_scales.shape == k_scales.shape
            and k_scales.is_contiguous() and v_scales.is_contiguous()
            and 0 <= dev == value.get_device() == slot_mapping.get_device() == k_cache.get_device() == v_cache.get_device()
            == k_scales.get_device() == v_scales.get_device() == _device()):
        _write_refuse(what, key, value, slot_mapping, _e4m3_checks(k_cache, v_cache, heads=ks[1] if len(ks) == 3 else -1)
                      + _scale_checks(k_scales, v_scales, k_cache))
    T, Hk, D = ks
    k0, k1, k2 = key.stride()
    v0, v1, v2 = value.stride()
    if (k2 != 1 or v2 != 1) and T * Hk:
        _refuse(what + ": the 128 dims of a row must be contiguous")
    k, v = _TokenRows(key.data_ptr(), k0, k1), _TokenRows(value.data_ptr(), v0, v1)
    st = lib.pda_reshape_and_cache_slot_scales(ctypes.addressof(k), ctypes.addressof(v), k_cache.data_ptr(),
                                               v_cache.data_ptr(), k_scales.data_ptr(), v_scales.data_ptr(),
                                               slot_mapping.data_ptr(), T, Hk, D, cs[3], cs[0], min_scale,
                                               _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        raise PdaError(st, "pda_reshape_and_cache_slot_scales")


def reshape_and_cache_fp4(key: torch.Tensor, value: torch.Tensor, kv_cache: torch.Tensor, slot_mapping: torch.Tensor,
                          k_scale: float, v_scale: float, *, stream=None) -> None:
    """``pda_reshape_and_cache_fp4``: write new tokens into a 4-bit cache ``[NB, Hk, 144 * bs]`` (``fp4_cache_shape``).

    key / value and slot_mapping as for ``reshape_and_cache_slot_scales``. Each
    16 dims get a scale of their own; ``k_scale`` / ``v_scale`` (about
    max|x| / 2688) are the tensors'.
    """
    what = "reshape_and_cache_fp4"
    lib = _lib or load()
    dev = key.get_device()
    ks, cs = key.shape, kv_cache.shape
    if not (len(ks) == 3 and len(cs) == 3 and value.shape == ks and key.dtype is _BF16 and value.dtype is _BF16
            and slot_mapping.dtype is _I64 and slot_mapping.shape == ks[:1] and slot_mapping.is_contiguous()
            and kv_cache.dtype is _U8 and kv_cache.is_contiguous() and cs[1] == ks[1] and cs[2] and cs[2] % 144 == 0
            and 0 <= dev == value.get_device() == slot_mapping.get_device() == kv_cache.get_device() == _device()):
        _write_refuse(what, key, value, slot_mapping, _fp4_checks(kv_cache, heads=ks[1] if len(ks) == 3 else -1))
    T, Hk, D = ks
    k0, k1, k2 = key.stride()
    v0, v1, v2 = value.stride()
    if (k2 != 1 or v2 != 1) and T * Hk:
        _refuse(what + ": the 128 dims of a row must be contiguous")
    k, v = _TokenRows(key.data_ptr(), k0, k1), _TokenRows(value.data_ptr(), v0, v1)
    st = lib.pda_reshape_and_cache_fp4(ctypes.addressof(k), ctypes.addressof(v), kv_cache.data_ptr(),
                                       slot_mapping.data_ptr(), T, Hk, D, cs[2] // 144, cs[0], k_scale, v_scale,
                                       _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        raise PdaError(st, "pda_reshape_and_cache_fp4")


def _gather_rows(what, block_tables, token_starts, first, num_tokens, Hk, k_out, v_out, dev, cache_ok, cache_checks):
    """(k_out, v_out, S, MB, first's address) of the checked arguments that the readers share."""
    bt = block_tables.shape
    shape = (num_tokens, Hk, 128)
    if not (cache_ok and len(bt) == 2 and token_starts.shape == (bt[0] + 1,) and block_tables.dtype is _I32
            and token_starts.dtype is _I32 and block_tables.is_contiguous() and token_starts.is_contiguous()
            and num_tokens >= 0 and 0 <= dev == block_tables.get_device() == token_starts.get_device() == _device()
            and (first is None or (first.shape == bt[:1] and first.dtype is _I32 and first.is_contiguous()
                                   and first.get_device() == dev))):
        _say_why(what, cache_checks() + [
            (lambda: len(bt) == 2 and token_starts.shape == (bt[0] + 1,) and (first is None or first.shape == bt[:1]),
             "shapes (block_tables [S, MB], token_starts [S + 1], first [S])"),
            (lambda: all(t is None or (t.dtype is _I32 and t.is_contiguous()) for t in (block_tables, token_starts, first)),
             "block_tables, token_starts and first must be contiguous int32"),
            (lambda: num_tokens >= 0, "num_tokens")])
    if k_out is None:
        k_out = torch.empty(shape, dtype=_BF16, device=block_tables.device)
    elif not (k_out.shape == shape and k_out.dtype is _BF16 and k_out.is_contiguous() and k_out.get_device() == dev):
        _refuse(what + ": k_out must be contiguous bf16 [num_tokens, Hk, 128] on the cache's device")
    if v_out is None:
        v_out = torch.empty_like(k_out)
    elif not (v_out.shape == shape and v_out.dtype is _BF16 and v_out.is_contiguous() and v_out.get_device() == dev):
        _refuse(what + ": v_out must be contiguous bf16 [num_tokens, Hk, 128] on the cache's device")
    return k_out, v_out, bt[0], bt[1], None if first is None else first.data_ptr()


def _e4m3_ok(k_cache, v_cache, dev, v_shuffled=False):
    cs = k_cache.shape
    return (len(cs) == 5 and cs[2] == 8 and cs[4] == 16 and k_cache.dtype in _CACHE_TYPES
            and v_cache.dtype in _CACHE_TYPES and k_cache.is_contiguous() and v_cache.is_contiguous()
            and v_cache.get_device() == dev
            and v_cache.shape == ((cs[0], cs[1], cs[3] // 16, 128, 16) if v_shuffled else (cs[0], cs[1], 128, cs[3])))


def gather_cache(k_cache: torch.Tensor, v_cache: torch.Tensor, block_tables: torch.Tensor, token_starts: torch.Tensor,
                 num_tokens: int, k_scale: float, v_scale: float, *, first: torch.Tensor | None = None,
                 v_shuffled: bool = False, k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
                 stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """``pda_gather_cache``: the keys and values of sequences' tokens as bf16 ``[num_tokens, Hk, 128]``, packed.

    Sequence s fills rows ``token_starts[s]`` up to ``token_starts[s + 1]``
    (int32 ``[S + 1]``) with its tokens from position ``first[s]`` (int32
    ``[S]``, default 0) on. Rows of no sequence are left as they are in
    ``k_out`` / ``v_out`` (uninitialised when not given).
    """
    lib = _lib or load()
    dev = k_cache.get_device()
    cs = k_cache.shape
    ok = _e4m3_ok(k_cache, v_cache, dev, v_shuffled)
    k, v, S, MB, at = _gather_rows("gather_cache", block_tables, token_starts, first, num_tokens, cs[1] if ok else 0, k_out,
                                   v_out, dev, ok, lambda: _e4m3_checks(k_cache, v_cache, v_shuffled))
    st = lib.pda_gather_cache(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_tables.data_ptr(),
                              token_starts.data_ptr(), at, num_tokens, S, cs[1], 128, cs[3], MB, cs[0], k_scale, v_scale,
                              PDA_KV_SHUFFLED_V if v_shuffled else PDA_KV_NATIVE,
                              _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        raise PdaError(st, "pda_gather_cache")
    return k, v


def gather_cache_slot_scales(k_cache: torch.Tensor, v_cache: torch.Tensor, k_scales: torch.Tensor,
                             v_scales: torch.Tensor, block_tables: torch.Tensor, token_starts: torch.Tensor,
                             num_tokens: int, *, first: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                             v_out: torch.Tensor | None = None, stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """``pda_gather_cache_slot_scales``: ``gather_cache`` with a scale per slot (float32 ``[NB, Hk, bs]``)."""
    lib = _lib or load()
    dev = k_cache.get_device()
    cs = k_cache.shape
    ok = (_e4m3_ok(k_cache, v_cache, dev) and k_scales.shape == (cs[0], cs[1], cs[3]) and v_scales.shape == k_scales.shape
          and k_scales.dtype is _F32 and v_scales.dtype is _F32 and k_scales.is_contiguous() and v_scales.is_contiguous()
          and dev == k_scales.get_device() == v_scales.get_device())
    k, v, S, MB, at = _gather_rows("gather_cache_slot_scales", block_tables, token_starts, first, num_tokens,
                                   cs[1] if ok else 0, k_out, v_out, dev, ok,
                                   lambda: _e4m3_checks(k_cache, v_cache) + _scale_checks(k_scales, v_scales, k_cache))
    st = lib.pda_gather_cache_slot_scales(k.data_ptr(), v.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(),
                                          k_scales.data_ptr(), v_scales.data_ptr(), block_tables.data_ptr(),
                                          token_starts.data_ptr(), at, num_tokens, S, cs[1], 128, cs[3], MB, cs[0],
                                          _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        raise PdaError(st, "pda_gather_cache_slot_scales")
    return k, v


def gather_cache_fp4(kv_cache: torch.Tensor, block_tables: torch.Tensor, token_starts: torch.Tensor, num_tokens: int,
                     k_scale: float, v_scale: float, *, first: torch.Tensor | None = None,
                     k_out: torch.Tensor | None = None, v_out: torch.Tensor | None = None,
                     stream=None) -> tuple[torch.Tensor, torch.Tensor]:
    """``pda_gather_cache_fp4``: ``gather_cache`` out of a 4-bit cache ``[NB, Hk, 144 * bs]``."""
    lib = _lib or load()
    dev = kv_cache.get_device()
    cs = kv_cache.shape
    ok = len(cs) == 3 and kv_cache.dtype is _U8 and kv_cache.is_contiguous() and cs[2] > 0 and cs[2] % 144 == 0
    k, v, S, MB, at = _gather_rows("gather_cache_fp4", block_tables, token_starts, first, num_tokens, cs[1] if ok else 0,
                                   k_out, v_out, dev, ok, lambda: _fp4_checks(kv_cache))
    st = lib.pda_gather_cache_fp4(k.data_ptr(), v.data_ptr(), kv_cache.data_ptr(), block_tables.data_ptr(),
                                  token_starts.data_ptr(), at, num_tokens, S, cs[1], 128, cs[2] // 144, MB, cs[0],
                                  k_scale, v_scale, _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        raise PdaError(st, "pda_gather_cache_fp4")
    return k, v


def decode_fp4(q: torch.Tensor, kv_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
               k_scale: float, v_scale: float, *, window: int = 0, sinks: torch.Tensor | None = None,
               output_scale: float | None = None, out: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """``pda_decode_fp4``: decode attention over a 4-bit cache ``[NB, Hk, 144 * bs]``.

    q ``[S, H, 128]`` bf16, block_tables ``[S, MB]`` and seq_lens ``[S]``
    int32, sinks and output_scale as for ``decode_ex``. ``window`` > 0 limits a
    sequence to its last ``window`` tokens. The first call on a stream makes its
    workspace; ``reserve_fp4`` does so ahead of a capture.
    """
    lib = _lib or load()
    dev = q.get_device()
    qs, cs, bt = q.shape, kv_cache.shape, block_tables.shape
    if not (len(qs) == 3 and len(cs) == 3 and len(bt) == 2 and bt[0] == qs[0] and seq_lens.shape == qs[:1]
            and q.dtype is _BF16 and kv_cache.dtype is _U8 and block_tables.dtype is _I32 and seq_lens.dtype is _I32
            and q.is_contiguous() and kv_cache.is_contiguous() and block_tables.is_contiguous()
            and seq_lens.is_contiguous() and cs[2] and cs[2] % 144 == 0
            and 0 <= dev == kv_cache.get_device() == block_tables.get_device() == seq_lens.get_device() == _device()):
        _say_why("decode_fp4", [
            (lambda: len(qs) == 3 and q.dtype is _BF16 and q.is_contiguous(), "q must be contiguous bf16 [S, H, 128]")]
            + _fp4_checks(kv_cache) + [
            (lambda: len(bt) == 2 and bt[0] == qs[0] and seq_lens.shape == qs[:1], "block_tables [S, MB] and seq_lens [S]"),
            (lambda: all(t.dtype is _I32 and t.is_contiguous() for t in (block_tables, seq_lens)),
             "block_tables and seq_lens must be contiguous int32")])
    fp8 = output_scale is not None
    if out is None:
        out = torch.empty_like(q, dtype=torch.float8_e4m3fn) if fp8 else torch.empty_like(q)
    elif not (out.shape == qs and out.dtype in (_CACHE_TYPES if fp8 else (_BF16,)) and out.is_contiguous()
              and out.get_device() == dev):
        _refuse("decode_fp4: out")
    if sinks is not None and not (sinks.dtype is _F32 and sinks.shape == qs[1:2] and sinks.is_contiguous()
                                  and sinks.get_device() == dev):
        _refuse("decode_fp4: sinks must be a contiguous float32 [num_heads] tensor on q's device")
    st = lib.pda_decode_fp4(out.data_ptr(), q.data_ptr(), kv_cache.data_ptr(), block_tables.data_ptr(),
                            seq_lens.data_ptr(), qs[0], qs[1], cs[1], qs[2], cs[2] // 144, bt[1], cs[0], scale, k_scale,
                            v_scale, window, None if sinks is None else sinks.data_ptr(),
                            PDA_OUT_E4M3 if fp8 else PDA_OUT_BF16, output_scale if fp8 else 1.0,
                            _raw_stream(dev) if stream is None else _stream_ptr(stream))
    if st:
        raise PdaError(st, "pda_decode_fp4")
    return out


def reserve_fp4(stream=None) -> None:
    """``pda_reserve_fp4``: make ``decode_fp4``'s workspace of the stream (before its first capture)."""
    _check(load().pda_reserve_fp4(_stream_ptr(stream)), "pda_reserve_fp4")
