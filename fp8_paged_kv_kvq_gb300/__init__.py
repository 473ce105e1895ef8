"""fp8_paged_kv_kvq_gb300 -- an FP8 E4M3 paged KV cache for NVIDIA GB300.

Python binding of ``libkvq.so`` (C ABI: ``include/kvq.h``).  Every function
here only marshals arguments -- PyTorch tensors in, raw device pointers, sizes
and the current CUDA stream out -- and calls the C entry point of the same
name; all computation happens in the library's sm_103a kernels.  There is no
fallback: if the library has not been built, or a call returns an error status,
a ``KvqError`` is raised.

Row format (ROCm/ATOM PR #2655 "fix(qwen4-exp): register the QSA FP8 scale
planes for KV offload", PR description; FlashML-org/FreeToken PR #354
"feat(kvcache): store the KV cache as fp8 e4m3 codes", PR description): every
cached (token, KV head) row of K or V is head_dim e4m3 bytes, in a uint8 buffer
shaped like the 16-bit cache, and one fp32 scale = row amax / 448.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading
from dataclasses import dataclass

import torch

__all__ = [
    "KvqError", "Cache", "load", "abi_version", "cache_bytes", "quantize_scatter",
    "paged_decode", "paged_decode_partials", "paged_decode_combine",
    "paged_decode_workspace_size", "paged_decode_partition_tokens", "dequant_rows",
    "header_functions", "LIB_PATH", "HEADER_PATH",
    "IndexCache", "INDEX_FP8", "INDEX_MXFP4", "index_cache_bytes", "index_quantize_scatter",
    "index_dequant_rows",
    "ERRF_SLOT_RANGE", "ERRF_BLOCK_RANGE", "ERRF_CONTEXT_RANGE",
    "CODES_E4M3", "CODES_E5M2", "quantize_scatter_unscaled", "paged_decode_codes",
    "paged_decode_codes_workspace_size",
    "ERRF_POSITION_RANGE", "ERRF_SEQUENCE_RANGE", "ROPE_HALVES", "ROPE_INTERLEAVED",
    "rope_quantize_scatter", "prompt_attention",
    "paged_decode_window", "paged_decode_window_workspace_size", "paged_decode_tree",
    "paged_decode_tree_workspace_size", "tree_commit", "PagePool", "pages_alloc", "pages_free",
    "pages_fork", "ERRF_PATH_RANGE", "ERRF_NO_PAGES", "ERRF_PAGE_STATE",
]

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "_build", "libkvq.so")
HEADER_PATH = os.path.join(os.path.dirname(_PKG), "include", "kvq.h")

INDEX_FP8 = 0
INDEX_MXFP4 = 1

CODES_E4M3 = 0
CODES_E5M2 = 1

ERRF_SLOT_RANGE = 1
ERRF_BLOCK_RANGE = 2
ERRF_CONTEXT_RANGE = 4
ERRF_POSITION_RANGE = 16
ERRF_SEQUENCE_RANGE = 32
ERRF_PATH_RANGE = 64
ERRF_NO_PAGES = 128
ERRF_PAGE_STATE = 256

ROPE_HALVES = 0
ROPE_INTERLEAVED = 1

_STATUS = {0: "KVQ_OK", 1: "KVQ_ERR_INVALID_ARGUMENT", 2: "KVQ_ERR_UNSUPPORTED",
           3: "KVQ_ERR_MISALIGNED", 4: "KVQ_ERR_WORKSPACE_TOO_SMALL", 5: "KVQ_ERR_CUDA"}


class KvqError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {_STATUS.get(status, status)} "
                         f"({load().kvq_status_string(status).decode()})")


class _CacheStruct(ctypes.Structure):
    _fields_ = [("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
                ("k_scales", ctypes.c_void_p), ("v_scales", ctypes.c_void_p),
                ("num_slots", ctypes.c_int64), ("num_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32)]


class _PagePoolStruct(ctypes.Structure):
    _fields_ = [("ref_counts", ctypes.c_void_p), ("free_pages", ctypes.c_void_p),
                ("state", ctypes.c_void_p), ("marks", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32)]


class _IndexCacheStruct(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("exponents", ctypes.c_void_p), ("num_slots", ctypes.c_int64),
                ("format", ctypes.c_int32), ("dim", ctypes.c_int32)]


_lock = threading.Lock()
_lib = None


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libkvq.so (built by ``fp8_paged_kv_kvq_gb300.build.build()``)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError(
                f"libkvq.so not found at {p}: build it with "
                "`python -c 'import __graft_entry__ as g; g.build()'` "
                "(or fp8_paged_kv_kvq_gb300/build.py); there is no CPU fallback")
        lib = ctypes.CDLL(p)
        P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
        CP = ctypes.POINTER(_CacheStruct)
        PP = ctypes.POINTER(_PagePoolStruct)
        sigs = {
            "kvq_status_string": (ctypes.c_char_p, [ctypes.c_int]),
            "kvq_abi_version": (i32, []),
            "kvq_cache_bytes": (sz, [i64, i32, i32]),
            "kvq_quantize_scatter": (ctypes.c_int, [CP, P, i64, P, i64, i64, P, P, P]),
            "kvq_rope_quantize_scatter": (ctypes.c_int, [CP, P, i64, i32, P, i64, P, i64, i64, P,
                                                         P, i64, i32, i32, P, P, i64, P, i64, P,
                                                         P]),
            "kvq_prompt_attention": (ctypes.c_int, [P, i64, P, i64, P, i64, i64, P, i32, i32, i32,
                                                    i32, i32, ctypes.c_float, P, i64, P, P]),
            "kvq_paged_decode_partition_tokens": (i32, [i32, i32, i32, i32, i32, i32]),
            "kvq_paged_decode_workspace_size": (sz, [i32, i32, i32, i32, i32, i32, i32, i32]),
            "kvq_paged_decode": (ctypes.c_int, [CP, P, i32, i32, i32, P, i32, P, i32,
                                                ctypes.c_float, i32, P, P, sz, P, P]),
            "kvq_paged_decode_partials": (ctypes.c_int, [CP, P, i32, i32, i32, P, i32, P, i32,
                                                         ctypes.c_float, i32, P, P, sz, P, P]),
            "kvq_paged_decode_combine": (ctypes.c_int, [CP, i32, i32, i32, i32, P, i32, i32,
                                                        P, P, sz, P]),
            "kvq_paged_decode_append_partials": (ctypes.c_int, [CP, P, i64, P, i64, P, i32, i32,
                                                                i32, P, i32, P, i32,
                                                                ctypes.c_float, i32, P, P, sz,
                                                                P, P]),
            "kvq_paged_decode_append": (ctypes.c_int, [CP, P, i64, P, i64, P, i32, i32, i32, P,
                                                       i32, P, i32, ctypes.c_float, i32, P, P,
                                                       sz, P, P]),
            "kvq_paged_decode_window_workspace_size": (sz, [i32, i32, i32, i32, i32, i32, i32, i32,
                                                            i32]),
            "kvq_paged_decode_window": (ctypes.c_int, [CP, P, i32, i32, i32, P, i32, P, i32, i32,
                                                       i32, ctypes.c_float, P, P, sz, P, P]),
            "kvq_paged_decode_tree_workspace_size": (sz, [i32, i32, i32, i32, i32, i32, i32]),
            "kvq_paged_decode_tree": (ctypes.c_int, [CP, P, P, i32, i32, i32, P, i32, P, i32,
                                                     ctypes.c_float, P, P, sz, P, P]),
            "kvq_tree_commit": (ctypes.c_int, [CP, P, P, i32, i32, P, i32, P, P, P, P]),
            "kvq_pages_alloc": (ctypes.c_int, [PP, P, i32, i32, P, P, P, P]),
            "kvq_pages_free": (ctypes.c_int, [PP, P, i32, i32, P, P, P, P]),
            "kvq_pages_fork": (ctypes.c_int, [CP, PP, P, i32, P, i32, i32, P, P, P, P, P]),
            "kvq_dequant_rows": (ctypes.c_int, [CP, P, i64, i32, P, P, P, P]),
            "kvq_quantize_scatter_unscaled": (ctypes.c_int, [CP, i32, P, i64, P, i64, i64, P,
                                                             P, P]),
            "kvq_paged_decode_codes_workspace_size": (sz, [i32, i32, i32, i32, i32, i32, i32]),
            "kvq_paged_decode_codes": (ctypes.c_int, [CP, i32, P, i32, i32, i32, P, i32, P, i32,
                                                      ctypes.c_float, P, P, sz, P, P]),
            "kvq_index_cache_bytes": (sz, [i64, i32, i32]),
            "kvq_index_quantize_scatter": (ctypes.c_int, [ctypes.POINTER(_IndexCacheStruct), P,
                                                          i64, i64, P, P, P]),
            "kvq_index_dequant_rows": (ctypes.c_int, [ctypes.POINTER(_IndexCacheStruct), P, i64,
                                                      i32, P, P, P]),
            "kvq_index_scores": (ctypes.c_int, [ctypes.POINTER(_IndexCacheStruct), i32, P, i32,
                                                i32, i32, P, i32, P, i32, P, P, P]),
        }
        for name, (res, args) in sigs.items():
            fn = getattr(lib, name)
            fn.restype = res
            fn.argtypes = args
        _lib = lib
        return lib


def header_functions(path: str = HEADER_PATH) -> list[str]:
    """Names of the functions declared in include/kvq.h."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(kvq_[a-z0-9_]+)\s*\(", text)))


def _check(status: int, where: str):
    if status != 0:
        raise KvqError(status, where)


def _stream(stream) -> ctypes.c_void_p:
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _current_stream_handle(device: int) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _torch_call(name: str, public):
    """torch's own call ``name`` without the checks and objects that ``public`` puts around
    it (1 us each, of 11 for a rotary store), or ``public`` where torch has none."""
    return getattr(torch._C, name, public)


_get_device = _torch_call("_cuda_getDevice", torch.cuda.current_device)
_get_raw_stream = _torch_call("_cuda_getCurrentRawStream", _current_stream_handle)


def _raw_stream(stream, device: int) -> int:
    """The cudaStream_t of ``stream``, or of ``device``'s current one."""
    if stream is None:
        return _get_raw_stream(device)
    if stream.device_index != device:
        raise ValueError(f"stream of device {stream.device_index}, not of the current one ({device})")
    return stream.cuda_stream


def _ptr(t) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


@dataclass
class Cache:
    """Device tensors of one FP8 paged cache; codes and scales travel together.

    k_codes, v_codes: uint8 [num_slots, num_kv_heads, head_dim]
    k_scales, v_scales: float32 [num_slots, num_kv_heads]"""
    k_codes: torch.Tensor
    v_codes: torch.Tensor
    k_scales: torch.Tensor
    v_scales: torch.Tensor
    block_size: int

    @staticmethod
    def empty(num_slots: int, num_kv_heads: int, head_dim: int = 128, block_size: int = 16,
              device="cuda") -> "Cache":
        return Cache(
            torch.zeros(num_slots, num_kv_heads, head_dim, dtype=torch.uint8, device=device),
            torch.zeros(num_slots, num_kv_heads, head_dim, dtype=torch.uint8, device=device),
            torch.zeros(num_slots, num_kv_heads, dtype=torch.float32, device=device),
            torch.zeros(num_slots, num_kv_heads, dtype=torch.float32, device=device),
            block_size)

    @property
    def num_slots(self) -> int:
        return self.k_codes.shape[0]

    @property
    def num_kv_heads(self) -> int:
        return self.k_codes.shape[1]

    @property
    def head_dim(self) -> int:
        return self.k_codes.shape[2]

    def struct(self) -> _CacheStruct:
        kc, vc, ks, vs = self.k_codes, self.v_codes, self.k_scales, self.v_scales
        u8, f32 = torch.uint8, torch.float32
        if not (kc.dtype is u8 and vc.dtype is u8 and ks.dtype is f32 and vs.dtype is f32 and
                kc.is_contiguous() and vc.is_contiguous() and ks.is_contiguous() and
                vs.is_contiguous()):
            raise ValueError("cache tensors must be contiguous uint8 codes / fp32 scales")
        shape = kc.shape
        return _CacheStruct(kc.data_ptr(), vc.data_ptr(), ks.data_ptr(), vs.data_ptr(),
                            shape[0], shape[1], shape[2], self.block_size)


def abi_version() -> int:
    return load().kvq_abi_version()


def cache_bytes(num_slots: int, num_kv_heads: int, head_dim: int = 128) -> int:
    return load().kvq_cache_bytes(num_slots, num_kv_heads, head_dim)


def _rows_view(x: torch.Tensor, H: int, D: int, name: str) -> int:
    """Token stride (elements) of a [T, H, D] (or [T, H*D]) bf16 view whose rows
    are contiguous within a token."""
    if x.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16")
    if x.dim() == 2:
        if x.shape[1] != H * D or x.stride(1) != 1:
            raise ValueError(f"{name}: expected [T, {H * D}] with unit inner stride")
    elif x.dim() == 3:
        if tuple(x.shape[1:]) != (H, D) or x.stride(2) != 1 or x.stride(1) != D:
            raise ValueError(f"{name}: expected [T, {H}, {D}] with contiguous heads")
    else:
        raise ValueError(f"{name}: expected a 2-D or 3-D view")
    return x.stride(0)


def quantize_scatter(cache: Cache, k: torch.Tensor, v: torch.Tensor, slot_ids: torch.Tensor,
                     err_flags: torch.Tensor | None = None, stream=None) -> None:
    """kvq_quantize_scatter: quantise bf16 K/V rows [T, H, D] (views allowed,
    each with its own token stride) into ``cache`` at device int64 ``slot_ids``."""
    H, D = cache.num_kv_heads, cache.head_dim
    ks = _rows_view(k, H, D, "k")
    vs = _rows_view(v, H, D, "v")
    T = k.shape[0]
    if v.shape[0] != T or slot_ids.numel() != T or slot_ids.dtype != torch.int64:
        raise ValueError("k, v and slot_ids (int64) must have the same token count")
    st = cache.struct()
    _check(load().kvq_quantize_scatter(ctypes.byref(st), _ptr(k), ks, _ptr(v), vs, T,
                                       _ptr(slot_ids), _ptr(err_flags), _stream(stream)),
           "kvq_quantize_scatter")


# The operators from here to pages_fork are called once per layer or step, on few
# tokens too, so their checks keep to a few tensor attribute reads each.

def _heads(x: torch.Tensor, name: str, T: int, heads: int, D: int) -> int:
    """Token stride (elements) of a bf16 view [T, heads, D] whose rows are
    contiguous within a token (of one token: the stride it would have)."""
    if x.dtype is not torch.bfloat16 or x.shape != (T, heads, D):
        raise ValueError(f"{name} must be a bfloat16 view [{T}, {heads}, {D}], "
                         f"not {x.dtype} {tuple(x.shape)}")
    s0, s1, s2 = x.stride()
    if T and (s2 != 1 or (heads > 1 and s1 != D)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    return s0 if T > 1 else heads * D


def _flat(x: torch.Tensor, name: str, dtype, n: int) -> None:
    if x.dtype is not dtype or x.numel() != n or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} with {n} entries")


def _one_device(tensors) -> int:
    """The index of the current CUDA device, on which every tensor (None: not
    given) has to be: a pointer of the host or of another device would fault in
    the kernel."""
    device = _get_device() if torch.cuda.is_initialized() else None
    for t in tensors:
        if t is not None and t.get_device() != device:
            raise ValueError(f"every tensor must be on the current CUDA device ({device}), "
                             f"not on {t.device}")
    return device


def _rows_like(x: torch.Tensor, stream) -> torch.Tensor:
    """An output like ``x``, allocated on the stream that writes it: memory that
    another stream has freed may still be read by work queued there."""
    if stream is None:
        return torch.empty(x.shape, dtype=x.dtype, device=x.device)
    with torch.cuda.stream(stream):
        return torch.empty(x.shape, dtype=x.dtype, device=x.device)


def _addr(t) -> int:
    return 0 if t is None else t.data_ptr()


def _flags(err_flags) -> None:
    if err_flags is not None and (err_flags.dtype is not torch.int32 or err_flags.numel() < 1):
        raise ValueError("err_flags must be an int32 tensor of one element")


def rope_quantize_scatter(cache: Cache, q: torch.Tensor | None, k: torch.Tensor, v: torch.Tensor,
                          positions: torch.Tensor, rope_table: torch.Tensor,
                          slot_ids: torch.Tensor, layout: int = ROPE_HALVES,
                          q_out: torch.Tensor | None = None, k_out: torch.Tensor | None = None,
                          err_flags: torch.Tensor | None = None,
                          stream=None) -> torch.Tensor | None:
    """kvq_rope_quantize_scatter: rotate query rows [T, Hq, D] and key rows
    [T, H, D] by their int64 ``positions`` in ``rope_table`` (fp32 [P, rotary_dim]:
    cosines, then sines) and quantise the rotated keys and the values into
    ``cache`` at int64 ``slot_ids``.  The rotated queries go to ``q_out`` (may be
    ``q`` itself; allocated here, by PyTorch on the call's stream, when not
    given), the rotated keys also to ``k_out`` where given (may be ``k``).  Rows
    of skipped tokens (slot id < 0) are not written.  Returns ``q_out`` (None
    without ``q``)."""
    T, (_, H, D) = k.shape[0], cache.k_codes.shape
    ks, vs = _heads(k, "k", T, H, D), _heads(v, "v", T, H, D)
    kos = 0 if k_out is None else _heads(k_out, "k_out", T, H, D)
    _flat(positions, "positions", torch.int64, T)
    _flat(slot_ids, "slot_ids", torch.int64, T)
    if rope_table.dtype is not torch.float32 or rope_table.dim() != 2 or \
            not rope_table.is_contiguous():
        raise ValueError("rope_table must be contiguous fp32 [positions, rotary_dim]")
    qs = qos = hq = 0
    if q is not None:
        if q.dim() != 3:
            raise ValueError(f"q must be a bfloat16 view [{T}, num_q_heads, {D}]")
        hq = q.shape[1]
        qs = _heads(q, "q", T, hq, D)
        if q_out is None:
            q_out = _rows_like(q, stream)
        qos = _heads(q_out, "q_out", T, hq, D)
    elif q_out is not None:
        raise ValueError("q_out without q")
    _flags(err_flags)
    device = _one_device((k, v, positions, rope_table, slot_ids, q, q_out, k_out, err_flags,
                          cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales))
    st = cache.struct()
    P, r = rope_table.shape
    status = load().kvq_rope_quantize_scatter(
        ctypes.byref(st), _addr(q), qs, hq, k.data_ptr(), ks, v.data_ptr(), vs, T,
        positions.data_ptr(), rope_table.data_ptr(), P, r, layout, slot_ids.data_ptr(),
        _addr(q_out), qos, _addr(k_out), kos, _addr(err_flags), _raw_stream(stream, device))
    if status:
        raise KvqError(status, "kvq_rope_quantize_scatter")
    return q_out


def prompt_attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, cu_seqlens: torch.Tensor,
                     max_seqlen: int, sm_scale: float, out: torch.Tensor | None = None,
                     err_flags: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvq_prompt_attention: causal attention of packed prompts -- bf16 queries
    [T, Hq, D] over keys and values [T, H, D] (views with their own token
    strides), sequence s holding the tokens cu_seqlens[s] .. cu_seqlens[s + 1] - 1
    (int32, on the device).  Returns ``out`` (bf16, shape of q; allocated here,
    by PyTorch on the call's stream, when not given).  Rows outside the sequences
    are not written."""
    if q.dim() != 3 or k.dim() != 3:
        raise ValueError("q, k and v must be bfloat16 views [T, heads, head_dim]")
    T, Hq, D = q.shape
    H = k.shape[1]
    qs, ks, vs = _heads(q, "q", T, Hq, D), _heads(k, "k", T, H, D), _heads(v, "v", T, H, D)
    if cu_seqlens.dim() != 1 or cu_seqlens.numel() < 1:
        raise ValueError("cu_seqlens must be int32 [num_seqs + 1]")
    N = cu_seqlens.numel() - 1
    _flat(cu_seqlens, "cu_seqlens", torch.int32, N + 1)
    if out is None:
        out = _rows_like(q, stream)
    outs = _heads(out, "out", T, Hq, D)
    _flags(err_flags)
    device = _one_device((q, k, v, cu_seqlens, out, err_flags))
    status = load().kvq_prompt_attention(
        q.data_ptr(), qs, k.data_ptr(), ks, v.data_ptr(), vs, T, cu_seqlens.data_ptr(), N,
        max_seqlen, Hq, H, D, sm_scale, out.data_ptr(), outs, _addr(err_flags),
        _raw_stream(stream, device))
    if status:
        raise KvqError(status, "kvq_prompt_attention")
    return out


def _int32(n: int) -> int:
    """n, or the nearest number that 32 bits hold: ctypes would drop the upper bits of a
    window that means all tokens (2**32 + 5: five)."""
    return n if -0x80000000 <= n <= 0x7FFFFFFF else (0x7FFFFFFF if n > 0 else -0x80000000)


def _masked_args(cache: Cache, q, block_tables, context_lens, R: int):
    """Requests, query heads, KV heads and table width of a windowed or tree call."""
    if q.dtype is not torch.bfloat16 or q.dim() != 3 or not q.is_contiguous():
        raise ValueError("q must be contiguous bfloat16 [num_requests * R, num_q_heads, head_dim]")
    if block_tables.dtype is not torch.int32 or block_tables.dim() != 2 or \
            not block_tables.is_contiguous():
        raise ValueError("block_tables must be contiguous int32 [num_requests, max_blocks]")
    n, width = block_tables.shape
    rows, hq, d = q.shape
    _, h, cd = cache.k_codes.shape
    if R < 1 or rows != n * R or d != cd:
        raise ValueError(f"q must have num_requests * R = {n} * {R} rows of {cd} dims")
    _flat(context_lens, "context_lens", torch.int32, n)
    return n, hq, h, width


def _masked_out(q, out, workspace, size: int, stream):
    """The output and the workspace (address and bytes) of a call; both are
    allocated on the stream that writes them when not given."""
    if out is None:
        out = _rows_like(q, stream)
    elif out.dtype is not torch.bfloat16 or out.shape != q.shape or not out.is_contiguous():
        raise ValueError("out must be contiguous bfloat16 of q's shape")
    if workspace is None:
        if stream is None:
            workspace = torch.empty(max(size, 1), dtype=torch.uint8, device=q.device)
        else:
            with torch.cuda.stream(stream):
                workspace = torch.empty(max(size, 1), dtype=torch.uint8, device=q.device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    return out, workspace


def paged_decode_window_workspace_size(num_requests: int, rows_per_request: int, num_q_heads: int,
                                       num_kv_heads: int, head_dim: int, block_size: int,
                                       max_context_len: int, window: int,
                                       num_sinks: int = 0) -> int:
    return load().kvq_paged_decode_window_workspace_size(
        num_requests, rows_per_request, num_q_heads, num_kv_heads, head_dim, block_size,
        _int32(max_context_len), _int32(window), _int32(num_sinks))


def paged_decode_window(cache: Cache, q: torch.Tensor, block_tables: torch.Tensor,
                        context_lens: torch.Tensor, max_context_len: int, window: int,
                        sm_scale: float, num_sinks: int = 0, rows_per_request: int = 1,
                        out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                        err_flags: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvq_paged_decode_window: paged_decode in which each row sees only the last
    ``window`` tokens up to its own and the first ``num_sinks``; block-table
    entries of tokens that no row of a request sees may hold anything.  Returns
    ``out`` (bf16, shape of q); ``out`` and ``workspace`` (uint8, >=
    paged_decode_window_workspace_size) are allocated here when not given."""
    R = rows_per_request
    n, hq, h, width = _masked_args(cache, q, block_tables, context_lens, R)
    max_context_len, window, num_sinks = _int32(max_context_len), _int32(window), _int32(num_sinks)
    lib = load()
    size = 0 if workspace is not None else lib.kvq_paged_decode_window_workspace_size(
        n, R, hq, h, 128, cache.block_size, max_context_len, window, num_sinks)
    out, workspace = _masked_out(q, out, workspace, size, stream)
    _flags(err_flags)
    device = _one_device((q, block_tables, context_lens, out, workspace, err_flags,
                          cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales))
    st = cache.struct()
    status = lib.kvq_paged_decode_window(
        ctypes.byref(st), q.data_ptr(), n, R, hq, block_tables.data_ptr(), width,
        context_lens.data_ptr(), max_context_len, window, num_sinks, sm_scale, out.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, _addr(err_flags), _raw_stream(stream, device))
    if status:
        raise KvqError(status, "kvq_paged_decode_window")
    return out


def paged_decode_tree_workspace_size(num_requests: int, rows_per_request: int, num_q_heads: int,
                                     num_kv_heads: int, head_dim: int, block_size: int,
                                     max_context_len: int) -> int:
    return load().kvq_paged_decode_tree_workspace_size(
        num_requests, rows_per_request, num_q_heads, num_kv_heads, head_dim, block_size,
        _int32(max_context_len))


def paged_decode_tree(cache: Cache, q: torch.Tensor, tree_mask: torch.Tensor,
                      block_tables: torch.Tensor, context_lens: torch.Tensor,
                      max_context_len: int, sm_scale: float, rows_per_request: int,
                      out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                      err_flags: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvq_paged_decode_tree: attention of ``rows_per_request`` drafted tokens, the
    last cached ones of each request, over the context before them and the drafted
    tokens whose bit ``tree_mask`` (int32 [num_requests, R, ceil(R / 32)], bit
    b % 32 of word b / 32) sets for the row.  Returns ``out`` (bf16, shape of q);
    ``out`` and ``workspace`` as for paged_decode_window."""
    R = rows_per_request
    n, hq, h, width = _masked_args(cache, q, block_tables, context_lens, R)
    _flat(tree_mask, "tree_mask", torch.int32, n * R * ((R + 31) // 32))
    max_context_len = _int32(max_context_len)
    lib = load()
    size = 0 if workspace is not None else lib.kvq_paged_decode_tree_workspace_size(
        n, R, hq, h, 128, cache.block_size, max_context_len)
    out, workspace = _masked_out(q, out, workspace, size, stream)
    _flags(err_flags)
    device = _one_device((q, tree_mask, block_tables, context_lens, out, workspace, err_flags,
                          cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales))
    st = cache.struct()
    status = lib.kvq_paged_decode_tree(
        ctypes.byref(st), q.data_ptr(), tree_mask.data_ptr(), n, R, hq, block_tables.data_ptr(),
        width, context_lens.data_ptr(), max_context_len, sm_scale, out.data_ptr(),
        workspace.data_ptr(), workspace.nbytes, _addr(err_flags), _raw_stream(stream, device))
    if status:
        raise KvqError(status, "kvq_paged_decode_tree")
    return out


def _table(x: torch.Tensor, name: str):
    if x.dtype is not torch.int32 or x.dim() != 2 or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32 [requests, max_blocks]")
    return x.shape


def tree_commit(cache: Cache, accepted: torch.Tensor, accepted_lens: torch.Tensor,
                block_tables: torch.Tensor, context_lens: torch.Tensor,
                new_lens: torch.Tensor | None = None, err_flags: torch.Tensor | None = None,
                stream=None) -> torch.Tensor:
    """kvq_tree_commit: the cache rows of the accepted drafted tokens (``accepted``
    int32 [N, R], ``accepted_lens`` int32 [N]) moved together behind each request's
    context.  Returns ``new_lens`` (int32 [N]: the context and the accepted tokens;
    may be ``context_lens`` itself; allocated here when not given)."""
    n, R = _table(accepted, "accepted")
    tn, width = _table(block_tables, "block_tables")
    if tn != n:
        raise ValueError("accepted and block_tables must have a row per request")
    _flat(accepted_lens, "accepted_lens", torch.int32, n)
    _flat(context_lens, "context_lens", torch.int32, n)
    if new_lens is None:
        new_lens = _rows_like(context_lens, stream)
    _flat(new_lens, "new_lens", torch.int32, n)
    _flags(err_flags)
    device = _one_device((accepted, accepted_lens, block_tables, context_lens, new_lens, err_flags,
                          cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales))
    st = cache.struct()
    status = load().kvq_tree_commit(
        ctypes.byref(st), accepted.data_ptr(), accepted_lens.data_ptr(), n, R,
        block_tables.data_ptr(), width, context_lens.data_ptr(), new_lens.data_ptr(),
        _addr(err_flags), _raw_stream(stream, device))
    if status:
        raise KvqError(status, "kvq_tree_commit")
    return new_lens


@dataclass
class PagePool:
    """Device tensors of a pool of pages (kvq_page_pool); int32 all.

    ref_counts: [num_pages], block tables that hold each page
    free_pages: [num_pages], a stack whose first state[0] entries are the free pages
    state: [4], the free pages' number first
    marks: [ceil(num_pages / 32)], zero between calls"""
    ref_counts: torch.Tensor
    free_pages: torch.Tensor
    state: torch.Tensor
    marks: torch.Tensor

    @staticmethod
    def empty(num_pages: int, device="cuda") -> "PagePool":
        """A pool whose pages are all free; the top of its stack is the last page."""
        def zeros(n):
            return torch.zeros(n, dtype=torch.int32, device=device)
        state = zeros(4)
        state[0] = num_pages
        return PagePool(zeros(num_pages), torch.arange(num_pages, dtype=torch.int32, device=device),
                        state, zeros((num_pages + 31) // 32))

    @property
    def num_pages(self) -> int:
        return self.ref_counts.shape[0]

    def tensors(self):
        return self.ref_counts, self.free_pages, self.state, self.marks

    def struct(self) -> _PagePoolStruct:
        refs, free, state, marks = self.tensors()
        n = refs.numel()
        _flat(refs, "ref_counts", torch.int32, n)
        _flat(free, "free_pages", torch.int32, n)
        _flat(state, "state", torch.int32, 4)
        _flat(marks, "marks", torch.int32, (n + 31) // 32)
        return _PagePoolStruct(refs.data_ptr(), free.data_ptr(), state.data_ptr(),
                               marks.data_ptr(), n)


def _page_ranges(name: str, pool: PagePool, block_tables, begin, end, err_flags, stream) -> None:
    n, width = _table(block_tables, "block_tables")
    _flat(begin, "begin", torch.int32, n)
    _flat(end, "end", torch.int32, n)
    _flags(err_flags)
    st = pool.struct()
    device = _one_device((*pool.tensors(), block_tables, begin, end, err_flags))
    status = getattr(load(), name)(ctypes.byref(st), block_tables.data_ptr(), n, width,
                                   begin.data_ptr(), end.data_ptr(), _addr(err_flags),
                                   _raw_stream(stream, device))
    if status:
        raise KvqError(status, name)


def pages_alloc(pool: PagePool, block_tables: torch.Tensor, begin: torch.Tensor,
                end: torch.Tensor, err_flags: torch.Tensor | None = None, stream=None) -> None:
    """kvq_pages_alloc: a page of the pool for each of the entries [begin[r], end[r])
    (int32 [N]) of request r's block table."""
    _page_ranges("kvq_pages_alloc", pool, block_tables, begin, end, err_flags, stream)


def pages_free(pool: PagePool, block_tables: torch.Tensor, begin: torch.Tensor,
               end: torch.Tensor, err_flags: torch.Tensor | None = None, stream=None) -> None:
    """kvq_pages_free: one reference given back for each of the entries [begin[r],
    end[r]) of request r's block table (entries < 0 are skipped)."""
    _page_ranges("kvq_pages_free", pool, block_tables, begin, end, err_flags, stream)


def pages_fork(cache: Cache, pool: PagePool, parents: torch.Tensor, block_tables: torch.Tensor,
               context_lens: torch.Tensor, child_tables: torch.Tensor, child_lens: torch.Tensor,
               err_flags: torch.Tensor | None = None, stream=None) -> None:
    """kvq_pages_fork: child i continues the sequence of request ``parents[i]`` (int32
    [M]): its row of ``child_tables`` [M, max_blocks] shares the parent's full pages
    and gets a copy of a partly filled last one, ``child_lens[i]`` its length."""
    num_parents, width = _table(block_tables, "block_tables")
    m, child_width = _table(child_tables, "child_tables")
    if child_width != width:
        raise ValueError("child_tables must be as wide as block_tables")
    _flat(parents, "parents", torch.int32, m)
    _flat(context_lens, "context_lens", torch.int32, num_parents)
    _flat(child_lens, "child_lens", torch.int32, m)
    _flags(err_flags)
    ps = pool.struct()
    device = _one_device((*pool.tensors(), parents, block_tables, context_lens, child_tables,
                          child_lens, err_flags, cache.k_codes, cache.v_codes, cache.k_scales,
                          cache.v_scales))
    st = cache.struct()
    status = load().kvq_pages_fork(
        ctypes.byref(st), ctypes.byref(ps), parents.data_ptr(), m, block_tables.data_ptr(),
        num_parents, width, context_lens.data_ptr(), child_tables.data_ptr(),
        child_lens.data_ptr(), _addr(err_flags), _raw_stream(stream, device))
    if status:
        raise KvqError(status, "kvq_pages_fork")


def paged_decode_partition_tokens(num_requests: int, rows_per_request: int, num_q_heads: int,
                                  num_kv_heads: int, block_size: int,
                                  max_context_len: int) -> int:
    return load().kvq_paged_decode_partition_tokens(num_requests, rows_per_request, num_q_heads,
                                                    num_kv_heads, block_size, max_context_len)


def paged_decode_workspace_size(num_requests: int, rows_per_request: int, num_q_heads: int,
                                num_kv_heads: int, head_dim: int, block_size: int,
                                max_context_len: int, partition_tokens: int = 0) -> int:
    return load().kvq_paged_decode_workspace_size(num_requests, rows_per_request, num_q_heads,
                                                  num_kv_heads, head_dim, block_size,
                                                  max_context_len, partition_tokens)


def _decode_args(cache, q, block_tables, context_lens, rows_per_request):
    if q.dtype != torch.bfloat16 or not q.is_contiguous() or q.dim() != 3:
        raise ValueError("q must be a contiguous bf16 [num_requests*R, Hq, D] tensor")
    if block_tables.dtype != torch.int32 or not block_tables.is_contiguous():
        raise ValueError("block_tables must be contiguous int32 [N, max_blocks]")
    if context_lens.dtype != torch.int32 or not context_lens.is_contiguous():
        raise ValueError("context_lens must be contiguous int32 [N]")
    N = block_tables.shape[0]
    if q.shape[0] != N * rows_per_request or context_lens.numel() != N:
        raise ValueError("q rows must equal num_requests * rows_per_request")
    return N, q.shape[1], block_tables.shape[1]


def paged_decode(cache: Cache, q: torch.Tensor, block_tables: torch.Tensor,
                 context_lens: torch.Tensor, max_context_len: int, sm_scale: float,
                 rows_per_request: int = 1, partition_tokens: int = 0,
                 out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                 err_flags: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvq_paged_decode: paged GQA decode / verify attention; returns ``out``
    (bf16, shape of q).  ``workspace`` (uint8, >= paged_decode_workspace_size;
    no initialisation needed) is allocated here, by PyTorch, when not given."""
    N, Hq, mb = _decode_args(cache, q, block_tables, context_lens, rows_per_request)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        need = paged_decode_workspace_size(N, rows_per_request, Hq, cache.num_kv_heads,
                                           cache.head_dim, cache.block_size, max_context_len,
                                           partition_tokens)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = cache.struct()
    _check(load().kvq_paged_decode(ctypes.byref(st), _ptr(q), N, rows_per_request, Hq,
                                   _ptr(block_tables), mb, _ptr(context_lens), max_context_len,
                                   float(sm_scale), partition_tokens, _ptr(out), _ptr(workspace),
                                   workspace.numel(), _ptr(err_flags), _stream(stream)),
           "kvq_paged_decode")
    return out


def _append_rows(cache: Cache, k_new, v_new, n_rows: int):
    H, D = cache.num_kv_heads, cache.head_dim
    ks = _rows_view(k_new, H, D, "k_new")
    vs = _rows_view(v_new, H, D, "v_new")
    if k_new.shape[0] != n_rows or v_new.shape[0] != n_rows:
        raise ValueError("k_new and v_new need num_requests * rows_per_request rows")
    return ks, vs


def paged_decode_append(cache: Cache, k_new: torch.Tensor, v_new: torch.Tensor,
                        q: torch.Tensor, block_tables: torch.Tensor, context_lens: torch.Tensor,
                        max_context_len: int, sm_scale: float, rows_per_request: int = 1,
                        partition_tokens: int = 0, out: torch.Tensor | None = None,
                        workspace: torch.Tensor | None = None,
                        err_flags: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvq_paged_decode_append: one decode step -- the step's new K/V rows
    [N*R, H, D] (views allowed) stored at positions L_r - R + i of each
    request's block table, then the attention over the cache that holds them;
    returns ``out`` (bf16, shape of q)."""
    N, Hq, mb = _decode_args(cache, q, block_tables, context_lens, rows_per_request)
    ks, vs = _append_rows(cache, k_new, v_new, N * rows_per_request)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        need = paged_decode_workspace_size(N, rows_per_request, Hq, cache.num_kv_heads,
                                           cache.head_dim, cache.block_size, max_context_len,
                                           partition_tokens)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = cache.struct()
    _check(load().kvq_paged_decode_append(
        ctypes.byref(st), _ptr(k_new), ks, _ptr(v_new), vs, _ptr(q), N, rows_per_request, Hq,
        _ptr(block_tables), mb, _ptr(context_lens), max_context_len, float(sm_scale),
        partition_tokens, _ptr(out), _ptr(workspace), workspace.numel(), _ptr(err_flags),
        _stream(stream)), "kvq_paged_decode_append")
    return out


def paged_decode_append_partials(cache: Cache, k_new, v_new, q, block_tables, context_lens,
                                 max_context_len: int, sm_scale: float, rows_per_request: int,
                                 partition_tokens: int, out: torch.Tensor,
                                 workspace: torch.Tensor | None,
                                 err_flags: torch.Tensor | None = None, stream=None) -> None:
    """kvq_paged_decode_append_partials (the step's store and split-K launch;
    kvq_paged_decode_combine follows)."""
    N, Hq, mb = _decode_args(cache, q, block_tables, context_lens, rows_per_request)
    ks, vs = _append_rows(cache, k_new, v_new, N * rows_per_request)
    st = cache.struct()
    _check(load().kvq_paged_decode_append_partials(
        ctypes.byref(st), _ptr(k_new), ks, _ptr(v_new), vs, _ptr(q), N, rows_per_request, Hq,
        _ptr(block_tables), mb, _ptr(context_lens), max_context_len, float(sm_scale),
        partition_tokens, _ptr(out), _ptr(workspace),
        0 if workspace is None else workspace.numel(), _ptr(err_flags), _stream(stream)),
        "kvq_paged_decode_append_partials")


def paged_decode_partials(cache: Cache, q, block_tables, context_lens, max_context_len: int,
                          sm_scale: float, rows_per_request: int, partition_tokens: int,
                          out: torch.Tensor, workspace: torch.Tensor | None,
                          err_flags: torch.Tensor | None = None, stream=None) -> None:
    """kvq_paged_decode_partials (the split-K launch of kvq_paged_decode)."""
    N, Hq, mb = _decode_args(cache, q, block_tables, context_lens, rows_per_request)
    st = cache.struct()
    _check(load().kvq_paged_decode_partials(
        ctypes.byref(st), _ptr(q), N, rows_per_request, Hq, _ptr(block_tables), mb,
        _ptr(context_lens), max_context_len, float(sm_scale), partition_tokens, _ptr(out),
        _ptr(workspace), 0 if workspace is None else workspace.numel(), _ptr(err_flags),
        _stream(stream)), "kvq_paged_decode_partials")


def paged_decode_combine(cache: Cache, num_requests: int, rows_per_request: int,
                         num_q_heads: int, max_blocks_per_req: int, context_lens: torch.Tensor,
                         max_context_len: int, partition_tokens: int, out: torch.Tensor,
                         workspace: torch.Tensor | None, stream=None) -> None:
    """kvq_paged_decode_combine (the merge launch of kvq_paged_decode)."""
    st = cache.struct()
    _check(load().kvq_paged_decode_combine(
        ctypes.byref(st), num_requests, rows_per_request, num_q_heads, max_blocks_per_req,
        _ptr(context_lens), max_context_len, partition_tokens, _ptr(out), _ptr(workspace),
        0 if workspace is None else workspace.numel(), _stream(stream)),
        "kvq_paged_decode_combine")


def quantize_scatter_unscaled(cache: Cache, k: torch.Tensor, v: torch.Tensor,
                              slot_ids: torch.Tensor, code_format: int = CODES_E4M3,
                              err_flags: torch.Tensor | None = None, stream=None) -> None:
    """kvq_quantize_scatter_unscaled: cast bf16 K/V rows to e4m3 or e5m2 codes
    with no scale (scale planes set to 1) -- the codec ablation's caches."""
    H, D = cache.num_kv_heads, cache.head_dim
    ks = _rows_view(k, H, D, "k")
    vs = _rows_view(v, H, D, "v")
    T = k.shape[0]
    if v.shape[0] != T or slot_ids.numel() != T or slot_ids.dtype != torch.int64:
        raise ValueError("k, v and slot_ids (int64) must have the same token count")
    st = cache.struct()
    _check(load().kvq_quantize_scatter_unscaled(ctypes.byref(st), code_format, _ptr(k), ks,
                                                _ptr(v), vs, T, _ptr(slot_ids), _ptr(err_flags),
                                                _stream(stream)),
           "kvq_quantize_scatter_unscaled")


def paged_decode_codes_workspace_size(num_requests: int, rows_per_request: int,
                                      num_q_heads: int, num_kv_heads: int, head_dim: int,
                                      block_size: int, max_context_len: int) -> int:
    return load().kvq_paged_decode_codes_workspace_size(num_requests, rows_per_request,
                                                        num_q_heads, num_kv_heads, head_dim,
                                                        block_size, max_context_len)


def paged_decode_codes(cache: Cache, code_format: int, q: torch.Tensor,
                       block_tables: torch.Tensor, context_lens: torch.Tensor,
                       max_context_len: int, sm_scale: float, rows_per_request: int = 1,
                       out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                       err_flags: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvq_paged_decode_codes: paged attention over a cache of e4m3 or e5m2
    codes (the rows-on-M kernel for every shape); returns ``out``."""
    N, Hq, mb = _decode_args(cache, q, block_tables, context_lens, rows_per_request)
    if out is None:
        out = torch.empty_like(q)
    if workspace is None:
        need = paged_decode_codes_workspace_size(N, rows_per_request, Hq, cache.num_kv_heads,
                                                 cache.head_dim, cache.block_size,
                                                 max_context_len)
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    st = cache.struct()
    _check(load().kvq_paged_decode_codes(ctypes.byref(st), code_format, _ptr(q), N,
                                         rows_per_request, Hq, _ptr(block_tables), mb,
                                         _ptr(context_lens), max_context_len, float(sm_scale),
                                         _ptr(out), _ptr(workspace), workspace.numel(),
                                         _ptr(err_flags), _stream(stream)),
           "kvq_paged_decode_codes")
    return out


def dequant_rows(cache: Cache, slot_ids: torch.Tensor, out_dtype=torch.float32,
                 out_k: torch.Tensor | None = None, out_v: torch.Tensor | None = None,
                 err_flags: torch.Tensor | None = None, stream=None):
    """kvq_dequant_rows: fp32 or bf16 rows [n, H, D] of K and V at ``slot_ids``."""
    if slot_ids.dtype != torch.int64:
        raise ValueError("slot_ids must be int64")
    code = {torch.float32: 0, torch.bfloat16: 1}[out_dtype]
    n = slot_ids.numel()
    shape = (n, cache.num_kv_heads, cache.head_dim)
    if out_k is None:
        out_k = torch.empty(shape, dtype=out_dtype, device=cache.k_codes.device)
    if out_v is None:
        out_v = torch.empty(shape, dtype=out_dtype, device=cache.k_codes.device)
    st = cache.struct()
    _check(load().kvq_dequant_rows(ctypes.byref(st), _ptr(slot_ids), n, code, _ptr(out_k),
                                   _ptr(out_v), _ptr(err_flags), _stream(stream)),
           "kvq_dequant_rows")
    return out_k, out_v


# ---------------------------------------------------------------------------
# compressed index keys

@dataclass
class IndexCache:
    """Device tensors of an index-key cache (one row of ``dim`` values per slot).

    FP8:   codes uint8 [num_slots, dim], scales float32 [num_slots]
    MXFP4: codes uint8 [num_slots, dim/2] (E2M1 pairs), exponents uint8
           [num_slots, dim/32] (E8M0)"""
    format: int
    codes: torch.Tensor
    scales: torch.Tensor | None = None
    exponents: torch.Tensor | None = None

    @staticmethod
    def empty(num_slots: int, format: int, dim: int = 128, device="cuda") -> "IndexCache":
        if format == INDEX_FP8:
            return IndexCache(format,
                              torch.zeros(num_slots, dim, dtype=torch.uint8, device=device),
                              scales=torch.zeros(num_slots, dtype=torch.float32, device=device))
        if format == INDEX_MXFP4:
            return IndexCache(format,
                              torch.zeros(num_slots, dim // 2, dtype=torch.uint8, device=device),
                              exponents=torch.zeros(num_slots, dim // 32, dtype=torch.uint8,
                                                    device=device))
        raise ValueError("format must be INDEX_FP8 or INDEX_MXFP4")

    @property
    def num_slots(self) -> int:
        return self.codes.shape[0]

    @property
    def dim(self) -> int:
        return self.codes.shape[1] * (1 if self.format == INDEX_FP8 else 2)

    def struct(self) -> _IndexCacheStruct:
        for t in (self.codes, self.scales, self.exponents):
            if t is not None and not t.is_contiguous():
                raise ValueError("index cache tensors must be contiguous")
        return _IndexCacheStruct(self.codes.data_ptr(),
                                 0 if self.scales is None else self.scales.data_ptr(),
                                 0 if self.exponents is None else self.exponents.data_ptr(),
                                 self.num_slots, self.format, self.dim)


def index_cache_bytes(num_slots: int, format: int, dim: int = 128) -> int:
    return load().kvq_index_cache_bytes(num_slots, format, dim)


def index_quantize_scatter(cache: IndexCache, x: torch.Tensor, slot_ids: torch.Tensor,
                           err_flags: torch.Tensor | None = None, stream=None) -> None:
    """kvq_index_quantize_scatter: bf16 rows [T, dim] (a view with unit inner
    stride; any token stride) into ``cache`` at device int64 ``slot_ids``."""
    if x.dtype != torch.bfloat16 or x.dim() != 2 or x.shape[1] != cache.dim or x.stride(1) != 1:
        raise ValueError(f"x: expected bf16 [T, {cache.dim}] with unit inner stride")
    if slot_ids.dtype != torch.int64 or slot_ids.numel() != x.shape[0]:
        raise ValueError("slot_ids must be int64 with one id per row")
    st = cache.struct()
    _check(load().kvq_index_quantize_scatter(ctypes.byref(st), _ptr(x), x.stride(0), x.shape[0],
                                             _ptr(slot_ids), _ptr(err_flags), _stream(stream)),
           "kvq_index_quantize_scatter")


def index_dequant_rows(cache: IndexCache, slot_ids: torch.Tensor, out_dtype=torch.float32,
                       err_flags: torch.Tensor | None = None, stream=None) -> torch.Tensor:
    """kvq_index_dequant_rows: fp32 or bf16 rows [n, dim] at ``slot_ids``."""
    if slot_ids.dtype != torch.int64:
        raise ValueError("slot_ids must be int64")
    code = {torch.float32: 0, torch.bfloat16: 1}[out_dtype]
    n = slot_ids.numel()
    out = torch.empty((n, cache.dim), dtype=out_dtype, device=cache.codes.device)
    st = cache.struct()
    _check(load().kvq_index_dequant_rows(ctypes.byref(st), _ptr(slot_ids), n, code, _ptr(out),
                                         _ptr(err_flags), _stream(stream)),
           "kvq_index_dequant_rows")
    return out


def index_scores(cache: IndexCache, block_size: int, q: torch.Tensor, block_tables: torch.Tensor,
                 context_lens: torch.Tensor, max_context_len: int,
                 out: torch.Tensor | None = None, err_flags: torch.Tensor | None = None,
                 stream=None) -> torch.Tensor:
    """kvq_index_scores: stacked index scores fp32 [N * R, max_context_len] for
    bf16 queries ``q`` [N, R, H, dim] over the paged index keys; -inf where a
    row does not see a token."""
    if q.dtype != torch.bfloat16 or not q.is_contiguous() or q.dim() != 4 \
            or q.shape[3] != cache.dim:
        raise ValueError(f"q must be a contiguous bf16 [N, R, H, {cache.dim}] tensor")
    if block_tables.dtype != torch.int32 or not block_tables.is_contiguous():
        raise ValueError("block_tables must be contiguous int32 [N, max_blocks]")
    if context_lens.dtype != torch.int32 or not context_lens.is_contiguous():
        raise ValueError("context_lens must be contiguous int32 [N]")
    N, R, H = q.shape[0], q.shape[1], q.shape[2]
    if block_tables.shape[0] != N or context_lens.numel() != N:
        raise ValueError("block_tables / context_lens must have one entry per request")
    if out is None:
        out = torch.empty((N * R, max_context_len), dtype=torch.float32, device=q.device)
    elif out.dtype != torch.float32 or not out.is_contiguous() \
            or tuple(out.shape) != (N * R, max_context_len):
        raise ValueError("out must be contiguous fp32 [N * R, max_context_len]")
    st = cache.struct()
    _check(load().kvq_index_scores(ctypes.byref(st), block_size, _ptr(q), N, R, H,
                                   _ptr(block_tables), block_tables.shape[1], _ptr(context_lens),
                                   max_context_len, _ptr(out), _ptr(err_flags), _stream(stream)),
           "kvq_index_scores")
    return out
