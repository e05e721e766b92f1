"""GB300 paged-KV decode library: Python binding of libpa.so (include/pa.h).

The binding only marshals arguments: shapes and dtypes are read from torch
tensors, pointers and the current CUDA stream are passed to the C entry
points of the same names, and a non-OK status raises ``PaError`` with the
library's detail string.  Every step of the computation runs in the CUDA
kernels of libpa.so; there is no fallback of any kind -- if the library has
not been built, every call raises.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libpa.so")

PA_F32, PA_F16, PA_BF16, PA_FP8_E4M3, PA_FP8_E5M2, PA_INT4 = 0, 1, 2, 3, 4, 5
PA_OK = 0
ERRBIT_BAD_BLOCK, ERRBIT_BAD_SLOT, ERRBIT_BAD_PAIR, ERRBIT_SEQ_TOO_LONG, ERRBIT_WAIT_TIMEOUT = 1, 2, 4, 8, 16
ERRBIT_BAD_QUERY, ERRBIT_BAD_POSITION = 32, 64

# entry points declared in include/pa.h
EXPORTED = ("pa_status_string", "pa_last_error_detail", "pa_decode_workspace_size", "pa_decode",
            "pa_decode_simt", "pa_decode_noalloc", "pa_reshape_and_cache", "pa_copy_blocks",
            "pa_copy_blocks_layers", "pa_swap_blocks", "pa_attention", "pa_attention_workspace_size",
            "pa_gather_cache", "pa_block_bytes", "pa_evict", "pa_evict_workspace_size",
            "pa_decode_weights", "pa_decode_weights_workspace_size", "pa_prefill", "pa_prefill_cached",
            "pa_prefill_workspace_size", "pa_rope_and_cache", "pa_decode_shared", "pa_decode_shared_workspace_size")
NOALLOC_SCRATCH_BYTES = 32 << 20

_DTYPE_CODE = {torch.float32: PA_F32, torch.float16: PA_F16, torch.bfloat16: PA_BF16,
               torch.uint8: PA_FP8_E4M3, torch.float8_e4m3fn: PA_FP8_E4M3, torch.float8_e5m2: PA_FP8_E5M2}
_NAME_CODE = {"f32": PA_F32, "f16": PA_F16, "bf16": PA_BF16, "fp8_e4m3": PA_FP8_E4M3, "fp8_e5m2": PA_FP8_E5M2, "int4": PA_INT4}


class PaError(RuntimeError):
    def __init__(self, status: int, detail: str):
        super().__init__(f"{status_string(status)}: {detail}")
        self.status = status


_lib = None


def build(force: bool = False) -> str:
    from . import build_lib as _b
    return _b.build(force=force)


def _configure(L):
    """Declare the C signatures of include/pa.h on a loaded library."""
    c_int, c_float, vp, sz = ctypes.c_int, ctypes.c_float, ctypes.c_void_p, ctypes.c_size_t
    L.pa_status_string.restype = ctypes.c_char_p
    L.pa_status_string.argtypes = [c_int]
    L.pa_last_error_detail.restype = ctypes.c_char_p
    L.pa_last_error_detail.argtypes = []
    L.pa_decode_workspace_size.restype = sz
    L.pa_decode_workspace_size.argtypes = [c_int, c_int, c_int, c_int, c_int]
    dec = [vp, vp, c_int, vp, vp, c_int, vp, c_int, vp, c_int, c_int, c_int, c_int, c_int, c_int,
           c_float, c_float, c_float, c_int, vp, sz, vp, vp]
    for name in ("pa_decode", "pa_decode_simt"):
        getattr(L, name).restype = c_int
        getattr(L, name).argtypes = dec
    L.pa_decode_noalloc.restype = c_int
    L.pa_decode_noalloc.argtypes = dec[:19] + [vp, vp]
    L.pa_reshape_and_cache.restype = c_int
    L.pa_reshape_and_cache.argtypes = [vp, vp, c_int, vp, vp, c_int, vp, c_int, c_int, c_int, c_int,
                                       c_int, c_float, c_float, vp, vp]
    L.pa_gather_cache.restype = c_int
    L.pa_gather_cache.argtypes = [vp, vp, c_int, vp, vp, c_int, vp, c_int, c_int, c_int, c_int, c_int, c_float,
                                  c_float, vp, vp]
    L.pa_block_bytes.restype = sz
    L.pa_block_bytes.argtypes = [c_int, c_int, c_int, c_int]
    L.pa_copy_blocks.restype = c_int
    L.pa_copy_blocks.argtypes = [vp, vp, c_int, vp, c_int, c_int, c_int, c_int, c_int, vp, vp]
    L.pa_copy_blocks_layers.restype = c_int
    L.pa_copy_blocks_layers.argtypes = [vp, vp, c_int, c_int, vp, c_int, c_int, c_int, c_int, c_int, vp, vp]
    L.pa_swap_blocks.restype = c_int
    L.pa_swap_blocks.argtypes = [vp, vp, c_int, vp, vp, c_int, c_int, vp, c_int, c_int, c_int, c_int, vp, vp]
    L.pa_attention_workspace_size.restype = sz
    L.pa_attention_workspace_size.argtypes = [c_int, c_int, c_int, c_int, c_int, c_int]
    L.pa_attention.restype = c_int
    L.pa_attention.argtypes = [vp, vp, c_int, vp, vp, c_int, vp, c_int, vp, vp, c_int, c_int, c_int, c_int, c_int,
                               c_int, c_int, c_int, c_float, c_float, c_float, c_int, vp, sz, vp, vp]
    L.pa_decode_weights_workspace_size.restype = sz
    L.pa_decode_weights_workspace_size.argtypes = [c_int, c_int, c_int, c_int]
    L.pa_decode_weights.restype = c_int
    L.pa_decode_weights.argtypes = [vp, vp, vp, c_int, vp, vp, c_int, vp, c_int, vp, vp, c_int, c_int, c_int, c_int,
                                    c_int, c_int, c_float, c_float, c_float, vp, sz, vp, vp]
    L.pa_rope_and_cache.restype = c_int
    L.pa_rope_and_cache.argtypes = [vp, vp, c_int, vp, vp, vp, vp, vp, c_int, vp, c_int, vp, vp, c_int, c_int, c_int, vp,
                                    c_int, c_int, c_int, c_int, c_int, c_int, c_float, c_float, vp, vp]
    L.pa_decode_shared_workspace_size.restype = sz
    L.pa_decode_shared_workspace_size.argtypes = [c_int] * 6
    L.pa_decode_shared.restype = c_int
    L.pa_decode_shared.argtypes = [vp, vp, c_int, vp, vp, c_int, vp, c_int, vp, vp, vp, c_int, c_int, c_int, c_int, c_int,
                                   c_int, c_int, c_float, vp, sz, vp, vp]
    L.pa_prefill_workspace_size.restype = sz
    L.pa_prefill_workspace_size.argtypes = [c_int] * 5
    L.pa_prefill.restype = c_int
    L.pa_prefill.argtypes = [vp, vp, vp, vp, c_int, vp, vp, c_int, c_int, c_int, c_int, c_int, c_int, c_float, vp, sz, vp,
                             vp]
    L.pa_prefill_cached.restype = c_int
    L.pa_prefill_cached.argtypes = [vp, vp, c_int, vp, vp, c_int, vp, c_int, vp, vp, c_int, c_int, c_int, c_int, c_int,
                                    c_int, c_int, c_float, vp, sz, vp, vp]
    L.pa_evict_workspace_size.restype = sz
    L.pa_evict_workspace_size.argtypes = [c_int, c_int, c_int, c_int]
    L.pa_evict.restype = c_int
    L.pa_evict.argtypes = [vp, vp, c_int, vp, vp, c_int, vp, vp, c_int, vp, vp, c_int, c_int, c_int, c_int, c_int,
                           c_int, c_int, c_int, vp, sz, vp, vp]
    return L


def lib():
    """The loaded libpa.so (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libpa.so is not built ({LIB_PATH}); run paged_kv_cache_69_gb300.build()")
        _lib = _configure(ctypes.CDLL(LIB_PATH))
    return _lib


def status_string(status: int) -> str:
    try:
        return lib().pa_status_string(int(status)).decode()
    except Exception:  # pragma: no cover
        return f"status {status}"


def _check(status: int):
    if status != PA_OK:
        raise PaError(status, lib().pa_last_error_detail().decode())


# (plain numbers: every argument of a pointer's type takes them; a c_void_p around each
# costs a call with 12 pointers 1.3-2.2 us)
def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _code(t: torch.Tensor, override=None) -> int:
    if override is not None:
        return _NAME_CODE[override] if isinstance(override, str) else int(override)
    if t.dtype not in _DTYPE_CODE:
        raise ValueError(f"libpa has no element type for {t.dtype}")
    return _DTYPE_CODE[t.dtype]


def _is_int4(kv_dtype) -> bool:
    return kv_dtype == "int4" or (isinstance(kv_dtype, int) and kv_dtype == PA_INT4)


# The current stream's handle without a Stream object around it (3 us less per
# call on a Grace host); None where torch has no such function.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream) -> int:
    if stream is None:
        if _raw_stream is not None:
            return _raw_stream(torch.cuda.current_device())
        stream = torch.cuda.current_stream()
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _scratch(nbytes: int, device, stream) -> torch.Tensor:
    """The workspace of one call, from the memory of the stream that the call
    runs on: torch hands it out again only to work behind the call's kernels."""
    if nbytes == 0:
        raise PaError(1, "invalid workspace bounds")
    if stream is None:
        return torch.empty(nbytes, dtype=torch.uint8, device=device)
    if not hasattr(stream, "cuda_stream"):
        stream = torch.cuda.ExternalStream(int(stream)) if int(stream) else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        return torch.empty(nbytes, dtype=torch.uint8, device=device)


def _nbytes(t: Optional[torch.Tensor]) -> int:
    return 0 if t is None else t.numel() * t.element_size()


def _dev(*ts):
    device = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError("libpa works on CUDA tensors only")
        if not t.is_contiguous():
            raise ValueError("libpa expects contiguous tensors")
        if device is None:
            device = torch.cuda.current_device()     # kernels launch there
        if t.get_device() != device:
            raise ValueError("libpa works on tensors of the current device")


def _pools(k: torch.Tensor, v: torch.Tensor, kv_dtype=None):
    """K and V pools of one shape and element type; returns (NB, bs, Hkv, D).
    A 4-bit pool is uint8 with head_dim / 2 + 4 bytes per row."""
    if k.dim() != 4 or tuple(v.shape) != tuple(k.shape) or v.dtype != k.dtype:
        raise ValueError("k_cache and v_cache must be [num_blocks, block_size, num_kv_heads, head_dim] "
                         "of one shape and dtype")
    if _is_int4(kv_dtype):
        if k.dtype != torch.uint8 or k.shape[3] <= 4:
            raise ValueError("4-bit pools must be uint8 [num_blocks, block_size, num_kv_heads, head_dim / 2 + 4]")
        return tuple(k.shape[:3]) + (2 * (k.shape[3] - 4),)
    return tuple(k.shape)


def _tables(block_tables: torch.Tensor, seq_lens: torch.Tensor, B: int):
    """int32 block tables with a row per sequence and int32 seq_lens [B]."""
    if block_tables.dtype != torch.int32 or seq_lens.dtype != torch.int32:
        raise ValueError("block_tables and seq_lens must be int32")
    if block_tables.dim() != 2 or block_tables.shape[0] < B or seq_lens.numel() != B:
        raise ValueError("block_tables must be [>= num_seqs, max_blocks] and seq_lens [num_seqs]")


def _flag(err_flag: Optional[torch.Tensor]):
    if err_flag is not None and (err_flag.dtype != torch.int32 or err_flag.numel() < 1):
        raise ValueError("err_flag must be an int32 tensor of at least one element")


# ---------------------------------------------------------------------------
def pa_decode_workspace_size(num_seqs: int, num_q_heads: int, max_seq_len: int, head_dim: int,
                             partition_tokens: int = 0) -> int:
    return int(lib().pa_decode_workspace_size(num_seqs, num_q_heads, max_seq_len, head_dim, partition_tokens))


def alloc_workspace(num_seqs: int, num_q_heads: int, max_seq_len: int, head_dim: int,
                    partition_tokens: int = 0, device=None) -> torch.Tensor:
    n = pa_decode_workspace_size(num_seqs, num_q_heads, max_seq_len, head_dim, partition_tokens)
    if n == 0:
        raise PaError(1, "invalid workspace bounds")
    return torch.empty(n, dtype=torch.uint8, device=device or "cuda")   # torch allocations are 256-B aligned


def alloc_int4_cache(num_blocks: int, block_size: int, num_kv_heads: int, head_dim: int, device=None) -> torch.Tensor:
    """A zeroed 4-bit K (or V) pool, uint8 [num_blocks, block_size,
    num_kv_heads, head_dim / 2 + 4]; kv_dtype="int4" in the calls.  Inside a
    block the codes of all rows come first, then their (step, low) pairs."""
    if head_dim not in (64, 128) or block_size % 8 or min(num_blocks, block_size, num_kv_heads) <= 0:
        raise ValueError("a 4-bit pool needs head_dim 64 or 128 and a block_size of a multiple of 8")
    return torch.zeros(num_blocks, block_size, num_kv_heads, head_dim // 2 + 4, dtype=torch.uint8,
                       device=device or "cuda")


def pa_decode(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
              block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float, kv_dtype=None, *,
              k_scale: float = 1.0, v_scale: float = 1.0, partition_tokens: int = 0,
              workspace: Optional[torch.Tensor] = None, err_flag: Optional[torch.Tensor] = None,
              stream=None, simt: bool = False) -> torch.Tensor:
    """out[i, h] = softmax(scale * q[i, h] K_i^T) V_i over the paged pool.
    q/out [B, Hq, D]; k_cache/v_cache [NB, bs, Hkv, D]; block_tables int32
    [B, MB]; seq_lens int32 [B].  ``kv_dtype`` defaults to the cache tensor's
    dtype (uint8 storage means fp8-e4m3; "int4" names a 4-bit pool)."""
    _dev(out, q, k_cache, v_cache, block_tables, seq_lens, workspace, err_flag)
    B, Hq, D = q.shape
    NB, bs, Hkv, D2 = _pools(k_cache, v_cache, kv_dtype)
    if D2 != D or tuple(out.shape) != (B, Hq, D) or out.dtype != q.dtype:
        raise ValueError("q and out must be [num_seqs, num_q_heads, head_dim] of one dtype, head_dim "
                         "that of the pools")
    _tables(block_tables, seq_lens, B)
    _flag(err_flag)
    MB = block_tables.shape[1]
    if workspace is None:
        workspace = _scratch(pa_decode_workspace_size(B, Hq, MB * bs, D, partition_tokens), q.device, stream)
    fn = lib().pa_decode_simt if simt else lib().pa_decode
    _check(fn(_ptr(out), _ptr(q), _code(q), _ptr(k_cache), _ptr(v_cache), _code(k_cache, kv_dtype),
              _ptr(block_tables), MB, _ptr(seq_lens), B, Hq, Hkv, D, bs, NB, float(scale),
              float(k_scale), float(v_scale), int(partition_tokens), _ptr(workspace),
              workspace.numel() * workspace.element_size(), _ptr(err_flag), _stream(stream)))
    return out


def pa_decode_noalloc(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float, kv_dtype=None, *,
                      k_scale: float = 1.0, v_scale: float = 1.0, partition_tokens: int = 0,
                      err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pa_decode without a workspace argument, for callers that cannot
    allocate one: the partials go to the library's built-in device scratch
    (NOALLOC_SCRATCH_BYTES per GPU, shared by all calls on that GPU)."""
    _dev(out, q, k_cache, v_cache, block_tables, seq_lens, err_flag)
    B, Hq, D = q.shape
    NB, bs, Hkv, D2 = _pools(k_cache, v_cache, kv_dtype)
    if D2 != D or tuple(out.shape) != (B, Hq, D) or out.dtype != q.dtype:
        raise ValueError("q and out must be [num_seqs, num_q_heads, head_dim] of one dtype, head_dim "
                         "that of the pools")
    _tables(block_tables, seq_lens, B)
    _flag(err_flag)
    _check(lib().pa_decode_noalloc(_ptr(out), _ptr(q), _code(q), _ptr(k_cache), _ptr(v_cache),
                                   _code(k_cache, kv_dtype), _ptr(block_tables), block_tables.shape[1],
                                   _ptr(seq_lens), B, Hq, Hkv, D, bs, NB, float(scale), float(k_scale),
                                   float(v_scale), int(partition_tokens), _ptr(err_flag), _stream(stream)))
    return out


def pa_decode_shared_workspace_size(num_seqs: int, num_groups: int, num_q_heads: int, num_kv_heads: int,
                                    max_seq_len: int, head_dim: int) -> int:
    return int(lib().pa_decode_shared_workspace_size(num_seqs, num_groups, num_q_heads, num_kv_heads, max_seq_len, head_dim))


def pa_decode_shared(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                     block_tables: torch.Tensor, seq_lens: torch.Tensor, group_start: torch.Tensor,
                     prefix_lens: torch.Tensor, scale: float, kv_dtype=None, *, workspace: Optional[torch.Tensor] = None,
                     err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pa_decode whose sequences group_start[j] .. group_start[j+1]-1 (int32
    [groups + 1]) share the blocks of their first prefix_lens[j] tokens (int32
    [groups]): a prefix's keys are read once for its group."""
    _dev(out, q, k_cache, v_cache, block_tables, seq_lens, group_start, prefix_lens, workspace, err_flag)
    B, Hq, D = q.shape
    NB, bs, Hkv, D2 = _pools(k_cache, v_cache, kv_dtype)
    if D2 != D or tuple(out.shape) != (B, Hq, D) or out.dtype != q.dtype:
        raise ValueError("q and out must be [num_seqs, num_q_heads, head_dim] of one dtype, head_dim "
                         "that of the pools")
    _tables(block_tables, seq_lens, B)
    NG = prefix_lens.numel()
    if prefix_lens.dtype != torch.int32 or group_start.dtype != torch.int32 or group_start.numel() != NG + 1:
        raise ValueError("group_start must be int32 [num_groups + 1] and prefix_lens int32 [num_groups]")
    _flag(err_flag)
    MB = block_tables.shape[1]
    if workspace is None and B > 0:
        workspace = _scratch(pa_decode_shared_workspace_size(B, NG, Hq, Hkv, MB * bs, D), q.device, stream)
    _check(lib().pa_decode_shared(_ptr(out), _ptr(q), _code(q), _ptr(k_cache), _ptr(v_cache), _code(k_cache, kv_dtype),
                                  _ptr(block_tables), MB, _ptr(seq_lens), _ptr(group_start), _ptr(prefix_lens), B, NG, Hq,
                                  Hkv, D, bs, NB, float(scale), _ptr(workspace), _nbytes(workspace), _ptr(err_flag),
                                  _stream(stream)))
    return out


def pa_reshape_and_cache(k_cache: torch.Tensor, v_cache: torch.Tensor, key: torch.Tensor,
                         value: torch.Tensor, slot_mapping: torch.Tensor, kv_dtype=None, *,
                         k_scale: float = 1.0, v_scale: float = 1.0,
                         err_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """Write key/value [T, Hkv, D] into pool slots slot_mapping (int64 [T])."""
    _dev(k_cache, v_cache, key, value, slot_mapping, err_flag)
    NB, bs, Hkv, D = _pools(k_cache, v_cache, kv_dtype)
    T = key.shape[0]
    if tuple(key.shape) != (T, Hkv, D) or tuple(value.shape) != (T, Hkv, D) or value.dtype != key.dtype:
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_dim] of one dtype")
    _flag(err_flag)
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != T:
        raise ValueError("slot_mapping must be int64 [num_tokens]")
    _check(lib().pa_reshape_and_cache(_ptr(k_cache), _ptr(v_cache), _code(k_cache, kv_dtype), _ptr(key),
                                      _ptr(value), _code(key), _ptr(slot_mapping), T, Hkv, D, bs, NB,
                                      float(k_scale), float(v_scale), _ptr(err_flag), _stream(stream)))


def rope_table(num_positions: int, rot_dim: int, base: float = 10000.0, device=None) -> torch.Tensor:
    """cos_sin of pa_rope_and_cache, float32 [num_positions, rot_dim]: cosines,
    then sines, of position * base^(-2i / rot_dim), the angles in 64 bits."""
    pair = torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device or "cuda")
    angle = torch.arange(num_positions, dtype=torch.float64, device=pair.device)[:, None] * base ** (-pair / rot_dim)
    return torch.cat([angle.cos(), angle.sin()], 1).float()


def pa_rope_and_cache(k_cache: torch.Tensor, v_cache: torch.Tensor, q_out: Optional[torch.Tensor],
                      q: Optional[torch.Tensor], key: torch.Tensor, value: torch.Tensor, positions: torch.Tensor,
                      cos_sin: torch.Tensor, slot_mapping: torch.Tensor, kv_dtype=None, *,
                      key_out: Optional[torch.Tensor] = None, sections=None, interleaved: bool = False,
                      k_scale: float = 1.0, v_scale: float = 1.0, err_flag: Optional[torch.Tensor] = None,
                      stream=None) -> None:
    """Rotate q [T, Hq, D] into q_out (it may be q) and key [T, Hkv, D] by
    positions (int64 [T], or [axes, T] with ``sections``, the rotated pairs of each
    axis), and write K/V into pool slots slot_mapping (int64 [T]).  cos_sin is
    float32 [positions, rot_dim] (rope_table); key_out receives the rotated keys.
    q and q_out may be None: keys and values alone."""
    _dev(k_cache, v_cache, q_out, q, key, value, positions, cos_sin, slot_mapping, key_out, err_flag)
    NB, bs, Hkv, D = _pools(k_cache, v_cache, kv_dtype)
    T = key.shape[0]
    if tuple(key.shape) != (T, Hkv, D) or tuple(value.shape) != (T, Hkv, D) or value.dtype != key.dtype:
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_dim] of one dtype")
    if key_out is not None and (tuple(key_out.shape) != (T, Hkv, D) or key_out.dtype != key.dtype):
        raise ValueError("key_out must have the shape and dtype of key")
    if (q is None) != (q_out is None):
        raise ValueError("q and q_out go together")
    Hq = 0
    if q is not None:
        Hq = q.shape[1] if q.dim() == 3 else 0
        for t in (q, q_out):
            if tuple(t.shape) != (T, Hq, D) or Hq == 0 or t.dtype != key.dtype:
                raise ValueError("q and q_out must be [num_tokens, num_q_heads, head_dim] of key's dtype")
    axes = 1 if sections is None else len(sections)
    if positions.dtype != torch.int64 or positions.numel() != axes * T or (axes > 1 and tuple(positions.shape) != (axes, T)):
        raise ValueError("positions must be int64 [num_tokens], or [len(sections), num_tokens]")
    if cos_sin.dtype != torch.float32 or cos_sin.dim() != 2:
        raise ValueError("cos_sin must be float32 [positions, rot_dim]")
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != T:
        raise ValueError("slot_mapping must be int64 [num_tokens]")
    _flag(err_flag)
    sec = None if sections is None else (ctypes.c_int * max(1, axes))(*[int(x) for x in sections])
    _check(lib().pa_rope_and_cache(_ptr(k_cache), _ptr(v_cache), _code(k_cache, kv_dtype), _ptr(q_out), _ptr(key_out),
                                   _ptr(q), _ptr(key), _ptr(value), _code(key), _ptr(positions), axes, sec, _ptr(cos_sin),
                                   cos_sin.shape[0], cos_sin.shape[1], int(bool(interleaved)), _ptr(slot_mapping), T, Hq,
                                   Hkv, D, bs, NB, float(k_scale), float(v_scale), _ptr(err_flag), _stream(stream)))


def pa_gather_cache(key: torch.Tensor, value: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    slot_mapping: torch.Tensor, kv_dtype=None, *, k_scale: float = 1.0, v_scale: float = 1.0,
                    err_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """Read pool slots slot_mapping (int64 [T]) back into key/value
    [T, Hkv, D]: bits of f32/f16/bf16 pools, values of fp8 and 4-bit pools."""
    _dev(key, value, k_cache, v_cache, slot_mapping, err_flag)
    NB, bs, Hkv, D = _pools(k_cache, v_cache, kv_dtype)
    T = key.shape[0]
    if tuple(key.shape) != (T, Hkv, D) or tuple(value.shape) != (T, Hkv, D) or value.dtype != key.dtype:
        raise ValueError("key/value must be [num_tokens, num_kv_heads, head_dim] of one dtype")
    _flag(err_flag)
    if slot_mapping.dtype != torch.int64 or slot_mapping.numel() != T:
        raise ValueError("slot_mapping must be int64 [num_tokens]")
    _check(lib().pa_gather_cache(_ptr(key), _ptr(value), _code(key), _ptr(k_cache), _ptr(v_cache),
                                 _code(k_cache, kv_dtype), _ptr(slot_mapping), T, Hkv, D, bs, NB, float(k_scale),
                                 float(v_scale), _ptr(err_flag), _stream(stream)))


def pa_copy_blocks(k_cache: torch.Tensor, v_cache: torch.Tensor, block_mapping: torch.Tensor,
                   kv_dtype=None, *, err_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """Copy whole blocks src -> dst for each row (src, dst) of block_mapping (int64 [P, 2])."""
    _dev(k_cache, v_cache, block_mapping, err_flag)
    NB, bs, Hkv, D = _pools(k_cache, v_cache, kv_dtype)
    _flag(err_flag)
    if block_mapping.dtype != torch.int64 or (block_mapping.numel() and block_mapping.shape[-1] != 2):
        raise ValueError("block_mapping must be int64 [num_pairs, 2]")
    P = block_mapping.numel() // 2
    _check(lib().pa_copy_blocks(_ptr(k_cache), _ptr(v_cache), _code(k_cache, kv_dtype), _ptr(block_mapping),
                                P, Hkv, D, bs, NB, _ptr(err_flag), _stream(stream)))


def pa_copy_blocks_layers(k_caches, v_caches, block_mapping: torch.Tensor, kv_dtype=None, *,
                          err_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """pa_copy_blocks over lists of per-layer pools of one shape."""
    if len(k_caches) != len(v_caches) or not k_caches:
        raise ValueError("k_caches and v_caches must be equal-length non-empty lists")
    _dev(*k_caches, *v_caches, block_mapping, err_flag)
    NB, bs, Hkv, D = _pools(k_caches[0], v_caches[0], kv_dtype)
    _flag(err_flag)
    for t in list(k_caches) + list(v_caches):
        if t.shape != k_caches[0].shape or t.dtype != k_caches[0].dtype:
            raise ValueError("all pools must have one shape and dtype")
    if block_mapping.dtype != torch.int64 or (block_mapping.numel() and block_mapping.shape[-1] != 2):
        raise ValueError("block_mapping must be int64 [num_pairs, 2]")
    L = len(k_caches)
    kp = (ctypes.c_void_p * L)(*[t.data_ptr() for t in k_caches])
    vp_ = (ctypes.c_void_p * L)(*[t.data_ptr() for t in v_caches])
    _check(lib().pa_copy_blocks_layers(kp, vp_, L, _code(k_caches[0], kv_dtype), _ptr(block_mapping),
                                       block_mapping.numel() // 2, Hkv, D, bs, NB, _ptr(err_flag),
                                       _stream(stream)))


def pa_swap_blocks(dst_k: torch.Tensor, dst_v: torch.Tensor, src_k: torch.Tensor, src_v: torch.Tensor,
                   block_mapping: torch.Tensor, kv_dtype=None, *, err_flag: Optional[torch.Tensor] = None,
                   stream=None) -> None:
    """Copy blocks src -> dst between two pools; either may be pinned host
    memory (torch pin_memory()), block_mapping must be on the device."""
    for t in (dst_k, dst_v, src_k, src_v):
        if not t.is_contiguous():
            raise ValueError("pools must be contiguous")
        if not (t.is_cuda or t.is_pinned()):
            raise ValueError("pools must be device memory or pinned host memory")
    _dev(block_mapping, err_flag)
    _flag(err_flag)
    NBd, bs, Hkv, D = _pools(dst_k, dst_v, kv_dtype)
    NBs = _pools(src_k, src_v, kv_dtype)[0]
    if src_k.shape[1:] != dst_k.shape[1:] or src_k.dtype != dst_k.dtype:
        raise ValueError("pools must share the block shape and dtype")
    if block_mapping.dtype != torch.int64 or (block_mapping.numel() and block_mapping.shape[-1] != 2):
        raise ValueError("block_mapping must be int64 [num_pairs, 2]")
    _check(lib().pa_swap_blocks(_ptr(dst_k), _ptr(dst_v), NBd, _ptr(src_k), _ptr(src_v), NBs,
                                _code(dst_k, kv_dtype), _ptr(block_mapping), block_mapping.numel() // 2,
                                Hkv, D, bs, _ptr(err_flag), _stream(stream)))


def pa_attention_workspace_size(num_seqs: int, max_q_len: int, num_q_heads: int, max_seq_len: int,
                                head_dim: int, partition_tokens: int = 0) -> int:
    return int(lib().pa_attention_workspace_size(num_seqs, max_q_len, num_q_heads, max_seq_len, head_dim,
                                                 partition_tokens))


def pa_attention(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                 block_tables: torch.Tensor, seq_lens: torch.Tensor, q_start: torch.Tensor, scale: float,
                 max_q_len: int, kv_dtype=None, *, k_scale: float = 1.0, v_scale: float = 1.0,
                 partition_tokens: int = 0, workspace: Optional[torch.Tensor] = None,
                 err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention of several query tokens per sequence over the paged
    pool.  q/out [T, Hq, D]; sequence i's query rows are q_start[i] ..
    q_start[i+1]-1 (int32 [B+1] on the device), the last tokens of its
    seq_lens[i]; max_q_len bounds every sequence's query count."""
    _dev(out, q, k_cache, v_cache, block_tables, seq_lens, q_start, workspace, err_flag)
    T, Hq, D = q.shape
    NB, bs, Hkv, D2 = _pools(k_cache, v_cache, kv_dtype)
    B = seq_lens.numel()
    if D2 != D or tuple(out.shape) != (T, Hq, D) or out.dtype != q.dtype:
        raise ValueError("q and out must be [total_q, num_q_heads, head_dim] of one dtype, head_dim "
                         "that of the pools")
    _tables(block_tables, seq_lens, B)
    _flag(err_flag)
    if q_start.dtype != torch.int32 or q_start.numel() != B + 1:
        raise ValueError("q_start must be int32 with num_seqs + 1 entries")
    MB = block_tables.shape[1]
    if workspace is None:
        n = pa_attention_workspace_size(B, max_q_len, Hq, MB * bs, D, partition_tokens)
        workspace = _scratch(n, q.device, stream)
    _check(lib().pa_attention(_ptr(out), _ptr(q), _code(q), _ptr(k_cache), _ptr(v_cache), _code(k_cache, kv_dtype),
                              _ptr(block_tables), MB, _ptr(seq_lens), _ptr(q_start), B, T, int(max_q_len), Hq, Hkv,
                              D, bs, NB, float(scale), float(k_scale), float(v_scale), int(partition_tokens),
                              _ptr(workspace), workspace.numel() * workspace.element_size(), _ptr(err_flag),
                              _stream(stream)))
    return out


def _starts(t: torch.Tensor, B: int, name: str):
    if t.dtype != torch.int32 or t.numel() != B + 1:
        raise ValueError(f"{name} must be int32 with num_seqs + 1 entries")


def pa_prefill_workspace_size(num_seqs: int, total_q: int, num_q_heads: int, num_kv_heads: int, head_dim: int) -> int:
    return int(lib().pa_prefill_workspace_size(num_seqs, total_q, num_q_heads, num_kv_heads, head_dim))


def pa_prefill(out: torch.Tensor, q: torch.Tensor, key: torch.Tensor, value: torch.Tensor, q_start: torch.Tensor,
               scale: float, *, k_start: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
               err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """Causal attention of whole prompts, packed.  q/out [T, Hq, D]; key/value
    [Tk, Hkv, D]; sequence i has query rows q_start[i] .. q_start[i+1]-1 and key
    rows k_start[i] .. k_start[i+1]-1 (int32 [B+1]; None: q_start), its query
    tokens being the last of its tokens."""
    _dev(out, q, key, value, q_start, k_start, workspace, err_flag)
    if q.dim() != 3 or key.dim() != 3 or tuple(out.shape) != tuple(q.shape) or out.dtype != q.dtype:
        raise ValueError("q and out must be [total_q, num_q_heads, head_dim] of one dtype")
    T, Hq, D = q.shape
    Tk, Hkv, D2 = key.shape
    if D2 != D or tuple(value.shape) != tuple(key.shape) or key.dtype != q.dtype or value.dtype != q.dtype:
        raise ValueError("key and value must be [total_k, num_kv_heads, head_dim], head_dim and dtype those of q")
    B = q_start.numel() - 1
    _starts(q_start, B, "q_start")
    if k_start is not None:
        _starts(k_start, B, "k_start")
    _flag(err_flag)
    if workspace is None and B > 0 and T > 0:
        workspace = _scratch(pa_prefill_workspace_size(B, T, Hq, Hkv, D), q.device, stream)
    _check(lib().pa_prefill(_ptr(out), _ptr(q), _ptr(key), _ptr(value), _code(q), _ptr(q_start), _ptr(k_start), B, T, Tk,
                            Hq, Hkv, D, float(scale), _ptr(workspace), _nbytes(workspace), _ptr(err_flag),
                            _stream(stream)))
    return out


def pa_prefill_cached(out: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                      block_tables: torch.Tensor, seq_lens: torch.Tensor, q_start: torch.Tensor, scale: float,
                      kv_dtype=None, *, workspace: Optional[torch.Tensor] = None,
                      err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pa_prefill over the paged pool: sequence i's query rows q_start[i] ..
    q_start[i+1]-1 (int32 [B+1]) are the last tokens of its seq_lens[i], all of
    them in the pool already; any number of query tokens."""
    _dev(out, q, k_cache, v_cache, block_tables, seq_lens, q_start, workspace, err_flag)
    if q.dim() != 3:
        raise ValueError("q and out must be [total_q, num_q_heads, head_dim]")
    T, Hq, D = q.shape
    NB, bs, Hkv, D2 = _pools(k_cache, v_cache, kv_dtype)
    B = seq_lens.numel()
    if D2 != D or tuple(out.shape) != (T, Hq, D) or out.dtype != q.dtype:
        raise ValueError("q and out must be [total_q, num_q_heads, head_dim] of one dtype, head_dim "
                         "that of the pools")
    _tables(block_tables, seq_lens, B)
    _starts(q_start, B, "q_start")
    _flag(err_flag)
    if workspace is None and B > 0 and T > 0:
        workspace = _scratch(pa_prefill_workspace_size(B, T, Hq, Hkv, D), q.device, stream)
    _check(lib().pa_prefill_cached(_ptr(out), _ptr(q), _code(q), _ptr(k_cache), _ptr(v_cache), _code(k_cache, kv_dtype),
                                   _ptr(block_tables), block_tables.shape[1], _ptr(seq_lens), _ptr(q_start), B, T, Hq,
                                   Hkv, D, bs, NB, float(scale), _ptr(workspace), _nbytes(workspace), _ptr(err_flag),
                                   _stream(stream)))
    return out


def _weights(weights: torch.Tensor, NB: int, Hkv: int, bs: int):
    if weights.dtype != torch.float32 or tuple(weights.shape) != (NB, Hkv, bs):
        raise ValueError("weights must be float32 [num_blocks, num_kv_heads, block_size]")


def pa_decode_weights_workspace_size(num_seqs: int, num_q_heads: int, max_seq_len: int, head_dim: int) -> int:
    return int(lib().pa_decode_weights_workspace_size(num_seqs, num_q_heads, max_seq_len, head_dim))


def pa_decode_weights(out: torch.Tensor, weights: torch.Tensor, q: torch.Tensor, k_cache: torch.Tensor,
                      v_cache: torch.Tensor, block_tables: torch.Tensor, seq_lens: torch.Tensor, scale: float,
                      kv_dtype=None, *, fresh: Optional[torch.Tensor] = None, k_scale: float = 1.0,
                      v_scale: float = 1.0, workspace: Optional[torch.Tensor] = None,
                      err_flag: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """pa_decode that also adds every key's softmax weight, summed over the
    heads of its group, to ``weights`` (float32 [NB, Hkv, bs]).  The entries of
    a sequence's last ``fresh`` tokens (int32 [B]; None: 1) start from 0."""
    _dev(out, weights, q, k_cache, v_cache, block_tables, seq_lens, fresh, workspace, err_flag)
    B, Hq, D = q.shape
    NB, bs, Hkv, D2 = _pools(k_cache, v_cache, kv_dtype)
    if D2 != D or tuple(out.shape) != (B, Hq, D) or out.dtype != q.dtype:
        raise ValueError("q and out must be [num_seqs, num_q_heads, head_dim] of one dtype, head_dim "
                         "that of the pools")
    _tables(block_tables, seq_lens, B)
    _weights(weights, NB, Hkv, bs)
    _flag(err_flag)
    if fresh is not None and (fresh.dtype != torch.int32 or fresh.numel() != B):
        raise ValueError("fresh must be int32 [num_seqs]")
    MB = block_tables.shape[1]
    if workspace is None:
        workspace = _scratch(pa_decode_weights_workspace_size(B, Hq, MB * bs, D), q.device, stream)
    _check(lib().pa_decode_weights(_ptr(out), _ptr(weights), _ptr(q), _code(q), _ptr(k_cache), _ptr(v_cache),
                                   _code(k_cache, kv_dtype), _ptr(block_tables), MB, _ptr(seq_lens), _ptr(fresh), B, Hq,
                                   Hkv, D, bs, NB, float(scale), float(k_scale), float(v_scale), _ptr(workspace),
                                   workspace.numel() * workspace.element_size(), _ptr(err_flag), _stream(stream)))
    return out


def pa_evict_workspace_size(num_seqs: int, num_kv_heads: int, max_seq_len: int, budget: int) -> int:
    return int(lib().pa_evict_workspace_size(num_seqs, num_kv_heads, max_seq_len, budget))


def pa_evict(k_cache: torch.Tensor, v_cache: torch.Tensor, weights: torch.Tensor, block_tables: torch.Tensor,
             seq_lens: torch.Tensor, new_seq_lens: torch.Tensor, budget: int, kv_dtype=None, *, num_sink: int = 0,
             num_recent: int = 0, new_block_tables: Optional[torch.Tensor] = None,
             kept: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
             err_flag: Optional[torch.Tensor] = None, stream=None) -> None:
    """Bring every sequence down to ``budget`` tokens per KV head: the first
    ``num_sink``, the last ``num_recent`` and the most heavily weighted between
    them.  weights float32 [NB, Hkv, bs] moves with the rows; new_seq_lens
    int32 [B] receives the lengths (it may be seq_lens); kept int32
    [B, Hkv, budget] the former positions.  In place, or into the blocks of
    ``new_block_tables`` (int32 [B, MB'], another tensor than block_tables)."""
    _dev(k_cache, v_cache, weights, block_tables, seq_lens, new_seq_lens, new_block_tables, kept, workspace, err_flag)
    NB, bs, Hkv, D = _pools(k_cache, v_cache, kv_dtype)
    B = seq_lens.numel()
    _tables(block_tables, seq_lens, B)
    _weights(weights, NB, Hkv, bs)
    _flag(err_flag)
    if new_seq_lens.dtype != torch.int32 or new_seq_lens.numel() != B:
        raise ValueError("new_seq_lens must be int32 [num_seqs]")
    if kept is not None and (kept.dtype != torch.int32 or tuple(kept.shape) != (B, Hkv, budget)):
        raise ValueError("kept must be int32 [num_seqs, num_kv_heads, budget]")
    if new_block_tables is not None and new_block_tables.data_ptr() == block_tables.data_ptr():
        new_block_tables = None
    if new_block_tables is not None:
        _tables(new_block_tables, seq_lens, B)
    MB = block_tables.shape[1]
    if workspace is None:
        workspace = _scratch(pa_evict_workspace_size(B, Hkv, MB * bs, int(budget)), k_cache.device, stream)
    _check(lib().pa_evict(_ptr(k_cache), _ptr(v_cache), _code(k_cache, kv_dtype), _ptr(weights), _ptr(block_tables), MB,
                          _ptr(seq_lens), _ptr(new_block_tables),
                          0 if new_block_tables is None else new_block_tables.shape[1], _ptr(new_seq_lens), _ptr(kept),
                          B, Hkv, D, bs, NB, int(budget), int(num_sink), int(num_recent), _ptr(workspace),
                          workspace.numel() * workspace.element_size(), _ptr(err_flag), _stream(stream)))
