"""libmimoattn: MiMo-V2.6-Flash hybrid attention forward on B200 (sm_100a).

Thin ctypes binding over the C ABI in include/mimoattn.h.  It marshals torch
tensors (device memory and streams only) into the argument structs; every step
of the attention runs in the library's CUDA kernels.  There is no fallback: if
the shared library is missing the import of `lib()` raises.
"""
from __future__ import annotations

import ctypes as C
import math
import os

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "lib", "libmimoattn.so")

MIMO_OK = 0
MIMO_ERR_INVALID_ARG = 1
MIMO_ERR_UNSUPPORTED = 2
MIMO_ERR_WORKSPACE = 3
MIMO_ERR_CUDA = 4
MIMO_ERR_TIMEOUT = 5
MIMO_STATUS_TIMEOUT = 1
MIMO_STATUS_BAD_INDEX = 2
MIMO_STATUS_RANGE = 4
MIMO_STATUS_BAD_SCALE = 8
MIMO_CACHE_NONE = 0
MIMO_CACHE_PAGED = 1
MIMO_CACHE_RING = 2
MIMO_DTYPE_BF16 = 0
MIMO_DTYPE_FP8_E4M3 = 1
MIMO_DTYPE_INT4 = 2
MIMO_INT4_K_SLOT_BYTES = 108
MIMO_INT4_V_SLOT_BYTES = 72
MIMO_SELECT_MAX_SLOTS = 393216
MIMO_RING_SLOTS_DEFAULT = 128
MIMO_RING_SLOTS_MAX = 512
MIMO_MAX_DRAFTS = 8

NUM_Q_HEADS = 64
HEAD_DIM_QK = 192
HEAD_DIM_V = 128
ROPE_DIM = 64
SOFTMAX_SCALE = 1.0 / math.sqrt(192.0)
V_SCALE = 0.707

EXPORTS = ("mimo_attn_prefill", "mimo_attn_prefill_workspace_size", "mimo_attn_prefill_stall_test", "mimo_attn_decode",
           "mimo_attn_decode_workspace_size", "mimo_attn_verify_workspace_size",
           "mimo_attn_decode_int4_workspace_size", "mimo_attn_decode_noalloc",
           "mimo_kv_append", "mimo_attn_weights", "mimo_kv_select", "mimo_kv_gather", "mimo_last_error",
           "mimo_status_poll", "mimo_version", "mimo_window_from_left_right")
DECODE_NOALLOC_MAX_BYTES = 16 << 20

_P = C.c_void_p
_PI = C.POINTER(C.c_int32)


class MimoLayer(C.Structure):
    _fields_ = [("num_q_heads", C.c_int), ("num_kv_heads", C.c_int), ("head_dim_qk", C.c_int),
                ("head_dim_v", C.c_int), ("rope_dim", C.c_int), ("rope_base", C.c_double),
                ("softmax_scale", C.c_float), ("v_scale", C.c_float), ("window", C.c_int), ("sink", _P)]


class MimoPrefillArgs(C.Structure):
    _fields_ = [("layer", MimoLayer), ("num_seqs", C.c_int), ("total_q", C.c_int), ("total_k", C.c_int),
                ("q", _P), ("k", _P), ("v", _P), ("cu_seqlens_q", _P), ("cu_seqlens_k", _P), ("cache_lens", _P),
                ("cache_kind", C.c_int), ("k_cache", _P), ("v_cache", _P), ("block_table", _P),
                ("max_pages", C.c_int), ("num_pages", C.c_int), ("out", _P), ("lse", _P), ("workspace", _P),
                ("workspace_bytes", C.c_size_t), ("ev_kernel_begin", _P), ("ev_kernel_end", _P),
                ("ring_slots", C.c_int)]


class MimoDecodeArgs(C.Structure):
    _fields_ = [("layer", MimoLayer), ("batch", C.c_int), ("max_seq_len", C.c_int), ("q", _P),
                ("seq_lens", _P), ("cache_kind", C.c_int), ("k_cache", _P), ("v_cache", _P),
                ("block_table", _P), ("max_pages", C.c_int), ("num_pages", C.c_int), ("out", _P), ("lse", _P),
                ("workspace", _P), ("workspace_bytes", C.c_size_t), ("ev_kernel_begin", _P),
                ("ev_kernel_end", _P), ("cache_dtype", C.c_int), ("k_dequant", _P), ("v_dequant", _P),
                ("ring_slots", C.c_int), ("q_len", C.c_int), ("positions", _P)]


class MimoAppendArgs(C.Structure):
    _fields_ = [("num_tokens", C.c_int), ("num_kv_heads", C.c_int), ("head_dim_qk", C.c_int),
                ("head_dim_v", C.c_int), ("rope_dim", C.c_int), ("rope_base", C.c_double), ("k_new", _P),
                ("v_new", _P), ("pos", _P), ("seq_idx", _P), ("cache_kind", C.c_int), ("k_cache", _P),
                ("v_cache", _P), ("num_seqs", C.c_int), ("block_table", _P), ("max_pages", C.c_int),
                ("num_pages", C.c_int), ("cache_dtype", C.c_int), ("k_dequant", _P), ("v_dequant", _P),
                ("ring_slots", C.c_int), ("slots", _P)]


class MimoWeightsArgs(C.Structure):
    _fields_ = [("layer", MimoLayer), ("batch", C.c_int), ("q_len", C.c_int), ("max_seq_len", C.c_int), ("q", _P),
                ("lse", _P), ("seq_lens", _P), ("positions", _P), ("k_cache", _P), ("block_table", _P),
                ("max_pages", C.c_int), ("num_pages", C.c_int), ("cache_dtype", C.c_int), ("k_dequant", _P),
                ("scores", _P), ("score_stride", C.c_int)]


class MimoSelectArgs(C.Structure):
    _fields_ = [("num_seqs", C.c_int), ("num_kv_heads", C.c_int), ("scores", _P), ("score_stride", C.c_int),
                ("seq_lens", _P), ("max_seq_len", C.c_int), ("keep", C.c_int), ("recent", C.c_int), ("first", C.c_int),
                ("idx", _P), ("counts", _P), ("scores_out", _P)]


class MimoGatherArgs(C.Structure):
    _fields_ = [("num_seqs", C.c_int), ("num_kv_heads", C.c_int), ("k_src", _P), ("v_src", _P),
                ("block_table_src", _P), ("max_pages_src", C.c_int), ("num_pages_src", C.c_int), ("k_dst", _P),
                ("v_dst", _P), ("block_table_dst", _P), ("max_pages_dst", C.c_int), ("num_pages_dst", C.c_int),
                ("counts", _P), ("idx", _P), ("idx_stride", C.c_int), ("max_count", C.c_int),
                ("cache_dtype", C.c_int), ("out_dtype", C.c_int), ("k_dequant", _P), ("v_dequant", _P)]


_lib = None


class MimoError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"[{code}] {msg}")
        self.code = code


def lib():
    """The loaded libmimoattn (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"libmimoattn is not built ({LIB_PATH} missing): run "
                               "python -m global_attention_attn_b200.build")
        L = C.CDLL(LIB_PATH)
        L.mimo_attn_prefill.argtypes = [C.POINTER(MimoPrefillArgs), _P]
        L.mimo_attn_prefill.restype = C.c_int
        L.mimo_attn_prefill_workspace_size.argtypes = [C.c_int, C.c_int, C.c_int, C.c_int, C.c_int]
        L.mimo_attn_prefill_workspace_size.restype = C.c_size_t
        L.mimo_attn_prefill_stall_test.argtypes = [C.POINTER(MimoPrefillArgs), _P, C.c_ulonglong]
        L.mimo_attn_prefill_stall_test.restype = C.c_int
        L.mimo_attn_decode.argtypes = [C.POINTER(MimoDecodeArgs), _P]
        L.mimo_attn_decode.restype = C.c_int
        L.mimo_attn_decode_workspace_size.argtypes = [C.c_int, C.c_int, C.c_int, C.c_int]
        L.mimo_attn_decode_workspace_size.restype = C.c_size_t
        L.mimo_attn_verify_workspace_size.argtypes = [C.c_int, C.c_int, C.c_int, C.c_int, C.c_int]
        L.mimo_attn_verify_workspace_size.restype = C.c_size_t
        L.mimo_attn_decode_int4_workspace_size.argtypes = [C.c_int] * 6
        L.mimo_attn_decode_int4_workspace_size.restype = C.c_size_t
        L.mimo_attn_decode_noalloc.argtypes = [C.POINTER(MimoDecodeArgs), _P]
        L.mimo_attn_decode_noalloc.restype = C.c_int
        L.mimo_kv_append.argtypes = [C.POINTER(MimoAppendArgs), _P]
        L.mimo_kv_append.restype = C.c_int
        L.mimo_attn_weights.argtypes = [C.POINTER(MimoWeightsArgs), _P]
        L.mimo_attn_weights.restype = C.c_int
        L.mimo_kv_select.argtypes = [C.POINTER(MimoSelectArgs), _P]
        L.mimo_kv_select.restype = C.c_int
        L.mimo_kv_gather.argtypes = [C.POINTER(MimoGatherArgs), _P]
        L.mimo_kv_gather.restype = C.c_int
        L.mimo_last_error.argtypes = []
        L.mimo_last_error.restype = C.c_char_p
        L.mimo_status_poll.argtypes = [C.POINTER(C.c_uint32)]
        L.mimo_status_poll.restype = C.c_int
        L.mimo_version.argtypes = []
        L.mimo_version.restype = C.c_char_p
        L.mimo_window_from_left_right.argtypes = [C.c_int, C.c_int, C.POINTER(C.c_int)]
        L.mimo_window_from_left_right.restype = C.c_int
        _lib = L
    return _lib


def _check(rc: int):
    if rc != MIMO_OK:
        raise MimoError(rc, lib().mimo_last_error().decode())


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(stream, t):
    """Handle of the stream that a call on tensor t goes to.  The library works on the current device:
    tensors of another one are refused, whatever the stream."""
    import torch
    if t.is_cuda and t.device.index != torch.cuda.current_device():
        raise ValueError(f"the tensors are on {t.device}, which is not the current device")
    if stream is None:
        # (the handle alone: making a torch.cuda.Stream of it takes 3 us, a quarter of a short decode)
        return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def _new(like, shape, dtype, stream):
    """A tensor for a call on `stream`, on the device of `like`.  Memory made for another stream than
    the current one is that stream's: a block of the current stream's may still be read there when
    the call runs, and one given back to it would be handed out again before the call has run.  The
    current stream is noted as a user of it, so that its reads are waited for too."""
    if stream is None or not like.is_cuda:
        return like.new_empty(shape, dtype=dtype)
    import torch
    here = torch.cuda.current_stream()
    handle = _stream(stream, like)
    if handle == here.cuda_stream:
        return like.new_empty(shape, dtype=dtype)
    if not isinstance(stream, torch.cuda.Stream):  # (0 and 1 are the legacy default stream)
        stream = torch.cuda.ExternalStream(handle) if handle > 1 else torch.cuda.default_stream()
    with torch.cuda.stream(stream):
        t = like.new_empty(shape, dtype=dtype)
    t.record_stream(here)
    return t


def _check32(t, size: int, name: str):
    if t.numel() != size or t.element_size() != 4 or not t.is_contiguous():
        raise ValueError(f"{name} is a contiguous 32-bit tensor of {size} elements")


def _check_input(t, size: int, name: str, like, dtype: str = "int32"):
    """A small input, which the kernels read `size` elements of."""
    if str(t.dtype) != "torch." + dtype or t.numel() < size or not t.is_contiguous() or t.device != like.device:
        raise ValueError(f"{name} is a contiguous {dtype} tensor of {size} elements on {like.device}")


def _check_table(t, rows: int, name: str, like):
    if t.ndim != 2:
        raise ValueError(f"{name} is a contiguous int32 [{rows}, pages] tensor")
    _check_input(t, rows * t.shape[1], name, like)


def make_layer(num_kv_heads: int, rope_base: float, window: int, sink=None, softmax_scale: float = SOFTMAX_SCALE,
               v_scale: float = V_SCALE) -> MimoLayer:
    L = MimoLayer()
    L.num_q_heads, L.num_kv_heads, L.head_dim_qk, L.head_dim_v, L.rope_dim = (NUM_Q_HEADS, num_kv_heads,
                                                                             HEAD_DIM_QK, HEAD_DIM_V, ROPE_DIM)
    L.rope_base, L.softmax_scale, L.v_scale, L.window = float(rope_base), float(softmax_scale), float(v_scale), int(window)
    L.sink = _ptr(sink)
    return L


def prefill_workspace_size(num_seqs: int, total_q: int, total_k: int, num_kv_heads: int, cache_kind: int) -> int:
    return int(lib().mimo_attn_prefill_workspace_size(num_seqs, total_q, total_k, num_kv_heads, cache_kind))


def decode_workspace_size(batch: int, max_seq_len: int, num_kv_heads: int, window: int, q_len: int = 1,
                          cache_dtype: int = MIMO_DTYPE_BF16, cache_kind: int = MIMO_CACHE_PAGED) -> int:
    if cache_dtype == MIMO_DTYPE_INT4:
        return int(lib().mimo_attn_decode_int4_workspace_size(batch, q_len, max_seq_len, num_kv_heads, window, cache_kind))
    if q_len == 1:
        return int(lib().mimo_attn_decode_workspace_size(batch, max_seq_len, num_kv_heads, window))
    return int(lib().mimo_attn_verify_workspace_size(batch, q_len, max_seq_len, num_kv_heads, window))


def _events(pair):
    """cudaEvent_t handles of a (begin, end) pair of torch.cuda.Event (None: no hooks)."""
    if pair is None:
        return None, None
    handles = [int(ev.cuda_event) for ev in pair]
    if len(handles) != 2 or not all(handles):
        raise ValueError("kernel_events: pass two torch.cuda.Event that have been recorded once")
    return handles[0], handles[1]


def mimo_attn_prefill(q, k, v, cu_seqlens_q, cu_seqlens_k, *, num_kv_heads: int, rope_base: float, window: int,
                      sink=None, cache_lens=None, cache_kind: int = MIMO_CACHE_NONE, k_cache=None, v_cache=None,
                      block_table=None, num_pages: int = 0, out=None, lse=None, workspace=None,
                      softmax_scale: float = SOFTMAX_SCALE, v_scale: float = V_SCALE, stream=None,
                      with_lse: bool = True, kernel_events=None, ring_slots: int = 0,
                      stall_test_wait_ns: int | None = None):
    """Varlen prefill (see include/mimoattn.h).  Tensors are CUDA tensors: q/k/v/caches bf16,
    index tensors int32, sink fp32.  kernel_events: optional (begin, end) pair of recorded-once
    torch.cuda.Event placed around the attention kernel.  ring_slots: slots per sequence of a
    ring cache (0 = 128).  stall_test_wait_ns: call mimo_attn_prefill_stall_test instead (the
    failure-detection test whose waits run out after that many ns).  Returns (out, lse)."""
    import torch
    total_q = q.shape[0]
    num_seqs = cu_seqlens_q.shape[0] - 1
    total_k = 0 if k is None else k.shape[0]
    if out is None:
        out = _new(q, (total_q, NUM_Q_HEADS, HEAD_DIM_V), torch.bfloat16, stream)
    if lse is None and with_lse:
        lse = _new(q, (total_q, NUM_Q_HEADS), torch.float32, stream)
    need = prefill_workspace_size(num_seqs, total_q, total_k, num_kv_heads, cache_kind)
    if workspace is None and need:
        workspace = _new(q, (need,), torch.uint8, stream)
    a = MimoPrefillArgs()
    a.layer = make_layer(num_kv_heads, rope_base, window, sink, softmax_scale, v_scale)
    a.num_seqs, a.total_q, a.total_k = num_seqs, total_q, total_k
    a.q, a.k, a.v = _ptr(q), _ptr(k), _ptr(v)
    a.cu_seqlens_q, a.cu_seqlens_k, a.cache_lens = _ptr(cu_seqlens_q), _ptr(cu_seqlens_k), _ptr(cache_lens)
    a.cache_kind = cache_kind
    a.k_cache, a.v_cache, a.block_table = _ptr(k_cache), _ptr(v_cache), _ptr(block_table)
    a.max_pages = 0 if block_table is None else block_table.shape[1]
    a.num_pages = num_pages
    a.out, a.lse = _ptr(out), _ptr(lse)
    a.workspace = _ptr(workspace)
    a.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    a.ev_kernel_begin, a.ev_kernel_end = _events(kernel_events)
    a.ring_slots = int(ring_slots)
    if stall_test_wait_ns is not None:
        _check(lib().mimo_attn_prefill_stall_test(C.byref(a), _stream(stream, q), int(stall_test_wait_ns)))
    else:
        _check(lib().mimo_attn_prefill(C.byref(a), _stream(stream, q)))
    return out, lse


def mimo_attn_decode(q, seq_lens, *, max_seq_len: int, num_kv_heads: int, rope_base: float, window: int,
                     cache_kind: int, k_cache, v_cache, block_table=None, num_pages: int = 0, sink=None, out=None,
                     lse=None, workspace=None, softmax_scale: float = SOFTMAX_SCALE, v_scale: float = V_SCALE,
                     stream=None, with_lse: bool = True, kernel_events=None, cache_dtype: int = MIMO_DTYPE_BF16,
                     k_dequant=None, v_dequant=None, ring_slots: int = 0, q_len: int = 1, positions=None):
    """Decode step (see include/mimoattn.h).  kernel_events as for mimo_attn_prefill (around the
    split kernel, not the combine).  ring_slots: slots per sequence of a ring cache (0 = 128).
    q_len: query tokens per sequence (draft tokens to verify; q holds batch * q_len rows).
    cache_dtype: MIMO_DTYPE_BF16, MIMO_DTYPE_FP8_E4M3 (with k_dequant / v_dequant) or
    MIMO_DTYPE_INT4 (uint8 caches, see empty_int4_cache).  positions: int32 [batch] rotary
    position of each sequence's last query token (None: seq_lens - 1), for evicted caches.
    Returns (out, lse)."""
    import torch
    rows = q.shape[0]
    if rows % q_len:
        raise ValueError("q holds batch * q_len rows")
    B = rows // q_len
    if positions is not None:
        _check_input(positions, B, "positions", q)
    if out is None:
        out = _new(q, (rows, NUM_Q_HEADS, HEAD_DIM_V), torch.bfloat16, stream)
    if lse is None and with_lse:
        lse = _new(q, (rows, NUM_Q_HEADS), torch.float32, stream)
    if workspace is None:
        need = decode_workspace_size(B, max_seq_len, num_kv_heads, window, q_len, cache_dtype, cache_kind)
        if need:
            workspace = _new(q, (need,), torch.uint8, stream)
    a = MimoDecodeArgs()
    a.layer = make_layer(num_kv_heads, rope_base, window, sink, softmax_scale, v_scale)
    a.batch, a.max_seq_len = B, int(max_seq_len)
    a.q, a.seq_lens = _ptr(q), _ptr(seq_lens)
    a.cache_kind = cache_kind
    a.k_cache, a.v_cache, a.block_table = _ptr(k_cache), _ptr(v_cache), _ptr(block_table)
    a.max_pages = 0 if block_table is None else block_table.shape[1]
    a.num_pages = num_pages
    a.out, a.lse = _ptr(out), _ptr(lse)
    a.workspace = _ptr(workspace)
    a.workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    a.ev_kernel_begin, a.ev_kernel_end = _events(kernel_events)
    a.cache_dtype, a.k_dequant, a.v_dequant = cache_dtype, _ptr(k_dequant), _ptr(v_dequant)
    a.ring_slots, a.q_len = int(ring_slots), int(q_len)
    a.positions = _ptr(positions)
    _check(lib().mimo_attn_decode(C.byref(a), _stream(stream, q)))
    return out, lse


def mimo_attn_decode_noalloc(q, seq_lens, *, max_seq_len: int, num_kv_heads: int, rope_base: float, window: int,
                             cache_kind: int, k_cache, v_cache, out, lse=None, block_table=None, num_pages: int = 0,
                             sink=None, softmax_scale: float = SOFTMAX_SCALE, v_scale: float = V_SCALE, stream=None,
                             cache_dtype: int = MIMO_DTYPE_BF16, k_dequant=None, v_dequant=None, ring_slots: int = 0,
                             q_len: int = 1, positions=None):
    """Decode that allocates nothing (see mimo_attn_decode_noalloc in include/mimoattn.h): the
    caller passes the output buffers; the split-KV partials go to the library's static
    device scratch (16 MiB), so concurrent calls must not overlap on the GPU.  q_len and positions
    as for mimo_attn_decode."""
    if q.shape[0] % q_len:
        raise ValueError("q holds batch * q_len rows")
    B = q.shape[0] // q_len
    if positions is not None:
        _check_input(positions, B, "positions", q)
    a = MimoDecodeArgs()
    a.layer = make_layer(num_kv_heads, rope_base, window, sink, softmax_scale, v_scale)
    a.batch, a.max_seq_len = B, int(max_seq_len)
    a.q, a.seq_lens = _ptr(q), _ptr(seq_lens)
    a.cache_kind = cache_kind
    a.k_cache, a.v_cache, a.block_table = _ptr(k_cache), _ptr(v_cache), _ptr(block_table)
    a.max_pages = 0 if block_table is None else block_table.shape[1]
    a.num_pages = num_pages
    a.out, a.lse = _ptr(out), _ptr(lse)
    a.cache_dtype, a.k_dequant, a.v_dequant = cache_dtype, _ptr(k_dequant), _ptr(v_dequant)
    a.ring_slots, a.q_len = int(ring_slots), int(q_len)
    a.positions = _ptr(positions)
    _check(lib().mimo_attn_decode_noalloc(C.byref(a), _stream(stream, q)))
    return out, lse


def mimo_kv_append(k_new, v_new, pos, seq_idx, *, rope_base: float, cache_kind: int, k_cache, v_cache,
                   num_seqs: int, block_table=None, num_pages: int = 0, stream=None,
                   cache_dtype: int = MIMO_DTYPE_BF16, k_dequant=None, v_dequant=None, ring_slots: int = 0,
                   slots=None):
    """Rotate and store new keys/values into the ring or paged cache (see include/mimoattn.h);
    an E4M3 cache (cache_dtype) quantises with the per-KV-head scales k_dequant / v_dequant, a
    4-bit cache with scales of its own.  ring_slots: slots per sequence of a ring cache (0 =
    128).  slots: int32 [tokens] cache slot of each token where it is not pos (paged caches)."""
    if slots is not None:
        _check_input(slots, k_new.shape[0], "slots", k_new)
    a = MimoAppendArgs()
    a.num_tokens, a.num_kv_heads = k_new.shape[0], k_new.shape[1]
    a.head_dim_qk, a.head_dim_v, a.rope_dim, a.rope_base = HEAD_DIM_QK, HEAD_DIM_V, ROPE_DIM, float(rope_base)
    a.k_new, a.v_new, a.pos, a.seq_idx = _ptr(k_new), _ptr(v_new), _ptr(pos), _ptr(seq_idx)
    a.cache_kind = cache_kind
    a.k_cache, a.v_cache = _ptr(k_cache), _ptr(v_cache)
    a.num_seqs = num_seqs
    a.block_table = _ptr(block_table)
    a.max_pages = 0 if block_table is None else block_table.shape[1]
    a.num_pages = num_pages
    a.cache_dtype, a.k_dequant, a.v_dequant = cache_dtype, _ptr(k_dequant), _ptr(v_dequant)
    a.ring_slots, a.slots = int(ring_slots), _ptr(slots)
    _check(lib().mimo_kv_append(C.byref(a), _stream(stream, k_new)))


def mimo_attn_weights(q, lse, scores, seq_lens, *, max_seq_len: int, num_kv_heads: int, rope_base: float, k_cache,
                      block_table, num_pages: int, cache_dtype: int = MIMO_DTYPE_BF16, k_dequant=None, positions=None,
                      q_len: int = 1, softmax_scale: float = SOFTMAX_SCALE, stream=None):
    """Adds the attention weights of a decode call (its q, lse, seq_lens, positions) to the float32
    scores [batch, num_kv_heads, slots] of a paged cache's slots (see include/mimoattn.h).
    Returns scores."""
    if q.shape[0] % q_len:
        raise ValueError("q holds batch * q_len rows")
    B = q.shape[0] // q_len
    if (scores.ndim != 3 or scores.shape[0] != B or scores.shape[1] != num_kv_heads or not scores.is_contiguous()
            or scores.element_size() != 4):
        raise ValueError("scores is a contiguous float32 [batch, num_kv_heads, slots] tensor")
    _check_input(lse, q.shape[0] * NUM_Q_HEADS, "lse", q, "float32")
    _check_input(seq_lens, B, "seq_lens", q)
    if positions is not None:
        _check_input(positions, B, "positions", q)
    _check_table(block_table, B, "block_table", q)
    a = MimoWeightsArgs()
    a.layer = make_layer(num_kv_heads, rope_base, 0, None, softmax_scale, 1.0)
    a.batch, a.q_len, a.max_seq_len = B, int(q_len), int(max_seq_len)
    a.q, a.lse, a.seq_lens, a.positions = _ptr(q), _ptr(lse), _ptr(seq_lens), _ptr(positions)
    a.k_cache, a.block_table = _ptr(k_cache), _ptr(block_table)
    a.max_pages, a.num_pages = block_table.shape[1], num_pages
    a.cache_dtype, a.k_dequant = cache_dtype, _ptr(k_dequant)
    a.scores, a.score_stride = _ptr(scores), scores.shape[2]
    _check(lib().mimo_attn_weights(C.byref(a), _stream(stream, q)))
    return scores


def mimo_kv_select(scores, seq_lens, *, max_seq_len: int, keep: int, recent: int = 0, first: int = 0, idx=None,
                   counts=None, scores_out=None, stream=None):
    """The slots that stay of every (sequence, KV head): the first `first`, the last `recent`, and the
    largest scores of the others, `keep` in all (see include/mimoattn.h).  scores: float32
    [num_seqs, num_kv_heads, slots].  Returns (idx int32 [num_seqs, num_kv_heads, keep] ascending,
    padded with -1; counts int32 [num_seqs]; the kept slots' scores, padded with 0)."""
    import torch
    if scores.ndim != 3 or not scores.is_contiguous() or scores.element_size() != 4:
        raise ValueError("scores is a contiguous float32 [num_seqs, num_kv_heads, slots] tensor")
    n, h, slots = scores.shape
    _check_input(seq_lens, n, "seq_lens", scores)
    if idx is None:
        idx = _new(scores, (n, h, keep), torch.int32, stream)
    else:
        _check32(idx, n * h * keep, "idx")
    if counts is None:
        counts = _new(scores, (n,), torch.int32, stream)
    else:
        _check32(counts, n, "counts")
    if scores_out is None:
        scores_out = _new(scores, (n, h, keep), torch.float32, stream)
    else:
        _check32(scores_out, n * h * keep, "scores_out")
    a = MimoSelectArgs()
    a.num_seqs, a.num_kv_heads, a.scores, a.score_stride = n, h, _ptr(scores), slots
    a.seq_lens, a.max_seq_len = _ptr(seq_lens), int(max_seq_len)
    a.keep, a.recent, a.first = int(keep), int(recent), int(first)
    a.idx, a.counts, a.scores_out = _ptr(idx), _ptr(counts), _ptr(scores_out)
    _check(lib().mimo_kv_select(C.byref(a), _stream(stream, scores)))
    return idx, counts, scores_out


def mimo_kv_gather(k_src, v_src, block_table_src, k_dst, v_dst, block_table_dst, counts, *, num_kv_heads: int,
                   num_pages: int, num_pages_out: int, idx=None, max_count: int | None = None,
                   cache_dtype: int = MIMO_DTYPE_BF16, out_dtype: int | None = None, k_dequant=None, v_dequant=None,
                   stream=None):
    """Moves slots idx[s, g, j] (None: slot j) of a paged cache to slots j < counts[s] of other pages
    (see include/mimoattn.h).  out_dtype: cache_dtype (None), or MIMO_DTYPE_BF16 to widen an E4M3 or
    4-bit cache.  max_count: upper bound of counts (None: what idx or the destination table holds)."""
    a = MimoGatherArgs()
    a.num_seqs, a.num_kv_heads = block_table_src.shape[0], num_kv_heads
    if block_table_dst.shape[0] != a.num_seqs or counts.shape[0] != a.num_seqs:
        raise ValueError("both block tables and counts have a row per sequence")
    _check_input(counts, a.num_seqs, "counts", k_src)
    _check_table(block_table_src, a.num_seqs, "block_table_src", k_src)
    _check_table(block_table_dst, a.num_seqs, "block_table_dst", k_src)
    if idx is not None and (idx.ndim != 3 or tuple(idx.shape[:2]) != (a.num_seqs, num_kv_heads) or not idx.is_contiguous()
                            or idx.element_size() != 4):
        raise ValueError("idx is a contiguous int32 [num_seqs, num_kv_heads, n] tensor")
    if max_count is None:
        max_count = block_table_dst.shape[1] * 128
        if idx is not None:
            max_count = min(max_count, idx.shape[2])
    a.k_src, a.v_src, a.block_table_src = _ptr(k_src), _ptr(v_src), _ptr(block_table_src)
    a.max_pages_src, a.num_pages_src = block_table_src.shape[1], num_pages
    a.k_dst, a.v_dst, a.block_table_dst = _ptr(k_dst), _ptr(v_dst), _ptr(block_table_dst)
    a.max_pages_dst, a.num_pages_dst = block_table_dst.shape[1], num_pages_out
    a.counts, a.idx, a.idx_stride = _ptr(counts), _ptr(idx), 0 if idx is None else idx.shape[2]
    a.max_count = int(max_count)
    a.cache_dtype, a.out_dtype = cache_dtype, cache_dtype if out_dtype is None else out_dtype
    a.k_dequant, a.v_dequant = _ptr(k_dequant), _ptr(v_dequant)
    _check(lib().mimo_kv_gather(C.byref(a), _stream(stream, k_src)))


def empty_int4_cache(blocks: int, num_kv_heads: int, ring_slots: int = 0, device="cuda"):
    """Zeroed (k_cache, v_cache) of a 4-bit cache: `blocks` pages of 128 slots, or (ring_slots > 0)
    `blocks` sequences' rings; uint8 [blocks, num_kv_heads, slots * bytes per slot]."""
    import torch
    n = ring_slots or 128
    return tuple(torch.zeros((blocks, num_kv_heads, n * b), dtype=torch.uint8, device=device)
                 for b in (MIMO_INT4_K_SLOT_BYTES, MIMO_INT4_V_SLOT_BYTES))


def mimo_window_from_left_right(left: int, right: int = 0) -> int:
    """`window` (keys in total including the query) of the (left, right) window form:
    (128, 0) -> 129, (127, 0) -> 128, (-1, 0) -> 0 (global)."""
    w = C.c_int(0)
    _check(lib().mimo_window_from_left_right(int(left), int(right), C.byref(w)))
    return int(w.value)


def status_poll() -> int:
    """Reads and clears the device status word (synchronises the device)."""
    st = C.c_uint32(0)
    rc = lib().mimo_status_poll(C.byref(st))
    if rc not in (MIMO_OK, MIMO_ERR_TIMEOUT):
        _check(rc)
    return int(st.value)
