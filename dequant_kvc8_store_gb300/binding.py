"""ctypes binding of libkvc8 (``include/kvc8.h``): argument marshalling only.

The functions carry the C names and argument order.  Tensor arguments may be
torch tensors (their ``data_ptr()`` is passed), plain integer addresses, or
None for NULL.  ``stream=None`` means torch's current CUDA stream.  A non-OK
status raises :class:`Kvc8Error`.  There is no fallback: if the library cannot
be built or loaded, importing the binding's functions fails loudly.
"""
from __future__ import annotations

import ctypes
import os
import re
import threading

from . import buildlib as _build

OK = 0
ERR_INVALID_ARG = 1
ERR_UNSUPPORTED = 2
ERR_CUDA = 3
ERR_DEVICE_BOUNDS = 4
ERR_WORKSPACE = 5

DEV_OK = 0
DEV_BAD_BLOCK_ID = 1
DEV_POS_BEYOND_TABLE = 2
DEV_OUT_ROW_RANGE = 3
DEV_BAD_LENGTH = 4
DEV_TIMEOUT = 5

ROPE_PLAIN = 0
ROPE_LINEAR = 1
ROPE_BASE = 2
ROPE_BY_PARTS = 3

HEADER = os.path.join(_build.INCLUDE, "kvc8.h")


class Kvc8Error(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_name(status)} ({status})")


class Geom(ctypes.Structure):
    """kvc8_geom."""
    _fields_ = [("num_seqs", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_blocks", ctypes.c_int32), ("max_blocks_per_seq", ctypes.c_int32),
                ("quant_mode", ctypes.c_int32)]

    def __repr__(self):
        return "Geom(" + ", ".join(f"{n}={getattr(self, n)}" for n, _ in self._fields_) + ")"


class RopeStruct(ctypes.Structure):
    """kvc8_rope."""
    _fields_ = [("rotary_dim", ctypes.c_int32), ("interleaved", ctypes.c_int32),
                ("attention_factor", ctypes.c_float), ("norm_eps", ctypes.c_float),
                ("freqs", ctypes.c_void_p), ("q_norm_weight", ctypes.c_void_p),
                ("k_norm_weight", ctypes.c_void_p), ("positions", ctypes.c_void_p)]


class Rope:
    """kvc8_rope with its device arrays: tensors, integer addresses or None,
    held here for as long as the calls may use them."""

    def __init__(self, rotary_dim, freqs, interleaved=0, attention_factor=1.0, norm_eps=1e-6,
                 q_norm_weight=None, k_norm_weight=None, positions=None):
        self.freqs, self.positions = freqs, positions
        self.q_norm_weight, self.k_norm_weight = q_norm_weight, k_norm_weight
        self.struct = RopeStruct(int(rotary_dim), int(interleaved), float(attention_factor),
                                 float(norm_eps), _p(freqs), _p(q_norm_weight), _p(k_norm_weight),
                                 _p(positions))


class RopeScaling(ctypes.Structure):
    """kvc8_rope_scaling."""
    _fields_ = [("kind", ctypes.c_int32), ("base", ctypes.c_double), ("factor", ctypes.c_double),
                ("original_positions", ctypes.c_double), ("low", ctypes.c_double),
                ("high", ctypes.c_double)]


_lock = threading.Lock()
_lib = None


def declared_functions() -> list:
    """Names of the functions that include/kvc8.h declares."""
    text = open(HEADER).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    return sorted(set(re.findall(r"\b(kvc8_\w+)\s*\(", text)))


def configure(lib: ctypes.CDLL) -> ctypes.CDLL:
    """Declare the C signatures of kvc8.h on a loaded copy of the library."""
    P, i32, i64, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    G = ctypes.POINTER(Geom)
    lib.kvc8_status_str.argtypes = [ctypes.c_int]
    lib.kvc8_status_str.restype = ctypes.c_char_p
    lib.kvc8_version.argtypes = []
    lib.kvc8_version.restype = i32
    lib.kvc8_store.argtypes = [G, i64, P, P, i64, i64, P, P, P, P, P, P, P, P, P]
    lib.kvc8_store.restype = ctypes.c_int
    lib.kvc8_gather_workspace_bytes.argtypes = [G]
    lib.kvc8_gather_workspace_bytes.restype = sz
    lib.kvc8_build_metadata.argtypes = [G, P, P, P, P, sz, P, P]
    lib.kvc8_build_metadata.restype = ctypes.c_int
    lib.kvc8_dequant_gather.argtypes = [G, P, P, P, P, P, P, P, P, P, i64, i64, i64, P, sz, P, P]
    lib.kvc8_dequant_gather.restype = ctypes.c_int
    lib.kvc8_dequant_gather_planned.argtypes = [G, P, P, P, P, P, P, P, P, i64, i64, i64, P, sz,
                                                P, P]
    lib.kvc8_dequant_gather_planned.restype = ctypes.c_int
    lib.kvc8_get_error.argtypes = [P, ctypes.POINTER(ctypes.c_int32), i32, P]
    lib.kvc8_get_error.restype = ctypes.c_int
    lib.kvc8_dequant_gather_noalloc.argtypes = [G, P, P, P, P, P, P, P, P, P, i64, i64, i64, P, P]
    lib.kvc8_dequant_gather_noalloc.restype = ctypes.c_int
    lib.kvc8_store_bf16.argtypes = [G, i64, P, P, i64, i64, P, P, P, P, P, P, P]
    lib.kvc8_store_bf16.restype = ctypes.c_int
    lib.kvc8_gather_bf16.argtypes = [G, P, P, P, P, P, P, P, i64, i64, i64, P, sz, P, P]
    lib.kvc8_gather_bf16.restype = ctypes.c_int
    lib.kvc8_attention_workspace_bytes.argtypes = [G, i32]
    lib.kvc8_attention_workspace_bytes.restype = sz
    lib.kvc8_paged_decode_attention.argtypes = [G, i32, P, i64, i64, P, P, P, P, P, P,
                                                ctypes.c_float, P, i64, i64, P, sz, P, P]
    lib.kvc8_paged_decode_attention.restype = ctypes.c_int
    lib.kvc8_append_gather.argtypes = [G, i64, P, P, i64, i64, P, P, P, P, P, P, P, P, P, P, i64,
                                       i64, i64, P, sz, P, P]
    lib.kvc8_append_gather.restype = ctypes.c_int
    lib.kvc8_build_append_metadata.argtypes = [G, P, P, P, P, P, sz, P, P]
    lib.kvc8_build_append_metadata.restype = ctypes.c_int
    lib.kvc8_append_gather_planned.argtypes = [G, i64, P, P, i64, i64, P, P, P, P, P, P, P, P, P,
                                               i64, i64, i64, P, sz, P, P]
    lib.kvc8_append_gather_planned.restype = ctypes.c_int
    R = ctypes.POINTER(RopeStruct)
    lib.kvc8_rope_frequencies.argtypes = [ctypes.POINTER(RopeScaling), i32,
                                          ctypes.POINTER(ctypes.c_uint64),
                                          ctypes.POINTER(ctypes.c_float)]
    lib.kvc8_rope_frequencies.restype = ctypes.c_int
    lib.kvc8_rope_store.argtypes = [G, R, i64, i32, P, i64, i64, P, i64, i64, P, P, i64, i64, P, P,
                                    P, P, P, P, P, P, P]
    lib.kvc8_rope_store.restype = ctypes.c_int
    lib.kvc8_rope_store_bf16.argtypes = [G, R, i64, i32, P, i64, i64, P, i64, i64, P, P, i64, i64,
                                         P, P, P, P, P, P, P]
    lib.kvc8_rope_store_bf16.restype = ctypes.c_int
    lib.kvc8_qk_norm_rope.argtypes = [R, i64, i32, i32, P, i64, i64, P, i64, i64, i32, P, i64, i64,
                                      P, i64, i64, P]
    lib.kvc8_qk_norm_rope.restype = ctypes.c_int
    lib.kvc8_shared_prefix_workspace_bytes.argtypes = [G, i32, i32]
    lib.kvc8_shared_prefix_workspace_bytes.restype = sz
    lib.kvc8_shared_prefix_attention.argtypes = [G, i32, P, i64, i64, P, P, P, P, P, i32, P, P, P,
                                                 ctypes.c_float, P, i64, i64, P, sz, P, P]
    lib.kvc8_shared_prefix_attention.restype = ctypes.c_int
    return lib


def load(build_if_needed: bool = True) -> ctypes.CDLL:
    """Load libkvc8.so (building it with nvcc first if it is missing or stale)."""
    global _lib
    if _lib is not None:
        return _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.build() if build_if_needed else _build.LIB_PATH
        if not os.path.exists(path):
            raise ImportError(f"libkvc8 is not built ({path}); run dequant_kvc8_store_gb300/buildlib.py")
        _lib = configure(ctypes.CDLL(path))
        return _lib


def status_name(status: int) -> str:
    try:
        return load().kvc8_status_str(int(status)).decode()
    except Exception:  # while reporting a load failure
        return "status"


def _p(x):
    """Device/host address of a tensor, int address, or None."""
    if x is None:
        return None
    if isinstance(x, int):
        return x
    return x.data_ptr()


_current_stream = None


def _find_current_stream():
    """torch's current stream as an address.  Asked for on every call, so by the
    lookup under torch.cuda.current_stream() where torch has it (0.3 us against
    2.9 us for the Stream object)."""
    import torch
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if raw is None:
        return lambda: torch.cuda.current_stream().cuda_stream
    return lambda: raw(torch.cuda.current_device())


def _stream(stream):
    global _current_stream
    if stream is None:
        if _current_stream is None:
            _current_stream = _find_current_stream()
        return _current_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _ok(status: int, where: str):
    if status != OK:
        raise Kvc8Error(status, where)


def kvc8_version() -> int:
    return int(load().kvc8_version())


def kvc8_status_str(status: int) -> str:
    return load().kvc8_status_str(int(status)).decode()


def kvc8_store(g: Geom, num_tokens, key_states, value_states, x_tok_stride, x_head_stride,
               key_cache, value_cache, key_scale, value_scale, block_table, cu_q_lens,
               context_kv_lens, dev_error=None, stream=None) -> None:
    st = load().kvc8_store(ctypes.byref(g), int(num_tokens), _p(key_states), _p(value_states),
                           int(x_tok_stride), int(x_head_stride), _p(key_cache),
                           _p(value_cache), _p(key_scale), _p(value_scale), _p(block_table),
                           _p(cu_q_lens), _p(context_kv_lens), _p(dev_error), _stream(stream))
    _ok(st, "kvc8_store")


def kvc8_gather_workspace_bytes(g: Geom) -> int:
    return int(load().kvc8_gather_workspace_bytes(ctypes.byref(g)))


def kvc8_build_metadata(g: Geom, context_lengths, context_seq_offset, offsets_out, workspace,
                        workspace_bytes, dev_error=None, stream=None) -> None:
    st = load().kvc8_build_metadata(ctypes.byref(g), _p(context_lengths), _p(context_seq_offset),
                                    _p(offsets_out), _p(workspace), int(workspace_bytes),
                                    _p(dev_error), _stream(stream))
    _ok(st, "kvc8_build_metadata")


def kvc8_dequant_gather(g: Geom, key_cache, value_cache, key_scale, value_scale, block_table,
                        context_lengths, context_seq_offset, key_out, value_out, out_rows,
                        out_tok_stride, out_head_stride, workspace, workspace_bytes,
                        dev_error=None, stream=None) -> None:
    st = load().kvc8_dequant_gather(ctypes.byref(g), _p(key_cache), _p(value_cache),
                                    _p(key_scale), _p(value_scale), _p(block_table),
                                    _p(context_lengths), _p(context_seq_offset), _p(key_out),
                                    _p(value_out), int(out_rows), int(out_tok_stride),
                                    int(out_head_stride), _p(workspace), int(workspace_bytes),
                                    _p(dev_error), _stream(stream))
    _ok(st, "kvc8_dequant_gather")


def kvc8_dequant_gather_planned(g: Geom, key_cache, value_cache, key_scale, value_scale,
                                block_table, context_lengths, key_out, value_out, out_rows,
                                out_tok_stride, out_head_stride, workspace, workspace_bytes,
                                dev_error=None, stream=None) -> None:
    st = load().kvc8_dequant_gather_planned(ctypes.byref(g), _p(key_cache), _p(value_cache),
                                            _p(key_scale), _p(value_scale), _p(block_table),
                                            _p(context_lengths), _p(key_out), _p(value_out),
                                            int(out_rows), int(out_tok_stride),
                                            int(out_head_stride), _p(workspace),
                                            int(workspace_bytes), _p(dev_error),
                                            _stream(stream))
    _ok(st, "kvc8_dequant_gather_planned")


NOALLOC_MAX_SEQS = 4096  # KVC8_NOALLOC_MAX_SEQS


def kvc8_dequant_gather_noalloc(g: Geom, key_cache, value_cache, key_scale, value_scale,
                                block_table, context_lengths, context_seq_offset, key_out,
                                value_out, out_rows, out_tok_stride, out_head_stride,
                                dev_error=None, stream=None) -> None:
    """kvc8_dequant_gather without a workspace, for callers that cannot allocate
    device memory: the plan lives in a fixed array inside the library (one per
    device, shared by all calls, at most NOALLOC_MAX_SEQS sequences).  Make the
    first call on a device before any stream capture; calls that overlap on the
    GPU race on the shared array."""
    st = load().kvc8_dequant_gather_noalloc(ctypes.byref(g), _p(key_cache), _p(value_cache),
                                            _p(key_scale), _p(value_scale), _p(block_table),
                                            _p(context_lengths), _p(context_seq_offset),
                                            _p(key_out), _p(value_out), int(out_rows),
                                            int(out_tok_stride), int(out_head_stride),
                                            _p(dev_error), _stream(stream))
    _ok(st, "kvc8_dequant_gather_noalloc")


def kvc8_store_bf16(g: Geom, num_tokens, key_states, value_states, x_tok_stride, x_head_stride,
                    key_cache, value_cache, block_table, cu_q_lens, context_kv_lens,
                    dev_error=None, stream=None) -> None:
    st = load().kvc8_store_bf16(ctypes.byref(g), int(num_tokens), _p(key_states),
                                _p(value_states), int(x_tok_stride), int(x_head_stride),
                                _p(key_cache), _p(value_cache), _p(block_table), _p(cu_q_lens),
                                _p(context_kv_lens), _p(dev_error), _stream(stream))
    _ok(st, "kvc8_store_bf16")


def kvc8_gather_bf16(g: Geom, key_cache, value_cache, block_table, context_lengths,
                     context_seq_offset, key_out, value_out, out_rows, out_tok_stride,
                     out_head_stride, workspace, workspace_bytes, dev_error=None,
                     stream=None) -> None:
    st = load().kvc8_gather_bf16(ctypes.byref(g), _p(key_cache), _p(value_cache),
                                 _p(block_table), _p(context_lengths), _p(context_seq_offset),
                                 _p(key_out), _p(value_out), int(out_rows), int(out_tok_stride),
                                 int(out_head_stride), _p(workspace), int(workspace_bytes),
                                 _p(dev_error), _stream(stream))
    _ok(st, "kvc8_gather_bf16")


def kvc8_append_gather(g: Geom, num_tokens, key_states, value_states, x_tok_stride,
                       x_head_stride, key_cache, value_cache, key_scale, value_scale, block_table,
                       cu_q_lens, context_kv_lens, context_seq_offset, key_out, value_out,
                       out_rows, out_tok_stride, out_head_stride, workspace, workspace_bytes,
                       dev_error=None, stream=None) -> None:
    st = load().kvc8_append_gather(
        ctypes.byref(g), int(num_tokens), _p(key_states), _p(value_states), int(x_tok_stride),
        int(x_head_stride), _p(key_cache), _p(value_cache), _p(key_scale), _p(value_scale),
        _p(block_table), _p(cu_q_lens), _p(context_kv_lens), _p(context_seq_offset),
        _p(key_out), _p(value_out), int(out_rows), int(out_tok_stride), int(out_head_stride),
        _p(workspace), int(workspace_bytes), _p(dev_error), _stream(stream))
    _ok(st, "kvc8_append_gather")


def kvc8_build_append_metadata(g: Geom, cu_q_lens, context_kv_lens, context_seq_offset,
                               offsets_out, workspace, workspace_bytes, dev_error=None,
                               stream=None) -> None:
    st = load().kvc8_build_append_metadata(
        ctypes.byref(g), _p(cu_q_lens), _p(context_kv_lens), _p(context_seq_offset),
        _p(offsets_out), _p(workspace), int(workspace_bytes), _p(dev_error), _stream(stream))
    _ok(st, "kvc8_build_append_metadata")


def kvc8_append_gather_planned(g: Geom, num_tokens, key_states, value_states, x_tok_stride,
                               x_head_stride, key_cache, value_cache, key_scale, value_scale,
                               block_table, cu_q_lens, context_kv_lens, key_out, value_out,
                               out_rows, out_tok_stride, out_head_stride, workspace,
                               workspace_bytes, dev_error=None, stream=None) -> None:
    st = load().kvc8_append_gather_planned(
        ctypes.byref(g), int(num_tokens), _p(key_states), _p(value_states), int(x_tok_stride),
        int(x_head_stride), _p(key_cache), _p(value_cache), _p(key_scale), _p(value_scale),
        _p(block_table), _p(cu_q_lens), _p(context_kv_lens), _p(key_out), _p(value_out),
        int(out_rows), int(out_tok_stride), int(out_head_stride), _p(workspace),
        int(workspace_bytes), _p(dev_error), _stream(stream))
    _ok(st, "kvc8_append_gather_planned")


def kvc8_attention_workspace_bytes(g: Geom, num_q_heads: int) -> int:
    return int(load().kvc8_attention_workspace_bytes(ctypes.byref(g), int(num_q_heads)))


def kvc8_paged_decode_attention(g: Geom, num_q_heads, query, q_seq_stride, q_head_stride,
                                key_cache, value_cache, key_scale, value_scale, block_table,
                                context_lengths, softmax_scale, out, out_seq_stride,
                                out_head_stride, workspace, workspace_bytes, dev_error=None,
                                stream=None) -> None:
    st = load().kvc8_paged_decode_attention(
        ctypes.byref(g), int(num_q_heads), _p(query), int(q_seq_stride), int(q_head_stride),
        _p(key_cache), _p(value_cache), _p(key_scale), _p(value_scale), _p(block_table),
        _p(context_lengths), float(softmax_scale), _p(out), int(out_seq_stride),
        int(out_head_stride), _p(workspace), int(workspace_bytes), _p(dev_error),
        _stream(stream))
    _ok(st, "kvc8_paged_decode_attention")


def kvc8_rope_frequencies(scaling: RopeScaling, rotary_dim: int):
    """(freqs, attention_factor): the fixed-point frequencies as a numpy uint64
    array, to be copied to the device once (as int64 bits), and the factor."""
    import numpy as np
    n = int(rotary_dim)
    freqs = np.zeros(max(n // 2, 1), np.uint64)
    factor = ctypes.c_float(0.0)
    st = load().kvc8_rope_frequencies(ctypes.byref(scaling), n,
                                      freqs.ctypes.data_as(ctypes.POINTER(ctypes.c_uint64)),
                                      ctypes.byref(factor))
    _ok(st, "kvc8_rope_frequencies")
    return freqs[: n // 2], float(factor.value)


def kvc8_rope_store(g: Geom, rope: Rope, num_tokens, num_q_heads, query, q_tok_stride,
                    q_head_stride, q_out, qo_tok_stride, qo_head_stride, key_states, value_states,
                    x_tok_stride, x_head_stride, key_cache, value_cache, key_scale, value_scale,
                    block_table, cu_q_lens, context_kv_lens, dev_error=None, stream=None) -> None:
    st = load().kvc8_rope_store(
        ctypes.byref(g), ctypes.byref(rope.struct), int(num_tokens), int(num_q_heads), _p(query),
        int(q_tok_stride), int(q_head_stride), _p(q_out), int(qo_tok_stride), int(qo_head_stride),
        _p(key_states), _p(value_states), int(x_tok_stride), int(x_head_stride), _p(key_cache),
        _p(value_cache), _p(key_scale), _p(value_scale), _p(block_table), _p(cu_q_lens),
        _p(context_kv_lens), _p(dev_error), _stream(stream))
    _ok(st, "kvc8_rope_store")


def kvc8_rope_store_bf16(g: Geom, rope: Rope, num_tokens, num_q_heads, query, q_tok_stride,
                         q_head_stride, q_out, qo_tok_stride, qo_head_stride, key_states,
                         value_states, x_tok_stride, x_head_stride, key_cache, value_cache,
                         block_table, cu_q_lens, context_kv_lens, dev_error=None,
                         stream=None) -> None:
    st = load().kvc8_rope_store_bf16(
        ctypes.byref(g), ctypes.byref(rope.struct), int(num_tokens), int(num_q_heads), _p(query),
        int(q_tok_stride), int(q_head_stride), _p(q_out), int(qo_tok_stride), int(qo_head_stride),
        _p(key_states), _p(value_states), int(x_tok_stride), int(x_head_stride), _p(key_cache),
        _p(value_cache), _p(block_table), _p(cu_q_lens), _p(context_kv_lens), _p(dev_error),
        _stream(stream))
    _ok(st, "kvc8_rope_store_bf16")


def kvc8_qk_norm_rope(rope: Rope, num_tokens, head_dim, num_q_heads, query, q_tok_stride,
                      q_head_stride, q_out, qo_tok_stride, qo_head_stride, kv_heads, key,
                      k_tok_stride, k_head_stride, k_out, ko_tok_stride, ko_head_stride,
                      stream=None) -> None:
    st = load().kvc8_qk_norm_rope(
        ctypes.byref(rope.struct), int(num_tokens), int(head_dim), int(num_q_heads), _p(query),
        int(q_tok_stride), int(q_head_stride), _p(q_out), int(qo_tok_stride), int(qo_head_stride),
        int(kv_heads), _p(key), int(k_tok_stride), int(k_head_stride), _p(k_out),
        int(ko_tok_stride), int(ko_head_stride), _stream(stream))
    _ok(st, "kvc8_qk_norm_rope")


def kvc8_shared_prefix_workspace_bytes(g: Geom, num_q_heads: int, max_prefix_blocks: int) -> int:
    return int(load().kvc8_shared_prefix_workspace_bytes(ctypes.byref(g), int(num_q_heads),
                                                         int(max_prefix_blocks)))


def kvc8_shared_prefix_attention(g: Geom, num_q_heads, query, q_seq_stride, q_head_stride,
                                 key_cache, value_cache, key_scale, value_scale, prefix_table,
                                 max_prefix_blocks, prefix_length, block_table, context_lengths,
                                 softmax_scale, out, out_seq_stride, out_head_stride, workspace,
                                 workspace_bytes, dev_error=None, stream=None) -> None:
    st = load().kvc8_shared_prefix_attention(
        ctypes.byref(g), int(num_q_heads), _p(query), int(q_seq_stride), int(q_head_stride),
        _p(key_cache), _p(value_cache), _p(key_scale), _p(value_scale), _p(prefix_table),
        int(max_prefix_blocks), _p(prefix_length), _p(block_table), _p(context_lengths),
        float(softmax_scale), _p(out), int(out_seq_stride), int(out_head_stride), _p(workspace),
        int(workspace_bytes), _p(dev_error), _stream(stream))
    _ok(st, "kvc8_shared_prefix_attention")


def kvc8_get_error(dev_error, reset: bool = False, stream=None) -> int:
    """Synchronise the stream and return the device error code (0 = none)."""
    code = ctypes.c_int32(0)
    st = load().kvc8_get_error(_p(dev_error), ctypes.byref(code), int(bool(reset)),
                               _stream(stream))
    if st not in (OK, ERR_DEVICE_BOUNDS):
        raise Kvc8Error(st, "kvc8_get_error")
    return int(code.value)
