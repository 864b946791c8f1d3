"""Thin Python binding of libpkv.so (the C ABI declared in include/pkv.h).

Each function has the name of its C entry point without the ``pkv_`` prefix and only
marshals arguments: it reads shapes and device pointers off torch tensors, passes the
current CUDA stream, and turns a negative status into :class:`PkvError`. Every step of the
computation runs in the library's CUDA kernels; there is no fallback path. Loading fails
loudly if the library is missing.
"""
from __future__ import annotations

import ctypes
import os
import threading

import numpy as np
import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
# PKV_LIB selects another build of the library (e.g. a pipeline-depth variant).
LIB_PATH = os.environ.get("PKV_LIB") or os.path.join(_HERE, "libpkv.so")

# Symbols the header declares (kept in sync with include/pkv.h; the CPU tests check both).
SYMBOLS = (
    "pkv_version", "pkv_device_error", "pkv_slot_mapping", "pkv_ring_slot_mapping",
    "pkv_kv_append", "pkv_copy_blocks", "pkv_decode_workspace_bytes", "pkv_workspace_init",
    "pkv_paged_attn_decode", "pkv_rope_table", "pkv_ring_attn_decode", "pkv_check_tables",
    "pkv_check_slots", "pkv_paged_attn_decode_noalloc", "pkv_paged_attn_decode_append",
    "pkv_kv_append_fp8", "pkv_paged_attn_decode_fp8", "pkv_paged_attn_decode_append_fp8",
    "pkv_pool_create", "pkv_pool_destroy", "pkv_pool_allocate", "pkv_pool_warm",
    "pkv_pool_release", "pkv_pool_fork", "pkv_pool_append", "pkv_pool_stats",
    "pkv_pool_refcount", "pkv_spec_verify", "pkv_set_early_start", "pkv_paged_prefill",
    "pkv_ring_attn_decode_append", "pkv_kv_append_int4", "pkv_widen_blocks_int4",
    "pkv_paged_attn_decode_int4", "pkv_paged_attn_decode_append_int4", "pkv_qk_norm_rope",
    "pkv_extend_tables", "pkv_truncate_tables", "pkv_kv_append_int8", "pkv_widen_blocks_int8",
    "pkv_copy_blocks_int8", "pkv_paged_attn_decode_int8", "pkv_selected_attn_decode_int8",
    "pkv_select_blocks",
)

OK, EINVAL, ERANGE, ENOSPC, ECUDA_BASE = 0, -22, -34, -28, -1000
DEVERR_BLOCK_ID, DEVERR_CONTEXT, DEVERR_SLOT, DEVERR_TIMEOUT, DEVERR_SEQ, DEVERR_POSITION = \
    1, 2, 4, 8, 16, 32
DEVERR_TOKEN = 64
DEVERR_SPACE = 128


class PkvError(RuntimeError):
    def __init__(self, fn: str, status: int):
        self.status = status
        if status <= ECUDA_BASE:
            what = f"CUDA error {ECUDA_BASE - status}"
        else:
            what = {EINVAL: "invalid argument", ERANGE: "index out of range",
                    ENOSPC: "workspace too small"}.get(status, "error")
        super().__init__(f"{fn} failed: {what} (status {status})")


_lock = threading.Lock()
_lib = None


def load() -> ctypes.CDLL:
    """Loads libpkv.so (built by paged_kv_cache_147_gb300.build); raises if it is missing."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: build it with "
                               "`python -m paged_kv_cache_147_gb300.build` (no CPU fallback)")
        _lib = _configure(ctypes.CDLL(LIB_PATH))
        return _lib


def load_variant(path: str) -> ctypes.CDLL:
    """Loads another build of the library (e.g. one compiled with different tuning macros)
    next to the default one, with the same signatures; the tests compare the two."""
    return _configure(ctypes.CDLL(path))


def _configure(lib: ctypes.CDLL) -> ctypes.CDLL:
    """Sets the argument and result types of every entry point on a loaded library."""
    P, i32, i64, sz, f32, f64 = (ctypes.c_void_p, ctypes.c_int, ctypes.c_int64,
                                 ctypes.c_size_t, ctypes.c_float, ctypes.c_double)
    sig = {
        "pkv_version": (i32, []),
        "pkv_device_error": (i32, [P, i32, P]),
        "pkv_slot_mapping": (i32, [P, P, i32, P, i32, i32, i32, P, P]),
        "pkv_ring_slot_mapping": (i32, [P, P, i32, P, i32, i32, i32, i32, i32, P, P]),
        "pkv_kv_append": (i32, [P, P, P, i32, P, P, i32, i32, i32, i32, P]),
        "pkv_copy_blocks": (i32, [P, P, P, P, i32, i64, i32, i32, i32, i32, i32, P]),
        "pkv_decode_workspace_bytes": (sz, [i32, i32, i32, i32, i32]),
        "pkv_workspace_init": (i32, [P, sz, P]),
        "pkv_paged_attn_decode": (i32, [P, P, P, P, i32, P, i32, P, i32, i32, i32, i32, i32,
                                        i32, f32, P, sz, P]),
        "pkv_rope_table": (i32, [P, i32, i32, f64]),
        "pkv_ring_attn_decode": (i32, [P, P, P, P, i32, P, i32, P, P, i32, i32, i32, i32,
                                       i32, i32, i32, i32, P, f32, P, sz, P]),
        "pkv_check_tables": (i32, [P, P, i32, i32, i32, i32, P]),
        "pkv_check_slots": (i32, [P, i32, i32, i32, P]),
        "pkv_paged_attn_decode_noalloc": (i32, [P, P, P, P, i32, P, i32, P, i32, i32, i32,
                                                i32, i32, i32, f32, P]),
        "pkv_paged_attn_decode_append": (i32, [P, P, P, P, P, P, i32, P, i32, P, i32, i32,
                                               i32, i32, i32, i32, f32, P, sz, P]),
        "pkv_kv_append_fp8": (i32, [P, P, P, i32, P, P, i32, i32, i32, i32, P, P, P]),
        "pkv_paged_attn_decode_fp8": (i32, [P, P, P, P, P, P, i32, P, i32, P, i32, i32, i32,
                                            i32, i32, i32, f32, P, sz, P]),
        "pkv_paged_attn_decode_append_fp8": (i32, [P, P, P, P, P, P, P, P, i32, P, i32, P, i32,
                                                   i32, i32, i32, i32, i32, f32, P, sz, P]),
        "pkv_set_early_start": (i32, [i32]),
        "pkv_ring_attn_decode_append": (i32, [P, P, P, P, P, P, i32, P, i32, P, P, i32, i32, i32,
                                              i32, i32, i32, i32, i32, P, f32, P, sz, P]),
        "pkv_paged_prefill": (i32, [P, P, P, P, i32, P, i32, P, i32, i32, i32, i32, i32, i32, f32,
                                    P]),
        "pkv_pool_create": (i32, [i32, i32, i32, P]),
        "pkv_pool_destroy": (None, [P]),
        "pkv_pool_allocate": (i32, [P, P, i32, i32, P, i32, P, P]),
        "pkv_pool_warm": (i32, [P, P, i32]),
        "pkv_pool_release": (i32, [P, P, i32]),
        "pkv_pool_fork": (i32, [P, P, i32]),
        "pkv_pool_append": (i32, [P, P, P, i32, i32, i32, P, P, P, i32, P]),
        "pkv_pool_stats": (i32, [P, P, P, P, P, P]),
        "pkv_pool_refcount": (i32, [P, i32]),
        "pkv_spec_verify": (i32, [P, P, P, P, P, i32, i32, i32, P, P, P]),
        "pkv_kv_append_int4": (i32, [P, P, P, i32, P, P, i32, i32, i32, i32, P]),
        "pkv_widen_blocks_int4": (i32, [P, P, P, P, i32, i32, P, P, i32, i32, i32, i32, P]),
        "pkv_paged_attn_decode_int4": (i32, [P, P, P, P, i32, P, i32, P, i32, i32, i32, i32, i32,
                                             i32, f32, P, sz, P]),
        "pkv_paged_attn_decode_append_int4": (i32, [P, P, P, P, P, P, i32, P, i32, P, i32, i32,
                                                    i32, i32, i32, i32, f32, P, sz, P]),
        "pkv_qk_norm_rope": (i32, [P, P, P, P, i64, i64, P, P, f32, P, P, i32, i32, i32, i32, i32,
                                   P]),
        "pkv_extend_tables": (i32, [P, P, P, i32, i32, i32, P, P, i32, P, P, P, P, i32, P]),
        "pkv_truncate_tables": (i32, [P, P, P, i32, i32, i32, P, P, i32, P]),
        "pkv_kv_append_int8": (i32, [P, P, P, i32, P, P, P, P, i32, i32, i32, i32, P]),
        "pkv_widen_blocks_int8": (i32, [P, P, P, P, P, i32, i32, P, P, i32, i32, i32, i32, P]),
        "pkv_copy_blocks_int8": (i32, [P, P, P, P, P, P, i32, i32, i32, i32, i32, i32, P]),
        "pkv_paged_attn_decode_int8": (i32, [P, P, P, P, P, i32, P, i32, P, i32, i32, i32, i32, i32,
                                             i32, f32, P, sz, P]),
        "pkv_selected_attn_decode_int8": (i32, [P, P, P, P, P, i32, P, i32, P, i32, i32, i32, i32,
                                                i32, i32, f32, P, sz, P]),
        "pkv_select_blocks": (i32, [P, P, P, P, P, i32, P, i32, P, i32, i32, i32, i32, i32, i32, i32,
                                    i32, i32, P]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name, None)    # an older build may lack newer entry points
        if f is not None:
            f.restype, f.argtypes = res, args
    return lib


def _check(fn: str, status: int) -> None:
    if status != OK:
        raise PkvError(fn, status)


def _stream(stream=None):
    s = torch.cuda.current_stream() if stream is None else stream
    return ctypes.c_void_p(s.cuda_stream)


def _empty(n: int, dtype: torch.dtype, device, stream=None) -> torch.Tensor:
    """A call's output, allocated on the stream that the call runs on: memory freed on another one
    may still be in use there."""
    if stream is None:
        return torch.empty(n, dtype=dtype, device=device)
    if not isinstance(stream, torch.cuda.Stream):   # another library's, or a bare handle's holder
        handle = stream.cuda_stream
        stream = (torch.cuda.ExternalStream(handle, device=device) if handle > 1 else
                  torch.cuda.default_stream(device))
    with torch.cuda.stream(stream):
        return torch.empty(n, dtype=dtype, device=device)


def _p(t: torch.Tensor | None):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


# The 4-bit, 8-bit, norm and table calls go through a compiled binding: it checks what the library cannot
# see through a bare pointer (element type, device, layout, shape), allocates the outputs and
# makes the call. Their kernels are shorter than the same steps in Python.
_TORCH_ENTRIES = ("kv_append_int4", "widen_blocks_int4", "paged_attn_decode_int4",
                  "paged_attn_decode_append_int4", "qk_norm_rope", "extend_tables",
                  "truncate_tables", "kv_append_int8", "widen_blocks_int8", "copy_blocks_int8",
                  "paged_attn_decode_int8", "selected_attn_decode_int8", "select_blocks")
_ops = None


def _torch_ops():
    """The compiled binding (built with the library), bound to the loaded library."""
    global _ops
    lib = load()
    try:
        from . import _pkv_torch
    except ImportError as e:
        raise RuntimeError("_pkv_torch.so is missing or does not fit the installed torch: build it "
                           "with `python -m paged_kv_cache_147_gb300.build`") from e
    _pkv_torch.bind(PkvError, *(ctypes.cast(getattr(lib, "pkv_" + n), ctypes.c_void_p).value
                                for n in _TORCH_ENTRIES))
    _ops = _pkv_torch
    return _ops


def version() -> int:
    return load().pkv_version()


def device_error(clear: bool = True, stream=None) -> int:
    out = ctypes.c_uint(0)
    _check("pkv_device_error", load().pkv_device_error(ctypes.byref(out), int(clear),
                                                        _stream(stream)))
    return out.value


# ------------------------------------------------------------------------------ slot mapping
def slot_mapping(seq_ids, positions, block_tables, block_size, out=None, stream=None):
    n = positions.numel()
    out = _empty(n, torch.int64, positions.device, stream) if out is None else out
    _check("pkv_slot_mapping", load().pkv_slot_mapping(
        _p(seq_ids), _p(positions), n, _p(block_tables), block_tables.shape[0],
        block_tables.shape[1], block_size, _p(out), _stream(stream)))
    return out


def ring_slot_mapping(seq_ids, positions, block_tables, sink, window, block_size, out=None,
                      stream=None):
    n = positions.numel()
    out = _empty(n, torch.int64, positions.device, stream) if out is None else out
    _check("pkv_ring_slot_mapping", load().pkv_ring_slot_mapping(
        _p(seq_ids), _p(positions), n, _p(block_tables), block_tables.shape[0],
        block_tables.shape[1], sink, window, block_size, _p(out), _stream(stream)))
    return out


# ------------------------------------------------------------------------------ cache edits
def kv_append(k, v, slots, k_cache, v_cache, stream=None):
    """k, v [T, Hkv, D]; k_cache, v_cache one layer [NB, Hkv, bs, D]."""
    nb, hkv, bs, d = k_cache.shape
    _check("pkv_kv_append", load().pkv_kv_append(
        _p(k), _p(v), _p(slots), slots.numel(), _p(k_cache), _p(v_cache), nb, hkv, d, bs,
        _stream(stream)))


def kv_append_fp8(k, v, slots, k_cache, v_cache, k_scale, v_scale, stream=None):
    """k, v fp16 [T, Hkv, D]; k_cache, v_cache one layer of uint8 E4M3 codes [NB, Hkv, bs, D];
    k_scale, v_scale float32 [Hkv] on the device."""
    nb, hkv, bs, d = k_cache.shape
    _check("pkv_kv_append_fp8", load().pkv_kv_append_fp8(
        _p(k), _p(v), _p(slots), slots.numel(), _p(k_cache), _p(v_cache), nb, hkv, d, bs,
        _p(k_scale), _p(v_scale), _stream(stream)))


def copy_blocks(k_cache, v_cache, src, dst, stream=None):
    """k_cache, v_cache [layers, NB, Hkv, bs, D] (or one layer [NB, Hkv, bs, D]) of any cache type:
    fp16 rows, uint8 E4M3 codes or uint8 4-bit rows (D = 80); copy_blocks_int8 copies those of an
    8-bit cache, whose scales go with them."""
    kc = k_cache if k_cache.dim() == 5 else k_cache.unsqueeze(0)
    layers, nb, hkv, bs, d = kc.shape
    row, layer = d * kc.element_size(), kc.stride(0) * kc.element_size()   # bytes
    if row % 2 or layer % 2 or v_cache.shape != k_cache.shape or v_cache.dtype != k_cache.dtype:
        raise PkvError("pkv_copy_blocks", EINVAL)
    # the library counts in fp16 elements
    _check("pkv_copy_blocks", load().pkv_copy_blocks(
        _p(k_cache), _p(v_cache), _p(src), _p(dst), src.numel(), layer // 2, layers, nb, hkv,
        row // 2, bs, _stream(stream)))


# ------------------------------------------------------------------------------ attention
def set_early_start(enable: bool) -> bool:
    """Lets the fused-append calls start while the previous kernel finishes (True, the
    default) or not; returns the previous setting. Process-wide."""
    return bool(load().pkv_set_early_start(1 if enable else 0))


def decode_workspace_bytes(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim=128) -> int:
    n = load().pkv_decode_workspace_bytes(num_seqs, q_len, num_q_heads, num_kv_heads, head_dim)
    if n == 0:
        raise PkvError("pkv_decode_workspace_bytes", EINVAL)
    return int(n)


def workspace_init(workspace, stream=None):
    _check("pkv_workspace_init", load().pkv_workspace_init(
        _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))


def make_workspace(num_seqs, q_len, num_q_heads, num_kv_heads, device="cuda", stream=None):
    """Allocates (through torch) and zeroes a decode workspace."""
    ws = _empty(decode_workspace_bytes(num_seqs, q_len, num_q_heads, num_kv_heads), torch.uint8,
                device, stream)
    workspace_init(ws, stream)
    return ws


def paged_attn_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale, workspace,
                      stream=None):
    """q, out [B, q_len, Hq, D]; k_cache, v_cache one layer [NB, Hkv, bs, D]."""
    B, q_len, hq, d = q.shape
    nb, hkv, bs, _ = k_cache.shape
    _check("pkv_paged_attn_decode", load().pkv_paged_attn_decode(
        _p(out), _p(q), _p(k_cache), _p(v_cache), nb, _p(block_tables), block_tables.shape[1],
        _p(context_lens), B, q_len, hq, hkv, d, bs, float(scale), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def paged_attn_decode_fp8(out, q, k_cache, v_cache, k_scale, v_scale, block_tables, context_lens,
                          scale, workspace, stream=None):
    """paged_attn_decode over an E4M3 cache: uint8 pools [NB, Hkv, bs, D], float32 per-kv-head
    scales [Hkv] (element value = code * scale)."""
    B, q_len, hq, d = q.shape
    nb, hkv, bs, _ = k_cache.shape
    _check("pkv_paged_attn_decode_fp8", load().pkv_paged_attn_decode_fp8(
        _p(out), _p(q), _p(k_cache), _p(v_cache), _p(k_scale), _p(v_scale), nb,
        _p(block_tables), block_tables.shape[1], _p(context_lens), B, q_len, hq, hkv, d, bs,
        float(scale), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return out


def paged_attn_decode_append_fp8(out, q, k_new, v_new, k_cache, v_cache, k_scale, v_scale,
                                 block_tables, context_lens, scale, workspace, stream=None):
    """paged_attn_decode_append over an E4M3 cache: the new fp16 rows are stored as
    kv_append_fp8 stores them and attended over with the rest of the cache."""
    B, q_len, hq, d = q.shape
    nb, hkv, bs, _ = k_cache.shape
    _check("pkv_paged_attn_decode_append_fp8", load().pkv_paged_attn_decode_append_fp8(
        _p(out), _p(q), _p(k_new), _p(v_new), _p(k_cache), _p(v_cache), _p(k_scale),
        _p(v_scale), nb, _p(block_tables), block_tables.shape[1], _p(context_lens), B, q_len, hq,
        hkv, d, bs, float(scale), _p(workspace), workspace.numel() * workspace.element_size(),
        _stream(stream)))
    return out


def paged_attn_decode_append(out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens,
                             scale, workspace, stream=None):
    """Decode step with the KV append fused in: k_new, v_new [B*q_len, Hkv, D] go to the slots of
    positions context_lens[b] - q_len + i, then attention runs over the cache including them.

    WARNING: by default this launch may start before the kernel ahead of it on the stream has
    finished, and it reads the K/V pools, block_tables and context_lens early. If the kernel
    right before it writes any of those (a torch op that advances context_lens, copy_blocks,
    ...), put another launch or a copy in between, or call set_early_start(False) first."""
    B, q_len, hq, d = q.shape
    nb, hkv, bs, _ = k_cache.shape
    _check("pkv_paged_attn_decode_append", load().pkv_paged_attn_decode_append(
        _p(out), _p(q), _p(k_new), _p(v_new), _p(k_cache), _p(v_cache), nb, _p(block_tables),
        block_tables.shape[1], _p(context_lens), B, q_len, hq, hkv, d, bs, float(scale),
        _p(workspace), workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def paged_prefill(out, q, k_cache, v_cache, block_tables, context_lens, scale, stream=None):
    """Chunked-prefill attention: q, out [B, q_len, Hq, D]; the chunk's K/V rows are already in
    the one-layer caches [NB, Hkv, bs, D]; query i of sequence b attends causally up to position
    context_lens[b] - q_len + i."""
    B, q_len, hq, d = q.shape
    nb, hkv, bs, _ = k_cache.shape
    _check("pkv_paged_prefill", load().pkv_paged_prefill(
        _p(out), _p(q), _p(k_cache), _p(v_cache), nb, _p(block_tables), block_tables.shape[1],
        _p(context_lens), B, q_len, hq, hkv, d, bs, float(scale), _stream(stream)))
    return out


def paged_attn_decode_noalloc(out, q, k_cache, v_cache, block_tables, context_lens, scale,
                              stream=None):
    """paged_attn_decode for callers that cannot allocate device memory: the library's fixed
    8 MiB scratch array replaces the workspace. Calls sharing it must not overlap on the GPU;
    the first call on a device must come before any stream capture."""
    B, q_len, hq, d = q.shape
    nb, hkv, bs, _ = k_cache.shape
    _check("pkv_paged_attn_decode_noalloc", load().pkv_paged_attn_decode_noalloc(
        _p(out), _p(q), _p(k_cache), _p(v_cache), nb, _p(block_tables), block_tables.shape[1],
        _p(context_lens), B, q_len, hq, hkv, d, bs, float(scale), _stream(stream)))
    return out


def rope_table(n_index, head_dim=128, base=10000.0) -> torch.Tensor:
    """Host float32 [n_index, head_dim/2, 2] (cos, sin) table; move it to the device."""
    t = torch.empty((n_index, head_dim // 2, 2), dtype=torch.float32)
    _check("pkv_rope_table", load().pkv_rope_table(_p(t), n_index, head_dim, float(base)))
    return t


def ring_attn_decode(out, q, k_cache, v_cache, block_tables, logical_len, high_water, sink,
                     window, rope_cos_sin, scale, workspace, stream=None):
    B, q_len, hq, d = q.shape
    nb, hkv, bs, _ = k_cache.shape
    _check("pkv_ring_attn_decode", load().pkv_ring_attn_decode(
        _p(out), _p(q), _p(k_cache), _p(v_cache), nb, _p(block_tables), block_tables.shape[1],
        _p(logical_len), _p(high_water), B, q_len, hq, hkv, d, bs, sink, window,
        _p(rope_cos_sin), float(scale), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


def ring_attn_decode_append(out, q, k_new, v_new, k_cache, v_cache, block_tables, logical_len,
                            high_water, sink, window, rope_cos_sin, scale, workspace,
                            stream=None):
    """Sink + ring decode step with the append fused in: k_new, v_new [B*q_len, Hkv, D] (before
    RoPE) go to the ring slots of positions logical_len[b] - q_len + i, then ring attention runs
    over the cache including them. Early-start caveat as for paged_attn_decode_append."""
    B, q_len, hq, d = q.shape
    nb, hkv, bs, _ = k_cache.shape
    _check("pkv_ring_attn_decode_append", load().pkv_ring_attn_decode_append(
        _p(out), _p(q), _p(k_new), _p(v_new), _p(k_cache), _p(v_cache), nb, _p(block_tables),
        block_tables.shape[1], _p(logical_len), _p(high_water), B, q_len, hq, hkv, d, bs, sink,
        window, _p(rope_cos_sin), float(scale), _p(workspace),
        workspace.numel() * workspace.element_size(), _stream(stream)))
    return out


# ------------------------------------------------------------------------------ 4-bit cache
INT4_ROW = 80   # bytes of one row (token, kv head) of a 4-bit pool


def kv_append_int4(k, v, slots, k_cache, v_cache, stream=None):
    """k, v fp16 [T, Hkv, 128]; slots int64 [T]; k_cache, v_cache one layer of uint8 4-bit rows
    [NB, Hkv, bs, 80]."""
    (_ops or _torch_ops()).kv_append_int4(k, v, slots, k_cache, v_cache, stream)


def widen_blocks_int4(k_cache, v_cache, src, dst, k_out, v_out, stream=None):
    """Blocks src[i] of the 4-bit pools [NB, Hkv, bs, 80] -> blocks dst[i] of the fp16 pools k_out,
    v_out [NB', Hkv, bs, 128]; src, dst int32."""
    (_ops or _torch_ops()).widen_blocks_int4(k_cache, v_cache, src, dst, k_out, v_out, stream)


def paged_attn_decode_int4(out, q, k_cache, v_cache, block_tables, context_lens, scale, workspace,
                           stream=None):
    """paged_attn_decode over a 4-bit cache: uint8 pools [NB, Hkv, bs, 80] (kv_append_int4's
    rows); everything else as there."""
    return (_ops or _torch_ops()).paged_attn_decode_int4(
        out, q, k_cache, v_cache, block_tables, context_lens, scale, workspace, stream)


def paged_attn_decode_append_int4(out, q, k_new, v_new, k_cache, v_cache, block_tables,
                                  context_lens, scale, workspace, stream=None):
    """paged_attn_decode_append over a 4-bit cache: the new fp16 rows k_new, v_new
    [B*q_len, Hkv, 128] are stored as kv_append_int4 stores them and attended over with the rest.
    Early-start caveat as there.

    WARNING: the last q_len positions of every context are written. A sequence without q_len new
    tokens (refused by extend_tables, or idle) needs a length of 0 in context_lens here: zeros come
    out and its rows stay. kv_append_int4 + paged_attn_decode_int4 go by the slots instead."""
    return (_ops or _torch_ops()).paged_attn_decode_append_int4(
        out, q, k_new, v_new, k_cache, v_cache, block_tables, context_lens, scale, workspace, stream)


# ------------------------------------------------------------------------------ 8-bit cache
def make_int8_cache(num_blocks, num_kv_heads, block_size, layers=None, bounds=True, device="cuda"):
    """A zeroed 8-bit cache: (k_cache, v_cache uint8 [NB, Hkv, bs, 128], kv_scales float32
    [NB, Hkv, 2], k_bounds uint8 [NB, Hkv, 2, 128] or None), with a leading dimension where `layers`
    is given. k_bounds are for select_blocks."""
    lead = () if layers is None else (layers,)

    def zeros(*shape, dtype=torch.uint8):
        return torch.zeros(*lead, num_blocks, num_kv_heads, *shape, dtype=dtype, device=device)

    return (zeros(block_size, 128), zeros(block_size, 128), zeros(2, dtype=torch.float32),
            zeros(2, 128) if bounds else None)


def kv_append_int8(k, v, slots, k_cache, v_cache, kv_scales, k_bounds=None, stream=None):
    """k, v fp16 [T, Hkv, 128]; slots int64 [T]; one layer of an 8-bit cache (make_int8_cache).
    A block's scale grows with the rows written into it; writing its first row starts it afresh,
    its other rows zero. The tokens of one block lie within block_size consecutive ones of the call."""
    (_ops or _torch_ops()).kv_append_int8(k, v, slots, k_cache, v_cache, kv_scales, k_bounds, stream)


def widen_blocks_int8(k_cache, v_cache, kv_scales, src, dst, k_out, v_out, stream=None):
    """Blocks src[i] of the 8-bit cache -> blocks dst[i] of the fp16 pools k_out, v_out
    [NB', Hkv, bs, 128]; src, dst int32."""
    (_ops or _torch_ops()).widen_blocks_int8(k_cache, v_cache, kv_scales, src, dst, k_out, v_out,
                                             stream)


def copy_blocks_int8(k_cache, v_cache, kv_scales, k_bounds, src, dst, stream=None):
    """copy_blocks for an 8-bit cache (one layer, or layers in a leading dimension): codes, scales
    and, unless None, bounds."""
    (_ops or _torch_ops()).copy_blocks_int8(k_cache, v_cache, kv_scales, k_bounds, src, dst, stream)


def paged_attn_decode_int8(out, q, k_cache, v_cache, kv_scales, block_tables, context_lens, scale,
                           workspace, stream=None):
    """paged_attn_decode over an 8-bit cache (make_int8_cache's pools and scales). block_tables
    [B, width], or [B, Hkv, width]: a table per kv head, with context_lens the tokens in it
    (select_blocks' two results)."""
    return (_ops or _torch_ops()).paged_attn_decode_int8(
        out, q, k_cache, v_cache, kv_scales, block_tables, context_lens, scale, workspace, stream)


def select_blocks(q, kv_scales, k_bounds, block_tables, context_lens, block_size, budget,
                  keep_first=1, keep_last=1, tables_out=None, lens_out=None, stream=None):
    """Blocks of each sequence that the queries q [B, q_len, Hq, 128] attend to, up to `budget` per kv
    head: the first keep_first, the last keep_last (and those of the last q_len tokens), and those
    whose keys may have the largest products with a query -> (tables int32 [B, Hkv, budget], -1
    behind the chosen blocks; lens int32 [B], the tokens in them), for paged_attn_decode_int8."""
    return (_ops or _torch_ops()).select_blocks(
        q, kv_scales, k_bounds, block_tables, context_lens, block_size, budget, keep_first,
        keep_last, tables_out, lens_out, stream)


# ------------------------------------------------------------------------------ norm + rotation
def qk_norm_rope(q, k, q_weight, k_weight, eps, positions, cos_sin, q_out=None, k_out=None,
                 stream=None):
    """Per-head RMS norm and rotation: q fp16 [T, Hq, 128], k fp16 [T, Hkv, 128] (each token's
    heads contiguous, tokens a stride of at least that apart, a multiple of 4: slices of a packed
    projection do), weights fp16 [128], positions int64 [T] (negative: padding, left as it is),
    cos_sin a rope_table on the device -> (q_out, k_out), contiguous."""
    return (_ops or _torch_ops()).qk_norm_rope(
        q, k, q_weight, k_weight, eps, positions, cos_sin, q_out, k_out, stream)


# ------------------------------------------------------------------------------ tables on the GPU
def extend_tables(block_tables, context_lens, new_lens, block_size, free_blocks, free_count,
                  max_tokens, out=None, stream=None):
    """Grows the tables (int32 [B, max_blocks]) and lengths (int32 [B]) for new_lens more tokens
    per sequence, blocks off the stack free_blocks (int32 [num_blocks], free_count of them free;
    all updated in place) -> (slots int64, seq_ids int32, positions int64 [max_tokens],
    cu_new_lens int32 [B + 1]); `out` gives the four to write into. A sequence that cannot be served
    keeps its table and length, and its tokens get -1: a fused append + decode behind this call
    needs a length of 0 for it (and a launch in between, see paged_attn_decode_append)."""
    return (_ops or _torch_ops()).extend_tables(
        block_tables, context_lens, new_lens, block_size, free_blocks, free_count, max_tokens,
        out if out is None else tuple(out), stream)


def truncate_tables(block_tables, context_lens, keep_lens, block_size, free_blocks, free_count,
                    stream=None):
    """Cuts sequences back to keep_lens tokens (int32 [B]; negative or past the length: as it is);
    their blocks go back on the stack. All updated in place."""
    (_ops or _torch_ops()).truncate_tables(
        block_tables, context_lens, keep_lens, block_size, free_blocks, free_count, stream)


# ------------------------------------------------------------------------------ host checks
def check_tables(block_tables, context_lens, block_size, num_blocks) -> int | None:
    """Host validation; returns None if valid, else the first bad sequence index."""
    bt = block_tables.detach().to("cpu", torch.int32).contiguous()
    cl = context_lens.detach().to("cpu", torch.int32).contiguous()
    bad = ctypes.c_int(-1)
    st = load().pkv_check_tables(_p(bt), _p(cl), bt.shape[0], bt.shape[1], block_size,
                                 num_blocks, ctypes.byref(bad))
    if st == ERANGE:
        return bad.value
    _check("pkv_check_tables", st)
    return None


def check_slots(slots, num_blocks, block_size) -> int | None:
    s = slots.detach().to("cpu", torch.int64).contiguous()
    bad = ctypes.c_int(-1)
    st = load().pkv_check_slots(_p(s), s.numel(), num_blocks, block_size, ctypes.byref(bad))
    if st == ERANGE:
        return bad.value
    _check("pkv_check_slots", st)
    return None


# ------------------------------------------------------------------------------ speculative verify
def spec_verify(target_logits, draft_logits, drafts, u_accept, u_sample, n_accept=None,
                next_token=None, stream=None):
    """target [B, K+1, V], draft [B, K, V] float32; drafts int32 [B, K]; u_accept [B, K],
    u_sample [B] float32 -> (n_accept, next_token) int32 [B] (device tensors)."""
    B, K1, V = target_logits.shape
    if n_accept is None:
        n_accept = _empty(B, torch.int32, target_logits.device, stream)
    if next_token is None:
        next_token = _empty(B, torch.int32, target_logits.device, stream)
    _check("pkv_spec_verify", load().pkv_spec_verify(
        _p(target_logits), _p(draft_logits), _p(drafts), _p(u_accept), _p(u_sample), B, K1 - 1,
        V, _p(n_accept), _p(next_token), _stream(stream)))
    return n_accept, next_token


# ------------------------------------------------------------------------------ host block pool
class BlockPool:
    """The library's host block pool (pkv_pool_*): block tables with prefix sharing, reference
    counts and copy-on-write pairs for pkv_copy_blocks. Tables are int32 numpy arrays."""

    def __init__(self, num_blocks: int, block_size: int, hash_bits: int = 64):
        self._lib = load()
        h = ctypes.c_void_p()
        _check("pkv_pool_create", self._lib.pkv_pool_create(num_blocks, block_size, hash_bits,
                                                             ctypes.byref(h)))
        self._h, self.num_blocks, self.block_size = h, num_blocks, block_size

    def close(self):
        if self._h:
            self._lib.pkv_pool_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    @staticmethod
    def _i32(a):
        return np.ascontiguousarray(np.asarray(a, dtype=np.int32))

    def allocate(self, tokens, max_tokens=None, table_cap=None):
        """-> (table, reused): the sequence's blocks and how many were shared."""
        t = self._i32(tokens)
        mt = len(t) if max_tokens is None else int(max_tokens)
        cap = table_cap or (max(mt, len(t)) // self.block_size + 2)
        table = np.empty(cap, np.int32)
        n, reused = ctypes.c_int(0), ctypes.c_int(0)
        _check("pkv_pool_allocate", self._lib.pkv_pool_allocate(
            self._h, t.ctypes.data, len(t), mt, table.ctypes.data, cap, ctypes.byref(n),
            ctypes.byref(reused)))
        return table[:n.value].copy(), reused.value

    def warm(self, tokens):
        t = self._i32(tokens)
        _check("pkv_pool_warm", self._lib.pkv_pool_warm(self._h, t.ctypes.data, len(t)))

    def release(self, table):
        t = self._i32(table)
        _check("pkv_pool_release", self._lib.pkv_pool_release(self._h, t.ctypes.data, len(t)))

    def fork(self, table):
        t = self._i32(table)
        _check("pkv_pool_fork", self._lib.pkv_pool_fork(self._h, t.ctypes.data, len(t)))
        return t.copy()

    def append(self, table, length, n_new, all_tokens=None):
        """-> (table, copies): copies is an int32 [n, 2] array of (src, dst) block pairs."""
        cap = (length + n_new) // self.block_size + 2
        t = np.empty(max(cap, len(table)), np.int32)
        t[:len(table)] = table
        n = ctypes.c_int(len(table))
        src, dst = np.empty(cap, np.int32), np.empty(cap, np.int32)
        nc = ctypes.c_int(0)
        at = None if all_tokens is None else self._i32(all_tokens)
        _check("pkv_pool_append", self._lib.pkv_pool_append(
            self._h, t.ctypes.data, ctypes.byref(n), len(t), int(length), int(n_new),
            None if at is None else at.ctypes.data, src.ctypes.data, dst.ctypes.data, cap,
            ctypes.byref(nc)))
        return t[:n.value].copy(), np.stack([src[:nc.value], dst[:nc.value]], axis=1)

    def stats(self) -> dict:
        v = [ctypes.c_int(0) for _ in range(5)]
        _check("pkv_pool_stats", self._lib.pkv_pool_stats(self._h, *[ctypes.byref(x) for x in v]))
        return dict(zip(("total", "used", "shared", "free", "warm"), (x.value for x in v)))

    def refcount(self, block: int) -> int:
        r = self._lib.pkv_pool_refcount(self._h, int(block))
        if r < 0:
            raise PkvError("pkv_pool_refcount", r)
        return r
