"""ctypes binding of libpagedkv.so (the C ABI in include/pagedkv.h).

Argument marshalling only: every function checks that the torch tensors it
is given have the dtype, device, shape and contiguity the C ABI documents,
then passes their device pointers, sizes and the current CUDA stream to the
entry point of the same name.  All computation happens in the library's CUDA
kernels; there is no fallback of any kind.  If the library is missing, the
first call raises ``RuntimeError`` (build it with ``__graft_entry__.build()``
or ``python -m paged_kv_cache_95_gb300.build``).
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import Optional

PKV_DTYPE_BF16 = 0
PKV_DTYPE_FLOAT32 = 1
PKV_DTYPE_FP8_E4M3 = 2

PKV_OK = 0
PKV_ERR_INVALID_ARG = -1
PKV_ERR_UNSUPPORTED = -2
PKV_ERR_WORKSPACE_TOO_SMALL = -3
PKV_ERR_CUDA = -4
PKV_ERR_OUT_OF_BLOCKS = -5

PKV_STATUS_BAD_CONTEXT_LEN = 0x1
PKV_STATUS_BAD_BLOCK_ID = 0x2
PKV_STATUS_BAD_Q_LEN = 0x4
PKV_STATUS_TIMEOUT = 0x8

PKV_VERIFY_AUTO = -1
PKV_VERIFY_DECODE_KERNEL = 0
PKV_VERIFY_PREFILL_KERNEL = 1

HEAD_DIM = 128
BLOCK_SIZE = 16
LATENT_DIM = 512  # latent attention: values of the shared latent a token
ROPE_DIM = 64     # and of its rotated key
STATIC_SCRATCH_BYTES = 16 * 1024 * 1024  # PKV_STATIC_SCRATCH_BYTES

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libpagedkv.so")
HEADER_PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "pagedkv.h")

_lock = threading.Lock()
_lib = None


class CacheDesc(ctypes.Structure):
    """Mirror of ``pkv_cache_desc``."""

    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32),
                ("num_kv_heads", ctypes.c_int32), ("head_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class LatentDesc(ctypes.Structure):
    """Mirror of ``pkv_latent_desc``."""

    _fields_ = [("num_blocks", ctypes.c_int32), ("block_size", ctypes.c_int32), ("latent_dim", ctypes.c_int32),
                ("rope_dim", ctypes.c_int32), ("dtype", ctypes.c_int32)]


class PagedKVError(RuntimeError):
    def __init__(self, fn: str, code: int):
        self.code = code
        super().__init__(f"{fn} failed: {status_string(code)} ({code})")


def load_library(path: Optional[str] = None) -> ctypes.CDLL:
    """Load libpagedkv.so and declare the C signatures."""
    global _lib
    if path is None:
        with _lock:
            if _lib is None:
                if not os.path.exists(LIB_PATH):
                    raise RuntimeError(f"{LIB_PATH} is missing: build the CUDA library first "
                                       "(python -c 'import __graft_entry__ as g; g.build()')")
                _lib = _declare(ctypes.CDLL(LIB_PATH))
            return _lib
    return _declare(ctypes.CDLL(path))


def _declare(lib):
    P, i32, f32, sz = ctypes.c_void_p, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t
    D = ctypes.POINTER(CacheDesc)
    lib.kv_reshape_and_cache.argtypes = [P, P, P, P, P, i32, D, P]
    lib.kv_reshape_and_cache.restype = ctypes.c_int
    lib.paged_attention_workspace_size.argtypes = [i32, i32, i32, i32, D]
    lib.paged_attention_workspace_size.restype = sz
    lib.paged_attention_decode_partitions.argtypes = [i32, i32, i32, i32, i32, D]
    lib.paged_attention_decode_partitions.restype = i32
    lib.paged_attention_decode.argtypes = [P, i32, P, P, P, P, P, i32, i32, i32, f32, i32, D, P, sz, P]
    lib.paged_attention_decode.restype = ctypes.c_int
    lib.paged_attention_decode_append.argtypes = [P, i32, P, P, P, P, P, P, P, i32, i32, i32, f32, i32, D, P, sz, P]
    lib.paged_attention_decode_append.restype = ctypes.c_int
    lib.paged_attention_decode_window.argtypes = [P, i32, P, P, P, P, P, i32, i32, i32, f32, i32, i32, D, P, sz, P]
    lib.paged_attention_decode_window.restype = ctypes.c_int
    lib.paged_attention_decode_fp8.argtypes = [P, i32, P, P, P, P, P, P, P, i32, i32, i32, f32, i32, i32, D, P, sz, P]
    lib.paged_attention_decode_fp8.restype = ctypes.c_int
    lib.paged_attention_verify_workspace_size.argtypes = [i32, i32, i32, i32, i32, D]
    lib.paged_attention_verify_workspace_size.restype = sz
    lib.paged_attention_verify.argtypes = [P, i32, P, i32, P, P, P, P, i32, i32, i32, f32, i32, D, P, sz, P]
    lib.paged_attention_verify.restype = ctypes.c_int
    lib.paged_attention_verify_window.argtypes = [P, i32, P, i32, P, P, P, P, i32, i32, i32, f32, i32, i32, D, P, sz,
                                                  P]
    lib.paged_attention_verify_window.restype = ctypes.c_int
    lib.paged_attention_verify_fp8.argtypes = [P, i32, P, i32, P, P, P, P, P, P, i32, i32, i32, f32, i32, i32, D, P,
                                               sz, P]
    lib.paged_attention_verify_fp8.restype = ctypes.c_int
    lib.paged_attention_verify_workspace_size_on.argtypes = [i32, i32, i32, i32, i32, i32, D]
    lib.paged_attention_verify_workspace_size_on.restype = sz
    lib.paged_attention_verify_on.argtypes = [i32, P, i32, P, i32, P, P, P, P, P, P, i32, i32, i32, f32, i32, i32, D,
                                              P, sz, P]
    lib.paged_attention_verify_on.restype = ctypes.c_int
    lib.kv_reshape_and_cache_fp8.argtypes = [P, P, P, P, P, P, P, i32, D, P]
    lib.kv_reshape_and_cache_fp8.restype = ctypes.c_int
    lib.paged_attention_prefill_workspace_size.argtypes = [i32, i32, D]
    lib.paged_attention_prefill_workspace_size.restype = sz
    lib.paged_attention_verify_on_prefill.argtypes = [i32, i32, i32, D]
    lib.paged_attention_verify_on_prefill.restype = ctypes.c_int
    lib.paged_attention_prefill_chunk_workspace_size.argtypes = [i32, i32, i32, i32, i32, D]
    lib.paged_attention_prefill_chunk_workspace_size.restype = sz
    lib.paged_attention_prefill_chunk.argtypes = [P, i32, P, P, i32, i32, P, P, P, P, i32, i32, i32, f32, D, P, sz, P]
    lib.paged_attention_prefill_chunk.restype = ctypes.c_int
    lib.paged_attention_prefill_chunk_window.argtypes = [P, i32, P, P, i32, i32, P, P, P, P, i32, i32, i32, f32, i32,
                                                         D, P, sz, P]
    lib.paged_attention_prefill_chunk_window.restype = ctypes.c_int
    lib.paged_attention_prefill_chunk_fp8.argtypes = [P, i32, P, P, i32, i32, P, P, P, P, P, P, i32, i32, i32, f32,
                                                      i32, D, P, sz, P]
    lib.paged_attention_prefill_chunk_fp8.restype = ctypes.c_int
    lib.paged_attention_decode_static_scratch.argtypes = [P, i32, P, P, P, P, P, i32, i32, i32, f32, i32, D, P, P]
    lib.paged_attention_decode_static_scratch.restype = ctypes.c_int
    lib.kv_copy_blocks.argtypes = [P, P, P, P, P, i32, D, P]
    lib.kv_copy_blocks.restype = ctypes.c_int
    i64, I = ctypes.c_int64, ctypes.c_int
    LD = ctypes.POINTER(LatentDesc)
    lib.latent_reshape_and_cache.argtypes = [P, i64, P, i64, P, P, i32, LD, P]
    lib.latent_reshape_and_cache.restype = I
    lib.latent_reshape_and_cache_fp8.argtypes = [P, i64, P, i64, P, P, P, P, i32, LD, P]
    lib.latent_reshape_and_cache_fp8.restype = I
    lib.latent_gather.argtypes = [P, P, P, P, P, P, i32, i32, i32, LD, P, P]
    lib.latent_gather.restype = I
    lib.latent_attention_workspace_size.argtypes = [i32, i32, i32, i32, LD]
    lib.latent_attention_workspace_size.restype = sz
    lib.latent_attention_decode.argtypes = [P, i32, P, i64, i64, P, i64, i64, P, P, P, i32, i32, i32, i32, f32, LD, P,
                                            sz, P]
    lib.latent_attention_decode.restype = I
    lib.latent_attention_decode_fp8.argtypes = [P, i32, P, i64, i64, P, i64, i64, P, P, P, P, P, i32, i32, i32, i32,
                                                f32, LD, P, sz, P]
    lib.latent_attention_decode_fp8.restype = I
    lib.latent_attention_prefill_workspace_size.argtypes = [i32, i32, i32, i32, i32]
    lib.latent_attention_prefill_workspace_size.restype = sz
    lib.latent_attention_prefill_chunk.argtypes = [P, i32, P, i64, i64, P, P, i64, i64, P, i64, P, P, i32, i32, i32,
                                                   i32, i32, f32, P, sz, P]
    lib.latent_attention_prefill_chunk.restype = I
    lib.pkv_bm_create.argtypes = [i32, ctypes.POINTER(P)]
    lib.pkv_bm_create.restype = I
    lib.pkv_bm_destroy.argtypes = [P]
    lib.pkv_bm_destroy.restype = None
    lib.pkv_bm_num_free.argtypes = [P]
    lib.pkv_bm_num_free.restype = i32
    lib.pkv_bm_ref_count.argtypes = [P, i32, P]
    lib.pkv_bm_ref_count.restype = I
    lib.pkv_bm_add_sequence.argtypes = [P, i64]
    lib.pkv_bm_add_sequence.restype = I
    lib.pkv_bm_fork.argtypes = [P, i64, i64]
    lib.pkv_bm_fork.restype = I
    lib.pkv_bm_append.argtypes = [P, i64, i32, P, P, P]
    lib.pkv_bm_append.restype = I
    lib.pkv_bm_append_batch.argtypes = [P, P, i32, P, P, P, P]
    lib.pkv_bm_append_batch.restype = I
    lib.pkv_bm_free_sequence.argtypes = [P, i64]
    lib.pkv_bm_free_sequence.restype = I
    lib.pkv_bm_sequence_length.argtypes = [P, i64, P]
    lib.pkv_bm_sequence_length.restype = I
    lib.pkv_bm_block_tables.argtypes = [P, P, i32, i32, i32, P, P]
    lib.pkv_bm_block_tables.restype = I
    lib.pkv_bm_publish.argtypes = [P, i64, P, i32]
    lib.pkv_bm_publish.restype = I
    lib.pkv_bm_add_sequence_cached.argtypes = [P, i64, P, i32, P]
    lib.pkv_bm_add_sequence_cached.restype = I
    lib.pagedkv_status_string.argtypes = [ctypes.c_int]
    lib.pagedkv_status_string.restype = ctypes.c_char_p
    lib.pagedkv_version.argtypes = []
    lib.pagedkv_version.restype = ctypes.c_int
    return lib


def status_string(code: int) -> str:
    try:
        return load_library().pagedkv_status_string(int(code)).decode()
    except RuntimeError:
        return f"status {code}"


def version() -> int:
    return int(load_library().pagedkv_version())


# ---- tensor marshalling ----------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t) -> int:
    return int(t.data_ptr())


def _stream(stream) -> int:
    torch = _torch()
    if stream is None:
        return int(torch.cuda.current_stream().cuda_stream)
    return int(stream.cuda_stream if hasattr(stream, "cuda_stream") else stream)


def _need(cond: bool, msg: str):
    if not cond:
        raise ValueError(msg)


def _new_workspace(nbytes, what, like, stream, clear=None):
    """Device scratch whose first ``clear`` bytes are zero (None: all), allocated and cleared on the call's stream (its
    handle): on another one the clear could come behind the kernel, and the memory still be in use."""
    torch = _torch()
    _need(nbytes > 0, f"invalid sizes for {what}")

    def new():
        workspace = torch.empty(nbytes, dtype=torch.uint8, device=like.device)
        (workspace if clear is None else workspace[:clear]).zero_()
        return workspace

    if stream == torch.cuda.current_stream(like.device).cuda_stream:
        return new()
    # (A handle of 0 is the default stream, which ExternalStream would take for a new one.)
    with torch.cuda.stream(torch.cuda.ExternalStream(stream, like.device) if stream else torch.cuda.default_stream(like.device)):
        return new()


def _check(t, name, dtype, ndim=None, last=None):
    torch = _torch()
    _need(isinstance(t, torch.Tensor), f"{name} must be a torch.Tensor")
    _need(t.is_cuda, f"{name} must be a CUDA tensor")
    _need(t.dtype == dtype, f"{name} must be {dtype}, got {t.dtype}")
    _need(t.is_contiguous(), f"{name} must be contiguous")
    if ndim is not None:
        _need(t.dim() == ndim, f"{name} must have {ndim} dims, got {tuple(t.shape)}")
    if last is not None:
        _need(t.shape[-1] == last, f"{name} last dim must be {last}")


def cache_desc(k_cache) -> CacheDesc:
    """Descriptor of a pool tensor [num_blocks, n_kv, 16, 128]: bf16, or FP8 E4M3 codes
    (torch.float8_e4m3fn or uint8)."""
    torch = _torch()
    fp8 = k_cache.dtype in (torch.uint8, torch.float8_e4m3fn)
    _check(k_cache, "k_cache", k_cache.dtype if fp8 else torch.bfloat16, ndim=4, last=HEAD_DIM)
    nb, n_kv, bs, d = k_cache.shape
    return CacheDesc(int(nb), int(bs), int(n_kv), int(d), PKV_DTYPE_FP8_E4M3 if fp8 else PKV_DTYPE_BF16)


def _out_dtype(out) -> int:
    torch = _torch()
    if out.dtype == torch.float32:
        return PKV_DTYPE_FLOAT32
    if out.dtype == torch.bfloat16:
        return PKV_DTYPE_BF16
    raise ValueError(f"out must be float32 or bfloat16, got {out.dtype}")


def _raise(fn, rc):
    if rc != PKV_OK:
        raise PagedKVError(fn, rc)


# ---- entry points (same names as the C ABI) ----------------------------------------

def kv_reshape_and_cache(key, value, k_cache, v_cache, slot_mapping, stream=None) -> None:
    torch = _torch()
    desc = cache_desc(k_cache)
    _check(v_cache, "v_cache", torch.bfloat16, ndim=4)
    _need(tuple(v_cache.shape) == tuple(k_cache.shape), "v_cache shape must equal k_cache shape")
    _check(key, "key", torch.bfloat16, ndim=3, last=HEAD_DIM)
    _check(value, "value", torch.bfloat16, ndim=3, last=HEAD_DIM)
    _check(slot_mapping, "slot_mapping", torch.int32, ndim=1)
    T = slot_mapping.shape[0]
    _need(tuple(key.shape) == (T, desc.num_kv_heads, HEAD_DIM), "key must be [num_tokens, n_kv, 128]")
    _need(tuple(value.shape) == tuple(key.shape), "value shape must equal key shape")
    rc = load_library().kv_reshape_and_cache(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
                                             _ptr(slot_mapping), int(T), ctypes.byref(desc), _stream(stream))
    _raise("kv_reshape_and_cache", rc)


def _check_fp8_pool(k_cache, v_cache, k_scale, v_scale):
    torch = _torch()
    desc = cache_desc(k_cache)
    _need(desc.dtype == PKV_DTYPE_FP8_E4M3, "k_cache must hold E4M3 codes (torch.float8_e4m3fn or uint8)")
    _check(v_cache, "v_cache", k_cache.dtype, ndim=4)
    _need(tuple(v_cache.shape) == tuple(k_cache.shape), "v_cache shape must equal k_cache shape")
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        _need(t is not None, f"{name} is required for an FP8 cache")
        _check(t, name, torch.float32, ndim=3)
        _need(tuple(t.shape) == tuple(k_cache.shape[:3]), f"{name} must be [num_blocks, n_kv, 16]")
    return desc


def kv_reshape_and_cache_fp8(key, value, k_cache, v_cache, k_scale, v_scale, slot_mapping, stream=None) -> None:
    """Quantise new tokens' K/V to E4M3 (one fp32 scale per token and KV head) into their slots."""
    torch = _torch()
    desc = _check_fp8_pool(k_cache, v_cache, k_scale, v_scale)
    _check(key, "key", torch.bfloat16, ndim=3, last=HEAD_DIM)
    _check(value, "value", torch.bfloat16, ndim=3, last=HEAD_DIM)
    _check(slot_mapping, "slot_mapping", torch.int32, ndim=1)
    T = slot_mapping.shape[0]
    _need(tuple(key.shape) == (T, desc.num_kv_heads, HEAD_DIM), "key must be [num_tokens, n_kv, 128]")
    _need(tuple(value.shape) == tuple(key.shape), "value shape must equal key shape")
    rc = load_library().kv_reshape_and_cache_fp8(_ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale),
                                                 _ptr(v_scale), _ptr(slot_mapping), int(T), ctypes.byref(desc),
                                                 _stream(stream))
    _raise("kv_reshape_and_cache_fp8", rc)


def kv_copy_blocks(k_cache, v_cache, block_pairs, k_scale=None, v_scale=None, stream=None) -> None:
    """Copy block pairs {source, destination} (int32 CUDA tensor [n, 2]) in both caches
    (and, for an FP8 cache, in both scale arrays)."""
    torch = _torch()
    desc = cache_desc(k_cache)
    _check(v_cache, "v_cache", k_cache.dtype, ndim=4)
    _need(tuple(v_cache.shape) == tuple(k_cache.shape), "v_cache shape must equal k_cache shape")
    _check(block_pairs, "block_pairs", torch.int32, ndim=2, last=2)
    fp8 = desc.dtype == PKV_DTYPE_FP8_E4M3
    _need(fp8 == (k_scale is not None) and fp8 == (v_scale is not None),
          "k_scale and v_scale are required for an FP8 cache and not allowed otherwise")
    if fp8:
        for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
            _check(t, name, torch.float32, ndim=3)
            _need(tuple(t.shape) == tuple(k_cache.shape[:3]), f"{name} must be [num_blocks, n_kv, 16]")
    rc = load_library().kv_copy_blocks(_ptr(k_cache), _ptr(v_cache), _ptr(k_scale) if fp8 else None,
                                       _ptr(v_scale) if fp8 else None, _ptr(block_pairs),
                                       int(block_pairs.shape[0]), ctypes.byref(desc), _stream(stream))
    _raise("kv_copy_blocks", rc)


class BlockManager:
    """Host block manager of the paged pool (``pkv_bm_*`` in include/pagedkv.h).

    Sequences are keyed by caller-chosen integers.  ``append`` returns the slot
    mapping of the new tokens and, when the sequence's shared last block had to
    be replaced first, the (source, destination) block pair to copy on the
    device with :func:`kv_copy_blocks` before writing the tokens.
    """

    def __init__(self, num_blocks: int):
        self._lib = load_library()
        h = ctypes.c_void_p()
        _raise("pkv_bm_create", self._lib.pkv_bm_create(int(num_blocks), ctypes.byref(h)))
        self._h = h
        self.num_blocks = int(num_blocks)

    def close(self):
        if getattr(self, "_h", None):
            self._lib.pkv_bm_destroy(self._h)
            self._h = None

    def __del__(self):
        self.close()

    @property
    def num_free(self) -> int:
        return int(self._lib.pkv_bm_num_free(self._h))

    def ref_count(self, block: int) -> int:
        c = ctypes.c_int32()
        _raise("pkv_bm_ref_count", self._lib.pkv_bm_ref_count(self._h, int(block), ctypes.byref(c)))
        return c.value

    def add(self, seq_id: int) -> None:
        _raise("pkv_bm_add_sequence", self._lib.pkv_bm_add_sequence(self._h, int(seq_id)))

    def fork(self, parent_id: int, child_id: int) -> None:
        _raise("pkv_bm_fork", self._lib.pkv_bm_fork(self._h, int(parent_id), int(child_id)))

    def append(self, seq_id: int, num_tokens: int):
        """Returns (slot_mapping int32 numpy [num_tokens], copy pair (src, dst) or None)."""
        import numpy as np
        slots = np.zeros(max(int(num_tokens), 1), dtype=np.int32)
        pair = np.zeros(2, dtype=np.int32)
        n = ctypes.c_int32()
        rc = self._lib.pkv_bm_append(self._h, int(seq_id), int(num_tokens), slots.ctypes.data,
                                     pair.ctypes.data, ctypes.byref(n))
        _raise("pkv_bm_append", rc)
        return slots[:int(num_tokens)], ((int(pair[0]), int(pair[1])) if n.value else None)

    def append_batch(self, seq_ids, num_tokens=None):
        """One call for a batch: returns (slot_mapping int32 [sum of num_tokens],
        copy pairs int32 [n_copies, 2]); num_tokens None means one token each."""
        import numpy as np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        n = len(ids)
        nt = None if num_tokens is None else np.ascontiguousarray(num_tokens, dtype=np.int32)
        total = n if nt is None else int(nt.sum())
        slots = np.zeros(max(total, 1), dtype=np.int32)
        pairs = np.zeros((max(n, 1), 2), dtype=np.int32)
        c = ctypes.c_int32()
        rc = self._lib.pkv_bm_append_batch(self._h, ids.ctypes.data, n, None if nt is None else nt.ctypes.data,
                                           slots.ctypes.data, pairs.ctypes.data, ctypes.byref(c))
        _raise("pkv_bm_append_batch", rc)
        return slots[:total], pairs[:c.value]

    def free(self, seq_id: int) -> None:
        _raise("pkv_bm_free_sequence", self._lib.pkv_bm_free_sequence(self._h, int(seq_id)))

    def length(self, seq_id: int) -> int:
        n = ctypes.c_int64()
        _raise("pkv_bm_sequence_length", self._lib.pkv_bm_sequence_length(self._h, int(seq_id), ctypes.byref(n)))
        return n.value

    def block_tables(self, seq_ids, max_blocks_per_seq: int, pad_block: int = 0):
        """Returns (block_tables int32 [B, max_blocks], context_lens int32 [B]) as numpy arrays."""
        import numpy as np
        ids = np.ascontiguousarray(seq_ids, dtype=np.int64)
        tables = np.zeros((max(len(ids), 1), int(max_blocks_per_seq)), dtype=np.int32)
        lens = np.zeros(max(len(ids), 1), dtype=np.int32)
        rc = self._lib.pkv_bm_block_tables(self._h, ids.ctypes.data, int(len(ids)), int(max_blocks_per_seq),
                                           int(pad_block), tables.ctypes.data, lens.ctypes.data)
        _raise("pkv_bm_block_tables", rc)
        return tables[:len(ids)], lens[:len(ids)]

    def publish(self, seq_id: int, tokens) -> None:
        import numpy as np
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        _raise("pkv_bm_publish", self._lib.pkv_bm_publish(self._h, int(seq_id), t.ctypes.data, int(t.shape[0])))

    def add_cached(self, seq_id: int, tokens) -> int:
        """New sequence for prompt `tokens`; returns how many leading tokens are already cached."""
        import numpy as np
        t = np.ascontiguousarray(tokens, dtype=np.int32)
        n = ctypes.c_int32()
        rc = self._lib.pkv_bm_add_sequence_cached(self._h, int(seq_id), t.ctypes.data, int(t.shape[0]),
                                                  ctypes.byref(n))
        _raise("pkv_bm_add_sequence_cached", rc)
        return n.value


def paged_attention_workspace_size(num_seqs: int, num_q_heads: int, max_blocks_per_seq: int,
                                   partition_size: int, cache: CacheDesc) -> int:
    return int(load_library().paged_attention_workspace_size(num_seqs, num_q_heads, max_blocks_per_seq,
                                                             partition_size, ctypes.byref(cache)))


def paged_attention_decode_partitions(num_seqs: int, num_q_heads: int, max_blocks_per_seq: int,
                                      partition_size: int, cache: CacheDesc, window: int = 0) -> int:
    """Partitions per sequence the decode entry points use (1: no merge kernel)."""
    n = int(load_library().paged_attention_decode_partitions(num_seqs, num_q_heads, max_blocks_per_seq,
                                                             partition_size, window, ctypes.byref(cache)))
    _raise("paged_attention_decode_partitions", min(n, 0))
    return n


def paged_attention_decode(out, q, k_cache, v_cache, block_tables, context_lens, scale: float,
                           workspace=None, partition_size: int = 0, stream=None, window: int = 0,
                           k_scale=None, v_scale=None):
    """Decode attention; ``workspace`` (uint8 CUDA tensor) is allocated if None.
    ``window`` > 0 calls paged_attention_decode_window (each row sees its newest
    ``window`` keys only).  An FP8 pool (E4M3 codes) with ``k_scale`` /
    ``v_scale`` calls paged_attention_decode_fp8."""
    torch = _torch()
    desc = cache_desc(k_cache)
    fp8 = desc.dtype == PKV_DTYPE_FP8_E4M3
    if fp8:
        _check_fp8_pool(k_cache, v_cache, k_scale, v_scale)
    else:
        _need(k_scale is None and v_scale is None, "scales are only for an FP8 cache")
        _check(v_cache, "v_cache", torch.bfloat16, ndim=4)
    _need(tuple(v_cache.shape) == tuple(k_cache.shape), "v_cache shape must equal k_cache shape")
    _check(q, "q", torch.bfloat16, ndim=3, last=HEAD_DIM)
    B, n_q, _ = q.shape
    _check(out, "out", out.dtype, ndim=3)
    _need(tuple(out.shape) == tuple(q.shape), "out must have q's shape")
    _check(block_tables, "block_tables", torch.int32, ndim=2)
    _check(context_lens, "context_lens", torch.int32, ndim=1)
    _need(block_tables.shape[0] == B and context_lens.shape[0] == B, "one table row and length per sequence")
    max_blocks = int(block_tables.shape[1])
    if workspace is None:
        nbytes = paged_attention_workspace_size(B, n_q, max_blocks, partition_size, desc)
        workspace = _new_workspace(nbytes, "paged_attention_decode", q, _stream(stream))  # status word starts clear
    _check(workspace, "workspace", torch.uint8, ndim=1)
    lib = load_library()
    if fp8:
        rc = lib.paged_attention_decode_fp8(
            _ptr(out), _out_dtype(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(k_scale), _ptr(v_scale),
            _ptr(block_tables), _ptr(context_lens), int(B), int(n_q), max_blocks, float(scale), int(window),
            int(partition_size), ctypes.byref(desc), _ptr(workspace), int(workspace.numel()), _stream(stream))
        _raise("paged_attention_decode_fp8", rc)
        return workspace
    if window:
        rc = lib.paged_attention_decode_window(
            _ptr(out), _out_dtype(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables),
            _ptr(context_lens), int(B), int(n_q), max_blocks, float(scale), int(window), int(partition_size),
            ctypes.byref(desc), _ptr(workspace), int(workspace.numel()), _stream(stream))
        _raise("paged_attention_decode_window", rc)
        return workspace
    rc = lib.paged_attention_decode(
        _ptr(out), _out_dtype(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        int(B), int(n_q), max_blocks, float(scale), int(partition_size), ctypes.byref(desc), _ptr(workspace),
        int(workspace.numel()), _stream(stream))
    _raise("paged_attention_decode", rc)
    return workspace


def paged_attention_verify(out, q, q_per_seq: int, k_cache, v_cache, block_tables, context_lens, scale: float,
                           workspace=None, partition_size: int = 0, stream=None, window: int = 0,
                           k_scale=None, v_scale=None, kernel: int = -1):
    """Verify k = q_per_seq draft positions per sequence: q / out [num_seqs * k, n_q, 128],
    row i of sequence b at position ctx_b - k + i (causal).  ``window`` > 0: row at pos
    sees pos - window < j <= pos.  An FP8 pool with ``k_scale`` / ``v_scale`` calls
    paged_attention_verify_fp8.  ``kernel`` (PKV_VERIFY_DECODE_KERNEL or
    PKV_VERIFY_PREFILL_KERNEL) forces one kernel through paged_attention_verify_on;
    PKV_VERIFY_AUTO lets the library's measured rule choose.  Returns the workspace."""
    torch = _torch()
    desc = cache_desc(k_cache)
    fp8 = desc.dtype == PKV_DTYPE_FP8_E4M3
    if fp8:
        _check_fp8_pool(k_cache, v_cache, k_scale, v_scale)
    else:
        _need(k_scale is None and v_scale is None, "scales are only for an FP8 cache")
        _check(v_cache, "v_cache", torch.bfloat16, ndim=4)
    _need(tuple(v_cache.shape) == tuple(k_cache.shape), "v_cache shape must equal k_cache shape")
    _check(q, "q", torch.bfloat16, ndim=3, last=HEAD_DIM)
    rows, n_q, _ = q.shape
    _check(out, "out", out.dtype, ndim=3)
    _need(tuple(out.shape) == tuple(q.shape), "out must have q's shape")
    _check(block_tables, "block_tables", torch.int32, ndim=2)
    _check(context_lens, "context_lens", torch.int32, ndim=1)
    B = int(context_lens.shape[0])
    _need(block_tables.shape[0] == B and rows == B * int(q_per_seq), "q must hold q_per_seq rows per sequence")
    max_blocks = int(block_tables.shape[1])
    lib = load_library()
    if workspace is None:
        nbytes = int(lib.paged_attention_verify_workspace_size_on(int(kernel), B, int(q_per_seq), n_q, max_blocks,
                                                                  int(partition_size), ctypes.byref(desc)))
        workspace = _new_workspace(nbytes, "paged_attention_verify", q, _stream(stream))
    _check(workspace, "workspace", torch.uint8, ndim=1)
    if kernel != PKV_VERIFY_AUTO:
        rc = lib.paged_attention_verify_on(int(kernel), _ptr(out), _out_dtype(out), _ptr(q), int(q_per_seq),
                                           _ptr(k_cache), _ptr(v_cache), _ptr(k_scale) if fp8 else None,
                                           _ptr(v_scale) if fp8 else None, _ptr(block_tables), _ptr(context_lens), B,
                                           int(n_q), max_blocks, float(scale), int(window), int(partition_size),
                                           ctypes.byref(desc), _ptr(workspace), int(workspace.numel()),
                                           _stream(stream))
        _raise("paged_attention_verify_on", rc)
        return workspace
    if fp8:
        rc = lib.paged_attention_verify_fp8(_ptr(out), _out_dtype(out), _ptr(q), int(q_per_seq), _ptr(k_cache),
                                            _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_tables),
                                            _ptr(context_lens), B, int(n_q), max_blocks, float(scale), int(window),
                                            int(partition_size), ctypes.byref(desc), _ptr(workspace),
                                            int(workspace.numel()), _stream(stream))
        _raise("paged_attention_verify_fp8", rc)
        return workspace
    if window:
        rc = lib.paged_attention_verify_window(_ptr(out), _out_dtype(out), _ptr(q), int(q_per_seq), _ptr(k_cache),
                                               _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), B, int(n_q),
                                               max_blocks, float(scale), int(partition_size), int(window),
                                               ctypes.byref(desc), _ptr(workspace), int(workspace.numel()),
                                               _stream(stream))
        _raise("paged_attention_verify_window", rc)
        return workspace
    rc = lib.paged_attention_verify(_ptr(out), _out_dtype(out), _ptr(q), int(q_per_seq), _ptr(k_cache),
                                    _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), B, int(n_q), max_blocks,
                                    float(scale), int(partition_size), ctypes.byref(desc), _ptr(workspace),
                                    int(workspace.numel()), _stream(stream))
    _raise("paged_attention_verify", rc)
    return workspace


def paged_attention_prefill_workspace_size(num_seqs: int, num_q_heads: int, cache: CacheDesc) -> int:
    return int(load_library().paged_attention_prefill_workspace_size(num_seqs, num_q_heads, ctypes.byref(cache)))


def paged_attention_prefill_chunk_workspace_size(num_seqs: int, num_q_heads: int, total_q_rows: int, max_q_len: int,
                                                 max_blocks_per_seq: int, cache: CacheDesc) -> int:
    """Workspace bytes with which the prefill chunk may split its keys (split-KV)."""
    return int(load_library().paged_attention_prefill_chunk_workspace_size(
        num_seqs, num_q_heads, total_q_rows, max_q_len, max_blocks_per_seq, ctypes.byref(cache)))


def paged_attention_prefill_chunk(out, q, cu_q_lens, max_q_len: int, k_cache, v_cache, block_tables, context_lens,
                                  scale: float, workspace=None, stream=None, window: int = 0, k_scale=None,
                                  v_scale=None):
    """Causal chunked-prefill attention; ``workspace`` is allocated if None.
    ``window`` > 0 calls paged_attention_prefill_chunk_window (row at pos sees
    keys pos - window < j <= pos); an FP8 cache with ``k_scale`` / ``v_scale``
    calls paged_attention_prefill_chunk_fp8."""
    torch = _torch()
    fp8 = k_scale is not None or v_scale is not None
    if fp8:
        desc = _check_fp8_pool(k_cache, v_cache, k_scale, v_scale)
    else:
        desc = cache_desc(k_cache)
        _check(v_cache, "v_cache", torch.bfloat16, ndim=4)
        _need(tuple(v_cache.shape) == tuple(k_cache.shape), "v_cache shape must equal k_cache shape")
    _check(q, "q", torch.bfloat16, ndim=3, last=HEAD_DIM)
    rows, n_q, _ = q.shape
    _check(out, "out", out.dtype, ndim=3)
    _need(tuple(out.shape) == tuple(q.shape), "out must have q's shape")
    _check(cu_q_lens, "cu_q_lens", torch.int32, ndim=1)
    _check(block_tables, "block_tables", torch.int32, ndim=2)
    _check(context_lens, "context_lens", torch.int32, ndim=1)
    B = int(context_lens.shape[0])
    _need(cu_q_lens.shape[0] == B + 1 and block_tables.shape[0] == B, "cu_q_lens is [B+1], block_tables [B, *]")
    if workspace is None:
        nbytes = paged_attention_prefill_chunk_workspace_size(B, n_q, int(rows), int(max_q_len),
                                                              int(block_tables.shape[1]), desc)
        workspace = _new_workspace(nbytes, "paged_attention_prefill_chunk", q, _stream(stream))  # status word starts clear
    _check(workspace, "workspace", torch.uint8, ndim=1)
    lib = load_library()
    if fp8:
        rc = lib.paged_attention_prefill_chunk_fp8(
            _ptr(out), _out_dtype(out), _ptr(q), _ptr(cu_q_lens), int(max_q_len), int(rows), _ptr(k_cache),
            _ptr(v_cache), _ptr(k_scale), _ptr(v_scale), _ptr(block_tables), _ptr(context_lens), B, int(n_q),
            int(block_tables.shape[1]), float(scale), int(window), ctypes.byref(desc), _ptr(workspace),
            int(workspace.numel()), _stream(stream))
        _raise("paged_attention_prefill_chunk_fp8", rc)
        return workspace
    if window:
        rc = lib.paged_attention_prefill_chunk_window(
            _ptr(out), _out_dtype(out), _ptr(q), _ptr(cu_q_lens), int(max_q_len), int(rows), _ptr(k_cache),
            _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), B, int(n_q), int(block_tables.shape[1]),
            float(scale), int(window), ctypes.byref(desc), _ptr(workspace), int(workspace.numel()), _stream(stream))
        _raise("paged_attention_prefill_chunk_window", rc)
        return workspace
    rc = lib.paged_attention_prefill_chunk(
        _ptr(out), _out_dtype(out), _ptr(q), _ptr(cu_q_lens), int(max_q_len), int(rows), _ptr(k_cache),
        _ptr(v_cache), _ptr(block_tables), _ptr(context_lens), B, int(n_q), int(block_tables.shape[1]),
        float(scale), ctypes.byref(desc), _ptr(workspace), int(workspace.numel()), _stream(stream))
    _raise("paged_attention_prefill_chunk", rc)
    return workspace


def paged_attention_decode_append(out, q, key, value, k_cache, v_cache, block_tables, context_lens, scale: float,
                                  workspace=None, partition_size: int = 0, stream=None):
    """One decode step in one launch: writes ``key`` / ``value`` (bf16
    [B, n_kv, 128], each sequence's row of position ctx - 1) into the pool and
    attends, as kv_reshape_and_cache + paged_attention_decode would."""
    torch = _torch()
    desc = cache_desc(k_cache)
    _check(v_cache, "v_cache", torch.bfloat16, ndim=4)
    _need(tuple(v_cache.shape) == tuple(k_cache.shape), "v_cache shape must equal k_cache shape")
    _check(q, "q", torch.bfloat16, ndim=3, last=HEAD_DIM)
    B, n_q, _ = q.shape
    n_kv = int(k_cache.shape[1])
    for name, t in (("key", key), ("value", value)):
        _check(t, name, torch.bfloat16, ndim=3, last=HEAD_DIM)
        _need(tuple(t.shape) == (B, n_kv, HEAD_DIM), f"{name} must be [num_seqs, num_kv_heads, 128]")
    _check(out, "out", out.dtype, ndim=3)
    _need(tuple(out.shape) == tuple(q.shape), "out must have q's shape")
    _check(block_tables, "block_tables", torch.int32, ndim=2)
    _check(context_lens, "context_lens", torch.int32, ndim=1)
    _need(block_tables.shape[0] == B and context_lens.shape[0] == B, "one table row and length per sequence")
    max_blocks = int(block_tables.shape[1])
    if workspace is None:
        nbytes = paged_attention_workspace_size(B, n_q, max_blocks, partition_size, desc)
        workspace = _new_workspace(nbytes, "paged_attention_decode_append", q, _stream(stream))
    _check(workspace, "workspace", torch.uint8, ndim=1)
    rc = load_library().paged_attention_decode_append(
        _ptr(out), _out_dtype(out), _ptr(q), _ptr(key), _ptr(value), _ptr(k_cache), _ptr(v_cache),
        _ptr(block_tables), _ptr(context_lens), int(B), int(n_q), max_blocks, float(scale), int(partition_size),
        ctypes.byref(desc), _ptr(workspace), int(workspace.numel()), _stream(stream))
    _raise("paged_attention_decode_append", rc)
    return workspace


def paged_attention_decode_static_scratch(out, q, k_cache, v_cache, block_tables, context_lens, scale: float,
                                          partition_size: int = 0, status=None, stream=None) -> None:
    """Decode attention that allocates nothing: the split-KV scratch is the
    library's fixed device array (STATIC_SCRATCH_BYTES), shared by all calls on
    a device, so calls must not overlap on the GPU.  ``status`` is an optional
    int32 CUDA tensor of one element that receives the call's status bits."""
    torch = _torch()
    desc = cache_desc(k_cache)
    _check(v_cache, "v_cache", torch.bfloat16, ndim=4)
    _need(tuple(v_cache.shape) == tuple(k_cache.shape), "v_cache shape must equal k_cache shape")
    _check(q, "q", torch.bfloat16, ndim=3, last=HEAD_DIM)
    B, n_q, _ = q.shape
    _check(out, "out", out.dtype, ndim=3)
    _need(tuple(out.shape) == tuple(q.shape), "out must have q's shape")
    _check(block_tables, "block_tables", torch.int32, ndim=2)
    _check(context_lens, "context_lens", torch.int32, ndim=1)
    if status is not None:
        _check(status, "status", torch.int32, ndim=1)
    rc = load_library().paged_attention_decode_static_scratch(
        _ptr(out), _out_dtype(out), _ptr(q), _ptr(k_cache), _ptr(v_cache), _ptr(block_tables), _ptr(context_lens),
        int(B), int(n_q), int(block_tables.shape[1]), float(scale), int(partition_size), ctypes.byref(desc),
        _ptr(status) if status is not None else None, _stream(stream))
    _raise("paged_attention_decode_static_scratch", rc)


# ---- latent attention ---------------------------------------------------------------
# (A decode of few tokens takes 10 us on the GPU: an argument is looked at once, and its error put into words only where
# something is wrong with it.  The tensors keep their names to the end of a call: an address alone would let a temporary
# be freed, and its memory handed out, before the launch.)

def _check_rows(t, name, ndim, last, device):
    """Raises what is wrong with a bf16 input of contiguous rows."""
    torch = _torch()
    _need(isinstance(t, torch.Tensor), f"{name} must be a torch.Tensor")
    _need(t.dtype == torch.bfloat16, f"{name} must be torch.bfloat16, got {t.dtype}")
    _need(t.dim() == ndim and t.shape[-1] == last, f"{name} must have {ndim} dims, the last {last}: {tuple(t.shape)}")
    _need(t.get_device() == device, f"{name} must be on the current CUDA device")
    _need(False, f"{name}'s innermost dimension must be contiguous")


def _rows(t, name, ndim, last, device):
    """Shape, strides and address of a bf16 input whose rows (innermost dimension) are contiguous; the outer strides are
    free, and packed where a dimension is never stepped (size 1)."""
    try:
        shape, strides = t.shape, t.stride()
        if (t.dtype is _torch().bfloat16 and len(strides) == ndim and shape[-1] == last and strides[-1] == 1
                and t.get_device() == device):
            if shape[0] == 1 or shape[-2] == 1:
                strides = tuple(n if size > 1 else last for size, n in zip(shape, strides))
            return shape, strides, t.data_ptr()
    except AttributeError:
        pass
    return _check_rows(t, name, ndim, last, device)


def _flat(t, name, dtype, ndim, device):
    """Shape and address of a contiguous tensor on the current device."""
    try:
        if t.dtype is dtype and t.get_device() == device and t.is_contiguous():
            shape = t.shape
            if len(shape) == ndim:
                return shape, t.data_ptr()
    except AttributeError:
        pass
    _check(t, name, dtype, ndim=ndim)
    raise ValueError(f"{name} must be on the current CUDA device")


def _latent_out(out, device):
    torch = _torch()
    dtype = getattr(out, "dtype", None)
    if dtype is torch.bfloat16:
        code = PKV_DTYPE_BF16
    elif dtype is torch.float32:
        code = PKV_DTYPE_FLOAT32
    else:
        raise ValueError(f"out must be float32 or bfloat16, got {dtype}")
    return code, *_flat(out, "out", dtype, 3, device)


_cuda_started = False


def _device_and_stream(stream):
    """The current device, and `stream` (None: the current one) as the ABI takes it."""
    global _cuda_started
    torch = _torch()
    if not _cuda_started:
        _need(torch.cuda.is_available(), "the latent entry points need a CUDA device")
        torch.cuda.init()
        _cuda_started = True
    device = torch._C._cuda_getDevice()
    return device, torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def latent_cache_desc(cache) -> LatentDesc:
    """Descriptor of a latent pool: bf16 [num_blocks, 16, 576], or FP8 E4M3 codes
    (torch.float8_e4m3fn or uint8) [num_blocks, 16, 512]."""
    torch = _torch()
    dtype = cache.dtype
    fp8 = dtype is torch.uint8 or dtype is torch.float8_e4m3fn
    _check(cache, "cache", dtype if fp8 else torch.bfloat16, ndim=3)
    blocks, slots, width = cache.shape
    want = LATENT_DIM if fp8 else LATENT_DIM + ROPE_DIM
    _need(width == want, f"cache rows must have {want} values, got {width}")
    return LatentDesc(blocks, slots, LATENT_DIM, ROPE_DIM, PKV_DTYPE_FP8_E4M3 if fp8 else PKV_DTYPE_BF16)


@functools.lru_cache(maxsize=64)
def _latent_desc(blocks, slots, dtype):
    return ctypes.byref(LatentDesc(blocks, slots, LATENT_DIM, ROPE_DIM, dtype))


def _latent_pool(cache, rope_cache, cache_scale, device):
    """(descriptor, FP8, addresses of cache, rope_cache and cache_scale)."""
    torch = _torch()
    dtype = getattr(cache, "dtype", None)
    fp8 = dtype is torch.uint8 or dtype is torch.float8_e4m3fn
    (blocks, slots, width), address = _flat(cache, "cache", dtype if fp8 else torch.bfloat16, 3, device)
    if width != (LATENT_DIM if fp8 else LATENT_DIM + ROPE_DIM):
        latent_cache_desc(cache)
    if fp8 != (rope_cache is not None) or fp8 != (cache_scale is not None):
        raise ValueError("rope_cache and cache_scale are required for an FP8 pool and not allowed otherwise")
    if not fp8:
        return _latent_desc(blocks, slots, PKV_DTYPE_BF16), False, address, None, None
    shape, rope = _flat(rope_cache, "rope_cache", torch.bfloat16, 3, device)
    if shape != (blocks, slots, ROPE_DIM):
        raise ValueError("rope_cache must be [num_blocks, 16, 64]")
    shape, scale = _flat(cache_scale, "cache_scale", torch.float32, 2, device)
    if shape != (blocks, slots):
        raise ValueError("cache_scale must be [num_blocks, 16]")
    return _latent_desc(blocks, slots, PKV_DTYPE_FP8_E4M3), True, address, rope, scale


def _latent_rows(latent, rope, slot_mapping, device):
    """(latent, its stride, rope, its stride, slots, tokens) of a write."""
    latent_shape, latent_strides, latent_at = _rows(latent, "latent", 2, LATENT_DIM, device)
    rope_shape, rope_strides, rope_at = _rows(rope, "rope", 2, ROPE_DIM, device)
    (tokens,), slots = _flat(slot_mapping, "slot_mapping", _torch().int32, 1, device)
    if latent_shape[0] != tokens or rope_shape[0] != tokens:
        raise ValueError("one latent and one rope row per slot")
    return latent_at, latent_strides[0], rope_at, rope_strides[0], slots, tokens


def latent_reshape_and_cache(latent, rope, cache, slot_mapping, stream=None) -> None:
    """Append rows [latent (512) | rope (64)] to the bf16 latent pool [num_blocks, 16, 576]
    through ``slot_mapping``; ``latent`` and ``rope`` may be slices of wider rows."""
    device, stream = _device_and_stream(stream)
    desc, _, pool, _, _ = _latent_pool(cache, None, None, device)
    rows = _latent_rows(latent, rope, slot_mapping, device)
    rc = (_lib or load_library()).latent_reshape_and_cache(*rows[:4], pool, *rows[4:], desc, stream)
    _raise("latent_reshape_and_cache", rc)


def latent_reshape_and_cache_fp8(latent, rope, cache, rope_cache, cache_scale, slot_mapping, stream=None) -> None:
    """The same into an FP8 pool: E4M3 codes of the latent with one fp32 scale a token
    (``cache_scale`` [num_blocks, 16]); the rotated key goes to ``rope_cache`` as it is."""
    device, stream = _device_and_stream(stream)
    desc, _, pool, rope_pool, scales = _latent_pool(cache, rope_cache, cache_scale, device)
    rows = _latent_rows(latent, rope, slot_mapping, device)
    rc = (_lib or load_library()).latent_reshape_and_cache_fp8(*rows[:4], pool, rope_pool, scales, *rows[4:], desc, stream)
    _raise("latent_reshape_and_cache_fp8", rc)


def latent_gather(out, cache, block_tables, cu_lens, rope_cache=None, cache_scale=None, status=None,
                  stream=None) -> None:
    """Read cached rows back in sequence order: row cu_lens[b] + i of ``out`` (bf16 [total, 576])
    is position i of sequence b; an FP8 pool is dequantised and rounded once.  ``status`` is
    an optional int32 CUDA tensor of one element into which status bits are ORed."""
    torch = _torch()
    device, stream = _device_and_stream(stream)
    desc, _, pool, rope_pool, scales = _latent_pool(cache, rope_cache, cache_scale, device)
    (rows, width), out_at = _flat(out, "out", torch.bfloat16, 2, device)
    if width != LATENT_DIM + ROPE_DIM:
        raise ValueError("out must be [total_rows, 576]")
    (B, max_blocks), tables = _flat(block_tables, "block_tables", torch.int32, 2, device)
    (n,), lens_at = _flat(cu_lens, "cu_lens", torch.int32, 1, device)
    if n != B + 1:
        raise ValueError("cu_lens must be [num_seqs + 1]")
    status_at = None if status is None else _flat(status, "status", torch.int32, 1, device)[1]
    rc = (_lib or load_library()).latent_gather(out_at, pool, rope_pool, scales, tables, lens_at, B, max_blocks, rows, desc,
                                                status_at, stream)
    _raise("latent_gather", rc)


def latent_attention_workspace_size(num_seqs: int, q_per_seq: int, num_q_heads: int, max_blocks_per_seq: int,
                                    desc: LatentDesc) -> int:
    return int(load_library().latent_attention_workspace_size(num_seqs, q_per_seq, num_q_heads, max_blocks_per_seq,
                                                              ctypes.byref(desc)))


def latent_attention_decode(out, q_latent, q_rope, cache, block_tables, context_lens, scale: float, workspace=None,
                            q_per_seq: int = 1, rope_cache=None, cache_scale=None, stream=None):
    """Absorbed latent attention over the paged pool: ``q_latent`` [num_seqs * q_per_seq, heads,
    512] and ``q_rope`` [.., heads, 64] (rows and heads may be strided), ``out`` [.., heads, 512]
    in float32 or bfloat16.  Row i of sequence b sits at position ctx_b - q_per_seq + i and
    sees the keys up to it.  An FP8 pool comes with ``rope_cache`` and ``cache_scale``
    (latent_attention_decode_fp8).  Returns the workspace (allocated if None)."""
    torch = _torch()
    device, stream = _device_and_stream(stream)
    desc, fp8, pool, rope_pool, scales = _latent_pool(cache, rope_cache, cache_scale, device)
    (rows, heads, _), ql_strides, ql = _rows(q_latent, "q_latent", 3, LATENT_DIM, device)
    shape, qr_strides, qr = _rows(q_rope, "q_rope", 3, ROPE_DIM, device)
    if shape != (rows, heads, ROPE_DIM):
        raise ValueError("q_rope must have q_latent's rows and heads")
    code, shape, out_at = _latent_out(out, device)
    if shape != (rows, heads, LATENT_DIM):
        raise ValueError("out must have q_latent's shape")
    (B, max_blocks), tables = _flat(block_tables, "block_tables", torch.int32, 2, device)
    (n,), lens = _flat(context_lens, "context_lens", torch.int32, 1, device)
    k = int(q_per_seq)
    if n != B or rows != B * k:
        raise ValueError("q_latent must hold q_per_seq rows per sequence")
    lib = _lib or load_library()
    if workspace is None:
        workspace = _new_workspace(lib.latent_attention_workspace_size(B, k, heads, max_blocks, desc), "latent_attention_decode", out,
                                   stream, clear=256)
    (size,), space = _flat(workspace, "workspace", torch.uint8, 1, device)
    if fp8:
        rc = lib.latent_attention_decode_fp8(out_at, code, ql, ql_strides[0], ql_strides[1], qr, qr_strides[0], qr_strides[1],
                                             pool, rope_pool, scales, tables, lens, B, k, heads, max_blocks, scale, desc, space,
                                             size, stream)
        _raise("latent_attention_decode_fp8", rc)
    else:
        rc = lib.latent_attention_decode(out_at, code, ql, ql_strides[0], ql_strides[1], qr, qr_strides[0], qr_strides[1],
                                         pool, tables, lens, B, k, heads, max_blocks, scale, desc, space, size, stream)
        _raise("latent_attention_decode", rc)
    return workspace


def latent_attention_prefill_workspace_size(num_seqs: int, num_heads: int, max_q_len: int, total_q_rows: int,
                                            total_k_rows: int) -> int:
    return int(load_library().latent_attention_prefill_workspace_size(num_seqs, num_heads, max_q_len, total_q_rows,
                                                                      total_k_rows))


def latent_attention_prefill_chunk(out, q, k_nope, v, k_rope, cu_q_lens, cu_k_lens, max_q_len: int, scale: float,
                                   workspace=None, stream=None):
    """Expanded latent attention of a causal chunk: ``q`` [total_q, heads, 192], ``k_nope`` and
    ``v`` [total_k, heads, 128] (usually the halves of one [total_k, heads, 256] product, so of
    equal strides), ``k_rope`` [total_k, 64] shared by the heads, ``out`` [total_q, heads, 128]
    in float32 or bfloat16.  Returns the workspace (allocated if None)."""
    torch = _torch()
    device, stream = _device_and_stream(stream)
    (tq, heads, _), q_strides, q_at = _rows(q, "q", 3, 192, device)
    k_shape, k_strides, k_at = _rows(k_nope, "k_nope", 3, 128, device)
    v_shape, v_strides, v_at = _rows(v, "v", 3, 128, device)
    rope_shape, rope_strides, rope_at = _rows(k_rope, "k_rope", 2, ROPE_DIM, device)
    tk = k_shape[0]
    if k_shape[1] != heads or v_shape != k_shape or rope_shape[0] != tk:
        raise ValueError("k_nope and v must be [total_k, heads, 128], k_rope [total_k, 64]")
    if k_strides != v_strides:
        raise ValueError("k_nope and v must have the same strides")
    code, shape, out_at = _latent_out(out, device)
    if shape != (tq, heads, 128):
        raise ValueError("out must be [total_q, heads, 128]")
    (n,), cu_q = _flat(cu_q_lens, "cu_q_lens", torch.int32, 1, device)
    (m,), cu_k = _flat(cu_k_lens, "cu_k_lens", torch.int32, 1, device)
    if m != n:
        raise ValueError("cu_q_lens and cu_k_lens must be [num_seqs + 1]")
    B, max_q_len = n - 1, int(max_q_len)
    lib = _lib or load_library()
    if workspace is None:
        workspace = _new_workspace(lib.latent_attention_prefill_workspace_size(B, heads, max_q_len, tq, tk),
                                   "latent_attention_prefill_chunk", out, stream, clear=256)
    (size,), space = _flat(workspace, "workspace", torch.uint8, 1, device)
    rc = lib.latent_attention_prefill_chunk(out_at, code, q_at, q_strides[0], q_strides[1], k_at, v_at, k_strides[0], k_strides[1],
                                            rope_at, rope_strides[0], cu_q, cu_k, B, heads, max_q_len, tq, tk, scale, space, size,
                                            stream)
    _raise("latent_attention_prefill_chunk", rc)
    return workspace
