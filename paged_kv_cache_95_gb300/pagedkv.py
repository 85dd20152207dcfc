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

def _torch():
    import torch
    return torch


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
        _need(nbytes > 0, "invalid sizes for paged_attention_decode")
        workspace = torch.zeros(nbytes, dtype=torch.uint8, device=q.device)  # status word starts clear
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
        _need(nbytes > 0, "invalid sizes for paged_attention_verify")
        workspace = torch.zeros(nbytes, dtype=torch.uint8, device=q.device)
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
        _need(nbytes > 0, "invalid sizes for paged_attention_prefill_chunk")
        workspace = torch.zeros(nbytes, dtype=torch.uint8, device=q.device)  # status word starts clear
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
        _need(nbytes > 0, "invalid sizes for paged_attention_decode_append")
        workspace = torch.zeros(nbytes, dtype=torch.uint8, device=q.device)
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

def _addr(t) -> int:
    return t.data_ptr()


def _check_rows(t, name, ndim, last, device):
    """A bf16 input whose rows (innermost dimension) are contiguous; the outer strides are free."""
    torch = _torch()
    if not (isinstance(t, torch.Tensor) and t.dtype is torch.bfloat16 and t.dim() == ndim and t.shape[-1] == last
            and t.get_device() == device and t.stride(-1) == 1):
        _need(isinstance(t, torch.Tensor), f"{name} must be a torch.Tensor")
        _need(t.dtype == torch.bfloat16, f"{name} must be torch.bfloat16, got {t.dtype}")
        _need(t.dim() == ndim and t.shape[-1] == last, f"{name} must have {ndim} dims, the last {last}: {tuple(t.shape)}")
        _need(t.get_device() == device, f"{name} must be on the current CUDA device")
        _need(False, f"{name}'s innermost dimension must be contiguous")


def _check_on(t, name, dtype, ndim, device):
    """A contiguous tensor on the current device."""
    if not (isinstance(t, _torch().Tensor) and t.dtype is dtype and t.dim() == ndim and t.get_device() == device
            and t.is_contiguous()):
        _check(t, name, dtype, ndim=ndim)
        _need(False, f"{name} must be on the current CUDA device")


def _outer_stride(t, dim: int) -> int:
    """The stride of an outer dimension; the packed one where its size is 1 (it is never stepped)."""
    return t.stride(dim) if t.shape[dim] > 1 else (t.shape[-1] + 7) // 8 * 8


def _device_and_stream(stream):
    """The current device, and `stream` (None: the current one) as the ABI takes it."""
    torch = _torch()
    if not torch.cuda.is_initialized():
        _need(torch.cuda.is_available(), "the latent entry points need a CUDA device")
        torch.cuda.init()
    device = torch._C._cuda_getDevice()
    return device, torch._C._cuda_getCurrentRawStream(device) if stream is None else _stream(stream)


def latent_cache_desc(cache) -> LatentDesc:
    """Descriptor of a latent pool: bf16 [num_blocks, 16, 576], or FP8 E4M3 codes
    (torch.float8_e4m3fn or uint8) [num_blocks, 16, 512]."""
    torch = _torch()
    dtype = cache.dtype
    fp8 = dtype is torch.uint8 or dtype is torch.float8_e4m3fn
    if not (cache.dim() == 3 and cache.is_cuda and cache.is_contiguous() and (fp8 or dtype is torch.bfloat16)):
        _check(cache, "cache", dtype if fp8 else torch.bfloat16, ndim=3)
    blocks, slots, width = cache.shape
    want = LATENT_DIM if fp8 else LATENT_DIM + ROPE_DIM
    if width != want:
        _need(False, f"cache rows must have {want} values, got {width}")
    return LatentDesc(blocks, slots, LATENT_DIM, ROPE_DIM, PKV_DTYPE_FP8_E4M3 if fp8 else PKV_DTYPE_BF16)


def _latent_pool(cache, rope_cache, cache_scale, device):
    torch = _torch()
    desc = latent_cache_desc(cache)
    fp8 = desc.dtype == PKV_DTYPE_FP8_E4M3
    if cache.get_device() != device:
        _need(False, "cache must be on the current CUDA device")
    if fp8 != (rope_cache is not None) or fp8 != (cache_scale is not None):
        _need(False, "rope_cache and cache_scale are required for an FP8 pool and not allowed otherwise")
    if fp8:
        _check_on(rope_cache, "rope_cache", torch.bfloat16, 3, device)
        _check_on(cache_scale, "cache_scale", torch.float32, 2, device)
        shape = cache.shape[:2]
        if rope_cache.shape[:2] != shape or rope_cache.shape[2] != ROPE_DIM:
            _need(False, "rope_cache must be [num_blocks, 16, 64]")
        if cache_scale.shape != shape:
            _need(False, "cache_scale must be [num_blocks, 16]")
    return desc, fp8


def _check_latent_rows(latent, rope, slot_mapping, device):
    torch = _torch()
    _check_rows(latent, "latent", 2, LATENT_DIM, device)
    _check_rows(rope, "rope", 2, ROPE_DIM, device)
    _check_on(slot_mapping, "slot_mapping", torch.int32, 1, device)
    T = slot_mapping.shape[0]
    _need(latent.shape[0] == T and rope.shape[0] == T, "one latent and one rope row per slot")
    return int(T)


def latent_reshape_and_cache(latent, rope, cache, slot_mapping, stream=None) -> None:
    """Append rows [latent (512) | rope (64)] to the bf16 latent pool [num_blocks, 16, 576]
    through ``slot_mapping``; ``latent`` and ``rope`` may be slices of wider rows."""
    device, stream = _device_and_stream(stream)
    desc, fp8 = _latent_pool(cache, None, None, device)
    T = _check_latent_rows(latent, rope, slot_mapping, device)
    rc = load_library().latent_reshape_and_cache(_addr(latent), _outer_stride(latent, 0), _addr(rope),
                                                 _outer_stride(rope, 0), _addr(cache), _addr(slot_mapping), T,
                                                 ctypes.byref(desc), stream)
    _raise("latent_reshape_and_cache", rc)


def latent_reshape_and_cache_fp8(latent, rope, cache, rope_cache, cache_scale, slot_mapping, stream=None) -> None:
    """The same into an FP8 pool: E4M3 codes of the latent with one fp32 scale a token
    (``cache_scale`` [num_blocks, 16]); the rotated key goes to ``rope_cache`` as it is."""
    device, stream = _device_and_stream(stream)
    desc, fp8 = _latent_pool(cache, rope_cache, cache_scale, device)
    T = _check_latent_rows(latent, rope, slot_mapping, device)
    rc = load_library().latent_reshape_and_cache_fp8(_addr(latent), _outer_stride(latent, 0), _addr(rope),
                                                     _outer_stride(rope, 0), _addr(cache), _addr(rope_cache),
                                                     _addr(cache_scale), _addr(slot_mapping), T, ctypes.byref(desc),
                                                     stream)
    _raise("latent_reshape_and_cache_fp8", rc)


def latent_gather(out, cache, block_tables, cu_lens, rope_cache=None, cache_scale=None, status=None,
                  stream=None) -> None:
    """Read cached rows back in sequence order: row cu_lens[b] + i of ``out`` (bf16 [total, 576])
    is position i of sequence b; an FP8 pool is dequantised and rounded once.  ``status`` is
    an optional int32 CUDA tensor of one element into which status bits are ORed."""
    torch = _torch()
    device, stream = _device_and_stream(stream)
    desc, fp8 = _latent_pool(cache, rope_cache, cache_scale, device)
    _check_on(out, "out", torch.bfloat16, 2, device)
    _need(out.shape[1] == LATENT_DIM + ROPE_DIM, "out must be [total_rows, 576]")
    _check_on(block_tables, "block_tables", torch.int32, 2, device)
    _check_on(cu_lens, "cu_lens", torch.int32, 1, device)
    B = int(block_tables.shape[0])
    _need(cu_lens.shape[0] == B + 1, "cu_lens must be [num_seqs + 1]")
    if status is not None:
        _check_on(status, "status", torch.int32, 1, device)
    rc = load_library().latent_gather(_addr(out), _addr(cache), _addr(rope_cache) if fp8 else None,
                                      _addr(cache_scale) if fp8 else None, _addr(block_tables), _addr(cu_lens), B,
                                      int(block_tables.shape[1]), int(out.shape[0]), ctypes.byref(desc),
                                      _addr(status) if status is not None else None, stream)
    _raise("latent_gather", rc)


def _latent_workspace(nbytes, device):
    """Device scratch whose status word starts clear (the rest is written before it is read)."""
    workspace = _torch().empty(nbytes, dtype=_torch().uint8, device=device)
    workspace[:256].zero_()
    return workspace


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
    desc, fp8 = _latent_pool(cache, rope_cache, cache_scale, device)
    _check_rows(q_latent, "q_latent", 3, LATENT_DIM, device)
    _check_rows(q_rope, "q_rope", 3, ROPE_DIM, device)
    rows, heads, _ = q_latent.shape
    _need(tuple(q_rope.shape[:2]) == (rows, heads), "q_rope must have q_latent's rows and heads")
    _check_on(out, "out", out.dtype, 3, device)
    _need(tuple(out.shape) == (rows, heads, LATENT_DIM), "out must have q_latent's shape")
    _check_on(block_tables, "block_tables", torch.int32, 2, device)
    _check_on(context_lens, "context_lens", torch.int32, 1, device)
    B, k = int(context_lens.shape[0]), int(q_per_seq)
    _need(block_tables.shape[0] == B and rows == B * k, "q_latent must hold q_per_seq rows per sequence")
    max_blocks = int(block_tables.shape[1])
    lib = load_library()
    if workspace is None:
        nbytes = int(lib.latent_attention_workspace_size(B, k, int(heads), max_blocks, ctypes.byref(desc)))
        _need(nbytes > 0, "invalid sizes for latent_attention_decode")
        workspace = _latent_workspace(nbytes, out.device)
    _check_on(workspace, "workspace", torch.uint8, 1, device)
    ql = (_addr(q_latent), _outer_stride(q_latent, 0), _outer_stride(q_latent, 1))
    qr = (_addr(q_rope), _outer_stride(q_rope, 0), _outer_stride(q_rope, 1))
    tail = (_addr(block_tables), _addr(context_lens), B, k, int(heads), max_blocks, float(scale), ctypes.byref(desc),
            _addr(workspace), int(workspace.numel()), stream)
    if fp8:
        rc = lib.latent_attention_decode_fp8(_addr(out), _out_dtype(out), *ql, *qr, _addr(cache), _addr(rope_cache),
                                             _addr(cache_scale), *tail)
        _raise("latent_attention_decode_fp8", rc)
    else:
        rc = lib.latent_attention_decode(_addr(out), _out_dtype(out), *ql, *qr, _addr(cache), *tail)
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
    _check_rows(q, "q", 3, 192, device)
    _check_rows(k_nope, "k_nope", 3, 128, device)
    _check_rows(v, "v", 3, 128, device)
    _check_rows(k_rope, "k_rope", 2, ROPE_DIM, device)
    tq, heads, _ = q.shape
    tk = int(k_nope.shape[0])
    _need(k_nope.shape[1] == heads and tuple(v.shape) == tuple(k_nope.shape) and k_rope.shape[0] == tk,
          "k_nope and v must be [total_k, heads, 128], k_rope [total_k, 64]")
    k_strides = (_outer_stride(k_nope, 0), _outer_stride(k_nope, 1))
    _need(k_strides == (_outer_stride(v, 0), _outer_stride(v, 1)), "k_nope and v must have the same strides")
    _check_on(out, "out", out.dtype, 3, device)
    _need(tuple(out.shape) == (tq, heads, 128), "out must be [total_q, heads, 128]")
    _check_on(cu_q_lens, "cu_q_lens", torch.int32, 1, device)
    _check_on(cu_k_lens, "cu_k_lens", torch.int32, 1, device)
    B = int(cu_q_lens.shape[0]) - 1
    _need(cu_k_lens.shape[0] == B + 1, "cu_q_lens and cu_k_lens must be [num_seqs + 1]")
    lib = load_library()
    if workspace is None:
        nbytes = int(lib.latent_attention_prefill_workspace_size(B, int(heads), int(max_q_len), int(tq), tk))
        _need(nbytes > 0, "invalid sizes for latent_attention_prefill_chunk")
        workspace = _latent_workspace(nbytes, out.device)
    _check_on(workspace, "workspace", torch.uint8, 1, device)
    rc = lib.latent_attention_prefill_chunk(_addr(out), _out_dtype(out), _addr(q), _outer_stride(q, 0),
                                            _outer_stride(q, 1), _addr(k_nope), _addr(v), *k_strides, _addr(k_rope),
                                            _outer_stride(k_rope, 0), _addr(cu_q_lens), _addr(cu_k_lens), B, int(heads),
                                            int(max_q_len), int(tq), tk, float(scale), _addr(workspace),
                                            int(workspace.numel()), stream)
    _raise("latent_attention_prefill_chunk", rc)
    return workspace
