"""Key-priority mixed-precision KV-cache quantization and decode attention for B200.

Thin ctypes binding over ``libkvq.so`` (the C ABI in ``include/kvq.h``).  The
functions keep the C names; arguments are marshalled from torch tensors
(device pointers) and the current CUDA stream.  Every step of the computation
runs in the library's CUDA kernels; there is no fallback: if the library is
missing, every call raises.

Typical use::

    cache = KVCache.allocate(batch, kv_heads, head_dim, capacity,
                             bits_k=4, bits_v=2, group=64, device="cuda")
    kvq_quantize_append(cache, k, v, pos)            # k, v: [B][Hkv][n][D]
    out = kvq_decode_attention(cache, q, seq_lens, max_seq_len)   # q: [B][Hq][D]
    # or both in one launch, the new rows at seq_lens - n .. seq_lens - 1:
    out = kvq_append_decode_attention(cache, k, v, q, seq_lens, max_seq_len)

A serving step whose rows bring different numbers of new tokens (prefill
chunks, draft tokens, single tokens), packed one after another::

    lens, cu, slots = kvq_plan_append(cache, old_lens, new_lens, k.shape[0], page_users)
    # then, for every layer:
    kvq_quantize_append_ragged(cache, k, v, slots)                # k, v: [T][Hkv][D]
    out = kvq_chunk_attention(cache, q, cu, lens, max_q, max_len)  # q: [T][Hq][D]

A paged cache (block tables) is allocated with ``page_size``, ``num_pages``
and an int32 ``block_table`` [batch][capacity / page_size].

With ``stream=`` a call runs on that stream: its results and workspace are
memory of that stream, and its arguments may be dropped right after the call.
Ordering it after the work that produces the arguments, and the reader of its
results after it, is up to the caller, as with any two streams.
"""
from __future__ import annotations

import ctypes
import dataclasses
import os
from typing import Optional

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIBRARY_PATH = os.path.join(_HERE, "libkvq.so")

KVQ_F32, KVQ_BF16, KVQ_F16 = 0, 1, 2
KVQ_OK, KVQ_ERR_INVALID_ARG, KVQ_ERR_UNSUPPORTED, KVQ_ERR_WORKSPACE, KVQ_ERR_CUDA = range(5)
KVQ_DEVERR_CAPACITY, KVQ_DEVERR_SEQ_LEN, KVQ_DEVERR_TIMEOUT, KVQ_DEVERR_BAD_POS = 1, 2, 4, 8
KVQ_DEVERR_BAD_PAGE, KVQ_DEVERR_NO_PAGE = 16, 32
KVQ_K_CODES, KVQ_V_CODES, KVQ_K_PARAMS, KVQ_V_PARAMS = range(4)
KVQ_FLAG_ROTATE_KEYS, KVQ_FLAG_PAGED = 1, 2

_DTYPE = {torch.float32: KVQ_F32, torch.bfloat16: KVQ_BF16, torch.float16: KVQ_F16}


class KvqError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {kvq_strerror(status)} (status {status})")
        self.status = status


class KvqCacheDesc(ctypes.Structure):
    _fields_ = [
        ("batch", ctypes.c_int32), ("kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32), ("capacity", ctypes.c_int32),
        ("bits_k", ctypes.c_int32), ("bits_v", ctypes.c_int32),
        ("group", ctypes.c_int32), ("flags", ctypes.c_int32),
        ("group_v", ctypes.c_int32), ("reserved", ctypes.c_int32),
        ("k_codes", ctypes.c_void_p), ("v_codes", ctypes.c_void_p),
        ("k_params", ctypes.c_void_p), ("v_params", ctypes.c_void_p),
        ("page_size", ctypes.c_int32), ("num_pages", ctypes.c_int32),
        ("block_table", ctypes.c_void_p),
    ]


_lib = None


def library() -> ctypes.CDLL:
    """The loaded libkvq.so; raises if it was not built."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIBRARY_PATH):
        raise RuntimeError(
            f"{LIBRARY_PATH} is missing: build it with `python -m kv_cache_mixed_kvq_b200.build`")
    lib = ctypes.CDLL(LIBRARY_PATH)
    P, I32, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_size_t
    D = ctypes.POINTER(KvqCacheDesc)
    lib.kvq_cache_bytes.argtypes = [I32] * 8
    lib.kvq_cache_bytes.restype = SZ
    lib.kvq_validate_cache.argtypes = [D]
    lib.kvq_validate_cache.restype = ctypes.c_int
    lib.kvq_quantize_append.argtypes = [D, P, P, I32, P, I32, P]
    lib.kvq_quantize_append.restype = ctypes.c_int
    lib.kvq_decode_workspace_bytes.argtypes = [D, I32, I32]
    lib.kvq_decode_workspace_bytes.restype = SZ
    lib.kvq_decode_split_tokens.argtypes = [D, I32, I32]
    lib.kvq_decode_split_tokens.restype = I32
    lib.kvq_decode_attention.argtypes = [D, P, I32, I32, P, I32, ctypes.c_float, P, I32, P, SZ, P]
    lib.kvq_decode_attention.restype = ctypes.c_int
    lib.kvq_append_decode_attention.argtypes = [D, P, P, I32, I32, P, I32, I32, P, I32,
                                                ctypes.c_float, P, I32, P, SZ, P]
    lib.kvq_append_decode_attention.restype = ctypes.c_int
    I64 = ctypes.c_int64
    lib.kvq_slot_map_entries.argtypes = [I32, I32]
    lib.kvq_slot_map_entries.restype = I32
    lib.kvq_plan_append.argtypes = [D, P, P, I32, P, P, P, P, I32, P]
    lib.kvq_plan_append.restype = ctypes.c_int
    lib.kvq_quantize_append_ragged.argtypes = [D, P, I64, P, I64, I32, I32, P, I32, P]
    lib.kvq_quantize_append_ragged.restype = ctypes.c_int
    lib.kvq_dequantize_ragged.argtypes = [D, P, I32, P, P, I32, I32, P]
    lib.kvq_dequantize_ragged.restype = ctypes.c_int
    lib.kvq_chunk_workspace_bytes.argtypes = [D, I32, I32, I32, I32]
    lib.kvq_chunk_workspace_bytes.restype = SZ
    lib.kvq_chunk_attention.argtypes = [D, P, I64, I32, I32, I32, P, P, I32, I32, I32,
                                        ctypes.c_float, P, I32, P, SZ, P]
    lib.kvq_chunk_attention.restype = ctypes.c_int
    lib.kvq_device_error_flags.argtypes = [P, ctypes.POINTER(ctypes.c_uint32)]
    lib.kvq_device_error_flags.restype = ctypes.c_int
    lib.kvq_last_device_error.argtypes = [P]
    lib.kvq_last_device_error.restype = ctypes.c_int
    lib.kvq_debug_inject_wait_timeout.argtypes = [I32, ctypes.c_int64]
    lib.kvq_debug_inject_wait_timeout.restype = ctypes.c_int
    lib.kvq_strerror.argtypes = [I32]
    lib.kvq_strerror.restype = ctypes.c_char_p
    _lib = lib
    return lib


def _stream_ptr(stream: Optional[torch.cuda.Stream]) -> int:
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _empty(shape, dtype: torch.dtype, device: torch.device,
           stream: Optional[torch.cuda.Stream], kept: bool = True) -> torch.Tensor:
    """Memory of the call's own.  It is taken on the stream that the call runs
    on: another stream's free memory may still be in use there, and what the
    call drops could be given out again while its kernels use it.  A result
    (kept) is also marked as used by the caller's stream, which will read it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        t = torch.empty(shape, dtype=dtype, device=device)
    if kept:
        t.record_stream(torch.cuda.current_stream(device))
    return t


def _used_on(stream: torch.cuda.Stream, *tensors: Optional[torch.Tensor]) -> None:
    """Marks tensors of other streams as used by the call's, so that their
    memory is not given out again before the call is done with it."""
    for t in tensors:
        if t is not None:
            t.record_stream(stream)


def _dev_ptr(t: torch.Tensor, name: str) -> int:
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _check(status: int, what: str) -> None:
    if status != KVQ_OK:
        raise KvqError(status, what)


# ------------------------------------------------------------- C-named calls
def kvq_strerror(status: int) -> str:
    return library().kvq_strerror(int(status)).decode()


def kvq_cache_bytes(batch, kv_heads, head_dim, capacity, bits_k, bits_v, group, which) -> int:
    return int(library().kvq_cache_bytes(batch, kv_heads, head_dim, capacity, bits_k, bits_v,
                                         group, which))


@dataclasses.dataclass
class KVCache:
    """One layer's packed cache: four caller-owned device buffers + shape."""
    batch: int
    kv_heads: int
    head_dim: int
    capacity: int
    bits_k: int
    bits_v: int
    group: int
    k_codes: torch.Tensor
    v_codes: torch.Tensor
    k_params: torch.Tensor
    v_params: torch.Tensor
    rotate_keys: bool = False  # KVQ_FLAG_ROTATE_KEYS: keys stored as H k
    group_v: int = 0           # values' group size (0: same as group)
    # KVQ_FLAG_PAGED: a pool of num_pages pages of page_size positions and an
    # int32 block table [batch][capacity / page_size] (device); 0 / None: slots
    page_size: int = 0
    num_pages: int = 0
    block_table: Optional[torch.Tensor] = None

    @classmethod
    def allocate(cls, batch, kv_heads, head_dim, capacity, bits_k, bits_v, group,
                 device="cuda", rotate_keys: bool = False, group_v: int = 0,
                 page_size: int = 0, num_pages: int = 0,
                 block_table: Optional[torch.Tensor] = None) -> "KVCache":
        """Zeroed buffers.  With page_size > 0 the cache is paged: a pool of
        num_pages pages and the given block table (int32 [batch][capacity /
        page_size], moved to `device`)."""
        gv = group_v or group
        rows, length = (num_pages, page_size) if page_size else (batch, capacity)
        sizes = [kvq_cache_bytes(rows, kv_heads, head_dim, length, bits_k, bits_v,
                                 gv if w == KVQ_V_PARAMS else group, w) for w in range(4)]
        if 0 in sizes:
            raise KvqError(KVQ_ERR_INVALID_ARG, "KVCache.allocate")
        if page_size:
            if block_table is None or capacity % page_size:
                raise KvqError(KVQ_ERR_INVALID_ARG, "KVCache.allocate (paged)")
            block_table = block_table.to(device=device, dtype=torch.int32).contiguous()
            if tuple(block_table.shape) != (batch, capacity // page_size):
                raise KvqError(KVQ_ERR_INVALID_ARG, "KVCache.allocate (block table shape)")
        bufs = [torch.zeros(n, dtype=torch.uint8, device=device) for n in sizes]
        return cls(batch, kv_heads, head_dim, capacity, bits_k, bits_v, group, *bufs,
                   rotate_keys=rotate_keys, group_v=group_v, page_size=page_size,
                   num_pages=num_pages if page_size else 0,
                   block_table=block_table if page_size else None)

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        self.__dict__.pop("_desc", None)

    def __getstate__(self):  # (copies and pickles build their own descriptor)
        return {k: v for k, v in self.__dict__.items() if k != "_desc"}

    def desc(self) -> KvqCacheDesc:
        """The C descriptor: a structure of the caller's own."""
        return KvqCacheDesc.from_buffer_copy(self._kept_desc())

    def _kept_desc(self) -> KvqCacheDesc:
        """The descriptor that the calls share; built and checked again when a
        field, or a buffer's address or layout, has changed since the last one."""
        k, v, kp, vp, bt = (self.k_codes, self.v_codes, self.k_params, self.v_params,
                            self.block_table)
        at = (k.data_ptr(), v.data_ptr(), kp.data_ptr(), vp.data_ptr(), k.is_contiguous(),
              v.is_contiguous(), kp.is_contiguous(), vp.is_contiguous(),
              bt is not None and (bt.data_ptr(), bt.is_contiguous()))
        kept = self.__dict__.get("_desc")
        if kept is None or kept[0] != at:
            kept = (at, self._build_desc())
            self.__dict__["_desc"] = kept
        return kept[1]

    def _buffers(self):
        """The cache's tensors (without pages the last one is None)."""
        return self.k_codes, self.v_codes, self.k_params, self.v_params, self.block_table

    def _build_desc(self) -> KvqCacheDesc:
        flags = (KVQ_FLAG_ROTATE_KEYS if self.rotate_keys else 0) | \
            (KVQ_FLAG_PAGED if self.page_size else 0)
        if any(t is not None and t.device != self.k_codes.device for t in self._buffers()):
            raise ValueError("the cache's buffers must be on one device")
        bt = _dev_ptr(self.block_table, "block_table") if self.block_table is not None else None
        return KvqCacheDesc(self.batch, self.kv_heads, self.head_dim, self.capacity,
                            self.bits_k, self.bits_v, self.group, flags, self.group_v, 0,
                            _dev_ptr(self.k_codes, "k_codes"), _dev_ptr(self.v_codes, "v_codes"),
                            _dev_ptr(self.k_params, "k_params"), _dev_ptr(self.v_params, "v_params"),
                            self.page_size, self.num_pages, bt)


def kvq_validate_cache(cache: KVCache) -> int:
    d = cache._kept_desc()
    return int(library().kvq_validate_cache(ctypes.byref(d)))


def kvq_quantize_append(cache: KVCache, k: torch.Tensor, v: torch.Tensor, pos: torch.Tensor,
                        stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantize k, v ([B][Hkv][n_new][D]) into positions pos[b] .. pos[b]+n_new-1."""
    if k.dtype != v.dtype or k.shape != v.shape or k.dim() != 4:
        raise ValueError("k and v must be [B][Hkv][n_new][D] tensors of one dtype")
    if pos.dtype != torch.int32:
        raise ValueError("pos must be int32")
    d = cache._kept_desc()
    st = library().kvq_quantize_append(ctypes.byref(d), _dev_ptr(k, "k"), _dev_ptr(v, "v"),
                                       _DTYPE[k.dtype], _dev_ptr(pos, "pos"), k.shape[2],
                                       _stream_ptr(stream))
    _check(st, "kvq_quantize_append")
    if stream is not None:
        _used_on(stream, k, v, pos, *cache._buffers())


def kvq_decode_workspace_bytes(cache: KVCache, num_q_heads: int, max_seq_len: int) -> int:
    d = cache._kept_desc()
    return int(library().kvq_decode_workspace_bytes(ctypes.byref(d), num_q_heads, max_seq_len))


def kvq_decode_split_tokens(cache: KVCache, num_q_heads: int, max_seq_len: int) -> int:
    d = cache._kept_desc()
    return int(library().kvq_decode_split_tokens(ctypes.byref(d), num_q_heads, max_seq_len))


def kvq_decode_attention(cache: KVCache, q: torch.Tensor, seq_lens: torch.Tensor,
                         max_seq_len: int, sm_scale: float = 0.0,
                         out: Optional[torch.Tensor] = None,
                         out_dtype: Optional[torch.dtype] = None,
                         workspace: Optional[torch.Tensor] = None,
                         stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of q ([B][Hq][D]) over positions [0, seq_lens[b]) of the cache."""
    if q.dim() != 3:
        raise ValueError("q must be [B][Hq][D]")
    if seq_lens.dtype != torch.int32:
        raise ValueError("seq_lens must be int32")
    if out is None:
        out = _empty(q.shape, out_dtype or q.dtype, q.device, stream)
    d = cache._kept_desc()
    lib = library()
    if workspace is None:  # (a given workspace is checked by the library itself)
        need = int(lib.kvq_decode_workspace_bytes(ctypes.byref(d), q.shape[1], max_seq_len))
        if need > 0:
            workspace = _empty(need, torch.uint8, q.device, stream, kept=False)
    ws_ptr = _dev_ptr(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.kvq_decode_attention(ctypes.byref(d), _dev_ptr(q, "q"), _DTYPE[q.dtype], q.shape[1],
                                  _dev_ptr(seq_lens, "seq_lens"), int(max_seq_len),
                                  float(sm_scale), _dev_ptr(out, "out"), _DTYPE[out.dtype],
                                  ws_ptr, ws_bytes, _stream_ptr(stream))
    _check(st, "kvq_decode_attention")
    if stream is not None:
        _used_on(stream, q, seq_lens, out, workspace, *cache._buffers())
    return out


def kvq_append_decode_attention(cache: KVCache, k_new: torch.Tensor, v_new: torch.Tensor,
                                q: torch.Tensor, seq_lens: torch.Tensor, max_seq_len: int,
                                sm_scale: float = 0.0, out: Optional[torch.Tensor] = None,
                                out_dtype: Optional[torch.dtype] = None,
                                workspace: Optional[torch.Tensor] = None,
                                stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Append k_new, v_new ([B][Hkv][n_new][D]) at positions seq_lens[b] - n_new ..
    seq_lens[b] - 1, then attend q ([B][Hq][D]) to [0, seq_lens[b]): one fused call."""
    if k_new.dtype != v_new.dtype or k_new.shape != v_new.shape or k_new.dim() != 4:
        raise ValueError("k_new and v_new must be [B][Hkv][n_new][D] tensors of one dtype")
    if q.dim() != 3:
        raise ValueError("q must be [B][Hq][D]")
    if seq_lens.dtype != torch.int32:
        raise ValueError("seq_lens must be int32")
    if out is None:
        out = _empty(q.shape, out_dtype or q.dtype, q.device, stream)
    d = cache._kept_desc()
    lib = library()
    if workspace is None:  # (a given workspace is checked by the library itself)
        need = int(lib.kvq_decode_workspace_bytes(ctypes.byref(d), q.shape[1], max_seq_len))
        if need > 0:
            workspace = _empty(need, torch.uint8, q.device, stream, kept=False)
    ws_ptr = _dev_ptr(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.kvq_append_decode_attention(
        ctypes.byref(d), _dev_ptr(k_new, "k_new"), _dev_ptr(v_new, "v_new"), _DTYPE[k_new.dtype],
        k_new.shape[2], _dev_ptr(q, "q"), _DTYPE[q.dtype], q.shape[1],
        _dev_ptr(seq_lens, "seq_lens"), int(max_seq_len), float(sm_scale), _dev_ptr(out, "out"),
        _DTYPE[out.dtype], ws_ptr, ws_bytes, _stream_ptr(stream))
    _check(st, "kvq_append_decode_attention")
    if stream is not None:
        _used_on(stream, k_new, v_new, q, seq_lens, out, workspace, *cache._buffers())
    return out


# ------------------------------------------- a serving step over a ragged batch
def _on_current(device: torch.device) -> None:
    """The library launches on the current device: its tensors must be there."""
    if device.type != "cuda":
        raise ValueError("the cache must be on a CUDA device")
    if device.index != torch._C._cuda_getDevice():
        raise ValueError(f"the cache is on {device}, the current device is "
                         f"cuda:{torch.cuda.current_device()}")


def _int32(t: torch.Tensor, numel: int, name: str, device: torch.device) -> int:
    """Data pointer of a contiguous int32 tensor of `numel` elements."""
    if t.dtype != torch.int32 or t.numel() != numel:
        raise ValueError(f"{name} must be an int32 tensor of {numel} elements")
    if t.device != device:
        raise ValueError(f"{name} must be on the cache's device")
    return _dev_ptr(t, name)


def _tokens(t: torch.Tensor, heads: Optional[int], D: int, name: str, device: torch.device):
    """(data pointer, elements from token to token) of packed tokens [T][heads][D];
    a slice along the heads of a larger packed tensor is accepted."""
    shape = t.shape
    if len(shape) != 3 or shape[2] != D or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [tokens][{heads or 'heads'}][{D}]")
    if t.dtype not in _DTYPE:
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    if t.device != device:
        raise ValueError(f"{name} must be on the cache's device")
    T, H, _ = shape
    if T == 0:
        return None, H * D
    strides = t.stride()
    stride = strides[0] if T > 1 else H * D
    if (strides[2] != 1 and D > 1) or (strides[1] != D and H > 1) or stride < H * D or \
            stride * t.element_size() % 16:
        raise ValueError(f"{name}: the heads of a token must be contiguous and tokens "
                         "a multiple of 16 bytes apart")
    return t.data_ptr(), stride


def _slots(slot_map: torch.Tensor, device: torch.device):
    if slot_map.dim() != 2 or slot_map.shape[1] != 4:
        raise ValueError("slot_map must be [entries][4]")
    return _int32(slot_map, slot_map.numel(), "slot_map", device)


def kvq_slot_map_entries(batch: int, num_tokens: int) -> int:
    """Entries of a slot map for num_tokens packed tokens in batch rows, at most."""
    return int(library().kvq_slot_map_entries(batch, num_tokens))


def kvq_plan_append(cache: KVCache, old_lens: torch.Tensor, new_lens: torch.Tensor,
                    num_tokens: int, page_users: Optional[torch.Tensor] = None,
                    stream: Optional[torch.cuda.Stream] = None):
    """Plan one ragged step: (lens, cu_tokens, slot_map) for rows that go from
    old_lens to new_lens with num_tokens new tokens in all (or more).

    A paged cache's block_table and page_users (int32 [num_pages], users of
    each page) are updated in place: growing rows take free pages, shrinking
    rows return theirs.  A row that gets no page keeps its old length in lens
    and flags KVQ_DEVERR_NO_PAGE."""
    device = cache.k_codes.device
    _on_current(device)
    B = cache.batch
    old, new = _int32(old_lens, B, "old_lens", device), _int32(new_lens, B, "new_lens", device)
    if cache.page_size:
        if page_users is None:
            raise ValueError("a paged cache needs page_users")
        users = _int32(page_users, cache.num_pages, "page_users", device)
    else:
        if page_users is not None:
            raise ValueError("page_users is for paged caches")
        users = None
    lib = library()
    E = lib.kvq_slot_map_entries(B, num_tokens)
    # (one allocation: three took half of the call's host time)
    results = _empty(4 * E + 2 * B + 1, torch.int32, device, stream)
    at = results.data_ptr()
    slot_map, lens, cu = results.split_with_sizes((4 * E, B, B + 1))
    slot_map = slot_map.view(E, 4)
    d = cache._kept_desc()
    st = lib.kvq_plan_append(ctypes.byref(d), old, new, num_tokens, users, at + 16 * E,
                             at + 16 * E + 4 * B, at if E else None, E,
                             _stream_ptr(stream))
    _check(st, "kvq_plan_append")
    if stream is not None:
        _used_on(stream, old_lens, new_lens, page_users, cache.block_table)
    return lens, cu, slot_map


def kvq_quantize_append_ragged(cache: KVCache, k: torch.Tensor, v: torch.Tensor,
                               slot_map: torch.Tensor,
                               stream: Optional[torch.cuda.Stream] = None) -> None:
    """Quantize packed tokens k, v ([T][Hkv][D]) into the places of a slot map."""
    device = cache.k_codes.device
    _on_current(device)
    if k.dtype != v.dtype or k.shape != v.shape:
        raise ValueError("k and v must be tensors of one shape and dtype")
    kp, ks = _tokens(k, cache.kv_heads, cache.head_dim, "k", device)
    vp, vs = _tokens(v, cache.kv_heads, cache.head_dim, "v", device)
    sp = _slots(slot_map, device)
    d = cache._kept_desc()
    st = library().kvq_quantize_append_ragged(ctypes.byref(d), kp, ks, vp, vs, _DTYPE[k.dtype],
                                              k.shape[0], sp, slot_map.shape[0],
                                              _stream_ptr(stream))
    _check(st, "kvq_quantize_append_ragged")
    if stream is not None:
        _used_on(stream, k, v, slot_map, *cache._buffers())


def kvq_dequantize_ragged(cache: KVCache, slot_map: torch.Tensor, num_tokens: int,
                          dtype: torch.dtype = torch.bfloat16,
                          k_out: Optional[torch.Tensor] = None,
                          v_out: Optional[torch.Tensor] = None,
                          stream: Optional[torch.cuda.Stream] = None):
    """(k, v) [num_tokens][Hkv][D] that the cache holds at the places of a slot
    map, as dtype (or into k_out, v_out, contiguous and of one dtype).  Tokens
    that no entry names are not written."""
    device = cache.k_codes.device
    _on_current(device)
    shape = (num_tokens, cache.kv_heads, cache.head_dim)
    if (k_out is None) != (v_out is None):
        raise ValueError("give both of k_out and v_out, or neither")
    if k_out is None:
        if dtype not in _DTYPE:
            raise ValueError("dtype must be float32, bfloat16 or float16")
        k_out = _empty(shape, dtype, device, stream)
        v_out = _empty(shape, dtype, device, stream)
    else:
        for t, name in ((k_out, "k_out"), (v_out, "v_out")):
            if tuple(t.shape) != shape or t.dtype not in _DTYPE or t.dtype != k_out.dtype or \
                    t.device != device:
                raise ValueError(f"{name} must be {list(shape)}, on the cache's device, of one "
                                 "dtype")
    sp = _slots(slot_map, device)
    d = cache._kept_desc()
    st = library().kvq_dequantize_ragged(ctypes.byref(d), sp, slot_map.shape[0],
                                         _dev_ptr(k_out, "k_out"), _dev_ptr(v_out, "v_out"),
                                         _DTYPE[k_out.dtype], num_tokens, _stream_ptr(stream))
    _check(st, "kvq_dequantize_ragged")
    if stream is not None:
        _used_on(stream, slot_map, k_out, v_out, *cache._buffers())
    return k_out, v_out


def kvq_chunk_workspace_bytes(cache: KVCache, num_q_heads: int, num_tokens: int, max_q_len: int,
                              max_seq_len: int) -> int:
    d = cache._kept_desc()
    return int(library().kvq_chunk_workspace_bytes(ctypes.byref(d), num_q_heads, num_tokens,
                                                   max_q_len, max_seq_len))


def kvq_chunk_attention(cache: KVCache, q: torch.Tensor, cu_tokens: torch.Tensor,
                        seq_lens: torch.Tensor, max_q_len: int, max_seq_len: int,
                        causal: bool = True, sm_scale: float = 0.0,
                        out: Optional[torch.Tensor] = None,
                        out_dtype: Optional[torch.dtype] = None,
                        workspace: Optional[torch.Tensor] = None,
                        stream: Optional[torch.cuda.Stream] = None) -> torch.Tensor:
    """Attention of packed queries q ([T][Hq][D]) over the cache, which holds
    their tokens already: query i of row b's n_b = cu_tokens[b+1] - cu_tokens[b]
    attends to positions [0, seq_lens[b] - n_b + i] (causal) or [0, seq_lens[b])."""
    device = cache.k_codes.device
    _on_current(device)
    qp, qs = _tokens(q, None, cache.head_dim, "q", device)
    T, Hq, D = q.shape
    cu = _int32(cu_tokens, cache.batch + 1, "cu_tokens", device)
    lens = _int32(seq_lens, cache.batch, "seq_lens", device)
    if out is None:
        out = _empty((T, Hq, D), out_dtype or q.dtype, device, stream)
    elif out.shape != q.shape or out.dtype not in _DTYPE or out.device != device:
        raise ValueError("out must be of q's shape, on the cache's device")
    d = cache._kept_desc()
    lib = library()
    if workspace is None:  # (a given workspace is checked by the library itself)
        need = lib.kvq_chunk_workspace_bytes(ctypes.byref(d), Hq, T, max_q_len, max_seq_len)
        if need > 0:
            workspace = _empty(need, torch.uint8, device, stream, kept=False)
    elif workspace.device != device:
        raise ValueError("workspace must be on the cache's device")
    ws_ptr = _dev_ptr(workspace, "workspace") if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    st = lib.kvq_chunk_attention(ctypes.byref(d), qp, qs, _DTYPE[q.dtype], Hq, T, cu, lens,
                                 max_q_len, max_seq_len, 1 if causal else 0, sm_scale,
                                 _dev_ptr(out, "out"), _DTYPE[out.dtype], ws_ptr, ws_bytes,
                                 _stream_ptr(stream))
    _check(st, "kvq_chunk_attention")
    if stream is not None:
        _used_on(stream, q, cu_tokens, seq_lens, out, workspace, *cache._buffers())
    return out


def kvq_debug_inject_wait_timeout(drop_stage: int, wait_limit_ns: int = 1_000_000) -> None:
    """Test knob: in the next decode or chunk launch, stage drop_stage (0 or 1) of the
    first warp's copy pipeline expects more bytes than its copies bring, so
    that a bounded wait runs out (see kvq.h); drop_stage < 0 disarms it."""
    _check(library().kvq_debug_inject_wait_timeout(int(drop_stage), int(wait_limit_ns)),
           "kvq_debug_inject_wait_timeout")


def kvq_device_error_flags(stream: Optional[torch.cuda.Stream] = None) -> int:
    flags = ctypes.c_uint32(0)
    st = library().kvq_device_error_flags(_stream_ptr(stream), ctypes.byref(flags))
    _check(st, "kvq_device_error_flags")
    return int(flags.value)


def kvq_last_device_error(stream: Optional[torch.cuda.Stream] = None) -> int:
    """Error-word bits (read and cleared); raises KvqError on a CUDA failure."""
    r = library().kvq_last_device_error(_stream_ptr(stream))
    if r < 0:
        _check(-r, "kvq_last_device_error")
    return int(r)
