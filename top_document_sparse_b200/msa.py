"""ctypes binding of libmsa.so (C ABI in include/msa.h).

Argument marshalling only: tensors become device pointers, streams become cudaStream_t handles,
statuses become exceptions.  Every step of the hot path runs in the library's CUDA kernels; there
is no CPU fallback, and importing this module fails loudly when the library cannot be loaded.
"""
from __future__ import annotations

import ctypes
import os

import numpy as np
import torch

from . import build as _build

_HERE = os.path.dirname(os.path.abspath(__file__))

MSA_F32, MSA_BF16 = 0, 1
DEVERR_BAD_DOC_ID, DEVERR_CACHE_OVERFLOW, DEVERR_WAIT_TIMEOUT = 0x1, 0x2, 0x4
DEVERR_BAD_LENGTH = 0x8
STATUS = {0: "MSA_OK", 1: "MSA_ERR_INVALID_ARG", 2: "MSA_ERR_UNSUPPORTED", 3: "MSA_ERR_CUDA",
          4: "MSA_ERR_OUT_OF_MEMORY", 5: "MSA_ERR_TIMEOUT", 6: "MSA_ERR_STATE"}
_DTYPE = {torch.float32: MSA_F32, torch.bfloat16: MSA_BF16}
_TORCH = {MSA_F32: torch.float32, MSA_BF16: torch.bfloat16}


class MsaError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"{STATUS.get(status, status)}: {message}")
        self.status = status


class MemoryConfig(ctypes.Structure):
    _fields_ = [("n_docs", ctypes.c_int32), ("doc_token_offsets", ctypes.POINTER(ctypes.c_int64)),
                ("chunk_len", ctypes.c_int32), ("n_kv_heads", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("n_router_heads", ctypes.c_int32),
                ("router_dim", ctypes.c_int32), ("dtype", ctypes.c_int),
                ("rope_theta", ctypes.c_double), ("max_local_position", ctypes.c_int32)]


class MemoryInfo(ctypes.Structure):
    _fields_ = [("n_tokens", ctypes.c_int64), ("n_chunks", ctypes.c_int64),
                ("max_doc_chunks", ctypes.c_int32), ("max_doc_tokens", ctypes.c_int64),
                ("elem_bytes", ctypes.c_size_t), ("router_key_bytes", ctypes.c_size_t),
                ("content_bytes", ctypes.c_size_t), ("doc_content_stride", ctypes.c_size_t)]


class DecodeState(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("top_k", ctypes.c_int32),
                ("n_q_heads", ctypes.c_int32), ("cache_capacity", ctypes.c_int32),
                ("pos_offset", ctypes.c_int32), ("state", ctypes.c_void_p),
                ("ids", ctypes.c_void_p), ("scores", ctypes.c_void_p),
                ("k_cache", ctypes.c_void_p), ("v_cache", ctypes.c_void_p),
                ("cache_len", ctypes.c_void_p), ("workspace", ctypes.c_void_p),
                ("workspace_bytes", ctypes.c_size_t)]


class RopeConfig(ctypes.Structure):
    _fields_ = [("head_dim", ctypes.c_int32), ("rotary_dim", ctypes.c_int32),
                ("theta", ctypes.c_double), ("layout", ctypes.c_int32),
                ("scaling", ctypes.c_int32), ("factor", ctypes.c_double),
                ("original_length", ctypes.c_int64), ("magnitude", ctypes.c_double)]


class Cache8Struct(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int32), ("capacity", ctypes.c_int32),
                ("block_len", ctypes.c_int32), ("format", ctypes.c_int32),
                ("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("cache_len", ctypes.c_void_p),
                ("weights", ctypes.c_void_p)]


_P = ctypes.c_void_p
_I32 = ctypes.c_int32
_I64 = ctypes.c_int64
_SZ = ctypes.c_size_t

# name -> (restype, argtypes); must match include/msa.h
SIGNATURES = {
    "msa_memory_create": (ctypes.c_int, [ctypes.POINTER(MemoryConfig), ctypes.POINTER(_P)]),
    "msa_memory_destroy": (ctypes.c_int, [_P]),
    "msa_memory_get_info": (ctypes.c_int, [_P, ctypes.POINTER(MemoryInfo)]),
    "msa_memory_doc_chunk_offsets": (ctypes.c_int, [_P, ctypes.POINTER(ctypes.c_int64)]),
    "msa_encode_memory": (ctypes.c_int, [_P, _I32, _I32, _P, _P, _P, _P, _P, _P, _P]),
    "msa_route_reset": (ctypes.c_int, [_P, _I64, _P]),
    "msa_route_workspace_size": (_SZ, [_P, _I32, _I32, _I32]),
    "msa_route": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _P, _P, _P, _P, _P, _SZ, _P]),
    "msa_attend_workspace_size": (_SZ, [_P, _I32, _I32, _I32, _I32]),
    "msa_sparse_attend": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P,
                                         _P, _I32, _I32, _P, _P, _SZ, _P]),
    "msa_sparse_attend_static": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _P,
                                                _P, _P, _P, _I32, _I32, _P, _P]),
    "msa_step_workspace_size": (_SZ, [_P, _I32, _I32, _I32]),
    "msa_step": (ctypes.c_int, [_P, _P, _P, ctypes.POINTER(DecodeState), _P, _P, _P, _P, _P, _P]),
    "msa_fetcher_create": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, ctypes.c_uint32,
                                          ctypes.POINTER(_P)]),
    "msa_fetcher_destroy": (ctypes.c_int, [_P]),
    "msa_fetcher_stats": (ctypes.c_int, [_P, ctypes.POINTER(_I64), ctypes.POINTER(_I64),
                                         ctypes.POINTER(_I64), ctypes.POINTER(_I64)]),
    "msa_fetch": (ctypes.c_int, [_P, _P, _I32, _I32, _P, _P]),
    "msa_sparse_attend_fetched": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _P,
                                                 _P, _P, _P, _I32, _I32, _P, _P, _SZ, _P]),
    "msa_step_host": (ctypes.c_int, [_P, _P, _P, ctypes.POINTER(DecodeState), _P, _P, _P, _P, _P,
                                     _P, _P]),
    "msa_interleave_workspace_size": (_SZ, [_P, _I32, _I32, _I32]),
    "msa_interleave": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _P, _SZ,
                                      _P]),
    "msa_interleave_adaptive": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _I32, ctypes.c_float,
                                               _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "msa_topk_merge": (ctypes.c_int, [_P, _P, _I32, _I32, _I32, ctypes.POINTER(_I32), _I32, _P,
                                      _P, _P]),
    "msa_route_backward": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _P, _P, _P, _P]),
    "msa_sparse_attend_backward": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _I32, _I32, _P, _P,
                                                  _P, _P, _I32, _I32, _P, _P, _P, _P, _P, _P]),
    "msa_rope_create": (ctypes.c_int, [ctypes.POINTER(RopeConfig), ctypes.POINTER(_P)]),
    "msa_rope_destroy": (ctypes.c_int, [_P]),
    "msa_rope_apply": (ctypes.c_int, [_P, ctypes.c_int, _I64, _P, _I32, _P, _I32, _I64, _P, _I64,
                                      _P, _I32, _I64, _P, _I64, _P]),
    "msa_cache8_append": (ctypes.c_int, [_P, _P, _P, _P, _I32, _I64, _I64, _I64, _I64, _P, _P,
                                         _P]),
    "msa_cache8_read": (ctypes.c_int, [_P, _P, _P, _I32, _P, _P, _P]),
    "msa_cache8_attend_workspace_size": (_SZ, [_P, _P, _I32, _I32, _I32]),
    "msa_cache8_attend": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _I32, _P, _P, _P, _P,
                                         ctypes.c_float, _P, _SZ, _P]),
    "msa_cache8_attend_fetched": (ctypes.c_int, [_P, _P, _P, _I32, _P, _I32, _I32, _P, _P, _P, _P,
                                                 ctypes.c_float, _P, _SZ, _P]),
    "msa_cache8_evict_workspace_size": (_SZ, [_P, _P]),
    "msa_cache8_evict": (ctypes.c_int, [_P, _P, _P, _I32, _I32, _P, _SZ, _P]),
    "msa_device_error": (ctypes.c_int, [ctypes.POINTER(ctypes.c_uint32), _P]),
    "msa_status_string": (ctypes.c_char_p, [ctypes.c_int]),
    "msa_last_error": (ctypes.c_char_p, []),
    "msa_version": (ctypes.c_int32, []),
    "msa_launch_count": (ctypes.c_uint64, []),
}


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load (building first when stale) libmsa.so; raises if it cannot be loaded."""
    if path is None:
        path = _build.LIB
        if _build.stale():
            _build.build()
    lib = ctypes.CDLL(path)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    return lib


_lib = load_library()


def lib() -> ctypes.CDLL:
    return _lib


def launch_count() -> int:
    """Kernels the library has enqueued (graph captures count once, at capture)."""
    return int(_lib.msa_launch_count())


def _check(status: int):
    if status != 0:
        raise MsaError(status, _lib.msa_last_error().decode())


def _ptr(t) -> int | None:
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor")
    if not t.is_contiguous():
        raise ValueError("tensors must be contiguous")
    return t.data_ptr()


def _stream(stream) -> int:
    if stream is None:
        stream = torch.cuda.current_stream()
    return stream.cuda_stream


def device_error(stream=None) -> int:
    """Read and clear the device error word (MSA_DEVERR_* bits)."""
    bits = ctypes.c_uint32(0)
    _lib.msa_device_error(ctypes.byref(bits), _stream(stream))
    return bits.value


class Memory:
    """One memory layout (documents, chunking, head shapes) and its device tables.

    Router keys and pooled content live in caller tensors: ``router_keys`` [C][H_r][d_r] and
    ``content`` [C][2][H_kv][D] (device, or pinned host for content)."""

    def __init__(self, doc_token_offsets, chunk_len: int, n_kv_heads: int, head_dim: int,
                 n_router_heads: int, router_dim: int, dtype: torch.dtype, rope_theta: float,
                 max_local_position: int):
        off = np.ascontiguousarray(np.asarray(doc_token_offsets, dtype=np.int64))
        self._off = off
        cfg = MemoryConfig(n_docs=off.size - 1,
                           doc_token_offsets=off.ctypes.data_as(ctypes.POINTER(ctypes.c_int64)),
                           chunk_len=chunk_len, n_kv_heads=n_kv_heads, head_dim=head_dim,
                           n_router_heads=n_router_heads, router_dim=router_dim,
                           dtype=_DTYPE[dtype], rope_theta=rope_theta,
                           max_local_position=max_local_position)
        h = _P()
        _check(_lib.msa_memory_create(ctypes.byref(cfg), ctypes.byref(h)))
        self.handle = h
        self.dtype = dtype
        self.n_docs = off.size - 1
        self.chunk_len, self.n_kv_heads, self.head_dim = chunk_len, n_kv_heads, head_dim
        self.n_router_heads, self.router_dim = n_router_heads, router_dim
        info = MemoryInfo()
        _check(_lib.msa_memory_get_info(h, ctypes.byref(info)))
        self.info = info
        self.n_chunks = info.n_chunks
        co = np.zeros(self.n_docs + 1, dtype=np.int64)
        _check(_lib.msa_memory_doc_chunk_offsets(h, co.ctypes.data_as(ctypes.POINTER(ctypes.c_int64))))
        self.doc_chunk_offsets = co

    def close(self):
        if getattr(self, "handle", None):
            _check(_lib.msa_memory_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- storage -----------------------------------------------------------------------------
    def new_router_keys(self, device="cuda") -> torch.Tensor:
        return torch.empty(self.n_chunks, self.n_router_heads, self.router_dim, dtype=self.dtype,
                           device=device)

    def new_content(self, device="cuda", pin_memory=False) -> torch.Tensor:
        t = torch.empty(self.n_chunks, 2, self.n_kv_heads, self.head_dim, dtype=self.dtype,
                        device=device, pin_memory=pin_memory)
        return t

    # -- calls -------------------------------------------------------------------------------
    def encode(self, doc_begin: int, doc_count: int, K, V, Kr, router_keys, content,
               router_mean=None, stream=None):
        _check(_lib.msa_encode_memory(self.handle, doc_begin, doc_count, _ptr(K), _ptr(V), _ptr(Kr),
                                      _ptr(router_keys), _ptr(content), _ptr(router_mean),
                                      _stream(stream)))

    def route_workspace_size(self, batch: int, tokens: int, k: int) -> int:
        return _lib.msa_route_workspace_size(self.handle, batch, tokens, k)

    def route(self, router_keys, Qr, k: int, state, ids, scores, workspace, exclude=None,
              stream=None):
        B = state.shape[0]
        T = Qr.shape[1] if Qr is not None else 0
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(_lib.msa_route(self.handle, _ptr(router_keys), _ptr(Qr), B, T, k, _ptr(exclude),
                              _ptr(state), _ptr(ids), _ptr(scores), _ptr(workspace), ws_bytes,
                              _stream(stream)))

    def attend_workspace_size(self, batch: int, tokens: int, k: int, n_q_heads: int) -> int:
        return _lib.msa_attend_workspace_size(self.handle, batch, tokens, k, n_q_heads)

    def sparse_attend(self, content, ids, Q, K_new, V_new, K_cache, V_cache, cache_len,
                      pos_offset: int, O, workspace, stream=None):
        B, T, H_q, _ = Q.shape
        k = ids.shape[1] if ids is not None else 0
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(_lib.msa_sparse_attend(self.handle, _ptr(content), _ptr(ids), B, k, T, H_q, _ptr(Q),
                                      _ptr(K_new), _ptr(V_new), _ptr(K_cache), _ptr(V_cache),
                                      _ptr(cache_len), K_cache.shape[1], pos_offset, _ptr(O),
                                      _ptr(workspace), ws_bytes, _stream(stream)))

    def sparse_attend_static(self, content, ids, Q, K_new, V_new, K_cache, V_cache, cache_len,
                             pos_offset: int, O, stream=None):
        """msa_sparse_attend without a workspace: scratch from the library's fixed array."""
        B, T, H_q, _ = Q.shape
        k = ids.shape[1] if ids is not None else 0
        _check(_lib.msa_sparse_attend_static(self.handle, _ptr(content), _ptr(ids), B, k, T, H_q,
                                             _ptr(Q), _ptr(K_new), _ptr(V_new), _ptr(K_cache),
                                             _ptr(V_cache), _ptr(cache_len), K_cache.shape[1],
                                             pos_offset, _ptr(O), _stream(stream)))

    def interleave(self, router_keys, Qr, k: int, rounds: int, stream=None):
        """Memory Interleave rounds (msa_interleave): returns (ids [rounds][B][k], scores,
        state [B][n_docs], taken [B][n_docs])."""
        B, T = Qr.shape[0], Qr.shape[1]
        dev = Qr.device
        state = torch.empty(B, self.n_docs, dtype=torch.float32, device=dev)
        taken = torch.empty(B, self.n_docs, dtype=torch.uint8, device=dev)
        ids = torch.empty(rounds, B, k, dtype=torch.int32, device=dev)
        scores = torch.empty(rounds, B, k, dtype=torch.float32, device=dev)
        ws = workspace(_lib.msa_interleave_workspace_size(self.handle, B, T, k), dev)
        _check(_lib.msa_interleave(self.handle, _ptr(router_keys), _ptr(Qr), B, T, k, rounds,
                                   _ptr(state), _ptr(taken), _ptr(ids), _ptr(scores), _ptr(ws),
                                   ws.numel(), _stream(stream)))
        return ids, scores, state, taken

    def interleave_adaptive(self, router_keys, Qr, k: int, max_rounds: int, stop_score: float,
                            stream=None):
        """Adaptive Memory Interleave (msa_interleave_adaptive): returns (ids [max_rounds][B][k],
        scores, state [B][n_docs], taken [B][n_docs], n_rounds [B])."""
        B, T = Qr.shape[0], Qr.shape[1]
        dev = Qr.device
        state = torch.empty(B, self.n_docs, dtype=torch.float32, device=dev)
        taken = torch.empty(B, self.n_docs, dtype=torch.uint8, device=dev)
        ids = torch.empty(max_rounds, B, k, dtype=torch.int32, device=dev)
        scores = torch.empty(max_rounds, B, k, dtype=torch.float32, device=dev)
        n_rounds = torch.empty(B, dtype=torch.int32, device=dev)
        ws = workspace(_lib.msa_interleave_workspace_size(self.handle, B, T, k), dev)
        _check(_lib.msa_interleave_adaptive(self.handle, _ptr(router_keys), _ptr(Qr), B, T, k,
                                            max_rounds, float(stop_score), _ptr(state),
                                            _ptr(taken), _ptr(ids), _ptr(scores), _ptr(n_rounds),
                                            _ptr(ws), ws.numel(), _stream(stream)))
        return ids, scores, state, taken, n_rounds

    def route_backward(self, router_mean, Qr, d_score, stream=None):
        """Gradients of sum(d_score * doc_score) of one routing call of Qr [B][T][H_r][d_r]
        (msa_route_backward): (d_Qr, d_router_mean), fp32."""
        B, T = Qr.shape[0], Qr.shape[1]
        dQr = torch.empty(Qr.shape, dtype=torch.float32, device=Qr.device)
        dM = torch.empty(router_mean.shape, dtype=torch.float32, device=Qr.device)
        _check(_lib.msa_route_backward(self.handle, _ptr(router_mean), _ptr(Qr), B, T,
                                       _ptr(d_score), _ptr(dQr), _ptr(dM), _stream(stream)))
        return dQr, dM

    def sparse_attend_backward(self, content, ids, Q, K_cache, V_cache, cache_len0,
                               pos_offset: int, dO, stream=None):
        """Gradients of sum(dO * O) of a msa_sparse_attend call (msa_sparse_attend_backward):
        (dQ, d_cache_k, d_cache_v, d_content), fp32."""
        B, T, H_q, _ = Q.shape
        k = ids.shape[1] if ids is not None else 0
        dev = Q.device
        dQ = torch.empty(Q.shape, dtype=torch.float32, device=dev)
        dKc = torch.empty(K_cache.shape, dtype=torch.float32, device=dev)
        dVc = torch.empty(V_cache.shape, dtype=torch.float32, device=dev)
        dC = torch.empty(content.shape, dtype=torch.float32, device=dev)
        _check(_lib.msa_sparse_attend_backward(
            self.handle, _ptr(content), _ptr(ids), B, k, T, H_q, _ptr(Q), _ptr(K_cache),
            _ptr(V_cache), _ptr(cache_len0), K_cache.shape[1], pos_offset, _ptr(dO), _ptr(dQ),
            _ptr(dKc), _ptr(dVc), _ptr(dC), _stream(stream)))
        return dQ, dKc, dVc, dC

    def step_workspace_size(self, batch: int, k: int, n_q_heads: int) -> int:
        return _lib.msa_step_workspace_size(self.handle, batch, k, n_q_heads)

    def step(self, router_keys, content, st: "LayerDecode", Qr_tok, Q_tok, K_tok, V_tok, O_tok,
             stream=None):
        _check(_lib.msa_step(self.handle, _ptr(router_keys), _ptr(content), ctypes.byref(st.c),
                             _ptr(Qr_tok), _ptr(Q_tok), _ptr(K_tok), _ptr(V_tok), _ptr(O_tok),
                             _stream(stream)))


FETCH_COLD = 0x1


class Fetcher:
    """Host tier of one layer's pooled content: pinned host content plus a device slot cache
    (msa_fetcher_*).  Owns neither buffer; keeps references so they outlive it."""

    def __init__(self, mem: Memory, content_host: torch.Tensor, n_slots: int, max_batch: int,
                 max_k: int, cold: bool = False, device="cuda"):
        if not content_host.is_pinned():
            raise ValueError("content_host must be pinned host memory")
        self.mem = mem
        self.content_host = content_host
        self.slot_cache = torch.empty(n_slots * mem.info.doc_content_stride, dtype=torch.uint8,
                                      device=device)
        h = _P()
        _check(_lib.msa_fetcher_create(mem.handle, content_host.data_ptr(),
                                       self.slot_cache.data_ptr(), n_slots, max_batch, max_k,
                                       FETCH_COLD if cold else 0, ctypes.byref(h)))
        self.handle = h

    def close(self):
        if getattr(self, "handle", None):
            _check(_lib.msa_fetcher_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def stats(self) -> dict:
        v = [_I64() for _ in range(4)]
        _check(_lib.msa_fetcher_stats(self.handle, *[ctypes.byref(x) for x in v]))
        return dict(zip(("hits", "misses", "copies", "bytes"), (x.value for x in v)))

    def fetch(self, ids, stream=None, fetch_stream=None):
        B, k = ids.shape
        _check(_lib.msa_fetch(self.handle, _ptr(ids), B, k, _stream(stream),
                              _stream(fetch_stream) if fetch_stream is not None else _stream(stream)))

    def sparse_attend(self, ids, Q, K_new, V_new, K_cache, V_cache, cache_len, pos_offset: int,
                      O, workspace, stream=None):
        B, T, H_q, _ = Q.shape
        k = ids.shape[1]
        ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
        _check(_lib.msa_sparse_attend_fetched(self.mem.handle, self.handle, _ptr(ids), B, k, T, H_q,
                                              _ptr(Q), _ptr(K_new), _ptr(V_new), _ptr(K_cache),
                                              _ptr(V_cache), _ptr(cache_len), K_cache.shape[1],
                                              pos_offset, _ptr(O), _ptr(workspace), ws_bytes,
                                              _stream(stream)))

    def step(self, router_keys, st: "LayerDecode", Qr_tok, Q_tok, K_tok, V_tok, O_tok,
             stream=None, fetch_stream=None):
        _check(_lib.msa_step_host(self.mem.handle, _ptr(router_keys), self.handle,
                                  ctypes.byref(st.c), _ptr(Qr_tok), _ptr(Q_tok), _ptr(K_tok),
                                  _ptr(V_tok), _ptr(O_tok), _stream(stream),
                                  _stream(fetch_stream) if fetch_stream is not None
                                  else _stream(stream)))


def topk_merge(cand_scores, cand_ids, shard_doc_base, k: int, stream=None):
    """Global top-k from every memory shard's candidates (msa_topk_merge).

    cand_scores / cand_ids: device [n_shards][B][k_cand] (each shard's msa_route output, ids
    local to the shard); shard_doc_base: the global id of each shard's document 0.  Returns
    (ids [B][k] global, scores [B][k])."""
    n_shards, B, kc = cand_ids.shape
    base = (ctypes.c_int32 * n_shards)(*[int(x) for x in shard_doc_base])
    ids = torch.empty(B, k, dtype=torch.int32, device=cand_ids.device)
    scores = torch.empty(B, k, dtype=torch.float32, device=cand_ids.device)
    _check(_lib.msa_topk_merge(_ptr(cand_scores), _ptr(cand_ids), n_shards, B, kc, base, k,
                               _ptr(ids), _ptr(scores), _stream(stream)))
    return ids, scores


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


class LayerDecode:
    """Per-layer decode buffers (all torch-allocated) bundled as an msa_decode_state."""

    def __init__(self, mem: Memory, batch: int, k: int, n_q_heads: int, cache_capacity: int,
                 pos_offset: int | None = None, device="cuda", cache_len=None):
        self.state = torch.full((batch, mem.n_docs), float("-inf"), dtype=torch.float32,
                                device=device)
        self.ids = torch.zeros(batch, k, dtype=torch.int32, device=device)
        self.scores = torch.zeros(batch, k, dtype=torch.float32, device=device)
        self.k_cache = torch.zeros(batch, cache_capacity, mem.n_kv_heads, mem.head_dim,
                                   dtype=mem.dtype, device=device)
        self.v_cache = torch.zeros_like(self.k_cache)
        # cache_len may be a caller's view (e.g. one row of a [layers][batch] tensor, so that
        # every layer's length can be set by one copy)
        if cache_len is None:
            cache_len = torch.zeros(batch, dtype=torch.int32, device=device)
        if cache_len.shape != (batch,) or cache_len.dtype != torch.int32:
            raise ValueError("cache_len must be int32 [batch]")
        self.cache_len = cache_len
        self.workspace = workspace(mem.step_workspace_size(batch, k, n_q_heads), device)
        self.pos_offset = k if pos_offset is None else pos_offset
        self.c = DecodeState(batch=batch, top_k=k, n_q_heads=n_q_heads,
                             cache_capacity=cache_capacity, pos_offset=self.pos_offset,
                             state=_ptr(self.state), ids=_ptr(self.ids), scores=_ptr(self.scores),
                             k_cache=_ptr(self.k_cache), v_cache=_ptr(self.v_cache),
                             cache_len=_ptr(self.cache_len), workspace=_ptr(self.workspace),
                             workspace_bytes=self.workspace.numel())


def _tensor(t, name: str, shape, dtype, index: int, contiguous: bool = True) -> int:
    """Check one argument of the rotary and 8-bit cache calls (on device `index`); its pointer."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name}: expected a torch.Tensor")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if t.get_device() != index:
        raise ValueError(f"{name}: expected a tensor on cuda:{index}, got {t.device}")
    if contiguous and not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    return t.data_ptr()


def _buffer(t, name: str, index: int):
    """(pointer, bytes) of a workspace."""
    if not isinstance(t, torch.Tensor) or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor on cuda:{index}")
    return t.data_ptr(), t.numel() * t.element_size()


def _call(fn, device, stream, *args):
    """One library call on `device` (made current for it) and `stream` (default: its current one).
    The raw accessors are the ones behind torch.cuda.current_stream() and current_device(), without
    building their objects: a small call's time is its issue."""
    if stream is None:
        raw = torch._C._cuda_getCurrentRawStream(device.index)
    elif stream.device != device:
        raise ValueError(f"the stream is on {stream.device}, the tensors are on {device}")
    else:
        raw = stream.cuda_stream
    if torch._C._cuda_getDevice() == device.index:
        status = fn(*args, raw)
    else:
        with torch.cuda.device(device):
            status = fn(*args, raw)
    if status != 0:
        _check(status)


def _output(stream, make, *args, **kw):
    """An output for a call on `stream`, from that stream's memory: a block that the current stream
    has freed may still be read by work queued there."""
    if stream is None:
        return make(*args, **kw)
    with torch.cuda.stream(stream):
        return make(*args, **kw)


def _device(device) -> torch.device:
    d = torch.device(device)
    if d.type != "cuda":
        raise ValueError(f"expected a CUDA device, got {d}")
    return d if d.index is not None else torch.device("cuda", torch.cuda.current_device())


class Rope:
    """Rotary positions of Q and K (msa_rope_*): the first ``rotary_dim`` elements of each head
    (None: all) in "half" or "interleaved" pairs, frequencies of base ``theta`` with scaling
    "none", "linear", "ntk" or "yarn".  The output feeds Cache8.append and Cache8.attend.

    q and k are [..., heads, head_dim] with the same leading dimensions as ``positions`` (int64),
    fp32 or bf16; heads of a token are dense and tokens evenly spaced, so slices of a joint
    projection are taken as they lie.  k may be None.  Outputs that are not given are allocated on
    the call's stream."""

    LAYOUTS = {"half": 0, "interleaved": 1}
    SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}

    def __init__(self, head_dim: int, rotary_dim: int | None = None, theta: float = 1e6,
                 layout: str = "half", scaling: str = "none", factor: float = 1.0,
                 original_length: int = 0, magnitude: float = 0.0, device="cuda"):
        if layout not in self.LAYOUTS:
            raise ValueError(f"layout must be one of {sorted(self.LAYOUTS)}, got {layout!r}")
        if scaling not in self.SCALINGS:
            raise ValueError(f"scaling must be one of {sorted(self.SCALINGS)}, got {scaling!r}")
        cfg = RopeConfig(head_dim=head_dim, rotary_dim=head_dim if rotary_dim is None else rotary_dim,
                         theta=theta, layout=self.LAYOUTS[layout], scaling=self.SCALINGS[scaling],
                         factor=factor, original_length=original_length, magnitude=magnitude)
        h = _P()
        self.handle = None
        self.device = _device(device)
        with torch.cuda.device(self.device):
            _check(_lib.msa_rope_create(ctypes.byref(cfg), ctypes.byref(h)))
        self.handle = h
        self.head_dim = head_dim

    def close(self):
        if getattr(self, "handle", None):
            _check(_lib.msa_rope_destroy(self.handle))
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    def _side(self, x, name, lead, dtype):
        """(pointer, heads, token stride) of one of Q and K."""
        if not isinstance(x, torch.Tensor):
            raise TypeError(f"{name}: expected a torch.Tensor")
        shape = x.shape
        if len(shape) < 2 or shape[:-2] != lead or shape[-1] != self.head_dim:
            raise ValueError(f"{name}: expected shape {(*lead, 'heads', self.head_dim)}, got "
                             f"{tuple(shape)}")
        if x.dtype is not dtype:
            raise ValueError(f"{name}: expected {dtype}, got {x.dtype}")
        if x.get_device() != self.device.index:
            raise ValueError(f"{name}: expected a tensor on {self.device}, got {x.device}")
        H, D = shape[-2], shape[-1]
        if x.is_contiguous():
            return x.data_ptr(), H, H * D
        st = x.stride()
        ok = st[-1] == 1 and (H == 1 or st[-2] == D)
        n, step = 1, None  # tokens so far, distance of consecutive ones
        for d in range(len(lead) - 1, -1, -1):
            if lead[d] != 1:
                step = st[d] if step is None else step
                ok = ok and st[d] == n * step
                n *= lead[d]
        if not ok:
            raise ValueError(f"{name}: heads must be dense and tokens evenly spaced")
        return x.data_ptr(), H, H * D if step is None else step

    def _apply(self, inverse, q, k, positions, q_out, k_out, stream):
        if not isinstance(positions, torch.Tensor):
            raise TypeError("positions: expected a torch.Tensor")
        lead = positions.shape
        pos = _tensor(positions, "positions", lead, torch.int64, self.device.index)
        if not isinstance(q, torch.Tensor) or q.dtype not in _DTYPE:
            raise TypeError("q: expected an fp32 or bf16 torch.Tensor")
        dtype = q.dtype
        qp, qh, qs = self._side(q, "q", lead, dtype)
        if q_out is None:
            q_out = _output(stream, torch.empty_like, q, memory_format=torch.contiguous_format)
            qo, qoh, qos = q_out.data_ptr(), qh, qh * self.head_dim
        else:
            qo, qoh, qos = self._side(q_out, "q_out", lead, dtype)
        kp, kh, ks, ko, koh, kos = None, 0, 0, None, 0, 0
        if k is not None:
            kp, kh, ks = self._side(k, "k", lead, dtype)
            if k_out is None:
                k_out = _output(stream, torch.empty_like, k, memory_format=torch.contiguous_format)
                ko, koh, kos = k_out.data_ptr(), kh, kh * self.head_dim
            else:
                ko, koh, kos = self._side(k_out, "k_out", lead, dtype)
        if qoh != qh or koh != kh:
            raise ValueError("the outputs must have the heads of the inputs")
        _call(_lib.msa_rope_apply, self.device, stream, self.handle, _DTYPE[dtype],
              positions.numel(), pos, inverse, qp, qh, qs, qo, qos, kp, kh, ks, ko, kos)
        return q_out, k_out

    def rotate(self, q, k, positions, q_out=None, k_out=None, stream=None):
        """Rotated (q, k); outputs may be given, and may be the inputs themselves."""
        return self._apply(0, q, k, positions, q_out, k_out, stream)

    def backward(self, d_q, d_k, positions, dq_out=None, dk_out=None, stream=None):
        """Gradients of rotate's inputs from the gradients of its outputs."""
        return self._apply(1, d_q, d_k, positions, dq_out, dk_out, stream)


class Cache8:
    """8-bit local K/V cache of one layer (msa_cache8_*), buffers torch-allocated: ``k``, ``v``
    [batch][H_kv][capacity][D] (int8 or float8_e4m3fn), ``k_scale``, ``v_scale`` fp32
    [batch][H_kv][capacity / block_len], ``cache_len`` int32 [batch] and, with ``track_weights``,
    ``weights`` fp32 [batch][H_kv][capacity]."""

    FORMATS = {"int8": (0, torch.int8), "e4m3": (1, torch.float8_e4m3fn)}

    def __init__(self, mem: Memory, batch: int, capacity: int, block_len: int = 64,
                 fmt: str = "int8", track_weights: bool = False, device="cuda"):
        if fmt not in self.FORMATS:
            raise ValueError(f"fmt must be one of {sorted(self.FORMATS)}, got {fmt!r}")
        if block_len not in (16, 32, 64, 128):
            raise ValueError(f"block_len must be 16, 32, 64 or 128, got {block_len}")
        if batch < 1 or capacity < 1 or capacity % block_len:
            raise ValueError(f"capacity={capacity} must be a positive multiple of block_len="
                             f"{block_len}, and batch={batch} positive")
        self.mem, self.batch, self.capacity, self.block_len = mem, batch, capacity, block_len
        self.fmt = fmt
        self.device = dev = _device(device)
        code, dtype = self.FORMATS[fmt]
        H, D = mem.n_kv_heads, mem.head_dim
        self.k = torch.zeros(batch, H, capacity, D, dtype=torch.int8, device=dev).view(dtype)
        self.v = torch.zeros(batch, H, capacity, D, dtype=torch.int8, device=dev).view(dtype)
        self.k_scale = torch.zeros(batch, H, capacity // block_len, device=dev)
        self.v_scale = torch.zeros_like(self.k_scale)
        self.cache_len = torch.zeros(batch, dtype=torch.int32, device=dev)
        self.weights = torch.zeros(batch, H, capacity, device=dev) if track_weights else None
        self.c = Cache8Struct(batch=batch, capacity=capacity, block_len=block_len, format=code,
                              k=self.k.data_ptr(), v=self.v.data_ptr(),
                              k_scale=self.k_scale.data_ptr(), v_scale=self.v_scale.data_ptr(),
                              cache_len=self.cache_len.data_ptr(),
                              weights=self.weights.data_ptr() if track_weights else None)
        self._ref = ctypes.byref(self.c)

    def _counts(self, t, name):
        return None if t is None else _tensor(t, name, (self.batch,), torch.int32, self.device.index)

    def append(self, K, V, n_tokens=None, start=None, stream=None):
        """Append [batch][tokens][H_kv][D] rows, K already rotated (msa_cache8_append).  K and V
        may be slices of a joint projection (H_kv and D dense, rows on 16 bytes)."""
        mem = self.mem
        if not isinstance(K, torch.Tensor) or K.dim() != 4:
            raise ValueError("K: expected [batch][tokens][H_kv][D]")
        T = K.shape[1]
        shape = (self.batch, T, mem.n_kv_heads, mem.head_dim)
        kp = _tensor(K, "K", shape, mem.dtype, self.device.index, contiguous=False)
        vp = _tensor(V, "V", shape, mem.dtype, self.device.index, contiguous=False)
        ks, vs = K.stride(), V.stride()
        for st in (ks, vs):
            if st[3] != 1 or (st[2] != mem.head_dim and mem.n_kv_heads > 1):
                raise ValueError("K, V: the heads of a token must be dense")
        # (the stride of a dimension of one means nothing)
        _call(_lib.msa_cache8_append, self.device, stream, mem.handle, self._ref, kp, vp, T,
              ks[0] if self.batch > 1 else 0, ks[1] if T > 1 else 0,
              vs[0] if self.batch > 1 else 0, vs[1] if T > 1 else 0,
              self._counts(n_tokens, "n_tokens"), self._counts(start, "start"))

    def read(self, begin, rows: int, K_out=None, V_out=None, stream=None):
        """Values of rows begin[b] .. begin[b] + rows - 1 (begin None: from 0) in the memory's
        dtype, token-major [batch][rows][H_kv][D] like the framework's caches; zeros past
        cache_len."""
        mem = self.mem
        shape = (self.batch, rows, mem.n_kv_heads, mem.head_dim)
        if K_out is None:
            K_out = _output(stream, torch.empty, shape, dtype=mem.dtype, device=self.device)
        if V_out is None:
            V_out = _output(stream, torch.empty_like, K_out)
        _call(_lib.msa_cache8_read, self.device, stream, mem.handle, self._ref,
              self._counts(begin, "begin"), rows,
              _tensor(K_out, "K_out", shape, mem.dtype, self.device.index),
              _tensor(V_out, "V_out", shape, mem.dtype, self.device.index))
        return K_out, V_out

    def attend_workspace_size(self, tokens: int, k: int, n_q_heads: int) -> int:
        with torch.cuda.device(self.device):  # (the library sizes for the current device)
            return _lib.msa_cache8_attend_workspace_size(self.mem.handle, self._ref, tokens, k,
                                                         n_q_heads)

    def attend(self, content, ids, Q, O, workspace, lse=None, n_tokens=None, weight_decay=None,
               stream=None):
        """Attention of the cache's newest tokens over the retrieved memory rows and the cached
        rows (msa_cache8_attend): Q, O [batch][tokens][n_q_heads][D], Q already rotated; lse
        [batch][tokens][n_q_heads] optional.  weight_decay None leaves ``weights`` alone.
        ``content`` is the memory's pooled content, or the Fetcher that just fetched ``ids``
        (msa_cache8_attend_fetched)."""
        mem, dev = self.mem, self.device.index
        if not isinstance(Q, torch.Tensor) or Q.dim() != 4:
            raise ValueError("Q: expected [batch][tokens][n_q_heads][D]")
        T, H_q = Q.shape[1], Q.shape[2]
        shape = (self.batch, T, H_q, mem.head_dim)
        k = ids.shape[1] if ids is not None else 0
        if weight_decay is not None and not weight_decay >= 0.0:
            raise ValueError(f"weight_decay must be >= 0 or None, got {weight_decay}")
        if isinstance(content, Fetcher):
            fn, rows = _lib.msa_cache8_attend_fetched, content.handle
        else:
            fn, rows = _lib.msa_cache8_attend, None
            if k:
                rows = _tensor(content, "content", (mem.n_chunks, 2, mem.n_kv_heads, mem.head_dim),
                               mem.dtype, dev)
        _call(fn, self.device, stream, mem.handle, rows,
              _tensor(ids, "ids", (self.batch, k), torch.int32, dev) if k else None, k, self._ref,
              T, H_q, _tensor(Q, "Q", shape, mem.dtype, dev), self._counts(n_tokens, "n_tokens"),
              _tensor(O, "O", shape, mem.dtype, dev),
              None if lse is None else _tensor(lse, "lse", shape[:3], torch.float32, dev),
              -1.0 if weight_decay is None else weight_decay,
              *_buffer(workspace, "workspace", dev))

    def evict_workspace_size(self) -> int:
        with torch.cuda.device(self.device):
            return _lib.msa_cache8_evict_workspace_size(self.mem.handle, self._ref)

    def evict(self, budget: int, recent: int, workspace, out: "Cache8 | None" = None, stream=None):
        """Keep at most ``budget`` rows a query: whole blocks leave by their accumulated attention
        weight, the last ``recent`` rows' blocks stay (msa_cache8_evict); in place, or into
        ``out``, a cache of the same batch, format and block_len."""
        if out is None:
            out = self
        elif out.device != self.device or (out.mem.n_kv_heads, out.mem.head_dim) != (
                self.mem.n_kv_heads, self.mem.head_dim):
            raise ValueError("out must be on the same device and have the same head shapes")
        _call(_lib.msa_cache8_evict, self.device, stream, self.mem.handle, self._ref, out._ref,
              budget, recent, *_buffer(workspace, "workspace", self.device.index))
