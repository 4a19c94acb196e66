"""Python binding over ``libsa.so``.

Argument marshalling only: torch tensors (device memory, streams) are turned
into the C structs of ``include/sa.h`` and passed to the library, which runs
every step of the path in its own CUDA kernels.  Nothing here computes.

A call runs on the device of its tensors, which must all be on one, and on
``stream`` (a torch.cuda.Stream of that device) or that device's current one.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass
from typing import Optional

import numpy as np
import torch

from . import _abi
from ._abi import SaCache, SaError, SaNewTokens, SaQuery, check

# (a torch without CUDA has neither; nor has it tensors that get this far)
_device = getattr(torch._C, "_cuda_getDevice", None)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)

_TORCH_RAW = {np.dtype(np.uint8): torch.uint8, np.dtype(np.uint16): torch.int16,
              np.dtype(np.float32): torch.float32, np.dtype(np.int32): torch.int32}


def _t(a: Optional[np.ndarray], device) -> Optional[torch.Tensor]:
    """numpy -> torch on `device`, raw bits preserved (bf16 travels as int16)."""
    if a is None:
        return None
    a = np.ascontiguousarray(a)
    if a.dtype == np.uint16:
        a = a.view(np.int16)
    return torch.from_numpy(a).to(device)


def _ptr(t: Optional[torch.Tensor]) -> Optional[int]:
    return None if t is None else t.data_ptr()


def _need(t, name: str, dtype=None, shape=None, optional: bool = False) -> None:
    """Marshalling precondition: a contiguous CUDA tensor (of `dtype` and `shape`
    when given).  The library reads raw pointers, so a host tensor, a strided
    view or an int64 index tensor would be misread; refuse them here."""
    if t is None:
        if optional:
            return
        raise SaError(_abi.SA_ERR_INVALID_ARG, f"{name} is required")
    # the usual case first: a call checks a dozen tensors
    if (type(t) is torch.Tensor and t.is_cuda and t.is_contiguous() and
            (dtype is None or t.dtype is dtype or (type(dtype) is tuple and t.dtype in dtype)) and
            (shape is None or t.shape == shape)):
        return
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SaError(_abi.SA_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    if not t.is_contiguous():
        raise SaError(_abi.SA_ERR_INVALID_ARG, f"{name} must be contiguous")
    if dtype is not None and t.dtype not in (dtype if isinstance(dtype, tuple) else (dtype,)):
        raise SaError(_abi.SA_ERR_INVALID_ARG, f"{name} has dtype {t.dtype}")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise SaError(_abi.SA_ERR_INVALID_ARG, f"{name} has shape {tuple(t.shape)}, "
                                               f"expected {tuple(shape)}")


def _need_rows(t, name: str, n_rows: int, min_cols: int) -> None:
    """A CUDA fp32 matrix whose rows may be padded (unit column stride)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise SaError(_abi.SA_ERR_INVALID_ARG, f"{name} must be a CUDA tensor")
    if t.dtype != torch.float32 or t.dim() != 2 or t.stride(1) != 1:
        raise SaError(_abi.SA_ERR_INVALID_ARG, f"{name} must be a float32 matrix with unit "
                                               "column stride")
    if t.shape[0] != n_rows or t.shape[1] < min_cols:
        raise SaError(_abi.SA_ERR_INVALID_ARG, f"{name} has shape {tuple(t.shape)}")


def _need_sums(t, name: str, batch: int, min_cols: int) -> int:
    """Per-sequence running sums: a contiguous CUDA fp32 matrix of `batch` rows
    (they are written up to their ends).  Returns the row length."""
    _need(t, name, torch.float32)
    if t.dim() != 2 or t.shape[0] != batch or t.shape[1] < max(1, min_cols):
        raise SaError(_abi.SA_ERR_INVALID_ARG, f"{name} has shape {tuple(t.shape)}, expected "
                                               f"({batch}, >= {max(1, min_cols)})")
    return int(t.shape[1])


def _need_here(where: str, *tensors) -> int:
    """The kernels run on the current device, which is that of the entry point's
    first argument (see _there): refuse tensors of another one.  Returns the raw
    handle of its current stream (a Stream object costs 3 us)."""
    here = _device()
    for t in tensors:
        if t is not None and t.get_device() != here:
            raise SaError(_abi.SA_ERR_INVALID_ARG, f"{where}: a tensor is on {t.device}, the "
                                                   f"call runs on cuda:{here}")
    return _raw_stream(here)


def _away(t) -> bool:
    """Whether an entry point's first argument is not on the current device."""
    d = t.get_device() if isinstance(t, torch.Tensor) else -1   # -1: the host
    return d < 0 or d != _device()


def _there(f, given: dict):
    """Entry point `f` with its arguments, on the device of the first one, whichever
    is current, and on ``stream``, or that device's current one.  Both are made
    current while it runs, so the buffers that the binding makes itself are allocated
    and filled there, and a workspace dropped on return goes back to that stream,
    behind the kernels that use it.  Results that it made may be used on the
    caller's stream, which the allocator is told."""
    first = next(iter(given.values()))
    first = getattr(first, "page_table", first)
    if not isinstance(first, torch.Tensor) or first.get_device() < 0:
        raise SaError(_abi.SA_ERR_INVALID_ARG, f"{f.__name__}: CUDA tensors only")
    stream = given.pop("stream")
    if stream is None:
        with torch.cuda.device(first.get_device()):
            return f(**given)
    if stream.device.index != first.get_device():
        raise SaError(_abi.SA_ERR_INVALID_ARG, f"{f.__name__}: the stream is on "
                                               f"{stream.device}, the tensors on {first.device}")
    caller = torch.cuda.current_stream(stream.device)
    with torch.cuda.stream(stream):
        made = f(**given)
    if caller != stream:
        own = {id(a) for a in given.values()}
        for t in made if isinstance(made, tuple) else (made,):
            if isinstance(t, torch.Tensor) and id(t) not in own:
                t.record_stream(caller)
    return made


@dataclass
class DeviceCache:
    """The paged index-key and latent caches of one layer, resident on the device."""

    page_table: torch.Tensor
    seq_len: torch.Tensor
    num_pages: int
    index_dtype: str
    k_index: torch.Tensor
    k_index_scale: Optional[torch.Tensor]
    kv_dtype: str
    kv: torch.Tensor
    kv_rope: Optional[torch.Tensor]
    kv_scale: Optional[torch.Tensor]
    d_index: int
    d_latent: int
    d_rope: int
    page_size: int = 64
    kv_scale_tile: tuple = (0, 0)   # (tokens, dims) per e4m3 scale; (0, 0): one per page

    def struct(self) -> SaCache:
        _need(self.page_table, "page_table", torch.int32)
        _need(self.seq_len, "seq_len", torch.int32)
        _need(self.k_index, "k_index", optional=True)
        _need(self.k_index_scale, "k_index_scale", optional=True)
        _need(self.kv, "kv", optional=True)
        _need(self.kv_rope, "kv_rope", optional=True)
        _need(self.kv_scale, "kv_scale", optional=True)
        if self.page_table.dim() != 2 or self.seq_len.numel() < self.page_table.shape[0]:
            raise SaError(_abi.SA_ERR_INVALID_ARG, "page_table must be [batch, max_pages] and "
                                                   "seq_len have an entry per sequence")
        # in the order of the struct's fields: by keyword the construction takes twice as long
        batch, max_pages = self.page_table.shape
        return SaCache(
            _ptr(self.page_table), _ptr(self.seq_len), batch, max_pages, self.num_pages,
            self.page_size,
            _abi.DTYPES[self.index_dtype], _ptr(self.k_index), _ptr(self.k_index_scale),
            self.d_index, _abi.DTYPES[self.kv_dtype], _ptr(self.kv), _ptr(self.kv_rope),
            _ptr(self.kv_scale), self.d_latent, self.d_rope, int(self.kv_scale_tile[0]),
            int(self.kv_scale_tile[1]))


@dataclass
class DeviceQueries:
    """One step's query tokens (indexer query, head weights, attention query)."""

    q_seq: torch.Tensor
    q_pos: torch.Tensor
    max_visible: int
    q_index: torch.Tensor
    q_index_scale: Optional[torch.Tensor]
    w: torch.Tensor
    h_index: int
    q_dtype: str
    q: torch.Tensor
    heads: int
    sm_scale: float
    # chunked prefill: queries 4i .. 4i+3 belong to one sequence (see sa_query.q_group)
    q_group: int = 1

    @property
    def n_q(self) -> int:
        return int(self.q_seq.shape[0])

    def struct(self) -> SaQuery:
        _need(self.q_seq, "q_seq", torch.int32)
        _need(self.q_pos, "q_pos", torch.int32)
        if self.q_pos.numel() < self.n_q:
            raise SaError(_abi.SA_ERR_INVALID_ARG, "q_pos must have an entry per query")
        for name in ("q_index", "q_index_scale", "w", "q"):
            _need(getattr(self, name), name, optional=True)
        return SaQuery(
            self.n_q, _ptr(self.q_seq), _ptr(self.q_pos), self.max_visible, _ptr(self.q_index),
            _ptr(self.q_index_scale), _ptr(self.w), self.h_index, _abi.DTYPES[self.q_dtype],
            _ptr(self.q), self.heads, self.sm_scale, self.q_group)

    def tensors(self) -> dict:
        return {"q_seq": self.q_seq, "q_pos": self.q_pos, "q_index": self.q_index,
                "q_index_scale": self.q_index_scale, "w": self.w, "q": self.q}

    def copy_from(self, host: dict, non_blocking: bool = True) -> int:
        """Copy a step's inputs (e.g. pinned host tensors) into these buffers.
        Returns the bytes copied."""
        n = 0
        for k, dst in self.tensors().items():
            src = host.get(k)
            if dst is None or src is None:
                continue
            dst.copy_(src, non_blocking=non_blocking)
            n += src.numel() * src.element_size()
        return n


def upload(wl, device="cuda") -> tuple[DeviceCache, DeviceQueries]:
    """Place a workload (numpy arrays) on the device."""
    sp = wl.spec
    if getattr(sp, "index_scale_group", 0):
        raise SaError(_abi.SA_ERR_UNSUPPORTED,
                      "upload: fp32 index scales per group of values have no kernel in this "
                      "library (its group-scaled index format is MXFP8: E8M0 scales per 32)")
    cache = DeviceCache(
        page_table=_t(wl.page_table, device), seq_len=_t(wl.seq_len, device),
        num_pages=int(wl.num_pages), index_dtype=sp.index_dtype,
        k_index=_t(wl.k_index, device), k_index_scale=_t(wl.k_index_scale, device),
        kv_dtype=sp.kv_dtype, kv=_t(wl.kv, device), kv_rope=_t(wl.kv_rope, device),
        kv_scale=_t(wl.kv_scale, device), d_index=sp.d_index, d_latent=sp.d_latent,
        d_rope=sp.d_rope, page_size=sp.page_size, kv_scale_tile=tuple(sp.kv_scale_tile))
    queries = DeviceQueries(
        q_seq=_t(wl.q_seq, device), q_pos=_t(wl.q_pos, device), max_visible=wl.max_visible,
        q_index=_t(wl.q_index, device), q_index_scale=_t(wl.q_index_scale, device),
        w=_t(wl.w, device), h_index=sp.h_index, q_dtype=sp.q_dtype, q=_t(wl.q, device),
        heads=sp.heads, sm_scale=sp.softmax_scale,
        q_group=4 if sp.queries[0] == "prefill" else 1)
    return cache, queries


def host_queries(wl, pin: bool = True) -> dict:
    """A step's query inputs as (pinned) host tensors, for end-to-end timing."""
    out = {}
    for k in ("q_seq", "q_pos", "q_index", "q_index_scale", "w", "q"):
        a = getattr(wl, k)
        if a is None:
            continue
        t = _t(a, "cpu")
        out[k] = t.pin_memory() if pin else t
    return out


# ---------------------------------------------------------------- workspace ---

def workspace_size(cache: DeviceCache, queries: Optional[DeviceQueries], top_k: int,
                   uses: int) -> int:
    """``queries`` may be None for SA_WS_APPEND and SA_WS_EVICT (top_k = the budget)."""
    c = cache.struct()
    q = None if queries is None else ctypes.byref(queries.struct())
    n = _abi.lib().sa_workspace_size(ctypes.byref(c), q, top_k, uses)
    if n == 0:
        raise SaError(_abi.SA_ERR_INVALID_ARG, "sa_workspace_size")
    return int(n)


def workspace(nbytes: int, device="cuda") -> torch.Tensor:
    """Device workspace (torch allocations are at least 256-byte aligned)."""
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def device_status(ws: torch.Tensor, stream=None) -> tuple[int, int]:
    """(status, detail) of the last call that used `ws`; synchronises the stream."""
    if stream is not None or _away(ws):
        return _there(device_status, locals())
    detail = ctypes.c_int32(0)
    st = _abi.lib().sa_device_status(_ptr(ws), ws.numel(), _raw_stream(_device()),
                                     ctypes.byref(detail))
    return int(st), int(detail.value)


# -------------------------------------------------------------- entry points ---

def indexer_score(cache: DeviceCache, queries: DeviceQueries, scores=None, ws=None,
                  stream=None) -> torch.Tensor:
    if stream is not None or _away(cache.page_table):
        return _there(indexer_score, locals())
    dev = queries.q_seq.device
    if scores is None:
        scores = torch.full((queries.n_q, max(1, queries.max_visible)), float("nan"),
                            dtype=torch.float32, device=dev)
    if ws is None:
        ws = workspace(workspace_size(cache, queries, 1, _abi.SA_WS_INDEXER), dev)
    _need_rows(scores, "scores", queries.n_q, queries.max_visible)
    _need(ws, "ws")
    c, q = cache.struct(), queries.struct()
    stream = _need_here("indexer_score", cache.k_index, queries.q_index, scores, ws)
    check(_abi.lib().sa_indexer_score(ctypes.byref(c), ctypes.byref(q), _ptr(scores),
                                      scores.stride(0), _ptr(ws), ws.numel(), stream),
          "sa_indexer_score")
    return scores


def topk(scores: torch.Tensor, valid_len: torch.Tensor, top_k: int, max_valid: int,
         idx=None, ws=None, stream=None) -> torch.Tensor:
    if stream is not None or _away(scores):
        return _there(topk, locals())
    n_q = scores.shape[0]
    if idx is None:
        idx = torch.empty((n_q, top_k), dtype=torch.int32, device=scores.device)
    if ws is None:
        ws = workspace(256, scores.device)
    _need_rows(scores, "scores", n_q, max_valid)
    _need(valid_len, "valid_len", torch.int32, (n_q,))
    _need(idx, "idx", torch.int32, (n_q, top_k))
    _need(ws, "ws")
    stream = _need_here("topk", valid_len, idx, ws)
    check(_abi.lib().sa_topk(_ptr(scores), scores.stride(0), _ptr(valid_len), n_q, max_valid,
                             top_k, _ptr(idx), _ptr(ws), ws.numel(), stream),
          "sa_topk")
    return idx


def _outputs(queries: DeviceQueries, d_latent: int, out, lse, out_dtype: str):
    dev = queries.q_seq.device
    dt = torch.bfloat16 if out_dtype == "bf16" else torch.float32
    if out is None:
        out = torch.empty((queries.n_q, queries.heads, d_latent), dtype=dt, device=dev)
    if lse is None:
        lse = torch.empty((queries.n_q, queries.heads), dtype=torch.float32, device=dev)
    _need(out, "out", dt, (queries.n_q, queries.heads, d_latent))
    _need(lse, "lse", torch.float32, (queries.n_q, queries.heads))
    return out, lse


def _to_store(out: torch.Tensor) -> torch.Tensor:
    """Where the attention writes `out`: the tensor-core kernel stores 16 bytes at a
    time, so an output off a 16-byte boundary is written elsewhere and copied."""
    return out if out.data_ptr() & 15 == 0 else torch.empty_like(out)


def sparse_mla_attn(cache: DeviceCache, queries: DeviceQueries, idx: torch.Tensor, top_k: int,
                    out=None, lse=None, out_dtype: str = "bf16", ws=None, stream=None):
    if stream is not None or _away(cache.page_table):
        return _there(sparse_mla_attn, locals())
    out, lse = _outputs(queries, cache.d_latent, out, lse, out_dtype)
    if ws is None:
        ws = workspace(workspace_size(cache, queries, top_k, _abi.SA_WS_ATTN), idx.device)
    _need(idx, "idx", torch.int32, (queries.n_q, top_k))
    _need(ws, "ws")
    c, q = cache.struct(), queries.struct()
    stream = _need_here("sparse_mla_attn", cache.kv, queries.q, idx, out, lse, ws)
    to = _to_store(out)
    check(_abi.lib().sa_sparse_mla_attn(ctypes.byref(c), ctypes.byref(q), _ptr(idx), top_k,
                                        _ptr(to), _abi.DTYPES[out_dtype], _ptr(lse), _ptr(ws),
                                        ws.numel(), stream),
          "sa_sparse_mla_attn")
    if to is not out:
        out.copy_(to)
    return out, lse


def decode(cache: DeviceCache, queries: DeviceQueries, top_k: int, out=None, lse=None,
           idx=None, out_dtype: str = "bf16", ws=None, stream=None, phase_events=None):
    """Fused indexer -> top-K -> sparse attention.  Returns (out, lse, idx-or-None).

    ``phase_events``: optional list of len(_abi.DECODE_PHASES) + 1 torch.cuda.Event
    objects recorded at the phase boundaries (sa_decode_traced)."""
    if stream is not None or _away(cache.page_table):
        return _there(decode, locals())
    out, lse = _outputs(queries, cache.d_latent, out, lse, out_dtype)
    if ws is None:
        ws = workspace(workspace_size(cache, queries, top_k, _abi.SA_WS_DECODE),
                       queries.q_seq.device)
    _need(idx, "idx", torch.int32, (queries.n_q, top_k), optional=True)
    _need(ws, "ws")
    c, q = cache.struct(), queries.struct()
    stream = _need_here("decode", cache.kv, queries.q, out, lse, idx, ws)
    to = _to_store(out)
    args = (ctypes.byref(c), ctypes.byref(q), top_k, _ptr(idx), _ptr(to),
            _abi.DTYPES[out_dtype], _ptr(lse), _ptr(ws), ws.numel(), stream)
    if phase_events is None:
        check(_abi.lib().sa_decode(*args), "sa_decode")
    else:
        if len(phase_events) != len(_abi.DECODE_PHASES) + 1:
            raise ValueError("need one event per phase boundary")
        for e in phase_events:
            if e.cuda_event == 0:       # torch creates the CUDA event on first record
                e.record(torch.cuda.current_stream())
        handles = (ctypes.c_void_p * len(phase_events))(*[e.cuda_event for e in phase_events])
        check(_abi.lib().sa_decode_traced(*args, handles), "sa_decode_traced")
    if to is not out:
        out.copy_(to)
    return out, lse, idx


# -------------------------------------------- context-parallel decode steps ---

def local_candidates(cache: DeviceCache, queries: DeviceQueries, top_k: int,
                     offset: torch.Tensor, score=None, pos=None, ws=None, stream=None):
    """This GPU's top_k of its context shard as (score fp32, position + offset
    int32), both [n_q, top_k], ascending positions, (-inf, -1) padding."""
    if stream is not None or _away(cache.page_table):
        return _there(local_candidates, locals())
    dev = queries.q_seq.device
    n_q = queries.n_q
    if score is None:
        score = torch.empty((n_q, top_k), dtype=torch.float32, device=dev)
    if pos is None:
        pos = torch.empty((n_q, top_k), dtype=torch.int32, device=dev)
    if ws is None:
        ws = workspace(workspace_size(cache, queries, top_k, _abi.SA_WS_DECODE), dev)
    _need(offset, "offset", torch.int32, (n_q,))
    _need(score, "score", torch.float32, (n_q, top_k))
    _need(pos, "pos", torch.int32, (n_q, top_k))
    _need(ws, "ws")
    c, q = cache.struct(), queries.struct()
    stream = _need_here("local_candidates", cache.kv, queries.q, offset, score, pos, ws)
    check(_abi.lib().sa_local_candidates(ctypes.byref(c), ctypes.byref(q), top_k, _ptr(offset),
                                         _ptr(score), _ptr(pos), _ptr(ws), ws.numel(), stream),
          "sa_local_candidates")
    return score, pos, ws


def merge_candidates(score: torch.Tensor, pos: torch.Tensor, top_k: int, lo: torch.Tensor,
                     hi: torch.Tensor, idx_global=None, idx_local=None, stream=None):
    """All ranks' candidates [n_ranks, n_q, top_k] -> (global top-K positions,
    the ones in [lo, hi) as local positions), both int32 [n_q, top_k]."""
    if stream is not None or _away(score):
        return _there(merge_candidates, locals())
    n_ranks, n_q, k = score.shape
    if k != top_k:
        raise SaError(_abi.SA_ERR_INVALID_ARG, "merge_candidates: candidate rows of top_k")
    _need(score, "score", torch.float32, (n_ranks, n_q, top_k))
    _need(pos, "pos", torch.int32, (n_ranks, n_q, top_k))
    _need(lo, "lo", torch.int32, (n_q,))
    _need(hi, "hi", torch.int32, (n_q,))
    if idx_global is None:
        idx_global = torch.empty((n_q, top_k), dtype=torch.int32, device=score.device)
    if idx_local is None:
        idx_local = torch.empty((n_q, top_k), dtype=torch.int32, device=score.device)
    _need(idx_global, "idx_global", torch.int32, (n_q, top_k))
    _need(idx_local, "idx_local", torch.int32, (n_q, top_k))
    stream = _need_here("merge_candidates", pos, lo, hi, idx_global, idx_local)
    check(_abi.lib().sa_merge_candidates(_ptr(score), _ptr(pos), n_ranks, n_q, top_k, _ptr(lo),
                                         _ptr(hi), _ptr(idx_global), _ptr(idx_local), stream),
          "sa_merge_candidates")
    return idx_global, idx_local


def combine_partials(o_part: torch.Tensor, lse_part: torch.Tensor, out=None, lse=None,
                     out_dtype: str = "bf16", stream=None):
    """Partial outputs [n_parts, n_q, heads, d] (fp32) with their lse [n_parts,
    n_q, heads] -> (out [n_q, heads, d], lse [n_q, heads])."""
    if stream is not None or _away(o_part):
        return _there(combine_partials, locals())
    n_parts, n_q, heads, d = o_part.shape
    _need(o_part, "o_part", torch.float32, (n_parts, n_q, heads, d))
    _need(lse_part, "lse_part", torch.float32, (n_parts, n_q, heads))
    dt = torch.bfloat16 if out_dtype == "bf16" else torch.float32
    if out is None:
        out = torch.empty((n_q, heads, d), dtype=dt, device=o_part.device)
    if lse is None:
        lse = torch.empty((n_q, heads), dtype=torch.float32, device=o_part.device)
    _need(out, "out", dt, (n_q, heads, d))
    _need(lse, "lse", torch.float32, (n_q, heads))
    stream = _need_here("combine_partials", lse_part, out, lse)
    check(_abi.lib().sa_combine_partials(_ptr(o_part), _ptr(lse_part), n_parts, n_q, heads, d,
                                         _ptr(out), _abi.DTYPES[out_dtype], _ptr(lse), stream),
          "sa_combine_partials")
    return out, lse


# ------------------------------------------------------- input preparation ---

_IN_DTYPES = {torch.bfloat16: "bf16", torch.float32: "f32"}


def _in_dtype(t: torch.Tensor) -> int:
    if t.dtype not in _IN_DTYPES:
        raise SaError(_abi.SA_ERR_UNSUPPORTED, "input dtype (bfloat16 or float32)")
    return _abi.DTYPES[_IN_DTYPES[t.dtype]]


def quantize_index_query(q: torch.Tensor, out=None, scale=None, stream=None):
    """Indexer query [n_q, h_index, d_index] (bfloat16 or float32) -> (e4m3 codes
    uint8 [n_q, h_index, d_index], fp32 scales [n_q, h_index])."""
    if stream is not None or _away(q):
        return _there(quantize_index_query, locals())
    _need(q, "q", (torch.bfloat16, torch.float32))
    n_q, h, d = q.shape
    if out is None:
        out = torch.empty((n_q, h, d), dtype=torch.uint8, device=q.device)
    if scale is None:
        scale = torch.empty((n_q, h), dtype=torch.float32, device=q.device)
    _need(out, "out", torch.uint8, (n_q, h, d))
    _need(scale, "scale", torch.float32, (n_q, h))
    stream = _need_here("quantize_index_query", out, scale)
    check(_abi.lib().sa_quantize_index_query(_ptr(q), _in_dtype(q), n_q, h, d, _ptr(out),
                                             _ptr(scale), stream),
          "sa_quantize_index_query")
    return out, scale


def append_tokens(cache: DeviceCache, seq: torch.Tensor, pos: torch.Tensor,
                  k_index: Optional[torch.Tensor] = None, kv: Optional[torch.Tensor] = None,
                  ws=None, stream=None) -> torch.Tensor:
    """Write new tokens (sequence, position) into the cache's pools in place:
    index keys [n_new, d_index] and latent + rope rows [n_new, d_latent + d_rope],
    both bfloat16 or both float32 (either may be None).  Returns the workspace,
    whose status word records skipped tokens (see device_status)."""
    if stream is not None or _away(cache.page_table):
        return _there(append_tokens, locals())
    if k_index is not None and kv is not None and k_index.dtype != kv.dtype:
        raise SaError(_abi.SA_ERR_INVALID_ARG, "append_tokens: k_index and kv dtypes differ")
    n_new = int(seq.numel())
    _need(seq, "seq", torch.int32, (n_new,))
    _need(pos, "pos", torch.int32, (n_new,))
    _need(k_index, "k_index", (torch.bfloat16, torch.float32), (n_new, cache.d_index),
          optional=True)
    _need(kv, "kv", (torch.bfloat16, torch.float32), (n_new, cache.d_latent + cache.d_rope),
          optional=True)
    rows = kv if kv is not None else k_index
    dt = _abi.SA_BF16 if rows is None else _in_dtype(rows)
    c = cache.struct()
    if ws is None:
        n = _abi.lib().sa_workspace_size(ctypes.byref(c), None, 0, _abi.SA_WS_APPEND)
        if n == 0:
            raise SaError(_abi.SA_ERR_INVALID_ARG, "sa_workspace_size")
        ws = workspace(n, seq.device)
    _need(ws, "ws")
    stream = _need_here("append_tokens", cache.kv, seq, pos, k_index, kv, ws)
    t = SaNewTokens(n_new, _ptr(seq), _ptr(pos), dt, _ptr(k_index), _ptr(kv))
    check(_abi.lib().sa_append_tokens(ctypes.byref(c), ctypes.byref(t), _ptr(ws), ws.numel(),
                                      stream),
          "sa_append_tokens")
    return ws


def read_tokens(cache: DeviceCache, seq: torch.Tensor, pos: torch.Tensor, out=None,
                out_dtype: str = "bf16", ws=None, stream=None):
    """Latent + rope rows of tokens (sequence, position) as the values the pool
    stands for: [n, d_latent + d_rope] in ``out_dtype`` ("bf16" or "f32"; taken
    from ``out`` when given).  Returns (out, ws): the workspace's status word
    records tokens that do not exist, whose rows are zero."""
    if stream is not None or _away(cache.page_table):
        return _there(read_tokens, locals())
    n = int(seq.numel())
    _need(seq, "seq", torch.int32, (n,))
    _need(pos, "pos", torch.int32, (n,))
    if out is None:
        if out_dtype not in _IN_DTYPES.values():
            raise SaError(_abi.SA_ERR_UNSUPPORTED, "read_tokens: out_dtype (bf16 or f32)")
        dt = torch.bfloat16 if out_dtype == "bf16" else torch.float32
        out = torch.empty((n, cache.d_latent + cache.d_rope), dtype=dt, device=seq.device)
    _need(out, "out", (torch.bfloat16, torch.float32), (n, cache.d_latent + cache.d_rope))
    if ws is None:
        ws = workspace(workspace_size(cache, None, 0, _abi.SA_WS_APPEND), seq.device)
    _need(ws, "ws")
    stream = _need_here("read_tokens", cache.kv, seq, pos, out, ws)
    c = cache.struct()
    check(_abi.lib().sa_read_tokens(ctypes.byref(c), n, _ptr(seq), _ptr(pos), _ptr(out),
                                    _in_dtype(out), _ptr(ws), ws.numel(), stream),
          "sa_read_tokens")
    return out, ws


# -------------------------------------- shrinking a cache by its attention ---

def accumulate_weights(cache: DeviceCache, queries: DeviceQueries, idx: torch.Tensor, top_k: int,
                       lse: torch.Tensor, acc: Optional[torch.Tensor], decay: float = 1.0,
                       out=None, ws=None, stream=None, return_ws: bool = False):
    """Attention weight that each cached position received from these queries,
    summed over heads and queries, on top of ``decay * acc``: fp32 rows [batch,
    >= max_visible] per sequence.  ``idx`` and ``lse`` are the attention's own.
    ``acc`` may be None (zeros); ``out`` defaults to ``acc`` (in place), or to a
    new zero-filled [batch, max_visible].  Both are contiguous, with rows of the
    same length; only positions below each sequence's length are written (bring
    ``out`` for sequences longer than max_visible, whose rest is reported otherwise).
    ``return_ws``: return (out, ws) instead of out; the workspace's status word
    records skipped entries and sequences longer than the rows (see device_status)."""
    if stream is not None or _away(cache.page_table):
        return _there(accumulate_weights, locals())
    batch = int(cache.page_table.shape[0])
    if out is None:
        out = acc if acc is not None else torch.zeros(
            (batch, max(1, queries.max_visible)), dtype=torch.float32, device=idx.device)
    _need(idx, "idx", torch.int32, (queries.n_q, top_k))
    _need(lse, "lse", torch.float32, (queries.n_q, queries.heads))
    ld = _need_sums(out, "out", batch, queries.max_visible)
    if acc is not None and _need_sums(acc, "acc", batch, queries.max_visible) != ld:
        raise SaError(_abi.SA_ERR_INVALID_ARG, "accumulate_weights: acc and out rows differ")
    if ws is None:
        ws = workspace(workspace_size(cache, queries, top_k, _abi.SA_WS_WEIGHTS), idx.device)
    _need(ws, "ws")
    c, q = cache.struct(), queries.struct()
    stream = _need_here("accumulate_weights", cache.kv, queries.q, idx, lse, acc, out, ws)
    check(_abi.lib().sa_accumulate_weights(ctypes.byref(c), ctypes.byref(q), _ptr(idx), top_k,
                                           _ptr(lse), _ptr(acc), decay, _ptr(out), ld, _ptr(ws),
                                           ws.numel(), stream),
          "sa_accumulate_weights")
    return (out, ws) if return_ws else out


def evict_tokens(cache: DeviceCache, acc: torch.Tensor, budget: int, dst: DeviceCache,
                 keep_first: int = 0, keep_last: int = 0, acc_out=None, src_pos=None, ws=None,
                 stream=None, return_ws: bool = False):
    """Keep at most ``budget`` tokens of every sequence -- the first
    ``keep_first``, the last ``keep_last`` and those of the largest ``acc``
    between -- and move them, in order, to the pages of ``dst`` (a cache of the
    same formats with its own page table and lengths, which are written; its
    pools may be the same).  ``acc_out`` [batch, >= budget] receives the kept
    sums, zeros behind them.  Returns the kept tokens' original positions,
    int32 [batch, budget], ascending, padded with -1.  ``return_ws``: return
    (positions, ws) instead; the workspace's status word records sequences that were
    skipped whole (see device_status)."""
    if stream is not None or _away(cache.page_table):
        return _there(evict_tokens, locals())
    batch = int(cache.page_table.shape[0])
    ld = _need_sums(acc, "acc", batch, 1)
    if src_pos is None:
        src_pos = torch.empty((batch, budget), dtype=torch.int32, device=acc.device)
    _need(src_pos, "src_pos", torch.int32, (batch, budget))
    ld_out = 0 if acc_out is None else _need_sums(acc_out, "acc_out", batch, budget)
    if ws is None:
        ws = workspace(workspace_size(cache, None, budget, _abi.SA_WS_EVICT), acc.device)
    _need(ws, "ws")
    c, d = cache.struct(), dst.struct()
    stream = _need_here("evict_tokens", cache.kv, dst.kv, dst.seq_len, acc, acc_out, src_pos, ws)
    check(_abi.lib().sa_evict_tokens(
        ctypes.byref(c), _ptr(acc), ld, budget, keep_first, keep_last, ctypes.byref(d),
        _ptr(acc_out), ld_out, _ptr(src_pos), _ptr(ws), ws.numel(), stream),
        "sa_evict_tokens")
    return (src_pos, ws) if return_ws else src_pos
