"""PyTorch-facing wrappers of the paged-cache entry points (argument marshalling only, in csrc/bind.cpp).

Each call is enqueued on the current stream of the tensors' device.  Without a
``ws`` it takes its scratch from torch's allocator (a block of its own per
call, so calls on several streams and captured graphs do not share one); pass
a Workspace to read the status word with status_check.  Token tensors are
[n_tokens, heads, head_dim] with each head's elements contiguous; rows and
heads may be strided (q, k, v as views of one fused row, say).
"""
from __future__ import annotations

import ctypes as C
import functools
from dataclasses import dataclass, fields

import torch

from ._lib import VxPagedCache, VxRopeCfg, lib
from .api import _STATUS_BYTES, Workspace


class _NoBind:
    """In the place of _bind.so where it cannot be loaded: the paged cache's calls raise, the rest of the package works."""

    def __init__(self, why: str):
        self._why = why

    def __getattr__(self, name):
        raise ImportError(f"_bind.so could not be loaded ({self._why}); build it with "
                          "`python sliding_window_attention_tcgen05_b200/build.py`")


try:
    from . import _bind
except ImportError as e:
    _bind = _NoBind(str(e))

_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def _ws(ws: Workspace | None, nbytes: int, device: int):
    """Address and size of a caller's workspace, grown to nbytes; (0, 0) without one."""
    if ws is None:
        return 0, 0
    if ws.buf.get_device() != device:
        raise ValueError(f"ws is on {ws.buf.device}, expected cuda:{device}")
    ws.get(nbytes)
    return ws.buf.data_ptr(), ws.buf.numel()


@dataclass(frozen=True)
class RopeCfg:
    """Rotary positions (mirrors vx_rope_cfg): rot_dim 0 rotates the whole head;
    scaling "none", "linear", "ntk" or "yarn" (see include/vx.h for the formulas)."""

    theta: float = 1e6
    rot_dim: int = 0
    interleaved: bool = False
    scaling: str = "none"
    factor: float = 1.0
    orig_len: int = 0
    beta_fast: float = 32.0
    beta_slow: float = 1.0
    mscale: float = 0.0

    @functools.cached_property
    def _c(self) -> VxRopeCfg:
        if self.scaling not in _SCALING:
            raise ValueError(f"unknown scaling {self.scaling!r}")
        return VxRopeCfg(self.rot_dim, int(self.interleaved), _SCALING[self.scaling], self.orig_len, self.theta,
                         self.factor, self.beta_fast, self.beta_slow, self.mscale)

    def c(self) -> VxRopeCfg:
        return self._c

    def __getstate__(self):   # a copy or another process makes its own C structure
        return {f.name: getattr(self, f.name) for f in fields(self)}

    @functools.cached_property
    def _address(self) -> int:
        return C.addressof(self._c)


def rope_fwd(x, pos, rope: RopeCfg = RopeCfg(), out=None):
    """Rotary positions of x [n, heads, head_dim] at pos [n] (int64); out may be x itself."""
    return _bind.rope_fwd(x, pos, rope._address, out)


class PagedCache:
    """Paged K/V cache (vx_paged_cache): k, v [layers, pages, kv_heads, page_size, head_dim],
    acc the same without head_dim (fp32; None without ``weights``), table
    [seqs, max_pages] int32 (-1: no page), lens and pos [seqs] int64.  The
    caller hands out the pages by writing table."""

    _TENSORS = ("k", "v", "acc", "table", "lens", "pos")

    def __init__(self, n_layers: int, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, n_seqs: int,
                 max_pages: int, dtype=torch.bfloat16, weights: bool = False, device=None):
        device = torch.device(device or "cuda")
        if dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"the cache must be float32 or bfloat16, not {dtype}")
        shape = (n_layers, n_pages, n_kv_heads, page_size, head_dim)
        self.k = torch.zeros(shape, dtype=dtype, device=device)
        self.v = torch.zeros(shape, dtype=dtype, device=device)
        self.acc = torch.zeros(shape[:4], dtype=torch.float32, device=device) if weights else None
        self.table = torch.full((n_seqs, max_pages), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(n_seqs, dtype=torch.int64, device=device)
        self.pos = torch.zeros(n_seqs, dtype=torch.int64, device=device)

    def __setattr__(self, name, value):
        object.__setattr__(self, name, value)
        if name in self._TENSORS:
            object.__setattr__(self, "_described", None)   # described and checked again by the next call

    def __getstate__(self):   # a copy or another process describes its own tensors
        return {**self.__dict__, "_described": None}

    @property
    def device(self):
        return self.k.device

    def _handle(self):
        h = self._described
        if h is None:
            h = _bind.Cache(self.k, self.v, self.acc, self.table, self.lens, self.pos)
            object.__setattr__(self, "_described", h)
        return h

    def c(self) -> VxPagedCache:
        """The C description, valid until a tensor is replaced."""
        return VxPagedCache.from_address(self._handle().address())


def paged_append(cache: PagedCache, layer: int, k, v, q_start, max_q: int, rope: RopeCfg | None = None, q=None,
                 q_out=None, ws: Workspace | None = None):
    """Writes the chunk's k (rotated with ``rope``) and v [n, kv_heads, head_dim] behind each sequence's tokens in
    one layer; with q, also rotates it and returns the result.  lens and pos are not advanced."""
    h = cache._handle()
    p, nb = (0, 0) if ws is None else _ws(ws, _STATUS_BYTES, h.dev)
    return _bind.paged_append(h, layer, k, v, q_start, max_q, 0 if rope is None else rope._address, q, q_out, p, nb)


def paged_advance(cache: PagedCache, q_start, n_tokens: int, max_q: int, ws: Workspace | None = None) -> None:
    """lens and pos of every sequence move on by its rows of the chunk."""
    h = cache._handle()
    p, nb = (0, 0) if ws is None else _ws(ws, _STATUS_BYTES, h.dev)
    _bind.paged_advance(h, q_start, n_tokens, max_q, p, nb)


def paged_attn_fwd(cache: PagedCache, layer: int, q, q_start, max_q: int, max_kv: int = 0, window: int = 0,
                   prefix=None, cap: float = 0.0, slopes=None, scale: float = 0.0, track: float | None = None,
                   return_lse: bool = False, out=None, lse=None, ws: Workspace | None = None):
    """Attention of the chunk q [n, heads, head_dim] over the cache that already holds its k and v.  ``track``: the
    decay of the accumulated weights (None: they are left alone).  Returns out, or (out, lse)."""
    h = cache._handle()
    p = nb = 0
    if ws is not None and q.dim() == 3:
        need = lib.vx_paged_attn_workspace(cache.c(), q.shape[1], q.shape[0], max_q, max_kv,
                                           int(lse is not None or return_lse), int(track is not None))
        p, nb = _ws(ws, need, h.dev)
    return _bind.paged_attn_fwd(h, layer, q, q_start, max_q, max_kv, window, prefix, cap, slopes, scale, track,
                                return_lse, out, lse, p, nb)


def paged_evict(cache: PagedCache, keep: int, recent: int, dst: PagedCache | None = None, kept=None,
                ws: Workspace | None = None) -> None:
    """Cuts every sequence to its last ``recent`` tokens and the others of most accumulated weight, ``keep`` in
    all, in place or into ``dst``; kept [layers, seqs, kv_heads, keep] int32 gets the slots they came from."""
    h = cache._handle()
    p = nb = 0
    if ws is not None:
        p, nb = _ws(ws, lib.vx_paged_evict_workspace(cache.c(), keep), h.dev)
    _bind.paged_evict(h, keep, recent, None if dst is None else dst._handle(), kept, p, nb)
