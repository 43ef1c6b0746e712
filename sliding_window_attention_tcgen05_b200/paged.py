"""PyTorch-facing wrappers of the paged-cache entry points (argument marshalling only).

Each call is enqueued on the current stream of the tensors' device.  Without a
``ws`` it takes its scratch from torch's allocator (a block of its own per
call, so calls on several streams and captured graphs do not share one); pass
a Workspace to read the status word with status_check.  Token tensors are
[n_tokens, heads, head_dim] with each head's elements contiguous; rows and
heads may be strided (q, k, v as views of one fused row, say).
"""
from __future__ import annotations

import functools
from dataclasses import dataclass

import torch

from ._lib import VX_BF16, VX_F32, VxAttnOpts, VxPagedCache, VxRopeCfg, VxRows, check, lib
from .api import Workspace

_DT = {torch.float32: VX_F32, torch.bfloat16: VX_BF16}
_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}
_STATUS_BYTES = 256    # a workspace that only holds the status word
_STATUS_BUF = 1024     # the largest workspace without scratch


def _dtype(t, what: str) -> int:
    dt = _DT.get(t.dtype)
    if dt is None:
        raise TypeError(f"{what} must be float32 or bfloat16, not {t.dtype}")
    return dt


def _on(index: int, t, name: str) -> None:
    """t is on CUDA device `index`."""
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.get_device() != index:
        raise ValueError(f"{name} is on {t.device}, expected cuda:{index}")


def _whole(t, name: str, dtype, index: int, numel: int | None = None):
    """Address of a contiguous index or state tensor of the given dtype (and size)."""
    if t is None:
        return None
    _on(index, t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, not {t.numel()}")
    return t.data_ptr()


def _rows(t, name: str, n_tokens: int, heads: int | None, dim: int, dtype, index: int) -> VxRows:
    _on(index, t, name)
    shape = t.shape
    if len(shape) != 3 or shape[0] != n_tokens or shape[2] != dim or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [{n_tokens}, {heads if heads is not None else 'heads'}, {dim}], "
                         f"not {list(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    row, head, el = t.stride()
    if dim > 1 and el != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return VxRows(t.data_ptr(), row, head)


def _new_rows(like):
    """A fresh contiguous tensor of the shape of [tokens, heads, head_dim] rows, and its description."""
    t = torch.empty_like(like, memory_format=torch.contiguous_format)   # half the time of torch.empty(shape, ...)
    _, heads, dim = t.shape
    return t, VxRows(t.data_ptr(), heads * dim, dim)


class _Device:
    """torch.cuda.device(index), entered only where another device is current (these calls take microseconds)."""

    __slots__ = ("ctx",)

    def __init__(self, index: int):
        self.ctx = None if torch.cuda.current_device() == index else torch.cuda.device(index)

    def __enter__(self):
        if self.ctx is not None:
            self.ctx.__enter__()

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)


_stream = torch._C._cuda_getCurrentRawStream   # the handle of the current stream of device `index`

_status: dict = {}   # device index -> a status word for calls without a workspace (it may be shared: nobody reads it)


def _scratch(ws: Workspace | None, nbytes: int, index: int):
    """Address and size of nbytes of scratch, and what keeps it alive until the call is enqueued."""
    if ws is None:
        if nbytes <= _STATUS_BUF:
            buf = _status.get(index)
            if buf is None:
                buf = _status[index] = torch.empty(_STATUS_BUF, dtype=torch.uint8, device=torch.device("cuda", index))
        else:
            buf = torch.empty(nbytes, dtype=torch.uint8, device=torch.device("cuda", index))
        return buf.data_ptr(), buf.numel(), buf
    if ws.buf.get_device() != index:
        raise ValueError(f"ws is on {ws.buf.device}, expected cuda:{index}")
    p, n = ws.get(nbytes)
    return p, n, ws


def _overlap(a, b) -> bool:
    """The storage ranges of two tensors meet."""
    if a.numel() == 0 or b.numel() == 0 or a.untyped_storage().data_ptr() != b.untyped_storage().data_ptr():
        return False

    def span(t):
        lo = t.data_ptr()
        return lo, lo + (sum((n - 1) * st for n, st in zip(t.shape, t.stride())) + 1) * t.element_size()

    (a0, a1), (b0, b1) = span(a), span(b)
    return a0 < b1 and b0 < a1


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


def rope_fwd(x, pos, rope: RopeCfg = RopeCfg(), out=None):
    """Rotary positions of x [n, heads, head_dim] at pos [n] (int64); out may be x itself."""
    if x.dim() != 3:
        raise ValueError(f"x must be [n, heads, head_dim], not {list(x.shape)}")
    n, heads, dim = x.shape
    dt = _dtype(x, "x")
    if not x.is_cuda:
        raise ValueError("x must be a CUDA tensor")
    dev = x.get_device()
    xr = _rows(x, "x", n, heads, dim, x.dtype, dev)
    if out is None:
        out, yr = _new_rows(x)
    else:
        if not (out.data_ptr() == x.data_ptr() and out.stride() == x.stride()) and _overlap(x, out):
            raise ValueError("out overlaps x without being x")
        yr = _rows(out, "out", n, heads, dim, x.dtype, dev)
    with _Device(dev):
        check(lib.vx_rope_fwd(xr, yr, dt, n, heads, dim, _whole(pos, "pos", torch.int64, dev, n), rope.c(),
                              _stream(dev)), "vx_rope_fwd")
    return out


class PagedCache:
    """Paged K/V cache (vx_paged_cache): k, v [layers, pages, kv_heads, page_size, head_dim],
    acc the same without head_dim (fp32; None without ``weights``), table
    [seqs, max_pages] int32 (-1: no page), lens and pos [seqs] int64.  The
    caller hands out the pages by writing table."""

    _TENSORS = ("k", "v", "acc", "table", "lens", "pos")

    def __init__(self, n_layers: int, n_pages: int, page_size: int, n_kv_heads: int, head_dim: int, n_seqs: int,
                 max_pages: int, dtype=torch.bfloat16, weights: bool = False, device=None):
        device = torch.device(device or "cuda")
        if dtype not in _DT:
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
            object.__setattr__(self, "_c", None)   # described and checked again by the next call

    @property
    def device(self):
        return self.k.device

    def _addresses(self):
        acc = self.acc
        return (self.k.data_ptr(), self.v.data_ptr(), None if acc is None else acc.data_ptr(), self.table.data_ptr(),
                self.lens.data_ptr(), self.pos.data_ptr())

    def c(self) -> VxPagedCache:
        """The C description; rebuilt when a tensor was replaced or its storage moved."""
        at = self._addresses()
        if self._c is not None and self._c[0] == at:
            return self._c[1]
        if self.k.dim() != 5 or self.v.shape != self.k.shape or self.v.dtype != self.k.dtype:
            raise ValueError("cache k and v must be [layers, pages, kv_heads, page_size, head_dim] of one dtype")
        L, P, H, page, D = self.k.shape
        if self.table.dim() != 2:
            raise ValueError("cache table must be [seqs, max_pages]")
        S, max_pages = self.table.shape
        dev = self.k.get_device()
        c = VxPagedCache(_whole(self.k, "k", self.k.dtype, dev), _whole(self.v, "v", self.k.dtype, dev),
                         _whole(self.acc, "acc", torch.float32, dev, self.k.numel() // max(D, 1)),
                         _whole(self.table, "table", torch.int32, dev), _whole(self.lens, "lens", torch.int64, dev, S),
                         _whole(self.pos, "pos", torch.int64, dev, S), _dtype(self.k, "k"), L, P, page, H, D, S,
                         max_pages)
        object.__setattr__(self, "_c", (at, c))
        return c


def paged_append(cache: PagedCache, layer: int, k, v, q_start, max_q: int, rope: RopeCfg | None = None, q=None,
                 q_out=None, ws: Workspace | None = None):
    """Writes the chunk's k (rotated with ``rope``) and v [n, kv_heads, head_dim] behind each sequence's tokens in
    one layer; with q, also rotates it and returns the result.  lens and pos are not advanced."""
    c = cache.c()
    dev = cache.k.get_device()
    n, D, dtype = k.shape[0], c.head_dim, cache.k.dtype
    kr, vr = _rows(k, "k", n, c.n_kv_heads, D, dtype, dev), _rows(v, "v", n, c.n_kv_heads, D, dtype, dev)
    qr = qo = None
    heads = 0
    if q is not None:
        qr = _rows(q, "q", n, None, D, dtype, dev)
        heads = q.shape[1]
        if q_out is None:
            q_out, qo = _new_rows(q)
        else:
            if not (q_out.data_ptr() == q.data_ptr() and q_out.stride() == q.stride()) and _overlap(q, q_out):
                raise ValueError("q_out overlaps q without being q")
            qo = _rows(q_out, "q_out", n, heads, D, dtype, dev)
    with _Device(dev):
        p, nb, _keep = _scratch(ws, _STATUS_BYTES, dev)
        check(lib.vx_paged_append(c, layer, None if rope is None else rope.c(), qr, qo, heads, kr, vr,
                                  _whole(q_start, "q_start", torch.int32, dev, c.n_seqs + 1), n, max_q, p, nb,
                                  _stream(dev)), "vx_paged_append")
    return q_out


def paged_advance(cache: PagedCache, q_start, n_tokens: int, max_q: int, ws: Workspace | None = None) -> None:
    """lens and pos of every sequence move on by its rows of the chunk."""
    c = cache.c()
    dev = cache.k.get_device()
    with _Device(dev):
        p, nb, _keep = _scratch(ws, _STATUS_BYTES, dev)
        check(lib.vx_paged_advance(c, _whole(q_start, "q_start", torch.int32, dev, c.n_seqs + 1), n_tokens, max_q,
                                   p, nb, _stream(dev)), "vx_paged_advance")


def paged_attn_fwd(cache: PagedCache, layer: int, q, q_start, max_q: int, max_kv: int = 0, window: int = 0,
                   prefix=None, cap: float = 0.0, slopes=None, scale: float = 0.0, track: float | None = None,
                   return_lse: bool = False, out=None, lse=None, ws: Workspace | None = None):
    """Attention of the chunk q [n, heads, head_dim] over the cache that already holds its k and v.  ``track``: the
    decay of the accumulated weights (None: they are left alone).  Returns out, or (out, lse)."""
    c = cache.c()
    dev = cache.k.get_device()
    if q.dim() != 3:
        raise ValueError(f"q must be [n, heads, head_dim], not {list(q.shape)}")
    n, heads, D = q.shape[0], q.shape[1], c.head_dim
    qr = _rows(q, "q", n, heads, D, cache.k.dtype, dev)
    if out is None:
        out, orr = _new_rows(q)
    else:
        if _overlap(q, out):
            raise ValueError("out overlaps q")
        orr = _rows(out, "out", n, heads, D, cache.k.dtype, dev)
    if lse is None and return_lse:
        lse = q.new_empty((n, heads), dtype=torch.float32)
    opts = VxAttnOpts(scale, cap, window, _whole(prefix, "prefix", torch.int32, dev, c.n_seqs),
                      _whole(slopes, "slopes", torch.float32, dev, heads))
    tr = track is not None
    need = lib.vx_paged_attn_workspace(c, heads, n, max_q, max_kv, lse is not None, tr)
    with _Device(dev):
        p, nb, _keep = _scratch(ws, need, dev)
        check(lib.vx_paged_attn_fwd(c, layer, qr, orr, _whole(lse, "lse", torch.float32, dev, n * heads), heads,
                                    _whole(q_start, "q_start", torch.int32, dev, c.n_seqs + 1), n, max_q, max_kv,
                                    opts, tr, track if tr else 0.0, p, nb, _stream(dev)), "vx_paged_attn_fwd")
    return (out, lse) if return_lse else out


def paged_evict(cache: PagedCache, keep: int, recent: int, dst: PagedCache | None = None, kept=None,
                ws: Workspace | None = None) -> None:
    """Cuts every sequence to its last ``recent`` tokens and the others of most accumulated weight, ``keep`` in
    all, in place or into ``dst``; kept [layers, seqs, kv_heads, keep] int32 gets the slots they came from."""
    c = cache.c()
    dev = cache.k.get_device()
    d = c
    if dst is not None:
        d = dst.c()
        _on(dev, dst.k, "dst")
    if kept is not None and kept.numel() == 0:
        kept = None
    need = _STATUS_BYTES if kept is not None else lib.vx_paged_evict_workspace(c, keep)
    with _Device(dev):
        p, nb, _keep = _scratch(ws, need, dev)
        check(lib.vx_paged_evict(c, d, keep, recent,
                                 _whole(kept, "kept", torch.int32, dev, c.n_layers * c.n_seqs * c.n_kv_heads * keep),
                                 p, nb, _stream(dev)), "vx_paged_evict")
