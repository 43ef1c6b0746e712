"""PyTorch-facing wrappers of the paged-cache entry points (argument marshalling only).

Each call is enqueued on the current stream of the tensors' device.  Without a
``ws`` it takes its scratch from torch's allocator (a block of its own per
call, so calls on several streams and captured graphs do not share one); pass
a Workspace to read the status word with status_check.  Token tensors are [n_tokens, heads, head_dim] with contiguous heads' elements; rows
and heads may be strided (q, k, v as views of one fused row, say).
"""
from __future__ import annotations

import ctypes as C
from dataclasses import dataclass

import torch

from ._lib import VX_BF16, VX_F32, VxAttnOpts, VxPagedCache, VxRopeCfg, VxRows, check, lib
from .api import Workspace

_DT = {torch.float32: VX_F32, torch.bfloat16: VX_BF16}
_SCALING = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def _dtype(t, what: str) -> int:
    if t.dtype not in _DT:
        raise TypeError(f"{what} must be float32 or bfloat16, not {t.dtype}")
    return _DT[t.dtype]


def _same_device(device, **tensors) -> None:
    for name, t in tensors.items():
        if t is None:
            continue
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        if t.device != device:
            raise ValueError(f"{name} is on {t.device}, expected {device}")


def _whole(t, name: str, dtype, numel: int | None = None):
    """A contiguous index or state tensor of the given dtype (and size)."""
    if t is None:
        return None
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if numel is not None and t.numel() != numel:
        raise ValueError(f"{name} must have {numel} elements, not {t.numel()}")
    return C.c_void_p(t.data_ptr())


def _rows(t, name: str, n_tokens: int, heads: int | None, dim: int, dtype) -> VxRows:
    if t.dim() != 3 or t.shape[0] != n_tokens or t.shape[2] != dim or (heads is not None and t.shape[1] != heads):
        raise ValueError(f"{name} must be [{n_tokens}, {heads if heads is not None else 'heads'}, {dim}], "
                         f"not {list(t.shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, not {t.dtype}")
    if dim > 1 and t.stride(2) != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return VxRows(C.c_void_p(t.data_ptr()), t.stride(0), t.stride(1))


def _stream(device) -> C.c_void_p:
    return C.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _scratch(ws: Workspace | None, nbytes: int, device):
    """Pointer and size of nbytes of scratch, and what keeps it alive until the call is enqueued."""
    if ws is None:
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)
        return C.c_void_p(buf.data_ptr()), C.c_size_t(buf.numel()), buf
    if ws.buf.device != device:
        raise ValueError(f"ws is on {ws.buf.device}, expected {device}")
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

    def c(self) -> VxRopeCfg:
        if self.scaling not in _SCALING:
            raise ValueError(f"unknown scaling {self.scaling!r}")
        return VxRopeCfg(self.rot_dim, int(self.interleaved), _SCALING[self.scaling], self.orig_len, self.theta,
                         self.factor, self.beta_fast, self.beta_slow, self.mscale)


def rope_fwd(x, pos, rope: RopeCfg = RopeCfg(), out=None):
    """Rotary positions of x [n, heads, head_dim] at pos [n] (int64); out may be x itself."""
    if x.dim() != 3:
        raise ValueError(f"x must be [n, heads, head_dim], not {list(x.shape)}")
    n, heads, dim = x.shape
    dt = _dtype(x, "x")
    if out is None:
        out = torch.empty(x.shape, dtype=x.dtype, device=x.device)
    _same_device(x.device, x=x, pos=pos, out=out)
    xr, yr = _rows(x, "x", n, heads, dim, x.dtype), _rows(out, "out", n, heads, dim, x.dtype)
    same = out.data_ptr() == x.data_ptr() and out.stride() == x.stride()
    if not same and _overlap(x, out):
        raise ValueError("out overlaps x without being x")
    r = rope.c()
    with torch.cuda.device(x.device):
        check(lib.vx_rope_fwd(C.byref(xr), C.byref(yr), dt, n, heads, dim, _whole(pos, "pos", torch.int64, n),
                              C.byref(r), _stream(x.device)), "vx_rope_fwd")
    return out


class PagedCache:
    """Paged K/V cache (vx_paged_cache): k, v [layers, pages, kv_heads, page_size, head_dim],
    acc the same without head_dim (fp32; None without ``weights``), table
    [seqs, max_pages] int32 (-1: no page), lens and pos [seqs] int64.  The
    caller hands out the pages by writing table."""

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

    @property
    def device(self):
        return self.k.device

    def c(self) -> VxPagedCache:
        if self.k.dim() != 5 or self.v.shape != self.k.shape or self.v.dtype != self.k.dtype:
            raise ValueError("cache k and v must be [layers, pages, kv_heads, page_size, head_dim] of one dtype")
        L, P, H, page, D = self.k.shape
        if self.table.dim() != 2:
            raise ValueError("cache table must be [seqs, max_pages]")
        S, max_pages = self.table.shape
        _same_device(self.k.device, k=self.k, v=self.v, acc=self.acc, table=self.table, lens=self.lens, pos=self.pos)
        return VxPagedCache(_whole(self.k, "k", self.k.dtype), _whole(self.v, "v", self.k.dtype),
                            _whole(self.acc, "acc", torch.float32, self.k.numel() // max(D, 1)),
                            _whole(self.table, "table", torch.int32), _whole(self.lens, "lens", torch.int64, S),
                            _whole(self.pos, "pos", torch.int64, S), _dtype(self.k, "k"), L, P, page, H, D, S,
                            max_pages)


def paged_append(cache: PagedCache, layer: int, k, v, q_start, max_q: int, rope: RopeCfg | None = None, q=None,
                 q_out=None, ws: Workspace | None = None):
    """Writes the chunk's k (rotated with ``rope``) and v [n, kv_heads, head_dim] behind each sequence's tokens in
    one layer; with q, also rotates it and returns the result.  lens and pos are not advanced."""
    c = cache.c()
    n, D, dtype = k.shape[0], cache.k.shape[4], cache.k.dtype
    kr, vr = _rows(k, "k", n, c.n_kv_heads, D, dtype), _rows(v, "v", n, c.n_kv_heads, D, dtype)
    qr = qo = None
    if q is not None:
        if q_out is None:
            q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        qr, qo = _rows(q, "q", n, None, D, dtype), _rows(q_out, "q_out", n, q.shape[1], D, dtype)
        if not (q_out.data_ptr() == q.data_ptr() and q_out.stride() == q.stride()) and _overlap(q, q_out):
            raise ValueError("q_out overlaps q without being q")
    _same_device(cache.device, k=k, v=v, q=q, q_out=q_out, q_start=q_start)
    r = rope.c() if rope is not None else None
    with torch.cuda.device(cache.device):
        p, nb, _keep = _scratch(ws, 256, cache.device)
        check(lib.vx_paged_append(C.byref(c), layer, C.byref(r) if r is not None else None,
                                  C.byref(qr) if qr is not None else None, C.byref(qo) if qo is not None else None,
                                  q.shape[1] if q is not None else 0, C.byref(kr), C.byref(vr),
                                  _whole(q_start, "q_start", torch.int32, c.n_seqs + 1), n, max_q, p, nb,
                                  _stream(cache.device)), "vx_paged_append")
    return q_out


def paged_advance(cache: PagedCache, q_start, n_tokens: int, max_q: int, ws: Workspace | None = None) -> None:
    """lens and pos of every sequence move on by its rows of the chunk."""
    c = cache.c()
    _same_device(cache.device, q_start=q_start)
    with torch.cuda.device(cache.device):
        p, nb, _keep = _scratch(ws, 256, cache.device)
        check(lib.vx_paged_advance(C.byref(c), _whole(q_start, "q_start", torch.int32, c.n_seqs + 1), n_tokens, max_q,
                                   p, nb, _stream(cache.device)), "vx_paged_advance")


def paged_attn_fwd(cache: PagedCache, layer: int, q, q_start, max_q: int, max_kv: int = 0, window: int = 0,
                   prefix=None, cap: float = 0.0, slopes=None, scale: float = 0.0, track: float | None = None,
                   return_lse: bool = False, out=None, lse=None, ws: Workspace | None = None):
    """Attention of the chunk q [n, heads, head_dim] over the cache that already holds its k and v.  ``track``: the
    decay of the accumulated weights (None: they are left alone).  Returns out, or (out, lse)."""
    c = cache.c()
    if q.dim() != 3:
        raise ValueError(f"q must be [n, heads, head_dim], not {list(q.shape)}")
    n, heads, D = q.shape[0], q.shape[1], cache.k.shape[4]
    if out is None:
        out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    qr, orr = _rows(q, "q", n, heads, D, cache.k.dtype), _rows(out, "out", n, heads, D, cache.k.dtype)
    if _overlap(q, out):
        raise ValueError("out overlaps q")
    if lse is None and return_lse:
        lse = torch.empty(n, heads, dtype=torch.float32, device=q.device)
    _same_device(cache.device, q=q, out=out, lse=lse, q_start=q_start, prefix=prefix, slopes=slopes)
    opts = VxAttnOpts(scale, cap, window, _whole(prefix, "prefix", torch.int32, c.n_seqs),
                      _whole(slopes, "slopes", torch.float32, heads))
    tr = track is not None
    need = lib.vx_paged_attn_workspace(C.byref(c), heads, n, max_q, max_kv, int(lse is not None), int(tr))
    with torch.cuda.device(cache.device):
        p, nb, _keep = _scratch(ws, need, cache.device)
        check(lib.vx_paged_attn_fwd(C.byref(c), layer, C.byref(qr), C.byref(orr),
                                    _whole(lse, "lse", torch.float32, n * heads), heads,
                                    _whole(q_start, "q_start", torch.int32, c.n_seqs + 1), n, max_q, max_kv,
                                    C.byref(opts), int(tr), track if tr else 0.0, p, nb, _stream(cache.device)),
              "vx_paged_attn_fwd")
    return (out, lse) if return_lse else out


def paged_evict(cache: PagedCache, keep: int, recent: int, dst: PagedCache | None = None, kept=None,
                ws: Workspace | None = None) -> None:
    """Cuts every sequence to its last ``recent`` tokens and the others of most accumulated weight, ``keep`` in
    all, in place or into ``dst``; kept [layers, seqs, kv_heads, keep] int32 gets the slots they came from."""
    c = cache.c()
    d = (dst or cache).c()
    _same_device(cache.device, dst=(dst or cache).k, kept=kept)
    if kept is not None and kept.numel() == 0:
        kept = None
    need = 256 if kept is not None else lib.vx_paged_evict_workspace(C.byref(c), keep)
    with torch.cuda.device(cache.device):
        p, nb, _keep = _scratch(ws, need, cache.device)
        check(lib.vx_paged_evict(C.byref(c), C.byref(d), keep, recent,
                                 _whole(kept, "kept", torch.int32, c.n_layers * c.n_seqs * c.n_kv_heads * keep),
                                 p, nb, _stream(cache.device)), "vx_paged_evict")
