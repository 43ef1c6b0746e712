"""GPU parity of the paged-cache operators (vx_rope_fwd, vx_paged_append,
vx_paged_advance, vx_paged_attn_fwd, vx_paged_evict) against the float64
statement in oracle/paged.py.

Tolerances, from the arithmetic (u = 2^-24, half a step of fp32; 2^-8, half a
step of bf16):
  scores  |ds| <= ((D + 8) sum|q k| scale) u, with a cap another cap 2^-21 (its
          exponential and reciprocal), with a bias the rounding of a sum of its size
  o       a weight's relative error 2 (ds + exp's 2^-21) + L u, bf16 weights 2^-8 more, times sum p |v|; bf16
          outputs 2^-8 |o| more
  lse     the score error, the exponential's and the logarithm's, L u
  weights the score's and lse's errors, relative to each weight
  rotary  the angle (2^-24 of a half turn, pi 2^-24) and sincos (2 u) times |a| + |b|
"""
import numpy as np
import pytest
import torch

import oracle.paged as paged

pytestmark = pytest.mark.gpu

U, B16 = 2.0 ** -24, 2.0 ** -8
BF, F32 = torch.bfloat16, torch.float32


def _vx():
    import sliding_window_attention_tcgen05_b200 as vx
    return vx


def _host(t):
    return t.detach().double().cpu().numpy()


def _randn(shape, dtype, gen, scale=1.0):
    return (torch.randn(shape, generator=gen, dtype=torch.float32) * scale).to(dtype)


def _within(got, want, tol, what):
    got, want, tol = np.asarray(got), np.asarray(want), np.broadcast_to(tol, np.shape(want))
    assert got.shape == want.shape, what
    inf = ~np.isfinite(want)
    assert np.array_equal(got[inf], want[inf], equal_nan=True), f"{what}: non-finite values differ"
    bad = ~(np.abs(got - want) <= tol) & ~inf
    if bad.any():
        i = np.unravel_index(np.argmax(np.where(bad, np.abs(got - want) / tol, 0)), want.shape)
        raise AssertionError(f"{what}: {bad.sum()} of {want.size} out; at {i}: {got[i]} for {want[i]} (tol {tol[i]:.3g})")


class Batch:
    """Sequences of `olds` cached tokens and `news` new ones on shuffled pages; everything outside them is NaN."""

    def __init__(self, olds, news, hq, hkv, D, page, dtype, seed=1, layers=1, weights=False, lead=0, tail=0, room=0,
                 scale=1.0):
        vx = _vx()
        gen = torch.Generator().manual_seed(seed)
        self.olds, self.news, self.hq, self.hkv, self.D, self.page, self.dtype = olds, news, hq, hkv, D, page, dtype
        self.layers, self.lead = layers, lead
        S = len(olds)
        total = [o + n for o, n in zip(olds, news)]
        need = [max(1, -(-(t + room) // page)) for t in total]
        P = sum(need) + 2
        order = torch.randperm(P, generator=gen)[:sum(need)]
        self.cache = c = vx.PagedCache(layers, P, page, hkv, D, S, max(need) + 1, dtype=dtype, weights=weights)
        at = 0
        for s, m in enumerate(need):
            c.table[s, :m] = order[at:at + m].to(torch.int32)
            at += m
        c.lens.copy_(torch.tensor(olds))
        c.pos.copy_(torch.tensor(olds))
        self.table = c.table.cpu().numpy()
        nan = float("nan")
        k = torch.full(c.k.shape, nan, dtype=dtype)
        v = torch.full(c.v.shape, nan, dtype=dtype)
        self.k = [_randn((layers, t, hkv, D), dtype, gen, scale) for t in total]
        self.v = [_randn((layers, t, hkv, D), dtype, gen) for t in total]
        for s in range(S):
            pg, off = self.slots(s, total[s])
            k[:, pg, :, off] = self.k[s].transpose(0, 1)
            v[:, pg, :, off] = self.v[s].transpose(0, 1)
        c.k.copy_(k)
        c.v.copy_(v)
        self.acc = None
        if weights:
            self.acc = [torch.rand((layers, hkv, t), generator=gen) for t in total]
            a = torch.full(c.acc.shape, nan)
            for s in range(S):
                pg, off = self.slots(s, total[s])
                a[:, pg, :, off] = self.acc[s].permute(2, 0, 1)
            c.acc.copy_(a)
        starts = np.concatenate([[lead], lead + np.cumsum(news)]).astype(np.int32)
        self.starts = starts
        self.n = int(starts[-1]) + tail
        self.q_start = torch.from_numpy(starts).cuda()
        self.q = _randn((self.n, hq, D), dtype, gen, scale)
        self.max_q, self.max_kv = max(news), max(total)

    def slots(self, s, n, first=0):
        j = np.arange(first, n)
        return torch.from_numpy(self.table[s][j // self.page].astype(np.int64)), torch.from_numpy(j % self.page)

    def gather(self, pool, s, n):
        """[layers, pages, heads, page, ...] -> [layers, n, heads, ...] of a sequence's slots."""
        pg, off = self.slots(s, n)
        return pool.cpu()[:, pg, :, off].transpose(0, 1)


def _check_attn(b, o, lse, layer=0, track=None, window=0, prefix=None, cap=0.0, slopes=None, scale=0.0, what=""):
    bf = b.dtype == BF
    o, lse = _host(o), None if lse is None else _host(lse)
    acc = None if track is None else b.cache.acc
    for s, (old, n) in enumerate(zip(b.olds, b.news)):
        if n == 0:
            continue
        rows = slice(b.starts[s], b.starts[s] + n)
        L = old + n
        r = paged.attention(_host(b.q)[rows], _host(b.k[s][layer]), _host(b.v[s][layer]), old, window=window,
                            prefix=0 if prefix is None else prefix[s], cap=cap,
                            slopes=None if slopes is None else np.asarray(slopes, dtype=np.float64), scale=scale)
        bias = 0.0 if slopes is None else float(np.max(slopes)) * L
        ds = ((b.D + 8) * r["smax"] + 4 * bias) * U + cap * 2.0 ** -21          # [n, Hq]
        rel = 2 * (ds + 2.0 ** -21) + (L + 8) * U + (B16 if bf else 0.0)
        tol = r["absv"] * rel[..., None] * 1.01 + (B16 if bf else 2 * U) * np.abs(r["o"]) + 1e-30
        _within(o[rows], r["o"], tol, f"{what} o of sequence {s}")
        dz = ds + 2.0 ** -20 + (L + 8) * U + 4 * U * np.abs(np.where(np.isfinite(r["lse"]), r["lse"], 0.0))
        if lse is not None:
            _within(lse[rows], r["lse"], dz, f"{what} lse of sequence {s}")
        if track is not None:
            got = _host(b.gather(acc, s, L))[layer].T                           # [hkv, L]
            before = track * _host(b.acc[s])[layer] if track else 0.0
            want = before + r["weights"]
            rel = ds.max() + dz.max() + 2.0 ** -20 + n * (b.hq // b.hkv) * U
            _within(got, want, 1.01 * r["weights"] * rel + 4 * U * np.abs(want) + 1e-30,
                    f"{what} weights of sequence {s}")


# ------------------------------------------------------------------- rotary

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("n,H,D,rot,inter,pad,scaling", [
    (1, 1, 64, 64, False, 0, {}),
    (5, 3, 128, 64, True, 1, dict(scaling="yarn", factor=8.0, orig_len=4096)),
    (700, 40, 128, 128, False, 8, dict(scaling="ntk", factor=4.0)),
    (333, 7, 64, 16, True, 0, dict(scaling="linear", factor=3.0)),
    (37, 5, 80, 80, False, 3, {}),
    (29, 3, 36, 12, False, 0, {}),          # no 16-byte vectors
    (29, 3, 36, 10, True, 1, {}),
    (16, 2, 2, 2, False, 0, {}),
    (9, 2, 256, 256, True, 0, dict(scaling="yarn", factor=2.0, orig_len=100, beta_fast=8.0, beta_slow=0.5,
                                   mscale=1.25))])
def test_rope(dtype, n, H, D, rot, inter, pad, scaling):
    vx = _vx()
    gen = torch.Generator().manual_seed(n)
    row = _randn((n, H + pad, D), dtype, gen)
    x = row.cuda()[:, :H]
    far = 1 << 20
    pos = torch.randint(-far, far, (n,), generator=gen)
    pos[0] = 0
    cfg = vx.RopeCfg(theta=1e6, rot_dim=rot, interleaved=inter, **scaling)
    got = vx.rope_fwd(x, pos.cuda(), cfg)
    want = paged.rope(_host(row)[:, :H], pos.numpy(), rot, inter, theta=1e6, **scaling)
    ms = paged.rope_freqs(rot, theta=1e6, **scaling)[1]
    a = np.abs(_host(row)[:, :H])
    part = a[..., :rot]
    pair = (np.repeat(part[..., 0::2] + part[..., 1::2], 2, -1) if inter
            else np.tile(part[..., :rot // 2] + part[..., rot // 2:], 2))
    # The oracle's own angle pos * f in fp64: 2^20 * 2^-53 is nothing beside pi 2^-24.
    tol = np.zeros_like(want)
    tol[..., :rot] = pair * ms * (np.pi + 5) * U + (B16 if dtype == BF else 0) * np.abs(want[..., :rot])
    _within(_host(got), want, tol, "rope")
    y = row.cuda()                                     # in place, on the strided view
    vx.rope_fwd(y[:, :H], pos.cuda(), cfg, out=y[:, :H])
    assert torch.equal(y[:, :H], got) and torch.equal(y[:, H:].cpu(), row[:, H:])


def test_rope_at_far_positions():
    # A table of fp32 angles is off by radians here; the turns are exact.
    vx = _vx()
    x = torch.ones(3, 1, 64, device="cuda")
    pos = [2 ** 40 + 12345, -(2 ** 35) - 7, 2 ** 62 + 1]
    got = _host(vx.rope_fwd(x, torch.tensor(pos).cuda(), vx.RopeCfg(theta=1.0)))
    import decimal
    decimal.getcontext().prec = 60
    pi = decimal.Decimal("3.14159265358979323846264338327950288419716939937510582097494459")
    for r, p in enumerate(pos[:2]):                    # theta 1: every pair turns by the position itself
        ang = float(decimal.Decimal(p) % (2 * pi))
        # a turn's 64-bit fraction is off by 2^-65, times the position
        tol = 2 * (abs(p) * 2.0 ** -65 * 2 * np.pi + (np.pi + 5) * U)
        np.testing.assert_allclose(got[r, 0, :32], np.cos(ang) - np.sin(ang), rtol=0, atol=tol)
    assert np.all(np.abs(got[2]) <= 1.5)


def test_rope_refusals():
    vx = _vx()
    x, pos = torch.zeros(4, 2, 64, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
    with pytest.raises(ValueError, match="heads"):
        vx.rope_fwd(x[0], pos)
    with pytest.raises(TypeError, match="float32 or bfloat16"):
        vx.rope_fwd(x.half(), pos)
    with pytest.raises(TypeError, match="pos"):
        vx.rope_fwd(x, pos.int())
    with pytest.raises(ValueError, match="pos"):
        vx.rope_fwd(x, pos[:3])
    with pytest.raises(ValueError, match="CUDA"):
        vx.rope_fwd(x, pos.cpu())
    with pytest.raises(ValueError, match="overlaps"):
        vx.rope_fwd(x[:3], pos[:3], out=x[1:])
    with pytest.raises(ValueError, match="contiguous"):
        vx.rope_fwd(torch.zeros(4, 64, 2, device="cuda").transpose(1, 2), pos)
    with pytest.raises(ValueError, match="scaling"):
        vx.rope_fwd(x, pos, vx.RopeCfg(scaling="other"))
    with pytest.raises(vx.VxError):
        vx.rope_fwd(x, pos, vx.RopeCfg(rot_dim=7))
    assert vx.rope_fwd(x[:0], pos[:0]).shape == (0, 2, 64)


# ------------------------------------------------------------------- append

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("olds,news,hq,hkv,D,page,rot,inter", [
    ([0], [1], 1, 1, 64, 16, 64, False),
    ([5, 0, 31, 16], [4, 4, 0, 4], 4, 2, 64, 16, 64, True),
    ([100, 3], [1, 77], 6, 2, 128, 7, 64, False),
    ([0] * 40, [3] * 40, 2, 2, 64, 1, 32, False),
    ([1000, 13, 7], [613, 1, 200], 8, 8, 64, 50, 0, False)])      # rot 0: no rotation
def test_append(dtype, olds, news, hq, hkv, D, page, rot, inter):
    vx = _vx()
    b = Batch(olds, news, hq, hkv, D, page, dtype, layers=2, weights=True, lead=2, tail=3)
    c = b.cache
    shift = torch.arange(len(olds)) * 5                # positions part from the slots, as after an eviction
    c.pos.add_(shift.cuda())
    gen = torch.Generator().manual_seed(9)
    row = _randn((b.n, hq + 2 * hkv, D), dtype, gen)
    dev = row.cuda()
    q, k, v = dev[:, :hq], dev[:, hq:hq + hkv], dev[:, hq + hkv:]
    k0, v0, a0 = c.k.cpu(), c.v.cpu(), c.acc.cpu()
    ws = vx.Workspace(256)
    vx.status_reset(ws)
    if rot:
        cfg = vx.RopeCfg(theta=1e4, rot_dim=rot, interleaved=inter, scaling="linear", factor=2.0)
        out = torch.full_like(row, 7.0).cuda()[:, :hq]
        got_q = vx.paged_append(c, 1, k, v, b.q_start, b.max_q, rope=cfg, q=q, q_out=out, ws=ws)
    else:
        cfg, got_q = None, None
        assert vx.paged_append(c, 1, k, v, b.q_start, b.max_q, ws=ws) is None
    assert vx.status_check(ws) == 0
    assert c.lens.tolist() == olds
    want_k, want_v, want_a = k0.clone(), v0.clone(), a0.clone()
    for s, (old, n) in enumerate(zip(olds, news)):
        if n == 0:
            continue
        rows = slice(b.starts[s], b.starts[s] + n)
        at = torch.arange(n) + old + int(shift[s])
        # The rotation itself is tested above: here the rows have to be bit for bit those of vx_rope_fwd.
        kr = vx.rope_fwd(k[rows].contiguous(), at.cuda(), cfg).cpu() if rot else k[rows].cpu()
        pg, off = b.slots(s, old + n, old)
        want_k[1, pg, :, off] = kr
        want_v[1, pg, :, off] = v[rows].cpu()
        want_a[1, pg, :, off] = 0.0
        if rot:
            assert torch.equal(got_q[rows], vx.rope_fwd(q[rows].contiguous(), at.cuda(), cfg))
    same = lambda x, y: torch.equal(x.view(torch.int16 if x.dtype == BF else torch.int32),
                                    y.view(torch.int16 if y.dtype == BF else torch.int32))
    assert same(c.k.cpu(), want_k) and same(c.v.cpu(), want_v) and same(c.acc.cpu(), want_a)
    if rot:                                            # rows of no sequence
        assert torch.all(got_q[:2] == 7.0) and torch.all(got_q[b.starts[-1]:] == 7.0)
    vx.paged_advance(c, b.q_start, b.n, b.max_q, ws=ws)
    assert c.lens.tolist() == [o + n for o, n in zip(olds, news)]
    assert c.pos.tolist() == [o + n + int(d) for o, n, d in zip(olds, news, shift)]
    assert vx.status_check(ws) == 0


def test_append_rotates_q_in_place():
    vx = _vx()
    b = Batch([3, 9], [5, 2], 4, 2, 64, 8, BF)
    gen = torch.Generator().manual_seed(3)
    q, k, v = (_randn((b.n, h, 64), BF, gen).cuda() for h in (4, 2, 2))
    cfg = vx.RopeCfg(theta=1e4, rot_dim=32)
    want = vx.paged_append(b.cache, 0, k, v, b.q_start, b.max_q, rope=cfg, q=q)
    got = q.clone()
    vx.paged_append(b.cache, 0, k, v, b.q_start, b.max_q, rope=cfg, q=got, q_out=got)
    assert torch.equal(got, want)


def test_full_tables_and_bad_pages_are_reported():
    vx = _vx()
    ws = vx.Workspace(1 << 20)
    b = Batch([30, 5], [4, 4], 2, 2, 64, 16, BF)
    c = b.cache
    gen = torch.Generator().manual_seed(4)
    k, v = (_randn((8, 2, 64), BF, gen).cuda() for _ in range(2))
    small = vx.PagedCache(1, c.k.shape[1], 16, 2, 64, 2, 2)              # 32 slots a sequence: two tokens too many
    small.k, small.v = c.k, c.v
    small.table.copy_(c.table[:, :2])
    small.lens.copy_(c.lens)
    before = c.k.clone()
    vx.status_reset(ws)
    vx.paged_append(small, 0, k, v, b.q_start, 4, ws=ws)
    assert vx.status_check(ws) == 1 and "sequence 0" in vx.lib.vx_last_error().decode()
    pg, off = b.slots(0, 32, 30)
    assert torch.equal(c.k.cpu()[0, pg, :, off], k[:2].cpu())
    changed = (c.k.view(torch.int16) != before.view(torch.int16)).any(-1).sum().item()
    assert changed <= (2 + 4) * 2
    vx.status_reset(ws)
    vx.paged_advance(small, b.q_start, 8, 4, ws=ws)
    assert small.lens.tolist() == [32, 9] and vx.status_check(ws) == 1
    for bad in (-1, c.k.shape[1], 2 ** 30):                              # a page that is none: zeros, reported
        d = Batch([20], [3], 2, 2, 64, 16, BF, weights=True)
        d.cache.table[0, 0] = bad
        for vv in (d.k[0], d.v[0]):
            vv[:, :16] = 0
        vx.status_reset(ws)
        o, lse = vx.paged_attn_fwd(d.cache, 0, d.q.cuda(), d.q_start, 3, track=0.0, return_lse=True, ws=ws)
        assert vx.status_check(ws) == 1
        _check_attn(d, o, lse, what="bad page")
        vx.status_reset(ws)
        vx.paged_evict(d.cache, 20, 4, ws=ws)
        assert vx.status_check(ws) == 1
    vx.status_reset(ws)
    assert vx.status_check(ws) == 0


# ---------------------------------------------------------------- attention

_ATTN = [   # olds, news, hq, hkv, D, page, options
    ([0], [1], 1, 1, 64, 16, {}),
    ([0], [1], 8, 1, 128, 16, {}),
    ([70, 0, 15, 16], [1, 1, 1, 1], 4, 2, 64, 16, {}),
    ([4000, 0, 17], [1, 1, 0], 8, 2, 128, 7, {}),
    ([2600], [1], 8, 2, 128, 64, {}),                                    # split keys
    ([2600, 0, 300], [4, 4, 4], 4, 4, 64, 16, dict(window=750)),
    ([900, 5], [8, 3], 8, 2, 128, 50, dict(window=33, prefix=[7, 100])),
    ([900, 5], [6, 6], 10, 2, 64, 1, dict(window=1)),                    # each token sees itself alone
    ([37, 1200], [5, 2], 6, 2, 128, 24, dict(cap=5.0, slopes=True)),
    ([37, 1200], [7, 4], 3, 1, 64, 24, dict(cap=30.0, prefix=[3, 600], window=200)),
    ([0], [33], 1, 1, 64, 16, {}),
    ([0], [40], 8, 8, 128, 16, {}),
    ([0, 100, 127], [127, 1, 129], 2, 1, 64, 16, {}),
    ([0, 513, 2], [257, 300, 90], 3, 1, 128, 128, dict(window=100)),
    ([1500, 0, 777], [65, 300, 0], 8, 2, 64, 48, dict(window=250, prefix=[16, 40, 5])),
    ([3000], [130], 4, 1, 128, 33, {}),                                  # split keys on the tensor cores
    ([200, 0, 64], [100, 260, 70], 12, 4, 64, 48, dict(cap=30.0, slopes=True, prefix=[100, 50, 3])),
    ([200, 0, 64], [100, 260, 70], 5, 1, 128, 8, dict(cap=8.0)),
    ([200, 31], [64, 200], 4, 2, 128, 100, dict(slopes=True, window=70)),
    ([0, 9], [200, 150], 2, 2, 64, 65536, dict(prefix=[500, 40])),       # a prefix behind the sequence's end
    ([300, 8], [90, 33], 4, 2, 64, 16, dict(scale=0.5)),
    ([300, 0], [300, 129], 2, 2, 64, 16, dict(window=1)),                # the warpgroups' tiles part
    ([1000, 77], [256, 300], 1, 1, 128, 128, dict(window=129)),
    ([520, 64], [700, 260], 1, 1, 128, 8, dict(window=40, prefix=[130, 3])),
    ([40, 3, 0], [2, 1, 3], 5, 1, 128, 16, dict(prefix=[9, 3, 0])),      # 9 to 16 rows
]


@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("olds,news,hq,hkv,D,page,opt", _ATTN)
@pytest.mark.parametrize("track", [None, 0.0, 0.5])
def test_attention(dtype, olds, news, hq, hkv, D, page, opt, track):
    vx = _vx()
    if page > 4096 and dtype == F32:
        pytest.skip("the pool of this page size is only built once")
    b = Batch(olds, news, hq, hkv, D, page, dtype, weights=track is not None, lead=1, tail=2)
    opt = dict(opt)
    slopes = prefix = None
    if opt.pop("slopes", False):
        slopes = torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)])
    if "prefix" in opt:
        prefix = opt.pop("prefix")
    ws = vx.Workspace(256)
    vx.status_reset(ws)
    out = torch.full((b.n, hq, D), 3.0, dtype=dtype, device="cuda")
    lse = torch.full((b.n, hq), 3.0, device="cuda")
    vx.paged_attn_fwd(b.cache, 0, b.q.cuda(), b.q_start, b.max_q, max_kv=b.max_kv,
                      prefix=None if prefix is None else torch.tensor(prefix, dtype=torch.int32).cuda(),
                      slopes=None if slopes is None else slopes.cuda(), track=track, out=out, lse=lse, ws=ws, **opt)
    assert vx.status_check(ws) == 0
    _check_attn(b, out, lse, track=track, prefix=prefix, slopes=None if slopes is None else slopes.numpy(), **opt)
    for t in (out, lse):                               # rows of no sequence are left alone
        assert torch.all(t[0] == 3.0) and torch.all(t[b.starts[-1]:] == 3.0)


@pytest.mark.parametrize("dtype,news,D", [(BF, [2, 1], 128), (BF, [70, 200], 64), (F32, [5, 9], 64)])
def test_attention_layers_strides_and_repeats(dtype, news, D):
    # A layer of several, q and o as views of wider rows, no bound on the lengths, the same bits each time.
    vx = _vx()
    b = Batch([600, 45], news, 6, 2, D, 16, dtype, layers=3, weights=True, room=500)
    wide = torch.zeros(b.n, 10, D, dtype=dtype, device="cuda")
    q = wide[:, 4:]
    q.copy_(b.q)
    res = []
    for kv in (0, b.max_kv):
        for _ in range(2):
            pg = torch.zeros(b.n, 8, D, dtype=dtype, device="cuda")
            o, lse = vx.paged_attn_fwd(b.cache, 2, q, b.q_start, b.max_q, max_kv=kv, window=300, track=0.0,
                                       return_lse=True, out=pg[:, 1:7])
            assert not pg[:, 0].any() and not pg[:, 7].any()
            _check_attn(b, o, lse, layer=2, track=0.0, window=300)
            res.append((o.clone(), lse, b.cache.acc[2].clone()))
        assert all(torch.equal(x.nan_to_num(), y.nan_to_num()) for x, y in zip(res[-1], res[-2]))
    for l in (0, 1):
        for s in range(2):
            got = b.gather(b.cache.acc, s, b.olds[s] + b.news[s])[l]
            assert torch.equal(got, b.acc[s][l].T)


@pytest.mark.parametrize("dtype,kv", [(BF, 200), (F32, 77), (BF, 1 << 20)])
def test_a_wrong_bound_on_the_lengths_costs_nothing_but_time(dtype, kv):
    vx = _vx()
    b = Batch([900, 45], [700, 300], 4, 2, 64, 16, dtype, weights=True)
    o, lse = vx.paged_attn_fwd(b.cache, 0, b.q.cuda(), b.q_start, b.max_q, max_kv=kv, track=0.25, return_lse=True)
    _check_attn(b, o, lse, track=0.25)


@pytest.mark.parametrize("dtype,n,D", [(BF, 1, 64), (BF, 100, 64), (BF, 100, 128), (F32, 3, 64)])
def test_queries_that_see_nothing(dtype, n, D):
    # Tokens past the table's slots have no key of their own; with a short window they see nothing at all.
    vx = _vx()
    b = Batch([64], [n], 2, 2, D, 16, dtype)
    c = vx.PagedCache(1, b.cache.k.shape[1], 16, 2, D, 1, 4, dtype=dtype, weights=True)
    c.k, c.v = b.cache.k, b.cache.v
    c.table.copy_(b.cache.table[:, :4])
    c.lens.copy_(b.cache.lens)
    ws = vx.Workspace(1 << 22)
    vx.status_reset(ws)
    o, lse = vx.paged_attn_fwd(c, 0, b.q.cuda(), b.q_start, n, window=1, track=0.0, return_lse=True, ws=ws)
    assert vx.status_check(ws) == 1
    assert not o.any() and torch.all(lse == -float("inf")) and not b.gather(c.acc, 0, 64).any()


@pytest.mark.parametrize("n,D", [(2, 64), (2, 128), (150, 64), (150, 128)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_large_scores_and_nan(n, D, dtype):
    # Scores of some thousands (a softmax that picks single keys), then a NaN that a query must pass on.
    vx = _vx()
    b = Batch([140], [n], 4, 2, D, 16, dtype, scale=30.0)
    o, lse = vx.paged_attn_fwd(b.cache, 0, b.q.cuda(), b.q_start, n, return_lse=True)
    _check_attn(b, o, lse)
    pg, off = b.slots(0, 4, 3)
    b.cache.k[0, pg.cuda(), :, off.cuda()] = float("nan")
    o, lse = vx.paged_attn_fwd(b.cache, 0, b.q.cuda(), b.q_start, n, return_lse=True)
    assert torch.isnan(o).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("dtype,n,D", [(BF, 2, 128), (BF, 150, 128), (BF, 150, 64), (F32, 2, 128), (F32, 70, 128)])
def test_pools_past_32_bit_offsets(dtype, n, D):
    # The sequences' pages at the end of a pool whose bytes and elements need more than 32 bits (5 GB of K).
    vx = _vx()
    b = Batch([300, 45], [n, n], 4, 2, D, 16, dtype, weights=True, room=2 * n)
    small = b.cache
    m = small.k.shape[1]
    P = (5 << 30) // (2 * 16 * D * small.k.element_size()) + m
    c = vx.PagedCache(1, P, 16, 2, D, 2, small.table.shape[1], dtype=dtype, weights=True)
    for name in ("k", "v", "acc"):
        getattr(c, name)[:, -m:] = getattr(small, name)
    c.table.copy_(torch.where(small.table >= 0, small.table + (P - m), small.table))
    c.lens.copy_(small.lens)
    c.pos.copy_(small.pos)
    ws = vx.Workspace(1 << 24)
    vx.status_reset(ws)
    gen = torch.Generator().manual_seed(5)
    row = _randn((2 * n, 4 + 2 * 2, D), dtype, gen).cuda()
    for cache in (small, c):
        q = vx.paged_append(cache, 0, row[:, 4:6], row[:, 6:], b.q_start, n, rope=vx.RopeCfg(theta=1e4), q=row[:, :4],
                            ws=ws)
        cache.out = vx.paged_attn_fwd(cache, 0, q, b.q_start, n, track=0.5, return_lse=True, ws=ws)
        vx.paged_advance(cache, b.q_start, 2 * n, n, ws=ws)
        vx.paged_evict(cache, 200, 20, ws=ws)
    assert vx.status_check(ws) == 0
    for x, y in zip(small.out, c.out):
        assert torch.equal(x, y)
    for name in ("k", "v", "acc"):
        assert torch.equal(getattr(c, name)[:, -m:].nan_to_num(), getattr(small, name).nan_to_num())
        assert not getattr(c, name)[:, :-m].any()
    assert torch.equal(c.lens, small.lens)


def test_rotary_configurations_are_copied_and_pickled():
    import copy
    import pickle
    vx = _vx()
    x, pos = torch.randn(4, 2, 64, device="cuda"), torch.arange(4, device="cuda")
    cfg = vx.RopeCfg(theta=1e4, rot_dim=32)
    want = vx.rope_fwd(x, pos, cfg)
    for other in (copy.deepcopy(cfg), copy.copy(cfg), pickle.loads(pickle.dumps(cfg))):
        assert other == cfg and other._address != cfg._address
        assert torch.equal(vx.rope_fwd(x, pos, other), want)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,D", [(2, 64), (12, 128), (150, 64), (150, 128)])
@pytest.mark.parametrize("scale,cap", [(0.5, 50.0), (1.0, 6.0), (8.0, 2.0), (60.0, 10.0)])
def test_capped_scores_small_and_large(dtype, n, D, scale, cap):
    # Scores well below the cap, around half of it, and far above it (both sides of the kernels' choice of formula).
    vx = _vx()
    b = Batch([140, 9], [n, n], 4, 2, D, 16, dtype, scale=scale, weights=True)
    o, lse = vx.paged_attn_fwd(b.cache, 0, b.q.cuda(), b.q_start, n, cap=cap, track=0.0, return_lse=True)
    _check_attn(b, o, lse, cap=cap, track=0.0)


@pytest.mark.parametrize("dtype,n,D,page,window,prefix", [
    (BF, 2, 64, 16, 40, 5), (BF, 2, 128, 7, 1, 0), (BF, 3, 128, 128, 129, 70), (BF, 150, 64, 128, 40, 3),
    (BF, 150, 128, 16, 33, 0), (BF, 150, 128, 7, 100, 61), (BF, 300, 64, 8, 1, 17), (F32, 2, 64, 16, 40, 5),
    (F32, 6, 128, 7, 1, 0), (F32, 90, 64, 16, 33, 21)])
def test_slots_that_no_query_sees_may_hold_anything(dtype, n, D, page, window, prefix):
    vx = _vx()
    b = Batch([700], [n], 4, 2, D, page, dtype, weights=True)
    pg, off = b.slots(0, 700 - window + 1, prefix)          # between the prefix and the first query's window
    for pool, x in ((b.cache.k, float("nan")), (b.cache.v, float("inf"))):
        pool[0, pg.cuda(), :, off.cuda()] = x
    o, lse = vx.paged_attn_fwd(b.cache, 0, b.q.cuda(), b.q_start, n, window=window, track=0.5, return_lse=True,
                               prefix=torch.tensor([prefix], dtype=torch.int32).cuda())
    _check_attn(b, o, lse, window=window, prefix=[prefix], track=0.5)


@pytest.mark.parametrize("case", ["empty", "none"])
def test_no_rows(case):
    vx = _vx()
    b = Batch([5, 6], [0, 0], 4, 2, 64, 16, BF, weights=True, tail=0 if case == "empty" else 3)
    b.cache.acc.zero_()
    k = torch.zeros(b.n, 2, 64, dtype=BF, device="cuda")
    vx.paged_append(b.cache, 0, k, k, b.q_start, b.n)
    o = vx.paged_attn_fwd(b.cache, 0, b.q.cuda(), b.q_start, b.n, track=0.0, out=torch.ones_like(b.q).cuda())
    vx.paged_advance(b.cache, b.q_start, b.n, b.n)
    assert torch.all(o == 1.0) and b.cache.lens.tolist() == [5, 6] and not b.cache.acc.any()


def test_attention_refusals():
    vx = _vx()
    b = Batch([5, 6], [3, 2], 4, 2, 64, 16, BF)
    q, go = b.q.cuda(), lambda **k: vx.paged_attn_fwd(b.cache, 0, **{**dict(q=q, q_start=b.q_start, max_q=3), **k})
    for kw, exc, word in [
            (dict(q=q.float()), TypeError, "q must be"), (dict(q=q[0]), ValueError, "heads"),
            (dict(q=q[:, :3]), vx.VxError, "multiple"), (dict(q_start=b.q_start[:2]), ValueError, "q_start"),
            (dict(q_start=b.q_start.long()), TypeError, "q_start"), (dict(out=q), ValueError, "overlaps"),
            (dict(prefix=torch.zeros(3, dtype=torch.int32, device="cuda")), ValueError, "prefix"),
            (dict(slopes=torch.zeros(2, device="cuda")), ValueError, "slopes"),
            (dict(track=0.0), vx.VxError, "acc"), (dict(window=-1), vx.VxError, "window"),
            (dict(cap=-1.0), vx.VxError, "cap"), (dict(prefix=torch.zeros(2, dtype=torch.int32)), ValueError, "CUDA"),
            (dict(q=torch.zeros(5, 4, 128, dtype=BF, device="cuda")), ValueError, "q must be"),
            (dict(q=torch.zeros(5 * 4 * 68, dtype=BF, device="cuda")[2:].as_strided((5, 4, 64), (272, 68, 1))),
             vx.VxError, "16-byte"),
            (dict(lse=torch.zeros(5, 3, device="cuda")), ValueError, "lse")]:
        with pytest.raises(exc, match=word):
            go(**kw)
    with pytest.raises(vx.VxError, match="layer"):
        vx.paged_attn_fwd(b.cache, 1, q, b.q_start, 3)
    with pytest.raises(ValueError, match="k must be"):
        vx.paged_append(b.cache, 0, q, q, b.q_start, 3)
    with pytest.raises(vx.VxError, match="rope"):
        vx.paged_append(b.cache, 0, q[:, :2], q[:, :2], b.q_start, 3, q=q)
    with pytest.raises(vx.VxError, match="acc"):
        vx.paged_evict(b.cache, 4, 2)


# ----------------------------------------------------------------- eviction

@pytest.mark.parametrize("dtype", [F32, BF])
@pytest.mark.parametrize("lens,hkv,D,page,keep,recent,kind", [
    ([1], 1, 64, 16, 1, 0, "rand"), ([1, 0, 2], 2, 64, 16, 1, 1, "rand"),
    ([100, 33, 29, 30], 2, 64, 16, 30, 10, "rand"), ([100, 33], 2, 128, 7, 30, 30, "rand"),
    ([100, 33], 2, 128, 7, 30, 50, "rand"), ([1500, 3000, 700], 3, 64, 50, 999, 1, "ties"),
    ([5000, 1025, 1024], 1, 64, 64, 1024, 0, "ties"), ([40, 70], 2, 64, 16, 20, 5, "odd"),
    ([40, 70], 2, 64, 16, 0, 5, "rand"), ([40, 70], 2, 64, 16, 1000, 5, "rand"),
    ([2600, 2100], 2, 64, 33, 2050, 7, "zero"), ([11000, 9000], 1, 64, 128, 3001, 64, "rand"),
    ([60000], 1, 64, 512, 20000, 100, "ties")])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict(dtype, lens, hkv, D, page, keep, recent, kind, in_place):
    vx = _vx()
    b = Batch(lens, [0] * len(lens), 1, hkv, D, page, dtype, layers=2, weights=True)
    c = b.cache
    gen = torch.Generator().manual_seed(8)
    for s, n in enumerate(lens):
        a = b.acc[s]
        if kind == "ties":
            a.copy_(torch.randint(0, 4, a.shape, generator=gen).float() / 4)
        if kind == "zero":
            a.zero_()
        if kind == "odd" and n:
            for j, x in enumerate((float("nan"), float("inf"), -float("inf"), -0.0, 0.0, -1.0, 1e-40)):
                a[..., j::11] = x
        pg, off = b.slots(s, n)
        c.acc[:, pg.cuda(), :, off.cuda()] = a.permute(2, 0, 1).cuda()
    c.lens.copy_(torch.tensor(lens))
    c.pos.copy_(torch.tensor(lens) * 3)
    S = len(lens)
    kept = torch.full((2, S, hkv, keep), -7, dtype=torch.int32, device="cuda")
    dst, table = c, b.table
    if not in_place:
        m = max(1, -(-max(min(n, keep) for n in lens) // page))
        dst = vx.PagedCache(2, S * m, page, hkv, D, S, m, dtype=dtype, weights=True)
        dst.table.copy_(torch.randperm(S * m, generator=gen).reshape(S, m))
        table = dst.table.cpu().numpy()
    ws = vx.Workspace(256)
    vx.status_reset(ws)
    vx.paged_evict(c, keep, recent, dst=None if in_place else dst, kept=kept, ws=ws)
    assert vx.status_check(ws) == 0
    assert dst.lens.tolist() == [min(n, keep) for n in lens] and dst.pos.tolist() == [3 * n for n in lens]
    if not in_place:
        assert c.lens.tolist() == lens
    dk, dv, da = dst.k.cpu(), dst.v.cpu(), dst.acc.cpu()
    kept = kept.cpu().numpy()
    for s, n in enumerate(lens):
        m = min(n, keep)
        j = np.arange(m)
        pg, off = torch.from_numpy(table[s][j // page].astype(np.int64)), torch.from_numpy(j % page)
        for l in range(2):
            for h in range(hkv):
                idx = paged.evict(b.acc[s][l, h].numpy(), keep, recent)
                assert np.array_equal(kept[l, s, h, :m], idx) and np.all(kept[l, s, h, m:] == -7)
                assert torch.equal(dk[l, pg, h, off], b.k[s][l, idx, h])
                assert torch.equal(dv[l, pg, h, off], b.v[s][l, idx, h])
                assert torch.equal(da[l, pg, h, off].view(torch.int32), b.acc[s][l, h, idx].view(torch.int32))


# ---------------------------------------------------------------- together

def _decode(vx, c, qkv, q_start, n, max_q, cfg, hq, hkv, **kw):
    q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    for l in range(c.k.shape[0]):
        qr = vx.paged_append(c, l, k, v, q_start, max_q, rope=cfg, q=q)
        o = vx.paged_attn_fwd(c, l, qr, q_start, max_q, track=0.9, **kw)
    vx.paged_advance(c, q_start, n, max_q)
    return o


@pytest.mark.parametrize("dtype", [BF, F32])
def test_prompt_steps_and_evictions_together(dtype):
    # Two layers: prompts, then steps of two tokens; after every third step the sequences are cut to 40 tokens.
    vx = _vx()
    hq, hkv, D, page, S = 4, 2, 64, 16, 3
    c = vx.PagedCache(2, 40, page, hkv, D, S, 12, dtype=dtype, weights=True)
    gen = torch.Generator().manual_seed(77)
    c.table.copy_(torch.randperm(40, generator=gen)[:36].reshape(S, 12))
    cfg = vx.RopeCfg(theta=1e4, scaling="linear", factor=2.0)
    model = [dict(k=np.zeros((2, 0, hkv, D)), v=np.zeros((2, 0, hkv, D)), acc=np.zeros((2, hkv, 0)), pos=0)
             for _ in range(S)]
    for step in range(8):
        news = [70, 3, 41] if step == 0 else [2, 2, 2]
        starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int32)
        qkv = _randn((sum(news), hq + 2 * hkv, D), dtype, gen)
        got = _decode(vx, c, qkv.cuda(), torch.from_numpy(starts).cuda(), sum(news), max(news), cfg, hq, hkv,
                      window=50, prefix=torch.full((S,), 4, dtype=torch.int32).cuda())
        for s in range(S):
            m, rows = model[s], slice(starts[s], starts[s] + news[s])
            x = _host(qkv[rows])
            at = m["pos"] + np.arange(news[s])
            rot = lambda z: torch.from_numpy(paged.rope(z, at, theta=1e4, scaling="linear", factor=2.0)).to(dtype)
            q, k = _host(rot(x[:, :hq])), _host(rot(x[:, hq:hq + hkv]))
            m["pos"] += news[s]
            old = m["k"].shape[1]
            for name, new in (("k", k), ("v", x[:, hq + hkv:])):
                m[name] = np.concatenate([m[name], np.broadcast_to(new, (2, *new.shape))], 1)
            m["acc"] = np.concatenate([m["acc"], np.zeros((2, hkv, news[s]))], 2)
            for l in range(2):
                r = paged.attention(q, m["k"][l], m["v"][l], old, window=50, prefix=4)
                m["acc"][l] = 0.9 * m["acc"][l] + r["weights"]
            # A rounding of q or k that falls the other way moves a score by smax times a step (2^-7).
            step_size = 2 * B16 if dtype == BF else 64 * U
            tol = r["absv"] * (4 * step_size * r["smax"][..., None] + 2 * step_size) + step_size
            _within(_host(got[rows]), r["o"], tol, f"step {step}, sequence {s}")
        assert c.lens.tolist() == [m["k"].shape[1] for m in model]
        assert c.pos.tolist() == [m["pos"] for m in model]
        if step % 3 == 2:
            kept = torch.full((2, S, hkv, 40), -1, dtype=torch.int32, device="cuda")
            vx.paged_evict(c, 40, 8, kept=kept)
            for s, m in enumerate(model):              # the cache's own choice, checked above, is followed
                n = min(40, m["k"].shape[1])
                idx = kept.cpu().numpy()[:, s, :, :n]
                new = {t: np.zeros((2, n, hkv, D)) for t in ("k", "v")}
                acc = np.zeros((2, hkv, n))
                for l in range(2):
                    for h in range(hkv):
                        for t in ("k", "v"):
                            new[t][l, :, h] = m[t][l, idx[l, h], h]
                        acc[l, h] = m["acc"][l, h, idx[l, h]]
                m.update(new, acc=acc)
            assert c.lens.tolist() == [m["k"].shape[1] for m in model]


@pytest.mark.parametrize("dtype,n", [(BF, 2), (BF, 40), (F32, 2)])
def test_captured_steps_replay_and_share_nothing(dtype, n):
    # Two captured graphs on caches of their own, replayed at the same time on two streams: each gives what eager
    # calls give.
    vx = _vx()
    hq, hkv, D = 4, 2, 64
    cfg = vx.RopeCfg(theta=1e4)

    def make(seed):
        b = Batch([300, 45], [n, n], hq, hkv, D, 16, dtype, seed=seed, weights=True, room=8 * n)
        qkv = _randn((2 * n, hq + 2 * hkv, D), dtype, torch.Generator().manual_seed(seed)).cuda()
        return b, qkv

    def step(b, qkv):
        o = _decode(vx, b.cache, qkv, b.q_start, 2 * n, n, cfg, hq, hkv)
        vx.paged_evict(b.cache, 320, 30)
        return o

    want = []
    for seed in (1, 2):
        b, qkv = make(seed)
        for _ in range(4):
            o = step(b, qkv)
        want.append((o.clone(), b.cache.lens.clone(), b.cache.k.clone()))
    torch.cuda.synchronize()
    live = []
    for seed in (1, 2):
        b, qkv = make(seed)
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            step(b, qkv)                               # first pass eager
        st.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            o = step(b, qkv)
        live.append((b, qkv, st, g, o))
    for _ in range(3):
        for b, qkv, st, g, o in live:
            with torch.cuda.stream(st):
                g.replay()
    torch.cuda.synchronize()
    for (b, _, _, _, o), (wo, wl, wk) in zip(live, want):
        assert torch.equal(o, wo) and torch.equal(b.cache.lens, wl)
        assert torch.equal(b.cache.k.nan_to_num(), wk.nan_to_num())
