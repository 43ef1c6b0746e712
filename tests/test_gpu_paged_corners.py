"""GPU tests of the paged-cache operators' corners, against the same float64
statement and with the same tolerances as test_gpu_paged.py."""
import numpy as np
import pytest
import torch

import oracle.paged as paged
from test_gpu_paged import BF, F32, U, Batch, _check_attn, _host, _randn, _vx, _within

pytestmark = pytest.mark.gpu


# ------------------------------------------- non-finite keys and queries

@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,D", [(2, 64), (2, 128), (6, 64), (12, 128), (150, 64), (150, 128)])
@pytest.mark.parametrize("cap", [0.0, 2.0, 1e4])
@pytest.mark.parametrize("kind", ["nan", "inf", "one inf"])
def test_a_key_that_is_not_finite_reaches_no_query_that_does_not_see_it(dtype, n, D, cap, kind):
    # The last token's key, V finite: the tokens before it do not see it.  Scores far above the cap of 2, far below 1e4.
    vx = _vx()
    b = Batch([140, 9], [n, n], 4, 2, D, 16, dtype, scale=8.0, weights=True)
    for s, old in enumerate(b.olds):
        at = slice(0, 1) if kind == "one inf" else slice(None)
        x = float("nan") if kind == "nan" else float("inf")
        b.k[s][0, -1, :, at] = x
        pg, off = b.slots(s, old + n, old + n - 1)
        b.cache.k[0, pg.cuda(), :, off.cuda(), at] = x
    o, lse = vx.paged_attn_fwd(b.cache, 0, b.q.cuda(), b.q_start, n, cap=cap, track=0.0, return_lse=True)
    with np.errstate(invalid="ignore"):
        for s, old in enumerate(b.olds):
            rows = slice(b.starts[s], b.starts[s] + n - 1)     # without the last token: nothing is off there
            r = paged.attention(_host(b.q)[rows], _host(b.k[s][0])[:-1], _host(b.v[s][0])[:-1], old, cap=cap)
            ds = ((D + 8) * r["smax"]) * U + cap * 2.0 ** -21
            rel = 2 * (ds + 2.0 ** -21) + (old + n + 8) * U + (2.0 ** -8 if dtype == BF else 0.0)
            tol = r["absv"] * rel[..., None] * 1.01 + (2.0 ** -8 if dtype == BF else 2 * U) * np.abs(r["o"]) + 1e-30
            _within(_host(o)[rows], r["o"], tol, f"o of sequence {s}")
            dz = ds + 2.0 ** -20 + (old + n + 8) * U + 4 * U * np.abs(r["lse"])
            _within(_host(lse)[rows], r["lse"], dz, f"lse of sequence {s}")
            last = b.starts[s] + n - 1
            if kind != "one inf":                              # inf - inf, or NaN: the query that sees it passes it on
                assert torch.isnan(o[last]).all() and torch.isnan(lse[last]).all()


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,D", [(2, 64), (2, 128), (4, 64), (12, 128), (18, 64), (150, 64), (150, 128)])
@pytest.mark.parametrize("cap", [0.0, 2.0])
@pytest.mark.parametrize("hq", [4, 2])
def test_a_query_that_is_not_finite_leaves_the_weights_of_slots_it_does_not_see(dtype, n, D, cap, hq):
    # One head of one token is NaN, under a window: the slots after it and before its window, and the other K/V head.
    vx = _vx()
    old, window, t = 140, 40, n // 2 - 1
    b = Batch([old], [n], hq, 2, D, 16, dtype, scale=8.0, weights=True)
    q = b.q.clone()
    q[t, 0] = float("nan")
    o, lse = vx.paged_attn_fwd(b.cache, 0, q.cuda(), b.q_start, n, window=window, cap=cap, track=0.0, return_lse=True)
    assert torch.isnan(o[t, 0]).all() and torch.isnan(lse[t, 0])
    assert not torch.isnan(o[t, 1:]).any() and not torch.isnan(lse[t, 1:]).any()
    r = paged.attention(_host(b.q), _host(b.k[0][0]), _host(b.v[0][0]), old, window=window, cap=cap)
    ds = ((D + 8) * r["smax"]) * U + cap * 2.0 ** -21
    dz = ds + 2.0 ** -20 + (old + n + 8) * U + 4 * U * np.abs(r["lse"])
    rel = ds.max() + dz.max() + 2.0 ** -20 + n * 2 * U
    got = _host(b.gather(b.cache.acc, 0, old + n))[0].T
    seen = paged.seen(old, n, window)[t]
    want = r["weights"].copy()                                 # a hidden slot has no part of the query's in it
    want[0, seen] = np.nan
    _within(got, want, 1.01 * r["weights"] * rel + 4 * U * r["weights"] + 1e-30, "weights")


# ------------------------------------------------------------------ same bits

@pytest.mark.parametrize("D,page", [(64, 16), (128, 16), (64, 50), (128, 50)])
def test_what_earlier_calls_left_in_shared_memory_changes_no_bit(D, page):
    # Capped scores over lists that end inside a tile, behind calls whose keys are large, tiny or not finite.
    vx = _vx()
    b = Batch([30] * 60, [40] * 60, 4, 2, D, page, BF, weights=True, scale=1.5)
    q, res = b.q.cuda(), []
    full = Batch([88] * 60, [40] * 60, 4, 2, D, page, BF)
    for x in (0.0, 1e30, 3.0, float("nan"), -1e30, float("inf")):
        full.cache.k.fill_(x)
        vx.paged_attn_fwd(full.cache, 0, full.q.cuda(), full.q_start, 40)
        o, lse = vx.paged_attn_fwd(b.cache, 0, q, b.q_start, 40, cap=12.0, track=0.0, return_lse=True)
        res.append((o, lse, b.cache.acc.clone()))
    _check_attn(b, *res[0][:2], cap=12.0)
    for r in res[1:]:
        assert all(torch.equal(x.nan_to_num(), y.nan_to_num()) for x, y in zip(r, res[0]))


# ------------------------------------------------------------ fp32 throughout

@pytest.mark.parametrize("n,hq,kv", [(1, 2, 0), (1, 2, 16), (4, 4, 0), (12, 2, 0), (70, 4, 0)])
def test_fp32_weights_below_the_smallest_normal_number_are_not_flushed(n, hq, kv):
    # Scores 0 and -92: a weight of exp(-92) = 1.1e-40.
    vx = _vx()
    old, D = 40, 64
    b = Batch([old], [n], hq, 2, D, 16, F32, weights=True)
    k, q = torch.zeros(old + n, 2, D), torch.zeros(n, hq, D)
    k[1:old, :, 0] = -92.0
    k[old:, :, 0] = -500.0
    q[..., 0] = 1.0
    pg, off = b.slots(0, old + n)
    b.cache.k[0, pg.cuda(), :, off.cuda()] = k.cuda()
    vx.paged_attn_fwd(b.cache, 0, q.cuda(), b.q_start, n, max_kv=kv, scale=1.0, track=0.0)
    got = _host(b.gather(b.cache.acc, 0, old + n))[0]
    want = n * (hq // 2) * np.exp(-92.0)
    # The score's rounding 92 * 2^-24 * log2 e, exp2's, and a denormal's step for each row's weight.
    tol = want * (92 * 4 * U + 2.0 ** -20) + n * (hq // 2) * 2.0 ** -149
    _within(got[1:old], np.full((old - 1, 2), want), tol, "weights")
    assert not got[old:].any()


# -------------------------------------------------------------- far angles

def _exact_angles(pos, rot, theta, scaling, factor, orig_len):
    """pos * f_m mod 2 pi in 60 digits, and the factor on cosine and sine; beta 32 and 1."""
    from decimal import Decimal as Dec, getcontext
    getcontext().prec = 60
    pi = Dec("3.14159265358979323846264338327950288419716939937510582097494459")
    theta, factor, ms = Dec(theta), Dec(factor), 1.0
    if scaling == "ntk":
        theta *= (factor.ln() * rot / (rot - 2)).exp()
    out = []
    for m in range(rot // 2):
        f = (theta.ln() * (-2 * m) / rot).exp()
        if scaling == "linear":
            f /= factor
        if scaling == "yarn":
            g = min(max((orig_len * f / (2 * pi) - 1) / 31, Dec(0)), Dec(1))
            f = g * f + (1 - g) * f / factor
            ms = 0.1 * np.log(float(factor)) + 1.0
        out.append([float(Dec(int(p)) * f % (2 * pi)) for p in pos])
    return np.array(out).T, ms


@pytest.mark.parametrize("rot,theta,scaling,factor,orig_len", [
    (64, 1e6, "none", 1.0, 0), (128, 1e4, "none", 1.0, 0), (64, 1.0, "none", 1.0, 0), (128, 5e5, "linear", 3.0, 0),
    (64, 1e6, "ntk", 4.0, 0), (128, 1e6, "yarn", 4.0, 32768), (34, 1e4, "yarn", 8.0, 2048)])
def test_rotary_angles_of_far_positions(rot, theta, scaling, factor, orig_len):
    # The bound that vx.h states: pi 2^-25 and |pos| 2^-61 turns; sine and cosine of an angle off by e are off by e.
    vx = _vx()
    pos = np.array([0, 1, -1, 12345, 2 ** 20 + 3, -(2 ** 31) - 5, 2 ** 35 - 1, 2 ** 40 + 12345, -(2 ** 45) + 7, 2 ** 50 + 1])
    x = torch.zeros(len(pos), 1, rot, device="cuda")
    x[..., :rot // 2] = 1.0                                  # y = (cos, sin), each rounded twice, sincos 2 U
    cfg = vx.RopeCfg(theta=theta, scaling=scaling, factor=factor, orig_len=orig_len)
    got = _host(vx.rope_fwd(x, torch.from_numpy(pos).cuda(), cfg))[:, 0]
    ang, ms = _exact_angles(pos, rot, theta, scaling, factor, orig_len)
    tol = ms * (np.pi * 2.0 ** -25 + np.abs(pos.astype(np.float64))[:, None] * 2.0 ** -61 * 2 * np.pi + 4 * U)
    _within(got[:, :rot // 2], ms * np.cos(ang), tol, "cosines")
    _within(got[:, rot // 2:], ms * np.sin(ang), tol, "sines")


def test_rotary_angles_wrap_exactly():
    # theta 1: all frequencies are 1, one turn's fraction is known to the bit and wraps in 64 bits at any position.
    vx = _vx()
    from decimal import Decimal as Dec, getcontext
    getcontext().prec = 60
    pi = Dec("3.14159265358979323846264338327950288419716939937510582097494459")
    turns = int(Dec(2) ** 64 / (2 * pi) + Dec("0.5"))
    pos = [2 ** 62 + 1, -(2 ** 63), 2 ** 63 - 1, -(2 ** 55) - 3]
    x = torch.zeros(len(pos), 1, 64, device="cuda")
    x[..., :32] = 1.0
    got = _host(vx.rope_fwd(x, torch.tensor(pos).cuda(), vx.RopeCfg(theta=1.0)))[:, 0]
    for r, p in enumerate(pos):
        # f = 1 is exact; 2 pi and the quotient are rounded to 64-bit mantissas: turns may be off by one
        angs = [float(Dec(p * (turns + e) % 2 ** 64) / 2 ** 63 * pi) for e in (-1, 0, 1)]
        tol = np.pi * 2.0 ** -25 + 4 * U
        assert any(np.all(np.abs(got[r, :32] - np.cos(a)) <= tol) and np.all(np.abs(got[r, 32:] - np.sin(a)) <= tol)
                   for a in angs)


# ---------------------------------------------- sequences without new tokens

@pytest.mark.parametrize("dtype,n", [(BF, 1), (BF, 12), (BF, 150), (F32, 1), (F32, 70)])
@pytest.mark.parametrize("track", [0.0, 0.5])
def test_weights_of_sequences_without_rows_stay(dtype, n, track):
    vx = _vx()
    b = Batch([90, 50, 7], [0, n, 0], 4, 2, 64, 16, dtype, weights=True)
    vx.paged_attn_fwd(b.cache, 0, b.q.cuda(), b.q_start, n, track=track)
    for s in (0, 2):
        assert torch.equal(b.gather(b.cache.acc, s, b.olds[s])[0], b.acc[s][0].T)
    assert not torch.equal(b.gather(b.cache.acc, 1, 50)[0], b.acc[1][0].T[:50])


# ------------------------------------------------------- status and scratch

def test_a_full_table_is_still_reported_after_the_workspace_has_grown():
    vx = _vx()
    b = Batch([30], [4], 2, 2, 64, 16, BF, weights=True)
    c = vx.PagedCache(1, b.cache.k.shape[1], 16, 2, 64, 1, 2, weights=True)      # 32 slots: two tokens too many
    c.table.copy_(b.cache.table[:, :2])
    c.lens.copy_(b.cache.lens)
    ws = vx.Workspace(256)
    vx.status_reset(ws)
    k = _randn((4, 2, 64), BF, torch.Generator().manual_seed(1)).cuda()
    vx.paged_append(c, 0, k, k, b.q_start, 4, ws=ws)
    c.lens.fill_(28)                                                            # nothing wrong from here on
    vx.paged_attn_fwd(c, 0, b.q.cuda(), b.q_start, 4, track=0.0, ws=ws)
    assert ws.buf.numel() > 256 and vx.status_check(ws) == 1


def test_a_captured_workspace_is_not_handed_out_again_when_it_grows():
    vx = _vx()
    b = Batch([300, 45], [40, 40], 4, 2, 64, 16, BF, weights=True)
    q, ws = b.q.cuda(), vx.Workspace(256)
    call = lambda: vx.paged_attn_fwd(b.cache, 0, q, b.q_start, 40, max_kv=b.max_kv, track=0.0, return_lse=True, ws=ws)
    st = torch.cuda.Stream()
    with torch.cuda.stream(st):
        want = [t.clone() for t in call()] + [b.cache.acc.clone()]
    st.synchronize()
    size, at = ws.buf.numel(), ws.buf.data_ptr()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=st):
        out = call()
    ws.get(4 * size)
    others = [torch.zeros(size, dtype=torch.uint8, device="cuda") for _ in range(8)]
    assert at not in [t.data_ptr() for t in others]
    b.cache.acc.zero_()
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    assert not any(t.any() for t in others)
    for x, y in zip([*out, b.cache.acc], want):
        assert torch.equal(x.nan_to_num(), y.nan_to_num())


def test_tensors_resized_in_place_are_described_again():
    # Host side only: nothing is launched on the old description.
    vx = _vx()
    make = lambda: vx.PagedCache(2, 8, 16, 2, 64, 3, 4, weights=True, device="cuda")
    c = make()
    assert (c.c().n_seqs, c.c().max_pages, c.c().n_pages) == (3, 4, 8)
    c.table.resize_(3, 2)
    assert c.c().max_pages == 2
    c.table.resize_(2, 2), c.lens.resize_(2), c.pos.resize_(2)
    assert c.c().n_seqs == 2
    for name in ("k", "v"):
        getattr(c, name).resize_(2, 5, 2, 16, 64)
    c.acc.resize_(2, 5, 2, 16)
    assert c.c().n_pages == 5
    for change, word in ((lambda c: c.lens.resize_(2), "lens"), (lambda c: c.pos.resize_(0), "pos"),
                         (lambda c: c.v.resize_(2, 5, 2, 16, 64), "k and v"), (lambda c: c.acc.resize_(2), "acc"),
                         (lambda c: c.table.t_(), "contiguous"), (lambda c: c.table.resize_(12), "table")):
        c = make()
        c.c()
        change(c)
        with pytest.raises(ValueError, match=word):
            c.c()
        with pytest.raises(ValueError, match=word):
            vx.paged_advance(c, torch.zeros(4, dtype=torch.int32, device="cuda"), 0, 0)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n,D,page", [(2, 64, 16), (12, 128, 16), (150, 64, 16), (150, 128, 64), (150, 128, 7), (70, 64, 256)])
def test_pages_outside_the_pool_read_as_zeros_and_are_reported(dtype, n, D, page):
    vx = _vx()
    b = Batch([300, 45], [n, n], 4, 2, D, page, dtype, weights=True)
    c, pages = b.cache, b.cache.k.shape[1]
    ws = vx.Workspace(1 << 24)
    first = min(64 // page, b.olds[0] // page - 1)
    for bad in (-1, pages, 2 ** 31 - 1, -2 ** 31):
        good = c.table[0, first].clone()
        c.table[0, first] = bad
        rows = slice(first * page, (first + 1) * page)
        k, v = b.k[0][:, rows].clone(), b.v[0][:, rows].clone()
        b.k[0][:, rows], b.v[0][:, rows] = 0, 0
        vx.status_reset(ws)
        o, lse = vx.paged_attn_fwd(c, 0, b.q.cuda(), b.q_start, n, return_lse=True, ws=ws)
        assert vx.status_check(ws) == 1 and "sequence 0" in vx.lib.vx_last_error().decode()
        _check_attn(b, o, lse)
        c.table[0, first] = good
        b.k[0][:, rows], b.v[0][:, rows] = k, v
    acc = c.acc.clone()
    c.table[0, first] = -1                                   # the weights of the other slots, none written for the page
    vx.status_reset(ws)
    vx.paged_attn_fwd(c, 0, b.q.cuda(), b.q_start, n, track=0.0, ws=ws)
    assert vx.status_check(ws) == 1
    lost = int(b.table[0][first])
    assert torch.equal(c.acc[:, lost].nan_to_num(), acc[:, lost].nan_to_num())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("n", [2, 12, 150])
def test_lengths_outside_the_table_are_clamped_and_reported(dtype, n):
    vx = _vx()
    b = Batch([100, 45], [n, n], 4, 2, 64, 16, dtype, weights=True)
    c, q, ws = b.cache, b.q.cuda(), vx.Workspace(1 << 24)
    gen = torch.Generator().manual_seed(6)
    k, v = (_randn((b.n, 2, 64), dtype, gen).cuda() for _ in range(2))
    cap = c.table.shape[1] * 16
    vx.paged_append(c, 0, k, v, b.q_start, n)
    want = vx.paged_attn_fwd(c, 0, q, b.q_start, n, track=0.0, return_lse=True)
    acc = b.gather(c.acc, 1, 45 + n)
    for bad in (-1, -2 ** 63, cap + 1, 2 ** 40, 2 ** 63 - 1):
        c.lens.copy_(torch.tensor([bad, 45]))
        calls = [lambda: vx.paged_append(c, 0, k, v, b.q_start, n, ws=ws),
                 lambda: vx.paged_attn_fwd(c, 0, q, b.q_start, n, track=0.0, return_lse=True, ws=ws),
                 lambda: vx.paged_advance(c, b.q_start, b.n, n, ws=ws)]
        for i, call in enumerate(calls):
            vx.status_reset(ws)
            got = call()
            assert vx.status_check(ws) == 1 and "sequence 0" in vx.lib.vx_last_error().decode()
            if i == 1:                                       # the other sequence does not notice
                for x, y in zip(got, want):
                    assert torch.equal(x[n:], y[n:])
                assert torch.equal(b.gather(c.acc, 1, 45 + n), acc)
        assert c.lens.tolist() == [min(n, cap) if bad < 0 else cap, 45 + n]
        c.lens.copy_(torch.tensor([bad, 45]))
        dst = vx.PagedCache(1, c.k.shape[1], 16, 2, 64, 2, c.table.shape[1], dtype=dtype, weights=True)
        dst.table.copy_(torch.arange(dst.table.numel()).reshape(dst.table.shape) % c.k.shape[1])
        dst.table[1] = torch.arange(dst.table.shape[1]) + c.k.shape[1] - dst.table.shape[1]
        vx.status_reset(ws)
        vx.paged_evict(c, 10, 4, dst=dst, ws=ws)
        assert vx.status_check(ws) == 1 and dst.lens.tolist() == [0 if bad < 0 else 10, 10]


# -------------------------------------------------- tensors in one fused row

def test_outputs_may_be_other_heads_of_the_inputs_rows():
    vx = _vx()
    b = Batch([30, 9], [5, 3], 4, 2, 64, 16, BF)
    cfg, gen = vx.RopeCfg(theta=1e4), torch.Generator().manual_seed(2)
    row = _randn((8, 12, 64), BF, gen).cuda()
    k, v = (_randn((8, 2, 64), BF, gen).cuda() for _ in range(2))
    pos = torch.arange(8, device="cuda")
    calls = {"rope_fwd": lambda q, out: vx.rope_fwd(q, pos, cfg, out=out),
             "append": lambda q, out: vx.paged_append(b.cache, 0, k, v, b.q_start, 5, rope=cfg, q=q, q_out=out),
             "attn": lambda q, out: vx.paged_attn_fwd(b.cache, 0, q, b.q_start, 5, out=out)}
    for name, call in calls.items():
        want = call(row[:, 4:8].clone(), None)
        for at in (0, 8):                              # before and behind the input's heads
            x = row.clone()
            got = call(x[:, 4:8], x[:, at:at + 4])
            rest = [i for i in range(12) if not at <= i < at + 4]
            assert torch.equal(got, want) and torch.equal(x[:, rest], row[:, rest]), name
        x = torch.zeros(9, 12, 64, dtype=BF, device="cuda")
        wrapped = torch.as_strided(x, (8, 4, 64), (768, 64, 1), 11 * 64)       # from a row's last head into the next row
        for q, bad in ((x[:8, 4:8], x[:8, 5:9]), (x[:8, 4:8], x[:8, 1:5]), (x[:8, 4:8], x[:8, 7:11]),
                       (x[:8, 4:8], x[1:, 4:8]), (x[:8, 0:4], wrapped), (wrapped, x[:8, 0:4])):
            with pytest.raises(ValueError, match="overlaps"):
                call(q, bad)


# ----------------------------------------------------------------- refusals

def test_a_kept_tensor_of_another_size_is_refused():
    vx = _vx()
    b = Batch([40, 70], [0, 0], 1, 2, 64, 16, BF, weights=True)
    kept = lambda *shape: torch.full(shape, -7, dtype=torch.int32, device="cuda")
    before = b.cache.lens.tolist()
    # 4 (sequence, head) pairs times 2^62 + 1 is 4 in 64 bits, times 2^62 nothing
    for keep, k in ((20, kept(0)), (20, kept(1, 2, 2, 19)), (20, kept(2, 2, 2, 20)), ((1 << 62) + 1, kept(4)),
                    (1 << 62, kept(0)), (1 << 61, kept(0))):
        with pytest.raises(ValueError, match="kept"):
            vx.paged_evict(b.cache, keep, 5, kept=k)
    with pytest.raises(vx.VxError, match="keep"):
        vx.paged_evict(b.cache, -1, 5, kept=kept(0))
    assert b.cache.lens.tolist() == before
    vx.paged_evict(b.cache, 0, 5, kept=kept(1, 2, 2, 0))
    assert b.cache.lens.tolist() == [0, 0]


def test_outputs_whose_rows_overlap_are_refused():
    vx = _vx()
    b = Batch([30, 9], [5, 3], 4, 2, 64, 16, BF)
    cfg, q = vx.RopeCfg(theta=1e4), b.q.cuda()
    k, v = (torch.zeros(8, 2, 64, dtype=BF, device="cuda") for _ in range(2))
    pos = torch.arange(8, device="cuda")
    calls = [lambda q, out: vx.rope_fwd(q, pos, cfg, out=out),
             lambda q, out: vx.paged_append(b.cache, 0, k, v, b.q_start, 5, rope=cfg, q=q, q_out=out),
             lambda q, out: vx.paged_attn_fwd(b.cache, 0, q, b.q_start, 5, out=out)]
    new = lambda *shape: torch.zeros(shape, dtype=BF, device="cuda")
    for call in calls:
        want = call(q, None)
        for bad in (new(1, 4, 64).expand(8, 4, 64), new(8, 1, 64).expand(8, 4, 64), new(64).expand(8, 4, 64),
                    torch.as_strided(new(4096), (8, 4, 64), (192, 64, 1)),
                    torch.as_strided(new(4096), (8, 4, 64), (256, 32, 1))):
            with pytest.raises(ValueError, match="overlap"):
                call(q, bad)
        heads_first = new(4, 8, 64).transpose(0, 1)
        padded = new(8, 5, 3, 64)[:, 1:, 2]
        for good in (heads_first, padded):
            call(q, good)
            assert torch.equal(good, want)
    x = new(1, 4, 64).expand(8, 4, 64)                 # as an input it may be
    vx.rope_fwd(x, pos, cfg)
    with pytest.raises(ValueError, match="overlap"):
        vx.rope_fwd(x, pos, cfg, out=x)


def test_an_output_for_no_queries_is_refused():
    vx = _vx()
    b = Batch([30], [5], 4, 2, 64, 16, BF)
    k = torch.zeros(5, 2, 64, dtype=BF, device="cuda")
    with pytest.raises(ValueError, match="q_out"):
        vx.paged_append(b.cache, 0, k, k, b.q_start, 5, rope=vx.RopeCfg(), q_out=torch.empty_like(b.q.cuda()))


# ----------------------------------------------------------------- eviction

@pytest.mark.parametrize("cap,lens,lanes", [(50000, 50000, 160), (50000, 700, 160), (9000, 9000, 160), (400000, 400000, 2)])
@pytest.mark.parametrize("kind", ["rand", "ties", "equal"])
def test_eviction_by_the_tables_capacity(cap, lens, lanes, kind):
    # Keys that fit in shared memory and keys that do not, by one CTA for each of many heads and by clusters for a few.
    vx = _vx()
    page, D, keep, recent = 500, 64, lens // 3, lens // 50
    pages = cap // page
    c = vx.PagedCache(1, pages, page, lanes, D, 1, pages, weights=True)
    gen = torch.Generator(device="cuda").manual_seed(3)
    c.table.copy_(torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)[None])
    a = torch.rand(lanes, lens, generator=gen, device="cuda")
    if kind == "ties":
        a = torch.randint(0, 5, (lanes, lens), generator=gen, device="cuda").float()
    if kind == "equal":
        a.fill_(0.25)
    j = torch.arange(lens, device="cuda")
    pg, off = c.table[0].long()[j // page], j % page
    c.acc[0][pg, :, off] = a.T
    c.k[0][pg, :, off] = (j % 251).to(BF)[:, None, None].expand(lens, lanes, D)
    c.v[0][pg, :, off] = (j % 241).to(BF)[:, None, None].expand(lens, lanes, D)
    c.lens.fill_(lens)
    kept = torch.full((1, 1, lanes, keep), -1, dtype=torch.int32, device="cuda")
    vx.paged_evict(c, keep, recent, kept=kept)
    best = torch.sort(a[:, :lens - recent], dim=1, descending=True, stable=True).indices[:, :keep - recent].sort(1).values
    want = torch.cat([best, torch.arange(lens - recent, lens, device="cuda").expand(lanes, recent)], 1)
    assert torch.equal(kept[0, 0].long(), want)
    i = torch.arange(keep, device="cuda")
    pg, off = c.table[0].long()[i // page], i % page
    assert torch.equal(c.acc[0][pg, :, off].T, a.gather(1, want))
    assert torch.equal(c.k[0][pg, :, off][..., 5].T, (want % 251).to(BF))
    assert torch.equal(c.v[0][pg, :, off][..., 60].T, (want % 241).to(BF))
