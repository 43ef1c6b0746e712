"""Pins of the oracle's paged-cache operators to facts outside them, and the
host-side refusals of their C entry points (both without a GPU)."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import oracle
import oracle.paged as paged


def _rand(shape, seed):
    return np.random.default_rng(seed).standard_normal(shape)


# ------------------------------------------------------------------- rotary

def test_plain_half_layout_is_the_encoders_rope():
    x = _rand((1, 9, 3, 64), 1)
    pos = np.arange(5, 14)
    np.testing.assert_allclose(paged.rope(x[0], pos), oracle.rope(x, pos, 1e6)[0], rtol=1e-12, atol=1e-13)


def test_interleaved_is_the_half_layout_of_permuted_elements():
    x = _rand((7, 2, 16), 2)
    pos = np.array([0, 1, -3, 1000, 7, 8, 123456])
    perm = np.concatenate([np.arange(0, 16, 2), np.arange(1, 16, 2)])
    y = paged.rope(x, pos, interleaved=True, theta=1e4)
    np.testing.assert_allclose(y[..., perm], paged.rope(x[..., perm], pos, theta=1e4), rtol=0, atol=1e-14)


def test_rotation_of_a_part_leaves_the_rest_and_the_norm():
    x = _rand((4, 2, 32), 3)
    y = paged.rope(x, np.array([3, 50, 7, 9]), rot=8, theta=1e4)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
    np.testing.assert_allclose(np.linalg.norm(y[..., :8], axis=-1), np.linalg.norm(x[..., :8], axis=-1), rtol=1e-13)


def test_scalings():
    plain, one = paged.rope_freqs(32, theta=1e4)
    lin, _ = paged.rope_freqs(32, theta=1e4, scaling="linear", factor=4.0)
    np.testing.assert_allclose(lin * 4, plain, rtol=1e-15)
    ntk, _ = paged.rope_freqs(32, theta=1e4, scaling="ntk", factor=4.0)
    assert ntk[0] == 1.0                                            # the fastest pair is unchanged,
    np.testing.assert_allclose(ntk[-1] * 4, plain[-1], rtol=1e-12)  # the slowest one is stretched by the factor
    yarn, ms = paged.rope_freqs(32, theta=1e4, scaling="yarn", factor=4.0, orig_len=4096)
    turns = 4096 * plain / (2 * math.pi)
    np.testing.assert_allclose(yarn[turns >= 32], plain[turns >= 32], rtol=1e-15)
    np.testing.assert_allclose(yarn[turns <= 1], plain[turns <= 1] / 4, rtol=1e-15)
    assert np.all((yarn <= plain) & (yarn >= plain / 4)) and ms == pytest.approx(0.1 * math.log(4) + 1) and one == 1.0


# ---------------------------------------------------------------- attention

@pytest.mark.parametrize("window", [1, 5, 40])
def test_chunk_over_a_cache_is_the_window_attention_of_the_whole(window):
    T, H, D, old = 33, 2, 8, 20
    q, k, v = (_rand((1, T, H, D), s) for s in (4, 5, 6))
    whole = oracle.swa_attention(q, k, v, window=window)[0]
    got = paged.attention(q[0, old:], k[0], v[0], old, window=window)
    np.testing.assert_allclose(got["o"], whole[old:], rtol=1e-12, atol=1e-13)


def test_grouped_heads_prefix_and_weights_against_torch():
    n, old, Hq, Hkv, D = 6, 7, 6, 2, 16
    q, k, v = _rand((n, Hq, D), 7), _rand((old + n, Hkv, D), 8), _rand((old + n, Hkv, D), 9)
    mask = torch.from_numpy(paged.seen(old, n, window=4, prefix=3))
    want = torch.nn.functional.scaled_dot_product_attention(
        torch.from_numpy(q).transpose(0, 1), torch.from_numpy(k).transpose(0, 1).repeat_interleave(3, 0),
        torch.from_numpy(v).transpose(0, 1).repeat_interleave(3, 0), attn_mask=mask).transpose(0, 1).numpy()
    got = paged.attention(q, k, v, old, window=4, prefix=3)
    np.testing.assert_allclose(got["o"], want, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(got["weights"].sum(1), n * 3, rtol=1e-12)   # every row's weights sum to one
    assert mask[0, :3].all() and not mask[0, 3] and mask[0, 4] and not mask[0, 8]


def test_cap_and_slopes_by_brute_force():
    n, old, H, D = 2, 3, 2, 4
    q, k, v = _rand((n, H, D), 10) * 3, _rand((old + n, H, D), 11), _rand((old + n, H, D), 12)
    slopes = np.array([0.5, 0.125])
    got = paged.attention(q, k, v, old, cap=2.0, slopes=slopes, scale=0.7)
    for t in range(n):
        for h in range(H):
            s = [2.0 * math.tanh(0.7 * float(q[t, h] @ k[j, h]) / 2.0) - slopes[h] * (old + t - j)
                 for j in range(old + t + 1)]
            e = [math.exp(x) for x in s]
            want = sum(a * v[j, h] for j, a in enumerate(e)) / sum(e)
            np.testing.assert_allclose(got["o"][t, h], want, rtol=1e-12)
            assert got["lse"][t, h] == pytest.approx(math.log(sum(e)), rel=1e-12)


# ----------------------------------------------------------------- eviction

def test_evict_order_ties_and_nan():
    nan = float("nan")
    assert list(paged.evict([1, 5, 5, 0, 5, 2, 9, 9], 4, 2)) == [1, 2, 6, 7]
    assert list(paged.evict([nan, 1.0, -np.inf, 2.0], 2, 0)) == [1, 3]
    assert list(paged.evict([nan, 1.0, -np.inf, 2.0], 3, 0)) == [1, 2, 3]
    assert list(paged.evict([3.0, 1.0, 2.0], 2, 5)) == [1, 2]
    assert list(paged.evict([3.0, 1.0], 5, 1)) == [0, 1]
    assert list(paged.evict([3.0, 1.0], 0, 1)) == []


# ------------------------------------------- host-side refusals (no GPU call)

def _lib():
    import sliding_window_attention_tcgen05_b200 as vx
    return vx, vx._lib


def _cache(L, **kw):
    # Pointers that are never followed: every call below is refused on the host.
    d = dict(k=4096, v=8192, acc=12288, table=16384, lens=20480, pos=24576, dt=1, n_layers=2, n_pages=8, page_size=16,
             n_kv_heads=2, head_dim=64, n_seqs=3, max_pages=4)
    d.update(kw)
    return L.VxPagedCache(*[d[n] for n, _ in L.VxPagedCache._fields_])


def _rope(L, **kw):
    d = dict(rot_dim=0, interleaved=0, scaling=0, orig_len=0, theta=1e4, factor=1.0, beta_fast=32.0, beta_slow=1.0,
             mscale=0.0)
    d.update(kw)
    return L.VxRopeCfg(*[d[n] for n, _ in L.VxRopeCfg._fields_])


def _attn(vx, L, cache, q=(1 << 20, 256, 64), o=(1 << 21, 256, 64), heads=4, layer=0, q_start=4096, n=5, mq=5,
          opts=None, track=0, decay=0.0, ws=1 << 22, nws=1 << 20):
    return vx.lib.vx_paged_attn_fwd(C.byref(cache), layer, C.byref(L.VxRows(*q)) if q else None,
                                    C.byref(L.VxRows(*o)) if o else None, None, heads, q_start, n, mq, 0,
                                    C.byref(L.VxAttnOpts(*opts)) if opts else None, track, decay, ws, nws, None)


@pytest.mark.parametrize("change,status,word", [
    (dict(k=None), 1, "null"), (dict(table=None), 1, "null"), (dict(lens=None), 1, "null"),
    (dict(k=4104), 1, "16-byte"), (dict(dt=7), 1, "dtype"), (dict(head_dim=96), 2, "head_dim"),
    (dict(n_layers=0), 1, "n_layers"), (dict(n_seqs=0), 1, "n_seqs"), (dict(n_seqs=70000), 1, "n_seqs"),
    (dict(page_size=0), 1, "page_size"), (dict(page_size=70000), 1, "page_size"),
    (dict(page_size=65536, max_pages=16384), 1, "2^30"), (dict(n_kv_heads=0), 1, "n_kv_heads"),
    (dict(lens=20484), 1, "aligned"), (dict(acc=12289), 1, "aligned")])
def test_bad_caches_are_refused(change, status, word):
    vx, L = _lib()
    assert _attn(vx, L, _cache(L, **change)) == status
    assert word in vx.lib.vx_last_error().decode()
    assert vx.lib.vx_paged_advance(C.byref(_cache(L, **change)), 4096, 5, 5, 1 << 22, 1 << 20, None) == status
    assert vx.lib.vx_paged_evict(C.byref(_cache(L, **change)), None, 4, 2, None, 1 << 22, 1 << 20, None) == status
    assert vx.lib.vx_paged_attn_workspace(C.byref(_cache(L, **change)), 4, 5, 5, 0, 0, 0) == 0


@pytest.mark.parametrize("kw,word", [
    (dict(layer=2), "layer"), (dict(layer=-1), "layer"), (dict(q_start=None), "q_start"),
    (dict(q_start=4098), "q_start"), (dict(n=-1), "n_tokens"), (dict(mq=-1), "max_q"), (dict(heads=3), "multiple"),
    (dict(heads=0), "multiple"), (dict(opts=(0.0, -1.0, 0, None, None)), "cap"),
    (dict(opts=(float("nan"), 0.0, 0, None, None)), "scale"), (dict(opts=(0.0, 0.0, -1, None, None)), "window"),
    (dict(opts=(0.0, 0.0, 0, 4097, None)), "misaligned"), (dict(track=1, decay=-0.5), "track_decay"),
    (dict(track=1, decay=float("inf")), "track_decay"), (dict(ws=None), "workspace"), (dict(ws=(1 << 22) + 8), "256"),
    (dict(nws=16), "too small")])
def test_bad_attention_calls_are_refused(kw, word):
    vx, L = _lib()
    assert _attn(vx, L, _cache(L), **kw) == 1
    assert word in vx.lib.vx_last_error().decode()


def test_track_needs_acc():
    vx, L = _lib()
    assert _attn(vx, L, _cache(L, acc=None), track=1) == 1
    assert "acc" in vx.lib.vx_last_error().decode()


@pytest.mark.parametrize("cfg,word", [
    (dict(rot_dim=3), "rot_dim"), (dict(rot_dim=66), "rot_dim"), (dict(rot_dim=-2), "rot_dim"),
    (dict(theta=0.5), "theta"), (dict(theta=float("nan")), "theta"), (dict(scaling=4), "scaling"),
    (dict(scaling=1, factor=0.5), "factor"), (dict(scaling=2, factor=2.0, rot_dim=2), "ntk"),
    (dict(scaling=3, factor=2.0), "yarn"), (dict(scaling=3, factor=2.0, orig_len=8, beta_fast=1.0), "yarn"),
    (dict(scaling=3, factor=2.0, orig_len=8, mscale=-1.0), "yarn")])
def test_bad_rope_configurations_are_refused(cfg, word):
    vx, L = _lib()
    r = L.VxRows(1 << 20, 256, 64)
    assert vx.lib.vx_rope_fwd(C.byref(r), C.byref(r), 1, 4, 2, 64, 4096, C.byref(_rope(L, **cfg)), None) == 1
    assert word in vx.lib.vx_last_error().decode()


def test_bad_rope_calls_are_refused():
    vx, L = _lib()
    r, rope = L.VxRows(1 << 20, 256, 64), _rope(L)

    def call(x=r, y=r, dt=1, n=4, heads=2, dim=64, pos=4096, cfg=rope):
        return vx.lib.vx_rope_fwd(C.byref(x) if x else None, C.byref(y) if y else None, dt, n, heads, dim, pos,
                                  C.byref(cfg) if cfg else None, None)
    for kw in (dict(x=None), dict(y=None), dict(dt=3), dict(n=-1), dict(heads=0), dict(dim=63), dict(dim=258),
               dict(pos=None), dict(pos=4100), dict(cfg=None), dict(x=L.VxRows((1 << 20) + 1, 256, 64)),
               dict(y=L.VxRows(1 << 20, 128, 64))):
        assert call(**kw) == 1, kw
    assert call(x=None, y=None, n=0, pos=None) == 0     # nothing to do


def test_append_and_evict_refusals():
    vx, L = _lib()
    rows = lambda p, row=128, head=64: C.byref(L.VxRows(p, row, head))
    k, v, q = 1 << 20, 1 << 21, 1 << 23

    def append(cache=_cache(L), rope=None, q_=None, qo=None, k_=rows(k), v_=rows(v), ws=1 << 22, nws=256):
        return vx.lib.vx_paged_append(C.byref(cache), 0, rope, q_, qo, 4, k_, v_, 4096, 5, 5, ws, nws, None)
    rope = C.byref(_rope(L))
    assert append(q_=rows(q, 256)) == 1 and "rope" in vx.lib.vx_last_error().decode()
    assert append(rope=C.byref(_rope(L, rot_dim=12))) == 2          # a pair's vector would be cut
    assert append(ws=None) == 1 and append(nws=128) == 1
    dst = _cache(L, k=1 << 24)
    assert vx.lib.vx_paged_evict(C.byref(_cache(L)), C.byref(dst), 4, 2, None, 1 << 22, 1 << 20, None) == 1
    for kw in (dict(head_dim=128), dict(n_seqs=2), dict(page_size=8), dict(dt=0), dict(acc=None), dict(n_layers=1)):
        d = _cache(L, **{**dict(k=1 << 24, v=1 << 25, acc=1 << 26, lens=1 << 27), **kw})
        assert vx.lib.vx_paged_evict(C.byref(_cache(L)), C.byref(d), 4, 2, None, 1 << 22, 1 << 20, None) == 1, kw
    c = C.byref(_cache(L))
    assert vx.lib.vx_paged_evict(c, None, -1, 0, None, 1 << 22, 1 << 20, None) == 1
    assert vx.lib.vx_paged_evict(c, None, 4, -1, None, 1 << 22, 1 << 20, None) == 1
    assert vx.lib.vx_paged_evict(c, None, 4, 2, None, 1 << 22, 16, None) == 1
    assert vx.lib.vx_paged_evict(C.byref(_cache(L, acc=None)), None, 4, 2, None, 1 << 22, 1 << 20, None) == 1
