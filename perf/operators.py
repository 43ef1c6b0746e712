"""The paged-cache operators as they are measured: rotary positions, the append
of new tokens to a paged K/V cache, attention of a chunk of new tokens over that
cache, and the eviction of cached tokens by accumulated attention weight.

``run`` computes each operator in its plain form (elementary torch operations
in fp32; float64 for rotary angles) or, with ``own`` set, calls the package.
``exact`` computes the same outputs in float64 from the definitions.

Definitions (one layer, one sequence; slots count the cached tokens):
  rope    y = R(pos) x on the first rot_dim dims, pairs (m, m + rot_dim/2) or
          (2m, 2m + 1), angle pos * f_m, f_m by the scaling rule, times mscale
  append  slot lens + t of the sequence's pages <- (R(pos + t) k_t, v_t)
  attn    query t sits at slot i = lens + t and sees slot j iff j < lens + n and
          (j < prefix or i - window < j <= i); s = q.k * scale, then
          cap * tanh(s / cap), then - slope_h * |i - j|; o = softmax(s) v,
          lse = log sum exp(s); acc_j = sum over queries and the group's heads
          of the softmax weights
  evict   the last `recent` slots and, of the others, the keep - recent with
          the largest acc (ties: the lowest slot) move, in slot order, to slots
          0 .. keep - 1 of the destination
"""
import math

import torch

own = False

_BF, _F32 = "bf16", "fp32"


def _dt(case):
    return torch.float32 if case["dtype"] == _F32 else torch.bfloat16


# ------------------------------------------------------------------- cases

def listed():
    return [
        # the encoder's streaming step: q and k of 64 streams x 4 new frames, 32 + 32 heads, a view of a fused qkv row
        dict(name="rope_step", op="rope", dtype=_BF, tokens=256, heads=64, pad_heads=32, dim=64, rot=64,
             inter=False, scaling="none", factor=1.0, theta=1e6, far=6000),
        # a decoder's prompt, 32 + 8 heads of 128, rotary on half of each head, stretched to 8 times its context
        dict(name="rope_prompt", op="rope", dtype=_BF, tokens=16384, heads=40, pad_heads=8, dim=128, rot=64,
             inter=True, scaling="yarn", factor=8.0, theta=1e6, far=60000),
        # the same step's 4 frames per stream rotated and written to their pages
        dict(name="append_step", op="append", dtype=_BF, seqs=64, new=4, ragged=False, kv=3000, hq=32, hkv=32, dim=64,
             page=16, inter=False, scaling="none", factor=1.0, theta=1e6),
        # prompts of several lengths at once, grouped heads
        dict(name="append_prompt", op="append", dtype=_BF, seqs=6, new=4001, ragged=True, kv=4100, hq=32, hkv=8,
             dim=128, page=64, inter=False, scaling="linear", factor=4.0, theta=1e6),
        # decoding: 64 sequences of very different lengths, one token each
        dict(name="attn_token", op="attn", dtype=_BF, seqs=64, new=1, ragged=False, kv=4096, hq=32, hkv=8, dim=128,
             page=64, window=0, prefix=0, cap=0.0, slopes=False, track=False),
        # decoding one long sequence, its weights accumulated for eviction
        dict(name="attn_long_token", op="attn", dtype=_BF, seqs=1, new=1, ragged=False, kv=40001, hq=32, hkv=8,
             dim=128, page=16, window=0, prefix=0, cap=0.0, slopes=False, track=True),
        # the encoder's streaming step over pages instead of a ring: window 750, 4 frames, 32 heads of 64
        dict(name="attn_step", op="attn", dtype=_BF, seqs=64, new=4, ragged=False, kv=3000, hq=32, hkv=32, dim=64,
             page=16, window=750, prefix=0, cap=0.0, slopes=False, track=False),
        # prompt chunks of up to 4096 tokens over caches that already hold as many
        dict(name="attn_prompt", op="attn", dtype=_BF, seqs=4, new=4096, ragged=True, kv=8192, hq=32, hkv=8, dim=128,
             page=64, window=0, prefix=0, cap=0.0, slopes=False, track=False),
        # capped scores with a distance bias over a shared prefix, three heads to a group, weights kept
        dict(name="attn_capped", op="attn", dtype=_BF, seqs=8, new=1501, ragged=True, kv=2003, hq=12, hkv=4, dim=64,
             page=48, window=0, prefix=100, cap=30.0, slopes=True, track=True),
        # the fp32 form, window with a visible prefix
        dict(name="attn_fp32", op="attn", dtype=_F32, seqs=3, new=67, ragged=True, kv=900, hq=8, hkv=2, dim=64,
             page=16, window=250, prefix=16, cap=0.0, slopes=False, track=False),
        # streams cut back to one window's worth of frames
        dict(name="evict_step", op="evict", dtype=_BF, seqs=64, kv=1000, hkv=32, dim=64, page=16, keep=750,
             recent=250),
        # long sequences cut to an eighth
        dict(name="evict_long", op="evict", dtype=_BF, seqs=4, kv=32768, hkv=8, dim=128, page=64, keep=4096,
             recent=512),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.5)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "attn", "attn", "attn", "attn", "evict"])
    dtype = _F32 if rng.random() < 0.2 else _BF
    dim = rng.choice([64, 128])
    page = rng.choice([8, 16, 24, 32, 48, 50, 64, 128])
    hkv = rng.choice([1, 2, 4, 8, 32 if dim == 64 else 8])
    group = rng.choice([1, 1, 2, 3, 4, 4, 5, 8])
    while hkv * group > 40:
        group = max(1, group // 2)
    rope = dict(inter=rng.random() < 0.5, scaling=rng.choice(["none", "linear", "ntk", "yarn"]),
                factor=rng.choice([2.0, 4.0, 8.0]), theta=rng.choice([1e4, 5e5, 1e6]))
    if op == "rope":
        heads = rng.randrange(1, 41)
        return dict(op=op, dtype=dtype, tokens=_log(rng, 1, 8192), heads=heads, pad_heads=rng.choice([0, 8]), dim=dim,
                    rot=rng.choice([dim, dim // 2, dim // 4]), far=_log(rng, 100, 1000000), **rope)
    if op == "append":
        seqs = _log(rng, 1, 64)
        new = _log(rng, 1, max(1, 16000 // seqs))
        return dict(op=op, dtype=dtype, seqs=seqs, new=new, ragged=rng.random() < 0.5, kv=new + _log(rng, 1, 2000),
                    hq=hkv * group, hkv=hkv, dim=dim, page=page, **rope)
    if op == "evict":
        seqs = _log(rng, 1, 64)
        kv = _log(rng, 16, min(32768, 1000000 // (seqs * hkv)))
        keep = rng.randrange(1, kv + 1)
        return dict(op=op, dtype=dtype, seqs=seqs, kv=kv, hkv=hkv, dim=dim, page=page, keep=keep,
                    recent=rng.randrange(0, keep + 1))
    seqs = _log(rng, 1, 64)
    small = rng.random() < 0.5
    budget = 1 << 27 if dtype == _F32 else 1 << 30          # rows x keys over all sequences and heads
    new = rng.randrange(1, 9) if small else _log(rng, 9, 4096)
    kv = new + _log(rng, 1, 40000 if small else 8192)
    while seqs * new * kv * hkv * group > budget and (seqs > 1 or kv > 2 * new):
        seqs, kv = (max(1, seqs // 2), kv) if seqs > 1 else (seqs, max(new, kv // 2))
    while new * kv * hkv * group > budget:
        new, kv = max(1, new // 2), max(1, kv // 2)
    seqs = max(1, min(seqs, 400000 // kv))
    return dict(op=op, dtype=dtype, seqs=seqs, new=new, ragged=rng.random() < 0.5, kv=kv, hq=hkv * group, hkv=hkv,
                dim=dim, page=page, window=rng.choice([0, 0, _log(rng, 1, 5000)]),
                prefix=rng.choice([0, 0, _log(rng, 1, 500)]), cap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                slopes=rng.random() < 0.25, track=rng.random() < 0.3)


# ----------------------------------------------------------------- lengths

def _new_lens(case):
    """New tokens of each sequence: all alike, or spread between an eighth and the whole of `new`."""
    S, n = case["seqs"], case["new"]
    if not case["ragged"]:
        return [n] * S
    return [max(1, n - (n * 7 * s) // (8 * S)) for s in range(S)]


def _old_lens(case, news):
    """Tokens each sequence holds already; with its new ones at most kv, the first sequence exactly kv."""
    S, kv = case["seqs"], case["kv"]
    room = kv - max(news)
    return [kv - news[0] if s == 0 else max(0, room - (room * ((5 * s) % S)) // S) for s in range(S)]


def _evict_lens(case):
    S, kv = case["seqs"], case["kv"]
    return [max(1, kv - (kv * ((5 * s) % S)) // (2 * S)) for s in range(S)]


# ----------------------------------------------------------------- prepare

def _randn(shape, gen, dtype):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).to(dtype)


def _pool(case, lens, seed, weights, n_extra=3):
    """k, v [1, pages, hkv, page, dim], acc, a table of shuffled pages and the pool's size."""
    page, hkv, D, dtype = case["page"], case["hkv"], case["dim"], _dt(case)
    need = [(n + page - 1) // page for n in lens]
    P = sum(need) + n_extra
    gen = torch.Generator(device="cuda").manual_seed(seed)
    order = torch.randperm(P, generator=gen, device="cuda").to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
    at = 0
    for s, m in enumerate(need):
        table[s, :m] = order[at:at + m]
        at += m
    k = torch.empty(1, P, hkv, page, D, dtype=dtype, device="cuda")
    v = torch.empty_like(k)
    for t in (k, v):
        for a in range(0, P, 4096):
            t[:, a:a + 4096] = _randn(t[:, a:a + 4096].shape, gen, dtype)
    acc = None
    if weights:   # what a softmax leaves: few large weights, many small ones
        acc = torch.rand(1, P, hkv, page, generator=gen, device="cuda").pow_(8)
    return k, v, acc, table, gen


def _own_cache(case, k, v, acc, table, lens, pos):
    import sliding_window_attention_tcgen05_b200 as vx
    cache = vx.PagedCache(1, k.shape[1], case["page"], case["hkv"], case["dim"], table.shape[0], table.shape[1],
                          dtype=k.dtype, weights=acc is not None)
    cache.k, cache.v = k, v
    if acc is not None:
        cache.acc = acc
    cache.table.copy_(table)
    cache.lens.copy_(lens)
    cache.pos.copy_(pos)
    return cache


def _own_rope(case):
    import sliding_window_attention_tcgen05_b200 as vx
    return vx.RopeCfg(theta=case["theta"], rot_dim=case.get("rot", case["dim"]), interleaved=case["inter"],
                      scaling=case["scaling"], factor=case["factor"], orig_len=8192)


def prepare(case, seed):
    dtype = _dt(case)
    st = dict(case=case)
    if case["op"] == "rope":
        gen = torch.Generator(device="cuda").manual_seed(seed)
        N, H, D = case["tokens"], case["heads"], case["dim"]
        row = _randn((N, H + case["pad_heads"], D), gen, dtype)
        st["x"] = row[:, :H]
        st["pos"] = torch.randint(0, case["far"], (N,), generator=gen, device="cuda", dtype=torch.int64)
        if own:
            st["rope"] = _own_rope(case)
        return st
    if case["op"] == "evict":
        lens = _evict_lens(case)
        k, v, acc, table, gen = _pool(case, lens, seed, True)
        keep = [min(n, case["keep"]) for n in lens]
        page = case["page"]
        need = [(n + page - 1) // page for n in keep]
        order = torch.randperm(sum(need), generator=gen, device="cuda").to(torch.int32)
        dst = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device="cuda")
        at = 0
        for s, m in enumerate(need):
            dst[s, :m] = order[at:at + m]
            at += m
        shape = (1, sum(need), case["hkv"], page, case["dim"])
        st.update(k=k, v=v, acc=acc, table=table, lens=torch.tensor(lens, dtype=torch.int64, device="cuda"),
                  host_lens=lens, dst_table=dst, dk=torch.zeros(shape, dtype=dtype, device="cuda"),
                  dv=torch.zeros(shape, dtype=dtype, device="cuda"), dacc=torch.zeros(shape[:-1], device="cuda"),
                  kept=torch.full((1, case["seqs"], case["hkv"], case["keep"]), -1, dtype=torch.int32, device="cuda"))
        if own:
            st["cache"] = _own_cache(case, k, v, acc, table, st["lens"], st["lens"])
            zero = torch.zeros_like(st["lens"])
            st["dst"] = _own_cache(case, st["dk"], st["dv"], st["dacc"], dst, zero, zero)
        return st
    news = _new_lens(case)
    olds = _old_lens(case, news)
    total = [a + b for a, b in zip(olds, news)]
    track = case["op"] == "attn" and case["track"]
    k, v, acc, table, gen = _pool(case, total, seed, track)
    N, D = sum(news), case["dim"]
    lens = torch.tensor(olds, dtype=torch.int64, device="cuda")
    starts = [0]
    for n in news:
        starts.append(starts[-1] + n)
    st.update(k=k, v=v, acc=acc, table=table, lens=lens, news=news, olds=olds, starts=starts,
              q_start=torch.tensor(starts, dtype=torch.int32, device="cuda"), max_q=max(news), max_kv=max(total))
    qkv = _randn((N, case["hq"] + 2 * case["hkv"], D), gen, dtype)
    st["q"] = qkv[:, :case["hq"]]
    if case["op"] == "append":
        st["kn"] = qkv[:, case["hq"]:case["hq"] + case["hkv"]]
        st["vn"] = qkv[:, case["hq"] + case["hkv"]:]
        if own:
            st["rope"] = _own_rope(case)
    else:
        st["q"] = st["q"].contiguous()
        S, H = case["seqs"], case["hq"]
        st["prefix"] = st["slopes"] = None
        if case["prefix"]:
            st["prefix"] = torch.tensor([(case["prefix"] * (s + 1)) // S for s in range(S)], dtype=torch.int32,
                                        device="cuda")
        if case["slopes"]:
            st["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)], device="cuda")
    if own:
        st["cache"] = _own_cache(case, k, v, acc, table, lens, lens)
    return st


# --------------------------------------------------------------- plain form

def _angles(case, rot):
    """f_m of the pairs and the factor on cosine and sine, in float64."""
    m = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    theta, s = case["theta"], case["factor"]
    if case["scaling"] == "ntk":
        theta = theta * s ** (rot / (rot - 2))
    f = theta ** (-2.0 * m / rot)
    scale = 1.0
    if case["scaling"] == "linear":
        f = f / s
    elif case["scaling"] == "yarn":
        g = ((8192 * f / (2 * math.pi) - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        f = (1 - g) * f / s + g * f
        scale = 0.1 * math.log(s) + 1.0
    return f, scale


def _rotate(x, pos, case, rot):
    f, scale = _angles(case, rot)
    ang = pos.double()[:, None, None] * f
    c, s = (ang.cos() * scale).float(), (ang.sin() * scale).float()
    xf = x.float()
    out = xf.clone()
    h = rot // 2
    if case["inter"]:
        a, b = xf[..., 0:rot:2], xf[..., 1:rot:2]
        out[..., 0:rot:2] = a * c - b * s
        out[..., 1:rot:2] = b * c + a * s
    else:
        a, b = xf[..., :h], xf[..., h:rot]
        out[..., :h] = a * c - b * s
        out[..., h:rot] = b * c + a * s
    return out.to(x.dtype)


def _slots(table_row, n, page):
    i = torch.arange(n, device="cuda")
    return table_row[i // page].long(), i % page


def _plain_append(st):
    case = st["case"]
    pos = torch.cat([a + torch.arange(n, device="cuda") for a, n in zip(st["olds"], st["news"])])
    q = _rotate(st["q"], pos, case, case["dim"])
    kr = _rotate(st["kn"], pos, case, case["dim"])
    for s, (old, n) in enumerate(zip(st["olds"], st["news"])):
        pg, off = _slots(st["table"][s], old + n, case["page"])
        pg, off = pg[old:], off[old:]
        rows = slice(st["starts"][s], st["starts"][s] + n)
        st["k"][0][pg, :, off] = kr[rows]
        st["v"][0][pg, :, off] = st["vn"][rows]
    return q, st["k"], st["v"]


def _plain_attn(st):
    case = st["case"]
    hq, hkv, D, page = case["hq"], case["hkv"], case["dim"], case["page"]
    G = hq // hkv
    out = torch.empty_like(st["q"])
    lse = torch.empty(st["q"].shape[0], hq, device="cuda")
    for s, (old, n) in enumerate(zip(st["olds"], st["news"])):
        L = old + n
        pg, off = _slots(st["table"][s], L, page)
        rows = slice(st["starts"][s], st["starts"][s] + n)
        i = old + torch.arange(n, device="cuda")[:, None]
        j = torch.arange(L, device="cuda")[None, :]
        seen = j <= i
        if case["window"]:
            seen &= j > i - case["window"]
        if st["prefix"] is not None:
            seen |= j < st["prefix"][s]
        dist = (i - j).abs().float() if case["slopes"] else None
        step = max(1, min(hkv, (1 << 28) // (G * n * L)))
        for h in range(0, hkv, step):
            hs = slice(h, min(hkv, h + step))
            k = st["k"][0][pg, hs, off].float().transpose(0, 1)            # [h, L, D]
            v = st["v"][0][pg, hs, off].float().transpose(0, 1)
            nh = k.shape[0]
            qs = st["q"][rows, h * G:(h + nh) * G].float().reshape(n, nh, G, D).permute(1, 2, 0, 3)
            x = torch.matmul(qs, k.transpose(1, 2)[:, None]) * D ** -0.5   # [h, G, n, L]
            if case["cap"]:
                x = case["cap"] * torch.tanh(x / case["cap"])
            if dist is not None:
                x = x - st["slopes"][h * G:(h + nh) * G].reshape(nh, G, 1, 1) * dist
            x = x.masked_fill(~seen, float("-inf"))
            top = x.amax(-1, keepdim=True)
            p = torch.exp(x - top)
            z = p.sum(-1, keepdim=True)
            p = p / z
            o = torch.matmul(p, v[:, None])
            out[rows, h * G:(h + nh) * G] = o.permute(2, 0, 1, 3).reshape(n, nh * G, D).to(out.dtype)
            lse[rows, h * G:(h + nh) * G] = (top + torch.log(z))[..., 0].permute(2, 0, 1).reshape(n, nh * G)
            if case["track"]:
                st["acc"][0][pg, hs, off] = p.sum((1, 2)).transpose(0, 1)
    return (out, lse, st["acc"]) if case["track"] else (out, lse)


def _plain_evict(st):
    case = st["case"]
    page, hkv, recent = case["page"], case["hkv"], case["recent"]
    new_lens = []
    for s, L in enumerate(st["host_lens"]):
        keep = min(L, case["keep"])
        r = min(recent, keep)
        pg, off = _slots(st["table"][s], L, page)
        a = st["acc"][0][pg, :, off].transpose(0, 1)                       # [hkv, L]
        best = torch.sort(a[:, :L - r], dim=1, descending=True, stable=True).indices[:, :keep - r]
        tail = torch.arange(L - r, L, device="cuda").expand(hkv, r)
        idx = torch.cat([best.sort(dim=1).values, tail], 1)                # [hkv, keep]
        dp, do = _slots(st["dst_table"][s], keep, page)
        heads = torch.arange(hkv, device="cuda")[:, None]
        sp, so = pg[idx], off[idx]
        for src, dst in ((st["k"], st["dk"]), (st["v"], st["dv"]), (st["acc"], st["dacc"])):
            dst[0][dp, :, do] = src[0][sp, heads, so].transpose(0, 1)
        st["kept"][0, s, :, :keep] = idx.to(torch.int32)
        new_lens.append(keep)
    return st["dk"], st["dv"], st["dacc"], torch.tensor(new_lens, device="cuda"), st["kept"]


# --------------------------------------------------------------------- run

def run(state):
    case = state["case"]
    op = case["op"]
    if not own:
        if op == "rope":
            return _rotate(state["x"], state["pos"], case, case["rot"])
        return {"append": _plain_append, "attn": _plain_attn, "evict": _plain_evict}[op](state)
    import sliding_window_attention_tcgen05_b200 as vx
    if op == "rope":
        return vx.rope_fwd(state["x"], state["pos"], state["rope"])
    if op == "append":
        q = vx.paged_append(state["cache"], 0, state["kn"], state["vn"], state["q_start"], state["max_q"],
                            rope=state["rope"], q=state["q"])
        return q, state["cache"].k, state["cache"].v
    if op == "attn":
        o, lse = vx.paged_attn_fwd(state["cache"], 0, state["q"], state["q_start"], state["max_q"],
                                   max_kv=state["max_kv"], window=case["window"], prefix=state["prefix"],
                                   cap=case["cap"], slopes=state["slopes"], track=0.0 if case["track"] else None,
                                   return_lse=True)
        return (o, lse, state["cache"].acc) if case["track"] else (o, lse)
    vx.paged_evict(state["cache"], case["keep"], case["recent"], dst=state["dst"], kept=state["kept"])
    dst = state["dst"]
    return dst.k, dst.v, dst.acc, dst.lens, state["kept"]


# -------------------------------------------------------------------- work

def _pairs(old, n, window, prefix):
    """Attended (query, key) pairs of one sequence, and the slots that some query sees."""
    t = torch.arange(n, dtype=torch.int64)
    i = old + t
    L = old + n
    lo = (i - window + 1).clamp(min=0) if window else torch.zeros_like(i)
    p = min(prefix, L)
    pairs = (i - lo + 1) + torch.minimum(lo, torch.tensor(p)) + (p - 1 - i).clamp(min=0)
    first = int(lo[0])
    seen = L - first + min(first, p)
    return int(pairs.sum()), seen


def work(case):
    es = 4 if case["dtype"] == _F32 else 2
    op, D = case["op"], case["dim"]
    if op == "rope":
        n = case["tokens"] * case["heads"]
        return {"bytes": 2 * n * D * es + 8 * case["tokens"], "flops": 3 * n * case["rot"]}
    if op == "append":
        N = sum(_new_lens(case))
        rows = N * (case["hq"] + 2 * case["hkv"])
        return {"bytes": 2 * rows * D * es, "flops": 3 * N * (case["hq"] + case["hkv"]) * D}
    if op == "evict":
        lens = _evict_lens(case)
        kept = sum(min(n, case["keep"]) for n in lens) * case["hkv"]
        return {"bytes": 4 * sum(lens) * case["hkv"] + kept * (4 * D * es + 4 + 4), "flops": sum(lens) * case["hkv"]}
    news = _new_lens(case)
    olds = _old_lens(case, news)
    pairs = keys = 0
    for s, (o, n) in enumerate(zip(olds, news)):
        a, b = _pairs(o, n, case["window"], (case["prefix"] * (s + 1)) // case["seqs"])
        pairs += a
        keys += b
    N = sum(news)
    total = sum(olds) + N
    by = 2 * keys * case["hkv"] * D * es + 2 * N * case["hq"] * D * es + 4 * N * case["hq"]
    if case["track"]:
        by += 4 * total * case["hkv"]
    return {"bytes": by, "flops": 4 * pairs * case["hq"] * D}


# ------------------------------------------------------------------- exact

def _exact_rope(x, pos, case, rot):
    """Each pair as a complex number times scale * exp(i * pos * f)."""
    half = rot // 2
    freqs, mag = [], 1.0
    for m in range(half):
        base = case["theta"]
        if case["scaling"] == "ntk":
            base *= case["factor"] ** (rot / (rot - 2))
        f = math.exp(-2.0 * m / rot * math.log(base))
        if case["scaling"] == "linear":
            f /= case["factor"]
        if case["scaling"] == "yarn":
            turns = 8192 * f / (2 * math.pi)
            share = min(1.0, max(0.0, (turns - 1.0) / 31.0))
            f = f * share + f / case["factor"] * (1.0 - share)
            mag = 1.0 + 0.1 * math.log(case["factor"])
        freqs.append(f)
    turn = torch.outer(pos.double(), torch.tensor(freqs, dtype=torch.float64, device="cuda"))
    w = torch.polar(torch.full_like(turn, mag), turn)[:, None]
    y = x.double().clone()
    part = y[..., :rot]
    if case["inter"]:
        z = torch.view_as_complex(part.reshape(*part.shape[:-1], half, 2).contiguous())
        y[..., :rot] = torch.view_as_real(z * w).flatten(-2)
    else:
        z = torch.complex(part[..., :half].contiguous(), part[..., half:].contiguous()) * w
        y[..., :rot] = torch.cat([z.real, z.imag], -1)
    return y


def exact(case, seed):
    global own
    was, own = own, False
    try:
        st = prepare(case, seed)
    finally:
        own = was
    op, page = case["op"], case["page"] if "page" in case else 0
    if op == "rope":
        return _exact_rope(st["x"], st["pos"], case, case["rot"])
    flat = {n: st[n][0].double() for n in ("k", "v", "acc") if st.get(n) is not None} if op != "attn" else {}

    def place(s, slot, name="table"):
        return int(st[name][s, slot // page]), slot % page

    if op == "append":
        pos = torch.tensor([o + t for o, n in zip(st["olds"], st["news"]) for t in range(n)], device="cuda")
        q = _exact_rope(st["q"], pos, case, case["dim"])
        kr = _exact_rope(st["kn"], pos, case, case["dim"])
        tab = st["table"].cpu()
        where = torch.tensor([[int(tab[s, (o + t) // page]), (o + t) % page]
                              for s, (o, n) in enumerate(zip(st["olds"], st["news"])) for t in range(n)],
                             device="cuda")
        flat["k"][where[:, 0], :, where[:, 1]] = kr
        flat["v"][where[:, 0], :, where[:, 1]] = st["vn"].double()
        return q, flat["k"][None], flat["v"][None]
    if op == "evict":
        dk, dv, da = (st[n][0].double() for n in ("dk", "dv", "dacc"))
        kept = st["kept"].clone()
        lens = []
        for s, L in enumerate(st["host_lens"]):
            K = min(L, case["keep"])
            R = min(case["recent"], K)
            slots = torch.arange(L, device="cuda")
            src = st["table"][s].long()[slots // page] * page + slots % page
            to = torch.arange(K, device="cuda")
            dst = st["dst_table"][s].long()[to // page] * page + to % page
            for h in range(case["hkv"]):
                a = flat["acc"][:, h].reshape(-1)[src]
                if K > R:   # the (K - R)-th largest of the old slots, then as many of its equals as still fit
                    old = a[:L - R]
                    bar = old.kthvalue(L - R - (K - R) + 1).values
                    more = old > bar
                    same = old == bar
                    more |= same & (same.cumsum(0) <= (K - R) - more.sum())
                    idx = torch.cat([more.nonzero()[:, 0], slots[L - R:]])
                else:
                    idx = slots[L - R:]
                kept[0, s, h, :K] = idx.to(torch.int32)
                for a_, b_ in ((flat["k"], dk), (flat["v"], dv)):
                    b_[dst // page, h, dst % page] = a_[src[idx] // page, h, src[idx] % page]
                da[dst // page, h, dst % page] = a[idx]
            lens.append(K)
        return dk[None], dv[None], da[None], torch.tensor(lens, device="cuda"), kept
    hq, hkv, D = case["hq"], case["hkv"], case["dim"]
    G = hq // hkv
    o = torch.zeros(st["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.zeros(st["q"].shape[:2], dtype=torch.float64, device="cuda")
    acc = st["acc"].double() if case["track"] else None
    for s, (old, n) in enumerate(zip(st["olds"], st["news"])):
        L = old + n
        slots = torch.arange(L, device="cuda")
        at = st["table"][s].long()[slots // page] * page + slots % page
        pre = 0 if st["prefix"] is None else int(st["prefix"][s])
        r0 = st["starts"][s]
        for h in range(hkv):
            k = st["k"][0][at // page, h, at % page].double()
            v = st["v"][0][at // page, h, at % page].double()
            total = torch.zeros(L, dtype=torch.float64, device="cuda")
            for g in range(h * G, (h + 1) * G):
                for a in range(0, n, 2048):
                    b = min(n, a + 2048)
                    back = (old + torch.arange(a, b, device="cuda"))[:, None] - slots    # i - j
                    x = st["q"][r0 + a:r0 + b, g].double() @ k.T / math.sqrt(D)
                    if case["cap"]:
                        x = torch.tanh(x / case["cap"]) * case["cap"]
                    if case["slopes"]:
                        x = x - float(st["slopes"][g]) * back.abs()
                    hidden = back < 0
                    if case["window"]:
                        hidden |= back >= case["window"]
                    hidden &= slots >= pre
                    x[hidden.expand_as(x)] = -math.inf
                    z = torch.logsumexp(x, 1)
                    p = torch.exp(x - z[:, None])
                    o[r0 + a:r0 + b, g] = p @ v
                    lse[r0 + a:r0 + b, g] = z
                    total += p.sum(0)
            if acc is not None:
                acc[0][at // page, h, at % page] = total
    return (o, lse, acc) if case["track"] else (o, lse)
