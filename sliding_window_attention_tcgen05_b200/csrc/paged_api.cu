// paged_api.cu -- the C entry points of the paged-cache operators
// (include/vx.h): argument checks, rotary tables, the choice of kernel and of
// the key split, workspace carving.
#include <cmath>
#include <climits>
#include <cstring>

#include "vx_api.h"
#include "paged_attn.cuh"

using namespace vx;

namespace vx {

// SMs the splits are sized for.
constexpr int64_t kPlanSms = 148;

PagedAttnPlan plan_paged_attn(bool bf16, int head_dim, int n_seqs, int n_kv_heads, int group, int max_q,
                              int64_t max_kv) {
  PagedAttnPlan p;
  const int64_t rows = static_cast<int64_t>(max_q) * group;
  const int64_t lanes = static_cast<int64_t>(n_seqs) * n_kv_heads;
  (void)head_dim;
  int64_t want, min_keys, ctas;
  if (!bf16) {
    p.kernel = 2;
    const int block = f32_block_rows(rows);
    ctas = lanes * ((rows + block - 1) / block);
    want = block == 64 ? 2 * kPlanSms : 6 * kPlanSms;
    min_keys = block == 8 ? 64 : 128;
  } else if (rows <= 32) {
    // A row block of the tcgen05 kernel would be at least three quarters padding.
    p.kernel = 0;
    ctas = lanes;
    want = 12 * kPlanSms;
    min_keys = 256;
  } else {
    p.kernel = 1;
    ctas = lanes * ((rows + 255) / 256);
    want = 1;
    min_keys = 128;
  }
  int64_t sp = (want + ctas - 1) / ctas;
  const int64_t most = max_kv / min_keys;
  if (sp > most) sp = most;
  if (sp > kMaxSplits) sp = kMaxSplits;
  if (p.kernel == 1) {
    // One CTA an SM: the split whose waves take least, in units of a tile of 128 keys (2 us), of which a CTA's start and
    // end cost about 4 and the joining of parts 3 (4 chunks of 100 tokens over 3000, 8 heads: 33 us in 128 CTAs, 36 us
    // in 160, which do not run at once).
    const int64_t tiles = (max_kv + 127) / 128;
    int64_t best = 0;
    for (int64_t c = 1; c <= kMaxSplits && c <= (most > 1 ? most : 1); ++c) {
      const int64_t cost = (ctas * c + kPlanSms - 1) / kPlanSms * ((tiles + c - 1) / c + 4) + (c > 1 ? 3 : 0);
      if (best == 0 || cost < best) {
        best = cost;
        sp = c;
      }
    }
  }
  // Where the rows kernel's CTAs can all run at once (three an SM) with few enough keys each, clusters of up to 8 join
  // their results themselves, which saves the combining launch; with more CTAs than that a cluster holds its places on
  // the SMs until its slowest CTA is done (64 sequences of up to 4096 tokens, 8 K/V heads: 96 us in clusters of 4, 92 us
  // without).
  p.cluster = 1;
  if (p.kernel == 0) {
    int c = 8;
    while (c > 1 && (ctas * c > 3 * kPlanSms || max_kv < c * 64)) c /= 2;
    if (max_kv <= c * 512 || sp <= c) {
      p.cluster = c;
      sp = c;
    }
  }
  p.splits = static_cast<int>(sp < 1 ? 1 : sp);
  // Sum of the weights: segments until there are about six CTAs for each place on the SMs (4 of 128 threads each), none
  // below four blocks of 64 rows.
  const int64_t w_ctas = lanes * ((max_kv + 127) / 128), most_segs = rows / 256;
  int64_t segs = (24 * kPlanSms + w_ctas - 1) / w_ctas;
  if (segs > most_segs) segs = most_segs;
  if (segs > 32) segs = 32;
  p.w_segs = static_cast<int>(segs < 1 ? 1 : segs);
  // Up to 8 rows: their scores, 4 bytes a key each, against another read of K (2 * head_dim bytes a key); not where
  // the tables' length would ask for a workspace of hundreds of megabytes.
  p.keep_scores = (p.kernel == 0 || p.kernel == 2) && rows <= 8 && lanes * rows * max_kv * 4 <= (256ll << 20);
  return p;
}

}  // namespace vx

namespace {

constexpr int64_t kMaxSlots = 1ll << 30;

vx_status check_cache(const vx_paged_cache* c, const char* what) {
  VX_CHECK_ARG(c != nullptr, "%s: the cache is null", what);
  VX_CHECK_ARG(c->k && c->v && c->table && c->lens && c->pos, "%s: a pointer of the cache is null", what);
  VX_CHECK_ARG(c->dt == VX_F32 || c->dt == VX_BF16, "%s: bad cache dtype %d", what, static_cast<int>(c->dt));
  VX_CHECK_ARG(aligned16(c->k) && aligned16(c->v), "%s: cache k/v must be 16-byte aligned", what);
  VX_CHECK_ARG((reinterpret_cast<uintptr_t>(c->table) & 3) == 0 && (reinterpret_cast<uintptr_t>(c->acc) & 3) == 0 &&
                   (reinterpret_cast<uintptr_t>(c->lens) & 7) == 0 && (reinterpret_cast<uintptr_t>(c->pos) & 7) == 0,
               "%s: table and acc must be 4-byte, lens and pos 8-byte aligned", what);
  if (c->head_dim != 64 && c->head_dim != 128) {
    set_error("%s: head_dim %d is not built (64 and 128 are)", what, c->head_dim);
    return VX_ERR_UNSUPPORTED;
  }
  VX_CHECK_ARG(c->n_layers >= 1 && c->n_layers <= 65535 && c->n_pages >= 1, "%s: bad n_layers or n_pages", what);
  VX_CHECK_ARG(c->n_kv_heads >= 1 && c->n_kv_heads <= 1024, "%s: n_kv_heads must be 1 .. 1024", what);
  VX_CHECK_ARG(c->n_seqs >= 1 && c->n_seqs <= 65535, "%s: n_seqs must be 1 .. 65535", what);
  VX_CHECK_ARG(c->page_size >= 1 && c->page_size <= 65536, "%s: page_size must be 1 .. 65536", what);
  VX_CHECK_ARG(static_cast<int64_t>(c->n_pages) * c->n_kv_heads * c->page_size < (1ll << 31),
               "%s: n_pages * n_kv_heads * page_size must be below 2^31", what);
  VX_CHECK_ARG(c->max_pages >= 1 && static_cast<int64_t>(c->max_pages) * c->page_size < kMaxSlots,
               "%s: max_pages * page_size must be 1 .. 2^30 - 1", what);
  return VX_OK;
}

vx_status check_chunk(const vx_paged_cache* c, int layer, const int32_t* q_start, int64_t n_tokens, int max_q,
                      const char* what) {
  VX_CHECK_ARG(layer >= 0 && layer < c->n_layers, "%s: layer %d of %d", what, layer, c->n_layers);
  VX_CHECK_ARG(q_start != nullptr && (reinterpret_cast<uintptr_t>(q_start) & 3) == 0,
               "%s: q_start is null or misaligned", what);
  VX_CHECK_ARG(n_tokens >= 0 && n_tokens < (1ll << 30), "%s: n_tokens must be 0 .. 2^30 - 1", what);
  VX_CHECK_ARG(max_q >= 0 && max_q < (1 << 30), "%s: max_q must be 0 .. 2^30 - 1", what);
  return VX_OK;
}

// Rows of heads read and written in 16-byte accesses.
vx_status check_rows(const vx_rows* r, int es, int n_heads, int64_t n_tokens, const char* what, const char* name) {
  VX_CHECK_ARG(r != nullptr && r->p != nullptr, "%s: %s is null", what, name);
  const int v = 16 / es;
  VX_CHECK_ARG(aligned16(r->p) && (r->row % v == 0 || n_tokens <= 1) && (r->head % v == 0 || n_heads <= 1),
               "%s: the rows of %s must start on 16-byte boundaries (strides %lld, %lld elements)", what, name,
               static_cast<long long>(r->row), static_cast<long long>(r->head));
  return VX_OK;
}

PagedView view_of(const vx_paged_cache* c) {
  PagedView v;
  v.table = c->table;
  v.lens = c->lens;
  v.page = FastDiv::make(static_cast<uint32_t>(c->page_size));
  v.n_pages = c->n_pages;
  v.n_heads = c->n_kv_heads;
  v.max_pages = c->max_pages;
  v.n_seqs = c->n_seqs;
  return v;
}

int64_t layer_rows(const vx_paged_cache* c) {
  return static_cast<int64_t>(c->n_pages) * c->n_kv_heads * c->page_size;
}
int elem_size(vx_dtype dt) { return dt == VX_BF16 ? 2 : 4; }

// f_m and mscale of the rotary positions, as fractions of a turn.
vx_status rope_table(const vx_rope_cfg* r, int head_dim, RopeTable* t, const char* what) {
  VX_CHECK_ARG(r != nullptr, "%s: rope is null", what);
  const int rot = r->rot_dim == 0 ? head_dim : r->rot_dim;
  VX_CHECK_ARG(rot >= 2 && rot % 2 == 0 && rot <= head_dim, "%s: rot_dim %d must be even and 2 .. head_dim (%d)", what,
               rot, head_dim);
  VX_CHECK_ARG(std::isfinite(r->theta) && r->theta >= 1.0, "%s: theta must be at least 1", what);
  VX_CHECK_ARG(r->scaling >= VX_ROPE_NONE && r->scaling <= VX_ROPE_YARN, "%s: unknown scaling %d", what, r->scaling);
  const bool scaled = r->scaling != VX_ROPE_NONE;
  VX_CHECK_ARG(!scaled || (std::isfinite(r->factor) && r->factor >= 1.0), "%s: factor must be at least 1", what);
  VX_CHECK_ARG(r->scaling != VX_ROPE_NTK || rot > 2, "%s: ntk scaling needs rot_dim above 2", what);
  const bool yarn = r->scaling == VX_ROPE_YARN;
  VX_CHECK_ARG(!yarn || (r->orig_len >= 1 && std::isfinite(r->beta_fast) && std::isfinite(r->beta_slow) &&
                         r->beta_fast > r->beta_slow && std::isfinite(r->mscale) && r->mscale >= 0.0),
               "%s: yarn needs orig_len >= 1, beta_fast > beta_slow and mscale >= 0", what);
  // The thread's last table: a model's calls all ask for the same one.
  struct Last {
    vx_rope_cfg cfg;   // no padding: compared as bytes
    int head_dim;
    RopeTable t;
  };
  static_assert(sizeof(vx_rope_cfg) == 4 * sizeof(int) + 5 * sizeof(double), "vx_rope_cfg has padding");
  static thread_local Last last = {};   // head_dim 0: none yet
  if (last.head_dim == head_dim && std::memcmp(&last.cfg, r, sizeof(*r)) == 0) {
    *t = last.t;
    return VX_OK;
  }
  long double theta = r->theta;
  if (r->scaling == VX_ROPE_NTK) theta *= powl(r->factor, static_cast<long double>(rot) / (rot - 2));
  const long double two_pi = 6.283185307179586476925286766559L;
  for (int m = 0; m < kMaxRotPairs; ++m) t->turns[m] = 0;
  // theta^(-2m / rot) as the product over m's bits: a power for each bit, one
  // multiplication for each m (64 powl calls take longer than the launch).
  long double bit[7], pw[kMaxRotPairs];
  for (int b = 0; b < 7; ++b) bit[b] = powl(theta, -2.0L * (1 << b) / rot);
  pw[0] = 1.0L;
  for (int m = 0; m < rot / 2; ++m) {
    if (m > 0) pw[m] = pw[m & (m - 1)] * bit[__builtin_ctz(m)];
    long double f = pw[m];
    if (r->scaling == VX_ROPE_LINEAR) f /= r->factor;
    if (yarn) {
      long double g = (r->orig_len * f / two_pi - r->beta_slow) /
                      (static_cast<long double>(r->beta_fast) - r->beta_slow);
      g = g < 0 ? 0 : g > 1 ? 1 : g;
      f = g * f + (1 - g) * f / r->factor;
    }
    t->turns[m] = static_cast<uint64_t>(f / two_pi * 18446744073709551616.0L + 0.5L);   // f <= 1: below 2^62
  }
  t->mscale = yarn ? static_cast<float>(r->mscale > 0.0 ? r->mscale : 0.1 * std::log(r->factor) + 1.0) : 1.f;
  t->pairs = rot / 2;
  t->interleaved = r->interleaved != 0;
  last.cfg = *r;
  last.head_dim = head_dim;
  last.t = *t;
  return VX_OK;
}

// Both layouts can be read in whole 16-byte vectors.
bool rope_vectors(const RopeTable& t, int head_dim, int es) {
  const int v = 16 / es;
  return head_dim % v == 0 && (t.interleaved ? (2 * t.pairs) % v == 0 : t.pairs % v == 0);
}

struct AttnCarve {
  float* lse;
  float* part_o;
  float2* part_ml;
  float* part_w;
  float* scores;
};
int64_t score_stride(int64_t max_kv) { return (max_kv + 3) / 4 * 4; }
AttnCarve carve_attn(Carve& cv, const vx_paged_cache* c, int64_t n_tokens, int n_q_heads, int max_q,
                     const PagedAttnPlan& p, int64_t max_kv, bool lse, bool track) {
  AttnCarve r = {};
  const int64_t rows_of_seq = static_cast<int64_t>(max_q) * (n_q_heads / c->n_kv_heads);
  const int64_t rows = n_tokens * n_q_heads;
  cv.take(kStatusBytes);
  if (track && !lse) r.lse = static_cast<float*>(cv.take(rows * 4));
  if (const int64_t parts = p.splits / p.cluster; parts > 1) {
    r.part_o = static_cast<float*>(cv.take(rows * parts * c->head_dim * 4));
    r.part_ml = static_cast<float2*>(cv.take(rows * parts * 8));
  }
  if (track && p.keep_scores)
    r.scores = static_cast<float*>(cv.take(c->n_seqs * c->n_kv_heads * rows_of_seq * score_stride(max_kv) * 4));
  else if (track && p.w_segs > 1)
    r.part_w = static_cast<float*>(cv.take(max_kv * p.w_segs * c->n_seqs * c->n_kv_heads * 4));
  return r;
}

int64_t bound_kv(const vx_paged_cache* c, int64_t max_kv) {
  const int64_t cap = static_cast<int64_t>(c->max_pages) * c->page_size;
  return max_kv <= 0 || max_kv > cap ? cap : max_kv;
}

}  // namespace

extern "C" {

vx_status vx_rope_fwd(const vx_rows* x, const vx_rows* y, vx_dtype dt, int64_t n_tokens, int n_heads, int head_dim,
                      const int64_t* pos, const vx_rope_cfg* rope, cudaStream_t stream) {
  const char* what = "vx_rope_fwd";
  VX_CHECK_ARG(dt == VX_F32 || dt == VX_BF16, "%s: bad dtype %d", what, static_cast<int>(dt));
  VX_CHECK_ARG(n_tokens >= 0 && n_tokens < (1ll << 30) && n_heads >= 1 && n_heads <= 65536,
               "%s: n_tokens must be 0 .. 2^30 - 1 and n_heads 1 .. 65536", what);
  VX_CHECK_ARG(head_dim >= 2 && head_dim <= 256 && head_dim % 2 == 0, "%s: head_dim must be even and 2 .. 256", what);
  RopeTable t;
  if (vx_status st = rope_table(rope, head_dim, &t, what)) return st;
  if (n_tokens == 0) return VX_OK;
  VX_CHECK_ARG(x && x->p && y && y->p && pos, "%s: x, y or pos is null", what);
  const int es = elem_size(dt);
  VX_CHECK_ARG(reinterpret_cast<uintptr_t>(x->p) % es == 0 && reinterpret_cast<uintptr_t>(y->p) % es == 0 &&
                   (reinterpret_cast<uintptr_t>(pos) & 7) == 0,
               "%s: x, y or pos is misaligned", what);
  RopeArgs2 a;
  a.x = {x->p, x->row, x->head};
  a.y = y->p;
  a.y_row = y->row;
  a.y_head = y->head;
  a.pos = pos;
  a.n_tokens = n_tokens;
  a.n_heads = n_heads;
  a.head_dim = head_dim;
  a.bf16 = dt == VX_BF16;
  const int v = 16 / es;
  auto whole = [&](const vx_rows* r) {
    return aligned16(r->p) && (r->row % v == 0 || n_tokens == 1) && (r->head % v == 0 || n_heads == 1);
  };
  a.vec = rope_vectors(t, head_dim, es) && whole(x) && whole(y);
  a.in_place = x->p == y->p;
  VX_CHECK_ARG(!a.in_place || ((x->row == y->row || n_tokens == 1) && (x->head == y->head || n_heads == 1)),
               "%s: y is x with other strides", what);
  Launch L{stream, nullptr, 0, 0};
  VX_CUDA(traced(L, "rope_fwd", 1, [&] { return launch_rope_rows(stream, a, t); }));
  return VX_OK;
}

vx_status vx_paged_append(const vx_paged_cache* cache, int layer, const vx_rope_cfg* rope, const vx_rows* q,
                          const vx_rows* q_out, int n_q_heads, const vx_rows* k, const vx_rows* v,
                          const int32_t* q_start, int64_t n_tokens, int max_q, void* ws, size_t ws_bytes,
                          cudaStream_t stream) {
  const char* what = "vx_paged_append";
  vx_status st;
  if ((st = check_cache(cache, what)) != VX_OK) return st;
  if ((st = check_chunk(cache, layer, q_start, n_tokens, max_q, what)) != VX_OK) return st;
  VX_CHECK_ARG(rope != nullptr || q == nullptr, "%s: q is only rotated, so it needs rope", what);
  VX_CHECK_ARG(q == nullptr || (n_q_heads >= 1 && n_q_heads <= 65536), "%s: bad n_q_heads %d", what, n_q_heads);
  const int es = elem_size(cache->dt);
  AppendArgs a = {};
  RopeTable t = {};
  if (rope) {
    if ((st = rope_table(rope, cache->head_dim, &t, what)) != VX_OK) return st;
    if (!rope_vectors(t, cache->head_dim, es)) {
      set_error("%s: rot_dim %d does not fill 16-byte vectors of this layout", what, 2 * t.pairs);
      return VX_ERR_UNSUPPORTED;
    }
  }
  Launch L;
  if ((st = make_launch(&L, ws, ws_bytes, kStatusBytes, stream)) != VX_OK) return st;
  if (n_tokens == 0 || max_q == 0) return VX_OK;
  if ((st = check_rows(k, es, cache->n_kv_heads, n_tokens, what, "k")) != VX_OK) return st;
  if ((st = check_rows(v, es, cache->n_kv_heads, n_tokens, what, "v")) != VX_OK) return st;
  if (q) {
    if ((st = check_rows(q, es, n_q_heads, n_tokens, what, "q")) != VX_OK) return st;
    if ((st = check_rows(q_out, es, n_q_heads, n_tokens, what, "q_out")) != VX_OK) return st;
    VX_CHECK_ARG(q->p != q_out->p || ((q->row == q_out->row || n_tokens == 1) &&
                                      (q->head == q_out->head || n_q_heads == 1)),
                 "%s: q_out is q with other strides", what);
    a.q = {q->p, q->row, q->head};
    a.q_out = q_out->p;
    a.qo_row = q_out->row;
    a.qo_head = q_out->head;
    a.n_q_heads = n_q_heads;
  }
  const int64_t base = layer * layer_rows(cache);
  a.c = view_of(cache);
  a.ch = {q_start, static_cast<int>(n_tokens), static_cast<int>(max_q < n_tokens ? max_q : n_tokens)};
  a.pos = cache->pos;
  a.k_pool = static_cast<uint8_t*>(cache->k) + base * cache->head_dim * es;
  a.v_pool = static_cast<uint8_t*>(cache->v) + base * cache->head_dim * es;
  a.acc = cache->acc ? cache->acc + base : nullptr;
  a.k = {k->p, k->row, k->head};
  a.v = {v->p, v->row, v->head};
  a.head_dim = cache->head_dim;
  a.bf16 = cache->dt == VX_BF16;
  a.status = L.status;
  VX_CUDA(traced(L, "paged_append", 1, [&] { return launch_paged_append(stream, a, t); }));
  return VX_OK;
}

vx_status vx_paged_advance(const vx_paged_cache* cache, const int32_t* q_start, int64_t n_tokens, int max_q, void* ws,
                           size_t ws_bytes, cudaStream_t stream) {
  const char* what = "vx_paged_advance";
  vx_status st;
  if ((st = check_cache(cache, what)) != VX_OK) return st;
  if ((st = check_chunk(cache, 0, q_start, n_tokens, max_q, what)) != VX_OK) return st;
  Launch L;
  if ((st = make_launch(&L, ws, ws_bytes, kStatusBytes, stream)) != VX_OK) return st;
  if (n_tokens == 0 || max_q == 0) return VX_OK;
  const ChunkArgs ch{q_start, static_cast<int>(n_tokens), static_cast<int>(max_q < n_tokens ? max_q : n_tokens)};
  VX_CUDA(traced(L, "paged_advance", 1, [&] {
    return launch_paged_advance(stream, view_of(cache), ch, cache->lens, cache->pos, L.status);
  }));
  return VX_OK;
}

size_t vx_paged_attn_workspace(const vx_paged_cache* cache, int n_q_heads, int64_t n_tokens, int max_q, int64_t max_kv,
                               int want_lse, int track) {
  if (check_cache(cache, "vx_paged_attn_workspace") != VX_OK || n_q_heads < 1 || n_tokens < 0 || max_q < 0) return 0;
  const int mq = static_cast<int>(max_q < n_tokens ? max_q : n_tokens);
  const int group = n_q_heads / cache->n_kv_heads;
  if (mq == 0 || group < 1) return kAlign;
  const int64_t kv = bound_kv(cache, max_kv);
  const PagedAttnPlan p = plan_paged_attn(cache->dt == VX_BF16, cache->head_dim, cache->n_seqs, cache->n_kv_heads,
                                          group, mq, kv);
  Carve cv{nullptr, 0};
  carve_attn(cv, cache, n_tokens, n_q_heads, mq, p, kv, want_lse, track);
  return align_up(cv.off, kAlign);
}

vx_status vx_paged_attn_fwd(const vx_paged_cache* cache, int layer, const vx_rows* q, const vx_rows* o, float* lse,
                            int n_q_heads, const int32_t* q_start, int64_t n_tokens, int max_q, int64_t max_kv,
                            const vx_attn_opts* opts, int track, float track_decay, void* ws, size_t ws_bytes,
                            cudaStream_t stream) {
  const char* what = "vx_paged_attn_fwd";
  vx_status st;
  if ((st = check_cache(cache, what)) != VX_OK) return st;
  if ((st = check_chunk(cache, layer, q_start, n_tokens, max_q, what)) != VX_OK) return st;
  VX_CHECK_ARG(n_q_heads >= 1 && n_q_heads % cache->n_kv_heads == 0,
               "%s: n_q_heads (%d) must be a multiple of n_kv_heads (%d)", what, n_q_heads, cache->n_kv_heads);
  VX_CHECK_ARG(!track || cache->acc, "%s: track needs the cache's acc", what);
  VX_CHECK_ARG(!track || (std::isfinite(track_decay) && track_decay >= 0.f), "%s: track_decay must be finite and >= 0",
               what);
  vx_attn_opts op = {};
  if (opts) op = *opts;
  VX_CHECK_ARG(op.window >= 0, "%s: window must be >= 0", what);
  // scale / cap and cap * 2 log2 e are formed in fp32.
  VX_CHECK_ARG(op.cap == 0.f || (op.cap >= 1e-18f && op.cap <= 1e18f), "%s: cap must be 0 or 1e-18 .. 1e18", what);
  VX_CHECK_ARG(std::isfinite(op.scale) && op.scale <= 1e18f, "%s: scale must be finite and at most 1e18", what);
  VX_CHECK_ARG((reinterpret_cast<uintptr_t>(op.prefix) & 3) == 0 && (reinterpret_cast<uintptr_t>(op.slopes) & 3) == 0 &&
                   (reinterpret_cast<uintptr_t>(lse) & 3) == 0,
               "%s: prefix, slopes or lse is misaligned", what);
  const int mq = static_cast<int>(max_q < n_tokens ? max_q : n_tokens);
  const int group = n_q_heads / cache->n_kv_heads;
  VX_CHECK_ARG(static_cast<int64_t>(mq) * group < (1ll << 30), "%s: max_q * (n_q_heads / n_kv_heads) must be below 2^30",
               what);
  const bool bf16 = cache->dt == VX_BF16;
  const int64_t kv = bound_kv(cache, max_kv);
  PagedAttnPlan plan = {0, 1, 1, 1, false};
  if (mq > 0) plan = plan_paged_attn(bf16, cache->head_dim, cache->n_seqs, cache->n_kv_heads, group, mq, kv);
  Carve cv{static_cast<uint8_t*>(ws), 0};
  const AttnCarve bf = carve_attn(cv, cache, n_tokens, n_q_heads, mq, plan, kv, lse != nullptr, track != 0);
  Launch L;
  if ((st = make_launch(&L, ws, ws_bytes, mq > 0 ? cv.off : kStatusBytes, stream)) != VX_OK) return st;
  if (mq == 0) return VX_OK;
  const int es = elem_size(cache->dt);
  if ((st = check_rows(q, es, n_q_heads, n_tokens, what, "q")) != VX_OK) return st;
  if ((st = check_rows(o, es, n_q_heads, n_tokens, what, "o")) != VX_OK) return st;
  const int64_t base = layer * layer_rows(cache);
  PagedAttnArgs a = {};
  a.c = view_of(cache);
  a.ch = {q_start, static_cast<int>(n_tokens), mq};
  a.k = static_cast<const uint8_t*>(cache->k) + base * cache->head_dim * es;
  a.v = static_cast<const uint8_t*>(cache->v) + base * cache->head_dim * es;
  a.q = {q->p, q->row, q->head};
  a.o = o->p;
  a.o_row = o->row;
  a.o_head = o->head;
  a.lse = lse ? lse : bf.lse;
  a.n_q_heads = n_q_heads;
  a.group = group;
  a.group_div = FastDiv::make(static_cast<uint32_t>(group));
  a.head_dim = cache->head_dim;
  a.window = op.window == 0 || op.window > kNoWindow ? kNoWindow : op.window;
  a.prefix = op.prefix;
  a.slopes = op.slopes;
  a.scale = op.scale > 0.f ? op.scale : 1.f / std::sqrt(static_cast<float>(cache->head_dim));
  a.cap = op.cap;
  a.acc = track ? cache->acc + base : nullptr;
  a.acc_decay = track_decay;
  a.splits = plan.splits;
  a.cluster = plan.cluster;
  a.parts = plan.splits / plan.cluster;
  a.part_o = bf.part_o;
  a.part_ml = bf.part_ml;
  a.w_segs = plan.w_segs;
  a.part_w = bf.part_w;
  a.part_stride = kv;
  a.scores = bf.scores;
  a.score_stride = score_stride(kv);
  a.status = L.status;
  a.limit_ns = L.limit_ns;
  const int64_t rows = static_cast<int64_t>(mq) * group;
  const int64_t blocks = plan.kernel == 1 ? (rows + 255) / 256 : plan.kernel == 2 ? (rows + 7) / 8 : 1;
  VX_CHECK_ARG(blocks * cache->n_seqs * cache->n_kv_heads * plan.splits < INT_MAX, "%s: too many row blocks", what);
  VX_CUDA(traced(L, plan.kernel == 0 ? "paged_attn_rows" : plan.kernel == 1 ? "paged_attn_tc" : "paged_attn_f32", 1, [&] {
    return plan.kernel == 0   ? launch_paged_attn_rows(L, a)
           : plan.kernel == 1 ? launch_paged_attn_tc(L, a)
                              : launch_paged_attn_f32(L, a);
  }));
  if (a.parts > 1 && a.scores == nullptr)   // with kept scores the sum of the weights does it
    VX_CUDA(traced(L, "paged_attn_combine", 1, [&] { return launch_paged_attn_combine(L, a, bf16); }));
  if (track)
    VX_CUDA(traced(L, "paged_attn_weights", plan.w_segs > 1 && !plan.keep_scores ? 2 : 1, [&] { return launch_paged_attn_weights(L, a, bf16, kv); }));
  return VX_OK;
}

size_t vx_paged_evict_workspace(const vx_paged_cache* cache, int64_t keep) {
  if (check_cache(cache, "vx_paged_evict_workspace") != VX_OK || keep < 0) return 0;
  const int64_t cap = static_cast<int64_t>(cache->max_pages) * cache->page_size;
  const int64_t m = keep < cap ? keep : cap;
  return align_up(kAlign + static_cast<size_t>(m) * cache->n_layers * cache->n_seqs * cache->n_kv_heads * 4, kAlign);
}

vx_status vx_paged_evict(const vx_paged_cache* cache, const vx_paged_cache* dst, int64_t keep, int64_t recent,
                         int32_t* kept, void* ws, size_t ws_bytes, cudaStream_t stream) {
  const char* what = "vx_paged_evict";
  vx_status st;
  if ((st = check_cache(cache, what)) != VX_OK) return st;
  if (dst == nullptr) dst = cache;
  if ((st = check_cache(dst, what)) != VX_OK) return st;
  VX_CHECK_ARG(cache->acc && dst->acc, "%s: the cache's acc is null", what);
  VX_CHECK_ARG(dst->dt == cache->dt && dst->n_layers == cache->n_layers && dst->n_kv_heads == cache->n_kv_heads &&
                   dst->head_dim == cache->head_dim && dst->n_seqs == cache->n_seqs &&
                   dst->page_size == cache->page_size,
               "%s: dst differs from the cache in dtype, layers, heads, head_dim, sequences or page_size", what);
  VX_CHECK_ARG((dst->k == cache->k) == (dst->v == cache->v) && (dst->k == cache->k) == (dst->acc == cache->acc),
               "%s: dst shares only some of k, v and acc with the cache", what);
  VX_CHECK_ARG(dst->k != cache->k || (dst->table == cache->table && dst->lens == cache->lens &&
                                      dst->n_pages == cache->n_pages && dst->max_pages == cache->max_pages),
               "%s: dst on the cache's own pages must be the cache itself", what);
  VX_CHECK_ARG(dst->k == cache->k || dst->lens != cache->lens, "%s: dst has pages of its own but the cache's lens", what);
  VX_CHECK_ARG(keep >= 0 && recent >= 0, "%s: keep and recent must be >= 0", what);
  VX_CHECK_ARG((reinterpret_cast<uintptr_t>(kept) & 3) == 0, "%s: kept is misaligned", what);
  const int64_t cap = static_cast<int64_t>(cache->max_pages) * cache->page_size;
  Launch L;
  const size_t need = kept ? kStatusBytes : vx_paged_evict_workspace(cache, keep);
  if ((st = make_launch(&L, ws, ws_bytes, need, stream)) != VX_OK) return st;
  EvictArgs a = {};
  a.src = view_of(cache);
  a.dst = view_of(dst);
  a.k = static_cast<const uint8_t*>(cache->k);
  a.v = static_cast<const uint8_t*>(cache->v);
  a.acc = cache->acc;
  a.dk = static_cast<uint8_t*>(dst->k);
  a.dv = static_cast<uint8_t*>(dst->v);
  a.dacc = dst->acc;
  a.src_pos = cache->pos;
  a.dst_lens = dst->lens;
  a.dst_pos = dst->pos;
  a.src_layer_rows = layer_rows(cache);
  a.dst_layer_rows = layer_rows(dst);
  a.n_layers = cache->n_layers;
  a.row_bytes = cache->head_dim * elem_size(cache->dt);
  a.keep = keep < cap ? keep : cap;
  a.recent = recent < cap ? recent : cap;
  a.kept_stride = keep < cap || kept == nullptr ? a.keep : keep;
  a.kept = kept ? kept : reinterpret_cast<int32_t*>(static_cast<uint8_t*>(ws) + kAlign);
  a.status = L.status;
  VX_CUDA(traced(L, "paged_evict", 2, [&] { return launch_paged_evict(L, a); }));
  return VX_OK;
}

}  // extern "C"
