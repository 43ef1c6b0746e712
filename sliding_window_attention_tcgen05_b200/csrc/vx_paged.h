// vx_paged.h -- the paged K/V cache as the kernels see it, and the launchers
// of the operators over it (rotary positions, append, attention, eviction).
#pragma once

#include "vx_internal.h"

namespace vx {

constexpr int kStatusBadCache = 1;   // DevStatus::code (VX_ERR_INVALID_ARG); `where` = the sequence

// n / d for 0 <= n < 2^31 by a multiplication (Granlund and Montgomery,
// "Division by Invariant Integers using Multiplication", 1994): with l =
// ceil(log2 d) and m = floor(2^32 (2^l - d) / d) + 1, n / d = (hi(m n) + n) >> l.
struct FastDiv {
  uint32_t d, m, l;
  __host__ static FastDiv make(uint32_t d) {
    uint32_t l = 0;
    while ((1ull << l) < d) ++l;
    const uint64_t m = ((1ull << 32) * ((1ull << l) - d)) / d + 1;
    return {d, static_cast<uint32_t>(m), l};
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const { return (__umulhi(m, n) + n) >> l; }
};

// One layer of the cache, passed to kernels by value.
struct PagedView {
  const int32_t* table;
  const int64_t* lens;
  FastDiv page;        // slots per page
  int n_pages, n_heads, max_pages, n_seqs;
};

// The rows of a chunk: q_start, clamped to the tensors' rows and to max_q.
struct ChunkArgs {
  const int32_t* q_start;
  int n_tokens, max_q;
};

// Sequence s: its first row, its row count and the slots it holds before the
// chunk (old) and with it (kv, at most the table's capacity).
struct SeqSpan {
  int row0, n, old, kv;
  bool over;           // old + n exceeded the capacity
};

__device__ __forceinline__ SeqSpan seq_span(const PagedView& c, const ChunkArgs& ch, int s) {
  SeqSpan r;
  const int a = min(max(ch.q_start[s], 0), ch.n_tokens);
  const int b = min(max(ch.q_start[s + 1], a), ch.n_tokens);
  const int64_t cap = static_cast<int64_t>(c.max_pages) * c.page.d;   // < 2^30
  const int64_t len = c.lens[s];
  r.row0 = a;
  r.n = min(b - a, ch.max_q);
  r.old = static_cast<int>(len < 0 ? 0 : len < cap ? len : cap);
  const int64_t kv = static_cast<int64_t>(r.old) + r.n;
  r.kv = static_cast<int>(kv < cap ? kv : cap);
  r.over = kv > cap || len < 0 || len > cap;
  return r;
}

__device__ __forceinline__ void report_bad_cache(DevStatus* st, int s) {
  if (st != nullptr && atomicCAS(&st->code, 0, kStatusBadCache) == 0) st->where = s;
}

// Row index ((page, head, row) flattened, in units of one head's row) of slot
// j, or -1 when the table's entry is not a page of the pool.  j must lie below
// max_pages * page size; a layer's pool has fewer than 2^31 rows.
__device__ __forceinline__ int slot_row(const PagedView& c, int s, int head, int j) {
  const uint32_t pg = c.page.div(static_cast<uint32_t>(j));
  const int id = c.table[static_cast<int64_t>(s) * c.max_pages + pg];
  if (id < 0 || id >= c.n_pages) return -1;
  const int page = static_cast<int>(c.page.d);
  return (id * c.n_heads + head) * page + (j - static_cast<int>(pg) * page);
}

// ---------------------------------------------------------------- rotary --
// Angles as fractions of a turn: turns[m] = round(f_m / 2 pi * 2^64), so
// pos * turns[m] mod 2^64 is the fraction of a turn of pos * f_m up to |pos|
// times the error of turns[m]: 2^-65 of its rounding and, f_m being a product of
// up to seven powers in 64-bit mantissas, a few 2^-64 of f_m's own, together
// below 2^-61.
constexpr int kMaxRotPairs = 128;
constexpr int kMaxTok = 32;   // tokens of a block
struct RopeTable {
  uint64_t turns[kMaxRotPairs];
  float mscale;
  int pairs;           // rot_dim / 2 (0: copies only)
  int interleaved;
};

// Strided rows of heads (element strides).
struct RowsView {
  const void* p;
  int64_t row, head;
};

struct RopeArgs2 {
  RowsView x;
  void* y;
  int64_t y_row, y_head;
  const int64_t* pos;
  int64_t n_tokens;
  int n_heads, head_dim;
  bool bf16, vec, in_place;   // vec: 16-byte accesses of 8 (bf16) or 4 (fp32) elements are possible
  FastDiv units, heads;       // work units of a head, heads (set by the launcher)
};
cudaError_t launch_rope_rows(cudaStream_t stream, const RopeArgs2& a, const RopeTable& t);

struct AppendArgs {
  PagedView c;
  ChunkArgs ch;
  const int64_t* pos;
  void *k_pool, *v_pool;   // of the layer
  float* acc;              // of the layer, or null
  RowsView q, k, v;
  void* q_out;
  int64_t qo_row, qo_head;
  int n_q_heads, head_dim;
  bool bf16;
  FastDiv units, per;      // work units of a rotated head, of a token (set by the launcher)
  DevStatus* status;
};
cudaError_t launch_paged_append(cudaStream_t stream, const AppendArgs& a, const RopeTable& t);
cudaError_t launch_paged_advance(cudaStream_t stream, const PagedView& c, const ChunkArgs& ch, int64_t* lens,
                                 int64_t* pos, DevStatus* status);

// ------------------------------------------------------------- attention --
struct PagedAttnArgs {
  PagedView c;
  ChunkArgs ch;
  const void *k, *v;       // pools of the layer
  RowsView q;
  void* o;
  int64_t o_row, o_head;
  float* lse;              // [n_tokens, n_q_heads] or null
  int n_q_heads, group, head_dim;
  FastDiv group_div;
  int window;              // > 0 (INT_MAX / 2 for none)
  const int32_t* prefix;   // [n_seqs] or null
  const float* slopes;     // [n_q_heads] or null
  float scale;             // of the raw scores
  float cap;               // 0 = none
  float* acc;              // of the layer (track) or null
  float acc_decay;
  int w_segs;              // segments of the rows in the sum of the weights
  float* scores;           // [n_seqs][n_heads][max_q * group][score_stride] (plan's keep_scores) or null
  int64_t score_stride;    // of list positions, a multiple of 4
  float* part_w;           // [w_segs][n_seqs][n_heads][part_stride] (w_segs > 1)
  int64_t part_stride;     // slots
  int splits;              // CTAs that every sequence's key range is cut into
  int cluster;             // of them join their results in shared memory (rows kernel)
  int parts;               // splits / cluster: results left to the combining kernel
  float* part_o;           // [parts][n_tokens][n_q_heads][head_dim] (parts > 1)
  float2* part_ml;         // [parts][n_tokens][n_q_heads]: running max (log2) and sum
  DevStatus* status;
  uint64_t limit_ns;
};

// Which kernel runs and into how many parts the keys are split.
struct PagedAttnPlan {
  int kernel;    // 0: warp-level rows kernel, 1: tcgen05 kernel, 2: fp32 kernel
  int splits;    // CTAs that every sequence's key range is cut into
  int cluster;   // of them that join their results themselves (1, 2, 4 or 8)
  int w_segs;    // segments of the rows in the sum of the weights (track)
  bool keep_scores;   // the rows kernel leaves its scores for the sum of the weights (track)
};
PagedAttnPlan plan_paged_attn(bool bf16, int head_dim, int n_seqs, int n_kv_heads, int group, int max_q,
                              int64_t max_kv);

// -------------------------------------------------------------- eviction --
struct EvictArgs {
  PagedView src, dst;
  const uint8_t *k, *v;
  const float* acc;
  uint8_t *dk, *dv;
  float* dacc;
  const int64_t* src_pos;
  int64_t *dst_lens, *dst_pos;
  int64_t src_layer_rows, dst_layer_rows;   // rows of one layer's pool
  int n_layers, row_bytes;
  int64_t keep, recent;
  int32_t* kept;           // [n_layers][n_seqs][n_heads][kept_stride]
  int64_t kept_stride;
  DevStatus* status;
};
cudaError_t launch_paged_evict(const Launch& L, const EvictArgs& a);

}  // namespace vx
