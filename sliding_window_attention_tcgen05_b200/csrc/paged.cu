// paged.cu -- rotary positions, the append to the paged K/V cache and the
// eviction from it (all bound by HBM, or by the launch for a step's few rows).
//
// rope_fwd_kernel: y = rotary(x) over strided rows of heads.
// paged_append_kernel: the chunk's K (rotated) and V rows into their pages,
//   q rotated into its output in the same launch.
// paged_advance_kernel: lens += n, pos += n.
// evict_select_kernel / evict_move_kernel: the slots with the largest
//   accumulated weight, and their move to the front.
#include "vx_paged.h"

namespace vx {

namespace {

// cos and sin (times mscale) of pos * f_m.  The product wraps modulo one turn
// in 64-bit arithmetic, so no range reduction is left to do: the top 32 bits,
// as a signed number, are the angle in units of 2^-31 * pi.
__device__ __forceinline__ float2 rope_cs(int64_t pos, uint64_t turns, float mscale) {
  const uint64_t frac = static_cast<uint64_t>(pos) * turns;
  const int32_t top = static_cast<int32_t>((frac + 0x80000000ull) >> 32);
  float s, c;
  sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  return make_float2(c * mscale, s * mscale);
}

template <bool BF16>
struct Vec {   // one 16-byte access
  static constexpr int N = BF16 ? 8 : 4;
  float f[N];
  __device__ __forceinline__ void load(const void* p) {
    if constexpr (BF16) {
      const uint4 a = *static_cast<const uint4*>(p);
      f[0] = bf16lo(a.x); f[1] = bf16hi(a.x); f[2] = bf16lo(a.y); f[3] = bf16hi(a.y);
      f[4] = bf16lo(a.z); f[5] = bf16hi(a.z); f[6] = bf16lo(a.w); f[7] = bf16hi(a.w);
    } else {
      const float4 a = *static_cast<const float4*>(p);
      f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    }
  }
  __device__ __forceinline__ void store(void* p) const {
    if constexpr (BF16)
      *static_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                           pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    else
      *static_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};

template <bool BF16>
__device__ __forceinline__ float ld1(const void* p, int64_t e) {
  if constexpr (BF16) return bf16_to_f(static_cast<const uint16_t*>(p)[e]);
  else return static_cast<const float*>(p)[e];
}
template <bool BF16>
__device__ __forceinline__ void st1(void* p, int64_t e, float x) {
  if constexpr (BF16) {
    const __nv_bfloat16 r = __float2bfloat16_rn(x);
    static_cast<uint16_t*>(p)[e] = *reinterpret_cast<const uint16_t*>(&r);
  } else {
    static_cast<float*>(p)[e] = x;
  }
}

// One head's work is cut into units.  Vector path (16-byte accesses, V
// elements): half layout: rot/2/V units of a vector at m and one at m + rot/2,
// interleaved: rot/V units of one vector; then (D - rot)/V copies.
template <bool BF16>
__device__ __forceinline__ int rope_units(int D, int pairs, bool inter) {
  constexpr int V = Vec<BF16>::N;
  return (inter ? 2 * pairs / V : pairs / V) + (D - 2 * pairs) / V;
}

// cs: the token's cosines and sines in shared memory (float2 per pair).
template <bool BF16>
__device__ __forceinline__ void rope_unit(const uint8_t* src, uint8_t* dst, int u, int pairs, bool inter,
                                          const float2* cs, bool skip_copy) {
  constexpr int V = Vec<BF16>::N;
  constexpr int ES = BF16 ? 2 : 4;
  const int nrot = inter ? 2 * pairs / V : pairs / V;
  if (u >= nrot) {
    if (skip_copy) return;
    const int e = 2 * pairs + (u - nrot) * V;
    *reinterpret_cast<uint4*>(dst + e * ES) = *reinterpret_cast<const uint4*>(src + e * ES);
    return;
  }
  if (inter) {
    Vec<BF16> a, y;
    a.load(src + u * V * ES);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float2 w = cs[u * (V / 2) + i / 2];
      y.f[i] = a.f[i] * w.x - a.f[i + 1] * w.y;
      y.f[i + 1] = a.f[i + 1] * w.x + a.f[i] * w.y;
    }
    y.store(dst + u * V * ES);
  } else {
    Vec<BF16> a, b, ya, yb;
    a.load(src + u * V * ES);
    b.load(src + (pairs + u * V) * ES);
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const float2 w = cs[u * V + i];
      ya.f[i] = a.f[i] * w.x - b.f[i] * w.y;
      yb.f[i] = b.f[i] * w.x + a.f[i] * w.y;
    }
    ya.store(dst + u * V * ES);
    yb.store(dst + (pairs + u * V) * ES);
  }
}

// Block: `tok` tokens of the chunk (their cosines and sines computed once in
// shared memory, for all heads), threads over (token, head, unit).
template <bool BF16>
__global__ void __launch_bounds__(256) rope_fwd_kernel(const __grid_constant__ RopeArgs2 a,
                                                       const __grid_constant__ RopeTable t, int tok) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float2 cs[];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok;
  const int nt = static_cast<int>(a.n_tokens - t0 < tok ? a.n_tokens - t0 : tok);
  for (int i = threadIdx.x; i < nt * t.pairs; i += blockDim.x)
    cs[i] = rope_cs(a.pos[t0 + i / t.pairs], t.turns[i % t.pairs], t.mscale);
  __syncthreads();
  constexpr int ES = BF16 ? 2 : 4;
  const bool inter = t.interleaved != 0;
  if (a.vec) {
    const int units = rope_units<BF16>(a.head_dim, t.pairs, inter);
    for (int i = threadIdx.x; i < nt * a.n_heads * units; i += blockDim.x) {
      const int u = i % units, h = (i / units) % a.n_heads, r = i / (units * a.n_heads);
      const uint8_t* src = static_cast<const uint8_t*>(a.x.p) + ((t0 + r) * a.x.row + h * a.x.head) * ES;
      uint8_t* dst = static_cast<uint8_t*>(a.y) + ((t0 + r) * a.y_row + h * a.y_head) * ES;
      rope_unit<BF16>(src, dst, u, t.pairs, inter, cs + r * t.pairs, a.in_place);
    }
  } else {   // element by element: unit = one pair, or one copied element
    const int units = t.pairs + a.head_dim - 2 * t.pairs;
    for (int i = threadIdx.x; i < nt * a.n_heads * units; i += blockDim.x) {
      const int u = i % units, h = (i / units) % a.n_heads, r = i / (units * a.n_heads);
      const int64_t xs = (t0 + r) * a.x.row + h * a.x.head, ys = (t0 + r) * a.y_row + h * a.y_head;
      if (u >= t.pairs) {
        if (!a.in_place) st1<BF16>(a.y, ys + t.pairs + u, ld1<BF16>(a.x.p, xs + t.pairs + u));
        continue;
      }
      const int e0 = inter ? 2 * u : u, e1 = inter ? 2 * u + 1 : u + t.pairs;
      const float2 w = cs[r * t.pairs + u];
      const float x0 = ld1<BF16>(a.x.p, xs + e0), x1 = ld1<BF16>(a.x.p, xs + e1);
      st1<BF16>(a.y, ys + e0, x0 * w.x - x1 * w.y);
      st1<BF16>(a.y, ys + e1, x1 * w.x + x0 * w.y);
    }
  }
}

// Grid (row blocks of a sequence, sequences).  Threads over (token, head,
// unit) with the heads numbered q, k, v; v (and all of them without rope) is
// copied in 16-byte units.
template <bool BF16>
__global__ void __launch_bounds__(256) paged_append_kernel(const __grid_constant__ AppendArgs a,
                                                           const __grid_constant__ RopeTable t, int tok) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ float2 cs[];
  __shared__ int64_t s_row[32];   // row of K/V head 0, or -1 (tok <= 32)
  const int s = blockIdx.y;
  const SeqSpan sp = seq_span(a.c, a.ch, s);
  const int t0 = blockIdx.x * tok;
  const int nt = min(sp.n - t0, tok);
  if (nt <= 0) return;
  if (sp.over && threadIdx.x == 0) report_bad_cache(a.status, s);
  const int64_t pos0 = a.rope ? a.pos[s] + t0 : 0;
  if (a.rope)
    for (int i = threadIdx.x; i < nt * t.pairs; i += blockDim.x)
      cs[i] = rope_cs(pos0 + i / t.pairs, t.turns[i % t.pairs], t.mscale);
  if (threadIdx.x < nt) {
    const int j = sp.old + t0 + static_cast<int>(threadIdx.x);
    const int64_t row = j < sp.kv ? slot_row(a.c, s, 0, j) : -1;
    if (row < 0) report_bad_cache(a.status, s);
    s_row[threadIdx.x] = row;
  }
  __syncthreads();
  constexpr int ES = BF16 ? 2 : 4;
  const int D = a.head_dim, V = 16 / ES, ps = a.c.page.d;
  const bool inter = t.interleaved != 0;
  const int Hk = a.c.n_heads, Hq = a.n_q_heads;
  const int64_t g0 = sp.row0 + t0;
  const int ru = a.rope ? rope_units<BF16>(D, t.pairs, inter) : D / V, cu = D / V;
  const int nrot = (Hq + Hk) * ru, per = nrot + Hk * cu;
  for (int i = threadIdx.x; i < nt * per; i += blockDim.x) {
    const int r = i / per, w = i - r * per;
    if (w < nrot) {
      const int h = w / ru, u = w - h * ru;
      const uint8_t* src;
      uint8_t* dst;
      bool same = false;
      if (h < Hq) {
        src = static_cast<const uint8_t*>(a.q.p) + ((g0 + r) * a.q.row + h * a.q.head) * ES;
        dst = static_cast<uint8_t*>(a.q_out) + ((g0 + r) * a.qo_row + h * a.qo_head) * ES;
        same = src == dst;
      } else {
        if (s_row[r] < 0) continue;
        src = static_cast<const uint8_t*>(a.k.p) + ((g0 + r) * a.k.row + (h - Hq) * a.k.head) * ES;
        dst = static_cast<uint8_t*>(a.k_pool) + (s_row[r] + static_cast<int64_t>(h - Hq) * ps) * D * ES;
      }
      if (a.rope)
        rope_unit<BF16>(src, dst, u, t.pairs, inter, cs + r * t.pairs, same);
      else
        *reinterpret_cast<uint4*>(dst + u * 16) = *reinterpret_cast<const uint4*>(src + u * 16);
    } else if (s_row[r] >= 0) {
      const int h = (w - nrot) / cu, u = (w - nrot) - h * cu;
      const int64_t row = s_row[r] + static_cast<int64_t>(h) * ps;
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(a.v_pool) + row * D * ES + u * 16) =
          *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(a.v.p) +
                                          ((g0 + r) * a.v.row + h * a.v.head) * ES + u * 16);
      if (a.acc != nullptr && u == 0) a.acc[row] = 0.f;
    }
  }
}

__global__ void paged_advance_kernel(const __grid_constant__ PagedView c, const __grid_constant__ ChunkArgs ch,
                                     int64_t* lens, int64_t* pos, DevStatus* status) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  if (s >= c.n_seqs) return;
  const SeqSpan sp = seq_span(c, ch, s);
  if (sp.over) report_bad_cache(status, s);
  lens[s] = sp.kv;
  pos[s] += sp.n;
}

// -------------------------------------------------------------- eviction --
// Order-preserving image of a weight: larger value, larger key; NaN lowest.
__device__ __forceinline__ uint32_t weight_key(float x) {
  if (x != x) return 0u;
  const uint32_t b = __float_as_uint(x == 0.f ? 0.f : x);   // -0 equals +0
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ int64_t evict_len(const EvictArgs& a, int s, bool* bad) {
  const int64_t cap = static_cast<int64_t>(a.src.max_pages) * a.src.page.d;
  const int64_t len = a.src.lens[s];
  *bad = len < 0 || len > cap;
  return len < 0 ? 0 : len < cap ? len : cap;
}

constexpr int kSelThreads = 1024;

// CTA per (head, sequence, layer): the bar (the (m - r)-th largest key among
// the first L - r slots) by a radix selection of four 8-bit digits, then one
// pass that writes the kept slots in slot order, counting equals of the bar
// from the lowest slot.
__global__ void __launch_bounds__(kSelThreads) evict_select_kernel(const __grid_constant__ EvictArgs a) {
  pdl_wait();
  pdl_trigger();
  __shared__ int hist[256];
  __shared__ int s_digit, s_rest;
  __shared__ int wsum[2][32];
  const int h = blockIdx.x, s = blockIdx.y, l = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad;
  const int L = static_cast<int>(evict_len(a, s, &bad));
  if (bad && tid == 0) report_bad_cache(a.status, s);
  const int m = static_cast<int>(a.keep < L ? a.keep : L);
  const int r = static_cast<int>(a.recent < m ? a.recent : m);
  const int n = L - r, want = m - r;
  int32_t* out = a.kept + ((static_cast<int64_t>(l) * a.src.n_seqs + s) * a.src.n_heads + h) * a.kept_stride;
  const float* acc = a.acc + l * a.src_layer_rows;
  for (int i = tid; i < r; i += kSelThreads) out[want + i] = n + i;
  if (want <= 0) return;
  auto key_at = [&](int j) -> uint32_t {
    const int64_t row = slot_row(a.src, s, h, j);
    return row < 0 ? 0u : weight_key(acc[row]);
  };
  uint32_t bar = 0, mask = 0;
  int rest = want;   // how many of the keys that match bar's known digits are wanted
  if (want < n) {
    for (int shift = 24; shift >= 0; shift -= 8) {
      if (tid < 256) hist[tid] = 0;
      __syncthreads();
      for (int j = tid; j < n; j += kSelThreads) {
        const uint32_t key = key_at(j);
        if ((key & mask) == bar) atomicAdd(&hist[(key >> shift) & 255u], 1);
      }
      __syncthreads();
      if (tid == 0) {
        int left = rest, d = 255;
        while (d > 0 && hist[d] < left) left -= hist[d--];
        s_digit = d;
        s_rest = left;
      }
      __syncthreads();
      bar |= static_cast<uint32_t>(s_digit) << shift;
      mask |= 255u << shift;
      rest = s_rest;
      __syncthreads();
    }
  }
  // Keys above the bar are kept, and the first `rest` of its equals (all of
  // the slots when none has to go).
  int kept = 0, equals = 0;
  for (int j0 = 0; j0 < n; j0 += kSelThreads) {
    const int j = j0 + tid;
    bool more = false, same = false;
    if (j < n) {
      if (want == n) {
        more = true;
      } else {
        const uint32_t key = key_at(j);
        more = key > bar;
        same = key == bar;
      }
    }
    const uint32_t bs = __ballot_sync(0xffffffffu, same);
    if (lane == 0) wsum[0][warp] = __popc(bs);
    __syncthreads();
    int before = equals, total = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) before += wsum[0][w];
      total += wsum[0][w];
    }
    const bool take = more || (same && before + __popc(bs & ((1u << lane) - 1)) < rest);
    const uint32_t bt = __ballot_sync(0xffffffffu, take);
    if (lane == 0) wsum[1][warp] = __popc(bt);
    __syncthreads();
    int at = kept, taken = 0;
    for (int w = 0; w < 32; ++w) {
      if (w < warp) at += wsum[1][w];
      taken += wsum[1][w];
    }
    if (take) out[at + __popc(bt & ((1u << lane) - 1))] = j;
    equals += total;
    kept += taken;
    __syncthreads();
  }
}

// Grid (head x slice, sequence, layer).  The kept rows move to the front in
// slot order.  In place a row's new slot is never above its old one, so a CTA
// that reads a chunk of rows before it writes that chunk, chunk after chunk,
// never overwrites a row it still has to read; the K and V rows are cut into
// slices of 64 bytes that different CTAs move, each for itself.
constexpr int kMoveThreads = 256;
constexpr int kSliceBytes = 64;                              // of a K or V row
constexpr int kMoveRows = kMoveThreads / (kSliceBytes / 16); // rows of a chunk: 64
constexpr int kMoveDeep = 4;                                 // chunks read together

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a, int slices) {
  pdl_wait();
  pdl_trigger();
  const int h = blockIdx.x / slices, slice = blockIdx.x % slices, s = blockIdx.y, l = blockIdx.z;
  bool bad;
  const int64_t L = evict_len(a, s, &bad);
  const int m = static_cast<int>(a.keep < L ? a.keep : L);
  const int64_t dcap = static_cast<int64_t>(a.dst.max_pages) * a.dst.page.d;
  const int32_t* kept = a.kept + ((static_cast<int64_t>(l) * a.src.n_seqs + s) * a.src.n_heads + h) * a.kept_stride;
  const bool in_place = a.k == a.dk;
  const int per_tensor = (slices - 1) / 2;   // slices of K, then of V, then one of acc
  auto rows_of = [&](int i, int64_t* from, int64_t* to) {
    *from = slot_row(a.src, s, h, kept[i]);
    *to = i < dcap ? slot_row(a.dst, s, h, i) : -1;
    if (*from < 0 || *to < 0) report_bad_cache(a.status, s);
  };
  if (slice == slices - 1) {
    const float* src = a.acc + l * a.src_layer_rows;
    float* dst = a.dacc + l * a.dst_layer_rows;
    for (int i0 = 0; i0 < m; i0 += kMoveThreads) {
      const int i = i0 + threadIdx.x;
      int64_t from = -1, to = -1;
      if (i < m) rows_of(i, &from, &to);
      const float x = from >= 0 ? src[from] : 0.f;
      if (in_place) __syncthreads();
      if (to >= 0 && !(in_place && from == to)) dst[to] = x;
    }
    return;
  }
  const bool is_v = slice >= per_tensor;
  const int64_t byte0 = static_cast<int64_t>(is_v ? slice - per_tensor : slice) * kSliceBytes +
                        (threadIdx.x % (kSliceBytes / 16)) * 16;
  const uint8_t* src = (is_v ? a.v : a.k) + l * a.src_layer_rows * a.row_bytes + byte0;
  uint8_t* dst = (is_v ? a.dv : a.dk) + l * a.dst_layer_rows * a.row_bytes + byte0;
  const int rr = threadIdx.x / (kSliceBytes / 16);
  for (int i0 = 0; i0 < m; i0 += kMoveRows * kMoveDeep) {
    uint4 x[kMoveDeep];
    int64_t from[kMoveDeep], to[kMoveDeep];
#pragma unroll
    for (int d = 0; d < kMoveDeep; ++d) {
      const int i = i0 + d * kMoveRows + rr;
      from[d] = to[d] = -1;
      x[d] = make_uint4(0u, 0u, 0u, 0u);
      if (i < m) rows_of(i, &from[d], &to[d]);
      if (from[d] >= 0 && !(in_place && from[d] == to[d])) x[d] = *reinterpret_cast<const uint4*>(src + from[d] * a.row_bytes);
    }
    if (in_place) __syncthreads();
#pragma unroll
    for (int d = 0; d < kMoveDeep; ++d)
      if (to[d] >= 0 && !(in_place && from[d] == to[d])) *reinterpret_cast<uint4*>(dst + to[d] * a.row_bytes) = x[d];
  }
}

__global__ void evict_lens_kernel(const __grid_constant__ EvictArgs a) {
  pdl_wait();
  pdl_trigger();
  const int s = blockIdx.x * blockDim.x + threadIdx.x;
  if (s >= a.src.n_seqs) return;
  bool bad;
  const int64_t L = evict_len(a, s, &bad);
  const int64_t dcap = static_cast<int64_t>(a.dst.max_pages) * a.dst.page.d;
  const int64_t m = a.keep < L ? a.keep : L;
  a.dst_lens[s] = m < dcap ? m : dcap;
  if (a.dst_pos != a.src_pos) a.dst_pos[s] = a.src_pos[s];
}

}  // namespace

cudaError_t launch_rope_rows(cudaStream_t stream, const RopeArgs2& a, const RopeTable& t) {
  // Tokens per block: about 16 KB of rows, so that few heads do not leave
  // blocks of a handful of threads' work, at most 32 tokens.
  const int64_t row = static_cast<int64_t>(a.n_heads) * a.head_dim * (a.bf16 ? 2 : 4);
  int64_t tok = (16384 + row - 1) / row;
  tok = tok < 1 ? 1 : tok > 32 ? 32 : tok;
  if (a.n_tokens < tok * 148) tok = 1;
  const unsigned grid = static_cast<unsigned>((a.n_tokens + tok - 1) / tok);
  const size_t smem = static_cast<size_t>(tok) * t.pairs * sizeof(float2);
  return a.bf16 ? launch_kernel(rope_fwd_kernel<true>, dim3(grid), dim3(256), smem, stream, a, t, static_cast<int>(tok))
                : launch_kernel(rope_fwd_kernel<false>, dim3(grid), dim3(256), smem, stream, a, t,
                                static_cast<int>(tok));
}

cudaError_t launch_paged_append(cudaStream_t stream, const AppendArgs& a, const RopeTable& t) {
  const int64_t row = static_cast<int64_t>(a.n_q_heads + 2 * a.c.n_heads) * a.head_dim * (a.bf16 ? 2 : 4);
  int64_t tok = (16384 + row - 1) / row;
  tok = tok < 1 ? 1 : tok > 32 ? 32 : tok;
  if (static_cast<int64_t>(a.ch.max_q) * a.c.n_seqs < tok * 148) tok = 1;
  const dim3 grid(static_cast<unsigned>((a.ch.max_q + tok - 1) / tok), static_cast<unsigned>(a.c.n_seqs));
  const size_t smem = a.rope ? static_cast<size_t>(tok) * t.pairs * sizeof(float2) : 0;
  return a.bf16 ? launch_kernel(paged_append_kernel<true>, grid, dim3(256), smem, stream, a, t, static_cast<int>(tok))
                : launch_kernel(paged_append_kernel<false>, grid, dim3(256), smem, stream, a, t,
                                static_cast<int>(tok));
}

cudaError_t launch_paged_advance(cudaStream_t stream, const PagedView& c, const ChunkArgs& ch, int64_t* lens,
                                 int64_t* pos, DevStatus* status) {
  return launch_kernel(paged_advance_kernel, dim3((c.n_seqs + 127) / 128), dim3(128), 0, stream, c, ch, lens, pos,
                       status);
}

cudaError_t launch_paged_evict(const Launch& L, const EvictArgs& a) {
  const unsigned S = static_cast<unsigned>(a.src.n_seqs), nl = static_cast<unsigned>(a.n_layers);
  const unsigned H = static_cast<unsigned>(a.src.n_heads);
  cudaError_t e = launch_kernel(evict_select_kernel, dim3(H, S, nl), dim3(kSelThreads), 0, L.stream, a);
  if (e != cudaSuccess) return e;
  const int slices = 2 * (a.row_bytes / kSliceBytes) + 1;
  e = launch_kernel(evict_move_kernel, dim3(H * slices, S, nl), dim3(kMoveThreads), 0, L.stream, a, slices);
  if (e != cudaSuccess) return e;
  return launch_kernel(evict_lens_kernel, dim3((S + 127) / 128), dim3(128), 0, L.stream, a);
}

}  // namespace vx
