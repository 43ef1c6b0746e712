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

// Eight bf16 or four fp32 elements: one 16-byte access, widened to fp32 and back.
template <bool BF16>
struct Vec {
  static constexpr int N = BF16 ? 8 : 4;
  float f[N];
  __device__ __forceinline__ explicit Vec(const uint4& a) {
    if constexpr (BF16) {
      f[0] = bf16lo(a.x); f[1] = bf16hi(a.x); f[2] = bf16lo(a.y); f[3] = bf16hi(a.y);
      f[4] = bf16lo(a.z); f[5] = bf16hi(a.z); f[6] = bf16lo(a.w); f[7] = bf16hi(a.w);
    } else {
      f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
    }
  }
  __device__ __forceinline__ uint4 bits() const {
    if constexpr (BF16)
      return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                        pack_bf16x2(f[6], f[7]));
    else
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
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

// One head's work is cut into units of 16-byte vectors of V elements.  Half
// layout: pairs / V units of a vector at m and one at m + pairs; interleaved:
// 2 pairs / V units of one vector; then (D - 2 pairs) / V copies.
//
// A thread takes one unit at a time: what counts is the number of threads in
// flight (16384 rows of 40 heads of 128, bf16: 59 us, 87% of copy bandwidth; two
// units a thread at 48 registers 66, four at 78 registers 77).
constexpr int kRopeBlocks = 6;   // resident blocks an SM: at most 40 registers
constexpr int kAppendBlocks = 5;   // 48 (prompts of up to 4001 tokens, 32 + 8 + 8 heads of 128: 68 us; at 64 registers 72)

// Place of pair m among a token's cosines and sines: a unit of G pairs reads
// them two by two, and the same two of neighbouring units are neighbours, so
// that the lanes of a warp read shared memory without conflicts.
template <bool BF16, bool INTER>
__device__ __forceinline__ int cs_place(int m, int pairs) {
  constexpr int G = INTER ? Vec<BF16>::N / 2 : Vec<BF16>::N;
  return ((m % G) / 2 * (pairs / G) + m / G) * 2 + m % 2;
}

struct Unit {
  const uint8_t* src;
  int first;            // its first two pairs among the token's float4s; below 0: a copy
  int at;               // bytes from the head's start, source and destination
};

// Unit u of a head whose elements start at src.
template <bool BF16, bool INTER>
__device__ __forceinline__ Unit rope_unit(const uint8_t* src, int u, int pairs) {
  const int nrot = (INTER ? 2 * pairs : pairs) / Vec<BF16>::N;
  const bool rot = u < nrot;
  const int o = (rot || INTER ? u : u + nrot) * 16;
  return {src + o, rot ? u : -1, o};
}

template <bool BF16, bool INTER>
__device__ __forceinline__ void load_unit(const Unit& w, int pairs, uint4& x, uint4& x1) {
  x = *reinterpret_cast<const uint4*>(w.src);
  if (!INTER && w.first >= 0) x1 = *reinterpret_cast<const uint4*>(w.src + pairs * (BF16 ? 2 : 4));
}

// dst: where the head's elements go; cs: the token's cosines and sines.
template <bool BF16, bool INTER>
__device__ __forceinline__ void store_unit(const Unit& w, int pairs, const uint4& x, const uint4& x1, uint8_t* dst,
                                           const float2* cs) {
  constexpr int V = Vec<BF16>::N;
  dst += w.at;
  if (w.first < 0) {
    *reinterpret_cast<uint4*>(dst) = x;
    return;
  }
  const float4* c4 = reinterpret_cast<const float4*>(cs) + w.first;
  const int nu = pairs / (INTER ? V / 2 : V);
  Vec<BF16> a(x);
  if constexpr (INTER) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      const float4 c = c4[i / 4 * nu];
      const float y = a.f[i] * c.x - a.f[i + 1] * c.y, z = a.f[i + 2] * c.z - a.f[i + 3] * c.w;
      a.f[i + 1] = a.f[i + 1] * c.x + a.f[i] * c.y;
      a.f[i + 3] = a.f[i + 3] * c.z + a.f[i + 2] * c.w;
      a.f[i] = y;
      a.f[i + 2] = z;
    }
  } else {
    const int half = pairs * (BF16 ? 2 : 4);   // bytes from m to m + pairs
    Vec<BF16> b(x1);
#pragma unroll
    for (int i = 0; i < V; i += 2) {
      const float4 c = c4[i / 2 * nu];
      const float y = a.f[i] * c.x - b.f[i] * c.y, z = a.f[i + 1] * c.z - b.f[i + 1] * c.w;
      b.f[i] = b.f[i] * c.x + a.f[i] * c.y;
      b.f[i + 1] = b.f[i + 1] * c.z + a.f[i + 1] * c.w;
      a.f[i] = y;
      a.f[i + 1] = z;
    }
    *reinterpret_cast<uint4*>(dst + half) = b.bits();
  }
  *reinterpret_cast<uint4*>(dst) = a.bits();
}

// Block: `tok` tokens of the chunk (their cosines and sines computed once in
// shared memory, for all heads), threads over (token, head, unit).
template <bool BF16, bool INTER>
__global__ void __launch_bounds__(256, kRopeBlocks) rope_fwd_kernel(const __grid_constant__ RopeArgs2 a,
                                                       const __grid_constant__ RopeTable t, int tok) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) float2 cs[];
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * tok;
  const int nt = static_cast<int>(a.n_tokens - t0 < tok ? a.n_tokens - t0 : tok);
  for (int i = threadIdx.x; i < nt * t.pairs; i += blockDim.x) {
    const int r = i / t.pairs, m = i - r * t.pairs;
    cs[a.vec ? r * t.pairs + cs_place<BF16, INTER>(m, t.pairs) : i] = rope_cs(a.pos[t0 + r], t.turns[m], t.mscale);
  }
  __syncthreads();
  constexpr int ES = BF16 ? 2 : 4;
  const int items = nt * a.n_heads * static_cast<int>(a.units.d);
  if (a.vec) {
    for (int i = threadIdx.x; i < items; i += 256) {
      const int rh = a.units.div(i), u = i - rh * static_cast<int>(a.units.d);
      const int r = a.heads.div(rh), h = rh - r * a.n_heads;
      const Unit w = rope_unit<BF16, INTER>(
          static_cast<const uint8_t*>(a.x.p) + ((t0 + r) * a.x.row + h * a.x.head) * ES, u, t.pairs);
      if (w.first < 0 && a.in_place) continue;
      uint4 x, x1;
      load_unit<BF16, INTER>(w, t.pairs, x, x1);
      store_unit<BF16, INTER>(w, t.pairs, x, x1, static_cast<uint8_t*>(a.y) + ((t0 + r) * a.y_row + h * a.y_head) * ES,
                              cs + r * t.pairs);
    }
  } else {   // element by element: unit = one pair, or one copied element
    for (int i = threadIdx.x; i < items; i += blockDim.x) {
      const int rh = a.units.div(i), u = i - rh * static_cast<int>(a.units.d);
      const int r = a.heads.div(rh), h = rh - r * a.n_heads;
      const int64_t xs = (t0 + r) * a.x.row + h * a.x.head, ys = (t0 + r) * a.y_row + h * a.y_head;
      if (u >= t.pairs) {
        if (!a.in_place) st1<BF16>(a.y, ys + t.pairs + u, ld1<BF16>(a.x.p, xs + t.pairs + u));
        continue;
      }
      const int e0 = INTER ? 2 * u : u, e1 = INTER ? 2 * u + 1 : u + t.pairs;
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
template <bool BF16, bool INTER>
__global__ void __launch_bounds__(256, kAppendBlocks) paged_append_kernel(const __grid_constant__ AppendArgs a,
                                                           const __grid_constant__ RopeTable t, int tok) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ __align__(16) float2 cs[];
  __shared__ int64_t s_row[kMaxTok];   // row of K/V head 0, or -1
  const int s = blockIdx.y;
  const SeqSpan sp = seq_span(a.c, a.ch, s);
  const int t0 = blockIdx.x * tok;
  const int nt = min(sp.n - t0, tok);
  if (nt <= 0) return;
  if (sp.over && threadIdx.x == 0) report_bad_cache(a.status, s);
  constexpr int ES = BF16 ? 2 : 4;
  const int row_bytes = a.head_dim * ES, cu_log2 = 31 - __clz(row_bytes / 16), ps = a.c.page.d;   // head_dim 64 or 128
  const int Hk = a.c.n_heads, Hq = a.n_q_heads, ru = a.units.d;
  const int64_t g0 = sp.row0 + t0;
  const int nrot = (Hq + Hk) * ru, items = nt * static_cast<int>(a.per.d);
  // Item i: its unit, token and head (q, k, v in turn).  A thread's next item is read while it works on one, the first
  // one under the page look-up and the angles.
  struct Item {
    Unit w;
    int r, h;
  };
  auto item = [&](int i) {
    Item it;
    it.r = a.per.div(i);
    const int x = i - it.r * static_cast<int>(a.per.d);
    if (x < nrot) {
      it.h = a.units.div(x);
      const uint8_t* src =
          it.h < Hq ? static_cast<const uint8_t*>(a.q.p) + ((g0 + it.r) * a.q.row + it.h * a.q.head) * ES
                    : static_cast<const uint8_t*>(a.k.p) + ((g0 + it.r) * a.k.row + (it.h - Hq) * a.k.head) * ES;
      it.w = rope_unit<BF16, INTER>(src, x - it.h * ru, t.pairs);
    } else {
      const int h = (x - nrot) >> cu_log2, o = ((x - nrot) - (h << cu_log2)) * 16;
      it.h = Hq + Hk + h;
      it.w = {static_cast<const uint8_t*>(a.v.p) + ((g0 + it.r) * a.v.row + h * a.v.head) * ES + o, -1, o};
    }
    return it;
  };
  Item next = {};
  uint4 n0, n1;
  if (static_cast<int>(threadIdx.x) < items) {
    next = item(threadIdx.x);
    load_unit<BF16, INTER>(next.w, t.pairs, n0, n1);
  }
  if (t.pairs > 0) {
    const int64_t pos0 = a.pos[s] + t0;
    for (int i = threadIdx.x; i < nt * t.pairs; i += blockDim.x) {
      const int r = i / t.pairs, m = i - r * t.pairs;
      cs[r * t.pairs + cs_place<BF16, INTER>(m, t.pairs)] = rope_cs(pos0 + r, t.turns[m], t.mscale);
    }
  }
  if (threadIdx.x < nt) {
    const int j = sp.old + t0 + static_cast<int>(threadIdx.x);
    const int64_t row = j < sp.kv ? slot_row(a.c, s, 0, j) : -1;
    if (row < 0) report_bad_cache(a.status, s);
    s_row[threadIdx.x] = row;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < items; i += 256) {
    const Item it = next;
    const uint4 x = n0, x1 = n1;
    if (i + 256 < items) {
      next = item(i + 256);
      load_unit<BF16, INTER>(next.w, t.pairs, n0, n1);
    }
    uint8_t* dst;
    if (it.h < Hq) {
      dst = static_cast<uint8_t*>(a.q_out) + ((g0 + it.r) * a.qo_row + it.h * a.qo_head) * ES;
    } else {
      const int64_t to = s_row[it.r];
      if (to < 0) continue;
      const bool is_v = it.h >= Hq + Hk;
      const int64_t row = to + static_cast<int64_t>(it.h - Hq - (is_v ? Hk : 0)) * ps;
      dst = static_cast<uint8_t*>(is_v ? a.v_pool : a.k_pool) + row * row_bytes;
      if (is_v && a.acc != nullptr && it.w.at == 0) a.acc[row] = 0.f;
    }
    store_unit<BF16, INTER>(it.w, t.pairs, x, x1, dst, cs + it.r * t.pairs);
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

// Cluster of C CTAs per (head, sequence, layer): the bar (the (m - r)-th
// largest key among the first n = L - r slots) by a radix selection of 8-bit
// digits, from keys read once into shared memory (when they fit), then the
// kept slots in slot order, with the bar's equals taken from the lowest slot.
// Each CTA owns a run of slots and each of its warps a run of those; the CTAs
// read one another's digit counts through distributed shared memory and all
// come to the same bar (4 sequences of 32768 slots, 8 heads: 49 us with one
// CTA each).  The histogram has kSelCopies copies, one per lane modulo
// kSelCopies, because weights crowd into few bins; the selection stops as soon
// as a whole bin is wanted.
constexpr int kSelCopies = 8;

// The same shared-memory word of the cluster's CTA `rank`.
__device__ __forceinline__ int ld_cluster(const int* p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(map_to_cta(smem_addr(p), rank)) : "memory");
  return v;
}

template <int T, int C>
__global__ void __cluster_dims__(C, 1, 1) __launch_bounds__(T)
evict_select_kernel(const __grid_constant__ EvictArgs a, int max_keys) {
  pdl_wait();
  pdl_trigger();
  extern __shared__ uint32_t keys[];                 // max_keys, of this CTA's run
  __shared__ int hist[kSelCopies][257];
  __shared__ int counts[2][256];                     // of this CTA: read by the others, in alternate passes
  __shared__ int s_digit, s_rest, s_whole;
  __shared__ int wsum[2][32], s_cta[2];
  const int h = blockIdx.x / C, c = blockIdx.x % C, s = blockIdx.y, l = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  auto cluster_sync = [&] {
    if constexpr (C > 1) cluster_sync_all(); else __syncthreads();
  };
  bool bad;
  const int L = static_cast<int>(evict_len(a, s, &bad));
  if (bad && tid == 0) report_bad_cache(a.status, s);
  const int m = static_cast<int>(a.keep < L ? a.keep : L);
  const int r = static_cast<int>(a.recent < m ? a.recent : m);
  const int n = L - r, want = m - r;
  int32_t* out = a.kept + ((static_cast<int64_t>(l) * a.src.n_seqs + s) * a.src.n_heads + h) * a.kept_stride;
  for (int i = c * T + tid; i < r; i += C * T) out[want + i] = n + i;
  if (want == n) {   // none has to go
    for (int i = c * T + tid; i < n; i += C * T) out[i] = i;
    return;
  }
  if (want <= 0) return;   // the same in all CTAs of the cluster
  const float* acc = a.acc + l * a.src_layer_rows;
  const int run = (n + C * T - 1) / (C * T) * 32;    // slots of a warp
  const int c0 = min(c * (T / 32) * run, n), c1 = min(c0 + (T / 32) * run, n);
  const bool fits = c1 - c0 <= max_keys;
  auto from_pool = [&](int j) -> uint32_t {
    const int row = slot_row(a.src, s, h, j);
    return row < 0 ? 0u : weight_key(acc[row]);
  };
  if (fits) {
#pragma unroll 4
    for (int j = c0 + tid; j < c1; j += T) keys[j - c0] = from_pool(j);
  }
  auto key_at = [&](int j) { return fits ? keys[j - c0] : from_pool(j); };
  uint32_t bar = 0, mask = 0;
  int rest = want;   // how many of the keys that match bar's known digits are wanted
  for (int shift = 24; shift >= 0; shift -= 8) {
    int* mine = counts[(shift >> 3) & 1];
    for (int i = tid; i < kSelCopies * 257; i += T) hist[0][i] = 0;
    __syncthreads();   // also: the keys are there
    for (int j = c0 + tid; j < c1; j += T) {
      const uint32_t key = key_at(j);
      if ((key & mask) == bar) atomicAdd(&hist[lane % kSelCopies][(key >> shift) & 255u], 1);
    }
    __syncthreads();
    int own = 0;
    if (tid < 256) {
#pragma unroll
      for (int k = 0; k < kSelCopies; ++k) own += hist[k][tid];
      mine[tid] = own;
    }
    cluster_sync();
    // Counts of the bins above: a suffix sum over the 256 bins, in 8 warps.
    int all = own, incl = 0;
    if (tid < 256) {
#pragma unroll
      for (int k = 1; k < C; ++k) all += ld_cluster(mine + tid, (c + k) % C);
      incl = all;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int y = __shfl_down_sync(0xffffffffu, incl, off);
        if (lane + off < 32) incl += y;
      }
      if (lane == 0) wsum[0][warp] = incl;
    }
    __syncthreads();
    if (tid < 256) {
      for (int w = warp + 1; w < 8; ++w) incl += wsum[0][w];
      if (incl >= rest && incl - all < rest) {
        s_digit = tid;
        s_rest = rest - (incl - all);
        s_whole = s_rest == all;
      }
    }
    __syncthreads();
    bar |= static_cast<uint32_t>(s_digit) << shift;
    mask |= 255u << shift;
    rest = s_rest;
    if (s_whole) break;
  }
  // Keys above the bar are kept, and the first `rest` of its equals (in the
  // digits looked at).  Each warp counts them in its run, then writes them
  // behind those of the warps before it.
  const int j0 = min(c0 + warp * run, n), j1 = min(j0 + run, n);
  int more = 0, same = 0;
  for (int j = j0 + lane; j < j1; j += 32) {
    const uint32_t key = key_at(j) & mask;
    more += key > bar;
    same += key == bar;
  }
  more = __reduce_add_sync(0xffffffffu, more);
  same = __reduce_add_sync(0xffffffffu, same);
  __syncthreads();
  if (lane == 0) {
    wsum[0][warp] = more;
    wsum[1][warp] = same;
  }
  __syncthreads();
  const int of = lane < T / 32 ? wsum[0][lane] : 0, os = lane < T / 32 ? wsum[1][lane] : 0;
  more = __reduce_add_sync(0xffffffffu, lane < warp ? of : 0);
  same = __reduce_add_sync(0xffffffffu, lane < warp ? os : 0);
  if constexpr (C > 1) {
    if (warp == 0) {
      const int tf = __reduce_add_sync(0xffffffffu, of), ts = __reduce_add_sync(0xffffffffu, os);
      if (lane == 0) {
        s_cta[0] = tf;
        s_cta[1] = ts;
      }
    }
    cluster_sync();
    more += __reduce_add_sync(0xffffffffu, lane < c ? ld_cluster(&s_cta[0], lane < c ? lane : 0) : 0);
    same += __reduce_add_sync(0xffffffffu, lane < c ? ld_cluster(&s_cta[1], lane < c ? lane : 0) : 0);
  }
  int at = more + min(same, rest);   // `same`: equals before this warp
  for (int j = j0; j < j1; j += 32) {
    const uint32_t key = j + lane < j1 ? key_at(j + lane) & mask : 0u;
    const bool eq = j + lane < j1 && key == bar;
    const uint32_t be = __ballot_sync(0xffffffffu, eq);
    const uint32_t below = (1u << lane) - 1u;
    const bool take = j + lane < j1 && (key > bar || (eq && same + __popc(be & below) < rest));
    const uint32_t bt = __ballot_sync(0xffffffffu, take);
    if (take) out[at + __popc(bt & below)] = j + lane;
    at += __popc(bt);
    same += __popc(be);
  }
  if constexpr (C > 1) cluster_sync_all();   // no CTA leaves while another may read its counts
}

// The kept rows move to the front in slot order: CTA per (layer, head, slice,
// block of rows, sequence).  The K and V rows of a slot are one row of 2 *
// row_bytes / 16 chunks, cut into `slices`; a block holds kMoveChunks chunks,
// so that a thread has kMoveDeep 16-byte loads in flight.  To pages of its own
// every block is a CTA.  In place a row's new slot is never above its old one,
// so a CTA that walks all blocks in order, reading a block before it writes it,
// never overwrites a row it still has to read (slices are independent).
constexpr int kMoveThreads = 256;
constexpr int kMoveDeep = 4;   // 2: 64 sequences of 1000 slots to 750 in 204 instead of 160 us, 8: no gain
constexpr int kMoveChunks = kMoveThreads * kMoveDeep;
constexpr int kMoveMaxRows = 256;   // of a block: slices of at least 4 chunks

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictArgs a, int slices_log2,
                                                                  int blocks) {
  pdl_wait();
  pdl_trigger();
  __shared__ int s_from[kMoveMaxRows], s_to[kMoveMaxRows];   // pool rows, or -1
  int id = blockIdx.x;
  const int blk = id % blocks;
  id /= blocks;
  const int slice = id & ((1 << slices_log2) - 1);
  id >>= slices_log2;
  const int h = id % a.src.n_heads, l = id / a.src.n_heads, s = blockIdx.y;
  const int tid = threadIdx.x;
  const bool in_place = a.k == a.dk;
  // In place another CTA may have stored the new length m already: min(keep, m) is m again.
  const int64_t dcap = static_cast<int64_t>(a.dst.max_pages) * a.dst.page.d;
  bool bad;
  const int64_t L = evict_len(a, s, &bad);
  const int m = static_cast<int>(a.keep < L ? a.keep : L);
  // The thread's chunk of a row is the same in all of its rows: tid >> cols_log2 and every row_step-th behind it.
  const int all_log2 = 31 - __clz(2 * a.row_bytes / 16), cols_log2 = all_log2 - slices_log2;
  const int rows = kMoveChunks >> cols_log2, row_step = kMoveThreads >> cols_log2, r0 = tid >> cols_log2;
  const int c = (slice << cols_log2) + (tid & ((1 << cols_log2) - 1));
  const bool is_v = (c >> (all_log2 - 1)) != 0;
  const int64_t off = (c - (is_v ? 1 << (all_log2 - 1) : 0)) * 16;
  const uint8_t* src = (is_v ? a.v : a.k) + l * a.src_layer_rows * a.row_bytes + off;
  uint8_t* dst = (is_v ? a.dv : a.dk) + l * a.dst_layer_rows * a.row_bytes + off;
  const int32_t* kept = a.kept + ((static_cast<int64_t>(l) * a.src.n_seqs + s) * a.src.n_heads + h) * a.kept_stride;
  for (int i0 = blk * rows; i0 < m; i0 += blocks * rows) {
    const int nr = min(rows, m - i0);
    float w = 0.f;
    int from = -1, to = -1;
    if (tid < nr) {
      const int i = i0 + tid;
      from = slot_row(a.src, s, h, kept[i]);
      to = i < dcap ? slot_row(a.dst, s, h, i) : -1;
      if (from < 0 || to < 0) report_bad_cache(a.status, s);
      if (in_place && from == to) to = -1;
      if (slice == 0 && from >= 0 && to >= 0) w = a.acc[l * a.src_layer_rows + from];
      s_from[tid] = from;
      s_to[tid] = to;
    }
    __syncthreads();
    uint4 x[kMoveDeep];
    int at[kMoveDeep];
#pragma unroll
    for (int d = 0; d < kMoveDeep; ++d) {
      const int r = r0 + d * row_step;
      x[d] = make_uint4(0u, 0u, 0u, 0u);
      at[d] = r < nr ? s_to[r] : -1;
      if (at[d] < 0 || s_from[r] < 0) continue;
      x[d] = *reinterpret_cast<const uint4*>(src + static_cast<int64_t>(s_from[r]) * a.row_bytes);
    }
    if (in_place) __syncthreads();
    if (slice == 0 && to >= 0) a.dacc[l * a.dst_layer_rows + to] = w;
#pragma unroll
    for (int d = 0; d < kMoveDeep; ++d)
      if (at[d] >= 0) *reinterpret_cast<uint4*>(dst + static_cast<int64_t>(at[d]) * a.row_bytes) = x[d];
    if (blocks * rows < m - i0) __syncthreads();   // s_from and s_to are rewritten
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (a.dst_pos != a.src_pos) a.dst_pos[s] = a.src_pos[s];
    a.dst_lens[s] = m < dcap ? m : dcap;
  }
}

template <bool BF16>
cudaError_t launch_rope_t(cudaStream_t stream, const RopeArgs2& a, const RopeTable& t, int tok) {
  const dim3 grid(static_cast<unsigned>((a.n_tokens + tok - 1) / tok));
  const size_t smem = static_cast<size_t>(tok) * t.pairs * sizeof(float2);
  return t.interleaved ? launch_kernel(rope_fwd_kernel<BF16, true>, grid, dim3(256), smem, stream, a, t, tok)
                       : launch_kernel(rope_fwd_kernel<BF16, false>, grid, dim3(256), smem, stream, a, t, tok);
}

template <bool BF16>
cudaError_t launch_append_t(cudaStream_t stream, const AppendArgs& a, const RopeTable& t, int tok) {
  const dim3 grid(static_cast<unsigned>((a.ch.max_q + tok - 1) / tok), static_cast<unsigned>(a.c.n_seqs));
  const size_t smem = static_cast<size_t>(tok) * t.pairs * sizeof(float2);
  return t.interleaved ? launch_kernel(paged_append_kernel<BF16, true>, grid, dim3(256), smem, stream, a, t, tok)
                       : launch_kernel(paged_append_kernel<BF16, false>, grid, dim3(256), smem, stream, a, t, tok);
}

// Tokens per block: about 32 KB of rows, to spread the angles and the page
// lookups over (16 KB: append of 12000 rows 3% slower, 64 KB as well); one
// token when that would leave SMs without a block.
int tokens_per_block(int64_t row_bytes, int64_t tokens) {
  int64_t tok = (32768 + row_bytes - 1) / row_bytes;
  tok = tok < 1 ? 1 : tok > kMaxTok ? kMaxTok : tok;
  return tokens < tok * 148 ? 1 : static_cast<int>(tok);
}

}  // namespace

cudaError_t launch_rope_rows(cudaStream_t stream, const RopeArgs2& in, const RopeTable& t) {
  RopeArgs2 a = in;
  const int es = a.bf16 ? 2 : 4;
  const int v = 16 / es, pairs = t.pairs, D = a.head_dim;
  a.heads = FastDiv::make(static_cast<uint32_t>(a.n_heads));
  a.units = FastDiv::make(static_cast<uint32_t>(a.vec ? (t.interleaved ? D : D - pairs) / v : D - pairs));
  const int tok = tokens_per_block(static_cast<int64_t>(a.n_heads) * D * es, a.n_tokens);
  return a.bf16 ? launch_rope_t<true>(stream, a, t, tok) : launch_rope_t<false>(stream, a, t, tok);
}

cudaError_t launch_paged_append(cudaStream_t stream, const AppendArgs& in, const RopeTable& t) {
  AppendArgs a = in;
  const int es = a.bf16 ? 2 : 4;
  const int v = 16 / es, D = a.head_dim;
  const int ru = (t.interleaved ? D : D - t.pairs) / v;
  a.units = FastDiv::make(static_cast<uint32_t>(ru));
  a.per = FastDiv::make(static_cast<uint32_t>((a.n_q_heads + a.c.n_heads) * ru + a.c.n_heads * (D / v)));
  const int tok = tokens_per_block(static_cast<int64_t>(a.n_q_heads + 2 * a.c.n_heads) * D * es,
                                   static_cast<int64_t>(a.ch.max_q) * a.c.n_seqs);
  return a.bf16 ? launch_append_t<true>(stream, a, t, tok) : launch_append_t<false>(stream, a, t, tok);
}

cudaError_t launch_paged_advance(cudaStream_t stream, const PagedView& c, const ChunkArgs& ch, int64_t* lens,
                                 int64_t* pos, DevStatus* status) {
  return launch_kernel(paged_advance_kernel, dim3((c.n_seqs + 127) / 128), dim3(128), 0, stream, c, ch, lens, pos,
                       status);
}

cudaError_t launch_paged_evict(const Launch& L, const EvictArgs& a) {
  const int64_t S = a.src.n_seqs, H = a.src.n_heads, nl = a.n_layers;
  // Few slots: 256 threads a CTA, of which several share an SM.  Many slots
  // and few (head, sequence, layer): 8 CTAs for each.  Keys in shared memory:
  // all that the tables can hold, up to 48 K.
  const int64_t cap = static_cast<int64_t>(a.src.max_pages) * a.src.page.d;
  const bool wide = cap > 8192 && H * S * nl < L.sm_count;
  const int64_t own = wide ? (cap + 8191) / 8192 * 1024 : cap;   // slots of a CTA
  const int max_keys = static_cast<int>(own < 49152 ? own : 49152);
  const dim3 sel(static_cast<unsigned>(wide ? H * 8 : H), static_cast<unsigned>(S), static_cast<unsigned>(nl));
  // launch_kernel raises a kernel's limit from 48 KB of dynamic shared memory on; the static arrays need room below it.
  size_t smem = static_cast<size_t>(max_keys) * 4;
  if (smem > 32 * 1024 && smem <= 48 * 1024) smem = 48 * 1024 + 16;
  cudaError_t e =
      wide          ? launch_kernel(evict_select_kernel<1024, 8>, sel, dim3(1024), smem, L.stream, a, max_keys)
      : cap <= 4096 ? launch_kernel(evict_select_kernel<256, 1>, sel, dim3(256), smem, L.stream, a, max_keys)
                    : launch_kernel(evict_select_kernel<1024, 1>, sel, dim3(1024), smem, L.stream, a, max_keys);
  if (e != cudaSuccess) return e;
  // To other pages: whole rows, every block a CTA.  In place: one CTA walks a
  // slice's blocks, so slices (of at least 64 bytes) are cut until there are
  // about four CTAs for each SM.
  const int all = 2 * a.row_bytes / 16;
  int slices_log2 = 0;
  int64_t blocks = 1;
  if (a.k == a.dk) {
    while (all >> slices_log2 > 4 && (nl * H * S << slices_log2) < 4 * L.sm_count) ++slices_log2;
  } else {
    const int rows = kMoveChunks / all;
    blocks = (a.keep + rows - 1) / rows;
    const int64_t most = (1ll << 30) / (nl * H);   // the grid's x dimension
    blocks = blocks < 1 ? 1 : blocks > most ? most : blocks;
  }
  return launch_kernel(evict_move_kernel, dim3(static_cast<unsigned>((nl * H << slices_log2) * blocks), static_cast<unsigned>(S)),
                       dim3(kMoveThreads), 0, L.stream, a, slices_log2, static_cast<int>(blocks));
}

}  // namespace vx
