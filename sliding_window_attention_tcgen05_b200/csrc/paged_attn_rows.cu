// paged_attn_rows.cu -- attention over the paged cache for few query rows
// (decoding, streaming steps), its fp32 form, the joining of split key ranges
// and the accumulated attention weights.
#include <type_traits>

#include "paged_attn.cuh"

namespace vx {

namespace {

// paged_attn_rows_kernel: CTA per (key range, K/V head, sequence), four warps.
// The up to 16 * MT query rows (token t, head g of the group: row t * G + g)
// are the M side of mma.sync tiles, so one read of a K/V row serves the whole
// group; tcgen05's M >= 64 tiles would be mostly padding.  With up to 8 rows
// (HALF) the tile's lower half is left out of the softmax.  Each warp walks its
// own tiles of KT keys through its own two cp.async stages (no CTA barrier in
// the loop; three CTAs an SM are worth more than a third stage), with the page
// of every row looked up one tile ahead; O is rescaled only when a row's
// maximum grows by more than 2^8; the four warps' softmax states, and those of
// up to 8 CTAs of a sequence (a cluster), are joined through shared memory at
// the end.  Weights are rounded to bf16 for the product with V (mma.sync takes
// both operands as bf16), as in the tcgen05 kernel; their sum is of the
// unrounded ones.
constexpr int kRowsThreads = 128;
constexpr int kRowsStages = 2;
constexpr int kRowsStageBytes = 8192;   // K and V of one warp tile
constexpr float kRowsSlack = 8.0f;

__device__ __forceinline__ float2 ld_cluster2(uint32_t addr, int rank) {   // 8 bytes of the cluster's CTA `rank`
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(map_to_cta(addr, rank)) : "memory");
  return v;
}

template <int D, int MT, bool HALF, bool MOD>
__global__ void __launch_bounds__(kRowsThreads)
paged_attn_rows_kernel(const __grid_constant__ PagedAttnArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int KT = kRowsStageBytes / (4 * D);   // 16 keys (D 128) or 32 (D 64)
  constexpr int NB = KT / 8;                      // 8-key blocks of a tile
  constexpr int NH = HALF ? 1 : 2;                // 8-row halves of a 16-row tile in use
  constexpr int CPR = D / 8;                      // 16-byte chunks of a row
  constexpr int RPI = 32 / CPR;                   // rows per warp-wide copy
  constexpr int ROWS = HALF ? 8 : 16 * MT;
  extern __shared__ __align__(128) uint8_t smem[];
  const int sp = blockIdx.x, kh = blockIdx.y, s = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SeqSpan q = seq_span(a.c, a.ch, s);
  if (q.n <= 0) return;
  if (q.over && threadIdx.x == 0) report_bad_cache(a.status, s);
  const int G = a.group, rows = q.n * G;
  const KeyList kl = key_list(q.old, q.old + q.n - 1, a.window, a.prefix ? a.prefix[s] : 0, q.kv);
  const int step = ((kl.total + a.splits - 1) / a.splits + KT - 1) / KT * KT;
  const int x0 = min(sp * step, kl.total), x1 = min(x0 + step, kl.total);
  const int tiles = (x1 - x0 + KT - 1) / KT;
  const int mine = tiles > warp ? (tiles - warp + 3) / 4 : 0;

  const uint32_t stage_addr = smem_addr(smem) + warp * kRowsStages * kRowsStageBytes;
  const int cc = lane % CPR, rl0 = lane / CPR;
  const uint8_t* kp = static_cast<const uint8_t*>(a.k) + cc * 16;
  const uint8_t* vp = static_cast<const uint8_t*>(a.v) + cc * 16;

  auto lookup = [&](int i) -> int {   // this lane's row of the warp's tile i, or -1
    const int x = x0 + (warp + 4 * i) * KT + (lane & (KT - 1));
    if (i >= mine || x >= x1) return -1;
    const int r = slot_row(a.c, s, kh, key_slot(kl, x));
    if (r < 0) report_bad_cache(a.status, s);
    return r;
  };
  auto issue = [&](int i, int row) {
    if (i < mine) {
      const uint32_t dst = stage_addr + (i % kRowsStages) * kRowsStageBytes + rl0 * (2 * D);
      int gr[KT / RPI];
#pragma unroll
      for (int it = 0; it < KT / RPI; ++it) gr[it] = __shfl_sync(0xffffffffu, row, it * RPI + rl0);
#pragma unroll
      for (int it = 0; it < KT / RPI; ++it) {
        const int64_t off = static_cast<int64_t>(max(gr[it], 0)) * (2 * D);
        const uint32_t d = dst + it * RPI * (2 * D) + ((cc ^ ((it * RPI + rl0) & 7)) << 4);
        cp_async16(d, kp + off, gr[it] >= 0);
        cp_async16(d + kRowsStageBytes / 2, vp + off, gr[it] >= 0);
      }
    }
    cp_async_commit();
  };
  issue(0, lookup(0));
  int next_row = lookup(1);

  // Query fragments (A operand) and each row's place: rows lane / 4 and + 8 of every 16-row tile.
  const int qr = lane >> 2, qc = (lane & 3) * 2;
  uint32_t qa[MT][D / 16][4];
  int xlo[MT][NH], xhi[MT][NH], qi[MT][NH];
  float slope2[MT][NH];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (half >= NH) {
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) qa[mt][ks][1] = qa[mt][ks][3] = 0u;
        continue;
      }
      const int r = mt * 16 + half * 8 + qr;
      const bool ok = r < rows;
      const int t = a.group_div.div(ok ? r : 0), g = (ok ? r : 0) - t * G;
      const int i = q.old + t;
      qi[mt][half] = i;
      xlo[mt][half] = max(0, i - a.window + 1 - kl.shift);
      xhi[mt][half] = i - kl.shift;
      slope2[mt][half] = MOD && a.slopes ? a.slopes[kh * G + g] * kLog2e : 0.f;
      const uint16_t* src = static_cast<const uint16_t*>(a.q.p) + (q.row0 + t) * a.q.row + (kh * G + g) * a.q.head;
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks) {
        qa[mt][ks][half] = ok ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + qc) : 0u;
        qa[mt][ks][half + 2] = ok ? *reinterpret_cast<const uint32_t*>(src + ks * 16 + 8 + qc) : 0u;
      }
    }
  const ScoreMod sm = score_mod(a);
  const float sc = MOD ? 1.f : sm.sl2;
  const int pre = min(kl.pre, x1);
  // Tiles inside [all_lo, all_hi] or below pre need no mask.
  const int all_lo = max(0, q.old + q.n - 1 - a.window + 1 - kl.shift), all_hi = min(q.old - kl.shift, x1 - 1);
  // Scores kept for the sum of the weights: this lane's row of them.
  float* kept = nullptr;
  if (HALF && a.scores != nullptr && qr < rows)
    kept = a.scores + ((static_cast<int64_t>(s) * a.c.n_heads + kh) * (a.ch.max_q * G) + qr) * a.score_stride;

  float o[MT][D / 8][4];
  float m_run[MT][NH], l_part[MT][NH];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
    for (int half = 0; half < NH; ++half) {
      m_run[mt][half] = -INFINITY;
      l_part[mt][half] = 0.f;
    }
#pragma unroll
    for (int nb = 0; nb < D / 8; ++nb) o[mt][nb][0] = o[mt][nb][1] = o[mt][nb][2] = o[mt][nb][3] = 0.f;
  }

  for (int i = 0; i < mine; ++i) {
    cp_async_wait<0>();
    __syncwarp();
    issue(i + 1, next_row);   // into the stage read in the last turn
    next_row = lookup(i + 2);
    const uint32_t kb = stage_addr + (i % kRowsStages) * kRowsStageBytes, vb = kb + kRowsStageBytes / 2;
    const int xb = x0 + (warp + 4 * i) * KT;
    float sa[MT][NB][4];
#pragma unroll
    for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) sa[mt][nb][0] = sa[mt][nb][1] = sa[mt][nb][2] = sa[mt][nb][3] = 0.f;
      const int kr = nb * 8 + (lane & 7);
#pragma unroll
      for (int h = 0; h < D / 32; ++h) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4(kb + kr * (2 * D) + (((h * 4 + (lane >> 3)) ^ (kr & 7)) << 4), b0, b1, b2, b3);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma_bf16_16816(sa[mt][nb], qa[mt][2 * h][0], qa[mt][2 * h][1], qa[mt][2 * h][2], qa[mt][2 * h][3], b0, b1);
          mma_bf16_16816(sa[mt][nb], qa[mt][2 * h + 1][0], qa[mt][2 * h + 1][1], qa[mt][2 * h + 1][2],
                         qa[mt][2 * h + 1][3], b2, b3);
        }
      }
    }
    const bool clean = (xb >= all_lo && xb + KT - 1 <= all_hi) || xb + KT - 1 < pre;
    uint32_t pa[MT][KT / 16][4];
    bool grew = false;
    float alpha[MT][NH];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        if (half >= NH) {
#pragma unroll
          for (int k = 0; k < KT / 16; ++k) pa[mt][k][1] = pa[mt][k][3] = 0u;
          continue;
        }
        float y[2 * NB];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
          y[2 * nb] = sa[mt][nb][2 * half];
          y[2 * nb + 1] = sa[mt][nb][2 * half + 1];
        }
        if constexpr (MOD) {
          scale_scores(sm, y);
          if (sm.bias)
#pragma unroll
            for (int e = 0; e < 2 * NB; ++e) {
              const int j = key_slot(kl, xb + (e >> 1) * 8 + qc + (e & 1));
              y[e] -= slope2[mt][half] * static_cast<float>(abs(qi[mt][half] - j));
            }
        }
        if (!clean) {
#pragma unroll
          for (int e = 0; e < 2 * NB; ++e) {
            const int x = xb + (e >> 1) * 8 + qc + (e & 1);
            y[e] = (x < pre || (x >= xlo[mt][half] && x <= xhi[mt][half] && x < x1)) ? y[e] : -INFINITY;
          }
        }
        if (HALF && kept != nullptr) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            const int x = xb + nb * 8 + qc;
            if (x < a.score_stride) *reinterpret_cast<float2*>(kept + x) = make_float2(y[2 * nb] * sc, y[2 * nb + 1] * sc);
          }
        }
        float cmax = fmaxf(y[0], y[1]);
#pragma unroll
        for (int e = 2; e < 2 * NB; e += 2) cmax = fmaxf(cmax, fmaxf(y[e], y[e + 1]));
        cmax = fmaxf(cmax, __shfl_xor_sync(0xffffffffu, cmax, 1));
        cmax = fmaxf(cmax, __shfl_xor_sync(0xffffffffu, cmax, 2)) * sc;
        alpha[mt][half] = 1.f;
        if (cmax > m_run[mt][half] + kRowsSlack) {
          alpha[mt][half] = ex2_approx(m_run[mt][half] - cmax);   // 0 for the first keys
          m_run[mt][half] = cmax;
          grew = true;
        }
        const float mu = m_run[mt][half] == -INFINITY ? 0.f : m_run[mt][half];
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 2 * NB; ++e) {
          y[e] = ex2_approx(fmaf(y[e], sc, -mu));
          sum += y[e];
        }
        l_part[mt][half] = l_part[mt][half] * alpha[mt][half] + sum;
#pragma unroll
        for (int k = 0; k < KT / 16; ++k) {
          pa[mt][k][half] = pack_bf16x2(y[4 * k], y[4 * k + 1]);
          pa[mt][k][half + 2] = pack_bf16x2(y[4 * k + 2], y[4 * k + 3]);
        }
      }
    if (__any_sync(0xffffffffu, grew)) {   // alpha is 1 for every row otherwise
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nb = 0; nb < D / 8; ++nb) {
          o[mt][nb][0] *= alpha[mt][0];
          o[mt][nb][1] *= alpha[mt][0];
          o[mt][nb][2] *= alpha[mt][NH - 1];
          o[mt][nb][3] *= alpha[mt][NH - 1];
        }
    }
#pragma unroll
    for (int k = 0; k < KT / 16; ++k) {
      const int vr = k * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
      for (int dc = 0; dc < D / 8; dc += 2) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(vb + vr * (2 * D) + (((dc + (lane >> 4)) ^ (vr & 7)) << 4), b0, b1, b2, b3);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          mma_bf16_16816(o[mt][dc], pa[mt][k][0], pa[mt][k][1], pa[mt][k][2], pa[mt][k][3], b0, b1);
          mma_bf16_16816(o[mt][dc + 1], pa[mt][k][0], pa[mt][k][1], pa[mt][k][2], pa[mt][k][3], b2, b3);
        }
      }
    }
  }
  cp_async_wait<0>();

  // Join the four warps (the stages are free once all of them are here), then
  // the CTAs of the cluster, each taking its share of the elements.
  float* sm_m = reinterpret_cast<float*>(smem);          // [4][ROWS]
  float* sm_l = sm_m + 4 * ROWS;                         // [4][ROWS]
  float2* sm_ml = reinterpret_cast<float2*>(sm_l + 4 * ROWS);   // [ROWS]: of the CTA
  float* sm_o = reinterpret_cast<float*>(sm_ml + ROWS);  // [4][ROWS][D], the CTA's own in [0]
  __syncthreads();
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int half = 0; half < NH; ++half) {
      float l = l_part[mt][half];
      l += __shfl_xor_sync(0xffffffffu, l, 1);
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      const int r = mt * 16 + half * 8 + qr;
      if (r < rows) {
        if ((lane & 3) == 0) {
          sm_m[warp * ROWS + r] = m_run[mt][half];
          sm_l[warp * ROWS + r] = l;
        }
#pragma unroll
        for (int nb = 0; nb < D / 8; ++nb)
          *reinterpret_cast<float2*>(sm_o + (warp * ROWS + r) * D + nb * 8 + qc) =
              make_float2(o[mt][nb][2 * half], o[mt][nb][2 * half + 1]);
      }
    }
  __syncthreads();
  auto store = [&](int r, int d, float M, float l, float y0, float y1) {
    const int t = a.group_div.div(r), h = kh * G + r - t * G;
    const int64_t tok = q.row0 + t;
    if (a.parts > 1) {
      const int64_t pr = (static_cast<int64_t>(sp / a.cluster) * a.ch.n_tokens + tok) * a.n_q_heads + h;
      if (l != 0.f) *reinterpret_cast<float2*>(a.part_o + pr * D + d) = make_float2(y0, y1);
      if (d == 0) a.part_ml[pr] = make_float2(M, l);
    } else {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      *reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.o) + tok * a.o_row + h * a.o_head + d) =
          pack_bf16x2(y0 * inv, y1 * inv);
      if (d == 0 && a.lse) a.lse[tok * a.n_q_heads + h] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
    }
  };
  for (int idx = threadIdx.x; idx < rows * (D / 2); idx += kRowsThreads) {
    const int r = idx / (D / 2), d = (idx % (D / 2)) * 2;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, sm_m[w * ROWS + r]);
    float l = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (sm_l[w * ROWS + r] == 0.f) continue;   // the warp saw no key (a NaN score leaves a NaN sum)
      const float f = ex2_approx(sm_m[w * ROWS + r] - M);
      const float2 y = *reinterpret_cast<const float2*>(sm_o + (w * ROWS + r) * D + d);
      l = fmaf(sm_l[w * ROWS + r], f, l);
      y0 = fmaf(y.x, f, y0);
      y1 = fmaf(y.y, f, y1);
    }
    if (a.cluster == 1) {
      store(r, d, M, l, y0, y1);
    } else {
      *reinterpret_cast<float2*>(sm_o + r * D + d) = make_float2(y0, y1);   // only this thread reads [.][r][d]
      if (d == 0) sm_ml[r] = make_float2(M, l);
    }
  }
  if (a.cluster == 1) return;
  cluster_sync_all();
  const int rank = sp % a.cluster;
  for (int idx = rank * kRowsThreads + threadIdx.x; idx < rows * (D / 2); idx += a.cluster * kRowsThreads) {
    const int r = idx / (D / 2), d = (idx % (D / 2)) * 2;
    const uint32_t ml_at = smem_addr(sm_ml + r), y_at = smem_addr(sm_o + r * D + d);
    float2 ml[8], y[8];
    float M = -INFINITY;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      ml[c] = make_float2(-INFINITY, 0.f);
      if (c < a.cluster) {
        ml[c] = ld_cluster2(ml_at, c);
        y[c] = ld_cluster2(y_at, c);
        M = fmaxf(M, ml[c].x);
      }
    }
    float l = 0.f, y0 = 0.f, y1 = 0.f;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (ml[c].y == 0.f) continue;
      const float f = ex2_approx(ml[c].x - M);
      l = fmaf(ml[c].y, f, l);
      y0 = fmaf(y[c].x, f, y0);
      y1 = fmaf(y[c].y, f, y1);
    }
    store(r, d, M, l, y0, y1);
  }
  cluster_sync_all();   // no CTA leaves while another may read its results
}

// ------------------------------------------------------------------- fp32 --
// paged_attn_f32_kernel: CTA per (block of 16 * RM rows x key range, K/V head,
// sequence), CUDA cores throughout (tensor-core tf32 would keep 10 mantissa
// bits).  256 threads as 16 x 16: a thread computes RM rows x 4 keys of a
// 64-key tile's scores and RM rows x D / 16 dims of the output, so that shared
// memory is read once for 8 (RM 4) or 5 multiply-adds; the V tile travels
// while the scores are computed and the next K tile while P V is.
constexpr int kF32Threads = 256;
constexpr int kF32Keys = 64;

template <int D, int RM>
struct F32Cfg {
  static constexpr int kRows = 16 * RM;
  static constexpr int kPitch = D + 4;          // of Q and K rows: neighbouring rows 16 bytes apart modulo the banks
  static constexpr int kPPitch = kF32Keys + 4;
  static constexpr size_t kSmem =
      (static_cast<size_t>(kRows + kF32Keys) * kPitch + kF32Keys * D + kRows * kPPitch) * 4 + 2 * kF32Keys * 4;
};

// Pool rows of the tile at list position xt (thread = key), -1 where there is none.
__device__ __forceinline__ int f32_row(const PagedAttnArgs& a, const KeyList& kl, int s, int kh, int x, int x1) {
  if (x >= x1) return -1;
  const int r = slot_row(a.c, s, kh, key_slot(kl, x));
  if (r < 0) report_bad_cache(a.status, s);
  return r;
}
// A tile's rows (PITCH floats apart in shared memory) by cp.async; the caller commits.
template <int D, int PITCH>
__device__ __forceinline__ void f32_tile(uint32_t dst, const float* pool, const int* rows) {
  for (int i = threadIdx.x; i < kF32Keys * (D / 4); i += kF32Threads) {
    const int r = i / (D / 4), c = i % (D / 4), gr = rows[r];
    cp_async16(dst + (r * PITCH + c * 4) * 4, pool + static_cast<int64_t>(max(gr, 0)) * D + c * 4, gr >= 0);
  }
}

template <int D, int RM>
__global__ void __launch_bounds__(kF32Threads) paged_attn_f32_kernel(const __grid_constant__ PagedAttnArgs a, int blocks) {
  pdl_wait();
  pdl_trigger();
  using Cfg = F32Cfg<D, RM>;
  constexpr int R = Cfg::kRows, KP = Cfg::kPitch, PP = Cfg::kPPitch, DV = D / 64;
  extern __shared__ __align__(16) float fsm[];
  float* sq = fsm;                       // [R][KP]
  float* sk = sq + R * KP;               // [64][KP]
  float* sv = sk + kF32Keys * KP;        // [64][D]
  float* spr = sv + kF32Keys * D;        // [R][PP]
  int* s_row = reinterpret_cast<int*>(spr + R * PP);   // [2][64]
  const int rb = blockIdx.x % blocks, sp = blockIdx.x / blocks, kh = blockIdx.y, s = blockIdx.z;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const SeqSpan q = seq_span(a.c, a.ch, s);
  const int G = a.group, rows = q.n * G, r0 = rb * R;
  if (r0 >= rows) return;
  if (q.over && tid == 0) report_bad_cache(a.status, s);
  const int rn = min(R, rows - r0);
  const int tf = a.group_div.div(r0), tl = a.group_div.div(r0 + rn - 1);
  const KeyList kl = key_list(q.old + tf, q.old + tl, a.window, a.prefix ? a.prefix[s] : 0, q.kv);
  const int step = ((kl.total + a.splits - 1) / a.splits + kF32Keys - 1) / kF32Keys * kF32Keys;
  const int x0 = min(sp * step, kl.total), x1 = min(x0 + step, kl.total);
  const int tiles = (x1 - x0 + kF32Keys - 1) / kF32Keys;
  const float* kp = static_cast<const float*>(a.k);
  const float* vp = static_cast<const float*>(a.v);
  if (tid < kF32Keys) s_row[tid] = f32_row(a, kl, s, kh, x0 + tid, x1);
  for (int i = tid; i < R * (D / 4); i += kF32Threads) {
    const int r = i / (D / 4), c = i % (D / 4);
    const bool ok = r < rn;
    const int t = a.group_div.div(r0 + (ok ? r : 0)), h = kh * G + r0 + (ok ? r : 0) - t * G;
    cp_async16(smem_addr(sq + r * KP + c * 4),
               static_cast<const float*>(a.q.p) + (q.row0 + t) * a.q.row + h * a.q.head + c * 4, ok);
  }
  __syncthreads();
  if (tiles > 0) f32_tile<D, KP>(smem_addr(sk), kp, s_row);
  cp_async_commit();
  const ScoreMod sm = score_mod(a);
  int qi[RM];
  float slope2[RM], m[RM], l[RM], o[RM][4 * DV];
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int r = min(r0 + ty * RM + i, rows - 1);
    const int t = a.group_div.div(r);
    qi[i] = q.old + t;
    slope2[i] = a.slopes ? a.slopes[kh * G + r - t * G] * kLog2e : 0.f;
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int e = 0; e < 4 * DV; ++e) o[i][e] = 0.f;
  }
  for (int u = 0; u < tiles; ++u) {
    const int xt = x0 + u * kF32Keys;
    int* row = s_row + (u & 1) * kF32Keys;
    cp_async_wait<0>();
    __syncthreads();                     // K (and Q) of this tile have landed, V's buffer is free
    f32_tile<D, D>(smem_addr(sv), vp, row);
    cp_async_commit();
    if (tid < kF32Keys && u + 1 < tiles) s_row[((u + 1) & 1) * kF32Keys + tid] = f32_row(a, kl, s, kh, xt + kF32Keys + tid, x1);
    float sc[RM][4];
#pragma unroll
    for (int i = 0; i < RM; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll 4
    for (int d = 0; d < D; d += 4) {
      float4 kk[4], qq[RM];
#pragma unroll
      for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * KP + d);
#pragma unroll
      for (int i = 0; i < RM; ++i) qq[i] = *reinterpret_cast<const float4*>(sq + (ty * RM + i) * KP + d);
#pragma unroll
      for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          sc[i][j] = fmaf(qq[i].x, kk[j].x, sc[i][j]);
          sc[i][j] = fmaf(qq[i].y, kk[j].y, sc[i][j]);
          sc[i][j] = fmaf(qq[i].z, kk[j].z, sc[i][j]);
          sc[i][j] = fmaf(qq[i].w, kk[j].w, sc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
      float cmax = -INFINITY;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int x = xt + tx + 16 * j, js = key_slot(kl, x);
        const bool seen = x < x1 && (js < kl.pre || (js <= qi[i] && js > qi[i] - a.window));
        sc[i][j] = seen ? score2(sm, sc[i][j], slope2[i], qi[i] - js) : -INFINITY;
        cmax = fmaxf(cmax, sc[i][j]);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) cmax = fmaxf(cmax, __shfl_xor_sync(0xffffffffu, cmax, off));
      const float m_new = fmaxf(m[i], cmax);
      const float mu = m_new == -INFINITY ? 0.f : m_new;
      const float alpha = exp2f(m[i] - mu);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float p = exp2f(sc[i][j] - mu);
        spr[(ty * RM + i) * PP + tx + 16 * j] = p;
        sum += p;
      }
      m[i] = m_new;
      l[i] = l[i] * alpha + sum;         // of this thread's keys
#pragma unroll
      for (int e = 0; e < 4 * DV; ++e) o[i][e] *= alpha;
    }
    cp_async_wait<0>();
    __syncthreads();                     // V has landed, P is written, K's buffer is free
    if (u + 1 < tiles) f32_tile<D, KP>(smem_addr(sk), kp, s_row + ((u + 1) & 1) * kF32Keys);
    cp_async_commit();
#pragma unroll 2
    for (int key = 0; key < kF32Keys; key += 4) {
      float4 p[RM];
#pragma unroll
      for (int i = 0; i < RM; ++i) p[i] = *reinterpret_cast<const float4*>(spr + (ty * RM + i) * PP + key);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk)
#pragma unroll
        for (int e = 0; e < DV; ++e) {
          const float4 v = *reinterpret_cast<const float4*>(sv + (key + kk) * D + tx * 4 + 64 * e);
#pragma unroll
          for (int i = 0; i < RM; ++i) {
            const float pk = kk == 0 ? p[i].x : kk == 1 ? p[i].y : kk == 2 ? p[i].z : p[i].w;
            o[i][4 * e] = fmaf(pk, v.x, o[i][4 * e]);
            o[i][4 * e + 1] = fmaf(pk, v.y, o[i][4 * e + 1]);
            o[i][4 * e + 2] = fmaf(pk, v.z, o[i][4 * e + 2]);
            o[i][4 * e + 3] = fmaf(pk, v.w, o[i][4 * e + 3]);
          }
        }
    }
  }
  cp_async_wait<0>();
#pragma unroll
  for (int i = 0; i < RM; ++i) {
    const int r = r0 + ty * RM + i;
    float sum = l[i];
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (r >= rows) continue;
    const int t = a.group_div.div(r), h = kh * G + r - t * G;
    const int64_t tok = q.row0 + t;
    float inv = 1.f;
    float* dst;
    if (a.parts > 1) {
      const int64_t pr = (static_cast<int64_t>(sp) * a.ch.n_tokens + tok) * a.n_q_heads + h;
      dst = a.part_o + pr * D;
      if (tx == 0) a.part_ml[pr] = make_float2(m[i], sum);
    } else {
      inv = sum == 0.f ? 0.f : 1.f / sum;
      dst = static_cast<float*>(a.o) + tok * a.o_row + h * a.o_head;
      if (tx == 0 && a.lse) a.lse[tok * a.n_q_heads + h] = sum == 0.f ? -INFINITY : (m[i] + log2f(sum)) * kLn2;
    }
#pragma unroll
    for (int e = 0; e < DV; ++e)
      *reinterpret_cast<float4*>(dst + tx * 4 + 64 * e) =
          make_float4(o[i][4 * e] * inv, o[i][4 * e + 1] * inv, o[i][4 * e + 2] * inv, o[i][4 * e + 3] * inv);
  }
}

// paged_attn_f32_rows_kernel: the fp32 form for few rows.  CTA per (block of 8
// rows x key range, K/V head, sequence), four warps.  D / 8 lanes share a key
// (8 dims each), which holds the 8 rows' queries and outputs of its dims in
// registers.  Each lane copies its own piece of K and V through a ring of
// cp.async stages in shared memory, several steps ahead.  The dot products' partial sums are added by an
// exchange that leaves row r's score in lane r of the key's lanes.
constexpr int kF32RowBlock = 8;
constexpr int kF32RowStages = 3;
constexpr int kF32RowDeep = 2;   // keys of a lane's step: two chains of shuffles and exponentials in flight
constexpr size_t kF32RowSmem = 128 * kF32RowStages * kF32RowDeep * 64;   // a lane's 64 bytes of a key

template <int D>
__global__ void __launch_bounds__(128) paged_attn_f32_rows_kernel(const __grid_constant__ PagedAttnArgs a, int blocks) {
  pdl_wait();
  pdl_trigger();
  constexpr int R = kF32RowBlock, LPK = D / 8, KPW = 32 / LPK;   // lanes of a key, keys of a warp's step
  constexpr int U = kF32RowDeep, WARP = U * KPW, STEP = 4 * WARP;   // keys of a warp's step and of the CTA's
  extern __shared__ __align__(16) float fsm[];
  float(*sm_m)[R] = reinterpret_cast<float(*)[R]>(fsm);                 // [4][R]: these once the ring is done
  float(*sm_l)[R] = sm_m + 4;                                           // [4][R]
  float(*sm_o)[R][D] = reinterpret_cast<float(*)[R][D]>(fsm + 8 * R);   // [4][R][D]
  const int rb = blockIdx.x % blocks, sp = blockIdx.x / blocks, kh = blockIdx.y, s = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane / LPK, e = lane % LPK, rl = lane & 7;
  const SeqSpan q = seq_span(a.c, a.ch, s);
  const int G = a.group, rows = q.n * G, r0 = rb * R;
  if (r0 >= rows) return;
  if (q.over && threadIdx.x == 0) report_bad_cache(a.status, s);
  const int rn = min(R, rows - r0);
  const int tf = a.group_div.div(r0), tl = a.group_div.div(r0 + rn - 1);
  const KeyList kl = key_list(q.old + tf, q.old + tl, a.window, a.prefix ? a.prefix[s] : 0, q.kv);
  const int step = ((kl.total + a.splits - 1) / a.splits + STEP - 1) / STEP * STEP;
  const int x0 = min(sp * step, kl.total), x1 = min(x0 + step, kl.total);
  const int steps = (x1 - x0 + STEP - 1) / STEP;
  const float* kp = static_cast<const float*>(a.k) + e * 4;
  const float* vp = static_cast<const float*>(a.v) + e * 4;
  auto key_of = [&](int i, int u) { return x0 + i * STEP + warp * WARP + u * KPW + g; };   // this lane's, in the list
  auto lookup = [&](int i, int (&row)[U]) {   // their pool rows, or -1
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = key_of(i, u);
      row[u] = -1;
      if (i >= steps || x >= x1) continue;
      row[u] = slot_row(a.c, s, kh, key_slot(kl, x));
      if (row[u] < 0) report_bad_cache(a.status, s);
    }
  };
  // Of each key, 4 x (32 lanes x 16 bytes): K dims 4 e .., K dims D / 2 + 4 e .., then V's.
  const uint32_t ring = smem_addr(fsm) + warp * (kF32RowStages * U * 2048) + lane * 16;
  auto fetch = [&](int i, const int (&row)[U]) {
    if (i < steps) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const uint32_t dst = ring + (i % kF32RowStages * U + u) * 2048;
        const int64_t at = static_cast<int64_t>(max(row[u], 0)) * D;
        cp_async16(dst, kp + at, row[u] >= 0);
        cp_async16(dst + 512, kp + at + D / 2, row[u] >= 0);
        cp_async16(dst + 1024, vp + at, row[u] >= 0);
        cp_async16(dst + 1536, vp + at + D / 2, row[u] >= 0);
      }
    }
    cp_async_commit();
  };
  int next_row[U];
#pragma unroll
  for (int i = 0; i < kF32RowStages - 1; ++i) {
    lookup(i, next_row);
    fetch(i, next_row);
  }
  lookup(kF32RowStages - 1, next_row);
  float qr[R][8], o[R][8];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int rr = min(r0 + r, rows - 1);
    const int t = a.group_div.div(rr), h = kh * G + rr - t * G;
    const float* src = static_cast<const float*>(a.q.p) + (q.row0 + t) * a.q.row + h * a.q.head + e * 4;
    const float4 x = *reinterpret_cast<const float4*>(src), y = *reinterpret_cast<const float4*>(src + D / 2);
    qr[r][0] = x.x; qr[r][1] = x.y; qr[r][2] = x.z; qr[r][3] = x.w;
    qr[r][4] = y.x; qr[r][5] = y.y; qr[r][6] = y.z; qr[r][7] = y.w;
#pragma unroll
    for (int d = 0; d < 8; ++d) o[r][d] = 0.f;
  }
  // This lane's row of the scores.
  const ScoreMod sm = score_mod(a);
  const int mr = min(r0 + rl, rows - 1), mt = a.group_div.div(mr), mi = q.old + mt;
  const float slope2 = a.slopes ? a.slopes[kh * G + mr - mt * G] * kLog2e : 0.f;
  float* kept = nullptr;
  if (a.scores != nullptr && rl < rn && e < 8)
    kept = a.scores + ((static_cast<int64_t>(s) * a.c.n_heads + kh) * (a.ch.max_q * G) + r0 + rl) * a.score_stride;
  float m = -INFINITY, l = 0.f;
  for (int i = 0; i < steps; ++i) {
    cp_async_wait<kF32RowStages - 2>();
    const float* st = fsm + (warp * kF32RowStages + i % kF32RowStages) * (U * 512) + lane * 4;   // what this lane copied
    float dot[U][R], v[U][8];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float k[8];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        *reinterpret_cast<float4*>(k + 4 * c) = *reinterpret_cast<const float4*>(st + u * 512 + c * 128);
        *reinterpret_cast<float4*>(v[u] + 4 * c) = *reinterpret_cast<const float4*>(st + u * 512 + 256 + c * 128);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        dot[u][r] = 0.f;
#pragma unroll
        for (int d = 0; d < 8; ++d) dot[u][r] = fmaf(qr[r][d], k[d], dot[u][r]);
      }
    }
    fetch(i + kF32RowStages - 1, next_row);   // into the stage of the last step
    lookup(i + kF32RowStages, next_row);
    if constexpr (LPK == 16) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < R; ++r) dot[u][r] += __shfl_xor_sync(0xffffffffu, dot[u][r], 8);
    }
    // Halve the rows and the lanes that share them, three times: lane rl ends with row rl.
#pragma unroll
    for (int w = 4; w > 0; w >>= 1) {
      const bool up = (lane & w) != 0;
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int r = 0; r < w; ++r) {
          const float keep = up ? dot[u][r + w] : dot[u][r], give = up ? dot[u][r] : dot[u][r + w];
          dot[u][r] = keep + __shfl_xor_sync(0xffffffffu, give, w);
        }
    }
    float y[U], cmax = -INFINITY;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int x = key_of(i, u), j = key_slot(kl, x);
      const bool seen = x < x1 && (j < kl.pre || (j <= mi && j > mi - a.window));
      y[u] = seen ? score2(sm, dot[u][0], slope2, mi - j) : -INFINITY;
      if (kept != nullptr && x < a.score_stride) kept[x] = y[u];
      cmax = fmaxf(cmax, y[u]);
    }
#pragma unroll
    for (int off = LPK; off < 32; off <<= 1) cmax = fmaxf(cmax, __shfl_xor_sync(0xffffffffu, cmax, off));
    const bool grew = cmax > m + kRowsSlack;
    float alpha = 1.f;
    if (grew) {
      alpha = exp2f(m - cmax);   // 0 for the first keys
      m = cmax;
    }
    if (__any_sync(0xffffffffu, grew)) {
      l *= alpha;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const float f = __shfl_sync(0xffffffffu, alpha, (lane & -LPK) | r);
#pragma unroll
        for (int d = 0; d < 8; ++d) o[r][d] *= f;
      }
    }
    float p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      p[u] = exp2f(y[u] - (m == -INFINITY ? 0.f : m));
      l += p[u];
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float f = __shfl_sync(0xffffffffu, p[u], (lane & -LPK) | r);
#pragma unroll
        for (int d = 0; d < 8; ++d) o[r][d] = fmaf(f, v[u][d], o[r][d]);
      }
  }
  cp_async_wait<0>();
  __syncthreads();   // the ring becomes the join's
  // Join the warp's keys, then the warps.
#pragma unroll
  for (int off = LPK; off < 32; off <<= 1) {
    l += __shfl_xor_sync(0xffffffffu, l, off);
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int d = 0; d < 8; ++d) o[r][d] += __shfl_xor_sync(0xffffffffu, o[r][d], off);
  }
  if (lane < R) {
    sm_m[warp][lane] = m;
    sm_l[warp][lane] = l;
  }
  if (g == 0) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      *reinterpret_cast<float4*>(&sm_o[warp][r][e * 4]) = make_float4(o[r][0], o[r][1], o[r][2], o[r][3]);
      *reinterpret_cast<float4*>(&sm_o[warp][r][D / 2 + e * 4]) = make_float4(o[r][4], o[r][5], o[r][6], o[r][7]);
    }
  }
  __syncthreads();
  for (int idx = threadIdx.x; idx < rn * (D / 4); idx += 128) {
    const int r = idx / (D / 4), d = idx % (D / 4) * 4;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < 4; ++w) M = fmaxf(M, sm_m[w][r]);
    float L = 0.f;
    float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (sm_l[w][r] == 0.f) continue;   // the warp saw no key (a NaN score leaves a NaN sum)
      const float f = exp2f(sm_m[w][r] - M);
      const float4 z = *reinterpret_cast<const float4*>(&sm_o[w][r][d]);
      L = fmaf(sm_l[w][r], f, L);
      y.x = fmaf(z.x, f, y.x);
      y.y = fmaf(z.y, f, y.y);
      y.z = fmaf(z.z, f, y.z);
      y.w = fmaf(z.w, f, y.w);
    }
    const int t = a.group_div.div(r0 + r), h = kh * G + r0 + r - t * G;
    const int64_t tok = q.row0 + t;
    if (a.parts > 1) {
      const int64_t pr = (static_cast<int64_t>(sp) * a.ch.n_tokens + tok) * a.n_q_heads + h;
      *reinterpret_cast<float4*>(a.part_o + pr * D + d) = y;
      if (d == 0) a.part_ml[pr] = make_float2(M, L);
    } else {
      const float inv = L == 0.f ? 0.f : 1.f / L;
      *reinterpret_cast<float4*>(static_cast<float*>(a.o) + tok * a.o_row + h * a.o_head + d) =
          make_float4(y.x * inv, y.y * inv, y.z * inv, y.w * inv);
      if (d == 0 && a.lse) a.lse[tok * a.n_q_heads + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * kLn2;
    }
  }
}

// ---------------------------------------------------------------- combine --
// W warps per (token, head): the parts' maxima and sums, then the weighted sum
// of their outputs, D / 32 elements per lane, the parts dealt to the warps and
// all of a warp's loads in flight together; the warps' sums are added in order.
constexpr int kCombineThreads = 256;
constexpr int kCombineDeep = 8;   // loads in flight

// The parts' largest maximum M, their factors 2^(m - M) and the sum l of a row,
// by one warp.
struct PartSums {
  float M, l, wt[kMaxSplits / 32];   // wt[i]: of part i * 32 + lane
};
__device__ __forceinline__ PartSums part_sums(const PagedAttnArgs& a, int64_t row) {
  const int64_t rows = static_cast<int64_t>(a.ch.n_tokens) * a.n_q_heads;
  const int lane = threadIdx.x & 31;
  PartSums r;
  r.M = -INFINITY;
  r.l = 0.f;
  float2 ml[kMaxSplits / 32];
#pragma unroll
  for (int i = 0; i < kMaxSplits / 32; ++i) {
    const int sp = i * 32 + lane;
    ml[i] = sp < a.parts ? a.part_ml[sp * rows + row] : make_float2(-INFINITY, 0.f);
    r.M = fmaxf(r.M, ml[i].x);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) r.M = fmaxf(r.M, __shfl_xor_sync(0xffffffffu, r.M, off));
#pragma unroll
  for (int i = 0; i < kMaxSplits / 32; ++i) {
    r.wt[i] = ml[i].y == 0.f ? 0.f : exp2f(ml[i].x - r.M);
    r.l += ml[i].y * r.wt[i];
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) r.l += __shfl_xor_sync(0xffffffffu, r.l, off);
  return r;
}

// The row of this thread's W warps; part: shared memory of all 8 warps.  Every thread of the block calls it.
template <int D, bool BF16, int W>
__device__ __forceinline__ void combine_row(const PagedAttnArgs& a, int64_t row, bool mine, float (*part)[D]) {
  constexpr int V = D / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, w = warp % W;
  const int64_t rows = static_cast<int64_t>(a.ch.n_tokens) * a.n_q_heads;
  const int64_t tok = row / a.n_q_heads;
  const int h = static_cast<int>(row - tok * a.n_q_heads);
  float M = -INFINITY, l = 0.f, y[V];
#pragma unroll
  for (int e = 0; e < V; ++e) y[e] = 0.f;
  if (mine) {
    const PartSums ps = part_sums(a, row);
    M = ps.M;
    l = ps.l;
    const float(&wt)[kMaxSplits / 32] = ps.wt;
#pragma unroll
    for (int i = 0; i < kMaxSplits / 32; ++i)
      for (int j0 = w; j0 < 32 && i * 32 + j0 < a.parts; j0 += W * kCombineDeep) {
        float x[kCombineDeep][V], ws[kCombineDeep];
#pragma unroll
        for (int k = 0; k < kCombineDeep; ++k) {
          const int j = j0 + k * W, sp = i * 32 + j;
          ws[k] = __shfl_sync(0xffffffffu, wt[i], j & 31);
          if (j >= 32 || sp >= a.parts) ws[k] = 0.f;
          const float* src = a.part_o + (sp * rows + row) * D + lane * V;
#pragma unroll
          for (int e = 0; e < V; ++e) x[k][e] = ws[k] == 0.f ? 0.f : src[e];   // an empty part wrote no output
        }
#pragma unroll
        for (int k = 0; k < kCombineDeep; ++k)
#pragma unroll
          for (int e = 0; e < V; ++e) y[e] = fmaf(x[k][e], ws[k], y[e]);
      }
  }
  if constexpr (W > 1) {
#pragma unroll
    for (int e = 0; e < V; ++e) part[warp][lane * V + e] = y[e];
    __syncthreads();
    if (w > 0) return;
#pragma unroll
    for (int k = 1; k < W; ++k)
#pragma unroll
      for (int e = 0; e < V; ++e) y[e] += part[warp + k][lane * V + e];
  }
  if (!mine) return;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  if constexpr (BF16) {
    uint16_t* dst = static_cast<uint16_t*>(a.o) + tok * a.o_row + h * a.o_head + lane * V;
#pragma unroll
    for (int e = 0; e < V; e += 2) *reinterpret_cast<uint32_t*>(dst + e) = pack_bf16x2(y[e] * inv, y[e + 1] * inv);
  } else {
    float* dst = static_cast<float*>(a.o) + tok * a.o_row + h * a.o_head + lane * V;
#pragma unroll
    for (int e = 0; e < V; ++e) dst[e] = y[e] * inv;
  }
  if (lane == 0 && a.lse) a.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * kLn2;
}

template <int D, bool BF16, int W>
__global__ void __launch_bounds__(kCombineThreads) paged_attn_combine_kernel(const __grid_constant__ PagedAttnArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int WARPS = kCombineThreads / 32;
  __shared__ float part[WARPS][D];
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (WARPS / W) + (threadIdx.x >> 5) / W;
  const int64_t tok = row / a.n_q_heads;
  bool mine = row < static_cast<int64_t>(a.ch.n_tokens) * a.n_q_heads;
  if (mine) {
    // Rows outside every sequence (or past max_q) have no parts: find the row's sequence.
    int lo = 0, hi = a.c.n_seqs;   // last s with q_start[s] <= tok
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (a.ch.q_start[mid] <= tok) lo = mid; else hi = mid;
    }
    const SeqSpan q = seq_span(a.c, a.ch, lo);
    mine = tok >= q.row0 && tok < q.row0 + q.n;
  }
  combine_row<D, BF16, W>(a, row, mine, part);
}

// ---------------------------------------------------------------- weights --
// Accumulated weights: acc_j = decay * acc_j + sum over the chunk's rows of
// exp(s - lse).  The keys are the M side (32 a warp, whose K fragments stay in
// registers), the rows stream past in blocks of 64, so every slot's sum stays in
// one thread group's registers: no atomics, a fixed order.  With 16 keys a warp
// each Q fragment read fed one product (4 chunks of 1000 tokens over 3000, 32/8
// heads of 128: 299 us, shared memory and mma pipe both under half busy).  CTA
// per (128 slots x segment
// of their row blocks, K/V head, sequence): early slots are seen by all rows
// and late ones by few, and cutting the rows into segments evens that out (8
// ragged chunks of 1500 tokens, 12 heads: 465 us without segments).  Segments'
// sums go to the workspace and are added up by paged_attn_weights_sum_kernel.
// Slots from part_stride on (a caller's max_kv that was too low) are left to
// the first segment, which then takes all their rows.
constexpr int kWKeys = 128;
constexpr int kWRows = 64;

// acc of slot j's row: decay * acc + x.
__device__ __forceinline__ void add_weight(const PagedAttnArgs& a, int64_t row, float x) {
  if (row >= 0) a.acc[row] = (a.acc_decay != 0.f ? a.acc_decay * a.acc[row] : 0.f) + x;
}
__device__ __forceinline__ float* weight_part(const PagedAttnArgs& a, int seg, int s, int kh) {
  return a.part_w + ((static_cast<int64_t>(seg) * a.c.n_seqs + s) * a.c.n_heads + kh) * a.part_stride;
}

template <int D, bool MOD>
__global__ void __launch_bounds__(128, D == 128 ? 4 : 5) paged_attn_weights_kernel(const __grid_constant__ PagedAttnArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int CPR = D / 8;
  static_assert(kWKeys == 2 * kWRows, "the K tile passes through the Q blocks' buffers");
  extern __shared__ __align__(128) uint8_t smem[];   // two Q blocks of 64 rows (before them the K tile), their places
  const uint32_t sq0 = smem_addr(smem);
  float* s_lse = reinterpret_cast<float*>(smem + 2 * kWRows * 2 * D);             // [2][64]
  float* s_sl = s_lse + 2 * kWRows;                                               // [2][64]
  int* s_i = reinterpret_cast<int*>(s_sl + 2 * kWRows);                           // [2][64]: i - first slot of the tile
  const int kh = blockIdx.y, s = blockIdx.z;
  const int seg = blockIdx.x % a.w_segs, tile0 = blockIdx.x / a.w_segs, tiles = gridDim.x / a.w_segs;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const SeqSpan q = seq_span(a.c, a.ch, s);
  if (q.n <= 0) return;
  const int G = a.group;
  const int pre = min(a.prefix ? max(a.prefix[s], 0) : 0, q.kv);
  const ScoreMod sm = score_mod(a);
  const uint16_t* kp = static_cast<const uint16_t*>(a.k);
  const uint16_t* qp = static_cast<const uint16_t*>(a.q.p);
  for (int tile = tile0; tile * kWKeys < q.kv; tile += tiles) {
    const int j0 = tile * kWKeys, j1 = min(j0 + kWKeys, q.kv);
    const bool cut = a.w_segs > 1 && j1 <= a.part_stride;
    if (!cut && seg > 0) continue;
    // Tokens that see some slot of the tile.
    int t0 = max(0, j0 - q.old);
    int t1 = min(q.n, j1 - 1 - q.old + min(a.window, kNoWindow - 1 - j1));
    if (j0 < pre) { t0 = 0; t1 = q.n; }
    int ra = t0 * G, rz = max(t1 * G, ra);
    if (cut) {
      const int64_t all = (rz - ra + kWRows - 1) / kWRows;
      const int b0 = static_cast<int>(all * seg / a.w_segs), b1 = static_cast<int>(all * (seg + 1) / a.w_segs);
      rz = min(rz, ra + b1 * kWRows);
      ra += b0 * kWRows;
    }
    auto stage_q = [&](int blk, int buf) {
      const int rbase = ra + blk * kWRows;
      for (int i = tid; i < kWRows * CPR; i += 128) {
        const int r = i / CPR, c = i % CPR;
        const bool ok = rbase + r < rz;
        const int t = a.group_div.div(ok ? rbase + r : 0), h = kh * G + (ok ? rbase + r : 0) - t * G;
        cp_async16(sq0 + buf * kWRows * 2 * D + r * 2 * D + ((c ^ (r & 7)) << 4),
                   qp + (q.row0 + t) * a.q.row + h * a.q.head + c * 8, ok);
      }
      if (tid < kWRows) {
        const bool ok = rbase + tid < rz;
        const int t = a.group_div.div(ok ? rbase + tid : 0), h = kh * G + (ok ? rbase + tid : 0) - t * G;
        const float z = ok ? a.lse[static_cast<int64_t>(q.row0 + t) * a.n_q_heads + h] : -INFINITY;
        s_lse[buf * kWRows + tid] = z == -INFINITY ? INFINITY : z * kLog2e;   // weight 0 without a sum
        s_i[buf * kWRows + tid] = q.old + t - j0;
        s_sl[buf * kWRows + tid] = MOD && a.slopes ? a.slopes[h] * kLog2e : 0.f;
      }
      cp_async_commit();
    };
    const int blocks = (rz - ra + kWRows - 1) / kWRows;
    uint32_t ka[2][D / 16][4];   // this warp's 2 x 16 keys as A fragments
    if (blocks > 0) {
      for (int i = tid; i < kWKeys * CPR; i += 128) {
        const int r = i / CPR, c = i % CPR;
        const int gr = j0 + r < j1 ? slot_row(a.c, s, kh, j0 + r) : -1;
        cp_async16(sq0 + r * 2 * D + ((c ^ (r & 7)) << 4), kp + static_cast<int64_t>(max(gr, 0)) * D + c * 8, gr >= 0);
      }
      cp_async_commit();
      cp_async_wait<0>();
      __syncthreads();
#pragma unroll
      for (int mk = 0; mk < 2; ++mk) {   // ldmatrix x4 = rows 0-7 / 8-15 at dims 0-7 / 8-15
        const int r = warp * 32 + mk * 16 + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks)
          ldsm_x4(sq0 + r * 2 * D + (((ks * 2 + (lane >> 4)) ^ (r & 7)) << 4), ka[mk][ks][0], ka[mk][ks][1],
                  ka[mk][ks][2], ka[mk][ks][3]);
      }
      __syncthreads();
      stage_q(0, 0);
    }
    int jr[2][2];   // this thread's keys, from j0
#pragma unroll
    for (int mk = 0; mk < 2; ++mk)
#pragma unroll
      for (int half = 0; half < 2; ++half) jr[mk][half] = warp * 32 + mk * 16 + half * 8 + (lane >> 2);
    const int pr = pre - j0;
    float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};
    for (int blk = 0; blk < blocks; ++blk) {
      const int buf = blk & 1;
      cp_async_wait<0>();
      __syncthreads();
      if (blk + 1 < blocks) stage_q(blk + 1, buf ^ 1);
      const uint32_t sq = sq0 + buf * kWRows * 2 * D;
      // Whether all rows of the block see all keys of the tile.
      const int r_first = ra + blk * kWRows, r_last = min(r_first + kWRows, rz) - 1;
      const int i_first = q.old + static_cast<int>(a.group_div.div(r_first)) - j0;
      const int i_last = q.old + static_cast<int>(a.group_div.div(r_last)) - j0;
      const bool clean = (i_first >= kWKeys - 1 && i_last - a.window < 0) || pr >= kWKeys;
      auto rows8 = [&](int nb, auto masked) {
        float c[2][4] = {};   // of each 16 keys: jr[0] (0, 1) and jr[1] (2, 3), rows col, col + 1
        const int r = nb * 8 + (lane & 7);
#pragma unroll
        for (int h = 0; h < D / 32; ++h) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4(sq + r * 2 * D + (((h * 4 + (lane >> 3)) ^ (r & 7)) << 4), b0, b1, b2, b3);
#pragma unroll
          for (int mk = 0; mk < 2; ++mk) {
            mma_bf16_16816(c[mk], ka[mk][2 * h][0], ka[mk][2 * h][1], ka[mk][2 * h][2], ka[mk][2 * h][3], b0, b1);
            mma_bf16_16816(c[mk], ka[mk][2 * h + 1][0], ka[mk][2 * h + 1][1], ka[mk][2 * h + 1][2], ka[mk][2 * h + 1][3],
                           b2, b3);
          }
        }
        const int col = buf * kWRows + nb * 8 + (lane & 3) * 2;
        const float2 z = *reinterpret_cast<const float2*>(s_lse + col);
        const int2 i = *reinterpret_cast<const int2*>(s_i + col);
        if constexpr (MOD) scale_scores(sm, reinterpret_cast<float(&)[8]>(c));
#pragma unroll
        for (int mk = 0; mk < 2; ++mk) {
          if constexpr (MOD) {
            if (sm.bias) {
              const float2 sl = *reinterpret_cast<const float2*>(s_sl + col);
              const float i0 = static_cast<float>(i.x), i1 = static_cast<float>(i.y);
              const float ja = static_cast<float>(jr[mk][0]), jb = ja + 8.f;
              c[mk][0] = fmaf(-sl.x, fabsf(i0 - ja), c[mk][0]);
              c[mk][1] = fmaf(-sl.y, fabsf(i1 - ja), c[mk][1]);
              c[mk][2] = fmaf(-sl.x, fabsf(i0 - jb), c[mk][2]);
              c[mk][3] = fmaf(-sl.y, fabsf(i1 - jb), c[mk][3]);
            }
          }
          const float sc = MOD ? 1.f : sm.sl2;
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float p0 = ex2_approx(fmaf(c[mk][2 * half], sc, -z.x)), p1 = ex2_approx(fmaf(c[mk][2 * half + 1], sc, -z.y));
            if constexpr (decltype(masked)::value) {
              const int j = jr[mk][half];
              p0 = (j < pr || (j <= i.x && j > i.x - a.window)) ? p0 : 0.f;
              p1 = (j < pr || (j <= i.y && j > i.y - a.window)) ? p1 : 0.f;
            }
            sum[mk][half] += p0 + p1;
          }
        }
      };
      if (clean) {
#pragma unroll 2
        for (int nb = 0; nb < kWRows / 8; ++nb) rows8(nb, std::false_type{});
      } else {
#pragma unroll 2
        for (int nb = 0; nb < kWRows / 8; ++nb) rows8(nb, std::true_type{});
      }
    }
#pragma unroll
    for (int mk = 0; mk < 2; ++mk)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        float x = sum[mk][half];
        x += __shfl_xor_sync(0xffffffffu, x, 1);
        x += __shfl_xor_sync(0xffffffffu, x, 2);
        const int j = j0 + jr[mk][half];
        if ((lane & 3) == 0 && j < j1) {
          if (cut) weight_part(a, seg, s, kh)[j] = x;
          else add_weight(a, slot_row(a.c, s, kh, j), x);
        }
      }
    __syncthreads();   // the tile's buffers are refilled
  }
}

// The same sum from the scores that the rows kernels kept (base 2, by list
// position; up to 8 rows, so that writing and reading them costs less than
// reading K again).  A thread per slot.  Where the keys were split, the grid has
// a block more for each row, which joins the row's parts, and the others take
// the rows' log-sum-exps from the parts themselves: one launch for both.
template <int D, bool BF16>
__global__ void __launch_bounds__(kCombineThreads)
paged_attn_weights_kept_kernel(const __grid_constant__ PagedAttnArgs a, int blocks) {
  pdl_wait();
  pdl_trigger();
  __shared__ float s_lse[8];
  __shared__ int s_i[8];   // slots of the rows' tokens
  __shared__ float part[kCombineThreads / 32][D];
  const int kh = blockIdx.y, s = blockIdx.z;
  const SeqSpan q = seq_span(a.c, a.ch, s);
  if (q.n <= 0) return;
  const int G = a.group, rows = q.n * G, cap = a.ch.max_q * G;
  auto row_of = [&](int r) -> int64_t {
    const int t = a.group_div.div(r);
    return static_cast<int64_t>(q.row0 + t) * a.n_q_heads + kh * G + r - t * G;
  };
  if (static_cast<int>(blockIdx.x) >= blocks) {
    const int r = static_cast<int>(blockIdx.x) - blocks;
    if (r < rows) combine_row<D, BF16, kCombineThreads / 32>(a, row_of(r), true, part);
    return;
  }
  const int warp = threadIdx.x >> 5;
  if (warp < rows) {   // base 2; +inf (weight 0) without a sum
    float z;
    if (a.parts > 1) {
      const PartSums ps = part_sums(a, row_of(warp));
      z = ps.l == 0.f ? INFINITY : ps.M + log2f(ps.l);
    } else {
      z = a.lse[row_of(warp)];
      z = z == -INFINITY ? INFINITY : z * kLog2e;
    }
    s_lse[warp] = z;
    s_i[warp] = q.old + a.group_div.div(warp);
  }
  __syncthreads();
  const KeyList kl = key_list(q.old, q.old + q.n - 1, a.window, a.prefix ? a.prefix[s] : 0, q.kv);
  const float* kept = a.scores + (static_cast<int64_t>(s) * a.c.n_heads + kh) * cap * a.score_stride;
  auto weight = [](float y) { return BF16 ? ex2_approx(y) : exp2f(y); };
  for (int j = blockIdx.x * kCombineThreads + threadIdx.x; j < q.kv; j += blocks * kCombineThreads) {
    const int x = j < kl.cut ? j : j - kl.shift;
    const int row = slot_row(a.c, s, kh, j);
    float sum = 0.f;
    if (x >= (j < kl.cut ? 0 : kl.cut) && x < kl.total) {
      if (x < a.score_stride) {
        for (int r = 0; r < rows; ++r) {
          const float w = weight(kept[r * a.score_stride + x] - s_lse[r]);
          const int i = s_i[r];
          sum += j < kl.pre || (j <= i && j > i - a.window) ? w : 0.f;   // a row whose sum is NaN gives none to what it does not see
        }
      } else if (row >= 0) {   // the caller's max_kv was too low: the product again
        const ScoreMod sm = score_mod(a);
        for (int r = 0; r < rows; ++r) {
          const int t = a.group_div.div(r), h = kh * G + r - t * G, i = q.old + t;
          if (!(j < kl.pre || (j <= i && j > i - a.window))) continue;
          const int64_t qe = (q.row0 + t) * a.q.row + h * a.q.head, ke = static_cast<int64_t>(row) * D;
          float dot = 0.f;
          for (int d = 0; d < D; ++d)
            dot = BF16 ? fmaf(bf16_to_f(static_cast<const uint16_t*>(a.q.p)[qe + d]),
                              bf16_to_f(static_cast<const uint16_t*>(a.k)[ke + d]), dot)
                       : fmaf(static_cast<const float*>(a.q.p)[qe + d], static_cast<const float*>(a.k)[ke + d], dot);
          sum += weight(score2(sm, dot, a.slopes ? a.slopes[h] * kLog2e : 0.f, i - j) - s_lse[r]);
        }
      }
    }
    add_weight(a, row, sum);
  }
}

// Adds up the segments' sums.
__global__ void __launch_bounds__(128) paged_attn_weights_sum_kernel(const __grid_constant__ PagedAttnArgs a, int keys) {
  pdl_wait();
  pdl_trigger();
  const int kh = blockIdx.y, s = blockIdx.z;
  const SeqSpan q = seq_span(a.c, a.ch, s);
  if (q.n <= 0) return;
  const int j = static_cast<int>(blockIdx.x) * 128 + threadIdx.x;
  const int tile_end = min((j / keys + 1) * keys, q.kv);   // as the segments saw it
  if (j >= q.kv || tile_end > a.part_stride) return;
  float x = 0.f;
  for (int seg = 0; seg < a.w_segs; ++seg) x += weight_part(a, seg, s, kh)[j];
  add_weight(a, slot_row(a.c, s, kh, j), x);
}

// fp32: CTA per 64 slots (and segment of their rows), 256 threads as 16 x 16,
// four rows x four slots each, the rows past in double-buffered blocks of 64.
constexpr int kWKeysF32 = kF32Keys;

template <int D>
__global__ void __launch_bounds__(kF32Threads) paged_attn_weights_f32_kernel(const __grid_constant__ PagedAttnArgs a) {
  pdl_wait();
  pdl_trigger();
  constexpr int KP = D + 4;
  extern __shared__ __align__(16) float fsm[];
  float* sk = fsm;                                        // [64][KP]
  float* sq = sk + kWKeysF32 * KP;                        // [2][64][KP]
  float* part = sq;                                       // [16][64], after the last block
  float* s_lse = sq + 2 * kWRows * KP;                    // [2][64]
  float* s_sl = s_lse + 2 * kWRows;                       // [2][64]
  int* s_i = reinterpret_cast<int*>(s_sl + 2 * kWRows);   // [2][64]
  const int kh = blockIdx.y, s = blockIdx.z;
  const int seg = blockIdx.x % a.w_segs, tile0 = blockIdx.x / a.w_segs, tiles = gridDim.x / a.w_segs;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const SeqSpan q = seq_span(a.c, a.ch, s);
  if (q.n <= 0) return;
  const int G = a.group;
  const int pre = min(a.prefix ? max(a.prefix[s], 0) : 0, q.kv);
  const ScoreMod sm = score_mod(a);
  for (int tile = tile0; tile * kWKeysF32 < q.kv; tile += tiles) {
    const int j0 = tile * kWKeysF32, j1 = min(j0 + kWKeysF32, q.kv);
    const bool cut = a.w_segs > 1 && j1 <= a.part_stride;
    if (!cut && seg > 0) continue;
    // Tokens that see some slot of the tile.
    int t0 = max(0, j0 - q.old), t1 = min(q.n, j1 - 1 - q.old + min(a.window, kNoWindow - 1 - j1));
    if (j0 < pre) { t0 = 0; t1 = q.n; }
    int ra = t0 * G, rz = max(t1 * G, ra);
    if (cut) {
      const int64_t all = (rz - ra + kWRows - 1) / kWRows;
      const int b0 = static_cast<int>(all * seg / a.w_segs), b1 = static_cast<int>(all * (seg + 1) / a.w_segs);
      rz = min(rz, ra + b1 * kWRows);
      ra += b0 * kWRows;
    }
    const int blocks = (rz - ra + kWRows - 1) / kWRows;
    auto stage_q = [&](int blk, int buf) {
      const int rbase = ra + blk * kWRows;
      for (int i = tid; i < kWRows * (D / 4); i += kF32Threads) {
        const int r = i / (D / 4), c = i % (D / 4);
        const bool ok = rbase + r < rz;
        const int t = a.group_div.div(ok ? rbase + r : 0), h = kh * G + (ok ? rbase + r : 0) - t * G;
        cp_async16(smem_addr(sq + (buf * kWRows + r) * KP + c * 4),
                   static_cast<const float*>(a.q.p) + (q.row0 + t) * a.q.row + h * a.q.head + c * 4, ok);
      }
      if (tid < kWRows) {
        const bool ok = rbase + tid < rz;
        const int t = a.group_div.div(ok ? rbase + tid : 0), h = kh * G + (ok ? rbase + tid : 0) - t * G;
        const float z = ok ? a.lse[static_cast<int64_t>(q.row0 + t) * a.n_q_heads + h] : -INFINITY;
        s_lse[buf * kWRows + tid] = z == -INFINITY ? INFINITY : z * kLog2e;   // weight 0 without a sum
        s_i[buf * kWRows + tid] = q.old + t;
        s_sl[buf * kWRows + tid] = a.slopes ? a.slopes[h] * kLog2e : 0.f;
      }
      cp_async_commit();
    };
    if (blocks > 0) {
      for (int i = tid; i < kWKeysF32 * (D / 4); i += kF32Threads) {
        const int r = i / (D / 4), c = i % (D / 4);
        const int gr = j0 + r < j1 ? slot_row(a.c, s, kh, j0 + r) : -1;
        cp_async16(smem_addr(sk + r * KP + c * 4),
                   static_cast<const float*>(a.k) + static_cast<int64_t>(max(gr, 0)) * D + c * 4, gr >= 0);
      }
      stage_q(0, 0);
    }
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    for (int blk = 0; blk < blocks; ++blk) {
      const int buf = blk & 1;
      cp_async_wait<0>();
      __syncthreads();
      if (blk + 1 < blocks) stage_q(blk + 1, buf ^ 1);
      float sc[4][4] = {};
#pragma unroll 4
      for (int d = 0; d < D; d += 4) {
        float4 kk[4], qq[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) kk[j] = *reinterpret_cast<const float4*>(sk + (tx + 16 * j) * KP + d);
#pragma unroll
        for (int i = 0; i < 4; ++i) qq[i] = *reinterpret_cast<const float4*>(sq + (buf * kWRows + ty * 4 + i) * KP + d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            sc[i][j] = fmaf(qq[i].x, kk[j].x, sc[i][j]);
            sc[i][j] = fmaf(qq[i].y, kk[j].y, sc[i][j]);
            sc[i][j] = fmaf(qq[i].z, kk[j].z, sc[i][j]);
            sc[i][j] = fmaf(qq[i].w, kk[j].w, sc[i][j]);
          }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int col = buf * kWRows + ty * 4 + i, pos = s_i[col];
        const float z = s_lse[col], sl = s_sl[col];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int slot = j0 + tx + 16 * j;
          const bool seen = slot < pre || (slot <= pos && slot > pos - a.window);
          sum[j] += seen ? exp2f(score2(sm, sc[i][j], sl, pos - slot) - z) : 0.f;
        }
      }
    }
    cp_async_wait<0>();
    __syncthreads();                     // the blocks' buffer becomes the sums'
#pragma unroll
    for (int j = 0; j < 4; ++j) part[ty * kWKeysF32 + tx + 16 * j] = sum[j];
    __syncthreads();
    if (tid < kWKeysF32 && j0 + tid < j1) {
      float x = 0.f;
#pragma unroll
      for (int k = 0; k < 16; ++k) x += part[k * kWKeysF32 + tid];
      if (cut) weight_part(a, seg, s, kh)[j0 + tid] = x;
      else add_weight(a, slot_row(a.c, s, kh, j0 + tid), x);
    }
    __syncthreads();
  }
}

template <int D, int MT, bool HALF, bool MOD>
cudaError_t launch_rows(const Launch& L, const PagedAttnArgs& a) {
  constexpr size_t ring = 4 * kRowsStages * kRowsStageBytes;
  constexpr size_t rows = HALF ? 8 : 16 * MT;
  constexpr size_t join = (10 * rows + 4 * rows * D) * sizeof(float);
  constexpr size_t smem = ring > join ? ring : join;
  const dim3 grid(a.splits, a.c.n_heads, a.c.n_seqs);
  return launch_clusters(paged_attn_rows_kernel<D, MT, HALF, MOD>, grid, dim3(kRowsThreads), smem, L.stream, a.cluster,
                         a);
}
template <int D, bool MOD>
cudaError_t launch_rows_d(const Launch& L, const PagedAttnArgs& a) {
  const int rows = a.ch.max_q * a.group;
  return rows <= 8    ? launch_rows<D, 1, true, MOD>(L, a)
         : rows <= 16 ? launch_rows<D, 1, false, MOD>(L, a)
                      : launch_rows<D, 2, false, MOD>(L, a);
}

template <int D, int RM>
cudaError_t launch_f32(const Launch& L, const PagedAttnArgs& a) {
  constexpr int R = F32Cfg<D, RM>::kRows;
  const int blocks = static_cast<int>((static_cast<int64_t>(a.ch.max_q) * a.group + R - 1) / R);
  const dim3 grid(static_cast<unsigned>(blocks) * a.splits, a.c.n_heads, a.c.n_seqs);
  return launch_kernel(paged_attn_f32_kernel<D, RM>, grid, dim3(kF32Threads), F32Cfg<D, RM>::kSmem, L.stream, a, blocks);
}
template <int D>
cudaError_t launch_weights_f32(const Launch& L, const PagedAttnArgs& a, const dim3& grid) {
  constexpr size_t smem = (static_cast<size_t>(kWKeysF32 + 2 * kWRows) * (D + 4) + 3 * 2 * kWRows) * 4;
  return launch_kernel(paged_attn_weights_f32_kernel<D>, grid, dim3(kF32Threads), smem, L.stream, a);
}

// Few rows get eight warps each, so that their parts are read by several SMs' worth of loads at once.
template <int D, bool BF16>
cudaError_t launch_combine(const Launch& L, const PagedAttnArgs& a) {
  const int64_t rows = static_cast<int64_t>(a.ch.n_tokens) * a.n_q_heads;
  const dim3 block(kCombineThreads);
  if (rows <= 8 * L.sm_count && a.parts >= 16)
    return launch_kernel(paged_attn_combine_kernel<D, BF16, 8>, dim3(static_cast<unsigned>(rows)), block, 0, L.stream, a);
  return launch_kernel(paged_attn_combine_kernel<D, BF16, 1>, dim3(static_cast<unsigned>((rows + 7) / 8)), block, 0,
                       L.stream, a);
}

template <int D, bool MOD>
cudaError_t launch_weights(const Launch& L, const PagedAttnArgs& a, const dim3& grid) {
  constexpr size_t smem = 2 * kWRows * 2 * D + 3 * 2 * kWRows * 4;
  return launch_kernel(paged_attn_weights_kernel<D, MOD>, grid, dim3(128), smem, L.stream, a);
}

}  // namespace

cudaError_t launch_paged_attn_rows(const Launch& L, const PagedAttnArgs& a) {
  const bool mod = a.cap > 0.f || a.slopes != nullptr;
  if (a.head_dim == 128) return mod ? launch_rows_d<128, true>(L, a) : launch_rows_d<128, false>(L, a);
  return mod ? launch_rows_d<64, true>(L, a) : launch_rows_d<64, false>(L, a);
}

cudaError_t launch_paged_attn_f32(const Launch& L, const PagedAttnArgs& a) {
  const int64_t all = static_cast<int64_t>(a.ch.max_q) * a.group;
  const int block = f32_block_rows(all);
  if (block == kF32RowBlock) {
    const int blocks = static_cast<int>((all + block - 1) / block);
    const dim3 grid(static_cast<unsigned>(blocks) * a.splits, a.c.n_heads, a.c.n_seqs);
    return a.head_dim == 128 ? launch_kernel(paged_attn_f32_rows_kernel<128>, grid, dim3(128), kF32RowSmem, L.stream, a, blocks)
                             : launch_kernel(paged_attn_f32_rows_kernel<64>, grid, dim3(128), kF32RowSmem, L.stream, a, blocks);
  }
  if (a.head_dim == 128) return block == 32 ? launch_f32<128, 2>(L, a) : launch_f32<128, 4>(L, a);
  return block == 32 ? launch_f32<64, 2>(L, a) : launch_f32<64, 4>(L, a);
}

cudaError_t launch_paged_attn_combine(const Launch& L, const PagedAttnArgs& a, bool bf16) {
  if (a.head_dim == 128) return bf16 ? launch_combine<128, true>(L, a) : launch_combine<128, false>(L, a);
  return bf16 ? launch_combine<64, true>(L, a) : launch_combine<64, false>(L, a);
}

cudaError_t launch_paged_attn_weights(const Launch& L, const PagedAttnArgs& a, bool bf16, int64_t max_kv) {
  const bool mod = a.cap > 0.f || a.slopes != nullptr;
  if (a.scores != nullptr) {
    const int blocks = static_cast<int>((max_kv + kCombineThreads - 1) / kCombineThreads);
    const dim3 g(static_cast<unsigned>(blocks + (a.parts > 1 ? a.ch.max_q * a.group : 0)), a.c.n_heads, a.c.n_seqs);
    const dim3 t(kCombineThreads);
    if (a.head_dim == 128)
      return bf16 ? launch_kernel(paged_attn_weights_kept_kernel<128, true>, g, t, 0, L.stream, a, blocks)
                  : launch_kernel(paged_attn_weights_kept_kernel<128, false>, g, t, 0, L.stream, a, blocks);
    return bf16 ? launch_kernel(paged_attn_weights_kept_kernel<64, true>, g, t, 0, L.stream, a, blocks)
                : launch_kernel(paged_attn_weights_kept_kernel<64, false>, g, t, 0, L.stream, a, blocks);
  }
  const int keys = bf16 ? kWKeys : kWKeysF32;
  const dim3 grid(static_cast<unsigned>((max_kv + keys - 1) / keys * a.w_segs), a.c.n_heads, a.c.n_seqs);
  cudaError_t e;
  if (!bf16)
    e = a.head_dim == 128 ? launch_weights_f32<128>(L, a, grid) : launch_weights_f32<64>(L, a, grid);
  else if (a.head_dim == 128)
    e = mod ? launch_weights<128, true>(L, a, grid) : launch_weights<128, false>(L, a, grid);
  else
    e = mod ? launch_weights<64, true>(L, a, grid) : launch_weights<64, false>(L, a, grid);
  if (e != cudaSuccess || a.w_segs == 1) return e;
  const dim3 g(static_cast<unsigned>((max_kv + 127) / 128), a.c.n_heads, a.c.n_seqs);
  return launch_kernel(paged_attn_weights_sum_kernel, g, dim3(128), 0, L.stream, a, keys);
}

}  // namespace vx
