// paged_attn_tc.cu -- attention of a chunk of tokens over the paged cache on
// the tcgen05 tensor cores.
#include "paged_attn.cuh"

namespace vx {

namespace {

// paged_attn_tc_kernel: CTA per (256-row block, K/V head, sequence, key
// range).  Rows are (token t, head g of the group), r = t * G + g, so a K/V
// tile serves the group's heads at once; softmax warpgroup X owns rows
// 128 X .. 128 X + 127 of the block (TMEM lane = row).  Keys are walked in
// tiles of 128 of the block's key list.  Pages may have any size, so a tile's
// rows lie anywhere: four producer warps copy them row by row with cp.async
// into the 128-byte-swizzled layout the tensor core reads (rows past the
// sequence as zeros), K and V tiles alternating in one ring.  One thread per
// warpgroup issues S = Q K^T into TMEM, waits for P (written over S as bf16)
// and issues O += P V; the two warpgroups' softmax phases and products
// overlap.  O is rescaled in place only when a row's maximum grows by more
// than 2^8.
constexpr int kTcThreads = 512;   // 2 x 4 softmax warps, 4 producer warps, 2 issuers + 2 idle
constexpr int kTcKeys = 128;
constexpr float kTcSlack = 8.0f;
// setmaxnreg: 256 x 200 + 256 x 56 = the 512 x 128 of the launch.
constexpr int kTcSoftmaxRegs = 200;
constexpr int kTcOtherRegs = 56;

template <int D>
struct TcCfg {
  static constexpr int kTile = kTcKeys * D * 2;               // one Q, K or V tile
  static constexpr int kStages = D == 128 ? 5 : 8;            // ring of K / V tiles
  static constexpr int kLag = kStages - 2;                    // copies in flight behind the newest
  static constexpr int kSmem = 2 * kTile + kStages * kTile + 1024 + 256;
};

struct TcItem {
  int s, kh, sp;
  int n_act;           // warpgroups with rows (1 or 2)
  int r0, rows;        // first row of the block, rows of the sequence
  KeyList kl;
  int x0, x1, nt;      // this CTA's part of the list, tiles
  SeqSpan q;
};

// The tile of keys [xt, xt + 128) meets what some row of warpgroup X sees.
__device__ __forceinline__ bool tc_tile_used(const PagedAttnArgs& a, const TcItem& it, int X, int xt) {
  const int ra = it.r0 + X * 128, rz = min(ra + 127, it.rows - 1);
  const int i_first = it.q.old + static_cast<int>(a.group_div.div(ra));
  const int i_last = it.q.old + static_cast<int>(a.group_div.div(rz));
  return xt < it.kl.pre || (xt <= i_last - it.kl.shift && xt + kTcKeys - 1 >= i_first - a.window + 1 - it.kl.shift);
}

template <int D, bool MOD>
__global__ void __launch_bounds__(kTcThreads, 1)
paged_attn_tc_kernel(const __grid_constant__ PagedAttnArgs a, int blocks) {
  using Cfg = TcCfg<D>;
  constexpr int NST = Cfg::kStages, LAG = Cfg::kLag, TILE = Cfg::kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                    // 2 tiles; a tile = D / 64 halves of [128 rows][128 bytes]
  uint8_t* sKV = smem + 2 * TILE;        // ring: K(0), V(0), K(1), V(1), ...
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + NST * TILE);
  constexpr int FULL = 0, EMPTY = NST, SF = 2 * NST, PF = SF + 2, PVD = PF + 2, DR = PVD + 2, NBAR = DR + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBAR);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  auto bar = [&](int i) { return smem_addr(bars + i); };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  pdl_wait();
  // Row blocks from the last (most keys under a causal mask) to the first.
  TcItem it;
  {
    int id = blockIdx.x;
    it.sp = id % a.splits;
    id /= a.splits;
    it.kh = id % a.c.n_heads;
    id /= a.c.n_heads;
    it.s = id % a.c.n_seqs;
    it.r0 = (blocks - 1 - id / a.c.n_seqs) * 256;
  }
  it.q = seq_span(a.c, a.ch, it.s);
  it.rows = it.q.n * a.group;
  if (it.r0 >= it.rows) return;
  it.n_act = it.rows - it.r0 > 128 ? 2 : 1;
  {
    const int tf = a.group_div.div(it.r0), tl = a.group_div.div(min(it.r0 + 255, it.rows - 1));
    it.kl = key_list(it.q.old + tf, it.q.old + tl, a.window, a.prefix ? a.prefix[it.s] : 0, it.q.kv);
    const int step = ((it.kl.total + a.splits - 1) / a.splits + kTcKeys - 1) / kTcKeys * kTcKeys;
    it.x0 = min(it.sp * step, it.kl.total);
    it.x1 = min(it.x0 + step, it.kl.total);
    it.nt = (it.x1 - it.x0 + kTcKeys - 1) / kTcKeys;
  }
  if (threadIdx.x == 0) {
    if (it.q.over) report_bad_cache(a.status, it.s);
    for (int i = 0; i < NST; ++i) { mbar_init(bar(FULL + i), 128); mbar_init(bar(EMPTY + i), it.n_act); }
    for (int X = 0; X < 2; ++X) {
      mbar_init(bar(SF + X), 1);
      mbar_init(bar(PF + X), 128);
      mbar_init(bar(PVD + X), 1);
      mbar_init(bar(DR + X), 1);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 12) {
    tmem_alloc(smem_addr(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_trigger();   // only now that the CTA holds its TMEM: a dependent CTA never keeps it from one
  const uint32_t tmem = *tmem_slot;
  const WaitCtx wc{a.status, abort_flag, a.limit_ns};

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kTcOtherRegs));
    if (warp < 12) {
      // ------------- producers: Q, then K(u), V(u) for every tile
      constexpr int CPR = D / 8, RPI = 32 / CPR;   // 16-byte chunks of a row, rows per warp-wide copy
      const int w = warp - 8, rbase = w * 32;      // this warp's 32 rows of every tile
      const int c = lane % CPR;
      const uint32_t coff = (c >> 3) * (kTcKeys * 128);
      const int ch = c & 7;
      const uint16_t* qp = static_cast<const uint16_t*>(a.q.p);
      for (int X = 0; X < it.n_act; ++X) {
        const uint32_t dst = smem_addr(sQ + X * TILE) + coff;
        for (int k = 0; k < 32 / RPI; ++k) {
          const int r = rbase + k * RPI + lane / CPR;
          const int rr = it.r0 + X * 128 + r;
          const bool ok = rr < it.rows;
          const int t = a.group_div.div(ok ? rr : 0), h = it.kh * a.group + (ok ? rr : 0) - t * a.group;
          cp_async16(dst + r * 128 + ((ch ^ (r & 7)) << 4),
                     qp + (it.q.row0 + t) * a.q.row + h * a.q.head + c * 8, ok);
        }
      }
      cp_async_commit();
      auto lookup = [&](int u) -> int64_t {
        const int x = it.x0 + u * kTcKeys + rbase + lane;
        if (u >= it.nt || x >= it.x1) return -1;
        const int64_t r = slot_row(a.c, it.s, it.kh, key_slot(it.kl, x));
        if (r < 0) report_bad_cache(a.status, it.s);
        return r;
      };
      int64_t row = 0, next = lookup(0);
      const int nb = 2 * it.nt;
      bool ok = true;
      for (int b = 0; b < nb; ++b) {
        const int st = b % NST;
        const bool w_ok = mbar_wait(bar(EMPTY + st), ((b / NST) & 1) ^ 1, wc, 70);
        if (!__all_sync(0xffffffffu, w_ok)) { ok = false; break; }
        if ((b & 1) == 0) {
          row = next;
          next = lookup(b / 2 + 1);
        }
        const uint16_t* pool = static_cast<const uint16_t*>((b & 1) ? a.v : a.k);
        const uint32_t dst = smem_addr(sKV + st * TILE) + coff;
#pragma unroll
        for (int k = 0; k < 32 / RPI; ++k) {
          const int rl = k * RPI + lane / CPR, r = rbase + rl;
          const int64_t gr = __shfl_sync(0xffffffffu, row, rl);
          cp_async16(dst + r * 128 + ((ch ^ (r & 7)) << 4), pool + (gr < 0 ? 0 : gr) * D + c * 8, gr >= 0);
        }
        cp_async_commit();
        if (b >= LAG) {   // the buffer LAG back (and Q with the first) has landed
          cp_async_wait<LAG>();
          fence_proxy_async_smem();
          mbar_arrive(bar(FULL + (b - LAG) % NST));
        }
      }
      cp_async_wait<0>();
      fence_proxy_async_smem();
      if (ok)
        for (int b = max(0, nb - LAG); b < nb; ++b) mbar_arrive(bar(FULL + b % NST));
    } else if (warp < 14 && lane == 0 && warp - 12 < it.n_act) {
      // ------------- tensor-core products of warpgroup X
      const int X = warp - 12;
      const uint32_t tS = tmem + X * 128, tO = tmem + 256 + X * D;
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, kTcKeys, 0);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, 1);
      const uint32_t qa = smem_addr(sQ + X * TILE);
      int t = 0;
      bool ok = true;
      for (int u = 0; ok && u < it.nt; ++u) {
        const int bk = 2 * u, bv = bk + 1, sk = bk % NST, sv = bv % NST;
        if (!(ok = mbar_wait(bar(FULL + sk), (bk / NST) & 1, wc, 71))) break;
        const bool used = tc_tile_used(a, it, X, it.x0 + u * kTcKeys);
        if (!used) {
          mbar_arrive(bar(EMPTY + sk));
          if (!(ok = mbar_wait(bar(FULL + sv), (bv / NST) & 1, wc, 72))) break;
          mbar_arrive(bar(EMPTY + sv));
          continue;
        }
        tc_fence_after();
        const uint32_t ka = smem_addr(sKV + sk * TILE), va = smem_addr(sKV + sv * TILE);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {   // S(t) overwrites P(t - 1), which the product before it has read
          const uint32_t o = (kk >> 2) * (kTcKeys * 128) + (kk & 3) * 32;
          umma_bf16(tS, smem_desc_sw128(qa + o, 16, 1024), smem_desc_sw128(ka + o, 16, 1024), idesc_s, kk > 0);
        }
        umma_commit(bar(SF + X));
        umma_commit(bar(EMPTY + sk));
        if (!(ok = mbar_wait(bar(FULL + sv), (bv / NST) & 1, wc, 73))) break;
        if (!(ok = mbar_wait(bar(PF + X), t & 1, wc, 74))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kTcKeys / 16; ++kk)   // 16 keys: 8 TMEM columns of P, 16 rows of V
          umma_bf16_ts(tO, tS + 8 * kk, smem_desc_sw128(va + kk * 2048, kTcKeys * 128, 1024), idesc_o,
                       (t > 0 || kk > 0) ? 1u : 0u);
        umma_commit(bar(PVD + X));
        umma_commit(bar(EMPTY + sv));
        ++t;
      }
      umma_commit(bar(DR + X));
      int zero = 0;
      WaitCtx dw = wc;
      dw.abort_flag = &zero;
      mbar_wait(bar(DR + X), 0, dw, 75);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcSoftmaxRegs));
    // ------------- softmax: warpgroup X, thread = row
    const int X = warp >> 2;
    if (X < it.n_act) {
      const int r = it.r0 + X * 128 + (threadIdx.x & 127);
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const uint32_t tS = tmem + X * 128 + lane_off, tO = tmem + 256 + X * D + lane_off;
      const ScoreMod sm = score_mod(a);
      // Rows past the sequence's follow its last one and are not stored.
      const int rc = min(r, it.rows - 1);
      const int tt = a.group_div.div(rc), h = it.kh * a.group + rc - tt * a.group;
      const int i = it.q.old + tt;
      const float slope2 = MOD && a.slopes ? a.slopes[h] * kLog2e : 0.f;
      const int xlo = max(0, i - a.window + 1 - it.kl.shift), xhi = min(i - it.kl.shift, it.x1 - 1);
      const int pre = min(it.kl.pre, it.x1);
      const int all_lo = __reduce_max_sync(0xffffffffu, xlo), all_hi = __reduce_min_sync(0xffffffffu, xhi);
      float m_used = -INFINITY, l_run = 0.f;
      int t = 0;
      bool ok = true;
      for (int u = 0; u < it.nt; ++u) {
        const int xt = it.x0 + u * kTcKeys;
        if (!tc_tile_used(a, it, X, xt)) continue;
        bool w = mbar_wait(bar(SF + X), t & 1, wc, 76);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        tc_fence_after();
        float sv[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t(&rr)[32] = *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * c);
          tmem_ld32(tS + 32 * c, rr);
        }
        tmem_ld_wait();
        if constexpr (MOD) {
#pragma unroll
          for (int e = 0; e < 128; ++e) sv[e] = score2(sm, sv[e], slope2, abs(i - key_slot(it.kl, xt + e)));
        }
        if (!((xt >= all_lo && xt + kTcKeys - 1 <= all_hi) || xt + kTcKeys - 1 < pre)) {
          const int lo = xlo - xt, hi = xhi - xt, pr = pre - xt;
#pragma unroll
          for (int e = 0; e < 128; ++e) sv[e] = ((e >= lo && e <= hi) || e < pr) ? sv[e] : -INFINITY;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 128; e += 4)
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = fmaxf(mx[k], sv[e + k]);
        const float sc = MOD ? 1.f : sm.sl2;
        const float m_tile = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sc;
        float corr = 1.f;
        if (m_tile > m_used + kTcSlack) {
          if (m_used != -INFINITY) corr = ex2_approx(m_used - m_tile);
          m_used = m_tile;
        }
        l_run *= corr;
        if (t > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
          w = mbar_wait(bar(PVD + X), (t - 1) & 1, wc, 77);
          if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t o[32];
            tmem_ld32(tO + 32 * c, o);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
            tmem_st32(tO + 32 * c, o);
          }
        }
        const float mu = m_used == -INFINITY ? 0.f : m_used;
        float rs[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pk[32];
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            const float p0 = ex2_approx(fmaf(sv[c * 64 + 2 * e], sc, -mu));
            const float p1 = ex2_approx(fmaf(sv[c * 64 + 2 * e + 1], sc, -mu));
            rs[e & 3] += p0 + p1;
            pk[e] = pack_bf16x2(p0, p1);
          }
          tmem_st32(tS + 32 * c, pk);
        }
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(bar(PF + X));
        l_run += (rs[0] + rs[1]) + (rs[2] + rs[3]);
        ++t;
      }
      if (ok && t > 0) {
        const bool w = mbar_wait(bar(PVD + X), (t - 1) & 1, wc, 78);
        ok = __all_sync(0xffffffffu, w);
        tc_fence_after();
      }
      if (ok) {
        const int64_t tok = it.q.row0 + tt;
        const bool mine = r < it.rows;
        const bool empty = l_run == 0.f;   // a NaN score leaves a NaN sum
        const float inv = empty ? 0.f : 1.f / l_run;
        const int64_t pr = (static_cast<int64_t>(it.sp) * a.ch.n_tokens + tok) * a.n_q_heads + h;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) {
          uint32_t o[32];
          if (t > 0) {
            tmem_ld32(tO + 32 * c, o);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (!mine) continue;
          if (a.splits > 1) {
            float* dst = a.part_o + pr * D + c * 32;
            if (!empty)
#pragma unroll
              for (int e = 0; e < 32; e += 4) st_global_v4(dst + e, o[e], o[e + 1], o[e + 2], o[e + 3]);
          } else {
            uint16_t* dst = static_cast<uint16_t*>(a.o) + tok * a.o_row + h * a.o_head + c * 32;
            uint32_t y[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              y[e] = empty ? 0u : pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
#pragma unroll
            for (int e = 0; e < 16; e += 4) st_global_v4(dst + 2 * e, y[e], y[e + 1], y[e + 2], y[e + 3]);
          }
        }
        if (mine) {
          if (a.splits > 1) a.part_ml[pr] = make_float2(m_used, l_run);
          else if (a.lse) a.lse[tok * a.n_q_heads + h] = empty ? -INFINITY : (m_used + log2f(l_run)) * kLn2;
        }
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool MOD>
cudaError_t launch_tc(const Launch& L, const PagedAttnArgs& a, int blocks) {
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(blocks) * a.c.n_seqs * a.c.n_heads * a.splits);
  return launch_kernel(paged_attn_tc_kernel<D, MOD>, dim3(grid), dim3(kTcThreads), TcCfg<D>::kSmem, L.stream, a,
                       blocks);
}

}  // namespace

cudaError_t launch_paged_attn_tc(const Launch& L, const PagedAttnArgs& a) {
  const int blocks = static_cast<int>((static_cast<int64_t>(a.ch.max_q) * a.group + 255) / 256);
  const bool mod = a.cap > 0.f || a.slopes != nullptr;
  if (a.head_dim == 128) return mod ? launch_tc<128, true>(L, a, blocks) : launch_tc<128, false>(L, a, blocks);
  return mod ? launch_tc<64, true>(L, a, blocks) : launch_tc<64, false>(L, a, blocks);
}

}  // namespace vx
