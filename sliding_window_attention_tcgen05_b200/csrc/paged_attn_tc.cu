// paged_attn_tc.cu -- attention of a chunk of tokens over the paged cache on
// the tcgen05 tensor cores.
#include "paged_attn.cuh"

namespace vx {

namespace {

// paged_attn_tc_kernel: CTA per (256-row block, K/V head, sequence, key
// range).  Rows are (token t, head g of the group), r = t * G + g, so a K/V
// tile serves the group's heads at once; softmax warpgroup X owns rows
// 128 X .. 128 X + 127 of the block (TMEM lane = row).  Keys are walked in
// tiles of 128 of the block's key list.  Pages may have any size and the list
// may start anywhere in one, so a tile's rows lie anywhere: where the page size
// is a multiple of 8 the list is cut into aligned runs of up to 128 rows that
// lie in one page, and one producer warp for K and one for V fetch each run by
// TMA; rows of a run that holds others than the block's keys, and all rows of
// odd page sizes, are copied with cp.async into the same 128-byte-swizzled
// layout (zeros for the others).  K and V tiles alternate in one ring.
// A warp per warpgroup issues O += P V as P arrives (written over S as bf16, 64
// keys at a time), then the next S = Q K^T.  O is rescaled in place only when
// a row's maximum grows by more than 2^8.  P is the one thing held in fewer
// bits than fp32: kind::f16 products take both operands as bf16 where V is
// bf16.  That rounding, 2^-9 of a weight at random, is as large as the output's
// own (against float64, relative: 2.0e-3 to 2.4e-3, of which the output's
// rounding alone makes 1.65e-3); P as two bf16 terms would double the products
// with V.  l sums the unrounded weights, so that lse has no part in it.
//
// What bounds it: a warpgroup's chain of softmax (about 1700 cycles a tile,
// 1024 of them MUFU issue), products (12 x 64 behind the last weights) and
// hand-overs; TMEM (two S, two O of 128 columns) has no room for a second S.
// So what counts is that one warpgroup's chain runs under the other's: the
// warps that share a scheduler take turns at their exponentials (left alone the
// warpgroups fall into step).  Measured for 4 ragged prompts of up to 4096
// tokens over 8192, 32/8 heads of 128 (819 GFLOP), 20 passes at 1965 MHz: 780 us
// (1050 TFLOP/s, 64% of cuBLAS's burst rate; back to back under the power cap,
// at 1.72 GHz, 875); without the turns 837; all weights handed over at once
// 828, in three parts 830; a quarter of the exponentials on the FMA pipe
// (range reduction and a polynomial) 895; rows all by cp.async, which feeds an
// SM 16 bytes a clock, 1026; TMA gathers of four rows 1276.
constexpr int kTcThreads = 384;   // 2 x 4 softmax warps, 2 issuers, 2 producer warps
constexpr int kTcKeys = 128;
constexpr float kTcSlack = 8.0f;
// setmaxnreg: 256 x 216 + 128 x 72 = the 384 x 168 of the launch.  A row's 128
// scores stay in registers (at 512 threads x 128 they spilled).
constexpr int kTcSoftmaxRegs = 216;
constexpr int kTcOtherRegs = 72;

template <int D>
struct TcCfg {
  static constexpr int kTile = kTcKeys * D * 2;               // one Q, K or V tile
  static constexpr int kStages = D == 128 ? 5 : 8;            // ring of K / V tiles
  static constexpr int kLag = 1;                              // a producer's cp.async tiles in flight behind the newest
  static constexpr int kBars = 2 * kStages + 19;              // mbarriers of the CTA
  static constexpr int kTail = (kBars + 1) * 8;               // behind the tiles: the barriers, the TMEM address, the abort flag
  static constexpr int kSmem = 2 * kTile + kStages * kTile + 1024 + kTail;   // 1024: the tiles' alignment
};

struct TcItem {
  int s, kh, sp;
  int n_act;           // warpgroups with rows (1 or 2)
  int r0, rows;        // first row of the block, rows of the sequence
  KeyList kl;
  int x0, x1, nt;      // this CTA's part of the list, tiles
  SeqSpan q;
};

// The tiles first .. end - 1 of the CTA's that warpgroup X uses: the others,
// at either end, hold no key that its rows see.
struct TcTiles {
  int first, end;
};
__device__ __forceinline__ TcTiles tc_tiles(const PagedAttnArgs& a, const TcItem& it, int X) {
  const int ra = it.r0 + X * 128, rz = min(ra + 127, it.rows - 1);
  const int i_first = it.q.old + static_cast<int>(a.group_div.div(ra));
  const int i_last = it.q.old + static_cast<int>(a.group_div.div(rz));
  const int lo = it.kl.pre > it.x0 ? it.x0 : max(it.x0, i_first - a.window + 1 - it.kl.shift);
  const int hi = max(i_last - it.kl.shift, it.kl.pre - 1);   // last key seen
  TcTiles t;
  t.first = min((lo - it.x0) / kTcKeys, it.nt);
  t.end = hi < it.x0 ? 0 : min((hi - it.x0) / kTcKeys + 1, it.nt);
  t.end = max(t.end, t.first);
  return t;
}

// Rows of tile u that the product with V reads: those of the list, rounded up
// to the 16 of a product.
__device__ __forceinline__ int tc_rows(const TcItem& it, int u) {
  return (min(kTcKeys, it.x1 - it.x0 - u * kTcKeys) + 15) & ~15;
}

template <class T>
__device__ __forceinline__ T uniform(T x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
// 32 columns of O (zeros where no product was issued).
__device__ __forceinline__ void tc_output(uint32_t addr, bool any, uint32_t (&o)[32]) {
  if (any) {
    tmem_ld32(addr, o);
    tmem_ld_wait();
  } else {
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = 0u;
  }
}

// mbar_wait, with a first sleep before it starts its clock: nearly every wait
// ends in that sleep, and reading the global timer takes longer than most.
__device__ __forceinline__ bool tc_wait(uint32_t bar, uint32_t parity, const WaitCtx& w, int where) {
  if (mbar_try_wait(bar, parity) || mbar_try_wait_sleep(bar, parity, 20000u)) return true;
  return mbar_wait(bar, parity, w, where);
}

__device__ __forceinline__ bool mbar_test_wait(uint32_t bar, uint32_t parity) {   // does not wait
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {   // no arrival
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ float ex2_ordered(float x) {   // keeps its place among the other asm statements
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The maximum of three.
__device__ __forceinline__ float fmax3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

template <int D, bool MOD>
__global__ void __launch_bounds__(kTcThreads, 1)
paged_attn_tc_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                     const __grid_constant__ PagedAttnArgs a, int blocks, int run) {
  using Cfg = TcCfg<D>;
  constexpr int NST = Cfg::kStages, TILE = Cfg::kTile;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;                    // 2 tiles; a tile = D / 64 halves of [128 rows][128 bytes]
  uint8_t* sKV = smem + 2 * TILE;        // ring: K(0), V(0), K(1), V(1), ...
  uint64_t* bars = reinterpret_cast<uint64_t*>(sKV + NST * TILE);
  // TK: the turns of warp w of each warpgroup at their scheduler's MUFU.
  constexpr int FULL = 0, EMPTY = NST, SF = 2 * NST, PF = SF + 2, PVD = PF + 4, DR = PVD + 2, TK = DR + 2, QF = TK + 8, NBAR = QF + 1;
  static_assert(NBAR == Cfg::kBars && NBAR * 8 + 8 <= Cfg::kTail, "shared memory behind the tiles");
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
    it.kl = key_list(it.q.old + tf, it.q.old + tl, a.window, a.prefix ? a.prefix[it.s] : 0, it.q.kv, run);
    const int step = ((it.kl.total + a.splits - 1) / a.splits + kTcKeys - 1) / kTcKeys * kTcKeys;
    it.x0 = min(it.sp * step, it.kl.total);
    it.x1 = min(it.x0 + step, it.kl.total);
    it.nt = (it.x1 - it.x0 + kTcKeys - 1) / kTcKeys;
  }
  // Pool rows of four rows of tile u, or -1: lane * 4 + k where runs are fetched
  // by TMA (so that a run's rows are R / 4 neighbouring lanes'), else lane + 32 k.
  const bool tma = run >= 8;
  auto lookup = [&](int u, int (&row)[4]) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int x = it.x0 + u * kTcKeys + (tma ? lane * 4 + k : lane + 32 * k);
      row[k] = -1;
      if (u >= it.nt || x >= it.x1) continue;
      const int j = key_slot(it.kl, x);
      if (!wanted(it.kl, j)) continue;
      row[k] = slot_row(a.c, it.s, it.kh, j);
      if (row[k] < 0) report_bad_cache(a.status, it.s);
    }
  };
  int next[4];
  if (warp >= 10) lookup(0, next);   // its table reads travel under the set-up

  if (threadIdx.x == 0) {
    if (it.q.over) report_bad_cache(a.status, it.s);
    for (int i = 0; i < NST; ++i) { mbar_init(bar(FULL + i), 32); mbar_init(bar(EMPTY + i), it.n_act); }
    for (int X = 0; X < 2; ++X) {
      mbar_init(bar(SF + X), 1);
      mbar_init(bar(PF + 2 * X), 128);       // P of keys 0 .. 63 of the tile
      mbar_init(bar(PF + 2 * X + 1), 128);   // and 64 .. 127
      mbar_init(bar(PVD + X), 1);
      mbar_init(bar(DR + X), 1);
      for (int w = 0; w < 4; ++w) mbar_init(bar(TK + 4 * X + w), 1);
    }
    mbar_init(bar(QF), 128 * it.n_act);
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 8) {
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
    if (warp >= 10) {
      // ------------- producers: warp 10 the K and warp 11 the V tiles
      constexpr int CPR = D / 8, RPI = 32 / CPR;      // 16-byte chunks of a row, rows per warp-wide copy
      const int c = lane % CPR, ch = c & 7, rl0 = lane / CPR;
      const uint32_t coff = (c >> 3) * (kTcKeys * 128);
      const bool is_v = warp == 11;
      const CUtensorMap* tm = is_v ? &tmV : &tmK;
      const uint8_t* pool = static_cast<const uint8_t*>(is_v ? a.v : a.k) + c * 16;
      if (lane == 0) tma_prefetch_desc(tm);
      int row[4];
      int u = 0, told = 0;   // tiles issued, tiles whose arrival the consumers were told of (cp.async)
      auto stage_of = [&](int v) { return (2 * v + (is_v ? 1 : 0)) % NST; };
      auto landed = [&](int in_flight) {   // tile `told` has landed once so many newer ones fly
        if (in_flight >= 1) cp_async_wait<1>(); else cp_async_wait<0>();
        fence_proxy_async_smem();
        mbar_arrive(bar(FULL + stage_of(told)));
        ++told;
      };
      for (; u < it.nt; ++u) {
        const int st = stage_of(u);
        const uint32_t full = bar(FULL + st), dst = smem_addr(sKV + st * TILE);
        const uint32_t empty = (((2 * u + (is_v ? 1 : 0)) / NST) & 1) ^ 1;
#pragma unroll
        for (int k = 0; k < 4; ++k) row[k] = next[k];
        // Rows that the product with V reads; of K all, where a cap's formula is chosen by a row's largest score (what lay
        // behind the list's end before may not choose it).
        const int used = MOD && !is_v && a.cap > 0.f ? kTcKeys : tc_rows(it, u);
        // No free buffer: nothing to issue, so pass on what lands meanwhile.
        if (!tma)
          while (told < u && !__all_sync(0xffffffffu, mbar_test_wait(bar(EMPTY + st), empty))) landed(u - told - 1);
        const bool w_ok = tc_wait(bar(EMPTY + st), empty, wc, 70);
        if (!__all_sync(0xffffffffu, w_ok)) break;
        if (tma) {
          const uint32_t have = __ballot_sync(0xffffffffu, min(min(row[0], row[1]), min(row[2], row[3])) >= 0);
          const int lanes = run / 4;                                   // of a run
          const uint32_t mine = (lanes == 32 ? 0xffffffffu : (1u << lanes) - 1u) << (lane & -lanes);
          const bool whole = (have & mine) == mine;
          const uint32_t runs = __ballot_sync(0xffffffffu, whole);     // a bit for each lane of a whole run
          // Announced alone: lane 0 arrives like the others, after its own copies have landed (their waits and fences
          // order no other lane's).
          if (lane == 0) mbar_expect_tx(full, __popc(runs) * (4 * D * 2));
          __syncwarp();
          if (whole && (lane & (lanes - 1)) == 0)
#pragma unroll
            for (int hf = 0; hf < D / 64; ++hf)
              tma_load_2d(dst + hf * (kTcKeys * 128) + lane * 512, tm, full, hf * 64, row[0]);
          if (runs != 0xffffffffu) {   // rows of runs that hold others than the block's keys, zeros for those
            for (int k = 0; k < used / RPI; ++k) {
              const int r = k * RPI + rl0;
              if ((runs >> (k * RPI / 4)) & 1u) continue;              // a warp-wide copy lies in one run
              int gr = -1;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const int y = __shfl_sync(0xffffffffu, row[j], r >> 2);
                if ((r & 3) == j) gr = y;
              }
              cp_async16(dst + coff + r * 128 + ((ch ^ (r & 7)) << 4),
                         pool + static_cast<int64_t>(max(gr, 0)) * (2 * D), gr >= 0);
            }
            cp_async_commit();
            cp_async_wait<0>();
            fence_proxy_async_smem();
          }
          mbar_arrive(full);
        } else {
#pragma unroll
          for (int k0 = 0; k0 < 128 / RPI; k0 += 8) {   // eight rows' numbers first: a shuffle before each copy takes 75 cycles a copy
            if (k0 * RPI >= used) break;
            int gr[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
              gr[k] = __shfl_sync(0xffffffffu, row[(k0 + k) * RPI / 32], ((k0 + k) * RPI + rl0) & 31);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const int r = (k0 + k) * RPI + rl0;
              cp_async16(dst + coff + r * 128 + ((ch ^ (r & 7)) << 4),
                         pool + static_cast<int64_t>(max(gr[k], 0)) * (2 * D), gr[k] >= 0);
            }
          }
          cp_async_commit();
          if (u - told >= Cfg::kLag) landed(Cfg::kLag);
        }
        lookup(u + 1, next);
      }
      while (!tma && u == it.nt && told < u) landed(u - told - 1);
      cp_async_wait<0>();
      if (tma && (u < it.nt || *abort_flag)) {   // gave up: the copies in flight must land before the CTA ends
        int zero = 0;
        WaitCtx dw = wc;
        dw.abort_flag = &zero;
        for (int v = max(0, u - NST / 2 - 1); v < u; ++v) {
          const int b = 2 * v + (is_v ? 1 : 0);
          tc_wait(bar(FULL + b % NST), (b / NST) & 1, dw, 80);
        }
      }
    } else if (warp - 8 < it.n_act) {
      // ------------- tensor-core products of warpgroup X: the whole warp walks the loop, so that the compiler knows its
      // values to be the same in all lanes and keeps them where the products want them (a product is then issued in 32
      // cycles, in 85 by a lone thread); one lane issues
      const int X = uniform(warp - 8), nt = uniform(it.nt);
      const uint32_t tm = uniform(tmem), tS = tm + X * 128, tO = tm + 256 + X * D;
      constexpr uint32_t idesc_s = idesc_bf16_f32(128, kTcKeys, 0);
      constexpr uint32_t idesc_o = idesc_bf16_f32(128, D, 1);
      TcTiles tiles = tc_tiles(a, it, X);
      tiles.first = uniform(tiles.first);
      tiles.end = uniform(tiles.end);
      const int rows_left = uniform(it.x1 - it.x0);
      // Descriptors of the first tiles; a stage or a K step further is an addition to the address field (built anew
      // for each product they take longer than the product).
      const uint32_t at_q = uniform(smem_addr(sQ + X * TILE)), at_kv = uniform(smem_addr(sKV));
      const uint64_t desc_q = smem_desc_sw128(at_q, 16, 1024);
      const uint64_t desc_k = smem_desc_sw128(at_kv, 16, 1024);
      const uint64_t desc_v = smem_desc_sw128(at_kv, kTcKeys * 128, 1024);
      const uint32_t b0 = uniform(bar(0));
      auto ubar = [&](int i) { return b0 + 8 * i; };
      const bool lead = elect_one();
      auto wait = [&](int i, uint32_t parity, int where) {
        return __all_sync(0xffffffffu, tc_wait(ubar(i), parity, wc, where)) != 0;
      };
      bool ok = nt == 0 || wait(QF, 0, 79);
      int sk = 0, sv = NST - 1;             // stages of K(u + 1) and V(u)
      uint32_t pk = 0, pvp = 1;             // and their parities
      for (int u = -1; ok && u < nt; ++u) {   // O += P V of tile u, then S of tile u + 1
        const int t = u - tiles.first;
        const bool pv = u >= tiles.first && u < tiles.end, sc = u + 1 >= tiles.first && u + 1 < tiles.end;
        const uint64_t dv = desc_v + static_cast<uint32_t>(sv * (TILE >> 4));
        const int used = (min(kTcKeys, rows_left - u * kTcKeys) + 15) & ~15;
        auto half_pv = [&](int half) {
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) {   // 16 keys: 8 TMEM columns of P, 16 rows of V
            const int kk = half * 4 + k4;
            if (kk * 16 < used) umma_bf16_ts(tO, tS + 8 * kk, dv + kk * (2048 >> 4), idesc_o, (t > 0 || kk > 0) ? 1u : 0u);
          }
        };
        if (u >= 0 && !(ok = wait(FULL + sv, pvp, 73))) break;
        if (pv) {
          if (!(ok = wait(PF + 2 * X, t & 1, 74))) break;
          tc_fence_after();
          if (lead) half_pv(0);
        } else if (u >= 0) {
          if (lead) mbar_arrive(ubar(EMPTY + sv));
        }
        if (u + 1 < nt && !(ok = wait(FULL + sk, pk, 71))) break;
        if (pv && !(ok = wait(PF + 2 * X + 1, t & 1, 74))) break;
        tc_fence_after();
        if (lead) {
          if (pv) half_pv(1);
          if (sc) {   // S(u + 1) overwrites P(u), which the product before it has read
            const uint64_t dk = desc_k + static_cast<uint32_t>(sk * (TILE >> 4));
            if (pv) {
              umma_commit(ubar(PVD + X));
              umma_commit(ubar(EMPTY + sv));
            }
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t o = ((kk >> 2) * (kTcKeys * 128) + (kk & 3) * 32) >> 4;
              umma_bf16(tS, desc_q + o, dk + o, idesc_s, kk > 0);
            }
            umma_commit(ubar(SF + X));
          }
          if (sc) {
            umma_commit(ubar(EMPTY + sk));
          } else {
            if (pv) {
              umma_commit(ubar(PVD + X));
              umma_commit(ubar(EMPTY + sv));
            }
            if (u + 1 < nt) mbar_arrive(ubar(EMPTY + sk));
          }
        }
        __syncwarp();
        sv = sk + 1 == NST ? 0 : sk + 1;
        pvp = sk + 1 == NST ? pk ^ 1 : pk;
        sk = sv + 1 == NST ? 0 : sv + 1;
        pk = sv + 1 == NST ? pvp ^ 1 : pvp;
      }
      if (lead) {
        umma_commit(ubar(DR + X));
        int zero = 0;
        WaitCtx dw = wc;
        dw.abort_flag = &zero;
        tc_wait(ubar(DR + X), 0, dw, 75);
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kTcSoftmaxRegs));
    // ------------- softmax: warpgroup X, thread = row
    const int X = warp >> 2;
    if (X < it.n_act) {
      {   // Q: the warp's 32 rows (those past the sequence's as zeros)
        constexpr int CPR = D / 8, RPI = 32 / CPR;
        const int c = lane % CPR;
        const uint32_t dst = smem_addr(sQ + X * TILE) + (c >> 3) * (kTcKeys * 128);
#pragma unroll
        for (int k = 0; k < 32 / RPI; ++k) {
          const int rl = (warp & 3) * 32 + k * RPI + lane / CPR, rr = it.r0 + X * 128 + rl;
          const bool ok = rr < it.rows;
          const int t = a.group_div.div(ok ? rr : 0), h = it.kh * a.group + (ok ? rr : 0) - t * a.group;
          cp_async16(dst + rl * 128 + (((c & 7) ^ (rl & 7)) << 4),
                     static_cast<const uint16_t*>(a.q.p) + (it.q.row0 + t) * a.q.row + h * a.q.head + c * 8, ok);
        }
        cp_async_commit();
        cp_async_wait<0>();
        fence_proxy_async_smem();
        mbar_arrive(bar(QF));
      }
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
      const TcTiles tiles = tc_tiles(a, it, X);
      const TcTiles other = tc_tiles(a, it, X ^ 1);
      const int turns = it.n_act == 2 ? min(tiles.end - tiles.first, other.end - other.first) : 0;
      const uint32_t turn_mine = bar(TK + 4 * X + (warp & 3)), turn_other = bar(TK + 4 * (X ^ 1) + (warp & 3));
      float m_used = -INFINITY, l_run = 0.f;
      int t = 0;
      bool ok = true;
      for (int u = tiles.first; u < tiles.end; ++u) {
        const int xt = it.x0 + u * kTcKeys;
        bool w = tc_wait(bar(SF + X), t & 1, wc, 76);
        if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        tc_fence_after();
        float sv[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t rr[32];
          tmem_ld32(tS + 32 * c, rr);
#pragma unroll
          for (int e = 0; e < 32; ++e) sv[32 * c + e] = __uint_as_float(rr[e]);
        }
        tmem_ld_wait();
        if constexpr (MOD) {
          const int gap = it.kl.cut - xt;   // the list's gap, if the tile holds it: slots lie `shift` further behind it
          const int near = i - xt, far = near - it.kl.shift;
          const bool split = gap > 0 && gap < kTcKeys;
          const int base = gap <= 0 ? far : near;
          if (sm.cap2 > 0.f || !sm.bias) scale_scores(sm, sv);
          if (sm.bias && !split && base >= kTcKeys - 1) {
            // All keys before the row: - slope (base - e) is linear in e, two keys at a time.
            const float b0 = -slope2 * static_cast<float>(base);
            const uint64_t sl = f2_pack(slope2, slope2), bb = f2_pack(b0, b0);
            const float one = sm.cap2 > 0.f ? 1.f : sm.sl2;
            const uint64_t k2 = f2_pack(one, one);
#pragma unroll
            for (int e = 0; e < 128; e += 2) {
              const uint64_t bias = ffma2(f2_pack(e, e + 1), sl, bb);
              f2_unpack(ffma2(f2_pack(sv[e], sv[e + 1]), k2, bias), sv[e], sv[e + 1]);
            }
          } else if (sm.bias) {
            const float one = sm.cap2 > 0.f ? 1.f : sm.sl2;
            const float fn = static_cast<float>(split ? near : base), ff = static_cast<float>(split ? far : base);
#pragma unroll
            for (int e = 0; e < 128; ++e)
              sv[e] = fmaf(-slope2, fabsf((e >= gap ? ff : fn) - e), sv[e] * one);
          }
        }
        if (!((xt >= all_lo && xt + kTcKeys - 1 <= all_hi) || xt + kTcKeys - 1 < pre)) {
          const int lo = xlo - xt, hi = xhi - xt, pr = pre - xt;
          if (pr <= 0 && xt >= all_lo) {   // only the causal edge (or the list's end)
#pragma unroll
            for (int e = 0; e < 128; ++e) sv[e] = e <= hi ? sv[e] : -INFINITY;
          } else {
#pragma unroll
            for (int e = 0; e < 128; ++e) sv[e] = ((e >= lo && e <= hi) || e < pr) ? sv[e] : -INFINITY;
          }
        }
        float mx[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
        for (int e = 4; e < 124; e += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k) mx[k] = fmax3(mx[k], sv[e + 2 * k], sv[e + 2 * k + 1]);
        mx[0] = fmax3(mx[0], sv[124], sv[125]);
        mx[1] = fmax3(mx[1], sv[126], sv[127]);
        const float sc = MOD ? 1.f : sm.sl2;
        const float m_tile = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]) * sc;
        float corr = 1.f;
        if (m_tile > m_used + kTcSlack) {
          if (m_used != -INFINITY) corr = ex2_approx(m_used - m_tile);
          m_used = m_tile;
        }
        l_run *= corr;
        if (t > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
          w = tc_wait(bar(PVD + X), (t - 1) & 1, wc, 77);
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
        const uint64_t sc2 = f2_pack(sc, sc), mu2 = f2_pack(-mu, -mu);
        uint64_t rs[2] = {0, 0};   // two packed sums
        auto args = [&](int c) {
#pragma unroll
          for (int e = c * 32; e < c * 32 + 32; e += 2)
            f2_unpack(ffma2(f2_pack(sv[e], sv[e + 1]), sc2, mu2), sv[e], sv[e + 1]);
        };
        args(0);
        if (t < turns) {
          w = tc_wait(turn_mine, (t & 1) ^ (X ^ 1), wc, 82);
          if (!__all_sync(0xffffffffu, w)) { ok = false; break; }
        }
        // Quarters of 32 keys: one quarter's sums and packing fill the gaps between the next one's exponentials (the
        // ordered asm keeps each store behind them).
        auto exps = [&](int c) {
#pragma unroll
          for (int e = 0; e < 32; ++e) sv[c * 32 + e] = ex2_ordered(sv[c * 32 + e]);
        };
        auto pack = [&](int c) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            rs[e & 1] = fadd2(rs[e & 1], f2_pack(sv[c * 32 + 2 * e], sv[c * 32 + 2 * e + 1]));
            p[e] = pack_bf16x2(sv[c * 32 + 2 * e], sv[c * 32 + 2 * e + 1]);
          }
          tmem_st16(tS + 16 * c, p);
        };
        auto hand_over = [&](int half) {
          tmem_st_wait();
          tc_fence_before();
          mbar_arrive(bar(PF + 2 * X + half));
        };
        args(1); exps(0);
        args(2); exps(1); args(3);
        pack(0);
        exps(2);
        pack(1);
        hand_over(0);
        exps(3);
        if (t < turns) {   // all exponentials are issued: the other warp's turn
          __syncwarp();
          if (lane == 0) mbar_arrive(turn_other);
        }
        pack(2);
        pack(3);
        hand_over(1);
        float r0, r1;
        f2_unpack(fadd2(rs[0], rs[1]), r0, r1);
        l_run += r0 + r1;
        ++t;
      }
      if (ok && t > 0) {
        const bool w = tc_wait(bar(PVD + X), (t - 1) & 1, wc, 78);
        ok = __all_sync(0xffffffffu, w);
        tc_fence_after();
      }
      if (ok) {
        // Rows go out through 4 KB of the warpgroup's Q tile (its products have read it) so that eight lanes write 128
        // bytes of a row: chunk g of row r at r * 128 + ((g ^ (r & 7)) << 4).
        const bool empty = l_run == 0.f;   // a NaN score leaves a NaN sum
        const float inv = empty ? 0.f : 1.f / l_run;
        const uint32_t stage = smem_addr(sQ + X * TILE) + (warp & 3) * 4096;
        const int rl = lane >> 3, g = lane & 7;
        int64_t at[8];   // of rows 4 k + rl: the row of the partial results, or the element of o; -1 past the sequence
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int ro = it.r0 + X * 128 + (warp & 3) * 32 + 4 * k + rl;
          const int to = a.group_div.div(min(ro, it.rows - 1)), ho = it.kh * a.group + min(ro, it.rows - 1) - to * a.group;
          const int64_t tok = it.q.row0 + to;
          at[k] = ro >= it.rows ? -1
                  : a.parts > 1 ? (static_cast<int64_t>(it.sp) * a.ch.n_tokens + tok) * a.n_q_heads + ho
                                : tok * a.o_row + ho * a.o_head;
        }
        constexpr int kWide = D / 32;   // 32-column chunks
        const int words = a.parts > 1 ? 1 : 2;   // columns of a staged word
        for (int c = 0; c < kWide; c += words) {
          uint32_t w[32];
          if (words == 1) {
            tc_output(tO + 32 * c, t > 0, w);
          } else {
            uint32_t o[32];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              tc_output(tO + 32 * (c + half), t > 0, o);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                w[16 * half + e] =
                    empty ? 0u : pack_bf16x2(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
            }
          }
#pragma unroll
          for (int k = 0; k < 8; ++k)
            st_shared_v4(stage + lane * 128 + ((k ^ (lane & 7)) << 4), w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
          __syncwarp();
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int rr = 4 * k + rl;
            const uint4 y = ld_shared_v4(stage + rr * 128 + ((g ^ (rr & 7)) << 4));
            if (at[k] < 0) continue;
            if (words == 1)
              st_global_v4(a.part_o + at[k] * D + c * 32 + g * 4, y.x, y.y, y.z, y.w);
            else
              st_global_v4(static_cast<uint16_t*>(a.o) + at[k] + c * 32 + g * 8, y.x, y.y, y.z, y.w);
          }
          __syncwarp();
        }
        if (r < it.rows) {
          const int64_t tok = it.q.row0 + tt;
          if (a.parts > 1)
            a.part_ml[(static_cast<int64_t>(it.sp) * a.ch.n_tokens + tok) * a.n_q_heads + h] = make_float2(m_used, l_run);
          else if (a.lse)
            a.lse[tok * a.n_q_heads + h] = empty ? -INFINITY : (m_used + log2f(l_run)) * kLn2;
        }
      }
      tc_fence_before();
    }
  }
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool MOD>
cudaError_t launch_tc(const Launch& L, const PagedAttnArgs& a, int blocks) {
  const uint64_t rows = static_cast<uint64_t>(a.c.n_pages) * a.c.n_heads * a.c.page.d;
  CUtensorMap tk, tv;
  const uint64_t dims[2] = {D, rows}, strides[1] = {D * 2};
  // Runs: the largest power of two that divides the page size, up to a tile.  Below 8 rows a TMA copy each costs more
  // than copying the rows with cp.async (2 chunks of 1000 tokens over 4000, 32/8 heads of 128: pages of 16 to 128 rows
  // 135 to 137 us, of 8 rows 154, of 8 rows by cp.async 184, of 50 rows by cp.async 172).
  int run = 1;
  while (run < kTcKeys && a.c.page.d % (2 * run) == 0) run *= 2;
  if (run < 8) run = 1;
  const uint32_t box[2] = {64, static_cast<uint32_t>(run)};
  if (!encode_tmap(&tk, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.k, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B) ||
      !encode_tmap(&tv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, a.v, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B))
    return cudaErrorInvalidValue;
  const unsigned grid = static_cast<unsigned>(static_cast<int64_t>(blocks) * a.c.n_seqs * a.c.n_heads * a.splits);
  return launch_kernel(paged_attn_tc_kernel<D, MOD>, dim3(grid), dim3(kTcThreads), TcCfg<D>::kSmem, L.stream, tk, tv, a,
                       blocks, run);
}

}  // namespace

cudaError_t launch_paged_attn_tc(const Launch& L, const PagedAttnArgs& a) {
  const int blocks = static_cast<int>((static_cast<int64_t>(a.ch.max_q) * a.group + 255) / 256);
  const bool mod = a.cap > 0.f || a.slopes != nullptr;
  if (a.head_dim == 128) return mod ? launch_tc<128, true>(L, a, blocks) : launch_tc<128, false>(L, a, blocks);
  return mod ? launch_tc<64, true>(L, a, blocks) : launch_tc<64, false>(L, a, blocks);
}

}  // namespace vx
