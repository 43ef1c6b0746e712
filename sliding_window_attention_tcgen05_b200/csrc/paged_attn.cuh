// paged_attn.cuh -- what the attention kernels over the paged cache share: the
// list of keys a block of queries sees, asynchronous row copies, the score
// transform.
//
// A block of queries (tokens t_first .. t_last of one sequence) sees the slots
// [0, pre) and [lo, hi).  They are walked as one list x = 0 .. total - 1: slot
// j = x for x < cut, x + shift behind it (shift 0 when the two ranges touch).
// In the list's coordinates token i sees x < pre or xlo(i) <= x <= xhi(i).
// With `align` above 1 (a power of two that divides the page size) every
// aligned run of the list is an aligned run of slots, so the list also holds
// the slots between pre and cut and up to align - 1 before lo: wanted() tells
// them apart, and no token sees them.
#pragma once

#include "vx_paged.h"

namespace vx {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kNoWindow = 1 << 30;

struct KeyList {
  int pre, lo, cut, shift, total;
};

__device__ __forceinline__ KeyList key_list(int i_first, int i_last, int window, int prefix, int kv, int align = 1) {
  KeyList k;
  k.lo = min(max(0, i_first - window + 1), kv);
  const int hi = min(i_last + 1, kv), lo = k.lo & -align;
  k.pre = min(max(prefix, 0), kv);
  k.cut = (k.pre + align - 1) & -align;
  if (k.cut >= lo) {
    k.shift = 0;
    k.total = max(hi, k.pre);
  } else {
    k.shift = lo - k.cut;
    k.total = k.cut + max(hi - lo, 0);
  }
  return k;
}
__device__ __forceinline__ int key_slot(const KeyList& k, int x) { return x + (x >= k.cut ? k.shift : 0); }
__device__ __forceinline__ bool wanted(const KeyList& k, int j) { return j < k.pre || j >= k.lo; }   // of x < total

// 16 bytes global -> shared, or zeros when !valid (src must be readable all the same: it is not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(addr));
}
__device__ __forceinline__ void ldsm_x4_t(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3) : "r"(addr));
}
// D = A(16x16, row) * B(16x8, col) + D, bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_bf16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Packed fp32 pairs (each half rounds like the scalar operation).
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t r, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r));
}
__device__ __forceinline__ uint64_t ffma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t fadd2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fmul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Scores to the exponent's base-2 units.  Without cap and slopes that is one
// multiplication by scale * log2(e).  A cap in bf16: where all of a thread's
// scores are at most half the cap, as they are nearly always, cap * tanh(z) =
// score * P(z^2) with the minimax polynomial P of tanh(z) / z on z^2 <= 1/4
// (relative error 2.8e-8), on the FMA pipe alone; else cap * (1 - 2 / (e^{2z} +
// 1)), from one exponential and half a reciprocal (absolute error about cap *
// 2^-22, where the hardware's own tanh would leave cap * 2^-11).  fp32: tanhf,
// whose error is relative to the score too.
struct ScoreMod {
  float sl2;       // scale * log2 e
  float cap2;      // cap * log2 e, 0 = no cap
  float z;         // scale / cap
  float two_z;     // 2 scale / cap * log2 e
  bool bias;       // slopes
};
__device__ __forceinline__ ScoreMod score_mod(const PagedAttnArgs& a) {
  ScoreMod m;
  m.sl2 = a.scale * kLog2e;
  m.cap2 = a.cap * kLog2e;
  m.z = a.cap > 0.f ? a.scale / a.cap : 0.f;
  m.two_z = 2.f * m.z * kLog2e;
  m.bias = a.slopes != nullptr;
  return m;
}
// N raw scores.
template <int N>
__device__ __forceinline__ void scale_scores(const ScoreMod& m, float (&s)[N]) {
  if (m.cap2 > 0.f) {
    float big = 0.f;
#pragma unroll
    for (int e = 0; e < N; ++e) big = fmaxf(big, fabsf(s[e]));
    if (big * fabsf(m.z) <= 0.5f) {
      const uint64_t z = f2_pack(m.z, m.z), sl = f2_pack(m.sl2, m.sl2);
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const uint64_t x = f2_pack(s[e], s[e + 1]), u = fmul2(x, z), w = fmul2(u, u);
        uint64_t p = f2_pack(0.0171350073f, 0.0171350073f);
        p = ffma2(p, w, f2_pack(-0.0529860742f, -0.0529860742f));
        p = ffma2(p, w, f2_pack(0.133247793f, 0.133247793f));
        p = ffma2(p, w, f2_pack(-0.333330691f, -0.333330691f));
        p = ffma2(p, w, f2_pack(1.f, 1.f));
        f2_unpack(fmul2(fmul2(x, sl), p), s[e], s[e + 1]);
      }
    } else {   // two at a time: 1 / a and 1 / b from one reciprocal of a b (exponents up to 2^60, beyond which tanh is 1
               // to the last bit, so that the product stays finite; a NaN counts as such a one in it and stays its own
               // score's, since the mask may hide it from a row that sees its partner)
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float x = s[e] * m.two_z, y = s[e + 1] * m.two_z;
        const float a = ex2_approx(fminf(x, 60.f)) + 1.f, b = ex2_approx(fminf(y, 60.f)) + 1.f;
        const float r = -2.f * m.cap2 * rcp_approx(a * b);
        s[e] = x != x ? x : fmaf(r, b, m.cap2);
        s[e + 1] = y != y ? y : fmaf(r, a, m.cap2);
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e) s[e] *= m.sl2;
  }
}
// A score of the fp32 kernels; slope2 = slope of the head * log2 e, dist = i - j.
__device__ __forceinline__ float score2(const ScoreMod& m, float s, float slope2, int dist) {
  const float y = m.cap2 > 0.f ? m.cap2 * tanhf(s * m.z) : s * m.sl2;
  return y - slope2 * static_cast<float>(abs(dist));
}

cudaError_t launch_paged_attn_rows(const Launch& L, const PagedAttnArgs& a);
cudaError_t launch_paged_attn_tc(const Launch& L, const PagedAttnArgs& a);
cudaError_t launch_paged_attn_f32(const Launch& L, const PagedAttnArgs& a);
cudaError_t launch_paged_attn_combine(const Launch& L, const PagedAttnArgs& a, bool bf16);
cudaError_t launch_paged_attn_weights(const Launch& L, const PagedAttnArgs& a, bool bf16, int64_t max_kv);

constexpr int kMaxSplits = 64;

// Rows of a block of the fp32 kernels, for sequences of up to `rows` rows: 8 is
// the kernel for few rows (twice over the keys for 9 to 16, from L2), 32 and
// 64 the tiled one.
inline int f32_block_rows(int64_t rows) { return rows <= 16 ? 8 : rows <= 32 ? 32 : 64; }

}  // namespace vx
