// dense.cuh -- what the kernels of the dense products share: values and activations,
// operand descriptors, scale words.
#pragma once

#include <type_traits>

#include <cuda_fp16.h>

#include "common.cuh"
#include "dense.h"

namespace mm {

// ------------------------------------------------------------------------- values
__device__ __forceinline__ float half_bits_to_float(uint32_t b) {
  return __half2float(__ushort_as_half((unsigned short)b));
}

__device__ __forceinline__ uint16_t bits16(float v, DenseType t) {
  return t == kFP16 ? __half_as_ushort(__float2half_rn(v)) : __bfloat16_as_ushort(__float2bfloat16_rn(v));
}

// Pairs of floats in one instruction.
struct F2 {
  uint64_t v;
};
__device__ __forceinline__ F2 f2(float a, float b) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void parts(F2 x, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(x.v)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal_fast(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// a = act(g) and d = act'(g) of two values.  With s the logistic function of z
//   silu               z = g,                             dz = 1
//   gelu (tanh form)   z = 2 sqrt(2/pi) (g + 0.044715 g^3), as tanh(z / 2) = 2 s - 1
//   a = g s,  d = s + s (1 - s) g dz  (silu: s (1 + (1 - s) g)).
// Far out s is 0 or 1, and g^2 is held at 400, where it has long been so, for dz to stay
// finite; g dz (87 g) need not be, so s (1 - s), 0 out there, comes before it.  s is good to
// about 2^-22 of itself by the hardware's exponential and reciprocal, and to |z| 2^-24 more by
// the rounding of the exponent, where s (1 - s) |z| is below 0.3.  (With these in pairs, not
// one by one with the special cases of division, the gradient's epilogue of a 256 x 256 tile
// has half the instructions.)
template <DenseAct ACT>
__device__ __forceinline__ void activate2(F2 g, F2& a, F2& d) {
  const F2 one = f2(1.f, 1.f);
  F2 z = g, dz = one;
  if constexpr (ACT == kGeluTanh) {
    float x, y;
    parts(mul2(g, g), x, y);
    const F2 gg = f2(fminf(x, 400.f), fminf(y, 400.f)), c = f2(1.5957691216f, 1.5957691216f);
    z = mul2(g, fma2(gg, f2(0.0713548163f, 0.0713548163f), c));
    dz = fma2(gg, f2(0.2140644488f, 0.2140644488f), c);
  }
  float x, y;
  parts(mul2(z, f2(-1.4426950409f, -1.4426950409f)), x, y);
  parts(add2(f2(exp2_fast(x), exp2_fast(y)), one), x, y);
  const F2 s = f2(reciprocal_fast(x), reciprocal_fast(y));
  a = mul2(g, s);
  const F2 q = fma2(s, f2(-1.f, -1.f), one);
  d = ACT == kSilu ? mul2(s, fma2(g, q, one)) : fma2(mul2(mul2(s, q), g), dz, s);
}

// u <- act(g) u
template <int N>
__device__ __forceinline__ void gate_values(DenseAct act, const float (&g)[N], float (&u)[N]) {
  auto all = [&](auto A) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      F2 a, d;
      activate2<decltype(A)::value>(f2(g[k], g[k + 1]), a, d);
      parts(mul2(a, f2(u[k], u[k + 1])), u[k], u[k + 1]);
    }
  };
  if (act == kSilu)
    all(std::integral_constant<DenseAct, kSilu>{});
  else
    all(std::integral_constant<DenseAct, kGeluTanh>{});
}

// g <- dh u act'(g), u <- dh act(g), dh <- act(g) u (h)
template <int N>
__device__ __forceinline__ void gradient_values(DenseAct act, float (&dh)[N], float (&g)[N], float (&u)[N]) {
  auto all = [&](auto A) {
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      F2 a, d;
      const F2 v = f2(dh[k], dh[k + 1]), w = f2(u[k], u[k + 1]);
      activate2<decltype(A)::value>(f2(g[k], g[k + 1]), a, d);
      parts(mul2(mul2(v, w), d), g[k], g[k + 1]);
      parts(mul2(v, a), u[k], u[k + 1]);
      parts(mul2(a, w), dh[k], dh[k + 1]);
    }
  };
  if (act == kSilu)
    all(std::integral_constant<DenseAct, kSilu>{});
  else
    all(std::integral_constant<DenseAct, kGeluTanh>{});
}

// What a block of 128 values with the largest magnitude `amax` is multiplied by before its
// rounding to E4M3 with the scale 2^e: 2^-e, or NaN where the block holds an infinity.  E4M3
// has none, and the conversion's 448 would pass for a number; so all of the block's codes are
// NaN, and with them the row of the product, as they are from a NaN.
__device__ __forceinline__ float block_factor(float amax, int e) {
  return __float_as_uint(amax) == 0x7F800000u ? __uint_as_float(0x7FFFFFFFu) : pow2_neg(e);
}

struct DenseArgs {
  int M, N, K;
  DenseAct act;
  DenseType type;
  const uint8_t *sa, *sb;
  int sa_pitch, sb_pitch;
  const uint16_t* x;  // the tokens in BF16 (quantised on the way), rows ldx elements apart
  int64_t ldx;
  void* out;
  int64_t ld_out;
  bool out_f32, vec;  // vec: columns in pieces of 8, rows on 16-byte boundaries (both of E4M3 products alone)
  void* saved;
  bool saved_f32;
  void* dgu;
  uint32_t* status;
  uint64_t wait_ns;  // limit of every wait
  bool withhold;     // a test: one copy is never made, so that a wait runs out
};

// A product on clusters that share K (dense_split.cu).
struct DenseSplit {
  int NT, tt, rt;        // tokens of a tile, tiles of them, tiles of weight rows
  int split, stages;     // CTAs that share a tile's K, ring places
  uint32_t tmem_cols, smem;
  bool early;            // the weights' first copies need not wait for the kernel before
  bool alone;            // at most one CTA per SM
  double us;             // its time by the model below
};
constexpr int kSpMaxTokens = 128;
constexpr int kSpMaxSmem = 104 * 1024;   // two CTAs, with what each has besides, in 228 KB
constexpr int kSpAloneSmem = 117248;     // two do not fit

cudaError_t dense_split_set_attributes();
DenseSplit dense_split_plan(const DenseGemm& g, int sms);
cudaError_t dense_split_launch(const CUtensorMap& a, const CUtensorMap& b, const DenseGemm& g, const DenseArgs& d,
                               const DenseSplit& p, cudaStream_t s);

// One lane of a converged warp.  The loops that issue copies and MMAs are run by whole warps
// and their instructions by the elected lane, so that descriptors stay in uniform
// registers: from one lane's branch every MMA took 76 clocks to issue.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xFFFFFFFF;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0u;
}

// Bounded wait of a whole warp: all of its lanes go on, or none.  (All of them poll: with one,
// whose branch the others wait for, short kernels took 5 to 8% longer.)
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* status,
                                          uint64_t limit_ns) {
  return __all_sync(0xFFFFFFFFu, mbar_wait<CLUSTER>(bar, parity, abort, status, limit_ns));
}

// Shared-memory descriptor of an MN-major operand with the 128-byte swizzle: 64 elements
// (128 bytes) per K row, 8 K rows 1024 bytes apart from the next 8 (stride offset), the
// next 64 elements one box of 64 K rows further (leading offset).
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);
  d |= (uint64_t)(8192u >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Instruction descriptor of kind::f16: FP32 sums (bits 4-5), A and B FP16 (0) or BF16 (1) at
// bits 7-9 and 10-12, MN-major operands bits 15 and 16, N >> 3, M >> 4.
__host__ __device__ constexpr uint32_t idesc_16(int M, int N, bool bf16, bool a_mn, bool b_mn) {
  return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)a_mn << 15) |
         ((uint32_t)b_mn << 16) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

__device__ __forceinline__ uint32_t pack16(float lo, float hi, DenseType t) {
  if (t != kFP16) return pack_bf16x2(lo, hi);
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

__device__ __forceinline__ void unpack16(uint32_t v, DenseType t, float& lo, float& hi) {
  lo = t == kFP16 ? half_bits_to_float(v & 0xFFFFu) : bf16_bits_to_float(v & 0xFFFFu);
  hi = t == kFP16 ? half_bits_to_float(v >> 16) : bf16_bits_to_float(v >> 16);
}

// Four K blocks' scale bytes of four rows, r, r + 32, r + 64, r + 96 (rows `pitch` bytes apart;
// past the last of `rows` rows the last one's, past the last block anything).  Aligned words
// only, all asked for before one is used: where rows begin within words, two for each row, of
// which the second is the first again unless it holds a byte of the row.  (Not
// by the read-only path: the kernel before may write them while this one has begun.)
__device__ __forceinline__ void scale_words(const uint8_t* s, int64_t r, int64_t rows, int pitch, int KB, int q,
                                            uint32_t (&w)[4]) {
  const uint8_t* p[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) p[i] = s + min(r + 32 * i, rows - 1) * pitch + 4 * q;
  if (((uintptr_t)s & 3) == 0 && (pitch & 3) == 0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const uint32_t*>(p[i]);
    return;
  }
  uint32_t off[4], lo[4], hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    off[i] = (uint32_t)(uintptr_t)p[i] & 3u;
    const uint32_t* a = reinterpret_cast<const uint32_t*>(p[i] - off[i]);
    lo[i] = *a;
    hi[i] = a[off[i] && 4 * q + 4 - (int)off[i] < KB ? 1 : 0];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = __funnelshift_r(lo[i], hi[i], 8 * off[i]);
}

// The same of one block of the matrix (whole words).
__device__ __forceinline__ uint32_t block_word(const uint8_t* s, int64_t block, int pitch, int q) {
  return __ldg(reinterpret_cast<const uint32_t*>(s + block * pitch) + q);
}

}  // namespace mm
