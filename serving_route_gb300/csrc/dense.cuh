// dense.cuh -- what the kernels of the dense products share: values and activations,
// operand descriptors, scale words.
#pragma once

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

// act(g) and act'(g).  silu = g s(g) with s the logistic function, s + silu (1 - s);
// gelu (tanh form) = g s(2z), z = sqrt(2/pi) (g + 0.044715 g^3), as tanh z = 2 s(2z) - 1.
__device__ __forceinline__ void activate(DenseAct act, float g, float& a, float& d) {
  const float z = act == kSilu ? g : g * (1.5957691216f + 0.0713548163f * g * g);
  const float dz = act == kSilu ? 1.0f : 1.5957691216f + 0.2140644488f * g * g;
  const float s = __fdividef(1.0f, 1.0f + __expf(-z));
  const float t = s * (1.0f - s);
  a = g * s;
  d = s + (t == 0.f ? 0.f : g * t * dz);  // (far out dz may be infinite)
}

struct DenseArgs {
  int M, N, K;
  int units, mt, nt;       // tiles of 256 rows, of the columns (kEpiGate: 128 h columns)
  DenseEpi epi;
  DenseAct act;
  DenseType type;
  const uint8_t *sa, *sb;
  void* out;
  int64_t ld_out;
  bool out_f32, accumulate, vec;  // vec: columns in pieces of 8, rows on 16-byte boundaries
  void* saved;
  bool saved_f32;
  void* dgu;
  uint32_t* status;
};

// A product on clusters that share K (dense_split.cu).
struct DenseSplit {
  int NT, tt, rt;        // tokens of a tile, tiles of them, tiles of weight rows
  int split, stages;     // CTAs that share a tile's K, ring places
  uint32_t tmem_cols, smem;
  bool early;            // the weights' first copies need not wait for the kernel before
};
constexpr int kSpMaxSmem = 230000;

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

__device__ __forceinline__ bool warp_test(uint32_t bar, uint32_t parity) {
  return __all_sync(0xFFFFFFFFu, mbar_test_wait(bar, parity));
}

// Bounded wait of a whole warp: all of its lanes go on, or none.
template <bool CLUSTER = false>
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* status) {
  return __all_sync(0xFFFFFFFFu, mbar_wait<CLUSTER>(bar, parity, abort, status));
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

// Four K blocks' scale bytes of one row (0 past the last block).
__device__ __forceinline__ uint32_t scale_word(const uint8_t* s, int64_t row, int KB, int q) {
  const uint8_t* p = s + row * KB + 4 * q;
  if ((KB & 3) == 0 && ((uintptr_t)s & 3) == 0) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t w = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    if (4 * q + j < KB) w |= (uint32_t)p[j] << (8 * j);
  return w;
}

}  // namespace mm
