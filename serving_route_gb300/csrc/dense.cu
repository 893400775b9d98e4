// dense.cu -- the dense products beside the MoE layer: x W^T in the layer's FP8 format
// (Fp8Linear) and the products of a gated feed-forward block and of its gradients
// (GatedMlp).
#include <cuda_fp16.h>

#include "common.cuh"
#include "dense.h"

namespace mm {

// ------------------------------------------------------------------------- rows to FP8
// One warp per 128 columns of a row: amax, the least power of two that brings it to at
// most 448, codes.  x * 2^-e is exact (but below E4M3's range, where it rounds once).
__global__ void __launch_bounds__(256) quantize_rows_kernel(const uint16_t* x, int64_t ld, int64_t blocks, int kb,
                                                            uint8_t* q, uint8_t* s) {
  const int lane = threadIdx.x & 31;
  for (int64_t b = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); b < blocks; b += (int64_t)gridDim.x * 8) {
    const int64_t t = b / kb;
    const int c = (int)(b - t * kb);
    const uint2 v = *reinterpret_cast<const uint2*>(x + t * ld + c * 128 + lane * 4);
    const float f[4] = {bf16_bits_to_float(v.x & 0xFFFFu), bf16_bits_to_float(v.x >> 16),
                        bf16_bits_to_float(v.y & 0xFFFFu), bf16_bits_to_float(v.y >> 16)};
    float m = fmaxf(fmaxf(fabsf(f[0]), fabsf(f[1])), fmaxf(fabsf(f[2]), fabsf(f[3])));
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
    const int e = pow2_scale_exp(m);
    const float inv = pow2_neg(e);
    *reinterpret_cast<uint32_t*>(q + b * 128 + lane * 4) =
        e4m3x4(f[0] * inv, f[1] * inv, f[2] * inv, f[3] * inv);
    if (lane == 0) s[b] = (uint8_t)(e + 127);
  }
}

cudaError_t dense_quantize_rows(const uint16_t* x, int64_t ld, int64_t T, int cols, uint8_t* q, uint8_t* s,
                                cudaStream_t stream) {
  const int64_t blocks = T * (cols / 128), ctas = (blocks + 7) / 8;
  quantize_rows_kernel<<<(int)(ctas < 152 * 8 ? ctas : 152 * 8), 256, 0, stream>>>(x, ld, blocks, cols / 128, q, s);
  return cudaGetLastError();
}

__global__ void scales_to_e8m0_kernel(const float* s, int64_t n, uint8_t* out, uint32_t* status) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const uint32_t b = __float_as_uint(s[i]);
    const bool ok = b == 0x00400000u || ((b & 0x807FFFFFu) == 0u && b != 0u && b < 0x7F800000u);
    if (!ok) record_status(status, MOE_DEV_BAD_SCALE);
    out[i] = (uint8_t)(b >> 23);  // 2^-127, subnormal, is byte 0
  }
}

cudaError_t dense_scales_to_e8m0(const float* s, int64_t n, uint8_t* out, uint32_t* status, cudaStream_t stream) {
  scales_to_e8m0_kernel<<<(int)((n + 255) / 256 < 1024 ? (n + 255) / 256 : 1024), 256, 0, stream>>>(s, n, out, status);
  return cudaGetLastError();
}

// ------------------------------------------------------------------------- values
__device__ __forceinline__ float half_bits_to_float(uint32_t b) {
  return __half2float(__ushort_as_half((unsigned short)b));
}

__device__ __forceinline__ float load16(const void* p, int64_t i, DenseType t) {
  const uint32_t b = reinterpret_cast<const uint16_t*>(p)[i];
  return t == kBF16 ? bf16_bits_to_float(b) : half_bits_to_float(b);
}

__device__ __forceinline__ uint16_t bits16(float v, DenseType t) {
  return t == kBF16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
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

// ------------------------------------------------------------------------- products
// The simple form: 64 x 64 outputs per block through shared memory, 4 x 4 per thread.
constexpr int kSimpleK = 16;

template <bool GATE>
__global__ void __launch_bounds__(256) dense_simple_kernel(const DenseGemm g) {
  __shared__ float as[kSimpleK][65], bs[GATE ? 2 : 1][kSimpleK][65];
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * 64, n0 = (int64_t)blockIdx.x * 64;
  const int KB = g.K / 128;
  auto value = [&](const DenseOperand& o, int64_t r, int k) -> float {
    if (g.type != kE4M3) return load16(o.p, o.mn ? k * o.ld + r : r * o.ld + k, g.type);
    const uint8_t c = reinterpret_cast<const uint8_t*>(o.p)[r * o.ld + k];
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
  };
  float d[GATE ? 2 : 1][4][4] = {}, sum[4][4] = {};
  for (int k0 = 0; k0 < g.K; k0 += kSimpleK) {
    for (int i = threadIdx.x; i < 64 * kSimpleK; i += 256) {
      const int r = i / kSimpleK, k = k0 + i % kSimpleK;
      as[i % kSimpleK][r] = m0 + r < g.M && k < g.K ? value(g.a, m0 + r, k) : 0.f;
#pragma unroll
      for (int h = 0; h < (GATE ? 2 : 1); ++h)
        bs[h][i % kSimpleK][r] = n0 + r < g.N && k < g.K ? value(g.b, n0 + r + (int64_t)h * g.N, k) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < kSimpleK; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int h = 0; h < (GATE ? 2 : 1); ++h)
            d[h][i][j] = fmaf(as[k][ty + 16 * i], bs[h][k][tx + 16 * j], d[h][i][j]);
    __syncthreads();
    if (!GATE && g.type == kE4M3 && (k0 + kSimpleK) % 128 == 0)  // a K block's sums, scaled
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) {
          const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
          if (m < g.M && n < g.N)
            sum[i][j] += scalbnf(d[0][i][j], (int)g.sa[m * KB + k0 / 128] + g.sb[n / 128 * KB + k0 / 128] - 254);
          d[0][i][j] = 0.f;
        }
  }
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      if (!GATE && g.type == kE4M3) d[0][i][j] = sum[i][j];
      const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= g.M || n >= g.N) continue;
      const int64_t at = m * g.ld_out + n, gate = m * 2 * g.N + n, up = gate + g.N;
      if (g.epi == kEpiStore) {
        float* f = reinterpret_cast<float*>(g.out) + at;
        if (g.out_f32)
          *f = g.accumulate ? *f + d[0][i][j] : d[0][i][j];
        else
          reinterpret_cast<uint16_t*>(g.out)[at] = bits16(d[0][i][j], g.type == kFP16 ? kFP16 : kBF16);
        continue;
      }
      float a, da;
      if (GATE) {
        const float gv = d[0][i][j], uv = d[GATE ? 1 : 0][i][j];
        activate(g.act, gv, a, da);
        reinterpret_cast<uint16_t*>(g.out)[at] = bits16(a * uv, g.type);
        if (g.saved && g.saved_f32) {
          reinterpret_cast<float*>(g.saved)[gate] = gv;
          reinterpret_cast<float*>(g.saved)[up] = uv;
        } else if (g.saved) {
          reinterpret_cast<uint16_t*>(g.saved)[gate] = bits16(gv, g.type);
          reinterpret_cast<uint16_t*>(g.saved)[up] = bits16(uv, g.type);
        }
      } else {
        const float gv = g.saved_f32 ? reinterpret_cast<const float*>(g.saved)[gate] : load16(g.saved, gate, g.type);
        const float uv = g.saved_f32 ? reinterpret_cast<const float*>(g.saved)[up] : load16(g.saved, up, g.type);
        activate(g.act, gv, a, da);
        const float dh = d[0][i][j];
        reinterpret_cast<uint16_t*>(g.dgu)[gate] = bits16(dh * uv * da, g.type);
        reinterpret_cast<uint16_t*>(g.dgu)[up] = bits16(dh * a, g.type);
        if (g.out) reinterpret_cast<uint16_t*>(g.out)[at] = bits16(a * uv, g.type);
      }
    }
}

cudaError_t dense_gemm(const DenseGemm& g, cudaStream_t s) {
  const dim3 grid((g.N + 63) / 64, (g.M + 63) / 64);
  if (g.epi == kEpiGate)
    dense_simple_kernel<true><<<grid, 256, 0, s>>>(g);
  else
    dense_simple_kernel<false><<<grid, 256, 0, s>>>(g);
  return cudaGetLastError();
}

}  // namespace mm
