// norm.cu -- residual addition, root-mean-square norm and 8-bit output in one
// pass over the rows (moe_add_rms_norm).
//
//   r = bf16(x + residual)                      (r = x without a residual)
//   y = r * rsqrt(mean(r^2) + eps) * weight     (float)
//   out: r, bf16(y), and E4M3 codes of y with the layer's scale rules
//        (per 128 or 32 columns the least power of two 2^e with amax <= 448 * 2^e,
//        or one static scale).
//
// The norm is taken of the stored (BF16) sum, so the residual stream that the
// next layer reads is exactly what was normed.  The 8-bit codes are rounded
// once, from the float y, not from its BF16 form.
//
// Bytes: 2 (x) + 2 (residual) read, 2 (r) + 2 (y) + 1 (q) written per element;
// everything between is held in registers, so the kernel is bound by HBM for
// many rows (8192 x 7168 with 1x128 codes: 77.2 us, 529 MB, 6.85 TB/s: the copy
// rate) and by one load -> reduce -> store latency chain for few (2.3 us in a
// stream of calls).
#include <cfloat>

#include "common.cuh"
#include "internal.h"

namespace mm {

struct NormArgs {
  const uint16_t* x;
  const uint16_t* res;   // nullptr: no residual
  const uint16_t* w;
  uint16_t* r_out;
  uint16_t* y;           // nullptr: no BF16 output
  uint8_t* q;            // nullptr: no 8-bit output
  uint8_t* sf;
  int64_t ldx, ldr;
  int H;
  float eps, rscale;     // rscale: 1 / static scale (per-tensor)
};

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// Sum over the block; every thread gets it.  red: 32 floats, one a warp.
__device__ __forceinline__ float block_sum(float v, float* red) {
  v = warp_sum(v);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  if (lane == 0) red[warp] = v;
  __syncthreads();
  return warp_sum(lane < nw ? red[lane] : 0.f);
}

__device__ __forceinline__ void bf16x8_to_float(const uint4 p, float (&v)[8]) {
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 float_to_bf16x8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// FMT: 0 no 8-bit output, 1 per 128 columns, 2 per 32 columns, 3 static scale.
// One block per row; thread t holds the 8-column vectors t, t + blockDim, ...
// (NV of them) in registers, so a 128-column block is one half warp.
template <int NV, int FMT>
__global__ void __launch_bounds__(1024) add_rms_norm_kernel(const NormArgs a) {
  __shared__ float red[32];
  pdl_wait();  // its launch overlaps the kernel before
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const int nvec = a.H >> 3;
  const uint4* x = reinterpret_cast<const uint4*>(a.x + row * a.ldx);
  uint4 r[NV];
  float ss = 0.f;
  if (a.res) {
    const uint4* res = reinterpret_cast<const uint4*>(a.res + row * a.ldr);
    uint4 p[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        r[i] = x[v];
        p[i] = res[v];
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) {
        float f[8], g[8];
        bf16x8_to_float(r[i], f);
        bf16x8_to_float(p[i], g);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] += g[j];
        r[i] = float_to_bf16x8(f);
        reinterpret_cast<uint4*>(a.r_out + row * a.H)[v] = r[i];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = threadIdx.x + i * blockDim.x;
      if (v < nvec) r[i] = x[v];
    }
  }
  // the weight does not wait for the sum
  uint4 w[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    if (v < nvec) {
      w[i] = reinterpret_cast<const uint4*>(a.w)[v];
      float f[8];
      bf16x8_to_float(r[i], f);
#pragma unroll
      for (int j = 0; j < 8; ++j) ss = fmaf(f[j], f[j], ss);
    }
  }
  ss = block_sum(ss, red);
  const float inv = rsqrtf(ss / (float)a.H + a.eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = threadIdx.x + i * blockDim.x;
    const bool on = v < nvec;
    float f[8];
    if (on) {
      float g[8];
      bf16x8_to_float(r[i], f);
      bf16x8_to_float(w[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) f[j] = f[j] * inv * g[j];
      if (a.y) reinterpret_cast<uint4*>(a.y + row * a.H)[v] = float_to_bf16x8(f);
    }
    if (FMT == 0) continue;
    float s = a.rscale;
    if (FMT != 3) {
      // v and the lane differ by a multiple of 32, so the columns of a scale
      // are 16 (or 4) neighbouring lanes, all on or all off
      float m = 0.f;
      if (on) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m = fmaxf(m, fabsf(f[j]));
      }
#pragma unroll
      for (int o = (FMT == 1 ? 8 : 2); o >= 1; o >>= 1)
        m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      const int e = pow2_scale_exp(m);
      s = pow2_neg(e);
      constexpr int L = FMT == 1 ? 16 : 4;
      if (on && (threadIdx.x & (L - 1)) == 0)
        a.sf[row * (a.H / (8 * L)) + v / L] = (uint8_t)(e + 127);
    }
    if (on) {
      uint2 q;
      q.x = e4m3x4(f[0] * s, f[1] * s, f[2] * s, f[3] * s);
      q.y = e4m3x4(f[4] * s, f[5] * s, f[6] * s, f[7] * s);
      reinterpret_cast<uint2*>(a.q + row * a.H)[v] = q;
    }
  }
}

// Any width, stride and alignment: element by element, the row read a second
// time (from L2) after the sum.  For widths that are no multiple of 8, above
// 16384, or pointers that are not 16-byte aligned.  A thread reads four columns
// before it stores any (the outputs may be the inputs, so the compiler would not).
template <int FMT>
__global__ void __launch_bounds__(1024) add_rms_norm_any_kernel(const NormArgs a) {
  __shared__ float red[32];
  pdl_wait();
  pdl_trigger();
  const int64_t row = blockIdx.x;
  const uint16_t* x = a.x + row * a.ldx;
  const uint16_t* res = a.res ? a.res + row * a.ldr : nullptr;
  float ss = 0.f;
  for (int c0 = threadIdx.x; c0 < a.H; c0 += 4 * blockDim.x) {
    float v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + j * blockDim.x;
      v[j] = c < a.H ? bf16_bits_to_float(x[c]) : 0.f;
      if (res && c < a.H) v[j] += bf16_bits_to_float(res[c]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + j * blockDim.x;
      if (res && c < a.H) {
        const uint32_t b = pack_bf16x2(v[j], 0.f) & 0xFFFFu;
        a.r_out[row * a.H + c] = (uint16_t)b;
        v[j] = bf16_bits_to_float(b);
      }
      ss = fmaf(v[j], v[j], ss);
    }
  }
  ss = block_sum(ss, red);  // its barrier also orders the stores of r_out before the reads below
  const float inv = rsqrtf(ss / (float)a.H + a.eps);
  const uint16_t* r = a.res ? a.r_out + row * a.H : x;
  const int lane = threadIdx.x & 31;
  for (int c0 = (threadIdx.x >> 5) * 128; c0 < a.H; c0 += (blockDim.x >> 5) * 128) {
    float f[4], m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + 32 * j + lane;
      f[j] = c < a.H ? bf16_bits_to_float(r[c]) * inv * bf16_bits_to_float(a.w[c]) : 0.f;
      m[j] = fabsf(f[j]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + 32 * j + lane;
      if (a.y && c < a.H) a.y[row * a.H + c] = (uint16_t)(pack_bf16x2(f[j], 0.f) & 0xFFFFu);
    }
    if (FMT == 0) continue;
    if (FMT == 1) m[0] = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
    float s = a.rscale;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = c0 + 32 * j + lane;
      if (FMT == 2 || (FMT == 1 && j == 0)) {
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m[j] = fmaxf(m[j], __shfl_xor_sync(0xFFFFFFFFu, m[j], o));
        const int e = pow2_scale_exp(m[j]);
        s = pow2_neg(e);
        constexpr int BL = FMT == 1 ? 128 : 32;
        if (lane == 0 && c < a.H) a.sf[row * (a.H / BL) + c / BL] = (uint8_t)(e + 127);
      }
      if (c < a.H) a.q[row * a.H + c] = (uint8_t)(e4m3x2(f[j] * s, 0.f) & 0xFFu);
    }
  }
}

template <int FMT>
static cudaError_t launch_norm(const NormArgs& a, int64_t T, bool vec, cudaStream_t s) {
  if (!vec) {
    // four columns a thread (7167 columns, one row: 3.7 us, 8192 rows: 158 us)
    const int nt = a.H >= 4096 ? 1024 : (a.H + 127) / 128 * 32;
    return launch_k(add_rms_norm_any_kernel<FMT>, dim3((unsigned)T), dim3(nt), 0, s, true, nullptr, a);
  }
  const int nvec = a.H >> 3;
  auto threads = [&](int nv) { return ((nvec + nv - 1) / nv + 31) / 32 * 32; };
  // few rows: as many threads as a block takes, so that the latency chain is
  // short (7168 columns, one row: 2.3 us, with four vectors a thread 2.6; 2048
  // columns: 1.6 and 2.3); many rows: four vectors a thread, so that several rows
  // are in flight on an SM (8192 rows: 77 us, with one vector a thread 88; between one and
  // 8192 rows neither has been measured, the border is one row an SM)
  if (T <= 152 && nvec <= 1024)
    return launch_k(add_rms_norm_kernel<1, FMT>, dim3((unsigned)T), dim3(threads(1)), 0, s, true, nullptr, a);
  if (T <= 152)
    return launch_k(add_rms_norm_kernel<2, FMT>, dim3((unsigned)T), dim3(threads(2)), 0, s, true, nullptr, a);
  return launch_k(add_rms_norm_kernel<4, FMT>, dim3((unsigned)T), dim3(threads(4)), 0, s, true, nullptr, a);
}

}  // namespace mm

using namespace mm;

extern "C" moe_status moe_add_rms_norm(const uint16_t* d_x, int64_t x_stride,
                                       const uint16_t* d_residual, int64_t residual_stride,
                                       const uint16_t* d_weight, float eps, int64_t num_tokens,
                                       int32_t hidden, uint16_t* d_residual_out, uint16_t* d_y,
                                       uint8_t* d_q, uint8_t* d_q_scale, uint32_t q_format,
                                       float q_static_scale, struct CUstream_st* stream) {
  if (num_tokens < 0 || hidden < 1 || !(eps >= 0.f) || eps > 1e30f) return MOE_ERR_INVALID_ARG;
  if (q_format != 0u && q_format != MOE_FLAG_MXFP8 && q_format != MOE_FLAG_PER_TENSOR)
    return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_OK;
  if (num_tokens > 0x7FFFFFFF || hidden > (1 << 20)) return MOE_ERR_UNSUPPORTED;
  if (!d_x || !d_weight || (!d_y && !d_q)) return MOE_ERR_INVALID_ARG;
  if (x_stride < hidden || (d_residual && residual_stride < hidden)) return MOE_ERR_INVALID_ARG;
  if ((d_residual != nullptr) != (d_residual_out != nullptr)) return MOE_ERR_INVALID_ARG;
  // in place only where both have the same rows
  if (d_residual && d_residual == d_residual_out && residual_stride != hidden)
    return MOE_ERR_INVALID_ARG;
  if (d_y && d_y == d_x && x_stride != hidden) return MOE_ERR_INVALID_ARG;
  int fmt = 0;
  float rscale = 1.f;
  if (d_q) {
    if (q_format == MOE_FLAG_PER_TENSOR) {
      if (!(q_static_scale > 0.f) || !(q_static_scale <= FLT_MAX)) return MOE_ERR_INVALID_ARG;
      fmt = 3;
      rscale = 1.f / q_static_scale;
    } else {
      if (!d_q_scale) return MOE_ERR_INVALID_ARG;
      fmt = q_format == MOE_FLAG_MXFP8 ? 2 : 1;
      if (hidden % (fmt == 2 ? 32 : 128)) return MOE_ERR_UNSUPPORTED;
    }
  }
  for (const void* p : {(const void*)d_x, (const void*)d_residual, (const void*)d_weight,
                        (const void*)d_residual_out, (const void*)d_y})
    if ((uintptr_t)p & 1) return MOE_ERR_INVALID_ARG;
  const NormArgs a = {d_x, d_residual, d_weight, d_residual_out, d_y, d_q, d_q_scale, x_stride,
                      residual_stride, hidden, eps, rscale};
  const uintptr_t low = (uintptr_t)d_x | (uintptr_t)d_residual | (uintptr_t)d_weight |
                        (uintptr_t)d_residual_out | (uintptr_t)d_y | ((uintptr_t)d_q << 1);
  const bool vec = hidden % 8 == 0 && hidden <= 16384 && x_stride % 8 == 0 &&
                   (!d_residual || residual_stride % 8 == 0) && (low & 15) == 0;
  cudaError_t e;
  switch (fmt) {
    case 0: e = launch_norm<0>(a, num_tokens, vec, stream); break;
    case 1: e = launch_norm<1>(a, num_tokens, vec, stream); break;
    case 2: e = launch_norm<2>(a, num_tokens, vec, stream); break;
    default: e = launch_norm<3>(a, num_tokens, vec, stream); break;
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
