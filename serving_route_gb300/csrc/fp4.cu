// fp4.cu -- few tokens on NVFP4 weights (E2M1 codes, an E4M3 scale per 16
// columns, a float scale per matrix): products of 1..16 vectors with one
// matrix (moe_fp4_linear) and the whole MoE layer (moe_fp4_forward).
//
//   v = e2m1(code) * e4m3(block scale) * global
//   linear: y = x W^T;   layer: out_t = sum_k w_tk * W2[e] (silu(g) * u),
//   (g; u) = W1[e] x_t, e = topk_idx[t, k].
#include <cstring>
#include <new>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace mm {

constexpr int kFp4MaxTokens = 16;

struct Fp4Matrix {
  const uint8_t* codes;   // [n, rows, cols/2]
  const uint8_t* scales;  // [n, rows, cols/16]
  const float* global;    // [n]
  int rows, cols;
};

// Four E2M1 pairs (one 32-bit word, low nibble first) to half2 values.
__device__ __forceinline__ void e2m1x8_to_half(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ float e4m3_to_float(uint32_t code) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)code));
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

// 16 values of block b of a row (without the matrix scale).
__device__ __forceinline__ void dequant16(const Fp4Matrix& m, int64_t row, int b, float (&v)[16]) {
  const uint2 c = *reinterpret_cast<const uint2*>(m.codes + row * (m.cols / 2) + 8 * b);
  const float s = e4m3_to_float(m.scales[row * (m.cols / 16) + b]);
  uint32_t h[8];
  e2m1x8_to_half(c.x, *reinterpret_cast<uint32_t(*)[4]>(h));
  e2m1x8_to_half(c.y, *reinterpret_cast<uint32_t(*)[4]>(h + 4));
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    v[2 * i] = f.x * s;
    v[2 * i + 1] = f.y * s;
  }
}

__device__ __forceinline__ float warp_total(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

// One warp per row of the matrix.
__global__ void __launch_bounds__(256) fp4_linear_kernel(Fp4Matrix m, const uint16_t* x, int64_t ldx,
                                                         int T, void* y, bool f32) {
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= m.rows) return;
  float acc[kFp4MaxTokens] = {};
  for (int b = lane; b < m.cols / 16; b += 32) {
    float v[16];
    dequant16(m, row, b, v);
#pragma unroll
    for (int t = 0; t < kFp4MaxTokens; ++t) {
      if (t >= T) break;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        acc[t] = fmaf(v[i], bf16_bits_to_float(x[t * ldx + 16 * b + i]), acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < kFp4MaxTokens; ++t) {
    if (t >= T) break;
    const float s = warp_total(acc[t]) * m.global[0];
    if (lane == 0) {
      if (f32)
        reinterpret_cast<float*>(y)[(int64_t)t * m.rows + row] = s;
      else
        reinterpret_cast<uint16_t*>(y)[(int64_t)t * m.rows + row] = pack_bf16x2(s, 0.f) & 0xFFFFu;
    }
  }
}

// Route checks: one thread per token.
__global__ void fp4_check_kernel(const int32_t* idx, const float* w, int T, int E, int K, bool check,
                                 uint32_t* status) {
  const int t = threadIdx.x;
  if (t == 0) *status = 0u;
  __syncthreads();
  if (t >= T) return;
  uint32_t bits = 0u;
  for (int k = 0; k < K; ++k) {
    const int e = idx[t * K + k];
    if (e < -1 || e >= E) bits |= MOE_DEV_ROUTE_RANGE;
    if (!check || e < 0 || e >= E) continue;
    if (!(fabsf(w[t * K + k]) < INFINITY)) bits |= MOE_DEV_ROUTE_NONFINITE;
    for (int j = 0; j < k; ++j)
      if (idx[t * K + j] == e) bits |= MOE_DEV_ROUTE_DUP;
  }
  if (bits) atomicOr(status, bits);
}

// h[route][i] = silu(g) * u: one warp per (i, route).
__global__ void __launch_bounds__(256) fp4_fc1_kernel(Fp4Matrix m, const uint16_t* x,
                                                      const int32_t* idx, int K, int E, float* h) {
  const int lane = threadIdx.x & 31, I = m.rows / 2, route = blockIdx.y;
  const int i = blockIdx.x * 8 + (threadIdx.x >> 5);
  const int e = idx[route];
  if (i >= I || e < 0 || e >= E) return;
  const uint16_t* xt = x + (int64_t)(route / K) * m.cols;
  float g = 0.f, u = 0.f;
  for (int b = lane; b < m.cols / 16; b += 32) {
    float vg[16], vu[16];
    dequant16(m, (int64_t)e * m.rows + i, b, vg);
    dequant16(m, (int64_t)e * m.rows + I + i, b, vu);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      const float xv = bf16_bits_to_float(xt[16 * b + j]);
      g = fmaf(vg[j], xv, g);
      u = fmaf(vu[j], xv, u);
    }
  }
  g = warp_total(g) * m.global[e];
  u = warp_total(u) * m.global[e];
  if (lane == 0) h[(int64_t)route * I + i] = swiglu(g, u);
}

// out[t][c] = sum_k w_tk * W2[e_tk][c] . h[t, k]: one warp per (c, t).
__global__ void __launch_bounds__(256) fp4_fc2_kernel(Fp4Matrix m, const float* h, const int32_t* idx,
                                                      const float* w, int K, int E, uint16_t* out) {
  const int lane = threadIdx.x & 31, t = blockIdx.y;
  const int c = blockIdx.x * 8 + (threadIdx.x >> 5);
  if (c >= m.rows) return;
  float acc = 0.f;
  for (int k = 0; k < K; ++k) {
    const int e = idx[t * K + k];
    if (e < 0 || e >= E) continue;
    float s = 0.f;
    for (int b = lane; b < m.cols / 16; b += 32) {
      float v[16];
      dequant16(m, (int64_t)e * m.rows + c, b, v);
#pragma unroll
      for (int j = 0; j < 16; ++j) s = fmaf(v[j], h[(int64_t)(t * K + k) * m.cols + 16 * b + j], s);
    }
    acc = fmaf(w[t * K + k], warp_total(s) * m.global[e], acc);
  }
  if (lane == 0) out[(int64_t)t * m.rows + c] = pack_bf16x2(acc, 0.f) & 0xFFFFu;
}

}  // namespace mm

using namespace mm;

struct moe_fp4_handle {
  bool layer;
  moe_dims dims;        // the layer
  Fp4Matrix w1, w2;     // the linear: w1
  int max_tokens, device;
  uint32_t* status;
  float* h;
};

namespace {

constexpr size_t kFp4Align = 256;

bool fp4_dims_ok(const moe_dims* d) {
  const bool hk = d->hidden >= 128 && d->hidden <= 16384 && d->hidden % 128 == 0;
  const bool ik = d->inter >= 128 && d->inter <= 16384 && d->inter % 128 == 0;
  const bool kk = d->top_k == 1 || d->top_k == 2 || d->top_k == 4 || d->top_k == 6 || d->top_k == 8;
  return hk && ik && kk && d->num_experts >= 1 && d->num_experts <= 1024 &&
         (d->flags & ~MOE_FLAG_CHECK_ROUTES) == 0;
}

moe_status fp4_device(int* dev) {
  int major = 0, minor = 0;
  if (cudaGetDevice(dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  return major == 10 && minor == 3 ? MOE_OK : MOE_ERR_UNSUPPORTED;  // built for sm_103a only
}

bool misaligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

}  // namespace

extern "C" {

moe_status moe_fp4_workspace_query(const moe_dims* dims, int64_t max_tokens, size_t* workspace_bytes) {
  if (!dims || !workspace_bytes || max_tokens < 1) return MOE_ERR_INVALID_ARG;
  if (!fp4_dims_ok(dims) || max_tokens > kFp4MaxTokens) return MOE_ERR_UNSUPPORTED;
  *workspace_bytes = 2 * kFp4Align + (size_t)max_tokens * dims->top_k * dims->inter * 4;
  return MOE_OK;
}

moe_status moe_fp4_create(const moe_dims* dims, int64_t max_tokens, const uint8_t* d_w1,
                          const uint8_t* d_w1_scale, const float* d_w1_global, const uint8_t* d_w2,
                          const uint8_t* d_w2_scale, const float* d_w2_global, void* d_workspace,
                          size_t workspace_bytes, struct CUstream_st* stream, moe_fp4_handle** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  size_t need = 0;
  moe_status st = moe_fp4_workspace_query(dims, max_tokens, &need);
  if (st != MOE_OK) return st;
  if (!d_w1 || !d_w1_scale || !d_w1_global || !d_w2 || !d_w2_scale || !d_w2_global || !d_workspace)
    return MOE_ERR_INVALID_ARG;
  if (misaligned(d_w1, 16) || misaligned(d_w1_scale, 16) || misaligned(d_w2, 16) ||
      misaligned(d_w2_scale, 16) || misaligned(d_w1_global, 4) || misaligned(d_w2_global, 4) ||
      misaligned(d_workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  int dev = 0;
  if ((st = fp4_device(&dev)) != MOE_OK) return st;
  moe_fp4_handle* h = new (std::nothrow) moe_fp4_handle;
  if (!h) return MOE_ERR_INVALID_ARG;
  memset(h, 0, sizeof(*h));
  h->layer = true;
  h->dims = *dims;
  h->w1 = {d_w1, d_w1_scale, d_w1_global, 2 * dims->inter, dims->hidden};
  h->w2 = {d_w2, d_w2_scale, d_w2_global, dims->hidden, dims->inter};
  h->max_tokens = (int)max_tokens;
  h->device = dev;
  uint8_t* b = reinterpret_cast<uint8_t*>(((uintptr_t)d_workspace + kFp4Align - 1) & ~(kFp4Align - 1));
  h->status = reinterpret_cast<uint32_t*>(b);
  h->h = reinterpret_cast<float*>(b + kFp4Align);
  if (cudaMemsetAsync(b, 0, kFp4Align, stream) != cudaSuccess) {
    delete h;
    return MOE_ERR_CUDA;
  }
  *out = h;
  return MOE_OK;
}

moe_status moe_fp4_forward(moe_fp4_handle* h, const uint16_t* d_x, const int32_t* d_topk_idx,
                           const float* d_topk_w, int64_t num_tokens, uint16_t* d_out,
                           struct CUstream_st* stream) {
  if (!h || !h->layer || num_tokens < 0) return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_OK;
  if (num_tokens > h->max_tokens) return MOE_ERR_CAPACITY;
  if (!d_x || !d_topk_idx || !d_topk_w || !d_out || misaligned(d_x, 16) ||
      misaligned(d_topk_idx, 4) || misaligned(d_topk_w, 4) || misaligned(d_out, 16))
    return MOE_ERR_INVALID_ARG;
  const moe_dims& d = h->dims;
  const int T = (int)num_tokens;
  fp4_check_kernel<<<1, 32, 0, stream>>>(d_topk_idx, d_topk_w, T, d.num_experts, d.top_k,
                                         (d.flags & MOE_FLAG_CHECK_ROUTES) != 0, h->status);
  fp4_fc1_kernel<<<dim3(d.inter / 8, T * d.top_k), 256, 0, stream>>>(h->w1, d_x, d_topk_idx, d.top_k,
                                                                     d.num_experts, h->h);
  fp4_fc2_kernel<<<dim3(d.hidden / 8, T), 256, 0, stream>>>(h->w2, h->h, d_topk_idx, d_topk_w, d.top_k,
                                                            d.num_experts, d_out);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_fp4_linear_workspace_query(int32_t rows, int32_t cols, int64_t max_tokens,
                                          size_t* workspace_bytes) {
  if (!workspace_bytes || max_tokens < 1 || rows < 1 || cols < 1) return MOE_ERR_INVALID_ARG;
  if (cols % 32 || cols > 32768 || rows > (1 << 24) || max_tokens > kFp4MaxTokens)
    return MOE_ERR_UNSUPPORTED;
  *workspace_bytes = 2 * kFp4Align;
  return MOE_OK;
}

moe_status moe_fp4_linear_create(int32_t rows, int32_t cols, int64_t max_tokens, const uint8_t* d_codes,
                                 const uint8_t* d_scales, const float* d_global, void* d_workspace,
                                 size_t workspace_bytes, struct CUstream_st* stream,
                                 moe_fp4_handle** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  size_t need = 0;
  moe_status st = moe_fp4_linear_workspace_query(rows, cols, max_tokens, &need);
  if (st != MOE_OK) return st;
  if (!d_codes || !d_scales || !d_global || !d_workspace || misaligned(d_codes, 16) ||
      misaligned(d_scales, 16) || misaligned(d_global, 4) || misaligned(d_workspace, 16))
    return MOE_ERR_INVALID_ARG;
  if (workspace_bytes < need) return MOE_ERR_WORKSPACE;
  int dev = 0;
  if ((st = fp4_device(&dev)) != MOE_OK) return st;
  moe_fp4_handle* h = new (std::nothrow) moe_fp4_handle;
  if (!h) return MOE_ERR_INVALID_ARG;
  memset(h, 0, sizeof(*h));
  h->w1 = {d_codes, d_scales, d_global, rows, cols};
  h->max_tokens = (int)max_tokens;
  h->device = dev;
  uint8_t* b = reinterpret_cast<uint8_t*>(((uintptr_t)d_workspace + kFp4Align - 1) & ~(kFp4Align - 1));
  h->status = reinterpret_cast<uint32_t*>(b);
  if (cudaMemsetAsync(b, 0, kFp4Align, stream) != cudaSuccess) {
    delete h;
    return MOE_ERR_CUDA;
  }
  *out = h;
  return MOE_OK;
}

moe_status moe_fp4_linear(moe_fp4_handle* h, const uint16_t* d_x, int64_t x_stride, int64_t num_tokens,
                          void* d_y, int32_t y_float32, struct CUstream_st* stream) {
  if (!h || h->layer || num_tokens < 0) return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_OK;
  if (num_tokens > h->max_tokens) return MOE_ERR_CAPACITY;
  if (!d_x || !d_y || x_stride < h->w1.cols || x_stride % 8 || misaligned(d_x, 16) ||
      misaligned(d_y, y_float32 ? 4 : 2))
    return MOE_ERR_INVALID_ARG;
  fp4_linear_kernel<<<(h->w1.rows + 7) / 8, 256, 0, stream>>>(h->w1, d_x, x_stride, (int)num_tokens,
                                                              d_y, y_float32 != 0);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_fp4_read_status(moe_fp4_handle* h, uint32_t* h_status, struct CUstream_st* stream) {
  if (!h || !h_status) return MOE_ERR_INVALID_ARG;
  if (cudaMemcpyAsync(h_status, h->status, 4, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (*h_status & MOE_DEV_TIMEOUT) return MOE_ERR_DEVICE_TIMEOUT;
  return *h_status ? MOE_ERR_BAD_ROUTE : MOE_OK;
}

void moe_fp4_destroy(moe_fp4_handle* h) { delete h; }

}  // extern "C"
