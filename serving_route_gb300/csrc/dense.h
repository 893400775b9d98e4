// dense.h -- what the dense products (Fp8Linear, GatedMlp) pass from their calls
// (dense_api.cu) to their kernels (dense.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/megamoe.h"

namespace mm {

constexpr int kFusedTokens = 16;

enum DenseType { kE4M3 = 0, kBF16 = 1, kFP16 = 2 };
enum DenseAct { kSilu = 0, kGeluTanh = 1 };

// What happens to a product's FP32 sums d[m, n]:
//   kEpiStore  y[m, n] = d (float or 16 bits; float: added to what is there, if asked)
//   kEpiGate   n over gate columns, with their up columns: h = act(g) * u, and g, u to
//              `saved` where it is given
//   kEpiGrad   d = dh: from the saved g, u -> dg, du (into dgu) and h
// Activations and derivatives are of the FP32 sums (kEpiGrad: of what was saved); h, dg and du are
// rounded once to the block's type, as they are the next product's operands and the tensor core
// takes no wider ones at this rate.  That costs y and the gradients 1.4 times a rounding of
// their own (BF16: 0.0023 of the norm in place of 0.0017).
enum DenseEpi { kEpiStore = 0, kEpiGate = 1, kEpiGrad = 2 };

// A[rows, K]: element (r, k) at r * ld + k, or with `mn` at k * ld + r.
struct DenseOperand {
  const void* p;
  int64_t ld;
  int rows;
  bool mn;
};

struct DenseGemm {
  DenseOperand a, b;       // d[m, n] = sum_k a[m, k] b[n, k]; kEpiGate: b holds 2 N rows, gate then up
  int M, N, K;
  DenseType type;
  DenseEpi epi;
  DenseAct act;
  const uint8_t* sa;       // E4M3: E8M0 scales of a's rows [M, K / 128], rows sa_pitch bytes apart
  const uint8_t* sb;       // E4M3: E8M0 scales of b's blocks [ceil(N / 128), scale_pitch(K)]
  int sa_pitch;
  const uint16_t* x;       // E4M3, up to kFusedTokens rows: a in BF16 instead, quantised on the way
  int64_t ldx;
  void* out;               // kEpiStore: y; else h [M, N] (kEpiGrad: or NULL)
  int64_t ld_out;
  bool out_f32, accumulate;
  void* saved;             // [M, 2N]: g, then u
  bool saved_f32;
  void* dgu;               // kEpiGrad: [M, 2N]
  uint32_t* status;
  bool withhold;           // a test of the waits: one copy is never made
  bool early;              // the kernel before in the stream is of the same call and does not write b
};

cudaError_t dense_set_attributes();  // of the kernels, on the current device
cudaError_t dense_gemm(const DenseGemm& g, int sms, cudaStream_t s);
// What dense_gemm, and dense_gemms of `count` products, would launch (sorts them).
moe_dense_launch dense_choice(DenseGemm* g, int count, int sms);
// Up to three products of 16-bit operands (kEpiStore), of which none reads what another writes, in one launch
// (sorts them).
cudaError_t dense_gemms(DenseGemm* g, int count, int sms, cudaStream_t s);

// Bytes from one row of E8M0 scales to the next where the library lays them out: whole words.
constexpr int scale_pitch(int K) { return (K / 128 + 3) / 4 * 4; }
// x BF16 [T, cols] (rows ld elements apart) -> E4M3 codes [T, cols] and E8M0 bytes [T, scale_pitch(cols)].
cudaError_t dense_quantize_rows(const uint16_t* x, int64_t ld, int64_t T, int cols, uint8_t* q, uint8_t* s, int sms,
                                cudaStream_t stream);
// Power-of-two float scales [rows, cols] to E8M0 bytes (rows pitch apart); others set MOE_DEV_BAD_SCALE in *status.
cudaError_t dense_scales_to_e8m0(const float* s, int64_t rows, int cols, int pitch, uint8_t* out, uint32_t* status,
                                 cudaStream_t stream);

}  // namespace mm
