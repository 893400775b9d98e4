// topk.cu -- gate logits to expert ids and weights (moe_topk_route), one warp
// per token.
//
//   softmax:  score p = softmax(l) over the row; the choice goes by l (same
//             order); a group's score is its largest logit.
//   sigmoid:  score p = 1 / (1 + exp(-l)); the choice goes by p + bias; a
//             group's score is the sum of its two largest choice values.
//   kept:     the top_groups groups of the highest score, then the top_k
//             experts among them, ties to the lowest index;
//   weight:   p of the chosen, divided by their sum (renormalize), times scale.
//
// An expert whose logit (or bias) is -inf is masked: it is never chosen, and
// slots without an expert get id -1 and weight 0, which the layer skips.  Nor is one chosen
// that holds a NaN, but a row with one has NaN weights and names at least one expert.
//
// Every lane holds E / 32 choice values in registers as integers of the same
// order (0: masked or taken), sorted, so a choice is a warp-wide integer
// maximum of the lanes' first ones and a ballot for who has it.  Bytes: the
// logits once, 8 per chosen expert; for few tokens the chain of top_k choices
// bounds it (256 experts, 4 of 8 groups, K = 8: 2.5 to 2.8 us in a stream of calls),
// for many the instructions issued (8192 tokens: 8.8 us, 6.9 without groups, where
// the bytes alone take 1.3 at 6782 GB/s).
#include <cfloat>

#include "common.cuh"
#include "internal.h"

namespace mm {

constexpr uint32_t kAll = 0xFFFFFFFFu;

// Integers in the order of the floats, all above 0 (-inf gives 0x007FFFFF).
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // -0 and +0 are the same choice
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// 1 / x of x = 1 + exp(-l), by the hardware's reciprocal of x / 8 and one Newton step: equal
// to the correctly rounded quotient for every float x from 1 on (compared on the hardware;
// subnormal scores are within one step of it), and not flushed to 0 for l in (-88.7, -87.3) as
// the reciprocal of x is.  Below that exp(-l) is infinite and the score 0.  (A general quotient
// with its check of x's range: 8192 tokens of 256 experts, 4 of 8 groups 9.15 us, so 8.8.)
__device__ __forceinline__ float sigmoid_score(float l) {
  const float y = fmaf(expf(-l), 0.125f, 0.125f);
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(y));
  return fmaf(r, fmaf(-fminf(y, FLT_MAX), r, 1.0f), r) * 0.125f;
}

// Descending, by the odd-even merge network (Batcher 1968): 5, 19, 63, 191 exchanges of
// 4, 8, 16, 32 values.
template <int V, int P = 1, int K = 1>
__device__ __forceinline__ void sort_descending(uint32_t (&s)[V]) {
  if constexpr (P < V) {
#pragma unroll
    for (int i = K % P; i < V - K; ++i)
      // pairs (i, i + K) of runs of 2 K from K mod P on, within one run of 2 P
      if ((i - K % P) / K % 2 == 0 && i / (2 * P) == (i + K) / (2 * P)) {
        const uint32_t hi = max(s[i], s[i + K]);
        s[i + K] = min(s[i], s[i + K]);
        s[i] = hi;
      }
    if constexpr (K > 1)
      sort_descending<V, P, K / 2>(s);
    else
      sort_descending<V, 2 * P, 2 * P>(s);
  }
}

struct TopkArgs {
  const void* logits;
  const float* bias;
  int32_t* idx;
  float* w;
  int64_t ld, T;
  int E, K, groups, top_groups;
  float scale;
  bool renorm;
};

template <bool BF16>
__device__ __forceinline__ float load_logit(const void* p, int64_t i) {
  return BF16 ? bf16_bits_to_float(reinterpret_cast<const uint16_t*>(p)[i])
              : reinterpret_cast<const float*>(p)[i];
}

// A predicated load: from a plain conditional one the compiler may make a branch, and
// put it behind the scores, where its latency is not hidden (one token 3.1 us, so 2.8).
__device__ __forceinline__ float load_if(const float* p, bool on) {
  float v;
  asm volatile(
      "{\n\t.reg .pred on;\n\t"
      "setp.ne.s32 on, %2, 0;\n\t"
      "mov.f32 %0, 0f00000000;\n\t"
      "@on ld.global.f32 %0, [%1];\n\t}"
      : "=f"(v)
      : "l"(p), "r"((int)on));
  return v;
}

// V values per lane: expert 32 i + lane.
template <int V, bool BF16, bool SIGMOID>
__global__ void __launch_bounds__(128) topk_route_kernel(const TopkArgs a) {
  // BF16 values leave half of the key for the index: no two are the same
  constexpr bool kUnique = BF16 && !SIGMOID;
  const int lane = threadIdx.x & 31;
  pdl_wait();  // its launch overlaps the kernel before
  pdl_trigger();
  const int64_t t = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  if (t >= a.T) return;
  const int64_t row = t * a.ld;
  float l[V], bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {  // all loads before the first use
    const int e = 32 * i + lane;
    l[i] = e < a.E ? load_logit<BF16>(a.logits, row + e) : -INFINITY;
    bias[i] = SIGMOID ? load_if(a.bias + e, a.bias && e < a.E) : 0.f;
  }
  uint32_t key[V];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int e = 32 * i + lane;
    float c = l[i];
    if (SIGMOID) c = sigmoid_score(c) + bias[i];
    bad |= c != c;  // also where l is NaN
    key[i] = l[i] > -INFINITY && c > -INFINITY ? order_key(c) : 0u;
    if (kUnique && key[i]) key[i] = (key[i] & 0xFFFF0000u) | (0xFFFFu - e);
  }
  const bool any_nan = __any_sync(kAll, bad);

  if (a.groups > 1) {
    const int gs = a.E / a.groups;
    uint32_t mine = 0u;  // this lane's group's score (0: no expert left)
    int shift = 0;       // that group: lane >> shift
    auto group_score = [&](uint32_t m1, uint32_t m2) {
      return SIGMOID && m1 ? order_key(key_value(m1) + (m2 ? key_value(m2) : 0.f)) : m1;
    };
    if (V > 1 && gs == 32) {
      // Row i is group i: the lanes exchange halves of their rows until each has
      // one, with its two largest values so far, then those.
      uint32_t m1[V], m2[V];
#pragma unroll
      for (int i = 0; i < V; ++i) {
        m1[i] = key[i];
        m2[i] = 0u;
      }
#pragma unroll
      for (int n = V, o = 16; o >= 1; n >>= 1, o >>= 1) {
        const bool up = n > 1 && (lane & o) != 0;
        const int h = n > 1 ? n / 2 : 0;
#pragma unroll
        for (int i = 0; i < (n > 1 ? n / 2 : 1); ++i) {
          const uint32_t r1 = __shfl_xor_sync(kAll, n > 1 && !up ? m1[i + h] : m1[i], o);
          const uint32_t r2 = n == V ? 0u : __shfl_xor_sync(kAll, n > 1 && !up ? m2[i + h] : m2[i], o);
          const uint32_t k1 = up ? m1[i + h] : m1[i], k2 = up ? m2[i + h] : m2[i];
          m2[i] = max(min(k1, r1), max(k2, r2));
          m1[i] = max(k1, r1);
        }
      }
      shift = V == 2 ? 4 : V == 4 ? 3 : V == 8 ? 2 : V == 16 ? 1 : 0;
      mine = group_score(m1[0], m2[0]);
    } else {
      for (int g = 0; g < a.groups; ++g) {
        uint32_t m1 = 0u, m2 = 0u;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const uint32_t k = (uint32_t)(32 * i + lane - g * gs) < (uint32_t)gs ? key[i] : 0u;
          if (SIGMOID) m2 = max(m2, min(m1, k));
          m1 = max(m1, k);
        }
        const uint32_t b1 = __reduce_max_sync(kAll, m1);
        uint32_t b2 = 0u;
        if (SIGMOID) {
          const int first = __ffs(__ballot_sync(kAll, m1 == b1)) - 1;
          b2 = __reduce_max_sync(kAll, lane == first ? m2 : m1);
        }
        if (lane == g) mine = group_score(b1, b2);
      }
    }
    uint32_t keep = 0u;
    for (int n = 0; n < a.top_groups; ++n) {
      const uint32_t b = __reduce_max_sync(kAll, mine);
      if (b == 0u) break;
      const int g = (__ffs(__ballot_sync(kAll, mine == b)) - 1) >> shift;
      keep |= 1u << g;
      if (lane >> shift == g) mine = 0u;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int g = gs == 32 ? i : (32 * i + lane) / gs;
      if (!((keep >> (g & 31)) & 1u)) key[i] = 0u;
    }
  }

  int my = -1;  // lane k: the k-th choice
  bool tied = true;
  if (kUnique || (V > 1 && a.K > 1)) {
    // Every lane's values in descending order: a choice is the largest of the lanes'
    // first ones, and its lane moves up.  Which row held it, the end tells.  (8192 tokens,
    // us, against a search of all rows per choice: 256 experts K = 8 7.9 / 10.1, K = 1 4.8 / 4.5;
    // 64 experts K = 6 4.4 / 4.7; 1024 experts K = 8 21.3 / 41.1, K = 1 16.4 / 15.0; 16
    // experts K = 4 3.8 / 3.6.)
    uint32_t s[V];
#pragma unroll
    for (int i = 0; i < V; ++i) s[i] = key[i];
    sort_descending(s);
    uint32_t taken = 0u, holders = 0u;  // lane k: the k-th choice and the lanes that have it
    uint32_t multi = 0u, last = 0u;
    for (int k = 0; k < a.K; ++k) {
      const uint32_t b = __reduce_max_sync(kAll, s[0]);
      if (b == 0u) break;
      const bool holds = s[0] == b;
      const uint32_t who = __ballot_sync(kAll, holds);
      if (!kUnique) multi |= (who & (who - 1u)) | (b == last ? 1u : 0u);
      last = b;
      if (lane == k) {
        taken = b;
        holders = who;
      }
      if (holds) {
#pragma unroll
        for (int i = 0; i + 1 < V; ++i) s[i] = s[i + 1];
        s[V - 1] = 0u;
      }
    }
    if (kUnique) {
      if (taken) my = 0xFFFF - (taken & 0xFFFFu);
      tied = false;
    } else if (multi == 0u) {
      const int from = (__ffs(holders) - 1) & 31;
      int at = 0;
#pragma unroll
      for (int i = V - 1; i >= 0; --i)
        if (__shfl_sync(kAll, key[i], from) == taken) at = i;
      if (taken) my = 32 * at + from;
      tied = false;
    }
  }
  // equal values among the choices, one choice or one row: the first row that holds the
  // largest, and there the first lane
  if (!kUnique && tied)
    for (int k = 0; k < a.K; ++k) {
      uint32_t m = 0u;
#pragma unroll
      for (int i = 0; i < V; ++i) m = max(m, key[i]);
      const uint32_t b = __reduce_max_sync(kAll, m);
      if (b == 0u) break;
      int at = -1;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (at < 0) {
          const uint32_t who = __ballot_sync(kAll, key[i] == b);
          if (who) {
            const int first = __ffs(who) - 1;
            at = 32 * i + first;
            if (lane == first) key[i] = 0u;
          }
        }
      }
      if (lane == k) my = at;
    }

  // Only NaN (and masked) experts: the first slot names the first one that holds a NaN, so
  // that its weight is seen; the layer skips slots of -1.
  if (any_nan && __all_sync(kAll, my < 0))
    for (int e0 = 0; e0 < a.E; e0 += 32) {
      const int e = e0 + lane;
      const float v = e < a.E ? load_logit<BF16>(a.logits, row + e) : 0.f;
      const float b = SIGMOID && a.bias && e < a.E ? a.bias[e] : 0.f;
      const uint32_t who = __ballot_sync(kAll, v != v || b != b);
      if (who) {
        if (lane == 0) my = e0 + __ffs(who) - 1;
        break;
      }
    }

  float p = 0.f;
  if (SIGMOID) {
    if (my >= 0) p = sigmoid_score(load_logit<BF16>(a.logits, row + my));
  } else {
    float m = -INFINITY, s = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    if (m > -INFINITY) {
#pragma unroll
      for (int i = 0; i < V; ++i) s += expf(l[i] - m);
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    if (my >= 0) p = expf(load_logit<BF16>(a.logits, row + my) - m) / s;
  }
  if (a.renorm) {
    float s = p;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
    p = s == 0.f ? 0.f : p / s;
  }
  if (lane < a.K) {
    a.idx[t * a.K + lane] = my;
    // a NaN logit or bias: NaN weights, which the layer's route check reports
    a.w[t * a.K + lane] = any_nan ? NAN : p * a.scale;
  }
}

template <int V>
static cudaError_t launch_topk(const TopkArgs& a, bool bf16, bool sigmoid, cudaStream_t s) {
  auto k = bf16 ? (sigmoid ? topk_route_kernel<V, true, true> : topk_route_kernel<V, true, false>)
                : (sigmoid ? topk_route_kernel<V, false, true> : topk_route_kernel<V, false, false>);
  return launch_k(k, dim3((unsigned)((a.T + 3) / 4)), dim3(128), 0, s, true, nullptr, a);
}

}  // namespace mm

using namespace mm;

extern "C" moe_status moe_topk_route(const void* d_logits, int32_t logits_bf16, int64_t logits_stride,
                                     const float* d_bias, int64_t num_tokens, int32_t num_experts,
                                     int32_t top_k, int32_t sigmoid, int32_t num_groups,
                                     int32_t top_groups, int32_t renormalize, float scale,
                                     int32_t* d_topk_idx, float* d_topk_w,
                                     struct CUstream_st* stream) {
  if (num_tokens < 0) return MOE_ERR_INVALID_ARG;
  if (num_experts < 1 || num_experts > 1024 || top_k < 1 || top_k > 32 || top_k > num_experts)
    return MOE_ERR_UNSUPPORTED;
  if (num_groups < 1 || num_groups > 32 || num_experts % num_groups || top_groups < 1 ||
      top_groups > num_groups || (d_bias && !sigmoid))
    return MOE_ERR_UNSUPPORTED;
  if (num_tokens == 0) return MOE_OK;
  if (num_tokens > 0x7FFFFFFF) return MOE_ERR_UNSUPPORTED;
  if (!d_logits || !d_topk_idx || !d_topk_w || logits_stride < num_experts) return MOE_ERR_INVALID_ARG;
  if (((uintptr_t)d_logits & (logits_bf16 ? 1 : 3)) || ((uintptr_t)d_bias & 3) ||
      ((uintptr_t)d_topk_idx & 3) || ((uintptr_t)d_topk_w & 3))
    return MOE_ERR_INVALID_ARG;
  const TopkArgs a = {d_logits,     d_bias, d_topk_idx, d_topk_w,   logits_stride,
                      num_tokens,   num_experts, top_k, num_groups, top_groups,
                      scale,        renormalize != 0};
  const int v = (num_experts + 31) / 32;
  const bool b = logits_bf16 != 0, g = sigmoid != 0;
  cudaError_t e = v <= 1   ? launch_topk<1>(a, b, g, stream)
                  : v <= 2 ? launch_topk<2>(a, b, g, stream)
                  : v <= 4 ? launch_topk<4>(a, b, g, stream)
                  : v <= 8 ? launch_topk<8>(a, b, g, stream)
                  : v <= 16 ? launch_topk<16>(a, b, g, stream)
                            : launch_topk<32>(a, b, g, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
