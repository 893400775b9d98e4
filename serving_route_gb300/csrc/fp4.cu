// fp4.cu -- few tokens on NVFP4 weights (E2M1 codes, an E4M3 scale per 16
// columns, a float scale per matrix): products of 1..16 vectors with one
// matrix (moe_fp4_linear) and the whole MoE layer (moe_fp4_forward), each one
// persistent kernel.
//
//   v = e2m1(code) * e4m3(block scale) * global
//   linear: y = x W^T;   layer: out_t = sum_k w_tk * W2[e] (silu(g) * u),
//   (g; u) = W1[e] x_t, e = topk_idx[t, k].
//
// What bounds it: the weights, 9/16 byte each, are read once and used for a
// few tokens, so the time is theirs through HBM.  At the copy rate an SM gets
// about 42 weights per clock, which leaves three issue slots per weight and
// lane; the loop below takes about 1.3:
//   * four codes pairs of a 32-bit word become half2 with one hardware convert
//     each, one half2 product applies the E4M3 scale (6 significant bits: both
//     exact in half), and m16n8k16 half MMAs with float accumulators take 8
//     tokens as their N side.  The checkpoint's order is kept: lane (g, t) owns
//     128 consecutive columns of rows g and g + 8, so a 16-byte load of codes
//     feeds eight MMAs of its own, and x is stored in shared memory in the order
//     in which the same lanes need it.
//   * x (BF16) and h (float) enter as half, each row multiplied by the power of
//     two that brings its largest value to [2^14, 2^15): for BF16 values exact
//     down to 2^-32 of the row's largest, below that rounded at 2^-40 of it; h
//     is rounded to 11 bits.  The inverse is applied to the float sums.
//   * a stage of the shared-memory ring is one warp's unit of work, 32 rows x
//     512 columns (8 KB of codes), copied by TMA as stored; eight warps take the
//     units in turn, so no barrier but the unit's own stands between the copies
//     and the MMAs.  The scales (one ninth of the bytes) go to registers, one
//     unit ahead.
//   * every CTA owns one contiguous range of the units (of the 152 per phase);
//     a tile of 32 rows that a range's end cuts is joined from float partial
//     sums by whichever CTA finishes it last, in the order of the CTAs.
//   * the layer is one cooperative launch: FC1 units, a grid barrier on h, FC2
//     units.  The weights' copies do not wait at the barrier: the ring fills
//     with FC2 weights while the last FC1 sums and h are on their way.
#include <cudaTypedefs.h>

#include <cstring>
#include <new>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace mm {

constexpr int kFp4MaxTokens = 16;
constexpr int kFp4MaxRoutes = 128;
constexpr int kFp4Grid = 152;        // one CTA per SM
constexpr int kConsumers = 8;        // warps 0..7: dequantise and multiply
constexpr int kWarpProducer = 8;     // one thread issues the TMA loads
constexpr int kWarpEpilogue = 9;     // adds the warps' sums, finishes and joins tiles
constexpr int kWarpLoader = 10;      // four warps: x and h rows to half in shared memory
constexpr int kLoaders = 4;
constexpr int kFp4Threads = 32 * (kWarpLoader + kLoaders);
constexpr int kUnitCols = 512;
constexpr int kStageBytes = 32 * kUnitCols / 2;
constexpr int kBoxBytes = 16 * 128;  // 16 rows x 256 columns
constexpr int kMaxStages = 24;
constexpr int kPartSlots = 3;
constexpr int kItems = 8;            // operand items in flight (rows ring)
constexpr int kMaxSmem = 232448;

struct Fp4Matrix {
  const uint8_t* scales;  // [n, rows, cols/16]
  const float* global;    // [n]
  int rows, cols;
};

struct Fp4Args {
  Fp4Matrix m[2];
  const uint16_t* x;
  int64_t ldx;
  const int32_t* idx;
  const float* w;
  float* h;             // [T*K, I]
  void* y;              // the layer's BF16 output, or the linear's
  uint32_t* status;
  uint32_t* ctl;        // [0] barrier, [1] finished CTAs, [2 + 152 p + c] joins of phase p
  float* part;          // [2][152][2][512]: a CTA's cut tiles, first and last
  int T, E, K, group;   // group: tokens of one operand item, at most 8 NT
  int stages, b_bytes;
  bool check, f32;
};

__host__ __device__ inline int padded_units(int cols) { return (cols + kUnitCols - 1) / kUnitCols; }
// 64 bytes of padding: rows of different parity lie in different halves of the banks
__host__ __device__ inline int row_bytes(int cols) { return padded_units(cols) * kUnitCols * 2 + 64; }

struct Fp4Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t pfull[kPartSlots], pempty[kPartSlots];
  uint64_t bfull[2][kItems], bempty[2][kItems];
  float out[kFp4MaxTokens][33];
  float rscale[2][kFp4MaxRoutes];       // per operand row: 2^-s
  float red[kLoaders];
  float route_w[kFp4MaxRoutes];         // by sorted position, as the next ones
  int16_t route_e[kFp4MaxRoutes], route_id[kFp4MaxRoutes];
  int16_t vstart[kFp4MaxRoutes + 1];    // first sorted position of every item
  int16_t vexp[kFp4MaxRoutes];
  int warp_cnt[4];
  int nv, nroutes;
  int abort;
};

template <bool MOE, int NT>
struct Fp4Ctx {
  const Fp4Args& a;
  Fp4Shared& sm;
  int nv;

  // One phase: `total` units in segments of U; a segment is a row tile times an item.
  struct Phase {
    int p, U, RT, nv, u0, u1, cols;
    __device__ int seg_begin() const { return u0 / U; }
    __device__ void split(int seg, int& v, int& j) const {
      if (p == 0) {
        v = seg / RT;
        j = seg - v * RT;
      } else {
        j = seg / nv;
        v = seg - j * nv;
      }
    }
    // units of the tile that holds seg
    __device__ int tile_units() const { return p == 0 ? U : nv * U; }
  };

  __device__ int64_t total_units(int p) const {
    const int U = padded_units(a.m[p].cols);
    const int RT = (a.m[p].rows + 31) / 32;
    return (int64_t)nv * RT * U;
  }

  __device__ Phase phase(int p) const {
    Phase f;
    f.p = p;
    f.cols = a.m[p].cols;
    f.U = padded_units(f.cols);
    f.RT = (a.m[p].rows + 31) / 32;
    f.nv = nv;
    const int64_t n = total_units(p), G = ctas(n);
    f.u0 = (int)(n * min((int64_t)blockIdx.x, G) / G);
    f.u1 = (int)(n * min((int64_t)blockIdx.x + 1, G) / G);
    return f;
  }
  // CTAs with work: none of them without a unit, so that a cut tile's CTAs are consecutive
  __device__ static int64_t ctas(int64_t n) { return min(n, (int64_t)gridDim.x); }

  __device__ int item_rows(int v) const { return sm.vstart[v + 1] - sm.vstart[v]; }
  __device__ int resident_rows(int p) const { return p == 0 ? a.T : sm.nroutes; }
  __device__ bool resident(int p) const {
    return (int64_t)resident_rows(p) * row_bytes(a.m[p].cols) <= a.b_bytes;
  }
  __device__ int ring_rows(int p) const {
    const int r = a.b_bytes / row_bytes(a.m[p].cols);
    return r < kFp4MaxRoutes ? r : kFp4MaxRoutes;
  }
  // matrix row of row r (0..31) of tile j of item v
  __device__ int64_t matrix_row(int p, int v, int j, int r) const {
    if (MOE) {
      const int64_t base = (int64_t)sm.vexp[v] * a.m[p].rows;
      if (p == 0)  // 16 gate rows, then their 16 up rows
        return base + (r < 16 ? 16 * j + r : a.m[0].rows / 2 + 16 * j + r - 16);
      return base + 32 * j + r;
    }
    return 32 * (int64_t)j + r;
  }
};

// Walks the operand items of a phase in segment order.  Resident: all rows stay
// for the phase and there is one item.  Ring: an item is the rows of one token
// group (first phase) or of one segment (second), at consecutive ring places.
struct ItemWalk {
  int item = -1, v = -1, pos = 0, rows = 0;
  template <class Ctx, class Ph>
  __device__ bool next(const Ctx& c, const Ph& f, bool resident, int R, int nv_) {
    if (resident) {
      const bool fresh = item < 0;
      item = 0;
      v = nv_;
      return fresh;
    }
    if (f.p == 0 && v == nv_) return false;
    if (item >= 0) pos = (pos + rows) % R;
    ++item;
    v = nv_;
    rows = c.item_rows(nv_);
    return true;
  }
};

__device__ __forceinline__ void e2m1x8_scaled(uint32_t w, uint32_t s, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(h[i]) : "r"(h[i]), "r"(s));
}

// Two E4M3 codes to half2.
__device__ __forceinline__ uint32_t e4m3x2_half2(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)codes));
  return h;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr));
  return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// Eight scale codes of a row: groups first..first + 7 of ng (0 past the end).
__device__ __forceinline__ uint2 load_scales(const uint8_t* row, int first, int ng, bool aligned8) {
  uint2 r = make_uint2(0u, 0u);
  if (aligned8) {
    if (first < ng) r = __ldg(reinterpret_cast<const uint2*>(row + first));
  } else {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      h[i] = first + 2 * i < ng ? __ldg(reinterpret_cast<const uint16_t*>(row + first + 2 * i)) : 0u;
    r = make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
  }
  return r;
}

// Eight consecutive values of an operand row.
__device__ __forceinline__ void load8(const uint16_t* src, int k, float (&v)[8]) {
  const uint4 p = __ldg(reinterpret_cast<const uint4*>(src + k));
  const uint32_t w[4] = {p.x, p.y, p.z, p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ void load8(const float* src, int k, float (&v)[8]) {
  // h was written by other SMs in this launch: read it from L2
  const float4 p = __ldcg(reinterpret_cast<const float4*>(src + k));
  const float4 q = __ldcg(reinterpret_cast<const float4*>(src + k + 4));
  v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w;
  v[4] = q.x, v[5] = q.y, v[6] = q.z, v[7] = q.w;
}

// One operand row: cols values (a multiple of 8) as half times 2^s, zeros up to
// the unit's end, in the order of the MMAs' lanes: within a unit of 512 columns
// lane t owns columns 128 t .. 128 t + 127 and takes its four 32-column chunks
// in the order j -> chunk j ^ (t >= 2 ? 2 : 0); 16-byte piece i of step j of lane
// t lies at ((j * 4 + i) * 4 + t) * 16.  team threads work on the row.
template <typename SRC>
__device__ __forceinline__ void fill_row(const SRC* src, int cols, uint32_t dst, int rank, int team,
                                         float* red, float* rscale) {
  const int n = cols >> 3, npad = padded_units(cols) * (kUnitCols / 8);
  float m = 0.f;
#pragma unroll 4
  for (int q = rank; q < n; q += team) {
    float v[8];
    load8(src, 8 * q, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(v[i]));
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
  if (team > 32) {
    if ((rank & 31) == 0) red[rank >> 5] = m;
    asm volatile("bar.sync 1, 128;" ::: "memory");
    m = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    asm volatile("bar.sync 1, 128;" ::: "memory");  // red is free for the next row
  }
  const int ef = (int)(__float_as_uint(m) >> 23);
  int s = 141 - (ef < 1 ? 1 : ef);
  s = m == 0.f ? 0 : (s > 126 ? 126 : s);
  const float up = __uint_as_float((uint32_t)(s + 127) << 23);
  if (rank == 0) *rscale = __uint_as_float((uint32_t)(127 - s) << 23);
#pragma unroll 4
  for (int q = rank; q < npad; q += team) {
    uint4 o = make_uint4(0u, 0u, 0u, 0u);
    if (q < n) {
      float v[8];
      load8(src, 8 * q, v);
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __half2 p = __floats2half2_rn(v[2 * i] * up, v[2 * i + 1] * up);
        h[i] = *reinterpret_cast<const uint32_t*>(&p);
      }
      o = make_uint4(h[0], h[1], h[2], h[3]);
    }
    const int u = q >> 6, r = q & 63;  // 64 pieces per unit
    const int t = r >> 4, c = (r >> 2) & 3, i = r & 3;
    const int j = c ^ ((t >> 1) << 1);
    sts128(dst + u * (kUnitCols * 2) + (((j * 4 + i) * 4 + t) << 4), o);
  }
}

// Sorted routes, and the items: runs of at most `group` tokens of one expert.
template <bool MOE>
__device__ void build_items(const Fp4Args& a, Fp4Shared& sm) {
  const int tid = threadIdx.x;
  if (!MOE) {  // token groups of the linear
    if (tid == 0) {
      int v = 0;
      for (int t = 0; t < a.T; t += a.group) {
        sm.vexp[v] = 0;
        sm.vstart[v++] = t;
      }
      sm.vstart[v] = a.T;
      sm.nv = v;
      sm.nroutes = a.T;
      if (blockIdx.x == 0) atomicExch(a.status, 0u);
    }
    if (tid < a.T) sm.route_id[tid] = tid;
    __syncthreads();
    return;
  }
  const int R = a.T * a.K;
  int e = -1;
  float w = 0.f;
  if (tid < kFp4MaxRoutes) {
    if (tid < R) {
      e = a.idx[tid];
      w = a.w[tid];
    }
    sm.route_e[tid] = e >= 0 && e < a.E ? e : -1;
  }
  uint32_t bits = 0u;
  if (tid < R && (e < -1 || e >= a.E)) bits = MOE_DEV_ROUTE_RANGE;
  if (e >= a.E) e = -1;
  __syncthreads();
  int pos = 0, within = 0, n = 0;
  if (tid < R) {
    const int t0 = tid / a.K * a.K;
    for (int r = 0; r < R; ++r) {
      const int o = sm.route_e[r];
      n += o >= 0;
      pos += o >= 0 && (o < e || (o == e && r < tid));
      within += o == e && r < tid;
      if (a.check && e >= 0 && o == e && r >= t0 && r < tid) bits |= MOE_DEV_ROUTE_DUP;
    }
    if (a.check && e >= 0 && !(fabsf(w) < INFINITY)) bits |= MOE_DEV_ROUTE_NONFINITE;
  }
  if (tid == 0) sm.nroutes = n;
  __syncthreads();  // route_e is rewritten in sorted order
  const bool live = tid < R && e >= 0;
  int16_t* first = reinterpret_cast<int16_t*>(sm.out);  // scratch: item starts by position
  if (tid < kFp4MaxRoutes) first[tid] = 0;
  __syncthreads();
  if (live) {
    sm.route_e[pos] = e;
    sm.route_id[pos] = tid;
    sm.route_w[pos] = w;
    first[pos] = within % a.group == 0;
  }
  __syncthreads();
  if (tid < kFp4MaxRoutes) {
    const bool f = first[tid] != 0;
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, f);
    if ((tid & 31) == 0) sm.warp_cnt[tid >> 5] = __popc(b);
    within = __popc(b & ((1u << (tid & 31)) - 1u));
  }
  __syncthreads();
  if (tid < kFp4MaxRoutes) {
    int v = within;
    for (int i = 0; i < (tid >> 5); ++i) v += sm.warp_cnt[i];
    if (first[tid]) {
      sm.vstart[v] = tid;
      sm.vexp[v] = sm.route_e[tid];
    }
    if (tid == 0) {
      const int nv = sm.warp_cnt[0] + sm.warp_cnt[1] + sm.warp_cnt[2] + sm.warp_cnt[3];
      sm.nv = nv;
      sm.vstart[nv] = sm.nroutes;
    }
  }
  __syncthreads();
  // the status word is this call's: the first CTA sets it
  if (blockIdx.x == 0 && tid < kFp4MaxRoutes) {
    const uint32_t all = __reduce_or_sync(0xFFFFFFFFu, bits);
    if ((tid & 31) == 0) sm.warp_cnt[tid >> 5] = (int)all;
  }
  __syncthreads();
  if (blockIdx.x == 0 && tid == 0)
    atomicExch(a.status, (uint32_t)(sm.warp_cnt[0] | sm.warp_cnt[1] | sm.warp_cnt[2] | sm.warp_cnt[3]));
}

// Bounded wait of a whole warp: all of its lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint64_t& bar, uint32_t parity, volatile int* abort,
                                          uint32_t* status) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&bar), parity, abort, status));
}

template <bool MOE, int NT>
__global__ void __launch_bounds__(kFp4Threads, 1)
    fp4_stream_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
                      const Fp4Args a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Fp4Shared sm;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t brow0 = ring + a.stages * kStageBytes;
  const uint32_t pbuf = brow0 + a.b_bytes;
  constexpr int kPartBytes = 2 * NT * 512;  // one warp's sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    prefetch_tensormap(&tm0);
    if (MOE) prefetch_tensormap(&tm1);
    sm.abort = 0;
    for (int i = 0; i < a.stages; ++i) {
      mbar_init(smem_u32(&sm.full[i]), 1);
      mbar_init(smem_u32(&sm.empty[i]), 1);
    }
    for (int i = 0; i < kPartSlots; ++i) {
      mbar_init(smem_u32(&sm.pfull[i]), kConsumers);
      mbar_init(smem_u32(&sm.pempty[i]), 1);
    }
    for (int p = 0; p < 2; ++p)
      for (int i = 0; i < kItems; ++i) {
        mbar_init(smem_u32(&sm.bfull[p][i]), kLoaders);
        mbar_init(smem_u32(&sm.bempty[p][i]), kConsumers + 1);
      }
    fence_mbar_init();
  }
  build_items<MOE>(a, sm);
  __syncthreads();

  using Ctx = Fp4Ctx<MOE, NT>;
  const Ctx c{a, sm, sm.nv};
  constexpr int kPhases = MOE ? 2 : 1;
  volatile int* abort = &sm.abort;

  if (MOE && c.nv == 0) {  // no active route: zeros
    uint4* o = reinterpret_cast<uint4*>(a.y);
    const int64_t n = (int64_t)a.T * a.m[1].rows / 8;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * blockDim.x)
      o[i] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }

  if (warp < kConsumers) {
    // ------------------------------------------------------------ consumers
    const int g = lane >> 2, t = lane & 3;
    int nbase = 0;      // units of the CTA before this phase
    int q = 0;          // segments of the CTA so far
    for (int p = 0; p < kPhases; ++p) {
      const auto f = c.phase(p);
      if (f.u0 >= f.u1) continue;
      const int ng = f.cols >> 4;
      const bool al8 = (f.cols & 127) == 0;
      const uint8_t* scales = a.m[p].scales;
      const int64_t nrows = MOE ? (int64_t)a.E * a.m[p].rows : a.m[p].rows;
      const int RB = row_bytes(f.cols);
      const bool res = c.resident(p);
      const int R = c.ring_rows(p);
      uint2 sc[4];
      auto fetch_scales = [&](int u) {
        const int seg = u / f.U, k = u - seg * f.U;
        int v, j;
        f.split(seg, v, j);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const int64_t row = c.matrix_row(p, v, j, 16 * m + g);
#pragma unroll
          for (int hi = 0; hi < 2; ++hi)
            sc[2 * m + hi] = row + 8 * hi < nrows
                                 ? load_scales(scales + (row + 8 * hi) * ng, 32 * k + 8 * t, ng, al8)
                                 : make_uint2(0u, 0u);
        }
      };
      // this warp's units: n = warp mod 8, counted over both phases
      int u = f.u0 + ((warp - nbase) & (kConsumers - 1));
      if (u < f.u1) fetch_scales(u);
      ItemWalk it;
      for (int seg = f.seg_begin(); seg * f.U < f.u1; ++seg, ++q) {
        const int ub = min(f.u1, (seg + 1) * f.U);
        int v, j;
        f.split(seg, v, j);
        const int last_item = it.item;
        if (it.next(c, f, res, R, v)) {
          if (last_item >= 0) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[p][last_item % kItems]));
          }
          if (!warp_wait(sm.bfull[p][it.item % kItems], (it.item / kItems) & 1, abort, a.status))
            goto done;
        }
        float acc[2][NT][4] = {};
        const bool any = u < ub;
        if (any) {
          const int n = c.item_rows(v), s0 = sm.vstart[v];
          uint32_t brow[NT];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int col = min(8 * nt + g, n - 1);  // columns past n repeat a row; nothing reads them
            const int slot = !res ? (it.pos + col) % R
                             : p == 1 ? s0 + col
                             : MOE ? sm.route_id[s0 + col] / a.K : s0 + col;
            brow[nt] = brow0 + slot * RB + t * 16;
          }
          for (; u < ub; u += kConsumers) {
            const int nu = nbase + u - f.u0;
            const int slot = nu % a.stages;
            const int k = u - seg * f.U;
            uint2 s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              s[i] = t < 2 ? sc[i] : make_uint2(sc[i].y, sc[i].x);  // chunk order of lanes t >= 2
            if (u + kConsumers < f.u1) fetch_scales(u + kConsumers);
            if (!warp_wait(sm.full[slot], (nu / a.stages) & 1, abort, a.status)) goto done;
            const uint32_t base = ring + slot * kStageBytes + (t >> 1) * kBoxBytes + g * 128;
            const uint32_t boff = (uint32_t)k * (kUnitCols * 2);
#pragma unroll
            for (int jj = 0; jj < 4; ++jj) {
              const uint32_t chunk = (uint32_t)(((t & 1) * 4 + (jj ^ ((t >> 1) << 1))) ^ g) << 4;
              uint32_t cw[2][2][4], sw[2][2];
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) {
                  const uint4 x = lds128(base + m * (2 * kBoxBytes) + hi * 1024 + chunk);
                  cw[m][hi][0] = x.x, cw[m][hi][1] = x.y, cw[m][hi][2] = x.z, cw[m][hi][3] = x.w;
                  const uint32_t word = jj < 2 ? s[2 * m + hi].x : s[2 * m + hi].y;
                  sw[m][hi] = e4m3x2_half2((jj & 1) ? word >> 16 : word & 0xFFFFu);
                }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                uint4 b[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) b[nt] = lds128(brow[nt] + boff + ((jj * 4 + i) << 6));
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                  uint32_t lo[4], hi[4];
                  const uint32_t sel = i < 2 ? 0x1010u : 0x3232u;
                  e2m1x8_scaled(cw[m][0][i], __byte_perm(sw[m][0], 0u, sel), lo);
                  e2m1x8_scaled(cw[m][1][i], __byte_perm(sw[m][1], 0u, sel), hi);
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt) {
                    mma_16816(acc[m][nt], lo[0], hi[0], lo[1], hi[1], b[nt].x, b[nt].y);
                    mma_16816(acc[m][nt], lo[2], hi[2], lo[3], hi[3], b[nt].z, b[nt].w);
                  }
                }
              }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.empty[slot]));
          }
        }
        const int ps = q % kPartSlots;
        if (!warp_wait(sm.pempty[ps], ((q / kPartSlots) & 1) ^ 1, abort, a.status)) goto done;
        if (any) {
          const uint32_t dst = pbuf + (ps * kConsumers + warp) * kPartBytes + lane * 16;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              sts128(dst + (m * NT + nt) * 512,
                     make_uint4(__float_as_uint(acc[m][nt][0]), __float_as_uint(acc[m][nt][1]),
                                __float_as_uint(acc[m][nt][2]), __float_as_uint(acc[m][nt][3])));
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.pfull[ps]));
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[p][it.item % kItems]));
      nbase += f.u1 - f.u0;
    }
  } else if (warp == kWarpProducer) {
    // ------------------------------------------------------------- producer
    if (lane == 0) {
      int nu = 0;
      bool ok = true;
      for (int p = 0; p < kPhases && ok; ++p) {
        const auto f = c.phase(p);
        const void* map = p == 0 ? &tm0 : &tm1;
        int seg = f.seg_begin(), k = f.u0 - seg * f.U;
        for (int u = f.u0; u < f.u1; ++u, ++nu) {
          int v, j;
          f.split(seg, v, j);
          const int slot = nu % a.stages;
          if (!mbar_wait(smem_u32(&sm.empty[slot]), ((nu / a.stages) & 1) ^ 1, abort, a.status)) {
            ok = false;
            break;
          }
          const int nbox = k * kUnitCols + kUnitCols / 2 < f.cols ? 2 : 1;  // 256-column boxes with columns
          const uint32_t bar = smem_u32(&sm.full[slot]), dst = ring + slot * kStageBytes;
          mbar_arrive_expect_tx(bar, 2 * nbox * kBoxBytes);
          for (int m = 0; m < 2; ++m)
            for (int b = 0; b < nbox; ++b)
              tma_load_2d(dst + (2 * m + b) * kBoxBytes, map, bar, k * (kUnitCols / 2) + 128 * b,
                          (int)c.matrix_row(p, v, j, 16 * m));
          if (++k == f.U) {
            k = 0;
            ++seg;
          }
        }
      }
      // no copy outlives the CTA, also when the other warps have given up
      int none = 0;
      for (int i = nu > a.stages ? nu - a.stages : 0; i < nu; ++i)
        mbar_wait_bounded(smem_u32(&sm.full[i % a.stages]), (i / a.stages) & 1, &none, nullptr, 100000000ull);
    }
  } else if (warp == kWarpEpilogue) {
    // ------------------------------------------------------------- epilogue
    const int g = lane >> 2, t = lane & 3;
    int nbase = 0, q = 0;
    for (int p = 0; p < kPhases; ++p) {
      const auto f = c.phase(p);
      const int64_t total = c.total_units(p);
      const bool res = c.resident(p);
      const int R = c.ring_rows(p);
      ItemWalk it;
      for (int seg = f.seg_begin(); seg * f.U < f.u1; ++seg, ++q) {
        const int ua = max(f.u0, seg * f.U), ub = min(f.u1, (seg + 1) * f.U);
        int v, j;
        f.split(seg, v, j);
        const int last_item = it.item;
        if (it.next(c, f, res, R, v) && last_item >= 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[p][last_item % kItems]));
        }
        const int ps = q % kPartSlots;
        if (!warp_wait(sm.pfull[ps], (q / kPartSlots) & 1, abort, a.status)) goto done;
        float acc[2][NT][4] = {};
        const int cnt = min(ub - ua, kConsumers);
        for (int i = 0; i < cnt; ++i) {
          const uint32_t src = pbuf +
                               (ps * kConsumers + ((nbase + ua - f.u0 + i) & (kConsumers - 1))) * kPartBytes +
                               lane * 16;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              const uint4 x = lds128(src + (m * NT + nt) * 512);
              acc[m][nt][0] += __uint_as_float(x.x);
              acc[m][nt][1] += __uint_as_float(x.y);
              acc[m][nt][2] += __uint_as_float(x.z);
              acc[m][nt][3] += __uint_as_float(x.w);
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.pempty[ps]));
        const int n = c.item_rows(v), s0 = sm.vstart[v];
        const float gl = __ldg(&a.m[p].global[sm.vexp[v]]);
        // lane (g, t) holds rows g and g + 8 of tokens 8 nt + 2 t and + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int col = 8 * nt + 2 * t + o;
            if (col < n) {
              const int slot = !res ? (it.pos + col) % R
                               : p == 1 ? s0 + col
                               : MOE ? sm.route_id[s0 + col] / a.K : s0 + col;
              const float rs = sm.rscale[p][slot] * gl;
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                acc[m][nt][o] *= rs;
                acc[m][nt][2 + o] *= rs;
              }
            }
          }
        const int tu = f.tile_units();
        const int tile = p == 0 ? seg : j;
        const int64_t tb = (int64_t)tile * tu, te = tb + tu;  // the tile's units
        if (p == 1) {
          // out[token][row] over the tile's experts
          if (ua == max((int64_t)f.u0, tb)) {
            for (int i = lane; i < kFp4MaxTokens * 33; i += 32) (&sm.out[0][0])[i] = 0.f;
          }
          __syncwarp();
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int col = 2 * t + o;
            if (col < n) {
              const int tok = sm.route_id[s0 + col] / a.K;
              const float w = sm.route_w[s0 + col];
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                sm.out[tok][16 * m + g] = fmaf(w, acc[m][0][o], sm.out[tok][16 * m + g]);
                sm.out[tok][16 * m + g + 8] = fmaf(w, acc[m][0][2 + o], sm.out[tok][16 * m + g + 8]);
              }
            }
          }
          __syncwarp();
          if (ub < min((int64_t)f.u1, te)) continue;  // more experts of this tile to come
        }
        const bool whole = tb >= f.u0 && te <= f.u1;
        if (!whole) {
          // join: this CTA's share goes to its slot; whoever arrives last adds the shares in CTA order
          const int64_t G = Ctx::ctas(total);
          const int c0 = (int)(((tb + 1) * G - 1) / total), c1 = (int)((te * G - 1) / total);
          auto slot = [&](int cta) { return a.part + ((size_t)(p * kFp4Grid + cta) * 2 + (cta == c0)) * 512; };
          float* mine = slot(blockIdx.x);
          if (p == 1) {
            for (int tok = 0; tok < a.T; ++tok) __stcg(&mine[tok * 32 + lane], sm.out[tok][lane]);
          } else {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                __stcg(reinterpret_cast<float4*>(mine) + (m * NT + nt) * 32 + lane,
                       make_float4(acc[m][nt][0], acc[m][nt][1], acc[m][nt][2], acc[m][nt][3]));
          }
          __threadfence();
          __syncwarp();
          uint32_t old = 0;
          uint32_t* cnt_p = &a.ctl[2 + p * kFp4Grid + c0];
          if (lane == 0) old = atomicAdd(cnt_p, 1u);
          old = __shfl_sync(0xFFFFFFFFu, old, 0);
          if (old != (uint32_t)(c1 - c0)) continue;
          __threadfence();
          if (lane == 0) *cnt_p = 0u;
          if (p == 1) {
            for (int tok = 0; tok < a.T; ++tok) {
              float s = 0.f;
              for (int i = c0; i <= c1; ++i) s += __ldcg(&slot(i)[tok * 32 + lane]);
              sm.out[tok][lane] = s;
            }
          } else {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int i = c0; i <= c1; ++i) {
                  const float4 z = __ldcg(reinterpret_cast<const float4*>(slot(i)) + (m * NT + nt) * 32 + lane);
                  s.x += z.x, s.y += z.y, s.z += z.z, s.w += z.w;
                }
                acc[m][nt][0] = s.x, acc[m][nt][1] = s.y, acc[m][nt][2] = s.z, acc[m][nt][3] = s.w;
              }
          }
        }
        if (p == 1) {
          __syncwarp();
          uint16_t* y = reinterpret_cast<uint16_t*>(a.y);
          for (int tok = 0; tok < a.T; ++tok)
            y[(int64_t)tok * a.m[1].rows + 32 * j + lane] = pack_bf16x2(sm.out[tok][lane], 0.f) & 0xFFFFu;
          __syncwarp();
          continue;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int col = 8 * nt + 2 * t + o;
            if (col >= n) continue;
            if (MOE) {
              float* h = a.h + (int64_t)sm.route_id[s0 + col] * (a.m[0].rows / 2) + 16 * j + g;
              __stcg(&h[0], swiglu(acc[0][nt][o], acc[1][nt][o]));
              __stcg(&h[8], swiglu(acc[0][nt][2 + o], acc[1][nt][2 + o]));
            } else {
              const int64_t at = (int64_t)(s0 + col) * a.m[0].rows;
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) {
                  const int row = 32 * j + 16 * m + 8 * hi + g;
                  if (row >= a.m[0].rows) continue;
                  const float val = acc[m][nt][2 * hi + o];
                  if (a.f32)
                    reinterpret_cast<float*>(a.y)[at + row] = val;
                  else
                    reinterpret_cast<uint16_t*>(a.y)[at + row] = pack_bf16x2(val, 0.f) & 0xFFFFu;
                }
            }
          }
      }
      if (f.u0 < f.u1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[p][it.item % kItems]));
      }
      if (MOE && p == 0) {  // every h value of this CTA is stored
        __threadfence();
        __syncwarp();
        if (lane == 0) atomicAdd(&a.ctl[0], 1u);
      }
      nbase += f.u1 - f.u0;
    }
  } else {
    // -------------------------------------------------------------- loaders
    const int lw = warp - kWarpLoader, lt = threadIdx.x - 32 * kWarpLoader;
    for (int p = 0; p < kPhases; ++p) {
      const auto f = c.phase(p);
      if (MOE && p == 1) {
        bool ok = true;
        if (lane == 0) {
          const uint64_t t0 = globaltimer_ns();
          while (ld_acquire_gpu_u32(&a.ctl[0]) < gridDim.x) {
            if (*abort) {
              ok = false;
              break;
            }
            if (globaltimer_ns() - t0 > kWaitLimitNs) {
              *abort = 1;
              record_status(a.status, MOE_DEV_TIMEOUT);
              ok = false;
              break;
            }
          }
        }
        if (!__shfl_sync(0xFFFFFFFFu, (int)ok, 0)) goto done;
      }
      if (f.u0 >= f.u1) continue;
      const int RB = row_bytes(f.cols);
      auto fill = [&](int src_row, int slot, int rank, int team) {
        // src_row: token (first phase) or sorted route position (second)
        if (p == 0)
          fill_row(a.x + (int64_t)src_row * a.ldx, f.cols, brow0 + slot * RB, rank, team, sm.red,
                   &sm.rscale[0][slot]);
        else
          fill_row(a.h + (int64_t)sm.route_id[src_row] * f.cols, f.cols, brow0 + slot * RB, rank, team,
                   sm.red, &sm.rscale[1][slot]);
      };
      if (c.resident(p)) {
        const int n = c.resident_rows(p);
        // (a named barrier of the four warps only where no wait that one of them
        // could give up on comes before it)
        if (p == 0 && n < kLoaders) {
          for (int r = 0; r < n; ++r) fill(r, r, lt, 32 * kLoaders);
        } else {
          for (int r = lw; r < n; r += kLoaders) fill(r, r, lane, 32);
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.bfull[p][0]));
        // the rows' memory is the next phase's when everyone is done with them
        if (p + 1 < kPhases && !warp_wait(sm.bempty[p][0], 0, abort, a.status)) goto done;
      } else {
        const int R = c.ring_rows(p);
        ItemWalk it;
        int oldest = 0, used = 0, counter = 0;
        int rows_of[kItems];  // rows of the items in flight
        auto retire = [&]() {
          if (!warp_wait(sm.bempty[p][oldest % kItems], (oldest / kItems) & 1, abort, a.status))
            return false;
#pragma unroll
          for (int i = 0; i < kItems; ++i)
            if (i == oldest % kItems) used -= rows_of[i];
          ++oldest;
          return true;
        };
        for (int seg = f.seg_begin(); seg * f.U < f.u1; ++seg) {
          int v, j;
          f.split(seg, v, j);
          if (!it.next(c, f, false, R, v)) continue;
          while (used + it.rows > R || it.item - oldest >= kItems)
            if (!retire()) goto done;
          used += it.rows;
#pragma unroll
          for (int i = 0; i < kItems; ++i)
            if (i == it.item % kItems) rows_of[i] = it.rows;
          for (int r = 0; r < it.rows; ++r, ++counter)
            if (counter % kLoaders == lw) {
              const int s = sm.vstart[v] + r;
              fill(p == 1 ? s : MOE ? sm.route_id[s] / a.K : s, (it.pos + r) % R, lane, 32);
            }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.bfull[p][it.item % kItems]));
        }
        if (p + 1 < kPhases)
          while (oldest <= it.item)
            if (!retire()) goto done;
      }
    }
  }
done:
  __syncthreads();
  // the last CTA leaves the counters at zero for the next call
  if (threadIdx.x == 0) {
    __threadfence();
    if (atomicAdd(&a.ctl[1], 1u) == gridDim.x - 1) {
      a.ctl[0] = 0u;
      a.ctl[1] = 0u;
      if (ld_acquire_gpu_u32(a.status) & MOE_DEV_TIMEOUT)
        for (int i = 0; i < 2 * kFp4Grid; ++i) a.ctl[2 + i] = 0u;
    }
  }
}

// Shared memory of a launch: the operand rows' share, and what is left for the ring.
struct Fp4Plan {
  int group, nt, stages, b_bytes, smem;
};

static int fp4_row_budget(int nt) {
  return kMaxSmem - (int)sizeof(Fp4Shared) - 2048 - kPartSlots * kConsumers * 2 * nt * 512 -
         8 * kStageBytes;  // at least eight stages
}

static void fp4_finish_plan(Fp4Plan* p) {
  p->b_bytes = (p->b_bytes + 127) / 128 * 128;
  const int left = fp4_row_budget(p->nt) - p->b_bytes;
  p->stages = 8 + left / kStageBytes;
  if (p->stages > kMaxStages) p->stages = kMaxStages;
  p->smem = 1024 + p->stages * kStageBytes + p->b_bytes + kPartSlots * kConsumers * 2 * p->nt * 512;
}

// The layer: tokens in groups of at most 8.  Rows stay for a phase where all of
// them fit (x: T rows, h: T * K), else they pass through a ring of the full budget.
static Fp4Plan fp4_plan_layer(int H, int I, int T, int K) {
  Fp4Plan p = {8, 1, 0, 0, 0};
  const int budget = fp4_row_budget(1) / 128 * 128, r1 = row_bytes(H), r2 = row_bytes(I);
  if (budget / r1 < p.group) p.group = budget / r1;
  if (budget / r2 < p.group) p.group = budget / r2;
  const int64_t n1 = (int64_t)T * r1, n2 = (int64_t)T * K * r2;
  p.b_bytes = n1 > budget || n2 > budget ? budget : (int)(n1 > n2 ? n1 : n2);
  fp4_finish_plan(&p);
  return p;
}

// The linear: one sweep over the matrix for up to 16 tokens where their rows
// fit, else equal groups, each with its own sweep (the second from L2, where
// the matrix fits there).
static Fp4Plan fp4_plan_linear(int cols, int T) {
  Fp4Plan p = {0, 1, 0, 0, 0};
  const int rb = row_bytes(cols);
  const int fit1 = fp4_row_budget(1) / 128 * 128 / rb, fit2 = fp4_row_budget(2) / 128 * 128 / rb;
  const int most = fit2 > 8 ? (fit2 < 16 ? fit2 : 16) : (fit1 < 8 ? fit1 : 8);
  const int groups = (T + most - 1) / most;
  p.group = (T + groups - 1) / groups;
  p.nt = p.group > 8 ? 2 : 1;
  const int budget = fp4_row_budget(p.nt) / 128 * 128;
  p.b_bytes = (int64_t)T * rb <= budget ? T * rb : budget;
  fp4_finish_plan(&p);
  return p;
}

template <bool MOE, int NT>
static cudaError_t fp4_launch(const CUtensorMap& t0, const CUtensorMap& t1, const Fp4Args& a, int grid,
                              int smem, cudaStream_t s) {
  cudaLaunchAttribute coop;
  coop.id = cudaLaunchAttributeCooperative;
  coop.val.cooperative = 1;
  // the layer's CTAs wait for one another (all resident, or the launch fails); the linear's do not
  return launch_k(fp4_stream_kernel<MOE, NT>, dim3(grid), dim3(kFp4Threads), smem, s, false,
                  MOE ? &coop : nullptr, t0, t1, a);
}

}  // namespace mm

using namespace mm;

struct moe_fp4_handle {
  bool layer;
  moe_dims dims;         // the layer
  Fp4Matrix m[2];        // the linear: the first
  CUtensorMap map[2];
  int max_tokens, grid;
  uint32_t* status;
  uint32_t* ctl;
  float* part;
  float* h;
};

namespace {

// Workspace: a line for the status word, counters, the cut tiles' shares, h.
constexpr size_t kFp4Align = 256;
constexpr size_t kFp4Ctl = 2048;
constexpr size_t kFp4Part = (size_t)kFp4Grid * 2 * 512 * 4;  // one phase
static_assert((2 + 2 * kFp4Grid) * 4 <= kFp4Ctl, "counters");

bool fp4_dims_ok(const moe_dims* d) {
  const bool hk = d->hidden >= 128 && d->hidden <= 16384 && d->hidden % 128 == 0;
  const bool ik = d->inter >= 128 && d->inter <= 16384 && d->inter % 128 == 0;
  const bool kk = d->top_k == 1 || d->top_k == 2 || d->top_k == 4 || d->top_k == 6 || d->top_k == 8;
  return hk && ik && kk && d->num_experts >= 1 && d->num_experts <= 1024 &&
         (d->flags & ~MOE_FLAG_CHECK_ROUTES) == 0;
}

bool misaligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// Codes [rows, cols/2] as a byte matrix; boxes of 16 rows x 128 bytes with the
// 128-byte swizzle; bytes past a row's or the matrix's end read as zero.
bool fp4_encode_map(CUtensorMap* m, const void* base, uint64_t rows, uint64_t cols) {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return false;
    fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }
  cuuint64_t dims[2] = {cols / 2, rows};
  cuuint64_t strides[1] = {cols / 2};
  cuuint32_t box[2] = {128, 16};
  cuuint32_t es[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The device checks, kernel attributes and workspace of a new handle.
moe_status fp4_set_up(moe_fp4_handle* h, void* d_workspace, cudaStream_t stream) {
  int dev = 0, major = 0, minor = 0, sms = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (major != 10 || minor != 3) return MOE_ERR_UNSUPPORTED;  // built for sm_103a only
  h->grid = sms < kFp4Grid ? sms : kFp4Grid;
  const int most = kMaxSmem - (int)sizeof(Fp4Shared) - 1024;
  const void* ks[3] = {(const void*)fp4_stream_kernel<true, 1>, (const void*)fp4_stream_kernel<false, 1>,
                       (const void*)fp4_stream_kernel<false, 2>};
  for (const void* k : ks)
    if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
      return MOE_ERR_CUDA;
  uint8_t* b = reinterpret_cast<uint8_t*>(((uintptr_t)d_workspace + kFp4Align - 1) & ~(kFp4Align - 1));
  h->status = reinterpret_cast<uint32_t*>(b);
  h->ctl = reinterpret_cast<uint32_t*>(b + kFp4Align);
  h->part = reinterpret_cast<float*>(b + kFp4Align + kFp4Ctl);
  h->h = reinterpret_cast<float*>(b + kFp4Align + kFp4Ctl + 2 * kFp4Part);
  return cudaMemsetAsync(b, 0, kFp4Align + kFp4Ctl, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

extern "C" {

moe_status moe_fp4_workspace_query(const moe_dims* dims, int64_t max_tokens, size_t* workspace_bytes) {
  if (!dims || !workspace_bytes || max_tokens < 1) return MOE_ERR_INVALID_ARG;
  if (!fp4_dims_ok(dims) || max_tokens > kFp4MaxTokens) return MOE_ERR_UNSUPPORTED;
  *workspace_bytes = 2 * kFp4Align + kFp4Ctl + 2 * kFp4Part +
                     (size_t)max_tokens * dims->top_k * dims->inter * 4;
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
  moe_fp4_handle* h = new (std::nothrow) moe_fp4_handle;
  if (!h) return MOE_ERR_INVALID_ARG;
  memset(h, 0, sizeof(*h));
  h->layer = true;
  h->dims = *dims;
  h->m[0] = {d_w1_scale, d_w1_global, 2 * dims->inter, dims->hidden};
  h->m[1] = {d_w2_scale, d_w2_global, dims->hidden, dims->inter};
  h->max_tokens = (int)max_tokens;
  st = fp4_set_up(h, d_workspace, stream);
  const uint64_t E = dims->num_experts;
  if (st == MOE_OK && (!fp4_encode_map(&h->map[0], d_w1, E * 2 * dims->inter, dims->hidden) ||
                       !fp4_encode_map(&h->map[1], d_w2, E * dims->hidden, dims->inter)))
    st = MOE_ERR_CUDA;
  if (st != MOE_OK) {
    delete h;
    return st;
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
  const Fp4Plan p = fp4_plan_layer(d.hidden, d.inter, (int)num_tokens, d.top_k);
  Fp4Args a = {};
  a.m[0] = h->m[0];
  a.m[1] = h->m[1];
  a.x = d_x;
  a.ldx = d.hidden;
  a.idx = d_topk_idx;
  a.w = d_topk_w;
  a.h = h->h;
  a.y = d_out;
  a.status = h->status;
  a.ctl = h->ctl;
  a.part = h->part;
  a.T = (int)num_tokens;
  a.E = d.num_experts;
  a.K = d.top_k;
  a.group = p.group;
  a.stages = p.stages;
  a.b_bytes = p.b_bytes;
  a.check = (d.flags & MOE_FLAG_CHECK_ROUTES) != 0;
  return fp4_launch<true, 1>(h->map[0], h->map[1], a, h->grid, p.smem, stream) == cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

moe_status moe_fp4_linear_workspace_query(int32_t rows, int32_t cols, int64_t max_tokens,
                                          size_t* workspace_bytes) {
  if (!workspace_bytes || max_tokens < 1 || rows < 1 || cols < 1) return MOE_ERR_INVALID_ARG;
  if (cols % 32 || cols > 32768 || rows > (1 << 24) || max_tokens > kFp4MaxTokens)
    return MOE_ERR_UNSUPPORTED;
  *workspace_bytes = 2 * kFp4Align + kFp4Ctl + 2 * kFp4Part;
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
  moe_fp4_handle* h = new (std::nothrow) moe_fp4_handle;
  if (!h) return MOE_ERR_INVALID_ARG;
  memset(h, 0, sizeof(*h));
  h->m[0] = {d_scales, d_global, rows, cols};
  h->max_tokens = (int)max_tokens;
  st = fp4_set_up(h, d_workspace, stream);
  if (st == MOE_OK && !fp4_encode_map(&h->map[0], d_codes, rows, cols)) st = MOE_ERR_CUDA;
  if (st != MOE_OK) {
    delete h;
    return st;
  }
  *out = h;
  return MOE_OK;
}

moe_status moe_fp4_linear(moe_fp4_handle* h, const uint16_t* d_x, int64_t x_stride, int64_t num_tokens,
                          void* d_y, int32_t y_float32, struct CUstream_st* stream) {
  if (!h || h->layer || num_tokens < 0) return MOE_ERR_INVALID_ARG;
  if (num_tokens == 0) return MOE_OK;
  if (num_tokens > h->max_tokens) return MOE_ERR_CAPACITY;
  const Fp4Matrix& m = h->m[0];
  if (!d_x || !d_y || x_stride < m.cols || x_stride % 8 || misaligned(d_x, 16) ||
      misaligned(d_y, y_float32 ? 4 : 2))
    return MOE_ERR_INVALID_ARG;
  const Fp4Plan p = fp4_plan_linear(m.cols, (int)num_tokens);
  Fp4Args a = {};
  a.m[0] = m;
  a.x = d_x;
  a.ldx = x_stride;
  a.y = d_y;
  a.status = h->status;
  a.ctl = h->ctl;
  a.part = h->part;
  a.T = (int)num_tokens;
  a.E = 1;
  a.K = 1;
  a.group = p.group;
  a.stages = p.stages;
  a.b_bytes = p.b_bytes;
  a.f32 = y_float32 != 0;
  const cudaError_t e = p.nt == 2
                            ? fp4_launch<false, 2>(h->map[0], h->map[0], a, h->grid, p.smem, stream)
                            : fp4_launch<false, 1>(h->map[0], h->map[0], a, h->grid, p.smem, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
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
