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
constexpr int kConsumers = 8;        // the first warps: dequantise and multiply
constexpr int kProducers = 2;        // then two that issue the copies of the weights, in turn
constexpr int kWarpProducer = kConsumers;
constexpr int kWarpEpilogue = kWarpProducer + kProducers;  // adds the warps' sums, finishes and joins tiles
constexpr int kWarpLoader = kWarpEpilogue + 1;             // x and h rows to half in shared memory
constexpr int kLoaders = 4;
constexpr int kFp4Threads = 32 * (kWarpLoader + kLoaders);
constexpr int kUnitCols = 512;
constexpr int kCodeBytes = 32 * kUnitCols / 2;
constexpr int kScaleBytes = 32 * kUnitCols / 16;
constexpr int kStageBytes = kCodeBytes + kScaleBytes;
constexpr int kBoxBytes = 16 * 128;  // 16 rows x 256 columns
// A multiple of kConsumers: then a slot's units are all one warp's, so no warp
// waits for a phase while an earlier phase of the slot is open (it would take
// the parity of the phase before that one for its own).
constexpr int kMaxStages = 2 * kConsumers;
constexpr int kItems = 8;            // operand items in flight (rows ring)
constexpr int kCutUnits = 15;        // units of imbalance that a tile's join costs (about 3 us)
constexpr int kTile2 = 128;          // output rows of an FC2 tile
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
  uint8_t* h;           // [T*K] records of half values and their block exponents
  void* y;              // the layer's BF16 output, or the linear's
  uint32_t* status;
  uint32_t* ctl;        // [0] barrier, [1] finished CTAs, [2 + 152 p + c] joins of phase p
  float* part[2];       // by phase, [152][2][..]: a CTA's cut tiles, first and last
  int T, E, K, group;   // group: tokens of one operand item, at most 8 NT
  int stages, b_bytes;
  bool check, f32;
};

__host__ __device__ inline int padded_units(int cols) { return (cols + kUnitCols - 1) / kUnitCols; }
// h of one route in global memory: halves, then one exponent byte per 16 of them
__host__ __device__ inline int exponent_bytes(int cols) { return (cols / 16 + 15) & ~15; }
__host__ __device__ inline int record_bytes(int cols) { return cols * 2 + exponent_bytes(cols); }
// An operand row in shared memory: whole units, the exponents of an h row, and 64 bytes
// past a multiple of 128, so that rows of different parity lie in different banks.
__host__ __device__ inline int row_bytes(int cols, bool h) {
  return ((padded_units(cols) * kUnitCols * 2 + (h ? exponent_bytes(cols) : 0) + 127) & ~127) + 64;
}

struct Fp4Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t pfull[kConsumers][2], pempty[kConsumers][2];
  uint64_t bfull[2][kItems], bempty[2][kItems];
  uint64_t raw[kLoaders];
  alignas(16) float out[kFp4MaxTokens][kTile2];
  alignas(16) int key[kFp4MaxRoutes];
  float rscale[2][kFp4MaxRoutes];       // per operand row: 2^-s
  float vglobal[2][kFp4MaxRoutes];      // the items' matrix scales
  float route_w[kFp4MaxRoutes];         // by sorted position, as the next ones
  int16_t route_e[kFp4MaxRoutes], route_id[kFp4MaxRoutes], route_tok[kFp4MaxRoutes];
  int16_t vstart[kFp4MaxRoutes + 1];    // first sorted position of every item
  int16_t vexp[kFp4MaxRoutes];
  uint8_t first[kFp4MaxRoutes];
  float red[kLoaders];
  int warp_cnt[4];
  int nv, nroutes;
  int abort;
};

// Where a walk over a phase stands: segment seg = the U units of item v's
// product with 32 matrix rows: block rb of tile j.
struct SegPos {
  int v, j, rb;
};

// One phase of one CTA: units [u0, u1), U to a segment.  Order of the segments:
// first phase  item, tile (RT of 32 rows each);
// second       tile (128 rows), item, block of 32 rows -- an item's rows serve four segments.
struct Phase {
  int p, U, RT, nv, u0, u1, cols;
  __device__ int seg_begin() const { return u0 / U; }
  __device__ SegPos at(int seg) const {
    SegPos s;
    if (p == 0) {
      s.v = seg / RT;
      s.j = seg - s.v * RT;
      s.rb = 0;
    } else {
      s.j = seg / (nv * 4);
      const int r = seg - s.j * nv * 4;
      s.v = r >> 2;
      s.rb = r & 3;
    }
    return s;
  }
  __device__ void step(SegPos& s) const {
    if (p == 0) {
      if (++s.j == RT) {
        s.j = 0;
        ++s.v;
      }
    } else if (++s.rb == 4) {
      s.rb = 0;
      if (++s.v == nv) {
        s.v = 0;
        ++s.j;
      }
    }
  }
  __device__ int tile_units() const { return p == 0 ? U : nv * 4 * U; }
};

template <bool MOE, int NT>
struct Fp4Ctx {
  const Fp4Args& a;
  Fp4Shared& sm;
  int nv;

  __device__ int64_t total_units(int p) const {
    return (int64_t)nv * ((a.m[p].rows + 31) / 32) * padded_units(a.m[p].cols);
  }
  // CTAs with work: none of them without a unit, so that a cut tile's CTAs are consecutive
  __device__ static int64_t ctas(int64_t n) { return min(n, (int64_t)gridDim.x); }

  __device__ Phase phase(int p) const {
    Phase f;
    f.p = p;
    f.cols = a.m[p].cols;
    f.U = padded_units(f.cols);
    f.RT = (a.m[p].rows + 31) / 32;
    f.nv = nv;
    // whole tiles, unless the CTA with one more than the others would work
    // longer than a join takes
    const int64_t n = total_units(p), tu = f.tile_units(), tiles = n / tu;
    const int64_t most = (tiles + gridDim.x - 1) / gridDim.x * tu;
    const int64_t G = ctas(n), step = most - (n + G - 1) / G > kCutUnits ? 1 : tu;
    const int64_t steps = n / step, H = min(steps, G);
    f.u0 = (int)(steps * min((int64_t)blockIdx.x, H) / H * step);
    f.u1 = (int)(steps * min((int64_t)blockIdx.x + 1, H) / H * step);
    return f;
  }

  __device__ int item_rows(int v) const { return sm.vstart[v + 1] - sm.vstart[v]; }
  // x rows stay for the whole phase where all of them fit; h rows always pass
  // through the ring, so that the first segment waits for its own rows only
  __device__ bool resident(int p) const {
    return p == 0 && (int64_t)a.T * row_bytes(a.m[0].cols, false) <= a.b_bytes;
  }
  __device__ int ring_rows(int p) const {
    return min(a.b_bytes / row_bytes(a.m[p].cols, p == 1), kFp4MaxRoutes);
  }
  // place of an item's column among the operand rows
  __device__ int row_slot(bool resident, int pos, int R, int s0, int col) const {
    if (resident) return sm.route_tok[s0 + col];
    return pos + col < R ? pos + col : pos + col - R;
  }
  // matrix row of row r (0..31) of a segment
  __device__ int64_t matrix_row(int p, const SegPos& s, int r) const {
    if (!MOE) return 32 * (int64_t)s.j + r;
    const int64_t base = (int64_t)sm.vexp[s.v] * a.m[p].rows;
    if (p == 0)  // 16 gate rows, then their 16 up rows
      return base + (r < 16 ? 16 * s.j + r : a.m[0].rows / 2 + 16 * s.j + r - 16);
    return base + kTile2 * s.j + 32 * s.rb + r;
  }
};

// Walks the operand items of a phase in segment order.  Resident: all rows stay
// for the phase and there is one item.  Ring: an item is the rows of one token
// group, for one run of segments, at consecutive ring places.
struct ItemWalk {
  int item = -1, v = -1, j = -1, pos = 0, rows = 0;
  // whether a new item starts with segment s
  template <class Ctx>
  __device__ bool next(const Ctx& c, const Phase& f, bool resident, int R, const SegPos& s) {
    if (resident) {
      const bool fresh = item < 0;
      item = 0;
      return fresh;
    }
    if (s.v == v && (f.p == 0 || s.j == j)) return false;
    pos += rows;
    if (pos >= R) pos -= R;
    ++item;
    v = s.v;
    j = s.j;
    rows = c.item_rows(s.v);
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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
}

// Asynchronous copy of N bytes, of which the first `valid` are read and the rest zero.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int valid) {
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(valid), "n"(N)
                 : "memory");
}

// The 32 scale bytes of one row of a unit (n of them in the matrix, the rest
// zero) to shared memory, in copies as wide as the rows' alignment allows.
template <int N>
__device__ __forceinline__ void copy_scale_row(uint32_t dst, const uint8_t* src, int n) {
#pragma unroll
  for (int o = 0; o < 32; o += N) {
    const int v = min(max(n - o, 0), N);
    cp_async<N>(dst + o, v > 0 ? src + o : src, v);
  }
}

// Bounded wait of a whole warp: all of its lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint64_t& bar, uint32_t parity, volatile int* abort,
                                          uint32_t* status) {
  return __all_sync(0xFFFFFFFFu, mbar_wait(smem_u32(&bar), parity, abort, status));
}

// Within a unit of 512 columns lane t of an MMA owns columns 128 t .. 128 t + 127
// and takes its four 32-column chunks in the order j -> chunk j ^ (t >= 2 ? 2 : 0);
// piece i (eight columns) of step j of lane t lies at ((j * 4 + i) * 4 + t) * 16.
__device__ __forceinline__ int piece_offset(int q) {
  const int t = q >> 4, ch = (q >> 2) & 3, i = q & 3;
  return (((ch ^ ((t >> 1) << 1)) * 4 + i) * 4 + t) << 4;
}

// s with max * 2^s in [2^14, 2^15), kept so that 2^s and 2^-s are normal; 126 for 0.
__device__ __forceinline__ int row_exponent(float max) {
  const int ef = (int)(__float_as_uint(max) >> 23);
  const int s = 141 - (ef < 1 ? 1 : ef);
  return max == 0.f || s > 126 ? 126 : s;
}

__device__ __forceinline__ float pow2f(int s) { return __uint_as_float((uint32_t)(s + 127) << 23); }

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Brings `bytes` (a multiple of 16) to shared memory and waits.  The places were
// read and written through the generic proxy before: a fence orders them.
__device__ __forceinline__ void raw_begin(uint64_t& bar, uint32_t bytes) {
  fence_proxy_async_smem();
  mbar_arrive_expect_tx(smem_u32(&bar), bytes);
}

// One x row (cols BF16 values, a multiple of 32) as half times 2^s, zeros up to
// the unit's end.  The row is copied as it is and turned in place, unit by unit;
// TEAM warps (one, or all loaders) work on it.
template <int TEAM>
__device__ __forceinline__ bool fill_x(const uint16_t* src, int cols, uint32_t dst, int rank,
                                       uint64_t& bar, uint32_t& parity, float* red, float* rscale,
                                       volatile int* abort, uint32_t* status) {
  const int lane = threadIdx.x & 31, n = cols >> 3, U = padded_units(cols);
  if (rank == 0 && lane == 0) {
    raw_begin(bar, cols * 2);
    bulk_load(dst, src, cols * 2, smem_u32(&bar));
  }
  const bool ok = warp_wait(bar, parity, abort, status);  // a team goes on to its barriers either way
  parity ^= 1;
  uint32_t m = 0u;  // the largest |value|, as BF16 bits
#pragma unroll 4
  for (int q = 32 * rank + lane; q < n; q += 32 * TEAM) {
    const uint4 v = lds128(dst + 16 * q);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] & 0x7FFFu, hi = (w[i] >> 16) & 0x7FFFu;
      // NaN does not set the scale (it stays NaN in half); infinity does
      m = max(m, max(lo > 0x7F80u ? 0u : lo, hi > 0x7F80u ? 0u : hi));
    }
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (TEAM > 1) {
    if (lane == 0) red[rank] = __uint_as_float(m);
    asm volatile("bar.sync 1, %0;" ::"n"(32 * TEAM) : "memory");
#pragma unroll
    for (int i = 0; i < TEAM; ++i) m = max(m, __float_as_uint(red[i]));
    asm volatile("bar.sync 1, %0;" ::"n"(32 * TEAM) : "memory");  // red is free for the next row
  }
  const int s = row_exponent(__uint_as_float(m << 16));
  const float up = pow2f(s);
  if (rank == 0 && lane == 0) *rscale = pow2f(-s);
  for (int u = rank; u < U; u += TEAM) {
    const uint32_t base = dst + u * (kUnitCols * 2);
    uint4 o[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int q = lane + 32 * k;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (64 * u + q < n) v = lds128(base + 16 * q);
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
      uint32_t h[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[i] = half2_bits(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
      o[k] = make_uint4(h[0], h[1], h[2], h[3]);
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k) sts128(base + piece_offset(lane + 32 * k), o[k]);
  }
  return ok;
}

// 2^-d in half, 0 below the subnormals.
__device__ __forceinline__ uint32_t half_pow2_neg(int d) {
  const uint32_t b = d <= 14 ? (uint32_t)(15 - d) << 10 : d <= 24 ? 1u << (24 - d) : 0u;
  return b | (b << 16);
}

// One h row: halves with one exponent per 16 (value = half * 2^-e) as halves of
// the row's common exponent, turned in place like x.
__device__ __forceinline__ bool fill_h(const uint8_t* src, int cols, uint32_t dst, uint64_t& bar,
                                       uint32_t& parity, float* rscale, volatile int* abort,
                                       uint32_t* status) {
  const int lane = threadIdx.x & 31, n = cols >> 3, U = padded_units(cols);
  const uint32_t ex = dst + U * (kUnitCols * 2);
  if (lane == 0) {
    raw_begin(bar, record_bytes(cols));
    bulk_load(dst, src, cols * 2, smem_u32(&bar));
    bulk_load(ex, src + cols * 2, exponent_bytes(cols), smem_u32(&bar));
  }
  if (!warp_wait(bar, parity, abort, status)) return false;
  parity ^= 1;
  auto exponent = [&](int block) {
    int e;
    asm volatile("ld.shared.s8 %0, [%1];" : "=r"(e) : "r"(ex + block) : "memory");
    return e;
  };
  int s = 126;
  for (int b = lane; b < (cols >> 4); b += 32) s = min(s, exponent(b));
  s = __reduce_min_sync(0xFFFFFFFFu, s);
  if (lane == 0) *rscale = pow2f(-s);
  for (int u = 0; u < U; ++u) {
    const uint32_t base = dst + u * (kUnitCols * 2);
    uint4 o[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int q = lane + 32 * k;
      o[k] = make_uint4(0u, 0u, 0u, 0u);
      if (64 * u + q < n) {
        const uint4 v = lds128(base + 16 * q);
        const int d = exponent((64 * u + q) >> 1) - s;
        const uint32_t f1 = half_pow2_neg(min(d, 14)), f2 = half_pow2_neg(d - min(d, 14));
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(f1));
          asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(f2));
        }
        o[k] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 2; ++k) sts128(base + piece_offset(lane + 32 * k), o[k]);
  }
  return true;
}

// Sorted routes, and the items: runs of at most `group` tokens of one expert.
template <bool MOE>
__device__ __forceinline__ void build_items(const Fp4Args& a, Fp4Shared& sm) {
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
    if (tid < a.T) sm.route_id[tid] = sm.route_tok[tid] = tid;
    return;
  }
  const int R = a.T * a.K;
  int e = -1;
  float w = 0.f;
  uint32_t bits = 0u;
  if (tid < R) {
    e = a.idx[tid];
    w = a.w[tid];
    if (e < -1 || e >= a.E) bits = MOE_DEV_ROUTE_RANGE;
    if (e >= a.E) e = -1;
  }
  const bool live = e >= 0;  // (threads past the routes: not live)
  const int mine = live ? e * kFp4MaxRoutes + tid : 0x7FFFFFFF;  // by expert, then by route
  if (tid < kFp4MaxRoutes) {
    sm.key[tid] = mine;
    sm.first[tid] = 0;
  }
  __syncthreads();
  int pos = 0, within = 0;
  if (live) {
    const int low = e * kFp4MaxRoutes;
#pragma unroll 4
    for (int r = 0; r < R; r += 4) {
      const int4 k4 = *reinterpret_cast<const int4*>(&sm.key[r]);
      const int k[4] = {k4.x, k4.y, k4.z, k4.w};  // past the routes: the largest key
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pos += k[i] < mine;
        within += k[i] < mine && k[i] >= low;
      }
    }
    if (a.check) {
      for (int r = tid / a.K * a.K; r < tid; ++r)
        if (sm.key[r] >= low && sm.key[r] < mine) bits |= MOE_DEV_ROUTE_DUP;
      if (!(fabsf(w) < INFINITY)) bits |= MOE_DEV_ROUTE_NONFINITE;
    }
    sm.route_e[pos] = e;
    sm.route_id[pos] = tid;
    sm.route_tok[pos] = tid / a.K;
    sm.route_w[pos] = w;
    sm.first[pos] = within % a.group == 0;
  }
  const int n = __syncthreads_count(live);
  if (tid < kFp4MaxRoutes) {
    const uint32_t b = __ballot_sync(0xFFFFFFFFu, sm.first[tid] != 0);
    if ((tid & 31) == 0) sm.warp_cnt[tid >> 5] = __popc(b);
    within = __popc(b & ((1u << (tid & 31)) - 1u));
  }
  // the status word is this call's: the first CTA sets it
  if (__syncthreads_or(bits != 0u)) {
    if (blockIdx.x == 0 && tid == 0) atomicExch(a.status, 0u);
    __syncthreads();
    if (blockIdx.x == 0 && bits) atomicOr(a.status, bits);
  } else if (blockIdx.x == 0 && tid == 0) {
    atomicExch(a.status, 0u);
  }
  if (tid < kFp4MaxRoutes) {
    int v = within;
    for (int i = 0; i < (tid >> 5); ++i) v += sm.warp_cnt[i];
    if (sm.first[tid]) {
      sm.vstart[v] = tid;
      sm.vexp[v] = sm.route_e[tid];
    }
    if (tid == 0) {
      const int nv = sm.warp_cnt[0] + sm.warp_cnt[1] + sm.warp_cnt[2] + sm.warp_cnt[3];
      sm.nv = nv;
      sm.nroutes = n;
      sm.vstart[nv] = n;
    }
  }
}

template <bool MOE, int NT>
__global__ void __launch_bounds__(kFp4Threads, 1)
    fp4_stream_kernel(const __grid_constant__ CUtensorMap tm0, const __grid_constant__ CUtensorMap tm1,
                      const Fp4Args a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Fp4Shared sm;
  const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint8_t* const smem = smem_raw + (ring - smem_u32(smem_raw));  // the same, for plain loads
  const uint32_t srow0 = ring + a.stages * kCodeBytes;   // the stages' scales
  const uint32_t brow0 = srow0 + a.stages * kScaleBytes; // operand rows
  const uint32_t pbuf = brow0 + a.b_bytes;               // the consumers' sums
  constexpr int kPartBytes = 2 * NT * 512;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  {
    const int i = threadIdx.x;
    if (i < kMaxStages) {
      // copies: one arrival with the codes' bytes, one per lane with its scales
      mbar_init(smem_u32(&sm.full[i]), 33);
      mbar_init(smem_u32(&sm.empty[i]), 1);
    } else if (i >= 32 && i < 32 + 2 * kConsumers) {
      mbar_init(smem_u32(&sm.pfull[0][0] + (i - 32)), 1);
      mbar_init(smem_u32(&sm.pempty[0][0] + (i - 32)), 1);
    } else if (i >= 64 && i < 64 + 2 * kItems) {
      mbar_init(smem_u32(&sm.bfull[0][0] + (i - 64)), kLoaders);
      mbar_init(smem_u32(&sm.bempty[0][0] + (i - 64)), kConsumers + 1);
    } else if (i >= 96 && i < 96 + kLoaders) {
      mbar_init(smem_u32(&sm.raw[i - 96]), 1);
    } else if (i == 128) {
      sm.abort = 0;
      prefetch_tensormap(&tm0);
      if (MOE) prefetch_tensormap(&tm1);
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
    int nbase = 0;  // units of the CTA before this phase
    int pc = 0;     // sums this warp has handed over
    for (int p = 0; p < kPhases; ++p) {
      const Phase f = c.phase(p);
      if (f.u0 >= f.u1) continue;
      const int RB = row_bytes(f.cols, p == 1);
      const bool res = c.resident(p);
      const int R = c.ring_rows(p);
      // this warp's units: every eighth, counted over both phases
      const int n0 = (warp + kConsumers - nbase % kConsumers) % kConsumers;
      int u = f.u0 + n0;
      int slot = (nbase + n0) % a.stages;
      uint32_t parity = ((nbase + n0) / a.stages) & 1;
      ItemWalk it;
      int seg = f.seg_begin();
      SegPos at = f.at(seg);
      for (; seg * f.U < f.u1; ++seg, f.step(at)) {
        const int ub = min(f.u1, (seg + 1) * f.U);
        const int last_item = it.item;
        if (it.next(c, f, res, R, at)) {
          if (last_item >= 0) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[p][last_item % kItems]));
          }
          if (!warp_wait(sm.bfull[p][it.item % kItems], (it.item / kItems) & 1, abort, a.status))
            goto done;
        }
        if (u >= ub) continue;
        // two sums per tile, so that consecutive MMAs do not wait for each other
        float acc[2][NT][2][4] = {};
        const int n = c.item_rows(at.v), s0 = sm.vstart[at.v];
        const uint8_t* brow[NT];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int col = min(8 * nt + g, n - 1);  // columns past n repeat a row; nothing reads them
          brow[nt] = smem + (brow0 - ring) + c.row_slot(res, it.pos, R, s0, col) * RB + t * 16;
        }
        for (; u < ub; u += kConsumers) {
          const int boff = (u - seg * f.U) * (kUnitCols * 2);
          if (!warp_wait(sm.full[slot], parity, abort, a.status)) goto done;
          const uint8_t* base = smem + slot * kCodeBytes + (t >> 1) * kBoxBytes + g * 128;
          const uint8_t* sbase = smem + (srow0 - ring) + slot * kScaleBytes + g * 32 + 8 * t;
          uint2 s[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // rows g, g + 8, g + 16, g + 24
            const uint2 v = *reinterpret_cast<const uint2*>(sbase + i * 256);
            s[i] = t < 2 ? v : make_uint2(v.y, v.x);  // chunk order of lanes t >= 2
          }
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) {
            const int chunk = (((t & 1) * 4 + (jj ^ ((t >> 1) << 1))) ^ g) << 4;
            uint32_t cw[2][2][4], sw[2][2];
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int hi = 0; hi < 2; ++hi) {
                const uint4 x = *reinterpret_cast<const uint4*>(base + m * (2 * kBoxBytes) + hi * 1024 + chunk);
                cw[m][hi][0] = x.x, cw[m][hi][1] = x.y, cw[m][hi][2] = x.z, cw[m][hi][3] = x.w;
                const uint32_t word = jj < 2 ? s[2 * m + hi].x : s[2 * m + hi].y;
                sw[m][hi] = e4m3x2_half2((jj & 1) ? word >> 16 : word & 0xFFFFu);
              }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 b[NT];
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                b[nt] = *reinterpret_cast<const uint4*>(brow[nt] + boff + ((jj * 4 + i) << 6));
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                uint32_t lo[4], hi[4];
                const uint32_t sel = i < 2 ? 0x1010u : 0x3232u;
                e2m1x8_scaled(cw[m][0][i], __byte_perm(sw[m][0], 0u, sel), lo);
                e2m1x8_scaled(cw[m][1][i], __byte_perm(sw[m][1], 0u, sel), hi);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  mma_16816(acc[m][nt][0], lo[0], hi[0], lo[1], hi[1], b[nt].x, b[nt].y);
                  mma_16816(acc[m][nt][1], lo[2], hi[2], lo[3], hi[3], b[nt].z, b[nt].w);
                }
              }
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.empty[slot]));
          slot += kConsumers;
          if (slot >= a.stages) {
            slot -= a.stages;
            parity ^= 1;
          }
        }
        if (!warp_wait(sm.pempty[warp][pc & 1], ((pc >> 1) & 1) ^ 1, abort, a.status)) goto done;
        const uint32_t dst = pbuf + (2 * warp + (pc & 1)) * kPartBytes + lane * 16;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            sts128(dst + (m * NT + nt) * 512,
                   make_uint4(__float_as_uint(acc[m][nt][0][0] + acc[m][nt][1][0]),
                              __float_as_uint(acc[m][nt][0][1] + acc[m][nt][1][1]),
                              __float_as_uint(acc[m][nt][0][2] + acc[m][nt][1][2]),
                              __float_as_uint(acc[m][nt][0][3] + acc[m][nt][1][3])));
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.pfull[warp][pc & 1]));
        ++pc;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[p][it.item % kItems]));
      nbase += f.u1 - f.u0;
    }
  } else if (warp < kWarpEpilogue) {
    // ------------------------------------------------------------ producers
    const int pw = warp - kWarpProducer;  // this one's units: n = pw mod 2, counted over both phases
    int nbase = 0;
    bool ok = true;
    for (int p = 0; p < kPhases && ok; ++p) {
      const Phase f = c.phase(p);
      if (f.u0 >= f.u1) continue;
      const void* map = p == 0 ? &tm0 : &tm1;
      const Fp4Matrix& m = a.m[p];
      const int ng = f.cols >> 4;
      const int first = (pw + kProducers - nbase % kProducers) % kProducers;
      int slot = (nbase + first) % a.stages;
      uint32_t parity = (((nbase + first) / a.stages) & 1) ^ 1;
      int k = (f.u0 + first) % f.U;
      SegPos at = f.at((f.u0 + first) / f.U);
      for (int u = f.u0 + first; u < f.u1; u += kProducers) {
        if (!warp_wait(sm.empty[slot], parity, abort, a.status)) {
          ok = false;
          break;
        }
        const uint32_t bar = smem_u32(&sm.full[slot]);
        if (lane == 0) {
          const uint32_t dst = ring + slot * kCodeBytes;
          const int x = k * (kUnitCols / 2), r0 = (int)c.matrix_row(p, at, 0), r1 = (int)c.matrix_row(p, at, 16);
          if (k * kUnitCols + kUnitCols / 2 < f.cols) {  // both 256-column boxes hold columns
            mbar_arrive_expect_tx(bar, 4 * kBoxBytes);
            tma_load_2d(dst, map, bar, x, r0);
            tma_load_2d(dst + kBoxBytes, map, bar, x + 128, r0);
            tma_load_2d(dst + 2 * kBoxBytes, map, bar, x, r1);
            tma_load_2d(dst + 3 * kBoxBytes, map, bar, x + 128, r1);
          } else {
            mbar_arrive_expect_tx(bar, 2 * kBoxBytes);
            tma_load_2d(dst, map, bar, x, r0);
            tma_load_2d(dst + 2 * kBoxBytes, map, bar, x, r1);
          }
        }
        __syncwarp();
        {
          const int64_t row = c.matrix_row(p, at, lane);
          const bool in = MOE || row < m.rows;
          const uint8_t* src = m.scales + (in ? row * ng + 32 * k : 0);
          const int n = in ? min(32, ng - 32 * k) : 0;
          const uint32_t dst = srow0 + slot * kScaleBytes + lane * 32;
          if ((ng & 15) == 0)
            copy_scale_row<16>(dst, src, n);
          else if ((ng & 7) == 0)
            copy_scale_row<8>(dst, src, n);
          else if ((ng & 3) == 0)
            copy_scale_row<4>(dst, src, n);
          else {  // rows on odd multiples of two bytes: through registers
            for (int o = 0; o < 32; o += 4) {
              uint32_t w = 0u;
              if (o < n) w = __ldg(reinterpret_cast<const uint16_t*>(src + o));
              if (o + 2 < n) w |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(src + o + 2)) << 16;
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(dst + o), "r"(w) : "memory");
            }
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
        }
        slot += kProducers;
        if (slot >= a.stages) {
          slot -= a.stages;
          parity ^= 1;
        }
        k += kProducers;
        while (k >= f.U) {
          k -= f.U;
          f.step(at);
        }
      }
      if (ok) nbase += f.u1 - f.u0;
    }
    // no copy outlives the CTA, also when the other warps have given up: every
    // slot's last fill has arrived, or is waited for
    asm volatile("cp.async.wait_all;" ::: "memory");
    int none = 0;
    if (*abort && lane < a.stages)
      for (int parity = 0; parity < 2; ++parity)
        mbar_wait_bounded(smem_u32(&sm.full[lane]), parity, &none, nullptr, 100000000ull);
  } else if (warp == kWarpEpilogue) {
    // ------------------------------------------------------------- epilogue
    const int g = lane >> 2, t = lane & 3;
    int nbase = 0;
    int taken = 0;  // lane w: sums taken from warp w
    for (int v = lane; v < c.nv; v += 32)
      for (int p = 0; p < kPhases; ++p) sm.vglobal[p][v] = __ldg(&a.m[p].global[sm.vexp[v]]);
    __syncwarp();
    for (int p = 0; p < kPhases; ++p) {
      const Phase f = c.phase(p);
      const int64_t total = c.total_units(p);
      const bool res = c.resident(p);
      const int R = c.ring_rows(p);
      const int tu = f.tile_units();
      ItemWalk it;
      int seg = f.seg_begin();
      SegPos at = f.at(seg);
      bool fresh = true;  // first segment of a tile in this CTA
      for (; seg * f.U < f.u1; ++seg, f.step(at)) {
        const int ua = max(f.u0, seg * f.U), ub = min(f.u1, (seg + 1) * f.U);
        const int last_item = it.item;
        if (it.next(c, f, res, R, at) && last_item >= 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[p][last_item % kItems]));
        }
        float acc[2][NT][4] = {};
        const int cnt = min(ub - ua, kConsumers), w0 = (nbase + ua - f.u0) % kConsumers;
        for (int i = 0; i < cnt; ++i) {
          const int w = (w0 + i) % kConsumers, tk = __shfl_sync(0xFFFFFFFFu, taken, w);
          if (!warp_wait(sm.pfull[w][tk & 1], (tk >> 1) & 1, abort, a.status)) goto done;
          const uint32_t src = pbuf + (2 * w + (tk & 1)) * kPartBytes + lane * 16;
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
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.pempty[w][tk & 1]));
          if (lane == w) ++taken;
        }
        const int n = c.item_rows(at.v), s0 = sm.vstart[at.v];
        const float gl = sm.vglobal[p][at.v];
        // lane (g, t) holds rows g and g + 8 of tokens 8 nt + 2 t and + 1
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int col = 8 * nt + 2 * t + o;
            if (col < n) {
              const float rs = sm.rscale[p][c.row_slot(res, it.pos, R, s0, col)] * gl;
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                acc[m][nt][o] *= rs;
                acc[m][nt][2 + o] *= rs;
              }
            }
          }
        const int tile = p == 0 ? seg : at.j;
        const int64_t tb = (int64_t)tile * tu, te = tb + tu;  // the tile's units
        if (p == 1) {
          // out[token][row] over the tile's experts
          if (fresh) {
            for (int i = lane; i < a.T * kTile2; i += 32) (&sm.out[0][0])[i] = 0.f;
            __syncwarp();
          }
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int col = 2 * t + o;
            if (col < n) {
              const float w = sm.route_w[s0 + col];
              float* row = &sm.out[sm.route_tok[s0 + col]][32 * at.rb + g];
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                row[16 * m] = fmaf(w, acc[m][0][o], row[16 * m]);
                row[16 * m + 8] = fmaf(w, acc[m][0][2 + o], row[16 * m + 8]);
              }
            }
          }
          __syncwarp();
          fresh = false;
          if (ub < min((int64_t)f.u1, te)) continue;  // more of this tile to come
          fresh = true;
        }
        const bool whole = tb >= f.u0 && te <= f.u1;
        if (!whole) {
          // join: this CTA's share goes to its slot; whoever arrives last adds the shares in CTA order
          const int64_t G = Ctx::ctas(total);
          const int c0 = (int)(((tb + 1) * G - 1) / total), c1 = (int)((te * G - 1) / total);
          constexpr int kSlot0 = 512, kSlot1 = kFp4MaxTokens * kTile2;
          auto share = [&](int cta) {
            return a.part[p] + (size_t)(2 * cta + (cta == c0)) * (p == 0 ? kSlot0 : kSlot1);
          };
          float* mine = share(blockIdx.x);
          if (p == 1) {
            for (int tok = 0; tok < a.T; ++tok)
              __stcg(reinterpret_cast<float4*>(mine + tok * kTile2) + lane,
                     *reinterpret_cast<const float4*>(&sm.out[tok][4 * lane]));
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
              float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
              for (int i = c0; i <= c1; ++i) {
                const float4 z = __ldcg(reinterpret_cast<const float4*>(share(i) + tok * kTile2) + lane);
                s.x += z.x, s.y += z.y, s.z += z.z, s.w += z.w;
              }
              *reinterpret_cast<float4*>(&sm.out[tok][4 * lane]) = s;
            }
          } else {
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
                for (int i = c0; i <= c1; ++i) {
                  const float4 z = __ldcg(reinterpret_cast<const float4*>(share(i)) + (m * NT + nt) * 32 + lane);
                  s.x += z.x, s.y += z.y, s.z += z.z, s.w += z.w;
                }
                acc[m][nt][0] = s.x, acc[m][nt][1] = s.y, acc[m][nt][2] = s.z, acc[m][nt][3] = s.w;
              }
          }
        }
        if (p == 1) {
          __syncwarp();
          uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + kTile2 * at.j + 4 * lane;
          for (int tok = 0; tok < a.T; ++tok) {
            const float4 v = *reinterpret_cast<const float4*>(&sm.out[tok][4 * lane]);
            *reinterpret_cast<uint2*>(y + (int64_t)tok * a.m[1].rows) =
                make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
          }
          __syncwarp();
          continue;
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int col = 8 * nt + 2 * t + o;
            if (MOE) {
              // 16 values of h: half times 2^s of their largest, and s
              const float h0 = swiglu(acc[0][nt][o], acc[1][nt][o]);
              const float h1 = swiglu(acc[0][nt][2 + o], acc[1][nt][2 + o]);
              float m = fmaxf(fabsf(h0), fabsf(h1));
#pragma unroll
              for (int x = 4; x <= 16; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, x));
              const int s = row_exponent(m);
              if (col < n) {
                const int I = a.m[1].cols;
                uint8_t* rec = a.h + (int64_t)sm.route_id[s0 + col] * record_bytes(I);
                const uint32_t b = half2_bits(h0 * pow2f(s), h1 * pow2f(s));
                uint16_t* hv = reinterpret_cast<uint16_t*>(rec) + 16 * at.j + g;
                hv[0] = (uint16_t)b;
                hv[8] = (uint16_t)(b >> 16);
                if (g == 0) reinterpret_cast<int8_t*>(rec)[2 * I + at.j] = (int8_t)s;
              }
            } else if (col < n) {
              const int64_t to = (int64_t)(s0 + col) * a.m[0].rows;
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int hi = 0; hi < 2; ++hi) {
                  const int row = 32 * at.j + 16 * m + 8 * hi + g;
                  if (row >= a.m[0].rows) continue;
                  const float val = acc[m][nt][2 * hi + o];
                  if (a.f32)
                    reinterpret_cast<float*>(a.y)[to + row] = val;
                  else
                    reinterpret_cast<uint16_t*>(a.y)[to + row] = pack_bf16x2(val, 0.f) & 0xFFFFu;
                }
            }
          }
      }
      if (f.u0 < f.u1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[p][it.item % kItems]));
      }
      if (MOE && p == 0) {  // every h value of this CTA is stored, also for bulk copies
        fence_proxy_async_global();
        __threadfence();
        __syncwarp();
        if (lane == 0) atomicAdd(&a.ctl[0], 1u);
      }
      nbase += f.u1 - f.u0;
    }
  } else {
    // -------------------------------------------------------------- loaders
    const int lw = warp - kWarpLoader;
    uint32_t raw_parity = 0;
    for (int p = 0; p < kPhases; ++p) {
      const Phase f = c.phase(p);
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
          fence_proxy_async_global();
        }
        if (!__shfl_sync(0xFFFFFFFFu, (int)ok, 0)) goto done;
      }
      if (f.u0 >= f.u1) continue;
      const int RB = row_bytes(f.cols, p == 1);
      if (c.resident(p)) {
        // all loader warps work on each row where there are few; a warp that gives
        // up on its copy still meets the others at their barrier
        bool ok = true;
        if (a.T < kLoaders) {
          for (int r = 0; r < a.T; ++r)
            ok &= fill_x<kLoaders>(a.x + r * a.ldx, f.cols, brow0 + r * RB, lw, sm.raw[0], raw_parity,
                                   sm.red, &sm.rscale[0][r], abort, a.status);
          // from here every warp has a barrier of its own
          if (lw > 0) raw_parity = 0;
        } else {
          for (int r = lw; r < a.T && ok; r += kLoaders)
            ok = fill_x<1>(a.x + r * a.ldx, f.cols, brow0 + r * RB, 0, sm.raw[lw], raw_parity, sm.red,
                           &sm.rscale[0][r], abort, a.status);
        }
        if (!ok) goto done;
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
        int seg = f.seg_begin();
        SegPos at = f.at(seg);
        for (; seg * f.U < f.u1; ++seg, f.step(at)) {
          if (!it.next(c, f, false, R, at)) continue;
          while (used + it.rows > R || it.item - oldest >= kItems)
            if (!retire()) goto done;
          used += it.rows;
#pragma unroll
          for (int i = 0; i < kItems; ++i)
            if (i == it.item % kItems) rows_of[i] = it.rows;
          for (int r = 0; r < it.rows; ++r, ++counter)
            if (counter % kLoaders == lw) {
              const int s = sm.vstart[at.v] + r, place = c.row_slot(false, it.pos, R, 0, r);
              const bool ok =
                  p == 0 ? fill_x<1>(a.x + sm.route_tok[s] * a.ldx, f.cols, brow0 + place * RB, 0,
                                     sm.raw[lw], raw_parity, sm.red, &sm.rscale[0][place], abort, a.status)
                         : fill_h(a.h + (int64_t)sm.route_id[s] * record_bytes(f.cols), f.cols,
                                  brow0 + place * RB, sm.raw[lw], raw_parity, &sm.rscale[1][place], abort,
                                  a.status);
              if (!ok) goto done;
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
  return kMaxSmem - (int)sizeof(Fp4Shared) - 2048 - 2 * kConsumers * 2 * nt * 512 -
         kConsumers * kStageBytes;  // the least number of stages
}

static void fp4_finish_plan(Fp4Plan* p) {
  p->b_bytes = (p->b_bytes + 127) / 128 * 128;
  const int left = fp4_row_budget(p->nt) - p->b_bytes;
  p->stages = left >= kConsumers * kStageBytes ? kMaxStages : kConsumers;
  p->smem = 1024 + p->stages * kStageBytes + p->b_bytes + 2 * kConsumers * 2 * p->nt * 512;
}

// The layer: tokens in groups of at most 8.
static Fp4Plan fp4_plan_layer(int H, int I, int T, int K) {
  Fp4Plan p = {8, 1, 0, 0, 0};
  const int budget = fp4_row_budget(1) / 128 * 128, r1 = row_bytes(H, false), r2 = row_bytes(I, true);
  if (budget / r1 < p.group) p.group = budget / r1;
  if (budget / r2 < p.group) p.group = budget / r2;
  // x: T rows, or one group's; h: two groups' or all, as far as they fit
  const int n1 = (int64_t)T * r1 <= budget ? T * r1 : p.group * r1;
  int rows2 = T * K < 2 * p.group ? T * K : 2 * p.group;
  if (rows2 > budget / r2) rows2 = budget / r2;
  p.b_bytes = n1 > rows2 * r2 ? n1 : rows2 * r2;
  fp4_finish_plan(&p);
  return p;
}

// The linear: one sweep over the matrix for up to 16 tokens where their rows
// fit, else equal groups, each with its own sweep (the second from L2, where
// the matrix fits there).
static Fp4Plan fp4_plan_linear(int cols, int T) {
  Fp4Plan p = {0, 1, 0, 0, 0};
  const int rb = row_bytes(cols, false);
  const int fit1 = fp4_row_budget(1) / 128 * 128 / rb, fit2 = fp4_row_budget(2) / 128 * 128 / rb;
  const int most = fit2 > 8 ? (fit2 < 16 ? fit2 : 16) : (fit1 < 8 ? fit1 : 8);
  const int groups = (T + most - 1) / most;
  p.group = (T + groups - 1) / groups;
  p.nt = p.group > 8 ? 2 : 1;
  const int budget = fp4_row_budget(p.nt) / 128 * 128;
  p.b_bytes = (int64_t)T * rb <= budget ? T * rb : p.group * rb;
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
  float* part[2];
  uint8_t* h;
};

namespace {

// Workspace: a line for the status word, counters, the cut tiles' shares, h.
constexpr size_t kFp4Align = 256;
constexpr size_t kFp4Ctl = 2048;
constexpr size_t kFp4Part0 = (size_t)kFp4Grid * 2 * 512 * 4;
constexpr size_t kFp4Part1 = (size_t)kFp4Grid * 2 * kFp4MaxTokens * kTile2 * 4;
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
  h->part[0] = reinterpret_cast<float*>(b + kFp4Align + kFp4Ctl);
  h->part[1] = reinterpret_cast<float*>(b + kFp4Align + kFp4Ctl + kFp4Part0);  // the layer
  h->h = b + kFp4Align + kFp4Ctl + kFp4Part0 + kFp4Part1;
  return cudaMemsetAsync(b, 0, kFp4Align + kFp4Ctl, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

extern "C" {

moe_status moe_fp4_workspace_query(const moe_dims* dims, int64_t max_tokens, size_t* workspace_bytes) {
  if (!dims || !workspace_bytes || max_tokens < 1) return MOE_ERR_INVALID_ARG;
  if (!fp4_dims_ok(dims) || max_tokens > kFp4MaxTokens) return MOE_ERR_UNSUPPORTED;
  *workspace_bytes = 2 * kFp4Align + kFp4Ctl + kFp4Part0 + kFp4Part1 +
                     (size_t)max_tokens * dims->top_k * record_bytes(dims->inter);
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
  a.part[0] = h->part[0];
  a.part[1] = h->part[1];
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
  *workspace_bytes = 2 * kFp4Align + kFp4Ctl + kFp4Part0;
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
  a.part[0] = h->part[0];
  a.part[1] = h->part[1];
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
