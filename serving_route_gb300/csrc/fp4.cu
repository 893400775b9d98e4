// fp4.cu -- few tokens on NVFP4 weights (E2M1 codes, an E4M3 scale per 16
// columns, a float scale per matrix): products of 1..16 vectors with one
// matrix (moe_fp4_linear) and the whole MoE layer (moe_fp4_forward), each one
// persistent kernel.
//
//   v = e2m1(code) * e4m3(block scale) * global
//   linear: y = x W^T;   layer: out_t = sum_k w_tk * W2[e] (silu(g) * u),
//   (g; u) = W1[e] x_t, e = topk_idx[t, k].
//
// What bounds it: the weights, 9/16 byte each, are read once and used for a few
// tokens, so the floor is their time through HBM.  At the copy rate an SM gets
// about 42 weights a clock; dequantising them costs one convert and one product
// per two weights, which is as much again, so the two have to overlap.  Measured
// for the layer of 256 experts, H 7168, I 2048, 16 tokens (2.52 GB): copies alone
// 374 us, products alone 374 us, the kernel 385 to 428 us, 5.9 to 6.5 TB/s.
//   * four code pairs of a 32-bit word become half2 with one hardware convert
//     each, one half2 product applies the E4M3 scale (6 significant bits: both
//     exact in half), and m16n8k16 half MMAs with float accumulators take 8
//     tokens as their N side: the weights go from registers to the tensor cores,
//     which are busy for 7% (linear) to 25% (layer) of the time.  (A tensor-memory
//     MMA could take them from tensor memory, with 8 or 16 tokens as N, after a
//     store to it instead of the operand registers: not tried.)  The
//     checkpoint's order is kept: lane (g, t) owns 128 consecutive columns of
//     rows g and g + 8, so a 16-byte load of codes feeds eight MMAs of its own,
//     and x is stored in shared memory in the order in which the lanes need it.
//   * x (BF16) and h (float) enter as half, each row multiplied by the power of
//     two that brings its largest value to [2^14, 2^15): for BF16 values exact
//     down to 2^-32 of the row's largest, below that rounded at 2^-40 of it; h
//     is rounded to 11 bits, or at 2^-39 of its row's largest value where that is
//     more: half is what the MMA takes, and of BF16 outputs the error against 64 bits
//     is 0.00167 with it, 0.00166 with a float h.  The inverse is applied to the float sums.
//   * a place of the shared-memory ring is one consumer warp's unit of work, 32
//     rows x 512 columns: 8 KB of codes, copied by TMA as stored, and 1 KB of
//     scales by asynchronous copies (their rows need not be multiples of 16
//     bytes).  Eight warps take the units in turn, so no barrier but the unit's
//     own stands between the copies and the MMAs; 12 to 16 places are in flight.
//   * every CTA owns one contiguous range of a phase's units; a tile that a
//     range's end cuts is joined from float partial sums by whichever CTA
//     finishes it last, in the order of the CTAs, so that results never change.
//   * the layer is one cooperative launch: FC1 units, a grid barrier on h, FC2
//     units.  The weights' copies do not wait at the barrier: the ring fills
//     with FC2 weights while the last FC1 sums and h are on their way.
// Where one token's 46 us go (H 7168, I 2048, 8 of 256 experts; 29.2 us at the copy
// rate): tables and the first copies 4.7 us, FC1 to 24, its last sums and the barrier
// to 28.2, h rows to 30.3, FC2 to 40, joining and leaving to 43, the launch.  FC2
// there is bound by its products (its first third is in the ring before the barrier
// opens; sending the rest to L2 ahead made it slower).  The linear (4096 x 7168, one
// token: 7.5 us, 2.4 at the copy rate) is bound by the same start, one tile's products
// and the launch.
#include <cudaTypedefs.h>

#include <cstring>
#include <new>
#include <type_traits>

#include <cuda_fp16.h>

#include "common.cuh"
#include "internal.h"

namespace mm {

constexpr int kFp4MaxTokens = 16;
constexpr int kFp4MaxRoutes = 128;
constexpr int kFp4Grid = 152;        // one CTA per SM
constexpr int kCtlPoison = 2 + 2 * kFp4Grid;  // not 0: a wait ran out, the counters may not be at zero
// The warps' roles.  More service warps than copies need by their number: each
// wait and each copy is a chain of round trips, and several chains overlap (two
// copying warps 449 us, four 409, at 16 tokens; one finishing FC1's tiles 36.9, two
// 35.6, at 3 tokens of H 2048, I 1408, 64 experts).
constexpr int kEpilogues = 2;        // add the consumers' sums, finish and join tiles: in turn, the
                                     // second phase's tiles by the first of them
constexpr int kProducers = 4;        // issue the copies of the weights, in turn
constexpr int kLoaders = 2;          // x and h rows to half in shared memory
constexpr int kConsumers = 8;        // dequantise and multiply
constexpr int kWarpEpilogue = 0;
constexpr int kWarpProducer = kWarpEpilogue + kEpilogues;
constexpr int kWarpLoader = kWarpProducer + kProducers;
constexpr int kWarpConsumer = kWarpLoader + kLoaders;
constexpr int kFp4Threads = 32 * (kWarpConsumer + kConsumers);
// Units in flight: at least what covers the latency of HBM at the copy rate; a
// multiple of kProducers, so that each place is one producer's (another one could
// wait for a phase two laps ahead, whose parity is that of the lap before)
constexpr int kMinStages = 12, kMaxStages = 16;
constexpr int kUnitCols = 512;
constexpr int kCodeBytes = 32 * kUnitCols / 2;
constexpr int kScaleBytes = 32 * kUnitCols / 16;
constexpr int kUnitBytes = kCodeBytes + kScaleBytes;
constexpr int kBoxBytes = 16 * 128;  // 16 rows x 256 columns
constexpr int kItems = 8;            // operand items in flight (rows ring)
// Ranges are cut within tiles where whole tiles would leave the fullest CTA with more
// than this many units above the mean: a join takes about 3 us, 15 units of copies (one
// token of H 7168, I 2048; other borders have not been measured)
constexpr int kCutUnits = 15;
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
  uint32_t* ctl;        // [0] barrier, [1] warps past it, [2 + 152 p + c] joins of phase p, kCtlPoison
  float* part[2];       // by phase, [152][2][..]: a CTA's cut tiles, first and last
  int T, E, K;
  int k_rcp;            // floor(2^16 / K) + 1: quotients of numbers below 128
  // how shared memory is divided: tokens of one operand item (at most 8 NT), bytes of
  // operand rows, places of the ring.  The layer may have a second division (group 0:
  // it has not), of which the routes choose.
  int group[2], b_bytes[2], stages[2];
  int group_rcp[2];     // as k_rcp
  uint32_t grid_rcp;    // floor(2^32 / CTAs) + 1
  uint64_t wait_ns;     // limit of every wait
  bool check, f32, watchdog_test;
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

// Where a walk over a phase stands: item v's product with the rows of tile j.
struct TilePos {
  int v, j;
};

// One phase of one CTA: units [u0, u1) in the order
//   first phase   item, tile: a tile is 32 matrix rows, U units of 512 columns;
//                 the CTA's n-th unit is warp n mod 8's.
//   second phase  tile, item: a tile is 128 rows, an item's share of it four
//                 blocks of 32 rows of U units.  Warp w has one half of block
//                 w / 2's units, so that few sums are to be added (I / 512 units
//                 are few), and the i-th units of the eight warps follow each
//                 other, so that none holds a place of the ring for long.
struct Phase {
  int p, U, RT, nv, u0, u1, cols;
  // the CTAs' shares: steps of `stride` units, `base` or (the first `extra` CTAs)
  // one more of them
  int stride, base, extra;
  TilePos start;  // the visit that u0 lies in, and its units before u0
  int ka;
  // the CTA that holds unit u
  __device__ int cta_of(int u) const {
    const int s = u / stride, big = extra * (base + 1);
    return s < big ? s / (base + 1) : extra + (s - big) / base;
  }
  __device__ int visit() const { return p == 0 ? U : 4 * U; }  // units of an item at a tile
  __device__ void step(TilePos& s) const {
    if (p == 0) {
      if (++s.j == RT) {
        s.j = 0;
        ++s.v;
      }
    } else if (++s.v == nv) {
      s.v = 0;
      ++s.j;
    }
  }
  // second phase: the i-th unit in order is warp w's with columns from 512 k
  __device__ void unit_of(int i, int& w, int& k) const {
    const int full = U >> 1, r = i >> 3;  // rounds in which all eight warps have a unit
    w = r < full ? i & 7 : 2 * (i - 8 * full);
    k = (w & 1) * (U - full) + (r < full ? r : full);
  }
  __device__ int tile_units() const { return p == 0 ? U : nv * 4 * U; }
};

// Codes as TMA tensors.  unit: 128-byte (256-column) blocks of the rows, a box is
// a unit's 32 rows x 2 blocks, block-major ({128 B, row, block}; FC1: {128 B, row
// of the half, gate or up, block, expert}).  box: the rows as they are, a box is
// 16 rows x 128 B.  128-byte swizzle; what lies past an extent reads as zero.
struct Fp4Maps {
  CUtensorMap unit[2], box[2];
};

// What bounds every wait: the CTA's abort flag (when one warp gives up the others
// do), the status word that it marks, and the time.  In shared memory, so that it
// costs registers only where a warp does wait.
struct WaitLimit {
  int abort;
  uint32_t* status;
  uint64_t ns;
};

struct Fp4Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t bfull[2][kItems], bempty[2][kItems];
  uint64_t raw[kLoaders], go;
  alignas(16) float out[kFp4MaxTokens][kTile2];
  alignas(16) int key[kFp4MaxRoutes];
  float rscale[2][kFp4MaxRoutes];       // per operand row: 2^-s
  float vglobal[2][kFp4MaxRoutes];      // the items' matrix scales
  float route_w[kFp4MaxRoutes];         // by sorted position, as the next ones
  int16_t route_e[kFp4MaxRoutes], route_id[kFp4MaxRoutes], route_tok[kFp4MaxRoutes];
  int16_t vstart[kFp4MaxRoutes + 1];    // first sorted position of every item
  int16_t vexp[kFp4MaxRoutes];
  uint8_t first[kFp4MaxRoutes];
  uint32_t row_max[kFp4MaxTokens];
  int warp_cnt[2][4], warp_live[4];
  uint32_t warp_bits[4];
  Phase phase[2];
  int issued[kProducers];               // units each producer has begun
  int done[kConsumers];                 // sums each consumer has left
  int taken[kConsumers][2];             // by place of a sum: how many were taken from it
  int nv, plan;
  WaitLimit lim;
};

template <bool MOE, int NT>
struct Fp4Ctx {
  const Fp4Args& a;
  Fp4Shared& sm;
  int nv;

  // n over the grid's CTAs, n below 2^32: the reciprocal's quotient is right or one too many
  __device__ uint32_t per_cta(uint32_t n) const {
    const uint32_t q = __umulhi(n, a.grid_rcp);
    return q * gridDim.x > n ? q - 1 : q;
  }
  // (units: below 2^30, also the linear's in 16 groups.  Divisions cost about 0.1 us each
  // here, where everyone waits: few, and once for all roles)
  __device__ Phase make_phase(int p) const {
    Phase f;
    f.p = p;
    f.cols = a.m[p].cols;
    f.U = padded_units(f.cols);
    f.RT = (a.m[p].rows + 31) / 32;
    f.nv = nv;
    // whole tiles, unless the CTA with one more than the others would work
    // longer than a join takes
    const int G = gridDim.x, tiles = p == 0 ? nv * f.RT : f.RT >> 2, tu = f.tile_units(), n = tiles * tu;
    const bool whole = (int)(per_cta(tiles + G - 1) * tu - per_cta(n + G - 1)) <= kCutUnits;
    f.stride = whole ? tu : p == 0 ? 1 : f.visit();
    const int steps = whole ? tiles : p == 0 ? n : nv * tiles;
    f.base = per_cta(steps);
    f.extra = steps - f.base * G;
    const int b = blockIdx.x, step0 = b * f.base + min(b, f.extra);
    f.u0 = step0 * f.stride;
    f.u1 = f.u0 + (f.base + (b < f.extra)) * f.stride;
    if (whole && p == 1) {
      f.ka = 0;
      f.start = {0, step0};
    } else {  // a step is a tile, a unit or an item's visit
      const int i = whole || p == 1 ? step0 : step0 / f.U, inner = p == 0 ? f.RT : nv, o = i / inner;
      f.ka = f.u0 - i * f.visit();
      f.start = p == 0 ? TilePos{o, i - o * inner} : TilePos{i - o * inner, o};
    }
    return f;
  }
  __device__ const Phase& phase(int p) const { return sm.phase[p]; }
  __device__ int b_bytes() const { return MOE && sm.plan ? a.b_bytes[1] : a.b_bytes[0]; }

  __device__ int item_rows(int v) const { return sm.vstart[v + 1] - sm.vstart[v]; }
  // x rows stay for the whole phase where all of them fit; h rows always pass
  // through the ring, so that the first item waits for its own rows only
  __device__ bool resident(int p) const {
    return p == 0 && (int64_t)a.T * row_bytes(a.m[0].cols, false) <= b_bytes();
  }
  __device__ int ring_rows(int p) const {
    return min(b_bytes() / row_bytes(a.m[p].cols, p == 1), kFp4MaxRoutes);
  }
  // place of an item's column among the operand rows
  __device__ int row_slot(bool resident, int pos, int R, int s0, int col) const {
    if (resident) return sm.route_tok[s0 + col];
    return pos + col < R ? pos + col : pos + col - R;
  }
  // matrix row of row r of a tile (0..31, second phase 0..127)
  __device__ int64_t matrix_row(int p, const TilePos& s, int r) const {
    if (!MOE) return 32 * (int64_t)s.j + r;
    const int64_t base = (int64_t)sm.vexp[s.v] * a.m[p].rows;
    if (p == 0)  // 16 gate rows, then their 16 up rows
      return base + (r < 16 ? 16 * s.j + r : a.m[0].rows / 2 + 16 * s.j + r - 16);
    return base + kTile2 * s.j + r;
  }
};

// Walks the operand items of a phase in the order of its visits.  Resident: all rows stay
// for the phase and there is one item.  Ring: an item is the rows of one token
// group, for its tiles in a row (first phase) or for one tile, at consecutive ring places.
struct ItemWalk {
  int item = -1, v = -1, j = -1, pos = 0, rows = 0;
  // whether a new item starts at s
  template <class Ctx>
  __device__ bool next(const Ctx& c, const Phase& f, bool resident, int R, const TilePos& s) {
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

// Four E2M1 pairs (one 32-bit word, low nibble first) times one half of the scale pair s.
template <int HI>
__device__ __forceinline__ void e2m1x8_scaled(uint32_t w, uint32_t s, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
  const __half2 sp = *reinterpret_cast<const __half2*>(&s), sd = HI ? __high2half2(sp) : __low2half2(sp);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 p = __hmul2(*reinterpret_cast<const __half2*>(&h[i]), sd);
    h[i] = *reinterpret_cast<const uint32_t*>(&p);
  }
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

// TMA loads and copies with an L2 policy: the weights pass once, and what else the
// kernel reads (instructions, x, h, tables) should stay.
__device__ __forceinline__ uint64_t policy_evict_first() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}

__device__ __forceinline__ void load_box_2d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4}], [%2], %5;" ::"r"(dst),
      "l"((uint64_t)map), "r"(bar), "r"(c0), "r"(c1), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void load_box_3d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1,
                                            int c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(dst),
      "l"((uint64_t)map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void load_box_5d(uint32_t dst, const void* map, uint32_t bar, int c0, int c1,
                                            int c2, int c3, int c4, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2], %8;" ::"r"(dst),
      "l"((uint64_t)map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "l"(policy)
      : "memory");
}

// Asynchronous copy of N bytes, of which the first `valid` are read and the rest zero.
template <int N>
__device__ __forceinline__ void cp_async(uint32_t dst, const void* src, int valid, uint64_t policy) {
  if (N == 16)
    asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2, %3;" ::"r"(dst), "l"(src),
                 "r"(valid), "l"(policy)
                 : "memory");
  else
    asm volatile("cp.async.ca.shared.global.L2::cache_hint [%0], [%1], %4, %2, %3;" ::"r"(dst), "l"(src),
                 "r"(valid), "l"(policy), "n"(N)
                 : "memory");
}

// The 32 scale bytes of one row of a unit (n of them in the matrix, the rest
// zero) to shared memory, in copies as wide as the rows' alignment allows.
template <int N>
__device__ __forceinline__ void copy_scale_row(uint32_t dst, const uint8_t* src, int n, uint64_t policy) {
#pragma unroll
  for (int o = 0; o < 32; o += N) {
    const int v = min(max(n - o, 0), N);
    cp_async<N>(dst + o, v > 0 ? src + o : src, v, policy);
  }
}

__device__ __forceinline__ bool gave_up(const WaitLimit& lim) {
  return *const_cast<const volatile int*>(&lim.abort) != 0;
}

// Counts in shared memory that one warp raises and others wait for: cheaper than
// an mbarrier where lanes wait on different ones.
__device__ __forceinline__ int load_count(const int* count) {
  int v;
  asm volatile("ld.acquire.cta.shared.s32 %0, [%1];" : "=r"(v) : "r"(smem_u32(count)) : "memory");
  return v;
}

__device__ __forceinline__ void store_count(int* count, int v) {
  asm volatile("st.release.cta.shared.s32 [%0], %1;" ::"r"(smem_u32(count)), "r"(v) : "memory");
}

__device__ __noinline__ bool wait_count_slow(const int* count, int n, WaitLimit& lim) {
  const uint64_t t0 = globaltimer_ns();
  bool ok;
  while (!(ok = __all_sync(0xFFFFFFFFu, load_count(count) >= n))) {
    if (__any_sync(0xFFFFFFFFu, gave_up(lim))) break;
    if (__any_sync(0xFFFFFFFFu, globaltimer_ns() - t0 > lim.ns)) {
      lim.abort = 1;
      record_status(lim.status, MOE_DEV_TIMEOUT);
      break;
    }
  }
  __syncwarp();
  return ok;
}

// Bounded wait of a whole warp until every lane's count has reached its n.
__device__ __forceinline__ bool wait_count(const int* count, int n, WaitLimit& lim) {
  if (__all_sync(0xFFFFFFFFu, load_count(count) >= n)) {
    __syncwarp();
    return true;
  }
  return wait_count_slow(count, n, lim);
}

__device__ __noinline__ bool bar_wait_slow(uint32_t bar, uint32_t parity, WaitLimit& lim) {
  return mbar_wait_bounded(bar, parity, &lim.abort, lim.status, lim.ns);
}

// Bounded wait of a whole warp: all of its lanes go on, or none.
__device__ __forceinline__ bool warp_wait(uint64_t& bar, uint32_t parity, WaitLimit& lim) {
  const uint32_t b = smem_u32(&bar);
  return __all_sync(0xFFFFFFFFu, mbar_test_wait(b, parity) || bar_wait_slow(b, parity, lim));
}

// The same for copies in flight to this CTA's memory, which must not outlive it: whoever
// gives up for another reason still gives them a while.
__device__ __forceinline__ bool copy_wait(uint64_t& bar, uint32_t parity, WaitLimit& lim) {
  if (warp_wait(bar, parity, lim)) return true;
  int none = 0;
  mbar_wait_bounded(smem_u32(&bar), parity, &none, nullptr, 100000000ull);
  return false;
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

// A row's scale 2^-s as the product of two normal numbers near its root: sums are multiplied
// by the first (exactly: they lie between 2^-34 and 2^42, or are 0), the matrix's scale by
// the second.  The product of the whole 2^-s and the matrix's scale may be subnormal
// although the result is not (x near 2^-112, say).
__device__ __forceinline__ float2 root_scales(float rscale) {
  const uint32_t e = __float_as_uint(rscale), one = 0x3F800000u, root = ((e + one) >> 1) & 0x7F800000u;
  return make_float2(__uint_as_float(root), __uint_as_float(e - root + one));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 p = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Before bulk copies of `bytes` to places that were read and written through the
// generic proxy before: a fence orders them.
__device__ __forceinline__ void raw_begin(uint64_t& bar, uint32_t bytes) {
  fence_proxy_async_smem();
  mbar_arrive_expect_tx(smem_u32(&bar), bytes);
}

// The largest magnitudes of BF16 values, in pairs.  NaN does not set the scale (it
// stays NaN in half); infinity does.
__device__ __forceinline__ uint32_t max_bf16x8(const uint4 v, uint32_t m) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[i] & 0x7FFF7FFFu));
  return m;
}

// The larger of a pair, over the warp, as BF16 bits.
__device__ __forceinline__ uint32_t warp_max_pair(uint32_t m) {
  return __reduce_max_sync(0xFFFFFFFFu, max(m & 0xFFFFu, m >> 16));
}

__device__ __forceinline__ uint4 bf16x8_to_half(const uint4 v, float up) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    h[i] = half2_bits(__uint_as_float(w[i] << 16) * up, __uint_as_float(w[i] & 0xFFFF0000u) * up);
  return make_uint4(h[0], h[1], h[2], h[3]);
}

// The two pieces of unit u that are this lane's, of a row of n pieces (zeros past them).
__device__ __forceinline__ void load_pieces(uint32_t row, int u, int n, uint4 (&v)[2]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int q = 64 * u + 32 * k + lane;
    v[k] = q < n ? lds128(row + 16 * q) : make_uint4(0u, 0u, 0u, 0u);
  }
}

__device__ __forceinline__ void turn_unit(uint32_t row, int u, uint4 (&v)[2], float up) {
  const int lane = threadIdx.x & 31;
  __syncwarp();  // all of the unit is in registers
#pragma unroll
  for (int k = 0; k < 2; ++k)
    sts128(row + u * (kUnitCols * 2) + piece_offset(32 * k + lane), bf16x8_to_half(v[k], up));
}

// One x row (cols BF16 values, a multiple of 32) by one warp: copied as it is,
// then turned in place, unit by unit, to half times 2^s with zeros up to the
// unit's end.
__device__ __forceinline__ bool fill_x(const uint16_t* src, int cols, uint32_t dst, uint64_t& bar,
                                       uint32_t& parity, float* rscale, WaitLimit& lim,
                                       uint64_t* go) {
  const int lane = threadIdx.x & 31, n = cols >> 3, U = padded_units(cols);
  if (lane == 0) {
    raw_begin(bar, cols * 2);
    bulk_load(dst, src, cols * 2, smem_u32(&bar));
    if (go) mbar_arrive(smem_u32(go));
  }
  if (!copy_wait(bar, parity, lim)) return false;
  parity ^= 1;
  uint32_t m = 0u;
#pragma unroll 2
  for (int u = 0; u < U; ++u) {
    uint4 v[2];
    load_pieces(dst, u, n, v);
    m = max_bf16x8(v[1], max_bf16x8(v[0], m));
  }
  const int s = row_exponent(__uint_as_float(warp_max_pair(m) << 16));
  if (lane == 0) *rscale = pow2f(-s);
  for (int u = 0; u < U; ++u) {
    uint4 v[2];
    load_pieces(dst, u, n, v);
    turn_unit(dst, u, v, pow2f(s));
  }
  return true;
}

// All T rows of a resident phase by `warps` warps, this one the rank-th: their
// copies have been asked for on `bar`.  Every warp meets the others at both
// barriers, also one that gave up on the copies.
__device__ __forceinline__ bool fill_x_rows(int T, int cols, uint32_t rows, int pitch, int rank, int warps,
                                            uint64_t& bar, uint32_t* row_max, float* rscale,
                                            WaitLimit& lim) {
  const int lane = threadIdx.x & 31, n = cols >> 3, U = padded_units(cols);
  const bool ok = copy_wait(bar, 0, lim);
  // (two units at a time)
  for (int i = rank; i < T * U; i += 2 * warps) {
    const int t0 = i / U, j = i + warps, t1 = j / U;
    uint4 v[2], w[2];
    load_pieces(rows + t0 * pitch, i - t0 * U, n, v);
    if (j < T * U) load_pieces(rows + t1 * pitch, j - t1 * U, n, w);
    const uint32_t m = warp_max_pair(max_bf16x8(v[1], max_bf16x8(v[0], 0u)));
    if (lane == 0) atomicMax(&row_max[t0], m);
    if (j < T * U) {
      const uint32_t m1 = warp_max_pair(max_bf16x8(w[1], max_bf16x8(w[0], 0u)));
      if (lane == 0) atomicMax(&row_max[t1], m1);
    }
  }
  asm volatile("bar.sync 1, %0;" ::"r"(32 * warps) : "memory");
  for (int i = rank; i < T * U; i += 2 * warps) {
    const int t0 = i / U, u0 = i - t0 * U, j = i + warps, t1 = j / U, u1 = j - t1 * U;
    uint4 v[2], w[2];
    load_pieces(rows + t0 * pitch, u0, n, v);
    if (j < T * U) load_pieces(rows + t1 * pitch, u1, n, w);
    const int s0 = row_exponent(__uint_as_float(row_max[t0] << 16));
    if (u0 == 0 && lane == 0) rscale[t0] = pow2f(-s0);
    turn_unit(rows + t0 * pitch, u0, v, pow2f(s0));
    if (j < T * U) {
      const int s1 = row_exponent(__uint_as_float(row_max[t1] << 16));
      if (u1 == 0 && lane == 0) rscale[t1] = pow2f(-s1);
      turn_unit(rows + t1 * pitch, u1, w, pow2f(s1));
    }
  }
  asm volatile("bar.sync 1, %0;" ::"r"(32 * warps) : "memory");
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
                                       uint32_t& parity, float* rscale, WaitLimit& lim) {
  const int lane = threadIdx.x & 31, n = cols >> 3, U = padded_units(cols);
  const uint32_t ex = dst + U * (kUnitCols * 2);
  if (lane == 0) {
    raw_begin(bar, record_bytes(cols));
    bulk_load(dst, src, cols * 2, smem_u32(&bar));
    bulk_load(ex, src + cols * 2, exponent_bytes(cols), smem_u32(&bar));
  }
  if (!copy_wait(bar, parity, lim)) return false;
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
  for (int u0 = 0; u0 < U; u0 += 2) {
    uint4 v[2][2];
    int d[2][2];
#pragma unroll
    for (int o = 0; o < 2; ++o)
      if (u0 + o < U) {
        load_pieces(dst, u0 + o, n, v[o]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int q = 64 * (u0 + o) + 32 * k + lane;
          d[o][k] = q < n ? exponent(q >> 1) - s : 0;
        }
      }
    __syncwarp();
#pragma unroll
    for (int o = 0; o < 2; ++o)
      if (u0 + o < U) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const uint32_t f1 = half_pow2_neg(min(d[o][k], 14)), f2 = half_pow2_neg(d[o][k] - min(d[o][k], 14));
          uint32_t w[4] = {v[o][k].x, v[o][k].y, v[o][k].z, v[o][k].w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(f1));
            asm("mul.rn.f16x2 %0, %0, %1;" : "+r"(w[i]) : "r"(f2));
          }
          sts128(dst + (u0 + o) * (kUnitCols * 2) + piece_offset(32 * k + lane),
                 make_uint4(w[0], w[1], w[2], w[3]));
        }
      }
  }
  return true;
}

// Sorted routes, and the items: runs of at most `group` tokens of one expert (the
// linear: groups of tokens).  By the first 128 threads; e, w: the thread's route; bad:
// status bits that the first CTA's first thread adds.
template <bool MOE>
__device__ __forceinline__ void build_items(const Fp4Args& a, Fp4Shared& sm, int e, float w, uint32_t bad) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (!MOE) {
    if (tid == 0) {
      int v = 0;
      for (int t = 0; t < a.T; t += a.group[0]) {
        sm.vexp[v] = 0;
        sm.vstart[v++] = t;
      }
      sm.vstart[v] = a.T;
      sm.nv = v;
      sm.plan = 0;
      if (blockIdx.x == 0) atomicExch(a.status, bad);
    }
    if (tid < a.T) sm.route_id[tid] = sm.route_tok[tid] = tid;
    return;
  }
  auto sync = [] { asm volatile("bar.sync 2, 128;" ::: "memory"); };
  const int R = a.T * a.K, token = tid * a.k_rcp >> 16;
  uint32_t bits = tid < R && (e < -1 || e >= a.E) ? MOE_DEV_ROUTE_RANGE : 0u;
  const bool live = tid < R && e >= 0 && e < a.E;
  const int low = e * kFp4MaxRoutes;
  const int mine = live ? low + tid : 0x7FFFFFFF;  // by expert, then by route
  sm.key[tid] = mine;
  sm.first[tid] = 0;
  sync();
  // routes before this one, with a lower expert, and neither with its expert and token
  int pos = 0, lower = 0, apart = 0;
  if (live) {
    const int same = low + token * a.K;
#pragma unroll 2
    for (int r = 0; r < R; r += 4) {
      const int4 k4 = *reinterpret_cast<const int4*>(&sm.key[r]);
      const int k[4] = {k4.x, k4.y, k4.z, k4.w};  // past the routes: the largest key
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        pos += k[i] < mine;
        lower += k[i] < low;
        apart += k[i] < same;
      }
    }
    const int within = pos - lower;
    if (a.check) {
      if (pos != apart) bits |= MOE_DEV_ROUTE_DUP;
      if (!(fabsf(w) < INFINITY)) bits |= MOE_DEV_ROUTE_NONFINITE;
    }
    sm.route_e[pos] = e;
    sm.route_id[pos] = tid;
    sm.route_tok[pos] = token;
    sm.route_w[pos] = w;
    auto starts = [&](int i) { return within == (within * a.group_rcp[i] >> 16) * a.group[i]; };
    sm.first[pos] = (int)starts(0) | (a.group[1] && starts(1) ? 2 : 0);
  }
  bits = __reduce_or_sync(0xFFFFFFFFu, bits);
  const int live_here = __popc(__ballot_sync(0xFFFFFFFFu, live));
  if (lane == 0) {
    sm.warp_bits[warp] = bits;
    sm.warp_live[warp] = live_here;
  }
  sync();
  const int first = sm.first[tid];
  const uint32_t firsts[2] = {__ballot_sync(0xFFFFFFFFu, first & 1), __ballot_sync(0xFFFFFFFFu, first & 2)};
  if (lane == 0) {
    sm.warp_cnt[0][warp] = __popc(firsts[0]);
    sm.warp_cnt[1][warp] = __popc(firsts[1]);
  }
  sync();
  // The second division has more places in the ring and takes fewer tokens at a time: an
  // expert with more of them is swept again.  For 16 tokens of 256 experts, H 7168, 16
  // places are 5% faster than 12 (402 and 424 us) and a sweep more is 1% of the products.
  // (The rule weighs items by that one shape; its border has not been measured.)
  auto items = [&](int i) { return sm.warp_cnt[i][0] + sm.warp_cnt[i][1] + sm.warp_cnt[i][2] + sm.warp_cnt[i][3]; };
  const int plan = a.group[1] && 17 * items(0) >= 16 * items(1), nv = items(plan);
  int v = __popc((plan ? firsts[1] : firsts[0]) & ((1u << lane) - 1u));
  for (int i = 0; i < warp; ++i) v += sm.warp_cnt[plan][i];
  if (first >> plan & 1) {
    sm.vstart[v] = tid;
    sm.vexp[v] = sm.route_e[tid];
  }
  if (tid == 0) {
    sm.plan = plan;
    sm.nv = nv;
    sm.vstart[nv] = sm.warp_live[0] + sm.warp_live[1] + sm.warp_live[2] + sm.warp_live[3];
    // the status word is this call's: the first CTA sets it
    if (blockIdx.x == 0)
      atomicExch(a.status, sm.warp_bits[0] | sm.warp_bits[1] | sm.warp_bits[2] | sm.warp_bits[3] | bad);
  }
}

template <bool MOE, int NT>
__global__ void __launch_bounds__(kFp4Threads, 1)
    fp4_stream_kernel(const __grid_constant__ Fp4Maps maps, const Fp4Args a) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ Fp4Shared sm;
  constexpr int kPartBytes = 2 * NT * 512;
  const uint32_t pbuf = (smem_u32(smem_raw) + 1023u) & ~1023u;  // the consumers' sums
  const uint32_t ring = pbuf + 2 * kConsumers * kPartBytes;     // the units: codes, then scales
  const uint8_t* const smem = smem_raw + (ring - smem_u32(smem_raw));  // the same, for plain loads
  const int warp_id = threadIdx.x >> 5, lane = threadIdx.x & 31;

  {
    const int i = threadIdx.x;
    if (i < kMaxStages) {
      // copies: one arrival with the codes' bytes, one per lane with its scales
      mbar_init(smem_u32(&sm.full[i]), 33);
      mbar_init(smem_u32(&sm.empty[i]), 1);
    } else if (i >= 96 && i < 96 + kFp4MaxTokens) {
      sm.row_max[i - 96] = 0u;
    } else if (i >= 32 && i < 32 + kConsumers) {
      sm.done[i - 32] = sm.taken[i - 32][0] = sm.taken[i - 32][1] = 0;
    } else if (i >= 64 && i < 64 + 2 * kItems) {
      mbar_init(smem_u32(&sm.bfull[0][0] + (i - 64)), kLoaders);
      mbar_init(smem_u32(&sm.bempty[0][0] + (i - 64)), kConsumers + (i - 64 < kItems ? kEpilogues : 1));
    } else if (i == 128) {
      mbar_init(smem_u32(&sm.go), kLoaders);
      sm.lim = {0, a.status, a.wait_ns};
      for (int k = 0; k < kProducers; ++k) sm.issued[k] = 0;
      for (int p = 0; p < (MOE ? 2 : 1); ++p) {
        prefetch_tensormap(&maps.unit[p]);
        prefetch_tensormap(&maps.box[p]);
      }
    }
    fence_mbar_init();
  }
  // The kernel before this one in the stream may still be at work; nothing above
  // reads global memory.  (So the linear is launched; the layer's cooperative launch
  // does not overlap, and returns from here at once.)
  pdl_wait();
  pdl_trigger();
  // x rows that stay are asked for before anything else: behind the first weights
  // they would wait for a full ring's copies
  // (the first division: with the second one they do not stay)
  const bool early = (int64_t)a.T * row_bytes(a.m[0].cols, false) <= a.b_bytes[0];
  const uint32_t early_rows = ring + a.stages[0] * kUnitBytes;
  const bool loader = warp_id >= kWarpLoader && warp_id < kWarpConsumer;
  if (loader && lane == 0) {
    uint64_t& bar = sm.raw[warp_id - kWarpLoader];
    mbar_init(smem_u32(&bar), 1);
    fence_mbar_init();
    if (early && warp_id == kWarpLoader) {
      raw_begin(bar, a.T * a.m[0].cols * 2);
      for (int r = 0; r < a.T; ++r)
        bulk_load(early_rows + r * row_bytes(a.m[0].cols, false), a.x + r * a.ldx, a.m[0].cols * 2, smem_u32(&bar));
    }
  }
  int route = -1;
  float route_w = 0.f;
  uint32_t bad = 0u;
  if (blockIdx.x == 0 && threadIdx.x == 0 && a.ctl[kCtlPoison]) bad = MOE_DEV_TIMEOUT;
  if (MOE && threadIdx.x < a.T * a.K) {
    route = a.idx[threadIdx.x];
    route_w = a.w[threadIdx.x];
  }
  __syncthreads();

  // Two groups of warps: the tables, after which the copies of the weights start at
  // once; and meanwhile, where the x rows stay, the loaders and consumers turn them.
  using Ctx = Fp4Ctx<MOE, NT>;
  constexpr int kTableThreads = 32 * kWarpLoader;
  static_assert(kTableThreads >= kFp4MaxRoutes, "one thread per route");
  bool rows_ok = true;
  WaitLimit& lim = sm.lim;
  if (warp_id < kWarpLoader) {
    if (threadIdx.x < kFp4MaxRoutes) {
      build_items<MOE>(a, sm, route, route_w, bad);
      asm volatile("bar.sync 2, 128;" ::: "memory");
      if (sm.nv > 0 && lane == 0 && warp_id < (MOE ? 2 : 1))
        sm.phase[warp_id] = Ctx{a, sm, sm.nv}.make_phase(warp_id);
    }
    asm volatile("bar.sync 3, %0;" ::"n"(kTableThreads) : "memory");
    asm volatile("bar.arrive 4, %0;" ::"n"(kFp4Threads) : "memory");
  } else {
    if (early) {
      if (loader && lane == 0) mbar_arrive(smem_u32(&sm.go));
      rows_ok = fill_x_rows(a.T, a.m[0].cols, early_rows, row_bytes(a.m[0].cols, false), warp_id - kWarpLoader,
                            kLoaders + kConsumers, sm.raw[0], sm.row_max, sm.rscale[0], lim);
    }
    asm volatile("bar.sync 4, %0;" ::"n"(kFp4Threads) : "memory");
  }
  const Ctx c{a, sm, sm.nv};
  constexpr int kPhases = MOE ? 2 : 1;
  const int stages = MOE && sm.plan ? a.stages[1] : a.stages[0];
  const uint32_t brow0 = ring + stages * kUnitBytes;  // operand rows

  if (MOE && c.nv == 0) {  // no active route: zeros
    uint4* o = reinterpret_cast<uint4*>(a.y);
    const int64_t n = (int64_t)a.T * a.m[1].rows / 8;
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < n;
         i += (int64_t)gridDim.x * blockDim.x)
      o[i] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }

  if (!rows_ok) goto done;

  if (warp_id >= kWarpConsumer) {
    // ------------------------------------------------------------ consumers
    const int warp = warp_id - kWarpConsumer, g = lane >> 2, t = lane & 3;
    int pc = 0;     // sums this warp has handed over
    int n0 = 0;     // the CTA's units before this visit; FC1: its n-th unit is warp n mod 8's
    auto consume = [&](auto phase_constant) {
      constexpr int p = decltype(phase_constant)::value;
      // what the walk needs of the phase, in registers: reading it where it is used costs a
      // round trip to shared memory each time (a tile's set-up took 1200 clocks)
      const Phase& f = c.phase(p);
      const int u0 = f.u0, u1 = f.u1, U = f.U, visit = f.visit(), inner = p == 0 ? f.RT : f.nv;
      if (u0 >= u1) return true;
      const int RB = row_bytes(f.cols, p == 1);
      const bool res = p == 0 && c.resident(0);
      const int R = c.ring_rows(p);
      int item = -1, pos = 0, rows = 0;
      const TilePos start = f.start;
      int v = start.v, left = inner - (p == 0 ? start.j : start.v);  // steps to the next item / tile
      bool fresh = true;        // a new item
      const uint8_t* brow[NT];  // this lane's operand rows
      int ka = f.ka;            // first unit of the visit (second phase: 0)
      // second phase: where the i-th of this warp's units of a visit comes in the order
      const int full = U >> 1, half = warp & 1;
      auto place = [&](int i) { return i < full ? 8 * i + warp : 8 * full + (warp >> 1); };
      // The warp's next unit: its count, place in the ring and lap's parity, and whether its
      // copies were seen to be there.  Only once the copies have begun is the place in this
      // lap's phase, and the parity that of this lap.
      int nu = p == 0 ? warp : n0 + place(0);
      int slot = (int)((uint32_t)nu % (uint32_t)stages), parity = (nu / stages) & 1;
      bool ready = false;
      for (int u = u0 - ka; u < u1; u += visit) {
        const int kb = min(visit, u1 - u);
        if (fresh) {
          if (!res) {
            if (item >= 0) {
              __syncwarp();
              if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[p][item % kItems]));
            }
            pos += rows;
            if (pos >= R) pos -= R;
            ++item;
            if (!warp_wait(sm.bfull[p][item % kItems], (item / kItems) & 1, lim)) return false;
          }
          const int s0 = sm.vstart[v];
          rows = sm.vstart[v + 1] - s0;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const int col = min(8 * nt + g, rows - 1);  // columns past the item repeat a row; nothing reads them
            brow[nt] = smem + (brow0 - ring) + c.row_slot(res, pos, R, s0, col) * RB + t * 16;
          }
        }
        // the next visit's item
        if (p == 0) {
          fresh = --left == 0;
          if (fresh) {
            ++v;
            left = inner;
          }
        } else if (--left == 0) {
          v = 0;
          left = inner;
        } else {
          ++v;
        }
        // this warp's units of the visit: columns from 512 k, k = first, first + dk, .. < last
        const int first = p == 0 ? ka + ((warp - n0) & (kConsumers - 1)) : half * (U - full);
        const int last = p == 0 ? kb : half ? U : U - full;
        constexpr int dk = p == 0 ? kConsumers : 1;
        if (first < last) {
          // two sums per tile, so that consecutive MMAs do not wait for each other
          float acc[2][NT][2][4] = {};
#pragma unroll 1
          for (int k = first; k < last; k += dk) {
            if (!ready) {
              if (!wait_count(&sm.issued[nu % kProducers], nu / kProducers + 1, lim)) return false;
              if (!warp_wait(sm.full[slot], parity, lim)) return false;
            }
            const uint8_t* base = smem + slot * kUnitBytes + (t >> 1) * (2 * kBoxBytes) + g * 128;
            const uint8_t* sbase = smem + slot * kUnitBytes + kCodeBytes + g * 32 + 8 * t;
            uint2 s[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // rows g, g + 8, g + 16, g + 24
              const uint2 v = *reinterpret_cast<const uint2*>(sbase + i * 256);
              s[i] = t < 2 ? v : make_uint2(v.y, v.x);  // chunk order of lanes t >= 2
            }
            // two of the four steps at a time: their codes to registers, and with the
            // second two the unit's place is free for the next copies
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint4 cw[2][2][2];  // [step][16-row half of the tile][rows g, g + 8]
#pragma unroll
              for (int jj = 0; jj < 2; ++jj) {
                const int chunk = (((t & 1) * 4 + ((2 * half + jj) ^ ((t >> 1) << 1))) ^ g) << 4;
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                  for (int hi = 0; hi < 2; ++hi)
                    cw[jj][m][hi] = *reinterpret_cast<const uint4*>(base + m * kBoxBytes + hi * 1024 + chunk);
              }
              if (half == 1) {
                __syncwarp();
                if (lane == 0) mbar_arrive(smem_u32(&sm.empty[slot]));
                // on to the next one (at most a lap further), looked at while this one's
                // products are under way
                const int i = k - first, step = p == 0 ? kConsumers
                                                : i + 1 < last - first ? place(i + 1) - place(i)
                                                                       : visit + place(0) - place(i);
                nu += step;
                slot += step;
                if (slot >= stages) {
                  slot -= stages;
                  parity ^= 1;
                }
                const bool begun = load_count(&sm.issued[nu % kProducers]) > nu / kProducers;
                ready = mbar_test_wait(smem_u32(&sm.full[slot]), parity) && begun;
                ready = __all_sync(0xFFFFFFFFu, ready);
              }
#pragma unroll
              for (int jj = 0; jj < 2; ++jj) {
                uint32_t sw[2][2];
#pragma unroll
                for (int m = 0; m < 2; ++m)
#pragma unroll
                  for (int hi = 0; hi < 2; ++hi) {
                    const uint32_t word = half == 0 ? s[2 * m + hi].x : s[2 * m + hi].y;
                    sw[m][hi] = e4m3x2_half2(jj ? word >> 16 : word & 0xFFFFu);
                  }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  uint4 b[NT];
#pragma unroll
                  for (int nt = 0; nt < NT; ++nt)
                    b[nt] = *reinterpret_cast<const uint4*>(brow[nt] + k * (kUnitCols * 2) +
                                                            (((2 * half + jj) * 4 + i) << 6));
#pragma unroll
                  for (int m = 0; m < 2; ++m) {
                    uint32_t lo[4], hi[4];
                    const uint4 wl = cw[jj][m][0], wh = cw[jj][m][1];
                    if (i < 2) {
                      e2m1x8_scaled<0>(i == 0 ? wl.x : wl.y, sw[m][0], lo);
                      e2m1x8_scaled<0>(i == 0 ? wh.x : wh.y, sw[m][1], hi);
                    } else {
                      e2m1x8_scaled<1>(i == 2 ? wl.z : wl.w, sw[m][0], lo);
                      e2m1x8_scaled<1>(i == 2 ? wh.z : wh.w, sw[m][1], hi);
                    }
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                      mma_16816(acc[m][nt][0], lo[0], hi[0], lo[1], hi[1], b[nt].x, b[nt].y);
                      mma_16816(acc[m][nt][1], lo[2], hi[2], lo[3], hi[3], b[nt].z, b[nt].w);
                    }
                  }
                }
              }
            }
          }
          if (!wait_count(&sm.taken[warp][pc & 1], pc >> 1, lim)) return false;
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
          ++pc;
          if (lane == 0) store_count(&sm.done[warp], pc);
        }
        n0 += kb - ka;
        ka = 0;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[p][max(item, 0) % kItems]));
      return true;
    };
    if (consume(std::integral_constant<int, 0>{})) {
      if constexpr (MOE) consume(std::integral_constant<int, 1>{});
    }
  } else if (warp_id >= kWarpProducer && warp_id < kWarpLoader) {
    // ------------------------------------------------------------ producers
    const uint64_t pass = policy_evict_first(), keep = policy_evict_normal();
    const int pw = warp_id - kWarpProducer;  // this one's units: every fourth, counted over both phases
    int slot = pw, mine = 0;
    uint32_t parity = 1;
    // the copies of a unit: columns from 512 k of the 32 rows from `row` on (FC1: 16
    // gate rows of `tile` and their up rows); lane_row: the lane's row.  False: gave up.
    auto issue = [&](auto phase_constant, const Phase& f, int k, int row, int row16, int64_t lane_row,
                     int tile, int expert, uint64_t policy) {
      constexpr int p = decltype(phase_constant)::value;
      if (!warp_wait(sm.empty[slot], parity, lim)) return false;
      const Fp4Matrix& m = a.m[p];
      const int ng = f.cols >> 4;
      const uint32_t bar = smem_u32(&sm.full[slot]), dst = ring + slot * kUnitBytes;
      if (lane == 0) {
        store_count(&sm.issued[pw], ++mine);
        // one copy, but for a unit that ends within a 256-column block, past which
        // lies the next row: a copy per 16 rows x 256 columns, cut off at the row's end
        const int blocks = (f.cols + 255) >> 8;
        if ((f.cols & 255) == 0 || 2 * k + 2 < blocks) {
          mbar_arrive_expect_tx(bar, kCodeBytes);
          if (MOE && p == 0)
            load_box_5d(dst, &maps.unit[0], bar, 0, 16 * tile, 0, 2 * k, expert, policy);
          else
            load_box_3d(dst, &maps.unit[p], bar, 0, row, 2 * k, policy);
        } else {
          mbar_arrive_expect_tx(bar, (blocks - 2 * k) * 2 * kBoxBytes);
          for (int b = 0; b < blocks - 2 * k; ++b) {
            load_box_2d(dst + 2 * b * kBoxBytes, &maps.box[p], bar, 128 * (2 * k + b), row, policy);
            load_box_2d(dst + (2 * b + 1) * kBoxBytes, &maps.box[p], bar, 128 * (2 * k + b), row16, policy);
          }
        }
      }
      __syncwarp();
      // lane: the scales of its row
      const bool in = MOE || lane_row < m.rows;
      const uint8_t* src = m.scales + (in ? lane_row * ng + 32 * k : 0);
      const int n = in ? min(32, ng - 32 * k) : 0;
      const uint32_t to = dst + kCodeBytes + lane * 32;
      if ((ng & 3) == 0) {
        if ((ng & 15) == 0) {
          cp_async<16>(to, src, n > 0 ? 16 : 0, policy);
          cp_async<16>(to + 16, n > 16 ? src + 16 : src, n > 16 ? 16 : 0, policy);
        } else if ((ng & 7) == 0)
          copy_scale_row<8>(to, src, n, policy);
        else
          copy_scale_row<4>(to, src, n, policy);
        asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
      } else {  // rows on odd multiples of two bytes: through registers
        for (int o = 0; o < 32; o += 4) {
          uint32_t x = 0u;
          if (o < n) x = __ldg(reinterpret_cast<const uint16_t*>(src + o));
          if (o + 2 < n) x |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(src + o + 2)) << 16;
          asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + o), "r"(x) : "memory");
        }
        // these are ordinary stores, which the arrival of the asynchronous copies does not
        // order: one that releases them
        mbar_arrive(bar);
      }
      slot += kProducers;
      if (slot >= stages) {
        slot -= stages;
        parity ^= 1;
      }
      return true;
    };
    // read again by the next item: the same matrix, more tokens
    auto item_policy = [&](int v) {
      return v + 1 < c.nv && sm.vexp[v + 1] == sm.vexp[v] ? keep : pass;
    };
    // the first operand rows go ahead of the weights
    bool ok = warp_wait(sm.go, 0, lim);
    if (MOE && a.watchdog_test && blockIdx.x == 0 && pw == 0) ok = false;  // its copies are missing
    int to_mine = pw;  // units until this warp's next one
    {
      const Phase& f = c.phase(0);
      TilePos at = f.start;
      int ka = f.ka;
      for (int u = f.u0 - ka; u < f.u1 && ok; u += f.U, f.step(at)) {
        const int kb = min(f.U, f.u1 - u);
        int k = ka + to_mine;
        if (k < kb) {
          const int64_t row = c.matrix_row(0, at, lane);
          const int r0 = __shfl_sync(0xFFFFFFFFu, (int)row, 0), r16 = __shfl_sync(0xFFFFFFFFu, (int)row, 16);
          const uint64_t policy = item_policy(at.v);
          for (; k < kb && ok; k += kProducers)
            ok = issue(std::integral_constant<int, 0>{}, f, k, r0, r16, row, at.j, sm.vexp[at.v], policy);
        }
        to_mine = k - kb;
        ka = 0;
      }
    }
    if constexpr (MOE) {
      const Phase& f = c.phase(1);
      TilePos at = f.start;
      const int visit = f.visit();
      for (int u = f.u0; u < f.u1 && ok; u += visit, f.step(at)) {
        const int r0 = (int)c.matrix_row(1, at, 0);
        const uint64_t policy = item_policy(at.v);
        int i = to_mine;
        for (; i < visit && ok; i += kProducers) {
          int w, k;
          f.unit_of(i, w, k);
          const int r = r0 + 32 * (w >> 1);
          ok = issue(std::integral_constant<int, 1>{}, f, k, r, r + 16, (int64_t)r + lane, 0, 0, policy);
        }
        to_mine = i - visit;
      }
    }
    // no copy outlives the CTA, also when the other warps have given up
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (gave_up(lim) && lane < stages) {
      int none = 0;
      for (int i = 0; i < 2; ++i)
        mbar_wait_bounded(smem_u32(&sm.full[lane]), i, &none, nullptr, 100000000ull);
    }
  } else if (warp_id < kWarpProducer) {
    // ------------------------------------------------------------- epilogue
    const int g = lane >> 2, t = lane & 3;
    int n0 = 0;     // the CTA's units before this tile
    int left = 0;   // lane w: sums that warp w has left before this tile
    for (int v = lane; v < c.nv; v += 32)
      for (int p = 0; p < kPhases; ++p) sm.vglobal[p][v] = __ldg(&a.m[p].global[sm.vexp[v]]);
    __syncwarp();
    // Where the sums of the warps first, first + step, .. (cnt of them) lie: lane i
    // gets the i-th one's warp and address, once all of them are there
    auto await_sums = [&](int first, int step, int cnt, int& from, uint32_t& src) {
      from = (first + step * lane) & (kConsumers - 1);
      const int n = __shfl_sync(0xFFFFFFFFu, left, from);
      src = pbuf + (2 * from + (n & 1)) * kPartBytes;
      return wait_count(&sm.done[from], lane < cnt ? n + 1 : 0, lim);
    };
    auto give_back = [&](int from, int cnt) {
      __syncwarp();
      const int n = __shfl_sync(0xFFFFFFFFu, left, from);
      if (lane < cnt) store_count(&sm.taken[from][n & 1], (n >> 1) + 1);
    };
    // on to the next tile
    auto count_sums = [&](int first, int step, int cnt) {
      const int i = ((lane - first) & (kConsumers - 1)) / step;
      left += ((lane - first) & (step - 1)) == 0 && i < cnt;
    };
    // A cut tile: this CTA's share goes to its slot, and the CTA that comes last
    // adds the shares in the order of the CTAs.  False: not the last one.
    auto last_to_join = [&](const Phase& f, int c0, int c1) {
      __threadfence();
      __syncwarp();
      uint32_t old = 0;
      uint32_t* count = &a.ctl[2 + f.p * kFp4Grid + c0];
      if (lane == 0) old = atomicAdd(count, 1u);
      old = __shfl_sync(0xFFFFFFFFu, old, 0);
      if (old != (uint32_t)(c1 - c0)) return false;
      __threadfence();
      if (lane == 0) *count = 0u;
      return true;
    };
    {
      const Phase& f = c.phase(0);
      const bool res = c.resident(0);
      const int R = c.ring_rows(0);
      ItemWalk it;
      TilePos at = f.start;
      int ka = f.ka, n = 0, s0 = 0;
      float factor[NT][2], factor2[NT][2];
      bool fresh = true;  // a new item since this warp's last tile
      int turn = 0;
      for (int u = f.u0 - ka; u < f.u1; u += f.U, f.step(at)) {
        const int units = min(f.U, f.u1 - u) - ka, last_item = it.item;
        if (it.next(c, f, res, R, at)) {
          fresh = true;
          if (last_item >= 0) {
            __syncwarp();
            if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[0][last_item % kItems]));
          }
        } else if (at.j == 0) {
          fresh = true;
        }
        const bool cut = units != f.U;
        const int cnt = min(units, kConsumers), first = n0;
        // a cut tile's CTAs, while its sums are on their way
        const int c0 = cut ? f.cta_of(u) : 0, c1 = cut ? f.cta_of(u + f.U - 1) : 0;
        n0 += units;
        ka = 0;
        turn ^= 1;
        if (turn == warp_id) {  // the other warp's
          count_sums(first, 1, cnt);
          continue;
        }
        // the sums of the warps that had units of the tile, in their order
        float acc[2][NT][4] = {};
        int from;
        uint32_t my_src;
        if (!await_sums(first, 1, cnt, from, my_src)) goto done;
#pragma unroll
        for (int i0 = 0; i0 < kConsumers; i0 += 4) {
          if (i0 >= cnt) break;
          uint4 x[4][2][NT];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t src = __shfl_sync(0xFFFFFFFFu, my_src, i0 + i) + lane * 16;
            if (i0 + i < cnt) {
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) x[i][m][nt] = lds128(src + (m * NT + nt) * 512);
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (i0 + i < cnt) {
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                  acc[m][nt][0] += __uint_as_float(x[i][m][nt].x);
                  acc[m][nt][1] += __uint_as_float(x[i][m][nt].y);
                  acc[m][nt][2] += __uint_as_float(x[i][m][nt].z);
                  acc[m][nt][3] += __uint_as_float(x[i][m][nt].w);
                }
            }
        }
        give_back(from, cnt);
        count_sums(first, 1, cnt);
        // lane (g, t) holds rows g and g + 8 of tokens 8 nt + 2 t and + 1; their factors:
        if (fresh) {
          fresh = false;
          n = c.item_rows(at.v);
          s0 = sm.vstart[at.v];
          const float gl = sm.vglobal[0][at.v];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const int col = 8 * nt + 2 * t + o;
              const float2 f2 =
                  col < n ? root_scales(sm.rscale[0][c.row_slot(res, it.pos, R, s0, col)]) : make_float2(0.f, 0.f);
              factor[nt][o] = f2.x;
              factor2[nt][o] = f2.y * gl;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int o = 0; o < 2; ++o)
#pragma unroll
            for (int m = 0; m < 2; ++m) {
              acc[m][nt][o] = acc[m][nt][o] * factor[nt][o] * factor2[nt][o];
              acc[m][nt][2 + o] = acc[m][nt][2 + o] * factor[nt][o] * factor2[nt][o];
            }
        if (cut) {
          auto share = [&](int cta) {
            return reinterpret_cast<float4*>(a.part[0] + (size_t)(2 * cta + (cta == c0)) * 512) + lane;
          };
          float4* mine = share(blockIdx.x);
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
              __stcg(mine + (m * NT + nt) * 32,
                     make_float4(acc[m][nt][0], acc[m][nt][1], acc[m][nt][2], acc[m][nt][3]));
          if (!last_to_join(f, c0, c1)) continue;
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
              for (int i = c0; i <= c1; ++i) {
                const float4 z = __ldcg(share(i) + (m * NT + nt) * 32);
                s.x += z.x, s.y += z.y, s.z += z.z, s.w += z.w;
              }
              acc[m][nt][0] = s.x, acc[m][nt][1] = s.y, acc[m][nt][2] = s.z, acc[m][nt][3] = s.w;
            }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int o = 0; o < 2; ++o) {
            const int col = 8 * nt + 2 * t + o;
            if (8 * nt + o >= n) continue;  // no lane has a column
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
        if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[0][it.item % kItems]));
      }
      if (MOE) {  // every h value of this CTA is stored, also for bulk copies
        fence_proxy_async_global();
        __syncwarp();
        if (lane == 0) red_release_gpu_add(reinterpret_cast<int32_t*>(&a.ctl[0]), 1);
      }
    }
    if (MOE && warp_id == kWarpEpilogue) {
      const Phase& f = c.phase(1);
      const int R = c.ring_rows(1), visit = f.visit(), tu = f.tile_units();
      const int step = f.U > 1 ? 1 : 2, cnt = kConsumers / step;  // the warps with units
      ItemWalk it;
      TilePos at = f.start;
      bool fresh = true;  // first visit of a tile by this CTA
      int c0 = 0, c1 = 0;  // the tile's CTAs
      for (int u = f.u0; u < f.u1; u += visit, f.step(at)) {
        const int last_item = it.item;
        it.next(c, f, false, R, at);
        if (last_item >= 0) {
          __syncwarp();
          if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[1][last_item % kItems]));
        }
        if (fresh) {
          for (int i = lane; i < a.T * kTile2 / 4; i += 32)
            reinterpret_cast<float4*>(&sm.out[0][0])[i] = make_float4(0.f, 0.f, 0.f, 0.f);
          fresh = false;
          c0 = f.cta_of(at.j * tu);
          c1 = f.cta_of(at.j * tu + tu - 1);
        }
        const int n = c.item_rows(at.v), s0 = sm.vstart[at.v];
        int from;
        uint32_t my_src;
        if (!await_sums(0, step, cnt, from, my_src)) goto done;
        // lane (g, t) holds rows g and g + 8 of tokens 2 t and 2 t + 1: their factors
        // and places in out[token][row], which sums over the tile's items
        const float gl = sm.vglobal[1][at.v];
        float factor[2], factor2[2];
        float* row[2];
#pragma unroll
        for (int o = 0; o < 2; ++o) {
          const int col = min(2 * t + o, n - 1), s = s0 + col;
          const float2 f2 = root_scales(sm.rscale[1][c.row_slot(false, it.pos, R, s0, col)]);
          factor[o] = f2.x;
          factor2[o] = f2.y * gl * sm.route_w[s];
          row[o] = &sm.out[sm.route_tok[s]][g];
        }
#pragma unroll
        for (int b = 0; b < 4; ++b) {  // blocks of 32 rows
          uint4 x[2][2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t src = __shfl_sync(0xFFFFFFFFu, my_src, f.U > 1 ? 2 * b + h : b) + lane * 16;
            if (h == 0 || f.U > 1) {
              x[h][0] = lds128(src);
              x[h][1] = lds128(src + 512);
            } else {
              x[h][0] = x[h][1] = make_uint4(0u, 0u, 0u, 0u);
            }
          }
#pragma unroll
          for (int o = 0; o < 2; ++o)
            if (2 * t + o < n) {
              float* to = row[o] + 32 * b;
              auto add = [&](const uint4& p, const uint4& q, int hi) {
                const uint32_t y = hi ? (o ? p.w : p.z) : (o ? p.y : p.x);
                const uint32_t z = hi ? (o ? q.w : q.z) : (o ? q.y : q.x);
                return (__uint_as_float(y) + __uint_as_float(z)) * factor[o];
              };
              const float r[4] = {to[0], to[8], to[16], to[24]};
              to[0] = fmaf(factor2[o], add(x[0][0], x[1][0], 0), r[0]);
              to[8] = fmaf(factor2[o], add(x[0][0], x[1][0], 1), r[1]);
              to[16] = fmaf(factor2[o], add(x[0][1], x[1][1], 0), r[2]);
              to[24] = fmaf(factor2[o], add(x[0][1], x[1][1], 1), r[3]);
            }
        }
        give_back(from, cnt);
        count_sums(0, step, cnt);
        const int tb = at.j * tu, te = tb + tu;  // the tile's units
        if (u + visit < min(f.u1, te)) continue;  // more of this tile to come
        fresh = true;
        if (c0 != c1) {
          auto share = [&](int cta) {
            return reinterpret_cast<float4*>(a.part[1] + (size_t)(2 * cta + (cta == c0)) *
                                                             (kFp4MaxTokens * kTile2)) + lane;
          };
          float4* mine = share(blockIdx.x);
          for (int tok = 0; tok < a.T; ++tok)
            __stcg(mine + tok * (kTile2 / 4), *reinterpret_cast<const float4*>(&sm.out[tok][4 * lane]));
          if (!last_to_join(f, c0, c1)) continue;
          for (int tok = 0; tok < a.T; ++tok) {
            float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
            for (int i = c0; i <= c1; ++i) {
              const float4 z = __ldcg(share(i) + tok * (kTile2 / 4));
              s.x += z.x, s.y += z.y, s.z += z.z, s.w += z.w;
            }
            *reinterpret_cast<float4*>(&sm.out[tok][4 * lane]) = s;
          }
        }
        __syncwarp();
        uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + kTile2 * at.j + 4 * lane;
        for (int tok = 0; tok < a.T; ++tok) {
          const float4 v = *reinterpret_cast<const float4*>(&sm.out[tok][4 * lane]);
          *reinterpret_cast<uint2*>(y + (int64_t)tok * a.m[1].rows) =
              make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
        __syncwarp();
      }
      if (f.u0 < f.u1) {
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&sm.bempty[1][it.item % kItems]));
      }
    }
  } else {
    // -------------------------------------------------------------- loaders
    const int lw = warp_id - kWarpLoader;
    uint32_t raw_parity = early && lw == 0;
    bool went = early;  // whether the producers need not wait for this warp's first copy
    for (int p = 0; p < kPhases; ++p) {
      const Phase& f = c.phase(p);
      if (MOE && p == 1) {
        bool ok = true;
        if (lane == 0) {
          const uint64_t t0 = globaltimer_ns();
          while (ld_acquire_gpu_u32(&a.ctl[0]) < kEpilogues * gridDim.x) {
            if (gave_up(lim)) {
              ok = false;
              break;
            }
            if (globaltimer_ns() - t0 > lim.ns) {
              lim.abort = 1;
              record_status(a.status, MOE_DEV_TIMEOUT);
              ok = false;
              break;
            }
          }
          fence_proxy_async_global();
        }
        if (!__shfl_sync(0xFFFFFFFFu, (int)ok, 0)) goto done;
      }
      if (f.u0 >= f.u1) {
        if (!went && lane == 0) mbar_arrive(smem_u32(&sm.go));
        went = true;
        continue;
      }
      const int RB = row_bytes(f.cols, p == 1);
      if (c.resident(p)) {
        // the rows' memory is the next phase's when everyone is done with them
        if (p + 1 < kPhases && !warp_wait(sm.bempty[p][0], 0, lim)) goto done;
      } else {
        const int R = c.ring_rows(p);
        ItemWalk it;
        int oldest = 0, used = 0, counter = 0;
        int rows_of[kItems];  // rows of the items in flight
        auto retire = [&]() {
          if (!warp_wait(sm.bempty[p][oldest % kItems], (oldest / kItems) & 1, lim))
            return false;
#pragma unroll
          for (int i = 0; i < kItems; ++i)
            if (i == oldest % kItems) used -= rows_of[i];
          ++oldest;
          return true;
        };
        TilePos at = f.start;
        const int visit = f.visit();
        for (int u = f.u0 - f.ka; u < f.u1; u += visit, f.step(at)) {
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
                  p == 0 ? fill_x(a.x + sm.route_tok[s] * a.ldx, f.cols, brow0 + place * RB, sm.raw[lw],
                                  raw_parity, &sm.rscale[0][place], lim, went ? nullptr : &sm.go)
                         : fill_h(a.h + (int64_t)sm.route_id[s] * record_bytes(f.cols), f.cols,
                                  brow0 + place * RB, sm.raw[lw], raw_parity, &sm.rscale[1][place], lim);
              went = true;
              if (!ok) goto done;
            }
          __syncwarp();
          if (lane == 0) {
            if (!went) mbar_arrive(smem_u32(&sm.go));
            mbar_arrive(smem_u32(&sm.bfull[p][it.item % kItems]));
          }
          went = true;
        }
        if (p + 1 < kPhases)
          while (oldest <= it.item)
            if (!retire()) goto done;
      }
    }
    // the last warp past the barrier leaves its counter at zero for the next call
    if (MOE && lane == 0 && atomicAdd(&a.ctl[1], 1u) == kLoaders * gridDim.x - 1) {
      a.ctl[0] = 0u;
      a.ctl[1] = 0u;
    }
  }
done:
  // whoever gave up leaves the counters as they are: every call says so until the host
  // has read the status and cleared them
  if (gave_up(lim) && lane == 0) a.ctl[kCtlPoison] = 1u;
}

// Shared memory of a launch: the operand rows' share, and what is left for the ring.
struct Fp4Plan {
  int group, nt, b_bytes, stages, smem;
};

static int fp4_part_bytes(int nt) { return kConsumers * 2 * 2 * nt * 512; }

static int fp4_row_budget(int nt) {
  return (kMaxSmem - (int)sizeof(Fp4Shared) - 2048 - fp4_part_bytes(nt) - kMinStages * kUnitBytes) / 128 * 128;
}

static void fp4_finish_plan(Fp4Plan* p) {
  p->b_bytes = (p->b_bytes + 127) / 128 * 128;
  p->stages = kMinStages + (fp4_row_budget(p->nt) - p->b_bytes) / (kProducers * kUnitBytes) * kProducers;
  if (p->stages > kMaxStages) p->stages = kMaxStages;
  p->smem = 1024 + p->stages * kUnitBytes + p->b_bytes + fp4_part_bytes(p->nt);
}

// The layer: tokens in groups of at most 8, with at most `budget` bytes of operand rows.
static Fp4Plan fp4_plan_layer(int H, int I, int T, int K, int budget) {
  Fp4Plan p = {8, 1, 0, 0, 0};
  const int r1 = row_bytes(H, false), r2 = row_bytes(I, true);
  if (budget / r1 < p.group) p.group = budget / r1;
  if (budget / r2 < p.group) p.group = budget / r2;
  if (p.group < 1) return p;
  // x: T rows, or one group's; h: two groups' or all, as far as they fit
  const int n1 = (int64_t)T * r1 <= budget ? T * r1 : p.group * r1;
  int rows2 = T * K < 2 * p.group ? T * K : 2 * p.group;
  if (rows2 > budget / r2) rows2 = budget / r2;
  p.b_bytes = n1 > rows2 * r2 ? n1 : rows2 * r2;
  fp4_finish_plan(&p);
  return p;
}

// The linear: one sweep over the matrix for up to 16 tokens where their rows
// fit (2048 columns; 8 tokens of 5120, 6 of 7168, 1 of 32768), else equal groups, each
// with its own sweep (the second from L2, where the matrix fits there).  4096 x 7168:
// 6 tokens 10.3 us, 7 to 12 (two sweeps) 14.1 to 16.3, 13 to 16 (three) 27.5; 4096 x 4096: 8
// tokens 8.2, 9 (two) 10.2.
static Fp4Plan fp4_plan_linear(int cols, int T) {
  Fp4Plan p = {0, 1, 0, 0, 0};
  const int rb = row_bytes(cols, false);
  const int fit1 = fp4_row_budget(1) / rb, fit2 = fp4_row_budget(2) / rb;
  const int most = fit2 > 8 ? (fit2 < 16 ? fit2 : 16) : (fit1 < 8 ? fit1 : 8);
  const int groups = (T + most - 1) / most;
  p.group = (T + groups - 1) / groups;
  p.nt = p.group > 8 ? 2 : 1;
  const int budget = fp4_row_budget(p.nt);
  p.b_bytes = (int64_t)T * rb <= budget ? T * rb : p.group * rb;
  fp4_finish_plan(&p);
  return p;
}

template <bool MOE, int NT>
static cudaError_t fp4_launch(const Fp4Maps& maps, const Fp4Args& a, int grid, int smem, cudaStream_t s) {
  cudaLaunchAttribute coop;
  coop.id = cudaLaunchAttributeCooperative;
  coop.val.cooperative = 1;
  // the layer's CTAs wait for one another (all resident, or the launch fails); the
  // linear's do not, and its launch and prologue overlap the kernel before (for
  // 4096 x 7168, T = 1, one after the other, 1.5 us less)
  return launch_k(fp4_stream_kernel<MOE, NT>, dim3(grid), dim3(kFp4Threads), smem, s, !MOE,
                  MOE ? &coop : nullptr, maps, a);
}

}  // namespace mm

using namespace mm;

struct moe_fp4_handle {
  bool layer;
  moe_dims dims;         // the layer
  Fp4Matrix m[2];        // the linear: the first
  Fp4Maps maps;
  int max_tokens, grid, device;
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
static_assert((kCtlPoison + 1) * 4 <= kFp4Ctl, "counters");

bool fp4_dims_ok(const moe_dims* d) {
  const bool hk = d->hidden >= 128 && d->hidden <= 16384 && d->hidden % 128 == 0;
  const bool ik = d->inter >= 128 && d->inter <= 16384 && d->inter % 128 == 0;
  const bool kk = d->top_k == 1 || d->top_k == 2 || d->top_k == 4 || d->top_k == 6 || d->top_k == 8;
  return hk && ik && kk && d->num_experts >= 1 && d->num_experts <= 1024 &&
         (d->flags & ~(MOE_FLAG_CHECK_ROUTES | MOE_FLAG_WATCHDOG_TEST)) == 0;
}

// Launches go to the current device: it has to be the one that the weights, the workspace
// and the kernels' attributes belong to.
bool elsewhere(const moe_fp4_handle* h) {
  int dev = -1;
  return cudaGetDevice(&dev) != cudaSuccess || dev != h->device;
}

bool misaligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) != 0; }

// The two maps of a matrix (Fp4Maps).  halves: FC1's, [E][gate, up][rows][cols],
// else [rows][cols].
bool fp4_encode_maps(CUtensorMap* unit, CUtensorMap* box, const void* base, uint64_t rows, uint64_t cols,
                     uint64_t experts) {
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
  auto encode = [&](CUtensorMap* m, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                    const cuuint32_t* b) {
    const cuuint32_t es[5] = {1, 1, 1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, rank, const_cast<void*>(base), dims, strides, b, es,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  const uint64_t pitch = cols / 2, all = rows * (experts ? 2 * experts : 1);
  // whole 256-column blocks (one, never used past its end, where there is none)
  const uint64_t blocks = cols / 256 ? cols / 256 : 1;
  const uint64_t inner = cols / 256 ? 128 : pitch < 128 ? pitch : 128;
  bool ok;
  if (experts) {
    const cuuint64_t dims[5] = {inner, rows, 2, blocks, experts};
    const cuuint64_t strides[4] = {pitch, rows * pitch, 128, 2 * rows * pitch};
    const cuuint32_t b[5] = {128, 16, 2, 2, 1};
    ok = encode(unit, 5, dims, strides, b);
  } else {
    const cuuint64_t dims[3] = {inner, all, blocks};
    const cuuint64_t strides[2] = {pitch, 128};
    const cuuint32_t b[3] = {128, 32, 2};
    ok = encode(unit, 3, dims, strides, b);
  }
  const cuuint64_t dims[2] = {pitch, all};
  const cuuint64_t strides[1] = {pitch};
  const cuuint32_t b[2] = {128, 16};
  return ok && encode(box, 2, dims, strides, b);
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
  h->device = dev;
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
  if (st == MOE_OK &&
      (!fp4_encode_maps(&h->maps.unit[0], &h->maps.box[0], d_w1, dims->inter, dims->hidden, E) ||
       !fp4_encode_maps(&h->maps.unit[1], &h->maps.box[1], d_w2, E * dims->hidden, dims->inter, 0)))
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
      misaligned(d_topk_idx, 4) || misaligned(d_topk_w, 4) || misaligned(d_out, 16) || elsewhere(h))
    return MOE_ERR_INVALID_ARG;
  const moe_dims& d = h->dims;
  const int budget = fp4_row_budget(1);
  const Fp4Plan p = fp4_plan_layer(d.hidden, d.inter, (int)num_tokens, d.top_k, budget);
  // where the x rows do not stay and the ring is short of its most places, the division
  // that is not
  const Fp4Plan p2 = p.stages == kMaxStages || num_tokens * row_bytes(d.hidden, false) <= budget
                         ? Fp4Plan{}
                         : fp4_plan_layer(d.hidden, d.inter, (int)num_tokens, d.top_k,
                                          budget - (kMaxStages - kMinStages) * kUnitBytes);
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
  a.group[0] = p.group;
  a.b_bytes[0] = p.b_bytes;
  a.stages[0] = p.stages;
  a.group[1] = p2.group;
  a.k_rcp = 65536 / d.top_k + 1;
  a.group_rcp[0] = 65536 / p.group + 1;
  a.group_rcp[1] = p2.group ? 65536 / p2.group + 1 : 0;
  a.b_bytes[1] = p2.b_bytes;
  a.stages[1] = p2.stages;
  a.check = (d.flags & MOE_FLAG_CHECK_ROUTES) != 0;
  a.watchdog_test = (d.flags & MOE_FLAG_WATCHDOG_TEST) != 0;
  a.grid_rcp = (uint32_t)(0x100000000ull / h->grid) + 1;
  a.wait_ns = a.watchdog_test ? 20000000ull : kWaitLimitNs;
  return fp4_launch<true, 1>(h->maps, a, h->grid, p.smem > p2.smem ? p.smem : p2.smem, stream) == cudaSuccess
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
  if (st == MOE_OK && !fp4_encode_maps(&h->maps.unit[0], &h->maps.box[0], d_codes, rows, cols, 0))
    st = MOE_ERR_CUDA;
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
      misaligned(d_y, y_float32 ? 4 : 2) || elsewhere(h))
    return MOE_ERR_INVALID_ARG;
  // a CTA that has finished stores y while others still read x
  const uintptr_t y0 = (uintptr_t)d_y, y1 = y0 + (size_t)num_tokens * m.rows * (y_float32 ? 4 : 2);
  for (int64_t t = 0; t < num_tokens; ++t) {
    const uintptr_t x0 = (uintptr_t)(d_x + t * x_stride);
    if (x0 < y1 && y0 < x0 + 2 * (size_t)m.cols) return MOE_ERR_INVALID_ARG;
  }
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
  a.group[0] = p.group;
  a.b_bytes[0] = p.b_bytes;
  a.stages[0] = p.stages;
  a.f32 = y_float32 != 0;
  a.grid_rcp = (uint32_t)(0x100000000ull / h->grid) + 1;
  a.wait_ns = kWaitLimitNs;
  const cudaError_t e = p.nt == 2
                            ? fp4_launch<false, 2>(h->maps, a, h->grid, p.smem, stream)
                            : fp4_launch<false, 1>(h->maps, a, h->grid, p.smem, stream);
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_fp4_read_status(moe_fp4_handle* h, uint32_t* h_status, struct CUstream_st* stream) {
  if (!h || !h_status || elsewhere(h)) return MOE_ERR_INVALID_ARG;
  if (cudaMemcpyAsync(h_status, h->status, 4, cudaMemcpyDeviceToHost, stream) != cudaSuccess ||
      cudaStreamSynchronize(stream) != cudaSuccess)
    return MOE_ERR_CUDA;
  if (*h_status & MOE_DEV_TIMEOUT) {
    if (cudaMemsetAsync(h->ctl, 0, kFp4Ctl, stream) != cudaSuccess || cudaStreamSynchronize(stream) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_ERR_DEVICE_TIMEOUT;
  }
  return *h_status ? MOE_ERR_BAD_ROUTE : MOE_OK;
}

void moe_fp4_destroy(moe_fp4_handle* h) { delete h; }

}  // extern "C"
