// dense.cu -- the dense products beside the MoE layer: x W^T in the layer's FP8 format
// (Fp8Linear) and the products of a gated feed-forward block and of its gradients
// (GatedMlp).
#include <utility>

#include <cudaTypedefs.h>

#include "dense.cuh"

namespace mm {

// ------------------------------------------------------------------------- rows to FP8
// Eight lanes per 128 columns of a row, 16 values each: amax, the least power of two that brings
// it to at most 448, codes.  x * 2^-e is exact (but below E4M3's range, where it rounds once).
// A stream: what bounds it is the bytes in flight, so a warp asks for four segments of four
// blocks before it uses one (8192 x 7168, 26 us at the copy rate: 35 us; with 8 bytes a
// lane and one block a warp at a time 70).
constexpr int kQuantTogether = 4;

__global__ void __launch_bounds__(256) quantize_rows_kernel(const uint16_t* x, int64_t ld, uint32_t units, uint32_t segs,
                                                            int kb, int pitch, uint8_t* q, uint8_t* s) {
  const int lane = threadIdx.x & 31;
  const uint32_t warps = gridDim.x * 8;
  pdl_wait();
  pdl_trigger();
  for (uint32_t u0 = blockIdx.x * 8 + (threadIdx.x >> 5); u0 < units; u0 += kQuantTogether * warps) {
    uint4 v[kQuantTogether][2];
    int64_t t[kQuantTogether];
    int c[kQuantTogether];
#pragma unroll
    for (int i = 0; i < kQuantTogether; ++i) {
      const uint32_t u = u0 + i * warps, row = u / segs;
      t[i] = row;
      c[i] = u < units ? (int)(u - row * segs) * 4 + (lane >> 3) : kb;
      if (c[i] >= kb) continue;
      const uint4* p = reinterpret_cast<const uint4*>(x + t[i] * ld + c[i] * 128 + (lane & 7) * 16);
      v[i][0] = p[0];
      v[i][1] = p[1];
    }
#pragma unroll
    for (int i = 0; i < kQuantTogether; ++i) {
      float f[16], m = 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t w[4] = {v[i][k].x, v[i][k].y, v[i][k].z, v[i][k].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          f[8 * k + 2 * e] = bf16_bits_to_float(w[e] & 0xFFFFu);
          f[8 * k + 2 * e + 1] = bf16_bits_to_float(w[e] >> 16);
        }
      }
#pragma unroll
      for (int k = 0; k < 16; ++k) m = fmaxf(m, fabsf(f[k]));
#pragma unroll
      for (int o = 4; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      if (c[i] >= kb) continue;
      const int e = pow2_scale_exp(m);
      const float inv = block_factor(m, e);
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        w[k] = e4m3x4(f[4 * k] * inv, f[4 * k + 1] * inv, f[4 * k + 2] * inv, f[4 * k + 3] * inv);
      *reinterpret_cast<uint4*>(q + (t[i] * kb + c[i]) * 128 + (lane & 7) * 16) = make_uint4(w[0], w[1], w[2], w[3]);
      if ((lane & 7) == 0) s[t[i] * pitch + c[i]] = (uint8_t)(e + 127);
    }
  }
}

cudaError_t dense_quantize_rows(const uint16_t* x, int64_t ld, int64_t T, int cols, uint8_t* q, uint8_t* s, int sms,
                                cudaStream_t stream) {
  const uint32_t segs = (uint32_t)(cols / 128 + 3) / 4, units = (uint32_t)T * segs;  // (below 2^30)
  const uint32_t ctas = (units + 7) / 8, most = (uint32_t)sms * 4;
  return launch_k(quantize_rows_kernel, dim3(ctas < most ? ctas : most), dim3(256), 0, stream, true, nullptr, x, ld,
                  units, segs, cols / 128, scale_pitch(cols), q, s);
}

__global__ void scales_to_e8m0_kernel(const float* s, int64_t n, int cols, int pitch, uint8_t* out,
                                      uint32_t* status) {
  for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (int64_t)gridDim.x * blockDim.x) {
    const uint32_t b = __float_as_uint(s[i]);
    const bool ok = b == 0x00400000u || ((b & 0x807FFFFFu) == 0u && b != 0u && b < 0x7F800000u);
    if (!ok) record_status(status, MOE_DEV_BAD_SCALE);
    out[i / cols * pitch + i % cols] = (uint8_t)(b >> 23);  // 2^-127, subnormal, is byte 0
  }
}

cudaError_t dense_scales_to_e8m0(const float* s, int64_t rows, int cols, int pitch, uint8_t* out, uint32_t* status,
                                 cudaStream_t stream) {
  const int64_t n = rows * cols;
  scales_to_e8m0_kernel<<<(int)((n + 255) / 256 < 1024 ? (n + 255) / 256 : 1024), 256, 0, stream>>>(s, n, cols, pitch,
                                                                                                out, status);
  return cudaGetLastError();
}

// ------------------------------------------------------------------------- products
// d[m, n] = sum_k a[m, k] b[n, k] on CTA pairs (tcgen05 cta_group::2): a pair owns a tile of
// 256 rows x BN columns, each CTA stages its 128 rows of A and half of B's rows, the
// leader issues the MMAs and each CTA drains its own 128 rows.  Persistent: the pairs take
// tiles in turn (PairArgs), of up to three products: the gradients of a block's input and
// weights need only what one kernel before them wrote, and fill each other's last wave;
// 8 row tiles share a sweep over the columns, so that what runs at one time reads few
// distinct operand rows.  BN is 256, or 192, 128, 64 where the tiles are few (pair_columns).
//   K-major operands (rows of K)      TMA boxes of rows x 128 bytes.
//   MN-major operands (K rows of it)  boxes of 64 K rows x 64 elements, two side by
//                                     side: gradients multiply the stored tensors as they
//                                     are, nothing is transposed in memory.
//   E4M3: block-scaled MMAs.  One warp builds the scale atoms (four K blocks of 128
//   rows) from the rows' and the matrix's E8M0 bytes, a slot ahead of the MMAs.
// Accumulators: two of up to 256 TMEM columns in turn.  With scales in TMEM (64 columns) two
// of 256 overlap by 64 columns, which the epilogue drains first.
// Warps: 0 and 3 loads, 1 MMAs, 2 scales, 4-11 epilogue (two per TMEM lane quadrant, a half
// of the columns each).
constexpr int kDThreads = 384;
constexpr int kDEpiWarps = 8;
constexpr int kDStages = 5;  // (with 6: 1% less time, with 4: 8% more; the fifth's room goes to the epilogue)
constexpr uint32_t kDBytesA = 16384, kDBytesB = 16384;
constexpr uint32_t kDStage = kDBytesA + kDBytesB;
constexpr int kSfSlots = 4;
constexpr uint32_t kSfSlotBytes = 1536;  // A atom, two B atoms
// Epilogue: per warp 32 rows x 128 bytes once (E4M3) or twice, through which sums and
// operands pass between thread = row and whole lines of memory.
template <bool F8>
struct PairSmem {
  static constexpr uint32_t kSf = kDStages * kDStage;
  static constexpr uint32_t kEpi = kSf + (F8 ? kSfSlots * kSfSlotBytes : 0u);
  static constexpr uint32_t kEpiWarp = F8 ? 4096u : 8192u;
  static constexpr uint32_t kBytes = kEpi + kDEpiWarps * kEpiWarp + 1024u;
};
constexpr uint32_t kDTmemSf = 448, kDSfCols = 16;

__device__ __forceinline__ void tc_mma_16_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// A warp's 32 rows x 128 bytes (or 64) in shared memory, in 16-byte pieces whose place is
// changed by the row, so that neither a thread's pieces of its row nor eight lanes' of one row
// meet in a bank.  Thread = row writes and reads pieces; memory is written and read
// eight (four) lanes to a row, whole lines at a time.  (Straight from the threads, 32 rows an
// instruction, the gradient's epilogue took 14 us of a 256 x 256 tile, most of it the
// load and store unit's time for 32 lines each.)
template <int BYTES>
__device__ __forceinline__ uint32_t piece_at(uint32_t buf, int row, int c) {
  return BYTES == 128 ? buf + row * 128 + ((c ^ (row & 7)) << 4) : buf + row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
}

__device__ __forceinline__ void sts_piece(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint4 lds_piece(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

// This thread's 32 values to its row: floats (128 bytes), or 16 bits from piece `first` on.
__device__ __forceinline__ void put_f32(uint32_t buf, int row, const float (&v)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    sts_piece(piece_at<128>(buf, row, c), __float_as_uint(v[4 * c]), __float_as_uint(v[4 * c + 1]),
              __float_as_uint(v[4 * c + 2]), __float_as_uint(v[4 * c + 3]));
}

template <int BYTES>
__device__ __forceinline__ void put_16(uint32_t buf, int row, int first, const float (&v)[32], DenseType t) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
    sts_piece(piece_at<BYTES>(buf, row, first + c), pack16(v[8 * c], v[8 * c + 1], t),
              pack16(v[8 * c + 2], v[8 * c + 3], t), pack16(v[8 * c + 4], v[8 * c + 5], t),
              pack16(v[8 * c + 6], v[8 * c + 7], t));
}

// The buffer's rows to dst (rows `pitch` bytes apart), `rows` of them and `bytes` of each
// (whole pieces).  ADD: floats, added to what is there.
template <int BYTES, bool ADD = false>
__device__ __forceinline__ void flush(uint32_t buf, uint8_t* dst, int64_t pitch, int rows, int bytes, int lane) {
  constexpr int kLanes = BYTES / 16, kRows = 32 / kLanes, kN = 32 / kRows;
  const int r0 = lane / kLanes, c = lane % kLanes;
  uint4 v[kN];  // (all read before the first is written: the reads' latency once)
#pragma unroll
  for (int i = 0; i < kN; ++i) v[i] = lds_piece(piece_at<BYTES>(buf, i * kRows + r0, c));
  if (16 * c >= bytes) return;
  uint4* p = reinterpret_cast<uint4*>(dst + r0 * pitch + 16 * c);
  const int64_t step = kRows * pitch / 16;
  if (ADD) {
    float4 o[kN];
#pragma unroll
    for (int i = 0; i < kN; ++i)
      if (i * kRows + r0 < rows) o[i] = *reinterpret_cast<const float4*>(p + i * step);
#pragma unroll
    for (int i = 0; i < kN; ++i) {
      v[i].x = __float_as_uint(__uint_as_float(v[i].x) + o[i].x);
      v[i].y = __float_as_uint(__uint_as_float(v[i].y) + o[i].y);
      v[i].z = __float_as_uint(__uint_as_float(v[i].z) + o[i].z);
      v[i].w = __float_as_uint(__uint_as_float(v[i].w) + o[i].w);
    }
  }
#pragma unroll
  for (int i = 0; i < kN; ++i)
    if (i * kRows + r0 < rows) p[i * step] = v[i];
}

// The same where rows begin anywhere: an element per lane.
template <typename E>
__device__ __forceinline__ void flush_elements(const uint8_t* buf, E* dst, int64_t ld, int rows, int cols, int lane) {
  constexpr int kPer = 16 / sizeof(E), kCols = 128 / sizeof(E) / 32;
#pragma unroll 1
  for (int r0 = 0; r0 < rows; r0 += 8) {
    E v[8][kCols];
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int k = 0; k < kCols; ++k) {
        const int c = lane + 32 * k;
        v[r][k] = *reinterpret_cast<const E*>(buf + (r0 + r) * 128 + (((c / kPer) ^ r) << 4) + c % kPer * sizeof(E));
      }
    E* p = dst + r0 * ld + lane;
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int k = 0; k < kCols; ++k)
        if (r0 + r < rows && lane + 32 * k < cols) p[r * ld + 32 * k] = v[r][k];
  }
}

// 32 columns of saved gate or up, asynchronously, zeros past the rows and columns.
__device__ __forceinline__ void fetch_saved(uint32_t buf, const uint8_t* src, int64_t pitch, int rows, int bytes, bool f32,
                                            int lane) {
  auto copy = [&](uint32_t at, int r, int c) {
    const bool in = r < rows && 16 * c < bytes;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(in ? src + r * pitch + 16 * c : src),
                 "r"(in ? 16 : 0)
                 : "memory");
  };
  if (f32) {
#pragma unroll
    for (int i = 0; i < 32; i += 4) copy(piece_at<128>(buf, i + lane / 8, lane % 8), i + lane / 8, lane % 8);
  } else {
#pragma unroll
    for (int i = 0; i < 32; i += 8) copy(piece_at<64>(buf, i + lane / 4, lane % 4), i + lane / 4, lane % 4);
  }
}

__device__ __forceinline__ void get_saved(uint32_t buf, int row, bool f32, DenseType t, float (&v)[32]) {
  if (f32) {
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint4 w = lds_piece(piece_at<128>(buf, row, c));
      v[4 * c] = __uint_as_float(w.x), v[4 * c + 1] = __uint_as_float(w.y);
      v[4 * c + 2] = __uint_as_float(w.z), v[4 * c + 3] = __uint_as_float(w.w);
    }
  } else {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 w = lds_piece(piece_at<64>(buf, row, c));
      unpack16(w.x, t, v[8 * c], v[8 * c + 1]);
      unpack16(w.y, t, v[8 * c + 2], v[8 * c + 3]);
      unpack16(w.z, t, v[8 * c + 4], v[8 * c + 5]);
      unpack16(w.w, t, v[8 * c + 6], v[8 * c + 7]);
    }
  }
}

__device__ __forceinline__ void as_floats(const uint32_t (&r)[32], float (&v)[32]) {
#pragma unroll
  for (int k = 0; k < 32; ++k) v[k] = __uint_as_float(r[k]);
}

struct PairProblem {
  CUtensorMap a, b;
  int M, N, K;
  int mt, nt, end;         // tiles of 256 rows, of columns; units of this product and those before
  bool amn, bmn;
  bool out_f32, accumulate;  // (accumulate: 16-bit operands)
  bool vec;                  // columns in pieces of 8, rows on 16-byte boundaries: always, but in E4M3
  void* out;
  int64_t ld_out;
};

constexpr int kPairProblems = 3;

// The pairs take the `heavy` first tiles, those of the products with the longest K, in turn: pair
// p tiles p, p + pairs, ...; `more` pairs then have one more of them than the others, which take
// `light` of the remaining tiles each to be even, and the rest goes round again, from pair
// `rest` on, the first that has less to do.
struct PairArgs {
  PairProblem p[kPairProblems];
  int BN, units;
  int heavy, more, light, rest;
  DenseAct act;
  DenseType type;
  const uint8_t *sa, *sb;
  int sa_pitch, sb_pitch;
  void* saved;
  bool saved_f32;
  void* dgu;
  uint32_t* status;
  uint64_t wait_ns;  // limit of every wait
  bool withhold;     // a test: one copy is never made, so that a wait runs out
};

template <bool F8, DenseEpi EPI>
__global__ void __launch_bounds__(kDThreads, 1) dense_pair_kernel(const __grid_constant__ PairArgs g) {
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[kDStages], empty_bar[kDStages];
  __shared__ __align__(8) uint64_t accf_bar[2], acce_bar[2], drain_bar;
  __shared__ __align__(8) uint64_t sff_bar[kSfSlots], sfe_bar[kSfSlots];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t sfbase = sbase + PairSmem<F8>::kSf;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int pair0 = (int)(blockIdx.x >> 1), pairs = (int)(gridDim.x >> 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kDStages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 2);  // A and B
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&accf_bar[i]), 1);
      mbar_init(smem_u32(&acce_bar[i]), 2 * kDEpiWarps);
    }
    for (int i = 0; i < kSfSlots; ++i) {
      mbar_init(smem_u32(&sff_bar[i]), 2);
      mbar_init(smem_u32(&sfe_bar[i]), 1);
    }
    mbar_init(smem_u32(&drain_bar), 1);
    abort_sh = 0;
    fence_mbar_init();
    prefetch_tensormap(&g.p[0].a);
    prefetch_tensormap(&g.p[0].b);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&tmem_base_sh), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  volatile int* abort = &abort_sh;
  pdl_wait();

  constexpr int kStep = F8 ? 128 : 64;  // elements of K per stage: 128 bytes
  constexpr int kRowM = 8;              // row tiles of one sweep
  const int BN = g.BN, hb = BN / 2;     // (kEpiGate: hb columns of h, their gate and up)
  const bool overlap = F8 && BN > 192;  // the accumulators share columns
  const uint32_t acc_next = F8 ? 192u : 256u;
  // the i-th unit of this pair, or `units`
  auto unit = [&](int i) {
    if (F8 || EPI != kEpiStore) return min(pair0 + i * pairs, g.units);
    int u = pair0 + i * pairs;
    if (u < g.heavy) return u;
    i -= (g.heavy - pair0 + pairs - 1) / pairs;  // those it had of the heavy ones
    const int others = pairs - g.more;
    if (pair0 >= g.more) {
      if (i < g.light) return min(g.heavy + pair0 - g.more + i * others, g.units);
      i -= g.light;
    }
    const int first = pair0 - g.rest + (pair0 < g.rest ? pairs : 0);
    return min(g.heavy + g.light * others + first + i * pairs, g.units);
  };
  // unit u -> product, row and column tile
  auto tile = [&](int u, int& m, int& n) -> const PairProblem& {
    int i = 0;
    if (!F8 && EPI == kEpiStore)
      while (u >= g.p[i].end) ++i;
    const PairProblem& p = g.p[i];
    if (i) u -= g.p[i - 1].end;
    const int band = u / (kRowM * p.nt), r = u - band * kRowM * p.nt;
    const int rows = min(kRowM, p.mt - band * kRowM);
    n = r / rows;
    m = band * kRowM + (r - n * rows);
    return p;
  };

  if (warp == 0 || warp == 3) {
    // ------------------------------------------------------------ loads
    // A warp for each operand; both CTAs' copies of it complete on the leader's barrier.
    const bool one = elect_one(), is_b = warp == 3;
    int stage = 0;
    uint32_t phase = 0, issued = 0, last_parity = 0;
    for (int i = 0, u; (u = unit(i)) < g.units && !__any_sync(0xFFFFFFFFu, *abort); ++i) {
      int m, n;
      const PairProblem& p = tile(u, m, n);
      const int KB = (p.K + kStep - 1) / kStep;
      const CUtensorMap* map = is_b ? &p.b : &p.a;
      const bool mn = !F8 && (is_b ? p.bmn : p.amn);
      // kEpiGate: the leader stages the gate rows, its peer the up rows
      const int row = !is_b             ? m * 256 + (int)rank * 128
                      : EPI == kEpiGate ? n * hb + (rank ? p.N : 0)
                                        : n * BN + (int)rank * hb;
      const int height = is_b ? hb : 128;
      const bool two = mn && height > 64;
      const uint32_t bytes = 2 * (mn ? (two ? 16384u : 8192u) : height * 128u), at = sbase + (is_b ? kDBytesA : 0u);
      bool ok = true;
      for (int kb = 0; kb < KB; ++kb) {
        if (!warp_wait(smem_u32(&empty_bar[stage]), phase ^ 1u, abort, g.status, g.wait_ns)) {
          ok = false;
          break;
        }
        const uint32_t st = at + stage * kDStage;
        const uint32_t fb = mapa_shared(smem_u32(&full_bar[stage]), 0);
        if (one) {
          if (leader) mbar_arrive_expect_tx(smem_u32(&full_bar[stage]), bytes);
          // (withheld: the leader expects the bytes all the same)
          if (!g.withhold || !is_b || blockIdx.x != 1 || i != 0 || kb != KB - 1) {
            tma_load_2d_pair(st, map, fb, mn ? row : kb * kStep, mn ? kb * kStep : row);
            if (two) tma_load_2d_pair(st + 8192, map, fb, row + 64, kb * kStep);
          }
        }
        issued |= 1u << stage;
        last_parity = (last_parity & ~(1u << stage)) | (phase << stage);
        if (++stage == kDStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!ok) break;
    }
    // Every copy has landed before the CTAs leave (the leader's barriers count both CTAs'
    // bytes); after an abort, when some may not have come, they get 100 us.
    const uint64_t t0 = globaltimer_ns();
    if (leader) {
      for (int s = 0; s < kDStages; ++s) {
        if (!(issued & (1u << s))) continue;
        while (!mbar_try_wait(smem_u32(&full_bar[s]), (last_parity >> s) & 1u) &&
               globaltimer_ns() - t0 < (*abort ? 100000ull : g.wait_ns)) {
        }
      }
    } else if (*abort) {
      while (globaltimer_ns() - t0 < 100000ull) {
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    if (leader) {
      const bool one = elect_one();
      const uint32_t idesc1 = (F8 ? idesc_mxf8_e4m3(256, 0) : idesc_16(256, 0, g.type == kBF16, false, false)) |
                              ((uint32_t)(BN >> 3) << 17);
      int stage = 0;
      uint32_t phase = 0, group = 0;
      // The next stage is probed between this one's MMAs and their commit, and the answer looked
      // at a K block later.  (In twos, as below, a K block of a tile alone takes 0.25 us, one by one
      // 0.26.)
      bool ready = mbar_test_wait_cluster(smem_u32(&full_bar[0]), 0);
      for (int i = 0, u; (u = unit(i)) < g.units; ++i) {
        int m, n;
        const PairProblem& p = tile(u, m, n);
        const int KB = (p.K + kStep - 1) / kStep;
        const bool amn = !F8 && p.amn, bmn = !F8 && p.bmn;
        const uint32_t idesc0 = idesc1 | ((uint32_t)amn << 15) | ((uint32_t)bmn << 16);
        const uint64_t step_a = amn ? 128 : 2, step_b = bmn ? 128 : 2;  // 16 K rows, or 32 bytes of a row
        const int b = i & 1;
        // overlapping: every warp has left the tile before last, and the tile before the columns
        // that both buffers have; else the tile before last
        if (!warp_wait<true>(smem_u32(&acce_bar[overlap ? 0 : b]), ((overlap ? i : i >> 1) & 1) ^ 1u, abort, g.status, g.wait_ns))
          break;
        tc_fence_after();
        const uint32_t acc = tmem + (b ? acc_next : 0u);
        bool ok = true;
        uint32_t sf = 0, slot = 0;
#pragma unroll 2
        for (int kb = 0; kb < KB; ++kb) {
          const uint32_t j = (uint32_t)kb & 3u;
          if (F8 && j == 0) {
            slot = group & (kSfSlots - 1);
            if (!warp_wait<true>(smem_u32(&sff_bar[slot]), (group / kSfSlots) & 1u, abort, g.status, g.wait_ns)) {
              ok = false;
              break;
            }
            ++group;
            sf = tmem + kDTmemSf + slot * kDSfCols;
          }
          if (!__all_sync(0xFFFFFFFFu, ready) &&
              !warp_wait<true>(smem_u32(&full_bar[stage]), phase, abort, g.status, g.wait_ns)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = sbase + stage * kDStage;
          const uint64_t ad = amn ? sdesc_mn_sw128(st) : sdesc_k_sw128(st);
          const uint64_t bd = bmn ? sdesc_mn_sw128(st + kDBytesA) : sdesc_k_sw128(st + kDBytesA);
          if (one) {
            if (F8 && j == 0) {
              const uint32_t sp = sfbase + slot * kSfSlotBytes;
              tc_cp_sf_atom_pair(sf, sdesc_sf_atom(sp));
              tc_cp_sf_atom_pair(sf + 8, sdesc_sf_atom(sp + 512));
              tc_cp_sf_atom_pair(sf + 12, sdesc_sf_atom(sp + 1024));
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const uint32_t add = (kb | k) != 0 ? 1u : 0u;
              const uint64_t da = ad + step_a * k, db = bd + step_b * k;
              if constexpr (F8)
                tc_mma_mxf8_pair(acc, da, db, idesc0 | (j << 4) | (j << 29), sf, sf + 8, add);
              else
                tc_mma_16_pair(acc, da, db, idesc0, add);
            }
          }
          const uint32_t done = smem_u32(&empty_bar[stage]);
          if (++stage == kDStages) {
            stage = 0;
            phase ^= 1u;
          }
          ready = mbar_test_wait_cluster(smem_u32(&full_bar[stage]), phase);
          if (one) {
            tc_commit_pair_multicast(done, 0x3);
            if (F8 && (j == 3 || kb == KB - 1)) tc_commit_pair_multicast(smem_u32(&sfe_bar[slot]), 0x3);
          }
        }
        if (!ok) break;
        if (one) tc_commit_pair_multicast(smem_u32(&accf_bar[b]), 0x3);
      }
      if (one) tc_commit_pair(smem_u32(&drain_bar));
      const uint64_t t0 = globaltimer_ns();
      while (!mbar_try_wait(smem_u32(&drain_bar), 0) && globaltimer_ns() - t0 < g.wait_ns) {
      }
    }
    __syncwarp();
  } else if (F8 && warp == 2) {
    // ------------------------------------------------------------ scales
    // Lane l holds the words of rows l, l + 32, l + 64, l + 96: 16 consecutive bytes of an
    // atom.  Rows past M have no scale (their sums are not stored).
    const PairProblem& p = g.p[0];
    const int KB = p.K / kStep, KQ = (KB + 3) / 4, NB = (p.N + 127) / 128;
    // The words of the next two groups of four K blocks are under way while one is written: a
    // load's time is that of a group's MMAs.
    struct Words {
      uint32_t w[4], b[3];  // of the rows, and of the up to three blocks that the columns are of
      int first;            // the tile's first column in its block, in groups of 32; -1: past the last tile
    } even, odd;
    int t = 0, q = 0, m = 0, n = 0, u = unit(0);
    if (u < g.units) tile(u, m, n);
    auto load = [&](Words& x) {
      x.first = u < g.units ? n * BN % 128 / 32 : -1;
      if (u >= g.units) return;
      scale_words(g.sa, (int64_t)m * 256 + rank * 128 + lane, p.M, g.sa_pitch, KB, q, x.w);
#pragma unroll
      for (int i = 0; i < 3; ++i) x.b[i] = block_word(g.sb, min(n * BN / 128 + i, NB - 1), g.sb_pitch, q);
      if (++q == KQ) {
        q = 0;
        if ((u = unit(++t)) < g.units) tile(u, m, n);
      }
    };
    uint32_t group = 0;
    auto emit = [&](const Words& x) {
      const uint32_t slot = group & (kSfSlots - 1);
      if (x.first < 0 || !warp_wait(smem_u32(&sfe_bar[slot]), ((group / kSfSlots) & 1u) ^ 1u, abort, g.status, g.wait_ns))
        return false;
      uint32_t c[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) c[i] = i + x.first < 4 ? x.b[0] : i + x.first < 8 ? x.b[1] : x.b[2];
      uint8_t* sp = smem + PairSmem<F8>::kSf + slot * kSfSlotBytes + lane * 16;
      *reinterpret_cast<uint4*>(sp) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
      *reinterpret_cast<uint4*>(sp + 512) = make_uint4(c[0], c[1], c[2], c[3]);
      *reinterpret_cast<uint4*>(sp + 1024) = make_uint4(c[4], c[5], c[6], c[7]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_u32(&sff_bar[slot]), 0));
      ++group;
      return true;
    };
    load(even);
    load(odd);
    while (emit(even)) {
      load(even);
      if (!emit(odd)) break;
      load(odd);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3, half = (warp - 4) >> 2;
    const uint32_t tlane = tmem + ((uint32_t)(q * 32) << 16);
    const uint32_t epi = PairSmem<F8>::kEpi + (uint32_t)(warp - 4) * PairSmem<F8>::kEpiWarp;
    const uint32_t buf = sbase + epi;
    for (int i = 0, u; (u = unit(i)) < g.units; ++i) {
      int m, n;
      const PairProblem& p = tile(u, m, n);
      const int N = p.N, b = i & 1;
      const int64_t row0 = (int64_t)m * 256 + rank * 128 + q * 32, ld = p.ld_out;
      const int rows = (int)max((int64_t)0, min((int64_t)32, p.M - row0));  // of this warp
      const int ss = g.saved_f32 ? 4 : 2;
      uint8_t* saved = reinterpret_cast<uint8_t*>(g.saved) + row0 * 2 * N * ss;
      const int64_t saved_pitch = (int64_t)2 * N * ss;
      auto fetch = [&](int up, int col) {  // gate to the first buffer, up to the second
        fetch_saved(buf + 4096 * up, saved + ((int64_t)up * N + col) * ss, saved_pitch, rows, (N - col) * ss, g.saved_f32,
                    lane);
      };
      if constexpr (EPI == kEpiGrad) {
        fetch(0, n * BN + half * hb);
        fetch(1, n * BN + half * hb);
      }
      if (!warp_wait(smem_u32(&accf_bar[b]), (i >> 1) & 1, abort, g.status, g.wait_ns)) break;
      tc_fence_after();
      const uint32_t acc = tlane + (b ? acc_next : 0u);
      auto release = [&](int bar) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster_relaxed(mapa_shared(smem_u32(&acce_bar[bar]), 0));
      };
      if constexpr (EPI == kEpiStore) {
        // the columns that both buffers have are the first one's last 64 and the second
        // one's first: their half drains them first, the other half has left the tile before
        if (overlap && half == b) release(0);
        const int groups = (hb + 63) / 64;
#pragma unroll 1
        for (int k = 0; k < groups; ++k) {
          const int cc = half * hb + (overlap && b == 0 ? k ^ 1 : k) * 64, width = min(64, half * hb + hb - cc);
          const int col = n * BN + cc, cols = min(width, N - col);
          uint32_t r[2][32];
          tmem_ld32(acc + cc, r[0]);
          if (width > 32) tmem_ld32(acc + cc + 32, r[1]);
          tmem_ld_wait();
          if (overlap ? k == 0 && half != b : k == groups - 1) release(overlap ? 0 : b);
          if (rows == 0 || cols <= 0) continue;
          float v[32];
          if (p.out_f32) {
            float* out = reinterpret_cast<float*>(p.out) + row0 * ld + col;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const int left = cols - 32 * h;
              if (left <= 0) break;
              as_floats(r[h], v);
              __syncwarp();
              put_f32(buf, lane, v);
              __syncwarp();
              uint8_t* dst = reinterpret_cast<uint8_t*>(out + 32 * h);
              if (F8 && !p.vec)
                flush_elements(smem + epi, out + 32 * h, ld, rows, left, lane);
              else if (!F8 && p.accumulate)
                flush<128, true>(buf, dst, ld * 4, rows, left * 4, lane);
              else
                flush<128>(buf, dst, ld * 4, rows, left * 4, lane);
            }
          } else {
            __syncwarp();
            as_floats(r[0], v);
            put_16<128>(buf, lane, 0, v, g.type);
            if (width > 32) {
              as_floats(r[1], v);
              put_16<128>(buf, lane, 4, v, g.type);
            }
            __syncwarp();
            uint16_t* out = reinterpret_cast<uint16_t*>(p.out) + row0 * ld + col;
            if (!F8 || p.vec)
              flush<128>(buf, reinterpret_cast<uint8_t*>(out), ld * 2, rows, cols * 2, lane);
            else
              flush_elements(smem + epi, out, ld, rows, cols, lane);
          }
        }
      } else if constexpr (EPI == kEpiGate) {
        // 32 columns at a time, in turn by the two halves
        const int chunks = hb / 32;
        if (half >= chunks) release(b);
#pragma unroll 1
        for (int c = half; c < chunks; c += 2) {
          const int cc = c * 32, col = n * hb + cc;
          uint32_t rg[32], ru[32];
          tmem_ld32(acc + cc, rg);
          tmem_ld32(acc + hb + cc, ru);
          tmem_ld_wait();
          if (c + 2 >= chunks) release(b);
          float gv[32], uv[32];
          as_floats(rg, gv);
          as_floats(ru, uv);
          if (g.saved && rows && col < N) {
            __syncwarp();
            const int bytes = (N - col) * ss;
            uint8_t* dst = saved + (int64_t)col * ss;
            if (g.saved_f32) {
              put_f32(buf, lane, gv);
              put_f32(buf + 4096, lane, uv);
              __syncwarp();
              flush<128>(buf, dst, saved_pitch, rows, bytes, lane);
              flush<128>(buf + 4096, dst + (int64_t)N * 4, saved_pitch, rows, bytes, lane);
            } else {
              put_16<64>(buf, lane, 0, gv, g.type);
              put_16<64>(buf + 4096, lane, 0, uv, g.type);
              __syncwarp();
              flush<64>(buf, dst, saved_pitch, rows, bytes, lane);
              flush<64>(buf + 4096, dst + (int64_t)N * 2, saved_pitch, rows, bytes, lane);
            }
          }
          gate_values(g.act, gv, uv);
          if (rows && col < N) {
            __syncwarp();
            put_16<64>(buf, lane, 0, uv, g.type);
            __syncwarp();
            flush<64>(buf, reinterpret_cast<uint8_t*>(p.out) + (row0 * ld + col) * 2, ld * 2, rows,
                      (N - col) * 2, lane);
          }
        }
      } else {
        // The saved gate and up of the next 32 columns are under way while these are
        // finished: up at once, gate when its buffer, which dg and du and then h leave
        // through, is free.
#pragma unroll 1
        for (int c = 0; c < hb / 32; ++c) {
          const int col = n * BN + half * hb + c * 32;
          asm volatile("cp.async.wait_all;" ::: "memory");
          __syncwarp();
          float gv[32], uv[32];
          get_saved(buf, lane, g.saved_f32, g.type, gv);
          get_saved(buf + 4096, lane, g.saved_f32, g.type, uv);
          __syncwarp();
          if (c < hb / 32 - 1) fetch(1, col + 32);
          uint32_t r[32];
          tmem_ld32(acc + half * hb + c * 32, r);
          tmem_ld_wait();
          if (c == hb / 32 - 1) release(b);
          float hv[32];
          as_floats(r, hv);
          gradient_values(g.act, hv, gv, uv);
          if (rows && col < N) {
            const int bytes = (N - col) * 2;
            put_16<64>(buf, lane, 0, gv, g.type);
            put_16<64>(buf + 2048, lane, 0, uv, g.type);
            __syncwarp();
            uint8_t* dst = reinterpret_cast<uint8_t*>(g.dgu) + (row0 * 2 * N + col) * 2;
            flush<64>(buf, dst, (int64_t)4 * N, rows, bytes, lane);
            flush<64>(buf + 2048, dst + (int64_t)2 * N, (int64_t)4 * N, rows, bytes, lane);
            if (p.out) {
              __syncwarp();
              put_16<64>(buf, lane, 0, hv, g.type);
              __syncwarp();
              flush<64>(buf, reinterpret_cast<uint8_t*>(p.out) + (row0 * ld + col) * 2, ld * 2, rows, bytes,
                        lane);
            }
          }
          __syncwarp();
          if (c < hb / 32 - 1) fetch(0, col + 32);
        }
      }
    }
    if (EPI == kEpiGrad) asm volatile("cp.async.wait_all;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  cluster_sync_all();  // neither CTA frees TMEM the pair still uses
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ------------------------------------------------------------------------- launches
constexpr uint64_t kWithheldNs = 20000000ull;  // the limit under the watchdog's test

static bool encode_map(CUtensorMap* map, const DenseOperand& o, int K, DenseType t, int box_rows) {
  // (looked up once, by whichever host thread comes first)
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool found = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                           cudaSuccess &&
                       q == cudaDriverEntryPointSuccess;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(found ? p : nullptr);
  }();
  if (!fn) return false;
  const cuuint64_t es = t == kE4M3 ? 1 : 2;
  const cuuint64_t dims[2] = {(cuuint64_t)(o.mn ? o.rows : K), (cuuint64_t)(o.mn ? K : o.rows)};
  const cuuint64_t strides[1] = {(cuuint64_t)o.ld * es};
  const cuuint32_t box[2] = {(cuuint32_t)(128 / es), (cuuint32_t)(o.mn ? 64 : box_rows)};
  const cuuint32_t one[2] = {1, 1};
  return fn(map,
            t == kE4M3  ? CU_TENSOR_MAP_DATA_TYPE_UINT8
            : t == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                         : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            2, const_cast<void*>(o.p), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <bool F8, DenseEpi EPI>
static cudaError_t launch_pair(const PairArgs& g, int pairs, cudaStream_t s) {
  cudaLaunchAttribute c;
  c.id = cudaLaunchAttributeClusterDimension;
  c.val.clusterDim.x = 2;
  c.val.clusterDim.y = 1;
  c.val.clusterDim.z = 1;
  return launch_k(dense_pair_kernel<F8, EPI>, dim3(2 * (g.units < pairs ? g.units : pairs)), dim3(kDThreads),
                  PairSmem<F8>::kBytes, s, true, &c, g);
}

cudaError_t dense_set_attributes() {
  const void* ks[4] = {(const void*)dense_pair_kernel<true, kEpiStore>, (const void*)dense_pair_kernel<false, kEpiStore>,
                       (const void*)dense_pair_kernel<false, kEpiGate>, (const void*)dense_pair_kernel<false, kEpiGrad>};
  for (int i = 0; i < 4; ++i) {
    const uint32_t bytes = i ? PairSmem<false>::kBytes : PairSmem<true>::kBytes;
    const cudaError_t e = cudaFuncSetAttribute(ks[i], cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e != cudaSuccess) return e;
  }
  return dense_split_set_attributes();
}

// The tiles' columns: the width with which the fullest pair has the least to do, and its time in
// microseconds.  Fitted, as the split kernel's, to the times of 90 E4M3 products (1 to 8192
// tokens, 64 to 8192 weight rows, K from 128 to 7168) in each width and split: one K block of 128
// bytes 0.31 us with 64 columns, 0.35 with 256; start, first copies and last tile 4.2 and 5.4
// us, 2.6 more with gate and gradient.  512 x 4096 x 2048 takes 9.3 us with 128 columns, 10.3
// with 256; 1021 x 4096 x 7168 44 and 25; 8192 x 256 x 7168 27 and 25 (20.3 by the split kernel).
// The outputs were BF16: float ones and rows off 16-byte boundaries take longer, which is not in
// it (1021 x 10007 x 1408 into float: 17 us by this, 27 measured).
static double pair_columns(const DenseGemm* g, int count, int pairs, int* columns) {
  double least = 0;
  for (int BN = 256; BN >= 64; BN -= 64) {
    const double w = BN / 256.0, block = 0.31 + 0.04 * w * w;
    double sum = 0, one = 0;
    int64_t units = 0;
    for (int i = 0; i < count; ++i) {
      const int cols = g[i].epi == kEpiGate ? BN / 2 : BN;
      const int64_t n = (int64_t)((g[i].M + 255) / 256) * ((g[i].N + cols - 1) / cols);
      const int KB = (g[i].K + (g[i].type == kE4M3 ? 127 : 63)) / (g[i].type == kE4M3 ? 128 : 64);
      double us = KB * block;
      if (count > 1) {
        // the gradients' MN-major operands come in boxes of 64: as many bytes for 192 columns as for
        // 256, half for 128; and a tile that sums few rows takes its stores' time (25 tokens, 3224 x
        // 1928: the step 45.8 us, by K alone 50.5)
        if (BN > 128) us += KB * 0.08;
        if (us < 0.7 + 2.2 * w) us = 0.7 + 2.2 * w;
      }
      us += 0.4;
      units += n;
      sum += n * us;
      if (us > one) one = us;
    }
    // one product: whole waves; several: their sum, and half a tile that does not fill up
    double us = count == 1 ? (double)((units + pairs - 1) / pairs) * one : sum / pairs + 0.5 * one;
    if (us < one) us = one;
    // a few tiles of long rows wait for memory: 2.9 TB/s, 100 GB/s for a pair
    const double mb = count == 1 ? ((double)g->M + g->N) * g->K * (g->type == kE4M3 ? 1e-6 : 2e-6) : 0;
    const double rate = units < 29 ? 0.1 * units : 2.9;
    if (us < mb / rate) us = mb / rate;
    us += 3.8 + (g->epi == kEpiStore ? 1.6 : 4.2) * w;
    if (BN == 256 || us < least) {
      least = us;
      *columns = BN;
    }
  }
  return least;
}

static cudaError_t pair_gemm(const DenseGemm* g, int count, int BN, int pairs, cudaStream_t s) {
  PairArgs d = {};
  d.BN = BN;
  for (int i = 0; i < count; ++i) {
    PairProblem& p = d.p[i];
    if (!encode_map(&p.a, g[i].a, g[i].K, g[i].type, 128) || !encode_map(&p.b, g[i].b, g[i].K, g[i].type, BN / 2))
      return cudaErrorInvalidValue;
    p.M = g[i].M;
    p.N = g[i].N;
    p.K = g[i].K;
    const int cols = g[i].epi == kEpiGate ? BN / 2 : BN;
    p.mt = (p.M + 255) / 256;
    p.nt = (p.N + cols - 1) / cols;
    d.units += p.mt * p.nt;
    p.end = d.units;
    p.amn = g[i].a.mn;
    p.bmn = g[i].b.mn;
    p.out_f32 = g[i].out_f32;
    p.accumulate = g[i].accumulate;
    p.vec = p.N % 8 == 0 && (uintptr_t)g[i].out % 16 == 0;
    p.out = g[i].out;
    p.ld_out = g[i].ld_out;
  }
  // (the products come with the longest K first)
  const int ctas = d.units < pairs ? d.units : pairs;
  for (int i = 0; i < count && g[i].K == g[0].K; ++i) d.heavy = d.p[i].end;
  d.more = d.heavy % ctas;
  d.light = count > 1 && d.heavy < d.units ? (g[0].K + g[count - 1].K / 2) / g[count - 1].K : 0;
  d.rest = (int64_t)d.light * g[count - 1].K > g[0].K ? 0 : d.more;
  d.act = g->act;
  d.type = g->type;
  d.sa = g->sa;
  d.sb = g->sb;
  d.sa_pitch = g->sa_pitch;
  d.sb_pitch = scale_pitch(g->K);
  d.saved = g->saved;
  d.saved_f32 = g->saved_f32;
  d.dgu = g->dgu;
  d.status = g->status;
  d.wait_ns = g->withhold ? kWithheldNs : kWaitLimitNs;
  d.withhold = g->withhold;
  if (g->type == kE4M3) return launch_pair<true, kEpiStore>(d, pairs, s);
  if (g->epi == kEpiGate) return launch_pair<false, kEpiGate>(d, pairs, s);
  if (g->epi == kEpiGrad) return launch_pair<false, kEpiGrad>(d, pairs, s);
  return launch_pair<false, kEpiStore>(d, pairs, s);
}

static cudaError_t split_gemm(const DenseGemm& g, DenseSplit p, cudaStream_t s) {
  CUtensorMap a, b;
  p.early = g.early;
  if ((!g.x && !encode_map(&a, g.a, g.K, g.type, p.NT)) || !encode_map(&b, g.b, g.K, g.type, g.epi == kEpiGate ? 64 : 128))
    return cudaErrorInvalidValue;
  DenseArgs d = {};
  d.M = g.M;
  d.N = g.N;
  d.K = g.K;
  d.act = g.act;
  d.type = g.type;
  d.sa = g.sa;
  d.sb = g.sb;
  d.sa_pitch = g.sa_pitch;
  d.sb_pitch = scale_pitch(g.K);
  d.x = g.x;
  d.ldx = g.ldx;
  d.out = g.out;
  d.ld_out = g.ld_out;
  d.out_f32 = g.out_f32;
  d.saved = g.saved;
  d.saved_f32 = g.saved_f32;
  d.dgu = g.dgu;
  d.status = g.status;
  d.wait_ns = g.withhold ? kWithheldNs : kWaitLimitNs;
  d.withhold = g.withhold;
  d.vec = g.N % 8 == 0 && (uintptr_t)g.out % 16 == 0;
  return dense_split_launch(a, b, g, d, p, s);
}

// Which kernel: the one that the measured times above say is faster.
struct DenseChoice {
  bool pairs;
  int BN;          // of the pairs
  DenseSplit split;
};

static DenseChoice choose(const DenseGemm& g, int sms) {
  DenseChoice c = {};
  const double pair_us = pair_columns(&g, 1, sms / 2, &c.BN);
  c.split = dense_split_plan(g, sms);
  c.pairs = !(c.split.us < pair_us || g.x);
  return c;
}

// The longest K first.
static void sort_products(DenseGemm* g, int count) {
  for (int i = 1; i < count; ++i)
    for (int j = i; j > 0 && g[j].K > g[j - 1].K; --j) std::swap(g[j], g[j - 1]);
}

cudaError_t dense_gemm(const DenseGemm& g, int sms, cudaStream_t s) {
  const DenseChoice c = choose(g, sms);
  return c.pairs ? pair_gemm(&g, 1, c.BN, sms / 2, s) : split_gemm(g, c.split, s);
}

cudaError_t dense_gemms(DenseGemm* g, int count, int sms, cudaStream_t s) {
  sort_products(g, count);
  int BN = 256;
  pair_columns(g, count, sms / 2, &BN);
  return pair_gemm(g, count, BN, sms / 2, s);
}

moe_dense_launch dense_choice(DenseGemm* g, int count, int sms) {
  DenseChoice c = {};
  if (count == 1) {
    c = choose(*g, sms);
  } else {
    c.pairs = true;
    sort_products(g, count);
    pair_columns(g, count, sms / 2, &c.BN);
  }
  moe_dense_launch l = {};
  l.pairs = c.pairs;
  l.width = c.pairs ? c.BN : c.split.NT;
  l.split = c.pairs ? 1 : c.split.split;
  for (int i = 0; i < count && c.pairs; ++i) {
    const int cols = g[i].epi == kEpiGate ? c.BN / 2 : c.BN;
    l.tiles += (int64_t)((g[i].M + 255) / 256) * ((g[i].N + cols - 1) / cols);
  }
  if (!c.pairs) l.tiles = (int64_t)c.split.tt * c.split.rt;
  return l;
}

}  // namespace mm
