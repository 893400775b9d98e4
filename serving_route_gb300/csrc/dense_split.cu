// dense_split.cu -- the dense products where a few tiles cannot fill the GPU: few tokens,
// small matrices.
//
// d^T[n, m] = sum_k b[n, k] a[m, k]: 128 rows of B (the weights) are the MMA's M operand and
// NT <= 128 rows of A (the tokens, a multiple of 16) its N operand, so a K block of a tile
// costs 16 KB of weights and 128 NT bytes of tokens.  What bounds these products is the
// weights' time, so every SM has to stream its share of them: the K blocks of a tile
// are split over a cluster of up to 8 CTAs, each of which sums its share in tensor
// memory.  The shares meet in the cluster's shared memory: every CTA leaves its FP32 sums in its
// own, and after one cluster barrier each finishes every s-th token of the tile, adding
// the shares in the order of the CTAs.  No workspace, no counters, no order that changes.
// Two CTAs per SM overlap one's join with the other's stream.
// FUSE (E4M3, up to 16 tokens): the tokens come in BF16 and the CTAs quantise what they need of
// them themselves, a warp for each ring place, straight into it: a kernel less before the
// stream (4096 x 7168, one token: 8.6 -> 7.2 us, 6.2 with what came after), for 16 x 256 bytes a K block from L2.
// Warps: 0 and 3 loads, 1 MMAs, 2 scales, 4-7 drain the accumulator (thread = weight row); all
// eight finish tokens (a lane has consecutive columns, so stores are whole lines).
#include "dense.cuh"

namespace mm {

constexpr int kSpThreads = 256;
constexpr int kSpWarps = kSpThreads / 32;
constexpr int kSpMaxStages = 8;
constexpr uint32_t kSpW = 16384;            // 128 weight rows x 128 bytes
constexpr uint32_t kSpSfBytes = 1024;       // weights' atom, tokens' atom
constexpr int kSpSfSlots = 4;
constexpr uint32_t kSpSfCols = 16;
constexpr int kSpFusedSlots = 7;  // more than ring places: a slot's MMAs are done when it comes again

__device__ __forceinline__ void tc_mma_16(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ float2 ld_cluster_v2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

// C consecutive columns of a row, of which those below n exist; whole where `vec`
// (n a multiple of C, rows on C elements' boundaries).
template <int C>
__device__ __forceinline__ void store_few(void* base, int64_t at, int c, int n, const float (&v)[C], bool f32,
                                          DenseType t, bool vec) {
  if (f32) {
    float* p = reinterpret_cast<float*>(base) + at;
    if (vec) {
      if (c >= n) return;
      if constexpr (C == 4)
        *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
      else
        *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (c + i < n) p[i] = v[i];
    }
    return;
  }
  uint16_t* p = reinterpret_cast<uint16_t*>(base) + at;
  if (vec) {
    if (c >= n) return;
    if constexpr (C == 4)
      *reinterpret_cast<uint2*>(p) = make_uint2(pack16(v[0], v[1], t), pack16(v[2], v[3], t));
    else
      *reinterpret_cast<uint32_t*>(p) = pack16(v[0], v[1], t);
  } else {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (c + i < n) p[i] = bits16(v[i], t);
  }
}

// (n a multiple of 4)
__device__ __forceinline__ float4 load_four(const void* base, int64_t at, bool f32, DenseType t) {
  if (f32) return *reinterpret_cast<const float4*>(reinterpret_cast<const float*>(base) + at);
  const uint2 w = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(base) + at);
  float4 v;
  unpack16(w.x, t, v.x, v.y);
  unpack16(w.y, t, v.z, v.w);
  return v;
}

// One K block of up to 16 tokens from BF16 to E4M3 with a power-of-two scale, as
// quantize_rows_kernel's: to `rows` as TMA's 128-byte swizzle would leave it, and the scales to
// an atom whose four bytes are alike.  Two lanes to a token, 64 columns each.
__device__ __forceinline__ void quantize_block(const uint16_t* x, int64_t ld, int tokens, uint32_t rows, uint32_t atom) {
  const int lane = threadIdx.x & 31, t = lane >> 1, h = lane & 1;
  uint4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    v[i] = t < tokens ? *reinterpret_cast<const uint4*>(x + t * ld + h * 64 + i * 8) : make_uint4(0u, 0u, 0u, 0u);
  uint32_t m = v[0].x & 0x7FFF7FFFu;  // the larger of each pair's halves (a NaN only where all are)
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
#pragma unroll
    for (int k = 0; k < 4; ++k) asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w[k] & 0x7FFF7FFFu));
  }
  asm("max.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(__shfl_xor_sync(0xFFFFFFFFu, m, 1)));
  const float amax = fmaxf(bf16_bits_to_float(m & 0xFFFFu), bf16_bits_to_float(m >> 16));
  const int e = pow2_scale_exp(amax);
  const float inv = block_factor(amax, e);
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 u = v[2 * c + i];
      q[2 * i] = e4m3x4(bf16_bits_to_float(u.x & 0xFFFFu) * inv, bf16_bits_to_float(u.x >> 16) * inv,
                        bf16_bits_to_float(u.y & 0xFFFFu) * inv, bf16_bits_to_float(u.y >> 16) * inv);
      q[2 * i + 1] = e4m3x4(bf16_bits_to_float(u.z & 0xFFFFu) * inv, bf16_bits_to_float(u.z >> 16) * inv,
                            bf16_bits_to_float(u.w & 0xFFFFu) * inv, bf16_bits_to_float(u.w >> 16) * inv);
    }
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(rows + t * 128 + (((4 * h + c) ^ (t & 7)) << 4)),
                 "r"(q[0]), "r"(q[1]), "r"(q[2]), "r"(q[3])
                 : "memory");
  }
  if (h == 0)
    asm volatile("st.shared.u32 [%0], %1;" ::"r"(atom + t * 16), "r"((uint32_t)(e + 127) * 0x01010101u) : "memory");
}

// (kEpiGrad multiplies W2 [K, N] as it lies: MN-major.)
template <bool F8, DenseEpi EPI, bool FUSE>
__global__ void __launch_bounds__(kSpThreads, 2)
    dense_split_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                       const DenseArgs g, const DenseSplit p) {
  constexpr bool BMN = EPI == kEpiGrad;
  extern __shared__ uint8_t dsmem[];
  __shared__ __align__(8) uint64_t full_bar[kSpMaxStages], empty_bar[kSpMaxStages];
  __shared__ __align__(8) uint64_t accf_bar, sff_bar[kSpSfSlots], sfe_bar[kSpSfSlots];
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  uint8_t* smem =
      reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(dsmem) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t stage_bytes = kSpW + (uint32_t)p.NT * 128u + (FUSE ? kSpSfBytes : 0u);
  uint8_t* sf_smem = smem + p.stages * stage_bytes;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = p.split > 1 ? (int)cluster_ctarank() : 0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(smem_u32(&full_bar[s]), 2);  // weights and tokens
      mbar_init(smem_u32(&empty_bar[s]), 1);
    }
    for (int i = 0; i < kSpSfSlots; ++i) {
      mbar_init(smem_u32(&sff_bar[i]), 1);
      mbar_init(smem_u32(&sfe_bar[i]), 1);
    }
    mbar_init(smem_u32(&accf_bar), 1);
    abort_sh = 0;
    fence_mbar_init();
    prefetch_tensormap(&tmA);
    prefetch_tensormap(&tmB);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&tmem_base_sh), p.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  volatile int* abort = &abort_sh;

  constexpr int kStep = F8 ? 128 : 64;
  const int KB = (g.K + kStep - 1) / kStep;
  const int unit = blockIdx.x / p.split;
  const int jt = unit / p.tt, m0 = (unit - jt * p.tt) * p.NT;  // weight tile, first token
  const int tokens = min(p.NT, g.M - m0);
  const int kb0 = (int)((int64_t)rank * KB / p.split), kb1 = (int)((int64_t)(rank + 1) * KB / p.split);
  const int n = kb1 - kb0;

  // The kernel before in the stream wrote the tokens, but not the weights where they are
  // `early`: their first loads do not wait for it.  (Beyond those the warp would only poll for
  // empty places, at the cost of the CTAs that still run.)
  if (warp != 0 || !p.early) {
    pdl_wait();
    pdl_trigger();  // (any thread's counts for the CTA: not before its wait)
  }
  if (warp == 0 || (warp == 3 && !FUSE)) {
    // ------------------------------------------------------------ loads
    // A warp for the weights, one for the tokens: wait, arrival and copy are a chain of
    // some 350 clocks a K block with both in one.
    const bool one = elect_one(), tokens_warp = warp == 3;
    const uint32_t bytes = tokens_warp ? (uint32_t)p.NT * 128u : kSpW;
    int st = 0, i = 0;
    uint32_t ph = 1u;
    for (; i < n; ++i) {
      if (i >= p.stages) {  // (the first places are free)
        if (i == p.stages && warp == 0 && p.early) pdl_wait();
        if (!warp_wait(smem_u32(&empty_bar[st]), ph, abort, g.status, g.wait_ns)) break;
      }
      if (one) {
        const uint32_t dst = sbase + st * stage_bytes + (tokens_warp ? kSpW : 0u), fb = smem_u32(&full_bar[st]);
        const int k = (kb0 + i) * kStep;
        mbar_arrive_expect_tx(fb, bytes);
        if (g.withhold && tokens_warp && blockIdx.x == 0 && i == n - 1) {
          // the bytes never come
        } else if (tokens_warp) {
          tma_load_2d(dst, &tmA, fb, k, m0);
        } else if (EPI == kEpiGate) {  // 64 gate rows, then their 64 up rows
          tma_load_2d(dst, &tmB, fb, k, jt * 64);
          tma_load_2d(dst + 8192, &tmB, fb, k, g.N + jt * 64);
        } else if (BMN) {
          tma_load_2d(dst, &tmB, fb, jt * 128, k);
          tma_load_2d(dst + 8192, &tmB, fb, jt * 128 + 64, k);
        } else {
          tma_load_2d(dst, &tmB, fb, k, jt * 128);
        }
      }
      if (++st == p.stages) {
        st = 0;
        ph ^= 1u;
      }
    }
    if (i <= p.stages && warp == 0 && p.early) pdl_wait();
    // Every copy has landed before the CTA leaves; after an abort, when one of the two may not
    // have come, they get 100 us.
    const uint64_t t0 = globaltimer_ns();
    for (int k = max(0, i - p.stages); k < i; ++k)
      while (!mbar_try_wait(smem_u32(&full_bar[k % p.stages]), (k / p.stages) & 1) &&
             globaltimer_ns() - t0 < (*abort ? 100000ull : g.wait_ns)) {
      }
    __syncwarp();
  }
  if (FUSE && warp >= 2) {
    // ------------------------------------------------------------ tokens, quantised here
    // A ring place is one warp's: a wait for its next use but one would take the parity of the
    // use before for it.
    const int st = warp - 2;
    uint32_t ph = 1u;
    for (int i = st; i < n && st < p.stages; i += p.stages, ph ^= 1u) {
      if (i >= p.stages && !warp_wait(smem_u32(&empty_bar[st]), ph, abort, g.status, g.wait_ns)) break;
      const uint32_t rows = sbase + st * stage_bytes + kSpW, atoms = rows + (uint32_t)p.NT * 128u;
      const uint32_t b = g.sb[(int64_t)jt * g.sb_pitch + kb0 + i] * 0x01010101u;  // one for the tile's weights
      quantize_block(g.x + m0 * g.ldx + (kb0 + i) * kStep, g.ldx, tokens, rows, atoms + 512u);
      asm volatile("st.shared.v4.u32 [%0], {%1,%1,%1,%1};" ::"r"(atoms + lane * 16), "r"(b) : "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && !(g.withhold && blockIdx.x == 0 && i == n - 1)) mbar_arrive(smem_u32(&full_bar[st]));
    }
    __syncwarp();
  }
  if (warp == 1) {
    // ------------------------------------------------------------ MMAs
    const bool one = elect_one();
    const uint32_t idesc0 = F8 ? idesc_mxf8_e4m3(128, 0) + ((uint32_t)(p.NT >> 3) << 17)
                               : idesc_16(128, 0, g.type == kBF16, BMN, false) + ((uint32_t)(p.NT >> 3) << 17);
    uint32_t sf = 0, slot = 0, group = 0;
    // The next place is probed between this one's MMAs and their commit.  (In twos a K block takes
    // 0.235 us, one by one 0.257, in fours 0.239: 128 x 7168 by one CTA.)
    int st = 0;
    uint32_t ph = 0;
    bool ready = mbar_test_wait(smem_u32(&full_bar[0]), 0);
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const uint32_t j = (uint32_t)(kb0 + i) & 3u;
      const bool fresh = F8 && !FUSE && (j == 0 || i == 0);
      if (fresh) {
        slot = group & (kSpSfSlots - 1);
        if (!warp_wait(smem_u32(&sff_bar[slot]), (group / kSpSfSlots) & 1u, abort, g.status, g.wait_ns)) break;
        ++group;
        sf = tmem + p.NT + slot * kSpSfCols;
      }
      if (!__all_sync(0xFFFFFFFFu, ready) && !warp_wait(smem_u32(&full_bar[st]), ph, abort, g.status, g.wait_ns)) break;
      tc_fence_after();
      const uint32_t wa = sbase + st * stage_bytes, ra = wa + kSpW;
      const uint64_t wd = BMN ? sdesc_mn_sw128(wa) : sdesc_k_sw128(wa);
      const uint64_t rd = sdesc_k_sw128(ra);
      if (FUSE) sf = tmem + p.NT + (uint32_t)(i % kSpFusedSlots) * kSpSfCols;
      if (one) {
        if (FUSE) {  // scales with every K block
          tc_cp_sf_atom(sf, sdesc_sf_atom(ra + p.NT * 128));
          tc_cp_sf_atom(sf + 8, sdesc_sf_atom(ra + p.NT * 128 + 512));
        } else if (fresh) {
          const uint32_t sp = smem_u32(sf_smem) + slot * kSpSfBytes;
          tc_cp_sf_atom(sf, sdesc_sf_atom(sp));
          tc_cp_sf_atom(sf + 8, sdesc_sf_atom(sp + 512));
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t add = (i | k) != 0 ? 1u : 0u;
          if constexpr (F8)
            tc_mma_mxf8(tmem, wd + 2 * k, rd + 2 * k, FUSE ? idesc0 : idesc0 | (j << 4) | (j << 29), sf, sf + 8, add);
          else
            tc_mma_16(tmem, wd + (BMN ? 128 : 2) * k, rd + 2 * k, idesc0, add);
        }
      }
      const uint32_t done = smem_u32(&empty_bar[st]);
      if (++st == p.stages) {
        st = 0;
        ph ^= 1u;
      }
      ready = mbar_test_wait(smem_u32(&full_bar[st]), ph);
      if (one) {
        tc_commit(done);
        if (F8 && !FUSE && (j == 3 || i == n - 1)) tc_commit(smem_u32(&sfe_bar[slot]));
      }
    }
    if (one) tc_commit(smem_u32(&accf_bar));
    __syncwarp();
  } else if (F8 && !FUSE && warp == 2) {
    // ------------------------------------------------------------ scales
    // Lane l holds the words of rows l, l + 32, l + 64, l + 96 of an atom; a weight tile
    // is one block of the matrix, all its rows have the same word.
    struct Words {
      uint32_t w[4], b;
    } even;
    const int q1 = (kb1 + 3) >> 2;
    int q = kb0 >> 2;
    auto load = [&](Words& x) {
      if (q >= q1) return;
      scale_words(g.sa, m0 + lane, g.M, g.sa_pitch, KB, q, x.w);
      x.b = block_word(g.sb, jt, g.sb_pitch, q++);
    };
    uint32_t group = 0;
    const uint32_t groups = q1 - q;
    auto emit = [&](const Words& x) {
      const uint32_t slot = group & (kSpSfSlots - 1);
      if (group == groups || !warp_wait(smem_u32(&sfe_bar[slot]), ((group / kSpSfSlots) & 1u) ^ 1u, abort, g.status, g.wait_ns))
        return false;
      uint8_t* sp = sf_smem + slot * kSpSfBytes + lane * 16;
      *reinterpret_cast<uint4*>(sp) = make_uint4(x.b, x.b, x.b, x.b);
      *reinterpret_cast<uint4*>(sp + 512) = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sff_bar[slot]));
      ++group;
      return true;
    };
    load(even);
    while (emit(even)) load(even);
    __syncwarp();
  } else if (warp >= 4) {
    // ------------------------------------------------------------ sums to shared memory
    // sums[token][row], over the ring: all its copies have been multiplied.
    const int q = warp & 3;
    const bool ok = warp_wait(smem_u32(&accf_bar), 0, abort, g.status, g.wait_ns);
    if (ok && !*abort) {
      tc_fence_after();
      float* sums = reinterpret_cast<float*>(smem) + q * 32 + lane;
      const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
      int c = 0;
      for (; c + 16 < tokens; c += 32) {
        uint32_t r[2][16];
        tmem_ld16(lanes + c, r[0]);
        tmem_ld16(lanes + c + 16, r[1]);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 32; ++k)
          sums[(c + k) * 128] = __uint_as_float(r[k / 16][k % 16]);
      }
      if (c < tokens) {
        uint32_t r[16];
        tmem_ld16(lanes + c, r);
        tmem_ld_wait();
#pragma unroll
        for (int k = 0; k < 16; ++k) sums[(c + k) * 128] = __uint_as_float(r[k]);
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  if (p.split > 1)
    cluster_sync_all();
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, p.tmem_cols);
  }

  // -------------------------------------------------------------- finish tokens
  // This CTA's tokens are rank, rank + split, ...: `mine` of them, in turn the warps'.  A warp
  // takes up to four at a time, whose loads overlap.
  const int mine = (tokens - rank + p.split - 1) / p.split;
  const int col = EPI == kEpiGate ? jt * 64 + 2 * lane : jt * 128 + 4 * lane;
  auto finish = [&](int i0, auto together) {
    constexpr int kN = decltype(together)::value;
    // a token's sums: columns 4 lane .. 4 lane + 3, or (kEpiGate) gate and up of h columns
    // 2 lane, 2 lane + 1
    uint32_t at[kN];
#pragma unroll
    for (int j = 0; j < kN; ++j)
      at[j] = sbase + (uint32_t)(rank + p.split * (i0 + kSpWarps * j)) * 512u + lane * (EPI == kEpiGate ? 8u : 16u);
    float v[kN][4] = {};
#pragma unroll(kN == 1 ? 4 : 2)
    for (int c = 0; c < p.split; ++c)
#pragma unroll
      for (int j = 0; j < kN; ++j) {
        const uint32_t a = mapa_shared(at[j], c);
        float4 x;
        if constexpr (EPI == kEpiGate) {
          const float2 gx = ld_cluster_v2(a), ux = ld_cluster_v2(a + 256);
          x = make_float4(gx.x, gx.y, ux.x, ux.y);
        } else {
          x = ld_cluster_v4(a);
        }
        v[j][0] += x.x, v[j][1] += x.y, v[j][2] += x.z, v[j][3] += x.w;
      }
    if (col >= g.N) return;
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int64_t m = m0 + rank + p.split * (i0 + kSpWarps * j);
      const int64_t o = m * g.ld_out + col;
      [[maybe_unused]] const int64_t s = m * 2 * g.N + col;
      if constexpr (EPI == kEpiGate) {
        const float gv[2] = {v[j][0], v[j][1]};
        float uv[2] = {v[j][2], v[j][3]};
        if (g.saved) {
          store_few(g.saved, s, col, g.N, gv, g.saved_f32, g.type, true);
          store_few(g.saved, s + g.N, col, g.N, uv, g.saved_f32, g.type, true);
        }
        gate_values(g.act, gv, uv);
        store_few(g.out, o, col, g.N, uv, false, g.type, true);
      } else if constexpr (EPI == kEpiStore) {
        store_few(g.out, o, col, g.N, v[j], F8 && g.out_f32, g.type, !F8 || g.vec);
      } else {
        const float4 gs = load_four(g.saved, s, g.saved_f32, g.type);
        const float4 us = load_four(g.saved, s + g.N, g.saved_f32, g.type);
        float gv[4] = {gs.x, gs.y, gs.z, gs.w}, uv[4] = {us.x, us.y, us.z, us.w};
        gradient_values(g.act, v[j], gv, uv);
        store_few(g.dgu, s, col, g.N, gv, false, g.type, true);
        store_few(g.dgu, s + g.N, col, g.N, uv, false, g.type, true);
        if (g.out) store_few(g.out, o, col, g.N, v[j], false, g.type, true);
      }
    }
  };
  for (int i = warp; i < mine;) {
    const int left = (mine - i + kSpWarps - 1) / kSpWarps;  // tokens of this warp
    if (left >= 4) {
      finish(i, std::integral_constant<int, 4>{});
      i += 4 * kSpWarps;
    } else if (left >= 2) {
      finish(i, std::integral_constant<int, 2>{});
      i += 2 * kSpWarps;
    } else {
      finish(i, std::integral_constant<int, 1>{});
      i += kSpWarps;
    }
  }
  if (p.split > 1) cluster_sync_all();  // the others have read this CTA's sums
}

template <bool F8, DenseEpi EPI, bool FUSE = false>
static cudaError_t launch_split(const CUtensorMap& a, const CUtensorMap& b, const DenseArgs& g, const DenseSplit& p,
                                cudaStream_t s) {
  cudaLaunchAttribute c;
  c.id = cudaLaunchAttributeClusterDimension;
  c.val.clusterDim.x = p.split;
  c.val.clusterDim.y = 1;
  c.val.clusterDim.z = 1;
  return launch_k(dense_split_kernel<F8, EPI, FUSE>, dim3((unsigned)(p.split * p.tt * p.rt)), dim3(kSpThreads),
                  p.smem, s, true, &c, a, b, g, p);
}

cudaError_t dense_split_set_attributes() {
  const void* ks[5] = {(const void*)dense_split_kernel<true, kEpiStore, true>,
                       (const void*)dense_split_kernel<true, kEpiStore, false>,
                       (const void*)dense_split_kernel<false, kEpiStore, false>,
                       (const void*)dense_split_kernel<false, kEpiGate, false>,
                       (const void*)dense_split_kernel<false, kEpiGrad, false>};
  for (const void* k : ks) {
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSpAloneSmem);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

// How a product is divided: tokens in equal tiles of at most 64 or 128, two CTAs per SM, K
// in 1, 2, 4 or 8 shares (others did not do better: clusters of them fill the GPU's parts
// unevenly).  By microseconds as measured (E4M3, 4096 x 7168, 32 tiles of 128 rows; K split by
// 1 / 2 / 4 / 8): 1 token 15.7 / 9.7 / 6.7 / 6.7, 64 tokens 16.4 / 10.5 / 7.9 / 9.2, 128
// tokens 19.6 / 12.8 / 10.7 / 13.7.  A K block of 128 bytes takes 0.25 us, 0.32 with 128
// tokens; start, drain and finish 2.8 us and 18 ns a token; the join through other CTAs'
// shared memory 5 or 9 ns a token for 4 or 8 shares; where SMs have two CTAs each of
// these takes longer, and so do joining and finishing gate and up.  Over 90 sizes
// (pair_columns) the choice by these figures and the pair's takes 0.3% longer than the best one,
// over 70 gated blocks 1.2%.
DenseSplit dense_split_plan(const DenseGemm& g, int sms) {
  DenseSplit best = {};
  const bool f8 = g.type == kE4M3;
  const int KB = (g.K + (f8 ? 127 : 63)) / (f8 ? 128 : 64);
  const double bytes = ((double)g.N * (g.epi == kEpiGate ? 2 : 1) + g.M) * g.K * (f8 ? 1e-6 : 2e-6);
  for (int most = 64; most <= kSpMaxTokens; most *= 2) {
    if (most > 64 && g.M <= most / 2) break;
    DenseSplit p = {};
    p.tt = (g.M + most - 1) / most;
    p.NT = ((g.M + p.tt - 1) / p.tt + 15) / 16 * 16;
    p.tt = (g.M + p.NT - 1) / p.NT;
    p.rt = g.epi == kEpiGate ? (g.N + 63) / 64 : (g.N + 127) / 128;
    const int64_t tiles = (int64_t)p.tt * p.rt;
    for (int split = 1; split <= 8 && split <= KB; split *= 2) {
      const int64_t ctas = tiles * split;
      const bool shared = ctas > sms;
      const double waves = (double)((ctas + 2 * sms - 1) / (2 * sms));
      double block = 0.24 + 0.0006 * p.NT, join = p.NT * (split == 8 ? 0.009 : split == 4 ? 0.0055 : 0.0);
      double us = 2.8 + 0.018 * p.NT;
      if (shared) block *= 1.11 + 0.0016 * p.NT, join *= 1.9, us += 0.023 * p.NT;
      if (g.epi == kEpiGate) us += (shared ? 0.03 : 0.02) * p.NT, join += split > 1 ? 1.0 : 0.0;
      us *= 0.5 + 0.5 * waves;  // (one's end overlaps another's start)
      // (fewer CTAs have less in flight than the memory needs)
      const double rate = ctas < 144 ? 0.045 * ctas : 6.5, stream_us = bytes / rate;
      const double stream = block * ((KB + split - 1) / split) * waves;
      us += join + (stream > stream_us ? stream : stream_us);
      if (best.split && us >= best.us) continue;
      best = p;
      best.split = split;
      best.us = us;
      best.alone = !shared;
    }
  }
  const int cols = best.NT + (g.x ? kSpFusedSlots : f8 ? kSpSfSlots : 0) * (int)kSpSfCols;
  best.tmem_cols = cols <= 32 ? 32 : cols <= 64 ? 64 : cols <= 128 ? 128 : 256;
  // two CTAs per SM (above 76 KB each and with at most 256 columns, so never three, and
  // two always find their tensor memory)
  const uint32_t stage = kSpW + best.NT * 128 + (g.x ? kSpSfBytes : 0u), fixed = kSpSfSlots * kSpSfBytes + 1024;
  best.stages = (int)((kSpMaxSmem - fixed) / stage);
  if (best.stages > (g.x ? kSpFusedSlots - 1 : kSpMaxStages)) best.stages = g.x ? kSpFusedSlots - 1 : kSpMaxStages;
  best.smem = best.stages * stage + fixed;
  // After the quantising kernel, whose CTAs leave some SMs emptier than others, at most one CTA
  // per SM are kept one: with more than half of the shared memory (200 tokens, 2048 x 7168: 15.1
  // -> 12.9 us; where a call's kernels follow others like them it only delays their start).
  if (best.alone && f8 && g.early) best.smem = kSpAloneSmem;
  return best;
}

cudaError_t dense_split_launch(const CUtensorMap& a, const CUtensorMap& b, const DenseGemm& g, const DenseArgs& d,
                               const DenseSplit& p, cudaStream_t s) {
  if (g.x) return launch_split<true, kEpiStore, true>(b, b, d, p, s);
  if (g.type == kE4M3) return launch_split<true, kEpiStore>(a, b, d, p, s);
  if (g.epi == kEpiGate) return launch_split<false, kEpiGate>(a, b, d, p, s);
  if (g.epi == kEpiGrad) return launch_split<false, kEpiGrad>(a, b, d, p, s);
  return launch_split<false, kEpiStore>(a, b, d, p, s);
}

}  // namespace mm
