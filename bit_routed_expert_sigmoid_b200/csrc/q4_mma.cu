// Linear products with 4-bit weights for more than 8 tokens (flint_q4_linear) on tcgen05.
//
// The weights are the M side of the MMA, decoded straight into tensor memory: a tile is up to 128 rows of W, and a
// cluster of CTAs splits a tile's K, so that tiles of equal height and K ranges fill the SMs whatever N is (8192 rows: 74
// tiles of 111 rows, two CTAs each). Two teams of four warps take 128-segments in turn (8192 x 8192 at T = 16: one team
// 23.5 us, two 21.6, four 24.0), a thread decoding one row's 128 codes to exact fp16; two warps issue the MMAs of a segment
// in turn (an instruction takes ~45 cycles to issue), each into an accumulator of the segment's own; eight warps add the
// accumulators, times the rows' group scales and the tokens' factors, to fp32 sums in registers, so that neither is rounded
// to fp16. At the end the CTAs of a cluster exchange their sums through distributed shared memory and add them in rank order.
// Codes come by TMA, 512 K of all rows per stage, the operand too, a pair of segments per stage (kF16Pair: the two parts of
// one), with its factors; rows of codes that are no multiple of 16 bytes (K % 32 = 16) are read by the decoding warps.
//
// 8192 x 8192 takes 20.3 us at T = 16 and 24.6 at T = 64, 5001 x 4112 NVFP4 15.6 at T = 37: calls in a CUDA graph, weights in
// L2, as all times in this file; with L2 flushed and the launch included 26.3, 32.0 and 35 (once through HBM 5.4, 5.6, 1.9).
// More than 64 tokens run in chunks that fetch and decode W again: 256 tokens 90 us, 2048 tokens 691 (tensor cores 20, 164).
// What bounds it is the chain of a segment, 0.4 us a team: codes to registers, decoding, the store to tensor memory, eight
// MMAs, the sums. 54 % of the issue slots are used; the warps wait for one another's results, and more stages, more teams or
// codes released before they are decoded only made them wait longer. (With the tokens on the M side every MMA reads 128
// operand rows from shared memory, 32 KB per segment whatever T is: that took 46 us for 8192 x 8192.)
#include <limits.h>

#include "kernels.cuh"
#include "ops.cuh"
#include "q4_operand.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace flint {

__device__ unsigned g_ops_error_q4mma;           // timeout bits of bounded waits (flint_ops_error_word)

namespace {

constexpr int kMmTeams = 2;                      // decoding teams of four warps
constexpr int kMmSums = 4 + 4 * kMmTeams;        // first of the 8 summing warps; before: copies 2, MMA 2, decoding
constexpr int kMmThreads = 32 * (kMmSums + 8);
constexpr int kMmTokens = 64;                    // tokens at a time at most
constexpr int kMmChunk = 4;                      // segments of codes per stage
constexpr int kMmA = 4;                          // decoded segments in tensor memory (64 columns each)
constexpr int kMmD = 4;                          // accumulators (64 columns each)
// Segments of factors kept for the sums: the MMA is at most kMmD segments ahead of them, copies at most kMmPairStages pairs
// ahead of the MMA.
constexpr int kMmRing = 16;
// Stages of codes (one where large tiles leave no room for two; up to four: 21.6 us against 21.1 for 8192 x 8192 at
// T = 16) and of the operand.
constexpr int kMmCodeStages = 2, kMmPairStages = 3;
constexpr int kMmMaxSplit = 8;                   // CTAs per tile (portable cluster size)
constexpr int kMmScaleBytes = 32 * 1024;

struct MmParams {
  CUtensorMap tm_codes;                          // boxed: [K / 256][N][128 bytes], else [N][K / 2 bytes]
  CUtensorMap tm_x;                              // operand [segs * parts * 2][T][64] fp16, boxes of 4 x TB x 64
  CUtensorMap tm_scales;                         // [N][scale bytes per row], boxes of scale_row x R
  Q4Params q;
  int R;                                         // rows of a tile
  int split, range;                              // CTAs per tile, segments of each
  int TB;                                        // tokens at a time, a multiple of 8
  int SC;                                        // stages of codes
  int boxed;
  int scale_row;                                 // bytes of a row's scales kept in shared memory, 0: none
};

struct MmBars {
  uint64_t c_full[kMmCodeStages], c_empty[kMmCodeStages], b_full[kMmPairStages], b_empty[kMmPairStages];
  uint64_t a_full[kMmA], a_empty[kMmA], d_full[kMmD], d_empty[kMmD], done[2], scales;
  uint32_t tmem;
  int abort;
};

__host__ __device__ inline int mm_code_stage(int R) { return (kMmChunk / 2 * R * 128 + 1023) & ~1023; }

// (a0, a1) += (d0, d1) s (f0, f1) in packed fp32 pairs, each step rounded once
__device__ __forceinline__ void add_scaled(float& a0, float& a1, uint32_t d0, uint32_t d1, float s, float f0, float f1) {
  uint64_t a, d, ss, ff;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(d0), "r"(d1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(ss) : "f"(s));
  asm("mov.b64 %0, {%1, %2};" : "=l"(ff) : "f"(f0), "f"(f1));
  asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(ff) : "l"(ss));
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(d), "l"(ff));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
}

// 16 consecutive columns of the warp's 32 lanes
__device__ __forceinline__ void tc_st16(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

template <int AR, int TYPE, bool TMA>
__global__ void __launch_bounds__(kMmThreads, 1) q4_mma_kernel(const __grid_constant__ MmParams mp) {
  const Q4Params& p = mp.q;
  constexpr bool kI4 = AR != kF16Nvfp4;
  constexpr int kSegs = 2 / kParts<AR>;          // segments of a stage of the operand: four 64-K blocks in all
  extern __shared__ uint8_t smem_raw[];
  __shared__ MmBars bb;
  __shared__ __align__(16) float s_factor[kMmRing][kMmTokens];   // of the tokens, per segment
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int all_segs = (p.K + 127) / 128;
  const int rank = blockIdx.x % mp.split, tile = blockIdx.x / mp.split;
  const int seg0 = rank * mp.range, segs = max(min(mp.range, all_segs - seg0), 0);     // this CTA's segments
  const int pairs = (segs + kSegs - 1) / kSegs, chunks = (segs + kMmChunk - 1) / kMmChunk;
  const int R = mp.R, TB = mp.TB, row0 = tile * R, rows = min(R, p.N - row0);
  const int b_stage = TB * 512, c_stage = TMA ? mm_code_stage(R) : 0;
  const int t0 = blockIdx.y * TB, N16 = (TB + 15) & ~15;
  uint8_t* sm_b = align1024(smem_raw);
  uint8_t* sm_c = sm_b + kMmPairStages * b_stage;
  uint8_t* sm_s = sm_c + mp.SC * c_stage;
  volatile int* abort = &bb.abort;
  unsigned* err = &g_ops_error_q4mma;
  const long long scale_row = kI4 ? p.K >> 6 : p.K >> 4;         // bytes

  if (threadIdx.x == 0) {
    for (int i = 0; i < kMmCodeStages; ++i) {
      mbar_init(&bb.c_full[i], 1);
      mbar_init(&bb.c_empty[i], 4 * kMmTeams);
    }
    for (int i = 0; i < kMmPairStages; ++i) {
      mbar_init(&bb.b_full[i], 1);
      mbar_init(&bb.b_empty[i], 2);
    }
    for (int i = 0; i < kMmA; ++i) {
      mbar_init(&bb.a_full[i], 4);
      mbar_init(&bb.a_empty[i], 1);
    }
    for (int i = 0; i < kMmD; ++i) {
      mbar_init(&bb.d_full[i], 1);
      mbar_init(&bb.d_empty[i], 8);
    }
    mbar_init(&bb.done[0], 1);
    mbar_init(&bb.done[1], 1);
    mbar_init(&bb.scales, 1);
    bb.abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bb.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bb.tmem, tmem_a = tmem + kMmD * 64;
  pdl_trigger();
  const int half = (warp - kMmSums) >> 2;             // sums: which 16 of every 32 tokens
  float acc[kMmTokens / 2];                      // sums: tokens 16 (2 b + half) + j at 16 b + j
#pragma unroll
  for (int j = 0; j < kMmTokens / 2; ++j) acc[j] = 0.f;

  if (warp == 0) {
    // ---- codes and scales: no predecessor's output, copied before griddepcontrol.wait
    if (lane == 0) {
      const uint64_t pol = l2_evict_first();
      if (mp.scale_row) {
        mbar_arrive_expect_tx(&bb.scales, R * mp.scale_row);
        tma_2d_hint(sm_s, &mp.tm_scales, seg0 * (kI4 ? 2 : 8) / 4, row0, &bb.scales, pol);
      }
      int it = 0;
      if constexpr (TMA) {
        for (; it < chunks; ++it) {
          const int slot = it % mp.SC;
          if (it >= mp.SC && !pf_wait(&bb.c_empty[slot], ((it / mp.SC) - 1) & 1, abort, err)) break;
          uint8_t* st = sm_c + slot * c_stage;
          mbar_arrive_expect_tx(&bb.c_full[slot], kMmChunk / 2 * R * 128);
          const int kb = seg0 / 2 + it * (kMmChunk / 2);         // 256-code block
          if (mp.boxed) {
            tma_3d_hint(st, &mp.tm_codes, 0, row0, kb, &bb.c_full[slot], pol);
          } else {
            for (int b = 0; b < kMmChunk / 2; ++b)
              tma_2d_hint(st + b * R * 128, &mp.tm_codes, (kb + b) * 32, row0, &bb.c_full[slot], pol);
          }
        }
        for (int j = max(it - mp.SC, 0); j < it; ++j) mbar_wait_bounded(&bb.c_full[j % mp.SC], (j / mp.SC) & 1, 1000000);
      }
      if (mp.scale_row) mbar_wait_bounded(&bb.scales, 0, 1000000);
    }
  } else if (warp == 1) {
    // ---- operand: a stage's four 64-K blocks (blocks behind K read as zeros), and the segments' factors
    if (lane == 0) {
      pdl_wait();
      const int tpad = (p.T + 3) & ~3, fbytes = min(TB, tpad - t0) * 4;
      const uint8_t* img = static_cast<const uint8_t*>(p.workspace);
      const float* fac = reinterpret_cast<const float*>(img + q4_rows_factors(p.T, all_segs, kParts<AR>)) + t0;
      int it = 0;
      for (; it < pairs; ++it) {
        const int slot = it % kMmPairStages, seg = kSegs * it, n = min(kSegs, segs - seg);
        if (it >= kMmPairStages && !pf_wait(&bb.b_empty[slot], ((it / kMmPairStages) - 1) & 1, abort, err)) break;
        mbar_arrive_expect_tx(&bb.b_full[slot], b_stage + n * fbytes);
        tma_3d(sm_b + slot * b_stage, &mp.tm_x, 0, t0, 4 / kSegs * (seg0 + seg), &bb.b_full[slot]);
        for (int j = 0; j < n; ++j)
          bulk_g2s(s_factor[(seg + j) % kMmRing], fac + static_cast<size_t>(seg0 + seg + j) * tpad, fbytes, &bb.b_full[slot]);
      }
      for (int j = max(it - kMmPairStages, 0); j < it; ++j)
        mbar_wait_bounded(&bb.b_full[j % kMmPairStages], (j / kMmPairStages) & 1, 1000000);
    }
  } else if (warp < 4) {
    // ---- MMA: segments of one parity. kMmA and kMmD are even, so that a place of either belongs to one warp; both
    // warps go through all stages of the operand.
    const int w = warp - 2;
    const uint32_t idesc = idesc_m128(N16, false);
    for (int it = 0; it < pairs; ++it) {
      const int seg = kSegs == 2 ? 2 * it + w : it, sb = it % kMmPairStages, sa = seg % kMmA, sd = seg % kMmD;
      if (!pf_wait_all(&bb.b_full[sb], (it / kMmPairStages) & 1, abort, err)) break;
      if (seg < segs && (seg & 1) == w) {
        if (seg >= kMmD && !pf_wait_all(&bb.d_empty[sd], ((seg / kMmD) - 1) & 1, abort, err)) break;
        if (!pf_wait_all(&bb.a_full[sa], (seg / kMmA) & 1, abort, err)) break;
        tc_fence_after();
        const uint32_t b0 = smem_u32(sm_b + sb * b_stage) + (kSegs == 2 ? w * TB * 256 : 0);
#pragma unroll
        for (int ks = 0; ks < 8 * kParts<AR>; ++ks)
          tc_mma_ta_w(tmem + sd * 64, tmem_a + sa * 64 + (ks & 7) * 8, sdesc_sw128(b0 + (ks >> 2) * TB * 128 + (ks & 3) * 32),
                      idesc, ks ? 1u : 0u);
        tc_commit_w(&bb.a_empty[sa]);
        tc_commit_w(&bb.d_full[sd]);
      }
      tc_commit_w(&bb.b_empty[sb]);
    }
    tc_commit_w(&bb.done[w]);
    pf_wait_all(&bb.done[w], 0, abort, err);
  } else if (warp < kMmSums) {
    // ---- decoding: a thread per row, 128 codes of every kMmTeams-th segment
    const int team = (warp - 4) >> 2, row = 32 * (warp & 3) + lane;
    const int n = min(row0 + min(row, R - 1), p.N - 1);
    const uint32_t lane_base = tmem_a + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    bool ok = kI4 || !mp.scale_row || pf_wait_all(&bb.scales, 0, abort, err);
    for (int c = 0; c < chunks && ok; ++c) {
      const int sc = c % mp.SC;
      if (TMA && !(ok = pf_wait_all(&bb.c_full[sc], (c / mp.SC) & 1, abort, err))) break;
      for (int j = team; j < kMmChunk; j += kMmTeams) {
        const int seg = c * kMmChunk + j, sa = seg % kMmA;
        if (seg >= segs) break;
        uint2 scale = make_uint2(0, 0);          // NVFP4: the eight block scales
        if constexpr (!kI4) {
          const int k = (seg0 + seg) * 128;
          if (mp.scale_row) {
            scale = *reinterpret_cast<const uint2*>(sm_s + min(row, R - 1) * mp.scale_row + 8 * seg);
          } else {
            uint32_t b[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              b[i] = k + 16 * i < p.K ? __ldg(p.scales + n * scale_row + (k >> 4) + i) : 0u;
            scale.x = b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24);
            scale.y = b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24);
          }
        }
        uint4 code[4];
        if constexpr (TMA) {
          const int at = (j >> 1) * R + min(row, R - 1);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            code[i] = *reinterpret_cast<const uint4*>(sm_c + sc * c_stage + at * 128 + (((4 * (j & 1) + i) ^ (at & 7)) << 4));
        } else {
          const uint8_t* src = p.codes + static_cast<size_t>(n) * (p.K >> 1) + (seg0 + seg) * 64;
          uint2 v[8];
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = (seg0 + seg) * 128 + 16 * i < p.K ? __ldg(reinterpret_cast<const uint2*>(src) + i) : make_uint2(0, 0);
#pragma unroll
          for (int i = 0; i < 4; ++i) code[i] = make_uint4(v[2 * i].x, v[2 * i].y, v[2 * i + 1].x, v[2 * i + 1].y);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {            // 32 codes: 16 columns
          uint32_t v[16];
          const uint32_t s2 = i < 2 ? scale.x : scale.y;
          decode_f16<kI4 ? kF16Int4 : kF16Nvfp4>(code[i], i & 1 ? s2 >> 16 : s2 & 0xFFFFu, v);
          if (i == 0) {
            if (seg >= kMmA && !(ok = pf_wait_all(&bb.a_empty[sa], ((seg / kMmA) - 1) & 1, abort, err))) break;
            tc_fence_after();
          }
          tc_st16(lane_base + sa * 64 + i * 16, v);
        }
        if (!ok) break;
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bb.a_full[sa]);
      }
      if (TMA && ok && lane == 0) mbar_arrive(&bb.c_empty[sc]);
    }
  } else {
    // ---- sums: a thread per row of W; the two sets of four warps take 16 tokens in turn
    const int row = 32 * (warp & 3) + lane;
    const uint32_t base = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const int n = min(row0 + min(row, R - 1), p.N - 1);
    const uint16_t* gs = reinterpret_cast<const uint16_t*>(p.scales + (kI4 ? n * scale_row : 0)) + seg0;
    const uint16_t* ss = reinterpret_cast<const uint16_t*>(sm_s + min(row, R - 1) * mp.scale_row);
    const float ts = p.tscale ? __ldg(p.tscale) : 1.f;
    bool ok = !kI4 || !mp.scale_row || pf_wait_all(&bb.scales, 0, abort, err);
    uint32_t next = kI4 && !mp.scale_row && segs > 0 ? __ldg(gs) : 0u;
    for (int seg = 0; seg < segs && ok; ++seg) {
      const int sd = seg % kMmD;
      float sc = 1.f;
      if constexpr (kI4) {
        const uint32_t now = next;
        if (!mp.scale_row && seg + 1 < segs) next = __ldg(gs + seg + 1);
        sc = bf16_bits_to_f32(static_cast<uint16_t>(mp.scale_row ? ss[seg] : now));
      }
      if (!(ok = pf_wait_all(&bb.d_full[sd], (seg / kMmD) & 1, abort, err))) break;
      tc_fence_after();
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int c0 = 16 * (2 * b + half);
        if (c0 < N16) {
          uint32_t d[16];
          tc_ld16(base + sd * 64 + c0, d);
          tc_wait_ld();
          const float* f = &s_factor[seg % kMmRing][c0];
#pragma unroll
          for (int i = 0; i < 16; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(f + i);
            add_scaled(acc[16 * b + i], acc[16 * b + i + 1], d[i], d[i + 1], sc, v.x, v.y);
            add_scaled(acc[16 * b + i + 2], acc[16 * b + i + 3], d[i + 2], d[i + 3], sc, v.z, v.w);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bb.d_empty[sd]);
    }
#pragma unroll
    for (int j = 0; j < kMmTokens / 2; ++j) acc[j] *= ts;
  }

  // ---- the CTAs of a tile add their sums: CTA r finishes the tokens of its share
  const bool summing = warp >= kMmSums;
  const int row = 32 * (warp & 3) + lane;
  if (mp.split == 1) {
    if (summing && row < rows) {
#pragma unroll
      for (int j = 0; j < kMmTokens / 2; ++j) {
        const int t = 16 * (2 * (j >> 4) + half) + (j & 15);
        if (t < TB && t0 + t < p.T) p.y[static_cast<long long>(t0 + t) * p.ldy + row0 + row] = from_f32<TYPE>(acc[j]);
      }
    }
  } else {
    const int share = (TB + mp.split - 1) / mp.split;
    float* part = reinterpret_cast<float*>(sm_b);                // [split][share][128]
    __syncwarp();
    cluster_sync();                              // every CTA is done with its rings
    if (summing) {
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        int t = 16 * (2 * b + half), to = t / share, at = t - to * share;
#pragma unroll
        for (int j = 0; j < 16; ++j, ++t) {
          if (t < TB) st_cluster_f32(part + (rank * share + at) * 128 + row, to, acc[16 * b + j]);
          if (++at == share) at = 0, ++to;
        }
      }
    }
    __syncwarp();
    cluster_sync();
    // a warp per token, four rows per lane
    for (int i = warp; i < share; i += kMmThreads / 32) {
      const int t = rank * share + i;
      if (t >= TB || t0 + t >= p.T) break;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k = 0; k < mp.split; ++k) {
        const float4 u = *reinterpret_cast<const float4*>(part + (k * share + i) * 128 + 4 * lane);
        v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
      }
      uint16_t* y = p.y + static_cast<long long>(t0 + t) * p.ldy + row0 + 4 * lane;
      const int left = rows - 4 * lane;
      if (left > 0) y[0] = from_f32<TYPE>(v.x);
      if (left > 1) y[1] = from_f32<TYPE>(v.y);
      if (left > 2) y[2] = from_f32<TYPE>(v.z);
      if (left > 3) y[3] = from_f32<TYPE>(v.w);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

constexpr int kAlone = 115 * 1024;               // more than half of an SM's 228 KB
constexpr int kMost = 226 * 1024 - static_cast<int>(sizeof(MmBars)) - kMmRing * 4 * kMmTokens - 256;

// Clusters of k CTAs that the device runs at once: fewer than SMs / k, as a cluster stays within a group of SMs.
int clusters_of(int dev, int sms, int k) {
  static std::atomic<int> known[kMaxDev][kMmMaxSplit + 1];
  int n = known[dev][k].load(std::memory_order_relaxed);
  if (n) return n;
  auto kernel = q4_mma_kernel<kF16Int4, kTBf16, true>;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(k);
  cfg.blockDim = dim3(kMmThreads);
  cfg.dynamicSmemBytes = kMost;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = k;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (k == 1) n = sms;
  else if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) != cudaSuccess ||
           cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
    (void)cudaGetLastError();
    n = -1;                                      // never taken
  }
  known[dev][k].store(n, std::memory_order_relaxed);
  return n;
}

template <int AR, int TYPE, bool TMA>
cudaError_t launch_mm(const Q4Params& p, cudaStream_t s) {
  constexpr bool kI4 = AR != kF16Nvfp4;
  int dev, sms;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  const int segs = (p.K + 127) / 128;
  MmParams mp;
  mp.q = p;
  // Tiles and splits: a CTA takes 0.4 us per segment (NVFP4 0.6), whatever the height of its tile. Of the splits for which
  // the tiles (as many as the SMs then hold, of at most 128 rows) make one wave, the one with the fewest segments per CTA
  // (2048 x 2048, T = 9: 12.6, 10.0, 9.2 and 8.5 us split 1, 2, 3 and 4 ways); more rows than one wave holds go unsplit.
  mp.split = 1;
  mp.R = 128;
  mp.range = INT_MAX;
  for (int k = 1; k <= kMmMaxSplit && k <= segs; ++k) {
    const int tiles = clusters_of(dev, sms, k), R = tiles > 0 ? (p.N + tiles - 1) / tiles : 129;
    if (R > 128) continue;
    int range = (segs + k - 1) / k;
    if (TMA) range = (range + 1) & ~1;           // it starts with a 256-code block
    if (range < mp.range) {
      mp.range = range;
      mp.split = k;
      mp.R = R < 8 ? 8 : R;
    }
  }
  if (mp.range > segs) mp.range = TMA ? (segs + 1) & ~1 : segs;
  const int tiles = (p.N + mp.R - 1) / mp.R;
  const int token_chunks = (p.T + kMmTokens - 1) / kMmTokens;
  mp.TB = ((p.T + token_chunks - 1) / token_chunks + 7) & ~7;
  mp.boxed = p.K % 256 == 0;
  const long long scale_row = kI4 ? p.K >> 6 : p.K >> 4;
  const int own = mp.range * (kI4 ? 2 : 8);
  mp.scale_row = scale_row % 16 == 0 && own % 16 == 0 && own <= 1024 && mp.R * own <= kMmScaleBytes &&
                         (reinterpret_cast<uintptr_t>(p.scales) & 15u) == 0
                     ? own
                     : 0;
  const int b_stage = mp.TB * 512, c_stage = TMA ? mm_code_stage(mp.R) : 0;
  const int fixed = 1024 + mp.R * mp.scale_row;
  mp.SC = TMA ? (kMost - fixed - kMmPairStages * b_stage) / c_stage : 1;
  if (mp.SC > kMmCodeStages) mp.SC = kMmCodeStages;
  if (mp.SC < 1) return cudaErrorInvalidConfiguration;
  int smem = fixed + kMmPairStages * b_stage + mp.SC * c_stage;
  const int parts = 1024 + mp.split * ((mp.TB + mp.split - 1) / mp.split) * 512;
  if (smem < parts) smem = parts;
  // the MMA reads N16 rows of the operand's last block, up to 8 more than there are
  if (smem < 1024 + kMmPairStages * b_stage + 1024) smem = 1024 + kMmPairStages * b_stage + 1024;
  // One CTA per SM, whatever its registers: a second one would wait for the first one's tensor memory, and two clusters
  // that share two SMs crosswise would wait for each other.
  if (smem < kAlone) smem = kAlone;
  if (smem > kMost) return cudaErrorInvalidConfiguration;
  if (TMA && !(mp.boxed ? encode_words_blocks(&mp.tm_codes, p.codes, p.N, p.K / 2, mp.R, kMmChunk / 2)
                        : encode_words(&mp.tm_codes, p.codes, p.N, p.K / 2, mp.R)))
    return cudaErrorInvalidValue;
  if (mp.scale_row && !encode_words_rows(&mp.tm_scales, p.scales, p.N, scale_row, mp.scale_row, mp.R))
    return cudaErrorInvalidValue;
  const uint64_t cols = static_cast<uint64_t>(segs) * 128 * kParts<AR>;
  if (!encode_16bit_blocks(&mp.tm_x, p.workspace, false, p.T, cols, cols, mp.TB, 4))
    return cudaErrorInvalidValue;
  if ((e = allow_smem_once<q4_mma_kernel<AR, TYPE, TMA>>(dev, kMost)) != cudaSuccess) return e;
  if ((e = launch_q4_operand<AR, TYPE, kRows>(p, sms, s)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(tiles * mp.split, (p.T + mp.TB - 1) / mp.TB);
  cfg.blockDim = dim3(kMmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = mp.split;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, q4_mma_kernel<AR, TYPE, TMA>, mp);
}

}  // namespace

cudaError_t launch_q4_mma(const Q4Params& p, cudaStream_t s) {
  if (p.fmt == kInt4) {
    if (p.type == kTBf16) return launch_mm<kF16Int4, kTBf16, true>(p, s);
    return p.rotated ? launch_mm<kF16Pair, kTF16, true>(p, s) : launch_mm<kF16Int4, kTF16, true>(p, s);
  }
  if (p.K % 32 == 0)
    return p.type == kTBf16 ? launch_mm<kF16Nvfp4, kTBf16, true>(p, s) : launch_mm<kF16Nvfp4, kTF16, true>(p, s);
  return p.type == kTBf16 ? launch_mm<kF16Nvfp4, kTBf16, false>(p, s) : launch_mm<kF16Nvfp4, kTF16, false>(p, s);
}

cudaError_t read_q4_mma_error(unsigned* out) {
  const unsigned zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_ops_error_q4mma, sizeof(unsigned));
  if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_ops_error_q4mma, &zero, sizeof(unsigned));
  return e;
}

}  // namespace flint
