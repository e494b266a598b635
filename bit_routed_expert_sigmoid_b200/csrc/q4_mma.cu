// Linear products with 4-bit weights for more than 8 tokens (flint_q4_linear) on tcgen05.
//
// The tokens are the M side of the MMA (up to 96 rows of the operand of q4_operand.cuh, the rest of 128 unused) and the
// rows of W its N side, so that W divides evenly over the SMs: a CTA has up to 64 rows per round, whatever N is. Work
// goes in pairs of 128-segments: two teams of four warps decode pairs in turn to exact fp16 in shared memory, two warps
// issue a segment's MMAs each, into an accumulator of the segment's own, and eight warps add the accumulators, times the
// rows' group scales and the tokens' factors, to fp32 sums in registers: scales of any range and tokens of any magnitude
// lose nothing. Every one of these steps has a long latency (tensor memory, the fence between a warp's stores and the
// tensor core's reads, small copies), which is why none takes one segment at a time: that took 56 us for 8192 x 8192 at
// T = 16. Codes come by TMA, 512 K of all rows per stage; the operand too, a pair per stage, with its factors.
#include "kernels.cuh"
#include "ops.cuh"
#include "q4_operand.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace flint {

__device__ unsigned g_ops_error_q4mma;           // timeout bits of bounded waits (flint_ops_error_word)

namespace {

constexpr int kMmThreads = 640;                  // copies: 2 warps, MMA: 2, decoding: 2 x 4, sums: 8
constexpr int kMmRows = 64;                      // rows of W per round at most
constexpr int kMmTokens = 96;                    // tokens at a time at most
constexpr int kMmChunk = 4;                      // segments of codes per stage: a pair for each team
constexpr int kMmGroup = 4;                      // segments per set of accumulators
constexpr int kMmSB = 2;                         // decoded pairs in flight, one of each team
// Segments of scales and factors kept for the sums: the MMA is at most two groups (4 pairs) ahead of them, decoding and
// copies at most 3 pairs ahead of the MMA, which makes the pair 8 back one that the sums are done with.
constexpr int kMmRing = 16;
constexpr int kMmMaxStages = 4;

struct MmParams {
  CUtensorMap tm_codes;                          // boxed: [K / 256][N][128 bytes], else [N][K / 2 bytes]
  CUtensorMap tm_x;                              // operand [segs * 2][T][64] fp16, boxes of 4 x TB x 64
  Q4Params q;
  int R, N16;                                    // rows of W per round; padded to 16
  int rounds;                                    // per CTA
  int TB;                                        // tokens at a time, a multiple of 8
  int SC, SA;                                    // stages of codes and of the operand
  int boxed, scale_bytes;
};

struct MmBars {
  uint64_t c_full[kMmMaxStages], c_empty[kMmMaxStages], a_full[kMmMaxStages], a_empty[kMmMaxStages];
  uint64_t b_full[kMmSB], b_empty[kMmSB], d_full[2], d_empty[2], done[2], scales;
  uint32_t tmem;
  int abort;
};

__host__ __device__ inline int mm_code_stage(int R) { return (kMmChunk / 2 * R * 128 + 1023) & ~1023; }

// (a0, a1) += (d0, d1) f (s0, s1), without the scales when !scaled: packed fp32 pairs, each step rounded once
__device__ __forceinline__ void add_scaled(float& a0, float& a1, uint32_t d0, uint32_t d1, float f, float s0, float s1,
                                           bool scaled) {
  uint64_t a, d, ff, ss;
  asm("mov.b64 %0, {%1, %2};" : "=l"(a) : "f"(a0), "f"(a1));
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(d0), "r"(d1));
  asm("mov.b64 %0, {%1, %1};" : "=l"(ff) : "f"(f));
  if (scaled) {
    asm("mov.b64 %0, {%1, %2};" : "=l"(ss) : "f"(s0), "f"(s1));
    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(d) : "l"(ff));
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(d), "l"(ss));
  } else {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(a) : "l"(d), "l"(ff));
  }
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a0), "=f"(a1) : "l"(a));
}

template <int AR, int TYPE>
__global__ void __launch_bounds__(kMmThreads, 1) q4_mma_kernel(const __grid_constant__ MmParams mp) {
  const Q4Params& p = mp.q;
  constexpr bool kI4 = AR == kF16Int4;
  extern __shared__ uint8_t smem_raw[];
  __shared__ MmBars bb;
  __shared__ __align__(16) float s_scale[kMmRing][kMmRows];      // of the rows, per segment
  __shared__ __align__(16) float s_factor[kMmRing][kMmTokens];   // of the tokens, per segment
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int segs = (p.K + 127) / 128, pairs = (segs + 1) / 2, chunks = (segs + kMmChunk - 1) / kMmChunk;
  const int groups = (segs + kMmGroup - 1) / kMmGroup;
  const int R = mp.R, N16 = mp.N16, TB = mp.TB;
  const int a_stage = TB * 512, b_stage = N16 * 512, c_stage = mm_code_stage(R);
  const int t0 = blockIdx.y * TB, first = blockIdx.x * mp.rounds, total = (p.N + R - 1) / R;
  const int rounds = min(mp.rounds, total - first);
  // operand first: the MMA reads 128 rows from a block's start, past its end into what follows (unused accumulator rows)
  uint8_t* sm_a = align1024(smem_raw);
  uint8_t* sm_b = sm_a + mp.SA * a_stage;
  uint8_t* sm_c = sm_b + kMmSB * b_stage;
  uint8_t* sm_s = sm_c + mp.SC * c_stage;
  volatile int* abort = &bb.abort;
  unsigned* err = &g_ops_error_q4mma;
  const size_t scale_row = kI4 ? p.K >> 6 : p.K >> 4;            // bytes

  if (threadIdx.x == 0) {
    for (int i = 0; i < mp.SC; ++i) {
      mbar_init(&bb.c_full[i], 1);
      mbar_init(&bb.c_empty[i], 8);
    }
    for (int i = 0; i < mp.SA; ++i) {
      mbar_init(&bb.a_full[i], 1);
      mbar_init(&bb.a_empty[i], 2);
    }
    for (int i = 0; i < kMmSB; ++i) {
      mbar_init(&bb.b_full[i], 4);
      mbar_init(&bb.b_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bb.d_full[i], 2);
      mbar_init(&bb.d_empty[i], 8);
      mbar_init(&bb.done[i], 1);
    }
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
  const uint32_t tmem = bb.tmem;

  if (warp == 0) {
    // ---- codes and scales: no predecessor's output, copied before griddepcontrol.wait
    if (lane == 0) {
      const uint64_t pol = l2_evict_first();
      if (mp.scale_bytes) {
        const int n = min(rounds * R, p.N - first * R) * static_cast<int>(scale_row);
        mbar_arrive_expect_tx(&bb.scales, n);
        bulk_g2s_hint(sm_s, p.scales + first * R * scale_row, n, &bb.scales, pol);
      }
      int it = 0;
      const int n = rounds * chunks;
      for (; it < n; ++it) {
        const int slot = it % mp.SC, rd = it / chunks, c = it - rd * chunks, row = (first + rd) * R;
        if (it >= mp.SC && !pf_wait(&bb.c_empty[slot], ((it / mp.SC) - 1) & 1, abort, err)) break;
        uint8_t* st = sm_c + slot * c_stage;
        mbar_arrive_expect_tx(&bb.c_full[slot], kMmChunk / 2 * R * 128);
        if (mp.boxed) {
          tma_3d_hint(st, &mp.tm_codes, 0, row, c * (kMmChunk / 2), &bb.c_full[slot], pol);
        } else {
          for (int b = 0; b < kMmChunk / 2; ++b)
            tma_2d_hint(st + b * R * 128, &mp.tm_codes, (c * (kMmChunk / 2) + b) * 32, row, &bb.c_full[slot], pol);
        }
      }
      for (int j = max(it - mp.SC, 0); j < it; ++j) mbar_wait_bounded(&bb.c_full[j % mp.SC], (j / mp.SC) & 1, 1000000);
      if (mp.scale_bytes) mbar_wait_bounded(&bb.scales, 0, 1000000);
    }
  } else if (warp == 1) {
    // ---- operand: a pair's four 64-K blocks (blocks behind K read as zeros), and the segments' factors
    if (lane == 0) {
      pdl_wait();
      const int tpad = (p.T + 3) & ~3, fbytes = min(TB, tpad - t0) * 4;
      const float* fac = reinterpret_cast<const float*>(static_cast<const uint8_t*>(p.workspace) + q4_rows_factors(p.T, segs)) + t0;
      int it = 0;
      for (; it < rounds * pairs; ++it) {
        const int slot = it % mp.SA, rd = it / pairs, seg = 2 * (it - rd * pairs), n = min(2, segs - seg);
        if (it >= mp.SA && !pf_wait(&bb.a_empty[slot], ((it / mp.SA) - 1) & 1, abort, err)) break;
        mbar_arrive_expect_tx(&bb.a_full[slot], a_stage + n * fbytes);
        tma_3d(sm_a + slot * a_stage, &mp.tm_x, 0, t0, 2 * seg, &bb.a_full[slot]);
        for (int j = 0; j < n; ++j)
          bulk_g2s(s_factor[(rd * segs + seg + j) % kMmRing], fac + static_cast<size_t>(seg + j) * tpad, fbytes, &bb.a_full[slot]);
      }
      for (int j = max(it - mp.SA, 0); j < it; ++j) mbar_wait_bounded(&bb.a_full[j % mp.SA], (j / mp.SA) & 1, 1000000);
    }
  } else if (warp < 4) {
    // ---- MMA: a segment of every pair for each of the two warps (an instruction takes ~45 cycles to issue)
    const int w = warp - 2;
    const uint32_t idesc = idesc_m128(N16, false);
    bool ok = true;
    for (int gi = 0; gi < rounds * groups && ok; ++gi) {
      const int rd = gi / groups, g = gi - rd * groups, set = gi & 1;
      if (gi >= 2 && !pf_wait_all(&bb.d_empty[set], ((gi >> 1) - 1) & 1, abort, err)) break;
      for (int j = 0; j < kMmGroup / 2 && kMmGroup / 2 * g + j < pairs; ++j) {
        const int it = rd * pairs + kMmGroup / 2 * g + j, sa = it % mp.SA, sb = it % kMmSB;
        if (!pf_wait_all(&bb.a_full[sa], (it / mp.SA) & 1, abort, err) ||
            !pf_wait_all(&bb.b_full[sb], (it / kMmSB) & 1, abort, err)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (kMmGroup * g + 2 * j + w < segs) {
          const uint32_t a0 = smem_u32(sm_a + sa * a_stage) + w * TB * 256, b0 = smem_u32(sm_b + sb * b_stage) + w * N16 * 256;
          const uint32_t d = tmem + (set * kMmGroup + 2 * j + w) * kMmRows;
#pragma unroll
          for (int ks = 0; ks < 8; ++ks)
            tc_mma_ss_w(d, sdesc_sw128(a0 + (ks >> 2) * TB * 128 + (ks & 3) * 32),
                        sdesc_sw128(b0 + (ks >> 2) * N16 * 128 + (ks & 3) * 32), idesc, ks ? 1u : 0u);
        }
        tc_commit_w(&bb.a_empty[sa]);
        tc_commit_w(&bb.b_empty[sb]);
      }
      if (ok) tc_commit_w(&bb.d_full[set]);
    }
    tc_commit_w(&bb.done[w]);
    pf_wait_all(&bb.done[w], 0, abort, err);
  } else if (warp < 12) {
    // ---- decoding: teams take pairs in turn; a thread has 32 codes of both segments of the rows row0 and row0 + 32
    const int team = (warp - 4) >> 2, id = (threadIdx.x - 128) & 127, row0 = id >> 2, q = id & 3;
    const bool resident = mp.scale_bytes > 0;
    bool ok = !resident || pf_wait_all(&bb.scales, 0, abort, err);
    for (int rd = 0; rd < rounds && ok; ++rd) {
      const int base = (first + rd) * R;
      for (int c = 0; c < chunks && ok; ++c) {
        const int ci = rd * chunks + c, sc = ci % mp.SC;
        if (!(ok = pf_wait_all(&bb.c_full[sc], (ci / mp.SC) & 1, abort, err))) break;
        for (int pp = 0; pp < kMmChunk / 2; ++pp) {
          const int pi = c * (kMmChunk / 2) + pp, it = rd * pairs + pi, sb = it % kMmSB;
          if (pi >= pairs || (it & 1) != team) continue;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int row = row0 + 32 * h, n = min(base + row, p.N - 1), at = pp * R + row;
            uint32_t v[2][16], scale[2] = {0, 0};
            if (row < R) {
              const uint8_t* sp = resident ? sm_s + (n - first * R) * scale_row : p.scales + n * scale_row;
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int seg = 2 * pi + j;
                if constexpr (kI4) {
                  if (seg < segs) scale[j] = reinterpret_cast<const uint16_t*>(sp)[seg];
                } else if (seg * 128 + 32 * q < p.K) {
                  scale[j] = *reinterpret_cast<const uint16_t*>(sp + 8 * seg + 2 * q);
                }
                decode_f16<AR>(*reinterpret_cast<const uint4*>(sm_c + sc * c_stage + at * 128 + (((4 * j + q) ^ (at & 7)) << 4)),
                               scale[j], v[j]);
              }
            }
            if (h == 0 && it >= kMmSB && !(ok = pf_wait_all(&bb.b_empty[sb], ((it / kMmSB) - 1) & 1, abort, err))) break;
            if (row < R) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                uint8_t* dst = sm_b + sb * b_stage + (2 * j + (q >> 1)) * N16 * 128 + row * 128;
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  *reinterpret_cast<uint4*>(dst + ((((q & 1) * 4 + i) ^ (row & 7)) << 4)) =
                      make_uint4(v[j][4 * i], v[j][4 * i + 1], v[j][4 * i + 2], v[j][4 * i + 3]);
                if (kI4 && q == j) s_scale[(rd * segs + 2 * pi + j) % kMmRing][row] = bf16_bits_to_f32(static_cast<uint16_t>(scale[j]));
              }
            }
          }
          if (!ok) break;
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) mbar_arrive(&bb.b_full[sb]);
        }
        if (ok && lane == 0) mbar_arrive(&bb.c_empty[sc]);
      }
    }
  } else {
    // ---- sums: a thread per token; the two sets of four warps take 16 rows in turn
    const int t = 32 * (warp & 3) + lane, half = (warp - 12) >> 2;
    const uint32_t base = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const float ts = p.tscale ? __ldg(p.tscale) : 1.f;
    const float* factors = s_factor[0] + min(t, kMmTokens - 1);
    bool ok = true;
    for (int rd = 0; rd < rounds && ok; ++rd) {
      float acc[kMmRows / 2];                    // rows 16 (2 b + half) + j at 16 b + j
#pragma unroll
      for (int j = 0; j < kMmRows / 2; ++j) acc[j] = 0.f;
      for (int g = 0; g < groups; ++g) {
        const int gi = rd * groups + g, set = gi & 1, s0 = g * kMmGroup, it0 = rd * segs + s0;
        if (!(ok = pf_wait_all(&bb.d_full[set], (gi >> 1) & 1, abort, err))) break;
        tc_fence_after();
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const int n0 = 16 * (2 * b + half);
          if (n0 < N16) {
#pragma unroll
            for (int jj = 0; jj < kMmGroup; jj += 2) {
              uint32_t d[2][16];
#pragma unroll
              for (int j = 0; j < 2; ++j) tc_ld16(base + (set * kMmGroup + jj + j) * kMmRows + n0, d[j]);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                if (s0 + jj + j < segs) {
                  const int ring = (it0 + jj + j) % kMmRing;
                  const float f = factors[ring * kMmTokens];
                  const float* sc = &s_scale[ring][n0];
#pragma unroll
                  for (int i = 0; i < 16; i += 4) {
                    float4 s = make_float4(1.f, 1.f, 1.f, 1.f);
                    if constexpr (kI4) s = *reinterpret_cast<const float4*>(sc + i);
                    add_scaled(acc[16 * b + i], acc[16 * b + i + 1], d[j][i], d[j][i + 1], f, s.x, s.y, kI4);
                    add_scaled(acc[16 * b + i + 2], acc[16 * b + i + 3], d[j][i + 2], d[j][i + 3], f, s.z, s.w, kI4);
                  }
                }
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bb.d_empty[set]);
      }
      if (!ok) break;
      const int r0 = (first + rd) * R, nn = min(R, p.N - r0);
      if (t < TB && t0 + t < p.T) {
        uint16_t* y = p.y + static_cast<long long>(t0 + t) * p.ldy + r0;
#pragma unroll
        for (int j = 0; j < kMmRows / 2; ++j) {
          const int row = 16 * (2 * (j >> 4) + half) + (j & 15);
          if (row < nn) y[row] = from_f32<TYPE>(acc[j] * ts);
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int AR, int TYPE>
cudaError_t launch_mm(const Q4Params& p, cudaStream_t s) {
  constexpr int kMost = 226 * 1024 - static_cast<int>(sizeof(MmBars)) - kMmRing * 4 * (kMmRows + kMmTokens) - 256;
  int dev, sms;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  const int segs = (p.K + 127) / 128;
  MmParams mp;
  mp.q = p;
  const int per_cta = (p.N + sms - 1) / sms;
  mp.rounds = (per_cta + kMmRows - 1) / kMmRows;
  mp.R = (per_cta + mp.rounds - 1) / mp.rounds;
  mp.N16 = (mp.R + 15) & ~15;
  const int token_chunks = (p.T + kMmTokens - 1) / kMmTokens;
  mp.TB = ((p.T + token_chunks - 1) / token_chunks + 7) & ~7;
  const long long scale_row = AR == kF16Int4 ? p.K >> 6 : p.K >> 4;
  const long long scale_all = (static_cast<long long>(mp.rounds) * mp.R * scale_row + 127) & ~127ll;
  const bool sc16 = scale_row % 16 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 15u) == 0;
  mp.scale_bytes = sc16 && scale_all <= 16 * 1024 ? static_cast<int>(scale_all) : 0;
  mp.boxed = p.K % 256 == 0;
  const int a_stage = mp.TB * 512, b_stage = mp.N16 * 512, c_stage = mm_code_stage(mp.R);
  const int fixed = 1024 + kMmSB * b_stage + mp.scale_bytes;
  mp.SA = mp.TB > 64 ? 2 : 3;
  mp.SC = (kMost - fixed - mp.SA * a_stage) / c_stage;
  if (mp.SC > kMmMaxStages) mp.SC = kMmMaxStages;
  if (mp.SC < 1) return cudaErrorInvalidConfiguration;
  int smem = fixed + mp.SA * a_stage + mp.SC * c_stage;
  // the last 64-K block of the operand's last stage is read 128 rows high
  const int over = 1024 + mp.SA * a_stage - mp.TB * 128 + 128 * 128;
  if (smem < over) smem = over;
  if (!(mp.boxed ? encode_words_blocks(&mp.tm_codes, p.codes, p.N, p.K / 2, mp.R, kMmChunk / 2)
                 : encode_words(&mp.tm_codes, p.codes, p.N, p.K / 2, mp.R)) ||
      !encode_16bit_blocks(&mp.tm_x, p.workspace, false, p.T, static_cast<uint64_t>(segs) * 128, static_cast<uint64_t>(segs) * 128,
                           mp.TB, 4))
    return cudaErrorInvalidValue;
  if ((e = allow_smem_once<q4_mma_kernel<AR, TYPE>>(dev, kMost)) != cudaSuccess) return e;
  if ((e = launch_q4_operand<AR, TYPE, kRows>(p, sms, s)) != cudaSuccess) return e;
  const int total = (p.N + mp.R - 1) / mp.R;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((total + mp.rounds - 1) / mp.rounds, (p.T + mp.TB - 1) / mp.TB);
  cfg.blockDim = dim3(kMmThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q4_mma_kernel<AR, TYPE>, mp);
}

}  // namespace

cudaError_t launch_q4_mma(const Q4Params& p, cudaStream_t s) {
  if (p.fmt == kInt4) return p.type == kTBf16 ? launch_mm<kF16Int4, kTBf16>(p, s) : launch_mm<kF16Int4, kTF16>(p, s);
  return p.type == kTBf16 ? launch_mm<kF16Nvfp4, kTBf16>(p, s) : launch_mm<kF16Nvfp4, kTF16>(p, s);
}

cudaError_t read_q4_mma_error(unsigned* out) {
  const unsigned zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_ops_error_q4mma, sizeof(unsigned));
  if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_ops_error_q4mma, &zero, sizeof(unsigned));
  return e;
}

}  // namespace flint
