// Linear products with 4-bit weights for more than 8 tokens (flint_q4_linear) on tcgen05.
//
// The tokens are the M side of the MMA (128 rows of the operand of q4_operand.cuh, those behind T unused) and the rows
// of W its N side, so that W divides evenly over the SMs: a CTA has up to 64 rows per round, whatever N is. Per
// 128-segment eight warps decode the codes to exact fp16 into shared memory, one of two warps (in turn) issues the MMAs
// into its own accumulator, and four warps add that accumulator, times the rows' group scales and the tokens' factors,
// to fp32 sums in registers: scales of any range and tokens of any magnitude lose nothing.
// Codes come by TMA, 1024 K of all rows per stage; the operand too, a segment per stage, with its factors.
// Bound by the MMA issue (about 45 cycles each, eight per segment, two issuers) against the weight stream.
#include "kernels.cuh"
#include "ops.cuh"
#include "q4_operand.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace flint {

__device__ unsigned g_ops_error_q4mma;           // timeout bits of bounded waits (flint_ops_error_word)

namespace {

constexpr int kMmThreads = 512;                  // copies: 2 warps, MMA: 2, decoding: 8, sums: 4
constexpr int kMmRows = 64;                      // rows of W per round at most
constexpr int kMmTokens = 128;
constexpr int kMmChunk = 8;                      // segments of codes per stage
constexpr int kMmSB = 3;                         // decoded segments in flight
constexpr int kMmRing = 8;                       // segments of scales and factors kept for the sums (see below)
constexpr int kMmMaxStages = 4;

struct MmParams {
  CUtensorMap tm_codes;                          // boxed: [K / 256][N][128 bytes], else [N][K / 2 bytes]
  CUtensorMap tm_x;                              // operand rows [T][segs * 128] fp16, 64 x TB boxes
  Q4Params q;
  int R, N16;                                    // rows of W per round; padded to 16
  int rounds;                                    // per CTA
  int TB;                                        // operand rows per stage: T rounded up to 8, at most 128
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

template <int AR, int TYPE>
__global__ void __launch_bounds__(kMmThreads, 1) q4_mma_kernel(const __grid_constant__ MmParams mp) {
  const Q4Params& p = mp.q;
  constexpr bool kI4 = AR == kF16Int4;
  extern __shared__ uint8_t smem_raw[];
  __shared__ MmBars bb;
  __shared__ __align__(16) float s_scale[kMmRing][kMmRows];      // of the rows, per segment
  __shared__ __align__(16) float s_factor[kMmRing][kMmTokens];   // of the tokens, per segment
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int segs = (p.K + 127) / 128, chunks = (segs + kMmChunk - 1) / kMmChunk;
  const int R = mp.R, N16 = mp.N16, TB = mp.TB;
  const int a_stage = TB * 256, b_stage = N16 * 256, c_stage = mm_code_stage(R);
  const int t0 = blockIdx.y * kMmTokens, first = blockIdx.x * mp.rounds, total = (p.N + R - 1) / R;
  const int rounds = min(mp.rounds, total - first);
  // operand first: the MMA reads 128 rows from a stage's start, past its end into what follows (unused accumulator rows)
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
      mbar_init(&bb.a_empty[i], 1);
    }
    for (int i = 0; i < kMmSB; ++i) {
      mbar_init(&bb.b_full[i], 8);
      mbar_init(&bb.b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bb.d_full[i], 1);
      mbar_init(&bb.d_empty[i], 4);
      mbar_init(&bb.done[i], 1);
    }
    mbar_init(&bb.scales, 1);
    bb.abort = 0;
    fence_mbar_init();
  }
  if (warp == 2) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 128;" ::"r"(smem_u32(&bb.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bb.tmem;
  const int steps = rounds * segs;               // segments of all rounds

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
    // ---- operand: 64 K per box, and the segment's factors
    if (lane == 0) {
      pdl_wait();
      const int tpad = (p.T + 3) & ~3, fbytes = min(kMmTokens, tpad - t0) * 4;
      const float* fac = reinterpret_cast<const float*>(static_cast<const uint8_t*>(p.workspace) + q4_rows_factors(p.T, segs)) + t0;
      int it = 0;
      for (; it < steps; ++it) {
        const int slot = it % mp.SA, seg = it % segs;
        if (it >= mp.SA && !pf_wait(&bb.a_empty[slot], ((it / mp.SA) - 1) & 1, abort, err)) break;
        uint8_t* st = sm_a + slot * a_stage;
        mbar_arrive_expect_tx(&bb.a_full[slot], a_stage + fbytes);
        tma_2d(st, &mp.tm_x, seg * 128, t0, &bb.a_full[slot]);
        tma_2d(st + a_stage / 2, &mp.tm_x, seg * 128 + 64, t0, &bb.a_full[slot]);
        bulk_g2s(s_factor[it % kMmRing], fac + static_cast<size_t>(seg) * tpad, fbytes, &bb.a_full[slot]);
      }
      for (int j = max(it - mp.SA, 0); j < it; ++j) mbar_wait_bounded(&bb.a_full[j % mp.SA], (j / mp.SA) & 1, 1000000);
    }
  } else if (warp < 4) {
    // ---- MMA: the two warps take segments in turn, each into its own 64 columns
    const int w = warp - 2;
    const uint32_t idesc = idesc_m128(N16, false), d = tmem + w * 64;
    for (int it = w, n = 0; it < steps; it += 2, ++n) {
      const int sa = it % mp.SA, sb = it % kMmSB;
      if (n > 0 && !pf_wait_all(&bb.d_empty[w], (n - 1) & 1, abort, err)) break;
      if (!pf_wait_all(&bb.a_full[sa], (it / mp.SA) & 1, abort, err) ||
          !pf_wait_all(&bb.b_full[sb], (it / kMmSB) & 1, abort, err))
        break;
      tc_fence_after();
      const uint32_t a0 = smem_u32(sm_a + sa * a_stage), b0 = smem_u32(sm_b + sb * b_stage);
#pragma unroll
      for (int ks = 0; ks < 8; ++ks)
        tc_mma_ss_w(d, sdesc_sw128(a0 + (ks >> 2) * (a_stage / 2) + (ks & 3) * 32),
                    sdesc_sw128(b0 + (ks >> 2) * (b_stage / 2) + (ks & 3) * 32), idesc, ks ? 1u : 0u);
      tc_commit_w(&bb.a_empty[sa]);
      tc_commit_w(&bb.b_empty[sb]);
      tc_commit_w(&bb.d_full[w]);
    }
    tc_commit_w(&bb.done[w]);
    pf_wait_all(&bb.done[w], 0, abort, err);
  } else if (warp < 12) {
    // ---- decoding: a thread per (row, 32 codes) of a segment
    const int id = threadIdx.x - 128, row = id >> 2, q = id & 3;
    const bool mine = row < R;
    uint8_t* dst = sm_b + (q >> 1) * (b_stage / 2) + row * 128;
    const bool resident = mp.scale_bytes > 0;
    bool ok = !resident || pf_wait_all(&bb.scales, 0, abort, err);
    for (int rd = 0; rd < rounds && ok; ++rd) {
      const int n = min((first + rd) * R + min(row, R - 1), p.N - 1);
      const uint8_t* gs = p.scales + n * scale_row;
      const uint8_t* ss = sm_s + (n - first * R) * scale_row;
      for (int seg = 0; seg < segs; ++seg) {
        const int it = rd * segs + seg, sb = it % kMmSB, ci = rd * chunks + seg / kMmChunk, sc = ci % mp.SC;
        uint32_t scale = 0;
        if (mine) {
          if constexpr (kI4) {
            if (q == 0) scale = resident ? reinterpret_cast<const uint16_t*>(ss)[seg] : __ldg(reinterpret_cast<const uint16_t*>(gs) + seg);
          } else if (seg * 128 + 32 * q < p.K) {
            scale = resident ? *reinterpret_cast<const uint16_t*>(ss + 8 * seg + 2 * q)
                             : __ldg(reinterpret_cast<const uint16_t*>(gs + 8 * seg + 2 * q));
          }
        }
        if (seg % kMmChunk == 0 && !(ok = pf_wait_all(&bb.c_full[sc], (ci / mp.SC) & 1, abort, err))) break;
        uint32_t v[16];
        if (mine) {
          const int kb = (seg % kMmChunk) >> 1, at = kb * R + row;
          decode_f16<AR>(*reinterpret_cast<const uint4*>(sm_c + sc * c_stage + at * 128 + (((4 * (seg & 1) + q) ^ (at & 7)) << 4)),
                         scale, v);
        }
        if (it >= kMmSB && !(ok = pf_wait_all(&bb.b_empty[sb], ((it / kMmSB) - 1) & 1, abort, err))) break;
        if (mine) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(dst + sb * b_stage + ((((q & 1) * 4 + i) ^ (row & 7)) << 4)) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          if (kI4 && q == 0) s_scale[it % kMmRing][row] = bf16_bits_to_f32(static_cast<uint16_t>(scale));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&bb.b_full[sb]);
          if (seg % kMmChunk == kMmChunk - 1 || seg == segs - 1) mbar_arrive(&bb.c_empty[sc]);
        }
      }
    }
  } else {
    // ---- sums: a thread per token, the rows in registers. The rings of scales and factors hold 8 segments: the MMA is
    // at most 2 segments ahead of the sums (two accumulators), decoding and copies at most kMmSB and SA <= 4 ahead of it.
    const int t = 32 * (warp & 3) + lane;
    const uint32_t base = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
    const float ts = p.tscale ? __ldg(p.tscale) : 1.f;
    bool ok = true;
    for (int rd = 0; rd < rounds && ok; ++rd) {
      float acc[kMmRows];
#pragma unroll
      for (int j = 0; j < kMmRows; ++j) acc[j] = 0.f;
      for (int seg = 0; seg < segs; ++seg) {
        const int it = rd * segs + seg, w = it & 1;
        if (!(ok = pf_wait_all(&bb.d_full[w], (it >> 1) & 1, abort, err))) break;
        tc_fence_after();
        const float f = s_factor[it % kMmRing][t];
#pragma unroll
        for (int j0 = 0; j0 < kMmRows; j0 += 16) {
          if (j0 < N16) {
            uint32_t d[16];
            tc_ld16(base + w * 64 + j0, d);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
              if constexpr (kI4) {
                const float4 s = *reinterpret_cast<const float4*>(&s_scale[it % kMmRing][j0 + j]);
                acc[j0 + j] = fmaf(__uint_as_float(d[j]) * f, s.x, acc[j0 + j]);
                acc[j0 + j + 1] = fmaf(__uint_as_float(d[j + 1]) * f, s.y, acc[j0 + j + 1]);
                acc[j0 + j + 2] = fmaf(__uint_as_float(d[j + 2]) * f, s.z, acc[j0 + j + 2]);
                acc[j0 + j + 3] = fmaf(__uint_as_float(d[j + 3]) * f, s.w, acc[j0 + j + 3]);
              } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[j0 + j + i] = fmaf(__uint_as_float(d[j + i]), f, acc[j0 + j + i]);
              }
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bb.d_empty[w]);
      }
      if (!ok) break;
      const int n0 = (first + rd) * R, nn = min(R, p.N - n0);
      if (t0 + t < p.T) {
        uint16_t* y = p.y + static_cast<long long>(t0 + t) * p.ldy + n0;
#pragma unroll
        for (int j = 0; j < kMmRows; ++j)
          if (j < nn) y[j] = from_f32<TYPE>(acc[j] * ts);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 2) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 128;" ::"r"(tmem));
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
  mp.TB = p.T >= kMmTokens ? kMmTokens : (p.T + 7) & ~7;
  const long long scale_row = AR == kF16Int4 ? p.K >> 6 : p.K >> 4;
  const long long scale_all = (static_cast<long long>(mp.rounds) * mp.R * scale_row + 127) & ~127ll;
  const bool sc16 = scale_row % 16 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 15u) == 0;
  mp.scale_bytes = sc16 && scale_all <= 32 * 1024 ? static_cast<int>(scale_all) : 0;
  mp.boxed = p.K % 256 == 0;
  // the operand's last stage is read 128 rows high: what follows it (decoded segments and codes) is at least as large
  const int a_stage = mp.TB * 256, b_stage = mp.N16 * 256, c_stage = mm_code_stage(mp.R);
  const int fixed = 1024 + kMmSB * b_stage + mp.scale_bytes;
  mp.SA = mp.TB > 64 ? 2 : 4;
  mp.SC = (kMost - fixed - mp.SA * a_stage) / c_stage;
  if (mp.SC > kMmMaxStages) mp.SC = kMmMaxStages;
  if (mp.SC < 1) return cudaErrorInvalidConfiguration;
  int smem = fixed + mp.SA * a_stage + mp.SC * c_stage;
  const int over = 1024 + (mp.SA - 1) * a_stage + a_stage / 2 + 128 * 128;
  if (smem < over) smem = over;
  if (!(mp.boxed ? encode_words_blocks(&mp.tm_codes, p.codes, p.N, p.K / 2, mp.R, kMmChunk / 2)
                 : encode_words(&mp.tm_codes, p.codes, p.N, p.K / 2, mp.R)) ||
      !encode_16bit(&mp.tm_x, p.workspace, false, p.T, static_cast<uint64_t>(segs) * 128, static_cast<uint64_t>(segs) * 128, mp.TB))
    return cudaErrorInvalidValue;
  if ((e = allow_smem_once<q4_mma_kernel<AR, TYPE>>(dev, kMost)) != cudaSuccess) return e;
  if ((e = launch_q4_operand<AR, TYPE, kRows>(p, sms, s)) != cudaSuccess) return e;
  const int total = (p.N + mp.R - 1) / mp.R;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((total + mp.rounds - 1) / mp.rounds, (p.T + kMmTokens - 1) / kMmTokens);
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
