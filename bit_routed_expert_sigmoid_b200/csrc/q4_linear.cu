// Linear products with 4-bit weights for few tokens (flint_q4_linear):
//   y[t][n] = ts * sum over 128-segments of  s[n] * (code[n] . x'[t]),  x' = x or blockdiag(Hn) x.
//
// Up to 8 tokens (this file; more: q4_mma.cu). 8192 x 8192 int4 takes 15.4 us at T = 8 and 13.1 at T = 1, NVFP4 22.8 at
// T = 8; T = 9 takes 20.1 in the other file. These, and all times in this file, are of calls in a CUDA graph, whose weights
// (36 MB here) stay in L2; with L2 flushed, and the launch included, 21.4, 19.6 and 29.2. Once through HBM the weights are
// 5.3 us, and a launch that only reads the codes takes 8.3. Nothing is near saturated: at T = 8 40 % of the issue slots are
// used, 25 % of DRAM, 13 % of the tensor pipe; a warp waits a third of its time for loads and stages (NVFP4: 54, 18 and 9 %,
// and more for the arithmetic pipes that decode, and for its turn, than for loads).
//
// The rows of W are divided evenly over one CTA per SM (not in units of a tile); the 16 warps of a CTA split K: a warp
// takes a 128-segment of one or two blocks of up to 16 rows at a time, as fragments of mma.sync. A fragment's K order is
// free as long as x has the same: a lane's 16 bytes are 32 neighbouring K of one row. The int4 group scale and the operand's
// factor (q4_operand.cuh) multiply the segment's sum in fp32.
//
// With few segments every CTA builds the operand itself in shared memory; with more, one kernel builds it once in the
// workspace and the product kernel, launched behind it as a programmatic dependent, starts its weight copies meanwhile.
#include "kernels.cuh"
#include "ops.cuh"
#include "q4_operand.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace flint {

__device__ unsigned g_ops_error_q4;              // timeout bits of bounded waits (flint_ops_error_word)

namespace {

constexpr int kQ4Threads = 512;
constexpr int kQ4Warps = kQ4Threads / 32;
// (token, segment) pairs up to which each CTA builds the operand itself: 64 pairs (8192 x 8192, T = 1) take 12.8 us so and
// 15.4 with the separate kernel, 128 (2048 x 2048, T = 8) 8.4 and 6.4.
constexpr int kQ4Inline = 64;

// d += A B on the integer tensor cores (m16n8k32): A s8, B s8 or u8
template <bool SIGNED_B>
__device__ __forceinline__ void mma_s8_16832(int (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (SIGNED_B)
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.u8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+r"(d[0]), "+r"(d[1]), "+r"(d[2]), "+r"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// The codes of rows g and g + 8 (a lane's 16 bytes each) as the A operand of one segment.
template <int AR>
struct AFrag {
  uint32_t a[2][16];
  __device__ __forceinline__ void decode(const uint4 (&c)[2], const uint32_t (&s)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) decode_f16<AR>(c[h], s[h], a[h]);
  }
  // sums over the segment of the lane's two rows (0, 1: row g, tokens 2q and 2q + 1; 2, 3: row g + 8), two chains
  __device__ __forceinline__ void times(const uint4 (&x)[4], float (&d)[4]) const {
    float e[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m0[4] = {a[0][4 * i], a[1][4 * i], a[0][4 * i + 1], a[1][4 * i + 1]};
      const uint32_t m1[4] = {a[0][4 * i + 2], a[1][4 * i + 2], a[0][4 * i + 3], a[1][4 * i + 3]};
      mma_f16_16816(d, m0, x[i].x, x[i].y);
      mma_f16_16816(e, m1, x[i].z, x[i].w);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] += e[j];
  }
};

template <>
struct AFrag<kLimbs> {
  uint32_t even[2][4], odd[2][4];                // int8 16 c: nibbles 0, 2, 4, 6 and 1, 3, 5, 7 of a word
  __device__ __forceinline__ void decode(const uint4 (&c)[2], const uint32_t (&)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w[4] = {c[h].x, c[h].y, c[h].z, c[h].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        even[h][i] = (w[i] << 4) & 0xF0F0F0F0u;
        odd[h][i] = w[i] & 0xF0F0F0F0u;
      }
    }
  }
  // |256 hi + lo| <= 128 * 128 * 2^15 < 2^31: exact
  __device__ __forceinline__ void times(const uint4 (&x)[4], float (&d)[4]) const {
    int hi[4] = {0, 0, 0, 0}, lo[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t m[4] = {even[0][i], even[1][i], odd[0][i], odd[1][i]};
      const uint4& xh = x[i >> 1];
      const uint4& xl = x[2 + (i >> 1)];
      mma_s8_16832<true>(hi, m, i & 1 ? xh.z : xh.x, i & 1 ? xh.w : xh.y);
      mma_s8_16832<false>(lo, m, i & 1 ? xl.z : xl.x, i & 1 ? xl.w : xl.y);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) d[j] = static_cast<float>(hi[j] * 256 + lo[j]);
  }
};

// ---------------------------------------------------------------------------------------------
// The product, codes streamed by TMA: one thread keeps a ring of stages full, a stage being 128 K per warp of a team
// for RB blocks of R rows per team. Blocks have the same R <= 16 rows everywhere (the rows of W divided evenly over the
// SMs), which is the height of the TMA box, so no row is read twice; a box holds all 256-code blocks of a stage (K a
// multiple of 256), or one of them. Rows are 128 bytes in the 128-byte swizzle, counted from the 1024-byte aligned
// ring. NVFP4 rows that are no multiple of 16 bytes (K % 32 = 16) have no tensor map: the warps read them themselves
// (TMA = false; the same blocks and order).
// Whatever a step needs comes through the ring, x and (where their rows are multiples of 16 bytes) the scales too: an
// ordinary load issued behind 150 KB of copies waits for all of them, which cost 5 us of 17 at 8192 x 8192, T = 8, for
// x and for the scales each.
constexpr int kRingThreads = kQ4Threads + 32;
constexpr int kRingMaxStages = 8;
// Warps of a team at most: 8, two teams sharing a stage's x (8192 x 8192, T = 8: 15.4 us; 4 or 16 warps 18.0, 16.3),
// but all 16 where a CTA has one block of rows (2048 x 2048, T = 8: 5.3 us against 6.4).
constexpr int kQ4Split = 8;
constexpr int kQ4ScaleBytes = 72 * 1024;         // scales kept in shared memory at most

struct RingParams {
  CUtensorMap tm;                                // boxed: [K / 256][N][128 bytes], else [N][K / 2 bytes]
  Q4Params q;
  int kw;                                        // warps of a team
  int R;                                         // rows of a block
  int blocks;                                    // blocks per CTA, a multiple of RB * teams
  int stages, boxed;
  int scale_bytes;                               // of the CTA's rows, kept in shared memory; 0: loaded when needed
};

struct RingBars {
  uint64_t full[kRingMaxStages], empty[kRingMaxStages], scales;
  int abort;
};

// Bytes of a block's rows in a stage: whole swizzle atoms, so that a lane's place in them is the same in every block.
__host__ __device__ inline int ring_region(int kw, int R) { return ((kw + 1) / 2 * R * 128 + 1023) & ~1023; }

template <int AR, int TYPE, int RB, bool TMA, bool INLINE>
__global__ void __launch_bounds__(kRingThreads, 1) q4_ring_kernel(const __grid_constant__ RingParams rp) {
  const Q4Params& p = rp.q;
  extern __shared__ uint8_t smem_raw[];
  __shared__ RingBars bb;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int segs = (p.K + 127) / 128, teams = kQ4Warps / rp.kw, chunks = (segs + rp.kw - 1) / rp.kw;
  constexpr bool kXRing = TMA && !INLINE;                        // x through the ring
  const int R = rp.R, kbs = (rp.kw + 1) / 2, region = ring_region(rp.kw, R);
  const int xstage = kXRing ? rp.kw * p.T * kTokenBytes : 0;
  const int stage = (teams * RB * region + xstage + 1023) & ~1023;
  const int total = (p.N + R - 1) / R, first = blockIdx.x * rp.blocks, rounds = rp.blocks / (teams * RB);
  constexpr bool kI4 = AR != kF16Nvfp4;
  const size_t scale_row = kI4 ? p.K >> 6 : p.K >> 4;            // bytes
  uint8_t* ring = align1024(smem_raw);
  float4* red = reinterpret_cast<float4*>(ring + rp.stages * stage);           // [warps][RB][32]
  uint8_t* sm_scales = reinterpret_cast<uint8_t*>(red + kQ4Warps * RB * 32);
  uint8_t* sm_x = sm_scales + rp.scale_bytes;                    // INLINE: the operand
  volatile int* abort = &bb.abort;

  if constexpr (TMA) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < rp.stages; ++i) {
        mbar_init(&bb.full[i], kXRing ? 2 : 1);
        mbar_init(&bb.empty[i], kQ4Warps);
      }
      mbar_init(&bb.scales, 1);
      bb.abort = 0;
      fence_mbar_init();
    }
    __syncthreads();
  }
  // Behind the operand kernel the weights may be read at once: all that ran before that one is complete.
  if constexpr (INLINE) pdl_wait();
  pdl_trigger();
  if (warp == kQ4Warps) {
    if (TMA && lane == 0) {
      // weights are no predecessor's output: copied before griddepcontrol.wait; x is the operand kernel's
      const uint64_t pol = l2_evict_first();
      const int steps = rounds * chunks;
      const uint8_t* img = static_cast<const uint8_t*>(p.workspace);
      auto copy_x = [&](int it, int slot) {
        const int c = it % chunks, n = min(rp.kw, segs - c * rp.kw) * p.T * kTokenBytes;
        mbar_arrive_expect_tx(&bb.full[slot], n);
        bulk_g2s(ring + slot * stage + teams * RB * region, img + static_cast<size_t>(c) * rp.kw * p.T * kTokenBytes, n,
                 &bb.full[slot]);
      };
      auto copy_codes = [&](int it, int slot) {
        const int rd = it / chunks, c = it - rd * chunks, b0 = first + rd * teams * RB, n = min(teams * RB, total - b0);
        uint8_t* st = ring + slot * stage;
        mbar_arrive_expect_tx(&bb.full[slot], max(n, 0) * kbs * R * 128);
        for (int j = 0; j < n; ++j, st += region) {
          if (rp.boxed) {
            tma_3d_hint(st, &rp.tm, 0, (b0 + j) * R, c * kbs, &bb.full[slot], pol);
          } else {
            for (int b = 0; b < kbs; ++b)
              tma_2d_hint(st + b * R * 128, &rp.tm, (c * kbs + b) * 32, (b0 + j) * R, &bb.full[slot], pol);
          }
        }
      };
      if (rp.scale_bytes) {
        const int rows = min(rp.blocks * R, p.N - first * R);
        mbar_arrive_expect_tx(&bb.scales, rows * static_cast<int>(scale_row));
        bulk_g2s_hint(sm_scales, p.scales + first * R * scale_row, rows * static_cast<int>(scale_row), &bb.scales, pol);
      }
      int it = 0;
      const int ahead = min(rp.stages, steps);
      for (; it < ahead; ++it) copy_codes(it, it);
      if constexpr (kXRing) {
        pdl_wait();
        for (int j = 0; j < ahead; ++j) copy_x(j, j);
      }
      for (; it < steps; ++it) {
        const int slot = it % rp.stages;
        if (!pf_wait(&bb.empty[slot], ((it / rp.stages) - 1) & 1, abort, &g_ops_error_q4)) break;
        if constexpr (kXRing) copy_x(it, slot);
        copy_codes(it, slot);
      }
      // no copy in flight when the CTA exits
      for (int j = max(it - rp.stages, 0); j < it; ++j)
        mbar_wait_bounded(&bb.full[j % rp.stages], (j / rp.stages) & 1, 1000000);
      if (rp.scale_bytes) mbar_wait_bounded(&bb.scales, 0, 1000000);
    }
    return;
  }

  const int kw = warp % rp.kw, team = warp / rp.kw, tid = kw * 32 + lane;
  const uint8_t* img = static_cast<const uint8_t*>(p.workspace);

  // the lane's place in a block: row g + 8 h (the last one repeated behind the block's end), its 16 bytes
  uint32_t place[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t row = (kw >> 1) * R + min(g + 8 * h, R - 1);
    place[h] = team * RB * region + row * 128 + (((4 * (kw & 1) + q) ^ (row & 7)) << 4);
  }
  // scales of the lane's rows (NVFP4: of its two 16-blocks), one step ahead of their use; rows behind N repeat the last
  const uint8_t* scales = p.scales + first * R * scale_row + (kI4 ? 0 : 2 * q);
  uint32_t srow[RB][2];                          // behind the CTA's first row
  auto scale_rows = [&](int rd) {
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = min(((rd * teams + team) * RB + r) * R + min(g + 8 * h, R - 1), p.N - 1 - first * R);
        srow[r][h] = static_cast<uint32_t>(row) * static_cast<uint32_t>(scale_row);
      }
  };
  uint32_t sc[RB][2];
  auto load_scales = [&](int seg) {
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (kI4) {
          sc[r][h] = __ldg(reinterpret_cast<const uint16_t*>(scales + (srow[r][h] + 2 * seg)));
        } else if constexpr (TMA) {
          sc[r][h] = seg * 128 + 32 * q < p.K ? __ldg(reinterpret_cast<const uint16_t*>(scales + (srow[r][h] + 8 * seg))) : 0u;
        } else {
          sc[r][h] = seg * 128 + 32 * q < p.K ? __ldg(scales + (srow[r][h] + 8 * seg)) : 0u;
          if (seg * 128 + 32 * q + 16 < p.K) sc[r][h] |= static_cast<uint32_t>(__ldg(scales + (srow[r][h] + 8 * seg + 1))) << 8;
        }
      }
  };
  scale_rows(0);
  const bool resident = TMA && rp.scale_bytes > 0;
  if (!resident && kw < segs) load_scales(kw);
  if constexpr (INLINE) {
    const int pairs = p.T * segs;
    for (int i0 = warp; i0 < pairs; i0 += 4 * kQ4Warps) {
      uint2 raw[4];
      OperandPlace o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = min(i0 + j * kQ4Warps, pairs - 1), t = i / segs, seg = i - t * segs;
        raw[j] = q4_fetch(p, t, seg);
        o[j] = q4_place<kTokens, 1>(sm_x, t, seg, p.T, segs);
        if (i0 + j * kQ4Warps >= pairs) o[j].at = nullptr;
      }
      q4_operand<AR, TYPE, 4>(raw, p.rotated != 0, o);
    }
    named_bar_sync(1, kQ4Threads);
  } else if constexpr (!kXRing) {
    pdl_wait();
  }
  bool ok = true;
  if (resident) ok = pf_wait_all(&bb.scales, 0, abort, &g_ops_error_q4);
  const float ts = p.tscale ? __ldg(p.tscale) : 1.f;

  int it = 0;
  for (int rd = 0; rd < rounds; ++rd) {
    float acc[RB][4];
#pragma unroll
    for (int r = 0; r < RB; ++r)
#pragma unroll
      for (int j = 0; j < 4; ++j) acc[r][j] = 0.f;
    for (int c = 0; c < chunks; ++c, ++it) {
      const int slot = it % rp.stages, seg = c * rp.kw + kw;
      if constexpr (TMA) ok = ok && pf_wait_all(&bb.full[slot], (it / rp.stages) & 1, abort, &g_ops_error_q4);
      if (seg < segs && ok) {
        // lanes behind the last token repeat it: their columns are not used
        const uint8_t* xs = INLINE ? sm_x + seg * p.T * kTokenBytes
                            : TMA  ? ring + slot * stage + teams * RB * region + kw * p.T * kTokenBytes
                                   : img + static_cast<size_t>(seg) * p.T * kTokenBytes;
        const uint8_t* xb = xs + min(g, p.T - 1) * kTokenBytes + 16 * q;
        uint4 x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4*>(xb + 64 * i);
        const float fx = *reinterpret_cast<const float*>(xs + min(2 * q, p.T - 1) * kTokenBytes + 256);
        const float fy = *reinterpret_cast<const float*>(xs + min(2 * q + 1, p.T - 1) * kTokenBytes + 256);
        if (resident) {
#pragma unroll
          for (int r = 0; r < RB; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h)
              sc[r][h] = *reinterpret_cast<const uint16_t*>(sm_scales + (srow[r][h] + (kI4 ? 2 * seg : 8 * seg + 2 * q)));
        }
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          uint4 code[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if constexpr (TMA) {
              code[h] = *reinterpret_cast<const uint4*>(ring + slot * stage + r * region + place[h]);
            } else {
              const int row = min((first + (rd * teams + team) * RB + r) * R + min(g + 8 * h, R - 1), p.N - 1);
              const uint8_t* s = p.codes + static_cast<size_t>(row) * (p.K >> 1) + seg * 64 + 16 * q;
              uint2 a = make_uint2(0, 0), b = a;
              if (seg * 128 + 32 * q < p.K) a = __ldg(reinterpret_cast<const uint2*>(s));
              if (seg * 128 + 32 * q + 16 < p.K) b = __ldg(reinterpret_cast<const uint2*>(s + 8));
              code[h] = make_uint4(a.x, a.y, b.x, b.y);
            }
          }
          AFrag<AR> a;
          a.decode(code, sc[r]);
          const float s0 = kI4 ? bf16_bits_to_f32(static_cast<uint16_t>(sc[r][0])) : 1.f;
          const float s1 = kI4 ? bf16_bits_to_f32(static_cast<uint16_t>(sc[r][1])) : 1.f;
          float d[4];
          a.times(x, d);
          acc[r][0] = fmaf(d[0], s0 * fx, acc[r][0]);
          acc[r][1] = fmaf(d[1], s0 * fy, acc[r][1]);
          acc[r][2] = fmaf(d[2], s1 * fx, acc[r][2]);
          acc[r][3] = fmaf(d[3], s1 * fy, acc[r][3]);
        }
        if (seg + rp.kw < segs) {
          if (!resident) load_scales(seg + rp.kw);
        } else if (rd + 1 < rounds) {
          scale_rows(rd + 1);
          if (!resident) load_scales(kw);
        }
      }
      if constexpr (TMA) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bb.empty[slot]);
      }
    }
    if (kw < segs) {
#pragma unroll
      for (int r = 0; r < RB; ++r) red[(warp * RB + r) * 32 + lane] = make_float4(acc[r][0], acc[r][1], acc[r][2], acc[r][3]);
    }
    if (named_bar_or(team, 32 * rp.kw, !ok)) break;              // a team gives up together
    // add the team's partial sums in warp order
    const float* rf = reinterpret_cast<const float*>(red) + team * rp.kw * RB * 128;
    const int parts = min(rp.kw, segs);
    for (int o = tid; o < RB * 128; o += 32 * rp.kw) {
      const int row = o & 15, t = (o >> 4) & 7, r = o >> 7;
      const int n = (first + (rd * teams + team) * RB + r) * R + row;
      if (t >= p.T || row >= R || n >= p.N) continue;
      const int at = (r * 32 + (row & 7) * 4 + (t >> 1)) * 4 + (row >> 3) * 2 + (t & 1);
      float v = 0.f;
#pragma unroll 4
      for (int w = 0; w < parts; ++w) v += rf[at + w * RB * 128];
      p.y[t * p.ldy + n] = from_f32<TYPE>(v * ts);
    }
    named_bar_sync(team, 32 * rp.kw);
  }
}

template <int AR, int TYPE, int RB, bool TMA, bool INLINE>
cudaError_t launch_rows(const Q4Params& p, int dev, int sms, int kw, cudaStream_t s) {
  constexpr int kRed = kQ4Warps * RB * 512, kMost = 226 * 1024 - static_cast<int>(sizeof(RingBars));
  const int segs = (p.K + 127) / 128, teams = kQ4Warps / kw;
  RingParams rp;
  rp.q = p;
  rp.kw = kw;
  const int per_cta = (p.N + sms - 1) / sms, round = teams * RB;
  rp.blocks = ((per_cta + 15) / 16 + round - 1) / round * round;
  rp.R = (per_cta + rp.blocks - 1) / rp.blocks;
  constexpr bool kI4 = AR != kF16Nvfp4;
  const long long scale_row = kI4 ? p.K >> 6 : p.K >> 4, scale_all = (rp.blocks * rp.R * scale_row + 127) & ~127ll;
  const bool sc16 = scale_row % 16 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 15u) == 0;
  rp.scale_bytes = TMA && sc16 && scale_all <= kQ4ScaleBytes ? static_cast<int>(scale_all) : 0;
  const int xstage = TMA && !INLINE ? kw * p.T * kTokenBytes : 0;
  const int stage = (teams * RB * ring_region(kw, rp.R) + xstage + 1023) & ~1023;
  const int rest = kRed + 1024 + rp.scale_bytes + (INLINE ? static_cast<int>(q4_operand_bytes(p.T, segs)) : 0);
  rp.stages = 0;
  rp.boxed = p.K % 256 == 0;
  if constexpr (TMA) {
    rp.stages = (kMost - rest) / stage;
    if (rp.stages > kRingMaxStages) rp.stages = kRingMaxStages;
    if (rp.stages < 1) return cudaErrorInvalidConfiguration;
    if (!(rp.boxed ? encode_words_blocks(&rp.tm, p.codes, p.N, p.K / 2, rp.R, (kw + 1) / 2)
                   : encode_words(&rp.tm, p.codes, p.N, p.K / 2, rp.R)))
      return cudaErrorInvalidValue;
  }
  cudaError_t e = allow_smem_once<q4_ring_kernel<AR, TYPE, RB, TMA, INLINE>>(dev, kMost);
  if (e != cudaSuccess) return e;
  const int total = (p.N + rp.R - 1) / rp.R;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((total + rp.blocks - 1) / rp.blocks);
  cfg.blockDim = dim3(kRingThreads);
  cfg.dynamicSmemBytes = rp.stages * stage + rest;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, q4_ring_kernel<AR, TYPE, RB, TMA, INLINE>, rp);
}

// Blocks of rows that a team works on at a time: two, sharing a segment's x, where there are as many (8192 x 8192, T = 8:
// 15.4 us; one at a time 17.6).
template <int AR, int TYPE, bool TMA, bool INLINE>
cudaError_t launch_ring(const Q4Params& p, int dev, int sms, cudaStream_t s) {
  const int segs = (p.K + 127) / 128;
  const int blocks = ((p.N + sms - 1) / sms + 15) / 16, split = blocks == 1 ? kQ4Warps : kQ4Split;
  int kw = 1;
  while (kw < segs && kw < split) kw *= 2;
  const int teams = kQ4Warps / kw;
  if (blocks <= teams) return launch_rows<AR, TYPE, 1, TMA, INLINE>(p, dev, sms, kw, s);
  return launch_rows<AR, TYPE, 2, TMA, INLINE>(p, dev, sms, kw, s);
}

template <int AR, int TYPE, bool TMA>
cudaError_t launch_tokens(const Q4Params& p, cudaStream_t s) {
  int dev, sms;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  if (q4_workspace_bytes(p.K, p.T) == 0) return launch_ring<AR, TYPE, TMA, true>(p, dev, sms, s);
  if ((e = launch_q4_operand<AR, TYPE, kTokens>(p, sms, s)) != cudaSuccess) return e;
  return launch_ring<AR, TYPE, TMA, false>(p, dev, sms, s);
}

template <int AR, bool TMA>
cudaError_t launch_type(const Q4Params& p, cudaStream_t s) {
  return p.type == kTBf16 ? launch_tokens<AR, kTBf16, TMA>(p, s) : launch_tokens<AR, kTF16, TMA>(p, s);
}

}  // namespace

cudaError_t read_q4_error(unsigned* out) {
  const unsigned zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(out, g_ops_error_q4, sizeof(unsigned));
  if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_ops_error_q4, &zero, sizeof(unsigned));
  unsigned more = 0;
  if (e == cudaSuccess) e = read_q4_mma_error(&more);
  *out |= more;
  return e;
}

size_t q4_workspace_bytes(int K, int T) {
  const int segs = (K + 127) / 128;
  if (T <= 8 && T * segs <= kQ4Inline) return 0;
  return q4_operand_bytes(T, segs);
}

cudaError_t launch_q4_linear(const Q4Params& p, cudaStream_t s) {
  if (p.T > 8) return launch_q4_mma(p, s);
  if (p.fmt == kInt4) return p.rotated ? launch_type<kLimbs, true>(p, s) : launch_type<kF16Int4, true>(p, s);
  // 16-byte rows of codes and 2-byte aligned pairs of scales where the width and the pointer allow
  const bool tma = p.K % 32 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 1u) == 0;
  return tma ? launch_type<kF16Nvfp4, true>(p, s) : launch_type<kF16Nvfp4, false>(p, s);
}

}  // namespace flint
