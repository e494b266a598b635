// Linear products with 4-bit weights for few tokens (flint_q4_linear):
//   y[t][n] = ts * sum over 128-segments of  s[n] * (code[n] . x'[t]),  x' = x or blockdiag(Hn) x.
//
// Bound by streaming the weights once. The rows of W are spread evenly over one CTA per SM (not in units of a
// tile), and the 16 warps of a CTA split K: a warp takes a 128-segment of up to 16 RB rows straight from global
// memory into the fragments of mma.sync m16n8k16 (a lane's 16 bytes are 32 neighbouring K of one row; x is stored
// in the same order), the next segment's loads in flight during this one's products. Codes become exact fp16
// (int4: -8..7; NVFP4: E2M1 x E4M3, six significant bits); the int4 group scale multiplies the segment's fp32 sum.
//
// x' enters as fp16 with one power of two per (token, segment) that brings the segment's largest finite value into
// [2^14, 2^15): 16-bit inputs stay exact down to 2^-29 of that value (2^-38 absolute), rotated ones are rounded to
// fp16's 11 bits, and the factor is taken out of the fp32 sum, so no range is lost for either type. With few
// (token, segment) pairs every CTA builds this operand itself in shared memory; with more, one kernel builds it
// once in the workspace and the product kernel, launched behind it as a programmatic dependent, starts its weight
// loads meanwhile.
#include "kernels.cuh"
#include "ops.cuh"
#include "tmap.cuh"

namespace flint {

namespace {

constexpr int kQ4Threads = 512;
constexpr int kQ4Warps = kQ4Threads / 32;
// (token, segment) pairs up to which each CTA builds the operand itself (8 per warp)
constexpr int kQ4Inline = 128;
constexpr size_t kQ4InlineBytes = 150 * 1024;    // beside at most 64 KB of partial sums

// The operand of one (token tile of 8, segment): [i 0..3][lane][8 halves], lane = 4 (token % 8) + q holding
// K = 32 q + 8 i .. + 7 of the segment in the order of the decoded pairs, and the eight inverse factors.
constexpr int kTileBytes = 2048;

__host__ __device__ inline size_t q4_operand_bytes(int tiles, int segs) {
  return static_cast<size_t>(tiles) * segs * (kTileBytes + 32);
}

// One (token, segment) by one warp. img: the operand of (tile 0, segment 0), indexed [segment][tile].
template <int FMT, int TYPE>
__device__ __forceinline__ void q4_operand(const Q4Params& p, int t, int seg, int tile, int tiles, uint8_t* img, float* fac) {
  const int lane = threadIdx.x & 31;
  const int k = seg * 128 + 4 * lane;
  float v[4] = {0.f, 0.f, 0.f, 0.f};
  if (k < p.K) {                                 // K is a multiple of 16: four neighbours are in or out together
    const uint2 r = __ldg(reinterpret_cast<const uint2*>(p.x + t * p.ldx + k));
    const float2 a = pair_to_f32<TYPE>(r.x), b = pair_to_f32<TYPE>(r.y);
    v[0] = a.x, v[1] = a.y, v[2] = b.x, v[3] = b.y;
  }
  if (FMT == kInt4 && p.rotated) fwht128_warp(v);
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = __float_as_uint(v[j]) & 0x7FFFFFFFu;
    if (a < 0x7F800000u) m = max(m, a);          // finite ones only: infinities and NaN pass through as they are
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  const int e = min(max(static_cast<int>(m >> 23), 15), 254);      // biased exponent of the largest value
  const float f = m ? __uint_as_float(static_cast<uint32_t>(268 - e) << 23) : 1.f;     // 2^(141 - e)
  const float inv = m ? __uint_as_float(static_cast<uint32_t>(e - 14) << 23) : 1.f;
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] *= f;
  uint8_t* at = img + (static_cast<size_t>(seg) * tiles + tile) * kTileBytes +
                (((lane >> 1) & 3) * 32 + (t & 7) * 4 + (lane >> 3)) * 16 + 8 * (lane & 1);
  uint2 u;
  if constexpr (FMT == kInt4) {                  // 8-block order 0,4,1,5,2,6,3,7: see int4x8_to_half2x4
    const bool odd = lane & 1;
    const float r0 = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[0] : v[2], 1);
    const float r1 = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[1] : v[3], 1);
    u = odd ? make_uint2(pack_half2(r0, v[2]), pack_half2(r1, v[3])) : make_uint2(pack_half2(v[0], r0), pack_half2(v[1], r1));
  } else {
    u = make_uint2(pack_half2(v[0], v[1]), pack_half2(v[2], v[3]));
  }
  *reinterpret_cast<uint2*>(at) = u;
  if (lane == 0) fac[(static_cast<size_t>(seg) * tiles + tile) * 8 + (t & 7)] = inv;
}

template <int FMT, int TYPE>
__global__ void __launch_bounds__(256) q4_operand_kernel(const __grid_constant__ Q4Params p) {
  pdl_trigger();                                 // the product kernel waits for this one before it reads the operand
  const int segs = (p.K + 127) / 128, tiles = (p.T + 7) / 8;
  uint8_t* img = static_cast<uint8_t*>(p.workspace);
  float* fac = reinterpret_cast<float*>(img + static_cast<size_t>(tiles) * segs * kTileBytes);
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < static_cast<long long>(p.T) * segs;
       i += static_cast<long long>(gridDim.x) * 8) {
    const int t = static_cast<int>(i / segs), seg = static_cast<int>(i - static_cast<long long>(t) * segs);
    q4_operand<FMT, TYPE>(p, t, seg, t >> 3, tiles, img, fac);
  }
}

// Rows g and g + 8 of a block: this lane's 16 bytes of codes and its scales.
struct Q4Frag {
  uint4 c[2];
  uint32_t s[2];
};

// n[h]: the lane's two rows, behind the row `base` points at.
template <int FMT, bool WIDE>
__device__ __forceinline__ void q4_load(const Q4Params& p, const uint8_t* codes, const uint8_t* scales, const int (&n)[2],
                                        int seg, Q4Frag& f) {
  const int q = threadIdx.x & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = seg * 128 + 32 * q;
    const uint8_t* c = codes + static_cast<uint32_t>(n[h]) * static_cast<uint32_t>(p.K >> 1) + (k >> 1);
    if constexpr (FMT == kInt4) {
      f.c[h] = ld_stream_v4(c);
      f.s[h] = __ldg(reinterpret_cast<const uint16_t*>(scales) + static_cast<uint32_t>(n[h]) * static_cast<uint32_t>(p.K >> 7) + seg);
    } else {
      const uint8_t* s = scales + static_cast<uint32_t>(n[h]) * static_cast<uint32_t>(p.K >> 4) + (k >> 4);
      f.c[h] = make_uint4(0, 0, 0, 0);
      f.s[h] = 0;
      if constexpr (WIDE) {                      // K a multiple of 32: codes in 16 bytes, both scales in one load
        if (k < p.K) {
          f.c[h] = ld_stream_v4(c);
          f.s[h] = __ldg(reinterpret_cast<const uint16_t*>(s));
        }
      } else {
        if (k < p.K) {
          const uint2 a = __ldg(reinterpret_cast<const uint2*>(c));
          f.c[h].x = a.x, f.c[h].y = a.y;
          f.s[h] = __ldg(s);
        }
        if (k + 16 < p.K) {
          const uint2 a = __ldg(reinterpret_cast<const uint2*>(c + 8));
          f.c[h].z = a.x, f.c[h].w = a.y;
          f.s[h] |= static_cast<uint32_t>(__ldg(s + 1)) << 8;
        }
      }
    }
  }
}

// The 32 codes of each of the two rows as fp16 pairs: a[w][j] of row h in d[h][4 w + j].
template <int FMT>
__device__ __forceinline__ void q4_decode(const Q4Frag& f, uint32_t (&d)[2][16]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t w[4] = {f.c[h].x, f.c[h].y, f.c[h].z, f.c[h].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (FMT == kInt4) {
        uint32_t pr[4];
        int4x8_to_half2x4(w[i], pr);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[h][4 * i + j] = pr[j];
      } else {
        const uint32_t s = e4m3_to_half_bits((f.s[h] >> (8 * (i >> 1))) & 0xFFu);
        const uint32_t s2 = s | (s << 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) d[h][4 * i + j] = hmul2_u32(e2m1x2_to_half2(w[i] >> (8 * j)), s2);
      }
    }
  }
}

// NT token tiles of 8 and RB blocks of 16 rows at a time; kw_n warps split K, kQ4Warps / kw_n of such teams take
// different rows.
template <int FMT, int TYPE, int NT, int RB, bool WIDE, bool INLINE>
__global__ void __launch_bounds__(kQ4Threads, 1) q4_linear_kernel(const __grid_constant__ Q4Params p, int kw_n) {
  extern __shared__ uint8_t sm[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int segs = (p.K + 127) / 128, kw = warp % kw_n, team = warp / kw_n, teams = kQ4Warps / kw_n;
  const int t0 = blockIdx.y * 8 * NT, tiles_all = INLINE ? NT : (p.T + 7) / 8;
  const int ntile = min(NT, (p.T - t0 + 7) / 8);
  float4* red = reinterpret_cast<float4*>(sm);   // [warps][RB][NT][32]
  const uint8_t* img;
  if constexpr (INLINE) img = sm + kQ4Warps * RB * NT * 512;
  else img = static_cast<const uint8_t*>(p.workspace);
  const float* fac = reinterpret_cast<const float*>(img + static_cast<size_t>(tiles_all) * segs * kTileBytes);

  // the CTA's rows [lo, lo + rows) in blocks of at most 16 and nearly equal size, a multiple of RB per team; lanes
  // behind the end of a block repeat its last row (the same sectors), their results are not used
  const int lo = static_cast<int>(static_cast<long long>(p.N) * blockIdx.x / gridDim.x);
  const int rows = static_cast<int>(static_cast<long long>(p.N) * (blockIdx.x + 1) / gridDim.x) - lo;
  const int round = teams * RB, blocks = ((rows + 15) / 16 + round - 1) / round * round;
  const int per = rows / blocks, more = rows % blocks;              // blocks of per + 1 rows, then of per
  auto block_row = [&](int b) { return b * per + min(b, more); };
  const uint8_t* codes = p.codes + static_cast<size_t>(lo) * (p.K >> 1);
  const uint8_t* scales = p.scales + static_cast<size_t>(lo) * (FMT == kInt4 ? p.K >> 6 : p.K >> 4);

  int n[RB][2];
  auto rows_of = [&](int b0) {
#pragma unroll
    for (int r = 0; r < RB; ++r) {
      const int first = block_row(b0 + r), last = max(block_row(b0 + r + 1) - 1, 0);
      n[r][0] = min(first + g, last);
      n[r][1] = min(first + g + 8, last);
    }
  };
  Q4Frag f[RB];
  rows_of(team * RB);
  if (kw < segs) {
#pragma unroll
    for (int r = 0; r < RB; ++r) q4_load<FMT, WIDE>(p, codes, scales, n[r], kw, f[r]);
  }
  if constexpr (INLINE) {
    for (int i = warp; i < p.T * segs; i += kQ4Warps) {       // one token chunk: t0 is 0
      const int t = i / segs, seg = i - t * segs;
      q4_operand<FMT, TYPE>(p, t, seg, t >> 3, NT, const_cast<uint8_t*>(img), const_cast<float*>(fac));
    }
    __syncthreads();
  } else {
    pdl_wait();
  }
  const float ts = p.tscale ? __ldg(p.tscale) : 1.f;

  for (int b0 = 0; b0 < blocks; b0 += round) {
    const int b = b0 + team * RB;
    if (kw < segs) {
      float acc[RB][NT][4];
#pragma unroll
      for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[r][t][j] = 0.f;
      for (int seg = kw; seg < segs; seg += kw_n) {
        const size_t tile0 = static_cast<size_t>(seg) * tiles_all + (INLINE ? 0 : (t0 >> 3));
        const bool same = seg + kw_n < segs;     // the next step is of the same rows
        const int next = same ? seg + kw_n : kw;
        if (!same && b0 + round < blocks) rows_of(b + round);
#pragma unroll
        for (int r = 0; r < RB; ++r) {
          uint32_t a[2][16];
          q4_decode<FMT>(f[r], a);
          const float s0 = FMT == kInt4 ? bf16_bits_to_f32(static_cast<uint16_t>(f[r].s[0])) : 1.f;
          const float s1 = FMT == kInt4 ? bf16_bits_to_f32(static_cast<uint16_t>(f[r].s[1])) : 1.f;
          if (same || b0 + round < blocks) q4_load<FMT, WIDE>(p, codes, scales, n[r], next, f[r]);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            if (NT == 1 || t < ntile) {
              const uint4* xb = reinterpret_cast<const uint4*>(img + (tile0 + t) * kTileBytes) + lane;
              float d[4] = {0.f, 0.f, 0.f, 0.f}, e[4] = {0.f, 0.f, 0.f, 0.f};      // two chains
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const uint4 x = xb[32 * i];
                const uint32_t m0[4] = {a[0][4 * i], a[1][4 * i], a[0][4 * i + 1], a[1][4 * i + 1]};
                const uint32_t m1[4] = {a[0][4 * i + 2], a[1][4 * i + 2], a[0][4 * i + 3], a[1][4 * i + 3]};
                mma_f16_16816(d, m0, x.x, x.y);
                mma_f16_16816(e, m1, x.z, x.w);
              }
              const float2 fx = *reinterpret_cast<const float2*>(fac + (tile0 + t) * 8 + 2 * q);
              acc[r][t][0] = fmaf(d[0] + e[0], s0 * fx.x, acc[r][t][0]);
              acc[r][t][1] = fmaf(d[1] + e[1], s0 * fx.y, acc[r][t][1]);
              acc[r][t][2] = fmaf(d[2] + e[2], s1 * fx.x, acc[r][t][2]);
              acc[r][t][3] = fmaf(d[3] + e[3], s1 * fx.y, acc[r][t][3]);
            }
          }
        }
      }
#pragma unroll
      for (int r = 0; r < RB; ++r)
#pragma unroll
        for (int t = 0; t < NT; ++t)
          red[((warp * RB + r) * NT + t) * 32 + lane] = make_float4(acc[r][t][0], acc[r][t][1], acc[r][t][2], acc[r][t][3]);
    }
    __syncthreads();
    // add the team's partial sums in warp order
    const float* rf = reinterpret_cast<const float*>(red);
    const int parts = min(kw_n, segs);
    for (int o = threadIdx.x; o < teams * RB * NT * 128; o += kQ4Threads) {
      const int row = o & 15, tok = (o >> 4) % (8 * NT), r = (o / (128 * NT)) % RB, tm = o / (128 * NT * RB);
      const int blk = b0 + tm * RB + r, m = block_row(blk) + row;
      if (t0 + tok >= p.T || m >= block_row(blk + 1)) continue;
      const int at = (((tm * kw_n * RB + r) * NT + (tok >> 3)) * 32 + (row & 7) * 4 + ((tok & 7) >> 1)) * 4 +
                     (row >> 3) * 2 + (tok & 1);
      float v = 0.f;
      for (int w = 0; w < parts; ++w) v += rf[at + w * RB * NT * 128];
      p.y[static_cast<long long>(t0 + tok) * p.ldy + lo + m] = from_f32<TYPE>(v * ts);
    }
    __syncthreads();
  }
}

template <int FMT, int TYPE, int NT, int RB, bool WIDE, bool INLINE>
cudaError_t launch_rows(const Q4Params& p, int dev, int sms, int kw, cudaStream_t s) {
  const int segs = (p.K + 127) / 128;
  const int smem = kQ4Warps * RB * NT * 512 + (INLINE ? static_cast<int>(q4_operand_bytes(NT, segs)) : 0);
  cudaError_t e = allow_smem_once<q4_linear_kernel<FMT, TYPE, NT, RB, WIDE, INLINE>>(dev, 227 * 1024);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(p.N < sms ? p.N : sms, (p.T + 8 * NT - 1) / (8 * NT));
  cfg.blockDim = dim3(kQ4Threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = INLINE ? 0 : 1;
  return cudaLaunchKernelEx(&cfg, q4_linear_kernel<FMT, TYPE, NT, RB, WIDE, INLINE>, p, kw);
}

// Blocks of rows at a time: as many as a team has, so that it keeps that many 1 KB loads in flight per warp.
template <int FMT, int TYPE, int NT, int RBMAX, bool WIDE, bool INLINE>
cudaError_t launch_q4(const Q4Params& p, int dev, int sms, cudaStream_t s) {
  const int segs = (p.K + 127) / 128;
  int kw = 1;
  while (kw < segs && kw < kQ4Warps) kw *= 2;
  const int blocks = ((p.N + sms - 1) / sms + 15) / 16, teams = kQ4Warps / kw;
  if (blocks <= teams) return launch_rows<FMT, TYPE, NT, 1, WIDE, INLINE>(p, dev, sms, kw, s);
  if (RBMAX == 2 || blocks <= 2 * teams) return launch_rows<FMT, TYPE, NT, 2, WIDE, INLINE>(p, dev, sms, kw, s);
  return launch_rows<FMT, TYPE, NT, RBMAX, WIDE, INLINE>(p, dev, sms, kw, s);
}

template <int FMT, int TYPE, bool WIDE>
cudaError_t launch_tokens(const Q4Params& p, cudaStream_t s) {
  int dev, sms;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  const int segs = (p.K + 127) / 128;
  if (q4_workspace_bytes(p.K, p.T) == 0)
    return p.T <= 8 ? launch_q4<FMT, TYPE, 1, 4, WIDE, true>(p, dev, sms, s) : launch_q4<FMT, TYPE, 4, 2, WIDE, true>(p, dev, sms, s);
  const long long pairs = static_cast<long long>(p.T) * segs, ctas = (pairs + 7) / 8;
  q4_operand_kernel<FMT, TYPE><<<static_cast<int>(ctas < 8 * sms ? ctas : 8 * sms), 256, 0, s>>>(p);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  if (p.T <= 8) return launch_q4<FMT, TYPE, 1, 4, WIDE, false>(p, dev, sms, s);
  if (p.T <= 16) return launch_q4<FMT, TYPE, 2, 2, WIDE, false>(p, dev, sms, s);
  return launch_q4<FMT, TYPE, 4, 2, WIDE, false>(p, dev, sms, s);
}

template <int FMT, bool WIDE>
cudaError_t launch_type(const Q4Params& p, cudaStream_t s) {
  return p.type == kTBf16 ? launch_tokens<FMT, kTBf16, WIDE>(p, s) : launch_tokens<FMT, kTF16, WIDE>(p, s);
}

}  // namespace

size_t q4_workspace_bytes(int K, int T) {
  const int segs = (K + 127) / 128;
  if (T <= 32 && T * segs <= kQ4Inline && q4_operand_bytes(T <= 8 ? 1 : 4, segs) <= kQ4InlineBytes) return 0;
  return q4_operand_bytes((T + 7) / 8, segs);
}

cudaError_t launch_q4_linear(const Q4Params& p, cudaStream_t s) {
  if (p.fmt == kInt4) return launch_type<kInt4, true>(p, s);
  // 16-byte rows of codes and 2-byte aligned scales where the widths and the pointers allow
  const bool wide = p.K % 32 == 0 && (reinterpret_cast<uintptr_t>(p.scales) & 1u) == 0;
  return wide ? launch_type<kNvfp4, true>(p, s) : launch_type<kNvfp4, false>(p, s);
}

}  // namespace flint
