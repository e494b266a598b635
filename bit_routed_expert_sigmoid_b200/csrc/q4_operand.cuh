// The activation operand of the 4-bit products (q4_linear.cu, q4_mma.cu): x, or blockdiag(Hn) x, per (token,
// 128-segment) as fp16 or as 16-bit fixed point, with the power of two that was taken out.
#pragma once

#include "ops.cuh"

namespace flint {

namespace {

// How codes meet x, per 128-segment:
//   kF16Int4, kF16Nvfp4  codes become exact fp16 (int4: -8..7; NVFP4: E2M1 x E4M3, six significant bits); x is fp16
//              after one power of two per (token, segment) that brings the segment's largest finite value into [2^14,
//              2^15): 16-bit inputs stay exact down to 2^-29 of it (2^-38 absolute). The factor is taken out of the fp32 sum
//              again. Rotated bf16 inputs are rounded to fp16's 11 bits, an eighth of the output's rounding: 2.0e-4 of the
//              result's norm beside 1.66e-3.
//   kF16Pair   rotated int4 of fp16 inputs, more tokens: there the same rounding would be as large as the output's (2.9e-4
//              of the norm in all against 2.07e-4), so Hn x enters as the sum of two fp16 numbers, 22 bits, at twice the
//              MMAs: 8192 x 8192 takes 24.8 us at T = 16 and 30.1 at T = 64, where one number takes 20.3 and 24.6 (warm L2).
//              Six stages of the operand instead of three: 26.5 and 33.6. An infinity's second part is NaN.
//   kLimbs     rotated int4, few tokens: Hn x is rounded to 16-bit fixed point per (token, segment), a unit being 2^-14
//              of the power of two below the segment's largest value (rotation spreads outliers, so that is finer than
//              fp16 for all but the smallest values); its signed high and unsigned low bytes multiply the exact int8
//              16 c on the integer tensor cores. Three instructions decode eight codes instead of nine.
enum Arith : int { kF16Int4, kF16Nvfp4, kLimbs, kF16Pair };

// fp16 numbers per element of the operand
template <int AR>
constexpr int kParts = AR == kF16Pair ? 2 : 1;

// A (token, segment) is four chunks of 16 bytes for each of the four lanes q that read it, K = 32 q .. 32 q + 31. fp16:
// chunk i holds K = 32 q + 8 i .. + 7 in the order of the decoded pairs (int4 0,4,1,5,2,6,3,7; NVFP4 0,1,2,6,4,5,3,7);
// limbs: chunk 2 limb + (i >> 1) holds at 8 (i & 1) the bytes of K = 32 q + 8 i + 0, 2, 4, 6 and of + 1, 3, 5, 7.
//   kTokens  [segment][token][chunk][q], then the inverse factor, kTokenBytes each
//   kRows    [token][segment][part][q][chunk]: K-major rows; then the factors [segment][tokens rounded up to 4]
// kTokens is for up to 8 tokens (q4_linear.cu), kRows for more (q4_mma.cu).
enum OperandLayout : int { kTokens, kRows };
constexpr int kTokenBytes = 272;

__host__ __device__ inline size_t q4_rows_factors(int T, int segs, int parts) {
  return static_cast<size_t>(T) * segs * parts * 256;
}
// of the form that takes most (more than 8 tokens: two parts)
__host__ __device__ inline size_t q4_operand_bytes(int T, int segs) {
  return T <= 8 ? static_cast<size_t>(T) * segs * kTokenBytes
                : q4_rows_factors(T, segs, 2) + static_cast<size_t>((T + 3) & ~3) * segs * 4;
}

struct OperandPlace {
  uint8_t* at;                                   // of chunk 0, q = 0
  int chunk, lane;                               // bytes from a chunk to the next, and from q to the next
  float* factor;
};

template <int LAYOUT, int PARTS>
__device__ __forceinline__ OperandPlace q4_place(uint8_t* img, int t, int seg, int T, int segs) {
  OperandPlace o;
  if constexpr (LAYOUT == kTokens) {
    o.at = img + (static_cast<size_t>(seg) * T + t) * kTokenBytes;
    o.chunk = 64, o.lane = 16;
    o.factor = reinterpret_cast<float*>(o.at + 256);
  } else {
    o.at = img + (static_cast<size_t>(t) * segs + seg) * (256 * PARTS);
    o.chunk = 16, o.lane = 64;
    o.factor = reinterpret_cast<float*>(img + q4_rows_factors(T, segs, PARTS)) + static_cast<size_t>(seg) * ((T + 3) & ~3) +
               t;
  }
  return o;
}

// A warp's four elements per lane of one (token, segment).
__device__ __forceinline__ uint2 q4_fetch(const Q4Params& p, int t, int seg) {
  const int k = seg * 128 + 4 * (threadIdx.x & 31);
  // K is a multiple of 16: four neighbours are in or out together
  return k < p.K ? __ldg(reinterpret_cast<const uint2*>(p.x + t * p.ldx + k)) : make_uint2(0, 0);
}

// The operands of NP (token, segment) pairs by one warp, their dependent steps interleaved. Every lane of the warp
// computes all of them; o[j].at is null for a pair that is not to be stored.
template <int AR, int TYPE, int NP>
__device__ __forceinline__ void q4_operand(const uint2 (&raw)[NP], bool rotate, const OperandPlace (&o)[NP]) {
  const int lane = threadIdx.x & 31;
  float v[NP][4];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const float2 a = pair_to_f32<TYPE>(raw[j].x), b = pair_to_f32<TYPE>(raw[j].y);
    v[j][0] = a.x, v[j][1] = a.y, v[j][2] = b.x, v[j][3] = b.y;
  }
  float back[NP];                                // power of two taken out before the rotation
#pragma unroll
  for (int j = 0; j < NP; ++j) back[j] = 1.f;
  if (rotate) {
    // A sum of 128 bf16 values may pass fp32's range: a segment with values of 2^120 or more is rotated at 2^-8 of its size
    // (exact but for values 2^-238 times the largest). fp16 values are far below.
    if constexpr (TYPE == kTBf16) {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        const float most = fmaxf(fmaxf(fabsf(v[j][0]), fabsf(v[j][1])), fmaxf(fabsf(v[j][2]), fabsf(v[j][3])));
        if (__any_sync(0xFFFFFFFFu, most >= 0x1p120f)) {
          back[j] = 0x1p8f;
#pragma unroll
          for (int i = 0; i < 4; ++i) v[j][i] *= 0x1p-8f;
        }
      }
    }
    // the butterfly of fwht128_warp, one fused multiply-add per step
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const float a = v[j][0] + v[j][1], b = v[j][0] - v[j][1], c = v[j][2] + v[j][3], d = v[j][2] - v[j][3];
      v[j][0] = a + c, v[j][1] = b + d, v[j][2] = a - c, v[j][3] = b - d;
    }
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const float sign = (lane & m) ? -1.f : 1.f;
#pragma unroll
      for (int j = 0; j < NP; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) v[j][i] = fmaf(sign, v[j][i], __shfl_xor_sync(0xFFFFFFFFu, v[j][i], m));
    }
#pragma unroll
    for (int j = 0; j < NP; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] *= 0.08838834764831845f;             // 1 / sqrt(128)
  }
  uint32_t m[NP];
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    m[j] = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = __float_as_uint(v[j][i]) & 0x7FFFFFFFu;
      m[j] = max(m[j], AR == kLimbs || a < 0x7F800000u ? a : 0u);  // fp16: infinities and NaN pass as they are
    }
  }
#pragma unroll
  for (int j = 0; j < NP; ++j) m[j] = __reduce_max_sync(0xFFFFFFFFu, m[j]);
  const int c = (lane >> 1) & 3;
  const bool odd = lane & 1;
#pragma unroll
  for (int j = 0; j < NP; ++j) {
    const int e = min(max(static_cast<int>(m[j] >> 23), 15), 254);             // biased exponent of the largest value
    const float f = m[j] ? __uint_as_float(static_cast<uint32_t>(268 - e) << 23) : 1.f;          // 2^(141 - e)
    float inv = m[j] ? back[j] * __uint_as_float(static_cast<uint32_t>(e - 14) << 23) : 1.f;
    uint2 u, low = make_uint2(0, 0);             // low: kF16Pair's second part
    int off;
    if constexpr (AR == kLimbs) {
      uint32_t n[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) n[i] = static_cast<uint32_t>(min(__float2int_rn(v[j][i] * f), 32767));
      // bytes 0, 1: elements 0, 2; bytes 2, 3: elements 1, 3
      const uint32_t hi = __byte_perm(__byte_perm(n[0], n[2], 0x0051), __byte_perm(n[1], n[3], 0x0051), 0x5410);
      const uint32_t lo = __byte_perm(__byte_perm(n[0], n[2], 0x0040), __byte_perm(n[1], n[3], 0x0040), 0x5410);
      // the even lane of a pair writes the high limbs of the eight, the odd lane the low ones
      const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, odd ? hi : lo, 1);
      const uint32_t first = odd ? got : hi, second = odd ? lo : got;
      u = make_uint2(__byte_perm(first, second, 0x5410), __byte_perm(first, second, 0x7632));
      off = (2 * odd + (c >> 1)) * o[j].chunk + (c & 1) * 8;
      // the codes enter as 16 c; what is infinite or no number stays so, for the token's whole sum
      inv = m[j] >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : inv * 0.0625f;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j][i] *= f;
      if constexpr (AR == kF16Int4 || AR == kF16Pair) {
        auto pairs = [&](const float (&w)[4]) {
          const float r0 = __shfl_xor_sync(0xFFFFFFFFu, odd ? w[0] : w[2], 1);
          const float r1 = __shfl_xor_sync(0xFFFFFFFFu, odd ? w[1] : w[3], 1);
          return odd ? make_uint2(pack_half2(r0, w[2]), pack_half2(r1, w[3]))
                     : make_uint2(pack_half2(w[0], r0), pack_half2(w[1], r1));
        };
        u = pairs(v[j]);
        if constexpr (AR == kF16Pair) {
#pragma unroll
          for (int i = 0; i < 4; ++i) v[j][i] -= __half2float(__float2half_rn(v[j][i]));       // exact
          low = pairs(v[j]);
        }
      } else {                                   // 0,1,2,6 by the even lane of a pair, 4,5,3,7 by the odd one
        const float r = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[j][2] : v[j][3], 1);
        u = odd ? make_uint2(pack_half2(v[j][0], v[j][1]), pack_half2(r, v[j][3]))
                : make_uint2(pack_half2(v[j][0], v[j][1]), pack_half2(v[j][2], r));
        inv *= 128.f;                            // see decode_f16
      }
      off = c * o[j].chunk + 8 * odd;
    }
    if (o[j].at) {
      *reinterpret_cast<uint2*>(o[j].at + (lane >> 3) * o[j].lane + off) = u;
      if constexpr (AR == kF16Pair) *reinterpret_cast<uint2*>(o[j].at + 256 + (lane >> 3) * o[j].lane + off) = low;
      if (lane == 0) *o[j].factor = inv;
    }
  }
}

// The whole operand in the workspace, a warp per (token, segment). Launched in stream order, so that what ran before it
// (weights written by a quantiser, say) is complete when it starts; the product kernel is its programmatic dependent, may
// start as soon as it has, and has to wait for the operand only. (As a programmatic dependent itself it would have to
// wait before it lets the product kernel start: 2048 x 2048 at T = 8 took 6.9 us against 6.3.)
template <int AR, int TYPE, int LAYOUT>
__global__ void __launch_bounds__(256) q4_operand_kernel(const __grid_constant__ Q4Params p) {
  pdl_trigger();
  const int segs = (p.K + 127) / 128;
  for (long long i = static_cast<long long>(blockIdx.x) * 8 + (threadIdx.x >> 5); i < static_cast<long long>(p.T) * segs;
       i += static_cast<long long>(gridDim.x) * 8) {
    const int t = static_cast<int>(i / segs), seg = static_cast<int>(i - static_cast<long long>(t) * segs);
    const uint2 raw[1] = {q4_fetch(p, t, seg)};
    const OperandPlace o[1] = {q4_place<LAYOUT, kParts<AR>>(static_cast<uint8_t*>(p.workspace), t, seg, p.T, segs)};
    q4_operand<AR, TYPE, 1>(raw, p.rotated != 0, o);
  }
}

template <int AR, int TYPE, int LAYOUT>
cudaError_t launch_q4_operand(const Q4Params& p, int sms, cudaStream_t s) {
  const long long pairs = static_cast<long long>(p.T) * ((p.K + 127) / 128), ctas = (pairs + 7) / 8;
  const int grid = static_cast<int>(ctas < 8 * sms ? ctas : 8 * sms);
  return launch_pdl_kernel(q4_operand_kernel<AR, TYPE, LAYOUT>, grid, 256, 0, false, s, p);
}

// ---------------------------------------------------------------------------------------------

// One row's 32 codes (16 bytes) as fp16 pairs, in the operand's order; s2: the two block scales (NVFP4).
template <int AR>
__device__ __forceinline__ void decode_f16(const uint4& c, uint32_t s2, uint32_t (&d)[16]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (AR == kF16Int4) {
      uint32_t pr[4];
      int4x8_to_half2x4(w[i], pr);
#pragma unroll
      for (int j = 0; j < 4; ++j) d[4 * i + j] = pr[j];
    } else {
      // Codes 0, 1 and 4, 5 by the hardware conversion, the pairs 2, 6 and 3, 7 by moving their bits: sign to bit 15,
      // exponent and fraction to bits 11-9, which is the value times 2^-14 (subnormals included). Both kinds of work
      // then run side by side. The products with the scale times 2^-7 and 2^7 are exact and share a factor of 2^-7.
      const uint32_t h = e4m3_to_half_bits((s2 >> (8 * (i >> 1))) & 0xFFu), hh = h | (h << 16);
      const uint32_t up = hmul2_u32(hh, 0x58005800u), down = hmul2_u32(hh, 0x20002000u);       // 2^7, 2^-7
      const uint32_t u = w[i] << 4;
      d[4 * i] = hmul2_u32(e2m1x2_to_half2(w[i]), down);
      d[4 * i + 1] = hmul2_u32((u & 0x80008000u) | ((u >> 3) & 0x0E000E00u), up);
      d[4 * i + 2] = hmul2_u32(e2m1x2_to_half2(w[i] >> 16), down);
      d[4 * i + 3] = hmul2_u32((w[i] & 0x80008000u) | ((w[i] >> 3) & 0x0E000E00u), up);
    }
  }
}

}  // namespace

}  // namespace flint
