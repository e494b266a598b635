// Linear products with 4-bit weights for few tokens (flint_q4_linear).
#include "kernels.cuh"
#include "ops.cuh"

namespace flint {

namespace {

// One weight of a row: code times its group scale.
template <int FMT>
__device__ __forceinline__ float q4_weight(const uint8_t* codes, const uint8_t* scales, int k) {
  const int nib = (codes[k >> 1] >> (4 * (k & 1))) & 15;
  if constexpr (FMT == kInt4) {
    const uint16_t s = reinterpret_cast<const uint16_t*>(scales)[k >> 7];
    return static_cast<float>((nib ^ 8) - 8) * bf16_bits_to_f32(s);
  } else {
    const float v = __half2float(__ushort_as_half(static_cast<uint16_t>(e2m1x2_to_half2(nib) & 0xFFFFu)));
    return v * __half2float(__ushort_as_half(e4m3_to_half_bits(scales[k >> 4])));
  }
}

// A CTA per 8 rows and token, a warp per row; 128-segments of x (rotated when asked) by all warps in turn.
template <int FMT, int TYPE>
__global__ void __launch_bounds__(256) q4_rows_kernel(const __grid_constant__ Q4Params p) {
  __shared__ float xs[8][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int n = blockIdx.x * 8 + warp;
  const float ts = p.tscale ? *p.tscale : 1.f;
  for (long long t = blockIdx.y; t < p.T; t += gridDim.y) {
    const uint16_t* x = p.x + t * p.ldx;
    float acc = 0.f;
    for (int k0 = 0; k0 < p.K; k0 += 1024) {
      __syncthreads();
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + 128 * warp + 4 * lane + j;
        v[j] = k < p.K ? to_f32<TYPE>(x[k]) : 0.f;
      }
      if (p.rotated) fwht128_warp(v);
#pragma unroll
      for (int j = 0; j < 4; ++j) xs[warp][4 * lane + j] = v[j];
      __syncthreads();
      if (n < p.N) {
        const uint8_t* codes = p.codes + static_cast<size_t>(n) * (p.K / 2);
        const uint8_t* scales = p.scales + static_cast<size_t>(n) * (FMT == kInt4 ? p.K / 64 : p.K / 16);
        for (int k = k0 + lane; k < min(p.K, k0 + 1024); k += 32)
          acc = fmaf(q4_weight<FMT>(codes, scales, k), xs[(k - k0) >> 7][(k - k0) & 127], acc);
      }
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, m);
    if (lane == 0 && n < p.N) p.y[t * p.ldy + n] = from_f32<TYPE>(acc * ts);
  }
}

}  // namespace

cudaError_t launch_q4_linear(const Q4Params& p, cudaStream_t s) {
  const dim3 grid((p.N + 7) / 8, p.T < 65535 ? p.T : 65535);
  if (p.fmt == kInt4) {
    if (p.type == kTBf16) q4_rows_kernel<kInt4, kTBf16><<<grid, 256, 0, s>>>(p);
    else q4_rows_kernel<kInt4, kTF16><<<grid, 256, 0, s>>>(p);
  } else {
    if (p.type == kTBf16) q4_rows_kernel<kNvfp4, kTBf16><<<grid, 256, 0, s>>>(p);
    else q4_rows_kernel<kNvfp4, kTF16><<<grid, 256, 0, s>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace flint
