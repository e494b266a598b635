// Products grouped by expert with 16-bit weights and ragged sizes (flint_grouped_linear).
#include "kernels.cuh"
#include "ops.cuh"

namespace flint {

namespace {

__device__ __forceinline__ int clamp_row(int v, int n) { return v < 0 ? 0 : v > n ? n : v; }

// The group that holds row p: the last e whose (clamped) offset is at or before p and whose end is behind it;
// -1 when none does.
__device__ __forceinline__ int group_of(const int* offsets, int E, int P, int p) {
  for (int e = 0; e < E; ++e)
    if (clamp_row(offsets[e], P) <= p && p < clamp_row(offsets[e + 1], P)) return e;
  return -1;
}

template <int TYPE>
__global__ void __launch_bounds__(256) grouped_rows_kernel(const __grid_constant__ GroupedParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nout = p.act ? p.N / 2 : p.N;
  __shared__ int group;
  for (int row = blockIdx.y; row < p.P; row += gridDim.y) {
    __syncthreads();
    if (threadIdx.x == 0) group = group_of(p.offsets, p.E, p.P, row);
    __syncthreads();
    const int e = group, n = blockIdx.x * 8 + warp;
    if (e < 0 || n >= nout) continue;
    const int r = p.row_of ? min(max(p.row_of[row] / p.row_div, 0), p.x_rows - 1) : row;
    const uint16_t* x = p.x + r * p.ldx;
    const uint16_t* w = p.w + (static_cast<size_t>(e) * p.N + n) * p.K;
    const uint16_t* u = w + static_cast<size_t>(nout) * p.K;
    float a = 0.f, b = 0.f;
    for (int k = lane; k < p.K; k += 32) {
      const float xv = to_f32<TYPE>(x[k]);
      a = fmaf(to_f32<TYPE>(w[k]), xv, a);
      if (p.act) b = fmaf(to_f32<TYPE>(u[k]), xv, b);
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
      a += __shfl_xor_sync(0xFFFFFFFFu, a, m);
      b += __shfl_xor_sync(0xFFFFFFFFu, b, m);
    }
    if (lane == 0) p.y[row * p.ldy + n] = from_f32<TYPE>(p.act ? silu(a) * b : a);
  }
}

}  // namespace

cudaError_t launch_grouped_linear(const GroupedParams& p, cudaStream_t s) {
  const int nout = p.act ? p.N / 2 : p.N;
  const dim3 grid((nout + 7) / 8, p.P < 65535 ? p.P : 65535);
  if (p.type == kTBf16) grouped_rows_kernel<kTBf16><<<grid, 256, 0, s>>>(p);
  else grouped_rows_kernel<kTF16><<<grid, 256, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace flint
