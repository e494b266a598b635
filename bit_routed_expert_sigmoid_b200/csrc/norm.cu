// The residual step around a block (flint_block_norm): post-norm of the branch, gate, residual add and the
// next block's pre-norm in one pass, every row read once and held in registers between the two reductions. Bound by HBM:
// 8192 x 4096 bf16 with a gate per element moves 336 MB in 58.0 us (5.8 TB/s); 2048 x 2048 with an fp32 residual 9.2 us
// (calls in a CUDA graph on rotating inputs, of which up to 126 MB are still in L2; flushed 68.5 and 16.4, launch included).
#include "kernels.cuh"
#include "ops.cuh"

namespace flint {

namespace {

constexpr int kNormWarps = 32;

// Sum over the CTA in a fixed order: the warp butterfly, then the warps in order.
__device__ __forceinline__ float block_sum(float v, float* wsum) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  const int warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  if ((threadIdx.x & 31) == 0) wsum[warp] = v;
  __syncthreads();
  float tot = 0.f;
  for (int w = 0; w < nw; ++w) tot += wsum[w];
  return tot;
}

// 1 / sqrt(mean + eps) over the row, from the thread's sum of squares. Values from 2^56 on may have a sum that passes
// fp32's range: all threads of the CTA then see it infinite and add the squares of 2^-80 times the values (`scaled`), at
// most 32768 of 2^96. An infinite or NaN value stays what it is.
template <bool WIDE, typename Scaled>
__device__ __forceinline__ float inv_rms(float s, int H, float eps, float* wsum, Scaled scaled) {
  const float sum = block_sum(s, wsum);
  if constexpr (WIDE) {
    if (sum > 3.402823466e38f) {
      __syncthreads();                           // wsum is written again
      return 0x1p-80f / sqrtf(block_sum(scaled(), wsum) / static_cast<float>(H) + eps * 0x1p-80f * 0x1p-80f);
    }
  }
  return 1.0f / sqrtf(sum / static_cast<float>(H) + eps);
}

// Element k (of 8 VPT) of a thread: 8 neighbours per step with 16-byte accesses, else one element per step so
// that a warp's accesses are neighbours.
template <bool VEC>
__device__ __forceinline__ int col_of(int k) {
  if constexpr (VEC) return ((k >> 3) * blockDim.x + threadIdx.x) * 8 + (k & 7);
  else return k * blockDim.x + threadIdx.x;
}

// Eight 16-bit elements as they were loaded, in pairs: converted where they are used, so that a row in flight costs
// few registers.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const uint16_t* row, int v, int H) {
  uint4 r = make_uint4(0, 0, 0, 0);
  if constexpr (VEC) {
    const int c = col_of<true>(8 * v);
    if (c < H) r = *reinterpret_cast<const uint4*>(row + c);
  } else {
    uint32_t w[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = col_of<false>(8 * v + j);
      w[j] = c < H ? row[c] : 0u;
    }
    r = make_uint4(w[0] | (w[1] << 16), w[2] | (w[3] << 16), w[4] | (w[5] << 16), w[6] | (w[7] << 16));
  }
  return r;
}

template <int TYPE>
__device__ __forceinline__ void widen8(const uint4& r, float (&out)[8]) {
  const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = pair_to_f32<TYPE>(w[j]);
    out[2 * j] = f.x;
    out[2 * j + 1] = f.y;
  }
}

template <bool VEC>
__device__ __forceinline__ void load8_f32(const float* row, int v, int H, float (&out)[8]) {
  if constexpr (VEC) {
    const int c = col_of<true>(8 * v);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f), b = a;
    if (c < H) {
      a = *reinterpret_cast<const float4*>(row + c);
      b = *reinterpret_cast<const float4*>(row + c + 4);
    }
    out[0] = a.x, out[1] = a.y, out[2] = a.z, out[3] = a.w;
    out[4] = b.x, out[5] = b.y, out[6] = b.z, out[7] = b.w;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = col_of<false>(8 * v + j);
      out[j] = c < H ? row[c] : 0.f;
    }
  }
}

template <int TYPE, bool VEC>
__device__ __forceinline__ void store8(uint16_t* row, int v, int H, const float (&in)[8]) {
  if constexpr (VEC) {
    const int c = col_of<true>(8 * v);
    if (c < H)
      *reinterpret_cast<uint4*>(row + c) =
          make_uint4(pair_from_f32<TYPE>(in[0], in[1]), pair_from_f32<TYPE>(in[2], in[3]),
                     pair_from_f32<TYPE>(in[4], in[5]), pair_from_f32<TYPE>(in[6], in[7]));
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int c = col_of<false>(8 * v + j);
      if (c < H) row[c] = from_f32<TYPE>(in[j]);
    }
  }
}

template <int TYPE, bool VEC>
__device__ __forceinline__ void load8_weight(const void* w, int w_f32, int v, int H, float (&out)[8]) {
  if (w_f32) load8_f32<VEC>(static_cast<const float*>(w), v, H, out);
  else widen8<TYPE>(load8<VEC>(static_cast<const uint16_t*>(w), v, H), out);
}

// 1 / (1 + e^-g) by the approximate base-2 exponential and reciprocal: within (1.3 |g| + 7) 2^-24 of itself. The argument's
// rounding and that of log2 e take 1.23 |g|, the exponential (2^-22) 4, the sum 1 and the reciprocal (2^-23) 2. It is 0
// where e^-g passes 2^126.
__device__ __forceinline__ float sigmoid_fast(float g) {
  float e, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(g * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + e));
  return r;
}

template <int VPT>
constexpr int kMaxThreads = VPT == 1 ? 1024 : VPT == 8 ? 512 : 256;

// VPT steps of 8 columns per thread. All of a row's loads are issued before the first reduction.
template <int TYPE, bool RES_F32, bool VEC, int VPT>
__global__ void __launch_bounds__(kMaxThreads<VPT>) block_norm_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sum_post[kNormWarps], sum_pre[kNormWarps];
  pdl_wait();
  pdl_trigger();
  const long long t = blockIdx.x;
  const int H = p.H;
  float x[VPT][8];
  uint4 xr[VPT], yr[VPT], gr[VPT];
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if constexpr (RES_F32) load8_f32<VEC>(static_cast<const float*>(p.x) + t * p.ldx, v, H, x[v]);
    else xr[v] = load8<VEC>(static_cast<const uint16_t*>(p.x) + t * p.ldx, v, H);
    if (p.y) yr[v] = load8<VEC>(p.y + t * p.ldy, v, H);
    if (p.gate) gr[v] = load8<VEC>(p.gate + t * p.ldg, v, H);
  }
  float norm = 1.f;
  if (p.post_norm) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      float b[8];
      widen8<TYPE>(yr[v], b);
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(b[j], b[j], s);
    }
    norm = inv_rms<TYPE == kTBf16>(s, H, p.eps, sum_post, [&] {   // from memory: the widened row is not kept for this
      float w = 0.f;
#pragma unroll 1
      for (int c = threadIdx.x; c < H; c += blockDim.x) {
        const float b = 0x1p-80f * to_f32<TYPE>(p.y[t * p.ldy + c]);
        w = fmaf(b, b, w);
      }
      return w;
    });
  }
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
    if constexpr (!RES_F32) widen8<TYPE>(xr[v], x[v]);
    if (p.y) {
      float b[8];
      widen8<TYPE>(yr[v], b);
      if (p.post_norm) {
#pragma unroll
        for (int j = 0; j < 8; ++j) b[j] *= norm;
        if (p.post_w) {
          float w[8];
          load8_weight<TYPE, VEC>(p.post_w, p.w_f32, v, H, w);
#pragma unroll
          for (int j = 0; j < 8; ++j) b[j] *= w[j];
        }
      }
      if (p.gate) {
        float g[8];
        widen8<TYPE>(gr[v], g);
        if (p.gate_act == 1) {
#pragma unroll
          for (int j = 0; j < 8; ++j) b[j] *= sigmoid_fast(g[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) b[j] *= g[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v][j] = fmaf(p.branch_scale, b[j], p.res_scale * x[v][j]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v][j] *= p.res_scale;
    }
  }
  if (p.x_out) {
#pragma unroll
    for (int v = 0; v < VPT; ++v) {
      if constexpr (RES_F32) {
        float* row = static_cast<float*>(p.x_out) + t * p.ldxo;
        if constexpr (VEC) {
          const int c = col_of<true>(8 * v);
          if (c < H) {
            *reinterpret_cast<float4*>(row + c) = make_float4(x[v][0], x[v][1], x[v][2], x[v][3]);
            *reinterpret_cast<float4*>(row + c + 4) = make_float4(x[v][4], x[v][5], x[v][6], x[v][7]);
          }
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int c = col_of<false>(8 * v + j);
            if (c < H) row[c] = x[v][j];
          }
        }
      } else {
        store8<TYPE, VEC>(static_cast<uint16_t*>(p.x_out) + t * p.ldxo, v, H, x[v]);
      }
    }
  }
  if (!p.z) return;
  auto squares = [&](float k) {
    float s = 0.f;
#pragma unroll
    for (int v = 0; v < VPT; ++v)
#pragma unroll
      for (int j = 0; j < 8; ++j) s = fmaf(k * x[v][j], k * x[v][j], s);       // columns behind H hold zeros
    return s;
  };
  // wide for any type: the scales of residual and branch may be large
  const float inv = inv_rms<true>(squares(1.f), H, p.eps, sum_pre, [&] { return squares(0x1p-80f); });
#pragma unroll
  for (int v = 0; v < VPT; ++v) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[v][j] *= inv;
    if (p.pre_w) {
      float w[8];
      load8_weight<TYPE, VEC>(p.pre_w, p.w_f32, v, H, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) x[v][j] *= w[j];
    }
    store8<TYPE, VEC>(p.z + t * p.ldz, v, H, x[v]);
  }
}

template <int TYPE, bool RES_F32, bool VEC>
cudaError_t launch_vpt(const NormParams& p, cudaStream_t s) {
  // Few rows: a thread per 8 columns, the shortest way through one row (4 x 2048: 2.3 us, 2.4 with two steps). Many rows:
  // 4 steps per thread, so that the reductions cost fewer warps and more loads of more rows are in flight (8192 x 4096
  // with a gate per element: 58.0 us, 63.4 with two steps, 76 with one).
  const int n8 = (p.H + 7) / 8;
  const int vpt = n8 > 1024 ? 8 : p.T >= 1024 && n8 > 256 ? 4 : 1;
  const int threads = ((n8 + vpt - 1) / vpt + 31) / 32 * 32;
  switch (vpt) {
    case 1: return launch_op(block_norm_kernel<TYPE, RES_F32, VEC, 1>, dim3(p.T), threads, 0, s, p);
    case 4: return launch_op(block_norm_kernel<TYPE, RES_F32, VEC, 4>, dim3(p.T), threads, 0, s, p);
    default: return launch_op(block_norm_kernel<TYPE, RES_F32, VEC, 8>, dim3(p.T), threads, 0, s, p);
  }
}

template <int TYPE>
cudaError_t launch_type(const NormParams& p, cudaStream_t s) {
  // 16-byte accesses where every row of every operand starts on 16 bytes
  const long long re = p.res_f32 ? 4 : 8;
  auto ok = [](const void* q, long long ld, long long e) {
    return !q || ((reinterpret_cast<uintptr_t>(q) & 15u) == 0 && ld % e == 0);
  };
  const bool vec = p.H % 8 == 0 && ok(p.x, p.ldx, re) && ok(p.x_out, p.ldxo, re) && ok(p.y, p.ldy, 8) &&
                   ok(p.gate, p.ldg, 8) && ok(p.z, p.ldz, 8) && ok(p.post_w, 0, 8) && ok(p.pre_w, 0, 8);
  if (p.res_f32) return vec ? launch_vpt<TYPE, true, true>(p, s) : launch_vpt<TYPE, true, false>(p, s);
  return vec ? launch_vpt<TYPE, false, true>(p, s) : launch_vpt<TYPE, false, false>(p, s);
}

}  // namespace

cudaError_t launch_block_norm(const NormParams& p, cudaStream_t s) {
  return p.type == kTBf16 ? launch_type<kTBf16>(p, s) : launch_type<kTF16>(p, s);
}

}  // namespace flint
