// Around the products grouped by expert: the expert-major permutation of (token, slot) pairs and the weighted
// combination of the experts' rows (flint_expert_permute, flint_expert_combine). Times are of calls in a CUDA graph on
// rotating inputs, of which up to 126 MB are still in L2.
#include <cooperative_groups.h>

#include "kernels.cuh"
#include "ops.cuh"
#include "tmap.cuh"

namespace flint {

namespace cg = cooperative_groups;

namespace {

// ---------------------------------------------------------------------------------------------
// Permutation: a counting sort that keeps pair order, in one launch of one cluster. Warp g of the cluster owns
// the pairs [g wlen, (g+1) wlen). It counts its pairs per expert in its own row of shared memory (counts do not
// depend on the order of the adds); the exclusive scans over the warps of a CTA, the CTAs of the cluster (read
// through distributed shared memory) and the experts then give each (warp, expert) its first position, and the
// warp hands out positions 32 pairs at a time by rank among equal ids (match.any). Deterministic throughout.
constexpr int kPermMaxThreads = 1024;
constexpr int kPermMaxE = 1024;                  // one per thread in the scan over the experts

__global__ void __launch_bounds__(kPermMaxThreads) expert_permute_kernel(const int* __restrict__ ids, int P, int E,
                                                                         int wlen, int* __restrict__ offsets,
                                                                         int* __restrict__ perm, int* __restrict__ inv) {
  extern __shared__ int sm_perm[];
  __shared__ int wtot[32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
  int* tot = sm_perm;                            // [E] this CTA's pairs per expert
  int* first = tot + E;                          // [E + 1] first position of this CTA's pairs; [E] = kept pairs
  int* cnt = first + E + 1;                      // [nw][E]
  cg::cluster_group cl = cg::this_cluster();
  const int rank = static_cast<int>(cl.block_rank()), ncta = static_cast<int>(cl.num_blocks());

  for (int i = threadIdx.x; i < nw * E; i += blockDim.x) cnt[i] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  const long long lo_ll = static_cast<long long>(rank * nw + warp) * wlen;
  const int lo = static_cast<int>(min(lo_ll, static_cast<long long>(P)));
  const int hi = static_cast<int>(min(lo_ll + wlen, static_cast<long long>(P)));
  int* mine = cnt + warp * E;
  for (int i0 = lo; i0 < hi; i0 += 128) {
    int v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = i0 + 32 * u + lane < hi ? __ldg(ids + i0 + 32 * u + lane) : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (v[u] >= 0 && v[u] < E) atomicAdd(mine + v[u], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    int run = 0;
#pragma unroll 8
    for (int w = 0; w < nw; ++w) {
      const int c = cnt[w * E + e];
      cnt[w * E + e] = run;
      run += c;
    }
    tot[e] = run;
  }
  cl.sync();
  // per expert: the cluster's pairs, and those of the CTAs before this one; then the exclusive scan over the
  // experts, blockDim of them at a time
  int base = 0;
  for (int e0 = 0; e0 < E; e0 += blockDim.x) {
    const int e = e0 + threadIdx.x;
    int all = 0, before = 0;
    if (e < E)
      for (int c = 0; c < ncta; ++c) {
        const int v = cl.map_shared_rank(tot, c)[e];
        if (c < rank) before += v;
        all += v;
      }
    int incl = all;
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, m);
      if (lane >= m) incl += o;
    }
    if (lane == 31) wtot[warp] = incl;
    __syncthreads();
    int off = base + incl - all, sum = 0;
    for (int w = 0; w < nw; ++w) {
      if (w < warp) off += wtot[w];
      sum += wtot[w];
    }
    if (e < E) {
      first[e] = off + before;
      if (rank == 0) offsets[e] = off;
    }
    base += sum;
    __syncthreads();
  }
  if (threadIdx.x == 0) {
    first[E] = base;
    if (rank == 0) offsets[E] = base;
  }
  cl.sync();                                     // nobody reads another CTA's memory behind this
  for (int i0 = lo; i0 < hi; i0 += 128) {
    int v[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) v[u] = i0 + 32 * u + lane < hi ? __ldg(ids + i0 + 32 * u + lane) : -1;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + 32 * u + lane;
      const int e = v[u] >= 0 && v[u] < E ? v[u] : -1;
      const unsigned peers = __match_any_sync(0xFFFFFFFFu, e);
      const int r = __popc(peers & ((1u << lane) - 1u));
      int pos = -1;
      if (e >= 0) pos = first[e] + mine[e] + r;
      __syncwarp();
      if (e >= 0 && r == 0) mine[e] += __popc(peers);
      __syncwarp();
      if (i < hi) {
        inv[i] = pos;
        if (pos >= 0) perm[pos] = i;
      }
    }
  }
  for (long long i = static_cast<long long>(base) + rank * blockDim.x + threadIdx.x; i < P;
       i += static_cast<long long>(ncta) * blockDim.x)
    perm[i] = -1;
}

// ---------------------------------------------------------------------------------------------
// Combination: y[t] = scale * sum_k w[t][k] o[inv[t][k]] + addend[t]. HBM-bound: every kept row of o is read
// once (8192 tokens of six rows of 2048: 215 MB in 40.7 us, 5.3 TB/s). A thread owns 8 columns (16-byte accesses) or one
// (any alignment), and issues the loads of 8 slots before their sum, which runs in slot order. Four CTAs per SM: three 47.7
// us, five 41.6.
template <int TYPE, bool VEC>
__global__ void __launch_bounds__(256, 4) expert_combine_kernel(const __grid_constant__ CombineParams p) {
  constexpr int kCols = VEC ? 8 : 1;
  pdl_wait();
  pdl_trigger();
  const long long t = blockIdx.x;
  const int c = (blockIdx.y * blockDim.x + threadIdx.x) * kCols;
  if (c >= p.H) return;
  float acc[kCols];
#pragma unroll
  for (int j = 0; j < kCols; ++j) acc[j] = 0.f;
  for (int k0 = 0; k0 < p.top_k; k0 += 8) {
    int row[8];
    float wk[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const bool in = k0 + k < p.top_k;
      row[k] = in ? __ldg(p.inv + t * p.top_k + k0 + k) : -1;
      wk[k] = in ? __ldg(p.w + t * p.top_k + k0 + k) : 0.f;
      if (row[k] >= p.P) row[k] = -1;
    }
    if constexpr (VEC) {
      uint4 v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (row[k] >= 0) v[k] = __ldg(reinterpret_cast<const uint4*>(p.o + row[k] * p.ldo + c));
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (row[k] < 0) continue;
        const uint32_t w[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = pair_to_f32<TYPE>(w[j]);
          acc[2 * j] = fmaf(wk[k], f.x, acc[2 * j]);
          acc[2 * j + 1] = fmaf(wk[k], f.y, acc[2 * j + 1]);
        }
      }
    } else {
      uint16_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (row[k] >= 0) v[k] = __ldg(p.o + row[k] * p.ldo + c);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (row[k] >= 0) acc[0] = fmaf(wk[k], to_f32<TYPE>(v[k]), acc[0]);
    }
  }
  if constexpr (VEC) {
    float a[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (p.addend) {                              // may be y itself: an ordinary load
      const uint4 r = *reinterpret_cast<const uint4*>(p.addend + t * p.lda + c);
      const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float2 f = pair_to_f32<TYPE>(w[j]);
        a[2 * j] = f.x;
        a[2 * j + 1] = f.y;
      }
    }
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      o[j] = pair_from_f32<TYPE>(fmaf(p.scale, acc[2 * j], a[2 * j]), fmaf(p.scale, acc[2 * j + 1], a[2 * j + 1]));
    *reinterpret_cast<uint4*>(p.y + t * p.ldy + c) = make_uint4(o[0], o[1], o[2], o[3]);
  } else {
    const float a = p.addend ? to_f32<TYPE>(p.addend[t * p.lda + c]) : 0.f;
    p.y[t * p.ldy + c] = from_f32<TYPE>(fmaf(p.scale, acc[0], a));
  }
}

// Size of the permutation's cluster: 16 where the device can hold such a one, else the portable 8. More CTAs
// share the scattered stores: 131072 pairs over 1000 experts 18.0 us with 16, 25.6 with 8, 152 with one.
int perm_ctas(int dev) {
  static std::atomic<int> known[kMaxDev];
  int n = known[dev].load(std::memory_order_relaxed);
  if (n) return n;
  n = 8;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(kPermMaxThreads);
  cfg.dynamicSmemBytes = 4 * (2 * kPermMaxE + 1 + kPermMaxThreads / 32 * kPermMaxE);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 16;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int fits = 0;
  if (cudaFuncSetAttribute(expert_permute_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
      cudaOccupancyMaxActiveClusters(&fits, expert_permute_kernel, &cfg) == cudaSuccess && fits > 0)
    n = 16;
  else
    (void)cudaGetLastError();
  known[dev].store(n, std::memory_order_relaxed);
  return n;
}

template <int TYPE>
cudaError_t launch_combine_type(const CombineParams& p, cudaStream_t s) {
  auto ok = [](const void* q, long long ld) {
    return !q || ((reinterpret_cast<uintptr_t>(q) & 15u) == 0 && ld % 8 == 0);
  };
  const bool vec = p.H % 8 == 0 && ok(p.o, p.ldo) && ok(p.addend, p.lda) && ok(p.y, p.ldy);
  const int units = vec ? p.H / 8 : p.H;
  const int threads = units >= 256 ? 256 : (units + 31) / 32 * 32;
  const dim3 grid(p.T, (units + threads - 1) / threads);
  return vec ? launch_op(expert_combine_kernel<TYPE, true>, grid, threads, 0, s, p)
             : launch_op(expert_combine_kernel<TYPE, false>, grid, threads, 0, s, p);
}

}  // namespace

cudaError_t launch_expert_permute(const int* ids, int P, int E, int* offsets, int* perm, int* inv, cudaStream_t s) {
  int dev, sms;
  cudaError_t err = current_device_sms(&dev, &sms);
  if (err != cudaSuccess) return err;
  constexpr int kSmem = 4 * (2 * kPermMaxE + 1 + kPermMaxThreads / 32 * kPermMaxE);
  if ((err = allow_smem_once<expert_permute_kernel>(dev, kSmem)) != cudaSuccess) return err;
  // one CTA or a cluster: 1200 pairs 5.6 us against 5.2, 4000 pairs 8.4 against 5.2; 30 pairs 3.3 us by one
  const int ncta = P <= 1024 ? 1 : perm_ctas(dev);
  int threads = ((P + ncta - 1) / ncta + 31) / 32 * 32;
  threads = threads < 256 ? 256 : threads > kPermMaxThreads ? kPermMaxThreads : threads;
  const int warps = ncta * (threads / 32);
  const int wlen = ((P + warps - 1) / warps + 31) / 32 * 32;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(ncta);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = 4 * (2 * E + 1 + threads / 32 * E);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ncta;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, expert_permute_kernel, ids, P, E, wlen, offsets, perm, inv);
}

cudaError_t launch_expert_combine(const CombineParams& p, cudaStream_t s) {
  return p.type == kTBf16 ? launch_combine_type<kTBf16>(p, s) : launch_combine_type<kTF16>(p, s);
}

}  // namespace flint
