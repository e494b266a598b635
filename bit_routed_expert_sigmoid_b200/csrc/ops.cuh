// Kernel launchers of the standalone operators (internal interface between ops_api.cu and the device code).
#pragma once

#include <cuda.h>

#include "common.cuh"

namespace flint {

enum OpType : int { kTBf16 = 0, kTF16 = 1, kTF32 = 2 };

struct Q4Params {
  int fmt, N, K, rotated;
  const uint8_t* codes;
  const uint8_t* scales;
  const float* tscale;
  const uint16_t* x;
  long long ldx;
  int T, type;
  uint16_t* y;
  long long ldy;
  void* workspace;                               // q4_workspace_bytes(K, T), 256-byte aligned
};
size_t q4_workspace_bytes(int K, int T);
cudaError_t launch_q4_linear(const Q4Params& p, cudaStream_t s);
cudaError_t launch_q4_mma(const Q4Params& p, cudaStream_t s);         // T > 8

struct GroupedParams {
  int E, N, K, act, type;
  const uint16_t* w;
  const uint16_t* x;
  long long ldx;
  int x_rows;
  const int* row_of;
  int row_div;
  const int* offsets;
  int P;
  uint16_t* y;
  long long ldy;
};
cudaError_t launch_grouped_linear(const GroupedParams& p, cudaStream_t s);
cudaError_t read_ops_error(unsigned* out);       // of the current device; waits for it, clears the words
cudaError_t read_q4_error(unsigned* out);
cudaError_t read_q4_mma_error(unsigned* out);

cudaError_t launch_expert_permute(const int* ids, int P, int E, int* offsets, int* perm, int* inv, cudaStream_t s);

struct CombineParams {
  const uint16_t* o;
  long long ldo;
  int P;
  const int* inv;
  const float* w;
  int T, top_k, H;
  float scale;
  const uint16_t* addend;
  long long lda;
  int type;
  uint16_t* y;
  long long ldy;
};
cudaError_t launch_expert_combine(const CombineParams& p, cudaStream_t s);

struct NormParams {
  const void* x;
  void* x_out;
  const uint16_t* y;
  const uint16_t* gate;
  const void* post_w;
  const void* pre_w;
  uint16_t* z;
  long long ldx, ldxo, ldy, ldg, ldz;
  int T, H, type, res_f32, w_f32, post_norm, gate_act;
  float res_scale, branch_scale, eps;
};
cudaError_t launch_block_norm(const NormParams& p, cudaStream_t s);

__device__ __forceinline__ void tma_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
          smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ void tma_3d_hint(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar,
                                            uint64_t pol) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%2, %3, %4}], [%5], %6;" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar)), "l"(pol)
      : "memory");
}

// Barrier over the CTAs of the cluster (all threads of each), ordering shared-memory accesses, remote ones too.
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Stores to the same place of CTA `rank`'s shared memory.
__device__ __forceinline__ void st_cluster_f32(float* p, int rank, float v) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(a), "f"(v) : "memory");
}

// Launches an operator's kernel as a programmatic dependent of what runs before it in the stream: its launch overlaps
// that kernel's end, and it calls pdl_wait before it touches memory (then pdl_trigger, for the next one).
template <typename Kern, typename... Args>
cudaError_t launch_op(Kern kernel, dim3 grid, int threads, int smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// 16-bit element of an activation tensor as fp32, and back (one rounding, to nearest even)
template <int TYPE>
__device__ __forceinline__ float to_f32(uint16_t b) {
  if constexpr (TYPE == kTBf16) return bf16_bits_to_f32(b);
  else return __half2float(__ushort_as_half(b));
}
template <int TYPE>
__device__ __forceinline__ uint16_t from_f32(float f) {
  if constexpr (TYPE == kTBf16) return f32_to_bf16_bits(f);
  else return __half_as_ushort(__float2half_rn(f));
}
template <int TYPE>
__device__ __forceinline__ float2 pair_to_f32(uint32_t w) {
  if constexpr (TYPE == kTBf16) return make_float2(bf16lo_to_f32(w), bf16hi_to_f32(w));
  else return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <int TYPE>
__device__ __forceinline__ uint32_t pair_from_f32(float lo, float hi) {
  if constexpr (TYPE == kTBf16) return pack_bf162(lo, hi);
  else return pack_half2(lo, hi);
}

}  // namespace flint
