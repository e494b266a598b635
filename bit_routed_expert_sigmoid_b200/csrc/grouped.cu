// Products grouped by expert with 16-bit weights and ragged sizes (flint_grouped_linear):
//   y[p] = W[e] x[r(p)] for p in [offsets[e], offsets[e+1]), or silu(gate) * up of W's two halves.
//
// Two kernels. grouped_mma_kernel is a persistent tcgen05 GEMM: the weights are its M side (128 rows a tile),
// a group's rows its N side (up to NMAX a tile, padded to 16), so a group with few rows costs few columns. Both
// operands are staged in the 128-byte swizzled K-major layout: the weights, and rows that are already in expert
// order, as TMA boxes; rows taken through row_of by four warps with 16-byte cp.async, so no gathered copy of x is
// ever written (TMA's gather4 measured ~70 cycles per four 128-byte rows: 4096^3 took 602 us with it). With few
// rows per expert it is bound by streaming the weights once; with many, by the tensor cores.
// grouped_few_kernel serves decode (P <= kFewRows): see there. 256 experts, gate|up 1024 x 2048: 12288 rows 160 us, 192
// rows 91, 24 rows 21.4; one group of 4096^3 106 us (tensor cores 82). These, and all times in this file, are of calls in a
// CUDA graph, where up to 126 MB of the weights are still in L2; with L2 flushed, and the launch included, 180, 104 and 28.0
// (once through HBM 167, 87, 14.9).
#include "kernels.cuh"
#include "ops.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace flint {

__device__ unsigned g_ops_error;                 // timeout bits of bounded waits (flint_ops_error_word)

namespace {

constexpr int kGrMaxE = 1024;
constexpr int kGrThreads = 384;                  // copies: 2 warps, MMA: 1, idle: 1, epilogue: 8; and 4 more that gather
constexpr int kGrTabWarps = 8;                   // warps that build the tile table
constexpr int kGrGather = 128;
constexpr int kGrABytes = 128 * 128;             // a stage of weights: 128 rows x 64 K
constexpr int kGrSlab = 2 * 2 * 16 * 64 * 4;      // SwiGLU: two teams x (gate, up) x 16 columns x 64 rows, fp32
// Rows up to which grouped_few_kernel is taken: 24 rows over 256 experts take 21.4 us there and 26.6 by the GEMM, 30 rows
// 25.1 and 26.7, 60 rows 44 and 38. It reads a group's weights once per eight of its rows, so with more than eight rows on
// average, counted in whole eights (P / 8 > E), the GEMM is taken: 28 rows of two experts, 4096 x 4096, 24.5 us and 20.4.
// Where that leaves a second reading, it still wins for one expert (12 rows, 4096 x 4096: 15.8 and 19.8) and for small
// matrices (20 rows of two, gate|up 1024 x 2048: 7.9 and 13.3), and loses for a few large ones (20 rows of two, 4096 x
// 4096: 23.5 and 20.2).
constexpr int kFewRows = 32;

// First row and number of rows of group e; offsets clamped to [0, P].
__device__ __forceinline__ int2 group_span(const int* offsets, int e, int P) {
  const int lo = min(max(__ldg(offsets + e), 0), P), hi = min(max(__ldg(offsets + e + 1), 0), P);
  return make_int2(lo, max(hi - lo, 0));
}

__device__ __forceinline__ int source_row(const GroupedParams& p, int row) {
  if (!p.row_of) return row;
  return min(max(__ldg(p.row_of + row) / p.row_div, 0), p.x_rows - 1);
}

struct GroupedMmaParams {
  CUtensorMap tm_w, tm_x;
  GroupedParams g;
  int m_tiles;                                   // tiles of 128 weight rows per group
};

// MB: 128-row blocks of weights per tile. Two share the tile's rows, which halves what has to be brought for them: with
// one, 256-row tiles are bound by the copies (48 KB per 512 cycles of MMA), most of all where rows are gathered.
template <int NMAX, int MB>
struct GrGeom {
  static constexpr int kA = MB * kGrABytes;
  static constexpr int kB = NMAX * 128;          // a stage of rows: NMAX rows x 64 K
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = 192 * 1024 / kStage;      // 8 (64), 6 (128), 4 (256), 3 (256, two blocks)
  static constexpr int kBox = NMAX == 256 ? 128 : 64;      // rows of a TMA box of x
};

struct GrTab {
  int start[kGrMaxE + 1];                        // first tile of group e
  int off[kGrMaxE], cnt[kGrMaxE];
  int wsum[kGrTabWarps];
  int pad;
};
static_assert(sizeof(GrTab) % 8 == 0, "the barriers behind it are 64-bit");

struct GrBars {
  uint64_t full[8], empty[8], acc_full[2], acc_empty[2], done;
  uint32_t tmem;
  int abort;
};

template <int NMAX, int MB>
constexpr int gr_smem() {
  return GrGeom<NMAX, MB>::kStages * GrGeom<NMAX, MB>::kStage + static_cast<int>(sizeof(GrTab) + sizeof(GrBars)) + kGrSlab + 1024;
}
static_assert(gr_smem<64, 1>() <= 227 * 1024 && gr_smem<128, 1>() <= 227 * 1024 && gr_smem<256, 1>() <= 227 * 1024 &&
                  gr_smem<256, 2>() <= 227 * 1024,
              "shared memory");

struct GrTile {
  int e, m, row0, n;                             // group, weight tile, first row, rows (1..NMAX)
  bool once;                                     // the group's weights are read by no other tile
};

// Tiles of a group: weight tiles outermost, its chunks of rows (of equal size, a multiple of 16) innermost, so
// that neighbouring CTAs share a weight tile in L2.
template <int NMAX>
__device__ __forceinline__ GrTile gr_tile(const GrTab& tt, int E, int t) {
  int lo = 0, hi = E - 1;
  while (lo < hi) {                              // last group with start <= t that has tiles
    const int mid = (lo + hi + 1) >> 1;
    if (tt.start[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int cnt = tt.cnt[lo], nch = (cnt + NMAX - 1) / NMAX, local = t - tt.start[lo];
  const int per = ((cnt + nch - 1) / nch + 15) & ~15;
  GrTile r;
  r.e = lo;
  r.m = local / nch;
  const int c = local - r.m * nch;
  r.row0 = tt.off[lo] + c * per;
  r.n = min(per, cnt - c * per);
  r.once = nch == 1;
  return r;
}

// 16 bytes to shared memory; zeros when !in
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// Arrives at `bar` (one of the arrivals it was made for) when this thread's copies so far have landed.
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }
// Orders shared-memory writes that this thread has observed (or made) before its later tensor-core reads of them.
__device__ __forceinline__ void fence_proxy_async_shared() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// Waits until the copies of iterations [max(it - stages, 0), it) have landed, so that none is in flight when the
// CTA exits. After an abort a stage may lack its other operand and never complete: each wait then ends after 1 ms,
// far longer than a copy takes.
__device__ __forceinline__ void drain_copies(uint64_t* full, int stages, int it) {
  for (int j = max(it - stages, 0); j < it; ++j) mbar_wait_bounded(&full[j % stages], (j / stages) & 1, 1000000);
}

// Warp 0: weights by TMA. Warp 1: MMA issue. Warp 2: rows by TMA, or the last four warps gather them. Warps 4-7 and 8-11:
// epilogue, of 32 columns in turn or of a block each. One block has two sets of accumulators, two blocks have one.
template <int TYPE, int ACT, int NMAX, bool GATHER, int MB>
__global__ void __launch_bounds__(kGrThreads + (GATHER ? kGrGather : 0), 1)
    grouped_mma_kernel(const __grid_constant__ GroupedMmaParams mp) {
  using G = GrGeom<NMAX, MB>;
  const GroupedParams& p = mp.g;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = align1024(smem_raw);
  GrTab& tt = *reinterpret_cast<GrTab*>(sm + G::kStages * G::kStage);
  GrBars& bb = *reinterpret_cast<GrBars*>(sm + G::kStages * G::kStage + sizeof(GrTab));
  float* slab = reinterpret_cast<float*>(sm + G::kStages * G::kStage + sizeof(GrTab) + sizeof(GrBars));
  volatile int* abort = &bb.abort;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int steps = (p.K + 63) / 64;
  const int nout = ACT ? p.N / 2 : p.N;

  if (threadIdx.x == 0) {
    for (int i = 0; i < G::kStages; ++i) {
      mbar_init(&bb.full[i], GATHER ? 1 + kGrGather : 2);
      mbar_init(&bb.empty[i], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&bb.acc_full[a], 1);
      mbar_init(&bb.acc_empty[a], 8);
    }
    mbar_init(&bb.done, 1);
    bb.abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&bb.tmem)));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  pdl_wait();
  pdl_trigger();
  // tile table: thread i owns the groups 4i..4i+3
  int tiles4 = 0, first4[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = 4 * threadIdx.x + j;           // warps behind the eighth own none
    first4[j] = tiles4;
    if (e < p.E) {
      const int2 s = group_span(p.offsets, e, p.P);
      tt.off[e] = s.x;
      tt.cnt[e] = s.y;
      tiles4 += mp.m_tiles * ((s.y + NMAX - 1) / NMAX);
    }
  }
  int incl = tiles4;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(kAll, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31 && warp < kGrTabWarps) tt.wsum[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  int base = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kGrTabWarps; ++w) {
    if (w < warp) base += tt.wsum[w];
    total += tt.wsum[w];
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int e = 4 * threadIdx.x + j;
    if (e < p.E) tt.start[e] = base + incl - tiles4 + first4[j];
  }
  __syncthreads();
  const uint32_t tmem = bb.tmem;

  if (warp == 0) {
    if (lane == 0) {
      const uint64_t pol = l2_evict_first();
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok && !*abort; t += gridDim.x) {
        const GrTile tl = gr_tile<NMAX>(tt, p.E, t);
        for (int s = 0; s < steps; ++s, ++it) {
          const int slot = it % G::kStages;
          if (it >= G::kStages && !pf_wait(&bb.empty[slot], ((it / G::kStages) - 1) & 1, abort, &g_ops_error)) {
            ok = false;
            break;
          }
          uint8_t* st = sm + slot * G::kStage;
          mbar_arrive_expect_tx(&bb.full[slot], G::kA);
#pragma unroll
          for (int b = 0; b < MB; ++b, st += kGrABytes) {
            if constexpr (ACT) {                 // 64 gate rows, then the 64 up rows of the same outputs
              const int r = tl.e * p.N + (tl.m * MB + b) * 64;
              if (tl.once) {
                tma_2d_hint(st, &mp.tm_w, s * 64, r, &bb.full[slot], pol);
                tma_2d_hint(st + kGrABytes / 2, &mp.tm_w, s * 64, r + nout, &bb.full[slot], pol);
              } else {
                tma_2d(st, &mp.tm_w, s * 64, r, &bb.full[slot]);
                tma_2d(st + kGrABytes / 2, &mp.tm_w, s * 64, r + nout, &bb.full[slot]);
              }
            } else if (tl.once) {
              tma_2d_hint(st, &mp.tm_w, s * 64, tl.e * p.N + (tl.m * MB + b) * 128, &bb.full[slot], pol);
            } else {
              tma_2d(st, &mp.tm_w, s * 64, tl.e * p.N + (tl.m * MB + b) * 128, &bb.full[slot]);
            }
          }
        }
      }
      drain_copies(bb.full, G::kStages, it);
    }
  } else if (!GATHER && warp == 2) {
    if (lane == 0) {
      int it = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < total && ok && !*abort; t += gridDim.x) {
        const GrTile tl = gr_tile<NMAX>(tt, p.E, t);
        const int boxes = (tl.n + G::kBox - 1) / G::kBox;    // rows behind the tile's only feed unused columns
        for (int s = 0; s < steps; ++s, ++it) {
          const int slot = it % G::kStages;
          if (it >= G::kStages && !pf_wait(&bb.empty[slot], ((it / G::kStages) - 1) & 1, abort, &g_ops_error)) {
            ok = false;
            break;
          }
          uint8_t* st = sm + slot * G::kStage + G::kA;
          mbar_arrive_expect_tx(&bb.full[slot], boxes * G::kBox * 128);
          for (int b = 0; b < boxes; ++b)
            tma_2d(st + b * G::kBox * 128, &mp.tm_x, s * 64, tl.row0 + b * G::kBox, &bb.full[slot]);
        }
      }
      drain_copies(bb.full, G::kStages, it);
    }
  } else if (GATHER && warp >= kGrThreads / 32) {
    // eight lanes per row of 128 bytes; a stage's barrier completes when every thread's copies have landed
    constexpr int kPass = NMAX / 16;
    const int tid = threadIdx.x - kGrThreads, c = tid & 7, r0 = tid >> 3;
    const uint32_t dst0 = smem_u32(sm) + G::kA + r0 * 128 + ((c ^ (r0 & 7)) << 4);
    int it = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x) {
      const GrTile tl = gr_tile<NMAX>(tt, p.E, t);
      const int passes = (tl.n + 15) >> 4;                   // rows behind the last one repeat it: unused columns
      const uint16_t* src[kPass];
#pragma unroll
      for (int i = 0; i < kPass; ++i)
        src[i] = p.x + (i < passes ? source_row(p, tl.row0 + min(r0 + 16 * i, tl.n - 1)) * p.ldx : 0);
      for (int s = 0; s < steps; ++s, ++it) {
        const int slot = it % G::kStages;
        if (it >= G::kStages && !pf_wait_all(&bb.empty[slot], ((it / G::kStages) - 1) & 1, abort, &g_ops_error)) {
          ok = false;
          break;
        }
        const int k = s * 64 + 8 * c;
        const bool in = k < p.K;
        const uint32_t dst = dst0 + slot * G::kStage;
#pragma unroll
        for (int i = 0; i < kPass; ++i)
          if (i < passes) cp_async16(dst + i * 2048, src[i] + (in ? k : 0), in);
        cp_async_arrive(&bb.full[slot]);
      }
    }
    cp_async_wait_all();
  } else if (warp == 1) {
    int it = 0, ti = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < total && ok; t += gridDim.x, ++ti) {
      const GrTile tl = gr_tile<NMAX>(tt, p.E, t);
      const uint32_t idesc = idesc_m128((tl.n + 15) & ~15, TYPE == kTBf16);
      const int sets = MB == 1 ? 2 : 1, as = ti % sets;
      const uint32_t d = tmem + as * 256;
      if (ti >= sets && !pf_wait_all(&bb.acc_empty[as], (ti / sets - 1) & 1, abort, &g_ops_error)) break;
      tc_fence_after();
      for (int s = 0; s < steps; ++s, ++it) {
        const int slot = it % G::kStages;
        if (!pf_wait_all(&bb.full[slot], (it / G::kStages) & 1, abort, &g_ops_error)) {
          ok = false;
          break;
        }
        if constexpr (GATHER) fence_proxy_async_shared();     // the rows were written by ordinary (cp.async) copies
        tc_fence_after();
        const uint32_t a0 = smem_u32(sm + slot * G::kStage), b0 = a0 + G::kA;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
#pragma unroll
          for (int b = 0; b < MB; ++b)
            tc_mma_ss_w(d + b * 256, sdesc_sw128(a0 + b * kGrABytes + ks * 32), sdesc_sw128(b0 + ks * 32), idesc,
                        (s | ks) ? 1u : 0u);
        tc_commit_w(&bb.empty[slot]);
      }
      if (ok) tc_commit_w(&bb.acc_full[as]);
    }
    tc_commit_w(&bb.done);
    pf_wait_all(&bb.done, 0, abort, &g_ops_error);
  } else if (warp >= 4 && warp < 12) {
    const int q = warp & 3, team = (warp - 4) >> 2, blk = MB == 2 ? team : 0;
    constexpr int kStep = MB == 2 ? 32 : 64;     // from 32 columns of a team to its next
    const uint32_t lane_base = tmem + (static_cast<uint32_t>(32 * q) << 16);
    int ti = 0;
    for (int t = blockIdx.x; t < total; t += gridDim.x, ++ti) {
      const GrTile tl = gr_tile<NMAX>(tt, p.E, t);
      const int sets = MB == 1 ? 2 : 1, as = ti % sets;
      const bool ok = pf_wait_all(&bb.acc_full[as], (ti / sets) & 1, abort, &g_ops_error);
      if (named_bar_or(1 + team, 128, !ok)) break;           // a team gives up together: it meets at barriers below
      tc_fence_after();
      const uint32_t d = lane_base + (as + blk) * 256;
      if constexpr (ACT) {
        // warps 0, 1 hold the gate and 2, 3 the up values of the same 64 outputs: of 32 columns, each side hands 16
        // to the other through shared memory and finishes the other 16
        const int r = 32 * (q & 1) + lane, n = (tl.m * MB + blk) * 64 + r, up = q >> 1;
        for (int j0 = MB == 2 ? 0 : 32 * team; j0 < tl.n; j0 += kStep) {
          uint32_t own[16], give[16];
          tc_ld16(d + j0 + 16 * up, own);
          tc_ld16(d + j0 + 16 * (up ^ 1), give);
          tc_wait_ld();
          float* to = slab + ((team * 2 + up) * 16) * 64 + r;
          const float* from = slab + ((team * 2 + (up ^ 1)) * 16) * 64 + r;
#pragma unroll
          for (int c = 0; c < 16; ++c) to[c * 64] = __uint_as_float(give[c]);
          named_bar_sync(1 + team, 128);
          uint16_t* yr = p.y + static_cast<long long>(tl.row0 + j0 + 16 * up) * p.ldy + n;
#pragma unroll
          for (int c = 0; c < 16; ++c) {
            const float o = from[c * 64], v = __uint_as_float(own[c]);
            const float h = up ? silu_fast(o) * v : silu_fast(v) * o;
            if (j0 + 16 * up + c < tl.n && n < nout) yr[c * p.ldy] = from_f32<TYPE>(h);
          }
          named_bar_sync(1 + team, 128);         // the slab is written again
        }
      } else {
        for (int j0 = MB == 2 ? 0 : 32 * team; j0 < tl.n; j0 += (j0 & 16) ? kStep - 16 : 16) {
          uint32_t v[16];
          tc_ld16(d + j0, v);
          tc_wait_ld();
          const int n = (tl.m * MB + blk) * 128 + 32 * q + lane;
          uint16_t* yr = p.y + static_cast<long long>(tl.row0 + j0) * p.ldy + n;
#pragma unroll
          for (int c = 0; c < 16; ++c)
            if (j0 + c < tl.n && n < nout) yr[c * p.ldy] = from_f32<TYPE>(__uint_as_float(v[c]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bb.acc_empty[as]);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

template <int TYPE, int ACT, int NMAX, bool GATHER, int MB = 1>
cudaError_t launch_mma(const GroupedParams& p, int dev, int sms, cudaStream_t s) {
  GroupedMmaParams mp;
  mp.g = p;
  const int nout = ACT ? p.N / 2 : p.N;
  mp.m_tiles = (nout + (ACT ? 64 : 128) * MB - 1) / ((ACT ? 64 : 128) * MB);
  if (!encode_16bit(&mp.tm_w, p.w, TYPE == kTBf16, static_cast<uint64_t>(p.E) * p.N, p.K, p.K, ACT ? 64 : 128) ||
      (!GATHER && !encode_16bit(&mp.tm_x, p.x, TYPE == kTBf16, p.x_rows, p.K, p.ldx, GrGeom<NMAX, MB>::kBox)))
    return cudaErrorInvalidValue;
  cudaError_t e = allow_smem_once<grouped_mma_kernel<TYPE, ACT, NMAX, GATHER, MB>>(dev, gr_smem<NMAX, MB>());
  if (e != cudaSuccess) return e;
  // tiles that the rows can make at most
  const long long chunks = p.P / NMAX + (p.E < p.P ? p.E : p.P);
  const long long most = chunks * mp.m_tiles;
  return launch_op(grouped_mma_kernel<TYPE, ACT, NMAX, GATHER, MB>, dim3(most < sms ? static_cast<int>(most) : sms),
                   kGrThreads + (GATHER ? kGrGather : 0), gr_smem<NMAX, MB>(), s, mp);
}

// ---------------------------------------------------------------------------------------------
// Few rows (P <= kFewRows): bound by streaming the active groups' weights once. A group makes an entry per eight of its
// rows (the MMA's columns; one entry, as a rule); the weight rows of all entries are cut into units of 16 (SwiGLU: 8 gate
// rows and their 8 up rows) and spread evenly over one CTA per SM, which a GEMM's 128-row tiles cannot do when a token has
// six experts. One thread keeps a ring of stages full: a stage is up to 1024 K of the units that the 16 other warps work
// on, in teams of eight or four warps per unit (fewer when K is short), one TMA box of up to 32 KB per unit (half a unit
// with SwiGLU). A warp takes 128 K of a stage and multiplies with mma.sync m16n8k16; any order of K serves as long as both
// operands have it, so a lane reads 8 neighbouring K at a time and x comes straight from global memory, through L1. A
// team's partial sums meet in shared memory and are added in warp order; teams do not wait for one another.
// Small copies starve it: bulk copies of one row (1 or 4 KB) and boxes of 2 KB all streamed ~11 bytes per cycle and
// SM, boxes of 8 KB and more over twice that.
constexpr int kFewWarps = 16;                    // consumers; one more warp copies
constexpr int kFewThreads = 32 * (kFewWarps + 1);
// Warps of a team at most, each with 128 K of a stage: 8 (fewer idle teams in the last round: 12 rows over 256 experts
// 14.7 us against 16.0, 30 rows 25.1 against 27.2), but 4 when a CTA has few units (6 rows 9.6 us against 10.7).
constexpr int kFewSplit = 8;
constexpr int kFewMaxStages = 8;

struct FewTab {
  uint64_t full[kFewMaxStages], empty[kFewMaxStages];
  int pad, abort;
  int wsum[kFewWarps + 1];
  int e[kFewRows], off[kFewRows], cnt[kFewRows];
  int src[kFewRows];                             // row of x of each row of y
};

struct FewParams {
  CUtensorMap tm;                                // blocks: [K / 64][E N][64], else [E N][K] (K % 64 != 0)
  GroupedParams g;
  int kw;                                        // warps that split a unit's K (a power of two)
  int stages;
  int blocks;                                    // 1: one box holds all 64-K blocks of a stage
};
constexpr int kFewStage = kFewWarps * 4096;      // 16 rows x 128 K per warp

template <int TYPE>
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                          uint32_t b1) {
  const uint32_t a[4] = {a0, a1, a2, a3};
  if constexpr (TYPE == kTBf16) mma_bf16_16816(d, a, b0, b1);
  else mma_f16_16816(d, a, b0, b1);
}

template <int TYPE, int ACT>
__global__ void __launch_bounds__(kFewThreads, 1) grouped_few_kernel(const __grid_constant__ FewParams ge) {
  const GroupedParams& p = ge.g;
  constexpr int kUnit = ACT ? 8 : 16;            // outputs per unit
  extern __shared__ uint8_t smem_raw[];
  __shared__ FewTab tab;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int nout = ACT ? p.N / 2 : p.N;
  const int units_per = (nout + kUnit - 1) / kUnit;
  const int teams = kFewWarps / ge.kw;
  uint8_t* ring = align1024(smem_raw);
  float4* red = reinterpret_cast<float4*>(ring + ge.stages * kFewStage);       // [warps][32]

  pdl_wait();
  pdl_trigger();
  // entries of up to eight rows of a group, in ascending order: thread i looks at the groups 2i, 2i + 1
  int2 span[2];
  int n = 0;
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int e = 2 * threadIdx.x + j;
    span[j] = e < p.E ? group_span(p.offsets, e, p.P) : make_int2(0, 0);
    n += (span[j].y + 7) / 8;
  }
  int incl = n;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(kAll, incl, d);
    if (lane >= d) incl += o;
  }
  if (lane == 31) tab.wsum[warp] = incl;
  if (threadIdx.x < p.P) tab.src[threadIdx.x] = source_row(p, threadIdx.x);
  if (threadIdx.x == 0) {
    for (int i = 0; i < ge.stages; ++i) {
      mbar_init(&tab.full[i], 1);
      mbar_init(&tab.empty[i], kFewWarps);
    }
    tab.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  int at = incl - n, total = 0;
#pragma unroll
  for (int w = 0; w <= kFewWarps; ++w) {
    if (w < warp) at += tab.wsum[w];
    total += tab.wsum[w];
  }
#pragma unroll
  for (int j = 0; j < 2; ++j)
    for (int i = 0; i < span[j].y; i += 8, ++at)
      if (at < kFewRows) {                       // groups that overlap (bad offsets) may be more: left out
        tab.e[at] = 2 * threadIdx.x + j;
        tab.off[at] = span[j].x + i;
        tab.cnt[at] = min(span[j].y - i, 8);
      }
  __syncthreads();
  const long long units = static_cast<long long>(min(total, kFewRows)) * units_per;
  const int u_lo = static_cast<int>(units * blockIdx.x / gridDim.x);
  const int u_hi = static_cast<int>(units * (blockIdx.x + 1) / gridDim.x);
  const int chunk = 128 * ge.kw, chunks = (p.K + chunk - 1) / chunk;
  volatile int* abort = &tab.abort;

  if (warp == kFewWarps) {
    // ---- weights
    if (lane == 0) {
      const uint64_t pol = l2_evict_first();
      const int kbs = 2 * ge.kw;                 // 64-K blocks of a stage
      int it = 0;
      bool ok = true;
      for (int u0 = u_lo; u0 < u_hi && ok; u0 += teams) {
        const int units_now = min(teams, u_hi - u0);
        for (int c = 0; c < chunks; ++c, ++it) {
          const int slot = it % ge.stages;
          if (it >= ge.stages && !pf_wait(&tab.empty[slot], ((it / ge.stages) - 1) & 1, abort, &g_ops_error)) {
            ok = false;
            break;
          }
          uint8_t* st = ring + slot * kFewStage;
          mbar_arrive_expect_tx(&tab.full[slot], units_now * kbs * 2048);
          for (int j = 0; j < units_now; ++j, st += kbs * 2048) {
            const int a = (u0 + j) / units_per;
            const int r = tab.e[a] * p.N + (u0 + j - a * units_per) * kUnit;
            if (ge.blocks) {
              tma_3d_hint(st, &ge.tm, 0, r, c * kbs, &tab.full[slot], pol);
              if constexpr (ACT) tma_3d_hint(st + kbs * 1024, &ge.tm, 0, r + nout, c * kbs, &tab.full[slot], pol);
            } else {
              for (int b = 0; b < kbs; ++b) {    // blocks behind K read as zeros
                const int x = (c * kbs + b) * 64;
                tma_2d_hint(st + b * kUnit * 128, &ge.tm, x, r, &tab.full[slot], pol);
                if constexpr (ACT) tma_2d_hint(st + kbs * 1024 + b * 1024, &ge.tm, x, r + nout, &tab.full[slot], pol);
              }
            }
          }
        }
      }
      drain_copies(tab.full, ge.stages, it);
    }
    return;
  }

  const int kw = warp % ge.kw, team = warp / ge.kw, tid = kw * 32 + lane;
  const float* rf = reinterpret_cast<const float*>(red) + team * ge.kw * 128;
  int it = 0;
  int ai = (u_lo + team) / units_per, un = u_lo + team - ai * units_per;       // unit `un` of entry ai
  bool ok = true;
  for (int u0 = u_lo; u0 < u_hi; u0 += teams) {
    const bool mine = u0 + team < u_hi;
    const int cnt = mine ? tab.cnt[ai] : 0, off = mine ? tab.off[ai] : 0;
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < chunks; ++c, ++it) {
      const int slot = it % ge.stages, k0 = c * chunk + kw * 128 + 8 * q;
      ok = ok && pf_wait_all(&tab.full[slot], (it / ge.stages) & 1, abort, &g_ops_error);
      if (mine && ok) {
        // rows of 128 bytes in the 128-byte swizzle: [64-K block][row], with SwiGLU the gate rows' blocks first
        const uint8_t* st = ring + slot * kFewStage + team * ge.kw * 4096;
        const uint8_t* lo = st + kw * 2 * kUnit * 128 + g * 128;
        const uint8_t* hi = lo + (ACT ? ge.kw * 2048 : 1024);
        uint4 a[8];                              // row g: 0..3, row g + 8: 4..7; K = k0 + 32 i .. + 7
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = (i >> 1) * kUnit * 128 + (((q + 4 * (i & 1)) ^ g) << 4);
          a[i] = *reinterpret_cast<const uint4*>(lo + at);
          a[4 + i] = *reinterpret_cast<const uint4*>(hi + at);
        }
        const bool tok = g < cnt;
        const uint16_t* x = p.x + (tok ? tab.src[off + g] * p.ldx : 0) + k0;
        float d[4] = {0.f, 0.f, 0.f, 0.f};       // two chains
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint4 v = make_uint4(0, 0, 0, 0);
          if (tok && k0 + 32 * i < p.K) v = ld_nc_v4(x + 32 * i);
          mma_16816<TYPE>(acc, a[i].x, a[4 + i].x, a[i].y, a[4 + i].y, v.x, v.y);
          mma_16816<TYPE>(d, a[i].z, a[4 + i].z, a[i].w, a[4 + i].w, v.z, v.w);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[j] += d[j];
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&tab.empty[slot]);
    }
    if (cnt) red[warp * 32 + lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    if (named_bar_or(team, 32 * ge.kw, !ok)) break;            // a team gives up together
    const int j = tid % kUnit, nn = un * kUnit + j;
    if (nn < nout)
      for (int tok = tid / kUnit; tok < cnt; tok += 32 * ge.kw / kUnit) {
        const int at4 = ((j & 7) * 4 + (tok >> 1)) * 4 + (tok & 1);
        float r0 = 0.f, r1 = 0.f;
        for (int w = 0; w < ge.kw; ++w) {
          r0 += rf[at4 + w * 128 + (ACT ? 0 : (j >> 3) * 2)];
          if constexpr (ACT) r1 += rf[at4 + w * 128 + 2];
        }
        p.y[static_cast<long long>(off + tok) * p.ldy + nn] = from_f32<TYPE>(ACT ? silu_fast(r0) * r1 : r0);
      }
    named_bar_sync(team, 32 * ge.kw);
    un += teams;
    while (un >= units_per) {
      un -= units_per;
      ++ai;
    }
  }
}

template <int TYPE, int ACT>
cudaError_t launch_few(const GroupedParams& p, int dev, int sms, cudaStream_t s) {
  constexpr int kRed = kFewWarps * 512;
  constexpr int kStages = (226 * 1024 - static_cast<int>(sizeof(FewTab)) - 1024 - kRed) / kFewStage;
  constexpr int kSmem = kStages * kFewStage + kRed + 1024;
  static_assert(kStages >= 2 && kStages <= kFewMaxStages, "stages");
  cudaError_t e = allow_smem_once<grouped_few_kernel<TYPE, ACT>>(dev, kSmem);
  if (e != cudaSuccess) return e;
  FewParams fp;
  fp.g = p;
  fp.kw = 1;
  const long long units = static_cast<long long>(p.E < p.P ? p.E : p.P) * (p.N / 16 + 1);     // at most
  const int split = units <= 4ll * sms ? kFewSplit / 2 : kFewSplit;
  while (fp.kw * 128 < p.K && fp.kw < split) fp.kw *= 2;
  fp.stages = kStages;
  fp.blocks = p.K % 64 == 0;
  const uint64_t rows = static_cast<uint64_t>(p.E) * p.N;
  const uint32_t box = ACT ? 8 : 16;
  if (!(fp.blocks ? encode_16bit_blocks(&fp.tm, p.w, TYPE == kTBf16, rows, p.K, p.K, box, 2 * fp.kw)
                  : encode_16bit(&fp.tm, p.w, TYPE == kTBf16, rows, p.K, p.K, box)))
    return cudaErrorInvalidValue;
  return launch_op(grouped_few_kernel<TYPE, ACT>, dim3(sms), kFewThreads, kSmem, s, fp);
}

template <int TYPE, int ACT>
cudaError_t launch_type(const GroupedParams& p, cudaStream_t s) {
  int dev, sms;
  cudaError_t e = current_device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  if (p.P <= kFewRows && (p.P <= 8 || p.P / 8 <= p.E)) return launch_few<TYPE, ACT>(p, dev, sms, s);
  const long long mean = p.P / p.E;
  const bool ga = p.row_of != nullptr;
  // Rows of a tile by the mean group: 48 rows 161 us with 64, 178 with 128 (12288 rows over 256 experts); 82 rows 24.8, 24.1
  // and 27.2 us with 64, 128 and 256 (5003 rows over 61 experts, uneven)
  if (mean <= 64) return ga ? launch_mma<TYPE, ACT, 64, true>(p, dev, sms, s) : launch_mma<TYPE, ACT, 64, false>(p, dev, sms, s);
  if (mean <= 128) return ga ? launch_mma<TYPE, ACT, 128, true>(p, dev, sms, s) : launch_mma<TYPE, ACT, 128, false>(p, dev, sms, s);
  // Two blocks where rows are gathered and the tiles then still fill the SMs: 16384 tokens over 256 experts, gate|up,
  // 642 -> 463 us, 4096^3 173 -> 120 us. Rows by TMA gain less (110 -> 104 us) or lose to the accumulators' single set
  // (SwiGLU, 8 experts: 177 -> 197 us).
  const int nout = ACT ? p.N / 2 : p.N;
  const long long chunks = p.P / 256 > p.E ? p.P / 256 : p.E, wide = (nout + (ACT ? 127 : 255)) / (ACT ? 128 : 256);
  if (ga && wide * chunks * 2 >= 3 * sms) return launch_mma<TYPE, ACT, 256, true, 2>(p, dev, sms, s);
  return ga ? launch_mma<TYPE, ACT, 256, true>(p, dev, sms, s) : launch_mma<TYPE, ACT, 256, false>(p, dev, sms, s);
}

}  // namespace

cudaError_t launch_grouped_linear(const GroupedParams& p, cudaStream_t s) {
  if (p.type == kTBf16) return p.act ? launch_type<kTBf16, 1>(p, s) : launch_type<kTBf16, 0>(p, s);
  return p.act ? launch_type<kTF16, 1>(p, s) : launch_type<kTF16, 0>(p, s);
}

// Reads and clears the current device's word (waits for the device's work).
cudaError_t read_ops_error(unsigned* out) {
  const unsigned zero = 0;
  *out = 0;
  cudaError_t e = cudaDeviceSynchronize();
  if (e == cudaSuccess) e = cudaMemcpyFromSymbol(out, g_ops_error, sizeof(unsigned));
  if (e == cudaSuccess && *out) e = cudaMemcpyToSymbol(g_ops_error, &zero, sizeof(unsigned));
  unsigned more = 0;
  if (e == cudaSuccess) e = read_q4_error(&more);
  *out |= more;
  return e;
}

}  // namespace flint
