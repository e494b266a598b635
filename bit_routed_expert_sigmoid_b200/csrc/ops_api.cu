// Host side of the standalone operators' C ABI (flint_ops.h): argument checks and launches.
#include "../../include/flint_ops.h"
#include "ops.cuh"

using namespace flint;

namespace {

bool aligned_to(const void* p, uintptr_t a) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool opt_aligned(const void* p, uintptr_t a) { return p == nullptr || aligned_to(p, a); }
bool is_16bit(int type) { return type == FLINT_T_BF16 || type == FLINT_T_F16; }

constexpr int kMaxOpK = 65536;
constexpr int kMaxQ4Tokens = 65536;              // chunks of at least 8 tokens are a grid dimension
constexpr int kMaxOpGroups = 1024;
constexpr int kMaxOpTopK = 64;
constexpr long long kMaxOpPairs = 1ll << 22;
constexpr int kMaxCombineH = 1 << 23;            // blocks of 256 columns are a grid dimension
constexpr int kMaxNormH = 32768;

flint_status status_of(cudaError_t e) { return e == cudaSuccess ? FLINT_OK : FLINT_ERR_CUDA; }

}  // namespace

extern "C" {

size_t flint_q4_linear_workspace_size(int K, int T) {
  return K < 1 || K > kMaxOpK || T < 1 ? 0 : q4_workspace_bytes(K, T);
}

flint_status flint_q4_linear(int fmt, int N, int K, int rotated, const void* codes, const void* scales,
                             const float* tscale, const void* x, long long ldx, int T, int type, void* y, long long ldy,
                             void* workspace, size_t workspace_bytes, void* stream) {
  if (fmt != FLINT_W_INT4_G128_FWHT128 && fmt != FLINT_W_NVFP4) return FLINT_ERR_INVALID_ARG;
  const bool i4 = fmt == FLINT_W_INT4_G128_FWHT128;
  if (N < 1 || K < 1 || K % (i4 ? 128 : 16) != 0 || T < 0) return FLINT_ERR_INVALID_ARG;
  // byte offsets inside the rows of one CTA (at least 1/1024 of them) are 32 bits wide
  if (K > kMaxOpK || T > kMaxQ4Tokens || N > (1 << 30) || static_cast<long long>(N) * K > (1ll << 37)) return FLINT_ERR_UNSUPPORTED;
  if ((rotated != 0 && rotated != 1) || (rotated && !i4) || !is_16bit(type)) return FLINT_ERR_INVALID_ARG;
  if (ldx < K || ldx % 8 != 0 || ldy < N) return FLINT_ERR_INVALID_ARG;
  if (T == 0) return FLINT_OK;
  if (!aligned_to(codes, 16) || !aligned_to(scales, i4 ? 2 : 1) || !aligned_to(x, 16) || !aligned_to(y, 2) || x == y)
    return FLINT_ERR_INVALID_ARG;
  if (i4 ? !opt_aligned(tscale, 4) : !aligned_to(tscale, 4)) return FLINT_ERR_INVALID_ARG;
  const size_t need = q4_workspace_bytes(K, T);
  if (need && (!aligned_to(workspace, 256) || workspace_bytes < need)) return FLINT_ERR_WORKSPACE;
  Q4Params p{};
  p.workspace = workspace;
  p.fmt = i4 ? kInt4 : kNvfp4;
  p.N = N;
  p.K = K;
  p.rotated = rotated;
  p.codes = static_cast<const uint8_t*>(codes);
  p.scales = static_cast<const uint8_t*>(scales);
  p.tscale = tscale;
  p.x = static_cast<const uint16_t*>(x);
  p.ldx = ldx;
  p.T = T;
  p.type = type;
  p.y = static_cast<uint16_t*>(y);
  p.ldy = ldy;
  return status_of(launch_q4_linear(p, static_cast<cudaStream_t>(stream)));
}

flint_status flint_grouped_linear(int E, int N, int K, int act, int type, const void* w, const void* x, long long ldx,
                                  int x_rows, const int* row_of, int row_div, const int* offsets, int P, void* y,
                                  long long ldy, void* stream) {
  if (E < 1 || N < 1 || K < 1 || K % 8 != 0 || P < 0 || x_rows < 0 || row_div < 1) return FLINT_ERR_INVALID_ARG;
  if (E > kMaxOpGroups || K > kMaxOpK || static_cast<long long>(E) * N > 0x7FFFFFFFll) return FLINT_ERR_UNSUPPORTED;
  // tiles of 64 outputs x 64 rows are counted in 32 bits, whatever the offsets hold
  if ((static_cast<long long>(N) / 64 + 1) * E > 0x7FFFFFFFll / (P / 64 + 1)) return FLINT_ERR_UNSUPPORTED;
  if ((act != FLINT_ACT_NONE && act != FLINT_ACT_SWIGLU) || !is_16bit(type)) return FLINT_ERR_INVALID_ARG;
  if (act == FLINT_ACT_SWIGLU && N % 2 != 0) return FLINT_ERR_INVALID_ARG;
  if (ldx < K || ldx % 8 != 0 || ldy < (act == FLINT_ACT_SWIGLU ? N / 2 : N)) return FLINT_ERR_INVALID_ARG;
  if (P == 0) return FLINT_OK;
  if (row_of ? x_rows < 1 : x_rows < P) return FLINT_ERR_INVALID_ARG;
  if (!aligned_to(w, 16) || !aligned_to(x, 16) || !aligned_to(y, 2) || !aligned_to(offsets, 4) || !opt_aligned(row_of, 4) ||
      x == y || w == y)
    return FLINT_ERR_INVALID_ARG;
  GroupedParams p{};
  p.E = E;
  p.N = N;
  p.K = K;
  p.act = act;
  p.type = type;
  p.w = static_cast<const uint16_t*>(w);
  p.x = static_cast<const uint16_t*>(x);
  p.ldx = ldx;
  p.x_rows = x_rows;
  p.row_of = row_of;
  p.row_div = row_div;
  p.offsets = offsets;
  p.P = P;
  p.y = static_cast<uint16_t*>(y);
  p.ldy = ldy;
  return status_of(launch_grouped_linear(p, static_cast<cudaStream_t>(stream)));
}

flint_status flint_expert_permute(const int* ids, int T, int top_k, int E, int* offsets, int* perm, int* inv,
                                  void* stream) {
  if (T < 0 || top_k < 1 || E < 1) return FLINT_ERR_INVALID_ARG;
  if (top_k > kMaxOpTopK || E > kMaxOpGroups || static_cast<long long>(T) * top_k > kMaxOpPairs) return FLINT_ERR_UNSUPPORTED;
  if (!aligned_to(offsets, 4)) return FLINT_ERR_INVALID_ARG;
  if (T > 0 && (!aligned_to(ids, 4) || !aligned_to(perm, 4) || !aligned_to(inv, 4))) return FLINT_ERR_INVALID_ARG;
  if (T > 0 && (perm == inv || offsets == perm || offsets == inv || ids == perm || ids == inv || ids == offsets))
    return FLINT_ERR_INVALID_ARG;
  return status_of(launch_expert_permute(ids, T * top_k, E, offsets, perm, inv, static_cast<cudaStream_t>(stream)));
}

flint_status flint_expert_combine(const void* o, long long ldo, int P, const int* inv, const float* w, int T, int top_k,
                                  int H, float scale, const void* addend, long long lda, int type, void* y,
                                  long long ldy, void* stream) {
  if (T < 0 || P < 0 || top_k < 1 || H < 1 || !is_16bit(type)) return FLINT_ERR_INVALID_ARG;
  if (top_k > kMaxOpTopK || H > kMaxCombineH) return FLINT_ERR_UNSUPPORTED;
  if (ldo < H || ldy < H || (addend && lda < H)) return FLINT_ERR_INVALID_ARG;
  if (T == 0) return FLINT_OK;
  if ((P > 0 && !aligned_to(o, 2)) || !aligned_to(inv, 4) || !aligned_to(w, 4) || !opt_aligned(addend, 2) ||
      !aligned_to(y, 2) || o == y || (addend == y && lda != ldy))
    return FLINT_ERR_INVALID_ARG;
  CombineParams p{};
  p.o = static_cast<const uint16_t*>(o);
  p.ldo = ldo;
  p.P = P;
  p.inv = inv;
  p.w = w;
  p.T = T;
  p.top_k = top_k;
  p.H = H;
  p.scale = scale;
  p.addend = static_cast<const uint16_t*>(addend);
  p.lda = lda;
  p.type = type;
  p.y = static_cast<uint16_t*>(y);
  p.ldy = ldy;
  return status_of(launch_expert_combine(p, static_cast<cudaStream_t>(stream)));
}

flint_status flint_block_norm(const flint_norm_args* a, void* stream) {
  if (!a || a->T < 0 || a->H < 1 || !(a->eps > 0.f)) return FLINT_ERR_INVALID_ARG;
  if (a->H > kMaxNormH) return FLINT_ERR_UNSUPPORTED;
  if (!is_16bit(a->type) || (a->res_type != FLINT_T_F32 && a->res_type != a->type) ||
      (a->w_type != FLINT_T_F32 && a->w_type != a->type))
    return FLINT_ERR_INVALID_ARG;
  if ((a->post_norm != 0 && a->post_norm != 1) || (a->post_norm && !a->y) ||
      (a->gate_act != FLINT_GATE_NONE && a->gate_act != FLINT_GATE_SIGMOID))
    return FLINT_ERR_INVALID_ARG;
  if ((a->gate && !a->y) || (a->post_weight && !a->post_norm) || (a->pre_weight && !a->z)) return FLINT_ERR_INVALID_ARG;
  if (a->ldx < a->H || (a->x_out && a->ldxo < a->H) || (a->y && a->ldy < a->H) || (a->z && a->ldz < a->H) ||
      (a->gate && a->ldg != 0 && a->ldg < a->H) || (a->x_out == a->x && a->ldxo != a->ldx))
    return FLINT_ERR_INVALID_ARG;
  if (a->T == 0 || (!a->x_out && !a->z)) return FLINT_OK;
  const uintptr_t rb = a->res_type == FLINT_T_F32 ? 4 : 2, wb = a->w_type == FLINT_T_F32 ? 4 : 2;
  if (!aligned_to(a->x, rb) || !opt_aligned(a->x_out, rb) || !opt_aligned(a->y, 2) || !opt_aligned(a->gate, 2) ||
      !opt_aligned(a->post_weight, wb) || !opt_aligned(a->pre_weight, wb) || !opt_aligned(a->z, 2))
    return FLINT_ERR_INVALID_ARG;
  if (a->z && (a->z == a->x || a->z == a->x_out || a->z == a->y || a->z == a->gate)) return FLINT_ERR_INVALID_ARG;
  if (a->x_out && (a->x_out == a->y || a->x_out == a->gate)) return FLINT_ERR_INVALID_ARG;
  NormParams p{};
  p.x = a->x;
  p.x_out = a->x_out;
  p.y = static_cast<const uint16_t*>(a->y);
  p.gate = static_cast<const uint16_t*>(a->gate);
  p.post_w = a->post_weight;
  p.pre_w = a->pre_weight;
  p.z = static_cast<uint16_t*>(a->z);
  p.ldx = a->ldx;
  p.ldxo = a->ldxo;
  p.ldy = a->ldy;
  p.ldg = a->ldg;
  p.ldz = a->ldz;
  p.T = a->T;
  p.H = a->H;
  p.type = a->type;
  p.res_f32 = a->res_type == FLINT_T_F32;
  p.w_f32 = a->w_type == FLINT_T_F32;
  p.post_norm = a->post_norm;
  p.gate_act = a->gate_act;
  p.res_scale = a->res_scale;
  p.branch_scale = a->branch_scale;
  p.eps = a->eps;
  return status_of(launch_block_norm(p, static_cast<cudaStream_t>(stream)));
}

flint_status flint_ops_error_word(unsigned* out) {
  if (!out) return FLINT_ERR_INVALID_ARG;
  return status_of(read_ops_error(out));
}

}  // extern "C"
