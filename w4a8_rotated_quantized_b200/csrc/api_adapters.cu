// api_adapters.cu -- the extern "C" entry points for low-rank adapters beside a projection (forward and
// backward), the 8-bit activation checkpoints and the packed layer's input gradient: argument validation
// on the host, device check, workspace carving and launches on the caller's stream.
//
// The adapters are the bf16 branch that the model cards keep beside a quantised layer ("Qwen-Image-Edit-
// 2511 -- W4A8 ConvRot", notes on LoRA: merged by requantising the weight, or kept as a branch of its own).

#include <cuda_runtime.h>

#include <cstdint>
#include <initializer_list>

#include "../../include/convrot.h"
#include "cr_internal.h"

namespace {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

inline cr_status cuda_status(cudaError_t e) { return e == cudaSuccess ? CR_OK : CR_ERR_CUDA; }

inline int* ws_status(void* workspace) {
  return reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + cr::kWsStatusOff);
}

// The status word of a call that launches no kernel to clear it.
inline cr_status clear_status(void* workspace, size_t workspace_bytes, cudaStream_t s) {
  if (!workspace || workspace_bytes < 16) return CR_OK;
  return cuda_status(cudaMemsetAsync(ws_status(workspace), 0, 16, s));
}

// Workspace of the adapter calls: the status word's 256 bytes, then the parts below, each on 256 bytes.
constexpr size_t kWsHead = 256;

inline size_t bytes_f32(int64_t n) { return cr::round_up(static_cast<size_t>(n) * 4, 256); }

// Splits, and with them the workspace, go by a B200's SM count whatever device is current: the size calls ask
// none, and the same call gives the same bits everywhere.
constexpr int kSizingSms = 148;

bool sizes_ok(int M, int N, int K, int rank, int L) {
  return M >= 0 && N >= 8 && N % 8 == 0 && N <= CR_MAX_K && K >= 8 && K % 8 == 0 && K <= CR_MAX_K && rank >= 4 &&
         rank <= CR_MAX_RANK && rank % 4 == 0 && L >= 1 && L <= CR_MAX_ADAPTERS;
}

struct GradSplits {
  int down = 0, up = 0;
};
GradSplits grad_splits(int M, int N, int K, int rank, int L, bool codes) {
  GradSplits g;
  cr::lora_grad_splits(M > 0 ? M : 1, K, N, rank, L, codes, kSizingSms, &g.down, &g.up);
  return g;
}

size_t backward_bytes(int M, int N, int K, int rank, int L, bool codes) {
  const GradSplits g = grad_splits(M, N, K, rank, L, codes);
  const int64_t per = static_cast<int64_t>(L) * rank;
  // (a gradient that is not split is written as it is)
  return kWsHead + bytes_f32(static_cast<int64_t>(M) * rank) + (g.down > 1 ? bytes_f32(g.down * per * K) : 0) +
         (g.up > 1 ? bytes_f32(g.up * per * N) : 0);
}

// An output may start at the very rows of the base that is added to it, and at no other operand's.
bool in_place_ok(const void* out, int64_t ldo, const void* base, int64_t ldb, int M, const void* a, const void* b) {
  if (out && (out == a || out == b)) return false;
  return !out || out != base || ldo == ldb || M <= 1;
}

cr_status check_rows(const void* p, int64_t ld, int cols) {
  if (ld < cols) return CR_ERR_INVALID_ARG;
  return (!aligned(p, 16) || ld % 8 != 0) ? CR_ERR_MISALIGNED : CR_OK;
}

}  // namespace

extern "C" {

size_t cr_lora_forward_workspace_size(int M, int N, int K, int rank, int num_adapters) {
  if (!sizes_ok(M, N, K, rank, num_adapters)) return kWsHead;
  if (cr::use_lora_rows(M, N, K, rank, num_adapters)) return 0;
  return kWsHead + bytes_f32(static_cast<int64_t>(M) * rank);
}

cr_status cr_lora_forward(const void* X, int64_t ldx, const int32_t* adapter, const void* down, const void* up,
                          const float* scale, const void* base, int64_t ldb, void* Y, int64_t ldy, void* V, int M,
                          int N, int K, int rank, int num_adapters, void* workspace, size_t workspace_bytes,
                          void* stream) {
  if (M < 0 || N < 0 || K < 0 || rank < 0 || num_adapters < 0 || ldx < 0 || ldb < 0 || ldy < 0)
    return CR_ERR_INVALID_ARG;
  if (M > 0 && (!X || !down || !up || !scale || !Y)) return CR_ERR_INVALID_ARG;
  if (M > 0 && !in_place_ok(Y, ldy, base, ldb, M, X, V)) return CR_ERR_INVALID_ARG;
  if (!sizes_ok(M, N, K, rank, num_adapters)) return CR_ERR_UNSUPPORTED_SHAPE;
  cr_status st = check_rows(X, ldx, K);
  if (st == CR_OK) st = check_rows(Y, ldy, N);
  if (st == CR_OK && base) st = check_rows(base, ldb, N);
  if (st != CR_OK) return st;
  if (!aligned(down, 16) || !aligned(up, 16) || !aligned(scale, 4) || !aligned(adapter, 4) || !aligned(V, 8))
    return CR_ERR_MISALIGNED;
  const size_t need = M > 0 ? cr_lora_forward_workspace_size(M, N, K, rank, num_adapters) : 0;
  // (of one that is given although none is needed, the status word is written)
  if ((need > 0 && (!workspace || workspace_bytes < need)) || !aligned(workspace, 256)) return CR_ERR_WORKSPACE;
  int nsm = 0;
  if ((st = static_cast<cr_status>(cr::check_current_device(&nsm))) != CR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0) return clear_status(workspace, workspace_bytes, s);
  float* v = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWsHead);
  uint16_t* vout = static_cast<uint16_t*>(V);
  int* status = ws_status(workspace);
  const uint16_t* x = static_cast<const uint16_t*>(X);
  const uint16_t* dn = static_cast<const uint16_t*>(down);
  const uint16_t* u = static_cast<const uint16_t*>(up);
  const uint16_t* b = static_cast<const uint16_t*>(base);
  uint16_t* y = static_cast<uint16_t*>(Y);
  const int L = num_adapters;
  if (cr::use_lora_rows(M, N, K, rank, L))
    return static_cast<cr_status>(
        cr::launch_lora_rows(x, ldx, adapter, dn, u, scale, b, ldb, y, ldy, nullptr, vout, M, N, K, rank, L,
                             workspace && workspace_bytes >= 16 ? status : nullptr, s));
  int r = cr::launch_lora_v_mma(x, ldx, adapter, dn, v, vout, M, K, rank, L, status, nsm, s);
  if (r == CR_OK) r = cr::launch_lora_y_mma(v, adapter, u, scale, b, ldb, y, ldy, M, N, rank, L, status, nsm, s);
  return static_cast<cr_status>(r);
}

size_t cr_lora_backward_workspace_size(int M, int N, int K, int rank, int num_adapters) {
  if (!sizes_ok(M, N, K, rank, num_adapters)) return kWsHead;
  // X as rows or as a checkpoint: the larger of the two
  const size_t rows = backward_bytes(M, N, K, rank, num_adapters, false);
  const size_t codes = backward_bytes(M, N, K, rank, num_adapters, true);
  return rows > codes ? rows : codes;
}

cr_status cr_lora_backward(const void* dY, int64_t lddy, const void* X, int64_t ldx, const void* codes,
                           const float* code_scales, const void* V, const int32_t* adapter, const void* down,
                           const void* up, const float* scale, const void* dX_base, int64_t ldb, void* dX, int64_t lddx,
                           void* d_down, void* d_up, int M, int N, int K, int rank, int num_adapters, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || rank < 0 || num_adapters < 0 || lddy < 0 || ldx < 0 || ldb < 0 || lddx < 0)
    return CR_ERR_INVALID_ARG;
  if (M > 0 && (!dY || !down || !up)) return CR_ERR_INVALID_ARG;
  if (!scale || (X && codes) || ((codes != nullptr) != (code_scales != nullptr))) return CR_ERR_INVALID_ARG;
  if (M > 0 && ((d_down && !X && !codes) || (d_up && !V))) return CR_ERR_INVALID_ARG;
  if (M > 0 && !in_place_ok(dX, lddx, dX_base, ldb, M, dY, X)) return CR_ERR_INVALID_ARG;
  if (!sizes_ok(M, N, K, rank, num_adapters) || (codes && K % 256 != 0)) return CR_ERR_UNSUPPORTED_SHAPE;
  cr_status st = check_rows(dY, lddy, N);
  if (st == CR_OK && X) st = check_rows(X, ldx, K);
  if (st == CR_OK && dX) st = check_rows(dX, lddx, K);
  if (st == CR_OK && dX && dX_base) st = check_rows(dX_base, ldb, K);
  if (st != CR_OK) return st;
  if (!aligned(codes, 16) || !aligned(code_scales, 4) || !aligned(V, 8) || !aligned(adapter, 4) || !aligned(down, 16) ||
      !aligned(up, 16) || !aligned(scale, 4) || !aligned(d_down, 16) || !aligned(d_up, 16))
    return CR_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < backward_bytes(M, N, K, rank, num_adapters, codes != nullptr) ||
      !aligned(workspace, 256))
    return CR_ERR_WORKSPACE;
  int nsm = 0;
  if ((st = static_cast<cr_status>(cr::check_current_device(&nsm))) != CR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int L = num_adapters;
  const int64_t nd = static_cast<int64_t>(L) * rank * K, nu = static_cast<int64_t>(L) * rank * N;
  if (M == 0) {  // no rows: the gradients are zero
    cudaError_t e = cudaMemsetAsync(ws_status(workspace), 0, 16, s);
    if (e == cudaSuccess && d_down) e = cudaMemsetAsync(d_down, 0, static_cast<size_t>(nd) * 2, s);
    if (e == cudaSuccess && d_up) e = cudaMemsetAsync(d_up, 0, static_cast<size_t>(nu) * 2, s);
    return cuda_status(e);
  }
  uint8_t* w = static_cast<uint8_t*>(workspace) + kWsHead;
  float* dv = reinterpret_cast<float*>(w);
  const GradSplits parts = grad_splits(M, N, K, rank, L, codes != nullptr);
  float* gd = reinterpret_cast<float*>(w + bytes_f32(static_cast<int64_t>(M) * rank));
  float* gu = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(gd) + (parts.down > 1 ? bytes_f32(parts.down * nd) : 0));
  int* status = ws_status(workspace);
  const uint16_t* dy = static_cast<const uint16_t*>(dY);
  const uint16_t* dn = static_cast<const uint16_t*>(down);
  const uint16_t* u = static_cast<const uint16_t*>(up);
  const uint16_t* xb = static_cast<const uint16_t*>(dX_base);
  uint16_t* dx = static_cast<uint16_t*>(dX);
  int r = CR_OK;
  if (dX && cr::use_lora_rows(M, K, N, rank, L)) {  // the forward's two products, up and down in each other's places
    r = cr::launch_lora_rows(dy, lddy, adapter, u, dn, scale, xb, ldb, dx, lddx, dv, nullptr, M, K, N, rank, L, status, s);
  } else if (dX || d_down) {
    r = cr::launch_lora_v_mma(dy, lddy, adapter, u, dv, nullptr, M, N, rank, L, status, nsm, s);
    if (r == CR_OK && dX)
      r = cr::launch_lora_y_mma(dv, adapter, dn, scale, xb, ldb, dx, lddx, M, K, rank, L, status, nsm, s);
  } else {
    r = clear_status(workspace, workspace_bytes, s);
  }
  if (r != CR_OK) return static_cast<cr_status>(r);
  if (d_down || d_up) {
    st = static_cast<cr_status>(cr::launch_lora_grad_mma(
        codes ? codes : X, ldx, code_scales, dY, lddy, dv, static_cast<const uint16_t*>(V), adapter, scale,
        gd, gu, static_cast<uint16_t*>(d_down), static_cast<uint16_t*>(d_up), M, K, N, rank, L, parts.down, parts.up,
        status, s));
    if (st != CR_OK) return st;
    uint16_t* split_down = parts.down > 1 ? static_cast<uint16_t*>(d_down) : nullptr;
    uint16_t* split_up = parts.up > 1 ? static_cast<uint16_t*>(d_up) : nullptr;
    if ((split_down || split_up) &&
        cr::launch_lora_grad_finish(gd, gu, parts.down, parts.up, static_cast<int64_t>(L) * rank, K, N, split_down,
                                    split_up, codes != nullptr, s) != cudaSuccess)
      return CR_ERR_CUDA;
  }
  return CR_OK;
}

cr_status cr_ckpt_save(const void* X, int M, int K, int64_t ldx, void* codes, float* scales, void* stream) {
  if (M < 0 || K < 0 || ldx < 0 || (M > 0 && (!X || !codes || !scales))) return CR_ERR_INVALID_ARG;
  if (K < 256 || K % 256 != 0 || K > CR_MAX_K) return CR_ERR_UNSUPPORTED_SHAPE;
  cr_status st = check_rows(X, ldx, K);
  if (st != CR_OK) return st;
  if (!aligned(codes, 16) || !aligned(scales, 4)) return CR_ERR_MISALIGNED;
  int nsm = 0;
  if ((st = static_cast<cr_status>(cr::check_current_device(&nsm))) != CR_OK) return st;
  if (M == 0) return CR_OK;
  return static_cast<cr_status>(cr::launch_ckpt_save(static_cast<const uint16_t*>(X), M, K, ldx,
                                                     static_cast<int8_t*>(codes), scales, nsm,
                                                     static_cast<cudaStream_t>(stream)));
}

cr_status cr_ckpt_load(const void* codes, const float* scales, int M, int K, void* X, int64_t ldx, void* stream) {
  if (M < 0 || K < 0 || ldx < 0 || (M > 0 && (!X || !codes || !scales))) return CR_ERR_INVALID_ARG;
  if (K < 256 || K % 256 != 0 || K > CR_MAX_K) return CR_ERR_UNSUPPORTED_SHAPE;
  cr_status st = check_rows(X, ldx, K);
  if (st != CR_OK) return st;
  if (!aligned(codes, 16) || !aligned(scales, 4)) return CR_ERR_MISALIGNED;
  int nsm = 0;
  if ((st = static_cast<cr_status>(cr::check_current_device(&nsm))) != CR_OK) return st;
  if (M == 0) return CR_OK;
  return static_cast<cr_status>(cr::launch_ckpt_load(static_cast<const int8_t*>(codes), scales, M, K,
                                                     static_cast<uint16_t*>(X), ldx, nsm,
                                                     static_cast<cudaStream_t>(stream)));
}

size_t cr_w4a4_grad_input_workspace_size(int M, int N, int K, int group) {
  (void)group;
  if (M < 0 || N <= 0 || K < 256 || K % 256 != 0) return kWsHead;
  if (M > 0 && cr::use_grad_input_few(M, N, K))
    return kWsHead + cr::round_up(cr::grad_input_few_operand_rows(M) * N * 2, 256) +
           bytes_f32(static_cast<int64_t>(M) * K * cr::grad_input_few_splits(M, N, K, kSizingSms));
  return kWsHead + cr::round_up(static_cast<size_t>(N) * static_cast<size_t>(K) * 2, 256);
}

cr_status cr_w4a4_grad_input(const void* dY, int64_t lddy, const void* Wq, const float* w_scale, void* dX, int64_t lddx,
                             int M, int N, int K, int group, void* workspace, size_t workspace_bytes, void* stream) {
  if (M < 0 || N < 0 || K < 0 || lddy < 0 || lddx < 0) return CR_ERR_INVALID_ARG;
  if (M > 0 && (!dX || (N > 0 && (!dY || !Wq || !w_scale || dX == dY)))) return CR_ERR_INVALID_ARG;
  if ((group != CR_GROUP_16 && group != CR_GROUP_64 && group != CR_GROUP_256 && group != CR_GROUP_1024) || K < 256 ||
      K % 256 != 0 || K % group != 0 || K > CR_MAX_K || N % 8 != 0 || N > CR_MAX_K)
    return CR_ERR_UNSUPPORTED_SHAPE;
  cr_status st = check_rows(dY, lddy, N);
  if (st == CR_OK) st = check_rows(dX, lddx, K);
  if (st != CR_OK) return st;
  if (!aligned(Wq, 16) || !aligned(w_scale, 4)) return CR_ERR_MISALIGNED;
  if (!workspace || workspace_bytes < cr_w4a4_grad_input_workspace_size(M, N, K, group) || !aligned(workspace, 256))
    return CR_ERR_WORKSPACE;
  int nsm = 0;
  if ((st = static_cast<cr_status>(cr::check_current_device(&nsm))) != CR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (M == 0 || N == 0) {
    st = clear_status(workspace, workspace_bytes, s);
    if (st != CR_OK || M == 0) return st;
    // no outputs: the gradient is zero
    return cuda_status(cudaMemset2DAsync(dX, static_cast<size_t>(lddx) * 2, 0, static_cast<size_t>(K) * 2,
                                         static_cast<size_t>(M), s));
  }
  uint16_t* w = reinterpret_cast<uint16_t*>(static_cast<uint8_t*>(workspace) + kWsHead);
  if (cr::use_grad_input_few(M, N, K)) {
    float* sums = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kWsHead +
                                           cr::round_up(cr::grad_input_few_operand_rows(M) * N * 2, 256));
    return static_cast<cr_status>(cr::launch_grad_input_few(
        static_cast<const uint16_t*>(dY), lddy, static_cast<const uint8_t*>(Wq), w_scale, w, sums,
        static_cast<uint16_t*>(dX), lddx, M, N, K, group, cr::grad_input_few_splits(M, N, K, kSizingSms),
        ws_status(workspace), s));
  }
  cudaError_t e = cr::launch_weight_values(static_cast<const uint8_t*>(Wq), w_scale, w, N, K, group,
                                           ws_status(workspace), s);
  if (e != cudaSuccess) return CR_ERR_CUDA;
  return static_cast<cr_status>(cr::launch_gemm_bf16(dY, lddy, w, dX, lddx, M, N, K, ws_status(workspace), nsm, s));
}

cr_status cr_read_timeouts(int* status, void* stream) {
  if (!status) return CR_ERR_INVALID_ARG;
  int nsm = 0;
  const cr_status st = static_cast<cr_status>(cr::check_current_device(&nsm));
  if (st != CR_OK) return st;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bool found = false;
  for (auto ask : {cr::lora_lost_wait, cr::ckpt_lost_wait, cr::gemm_bf16_lost_wait, cr::grad_input_few_lost_wait,
                   cr::selftest_lost_wait})
    if (ask(s, &found) != cudaSuccess) return CR_ERR_CUDA;
  *status = found ? CR_ERR_TIMEOUT : CR_OK;
  return CR_OK;
}

}  // extern "C"
