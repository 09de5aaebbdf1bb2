// C ABI of the operators around the layer (layer norm, gated linear recurrence, linear layer):
// argument checks on the host and dispatch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include <initializer_list>

#include "../../include/ttt.h"
#include "kernels.h"

namespace tttk {
ttt_status launch_status(cudaError_t e);  // api.cu
}
using namespace tttk;

namespace {

bool aligned16(std::initializer_list<const void*> ptrs) {
  for (const void* p : ptrs)
    if (reinterpret_cast<uintptr_t>(p) & 15u) return false;
  return true;
}

ttt_status check_norm(const ttt_norm_config* c, NormArgs* a) {
  if (!c || c->B < 1 || c->H < 1 || c->T < 1 || c->d < 1) return TTT_ERR_INVALID_ARG;
  if (c->dtype != TTT_F32 && c->dtype != TTT_BF16) return TTT_ERR_INVALID_ARG;
  if (c->token_major != 0 && c->token_major != 1) return TTT_ERR_INVALID_ARG;
  if (!isfinite(c->eps) || c->eps <= 0.f) return TTT_ERR_INVALID_ARG;
  // row indices are 32-bit inside the kernels, and walks step past the last row; element offsets
  // are 64-bit
  constexpr long long kMaxRows = (1ll << 31) - (1 << 16);
  if ((long long)c->B * c->H > kMaxRows || (long long)c->B * c->H * c->T > kMaxRows)
    return TTT_ERR_INVALID_ARG;
  if ((long long)c->B * c->H * c->T * c->d > (1ll << 40)) return TTT_ERR_INVALID_ARG;
  *a = NormArgs{};
  a->B = c->B; a->H = c->H; a->T = c->T; a->d = c->d;
  a->bf16 = c->dtype == TTT_BF16;
  a->token_major = c->token_major != 0;
  a->eps = c->eps;
  return norm_supported(*a) ? TTT_OK : TTT_ERR_UNSUPPORTED;
}

ttt_status check_recur(const ttt_recur_config* c, RecurArgs* a) {
  if (!c || c->B < 1 || c->T < 1 || c->D < 1) return TTT_ERR_INVALID_ARG;
  if (c->dtype != TTT_F32 && c->dtype != TTT_BF16) return TTT_ERR_INVALID_ARG;
  if (c->gate != TTT_GATE_DECAY && c->gate != TTT_GATE_SIGMOID) return TTT_ERR_INVALID_ARG;
  if ((long long)c->B * c->T >= (1ll << 31)) return TTT_ERR_INVALID_ARG;
  // blocks of features reach past the last one: their indices stay below 2^31
  if (c->D > 2147483647 - 512) return TTT_ERR_INVALID_ARG;
  if ((long long)c->B * c->T * c->D > (1ll << 40)) return TTT_ERR_INVALID_ARG;
  *a = RecurArgs{};
  a->B = c->B; a->T = c->T; a->D = c->D;
  a->bf16 = c->dtype == TTT_BF16;
  a->sigmoid = c->gate == TTT_GATE_SIGMOID;
  return TTT_OK;
}

ttt_status check_linear(int M, int N, int K, int act) {
  if (M < 1 || N < 1 || K < 1) return TTT_ERR_INVALID_ARG;
  if (act != TTT_ACT_ID && act != TTT_ACT_SILU) return TTT_ERR_INVALID_ARG;
  // tiles reach past the last row: their indices stay below 2^31
  constexpr int kMax = 2147483647 - 512;
  if (M > kMax || N > kMax || K > kMax) return TTT_ERR_INVALID_ARG;
  const long long lim = 1ll << 40;
  if ((long long)M * N > lim || (long long)M * K > lim || (long long)N * K > lim)
    return TTT_ERR_INVALID_ARG;
  // rows of every matrix start on 16-byte boundaries (the TMA's row stride)
  return N % 8 || K % 8 ? TTT_ERR_UNSUPPORTED : TTT_OK;
}

}  // namespace

extern "C" {

ttt_status ttt_norm_fwd(const ttt_norm_config* cfg, const void* X, const void* residual,
                        const float* weight, const float* bias, void* Y, void* S, float* mean,
                        float* rstd, void* stream) {
  NormArgs a;
  const ttt_status st = check_norm(cfg, &a);
  if (st != TTT_OK) return st;
  if (!X || !Y || (S && !residual)) return TTT_ERR_INVALID_ARG;
  if (!aligned16({X, residual, weight, bias, Y, S, mean, rstd})) return TTT_ERR_ALIGNMENT;
  a.X = X; a.residual = residual; a.weight = weight; a.bias = bias; a.Y = Y; a.S = S;
  a.mean = mean; a.rstd = rstd;
  a.err = current_error_word();
  if (!a.err) return TTT_ERR_CUDA;
  return launch_status(norm_fwd(a, static_cast<cudaStream_t>(stream)));
}

size_t ttt_norm_bwd_workspace_bytes(const ttt_norm_config* cfg) {
  NormArgs a;
  return check_norm(cfg, &a) == TTT_OK ? norm_bwd_workspace(a) : (size_t)-1;
}

ttt_status ttt_norm_bwd(const ttt_norm_config* cfg, const void* S, const float* weight,
                        const float* mean, const float* rstd, const void* dY, const void* dS,
                        void* dX, float* dweight, float* dbias, void* workspace,
                        size_t workspace_bytes, void* stream) {
  NormArgs a;
  const ttt_status st = check_norm(cfg, &a);
  if (st != TTT_OK) return st;
  if (!S || !mean || !rstd || !dY || !dX) return TTT_ERR_INVALID_ARG;
  if (!aligned16({S, weight, mean, rstd, dY, dS, dX, dweight, dbias, workspace}))
    return TTT_ERR_ALIGNMENT;
  const size_t need = dweight || dbias ? norm_bwd_workspace(a) : 0;
  if (need && (!workspace || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  a.X = S; a.weight = weight; a.mean = const_cast<float*>(mean);
  a.rstd = const_cast<float*>(rstd); a.dY = dY; a.dS = dS; a.dX = dX; a.dweight = dweight;
  a.dbias = dbias; a.ws = workspace;
  a.err = current_error_word();
  if (!a.err) return TTT_ERR_CUDA;
  return launch_status(norm_bwd(a, static_cast<cudaStream_t>(stream)));
}

ttt_status ttt_recur_fwd(const ttt_recur_config* cfg, const void* X, const void* G,
                         const unsigned char* reset, const float* h0, void* H, float* h_final,
                         void* stream) {
  RecurArgs a;
  const ttt_status st = check_recur(cfg, &a);
  if (st != TTT_OK) return st;
  if (!X || !G || !H) return TTT_ERR_INVALID_ARG;
  if (!aligned16({X, G, reset, h0, H, h_final})) return TTT_ERR_ALIGNMENT;
  a.X = X; a.G = G; a.reset = reset; a.h0 = h0; a.H = H; a.h_final = h_final;
  a.err = current_error_word();
  if (!a.err) return TTT_ERR_CUDA;
  return launch_status(recur_fwd(a, static_cast<cudaStream_t>(stream)));
}

ttt_status ttt_recur_bwd(const ttt_recur_config* cfg, const void* X, const void* G,
                         const unsigned char* reset, const float* h0, const void* H,
                         const void* dH, const float* dh_final, void* dX, void* dG, float* dh0,
                         void* stream) {
  RecurArgs a;
  const ttt_status st = check_recur(cfg, &a);
  if (st != TTT_OK) return st;
  if ((a.sigmoid && !X) || !G || !H || !dH || !dX || !dG) return TTT_ERR_INVALID_ARG;
  if (!aligned16({X, G, reset, h0, H, dH, dh_final, dX, dG, dh0})) return TTT_ERR_ALIGNMENT;
  a.X = X; a.G = G; a.reset = reset; a.h0 = h0; a.H_in = H; a.dH = dH; a.dh_final = dh_final;
  a.dX = dX; a.dG = dG; a.dh0 = dh0;
  a.err = current_error_word();
  if (!a.err) return TTT_ERR_CUDA;
  return launch_status(recur_bwd(a, static_cast<cudaStream_t>(stream)));
}

ttt_status ttt_recur_step(const ttt_recur_config* cfg, const void* X, const void* G,
                          const int* slots, int n_slots, float* state, void* Y, void* stream) {
  RecurArgs a;
  const ttt_status st = check_recur(cfg, &a);
  if (st != TTT_OK) return st;
  if (cfg->T != 1 || n_slots < 1 || !X || !G || !state || !Y) return TTT_ERR_INVALID_ARG;
  if (!slots && n_slots < cfg->B) return TTT_ERR_INVALID_ARG;
  // every row looks for its slot among all rows'
  if (slots && cfg->B > (1 << 20)) return TTT_ERR_UNSUPPORTED;
  if (!aligned16({X, G, slots, state, Y})) return TTT_ERR_ALIGNMENT;
  a.err = current_error_word();
  if (!a.err) return TTT_ERR_CUDA;
  a.X = X; a.G = G; a.slots = slots; a.n_slots = n_slots; a.state = state; a.H = Y;
  return launch_status(recur_step(a, static_cast<cudaStream_t>(stream)));
}

size_t ttt_linear_workspace_bytes(int M, int N, int K, int for_bwd) {
  if (check_linear(M, N, K, TTT_ACT_ID) != TTT_OK || (for_bwd != 0 && for_bwd != 1))
    return (size_t)-1;
  return for_bwd ? linear_bwd_workspace(M, N, K) : linear_fwd_workspace(M, N, K);
}

ttt_status ttt_linear_fwd(int M, int N, int K, int act, const void* X, const void* W,
                          const float* bias, const void* mul, const void* residual, void* Y,
                          void* P, void* workspace, size_t workspace_bytes, void* stream) {
  const ttt_status st = check_linear(M, N, K, act);
  if (st != TTT_OK) return st;
  if (!X || !W || !Y) return TTT_ERR_INVALID_ARG;
  if (!aligned16({X, W, bias, mul, residual, Y, P, workspace})) return TTT_ERR_ALIGNMENT;
  const size_t need = linear_fwd_workspace(M, N, K);
  if (need && (!workspace || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  LinearArgs a{};
  a.M = M; a.N = N; a.K = K; a.silu = act == TTT_ACT_SILU;
  a.X = X; a.W = W; a.bias = bias; a.mul = mul; a.residual = residual; a.Y = Y; a.P = P;
  a.ws = workspace;
  a.err = current_error_word();
  if (!a.err) return TTT_ERR_CUDA;
  return launch_status(linear_fwd(a, static_cast<cudaStream_t>(stream)));
}

ttt_status ttt_linear_bwd(int M, int N, int K, int act, const void* X, const void* W,
                          const void* P, const void* mul, const void* dY, void* dX, void* dW,
                          float* dbias, void* dmul, void* workspace, size_t workspace_bytes,
                          void* stream) {
  const ttt_status st = check_linear(M, N, K, act);
  if (st != TTT_OK) return st;
  if (!dY || (!dX && !dW && !dbias && !dmul)) return TTT_ERR_INVALID_ARG;
  if ((dX && !W) || (dW && !X) || (dmul && !mul)) return TTT_ERR_INVALID_ARG;
  if (!P && (act != TTT_ACT_ID || mul)) return TTT_ERR_INVALID_ARG;
  if (!aligned16({X, W, P, mul, dY, dX, dW, dbias, dmul, workspace})) return TTT_ERR_ALIGNMENT;
  const size_t need = linear_bwd_workspace(M, N, K);
  if (need && (!workspace || workspace_bytes < need)) return TTT_ERR_WORKSPACE;
  LinearArgs a{};
  a.M = M; a.N = N; a.K = K; a.silu = act == TTT_ACT_SILU;
  a.X = X; a.W = W; a.P_in = act != TTT_ACT_ID || mul ? P : nullptr; a.mul = mul; a.dY = dY;
  a.dX = dX; a.dW = dW; a.dbias = dbias; a.dmul = dmul; a.ws = workspace;
  a.err = current_error_word();
  if (!a.err) return TTT_ERR_CUDA;
  return launch_status(linear_bwd(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
