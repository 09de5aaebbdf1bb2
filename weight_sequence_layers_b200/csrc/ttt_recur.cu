// Gated linear recurrence h_t = a_t h_{t-1} + u_t per feature, forward, backward and the
// single-token step on a state cache (include/ttt.h). One thread per (sequence, feature) walks
// the tokens.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "kernels.h"
#include "simt_util.cuh"

namespace tttk {
namespace {

constexpr int kThreads = 128;

// a and 1 - a from a gate logit: both from the exponential, so that neither is a difference.
__device__ __forceinline__ void gate_of(float g, float& a, float& na) {
  const float e = expf(-fabsf(g)), big = 1.f / (1.f + e), small = e * big;
  a = g >= 0.f ? big : small;
  na = g >= 0.f ? small : big;
}

template <typename E, typename GT, bool SIG>
__global__ void __launch_bounds__(kThreads) recur_fwd_kernel(const RecurArgs a) {
  const int j = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
  if (j >= a.D) return;
  float h = a.h0 ? a.h0[(size_t)b * a.D + j] : 0.f;
  for (int t = 0; t < a.T; ++t) {
    const size_t row = (size_t)b * a.T + t, i = row * a.D + j;
    const float x = ldf(static_cast<const E*>(a.X) + i), g = ldf(static_cast<const GT*>(a.G) + i);
    float aa = g, u = x;
    if (SIG) {
      float na;
      gate_of(g, aa, na);
      u = na * x;
    }
    h = a.reset && a.reset[row] ? u : fmaf(aa, h, u);
    stf(static_cast<E*>(a.H) + i, h);
  }
  if (a.h_final) a.h_final[(size_t)b * a.D + j] = h;
}

template <typename E, typename GT, bool SIG>
__global__ void __launch_bounds__(kThreads) recur_bwd_kernel(const RecurArgs a) {
  const int j = blockIdx.x * kThreads + threadIdx.x, b = blockIdx.y;
  if (j >= a.D) return;
  const size_t bd = (size_t)b * a.D + j;
  float c = a.dh_final ? a.dh_final[bd] : 0.f;
  for (int t = a.T - 1; t >= 0; --t) {
    const size_t row = (size_t)b * a.T + t, i = row * a.D + j;
    const bool rs = a.reset && a.reset[row];
    const float g = ldf(static_cast<const GT*>(a.G) + i);
    const float Dt = ldf(static_cast<const E*>(a.dH) + i) + c;
    float prev = 0.f;
    if (!rs) prev = t > 0 ? ldf(static_cast<const E*>(a.H_in) + i - a.D) : a.h0 ? a.h0[bd] : 0.f;
    float aa = g;
    if (SIG) {
      float na;
      gate_of(g, aa, na);
      stf(static_cast<E*>(a.dX) + i, na * Dt);
      stf(static_cast<GT*>(a.dG) + i,
          Dt * (prev - ldf(static_cast<const E*>(a.X) + i)) * aa * na);
    } else {
      stf(static_cast<E*>(a.dX) + i, Dt);
      stf(static_cast<GT*>(a.dG) + i, rs ? 0.f : Dt * prev);
    }
    c = rs ? 0.f : aa * Dt;
  }
  if (a.dh0) a.dh0[bd] = c;
}

template <typename E, typename GT, bool SIG>
__global__ void __launch_bounds__(kThreads) recur_step_kernel(const RecurArgs a) {
  const int j = blockIdx.x * kThreads + threadIdx.x;
  if (j >= a.D) return;
  for (int b = 0; b < a.B; ++b) {
    const int slot = a.slots ? a.slots[b] : b;
    if (slot < 0) continue;
    if (slot >= a.n_slots) {
      if (j == 0) atomicOr(a.err, ERR_RANGE);
      continue;
    }
    const size_t i = (size_t)b * a.D + j, si = (size_t)slot * a.D + j;
    const float x = ldf(static_cast<const E*>(a.X) + i), g = ldf(static_cast<const GT*>(a.G) + i);
    float aa = g, u = x;
    if (SIG) {
      float na;
      gate_of(g, aa, na);
      u = na * x;
    }
    const float h = fmaf(aa, a.state[si], u);
    a.state[si] = h;
    stf(static_cast<E*>(a.H) + i, h);
  }
}

}  // namespace

#define RECUR_LAUNCH(kernel, grid)                                                            \
  do {                                                                                        \
    if (a.bf16 && a.sigmoid)                                                                  \
      kernel<__nv_bfloat16, __nv_bfloat16, true><<<grid, kThreads, 0, s>>>(a);                \
    else if (a.bf16)                                                                          \
      kernel<__nv_bfloat16, float, false><<<grid, kThreads, 0, s>>>(a);                       \
    else if (a.sigmoid)                                                                       \
      kernel<float, float, true><<<grid, kThreads, 0, s>>>(a);                                \
    else                                                                                      \
      kernel<float, float, false><<<grid, kThreads, 0, s>>>(a);                               \
    count_launches(1);                                                                        \
    return cudaGetLastError();                                                                \
  } while (0)

cudaError_t recur_fwd(const RecurArgs& a, cudaStream_t s) {
  RECUR_LAUNCH(recur_fwd_kernel, dim3((a.D + kThreads - 1) / kThreads, a.B));
}
cudaError_t recur_bwd(const RecurArgs& a, cudaStream_t s) {
  RECUR_LAUNCH(recur_bwd_kernel, dim3((a.D + kThreads - 1) / kThreads, a.B));
}
cudaError_t recur_step(const RecurArgs& a, cudaStream_t s) {
  RECUR_LAUNCH(recur_step_kernel, dim3((a.D + kThreads - 1) / kThreads));
}

}  // namespace tttk
