// Layer norm over rows of d features with one weight group per head, forward and backward
// (include/ttt.h). One CTA per row, three passes over it; the weight gradients with one thread
// per feature over all rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "simt_util.cuh"

namespace tttk {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float block_sum(float v, float* red) {
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  __syncthreads();
  if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
  __syncthreads();
  float t = 0.f;
  for (int w = 0; w < kThreads / 32; ++w) t += red[w];
  return t;
}

__device__ __forceinline__ size_t y_row(const NormArgs& a, int row) {
  if (!a.token_major) return row;
  const int t = row % a.T, bh = row / a.T;
  return ((size_t)(bh / a.H) * a.T + t) * a.H + bh % a.H;
}

template <typename E>
__global__ void __launch_bounds__(kThreads) norm_fwd_kernel(const NormArgs a) {
  __shared__ float red[kThreads / 32];
  const int row = blockIdx.x, h = (row / a.T) % a.H;
  const E* x = static_cast<const E*>(a.X) + (size_t)row * a.d;
  const E* r = a.residual ? static_cast<const E*>(a.residual) + (size_t)row * a.d : nullptr;
  E* y = static_cast<E*>(a.Y) + y_row(a, row) * a.d;
  E* so = a.S ? static_cast<E*>(a.S) + (size_t)row * a.d : nullptr;
  auto s_at = [&](int j) { return ldf(x + j) + (r ? ldf(r + j) : 0.f); };
  float sum = 0.f;
  for (int j = threadIdx.x; j < a.d; j += kThreads) sum += s_at(j);
  const float mean = block_sum(sum, red) / a.d;
  float sq = 0.f;
  for (int j = threadIdx.x; j < a.d; j += kThreads) {
    const float c = s_at(j) - mean;
    sq += c * c;
  }
  const float rstd = 1.f / sqrtf(block_sum(sq, red) / a.d + a.eps);
  for (int j = threadIdx.x; j < a.d; j += kThreads) {
    const float s = s_at(j), w = a.weight ? a.weight[(size_t)h * a.d + j] : 1.f;
    stf(y + j, (s - mean) * rstd * w + (a.bias ? a.bias[(size_t)h * a.d + j] : 0.f));
    if (so) stf(so + j, s);
  }
  if (threadIdx.x == 0) {
    if (a.mean) a.mean[row] = mean;
    if (a.rstd) a.rstd[row] = rstd;
  }
}

template <typename E>
__global__ void __launch_bounds__(kThreads) norm_bwd_kernel(const NormArgs a) {
  __shared__ float red[kThreads / 32];
  const int row = blockIdx.x, h = (row / a.T) % a.H;
  const E* x = static_cast<const E*>(a.X) + (size_t)row * a.d;
  const E* dy = static_cast<const E*>(a.dY) + y_row(a, row) * a.d;
  const float mean = a.mean[row], rstd = a.rstd[row];
  auto g_at = [&](int j) { return ldf(dy + j) * (a.weight ? a.weight[(size_t)h * a.d + j] : 1.f); };
  float s1 = 0.f, s2 = 0.f;
  for (int j = threadIdx.x; j < a.d; j += kThreads) {
    s1 += g_at(j);
    s2 += g_at(j) * (ldf(x + j) - mean) * rstd;
  }
  const float c1 = block_sum(s1, red) / a.d, c2 = block_sum(s2, red) / a.d;
  for (int j = threadIdx.x; j < a.d; j += kThreads) {
    const size_t i = (size_t)row * a.d + j;
    const float xh = (ldf(x + j) - mean) * rstd;
    stf(static_cast<E*>(a.dX) + i, rstd * (g_at(j) - c1 - xh * c2) +
                                       (a.dS ? ldf(static_cast<const E*>(a.dS) + i) : 0.f));
  }
}

template <typename E>
__global__ void __launch_bounds__(kThreads) norm_dw_kernel(const NormArgs a) {
  const int j = blockIdx.x * kThreads + threadIdx.x, h = blockIdx.y;
  if (j >= a.d) return;
  float dw = 0.f, db = 0.f;
  for (int b = 0; b < a.B; ++b)
    for (int t = 0; t < a.T; ++t) {
      const int row = (b * a.H + h) * a.T + t;
      const float g = ldf(static_cast<const E*>(a.dY) + y_row(a, row) * a.d + j);
      db += g;
      dw += g * (ldf(static_cast<const E*>(a.X) + (size_t)row * a.d + j) - a.mean[row]) *
            a.rstd[row];
    }
  if (a.dweight) a.dweight[(size_t)h * a.d + j] = dw;
  if (a.dbias) a.dbias[(size_t)h * a.d + j] = db;
}

}  // namespace

bool norm_supported(const NormArgs& a) { return a.d <= 16384; }
size_t norm_bwd_workspace(const NormArgs&) { return 0; }

cudaError_t norm_fwd(const NormArgs& a, cudaStream_t s) {
  const int rows = a.B * a.H * a.T;
  if (a.bf16) norm_fwd_kernel<__nv_bfloat16><<<rows, kThreads, 0, s>>>(a);
  else norm_fwd_kernel<float><<<rows, kThreads, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t norm_bwd(const NormArgs& a, cudaStream_t s) {
  const int rows = a.B * a.H * a.T;
  const dim3 gw((a.d + kThreads - 1) / kThreads, a.H);
  // the weight gradients first: dX may be dS, never dY or S
  if (a.dweight || a.dbias) {
    if (a.bf16) norm_dw_kernel<__nv_bfloat16><<<gw, kThreads, 0, s>>>(a);
    else norm_dw_kernel<float><<<gw, kThreads, 0, s>>>(a);
    count_launches(1);
  }
  if (a.bf16) norm_bwd_kernel<__nv_bfloat16><<<rows, kThreads, 0, s>>>(a);
  else norm_bwd_kernel<float><<<rows, kThreads, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace tttk
