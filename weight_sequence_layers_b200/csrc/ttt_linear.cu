// Linear layer with bias, activation, multiplier and residual in its epilogue, forward and
// backward (include/ttt.h): 64 x 64 tiles on CUDA cores, bf16 operands, float32 sums.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "kernels.h"
#include "simt_util.cuh"

namespace tttk {
namespace {

using bf16 = __nv_bfloat16;
constexpr int TS = 64, TK = 16;

// acc[i][j] of rows r0 + 4 ty + i, columns c0 + 4 tx + j of A B with A(m, k), B(k, n) given by
// strides.
struct View {
  const bf16* p;
  size_t s0, s1;  // strides of the (row or column, k) indices
};
__device__ __forceinline__ void tile_product(const View& A, const View& B, int M, int N, int K,
                                             int r0, int c0, float (&acc)[4][4]) {
  __shared__ float sa[TK][TS + 1], sb[TK][TS + 1];
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
  for (int k0 = 0; k0 < K; k0 += TK) {
    for (int e = threadIdx.x; e < TS * TK; e += 256) {
      const int k = e % TK, m = e / TK;
      sa[k][m] = r0 + m < M && k0 + k < K ? ldf(A.p + (r0 + m) * A.s0 + (k0 + k) * A.s1) : 0.f;
      sb[k][m] = c0 + m < N && k0 + k < K ? ldf(B.p + (c0 + m) * B.s0 + (k0 + k) * B.s1) : 0.f;
    }
    __syncthreads();
    for (int k = 0; k < TK; ++k)
      for (int i = 0; i < 4; ++i)
        for (int j = 0; j < 4; ++j) acc[i][j] = fmaf(sa[k][4 * ty + i], sb[k][4 * tx + j], acc[i][j]);
    __syncthreads();
  }
}

__global__ void __launch_bounds__(256) linear_fwd_kernel(const LinearArgs a) {
  float acc[4][4];
  const int r0 = blockIdx.y * TS, c0 = blockIdx.x * TS;
  tile_product({static_cast<const bf16*>(a.X), (size_t)a.K, 1},
               {static_cast<const bf16*>(a.W), (size_t)a.K, 1}, a.M, a.N, a.K, r0, c0, acc);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + 4 * (threadIdx.x / 16) + i, c = c0 + 4 * (threadIdx.x % 16) + j;
      if (r >= a.M || c >= a.N) continue;
      const size_t o = (size_t)r * a.N + c;
      const float p = acc[i][j] + (a.bias ? a.bias[c] : 0.f);
      if (a.P) static_cast<bf16*>(a.P)[o] = __float2bfloat16_rn(p);
      float y = actf(a.silu, p);
      if (a.mul) y *= ldf(static_cast<const bf16*>(a.mul) + o);
      if (a.residual) y += ldf(static_cast<const bf16*>(a.residual) + o);
      static_cast<bf16*>(a.Y)[o] = __float2bfloat16_rn(y);
    }
}

__global__ void __launch_bounds__(256)
    product_kernel(View A, View B, int M, int N, int K, bf16* out) {
  float acc[4][4];
  const int r0 = blockIdx.y * TS, c0 = blockIdx.x * TS;
  tile_product(A, B, M, N, K, r0, c0, acc);
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      const int r = r0 + 4 * (threadIdx.x / 16) + i, c = c0 + 4 * (threadIdx.x % 16) + j;
      if (r < M && c < N) out[(size_t)r * N + c] = __float2bfloat16_rn(acc[i][j]);
    }
}

// dP (bf16), dmul and the bias gradient; one thread per column.
__global__ void __launch_bounds__(64) linear_dp_kernel(const LinearArgs a, bf16* dP) {
  const int c = blockIdx.x * 64 + threadIdx.x;
  if (c >= a.N) return;
  float sum = 0.f;
  for (int r = 0; r < a.M; ++r) {
    const size_t o = (size_t)r * a.N + c;
    const float dy = ldf(static_cast<const bf16*>(a.dY) + o);
    float dp = dy;
    if (a.P_in) {
      const float p = ldf(static_cast<const bf16*>(a.P_in) + o);
      if (a.dmul) static_cast<bf16*>(a.dmul)[o] = __float2bfloat16_rn(dy * actf(a.silu, p));
      dp *= act1(a.silu, p);
      if (a.mul) dp *= ldf(static_cast<const bf16*>(a.mul) + o);
    }
    dP[o] = __float2bfloat16_rn(dp);
    sum += dp;
  }
  if (a.dbias) a.dbias[c] = sum;
}

}  // namespace

size_t linear_fwd_workspace(int, int, int) { return 0; }
size_t linear_bwd_workspace(int M, int N, int) { return (size_t)M * N * 2; }

cudaError_t linear_fwd(const LinearArgs& a, cudaStream_t s) {
  linear_fwd_kernel<<<dim3((a.N + TS - 1) / TS, (a.M + TS - 1) / TS), 256, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t linear_bwd(const LinearArgs& a, cudaStream_t s) {
  bf16* dP = static_cast<bf16*>(a.ws);
  const size_t M = a.M, N = a.N, K = a.K;
  linear_dp_kernel<<<(a.N + 63) / 64, 64, 0, s>>>(a, dP);
  count_launches(1);
  if (a.dX) {
    product_kernel<<<dim3((K + TS - 1) / TS, (M + TS - 1) / TS), 256, 0, s>>>(
        {dP, N, 1}, {static_cast<const bf16*>(a.W), 1, K}, a.M, a.K, a.N,
        static_cast<bf16*>(a.dX));
    count_launches(1);
  }
  if (a.dW) {
    product_kernel<<<dim3((K + TS - 1) / TS, (N + TS - 1) / TS), 256, 0, s>>>(
        {dP, 1, N}, {static_cast<const bf16*>(a.X), 1, K}, a.N, a.K, a.M,
        static_cast<bf16*>(a.dW));
    count_launches(1);
  }
  return cudaGetLastError();
}

}  // namespace tttk
