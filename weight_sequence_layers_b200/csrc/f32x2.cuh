// Pairs of float32 in one instruction (add, mul, fma on f32x2). Streaming kernels on bf16 data are
// bound by the instructions they issue before they are by HBM (a 16-byte access holds eight
// values), and a pair costs one issue slot.
#pragma once
#include <cuda_runtime.h>

namespace tttk {

__device__ __forceinline__ float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

}  // namespace tttk
