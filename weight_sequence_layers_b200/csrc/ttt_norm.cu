// Layer norm over rows of d features with one weight group per head, forward and backward
// (include/ttt.h).
//
// Both passes are bound by HBM: a row is read once into registers, reduced twice there (the
// mean, then the centred squares: no cancellation for rows with a large mean) and written once.
// A row belongs to a group of threads: 8 to 32 lanes of a warp for narrow rows (several rows
// per CTA, sums by shuffles alone), the whole CTA for wide ones. CTA (h, s) walks a contiguous
// run of the rows of head h, so that the head's weights stay in registers, and loads the next
// row before it reduces the current one.
//
// The backward keeps its share of dweight and dbias in registers over its run; the CTAs' shares
// go to the workspace and a second kernel adds them in a fixed order (no atomics). That kernel
// starts while the first one drains (programmatic launch) and waits for it on the device.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "kernels.h"
#include "simt_util.cuh"

namespace tttk {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kSMs = 148;
constexpr int kNarrowThreads = 128;  // CTA of the narrow-row kernels

// VEC elements of a row: one 16-byte access, or one element where the width does not keep rows
// on 16-byte boundaries. Plain (coherent) loads: S may be X or residual, dX may be dS.
template <typename E, int VEC>
struct Pack;
template <>
struct Pack<bf16, 8> {
  uint4 r;
  __device__ __forceinline__ void load(const bf16* p) {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = __uint_as_float(w[k] << 16);
      v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(bf16* p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
      w[k] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Pack<float, 4> {
  float4 r;
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];"
                 : "=f"(r.x), "=f"(r.y), "=f"(r.z), "=f"(r.w) : "l"(p) : "memory");
  }
  __device__ __forceinline__ void get(float (&v)[4]) const {
    v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&v)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <typename E>
struct Pack<E, 1> {
  E r;
  __device__ __forceinline__ void load(const E* p) { r = *p; }
  __device__ __forceinline__ void get(float (&v)[1]) const { v[0] = ldf(&r); }
  static __device__ __forceinline__ void store(E* p, const float (&v)[1]) { stf(p, v[0]); }
};

template <int VEC>
__device__ __forceinline__ void load_f32(const float* p, float (&v)[VEC]) {
  if constexpr (VEC == 1) {
    v[0] = *p;
  } else {
#pragma unroll
    for (int k = 0; k < VEC; k += 4) {
      const float4 f = *reinterpret_cast<const float4*>(p + k);
      v[k] = f.x; v[k + 1] = f.y; v[k + 2] = f.z; v[k + 3] = f.w;
    }
  }
}

// How a launch cuts the rows: head h's B T rows into S runs of L, CTA h S + s.
struct Split {
  int S, L;
};

struct Rows {
  int lo, hi, h, T, H, d;
  bool token_major;
  // offset of the head's i-th row in the [B, H, T, d] tensors, and in Y and dY
  __device__ __forceinline__ size_t row(int i) const {
    const int b = i / T, t = i - b * T;
    return ((size_t)b * H + h) * T + t;
  }
  __device__ __forceinline__ size_t yrow(int i) const {
    return token_major ? (size_t)i * H + h : row(i);  // i = b T + t
  }
};
__device__ __forceinline__ Rows rows_of(const NormArgs& a, const Split& sp) {
  Rows r;
  r.h = blockIdx.x / sp.S;
  const int s = blockIdx.x - r.h * sp.S;
  r.lo = (int)min((long long)s * sp.L, (long long)a.B * a.T);
  r.hi = (int)min((long long)r.lo + sp.L, (long long)a.B * a.T);
  r.T = a.T; r.H = a.H; r.d = a.d;
  r.token_major = a.token_major;
  return r;
}

// Sums v over the row's group: G lanes of a warp, or (G = 0) the CTA through red[buf]. The two
// buffers alternate, so that one barrier per sum is enough: nobody writes a buffer before all
// have passed the barrier of the sum after the one that last read it.
template <int G>
__device__ __forceinline__ float group_sum(float v, float* red) {
#pragma unroll
  for (int o = (G ? G : 32) / 2; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if constexpr (G == 0) {
    const int nw = blockDim.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = lane < nw ? red[lane] : 0.f;
#pragma unroll
    for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  }
  return v;
}

// E: storage type; VEC: elements of one access; NV: accesses per thread; G: lanes per row (0:
// the CTA).
template <typename E, int VEC, int NV, int G>
__global__ void __launch_bounds__(G ? kNarrowThreads : 512)
    norm_fwd_kernel(const __grid_constant__ NormArgs a, const Split sp) {
  __shared__ float red[2][32];
  const Rows R = rows_of(a, sp);
  const int gsz = G ? G : blockDim.x, ngrp = G ? kNarrowThreads / G : 1;
  const int grp = G ? threadIdx.x / gsz : 0, tid = G ? threadIdx.x % gsz : threadIdx.x;
  const int d = a.d;
  const float inv_d = 1.f / (float)d;
  const E* X = static_cast<const E*>(a.X);
  const E* Rs = static_cast<const E*>(a.residual);
  E* Y = static_cast<E*>(a.Y);
  E* S = static_cast<E*>(a.S);
  float w[NV][VEC], bb[NV][VEC];
  bool ok[NV];
  int col[NV];
  Pack<E, VEC> px[NV], pr[NV];
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    col[n] = (tid + n * gsz) * VEC;
    ok[n] = col[n] < d;
  }
  auto fetch = [&](int i) {
    if (i >= R.hi) return;
    const size_t o = R.row(i) * d;
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (ok[n]) {
        px[n].load(X + o + col[n]);
        if (Rs) pr[n].load(Rs + o + col[n]);
      }
  };
  fetch(R.lo + grp);
#pragma unroll
  for (int n = 0; n < NV; ++n) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) { w[n][k] = 1.f; bb[n][k] = 0.f; }
    if (ok[n]) {
      if (a.weight) load_f32<VEC>(a.weight + (size_t)R.h * d + col[n], w[n]);
      if (a.bias) load_f32<VEC>(a.bias + (size_t)R.h * d + col[n], bb[n]);
    }
  }
  for (int i0 = R.lo; i0 < R.hi; i0 += ngrp) {  // uniform over the CTA
    const int i = i0 + grp;
    const bool live = i < R.hi;
    float v[NV][VEC];
    float sum = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
#pragma unroll
      for (int k = 0; k < VEC; ++k) v[n][k] = 0.f;
      if (live && ok[n]) {
        px[n].get(v[n]);
        if (Rs) {
          float r[VEC];
          pr[n].get(r);
#pragma unroll
          for (int k = 0; k < VEC; ++k) v[n][k] += r[k];
          if (S) Pack<E, VEC>::store(S + R.row(i) * d + col[n], v[n]);
        }
#pragma unroll
        for (int k = 0; k < VEC; ++k) sum += v[n][k];
      }
    }
    fetch(i + ngrp);
    const float mean = group_sum<G>(sum, red[0]) * inv_d;
    float sq = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (ok[n])
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          v[n][k] -= mean;
          sq = fmaf(v[n][k], v[n][k], sq);
        }
    const float rstd = 1.f / sqrtf(group_sum<G>(sq, red[1]) * inv_d + a.eps);
    if (!live) continue;
    E* y = Y + R.yrow(i) * d;
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (ok[n]) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) v[n][k] = fmaf(v[n][k] * rstd, w[n][k], bb[n][k]);
        Pack<E, VEC>::store(y + col[n], v[n]);
      }
    if (tid == 0) {
      if (a.mean) a.mean[R.row(i)] = mean;
      if (a.rstd) a.rstd[R.row(i)] = rstd;
    }
  }
}

// The CTA's shares of dweight and dbias go to dw0 + s ldp and db0 + s ldp (S = 1: the outputs
// themselves).
struct Partials {
  float *dw0, *db0;  // each nullable
  size_t ldp;
};

template <typename E, int VEC, int NV, int G>
__global__ void __launch_bounds__(G ? kNarrowThreads : 512)
    norm_bwd_kernel(const __grid_constant__ NormArgs a, const Split sp, const Partials pt) {
  __shared__ float red[2][2][32];
  __shared__ float join[G ? 2 * kNarrowThreads * NV * VEC : 1];
  asm volatile("griddepcontrol.launch_dependents;");
  const Rows R = rows_of(a, sp);
  const int gsz = G ? G : blockDim.x, ngrp = G ? kNarrowThreads / G : 1;
  const int grp = G ? threadIdx.x / gsz : 0, tid = G ? threadIdx.x % gsz : threadIdx.x;
  const int d = a.d;
  const float inv_d = 1.f / (float)d;
  const E* X = static_cast<const E*>(a.X);
  const E* dY = static_cast<const E*>(a.dY);
  const E* dS = static_cast<const E*>(a.dS);
  E* dX = static_cast<E*>(a.dX);
  float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
  bool ok[NV];
  int col[NV];
  Pack<E, VEC> px[NV], py[NV], ps[NV];
  float nmean = 0.f, nrstd = 0.f;
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    col[n] = (tid + n * gsz) * VEC;
    ok[n] = col[n] < d;
  }
  auto fetch = [&](int i) {
    if (i >= R.hi) return;
    const size_t row = R.row(i), o = row * d, oy = R.yrow(i) * d;
    nmean = a.mean[row];
    nrstd = a.rstd[row];
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (ok[n]) {
        px[n].load(X + o + col[n]);
        py[n].load(dY + oy + col[n]);
        if (dS) ps[n].load(dS + o + col[n]);
      }
  };
  fetch(R.lo + grp);
#pragma unroll
  for (int n = 0; n < NV; ++n) {
#pragma unroll
    for (int k = 0; k < VEC; ++k) { w[n][k] = 1.f; dw[n][k] = db[n][k] = 0.f; }
    if (ok[n] && a.weight) load_f32<VEC>(a.weight + (size_t)R.h * d + col[n], w[n]);
  }
  int it = 0;
  for (int i0 = R.lo; i0 < R.hi; i0 += ngrp, ++it) {  // uniform over the CTA
    const int i = i0 + grp;
    const bool live = i < R.hi;
    const float mean = nmean, rstd = nrstd;
    float xh[NV][VEC], g[NV][VEC], s[NV][VEC];
    float s1 = 0.f, s2 = 0.f;
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (live && ok[n]) {
        px[n].get(xh[n]);
        py[n].get(g[n]);
        if (dS) ps[n].get(s[n]);
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          xh[n][k] = (xh[n][k] - mean) * rstd;
          db[n][k] += g[n][k];
          dw[n][k] = fmaf(g[n][k], xh[n][k], dw[n][k]);
          g[n][k] *= w[n][k];
          s1 += g[n][k];
          s2 = fmaf(g[n][k], xh[n][k], s2);
        }
      }
    fetch(i + ngrp);
#pragma unroll
    for (int o = (G ? G : 32) / 2; o; o >>= 1) {
      s1 += __shfl_xor_sync(~0u, s1, o);
      s2 += __shfl_xor_sync(~0u, s2, o);
    }
    if constexpr (G == 0) {  // both sums behind one barrier
      const int nw = blockDim.x >> 5, lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
      if (lane == 0) { red[it & 1][0][wp] = s1; red[it & 1][1][wp] = s2; }
      __syncthreads();
      s1 = lane < nw ? red[it & 1][0][lane] : 0.f;
      s2 = lane < nw ? red[it & 1][1][lane] : 0.f;
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        s1 += __shfl_xor_sync(~0u, s1, o);
        s2 += __shfl_xor_sync(~0u, s2, o);
      }
    }
    if (!live) continue;
    const float c1 = s1 * inv_d, c2 = s2 * inv_d;
    E* dx = dX + R.row(i) * d;
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (ok[n]) {
#pragma unroll
        for (int k = 0; k < VEC; ++k) {
          const float v = rstd * (g[n][k] - c1 - xh[n][k] * c2);
          g[n][k] = dS ? v + s[n][k] : v;
        }
        Pack<E, VEC>::store(dx + col[n], g[n]);
      }
  }
  if (!pt.dw0 && !pt.db0) return;
  const size_t base = (size_t)(blockIdx.x - R.h * sp.S) * pt.ldp + (size_t)R.h * d;
  if constexpr (G == 0) {
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (ok[n]) {
        if (pt.dw0)
#pragma unroll
          for (int k = 0; k < VEC; ++k) pt.dw0[base + col[n] + k] = dw[n][k];
        if (pt.db0)
#pragma unroll
          for (int k = 0; k < VEC; ++k) pt.db0[base + col[n] + k] = db[n][k];
      }
  } else {
    constexpr int W = G * NV * VEC;  // columns of a group, padded
#pragma unroll
    for (int n = 0; n < NV; ++n)
#pragma unroll
      for (int k = 0; k < VEC; ++k) {
        join[grp * W + col[n] + k] = dw[n][k];
        join[kNarrowThreads * NV * VEC + grp * W + col[n] + k] = db[n][k];
      }
    __syncthreads();
    for (int j = threadIdx.x; j < d; j += kNarrowThreads) {
      float tw = 0.f, tb = 0.f;
#pragma unroll
      for (int g = 0; g < kNarrowThreads / G; ++g) {
        tw += join[g * W + j];
        tb += join[kNarrowThreads * NV * VEC + g * W + j];
      }
      if (pt.dw0) pt.dw0[base + j] = tw;
      if (pt.db0) pt.db0[base + j] = tb;
    }
  }
}

// dweight[j] = sum over s of part[s][0][j], dbias likewise from part[s][1]: 32 columns per CTA,
// 8 warps over s.
constexpr int kJoinWarps = 8;
__global__ void __launch_bounds__(32 * kJoinWarps)
    norm_join_kernel(const float* part, int S, size_t cols, float* dweight, float* dbias) {
  __shared__ float red[kJoinWarps][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x % 32, wp = threadIdx.x / 32;
  const size_t c = (size_t)blockIdx.x * 32 + lane;  // column of [dweight | dbias]
  float t0 = 0.f, t1 = 0.f, t2 = 0.f, t3 = 0.f;
  if (c < 2 * cols) {
    int s = wp;
    for (; s + 3 * kJoinWarps < S; s += 4 * kJoinWarps) {
      t0 += part[(size_t)s * 2 * cols + c];
      t1 += part[(size_t)(s + kJoinWarps) * 2 * cols + c];
      t2 += part[(size_t)(s + 2 * kJoinWarps) * 2 * cols + c];
      t3 += part[(size_t)(s + 3 * kJoinWarps) * 2 * cols + c];
    }
    for (; s < S; s += kJoinWarps) t0 += part[(size_t)s * 2 * cols + c];
  }
  red[wp][lane] = (t0 + t1) + (t2 + t3);
  __syncthreads();
  if (wp == 0 && c < 2 * cols) {
    float t = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k) t += red[k][lane];
    float* out = c < cols ? dweight : dbias;
    if (out) out[c < cols ? c : c - cols] = t;
  }
}

// ------------------------------------------------------------------------------ launch rules
struct Shape {
  int vec, nv, g, threads;  // g = 0: one CTA of `threads` per row
};
// Narrow rows take as few lanes as hold the row in at most two (scalar: eight) accesses each;
// wide rows one access per thread up to 512 threads, then more accesses.
Shape shape_of(const NormArgs& a) {
  const int v = a.bf16 ? 8 : 4;
  Shape s;
  s.vec = a.d % v == 0 ? v : 1;
  const int n = (a.d + s.vec - 1) / s.vec;
  s.threads = kNarrowThreads;
  if (s.vec > 1) {
    if (n <= 8) { s.g = 8; s.nv = 1; return s; }
    if (n <= 16) { s.g = 16; s.nv = 1; return s; }
    if (n <= 32) { s.g = 32; s.nv = 1; return s; }
    if (n <= 64) { s.g = 32; s.nv = 2; return s; }
    s.nv = n <= 512 ? 1 : n <= 1024 ? 2 : n <= 2048 ? 4 : 8;
  } else {
    if (n <= 32) { s.g = 32; s.nv = 1; return s; }
    if (n <= 128) { s.g = 32; s.nv = 4; return s; }
    if (n <= 256) { s.g = 32; s.nv = 8; return s; }
    s.nv = n <= 2048 ? 4 : n <= 4096 ? 8 : 32;
  }
  s.g = 0;
  s.threads = ((n + s.nv - 1) / s.nv + 31) / 32 * 32;
  return s;
}

// CTAs that run at once, from the threads of an SM that the kernels' registers allow.
Split split_of(const NormArgs& a, const Shape& sh, int threads_per_sm, int min_rows) {
  const long long bt = (long long)a.B * a.T;
  const int ngrp = sh.g ? kNarrowThreads / sh.g : 1;
  const long long slots = (long long)kSMs * std::max(1, threads_per_sm / sh.threads);
  // every SM gets a CTA before any run is longer than one row per group; beyond that a run has
  // at least min_rows per group
  const long long one = (bt + ngrp - 1) / ngrp, few = (one + min_rows - 1) / min_rows;
  long long S = std::min(std::max(1ll, slots / a.H),
                         std::max(few, std::min(one, (long long)(kSMs + a.H - 1) / a.H)));
  Split sp;
  sp.L = (int)((bt + S - 1) / S);
  sp.L = (int)std::min(bt, (long long)(sp.L + ngrp - 1) / ngrp * ngrp);
  sp.S = (int)((bt + sp.L - 1) / sp.L);
  return sp;
}
Split fwd_split(const NormArgs& a, const Shape& sh) { return split_of(a, sh, 1024, 1); }
Split bwd_split(const NormArgs& a, const Shape& sh) { return split_of(a, sh, 640, 4); }

template <typename E, int VEC, int NV, int G>
void launch_fwd(const NormArgs& a, const Shape& sh, cudaStream_t s) {
  const Split sp = fwd_split(a, sh);
  norm_fwd_kernel<E, VEC, NV, G><<<(unsigned)a.H * sp.S, sh.threads, 0, s>>>(a, sp);
}
template <typename E, int VEC, int NV, int G>
void launch_bwd(const NormArgs& a, const Shape& sh, cudaStream_t s) {
  const Split sp = bwd_split(a, sh);
  const size_t cols = (size_t)a.H * a.d;
  Partials pt{};
  if (a.dweight || a.dbias) {
    float* ws = static_cast<float*>(a.ws);
    pt = sp.S == 1 ? Partials{a.dweight, a.dbias, 0} : Partials{ws, ws + cols, 2 * cols};
  }
  norm_bwd_kernel<E, VEC, NV, G><<<(unsigned)a.H * sp.S, sh.threads, 0, s>>>(a, sp, pt);
}

// Calls F::run<E, VEC, NV, G>(a, sh, s) for the shape's instance.
#define NORM_DISPATCH(F)                                                                     \
  do {                                                                                       \
    const Shape sh = shape_of(a);                                                            \
    if (a.bf16 && sh.vec == 8) {                                                             \
      if (sh.g == 8) F<bf16, 8, 1, 8>(a, sh, s);                                             \
      else if (sh.g == 16) F<bf16, 8, 1, 16>(a, sh, s);                                      \
      else if (sh.g == 32 && sh.nv == 1) F<bf16, 8, 1, 32>(a, sh, s);                        \
      else if (sh.g == 32) F<bf16, 8, 2, 32>(a, sh, s);                                      \
      else if (sh.nv == 1) F<bf16, 8, 1, 0>(a, sh, s);                                       \
      else if (sh.nv == 2) F<bf16, 8, 2, 0>(a, sh, s);                                       \
      else F<bf16, 8, 4, 0>(a, sh, s);                                                       \
    } else if (!a.bf16 && sh.vec == 4) {                                                     \
      if (sh.g == 8) F<float, 4, 1, 8>(a, sh, s);                                            \
      else if (sh.g == 16) F<float, 4, 1, 16>(a, sh, s);                                     \
      else if (sh.g == 32 && sh.nv == 1) F<float, 4, 1, 32>(a, sh, s);                       \
      else if (sh.g == 32) F<float, 4, 2, 32>(a, sh, s);                                     \
      else if (sh.nv == 1) F<float, 4, 1, 0>(a, sh, s);                                      \
      else if (sh.nv == 2) F<float, 4, 2, 0>(a, sh, s);                                      \
      else if (sh.nv == 4) F<float, 4, 4, 0>(a, sh, s);                                      \
      else F<float, 4, 8, 0>(a, sh, s);                                                      \
    } else if (a.bf16) {                                                                     \
      NORM_SCALAR(F, bf16);                                                                  \
    } else {                                                                                 \
      NORM_SCALAR(F, float);                                                                 \
    }                                                                                        \
  } while (0)
#define NORM_SCALAR(F, E)                                                                    \
  do {                                                                                       \
    if (sh.g == 32 && sh.nv == 1) F<E, 1, 1, 32>(a, sh, s);                                  \
    else if (sh.g == 32 && sh.nv == 4) F<E, 1, 4, 32>(a, sh, s);                             \
    else if (sh.g == 32) F<E, 1, 8, 32>(a, sh, s);                                           \
    else if (sh.nv == 4) F<E, 1, 4, 0>(a, sh, s);                                            \
    else if (sh.nv == 8) F<E, 1, 8, 0>(a, sh, s);                                            \
    else F<E, 1, 32, 0>(a, sh, s);                                                           \
  } while (0)

}  // namespace

bool norm_supported(const NormArgs& a) { return a.d <= 16384; }

size_t norm_bwd_workspace(const NormArgs& a) {
  const Split sp = bwd_split(a, shape_of(a));
  return sp.S == 1 ? 0 : (size_t)sp.S * 2 * a.H * a.d * sizeof(float);
}

cudaError_t norm_fwd(const NormArgs& a, cudaStream_t s) {
  NORM_DISPATCH(launch_fwd);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t norm_bwd(const NormArgs& a, cudaStream_t s) {
  NORM_DISPATCH(launch_bwd);
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  const Split sp = bwd_split(a, shape_of(a));
  if (e != cudaSuccess || sp.S == 1 || !(a.dweight || a.dbias)) return e;
  const size_t cols = (size_t)a.H * a.d;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)((2 * cols + 31) / 32));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, norm_join_kernel, static_cast<const float*>(a.ws), sp.S, cols,
                         a.dweight, a.dbias);
  count_launches(1);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace tttk
