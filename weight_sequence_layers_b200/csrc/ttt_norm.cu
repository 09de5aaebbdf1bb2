// Layer norm over rows of d features with one weight group per head, forward and backward
// (include/ttt.h).
//
// A row is read once into registers, reduced twice there (the mean, then the centred squares: no
// cancellation for rows with a large mean) and written once. Bound by HBM and, close behind, by the
// instructions issued (16 and 22 for 32 values): 262144 x 128 bf16 forward 28 us = 4.9 TB/s,
// 32768 x 2560 bf16 backward with dS 113 us = 5.9 TB/s and 8 us for the weight gradients' join
// (one CTA per row with the row read three times: 734 us and 5.8 ms).
// A row belongs to a group of threads: 8 to 32 lanes of a warp for narrow rows (several rows
// per CTA, sums by shuffles alone), the whole CTA for wide ones. CTA (h, s) walks a contiguous
// run of the rows of head h, so that the head's weights stay in registers, with the next rows'
// loads in flight.
//
// The backward keeps its share of dweight and dbias in registers over its run; the CTAs' shares
// go to the workspace and a second kernel adds them in a fixed order (no atomics). That kernel
// starts while the first one drains (programmatic launch) and waits for it on the device.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "simt_util.cuh"

namespace tttk {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kSMs = 148;
constexpr int kNarrowThreads = 128;  // CTA of the narrow-row kernels
// Of them on an SM, and the threads of the wide-row kernels on an SM, by the floats of a row that
// a thread holds: what the registers leave room for.
constexpr int narrow_ctas(int floats) { return floats < 16 ? 4 : 3; }
constexpr int fwd_threads(int floats) { return floats <= 8 ? 1024 : 512; }
constexpr int bwd_threads(int floats) { return floats <= 8 ? 640 : 512; }

// VEC elements of a row: one 16-byte access; where the width does not keep rows on 16-byte
// boundaries, a pair for even widths and one element for odd ones. Coherent loads, since S may be X or residual and dX may be dS.
template <typename E, int VEC>
struct Pack;
template <>
struct Pack<bf16, 8> {
  uint4 r;
  __device__ __forceinline__ void load(const bf16* p) {
    asm volatile("ld.global.L1::no_allocate.v4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  }
  __device__ __forceinline__ void get(float2* v) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u));
  }
  static __device__ __forceinline__ void store(bf16* p, const float2* v) {
    uint32_t w[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) w[k] = pack_bf16x2(v[k].x, v[k].y);
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
  __device__ __forceinline__ void get(float2* v) const {
    v[0] = make_float2(r.x, r.y);
    v[1] = make_float2(r.z, r.w);
  }
  static __device__ __forceinline__ void store(float* p, const float2* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0].x, v[0].y, v[1].x, v[1].y);
  }
};
template <>
struct Pack<bf16, 2> {
  uint32_t r;
  __device__ __forceinline__ void load(const bf16* p) {
    asm volatile("ld.global.L1::no_allocate.b32 %0, [%1];" : "=r"(r) : "l"(p) : "memory");
  }
  __device__ __forceinline__ void get(float2* v) const { v[0] = make_float2(bf16lo(r), bf16hi(r)); }
  static __device__ __forceinline__ void store(bf16* p, const float2* v) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v[0].x, v[0].y);
  }
};
template <>
struct Pack<float, 2> {
  float2 r;
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.L1::no_allocate.v2.f32 {%0,%1}, [%2];" : "=f"(r.x), "=f"(r.y) : "l"(p) : "memory");
  }
  __device__ __forceinline__ void get(float2* v) const { v[0] = r; }
  static __device__ __forceinline__ void store(float* p, const float2* v) { *reinterpret_cast<float2*>(p) = v[0]; }
};
template <typename E>
struct Pack<E, 1> {
  E r;
  __device__ __forceinline__ void load(const E* p) { r = *p; }
};

// A thread's part of a row: NV accesses of VEC elements, `step` columns apart, as pairs (VEC = 1
// has an odd element only with NV = 1: the pair's second half). An access past the row's end
// reads the row's last elements again (at()), or zeros behind its slot of shared memory (at_slot()):
// its columns are told apart by mask() only, which costs less than a predicate on every access and
// value.
template <typename E, int VEC, int NV>
struct Frag {
  static constexpr int NP = VEC == 1 ? (NV + 1) / 2 : NV * VEC / 2;  // pairs
  int first, step, d;  // this thread's first column and the columns between its accesses
  __device__ __forceinline__ int col(int n) const { return first + n * step; }
  __device__ __forceinline__ bool ok(int n) const { return n < NV && col(n) < d; }
  __device__ __forceinline__ int at(int n) const { return min(col(n), d - VEC); }
  __device__ __forceinline__ int at_slot(int n, int zeros) const { return ok(n) ? col(n) : zeros; }
  // 1 for the pair's columns that are the row's, else 0
  __device__ __forceinline__ void mask(float2 (&m)[NP]) const {
#pragma unroll
    for (int i = 0; i < NP; ++i)
      m[i] = VEC > 1 ? both(ok(2 * i / VEC) ? 1.f : 0.f)
                     : make_float2(ok(2 * i) ? 1.f : 0.f, ok(2 * i + 1) ? 1.f : 0.f);
  }
  // unpacks loaded accesses
  __device__ __forceinline__ void get(const Pack<E, VEC> (&p)[NV], float2 (&v)[NP]) const {
    if constexpr (VEC > 1) {
#pragma unroll
      for (int n = 0; n < NV; ++n) p[n].get(v + n * VEC / 2);
    } else {
#pragma unroll
      for (int n = 0; n < 2 * NP; n += 2)
        v[n / 2] = make_float2(ldf(&p[n].r), n + 1 < NV ? ldf(&p[n + 1 < NV ? n + 1 : 0].r) : 0.f);
    }
  }
  template <typename L>
  __device__ __forceinline__ void each_f32(L f) const {  // f(pair, half, column) where valid
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (ok(n))
#pragma unroll
        for (int k = 0; k < VEC; ++k) f((n * VEC + k) / 2, (n * VEC + k) & 1, col(n) + k);
  }
  // float32 parameters of the columns (`none` without an array), 0 past the end
  __device__ __forceinline__ void get_f32(const float* p, float none, float2 (&v)[NP]) const {
#pragma unroll
    for (int k = 0; k < NP; ++k) v[k] = both(0.f);
    each_f32([&](int i, int h, int c) { (h ? v[i].y : v[i].x) = p ? p[c] : none; });
  }
  __device__ __forceinline__ void store(E* p, const float2 (&v)[NP]) const {
#pragma unroll
    for (int n = 0; n < NV; ++n)
      if (ok(n)) {
        if constexpr (VEC > 1) Pack<E, VEC>::store(p + col(n), v + n * VEC / 2);
        else stf(p + col(n), n & 1 ? v[n / 2].y : v[n / 2].x);
      }
  }
};
// The masked sum, x - mean (0 past the end), and the sum of squares of that. The masks multiply: an
// infinity or NaN that is read again past the end makes a NaN of the sum, which is then taken again
// from the row's own columns alone (selected).
template <int NP>
__device__ __forceinline__ float selected(const float2 (&v)[NP], const float2 (&m)[NP]) {
  float t = 0.f;
#pragma unroll
  for (int i = 0; i < NP; ++i) t += (m[i].x != 0.f ? v[i].x : 0.f) + (m[i].y != 0.f ? v[i].y : 0.f);
  return t;
}
template <int NP>
__device__ __forceinline__ float selected(const float2 (&v)[NP], const float2 (&x)[NP],
                                          const float2 (&m)[NP]) {
  float2 q[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) q[i] = mul2(v[i], x[i]);
  return selected(q, m);
}
template <int N>
__device__ __forceinline__ bool any_nan(const float (&t)[N]) {
  bool nan = false;
#pragma unroll
  for (int n = 0; n < N; ++n) nan = nan || t[n] != t[n];
  return nan;
}
// Sums that are not NaN stay to the last bit, whatever the rows beside them hold.
template <int N>
__device__ __forceinline__ void replace_nan(float (&t)[N], const float (&s)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) t[n] = t[n] != t[n] ? s[n] : t[n];
}
template <int NP>
__device__ __forceinline__ float total(const float2 (&v)[NP], const float2 (&m)[NP]) {
  float2 t = mul2(v[0], m[0]);
#pragma unroll
  for (int i = 1; i < NP; ++i) t = fma2(v[i], m[i], t);
  return t.x + t.y;
}
template <int NP>
__device__ __forceinline__ void centre(float mean, const float2 (&m)[NP], float2 (&v)[NP]) {
  const float2 c = both(-mean);
#pragma unroll
  for (int i = 0; i < NP; ++i) v[i] = fma2(v[i], m[i], mul2(c, m[i]));
}
template <int NP>
__device__ __forceinline__ float total_sq(const float2 (&v)[NP]) {
  float2 t = mul2(v[0], v[0]);
#pragma unroll
  for (int i = 1; i < NP; ++i) t = fma2(v[i], v[i], t);
  return t.x + t.y;
}
template <int NP>
__device__ __forceinline__ void scale_shift(float rstd, const float2 (&w)[NP],
                                            const float2 (&b)[NP], float2 (&v)[NP]) {
  const float2 r = both(rstd);
#pragma unroll
  for (int i = 0; i < NP; ++i) v[i] = fma2(mul2(v[i], r), w[i], b[i]);
}
// The backward of one row in two halves. first: x -> xh, g (dY) -> g w, the weight gradients'
// terms, and the sums of g w and g w xh (w is 0 past the row's end); second: g w -> dX without dS.
template <int NP>
__device__ __forceinline__ void bwd_first(float mean, float rstd, const float2 (&w)[NP],
                                          float2 (&x)[NP], float2 (&g)[NP], float2 (&dw)[NP],
                                          float2 (&db)[NP], float& s1, float& s2) {
  const float2 r = both(rstd), m = both(-mean);
  float2 t1 = both(0.f), t2 = both(0.f);
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    x[i] = mul2(add2(x[i], m), r);
    db[i] = add2(db[i], g[i]);
    dw[i] = fma2(g[i], x[i], dw[i]);
    g[i] = mul2(g[i], w[i]);
    t1 = add2(t1, g[i]);
    t2 = fma2(g[i], x[i], t2);
  }
  s1 = t1.x + t1.y;
  s2 = t2.x + t2.y;
}
template <int NP>
__device__ __forceinline__ void bwd_second(float rstd, float c1, float c2, const float2 (&x)[NP],
                                           float2 (&g)[NP]) {
  const float2 r = both(rstd), n1 = both(-c1), n2 = both(-c2);
#pragma unroll
  for (int i = 0; i < NP; ++i) g[i] = mul2(r, fma2(x[i], n2, add2(g[i], n1)));
}

// How a launch cuts the rows: head h's B T rows (i = b T + t) into S runs of L, CTA h S + s.
struct Split {
  int S, L;
};
// A walk over a head's rows i, i + step, ...: the row in the [B, H, T, d] tensors without a
// division per step.
struct Walk {
  int i, t;      // the head's row and its token
  size_t row;    // (b H + h) T + t
  __device__ __forceinline__ void start(int i0, int T, int H, int h) {
    i = i0;
    const int b = i0 / T;
    t = i0 - b * T;
    row = ((size_t)b * H + h) * T + t;
  }
  __device__ __forceinline__ void next(int step, int T, int H) {
    i += step;
    row += step;
    if (H == 1) return;
    t += step;
    while (t >= T) {
      t -= T;
      row += (size_t)(H - 1) * T;
    }
  }
};
struct Rows {
  int lo, hi, s, h;
  __device__ __forceinline__ Rows(const NormArgs& a, const Split& sp) {
    h = blockIdx.x / sp.S;
    s = blockIdx.x - h * sp.S;
    const long long bt = (long long)a.B * a.T;
    lo = (int)min((long long)s * sp.L, bt);
    hi = (int)min((long long)lo + sp.L, bt);
  }
};
// The row of Y and dY.
__device__ __forceinline__ size_t y_row(const NormArgs& a, const Rows& R, const Walk& w) {
  return a.token_major ? (size_t)w.i * a.H + R.h : w.row;
}

template <int G, int N>
__device__ __forceinline__ void lanes_sum(float (&v)[N]) {
#pragma unroll
  for (int o = G / 2; o; o >>= 1)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor_sync(~0u, v[n], o);
}

// ------------------------------------------------------------------------------ narrow rows
// G lanes per row, NV accesses of VEC elements each, RU rows per group and step: RU rows are
// loaded ahead while RU are reduced, which keeps enough bytes in flight. RES: with a residual,
// which doubles a row's bytes. PAST: the lanes' accesses go past the row's end.
template <typename E, int VEC, int NV, int G, int RU, bool RES, bool PAST>
__global__ void __launch_bounds__(kNarrowThreads, narrow_ctas(NV * VEC))
    norm_fwd_narrow(const __grid_constant__ NormArgs a, const Split sp) {
  using F = Frag<E, VEC, NV>;
  constexpr int NG = kNarrowThreads / G, STEP = RU * NG;
  const Rows R(a, sp);
  const int grp = threadIdx.x / G, tid = threadIdx.x % G, d = a.d;
  const F f{tid * VEC, G * VEC, d};
  const float inv_d = 1.f / (float)d;
  const E* X = static_cast<const E*>(a.X);
  const E* Rs = static_cast<const E*>(a.residual);
  E* Y = static_cast<E*>(a.Y);
  E* S = static_cast<E*>(a.S);
  float2 w[F::NP], bb[F::NP], mk[F::NP];
  f.mask(mk);
  Pack<E, VEC> px[RU][NV], pr[RES ? RU : 1][NV];
  Walk at[RU];
  auto fetch = [&]() {
#pragma unroll
    for (int u = 0; u < RU; ++u)
      if (at[u].i < R.hi) {
        const size_t o = at[u].row * d;
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          px[u][n].load(X + o + f.at(n));
          if constexpr (RES) pr[u][n].load(Rs + o + f.at(n));
        }
      }
  };
#pragma unroll
  for (int u = 0; u < RU; ++u) at[u].start(R.lo + u * NG + grp, a.T, a.H, R.h);
  fetch();
  f.get_f32(a.weight ? a.weight + (size_t)R.h * d : nullptr, 1.f, w);
  f.get_f32(a.bias ? a.bias + (size_t)R.h * d : nullptr, 0.f, bb);
  for (int i0 = R.lo; i0 < R.hi; i0 += STEP) {  // uniform over the CTA
    float2 v[RU][F::NP];
    float t[RU], mean[RU];
    size_t row[RU], yrow[RU];
    bool live[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      live[u] = at[u].i < R.hi;
      row[u] = at[u].row;
      yrow[u] = y_row(a, R, at[u]);
      f.get(px[u], v[u]);
      if constexpr (RES) {
        float2 r[F::NP];
        f.get(pr[u], r);
#pragma unroll
        for (int i = 0; i < F::NP; ++i) v[u][i] = add2(v[u][i], r[i]);
        if (S && live[u]) f.store(S + row[u] * d, v[u]);
      }
      t[u] = total(v[u], mk);
      at[u].next(STEP, a.T, a.H);
    }
    fetch();
    lanes_sum<G>(t);
    if (PAST && __any_sync(~0u, any_nan(t))) {
      float s[RU];
#pragma unroll
      for (int u = 0; u < RU; ++u) s[u] = selected(v[u], mk);
      lanes_sum<G>(s);
      replace_nan(t, s);
    }
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      mean[u] = t[u] * inv_d;
      centre(mean[u], mk, v[u]);
      t[u] = total_sq(v[u]);
    }
    lanes_sum<G>(t);
#pragma unroll
    for (int u = 0; u < RU; ++u)
      if (live[u]) {
        const float rstd = rsqrtf(fmaf(t[u], inv_d, a.eps));
        scale_shift(rstd, w, bb, v[u]);
        f.store(Y + yrow[u] * d, v[u]);
        if (tid == 0) {
          if (a.mean) a.mean[row[u]] = mean[u];
          if (a.rstd) a.rstd[row[u]] = rstd;
        }
      }
  }
}

// The CTA's shares of dweight and dbias go to dw0 + s ldp and db0 + s ldp (S = 1: the outputs
// themselves).
struct Partials {
  float *dw0, *db0;  // each nullable
  size_t ldp;
};

template <typename E, int VEC, int NV, int G, int RU, bool PAST>
__global__ void __launch_bounds__(kNarrowThreads, narrow_ctas(NV * VEC))
    norm_bwd_narrow(const __grid_constant__ NormArgs a, const Split sp, const Partials pt) {
  using F = Frag<E, VEC, NV>;
  constexpr int NG = kNarrowThreads / G, STEP = RU * NG;
  constexpr int W = G * NV * VEC;  // columns of a group, padded
  __shared__ float join[2][NG][W];
  asm volatile("griddepcontrol.launch_dependents;");
  const Rows R(a, sp);
  const int grp = threadIdx.x / G, tid = threadIdx.x % G, d = a.d;
  const F f{tid * VEC, G * VEC, d};
  const float inv_d = 1.f / (float)d;
  const E* X = static_cast<const E*>(a.X);
  const E* dY = static_cast<const E*>(a.dY);
  const E* dS = static_cast<const E*>(a.dS);
  E* dX = static_cast<E*>(a.dX);
  float2 w[F::NP], dw[F::NP], db[F::NP];
  Pack<E, VEC> px[RU][NV], py[RU][NV], ps[RU][NV];
  Walk at[RU];
  float nmean[RU], nrstd[RU];
  auto fetch = [&]() {
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      nmean[u] = nrstd[u] = 0.f;
      if (at[u].i < R.hi) {
        const size_t o = at[u].row * d, oy = y_row(a, R, at[u]) * d;
        nmean[u] = a.mean[at[u].row];
        nrstd[u] = a.rstd[at[u].row];
#pragma unroll
        for (int n = 0; n < NV; ++n) {
          px[u][n].load(X + o + f.at(n));
          py[u][n].load(dY + oy + f.at(n));
          if (dS) ps[u][n].load(dS + o + f.at(n));
        }
      }
    }
  };
#pragma unroll
  for (int u = 0; u < RU; ++u) at[u].start(R.lo + u * NG + grp, a.T, a.H, R.h);
  fetch();
  f.get_f32(a.weight ? a.weight + (size_t)R.h * d : nullptr, 1.f, w);
#pragma unroll
  for (int i = 0; i < F::NP; ++i) dw[i] = db[i] = both(0.f);
  for (int i0 = R.lo; i0 < R.hi; i0 += STEP) {  // uniform over the CTA
    float2 xh[RU][F::NP], g[RU][F::NP];
    Pack<E, VEC> s[RU][NV];
    float t[2 * RU], rstd[RU];
    size_t row[RU];
    bool live[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      live[u] = at[u].i < R.hi;
      row[u] = at[u].row;
      rstd[u] = nrstd[u];
      t[2 * u] = t[2 * u + 1] = 0.f;
      if (live[u]) {
        f.get(px[u], xh[u]);
        f.get(py[u], g[u]);
        bwd_first(nmean[u], rstd[u], w, xh[u], g[u], dw, db, t[2 * u], t[2 * u + 1]);
        if (dS)
#pragma unroll
          for (int n = 0; n < NV; ++n) s[u][n] = ps[u][n];
      }
      at[u].next(STEP, a.T, a.H);
    }
    fetch();
    lanes_sum<G>(t);
    if (PAST && __any_sync(~0u, any_nan(t))) {
      float2 m[F::NP];
      float r[2 * RU];
      f.mask(m);
#pragma unroll
      for (int u = 0; u < RU; ++u) {
        r[2 * u] = live[u] ? selected(g[u], m) : 0.f;
        r[2 * u + 1] = live[u] ? selected(g[u], xh[u], m) : 0.f;
      }
      lanes_sum<G>(r);
      replace_nan(t, r);
    }
#pragma unroll
    for (int u = 0; u < RU; ++u)
      if (live[u]) {
        bwd_second(rstd[u], t[2 * u] * inv_d, t[2 * u + 1] * inv_d, xh[u], g[u]);
        if (dS) {
          float2 sv[F::NP];
          f.get(s[u], sv);
#pragma unroll
          for (int i = 0; i < F::NP; ++i) g[u][i] = add2(g[u][i], sv[i]);
        }
        f.store(dX + row[u] * d, g[u]);
      }
  }
  if (!pt.dw0 && !pt.db0) return;
  f.each_f32([&](int i, int h, int c) {
    join[0][grp][c] = h ? dw[i].y : dw[i].x;
    join[1][grp][c] = h ? db[i].y : db[i].x;
  });
  __syncthreads();
  const size_t base = R.s * pt.ldp + (size_t)R.h * d;
  for (int j = threadIdx.x; j < d; j += kNarrowThreads) {
    float tw = 0.f, tb = 0.f;
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      tw += join[0][g][j];
      tb += join[1][g][j];
    }
    if (pt.dw0) pt.dw0[base + j] = tw;
    if (pt.db0) pt.db0[base + j] = tb;
  }
}

// -------------------------------------------------------------------------------- wide rows
// One CTA per row. Rows come into a ring of shared-memory stages by bulk copies (TMA, untiled)
// that one thread issues several rows ahead, so that the bytes in flight cost no registers.
// A stage is refilled behind the barrier of its row's sum, when all threads hold the row in
// registers. A bulk copy moves whole 16-byte blocks: where rows start off such a boundary
// (VEC of 1 and 2) the stage holds the blocks around the row and the row starts `off` bytes in; the
// copy never goes past the tensor's last whole block, and the elements behind it (of the last
// row only) are read directly. Behind each slot's blocks are kZeros bytes of zeros, which accesses
// past the row's end read (wherever in its first block the row starts).
constexpr uint32_t kZeros = 32;
struct Ring {
  int stages;
  uint32_t slot;  // bytes of one row's slot, a multiple of 16, with the zeros at its end
};
struct RowView {
  uint32_t off;  // bytes from the slot's start to the row
  int in_slot;   // elements of the row that the slot holds
};
// The view of a row that starts at element x of a tensor of `total` elements.
template <typename E, int VEC>
__device__ __forceinline__ RowView row_view(size_t x, int d, size_t total) {
  if (VEC * sizeof(E) == 16) return {0u, d};
  const size_t b0 = x * sizeof(E), end = total * sizeof(E) & ~(size_t)15;
  const size_t held = end > b0 ? (end - b0) / sizeof(E) : 0;
  return {(uint32_t)(b0 & 15), held < (size_t)d ? (int)held : d};
}
// Bytes that its copy moves.
template <typename E, int VEC>
__device__ __forceinline__ uint32_t row_bytes(size_t x, int d, size_t total) {
  const size_t es = sizeof(E), b0 = x * es;
  if (VEC * sizeof(E) == 16) return (uint32_t)(d * es);
  const size_t from = b0 & ~(size_t)15, end = total * es & ~(size_t)15;
  const size_t to = (b0 + d * es + 15) & ~(size_t)15;
  const size_t stop = to < end ? to : end;
  return stop > from ? (uint32_t)(stop - from) : 0u;
}
template <typename E>
__device__ __forceinline__ void row_copy(uint32_t slot, const E* row, uint32_t bytes, uint32_t bar) {
  if (!bytes) return;
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
      ::"r"(slot), "l"(reinterpret_cast<uintptr_t>(row) & ~(uintptr_t)15), "r"(bytes), "r"(bar)
      : "memory");
}
// A thread's accesses in a slot, from the row's start. HOLD keeps them in registers, where the compiler
// would make them again for every row (4098 x 1021 float32 backward 23.0 us against 25.0); the
// backward of 8 and more accesses has no registers for them (45288 x 1403: 223 us against 262).
template <bool HOLD, typename E, int VEC, int NV>
__device__ __forceinline__ void slot_indices(const Frag<E, VEC, NV>& f, const Ring& rg, int (&idx)[NV]) {
#pragma unroll
  for (int n = 0; n < NV; ++n) {
    idx[n] = f.at_slot(n, (rg.slot - kZeros) / (uint32_t)sizeof(E));
    if constexpr (HOLD) asm volatile("" : "+r"(idx[n]));
  }
}
template <typename E, int VEC, int NV>
__device__ __forceinline__ void slot_read(const Frag<E, VEC, NV>& f, const uint8_t* slot,
                                          const RowView& rv, const E* row, const int (&idx)[NV],
                                          float2 (&v)[Frag<E, VEC, NV>::NP]) {
  Pack<E, VEC> p[NV];
  using R = decltype(p[0].r);
  const E* sp = reinterpret_cast<const E*>(slot + rv.off);
  if (VEC * sizeof(E) == 16 || rv.in_slot >= f.d) {
#pragma unroll
    for (int n = 0; n < NV; ++n) p[n].r = *reinterpret_cast<const R*>(sp + idx[n]);
  } else {  // the tensor's last row, off a 16-byte boundary
#pragma unroll
    for (int n = 0; n < NV; ++n)
      p[n].r = *reinterpret_cast<const R*>(f.ok(n) && f.col(n) >= rv.in_slot ? row + f.col(n)
                                                                             : sp + idx[n]);
  }
  f.get(p, v);
}

constexpr int kMaxStages = 8;
struct __align__(16) RingBars {
  float red[2][4][16];  // [buffer][value][warp]
  uint64_t full[kMaxStages];
  int abort_flag;
};
// Sums of N (1, 2 or 4) values over the CTA (at most 16 warps) through one barrier. Values are
// halved among the lanes while they are summed (lanes 32/N v .. hold value v), so that N values
// cost little more than one. Two buffers alternate: nobody writes a buffer before all have passed
// the barrier of the sum after the one that last read it. Unused warps' entries are zero.
template <int N>
__device__ __forceinline__ void cta_sum(float (&v)[N], float (*red)[16]) {
  static_assert(N == 1 || N == 2 || N == 4, "N");
  constexpr int L = 32 / N;  // lanes of a value
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5, mine = lane / L;
  float c;
  if constexpr (N == 4) {
    const bool hi = lane & 16, hi2 = lane & 8;
    const float a0 = (hi ? v[2] : v[0]) + __shfl_xor_sync(~0u, hi ? v[0] : v[2], 16);
    const float a1 = (hi ? v[3] : v[1]) + __shfl_xor_sync(~0u, hi ? v[1] : v[3], 16);
    c = (hi2 ? a1 : a0) + __shfl_xor_sync(~0u, hi2 ? a0 : a1, 8);
  } else if constexpr (N == 2) {
    const bool hi = lane & 16;
    c = (hi ? v[1] : v[0]) + __shfl_xor_sync(~0u, hi ? v[0] : v[1], 16);
  } else {
    c = v[0];
  }
#pragma unroll
  for (int o = L / 2; o; o >>= 1) c += __shfl_xor_sync(~0u, c, o);
  if (lane % L == 0) red[mine][wp] = c;
  __syncthreads();
  constexpr int P = L < 16 ? L : 16;  // lanes that read a value's 16 entries
  if constexpr (P == 8) {
    const float2 q = reinterpret_cast<const float2*>(red[mine])[lane % 8];
    c = q.x + q.y;
  } else {
    c = red[mine][lane % 16];
  }
#pragma unroll
  for (int o = P / 2; o; o >>= 1) c += __shfl_xor_sync(~0u, c, o);
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = N == 1 ? c : __shfl_sync(~0u, c, n * L);
}
__device__ __forceinline__ void ring_init(RingBars& bars, const Ring& rg, uint8_t* slots, int nslots) {
  for (int k = threadIdx.x; k < nslots * (int)(kZeros / 4); k += blockDim.x) {
    const int slot = k / (int)(kZeros / 4), word = k % (int)(kZeros / 4);
    *reinterpret_cast<uint32_t*>(slots + (size_t)(slot + 1) * rg.slot - kZeros + 4 * word) = 0u;
  }
  for (int k = threadIdx.x; k < 2 * 4 * 16; k += blockDim.x) (&bars.red[0][0][0])[k] = 0.f;
  if (threadIdx.x == 0) {
    for (int s = 0; s < rg.stages; ++s) mbar_init(smem_u32(&bars.full[s]), 1);
    bars.abort_flag = 0;
    fence_barrier_init();
  }
  __syncthreads();
}

// A walk over a head's rows one by one, in elements: the row's start in the [B, H, T, d] tensors
// and in Y, and its index for mean and rstd.
struct RowWalk {
  int i, t;
  size_t x, y, row;
  __device__ __forceinline__ RowWalk(const NormArgs& a, const Rows& R) {
    Walk w;
    w.start(R.lo, a.T, a.H, R.h);
    i = w.i;
    t = w.t;
    row = w.row;
    x = row * a.d;
    y = y_row(a, R, w) * a.d;
  }
  __device__ __forceinline__ void next(const NormArgs& a) {
    ++i;
    ++row;
    x += a.d;
    y += a.token_major ? (size_t)a.H * a.d : (size_t)a.d;
    if (a.H > 1 && ++t == a.T) {
      t = 0;
      const size_t skip = (size_t)(a.H - 1) * a.T;
      row += skip;
      x += skip * a.d;
      if (!a.token_major) y += skip * a.d;
    }
  }
};
// Row loads of one thread into the ring, stage after stage.
template <typename E, int VEC>
struct Loader {
  RowWalk at;
  int st = 0;
  uint32_t slots, bars;
  size_t total;  // elements of a tensor
  __device__ __forceinline__ Loader(const NormArgs& a, const Rows& R, uint32_t slots_, uint32_t bars_)
      : at(a, R), slots(slots_), bars(bars_), total((size_t)a.B * a.H * a.T * a.d) {}
  // n rows of the tensors s0, s1 (by x) and sy (by y; each nullable) into the next stages
  __device__ __forceinline__ void issue(int n, const NormArgs& a, const Rows& R, const Ring& rg,
                                        const E* s0, const E* sy, const E* s1) {
    const int nsrc = 1 + (sy != nullptr) + (s1 != nullptr);
    for (; n > 0 && at.i < R.hi; --n) {
      const uint32_t nx = row_bytes<E, VEC>(at.x, a.d, total), ny = row_bytes<E, VEC>(at.y, a.d, total);
      uint32_t slot = slots + st * nsrc * rg.slot;
      const uint32_t bar = bars + 8 * st;
      mbar_arrive_expect_tx(bar, nx * (s1 ? 2 : 1) + (sy ? ny : 0));
      row_copy(slot, s0 + at.x, nx, bar);
      if (sy) row_copy(slot += rg.slot, sy + at.y, ny, bar);
      if (s1) row_copy(slot + rg.slot, s1 + at.x, nx, bar);
      at.next(a);
      if (++st == rg.stages) st = 0;
    }
  }
};

template <typename E, int VEC, int NV>
__global__ void __launch_bounds__(512, fwd_threads(NV * VEC) / 512)
    norm_fwd_wide(const __grid_constant__ NormArgs a, const Split sp, const Ring rg) {
  using F = Frag<E, VEC, NV>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ RingBars bars;
  const Rows R(a, sp);
  const int tid = threadIdx.x, d = a.d;
  const F f{tid * VEC, (int)blockDim.x * VEC, d};
  const float inv_d = 1.f / (float)d;
  const E* X = static_cast<const E*>(a.X);
  const E* Rs = static_cast<const E*>(a.residual);
  E* Y = static_cast<E*>(a.Y);
  E* S = static_cast<E*>(a.S);
  const Abort ab{&bars.abort_flag, a.err};
  const int nsrc = Rs ? 2 : 1;
  ring_init(bars, rg, smem, rg.stages * nsrc);
  int idx[NV];
  slot_indices<true>(f, rg, idx);
  Loader<E, VEC> ld(a, R, smem_u32(smem), smem_u32(bars.full));
  if (tid == 0) ld.issue(rg.stages, a, R, rg, X, nullptr, Rs);
  float2 w[F::NP], bb[F::NP], mk[F::NP];
  f.mask(mk);
  f.get_f32(a.weight ? a.weight + (size_t)R.h * d : nullptr, 1.f, w);
  f.get_f32(a.bias ? a.bias + (size_t)R.h * d : nullptr, 0.f, bb);
  int st = 0;
  uint32_t ph = 0;
  for (RowWalk at(a, R); at.i < R.hi; at.next(a)) {
    const RowView rv = row_view<E, VEC>(at.x, d, ld.total);
    const uint8_t* slot = smem + st * nsrc * rg.slot;
    // a wait that runs out is recorded; the loop goes on without waiting, so that all threads
    // keep meeting at the barriers
    mbar_wait(smem_u32(&bars.full[st]), ph, ab);
    float2 v[F::NP];
    float t[1];
    slot_read(f, slot, rv, X + at.x, idx, v);
    if (Rs) {
      float2 r[F::NP];
      slot_read(f, slot + rg.slot, rv, Rs + at.x, idx, r);
#pragma unroll
      for (int i = 0; i < F::NP; ++i) v[i] = add2(v[i], r[i]);
    }
    t[0] = total(v, mk);
    cta_sum(t, bars.red[0]);
    if (tid == 0) ld.issue(1, a, R, rg, X, nullptr, Rs);
    if (++st == rg.stages) { st = 0; ph ^= 1; }
    const float mean = t[0] * inv_d;
    if (S) f.store(S + at.x, v);
    centre(mean, mk, v);
    t[0] = total_sq(v);
    cta_sum(t, bars.red[1]);
    const float rstd = rsqrtf(fmaf(t[0], inv_d, a.eps));
    scale_shift(rstd, w, bb, v);
    f.store(Y + at.y, v);
    if (tid == 0) {
      if (a.mean) a.mean[at.row] = mean;
      if (a.rstd) a.rstd[at.row] = rstd;
    }
  }
  if (bars.abort_flag) __nanosleep(100000);  // let any load issued before the abort land
}

// RU rows per step share one barrier; a stage is refilled behind the next step's barrier, so that
// dS is read from it after the sums instead of being held in registers.
template <typename E, int VEC, int NV, int RU, int MAXT>
__global__ void __launch_bounds__(MAXT, 640 / MAXT)
    norm_bwd_wide(const __grid_constant__ NormArgs a, const Split sp, const Ring rg,
                  const Partials pt) {
  using F = Frag<E, VEC, NV>;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ RingBars bars;
  asm volatile("griddepcontrol.launch_dependents;");
  const Rows R(a, sp);
  const int tid = threadIdx.x, d = a.d;
  const F f{tid * VEC, (int)blockDim.x * VEC, d};
  const float inv_d = 1.f / (float)d;
  const E* X = static_cast<const E*>(a.X);
  const E* dY = static_cast<const E*>(a.dY);
  const E* dS = static_cast<const E*>(a.dS);
  E* dX = static_cast<E*>(a.dX);
  const Abort ab{&bars.abort_flag, a.err};
  const int nsrc = dS ? 3 : 2;
  ring_init(bars, rg, smem, rg.stages * nsrc);
  int idx[NV];
  slot_indices<NV <= 4>(f, rg, idx);
  Loader<E, VEC> ld(a, R, smem_u32(smem), smem_u32(bars.full));
  if (tid == 0) ld.issue(rg.stages, a, R, rg, X, dY, dS);
  float2 w[F::NP], dw[F::NP], db[F::NP];
  f.get_f32(a.weight ? a.weight + (size_t)R.h * d : nullptr, 1.f, w);
#pragma unroll
  for (int i = 0; i < F::NP; ++i) dw[i] = db[i] = both(0.f);
  int st = 0, buf = 0;
  uint32_t ph = 0;
  float nmean[RU], nrstd[RU];
  RowWalk at(a, R);
  // the next step's statistics, a step ahead; rows past the run's end read the last row's
  size_t stat = at.row;
  int stat_t = at.t, left = R.hi - R.lo;
  auto stats = [&]() {
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      nmean[u] = a.mean[stat];
      nrstd[u] = a.rstd[stat];
      if (--left > 0) {
        ++stat;
        if (a.H > 1 && ++stat_t == a.T) {
          stat_t = 0;
          stat += (size_t)(a.H - 1) * a.T;
        }
      }
    }
  };
  if (left > 0) stats();
  const bool tight = rg.stages < 2 * RU;
  for (bool first = true; at.i < R.hi; first = false) {  // uniform over the CTA
    float2 xh[RU][F::NP], g[RU][F::NP];
    float t[2 * RU], rstd[RU];
    size_t x[RU];
    const uint8_t* slot[RU];
    bool live[RU];
#pragma unroll
    for (int u = 0; u < RU; ++u) {
      live[u] = at.i < R.hi;
      x[u] = at.x;
      slot[u] = smem + st * nsrc * rg.slot;
      rstd[u] = nrstd[u];
      t[2 * u] = t[2 * u + 1] = 0.f;
      if (live[u]) {
        // a wait that runs out is recorded; the loop goes on without waiting, so that all
        // threads keep meeting at the barriers
        mbar_wait(smem_u32(&bars.full[st]), ph, ab);
        slot_read(f, slot[u], row_view<E, VEC>(at.x, d, ld.total), X + at.x, idx, xh[u]);
        slot_read(f, slot[u] + rg.slot, row_view<E, VEC>(at.y, d, ld.total), dY + at.y, idx, g[u]);
        bwd_first(nmean[u], rstd[u], w, xh[u], g[u], dw, db, t[2 * u], t[2 * u + 1]);
        if (++st == rg.stages) { st = 0; ph ^= 1; }
        at.next(a);
      }
    }
    stats();
    cta_sum(t, bars.red[buf]);
    buf ^= 1;
    if (tid == 0 && !first && !tight) ld.issue(RU, a, R, rg, X, dY, dS);  // the last step's stages
#pragma unroll
    for (int u = 0; u < RU; ++u)
      if (live[u]) {
        bwd_second(rstd[u], t[2 * u] * inv_d, t[2 * u + 1] * inv_d, xh[u], g[u]);
        if (dS) {
          float2 s[F::NP];
          slot_read(f, slot[u] + 2 * rg.slot, row_view<E, VEC>(x[u], d, ld.total), dS + x[u], idx, s);
#pragma unroll
          for (int i = 0; i < F::NP; ++i) g[u][i] = add2(g[u][i], s[i]);
        }
        f.store(dX + x[u], g[u]);
      }
    if (tight) {
      __syncthreads();
      if (tid == 0) ld.issue(RU, a, R, rg, X, dY, dS);
    }
  }
  const size_t base = R.s * pt.ldp + (size_t)R.h * d;
  f.each_f32([&](int i, int h, int c) {
    if (pt.dw0) pt.dw0[base + c] = h ? dw[i].y : dw[i].x;
    if (pt.db0) pt.db0[base + c] = h ? db[i].y : db[i].x;
  });
  if (bars.abort_flag) __nanosleep(100000);
}

// dweight[j] = sum over s of part[s][0][j], dbias likewise from part[s][1]: 32 columns per CTA,
// the warps over s.
constexpr int kJoinWarps = 16;
__global__ void __launch_bounds__(32 * kJoinWarps)
    norm_join_kernel(const float* part, int S, size_t cols, float* dweight, float* dbias) {
  __shared__ float red[kJoinWarps][33];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x % 32, wp = threadIdx.x / 32;
  const size_t c = (size_t)blockIdx.x * 32 + lane;  // column of [dweight | dbias]
  constexpr int kFlight = 8;
  float t[kFlight];
#pragma unroll
  for (int k = 0; k < kFlight; ++k) t[k] = 0.f;
  if (c < 2 * cols)
    for (int s = wp; s < S; s += kFlight * kJoinWarps)
#pragma unroll
      for (int k = 0; k < kFlight; ++k)
        if (s + k * kJoinWarps < S) t[k] += part[(size_t)(s + k * kJoinWarps) * 2 * cols + c];
  red[wp][lane] = ((t[0] + t[1]) + (t[2] + t[3])) + ((t[4] + t[5]) + (t[6] + t[7]));
  __syncthreads();
  if (wp == 0 && c < 2 * cols) {
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < kJoinWarps; ++k) sum += red[k][lane];
    float* out = c < cols ? dweight : dbias;
    if (out) out[c < cols ? c : c - cols] = sum;
  }
}

// ------------------------------------------------------------------------------ launch rules
struct Shape {
  int vec, nv, g, threads;  // g = 0: a wide row, one CTA of `threads`
};
// Narrow rows take as few lanes as hold the row in at most two (small accesses: eight;
// single elements in the forward: sixteen) each.
// Wide rows: the forward takes one access (small ones: four) per thread up to 512 threads, then more.
// The backward takes 16 values per thread: its work around a row is the same for 8 (32768 x 2560:
// 110 us against 143 with twice the threads and two rows per barrier).
Shape shape_of(const NormArgs& a, bool bwd) {
  const int v = a.bf16 ? 8 : 4;
  Shape s;
  s.vec = a.d % v == 0 ? v : a.d % 2 == 0 ? 2 : 1;
  const int n = a.d / s.vec;
  s.threads = kNarrowThreads;
  if (s.vec == v) {
    if (n <= 8) { s.g = 8; s.nv = 1; return s; }
    if (n <= 16) { s.g = 16; s.nv = 1; return s; }
    if (n <= 32) { s.g = 32; s.nv = 1; return s; }
    if (n <= 64) { s.g = 32; s.nv = 2; return s; }
    s.nv = n <= 512 ? 1 : n <= 1024 ? 2 : n <= 2048 ? 4 : 8;
    if (bwd) s.nv = std::max(s.nv, 16 / s.vec);
  } else {
    if (n <= 32) { s.g = 32; s.nv = 1; return s; }
    if (n <= 64) { s.g = 32; s.nv = 2; return s; }
    if (n <= 128) { s.g = 32; s.nv = 4; return s; }
    if (n <= 256) { s.g = 32; s.nv = 8; return s; }
    if (n <= 512 && s.vec == 1 && !bwd) { s.g = 32; s.nv = 16; return s; }
    s.nv = n <= 2048 ? 4 : n <= 4096 ? 8 : n <= 8192 ? 16 : 32;
    // 4 single elements with two rows per barrier against 8 with one: where runs are short or rows
    // narrow the 4 (us, 4098 x 1263 float32 25.0 against 27.3, 6144 x 1021 31.2 against 31.4; 45288 x 601
    // bf16 104 against 117), else the 8 (8800 x 1021 bf16 39.4 against 42.2, 45288 x 641 119 against 142)
    const bool long_runs = (long long)a.B * a.H * a.T >= 64 * kSMs;
    if (bwd && (s.vec == 2 || n > 1280 || (n > 640 && long_runs))) s.nv = std::max(s.nv, 8);
  }
  s.g = 0;
  s.threads = ((n + s.nv - 1) / s.nv + 31) / 32 * 32;
  return s;
}

// CTAs of an SM, from the threads that the kernels' registers leave room for.
int ctas_per_sm(const Shape& sh, bool bwd) {
  const int floats = sh.nv * sh.vec;
  if (sh.g) return narrow_ctas(floats);
  const int threads = bwd ? bwd_threads(floats) : fwd_threads(floats);
  return std::max(1, std::min(8, threads / sh.threads));
}
// A run of the backward has at least four rows per group, so that the shares of the weight
// gradients it writes are few against the rows it reads.
Split split_of(const NormArgs& a, const Shape& sh, bool bwd) {
  const int min_rows = bwd ? 4 : 1;
  const long long bt = (long long)a.B * a.T;
  const int ngrp = sh.g ? kNarrowThreads / sh.g : 1;
  const long long slots = (long long)kSMs * ctas_per_sm(sh, bwd);
  // every SM gets a CTA before any run is longer than one row per group; beyond that a run has
  // at least min_rows per group
  const long long one = (bt + ngrp - 1) / ngrp, few = (one + min_rows - 1) / min_rows;
  const long long S = std::min(std::max(1ll, slots / a.H),
                               std::max(few, std::min(one, (long long)(kSMs + a.H - 1) / a.H)));
  Split sp{};
  const long long L = (bt + S - 1) / S;
  sp.L = (int)std::min(bt, (L + ngrp - 1) / ngrp * ngrp);
  sp.S = (int)((bt + sp.L - 1) / sp.L);
  return sp;
}
Split fwd_split(const NormArgs& a, const Shape& sh) { return split_of(a, sh, false); }
Split bwd_split(const NormArgs& a, const Shape& sh) { return split_of(a, sh, true); }

constexpr uint32_t kRingBytes = 200 << 10;  // of an SM's shared memory, for all its CTAs
Ring ring_of(const NormArgs& a, const Shape& sh, int nsrc, bool bwd) {
  const uint32_t es = a.bf16 ? 2 : 4;
  Ring r;
  // off a 16-byte boundary a row touches up to one block more on each side
  r.slot = (sh.vec * es == 16 ? a.d * es : (a.d * es + 30) / 16 * 16) + kZeros;
  const uint32_t room = kRingBytes / ctas_per_sm(sh, bwd) / (nsrc * r.slot);
  r.stages = (int)std::max(1u, std::min((uint32_t)kMaxStages, room));
  return r;
}
template <typename K>
cudaError_t ring_room(K kernel, size_t smem) {
  return smem > (40 << 10) ? cudaFuncSetAttribute(
             kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) : cudaSuccess;
}

Partials partials_of(const NormArgs& a, const Split& sp) {
  const size_t cols = (size_t)a.H * a.d;
  if (!a.dweight && !a.dbias) return {};
  if (sp.S == 1) return {a.dweight, a.dbias, 0};
  float* ws = static_cast<float*>(a.ws);
  return {ws, ws + cols, 2 * cols};
}

struct Fwd {
  static constexpr bool kBwd = false;
  template <typename E, int VEC, int NV, int G, int RU>
  static cudaError_t narrow(const NormArgs& a, const Shape& sh, cudaStream_t s) {
    const Split sp = fwd_split(a, sh);
    const unsigned grid = (unsigned)a.H * sp.S;
    if (a.d == G * NV * VEC) {
      if (a.residual) norm_fwd_narrow<E, VEC, NV, G, RU, true, false><<<grid, sh.threads, 0, s>>>(a, sp);
      else norm_fwd_narrow<E, VEC, NV, G, 2 * RU, false, false><<<grid, sh.threads, 0, s>>>(a, sp);
    } else {
      if (a.residual) norm_fwd_narrow<E, VEC, NV, G, RU, true, true><<<grid, sh.threads, 0, s>>>(a, sp);
      else norm_fwd_narrow<E, VEC, NV, G, 2 * RU, false, true><<<grid, sh.threads, 0, s>>>(a, sp);
    }
    return cudaGetLastError();
  }
  template <typename E, int VEC, int NV>
  static cudaError_t wide(const NormArgs& a, const Shape& sh, cudaStream_t s) {
    const Split sp = fwd_split(a, sh);
    const int nsrc = a.residual ? 2 : 1;
    const Ring rg = ring_of(a, sh, nsrc, false);
    const size_t smem = (size_t)rg.stages * nsrc * rg.slot;
    const cudaError_t e = ring_room(norm_fwd_wide<E, VEC, NV>, smem);
    if (e != cudaSuccess) return e;
    norm_fwd_wide<E, VEC, NV><<<(unsigned)a.H * sp.S, sh.threads, smem, s>>>(a, sp, rg);
    return cudaGetLastError();
  }
};
struct Bwd {
  static constexpr bool kBwd = true;
  template <typename E, int VEC, int NV, int G, int RU>
  static cudaError_t narrow(const NormArgs& a, const Shape& sh, cudaStream_t s) {
    const Split sp = bwd_split(a, sh);
    const unsigned grid = (unsigned)a.H * sp.S;
    if (a.d == G * NV * VEC)
      norm_bwd_narrow<E, VEC, NV, G, RU, false><<<grid, sh.threads, 0, s>>>(a, sp, partials_of(a, sp));
    else
      norm_bwd_narrow<E, VEC, NV, G, RU, true><<<grid, sh.threads, 0, s>>>(a, sp, partials_of(a, sp));
    return cudaGetLastError();
  }
  template <typename E, int VEC, int NV>
  static cudaError_t wide(const NormArgs& a, const Shape& sh, cudaStream_t s) {
    const Split sp = bwd_split(a, sh);
    const int nsrc = a.dS ? 3 : 2;
    const Ring rg = ring_of(a, sh, nsrc, true);
    const size_t smem = (size_t)rg.stages * nsrc * rg.slot;
    constexpr int RU = NV * VEC <= 4 ? 2 : 1, MAXT = RU == 2 ? 320 : 512;
    return wide_launch(norm_bwd_wide<E, VEC, NV, RU, MAXT>, a, sh, sp, rg, smem, s);
  }
  template <typename K>
  static cudaError_t wide_launch(K kernel, const NormArgs& a, const Shape& sh, const Split& sp,
                                 const Ring& rg, size_t smem, cudaStream_t s) {
    const cudaError_t e = ring_room(kernel, smem);
    if (e != cudaSuccess) return e;
    kernel<<<(unsigned)a.H * sp.S, sh.threads, smem, s>>>(a, sp, rg, partials_of(a, sp));
    return cudaGetLastError();
  }
};

// The instance of a row shape. RU (rows per group and step; twice that in a forward without
// residual) is what the registers leave room for.
template <typename F, typename E, int VEC>
cudaError_t dispatch_vec(const NormArgs& a, const Shape& sh, cudaStream_t s) {
  if (sh.g == 8) return F::template narrow<E, VEC, 1, 8, 2>(a, sh, s);
  if (sh.g == 16) return F::template narrow<E, VEC, 1, 16, 2>(a, sh, s);
  if (sh.g == 32 && sh.nv == 1) return F::template narrow<E, VEC, 1, 32, 2>(a, sh, s);
  if (sh.g == 32) return F::template narrow<E, VEC, 2, 32, 1>(a, sh, s);
  if constexpr (!F::kBwd) {
    if (sh.nv == 1) return F::template wide<E, VEC, 1>(a, sh, s);
  }
  if constexpr (!F::kBwd || VEC == 8) {
    if (sh.nv == 2) return F::template wide<E, VEC, 2>(a, sh, s);
  }
  if (sh.nv == 4) return F::template wide<E, VEC, 4>(a, sh, s);
  if constexpr (VEC == 4) return F::template wide<E, VEC, 8>(a, sh, s);  // float32 rows only
  return cudaErrorInvalidValue;
}
template <typename F, typename E, int VEC>
cudaError_t dispatch_small(const NormArgs& a, const Shape& sh, cudaStream_t s) {
  constexpr int RU = VEC == 1 ? 2 : 1;
  if (sh.g == 32 && sh.nv == 1) return F::template narrow<E, VEC, 1, 32, 2>(a, sh, s);
  if (sh.g == 32 && sh.nv == 2) return F::template narrow<E, VEC, 2, 32, 2>(a, sh, s);
  if (sh.g == 32 && sh.nv == 4) return F::template narrow<E, VEC, 4, 32, RU>(a, sh, s);
  if (sh.g == 32 && sh.nv == 8) return F::template narrow<E, VEC, 8, 32, 1>(a, sh, s);
  if constexpr (VEC == 1 && !F::kBwd) {
    if (sh.g == 32) return F::template narrow<E, 1, 16, 32, 1>(a, sh, s);
  }
  if constexpr (!F::kBwd || VEC == 1) {
    if (sh.nv == 4) return F::template wide<E, VEC, 4>(a, sh, s);
  }
  if (sh.nv == 8) return F::template wide<E, VEC, 8>(a, sh, s);
  if constexpr (VEC == 1) {
    if (sh.nv == 32) return F::template wide<E, VEC, 32>(a, sh, s);
  }
  return F::template wide<E, VEC, 16>(a, sh, s);
}
template <typename F>
cudaError_t dispatch(const NormArgs& a, cudaStream_t s) {
  const Shape sh = shape_of(a, F::kBwd);
  count_launches(1);
  if (sh.vec == 8) return dispatch_vec<F, bf16, 8>(a, sh, s);
  if (sh.vec == 4) return dispatch_vec<F, float, 4>(a, sh, s);
  if (sh.vec == 2)
    return a.bf16 ? dispatch_small<F, bf16, 2>(a, sh, s) : dispatch_small<F, float, 2>(a, sh, s);
  return a.bf16 ? dispatch_small<F, bf16, 1>(a, sh, s) : dispatch_small<F, float, 1>(a, sh, s);
}

}  // namespace

bool norm_supported(const NormArgs& a) { return a.d <= 16384; }

size_t norm_bwd_workspace(const NormArgs& a) {
  const Split sp = bwd_split(a, shape_of(a, true));
  return sp.S == 1 ? 0 : (size_t)sp.S * 2 * a.H * a.d * sizeof(float);
}

cudaError_t norm_fwd(const NormArgs& a, cudaStream_t s) { return dispatch<Fwd>(a, s); }

cudaError_t norm_bwd(const NormArgs& a, cudaStream_t s) {
  cudaError_t e = dispatch<Bwd>(a, s);
  const Split sp = bwd_split(a, shape_of(a, true));
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
