// Gated linear recurrence h_t = a_t h_{t-1} + u_t per feature, forward, backward and the
// single-token step on a state cache (include/ttt.h).
//
// The scans are bound by HBM: X, G (and dH, H) are read once, H (or dX, dG) written once. The map
// of a run of tokens, h -> A h + U with A the product of its decays and U its state from 0, is
// found without the state that enters it, so runs are taken in parallel and joined:
//   thread: R tokens of VC features, held in registers between the two passes over them;
//   warp:   R tokens of 32 VC features (a row's loads are one contiguous piece);
//   CTA:    kWarps such runs, joined through shared memory;
//   cluster: up to 8 CTAs along the sequence where batch and features alone give too few CTAs,
//           joined through distributed shared memory, so that no workspace is needed.
// The cluster walks the sequence in rounds of all its runs; every warp carries the state of its
// features from round to round. The next round's loads are issued before the joins. The order of
// all sums is fixed by the shape.
//
// A run that holds a document's first token maps every state to its U: joins select on a flag
// (and not by A = 0), so that an infinity or NaN of one document does not reach the next.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "simt_util.cuh"

namespace tttk {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kSMs = 148;
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;

// a = sigmoid(g) = 1 / (1 + e) and 1 - a = e a with e = exp(-g): neither is a difference. e is
// held at 2^126, where a is the smallest normal number and 1 - a is 1; a NaN stays one.
__device__ __forceinline__ void gate_of(float g, float& a, float& na) {
  float x = g * -1.44269504f, e, r;
  asm("min.NaN.f32 %0, %0, 0f42FC0000;" : "+f"(x));  // 126
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  a = r;
  na = e * r;
}

// VC neighbouring elements of a row as they lie in memory.
template <typename E, int VC>
struct Raw;
template <>
struct Raw<bf16, 1> {
  unsigned short r;
  __device__ __forceinline__ void load(const bf16* p) {
    asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(r) : "l"(p));
  }
  __device__ __forceinline__ float get(int) const { return __uint_as_float((uint32_t)r << 16); }
  static __device__ __forceinline__ void store(bf16* p, const float* v) { *p = __float2bfloat16_rn(v[0]); }
};
template <>
struct Raw<bf16, 2> {
  uint32_t r;
  __device__ __forceinline__ void load(const bf16* p) {
    asm volatile("ld.global.nc.L1::no_allocate.b32 %0, [%1];" : "=r"(r) : "l"(p));
  }
  __device__ __forceinline__ float get(int k) const { return k ? bf16hi(r) : bf16lo(r); }
  static __device__ __forceinline__ void store(bf16* p, const float* v) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v[0], v[1]);
  }
};
template <>
struct Raw<float, 1> {
  float r;
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.nc.L1::no_allocate.f32 %0, [%1];" : "=f"(r) : "l"(p));
  }
  __device__ __forceinline__ float get(int) const { return r; }
  static __device__ __forceinline__ void store(float* p, const float* v) { *p = v[0]; }
};
template <>
struct Raw<float, 2> {
  float2 r;
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.f32 {%0,%1}, [%2];" : "=f"(r.x), "=f"(r.y) : "l"(p));
  }
  __device__ __forceinline__ float get(int k) const { return k ? r.y : r.x; }
  static __device__ __forceinline__ void store(float* p, const float* v) {
    *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
  }
};

// ------------------------------------------------------------------------------------- joins
template <int VC>
struct __align__(8 * VC) Map {
  float A[VC], U[VC];
};
template <int VC>
struct Joins {  // two buffers in turn: a buffer is written again two joins later
  Map<VC> seg[2][kWarps][32], cta[2][kMaxCluster][32];
  unsigned seg_reset[2][kWarps], cta_reset[2][kMaxCluster];
};
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ uint32_t remote(uint32_t addr, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
template <int VC>
__device__ __forceinline__ void st_remote(uint32_t addr, const Map<VC>& m) {
#pragma unroll
  for (int k = 0; k < VC; ++k) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr + 4 * k), "f"(m.A[k]) : "memory");
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr + 4 * (VC + k)), "f"(m.U[k]) : "memory");
  }
}

// Joins the warps' maps m (reset: it holds a document's first token) of one round: `carry` goes
// from the state that enters the round to the one that leaves it, `in` is the state that enters
// this warp's run. All threads of the cluster call it the same number of times.
template <int VC>
__device__ __forceinline__ void join_runs(Joins<VC>& js, int buf, int cl, int rank,
                                          const Map<VC>& m, bool reset, float (&carry)[VC],
                                          float (&in)[VC]) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  js.seg[buf][w][lane] = m;
  if (lane == 0) js.seg_reset[buf][w] = reset;
  __syncthreads();
  const unsigned rs = __ballot_sync(~0u, lane < kWarps && js.seg_reset[buf][lane & (kWarps - 1)]);
  float h[VC];
#pragma unroll
  for (int k = 0; k < VC; ++k) h[k] = carry[k];
  if (cl > 1) {
    Map<VC> c;
#pragma unroll
    for (int k = 0; k < VC; ++k) c.A[k] = 1.f, c.U[k] = 0.f;
#pragma unroll
    for (int s = 0; s < kWarps; ++s) {
      const Map<VC> q = js.seg[buf][s][lane];
#pragma unroll
      for (int k = 0; k < VC; ++k) {
        c.A[k] *= q.A[k];
        c.U[k] = rs >> s & 1 ? q.U[k] : fmaf(q.A[k], c.U[k], q.U[k]);
      }
    }
    if (w < cl) {  // warp w hands the CTA's map to CTA w
      st_remote(remote(smem_u32(&js.cta[buf][rank][lane]), w), c);
      if (lane == 0)
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                         remote(smem_u32(&js.cta_reset[buf][rank]), w)), "r"(rs) : "memory");
    }
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    const unsigned crs = __ballot_sync(~0u, lane < cl && js.cta_reset[buf][lane & (kMaxCluster - 1)]);
    for (int s = 0; s < cl; ++s) {
      const Map<VC> q = js.cta[buf][s][lane];
#pragma unroll
      for (int k = 0; k < VC; ++k) {
        if (s == rank) in[k] = h[k];
        h[k] = crs >> s & 1 ? q.U[k] : fmaf(q.A[k], h[k], q.U[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      carry[k] = h[k];
      h[k] = in[k];
    }
  }
#pragma unroll
  for (int s = 0; s < kWarps; ++s) {
    const Map<VC> q = js.seg[buf][s][lane];
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      if (s == w) in[k] = h[k];
      h[k] = rs >> s & 1 ? q.U[k] : fmaf(q.A[k], h[k], q.U[k]);
    }
  }
  if (cl == 1)
#pragma unroll
    for (int k = 0; k < VC; ++k) carry[k] = h[k];
}

// This thread's place: features c.. of batch row b, run w of CTA `rank` of the cluster.
template <int VC>
struct Place {
  int b, c, cl, rank;
  bool ok;
  __device__ __forceinline__ Place(const RecurArgs& a, int cluster) {
    cl = cluster;
    rank = cl > 1 ? (int)cluster_rank() : 0;
    const int blocks = (a.D + 32 * VC - 1) / (32 * VC), i = blockIdx.x / cl;
    b = i / blocks;
    c = (i - b * blocks) * 32 * VC + (threadIdx.x & 31) * VC;
    ok = c < a.D;
  }
};
// A CTA's shared memory may be written by the others once all have started.
__device__ __forceinline__ void cluster_sync(int cl) {
  if (cl == 1) return;
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
template <int VC>
__device__ __forceinline__ void load_state(const float* p, const RecurArgs& a, const Place<VC>& at,
                                           float (&v)[VC]) {
#pragma unroll
  for (int k = 0; k < VC; ++k) v[k] = p && at.ok ? p[(size_t)at.b * a.D + at.c + k] : 0.f;
}
template <int VC>
__device__ __forceinline__ void store_state(float* p, const RecurArgs& a, const Place<VC>& at,
                                            const float (&v)[VC]) {
  if (p && at.ok && at.rank == 0 && threadIdx.x < 32)
#pragma unroll
    for (int k = 0; k < VC; ++k) p[(size_t)at.b * a.D + at.c + k] = v[k];
}
// R documents' marks from position pos of a walk (position p is token p, or T - 1 - p with REV):
// lane i loads that of position pos + i.
template <int R, bool REV>
__device__ __forceinline__ unsigned load_reset(const RecurArgs& a, int b, unsigned pos) {
  const unsigned p = pos + (threadIdx.x & 31);
  if (!a.reset || (threadIdx.x & 31) >= R || p >= (unsigned)a.T) return 0;
  return a.reset[(size_t)b * a.T + (REV ? a.T - 1 - p : p)];
}

// ----------------------------------------------------------------------------------- forward
template <typename E, typename GT, bool SIG, int VC, int R, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS)
    recur_fwd_kernel(const __grid_constant__ RecurArgs a, const int cluster) {
  __shared__ Joins<VC> js;
  const Place<VC> at(a, cluster);
  const unsigned T = a.T, stride = (unsigned)at.cl * kWarps * R;
  const size_t D = a.D, base = (size_t)at.b * T * D + at.c;
  const E* X = static_cast<const E*>(a.X) + base;
  const GT* G = static_cast<const GT*>(a.G) + base;
  E* H = static_cast<E*>(a.H) + base;
  Raw<E, VC> rx[R];
  Raw<GT, VC> rg[R];
  unsigned mark;
  auto fetch = [&](unsigned p) {
    mark = load_reset<R, false>(a, at.b, p);
    if (!at.ok || p >= T) return;
    const E* x = X + p * D;
    const GT* g = G + p * D;
    const int n = min(T - p, (unsigned)R);
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i < n) {
        rx[i].load(x + i * D);
        rg[i].load(g + i * D);
      }
  };
  unsigned pos = ((unsigned)at.rank * kWarps + (threadIdx.x >> 5)) * R;
  const unsigned rounds = (T + stride - 1) / stride;
  fetch(pos);
  cluster_sync(at.cl);
  float carry[VC];
  load_state(a.h0, a, at, carry);
  for (unsigned round = 0; round < rounds; ++round, pos += stride) {
    float av[R][VC], u[R][VC];
    const int n = pos >= T ? 0 : (int)min(T - pos, (unsigned)R);
    const unsigned rs = __ballot_sync(~0u, mark != 0);
#pragma unroll
    for (int i = 0; i < R; ++i)
#pragma unroll
      for (int k = 0; k < VC; ++k) {
        const float x = rx[i].get(k), g = rg[i].get(k);
        av[i][k] = g;
        u[i][k] = x;
        if constexpr (SIG) {
          float na;
          gate_of(g, av[i][k], na);
          u[i][k] = na * x;
        }
        if (i >= n) av[i][k] = 1.f, u[i][k] = 0.f;
      }
    fetch(pos + stride);
    Map<VC> m;
#pragma unroll
    for (int k = 0; k < VC; ++k) m.A[k] = 1.f, m.U[k] = 0.f;
    if (rs == 0) {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < VC; ++k) {
          m.A[k] *= av[i][k];
          m.U[k] = fmaf(av[i][k], m.U[k], u[i][k]);
        }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
#pragma unroll
        for (int k = 0; k < VC; ++k)
          m.U[k] = rs >> i & 1 ? u[i][k] : fmaf(av[i][k], m.U[k], u[i][k]);
    }
    float h[VC];
    join_runs(js, round & 1, at.cl, at.rank, m, rs != 0, carry, h);
    if (at.ok) {
      E* out = H + pos * D;
      if (rs == 0 && n == R) {
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
          for (int k = 0; k < VC; ++k) h[k] = fmaf(av[i][k], h[k], u[i][k]);
          Raw<E, VC>::store(out + i * D, h);
        }
      } else {
#pragma unroll
        for (int i = 0; i < R; ++i)
          if (i < n) {
#pragma unroll
            for (int k = 0; k < VC; ++k)
              h[k] = rs >> i & 1 ? u[i][k] : fmaf(av[i][k], h[k], u[i][k]);
            Raw<E, VC>::store(out + i * D, h);
          }
      }
    }
  }
  store_state(a.h_final, a, at, carry);
}

// ---------------------------------------------------------------------------------- backward
// The adjoint runs backwards over the tokens: with c the part of D_{t-1} that comes from token t,
//   D_t = dH_t + c_{t+1},  c_t = a_t D_t  (0 at a document's first token),
// a recurrence in c of the same form, walked from the last token.
template <typename E, typename GT, bool SIG, int VC, int R, int CTAS>
__global__ void __launch_bounds__(kThreads, CTAS)
    recur_bwd_kernel(const __grid_constant__ RecurArgs a, const int cluster) {
  __shared__ Joins<VC> js;
  const Place<VC> at(a, cluster);
  const unsigned T = a.T, stride = (unsigned)at.cl * kWarps * R;
  const size_t D = a.D, base = (size_t)at.b * T * D + at.c;
  const E* X = static_cast<const E*>(a.X) + base;
  const GT* G = static_cast<const GT*>(a.G) + base;
  const E* H = static_cast<const E*>(a.H_in) + base;
  const E* dH = static_cast<const E*>(a.dH) + base;
  E* dX = static_cast<E*>(a.dX) + base;
  GT* dG = static_cast<GT*>(a.dG) + base;
  Raw<E, VC> rd[R], rx[SIG ? R : 1], rh[R];
  Raw<GT, VC> rg[R];
  unsigned mark;
  // position p is token T - 1 - p; rh holds the state before the token, row T - 2 - p
  auto fetch = [&](unsigned p) {
    mark = load_reset<R, true>(a, at.b, p);
    if (!at.ok || p >= T) return;
    const size_t o = (T - 1 - p) * D;
    const int n = min(T - p, (unsigned)R), nh = min(T - 1 - p, (unsigned)R);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      if (i < n) {
        rg[i].load(G + o - i * D);
        rd[i].load(dH + o - i * D);
        if constexpr (SIG) rx[i].load(X + o - i * D);
      }
      if (i < nh) rh[i].load(H + o - (i + 1) * D);
    }
  };
  unsigned pos = ((unsigned)at.rank * kWarps + (threadIdx.x >> 5)) * R;
  const unsigned rounds = (T + stride - 1) / stride;
  fetch(pos);
  cluster_sync(at.cl);
  float carry[VC], h0[VC];
  load_state(a.dh_final, a, at, carry);
  load_state(a.h0, a, at, h0);
  for (unsigned round = 0; round < rounds; ++round, pos += stride) {
    // dg: dG / (D) before the adjoint is known: h_{t-1}, or (h_{t-1} - x) a (1 - a)
    float av[R][VC], na[SIG ? R : 1][VC], dg[R][VC];
    Raw<E, VC> dh[R];
    const int n = pos >= T ? 0 : (int)min(T - pos, (unsigned)R);
    const unsigned rs = __ballot_sync(~0u, mark != 0);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      dh[i] = rd[i];
#pragma unroll
      for (int k = 0; k < VC; ++k) {
        av[i][k] = rg[i].get(k);
        float prev = pos + i == T - 1 ? h0[k] : rh[i].get(k);
        if (rs >> i & 1) prev = 0.f;
        dg[i][k] = prev;
        if constexpr (SIG) {
          gate_of(av[i][k], av[i][k], na[i][k]);
          dg[i][k] = (prev - rx[i].get(k)) * (av[i][k] * na[i][k]);
        }
      }
    }
    fetch(pos + stride);
    Map<VC> m;
#pragma unroll
    for (int k = 0; k < VC; ++k) m.A[k] = 1.f, m.U[k] = 0.f;
#pragma unroll
    for (int i = 0; i < R; ++i)
      if (i < n)
#pragma unroll
        for (int k = 0; k < VC; ++k) {
          m.A[k] *= av[i][k];
          m.U[k] = rs >> i & 1 ? 0.f : av[i][k] * (dh[i].get(k) + m.U[k]);
        }
    float c[VC];
    join_runs(js, round & 1, at.cl, at.rank, m, rs != 0, carry, c);
    if (at.ok && n > 0) {
      const size_t o = (T - 1 - pos) * D;
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n) {
          const bool first = rs >> i & 1;
          float x[VC], g[VC];
#pragma unroll
          for (int k = 0; k < VC; ++k) {
            const float Dt = dh[i].get(k) + c[k];
            x[k] = SIG ? na[SIG ? i : 0][k] * Dt : Dt;
            g[k] = !SIG && first ? 0.f : Dt * dg[i][k];
            c[k] = first ? 0.f : av[i][k] * Dt;
          }
          Raw<E, VC>::store(dX + o - i * D, x);
          Raw<GT, VC>::store(dG + o - i * D, g);
        }
    }
  }
  store_state(a.dh0, a, at, carry);
}

// -------------------------------------------------------------------------------------- step
// CTA (j, b): VC features a thread of row b. Rows that name one slot are one chain: the first of
// them applies all in order, the others leave.
constexpr int kStepThreads = 128;
template <typename E, typename GT, bool SIG, int VC>
__global__ void __launch_bounds__(kStepThreads) recur_step_kernel(const __grid_constant__ RecurArgs a) {
  const int b = blockIdx.x, c = (blockIdx.y * kStepThreads + threadIdx.x) * VC;
  const bool ok = c < a.D;
  const int slot = a.slots ? a.slots[b] : b;
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    if (blockIdx.y == 0 && threadIdx.x == 0) atomicOr(a.err, ERR_RANGE);
    return;
  }
  float* st = a.state + (size_t)slot * a.D + c;
  Raw<E, VC> rx;
  Raw<GT, VC> rg;
  float h[VC];
  auto fetch = [&](int row) {
    rx.load(static_cast<const E*>(a.X) + (size_t)row * a.D + c);
    rg.load(static_cast<const GT*>(a.G) + (size_t)row * a.D + c);
  };
  auto token = [&](int row) {
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      float aa = rg.get(k), u = rx.get(k), na;
      if constexpr (SIG) {
        gate_of(aa, aa, na);
        u *= na;
      }
      h[k] = fmaf(aa, h[k], u);
    }
    Raw<E, VC>::store(static_cast<E*>(a.H) + (size_t)row * a.D + c, h);
  };
  if (ok) {
    fetch(b);
#pragma unroll
    for (int k = 0; k < VC; ++k) h[k] = st[k];
  }
  bool later = false;
  if (a.slots) {
    bool before = false;
    for (int r = threadIdx.x; r < a.B; r += kStepThreads)
      if (a.slots[r] == slot) {
        before |= r < b;
        later |= r > b;
      }
    if (__syncthreads_or(before)) return;
    later = __syncthreads_or(later);
  }
  if (!ok) return;
  token(b);
  if (later)
    for (int r = b + 1; r < a.B; ++r)
      if (a.slots[r] == slot) {
        fetch(r);
        token(r);
      }
  Raw<float, VC>::store(st, h);
}

// ------------------------------------------------------------------------------------ launch
// CTAs along the sequence: as few as bring the grid to two CTAs per SM, and no more than have a
// run each.
int cluster_of(const RecurArgs& a, int vc, int run) {
  const long long ctas = (long long)a.B * ((a.D + 32 * vc - 1) / (32 * vc));
  int cl = 1;
  while (cl < kMaxCluster && ctas * cl < 2 * kSMs && (long long)cl * kWarps * run < a.T) cl *= 2;
  return cl;
}
template <typename K>
cudaError_t launch(K kernel, const RecurArgs& a, int vc, int run, cudaStream_t s) {
  const int cl = cluster_of(a, vc, run);
  const long long ctas = (long long)a.B * ((a.D + 32 * vc - 1) / (32 * vc)) * cl;
  if (ctas >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = cl;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = cl > 1;
  count_launches(1);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a, cl);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Two features a thread where rows start on a pair's boundary and pairs are 32 bits (bf16 X).
#ifndef RF
#define RF 8
#define RB 8
#define CF 3
#define CB 2
#endif
cudaError_t recur_fwd(const RecurArgs& a, cudaStream_t s) {
  const bool two = a.bf16 && a.D % 2 == 0;
  if (two && a.sigmoid) return launch(recur_fwd_kernel<bf16, bf16, true, 2, RF, CF>, a, 2, RF, s);
  if (two) return launch(recur_fwd_kernel<bf16, float, false, 2, RF, CF>, a, 2, RF, s);
  if (a.bf16 && a.sigmoid) return launch(recur_fwd_kernel<bf16, bf16, true, 1, 16, 3>, a, 1, 16, s);
  if (a.bf16) return launch(recur_fwd_kernel<bf16, float, false, 1, 16, 3>, a, 1, 16, s);
  if (a.sigmoid) return launch(recur_fwd_kernel<float, float, true, 1, 16, 3>, a, 1, 16, s);
  return launch(recur_fwd_kernel<float, float, false, 1, 16, 3>, a, 1, 16, s);
}
cudaError_t recur_bwd(const RecurArgs& a, cudaStream_t s) {
  const bool two = a.bf16 && a.D % 2 == 0;
  if (two && a.sigmoid) return launch(recur_bwd_kernel<bf16, bf16, true, 2, RB, CB>, a, 2, RB, s);
  if (two) return launch(recur_bwd_kernel<bf16, float, false, 2, RB, CB>, a, 2, RB, s);
  if (a.bf16 && a.sigmoid) return launch(recur_bwd_kernel<bf16, bf16, true, 1, 8, 2>, a, 1, 8, s);
  if (a.bf16) return launch(recur_bwd_kernel<bf16, float, false, 1, 8, 2>, a, 1, 8, s);
  if (a.sigmoid) return launch(recur_bwd_kernel<float, float, true, 1, 8, 2>, a, 1, 8, s);
  return launch(recur_bwd_kernel<float, float, false, 1, 8, 2>, a, 1, 8, s);
}
cudaError_t recur_step(const RecurArgs& a, cudaStream_t s) {
  const int vc = a.D % 2 == 0 ? 2 : 1;
  const int cols = kStepThreads * vc;
  const dim3 grid(a.B, (a.D + cols - 1) / cols);
  count_launches(1);
  if (vc == 2) {
    if (a.bf16 && a.sigmoid) recur_step_kernel<bf16, bf16, true, 2><<<grid, kStepThreads, 0, s>>>(a);
    else if (a.bf16) recur_step_kernel<bf16, float, false, 2><<<grid, kStepThreads, 0, s>>>(a);
    else if (a.sigmoid) recur_step_kernel<float, float, true, 2><<<grid, kStepThreads, 0, s>>>(a);
    else recur_step_kernel<float, float, false, 2><<<grid, kStepThreads, 0, s>>>(a);
  } else {
    if (a.bf16 && a.sigmoid) recur_step_kernel<bf16, bf16, true, 1><<<grid, kStepThreads, 0, s>>>(a);
    else if (a.bf16) recur_step_kernel<bf16, float, false, 1><<<grid, kStepThreads, 0, s>>>(a);
    else if (a.sigmoid) recur_step_kernel<float, float, true, 1><<<grid, kStepThreads, 0, s>>>(a);
    else recur_step_kernel<float, float, false, 1><<<grid, kStepThreads, 0, s>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace tttk
