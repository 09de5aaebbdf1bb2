// Gated linear recurrence h_t = a_t h_{t-1} + u_t per feature, forward, backward and the
// single-token step on a state cache (include/ttt.h).
//
// X, G (and dH, H) are read once, H (or dX, dG) written once. The map of a run of tokens,
// h -> A h + U with A the product of its decays and U its state from 0, is found without the state
// that enters it, so runs are taken in parallel and joined:
//   thread: R tokens of VC features, held in registers between the two passes over them;
//   warp:   R tokens of 32 VC features (a row's loads are one contiguous piece), which come into
//           shared memory by asynchronous copies a round or two ahead;
//   CTA:    kWarps such runs, joined through shared memory by scans over eight lanes;
//   cluster: up to 8 CTAs along the sequence where batch and features alone give too few CTAs,
//           joined through distributed shared memory, so that no workspace is needed.
// The cluster walks the sequence in rounds of all its runs. The order of all sums is fixed by the
// shape.
//
// Bound by the time of a round (about 4,700 cycles: the gates' exponentials and reciprocals 1,500,
// the join and its exchange 1,900, loads, outputs) before HBM: 32768 x 2560 bf16 forward 128 us =
// 3.9 TB/s (one thread per feature: 19.8 ms), 8 x 2048 x 2048 backward 73 us = 5.5 TB/s. Measured
// and not kept: CTAs of 4 warps on 32 features (the same), three or four CTAs per SM with shorter
// runs (192 us and more), joins by a releasing cluster barrier, which waits for the outputs'
// stores too (371 us against 195 at the time).
//
// A run that holds a document's first token maps every state to its U: joins select on a flag
// (and not by A = 0), so that an infinity or NaN of one document does not reach the next.
//
// Decays given as values may be above 1, and the products that join runs can then leave float32's
// range where every state stays in it (a zero or tiny state over tokens that would double it). A
// round in which any product of its scans is not finite is walked run after run instead, each from
// the state that the one before left, with the arithmetic of the single-token step. (The way costs
// the decay forward of 32768 x 2560 bf16 143 -> 154 us without being taken, shorter ones nothing.)
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <float.h>

#include <algorithm>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "pair_tc.cuh"
#include "simt_util.cuh"

namespace tttk {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kWarps = 8, kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;

// A thread's features of one token: one float, or two in a pair (f32x2 arithmetic).
template <int VC>
struct VecOf { using T = float; };
template <>
struct VecOf<2> { using T = float2; };
template <int VC>
using Vec = typename VecOf<VC>::T;
__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ float2 add(float2 a, float2 b) { return add2(a, b); }
__device__ __forceinline__ float mul(float a, float b) { return a * b; }
__device__ __forceinline__ float2 mul(float2 a, float2 b) { return mul2(a, b); }
__device__ __forceinline__ float fma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) { return fma2(a, b, c); }
template <int VC>
__device__ __forceinline__ Vec<VC> all(float v) {
  if constexpr (VC == 1) return v;
  else return both(v);
}
template <typename V>
__device__ __forceinline__ V pick(bool c, V a, V b) {
  if constexpr (sizeof(V) == 4) return c ? a : b;
  else return make_float2(c ? a.x : b.x, c ? a.y : b.y);
}

// a = sigmoid(g) = 1 / (1 + e) and 1 - a = e a with e = exp(-g): neither is a difference. Logits
// come held at -87 (Raw::hold), where a is 2e-38 and 1 - a is 1: beyond, e would overflow.
// E is the logits' type. bf16: the hardware's base-2 exponential of g log2(e); the rounding of that
// product enters the exponent, so that e is off by about a step of float32 for every unit of |g|,
// which bf16 outputs hide (half a step of theirs is 2^16 of those). float32: with x the rounded
// product and r what it lost (by one multiply-add, and log2(e) beyond its own float32),
// exp(-g) = 2^x 2^r = 2^x (1 + r ln 2) to 2^-33: the hardware's own two steps are left, whatever |g|
// is. (The library's expf and a rounded reciprocal: 32768 x 2560 forward 246 us.)
__device__ __forceinline__ float exp2_of(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x));
  return e;
}
__device__ __forceinline__ float recip(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
constexpr double kLog2e = 1.4426950408889634;
constexpr float kNegLog2e = (float)-kLog2e, kNegLog2eRest = (float)(-kLog2e - (double)kNegLog2e);
constexpr float kLn2 = 0.693147181f;
template <typename E>
__device__ __forceinline__ void gate_of(float g, float& a, float& na) {
  if constexpr (sizeof(E) == 4) {
    const float x = g * kNegLog2e, r = fmaf(g, kNegLog2eRest, fmaf(g, kNegLog2e, -x));
    const float p = exp2_of(x), e = fmaf(p, r * kLn2, p);
    a = recip(1.f + e);
    na = e * a;
  } else {
    const float e = exp2_of(g * kNegLog2e);
    a = recip(1.f + e);
    na = e * a;
  }
}
template <typename E>
__device__ __forceinline__ void gate_of(float2 g, float2& a, float2& na) {
  if constexpr (sizeof(E) == 4) {
    gate_of<E>(g.x, a.x, na.x);
    gate_of<E>(g.y, a.y, na.y);
  } else {
    const float2 x = mul2(g, both(kNegLog2e));
    const float2 e = make_float2(exp2_of(x.x), exp2_of(x.y));
    const float2 q = add2(e, both(1.f));
    a = make_float2(recip(q.x), recip(q.y));
    na = mul2(e, a);
  }
}

// VC neighbouring elements of a row as they lie in memory. hold: at least -87 (0xC2AE in bf16), and
// in float32, where an infinity would leave the product's rest NaN, at most 126 (1 - a is 0 from 88
// on); a NaN stays one.
__device__ __forceinline__ float held(float g) {
  asm("max.NaN.f32 %0, %0, 0fC2AE0000;\n\tmin.NaN.f32 %0, %0, 0f42FC0000;" : "+f"(g));
  return g;
}
template <typename E, int VC>
struct Raw;
template <>
struct Raw<bf16, 1> {
  unsigned short r;
  __device__ __forceinline__ void load(const bf16* p) {
    asm volatile("ld.global.nc.L1::no_allocate.u16 %0, [%1];" : "=h"(r) : "l"(p));
  }
  __device__ __forceinline__ void hold() { asm("max.NaN.bf16 %0, %0, %1;" : "+h"(r) : "h"((unsigned short)0xC2AE)); }
  __device__ __forceinline__ float get() const { return __uint_as_float((uint32_t)r << 16); }
  static __device__ __forceinline__ void store(bf16* p, float v) { *p = __float2bfloat16_rn(v); }
};
template <>
struct Raw<bf16, 2> {
  uint32_t r;
  __device__ __forceinline__ void load(const bf16* p) {
    asm volatile("ld.global.nc.L1::no_allocate.b32 %0, [%1];" : "=r"(r) : "l"(p));
  }
  __device__ __forceinline__ void hold() { asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(r) : "r"(0xC2AEC2AEu)); }
  __device__ __forceinline__ float2 get() const { return make_float2(bf16lo(r), bf16hi(r)); }
  static __device__ __forceinline__ void store(bf16* p, float2 v) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16x2(v.x, v.y);
  }
};
template <>
struct Raw<float, 1> {
  float r;
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.nc.L1::no_allocate.f32 %0, [%1];" : "=f"(r) : "l"(p));
  }
  __device__ __forceinline__ void hold() { r = held(r); }
  __device__ __forceinline__ float get() const { return r; }
  static __device__ __forceinline__ void store(float* p, float v) { *p = v; }
};
template <>
struct Raw<float, 2> {
  float2 r;
  __device__ __forceinline__ void load(const float* p) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.f32 {%0,%1}, [%2];" : "=f"(r.x), "=f"(r.y) : "l"(p));
  }
  __device__ __forceinline__ void hold() { r = make_float2(held(r.x), held(r.y)); }
  __device__ __forceinline__ float2 get() const { return r; }
  static __device__ __forceinline__ void store(float* p, float2 v) { *reinterpret_cast<float2*>(p) = v; }
};
// i rows of D elements (i a constant: one wide multiply-add on the pointer).
template <typename E>
__device__ __forceinline__ E* rows(E* p, int i, unsigned D) {
  return reinterpret_cast<E*>(reinterpret_cast<uintptr_t>(p) +
                              (uint64_t)D * (uint32_t)(i * sizeof(E)));
}
template <typename E>
__device__ __forceinline__ E* rows_back(E* p, int i, unsigned D) {
  return reinterpret_cast<E*>(reinterpret_cast<uintptr_t>(p) -
                              (uint64_t)D * (uint32_t)(i * sizeof(E)));
}

// ------------------------------------------------------------------------------------- joins
// A CTA's runs and a cluster's CTAs are joined by scans over eight lanes: in warp w, lane 8 q + s
// takes the maps s (of run s, or of CTA s) of features kScan w + q + 4 k, k < VC, so that a scan
// is three shuffles deep and all warps share the work.
template <int VC>
struct Joins {
  static constexpr int kCols = 32 * VC, kScan = kCols / kWarps;
  static constexpr int kPitch = kCols + 4;  // rows of neighbouring s fall into different banks
  float A[kWarps][kPitch], U[kWarps][kPitch];  // the runs' maps
  float in[kWarps][kPitch];                    // the states that enter the runs
  float2 cta[2][kMaxCluster][kPitch];          // the CTAs' maps, two rounds in turn
  unsigned run_reset[kWarps], cta_reset[2][kMaxCluster];
  uint64_t full[2];  // the cluster's maps of the round have arrived in cta and cta_reset
  int abort_flag;
};
// Stores to a CTA of the cluster that count their bytes on its barrier: the receiver waits for
// the data alone, where a release would make every round wait for the outputs' stores too.
__device__ __forceinline__ void st_async(uint32_t addr, float a, float u, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1,%2}, [%3];"
               ::"r"(addr), "f"(a), "f"(u), "r"(bar) : "memory");
}
__device__ __forceinline__ void st_async(uint32_t addr, uint32_t v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.u32 [%0], %1, [%2];"
               ::"r"(addr), "r"(v), "r"(bar) : "memory");
}
// Before the first join: the barriers, and that all CTAs of the cluster have started.
template <int VC>
__device__ __forceinline__ void join_init(Joins<VC>& js, int cl) {
  if (cl == 1) return;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&js.full[0]), 1);
    mbar_init(smem_u32(&js.full[1]), 1);
    js.abort_flag = 0;
    fence_barrier_init();
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Inclusive scan of the maps of lanes s = 0..7 of each group: afterwards lane s holds map s after
// ... after map 0. resets: bit s for map s; a map that holds a reset does not see what is before.
template <int VC>
__device__ __forceinline__ void scan8(float (&A)[VC], float (&U)[VC], unsigned resets) {
  const int s = threadIdx.x & 7;
#pragma unroll
  for (int o = 1; o < 8; o *= 2) {
    float a[VC], u[VC];
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      a[k] = __shfl_up_sync(~0u, A[k], o, 8);
      u[k] = __shfl_up_sync(~0u, U[k], o, 8);
    }
    // maps s - o + 1 .. s are in (A, U); lanes without a map before theirs keep them
    const bool in = s >= o, see = in && (resets >> (s - o + 1) & ((1u << o) - 1)) == 0;
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      U[k] = see ? fmaf(A[k], u[k], U[k]) : U[k];
      A[k] = in ? A[k] * a[k] : A[k];
    }
  }
}

// All threads of the cluster meet.
__device__ __forceinline__ void meet(int cl) {
  __syncwarp();
  if (cl > 1) cluster_sync_all();
  else __syncthreads();
}
// A round without products: run after run, CTA after CTA, `through` takes a run's threads from the
// state that enters it to the one that leaves it; the state that enters the round is in CTA 0's
// in[0], the one that leaves it comes into every CTA's A[0]. All threads of the cluster call it,
// behind a barrier of their CTA after join_runs' last use of js.
template <int VC, typename Through>
__device__ __forceinline__ void join_serial(Joins<VC>& js, int cl, int rank, const Through& through) {
  using V = Vec<VC>;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  auto send = [&](float* to, int cta, V h) {
    const uint32_t at = peer_addr(smem_u32(to), cta);
    if constexpr (VC == 1) {
      asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(h) : "memory");
    } else {
      asm volatile("st.shared::cluster.v2.f32 [%0], {%1,%2};" ::"r"(at), "f"(h.x), "f"(h.y) : "memory");
    }
  };
#pragma unroll 1
  for (int r = 0; r < cl; ++r) {
    meet(cl);  // the state that enters CTA r is in its in[0]
    if (r != rank) continue;
#pragma unroll 1
    for (int q = 0; q < kWarps; ++q) {
      if (w == q) {
        const V h = through(*reinterpret_cast<const V*>(&js.in[q][lane * VC]));
        if (q + 1 < kWarps) *reinterpret_cast<V*>(&js.in[q + 1][lane * VC]) = h;
        else if (r + 1 < cl) send(&js.in[0][lane * VC], r + 1, h);
        else if (cl == 1) *reinterpret_cast<V*>(&js.A[0][lane * VC]) = h;
        else
#pragma unroll 1
          for (int c = 0; c < cl; ++c) send(&js.A[0][lane * VC], c, h);
      }
      __syncthreads();
    }
  }
  meet(cl);
}
__device__ __forceinline__ bool within(float x, float most) { return fabsf(x) <= most; }
__device__ __forceinline__ bool within(float2 x, float most) { return within(x.x, most) && within(x.y, most); }

// Joins the runs' maps (A, U) (reset: the run holds a document's first token) of one round:
// carry goes from the state that enters the round to the one that leaves it (in the layout of the
// scans); returns the state that enters this warp's run. All threads of the cluster call it the
// same number of times. A buffer of `cta` is free again when the next round's maps arrive: a CTA
// sends those behind a barrier that all its threads reach after reading it, and sends into the
// buffer again only after it has them from all.
// WIDE: products may leave the range, where a run's A is above kSafe in size (marked beside its
// reset). A product that did stays an infinity or NaN to the end of its lane's scan. In the scan of
// the CTAs' maps, which all CTAs make alike, it sends the whole cluster the serial way; in the scan
// of the runs, where the CTA's own map (lane 7's) is sound, this CTA alone.
constexpr float kSafe = 3.9f;  // to the power of the 64 runs of a round: below 2^127
template <int VC, bool WIDE, typename Through>
__device__ __forceinline__ Vec<VC> join_runs(Joins<VC>& js, unsigned round, int cl, int rank,
                                             Vec<VC> A, Vec<VC> U, bool reset, float (&carry)[VC],
                                             unsigned* err, const Through& through) {
  using J = Joins<VC>;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31, buf = round & 1;
  const int s = lane & 7, col = w * J::kScan + (lane >> 3);
  *reinterpret_cast<Vec<VC>*>(&js.A[w][lane * VC]) = A;
  *reinterpret_cast<Vec<VC>*>(&js.U[w][lane * VC]) = U;
  unsigned mark = reset;
  if constexpr (WIDE) mark |= __any_sync(~0u, !within(A, kSafe)) ? 2u : 0u;
  if (lane == 0) js.run_reset[w] = mark;
  const uint32_t full = smem_u32(&js.full[buf]);
  if (cl > 1 && threadIdx.x == 0) mbar_arrive_expect_tx(full, cl * (J::kCols * 8 + 4));
  __syncthreads();
  mark = lane < kWarps ? js.run_reset[s] : 0u;
  const unsigned rs = __ballot_sync(~0u, mark & 1);
  unsigned wide = WIDE ? __ballot_sync(~0u, mark & 2) : 0u;
  float a[VC], u[VC], in[VC];
#pragma unroll
  for (int k = 0; k < VC; ++k) {
    a[k] = js.A[s][col + 4 * k];
    u[k] = js.U[s][col + 4 * k];
    in[k] = carry[k];
  }
  scan8(a, u, rs);
  bool own = false, out = false;  // a product of the runs' scan, of the CTAs' is out of range
  if (wide)
#pragma unroll
    for (int k = 0; k < VC; ++k) own = own || !within(a[k], FLT_MAX);
  if (cl > 1) {
    const uint32_t bar = peer_addr(full, s < cl ? s : 0);  // lane s of a group sends to CTA s
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      const float ta = __shfl_sync(~0u, a[k], 7, 8), tu = __shfl_sync(~0u, u[k], 7, 8);
      if (s < cl) st_async(peer_addr(smem_u32(&js.cta[buf][rank][col + 4 * k]), s), ta, tu, bar);
    }
    if (w == 0 && lane < cl)
      st_async(peer_addr(smem_u32(&js.cta_reset[buf][rank]), lane), rs | (wide ? 0x100u : 0u), bar);
    // a wait that runs out is recorded, and the rounds go on without waiting
    if (!mbar_try_wait_cluster(full, round >> 1 & 1))
      mbar_wait_cluster(full, round >> 1 & 1, {&js.abort_flag, err});
    __syncwarp();
    mark = lane < cl ? js.cta_reset[buf][s] : 0u;
    const unsigned crs = __ballot_sync(~0u, mark & 0xFF);
    if constexpr (WIDE) wide = __ballot_sync(~0u, mark & 0x100);
    float ca[VC], cu[VC];
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      const float2 q = js.cta[buf][s][col + 4 * k];
      ca[k] = s < cl ? q.x : 1.f;
      cu[k] = s < cl ? q.y : 0.f;
    }
    scan8(ca, cu, crs);
    if (wide)
#pragma unroll
      for (int k = 0; k < VC; ++k) out = out || !within(ca[k], FLT_MAX);
#pragma unroll
    for (int k = 0; k < VC; ++k) {
      const float h = (crs & ((2u << s) - 1)) ? cu[k] : fmaf(ca[k], carry[k], cu[k]);  // after CTA s
      const float before = __shfl_sync(~0u, h, rank - 1, 8);
      in[k] = rank == 0 ? carry[k] : before;
      carry[k] = __shfl_sync(~0u, h, 7, 8);
    }
  }
#pragma unroll
  for (int k = 0; k < VC; ++k) {
    const float h = (rs & ((2u << s) - 1)) ? u[k] : fmaf(a[k], in[k], u[k]);  // after run s
    const float before = __shfl_up_sync(~0u, h, 1, 8);
    js.in[s][col + 4 * k] = s == 0 ? in[k] : before;
    if (cl == 1) carry[k] = __shfl_sync(~0u, h, 7, 8);
  }
  __syncthreads();
  if constexpr (WIDE) {
    if (wide) {  // the same in all threads of the cluster
      const bool all = cl == 1 || __syncthreads_or(out);
      if (__syncthreads_or(own || out)) {
        join_serial(js, all ? cl : 1, all ? rank : 0, through);
        if (all)
#pragma unroll
          for (int k = 0; k < VC; ++k) carry[k] = js.A[0][col + 4 * k];
        __syncthreads();  // A is written by the next round
      }
    }
  }
  return *reinterpret_cast<const Vec<VC>*>(&js.in[w][lane * VC]);
}

// This thread's place: features c.. of batch row b, run w of CTA `rank` of the cluster.
template <int VC>
struct Place {
  int b, c0, c, cl, rank;
  bool ok, two;  // the thread has a feature, has VC of them
  __device__ __forceinline__ Place(const RecurArgs& a, int cluster) {
    cl = cluster;
    rank = cl > 1 ? (int)cluster_rank() : 0;
    const int blocks = (a.D + 32 * VC - 1) / (32 * VC), i = blockIdx.x / cl;
    b = i / blocks;
    c0 = (i - b * blocks) * 32 * VC;
    c = c0 + (threadIdx.x & 31) * VC;
    ok = c < a.D;
    two = c + VC <= a.D;
  }
  // A map's A with 1 for columns that are not the thread's own: what is read for them is not data.
  __device__ __forceinline__ Vec<VC> only_own(Vec<VC> A) const {
    if constexpr (VC == 1) return ok ? A : 1.f;
    else return make_float2(ok ? A.x : 1.f, two ? A.y : 1.f);
  }
};
template <int VC>
__device__ __forceinline__ Vec<VC> load_state(const float* p, const RecurArgs& a,
                                              const Place<VC>& at) {
  if (!p || !at.ok) return all<VC>(0.f);
  p += (size_t)at.b * a.D + at.c;
  if constexpr (VC == 1) return *p;
  else return make_float2(p[0], at.two ? p[1] : 0.f);
}
// Stores a thread's elements; of an odd row's pairs element by element, `two` of them or one.
template <typename E, int VC, bool ODD>
__device__ __forceinline__ void put(E* p, Vec<VC> v, bool two) {
  if constexpr (ODD && VC == 2) {
    Raw<E, 1>::store(p, v.x);
    if (two) Raw<E, 1>::store(p + 1, v.y);
  } else {
    Raw<E, VC>::store(p, v);
  }
}
// The state in the layout of the scans.
template <int VC>
__device__ __forceinline__ void load_carry(const float* p, const RecurArgs& a, const Place<VC>& at,
                                           float (&v)[VC]) {
  const int c = at.c0 + (threadIdx.x >> 5) * Joins<VC>::kScan + (threadIdx.x >> 3 & 3);
#pragma unroll
  for (int k = 0; k < VC; ++k) v[k] = p && c + 4 * k < a.D ? p[(size_t)at.b * a.D + c + 4 * k] : 0.f;
}
template <int VC>
__device__ __forceinline__ void store_carry(float* p, const RecurArgs& a, const Place<VC>& at,
                                            const float (&v)[VC]) {
  const int c = at.c0 + (threadIdx.x >> 5) * Joins<VC>::kScan + (threadIdx.x >> 3 & 3);
  if (p && at.rank == 0 && (threadIdx.x & 7) == 0)
#pragma unroll
    for (int k = 0; k < VC; ++k)
      if (c + 4 * k < a.D) p[(size_t)at.b * a.D + c + 4 * k] = v[k];
}
// The documents' marks of R positions from pos of a walk (position p is token p, or T - 1 - p
// with REV): lane i loads that of position pos + i.
template <int R, bool REV>
__device__ __forceinline__ unsigned load_reset(const RecurArgs& a, int b, unsigned pos) {
  const unsigned p = pos + (threadIdx.x & 31);
  if (!a.reset || (threadIdx.x & 31) >= R || p >= (unsigned)a.T) return 0;
  return a.reset[(size_t)b * a.T + (REV ? a.T - 1 - p : p)];
}

// --------------------------------------------------------------------------------- row loads
// A warp's R rows of 32 VC elements in shared memory, filled ahead by asynchronous copies of CB
// bytes: 16 where all rows start on such a boundary, else 4. ODD: rows of an odd number of
// elements. Of bf16 every second one then starts in the middle of a 4-byte word: the tile holds
// the words around a row (one more than its own), and `half` (0 or 1) is the element of the first
// word that the row starts at.
template <typename E, int VC, int R, int CB, bool ODD>
struct RowTile {
  static constexpr bool kHalves = ODD && sizeof(E) == 2;
  static constexpr int kRow = 32 * VC * (int)sizeof(E) + (kHalves ? 4 : 0);
  static constexpr int kBytes = (R * kRow + 15) / 16 * 16;
  static_assert(!kHalves || VC == 2, "a word per thread");
  // Rows row0, row0 +- D, ...: n of them; `width` elements of each are the tensor's, which ends at
  // `end`.
  template <bool REV>
  static __device__ __forceinline__ void fetch(uint32_t dst, const E* row0, unsigned D, int n,
                                               int width, const E* end) {
    const int lane = threadIdx.x & 31;
    if constexpr (kHalves) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const uintptr_t p = reinterpret_cast<uintptr_t>(REV ? rows_back(row0, i, D) : rows(row0, i, D));
        const int words = ((int)(p & 2) / 2 + min(width, 64) + 1) / 2;
        const uintptr_t src = (p & ~(uintptr_t)3) + 4 * lane;
        const uint32_t to = dst + i * kRow + 4 * lane;
        // the tensor's last word may hold one element only
        auto copy = [&](uint32_t t, uintptr_t q) {
          const int bytes = q + 4 <= reinterpret_cast<uintptr_t>(end) ? 4 : 2;
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(t), "l"(q), "r"(bytes) : "memory");
        };
        if (i < n && lane < words) copy(to, src);
        if (i < n && lane == 0 && words == 33) copy(to + 128, src + 128);
      }
    } else if constexpr (CB == 4 && kRow == 256) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        const E* src = (REV ? rows_back(row0, i, D) : rows(row0, i, D)) + lane;
        const uint32_t to = dst + i * kRow + 4 * lane;
        if (i < n && lane < width)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(src) : "memory");
        if (i < n && lane + 32 < width)
          asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + 128), "l"(src + 32) : "memory");
      }
    } else {
      constexpr int kLanes = kRow / CB, kStep = 32 / kLanes;
      static_assert(kLanes <= 32 && R % kStep == 0, "whole rows per copy");
      const int r0 = lane / kLanes, col = (lane % kLanes) * CB;
      const bool in = col < width * (int)sizeof(E);
      const E* src = (REV ? row0 - (size_t)r0 * D : row0 + (size_t)r0 * D) + col / (int)sizeof(E);
      const uint32_t to = dst + r0 * kRow + col;
#pragma unroll
      for (int i = 0; i < R; i += kStep) {
        const E* p = REV ? rows_back(src, i, D) : rows(src, i, D);
        if (in && i + r0 < n) {
          if constexpr (CB == 16)
            asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to + i * kRow), "l"(p) : "memory");
          else
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to + i * kRow), "l"(p) : "memory");
        }
      }
    }
  }
  static __device__ __forceinline__ Raw<E, VC> get(const uint8_t* tile, int i, int half) {
    const uint8_t* p = tile + i * kRow + (threadIdx.x & 31) * VC * (int)sizeof(E);
    if constexpr (kHalves) {
      const unsigned short* q = reinterpret_cast<const unsigned short*>(p) + half;
      return {(uint32_t)q[0] | (uint32_t)q[1] << 16};
    } else {
      return *reinterpret_cast<const Raw<E, VC>*>(p);
    }
  }
};
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }
// Rounds in shared memory: the one at hand and two on their way; odd rows are a word longer, and two
// CTAs per SM have room for one round less.
template <bool ODD>
constexpr int kStagesOf = ODD ? 2 : 3;

// ----------------------------------------------------------------------------------- forward
template <typename E, typename GT, int VC, int R, int CB, bool ODD>
struct FwdTiles {
  using X = RowTile<E, VC, R, CB, ODD>;
  using G = RowTile<GT, VC, R, CB, ODD>;
  static constexpr int kStage = X::kBytes + G::kBytes;  // of one warp
  static constexpr size_t kSmem = (size_t)kWarps * kStagesOf<ODD> * kStage;
};
// A run of decays given as values, token by token from its tile (which stays until the next round's
// first copies).
template <typename Tl, int VC>
struct FwdRun {
  const uint8_t* tile;
  unsigned odd0, rs;
  int n;
  __device__ __forceinline__ Vec<VC> operator()(Vec<VC> h) const {
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int half = (int)(odd0 + i) & 1;
      const auto x = Tl::X::get(tile, i, half).get();
      h = pick(rs >> i & 1, x, fma(Tl::G::get(tile + Tl::X::kBytes, i, half).get(), h, x));
    }
    return h;
  }
};
template <typename E, typename GT, bool SIG, int VC, int R, int CB, bool ODD>
__global__ void __launch_bounds__(kThreads, 2)
    recur_fwd_kernel(const __grid_constant__ RecurArgs a, const int cluster) {
  using V = Vec<VC>;
  using Tl = FwdTiles<E, GT, VC, R, CB, ODD>;
  constexpr int kStages = kStagesOf<ODD>;
  extern __shared__ __align__(16) uint8_t tiles[];
  __shared__ Joins<VC> js;
  const Place<VC> at(a, cluster);
  const unsigned T = a.T, D = a.D, stride = (unsigned)at.cl * kWarps * R;
  const int w = threadIdx.x >> 5;
  uint8_t* mine = tiles + w * kStages * Tl::kStage;
  const size_t base = (size_t)at.b * T * D + at.c0, all_n = (size_t)a.B * T * D;
  const E* X = static_cast<const E*>(a.X) + base;
  const GT* G = static_cast<const GT*>(a.G) + base;
  E* H = static_cast<E*>(a.H) + base + (at.c - at.c0);
  unsigned mark[kStages - 1];
  auto fetch = [&](unsigned p, int st) {
    if (p < T) {
      const int n = min(T - p, (unsigned)R);
      const uint32_t dst = smem_u32(mine) + st * Tl::kStage;
      Tl::X::template fetch<false>(dst, X + (size_t)p * D, D, n, a.D - at.c0, static_cast<const E*>(a.X) + all_n);
      Tl::G::template fetch<false>(dst + Tl::X::kBytes, G + (size_t)p * D, D, n, a.D - at.c0,
                                   static_cast<const GT*>(a.G) + all_n);
    }
    cp_commit();
  };
  unsigned pos = ((unsigned)at.rank * kWarps + w) * R;
  const unsigned rounds = (T + stride - 1) / stride;
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) {
    fetch(pos + k * stride, k);
    mark[k] = load_reset<R, false>(a, at.b, pos + k * stride);
  }
  float carry[VC];
  load_carry(a.h0, a, at, carry);
  join_init(js, at.cl);  // (behind the loads of h0, which h_final may overwrite)
  int st = 0, ahead = kStages - 1;
  for (unsigned round = 0; round < rounds; ++round, pos += stride) {
    V av[R], u[R];
    const int n = pos >= T ? 0 : (int)min(T - pos, (unsigned)R);
    const unsigned rs = __ballot_sync(~0u, mark[0] != 0);
#pragma unroll
    for (int k = 0; k + 1 < kStages - 1; ++k) mark[k] = mark[k + 1];
    mark[kStages - 2] = load_reset<R, false>(a, at.b, pos + (kStages - 1) * stride);
    fetch(pos + (kStages - 1) * stride, ahead);
    cp_wait<kStages - 1>();
    __syncwarp();
    const uint8_t* tile = mine + st * Tl::kStage;
    if (++st == kStages) st = 0;
    if (++ahead == kStages) ahead = 0;
    V mA = all<VC>(1.f), mU = all<VC>(0.f);
    const unsigned odd0 = (unsigned)at.b * T + pos;  // its parity is that of the first row's start
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const int half = (int)(odd0 + i) & 1;
      u[i] = Tl::X::get(tile, i, half).get();
      Raw<GT, VC> g = Tl::G::get(tile + Tl::X::kBytes, i, half);
      if constexpr (SIG) {
        g.hold();
        V na;
        gate_of<GT>(g.get(), av[i], na);
        u[i] = mul(na, u[i]);
      } else {
        av[i] = g.get();
      }
    }
    __syncwarp();  // the stage may be filled again
    if (rs == 0 && n == R) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        mA = mul(mA, av[i]);
        mU = fma(av[i], mU, u[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n) {
          mA = mul(mA, av[i]);
          mU = pick(rs >> i & 1, u[i], fma(av[i], mU, u[i]));
        }
    }
    if constexpr (!SIG) mA = at.only_own(mA);
    V h = join_runs<VC, !SIG>(js, round, at.cl, at.rank, mA, mU, rs != 0, carry, a.err,
                              FwdRun<Tl, VC>{tile, odd0, rs, n});
    if (!at.ok) continue;
    E* out = H + (size_t)pos * D;
    if (rs == 0 && n == R) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        h = fma(av[i], h, u[i]);
        put<E, VC, ODD>(rows(out, i, D), h, at.two);
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n) {
          h = pick(rs >> i & 1, u[i], fma(av[i], h, u[i]));
          put<E, VC, ODD>(rows(out, i, D), h, at.two);
        }
    }
  }
  store_carry(a.h_final, a, at, carry);
  if (at.cl > 1 && js.abort_flag) __nanosleep(100000);  // let what the others send land
}

// ---------------------------------------------------------------------------------- backward
// The adjoint runs backwards over the tokens: with c the part of D_{t-1} that comes from token t,
//   D_t = dH_t + c_{t+1},  c_t = a_t D_t  (0 at a document's first token),
// a recurrence in c of the same form, walked from the last token. The decays stay in registers
// between the two passes over a run; the other inputs are read from shared memory again.
template <typename E, typename GT, bool SIG, int VC, int R, int CB, bool ODD>
struct BwdTiles {
  using X = RowTile<E, VC, R, CB, ODD>;
  using G = RowTile<GT, VC, R, CB, ODD>;
  static constexpr int oD = G::kBytes, oH = oD + X::kBytes, oX = oH + X::kBytes;
  static constexpr int kStage = oX + (SIG ? X::kBytes : 0);  // of one warp
  static constexpr size_t kSmem = (size_t)kWarps * kStagesOf<ODD> * kStage;
};
template <typename Tl, int VC>
struct BwdRun {
  const uint8_t* tile;
  unsigned odd0, rs;
  int n;
  __device__ __forceinline__ Vec<VC> operator()(Vec<VC> c) const {
#pragma unroll 1
    for (int i = 0; i < n; ++i) {
      const int half = (int)(odd0 + i) & 1;
      const Vec<VC> Dt = add(Tl::X::get(tile + Tl::oD, i, half).get(), c);
      c = pick(rs >> i & 1, all<VC>(0.f), mul(Tl::G::get(tile, i, half).get(), Dt));
    }
    return c;
  }
};
template <typename E, typename GT, bool SIG, int VC, int R, int CB, bool ODD>
__global__ void __launch_bounds__(kThreads, 2)
    recur_bwd_kernel(const __grid_constant__ RecurArgs a, const int cluster) {
  using V = Vec<VC>;
  using Tl = BwdTiles<E, GT, SIG, VC, R, CB, ODD>;
  constexpr int kStages = kStagesOf<ODD>;
  extern __shared__ __align__(16) uint8_t tiles[];
  __shared__ Joins<VC> js;
  const Place<VC> at(a, cluster);
  const unsigned T = a.T, D = a.D, stride = (unsigned)at.cl * kWarps * R;
  const int w = threadIdx.x >> 5;
  uint8_t* mine = tiles + w * kStages * Tl::kStage;
  const size_t base = (size_t)at.b * T * D + at.c0, all_n = (size_t)a.B * T * D;
  const E* X = static_cast<const E*>(a.X) + base;
  const GT* G = static_cast<const GT*>(a.G) + base;
  const E* H = static_cast<const E*>(a.H_in) + base;
  const E* dH = static_cast<const E*>(a.dH) + base;
  E* dX = static_cast<E*>(a.dX) + base + (at.c - at.c0);
  GT* dG = static_cast<GT*>(a.dG) + base + (at.c - at.c0);
  unsigned mark[kStages - 1];
  // position p is token T - 1 - p; the H tile holds the states before the tokens, from row T - 2 - p
  auto fetch = [&](unsigned p, int st) {
    if (p < T) {
      const int n = min(T - p, (unsigned)R), nh = min(T - 1 - p, (unsigned)R), width = a.D - at.c0;
      const uint32_t dst = smem_u32(mine) + st * Tl::kStage;
      const size_t o = (size_t)(T - 1 - p) * D;
      Tl::G::template fetch<true>(dst, G + o, D, n, width, static_cast<const GT*>(a.G) + all_n);
      Tl::X::template fetch<true>(dst + Tl::oD, dH + o, D, n, width, static_cast<const E*>(a.dH) + all_n);
      if (nh > 0)
        Tl::X::template fetch<true>(dst + Tl::oH, H + o - D, D, nh, width, static_cast<const E*>(a.H_in) + all_n);
      if constexpr (SIG)
        Tl::X::template fetch<true>(dst + Tl::oX, X + o, D, n, width, static_cast<const E*>(a.X) + all_n);
    }
    cp_commit();
  };
  unsigned pos = ((unsigned)at.rank * kWarps + w) * R;
  const unsigned rounds = (T + stride - 1) / stride;
#pragma unroll
  for (int k = 0; k < kStages - 1; ++k) {
    fetch(pos + k * stride, k);
    mark[k] = load_reset<R, true>(a, at.b, pos + k * stride);
  }
  float carry[VC];
  load_carry(a.dh_final, a, at, carry);
  join_init(js, at.cl);  // (behind the loads of dh_final, which dh0 may overwrite)
  int st = 0, ahead = kStages - 1;
  for (unsigned round = 0; round < rounds; ++round, pos += stride) {
    V av[R], na[SIG ? R : 1];
    const int n = pos >= T ? 0 : (int)min(T - pos, (unsigned)R);
    const unsigned rs = __ballot_sync(~0u, mark[0] != 0);
#pragma unroll
    for (int k = 0; k + 1 < kStages - 1; ++k) mark[k] = mark[k + 1];
    mark[kStages - 2] = load_reset<R, true>(a, at.b, pos + (kStages - 1) * stride);
    __syncwarp();  // all lanes have left the last round's tile, which is filled next
    fetch(pos + (kStages - 1) * stride, ahead);
    cp_wait<kStages - 1>();
    __syncwarp();
    const uint8_t* tile = mine + st * Tl::kStage;
    if (++st == kStages) st = 0;
    if (++ahead == kStages) ahead = 0;
    V mA = all<VC>(1.f), mU = all<VC>(0.f);
    const unsigned odd0 = (unsigned)at.b * T + T - 1 - pos;  // parity of the first row's start
#pragma unroll
    for (int i = 0; i < R; ++i) {
      Raw<GT, VC> g = Tl::G::get(tile, i, (int)(odd0 + i) & 1);
      if constexpr (SIG) {
        g.hold();
        gate_of<GT>(g.get(), av[i], na[i]);
      } else {
        av[i] = g.get();
      }
    }
    const bool plain = rs == 0 && n == R && pos + R < T;
    if (plain) {
#pragma unroll
      for (int i = 0; i < R; ++i) {
        mA = mul(mA, av[i]);
        mU = mul(av[i], add(Tl::X::get(tile + Tl::oD, i, (int)(odd0 + i) & 1).get(), mU));
      }
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n) {
          mA = mul(mA, av[i]);
          mU = pick(rs >> i & 1, all<VC>(0.f),
                     mul(av[i], add(Tl::X::get(tile + Tl::oD, i, (int)(odd0 + i) & 1).get(), mU)));
        }
    }
    if constexpr (!SIG) mA = at.only_own(mA);
    V c = join_runs<VC, !SIG>(js, round, at.cl, at.rank, mA, mU, rs != 0, carry, a.err,
                              BwdRun<Tl, VC>{tile, odd0, rs, n});
    if (!at.ok || n == 0) continue;
    const size_t o = (size_t)(T - 1 - pos) * D;
    auto token = [&](int i, V prev, bool first) {
      const V Dt = add(Tl::X::get(tile + Tl::oD, i, (int)(odd0 + i) & 1).get(), c);
      c = mul(av[i], Dt);
      V x = Dt, g;
      if constexpr (SIG) {
        x = mul(na[i], Dt);
        // D_t (h_{t-1} - x) a (1 - a)
        g = mul(mul(c, na[i]), fma(Tl::X::get(tile + Tl::oX, i, (int)(odd0 + i) & 1).get(), all<VC>(-1.f), prev));
      } else {
        g = first ? all<VC>(0.f) : mul(Dt, prev);
      }
      if (first) c = all<VC>(0.f);
      put<E, VC, ODD>(rows_back(dX + o, i, D), x, at.two);
      put<GT, VC, ODD>(rows_back(dG + o, i, D), g, at.two);
    };
    if (plain) {
#pragma unroll
      for (int i = 0; i < R; ++i) token(i, Tl::X::get(tile + Tl::oH, i, (int)(odd0 + i + 1) & 1).get(), false);
    } else {
#pragma unroll
      for (int i = 0; i < R; ++i)
        if (i < n) {
          const bool first = rs >> i & 1;
          V prev = all<VC>(0.f);
          if (!first) {
            if (pos + i == T - 1) prev = load_state<VC>(a.h0, a, at);
            else prev = Tl::X::get(tile + Tl::oH, i, (int)(odd0 + i + 1) & 1).get();
          }
          token(i, prev, first);
        }
    }
  }
  store_carry(a.dh0, a, at, carry);
  if (at.cl > 1 && js.abort_flag) __nanosleep(100000);
}

// -------------------------------------------------------------------------------------- step
// CTA (b, y, z): a block of VC features a thread of row b; a grid's y ends at 65535, so that very wide
// rows go on in z. Rows that name one slot are one chain: the first of them applies all in order,
// the others leave.
constexpr int kStepThreads = 128;
template <typename E, typename GT, bool SIG, int VC>
__global__ void __launch_bounds__(kStepThreads) recur_step_kernel(const __grid_constant__ RecurArgs a) {
  const int b = blockIdx.x;
  const unsigned block = blockIdx.z * gridDim.y + blockIdx.y;
  const unsigned c = (block * kStepThreads + threadIdx.x) * VC;  // (below 2^31 + 2^17)
  const bool ok = c < (unsigned)a.D;
  const int slot = a.slots ? a.slots[b] : b;
  if (slot < 0) return;
  if (slot >= a.n_slots) {
    if (block == 0 && threadIdx.x == 0) atomicOr(a.err, ERR_RANGE);
    return;
  }
  float* st = a.state + (size_t)slot * a.D + c;
  Raw<E, VC> rx;
  Raw<GT, VC> rg;
  Vec<VC> h;
  auto fetch = [&](int row) {
    rx.load(static_cast<const E*>(a.X) + (size_t)row * a.D + c);
    rg.load(static_cast<const GT*>(a.G) + (size_t)row * a.D + c);
  };
  auto token = [&](int row) {
    if constexpr (SIG) rg.hold();
    Vec<VC> aa = rg.get(), u = rx.get(), na;
    if constexpr (SIG) {
      gate_of<GT>(aa, aa, na);
      u = mul(u, na);
    }
    h = fma(aa, h, u);
    Raw<E, VC>::store(static_cast<E*>(a.H) + (size_t)row * a.D + c, h);
  };
  if (ok) {
    fetch(b);
    if constexpr (VC == 1) h = *st;
    else h = *reinterpret_cast<const float2*>(st);
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
// CTAs along the sequence. A cluster lies within one GPC, so that fewer CTAs than two per SM are
// resident with the larger sizes (kResident, from the occupancy query). The choice is the least
// time by the measured times of a round, with two rounds more per wave for its start and end
// (32768 x 2560 forward: 407 us with 1, 188 with 3, 139 with 6, 199 with 8).
int cluster_of(const RecurArgs& a, long long ctas, int run) {
  constexpr int kResident[kMaxCluster + 1] = {0, 296, 296, 279, 284, 280, 270, 259, 264};
  int best = 1;
  long long least = 0;
  for (int cl = 1; cl <= kMaxCluster; ++cl) {
    if (cl > 1 && (long long)(cl - 1) * kWarps * run >= a.T) break;  // CTAs without a token
    const long long waves = (ctas * cl + kResident[cl] - 1) / kResident[cl];
    const long long tile = (long long)cl * kWarps * run, rounds = (a.T + tile - 1) / tile;
    // tenths of a microsecond: a round of a CTA alone on its SM, the join of a cluster, a second CTA
    const long long round = 15 + (cl > 1 ? 6 : 0) + (ctas * cl > kResident[1] / 2 ? 10 : 0);
    const long long cost = waves * (rounds + 2) * round;
    if (cl == 1 || cost < least) best = cl, least = cost;
  }
  return best;
}
template <typename K>
cudaError_t launch(K kernel, size_t smem, const RecurArgs& a, int vc, int run, cudaStream_t s) {
  const long long blocks = (long long)a.B * ((a.D + 32 * vc - 1) / (32 * vc));
  const int cl = cluster_of(a, blocks, run);
  if (blocks * cl >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(blocks * cl));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = cl;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = cl > 1;
  count_launches(1);
  e = cudaLaunchKernelEx(&cfg, kernel, a, cl);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename E, typename GT, bool SIG, int VC, int CB, bool ODD>
cudaError_t fwd(const RecurArgs& a, cudaStream_t s) {
  constexpr int R = sizeof(GT) * VC == 8 ? 8 : 16;  // what a stage of shared memory has room for
  return launch(recur_fwd_kernel<E, GT, SIG, VC, R, CB, ODD>, FwdTiles<E, GT, VC, R, CB, ODD>::kSmem, a, VC, R, s);
}
template <typename E, typename GT, bool SIG, int VC, int CB, bool ODD>
cudaError_t bwd(const RecurArgs& a, cudaStream_t s) {
  constexpr int R = 8;
  return launch(recur_bwd_kernel<E, GT, SIG, VC, R, CB, ODD>, BwdTiles<E, GT, SIG, VC, R, CB, ODD>::kSmem, a, VC, R, s);
}

}  // namespace

// bf16 takes two features a thread; copies are of 16 bytes where all rows start on such a boundary.
#define RECUR_DISPATCH(f)                                                \
  do {                                                                   \
    if (a.bf16 && a.sigmoid)                                             \
      return a.D % 8 == 0   ? f<bf16, bf16, true, 2, 16, false>(a, s)    \
             : a.D % 2 == 0 ? f<bf16, bf16, true, 2, 4, false>(a, s)     \
                            : f<bf16, bf16, true, 2, 4, true>(a, s);     \
    if (a.bf16)                                                          \
      return a.D % 8 == 0   ? f<bf16, float, false, 2, 16, false>(a, s)  \
             : a.D % 2 == 0 ? f<bf16, float, false, 2, 4, false>(a, s)   \
                            : f<bf16, float, false, 2, 4, true>(a, s);   \
    if (a.sigmoid)                                                       \
      return a.D % 4 == 0 ? f<float, float, true, 1, 16, false>(a, s)    \
                          : f<float, float, true, 1, 4, false>(a, s);    \
    return a.D % 4 == 0 ? f<float, float, false, 1, 16, false>(a, s)     \
                        : f<float, float, false, 1, 4, false>(a, s);     \
  } while (0)

cudaError_t recur_fwd(const RecurArgs& a, cudaStream_t s) { RECUR_DISPATCH(fwd); }
cudaError_t recur_bwd(const RecurArgs& a, cudaStream_t s) { RECUR_DISPATCH(bwd); }
cudaError_t recur_step(const RecurArgs& a, cudaStream_t s) {
  const int vc = a.D % 2 == 0 ? 2 : 1;
  const int cols = kStepThreads * vc;
  const int blocks = (a.D + cols - 1) / cols, z = (blocks + 65534) / 65535;
  const dim3 grid(a.B, (blocks + z - 1) / z, z);
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
