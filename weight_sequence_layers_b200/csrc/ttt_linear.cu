// Linear layer with bias, activation, multiplier and residual in its epilogue, forward and
// backward (include/ttt.h), on the tensor cores.
//
// Every product is D[i, j] = sum_k A[i, k] B[j, k] with bf16 operands, each stored with k
// contiguous (K-major) or with its own index contiguous (MN-major):
//   forward  P  = X W^T   rows tokens,    columns outputs, k inputs:  X, W K-major
//   dX = dP W             rows tokens,    columns inputs,  k outputs: dP K-major, W MN-major
//   dW = dP^T X           rows outputs,   columns inputs,  k tokens:  dP, X MN-major
// TMA fills what lies outside a matrix with zeros, so that every size is a number of full tiles.
//
// Two kernels:
//   pair: 256 x 256 tiles on CTA pairs (cta_group::2), persistent, two accumulators in TMEM so
//         that the epilogue of one tile runs under the products of the next. Bound by the tensor
//         cores.
//   split: 128 x NT tiles with the roles of rows and columns exchanged (the weights' rows are the
//         MMA's 128 rows, NT = 16..128 tokens its columns), one tile a CTA and several CTAs an
//         SM; the CTAs of a cluster share the contraction of one tile and add their parts through
//         distributed shared memory in a fixed order. For few tiles: decode steps, which read the
//         weights once (bound by HBM), and small matrices.
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "pair_tc.cuh"

namespace tttk {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kSMs = 148;
constexpr int BK = 64;  // contraction per stage: one 128-byte swizzled row

// sigmoid with the hardware's exponential and reciprocal: 2 steps of float32 each and one for
// every unit of |z|, below the bf16 result's half step
__device__ __forceinline__ float sigm(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// The epilogue: P = D + bias, Y = act(P) mul + residual at [row, col] of a row-major matrix.
struct Epi {
  const float* bias;  // by column
  const bf16 *mul, *residual;
  bf16 *Y, *P;
  size_t ld;
  int silu;
};

// ================================================================================ pair tiles
constexpr int PT = 256;  // tile rows and columns
constexpr int kPairThreads = 320, kEpiWarps = 8;
constexpr int kPairStages = 6;
constexpr uint32_t kHalf = 128 * BK * 2;      // 16 KB: this CTA's 128 rows of A, or of B
constexpr uint32_t kPairStage = 2 * kHalf;
constexpr uint32_t kTurn = 32 * 32 * 4;       // an epilogue warp's block of the accumulator
struct __align__(8) PairBars {
  uint64_t full[kPairStages], empty[kPairStages], acc_full[2], acc_empty[2];
  uint32_t tmem_base;
  int abort_flag;
};
constexpr size_t kPairSmem = kPairStages * kPairStage + kEpiWarps * kTurn + sizeof(PairBars) + 1024;
static_assert(kPairSmem <= 232448, "shared memory of one CTA");

struct PairArgs {
  int rows, cols, nkb;     // of D; 64-wide blocks of k
  int tm, tn;              // tiles
  Epi e;
  unsigned* err;
};
// Tile t: groups of kGroup tile rows, column by column, so that the tiles at work at one time
// share their rows of A and of B in L2.
constexpr int kGroup = 8;
__device__ __forceinline__ void pair_tile(const PairArgs& p, int t, int& m0, int& n0) {
  const int g = t / (kGroup * p.tn), rem = t - g * kGroup * p.tn;
  const int gm = min(kGroup, p.tm - g * kGroup), n = rem / gm;
  m0 = (g * kGroup + rem - n * gm) * PT;
  n0 = n * PT;
}
// A tile's half operand (128 rows of A, or 128 of B) for k block kb.
template <bool MN>
__device__ __forceinline__ void pair_load(uint32_t dst, const CUtensorMap* m, uint32_t bar, int r0,
                                          int kb) {
  if constexpr (MN) {
    tma_load_2d_pair(dst, m, bar, r0, kb * BK);
    tma_load_2d_pair(dst + kHalf / 2, m, bar, r0 + 64, kb * BK);
  } else {
    tma_load_2d_pair(dst, m, bar, kb * BK, r0);
  }
}
template <bool MN>
__device__ __forceinline__ uint64_t operand(uint32_t addr, int kk) {
  return MN ? sdesc_sw128(addr + kk * 2048, kHalf / 2, 1024) : sdesc_sw128(addr + kk * 32, 16, 1024);
}
__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) v[2 * k] = bf16lo(w[k]), v[2 * k + 1] = bf16hi(w[k]);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}

// Eight neighbouring outputs from their sums y (w: scratch).
template <bool AUX>
__device__ __forceinline__ void finish8(const Epi& e, size_t o, const float (&b)[8], const uint4& mu,
                                        const uint4& re, float (&y)[8], float (&w)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] += b[k];
  if (e.P) *reinterpret_cast<uint4*>(e.P + o) = pack8(y);
  if (e.silu)
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] *= sigm(y[k]);
  if (AUX && e.mul) {
    unpack8(mu, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] *= w[k];
  }
  if (AUX && e.residual) {
    unpack8(re, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] += w[k];
  }
  *reinterpret_cast<uint4*>(e.Y + o) = pack8(y);
}

// Warps: 0 TMA loads, 1 MMA (the leader's), 2-9 epilogue (two per TMEM lane quadrant, 128
// columns each). The leader's barriers count both CTAs' loads and drained accumulators; commits
// arrive on both CTAs' stage and accumulator barriers.
template <bool AMN, bool BMN, bool AUX>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                       const __grid_constant__ PairArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  PairBars* bars = reinterpret_cast<PairBars*>(smem + kPairStages * kPairStage + kEpiWarps * kTurn);
  const uint32_t stage0 = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int half = (int)rank * 128;
  const int tiles = p.tm * p.tn, first = blockIdx.x / 2, step = gridDim.x / 2;
  const Abort ab{&bars->abort_flag, p.err};
#define PB(x) smem_u32(&bars->x)
  if (threadIdx.x == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(PB(full[s]), 1);
      mbar_init(PB(empty[s]), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(PB(acc_full[a]), 1);
      mbar_init(PB(acc_empty[a]), 2 * kEpiWarps);
    }
    bars->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&ta);
    tma_prefetch_desc(&tb);
  }
  if (warp == 1) {
    tmem_alloc_pair(PB(tmem_base), 2 * PT);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        int m0, n0;
        pair_tile(p, t, m0, n0);
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!(ok = mbar_wait(PB(empty[s]), ph ^ 1, ab))) break;
          if (leader) mbar_arrive_expect_tx(PB(full[s]), 2 * kPairStage);
          const uint32_t bar = peer_addr(PB(full[s]), 0), sa = stage0 + s * kPairStage;
          pair_load<AMN>(sa, &ta, bar, m0 + half, kb);
          pair_load<BMN>(sa + kHalf, &tb, bar, n0 + half, kb);
          if (++s == kPairStages) { s = 0; ph ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      constexpr uint32_t id = idesc_bf16(PT, PT, AMN, BMN);
      bool ok = true;
      for (int t = first; t < tiles && ok; t += step) {
        if (!(ok = mbar_wait_cluster(PB(acc_empty[acc]), aph ^ 1, ab))) break;
        tc_fence_after();
        for (int kb = 0; kb < p.nkb; ++kb) {
          if (!(ok = mbar_wait(PB(full[s]), ph, ab))) break;
          tc_fence_after();
          const uint32_t sa = stage0 + s * kPairStage;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            mma_bf16_pair(tmem + acc * PT, operand<AMN>(sa, kk), operand<BMN>(sa + kHalf, kk), id,
                          (kb | kk) != 0);
          mma_commit_pair(PB(empty[s]));
          if (++s == kPairStages) { s = 0; ph ^= 1; }
        }
        if (ok) mma_commit_pair(PB(acc_full[acc]));
        if (++acc == 2) { acc = 0; aph ^= 1; }
      }
    }
  } else {
    // A thread reads a row of the accumulator. Alone, an output is written as such, 64 bytes of a
    // row a thread (16384 x 2048 x 2048: 94 us; 98 by the other way). With a multiplier or a
    // residual (AUX), rows are read and written best by several threads: each 32 x 32 block goes
    // through shared memory (16-byte chunks swizzled by the row) and comes back as 8 columns of 4
    // rows a thread, a row's 4 threads side by side (100 us; 108 row by row).
    const int q = warp & 3, h = (warp - 2) / 4;
    float* turn = reinterpret_cast<float*>(smem + kPairStages * kPairStage + (warp - 2) * kTurn);
    const int c8 = 8 * (lane % 4), r8 = lane / 4;
    const Epi& e = p.e;
    int acc = 0;
    uint32_t aph = 0;
    for (int t = first; t < tiles; t += step) {
      int m0, n0;
      pair_tile(p, t, m0, n0);
      m0 += half + q * 32;
      if (!mbar_wait(PB(acc_full[acc]), aph, ab)) break;
      __syncwarp();
      tc_fence_after();
#pragma unroll 1
      for (int cb = 4 * h; cb < 4 * h + 4; ++cb) {
        float v[32];
        if constexpr (!AUX) {
          tmem_ld32(tmem_addr(tmem, q * 32, acc * PT + cb * 32), v);
          tmem_wait_ld();
          const int row = m0 + lane, c0 = n0 + 32 * cb;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int col = c0 + 8 * j;
            if (row >= p.rows || col >= p.cols) continue;
            float b[8], y[8], w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) b[k] = 0.f, y[k] = v[8 * j + k];
            if (e.bias) {
              *reinterpret_cast<float4*>(b) = *reinterpret_cast<const float4*>(e.bias + col);
              *reinterpret_cast<float4*>(b + 4) = *reinterpret_cast<const float4*>(e.bias + col + 4);
            }
            const uint4 none = make_uint4(0, 0, 0, 0);
            finish8<false>(e, (size_t)row * e.ld + col, b, none, none, y, w);
          }
          __syncwarp();
          continue;
        }
        const int col = n0 + 32 * cb + c8;
        const bool cok = col < p.cols;  // columns come in eights
        uint4 mu[4], re[4];
        float b[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = m0 + 8 * i + r8;
          const size_t o = (size_t)row * e.ld + col;
          if (cok && row < p.rows) {
            if (e.mul) mu[i] = *reinterpret_cast<const uint4*>(e.mul + o);
            if (e.residual) re[i] = *reinterpret_cast<const uint4*>(e.residual + o);
          }
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) b[k] = 0.f;
        if (e.bias && cok) {
          *reinterpret_cast<float4*>(b) = *reinterpret_cast<const float4*>(e.bias + col);
          *reinterpret_cast<float4*>(b + 4) = *reinterpret_cast<const float4*>(e.bias + col + 4);
        }
        tmem_ld32(tmem_addr(tmem, q * 32, acc * PT + cb * 32), v);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 8; ++c)
          *reinterpret_cast<float4*>(turn + lane * 32 + ((c ^ (lane & 7)) << 2)) =
              make_float4(v[4 * c], v[4 * c + 1], v[4 * c + 2], v[4 * c + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int r = 8 * i + r8, row = m0 + r;
          if (!cok || row >= p.rows) continue;
          float y[8], w[8];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float4 x = *reinterpret_cast<const float4*>(
                turn + r * 32 + (((c8 / 4 + k) ^ (r & 7)) << 2));
            y[4 * k] = x.x; y[4 * k + 1] = x.y; y[4 * k + 2] = x.z; y[4 * k + 3] = x.w;
          }
          finish8<true>(e, (size_t)row * e.ld + col, b, mu[i], re[i], y, w);
        }
        __syncwarp();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(PB(acc_empty[acc]));
        else mbar_arrive_cluster(peer_addr(PB(acc_empty[acc]), 0));
      }
      if (++acc == 2) { acc = 0; aph ^= 1; }
    }
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // no MMA of the leader still writes the peer's TMEM
  if (bars->abort_flag) __nanosleep(100000);  // let any load issued before the abort land
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 2 * PT);
  }
#undef PB
}

// =============================================================================== split tiles
// D^T tiles: 128 rows are "features" f (rows of operand A), NT columns "tokens" t (of B); the
// output at [t, f] is row-major with f contiguous, so that a warp's 32 rows are one 64-byte piece
// of a token's row. Warps: 0 TMA, 1 MMA, 2-5 epilogue.
constexpr int kSplitThreads = 192;
constexpr int kMaxSplit = 8;
struct SplitArgs {
  int feats, toks, nkb;
  int tf, tt, split;  // tiles of features and of tokens, CTAs of a cluster
  Epi e;
  unsigned* err;
};
template <int NT>
struct SplitLayout {
  static constexpr uint32_t kA = 128 * BK * 2, kB = NT * BK * 2, kStage = kA + kB;
  static constexpr int kStages = NT == 16 ? 3 : NT <= 64 ? 4 : 3;  // two CTAs an SM, three with NT = 16
  // The parts of a tile that come from the cluster's CTAs: in their own place where that is
  // small, else over the stages, once all CTAs have read these.
  static constexpr bool kOwnParts = NT <= 32;
  static constexpr uint32_t kParts = NT * 128 * 4, kOffParts = kOwnParts ? kStages * kStage : 0;
  static constexpr uint32_t kOffBars = kStages * kStage + (kOwnParts ? kParts : 0);
  static_assert(kOwnParts || kStages * kStage >= kParts, "room for the parts");
};
struct __align__(8) SplitBars {
  uint64_t full[4], empty[4], acc;
  uint32_t tmem_base;
  int abort_flag;
};
template <int NT>
constexpr size_t split_smem() { return SplitLayout<NT>::kOffBars + sizeof(SplitBars) + 1024; }

template <int NT, bool AMN, bool BMN>
__global__ void __launch_bounds__(kSplitThreads)
    linear_split_kernel(const __grid_constant__ CUtensorMap ta, const __grid_constant__ CUtensorMap tb,
                        const __grid_constant__ SplitArgs p) {
  static_assert(!BMN || NT >= 64, "an MN-major operand comes in panels of 64");
  using L = SplitLayout<NT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  SplitBars* bars = reinterpret_cast<SplitBars*>(smem + L::kOffBars);
  const uint32_t stage0 = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int S = p.split, rank = S > 1 ? (int)cluster_rank() : 0;
  const int tile = blockIdx.x / S, f0 = (tile % p.tf) * 128, t0 = (tile / p.tf) * NT;
  const int k_lo = (int)((long long)p.nkb * rank / S), k_hi = (int)((long long)p.nkb * (rank + 1) / S);
  const Abort ab{&bars->abort_flag, p.err};
  constexpr uint32_t kCols = NT < 32 ? 32 : NT;
#define SB(x) smem_u32(&bars->x)
  auto load = [&](int kb) {
    const int st = (kb - k_lo) % L::kStages;
    const uint32_t bar = SB(full[st]), sa = stage0 + st * L::kStage, sb = sa + L::kA;
    mbar_arrive_expect_tx(bar, L::kStage);
    if constexpr (AMN) {
      tma_load_2d(sa, &ta, bar, f0, kb * BK);
      tma_load_2d(sa + 8192, &ta, bar, f0 + 64, kb * BK);
    } else {
      tma_load_2d(sa, &ta, bar, kb * BK, f0);
    }
    if constexpr (BMN) {
#pragma unroll
      for (int j = 0; j < NT / 64; ++j) tma_load_2d(sb + 8192 * j, &tb, bar, t0 + 64 * j, kb * BK);
    } else {
      tma_load_2d(sb, &tb, bar, kb * BK, t0);
    }
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(SB(full[s]), 1);
      mbar_init(SB(empty[s]), 1);
    }
    mbar_init(SB(acc), 1);
    bars->abort_flag = 0;
    fence_barrier_init();
    // the first loads run while the other warps get ready
    for (int kb = k_lo; kb < min(k_hi, k_lo + L::kStages); ++kb) load(kb);
  }
  if (warp == 1) {
    tmem_alloc(SB(tmem_base), kCols);
    tmem_relinquish();
  }
  // (a CTA's shared memory may be written by the others once all have started)
  __syncwarp();
  if (S > 1 && L::kOwnParts) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  if (warp == 0) {
    if (lane == 0)
      for (int kb = k_lo + L::kStages; kb < k_hi; ++kb) {
        const int i = kb - k_lo;
        if (!mbar_wait(SB(empty[i % L::kStages]), (i / L::kStages - 1) & 1, ab)) break;
        load(kb);
      }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t id = idesc_bf16(128, NT, AMN, BMN);
      for (int kb = k_lo; kb < k_hi; ++kb) {
        const int i = kb - k_lo, s = i % L::kStages;
        if (!mbar_wait(SB(full[s]), (i / L::kStages) & 1, ab)) break;
        tc_fence_after();
        const uint32_t sa = stage0 + s * L::kStage, sb = sa + L::kA;
#pragma unroll
        for (int kk = 0; kk < BK / 16; ++kk)
          mma_bf16_ss(tmem, AMN ? sdesc_sw128(sa + kk * 2048, 8192, 1024) : sdesc_sw128(sa + kk * 32, 16, 1024),
                      BMN ? sdesc_sw128(sb + kk * 2048, 8192, 1024) : sdesc_sw128(sb + kk * 32, 16, 1024),
                      id, i > 0 || kk > 0);
        mma_commit(SB(empty[s]));
      }
      mma_commit(SB(acc));
    }
  }
  __syncwarp();
  // The outputs of this CTA: its share of the tile's tokens, 8 features (16 bytes) at a time, a
  // token's 16 pieces side by side. The first items' operands are loaded before the sums are
  // there.
  const Epi& e = p.e;
  const int share = NT / S, first = t0 + rank * share, items = share * 16;
  constexpr int kBatch = 4;
  uint4 mu[kBatch], re[kBatch];
  const int f = f0 + 8 * (threadIdx.x % 16);  // the same piece for all of a thread's items
  auto fetch = [&](int it0) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int it = it0 + u * kSplitThreads, t = first + it / 16;
      if (it < items && t < p.toks && f < p.feats) {
        const size_t o = (size_t)t * e.ld + f;
        if (e.mul) mu[u] = *reinterpret_cast<const uint4*>(e.mul + o);
        if (e.residual) re[u] = *reinterpret_cast<const uint4*>(e.residual + o);
      }
    }
  };
  fetch(threadIdx.x);
  float b[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) b[k] = 0.f;
  if (e.bias && f < p.feats) {
    *reinterpret_cast<float4*>(b) = *reinterpret_cast<const float4*>(e.bias + f);
    *reinterpret_cast<float4*>(b + 4) = *reinterpret_cast<const float4*>(e.bias + f + 4);
  }
  if (warp >= 2) {
    mbar_wait(SB(acc), 0, ab);
    __syncwarp();
    tc_fence_after();
  }
  __syncwarp();
  if (S > 1 && L::kOwnParts) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  else if (S > 1) cluster_sync_all();  // the MMAs of all CTAs have read their stages
  else if (!L::kOwnParts) __syncthreads();
  // part of CTA c, token j of a CTA's share, feature i: parts[(c share + j) 128 + i]
  if (warp >= 2) {
    const int q = warp & 3;
#pragma unroll
    for (int c = 0; c < NT / 16; ++c) {
      if (t0 + c * 16 >= p.toks) break;
      float v[16];
      tmem_ld16(tmem_addr(tmem, q * 32, c * 16), v);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const int t = c * 16 + j, to = t / share;
        const uint32_t local = stage0 + L::kOffParts + (uint32_t)((rank * share + t - to * share) * 128 + q * 32 + lane) * 4;
        if (t0 + t < p.toks) {
          if (S > 1)
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer_addr(local, to)), "f"(v[j]) : "memory");
          else
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(local), "f"(v[j]) : "memory");
        }
      }
      __syncwarp();
    }
  }
  __syncwarp();
  if (S > 1) cluster_sync_all();
  else __syncthreads();
  const float* parts = reinterpret_cast<const float*>(smem + L::kOffParts) + 8 * (threadIdx.x % 16);
  for (int it0 = threadIdx.x; it0 < items; it0 += kBatch * kSplitThreads) {
    if (it0 != threadIdx.x) fetch(it0);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int it = it0 + u * kSplitThreads, j = it / 16, t = first + j;
      if (it >= items || t >= p.toks || f >= p.feats) continue;
      float y[8], w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = 0.f;
      for (int c = 0; c < S; ++c) {
        const float4* x = reinterpret_cast<const float4*>(parts + (c * share + j) * 128);
        const float4 lo = x[0], hi = x[1];
        y[0] += lo.x; y[1] += lo.y; y[2] += lo.z; y[3] += lo.w;
        y[4] += hi.x; y[5] += hi.y; y[6] += hi.z; y[7] += hi.w;
      }
      const size_t o = (size_t)t * e.ld + f;
      finish8<true>(e, o, b, mu[u], re[u], y, w);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (bars->abort_flag) __nanosleep(100000);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kCols);
  }
#undef SB
}

// ============================================================================ dP, dmul, dbias
// One pass over dY, P and mul: dP (rounded to bf16 for the products), dmul, and the column sums
// of dP for dbias. A thread takes 8 columns of every kRowsY-th row of its CTA's rows; the CTAs'
// sums go to `part` [gridDim.y, N] and are added in a fixed order.
constexpr int kDpX = 32, kDpY = 8;
struct DpArgs {
  int M, N, rows;  // rows of a CTA
  int silu;
  const bf16 *dY, *P, *mul;
  bf16 *dP, *dmul;  // nullable
  float* part;      // nullable
};
__global__ void __launch_bounds__(kDpX* kDpY) linear_dp_kernel(const DpArgs a) {
  __shared__ float join[kDpY][kDpX * 8 + 8];
  const int tx = threadIdx.x % kDpX, ty = threadIdx.x / kDpX;
  const int col = (blockIdx.x * kDpX + tx) * 8;
  const long long lo = (long long)blockIdx.y * a.rows, hi = min((long long)a.M, lo + a.rows);
  float sum[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) sum[k] = 0.f;
  constexpr int kBatch = 4;  // rows in flight
  if (col < a.N)
    for (long long r0 = lo + ty; r0 < hi; r0 += kBatch * kDpY) {
      uint4 qy[kBatch], qp[kBatch], qm[kBatch];
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const long long r = r0 + u * kDpY;
        const size_t o = (size_t)r * a.N + col;
        qy[u] = make_uint4(0, 0, 0, 0);
        if (r < hi) {
          qy[u] = *reinterpret_cast<const uint4*>(a.dY + o);
          if (a.P) qp[u] = *reinterpret_cast<const uint4*>(a.P + o);
          if (a.mul) qm[u] = *reinterpret_cast<const uint4*>(a.mul + o);
        }
      }
#pragma unroll
      for (int u = 0; u < kBatch; ++u) {
        const long long r = r0 + u * kDpY;
        if (r >= hi) break;
        const size_t o = (size_t)r * a.N + col;
        float dy[8];
        unpack8(qy[u], dy);
        if (a.P) {
          float p[8], m[8];
          unpack8(qp[u], p);
          if (a.dmul) {
#pragma unroll
            for (int k = 0; k < 8; ++k) m[k] = dy[k] * (a.silu ? p[k] * sigm(p[k]) : p[k]);
            *reinterpret_cast<uint4*>(a.dmul + o) = pack8(m);
          }
          if (a.silu)
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float s = sigm(p[k]);
              dy[k] *= s * (1.f + p[k] * (1.f - s));
            }
          if (a.mul) {
            unpack8(qm[u], m);
#pragma unroll
            for (int k = 0; k < 8; ++k) dy[k] *= m[k];
          }
          if (a.dP) *reinterpret_cast<uint4*>(a.dP + o) = pack8(dy);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) sum[k] += dy[k];
      }
    }
  if (!a.part) return;
#pragma unroll
  for (int k = 0; k < 8; ++k) join[ty][tx * 8 + k] = sum[k];
  __syncthreads();
  const int c = threadIdx.x;  // kDpX * 8 columns, kDpX * kDpY threads
  if (blockIdx.x * kDpX * 8 + c < a.N) {
    float t = 0.f;
#pragma unroll
    for (int y = 0; y < kDpY; ++y) t += join[y][c];
    a.part[(size_t)blockIdx.y * a.N + blockIdx.x * kDpX * 8 + c] = t;
  }
}
static_assert(kDpX * 8 == kDpX * kDpY, "a thread per column in the join");
__global__ void __launch_bounds__(256) linear_dbias_kernel(const float* part, int n, int N, float* dbias) {
  __shared__ float join[8][33];
  const int lane = threadIdx.x % 32, w = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
  float t = 0.f;
  if (c < N) {
    float u[4] = {0.f, 0.f, 0.f, 0.f};
    for (int i = w; i < n; i += 32)
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + 8 * k < n) u[k] += part[(size_t)(i + 8 * k) * N + c];
    t = (u[0] + u[1]) + (u[2] + u[3]);
  }
  join[w][lane] = t;
  __syncthreads();
  if (w == 0 && c < N) {
    t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += join[i][lane];
    dbias[c] = t;
  }
}

// ------------------------------------------------------------------------------------ launch
// A product D [rows, cols] = A B^T with contraction k; A is [rows, k] (or [k, rows] when AMN), B
// [cols, k] (or [k, cols] when BMN). Row-major output, row length e.ld.
struct Product {
  const void *A, *B;
  int rows, cols, k;
  Epi e;
  unsigned* err;
};
int ceil_div(long long a, int b) { return (int)((a + b - 1) / b); }

bool operand_map(CUtensorMap* m, const void* p, bool mn, int rows, int k, int box_rows) {
  return mn ? make_tmap_bf16(m, p, rows, k, rows, 64, 64) : make_tmap_bf16(m, p, k, rows, k, 64, box_rows);
}

template <typename K>
cudaError_t with_smem(K kernel, size_t smem) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
}

template <bool AMN, bool BMN>
cudaError_t run_pair(const Product& g, cudaStream_t s) {
  CUtensorMap ta, tb;
  if (!operand_map(&ta, g.A, AMN, g.rows, g.k, 128) || !operand_map(&tb, g.B, BMN, g.cols, g.k, 128))
    return cudaErrorInvalidValue;
  PairArgs p{g.rows, g.cols, ceil_div(g.k, BK), ceil_div(g.rows, PT), ceil_div(g.cols, PT), g.e, g.err};
  const bool aux = g.e.mul || g.e.residual;
  if (aux && (AMN || BMN)) return cudaErrorInvalidValue;  // only the forward has them
  auto kernel = aux && !AMN && !BMN ? linear_pair_kernel<false, false, true>
                                    : linear_pair_kernel<AMN, BMN, false>;
  const cudaError_t e = with_smem(kernel, kPairSmem);
  if (e != cudaSuccess) return e;
  const int pairs = (int)std::min((long long)p.tm * p.tn, (long long)kSMs / 2);
  kernel<<<2 * pairs, kPairThreads, kPairSmem, s>>>(ta, tb, p);
  count_launches(1);
  return cudaGetLastError();
}

// The split kernel takes the columns' operand as its rows.
template <int NT, bool AMN, bool BMN>
cudaError_t run_split_nt(const Product& g, cudaStream_t s) {
  CUtensorMap ta, tb;
  if (!operand_map(&ta, g.B, BMN, g.cols, g.k, 128) || !operand_map(&tb, g.A, AMN, g.rows, g.k, NT))
    return cudaErrorInvalidValue;
  SplitArgs p{g.cols, g.rows, ceil_div(g.k, BK), ceil_div(g.cols, 128), ceil_div(g.rows, NT), 1, g.e, g.err};
  // As many CTAs as are resident at a time, each with four blocks of k at least. Wide tiles stop
  // at about one CTA per SM: their parts cost more than a second CTA brings (200 x 2560 x 2560:
  // split 4 ways 22.5 us, 8 ways 30.8).
  const long long tiles = (long long)p.tf * p.tt, most = NT <= 32 ? 2 * kSMs + 29 : kSMs + 29;
  while (p.split < kMaxSplit && 2 * tiles * p.split <= most && p.nkb / (2 * p.split) >= 4) p.split *= 2;
  if (tiles * p.split >= (1ll << 31)) return cudaErrorInvalidConfiguration;
  constexpr size_t smem = split_smem<NT>();
  cudaError_t e = with_smem(linear_split_kernel<NT, BMN, AMN>, smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(tiles * p.split));
  cfg.blockDim = dim3(kSplitThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = p.split;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = p.split > 1;
  count_launches(1);
  e = cudaLaunchKernelEx(&cfg, linear_split_kernel<NT, BMN, AMN>, ta, tb, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <bool AMN, bool BMN>
cudaError_t run(const Product& g, cudaStream_t s) {
  // Few rows, or few tiles that are deep: the contraction is split (200 x 2560 x 2560: 22.5 us
  // against 26.7; 1537 x 1000 x 520, a shallow one: 22.5 against the pair kernel's 18.4).
  const long long tiles = (long long)ceil_div(g.rows, PT) * ceil_div(g.cols, PT);
  if (g.rows > 64 && (tiles > kSMs / 8 || g.k < 24 * BK)) return run_pair<AMN, BMN>(g, s);
  if constexpr (!AMN) {
    if (g.rows <= 16) return run_split_nt<16, AMN, BMN>(g, s);
    if (g.rows <= 32) return run_split_nt<32, AMN, BMN>(g, s);
  }
  if (g.rows <= 64) return run_split_nt<64, AMN, BMN>(g, s);
  return run_split_nt<128, AMN, BMN>(g, s);
}

struct BwdPlan {
  int bx, by, rows;
  size_t dp_bytes, part_bytes;
};
// The pass over dY: six CTAs per SM (two rounds of those that are resident), each with 32 rows at
// least.
BwdPlan bwd_plan(int M, int N) {
  BwdPlan b;
  b.bx = ceil_div(N, kDpX * 8);
  const long long want = std::max(1, 6 * kSMs / b.bx);
  b.rows = (int)std::min<long long>(M, std::max<long long>(32, (M + want - 1) / want));
  b.by = ceil_div(M, b.rows);
  b.dp_bytes = ((size_t)M * N * sizeof(bf16) + 255) & ~(size_t)255;
  b.part_bytes = (size_t)b.by * N * sizeof(float);
  return b;
}

}  // namespace

size_t linear_fwd_workspace(int, int, int) { return 0; }
size_t linear_bwd_workspace(int M, int N, int) {
  const BwdPlan b = bwd_plan(M, N);
  return b.dp_bytes + b.part_bytes;
}

cudaError_t linear_fwd(const LinearArgs& a, cudaStream_t s) {
  const Epi e{a.bias, static_cast<const bf16*>(a.mul), static_cast<const bf16*>(a.residual),
              static_cast<bf16*>(a.Y), static_cast<bf16*>(a.P), (size_t)a.N, a.silu};
  return run<false, false>({a.X, a.W, a.M, a.N, a.K, e, a.err}, s);
}

cudaError_t linear_bwd(const LinearArgs& a, cudaStream_t s) {
  const BwdPlan b = bwd_plan(a.M, a.N);
  bf16* dP = static_cast<bf16*>(a.ws);
  float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + b.dp_bytes);
  const bool products = a.dX || a.dW;
  // without an activation and a multiplier dP is dY
  const void* dp = a.P_in ? dP : a.dY;
  cudaError_t e = cudaSuccess;
  if (a.dbias || (a.P_in && (products || a.dmul))) {
    const DpArgs d{a.M, a.N, b.rows, a.silu, static_cast<const bf16*>(a.dY),
                   static_cast<const bf16*>(a.P_in), static_cast<const bf16*>(a.mul),
                   products && a.P_in ? dP : nullptr, static_cast<bf16*>(a.dmul), a.dbias ? part : nullptr};
    linear_dp_kernel<<<dim3(b.bx, b.by), kDpX * kDpY, 0, s>>>(d);
    count_launches(1);
    if (a.dbias) {
      linear_dbias_kernel<<<(a.N + 31) / 32, 256, 0, s>>>(part, b.by, a.N, a.dbias);
      count_launches(1);
    }
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && a.dX) {
    const Epi out{nullptr, nullptr, nullptr, static_cast<bf16*>(a.dX), nullptr, (size_t)a.K, 0};
    e = run<false, true>({dp, a.W, a.M, a.K, a.N, out, a.err}, s);
  }
  if (e == cudaSuccess && a.dW) {
    const Epi out{nullptr, nullptr, nullptr, static_cast<bf16*>(a.dW), nullptr, (size_t)a.K, 0};
    e = run<true, true>({dp, a.X, a.N, a.K, a.M, out, a.err}, s);
  }
  return e;
}

}  // namespace tttk
