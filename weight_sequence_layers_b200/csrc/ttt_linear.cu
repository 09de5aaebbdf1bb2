// Linear layer with bias, activation, multiplier and residual in its epilogue, forward and
// backward (include/ttt.h), on the tensor cores.
//
// Every product is D[i, j] = sum_k A[i, k] B[j, k] with bf16 operands, each stored with k
// contiguous (K-major) or with its own index contiguous (MN-major):
//   forward  P  = X W^T   rows tokens,    columns outputs, k inputs:  X, W K-major
//   dX = dP W             rows tokens,    columns inputs,  k outputs: dP K-major, W MN-major
//   dW = dP^T X           rows outputs,   columns inputs,  k tokens:  dP, X MN-major
// TMA fills what lies outside a matrix with zeros, so that every size is a number of full tiles.
// A launch takes one product or two (the backward's): both then share the machine.
//
// Two kernels:
//   pair: 256 x 256 tiles on CTA pairs (cta_group::2), persistent, two accumulators in TMEM so
//         that the epilogue of one tile runs under the products of the next. Bound by the tensor
//         cores: 16384 x 2048 x 2048 backward, both products 187 us = 1.47 PFLOP/s, and by power
//         over longer times (32768 x 9728 x 2560 with SiLU and multiplier 1.14 to 1.18 ms alone, 1.40
//         to 1.45 ms back to back at 1.3 GHz, with P 1.25 and 1.52; the plain product 1.08 and 1.33,
//         the library's 1.03 and 1.24). Operands
//         of the epilogue by plain loads through shared memory were 2 % slower there and 20 % on
//         small products.
//   split: 128 x NT tiles with the roles of rows and columns exchanged (the weights' rows are the
//         MMA's 128 rows, NT = 16, 32 or 64 tokens its columns), one tile a CTA and several CTAs an
//         SM; the CTAs of a cluster share the contraction of one tile and add their parts through
//         distributed shared memory in a fixed order. For few tiles: decode steps, which read the
//         weights once (bound by HBM: 8 x 9728 x 2560 14 us, of which the weights' stream is 9),
//         and small matrices (bound by their latency).
#include <cuda_bf16.h>

#include <algorithm>
#include <type_traits>

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
constexpr int kMaxStages = 6, kRing = 4;
constexpr int kTileReaders = 2 * (1 + kEpiWarps);  // leader: MMA, peer: loads, both: epilogue
constexpr uint32_t kHalf = 128 * BK * 2;      // 16 KB: this CTA's 128 rows of A, or of B
constexpr uint32_t kPairStage = 2 * kHalf;
constexpr uint32_t kPanel = 32 * 128;         // 32 rows of 64 columns of an epilogue warp
struct __align__(8) PairBars {
  uint64_t full[kMaxStages], empty[kMaxStages], acc_full[2], acc_empty[2], tile_full[kRing],
      tile_empty[kRing], panel_full[kEpiWarps][2];
  int ring[kRing];  // tiles handed out, a few ahead
  uint32_t tmem_base;
  int abort_flag;
};
// AUX: the epilogue has a multiplier, a residual or P, and takes two panels a warp.
template <bool AUX>
struct PairLayout {
  static constexpr int kStages = AUX ? 5 : 6, kPanels = AUX ? 2 : 1;
  static constexpr uint32_t kOffPanels = kStages * kPairStage;
  static constexpr uint32_t kOffBars = kOffPanels + kEpiWarps * kPanels * kPanel;
  static constexpr size_t kSmem = kOffBars + sizeof(PairBars) + 1024;
  static_assert(kSmem <= 232448, "shared memory of one CTA");
};

struct PairProb {
  int rows, cols, nkb;  // of D; 64-wide blocks of k
  int tm, tn;           // tiles
  int a_mn, b_mn;
  Epi e;
};
// The sums of `part` [n, N] over its rows, which a launch takes along (part: nullable).
struct Sums {
  const float* part;
  int n, N;
  float* out;
};
struct PairArgs {
  PairProb p[2];
  int tiles0, tiles;  // of the first product, of both
  int* counter;       // hands out the tiles; NULL: pair c takes tiles c, c + pairs and so on
  Sums sums;
  unsigned* err;
};
// Tile t: groups of kGroup tile rows, column by column, so that the tiles at work at one time
// share their rows of A and of B in L2.
constexpr int kGroup = 8;
__device__ __forceinline__ const PairProb& pair_tile(const PairArgs& a, int t, int& m0, int& n0) {
  const PairProb& p = a.p[t >= a.tiles0];
  if (t >= a.tiles0) t -= a.tiles0;
  const int g = t / (kGroup * p.tn), rem = t - g * kGroup * p.tn;
  const int gm = min(kGroup, p.tm - g * kGroup), n = rem / gm;
  m0 = (g * kGroup + rem - n * gm) * PT;
  n0 = n * PT;
  return p;
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
// 128 rows of an operand in a stage, at 16-wide step kk of its block of k.
template <bool MN>
__device__ __forceinline__ uint64_t operand(uint32_t addr, int kk) {
  return MN ? sdesc_sw128(addr + kk * 2048, kHalf / 2, 1024) : sdesc_sw128(addr + kk * 32, 16, 1024);
}
template <bool MN>
using Major = std::bool_constant<MN>;
// f with the operands' layouts as constants: the loops over k that issue loads and products are
// one thread's, and slow down with descriptors made from run-time layouts (16384 x 2048 x 2048:
// 96 -> 112 us).
template <typename F>
__device__ __forceinline__ bool with_layouts(bool a_mn, bool b_mn, F f) {
  if (!b_mn) return f(Major<false>{}, Major<false>{});  // the forward
  if (!a_mn) return f(Major<false>{}, Major<true>{});   // dX
  return f(Major<true>{}, Major<true>{});               // dW
}
// Column sums by W warps (threads 0.. of `tid`), 32 columns at a time. A column's rows fall to
// eight parts whatever W is, so that the order of the sum is the same in every kernel. The walk
// counts blocks of columns: a column's index plus a step of all CTAs can pass 2^31.
constexpr int kSumParts = 8;
template <int W>
__device__ __forceinline__ void column_sums(const Sums& s, int tid, int block, int blocks, float* join) {
  const int lane = tid % 32, w = tid / 32;
  const int last = (s.N - 1) / 32;
  for (int i = block; i <= last; i += blocks) {
    const int c = 32 * i + lane;
#pragma unroll
    for (int v = w; v < kSumParts; v += W) {
      float t[4] = {0.f, 0.f, 0.f, 0.f};
      if (c < s.N)
        for (int i = v; i < s.n; i += 4 * kSumParts)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (i + k * kSumParts < s.n) t[k] += s.part[(size_t)(i + k * kSumParts) * s.N + c];
      join[v * 32 + lane] = (t[0] + t[1]) + (t[2] + t[3]);
    }
    asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory");
    if (w == 0 && c < s.N) {
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < kSumParts; ++i) sum += join[i * 32 + lane];
      s.out[c] = sum;
    }
    asm volatile("bar.sync 1, %0;" ::"n"(32 * W) : "memory");
  }
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
__device__ __forceinline__ void finish8(const Epi& e, size_t o, const float (&b)[8], const uint4& mu,
                                        const uint4& re, float (&y)[8], float (&w)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) y[k] += b[k];
  if (e.P) *reinterpret_cast<uint4*>(e.P + o) = pack8(y);
  if (e.silu)
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] *= sigm(y[k]);
  if (e.mul) {
    unpack8(mu, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] *= w[k];
  }
  if (e.residual) {
    unpack8(re, w);
#pragma unroll
    for (int k = 0; k < 8; ++k) y[k] += w[k];
  }
  *reinterpret_cast<uint4*>(e.Y + o) = pack8(y);
}

// Warps: 0 TMA loads, 1 MMA (the leader's), 2-9 epilogue (two per TMEM lane quadrant, 128
// columns each). The leader's barriers count both CTAs' loads and drained accumulators; commits
// arrive on both CTAs' stage and accumulator barriers. The leader's loading thread takes the
// tiles and hands each to the roles of both CTAs.
template <bool AUX>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap ta0, const __grid_constant__ CUtensorMap tb0,
                       const __grid_constant__ CUtensorMap ta1, const __grid_constant__ CUtensorMap tb1,
                       const __grid_constant__ CUtensorMap ty0, const __grid_constant__ CUtensorMap ty1,
                       const __grid_constant__ PairArgs p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  using L = PairLayout<AUX>;
  constexpr int kPairStages = L::kStages;
  PairBars* bars = reinterpret_cast<PairBars*>(smem + L::kOffBars);
  const uint32_t stage0 = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int half = (int)rank * 128;
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
    for (int w = 0; w < 2 * kEpiWarps; ++w) mbar_init(PB(panel_full[w / 2][w % 2]), 1);
    for (int r = 0; r < kRing; ++r) {
      mbar_init(PB(tile_full[r]), 1);
      mbar_init(PB(tile_empty[r]), kTileReaders);
    }
    bars->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&ta0);
    tma_prefetch_desc(&tb0);
    if (p.tiles > p.tiles0) {
      tma_prefetch_desc(&ta1);
      tma_prefetch_desc(&tb1);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(PB(tmem_base), 2 * PT);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // what the launch before this one wrote
  // A reader's next tile; p.tiles or more: none left, or a wait that ran out. Without a counter
  // all roles know the order, and the ring is not used.
  int ring = 0, mine = blockIdx.x / 2;
  uint32_t ring_ph = 0;
  auto next_tile = [&](bool one_thread) {
    if (!p.counter) {
      const int t = mine;
      mine += gridDim.x / 2;
      return t;
    }
    if (!mbar_wait_cluster(PB(tile_full[ring]), ring_ph, ab)) return 0x7FFFFFFF;
    const int t = bars->ring[ring];
    if (!one_thread) __syncwarp();
    if (one_thread || lane == 0) {
      if (leader) mbar_arrive(PB(tile_empty[ring]));
      else mbar_arrive_cluster(peer_addr(PB(tile_empty[ring]), 0));
    }
    if (++ring == kRing) { ring = 0; ring_ph ^= 1; }
    return t;
  };

  if (warp == 0) {
    if (lane == 0) {
      int s = 0;
      uint32_t ph = 0;
      bool ok = true;
      while (ok) {
        int t;
        if (leader && p.counter) {
          if (!mbar_wait_cluster(PB(tile_empty[ring]), ring_ph ^ 1, ab)) break;
          t = atomicAdd(p.counter, 1);
          bars->ring[ring] = t;
          st_cluster_u32(peer_addr(PB(ring[ring]), 1), t);
          mbar_arrive(PB(tile_full[ring]));
          mbar_arrive_cluster(peer_addr(PB(tile_full[ring]), 1));
          if (++ring == kRing) { ring = 0; ring_ph ^= 1; }
        } else {
          t = next_tile(true);
        }
        if (t >= p.tiles) break;
        int m0, n0;
        const PairProb& g = pair_tile(p, t, m0, n0);
        const int nkb = g.nkb;
        const CUtensorMap *ta = t < p.tiles0 ? &ta0 : &ta1, *tb = t < p.tiles0 ? &tb0 : &tb1;
        ok = with_layouts(g.a_mn, g.b_mn, [&](auto am, auto bm) {
          for (int kb = 0; kb < nkb; ++kb) {
            if (!mbar_wait(PB(empty[s]), ph ^ 1, ab)) return false;
            if (leader) mbar_arrive_expect_tx(PB(full[s]), 2 * kPairStage);
            const uint32_t bar = peer_addr(PB(full[s]), 0), sa = stage0 + s * kPairStage;
            pair_load<am.value>(sa, ta, bar, m0 + half, kb);
            pair_load<bm.value>(sa + kHalf, tb, bar, n0 + half, kb);
            if (++s == kPairStages) { s = 0; ph ^= 1; }
          }
          return true;
        });
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      int s = 0, acc = 0;
      uint32_t ph = 0, aph = 0;
      bool ok = true;
      for (int t; ok && (t = next_tile(true)) < p.tiles;) {
        const PairProb& g = p.p[t >= p.tiles0];
        const int nkb = g.nkb;
        if (!(ok = mbar_wait_cluster(PB(acc_empty[acc]), aph ^ 1, ab))) break;
        tc_fence_after();
        ok = with_layouts(g.a_mn, g.b_mn, [&](auto am, auto bm) {
          constexpr uint32_t id = idesc_bf16(PT, PT, am.value, bm.value);
          for (int kb = 0; kb < nkb; ++kb) {
            if (!mbar_wait(PB(full[s]), ph, ab)) return false;
            tc_fence_after();
            const uint32_t sa = stage0 + s * kPairStage;
#pragma unroll
            for (int kk = 0; kk < BK / 16; ++kk)
              mma_bf16_pair(tmem + acc * PT, operand<am.value>(sa, kk), operand<bm.value>(sa + kHalf, kk),
                            id, (kb | kk) != 0);
            mma_commit_pair(PB(empty[s]));
            if (++s == kPairStages) { s = 0; ph ^= 1; }
          }
          return true;
        });
        if (ok) mma_commit_pair(PB(acc_full[acc]));
        if (++acc == 2) { acc = 0; aph ^= 1; }
      }
    }
  } else {
    // A thread takes a row of the accumulator. Outputs leave by TMA: 32 rows of 64 columns go to a
    // swizzled panel of the warp and from there in one bulk store (clipped at the edges). A
    // multiplier or a residual comes into the panel the same way, ahead of the accumulator; a warp
    // has one panel for each of its two blocks of a tile, or, with both operands, one for each of
    // them (the maps of the second product, which a launch with operands does not have).
    const int q = warp & 3, h = (warp - 2) / 4, ew = warp - 2;
    const uint32_t panels = stage0 + L::kOffPanels + ew * L::kPanels * kPanel;
    uint32_t panel_ph = 0;  // bit b: the parity of panel_full[ew][b]
    int acc = 0;
    uint32_t aph = 0;
    if (p.sums.part) {  // before the first tile's sums are there
      column_sums<kEpiWarps>(p.sums, threadIdx.x - 64, blockIdx.x, gridDim.x,
                             reinterpret_cast<float*>(smem + L::kOffPanels));
    }
    for (int t; (t = next_tile(false)) < p.tiles;) {
      int m0, n0;
      const PairProb& g = pair_tile(p, t, m0, n0);
      const Epi e = g.e;
      const int rows = g.rows, cols = g.cols;
      m0 += half + q * 32;
      const bool both = AUX && e.mul && e.residual, any = AUX && (e.mul || e.residual);
      // block b of the warp's two: its columns, whether the matrix has any of it, and its panel
      auto col0 = [&](int b) { return n0 + 64 * (2 * h + b); };
      auto inside = [&](int b) { return m0 < rows && col0(b) < cols; };
      auto panel_of = [&](int b) { return panels + (L::kPanels == 2 && !both ? b : 0) * kPanel; };
      auto fetch = [&](int b) {  // one thread
        if (!inside(b)) return;
        const uint32_t bar = PB(panel_full[ew][both ? 0 : b]);
        mbar_arrive_expect_tx(bar, (both ? 2 : 1) * kPanel);
        tma_load_2d(panel_of(b), e.mul ? &ta1 : &tb1, bar, col0(b), m0);
        if (both) tma_load_2d(panel_of(b) + kPanel, &tb1, bar, col0(b), m0);
      };
      if (AUX && lane == 0) {
        bulk_wait_read0();  // the last tile's stores have left the panels
        if (any) fetch(0);
        if (any && !both) fetch(1);
      }
      if (!mbar_wait(PB(acc_full[acc]), aph, ab)) break;
      __syncwarp();
      tc_fence_after();
#pragma unroll 1
      for (int b = 0; b < 2; ++b) {
        const int c0 = col0(b);
        const uint32_t panel = panel_of(b);
        if (lane == 0 && (!AUX || (both && b == 1))) {
          bulk_wait_read0();  // the store before this one has left the panel
          if (both) fetch(1);
        }
        __syncwarp();
        if (any && inside(b)) {
          const int bar = both ? 0 : b;
          mbar_wait(PB(panel_full[ew][bar]), panel_ph >> bar & 1, ab);
          panel_ph ^= 1u << bar;
          __syncwarp();
        }
#pragma unroll
        for (int part = 0; part < 2; ++part) {
          float v[32];
          tmem_ld32(tmem_addr(tmem, q * 32, acc * PT + (2 * h + b) * 64 + part * 32), v);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int col = c0 + part * 32 + 8 * k;
            const uint32_t at = panel + sw128_off(lane, part * 4 + k);
            float y[8], w[8];
#pragma unroll
            for (int x = 0; x < 8; ++x) y[x] = v[8 * k + x];
            if (e.bias && col < cols) {  // columns come in eights
              const float4 lo = *reinterpret_cast<const float4*>(e.bias + col);
              const float4 hi = *reinterpret_cast<const float4*>(e.bias + col + 4);
              y[0] += lo.x; y[1] += lo.y; y[2] += lo.z; y[3] += lo.w;
              y[4] += hi.x; y[5] += hi.y; y[6] += hi.z; y[7] += hi.w;
            }
            if (AUX && e.P && col < cols && m0 + lane < rows)
              *reinterpret_cast<uint4*>(e.P + (size_t)(m0 + lane) * e.ld + col) = pack8(y);
            if (e.silu)
#pragma unroll
              for (int x = 0; x < 8; ++x) y[x] *= sigm(y[x]);
            if (AUX && e.mul) {
              uint4 o;
              ld_shared_v4(at, o.x, o.y, o.z, o.w);
              unpack8(o, w);
#pragma unroll
              for (int x = 0; x < 8; ++x) y[x] *= w[x];
            }
            if (AUX && e.residual) {
              uint4 o;
              ld_shared_v4(at + (both ? kPanel : 0), o.x, o.y, o.z, o.w);
              unpack8(o, w);
#pragma unroll
              for (int x = 0; x < 8; ++x) y[x] += w[x];
            }
            const uint4 o = pack8(y);
            st_shared_v4(at, o.x, o.y, o.z, o.w);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && inside(b)) {
          tma_store_2d(t < p.tiles0 ? &ty0 : &ty1, panel, c0, m0);
          bulk_commit();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (leader) mbar_arrive(PB(acc_empty[acc]));
        else mbar_arrive_cluster(peer_addr(PB(acc_empty[acc]), 0));
      }
      if (++acc == 2) { acc = 0; aph ^= 1; }
    }
    if (lane == 0) bulk_wait0();
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
// 32 lanes x 16 columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,"
      "%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]),
        "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
// D^T tiles: 128 rows are "features" f (rows of operand A), NT columns "tokens" t (of B); the
// output at [t, f] is row-major with f contiguous, so that a warp's 32 rows are one 64-byte piece
// of a token's row. Warps: 0 TMA, 1 MMA, 2-5 epilogue.
constexpr int kSplitThreads = 192;
constexpr int kMaxSplit = 8;
struct SplitProb {
  int feats, toks, nkb;
  int tf;  // tiles of features
  int a_mn, b_mn;
  Epi e;
};
struct SplitArgs {
  SplitProb p[2];
  int tiles0, split;  // tiles of the first product, CTAs of a cluster
  Sums sums;
  unsigned* err;
};
template <int NT>
struct SplitLayout {
  static constexpr uint32_t kA = 128 * BK * 2, kB = NT * BK * 2, kStage = kA + kB;
  static constexpr int kStages = NT == 16 ? 3 : 4;  // two CTAs an SM, three with NT = 16
  // The parts of a tile that come from the cluster's CTAs: in their own place where that is
  // small, else over the stages, once all CTAs have read these.
  static constexpr bool kOwnParts = NT <= 32;
  static constexpr uint32_t kParts = NT * 128 * 4, kOffParts = kOwnParts ? kStages * kStage : 0;
  static constexpr uint32_t kOffBars = kStages * kStage + (kOwnParts ? kParts : 0);
  static_assert(kOwnParts || kStages * kStage >= kParts, "room for the parts");
};
struct __align__(8) SplitBars {
  uint64_t full[4], empty[4], acc, parts;
  uint32_t tmem_base;
  int abort_flag;
  float join[kSumParts * 32];
};
template <int NT>
constexpr size_t split_smem() { return SplitLayout<NT>::kOffBars + sizeof(SplitBars) + 1024; }

template <int NT>
__global__ void __launch_bounds__(kSplitThreads)
    linear_split_kernel(const __grid_constant__ CUtensorMap ta0, const __grid_constant__ CUtensorMap tb0,
                        const __grid_constant__ CUtensorMap ta1, const __grid_constant__ CUtensorMap tb1,
                        const __grid_constant__ SplitArgs a) {
  using L = SplitLayout<NT>;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  SplitBars* bars = reinterpret_cast<SplitBars*>(smem + L::kOffBars);
  const uint32_t stage0 = smem_u32(smem);
  const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
  const int S = a.split, rank = S > 1 ? (int)cluster_rank() : 0;
  int tile = blockIdx.x / S;
  const bool second = tile >= a.tiles0;
  if (second) tile -= a.tiles0;
  const SplitProb p = a.p[second];
  const CUtensorMap *ta = second ? &ta1 : &ta0, *tb = second ? &tb1 : &tb0;
  const int f0 = (tile % p.tf) * 128, t0 = (tile / p.tf) * NT;
  const int k_lo = (int)((long long)p.nkb * rank / S), k_hi = (int)((long long)p.nkb * (rank + 1) / S);
  const Abort ab{&bars->abort_flag, a.err};
  constexpr uint32_t kCols = NT < 32 ? 32 : NT;
#define SB(x) smem_u32(&bars->x)
  auto load = [&](int kb) {
    const int st = (kb - k_lo) % L::kStages;
    const uint32_t bar = SB(full[st]), sa = stage0 + st * L::kStage, sb = sa + L::kA;
    mbar_arrive_expect_tx(bar, L::kStage);
    if (p.a_mn) {
      tma_load_2d(sa, ta, bar, f0, kb * BK);
      tma_load_2d(sa + 8192, ta, bar, f0 + 64, kb * BK);
    } else {
      tma_load_2d(sa, ta, bar, kb * BK, f0);
    }
    if (NT >= 64 && p.b_mn) {  // panels of 64
#pragma unroll
      for (int j = 0; j < NT / 64; ++j) tma_load_2d(sb + 8192 * j, tb, bar, t0 + 64 * j, kb * BK);
    } else {
      tma_load_2d(sb, tb, bar, kb * BK, t0);
    }
  };
  if (threadIdx.x == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(SB(full[s]), 1);
      mbar_init(SB(empty[s]), 1);
    }
    mbar_init(SB(acc), 1);
    mbar_init(SB(parts), 1);
    bars->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(ta);
    tma_prefetch_desc(tb);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what the launch before this one wrote
    // the first loads run while the other warps get ready
    for (int kb = k_lo; kb < min(k_hi, k_lo + L::kStages); ++kb) load(kb);
  }
  if (warp == 1) {
    tmem_alloc(SB(tmem_base), kCols);
    tmem_relinquish();
  }
  // (a CTA's shared memory may be written by the others once all have started)
  __syncwarp();
  if (S > 1 && L::kOwnParts) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
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
      with_layouts(p.b_mn, p.a_mn, [&](auto bm, auto am) {  // (its operands are exchanged)
        constexpr uint32_t id = idesc_bf16(128, NT, am.value, bm.value);
        for (int kb = k_lo; kb < k_hi; ++kb) {
          const int i = kb - k_lo, s = i % L::kStages;
          if (!mbar_wait(SB(full[s]), (i / L::kStages) & 1, ab)) return false;
          tc_fence_after();
          const uint32_t sa = stage0 + s * L::kStage, sb = sa + L::kA;
#pragma unroll
          for (int kk = 0; kk < BK / 16; ++kk)
            mma_bf16_ss(tmem, operand<am.value>(sa, kk), operand<bm.value>(sb, kk), id, i > 0 || kk > 0);
          mma_commit(SB(empty[s]));
        }
        return true;
      });
      mma_commit(SB(acc));
    }
  }
  __syncwarp();
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (a.sums.part && warp >= 2)
    column_sums<4>(a.sums, threadIdx.x - 64, blockIdx.x, gridDim.x, bars->join);
  __syncwarp();
  // The outputs of this CTA: of the tile's tokens t those with t % S = rank, 8 features (16 bytes)
  // at a time, a token's 16 pieces side by side. Operands are loaded a batch of items ahead.
  const Epi& e = p.e;
  const int split_log = __ffs(S) - 1, items = (NT >> split_log) * 16;  // S is a power of two
  constexpr int kBatch = 4;
  struct Operands {
    uint4 mu[kBatch], re[kBatch];
  } now, next;
  const int f = f0 + 8 * (threadIdx.x % 16);  // the same piece for all of a thread's items
  auto token_of = [&](int it) { return t0 + ((it / 16) << split_log) + rank; };
  auto fetch = [&](int it0, Operands& o) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int it = it0 + u * kSplitThreads, t = token_of(it);
      if (it < items && t < p.toks && f < p.feats) {
        const size_t at = (size_t)t * e.ld + f;
        if (e.mul) o.mu[u] = *reinterpret_cast<const uint4*>(e.mul + at);
        if (e.residual) o.re[u] = *reinterpret_cast<const uint4*>(e.residual + at);
      }
    }
  };
  fetch(threadIdx.x, now);
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
  // part of CTA c, token number j of a CTA's, feature i: parts[(c NT / S + j) 128 + i]
  const int q = warp & 3;
  const uint32_t part0 = stage0 + L::kOffParts + (uint32_t)((rank * NT >> split_log) * 128 + q * 32 + lane) * 4;
  if (S == 1) {
    if (warp >= 2)
#pragma unroll 1
      for (int c = 0; c < NT / 16 && t0 + c * 16 < p.toks; ++c) {
        float v[16];
        __syncwarp();
        tmem_ld16(tmem_addr(tmem, q * 32, c * 16), v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j)
          asm volatile("st.shared.f32 [%0], %1;" ::"r"(part0 + (c * 16 + j) * 512), "f"(v[j]) : "memory");
      }
    __syncthreads();
  } else {
    // With a place of their own the parts are counted where they arrive; over the stages a
    // barrier of the cluster follows them.
    const uint32_t bar = SB(parts);
    const int valid = min(NT, p.toks - t0);
    const int mine = valid > rank ? ((valid - rank - 1) >> split_log) + 1 : 0;  // tokens
    if (L::kOwnParts && threadIdx.x == 0) mbar_arrive_expect_tx(bar, mine * S * 512);
    if (warp >= 2) {
      uint32_t to[8], bars_at[8];  // CTA j % S
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        to[k] = peer_addr(part0, k & (S - 1));
        bars_at[k] = peer_addr(bar, k & (S - 1));
      }
#pragma unroll 1
      for (int c = 0; c < NT / 16 && c * 16 < valid; ++c) {
        float v[16];
        __syncwarp();
        tmem_ld16(tmem_addr(tmem, q * 32, c * 16), v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int t = c * 16 + j;
          const uint32_t at = to[j & 7] + (t >> split_log) * 512;
          if (t < valid) {
            if (L::kOwnParts)
              asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.f32 [%0], %1, [%2];"
                           ::"r"(at), "f"(v[j]), "r"(bars_at[j & 7]) : "memory");
            else
              asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(at), "f"(v[j]) : "memory");
          }
        }
      }
    }
    __syncwarp();
    if (L::kOwnParts) {
      if (!mbar_try_wait_cluster(bar, 0)) mbar_wait_cluster(bar, 0, ab);
      __syncwarp();
    } else {
      cluster_sync_all();
    }
  }
  const float* parts = reinterpret_cast<const float*>(smem + L::kOffParts) + 8 * (threadIdx.x % 16);
#pragma unroll 1
  for (int it0 = threadIdx.x; it0 < items; it0 += kBatch * kSplitThreads) {
    fetch(it0 + kBatch * kSplitThreads, next);
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int it = it0 + u * kSplitThreads, t = token_of(it);
      if (it >= items || t >= p.toks || f >= p.feats) continue;
      float y[8], w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = 0.f;
      for (int c = 0; c < S; ++c) {
        const float4* x = reinterpret_cast<const float4*>(parts + ((c * NT >> split_log) + it / 16) * 128);
        const float4 lo = x[0], hi = x[1];
        y[0] += lo.x; y[1] += lo.y; y[2] += lo.z; y[3] += lo.w;
        y[4] += hi.x; y[5] += hi.y; y[6] += hi.z; y[7] += hi.w;
      }
      finish8(e, (size_t)t * e.ld + f, b, now.mu[u], now.re[u], y, w);
    }
    now = next;
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
// of dP for dbias. A thread takes 8 columns of every kDpY-th row of its CTA's rows; the CTAs'
// sums go to `part` [gridDim.y, N] and are added in a fixed order.
constexpr int kDpX = 32, kDpY = 8;
struct DpArgs {
  int M, N, rows;  // rows of a CTA
  int silu;
  const bf16 *dY, *P, *mul;
  bf16 *dP, *dmul;  // nullable
  float* part;      // nullable
  int* counter;     // the products' tiles, from 0
};
__global__ void __launch_bounds__(kDpX* kDpY) linear_dp_kernel(const DpArgs a) {
  __shared__ float join[kDpY][kDpX * 8 + 8];
  asm volatile("griddepcontrol.launch_dependents;");
  if (blockIdx.x == 0 && blockIdx.y == 0 && threadIdx.x == 0) *a.counter = 0;
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
__global__ void __launch_bounds__(256) linear_sums_kernel(const __grid_constant__ Sums s) {
  __shared__ float join[kSumParts * 32];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  column_sums<8>(s, threadIdx.x, blockIdx.x, gridDim.x, join);
}

// ------------------------------------------------------------------------------------ launch
// A product D [rows, cols] = A B^T with contraction k; A is [rows, k] (or [k, rows] when a_mn), B
// [cols, k] (or [k, cols] when b_mn). Row-major output, row length e.ld.
struct Product {
  const void *A, *B;
  int rows, cols, k;
  bool a_mn, b_mn;
  Epi e;
};
int ceil_div(long long a, int b) { return (int)((a + b - 1) / b); }

bool operand_map(CUtensorMap* m, const void* p, bool mn, int rows, int k, int box_rows) {
  return mn ? make_tmap_bf16(m, p, rows, k, rows, 64, 64) : make_tmap_bf16(m, p, k, rows, k, 64, box_rows);
}

// after: the launch may start before the one in front of it has ended, and waits on the device.
template <typename... P, typename... A>
cudaError_t launch(void (*kernel)(P...), unsigned grid, int threads, size_t smem, int cluster,
                   bool after, cudaStream_t s, A... args) {
  cudaError_t e = smem > (48 << 10) ? cudaFuncSetAttribute(
      kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) : cudaSuccess;
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[2]{};
  if (cluster > 1) {
    at[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    at[cfg.numAttrs].val.clusterDim.x = cluster;
    at[cfg.numAttrs].val.clusterDim.y = at[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
  }
  if (after) {
    at[cfg.numAttrs].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[cfg.numAttrs].val.programmaticStreamSerializationAllowed = 1;
    ++cfg.numAttrs;
  }
  cfg.attrs = at;
  count_launches(1);
  e = cudaLaunchKernelEx(&cfg, kernel, args...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

// One or two products (n); the first should be the one with the longer contraction.
cudaError_t run_pair(const Product* g, int n, int* counter, const Sums& sums, bool after,
                     unsigned* err, cudaStream_t s) {
  CUtensorMap t[6];
  PairArgs p{};
  const bool aux = g[0].e.mul || g[0].e.residual || g[0].e.P;
  for (int i = 0; i < n; ++i) {
    const Product& q = g[i];
    if (!operand_map(&t[2 * i], q.A, q.a_mn, q.rows, q.k, 128) ||
        !operand_map(&t[2 * i + 1], q.B, q.b_mn, q.cols, q.k, 128) ||
        !make_tmap_bf16(&t[4 + i], q.e.Y, q.cols, q.rows, q.e.ld, 64, 32))
      return cudaErrorInvalidValue;
    p.p[i] = {q.rows, q.cols, ceil_div(q.k, BK), ceil_div(q.rows, PT), ceil_div(q.cols, PT), q.a_mn, q.b_mn, q.e};
    p.tiles += p.p[i].tm * p.p[i].tn;
    if (i == 0) p.tiles0 = p.tiles;
  }
  // what the launch does not use repeats the first operand's map
  if (n == 1) t[2] = t[3] = t[5] = t[0];
  if (aux) {
    if (n > 1) return cudaErrorInvalidValue;  // (the operands take the second product's maps)
    const Epi& e = g[0].e;
    if ((e.mul && !make_tmap_bf16(&t[2], e.mul, g[0].cols, g[0].rows, e.ld, 64, 32)) ||
        (e.residual && !make_tmap_bf16(&t[3], e.residual, g[0].cols, g[0].rows, e.ld, 64, 32)))
      return cudaErrorInvalidValue;
  }
  p.counter = n > 1 ? counter : nullptr;  // tiles of one product are alike
  p.sums = sums;
  p.err = err;
  return launch(aux ? linear_pair_kernel<true> : linear_pair_kernel<false>,
                2 * std::min(p.tiles, kSMs / 2), kPairThreads,
                aux ? PairLayout<true>::kSmem : PairLayout<false>::kSmem, 1, after, s, t[0], t[1],
                t[2], t[3], t[4], t[5], p);
}

// The kernel of a product and the CTAs that share a tile's contraction (0: the pair kernel). The
// choice hangs on the product alone, so that its sums come out the same in any call.
// Split tiles as long as all of them are resident at a time, two an SM (543 x 3936 x 1696, 279
// tiles: 23.4 us against the pair kernel's 25.5; 512 x 1024 x 1024: 14.3 against 20.5; beyond,
// 200 rows' dW of 2560 x 2560: 27.6 against 21.3). With 32 rows or fewer always: the product is a
// read of the weights. The backward's products stay with the pair kernel, which takes two in one
// launch, unless they are deep (1024 x 2048 x 2048, both: 33.8 us against 44; 1024 x 1024 x 1024,
// 17.4 against 25.0; 117 x 6440 x 24 with its 101 blocks of k: 29.7 against 47.8). The price is a call
// for one product of few tiles and a middling depth: dX of 64 x 2048 x 2048 takes 19.5 us, split 15.0.
int tokens_of(const Product& g) {  // columns of a split tile
  return !g.a_mn && g.rows <= 16 ? 16 : !g.a_mn && g.rows <= 32 ? 32 : 64;
}
int split_of(const Product& g) {
  const int nt = tokens_of(g), nkb = ceil_div(g.k, BK);
  const long long tiles = (long long)ceil_div(g.rows, nt) * ceil_div(g.cols, 128);
  if (nt > 32 && tiles > 2 * kSMs) return 0;
  if (g.b_mn && nkb < 50) return 0;
  // The contraction is shared as long as all CTAs stay resident (a cluster lies within one GPC, so
  // that fewer fit with the larger ones: kResident at two an SM, by the occupancy query; three with
  // 16 tokens), each with four blocks of k at least. us on both sides of the limit, K = 2560, for a
  // split of 2 / 4: 16 tokens, limit 426 CTAs: 23.3 / 22.6 at 100 tiles, 24.7 / 28.0 at 111; 32 tokens,
  // limit 284: 20.5 / 18.7 at 70, 20.5 / 24.6 at 74; 64 tokens: 22.6 / 22.3 at 70, 23.1 / 28.8 at 74.
  constexpr int kResident[kMaxSplit + 1] = {0, 2 * kSMs, 2 * kSMs, 0, 284, 0, 0, 0, 264};
  auto resident = [&](int split) { return kResident[split] * (nt == 16 ? 3 : 2) / 2; };
  int split = 1;
  while (split < kMaxSplit && 2 * tiles * split <= resident(2 * split) && nkb / (2 * split) >= 4) split *= 2;
  return split;
}

// The split kernel takes the columns' operand as its rows.
template <int NT>
cudaError_t run_split_nt(const Product* g, int n, int split, const Sums& sums, bool after,
                         unsigned* err, cudaStream_t s) {
  CUtensorMap t[4];
  SplitArgs p{};
  long long tiles = 0;
  for (int i = 0; i < n; ++i) {
    const Product& q = g[i];
    if (!operand_map(&t[2 * i], q.B, q.b_mn, q.cols, q.k, 128) ||
        !operand_map(&t[2 * i + 1], q.A, q.a_mn, q.rows, q.k, NT))
      return cudaErrorInvalidValue;
    p.p[i] = {q.cols, q.rows, ceil_div(q.k, BK), ceil_div(q.cols, 128), q.b_mn, q.a_mn, q.e};
    tiles += (long long)p.p[i].tf * ceil_div(q.rows, NT);
    if (tiles * split >= (1ll << 31)) return cudaErrorInvalidConfiguration;
    if (i == 0) p.tiles0 = (int)tiles;
  }
  if (n == 1) t[2] = t[3] = t[0];  // not used
  p.split = split;
  p.sums = sums;
  p.err = err;
  return launch(linear_split_kernel<NT>, (unsigned)(tiles * split), kSplitThreads, split_smem<NT>(),
                split, after, s, t[0], t[1], t[2], t[3], p);
}
cudaError_t run_split(const Product* g, int n, int split, const Sums& sums, bool after, unsigned* err,
                      cudaStream_t s) {
  const int nt = n > 1 ? std::max(tokens_of(g[0]), tokens_of(g[1])) : tokens_of(g[0]);
  if (nt == 16) return run_split_nt<16>(g, n, split, sums, after, err, s);
  if (nt == 32) return run_split_nt<32>(g, n, split, sums, after, err, s);
  return run_split_nt<64>(g, n, split, sums, after, err, s);
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
  b.part_bytes = ((size_t)b.by * N * sizeof(float) + 255) & ~(size_t)255;
  return b;
}

}  // namespace

size_t linear_fwd_workspace(int, int, int) { return 0; }
size_t linear_bwd_workspace(int M, int N, int) {
  const BwdPlan b = bwd_plan(M, N);
  return b.dp_bytes + b.part_bytes + 256;  // and the tile counter
}

cudaError_t linear_fwd(const LinearArgs& a, cudaStream_t s) {
  const Epi e{a.bias, static_cast<const bf16*>(a.mul), static_cast<const bf16*>(a.residual),
              static_cast<bf16*>(a.Y), static_cast<bf16*>(a.P), (size_t)a.N, a.silu};
  const Product g{a.X, a.W, a.M, a.N, a.K, false, false, e};
  const int split = split_of(g);
  return split ? run_split(&g, 1, split, {}, false, a.err, s)
               : run_pair(&g, 1, nullptr, {}, false, a.err, s);
}

cudaError_t linear_bwd(const LinearArgs& a, cudaStream_t s) {
  const BwdPlan b = bwd_plan(a.M, a.N);
  bf16* dP = static_cast<bf16*>(a.ws);
  float* part = reinterpret_cast<float*>(static_cast<char*>(a.ws) + b.dp_bytes);
  int* counter = reinterpret_cast<int*>(static_cast<char*>(a.ws) + b.dp_bytes + b.part_bytes);
  // without an activation and a multiplier dP is dY
  const void* dp = a.P_in ? dP : a.dY;
  Product g[2];  // the longer contraction first
  int n = 0;
  auto product = [&](void* out, const void* A, const void* B, int rows, int k, bool a_mn) {
    if (out) g[n++] = {A, B, rows, a.K, k, a_mn, true,
                       {nullptr, nullptr, nullptr, static_cast<bf16*>(out), nullptr, (size_t)a.K, 0}};
  };
  if (a.M < a.N) product(a.dX, dp, a.W, a.M, a.N, false);
  product(a.dW, dp, a.X, a.N, a.M, true);
  if (a.M >= a.N) product(a.dX, dp, a.W, a.M, a.N, false);
  bool after = false;  // a launch of this call is in front of the next one
  Sums sums{};
  if (a.dbias || (a.P_in && (n || a.dmul))) {
    const DpArgs d{a.M, a.N, b.rows, a.silu, static_cast<const bf16*>(a.dY),
                   static_cast<const bf16*>(a.P_in), static_cast<const bf16*>(a.mul),
                   n && a.P_in ? dP : nullptr, static_cast<bf16*>(a.dmul), a.dbias ? part : nullptr, counter};
    linear_dp_kernel<<<dim3(b.bx, b.by), kDpX * kDpY, 0, s>>>(d);
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    if (a.dbias) sums = {part, b.by, a.N, a.dbias};
    after = true;
  }
  int* tiles = after ? counter : nullptr;
  if (n == 0)
    return sums.part ? launch(linear_sums_kernel, std::min(ceil_div(a.N, 32), 4 * kSMs), 256, 0, 1, true, s, sums)
                     : cudaSuccess;
  const int split[2] = {split_of(g[0]), n > 1 ? split_of(g[1]) : 0};
  const int together = n > 1 && split[0] == split[1] ? 2 : 1;
  for (int i = 0; i < n; i += together) {
    const cudaError_t e = split[i] ? run_split(g + i, together, split[i], sums, after, a.err, s)
                                   : run_pair(g + i, together, tiles, sums, after, a.err, s);
    if (e != cudaSuccess) return e;
    sums = {};
    after = false;
  }
  return cudaSuccess;
}

}  // namespace tttk
