// The dense layer with bias for many rows, on pairs of SMs.
//
// What it computes: Y = act(A W^T + bias) (+ R), as the other forms (wave_few.cu).
//
// What bounds it: the tensor pipe, if the operands arrive. An SM takes in about
// 60 bytes a clock through TMA; a 128 x 256 tile of one SM wants 48 KB per 512
// tensor cycles, 96 a clock, so it stops at two thirds. Here a cluster of two
// CTAs computes a 256 x 256 (or 192) tile with cta_group::2 MMAs: each CTA holds its
// own 128 rows of A and half of W's rows, 32 KB per 512 cycles.
//
// How: 74 persistent pairs walk the tiles row-tile-major (A comes from HBM once,
// the weights stay in L2). Per CTA: warp 0 lane 0 feeds a 3-stage ring (K = 128 each) by TMA,
// both CTAs' bytes counted on the even CTA's barrier; warp 1 lane 0 of the even
// CTA issues the MMAs of both into one of two 256-column TMEM accumulators;
// warps 2..9 are the epilogue, two warps per 32 rows, while the other accumulator
// fills. SPLIT: too few tiles for the SMs; a cluster of 2 S CTAs takes one tile,
// its S pairs a share of K each, and the partial tiles are summed through
// distributed shared memory in pair order.
//
// Every wait is bounded. A pair that gives up leaves in step: the cluster's last
// barrier is behind every copy that either CTA has issued.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "ptx.cuh"
#include "wave_dense.cuh"
#include "wave_internal.h"
#include "wave_wait.cuh"

using namespace wptx;

namespace wavei {
namespace {

constexpr int kPairThreads = 320;

// NT: columns of a tile, 192 or 256 (192 fills the SMs better at some sizes).
template <int NT>
struct PairCfg {
  static constexpr int kATile = 128 * 128;      // 128 rows x 64 bf16
  static constexpr int kWTile = NT / 2 * 128;   // half of the columns' rows of W
  static constexpr int kStage = 2 * (kATile + kWTile);   // two panels of 64 of each: K = 128
  static constexpr int kStages = 204800 / kStage;
  static constexpr int kBarOff = kStages * kStage;
  static constexpr int kFull = 0, kEmpty = kStages, kAccFull = 2 * kStages, kAccEmpty = kAccFull + 2,
                       kDrain = kAccEmpty + 2, kBars = kDrain + 1;
  static constexpr int kSmemBytes = kBarOff + kBars * 8 + 16 + 1024;
  static constexpr int kPartRow = NT + 4;  // padded row of a partial tile, as in wave_few.cu
  static_assert(4 * 32 * kPartRow * 4 <= kBarOff && 3 * 43 * kPartRow * 4 <= kBarOff, "partials reuse the ring");
  // kind::f16, cta_group::2: fp32 accumulate, bf16 A and B, K-major, M = 256, N = NT.
  static constexpr uint32_t kIdesc =
      (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(NT >> 3) << 17) | ((256u >> 4) << 24);
};

struct PairParams {
  CUtensorMap tm_a;  // A [M][K], box 64 x 128
  CUtensorMap tm_w;  // W [N][K], box 64 x NT / 2
  int32_t* status;
  uint64_t wait_ns;
  int32_t k_slices, n_ntiles, n_tiles, splits;
  int32_t M, N;
  uint16_t* y;
  const uint16_t* resid;
  const uint16_t* bias;
  int64_t ldr, ldy;
  int32_t wide;
};

// `addr` of this CTA's shared memory, in the cluster's CTA `rank`.
__device__ __forceinline__ uint32_t in_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// A tile of this GPU's memory into this CTA's shared memory; the bytes count on
// the mbarrier `bar` of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const CUtensorMap* m, int32_t x, int32_t y, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(m)), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
// The four K = 16 steps of a 64-wide slice in one block: low descriptor words
// a, b and 32 bytes on for each step, common high word.
__device__ __forceinline__ void mma_pair_slice(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                               uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 x, y;\n\t.reg .b32 l, m;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, %5, %5;\n\t"
      "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %4, p;\n\t"
      "add.u32 l, %1, 2;\n\tadd.u32 m, %2, 2;\n\tmov.b64 x, {l, %3};\n\tmov.b64 y, {m, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %4, t;\n\t"
      "add.u32 l, %1, 4;\n\tadd.u32 m, %2, 4;\n\tmov.b64 x, {l, %3};\n\tmov.b64 y, {m, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %4, t;\n\t"
      "add.u32 l, %1, 6;\n\tadd.u32 m, %2, 6;\n\tmov.b64 x, {l, %3};\n\tmov.b64 y, {m, %3};\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %4, t;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(hi), "r"(idesc),
      "r"(accumulate)
      : "memory");
}
// Arrive on `bar` (the same offset in each CTA of `mask`) once all MMAs issued
// so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(mask)
      : "memory");
}
__device__ __forceinline__ void arrive_rank(uint32_t cluster_addr) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}
template <int NT, int ACT, bool SPLIT>
__global__ void __launch_bounds__(kPairThreads, 1) pair_rows_kernel(const __grid_constant__ PairParams p) {
  using C = PairCfg<NT>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_addr(smem);
  auto bar = [&](int i) -> uint32_t { return sb + C::kBarOff + 8u * i; };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::kBarOff + 8 * C::kBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBarOff + 8 * C::kBars + 4);
  const Ctl ctl{abort_flag, p.status, p.wait_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Ranks in the cluster: pair `pair`, CTA `half` of it; the pair's even CTA leads.
  const int ctas = SPLIT ? 2 * p.splits : 2;
  const int rank = blockIdx.x % ctas;
  const int pair = rank >> 1, half = rank & 1;
  const uint32_t lead = rank & ~1;
  const uint16_t both = (uint16_t)(3u << lead);
  const int tile0 = blockIdx.x / ctas, tile_step = SPLIT ? p.n_tiles : gridDim.x / 2;
  const int k0 = SPLIT ? (int)((int64_t)pair * p.k_slices / p.splits) : 0;
  const int k1 = SPLIT ? (int)((int64_t)(pair + 1) * p.k_slices / p.splits) : p.k_slices;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bar(C::kFull + s), 1);
      mbar_init(bar(C::kEmpty + s), 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(bar(C::kAccFull + a), 1);
      mbar_init(bar(C::kAccEmpty + a), 2 * 8);  // the epilogue warps of both CTAs
    }
    mbar_init(bar(C::kDrain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&p.tm_a);
    prefetch_tmap(&p.tm_w);
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // every CTA's barriers exist before another CTA signals them
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  chain_begin();
  chain_wait();

  if (warp == 0) {
    if (lane == 0) {
      const uint32_t full0 = in_rank(bar(C::kFull), lead);
      int g = 0, s = 0;
      uint32_t ph = 1;
      bool ok = true;
      for (int t = tile0; t < p.n_tiles && ok; t += tile_step) {
        const int mt = t / p.n_ntiles, nt = t - mt * p.n_ntiles;
        for (int k = k0; k < k1; ++k, ++g) {
          if (g >= S && !wait_within(bar(C::kEmpty + s), ph, ctl, 0x601)) {
            ok = false;
            break;
          }
          const uint32_t a = sb + s * C::kStage;
          if (half == 0) mbar_arrive_expect_tx(bar(C::kFull + s), 2 * C::kStage);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            tma_load_pair(a + j * C::kATile, &p.tm_a, k * 128 + j * 64, mt * 256 + half * 128, full0 + 8u * s);
            tma_load_pair(a + 2 * C::kATile + j * C::kWTile, &p.tm_w, k * 128 + j * 64, nt * NT + half * (NT / 2),
                          full0 + 8u * s);
          }
          if (++s == S) s = 0, ph ^= 1;
        }
      }
      // Copies still in flight land before the ring is reused or the pair leaves:
      // the even CTA's barrier counts both CTAs' bytes.
      if (half == 0)
        for (int k = g > S ? g - S : 0; k < g; ++k) drain_wait(bar(C::kFull + k % S), (k / S) & 1);
      if (!ok) {  // gave up: time for copies that no barrier of this CTA counts
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 200000) {
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && half == 0) {
      // This thread's own time bounds the loop unless it is short against the MMAs it
      // issues, and more so while the epilogue's warps take issue slots: 604 cycles
      // per 64 of K (512 of the tensor pipe's) with a division, a fence and a 64-bit
      // descriptor per MMA; 563, and 660 under a GELU epilogue, with the ring's
      // position kept and four MMAs in one block; 524 and 535 with 128 of K per
      // wait and commit.
      const uint64_t desc = desc_k(sb);
      const uint32_t hi = (uint32_t)(desc >> 32), lo0 = (uint32_t)desc;
      int s = 0, i = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = tile0; t < p.n_tiles && ok; t += tile_step, ++i) {
        const int acc = i & 1;
        if (i >= 2 && !wait_within(bar(C::kAccEmpty + acc), ((i >> 1) - 1) & 1, ctl, 0x602)) break;
        tc_fence_after();
        uint32_t accumulate = 0;
        for (int k = k0; k < k1; ++k) {
          if (!wait_within(bar(C::kFull + s), ph, ctl, 0x603)) {
            ok = false;
            break;
          }
          const uint32_t lo = lo0 + (uint32_t)s * (C::kStage >> 4);
          mma_pair_slice(tmem + 256 * acc, lo, lo + (2 * C::kATile >> 4), hi, C::kIdesc, accumulate);
          mma_pair_slice(tmem + 256 * acc, lo + (C::kATile >> 4), lo + ((2 * C::kATile + C::kWTile) >> 4), hi, C::kIdesc, 1);
          accumulate = 1;
          commit_pair(bar(C::kEmpty + s), both);
          if (++s == S) s = 0, ph ^= 1;
        }
        if (ok) commit_pair(bar(C::kAccFull + acc), both);
      }
      // Every MMA issued above completes before TMEM is released.
      commit_pair(bar(C::kDrain), (uint16_t)(1u << lead));
      drain_wait(bar(C::kDrain), 0);
    }
  } else {
    // Warps w and w + 4 own rows 32 (w % 4) .. (TMEM lanes) and half the columns each.
    const int quarter = warp & 3, side = (warp - 2) >> 2;
    const int row = quarter * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
    int i = 0;
    for (int t = tile0; t < p.n_tiles; t += tile_step, ++i) {
      const int acc = i & 1;
      bool ok = false;
      auto wait = [&] {
        ok = __all_sync(0xffffffffu, wait_within(bar(C::kAccFull + acc), (i >> 1) & 1, ctl, 0x604));
        tc_fence_after();
        return ok;
      };
      if constexpr (SPLIT) {
        wait();
      } else {
        const int mt = t / p.n_ntiles, nt = t - mt * p.n_ntiles;
        const int64_t m = (int64_t)mt * 256 + half * 128 + row;
        finish_row<ACT>(p, trow + 256 * acc, m, nt * NT, NT / 2 * side, NT / 2 * (side + 1), m < p.M, wait);
        if (!ok) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_rank(in_rank(bar(C::kAccEmpty + acc), lead));
      }
    }
  }
  __syncwarp();
  if constexpr (SPLIT) {
    // Sum the pairs' partial tiles: of the 128 rows of this half, pair o gets rows
    // o * per .., from the same half of every pair, as [pair][row][kPartRow].
    const int mt = tile0 / p.n_ntiles, nt = tile0 - mt * p.n_ntiles;
    const int rows = max(0, min(128, p.M - mt * 256 - half * 128));
    const int cols = min(NT, p.N - nt * NT);
    const int per = max(1, (rows + p.splits - 1) / p.splits);
    cluster_sync();  // every CTA of the cluster is done with its ring
    if (warp >= 2) {
      const int quarter = warp & 3, side = (warp - 2) >> 2;
      const int row = quarter * 32 + lane;
      const uint32_t trow = tmem + ((uint32_t)(quarter * 32) << 16);
      const int owner = row < rows ? row / per : pair;
      const uint32_t remote =
          in_rank(sb + (uint32_t)((pair * per + row - owner * per) * C::kPartRow) * 4, 2 * owner + half);
#pragma unroll 1
      for (int c = NT / 2 * side; c < min(cols, NT / 2 * (side + 1)); c += 32) {
        uint32_t v[32];
        tmem_ld32_wait(trow + c, v);
        if (row < rows) {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(remote + (uint32_t)(c + 4 * j) * 4),
                         "r"(v[4 * j]), "r"(v[4 * j + 1]), "r"(v[4 * j + 2]), "r"(v[4 * j + 3])
                         : "memory");
        }
        __syncwarp();
      }
    }
    __syncwarp();
    sum_tiles<ACT, kPairThreads>(p, reinterpret_cast<const float*>(smem), p.splits, per, C::kPartRow,
                                 min(per, rows - pair * per), cols, (int64_t)mt * 256 + half * 128 + pair * per,
                                 nt * NT, [] { __syncwarp(); cluster_sync(); });
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA leaves while the other's MMAs or signals reach into it
  if (warp == 1) {
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
  }
}

template <int NT, int ACT, bool SPLIT>
int launch_pair(const PairParams& p, int ctas, int cluster, int device, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  if (int rc = allow_shared(reinterpret_cast<const void*>(&pair_rows_kernel<NT, ACT, SPLIT>), PairCfg<NT>::kSmemBytes, device, done)) return rc;
  const cudaError_t e = launch_chained(pair_rows_kernel<NT, ACT, SPLIT>, dim3((unsigned)ctas), kPairThreads,
                                       PairCfg<NT>::kSmemBytes, s, (unsigned)cluster, p);
  if (e != cudaSuccess)
    return fail(WAVE_ERR_CUDA, "pair_rows_kernel launch: %s", cudaGetErrorString(e));
  return WAVE_OK;
}

template <int NT, int ACT>
int launch_pair_any(const PairParams& p, int ctas, int cluster, int device, cudaStream_t s) {
  return cluster > 2 ? launch_pair<NT, ACT, true>(p, ctas, cluster, device, s)
                     : launch_pair<NT, ACT, false>(p, ctas, cluster, device, s);
}
template <int NT>
int launch_pair_act(const PairParams& p, int act, int ctas, int cluster, int device, cudaStream_t s) {
  switch (act) {
    case WAVE_ACT_GELU_TANH: return launch_pair_any<NT, WAVE_ACT_GELU_TANH>(p, ctas, cluster, device, s);
    case WAVE_ACT_GELU_ERF: return launch_pair_any<NT, WAVE_ACT_GELU_ERF>(p, ctas, cluster, device, s);
    case WAVE_ACT_SILU: return launch_pair_any<NT, WAVE_ACT_SILU>(p, ctas, cluster, device, s);
    default: return launch_pair_any<NT, WAVE_ACT_NONE>(p, ctas, cluster, device, s);
  }
}

}  // namespace

int pair_rows_launch(const wave_kv* kv, const DenseArgs& a, int nt, int splits, cudaStream_t s) {
  PairParams p = {};
  if (int rc = encode_kmajor(&p.tm_a, a.A, a.M, a.K, 128, "A", a.lda)) return rc;
  if (int rc = encode_kmajor(&p.tm_w, a.W, a.N, a.K, (uint32_t)nt / 2, "W")) return rc;
  p.status = static_cast<int32_t*>(kv->cfg.pool);
  p.wait_ns = wait_limit_ns(kv);
  p.k_slices = (a.K + 127) / 128;  // the tensor maps fill K's tail with zeros
  p.n_ntiles = (a.N + nt - 1) / nt;
  const int64_t tiles = ((int64_t)a.M + 255) / 256 * p.n_ntiles;
  if (tiles >= (1LL << 28)) return fail(WAVE_ERR_ARG, "M x N too large");
  p.n_tiles = (int32_t)tiles;
  p.splits = splits;
  p.M = a.M;
  p.N = a.N;
  p.y = a.Y;
  p.resid = a.R;
  p.bias = a.bias;
  p.ldr = a.ldr;
  p.ldy = a.ldy;
  p.wide = wide_rows(a.Y, a.ldy);
  const int cluster = 2 * splits;
  const int ctas = splits > 1 ? p.n_tiles * cluster : 2 * std::min(p.n_tiles, kv->num_sms / 2);
  return nt == 192 ? launch_pair_act<192>(p, a.act, ctas, cluster, kv->device, s)
                   : launch_pair_act<256>(p, a.act, ctas, cluster, kv->device, s);
}

}  // namespace wavei
