// The dense layer with bias where the wide GEMM's tiles would leave SMs idle:
// single tokens, and rows up to a streaming unit.
//
// What both kernels compute: Y = act(A W^T + bias) (+ R), sums, bias, activation and
// residual in fp32, one rounding to bf16.
//
// token_rows_kernel, up to 16 rows. Every weight is used once or a few times,
// so the time is that of reading W from HBM, and for small layers that of one
// trip to memory. No shared-memory ring: a lane loads 16 bytes of a feature's
// row straight into the register operand of m16n8k16 MMAs (the order of the
// contracted index is free, so a lane's eight consecutive k serve two MMAs),
// rows of A likewise. A block takes 8 FT features; its 8 or 16 warps take
// neighbouring 32-wide chunks of K, and their sums meet in shared memory in a
// fixed order. One token, 1536 -> 8960: 4.8 us back to back, 6.3 (4.4 TB/s) with its
// 27.5 MB of weights from HBM; 8192 -> 8192 26.8 (5.0 TB/s).
//
// split_rows_kernel, more rows. Tiles of 128 rows x NF features on tcgen05, K
// cut over the CTAs of a cluster (any number up to 8) until the tiles fill the
// SMs; each CTA streams its share of K through a TMA ring of 192 KB, 128 of K a stage,
// accumulates in TMEM, and the partial tiles are summed through distributed
// shared memory in rank order: no workspace, no atomics, one launch. 192
// threads: warp 0 lane 0 TMA, warp 1 lane 0 tcgen05, warps 2..5 the epilogue.
// Every wait is bounded.
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

__device__ __forceinline__ float bf16_value(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }
__device__ __forceinline__ uint16_t to_bf16(float f) { return (uint16_t)(pack_bf16x2(f, 0.f) & 0xFFFF); }

// ---------------------------------------------------------------- up to 16 rows

struct TokenRowsParams {
  const uint16_t* a;
  const uint16_t* w;
  uint16_t* y;
  const uint16_t* resid;
  const uint16_t* bias;
  int64_t lda, ldr, ldy;
  int32_t M, K, N;
  int32_t ahead;  // bytes of each weight row that go into L2 before chain_wait
};

// 16 bytes, or zeros without a load (predicated, so that a batch of loads stays
// straight-line code with all of them in flight). Weights pass by L1.
__device__ __forceinline__ uint4 ld_weights(const uint16_t* p, bool in) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w) : "l"(p), "r"((int)in));
  return v;
}
__device__ __forceinline__ uint4 ld_rows(const uint16_t* p, bool in) {
  uint4 v;
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b32 %0, 0;\n\tmov.b32 %1, 0;\n\tmov.b32 %2, 0;\n\tmov.b32 %3, 0;\n\t"
      "@p ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=&r"(v.x), "=&r"(v.y), "=&r"(v.z), "=&r"(v.w) : "l"(p), "r"((int)in));
  return v;
}
// `bytes` (a multiple of 16, as `p` is aligned) on their way into L2.
__device__ __forceinline__ void prefetch_l2(const void* p, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
// WARPS: warps that share K; FT: n-tiles of 8 features per block; R16: more than 8 rows.
template <int WARPS, int FT, bool R16, int ACT>
__global__ void __launch_bounds__(32 * WARPS) token_rows_kernel(const __grid_constant__ TokenRowsParams p) {
  constexpr int U = FT == 1 ? 4 : 2;  // chunks of K in a batch
  __shared__ float red[WARPS][16][8 * FT];
  chain_begin();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int r8 = lane >> 2, q4 = lane & 3;
  const int f0 = blockIdx.x * 8 * FT;
  {
    // While the kernel before still runs, the weights are sent for: into L2, which a
    // write by that kernel would reach too, and not read. Thread t: piece t % pieces
    // of row t / pieces.
    const int rows = min(8 * FT, p.N - f0), pieces = (p.ahead + 2047) >> 11;
    const char* w = reinterpret_cast<const char*>(p.w + (int64_t)f0 * p.K);
    for (int t = threadIdx.x; t < rows * pieces; t += 32 * WARPS) {
      const int r = t / pieces, at = (t - r * pieces) << 11;
      prefetch_l2(w + (int64_t)r * p.K * 2 + at, (uint32_t)min(2048, p.ahead - at));
    }
  }
  chain_wait();
  const uint16_t* wrow[FT];
  bool win[FT];
#pragma unroll
  for (int t = 0; t < FT; ++t) {
    const int f = f0 + 8 * t + r8;
    win[t] = f < p.N;
    wrow[t] = p.w + (int64_t)(win[t] ? f : 0) * p.K + 8 * q4;
  }
  const bool in0 = r8 < p.M, in1 = R16 && r8 + 8 < p.M;
  const uint16_t* a0 = p.a + (in0 ? r8 : 0) * p.lda + 8 * q4;
  const uint16_t* a1 = p.a + (in1 ? r8 + 8 : 0) * p.lda + 8 * q4;
  float acc[FT][4] = {};
  const int chunks = (p.K + 31) >> 5;
  // Two batches of loads: one in flight while the other goes through the MMAs.
  uint4 w[2][U][FT], x0[2][U], x1[2][U];
  auto load = [&](int c0, int at) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int k = (c0 + u * WARPS) * 32;
      const bool in = k + 8 * q4 < p.K;
#pragma unroll
      for (int t = 0; t < FT; ++t) w[at][u][t] = ld_weights(wrow[t] + k, in && win[t]);
      x0[at][u] = ld_rows(a0 + k, in && in0);
      x1[at][u] = make_uint4(0, 0, 0, 0);
      if (R16) x1[at][u] = ld_rows(a1 + k, in && in1);
    }
  };
  auto multiply = [&](int at) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int t = 0; t < FT; ++t) {
        mma_16816<false>(acc[t], {x0[at][u].x, x1[at][u].x, x0[at][u].y, x1[at][u].y}, w[at][u][t].x, w[at][u][t].y);
        mma_16816<false>(acc[t], {x0[at][u].z, x1[at][u].z, x0[at][u].w, x1[at][u].w}, w[at][u][t].z, w[at][u][t].w);
      }
  };
  constexpr int kStep = WARPS * U;
  load(warp, 0);
#pragma unroll 1
  for (int c0 = warp; c0 < chunks; c0 += 2 * kStep) {
    load(c0 + kStep, 1);
    multiply(0);
    load(c0 + 2 * kStep, 0);
    multiply(1);
  }
#pragma unroll
  for (int t = 0; t < FT; ++t) {
    *reinterpret_cast<float2*>(&red[warp][r8][8 * t + 2 * q4]) = make_float2(acc[t][0], acc[t][1]);
    if (R16) *reinterpret_cast<float2*>(&red[warp][r8 + 8][8 * t + 2 * q4]) = make_float2(acc[t][2], acc[t][3]);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < p.M * 8 * FT; i += 32 * WARPS) {
    const int m = i / (8 * FT), f = i - m * 8 * FT;
    if (f0 + f >= p.N) continue;
    float v = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) v += red[k][m][f];
    if (p.bias) v += bf16_value(p.bias[f0 + f]);
    v = activate<ACT>(v);
    if (p.resid) v += bf16_value(p.resid[m * p.ldr + f0 + f]);
    p.y[m * p.ldy + f0 + f] = to_bf16(v);
  }
}

template <int WARPS, int FT, bool R16>
cudaError_t launch_token_rows(const TokenRowsParams& p, int act, cudaStream_t s) {
  const dim3 grid((unsigned)((p.N + 8 * FT - 1) / (8 * FT)));
  const unsigned threads = 32 * WARPS;
  switch (act) {
    case WAVE_ACT_GELU_TANH:
      return launch_chained(token_rows_kernel<WARPS, FT, R16, WAVE_ACT_GELU_TANH>, grid, threads, 0, s, 1, p);
    case WAVE_ACT_GELU_ERF:
      return launch_chained(token_rows_kernel<WARPS, FT, R16, WAVE_ACT_GELU_ERF>, grid, threads, 0, s, 1, p);
    case WAVE_ACT_SILU:
      return launch_chained(token_rows_kernel<WARPS, FT, R16, WAVE_ACT_SILU>, grid, threads, 0, s, 1, p);
    default:
      return launch_chained(token_rows_kernel<WARPS, FT, R16, WAVE_ACT_NONE>, grid, threads, 0, s, 1, p);
  }
}

// ------------------------------------------------------------------- more rows
constexpr int kSplitThreads = 192;

template <int NF>
struct SplitCfg {
  static constexpr int kATile = 128 * 128;  // 128 rows x 64 bf16
  static constexpr int kWTile = NF * 128;
  static constexpr int kStage = 2 * (kATile + kWTile);  // two panels of 64 of each: K = 128
  static constexpr int kStages = 196608 / kStage;
  static constexpr int kBarOff = kStages * kStage;
  static constexpr int kFull = 0, kEmpty = kStages, kAccFull = 2 * kStages, kDrain = kAccFull + 1,
                       kBars = kDrain + 1;
  static constexpr int kSmemBytes = kBarOff + kBars * 8 + 16 + 1024;
  // A row of a partial tile: four floats of padding, so that the 16-byte
  // stores of eight lanes (eight rows) fall into different banks.
  static constexpr int kPartRow = NF + 4;
  static_assert(8 * 16 * kPartRow * 4 <= kBarOff && 7 * 19 * kPartRow * 4 <= kBarOff, "partials reuse the ring");
  // kind::f16: fp32 accumulate, bf16 A and B, both K-major, N = NF, M = 128.
  static constexpr uint32_t kIdesc =
      (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(NF >> 3) << 17) | ((128u >> 4) << 24);
};

struct SplitParams {
  CUtensorMap tm_a;  // A [M][K], box 64 x box_rows
  CUtensorMap tm_w;  // W [N][K], box 64 x NF
  int32_t* status;
  uint64_t wait_ns;
  int32_t k_slices, n_ftiles, splits, box_rows;
  int32_t M, N;
  uint16_t* y;
  const uint16_t* resid;
  const uint16_t* bias;
  int64_t ldr, ldy;
  int32_t wide;
};

// The four K = 16 steps of a 64-wide slice in one block: low descriptor words
// a, b and 32 bytes on for each step, common high word.
__device__ __forceinline__ void mma_slice(uint32_t d, uint32_t a, uint32_t b, uint32_t hi, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, t;\n\t.reg .b64 x, y;\n\t.reg .b32 l, m;\n\t"
      "setp.ne.b32 p, %5, 0;\n\tsetp.eq.b32 t, %5, %5;\n\t"
      "mov.b64 x, {%1, %3};\n\tmov.b64 y, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, p;\n\t"
      "add.u32 l, %1, 2;\n\tadd.u32 m, %2, 2;\n\tmov.b64 x, {l, %3};\n\tmov.b64 y, {m, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n\t"
      "add.u32 l, %1, 4;\n\tadd.u32 m, %2, 4;\n\tmov.b64 x, {l, %3};\n\tmov.b64 y, {m, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n\t"
      "add.u32 l, %1, 6;\n\tadd.u32 m, %2, 6;\n\tmov.b64 x, {l, %3};\n\tmov.b64 y, {m, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %4, t;\n\t}" ::"r"(d), "r"(a), "r"(b), "r"(hi), "r"(idesc),
      "r"(accumulate)
      : "memory");
}

template <int NF, int ACT>
__global__ void __launch_bounds__(kSplitThreads, 1) split_rows_kernel(const __grid_constant__ SplitParams p) {
  using C = SplitCfg<NF>;
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
  const int rank = blockIdx.x % p.splits;  // the CTA's rank in its cluster
  const int tile = blockIdx.x / p.splits;
  const int mt = tile / p.n_ftiles, ft = tile - mt * p.n_ftiles;
  const int k0 = (int)((int64_t)rank * p.k_slices / p.splits);
  const int k1 = (int)((int64_t)(rank + 1) * p.k_slices / p.splits);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(bar(C::kFull + s), 1);
      mbar_init(bar(C::kEmpty + s), 1);
    }
    mbar_init(bar(C::kAccFull), 1);
    mbar_init(bar(C::kDrain), 1);
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&p.tm_a);
    prefetch_tmap(&p.tm_w);
  }
  if (warp == 1) {
    tmem_alloc(smem_addr(tmem_slot), NF);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  chain_begin();
  chain_wait();
  const int rows = min(128, p.M - mt * 128);   // rows of this tile
  const int cols = min(NF, p.N - ft * NF);     // columns of this tile, a multiple of 8

  if (warp == 0) {
    if (lane == 0) {
      // Rows past box_rows are left as they are: they only reach unused rows.
      const uint32_t bytes = 2 * (NF * 128 + p.box_rows * 128);
      int n = 0;
      int s = 0;
      uint32_t ph = 1;
      for (int k = k0; k < k1; ++k, ++n) {
        if (n >= S && !wait_within(bar(C::kEmpty + s), ph, ctl, 0x501)) break;
        mbar_arrive_expect_tx(bar(C::kFull + s), bytes);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t a = sb + s * C::kStage + j * C::kATile, w = sb + s * C::kStage + 2 * C::kATile + j * C::kWTile;
          tma_load_2d(w, &p.tm_w, k * 128 + j * 64, ft * NF, bar(C::kFull + s));
          tma_load_2d(a, &p.tm_a, k * 128 + j * 64, mt * 128, bar(C::kFull + s));
        }
        if (++s == S) s = 0, ph ^= 1;
      }
      // Copies still in flight land before the ring is reused or the CTA exits.
      for (int k = n > S ? n - S : 0; k < n; ++k) drain_wait(bar(C::kFull + k % S), (k / S) & 1);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint64_t desc = desc_k(sb);
      const uint32_t hi = (uint32_t)(desc >> 32), lo0 = (uint32_t)desc;
      bool ok = true;
      int s = 0;
      uint32_t ph = 0;
      for (int n = 0; n < k1 - k0; ++n) {
        if (!wait_within(bar(C::kFull + s), ph, ctl, 0x502)) {
          ok = false;
          break;
        }
        const uint32_t lo = lo0 + (uint32_t)s * (C::kStage >> 4);
        mma_slice(tmem, lo, lo + (2 * C::kATile >> 4), hi, C::kIdesc, n != 0);
        mma_slice(tmem, lo + (C::kATile >> 4), lo + ((2 * C::kATile + C::kWTile) >> 4), hi, C::kIdesc, 1);
        tc_commit(bar(C::kEmpty + s));
        if (++s == S) s = 0, ph ^= 1;
      }
      if (ok) tc_commit(bar(C::kAccFull));
      // Every MMA issued above completes before TMEM is released.
      tc_commit(bar(C::kDrain));
      drain_wait(bar(C::kDrain), 0);
    }
  } else {
    if (p.splits > 1) {
      __all_sync(0xffffffffu, wait_within(bar(C::kAccFull), 0, ctl, 0x503));
      tc_fence_after();
    }
  }
  __syncwarp();
  // Thread of warps 2..5: row of the tile (TMEM lane; warp w may read lanes 32 (w % 4) ..).
  const int row = (warp & 3) * 32 + lane;
  const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
  if (p.splits == 1) {
    if (warp >= 2)
      finish_row<ACT>(p, trow, (int64_t)mt * 128 + row, ft * NF, 0, NF, row < rows, [&] {
        const bool ok = __all_sync(0xffffffffu, wait_within(bar(C::kAccFull), 0, ctl, 0x503));
        tc_fence_after();
        return ok;
      });
  } else {
    // Sum the cluster's partial tiles: the CTA of rank o gets rows o * per ..
    // of every CTA's tile, as [source rank][row][kPartRow], in its ring.
    const int per = (rows + p.splits - 1) / p.splits;
    cluster_sync();  // every CTA of the cluster is done with its ring
    if (warp >= 2) {
      const int owner = row < rows ? row / per : rank;
      const uint32_t local = sb + (uint32_t)((rank * per + row - owner * per) * C::kPartRow) * 4;
      uint32_t remote;
      asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(local), "r"(owner));
#pragma unroll 1
      for (int c = 0; c < cols; c += 32) {
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
    sum_tiles<ACT, kSplitThreads>(p, reinterpret_cast<const float*>(smem), p.splits, per, C::kPartRow,
                                  min(per, rows - rank * per), cols, (int64_t)mt * 128 + rank * per, ft * NF,
                                  [] { __syncwarp(); cluster_sync(); });
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, NF);
  }
}

template <int NF, int ACT>
int launch_split(const SplitParams& p, int tiles, int device, cudaStream_t s) {
  static std::atomic<uint64_t> done{0};
  if (int rc = allow_shared(reinterpret_cast<const void*>(&split_rows_kernel<NF, ACT>), SplitCfg<NF>::kSmemBytes, device, done)) return rc;
  const cudaError_t e = launch_chained(split_rows_kernel<NF, ACT>, dim3((unsigned)(tiles * p.splits)), kSplitThreads,
                                       SplitCfg<NF>::kSmemBytes, s, (unsigned)p.splits, p);
  if (e != cudaSuccess)
    return fail(WAVE_ERR_CUDA, "split_rows_kernel launch: %s", cudaGetErrorString(e));
  return WAVE_OK;
}

template <int NF>
int launch_split_act(const SplitParams& p, int tiles, int act, int device, cudaStream_t s) {
  switch (act) {
    case WAVE_ACT_GELU_TANH: return launch_split<NF, WAVE_ACT_GELU_TANH>(p, tiles, device, s);
    case WAVE_ACT_GELU_ERF: return launch_split<NF, WAVE_ACT_GELU_ERF>(p, tiles, device, s);
    case WAVE_ACT_SILU: return launch_split<NF, WAVE_ACT_SILU>(p, tiles, device, s);
    default: return launch_split<NF, WAVE_ACT_NONE>(p, tiles, device, s);
  }
}

}  // namespace

int token_rows_launch(const DenseArgs& a, int ft, int warps, cudaStream_t s) {
  // Ahead of the wait go 16 MB in all, of each row its first part (chained, cold, us,
  // with none / 4 / 16 / 64 MB: 1536 -> 8960 7.2 / 6.5 / 6.3 / 6.7; 8960 -> 1536 9.3 /
  // 8.8 / 8.3 / 8.1; 8192 -> 8192 26.8 / 26.5 / 26.7 / 28.3; a block's whole step of
  // seven calls 48.4 / 47.4 / 46.7 / 48.8).
  const int64_t ahead = std::min<int64_t>(2LL * a.K, (16 << 20) / a.N & ~15);
  const TokenRowsParams p{static_cast<const uint16_t*>(a.A), static_cast<const uint16_t*>(a.W), a.Y, a.R, a.bias,
                          a.lda, a.ldr, a.ldy, a.M, a.K, a.N, (int32_t)ahead};
  const bool r16 = a.M > 8;
  const cudaError_t e =
      warps == 16 ? launch_token_rows<16, 1, false>(p, a.act, s)
      : ft == 1   ? (r16 ? launch_token_rows<8, 1, true>(p, a.act, s) : launch_token_rows<8, 1, false>(p, a.act, s))
                  : (r16 ? launch_token_rows<8, 2, true>(p, a.act, s) : launch_token_rows<8, 2, false>(p, a.act, s));
  if (e != cudaSuccess) return fail(WAVE_ERR_CUDA, "token_rows_kernel launch: %s", cudaGetErrorString(e));
  return WAVE_OK;
}

int split_rows_launch(const wave_kv* kv, const DenseArgs& a, int nf, int splits, cudaStream_t s) {
  SplitParams p = {};
  p.box_rows = std::min(128, (a.M + 15) / 16 * 16);
  if (int rc = encode_kmajor(&p.tm_w, a.W, a.N, a.K, (uint32_t)nf, "W")) return rc;
  if (int rc = encode_kmajor(&p.tm_a, a.A, a.M, a.K, (uint32_t)p.box_rows, "A", a.lda)) return rc;
  p.status = static_cast<int32_t*>(kv->cfg.pool);
  p.wait_ns = wait_limit_ns(kv);
  p.k_slices = (a.K + 127) / 128;  // the tensor maps fill K's tail with zeros
  p.n_ftiles = (a.N + nf - 1) / nf;
  p.splits = splits;
  p.M = a.M;
  p.N = a.N;
  p.y = a.Y;
  p.resid = a.R;
  p.bias = a.bias;
  p.ldr = a.ldr;
  p.ldy = a.ldy;
  p.wide = wide_rows(a.Y, a.ldy);
  const int tiles = p.n_ftiles * ((a.M + 127) / 128);
  return nf == 64 ? launch_split_act<64>(p, tiles, a.act, kv->device, s)
                  : launch_split_act<128>(p, tiles, a.act, kv->device, s);
}

}  // namespace wavei
