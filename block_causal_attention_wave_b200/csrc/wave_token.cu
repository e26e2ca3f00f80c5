// Attention of single query tokens over the paged (chunk, level) cache, cut
// over the cache's length and joined.
//
// What it computes: for query token i, query head x and K/V head h = x / g,
//   O = sum_k p_k V_k / sum_k p_k,  p_k = exp(Q . K_k / sqrt(d)),
// over the tokens of the query's key list. Any cut of the list into parts with
// (m, l, O') = (max score, sum of exp(score - m), sum of exp(score - m) V) gives
// the same result: M = max m, O = sum e^(m - M) O' / sum e^(m - M) l.
//
// What bounds it: HBM. Every cached byte is used for one multiply-add per
// query, far below the tensor pipe's ratio, so the kernel is built around
// keeping page tiles in flight.
//
// How:
//   - A list item is a page together with the number of its tokens seen and a
//     16-bit mask of the query rows that see them; up to 16 query rows
//     (consecutive queries times g heads) form a group, whose distinct items are
//     read once. A list is a group's items for one K/V head. A cluster of 1 to 8
//     CTAs takes a list, each CTA an equal run of its items, and joins the parts
//     through distributed shared memory: one launch, no workspace. An SM draws at
//     most about 95 GB/s through TMA, so 70 of them already saturate HBM, and
//     clusters that do not pack all 148 cost nothing. Fewer than 8 long lists
//     are cut into parts for several clusters each, which leave their (m, l, O')
//     in the workspace for a second kernel.
//   - Warps are two or three teams that take every other unit; a warp takes 32 of
//     the page's 128 keys, for all rows, with its own running maximum, sum
//     and O: no exchange between warps until the CTA's items end.
//   - A further warp per team feeds it, K and V tiles by TMA through a ring of the
//     team's own (192 KB in flight per SM in all). A ring that the teams shared
//     would need every warp at every slot: a parity wait tells apart only the
//     phase after the last one its waiter saw, so a team that skipped the other
//     team's fill of a slot could take it for its own.
//   - Both products are m16n8k16 MMAs with the cache as the operand of sixteen rows:
//     S^T = K Q^T (16 keys x 8 query rows) and O^T += V^T P^T (16 d x 8 query
//     rows), QT = 1 or 2 tiles of query rows. With the queries as the sixteen rows
//     one token filled one of them: twice the MMAs, exponentials and registers
//     (32 FP8 units: 50.7 us, this way 40.8, and 38.1 with launches chained).
//   - Within an MMA the order of the contracted index, and which d is which row,
//     are free, so a lane's operand is whole 16-byte vectors of a token's row, all
//     conflict-free under the swizzle; P is turned into its operand's layout by
//     one movmatrix per 8 keys.
//   - FP8 tiles: codes are exact in f16, so both MMAs run in f16 on converted
//     codes (e4m3 MMAs on the codes themselves, with Q and P as sums of two E4M3
//     values, took 80 us for those 50: this GPU has no fast form of them outside
//     tcgen05). Q is scaled by a power of two per row to fit f16 (its 8 bits of
//     mantissa stay exact down to 2^-24 of the row's largest value). P, in
//     [0, 1], is scaled by 2^15, so what f16 drops is below 2^-39; V's scale is
//     applied to each page's product in fp32.
//   - bf16: P goes in as two bf16, its leading eight bits and the rest (what is
//     dropped is below 2^-15 of it), one MMA each: rounded to one, the few
//     weights of a peaked softmax would be off by up to 2^-8 each (seven chunks of 4680
//     tokens, 12 heads: 34.4 us so, 34.7 with both; with more than eight query rows,
//     whose products are twice as many, 5 to 10 % more). The rest of a weight is a
//     positive number wherever the weight is (down to 2^-109), so that an infinite V
//     that is seen gives an infinity, not the NaN of its product with zero.
//   - Rows that do not see an item keep their O by selection, not by a zero
//     weight, and V rows past the seen tokens are zeroed: whatever stands
//     there, infinities and NaN included, reaches nothing.
#include <cuda.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <new>
#include <type_traits>
#include <utility>
#include <vector>

#include "ptx.cuh"
#include "wave_dense.cuh"
#include "wave_internal.h"
#include "wave_wait.cuh"

using namespace wptx;

namespace wavei {
namespace {

constexpr int kTokTeam = 4;                        // warps of a unit, 32 keys each
constexpr int kTokRows = 16;                       // query rows of a group

struct TokGroup {
  int32_t item0;    // first item in the tables
  int32_t n_items;
  int32_t q0;       // first query
  int32_t rows;     // query rows: queries * heads_per_kv
};

struct TokHead {
  CUtensorMap tm;            // pool pages
  const float* scales;       // FP8: [max_pages][2][H]
  const uint16_t* q;
  uint16_t* o;
  float* lse;                // or null
  float* part_o;             // [list][part][rows_max][d]
  float2* part_ml;           // [list][part][rows_max]
  int64_t ldq, ldo;
  int32_t* status;
  uint64_t wait_ns;
  float scale_log2;          // log2(e) / sqrt(d)
  int32_t heads;             // K/V heads
  int32_t per_kv;            // query heads per K/V head
  int32_t n_groups;
  int32_t cluster;           // CTAs per cluster
  int32_t parts;             // clusters per list
  int32_t rows_max;
  TokGroup g[WAVE_MAX_NODES];
};

// The tables travel in the parameter block: 512 items where they suffice.
template <int CAP>
struct TokParams {
  TokHead h;
  uint32_t page[CAP];   // page | (tokens seen - 1) << 25
  uint16_t mask[CAP];   // query rows that see it
};
constexpr int kTokCapSmall = 512;
static_assert(sizeof(TokParams<WAVE_MAX_TOKEN_PAGES>) <= 32760, "kernel parameter space is 32 KB");

template <int D, bool FP8, int QT>
struct TokCfg {
  // Unit n of a CTA goes to team n % kTeams. Three teams hide more of the codes'
  // conversion (12 heads of d = 128 over seven FP8 chunks: 24.7 us, with two 27.7);
  // bf16 is bound by HBM either way and ends sooner with two (77 own tokens: 6.5
  // us, with three 7.0).
  static constexpr int kTeams = FP8 && QT == 1 ? 3 : 2;
  static constexpr int kWarps = kTokTeam * kTeams;   // consumers
  // A warpgroup of producers follows, one warp per team and idle ones: registers
  // move between whole warpgroups.
  static constexpr int kThreads = 32 * (kWarps + 4);
  // d = 128: registers a thread at launch, then of producers and consumers: 128 * 72
  // + 256 * 216 = 64,512 or 128 * 40 + 384 * 152 = 63,488 of the launch's 64,512 or
  // 65,536.
  static constexpr int kRegsLaunch = kTeams == 3 ? 128 : 168, kRegsFeed = kTeams == 3 ? 40 : 72,
                       kRegsWork = kTeams == 3 ? 152 : 216;
  static_assert(128 * kRegsFeed + 32 * kWarps * kRegsWork <= kThreads * kRegsLaunch, "register split");
  static constexpr int kTile = 128 * D * (FP8 ? 1 : 2);
  static constexpr int kSlots = 196608 / kTeams / kTile;              // of each team's ring
  static constexpr int kStatOff = kTeams * kSlots * kTile;         // [8][16] float2
  static constexpr int kMlOff = kStatOff + kWarps * kTokRows * 8;  // [16] float2: the CTA's
  static constexpr int kBarOff = kMlOff + kTokRows * 8;
  static constexpr int kSmemBytes = kBarOff + 2 * kTeams * kSlots * 8 + 16 + 1024;
  // After the last tile the ring holds the warps' O, [8][16][kRow] fp32, and
  // behind it the CTA's, [16][kRow].
  static constexpr int kRow = D + 4;
  static constexpr int kCtaOff = kWarps * kTokRows * kRow * 4;
  static_assert(kCtaOff + kTokRows * kRow * 4 <= kStatOff, "the joins reuse the ring");
  static constexpr int kTiles = D / 16;   // tiles of 16 d of O^T
  static constexpr int kSteps = D / 16;   // k-steps of K Q^T
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
// Two E4M3 codes (low 16 bits of w) to two f16 values.
__device__ __forceinline__ uint32_t e4m3_f16x2(uint32_t w) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)w));
  return h;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
// A float (pair) at shared address `addr` of the cluster's CTA `rank`.
__device__ __forceinline__ float lds_rank(uint32_t addr, int rank) {
  float v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %1, %2;\n\tld.shared::cluster.f32 %0, [a];\n\t}"
               : "=f"(v) : "r"(addr), "r"(rank) : "memory");
  return v;
}
__device__ __forceinline__ float2 lds_rank2(uint32_t addr, int rank) {
  float2 v;
  asm volatile("{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %2, %3;\n\tld.shared::cluster.v2.f32 {%0, %1}, [a];\n\t}"
               : "=f"(v.x), "=f"(v.y) : "r"(addr), "r"(rank) : "memory");
  return v;
}
template <int THREADS>
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// First d of the two that lane row r holds of O^T's tile t (the next tile's follow).
template <int D, bool FP8>
__device__ __forceinline__ int tok_d(int t, int r) {
  if (!FP8) return 64 * (t >> 2) + 8 * r + 2 * (t & 3);
  return (D == 128 ? 16 : 8) * r + 2 * t;
}
// 8 x 8 values of 16 bits, transposed across the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int D, bool FP8, int QT, int CAP>
__global__ void __launch_bounds__(TokCfg<D, FP8, QT>::kThreads, 1)
    token_attn_kernel(const __grid_constant__ TokParams<CAP> p) {
  using C = TokCfg<D, FP8, QT>;
  constexpr int S = C::kSlots;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_addr(smem);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBarOff + 16 * C::kTeams * S);
  const TokHead& h = p.h;
  const Ctl ctl{abort_flag, h.status, h.wait_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // This CTA's list (group, K/V head), part, rank in the cluster, and items.
  const int rank = blockIdx.x % h.cluster;
  const int part_id = blockIdx.x / h.cluster % h.parts;
  const int list = blockIdx.x / (h.cluster * h.parts);
  const int head = list % h.heads;
  const TokGroup& grp = h.g[list / h.heads];
  const int share = part_id * h.cluster + rank, shares = h.cluster * h.parts;
  const int u0 = (int)((int64_t)grp.n_items * share / shares);
  const int u1 = (int)((int64_t)grp.n_items * (share + 1) / shares);
  const uint32_t* pages = p.page + grp.item0;
  const uint16_t* masks = p.mask + grp.item0;
  // The ring of this warp's team: fill f (K of the team's unit j is fill 2 j, V
  // fill 2 j + 1) is in slot f % S, in phase f / S of its barriers.
  const int team = warp < C::kWarps ? warp / kTokTeam : warp - C::kWarps;
  const uint32_t ring = sb + team * S * C::kTile;
  const uint32_t bars = sb + C::kBarOff + 16u * S * team;
  auto full = [&](int s) -> uint32_t { return bars + 8u * s; };
  auto empty = [&](int s) -> uint32_t { return bars + 8u * (S + s); };

  chain_begin();
  if (threadIdx.x == 0) {
    for (int t = 0; t < C::kTeams; ++t)
      for (int s = 0; s < S; ++s) {
        mbar_init(sb + C::kBarOff + 16u * S * t + 8u * s, 1);
        mbar_init(sb + C::kBarOff + 16u * S * t + 8u * (S + s), kTokTeam);
      }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&h.tm);
  }
  __syncthreads();
  chain_wait();

  if (warp >= C::kWarps) {
    if constexpr (D == 128) regs_dec<C::kRegsFeed>();
    if (lane == 0 && team < C::kTeams) {
      int f = 0;
      bool ok = true;
      for (int u = u0 + team; u < u1 && ok; u += C::kTeams) {
        const int page = (int)(pages[u] & 0x1FFFFFFu);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int s = f % S;
          if (f >= S && !wait_within(empty(s), (f / S - 1) & 1, ctl, 0x401)) {
            ok = false;
            break;
          }
          const uint32_t dst = ring + s * C::kTile;
          const int tile = (page * 2 + kv) * h.heads + head;
          mbar_arrive_expect_tx(full(s), C::kTile);
          if constexpr (FP8) {
            tma_load_2d(dst, &h.tm, 0, tile * D, full(s));
          } else {
#pragma unroll
            for (int b = 0; b < D / 64; ++b) tma_load_2d(dst + b * 16384, &h.tm, 64 * b, tile * 128, full(s));
          }
          ++f;
        }
      }
      // Copies still in flight land before the CTA exits.
      for (int k = f > S ? f - S : 0; k < f; ++k) drain_wait(full(k % S), (k / S) & 1);
    }
    // These warps end here (the cluster's barriers wait for threads that have not
    // exited): what follows may use more registers than they kept.
    return;
  }
  if constexpr (D == 128) regs_inc<C::kRegsWork>();
  {
  // ---- consumers: keys 32 (warp % 4) .. + 31 of every other page
  const int key0 = 32 * (warp % kTokTeam);
  const int r8 = lane >> 2, q4 = lane & 3;   // fragment row, lane quarter
  float o[QT][C::kTiles][4];                 // O^T: d tok_d + (c >> 1), query row 8 t + 2 q4 + (c & 1)
  uint32_t qf[QT][C::kSteps][2];             // Q of query row 8 t + r8
  float m[QT][2], l[QT][2], qs[QT][2];       // of query rows 8 t + 2 q4 (+ 1): maximum (log2), this
                                             // lane's part of the sum, score factor
  bool dead = false;
  const int rows = grp.rows;
  const uint32_t all_rows = (1u << rows) - 1;
#pragma unroll
    for (int t = 0; t < QT; ++t) {
      const int row = 8 * t + r8;
      const uint16_t* src = h.q + (grp.q0 + row / h.per_kv) * h.ldq +
                            (int64_t)(head * h.per_kv + row % h.per_kv) * D;
      const bool in = row < rows;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[t][i] = -INFINITY;
        l[t][i] = 0.f;
        qs[t][i] = h.scale_log2;
      }
      if constexpr (!FP8) {
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in) v = *reinterpret_cast<const uint4*>(src + 64 * b + 8 * (2 * q4 + hh));
            const int st = (b * 2 + hh) * 2;
            qf[t][st][0] = v.x;
            qf[t][st][1] = v.y;
            qf[t][st + 1][0] = v.z;
            qf[t][st + 1][1] = v.w;
          }
      } else {
        // Lane quarter q4 holds d = 16 (D / 64 q4 + hh) .. + 15, hh < D / 64.
        uint32_t raw[C::kSteps * 2];
#pragma unroll
        for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in) v = *reinterpret_cast<const uint4*>(src + 16 * (D / 64 * q4 + hh) + 8 * j);
            raw[hh * 8 + j * 4] = v.x;
            raw[hh * 8 + j * 4 + 1] = v.y;
            raw[hh * 8 + j * 4 + 2] = v.z;
            raw[hh * 8 + j * 4 + 3] = v.w;
          }
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < C::kSteps * 2; ++j)
          top = fmaxf(top, fmaxf(fabsf(__uint_as_float(raw[j] << 16)),
                                 fabsf(__uint_as_float(raw[j] & 0xFFFF0000u))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // 2^e brings the row's largest magnitude into [2^13, 2^14).
        int e = 0;
        if (top > 0.f && top < INFINITY)
          e = min(13 - ((int)(__float_as_uint(top) >> 23) - 127), 120);
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int i = 0; i < 2; ++i) qs[t][i] *= __shfl_sync(0xffffffffu, down, 8 * q4 + 4 * i);
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t v = raw[st * 2 + j];
            qf[t][st][j] = pack_f16x2(__uint_as_float(v << 16) * up, __uint_as_float(v & 0xFFFF0000u) * up);
          }
      }
#pragma unroll
      for (int x = 0; x < C::kTiles; ++x)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[t][x][c] = 0.f;
    }

    // One unit: S^T = K Q^T, the softmax's step, O^T += V^T P^T, for the warp's 32
    // keys. false: a wait ran out. WHOLE: every row sees all 128 tokens.
    auto unit = [&](auto whole_c, int ks, int vs, int vp, int seen, uint32_t mask, float sk, float sv) -> bool {
      constexpr bool WHOLE = decltype(whole_c)::value;
      const bool some = WHOLE || key0 < seen;   // the warp has a key that is seen
      uint32_t pb[QT][2][2];                    // P^T of the warp's two blocks of sixteen keys
      [[maybe_unused]] uint32_t pr[FP8 ? 1 : QT][2][2];   // bf16: what pb leaves of it
      auto sees = [&](int t, int i) { return (mask >> (8 * t + 2 * q4 + i) & 1) != 0; };
      if (some) {
        const uint32_t kt = ring + ks * C::kTile;
        // ---- S^T: block kb, keys r8 (c = 0, 1) and r8 + 8 (c = 2, 3)
        float sc[QT][2][4];
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[t][kb][c] = 0.f;
        if constexpr (!FP8) {
#pragma unroll
          for (int b = 0; b < D / 64; ++b)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int kb = 0; kb < 2; ++kb) {
                const uint32_t row = kt + b * 16384 + (key0 + kb * 16 + r8) * 128 + (((2 * q4 + hh) ^ r8) << 4);
                const uint4 u = lds128(row), v = lds128(row + 8 * 128);
                const uint32_t a0[4] = {u.x, v.x, u.y, v.y}, a1[4] = {u.z, v.z, u.w, v.w};
                const int st = (b * 2 + hh) * 2;
#pragma unroll
                for (int t = 0; t < QT; ++t) {
                  mma_16816<false>(sc[t][kb], a0, qf[t][st][0], qf[t][st][1]);
                  mma_16816<false>(sc[t][kb], a1, qf[t][st + 1][0], qf[t][st + 1][1]);
                }
              }
        } else {
#pragma unroll
          for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
              uint32_t wd[2][4];
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int key = key0 + kb * 16 + k * 8 + r8;
                const int line = D == 128 ? key : key >> 1;
                const int chunk = D == 128 ? 2 * q4 + hh : (key & 1) * 4 + q4;
                const uint4 v = lds128(kt + line * 128 + ((chunk ^ (line & 7)) << 4));
                wd[k][0] = v.x; wd[k][1] = v.y; wd[k][2] = v.z; wd[k][3] = v.w;
              }
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const uint32_t a[4] = {e4m3_f16x2(wd[0][j] & 0xFFFF), e4m3_f16x2(wd[1][j] & 0xFFFF),
                                       e4m3_f16x2(wd[0][j] >> 16), e4m3_f16x2(wd[1][j] >> 16)};
#pragma unroll
                for (int t = 0; t < QT; ++t) mma_16816<true>(sc[t][kb], a, qf[t][hh * 4 + j][0], qf[t][hh * 4 + j][1]);
              }
            }
        }
        // ---- softmax of this warp's keys; query rows 2 q4 (c = 0, 2) and 2 q4 + 1 (c = 1, 3)
        bool grew = false;
        float top[QT][2], shift[QT][2];
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float f = FP8 ? qs[t][i] * sk : qs[t][i];
            top[t][i] = -INFINITY;
#pragma unroll
            for (int kb = 0; kb < 2; ++kb)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                float& x = sc[t][kb][2 * k + i];
                x *= f;
                if (!WHOLE && (!sees(t, i) || key0 + kb * 16 + k * 8 + r8 >= seen)) x = -INFINITY;
                top[t][i] = fmaxf(top[t][i], x);
              }
#pragma unroll
            for (int x = 4; x < 32; x *= 2) top[t][i] = fmaxf(top[t][i], __shfl_xor_sync(0xffffffffu, top[t][i], x));
            top[t][i] = fmaxf(top[t][i], m[t][i]);
            grew |= top[t][i] > m[t][i];
            shift[t][i] = top[t][i] == -INFINITY ? 0.f : top[t][i];
          }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int t = 0; t < QT; ++t)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              if (top[t][i] > m[t][i]) {
                const float f = ex2_approx(m[t][i] - shift[t][i]);
                l[t][i] *= f;
                m[t][i] = top[t][i];
#pragma unroll
                for (int x = 0; x < C::kTiles; ++x) {
                  o[t][x][i] *= f;
                  o[t][x][2 + i] *= f;
                }
              }
        }
#pragma unroll
        for (int t = 0; t < QT; ++t)
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float a = ex2_approx(sc[t][kb][2 * k] - shift[t][0]);
              const float b = ex2_approx(sc[t][kb][2 * k + 1] - shift[t][1]);
              l[t][0] += a;
              l[t][1] += b;
              if constexpr (FP8) {
                pb[t][kb][k] = transpose8(pack_f16x2(a * 32768.f, b * 32768.f));
              } else {
                const uint32_t ha = __float_as_uint(a) & 0xFFFF0000u, hb = __float_as_uint(b) & 0xFFFF0000u;
                pb[t][kb][k] = transpose8(ha >> 16 | hb);
                pr[t][kb][k] = transpose8(pack_bf16x2(fmaf(a, 0x1p-24f, a - __uint_as_float(ha)),
                                                      fmaf(b, 0x1p-24f, b - __uint_as_float(hb))));
              }
            }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(ks));
      if (!__all_sync(0xffffffffu, wait_within(full(vs), vp, ctl, 0x403))) return false;
      if (some) {
        // ---- O^T += V^T P^T: of each block, a lane's keys are 2 q4, + 1, + 8, + 9
        const uint32_t vt = ring + vs * C::kTile;
        auto key_of = [&](int kb, int k) { return key0 + 16 * kb + 2 * q4 + (k & 1) + 8 * (k >> 1); };
        if constexpr (!FP8) {
#pragma unroll
          for (int b = 0; b < D / 64; ++b)
#pragma unroll
            for (int kb = 0; kb < 2; ++kb) {
              uint32_t x[4][4];
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const int key = key_of(kb, k);
                uint4 v = lds128(vt + b * 16384 + key * 128 + ((r8 ^ (key & 7)) << 4));
                if (!WHOLE && key >= seen) v = make_uint4(0, 0, 0, 0);
                x[k][0] = v.x; x[k][1] = v.y; x[k][2] = v.z; x[k][3] = v.w;
              }
              uint32_t a[4][4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                a[e][0] = __byte_perm(x[0][e], x[1][e], 0x5410);
                a[e][1] = __byte_perm(x[0][e], x[1][e], 0x7632);
                a[e][2] = __byte_perm(x[2][e], x[3][e], 0x5410);
                a[e][3] = __byte_perm(x[2][e], x[3][e], 0x7632);
              }
              if constexpr (WHOLE) {
#pragma unroll
                for (int e = 0; e < 4; ++e)
#pragma unroll
                  for (int t = 0; t < QT; ++t) {
                    mma_16816<false>(o[t][b * 4 + e], a[e], pr[t][kb][0], pr[t][kb][1]);
                    mma_16816<false>(o[t][b * 4 + e], a[e], pb[t][kb][0], pb[t][kb][1]);
                  }
              } else {
                // Two tiles of query rows: products apart, then added (16 queries over 632
                // MB of pages: 120 us, else 125); one: carried through and selected (one
                // token, 77 keys of its own: 5.32 us, else 5.45).
#pragma unroll
                for (int e0 = 0; e0 < 4; e0 += 2) {
                  float d[2][QT][4] = {};
                  if constexpr (QT == 1) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) d[i >> 2][0][i & 3] = o[0][b * 4 + e0 + (i >> 2)][i & 3];
                  }
#pragma unroll
                  for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int t = 0; t < QT; ++t) mma_16816<false>(d[e][t], a[e0 + e], pr[t][kb][0], pr[t][kb][1]);
#pragma unroll
                  for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int t = 0; t < QT; ++t) {
                      mma_16816<false>(d[e][t], a[e0 + e], pb[t][kb][0], pb[t][kb][1]);
                      float (&acc)[4] = o[t][b * 4 + e0 + e];
#pragma unroll
                      for (int c = 0; c < 4; ++c)
                        if (sees(t, c & 1)) acc[c] = QT == 1 ? d[e][t][c] : acc[c] + d[e][t][c];
                    }
                }
              }
            }
        } else {
          const float f = sv * 0x1p-15f;
          uint32_t x[2][4][D / 32];
#pragma unroll
          for (int kb = 0; kb < 2; ++kb)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int key = key_of(kb, k);
              if constexpr (D == 128) {
                const uint4 v = lds128(vt + key * 128 + ((r8 ^ (key & 7)) << 4));
                x[kb][k][0] = v.x; x[kb][k][1] = v.y; x[kb][k][2] = v.z; x[kb][k][3] = v.w;
              } else {
                const int line = key >> 1, chunk = (key & 1) * 4 + (r8 >> 1);
                const uint2 v = lds64(vt + line * 128 + ((chunk ^ (line & 7)) << 4) + (r8 & 1) * 8);
                x[kb][k][0] = v.x; x[kb][k][1] = v.y;
              }
              if (!WHOLE && key >= seen) {
#pragma unroll
                for (int j = 0; j < D / 32; ++j) x[kb][k][j] = 0;
              }
            }
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              // codes of d 4 j + 2 half (low 16 bits) and the next: keys (0, 1) and (8, 9)
              const uint32_t sel = half ? 0x7362 : 0x5140;
              float d[QT][4] = {};
#pragma unroll
              for (int kb = 0; kb < 2; ++kb) {
                const uint32_t k01 = __byte_perm(x[kb][0][j], x[kb][1][j], sel);
                const uint32_t k89 = __byte_perm(x[kb][2][j], x[kb][3][j], sel);
                const uint32_t a[4] = {e4m3_f16x2(k01 & 0xFFFF), e4m3_f16x2(k01 >> 16), e4m3_f16x2(k89 & 0xFFFF),
                                       e4m3_f16x2(k89 >> 16)};
#pragma unroll
                for (int t = 0; t < QT; ++t) mma_16816<true>(d[t], a, pb[t][kb][0], pb[t][kb][1]);
              }
#pragma unroll
              for (int t = 0; t < QT; ++t)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                  if (WHOLE || sees(t, c & 1)) o[t][2 * j + half][c] = fmaf(f, d[t][c], o[t][2 * j + half][c]);
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(vs));
      return true;
    };
    int f = 0;   // the team's fills taken
    // The next unit's table words and scales are fetched a unit ahead: a scale is a
    // trip to L2, which a unit of its own could not hide.
    uint32_t next_word = 0, next_mask = 0;
    float next_sk = 1.f, next_sv = 1.f;
    auto fetch = [&](int u) {
      if (u >= u1) return;
      next_word = pages[u];
      next_mask = masks[u];
      if constexpr (FP8) {
        const int64_t page = next_word & 0x1FFFFFFu;
        next_sk = h.scales[(page * 2) * h.heads + head];
        next_sv = h.scales[(page * 2 + 1) * h.heads + head];
      }
    };
    fetch(u0 + team);
    for (int u = u0 + team; u < u1; u += C::kTeams) {
      const int ks = f % S, kp = (f / S) & 1, vs = (f + 1) % S, vp = ((f + 1) / S) & 1;
      f += 2;
      const int seen = (int)(next_word >> 25) + 1;
      const uint32_t mask = next_mask;
      const float sk = next_sk, sv = next_sv;
      fetch(u + C::kTeams);
      if (!dead) dead = !__all_sync(0xffffffffu, wait_within(full(ks), kp, ctl, 0x402));
      if (dead) continue;
      // The common unit, of which every row sees every token, has code of its own:
      // with the others' selections in line (predicated by the compiler) a unit
      // took twice the instructions (919 a warp, then 473, with the queries still
      // as the sixteen rows).
      const bool whole = seen == kPageTokens && (mask & all_rows) == all_rows;
      if (whole) dead = !unit(std::true_type{}, ks, vs, vp, seen, mask, sk, sv);
      else dead = !unit(std::false_type{}, ks, vs, vp, seen, mask, sk, sv);
    }

    // ---- join the warps: O of each, scaled to the CTA's maximum, goes into
    // the ring, whose tiles all warps are done with at the first barrier.
    float2* stat = reinterpret_cast<float2*>(smem + C::kStatOff);
    float* red = reinterpret_cast<float*>(smem);
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
#pragma unroll
        for (int x = 4; x < 32; x *= 2) l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], x);
        if (r8 == 0) stat[warp * kTokRows + 8 * t + 2 * q4 + i] = make_float2(m[t][i], l[t][i]);
      }
    consumers_sync<32 * C::kWarps>();
#pragma unroll
    for (int t = 0; t < QT; ++t)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * t + 2 * q4 + i;
        if (row >= rows) continue;
        float top = -INFINITY;
#pragma unroll
        for (int k = 0; k < C::kWarps; ++k) top = fmaxf(top, stat[k * kTokRows + row].x);
        const float fac = ex2_approx(m[t][i] - (top == -INFINITY ? 0.f : top));
        float* dst = red + (warp * kTokRows + row) * C::kRow;
#pragma unroll
        for (int x = 0; x < C::kTiles; x += 2)
          *reinterpret_cast<float4*>(dst + tok_d<D, FP8>(x, r8)) =
              make_float4(o[t][x][i] * fac, o[t][x][2 + i] * fac, o[t][x + 1][i] * fac, o[t][x + 1][2 + i] * fac);
      }
    consumers_sync<32 * C::kWarps>();
    float* cta = reinterpret_cast<float*>(smem + C::kCtaOff);
    for (int x = threadIdx.x; x < rows * D; x += 32 * C::kWarps) {
      const int row = x / D, d = x % D;
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < C::kWarps; ++k) sum += red[(k * kTokRows + row) * C::kRow + d];
      cta[row * C::kRow + d] = sum;
    }
    if (threadIdx.x < rows) {
      float top = -INFINITY, den = 0.f;
#pragma unroll
      for (int k = 0; k < C::kWarps; ++k) top = fmaxf(top, stat[k * kTokRows + threadIdx.x].x);
#pragma unroll
      for (int k = 0; k < C::kWarps; ++k) {
        const float2 ml = stat[k * kTokRows + threadIdx.x];
        den += ml.y * ex2_approx(ml.x - (top == -INFINITY ? 0.f : top));
      }
      reinterpret_cast<float2*>(smem + C::kMlOff)[threadIdx.x] = make_float2(top, den);
    }
  }

  // ---- join the cluster's CTAs, in rank order; rank r finishes every cluster-th
  // run of columns
  __syncwarp();
  if (h.cluster > 1) cluster_sync();
  else consumers_sync<32 * C::kWarps>();
  constexpr int kWorkers = 32 * C::kWarps;
  for (int x = rank * kWorkers + threadIdx.x; x < grp.rows * D; x += h.cluster * kWorkers) {
    const int row = x / D, d = x % D;
    const uint32_t at = sb + C::kCtaOff + (uint32_t)(row * C::kRow + d) * 4, ml_at = sb + C::kMlOff + row * 8;
    float top = -INFINITY, den = 0.f, sum = 0.f;
    for (int r = 0; r < h.cluster; ++r) top = fmaxf(top, lds_rank2(ml_at, r).x);
    const float shift = top == -INFINITY ? 0.f : top;
    for (int r = 0; r < h.cluster; ++r) {
      const float2 ml = lds_rank2(ml_at, r);
      const float e = ex2_approx(ml.x - shift);
      den += e * ml.y;
      sum += e * lds_rank(at, r);
    }
    if (h.parts > 1) {
      const int64_t slot = (int64_t)(list * h.parts + part_id) * h.rows_max + row;
      h.part_o[slot * D + d] = sum;
      if (d == 0) h.part_ml[slot] = make_float2(top, den);
    } else {
      const int64_t query = grp.q0 + row / h.per_kv;
      const int qhead = head * h.per_kv + row % h.per_kv;
      const float v = den == 0.f ? 0.f : sum / den;  // 0: no token seen; NaN scores have a NaN sum
      h.o[query * h.ldo + (int64_t)qhead * D + d] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFF);
      if (h.lse && d == 0)
        h.lse[query * (h.heads * h.per_kv) + qhead] =
            den == 0.f ? -INFINITY : (top + log2f(den)) * 0.6931471805599453f;
    }
  }
  __syncwarp();
  if (h.cluster > 1) cluster_sync();  // no CTA leaves while another reads it
}

// The join of a list's parts: one warp per (query, query head).
constexpr int kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) token_join_kernel(const __grid_constant__ TokHead h,
                                                                    const int n_queries) {
  constexpr int V = D / 32;
  chain_begin();
  chain_wait();
  const int lane = threadIdx.x & 31;
  const int q_heads = h.heads * h.per_kv;
  const int at = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (at >= n_queries * q_heads) return;
  const int query = at / q_heads, qhead = at - query * q_heads;
  int g = 0;
  while (g + 1 < h.n_groups && query >= h.g[g + 1].q0) ++g;
  const int head = qhead / h.per_kv;
  const int row = (query - h.g[g].q0) * h.per_kv + qhead - head * h.per_kv;
  const int64_t base = (int64_t)(g * h.heads + head) * h.parts * h.rows_max + row;
  float mx = -INFINITY, den = 0.f, acc[V] = {};
  for (int c = 0; c < h.parts; ++c) mx = fmaxf(mx, h.part_ml[base + (int64_t)c * h.rows_max].x);
  const float shift = mx == -INFINITY ? 0.f : mx;
#pragma unroll 4
  for (int c = 0; c < h.parts; ++c) {
    const int64_t slot = base + (int64_t)c * h.rows_max;
    const float2 ml = h.part_ml[slot];
    const float e = ex2_approx(ml.x - shift);
    den += e * ml.y;
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] += e * h.part_o[slot * D + lane * V + i];
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  uint16_t* dst = h.o + query * h.ldo + (int64_t)qhead * D + lane * V;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t*>(dst + i) =
        den == 0.f ? 0u : pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
  if (h.lse && lane == 0)
    h.lse[at] = den == 0.f ? -INFINITY : (mx + log2f(den)) * 0.6931471805599453f;
}

template <int D, bool FP8, int QT, int CAP>
int launch_token(const TokParams<CAP>& p, int device, cudaStream_t s) {
  using C = TokCfg<D, FP8, QT>;
  static std::atomic<uint64_t> done{0};
  const void* fn = reinterpret_cast<const void*>(&token_attn_kernel<D, FP8, QT, CAP>);
  if (int rc = allow_shared(fn, C::kSmemBytes, device, done)) return rc;
  static std::atomic<int32_t> known{0};
  int32_t regs;
  if (int rc = wavei_kernel_registers(fn, &known, &regs)) return rc;
  // setmaxnreg.inc waits until registers are free: with fewer at launch than the
  // split assumes it would never return.
  if (D == 128 && regs < C::kRegsLaunch)
    return fail(WAVE_ERR_UNSUPPORTED, "token_attn_kernel compiled with %d registers per thread; its "
                "register split needs %d", regs, C::kRegsLaunch);
  const unsigned grid = (unsigned)(p.h.n_groups * p.h.heads * p.h.parts * p.h.cluster);
  const cudaError_t e = launch_chained(token_attn_kernel<D, FP8, QT, CAP>, dim3(grid), C::kThreads, C::kSmemBytes, s,
                                       (unsigned)p.h.cluster, p);
  if (e != cudaSuccess) return fail(WAVE_ERR_CUDA, "token_attn_kernel launch: %s", cudaGetErrorString(e));
  return WAVE_OK;
}

template <int QT, int CAP>
int launch_token_any(const wave_kv* kv, const TokParams<CAP>& p, cudaStream_t s) {
  if (kv->cfg.head_dim == 128)
    return kv->fp8 ? launch_token<128, true, QT, CAP>(p, kv->device, s) : launch_token<128, false, QT, CAP>(p, kv->device, s);
  return kv->fp8 ? launch_token<64, true, QT, CAP>(p, kv->device, s) : launch_token<64, false, QT, CAP>(p, kv->device, s);
}
template <int CAP>
int launch_token_rows(const wave_kv* kv, const TokParams<CAP>& p, cudaStream_t s) {
  return p.h.rows_max <= 8 ? launch_token_any<1>(kv, p, s) : launch_token_any<2>(kv, p, s);
}

// Lists of a call: groups of consecutive queries with their distinct items.
// kv->page_mark holds, per page, generation << 16 | index of the newest item of
// that page in the group being built (items of one page with other counts are
// chained through `prev`).
struct TokLists {
  TokParams<WAVE_MAX_TOKEN_PAGES> p;
  int32_t prev[WAVE_MAX_TOKEN_PAGES];
};

int build_lists(wave_kv* kv, const wave_node* active, int32_t n, int32_t policy,
                const int32_t* own_tokens, int32_t per_kv, TokLists& t) {
  TokHead& h = t.p.h;
  const int H = kv->cfg.heads;
  const int queries = kTokRows / per_kv;
  if ((int64_t)kv->page_mark.size() < kv->max_pages) kv->page_mark.resize(kv->max_pages, 0);
  std::vector<std::pair<int32_t, int32_t>> keys;
  int32_t items = 0, longest = 0;
  h.n_groups = 0;
  h.rows_max = 0;
  for (int32_t q0 = 0; q0 < n; q0 += queries) {
    TokGroup& g = h.g[h.n_groups++];
    const int32_t nq = std::min(queries, n - q0);
    g.q0 = q0;
    g.rows = nq * per_kv;
    g.item0 = items;
    h.rows_max = std::max(h.rows_max, g.rows);
    const int64_t gen = ++kv->mark_gen;
    for (int32_t i = 0; i < nq; ++i) {
      const wave_node node = active[q0 + i];
      if (int rc = check_query_node(kv, node)) return rc;
      if (int rc = check_history(kv, node, policy)) return rc;
      const uint16_t rows = (uint16_t)(((1u << per_kv) - 1) << (i * per_kv));
      key_entries(kv, node, policy, keys);
      for (size_t e = 0; e < keys.size(); ++e) {
        const bool own = e + 1 == keys.size();
        const int32_t want = own && own_tokens ? own_tokens[q0 + i] : -1;
        if (want < -1 || (own && own_tokens && want < 0))
          return fail(WAVE_ERR_ARG, "own_tokens[%d] is %d", q0 + i, own_tokens[q0 + i]);
        if (want == 0) continue;
        const auto it = kv->entries.find(keys[e]);
        if (it == kv->entries.end())
          return fail(WAVE_ERR_MISSING_KV, "K/V of (%d, %d) read by node (%d, %d) is not cached",
                      keys[e].first, keys[e].second, node.chunk, node.level);
        const wave_entry& ent = it->second;
        if (want > ent.ntokens)
          return fail(WAVE_ERR_ARG, "own_tokens[%d] is %d, the entry (%d, %d) holds %d", q0 + i, want,
                      keys[e].first, keys[e].second, ent.ntokens);
        const int32_t tokens = want < 0 ? ent.ntokens : want;
        for (int32_t j = 0; j * kPageTokens < tokens; ++j) {
          const int32_t page = ent.pages[j];
          const uint32_t word = (uint32_t)page |
                                (uint32_t)(std::min(kPageTokens, tokens - j * kPageTokens) - 1) << 25;
          int32_t at = kv->page_mark[page] >> 16 == gen ? (int32_t)(kv->page_mark[page] & 0xFFFF) : -1;
          const int32_t newest = at;
          while (at >= 0 && t.p.page[at] != word) at = t.prev[at];
          if (at >= 0) {
            t.p.mask[at] |= rows;
            continue;
          }
          if (items == WAVE_MAX_TOKEN_PAGES)
            return fail(WAVE_ERR_CAPACITY, "more than %d pages in one call", WAVE_MAX_TOKEN_PAGES);
          t.p.page[items] = word;
          t.p.mask[items] = rows;
          t.prev[items] = newest;
          kv->page_mark[page] = gen << 16 | items;
          ++items;
        }
      }
    }
    g.n_items = items - g.item0;
    longest = std::max(longest, g.n_items);
  }
  h.heads = H;
  h.per_kv = per_kv;
  int32_t cut[2];
  wavei_token_cut(kv->num_sms, (int64_t)h.n_groups * H, longest, cut);
  h.cluster = cut[0];
  h.parts = cut[1];
  return items;
}

// Workspace: per (list, part) slot, rows_max rows of d fp32 and (m, l).
uint64_t token_rows(const TokHead& h) {
  return h.parts > 1 ? (uint64_t)h.n_groups * h.heads * h.parts * h.rows_max : 0;
}

int token_check(const wave_kv* kv, const wave_node* active, int32_t n_active, int32_t policy,
                int32_t q_heads) {
  if (!kv) return fail(WAVE_ERR_ARG, "NULL handle");
  if (!kv->on_device) return fail(WAVE_ERR_ARG, "host-only handle (pool == NULL)");
  if (!valid_policy(policy)) return fail(WAVE_ERR_ARG, "unknown policy %d", policy);
  if (n_active < 0 || (n_active > 0 && !active)) return fail(WAVE_ERR_ARG, "bad active list");
  if (n_active > WAVE_MAX_NODES)
    return fail(WAVE_ERR_CAPACITY, "%d query tokens exceed %d", n_active, WAVE_MAX_NODES);
  if (q_heads < 1 || q_heads % kv->cfg.heads || q_heads / kv->cfg.heads > kTokRows)
    return fail(WAVE_ERR_ARG, "q_heads %d must be a multiple of the %d K/V heads, at most %d times",
                q_heads, kv->cfg.heads, kTokRows);
  return WAVE_OK;
}

thread_local TokLists t_lists;  // large: keep off the stack; launches copy it

}  // namespace
}  // namespace wavei

using namespace wavei;

extern "C" void wavei_token_cut(int32_t sms, int64_t lists, int32_t longest, int32_t* cut) {
  // Of 20 cases measured (kept under profiles/) the choice is the best of clusters of
  // 1 to 8 and of several clusters a list, or within a tenth of it.
  int32_t cluster = 1;
  double best = 1e30;
  for (int s = 1; s <= 8 && s <= std::max(1, longest); ++s) {
    // Waves of clusters; in units of an item's time at one SM's share of HBM's rate, an
    // item takes 0.6 when an SM draws all it can, more once the SMs share HBM, and
    // a wave two to start and end.
    const int64_t held = clusters_held(s, sms);
    const double waves = (double)((lists + held - 1) / held);
    const double active = (double)(std::min(lists, held) * s);
    const double t = waves * ((longest + s - 1) / s * std::max(0.6, active / sms) + 2.0);
    if (t < best) best = t, cluster = s;
  }
  cut[0] = cluster;
  cut[1] = 1;
  // Fewer than 8 long lists: several clusters each, while every CTA keeps eight
  // items. The second kernel takes 6 us: one head over 41 chunks of 4680 tokens
  // takes 25 us in 15 clusters, 108 in one; 8 lists of 71 items lose (10.8 us and 17.6).
  if (lists * 8 < 64 && longest >= 128) {
    cut[0] = 8;
    cut[1] = (int32_t)std::max<int64_t>(1, std::min<int64_t>(clusters_held(8, sms) / lists, longest / 64));
  }
}

extern "C" int wave_token_attn_workspace(wave_kv* kv, const wave_node* active, int32_t n_active,
                                         int32_t policy, const int32_t* own_tokens,
                                         int32_t q_heads, uint64_t* bytes) {
  clear_error();
  if (!bytes) return fail(WAVE_ERR_ARG, "NULL argument");
  if (int rc = token_check(kv, active, n_active, policy, q_heads)) return rc;
  *bytes = 0;
  if (n_active == 0) return WAVE_OK;
  try {
    TokLists& t = t_lists;
    const int rc = build_lists(kv, active, n_active, policy, own_tokens, q_heads / kv->cfg.heads, t);
    if (rc < 0) return rc;
    *bytes = token_rows(t.p.h) * (kv->cfg.head_dim + 2) * sizeof(float);
  } catch (const std::bad_alloc&) {
    return no_host_memory();
  }
  return WAVE_OK;
}

extern "C" int wave_token_attn(wave_kv* kv, const wave_node* active, int32_t n_active,
                               int32_t policy, const int32_t* own_tokens, int32_t q_heads,
                               const void* Q, int64_t ldq, void* O, int64_t ldo, float* lse,
                               void* workspace, uint64_t workspace_bytes, void* stream) {
  clear_error();
  if (int rc = token_check(kv, active, n_active, policy, q_heads)) return rc;
  if (n_active == 0) return WAVE_OK;
  const int D = kv->cfg.head_dim;
  if (!Q || !O || !aligned16(Q) || !aligned16(O) || (reinterpret_cast<uintptr_t>(lse) & 3))
    return fail(WAVE_ERR_ARG, "Q and O must be non-NULL and 16-byte aligned, lse 4-byte aligned");
  const int64_t row = (int64_t)q_heads * D;
  if (ldq < row || ldq % 8 || ldq >= (1LL << 40) || ldo < row || ldo % 8 || ldo >= (1LL << 40))
    return fail(WAVE_ERR_ARG, "row strides must be multiples of 8 and cover q_heads * %d", D);
  TokLists& t = t_lists;
  int items;
  try {
    items = build_lists(kv, active, n_active, policy, own_tokens, q_heads / kv->cfg.heads, t);
  } catch (const std::bad_alloc&) {
    return no_host_memory();
  }
  if (items < 0) return items;
  TokHead& h = t.p.h;
  if ((int64_t)h.n_groups * h.heads * h.parts * h.cluster >= (1LL << 31))
    return fail(WAVE_ERR_CAPACITY, "too many lists");
  const uint64_t rows = token_rows(h);
  const uint64_t need = rows * (D + 2) * sizeof(float);
  if (need > 0 && (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255)))
    return fail(WAVE_ERR_ARG, "needs a 256-byte aligned workspace of %llu bytes (got %llu)",
                (unsigned long long)need, (unsigned long long)workspace_bytes);
  if (int rc = check_current_device(kv)) return rc;
  if (kv->fp8 && !kv->codes_mapped) {
    auto encode = tensor_map_encoder();
    if (!encode) return fail(WAVE_ERR_CUDA, "cuTensorMapEncodeTiled entry point unavailable");
    cuuint64_t dims[2] = {128, (cuuint64_t)kv->max_pages * 2 * kv->cfg.heads * D};
    cuuint64_t strides[1] = {128};
    cuuint32_t box[2] = {128, (cuuint32_t)D};
    cuuint32_t estr[2] = {1, 1};
    CUresult r = encode(&kv->tm_codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2,
                        static_cast<uint8_t*>(kv->cfg.pool) + kv->data_offset, dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) return fail(WAVE_ERR_CUDA, "cuTensorMapEncodeTiled(codes) failed: %d", (int)r);
    kv->codes_mapped = true;
  }
  h.tm = kv->fp8 ? kv->tm_codes : kv->tm_kv;
  uint8_t* pool = static_cast<uint8_t*>(kv->cfg.pool);
  h.scales = kv->fp8 ? reinterpret_cast<const float*>(pool + kv->scale_offset) : nullptr;
  h.q = static_cast<const uint16_t*>(Q);
  h.o = static_cast<uint16_t*>(O);
  h.lse = lse;
  h.part_o = static_cast<float*>(workspace);
  h.part_ml = need ? reinterpret_cast<float2*>(h.part_o + rows * D) : nullptr;
  h.ldq = ldq;
  h.ldo = ldo;
  h.status = reinterpret_cast<int32_t*>(pool);
  h.wait_ns = wait_limit_ns(kv);
  h.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)D));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  int rc;
  if (items <= kTokCapSmall) {
    static thread_local TokParams<kTokCapSmall> small;
    std::memcpy(&small.h, &h, sizeof h);
    std::memcpy(small.page, t.p.page, items * sizeof(uint32_t));
    std::memcpy(small.mask, t.p.mask, items * sizeof(uint16_t));
    rc = launch_token_rows(kv, small, s);
  } else {
    rc = launch_token_rows(kv, t.p, s);
  }
  if (rc || h.parts == 1) return rc;
  const dim3 grid((unsigned)(((int64_t)n_active * q_heads + kJoinWarps - 1) / kJoinWarps));
  const cudaError_t e = D == 128 ? launch_chained(token_join_kernel<128>, grid, 32 * kJoinWarps, 0, s, 1, h, (int)n_active)
                                 : launch_chained(token_join_kernel<64>, grid, 32 * kJoinWarps, 0, s, 1, h, (int)n_active);
  if (e != cudaSuccess)
    return fail(WAVE_ERR_CUDA, "token_join_kernel launch: %s", cudaGetErrorString(e));
  return WAVE_OK;
}
