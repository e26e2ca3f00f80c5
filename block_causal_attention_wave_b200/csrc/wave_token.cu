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
//     read once. A unit is (group, head, item); the units, in that order, are
//     cut into equal runs, one per SM, wherever the cut falls. A run's part of
//     one (group, head) is a segment: a whole (group, head) goes straight to O,
//     others leave their (m, l, O') in the workspace for the join kernel.
//   - Warp 8 feeds a ring of K and V tiles by TMA (192 KB in flight per SM).
//   - Warps 0..7 take 16 of the page's 128 keys each, for all 16 rows, with
//     their own running maximum, sum and O: no exchange between warps until the
//     segment ends. S = Q K^T and O += P V are m16n8k16 MMAs on fragments read
//     from shared memory; one token fills one of 16 rows, but at a byte a cycle
//     a thread the tensor pipe idles either way, and 16 rows cost what one costs.
//   - Within an MMA the order of the contracted index is free, so a lane's
//     operand is whole 16-byte vectors of a token's row (d permuted alike in Q
//     and K; P's key order is that of S), all conflict-free under the swizzle.
//   - FP8 tiles: codes are exact in f16, so both MMAs run in f16 on converted
//     codes. Q is scaled by a power of two per row to fit f16 (its 8 bits of
//     mantissa stay exact down to 2^-24 of the row's largest value). P, in
//     [0, 1], is scaled by 2^15, so what f16 drops is below 2^-39; V's scale is
//     applied to each page's product in fp32.
//   - bf16: P is rounded to bf16 (2^-9 relative, errors of either sign over
//     many keys), as in the round's attention; sums are of the unrounded P.
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
#include <mutex>
#include <new>
#include <utility>
#include <vector>

#include "ptx.cuh"
#include "wave_internal.h"
#include "wave_sync.cuh"

using namespace wptx;

namespace wavei {
namespace {

constexpr int kTokWarps = 8;                       // consumers, 16 keys each
constexpr int kTokThreads = 32 * (kTokWarps + 1);  // and a producer warp
constexpr int kTokRows = 16;                       // query rows of a group

struct TokGroup {
  int32_t unit0;    // first unit of the group
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
  float* part_o;             // [slot][rows_max][d]
  float2* part_ml;           // [slot][rows_max]
  int64_t ldq, ldo;
  int32_t* status;
  uint64_t wait_ns;
  float scale_log2;          // log2(e) / sqrt(d)
  int32_t heads;             // K/V heads
  int32_t per_kv;            // query heads per K/V head
  int32_t n_groups;
  int32_t units;
  int32_t ctas;
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

template <int D, bool FP8>
struct TokCfg {
  static constexpr int kTile = 128 * D * (FP8 ? 1 : 2);
  static constexpr int kStage = 2 * kTile;
  static constexpr int kStages = 196608 / kStage;
  static constexpr int kRedOff = kStages * kStage;                    // [8][16][32] fp32
  static constexpr int kStatOff = kRedOff + kTokWarps * kTokRows * 32 * 4;  // [8][16] float2
  static constexpr int kBarOff = kStatOff + kTokWarps * kTokRows * 8;
  static constexpr int kSmemBytes = kBarOff + 2 * kStages * 8 + 16 + 1024;
  static constexpr int kTiles = D / 8;    // n-tiles of O
  static constexpr int kSteps = D / 16;   // k-steps of Q K^T
};

// First unit of CTA c, and the CTA that holds unit u.
__host__ __device__ __forceinline__ int tok_first(int c, int units, int ctas) {
  return (int)((int64_t)c * units / ctas);
}
__device__ __forceinline__ int tok_cta(int u, int units, int ctas) {
  return (int)((((int64_t)u + 1) * ctas - 1) / units);
}

// Walk over a CTA's units: group, head, item.
struct TokWalk {
  int g, head, item;
  __device__ __forceinline__ void start(const TokHead& p, int u) {
    g = 0;
    while (g + 1 < p.n_groups && u >= p.g[g + 1].unit0) ++g;
    const int local = u - p.g[g].unit0;
    head = local / p.g[g].n_items;
    item = local - head * p.g[g].n_items;
  }
  __device__ __forceinline__ void next(const TokHead& p) {
    if (++item < p.g[g].n_items) return;
    item = 0;
    if (++head < p.heads) return;
    head = 0;
    do ++g;
    while (g < p.n_groups && p.g[g].n_items == 0);
  }
};

template <bool F16>
__device__ __forceinline__ void tok_mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
        "{%8, %9}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

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
__device__ __forceinline__ void consumers_sync() {
  asm volatile("bar.sync 1, %0;" ::"n"(32 * kTokWarps) : "memory");
}

// d of column c (0, 1) of n-tile t in lane quarter q of O's fragment.
template <int D, bool FP8>
__device__ __forceinline__ int tok_col(int t, int q, int c) {
  if (!FP8) return 64 * (t >> 3) + 16 * q + 8 * c + (t & 7);
  return D == 128 ? 32 * q + 16 * c + t : 16 * q + 8 * c + t;
}

template <int D, bool FP8, int CAP>
__global__ void __launch_bounds__(kTokThreads, 1)
    token_attn_kernel(const __grid_constant__ TokParams<CAP> p) {
  using C = TokCfg<D, FP8>;
  constexpr int S = C::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const uint32_t sb = smem_addr(smem);
  auto full = [&](int s) -> uint32_t { return sb + C::kBarOff + 8u * s; };
  auto empty = [&](int s) -> uint32_t { return sb + C::kBarOff + 8u * (S + s); };
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::kBarOff + 16 * S);
  const TokHead& h = p.h;
  const Ctl ctl{abort_flag, h.status, h.wait_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int u0 = tok_first(blockIdx.x, h.units, h.ctas);
  const int u1 = tok_first(blockIdx.x + 1, h.units, h.ctas);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full(s), 1);
      mbar_init(empty(s), kTokWarps);
    }
    *abort_flag = 0;
    fence_mbar_init();
    prefetch_tmap(&h.tm);
  }
  __syncthreads();
  if (u0 >= u1) return;

  if (warp == kTokWarps) {
    if (lane == 0) {
      TokWalk w;
      w.start(h, u0);
      int n = 0;
      for (int u = u0; u < u1; ++u, ++n, w.next(h)) {
        const int s = n % S;
        if (n >= S && !wait_bar(empty(s), (n / S - 1) & 1, ctl, 0x401)) break;
        const int item = h.g[w.g].item0 + w.item;
        const int page = (int)(p.page[item] & 0x1FFFFFFu);
        const uint32_t dst = sb + s * C::kStage;
        mbar_arrive_expect_tx(full(s), C::kStage);
#pragma unroll
        for (int kv = 0; kv < 2; ++kv) {
          const int tile = (page * 2 + kv) * h.heads + w.head;
          if constexpr (FP8) {
            tma_load_2d(dst + kv * C::kTile, &h.tm, 0, tile * D, full(s));
          } else {
#pragma unroll
            for (int b = 0; b < D / 64; ++b)
              tma_load_2d(dst + kv * C::kTile + b * 16384, &h.tm, 64 * b, tile * 128, full(s));
          }
        }
      }
      // Copies still in flight land before the CTA exits.
      for (int k = n > S ? n - S : 0; k < n; ++k) drain_wait(full(k % S), (k / S) & 1);
    }
    return;
  }

  // ---- consumers: keys 16 warp .. 16 warp + 15 of every page
  const int r8 = lane >> 2, q4 = lane & 3;   // fragment row (and column group), lane quarter
  float o[C::kTiles][4];
  uint32_t qa[C::kSteps][4];
  float m[2], l[2], qs[2];   // rows r8 and r8 + 8: maximum (log2), this lane's sum, score factor
  float2* stat = reinterpret_cast<float2*>(smem + C::kStatOff);
  float* red = reinterpret_cast<float*>(smem + C::kRedOff);
  bool dead = false;
  TokWalk w;
  w.start(h, u0);
  float next_sk = 0.f, next_sv = 0.f;
  auto fetch_scales = [&](const TokWalk& at) {
    if constexpr (FP8) {
      const int64_t page = p.page[h.g[at.g].item0 + at.item] & 0x1FFFFFFu;
      next_sk = __ldg(h.scales + (page * 2) * h.heads + at.head);
      next_sv = __ldg(h.scales + (page * 2 + 1) * h.heads + at.head);
    }
  };
  fetch_scales(w);
  int n = 0;
  for (int u = u0; u < u1;) {
    // ---- a segment: units of one (group, head)
    const TokGroup& grp = h.g[w.g];
    const int seg_head = w.head, seg_g = w.g;
    const int seg_end = min(u1, u + grp.n_items - w.item);
    const int rows = grp.rows;
    const uint32_t all_rows = (1u << rows) - 1;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = r8 + 8 * i;
      const uint16_t* src = h.q + (grp.q0 + row / h.per_kv) * h.ldq +
                            (int64_t)(seg_head * h.per_kv + row % h.per_kv) * D;
      const bool in = row < rows;
      m[i] = -INFINITY;
      l[i] = 0.f;
      qs[i] = h.scale_log2;
      if constexpr (!FP8) {
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (in) v = *reinterpret_cast<const uint4*>(src + 64 * b + 8 * (2 * q4 + hh));
            const int st = (b * 2 + hh) * 2;
            qa[st][i] = v.x;
            qa[st][2 + i] = v.y;
            qa[st + 1][i] = v.z;
            qa[st + 1][2 + i] = v.w;
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
        qs[i] *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int st = 0; st < C::kSteps; ++st)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t v = raw[st * 2 + j];
            qa[st][2 * j + i] = pack_f16x2(__uint_as_float(v << 16) * up,
                                           __uint_as_float(v & 0xFFFF0000u) * up);
          }
      }
    }
#pragma unroll
    for (int t = 0; t < C::kTiles; ++t)
#pragma unroll
      for (int c = 0; c < 4; ++c) o[t][c] = 0.f;

    for (; u < seg_end; ++u, ++n) {
      const int s = n % S;
      const int item = grp.item0 + w.item;
      const int seen = (int)(p.page[item] >> 25) + 1;
      const uint32_t mask = p.mask[item];
      const float sk = next_sk, sv = next_sv;
      w.next(h);
      if (FP8 && u + 1 < u1) fetch_scales(w);
      if (!dead) dead = !__all_sync(0xffffffffu, wait_bar(full(s), (n / S) & 1, ctl, 0x402));
      if (dead) continue;
      const int key0 = 16 * warp;
      if (key0 < seen) {
        const uint32_t kt = sb + s * C::kStage, vt = kt + C::kTile;
        float sc[2][4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[nt][c] = 0.f;
        if constexpr (!FP8) {
#pragma unroll
          for (int b = 0; b < D / 64; ++b)
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
              for (int nt = 0; nt < 2; ++nt) {
                const uint32_t row = kt + b * 16384 + (key0 + nt * 8 + r8) * 128;
                const uint4 v = lds128(row + (((2 * q4 + hh) ^ r8) << 4));
                const int st = (b * 2 + hh) * 2;
                tok_mma<false>(sc[nt], qa[st], v.x, v.y);
                tok_mma<false>(sc[nt], qa[st + 1], v.z, v.w);
              }
        } else {
#pragma unroll
          for (int hh = 0; hh < D / 64; ++hh)
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
              const int key = key0 + nt * 8 + r8;
              const int line = D == 128 ? key : key >> 1;
              const int chunk = D == 128 ? 2 * q4 + hh : (key & 1) * 4 + q4;
              const uint4 v = lds128(kt + line * 128 + ((chunk ^ (line & 7)) << 4));
              const uint32_t wd[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
              for (int j = 0; j < 4; ++j)
                tok_mma<true>(sc[nt], qa[hh * 4 + j], e4m3_f16x2(wd[j] & 0xFFFF), e4m3_f16x2(wd[j] >> 16));
            }
        }
        // ---- softmax of this warp's 16 keys; rows r8 (c = 0, 1) and r8 + 8 (c = 2, 3)
        const bool part[2] = {(mask >> r8 & 1) != 0, (mask >> (r8 + 8) & 1) != 0};
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const int key = key0 + nt * 8 + 2 * q4 + (c & 1);
            const float f = FP8 ? qs[c >> 1] * sk : qs[c >> 1];
            sc[nt][c] = part[c >> 1] && key < seen ? sc[nt][c] * f : -INFINITY;
            top[c >> 1] = fmaxf(top[c >> 1], sc[nt][c]);
          }
        bool grew = false;
        float shift[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
          top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
          top[i] = fmaxf(top[i], m[i]);
          grew |= top[i] > m[i];
          shift[i] = top[i] == -INFINITY ? 0.f : top[i];
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float f = ex2_approx(m[i] - shift[i]);
            if (top[i] > m[i]) {
              l[i] *= f;
              m[i] = top[i];
#pragma unroll
              for (int t = 0; t < C::kTiles; ++t) {
                o[t][2 * i] *= f;
                o[t][2 * i + 1] *= f;
              }
            }
          }
        }
        uint32_t pa[4];
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float a = ex2_approx(sc[nt][2 * i] - shift[i]);
            const float b = ex2_approx(sc[nt][2 * i + 1] - shift[i]);
            l[i] += a + b;
            pa[2 * nt + i] = FP8 ? pack_f16x2(a * 32768.f, b * 32768.f) : pack_bf16x2(a, b);
          }
        // ---- O += P V: keys 2 q4, + 1, + 8, + 9 of the warp's sixteen
        const bool partial = seen < key0 + 16;
        const bool mixed = (mask & all_rows) != all_rows;
        bool live[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) live[k] = key0 + 2 * q4 + (k & 1) + 8 * (k >> 1) < seen;
        if constexpr (!FP8) {
#pragma unroll
          for (int b = 0; b < D / 64; ++b) {
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const int key = key0 + 2 * q4 + (k & 1) + 8 * (k >> 1);
              v[k] = lds128(vt + b * 16384 + key * 128 + ((r8 ^ (key & 7)) << 4));
              if (partial && !live[k]) v[k] = make_uint4(0, 0, 0, 0);
            }
            const uint32_t x[4][4] = {{v[0].x, v[0].y, v[0].z, v[0].w}, {v[1].x, v[1].y, v[1].z, v[1].w},
                                      {v[2].x, v[2].y, v[2].z, v[2].w}, {v[3].x, v[3].y, v[3].z, v[3].w}};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              const uint32_t sel = e & 1 ? 0x7632 : 0x5410;
              const uint32_t b0 = __byte_perm(x[0][e >> 1], x[1][e >> 1], sel);
              const uint32_t b1 = __byte_perm(x[2][e >> 1], x[3][e >> 1], sel);
              float (&acc)[4] = o[b * 8 + e];
              if (!mixed) {
                tok_mma<false>(acc, pa, b0, b1);
              } else {
                float d[4] = {acc[0], acc[1], acc[2], acc[3]};
                tok_mma<false>(d, pa, b0, b1);
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[c] = part[c >> 1] ? d[c] : acc[c];
              }
            }
          }
        } else {
          const float f = sv * 0x1p-15f;
          uint32_t x[4][D / 32];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int key = key0 + 2 * q4 + (k & 1) + 8 * (k >> 1);
            if constexpr (D == 128) {
              const uint4 v = lds128(vt + key * 128 + ((r8 ^ (key & 7)) << 4));
              x[k][0] = v.x; x[k][1] = v.y; x[k][2] = v.z; x[k][3] = v.w;
            } else {
              const int line = key >> 1, chunk = (key & 1) * 4 + (r8 >> 1);
              const uint2 v = lds64(vt + line * 128 + ((chunk ^ (line & 7)) << 4) + (r8 & 1) * 8);
              x[k][0] = v.x; x[k][1] = v.y;
            }
            if (partial && !live[k]) {
#pragma unroll
              for (int j = 0; j < D / 32; ++j) x[k][j] = 0;
            }
          }
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              // codes of d 4 j + 2 half (low 16 bits) and the next: keys (0, 1) and (8, 9)
              const uint32_t sel = half ? 0x7362 : 0x5140;
              const uint32_t k01 = __byte_perm(x[0][j], x[1][j], sel);
              const uint32_t k89 = __byte_perm(x[2][j], x[3][j], sel);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                float d[4] = {0.f, 0.f, 0.f, 0.f};
                tok_mma<true>(d, pa, e4m3_f16x2(e ? k01 >> 16 : k01 & 0xFFFF),
                              e4m3_f16x2(e ? k89 >> 16 : k89 & 0xFFFF));
                float (&acc)[4] = o[4 * j + 2 * half + e];
#pragma unroll
                for (int c = 0; c < 4; ++c) acc[c] = part[c >> 1] ? fmaf(f, d[c], acc[c]) : acc[c];
              }
            }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty(s));
    }

    // ---- segment end: join the eight warps
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
      if (q4 == 0) stat[warp * kTokRows + r8 + 8 * i] = make_float2(m[i], l[i]);
    }
    consumers_sync();
    float f[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float top = -INFINITY;
#pragma unroll
      for (int k = 0; k < kTokWarps; ++k) top = fmaxf(top, stat[k * kTokRows + r8 + 8 * i].x);
      f[i] = ex2_approx(m[i] - (top == -INFINITY ? 0.f : top));
    }
    const int gh = seg_g * h.heads + seg_head;
    const int list0 = grp.unit0 + seg_head * grp.n_items;
    const bool whole = u0 <= list0 && list0 + grp.n_items <= u1;
    const int64_t slot = (int64_t)(blockIdx.x + gh) * h.rows_max;
    // 32 columns (4 n-tiles) at a time; thread: row threadIdx.x / 16, columns x, x + 16.
    const int row = threadIdx.x >> 4;
    float top = -INFINITY, den = 0.f;
    if (row < rows) {
#pragma unroll
      for (int k = 0; k < kTokWarps; ++k) top = fmaxf(top, stat[k * kTokRows + row].x);
#pragma unroll
      for (int k = 0; k < kTokWarps; ++k) {
        const float2 ml = stat[k * kTokRows + row];
        den += ml.y * ex2_approx(ml.x - (top == -INFINITY ? 0.f : top));
      }
    }
    const int64_t query = grp.q0 + row / h.per_kv;
    const int qhead = seg_head * h.per_kv + row % h.per_kv;
    const float inv = top == -INFINITY ? 0.f : 1.f / den;
#pragma unroll
    for (int blk = 0; blk < C::kTiles / 4; ++blk) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (r8 + 8 * i >= rows) continue;
        float* dst = red + (warp * kTokRows + r8 + 8 * i) * 32 + q4 * 8;
#pragma unroll
        for (int tt = 0; tt < 4; ++tt)
#pragma unroll
          for (int c = 0; c < 2; ++c) dst[tt * 2 + c] = o[blk * 4 + tt][2 * i + c] * f[i];
      }
      consumers_sync();
      if (row < rows) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int x = (threadIdx.x & 15) + 16 * j;
          float sum = 0.f;
#pragma unroll
          for (int k = 0; k < kTokWarps; ++k) sum += red[(k * kTokRows + row) * 32 + x];
          const int d = tok_col<D, FP8>(blk * 4 + ((x >> 1) & 3), x >> 3, x & 1);
          if (whole) {
            const float v = top == -INFINITY ? 0.f : sum * inv;
            h.o[query * h.ldo + (int64_t)qhead * D + d] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFF);
          } else {
            h.part_o[(slot + row) * D + d] = sum;
          }
        }
      }
      consumers_sync();
    }
    if (row < rows && (threadIdx.x & 15) == 0) {
      if (!whole)
        h.part_ml[slot + row] = make_float2(top, den);
      else if (h.lse)
        h.lse[query * (h.heads * h.per_kv) + qhead] =
            top == -INFINITY ? -INFINITY : (top + log2f(den)) * 0.6931471805599453f;
    }
  }
}

// The join: one warp per (query, query head). Lists that one CTA held whole are
// done already; lists of no item give zeros.
constexpr int kJoinWarps = 4;
template <int D>
__global__ void __launch_bounds__(32 * kJoinWarps) token_join_kernel(const __grid_constant__ TokHead h,
                                                                    const int n_queries) {
  constexpr int V = D / 32;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int q_heads = h.heads * h.per_kv;
  const int at = blockIdx.x * kJoinWarps + (threadIdx.x >> 5);
  if (at >= n_queries * q_heads) return;
  const int query = at / q_heads, qhead = at - query * q_heads;
  int g = 0;
  while (g + 1 < h.n_groups && query >= h.g[g + 1].q0) ++g;
  const TokGroup& grp = h.g[g];
  const int head = qhead / h.per_kv;
  const int row = (query - grp.q0) * h.per_kv + qhead - head * h.per_kv;
  uint16_t* dst = h.o + query * h.ldo + (int64_t)qhead * D + lane * V;
  float acc[V] = {};
  float mx = -INFINITY, den = 0.f;
  if (grp.n_items > 0) {
    const int first = grp.unit0 + head * grp.n_items;
    const int c0 = tok_cta(first, h.units, h.ctas), c1 = tok_cta(first + grp.n_items - 1, h.units, h.ctas);
    if (c0 == c1) return;
    const int64_t base = (int64_t)(g * h.heads + head) * h.rows_max + row;
    for (int c = c0 + lane; c <= c1; c += 32)
      mx = fmaxf(mx, h.part_ml[base + (int64_t)c * h.rows_max].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    const float shift = mx == -INFINITY ? 0.f : mx;
#pragma unroll 8
    for (int c = c0; c <= c1; ++c) {
      const int64_t slot = base + (int64_t)c * h.rows_max;
      const float2 ml = h.part_ml[slot];
      const float e = exp2f(ml.x - shift);
      den += e * ml.y;
      const float* po = h.part_o + slot * D + lane * V;
#pragma unroll
      for (int i = 0; i < V; ++i) acc[i] += e * po[i];
    }
  }
  const float inv = mx == -INFINITY ? 0.f : 1.f / den;
#pragma unroll
  for (int i = 0; i < V; i += 2)
    *reinterpret_cast<uint32_t*>(dst + i) =
        mx == -INFINITY ? 0u : pack_bf16x2(acc[i] * inv, acc[i + 1] * inv);
  if (h.lse && lane == 0)
    h.lse[at] = mx == -INFINITY ? -INFINITY : (mx + log2f(den)) * 0.6931471805599453f;
}

template <int D, bool FP8, int CAP>
int launch_token(const TokParams<CAP>& p, cudaStream_t s) {
  using C = TokCfg<D, FP8>;
  static std::once_flag once;
  static cudaError_t attr_err = cudaSuccess;
  std::call_once(once, [] {
    attr_err = cudaFuncSetAttribute(token_attn_kernel<D, FP8, CAP>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  });
  if (attr_err != cudaSuccess)
    return fail(WAVE_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(attr_err));
  token_attn_kernel<D, FP8, CAP><<<p.h.ctas, kTokThreads, C::kSmemBytes, s>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return fail(WAVE_ERR_CUDA, "token_attn_kernel launch: %s", cudaGetErrorString(e));
  return WAVE_OK;
}

template <int CAP>
int launch_token_any(const wave_kv* kv, const TokParams<CAP>& p, cudaStream_t s) {
  if (kv->cfg.head_dim == 128)
    return kv->fp8 ? launch_token<128, true, CAP>(p, s) : launch_token<128, false, CAP>(p, s);
  return kv->fp8 ? launch_token<64, true, CAP>(p, s) : launch_token<64, false, CAP>(p, s);
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
  int32_t items = 0;
  int64_t units = 0;
  h.n_groups = 0;
  h.rows_max = 0;
  for (int32_t q0 = 0; q0 < n; q0 += queries) {
    TokGroup& g = h.g[h.n_groups++];
    const int32_t nq = std::min(queries, n - q0);
    g.q0 = q0;
    g.rows = nq * per_kv;
    g.item0 = items;
    g.unit0 = (int32_t)units;
    h.rows_max = std::max(h.rows_max, g.rows);
    const int64_t gen = ++kv->mark_gen;
    for (int32_t i = 0; i < nq; ++i) {
      const wave_node node = active[q0 + i];
      if (int rc = check_query_node(kv, node)) return rc;
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
    units += (int64_t)g.n_items * H;
    if (units >= (1LL << 30)) return fail(WAVE_ERR_CAPACITY, "too many work units");
  }
  h.heads = H;
  h.per_kv = per_kv;
  h.units = (int32_t)units;
  h.ctas = (int32_t)std::min<int64_t>(units, kv->num_sms);
  return items;
}

bool join_needed(const TokHead& h) {
  // Some group without items (its rows are zeroed there), or some (group,
  // head) that two CTAs share.
  for (int g = 0; g < h.n_groups; ++g) {
    const TokGroup& gr = h.g[g];
    if (gr.n_items == 0) return true;
    for (int head = 0; head < h.heads; ++head) {
      const int64_t a = gr.unit0 + (int64_t)head * gr.n_items, b = a + gr.n_items - 1;
      if (((a + 1) * h.ctas - 1) / h.units != ((b + 1) * h.ctas - 1) / h.units) return true;
    }
  }
  return false;
}

// Workspace: per (CTA, group, head) slot, rows_max rows of d fp32 and (m, l).
uint64_t token_slots(const TokHead& h) { return (uint64_t)h.ctas + (uint64_t)h.n_groups * h.heads; }

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
    if (t.p.h.units > 0 && join_needed(t.p.h))
      *bytes = token_slots(t.p.h) * t.p.h.rows_max * (kv->cfg.head_dim + 2) * sizeof(float);
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
  const bool join = join_needed(h);
  const uint64_t slots = token_slots(h) * h.rows_max;
  if (join && h.units > 0) {
    const uint64_t need = slots * (D + 2) * sizeof(float);
    if (!workspace || workspace_bytes < need || (reinterpret_cast<uintptr_t>(workspace) & 255))
      return fail(WAVE_ERR_ARG, "needs a 256-byte aligned workspace of %llu bytes (got %llu)",
                  (unsigned long long)need, (unsigned long long)workspace_bytes);
  }
  if (int rc = check_current_device(kv)) return rc;
  h.tm = kv->tm_kv;
  uint8_t* pool = static_cast<uint8_t*>(kv->cfg.pool);
  h.scales = kv->fp8 ? reinterpret_cast<const float*>(pool + kv->scale_offset) : nullptr;
  h.q = static_cast<const uint16_t*>(Q);
  h.o = static_cast<uint16_t*>(O);
  h.lse = lse;
  h.part_o = static_cast<float*>(workspace);
  h.part_ml = reinterpret_cast<float2*>(h.part_o + slots * D);
  h.ldq = ldq;
  h.ldo = ldo;
  h.status = reinterpret_cast<int32_t*>(pool);
  h.wait_ns = wait_limit_ns(kv);
  h.scale_log2 = (float)(1.4426950408889634 / std::sqrt((double)D));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (h.units > 0) {
    int rc;
    if (items <= kTokCapSmall) {
      static thread_local TokParams<kTokCapSmall> small;
      std::memcpy(&small.h, &h, sizeof h);
      std::memcpy(small.page, t.p.page, items * sizeof(uint32_t));
      std::memcpy(small.mask, t.p.mask, items * sizeof(uint16_t));
      rc = launch_token_any(kv, small, s);
    } else {
      rc = launch_token_any(kv, t.p, s);
    }
    if (rc) return rc;
  }
  if (!join) return WAVE_OK;
  // The join may be launched while the first kernel runs (its blocks wait for
  // it to finish): the launch's latency is hidden behind the first kernel.
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(((int64_t)n_active * q_heads + kJoinWarps - 1) / kJoinWarps));
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = h.units > 0 ? 1 : 0;
  cudaError_t e = D == 128 ? cudaLaunchKernelEx(&cfg, token_join_kernel<128>, h, (int)n_active)
                           : cudaLaunchKernelEx(&cfg, token_join_kernel<64>, h, (int)n_active);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(WAVE_ERR_CUDA, "token_join_kernel launch: %s", cudaGetErrorString(e));
  }
  return WAVE_OK;
}
