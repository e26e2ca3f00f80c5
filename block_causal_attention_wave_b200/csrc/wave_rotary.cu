// Rotary embedding of tokens at positions of their own.
//
// What it computes: the rotation that the round projection fuses for whole
// chunks (see wave_gemm.cu), for any token: pair (a, b) of a head becomes
// (a cos t - b sin t, a sin t + b cos t), t = position[axis] * frequency.
//
// The angle: a pair turns by f = frequency / (2 pi) turns a position step, f
// in (0, 0.16]. The host keeps f as a 64-bit fraction of a turn, and position *
// f modulo one turn is a 64-bit product that wraps: exact for every int32
// position, where a float32 angle is off by 2^-24 of itself (0.06 rad at a
// million). The upper 32 bits, as a signed fraction of half a turn, go to
// sincospif.
//
// What bounds it: HBM. A thread owns 16 bytes of a head (or 16 + 16 where the
// partner sits d/2 away), works its sines and cosines out once and takes them
// through several heads, whose loads are all in flight before the first store.
// 18720 rows of 12 + 12 heads of 128 (230 MB): 37.6 us back to back, 6.1 TB/s, 0.93 of a
// plain copy's rate (39.5 us with inputs of which L2 holds nothing); with load and store in
// turn a fifth more.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "ptx.cuh"
#include "wave_internal.h"
#include "wave_wait.cuh"

namespace wavei {
namespace {

constexpr int kRotaryThreads = 128;

struct RotaryParams {
  const int32_t* pos;        // [rows][3]
  const uint16_t* x[2];      // Q, K
  uint16_t* y[2];
  int64_t ldx[2], ldy[2];    // row strides in elements
  int32_t q_heads, heads;    // heads of Q; of Q and K together
  int32_t rows;
  int32_t heads_per_thread;
  uint64_t turn[64];         // turns per position step, in 2^-64 turns; 0: pair is copied
  int8_t axis[64];
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

template <int D, bool HALVES>
__global__ void __launch_bounds__(kRotaryThreads) rotary_kernel(const __grid_constant__ RotaryParams p,
                                                               const float sign) {
  constexpr int kPairs = HALVES ? 8 : 4;            // pairs of one thread
  constexpr int kLanes = D / 2 / kPairs;            // threads of one row
  chain_begin();
  __shared__ uint64_t turn[D / 2];
  __shared__ int8_t axis[D / 2];
  if (threadIdx.x < D / 2) {
    turn[threadIdx.x] = p.turn[threadIdx.x];
    axis[threadIdx.x] = p.axis[threadIdx.x];
  }
  __syncthreads();
  const int64_t at = (int64_t)blockIdx.x * kRotaryThreads + threadIdx.x;
  const int64_t row = at / kLanes;
  const int v = (int)(at % kLanes);
  if (row >= p.rows) return;
  chain_wait();
  float cs[kPairs], sn[kPairs];
  uint32_t copied = 0;
  {
    const int32_t* ps = p.pos + row * 3;
    const int32_t where[3] = {ps[0], ps[1], ps[2]};
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      const int pr = v * kPairs + i;
      const int ax = axis[pr];
      const int64_t w = ax == 0 ? where[0] : ax == 1 ? where[1] : where[2];
      const uint64_t t = turn[pr];
      const uint64_t angle = (uint64_t)w * t;  // modulo one turn
      sincospif((float)(int32_t)(angle >> 32) * 0x1p-31f, &sn[i], &cs[i]);
      sn[i] *= sign;
      if (t == 0) copied |= 1u << i;
    }
  }
  // Heads in batches whose loads are all issued before the first store (which the
  // compiler may not do, since the outputs may be the inputs).
  constexpr int kBatch = HALVES ? 4 : 8;
  const int h0 = blockIdx.y * p.heads_per_thread;
  const int h1 = min(p.heads, h0 + p.heads_per_thread);
  const uint16_t* x[2] = {p.x[0] + row * p.ldx[0] + v * 8,
                          p.x[1] + row * p.ldx[1] + v * 8 - p.q_heads * D};
  uint16_t* y[2] = {p.y[0] + row * p.ldy[0] + v * 8, p.y[1] + row * p.ldy[1] + v * 8 - p.q_heads * D};
  for (int hb = h0; hb < h1; hb += kBatch) {
    uint4 in[kBatch], hi[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = hb + j;
      if (h >= h1) break;
      const uint16_t* src = (h < p.q_heads ? x[0] : x[1]) + h * D;
      in[j] = *reinterpret_cast<const uint4*>(src);
      if constexpr (HALVES) hi[j] = *reinterpret_cast<const uint4*>(src + D / 2);
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = hb + j;
      if (h >= h1) break;
      uint16_t* dst = (h < p.q_heads ? y[0] : y[1]) + h * D;
      const uint32_t a[4] = {in[j].x, in[j].y, in[j].z, in[j].w};
      if constexpr (HALVES) {
        const uint32_t b[4] = {hi[j].x, hi[j].y, hi[j].z, hi[j].w};
        uint32_t oa[4], ob[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float ra[2], rb[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const float fa = e ? bf16_hi(a[i]) : bf16_lo(a[i]), fb = e ? bf16_hi(b[i]) : bf16_lo(b[i]);
            const float c = cs[2 * i + e], s = sn[2 * i + e];
            const bool keep = copied >> (2 * i + e) & 1;
            ra[e] = keep ? fa : fa * c - fb * s;
            rb[e] = keep ? fb : fa * s + fb * c;
          }
          oa[i] = wptx::pack_bf16x2(ra[0], ra[1]);
          ob[i] = wptx::pack_bf16x2(rb[0], rb[1]);
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(oa[0], oa[1], oa[2], oa[3]);
        *reinterpret_cast<uint4*>(dst + D / 2) = make_uint4(ob[0], ob[1], ob[2], ob[3]);
      } else {
        uint32_t o[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float fa = bf16_lo(a[i]), fb = bf16_hi(a[i]);
          const bool keep = copied >> i & 1;
          o[i] = wptx::pack_bf16x2(keep ? fa : fa * cs[i] - fb * sn[i],
                                   keep ? fb : fa * sn[i] + fb * cs[i]);
        }
        *reinterpret_cast<uint4*>(dst) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

template <int D, bool HALVES>
cudaError_t launch_rotary(const RotaryParams& p, float sign, cudaStream_t s) {
  constexpr int kLanes = D / 2 / (HALVES ? 8 : 4);
  const int64_t blocks = ((int64_t)p.rows * kLanes + kRotaryThreads - 1) / kRotaryThreads;
  const int groups = (p.heads + p.heads_per_thread - 1) / p.heads_per_thread;
  return launch_chained(rotary_kernel<D, HALVES>, dim3((unsigned)blocks, (unsigned)groups), kRotaryThreads, 0, s, 1, p,
                        sign);
}

// The pairs' turns and axes. The last spec's are kept: working them out takes a
// microsecond, a third of the call.
void turns_of(const wave_rotary_spec& spec, int D, RotaryParams& p) {
  static thread_local struct {
    wave_rotary_spec spec;
    int D = 0;
    uint64_t turn[64];
    int8_t axis[64];
  } last;
  if (last.D == D && std::memcmp(&last.spec, &spec, sizeof spec) == 0) {
    std::memcpy(p.turn, last.turn, sizeof p.turn);
    std::memcpy(p.axis, last.axis, sizeof p.axis);
    return;
  }
  const int32_t* n = spec.pairs;
  // Frequencies by running products in 64-bit mantissas: after 64 steps off by
  // 2^-58 of themselves, 2^-29 turns at the farthest position.
  int pr = 0;
  long double freq = 1.0L;
  const bool one_ladder = spec.ladder == WAVE_ROTARY_LADDER;
  long double step = one_ladder ? powl((long double)spec.base, -2.0L / D) : 1.0L;
  for (int axis = 0; axis < 3; ++axis) {
    if (!one_ladder) {
      freq = 1.0L;
      if (n[axis] > 1) step = powl((long double)spec.base, -1.0L / n[axis]);
    }
    for (int i = 0; i < n[axis]; ++i, ++pr, freq *= step) {
      // freq / (2 pi), as a 64-bit fraction of a turn; at least one unit, so a
      // pair that turns is told from one that is copied.
      constexpr long double kUnits = 18446744073709551616.0L / 6.283185307179586476925286766559L;
      p.turn[pr] = std::max<uint64_t>(1, (uint64_t)(freq * kUnits + 0.5L));
      p.axis[pr] = (int8_t)axis;
    }
  }
  last.spec = spec;
  last.D = D;
  std::memcpy(last.turn, p.turn, sizeof p.turn);
  std::memcpy(last.axis, p.axis, sizeof p.axis);
}

bool stride_ok(int64_t ld, int64_t row) { return ld >= row && ld % 8 == 0 && ld < (1LL << 40); }

}  // namespace
}  // namespace wavei

using namespace wavei;

extern "C" int wave_rotary(wave_kv* kv, const wave_rotary_spec* spec, const int32_t* positions,
                           int32_t rows, const void* Q, int64_t ldq, int32_t q_heads, void* Qout,
                           int64_t ldqo, const void* K, int64_t ldk, int32_t k_heads, void* Kout,
                           int64_t ldko, void* stream) {
  clear_error();
  if (!kv) return fail(WAVE_ERR_ARG, "NULL handle");
  if (!kv->on_device) return fail(WAVE_ERR_ARG, "host-only handle (pool == NULL) cannot launch");
  const int D = kv->cfg.head_dim;
  if (!spec) return fail(WAVE_ERR_ARG, "NULL spec");
  const int32_t* n = spec->pairs;
  if (n[0] < 0 || n[1] < 0 || n[2] < 0 || (int64_t)n[0] + n[1] + n[2] > D / 2)
    return fail(WAVE_ERR_ARG, "pairs %d + %d + %d must be >= 0 and at most %d together", n[0], n[1],
                n[2], D / 2);
  if (!(spec->base > 1.f) || !std::isfinite(spec->base))
    return fail(WAVE_ERR_ARG, "base must be finite and > 1");
  if ((spec->layout != WAVE_ROTARY_INTERLEAVED && spec->layout != WAVE_ROTARY_HALVES) ||
      (spec->ladder != WAVE_ROTARY_PER_AXIS && spec->ladder != WAVE_ROTARY_LADDER) ||
      (spec->inverse != 0 && spec->inverse != 1))
    return fail(WAVE_ERR_ARG, "unknown layout %d, ladder %d or inverse %d", spec->layout,
                spec->ladder, spec->inverse);
  if (rows < 0) return fail(WAVE_ERR_ARG, "rows must be >= 0, got %d", rows);
  if (!K) k_heads = 0;
  if (q_heads < 1 || q_heads > (1 << 16) || (K && (k_heads < 1 || k_heads > (1 << 16))))
    return fail(WAVE_ERR_ARG, "need 1..65536 heads, got %d of Q and %d of K", q_heads, k_heads);
  if (rows == 0) return WAVE_OK;
  if (!positions || (reinterpret_cast<uintptr_t>(positions) & 3))
    return fail(WAVE_ERR_ARG, "positions must be non-NULL and 4-byte aligned");
  if (!Q || !Qout || !aligned16(Q) || !aligned16(Qout) ||
      (K && (!Kout || !aligned16(K) || !aligned16(Kout))))
    return fail(WAVE_ERR_ARG, "Q, Qout (and K, Kout) must be non-NULL and 16-byte aligned");
  if (!stride_ok(ldq, (int64_t)q_heads * D) || !stride_ok(ldqo, (int64_t)q_heads * D) ||
      (K && (!stride_ok(ldk, (int64_t)k_heads * D) || !stride_ok(ldko, (int64_t)k_heads * D))))
    return fail(WAVE_ERR_ARG, "row strides must be multiples of 8 and cover heads * %d", D);
  if ((Q == Qout && ldq != ldqo) || (K && K == Kout && ldk != ldko))
    return fail(WAVE_ERR_ARG, "a rotation in place needs equal strides");
  if (int rc = check_current_device(kv)) return rc;

  RotaryParams p;
  std::memset(&p, 0, sizeof p);
  p.pos = positions;
  p.x[0] = static_cast<const uint16_t*>(Q);
  p.y[0] = static_cast<uint16_t*>(Qout);
  p.ldx[0] = ldq;
  p.ldy[0] = ldqo;
  p.x[1] = static_cast<const uint16_t*>(K);
  p.y[1] = static_cast<uint16_t*>(Kout);
  p.ldx[1] = ldk;
  p.ldy[1] = ldko;
  p.q_heads = q_heads;
  p.heads = q_heads + k_heads;
  p.rows = rows;
  turns_of(*spec, D, p);
  // A thread takes its angles through as many heads as leave the GPU about four
  // blocks per SM, at most one batch (us, in a graph, inputs from HBM: 18720 rows of
  // 12 + 12 heads of 128: 4 heads a thread 45.5, 8 39.5, 24 40.3; 984 rows of 24 + 24
  // heads of 64, halves: 1 8.3, 3 4.8, 8 6.3).
  const int lanes = D / 2 / (spec->layout == WAVE_ROTARY_HALVES ? 8 : 4);
  const int64_t row_blocks = ((int64_t)rows * lanes + kRotaryThreads - 1) / kRotaryThreads;
  const int64_t groups = std::min<int64_t>(p.heads, (4LL * kv->num_sms + row_blocks - 1) / row_blocks);
  p.heads_per_thread = (int)std::min<int64_t>(8, (p.heads + groups - 1) / groups);
  const float sign = spec->inverse ? -1.f : 1.f;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool halves = spec->layout == WAVE_ROTARY_HALVES;
  const cudaError_t e = D == 128 ? (halves ? launch_rotary<128, true>(p, sign, s) : launch_rotary<128, false>(p, sign, s))
                                 : (halves ? launch_rotary<64, true>(p, sign, s) : launch_rotary<64, false>(p, sign, s));
  if (e != cudaSuccess) return fail(WAVE_ERR_CUDA, "rotary_kernel launch: %s", cudaGetErrorString(e));
  return WAVE_OK;
}
