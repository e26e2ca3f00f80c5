// What the dense layers' kernels share: activations, their arguments, and the
// tensor map of a K-major operand.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "ptx.cuh"
#include "wave.h"

namespace wavei {

// C += A B on registers, 16 x 8 x 16, f16 or bf16.
template <bool F16>
__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
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

// GELU, tanh form, through 0.5 (1 + tanh u) = 1 / (1 + e^(-2u)): one
// exponential and one division on the special-function unit, with relative
// accuracy everywhere (the tail where 1 + tanh u is tiny included).
__device__ __forceinline__ float gelu_tanh(float x) {
  const float u = 0.7978845608028654f * fmaf(0.044715f * x, x * x, x);
  return __fdividef(x, 1.f + __expf(-2.f * u));
}

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The activations of wave_linear_bias, written for the epilogue's instruction
// count (18720 x 1536 x 8960, sustained, us: none 402, tanh-GELU 417, SiLU 408, erf-GELU
// 455; tanh-GELU by the form above was 32 us slower than by this one):
// - tanh-GELU and SiLU are x / (1 + 2^w) with w folded into one polynomial;
// - erf-GELU is x (1 - E / 2) or, for x < 0, x E / 2, with E = erfc(|x| / sqrt 2).
//   The second needs E's relative accuracy: E = e^(-x^2 / 2) t P(t), t = 1 / (1 +
//   0.375 z), z = |x| / sqrt 2, P of degree 6 fitted to t P(t) = e^(z^2) erfc(z) over
//   0 <= z <= 9.6 with the least largest relative error (6.4e-7; with float32's
//   roundings 2.1e-6 up to |x| = 5 and 2^-16 to the end).
// An infinite 2^w gives a reciprocal of zero.
template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == WAVE_ACT_GELU_TANH) {
    // w = -2 log2(e) sqrt(2 / pi) (x + 0.044715 x^3)
    const float w = x * fmaf(x * x, -2.302208198f * 0.044715f, -2.302208198f);
    return x * rcp_approx(1.f + wptx::ex2_approx(w));
  }
  if constexpr (ACT == WAVE_ACT_SILU) return x * rcp_approx(1.f + wptx::ex2_approx(-1.442695041f * x));
  if constexpr (ACT == WAVE_ACT_GELU_ERF) {
    const float t = rcp_approx(fmaf(0.375f * 0.7071067812f, fabsf(x), 1.f));
    float e = fmaf(-0.135095909f, t, 0.387937844f);
    e = fmaf(e, t, -0.129597321f);
    e = fmaf(e, t, 0.283061564f);
    e = fmaf(e, t, 0.166664556f);
    e = fmaf(e, t, 0.215689182f);
    e = fmaf(e, t, 0.211339444f);
    const float h = 0.5f * x * (e * t * wptx::ex2_approx(x * x * -0.7213475204f));
    return x < 0.f ? h : x < 16.f ? x - h : x;  // from 16 on h is less than half a step; at infinity, NaN
  }
  return x;
}

// Bias and residual of eight columns of a row, fetched ahead of their use (a trip
// to L2 is as long as a tile's 32 columns take): P has bias, resid, ldr, y, ldy
// and wide (y and ldy allow 32-byte stores).
struct Eight {
  uint4 b, r;
};
template <class P>
__device__ __forceinline__ Eight fetch8(const P& p, int64_t m, int col, bool in) {
  Eight e{make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
  if (in && p.bias) e.b = *reinterpret_cast<const uint4*>(p.bias + col);
  if (in && p.resid) e.r = *reinterpret_cast<const uint4*>(p.resid + m * p.ldr + col);
  return e;
}
// Element i of eight bf16.
__device__ __forceinline__ float bf16_at(const uint4& v, int i) {
  const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
  return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
}
// act(f + bias) + R, as eight bf16.
template <int ACT>
__device__ __forceinline__ uint4 finish8(const float (&f)[8], const Eight& e) {
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = activate<ACT>(f[i] + bf16_at(e.b, i)) + bf16_at(e.r, i);
  return make_uint4(wptx::pack_bf16x2(v[0], v[1]), wptx::pack_bf16x2(v[2], v[3]),
                    wptx::pack_bf16x2(v[4], v[5]), wptx::pack_bf16x2(v[6], v[7]));
}

// Sum partial tiles [source][row][stride] (fp32, shared memory) of `rows` rows x
// `cols` columns in source order, finish and store them; row 0 is row m0 of Y,
// column 0 its column col0. `ready` is called once, after the first bias and
// residual loads are under way and before any partial is read.
template <int ACT, int THREADS, class P, class F>
__device__ __forceinline__ void sum_tiles(const P& p, const float* part, int sources, int per, int stride, int rows,
                                          int cols, int64_t m0, int col0, F ready) {
  constexpr int kBatch = 4;
  const int vec = cols >> 3, total = max(rows, 0) * vec;
  Eight e[kBatch];
  auto fetch = [&](int i0) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * THREADS, r = i / vec;
      e[k] = fetch8(p, m0 + r, col0 + (i - r * vec) * 8, i < total);
    }
  };
  fetch(threadIdx.x);
  ready();
  for (int i0 = threadIdx.x; i0 < total; i0 += kBatch * THREADS) {
    if (i0 != (int)threadIdx.x) fetch(i0);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int i = i0 + k * THREADS, r = i / vec, c = (i - r * vec) * 8;
      if (i >= total) break;
      float f[8] = {};
      for (int s = 0; s < sources; ++s) {
        const float4* src = reinterpret_cast<const float4*>(part + (s * per + r) * stride + c);
        const float4 lo = src[0], hi = src[1];
        f[0] += lo.x; f[1] += lo.y; f[2] += lo.z; f[3] += lo.w;
        f[4] += hi.x; f[5] += hi.y; f[6] += hi.z; f[7] += hi.w;
      }
      *reinterpret_cast<uint4*>(p.y + (m0 + r) * p.ldy + col0 + c) = finish8<ACT>(f, e[k]);
    }
  }
}

__device__ __forceinline__ void st_global_32(uint16_t* p, const uint4& a, const uint4& b) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a.x), "r"(a.y), "r"(a.z),
               "r"(a.w), "r"(b.x), "r"(b.y), "r"(b.z), "r"(b.w)
               : "memory");
}

// Columns c0 .. c1 - 1 (of p.N) of one row from TMEM (column 0 of the tile at
// `tmem`), finished and stored, 32 at a time with the next 32 columns' bias and
// residual on their way. All 32 lanes call it; `in`: the lane's row exists.
// `ready`: called after the first loads, before TMEM is read.
template <int ACT, class P, class F>
__device__ __forceinline__ void finish_row(const P& p, uint32_t tmem, int64_t m, int col0, int c0, int c1, bool in,
                                           F ready) {
  Eight e[4], n[4];
  auto fetch = [&](Eight (&x)[4], int c) {
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = fetch8(p, m, col0 + c + 8 * j, in && c + 8 * j < c1 && col0 + c + 8 * j < p.N);
  };
  fetch(e, c0);
  if (!ready()) return;
#pragma unroll 1
  for (int c = c0; c < c1 && col0 + c < p.N; c += 32) {
    fetch(n, c + 32);
    uint32_t v[32];
    uint4 out[4];
    wptx::tmem_ld32_wait(tmem + c, v);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(v[8 * j + i]);
      out[j] = finish8<ACT>(f, e[j]);
      e[j] = n[j];
    }
    uint16_t* y = p.y + m * p.ldy + col0 + c;
    if (p.wide && col0 + c + 32 <= p.N) {
      // whole 32-byte sectors: half the write requests
      if (in) {
        st_global_32(y, out[0], out[1]);
        st_global_32(y + 16, out[2], out[3]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (in && col0 + c + 8 * j < p.N) *reinterpret_cast<uint4*>(y + 8 * j) = out[j];
    }
    __syncwarp();  // reconverge before the next tcgen05.ld
  }
}

inline bool wide_rows(const uint16_t* y, int64_t ldy) {
  return (reinterpret_cast<uintptr_t>(y) & 31) == 0 && ldy % 16 == 0;
}

// Let kernel `fn` use `bytes` of dynamic shared memory on the current device, once
// per device (an attribute belongs to a device): `done` is the kernel's own word,
// a bit per device.
int allow_shared(const void* fn, int bytes, int device, std::atomic<uint64_t>& done);

// The kernel that takes a call of wave_linear_bias, by its sizes alone.
enum : int32_t { kDenseTokens = 0, kDenseTiles = 1, kDensePairs = 2 };
struct DenseForm {
  int32_t kind;
  int32_t cols;   // features of a block (tokens) or columns of a tile
  int32_t parts;  // warps of a block (tokens) or parts that K is cut into
};

// A checked call of wave_linear_bias.
struct DenseArgs {
  const void* A;
  int64_t lda;
  int32_t M, K;
  const void* W;
  int32_t N;
  const uint16_t* bias;
  const uint16_t* R;
  int64_t ldr;
  int32_t act;
  uint16_t* Y;
  int64_t ldy;
};

// Tensor map over a K-major bf16 matrix, `rows` rows of k (ld apart; 0: k) with
// a box of 64 x box_rows.
int encode_kmajor(CUtensorMap* map, const void* base, int64_t rows, int64_t k, uint32_t box_rows,
                  const char* what, int64_t ld = 0);

// wave_few.cu. At most 16 rows, blocks of 8 ft features (ft = 1 or 2) and 8 warps,
// or (ft = 1, at most 8 rows) 16.
int token_rows_launch(const DenseArgs& a, int ft, int warps, cudaStream_t s);
// wave_few.cu. Tiles of 128 rows x nf features (64 or 128), K cut over clusters of
// `splits` CTAs (1 .. 8, at most the 128-wide slices of K).
int split_rows_launch(const struct ::wave_kv* kv, const DenseArgs& a, int nf, int splits, cudaStream_t s);
// wave_pair.cu. Tiles of 256 rows x nt columns (192 or 256) on pairs of SMs; splits > 1
// (2 .. 4, at most the 128-wide slices of K): K cut over the pairs of a cluster.
int pair_rows_launch(const struct ::wave_kv* kv, const DenseArgs& a, int nt, int splits, cudaStream_t s);

}  // namespace wavei

// Registers a thread of kernel `fn`, asked for once and kept in the kernel's own word
// `known` (0 until then; a failed query is returned, and asked again by the next call).
extern "C" int wavei_kernel_registers(const void* fn, std::atomic<int32_t>* known, int32_t* regs);

// The choice on a GPU of `sms` SMs. Host only; C linkage, so that a test can ask
// which form its sizes reach.
extern "C" void wavei_dense_form(int32_t sms, int32_t M, int32_t K, int32_t N, wavei::DenseForm* form);
