// What the dense layers' kernels share: activations, their arguments, and the
// tensor map of a K-major operand.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "wave.h"

namespace wavei {

// GELU, tanh form, through 0.5 (1 + tanh u) = 1 / (1 + e^(-2u)): one
// exponential and one division on the special-function unit, with relative
// accuracy everywhere (the tail where 1 + tanh u is tiny included).
__device__ __forceinline__ float gelu_tanh(float x) {
  const float u = 0.7978845608028654f * fmaf(0.044715f * x, x * x, x);
  return __fdividef(x, 1.f + __expf(-2.f * u));
}

template <int ACT>
__device__ __forceinline__ float activate(float x) {
  if constexpr (ACT == WAVE_ACT_GELU_TANH) return gelu_tanh(x);
  if constexpr (ACT == WAVE_ACT_GELU_ERF) return 0.5f * x * (1.f + erff(0.7071067811865476f * x));
  if constexpr (ACT == WAVE_ACT_SILU) return __fdividef(x, 1.f + __expf(-x));
  return x;
}

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

// wave_few.cu. At most 16 rows, blocks of 8 ft features (ft = 1 or 2) and 8 or 16 warps.
int token_rows_launch(const DenseArgs& a, int ft, int warps, cudaStream_t s);
// wave_few.cu. Tiles of 128 rows x nf features (64, 128 or 256), K cut over clusters
// of `splits` CTAs (1 .. 8, at most the 64-wide slices of K).
int split_rows_launch(const struct ::wave_kv* kv, const DenseArgs& a, int nf, int splits, cudaStream_t s);

}  // namespace wavei
