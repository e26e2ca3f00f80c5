// wave_linear_bias: its checks, and which kernel takes a call.
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "wave_dense.cuh"
#include "wave_internal.h"

namespace wavei {
namespace {

// Up to 16 rows: token_rows_kernel (wave_few.cu), by waves of its blocks: an SM holds
// four of 8 warps (three with more than 8 rows), two of 16. Blocks of 8 features while
// they are one wave, else of 16 (chained, weights from HBM, one row, us, 8 and 16
// features: 1536 -> 1536 3.0 and 3.8, 2048 -> 4736 5.1 and 6.5, 1536 -> 8960 7.4 and
// 6.2, 8192 -> 8192 25.8 and 25.7). Sixteen warps to a block where that is one wave and
// K is long (8 and 16 warps: 8960 -> 1536 11.1 and 8.6, 4096 -> 2048 6.2 and 5.1, 1536
// -> 1536 3.0 and 3.5, 4096 -> 4096 7.3 and 8.9).
// With 9 to 16 rows a block reads more of A than of W, and tiles take over beyond one
// wave or where K is long (token rows and the best tiles: 16 rows 1536 -> 4608 6.6 and
// 7.6, 4096 -> 4096 11.8 both, 8960 -> 1536 14.3 and 11.0, 8192 -> 8192 39.3 and 26.7; 12
// rows 1536 -> 8960 10.2 and 9.2, 4096 -> 2048 7.8 and 8.8). Of 40 sizes of up to 16 rows
// measured, the rule takes the fastest form in each (the sweep is kept under profiles/).
bool takes_tokens(int sms, int32_t M, int32_t K, int32_t N) { return M <= 8 || (M <= 16 && K <= 4096 && N <= 3 * 16 * sms); }
DenseForm tokens_form(int sms, int32_t M, int32_t K, int32_t N) {
  const int held = M <= 8 ? 4 : 3;
  if (N > held * 8 * sms) return {kDenseTokens, 16, 8};
  return {kDenseTokens, 8, M <= 8 && K >= 4096 && N <= 2 * 8 * sms ? 16 : 8};
}

// More rows: the cheapest form by its cost in us: a start and end, more where the
// parts of K are joined, and what a 128-wide slice of K takes (for pairs in several
// waves, at the clock under load), fitted to 55 sizes, M = 40 .. 4680 and K x N = 1536 x
// 1536 .. 4096 x 4096, of which it takes the best form in 49 and one within 7 % in the
// others (the sweep is kept under profiles/). Both sides: 984 x 8960 x 1536: 192-column pairs with
// K in two 29.8, 256-column 33.8, 128-column tiles 38.3; 256 x 1536 x 1536: 64-column
// tiles with K in two 8.4, 128-column in four 9.6, pairs 11.8; 512 x 1536 x 4608:
// 128-column tiles 11.2, pairs 13.6; 2000 x 1536 x 8960: 256-column pairs 43.5,
// 192-column 49.3, 128-column tiles 82.
DenseForm rows_form(int sms, int32_t M, int32_t K, int32_t N) {
  struct Form {
    int rows, cols, ctas, most;         // tile, CTAs that share one, most parts of K
    double start, join, slice, loaded;  // `loaded`: a slice in more than one wave
  };
  constexpr Form kForms[4] = {{128, 64, 1, 8, 4.5, 1.5, 0.40, 0.40},
                              {128, 128, 1, 8, 5.3, 3.5, 0.49, 0.49},
                              {256, 192, 2, 4, 6.7, 3.5, 0.55, 0.62},
                              {256, 256, 2, 4, 8.2, 3.5, 0.60, 0.72}};
  const int64_t slices = (K + 127) / 128;
  double best = 1e30;
  DenseForm form{kDensePairs, 256, 1};
  for (int f = 0; f < 4; ++f)
    for (int n = 1; n <= kForms[f].most && n <= slices; ++n) {
      const Form& x = kForms[f];
      const int64_t tiles = ((int64_t)M + x.rows - 1) / x.rows * ((N + x.cols - 1) / x.cols);
      const int64_t held = clusters_held(x.ctas * n, sms);
      const double waves = (double)((tiles + held - 1) / held);
      // Pairs that do not share K are persistent: their tiles follow without a gap.
      const bool persistent = x.ctas == 2 && n == 1;
      const double t = (persistent ? 1.0 : waves) * (x.start + (n > 1 ? x.join : 0.0)) +
                       waves * (double)((slices + n - 1) / n) * (waves > 1 ? x.loaded : x.slice);
      if (t < best) best = t, form = {x.ctas == 2 ? kDensePairs : kDenseTiles, x.cols, n};
    }
  return form;
}

}  // namespace

int allow_shared(const void* fn, int bytes, int device, std::atomic<uint64_t>& done) {
  const bool counted = device >= 0 && device < 64;
  if (counted && (done.load(std::memory_order_acquire) >> device & 1)) return WAVE_OK;
  const cudaError_t e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return fail(WAVE_ERR_CUDA, "cudaFuncSetAttribute: %s", cudaGetErrorString(e));
  if (counted) done.fetch_or(1ull << device, std::memory_order_release);
  return WAVE_OK;
}

}  // namespace wavei

using namespace wavei;

extern "C" int wavei_kernel_registers(const void* fn, std::atomic<int32_t>* known, int32_t* regs) {
  *regs = known->load(std::memory_order_relaxed);
  if (*regs > 0) return WAVE_OK;
  cudaFuncAttributes a;
  const cudaError_t e = cudaFuncGetAttributes(&a, fn);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(WAVE_ERR_CUDA, "cudaFuncGetAttributes: %s", cudaGetErrorString(e));
  }
  *regs = a.numRegs;
  known->store(a.numRegs, std::memory_order_relaxed);
  return WAVE_OK;
}

extern "C" void wavei_dense_form(int32_t sms, int32_t M, int32_t K, int32_t N, DenseForm* form) {
  *form = takes_tokens(sms, M, K, N) ? tokens_form(sms, M, K, N) : rows_form(sms, M, K, N);
}

extern "C" int wave_linear_bias(wave_kv* kv, const void* A, int64_t lda, int32_t M, int32_t K,
                                const void* W, int32_t N, const void* bias, const void* R,
                                int64_t ldr, int32_t act, void* Y, int64_t ldy, void* stream) {
  clear_error();
  if (!kv) return fail(WAVE_ERR_ARG, "NULL handle");
  if (!kv->on_device) return fail(WAVE_ERR_ARG, "host-only handle (pool == NULL) cannot launch");
  if (M < 0 || M > (1 << 30) || K < 8 || K % 8 != 0 || K > (1 << 16) || N < 8 || N % 8 != 0 || N > (1 << 16))
    return fail(WAVE_ERR_ARG, "need 0 <= M <= 2^30, K and N positive multiples of 8 (at most 65536); got "
                "M %d, K %d, N %d", M, K, N);
  if ((int64_t)M * N >= (1LL << 40)) return fail(WAVE_ERR_ARG, "M x N too large");
  if (act < WAVE_ACT_NONE || act > WAVE_ACT_SILU) return fail(WAVE_ERR_ARG, "unknown activation %d", act);
  const int64_t most = 1LL << 38;  // the tensor map's stride is below 2^40 bytes
  if (lda < K || lda % 8 || lda >= most || ldy < N || ldy % 8 || ldy >= most ||
      (R && (ldr < N || ldr % 8 || ldr >= most)))
    return fail(WAVE_ERR_ARG, "row strides must be multiples of 8 and cover the row; got lda %lld, "
                "ldr %lld, ldy %lld", (long long)lda, (long long)ldr, (long long)ldy);
  if (Y && (Y == A || Y == W || Y == bias)) return fail(WAVE_ERR_ARG, "Y may overlap nothing but R");
  if (R && R == Y && ldr != ldy) return fail(WAVE_ERR_ARG, "Y = R needs ldy = ldr");
  if (M == 0) return WAVE_OK;
  if (!A || !W || !Y || !aligned16(A) || !aligned16(W) || !aligned16(Y) || (R && !aligned16(R)) ||
      (bias && !aligned16(bias)))
    return fail(WAVE_ERR_ARG, "A, W, Y (and bias, R) must be non-NULL and 16-byte aligned");
  if (int rc = check_current_device(kv)) return rc;
  if (((int64_t)M + 127) / 128 * ((N + 63) / 64) >= (1LL << 27)) return fail(WAVE_ERR_ARG, "M x N too large");
  const DenseArgs a{A, lda, M, K, W, N, static_cast<const uint16_t*>(bias), static_cast<const uint16_t*>(R),
                    ldr, act, static_cast<uint16_t*>(Y), ldy};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  DenseForm f;
  wavei_dense_form(kv->num_sms, M, K, N, &f);
  if (f.kind == kDenseTokens) return token_rows_launch(a, f.cols / 8, f.parts, s);
  return f.kind == kDensePairs ? pair_rows_launch(kv, a, f.cols, f.parts, s) : split_rows_launch(kv, a, f.cols, f.parts, s);
}
