// Token writes into cache entries that already have their pages: the append of
// tokens that arrive one by one or a few at a time.
//
// The work unit is the append kernel's tile: one page's rows of one head, of K
// or of V, one block each. bf16: the block copies the page's new rows, and
// where the page holds no token yet also zeroes the rows behind them. FP8: the
// block also reads the codes that the tile keeps, since a larger new token
// raises the tile's scale; it rewrites them only if the scale grew.
//
// What bounds it: for single tokens the launch (a 256-byte row per tile and,
// FP8, 16 KB of codes to look through): one token in each of four entries 1.4 us
// (FP8 3.4). For long runs HBM: 18720 tokens of 12 heads of 128, bf16, 37.5 us =
// 6.1 TB/s; FP8, whose blocks wait for their tile's maximum, 47 us = 3.7 TB/s.
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstddef>
#include <cstdint>
#include <cstring>
#include <utility>

#include "ptx.cuh"
#include "wave_internal.h"
#include "wave_wait.cuh"

namespace wavei {
namespace {

constexpr int kWriteThreads = 256;
constexpr int kWritePer = WAVE_PAGE_TOKENS * 16 / kWriteThreads;  // vectors per thread, d = 128

struct WriteEntry {
  int64_t row0;     // row of K and V that holds the entry's first new token
  int32_t first;    // tokens first .. first + count - 1 are written
  int32_t count;
  int32_t written;  // tokens the entry held before
  int32_t page_lo;  // first touched page, counted within the entry
  int32_t page0;    // its place in `pages`
  int32_t tile0;    // the entry's first tile
};

// The tables travel in the parameter block; a launch copies it, and 31 KB of
// it take about 3 us longer than the small form's 1 KB.
template <int ENTRIES, int PAGES>
struct WriteParamsOf {
  const uint16_t* k;
  const uint16_t* v;
  int64_t ldk, ldv;     // row strides in elements
  uint8_t* data;        // pool + data_offset
  float* scales;        // FP8: [max_pages][2][H]
  int64_t page_bytes;
  int32_t heads;
  int32_t log2_vec;     // 16-byte vectors per token row: 8 or 16
  int32_t n_entries;
  int32_t n_tiles;
  WriteEntry e[ENTRIES];
  int32_t pages[PAGES];
};
using WriteParams = WriteParamsOf<WAVE_MAX_APPEND_ENTRIES, WAVE_MAX_APPEND_PAGES>;
using WriteParamsSmall = WriteParamsOf<8, 64>;
static_assert(sizeof(WriteParams) <= 32760, "kernel parameter space is 32 KB");

// A block's tile: page, K or V, head, and which rows are new.
struct WriteTile {
  int64_t page;
  int kv, head;
  int64_t row;     // source row of the page's row r0
  int r0, r1;      // rows r0 .. r1 - 1 are new
  int held;        // rows held before the write (0: the page is fresh, and r0 = 0)
};

template <class P>
__device__ __forceinline__ WriteTile write_tile(const P& p, int tile) {
  int ei = 0;
  while (ei + 1 < p.n_entries && tile >= p.e[ei + 1].tile0) ++ei;
  const WriteEntry& en = p.e[ei];
  const int local = tile - en.tile0;
  const int per_page = 2 * p.heads;
  const int pi = local / per_page;
  const int kvh = local - pi * per_page;
  WriteTile t;
  t.page = p.pages[en.page0 + pi];
  t.kv = kvh >= p.heads;
  t.head = kvh - t.kv * p.heads;
  const int base = (en.page_lo + pi) * WAVE_PAGE_TOKENS;
  t.r0 = max(en.first - base, 0);
  t.r1 = min(en.first + en.count - base, WAVE_PAGE_TOKENS);
  t.row = en.row0 + (base + t.r0 - en.first);
  t.held = min(max(en.written - base, 0), WAVE_PAGE_TOKENS);
  return t;
}

template <class P>
__global__ void __launch_bounds__(kWriteThreads) kv_write_kernel(const __grid_constant__ P p) {
  chain_begin();
  const WriteTile t = write_tile(p, blockIdx.x);
  const int vec = 1 << p.log2_vec;
  const uint16_t* src = (t.kv ? p.v : p.k) + (t.row - t.r0) * (t.kv ? p.ldv : p.ldk) +
                        (int64_t)t.head * vec * 8;
  const int64_t ld = t.kv ? p.ldv : p.ldk;
  uint4* dst = reinterpret_cast<uint4*>(p.data + t.page * p.page_bytes) +
               ((int64_t)t.kv * p.heads + t.head) * WAVE_PAGE_TOKENS * vec;
  const int from = t.r0 * vec;
  const int to = (t.held == 0 ? WAVE_PAGE_TOKENS : t.r1) * vec;
  chain_wait();
  uint4 val[kWritePer];
#pragma unroll
  for (int u = 0; u < kWritePer; ++u) {
    const int i = from + threadIdx.x + u * kWriteThreads;
    const int r = i >> p.log2_vec;
    val[u] = make_uint4(0, 0, 0, 0);
    if (i < to && r < t.r1)
      val[u] = *(reinterpret_cast<const uint4*>(src + r * ld) + (i & (vec - 1)));
  }
#pragma unroll
  for (int u = 0; u < kWritePer; ++u) {
    const int i = from + threadIdx.x + u * kWriteThreads;
    if (i < to) dst[i] = val[u];
  }
}

__device__ __forceinline__ uint16_t write_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 write_decode2(uint16_t pair) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(pair));
  return make_float2(__half2float(__ushort_as_half((unsigned short)(h & 0xFFFF))),
                     __half2float(__ushort_as_half((unsigned short)(h >> 16))));
}

// E4M3(x / s), the quotient rounded to float32 first, for eight values. An IEEE
// division takes about twenty instructions, so the quotient is only bracketed:
// x times two reciprocals a factor 1 -+ 2^-21 apart from 1 / s lies on either
// side of it (their own roundings are below 3 * 2^-24), and where both round to
// the same code, so does everything between. Where they do not (a few values in
// a million), or s is so small or large that a reciprocal leaves float32's
// normal range, the division is done.
struct Quantizer {
  float s, lo, hi;
  bool bracket;
  __device__ __forceinline__ explicit Quantizer(float scale) : s(scale) {
    const float r = __frcp_rn(scale);
    lo = r * (1.f - 0x1p-21f);
    hi = r * (1.f + 0x1p-21f);
    bracket = scale >= 0x1p-100f && scale <= 0x1p100f;
  }
  __device__ __forceinline__ uint2 operator()(const float (&x)[8]) const {
    uint32_t a[4], b[4], differ = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = write_e4m3x2(x[2 * i] * lo, x[2 * i + 1] * lo);
      b[i] = write_e4m3x2(x[2 * i] * hi, x[2 * i + 1] * hi);
      differ |= a[i] ^ b[i];
    }
    if (differ != 0 || !bracket) {
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = write_e4m3x2(__fdiv_rn(x[2 * i], s), __fdiv_rn(x[2 * i + 1], s));
    }
    return make_uint2(a[0] | a[1] << 16, a[2] | a[3] << 16);
  }
};

// Row r of an FP8 tile is new (r0 <= r < r1), kept (r < held, not new) or zero.
// THREADS: 512 while the tiles leave SMs room, 256 in long writes, whose blocks then
// overlap their phases (loads, maximum, codes) better (us: 500 tokens of 24 heads
// 6.9 and 7.9; 18720 tokens of 12 heads 57 and 48).
template <int THREADS, class P>
__global__ void __launch_bounds__(THREADS) kv_write_fp8_kernel(const __grid_constant__ P p) {
  constexpr int kPer = WAVE_PAGE_TOKENS * 16 / THREADS;  // vectors per thread, d = 128
  __shared__ float warp_max[THREADS / 32];
  chain_begin();
  const WriteTile t = write_tile(p, blockIdx.x);
  const int vec = 1 << p.log2_vec;  // 8-value vectors per row
  const uint16_t* src = (t.kv ? p.v : p.k) + (t.row - t.r0) * (t.kv ? p.ldv : p.ldk) +
                        (int64_t)t.head * vec * 8;
  const int64_t ld = t.kv ? p.ldv : p.ldk;
  uint2* dst = reinterpret_cast<uint2*>(p.data + t.page * p.page_bytes) +
               ((int64_t)t.kv * p.heads + t.head) * WAVE_PAGE_TOKENS * vec;
  float* scale = p.scales + (t.page * 2 + t.kv) * p.heads + t.head;
  chain_wait();
  const float old = *scale;
  uint4 val[kPer];  // new rows: 8 bf16 values; kept rows: 8 codes in x, y
  float amax = 0.f;
  bool kept_some = false;
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = threadIdx.x + u * THREADS;
    const int r = i >> p.log2_vec;
    val[u] = make_uint4(0, 0, 0, 0);
    if (r >= t.r0 && r < t.r1) {
      val[u] = *(reinterpret_cast<const uint4*>(src + r * ld) + (i & (vec - 1)));
    } else if (r < t.held) {
      const uint2 c = dst[i];
      val[u].x = c.x;
      val[u].y = c.y;
    }
  }
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int r = (threadIdx.x + u * THREADS) >> p.log2_vec;
    if (r >= t.r0 && r < t.r1) {
      const uint32_t w[4] = {val[u].x, val[u].y, val[u].z, val[u].w};
#pragma unroll
      for (int e = 0; e < 4; ++e)
        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(w[e] << 16)),
                                 fabsf(__uint_as_float(w[e] & 0xFFFF0000u))));
    } else {
      kept_some |= ((val[u].x | val[u].y) & 0x7F7F7F7Fu) != 0;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  if ((threadIdx.x & 31) == 0) warp_max[threadIdx.x >> 5] = amax;
  // Also: every thread has read the old scale and its codes before any is replaced.
  const bool some = __syncthreads_or(kept_some);
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) amax = fmaxf(amax, warp_max[w]);
  const float want = __fdiv_rn(amax, 448.f);
  const float s = some ? fmaxf(old, want) : (amax > 0.f ? want : 1.f);
  const bool grew = some && s != old;
  if (threadIdx.x == 0) *scale = s;
  const Quantizer quantize(s);
#pragma unroll
  for (int u = 0; u < kPer; ++u) {
    const int i = threadIdx.x + u * THREADS;
    const int r = i >> p.log2_vec;
    if (r >= WAVE_PAGE_TOKENS) continue;
    const bool fresh = r >= t.r0 && r < t.r1;
    uint2 q = make_uint2(0, 0);
    if (fresh) {
      const uint32_t w[4] = {val[u].x, val[u].y, val[u].z, val[u].w};
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
      q = quantize(x);
    } else if (r < t.held) {
      if (!grew) continue;
      const uint32_t w[2] = {val[u].x, val[u].y};
      float x[8];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 v = write_decode2((uint16_t)(w[e >> 1] >> (16 * (e & 1))));
        x[2 * e] = v.x * old;
        x[2 * e + 1] = v.y * old;
      }
      q = quantize(x);
    } else if (t.held != 0) {
      continue;  // zero since the page's first write
    }
    dst[i] = q;
  }
}

template <class P>
cudaError_t launch_write(bool fp8, const P& p, int sms, cudaStream_t s) {
  const dim3 grid((unsigned)p.n_tiles);
  if (!fp8) return launch_chained(kv_write_kernel<P>, grid, kWriteThreads, 0, s, 1, p);
  return p.n_tiles <= 4 * sms ? launch_chained(kv_write_fp8_kernel<512, P>, grid, 512, 0, s, 1, p)
                              : launch_chained(kv_write_fp8_kernel<256, P>, grid, 256, 0, s, 1, p);
}

}  // namespace
}  // namespace wavei

using namespace wavei;

extern "C" int wave_kv_write_tokens(wave_kv* kv, int32_t n_entries, const wave_node* entries,
                                    const int32_t* first, const int32_t* ntokens, const void* K,
                                    int64_t ldk, const void* V, int64_t ldv, void* stream) {
  clear_error();
  if (!kv) return fail(WAVE_ERR_ARG, "NULL handle");
  if (!kv->on_device) return fail(WAVE_ERR_ARG, "host-only handle (pool == NULL) cannot write");
  if (n_entries < 0 || (n_entries > 0 && (!entries || !first || !ntokens)))
    return fail(WAVE_ERR_ARG, "bad arguments");
  if (n_entries > WAVE_MAX_APPEND_ENTRIES)
    return fail(WAVE_ERR_CAPACITY, "%d entries exceed %d per write call", n_entries,
                WAVE_MAX_APPEND_ENTRIES);
  const int64_t row = (int64_t)kv->cfg.heads * kv->cfg.head_dim;
  static thread_local WriteParams p;  // large: keep off the stack; launch copies it
  wave_entry* ents[WAVE_MAX_APPEND_ENTRIES];
  int64_t pages = 0, tiles = 0, rows = 0;
  int n = 0;
  for (int32_t i = 0; i < n_entries; ++i) {
    const auto it = kv->entries.find(std::make_pair(entries[i].chunk, entries[i].level));
    if (it == kv->entries.end())
      return fail(WAVE_ERR_MISSING_KV, "(%d, %d) has no pages", entries[i].chunk, entries[i].level);
    wave_entry& ent = it->second;
    for (int32_t j = 0; j < i; ++j)
      if (entries[j].chunk == entries[i].chunk && entries[j].level == entries[i].level)
        return fail(WAVE_ERR_ARG, "(%d, %d) named twice in one write call", entries[i].chunk,
                    entries[i].level);
    if (first[i] < 0 || ntokens[i] < 0 || (int64_t)first[i] + ntokens[i] > ent.ntokens)
      return fail(WAVE_ERR_ARG, "tokens %d .. %lld do not lie in the %d tokens of (%d, %d)",
                  first[i], (long long)first[i] + ntokens[i] - 1, ent.ntokens, entries[i].chunk,
                  entries[i].level);
    if (first[i] > ent.written)
      return fail(WAVE_ERR_ARG, "write at token %d of (%d, %d) would leave a hole: %d are written",
                  first[i], entries[i].chunk, entries[i].level, ent.written);
    if (ntokens[i] == 0) continue;
    const int32_t lo = first[i] / kPageTokens, hi = (first[i] + ntokens[i] - 1) / kPageTokens;
    if (pages + hi - lo + 1 > WAVE_MAX_APPEND_PAGES)
      return fail(WAVE_ERR_CAPACITY, "more than %d pages in one write", WAVE_MAX_APPEND_PAGES);
    p.e[n] = WriteEntry{rows, first[i], ntokens[i], ent.written, lo, (int32_t)pages, (int32_t)tiles};
    std::memcpy(p.pages + pages, ent.pages.data() + lo, (hi - lo + 1) * sizeof(int32_t));
    ents[n++] = &ent;
    pages += hi - lo + 1;
    tiles += (int64_t)(hi - lo + 1) * 2 * kv->cfg.heads;
    rows += ntokens[i];
    if (tiles >= (1LL << 31)) return fail(WAVE_ERR_CAPACITY, "too many page tiles in one write");
  }
  if (n == 0) return WAVE_OK;
  if (!K || !V || !aligned16(K) || !aligned16(V))
    return fail(WAVE_ERR_ARG, "K and V must be non-NULL and 16-byte aligned");
  if (ldk < row || ldk % 8 || ldk >= (1LL << 40) || ldv < row || ldv % 8 || ldv >= (1LL << 40))
    return fail(WAVE_ERR_ARG, "row strides must be multiples of 8 and cover heads * head_dim");
  if (int rc = check_current_device(kv)) return rc;
  p.k = static_cast<const uint16_t*>(K);
  p.v = static_cast<const uint16_t*>(V);
  p.ldk = ldk;
  p.ldv = ldv;
  uint8_t* pool = static_cast<uint8_t*>(kv->cfg.pool);
  p.data = pool + kv->data_offset;
  p.scales = kv->fp8 ? reinterpret_cast<float*>(pool + kv->scale_offset) : nullptr;
  p.page_bytes = kv->page_bytes;
  p.heads = kv->cfg.heads;
  p.log2_vec = kv->cfg.head_dim == 128 ? 4 : 3;
  p.n_entries = n;
  p.n_tiles = (int32_t)tiles;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (n <= 8 && pages <= 64) {
    WriteParamsSmall q;
    std::memcpy(&q, &p, offsetof(WriteParamsSmall, e));
    std::memcpy(q.e, p.e, n * sizeof(WriteEntry));
    std::memcpy(q.pages, p.pages, pages * sizeof(int32_t));
    e = launch_write(kv->fp8, q, kv->num_sms, s);
  } else {
    e = launch_write(kv->fp8, p, kv->num_sms, s);
  }
  if (e != cudaSuccess)
    return fail(WAVE_ERR_CUDA, "kv_write_kernel launch: %s", cudaGetErrorString(e));
  for (int i = 0; i < n; ++i)
    ents[i]->written = std::max(ents[i]->written, p.e[i].first + p.e[i].count);
  return WAVE_OK;
}
