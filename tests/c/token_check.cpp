// White-box check of what the single-token calls refuse, without a GPU. The
// handle is created host-only and then marked, through the library's internal
// struct, as a device handle of a device that no machine has: an argument that a
// call has to refuse comes back with its own code, and a call with good
// arguments stops at the device check (WAVE_ERR_ARG with a GPU, WAVE_ERR_CUDA
// without one), so nothing is launched and no pointer is read either way.
// Usage: token_check <1 if a CUDA device is visible, else 0>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <limits>
#include <vector>

#include "wave.h"
#include "wave_internal.h"

static int g_fail = 0;
alignas(256) static uint16_t buf[65536];

static void expect(long long got, long long want, const char* what) {
  if (got != want) {
    std::fprintf(stderr, "FAIL %s: %lld, want %lld (%s)\n", what, got, want, wave_last_error_detail());
    g_fail = 1;
  } else {
    std::printf("ok %s\n", what);
  }
}

static wave_kv* handle(int heads, int d, int tokens, int levels, int window, int prefix, int pages,
                       bool fake) {
  wave_kv_config cfg;
  std::memset(&cfg, 0, sizeof cfg);
  cfg.heads = heads;
  cfg.head_dim = d;
  cfg.tokens_per_chunk = tokens;
  cfg.num_levels = levels;
  cfg.window = window;
  cfg.prefix_tokens = prefix;
  cfg.pool_bytes = 4096 + (uint64_t)pages * 2 * heads * 128 * d * 2;
  wave_kv* kv = nullptr;
  if (wave_kv_create(&cfg, &kv) != WAVE_OK) {
    std::fprintf(stderr, "FAIL create: %s\n", wave_last_error_detail());
    std::exit(1);
  }
  if (fake) {
    kv->on_device = true;
    kv->device = 1 << 20;
    kv->num_sms = 148;
  }
  return kv;
}

int main(int argc, char** argv) {
  const int stop = argc > 1 && std::atoi(argv[1]) == 1 ? WAVE_ERR_ARG : WAVE_ERR_CUDA;
  uint16_t *p = buf, *odd = buf + 1;
  const int bad = WAVE_ERR_ARG;

  // ---- host-only handles and NULL
  wave_kv* host = handle(2, 64, 256, 2, 0, 0, 16, false);
  wave_rotary_spec spec = {{12, 10, 10}, 10000.f, 0, 0, 0};
  int32_t pos[3] = {0, 0, 0}, one = 1, zero = 0;
  const wave_node node{0, 1};
  uint64_t bytes = 0;
  for (wave_kv* kv : {host, (wave_kv*)nullptr}) {
    expect(wave_linear_bias(kv, p, 64, 1, 64, p, 64, nullptr, nullptr, 0, 0, p, 64, nullptr), bad, "linear: no device");
    expect(wave_rotary(kv, &spec, pos, 1, p, 128, 2, p, 128, nullptr, 0, 0, nullptr, 0, nullptr), bad, "rotary: no device");
    expect(wave_kv_write_tokens(kv, 1, &node, &zero, &one, p, 128, p, 128, nullptr), bad, "write: no device");
    expect(wave_token_attn(kv, &node, 1, 0, nullptr, 2, p, 128, p, 128, nullptr, nullptr, 0, nullptr), bad, "attention: no device");
    expect(wave_token_attn_workspace(kv, &node, 1, 0, nullptr, 2, &bytes), bad, "workspace: no device");
  }
  wave_kv_destroy(host);

  wave_kv* kv = handle(2, 64, 256, 2, 0, 100, 40, true);

  // ---- dense layer
  const uint16_t *a = p + 1024, *w = p + 2048;
  auto lin = [&](const void* A, int64_t lda, int M, int K, const void* W, int N, const void* b, const void* R,
                 int64_t ldr, int act, void* Y, int64_t ldy) {
    return wave_linear_bias(kv, A, lda, M, K, W, N, b, R, ldr, act, Y, ldy, nullptr);
  };
  expect(lin(a, 64, 3, 64, w, 64, a, p, 64, 3, p, 64), stop, "linear: good arguments reach the device check");
  expect(lin(nullptr, 64, 0, 64, nullptr, 64, nullptr, nullptr, 0, 0, nullptr, 64), WAVE_OK, "linear: no rows");
  expect(lin(a, 64, -1, 64, w, 64, a, p, 64, 0, p, 64), bad, "linear: M < 0");
  expect(lin(a, 64, (1 << 30) + 1, 64, w, 8, a, p, 64, 0, p, 64), bad, "linear: M > 2^30");
  expect(lin(a, 64, 3, 60, w, 64, a, p, 64, 0, p, 64), bad, "linear: K % 8");
  expect(lin(a, 64, 3, 64, w, 60, a, p, 64, 0, p, 64), bad, "linear: N % 8");
  expect(lin(a, 64, 3, 0, w, 64, a, p, 64, 0, p, 64), bad, "linear: K = 0");
  expect(lin(a, 64, 3, 64, w, 0, a, p, 64, 0, p, 64), bad, "linear: N = 0");
  expect(lin(a, 65544, 3, 65544, w, 64, a, p, 64, 0, p, 64), bad, "linear: K > 65536");
  expect(lin(a, 56, 3, 64, w, 64, a, p, 64, 0, p, 64), bad, "linear: lda < K");
  expect(lin(a, 68, 3, 64, w, 64, a, p, 64, 0, p, 64), bad, "linear: lda % 8");
  expect(lin(a, 1LL << 39, 3, 64, w, 64, a, p, 64, 0, p, 64), bad, "linear: lda past the tensor map");
  expect(lin(a, 64, 3, 64, w, 64, a, p, 56, 0, p, 64), bad, "linear: ldr < N");
  expect(lin(a, 64, 3, 64, w, 64, a, p, 64, 0, p, 56), bad, "linear: ldy < N");
  expect(lin(a, 64, 3, 64, w, 64, a, p, 72, 0, p, 64), bad, "linear: in place with other strides");
  expect(lin(a, 64, 3, 64, w, 64, a, p, 64, 4, p, 64), bad, "linear: activation");
  expect(lin(a, 64, 3, 64, w, 64, a, p, 64, -1, p, 64), bad, "linear: activation < 0");
  expect(lin(odd, 64, 3, 64, w, 64, a, p, 64, 0, p, 64), bad, "linear: A misaligned");
  expect(lin(a, 64, 3, 64, odd, 64, a, p, 64, 0, p, 64), bad, "linear: W misaligned");
  expect(lin(a, 64, 3, 64, w, 64, odd, p, 64, 0, p, 64), bad, "linear: bias misaligned");
  expect(lin(a, 64, 3, 64, w, 64, a, odd, 64, 0, p, 64), bad, "linear: R misaligned");
  expect(lin(a, 64, 3, 64, w, 64, a, p, 64, 0, odd, 64), bad, "linear: Y misaligned");
  expect(lin(a, 64, 3, 64, w, 64, a, p, 64, 0, nullptr, 64), bad, "linear: no Y");
  expect(lin(p, 64, 3, 64, w, 64, a, nullptr, 0, 0, p, 64), bad, "linear: Y is A");
  expect(lin(a, 64, 3, 64, p, 64, a, nullptr, 0, 0, p, 64), bad, "linear: Y is W");
  expect(lin(a, 64, 3, 64, w, 64, p, nullptr, 0, 0, p, 64), bad, "linear: Y is bias");
  expect(wave_linear(kv, p, 3, 64, p, 256, nullptr, WAVE_ACT_SILU, p, nullptr) < 0, 1, "wave_linear refuses SiLU");

  // ---- rotary
  auto rot = [&](wave_rotary_spec s, const int32_t* ps, int rows, const void* q, int64_t ldq, int qh, void* qo,
                 int64_t ldqo, const void* k, int64_t ldk, int kh, void* ko, int64_t ldko) {
    return wave_rotary(kv, &s, ps, rows, q, ldq, qh, qo, ldqo, k, ldk, kh, ko, ldko, nullptr);
  };
  auto with = [&](int a, int b, int c, float base, int layout, int ladder, int inverse) {
    return rot({{a, b, c}, base, layout, ladder, inverse}, pos, 1, p, 128, 2, p + 512, 128, nullptr, 0, 0, nullptr, 0);
  };
  const float inf = std::numeric_limits<float>::infinity(), nan = std::numeric_limits<float>::quiet_NaN();
  expect(with(12, 10, 10, 10000.f, 1, 1, 1), stop, "rotary: good arguments reach the device check");
  expect(with(12, 10, 11, 10000.f, 0, 0, 0), bad, "rotary: too many pairs");
  expect(with(-1, 10, 10, 10000.f, 0, 0, 0), bad, "rotary: pairs < 0");
  expect(with(2147483647, 2147483647, 2, 10000.f, 0, 0, 0), bad, "rotary: pairs that wrap");
  expect(with(12, 10, 10, 1.f, 0, 0, 0), bad, "rotary: base 1");
  expect(with(12, 10, 10, inf, 0, 0, 0), bad, "rotary: base inf");
  expect(with(12, 10, 10, nan, 0, 0, 0), bad, "rotary: base NaN");
  expect(with(12, 10, 10, 10000.f, 2, 0, 0), bad, "rotary: layout");
  expect(with(12, 10, 10, 10000.f, 0, 2, 0), bad, "rotary: ladder");
  expect(with(12, 10, 10, 10000.f, 0, 0, 2), bad, "rotary: inverse");
  expect(rot(spec, pos, 0, nullptr, 128, 2, nullptr, 128, nullptr, 0, 0, nullptr, 0), WAVE_OK, "rotary: no rows");
  expect(rot(spec, pos, -1, p, 128, 2, p, 128, nullptr, 0, 0, nullptr, 0), bad, "rotary: rows < 0");
  expect(rot(spec, nullptr, 1, p, 128, 2, p, 128, nullptr, 0, 0, nullptr, 0), bad, "rotary: no positions");
  expect(rot(spec, pos, 1, p, 128, 0, p, 128, nullptr, 0, 0, nullptr, 0), bad, "rotary: no heads");
  expect(rot(spec, pos, 1, p, 120, 2, p, 128, nullptr, 0, 0, nullptr, 0), bad, "rotary: ldq short");
  expect(rot(spec, pos, 1, p, 128, 2, p, 132, nullptr, 0, 0, nullptr, 0), bad, "rotary: ldqo % 8");
  expect(rot(spec, pos, 1, p, 128, 2, p, 136, nullptr, 0, 0, nullptr, 0), bad, "rotary: in place with other strides");
  expect(rot(spec, pos, 1, odd, 128, 2, p, 128, nullptr, 0, 0, nullptr, 0), bad, "rotary: Q misaligned");
  expect(rot(spec, pos, 1, p, 128, 2, p, 128, p, 128, 2, nullptr, 128), bad, "rotary: K without Kout");
  expect(rot(spec, pos, 1, p, 128, 2, p, 128, p, 64, 2, p, 64), bad, "rotary: ldk short");

  // ---- token writes
  expect(wave_kv_alloc(kv, -1, 0, 100), WAVE_OK, "alloc prefix");
  expect(wave_kv_alloc(kv, 0, 1, 256), WAVE_OK, "alloc (0, 1)");
  expect(wave_kv_alloc(kv, 1, 1, 256), WAVE_OK, "alloc (1, 1)");
  auto wr = [&](std::vector<wave_node> e, std::vector<int32_t> f, std::vector<int32_t> n, const void* k = buf,
                int64_t ldk = 128, const void* v = buf, int64_t ldv = 128) {
    return wave_kv_write_tokens(kv, (int)e.size(), e.data(), f.data(), n.data(), k, ldk, v, ldv, nullptr);
  };
  expect(wr({{0, 1}, {-1, 0}}, {0, 0}, {256, 100}), stop, "write: good arguments reach the device check");
  expect(wr({{0, 1}}, {1}, {1}), bad, "write: nothing was counted, so a hole");
  kv->entries.at({0, 1}).written = 130;
  expect(wr({{0, 1}}, {130}, {1}), stop, "write: the next token");
  expect(wr({{0, 1}}, {131}, {1}), bad, "write: a hole");
  expect(wr({{0, 1}}, {100}, {156}), stop, "write: up to the end");
  expect(wr({{0, 1}}, {100}, {157}), bad, "write: past the end");
  expect(wr({{0, 1}}, {-1}, {1}), bad, "write: first < 0");
  expect(wr({{0, 1}}, {0}, {-1}), bad, "write: count < 0");
  expect(wr({{0, 1}}, {100}, {2147483647}), bad, "write: count that wraps");
  expect(wr({{0, 1}, {1, 1}, {0, 1}}, {0, 0, 5}, {1, 1, 1}), bad, "write: an entry twice");
  expect(wr({{0, 2}}, {0}, {1}), WAVE_ERR_MISSING_KV, "write: no such entry");
  expect(wr({{0, 1}, {1, 1}}, {130, 0}, {0, 0}, nullptr, 0, nullptr, 0), WAVE_OK, "write: nothing");
  expect(wr({}, {}, {}), WAVE_OK, "write: no entries");
  expect(wr({{0, 1}}, {0}, {1}, nullptr), bad, "write: no K");
  expect(wr({{0, 1}}, {0}, {1}, odd), bad, "write: K misaligned");
  expect(wr({{0, 1}}, {0}, {1}, p, 120), bad, "write: ldk short");
  expect(wr({{0, 1}}, {0}, {1}, p, 128, p, 130), bad, "write: ldv % 8");
  expect(wave_kv_write_tokens(kv, 65, &node, &zero, &one, p, 128, p, 128, nullptr), WAVE_ERR_CAPACITY, "write: 65 entries");
  expect(wave_kv_write_tokens(kv, 1, nullptr, &zero, &one, p, 128, p, 128, nullptr), bad, "write: no list");
  expect(kv->entries.at({0, 1}).written, 130, "a refused write counts nothing");

  // ---- token attention
  auto att = [&](std::vector<wave_node> a, std::vector<int32_t> own, int qh = 2, int policy = WAVE_POLICY_SAME,
                 const void* q = buf, int64_t ldq = 1024, void* o = buf, int64_t ldo = 1024, void* ws = buf,
                 uint64_t n = sizeof buf) {
    return wave_token_attn(kv, a.data(), (int)a.size(), policy, own.empty() ? nullptr : own.data(), qh, q, ldq, o,
                           ldo, nullptr, ws, n, nullptr);
  };
  expect(att({{1, 1}}, {256}), stop, "attention: good arguments reach the device check");
  expect(att({{1, 1}}, {}), stop, "attention: whole entries");
  expect(att({}, {}), WAVE_OK, "attention: no queries");
  expect(att({{1, 1}}, {257}), bad, "attention: own_tokens past the entry");
  expect(att({{1, 1}}, {-1}), bad, "attention: own_tokens < 0");
  expect(att({{2, 1}}, {0}), stop, "attention: own entry not needed");
  expect(att({{2, 1}}, {1}), WAVE_ERR_MISSING_KV, "attention: own entry missing");
  expect(att({{1, 2}}, {0}), WAVE_ERR_MISSING_KV, "attention: history missing");
  expect(att({{1, 3}}, {}), bad, "attention: level");
  expect(att({{-1, 0}}, {}), bad, "attention: the prefix asks nothing");
  expect(att({{1, 1}}, {}, 2, 3), bad, "attention: policy");
  expect(att({{1, 1}}, {}, 3), bad, "attention: q_heads not a multiple");
  expect(att({{1, 1}}, {}, 34), bad, "attention: q_heads over 16 times");
  expect(att({{1, 1}}, {}, 0), bad, "attention: no q_heads");
  expect(att({{1, 1}}, {}, 2, WAVE_POLICY_SAME, nullptr), bad, "attention: no Q");
  expect(att({{1, 1}}, {}, 2, WAVE_POLICY_SAME, odd), bad, "attention: Q misaligned");
  expect(att({{1, 1}}, {}, 2, WAVE_POLICY_SAME, p, 120), bad, "attention: ldq short");
  expect(att({{1, 1}}, {}, 2, WAVE_POLICY_SAME, p, 128, p, 132), bad, "attention: ldo % 8");
  expect(att({{1, 1}}, {}, 2, WAVE_POLICY_SAME, p, 128, p, 128, nullptr, 0), stop, "attention: a short list needs no workspace");
  expect(wave_token_attn(kv, std::vector<wave_node>(65, {1, 1}).data(), 65, 1, nullptr, 2, p, 128, p, 128, nullptr,
                         p, sizeof buf, nullptr), WAVE_ERR_CAPACITY, "attention: 65 queries");
  wave_kv_destroy(kv);

  // ---- list lengths: 5120 items a call
  kv = handle(1, 64, 128 * 1024, 1, 0, 0, 5 * 1024 + 8, true);
  for (int c = 0; c < 5; ++c) expect(wave_kv_alloc(kv, c, 1, 128 * 1024), WAVE_OK, "alloc 1024 pages");
  const wave_node last{4, 1}, two[2] = {{4, 1}, {4, 1}};
  int32_t own[2] = {128 * 1024, 128 * 1024};
  expect(wave_token_attn_workspace(kv, &last, 1, 1, own, 1, &bytes), WAVE_OK, "5120 pages");
  expect((long long)bytes, 15 * (64 + 2) * 4, "one list over 15 clusters");
  auto late = [&](void* ws, uint64_t n) {
    return wave_token_attn(kv, &last, 1, 1, own, 1, p, 64, p, 64, nullptr, ws, n, nullptr);
  };
  expect(late(p, bytes), stop, "attention: workspace as told");
  expect(late(p, bytes - 1), bad, "attention: short workspace");
  expect(late(p + 8, bytes), bad, "attention: workspace misaligned");
  expect(late(nullptr, bytes), bad, "attention: no workspace");
  expect(wave_token_attn_workspace(kv, two, 2, 1, own, 1, &bytes), WAVE_OK, "5120 pages, shared by two queries");
  expect((long long)bytes, 15 * 2 * (64 + 2) * 4, "two rows a part");
  own[1] -= 1;  // its last page is an item of its own
  expect(wave_token_attn_workspace(kv, two, 2, 1, own, 1, &bytes), WAVE_ERR_CAPACITY, "5121 items");
  own[1] -= 127;
  expect(wave_token_attn_workspace(kv, two, 2, 1, own, 1, &bytes), WAVE_OK, "a page less is not another item");
  expect(wave_token_attn_workspace(kv, two, 2, 1, nullptr, 16, &bytes), WAVE_ERR_CAPACITY, "two groups share nothing");
  int32_t few = 100;
  const wave_node head{0, 1};
  expect(wave_token_attn_workspace(kv, &head, 1, 1, &few, 1, &bytes), WAVE_OK, "one page");
  expect((long long)bytes, 0, "a short list needs no workspace");
  few = 0;
  expect(wave_token_attn_workspace(kv, &head, 1, 1, &few, 1, &bytes), WAVE_OK, "no token");
  expect((long long)bytes, 0, "nothing to join");
  wave_kv_destroy(kv);

  // ---- writes: 7168 touched pages a call
  kv = handle(1, 64, 128 * 3700, 1, 0, 0, 7500, true);
  wave_kv_alloc(kv, 0, 1, 128 * 3700);
  wave_kv_alloc(kv, 1, 1, 128 * 3700);
  auto big = [&](int n) {
    const wave_node e[2] = {{0, 1}, {1, 1}};
    const int32_t f[2] = {0, 0}, c[2] = {128 * 3700, n};
    return wave_kv_write_tokens(kv, 2, e, f, c, p, 64, p, 64, nullptr);
  };
  expect(big(128 * 3468), stop, "write: 7168 pages");
  expect(big(128 * 3468 + 1), WAVE_ERR_CAPACITY, "write: 7169 pages");
  wave_kv_destroy(kv);
  return g_fail;
}
