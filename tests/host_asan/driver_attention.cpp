// Host-side exercise of the entry points between a QKV projection and an
// output projection under AddressSanitizer and UndefinedBehaviorSanitizer:
// argument validation, workspace sizing and the table of rotations over random
// and extreme arguments. Every call here returns before any device work: each
// has an argument that is refused, or nothing to do. Exit status 0 when every
// check holds.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>
#include <random>
#include <vector>

#include "qlinear.h"

static int failures = 0;
#define CHECK(cond)                                                           \
  do {                                                                        \
    if (!(cond)) {                                                            \
      std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
      ++failures;                                                             \
    }                                                                         \
  } while (0)

static const int64_t kSizes[] = {INT64_MIN, -1, 0, 1, 4, 7, 8, 64, 256, 264, 65536, 65537, int64_t(1) << 20, int64_t(1) << 22,
                                 int64_t(1) << 30, (int64_t(1) << 30) + 1, INT32_MAX, int64_t(1) << 40, INT64_MAX};
template <typename Rng> static int64_t size_of(Rng &rng) { return kSizes[rng() % (sizeof(kSizes) / sizeof(kSizes[0]))]; }

int main() {
  std::mt19937_64 rng(7);
  CHECK(qlinear_qk_norm_rope(nullptr, nullptr) == QL_EINVAL);
  CHECK(qlinear_attention(nullptr, nullptr) == QL_EINVAL);
  for (int i = 0; i < 40000; ++i) {
    ql_qk_args a;
    std::memset(&a, 0, sizeof(a));
    a.M = size_of(rng), a.head_dim = size_of(rng), a.q_heads = size_of(rng), a.kv_heads = size_of(rng);
    a.q_ld = size_of(rng), a.q_out_ld = size_of(rng), a.pairs = size_of(rng), a.axes = size_of(rng);
    a.norm = (int)(rng() % 5) - 1, a.rope = (int)(rng() % 4) - 1, a.in_dtype = (int)(rng() % 4) - 1;
    a.eps = rng() % 2 ? 1e-6f : std::numeric_limits<float>::quiet_NaN();
    a.q = rng() % 2 ? reinterpret_cast<const void *>(0x1000) : nullptr;
    // no output for q, or no part at all: nothing can run (M == 0 is nothing to do)
    const int st = qlinear_qk_norm_rope(&a, nullptr);
    CHECK(st != QL_OK || a.M == 0);
  }
  for (int i = 0; i < 40000; ++i) {
    ql_attention_args a;
    std::memset(&a, 0, sizeof(a));
    a.Mq = size_of(rng), a.Mk = size_of(rng), a.q_heads = size_of(rng), a.kv_heads = size_of(rng);
    a.head_dim = size_of(rng), a.samples = size_of(rng), a.q_ld = size_of(rng), a.out_ld = size_of(rng);
    a.k_ld = size_of(rng), a.v_ld = size_of(rng);
    a.scale = rng() % 2 ? 0.125f : rng() % 2 ? -1.f : std::numeric_limits<float>::infinity();
    if (rng() % 2) a.q_offsets = reinterpret_cast<const int32_t *>(0x1000);
    if (rng() % 2) a.k_offsets = reinterpret_cast<const int32_t *>(0x2000);
    // no output: nothing can run (no queries or no samples are nothing to do)
    const int st = qlinear_attention(&a, nullptr);
    CHECK(st != QL_OK || a.Mq == 0 || (a.q_offsets && a.samples == 0));
    const size_t ws = qlinear_attention_workspace_bytes(a.Mq, a.Mk, a.samples, a.q_heads, a.kv_heads, a.head_dim);
    CHECK(ws % 4 == 0);
    if (a.Mq <= 0 || a.Mk <= 0 || a.samples <= 0 || a.q_heads <= 0 || a.kv_heads <= 0 || a.head_dim <= 0 || a.head_dim % 8)
      CHECK(ws == 0);
  }
  // a workspace is bounded by what the card's blocks can cut, whatever the sizes
  for (int64_t q : {1, 16, 33, 4608, 1 << 20, 1 << 30})
    for (int64_t k : {1, 600, 4608, 1 << 30})
      for (int64_t s : {1, 16, 1000, 1 << 20})
        for (int64_t h : {1, 8, 18})
          for (int64_t d : {8, 64, 72, 128, 136, 256})
            CHECK(qlinear_attention_workspace_bytes(q, k, s, h, h, d) <= (size_t)600 << 20);
  for (int i = 0; i < 2000; ++i) {
    const int64_t axes = 1 + (int64_t)(rng() % 5);
    std::vector<int64_t> n((size_t)axes);
    int64_t pairs = 0;
    for (auto &x : n) pairs += x = (int64_t)(rng() % 40);
    std::vector<float> f((size_t)pairs + 1, -1.f);
    std::vector<int32_t> ax((size_t)pairs + 1, -1);
    const int order = (int)(rng() % 3);
    CHECK(qlinear_rope_table_host(10000.0, axes, n.data(), order, f.data(), ax.data()) == QL_OK);
    std::vector<int64_t> seen((size_t)axes, 0);
    for (int64_t j = 0; j < pairs; ++j) {
      CHECK(ax[(size_t)j] >= 0 && ax[(size_t)j] < axes && f[(size_t)j] > 0.f && f[(size_t)j] <= 1.f);
      ++seen[(size_t)ax[(size_t)j]];
    }
    CHECK(seen == n && f[(size_t)pairs] == -1.f && ax[(size_t)pairs] == -1);
  }
  int64_t n[2] = {4, -1};
  float f[8];
  int32_t ax[8];
  CHECK(qlinear_rope_table_host(10000.0, 2, n, 0, f, ax) == QL_EINVAL);
  n[1] = INT64_MAX;
  CHECK(qlinear_rope_table_host(10000.0, 2, n, 0, f, ax) == QL_EINVAL);
  for (double theta : {0.0, -1.0, (double)INFINITY, (double)NAN}) CHECK(qlinear_rope_table_host(theta, 1, n, 0, f, ax) == QL_EINVAL);
  if (failures) return 1;
  std::printf("host checks passed\n");
  return 0;
}
