// Host-side exercise of the entry points around a projection under
// AddressSanitizer and UndefinedBehaviorSanitizer: argument validation and
// workspace sizing of qlinear_block_norm and qlinear_adapters over random and
// extreme arguments. Every call here returns before any device work: each has
// an argument that is refused, or nothing to do. Exit status 0 when every
// check holds.
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <limits>
#include <random>

#include "qlinear.h"

static int failures = 0;
#define CHECK(cond)                                                           \
  do {                                                                        \
    if (!(cond)) {                                                            \
      std::fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #cond); \
      ++failures;                                                             \
    }                                                                         \
  } while (0)

static const int64_t kSizes[] = {INT64_MIN, -1, 0, 1, 7, 64, 256, 4608, 65536, 65537, INT32_MAX, int64_t(INT32_MAX) + 1,
                                 int64_t(1) << 40, INT64_MAX};
template <typename Rng> static int64_t size_of(Rng &rng) { return kSizes[rng() % (sizeof(kSizes) / sizeof(kSizes[0]))]; }

int main() {
  std::mt19937_64 rng(5);
  CHECK(qlinear_block_norm(nullptr, nullptr) == QL_EINVAL);
  CHECK(qlinear_adapters(nullptr, nullptr) == QL_EINVAL);
  for (int i = 0; i < 20000; ++i) {
    ql_block_norm_args a;
    std::memset(&a, 0, sizeof(a));
    a.M = size_of(rng), a.D = size_of(rng), a.gate_ld = size_of(rng), a.scale_ld = size_of(rng);
    a.shift_ld = size_of(rng), a.mod_rows = size_of(rng), a.samples = size_of(rng);
    a.post_norm = (int)(rng() % 5) - 1, a.pre_norm = (int)(rng() % 5) - 1;
    a.post_eps = rng() % 2 ? 1e-6f : -1.f, a.pre_eps = rng() % 2 ? 1e-6f : std::numeric_limits<float>::quiet_NaN();
    a.residual_scale = rng() % 2 ? 1.f : std::numeric_limits<float>::infinity();
    a.y_dtype = (int)(rng() % 4) - 1, a.residual_dtype = (int)(rng() % 4) - 1;
    // no residual: nothing can run (M == 0 is nothing to do)
    const int st = qlinear_block_norm(&a, nullptr);
    CHECK(st != QL_OK || a.M == 0);
  }
  for (int i = 0; i < 20000; ++i) {
    ql_adapter_args a;
    std::memset(&a, 0, sizeof(a));
    a.M = size_of(rng), a.N = size_of(rng), a.K = size_of(rng), a.adapters = size_of(rng), a.rank = size_of(rng);
    a.epilogue = (int)(rng() % 5) - 1, a.ab_dtype = (int)(rng() % 4) - 1, a.out_dtype = (int)(rng() % 4) - 1;
    a.gate_rows = size_of(rng);
    // no output: nothing can run (M == 0 or N == 0 is nothing to do)
    const int st = qlinear_adapters(&a, nullptr);
    CHECK(st != QL_OK || a.M == 0 || a.N == 0);
    const size_t ws = qlinear_adapters_workspace_bytes(a.M, a.N, a.K, a.rank, a.adapters);
    CHECK(ws % 4 == 0);
    if (a.M <= 0 || a.N <= 0 || a.K < 0 || a.K % 64 || a.adapters <= 0 || a.rank % 8) CHECK(ws == 0);
  }
  for (int64_t M : {1, 15, 16, 17, 1024, 1025, 4096, INT32_MAX})
    for (int64_t N : {1, 64, 4608, 1 << 22})
      for (int64_t K : {0, 64, 4608, 1 << 22})
        for (int64_t rank : {8, 16, 24, 32, 64, 72, 256})
          for (int64_t n : {1, 3, 1000, INT32_MAX}) {
            const size_t ws = qlinear_adapters_workspace_bytes(M, N, K, rank, n);
            CHECK(ws >= (size_t)M * rank * 4 && ws <= (size_t)M * rank * 4 * 8 && ws % ((size_t)M * rank * 4) == 0);
          }
  if (failures) return 1;
  std::printf("host checks passed\n");
  return 0;
}
