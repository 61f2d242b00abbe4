// Host-only check of the 8-bit operators' plans (plan.cpp), built with g++
// under AddressSanitizer and UndefinedBehaviorSanitizer by
// tests/test_fp8_plan_sanitized.py: splits of K that cover it with none empty,
// workspaces large enough for what the kernels write, sizes up to the largest
// accepted.
#include <stdio.h>

#include <vector>

#include "plan.h"

using namespace ortho;

static long checks = 0;
static int failures = 0;
#define EXPECT(cond, m, n, k)                                                              \
  do {                                                                                     \
    ++checks;                                                                              \
    if (!(cond)) {                                                                         \
      ++failures;                                                                          \
      fprintf(stderr, "FAIL %s at %lld x %lld x %lld\n", #cond, (long long)(m), (long long)(n), (long long)(k)); \
    }                                                                                      \
  } while (0)

int main() {
  const std::vector<int64_t> dims = {1,   2,    31,   32,   33,   64,   127,  128,   129,   200,   256,
                                     300, 1000, 1024, 1537, 2048, 4096, 8192, 16384, 53248, 131072};
  for (int64_t m : dims)
    for (int64_t n : dims)
      for (int64_t k : dims) {
        Fp8MatmulPlan p;
        EXPECT(plan_fp8_matmul(m, n, k, &p), m, n, k);
        const int64_t nkb = (k + 127) / 128, tiles = ((m + 127) / 128) * ((n + 127) / 128);
        EXPECT(p.splits >= 1 && p.kchunk >= 1, m, n, k);
        EXPECT((int64_t)p.splits * p.kchunk >= nkb, m, n, k);
        EXPECT((int64_t)(p.splits - 1) * p.kchunk < nkb, m, n, k);   // the last one is not empty
        EXPECT(p.ldp >= n && p.ldp % 4 == 0 && p.ldp < n + 4, m, n, k);
        EXPECT(p.total_bytes % kWsAlign == 0 && p.total_bytes > 0, m, n, k);
        if (p.splits > 1) {
          EXPECT(p.total_bytes >= (size_t)p.splits * m * p.ldp * 4, m, n, k);
          EXPECT(m > kFewRowsMax && tiles * p.splits <= 256 && p.kchunk >= 3, m, n, k);
          // what a launch for large results takes is never split
          EXPECT(m * n < 256 * 256 * 160, m, n, k);
        }
      }
  for (int64_t m : dims)
    for (int64_t n : dims) {
      NormGradPlan p;
      EXPECT(plan_norm_grad(m, n, &p) == (n <= kNormMaxCols), m, n, 0);
      if (n > kNormMaxCols) continue;
      EXPECT(p.groups >= 1 && p.groups <= m && p.ld >= n && p.ld % 8 == 0, m, n, 0);
      EXPECT(p.total_bytes >= (size_t)p.groups * p.ld * 4 && p.total_bytes % kWsAlign == 0, m, n, 0);
    }
  const int64_t big = int64_t{1} << 30;
  Fp8MatmulPlan p;
  NormGradPlan g;
  EXPECT(plan_fp8_matmul(big, 128, big, &p), big, 128, big);
  EXPECT(plan_fp8_matmul(1, big, big, &p) && p.splits == 1, 1, big, big);
  EXPECT(!plan_fp8_matmul(big, big, 1, &p), big, big, 1);
  EXPECT(!plan_fp8_matmul(big, 129, 1, &p), big, 129, 1);   // 2^24 tiles: 2^32 threads
  EXPECT(!plan_fp8_matmul(big + 1, 1, 1, &p), big + 1, 1, 1);
  EXPECT(!plan_fp8_matmul(0, 1, 1, &p) && !plan_fp8_matmul(1, 1, 0, &p), 0, 1, 1);
  EXPECT(plan_norm_grad(big, 1, &g) && !plan_norm_grad(1, 0, &g), big, 1, 0);
  printf("fp8_plan_check: %ld checks, %d failures\n", checks, failures);
  return failures == 0 ? 0 : 1;
}
