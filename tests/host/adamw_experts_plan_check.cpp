// Host-only check of the plans and of the overlap test behind AdamW and the tokens by
// expert (plan.cpp), built with g++ under AddressSanitizer and
// UndefinedBehaviorSanitizer by tests/test_adamw_experts_plan_sanitized.py.
#include <stdio.h>

#include <random>
#include <set>
#include <vector>

#include "plan.h"

using namespace ortho;

static long checks = 0;
static int failures = 0;
#define EXPECT(cond, ...)                          \
  do {                                             \
    ++checks;                                      \
    if (!(cond)) {                                 \
      if (++failures < 20) {                       \
        fprintf(stderr, "FAIL %s: ", #cond);       \
        fprintf(stderr, __VA_ARGS__);              \
        fprintf(stderr, "\n");                     \
      }                                            \
    }                                              \
  } while (0)

// Every element of a matrix belongs to one thread's piece, none to two.
static void check_deal(int64_t rows, int64_t cols, int64_t piece, int64_t slack = 8) {
  const Deal d = deal(rows, cols, piece, slack);
  EXPECT(d.lanes >= 4 && d.lanes <= 8, "%lld x %lld", (long long)rows, (long long)cols);
  const int64_t wide = piece << d.lanes, high = 256 >> d.lanes;
  EXPECT(d.across * wide >= cols && (d.across - 1) * wide < cols, "%lld", (long long)cols);
  EXPECT(d.units == d.across * ((rows + high - 1) / high), "%lld", (long long)rows);
  const int64_t least = (cols + 16 * piece - 1) / (16 * piece) * 16 * piece;
  EXPECT(d.across * wide <= least + least / slack, "%lld", (long long)cols);
  // (32-bit numbers in the kernels on up to 2^40 elements; pieces of bytes count in 64)
  if (piece >= 8 && rows <= kMaxElements / cols) EXPECT(d.units < int64_t{1} << 31 && d.across < int64_t{1} << 31, "units");
}

static ortho_mat mat(uintptr_t at, int64_t rows, int64_t cols, int64_t ld, int32_t dtype) {
  return {reinterpret_cast<void*>(at), rows, cols, ld, dtype};
}

// The bytes of a small matrix.
static std::set<uintptr_t> bytes(const ortho_mat& a) {
  std::set<uintptr_t> s;
  const int64_t e = a.dtype == ORTHO_F32 ? 4 : (a.dtype == ORTHO_BF16 ? 2 : 1);
  for (int64_t r = 0; r < a.rows; ++r)
    for (int64_t b = 0; b < a.cols * e; ++b) s.insert(reinterpret_cast<uintptr_t>(a.data) + r * a.ld * e + b);
  return s;
}

static bool meet(const std::set<uintptr_t>& a, const std::set<uintptr_t>& b) {
  for (uintptr_t x : a)
    if (b.count(x)) return true;
  return false;
}

int main() {
  const std::vector<int64_t> sizes = {1,    2,    7,    8,    15,   16,   127,  128,   129,   255,    256,    257,    511,
                                      512,  513,  1023, 1024, 1025, 2001, 2047, 2048,  2049,  2056,   4096,   4097,   8192,
                                      8193, 1 << 20, (1 << 20) + 1, 1 << 30};
  for (int64_t r : sizes)
    for (int64_t c : sizes)
      for (int64_t p : {1, 8, 32}) {
        check_deal(r, c, p);
        check_deal(r, c, p, 4);
      }
  check_deal(1, kMaxElements, 8);
  check_deal(1, kMaxElements, 32);

  for (int64_t tokens : {1, 2, 511, 512, 513, 4096, 4097, 131072, 1 << 20, (1 << 30) - 1})
    for (int32_t choices : {1, 2, 8, 64})
      for (int32_t experts : {1, 5, 64, 1023, 1024}) {
        ExpertSortPlan p;
        const bool ok = plan_expert_sort(tokens, choices, experts, &p);
        EXPECT(ok == (tokens * choices < (int64_t{1} << 30)), "%lld", (long long)tokens);
        if (!ok) continue;
        EXPECT(p.pairs == tokens * choices && p.tile % 1024 == 0 && p.tiles >= 1 && p.tiles <= 1024, "plan");
        EXPECT((int64_t)p.tiles * p.tile >= p.pairs && (int64_t)(p.tiles - 1) * p.tile < p.pairs, "cover");
        EXPECT(p.total_bytes % kWsAlign == 0 && (p.tiles == 1 || p.total_bytes >= (size_t)p.tiles * experts * 4), "ws");
        for (int32_t align : {1, 3, 128, 4096}) {
          const int64_t rows = expert_rows(tokens, choices, experts, align);
          const int64_t want = tokens * choices + (int64_t)experts * (align - 1);
          EXPECT(rows == (want < (int64_t{1} << 30) ? want : 0), "rows");
        }
      }

  // Random small tensors in a small memory: refused as overlapping exactly if a byte that
  // one writes is another's too.
  std::mt19937 rng(7);
  auto pick = [&](int64_t lo, int64_t hi) { return lo + (int64_t)(rng() % (uint64_t)(hi - lo + 1)); };
  ortho_adamw h{};
  h.lr = 0.1;
  h.beta1 = 0.9;
  h.beta2 = 0.99;
  h.eps = 1e-8;
  h.step = 1;
  long refused = 0, taken = 0;
  for (int round = 0; round < 3000; ++round) {
    const int count = (int)pick(1, 20);   // (more than 64 matrices: the list that is allocated)
    const int64_t room = count * pick(400, 6000);
    std::vector<ortho_mat> l[6];
    std::vector<std::set<uintptr_t>> written, read;
    const bool slices = pick(0, 3) == 0;   // columns of one wide matrix
    const int64_t wide = 4 * count * 5;
    for (int i = 0; i < count; ++i) {
      const int64_t rows = pick(1, 4), cols = slices ? pick(3, 5) : pick(1, 9);
      const int32_t s = pick(0, 1) ? ORTHO_E4M3 : ORTHO_F32;
      for (int k = 0; k < 6; ++k) {
        const int32_t type = k < 2 ? (pick(0, 1) ? ORTHO_F32 : ORTHO_BF16) : (k < 4 ? s : ORTHO_F32);
        const int64_t c = k < 4 ? cols : 1;
        ortho_mat a = mat(0x10000 + (uintptr_t)(k * room + pick(0, room)), rows, c, c + pick(0, 6), type);
        if (slices && k == 0) a = mat(0x10000 + (uintptr_t)(4 * (5 * i) + (pick(0, 40) ? 0 : 4)), rows, 4, wide, ORTHO_F32);
        if (slices && k != 0 && k < 4) a = mat(0x10000 + (uintptr_t)(k * 1000000 + i * 10000), rows, 4, 4, k < 2 ? type : s);
        if (slices && k >= 4) a = mat(0x10000 + (uintptr_t)(k * 1000000 + i * 10000), rows, 1, 1, ORTHO_F32);
        l[k].push_back(a);
        if (k >= 4 && s == ORTHO_F32) continue;
        (k == 1 ? read : written).push_back(bytes(a));
      }
    }
    bool clash = false;
    for (size_t i = 0; i < written.size(); ++i) {
      for (size_t j = 0; j < i; ++j) clash |= meet(written[i], written[j]);
      for (const auto& r : read) clash |= meet(written[i], r);
    }
    const ortho_status st = validate_adamw(count, l[0].data(), l[1].data(), l[2].data(), l[3].data(), l[4].data(), l[5].data(), &h);
    // (rows that lie between rows of another pitch are refused, too)
    bool between = false;
    for (size_t i = 0; i < written.size(); ++i)
      for (size_t j = 0; j < written.size() + read.size(); ++j) {
        const auto& a = written[i];
        const auto& b = j < written.size() ? written[j] : read[j - written.size()];
        between |= i != j && !slices && *a.begin() <= *b.rbegin() && *b.begin() <= *a.rbegin();
      }
    if (clash || !between) EXPECT(st == (clash ? ORTHO_E_LAYOUT : ORTHO_OK), "round %d: status %d, clash %d", round, (int)st, (int)clash);
    (clash ? refused : taken)++;
  }
  EXPECT(refused > 300 && taken > 300, "refused %ld, taken %ld", refused, taken);
  // the largest descriptors: extents beyond 64 bits
  const ortho_mat big = mat(0x10000, 1 << 30, 4, (int64_t{1} << 32) - 64, ORTHO_F32);
  const ortho_mat far = mat(0x20000, 1 << 30, 4, (int64_t{1} << 32) - 64, ORTHO_F32), m = mat(0x30000, 1 << 30, 4, (int64_t{1} << 32) - 64, ORTHO_F32),
                  v = mat(0x40000, 1 << 30, 4, (int64_t{1} << 32) - 64, ORTHO_F32);
  EXPECT(validate_adamw(1, &big, &far, &m, &v, nullptr, nullptr, &h) == ORTHO_OK, "far");
  EXPECT(validate_adamw(1, &big, &far, &m, &far, nullptr, nullptr, &h) == ORTHO_E_LAYOUT, "far");
  const ortho_mat further = mat(0x20000, 1 << 30, 4, int64_t{1} << 32, ORTHO_F32);
  EXPECT(validate_adamw(1, &big, &further, &m, &v, nullptr, nullptr, &h) == ORTHO_E_LAYOUT, "further");
  printf("%ld checks, %d failures\n", checks, failures);
  return failures != 0;
}
