// The 8-bit product for few rows of A (a decoding step's tokens): bound by
// reading B once.
#include <type_traits>

#include "fp8_gemm.h"

namespace ortho {

namespace {

// 16 kMB rows of A against 16 rows of B per workgroup.  The kWaves waves share
// the blocks of K among them (block b goes to wave b % kWaves), hold kAhead
// blocks' loads in flight straight from memory into registers, and their sums
// are added in LDS in a fixed order.  Codes become bf16, which holds them
// exactly, whatever C's type: at this size the conversions are free.
//
// The workgroups that share 16 rows of B follow each other on one XCD
// (workgroup id mod 8), where all but the first find them in the L2.
template <bool kE8m0, int kMB, int kWaves, int kAhead>
__global__ __launch_bounds__(kWaves * 64) void fp8_few_kernel(Fp8GemmArgs p) {
  __shared__ __attribute__((aligned(16))) float part[kWaves][kMB][16][20];   // [m][n], rows 16 bytes apart in banks
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int l16 = lane & 15, lg = lane >> 4;
  const int parts = (p.M + 16 * kMB - 1) / (16 * kMB), turn = blockIdx.x >> 3;
  const int m0 = turn % parts * (16 * kMB), n0 = ((blockIdx.x & 7) + 8 * (turn / parts)) * 16;
  if (n0 >= p.N) return;
  const int nkb = (p.K + kFp8Block - 1) / kFp8Block;
  // Lane l holds codes 16 lg .. and 64 + 16 lg .. of row l16 of a block (the
  // order of k within a block is free).
  const uint8_t* const brow = p.b + (int64_t)min(n0 + l16, p.N - 1) * p.ldb;
  floatx4 acc[kMB];
#pragma unroll
  for (int i = 0; i < kMB; ++i) acc[i] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int64_t srow = min(n0 + lg * 4, p.N - 1);   // kept in bounds below, too
  bool lost = false;   // a product of scales left fp32's range
  auto step = [&](int b0, auto ahead, auto checked) __attribute__((always_inline)) {
    constexpr int kN = decltype(ahead)::value;
    uint4 rb[kN][2], ra[kN][kMB][2];
    float sa[kN][kMB], sb[kN][4];
#pragma unroll
    for (int x = 0; x < kN; ++x) {
      const int kb = b0 + x * kWaves, k = kb * 128 + lg * 16;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if constexpr (decltype(checked)::value) rb[x][h] = load_codes16(brow, k + 64 * h, p.K);
        else __builtin_memcpy(&rb[x][h], brow + k + 64 * h, 16);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (p.sb.shift != 0 && e > 0) {   // 128 rows of B share a scale, and 16 never lie in two blocks
          sb[x][e] = sb[x][0];
        } else {
          const int64_t r = (p.sb.shift != 0 ? n0 : min(static_cast<int>(srow) + e, p.N - 1)) >> p.sb.shift;
          sb[x][e] = load_scale<kE8m0>(p.sb.p, r * p.sb.ld + kb);
        }
      }
#pragma unroll
      for (int i = 0; i < kMB; ++i) {
        const int m = min(m0 + i * 16 + l16, p.M - 1);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if constexpr (decltype(checked)::value) ra[x][i][h] = load_codes16(p.a + m * p.lda, k + 64 * h, p.K);
          else __builtin_memcpy(&ra[x][i][h], p.a + m * p.lda + k + 64 * h, 16);
        }
        sa[x][i] = load_scale<kE8m0>(p.sa.p, (m >> p.sa.shift) * p.sa.ld + kb);
      }
    }
#pragma unroll
    for (int x = 0; x < kN; ++x)
#pragma unroll
      for (int i = 0; i < kMB; ++i) {
        floatx4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 ub = rb[x][h], ua = ra[x][i][h];
          s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_to_bf16(ub.x, ub.y), codes_to_bf16(ua.x, ua.y), s, 0, 0, 0);
          s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_to_bf16(ub.z, ub.w), codes_to_bf16(ua.z, ua.w), s, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float f = sa[x][i] * sb[x][e];
          lost |= leaves_range<kE8m0>(f, sa[x][i], sb[x][e]);
          acc[i][e] = fmaf(s[e], f, acc[i][e]);
        }
      }
  };
  // whole blocks without bounds checks (a check per load would make each wait
  // for the one before), then what is left of K
  const int whole = p.K / kFp8Block;
  int kb = wave;
  for (; kb + (kAhead - 1) * kWaves < whole; kb += kAhead * kWaves)
    step(kb, std::integral_constant<int, kAhead>{}, std::false_type{});
  if constexpr (kAhead > 1)
    for (; kb < whole; kb += kWaves) step(kb, std::integral_constant<int, 1>{}, std::false_type{});
  if (kb < nkb) step(kb, std::integral_constant<int, 1>{}, std::true_type{});
  if (!__any(lost)) {
#pragma unroll
    for (int i = 0; i < kMB; ++i) *reinterpret_cast<floatx4*>(&part[wave][i][l16][lg * 4]) = acc[i];
  } else {
    // with the excess of far scales in the conversions
    const Fp8GemmArgs r = args_again();
#pragma unroll 1
    for (int i = 0; i < kMB; ++i) {
      const int64_t ra = min(m0 + i * 16 + l16, r.M - 1), rb = min(n0 + l16, r.N - 1);
      floatx4 to = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      for (kb = wave; kb < nkb; kb += kWaves) {
        const float sa = load_scale<kE8m0>(r.sa.p, (ra >> r.sa.shift) * r.sa.ld + kb);
        const float by_a = __builtin_ldexpf(1.f, excess(sa));
        const float by_b = __builtin_ldexpf(1.f, excess(load_scale<kE8m0>(r.sb.p, (rb >> r.sb.shift) * r.sb.ld + kb)));
        floatx4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int k = kb * 128 + h * 64 + lg * 16;
          const uint4 a = load_codes16(r.a + ra * r.lda, k, r.K), b = load_codes16(r.b + rb * r.ldb, k, r.K);
          s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_to_bf16(b.x, b.y, by_b), codes_to_bf16(a.x, a.y, by_a), s, 0, 0, 0);
          s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_to_bf16(b.z, b.w, by_b), codes_to_bf16(a.z, a.w, by_a), s, 0, 0, 0);
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t row = min(n0 + lg * 4 + e, r.N - 1);
          to[e] = fmaf(s[e], moved(sa) * moved(load_scale<kE8m0>(r.sb.p, (row >> r.sb.shift) * r.sb.ld + kb)), to[e]);
        }
      }
      *reinterpret_cast<floatx4*>(&part[wave][i][l16][lg * 4]) = to;
    }
  }
  __syncthreads();
  for (int x = threadIdx.x; x < kMB * 256; x += kWaves * 64) {
    const int i = x >> 8, m = (x >> 4) & 15, n = x & 15;
    float v = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) v += part[w][i][m][n];
    const int64_t row = m0 + i * 16 + m;
    if (row >= p.M || n0 + n >= p.N) continue;
    if (p.add)
      v += p.add_bf ? bf16_bits_to_f32(static_cast<const uint16_t*>(p.add)[row * p.ldadd + n0 + n])
                    : static_cast<const float*>(p.add)[row * p.ldadd + n0 + n];
    if (p.c_bf) static_cast<uint16_t*>(p.c)[row * p.ldc + n0 + n] = to_bf16_bits(v);
    else static_cast<float*>(p.c)[row * p.ldc + n0 + n] = v;
  }
}

template <bool kE8m0, int kMB, int kAhead>
void by_depth(const Fp8GemmArgs& a, hipStream_t s) {
  // one wave for every kAhead blocks of K, 4 to 16
  const int tiles = (a.N + 15) / 16, parts = (a.M + 16 * kMB - 1) / (16 * kMB);
  const dim3 grid((tiles + 7) / 8 * 8 * parts);
  const int nkb = (a.K + kFp8Block - 1) / kFp8Block;
  if (nkb <= 4 * kAhead)
    hipLaunchKernelGGL((fp8_few_kernel<kE8m0, kMB, 4, kAhead>), grid, dim3(256), 0, s, a);
  else if (nkb <= 8 * kAhead)
    hipLaunchKernelGGL((fp8_few_kernel<kE8m0, kMB, 8, kAhead>), grid, dim3(512), 0, s, a);
  else
    hipLaunchKernelGGL((fp8_few_kernel<kE8m0, kMB, 16, kAhead>), grid, dim3(1024), 0, s, a);
}

template <bool kE8m0>
void by_rows(const Fp8GemmArgs& a, hipStream_t s) {
  // 16 or 32 rows of A per workgroup.  Where B's rows alone do not give every
  // CU one, 16 (24 x 2048 x 8192: 14.9 us with 32 rows, 11.7 with 16;
  // 32 x 8192 x 2048: 10.0 and 12.3 us).
  if (a.M <= 16) by_depth<kE8m0, 1, 4>(a, s);
  else if ((a.N + 15) / 16 >= 256) by_depth<kE8m0, 2, 2>(a, s);
  else by_depth<kE8m0, 1, 2>(a, s);
}

}  // namespace

hipError_t launch_fp8_few(const Fp8GemmArgs& a, hipStream_t s) {
  if (a.e8m0) by_rows<true>(a, s);
  else by_rows<false>(a, s);
  return hipGetLastError();
}

}  // namespace ortho
