// The 8-bit product with an fp32 C: every product counts in full (the 8-bit
// matrix instruction would cut small ones; kernels_fp8_gemm.hip), so the codes
// are converted to bf16, which holds them exactly, and multiplied with the bf16
// instruction, whose sums keep fp32 precision.  A block of 128 is summed from
// zero, scaled in fp32 and added to the accumulators.
#include "fp8_gemm.h"

namespace ortho {

namespace {

// 128 x 128 of C per workgroup, 64 x 64 per wave as 2 x 2 of 32 x 32 x 16
// instructions (B's rows are the instruction's rows: a lane holds groups of
// four columns of one row of C).  Two workgroups share a CU, so that one's
// conversions and block ends run under the other's products: per block of 128
// a wave has 32 products (1024 cycles of the matrix core) and 128 conversions
// and 64 or 128 scalings (768 or 1024 cycles of the vector unit).
//
// A k tile is one block, 128-byte LDS rows of eight chunks (swz), two stages.
// A lane takes chunks 4 h .. 4 h + 3 of its row (h = lane / 32; the order of k
// within a block is free), one chunk ahead of the products.  The barrier sits
// before the last chunk's products: the stage is then free, and the copies of
// the tile after next have a whole tile's time to arrive.
//
// 8192 x 2048 x 8192 takes 252 us with fp32 or e8m0 scales, 1.09 PFLOP/s, and 285
// (e8m0 318) where B has a scale per row, with the matrix cores busy 43% of it.
template <bool kE8m0, bool kRowB, bool kDma>
__global__ __launch_bounds__(256, 2) void fp8_exact_kernel(Fp8GemmArgs p) {
  constexpr int BM = 128, BN = 128, kStage = (BM + BN) * 128, kCopies = 8;
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStage];
  __shared__ __attribute__((aligned(16))) uint32_t scales[3][BM + BN];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;

  const int nkb = (p.K + kFp8Block - 1) / kFp8Block;
  // Each XCD (workgroup id mod 8) gets a contiguous run of units (tiles of C
  // times splits of K), walked in groups of 8 tile rows.
  const int tiles_n = (p.N + BN - 1) / BN, tiles_m = (p.M + BM - 1) / BM;
  const int tiles = tiles_n * tiles_m, units = tiles * p.splits;
  const int xcd = blockIdx.x & 7, each = units >> 3, rest = units & 7;
  const int unit = xcd * each + min(xcd, rest) + (blockIdx.x >> 3);
  const int split = unit / tiles, tile = unit - split * tiles;
  const int group = 8 * tiles_n, first_m = tile / group * 8, gsize = min(tiles_m - first_m, 8);
  const int in = tile % group;
  const int m0 = (first_m + in % gsize) * BM, n0 = in / gsize * BN;
  const int kt_begin = split * p.kchunk, kt_end = min(kt_begin + p.kchunk, nkb);
  const int tail = p.K % kFp8Block, tail_kt = tail != 0 ? nkb - 1 : nkb;

  // copy g of this wave: rows 8 (8 wave + g) .. + 7 of the stage (A's, then
  // B's); lane = 8 * (row of the 8) + chunk position
  const bool is_a = wave < 2;
  const int last = pick(is_a, p.M, p.N) - 1, row0 = is_a ? m0 : n0 - BM;
  const int64_t ld = pick(is_a, p.lda, p.ldb);
  const uint8_t* const matrix = pick(is_a, p.a, p.b);
  auto stage_row = [&](int g) ORTHO_INLINE { return (wave * 8 + g) * 8 + (lane >> 3); };
  auto matrix_row = [&](int r) ORTHO_INLINE { return min(row0 + r, last); };
  auto chunk_of = [&](int g) ORTHO_INLINE { return swz<false>(stage_row(g), lane & 7); };
  const int from = min(row0 + wave * 64, last);
  const uint8_t* const base = uniform_ptr(matrix + (int64_t)from * ld);
  unsigned voff[kCopies];
#pragma unroll
  for (int g = 0; g < kCopies; ++g)
    voff[g] = (matrix_row(stage_row(g)) - from) * static_cast<unsigned>(ld) + chunk_of(g) * 16;
  const unsigned lds0 = uniform((unsigned)(uintptr_t)(lds_ptr_t)(smem));
  const unsigned scales0 = uniform((unsigned)(uintptr_t)(lds_ptr_t)(&scales[0][0]));
  // scales: the wave's 64 rows of the stage, one per lane (bytes as words)
  const int shift = pick(is_a, p.sa.shift, p.sb.shift);
  const int64_t s_ld = pick(is_a, p.sa.ld, p.sb.ld) * (kE8m0 ? 1 : 4);
  const uint8_t* const s_base =
      uniform_ptr(static_cast<const uint8_t*>(pick(is_a, p.sa.p, p.sb.p)) + (from >> shift) * s_ld);
  const int s_row = (matrix_row(wave * 64 + lane) >> shift) - (from >> shift);

  auto copy_scales = [&](int kt, int buf) ORTHO_INLINE {
    const uint8_t* src = s_base + (int64_t)kt * (kE8m0 ? 1 : 4);
    if constexpr (kDma) {
      const unsigned at = uniform(scales0 + (buf * (BM + BN) + wave * 64) * 4);
      const unsigned off = s_row * static_cast<unsigned>(s_ld);
      if constexpr (kE8m0) dma1(off, uniform_ptr(src), at);
      else dma4(off, uniform_ptr(src), at);
    } else {
      src += s_row * s_ld;
      scales[buf][wave * 64 + lane] = kE8m0 ? *src : *reinterpret_cast<const uint32_t*>(src);
    }
  };
  auto copy = [&](int g, int kt, int st) ORTHO_INLINE {
    if constexpr (kDma) {
      const int64_t k0 = kt == tail_kt ? 0 : (int64_t)kt * 128;   // the short tile's offsets hold its k
      dma16(voff[g], uniform_ptr(base + k0), uniform(lds0 + st * kStage + (wave * 8 + g) * 1024));
    } else {
      *reinterpret_cast<uint4*>(smem + st * kStage + (wave * 8 + g) * 1024 + lane * 16) =
          load_codes16(matrix + matrix_row(stage_row(g)) * ld, kt * 128 + chunk_of(g) * 16, p.K);
    }
  };
  // Before the copies of a short last tile: a chunk that is not whole is taken
  // from column 0 instead, and patch_tail replaces it.
  auto tail_offsets = [&]() ORTHO_INLINE {
#pragma unroll
    for (int g = 0; g < kCopies; ++g) {
      const int k = (nkb - 1) * 128 + chunk_of(g) * 16;
      voff[g] = voff[g] - chunk_of(g) * 16 + (k + 16 <= p.K ? k : 0);
    }
  };
  auto patch_tail = [&](int st) ORTHO_INLINE {
    int r = wave * 64 + lane;
    asm volatile("" : "+v"(r));   // nothing of this is worked out ahead of the loop over k
    uint4 u = load_codes16(matrix + matrix_row(r) * ld, (nkb - 1) * 128 + (tail & ~15), p.K);
#pragma unroll 1
    for (int c = tail >> 4; c < 8; ++c) {
      *reinterpret_cast<uint4*>(smem + st * kStage + (r * 8 + swz<false>(r, c)) * 16) = u;
      u = make_uint4(0, 0, 0, 0);
    }
  };
  auto scale_value = [&](uint32_t u) ORTHO_INLINE {
    if constexpr (kE8m0) u = u == 0 ? 0x00400000u : (u == 255 ? 0x7fc00000u : u << 23);
    return __uint_as_float(u);
  };

  // fragment f: rows 32 f .. of the wave's 64 of A (f = 0, 1) or B (2, 3)
  const int l32 = lane & 31, half = lane >> 5;
  auto chunk = [&](int st, int f, int q) ORTHO_INLINE {
    const int r = (f < 2 ? wm : BM + wn - 64) + f * 32 + l32;
    return *reinterpret_cast<const uint4*>(smem + st * kStage + (r * 8 + swz<false>(l32, half * 4 + q)) * 16);
  };

  floatx16 acc[2][2], sum[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.f;

  auto all_copies = [&](int kt, int st) ORTHO_INLINE {
    if (kDma && kt == tail_kt) tail_offsets();
    copy_scales(kt, st);
#pragma unroll
    for (int g = 0; g < kCopies; ++g) copy(g, kt, st);
  };
  all_copies(kt_begin, 0);
  if (kt_begin + 1 < kt_end) {
    all_copies(kt_begin + 1, 1);
    sync<1 + kCopies>();
  } else {
    sync<0>();
  }
  if (kDma && kt_begin == tail_kt) {
    patch_tail(0);
    __syncthreads();
  }
  uint4 raw[2][4];
#pragma unroll
  for (int f = 0; f < 4; ++f) raw[0][f] = chunk(0, f, 0);

  ScaleRange<1, 1> range;          // where B's rows have scales of their own
  bool left[2] = {false, false};   // elsewhere: whether a product of scales left fp32's range
  int cur = 0, cur3 = 0;   // stage, and buffer of scales, of the tile being computed
  for (int kt = kt_begin; kt < kt_end; ++kt) {
    const int ahead3 = cur3 == 0 ? 2 : cur3 - 1;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q == 3) {
        sync<0>();
        if (kDma && kt + 1 == tail_kt && kt + 1 < kt_end) {
          patch_tail(cur ^ 1);
          __syncthreads();
        }
        if (kDma && kt + 2 == tail_kt && kt + 2 < kt_end) tail_offsets();
      }
#pragma unroll
      for (int f = 0; f < 4; ++f) raw[(q + 1) & 1][f] = q < 3 ? chunk(cur, f, q + 1) : chunk(cur ^ 1, f, 0);
      // (the reads stay ahead of the products that hide them)
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        bf16x8 x[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) {
          const uint4 u = raw[q & 1][f];
          x[f] = codes_to_bf16(s ? u.z : u.x, s ? u.w : u.y);
        }
        if (q == 3 && kt + 2 < kt_end) {
          if (s == 0) copy_scales(kt + 2, ahead3);
#pragma unroll
          for (int g = 0; g < kCopies / 2; ++g) copy(s * (kCopies / 2) + g, kt + 2, cur);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            if (q == 0 && s == 0) {
              floatx16 z;
#pragma unroll
              for (int e = 0; e < 16; ++e) z[e] = 0.f;
              sum[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[2 + j], x[i], z, 0, 0, 0);
            } else {
              sum[i][j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(x[2 + j], x[i], sum[i][j], 0, 0, 0);
            }
          }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    // the block's sums, scaled
    float sa[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) sa[i] = scale_value(scales[cur3][wm + i * 32 + l32]);
    if constexpr (kRowB) {
      range.a(0, scale_value(scales[cur3][wm + lane]));
      range.b(scale_value(scales[cur3][BM + wn + lane]));
    } else {
      const float sb = scale_value(scales[cur3][BM + wn]);
#pragma unroll
      for (int i = 0; i < 2; ++i) left[i] |= leaves_range<kE8m0>(sa[i] * sb, sa[i], sb);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        floatx4 sb;
        if constexpr (kRowB) {
          const uint4 u = *reinterpret_cast<const uint4*>(&scales[cur3][BM + wn + j * 32 + g * 8 + half * 4]);
          sb = floatx4{scale_value(u.x), scale_value(u.y), scale_value(u.z), scale_value(u.w)};
        } else {
          const float v = scale_value(scales[cur3][BM + wn]);
          sb = floatx4{v, v, v, v};
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            acc[i][j][g * 4 + e] = fmaf(sum[i][j][g * 4 + e], sa[i] * sb[e], acc[i][j][g * 4 + e]);
      }
    cur ^= 1;
    cur3 = cur3 == 2 ? 0 : cur3 + 1;
  }

  // What a lane holds of one 32 x 32 of C: four columns in four places.
  auto store = [&](const Fp8GemmArgs& to, int i, int j, const floatx16& c) ORTHO_INLINE {
    const int m = m0 + wm + i * 32 + l32;
    if (m >= to.M) return;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int n = n0 + wn + j * 32 + g * 8 + half * 4;
      floatx4 v = {c[g * 4], c[g * 4 + 1], c[g * 4 + 2], c[g * 4 + 3]};
      if (to.part) {   // rows of whole quads
        if (n < to.N)
          *reinterpret_cast<floatx4*>(to.part + ((int64_t)split * to.M + m) * to.ldp + n) = v;
        continue;
      }
      if (to.add) v += load_add4(to, m, n);
      store_c4<float>(to, m, n, v);
    }
  };
  bool lost[2];
  if constexpr (kRowB) {
    const uint32_t rows = range.lost();
    lost[0] = (rows & 3) != 0;
    lost[1] = (rows & 12) != 0;
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) lost[i] = __any(left[i]);
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if (lost[i]) continue;
#pragma unroll
    for (int j = 0; j < 2; ++j) store(p, i, j, acc[i][j]);
  }
  if (!lost[0] && !lost[1]) return;
  // Straight from memory, with the excess of far scales in the conversions.
  const Fp8GemmArgs r = args_again();
#pragma unroll 1
  for (int ij = 0; ij < 4; ++ij) {
    const int i = ij >> 1, j = ij & 1;
    if (!(i == 0 ? lost[0] : lost[1])) continue;
    const int64_t ra = min(m0 + wm + i * 32 + l32, r.M - 1), rb = min(n0 + wn + j * 32 + l32, r.N - 1);
    floatx16 to;
#pragma unroll
    for (int e = 0; e < 16; ++e) to[e] = 0.f;
#pragma unroll 1
    for (int kt = kt_begin; kt < kt_end; ++kt) {
      const float sa = load_scale<kE8m0>(r.sa.p, (ra >> r.sa.shift) * r.sa.ld + kt);
      const float by_a = __builtin_ldexpf(1.f, excess(sa));
      const float by_b = __builtin_ldexpf(1.f, excess(load_scale<kE8m0>(r.sb.p, (rb >> r.sb.shift) * r.sb.ld + kt)));
      floatx16 s;
#pragma unroll
      for (int e = 0; e < 16; ++e) s[e] = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int k = kt * 128 + (half * 4 + q) * 16;
        const uint4 a = kDma ? load_codes16_of_long_rows(r.a + ra * r.lda, k, r.K) : load_codes16(r.a + ra * r.lda, k, r.K);
        const uint4 b = kDma ? load_codes16_of_long_rows(r.b + rb * r.ldb, k, r.K) : load_codes16(r.b + rb * r.ldb, k, r.K);
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(codes_to_bf16(b.x, b.y, by_b), codes_to_bf16(a.x, a.y, by_a), s, 0, 0, 0);
        s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(codes_to_bf16(b.z, b.w, by_b), codes_to_bf16(a.z, a.w, by_a), s, 0, 0, 0);
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t n = min(n0 + wn + j * 32 + (e >> 2) * 8 + half * 4 + (e & 3), r.N - 1);
        const float sb = load_scale<kE8m0>(r.sb.p, (n >> r.sb.shift) * r.sb.ld + kt);
        to[e] = fmaf(s[e], moved(sa) * moved(sb), to[e]);
      }
    }
    store(r, i, j, to);
  }
}

template <bool kE8m0, bool kRowB>
void launch(const Fp8GemmArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)((a.N + 127) / 128) * ((a.M + 127) / 128) * a.splits;
  const dim3 grid(static_cast<uint32_t>(units));
  if (a.dma && a.K >= 16) hipLaunchKernelGGL((fp8_exact_kernel<kE8m0, kRowB, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((fp8_exact_kernel<kE8m0, kRowB, false>), grid, dim3(256), 0, s, a);
}

}  // namespace

hipError_t launch_fp8_exact(const Fp8GemmArgs& a, hipStream_t s) {
  const bool row_b = a.sb.shift == 0;
  if (a.e8m0) row_b ? launch<true, true>(a, s) : launch<true, false>(a, s);
  else row_b ? launch<false, true>(a, s) : launch<false, false>(a, s);
  return hipGetLastError();
}

}  // namespace ortho
