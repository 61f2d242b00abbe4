// Product of 8-bit matrices with a scale for each block of 128:
//   C[i, j] = sum over blocks b of K of sa[i, b] sb[j, b] (sum over k in b of
//             a[i, k] b[j, k])  (+ Add[i, j])
//
// Which matrix instruction forms a block's sum goes by C's type.  The 8-bit one
// aligns each group of eight consecutive products to the largest of them and
// cuts what lies below 2^-13 of its power of two (measured: a product of 2^-13
// of the largest still counts, one of 2^-14 is lost, while other groups and the
// accumulator are added at full fp32 precision).  Relative to the sum that is
// about 1e-5 for normally distributed operands: far below the rounding of a
// bf16 C, but 20 times what fp32 sums reach.  An fp32 C therefore converts the
// codes to bf16 (exact) and multiplies with the bf16 instruction, whose sums
// keep fp32 precision, at half the rate.
//
// Power-of-two scales are operands of the 8-bit instruction, which then
// accumulates across blocks by itself.  With fp32 scales, and with the bf16
// instruction, a block's sum starts at zero and joins the accumulators with
// one fused multiply-add per element.
#include <limits.h>

#include "fp8_gemm.h"

namespace ortho {

namespace {

enum { kScaled = 0, kHardware = 1 };

// The units of work, tiles of C times splits of K, of this workgroup: first,
// first + step, ... below end.  Each XCD (workgroup id mod 8) gets a contiguous run
// of them, walked in groups of 4 tile rows so that what runs together shares row
// blocks in that XCD's L2.
struct Walk {
  int bm, bn, tiles_n, tiles_m, tiles, first, end, step;
  __device__ __forceinline__ Walk(const Fp8GemmArgs& p, int bm_, int bn_) : bm(bm_), bn(bn_) {
    tiles_n = (p.N + bn - 1) / bn;
    tiles_m = (p.M + bm - 1) / bm;
    tiles = tiles_n * tiles_m;
    const int units = tiles * p.splits, xcd = blockIdx.x & 7, each = units >> 3, rest = units & 7;
    const int run_first = xcd * each + min(xcd, rest);
    end = run_first + each + (xcd < rest ? 1 : 0);
    step = static_cast<int>(gridDim.x) < units ? gridDim.x >> 3 : units;
    first = run_first + (blockIdx.x >> 3);
  }
  __device__ __forceinline__ void place(int u, int& m, int& n, int& sp) const {
    sp = u / tiles;
    const int tile = u - sp * tiles, group = 4 * tiles_n, g = tile / group;
    const int gsize = min(tiles_m - g * 4, 4), in = tile - g * group, col = in / gsize;
    m = (g * 4 + in - col * gsize) * bm;
    n = col * bn;
  }
};

// Of a wave's (16 kMI) x 64 of C from row m0 and column n0 on, the rows 16 i .. 16 i +
// 15 of each bit i of `lost`, straight from memory, with what far fp32 scales have in
// excess as operands of the instruction.  kLook: `lost` is found anew.
template <int kMI, int kRanges, bool kLook, bool kLongRows>
__device__ __forceinline__ void redo_rows(const Fp8GemmArgs& p, int m0, int n0, int split, uint32_t lost) {
  const int lane = __builtin_amdgcn_mbcnt_hi(~0u, __builtin_amdgcn_mbcnt_lo(~0u, 0)), l16 = lane & 15, lg = lane >> 4;
  const int nkb = (p.K + kFp8Block - 1) / kFp8Block;
  const int kt_begin = split * p.kchunk, kt_end = min(kt_begin + p.kchunk, nkb);
  auto scale_a = [&](int64_t row, int kt) ORTHO_INLINE {
    return load_scale<false>(p.sa.p, (min(row, (int64_t)p.M - 1) >> p.sa.shift) * p.sa.ld + kt);
  };
  auto scale_b = [&](int64_t row, int kt) ORTHO_INLINE {
    return load_scale<false>(p.sb.p, (min(row, (int64_t)p.N - 1) >> p.sb.shift) * p.sb.ld + kt);
  };
  if constexpr (kLook) {
    ScaleRange<kMI / 4, kRanges> range;
#pragma unroll 1
    for (int kt = kt_begin; kt < kt_end; ++kt) {
#pragma unroll
      for (int h = 0; h < kMI / 4; ++h) range.a(h, scale_a(m0 + h * 64 + lane, kt));
      range.b(scale_b(n0 + lane, kt));
    }
    lost = range.lost();
  }
#pragma unroll 1
  for (int ij = 0; ij < kMI * 4; ++ij) {
    if (!(lost >> ij / 4 & 1)) continue;
    const int m = m0 + ij / 4 * 16 + l16, n = n0 + lg * 16 + ij % 4 * 4;
    const int row_b = n0 + l16 / 4 * 16 + l16 % 4 + ij % 4 * 4;   // the lane's of the fragment
    const uint8_t* const src_a = p.a + (int64_t)min(m, p.M - 1) * p.lda;
    const uint8_t* const src_b = p.b + (int64_t)min(row_b, p.N - 1) * p.ldb;
    auto codes = [&](const uint8_t* row, int k) ORTHO_INLINE {
      const uint4 x = kLongRows ? load_codes16_of_long_rows(row, k, p.K) : load_codes16(row, k, p.K);
      const uint4 y = kLongRows ? load_codes16_of_long_rows(row, k + 64, p.K) : load_codes16(row, k + 64, p.K);
      return intx8{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
    };
    floatx4 c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int kt = kt_begin; kt < kt_end; ++kt) {
      const int k = kt * 128 + lg * 16;
      const float a = scale_a(m, kt);
      floatx4 s = {0.f, 0.f, 0.f, 0.f};
      s = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes(src_b, k), codes(src_a, k), s, 0, 0, 0,
                                                           127 + excess(scale_b(row_b, kt)), 0, 127 + excess(a));
#pragma unroll
      for (int e = 0; e < 4; ++e) c[e] = fmaf(s[e], moved(a) * moved(scale_b(n + e, kt)), c[e]);
    }
    if (m >= p.M) continue;
    if (p.part) {
      if (n < p.N) *reinterpret_cast<floatx4*>(p.part + ((int64_t)split * p.M + m) * p.ldp + n) = c;
      continue;
    }
    if (p.add) c += load_add4(p, m, n);
    store_c4<uint16_t>(p, m, n, c);
  }
}

// A BM x BN tile of C per workgroup, kWM x kWN waves of (16 kMI) x 64.  The
// rows of B are the matrix instruction's rows and the rows of A its columns, so
// a lane holds four columns of one row of C per instruction and needs one scale
// of A per 16 rows; the scale of a 128 x 128 block of B is the same for the
// whole wave.  Which row of B is which row of instruction j is free: row
// 4 g + e is column 16 g + 4 j + e of the wave's 64, so that lane group g ends
// up with 16 consecutive columns and stores them as two 16-byte pieces (at any
// element: no alignment is needed).  C is
// written straight from the accumulators, so the LDS is free at once for the
// next copies, which overlap the stores.  (kWhole: M, N multiples of 256 and K of
// 128.  8192 x 8192 x 2048 takes 135 us with fp32 scales, 2.04 PFLOP/s, and 123
// with e8m0 ones; its C alone is 26 us of a copy's rate.  8190 rows, and with
// them one tile per workgroup and checked rows, take 146 and 133.)
//
// A k tile is one block of 128: 128-byte LDS rows of eight 16-byte chunks, two
// stages.  B's fragments and the scales of a tile sit in registers from its
// start and A's are read 16 rows at a time, so a stage empties in two steps,
// each at a barrier, and each step's copies of the tile after next go out at
// once, spread over the products that follow:
//   barrier M, before the last products of the first half of A's rows:
//     B and that half are free;  the second half has arrived
//   barrier E, before the tile's last 16 rows of products:
//     the second half is free;  the next tile's B, scales and first half have
//     arrived, and its first fragments are read under those products
// A copy thus has one and a half tiles' time to arrive, in two stages.  (With
// one barrier per tile a copy has at most one, and the 256 x 256 tiles of
// 8192^3 took 545 us.)  Copies go straight from L2 into LDS (kDma; rows at
// multiples of 16 bytes), or through registers (rows at any byte).
template <int kMode, bool kRowB, int kWM, int kWN, int kMI, int kNJ, bool kDma, bool kWhole>
__global__ __launch_bounds__(kWM * kWN * 64, 2) void fp8_gemm_kernel(Fp8GemmArgs p) {
  constexpr int kThreads = kWM * kWN * 64, BM = kWM * kMI * 16, BN = kWN * kNJ * 16;
  constexpr int kStage = (BM + BN) * 128;
  constexpr int kWaves = kWM * kWN;
  constexpr int kSlots = kMI * kNJ;
  // 8-row copies per wave and tile: B's, the first half of A's rows, the second
  constexpr int kCopyB = BN / 8 / kWaves, kCopyA = BM / 16 / kWaves, kCopies = kCopyB + 2 * kCopyA;
  // A's fragments are read kDepth groups of products ahead, so all of a half has
  // been read kDepth groups before its end: the groups behind the barriers.
  constexpr int kDepth = 2, kM = kMI / 2 - kDepth, kE = kMI - kDepth;
  static_assert(kMI % 4 == 0 && kNJ == 4, "");
  static_assert(kThreads == BM + BN && kCopyB * kWaves * 8 == BN && kCopyA * kWaves * 16 == BM, "");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * kStage];
  __shared__ __attribute__((aligned(16))) uint32_t scales[3][BM + BN];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = (wave / kWN) * (kMI * 16), wn = (wave % kWN) * (kNJ * 16);

  const Walk walk(p, BM, BN);
  const int run_end = walk.end, run_step = walk.step;   // step < units: kWhole only
  auto place_unit = [&](int u, int& m, int& n, int& sp) ORTHO_INLINE { walk.place(u, m, n, sp); };
  int unit = walk.first, m0, n0, split;
  place_unit(unit, m0, n0, split);

  const int nkb = (p.K + kFp8Block - 1) / kFp8Block;
  int kt_begin = split * p.kchunk, kt_end = min(kt_begin + p.kchunk, nkb);
  const int tail = kWhole ? 0 : p.K % kFp8Block;   // codes in the last tile, 0: all
  const int tail_kt = tail != 0 ? nkb - 1 : nkb;

  // copy g of this wave: 8 rows of the stage (A's rows, then B's), lane = 8 *
  // (row of the 8) + chunk position; g < kCopyB: B; then the halves of A (the
  // first or second 8 kMI rows of every wave)
  auto rows8 = [&](int g) ORTHO_INLINE {
    if (g < kCopyB) return BM + (wave * kCopyB + g) * 8;
    const int half = (g - kCopyB) / kCopyA, x = (wave * kCopyA + (g - kCopyB) % kCopyA) * 8;
    return x / (8 * kMI) * (16 * kMI) + half * (8 * kMI) + x % (8 * kMI);
  };
  auto place = [&](int r, int c) ORTHO_INLINE { return r < BM ? swz<false>(r, c) : swz<true>(r - BM, c); };
  const int sub = lane >> 3;
  auto chunk_of = [&](int g) ORTHO_INLINE {
    return g < kCopyB ? swz<true>(rows8(g) - BM + sub, lane & 7) : swz<false>(rows8(g) + sub, lane & 7);
  };
  auto row_of = [&](int g) ORTHO_INLINE {   // of the operand
    if (g < kCopyB) return min(n0 + rows8(g) - BM + sub, kWhole ? INT_MAX : p.N - 1);
    return min(m0 + rows8(g) + sub, kWhole ? INT_MAX : p.M - 1);
  };
  auto matrix_row = [&](int r) ORTHO_INLINE {
    if (kWhole) return r < BM ? m0 + r : n0 + r - BM;
    return r < BM ? min(m0 + r, p.M - 1) : min(n0 + r - BM, p.N - 1);
  };
  // What a lane adds to a copy's base address.  kWhole: its row of the 8, and
  // the chunk that belongs at its position (the part of swz that depends on
  // the 8 rows is uniform); otherwise rows past the matrix are the last row.
  const unsigned row_a = sub * static_cast<unsigned>(p.lda), row_b = sub * static_cast<unsigned>(p.ldb);
  const unsigned chunk_a = swz<false>(sub, lane & 7) * 16, chunk_b = swz<true>(sub, lane & 7) * 16;
  unsigned voff[kWhole ? 1 : kCopies];
  if constexpr (!kWhole) {
#pragma unroll
    for (int g = 0; g < kCopies; ++g)
      voff[g] = (g < kCopyB ? (row_of(g) - n0) * static_cast<unsigned>(p.ldb)
                            : (row_of(g) - m0) * static_cast<unsigned>(p.lda)) + chunk_of(g) * 16;
  }
  const unsigned scales0 = __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)(lds_ptr_t)(&scales[0][0]));
  const unsigned lds0 = __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)(lds_ptr_t)(smem));
  const uint8_t* a0 = uniform_ptr(p.a + (int64_t)m0 * p.lda);
  const uint8_t* b0 = uniform_ptr(p.b + (int64_t)n0 * p.ldb);
  // Before the copies of the last tile, if it is short: a chunk that is not
  // whole is taken from column 0 instead, and patch_tail replaces it.
  auto tail_offsets = [&]() ORTHO_INLINE {
    if constexpr (!kWhole)
#pragma unroll
    for (int g = 0; g < kCopies; ++g) {
      const int k = (nkb - 1) * 128 + chunk_of(g) * 16;
      voff[g] = voff[g] - chunk_of(g) * 16 + (k + 16 <= p.K ? k : 0);
    }
  };
  auto copy_group = [&](int g, int kt, int st) ORTHO_INLINE {
    const int r8 = rows8(g);
    const bool is_a = g >= kCopyB;
    const unsigned at = uniform(lds0 + st * kStage + r8 * 128);
    if constexpr (kDma && kWhole) {
      const unsigned key = is_a ? swz<false>(r8, 0) : swz<true>(r8 - BM, 0);
      const uint8_t* base = (is_a ? a0 + r8 * p.lda : b0 + (r8 - BM) * p.ldb) + (int64_t)kt * 128;
      dma16((is_a ? row_a : row_b) + ((is_a ? chunk_a : chunk_b) ^ (key * 16)), uniform_ptr(base), at);
    } else if constexpr (kDma) {
      const int64_t k0 = kt == tail_kt ? 0 : (int64_t)kt * 128;   // the last tile's offsets hold its k
      dma16(voff[g], uniform_ptr((is_a ? a0 : b0) + k0), at);
    } else {
      const uint8_t* src = g < kCopyB ? p.b + row_of(g) * p.ldb : p.a + row_of(g) * p.lda;
      *reinterpret_cast<uint4*>(smem + st * kStage + r8 * 128 + lane * 16) =
          load_codes16(src, kt * 128 + chunk_of(g) * 16, p.K);
    }
  };
  // The last tile's codes from the first chunk that is not whole on.
  auto patch_tail = [&](int st) ORTHO_INLINE {
    int r = t;
    asm volatile("" : "+v"(r));   // nothing of this is worked out ahead of the loop over k
    const int mr = matrix_row(r);
    const uint8_t* src = r < BM ? p.a + (int64_t)mr * p.lda : p.b + (int64_t)mr * p.ldb;
    uint4 u = load_codes16(src, (nkb - 1) * 128 + (tail & ~15), p.K);
#pragma unroll 1
    for (int c = tail >> 4; c < 8; ++c) {
      *reinterpret_cast<uint4*>(smem + st * kStage + (r * 8 + place(r, c)) * 16) = u;
      u = make_uint4(0, 0, 0, 0);
    }
  };

  // scales: the wave's 64 rows of the stage, one per lane (bytes as words)
  constexpr bool kByteOnly = kMode == kHardware;
  constexpr int scale_size = kByteOnly ? 1 : 4;
  const bool scales_a = wave * 64 < BM;
  const int s_shift = pick(scales_a, p.sa.shift, p.sb.shift);
  const int64_t s_ld = pick(scales_a, p.sa.ld, p.sb.ld) * scale_size;
  const uint8_t* const s_all = static_cast<const uint8_t*>(pick(scales_a, p.sa.p, p.sb.p));
  const int s_first = (scales_a ? m0 : n0) >> s_shift;
  const uint8_t* s0 = uniform_ptr(s_all + s_first * s_ld);
  const int s_at = (scales_a ? m0 : n0 - BM) + wave * 64 + lane;
  const int s_row = ((kWhole ? s_at : min(s_at, pick(scales_a, p.M, p.N) - 1)) >> s_shift) - s_first;
  auto copy_scales = [&](int kt, int st) ORTHO_INLINE {
    const uint8_t* base = s0 + (int64_t)kt * scale_size;
    if constexpr (kDma) {
      const unsigned at = uniform(scales0 + (st * (BM + BN) + wave * 64) * 4);
      base = uniform_ptr(base);
      if (scale_size == 1) dma1(s_row * static_cast<unsigned>(s_ld), base, at);
      else dma4(s_row * static_cast<unsigned>(s_ld), base, at);
    } else {
      base += s_row * s_ld;
      scales[st][wave * 64 + lane] = scale_size == 1 ? *base : *reinterpret_cast<const uint32_t*>(base);
    }
  };

  floatx4 acc[kMI][kNJ];

  // 16 rows of 128 codes: lane l takes chunks l / 16 and l / 16 + 4 of its row
  // (the order of k within a block is free, if both operands share it)
  auto chunks = [&](int row, int lo, int hi) ORTHO_INLINE {
    const uint4 x = *reinterpret_cast<const uint4*>(smem + row + lo);
    const uint4 y = *reinterpret_cast<const uint4*>(smem + row + hi);
    return intx8{(int)x.x, (int)x.y, (int)x.z, (int)x.w, (int)y.x, (int)y.y, (int)y.z, (int)y.w};
  };
  const int l16 = lane & 15, lg = lane >> 4;
  const int alo = (l16 * 8 + swz<false>(l16, lg)) * 16, ahi = (l16 * 8 + swz<false>(l16, lg + 4)) * 16;
  const int brow = l16 / 4 * 16 + l16 % 4;
  constexpr int kBStep = 4;   // rows of B between fragments (rows 4 apart within 16 share a place)
  const int blo = (brow * 8 + swz<true>(brow, lg)) * 16, bhi = (brow * 8 + swz<true>(brow, lg + 4)) * 16;
  auto frag_a = [&](int off) ORTHO_INLINE { return chunks(off, alo, ahi); };
  auto frag_b = [&](int off) ORTHO_INLINE { return chunks(off, blo, bhi); };
  const int offa = wm * 128, offb = (BM + wn) * 128;
  const uint32_t* const my_sa = &scales[0][wm + l16];
  const uint32_t* const my_sb =
      &scales[0][BM + wn + (kMode == kHardware ? brow : (kRowB ? lg * 16 : 0))];

  intx8 fa[4], fb[kNJ];
  floatx4 sum[4];                        // block sums of the last slots,
  floatx4 factor[4];                     // and what they are multiplied by
  uint32_t sa[4];                        // scales as they were copied: A's of the
  floatx4 sb[kRowB ? kNJ : 1];           // 16 rows at hand, B's of the tile
  int eb[kNJ];                           // (kHardware: bytes)
  auto load_sb = [&](int j, int buf) ORTHO_INLINE {
    if constexpr (kMode == kHardware) {
      eb[j] = my_sb[buf * (BM + BN) + j * kBStep];
    } else if constexpr (kRowB) {
      const uint4 u = *reinterpret_cast<const uint4*>(my_sb + buf * (BM + BN) + j * kBStep);
      sb[j] = floatx4{__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z), __uint_as_float(u.w)};
    } else {
      if (j == kNJ - 1) sb[0][0] = __uint_as_float(my_sb[buf * (BM + BN)]);
    }
  };

  // The copies of a tile, in this order (the waits count them): scales, B, the
  // first half of A, the second half.
  constexpr int kPerTile = 1 + kCopies;
  auto first_copies = [&](int kt, int st) ORTHO_INLINE {
    copy_scales(kt, st);
#pragma unroll
    for (int g = 0; g < kCopies; ++g) copy_group(g, kt, st);
  };
  // The k tile to be copied next, two on from the one being computed.  kWhole:
  // the next unit's follow this one's, so that its first tiles arrive under
  // this one's last products and stores.
  int ahead = kt_begin, ahead_end = kt_end, ahead_unit = unit;
  bool more = true;
  auto advance = [&]() ORTHO_INLINE {
    if (++ahead < ahead_end) return;
    if constexpr (!kWhole) {
      more = false;
    } else {
      ahead_unit += run_step;
      more = ahead_unit < run_end;
      if (!more) return;
      int m, n, sp;
      place_unit(ahead_unit, m, n, sp);
      a0 = uniform_ptr(p.a + (int64_t)m * p.lda);
      b0 = uniform_ptr(p.b + (int64_t)n * p.ldb);
      s0 = uniform_ptr(s_all + ((scales_a ? m : n) >> s_shift) * s_ld);
      ahead = sp * p.kchunk;
      ahead_end = min(ahead + p.kchunk, nkb);
    }
  };
  if (kDma && kt_begin == tail_kt) tail_offsets();
  first_copies(ahead, 0);
  advance();
  if (more) {
    if (kDma && ahead == tail_kt) tail_offsets();
    first_copies(ahead, 1);
    advance();
    sync<kPerTile>();
  } else {
    sync<0>();
  }
  if (kDma && kt_begin == tail_kt) {
    patch_tail(0);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < kDepth; ++i) {
    fa[i] = frag_a(offa + i * 2048);
    sa[i] = my_sa[i * 16];
  }
#pragma unroll
  for (int j = 0; j < kNJ; ++j) {
    fb[j] = frag_b(offb + j * kBStep * 128);
    load_sb(j, 0);
  }
  // kWhole: the stores of a unit count among the outstanding accesses like
  // copies; the three waits after them are for copies issued before them.
  constexpr int kStores = kMI * 2;
  int stores_ahead = 0;
  // (one register for both halves of the rows where B's scales take 16)
  constexpr int kRanges = kRowB ? 1 : kMI / 4;
  ScaleRange<kMI / 4, kRanges> range;   // (fp32 scales) of this unit, and the rows of
  uint32_t lost_ever = 0;               // any unit whose products left fp32's range
  float met[kMI / 4 + 1];
  int cur = 0, cur3 = 0;   // stage, and buffer of scales, of the k tile being computed

  for (;;) {
#pragma unroll
  for (int i = 0; i < kMI; ++i)
#pragma unroll
    for (int j = 0; j < kNJ; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    sum[q] = floatx4{0.f, 0.f, 0.f, 0.f};
    factor[q] = floatx4{0.f, 0.f, 0.f, 0.f};
  }
  for (int kt = kt_begin; kt < kt_end; ++kt, cur ^= 1, cur3 = cur3 == 2 ? 0 : cur3 + 1) {
    const int here = cur * kStage, next = (cur ^ 1) * kStage;
    const int next3 = cur3 == 2 ? 0 : cur3 + 1, ahead3 = next3 == 2 ? 0 : next3 + 1;
#pragma unroll
    for (int i = 0; i < kMI; ++i) {
      if (i == kM || i == kE) {
        // Since the copies that have to be here by now, one tile's worth was
        // issued; near the end there are fewer, and the wait is for all.
        if (!more) {
          sync<0>();
        } else if (kWhole && stores_ahead > 0) {
          --stores_ahead;
          sync<kPerTile + kStores>();
        } else {
          sync<kPerTile>();
        }
        if (kDma && i == kE && kt + 1 == tail_kt && kt + 1 < kt_end) {
          patch_tail(cur ^ 1);
          __syncthreads();
        }
        if (kDma && i == kM && more && ahead == tail_kt) tail_offsets();
      }
#pragma unroll
      for (int j = 0; j < kNJ; ++j) {
        const int slot = i * kNJ + j;
        if (j == 0) {
          constexpr int kLast = kMI - kDepth;
          fa[(i + kDepth) & 3] = frag_a((i < kLast ? here : next) + offa + (i + kDepth) % kMI * 2048);
          sa[(i + kDepth) & 3] = my_sa[(i < kLast ? cur3 : next3) * (BM + BN) + (i + kDepth) % kMI * 16];
        }
        if constexpr (kMode == kHardware) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa[i & 3], acc[i][j], 0, 0, 0,
                                                                       eb[j], 0, sa[i & 3]);
          const int ds = (slot + kSlots - 4) % kSlots;   // keeps the products in this order
          asm volatile("" : "+v"(acc[ds / kNJ][ds % kNJ]));
        } else {
          floatx4 s = {0.f, 0.f, 0.f, 0.f};
          s = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa[i & 3], s, 0, 0, 0, 0, 0, 0);
          // the sum of two slots ago joins its accumulators (pinned here: left
          // alone, the compiler gathers the additions at the tile's end and
          // keeps every sum alive until then)
          const int d = (slot + 2) & 3, ds = (slot + kSlots - 2) % kSlots;
          floatx4& to = acc[ds / kNJ][ds % kNJ];
#pragma unroll
          for (int e = 0; e < 4; ++e) to[e] = fmaf(sum[d][e], factor[d][kRowB ? e : 0], to[e]);
          asm volatile("" : "+v"(to));
          sum[slot & 3] = s;
          if constexpr (kRowB) {
#pragma unroll
            for (int e = 0; e < 4; ++e) factor[slot & 3][e] = __uint_as_float(sa[i & 3]) * sb[j][e];
          } else {
            factor[slot & 3][0] = __uint_as_float(sa[i & 3]) * sb[0][0];
          }
        }
        if (i == kMI - 1) {
          fb[j] = frag_b(next + offb + j * kBStep * 128);
          load_sb(j, next3);
        }
        if constexpr (kMode == kScaled) {
          // the tile's scales, read and looked at where little else is (1000 x 1537 x
          // 1111 with a scale per row of B 17.0 us, 17.6 at slots 2 and 5)
          constexpr int kReadAt = kMI == 8 ? 2 : 8;
          if (slot == kReadAt) {
            const float* const rows = reinterpret_cast<const float*>(&scales[cur3][0]);
#pragma unroll
            for (int h = 0; h < kMI / 4; ++h) met[h] = rows[wm + h * 64 + lane];
            if (kRowB) met[kMI / 4] = rows[BM + wn + lane];
          } else if (slot == kReadAt + 3) {
#pragma unroll
            for (int h = 0; h < kMI / 4; ++h) range.a(h, met[h]);
            range.b(kRowB ? met[kMI / 4] : sb[0][0]);
          }
        }
        // the copies behind barrier M, one every second or third slot, and
        // those behind barrier E
        if (more) {
          constexpr int kStep = (kE - kM) * kNJ / (1 + kCopyB + kCopyA);
          const int x = slot - kM * kNJ;
          if (x >= 0 && x % kStep == 0 && x / kStep <= kCopyB + kCopyA) {
            if (x == 0) copy_scales(ahead, ahead3);
            else copy_group(x / kStep - 1, ahead, cur);
          }
          if (i == kE) {
#pragma unroll
            for (int g = j * kCopyA / kNJ; g < (j + 1) * kCopyA / kNJ; ++g)
              copy_group(kCopyB + kCopyA + g, ahead, cur);
            if (j == kNJ - 1) advance();
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  }
  if constexpr (kMode != kHardware) {
#pragma unroll
    for (int slot = kSlots; slot < kSlots + 2; ++slot) {
      const int d = (slot + 2) & 3, ds = slot - 2;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        acc[ds / kNJ][ds % kNJ][e] = fmaf(sum[d][e], factor[d][kRowB ? e : 0], acc[ds / kNJ][ds % kNJ][e]);
    }
  }

  uint32_t lost = 0;
  if constexpr (kMode == kScaled) lost = range.lost();
  // Columns of piece j of a lane: four, next to those of piece j + 1.
  const bool whole = kWhole || n0 + wn + 64 <= p.N;
#pragma unroll
  for (int i = 0; i < kMI; ++i) {
    if (kMode == kScaled && (lost >> i & 1)) continue;   // below
    const int m = m0 + wm + i * 16 + l16;
    if (!kWhole && m >= p.M) continue;
    const int nl = n0 + wn + lg * 16;
    if (!kWhole && p.part) {
      float* o = p.part + ((int64_t)split * p.M + m) * p.ldp;
#pragma unroll
      for (int j = 0; j < kNJ; ++j)
        if (nl + j * 4 < p.N) *reinterpret_cast<floatx4*>(o + nl + j * 4) = acc[i][j];
      continue;
    }
    if (p.add) {
#pragma unroll
      for (int j = 0; j < kNJ; ++j) acc[i][j] += load_add4(p, m, nl + j * kBStep);
    }
    if (whole) {
      uint16_t* const o = static_cast<uint16_t*>(p.c) + m * p.ldc + nl;
#pragma unroll
      for (int j = 0; j < kNJ; j += 2) {
        const uint2 lo = pack_bf16x4(acc[i][j]), hi = pack_bf16x4(acc[i][j + 1]);
        const uint4 u = make_uint4(lo.x, lo.y, hi.x, hi.y);
        __builtin_memcpy(o + j * 4, &u, 16);
      }
    } else {
#pragma unroll
      for (int j = 0; j < kNJ; ++j) store_c4<uint16_t>(p, m, nl + j * 4, acc[i][j]);
    }
  }
  if constexpr (kWhole) {
    // with Add its loads were waited for, and with them all before
    stores_ahead = p.add || lost != 0 ? 0 : 3;
    lost_ever |= lost;
    range = {};
    unit += run_step;
    if (unit >= run_end) break;
    place_unit(unit, m0, n0, split);
    kt_begin = split * p.kchunk;
    kt_end = min(kt_begin + p.kchunk, nkb);
  } else {
    lost_ever = lost;
    break;
  }
  }
  if (lost_ever == 0) return;
  // After the pipeline, and from the arguments read again: nothing of this is held in
  // registers before (redone at a unit's end it cost 8192 x 8192 x 2048 12%).
  if constexpr (kMode == kScaled) {
    const Fp8GemmArgs again = args_again();
    const Walk walk(again, BM, BN);
    for (int u = walk.first; u < walk.end; u += walk.step) {
      int m, n, sp;
      walk.place(u, m, n, sp);
      redo_rows<kMI, kRanges, kWhole, kDma>(again, m + wm, n + wn, sp, lost_ever);
      if (!kWhole) break;
    }
  }
}

// C from the splits' sums: four columns per thread, the splits in order.
template <typename T>
__global__ __launch_bounds__(256) void fp8_join_kernel(Fp8GemmArgs p) {
  const int64_t quads = p.ldp / 4, x = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (x >= p.M * quads) return;
  const int64_t m = x / quads;
  const int n = static_cast<int>(x % quads) * 4;
  const float* src = p.part + m * p.ldp + n;
  floatx4 v = *reinterpret_cast<const floatx4*>(src);
#pragma unroll 4
  for (int i = 1; i < p.splits; ++i) v += *reinterpret_cast<const floatx4*>(src + i * (p.M * p.ldp));
  if (p.add) v += load_add4(p, m, n);
  store_c4<T>(p, m, n, v);
}

constexpr int kResident = 256;   // workgroups of eight waves that the chip holds at once

template <int kMode, bool kRowB, int kWM, int kWN, int kMI, int kNJ, bool kDma, bool kWhole>
void launch(const Fp8GemmArgs& a, hipStream_t s) {
  constexpr int BM = kWM * kMI * 16, BN = kWN * kNJ * 16;
  const int64_t units = (int64_t)((a.N + BN - 1) / BN) * ((a.M + BM - 1) / BM) * a.splits;
  const int64_t grid = kWhole && units > kResident ? kResident : units;
  hipLaunchKernelGGL((fp8_gemm_kernel<kMode, kRowB, kWM, kWN, kMI, kNJ, kDma, kWhole>),
                     dim3(static_cast<uint32_t>(grid)), dim3(kWM * kWN * 64), 0, s, a);
}

template <int kMode, bool kRowB>
void by_tile(const Fp8GemmArgs& a, hipStream_t s) {
  const bool whole = a.M % 256 == 0 && a.N % 256 == 0 && a.K % kFp8Block == 0;
  // (codes at any byte go through registers: 8192 x 8192 x 2047 150 us with rows at
  // multiples of 16 bytes, 476 without)
  if (!a.dma || a.K < 16) return launch<kMode, kRowB, 2, 2, 4, 4, false, false>(a, s);
  // 256 x 256 tiles from a C of 160 of them on (below, the CUs without one cost
  // more than twice the copies do: 4096 x 2048 x 2048 32.7 us with them, 25.4 on
  // 128 x 128; 4096 x 2800 x 2048 35.2 and 39.3 us, 8192^3 486 and 645).  The rule
  // looks at the area alone: where M or N is under 256, parts of the tiles are
  // empty (96 x 131072 x 2048: 77 us, 65 on 128 x 128).
  if ((int64_t)a.M * a.N >= 256 * 256 * 160) {
    if (whole) return launch<kMode, kRowB, 2, 4, 8, 4, true, true>(a, s);
    return launch<kMode, kRowB, 2, 4, 8, 4, true, false>(a, s);
  }
  launch<kMode, kRowB, 2, 2, 4, 4, true, false>(a, s);
}

}  // namespace

hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, hipStream_t s) {
  if (a.e8m0) by_tile<kHardware, false>(a, s);
  else if (a.sb.shift == 0) by_tile<kScaled, true>(a, s);
  else by_tile<kScaled, false>(a, s);
  return hipGetLastError();
}

hipError_t launch_fp8_matmul(const Fp8GemmArgs& a, hipStream_t s) {
  // (from 2^25 rows of B on its launch could pass 2^32 threads)
  if (a.M <= kFewRows && a.N < 1 << 25) return launch_fp8_few(a, s);
  const hipError_t e = a.c_bf ? launch_fp8_gemm(a, s) : launch_fp8_exact(a, s);
  if (e != hipSuccess || a.splits == 1) return e;
  const int64_t quads = (int64_t)a.M * (a.ldp / 4);
  const dim3 grid(static_cast<uint32_t>((quads + 255) / 256));
  if (a.c_bf) hipLaunchKernelGGL(fp8_join_kernel<uint16_t>, grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL(fp8_join_kernel<float>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace ortho
