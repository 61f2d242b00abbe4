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
#include "fp8.h"

namespace ortho {

namespace {

typedef int intx8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

enum { kScaled = 0, kHardware = 1, kExact = 2 };

// Eight codes as eight bf16 (exact; the NaN code gives NaN).
__device__ __forceinline__ bf16x8 codes_to_bf16(int lo, int hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ int swz(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// 16 bytes per lane from global memory into LDS at lds + 16 * lane.  lds must
// be wave-uniform.  The compiler does not look inside the assembly for
// hazards, so it carries its own wait states: five before anything in it (a
// vector instruction that wrote an SGPR the load reads needs five before a
// vector memory instruction), and one between the M0 write and the load.  The
// caller waits (vmcnt) before the LDS is read.
__device__ __forceinline__ void dma16(unsigned voff, const uint8_t* sbase, unsigned lds) {
  asm volatile("s_nop 4\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
               :: "v"(voff), "s"(sbase), "s"(lds) : "memory");
}

__device__ __forceinline__ const uint8_t* uniform_ptr(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const uint8_t*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// 16 codes from column k of a row; zero codes from column K on.  Any byte.
__device__ __forceinline__ uint4 load_codes16(const uint8_t* row, int k, int K) {
  uint4 u = make_uint4(0, 0, 0, 0);
  if (k + 16 <= K) {
    __builtin_memcpy(&u, row + k, 16);
    return u;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (k + j < K) w[j >> 2] |= static_cast<uint32_t>(row[k + j]) << (8 * (j & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A BM x BN tile of C per workgroup, kWM x kWN waves of (16 kMI) x (16 kNJ).
// The rows of B are the matrix instruction's rows and the rows of A its
// columns, so a lane holds four consecutive columns of one row of C and needs
// one scale of A per 16 rows; the scale of a 128 x 128 block of B is the same
// for the whole wave.
//
// A k tile is one block of 128: 128-byte LDS rows of eight 16-byte chunks,
// chunk c of row r at c ^ ((r >> 1) & 7) so that 16 consecutive rows hit 64
// distinct banks.  Two stages.  The barrier of a tile sits before its last row
// of products, when the last fragments are in registers: the copies of the
// tile after next and the next tile's first fragment reads go out under those
// products, and a copy has a whole tile's time to arrive.  Copies go straight
// from L2 into LDS (kDma; rows at multiples of 16 bytes) or through registers
// (rows at any byte).
template <int kMode, bool kRowB, int kWM, int kWN, int kMI, int kNJ, bool kDma>
__global__ __launch_bounds__(kWM * kWN * 64, 2) void fp8_gemm_kernel(Fp8GemmArgs p) {
  constexpr int kThreads = kWM * kWN * 64, BM = kWM * kMI * 16, BN = kWN * kNJ * 16;
  constexpr int kStage = (BM + BN) * 128;
  constexpr int kGroups = (BM + BN) / 8 / (kWM * kWN);   // 8-row copies per wave and tile
  constexpr int kSlots = kMI * kNJ;
  constexpr int kScaleRows = (BM + BN + kThreads - 1) / kThreads;
  // The result leaves through LDS in kPasses passes of BM / kPasses rows.
  constexpr int kPasses = BM * BN * 4 > 2 * kStage + BM * 16 ? 2 : 1;
  constexpr int kOutRow = BN + 4;                         // floats; rows 16 bytes apart in banks
  constexpr int kOutBytes = BM / kPasses * kOutRow * 4;
  constexpr int kLds = kOutBytes > 2 * kStage ? kOutBytes : 2 * kStage;
  static_assert(kSlots % 4 == 0 && kMI % kPasses == 0, "");
  static_assert(kThreads <= BM + BN && (BM + BN) % kThreads == 0, "");
  __shared__ __attribute__((aligned(1024))) uint8_t smem[kLds];
  __shared__ __attribute__((aligned(16))) float scales[2][BM + BN];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int wm = (wave / kWN) * (kMI * 16), wn = (wave % kWN) * (kNJ * 16);

  // Each XCD (workgroup id mod 8) gets a contiguous run of tiles, walked in
  // groups of 4 tile rows, so that a run shares row blocks in that XCD's L2.
  const int tiles_n = (p.N + BN - 1) / BN, tiles_m = (p.M + BM - 1) / BM;
  const int nwg = tiles_n * tiles_m;
  int tile = blockIdx.x % nwg;
  const int split = blockIdx.x / nwg;
  {
    const int xcd = tile & 7, each = nwg >> 3, rest = nwg & 7;
    tile = xcd * each + min(xcd, rest) + (tile >> 3);
  }
  const int group = 4 * tiles_n, first_m = (tile / group) * 4, gsize = min(tiles_m - first_m, 4);
  const int m0 = (first_m + (tile % group) % gsize) * BM, n0 = ((tile % group) / gsize) * BN;

  const int nkb = (p.K + kFp8Block - 1) / kFp8Block;
  const int kt_begin = split * p.kchunk, kt_end = min(kt_begin + p.kchunk, nkb);
  const int tail = p.K % kFp8Block;   // codes in the last tile, 0: all
  const int tail_kt = tail != 0 ? nkb - 1 : nkb;

  // copies: group g of this wave is rows 8 (wave kGroups + g) .. + 7 of the
  // stage (A's rows, then B's); lane = 8 * (row of the group) + chunk position
  auto row_of = [&](int g) { return (wave * kGroups + g) * 8 + (lane >> 3); };
  auto chunk_of = [&](int g) { return swz(row_of(g), lane & 7); };
  auto matrix_row = [&](int r) { return r < BM ? min(m0 + r, p.M - 1) : min(n0 + r - BM, p.N - 1); };
  unsigned voff[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const int r = row_of(g), mr = matrix_row(r);
    voff[g] = static_cast<unsigned>(r < BM ? (mr - m0) * p.lda : (mr - n0) * p.ldb) + chunk_of(g) * 16;
  }
  const unsigned lds0 = __builtin_amdgcn_readfirstlane((unsigned)(uintptr_t)(lds_ptr_t)(smem));
  const uint8_t* const a0 = uniform_ptr(p.a + (int64_t)m0 * p.lda);
  const uint8_t* const b0 = uniform_ptr(p.b + (int64_t)n0 * p.ldb);
  // Before the copies of the last tile, if it is short: a chunk that is not
  // whole is taken from column 0 instead, and patch_tail replaces it.
  auto tail_offsets = [&]() {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const int k = (nkb - 1) * 128 + chunk_of(g) * 16;
      voff[g] = voff[g] - chunk_of(g) * 16 + (k + 16 <= p.K ? k : 0);
    }
  };
  auto copy_group = [&](int g, int kt, int st) {
    const int r8 = (wave * kGroups + g) * 8;
    if constexpr (kDma) {
      const int64_t k0 = kt == tail_kt ? 0 : (int64_t)kt * 128;   // the last tile's offsets hold its k
      dma16(voff[g], (r8 < BM ? a0 : b0) + k0, lds0 + st * kStage + r8 * 128);
    } else {
      const int r = row_of(g), mr = matrix_row(r);
      const uint8_t* src = r < BM ? p.a + (int64_t)mr * p.lda : p.b + (int64_t)mr * p.ldb;
      *reinterpret_cast<uint4*>(smem + st * kStage + r8 * 128 + lane * 16) =
          load_codes16(src, kt * 128 + chunk_of(g) * 16, p.K);
    }
  };
  auto copy_tile = [&](int kt, int st) {
    if (kDma && kt == tail_kt) tail_offsets();
#pragma unroll
    for (int g = 0; g < kGroups; ++g) copy_group(g, kt, st);
  };
  // The last tile's codes from the first chunk that is not whole on.
  auto patch_tail = [&](int st) {
#pragma unroll 1
    for (int x = t; x < (BM + BN) * 8; x += kThreads) {
      const int r = x >> 3, c = x & 7;
      if (c < (tail >> 4)) continue;
      const int mr = matrix_row(r);
      const uint8_t* src = r < BM ? p.a + (int64_t)mr * p.lda : p.b + (int64_t)mr * p.ldb;
      *reinterpret_cast<uint4*>(smem + st * kStage + (r * 8 + swz(r, c)) * 16) =
          load_codes16(src, (nkb - 1) * 128 + c * 16, p.K);
    }
  };

  // scales of tile kt for the stage rows t, t + kThreads, ...
  auto load_scales = [&](int kt, float (&s)[kScaleRows]) {
    kt = min(kt, nkb - 1);
#pragma unroll
    for (int q = 0; q < kScaleRows; ++q) {
      const int r = t + q * kThreads, mr = matrix_row(r);
      const void* sp = r < BM ? p.sa.p : p.sb.p;
      const int64_t at = (int64_t)(mr >> (r < BM ? p.sa.shift : p.sb.shift)) * (r < BM ? p.sa.ld : p.sb.ld) + kt;
      if constexpr (kMode == kHardware)
        s[q] = __uint_as_float(static_cast<const uint8_t*>(sp)[at]);
      else if constexpr (kMode == kScaled)
        s[q] = load_scale<false>(sp, at);
      else
        s[q] = p.e8m0 ? load_scale<true>(sp, at) : load_scale<false>(sp, at);
    }
  };
  auto put_scales = [&](int buf, const float (&s)[kScaleRows]) {
#pragma unroll
    for (int q = 0; q < kScaleRows; ++q) scales[buf][t + q * kThreads] = s[q];
  };

  floatx4 acc[kMI][kNJ];
#pragma unroll
  for (int i = 0; i < kMI; ++i)
#pragma unroll
    for (int j = 0; j < kNJ; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  // 16 rows of 128 codes (row: a multiple of 16): lane l takes chunks l / 16
  // and l / 16 + 4 of row l % 16 (the order of k within a block is free, if
  // both operands share it)
  const int flo = ((lane & 15) * 8 + swz(lane & 15, lane >> 4)) * 16;
  const int fhi = ((lane & 15) * 8 + swz(lane & 15, (lane >> 4) + 4)) * 16;
  auto frag = [&](int off) {
    const uint4 lo = *reinterpret_cast<const uint4*>(smem + flo + off);
    const uint4 hi = *reinterpret_cast<const uint4*>(smem + fhi + off);
    return intx8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
  };
  const int offa = wm * 128, offb = (BM + wn) * 128;
  const float* const my_sa = &scales[0][wm + (lane & 15)];
  const float* const my_sb = &scales[0][BM + wn + (kMode == kHardware ? (lane & 15) : (kRowB ? (lane >> 4) * 4 : 0))];

  intx8 fa[2], fb[kNJ];
  bf16x8 xa[4], xb[kNJ][4];              // kExact: the fragments as bf16
  floatx4 sum[4];                        // block sums of the last slots,
  floatx4 factor[4];                     // and what they are multiplied by
  float sa[kMI];
  floatx4 sb[kRowB ? kNJ : 1];
  int ea[kMI], eb[kNJ];                  // kHardware: scale bytes

  float next_scales[kScaleRows];
  {
    float s[kScaleRows];
    load_scales(kt_begin, s);
    put_scales(0, s);
    load_scales(kt_begin + 1, s);
    put_scales(1, s);
  }
  copy_tile(kt_begin, 0);
  if (kt_begin + 1 < kt_end) copy_tile(kt_begin + 1, 1);
  load_scales(kt_begin + 2, next_scales);
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  if (kDma && kt_begin == tail_kt) {
    patch_tail(0);
    __syncthreads();
  }
  fa[0] = frag(offa);
#pragma unroll
  for (int j = 0; j < kNJ; ++j) fb[j] = frag(offb + j * 2048);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    sum[q] = floatx4{0.f, 0.f, 0.f, 0.f};
    factor[q] = floatx4{0.f, 0.f, 0.f, 0.f};
  }

  for (int kt = kt_begin; kt < kt_end; ++kt) {
    const int cur = (kt - kt_begin) & 1;
    const int here = cur * kStage, next = (cur ^ 1) * kStage;
    // this tile's scales
    if constexpr (kMode == kHardware) {
#pragma unroll
      for (int i = 0; i < kMI; ++i) ea[i] = __float_as_int(my_sa[cur * (BM + BN) + i * 16]);
#pragma unroll
      for (int j = 0; j < kNJ; ++j) eb[j] = __float_as_int(my_sb[cur * (BM + BN) + j * 16]);
    } else {
#pragma unroll
      for (int i = 0; i < kMI; ++i) sa[i] = my_sa[cur * (BM + BN) + i * 16];
#pragma unroll
      for (int j = 0; j < (kRowB ? kNJ : 1); ++j) {
        if constexpr (kRowB) sb[j] = *reinterpret_cast<const floatx4*>(my_sb + cur * (BM + BN) + j * 16);
        else sb[j][0] = my_sb[cur * (BM + BN)];
      }
    }
#pragma unroll
    for (int i = 0; i < kMI; ++i) {
      if (i == kMI - 1) {
        // the tile's last fragments are in registers and the next tile has
        // arrived: hand this stage to the tile after next
        asm volatile("" ::: "memory");
        __builtin_amdgcn_s_waitcnt(0);
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        if (kDma && kt + 1 == tail_kt && kt + 1 < kt_end) {
          patch_tail(cur ^ 1);
          __syncthreads();
        }
        if (kDma && kt + 2 == tail_kt && kt + 2 < kt_end) tail_offsets();
      }
      if constexpr (kMode == kExact) {
#pragma unroll
        for (int q = 0; q < 4; ++q) xa[q] = codes_to_bf16(fa[i & 1][2 * q], fa[i & 1][2 * q + 1]);
      }
#pragma unroll
      for (int j = 0; j < kNJ; ++j) {
        const int slot = i * kNJ + j;
        if (j == 0) fa[(i + 1) & 1] = frag(i + 1 < kMI ? here + offa + (i + 1) * 2048 : next + offa);
        if constexpr (kMode == kHardware) {
          acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa[i & 1], acc[i][j], 0, 0, 0,
                                                                       eb[j], 0, ea[i]);
          const int ds = (slot + kSlots - 4) % kSlots;   // keeps the products in this order
          asm volatile("" : "+v"(acc[ds / kNJ][ds % kNJ]));
        } else {
          floatx4 s = {0.f, 0.f, 0.f, 0.f};
          if constexpr (kMode == kScaled) {
            s = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa[i & 1], s, 0, 0, 0, 0, 0, 0);
          } else {
            if (i == 0) {
#pragma unroll
              for (int q = 0; q < 4; ++q) xb[j][q] = codes_to_bf16(fb[j][2 * q], fb[j][2 * q + 1]);
            }
#pragma unroll
            for (int q = 0; q < 4; ++q)
              s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(xb[j][q], xa[q], s, 0, 0, 0);
          }
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
            for (int e = 0; e < 4; ++e) factor[slot & 3][e] = sa[i] * sb[j][e];
          } else {
            factor[slot & 3][0] = sa[i] * sb[0][0];
          }
        }
        if (i == kMI - 1) {
          fb[j] = frag(next + offb + j * 2048);
          if (kt + 2 < kt_end) {
#pragma unroll
            for (int g = j * kGroups / kNJ; g < (j + 1) * kGroups / kNJ; ++g) copy_group(g, kt + 2, cur);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (i == kMI - 1) {
        put_scales(cur, next_scales);
        load_scales(kt + 3, next_scales);
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

  // The result through LDS, then whole rows, four columns per lane.
  constexpr bool kBf = kMode != kExact;
  constexpr int kIters = BM / kPasses * BN / 4 / kThreads;
  float* const stage = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kMI / kPasses; ++i)
#pragma unroll
      for (int j = 0; j < kNJ; ++j)
        *reinterpret_cast<floatx4*>(stage + (wm / kPasses + i * 16 + (lane & 15)) * kOutRow + wn + j * 16 +
                                    (lane >> 4) * 4) = acc[pass * (kMI / kPasses) + i][j];
    __syncthreads();
#pragma unroll 2
    for (int q = 0; q < kIters; ++q) {
      const int x = q * kThreads + t, r = x / (BN / 4), c = x % (BN / 4) * 4;
      // LDS row r is row r / h * (kPasses h) + pass h + r % h of the tile, h = 16 kMI / kPasses
      constexpr int h = kMI * 16 / kPasses;
      const int m = m0 + r / h * (kMI * 16) + pass * h + r % h, n = n0 + c;
      if (m >= p.M || n >= p.N) continue;
      floatx4 v = *reinterpret_cast<const floatx4*>(stage + r * kOutRow + c);
      if (p.part) {
        float* o = p.part + ((int64_t)split * p.M + m) * p.N;
        if (p.N % 4 == 0) {
          *reinterpret_cast<floatx4*>(o + n) = v;
        } else {
          for (int e = 0; e < 4; ++e)
            if (n + e < p.N) o[n + e] = v[e];
        }
        continue;
      }
      if (p.add) {
        const float4 ad = p.add_bf ? load4<uint16_t>(static_cast<const uint16_t*>(p.add) + m * p.ldadd, n, p.N, p.cvec)
                                   : load4<float>(static_cast<const float*>(p.add) + m * p.ldadd, n, p.N, p.cvec);
        v[0] += ad.x; v[1] += ad.y; v[2] += ad.z; v[3] += ad.w;
      }
      if constexpr (kBf) {
        uint16_t* o = static_cast<uint16_t*>(p.c) + m * p.ldc;
        if (p.cvec && n + 4 <= p.N) {
          *reinterpret_cast<uint2*>(o + n) = pack_bf16x4(v);
        } else {
          for (int e = 0; e < 4; ++e)
            if (n + e < p.N) o[n + e] = to_bf16_bits(v[e]);
        }
      } else {
        float* o = static_cast<float*>(p.c) + m * p.ldc;
        if (p.cvec && n + 4 <= p.N) {
          *reinterpret_cast<floatx4*>(o + n) = v;
        } else {
          for (int e = 0; e < 4; ++e)
            if (n + e < p.N) o[n + e] = v[e];
        }
      }
    }
  }
}

template <int kMode, bool kRowB, int kWM, int kWN, int kMI, int kNJ, bool kDma>
void launch(const Fp8GemmArgs& a, hipStream_t s) {
  constexpr int BM = kWM * kMI * 16, BN = kWN * kNJ * 16;
  const int64_t tiles = (int64_t)((a.N + BN - 1) / BN) * ((a.M + BM - 1) / BM);
  hipLaunchKernelGGL((fp8_gemm_kernel<kMode, kRowB, kWM, kWN, kMI, kNJ, kDma>),
                     dim3(static_cast<uint32_t>(tiles * a.splits)), dim3(kWM * kWN * 64), 0, s, a);
}

template <int kMode, bool kRowB>
void by_tile(const Fp8GemmArgs& a, hipStream_t s) {
  const bool dma = a.dma && a.K >= 16;
  if (!dma) launch<kMode, kRowB, 2, 2, 4, 4, false>(a, s);
  else if (kMode != kExact && (int64_t)a.M * a.N >= 256 * 256 * 128) launch<kMode, kRowB, 2, 4, 8, 4, true>(a, s);
  else launch<kMode, kRowB, 2, 2, 4, 4, true>(a, s);
}

}  // namespace

hipError_t launch_fp8_matmul(const Fp8GemmArgs& a0, bool c_bf, bool e8m0, hipStream_t s) {
  Fp8GemmArgs a = a0;
  a.e8m0 = e8m0;
  a.splits = 1;
  a.part = nullptr;
  a.kchunk = (a.K + kFp8Block - 1) / kFp8Block;
  const bool row_b = a.sb.shift == 0;
  if (!c_bf) {
    if (row_b) by_tile<kExact, true>(a, s);
    else by_tile<kExact, false>(a, s);
  } else if (e8m0) {
    by_tile<kHardware, false>(a, s);
  } else {
    if (row_b) by_tile<kScaled, true>(a, s);
    else by_tile<kScaled, false>(a, s);
  }
  return hipGetLastError();
}

}  // namespace ortho
