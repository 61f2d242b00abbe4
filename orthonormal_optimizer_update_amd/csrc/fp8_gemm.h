// What the kernels of the 8-bit product share: matrix operand types, copies into
// LDS, LDS places, conversion to bf16.
#pragma once

#include "fp8.h"

namespace ortho {

// The kernel's lambdas share its state by reference: inlined, it stays in registers.
#define ORTHO_INLINE __attribute__((always_inline))

typedef int intx8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) void* lds_ptr_t;

// Eight codes times the power of two `by` as eight bf16 (exact while that is a
// normal number; the NaN code gives NaN).
__device__ __forceinline__ bf16x8 codes_to_bf16(int lo, int hi, float by = 1.f) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, by, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, by, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, by, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, by, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Position of a 16-byte chunk in the 128-byte LDS row `row` of a tile, such that
// the 16 rows of a fragment hit 64 distinct banks: rows r .. r + 15 of A (and of
// B for an fp32 C), rows 16 (i / 4) + i % 4 + 4 j of B for a bf16 C.
template <bool kSpread>
__device__ __forceinline__ int swz(int row, int chunk) {
  if constexpr (kSpread) return chunk ^ (((row >> 1) & 1) | ((row >> 3) & 6));
  return chunk ^ ((row >> 1) & 7);
}

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

// Four bytes, or one byte as a word, per lane into LDS at lds + 4 * lane.
__device__ __forceinline__ void dma4(unsigned voff, const uint8_t* sbase, unsigned lds) {
  asm volatile("s_nop 4\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dword %0, %1"
               :: "v"(voff), "s"(sbase), "s"(lds) : "memory");
}
__device__ __forceinline__ void dma1(unsigned voff, const uint8_t* sbase, unsigned lds) {
  asm volatile("s_nop 4\n\ts_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_ubyte %0, %1"
               :: "v"(voff), "s"(sbase), "s"(lds) : "memory");
}

// Waits until at most kOutstanding of the wave's copies are under way and its
// LDS reads and writes are done, then for the workgroup.
template <int kOutstanding>
__device__ __forceinline__ void sync() {
  static_assert(kOutstanding < 64, "");
  asm volatile("" ::: "memory");
  // vmcnt kOutstanding, expcnt off, lgkmcnt 0
  __builtin_amdgcn_s_waitcnt((kOutstanding & 15) | (kOutstanding >> 4) << 14 | 7 << 4);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

__device__ __forceinline__ unsigned uniform(unsigned x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ const uint8_t* uniform_ptr(const uint8_t* p) {
  const uint64_t v = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v));
  const uint32_t hi = __builtin_amdgcn_readfirstlane(static_cast<uint32_t>(v >> 32));
  return reinterpret_cast<const uint8_t*>((static_cast<uint64_t>(hi) << 32) | lo);
}

// One of two kernel arguments by a condition that is the same for the whole
// wave.  Both are read by scalar loads first: left alone, the compiler chooses
// between their addresses and reads the argument block through vector memory.
template <typename T>
__device__ __forceinline__ T pick(bool first, T a, T b) {
  asm("" : "+s"(a), "+s"(b));
  return first ? a : b;
}

// A block's sum is 2^-18 to 2^24.7 (or 0), so sum sa sb can be a number though
// sa sb is subnormal, zero or infinite (0 with a block of zeros beside an infinite
// one).  That is rare: a wave keeps the range of the scales that it met, and the
// rows of C where a product could have left fp32's are formed anew, in the same
// order, with what a scale has beyond 2^-63 .. 2^62 (an exact power of two) in the
// codes' products and only the rest, whose products are normal numbers, in the
// factor.  Elements with no such scale come out the same either way.
constexpr int kFar = 62;
__device__ __forceinline__ int excess(float s) {
  const int e = __builtin_amdgcn_frexp_expf(s);   // 0 for zero, infinities and NaN
  return e - min(max(e, -kFar), kFar);
}
__device__ __forceinline__ float moved(float s) { return __builtin_ldexpf(s, -excess(s)); }

// Whether the product f of two scales left fp32's normal range (power-of-two scales
// are never 0).
template <bool kE8m0>
__device__ __forceinline__ bool leaves_range(float f, float sa, float sb) {
  const bool odd = __builtin_amdgcn_classf(f, 0x2f4);   // infinite, subnormal or zero, of either sign
  if constexpr (kE8m0) return odd;
  return odd && sa != 0.f && sb != 0.f;
}

// Smallest exponents of the scales of a wave's 64 kRows rows of A (lane l: rows
// 64 h + l, in one of kH registers) and of its rows of B (spread over the lanes in
// any way), and the largest of both: s in [2^(e-1), 2^e).
template <int kRows, int kH>
struct ScaleRange {
  int lo_a[kH] = {}, lo_b = 0, hi = 0;
  __device__ __forceinline__ void a(int h, float s) {
    const int e = __builtin_amdgcn_frexp_expf(s);
    lo_a[h % kH] = min(lo_a[h % kH], e);
    hi = max(hi, e);
  }
  __device__ __forceinline__ void b(float s) {
    const int e = __builtin_amdgcn_frexp_expf(s);
    lo_b = min(lo_b, e);
    hi = max(hi, e);
  }
  // Bit i: whether a product with one of the rows 16 i .. 16 i + 15 may have left
  // fp32's normal range.  The same for the wave.
  __device__ __forceinline__ uint32_t lost() const {
    int lo = lo_b;
#pragma unroll
    for (int h = 0; h < kH; ++h) lo = min(lo, lo_a[h]);
    if (!__any(lo < -kFar || hi > kFar)) return 0;
    int y = lo_b;
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) y = min(y, __shfl_xor(y, o, 64));
    const bool all = __any(hi > kFar);
    uint32_t rows = 0;
#pragma unroll
    for (int h = 0; h < kRows; ++h) {
      const uint64_t some = __ballot(all || lo_a[h % kH] + y < -124);   // 2^(x-1) 2^(y-1) < 2^-126
#pragma unroll
      for (int q = 0; q < 4; ++q) rows |= (some >> 16 * q & 0xffff) != 0 ? 1u << (4 * h + q) : 0u;
    }
    return rows;
  }
};

// The kernel's arguments (its only parameter) read anew from here on: a rare path
// that uses them then does not keep them in scalar registers through the others.
__device__ __forceinline__ Fp8GemmArgs args_again() {
  auto* q = __builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(q));
  return *(const Fp8GemmArgs*)(const void*)q;
}

// 16 codes from column k of a row of K; zero codes from column K on.  Any byte.
// A piece that the row's end cuts is loaded from 16 columns before the end and
// shifted, so that no load depends on a branch.
__device__ __forceinline__ uint4 load_codes16_of_long_rows(const uint8_t* row, int k, int K) {   // K >= 16
  uint4 u;
  __builtin_memcpy(&u, row + min(k, K - 16), 16);
  const int cut = k + 16 - K;   // bytes of the piece that lie past the end
  return cut <= 0 ? u : cut16(u, min(cut, 16));
}
__device__ __forceinline__ uint4 load_codes16(const uint8_t* row, int k, int K) {
  if (K >= 16) return load_codes16_of_long_rows(row, k, K);   // uniform
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint32_t c = row[min(k + j, K - 1)];
    w[j >> 2] |= (k + j < K ? c : 0u) << (8 * (j & 3));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Four elements of Add from column n of row m, and four of C to it (C's type
// T); rows of either may start at any element (the accesses need no alignment).
__device__ __forceinline__ floatx4 load_add4(const Fp8GemmArgs& p, int64_t m, int n) {
  floatx4 v = {0.f, 0.f, 0.f, 0.f};
  if (p.add_bf) {
    const uint16_t* src = static_cast<const uint16_t*>(p.add) + m * p.ldadd + n;
    if (n + 4 <= p.N) {
      uint2 u;
      __builtin_memcpy(&u, src, 8);
      return floatx4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                     __uint_as_float(u.y & 0xffff0000u)};
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < p.N) v[e] = bf16_bits_to_f32(src[e]);
    return v;
  }
  const float* src = static_cast<const float*>(p.add) + m * p.ldadd + n;
  if (n + 4 <= p.N) {
    __builtin_memcpy(&v, src, 16);
    return v;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < p.N) v[e] = src[e];
  return v;
}
template <typename T>
__device__ __forceinline__ void store_c4(const Fp8GemmArgs& p, int64_t m, int n, floatx4 v) {
  T* const dst = static_cast<T*>(p.c) + m * p.ldc + n;
  if (n + 4 <= p.N) {
    if constexpr (sizeof(T) == 2) {
      const uint2 u = pack_bf16x4(v);
      __builtin_memcpy(dst, &u, 8);
    } else {
      __builtin_memcpy(dst, &v, 16);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (n + e < p.N) store_from_f32<T>(dst, e, v[e]);
}

}  // namespace ortho
