// 8-bit matrices with a scale for each block of 128: device helpers and the
// launchers' argument blocks (internal to libortho.so).  gfx950 only.
//
// A code is an OCP e4m3 byte (1 sign, 4 exponent, 3 mantissa bits; largest
// value 448, one NaN, no infinities).  The scales of an R x C matrix hold one
// value for each block of 1 x 128 or 128 x 128 elements (the last block of a
// row or column may be shorter), as fp32 or as e8m0 (byte b stands for
// 2^(b - 127), 255 for NaN).  Element = code * scale.
#pragma once

#include "common.h"

namespace ortho {

constexpr int kFp8Block = 128;
constexpr float kFp8Top = 448.f;

// Scales as a kernel sees them: the row of scales that covers matrix row i is
// i >> shift (shift 0: a row of its own, 7: shared by 128 rows).
struct ScaleArg {
  const void* p;
  int64_t ld;
  int shift;
};

struct QuantArgs {
  const void* x;
  int64_t ldx;
  uint8_t *q, *qt;          // codes by rows (m x n) and transposed (n x m); either may be null
  int64_t ldq, ldqt;
  void *s, *st;
  int64_t lds, ldst;
  int m, n;
};
hipError_t launch_fp8_quantize(const QuantArgs& a, bool bf, bool e8m0, bool tiles, hipStream_t s);

struct NormArgs {
  const void *x, *res, *w;
  int64_t ldx, ldres;
  void *sum, *y;
  int64_t ldsum, ldy;
  uint8_t* q;
  int64_t ldq;
  void* s;
  int64_t lds;
  float eps;
  int m, n;
  int w_bf;                 // W is bf16
};
hipError_t launch_rms_norm_fp8(const NormArgs& a, bool bf, bool e8m0, hipStream_t s);

struct NormGradArgs {
  const void *dy, *x, *w, *dsum;
  int64_t lddy, ldx, lddsum;
  void* dx;
  int64_t lddx;
  float* dw;
  float* part;              // groups x n partial sums of dw, rows of ldpart (multiple of 8)
  int64_t ldpart;
  float eps;
  int m, n, groups;
  int w_bf;
};
hipError_t launch_rms_norm_backward(const NormGradArgs& a, bool bf, hipStream_t s);

struct Fp8GemmArgs {
  const uint8_t *a, *b;     // M x K and N x K codes
  int64_t lda, ldb;
  ScaleArg sa, sb;
  void* c;
  const void* add;
  int64_t ldc, ldadd;
  int add_bf;
  int M, N, K;
  int dma;                  // A's and B's rows at multiples of 16 bytes, 256 of them within 2 GiB
  int e8m0, c_bf;           // scale type, C's type
  int splits, kchunk;       // splits of K, blocks of 128 in each
  float* part;              // splits x M x ldp partial sums (splits > 1), else null
  int64_t ldp;
};
constexpr int kFewRows = 32;         // rows of A that launch_fp8_few takes (must match plan.h)
hipError_t launch_fp8_few(const Fp8GemmArgs& a, hipStream_t s);     // M <= kFewRows
hipError_t launch_fp8_gemm(const Fp8GemmArgs& a, hipStream_t s);    // bf16 C
hipError_t launch_fp8_exact(const Fp8GemmArgs& a, hipStream_t s);   // fp32 C
hipError_t launch_fp8_matmul(const Fp8GemmArgs& a, hipStream_t s);

// Scale of a block whose largest finite magnitude is `top`, and the factor
// that takes the block's elements to codes.  fp32: top / 448, not below 2^-126
// so that the factor 1 / scale is finite; the factor is rounded once.  e8m0:
// the smallest power of two with top <= 448 * scale, so both are exact.  A
// block of zeros (or without a finite element) has scale 1.
template <bool kE8m0>
__device__ __forceinline__ void block_scale(float top, float& scale, float& factor) {
  if constexpr (kE8m0) {
    // top = f 2^e with f in [0.5, 1): 448 = 0.875 * 2^9
    int e;
    const float f = __builtin_frexpf(top, &e);
    e = e - 9 + (f > 0.875f ? 1 : 0);
    e = e < -126 ? -126 : e;
    e = top == 0.f ? 0 : e;
    scale = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
    factor = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
  } else {
    float s = top / kFp8Top;
    s = s < 0x1p-126f ? 0x1p-126f : s;
    scale = top == 0.f ? 1.f : s;
    factor = 1.f / scale;
  }
}

template <bool kE8m0>
__device__ __forceinline__ void store_scale(void* p, int64_t idx, float scale) {
  if constexpr (kE8m0)
    static_cast<uint8_t*>(p)[idx] = static_cast<uint8_t>(__float_as_uint(scale) >> 23);
  else
    static_cast<float*>(p)[idx] = scale;
}

template <bool kE8m0>
__device__ __forceinline__ float load_scale(const void* p, int64_t idx) {
  if constexpr (kE8m0) {
    const uint32_t b = static_cast<const uint8_t*>(p)[idx];
    return __uint_as_float(b == 0 ? 0x00400000u : (b == 255 ? 0x7fc00000u : b << 23));
  } else {
    return static_cast<const float*>(p)[idx];
  }
}

// |x| if finite, else 0: what a block's scale is taken from.
__device__ __forceinline__ float finite_abs(float x) {
  const float a = __builtin_fabsf(x);
  return a < __builtin_inff() ? a : 0.f;
}

// Eight consecutive elements as stored: fp32 in two registers of four, bf16 in
// one of eight.
template <typename T> struct Raw8;
template <> struct Raw8<uint16_t> { uint4 a; };
template <> struct Raw8<float> { uint4 a, b; };

__device__ __forceinline__ void unpack8(const Raw8<uint16_t>& r, float (&v)[8]) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = __uint_as_float(w[j] << 16);
    v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
  }
}
__device__ __forceinline__ void unpack8(const Raw8<float>& r, float (&v)[8]) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(w[j]);
}

// The 16 bytes u without its first `cut` (a multiple of 2, 1 .. 16), zeros behind.
__device__ __forceinline__ uint4 cut16(uint4 u, int cut) {
  uint64_t lo = u.x | static_cast<uint64_t>(u.y) << 32, hi = u.z | static_cast<uint64_t>(u.w) << 32;
  if (cut >= 8) {
    lo = hi;
    hi = 0;
  }
  const int s = (cut & 7) * 8;
  if (s != 0) {
    lo = lo >> s | hi << (64 - s);
    hi >>= s;
  }
  if (cut >= 16) lo = hi = 0;
  return make_uint4(static_cast<uint32_t>(lo), static_cast<uint32_t>(lo >> 32), static_cast<uint32_t>(hi),
                    static_cast<uint32_t>(hi >> 32));
}

// 16 and 8 bytes at any address; kOnce: such as pass through the chip once, so that the
// caches need not keep them.
template <typename V, bool kOnce>
__device__ __forceinline__ V load_any(const void* p) {
  typedef uint32_t Words __attribute__((ext_vector_type(sizeof(V) / 4), aligned(1)));
  const Words* const w = static_cast<const Words*>(p);
  const Words u = kOnce ? __builtin_nontemporal_load(w) : *w;
  V v;
  __builtin_memcpy(&v, &u, sizeof(V));
  return v;
}
template <bool kOnce, typename V>
__device__ __forceinline__ void store_any(void* p, const V& v) {
  typedef uint32_t Words __attribute__((ext_vector_type(sizeof(V) / 4), aligned(1)));
  Words u;
  __builtin_memcpy(&u, &v, sizeof(V));
  if constexpr (kOnce) __builtin_nontemporal_store(u, static_cast<Words*>(p));
  else *static_cast<Words*>(p) = u;
}

// Eight elements at `row`, all inside.
template <bool kOnce, typename T>
__device__ __forceinline__ Raw8<T> load_whole8(const T* row) {
  Raw8<T> r;
  r.a = load_any<uint4, kOnce>(row);
  if constexpr (sizeof(T) == 4) r.b = load_any<uint4, kOnce>(row + 4);
  return r;
}
template <bool kOnce>
__device__ __forceinline__ void store_whole8(uint16_t* row, const float (&v)[8]) {
  const uint2 lo = pack_bf16x4(floatx4{v[0], v[1], v[2], v[3]});
  const uint2 hi = pack_bf16x4(floatx4{v[4], v[5], v[6], v[7]});
  store_any<kOnce>(row, make_uint4(lo.x, lo.y, hi.x, hi.y));
}
template <bool kOnce>
__device__ __forceinline__ void store_whole8(float* row, const float (&v)[8]) {
  store_any<kOnce>(row, floatx4{v[0], v[1], v[2], v[3]});
  store_any<kOnce>(row + 4, floatx4{v[4], v[5], v[6], v[7]});
}

// 16 bytes' worth of elements from column c of a row of `limit` columns; zeros
// past its end.  The row may start at any element (the accesses need no
// alignment); what its end cuts is loaded from further left and shifted, so
// that no load depends on a branch.
template <typename T>
__device__ __forceinline__ uint4 load16(const T* row, int c, int limit) {
  constexpr int kN = 16 / sizeof(T);
  if (limit >= kN) {   // uniform
    uint4 u;
    __builtin_memcpy(&u, row + (c < limit - kN ? c : limit - kN), 16);
    const int over = c - (limit - kN);
    return over > 0 ? cut16(u, (over < kN ? over : kN) * static_cast<int>(sizeof(T))) : u;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const T e = row[c + j < limit ? c + j : 0];
    if (c + j < limit) {
      if constexpr (sizeof(T) == 2) w[j >> 1] |= static_cast<uint32_t>(e) << (16 * (j & 1));
      else w[j] = __float_as_uint(e);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ Raw8<uint16_t> load_raw8(const uint16_t* row, int c, int limit) {
  return {load16(row, c, limit)};
}
__device__ __forceinline__ Raw8<float> load_raw8(const float* row, int c, int limit) {
  return {load16(row, c, limit), load16(row, c + 4, limit)};
}
template <typename T>
__device__ __forceinline__ void load8(const T* row, int c, int limit, float (&v)[8]) {
  unpack8(load_raw8(row, c, limit), v);
}

// Eight elements to column c of a row of `limit` columns.
__device__ __forceinline__ void store8(uint16_t* row, int c, int limit, const float (&v)[8]) {
  const uint2 lo = pack_bf16x4(floatx4{v[0], v[1], v[2], v[3]});
  const uint2 hi = pack_bf16x4(floatx4{v[4], v[5], v[6], v[7]});
  const uint4 u = make_uint4(lo.x, lo.y, hi.x, hi.y);
  if (c + 8 <= limit) {
    __builtin_memcpy(row + c, &u, 16);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < limit) row[c + j] = to_bf16_bits(v[j]);
}
__device__ __forceinline__ void store8(float* row, int c, int limit, const float (&v)[8]) {
  if (c + 8 <= limit) {
    const floatx4 lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
    __builtin_memcpy(row + c, &lo, 16);
    __builtin_memcpy(row + c + 4, &hi, 16);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < limit) row[c + j] = v[j];
}

// Magnitudes as integers, which order like the values: bf16 two to a register,
// fp32 one.  Infinities and NaN are the largest, so a maximum from kTop on
// says that there is one.
typedef uint16_t ushort2v __attribute__((ext_vector_type(2)));
template <typename T> struct Mags;
template <> struct Mags<uint16_t> { ushort2v m[4]; };
template <> struct Mags<float> { uint32_t m[8]; };

__device__ __forceinline__ Mags<uint16_t> magnitudes(const Raw8<uint16_t>& r) {
  const uint32_t w[4] = {r.a.x, r.a.y, r.a.z, r.a.w};
  Mags<uint16_t> o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o.m[j] = __builtin_bit_cast(ushort2v, w[j] & 0x7fff7fffu);
  return o;
}
__device__ __forceinline__ Mags<float> magnitudes(const Raw8<float>& r) {
  const uint32_t w[8] = {r.a.x, r.a.y, r.a.z, r.a.w, r.b.x, r.b.y, r.b.z, r.b.w};
  Mags<float> o;
#pragma unroll
  for (int j = 0; j < 8; ++j) o.m[j] = w[j] & 0x7fffffffu;
  return o;
}
template <typename T>
__device__ __forceinline__ Mags<T> max_of(const Mags<T>& a, const Mags<T>& b) {
  Mags<T> o;
#pragma unroll
  for (int j = 0; j < (sizeof(T) == 2 ? 4 : 8); ++j) o.m[j] = __builtin_elementwise_max(a.m[j], b.m[j]);
  return o;
}
// Element j's magnitude, and the largest of the eight, as fp32 bits.
__device__ __forceinline__ uint32_t element(const Mags<uint16_t>& a, int j) {
  return static_cast<uint32_t>(a.m[j >> 1][j & 1]) << 16;
}
__device__ __forceinline__ uint32_t element(const Mags<float>& a, int j) { return a.m[j]; }
__device__ __forceinline__ uint32_t largest(const Mags<uint16_t>& a) {
  const ushort2v m = __builtin_elementwise_max(__builtin_elementwise_max(a.m[0], a.m[1]),
                                               __builtin_elementwise_max(a.m[2], a.m[3]));
  return static_cast<uint32_t>(m[0] > m[1] ? m[0] : m[1]) << 16;
}
__device__ __forceinline__ uint32_t largest(const Mags<float>& a) {
  uint32_t m = a.m[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) m = m > a.m[j] ? m : a.m[j];
  return m;
}
constexpr uint32_t kInfBits = 0x7f800000u;

// Four fp32 values as four e4m3 codes, round to nearest even; infinities and
// NaN give the NaN code.
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  int u = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, u, true));
}

// Eight codes to column c of a row of `limit` columns.
__device__ __forceinline__ void store_codes8(uint8_t* row, int c, int limit, uint2 u) {
  if (c + 8 <= limit) {
    __builtin_memcpy(row + c, &u, 8);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < limit) row[c + j] = static_cast<uint8_t>((j < 4 ? u.x : u.y) >> (8 * (j & 3)));
}

}  // namespace ortho
