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
  int vec;                  // X's rows start at multiples of 16 bytes
  uint8_t *q, *qt;          // codes by rows (m x n) and transposed (n x m); either may be null
  int64_t ldq, ldqt;
  int qvec, qtvec;          // rows of 16-byte multiples
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
  int vec;                  // x, res, sum, y rows of 16-byte multiples
  int qvec;                 // q rows of 8-byte multiples
  int w_bf, wvec;           // W is bf16; 16-byte aligned
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
  int vec;
  int w_bf, wvec;
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
  int cvec;                 // C's (and Add's) rows at multiples of 16 bytes
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

// From column c of a row of `limit` columns; zeros past its end.
__device__ __forceinline__ Raw8<uint16_t> load_raw8(const uint16_t* row, int c, int limit, bool vec) {
  Raw8<uint16_t> r;
  if (vec && c + 8 <= limit) {
    r.a = *reinterpret_cast<const uint4*>(row + c);
    return r;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < limit) w[j >> 1] |= static_cast<uint32_t>(row[c + j]) << (16 * (j & 1));
  r.a = make_uint4(w[0], w[1], w[2], w[3]);
  return r;
}
__device__ __forceinline__ Raw8<float> load_raw8(const float* row, int c, int limit, bool vec) {
  Raw8<float> r;
  if (vec && c + 8 <= limit) {
    r.a = *reinterpret_cast<const uint4*>(row + c);
    r.b = *reinterpret_cast<const uint4*>(row + c + 4);
    return r;
  }
  uint32_t w[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) w[j] = c + j < limit ? __float_as_uint(row[c + j]) : 0u;
  r.a = make_uint4(w[0], w[1], w[2], w[3]);
  r.b = make_uint4(w[4], w[5], w[6], w[7]);
  return r;
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

// Eight consecutive elements from column c of a row of `limit` columns.
template <typename T>
__device__ __forceinline__ void load8(const T* row, int c, int limit, bool vec, float (&v)[8]);
template <>
__device__ __forceinline__ void load8<uint16_t>(const uint16_t* row, int c, int limit, bool vec,
                                                float (&v)[8]) {
  if (vec && c + 8 <= limit) {
    const uint4 u = *reinterpret_cast<const uint4*>(row + c);
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = __uint_as_float(w[j] << 16);
      v[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = c + j < limit ? bf16_bits_to_f32(row[c + j]) : 0.f;
}
template <>
__device__ __forceinline__ void load8<float>(const float* row, int c, int limit, bool vec,
                                             float (&v)[8]) {
  if (vec && c + 8 <= limit) {
    const float4 u = *reinterpret_cast<const float4*>(row + c);
    const float4 w = *reinterpret_cast<const float4*>(row + c + 4);
    v[0] = u.x; v[1] = u.y; v[2] = u.z; v[3] = u.w;
    v[4] = w.x; v[5] = w.y; v[6] = w.z; v[7] = w.w;
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = c + j < limit ? row[c + j] : 0.f;
}

template <typename T>
__device__ __forceinline__ void store8(T* row, int c, int limit, bool vec, const float (&v)[8]);
template <>
__device__ __forceinline__ void store8<uint16_t>(uint16_t* row, int c, int limit, bool vec,
                                                 const float (&v)[8]) {
  if (vec && c + 8 <= limit) {
    const uint2 lo = pack_bf16x4(floatx4{v[0], v[1], v[2], v[3]});
    const uint2 hi = pack_bf16x4(floatx4{v[4], v[5], v[6], v[7]});
    *reinterpret_cast<uint4*>(row + c) = make_uint4(lo.x, lo.y, hi.x, hi.y);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < limit) row[c + j] = to_bf16_bits(v[j]);
}
template <>
__device__ __forceinline__ void store8<float>(float* row, int c, int limit, bool vec,
                                              const float (&v)[8]) {
  if (vec && c + 8 <= limit) {
    *reinterpret_cast<float4*>(row + c) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(row + c + 4) = make_float4(v[4], v[5], v[6], v[7]);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < limit) row[c + j] = v[j];
}

// Eight codes to column c of a row of `limit` columns.
__device__ __forceinline__ void store_codes8(uint8_t* row, int c, int limit, bool vec, uint2 u) {
  if (vec && c + 8 <= limit) {
    *reinterpret_cast<uint2*>(row + c) = u;
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < limit) row[c + j] = static_cast<uint8_t>((j < 4 ? u.x : u.y) >> (8 * (j & 3)));
}

}  // namespace ortho
