// AdamW on many tensors per launch, and the gradients' norm.
#include "adamw.h"
#include "fp8.h"

// Products and sums join where the code says so and nowhere else: a tensor comes
// out the same whichever kernel its layout picks.  m and v take the separate
// roundings of the formula written in elementary operations, so that their codes
// are the same as such a form's: a code that goes the other way at a tie can be its
// block's largest, and then the next step's scale differs.
#pragma clang fp contract(off)

namespace ortho {

namespace {

static_assert(sizeof(AdamwFlat) <= 4096 && sizeof(AdamwRows) <= 4096 && sizeof(NormParts) <= 4096, "");

// ---- random bits (the definition is in ortho.h) ----

__device__ __forceinline__ uint32_t mix(uint32_t h) {
  h = (h ^ h >> 16) * 0x7feb352du;
  h = (h ^ h >> 15) * 0x846ca68bu;
  return h ^ h >> 16;
}
constexpr uint32_t kStride = 0x9e3779b9u;

__device__ __forceinline__ uint32_t tensor_key(const AdamwScalars& h, int64_t step, int index) {
  uint32_t key = mix(h.seed_lo);
  key = mix(key ^ mix(h.seed_hi + kStride));
  key = mix(key ^ mix(static_cast<uint32_t>(step) + kStride));
  key = mix(key ^ mix(static_cast<uint32_t>(static_cast<uint64_t>(step) >> 32) + kStride));
  return mix(key ^ mix(static_cast<uint32_t>(index) + kStride));
}

// The bits of the elements from `element` on, as seeds of the conversion
// instructions, which take a seed's top 20 (e4m3) and 16 bits (bf16).
struct Bits {
  uint32_t low, key, next;   // next: the key behind a multiple of 2^32
  __device__ __forceinline__ Bits(uint32_t tensor, int64_t element) {
    low = static_cast<uint32_t>(element);
    key = tensor + kStride * static_cast<uint32_t>(static_cast<uint64_t>(element) >> 32);
    next = key + kStride;
  }
  // m's seeds, and sqrt(v)'s, of kN elements.
  template <int kN>
  __device__ __forceinline__ void all(uint32_t (&a)[kN], uint32_t (&b)[kN]) const {
    if (__any(low > ~0u - (kN - 1))) {   // a multiple of 2^32 among them
#pragma unroll
      for (int j = 0; j < kN; ++j) a[j] = mix((low + j) ^ (low + j < low ? next : key));
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) a[j] = mix((low + j) ^ key);
    }
#pragma unroll
    for (int j = 0; j < kN; ++j) b[j] = mix(a[j] + kStride);
  }
  // The weight's: a's low 12 bits, then b's low 4.
  static __device__ __forceinline__ uint32_t weight(uint32_t a, uint32_t b) {
    return __builtin_amdgcn_alignbit(a, b << 28, 12);
  }
};

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two weights, rounded by their seeds.
__device__ __forceinline__ uint32_t weights2(float x0, float x1, uint32_t seed0, uint32_t seed1) {
  bf16x2 p = {0, 0};
  p = __builtin_amdgcn_cvt_sr_bf16_f32(p, x0, seed0, false);
  p = __builtin_amdgcn_cvt_sr_bf16_f32(p, x1, seed1, true);
  return __builtin_bit_cast(uint32_t, p);
}

// Eight weights to column c of a row of `limit`, rounded by their seeds.
template <bool kOnce>
__device__ __forceinline__ void store_weights8(uint16_t* row, int c, int limit, const float (&x)[8],
                                               const uint32_t (&seed)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = weights2(x[2 * j], x[2 * j + 1], seed[2 * j], seed[2 * j + 1]);
  if (c + 8 <= limit) {
    const uint4 u = make_uint4(w[0], w[1], w[2], w[3]);
    store_any<kOnce>(row + c, u);
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (c + j < limit) row[c + j] = static_cast<uint16_t>(w[j >> 1] >> 16 * (j & 1));
}

// ---- the step ----

struct StepScalars {
  float keep, size, root, factor;
  int64_t step;
  bool skip;
};

// (Rate or step read on the device: every wave works the rest out in fp64 again.  Calls
// that wait for memory lose nothing by it, 604 million bf16 weights 2534 us for 2528;
// 67 million with states in codes, rounded stochastically, a sixth, 174 us for 150.)
__device__ __forceinline__ StepScalars step_scalars(const AdamwScalars& h) {
  StepScalars s = {h.keep, h.size, h.root, 1.f, h.step, false};
  if (h.factor) {
    s.factor = *h.factor;
    s.skip = s.factor != s.factor;
  }
  if (h.lr_dev || h.step_dev) {
    const double lr = h.lr_dev ? static_cast<double>(*h.lr_dev) : h.lr;
    if (h.step_dev) s.step = *h.step_dev < 1 ? 1 : *h.step_dev;
    const double t = static_cast<double>(s.step);
    s.keep = static_cast<float>(1.0 - lr * h.wd);
    s.size = static_cast<float>(lr / -expm1(t * h.log_b1));
    s.root = static_cast<float>(1.0 / __builtin_sqrt(-expm1(t * h.log_b2)));
  }
  return s;
}

// m and v are fp32 from here to the next step's start; only storage rounds them.
__device__ __forceinline__ void moments(const AdamwScalars& h, const StepScalars& s, float g, float& m, float& v) {
  g *= s.factor;
  m = h.b1 * m + h.c1 * g;
  v = h.b2 * v + h.c2 * (g * g);
}

// The weight takes the reciprocal's rounding (one unit in the last place) in place of
// a division's.  (eps and the root's bounds keep the divisor from 2^-126 to 2^126,
// where the instruction's result is a normal number.)
__device__ __forceinline__ float weight(const AdamwScalars& h, const StepScalars& s, float x, float m, float root) {
  return fmaf(-s.size, m * __builtin_amdgcn_rcpf(fmaf(root, s.root, h.eps)), s.keep * x);
}

// sqrt(v), correctly rounded, for v = 2^-100 to the largest number and NaN, with kZero
// for 0 too: coupled Newton steps for sqrt(v) and 1 / (2 sqrt(v)) from the reciprocal
// root, and the residual's correction (eight instructions; the library's function,
// which takes all of fp32, has seventeen).
template <bool kZero>
__device__ __forceinline__ float root_of(float v) {
  const uint32_t bits = __float_as_uint(v);
  const float y = __builtin_amdgcn_rsqf(__uint_as_float(kZero ? max(bits, 0x00800000u) : bits));
  float g = v * y, h = 0.5f * y;
  const float r = fmaf(-h, g, 0.5f);
  g = fmaf(g, r, g);
  h = fmaf(h, r, h);
  return fmaf(fmaf(-g, g, v), h, g);
}
constexpr uint32_t kLeastRoot = 0x0d800000u, kInfinity = 0x7f800000u;   // 2^-100's bits

// What a wave's values may be beside ordinary ones.
struct Among {
  bool zeros, far;   // far: infinite or NaN
};

// The roots of eight values that are not negative.  Most waves hold no zero and nothing
// tiny, infinite or NaN, and one look tells.
__device__ __forceinline__ Among roots8(float (&v)[8]) {
  uint32_t low = ~0u, high = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    low = min(low, __float_as_uint(v[j]));
    high = max(high, __float_as_uint(v[j]));
  }
  if (!__any(low < kLeastRoot || high >= kInfinity)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = root_of<false>(v[j]);
    return {false, false};
  }
  const bool far = __any(high >= kInfinity);
  uint32_t least = ~0u;
#pragma unroll
  for (int j = 0; j < 8; ++j) least = min(least, __float_as_uint(v[j]) - 1);   // (0 counts for nothing)
  if (far || __any(least < kLeastRoot - 1)) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __builtin_sqrtf(v[j]);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = root_of<true>(v[j]);
  }
  return {true, far};
}

__device__ __forceinline__ float value_of(float g) { return g; }
__device__ __forceinline__ float value_of(uint16_t g) { return bf16_bits_to_f32(g); }
__device__ __forceinline__ float value_of(uint8_t code, float scale) {
  return __builtin_amdgcn_cvt_f32_fp8(code, 0) * scale;
}

// The weight of an element whose v came out infinite or NaN in fp32, and sqrt(v) in
// place of it.  A root kept as a code, or a gradient, may have a square beyond fp32's
// range; scaled by a power of two it has not, and the root is back within the range.
// (Formed so where nothing is far, a square would be lost at the other end.)
__device__ __forceinline__ float far_weight(const AdamwScalars& h, const StepScalars& s, float x, float g, float m,
                                            float kept, float& root) {
  g *= s.factor;
  kept = h.b2 == 0.f ? 0.f * kept : kept;
  const int e = max(0, __builtin_amdgcn_frexp_expf(fmaxf(__builtin_fabsf(kept), __builtin_fabsf(g))));
  g = __builtin_ldexpf(g, -e);
  kept = __builtin_ldexpf(kept, -e);
  const float r = __builtin_sqrtf(h.b2 * (kept * kept) + h.c2 * (g * g));
  root = r < __builtin_inff() ? fminf(__builtin_ldexpf(r, e), __FLT_MAX__) : r;
  const float down = fmaf(r, s.root, __builtin_ldexpf(h.eps, -e));
  return fmaf(-s.size, __builtin_ldexpf(m, -e) * __builtin_amdgcn_rcpf(down), s.keep * x);
}

// The tensor of a unit; `first` is this lane's.
template <typename I>
__device__ __forceinline__ int tensor_of(I first, I unit) {
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(first <= unit)) - 1);
}


// Four elements at p.
template <bool kOnce>
__device__ __forceinline__ void load4(const float* p, float* v) {
  const uint4 u = load_any<uint4, kOnce>(p);
  v[0] = __uint_as_float(u.x); v[1] = __uint_as_float(u.y); v[2] = __uint_as_float(u.z); v[3] = __uint_as_float(u.w);
}
template <bool kOnce>
__device__ __forceinline__ void load4(const uint16_t* p, float* v) {
  const uint2 u = load_any<uint2, kOnce>(p);
  v[0] = __uint_as_float(u.x << 16); v[1] = __uint_as_float(u.x & 0xffff0000u);
  v[2] = __uint_as_float(u.y << 16); v[3] = __uint_as_float(u.y & 0xffff0000u);
}
template <bool kOnce>
__device__ __forceinline__ void store4(float* p, const float* v) {
  store_any<kOnce>(p, floatx4{v[0], v[1], v[2], v[3]});
}
template <bool kOnce>
__device__ __forceinline__ void store4(uint16_t* p, const float* v) {
  store_any<kOnce>(p, pack_bf16x4(floatx4{v[0], v[1], v[2], v[3]}));
}

// A whole unit: a thread has four elements in each half of it, so that every access of
// a wave covers whole lines whatever the type.
template <typename TX, typename TG, bool kStochastic, bool kOnce>
__device__ __forceinline__ void flat_whole(const AdamwScalars& h, const StepScalars& s, const FlatTensor& t,
                                           int64_t base, uint32_t key) {
  constexpr int kHalf = kUnit / 2;
  base += threadIdx.x * 4;
  TX* const x = static_cast<TX*>(t.x) + base;
  const TG* const g = static_cast<const TG*>(t.g) + base;
  float *const m = t.m + base, *const v = t.v + base;
  float xv[8], gv[8], mv[8], vv[8];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    load4<kOnce>(x + q * kHalf, xv + 4 * q);
    load4<kOnce>(g + q * kHalf, gv + 4 * q);
    load4<kOnce>(m + q * kHalf, mv + 4 * q);
    load4<kOnce>(v + q * kHalf, vv + 4 * q);
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    moments(h, s, gv[j], mv[j], vv[j]);
    xv[j] = weight(h, s, xv[j], mv[j], __builtin_sqrtf(vv[j]));
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if constexpr (kStochastic && sizeof(TX) == 2) {
      uint32_t a[4], b[4];
      Bits(key, base + q * kHalf).all(a, b);
      store_any<kOnce>(x + q * kHalf, make_uint2(weights2(xv[4 * q], xv[4 * q + 1], Bits::weight(a[0], b[0]), Bits::weight(a[1], b[1])),
                                                 weights2(xv[4 * q + 2], xv[4 * q + 3], Bits::weight(a[2], b[2]), Bits::weight(a[3], b[3]))));
    } else {
      store4<kOnce>(x + q * kHalf, xv + 4 * q);
    }
    store4<kOnce>(m + q * kHalf, mv + 4 * q);
    store4<kOnce>(v + q * kHalf, vv + 4 * q);
  }
}

// A tensor's last unit, of `limit` elements.
template <typename TX, typename TG, bool kStochastic>
__device__ __forceinline__ void flat_part(const AdamwScalars& h, const StepScalars& s, const FlatTensor& t,
                                          int64_t base, int limit, uint32_t key) {
  TX* const x = static_cast<TX*>(t.x) + base;
  const TG* const g = static_cast<const TG*>(t.g) + base;
  float *const m = t.m + base, *const v = t.v + base;
  const int c = threadIdx.x * 8;
  float xv[8], gv[8], mv[8], vv[8];
  const auto rx = load_raw8(x, c, limit);
  const auto rg = load_raw8(g, c, limit);
  const auto rm = load_raw8(m, c, limit);
  const auto rv = load_raw8(v, c, limit);
  unpack8(rx, xv);
  unpack8(rg, gv);
  unpack8(rm, mv);
  unpack8(rv, vv);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    moments(h, s, gv[j], mv[j], vv[j]);
    xv[j] = weight(h, s, xv[j], mv[j], __builtin_sqrtf(vv[j]));
  }
  if constexpr (kStochastic && sizeof(TX) == 2) {
    const Bits bits(key, base + c);
    uint32_t a[8], b[8], seed[8];
    bits.all(a, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) seed[j] = Bits::weight(a[j], b[j]);
    store_weights8<false>(x, c, limit, xv, seed);
  } else {
    store8(x, c, limit, xv);
  }
  store8(m, c, limit, mv);
  store8(v, c, limit, vv);
}

template <typename TX, typename TG, bool kStochastic, bool kOnce>
__device__ __forceinline__ void flat_unit(const AdamwScalars& h, const StepScalars& s, const FlatTensor& t,
                                          int64_t base, int64_t left, uint32_t key) {
  if (left >= kUnit) flat_whole<TX, TG, kStochastic, kOnce>(h, s, t, base, key);
  else flat_part<TX, TG, kStochastic>(h, s, t, base, static_cast<int>(left), key);
}

// Tensors of consecutive elements, states in 32 bits.  Bound by HBM: 134 million weights
// and gradients in bf16 take 501 us (22 bytes each, 5.9 TB/s; a copy reaches 5.1).  Every
// element is touched once, so nothing is staged: each thread has its 8 elements' loads
// under way together, a new workgroup per unit keeps memory busier than workgroups that
// stay (8% on 604 million; two and four units per workgroup: no gain), and what is large
// goes past the caches, in whole lines and both ways (551 us through them; 545 past them
// with lines in halves, 541 with only the loads, 551 with only the stores past them).
// 100352 fp32 weights in 49 tensors take 4.0 us, a launch's latency.
template <bool kStochastic, bool kOnce>
__global__ __launch_bounds__(256) void adamw_flat_kernel(AdamwFlat a) {
  const int first = a.first[threadIdx.x & (kLanes - 1)];
  const StepScalars s = step_scalars(a.h);
  if (s.skip) return;
  for (int unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const int i = tensor_of(first, unit);
    const FlatTensor& t = a.t[i];
    const int64_t base = (int64_t)(unit - a.first[i]) * kUnit, left = t.n - base;
    const uint32_t key = kStochastic ? tensor_key(a.h, s.step, t.index) : 0;
    switch (t.kind) {
      case 0: flat_unit<float, float, kStochastic, kOnce>(a.h, s, t, base, left, key); break;
      case kBf16Weight: flat_unit<uint16_t, float, kStochastic, kOnce>(a.h, s, t, base, left, key); break;
      case kBf16Gradient: flat_unit<float, uint16_t, kStochastic, kOnce>(a.h, s, t, base, left, key); break;
      default: flat_unit<uint16_t, uint16_t, kStochastic, kOnce>(a.h, s, t, base, left, key);
    }
  }
}

// Eight codes from column c of a row of `limit`, zeros past its end.
__device__ __forceinline__ uint2 load_codes8(const uint8_t* row, int c, int limit) {
  uint64_t u = 0;
  if (limit >= 8) {   // uniform for the row
    __builtin_memcpy(&u, row + (c < limit - 8 ? c : limit - 8), 8);
    const int over = c - (limit - 8);
    if (over > 0) u = over >= 8 ? 0 : u >> 8 * over;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const uint64_t e = row[c + j < limit ? c + j : 0];
      if (c + j < limit) u |= e << 8 * j;
    }
  }
  return make_uint2(static_cast<uint32_t>(u), static_cast<uint32_t>(u >> 32));
}

__device__ __forceinline__ void values8(uint2 u, float scale, float (&v)[8]) {
  typedef float float2v __attribute__((ext_vector_type(2)));
  const float2v a = __builtin_amdgcn_cvt_pk_f32_fp8(u.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8(u.x, true);
  const float2v c = __builtin_amdgcn_cvt_pk_f32_fp8(u.y, false), d = __builtin_amdgcn_cvt_pk_f32_fp8(u.y, true);
  v[0] = a[0] * scale; v[1] = a[1] * scale; v[2] = b[0] * scale; v[3] = b[1] * scale;
  v[4] = c[0] * scale; v[5] = c[1] * scale; v[6] = d[0] * scale; v[7] = d[1] * scale;
}

// The largest of 16 lanes' values (a row of the wave), NaN if there is one.
template <int kRotate>
__device__ __forceinline__ float rotated(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x120 + kRotate, 0xf, 0xf, false));
}
__device__ __forceinline__ float max_of_16_lanes(float v) {
  v = __builtin_elementwise_maximum(v, rotated<8>(v));
  v = __builtin_elementwise_maximum(v, rotated<4>(v));
  v = __builtin_elementwise_maximum(v, rotated<2>(v));
  return __builtin_elementwise_maximum(v, rotated<1>(v));
}

// 1 / s for s from 2^-126 to 2^126: the reciprocal instruction's result and one
// correction by the residual, which is the correctly rounded quotient for every such s
// (all of them tried on the chip).
__device__ __forceinline__ float inverse(float s) {
  const float y = __builtin_amdgcn_rcpf(s);
  return fmaf(fmaf(-s, y, 1.f), y, y);
}

// Codes of a block's eight elements here, the 16 lanes of a block together.  A block
// with an infinity or NaN (its largest magnitude says so) looks at its finite
// elements once more.
// kPositive: no element is below 0; those above 0 get no code of 0, and `zeros` says
// whether there may be others.
template <bool kStochastic, bool kPositive>
__device__ __forceinline__ uint2 to_codes8(const float (&v)[8], const uint32_t (&seed)[8], bool zeros, float& scale) {
  float top = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = __builtin_elementwise_maximum(top, kPositive ? v[j] : __builtin_fabsf(v[j]));
  top = max_of_16_lanes(top);
  uint32_t lost = 0;   // bit j: element j is no number
  if (!(top < __builtin_inff())) {
    top = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const bool number = __builtin_fabsf(v[j]) < __builtin_inff();
      top = fmaxf(top, number ? __builtin_fabsf(v[j]) : 0.f);
      lost |= number ? 0u : 1u << j;
    }
    top = max_of_16_lanes(top);
  }
  const float s = fmaxf(top * (1.f / kFp8Top), 0x1p-126f);
  scale = top == 0.f ? 1.f : s;
  const float f = inverse(scale);
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) q[j] = v[j] * f;
  // (the largest may come out a rounding above 448)
  if constexpr (kPositive) {
    if (zeros) {
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = __builtin_amdgcn_fmed3f(q[j], v[j] > 0.f ? 0x1p-9f : 0.f, kFp8Top);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) q[j] = __builtin_amdgcn_fmed3f(q[j], 0x1p-9f, kFp8Top);
    }
  } else if constexpr (kStochastic) {
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __builtin_amdgcn_fmed3f(q[j], -kFp8Top, kFp8Top);
  }
  if (lost != 0) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (lost >> j & 1) q[j] = __builtin_nanf("");
  }
  if constexpr (kStochastic) {
    uint32_t u[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      int w = 0;
      w = __builtin_amdgcn_cvt_sr_fp8_f32(q[4 * i], seed[4 * i], w, 0);
      w = __builtin_amdgcn_cvt_sr_fp8_f32(q[4 * i + 1], seed[4 * i + 1], w, 1);
      w = __builtin_amdgcn_cvt_sr_fp8_f32(q[4 * i + 2], seed[4 * i + 2], w, 2);
      w = __builtin_amdgcn_cvt_sr_fp8_f32(q[4 * i + 3], seed[4 * i + 3], w, 3);
      u[i] = static_cast<uint32_t>(w);
    }
    return make_uint2(u[0], u[1]);
  } else {
    return make_uint2(pack_e4m3x4(q[0], q[1], q[2], q[3]), pack_e4m3x4(q[4], q[5], q[6], q[7]));
  }
}

// Eight codes at c of a row of `cols`.
template <bool kWhole, bool kOnce>
__device__ __forceinline__ uint2 unit_load_codes(const uint8_t* row, int c, int cols) {
  if constexpr (kWhole) return load_any<uint2, kOnce>(row + c);
  else return load_codes8(row, c, cols);
}

// Eight elements at c of a row of `cols`.  fp32, of which a wave's 16-byte accesses take
// every other 16, does not go past the caches, which join the halves of a line (67
// million weights with gradients in fp32: 184 us, 197 past them).
template <bool kWhole, bool kOnce, typename T>
__device__ __forceinline__ Raw8<T> unit_load(const T* p, int c, int limit) {
  if constexpr (kWhole) return load_whole8<kOnce && sizeof(T) == 2>(p + c);
  else return load_raw8(p, c, limit);
}

// (pitch and row as they are, unsigned: the address takes one multiplication)
template <typename T>
__device__ __forceinline__ T* row_at(void* base, uint32_t ld, uint32_t row) {
  return static_cast<T*>(base) + static_cast<uint64_t>(ld) * row;
}

// One thread's eight elements of a row.  kWhole: all inside.  kCodes: states in 8
// bits, else either.
template <typename TX, typename TG, bool kStochastic, bool kCodes, bool kOnce, bool kWhole>
__device__ __forceinline__ void row_piece(const AdamwScalars& h, const StepScalars& s, const RowTensor& t, uint32_t row, int c,
                                          uint32_t key) {
  int cols = t.cols;
  TX* const x = row_at<TX>(t.x, t.ldx, row);
  const TG* const g = row_at<const TG>(const_cast<void*>(t.g), t.ldg, row);
  float xv[8], gv[8], mv[8], vv[8];
  const auto rx = unit_load<kWhole, kOnce>(x, c, cols);
  const auto rg = unit_load<kWhole, kOnce>(g, c, cols);
  const Bits bits(key, static_cast<uint64_t>(row) * static_cast<uint32_t>(cols) + c);
  uint32_t seed_m[8] = {}, seed_v[8] = {};
  if (!kCodes && t.sm == nullptr) {
    float* const m = row_at<float>(t.m, t.ldm, row);
    float* const v = row_at<float>(t.v, t.ldv, row);
    const auto rm = unit_load<kWhole, kOnce>(m, c, cols);
    const auto rv = unit_load<kWhole, kOnce>(v, c, cols);
    unpack8(rx, xv);
    unpack8(rg, gv);
    unpack8(rm, mv);
    unpack8(rv, vv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      moments(h, s, gv[j], mv[j], vv[j]);
      xv[j] = weight(h, s, xv[j], mv[j], __builtin_sqrtf(vv[j]));
    }
    if constexpr (kStochastic && sizeof(TX) == 2) bits.all(seed_m, seed_v);
    if constexpr (kWhole) cols = c + 8;
    store8(m, c, cols, mv);
    store8(v, c, cols, vv);
  } else {
    uint8_t* const m = row_at<uint8_t>(t.m, t.ldm, row);
    uint8_t* const v = row_at<uint8_t>(t.v, t.ldv, row);
    float* const sm = row_at<float>(t.sm, t.ldsm, row) + (c >> 7);
    float* const sv = row_at<float>(t.sv, t.ldsv, row) + (c >> 7);
    const uint2 qm = unit_load_codes<kWhole, kOnce>(m, c, cols), qv = unit_load_codes<kWhole, kOnce>(v, c, cols);
    const float ms = *sm, vs = *sv;
    unpack8(rx, xv);
    unpack8(rg, gv);
    values8(qm, ms, mv);
    values8(qv, vs, vv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      vv[j] *= vv[j];
      moments(h, s, gv[j], mv[j], vv[j]);
    }
    const Among among = roots8(vv);
#pragma unroll
    for (int j = 0; j < 8; ++j) xv[j] = weight(h, s, xv[j], mv[j], vv[j]);
    if (__builtin_expect(among.far, false)) {   // (read anew: kept until here it would cost every launch registers)
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (!(vv[j] < __builtin_inff()) && c + j < cols)
          xv[j] = far_weight(h, s, value_of(x[c + j]), value_of(g[c + j]), mv[j], value_of(v[c + j], *sv), vv[j]);
    }
    if constexpr (kStochastic) bits.all(seed_m, seed_v);
    // past the row's end: zeros, which enter no maximum
    if constexpr (!kWhole) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j >= cols) mv[j] = vv[j] = 0.f;
    }
    float ms2, vs2;
    const uint2 um = to_codes8<kStochastic, false>(mv, seed_m, false, ms2);
    const uint2 uv = to_codes8<kStochastic, true>(vv, seed_v, among.zeros, vs2);
    if constexpr (kWhole) cols = c + 8;
    if constexpr (kWhole) {
      store_any<kOnce>(m + c, um);
      store_any<kOnce>(v + c, uv);
    } else {
      store_codes8(m, c, cols, um);
      store_codes8(v, c, cols, uv);
    }
    if ((threadIdx.x & 15) == 0) {
      *sm = ms2;
      *sv = vs2;
    }
  }
  if constexpr (kStochastic && sizeof(TX) == 2) {
    uint32_t seed[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) seed[j] = Bits::weight(seed_m[j], seed_v[j]);
    store_weights8<kOnce>(x, c, cols, xv, seed);
  } else if constexpr (kWhole) {
    store_whole8<kOnce && sizeof(TX) == 2>(x + c, xv);
  } else {
    store8(x, c, cols, xv);
  }
}

template <typename TX, typename TG, bool kStochastic, bool kCodes, bool kOnce>
__device__ __forceinline__ void row_unit(const AdamwScalars& h, const StepScalars& s, const RowTensor& t, int at,
                                         uint32_t key) {
  const int lanes = t.lanes, across = t.across, down = at / across;
  const int row = (down << (8 - lanes)) + (threadIdx.x >> lanes);
  const int c = (((at - down * across) << lanes) + (threadIdx.x & ((1 << lanes) - 1))) * 8;
  // (the 16 lanes of a block share the row)
  if (row >= t.rows || (c & ~127) >= t.cols) return;
  if (__all(c + 8 <= t.cols)) row_piece<TX, TG, kStochastic, kCodes, kOnce, true>(h, s, t, row, c, key);
  else row_piece<TX, TG, kStochastic, kCodes, kOnce, false>(h, s, t, row, c, key);
}

// Tensors of any kind: rows of their own pitch, or states in 8 bits beside other kinds.
// The states' codes are formed where they lie: 16 lanes hold a block of 128, whose
// maximum they find with four rotations of the lanes, so m and sqrt(v) meet memory only
// as codes.  67 million bf16 weights with codes, stochastically, 152 us (4.5 TB/s); with
// states in fp32 and rows 8 elements apart, to nearest, 269 (5.5), fp32 weights 353 (5.3).
template <bool kStochastic>
__global__ __launch_bounds__(256, 5) void adamw_rows_kernel(AdamwRows a) {
  const int first = a.first[threadIdx.x & (kLanes - 1)];
  const StepScalars s = step_scalars(a.h);
  if (s.skip) return;
  for (int unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const int i = tensor_of(first, unit);
    const RowTensor& t = a.t[i];
    const int at = unit - a.first[i];
    const uint32_t key = kStochastic ? tensor_key(a.h, s.step, t.index) : 0;
    switch (t.kind) {
      case 0: row_unit<float, float, kStochastic, false, false>(a.h, s, t, at, key); break;
      case kBf16Weight: row_unit<uint16_t, float, kStochastic, false, false>(a.h, s, t, at, key); break;
      case kBf16Gradient: row_unit<float, uint16_t, kStochastic, false, false>(a.h, s, t, at, key); break;
      default: row_unit<uint16_t, uint16_t, kStochastic, false, false>(a.h, s, t, at, key);
    }
  }
}

// Tensors with states in 8 bits, all of one kind.  Bound by HBM to nearest: 67 million
// weights with gradients in bf16 112 us (10.1 bytes each, 6.1 TB/s; 123 through the
// caches), in fp32 184 (5.9); stochastically the vector unit has as much to do in bf16
// (132 us; 152 in the kernel above), about 20 instructions an element for its random
// bits.  Six waves per SIMD hide 2% more of it than five; weights in fp32 take five and
// no more (with gradients in fp32, stochastically, 183 us, to nearest 184; with as many
// as fit, 187 and 188).
template <typename TX, typename TG, bool kStochastic, bool kOnce>
__global__ __launch_bounds__(256)
    __attribute__((amdgpu_waves_per_eu(sizeof(TX) == 4 ? 5 : 6, sizeof(TX) == 4 ? 5 : 8))) void adamw_codes_kernel(
        AdamwRows a) {
  const int first = a.first[threadIdx.x & (kLanes - 1)];
  const StepScalars s = step_scalars(a.h);
  if (s.skip) return;
  for (int unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const int i = tensor_of(first, unit);
    const RowTensor& t = a.t[i];
    const uint32_t key = kStochastic ? tensor_key(a.h, s.step, t.index) : 0;
    row_unit<TX, TG, kStochastic, true, kOnce>(a.h, s, t, unit - a.first[i], key);
  }
}

// ---- the gradients' norm ----

__device__ __forceinline__ double sum_of_wave(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

// A thread's four pieces of 16 bytes of a unit.
struct Pieces {
  uint4 u[4];
  int bf;
};

template <typename T>
__device__ __forceinline__ void load_pieces(const NormTensor& t, int64_t row, int64_t at, uint4 (&u)[4]) {
  constexpr int kN = 16 / sizeof(T);
  const T* const p = static_cast<const T*>(t.g) + row * t.ld;
  const int step = kN << t.lanes;
  const int64_t c = at * kN;
  if (row < t.rows && c + 3 * step + kN <= t.cols) {
#pragma unroll
    for (int q = 0; q < 4; ++q) __builtin_memcpy(&u[q], p + c + q * step, 16);
    return;
  }
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t left = row < t.rows ? t.cols - (c + q * step) : 0;
    u[q] = left > 0 ? load16(p + c + q * step, 0, left < kN ? static_cast<int>(left) : kN) : make_uint4(0, 0, 0, 0);
  }
}

__device__ __forceinline__ Pieces load_unit(const NormParts& a, int64_t first, int64_t unit) {
  const int i = tensor_of(first, unit);
  const NormTensor& t = a.t[i];
  const int lanes = t.lanes, at = static_cast<int>(unit - a.first[i]), across = t.across;
  const int down = at / across;
  const int64_t row = ((int64_t)down << (8 - lanes)) + (threadIdx.x >> lanes);
  const int64_t c = ((int64_t)(at - down * across) << (lanes + 2)) + (threadIdx.x & ((1 << lanes) - 1));
  Pieces p;
  p.bf = t.bf;
  if (p.bf) load_pieces<uint16_t>(t, row, c, p.u);
  else load_pieces<float>(t, row, c, p.u);
  return p;
}

__device__ __forceinline__ double add_square(double sum, uint32_t bits) {
  const double d = static_cast<double>(__uint_as_float(bits));
  return fma(d, d, sum);
}

// The squares' sum in fp64, where an fp32 square is exact.  The next unit's loads are
// under way while this one's squares are added.  Bound by HBM: 134 MB take 27 us (5.0
// TB/s), 1.2 GB 206 (5.9), with the 2048 workgroups that the chip holds at once (1024:
// 28.5 and 207; 16384: 27.7 and 201, but eight times the sums to join).
__global__ __launch_bounds__(256) void grad_norm_parts_kernel(NormParts a) {
  __shared__ double red[4];
  const int64_t first = a.first[threadIdx.x & (kLanes - 1)];
  double part[4] = {};
  Pieces p = load_unit(a, first, blockIdx.x);   // (no more workgroups than units)
  for (int64_t unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const Pieces now = p;
    if (unit + gridDim.x < a.units) p = load_unit(a, first, unit + gridDim.x);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t w[4] = {now.u[q].x, now.u[q].y, now.u[q].z, now.u[q].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (now.bf) part[q] = add_square(part[q], w[j] << 16);
        part[q] = add_square(part[q], now.bf ? w[j] & 0xffff0000u : w[j]);
      }
    }
  }
  double sum = (part[0] + part[1]) + (part[2] + part[3]);
  sum = sum_of_wave(sum);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) a.part[blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

// The workgroups' sums in a fixed order, by a launch of its own: 2 us for 1023 of them,
// 2 to 5 for 2048.
__global__ __launch_bounds__(1024) void grad_norm_join_kernel(const double* part, int count, double max_norm,
                                                              float* out) {
  __shared__ double red[16];
  double sum = 0.0;
#pragma unroll 8
  for (int i = threadIdx.x; i < count; i += 1024) sum += part[i];
  sum = sum_of_wave(sum);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) {
    double total = 0.0;
#pragma unroll
    for (int w = 0; w < 16; ++w) total += red[w];
    const double norm = __builtin_sqrt(total);
    out[0] = static_cast<float>(norm);
    out[1] = norm < __builtin_inf() ? (norm > max_norm ? static_cast<float>(max_norm / norm) : 1.f)
                                    : __builtin_nanf("");
  }
}

// A workgroup per unit, as far as a launch goes (2^32 threads); more are walked.
constexpr int kMostGroups = (1 << 24) - 1;

// Units from which on a launch goes past the caches, which would keep too little of it
// until the next step (bf16 weights and gradients, states in 32 bits: 8192 units 61.4 us
// past the caches and 71.4 through them, 4096 32.3 both ways, 2048 17.5 and 15.4; in 8
// bits: 16384 units 59.9 and 64.4, 8192 32 both ways).
constexpr int kPastUnits = 1 << 13;

inline dim3 grid_of(int units) { return dim3(units < kMostGroups ? units : kMostGroups); }

}  // namespace

hipError_t launch_adamw_flat(const AdamwFlat& a, bool stochastic, hipStream_t s) {
  const bool once = a.units >= kPastUnits;
  const auto kernel = stochastic ? (once ? adamw_flat_kernel<true, true> : adamw_flat_kernel<true, false>)
                                 : (once ? adamw_flat_kernel<false, true> : adamw_flat_kernel<false, false>);
  hipLaunchKernelGGL(kernel, grid_of(a.units), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <bool kStochastic, bool kOnce>
static hipError_t codes(const AdamwRows& a, int kind, hipStream_t s) {
  const auto kernel = kind == 0               ? adamw_codes_kernel<float, float, kStochastic, kOnce>
                      : kind == kBf16Weight   ? adamw_codes_kernel<uint16_t, float, kStochastic, kOnce>
                      : kind == kBf16Gradient ? adamw_codes_kernel<float, uint16_t, kStochastic, kOnce>
                                              : adamw_codes_kernel<uint16_t, uint16_t, kStochastic, kOnce>;
  hipLaunchKernelGGL(kernel, grid_of(a.units), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_adamw_rows(const AdamwRows& a, int kind, bool stochastic, hipStream_t s) {
  if (kind < 0) {
    const auto kernel = stochastic ? adamw_rows_kernel<true> : adamw_rows_kernel<false>;
    hipLaunchKernelGGL(kernel, grid_of(a.units), dim3(256), 0, s, a);
    return hipGetLastError();
  }
  if (a.units >= kPastUnits) return stochastic ? codes<true, true>(a, kind, s) : codes<false, true>(a, kind, s);
  return stochastic ? codes<true, false>(a, kind, s) : codes<false, false>(a, kind, s);
}

hipError_t launch_grad_norm_parts(const NormParts& a, int groups, hipStream_t s) {
  hipLaunchKernelGGL(grad_norm_parts_kernel, dim3(groups), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_grad_norm_join(const double* part, int count, double max_norm, float* out, hipStream_t s) {
  hipLaunchKernelGGL(grad_norm_join_kernel, dim3(1), dim3(1024), 0, s, part, count, max_norm, out);
  return hipGetLastError();
}

}  // namespace ortho
