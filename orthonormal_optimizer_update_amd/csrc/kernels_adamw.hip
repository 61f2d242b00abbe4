// AdamW on many tensors per launch, and the gradients' norm.
#include "adamw.h"
#include "fp8.h"

// Products and sums join where the code says so and nowhere else: a tensor comes
// out the same whichever kernel its layout picks.
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

struct Bits {
  uint32_t a, b;
  __device__ __forceinline__ Bits(uint32_t key, int64_t element) {
    const uint64_t e = static_cast<uint64_t>(element);
    a = mix(static_cast<uint32_t>(e) ^ (key + kStride * static_cast<uint32_t>(e >> 32)));
    b = mix(a + kStride);
  }
  __device__ __forceinline__ uint32_t m() const { return a >> 12; }
  __device__ __forceinline__ uint32_t v() const { return b >> 12; }
  __device__ __forceinline__ uint32_t x() const { return (a & 4095u) << 4 | (b & 15u); }
};

// x with `bits` added below its bit kFrom and cut there; infinities and NaN stay.
template <int kFrom>
__device__ __forceinline__ float cut(float x, uint32_t bits) {
  const uint32_t u = (__float_as_uint(x) + bits) & ~((1u << kFrom) - 1);
  return __builtin_fabsf(x) < __builtin_inff() ? __uint_as_float(u) : x;
}

// |q| <= 448 to a value that e4m3 holds: below 2^-6 its steps are 2^-9, which are
// fp32's bit 20 after 2^-6 is added.
__device__ __forceinline__ float cut_e4m3(float q, uint32_t bits) {
  const float a = __builtin_fabsf(q), shift = a < 0x1p-6f ? 0x1p-6f : 0.f;
  const float c = cut<20>(a + shift, bits) - shift;
  return __builtin_copysignf(c, q);
}

// ---- the step ----

struct StepScalars {
  float keep, size, root, factor;
  int64_t step;
  bool skip;
};

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
__device__ __forceinline__ void adamw(const AdamwScalars& h, const StepScalars& s, float& x, float g, float& m,
                                      float& v) {
  g *= s.factor;
  m = fmaf(h.b1, m, h.c1 * g);
  v = fmaf(h.b2, v, h.c2 * (g * g));
  const float down = fmaf(__builtin_sqrtf(v), s.root, h.eps);
  x = fmaf(s.keep, x, -(s.size * (m / down)));
}

// The tensor of a unit; `first` is this lane's.
template <typename I>
__device__ __forceinline__ int tensor_of(I first, I unit) {
  return __builtin_amdgcn_readfirstlane(__popcll(__ballot(first <= unit)) - 1);
}

// Eight elements at c of a unit's `limit`; a whole unit needs no look at its end.
template <bool kWhole, typename T>
__device__ __forceinline__ Raw8<T> unit_load(const T* p, int c, int limit) {
  if constexpr (!kWhole) return load_raw8(p, c, limit);
  Raw8<T> r;
  __builtin_memcpy(&r, p + c, sizeof(r));
  return r;
}

template <typename TX, typename TG, bool kStochastic, bool kWhole>
__device__ __forceinline__ void flat_unit(const AdamwScalars& h, const StepScalars& s, const FlatTensor& t,
                                          int64_t base, int limit, uint32_t key) {
  TX* const x = static_cast<TX*>(t.x) + base;
  const TG* const g = static_cast<const TG*>(t.g) + base;
  float *const m = t.m + base, *const v = t.v + base;
  const int c = threadIdx.x * 8;
  float xv[8], gv[8], mv[8], vv[8];
  const auto rx = unit_load<kWhole>(x, c, limit);
  const auto rg = unit_load<kWhole>(g, c, limit);
  const auto rm = unit_load<kWhole>(m, c, limit);
  const auto rv = unit_load<kWhole>(v, c, limit);
  unpack8(rx, xv);
  unpack8(rg, gv);
  unpack8(rm, mv);
  unpack8(rv, vv);
#pragma unroll
  for (int j = 0; j < 8; ++j) adamw(h, s, xv[j], gv[j], mv[j], vv[j]);
  if constexpr (kStochastic && sizeof(TX) == 2) {
#pragma unroll
    for (int j = 0; j < 8; ++j) xv[j] = cut<16>(xv[j], Bits(key, base + c + j).x());
  }
  if constexpr (kWhole) limit = kUnit;
  store8(x, c, limit, xv);
  store8(m, c, limit, mv);
  store8(v, c, limit, vv);
}

template <bool kStochastic, bool kWhole>
__device__ __forceinline__ void flat_by_kind(const AdamwScalars& h, const StepScalars& s, const FlatTensor& t,
                                             int64_t base, int limit, uint32_t key) {
  switch (t.kind) {
    case 0: flat_unit<float, float, kStochastic, kWhole>(h, s, t, base, limit, key); break;
    case kBf16Weight: flat_unit<uint16_t, float, kStochastic, kWhole>(h, s, t, base, limit, key); break;
    case kBf16Gradient: flat_unit<float, uint16_t, kStochastic, kWhole>(h, s, t, base, limit, key); break;
    default: flat_unit<uint16_t, uint16_t, kStochastic, kWhole>(h, s, t, base, limit, key);
  }
}

template <bool kStochastic>
__global__ __launch_bounds__(256) void adamw_flat_kernel(AdamwFlat a) {
  const int first = a.first[threadIdx.x & (kLanes - 1)];
  const StepScalars s = step_scalars(a.h);
  if (s.skip) return;
  for (int unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const int i = tensor_of(first, unit);
    const FlatTensor& t = a.t[i];
    const int64_t base = (int64_t)(unit - a.first[i]) * kUnit, left = t.n - base;
    const uint32_t key = kStochastic ? tensor_key(a.h, s.step, t.index) : 0;
    if (left >= kUnit) flat_by_kind<kStochastic, true>(a.h, s, t, base, kUnit, key);
    else flat_by_kind<kStochastic, false>(a.h, s, t, base, static_cast<int>(left), key);
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

__device__ __forceinline__ float max_of_16_lanes(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

// Codes of a block's eight elements here, the 16 lanes of a block together.
template <bool kStochastic, bool kPositive>
__device__ __forceinline__ uint2 to_codes8(const float (&v)[8], const uint32_t (&bits)[8], float& scale) {
  float top = 0.f, f;
#pragma unroll
  for (int j = 0; j < 8; ++j) top = fmaxf(top, finite_abs(v[j]));
  block_scale<false>(max_of_16_lanes(top), scale, f);
  float q[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    q[j] = v[j] * f;
    if constexpr (kStochastic) {
      // (the largest may come out a rounding above 448; infinities and NaN stay)
      const float in = __builtin_fabsf(q[j]) < 512.f ? __builtin_copysignf(fminf(__builtin_fabsf(q[j]), kFp8Top), q[j]) : q[j];
      q[j] = cut_e4m3(in, bits[j]);
    }
    if constexpr (kPositive) q[j] = v[j] > 0.f && q[j] < 0x1p-9f ? 0x1p-9f : q[j];
  }
  return make_uint2(pack_e4m3x4(q[0], q[1], q[2], q[3]), pack_e4m3x4(q[4], q[5], q[6], q[7]));
}

template <typename TX, typename TG, bool kStochastic>
__device__ __forceinline__ void row_unit(const AdamwScalars& h, const StepScalars& s, const RowTensor& t, int at,
                                         uint32_t key) {
  const int lanes = t.lanes, across = t.across, cols = t.cols, down = at / across;
  const int row = (down << (8 - lanes)) + (threadIdx.x >> lanes);
  const int c = (((at - down * across) << lanes) + (threadIdx.x & ((1 << lanes) - 1))) * 8;
  // (the 16 lanes of a block share the row)
  if (row >= t.rows || (c & ~127) >= cols) return;
  TX* const x = static_cast<TX*>(t.x) + row * t.ldx;
  const TG* const g = static_cast<const TG*>(t.g) + row * t.ldg;
  const int64_t element = (int64_t)row * cols + c;
  float xv[8], gv[8], mv[8], vv[8];
  const auto rx = load_raw8(x, c, cols);
  const auto rg = load_raw8(g, c, cols);
  if (t.sm == nullptr) {
    float* const m = static_cast<float*>(t.m) + row * t.ldm;
    float* const v = static_cast<float*>(t.v) + row * t.ldv;
    const auto rm = load_raw8(m, c, cols);
    const auto rv = load_raw8(v, c, cols);
    unpack8(rx, xv);
    unpack8(rg, gv);
    unpack8(rm, mv);
    unpack8(rv, vv);
#pragma unroll
    for (int j = 0; j < 8; ++j) adamw(h, s, xv[j], gv[j], mv[j], vv[j]);
    if constexpr (kStochastic && sizeof(TX) == 2) {
#pragma unroll
      for (int j = 0; j < 8; ++j) xv[j] = cut<16>(xv[j], Bits(key, element + j).x());
    }
    store8(m, c, cols, mv);
    store8(v, c, cols, vv);
  } else {
    uint8_t* const m = static_cast<uint8_t*>(t.m) + row * t.ldm;
    uint8_t* const v = static_cast<uint8_t*>(t.v) + row * t.ldv;
    float* const sm = t.sm + row * t.ldsm + (c >> 7);
    float* const sv = t.sv + row * t.ldsv + (c >> 7);
    const uint2 qm = load_codes8(m, c, cols), qv = load_codes8(v, c, cols);
    const float ms = *sm, vs = *sv;
    unpack8(rx, xv);
    unpack8(rg, gv);
    values8(qm, ms, mv);
    values8(qv, vs, vv);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      vv[j] *= vv[j];
      adamw(h, s, xv[j], gv[j], mv[j], vv[j]);
      // (its code could not say infinite)
      vv[j] = __builtin_sqrtf(vv[j] > __FLT_MAX__ ? __FLT_MAX__ : vv[j]);
    }
    uint32_t bm[8] = {}, bv[8] = {};
    if constexpr (kStochastic) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const Bits r(key, element + j);
        bm[j] = r.m();
        bv[j] = r.v();
        if constexpr (sizeof(TX) == 2) xv[j] = cut<16>(xv[j], r.x());
      }
    }
    // past the row's end: zeros, which enter no maximum
    if (c + 8 > cols) {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j >= cols) mv[j] = vv[j] = 0.f;
    }
    float ms2, vs2;
    const uint2 um = to_codes8<kStochastic, false>(mv, bm, ms2);
    const uint2 uv = to_codes8<kStochastic, true>(vv, bv, vs2);
    store_codes8(m, c, cols, um);
    store_codes8(v, c, cols, uv);
    if ((threadIdx.x & 15) == 0) {
      *sm = ms2;
      *sv = vs2;
    }
  }
  store8(x, c, cols, xv);
}

template <bool kStochastic>
__global__ __launch_bounds__(256) void adamw_rows_kernel(AdamwRows a) {
  const int first = a.first[threadIdx.x & (kLanes - 1)];
  const StepScalars s = step_scalars(a.h);
  if (s.skip) return;
  for (int unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const int i = tensor_of(first, unit);
    const RowTensor& t = a.t[i];
    const int at = unit - a.first[i];
    const uint32_t key = kStochastic ? tensor_key(a.h, s.step, t.index) : 0;
    switch (t.kind) {
      case 0: row_unit<float, float, kStochastic>(a.h, s, t, at, key); break;
      case kBf16Weight: row_unit<uint16_t, float, kStochastic>(a.h, s, t, at, key); break;
      case kBf16Gradient: row_unit<float, uint16_t, kStochastic>(a.h, s, t, at, key); break;
      default: row_unit<uint16_t, uint16_t, kStochastic>(a.h, s, t, at, key);
    }
  }
}

// ---- the gradients' norm ----

__device__ __forceinline__ double sum_of_wave(double x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o, 64);
  return x;
}

template <typename T>
__device__ __forceinline__ double squares(const T* row, int64_t c, int64_t cols, int step) {
  Raw8<T> r[4];
  if (c + 3 * step + 8 <= cols) {
#pragma unroll
    for (int q = 0; q < 4; ++q) r[q] = load_raw8(row + c + q * step, 0, 8);
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int64_t at = c + q * step, left = cols - at;
      r[q] = left > 0 ? load_raw8(row + at, 0, left < 8 ? static_cast<int>(left) : 8) : Raw8<T>{};
    }
  }
  double sum = 0.0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float v[8];
    unpack8(r[q], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const double d = static_cast<double>(v[j]);
      sum = fma(d, d, sum);
    }
  }
  return sum;
}

__global__ __launch_bounds__(256) void grad_norm_parts_kernel(NormParts a) {
  __shared__ double red[4];
  const int64_t first = a.first[threadIdx.x & (kLanes - 1)];
  double sum = 0.0;
  for (int64_t unit = blockIdx.x; unit < a.units; unit += gridDim.x) {
    const int i = tensor_of(first, unit);
    const NormTensor& t = a.t[i];
    const int lanes = t.lanes, at = static_cast<int>(unit - a.first[i]), across = t.across;
    const int down = at / across;
    const int64_t row = ((int64_t)down << (8 - lanes)) + (threadIdx.x >> lanes);
    const int64_t c = ((int64_t)(at - down * across) << (lanes + 5)) + (threadIdx.x & ((1 << lanes) - 1)) * 8;
    if (row < t.rows) {
      if (t.bf) sum += squares(static_cast<const uint16_t*>(t.g) + row * t.ld, c, t.cols, 8 << lanes);
      else sum += squares(static_cast<const float*>(t.g) + row * t.ld, c, t.cols, 8 << lanes);
    }
  }
  sum = sum_of_wave(sum);
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x == 0) a.part[blockIdx.x] = red[0] + red[1] + red[2] + red[3];
}

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

// Workgroups of 256 that the chip holds at once; more units than that are walked.
constexpr int kResident = 2048;

inline dim3 grid_of(int units) { return dim3(units < kResident ? units : kResident); }

}  // namespace

hipError_t launch_adamw_flat(const AdamwFlat& a, bool stochastic, hipStream_t s) {
  if (stochastic) hipLaunchKernelGGL(adamw_flat_kernel<true>, grid_of(a.units), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(adamw_flat_kernel<false>, grid_of(a.units), dim3(256), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_adamw_rows(const AdamwRows& a, bool stochastic, hipStream_t s) {
  if (stochastic) hipLaunchKernelGGL(adamw_rows_kernel<true>, grid_of(a.units), dim3(256), 0, s, a);
  else hipLaunchKernelGGL(adamw_rows_kernel<false>, grid_of(a.units), dim3(256), 0, s, a);
  return hipGetLastError();
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
