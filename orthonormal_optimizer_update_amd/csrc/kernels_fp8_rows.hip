// Conversion to 8-bit codes with block scales, and the RMS norm around it: the
// residual's addition, the 8-bit output and the gradient.  All are bound by
// HBM traffic: each element is read once, held in registers, and written once
// per output.  In bf16, with new operands in every call: quantisation by rows of
// 8192 x 4096 24.0 us (4.2 TB/s), both orientations 34.8 (3.9); the norm with
// residual, sum and y 58.6 (5.2); the gradient with dSum 59.9 (4.5).  In fp32, 4096 x
// 8192: 30.1 (5.6), 47.6 (4.2), 124 (4.6), 117 (4.6).  (A copy of 1 GiB: 5.1.)
//
// Not so for the norms' longest rows: over 16384 columns (the fp32 gradient: over
// 8192) a thread's pieces pass its 128 registers and go through scratch.  1024 x
// 32768 in bf16: norm 164 us (66.8 as 2048 x 16384), gradient 232 (82.9); in fp32
// 249 (126) and 383 (145).  Nor for rows of 128, which fill a quarter of a wave:
// 131072 x 128 in bf16 takes 104 us (1.5 TB/s), its gradient 165.
#include <type_traits>

#include "fp8.h"

namespace ortho {

namespace {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Largest value over the 16 lanes that hold one block of 128 (8 per lane).
__device__ __forceinline__ float max16(float v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o, 64));
  return v;
}

__device__ __forceinline__ uint32_t max16(uint32_t v) {
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) {
    const uint32_t w = __shfl_xor(v, o, 64);
    v = v > w ? v : w;
  }
  return v;
}

__device__ __forceinline__ float top8(const float (&v)[8]) {
  float t = 0.f;
#pragma unroll
  for (int j = 0; j < 8; ++j) t = fmaxf(t, finite_abs(v[j]));
  return t;
}

__device__ __forceinline__ uint2 codes8(const float (&v)[8], float f) {
  return make_uint2(pack_e4m3x4(v[0] * f, v[1] * f, v[2] * f, v[3] * f),
                    pack_e4m3x4(v[4] * f, v[5] * f, v[6] * f, v[7] * f));
}

// Codes by rows with a scale per 1 x 128 block: 16 lanes per block.
template <typename T, bool kE8m0>
__global__ __launch_bounds__(256) void quant_rows_kernel(QuantArgs a) {
  const int nb = (a.n + kFp8Block - 1) / kFp8Block;
  const int64_t blk = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);
  if (blk >= (int64_t)a.m * nb) return;
  const int row = static_cast<int>(blk / nb), b = static_cast<int>(blk % nb);
  const int c = b * kFp8Block + (threadIdx.x & 15) * 8;
  float v[8];
  load8(static_cast<const T*>(a.x) + row * a.ldx, c, a.n, v);
  float scale, f;
  block_scale<kE8m0>(max16(top8(v)), scale, f);
  store_codes8(a.q + row * a.ldq, c, a.n, codes8(v, f));
  if ((threadIdx.x & 15) == 0) store_scale<kE8m0>(a.s, row * a.lds + b, scale);
}

// A 128 x 128 tile per workgroup, 8 x 8 elements per thread (columns of 16
// threads, rows of 16 groups): codes by rows, transposed, or both, from one
// read.  kTiles: one scale for the tile; otherwise one per row for the codes
// by rows and one per column for the transposed ones.  The largest magnitudes
// are found on the elements' bits (two bf16 per instruction); only a tile that
// holds an infinity or NaN looks at the elements one by one.
template <typename T, bool kE8m0, bool kTiles>
__global__ __launch_bounds__(256, sizeof(T) == 2 ? 4 : 1) void quant_tile_kernel(QuantArgs a) {
  constexpr int kPitch = 128 + 16;   // bytes per LDS row of transposed codes
  __shared__ __attribute__((aligned(16))) uint8_t tile[128 * kPitch];
  __shared__ uint32_t red[4][128];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int nbn = (a.n + 127) / 128;
  const int tn = blockIdx.x % nbn, tm = blockIdx.x / nbn;
  const int cl = (t & 15) * 8, rl = (t >> 4) * 8;
  const int c = tn * 128 + cl, r0 = tm * 128 + rl;
  Raw8<T> x[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    if (r0 + i < a.m) x[i] = load_raw8(static_cast<const T*>(a.x) + (r0 + i) * a.ldx, c, a.n);
    else x[i] = Raw8<T>{};
  }
  // largest finite magnitudes: of each row's 8 elements, and of each column's
  uint32_t rows[8], cols[8];
  Mags<T> down = magnitudes(x[0]);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const Mags<T> m = magnitudes(x[i]);
    rows[i] = largest(m);
    if (i > 0) down = max_of(down, m);
  }
  if (largest(down) >= kInfBits) {
#pragma unroll
    for (int j = 0; j < 8; ++j) cols[j] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      rows[i] = 0;
      const Mags<T> m = magnitudes(x[i]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t e = element(m, j) < kInfBits ? element(m, j) : 0;
        rows[i] = rows[i] > e ? rows[i] : e;
        cols[j] = cols[j] > e ? cols[j] : e;
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) cols[j] = element(down, j);
  }
  float fr[8], fc[8];   // factors by row and by column
  if constexpr (kTiles) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = top > rows[i] ? top : rows[i];
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) {
      const uint32_t w = __shfl_xor(top, o, 64);
      top = top > w ? top : w;
    }
    if (lane == 0) red[0][wave] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) top = top > red[0][w] ? top : red[0][w];
    float scale, f;
    block_scale<kE8m0>(__uint_as_float(top), scale, f);
#pragma unroll
    for (int i = 0; i < 8; ++i) fr[i] = fc[i] = f;
    if (t == 0) {
      if (a.q) store_scale<kE8m0>(a.s, tm * a.lds + tn, scale);
      if (a.qt) store_scale<kE8m0>(a.st, tn * a.ldst + tm, scale);
    }
  } else {
    if (a.qt) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t top = cols[j];
#pragma unroll
        for (int o = 16; o <= 32; o <<= 1) {
          const uint32_t w = __shfl_xor(top, o, 64);
          top = top > w ? top : w;
        }
        cols[j] = top;
      }
      if (lane < 16) {
        *reinterpret_cast<uint4*>(&red[wave][cl]) = make_uint4(cols[0], cols[1], cols[2], cols[3]);
        *reinterpret_cast<uint4*>(&red[wave][cl + 4]) = make_uint4(cols[4], cols[5], cols[6], cols[7]);
      }
    }
    if (a.q) {
      // lane l of a row's 16 works out the scale of row l / 2
      uint32_t mine = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t top = max16(rows[i]);
        if ((lane & 15) >> 1 == i) mine = top;
      }
      float scale, f;
      block_scale<kE8m0>(__uint_as_float(mine), scale, f);
      const int r = r0 + ((lane & 15) >> 1);
      if ((lane & 1) == 0 && r < a.m) store_scale<kE8m0>(a.s, r * a.lds + tn, scale);
#pragma unroll
      for (int i = 0; i < 8; ++i) fr[i] = __shfl(f, (lane & 48) + 2 * i, 64);
    }
    if (a.qt) {
      __syncthreads();
      // thread c (of 128) works out the scale of column c
      float* const factors = reinterpret_cast<float*>(&red[0][0]);
      float f = 0.f;
      if (t < 128) {
        uint32_t top = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) top = top > red[w][t] ? top : red[w][t];
        float scale;
        block_scale<kE8m0>(__uint_as_float(top), scale, f);
        if (tn * 128 + t < a.n) store_scale<kE8m0>(a.st, (tn * 128 + t) * a.ldst + tm, scale);
        factors[t] = f;   // its own column's, which no one else reads above
      }
      __syncthreads();
#pragma unroll
      for (int j = 0; j < 8; ++j) fc[j] = factors[cl + j];
    }
  }
  float v[8][8];
#pragma unroll
  for (int i = 0; i < 8; ++i) unpack8(x[i], v[i]);
  if (a.q) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (r0 + i < a.m) store_codes8(a.q + (r0 + i) * a.ldq, c, a.n, codes8(v[i], fr[i]));
  }
  if (a.qt) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float col[8] = {v[0][j], v[1][j], v[2][j], v[3][j], v[4][j], v[5][j], v[6][j], v[7][j]};
      *reinterpret_cast<uint2*>(tile + (cl + j) * kPitch + rl) = codes8(col, fc[j]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int cc = (t >> 3) + 32 * i, k = (t & 7) * 16;   // column of X, offset along its rows
      if (tn * 128 + cc >= a.n) continue;
      const uint4 u = *reinterpret_cast<const uint4*>(tile + cc * kPitch + k);
      uint8_t* dst = a.qt + (tn * 128 + cc) * a.ldqt;
      const int m0 = tm * 128 + k;
      if (m0 + 16 <= a.m) {
        __builtin_memcpy(dst + m0, &u, 16);
      } else {
        store_codes8(dst, m0, a.m, make_uint2(u.x, u.y));
        store_codes8(dst, m0 + 8, a.m, make_uint2(u.z, u.w));
      }
    }
  }
}

// Sums of two values over the workgroup in a fixed order; every thread gets
// the totals.  One barrier: calls alternate between two buffers.
template <int kThreads>
__device__ __forceinline__ void block_sum2(float& x, float& y, float (*red)[2][kThreads / 64], int turn) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    x += __shfl_xor(x, o, 64);
    y += __shfl_xor(y, o, 64);
  }
  if constexpr (kThreads > 64) {
    if ((threadIdx.x & 63) == 0) {
      red[turn][0][threadIdx.x >> 6] = x;
      red[turn][1][threadIdx.x >> 6] = y;
    }
    __syncthreads();
    x = y = 0.f;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
      x += red[turn][0][w];
      y += red[turn][1][w];
    }
  }
}

__device__ __forceinline__ void load_w8(const void* w, int w_bf, int c, int n, float (&v)[8]) {
  if (w_bf) load8(static_cast<const uint16_t*>(w), c, n, v);
  else load8(static_cast<const float*>(w), c, n, v);
}

// A workgroup takes the rows g, g + groups, ..., 8 kC elements per thread.  Up
// to kC = 2 W stays in registers, and the next row's loads go out before this
// row's sum is waited for; longer rows need more registers than there are (so
// do fp32 rows of over 8192 in the gradient).
//   r = round(x + res), t = 1 / sqrt(mean r^2 + eps), y = r t w
// The sum is rounded to its storage type first and the rounded one is
// normalised, so that the gradient, which sees only the stored sum, is that of
// what was computed.
//
// The codes do not see the rounding of y: with u = r w, a block's codes are
// u (448 / max|u|), in which t cancels (power-of-two scales: u (t / s), t kept
// in fp64), and u and the factor each carry their rounding error as a second
// fp32.  What is left are the roundings of max|u| (of the row's sum, with
// power-of-two scales) and of the result before the one to e4m3: of the 33.5
// million codes of 8192 x 4096 about 14 are on the other side of a tie (20
// without the second fp32s, which cost 4% of the time in bf16).  Blocks whose u is
// no number that stands for y take the codes from y.
template <typename T, bool kE8m0, int kThreads, int kC>
__global__ __launch_bounds__(kThreads) void rms_norm_fp8_kernel(NormArgs a) {
  __shared__ float red[2][2][kThreads / 64];
  const int t = threadIdx.x;
  constexpr bool kAhead = kC <= 2;
  float w[kAhead ? kC : 1][8];
  Raw8<T> x[kC], res[kC];
  if constexpr (kAhead) {
#pragma unroll
    for (int i = 0; i < kC; ++i) load_w8(a.w, a.w_bf, (i * kThreads + t) * 8, a.n, w[i]);
  }
  auto load_row = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = (i * kThreads + t) * 8;
      x[i] = load_raw8(static_cast<const T*>(a.x) + row * a.ldx, c, a.n);
      if (a.res) res[i] = load_raw8(static_cast<const T*>(a.res) + row * a.ldres, c, a.n);
    }
  };
  if (kAhead) load_row(blockIdx.x);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x, turn ^= 1) {
    if (!kAhead) load_row(row);
    float v[kC][8];
    float sq = 0.f, unused = 0.f;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      unpack8(x[i], v[i]);
      if (a.res) {
        float r[8];
        unpack8(res[i], r);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] += r[j];
          if constexpr (sizeof(T) == 2) v[i][j] = static_cast<float>(to_bf16(v[i][j]));
        }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) sq += v[i][j] * v[i][j];
    }
    if (kAhead && row + gridDim.x < a.m) load_row(row + gridDim.x);
    if (a.sum) {
#pragma unroll
      for (int i = 0; i < kC; ++i)
        store8(static_cast<T*>(a.sum) + row * a.ldsum, (i * kThreads + t) * 8, a.n, v[i]);
    }
    block_sum2<kThreads>(sq, unused, red, turn);
    const double rsd = 1.0 / __builtin_sqrt(static_cast<double>(sq / a.n + a.eps));
    const float rs = static_cast<float>(rsd);
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = (i * kThreads + t) * 8;
      if (c - (t & 15) * 8 >= a.n) continue;   // whole block past the row's end
      float u[8], ul[8], q[8];
      float (&wi)[8] = w[kAhead ? i : 0];
      if (!kAhead) load_w8(a.w, a.w_bf, c, a.n, wi);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = v[i][j] * wi[j];
        ul[j] = fmaf(v[i][j], wi[j], -u[j]);
      }
      if (a.y) {
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = v[i][j] * rs * wi[j];
        store8(static_cast<T*>(a.y) + row * a.ldy, c, a.n, y);
      }
      // (NaN counts for nothing here, and below the codes are of y itself)
      float top = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, __builtin_fabsf(u[j]));
      top = max16(top);
      float scale, f, gh, gl;
      if (top >= 0x1p-100f && top < __builtin_inff() && rsd > 0.0 && rsd < 1e300) {
        block_scale<kE8m0>(static_cast<float>(top * rsd), scale, f);
        // fp32 scales: 448 / top, unless the scale is the smallest
        const double g = !kE8m0 && scale > 0x1p-126f ? 448.0 / top : rsd / scale;
        gh = static_cast<float>(g);
        gl = static_cast<float>(g - gh);
      } else {
        // u is not a number that stands for y: infinite (as r may be, or only the
        // product), too small to hold its rounding error, or of a row without a factor
        float y[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = v[i][j] * rs * wi[j];
        block_scale<kE8m0>(max16(top8(y)), scale, f);
        gh = gl = __builtin_nanf("");
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float e = fmaf(u[j], gh, fmaf(ul[j], gh, u[j] * gl));
        // (not finite: the product as it is, so that infinities give NaN codes)
        q[j] = __builtin_fabsf(e) <= 512.f ? e : v[i][j] * rs * wi[j] * f;
      }
      store_codes8(a.q + row * a.ldq, c, a.n, codes8(q, 1.f));
      if ((t & 15) == 0) store_scale<kE8m0>(a.s, row * a.lds + c / kFp8Block, scale);
    }
  }
}

// Unpacks r anew from here on: four registers of bf16 instead of eight of
// fp32 stay alive across the sums.
__device__ __forceinline__ void again(Raw8<uint16_t>& r) {
  asm volatile("" : "+v"(r.a.x), "+v"(r.a.y), "+v"(r.a.z), "+v"(r.a.w));
}
__device__ __forceinline__ void again(Raw8<float>&) {}

// Gradient of the norm.  With h = dy w, u = x t:
//   dx = t (h - u mean(h u)) (+ dsum),  dw = sum over rows of dy u
// Workgroup g takes the rows g, g + groups, ..., as above, and keeps its part
// of dw in registers; the parts are added in a fixed order by a second launch.
template <typename T, int kThreads, int kC>
__global__ __launch_bounds__(kThreads, kC <= 2 && sizeof(T) == 2 ? 4 : 1) void rms_norm_grad_kernel(NormGradArgs a) {
  __shared__ float red[2][2][kThreads / 64];
  const int t = threadIdx.x;
  constexpr bool kAhead = kC <= 2 && (sizeof(T) == 2 || kThreads <= 512);
  float w[kAhead ? kC : 1][8], dw[kC][8];
  Raw8<T> nx[kC], ng[kC], nd[kAhead ? kC : 1];
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    if (kAhead) load_w8(a.w, a.w_bf, (i * kThreads + t) * 8, a.n, w[kAhead ? i : 0]);
#pragma unroll
    for (int j = 0; j < 8; ++j) dw[i][j] = 0.f;
  }
  auto load_row = [&](int64_t row) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = (i * kThreads + t) * 8;
      nx[i] = load_raw8(static_cast<const T*>(a.x) + row * a.ldx, c, a.n);
      ng[i] = load_raw8(static_cast<const T*>(a.dy) + row * a.lddy, c, a.n);
      if (kAhead && a.dsum)
        nd[kAhead ? i : 0] = load_raw8(static_cast<const T*>(a.dsum) + row * a.lddsum, c, a.n);
    }
  };
  if (kAhead) load_row(blockIdx.x);
  int turn = 0;
  for (int64_t row = blockIdx.x; row < a.m; row += a.groups, turn ^= 1) {
    if (!kAhead) load_row(row);
    Raw8<T> rx[kC], rg[kC], rd[kAhead ? kC : 1];
    float sq = 0.f, dot = 0.f, unused;
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      rx[i] = nx[i];
      rg[i] = ng[i];
      if (kAhead) rd[kAhead ? i : 0] = nd[kAhead ? i : 0];
      float x[8], g[8];
      unpack8(rx[i], x);
      unpack8(rg[i], g);
      float (&wi)[8] = w[kAhead ? i : 0];
      if (!kAhead) load_w8(a.w, a.w_bf, (i * kThreads + t) * 8, a.n, wi);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        sq += x[j] * x[j];
        dot += x[j] * (g[j] * wi[j]);
      }
    }
    if (kAhead && row + a.groups < a.m) load_row(row + a.groups);
    block_sum2<kThreads>(sq, dot, red, turn);
    const float rs = 1.f / __builtin_sqrtf(sq / a.n + a.eps);
    float mean = dot * rs / a.n;   // mean(h u)
    // Of rows far from 1 (no eps, or huge), x h may leave fp32's range where u h
    // does not: their sums are formed of u.  (The same for the workgroup.)
    if (!(rs >= 0x1p-16f && rs <= 0x1p16f && __builtin_fabsf(dot) < __builtin_inff())) {
      dot = unused = 0.f;
#pragma unroll
      for (int i = 0; i < kC; ++i) {
        float x[8], g[8];
        again(rx[i]);
        again(rg[i]);
        unpack8(rx[i], x);
        unpack8(rg[i], g);
        float (&wi)[8] = w[kAhead ? i : 0];
        if (!kAhead) load_w8(a.w, a.w_bf, (i * kThreads + t) * 8, a.n, wi);
#pragma unroll
        for (int j = 0; j < 8; ++j) dot += x[j] * rs * (g[j] * wi[j]);
      }
      turn ^= 1;
      block_sum2<kThreads>(dot, unused, red, turn);
      mean = dot / a.n;
    }
#pragma unroll
    for (int i = 0; i < kC; ++i) {
      const int c = (i * kThreads + t) * 8;
      float o[8], x[8], g[8], d[8];
      float (&wi)[8] = w[kAhead ? i : 0];
      if (!kAhead) {
        load_w8(a.w, a.w_bf, c, a.n, wi);
        if (a.dsum) rd[0] = load_raw8(static_cast<const T*>(a.dsum) + row * a.lddsum, c, a.n);
      }
      again(rx[i]);
      again(rg[i]);
      unpack8(rx[i], x);
      unpack8(rg[i], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = x[j] * rs;
        dw[i][j] += g[j] * u;
        o[j] = rs * (g[j] * wi[j] - u * mean);
      }
      if (a.dsum) {
        unpack8(rd[kAhead ? i : 0], d);
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] += d[j];
      }
      store8(static_cast<T*>(a.dx) + row * a.lddx, c, a.n, o);
    }
  }
#pragma unroll
  for (int i = 0; i < kC; ++i)
    store8(a.part + (int64_t)blockIdx.x * a.ldpart, (i * kThreads + t) * 8, a.n, dw[i]);
}

// dw: kCols columns per workgroup, the parts shared among 1024 / kCols threads
// of each and added in a fixed order.
template <int kCols>
__global__ __launch_bounds__(1024) void rms_norm_dw_kernel(NormGradArgs a) {
  constexpr int kSlices = 1024 / kCols;
  __shared__ float red[kSlices][kCols];
  const int x = threadIdx.x % kCols, slice = threadIdx.x / kCols;
  const int c = blockIdx.x * kCols + x;
  float sum = 0.f;
  if (c < a.n) {
#pragma unroll 16
    for (int g = slice; g < a.groups; g += kSlices) sum += a.part[(int64_t)g * a.ldpart + c];
  }
  red[slice][x] = sum;
  __syncthreads();
  if (slice == 0 && c < a.n) {
    float total = 0.f;
#pragma unroll
    for (int w = 0; w < kSlices; ++w) total += red[w][x];
    a.dw[c] = total;
  }
}

// f(threads, elements per thread / 8) at the smallest workgroup that holds a
// row of n elements; n <= 32768.
template <class F>
hipError_t by_width(int n, F f) {
  if (n <= 512) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  else if (n <= 1024) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  else if (n <= 2048) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 1>{});
  else if (n <= 4096) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  else if (n <= 8192) f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  else if (n <= 16384) f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
  else if (n <= 32768) f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 4>{});
  else return hipErrorInvalidValue;
  return hipGetLastError();
}

template <typename T, bool kE8m0>
hipError_t quantize(const QuantArgs& a, bool tiles, hipStream_t s) {
  const int64_t blocks = cdiv((int64_t)a.m * cdiv(a.n, kFp8Block), 16);
  // (more workgroups of 256 would be 2^32 threads, too many for one launch)
  if (!tiles && a.qt == nullptr && blocks < int64_t{1} << 24) {
    hipLaunchKernelGGL((quant_rows_kernel<T, kE8m0>), dim3(static_cast<uint32_t>(blocks)), dim3(256),
                       0, s, a);
    return hipGetLastError();
  }
  const dim3 grid(static_cast<uint32_t>(cdiv(a.n, 128) * cdiv(a.m, 128)));
  if (tiles) hipLaunchKernelGGL((quant_tile_kernel<T, kE8m0, true>), grid, dim3(256), 0, s, a);
  else hipLaunchKernelGGL((quant_tile_kernel<T, kE8m0, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

// Workgroups of the forward norm: rows are shared among as many as the chip
// holds at eight waves per SIMD.
inline int64_t norm_groups(int64_t m, int threads) {
  const int64_t most = 256 * 4 * 8 * 64 / threads;
  return m < most ? m : most;
}

template <typename T, bool kE8m0>
hipError_t norm(const NormArgs& a, hipStream_t s) {
  return by_width(a.n, [&](auto th, auto c) {
    hipLaunchKernelGGL((rms_norm_fp8_kernel<T, kE8m0, decltype(th)::value, decltype(c)::value>),
                       dim3(static_cast<uint32_t>(norm_groups(a.m, decltype(th)::value))),
                       dim3(decltype(th)::value), 0, s, a);
  });
}

template <typename T>
hipError_t norm_grad(const NormGradArgs& a, hipStream_t s) {
  hipError_t e = by_width(a.n, [&](auto th, auto c) {
    hipLaunchKernelGGL((rms_norm_grad_kernel<T, decltype(th)::value, decltype(c)::value>),
                       dim3(a.groups), dim3(decltype(th)::value), 0, s, a);
  });
  if (e != hipSuccess) return e;
  // 16 columns per workgroup (64-byte pieces of a part) where 64 would leave
  // most CUs idle
  if (a.n <= 4096) hipLaunchKernelGGL(rms_norm_dw_kernel<16>, dim3(static_cast<uint32_t>(cdiv(a.n, 16))), dim3(1024), 0, s, a);
  else hipLaunchKernelGGL(rms_norm_dw_kernel<64>, dim3(static_cast<uint32_t>(cdiv(a.n, 64))), dim3(1024), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_quantize(const QuantArgs& a, bool bf, bool e8m0, bool tiles, hipStream_t s) {
  if (bf) return e8m0 ? quantize<uint16_t, true>(a, tiles, s) : quantize<uint16_t, false>(a, tiles, s);
  return e8m0 ? quantize<float, true>(a, tiles, s) : quantize<float, false>(a, tiles, s);
}

hipError_t launch_rms_norm_fp8(const NormArgs& a, bool bf, bool e8m0, hipStream_t s) {
  if (bf) return e8m0 ? norm<uint16_t, true>(a, s) : norm<uint16_t, false>(a, s);
  return e8m0 ? norm<float, true>(a, s) : norm<float, false>(a, s);
}

hipError_t launch_rms_norm_backward(const NormGradArgs& a, bool bf, hipStream_t s) {
  return bf ? norm_grad<uint16_t>(a, s) : norm_grad<float>(a, s);
}

}  // namespace ortho
