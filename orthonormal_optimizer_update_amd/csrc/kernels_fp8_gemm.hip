// Product of 8-bit matrices with a scale for each block of 128:
//   C[i, j] = sum over blocks b of K of sa[i, b] sb[j, b] (sum over k in b of
//             a[i, k] b[j, k])  (+ Add[i, j])
// A block's sum is scaled in fp32 and added to the fp32 accumulators.
//
// Which matrix instruction forms a block's sum goes by C's type.  The 8-bit one
// aligns each group of eight consecutive products to the largest of them and
// cuts what lies below 2^-13 of its power of two (measured: a product of 2^-13
// of the largest still counts, one of 2^-14 is lost, while other groups and the
// accumulator are added at full fp32 precision).  Relative to the sum that is
// about 1e-5 for normally distributed operands: far below the rounding of a
// bf16 C, but 20 times what fp32 sums reach.  An fp32 C therefore converts the
// codes to bf16 (exact) and multiplies with the bf16 instruction, whose sums
// keep fp32 precision.
#include "fp8.h"

namespace ortho {

namespace {

typedef int intx8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Eight codes as eight bf16 (exact; the NaN code gives NaN).
__device__ __forceinline__ bf16x8 codes_to_bf16(int lo, int hi) {
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

__device__ __forceinline__ int swz(int row, int chunk) { return chunk ^ ((row >> 1) & 7); }

// 16 codes from column k of row `row`; zero codes outside the matrix.  Rows
// may start at any byte.
__device__ __forceinline__ uint4 load_codes16(const uint8_t* p, int64_t ld, int row, int k, int rows,
                                              int K) {
  uint4 u = make_uint4(0, 0, 0, 0);
  if (row >= rows || k >= K) return u;
  const uint8_t* src = p + row * ld + k;
  if (k + 16 <= K) {
    __builtin_memcpy(&u, src, 16);
    return u;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (k + j < K) w[j >> 2] |= static_cast<uint32_t>(src[j]) << (8 * (j & 3));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 128 x 128 tile of C per workgroup, 64 x 64 per wave.  The rows of B are the
// matrix instruction's rows and the rows of A its columns, so a lane holds
// four consecutive columns of one row of C and one scale of A.
template <bool kE8m0, bool kBf>
__global__ __launch_bounds__(256) void fp8_gemm_kernel(Fp8GemmArgs p) {
  __shared__ __attribute__((aligned(16))) uint8_t ta[128 * 128], tb[128 * 128];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int tiles_n = (p.N + 127) / 128;
  const int m0 = (blockIdx.x / tiles_n) * 128, n0 = (blockIdx.x % tiles_n) * 128;
  const int wm = (wave >> 1) * 64, wn = (wave & 1) * 64;
  floatx4 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};
  const int nkb = (p.K + kFp8Block - 1) / kFp8Block;
  for (int kb = 0; kb < nkb; ++kb) {
    uint4 ra[4], rb[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = (t >> 3) + 32 * q, c = t & 7;
      ra[q] = load_codes16(p.a, p.lda, m0 + r, kb * 128 + c * 16, p.M, p.K);
      rb[q] = load_codes16(p.b, p.ldb, n0 + r, kb * 128 + c * 16, p.N, p.K);
    }
    float sa[4], sb[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int m = min(m0 + wm + i * 16 + (lane & 15), p.M - 1);
      sa[i] = load_scale<kE8m0>(p.sa.p, (m >> p.sa.shift) * p.sa.ld + kb);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int n = min(n0 + wn + i * 16 + (lane >> 4) * 4 + e, p.N - 1);
        sb[i][e] = load_scale<kE8m0>(p.sb.p, (n >> p.sb.shift) * p.sb.ld + kb);
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int r = (t >> 3) + 32 * q, c = t & 7;
      *reinterpret_cast<uint4*>(ta + (r * 8 + swz(r, c)) * 16) = ra[q];
      *reinterpret_cast<uint4*>(tb + (r * 8 + swz(r, c)) * 16) = rb[q];
    }
    __syncthreads();
    auto frag = [&](const uint8_t* tile, int row) {
      const int g = lane >> 4;
      const uint4 lo = *reinterpret_cast<const uint4*>(tile + (row * 8 + swz(row, g)) * 16);
      const uint4 hi = *reinterpret_cast<const uint4*>(tile + (row * 8 + swz(row, g + 4)) * 16);
      return intx8{(int)lo.x, (int)lo.y, (int)lo.z, (int)lo.w, (int)hi.x, (int)hi.y, (int)hi.z, (int)hi.w};
    };
    // 16 x 16 x 128 product, zero start; the k order within a block is the same
    // for both operands and otherwise free
    auto product = [](const intx8& b, const intx8& a) -> floatx4 {
      floatx4 s = {0.f, 0.f, 0.f, 0.f};
      if constexpr (kBf)
        return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, s, 0, 0, 0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < 4; ++q)
        s = __builtin_amdgcn_mfma_f32_16x16x32_bf16(codes_to_bf16(b[2 * q], b[2 * q + 1]),
                                                    codes_to_bf16(a[2 * q], a[2 * q + 1]), s, 0, 0, 0);
      return s;
    };
    intx8 fa[4], fb[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      fa[i] = frag(ta, wm + i * 16 + (lane & 15));
      fb[i] = frag(tb, wn + i * 16 + (lane & 15));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const floatx4 s = product(fb[j], fa[i]);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = fmaf(s[e], sa[i] * sb[j][e], acc[i][j][e]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int m = m0 + wm + i * 16 + (lane & 15);
    if (m >= p.M) continue;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = n0 + wn + j * 16 + (lane >> 4) * 4;
      floatx4 v = acc[i][j];
      if (p.add) {
        const float4 ad = p.add_bf ? load4<uint16_t>(static_cast<const uint16_t*>(p.add) + m * p.ldadd, n, p.N, p.cvec)
                                   : load4<float>(static_cast<const float*>(p.add) + m * p.ldadd, n, p.N, p.cvec);
        v[0] += ad.x; v[1] += ad.y; v[2] += ad.z; v[3] += ad.w;
      }
      if constexpr (kBf) {
        uint16_t* c = static_cast<uint16_t*>(p.c) + m * p.ldc;
        if (p.cvec && n + 4 <= p.N) {
          *reinterpret_cast<uint2*>(c + n) = pack_bf16x4(v);
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < p.N) c[n + e] = to_bf16_bits(v[e]);
        }
      } else {
        float* c = static_cast<float*>(p.c) + m * p.ldc;
        if (p.cvec && n + 4 <= p.N) {
          *reinterpret_cast<floatx4*>(c + n) = v;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (n + e < p.N) c[n + e] = v[e];
        }
      }
    }
  }
}

}  // namespace

hipError_t launch_fp8_matmul(const Fp8GemmArgs& a, bool c_bf, bool e8m0, hipStream_t s) {
  const int64_t tiles = (int64_t)((a.N + 127) / 128) * ((a.M + 127) / 128);
  const dim3 grid(static_cast<uint32_t>(tiles));
  if (e8m0) {
    if (c_bf) hipLaunchKernelGGL((fp8_gemm_kernel<true, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((fp8_gemm_kernel<true, false>), grid, dim3(256), 0, s, a);
  } else {
    if (c_bf) hipLaunchKernelGGL((fp8_gemm_kernel<false, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((fp8_gemm_kernel<false, false>), grid, dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace ortho
