// Tokens to rows by expert, and back.
#include <type_traits>

#include "experts.h"
#include "fp8.h"

namespace ortho {

namespace {

inline int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// ---- the sort ----
//
// A stable counting sort.  Counts of each tile's experts meet in memory; then each
// workgroup adds what it needs of them itself (64 tiles of 128 experts are 32 KB
// from L2, less than another launch takes), and its 16 waves place their pairs, 64 at
// a time, in order.  One tile needs no other's counts and no first launch.  Bound by
// latency: 16384 x 8 pairs, 128 experts take 2.0 and 6.6 us, 33 x 8 pairs 4.2.  (What the
// workgroups add up grows with the square of the tiles: 131072 x 8 pairs of 256 experts
// take 32 us in all, 262144 x 8 of 512 160.)
constexpr int kSortThreads = 1024, kSortWaves = kSortThreads / 64, kExperts = 1024;

__device__ __forceinline__ int expert_of(const ExpertSortArgs& a, int pair) {
  if (pair >= a.pairs) return -1;
  const int64_t e = a.wide ? static_cast<const int64_t*>(a.chosen)[pair]
                           : static_cast<int64_t>(static_cast<const int32_t*>(a.chosen)[pair]);
  return e >= 0 && e < a.experts ? static_cast<int>(e) : -1;
}

__global__ __launch_bounds__(kSortThreads) void expert_count_kernel(ExpertSortArgs a) {
  __shared__ int32_t count[kExperts];
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) count[e] = 0;
  __syncthreads();
  const int first = blockIdx.x * a.tile;
  for (int i = threadIdx.x; i < a.tile; i += kSortThreads) {
    const int e = expert_of(a, first + i);
    if (e >= 0) atomicAdd(&count[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSortThreads) a.part[(int64_t)blockIdx.x * a.experts + e] = count[e];
}

// Lanes of the wave with this lane's expert, by one ballot per bit of its number
// (bit `bits` is set for pairs without one).
__device__ __forceinline__ uint64_t same_lanes(int expert, int bits) {
  uint64_t same = ~uint64_t{0};
  for (int b = 0; b <= bits; ++b) {
    const bool set = expert >> b & 1;
    const uint64_t with = __ballot(set);
    same &= set ? with : ~with;
  }
  return same;
}

// kBatch x 64 pairs of a wave's `each`, from pair `first` + i0 on: their experts, all
// loads under way together.
constexpr int kBatch = 2;
__device__ __forceinline__ void load_experts(const ExpertSortArgs& a, int first, int i0, int each, int (&e)[kBatch]) {
#pragma unroll
  for (int q = 0; q < kBatch; ++q) {
    const int i = i0 + q * 64 + (threadIdx.x & 63);
    e[q] = i < each ? expert_of(a, first + i) : -1;
  }
}

__global__ __launch_bounds__(kSortThreads) void expert_place_kernel(ExpertSortArgs a) {
  __shared__ int32_t place[kSortWaves][kExperts];   // counts, then next rows, of each wave
  __shared__ int32_t begin[kExperts + 1], total[kExperts];
  __shared__ int32_t sums[kSortWaves];
  __shared__ int32_t parts[2][kSortThreads];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int each = a.tile / kSortWaves, first = blockIdx.x * a.tile + wave * each;
  for (int e = lane; e < a.experts; e += 64) place[wave][e] = 0;
  // All tiles' counts of expert t mod 2^k, and those of the tiles before this one: the
  // tiles are dealt to the 2^(10 - k) threads that have the same expert.
  int log = 6;
  while (1 << log < a.experts) ++log;
  if (a.tiles > 1) {
    const int e = t & ((1 << log) - 1), group = t >> log, groups = kSortThreads >> log;
    int all = 0, before = 0;
    if (e < a.experts) {
#pragma unroll 8
      for (int i = group; i < a.tiles; i += groups) {
        const int c = a.part[(int64_t)i * a.experts + e];
        all += c;
        before += i < static_cast<int>(blockIdx.x) ? c : 0;
      }
    }
    parts[0][t] = all;
    parts[1][t] = before;
  }
  __syncthreads();
  int es[kBatch];
  for (int i0 = 0; i0 < each; i0 += kBatch * 64) {
    load_experts(a, first, i0, each, es);
#pragma unroll
    for (int q = 0; q < kBatch; ++q)
      if (es[q] >= 0) atomicAdd(&place[wave][es[q]], 1);
  }
  __syncthreads();
  int all = 0, before = 0;
  if (t < a.experts) {
    if (a.tiles == 1) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) all += place[w][t];
    } else {
      for (int i = t; i < kSortThreads; i += 1 << log) {
        all += parts[0][i];
        before += parts[1][i];
      }
    }
  }
  // Where expert t begins: the padded counts before it.
  const int padded = (all + a.align - 1) / a.align * a.align;
  int up = padded;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int v = __shfl_up(up, o, 64);
    up += lane >= o ? v : 0;
  }
  if (lane == 63) sums[wave] = up;
  __syncthreads();
  int start = up - padded;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) start += w < wave ? sums[w] : 0;
  if (t < a.experts) {
    begin[t] = start;
    total[t] = all;
    if (t == a.experts - 1) begin[a.experts] = start + padded;
    int at = start + before;
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int c = place[w][t];
      place[w][t] = at;
      at += c;
    }
    if (blockIdx.x == 0) {
      a.offsets[t] = start;
      a.counts[t] = all;
      if (t == a.experts - 1) a.offsets[a.experts] = start + padded;
    }
  }
  __syncthreads();
  int bits = 1;
  while (1 << bits < a.experts) ++bits;
  for (int i0 = 0; i0 < each && first + i0 < a.pairs; i0 += kBatch * 64) {
    if (each > kBatch * 64) load_experts(a, first, i0, each, es);   // (else they are here)
#pragma unroll
    for (int q = 0; q < kBatch; ++q) {
      const int e = es[q], i = i0 + q * 64 + lane, pair = first + i;
      const uint64_t same = same_lanes(e < 0 ? 1 << bits : e, bits);
      const int rank = __popcll(same & ((uint64_t{1} << lane) - 1));
      const int base = e >= 0 ? place[wave][e] : 0;
      // (the wave's own row of LDS, whose accesses keep their order)
      __builtin_amdgcn_wave_barrier();
      if (e >= 0 && rank == 0) place[wave][e] = base + __popcll(same);
      __builtin_amdgcn_wave_barrier();
      if (i < each && pair < a.pairs) {
        a.slot[pair] = e >= 0 ? base + rank : -1;
        if (a.source && e >= 0) a.source[base + rank] = pair;
      }
    }
  }
  if (a.source == nullptr) return;
  // Rows without a pair: each expert's padding, and what lies behind the last.
  for (int e = blockIdx.x * kSortWaves + wave; e < a.experts; e += gridDim.x * kSortWaves)
    for (int r = begin[e] + total[e] + lane; r < begin[e + 1]; r += 64) a.source[r] = -1;
  for (int64_t r = (int64_t)begin[a.experts] + blockIdx.x * kSortThreads + t; r < a.rows;
       r += gridDim.x * kSortThreads)
    a.source[r] = -1;
}

// ---- rows as bytes ----

// 16 bytes of a row of at least 16, from byte 16 p on; a piece that the row's end
// cuts starts earlier, so that it lies inside (its bytes are the same either way).
__device__ __forceinline__ int64_t piece_at(int64_t p, int64_t bytes) {
  return p * 16 + 16 <= bytes ? p * 16 : bytes - 16;
}

template <bool kOnce>
__device__ __forceinline__ void copy_piece(uint8_t* dst, const uint4& u, int64_t p, int64_t bytes) {
  if (bytes >= 16) {
    store_any<kOnce>(dst + piece_at(p, bytes), u);
    return;
  }
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (j < bytes) dst[j] = static_cast<uint8_t>(w[j >> 2] >> 8 * (j & 3));
}

__device__ __forceinline__ uint4 load_piece(const uint8_t* src, int64_t p, int64_t bytes) {
  uint4 u;
  if (bytes >= 16) {
    __builtin_memcpy(&u, src + piece_at(p, bytes), 16);
    return u;
  }
  uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < 16; ++j)
    if (j < bytes) w[j >> 2] |= static_cast<uint32_t>(src[j]) << 8 * (j & 3);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Zeros in the rows of padding of expert e's part `part` of `parts`, `pieces` of
// `bytes` each.
template <bool kOnce>
__device__ __forceinline__ void clear_padding(const ExpertRowsArgs& r, int e, int part, int parts, uint8_t* y,
                                              int64_t pitch, int64_t bytes, uint8_t* s, int64_t pitch_s, int blocks,
                                              int scale_bytes) {
  const int64_t from = max(0, r.offsets[e]) + static_cast<int64_t>(max(0, r.counts[e]));
  const int64_t to = min(static_cast<int64_t>(r.offsets[e + 1]), r.rows);
  const int64_t pieces = (bytes + 15) >> 4;
  for (int64_t row = from + part; row < to; row += parts) {
    for (int64_t p = threadIdx.x; p < pieces; p += 256)
      copy_piece<kOnce>(y + row * pitch, make_uint4(0, 0, 0, 0), p, bytes);
    if (s)
      for (int i = threadIdx.x; i < blocks; i += 256) {
        if (scale_bytes == 4) reinterpret_cast<float*>(s + row * pitch_s)[i] = 1.f;
        else s[row * pitch_s + i] = 127;
      }
  }
}

constexpr int kPadParts = 4;   // workgroups per expert's padding

// The row of a pair, or -1.
__device__ __forceinline__ int64_t row_of(const ExpertRowsArgs& r, int64_t pair) {
  const int s = r.slot[pair];
  return s >= 0 && s < r.rows ? s : -1;
}

// A token's row is read once and written `choices` times.  A workgroup's unit is
// 256 >> lanes tokens by 1 << lanes pieces of 16 bytes.  Bound by the writes: 8192
// tokens x 2048 codes to 8 of 64 experts (rows padded to 128) take 32 us, 4.9 TB/s, with
// rows written past the caches (36 through them; reading past them too 35).  The scales,
// scattered in pieces of 64 bytes, are 4 us of it (6 written beside each 128 codes by the
// thread that has them).  A wave per token with scalar rows took a quarter more, a thread
// row per (token, choice), which reads the token anew, twice as long.
template <bool kOnce>
__global__ __launch_bounds__(256) void expert_gather_kernel(ExpertGatherArgs a, int lanes, int across, int64_t units) {
  if (blockIdx.x >= gridDim.x - a.r.experts * kPadParts) {
    const int at = blockIdx.x - (gridDim.x - a.r.experts * kPadParts);
    clear_padding<kOnce>(a.r, at / kPadParts, at % kPadParts, kPadParts, a.y, a.pitch_y, a.bytes, a.sy, a.pitch_sy, a.blocks,
                  a.scale_bytes);
    return;
  }
  const int64_t pieces = (a.bytes + 15) >> 4;
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x - a.r.experts * kPadParts) {
    const int64_t down = unit / across;
    const int col = static_cast<int>(unit - down * across);
    const int64_t token = (down << (8 - lanes)) + (threadIdx.x >> lanes);
    const int64_t p = ((int64_t)col << lanes) + (threadIdx.x & ((1 << lanes) - 1));
    if (token >= a.r.tokens) continue;
    if (p >= pieces) continue;
    const int64_t pair = token * a.r.choices;
    const uint4 u = load_piece(a.x + token * a.pitch_x, p, a.bytes);
#pragma unroll 4
    for (int j = 0; j < a.r.choices; ++j) {
      const int64_t row = row_of(a.r, pair + j);
      if (row >= 0) copy_piece<kOnce>(a.y + row * a.pitch_y, u, p, a.bytes);
    }
  }
  if (a.s == nullptr) return;
  const int wide = a.scale_lanes;
  const int64_t step = (int64_t)(gridDim.x - a.r.experts * kPadParts) << (8 - wide);
  for (int64_t token = ((int64_t)blockIdx.x << (8 - wide)) + (threadIdx.x >> wide); token < a.r.tokens; token += step) {
    const int64_t pair = token * a.r.choices;
    const uint8_t* const src = a.s + token * a.pitch_s;
    for (int b = threadIdx.x & ((1 << wide) - 1); b < a.blocks; b += 1 << wide) {
      const uint32_t scale = a.scale_bytes == 4 ? reinterpret_cast<const uint32_t*>(src)[b] : src[b];
#pragma unroll 4
      for (int j = 0; j < a.r.choices; ++j) {
        const int64_t row = row_of(a.r, pair + j);
        if (row < 0) continue;
        uint8_t* const to = a.sy + row * a.pitch_sy;
        if (a.scale_bytes == 4) reinterpret_cast<uint32_t*>(to)[b] = scale;
        else to[b] = static_cast<uint8_t>(scale);
      }
    }
  }
}

// ---- back to tokens ----

__device__ __forceinline__ float weight_of(const void* w, int w_bf, int64_t at) {
  if (w == nullptr) return 1.f;
  return w_bf ? bf16_bits_to_f32(static_cast<const uint16_t*>(w)[at]) : static_cast<const float*>(w)[at];
}

// kAtOnce choices' loads are under way together.
template <typename T, int kAtOnce>
__global__ __launch_bounds__(256) void expert_combine_narrow_kernel(ExpertCombineArgs a, int lanes, int across,
                                                             int64_t units) {
  for (int64_t unit = blockIdx.x; unit < units; unit += gridDim.x) {
    const int64_t down = unit / across;
    const int col = static_cast<int>(unit - down * across);
    const int64_t token = (down << (8 - lanes)) + (threadIdx.x >> lanes);
    const int c = ((col << lanes) + (threadIdx.x & ((1 << lanes) - 1))) * 8;
    if (token >= a.r.tokens || c >= a.n) continue;
    float sum[8] = {};
    for (int j0 = 0; j0 < a.r.choices; j0 += kAtOnce) {
      Raw8<T> y[kAtOnce];
      float w[kAtOnce];
      bool has[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int at = min(j0 + j, a.r.choices - 1);
        const int64_t row = row_of(a.r, token * a.r.choices + at);
        has[j] = row >= 0 && j0 + j < a.r.choices;
        w[j] = weight_of(a.w, a.w_bf, token * a.ldw + at);
        // (row 0 for pairs without one: no load depends on a branch)
        y[j] = load_raw8(static_cast<const T*>(a.y) + max(row, (int64_t)0) * a.ldy, c, a.n);
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        float v[8];
        unpack8(y[j], v);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[e] = has[j] ? fmaf(w[j], v[e], sum[e]) : sum[e];
      }
    }
    if (a.add) {
      float v[8];
      if (a.add_bf) load8(static_cast<const uint16_t*>(a.add) + token * a.ldadd, c, a.n, v);
      else load8(static_cast<const float*>(a.add) + token * a.ldadd, c, a.n, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += v[e];
    }
    store8(static_cast<T*>(a.out) + token * a.ldout, c, a.n, sum);
  }
}

// ---- a wave for 512 elements of a token ----
//
// Lane j holds the row and the weight of choice j; readlane makes them scalars, so
// that a row's address is scalar too.  All lanes go through all of it: past a row's
// end they read zeros and write nothing.
struct Choices {
  int row;       // -1: none
  float weight;
};
__device__ __forceinline__ Choices lane_choices(const ExpertRowsArgs& r, int64_t token, const void* w, int w_bf, int64_t ldw) {
  Choices c = {-1, 0.f};
  const int lane = threadIdx.x & 63;
  if (lane < r.choices) {
    const int s = r.slot[token * r.choices + lane];
    c.row = s >= 0 && s < r.rows ? s : -1;
    c.weight = weight_of(w, w_bf, token * ldw + lane);
  }
  return c;
}
__device__ __forceinline__ int scalar_row(const Choices& c, int j) { return __builtin_amdgcn_readlane(c.row, j); }
__device__ __forceinline__ float scalar_weight(const Choices& c, int j) {
  return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(c.weight), j));
}

constexpr int kWaveColumns = 512;

// This lane's eight elements of the 512 of a row of n from column c on; kWhole: all
// inside.  Where rows are fp32 (kHalves) a lane of a whole 512 has four elements in each
// half, so that every access of a wave covers whole lines.
template <bool kWhole, bool kHalves, bool kOnce, typename T>
__device__ __forceinline__ Raw8<T> piece8(const T* row, int c, int n) {
  const int lane = threadIdx.x & 63;
  Raw8<T> r;
  if constexpr (!kWhole) {
    r = load_raw8(row, c + lane * 8, n);
  } else if constexpr (!kHalves) {
    r = load_whole8<kOnce>(row + c + lane * 8);
  } else if constexpr (sizeof(T) == 4) {
    r.a = load_any<uint4, kOnce>(row + c + lane * 4);
    r.b = load_any<uint4, kOnce>(row + c + kWaveColumns / 2 + lane * 4);
  } else {
    const uint2 lo = load_any<uint2, kOnce>(row + c + lane * 4);
    const uint2 hi = load_any<uint2, kOnce>(row + c + kWaveColumns / 2 + lane * 4);
    r.a = make_uint4(lo.x, lo.y, hi.x, hi.y);
  }
  return r;
}
template <bool kWhole, bool kHalves, bool kOnce, typename T>
__device__ __forceinline__ void store_piece8(T* row, int c, int n, const float (&v)[8]) {
  const int lane = threadIdx.x & 63;
  if constexpr (!kWhole) {
    store8(row, c + lane * 8, n, v);
  } else if constexpr (!kHalves) {
    store_whole8<kOnce>(row + c + lane * 8, v);
  } else {
    static_assert(sizeof(T) == 4, "");
    store_any<kOnce>(row + c + lane * 4, floatx4{v[0], v[1], v[2], v[3]});
    store_any<kOnce>(row + c + kWaveColumns / 2 + lane * 4, floatx4{v[4], v[5], v[6], v[7]});
  }
}

template <typename T, int kAtOnce, bool kWhole, bool kOnce>
__device__ __forceinline__ void combine_chunk(const ExpertCombineArgs& a, int64_t token, const Choices& ch, int c) {
  constexpr bool kHalves = sizeof(T) == 4;
  float sum[8] = {};
  for (int j0 = 0; j0 < a.r.choices; j0 += kAtOnce) {
    Raw8<T> y[kAtOnce];
    int row[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      row[j] = j0 + j < a.r.choices ? scalar_row(ch, j0 + j) : -1;
      y[j] = piece8<kWhole, kHalves, kOnce>(static_cast<const T*>(a.y) + max(row[j], 0) * a.ldy, c, a.n);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (row[j] < 0) continue;
      const float w = scalar_weight(ch, j0 + j);
      float v[8];
      unpack8(y[j], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] = fmaf(w, v[e], sum[e]);
    }
  }
  if (a.add) {
    float v[8];
    if (a.add_bf) unpack8(piece8<kWhole, kHalves, kOnce>(static_cast<const uint16_t*>(a.add) + token * a.ldadd, c, a.n), v);
    else unpack8(piece8<kWhole, kHalves, kOnce>(static_cast<const float*>(a.add) + token * a.ldadd, c, a.n), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] += v[e];
  }
  store_piece8<kWhole, kHalves, kOnce>(static_cast<T*>(a.out) + token * a.ldout, c, a.n, sum);
}

// Bound by HBM: 8192 tokens x 2048 bf16 from 8 experts each 50 us (6.0 TB/s), 59 through
// the caches, 67 with the rows' addresses in vector registers.
template <typename T, int kAtOnce, bool kOnce>
__global__ __launch_bounds__(256) void expert_combine_kernel(ExpertCombineArgs a, int chunks, int64_t tasks) {
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  for (int64_t task = (int64_t)blockIdx.x * 4 + wave; task < tasks; task += 4 * (int64_t)gridDim.x) {
    const int64_t token = task / chunks;
    const int c = static_cast<int>(task - token * chunks) * kWaveColumns;
    const Choices ch = lane_choices(a.r, token, a.w, a.w_bf, a.ldw);
    if (c + kWaveColumns <= a.n) combine_chunk<T, kAtOnce, true, kOnce>(a, token, ch, c);
    else combine_chunk<T, kAtOnce, false, kOnce>(a, token, ch, c);
  }
}

template <int kRotate>
__device__ __forceinline__ float turned(float v) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(v), 0x120 + kRotate, 0xf, 0xf, false));
}
__device__ __forceinline__ float sum_of_wave(float v) {
  v += turned<8>(v);
  v += turned<4>(v);
  v += turned<2>(v);
  v += turned<1>(v);
  v += __shfl_xor(v, 16, 64);
  return v + __shfl_xor(v, 32, 64);
}

template <typename T, int kAtOnce, bool kWhole, bool kOnce>
__device__ __forceinline__ void grad_chunk(const ExpertCombineGradArgs& a, int64_t token, const int (&row)[kAtOnce],
                                           const float (&w)[kAtOnce], float (&dot)[kAtOnce], int c) {
  constexpr bool kHalves = sizeof(T) == 4;
  const Raw8<T> rd = piece8<kWhole, kHalves, kOnce>(static_cast<const T*>(a.dout) + token * a.lddout, c, a.n);
  float d[8];
  if (a.y) {
    Raw8<T> y[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) y[j] = piece8<kWhole, kHalves, kOnce>(static_cast<const T*>(a.y) + max(row[j], 0) * a.ldy, c, a.n);
    unpack8(rd, d);
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      float v[8];
      unpack8(y[j], v);
#pragma unroll
      for (int e = 0; e < 8; ++e) dot[j] = fmaf(d[e], v[e], dot[j]);
    }
  } else {
    unpack8(rd, d);
  }
#pragma unroll
  for (int j = 0; j < kAtOnce; ++j) {
    if (row[j] < 0) continue;
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = w[j] * d[e];
    store_piece8<kWhole, kHalves, kOnce>(static_cast<T*>(a.dy) + row[j] * a.lddy, c, a.n, v);
  }
}

// kWaves waves per token, kAtOnce choices at a time: their rows of Y are read, the
// products with dOut summed, their rows of dY written.  Bound by HBM: 8192 tokens x
// 2048 bf16, 8 choices 107 to 113 us (5.2 TB/s), 114 to 119 through the caches; fp32 228
// (5.0).  Columns that the four waves' chunks do not share evenly, or rows that begin
// inside a line, take longer: bf16 x 1100 131 us (2.3 TB/s), x 2001 170, x 2100 186.
template <typename T, int kAtOnce, int kWaves, bool kOnce>
__global__ __launch_bounds__(256) void expert_combine_grad_kernel(ExpertCombineGradArgs a, int64_t groups) {
  __shared__ float red[2][4][64];
  if (blockIdx.x >= gridDim.x - a.r.experts * kPadParts) {
    const int at = blockIdx.x - (gridDim.x - a.r.experts * kPadParts);
    clear_padding<kOnce>(a.r, at / kPadParts, at % kPadParts, kPadParts, static_cast<uint8_t*>(a.dy), a.lddy * sizeof(T),
                  (int64_t)a.n * sizeof(T), nullptr, 0, 0, 0);
    return;
  }
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int turn = 0;
  for (int64_t group = blockIdx.x; group < groups; group += gridDim.x - a.r.experts * kPadParts) {
    const int64_t token = kWaves == 1 ? group * 4 + wave : group;
    if (token >= a.r.tokens) continue;
    const Choices ch = lane_choices(a.r, token, a.w, a.w_bf, a.ldw);
    float mine = 0.f;   // lane j: choice j's sum
    for (int j0 = 0; j0 < a.r.choices; j0 += kAtOnce) {
      int row[kAtOnce];
      float w[kAtOnce], dot[kAtOnce];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        row[j] = j0 + j < a.r.choices ? scalar_row(ch, j0 + j) : -1;
        w[j] = scalar_weight(ch, min(j0 + j, 63));
        dot[j] = 0.f;
      }
      for (int c = kWaves == 1 ? 0 : wave * kWaveColumns; c < a.n; c += kWaves * kWaveColumns) {
        if (c + kWaveColumns <= a.n) grad_chunk<T, kAtOnce, true, kOnce>(a, token, row, w, dot, c);
        else grad_chunk<T, kAtOnce, false, kOnce>(a, token, row, w, dot, c);
      }
      if (a.y == nullptr) continue;
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const float sum = sum_of_wave(dot[j]);
        mine = lane == j0 + j ? sum : mine;
      }
    }
    if (a.y == nullptr) continue;
    if constexpr (kWaves > 1) {
      red[turn][wave][lane] = mine;
      __syncthreads();
      mine = red[turn][0][lane] + red[turn][1][lane] + red[turn][2][lane] + red[turn][3][lane];
      turn ^= 1;
      if (wave != 0) continue;
    }
    if (lane < a.r.choices) a.dw[token * a.lddw + lane] = ch.row >= 0 ? mine : 0.f;
  }
}

constexpr int64_t kMostGroups = 1 << 20;   // workgroups of a launch; more units are walked

// Whether the rows by expert that a call reads and writes, `row_bytes` for a pair, are
// more than the last-level cache of 256 MB would keep (bf16, 8 choices x 2048, past the
// caches and through them: combine of 2048 tokens, 67 MB, 14.6 and 13.3 us, of 4096 28.7
// and 33.2, of 8192 55.5 and 63.0; its gradient, of 1024, 67 MB, 15.0 and 13.2 us, of 2048
// 29.7 and 34.8; codes gathered for 4096, 67 MB, 19.6 and 19.7, for 8192 32.4 and 36.7).
// Each was timed alone, without the call that reads what it writes.
bool passes_once(const ExpertRowsArgs& r, int64_t row_bytes) {
  return static_cast<int64_t>(r.tokens) * r.choices * row_bytes >= int64_t{1} << 27;
}

}  // namespace

hipError_t launch_expert_sort(const ExpertSortArgs& a, hipStream_t s) {
  if (a.tiles > 1) {
    hipLaunchKernelGGL(expert_count_kernel, dim3(a.tiles), dim3(kSortThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(expert_place_kernel, dim3(a.tiles), dim3(kSortThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_expert_gather(const ExpertGatherArgs& a, int lanes, int64_t across, int64_t units, hipStream_t s) {
  const int64_t groups = units < kMostGroups ? units : kMostGroups;
  const dim3 grid(static_cast<uint32_t>(groups + a.r.experts * kPadParts));
  const auto kernel = passes_once(a.r, a.bytes) ? expert_gather_kernel<true> : expert_gather_kernel<false>;
  hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a, lanes, static_cast<int>(across), units);
  return hipGetLastError();
}

// f(choices at once): the least power of two that holds them, at most eight.
template <class F>
hipError_t by_choices(int choices, F f) {
  if (choices <= 1) f(std::integral_constant<int, 1>{});
  else if (choices <= 2) f(std::integral_constant<int, 2>{});
  else if (choices <= 4) f(std::integral_constant<int, 4>{});
  else f(std::integral_constant<int, 8>{});
  return hipGetLastError();
}

template <typename T>
static hipError_t combine(const ExpertCombineArgs& a, int lanes, int64_t across, int64_t units, hipStream_t s) {
  const dim3 grid(static_cast<uint32_t>(units < kMostGroups ? units : kMostGroups));
  return by_choices(a.r.choices, [&](auto k) {
    hipLaunchKernelGGL((expert_combine_narrow_kernel<T, decltype(k)::value>), grid, dim3(256), 0, s, a, lanes,
                       static_cast<int>(across), units);
  });
}

template <typename T>
static hipError_t combine_wide(const ExpertCombineArgs& a, hipStream_t s) {
  const int64_t chunks = cdiv(a.n, kWaveColumns), tasks = chunks * a.r.tokens, groups = cdiv(tasks, 4);
  const dim3 grid(static_cast<uint32_t>(groups < kMostGroups ? groups : kMostGroups));
  const bool once = passes_once(a.r, static_cast<int64_t>(a.n) * sizeof(T));
  return by_choices(a.r.choices, [&](auto k) {
    constexpr int kAtOnce = decltype(k)::value;
    const auto kernel = once ? expert_combine_kernel<T, kAtOnce, true> : expert_combine_kernel<T, kAtOnce, false>;
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, a, static_cast<int>(chunks), tasks);
  });
}

template <typename T, int kWaves, bool kOnce>
static hipError_t combine_grad(const ExpertCombineGradArgs& a, hipStream_t s) {
  const int64_t units = cdiv(a.r.tokens, 4 / kWaves);
  const dim3 grid(static_cast<uint32_t>((units < kMostGroups ? units : kMostGroups) + a.r.experts * kPadParts));
  return by_choices(a.r.choices, [&](auto k) {
    hipLaunchKernelGGL((expert_combine_grad_kernel<T, decltype(k)::value, kWaves, kOnce>), grid, dim3(256), 0, s, a, units);
  });
}

hipError_t launch_expert_combine(const ExpertCombineArgs& a, bool bf, int lanes, int64_t across, int64_t units,
                                 hipStream_t s) {
  // rows that fill less than half of a wave share it (bf16, 8 choices: 16384 x 128
  // 8.6 us, 12.0 a wave each; x 256 14.6 both ways; x 384 29.2 and 24.3)
  if (a.n < kWaveColumns / 2)
    return bf ? combine<uint16_t>(a, lanes, across, units, s) : combine<float>(a, lanes, across, units, s);
  return bf ? combine_wide<uint16_t>(a, s) : combine_wide<float>(a, s);
}

hipError_t launch_expert_combine_grad(const ExpertCombineGradArgs& a, bool bf, hipStream_t s) {
  // one wave per token below 1024 columns (bf16, 8 choices: 16384 x 512 60 us, 78 with
  // four; x 768 89 and 94; x 1024 117 and 113; 8192 x 2048 131 and 115; 64 x 8192 26
  // and 11)
  if (a.n < 1024) return bf ? combine_grad<uint16_t, 1, false>(a, s) : combine_grad<float, 1, false>(a, s);
  if (passes_once(a.r, static_cast<int64_t>(a.n) * (bf ? 2 : 4) * (a.y ? 2 : 1)))
    return bf ? combine_grad<uint16_t, 4, true>(a, s) : combine_grad<float, 4, true>(a, s);
  return bf ? combine_grad<uint16_t, 4, false>(a, s) : combine_grad<float, 4, false>(a, s);
}

}  // namespace ortho
