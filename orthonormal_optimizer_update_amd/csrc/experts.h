// Tokens by expert: the launchers' argument blocks (internal to libortho.so).
// gfx950 only.
#pragma once

#include "common.h"

namespace ortho {

struct ExpertSortArgs {
  const void* chosen;
  int wide;                      // int64, else int32
  int pairs, experts, align;
  int tiles, tile;               // pairs per workgroup, a multiple of 1024
  int32_t *slot, *source, *offsets, *counts;   // source may be null
  int rows;                      // of source
  int32_t* part;                 // tiles x experts counts (tiles > 1)
};
hipError_t launch_expert_sort(const ExpertSortArgs& a, hipStream_t s);

// Rows of a matrix of any type as bytes, and the rows of scales beside them.
struct ExpertRowsArgs {
  const int32_t *slot, *offsets, *counts;
  int tokens, choices, experts;
  int64_t rows;                  // of the sorted matrix
};

struct ExpertGatherArgs {
  ExpertRowsArgs r;
  const uint8_t* x;
  uint8_t* y;
  int64_t pitch_x, pitch_y, bytes;
  const uint8_t* s;              // null: no scales
  uint8_t* sy;
  int64_t pitch_s, pitch_sy;
  int blocks, scale_bytes;       // scales per row, and the bytes of one
  int scale_lanes;               // 1 << scale_lanes threads per row of scales
};
hipError_t launch_expert_gather(const ExpertGatherArgs& a, int lanes, int64_t across, int64_t units, hipStream_t s);

struct ExpertCombineArgs {
  ExpertRowsArgs r;
  const void* y;
  const void* w;                 // null: ones
  const void* add;
  void* out;
  int64_t ldy, ldw, ldadd, ldout;
  int n, w_bf, add_bf;
};
hipError_t launch_expert_combine(const ExpertCombineArgs& a, bool bf, int lanes, int64_t across, int64_t units,
                                 hipStream_t s);

struct ExpertCombineGradArgs {
  ExpertRowsArgs r;
  const void* dout;
  const void* w;
  const void* y;                 // null: no dw
  void* dy;
  float* dw;
  int64_t lddout, ldw, ldy, lddy, lddw;
  int n, w_bf;
};
hipError_t launch_expert_combine_grad(const ExpertCombineGradArgs& a, bool bf, hipStream_t s);

}  // namespace ortho
