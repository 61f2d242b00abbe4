// AdamW over many tensors and the gradients' norm: the launchers' argument blocks
// (internal to libortho.so).  gfx950 only.
#pragma once

#include <stddef.h>

#include "common.h"

namespace ortho {

// Work is dealt in units of up to 2048 elements, eight per thread of a workgroup.
// Tensor i of a launch has the units first[i] .. first[i + 1] - 1.  A table has at
// most one tensor per lane of a wave: lane l holds first[l], and a unit's tensor is
// the last of the lanes whose first unit is not beyond it (one comparison, one
// count).  What is not used of `first` is the type's largest value.
//
// A tensor's entry is read by scalar loads, which drop the two low bits of both
// parts of an address: entries hold no type of less than four bytes.  The assertions
// below add up their members, so that another member has to be looked at there.
constexpr int kUnit = 2048;
constexpr int kLanes = 64;

// What the step reads that is the same for all tensors.
struct AdamwScalars {
  float b1, c1, b2, c2;         // beta and 1 - beta
  float eps;
  float keep, size, root;       // 1 - lr wd, lr / (1 - b1^t), 1 / sqrt(1 - b2^t)
  double lr, wd;                // for what is read on the device in their place
  double log_b1, log_b2;
  int64_t step;
  uint32_t seed_lo, seed_hi;
  const float* lr_dev;
  const int64_t* step_dev;
  const float* factor;
};

enum { kBf16Weight = 1, kBf16Gradient = 2 };

// Tensors of consecutive elements with states in 32 bits.
struct FlatTensor {
  void* x;
  const void* g;
  float *m, *v;
  int64_t n;
  int32_t index;                 // of the tensor in the call
  int32_t kind;
};
static_assert(sizeof(FlatTensor) == 4 * 8 + 8 + 2 * 4 && alignof(FlatTensor) == 8 && offsetof(FlatTensor, n) == 4 * 8,
              "pointers at multiples of 8, nothing below four bytes, no gap");
struct AdamwFlat {
  static constexpr int kMost = 64;
  AdamwScalars h;
  FlatTensor t[kMost];           // 48 bytes each: the argument block stays below 4 KB
  int32_t first[kLanes];
  int32_t units;
};

// Tensors with rows of their own pitch, or with states in 8 bits.  A unit is
// 256 >> lanes rows of 8 << lanes columns: 1 << lanes threads (16 to 256) per row.
struct RowTensor {
  void* x;
  const void* g;
  void *m, *v;
  float *sm, *sv;                // null: states in 32 bits
  uint32_t ldx, ldg, ldm, ldv, ldsm, ldsv;
  int32_t rows, cols;
  int32_t across;                // units next to each other along the columns
  int32_t lanes;
  int32_t index, kind;
};
static_assert(sizeof(RowTensor) == 6 * 8 + 12 * 4 && alignof(RowTensor) == 8 && offsetof(RowTensor, ldx) == 6 * 8,
              "pointers at multiples of 8, nothing below four bytes, no gap");
struct AdamwRows {
  static constexpr int kMost = 38;   // 96 bytes each
  AdamwScalars h;
  RowTensor t[kMost];
  int32_t first[kLanes];
  int32_t units;
};

// Gradients: units of 256 >> lanes rows of 4 << lanes pieces of 16 bytes.
struct NormTensor {
  const void* g;
  int64_t ld, cols;
  int32_t rows, across, lanes, bf;
};
static_assert(sizeof(NormTensor) == 3 * 8 + 4 * 4 && alignof(NormTensor) == 8 && offsetof(NormTensor, rows) == 3 * 8,
              "pointers at multiples of 8, nothing below four bytes, no gap");
struct NormParts {
  static constexpr int kMost = 64;
  NormTensor t[kMost];
  int64_t first[kLanes];         // (gradients may overlap: many long ones pass 2^31 units)
  int64_t units;
  double* part;                  // one sum per workgroup
};

static_assert(offsetof(AdamwFlat, t) % 8 == 0 && offsetof(AdamwRows, t) % 8 == 0 && offsetof(NormParts, t) % 8 == 0 &&
                  offsetof(AdamwFlat, first) % 4 == 0 && offsetof(AdamwRows, first) % 4 == 0 &&
                  offsetof(NormParts, first) % 8 == 0,
              "the tables' places in a launch's arguments");

hipError_t launch_adamw_flat(const AdamwFlat& a, bool stochastic, hipStream_t s);
// kind: all tensors', if they have one and their states are codes, else -1.
hipError_t launch_adamw_rows(const AdamwRows& a, int kind, bool stochastic, hipStream_t s);
hipError_t launch_grad_norm_parts(const NormParts& a, int groups, hipStream_t s);
hipError_t launch_grad_norm_join(const double* part, int count, double max_norm, float* out, hipStream_t s);

}  // namespace ortho
