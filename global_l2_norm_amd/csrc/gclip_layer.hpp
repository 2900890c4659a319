// gclip_layer.hpp -- what the layer calls' host side hands to their kernels
// (include/gclip_layer.h; internal to libgclip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gclip_layer.h"

namespace gclip {

struct DropArgs {
  uint32_t k0, k1, step, site;
  const uint32_t* d_step;
  uint32_t threshold;  // t: halves below it are dropped; 0: nothing is
  float scale;
};

// A matrix: its address and the distance of its rows in bytes.
struct Rows {
  uint64_t at;
  uint64_t ld;
};

struct FwdArgs {
  Rows x, residual, h, y;
  uint64_t weight, bias;
  float *mean, *rstd;
  uint32_t rows, size;
  int32_t wdt;
  float eps, rstd_max;  // rstd_max: 1 / sqrt(eps)
};

struct BwdArgs {
  Rows dy, dh, x, dres, dx;  // dh.at 0: none; the plain norm writes dres alone, a residual step without dropout too
  const float *mean, *rstd;
  uint64_t weight, dweight, dbias;
  float* partials;  // [parts][2][size]: sums of dy * n, then of dy
  uint32_t rows, size;
  int32_t wdt, gdt, accumulate;
  uint32_t parts;
};

// The norms' kernels hold a row of kRegistersMin to kRegistersMax columns in
// registers, `lanes` lanes with `groups` groups of eight columns each: the
// least of these shapes that holds the row.  Other rows go through the
// kernels of gclip_layer_any.hip.
constexpr uint32_t kRegistersMin = 8, kRegistersMax = 16384;
struct RowShape {
  uint32_t lanes, groups;
};
#ifndef GCLIP_FWD_SHAPES
#define GCLIP_FWD_SHAPES {8, 1}, {16, 1}, {32, 1}, {64, 1}, {32, 3}, {64, 2}, {64, 3}, {64, 4}, {256, 2}, {256, 3}, {256, 4}, {512, 3}, {512, 4}
#endif
#ifndef GCLIP_BWD_SHAPES
#define GCLIP_BWD_SHAPES {8, 1}, {16, 1}, {32, 1}, {64, 1}, {32, 3}, {64, 2}, {64, 3}, {128, 2}, {256, 2}, {256, 3}, {512, 2}, {512, 3}, {512, 4}
#endif
constexpr RowShape kFwdShapes[] = {GCLIP_FWD_SHAPES};
constexpr RowShape kBwdShapes[] = {GCLIP_BWD_SHAPES};
template <int N>
constexpr int row_shape_of(const RowShape (&shapes)[N], uint32_t size) {
  int i = 0;
  while (shapes[i].lanes * shapes[i].groups * 8 < size) ++i;
  return i;
}
inline bool in_registers(uint32_t size) { return size >= kRegistersMin && size <= kRegistersMax; }

// Threads of a workgroup of the backward kernel, and the most workgroups,
// each of which leaves one partial sum of the weights' gradients.
constexpr uint32_t kBwdThreads = 512;
#ifndef GCLIP_BWD_WGS
#define GCLIP_BWD_WGS 1
#endif
constexpr uint32_t kBwdParts = 256 * GCLIP_BWD_WGS;

// Partial sums of the weights' gradients for a matrix of this shape.
uint32_t layer_parts(int64_t rows, int64_t size);

// residual: the residual step; drop: null for none.
hipError_t launch_layer_forward(const FwdArgs& a, int32_t dtype, bool residual, const DropArgs* drop, hipStream_t st);
hipError_t launch_layer_backward(const BwdArgs& a, int32_t dtype, bool residual, const DropArgs* drop, hipStream_t st);
hipError_t launch_dropout(const Rows& x, const Rows& y, uint32_t rows, uint32_t size, int32_t dtype,
                          const DropArgs& drop, hipStream_t st);

// Their parts for one storage format: rows in registers, and the join of the
// partial sums.
template <int DT>
hipError_t forward_rows(const FwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st);
template <int DT>
hipError_t backward_rows(const BwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st);
template <int DT>
hipError_t join_weight_grads(const BwdArgs& a, hipStream_t st);

}  // namespace gclip
