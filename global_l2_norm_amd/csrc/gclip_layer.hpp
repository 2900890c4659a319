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
  int32_t streamed;     // see kStreamBytes
};

struct BwdArgs {
  Rows dy, dh, x, dres, dx;  // dh.at 0: none; the plain norm writes dres alone, a residual step without dropout too
  const float *mean, *rstd;
  uint64_t weight, dweight, dbias;
  float* partials;  // [parts][2][size]: sums of dy * n, then of dy
  uint32_t rows, size;
  int32_t wdt, gdt, accumulate;
  uint32_t parts;
  int32_t streamed;  // see kStreamBytes
};

// The norms' kernels hold a row of kRegistersMin to kRegistersMax columns in
// registers, `lanes` lanes with `units` units of 16 bytes each: the least of
// these shapes that holds the row.  Other rows go through the kernels of
// gclip_layer_any.hip.
constexpr uint32_t kRegistersMin = 8, kRegistersMax = 16384;
struct RowShape {
  uint32_t lanes, units;
};
template <int DT>
constexpr RowShape kFwdShapes[] = {{8, 1},  {16, 1}, {32, 1},  {64, 1},  {32, 3},  {64, 2}, {64, 3},
                                   {64, 4}, {256, 2}, {256, 3}, {256, 4}, {512, 3}, {512, 4}};
template <>
inline constexpr RowShape kFwdShapes<GCLIP_F32>[] = {{16, 1}, {32, 1},  {64, 1},  {64, 2},  {64, 3},  {64, 4}, {64, 6},
                                                     {64, 8}, {256, 4}, {256, 6}, {256, 8}, {512, 6}, {512, 8}};
// Few rows: more lanes each.
#ifndef GCLIP_FEW_ROWS
#define GCLIP_FEW_ROWS 512
#endif
constexpr uint32_t kFewRows = GCLIP_FEW_ROWS;
template <int DT>
constexpr RowShape kFewShapes[] = {{8, 1},   {16, 1},  {32, 1},   {64, 1},  {128, 1},
                                   {256, 1}, {512, 1}, {1024, 1}, {1024, 2}};
template <>
inline constexpr RowShape kFewShapes<GCLIP_F32>[] = {{16, 1},  {32, 1},  {64, 1},   {128, 1}, {256, 1},
                                                     {512, 1}, {1024, 1}, {1024, 2}, {1024, 4}};
#ifndef GCLIP_BWD_F32
#define GCLIP_BWD_F32 {64, 3}, {64, 4}, {128, 3}, {128, 4}
#endif
template <int DT>
constexpr RowShape kBwdShapes[] = {{8, 1},   {16, 1},  {32, 1},  {64, 1},  {64, 2},
                                   {128, 2}, {256, 2}, {512, 2}, {1024, 2}};
template <>
inline constexpr RowShape kBwdShapes<GCLIP_F32>[] = {{16, 1}, {32, 1}, {64, 1}, {64, 2}, GCLIP_BWD_F32,
                                                     {256, 4}, {512, 4}, {1024, 4}};
template <int N>
constexpr int row_shape_of(const RowShape (&shapes)[N], uint32_t unit, uint32_t size) {
  int i = 0;
  while (shapes[i].lanes * shapes[i].units * unit < size) ++i;
  return i;
}
// Units of shape i that lie in every row it is used for.
template <int N>
constexpr int sure_units(const RowShape (&shapes)[N], int i) {
  return i == 0 ? 0 : (int)(shapes[i - 1].lanes * shapes[i - 1].units / shapes[i].lanes);
}
inline bool in_registers(uint32_t size) { return size >= kRegistersMin && size <= kRegistersMax; }

// Threads of a workgroup of the backward kernel: all that a compute unit's
// registers hold, so that each unit leaves one partial sum of the weights'
// gradients, of kBwdParts at most.
constexpr uint32_t bwd_threads(uint32_t lanes, uint32_t columns) { return columns <= 8 || lanes > 512 ? 1024 : 512; }
constexpr uint32_t kBwdParts = 256;
template <int DT>
inline uint32_t bwd_parts(uint32_t rows, uint32_t size) {
  const uint32_t unit = DT == GCLIP_F32 ? 4 : 8;
  const RowShape s = kBwdShapes<DT>[row_shape_of(kBwdShapes<DT>, unit, size)];
  const uint32_t at_once = bwd_threads(s.lanes, s.units * unit) / s.lanes, need = (rows - 1) / at_once + 1;
  return need < kBwdParts ? need : kBwdParts;
}

// What a call moves decides how.  Up to kStreamBytes the matrices may lie in
// the 256 MB cache before memory, where the kernel before has left them:
// ordinary loads find them there, and nontemporal stores leave them there.
// Above, nontemporal loads and ordinary stores are faster.
#ifndef GCLIP_STREAM_MB
#define GCLIP_STREAM_MB 144
#endif
constexpr uint64_t kStreamBytes = (uint64_t)GCLIP_STREAM_MB << 20;

// The most partial sums of the weights' gradients for a matrix of this shape
// in any format.
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
