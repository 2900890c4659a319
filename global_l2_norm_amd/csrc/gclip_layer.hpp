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
  float* sums;      // [rows][2], long rows: their means of dy * weight and of that times n
  uint32_t rows, size;
  int32_t wdt, gdt, accumulate;
  uint32_t parts;
  int32_t streamed;  // see kStreamBytes
};

// The norms' kernels hold a row in registers, `lanes` lanes with `units` units
// of 16 bytes each: the least of the shapes below that holds the row.  The
// backward kernel keeps the columns' sums there too, for rows of half the
// length.  Shorter and longer rows go through the kernels of
// gclip_layer_any.hip.  Idle lanes cost what working ones do: with powers of
// two alone from 64 columns on, 16.8M bfloat16 elements in rows of 8 took
// 66 us (15 now), of 257 24 us (16), and residual gradients of 1025 and 1200
// columns 59 and 47 us (44 and 38).
constexpr uint32_t kRegistersMin = 8, kFwdMax = 16384, kBwdMax = 8192;
struct RowShape {
  uint32_t lanes, units;
};
template <int DT>
constexpr RowShape kFwdShapes[] = {{1, 1},  {2, 1},  {4, 1},   {8, 1},   {16, 1},  {8, 3},   {32, 1},
                                   {16, 3}, {64, 1}, {32, 3},  {64, 2},  {64, 3},  {64, 4},  {128, 3},
                                   {256, 2}, {256, 3}, {256, 4}, {512, 3}, {512, 4}};
template <>
inline constexpr RowShape kFwdShapes<GCLIP_F32>[] = {
    {2, 1},  {4, 1},  {8, 1},  {16, 1}, {32, 1},  {16, 3},  {64, 1},  {32, 3},  {64, 2}, {64, 3},
    {64, 4}, {64, 6}, {64, 8}, {256, 3}, {256, 4}, {256, 6}, {256, 8}, {512, 6}, {512, 8}};
// Few rows: more lanes each, which shortens the way from a row's loads to its
// stores while compute units are idle anyway.  256 x 2048 in bfloat16 takes
// 3.4 us (3.8 with a wave a row), 512 rows 3.6 (4.0), but 1024 rows 4.4 (4.3)
// and 2048 rows 6.5 (5.8).
constexpr uint32_t kFewRows = 512;
template <int DT>
constexpr RowShape kFewShapes[] = {{8, 1},   {16, 1},  {32, 1},   {64, 1},  {128, 1},
                                   {256, 1}, {512, 1}, {1024, 1}, {1024, 2}};
template <>
inline constexpr RowShape kFewShapes<GCLIP_F32>[] = {{16, 1},  {32, 1},  {64, 1},   {128, 1}, {256, 1},
                                                     {512, 1}, {1024, 1}, {1024, 2}, {1024, 4}};
template <int DT>
constexpr RowShape kBwdShapes[] = {{1, 1},  {2, 1},  {4, 1},  {8, 1},   {16, 1},  {8, 3},   {32, 1},  {16, 3}, {64, 1},
                                   {32, 3}, {64, 2}, {64, 3}, {128, 2}, {128, 3}, {256, 2}, {256, 3}, {512, 2}};
template <>
inline constexpr RowShape kBwdShapes<GCLIP_F32>[] = {{2, 1},  {4, 1},  {8, 1},   {16, 1},  {32, 1},  {16, 3},
                                                     {64, 1}, {32, 3}, {64, 2},  {64, 3},  {64, 4},  {128, 3},
                                                     {128, 4}, {256, 3}, {256, 4}, {512, 3}, {512, 4}};
// Few rows of a 16-bit format backward, of up to 2048 columns: no shape whose
// rows leave half of the compute units without one (1021 x 1111 in bfloat16
// 9.3 us instead of 10.9, 2048 x 768 8.1 instead of 10.4; from 4096 rows on
// the shapes that hold a row with fewer idle lanes are faster, and in binary32
// no others are).
constexpr uint32_t kFewBwdRows = 2048, kFewBwdMax = 2048;
constexpr RowShape kFewBwdShapes[] = {{1, 1}, {2, 1}, {4, 1}, {8, 1}, {16, 1}, {32, 1}, {64, 1}, {64, 2}, {128, 2}};
template <int DT>
constexpr bool few_bwd(uint32_t rows, uint32_t size) {
  return DT != GCLIP_F32 && rows <= kFewBwdRows && size <= kFewBwdMax;
}
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
inline bool in_registers(uint32_t size, uint32_t most) { return size >= kRegistersMin && size <= most; }

// Threads of a workgroup of the backward kernel: all that a compute unit's
// registers hold, so that each unit leaves one partial sum of the weights'
// gradients, of kBwdParts at most.
constexpr uint32_t bwd_threads(uint32_t columns) { return columns <= 8 ? 1024 : 512; }
constexpr uint32_t kBwdParts = 256;
template <int DT>
inline uint32_t bwd_parts(uint32_t rows, uint32_t size) {
  const uint32_t unit = DT == GCLIP_F32 ? 4 : 8;
  const RowShape s = few_bwd<DT>(rows, size) ? kFewBwdShapes[row_shape_of(kFewBwdShapes, unit, size)]
                                             : kBwdShapes<DT>[row_shape_of(kBwdShapes<DT>, unit, size)];
  const uint32_t at_once = bwd_threads(s.units * unit) / s.lanes, need = (rows - 1) / at_once + 1;
  return need < kBwdParts ? need : kBwdParts;
}

// What a call moves decides how.  Up to kStreamBytes the matrices may lie in
// the 256 MB cache before memory, where the kernel before has left them:
// ordinary loads find them there, and nontemporal stores, which pass the L2
// by, are written there.  Above, nontemporal loads and ordinary stores are
// faster.  Measured in bfloat16 (in turn streamed, not): norm 16384 x 2048,
// 134 MB, 26.4 and 23.4 us; residual step 8192 x 2048, 134 MB, 28.2 and 23.5;
// norm gradient 12288 x 2048, 151 MB, 32.3 and 34.0; residual gradient
// 8192 x 2048, 168 MB, 36.8 and 37.8; residual step 16384 x 2048, 268 MB, 46.6
// and 49.6.
constexpr uint64_t kStreamBytes = 144ull << 20;

// A dispatch counts its lanes in each direction in 32 bits, and the largest
// matrices have more units than that (a dropout of 2^32 units left some of
// them undone, with no error): workgroups beyond kGridRow go into further
// rows of the grid, whose end no work is left for.
constexpr uint32_t kGridRow = 1u << 20;
inline dim3 grid_of(uint64_t workgroups, uint32_t layers = 1) {
  const uint64_t x = workgroups < kGridRow ? workgroups : kGridRow;
  return dim3((uint32_t)x, (uint32_t)((workgroups + x - 1) / x), layers);
}

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
