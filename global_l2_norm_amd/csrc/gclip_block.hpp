// gclip_block.hpp -- what the host side of the block calls hands to their
// kernels (include/gclip_block.h; internal to libgclip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gclip_block.h"
#include "gclip_layer.hpp"

namespace gclip {

// A matrix in 8 bits: its values (rows of ld bytes) and `count` scales a row,
// one for every GCLIP_SCALE_BLOCK columns, or one (row).
struct Eight {
  uint64_t at, ld, scales;
  uint32_t count, row;
};

struct RmsFwdArgs {
  Rows x, residual, h, y;
  Eight y8, kept;  // y8.at: y is not written
  uint64_t weight;
  float* rstd;
  uint32_t rows, size;
  int32_t wdt;
  float eps;
  int32_t streamed;  // see kStreamBytes
};

struct RmsBwdArgs {
  Rows dy, dh, x, dres, dx;  // dh.at 0: none; the plain norm writes dres alone, a residual step without dropout too
  Eight x8;                  // x8.at: in the place of x
  const float* rstd;
  uint64_t weight, dweight;
  float* partials;  // [parts][part_columns(size)]: sums of dy * n
  float* sums;      // [rows], long rows: their means of dy * weight * n
  uint32_t rows, size;
  int32_t wdt, gdt, accumulate;
  uint32_t parts;
  uint32_t row_groups, strips;  // rows in registers: workgroups that take rows, and before them the weight's gradient
  int32_t streamed;
};

// A part's columns lie at whole units of 16 bytes.
__host__ __device__ constexpr uint64_t part_columns(uint32_t size) { return ((uint64_t)size + 3) / 4 * 4; }

// Few rows in registers: the weight's gradient is taken by workgroups of its
// own, and leaves no parts.  Residual gradients with dropout, so and by parts:
// 256 x 2048 in bfloat16 5.9 and 9.3 us, 512 x 2048 8.3 and 10.8, 1021 x 2048
// 13.4 and 11.3; in binary32 256 x 8192 13.2 and 16.3, 512 x 4096 13.7 and
// 13.9, 512 x 8192 20.5 and 19.4.
constexpr uint32_t kStripRows = 256, kStripMoreRows = 512, kStripMoreMax = 4096;
inline bool weight_by_strips(uint32_t rows, uint32_t size) {
  return rows <= kStripRows || (rows <= kStripMoreRows && size <= kStripMoreMax);
}

// Gradients of rows in registers: the shapes of the layer norm's for shorter
// rows, and for longer ones 1024 lanes, a workgroup, each.  By them and by
// the other shapes: 2048 x 8192 norms with a checkpoint in bfloat16 21.0 and
// 22.6 us, in binary32 30.3 and 33.7, 4000 x 4100 30.4 and 34.3; but 4000 x
// 4100 residual gradients with dropout in bfloat16, which leave half of the
// lanes idle, 47.3 and 39.4.  2048 x 16384 in bfloat16 44.9 us in one pass,
// 64.6 in two; with residual and dropout 78 and 87, in binary32 147 and 167.
constexpr uint32_t kRmsBwdMax = 16384, kRmsBwdLanes = 1024;
template <int DT>
constexpr uint32_t kRmsShortMax = DT == GCLIP_F32 ? 4096 : 6144;
template <int DT>
constexpr RowShape kRmsLongShapes[] = {{kRmsBwdLanes, 1}, {kRmsBwdLanes, 2}};
template <>
inline constexpr RowShape kRmsLongShapes<GCLIP_F32>[] = {{kRmsBwdLanes, 2}, {kRmsBwdLanes, 3}, {kRmsBwdLanes, 4}};
template <int DT>
inline uint32_t rms_bwd_parts(uint32_t rows, uint32_t size) {
  return size <= kRmsShortMax<DT> ? bwd_parts<DT>(rows, size) : rows < kBwdParts ? rows : kBwdParts;
}

struct ActArgs {
  Rows gate, up, y, dy, dgate, dup;  // up.at, y.at 0: none
  Eight gate8, up8;
  uint32_t rows, size;
};

// The most partial sums of the weight's gradient for a matrix of this shape
// in any format.
uint32_t rms_parts(int64_t rows, int64_t size);

// residual: the residual step; drop: null for none.
hipError_t launch_rms_forward(const RmsFwdArgs& a, int32_t dtype, bool residual, const DropArgs* drop, hipStream_t st);
hipError_t launch_rms_backward(const RmsBwdArgs& a, int32_t dtype, bool residual, const DropArgs* drop,
                               hipStream_t st);
hipError_t launch_activation(const ActArgs& a, int32_t dtype, int32_t kind, bool backward, bool streamed,
                             hipStream_t st);
hipError_t launch_pack8(const Rows& x, const Eight& out, uint32_t rows, uint32_t size, int32_t dtype, hipStream_t st);
hipError_t launch_unpack8(const Eight& x, const Rows& out, uint32_t rows, uint32_t size, int32_t dtype,
                          hipStream_t st);

// Their parts for one storage format: rows in registers, without and with
// matrices in 8 bits; rows of other lengths; the join of the partial sums.
template <int DT, bool EIGHT>
hipError_t rms_forward_rows(const RmsFwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st);
template <int DT, bool EIGHT>
hipError_t rms_backward_rows(const RmsBwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st);
template <int DT>
hipError_t rms_join_weight_grad(const RmsBwdArgs& a, hipStream_t st);
template <int DT>
hipError_t activation_of(const ActArgs& a, int32_t kind, bool backward, bool streamed, hipStream_t st);

}  // namespace gclip
