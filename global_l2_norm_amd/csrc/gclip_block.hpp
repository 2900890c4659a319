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
  float* partials;  // [parts][size]: sums of dy * n
  float* sums;      // [rows], long rows: their means of dy * weight * n
  uint32_t rows, size;
  int32_t wdt, gdt, accumulate;
  uint32_t parts;
  uint32_t row_groups;  // rows in registers: the workgroups that take rows
  int32_t streamed;
};

// Rows in registers, and no more than so many: the weight's gradient is taken
// by workgroups of its own.
constexpr uint32_t kStripRows = 128;

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
