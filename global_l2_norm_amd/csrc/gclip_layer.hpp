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
  float eps;
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

// Partial sums of the weights' gradients for a matrix of this shape.
uint32_t layer_parts(int64_t rows, int64_t size);

// residual: the residual step; drop: null for none.
hipError_t launch_layer_forward(const FwdArgs& a, int32_t dtype, bool residual, const DropArgs* drop, hipStream_t st);
hipError_t launch_layer_backward(const BwdArgs& a, int32_t dtype, const DropArgs* drop, hipStream_t st);
hipError_t launch_dropout(const Rows& x, const Rows& y, uint32_t rows, uint32_t size, int32_t dtype,
                          const DropArgs& drop, hipStream_t st);

}  // namespace gclip
