// gclip_logprob.hpp -- what the host side of the log probability calls hands
// to their kernels (include/gclip_logprob.h; internal to libgclip).
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/gclip_logprob.h"
#include "gclip_layer.hpp"

namespace gclip {

constexpr uint32_t kLogpThreads = 256, kLogpNarrow = 64;
// Many rows: a wave each, while its lanes take few enough units (8192 x 4000 in
// bfloat16 22 us, 32 by 256 threads a row; but 1100 x 131072 84 and 60).
constexpr uint32_t kLogpManyRows = 1536, kLogpNarrowTurns = 64;
// Few rows: workgroups of more threads, one a row, which take a few units
// each, and more the more rows there are to fill the compute units; longer
// rows in segments, a workgroup each, and a join: at most a wave's lanes,
// which the join's first wave holds one each.  In bfloat16, so and in
// segments: 256 x 80000 13.9 and 16.6 us, 160 x 131072 15.3 and 17.4, 8 x
// 131072 13.3 and 8.0.
constexpr uint32_t kLogpFewRows = 256, kLogpWide = 1024, kLogpTurns = 8, kLogpRowsATurn = 8, kLogpSegments = 64;

struct LogpArgs {
  Rows x, dx;
  const int64_t* targets;
  int64_t ignore;
  float *stats, *logp, *entropy, *top_logp;
  int64_t* top_ids;
  const float *dlogp, *dentropy;
  float* parts;    // [rows][segments][4]: largest, sum, weighted sum of a segment
  uint64_t* keys;  // [rows][segments][top]
  uint32_t rows, size, top;
  uint32_t segments, turns;  // of a row; units of a thread in each
  uint32_t threads;          // of a workgroup
  int32_t streamed;          // see kStreamBytes
};

// Rows of up to so many columns lie in a wave's registers.
constexpr uint32_t kShortRow = 2048;

// How the rows of a shape are cut; no segments: short rows.
struct LogpCut {
  uint32_t segments, turns, threads;
};
LogpCut logp_cut(uint32_t rows, uint32_t size, int32_t dtype);

hipError_t launch_logprob_forward(const LogpArgs& a, int32_t dtype, hipStream_t st);
hipError_t launch_logprob_backward(const LogpArgs& a, int32_t dtype, hipStream_t st);

}  // namespace gclip
