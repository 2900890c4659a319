// gclip_rms_backward.hpp -- the gradients of the RMS norm and of its residual
// step for rows that fit into registers, and the join of the weight's
// gradient; instantiated for one storage format, without or with the normed
// matrix in 8 bits, in each of gclip_rms_backward_*.hip.
#pragma once

#include "gclip_block_device.hpp"

namespace gclip {

typedef float f32x4 __attribute__((ext_vector_type(4)));

template <int DT>
__device__ __forceinline__ void store_rms_weight_grad(const RmsBwdArgs& a, uint32_t c, float t) {
  if (DT == GCLIP_F32 || a.gdt == GCLIP_F32) {
    const uint64_t p = a.dweight + c * 4ull;
    if (a.accumulate) t += elem_float<GCLIP_F32>(load_elem<GCLIP_F32>(p));
    store_elem<GCLIP_F32>(p, elem_bits<GCLIP_F32>(t));
  } else {
    const uint64_t p = a.dweight + c * 2ull;
    if (a.accumulate) t += elem_float<DT>(load_elem<DT>(p));
    store_elem<DT>(p, elem_bits<DT>(t));
  }
}

// The weight's gradient of few rows: it takes neither the rows' sums nor their
// results, so workgroups of their own, in the same launch, take a strip of
// columns each down all rows, from the caches, and no parts are left to join.
// Where the results go in place over what the strips read, the strips have a
// launch of their own, before the rows'.  A lane's loads of eight rows at once
// instead of four, 256 x 9000 in binary32 18.8 us and 14.6; strips of 64 units
// 256 x 2048 in bfloat16 9.1 and 5.9.
constexpr uint32_t kStripLanes = 16;  // units of a strip
template <int DT, bool EIGHT, uint32_t WAVES>
__device__ __forceinline__ void strip_weight_grad(const RmsBwdArgs& a, uint32_t strip, float* meet) {
  constexpr uint32_t kU = kUnit<DT>, kRows = 64 / kStripLanes * WAVES, kCols = kStripLanes * kU;
  const uint32_t lane = threadIdx.x % kStripLanes, slot = threadIdx.x / kStripLanes;
  const uint32_t unit = strip * kStripLanes + lane, c = unit * kU, c8 = min(c, (a.size - 1) / kU * kU);
  constexpr int kAtOnce = 4;  // rows of a lane under way
  float dw[kU] = {};
  for (uint32_t first = 0; first < a.rows; first += kAtOnce * kRows) {
    u32x4 ny[kAtOnce], nx[kAtOnce];
    Unit8<DT> n8[kAtOnce];
    float ns[kAtOnce], rstd[kAtOnce];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const uint32_t r = min(first + i * kRows + slot, a.rows - 1);
      ny[i] = load_columns<DT, 1, 0, false>(a.dy.at + r * a.dy.ld, unit, 0, a.size);
      if constexpr (EIGHT) {
        n8[i] = load_eight<DT, false>(a.x8.at + r * a.x8.ld, c8);
        ns[i] = load_scale(a.x8, r, c8);
      } else {
        nx[i] = load_columns<DT, 1, 0, false>(a.x.at + r * a.x.ld, unit, 0, a.size);
      }
      rstd[i] = a.rstd[r];
    }
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      if (first + i * kRows + slot >= a.rows) break;
      float y[kU], n[kU];
      settle<DT, 1, 0>(ny[i], unit, 0, a.size);
      unpack_unit<DT>(ny[i], y);
      if constexpr (EIGHT) {
        unit_value<DT>(n8[i], ns[i], n);  // past the row's end y is 0, and nothing is stored
      } else {
        settle<DT, 1, 0>(nx[i], unit, 0, a.size);
        unpack_unit<DT>(nx[i], n);
      }
#pragma unroll
      for (uint32_t j = 0; j < kU; ++j) dw[j] = __builtin_fmaf(y[j], n[j] * rstd[i], dw[j]);
    }
  }
#pragma unroll
  for (uint32_t j = 0; j < kU; ++j) {
    const float t = across_rows<kStripLanes>(dw[j]);
    if (threadIdx.x % 64 < kStripLanes) meet[threadIdx.x / 64 * kCols + lane * kU + j] = t;
  }
  __syncthreads();
  if (threadIdx.x < kCols) {
    float t = meet[threadIdx.x];
#pragma unroll
    for (uint32_t k = 1; k < WAVES; ++k) t += meet[k * kCols + threadIdx.x];
    const uint32_t column = strip * kCols + threadIdx.x;
    if (column < a.size) store_rms_weight_grad<DT>(a, column, t);
  }
}

template <int LANES>
constexpr uint32_t rms_bwd_threads(uint32_t columns) {
  return LANES > (int)bwd_threads(columns) ? LANES : bwd_threads(columns);
}

// With n = x rstd and g = dy weight:
//   dx = rstd (g - n sum(g n) / size),  dweight = sum over rows of dy n
// in one pass: a row's dy and x are read once, into the registers of LANES
// lanes, where the row's sum and then dx are taken from them; the columns'
// sums stay in registers over all rows of the workgroup, whose rows meet in
// shared memory at the end, and each workgroup -- one for each compute unit --
// leaves one part of them.  While a row is worked on, the loads of the
// workgroup's next one are under way.  x in 8 bits is half of a 16-bit
// matrix's bytes, and four operations more for each four elements.
// Bound by memory: 16384 x 2048 bfloat16 residual gradients with dropout, x in
// 8 bits, 49.4 us, 303 MB at 6.1 TB/s (and 4.8 us for the join).  Where a row
// fills a workgroup its waves wait for each other twice a row: 2048 x 16384
// 38.6 us, 201 MB at 5.2 TB/s; with dropout in binary32 130 us, 5.2 TB/s,
// where 25 registers of a lane do not fit and go through memory.
template <int DT, int LANES, int NV, int SURE, bool RES, bool DROP, bool EIGHT, bool STREAMED>
__global__ __launch_bounds__(rms_bwd_threads<LANES>(NV * kUnit<DT>)) void k_rms_rows_grad(RmsBwdArgs a, DropArgs d) {
  constexpr uint32_t kBwdThreads = rms_bwd_threads<LANES>(NV * kUnit<DT>);
  constexpr uint32_t kRows = kBwdThreads / LANES;  // of a workgroup at a time
  constexpr uint32_t kCols = LANES * NV * kUnit<DT>;
  constexpr uint32_t kMeet = LANES < 64 ? kBwdThreads / 64 : kRows;  // sums of a column that meet
  // More than eight columns for each of 1024 lanes: their registers do not hold
  // the weight and the columns' sums besides, which lie in shared memory, nor
  // in binary32 the next row's dh.
  constexpr bool kAside = LANES == (int)kRmsBwdLanes && NV * kUnit<DT> > 8, kLate = kAside && DT == GCLIP_F32;
  constexpr int kFours = NV * (int)kUnit<DT> / 4;
  __shared__ f32x4 aside[kAside ? 2 : 1][kAside ? kFours * LANES : 1];
  __shared__ float red[2][kBwdThreads / 64];
  constexpr uint32_t kStripFloats = kBwdThreads / 64 * kStripLanes * kUnit<DT>;  // see strip_weight_grad()
  constexpr uint32_t kSums = kMeet > 1 ? kMeet * kCols : 1;
  __shared__ float own_sums[kAside ? 1 : kSums > kStripFloats ? kSums : kStripFloats];
  float* sums = kAside ? reinterpret_cast<float*>(aside) : own_sums;
  if (blockIdx.x < a.strips) {
    strip_weight_grad<DT, EIGHT, kBwdThreads / 64>(a, blockIdx.x, sums);
    return;
  }
  const uint32_t group = blockIdx.x - a.strips;
  const uint32_t lane = threadIdx.x % LANES;
  uint32_t slot = threadIdx.x / LANES;
  if constexpr (LANES >= 64) slot = __builtin_amdgcn_readfirstlane(slot);
  const uint32_t step = DROP ? drop_step(d) : 0u;

  u32x4 ny[NV], nx[EIGHT ? 1 : NV], nh[RES && !kLate ? NV : 1];
  Unit8<DT> n8[EIGHT ? NV : 1];
  float ns[EIGHT ? NV : 1];
  float nrstd;
  uint32_t base = group * kRows;
  const uint32_t last8 = (a.size - 1) / kUnit<DT> * kUnit<DT>;
  const auto fetch = [&](uint32_t first) {
    // rows past the end are read as the last one; they count for nothing
    const uint32_t r = min(first + slot, a.rows - 1);
    const uint64_t dy = a.dy.at + r * a.dy.ld, x = a.x.at + r * a.x.ld;
    [[maybe_unused]] const uint64_t dh = a.dh.at + r * a.dh.ld;
    nrstd = a.rstd[r];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      ny[k] = load_columns<DT, LANES, SURE, STREAMED>(dy, lane, k, a.size);
      if constexpr (EIGHT) {
        const uint32_t c = k < SURE ? column_of<DT>(lane, LANES, k) : min(column_of<DT>(lane, LANES, k), last8);
        n8[k] = load_eight<DT, STREAMED>(a.x8.at + r * a.x8.ld, c);
        ns[k] = load_scale(a.x8, r, c);
      } else {
        nx[k] = load_columns<DT, LANES, SURE, STREAMED>(x, lane, k, a.size);
      }
      if constexpr (RES && !kLate)
        nh[k] = a.dh.at ? load_columns<DT, LANES, SURE, STREAMED>(dh, lane, k, a.size) : u32x4{0u, 0u, 0u, 0u};
    }
  };
  fetch(base);
  float w[NV][kUnit<DT>], dw[kAside ? 1 : NV][kUnit<DT>];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    weight_columns<DT, LANES, SURE>(a.weight, a.wdt, lane, k, a.size, 1.0f, w[k]);
    if constexpr (kAside) {
#pragma unroll
      for (int f = 0; f < (int)kUnit<DT> / 4; ++f) {
        const int at = (k * (int)kUnit<DT> / 4 + f) * LANES + lane;
        aside[0][at] = f32x4{w[k][4 * f], w[k][4 * f + 1], w[k][4 * f + 2], w[k][4 * f + 3]};
        aside[1][at] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      }
    } else {
#pragma unroll
      for (uint32_t j = 0; j < kUnit<DT>; ++j) dw[k][j] = 0.0f;
    }
  }
  const float count = (float)a.size, inverse = 1.0f / count;
  const bool full = a.size == kCols;
  uint32_t turn = 0;

  while (base < a.rows) {
    const uint32_t r = base + slot;
    const float rstd = nrstd;
    float g[NV][kUnit<DT>], n[NV][kUnit<DT>];
    u32x4 hh[RES ? NV : 1];
    if constexpr (RES && kLate) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        hh[k] = a.dh.at ? load_columns<DT, LANES, SURE, STREAMED>(a.dh.at + min(r, a.rows - 1) * a.dh.ld, lane, k, a.size)
                        : u32x4{0u, 0u, 0u, 0u};
    }
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      settle<DT, LANES, SURE>(ny[k], lane, k, a.size, full);
      if constexpr (EIGHT) {
        if (k >= SURE && !full) settle_eight<DT>(n8[k], column_of<DT>(lane, LANES, k), a.size);
        unit_value<DT>(n8[k], ns[k], n[k]);
      } else {
        settle<DT, LANES, SURE>(nx[k], lane, k, a.size, full);
        unpack_unit<DT>(nx[k], n[k]);
      }
      // nothing past the row's end or the last row enters the sums, where an
      // infinite rstd or scale would make it a NaN
      const float rk = r < a.rows && (k < SURE || column_of<DT>(lane, LANES, k) < a.size) ? rstd : 0.0f;
      if (r >= a.rows) {
        ny[k] = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
        for (uint32_t j = 0; j < kUnit<DT>; ++j) n[k][j] = 0.0f;
      }
      unpack_unit<DT>(ny[k], g[k]);
      if constexpr (RES && !kLate) {
        settle<DT, LANES, SURE>(nh[k], lane, k, a.size, full);
        hh[k] = nh[k];
      }
      if constexpr (kAside) {
#pragma unroll
        for (int f = 0; f < (int)kUnit<DT> / 4; ++f) {
          const int at = (k * (int)kUnit<DT> / 4 + f) * LANES + lane;
          const f32x4 wf = aside[0][at];
          f32x4 sum = aside[1][at];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int j = 4 * f + i;
            n[k][j] *= rk;
            sum[i] = __builtin_fmaf(g[k][j], n[k][j], sum[i]);
            g[k][j] *= wf[i];
            s = __builtin_fmaf(g[k][j], n[k][j], s);
          }
          aside[1][at] = sum;
        }
      } else {
#pragma unroll
        for (uint32_t j = 0; j < kUnit<DT>; ++j) {
          n[k][j] *= rk;
          dw[k][j] = __builtin_fmaf(g[k][j], n[k][j], dw[k][j]);
          g[k][j] *= w[k][j];
          s = __builtin_fmaf(g[k][j], n[k][j], s);
        }
      }
    }
    const uint32_t next = base + a.row_groups * kRows;
    if (next < a.rows) fetch(next);
    // the next row's sum uses the other words
    const float c2 = rstd * divided(row_sum<LANES>(s, red[turn]), count, inverse);
    turn ^= 1u;
    if (r < a.rows) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t c = column_of<DT>(lane, LANES, k);
        float v[kUnit<DT>];
#pragma unroll
        for (uint32_t j = 0; j < kUnit<DT>; ++j) v[j] = __builtin_fmaf(rstd, g[k][j], -(n[k][j] * c2));
        if constexpr (RES) {
          float q[kUnit<DT>];
          if constexpr (kLate) settle<DT, LANES, SURE>(hh[k], lane, k, a.size, full);
          unpack_unit<DT>(hh[k], q);
#pragma unroll
          for (uint32_t j = 0; j < kUnit<DT>; ++j) v[j] += q[j];
        }
        store_columns<DT, LANES, SURE, !STREAMED>(a.dres.at + r * a.dres.ld, lane, k, a.size, pack_unit<DT>(v));
        if constexpr (DROP) {
          drop_unit<DT>(d, step, r, c, v);
          store_columns<DT, LANES, SURE, !STREAMED>(a.dx.at + r * a.dx.ld, lane, k, a.size, pack_unit<DT>(v));
        }
      }
    }
    base = next;
  }

  // this workgroup's part of the columns' sums
  if (!a.dweight || a.strips > 0) return;
  float* part = a.partials + group * part_columns(a.size);
  if constexpr (kMeet > 1) {
    const uint32_t row = LANES < 64 ? threadIdx.x / 64 : slot;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (uint32_t j = 0; j < kUnit<DT>; ++j) {
        const float t = across_rows<LANES>(dw[k][j]);
        if (LANES >= 64 || threadIdx.x % 64 < LANES) sums[row * kCols + column_of<DT>(lane, LANES, k) + j] = t;
      }
    }
    __syncthreads();
    for (uint32_t c = threadIdx.x; c < a.size; c += kBwdThreads) {
      float t = sums[c];
#pragma unroll
      for (uint32_t i = 1; i < kMeet; ++i) t += sums[i * kCols + c];
      if (a.parts == 1) store_rms_weight_grad<DT>(a, c, t);
      else part[c] = t;
    }
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
#pragma unroll
      for (int f = 0; f < (int)kUnit<DT> / 4; ++f) {
        const uint32_t c = column_of<DT>(lane, LANES, k) + 4 * f;
        f32x4 t;
        if constexpr (kAside) t = aside[1][(k * (int)kUnit<DT> / 4 + f) * LANES + lane];
        else t = f32x4{dw[k][4 * f], dw[k][4 * f + 1], dw[k][4 * f + 2], dw[k][4 * f + 3]};
        if (c >= a.size) continue;
        if (a.parts > 1) {
          *reinterpret_cast<f32x4*>(part + c) = t;
        } else {
#pragma unroll
          for (uint32_t j = 0; j < 4; ++j)
            if (c + j < a.size) store_rms_weight_grad<DT>(a, c + j, t[j]);
        }
      }
    }
  }
}

// The sum of the parts: a workgroup takes 64 columns, its sixteen waves share
// the parts, in a fixed order, all loads of a wave under way at once.  256
// parts of 2048 columns 4.8 us, of 16384 4.8: a launch and one way to the
// cache behind the kernel before.
constexpr uint32_t kRmsJoinThreads = 1024;
template <int DT>
__global__ __launch_bounds__(kRmsJoinThreads) void k_rms_join(RmsBwdArgs a) {
  constexpr uint32_t kWavesOf = kRmsJoinThreads / 64;
  __shared__ float red[kWavesOf][64];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t i = workgroup_of_grid() * 64 + lane;
  float t = 0.0f;
  if (i < a.size) {
#pragma unroll 16
    for (uint32_t p = wave; p < a.parts; p += kWavesOf) t += a.partials[p * part_columns(a.size) + i];
  }
  red[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && i < a.size) {
#pragma unroll
    for (uint32_t k = 1; k < kWavesOf; ++k) t += red[k][lane];
    store_rms_weight_grad<DT>(a, (uint32_t)i, t);
  }
}

template <int DT>
hipError_t rms_join_weight_grad(const RmsBwdArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((k_rms_join<DT>), grid_of(((uint64_t)a.size + 63) / 64), dim3(kRmsJoinThreads), 0, st, a);
  return hipGetLastError();
}

// Rows' workgroups (a.row_groups of them) and strips'.
template <int DT, bool EIGHT, int LANES, int NV, int SURE, bool STREAMED>
hipError_t rms_backward_launch(const RmsBwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  const dim3 grid(a.row_groups + a.strips), block(rms_bwd_threads<LANES>(NV * kUnit<DT>));
  const DropArgs none{};
  if (!residual)
    hipLaunchKernelGGL((k_rms_rows_grad<DT, LANES, NV, SURE, false, false, EIGHT, STREAMED>), grid, block, 0, st, a, none);
  else if (!drop)
    hipLaunchKernelGGL((k_rms_rows_grad<DT, LANES, NV, SURE, true, false, EIGHT, STREAMED>), grid, block, 0, st, a, none);
  else
    hipLaunchKernelGGL((k_rms_rows_grad<DT, LANES, NV, SURE, true, true, EIGHT, STREAMED>), grid, block, 0, st, a, *drop);
  return hipGetLastError();
}

template <int DT, bool EIGHT, int LANES, int NV, int SURE, bool STREAMED>
hipError_t rms_backward_shape(RmsBwdArgs a, bool residual, const DropArgs* drop, hipStream_t st) {
  a.parts = a.row_groups = rms_bwd_parts<DT>(a.rows, a.size);
  if (a.dweight && a.parts > 1 && weight_by_strips(a.rows, a.size)) {
    a.strips = (a.size - 1) / (kStripLanes * kUnit<DT>) + 1;
    const auto over = [&](uint64_t out) { return out != 0 && (out == a.dy.at || out == a.x.at); };
    if (over(a.dres.at) || over(a.dx.at)) {
      RmsBwdArgs weight_alone = a;
      weight_alone.row_groups = 0;
      const hipError_t e =
          rms_backward_launch<DT, EIGHT, LANES, NV, SURE, STREAMED>(weight_alone, residual, drop, st);
      if (e != hipSuccess) return e;
      a.dweight = 0;
      a.strips = 0;
    }
    return rms_backward_launch<DT, EIGHT, LANES, NV, SURE, STREAMED>(a, residual, drop, st);
  }
  const hipError_t e = rms_backward_launch<DT, EIGHT, LANES, NV, SURE, STREAMED>(a, residual, drop, st);
  if (e != hipSuccess || a.parts == 1 || !a.dweight) return e;
  return rms_join_weight_grad<DT>(a, st);
}

template <int DT, bool EIGHT, int I = 0>
hipError_t rms_backward_of(int shape, const RmsBwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  constexpr RowShape s = kBwdShapes<DT>[I];
  if constexpr (s.lanes * s.units * kUnit<DT> < kRmsShortMax<DT>) {
    if (shape != I) return rms_backward_of<DT, EIGHT, I + 1>(shape, a, residual, drop, st);
  }
  constexpr int sure = sure_units(kBwdShapes<DT>, I);
  return a.streamed ? rms_backward_shape<DT, EIGHT, s.lanes, s.units, sure, true>(a, residual, drop, st)
                    : rms_backward_shape<DT, EIGHT, s.lanes, s.units, sure, false>(a, residual, drop, st);
}

template <int DT, bool EIGHT, int I = 0>
hipError_t rms_backward_few(int shape, const RmsBwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if constexpr (I + 1 < (int)(sizeof(kFewBwdShapes) / sizeof(RowShape))) {
    if (shape != I) return rms_backward_few<DT, EIGHT, I + 1>(shape, a, residual, drop, st);
  }
  constexpr RowShape s = kFewBwdShapes[I];
  return rms_backward_shape<DT, EIGHT, s.lanes, s.units, sure_units(kFewBwdShapes, I), false>(a, residual, drop, st);
}

template <int DT, bool EIGHT, int I = 0>
hipError_t rms_backward_long(int shape, const RmsBwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if constexpr (I + 1 < (int)(sizeof(kRmsLongShapes<DT>) / sizeof(RowShape))) {
    if (shape != I) return rms_backward_long<DT, EIGHT, I + 1>(shape, a, residual, drop, st);
  }
  constexpr RowShape s = kRmsLongShapes<DT>[I];
  constexpr int sure = I > 0 ? sure_units(kRmsLongShapes<DT>, I) : kRmsShortMax<DT> / kUnit<DT> / s.lanes;
  return a.streamed ? rms_backward_shape<DT, EIGHT, s.lanes, s.units, sure, true>(a, residual, drop, st)
                    : rms_backward_shape<DT, EIGHT, s.lanes, s.units, sure, false>(a, residual, drop, st);
}

template <int DT, bool EIGHT>
hipError_t rms_backward_rows(const RmsBwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if constexpr (DT != GCLIP_F32) {
    if (few_bwd<DT>(a.rows, a.size))
      return rms_backward_few<DT, EIGHT>(row_shape_of(kFewBwdShapes, kUnit<DT>, a.size), a, residual, drop, st);
  }
  if (a.size > kRmsShortMax<DT>)
    return rms_backward_long<DT, EIGHT>(row_shape_of(kRmsLongShapes<DT>, kUnit<DT>, a.size), a, residual, drop, st);
  return rms_backward_of<DT, EIGHT>(row_shape_of(kBwdShapes<DT>, kUnit<DT>, a.size), a, residual, drop, st);
}

}  // namespace gclip
