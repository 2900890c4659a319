// gclip_layer_forward.hpp -- the norm and the residual step for rows that
// fit into registers; instantiated for one storage format in each of
// gclip_layer_forward_*.hip.
#pragma once

#include "gclip_layer_device.hpp"

namespace gclip {

// The most threads of a workgroup: four waves, of which rows of up to a wave
// share one; workgroups of a wave each where the rows are few.  Two rows of
// 128 lanes share one in 16-bit formats (2000 x 2500 residual with dropout
// 11.7 us, 512 x 1000 4.0; a workgroup each: 12.5 and 4.2), and have one each
// in binary32 (256 x 384 norm 3.1 us; shared: 3.2).
template <int DT, int LANES>
constexpr int kFwdThreads = LANES > 256 || (LANES == 128 && DT == GCLIP_F32) ? LANES : 256;

// Workgroups of four waves for each compute unit, by the columns that a lane
// holds: as many as its registers let run at once, so that each goes through
// its rows with the next one's loads under way.  Measured: 2 for 32 columns
// (4096 x 2048 binary32 residual 21.4 us; 3: 24.0, 4: 27.4), 4 for 12 to 24
// (8192 x 1024 bfloat16 norm 7.3 us; 2: 7.9), 8 for up to 8 (131072 x 64:
// 7.8 us; 4: 8.1, 16: 8.4).
constexpr uint32_t fwd_workgroups(uint32_t columns) { return columns <= 8 ? 8 : columns <= 24 ? 4 : 2; }

// y = (x - mean) rstd weight + bias, in one pass: a row's elements are read
// once, into the registers of LANES lanes, where its mean, its squared
// deviations from it (of the mean, not of zero: no cancellation) and y are
// taken from them in turn.  While a row is worked on, the loads of the
// workgroup's next one are under way; weight and bias stay in registers.
//
// Bound by memory: 16384 x 2048 in bfloat16 takes 22.0 us, 6.1 TB/s of one
// read and one write (a copy of these bytes: 22.7), the residual step with
// dropout 44.0 us, 6.1 TB/s; 8192 x 768 in binary32 9.3 us, 5.4 TB/s.  With a
// workgroup a row and three passes through the caches the first took 45.9 us.
// Reading rows past the end as the last one, rather than not, keeps the loads
// of the next row out of a branch, which would be waited for at its end
// (residual step: 53.7 us against 46.0).
template <int DT, int LANES, int NV, int SURE, bool RES, bool DROP, bool STREAMED>
__global__ __launch_bounds__((kFwdThreads<DT, LANES>)) void k_norm_rows(FwdArgs a, DropArgs d) {
  constexpr int kThreads = kFwdThreads<DT, LANES>;
  const uint32_t at_once = LANES > 64 ? kThreads / LANES : blockDim.x / LANES;  // rows of a workgroup
  __shared__ float red[3][kThreads / 64];
  const uint32_t lane = threadIdx.x % LANES;
  uint32_t slot = threadIdx.x / LANES;
  if constexpr (LANES >= 64) slot = __builtin_amdgcn_readfirstlane(slot);
  const uint32_t step = DROP ? drop_step(d) : 0u;

  u32x4 nx[NV], nr[NV];
  uint32_t base = blockIdx.x * at_once;
  const auto fetch = [&](uint32_t first) {
    // rows past the end are read as the last one, and not written
    const uint32_t r = min(first + slot, a.rows - 1);
    const uint64_t x = a.x.at + r * a.x.ld, q = a.residual.at + r * a.residual.ld;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      nx[k] = load_columns<DT, LANES, SURE, STREAMED>(x, lane, k, a.size);
      if constexpr (RES) nr[k] = load_columns<DT, LANES, SURE, STREAMED>(q, lane, k, a.size);
    }
  };
  fetch(base);
  float w[NV][kUnit<DT>], b[NV][kUnit<DT>];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    weight_columns<DT, LANES, SURE>(a.weight, a.wdt, lane, k, a.size, 1.0f, w[k]);
    weight_columns<DT, LANES, SURE>(a.bias, a.wdt, lane, k, a.size, 0.0f, b[k]);
  }
  const float count = (float)a.size, inverse = 1.0f / count;
  const bool full = a.size == LANES * NV * kUnit<DT>;

  while (base < a.rows) {
    const uint32_t r = base + slot;
    float v[NV][kUnit<DT>];
    u32x4 o[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const uint32_t c = column_of<DT>(lane, LANES, k);
      settle<DT, LANES, SURE>(nx[k], lane, k, a.size, full);
      unpack_unit<DT>(nx[k], v[k]);
      if constexpr (RES) {
        float q[kUnit<DT>];
        settle<DT, LANES, SURE>(nr[k], lane, k, a.size, full);
        unpack_unit<DT>(nr[k], q);
        if constexpr (DROP) drop_unit<DT>(d, step, r, c, v[k]);
#pragma unroll
        for (uint32_t j = 0; j < kUnit<DT>; ++j) v[k][j] += q[j];
        o[k] = pack_unit<DT>(v[k]);
        unpack_unit<DT>(o[k], v[k]);
      }
    }
    const uint32_t next = base + gridDim.x * at_once;
    if (next < a.rows) fetch(next);
    if constexpr (RES) {
      if (r < a.rows) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
          store_columns<DT, LANES, SURE, !STREAMED>(a.h.at + r * a.h.ld, lane, k, a.size, o[k]);
      }
    }

    // the mean, then the squares of what is left of it and, where the sum may
    // round, what is left itself: in a row of little spread it takes the sum's
    // own error off, so a constant row's mean is its value, and its y the bias
    // (a row's sum of equal bfloat16 elements is exact up to 2^16 of them, of
    // binary16 ones up to 2^13); rows whose sums, or whose var + eps, leave
    // binary32 go through this again, scaled by a power of two (so does a row
    // with a NaN or an infinity, to no effect)
    constexpr bool kRounds = DT == GCLIP_F32 || (DT == GCLIP_F16 && LANES * NV * kUnit<DT> > 8192);
    float scale = 1.0f, mean, var;
    for (bool first = true;; first = false) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < NV; ++k)
#pragma unroll
        for (uint32_t j = 0; j < kUnit<DT>; ++j) s = __builtin_fmaf(v[k][j], scale, s);
      mean = divided(row_sum<LANES>(s, red[0]), count, inverse);
      s = 0.0f;
      float rest = 0.0f;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t c = column_of<DT>(lane, LANES, k);
        if (k < SURE || full || c + kUnit<DT> <= a.size) {
#pragma unroll
          for (uint32_t j = 0; j < kUnit<DT>; ++j) {
            const float t = __builtin_fmaf(v[k][j], scale, -mean);
            if (kRounds) rest += t;
            s = __builtin_fmaf(t, t, s);
          }
        } else {
          uint32_t left = c < a.size ? a.size - c : 0u;
          // recomputed for each row: the conditions would else be kept
          // in scalar registers over the loop, more than there are
          asm volatile("" : "+v"(left));
#pragma unroll
          for (uint32_t j = 0; j < kUnit<DT>; ++j) {
            const float t = j < left ? __builtin_fmaf(v[k][j], scale, -mean) : 0.0f;
            if (kRounds) rest += t;
            s = __builtin_fmaf(t, t, s);
          }
        }
      }
      if constexpr (kRounds) {
        row_sums<LANES>(s, rest, red[1], red[2]);
        rest = divided(rest, count, inverse);
        var = divided(s, count, inverse);
        // little: at most an eighth of the mean, where the subtractions are
        // exact but for outliers.  Elsewhere their roundings are more than
        // what the sum's own come to (twice the mean's error in rows around
        // zero).
        if (var <= mean * (mean * 0x1p-6f)) {
          mean += rest;
          var = __builtin_fmaf(-rest, rest, var);
          if (var < 0.0f) var = 0.0f;  // of a constant row, by rounding
        }
      } else {
        var = divided(row_sum<LANES>(s, red[1]), count, inverse);
      }
      if (!first) break;
      // rows that meet go through it again together, if one of them has to:
      // those of a wave, or of a workgroup, whose barriers all of its waves
      // have to reach equally often
      const auto leaves = [&](float t) { return !(t + a.eps <= 0x1.fffffep+127f); };
      bool again = leaves(var);
      if constexpr (LANES > 64) {
        static_assert(kThreads == LANES || !kRounds, "the sum of squares alone decides");
        for (int i = 0; kThreads > LANES && i < kThreads / 64; i += LANES / 64)
          again |= leaves(divided(waves_sum<LANES>(red[1] + i), count, inverse));
        again = __builtin_amdgcn_readfirstlane(again);
      } else {
        again = __any(again);
      }
      if (!again) break;
      if (leaves(var)) scale = 0x1p-96f;
    }
    float rstd = scale / sqrtf(var + a.eps * scale * scale);
    if (scale != 1.0f) {
      mean *= 0x1p+96f;
      rstd = rstd > a.rstd_max ? a.rstd_max : rstd;  // a constant row
    }

    if (r < a.rows) {
      const float hm = 0.5f * mean, tr = 2.0f * rstd;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (uint32_t j = 0; j < kUnit<DT>; ++j) v[k][j] = __builtin_fmaf(normed(v[k][j], hm, tr), w[k][j], b[k][j]);
        store_columns<DT, LANES, SURE, !STREAMED>(a.y.at + r * a.y.ld, lane, k, a.size, pack_unit<DT>(v[k]));
      }
      if (a.mean && lane == 0) {
        a.mean[r] = mean;
        a.rstd[r] = rstd;
      }
    }
    base = next;
  }
}

template <int DT, int LANES, int NV, int SURE, bool STREAMED>
hipError_t forward_shape(const FwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  // workgroups of a wave until there are four for each compute unit
  const uint32_t threads = LANES <= 64 && a.rows < 1024 * (64 / LANES) ? 64 : kFwdThreads<DT, LANES>;
  const uint32_t at_once = threads / LANES;
  const uint32_t most = 256u * fwd_workgroups(NV * kUnit<DT>) * 256 / threads;
  const uint32_t need = (a.rows + at_once - 1) / at_once;
  const dim3 grid(need < most ? need : most), block(threads);
  if (!residual)
    hipLaunchKernelGGL((k_norm_rows<DT, LANES, NV, SURE, false, false, STREAMED>), grid, block, 0, st, a, DropArgs{});
  else if (!drop)
    hipLaunchKernelGGL((k_norm_rows<DT, LANES, NV, SURE, true, false, STREAMED>), grid, block, 0, st, a, DropArgs{});
  else
    hipLaunchKernelGGL((k_norm_rows<DT, LANES, NV, SURE, true, true, STREAMED>), grid, block, 0, st, a, *drop);
  return hipGetLastError();
}

template <int DT, int I = 0>
hipError_t forward_of(int shape, const FwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if constexpr (I + 1 < (int)(sizeof(kFwdShapes<DT>) / sizeof(RowShape))) {
    if (shape != I) return forward_of<DT, I + 1>(shape, a, residual, drop, st);
  }
  constexpr RowShape s = kFwdShapes<DT>[I];
  return a.streamed ? forward_shape<DT, s.lanes, s.units, sure_units(kFwdShapes<DT>, I), true>(a, residual, drop, st)
                    : forward_shape<DT, s.lanes, s.units, sure_units(kFwdShapes<DT>, I), false>(a, residual, drop, st);
}

template <int DT, int I = 0>
hipError_t forward_few(int shape, const FwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if constexpr (I + 1 < (int)(sizeof(kFewShapes<DT>) / sizeof(RowShape))) {
    if (shape != I) return forward_few<DT, I + 1>(shape, a, residual, drop, st);
  }
  constexpr RowShape s = kFewShapes<DT>[I];
  return forward_shape<DT, s.lanes, s.units, sure_units(kFewShapes<DT>, I), false>(a, residual, drop, st);
}

template <int DT>
hipError_t forward_rows(const FwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  static_assert((uint64_t)kFewRows * kFwdMax * 4 * 4 <= kStreamBytes, "few rows are not streamed");
  if (a.rows <= kFewRows)
    return forward_few<DT>(row_shape_of(kFewShapes<DT>, kUnit<DT>, a.size), a, residual, drop, st);
  return forward_of<DT>(row_shape_of(kFwdShapes<DT>, kUnit<DT>, a.size), a, residual, drop, st);
}

}  // namespace gclip
