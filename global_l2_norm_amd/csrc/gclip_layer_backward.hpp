// gclip_layer_backward.hpp -- the gradients of the norm and of the residual
// step for rows that fit into registers, and the join of the weights'
// gradients; instantiated for one storage format in each of
// gclip_layer_backward_*.hip.
#pragma once

#include "gclip_layer_device.hpp"

namespace gclip {

// With n = (x - mean) rstd and g = dy weight:
//   dx = rstd (g - sum(g) / size - n sum(g n) / size)
//   dweight = sum over rows of dy n, dbias = sum over rows of dy
// in one pass: a row's dy and x are read once, into the registers of LANES
// lanes, where the row's two sums and then dx are taken from them; the
// columns' sums stay in registers over all rows of the workgroup, whose rows
// meet in shared memory at the end, and each workgroup -- one for each compute
// unit -- leaves one part of them.  While a row is worked on, the loads of
// the workgroup's next one are under way.
//
// Bound by memory: 16384 x 2048 in bfloat16 takes 36.1 us, 5.6 TB/s of two
// reads and a write, and 4.6 us for the join of the parts (4 MB written and
// read); the residual step's with dropout 54.3 us, 6.2 TB/s; 8192 x 768 in
// binary32 13.9 us and 3.9.  Two workgroups a unit leave twice the parts: 22.6
// -> 26.7 us for the last in all, then.  Rows that share a wave (131071 x 64:
// 11.6 us, 4.3 TB/s) have vector instructions under way for 71 % of the time
// that a SIMD's four waves are there; the rest is the first load and the
// meeting at the end, with four rows' turns between them.
template <int DT, int LANES, int NV, int SURE, bool RES, bool DROP, bool STREAMED>
__global__ __launch_bounds__(bwd_threads(NV * kUnit<DT>)) void k_norm_rows_grad(BwdArgs a, DropArgs d) {
  constexpr uint32_t kBwdThreads = bwd_threads(NV * kUnit<DT>);
  constexpr uint32_t kRows = kBwdThreads / LANES;  // of a workgroup at a time
  constexpr uint32_t kCols = LANES * NV * kUnit<DT>;
  constexpr uint32_t kMeet = LANES < 64 ? kBwdThreads / 64 : kRows;  // sums of a column that meet
  __shared__ float red[2][2][kBwdThreads / 64];
  __shared__ float sums[kMeet > 1 ? kMeet * kCols : 1];
  const uint32_t lane = threadIdx.x % LANES;
  uint32_t slot = threadIdx.x / LANES;
  if constexpr (LANES >= 64) slot = __builtin_amdgcn_readfirstlane(slot);
  const uint32_t step = DROP ? drop_step(d) : 0u;

  u32x4 ny[NV], nx[NV], nh[NV];
  float nmean, nrstd;
  uint32_t base = blockIdx.x * kRows;
  const auto fetch = [&](uint32_t first) {
    // rows past the end are read as the last one; they count for nothing
    const uint32_t r = min(first + slot, a.rows - 1);
    const uint64_t dy = a.dy.at + r * a.dy.ld, x = a.x.at + r * a.x.ld, dh = a.dh.at + r * a.dh.ld;
    nmean = a.mean[r];
    nrstd = a.rstd[r];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      ny[k] = load_columns<DT, LANES, SURE, STREAMED>(dy, lane, k, a.size);
      nx[k] = load_columns<DT, LANES, SURE, STREAMED>(x, lane, k, a.size);
      if constexpr (RES)
        nh[k] = a.dh.at ? load_columns<DT, LANES, SURE, STREAMED>(dh, lane, k, a.size) : u32x4{0u, 0u, 0u, 0u};
    }
  };
  fetch(base);
  float w[NV][kUnit<DT>], dw[NV][kUnit<DT>], db[NV][kUnit<DT>];
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    weight_columns<DT, LANES, SURE>(a.weight, a.wdt, lane, k, a.size, 1.0f, w[k]);
#pragma unroll
    for (uint32_t j = 0; j < kUnit<DT>; ++j) dw[k][j] = db[k][j] = 0.0f;
  }
  const float count = (float)a.size, inverse = 1.0f / count;
  const bool full = a.size == kCols;
  uint32_t turn = 0;

  while (base < a.rows) {
    const uint32_t r = base + slot;
    const float rstd = nrstd, hm = r < a.rows ? 0.5f * nmean : 0.0f, tr = 2.0f * rstd;
    float g[NV][kUnit<DT>], n[NV][kUnit<DT>];
    u32x4 hh[NV];
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      settle<DT, LANES, SURE>(ny[k], lane, k, a.size, full);
      settle_round<DT, LANES, SURE>(nx[k], lane, k, a.size, full);
      if (r >= a.rows) ny[k] = nx[k] = u32x4{0u, 0u, 0u, 0u};
      unpack_unit<DT>(ny[k], g[k]);
      unpack_unit<DT>(nx[k], n[k]);
      if constexpr (RES) {
        settle<DT, LANES, SURE>(nh[k], lane, k, a.size, full);
        hh[k] = nh[k];
      }
      // past the row's end and the last row x is 0: n is too, from a mean of 0
      const float hk = k < SURE || column_of<DT>(lane, LANES, k) < a.size ? hm : 0.0f;
#pragma unroll
      for (uint32_t j = 0; j < kUnit<DT>; ++j) {
        n[k][j] = normed(n[k][j], hk, tr);
        dw[k][j] = __builtin_fmaf(g[k][j], n[k][j], dw[k][j]);
        db[k][j] += g[k][j];
        g[k][j] *= w[k][j];
        s1 += g[k][j];
        s2 = __builtin_fmaf(g[k][j], n[k][j], s2);
      }
    }
    const uint32_t next = base + gridDim.x * kRows;
    if (next < a.rows) fetch(next);
    // the next row's sums use the other words
    row_sums<LANES>(s1, s2, red[turn][0], red[turn][1]);
    turn ^= 1u;
    const float c1 = divided(s1, count, inverse), c2 = rstd * divided(s2, count, inverse);
    if (r < a.rows) {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
        const uint32_t c = column_of<DT>(lane, LANES, k);
        float v[kUnit<DT>];
#pragma unroll
        for (uint32_t j = 0; j < kUnit<DT>; ++j) v[j] = __builtin_fmaf(rstd, g[k][j] - c1, -(n[k][j] * c2));
        if constexpr (RES) {
          float q[kUnit<DT>];
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

  // this workgroup's part of the columns' sums: dweight, then dbias
  if (!a.dweight && !a.dbias) return;
#pragma unroll
  for (uint32_t which = 0; which < 2; ++which) {
    float(&v)[NV][kUnit<DT>] = which ? db : dw;
    if constexpr (kMeet > 1) {
      const uint32_t row = LANES < 64 ? threadIdx.x / 64 : slot;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (uint32_t j = 0; j < kUnit<DT>; ++j) {
          const float t = across_rows<LANES>(v[k][j]);
          if (LANES >= 64 || threadIdx.x % 64 < LANES) sums[row * kCols + column_of<DT>(lane, LANES, k) + j] = t;
        }
      }
      __syncthreads();
      for (uint32_t c = threadIdx.x; c < a.size; c += kBwdThreads) {
        float t = sums[c];
#pragma unroll
        for (uint32_t i = 1; i < kMeet; ++i) t += sums[i * kCols + c];
        if (a.parts == 1) store_weight_grad<DT>(a, which, c, t);
        else a.partials[((uint64_t)blockIdx.x * 2 + which) * a.size + c] = t;
      }
    } else {
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (uint32_t j = 0; j < kUnit<DT>; ++j) {
          const uint32_t c = column_of<DT>(lane, LANES, k) + j;
          if (c < a.size) {
            if (a.parts == 1) store_weight_grad<DT>(a, which, c, v[k][j]);
            else a.partials[((uint64_t)blockIdx.x * 2 + which) * a.size + c] = v[k][j];
          }
        }
      }
    }
  }
}

// The sum of the parts: a workgroup takes 64 columns, its sixteen waves share
// the parts, in a fixed order, all loads of a wave under way at once.  Bound
// by latency: 256 parts of 128 columns take 2.2 to 3.8 us, of 4096 columns 3.5
// to 4.6.
constexpr uint32_t kJoinThreads = 1024;
template <int DT>
__global__ __launch_bounds__(kJoinThreads) void k_join_weight_grads(BwdArgs a) {
  constexpr uint32_t kWavesOf = kJoinThreads / 64;
  __shared__ float red[kWavesOf][64];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const uint64_t i = workgroup_of_grid() * 64 + lane, width = 2ull * a.size;
  float t = 0.0f;
  if (i < width) {
#pragma unroll 16
    for (uint32_t p = wave; p < a.parts; p += kWavesOf) t += a.partials[p * width + i];
  }
  red[wave][lane] = t;
  __syncthreads();
  if (wave == 0 && i < width) {
#pragma unroll
    for (uint32_t k = 1; k < kWavesOf; ++k) t += red[k][lane];
    store_weight_grad<DT>(a, i >= a.size, (uint32_t)(i < a.size ? i : i - a.size), t);
  }
}

template <int DT>
hipError_t join_weight_grads(const BwdArgs& a, hipStream_t st) {
  hipLaunchKernelGGL((k_join_weight_grads<DT>), grid_of((2ull * a.size + 63) / 64), dim3(kJoinThreads), 0, st, a);
  return hipGetLastError();
}

template <int DT, int LANES, int NV, int SURE, bool STREAMED>
hipError_t backward_shape(BwdArgs a, bool residual, const DropArgs* drop, hipStream_t st) {
  a.parts = bwd_parts<DT>(a.rows, a.size);
  const dim3 grid(a.parts), block(bwd_threads(NV * kUnit<DT>));
  const DropArgs none{};
  if (!residual)
    hipLaunchKernelGGL((k_norm_rows_grad<DT, LANES, NV, SURE, false, false, STREAMED>), grid, block, 0, st, a, none);
  else if (!drop)
    hipLaunchKernelGGL((k_norm_rows_grad<DT, LANES, NV, SURE, true, false, STREAMED>), grid, block, 0, st, a, none);
  else
    hipLaunchKernelGGL((k_norm_rows_grad<DT, LANES, NV, SURE, true, true, STREAMED>), grid, block, 0, st, a, *drop);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.parts == 1 || (!a.dweight && !a.dbias)) return e;
  return join_weight_grads<DT>(a, st);
}

template <int DT, int I = 0>
hipError_t backward_of(int shape, const BwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if constexpr (I + 1 < (int)(sizeof(kBwdShapes<DT>) / sizeof(RowShape))) {
    if (shape != I) return backward_of<DT, I + 1>(shape, a, residual, drop, st);
  }
  constexpr RowShape s = kBwdShapes<DT>[I];
  return a.streamed ? backward_shape<DT, s.lanes, s.units, sure_units(kBwdShapes<DT>, I), true>(a, residual, drop, st)
                    : backward_shape<DT, s.lanes, s.units, sure_units(kBwdShapes<DT>, I), false>(a, residual, drop, st);
}

template <int DT, int I = 0>
hipError_t backward_few(int shape, const BwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if constexpr (I + 1 < (int)(sizeof(kFewBwdShapes) / sizeof(RowShape))) {
    if (shape != I) return backward_few<DT, I + 1>(shape, a, residual, drop, st);
  }
  static_assert((uint64_t)kFewBwdRows * kFewBwdMax * 2 * 5 <= kStreamBytes, "few rows are not streamed");
  constexpr RowShape s = kFewBwdShapes[I];
  return backward_shape<DT, s.lanes, s.units, sure_units(kFewBwdShapes, I), false>(a, residual, drop, st);
}

template <int DT>
hipError_t backward_rows(const BwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if constexpr (DT != GCLIP_F32) {
    if (few_bwd<DT>(a.rows, a.size))
      return backward_few<DT>(row_shape_of(kFewBwdShapes, kUnit<DT>, a.size), a, residual, drop, st);
  }
  return backward_of<DT>(row_shape_of(kBwdShapes<DT>, kUnit<DT>, a.size), a, residual, drop, st);
}

}  // namespace gclip
