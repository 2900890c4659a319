// gclip_rms_forward.hpp -- RMS norm and its residual step for rows that fit
// into registers; instantiated for one storage format, without or with
// matrices in 8 bits, in each of gclip_rms_forward_*.hip.
#pragma once

#include "gclip_block_device.hpp"

namespace gclip {

// Threads of a workgroup: rows of up to a wave share four waves, longer ones
// have a workgroup each.
template <int LANES>
constexpr int kRmsThreads = LANES > 64 ? LANES : 256;

// Workgroups of four waves for each compute unit, by the columns that a lane
// holds: as many as its registers let run at once, which take the other rows
// in turn with their weight kept.
constexpr uint32_t rms_workgroups(uint32_t columns) { return columns <= 8 ? 8 : columns <= 24 ? 4 : 2; }

// Few rows take shapes of more lanes each, while these are no more than all
// compute units hold at once (1024 each): 396 x 4608 bfloat16 residual steps
// with dropout 5.5 us by 256 lanes and 6.3 by 1024, 1021 x 1111 in 8 bits too
// 6.2 us by 256 and 6.5 by 64, 900 x 2048 norms 4.7 by 256 and 4.9 by 64.
constexpr uint32_t kFewLanes = 1u << 18;

// Sum and largest of a row's LANES lanes behind one barrier; rows of more
// than a wave meet in redp and redq, a word for each wave of their workgroup.
template <int LANES>
__device__ __forceinline__ void row_sum_max(float& s, uint32_t& m, float* redp, uint32_t* redq) {
  s = lanes_sum<(LANES < 64 ? LANES : 64)>(s);
  m = lanes_max<(LANES < 64 ? LANES : 64)>(m);
  if constexpr (LANES > 64) {
    const uint32_t wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) {
      redp[wave] = s;
      redq[wave] = m;
    }
    __syncthreads();
    s = waves_sum<LANES>(redp);
    m = redq[0];
#pragma unroll
    for (int i = 1; i < LANES / 64; ++i) m = max(m, redq[i]);
  }
}

// A row's checkpoint, from its stored elements (zeros past the end).  A block
// is an aligned run of lanes of one unit, or several units of rows whose lanes
// hold less than a block.
template <int DT, int LANES, int NV, bool NT>
__device__ __forceinline__ void keep_row(const Eight& e, uint64_t r, uint32_t lane, uint32_t size, const u32x4 (&q)[NV]) {
  constexpr int kRun = LANES < kBlockLanes<DT> ? LANES : kBlockLanes<DT>;
  constexpr int kUnits = LANES < kBlockLanes<DT> ? kBlockLanes<DT> / LANES : 1;  // of a block
#pragma unroll
  for (int k = 0; k < NV; k += kUnits) {
    uint32_t m = 0, f = 0;
#pragma unroll
    for (int i = k; i < k + kUnits && i < NV; ++i) m = max(m, unit_magnitude<DT>(q[i]));
    m = lanes_max<kRun>(m);
    if (m >= kInfBits<DT>) {  // the run's lanes together
#pragma unroll
      for (int i = k; i < k + kUnits && i < NV; ++i) f = max(f, unit_magnitude_finite<DT>(q[i]));
      m = lanes_max<kRun>(f);
    }
    const float scale = scale_of(elem_float<DT>(m)), inverse = 1.0f / scale;
#pragma unroll
    for (int i = k; i < k + kUnits && i < NV; ++i) {
      const uint32_t c = column_of<DT>(lane, LANES, i);
      float v[kUnit<DT>];
      unpack_unit<DT>(q[i], v);
      if (c < size) store_eight<DT, NT>(e.at + r * e.ld, c, unit_eight<DT>(v, inverse));
      if (c < size && i == k && lane % kRun == 0) store_scale(e, r, c / kBlock, scale);
    }
  }
}

// The largest magnitude's bits among values in binary32; finite: of those.
template <uint32_t N>
__device__ __forceinline__ uint32_t largest(const float (&v)[N], bool finite) {
  uint32_t m = 0;
#pragma unroll
  for (uint32_t j = 0; j < N; ++j) {
    const uint32_t b = __float_as_uint(v[j]) & 0x7fffffffu;
    m = max(m, finite && b >= 0x7f800000u ? 0u : b);
  }
  return m;
}

// y = x rstd weight, rstd = 1 / sqrt(sum(x^2) / size + eps), in one pass: a
// row's elements are read once, into the registers of LANES lanes, where the
// sum and y are taken from them.  While a row is worked on, the loads of the
// workgroup's next one are under way; the weight stays in registers.
// Bound by memory: 8192 x 768 binary32 residual steps with dropout and a
// checkpoint 17.5 us, 107 MB at 6.1 TB/s, which a copy of so much reaches 5.6
// of; one token of 2048 columns 2.4 us, of which all but 0.1 are a launch and
// two ways to memory and back.
//
// y in 8 bits with a scale a row: the largest |x weight| comes with the sum
// of squares, behind the same barrier, and is the largest |y| but for rstd.
template <int DT, int LANES, int NV, int SURE, bool RES, bool DROP, bool EIGHT, bool STREAMED>
__global__ __launch_bounds__((kRmsThreads<LANES>)) void k_rms_rows(RmsFwdArgs a, DropArgs d) {
  constexpr int kThreads = kRmsThreads<LANES>;
  const uint32_t at_once = LANES > 64 ? 1u : blockDim.x / LANES;  // rows of a workgroup
  __shared__ float reds[2][kThreads / 64];
  __shared__ uint32_t redm[2][kThreads / 64];
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
  float w[NV][kUnit<DT>];
#pragma unroll
  for (int k = 0; k < NV; ++k) weight_columns<DT, LANES, SURE>(a.weight, a.wdt, lane, k, a.size, 1.0f, w[k]);
  const float inverse = 1.0f / (float)a.size;
  const bool full = a.size == LANES * NV * kUnit<DT>;
  const bool by_row = EIGHT && a.y8.at && a.y8.row;
  uint32_t turn = 0;  // a barrier lies between two uses of the same words

  while (base < a.rows) {
    const uint32_t r = base + slot;
    float v[NV][kUnit<DT>];
    u32x4 o[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const uint32_t c = column_of<DT>(lane, LANES, k);
      settle<DT, LANES, SURE>(nx[k], lane, k, a.size, full);
      unpack_unit<DT>(nx[k], v[k]);
      o[k] = nx[k];
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
    if (r < a.rows) {
      if constexpr (RES) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
          store_columns<DT, LANES, SURE, !STREAMED>(a.h.at + r * a.h.ld, lane, k, a.size, o[k]);
      }
      if constexpr (EIGHT) {
        if (a.kept.at) keep_row<DT, LANES, NV, !STREAMED>(a.kept, r, lane, a.size, o);
      }
    }

    // the squares; rows whose sum of them leaves binary32 go through this
    // again, scaled by a power of two (so does a row with a NaN or an
    // infinity, to no effect).  Rows that share a wave go together.
    float ms, up = 1.0f;  // up: the power of two, undone
    uint32_t most;
    for (bool first = true;; first = false) {
      float s = 0.0f;
      most = 0;
#pragma unroll
      for (int k = 0; k < NV; ++k) {
#pragma unroll
        for (uint32_t j = 0; j < kUnit<DT>; ++j) s = __builtin_fmaf(v[k][j], v[k][j], s);
        if constexpr (EIGHT) {
          if (by_row) {
            float t[kUnit<DT>];
#pragma unroll
            for (uint32_t j = 0; j < kUnit<DT>; ++j) t[j] = v[k][j] * w[k][j];
            most = max(most, largest<kUnit<DT>>(t, false));
          }
        }
      }
      if constexpr (EIGHT) row_sum_max<LANES>(s, most, reds[turn], redm[turn]);
      else s = row_sum<LANES>(s, reds[turn]);
      turn ^= 1u;
      ms = s * inverse;  // an infinite sum stays one
      const bool leaves = !(ms + a.eps <= 0x1.fffffep+127f);
      if (!first || !(LANES > 64 ? __builtin_amdgcn_readfirstlane(leaves) : __any(leaves))) break;
      if (leaves) {
        up = 0x1p+96f;
#pragma unroll
        for (int k = 0; k < NV; ++k)
#pragma unroll
          for (uint32_t j = 0; j < kUnit<DT>; ++j) v[k][j] *= 0x1p-96f;
      }
    }
    const float rstd = 1.0f / sqrtf(ms + (up == 1.0f ? a.eps : a.eps * 0x1p-96f * 0x1p-96f));
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (uint32_t j = 0; j < kUnit<DT>; ++j) v[k][j] = v[k][j] * rstd * w[k][j];

    if constexpr (EIGHT) {
      if (by_row) {
        float top = __uint_as_float(most) * rstd;
        // products that leave binary32 although y does not, or are so small
        // that they have lost bits: y's own largest, for the row's lanes together
        if (!(most >= 0x21800000u && top <= 0x1.fffffep+127f)) {  // 2^-60
          most = 0;
#pragma unroll
          for (int k = 0; k < NV; ++k) most = max(most, largest<kUnit<DT>>(v[k], true));
          float none = 0.0f;
          row_sum_max<LANES>(none, most, reds[turn], redm[turn]);
          turn ^= 1u;
          top = __uint_as_float(most);
        }
        const float scale = scale_of(top), factor = 1.0f / scale;
        if (r < a.rows) {
#pragma unroll
          for (int k = 0; k < NV; ++k) {
            const uint32_t c = column_of<DT>(lane, LANES, k);
            if (k < SURE || c < a.size)
              store_eight<DT, !STREAMED>(a.y8.at + r * a.y8.ld, c, unit_eight<DT>(v[k], factor));
          }
          if (lane == 0) store_scale(a.y8, r, 0, scale);
        }
      } else if (a.y8.at && r < a.rows) {
        constexpr int kRun = LANES < kBlockLanes<DT> ? LANES : kBlockLanes<DT>;
        constexpr int kUnits = LANES < kBlockLanes<DT> ? kBlockLanes<DT> / LANES : 1;  // see keep_row()
#pragma unroll
        for (int k = 0; k < NV; k += kUnits) {
          uint32_t m = 0;
#pragma unroll
          for (int i = k; i < k + kUnits && i < NV; ++i) m = max(m, largest<kUnit<DT>>(v[i], false));
          m = lanes_max<kRun>(m);
          if (m >= 0x7f800000u) {
            m = 0;
#pragma unroll
            for (int i = k; i < k + kUnits && i < NV; ++i) m = max(m, largest<kUnit<DT>>(v[i], true));
            m = lanes_max<kRun>(m);
          }
          const float scale = scale_of(__uint_as_float(m)), factor = 1.0f / scale;
#pragma unroll
          for (int i = k; i < k + kUnits && i < NV; ++i) {
            const uint32_t c = column_of<DT>(lane, LANES, i);
            if (c >= a.size) continue;
            store_eight<DT, !STREAMED>(a.y8.at + r * a.y8.ld, c, unit_eight<DT>(v[i], factor));
            if (i == k && lane % kRun == 0) store_scale(a.y8, r, c / kBlock, scale);
          }
        }
      }
    }
    if (r < a.rows) {
      if (!EIGHT || !a.y8.at) {
#pragma unroll
        for (int k = 0; k < NV; ++k)
          store_columns<DT, LANES, SURE, !STREAMED>(a.y.at + r * a.y.ld, lane, k, a.size, pack_unit<DT>(v[k]));
      }
      if (a.rstd && lane == 0) a.rstd[r] = up == 1.0f ? rstd : rstd * 0x1p-96f;
    }
    base = next;
  }
}

template <int DT, bool EIGHT, int LANES, int NV, int SURE, bool STREAMED>
hipError_t rms_forward_shape(const RmsFwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  // workgroups of a wave until there are four for each compute unit
  const uint32_t threads = LANES <= 64 && a.rows < 1024 * (64 / LANES) ? 64 : kRmsThreads<LANES>;
  const uint32_t at_once = threads / LANES;
  const uint32_t most = 256u * rms_workgroups(NV * kUnit<DT>) * 256 / threads;
  const uint32_t need = (a.rows - 1) / at_once + 1;
  const dim3 grid(need < most ? need : most), block(threads);
  if (!residual)
    hipLaunchKernelGGL((k_rms_rows<DT, LANES, NV, SURE, false, false, EIGHT, STREAMED>), grid, block, 0, st, a, DropArgs{});
  else if (!drop)
    hipLaunchKernelGGL((k_rms_rows<DT, LANES, NV, SURE, true, false, EIGHT, STREAMED>), grid, block, 0, st, a, DropArgs{});
  else
    hipLaunchKernelGGL((k_rms_rows<DT, LANES, NV, SURE, true, true, EIGHT, STREAMED>), grid, block, 0, st, a, *drop);
  return hipGetLastError();
}

template <int DT, bool EIGHT, int I = 0>
hipError_t rms_forward_of(int shape, const RmsFwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if constexpr (I + 1 < (int)(sizeof(kFwdShapes<DT>) / sizeof(RowShape))) {
    if (shape != I) return rms_forward_of<DT, EIGHT, I + 1>(shape, a, residual, drop, st);
  }
  constexpr RowShape s = kFwdShapes<DT>[I];
  constexpr int sure = sure_units(kFwdShapes<DT>, I);
  return a.streamed ? rms_forward_shape<DT, EIGHT, s.lanes, s.units, sure, true>(a, residual, drop, st)
                    : rms_forward_shape<DT, EIGHT, s.lanes, s.units, sure, false>(a, residual, drop, st);
}

template <int DT, bool EIGHT, int I = 0>
hipError_t rms_forward_few(int shape, const RmsFwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if constexpr (I + 1 < (int)(sizeof(kFewShapes<DT>) / sizeof(RowShape))) {
    if (shape != I) return rms_forward_few<DT, EIGHT, I + 1>(shape, a, residual, drop, st);
  }
  constexpr RowShape s = kFewShapes<DT>[I];
  return rms_forward_shape<DT, EIGHT, s.lanes, s.units, sure_units(kFewShapes<DT>, I), false>(a, residual, drop, st);
}

template <int DT, bool EIGHT>
hipError_t rms_forward_rows(const RmsFwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  const int few = row_shape_of(kFewShapes<DT>, kUnit<DT>, a.size);
  if ((uint64_t)a.rows * kFewShapes<DT>[few].lanes <= kFewLanes) return rms_forward_few<DT, EIGHT>(few, a, residual, drop, st);
  return rms_forward_of<DT, EIGHT>(row_shape_of(kFwdShapes<DT>, kUnit<DT>, a.size), a, residual, drop, st);
}

}  // namespace gclip
