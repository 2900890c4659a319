// gclip_activation.hpp -- the (gated) activation and its gradient;
// instantiated for one storage format in each of gclip_activation_*.hip.
#pragma once

#include "gclip_block_device.hpp"

namespace gclip {

constexpr int kActThreads = 256;

// e^x: of the 16-bit formats by the hardware's power of two alone, whose
// error (|x| 2^-24 of the result) is far below the format's step; in binary32
// with what the product with log2(e) loses put back, within 3 u.
template <int DT>
__device__ __forceinline__ float exponential(float x) {
  constexpr float kLog2e = 1.44269504088896f;
  if constexpr (DT == GCLIP_F32) {
    const float p = x * kLog2e;
    const float lost = __builtin_fmaf(x, 1.92596299e-8f, __builtin_fmaf(x, kLog2e, -p));
    // 0 and infinity are not corrected: an infinite p has lost everything
    return __builtin_amdgcn_exp2f(p) * (fabsf(p) < 300.0f ? __builtin_fmaf(lost, 0.693147180559945f, 1.0f) : 1.0f);
  } else {
    return __builtin_amdgcn_exp2f(x * kLog2e);
  }
}
// 1 / x of x >= 1; in binary32 with a step of Newton's, within 2 u (of an
// infinite x too).
template <int DT>
__device__ __forceinline__ float reciprocal(float x) {
  const float r = __builtin_amdgcn_rcpf(x);
  if constexpr (DT == GCLIP_F32) {
    const float d = fminf(x, 0x1.fffffep+127f);
    return __builtin_fmaf(__builtin_fmaf(-d, r, 1.0f), r, r);
  }
  return r;
}

// act(x) and, where wanted, its derivative.  With p = 1 / (1 + e^-x), 1 - p is
// taken from e^-x p where p is near 1.
template <int DT, int KIND, bool SLOPE>
__device__ __forceinline__ float activated(float x, float& slope) {
  if constexpr (KIND == GCLIP_ACT_RELU) {
    if (SLOPE) slope = x > 0.0f ? 1.0f : x != x ? x : 0.0f;
    return x < 0.0f ? 0.0f : x;
  } else if constexpr (KIND == GCLIP_ACT_SILU) {
    const float e = exponential<DT>(-x), p = reciprocal<DT>(1.0f + e);
    if (SLOPE) slope = p * __builtin_fmaf(x, x > 0.0f ? e * p : 1.0f - p, 1.0f);
    return x * p;
  } else if constexpr (KIND == GCLIP_ACT_GELU) {
    // h = erfc(z) / 2 of z = |x| / sqrt(2) as e^(-z^2) t P(t), t = 1 / (1 + 0.3 z):
    // P of degree 8 fitted to e^(z^2) erfc(z) / (2 t) for z up to 10, 3.5e-8 off
    // at most (0.6 u), relative.  The power serves the derivative too.  2047 x 1367 in
    // binary32, kept, 7.4 us, and 8.6 with the library's erfc and exponential.
    const float e = exponential<DT>(-0.5f * x * x), t = reciprocal<DT>(__builtin_fmaf(fabsf(x), 0.212132034355964f, 1.0f));
    float h = -0.06476137042f;
    h = __builtin_fmaf(h, t, 0.24278119206f);
    h = __builtin_fmaf(h, t, -0.25613820553f);
    h = __builtin_fmaf(h, t, 0.27385905385f);
    h = __builtin_fmaf(h, t, -0.04732470214f);
    h = __builtin_fmaf(h, t, 0.10746274889f);
    h = __builtin_fmaf(h, t, 0.07416965812f);
    h = __builtin_fmaf(h, t, 0.08535760641f);
    h = __builtin_fmaf(h, t, 0.08459400386f);
    h = e * t * h;
    const float c = x > 0.0f ? 1.0f - h : h;
    if (SLOPE) slope = __builtin_fmaf(x * 0.398942280401432678f, e, c);
    return x * c;
  } else {
    // (1 + tanh(u)) / 2 = 1 / (1 + e^-2u), u = sqrt(2 / pi) (x + 0.044715 x^3)
    const float xx = x * x, t = 1.59576912160573071f * x * __builtin_fmaf(xx, 0.044715f, 1.0f);  // 2 u
    const float e = exponential<DT>(-t), p = reciprocal<DT>(1.0f + e);
    if (SLOPE) {
      // beyond 16 the slope is 0 or 1, and the polynomial would leave binary32
      const float s = fminf(fmaxf(x, -16.0f), 16.0f), du = 1.59576912160573071f * __builtin_fmaf(s * s, 3.0f * 0.044715f, 1.0f);
      slope = p * __builtin_fmaf(s * du, x > 0.0f ? e * p : 1.0f - p, 1.0f);
    }
    return x * p;
  }
}

// y = act(gate) up, a unit of 16 bytes a lane; with KEEP the lanes of a block
// also share their scale and leave gate and up in 8 bits.  Bound by memory:
// 16384 x 5504 bfloat16 silu, gated and kept, 117 us, 727 MB at 6.2 TB/s.
template <int DT, int KIND, bool GATED, bool KEEP, bool STREAMED>
__global__ __launch_bounds__(kActThreads) void k_activation(ActArgs a, Split split) {
  constexpr uint32_t kU = kUnit<DT>;
  const uint64_t i = workgroup_of_grid() * kActThreads + threadIdx.x;
  const uint32_t r = row_of(i, split);
  if (r >= a.rows) return;  // whole blocks of lanes
  const uint32_t c = (uint32_t)(i - r * split.of) * kU;
  const bool in = c < a.size;
  if (!KEEP && !in) return;
  u32x4 g{0u, 0u, 0u, 0u}, u{0u, 0u, 0u, 0u};
  if (in) {
    g = load_unit_at<DT, STREAMED>(a.gate.at + r * a.gate.ld, c, a.size);
    if (GATED) u = load_unit_at<DT, STREAMED>(a.up.at + r * a.up.ld, c, a.size);
  }
  float x[kU], y[kU], b[kU], none;
  unpack_unit<DT>(g, x);
  unpack_unit<DT>(u, b);
#pragma unroll
  for (uint32_t j = 0; j < kU; ++j) {
    y[j] = activated<DT, KIND, false>(x[j], none);
    if (GATED) y[j] *= b[j];
  }
  if (in) store_unit<DT, true>(a.y.at + r * a.y.ld, c / kU, a.size, pack_unit<DT>(y));
  if constexpr (KEEP) {
    const bool first = threadIdx.x % kBlockLanes<DT> == 0;
    const float sg = block_scale<DT, kBlockLanes<DT>>(g);
    if (in) store_eight<DT, true>(a.gate8.at + r * a.gate8.ld, c, unit_eight<DT>(x, 1.0f / sg));
    if (in && first) store_scale(a.gate8, r, c / kBlock, sg);
    if constexpr (GATED) {
      const float su = block_scale<DT, kBlockLanes<DT>>(u);
      if (in) store_eight<DT, true>(a.up8.at + r * a.up8.ld, c, unit_eight<DT>(b, 1.0f / su));
      if (in && first) store_scale(a.up8, r, c / kBlock, su);
    }
  }
}

// dgate = dy up act'(gate), dup = dy act(gate), and y again where wanted.
// Bound by memory: 16384 x 5504 in bfloat16 from 8 bits, y too, 145 us, 907 MB
// at 6.3 TB/s.
template <int DT, int KIND, bool GATED, bool EIGHT, bool STREAMED>
__global__ __launch_bounds__(kActThreads) void k_activation_grad(ActArgs a, Split split) {
  constexpr uint32_t kU = kUnit<DT>;
  const uint64_t i = workgroup_of_grid() * kActThreads + threadIdx.x;
  const uint32_t r = row_of(i, split);
  if (r >= a.rows) return;
  const uint32_t c = (uint32_t)(i - r * split.of) * kU;
  float x[kU], b[kU], d[kU];
  const u32x4 dy = load_unit_at<DT, STREAMED>(a.dy.at + r * a.dy.ld, c, a.size);
  if constexpr (EIGHT) {
    const Unit8<DT> g = load_eight<DT, STREAMED>(a.gate8.at + r * a.gate8.ld, c);
    const float sg = load_scale(a.gate8, r, c);
    if constexpr (GATED) {
      const Unit8<DT> u = load_eight<DT, STREAMED>(a.up8.at + r * a.up8.ld, c);
      unit_value<DT>(u, load_scale(a.up8, r, c), b);
    }
    unit_value<DT>(g, sg, x);
  } else {
    const u32x4 g = load_unit_at<DT, STREAMED>(a.gate.at + r * a.gate.ld, c, a.size);
    if constexpr (GATED) unpack_unit<DT>(load_unit_at<DT, STREAMED>(a.up.at + r * a.up.ld, c, a.size), b);
    unpack_unit<DT>(g, x);
  }
  unpack_unit<DT>(dy, d);
  float y[kU], dg[kU], du[kU];
#pragma unroll
  for (uint32_t j = 0; j < kU; ++j) {
    float slope;
    y[j] = activated<DT, KIND, true>(x[j], slope);
    if constexpr (GATED) {
      dg[j] = d[j] * b[j] * slope;
      du[j] = d[j] * y[j];
      y[j] *= b[j];
    } else {
      dg[j] = d[j] * slope;
    }
  }
  store_unit<DT, true>(a.dgate.at + r * a.dgate.ld, c / kU, a.size, pack_unit<DT>(dg));
  if constexpr (GATED) store_unit<DT, true>(a.dup.at + r * a.dup.ld, c / kU, a.size, pack_unit<DT>(du));
  if (a.y.at) store_unit<DT, true>(a.y.at + r * a.y.ld, c / kU, a.size, pack_unit<DT>(y));
}

template <int DT, int KIND, bool GATED, bool STREAMED>
hipError_t activation_launch(const ActArgs& a, bool backward, hipStream_t st) {
  const bool keep = !backward && a.gate8.at, eight = backward && a.gate8.at;
  // lanes of a row: its units, or whole blocks where lanes share a scale
  const uint64_t of = keep ? (uint64_t)a.gate8.count * kBlockLanes<DT> : (a.size - 1) / kUnit<DT> + 1;
  const Split split{of, 1.0 / (double)of};
  const dim3 grid = grid_of((of * a.rows + kActThreads - 1) / kActThreads), block(kActThreads);
  if (keep) hipLaunchKernelGGL((k_activation<DT, KIND, GATED, true, STREAMED>), grid, block, 0, st, a, split);
  else if (!backward) hipLaunchKernelGGL((k_activation<DT, KIND, GATED, false, STREAMED>), grid, block, 0, st, a, split);
  else if (eight) hipLaunchKernelGGL((k_activation_grad<DT, KIND, GATED, true, STREAMED>), grid, block, 0, st, a, split);
  else hipLaunchKernelGGL((k_activation_grad<DT, KIND, GATED, false, STREAMED>), grid, block, 0, st, a, split);
  return hipGetLastError();
}

template <int DT, int KIND>
hipError_t activation_kind(const ActArgs& a, bool backward, bool streamed, hipStream_t st) {
  const bool gated = a.up.at || a.up8.at;
  if (gated) return streamed ? activation_launch<DT, KIND, true, true>(a, backward, st)
                             : activation_launch<DT, KIND, true, false>(a, backward, st);
  return streamed ? activation_launch<DT, KIND, false, true>(a, backward, st)
                  : activation_launch<DT, KIND, false, false>(a, backward, st);
}

template <int DT>
hipError_t activation_of(const ActArgs& a, int32_t kind, bool backward, bool streamed, hipStream_t st) {
  switch (kind) {
    case GCLIP_ACT_SILU: return activation_kind<DT, GCLIP_ACT_SILU>(a, backward, streamed, st);
    case GCLIP_ACT_GELU: return activation_kind<DT, GCLIP_ACT_GELU>(a, backward, streamed, st);
    case GCLIP_ACT_GELU_TANH: return activation_kind<DT, GCLIP_ACT_GELU_TANH>(a, backward, streamed, st);
    default: return activation_kind<DT, GCLIP_ACT_RELU>(a, backward, streamed, st);
  }
}

}  // namespace gclip
