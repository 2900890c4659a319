// gclip_layer_any.hip -- the layer calls for rows of any length: a workgroup
// goes through a row in passes, and through the caches again in each.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gclip_layer_device.hpp"

namespace gclip {
namespace {

constexpr int kAnyThreads = 256;
constexpr int kAnyWaves = kAnyThreads / 64;

// Sum over the workgroup, the same bits in every thread.
__device__ __forceinline__ double any_sum(double v, double* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  __syncthreads();  // red may still be read by a previous call
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = red[0];
#pragma unroll
  for (int i = 1; i < kAnyWaves; ++i) t += red[i];
  return t;
}

// Three passes over a row: h and the sum, the squares, y.  A thread reads in
// a later pass only the groups that it wrote itself.  The sums are binary64,
// so no finite row overflows them.
template <int DT, bool RES, bool DROP>
__global__ __launch_bounds__(kAnyThreads) void k_norm_any(FwdArgs a, DropArgs d) {
  __shared__ double red[kAnyWaves];
  const uint32_t groups = (a.size + kGroup - 1) / kGroup;
  const uint32_t step = DROP ? drop_step(d) : 0u;
  for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const uint64_t x = a.x.at + r * a.x.ld, y = a.y.at + r * a.y.ld;
    const uint64_t h = RES ? a.h.at + r * a.h.ld : x;
    double s = 0.0;
    for (uint32_t g = threadIdx.x; g < groups; g += kAnyThreads) {
      float v[8];
      unpack<DT>(load_group8<DT, false>(x, g, a.size), v);
      if constexpr (RES) {
        float q[8];
        if constexpr (DROP) drop_group(d, step, r, g, v);
        unpack<DT>(load_group8<DT, false>(a.residual.at + r * a.residual.ld, g, a.size), q);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += q[k];
        const Raw8<DT> o = pack<DT>(v);
        store_group8<DT, false>(h, g, a.size, o);
        unpack<DT>(o, v);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) s += g * kGroup + k < a.size ? (double)v[k] : 0.0;
    }
    const double mean = any_sum(s, red) / (double)a.size;
    double ss = 0.0;
    for (uint32_t g = threadIdx.x; g < groups; g += kAnyThreads) {
      float v[8];
      unpack<DT>(load_group8<DT, false>(h, g, a.size), v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double t = (double)v[k] - mean;
        ss += g * kGroup + k < a.size ? t * t : 0.0;
      }
    }
    const float rstd = (float)(1.0 / sqrt(any_sum(ss, red) / (double)a.size + (double)a.eps));
    const float m = (float)mean;
    for (uint32_t g = threadIdx.x; g < groups; g += kAnyThreads) {
      float v[8], w[8], b[8];
      unpack<DT>(load_group8<DT, false>(h, g, a.size), v);
      weight_group<DT>(a.weight, a.wdt, g, a.size, 1.0f, w);
      weight_group<DT>(a.bias, a.wdt, g, a.size, 0.0f, b);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = (v[k] - m) * rstd * w[k] + b[k];
      store_group8<DT, false>(y, g, a.size, pack<DT>(v));
    }
    if (a.mean && threadIdx.x == 0) {
      a.mean[r] = m;
      a.rstd[r] = rstd;
    }
  }
}

// The rows' gradients: a pass for the two sums, a pass for the result.
template <int DT, bool DROP>
__global__ __launch_bounds__(kAnyThreads) void k_norm_rows_grad_any(BwdArgs a, DropArgs d) {
  __shared__ double red[kAnyWaves];
  const uint32_t groups = (a.size + kGroup - 1) / kGroup;
  const uint32_t step = DROP ? drop_step(d) : 0u;
  for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const uint64_t dy = a.dy.at + r * a.dy.ld, x = a.x.at + r * a.x.ld;
    const float mean = a.mean[r], rstd = a.rstd[r];
    double s1 = 0.0, s2 = 0.0;
    for (uint32_t g = threadIdx.x; g < groups; g += kAnyThreads) {
      float u[8], v[8], w[8];
      unpack<DT>(load_group8<DT, false>(dy, g, a.size), u);
      unpack<DT>(load_group8<DT, false>(x, g, a.size), v);
      weight_group<DT>(a.weight, a.wdt, g, a.size, 1.0f, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        if (g * kGroup + k < a.size) {
          const float t = u[k] * w[k];
          s1 += (double)t;
          s2 += (double)(t * ((v[k] - mean) * rstd));
        }
      }
    }
    const float c1 = (float)(any_sum(s1, red) / (double)a.size);
    const float c2 = (float)(any_sum(s2, red) / (double)a.size);
    for (uint32_t g = threadIdx.x; g < groups; g += kAnyThreads) {
      float u[8], v[8], w[8];
      unpack<DT>(load_group8<DT, false>(dy, g, a.size), u);
      unpack<DT>(load_group8<DT, false>(x, g, a.size), v);
      weight_group<DT>(a.weight, a.wdt, g, a.size, 1.0f, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = rstd * (u[k] * w[k] - c1 - (v[k] - mean) * rstd * c2);
      if (a.dh.at) {
        unpack<DT>(load_group8<DT, false>(a.dh.at + r * a.dh.ld, g, a.size), u);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += u[k];
      }
      store_group8<DT, false>(a.dres.at + r * a.dres.ld, g, a.size, pack<DT>(v));
      if constexpr (DROP) {
        drop_group(d, step, r, g, v);
        store_group8<DT, false>(a.dx.at + r * a.dx.ld, g, a.size, pack<DT>(v));
      }
    }
  }
}

// Part p of the weights' gradients: the rows r with r mod parts == p, in a
// fixed order.  A wave takes 64 groups of columns, the workgroup's waves
// share the part's rows.
template <int DT>
__global__ __launch_bounds__(kAnyThreads) void k_norm_cols_grad_any(BwdArgs a) {
  __shared__ float red[kAnyWaves][64][17];
  const uint32_t lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = blockIdx.x * 64 + lane;
  float dw[8] = {}, db[8] = {};
  if (g * kGroup < a.size) {
    for (uint64_t r = blockIdx.y + (uint64_t)wave * a.parts; r < a.rows; r += (uint64_t)kAnyWaves * a.parts) {
      float u[8], v[8];
      unpack<DT>(load_group8<DT, false>(a.dy.at + r * a.dy.ld, g, a.size), u);
      unpack<DT>(load_group8<DT, false>(a.x.at + r * a.x.ld, g, a.size), v);
      const float mean = a.mean[r], rstd = a.rstd[r];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        dw[k] += u[k] * ((v[k] - mean) * rstd);
        db[k] += u[k];
      }
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    red[wave][lane][k] = dw[k];
    red[wave][lane][8 + k] = db[k];
  }
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < 64 * 16; i += kAnyThreads) {
    const uint32_t which = i / 512, l = (i % 512) / 8, k = i % 8, c = (blockIdx.x * 64 + l) * kGroup + k;
    float t = red[0][l][8 * which + k];
#pragma unroll
    for (int w = 1; w < kAnyWaves; ++w) t += red[w][l][8 * which + k];
    if (c < a.size) a.partials[((uint64_t)blockIdx.y * 2 + which) * a.size + c] = t;
  }
}

// A lane takes a unit of 16 bytes.  A unit of a 16-bit format is a group; of
// binary32 half of one, whose two lanes run the generator both: a wave's
// accesses are adjacent then, and there is twice the time for it.  Bound by
// memory, with the generator's products (20 for eight elements, at a quarter
// of the full rate) close behind in 16 bits: 1.3B's 16384 x 2048 in bfloat16
// takes 23.5 us (two units a lane: 24.1), 5.7 TB/s.
template <int DT, bool STREAMED>
__global__ __launch_bounds__(kAnyThreads) void k_dropout(Rows x, Rows y, uint32_t rows, uint32_t size, DropArgs d) {
  const uint32_t units = (size + kUnit<DT> - 1) / kUnit<DT>;
  const uint64_t i = (uint64_t)blockIdx.x * kAnyThreads + threadIdx.x;
  const uint64_t row = i / units;
  if (row >= rows) return;
  const uint32_t r = (uint32_t)row, u = (uint32_t)(i % units);
  float v[kUnit<DT>];
  unpack_unit<DT>(load_unit<DT, STREAMED>(x.at + r * x.ld, u, size), v);
  drop_unit<DT>(d, drop_step(d), r, u * kUnit<DT>, v);
  store_unit<DT, true>(y.at + r * y.ld, u, size, pack_unit<DT>(v));
}

template <int DT>
hipError_t forward_any(const FwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  const dim3 grid(std::min<uint32_t>(a.rows, 1u << 20)), block(kAnyThreads);
  if (!residual) hipLaunchKernelGGL((k_norm_any<DT, false, false>), grid, block, 0, st, a, DropArgs{});
  else if (!drop) hipLaunchKernelGGL((k_norm_any<DT, true, false>), grid, block, 0, st, a, DropArgs{});
  else hipLaunchKernelGGL((k_norm_any<DT, true, true>), grid, block, 0, st, a, *drop);
  return hipGetLastError();
}

// The weights' gradients first: dx may be written over dy or x.
template <int DT>
hipError_t backward_any(const BwdArgs& a, const DropArgs* drop, hipStream_t st) {
  const dim3 block(kAnyThreads);
  const uint32_t groups = (a.size + kGroup - 1) / kGroup;
  if (a.dweight || a.dbias) {
    hipLaunchKernelGGL((k_norm_cols_grad_any<DT>), dim3((groups + 63) / 64, a.parts), block, 0, st, a);
    const hipError_t e = join_weight_grads<DT>(a, st);
    if (e != hipSuccess) return e;
  }
  if (a.rows > 0) {
    const dim3 grid(std::min<uint32_t>(a.rows, 1u << 20));
    if (drop) hipLaunchKernelGGL((k_norm_rows_grad_any<DT, true>), grid, block, 0, st, a, *drop);
    else hipLaunchKernelGGL((k_norm_rows_grad_any<DT, false>), grid, block, 0, st, a, DropArgs{});
  }
  return hipGetLastError();
}

template <int DT>
hipError_t dropout(const Rows& x, const Rows& y, uint32_t rows, uint32_t size, const DropArgs& d, hipStream_t st) {
  const uint64_t total = (uint64_t)rows * ((size + kUnit<DT> - 1) / kUnit<DT>);
  const dim3 grid((uint32_t)((total + kAnyThreads - 1) / kAnyThreads)), block(kAnyThreads);
  if (total * 32 > kStreamBytes) hipLaunchKernelGGL((k_dropout<DT, true>), grid, block, 0, st, x, y, rows, size, d);
  else hipLaunchKernelGGL((k_dropout<DT, false>), grid, block, 0, st, x, y, rows, size, d);
  return hipGetLastError();
}

}  // namespace

// A part for each workgroup of the kernel with rows in registers.  Else as
// many as leave each at least 16 rows, at most 256, and at most 64 MiB of
// them for long rows.
uint32_t layer_parts(int64_t rows, int64_t size) {
  if (rows > 0 && in_registers((uint32_t)size)) {
    const uint32_t n = (uint32_t)rows;
    return std::max(bwd_parts<GCLIP_F32>(n, (uint32_t)size), bwd_parts<GCLIP_BF16>(n, (uint32_t)size));
  }
  const int64_t by_rows = std::max<int64_t>(1, (rows + 15) / 16);
  const int64_t by_bytes = std::max<int64_t>(1, (64ll << 20) / (8 * size));
  return (uint32_t)std::min<int64_t>({by_rows, by_bytes, 256});
}

hipError_t launch_layer_forward(const FwdArgs& a, int32_t dtype, bool residual, const DropArgs* drop, hipStream_t st) {
  const bool regs = in_registers(a.size);
  switch (dtype) {
    case GCLIP_F32:
      return regs ? forward_rows<GCLIP_F32>(a, residual, drop, st) : forward_any<GCLIP_F32>(a, residual, drop, st);
    case GCLIP_F16:
      return regs ? forward_rows<GCLIP_F16>(a, residual, drop, st) : forward_any<GCLIP_F16>(a, residual, drop, st);
    default:
      return regs ? forward_rows<GCLIP_BF16>(a, residual, drop, st) : forward_any<GCLIP_BF16>(a, residual, drop, st);
  }
}

hipError_t launch_layer_backward(const BwdArgs& a, int32_t dtype, bool residual, const DropArgs* drop, hipStream_t st) {
  const bool regs = a.rows > 0 && in_registers(a.size);
  switch (dtype) {
    case GCLIP_F32:
      return regs ? backward_rows<GCLIP_F32>(a, residual, drop, st) : backward_any<GCLIP_F32>(a, drop, st);
    case GCLIP_F16:
      return regs ? backward_rows<GCLIP_F16>(a, residual, drop, st) : backward_any<GCLIP_F16>(a, drop, st);
    default:
      return regs ? backward_rows<GCLIP_BF16>(a, residual, drop, st) : backward_any<GCLIP_BF16>(a, drop, st);
  }
}

hipError_t launch_dropout(const Rows& x, const Rows& y, uint32_t rows, uint32_t size, int32_t dtype, const DropArgs& d,
                          hipStream_t st) {
  switch (dtype) {
    case GCLIP_F32: return dropout<GCLIP_F32>(x, y, rows, size, d, st);
    case GCLIP_F16: return dropout<GCLIP_F16>(x, y, rows, size, d, st);
    default: return dropout<GCLIP_BF16>(x, y, rows, size, d, st);
  }
}

}  // namespace gclip
