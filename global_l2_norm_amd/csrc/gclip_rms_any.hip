// gclip_rms_any.hip -- the RMS norm of rows that the kernels with rows in
// registers do not take, shorter and longer ones.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gclip_block_device.hpp"

namespace gclip {
namespace {

constexpr int kShortThreads = 256;
constexpr int kLongThreads = 512;
constexpr int kLongWaves = kLongThreads / 64;

// Sum over the workgroup, the same bits in every thread.
__device__ __forceinline__ double workgroup_sum(double v, double* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  __syncthreads();  // red may still be read by a previous call
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = red[0];
#pragma unroll
  for (int i = 1; i < kLongWaves; ++i) t += red[i];
  return t;
}

__device__ __forceinline__ uint32_t workgroup_max(uint32_t v, uint32_t* red) {
  v = lanes_max<64>(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int i = 1; i < kLongWaves; ++i) v = max(v, red[i]);
  return v;
}

__device__ __forceinline__ uint32_t largest_finite(const float (&v)[8]) {
  uint32_t m = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t b = __float_as_uint(v[k]) & 0x7fffffffu;
    m = max(m, b < 0x7f800000u ? b : 0u);
  }
  return m;
}

// A group of eight values in 8 bits at column c of a row.
__device__ __forceinline__ void store_eight_group(const Eight& e, uint64_t r, uint32_t c, const float (&v)[8],
                                                  float scale) {
  store_eight<GCLIP_BF16, false>(e.at + r * e.ld, c, unit_eight<GCLIP_BF16>(v, 1.0f / scale));
}

// The same with the scale of its block, which sixteen lanes hold together.
__device__ __forceinline__ void store_eight_block(const Eight& e, uint64_t r, uint32_t c, uint32_t size,
                                                  const float (&v)[8]) {
  const float scale = scale_of(__uint_as_float(lanes_max<16>(largest_finite(v))));
  if (c >= size) return;
  store_eight_group(e, r, c, v, scale);
  if (c % kBlock == 0) store_scale(e, r, c / kBlock, scale);
}

// Two passes over a row, h and the squares, then y, which finds the row in the
// caches; y in 8 bits with a scale a row takes one more between them.  A
// thread reads there only the groups that it wrote itself.  The sums are
// binary64, so no finite row overflows them.  Bound by the passes' latency:
// 1000 x 40000 residual steps in bfloat16 77 us, 320 MB at 4.2 TB/s.
template <int DT, bool RES, bool DROP>
__global__ __launch_bounds__(kLongThreads) void k_rms_long(RmsFwdArgs a, DropArgs d) {
  __shared__ double red[kLongWaves];
  __shared__ uint32_t redm[kLongWaves];
  // whole blocks of lanes take part in a block's largest
  const uint32_t groups = (a.size + kGroup - 1) / kGroup, turns = (groups + 15) / 16 * 16;
  const uint32_t step = DROP ? drop_step(d) : 0u;
  for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const uint64_t x = a.x.at + r * a.x.ld, y = a.y.at + r * a.y.ld;
    const uint64_t h = RES ? a.h.at + r * a.h.ld : x;
    double s = 0.0;
    for (uint32_t g = threadIdx.x; g < turns; g += kLongThreads) {
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
      for (int k = 0; k < 8; ++k) {
        if (g * kGroup + k >= a.size) v[k] = 0.0f;
        s = __builtin_fma((double)v[k], (double)v[k], s);
      }
      if (a.kept.at) store_eight_block(a.kept, r, g * kGroup, a.size, v);
    }
    const double rs = 1.0 / sqrt(workgroup_sum(s, red) / (double)a.size + (double)a.eps);
    const float rstd = (float)rs;
    // rows of the largest elements: rstd alone would lose bits below binary32
    const float low = rs < 0x1p-100 ? 0x1p-96f : 1.0f, high = (float)(rs / (double)low);
    const auto normed_group = [&](uint32_t g, float(&v)[8]) {
      float w[8];
      unpack<DT>(load_group8<DT, false>(h, g, a.size), v);
      weight_group<DT>(a.weight, a.wdt, g, a.size, 1.0f, w);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = g * kGroup + k < a.size ? v[k] * low * high * w[k] : 0.0f;
    };
    float row_scale = 1.0f;
    if (a.y8.at && a.y8.row) {
      uint32_t most = 0;
      for (uint32_t g = threadIdx.x; g < groups; g += kLongThreads) {
        float v[8];
        normed_group(g, v);
        most = max(most, largest_finite(v));
      }
      row_scale = scale_of(__uint_as_float(workgroup_max(most, redm)));
      if (threadIdx.x == 0) store_scale(a.y8, r, 0, row_scale);
    }
    for (uint32_t g = threadIdx.x; g < turns; g += kLongThreads) {
      float v[8];
      normed_group(g, v);
      if (!a.y8.at) store_group8<DT, false>(y, g, a.size, pack<DT>(v));
      else if (!a.y8.row) store_eight_block(a.y8, r, g * kGroup, a.size, v);
      else if (g < groups) store_eight_group(a.y8, r, g * kGroup, v, row_scale);
    }
    if (a.rstd && threadIdx.x == 0) a.rstd[r] = rstd;
  }
}

// ---------------------------------------------------------------- gradients of long rows
// Two passes, for rows whose columns' sums would fill a compute unit's
// registers and more.  The first leaves a row's mean; the second takes strips
// of columns down many rows, whose sums stay in registers, and reads the
// matrices again, mostly from the cache before memory.  Workgroups of the
// second: kLongStrips in a 16-bit format, two for each compute unit, and twice
// as many in binary32, whose strips are half as wide.  1000 x 40000 residual
// gradients in bfloat16 41.9 and 48.4 us, and 4.8 for the join: 400 MB at 4.2
// TB/s, of which 320 would do.
constexpr uint32_t kLongStrips = 512;

// The eight values of group g of what was normed, zeros past the row's end.
template <int DT>
__device__ __forceinline__ void normed_input(const RmsBwdArgs& a, uint32_t r, uint32_t g, float (&v)[8]) {
  if (a.x8.at) {
    const uint32_t c = g * kGroup;
    if (c < a.size) {
      Unit8<GCLIP_BF16> u = load_eight<GCLIP_BF16, false>(a.x8.at + r * a.x8.ld, c);
      settle_eight<GCLIP_BF16>(u, c, a.size);
      unit_value<GCLIP_BF16>(u, load_scale(a.x8, r, c), v);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = 0.0f;
    }
  } else {
    unpack<DT>(load_group8<DT, false>(a.x.at + r * a.x.ld, g, a.size), v);
  }
}

template <int DT>
__global__ __launch_bounds__(kLongThreads) void k_rms_row_means(RmsBwdArgs a) {
  __shared__ double red[kLongWaves];
  const uint32_t groups = (a.size + kGroup - 1) / kGroup;
  for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const float rstd = a.rstd[r];
    double s = 0.0;  // of each group's binary32 sums
    for (uint32_t g = threadIdx.x; g < groups; g += kLongThreads) {
      float y[8], n[8], w[8], t = 0.0f;
      unpack<DT>(load_group8<DT, false>(a.dy.at + r * a.dy.ld, g, a.size), y);
      normed_input<DT>(a, r, g, n);
      weight_group<DT>(a.weight, a.wdt, g, a.size, 1.0f, w);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (g * kGroup + k < a.size) t = __builtin_fmaf(y[k] * w[k], n[k] * rstd, t);
      s += (double)t;
    }
    s = workgroup_sum(s, red);
    if (threadIdx.x == 0) a.sums[r] = (float)(s / (double)a.size);
  }
}

// Unit u's place in a row: a unit that passes the row's end is read as its last
// 16 bytes, and settled afterwards.
template <int DT>
__device__ __forceinline__ u32x4 load_clamped(uint64_t row, uint32_t c, uint32_t size) {
  return load16<DT, false>(row + (uint64_t)min(c, size - kUnit<DT>) * kElem<DT>);
}
template <int DT>
__device__ __forceinline__ void settle_unit(u32x4& q, uint32_t c, uint32_t size) {
  if (c + kUnit<DT> > size) q = c < size ? moved_down<DT>(q, kUnit<DT> - size % kUnit<DT>) : u32x4{0u, 0u, 0u, 0u};
}

// A workgroup takes a strip of 64 units of columns and part blockIdx.z of the
// rows, its waves in turn; a row's loads are under way while the one before is
// worked on.
template <int DT, bool RES, bool DROP, bool EIGHT>
__global__ __launch_bounds__(kLongThreads) void k_rms_grad_long(RmsBwdArgs a, DropArgs d) {
  constexpr uint32_t kU = kUnit<DT>;
  __shared__ float red[kLongWaves][64 * kU + 1];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t strip = workgroup_of_grid() * (64 * kU);
  if (strip >= a.size) return;
  const uint32_t c = (uint32_t)strip + lane * kU, c8 = min(c, (a.size - 1) / kU * kU);
  const uint32_t step = DROP ? drop_step(d) : 0u;
  const uint32_t stride = gridDim.z * kLongWaves;
  float w[kU], dw[kU] = {};
  if (a.weight == 0) {
#pragma unroll
    for (uint32_t j = 0; j < kU; ++j) w[j] = 1.0f;
  } else if (DT != GCLIP_F32 && a.wdt == GCLIP_F32) {
    float t[8];
    weight_group<DT>(a.weight, a.wdt, c / kGroup, a.size, 1.0f, t);
#pragma unroll
    for (uint32_t j = 0; j < kU; ++j) w[j] = t[j];
  } else {
    u32x4 q = load_clamped<DT>(a.weight, c, a.size);
    settle_unit<DT>(q, c, a.size);
    unpack_unit<DT>(q, w);
  }
  u32x4 ny, nx{0u, 0u, 0u, 0u}, nh{0u, 0u, 0u, 0u};
  Unit8<DT> n8{};
  float ns = 0.0f, nrstd = 0.0f, nc2 = 0.0f;
  const auto fetch = [&](uint32_t r) {
    ny = load_clamped<DT>(a.dy.at + r * a.dy.ld, c, a.size);
    if constexpr (EIGHT) {
      n8 = load_eight<DT, false>(a.x8.at + r * a.x8.ld, c8);
      ns = load_scale(a.x8, r, c8);
    } else {
      nx = load_clamped<DT>(a.x.at + r * a.x.ld, c, a.size);
    }
    if (RES && a.dh.at) nh = load_clamped<DT>(a.dh.at + r * a.dh.ld, c, a.size);
    nrstd = a.rstd[r];
    nc2 = a.sums[r];
  };
  uint32_t r = blockIdx.z * kLongWaves + wave;
  if (r < a.rows) fetch(r);
  while (r < a.rows) {
    float y[kU], n[kU], h[kU];
    const float rstd = nrstd, c2 = nc2;
    settle_unit<DT>(ny, c, a.size);
    unpack_unit<DT>(ny, y);
    if constexpr (EIGHT) {
      settle_eight<DT>(n8, c, a.size);
      unit_value<DT>(n8, ns, n);
    } else {
      settle_unit<DT>(nx, c, a.size);
      unpack_unit<DT>(nx, n);
    }
    if constexpr (RES) {
      settle_unit<DT>(nh, c, a.size);
      unpack_unit<DT>(nh, h);
    }
    const uint32_t next = r + stride;
    if (next < a.rows) fetch(next);
#pragma unroll
    for (uint32_t j = 0; j < kU; ++j) {
      n[j] *= rstd;
      dw[j] = __builtin_fmaf(y[j], n[j], dw[j]);
      n[j] = rstd * (y[j] * w[j] - n[j] * c2);
      if constexpr (RES) n[j] += h[j];
    }
    if (c < a.size) {
      store_unit<DT, true>(a.dres.at + r * a.dres.ld, c / kU, a.size, pack_unit<DT>(n));
      if constexpr (DROP) {
        drop_unit<DT>(d, step, r, c, n);
        store_unit<DT, true>(a.dx.at + r * a.dx.ld, c / kU, a.size, pack_unit<DT>(n));
      }
    }
    r = next;
  }
  if (!a.dweight) return;
#pragma unroll
  for (uint32_t j = 0; j < kU; ++j) red[wave][lane * kU + j] = dw[j];
  __syncthreads();
  for (uint32_t i = threadIdx.x; i < 64 * kU; i += kLongThreads) {
    const uint64_t col = strip + i;
    float t = red[0][i];
#pragma unroll
    for (int k = 1; k < kLongWaves; ++k) t += red[k][i];
    if (col < a.size) a.partials[blockIdx.z * part_columns(a.size) + col] = t;
  }
}

// ---------------------------------------------------------------- rows of fewer than eight columns
// A lane takes a row, element by element; it is a block of its own.
template <int DT>
__device__ __forceinline__ void load_short(uint64_t row, uint32_t size, float (&v)[8]) {
#pragma unroll
  for (uint32_t k = 0; k < 8; ++k) v[k] = k < size && k < 7 ? elem_float<DT>(load_elem<DT>(row + k * kElem<DT>)) : 0.0f;
}
template <int DT>
__device__ __forceinline__ void store_short(uint64_t row, uint32_t size, const float (&v)[8]) {
#pragma unroll
  for (uint32_t k = 0; k < 7; ++k)
    if (k < size) store_elem<DT>(row + k * kElem<DT>, elem_bits<DT>(v[k]));
}
template <int DT>
__device__ __forceinline__ void weight_short(uint64_t w, int wdt, uint32_t size, float (&v)[8]) {
  if (w == 0) {
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) v[k] = 1.0f;
  } else if (DT == GCLIP_F32 || wdt == GCLIP_F32) {
    load_short<GCLIP_F32>(w, size, v);
  } else {
    load_short<DT>(w, size, v);
  }
}
__device__ __forceinline__ void store_eight_short(const Eight& e, uint64_t r, const float (&v)[8]) {
  const float scale = scale_of(__uint_as_float(largest_finite(v)));
  store_eight_group(e, r, 0, v, scale);
  store_scale(e, r, 0, scale);
}

template <int DT, bool RES, bool DROP>
__global__ __launch_bounds__(kShortThreads) void k_rms_short(RmsFwdArgs a, DropArgs d) {
  const uint32_t r = blockIdx.x * kShortThreads + threadIdx.x;
  if (r >= a.rows) return;
  float v[8], w[8];
  load_short<DT>(a.x.at + r * a.x.ld, a.size, v);
  if constexpr (RES) {
    float q[8];
    if constexpr (DROP) drop_group(d, drop_step(d), r, 0, v);
    load_short<DT>(a.residual.at + r * a.residual.ld, a.size, q);
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) v[k] = k < a.size ? elem_float<DT>(elem_bits<DT>(v[k] + q[k])) : 0.0f;
    store_short<DT>(a.h.at + r * a.h.ld, a.size, v);
  }
  if (a.kept.at) store_eight_short(a.kept, r, v);
  weight_short<DT>(a.weight, a.wdt, a.size, w);
  double s = 0.0;
#pragma unroll
  for (int k = 0; k < 7; ++k) s = __builtin_fma((double)v[k], (double)v[k], s);
  const double rs = 1.0 / sqrt(s / (double)a.size + (double)a.eps);
  const float low = rs < 0x1p-100 ? 0x1p-96f : 1.0f, high = (float)(rs / (double)low);  // see k_rms_long
#pragma unroll
  for (uint32_t k = 0; k < 8; ++k) v[k] = k < a.size ? v[k] * low * high * w[k] : 0.0f;
  if (a.y8.at) store_eight_short(a.y8, r, v);
  else store_short<DT>(a.y.at + r * a.y.ld, a.size, v);
  if (a.rstd) a.rstd[r] = (float)rs;
}

template <int DT, bool RES, bool DROP>
__global__ __launch_bounds__(kShortThreads) void k_rms_grad_short(RmsBwdArgs a, DropArgs d) {
  __shared__ float red[kShortThreads / 64][8];
  const uint32_t step = DROP ? drop_step(d) : 0u;
  float w[8], dw[8] = {};
  weight_short<DT>(a.weight, a.wdt, a.size, w);
  for (uint64_t i = blockIdx.x * (uint64_t)kShortThreads + threadIdx.x; i < a.rows; i += (uint64_t)gridDim.x * kShortThreads) {
    const uint32_t r = (uint32_t)i;
    float g[8], n[8], c2 = 0.0f;
    load_short<DT>(a.dy.at + r * a.dy.ld, a.size, g);
    if (a.x8.at) normed_input<DT>(a, r, 0, n);
    else load_short<DT>(a.x.at + r * a.x.ld, a.size, n);
    const float rstd = a.rstd[r];
#pragma unroll
    for (uint32_t k = 0; k < 7; ++k) {
      n[k] = k < a.size ? n[k] * rstd : 0.0f;
      dw[k] = __builtin_fmaf(g[k], n[k], dw[k]);
      g[k] *= w[k];
      c2 = __builtin_fmaf(g[k], n[k], c2);
    }
    c2 /= (float)a.size;
#pragma unroll
    for (int k = 0; k < 7; ++k) n[k] = rstd * (g[k] - n[k] * c2);
    if (RES && a.dh.at) {
      load_short<DT>(a.dh.at + r * a.dh.ld, a.size, g);
#pragma unroll
      for (int k = 0; k < 7; ++k) n[k] += g[k];
    }
    store_short<DT>(a.dres.at + r * a.dres.ld, a.size, n);
    if constexpr (DROP) {
      drop_group(d, step, r, 0, n);
      store_short<DT>(a.dx.at + r * a.dx.ld, a.size, n);
    }
  }
  if (!a.dweight) return;
#pragma unroll
  for (int k = 0; k < 7; ++k) {
    const float p = lanes_sum<64>(dw[k]);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6][k] = p;
  }
  __syncthreads();
  if (threadIdx.x < a.size) {
    float t = red[0][threadIdx.x];
#pragma unroll
    for (int i = 1; i < kShortThreads / 64; ++i) t += red[i][threadIdx.x];
    a.partials[blockIdx.x * part_columns(a.size) + threadIdx.x] = t;
  }
}

template <int DT>
hipError_t forward_any(const RmsFwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if (a.size < kRegistersMin) {
    const dim3 grid((a.rows - 1) / kShortThreads + 1), block(kShortThreads);
    if (!residual) hipLaunchKernelGGL((k_rms_short<DT, false, false>), grid, block, 0, st, a, DropArgs{});
    else if (!drop) hipLaunchKernelGGL((k_rms_short<DT, true, false>), grid, block, 0, st, a, DropArgs{});
    else hipLaunchKernelGGL((k_rms_short<DT, true, true>), grid, block, 0, st, a, *drop);
    return hipGetLastError();
  }
  const dim3 grid(std::min<uint32_t>(a.rows, 1u << 20)), block(kLongThreads);
  if (!residual) hipLaunchKernelGGL((k_rms_long<DT, false, false>), grid, block, 0, st, a, DropArgs{});
  else if (!drop) hipLaunchKernelGGL((k_rms_long<DT, true, false>), grid, block, 0, st, a, DropArgs{});
  else hipLaunchKernelGGL((k_rms_long<DT, true, true>), grid, block, 0, st, a, *drop);
  return hipGetLastError();
}

template <int DT, bool EIGHT>
void launch_long(const RmsBwdArgs& a, bool residual, const DropArgs* drop, dim3 strips, dim3 block, hipStream_t st) {
  if (!residual) hipLaunchKernelGGL((k_rms_grad_long<DT, false, false, EIGHT>), strips, block, 0, st, a, DropArgs{});
  else if (!drop) hipLaunchKernelGGL((k_rms_grad_long<DT, true, false, EIGHT>), strips, block, 0, st, a, DropArgs{});
  else hipLaunchKernelGGL((k_rms_grad_long<DT, true, true, EIGHT>), strips, block, 0, st, a, *drop);
}

template <int DT>
hipError_t backward_any(const RmsBwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if (a.rows > 0 && a.size < kRegistersMin) {
    const dim3 grid(a.parts), block(kShortThreads);
    if (!residual) hipLaunchKernelGGL((k_rms_grad_short<DT, false, false>), grid, block, 0, st, a, DropArgs{});
    else if (!drop) hipLaunchKernelGGL((k_rms_grad_short<DT, true, false>), grid, block, 0, st, a, DropArgs{});
    else hipLaunchKernelGGL((k_rms_grad_short<DT, true, true>), grid, block, 0, st, a, *drop);
  } else if (a.rows > 0) {
    const dim3 block(kLongThreads), strips = grid_of((a.size - 1) / (64 * kUnit<DT>) + 1, a.parts);
    hipLaunchKernelGGL((k_rms_row_means<DT>), dim3(std::min<uint32_t>(a.rows, 1u << 20)), block, 0, st, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (a.x8.at) launch_long<DT, true>(a, residual, drop, strips, block, st);
    else launch_long<DT, false>(a, residual, drop, strips, block, st);
  }
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || !a.dweight ? e : rms_join_weight_grad<DT>(a, st);
}

template <int DT>
hipError_t forward(const RmsFwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if (!in_registers(a.size, kFwdMax)) return forward_any<DT>(a, residual, drop, st);
  return a.y8.at || a.kept.at ? rms_forward_rows<DT, true>(a, residual, drop, st)
                              : rms_forward_rows<DT, false>(a, residual, drop, st);
}

template <int DT>
hipError_t backward(const RmsBwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if (a.rows == 0 || !in_registers(a.size, kRmsBwdMax)) return backward_any<DT>(a, residual, drop, st);
  return a.x8.at ? rms_backward_rows<DT, true>(a, residual, drop, st) : rms_backward_rows<DT, false>(a, residual, drop, st);
}

}  // namespace

// Rows in registers: a part for each workgroup.  Shorter rows: as many as
// leave each lane four rows.  Longer ones: as many as make kLongStrips
// workgroups of strips of 512 columns, those of a 16-bit format, and leave each
// wave two rows: the workspace serves any format.
uint32_t rms_parts(int64_t rows, int64_t size) {
  if (rows == 0) return 0;
  const uint32_t n = (uint32_t)rows, c = (uint32_t)size;
  if (in_registers(c, kRmsBwdMax)) return std::max(rms_bwd_parts<GCLIP_F32>(n, c), rms_bwd_parts<GCLIP_BF16>(n, c));
  if (c < kRegistersMin) return std::min<uint32_t>((n - 1) / (4 * kShortThreads) + 1, kBwdParts);
  const uint32_t strips = (c - 1) / 512 + 1;
  return std::min<uint32_t>({std::max<uint32_t>(kLongStrips / strips, 1), (n - 1) / (2 * kLongWaves) + 1, kBwdParts});
}

hipError_t launch_rms_forward(const RmsFwdArgs& a, int32_t dtype, bool residual, const DropArgs* drop, hipStream_t st) {
  switch (dtype) {
    case GCLIP_F32: return forward<GCLIP_F32>(a, residual, drop, st);
    case GCLIP_F16: return forward<GCLIP_F16>(a, residual, drop, st);
    default: return forward<GCLIP_BF16>(a, residual, drop, st);
  }
}

hipError_t launch_rms_backward(const RmsBwdArgs& a, int32_t dtype, bool residual, const DropArgs* drop,
                               hipStream_t st) {
  switch (dtype) {
    case GCLIP_F32: return backward<GCLIP_F32>(a, residual, drop, st);
    case GCLIP_F16: return backward<GCLIP_F16>(a, residual, drop, st);
    default: return backward<GCLIP_BF16>(a, residual, drop, st);
  }
}

}  // namespace gclip
