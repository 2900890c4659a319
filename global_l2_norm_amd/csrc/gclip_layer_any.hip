// gclip_layer_any.hip -- the norms of rows that the kernels with rows in
// registers do not take, shorter and longer ones, and dropout.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gclip_layer_device.hpp"

namespace gclip {
namespace {

constexpr int kAnyThreads = 256;
constexpr int kAnyWaves = kAnyThreads / 64;
constexpr int kRowThreads = 512;
constexpr int kRowWaves = kRowThreads / 64;

// Sum over the workgroup, the same bits in every thread.
__device__ __forceinline__ double any_sum(double v, double* red) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) v += __shfl_xor(v, off, 64);
  __syncthreads();  // red may still be read by a previous call
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  double t = red[0];
#pragma unroll
  for (int i = 1; i < kRowWaves; ++i) t += red[i];
  return t;
}

// Three passes over a row: h and the sum, the squares, y; the later ones find
// the row in the caches.  A thread reads there only the groups that it wrote
// itself.  The sums are binary64, so no finite row overflows them.  Bound by
// the passes' latency: 512 x 40000 in bfloat16 takes 28.3 us, 2.9 TB/s of the
// row's one read and one write, and fetches it 2.7 times into the L2 (1024
// lanes a row: 33.0 us).
template <int DT, bool RES, bool DROP>
__global__ __launch_bounds__(kRowThreads) void k_norm_any(FwdArgs a, DropArgs d) {
  __shared__ double red[kRowWaves];
  const uint32_t groups = (a.size + kGroup - 1) / kGroup;
  const uint32_t step = DROP ? drop_step(d) : 0u;
  for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const uint64_t x = a.x.at + r * a.x.ld, y = a.y.at + r * a.y.ld;
    const uint64_t h = RES ? a.h.at + r * a.h.ld : x;
    double s = 0.0;
    for (uint32_t g = threadIdx.x; g < groups; g += kRowThreads) {
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
    for (uint32_t g = threadIdx.x; g < groups; g += kRowThreads) {
      float v[8];
      unpack<DT>(load_group8<DT, false>(h, g, a.size), v);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const double t = (double)v[k] - mean;
        ss += g * kGroup + k < a.size ? t * t : 0.0;
      }
    }
    const float rstd = (float)(1.0 / sqrt(any_sum(ss, red) / (double)a.size + (double)a.eps));
    const float m = (float)mean, hm = 0.5f * m, tr = 2.0f * rstd;
    for (uint32_t g = threadIdx.x; g < groups; g += kRowThreads) {
      float v[8], w[8], b[8];
      unpack<DT>(load_group8<DT, false>(h, g, a.size), v);
      weight_group<DT>(a.weight, a.wdt, g, a.size, 1.0f, w);
      weight_group<DT>(a.bias, a.wdt, g, a.size, 0.0f, b);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = normed(v[k], hm, tr) * w[k] + b[k];
      store_group8<DT, false>(y, g, a.size, pack<DT>(v));
    }
    if (a.mean && threadIdx.x == 0) {
      a.mean[r] = m;
      a.rstd[r] = rstd;
    }
  }
}

// ---------------------------------------------------------------- gradients of long rows
// Two passes, for rows whose columns' sums would fill a compute unit's
// registers and more: with a workgroup a row, each of 256 workgroups would
// leave partial sums as long as the row (2048 x 16384 in bfloat16: 34 MB
// written and read again, 68 us).  The first pass leaves a row's two means;
// the second takes strips of columns down many rows, whose sums stay in
// registers, and reads the matrices again, mostly from the cache before
// memory.
constexpr int kLongThreads = 512;
constexpr int kLongWaves = kLongThreads / 64;
// Workgroups of the second pass: 512, two for each compute unit, took 63.3 us
// for 2048 x 16384 in bfloat16, 1024 of them 65.6 and 2048 of them 67.1.
constexpr uint32_t kLongStrips = 512;

template <int DT>
__device__ __forceinline__ void unit_settled(u32x4& q, uint32_t c, uint32_t size) {
  if (c + kUnit<DT> > size)
    q = c < size ? moved_down<DT>(q, kUnit<DT> - size % kUnit<DT>) : u32x4{0u, 0u, 0u, 0u};
}
// Past the row's end other elements of the row, see settle_round().
template <int DT>
__device__ __forceinline__ void unit_settled_round(u32x4& q, uint32_t c, uint32_t size) {
  if (c < size && c + kUnit<DT> > size) q = moved_down<DT, true>(q, kUnit<DT> - size % kUnit<DT>);
}
template <int DT>
__device__ __forceinline__ uint64_t unit_place(uint32_t c, uint32_t size) {
  return (uint64_t)(c + kUnit<DT> <= size ? c : size - kUnit<DT>) * kElem<DT>;
}
template <int DT>
__device__ __forceinline__ u32x4 unit_clamped(uint64_t row, uint32_t c, uint32_t size) {
  return load16<DT, false>(row + unit_place<DT>(c, size));
}
template <int DT>
__device__ __forceinline__ void weight_unit(uint64_t w, int wdt, uint32_t c, uint32_t size, float (&v)[kUnit<DT>]) {
  if constexpr (DT == GCLIP_F32) {
    if (w == 0) {
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = 1.0f;
    } else {
      u32x4 q = unit_clamped<DT>(w, c, size);
      unit_settled<DT>(q, c, size);
      unpack_unit<DT>(q, v);
    }
  } else {
    weight_group<DT>(w, wdt, c / kGroup, size, 1.0f, v);
  }
}

template <int DT>
__global__ __launch_bounds__(kLongThreads) void k_row_means_long(BwdArgs a) {
  __shared__ double red[2][kLongWaves];
  const uint32_t units = (a.size + kUnit<DT> - 1) / kUnit<DT>;
  for (uint32_t r = blockIdx.x; r < a.rows; r += gridDim.x) {
    const uint64_t dy = a.dy.at + r * a.dy.ld, x = a.x.at + r * a.x.ld;
    const float hm = 0.5f * a.mean[r], tr = 2.0f * a.rstd[r];
    double s1 = 0.0, s2 = 0.0;  // of each unit's binary32 sums
    for (uint32_t u = threadIdx.x; u < units; u += kLongThreads) {
      const uint32_t c = u * kUnit<DT>;
      u32x4 p = unit_clamped<DT>(dy, c, a.size), q = unit_clamped<DT>(x, c, a.size);
      float g[kUnit<DT>], n[kUnit<DT>], w[kUnit<DT>];
      weight_unit<DT>(a.weight, a.wdt, c, a.size, w);
      unit_settled<DT>(p, c, a.size);
      unit_settled_round<DT>(q, c, a.size);
      unpack_unit<DT>(p, g);
      unpack_unit<DT>(q, n);
      float t1 = 0.0f, t2 = 0.0f;
#pragma unroll
      for (uint32_t j = 0; j < kUnit<DT>; ++j) {
        const float t = g[j] * w[j];
        t1 += t;
        t2 = __builtin_fmaf(t, normed(n[j], hm, tr), t2);
      }
      s1 += (double)t1;
      s2 += (double)t2;
    }
#pragma unroll
    for (int off = 32; off > 0; off >>= 1) {
      s1 += __shfl_xor(s1, off, 64);
      s2 += __shfl_xor(s2, off, 64);
    }
    __syncthreads();  // red may still be read for the row before
    if ((threadIdx.x & 63) == 0) {
      red[0][threadIdx.x >> 6] = s1;
      red[1][threadIdx.x >> 6] = s2;
    }
    __syncthreads();
    if (threadIdx.x < 2) {
      double t = red[threadIdx.x][0];
#pragma unroll
      for (int i = 1; i < kLongWaves; ++i) t += red[threadIdx.x][i];
      a.sums[2 * (uint64_t)r + threadIdx.x] = (float)(t / (double)a.size);
    }
  }
}

// A workgroup takes a strip of 64 units of columns and part blockIdx.z of the
// rows, its waves in turn; a row's loads are under way while the one before
// is worked on.
template <int DT, bool RES, bool DROP>
__global__ __launch_bounds__(kLongThreads) void k_norm_grad_long(BwdArgs a, DropArgs d) {
  __shared__ float red[kLongWaves][64 * kUnit<DT> + 1];
  const uint32_t lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint64_t strip = workgroup_of_grid() * (64 * kUnit<DT>);
  if (strip >= a.size) return;
  const uint32_t c = (uint32_t)strip + lane * kUnit<DT>;
  const uint32_t step = DROP ? drop_step(d) : 0u;
  const uint32_t stride = gridDim.z * kLongWaves;
  float w[kUnit<DT>], dw[kUnit<DT>] = {}, db[kUnit<DT>] = {};
  weight_unit<DT>(a.weight, a.wdt, c, a.size, w);
  u32x4 ny, nx, nh{0u, 0u, 0u, 0u};
  float nmean = 0.0f, nrstd = 0.0f, nc1 = 0.0f, nc2 = 0.0f;
  const auto fetch = [&](uint32_t r) {
    ny = unit_clamped<DT>(a.dy.at + r * a.dy.ld, c, a.size);
    nx = unit_clamped<DT>(a.x.at + r * a.x.ld, c, a.size);
    if (RES && a.dh.at) nh = unit_clamped<DT>(a.dh.at + r * a.dh.ld, c, a.size);
    nmean = a.mean[r];
    nrstd = a.rstd[r];
    nc1 = a.sums[2 * (uint64_t)r];
    nc2 = a.sums[2 * (uint64_t)r + 1];
  };
  uint32_t r = blockIdx.z * kLongWaves + wave;
  if (r < a.rows) fetch(r);
  while (r < a.rows) {
    float g[kUnit<DT>], n[kUnit<DT>], h[kUnit<DT>];
    const float rstd = nrstd, hm = 0.5f * nmean, tr = 2.0f * rstd, c1 = nc1, c2 = nc2;
    unit_settled<DT>(ny, c, a.size);
    unit_settled<DT>(nx, c, a.size);
    unpack_unit<DT>(ny, g);
    unpack_unit<DT>(nx, n);
    if constexpr (RES) {
      unit_settled<DT>(nh, c, a.size);
      unpack_unit<DT>(nh, h);
    }
    const uint32_t next = r + stride;
    if (next < a.rows) fetch(next);
#pragma unroll
    for (uint32_t j = 0; j < kUnit<DT>; ++j) {
      n[j] = normed(n[j], hm, tr);
      dw[j] = __builtin_fmaf(g[j], n[j], dw[j]);
      db[j] += g[j];
      n[j] = rstd * (g[j] * w[j] - c1 - n[j] * c2);
      if constexpr (RES) n[j] += h[j];
    }
    if (c < a.size) {
      store_unit<DT, true>(a.dres.at + r * a.dres.ld, c / kUnit<DT>, a.size, pack_unit<DT>(n));
      if constexpr (DROP) {
        drop_unit<DT>(d, step, r, c, n);
        store_unit<DT, true>(a.dx.at + r * a.dx.ld, c / kUnit<DT>, a.size, pack_unit<DT>(n));
      }
    }
    r = next;
  }
  if (!a.dweight && !a.dbias) return;
#pragma unroll
  for (uint32_t which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (uint32_t j = 0; j < kUnit<DT>; ++j) red[wave][lane * kUnit<DT> + j] = which ? db[j] : dw[j];
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < 64 * kUnit<DT>; i += kLongThreads) {
      const uint32_t col = (uint32_t)strip + i;
      float t = red[0][i];
#pragma unroll
      for (int k = 1; k < kLongWaves; ++k) t += red[k][i];
      if (col < a.size) a.partials[((uint64_t)blockIdx.z * 2 + which) * a.size + col] = t;
    }
  }
}

// ---------------------------------------------------------------- rows of fewer than eight columns
// A lane takes a row, element by element.
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
__device__ __forceinline__ void weight_short(uint64_t w, int wdt, uint32_t size, float def, float (&v)[8]) {
  if (w == 0) {
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) v[k] = def;
  } else if (DT == GCLIP_F32 || wdt == GCLIP_F32) {
    load_short<GCLIP_F32>(w, size, v);
  } else {
    load_short<DT>(w, size, v);
  }
}

template <int DT, bool RES, bool DROP>
__global__ __launch_bounds__(kAnyThreads) void k_norm_short(FwdArgs a, DropArgs d) {
  const uint32_t r = blockIdx.x * kAnyThreads + threadIdx.x;
  if (r >= a.rows) return;
  float v[8], w[8], b[8];
  load_short<DT>(a.x.at + r * a.x.ld, a.size, v);
  if constexpr (RES) {
    float q[8];
    if constexpr (DROP) drop_group(d, drop_step(d), r, 0, v);
    load_short<DT>(a.residual.at + r * a.residual.ld, a.size, q);
#pragma unroll
    for (uint32_t k = 0; k < 8; ++k) v[k] = k < a.size ? elem_float<DT>(elem_bits<DT>(v[k] + q[k])) : 0.0f;
    store_short<DT>(a.h.at + r * a.h.ld, a.size, v);
  }
  weight_short<DT>(a.weight, a.wdt, a.size, 1.0f, w);
  weight_short<DT>(a.bias, a.wdt, a.size, 0.0f, b);
  double s = 0.0, ss = 0.0;
#pragma unroll
  for (int k = 0; k < 7; ++k) s += (double)v[k];
  const double mean = s / (double)a.size;
#pragma unroll
  for (uint32_t k = 0; k < 7; ++k) {
    const double t = k < a.size ? (double)v[k] - mean : 0.0;
    ss += t * t;
  }
  const float rstd = (float)(1.0 / sqrt(ss / (double)a.size + (double)a.eps)), m = (float)mean, hm = 0.5f * m,
              tr = 2.0f * rstd;
#pragma unroll
  for (int k = 0; k < 7; ++k) v[k] = __builtin_fmaf(normed(v[k], hm, tr), w[k], b[k]);
  store_short<DT>(a.y.at + r * a.y.ld, a.size, v);
  if (a.mean) {
    a.mean[r] = m;
    a.rstd[r] = rstd;
  }
}

template <int DT, bool RES, bool DROP>
__global__ __launch_bounds__(kAnyThreads) void k_norm_grad_short(BwdArgs a, DropArgs d) {
  __shared__ float red[kAnyWaves][16];
  const uint32_t step = DROP ? drop_step(d) : 0u;
  float w[8], dw[8] = {}, db[8] = {};
  weight_short<DT>(a.weight, a.wdt, a.size, 1.0f, w);
  for (uint32_t r = blockIdx.x * kAnyThreads + threadIdx.x; r < a.rows; r += gridDim.x * kAnyThreads) {
    float g[8], n[8];
    load_short<DT>(a.dy.at + r * a.dy.ld, a.size, g);
    load_short<DT>(a.x.at + r * a.x.ld, a.size, n);
    const float rstd = a.rstd[r], hm = 0.5f * a.mean[r], tr = 2.0f * rstd;
    float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
    for (uint32_t k = 0; k < 7; ++k) {
      n[k] = k < a.size ? normed(n[k], hm, tr) : 0.0f;  // past the end: see settle_round()
      dw[k] = __builtin_fmaf(g[k], n[k], dw[k]);
      db[k] += g[k];
      g[k] *= w[k];
      c1 += g[k];
      c2 = __builtin_fmaf(g[k], n[k], c2);
    }
    c1 /= (float)a.size;
    c2 /= (float)a.size;
#pragma unroll
    for (int k = 0; k < 7; ++k) n[k] = rstd * (g[k] - c1 - n[k] * c2);
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
  if (!a.dweight && !a.dbias) return;
#pragma unroll
  for (int k = 0; k < 7; ++k) {
    const float p = lanes_sum<64>(dw[k]), q = lanes_sum<64>(db[k]);
    if ((threadIdx.x & 63) == 0) {
      red[threadIdx.x >> 6][k] = p;
      red[threadIdx.x >> 6][8 + k] = q;
    }
  }
  __syncthreads();
  if (threadIdx.x < 2 * a.size) {
    const uint32_t which = threadIdx.x >= a.size, col = threadIdx.x - which * a.size;
    float t = red[0][8 * which + col];
#pragma unroll
    for (int i = 1; i < kAnyWaves; ++i) t += red[i][8 * which + col];
    a.partials[((uint64_t)blockIdx.x * 2 + which) * a.size + col] = t;
  }
}

// ---------------------------------------------------------------- dropout
// A lane takes a unit of 16 bytes.  A unit of a 16-bit format is a group; of
// binary32 half of one, whose two lanes run the generator both: a wave's
// accesses are adjacent then, and there is twice the time for it.  Bound by
// memory, with the generator's products (20 for eight elements, at a quarter
// of the full rate) close behind in 16 bits: 1.3B's 16384 x 2048 in bfloat16
// takes 22.3 us, 6.0 TB/s (two units a lane 0.6 us more, four 1.6).
template <int DT, bool STREAMED>
__global__ __launch_bounds__(kAnyThreads) void k_dropout(Rows x, Rows y, uint32_t rows, uint32_t size, DropArgs d) {
  const uint32_t units = (size + kUnit<DT> - 1) / kUnit<DT>;
  const uint64_t i = workgroup_of_grid() * kAnyThreads + threadIdx.x;
  const uint64_t row = i / units;
  if (row >= rows) return;
  const uint32_t r = (uint32_t)row, u = (uint32_t)(i % units);
  u32x4 q;
  if (size % kUnit<DT> == 0) {
    q = load16<DT, STREAMED>(x.at + r * x.ld + u * 16ull);
  } else if (size >= kGroup) {
    q = load16<DT, STREAMED>(x.at + r * x.ld + unit_place<DT>(u * kUnit<DT>, size));
    unit_settled<DT>(q, u * kUnit<DT>, size);
  } else {
    q = load_unit<DT, STREAMED>(x.at + r * x.ld, u, size);
  }
  float v[kUnit<DT>];
  unpack_unit<DT>(q, v);
  drop_unit<DT>(d, drop_step(d), r, u * kUnit<DT>, v);
  store_unit<DT, true>(y.at + r * y.ld, u, size, pack_unit<DT>(v));
}

template <int DT>
hipError_t forward_any(const FwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  const dim3 block(kAnyThreads);
  if (a.size < kRegistersMin) {
    const dim3 grid((a.rows - 1) / kAnyThreads + 1);
    if (!residual) hipLaunchKernelGGL((k_norm_short<DT, false, false>), grid, block, 0, st, a, DropArgs{});
    else if (!drop) hipLaunchKernelGGL((k_norm_short<DT, true, false>), grid, block, 0, st, a, DropArgs{});
    else hipLaunchKernelGGL((k_norm_short<DT, true, true>), grid, block, 0, st, a, *drop);
    return hipGetLastError();
  }
  const dim3 grid(std::min<uint32_t>(a.rows, 1u << 20)), row(kRowThreads);
  if (!residual) hipLaunchKernelGGL((k_norm_any<DT, false, false>), grid, row, 0, st, a, DropArgs{});
  else if (!drop) hipLaunchKernelGGL((k_norm_any<DT, true, false>), grid, row, 0, st, a, DropArgs{});
  else hipLaunchKernelGGL((k_norm_any<DT, true, true>), grid, row, 0, st, a, *drop);
  return hipGetLastError();
}

template <int DT>
hipError_t backward_any(const BwdArgs& a, bool residual, const DropArgs* drop, hipStream_t st) {
  if (a.rows > 0 && a.size < kRegistersMin) {
    const dim3 grid(a.parts), block(kAnyThreads);
    if (!residual) hipLaunchKernelGGL((k_norm_grad_short<DT, false, false>), grid, block, 0, st, a, DropArgs{});
    else if (!drop) hipLaunchKernelGGL((k_norm_grad_short<DT, true, false>), grid, block, 0, st, a, DropArgs{});
    else hipLaunchKernelGGL((k_norm_grad_short<DT, true, true>), grid, block, 0, st, a, *drop);
  } else if (a.rows > 0) {
    const dim3 block(kLongThreads), strips = grid_of((a.size - 1) / (64 * kUnit<DT>) + 1, a.parts);
    hipLaunchKernelGGL((k_row_means_long<DT>), dim3(std::min<uint32_t>(a.rows, 1u << 20)), block, 0, st, a);
    if (!residual) hipLaunchKernelGGL((k_norm_grad_long<DT, false, false>), strips, block, 0, st, a, DropArgs{});
    else if (!drop) hipLaunchKernelGGL((k_norm_grad_long<DT, true, false>), strips, block, 0, st, a, DropArgs{});
    else hipLaunchKernelGGL((k_norm_grad_long<DT, true, true>), strips, block, 0, st, a, *drop);
  }
  const hipError_t e = hipGetLastError();
  return e != hipSuccess || (!a.dweight && !a.dbias) ? e : join_weight_grads<DT>(a, st);
}

template <int DT>
hipError_t dropout(const Rows& x, const Rows& y, uint32_t rows, uint32_t size, const DropArgs& d, hipStream_t st) {
  const uint64_t total = (uint64_t)rows * ((size + kUnit<DT> - 1) / kUnit<DT>);
  const dim3 grid = grid_of((total + kAnyThreads - 1) / kAnyThreads), block(kAnyThreads);
  if (total * 32 > kStreamBytes) hipLaunchKernelGGL((k_dropout<DT, true>), grid, block, 0, st, x, y, rows, size, d);
  else hipLaunchKernelGGL((k_dropout<DT, false>), grid, block, 0, st, x, y, rows, size, d);
  return hipGetLastError();
}

}  // namespace

// Rows in registers: a part for each workgroup.  Shorter rows: as many as
// leave each lane four rows.  Longer ones: as many as make kLongStrips
// workgroups of strips of 512 columns, and leave each wave two rows.
uint32_t layer_parts(int64_t rows, int64_t size) {
  if (rows == 0) return 0;
  const uint32_t n = (uint32_t)rows, c = (uint32_t)size;
  if (in_registers(c, kBwdMax)) return std::max(bwd_parts<GCLIP_F32>(n, c), bwd_parts<GCLIP_BF16>(n, c));
  if (c < kRegistersMin) return std::min<uint32_t>((n - 1) / (4 * kAnyThreads) + 1, kBwdParts);
  const uint32_t strips = (c - 1) / 512 + 1;
  return std::min<uint32_t>({std::max<uint32_t>(kLongStrips / strips, 1), (n - 1) / (2 * kLongWaves) + 1, kBwdParts});
}

hipError_t launch_layer_forward(const FwdArgs& a, int32_t dtype, bool residual, const DropArgs* drop, hipStream_t st) {
  const bool regs = in_registers(a.size, kFwdMax);
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
  const bool regs = a.rows > 0 && in_registers(a.size, kBwdMax);
  switch (dtype) {
    case GCLIP_F32:
      return regs ? backward_rows<GCLIP_F32>(a, residual, drop, st) : backward_any<GCLIP_F32>(a, residual, drop, st);
    case GCLIP_F16:
      return regs ? backward_rows<GCLIP_F16>(a, residual, drop, st) : backward_any<GCLIP_F16>(a, residual, drop, st);
    default:
      return regs ? backward_rows<GCLIP_BF16>(a, residual, drop, st) : backward_any<GCLIP_BF16>(a, residual, drop, st);
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
