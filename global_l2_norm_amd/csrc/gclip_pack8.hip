// gclip_pack8.hip -- matrices into 8 bits and out of them.
#include <algorithm>

#include "gclip_block_device.hpp"

namespace gclip {
namespace {

constexpr int kPackThreads = 256;

// A scale a block: its lanes hold a unit each and share it.  Bound by memory:
// 16384 x 2048 in bfloat16 18.1 us, 102 MB at 5.6 TB/s (a copy of 100 MB: 5.6);
// out of 8 bits 15.8 us, 6.5 TB/s.
template <int DT, bool STREAMED>
__global__ __launch_bounds__(kPackThreads) void k_pack8(Rows x, Eight out, uint32_t rows, uint32_t size, Split split) {
  constexpr uint32_t kU = kUnit<DT>;
  const uint64_t i = workgroup_of_grid() * kPackThreads + threadIdx.x;
  const uint32_t r = row_of(i, split);
  if (r >= rows) return;  // whole blocks of lanes
  const uint32_t c = (uint32_t)(i - r * split.of) * kU;
  u32x4 q{0u, 0u, 0u, 0u};
  if (c < size) q = load_unit_at<DT, STREAMED>(x.at + r * x.ld, c, size);
  const float scale = block_scale<DT, kBlockLanes<DT>>(q);
  if (c >= size) return;
  float v[kU];
  unpack_unit<DT>(q, v);
  store_eight<DT, true>(out.at + r * out.ld, c, unit_eight<DT>(v, 1.0f / scale));
  if (threadIdx.x % kBlockLanes<DT> == 0) store_scale(out, r, c / kBlock, scale);
}

// A scale a row, which LANES lanes hold: in registers up to kHeld units each,
// else read again, from the caches.
constexpr int kHeld = 8;
template <int LANES>
__device__ __forceinline__ uint32_t row_most(uint32_t m, uint32_t* red) {
  m = lanes_max<64>(m);
  if constexpr (LANES > 64) {
    __syncthreads();  // red may still be read for the row before
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int i = 1; i < LANES / 64; ++i) m = max(m, red[i]);
  }
  return m;
}
template <int DT, int LANES>
__global__ __launch_bounds__((LANES > kPackThreads ? LANES : kPackThreads)) void k_pack8_row(Rows x, Eight out,
                                                                                            uint32_t rows,
                                                                                            uint32_t size) {
  constexpr uint32_t kU = kUnit<DT>;
  __shared__ uint32_t red[LANES / 64];
  const uint32_t lane = threadIdx.x % LANES, at_once = blockDim.x / LANES;
  const uint32_t units = (size - 1) / kU + 1;
  const bool held = units <= LANES * kHeld;
  for (uint64_t row = blockIdx.x * (uint64_t)at_once + threadIdx.x / LANES; row < rows; row += (uint64_t)gridDim.x * at_once) {
    const uint32_t r = (uint32_t)row;
    const uint64_t from = x.at + r * x.ld, to = out.at + r * out.ld;
    u32x4 q[kHeld];
    uint32_t m = 0;
    if (held) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const uint32_t u = lane + k * LANES;
        q[k] = u32x4{0u, 0u, 0u, 0u};
        if (u < units) q[k] = load_unit_at<DT, false>(from, u * kU, size);
      }
#pragma unroll
      for (int k = 0; k < kHeld; ++k) m = max(m, unit_magnitude_finite<DT>(q[k]));
    } else {
      for (uint32_t u = lane; u < units; u += LANES)
        m = max(m, unit_magnitude_finite<DT>(load_unit_at<DT, false>(from, u * kU, size)));
    }
    const float scale = scale_of(elem_float<DT>(row_most<LANES>(m, red))), inverse = 1.0f / scale;
    if (held) {
#pragma unroll
      for (int k = 0; k < kHeld; ++k) {
        const uint32_t u = lane + k * LANES;
        float v[kU];
        unpack_unit<DT>(q[k], v);
        if (u < units) store_eight<DT, true>(to, u * kU, unit_eight<DT>(v, inverse));
      }
    } else {
      for (uint32_t u = lane; u < units; u += LANES) {
        float v[kU];
        unpack_unit<DT>(load_unit_at<DT, false>(from, u * kU, size), v);
        store_eight<DT, true>(to, u * kU, unit_eight<DT>(v, inverse));
      }
    }
    if (lane == 0) store_scale(out, r, 0, scale);
  }
}

template <int DT, bool STREAMED>
__global__ __launch_bounds__(kPackThreads) void k_unpack8(Eight x, Rows out, uint32_t rows, uint32_t size, Split split) {
  constexpr uint32_t kU = kUnit<DT>;
  const uint64_t i = workgroup_of_grid() * kPackThreads + threadIdx.x;
  const uint32_t r = row_of(i, split);
  if (r >= rows) return;
  const uint32_t c = (uint32_t)(i - r * split.of) * kU;
  float v[kU];
  unit_value<DT>(load_eight<DT, STREAMED>(x.at + r * x.ld, c), load_scale(x, r, c), v);
  store_unit<DT, true>(out.at + r * out.ld, c / kU, size, pack_unit<DT>(v));
}

template <int DT>
hipError_t pack(const Rows& x, const Eight& out, uint32_t rows, uint32_t size, hipStream_t st) {
  const uint32_t units = (size - 1) / kUnit<DT> + 1;
  if (out.row && size > kBlock) {
    if (units <= 64 * kHeld)
      hipLaunchKernelGGL((k_pack8_row<DT, 64>), dim3(std::min<uint32_t>((rows - 1) / 4 + 1, 1u << 20)), dim3(kPackThreads), 0, st, x, out, rows, size);
    else
      hipLaunchKernelGGL((k_pack8_row<DT, 512>), dim3(std::min<uint32_t>(rows, 1u << 20)), dim3(512), 0, st, x, out, rows, size);
    return hipGetLastError();
  }
  const uint64_t of = ((uint64_t)(size - 1) / kBlock + 1) * kBlockLanes<DT>;
  const Split split{of, 1.0 / (double)of};
  const dim3 grid = grid_of((of * rows + kPackThreads - 1) / kPackThreads), block(kPackThreads);
  if ((uint64_t)rows * size * (kElem<DT> + 1) > kStreamBytes)
    hipLaunchKernelGGL((k_pack8<DT, true>), grid, block, 0, st, x, out, rows, size, split);
  else
    hipLaunchKernelGGL((k_pack8<DT, false>), grid, block, 0, st, x, out, rows, size, split);
  return hipGetLastError();
}

template <int DT>
hipError_t unpack(const Eight& x, const Rows& out, uint32_t rows, uint32_t size, hipStream_t st) {
  const uint64_t of = (size - 1) / kUnit<DT> + 1;
  const Split split{of, 1.0 / (double)of};
  const dim3 grid = grid_of((of * rows + kPackThreads - 1) / kPackThreads), block(kPackThreads);
  if ((uint64_t)rows * size * (kElem<DT> + 1) > kStreamBytes)
    hipLaunchKernelGGL((k_unpack8<DT, true>), grid, block, 0, st, x, out, rows, size, split);
  else
    hipLaunchKernelGGL((k_unpack8<DT, false>), grid, block, 0, st, x, out, rows, size, split);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_pack8(const Rows& x, const Eight& out, uint32_t rows, uint32_t size, int32_t dtype, hipStream_t st) {
  switch (dtype) {
    case GCLIP_F32: return pack<GCLIP_F32>(x, out, rows, size, st);
    case GCLIP_F16: return pack<GCLIP_F16>(x, out, rows, size, st);
    default: return pack<GCLIP_BF16>(x, out, rows, size, st);
  }
}

hipError_t launch_unpack8(const Eight& x, const Rows& out, uint32_t rows, uint32_t size, int32_t dtype,
                          hipStream_t st) {
  switch (dtype) {
    case GCLIP_F32: return unpack<GCLIP_F32>(x, out, rows, size, st);
    case GCLIP_F16: return unpack<GCLIP_F16>(x, out, rows, size, st);
    default: return unpack<GCLIP_BF16>(x, out, rows, size, st);
  }
}

hipError_t launch_activation(const ActArgs& a, int32_t dtype, int32_t kind, bool backward, bool streamed,
                             hipStream_t st) {
  switch (dtype) {
    case GCLIP_F32: return activation_of<GCLIP_F32>(a, kind, backward, streamed, st);
    case GCLIP_F16: return activation_of<GCLIP_F16>(a, kind, backward, streamed, st);
    default: return activation_of<GCLIP_BF16>(a, kind, backward, streamed, st);
  }
}

}  // namespace gclip
