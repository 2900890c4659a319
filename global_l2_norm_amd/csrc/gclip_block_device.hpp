// gclip_block_device.hpp -- device code shared by the block kernels
// (include/gclip_block.h): matrices in 8 bits.
#pragma once

#include "gclip_block.hpp"
#include "gclip_layer_device.hpp"

namespace gclip {

constexpr uint32_t kBlock = GCLIP_SCALE_BLOCK;

// Magnitudes are compared as bit patterns, which order the finite ones, the
// infinity and the NaNs: no instruction quiets or drops a NaN on the way, and
// two 16-bit elements take one operation.  A largest magnitude that is not
// finite is found again among the finite ones.
template <int DT>
constexpr uint32_t kInfBits = DT == GCLIP_F32 ? 0x7f800000u : DT == GCLIP_F16 ? 0x7c00u : 0x7f80u;

__device__ __forceinline__ uint32_t max_pair(uint32_t a, uint32_t b) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

// The largest magnitude of a unit of stored elements, as the format's bits.
template <int DT>
__device__ __forceinline__ uint32_t unit_magnitude(const u32x4& q) {
  if constexpr (DT == GCLIP_F32) {
    return max(max(q[0] & 0x7fffffffu, q[1] & 0x7fffffffu), max(q[2] & 0x7fffffffu, q[3] & 0x7fffffffu));
  } else {
    const uint32_t m = 0x7fff7fffu;
    const uint32_t t = max_pair(max_pair(q[0] & m, q[1] & m), max_pair(q[2] & m, q[3] & m));
    return max(t & 0xffffu, t >> 16);
  }
}

// The same of the finite ones alone.
template <int DT>
__device__ __forceinline__ uint32_t unit_magnitude_finite(const u32x4& q) {
  uint32_t most = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == GCLIP_F32) {
      const uint32_t b = q[k] & 0x7fffffffu;
      most = max(most, b < kInfBits<DT> ? b : 0u);
    } else {
      const uint32_t lo = q[k] & 0x7fffu, hi = (q[k] >> 16) & 0x7fffu;
      most = max(most, max(lo < kInfBits<DT> ? lo : 0u, hi < kInfBits<DT> ? hi : 0u));
    }
  }
  return most;
}

// The largest of the N lanes of an aligned run, in all of them.
template <int N>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  const auto by = [](uint32_t a, int b) { return max(a, (uint32_t)b); };
  if constexpr (N >= 2) v = by(v, __builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));
  if constexpr (N >= 4) v = by(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));
  if constexpr (N >= 8) v = by(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));
  if constexpr (N >= 16) v = by(v, __builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));
  if constexpr (N >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    v = max(s[0], s[1]);
  }
  if constexpr (N >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    v = max(s[0], s[1]);
  }
  return v;
}

// most / 448 by the rounded reciprocal: within 2 u of it, and a division less.
__device__ __forceinline__ float scale_of(float most) {
  const float s = most * (1.0f / 448.0f);
  return s > 0x1p-112f ? s : 0x1p-112f;
}

// Four values in e4m3, the first in the lowest byte.  The conversion rounds
// to nearest even; what it is given is at most 448 but for the roundings of
// the scale's reciprocal and the product, which come to less than half a step
// there, or not finite, which gives a NaN.
__device__ __forceinline__ uint32_t eight_word(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// A unit's values in 8 bits: a word of binary32's four, two of the others'
// eight.
template <int DT>
struct Unit8 {
  uint32_t w[DT == GCLIP_F32 ? 1 : 2];
};

template <int DT>
__device__ __forceinline__ Unit8<DT> unit_eight(const float (&v)[kUnit<DT>], float inverse) {
  Unit8<DT> u;
#pragma unroll
  for (uint32_t i = 0; i < kUnit<DT> / 4; ++i)
    u.w[i] = eight_word(v[4 * i] * inverse, v[4 * i + 1] * inverse, v[4 * i + 2] * inverse, v[4 * i + 3] * inverse);
  return u;
}

// The values that a unit stands for.
template <int DT>
__device__ __forceinline__ void unit_value(const Unit8<DT>& u, float scale, float (&v)[kUnit<DT>]) {
#pragma unroll
  for (uint32_t i = 0; i < kUnit<DT> / 4; ++i) {
    const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)u.w[i], false);
    const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)u.w[i], true);
    v[4 * i] = lo[0] * scale;
    v[4 * i + 1] = lo[1] * scale;
    v[4 * i + 2] = hi[0] * scale;
    v[4 * i + 3] = hi[1] * scale;
  }
}

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The unit that begins at column c (a multiple of the unit's columns) of a
// row of values: inside the row's groups of eight bytes where c < size.
template <int DT, bool NT>
__device__ __forceinline__ Unit8<DT> load_eight(uint64_t row, uint32_t c) {
  Unit8<DT> u;
  if constexpr (DT == GCLIP_F32) {
    const g_u32* p = reinterpret_cast<const g_u32*>(row + c);
    u.w[0] = NT ? __builtin_nontemporal_load(p) : *p;
  } else {
    typedef __attribute__((address_space(1))) u32x2 g_t;
    const g_t* p = reinterpret_cast<const g_t*>(row + c);
    const u32x2 q = NT ? __builtin_nontemporal_load(p) : *p;
    u.w[0] = q[0];
    u.w[1] = q[1];
  }
  return u;
}

template <int DT, bool NT>
__device__ __forceinline__ void store_eight(uint64_t row, uint32_t c, const Unit8<DT>& u) {
  if constexpr (DT == GCLIP_F32) {
    g_u32* p = reinterpret_cast<g_u32*>(row + c);
    if constexpr (NT) __builtin_nontemporal_store(u.w[0], p);
    else *p = u.w[0];
  } else {
    typedef __attribute__((address_space(1))) u32x2 g_t;
    g_t* p = reinterpret_cast<g_t*>(row + c);
    const u32x2 q{u.w[0], u.w[1]};
    if constexpr (NT) __builtin_nontemporal_store(q, p);
    else *p = q;
  }
}

// The same with nothing in the bytes past the row's end.
template <int DT>
__device__ __forceinline__ void settle_eight(Unit8<DT>& u, uint32_t c, uint32_t size) {
#pragma unroll
  for (uint32_t i = 0; i < kUnit<DT> / 4; ++i) {
    const uint32_t first = c + 4 * i, left = first < size ? size - first : 0u;
    if (left < 4) u.w[i] &= left == 0 ? 0u : 0xffffffffu >> (8 * (4 - left));
  }
}

__device__ __forceinline__ float load_scale(const Eight& e, uint64_t row, uint32_t c) {
  typedef __attribute__((address_space(1))) float g_t;
  return reinterpret_cast<const g_t*>(e.scales)[row * e.count + (e.row ? 0u : c / kBlock)];
}

__device__ __forceinline__ void store_scale(const Eight& e, uint64_t row, uint32_t block, float scale) {
  typedef __attribute__((address_space(1))) float g_t;
  reinterpret_cast<g_t*>(e.scales)[row * e.count + block] = scale;
}

// Lanes that hold a block, one unit each.
template <int DT>
constexpr int kBlockLanes = (int)(kBlock / kUnit<DT>);

// The scale of a block whose units an aligned run of lanes holds, one each.
template <int DT, int LANES>
__device__ __forceinline__ float block_scale(const u32x4& q) {
  uint32_t m = lanes_max<LANES>(unit_magnitude<DT>(q));
  if (m >= kInfBits<DT>) m = lanes_max<LANES>(unit_magnitude_finite<DT>(q));  // the run's lanes together
  return scale_of(elem_float<DT>(m));
}

// ---------------------------------------------------------------- elementwise kernels
// A lane takes a unit of a row, which it finds by a division: of a number
// below 2^52 by one of at most 2^31, through binary64 and to the nearest
// half, which is further from any whole quotient than its roundings are.
struct Split {
  uint64_t of;     // units (or lanes) of a row
  double inverse;  // 1 / of
};
__device__ __forceinline__ uint32_t row_of(uint64_t i, const Split& s) {
  return (uint32_t)(((double)i + 0.5) * s.inverse);
}

// The unit at column c of a row, zeros past the row's end; c < size.
template <int DT, bool NT>
__device__ __forceinline__ u32x4 load_unit_at(uint64_t row, uint32_t c, uint32_t size) {
  constexpr uint32_t kU = kUnit<DT>;
  if (size % kU == 0) return load16<DT, NT>(row + (uint64_t)c * kElem<DT>);
  if (size < kGroup) return load_unit<DT, NT>(row, c / kU, size);
  const bool ends = c + kU > size;
  u32x4 q = load16<DT, NT>(row + (uint64_t)(ends ? size - kU : c) * kElem<DT>);
  if (ends) q = moved_down<DT>(q, kU - size % kU);
  return q;
}

}  // namespace gclip
