// gclip_layer_device.hpp -- device code shared by the layer kernels
// (include/gclip_layer.h): groups of eight columns in registers, the
// counter-based generator and the dropout map.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "gclip_device.hpp"
#include "gclip_layer.hpp"

namespace gclip {

// A lane works on groups of eight adjacent columns: one 16-byte access of a
// 16-bit format (two of binary32), and one call of the generator.  Rows may
// begin at any element, so the vector types carry the element's alignment
// only; gfx950 does such accesses in one instruction, and aligned addresses
// lose nothing by it.
constexpr uint32_t kGroup = 8;
typedef u32x4 u32x4_any2 __attribute__((aligned(2)));
typedef u32x4 u32x4_any4 __attribute__((aligned(4)));
typedef uint64_t u64_any2 __attribute__((aligned(2)));
typedef uint64_t u64_any4 __attribute__((aligned(4)));
typedef uint32_t u32_any2 __attribute__((aligned(2)));

// Number of this workgroup in a layer of a grid_of().
__device__ __forceinline__ uint64_t workgroup_of_grid() { return (uint64_t)blockIdx.y * gridDim.x + blockIdx.x; }

template <int DT>
constexpr uint32_t kElem = DT == GCLIP_F32 ? 4u : 2u;

// The storage of eight elements.
template <int DT>
struct Raw8 {
  u32x4 q[DT == GCLIP_F32 ? 2 : 1];
};

template <int DT>
__device__ __forceinline__ float elem_float(uint32_t bits) {
  if constexpr (DT == GCLIP_F32) return __uint_as_float(bits);
  else if constexpr (DT == GCLIP_F16) return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  else return __uint_as_float(bits << 16);
}

template <int DT>
__device__ __forceinline__ uint32_t elem_bits(float v) {
  if constexpr (DT == GCLIP_F32) return __float_as_uint(v);
  else if constexpr (DT == GCLIP_F16) return (uint32_t)__builtin_bit_cast(uint16_t, (_Float16)v);
  else return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)v);
}

// Two values rounded to a 16-bit format, in one conversion.
template <int DT>
__device__ __forceinline__ uint32_t pair_bits(float lo, float hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
  if constexpr (DT == GCLIP_F16) {
    typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), f16x2));
  } else {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
  }
}

template <int DT>
__device__ __forceinline__ void unpack(const Raw8<DT>& r, float (&v)[8]) {
  if constexpr (DT == GCLIP_F32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = __uint_as_float(r.q[k >> 2][k & 3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[2 * k] = elem_float<DT>(r.q[0][k] & 0xffffu);
      v[2 * k + 1] = elem_float<DT>(r.q[0][k] >> 16);
    }
  }
}

template <int DT>
__device__ __forceinline__ Raw8<DT> pack(const float (&v)[8]) {
  Raw8<DT> r;
  if constexpr (DT == GCLIP_F32) {
#pragma unroll
    for (int k = 0; k < 8; ++k) r.q[k >> 2][k & 3] = __float_as_uint(v[k]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) r.q[0][k] = pair_bits<DT>(v[2 * k], v[2 * k + 1]);
  }
  return r;
}

template <int DT>
__device__ __forceinline__ Raw8<DT> zero8() {
  Raw8<DT> r;
  r.q[0] = u32x4{0u, 0u, 0u, 0u};
  if constexpr (DT == GCLIP_F32) r.q[1] = u32x4{0u, 0u, 0u, 0u};
  return r;
}

// Eight elements from an address of the element's alignment.
template <int DT, bool NT>
__device__ __forceinline__ Raw8<DT> load8(uint64_t a) {
  Raw8<DT> r;
  if constexpr (DT == GCLIP_F32) {
    typedef __attribute__((address_space(1))) u32x4_any4 g_t;
    const g_t* p = reinterpret_cast<const g_t*>(a);
    r.q[0] = NT ? __builtin_nontemporal_load(p) : *p;
    r.q[1] = NT ? __builtin_nontemporal_load(p + 1) : p[1];
  } else {
    typedef __attribute__((address_space(1))) u32x4_any2 g_t;
    const g_t* p = reinterpret_cast<const g_t*>(a);
    r.q[0] = NT ? __builtin_nontemporal_load(p) : *p;
  }
  return r;
}

template <int DT, bool NT>
__device__ __forceinline__ void store8(uint64_t a, const Raw8<DT>& r) {
  if constexpr (DT == GCLIP_F32) {
    typedef __attribute__((address_space(1))) u32x4_any4 g_t;
    g_t* p = reinterpret_cast<g_t*>(a);
    if constexpr (NT) {
      __builtin_nontemporal_store(r.q[0], p);
      __builtin_nontemporal_store(r.q[1], p + 1);
    } else {
      p[0] = r.q[0];
      p[1] = r.q[1];
    }
  } else {
    typedef __attribute__((address_space(1))) u32x4_any2 g_t;
    g_t* p = reinterpret_cast<g_t*>(a);
    if constexpr (NT) __builtin_nontemporal_store(r.q[0], p);
    else *p = r.q[0];
  }
}

// The elements of 16 or 32 bytes moved down by n places, zeros after them or,
// with ROUND, those that were moved out.  n is the same in every lane (what a row's ragged end lacks), and moves by
// words and half words: a 64-bit shift by a vector register gave wrong bits
// on gfx950 when that register was the last one of the wave's allocation.
template <int DT, bool ROUND = false>
__device__ __forceinline__ u32x4 moved_down(u32x4 q, uint32_t n) {
  const uint32_t bits = __builtin_amdgcn_readfirstlane(n * 8u * kElem<DT>);
  if (bits & 64u) q = u32x4{q[2], q[3], ROUND ? q[0] : 0u, ROUND ? q[1] : 0u};
  if (bits & 32u) q = u32x4{q[1], q[2], q[3], ROUND ? q[0] : 0u};
  if (DT != GCLIP_F32 && (bits & 16u))
    q = u32x4{(q[0] >> 16) | (q[1] << 16), (q[1] >> 16) | (q[2] << 16), (q[2] >> 16) | (q[3] << 16),
              (q[3] >> 16) | (ROUND ? q[0] << 16 : 0u)};
  return q;
}

template <int DT>
__device__ __forceinline__ Raw8<DT> moved_down(Raw8<DT> r, uint32_t n) {
  if constexpr (DT == GCLIP_F32) {
    if (__builtin_amdgcn_readfirstlane(n) & 4u) {
      r.q[0] = r.q[1];
      r.q[1] = u32x4{0u, 0u, 0u, 0u};
    }
    const uint32_t by = __builtin_amdgcn_readfirstlane(n) & 3u;
    const uint32_t v[8] = {r.q[0][0], r.q[0][1], r.q[0][2], r.q[0][3], r.q[1][0], r.q[1][1], r.q[1][2], r.q[1][3]};
    if (by == 1) r = Raw8<DT>{{u32x4{v[1], v[2], v[3], v[4]}, u32x4{v[5], v[6], v[7], 0u}}};
    if (by == 2) r = Raw8<DT>{{u32x4{v[2], v[3], v[4], v[5]}, u32x4{v[6], v[7], 0u, 0u}}};
    if (by == 3) r = Raw8<DT>{{u32x4{v[3], v[4], v[5], v[6]}, u32x4{v[7], 0u, 0u, 0u}}};
  } else {
    r.q[0] = moved_down<DT>(r.q[0], n);
  }
  return r;
}

// The n (1 to 7) elements at a, zeros after them.  Elements in front of a
// belong to the same row when front is set: then one vector ending at the
// row's end is read and moved down; a row of fewer than eight elements is read
// one by one.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_tail(uint64_t a, uint32_t n, bool front) {
  if (front) return moved_down<DT>(load8<DT, false>(a - (uint64_t)(kGroup - n) * kElem<DT>), kGroup - n);
  Raw8<DT> r = zero8<DT>();
#pragma unroll
  for (uint32_t k = 0; k < 7; ++k) {
    if (k < n) {
      const uint32_t e = load_elem<DT>(a + (uint64_t)k * kElem<DT>);
      if constexpr (DT == GCLIP_F32) r.q[k >> 2][k & 3] = e;
      else r.q[0][k >> 1] |= e << (16 * (k & 1));
    }
  }
  return r;
}

// The first n (1 to 7) elements of r, in pieces of four, two and one.
template <int DT>
__device__ __forceinline__ void store_tail(uint64_t a, const Raw8<DT>& r, uint32_t n) {
  if constexpr (DT == GCLIP_F32) {
    uint32_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = r.q[k >> 2][k & 3];
#pragma unroll
    for (uint32_t k = 0; k < 7; ++k)
      if (k < n) store_elem<DT>(a + (uint64_t)k * 4u, v[k]);
  } else {
    uint64_t lo = (uint64_t)r.q[0][0] | ((uint64_t)r.q[0][1] << 32);
    uint64_t hi = (uint64_t)r.q[0][2] | ((uint64_t)r.q[0][3] << 32);
    if (n & 4) {
      typedef __attribute__((address_space(1))) u64_any2 g_t;
      *reinterpret_cast<g_t*>(a) = lo;
      a += 8;
      lo = hi;
    }
    if (n & 2) {
      typedef __attribute__((address_space(1))) u32_any2 g_t;
      *reinterpret_cast<g_t*>(a) = (uint32_t)lo;
      a += 4;
      lo >>= 32;
    }
    if (n & 1) store_elem<DT>(a, (uint32_t)lo & 0xffffu);
  }
}

// Group g of a row of `size` columns that begins at `row`: zeros past its end.
template <int DT, bool NT>
__device__ __forceinline__ Raw8<DT> load_group8(uint64_t row, uint32_t g, uint32_t size) {
  const uint32_t c = g * kGroup;
  if (c + kGroup <= size) return load8<DT, NT>(row + (uint64_t)c * kElem<DT>);
  if (c < size) return load_tail<DT>(row + (uint64_t)c * kElem<DT>, size - c, size >= kGroup);
  return zero8<DT>();
}

template <int DT, bool NT>
__device__ __forceinline__ void store_group8(uint64_t row, uint32_t g, uint32_t size, const Raw8<DT>& r) {
  const uint32_t c = g * kGroup;
  if (c + kGroup <= size) store8<DT, NT>(row + (uint64_t)c * kElem<DT>, r);
  else if (c < size) store_tail<DT>(row + (uint64_t)c * kElem<DT>, r, size - c);
}

// Columns of a unit of 16 bytes: a group, or half of one of binary32.
template <int DT>
constexpr uint32_t kUnit = DT == GCLIP_F32 ? 4u : 8u;

// Unit u of a row: zeros past its end.
template <int DT, bool NT>
__device__ __forceinline__ u32x4 load_unit(uint64_t row, uint32_t u, uint32_t size) {
  if constexpr (DT == GCLIP_F32) {
    typedef __attribute__((address_space(1))) u32x4_any4 g_t;
    const uint32_t c = u * kUnit<DT>;
    if (c + 4 <= size) {
      const g_t* p = reinterpret_cast<const g_t*>(row + c * 4ull);
      return NT ? __builtin_nontemporal_load(p) : *p;
    }
    u32x4 q{0u, 0u, 0u, 0u};
#pragma unroll
    for (uint32_t k = 0; k < 3; ++k)
      if (c + k < size) q[k] = load_elem<DT>(row + (c + k) * 4ull);
    return q;
  } else {
    return load_group8<DT, NT>(row, u, size).q[0];
  }
}
template <int DT, bool NT>
__device__ __forceinline__ void store_unit(uint64_t row, uint32_t u, uint32_t size, const u32x4& q) {
  if constexpr (DT == GCLIP_F32) {
    typedef __attribute__((address_space(1))) u32x4_any4 g_t;
    const uint32_t c = u * 4;
    if (c + 4 <= size) {
      g_t* p = reinterpret_cast<g_t*>(row + c * 4ull);
      if constexpr (NT) __builtin_nontemporal_store(q, p);
      else *p = q;
    } else {
#pragma unroll
      for (uint32_t k = 0; k < 3; ++k)
        if (c + k < size) store_elem<DT>(row + (c + k) * 4ull, q[k]);
    }
  } else {
    store_group8<DT, NT>(row, u, size, Raw8<DT>{{q}});
  }
}

// ---------------------------------------------------------------- weights
// Eight elements of weight or bias (binary32 or the matrices' format; `def`
// where there is none).
template <int DT>
__device__ __forceinline__ void weight_group(uint64_t w, int wdt, uint32_t g, uint32_t size, float def, float (&v)[8]) {
  if (w == 0) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = def;
  } else if (DT == GCLIP_F32 || wdt == GCLIP_F32) {
    unpack<GCLIP_F32>(load_group8<GCLIP_F32, false>(w, g, size), v);
  } else {
    unpack<DT>(load_group8<DT, false>(w, g, size), v);
  }
}

// ---------------------------------------------------------------- dropout
// Philox4x32-10 as published: ten rounds of two 32 x 32 -> 64-bit products.
struct Words4 {
  uint32_t w[4];
};
__device__ __forceinline__ Words4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = (uint64_t)0xD2511F53u * c0, b = (uint64_t)0xCD9E8D57u * c2;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return Words4{{c0, c1, c2, c3}};
}

__device__ __forceinline__ uint32_t drop_step(const DropArgs& d) { return d.step + (d.d_step ? *d.d_step : 0u); }

// The generator's halves for one half of a group.
__device__ __forceinline__ uint64_t philox_half(const DropArgs& d, uint32_t step, uint32_t row, uint32_t g,
                                                uint32_t h) {
  const Words4 b = philox(g, row, d.site, step, d.k0, d.k1);
  const uint64_t lo = (uint64_t)b.w[0] | ((uint64_t)b.w[1] << 32), hi = (uint64_t)b.w[2] | ((uint64_t)b.w[3] << 32);
  return h ? hi : lo;
}

// v * scale where kept, else 0 (a select: a dropped NaN is 0).  The product
// is rounded before whatever is added to it, so the residual step's h does
// not depend on what the compiler contracts.
__device__ __forceinline__ void drop_group(const DropArgs& d, uint32_t step, uint32_t row, uint32_t g, float (&v)[8]) {
#pragma clang fp contract(off)
  const Words4 b = philox(g, row, d.site, step, d.k0, d.k1);
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t u = k & 1 ? b.w[k >> 1] >> 16 : b.w[k >> 1] & 0xffffu;
    v[k] = u >= d.threshold ? v[k] * d.scale : 0.0f;
  }
}

template <int DT>
__device__ __forceinline__ void drop_unit(const DropArgs& d, uint32_t step, uint32_t row, uint32_t c,
                                          float (&v)[kUnit<DT>]) {
#pragma clang fp contract(off)
  if constexpr (DT == GCLIP_F32) {
    const uint64_t b = philox_half(d, step, row, c / kGroup, c & 4u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t u = (uint32_t)(b >> (16 * j)) & 0xffffu;
      v[j] = u >= d.threshold ? v[j] * d.scale : 0.0f;
    }
  } else {
    drop_group(d, step, row, c / kGroup, v);
  }
}

// ---------------------------------------------------------------- rows in registers
// A row of at least eight columns is held by LANES lanes, NV units of 16
// bytes each: lane l takes the units l, l + LANES, ..., so a wave's accesses
// are adjacent.  Loads are unconditional -- a lane whose unit passes the
// row's end reads the row's last 16 bytes instead -- and settled afterwards:
// shifted where the unit is the row's ragged end, zero past it.  So a row's
// loads are all under way before anything is waited for, and none leaves the
// row.
template <int DT>
__device__ __forceinline__ uint32_t column_of(uint32_t lane, uint32_t lanes, int k) {
  return (lane + (uint32_t)k * lanes) * kUnit<DT>;
}

template <int DT>
__device__ __forceinline__ void unpack_unit(const u32x4& q, float (&v)[kUnit<DT>]) {
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == GCLIP_F32) {
      v[k] = __uint_as_float(q[k]);
    } else {
      v[2 * k] = elem_float<DT>(q[k] & 0xffffu);
      v[2 * k + 1] = elem_float<DT>(q[k] >> 16);
    }
  }
}

template <int DT>
__device__ __forceinline__ u32x4 pack_unit(const float (&v)[kUnit<DT>]) {
  u32x4 q;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (DT == GCLIP_F32) q[k] = __float_as_uint(v[k]);
    else q[k] = pair_bits<DT>(v[2 * k], v[2 * k + 1]);
  }
  return q;
}

template <int DT, bool NT>
__device__ __forceinline__ u32x4 load16(uint64_t at) {
  if constexpr (DT == GCLIP_F32) {
    typedef __attribute__((address_space(1))) u32x4_any4 g_t;
    const g_t* p = reinterpret_cast<const g_t*>(at);
    return NT ? __builtin_nontemporal_load(p) : *p;
  } else {
    typedef __attribute__((address_space(1))) u32x4_any2 g_t;
    const g_t* p = reinterpret_cast<const g_t*>(at);
    return NT ? __builtin_nontemporal_load(p) : *p;
  }
}

template <int DT, bool NT>
__device__ __forceinline__ void store16(uint64_t at, const u32x4& q) {
  if constexpr (DT == GCLIP_F32) {
    typedef __attribute__((address_space(1))) u32x4_any4 g_t;
    g_t* p = reinterpret_cast<g_t*>(at);
    if constexpr (NT) __builtin_nontemporal_store(q, p);
    else *p = q;
  } else {
    typedef __attribute__((address_space(1))) u32x4_any2 g_t;
    g_t* p = reinterpret_cast<g_t*>(at);
    if constexpr (NT) __builtin_nontemporal_store(q, p);
    else *p = q;
  }
}

// The units k < SURE lie in every row that a shape is used for (the shape
// before it would hold the others): nothing is clamped or settled there.
template <int DT, int LANES, int SURE, bool NT>
__device__ __forceinline__ u32x4 load_columns(uint64_t row, uint32_t lane, int k, uint32_t size) {
  if (k < SURE) return load16<DT, NT>(row + (uint64_t)(k * LANES * 16) + lane * 16u);
  const uint32_t c = column_of<DT>(lane, LANES, k);
  return load16<DT, NT>(row + (c + kUnit<DT> <= size ? c : size - kUnit<DT>) * kElem<DT>);
}

// full: the row fills its shape, the same for a whole launch.
template <int DT, int LANES, int SURE>
__device__ __forceinline__ void settle(u32x4& q, uint32_t lane, int k, uint32_t size, bool full = false) {
  if (k < SURE || full) return;
  const uint32_t c = column_of<DT>(lane, LANES, k);
  if (c + kUnit<DT> > size)
    q = c < size ? moved_down<DT>(q, kUnit<DT> - size % kUnit<DT>) : u32x4{0u, 0u, 0u, 0u};
}

// As settle(), but in the unit of the row's end other elements of the row
// come after it, not zeros: for the matrix that was normed, where a zero's
// (0 - mean) rstd may be infinite though every element's is finite, and
// nothing times that is NaN in the row's sums.
template <int DT, int LANES, int SURE>
__device__ __forceinline__ void settle_round(u32x4& q, uint32_t lane, int k, uint32_t size, bool full) {
  if (k < SURE || full) return;
  const uint32_t c = column_of<DT>(lane, LANES, k);
  if (c + kUnit<DT> > size)
    q = c < size ? moved_down<DT, true>(q, kUnit<DT> - size % kUnit<DT>) : u32x4{0u, 0u, 0u, 0u};
}

template <int DT, int LANES, int SURE, bool NT>
__device__ __forceinline__ void store_columns(uint64_t row, uint32_t lane, int k, uint32_t size, const u32x4& q) {
  const uint32_t c = column_of<DT>(lane, LANES, k);
  if (k < SURE) store16<DT, NT>(row + (uint64_t)(k * LANES * 16) + lane * 16u, q);
  else if (c < size) store_unit<DT, NT>(row, c / kUnit<DT>, size, q);
}

// The columns of unit k of weight or bias as settle() leaves a row's.
template <int DT, int LANES, int SURE>
__device__ __forceinline__ void weight_columns(uint64_t w, int wdt, uint32_t lane, int k, uint32_t size, float def,
                                               float (&v)[kUnit<DT>]) {
  if (w == 0) {
#pragma unroll
    for (uint32_t j = 0; j < kUnit<DT>; ++j) v[j] = def;
  } else if (DT != GCLIP_F32 && wdt == GCLIP_F32) {
    if constexpr (DT != GCLIP_F32) {
      const uint32_t c = column_of<DT>(lane, LANES, k);
      Raw8<GCLIP_F32> r = load8<GCLIP_F32, false>(w + (k < SURE || c + kGroup <= size ? c : size - kGroup) * 4ull);
      if (k >= SURE && c + kGroup > size)
        r = c < size ? moved_down<GCLIP_F32>(r, kGroup - size % kGroup) : zero8<GCLIP_F32>();
      unpack<GCLIP_F32>(r, v);
    }
  } else {
    u32x4 q = load_columns<DT, LANES, SURE, false>(w, lane, k, size);
    settle<DT, LANES, SURE>(q, lane, k, size);
    unpack_unit<DT>(q, v);
  }
}

// Sum over each aligned run of N lanes of a wave, the same bits in all of
// them (a + b == b + a at every level), by register permutations alone:
// quads, mirrored halves and rows of sixteen, then swaps between the rows.
template <int CTRL>
__device__ __forceinline__ float permuted(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, 0xf, 0xf, true));
}
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (N >= 2) v += permuted<0xB1>(v);   // quad_perm 1,0,3,2
  if constexpr (N >= 4) v += permuted<0x4E>(v);   // quad_perm 2,3,0,1
  if constexpr (N >= 8) v += permuted<0x141>(v);  // row_half_mirror
  if constexpr (N >= 16) v += permuted<0x140>(v); // row_mirror
  if constexpr (N >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if constexpr (N >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return v;
}

// The sum of a row's waves, from the words that they left.
template <int LANES>
__device__ __forceinline__ float waves_sum(const float* own) {
  float v = own[0];
#pragma unroll
  for (int i = 1; i < LANES / 64; ++i) v += own[i];
  return v;
}

// Sum over the LANES lanes of a row, the same bits in all of them.  Rows of
// more than a wave meet in `red`, a word for each wave of the workgroup; one
// barrier, so two sums in a row need two `red`s, and the third may use the
// first again.
template <int LANES>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = lanes_sum<(LANES < 64 ? LANES : 64)>(v);
  if constexpr (LANES > 64) {
    constexpr int kWavesOfRow = LANES / 64;
    const uint32_t wave = threadIdx.x >> 6;
    if ((threadIdx.x & 63) == 0) red[wave] = v;
    __syncthreads();
    v = waves_sum<LANES>(red + wave / kWavesOfRow * kWavesOfRow);
  }
  return v;
}

// Two of them behind one barrier.
template <int LANES>
__device__ __forceinline__ void row_sums(float& p, float& q, float* redp, float* redq) {
  p = lanes_sum<(LANES < 64 ? LANES : 64)>(p);
  q = lanes_sum<(LANES < 64 ? LANES : 64)>(q);
  if constexpr (LANES > 64) {
    constexpr int kWavesOfRow = LANES / 64;
    const uint32_t wave = threadIdx.x >> 6, own = wave / kWavesOfRow * kWavesOfRow;
    if ((threadIdx.x & 63) == 0) {
      redp[wave] = p;
      redq[wave] = q;
    }
    __syncthreads();
    p = redp[own];
    q = redq[own];
#pragma unroll
    for (int i = 1; i < kWavesOfRow; ++i) {
      p += redp[own + i];
      q += redq[own + i];
    }
  }
}

// t / n by n's reciprocal and one correction, exact where n divides t (a
// constant row's mean is its value), in a quarter of a division's operations.
__device__ __forceinline__ float divided(float t, float n, float inverse) {
  const float q = t * inverse;
  return __builtin_fmaf(__builtin_fmaf(-q, n, t), inverse, q);
}

// (x - mean) rstd, from half of the mean and twice rstd: x - mean alone may
// leave binary32 (elements at both of its ends).  The same bits otherwise,
// as both factors are powers of two.
__device__ __forceinline__ float normed(float x, float half_mean, float twice_rstd) {
  return __builtin_fmaf(x, 0.5f, -half_mean) * twice_rstd;
}

// Sum over the lanes of a wave that hold the same column of its 64 / LANES
// rows, in the first LANES lanes.
template <int LANES>
__device__ __forceinline__ float across_rows(float v) {
  if constexpr (LANES <= 1) v += permuted<0x121>(v);  // row_ror 1, 2, 4, 8
  if constexpr (LANES <= 2) v += permuted<0x122>(v);
  if constexpr (LANES <= 4) v += permuted<0x124>(v);
  if constexpr (LANES <= 8) v += permuted<0x128>(v);
  if constexpr (LANES <= 16) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  if constexpr (LANES <= 32) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = __uint_as_float(s[0]) + __uint_as_float(s[1]);
  }
  return v;
}

// A column's gradient into dweight (which 0) or dbias (1), unless unwanted.
template <int DT>
__device__ __forceinline__ void store_weight_grad(const BwdArgs& a, uint32_t which, uint32_t c, float t) {
  const uint64_t out = which ? a.dbias : a.dweight;
  if (!out) return;
  if (DT == GCLIP_F32 || a.gdt == GCLIP_F32) {
    const uint64_t p = out + c * 4ull;
    if (a.accumulate) t += elem_float<GCLIP_F32>(load_elem<GCLIP_F32>(p));
    store_elem<GCLIP_F32>(p, elem_bits<GCLIP_F32>(t));
  } else {
    const uint64_t p = out + c * 2ull;
    if (a.accumulate) t += elem_float<DT>(load_elem<DT>(p));
    store_elem<DT>(p, elem_bits<DT>(t));
  }
}

}  // namespace gclip
