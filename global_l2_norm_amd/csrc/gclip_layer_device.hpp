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
    for (int k = 0; k < 4; ++k) r.q[0][k] = elem_bits<DT>(v[2 * k]) | (elem_bits<DT>(v[2 * k + 1]) << 16);
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

// The n (1 to 7) elements at a, zeros after them.  Elements in front of a
// belong to the same row when front is set: then one vector ending at the
// row's end is read and shifted, which keeps the tail's load in step with the
// others; a row of fewer than eight elements is read one by one.
template <int DT>
__device__ __forceinline__ Raw8<DT> load_tail(uint64_t a, uint32_t n, bool front) {
  Raw8<DT> r = zero8<DT>();
  if (front) {
    const Raw8<DT> s = load8<DT, false>(a - (uint64_t)(kGroup - n) * kElem<DT>);
    if constexpr (DT == GCLIP_F32) {
      uint32_t v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = s.q[k >> 2][k & 3];
      const uint32_t sh = kGroup - n;
#pragma unroll
      for (uint32_t b = 4; b > 0; b >>= 1) {
        if (sh & b) {
#pragma unroll
          for (uint32_t k = 0; k < 8; ++k) v[k] = k + b < 8 ? v[k + b < 8 ? k + b : 0] : 0u;
        }
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) r.q[k >> 2][k & 3] = v[k];
    } else {
      uint64_t lo = (uint64_t)s.q[0][0] | ((uint64_t)s.q[0][1] << 32);
      uint64_t hi = (uint64_t)s.q[0][2] | ((uint64_t)s.q[0][3] << 32);
      const uint32_t sh = 16u * (kGroup - n);  // 16 to 112 bits
      if (sh >= 64) {
        lo = hi >> (sh - 64);
        hi = 0;
      } else {
        lo = (lo >> sh) | (hi << (64 - sh));
        hi >>= sh;
      }
      r.q[0] = u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
    }
  } else {
#pragma unroll
    for (uint32_t k = 0; k < 7; ++k) {
      if (k < n) {
        const uint32_t e = load_elem<DT>(a + (uint64_t)k * kElem<DT>);
        if constexpr (DT == GCLIP_F32) r.q[k >> 2][k & 3] = e;
        else r.q[0][k >> 1] |= e << (16 * (k & 1));
      }
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

}  // namespace gclip
