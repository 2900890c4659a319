// gclip_operand.hpp -- the operands of a call as the host checks them: their
// extents in bytes and which of them may not touch (internal to libgclip).
#pragma once

#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "gclip_block.hpp"
#include "gclip_host.hpp"

namespace gclip {

inline uint64_t address_of(const void* p) { return reinterpret_cast<uint64_t>(p); }
inline bool format_ok(int32_t t) { return t == GCLIP_F32 || t == GCLIP_F16 || t == GCLIP_BF16; }
inline bool weight_format_ok(int32_t w, int32_t t) { return w == GCLIP_F32 || w == t; }
inline uint64_t format_bytes(int32_t t) { return t == GCLIP_F32 ? 4u : 2u; }
inline bool extents_fit(int64_t rows, int64_t size) {
  return rows >= 0 && rows <= GCLIP_LAYER_MAX_EXTENT && size >= 1 && size <= GCLIP_LAYER_MAX_EXTENT;
}

// `rows` runs of `row` bytes, `ld` bytes from one to the next.  matrix: one
// that a call may read and write in place.
struct Span {
  uint64_t at = 0, ld = 0, row = 0, extent = 0;
  bool written = false, matrix = false;
  Rows device() const { return Rows{at, ld}; }
};

// Fills *s; false for an address, a distance or an extent that no call takes.
inline bool span_of(const void* p, uint64_t align, int64_t rows, uint64_t row, uint64_t ld, bool written, bool matrix,
                    Span* s) {
  *s = Span{address_of(p), 0, 0, 0, written, matrix};
  if (rows == 0 || row == 0) return true;
  const __uint128_t extent = (__uint128_t)(uint64_t)(rows - 1) * ld + row;
  if (!p || address_of(p) % align != 0 || (written && rows > 1 && ld < row)) return false;
  if (extent > (1ull << 60) || (__uint128_t)address_of(p) + extent > ~0ull) return false;
  s->ld = rows > 1 ? ld : row;
  s->row = row;
  s->extent = (uint64_t)extent;
  return true;
}

inline bool matrix_of(const void* p, int64_t ld, int64_t rows, int64_t size, uint64_t es, bool written, Span* s) {
  if (rows > 0 && (ld < 0 || ld > (int64_t)(1ull << 60))) return false;
  return span_of(p, es, rows, (uint64_t)size * es, (uint64_t)ld * es, written, true, s);
}

// A vector of n elements; none where p is null.
inline bool vector_of(const void* p, int64_t n, uint64_t es, bool written, Span* s) {
  *s = Span{};
  return !p || span_of(p, es, 1, (uint64_t)n * es, 0, written, false, s);
}

inline uint32_t scales_of(int64_t size, int32_t mode) {
  return mode == GCLIP_SCALES_ROW ? 1u : (uint32_t)((size + GCLIP_SCALE_BLOCK - 1) / GCLIP_SCALE_BLOCK);
}

// A matrix in 8 bits, its values and its scales; none where it has no values
// (and then no scales either).  any_mode: by row too.
inline bool packed_of(const gclip_packed8& p, int64_t rows, int64_t size, bool written, bool any_mode, Eight* e,
                      Span* values, Span* scales) {
  *e = Eight{};
  *values = *scales = Span{};
  if (!p.values) return !p.scales;
  if (p.mode != GCLIP_SCALES_BLOCK && !(any_mode && p.mode == GCLIP_SCALES_ROW)) return false;
  if (p.reserved != 0 || p.ld < 0 || (rows > 0 && (p.ld % 8 != 0 || (rows > 1 && p.ld < size)))) return false;
  const uint32_t n = scales_of(size, p.mode);
  if (!span_of(p.values, 8, rows, ((uint64_t)size + 7) / 8 * 8, (uint64_t)p.ld, written, false, values)) return false;
  if (!span_of(p.scales, 4, rows, 4ull * n, 4ull * n, written, false, scales)) return false;
  *e = Eight{address_of(p.values), rows > 1 ? (uint64_t)p.ld : 0u, address_of(p.scales), n,
             p.mode == GCLIP_SCALES_ROW ? 1u : 0u};
  return true;
}

// Whether two operands, one of them written, touch a byte in common -- other
// than as the same matrix, read and written in place.  Rows at one distance,
// each clear of the other's in the same row and in the next, are columns of
// one buffer.
inline bool touch(const Span& a, const Span& b) {
  if (!(a.written || b.written) || a.extent == 0 || b.extent == 0) return false;
  if (a.at + a.extent <= b.at || b.at + b.extent <= a.at) return false;
  if (a.matrix && b.matrix && a.at == b.at && a.ld == b.ld && a.extent == b.extent) return a.written && b.written;
  if (a.ld == b.ld && a.ld > 0 && a.extent > a.row && b.extent > b.row) {
    const uint64_t off = a.at > b.at ? (a.at - b.at) % a.ld : (a.ld - (b.at - a.at) % a.ld) % a.ld;
    return off < b.row || off + a.row > a.ld;
  }
  return true;
}

inline bool none_touch(std::initializer_list<Span> all) {
  for (auto i = all.begin(); i != all.end(); ++i)
    for (auto j = i + 1; j != all.end(); ++j)
      if (touch(*i, *j)) return false;
  return true;
}

// Whether a call that moves so many bytes streams them, see kStreamBytes.
inline int32_t streams(int64_t rows, int64_t size, uint64_t bytes_an_element) {
  return (__uint128_t)(uint64_t)rows * (uint64_t)size * bytes_an_element > kStreamBytes ? 1 : 0;
}

inline gclip_status launched(hipError_t e) { return e == hipSuccess ? GCLIP_OK : hip_fail(e); }

}  // namespace gclip
