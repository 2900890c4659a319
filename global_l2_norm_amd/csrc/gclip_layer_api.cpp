// gclip_layer_api.cpp -- the layer calls of the C ABI (include/gclip_layer.h):
// argument checks, then the launch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "gclip_host.hpp"
#include "gclip_layer.hpp"

namespace {

using gclip::DropArgs;
using gclip::Rows;

inline uint64_t address(const void* p) { return reinterpret_cast<uint64_t>(p); }
inline bool dtype_ok(int32_t t) { return t == GCLIP_F32 || t == GCLIP_F16 || t == GCLIP_BF16; }
inline uint64_t elem(int32_t t) { return t == GCLIP_F32 ? 4u : 2u; }

// A matrix or vector operand: bytes [at, at + extent), rows of `row` bytes
// every `ld` bytes.
struct Operand {
  uint64_t at, ld, row, extent;
  bool written, rows;  // rows: a matrix
};

// The operand of a matrix argument; false for one that no call takes.
bool matrix(const void* p, int64_t ld, int64_t rows, int64_t size, uint64_t es, bool written, Operand* o) {
  *o = Operand{address(p), 0, 0, 0, written, true};
  if (rows == 0 || size == 0) return true;
  if (!p || address(p) % es != 0 || ld < 0 || (written && rows > 1 && ld < size)) return false;
  const uint64_t row = (uint64_t)size * es;
  const __uint128_t extent = (__uint128_t)(uint64_t)(rows - 1) * (uint64_t)ld * es + row;
  if (extent > (1ull << 60) || (__uint128_t)address(p) + extent > ~0ull) return false;
  *o = Operand{address(p), rows > 1 ? (uint64_t)ld * es : row, row, (uint64_t)extent, written, true};
  return true;
}

bool vector(const void* p, int64_t n, uint64_t es, bool written, Operand* o) {
  *o = Operand{address(p), 0, 0, 0, written, false};
  if (!p || n == 0) return true;
  if (address(p) % es != 0) return false;
  const uint64_t bytes = (uint64_t)n * es;
  *o = Operand{address(p), bytes, bytes, bytes, written, false};
  return true;
}

// Whether two operands, one of them written, touch a byte in common -- other
// than as the same matrix, read and written in place.
bool clash(const Operand& a, const Operand& b) {
  if (!(a.written || b.written) || a.extent == 0 || b.extent == 0) return false;
  if (a.at + a.extent <= b.at || b.at + b.extent <= a.at) return false;
  if (a.rows && b.rows && a.at == b.at && a.ld == b.ld && a.extent == b.extent) return a.written && b.written;
  // columns of one buffer: rows at the same distance, each clear of the
  // other's both in the same row and in the next
  if (a.ld == b.ld && a.ld > 0 && a.extent > a.row && b.extent > b.row) {
    const uint64_t off = a.at > b.at ? (a.at - b.at) % a.ld : (a.ld - (b.at - a.at) % a.ld) % a.ld;
    return off < b.row || off + a.row > a.ld;
  }
  return true;
}

bool apart(std::initializer_list<Operand> all) {
  for (auto i = all.begin(); i != all.end(); ++i)
    for (auto j = i + 1; j != all.end(); ++j)
      if (clash(*i, *j)) return false;
  return true;
}

bool extents_ok(int64_t rows, int64_t size, int64_t least) {
  return rows >= 0 && rows <= GCLIP_LAYER_MAX_EXTENT && size >= least && size <= GCLIP_LAYER_MAX_EXTENT;
}

// The kernel's form of a dropout; *any is whether it can drop something.
bool dropout_args(const gclip_dropout* d, DropArgs* out, bool* any) {
  *out = DropArgs{};
  *any = false;
  if (!d) return true;
  if (!(d->p >= 0.0 && d->p <= 1.0) || address(d->d_step) % 4 != 0) return false;
  // floor(65536 p + 1/2): the sum itself rounds up to 1 just below 1/2
  const double q = 65536.0 * d->p;
  const uint32_t t = (uint32_t)q + (q - std::floor(q) >= 0.5 ? 1u : 0u);
  *out = DropArgs{(uint32_t)d->seed, (uint32_t)(d->seed >> 32), d->step, d->site, d->d_step, t,
                  t < 65536u ? (float)(65536.0 / (65536.0 - t)) : 0.0f};
  *any = t > 0;
  return true;
}

// Whether a call that reads and writes `matrices` of this shape streams them.
int32_t streamed(int64_t rows, int64_t size, uint64_t es, uint64_t matrices) {
  return (__uint128_t)(uint64_t)rows * (uint64_t)size * es * matrices > gclip::kStreamBytes ? 1 : 0;
}

// A workspace begins with the partial sums; the long rows' means follow.
inline int64_t partial_floats(int64_t rows, int64_t size) { return (int64_t)gclip::layer_parts(rows, size) * 2 * size; }

gclip_status status_of(hipError_t e) { return e == hipSuccess ? GCLIP_OK : gclip::hip_fail(e); }

gclip_status forward(const gclip_layer_forward* a, bool residual, const gclip_dropout* drop, void* stream) {
  if (!a || !extents_ok(a->rows, a->size, 1)) return GCLIP_EINVAL;
  if (!dtype_ok(a->dtype) || !(a->weight_dtype == GCLIP_F32 || a->weight_dtype == a->dtype)) return GCLIP_EDTYPE;
  const uint64_t es = elem(a->dtype), ws = elem(a->weight_dtype);
  if (!std::isfinite(a->eps) || a->eps < 0x1p-126 || !a->mean != !a->rstd) return GCLIP_EINVAL;
  if (a->eps > 0x1.fffffep+127) return GCLIP_EINVAL;  // not finite in binary32
  if (!residual && (a->residual || a->h)) return GCLIP_EINVAL;
  Operand x, r{}, h{}, y, w, b, m, s;
  DropArgs d;
  bool drops;
  if (!matrix(a->x, a->ldx, a->rows, a->size, es, false, &x) ||
      !matrix(a->y, a->ldy, a->rows, a->size, es, true, &y) || !vector(a->weight, a->size, ws, false, &w) ||
      !vector(a->bias, a->size, ws, false, &b) || !vector(a->mean, a->rows, 4, true, &m) ||
      !vector(a->rstd, a->rows, 4, true, &s) || !dropout_args(drop, &d, &drops))
    return GCLIP_EINVAL;
  if (residual && (!matrix(a->residual, a->ldresidual, a->rows, a->size, es, false, &r) ||
                   !matrix(a->h, a->ldh, a->rows, a->size, es, true, &h)))
    return GCLIP_EINVAL;
  if (!apart({x, r, h, y, w, b, m, s})) return GCLIP_EINVAL;
  if (a->rows == 0) return GCLIP_OK;
  const gclip::FwdArgs k{{x.at, x.ld}, {r.at, r.ld}, {h.at, h.ld}, {y.at, y.ld}, address(a->weight), address(a->bias),
                         a->mean, a->rstd, (uint32_t)a->rows, (uint32_t)a->size, a->weight_dtype, (float)a->eps,
                         (float)(1.0 / std::sqrt((double)(float)a->eps)),
                         streamed(a->rows, a->size, es, residual ? 4 : 2)};
  return status_of(gclip::launch_layer_forward(k, a->dtype, residual, drops ? &d : nullptr,
                                               static_cast<hipStream_t>(stream)));
}

gclip_status backward(const gclip_layer_backward* a, bool residual, const gclip_dropout* drop, void* stream) {
  if (!a || !extents_ok(a->rows, a->size, 1)) return GCLIP_EINVAL;
  if (!dtype_ok(a->dtype) || !(a->weight_dtype == GCLIP_F32 || a->weight_dtype == a->dtype) ||
      !(a->grad_dtype == GCLIP_F32 || a->grad_dtype == a->dtype))
    return GCLIP_EDTYPE;
  const uint64_t es = elem(a->dtype), ws = elem(a->weight_dtype), gs = elem(a->grad_dtype);
  Operand dy, dh{}, x, dr{}, dx{}, w, dw, db, m, s, wk{};
  DropArgs d;
  bool drops;
  if (!dropout_args(drop, &d, &drops)) return GCLIP_EINVAL;
  // without dropout the residual step has one result for both of its inputs
  if (!residual ? (a->dh || a->dresidual) : (!drop && a->dx)) return GCLIP_EINVAL;
  const bool two = residual && drop;
  if (!matrix(a->dy, a->lddy, a->rows, a->size, es, false, &dy) ||
      !matrix(a->x, a->ldx, a->rows, a->size, es, false, &x) ||
      !vector(a->mean, a->rows, 4, false, &m) || !vector(a->rstd, a->rows, 4, false, &s) ||
      !vector(a->weight, a->size, ws, false, &w) || !vector(a->dweight, a->size, gs, true, &dw) ||
      !vector(a->dbias, a->size, gs, true, &db))
    return GCLIP_EINVAL;
  if (a->rows > 0 && (!a->mean || !a->rstd)) return GCLIP_EINVAL;
  if (a->dh && !matrix(a->dh, a->lddh, a->rows, a->size, es, false, &dh)) return GCLIP_EINVAL;
  if (residual && !matrix(a->dresidual, a->lddresidual, a->rows, a->size, es, true, &dr)) return GCLIP_EINVAL;
  if ((!residual || two) && !matrix(a->dx, a->lddx, a->rows, a->size, es, true, &dx)) return GCLIP_EINVAL;
  const int64_t need = gclip_layer_workspace(a->rows, a->size);
  if ((need > 0 && !a->workspace) || a->workspace_bytes < need || address(a->workspace) % 16 != 0) return GCLIP_EINVAL;
  if (!vector(a->workspace, need, 1, true, &wk)) return GCLIP_EINVAL;
  if (!apart({dy, dh, x, dr, dx, w, dw, db, m, s, wk})) return GCLIP_EINVAL;
  if (a->rows == 0 && ((!a->dweight && !a->dbias) || a->accumulate)) return GCLIP_OK;
  const Operand& out = residual ? dr : dx;
  const gclip::BwdArgs k{{dy.at, dy.ld}, {dh.at, dh.ld}, {x.at, x.ld}, {out.at, out.ld}, {dx.at, dx.ld},
                         a->mean, a->rstd,
                         address(a->weight), address(a->dweight), address(a->dbias), static_cast<float*>(a->workspace),
                         static_cast<float*>(a->workspace) + partial_floats(a->rows, a->size),
                         (uint32_t)a->rows, (uint32_t)a->size, a->weight_dtype, a->grad_dtype, a->accumulate ? 1 : 0,
                         gclip::layer_parts(a->rows, a->size),
                         streamed(a->rows, a->size, es, 3 + (a->dh ? 1 : 0) + (two ? 1 : 0))};
  return status_of(gclip::launch_layer_backward(k, a->dtype, residual, two ? &d : nullptr,
                                                static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

gclip_status gclip_layernorm_forward(const gclip_layer_forward* a, void* stream) {
  return forward(a, false, nullptr, stream);
}

gclip_status gclip_residual_forward(const gclip_layer_forward* a, const gclip_dropout* drop, void* stream) {
  return forward(a, true, drop, stream);
}

gclip_status gclip_layernorm_backward(const gclip_layer_backward* a, void* stream) {
  return backward(a, false, nullptr, stream);
}

gclip_status gclip_residual_backward(const gclip_layer_backward* a, const gclip_dropout* drop, void* stream) {
  return backward(a, true, drop, stream);
}

gclip_status gclip_dropout_apply(const void* x, int64_t ldx, void* y, int64_t ldy, int64_t rows, int64_t size,
                                 int32_t dtype, const gclip_dropout* drop, void* stream) {
  if (!drop || !extents_ok(rows, size, 0)) return GCLIP_EINVAL;
  if (!dtype_ok(dtype)) return GCLIP_EDTYPE;
  Operand i, o;
  DropArgs d;
  bool drops;
  if (!matrix(x, ldx, rows, size, elem(dtype), false, &i) || !matrix(y, ldy, rows, size, elem(dtype), true, &o) ||
      !dropout_args(drop, &d, &drops) || !apart({i, o}))
    return GCLIP_EINVAL;
  if (rows == 0 || size == 0) return GCLIP_OK;
  return status_of(gclip::launch_dropout({i.at, i.ld}, {o.at, o.ld}, (uint32_t)rows, (uint32_t)size, dtype, d,
                                         static_cast<hipStream_t>(stream)));
}

int64_t gclip_layer_workspace(int64_t rows, int64_t size) {
  if (!extents_ok(rows, size, 1)) return 0;
  return 4 * (partial_floats(rows, size) + (size > gclip::kBwdMax ? 2 * rows : 0));
}

}  // extern "C"
