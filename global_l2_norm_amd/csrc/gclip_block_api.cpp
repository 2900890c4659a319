// gclip_block_api.cpp -- the block calls of the C ABI (include/gclip_block.h):
// argument checks, then the launch.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "gclip_operand.hpp"

namespace {

using namespace gclip;

// The kernel's form of a dropout; *any is whether it can drop something.
bool dropout_of(const gclip_dropout* d, DropArgs* out, bool* any) {
  *out = DropArgs{};
  *any = false;
  if (!d) return true;
  if (!(d->p >= 0.0 && d->p <= 1.0) || address_of(d->d_step) % 4 != 0) return false;
  // floor(65536 p + 1/2): the sum itself rounds up to 1 just below 1/2
  const double q = 65536.0 * d->p;
  const uint32_t t = (uint32_t)q + (q - std::floor(q) >= 0.5 ? 1u : 0u);
  *out = DropArgs{(uint32_t)d->seed, (uint32_t)(d->seed >> 32), d->step, d->site, d->d_step, t,
                  t < 65536u ? (float)(65536.0 / (65536.0 - t)) : 0.0f};
  *any = t > 0;
  return true;
}

int64_t part_floats(int64_t rows, int64_t size) { return (int64_t)rms_parts(rows, size) * (int64_t)part_columns((uint32_t)size); }
// The long rows' means follow the partial sums.  Few rows in registers leave
// none.
int64_t workspace_bytes(int64_t rows, int64_t size) {
  if (in_registers((uint32_t)size, kRmsBwdMax) && weight_by_strips((uint32_t)rows, (uint32_t)size)) return 0;
  return 4 * (part_floats(rows, size) + (size > kRmsBwdMax ? rows : 0));
}

gclip_status forward(const gclip_rms_forward* a, bool residual, const gclip_dropout* drop, void* stream) {
  if (!a || !extents_fit(a->rows, a->size)) return GCLIP_EINVAL;
  if (!format_ok(a->dtype) || !weight_format_ok(a->weight_dtype, a->dtype)) return GCLIP_EDTYPE;
  const uint64_t es = format_bytes(a->dtype), ws = format_bytes(a->weight_dtype);
  if (!std::isfinite(a->eps) || a->eps < 0x1p-126 || a->eps > 0x1.fffffep+127) return GCLIP_EINVAL;
  if (!residual && (a->residual || a->h)) return GCLIP_EINVAL;
  Span x, r, h, y, y8, ys, k8, ks, w, s;
  Eight ey, ek;
  DropArgs d;
  bool drops;
  if (!matrix_of(a->x, a->ldx, a->rows, a->size, es, false, &x) ||
      !packed_of(a->y8, a->rows, a->size, true, true, &ey, &y8, &ys) ||
      !packed_of(a->kept, a->rows, a->size, true, false, &ek, &k8, &ks) ||
      !vector_of(a->weight, a->size, ws, false, &w) || !vector_of(a->rstd, a->rows, 4, true, &s) ||
      !dropout_of(drop, &d, &drops))
    return GCLIP_EINVAL;
  if (a->y8.values ? a->y != nullptr : !matrix_of(a->y, a->ldy, a->rows, a->size, es, true, &y)) return GCLIP_EINVAL;
  if (residual && (!matrix_of(a->residual, a->ldresidual, a->rows, a->size, es, false, &r) ||
                   !matrix_of(a->h, a->ldh, a->rows, a->size, es, true, &h)))
    return GCLIP_EINVAL;
  if (!none_touch({x, r, h, y, y8, ys, k8, ks, w, s})) return GCLIP_EINVAL;
  if (a->rows == 0) return GCLIP_OK;
  const uint64_t moved = (residual ? 3 : 1) * es + (a->y8.values ? 1 : es) + (a->kept.values ? 1 : 0);
  const RmsFwdArgs k{x.device(), r.device(), h.device(), y.device(), ey, ek, address_of(a->weight), a->rstd,
                     (uint32_t)a->rows, (uint32_t)a->size, a->weight_dtype, (float)a->eps,
                     streams(a->rows, a->size, moved)};
  return launched(launch_rms_forward(k, a->dtype, residual, drops ? &d : nullptr, static_cast<hipStream_t>(stream)));
}

gclip_status backward(const gclip_rms_backward* a, bool residual, const gclip_dropout* drop, void* stream) {
  if (!a || !extents_fit(a->rows, a->size)) return GCLIP_EINVAL;
  if (!format_ok(a->dtype) || !weight_format_ok(a->weight_dtype, a->dtype) ||
      !weight_format_ok(a->grad_dtype, a->dtype))
    return GCLIP_EDTYPE;
  const uint64_t es = format_bytes(a->dtype), ws = format_bytes(a->weight_dtype), gs = format_bytes(a->grad_dtype);
  Span dy, dh, x, x8, xs, dr, dx, w, dw, s, wk;
  Eight ex;
  DropArgs d;
  bool drops;
  if (!dropout_of(drop, &d, &drops)) return GCLIP_EINVAL;
  // without dropout the residual step has one result for both of its inputs
  if (!residual ? (a->dh || a->dresidual) : (!drop && a->dx)) return GCLIP_EINVAL;
  const bool two = residual && drop;
  if (!matrix_of(a->dy, a->lddy, a->rows, a->size, es, false, &dy) ||
      !packed_of(a->x8, a->rows, a->size, false, true, &ex, &x8, &xs) ||
      !vector_of(a->rstd, a->rows, 4, false, &s) || !vector_of(a->weight, a->size, ws, false, &w) ||
      !vector_of(a->dweight, a->size, gs, true, &dw))
    return GCLIP_EINVAL;
  if (a->x8.values ? a->x != nullptr : !matrix_of(a->x, a->ldx, a->rows, a->size, es, false, &x)) return GCLIP_EINVAL;
  if (a->rows > 0 && !a->rstd) return GCLIP_EINVAL;
  if (a->dh && !matrix_of(a->dh, a->lddh, a->rows, a->size, es, false, &dh)) return GCLIP_EINVAL;
  if (residual && !matrix_of(a->dresidual, a->lddresidual, a->rows, a->size, es, true, &dr)) return GCLIP_EINVAL;
  if ((!residual || two) && !matrix_of(a->dx, a->lddx, a->rows, a->size, es, true, &dx)) return GCLIP_EINVAL;
  const int64_t need = workspace_bytes(a->rows, a->size);
  if ((need > 0 && !a->workspace) || a->workspace_bytes < need || address_of(a->workspace) % 16 != 0 ||
      !vector_of(a->workspace, need, 1, true, &wk))
    return GCLIP_EINVAL;
  if (!none_touch({dy, dh, x, x8, xs, dr, dx, w, dw, s, wk})) return GCLIP_EINVAL;
  if (a->rows == 0 && (!a->dweight || a->accumulate)) return GCLIP_OK;
  const uint64_t moved = es * (2 + (a->dh ? 1 : 0) + (two ? 1 : 0)) + (a->x8.values ? 1 : es);
  const RmsBwdArgs k{dy.device(), dh.device(), x.device(), (residual ? dr : dx).device(), dx.device(), ex, a->rstd,
                     address_of(a->weight), address_of(a->dweight), static_cast<float*>(a->workspace),
                     static_cast<float*>(a->workspace) + part_floats(a->rows, a->size), (uint32_t)a->rows,
                     (uint32_t)a->size, a->weight_dtype, a->grad_dtype, a->accumulate ? 1 : 0,
                     rms_parts(a->rows, a->size), 0, 0, streams(a->rows, a->size, moved)};
  return launched(launch_rms_backward(k, a->dtype, residual, two ? &d : nullptr, static_cast<hipStream_t>(stream)));
}

gclip_status activate(const gclip_activate* a, bool backward, void* stream) {
  if (!a || !extents_fit(a->rows, a->size)) return GCLIP_EINVAL;
  if (!format_ok(a->dtype)) return GCLIP_EDTYPE;
  if (a->kind < GCLIP_ACT_SILU || a->kind > GCLIP_ACT_RELU) return GCLIP_EINVAL;
  const uint64_t es = format_bytes(a->dtype);
  const bool eight = a->gate8.values != nullptr;
  const bool gated = backward && eight ? a->up8.values != nullptr : a->up != nullptr;
  Span g, u, y, dy, dg, du, g8, gs, u8, us;
  Eight eg, eu;
  if (!packed_of(a->gate8, a->rows, a->size, !backward, false, &eg, &g8, &gs) ||
      !packed_of(a->up8, a->rows, a->size, !backward, false, &eu, &u8, &us))
    return GCLIP_EINVAL;
  if ((a->up8.values != nullptr) != (eight && gated)) return GCLIP_EINVAL;
  if (backward && eight) {
    if (a->gate || a->up) return GCLIP_EINVAL;
  } else if (!matrix_of(a->gate, a->ldgate, a->rows, a->size, es, false, &g) ||
             (gated && !matrix_of(a->up, a->ldup, a->rows, a->size, es, false, &u))) {
    return GCLIP_EINVAL;
  }
  if ((!backward || a->y) && !matrix_of(a->y, a->ldy, a->rows, a->size, es, true, &y)) return GCLIP_EINVAL;
  if (!backward) {
    if (a->dy || a->dgate || a->dup) return GCLIP_EINVAL;
  } else {
    if (!matrix_of(a->dy, a->lddy, a->rows, a->size, es, false, &dy) ||
        !matrix_of(a->dgate, a->lddgate, a->rows, a->size, es, true, &dg) ||
        (gated ? !matrix_of(a->dup, a->lddup, a->rows, a->size, es, true, &du) : a->dup != nullptr))
      return GCLIP_EINVAL;
  }
  if (!none_touch({g, u, y, dy, dg, du, g8, gs, u8, us})) return GCLIP_EINVAL;
  if (a->rows == 0) return GCLIP_OK;
  const uint64_t inputs = (gated ? 2 : 1) * (backward && eight ? 1 : es);
  const uint64_t moved = backward ? inputs + es * ((gated ? 3 : 2) + (a->y ? 1 : 0))
                                  : inputs + es + (eight ? gated ? 2 : 1 : 0);
  const ActArgs k{g.device(), u.device(), y.device(), dy.device(), dg.device(), du.device(), eg, eu,
                  (uint32_t)a->rows, (uint32_t)a->size};
  return launched(launch_activation(k, a->dtype, a->kind, backward, streams(a->rows, a->size, moved) != 0,
                                    static_cast<hipStream_t>(stream)));
}

}  // namespace

extern "C" {

gclip_status gclip_rmsnorm_forward(const gclip_rms_forward* a, void* stream) {
  return forward(a, false, nullptr, stream);
}

gclip_status gclip_residual_rms_forward(const gclip_rms_forward* a, const gclip_dropout* drop, void* stream) {
  return forward(a, true, drop, stream);
}

gclip_status gclip_rmsnorm_backward(const gclip_rms_backward* a, void* stream) {
  return backward(a, false, nullptr, stream);
}

gclip_status gclip_residual_rms_backward(const gclip_rms_backward* a, const gclip_dropout* drop, void* stream) {
  return backward(a, true, drop, stream);
}

int64_t gclip_rms_workspace(int64_t rows, int64_t size) {
  return extents_fit(rows, size) ? workspace_bytes(rows, size) : 0;
}

gclip_status gclip_activation_forward(const gclip_activate* a, void* stream) { return activate(a, false, stream); }

gclip_status gclip_activation_backward(const gclip_activate* a, void* stream) { return activate(a, true, stream); }

gclip_status gclip_pack(const void* x, int64_t ldx, const gclip_packed8* out, int64_t rows, int64_t size,
                         int32_t dtype, void* stream) {
  if (!out || !extents_fit(rows, size)) return GCLIP_EINVAL;
  if (!format_ok(dtype)) return GCLIP_EDTYPE;
  Span i, o, s;
  Eight e;
  if (!matrix_of(x, ldx, rows, size, format_bytes(dtype), false, &i) ||
      !packed_of(*out, rows, size, true, true, &e, &o, &s) || !none_touch({i, o, s}))
    return GCLIP_EINVAL;
  if (rows == 0) return GCLIP_OK;
  if (!out->values) return GCLIP_EINVAL;
  return launched(launch_pack8(i.device(), e, (uint32_t)rows, (uint32_t)size, dtype, static_cast<hipStream_t>(stream)));
}

gclip_status gclip_unpack(const gclip_packed8* x, void* out, int64_t ldout, int64_t rows, int64_t size,
                           int32_t dtype, void* stream) {
  if (!x || !extents_fit(rows, size)) return GCLIP_EINVAL;
  if (!format_ok(dtype)) return GCLIP_EDTYPE;
  Span i, o, s;
  Eight e;
  if (!matrix_of(out, ldout, rows, size, format_bytes(dtype), true, &o) ||
      !packed_of(*x, rows, size, false, true, &e, &i, &s) || !none_touch({i, o, s}))
    return GCLIP_EINVAL;
  if (rows == 0) return GCLIP_OK;
  if (!x->values) return GCLIP_EINVAL;
  return launched(launch_unpack8(e, o.device(), (uint32_t)rows, (uint32_t)size, dtype, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
