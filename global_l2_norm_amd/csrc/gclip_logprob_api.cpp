// gclip_logprob_api.cpp -- the log probability calls of the C ABI
// (include/gclip_logprob.h): argument checks, then the launch.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "gclip_logprob.hpp"
#include "gclip_operand.hpp"

namespace {

using namespace gclip;

bool top_ok(int64_t size, int32_t top) { return top >= 0 && top <= GCLIP_LOGPROB_MAX_TOP && top <= size; }

// Of any format: the keys of the segments come first, then their sums.
int64_t segments_most(int64_t rows, int64_t size) {
  const uint32_t a = logp_cut((uint32_t)rows, (uint32_t)size, GCLIP_F32).segments;
  const uint32_t b = logp_cut((uint32_t)rows, (uint32_t)size, GCLIP_BF16).segments;
  const uint32_t n = a > b ? a : b;
  return n > 1 ? n : 0;
}
int64_t workspace_bytes(int64_t rows, int64_t size, int32_t top) {
  return rows == 0 ? 0 : rows * segments_most(rows, size) * (8ll * top + 16);
}

}  // namespace

extern "C" {

gclip_status gclip_logprob_forward(const gclip_logprobs* a, void* stream) {
  if (!a || !extents_fit(a->rows, a->size)) return GCLIP_EINVAL;
  if (!format_ok(a->dtype)) return GCLIP_EDTYPE;
  if (!top_ok(a->size, a->top) || a->dlogp || a->dentropy || a->dlogits) return GCLIP_EINVAL;
  Span x, t, l, p, e, tl, ti, wk;
  if (!matrix_of(a->logits, a->ld, a->rows, a->size, format_bytes(a->dtype), false, &x) ||
      !vector_of(a->targets, a->rows, 8, false, &t) || !vector_of(a->stats, 2 * a->rows, 4, true, &l) ||
      !vector_of(a->logp, a->rows, 4, true, &p) || !vector_of(a->entropy, a->rows, 4, true, &e) ||
      !vector_of(a->top_logp, a->rows * a->top, 4, true, &tl) || !vector_of(a->top_ids, a->rows * a->top, 8, true, &ti))
    return GCLIP_EINVAL;
  if (a->rows > 0 && (!a->targets != !a->logp || (a->top > 0) != (a->top_logp != nullptr) ||
                      (a->top > 0) != (a->top_ids != nullptr)))
    return GCLIP_EINVAL;
  const int64_t need = workspace_bytes(a->rows, a->size, a->top);
  if ((need > 0 && !a->workspace) || a->workspace_bytes < need || address_of(a->workspace) % 16 != 0 ||
      !vector_of(a->workspace, need, 1, true, &wk))
    return GCLIP_EINVAL;
  if (!none_touch({x, t, l, p, e, tl, ti, wk})) return GCLIP_EINVAL;
  if (a->rows == 0) return GCLIP_OK;
  const LogpCut cut = logp_cut((uint32_t)a->rows, (uint32_t)a->size, a->dtype);
  LogpArgs k{};
  k.x = x.device();
  k.targets = a->targets;
  k.ignore = a->ignore;
  k.stats = a->stats;
  k.logp = a->logp;
  k.entropy = a->entropy;
  k.top_logp = a->top_logp;
  k.top_ids = a->top_ids;
  k.keys = static_cast<uint64_t*>(a->workspace);
  k.parts = reinterpret_cast<float*>(address_of(a->workspace) + (uint64_t)a->rows * cut.segments * 8u * (uint64_t)a->top);
  k.rows = (uint32_t)a->rows;
  k.size = (uint32_t)a->size;
  k.top = (uint32_t)a->top;
  k.segments = cut.segments;
  k.turns = cut.turns;
  k.threads = cut.threads;
  k.streamed = streams(a->rows, a->size, format_bytes(a->dtype));
  return launched(launch_logprob_forward(k, a->dtype, static_cast<hipStream_t>(stream)));
}

gclip_status gclip_logprob_backward(const gclip_logprobs* a, void* stream) {
  if (!a || !extents_fit(a->rows, a->size)) return GCLIP_EINVAL;
  if (!format_ok(a->dtype)) return GCLIP_EDTYPE;
  if (a->top != 0 || a->logp || a->top_logp || a->top_ids) return GCLIP_EINVAL;
  Span x, t, l, p, e, d, o;
  const uint64_t es = format_bytes(a->dtype);
  if (!matrix_of(a->logits, a->ld, a->rows, a->size, es, false, &x) ||
      !matrix_of(a->dlogits, a->lddlogits, a->rows, a->size, es, true, &o) ||
      !vector_of(a->targets, a->rows, 8, false, &t) || !vector_of(a->stats, 2 * a->rows, 4, false, &l) ||
      !vector_of(a->entropy, a->rows, 4, false, &e) || !vector_of(a->dlogp, a->rows, 4, false, &p) ||
      !vector_of(a->dentropy, a->rows, 4, false, &d))
    return GCLIP_EINVAL;
  if (a->rows > 0 && (!a->targets || !a->stats || !a->dlogp || (a->dentropy && !a->entropy))) return GCLIP_EINVAL;
  if (!none_touch({x, t, l, p, e, d, o})) return GCLIP_EINVAL;
  if (a->rows == 0) return GCLIP_OK;
  LogpArgs k{};
  k.x = x.device();
  k.dx = o.device();
  k.targets = a->targets;
  k.ignore = a->ignore;
  k.stats = a->stats;
  k.entropy = a->entropy;
  k.dlogp = a->dlogp;
  k.dentropy = a->dentropy;
  k.rows = (uint32_t)a->rows;
  k.size = (uint32_t)a->size;
  k.streamed = streams(a->rows, a->size, 2 * es);
  return launched(launch_logprob_backward(k, a->dtype, static_cast<hipStream_t>(stream)));
}

int64_t gclip_logprob_workspace(int64_t rows, int64_t size, int32_t top) {
  return extents_fit(rows, size) && top_ok(size, top) ? workspace_bytes(rows, size, top) : 0;
}

}  // extern "C"
