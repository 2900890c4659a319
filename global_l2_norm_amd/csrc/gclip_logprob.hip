// gclip_logprob.hip -- log probabilities of given tokens, with the entropy
// and the likeliest alternatives, and their gradient.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cstdint>

#include "gclip_block_device.hpp"
#include "gclip_logprob.hpp"

namespace gclip {
namespace {

constexpr int kChunk = 4;  // units of a lane at a time
constexpr uint32_t kCandidates = 1024;
static_assert(GCLIP_LOGPROB_MAX_TOP * GCLIP_LOGPROB_MAX_TOP <= kCandidates, "the join's candidates");
constexpr float kLog2e = 1.44269504088896f;
constexpr float kLowest = -0x1.fffffep+127f;
constexpr float kNone = -__builtin_huge_valf();

// ---------------------------------------------------------------- a softmax on the way
// Of the logits so far: the largest, m (-infinity: none that can come), and
// relative to r = max(m, the lowest finite number) the sums of e^(x - r) and
// of (x - r) e^(x - r).  Differences are taken before anything is multiplied,
// so logits of any size, the lowest finite ones too, keep theirs.  A NaN or
// an infinity in a row makes s a NaN, which stays.
struct Softmax {
  float m, s, t;
};
__device__ __forceinline__ float reference(float m) { return fmaxf(m, kLowest); }
// The difference of two references; finite, and so times any sum of 2^31
// exponentials, so that nothing times either is nothing.
constexpr float kFar = -1e28f;
__device__ __forceinline__ float drop_to(float from, float to) { return fmaxf(reference(from) - reference(to), kFar); }

template <bool ENTROPY>
__device__ __forceinline__ void rebase(Softmax& z, float m) {
  const float delta = drop_to(z.m, m), f = __builtin_amdgcn_exp2f(delta * kLog2e);
  if (ENTROPY) z.t = f * __builtin_fmaf(delta, z.s, z.t);
  z.s *= f;
  z.m = m;
}

template <bool ENTROPY, int N>
__device__ __forceinline__ void take(Softmax& z, const float (&v)[N]) {
  float m = z.m;
#pragma unroll
  for (int j = 0; j < N; ++j) m = fmaxf(m, v[j]);
  rebase<ENTROPY>(z, m);
  const float r = reference(m);
  float s = 0.0f, t = 0.0f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float d = v[j] - r, e = __builtin_amdgcn_exp2f(d * kLog2e);
    s += e;
    if (ENTROPY) t = __builtin_fmaf(e, fmaxf(d, kFar), t);
  }
  z.s += s;
  if (ENTROPY) z.t += t;
}

template <int N>
__device__ __forceinline__ float lanes_largest(float v) {
  if constexpr (N >= 2) v = fmaxf(v, permuted<0xB1>(v));
  if constexpr (N >= 4) v = fmaxf(v, permuted<0x4E>(v));
  if constexpr (N >= 8) v = fmaxf(v, permuted<0x141>(v));
  if constexpr (N >= 16) v = fmaxf(v, permuted<0x140>(v));
  if constexpr (N >= 32) {
    const auto s = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
  }
  if constexpr (N >= 64) {
    const auto s = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    v = fmaxf(__uint_as_float(s[0]), __uint_as_float(s[1]));
  }
  return v;
}

// The softmax of the workgroup's WAVES waves from its threads', in all of
// them, in a fixed order.
template <int WAVES, bool ENTROPY>
__device__ __forceinline__ Softmax joined(Softmax z, float (*red)[4]) {
#pragma unroll
  for (int pass = 0; pass < 2; ++pass) {
    rebase<ENTROPY>(z, lanes_largest<64>(z.m));
    z.s = lanes_sum<64>(z.s);
    if (ENTROPY) z.t = lanes_sum<64>(z.t);
    if (pass == 1) break;
    const uint32_t lane = threadIdx.x & 63;
    if (lane == 0) {
      red[threadIdx.x >> 6][0] = z.m;
      red[threadIdx.x >> 6][1] = z.s;
      red[threadIdx.x >> 6][2] = z.t;
    }
    __syncthreads();
    z = lane < WAVES ? Softmax{red[lane][0], red[lane][1], red[lane][2]} : Softmax{kNone, 0.0f, 0.0f};
  }
  return z;
}

// What a row's numbers come to: its softmax, its target's logit (column:
// there is one) and s = log(sum).
template <bool ENTROPY>
__device__ __forceinline__ void store_row(const LogpArgs& a, uint32_t r, const Softmax& all, double s, bool column,
                                          float given) {
  const bool none = all.s == 0.0f;  // nothing that can come
  if (a.stats) {
    a.stats[2ull * r] = none ? kNone : all.m;
    a.stats[2ull * r + 1] = (float)s;
  }
  if (a.logp) a.logp[r] = !column ? __uint_as_float(0x7fc00000u) : none ? kNone : (float)((double)given - (double)all.m - s);
  if (ENTROPY) a.entropy[r] = none ? 0.0f : (float)(s - (double)all.t / (double)all.s);
}

// A row that counts for nothing.
template <bool ENTROPY>
__device__ __forceinline__ void store_nothing(const LogpArgs& a, uint32_t r) {
  if (a.stats) a.stats[2ull * r] = a.stats[2ull * r + 1] = 0.0f;
  if (a.logp) a.logp[r] = 0.0f;
  if (ENTROPY) a.entropy[r] = 0.0f;
}
template <bool ENTROPY, bool TOP>
__device__ __forceinline__ void store_no_row(const LogpArgs& a, uint32_t r) {
  if (threadIdx.x == 0) store_nothing<ENTROPY>(a, r);
  if (TOP && threadIdx.x < a.top) {
    a.top_logp[(uint64_t)r * a.top + threadIdx.x] = kNone;
    a.top_ids[(uint64_t)r * a.top + threadIdx.x] = -1;
  }
}

// ---------------------------------------------------------------- the likeliest
// A key orders logits, and columns of equal logits from the last to the
// first; every column has another.  0 is none, and none is all ones.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.0f);  // both zeros are one
  return v != v ? 0xffffffffu : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return k == 0xffffffffu ? __uint_as_float(0x7fc00000u) : __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t key_of(float v, uint32_t column) {
  return ((uint64_t)ordered(v) << 32) | (0x7fffffffu - column);
}

// The largest of a wave's words, in all lanes.
__device__ __forceinline__ uint32_t lanes_most(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xf, 0xf, true));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xf, 0xf, true));
  const auto a = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  v = max(a[0], a[1]);
  const auto b = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return max(b[0], b[1]);
}

// The k-th largest of a wave's words but for their lowest bits, the same in
// all lanes: no more than the k-th largest.
template <int IDLE = 0>
__device__ __forceinline__ uint32_t kth_largest(uint32_t v, uint32_t k) {
  uint32_t t = 0;
#pragma unroll 4
  for (int bit = 31; bit >= IDLE; --bit) {
    const uint32_t c = t | (1u << bit);
    if ((uint32_t)__popcll(__ballot(v >= c)) >= k) t = c;
  }
  return t;
}
// Lowest bits of a converted element that say nothing.
template <int DT>
constexpr int kIdleBits = DT == GCLIP_F32 ? 0 : DT == GCLIP_F16 ? 13 : 16;

template <int THREADS>
struct Top {
  uint64_t candidate[kCandidates];
  uint64_t best[GCLIP_LOGPROB_MAX_TOP];
  uint64_t largest[THREADS / 64];
  union {
    uint32_t chosen[THREADS];
    uint64_t first[64];
  };
  uint32_t threshold[2][THREADS / 64];
  uint32_t n, chosen_n;
};

// One more candidate, if there is room for it; n counts it either way.  The
// only store to candidate[]: others of the workgroup may have filled it.
template <int THREADS>
__device__ __forceinline__ bool offer(Top<THREADS>& w, uint64_t key) {
  const uint32_t at = atomicAdd(&w.n, 1u);
  if (at >= kCandidates) return false;
  w.candidate[at] = key;
  return true;
}

// best[] from the candidates, n of them at most kCandidates: a candidate's
// place is the number of larger ones.
template <int THREADS>
__device__ __forceinline__ void rank_candidates(Top<THREADS>& w, uint32_t n, uint32_t k) {
  for (uint32_t i = threadIdx.x; i < n; i += THREADS) {
    const uint64_t own = w.candidate[i];
    uint32_t place = 0;
#pragma unroll 8
    for (uint32_t j = 0; j < n; ++j) place += w.candidate[j] > own ? 1u : 0u;
    if (place < k) w.best[place] = own;
  }
}

// ---------------------------------------------------------------- reading a segment
// Unit u of a row: where it passes the row's end its columns there are
// -infinity.  Loads of units past the end stay inside the row.
template <int DT, bool NT>
__device__ __forceinline__ u32x4 logits_raw(uint64_t row, uint32_t u, uint32_t size) {
  constexpr uint32_t kU = kUnit<DT>;
  if (size < kU) return load_unit<DT, false>(row, 0, size);
  const uint64_t c = (uint64_t)u * kU;
  return load16<DT, NT>(row + (c + kU <= size ? c : size - kU) * kElem<DT>);
}
template <int DT>
__device__ __forceinline__ void logits_settled(u32x4 q, uint32_t u, uint32_t size, float* v) {
  constexpr uint32_t kU = kUnit<DT>;
  const uint64_t c = (uint64_t)u * kU;
  if (size >= kU && c < size && c + kU > size) q = moved_down<DT>(q, kU - size % kU);
  float t[kU];
  unpack_unit<DT>(q, t);
#pragma unroll
  for (uint32_t j = 0; j < kU; ++j) v[j] = c + j < size ? t[j] : kNone;
}

// One pass over a segment of a row (all of it, with many rows), a unit of 16
// bytes a lane, kChunk of them at a time with the next ones under way.  What a
// lane has seen as its largest logit then chooses the few lanes that can hold
// one of the likeliest, and those read theirs again, from the caches: the k-th
// largest logit is at least the k-th largest of any wave's lanes' largest, and
// at least what, in every wave, k / waves of those reach.  Rows of so many equal
// logits that the candidates do not fit, and those with NaNs or infinities, are
// searched k times instead.
//
// Long rows of 16-bit logits are bound by the exponentials: 4096 x 50304 with
// entropies 69.6 us, 412 MB at 5.9 TB/s with the vector units full; 8192 x 8449
// in binary32 by memory, 49.4 us, 277 MB at 5.6 TB/s.  Few rows by latency: 8 x
// 131072 in segments 8.0 us with 20 alternatives and 5.8 for the join; their
// lanes have one unit each and read kChunk, 7 MB of the 2 that it takes.
template <int DT, int THREADS, bool ENTROPY, bool TOP, bool STREAMED>
__global__ __launch_bounds__(THREADS) void k_logp(LogpArgs a) {
  constexpr uint32_t kU = kUnit<DT>;
  constexpr int kWaves = THREADS / 64;
  __shared__ float red[kWaves][4];
  [[maybe_unused]] __shared__ Top<THREADS> top;
  const uint64_t wg = workgroup_of_grid();
  const uint32_t r = (uint32_t)(wg / a.segments), seg = (uint32_t)(wg % a.segments);
  if (r >= a.rows) return;
  const uint32_t tid = threadIdx.x;
  const int64_t target = a.targets ? a.targets[r] : 0;
  if (a.targets && target == a.ignore) {
    if (a.segments == 1) store_no_row<ENTROPY, TOP>(a, r);  // else the join does
    return;
  }
  const uint64_t row = a.x.at + r * a.x.ld;
  const uint32_t first = seg * (a.turns * (uint32_t)THREADS) + tid;  // unit
  const bool column = a.logp && target >= 0 && target < (int64_t)a.size;
  float given = 0.0f;
  if (a.segments == 1 && column) given = elem_float<DT>(load_elem<DT>(row + (uint64_t)target * kElem<DT>));

  Softmax z{kNone, 0.0f, 0.0f};
  u32x4 next[kChunk];
  const auto fetch = [&](uint32_t turn) {
#pragma unroll
    for (int k = 0; k < kChunk; ++k) next[k] = logits_raw<DT, STREAMED>(row, first + (turn + k) * (uint32_t)THREADS, a.size);
  };
  fetch(0);
  for (uint32_t turn = 0; turn < a.turns; turn += kChunk) {
    u32x4 q[kChunk];
#pragma unroll
    for (int k = 0; k < kChunk; ++k) q[k] = next[k];
    if (turn + kChunk < a.turns) fetch(turn + kChunk);
    // all of the workgroup's units of these turns lie in the row, and in the segment
    const uint64_t end = ((uint64_t)seg * a.turns * (uint32_t)THREADS + (uint64_t)(turn + kChunk) * (uint32_t)THREADS) * kU;
    if (end <= a.size && turn + kChunk <= a.turns) {
      float v[kChunk * kU];
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        float t[kU];
        unpack_unit<DT>(q[k], t);
#pragma unroll
        for (uint32_t j = 0; j < kU; ++j) v[k * kU + j] = t[j];
      }
      take<ENTROPY>(z, v);
    } else {
#pragma unroll
      for (int k = 0; k < kChunk; ++k) {
        if (turn + k < a.turns) {
          float t[kU];
          logits_settled<DT>(q[k], first + (turn + k) * (uint32_t)THREADS, a.size, t);
          take<ENTROPY>(z, t);
        }
      }
    }
  }

  const float own = z.m;
  const Softmax all = joined<kWaves, ENTROPY>(z, red);
  double sum_log = 0.0;
  if (a.segments == 1) {
    sum_log = log((double)all.s);
    if (tid == 0) store_row<ENTROPY>(a, r, all, sum_log, column, given);
  } else if (tid == 0) {
    float* p = a.parts + wg * 4;
    p[0] = all.m;
    p[1] = all.s;
    p[2] = all.t;
  }
  if constexpr (TOP) {
    const uint32_t mine = ordered(own);
    const uint32_t share = (a.top + kWaves - 1) / kWaves;
    const uint32_t kth = kth_largest<kIdleBits<DT>>(mine, a.top), part = kth_largest<kIdleBits<DT>>(mine, share);
    if ((tid & 63) == 0) {
      top.threshold[0][tid >> 6] = kth;
      top.threshold[1][tid >> 6] = part;
    }
    if (tid == 0) top.n = top.chosen_n = 0;
    if (tid < GCLIP_LOGPROB_MAX_TOP) top.best[tid] = 0;
    __syncthreads();
    uint32_t least = top.threshold[0][0], every = top.threshold[1][0];
#pragma unroll
    for (int i = 1; i < kWaves; ++i) {
      least = max(least, top.threshold[0][i]);
      every = min(every, top.threshold[1][i]);
    }
    least = max(least, every);
    const bool regular = all.s == all.s;
    // where fewer than k lanes have anything that can come, all that can, and
    // of what cannot the first columns, of which at most n can: enough of them
    const bool scarce = least <= ordered(kNone);
    if (scarce) least = ordered(kNone) + 1;
    uint32_t n = kCandidates + 1;
    if (regular) {
      if (mine >= least) top.chosen[atomicAdd(&top.chosen_n, 1u)] = tid;
      __syncthreads();
      const uint32_t items = top.chosen_n * a.turns;
      bool room = true;
      const uint64_t begin = (uint64_t)seg * a.turns * (uint32_t)THREADS * kU + tid;
      if (scarce && tid < a.top && begin < a.size) {
        const float v = elem_float<DT>(load_elem<DT>(row + begin * kElem<DT>));
        if (v == kNone) room = offer(top, key_of(v, (uint32_t)begin));
      }
      for (uint32_t i = tid; room && i < items; i += (uint32_t)THREADS) {
        const uint32_t u = seg * (a.turns * (uint32_t)THREADS) + top.chosen[i / a.turns] + i % a.turns * (uint32_t)THREADS;
        const uint64_t c = (uint64_t)u * kU;
        if (c >= a.size) continue;
        float v[kU];
        logits_settled<DT>(logits_raw<DT, false>(row, u, a.size), u, a.size, v);
#pragma unroll
        for (uint32_t j = 0; j < kU; ++j) {
          if (c + j < a.size && ordered(v[j]) >= least) room &= offer(top, key_of(v[j], (uint32_t)c + j));
        }
      }
      __syncthreads();
      n = top.n;
      if (n <= kCandidates) rank_candidates(top, n, a.top);
    }
    if (n > kCandidates) {
      uint64_t last = ~0ull;
      for (uint32_t i = 0; i < a.top; ++i) {
        uint64_t best = 0;
        for (uint32_t turn = 0; turn < a.turns; ++turn) {
          const uint32_t u = first + turn * (uint32_t)THREADS;
          const uint64_t c = (uint64_t)u * kU;
          if (c >= a.size) break;
          float v[kU];
          logits_settled<DT>(logits_raw<DT, false>(row, u, a.size), u, a.size, v);
#pragma unroll
          for (uint32_t j = 0; j < kU; ++j) {
            const uint64_t key = key_of(v[j], (uint32_t)c + j);
            if (c + j < a.size && key < last && key > best) best = key;
          }
        }
#pragma unroll
        for (int off = 32; off > 0; off >>= 1) {
          const uint64_t other = __shfl_xor((unsigned long long)best, off, 64);
          if (other > best) best = other;
        }
        if ((tid & 63) == 0) top.largest[tid >> 6] = best;
        __syncthreads();
        best = top.largest[0];
#pragma unroll
        for (int k = 1; k < kWaves; ++k)
          if (top.largest[k] > best) best = top.largest[k];
        if (tid == 0) top.best[i] = best;
        last = best;
        __syncthreads();  // largest[] may still be read
      }
    }
    __syncthreads();
    if (tid < a.top) {
      const uint64_t key = top.best[tid];
      if (a.segments == 1) {
        a.top_logp[(uint64_t)r * a.top + tid] = all.s == 0.0f ? kNone : (float)((double)unordered((uint32_t)(key >> 32)) - (double)all.m - sum_log);
        a.top_ids[(uint64_t)r * a.top + tid] = (int64_t)(0x7fffffffu - (uint32_t)key);
      } else {
        a.keys[wg * a.top + tid] = key;
      }
    }
  }
}

// ---------------------------------------------------------------- short rows
// A row lies in the registers of LANES lanes, NV units each, is read once, and
// its largest and its sums are taken from there.  The likeliest: those logits
// that reach the k-th largest of the lanes' largest, found and ordered within
// the wave; rows with NaNs or infinities, and those whose candidates do not
// fit, are searched k times.  Bound by the vector units: 59629 x 382 in
// bfloat16 14.4 us, 45 MB; 28860 x 186 with 20 alternatives 23.5 us, which
// were 137 by k_logp's way.
constexpr uint32_t kRowCandidates = 128;
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// Many rows have fewer lanes each, for what each row costs whatever its
// length: 59629 x 382 bfloat16 15.2 us by 16 lanes and 23.0 by 64.
constexpr uint32_t kManyShort = 8192;

// The likeliest of rows of up to kScattered columns: a lane holds every 64th
// column, so that every lane has some to choose from.
constexpr uint32_t kScattered = 512;
template <int DT, int LANES, int NV, bool ENTROPY, bool TOP, bool SCATTERED>
__global__ __launch_bounds__(kLogpThreads) void k_logp_rows(LogpArgs a) {
  constexpr uint32_t kU = kUnit<DT>;
  static_assert(!SCATTERED || (LANES == 64 && NV * kU == kScattered / 64), "columns of a lane");
  [[maybe_unused]] __shared__ uint64_t lists[kLogpThreads / 64][kRowCandidates];
  const uint64_t at = workgroup_of_grid() * (kLogpThreads / LANES) + threadIdx.x / LANES;
  if (LANES == 64 && at >= a.rows) return;
  const uint32_t lane = threadIdx.x % LANES;
  uint32_t r = (uint32_t)(at < a.rows ? at : a.rows - 1);
  if constexpr (LANES == 64) r = __builtin_amdgcn_readfirstlane(r);
  const int64_t target = a.targets ? a.targets[r] : 0;
  const bool ignored = a.targets && target == a.ignore, column = a.logp && target >= 0 && target < (int64_t)a.size;
  const uint64_t row = a.x.at + r * a.x.ld;
  // A row that counts for nothing is not read, where it has a wave to itself:
  // 8192 x 2048 bfloat16 10.3 us where all rows count, 8.7 where half do, and
  // 10.2 with the target looked at behind the loads.
  if (LANES == 64 && ignored) {
    if (lane == 0) store_nothing<ENTROPY>(a, r);
    if (TOP && lane < a.top) {
      a.top_logp[(uint64_t)r * a.top + lane] = kNone;
      a.top_ids[(uint64_t)r * a.top + lane] = -1;
    }
    return;
  }
  float given = 0.0f;
  if (column && !ignored && lane == 0) given = elem_float<DT>(load_elem<DT>(row + (uint64_t)target * kElem<DT>));
  u32x4 q[NV];
  float v[NV * kU];
  const auto column_at = [&](uint32_t j) { return SCATTERED ? lane + j * 64u : (lane + j / kU * LANES) * kU + j % kU; };
  if constexpr (SCATTERED) {
#pragma unroll
    for (uint32_t j = 0; j < NV * kU; ++j)
      v[j] = elem_float<DT>(load_elem<DT>(row + (uint64_t)min(column_at(j), a.size - 1) * kElem<DT>));
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) q[k] = logits_raw<DT, false>(row, lane + k * LANES, a.size);
  }
  float m = kNone;
  if constexpr (SCATTERED) {
#pragma unroll
    for (uint32_t j = 0; j < NV * kU; ++j) v[j] = column_at(j) < a.size ? v[j] : kNone;
  } else {
#pragma unroll
    for (int k = 0; k < NV; ++k) logits_settled<DT>(q[k], lane + k * LANES, a.size, v + k * kU);
  }
#pragma unroll
  for (uint32_t j = 0; j < NV * kU; ++j) m = fmaxf(m, v[j]);
  const float own = m;
  m = lanes_largest<LANES>(m);
  const float ref = reference(m);
  float s = 0.0f, t = 0.0f;
#pragma unroll
  for (uint32_t j = 0; j < NV * kU; ++j) {
    const float d = v[j] - ref, e = __builtin_amdgcn_exp2f(d * kLog2e);
    s += e;
    if (ENTROPY) t = __builtin_fmaf(e, fmaxf(d, kFar), t);
  }
  s = lanes_sum<LANES>(s);
  if (ENTROPY) t = lanes_sum<LANES>(t);
  const bool none = s == 0.0f;
  const float sum_log = logf(s);
  if (lane == 0 && at < a.rows) {
    if (ignored) {
      store_nothing<ENTROPY>(a, r);
    } else {
      if (a.stats) {
        a.stats[2ull * r] = none ? kNone : m;
        a.stats[2ull * r + 1] = sum_log;
      }
      if (a.logp) a.logp[r] = !column ? __uint_as_float(0x7fc00000u) : none ? kNone : given - ref - sum_log;
      if (ENTROPY) a.entropy[r] = none ? 0.0f : sum_log - t / s;
    }
  }
  if constexpr (TOP) {
    static_assert(LANES == 64, "the likeliest are a wave's");
    uint64_t* list = lists[threadIdx.x >> 6];
    uint32_t least = kth_largest<kIdleBits<DT>>(ordered(own), a.top), n = 0;
    const bool scarce = least <= ordered(kNone);  // as in k_logp
    if (scarce) least = ordered(kNone) + 1;
    const auto put = [&](bool mine, uint64_t key) {
      const uint64_t who = __ballot(mine);
      if (!who) return;
      const uint32_t place = n + __builtin_amdgcn_mbcnt_hi((uint32_t)(who >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)who, 0u));
      if (mine && place < kRowCandidates) list[place] = key;
      n += (uint32_t)__popcll(who);
    };
    if (s == s) {
      if (scarce) {
        const bool first = lane < a.top;
        const float x = first ? elem_float<DT>(load_elem<DT>(row + (uint64_t)lane * kElem<DT>)) : 0.0f;
        put(first && x == kNone, key_of(x, lane));
      }
#pragma unroll
      for (uint32_t j = 0; j < NV * kU; ++j)
        put(ordered(v[j]) >= least && column_at(j) < a.size, key_of(v[j], column_at(j)));
    } else {
      n = kRowCandidates + 1;
    }
    const auto store = [&](uint32_t place, uint64_t key) {
      a.top_logp[(uint64_t)r * a.top + place] = none ? kNone : unordered((uint32_t)(key >> 32)) - ref - sum_log;
      a.top_ids[(uint64_t)r * a.top + place] = (int64_t)(0x7fffffffu - (uint32_t)key);
    };
    if (n <= kRowCandidates) {
      wave_sync();
      for (uint32_t i = lane; i < n; i += 64) {
        const uint64_t key = list[i];
        uint32_t place = 0;
#pragma unroll 8
        for (uint32_t j = 0; j < n; ++j) place += list[j] > key ? 1u : 0u;
        if (place < a.top) store(place, key);
      }
    } else {
      uint64_t last = ~0ull;
      for (uint32_t i = 0; i < a.top; ++i) {
        uint64_t best = 0;
#pragma unroll
        for (uint32_t j = 0; j < NV * kU; ++j) {
          const uint64_t key = column_at(j) < a.size ? key_of(v[j], column_at(j)) : 0;
          if (key < last && key > best) best = key;
        }
        const uint32_t high = lanes_most((uint32_t)(best >> 32));
        const uint32_t low = lanes_most((uint32_t)(best >> 32) == high ? (uint32_t)best : 0u);
        last = ((uint64_t)high << 32) | low;
        if (lane == 0) store(i, last);
      }
    }
  }
}

// The join of a row's segments: a lane of the first wave has one, its sums
// and its largest keys in order.  No more than k segments' first keys reach
// the k-th largest of them, so at most k k keys are left.
template <int DT, bool ENTROPY, bool TOP>
__global__ __launch_bounds__(kLogpThreads) void k_logp_join(LogpArgs a) {
  constexpr int kWaves = kLogpThreads / 64;
  __shared__ float red[kWaves][4];
  [[maybe_unused]] __shared__ Top<kLogpThreads> top;
  const uint64_t row_at = workgroup_of_grid();
  if (row_at >= a.rows) return;
  const uint32_t r = (uint32_t)row_at, tid = threadIdx.x;
  const int64_t target = a.targets ? a.targets[r] : 0;
  if (a.targets && target == a.ignore) {
    store_no_row<ENTROPY, TOP>(a, r);
    return;
  }
  const bool column = a.logp && target >= 0 && target < (int64_t)a.size;
  float given = 0.0f;
  if (column) given = elem_float<DT>(load_elem<DT>(a.x.at + r * a.x.ld + (uint64_t)target * kElem<DT>));
  Softmax z{kNone, 0.0f, 0.0f};
  if (tid < a.segments) {
    const float* p = a.parts + (row_at * a.segments + tid) * 4;
    z = Softmax{p[0], p[1], p[2]};
  }
  // every key is under way while the sums are joined
  constexpr int kKeys = GCLIP_LOGPROB_MAX_TOP * kLogpSegments / kLogpThreads;
  const uint64_t* keys = TOP ? a.keys + row_at * a.segments * a.top : nullptr;
  uint64_t own[TOP ? kKeys : 1], mine = 0;
  if constexpr (TOP) {
#pragma unroll
    for (int i = 0; i < kKeys; ++i) {
      const uint32_t at = tid + i * kLogpThreads;
      own[i] = at < a.segments * a.top ? keys[at] : 0;
    }
    if (tid < a.segments) mine = keys[(uint64_t)tid * a.top];
  }
  const Softmax all = joined<kWaves, ENTROPY>(z, red);
  const double sum_log = log((double)all.s);
  if (tid == 0) store_row<ENTROPY>(a, r, all, sum_log, column, given);
  if constexpr (TOP) {
    if (tid == 0) top.n = 0;
    if (tid < GCLIP_LOGPROB_MAX_TOP) top.best[tid] = 0;
    // the k-th largest of the first keys, 0 where there are fewer
    if (tid < 64) top.first[tid] = mine;
    if (tid == 0) top.largest[0] = 0;
    __syncthreads();
    if (tid < a.segments) {
      uint32_t place = 0;
#pragma unroll 16
      for (uint32_t j = 0; j < kLogpSegments; ++j) place += top.first[j] > mine ? 1u : 0u;
      if (place == a.top - 1) top.largest[0] = mine;
    }
    __syncthreads();
    const uint64_t least = top.largest[0];
#pragma unroll
    for (int i = 0; i < kKeys; ++i)
      if (own[i] != 0 && own[i] >= least) offer(top, own[i]);  // all have room
    __syncthreads();
    rank_candidates(top, top.n, a.top);
    __syncthreads();
    if (tid < a.top) {
      const uint64_t key = top.best[tid];
      a.top_logp[row_at * a.top + tid] = all.s == 0.0f ? kNone : (float)((double)unordered((uint32_t)(key >> 32)) - (double)all.m - sum_log);
      a.top_ids[row_at * a.top + tid] = (int64_t)(0x7fffffffu - (uint32_t)key);
    }
  }
}

// dx = dlogp (1[t] - p) - dentropy p (log p + entropy), log p = x - m - s: a unit
// of 16 bytes a lane over all rows, whose numbers come from the caches.  A
// workgroup for four units a thread of one row loses what its last one does
// not fill: 7544 x 11328 bfloat16 68 us (63), 8192 x 8449 binary32 97 (91).
// Bound by memory: 8192 x 8449 binary32 with entropies 92.8 us, 554 MB at 6.0
// TB/s; 4096 x 50304 bfloat16 133 us, 824 MB at 6.2.
// Rows that count for nothing are read too: with their targets looked at first,
// by lanes or as scalars, a wave lives longer than its bytes are worth, 4096 x
// 50304 131 us and 152 where all rows count, 128 and 120 where half do.
template <int DT, bool ENTROPY, bool STREAMED>
__global__ __launch_bounds__(kLogpThreads) void k_logp_grad(LogpArgs a, Split split) {
  constexpr uint32_t kU = kUnit<DT>;
  const uint64_t i = workgroup_of_grid() * kLogpThreads + threadIdx.x;
  const uint32_t r = row_of(i, split);
  if (r >= a.rows) return;
  const uint32_t u = (uint32_t)(i - r * split.of), c = u * kU;
  u32x4 q = logits_raw<DT, STREAMED>(a.x.at + r * a.x.ld, u, a.size);
  const int64_t target = a.targets[r];
  const float m = a.stats[2ull * r], s = a.stats[2ull * r + 1], dlogp = a.dlogp[r];
  const float entropy = ENTROPY ? a.entropy[r] : 0.0f, dent = ENTROPY ? a.dentropy[r] : 0.0f;
  // s of -infinity: nothing that can come; m alone is that in a row of NaNs too
  const bool counts = target != a.ignore && s != kNone, valid = target >= 0 && target < (int64_t)a.size;
  if (a.size >= kU && c + kU > a.size) q = moved_down<DT>(q, kU - a.size % kU);
  float v[kU];
  unpack_unit<DT>(q, v);
#pragma unroll
  for (uint32_t j = 0; j < kU; ++j) {
    const float d = v[j] - m - s, p = __builtin_amdgcn_exp2f(d * kLog2e);
    const float f = ENTROPY ? __builtin_fmaf(dent, d + entropy, dlogp) : dlogp;
    v[j] = p == 0.0f ? 0.0f : -p * f;
  }
  if ((uint64_t)target - c < kU) {
#pragma unroll
    for (uint32_t j = 0; j < kU; ++j)
      if ((uint64_t)target - c == j) v[j] += dlogp;
  }
  if (!counts || !valid) {
#pragma unroll
    for (uint32_t j = 0; j < kU; ++j) v[j] = counts ? __uint_as_float(0x7fc00000u) : 0.0f;
  }
  store_unit<DT, true>(a.dx.at + r * a.dx.ld, u, a.size, pack_unit<DT>(v));
}

template <int DT, bool ENTROPY, bool TOP, int LANES, int NV, bool SCATTERED = false>
hipError_t forward_short(const LogpArgs& a, hipStream_t st) {
  constexpr uint32_t kRows = kLogpThreads / LANES;
  hipLaunchKernelGGL((k_logp_rows<DT, LANES, NV, ENTROPY, TOP, SCATTERED>), grid_of(((uint64_t)a.rows + kRows - 1) / kRows),
                     dim3(kLogpThreads), 0, st, a);
  return hipGetLastError();
}

template <int DT, bool ENTROPY, bool TOP>
hipError_t forward_short(const LogpArgs& a, hipStream_t st) {
  const uint32_t units = (a.size - 1) / kUnit<DT> + 1;
  if constexpr (!TOP) {
    const bool many = a.rows >= kManyShort;
    if (units <= 1) return forward_short<DT, ENTROPY, TOP, 1, 1>(a, st);
    if (units <= 2) return forward_short<DT, ENTROPY, TOP, 2, 1>(a, st);
    if (units <= 4) return forward_short<DT, ENTROPY, TOP, 4, 1>(a, st);
    if (units <= 8) return many ? forward_short<DT, ENTROPY, TOP, 4, 2>(a, st) : forward_short<DT, ENTROPY, TOP, 8, 1>(a, st);
    if (units <= 16) return many ? forward_short<DT, ENTROPY, TOP, 8, 2>(a, st) : forward_short<DT, ENTROPY, TOP, 16, 1>(a, st);
    if (units <= 32) return many ? forward_short<DT, ENTROPY, TOP, 8, 4>(a, st) : forward_short<DT, ENTROPY, TOP, 32, 1>(a, st);
    if (many && units <= 64) return forward_short<DT, ENTROPY, TOP, 16, 4>(a, st);
    if (many && units <= 128) return forward_short<DT, ENTROPY, TOP, 32, 4>(a, st);
  } else if (a.size <= kScattered) {
    return forward_short<DT, ENTROPY, TOP, 64, kScattered / 64 / kUnit<DT>, true>(a, st);
  }
  if (units <= 64) return forward_short<DT, ENTROPY, TOP, 64, 1>(a, st);
  if (units <= 128) return forward_short<DT, ENTROPY, TOP, 64, 2>(a, st);
  if (DT != GCLIP_F32 || units <= 256) return forward_short<DT, ENTROPY, TOP, 64, 4>(a, st);
  return forward_short<DT, ENTROPY, TOP, 64, DT == GCLIP_F32 ? 8 : 4>(a, st);
}

template <int DT, bool ENTROPY, bool TOP>
hipError_t forward_top(const LogpArgs& a, hipStream_t st) {
  if (a.segments == 0) return forward_short<DT, ENTROPY, TOP>(a, st);
  const dim3 grid = grid_of((uint64_t)a.rows * a.segments), block(a.threads);
  if (a.threads == kLogpWide) hipLaunchKernelGGL((k_logp<DT, kLogpWide, ENTROPY, TOP, false>), grid, block, 0, st, a);
  else if (a.threads == kLogpNarrow && a.streamed)
    hipLaunchKernelGGL((k_logp<DT, kLogpNarrow, ENTROPY, TOP, true>), grid, block, 0, st, a);
  else if (a.threads == kLogpNarrow)
    hipLaunchKernelGGL((k_logp<DT, kLogpNarrow, ENTROPY, TOP, false>), grid, block, 0, st, a);
  else if (a.streamed) hipLaunchKernelGGL((k_logp<DT, kLogpThreads, ENTROPY, TOP, true>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_logp<DT, kLogpThreads, ENTROPY, TOP, false>), grid, block, 0, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.segments == 1) return e;
  hipLaunchKernelGGL((k_logp_join<DT, ENTROPY, TOP>), grid_of(a.rows), dim3(kLogpThreads), 0, st, a);
  return hipGetLastError();
}

template <int DT>
hipError_t forward(const LogpArgs& a, hipStream_t st) {
  if (a.top) return a.entropy ? forward_top<DT, true, true>(a, st) : forward_top<DT, false, true>(a, st);
  return a.entropy ? forward_top<DT, true, false>(a, st) : forward_top<DT, false, false>(a, st);
}

template <int DT>
hipError_t backward(const LogpArgs& a, hipStream_t st) {
  const uint64_t units = (a.size - 1) / kUnit<DT> + 1;
  const Split split{units, 1.0 / (double)units};
  const dim3 grid = grid_of((units * a.rows + kLogpThreads - 1) / kLogpThreads), block(kLogpThreads);
  if (a.dentropy) {
    if (a.streamed) hipLaunchKernelGGL((k_logp_grad<DT, true, true>), grid, block, 0, st, a, split);
    else hipLaunchKernelGGL((k_logp_grad<DT, true, false>), grid, block, 0, st, a, split);
  } else {
    if (a.streamed) hipLaunchKernelGGL((k_logp_grad<DT, false, true>), grid, block, 0, st, a, split);
    else hipLaunchKernelGGL((k_logp_grad<DT, false, false>), grid, block, 0, st, a, split);
  }
  return hipGetLastError();
}

}  // namespace

LogpCut logp_cut(uint32_t rows, uint32_t size, int32_t dtype) {
  if (size <= kShortRow) return LogpCut{0, 0, 0};
  const uint32_t units = (size - 1) / (dtype == GCLIP_F32 ? 4u : 8u) + 1, most = (units - 1) / kLogpThreads + 1;
  if (rows >= kLogpManyRows && units <= kLogpNarrow * kLogpNarrowTurns)
    return LogpCut{1, (units - 1) / kLogpNarrow + 1, kLogpNarrow};
  if (rows > kLogpFewRows) return LogpCut{1, most, kLogpThreads};
  if (units <= kLogpWide * std::max(kLogpTurns, rows / kLogpRowsATurn)) return LogpCut{1, (units - 1) / kLogpWide + 1, kLogpWide};
  const uint32_t wanted = std::min(kLogpSegments, 4 * kLogpFewRows / std::max(rows, 1u));
  const uint32_t turns = (most - 1) / wanted + 1;
  return LogpCut{(most - 1) / turns + 1, turns, kLogpThreads};
}

hipError_t launch_logprob_forward(const LogpArgs& a, int32_t dtype, hipStream_t st) {
  switch (dtype) {
    case GCLIP_F32: return forward<GCLIP_F32>(a, st);
    case GCLIP_F16: return forward<GCLIP_F16>(a, st);
    default: return forward<GCLIP_BF16>(a, st);
  }
}

hipError_t launch_logprob_backward(const LogpArgs& a, int32_t dtype, hipStream_t st) {
  switch (dtype) {
    case GCLIP_F32: return backward<GCLIP_F32>(a, st);
    case GCLIP_F16: return backward<GCLIP_F16>(a, st);
    default: return backward<GCLIP_BF16>(a, st);
  }
}

}  // namespace gclip
