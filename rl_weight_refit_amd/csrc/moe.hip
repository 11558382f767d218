// HIP kernels around the experts' products, written for gfx950 (CDNA4,
// wave64): routing, the slots' order by expert, the combination of the
// experts' rows, and the backward passes of routing and combination.
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "ops.hpp"
#include "ops_device.hpp"

namespace rs {
namespace {

// --------------------------------------------------------------------------
// Routing.
//
// Sixteen lanes hold one token's experts (four tokens per wave), the row of
// a DPP operation, so every reduction over a token is four DPP steps.  A
// group of experts takes 16 / G' lanes (G' = the groups rounded up to a power
// of two) and each lane a run of consecutive experts of one group, so a
// group's score is a scan of the lane's own values and a merge over its
// lanes.
//
// The choice is made on 32-bit keys: the float's bits in ascending order,
// their lowest bits replaced by the place within the lane's run.  The largest
// key below the last one chosen is best + max(key - best) in wrapping
// arithmetic (chosen and absent ones wrap to small numbers), so nothing is
// removed and no index is carried along.  What the replaced bits and float32
// scores can get wrong is bounded afterwards, all slots at once; a token with
// two neighbours nearer than that bound is chosen again in double precision.
// Where order does not depend on the scores (no bias, no sums) the keys are
// the logits', and logits of 16-bit precision leave room for the whole expert
// number: then every choice is exact, equal logits included.
// --------------------------------------------------------------------------

struct RouteArgs {
  const void* logits;
  const float* bias;
  const uint8_t* mask;
  int32_t* ids;
  float* weights;
  int64_t n_tokens, stride;
  int32_t n_experts, top_k, n_groups, top_groups, group_top, renormalise, sigmoid, dtype;
  int32_t group_size, lanes_shift, run;  // experts a group, log2 of the lanes a group, experts a lane
  int32_t by_logit;                      // order by logits
  float scale;
};

// Reductions over the sixteen lanes of a token, all lanes receiving the
// result: partners by quad permutes, then mirrored halves and rows.
template <int CTRL>
__device__ __forceinline__ int dpp(int v) {
  return __builtin_amdgcn_update_dpp(0, v, CTRL, 0xF, 0xF, true);  // every lane has a partner
}
template <typename Op>
__device__ __forceinline__ int row16(int v, Op op) {
  v = op(v, dpp<0xB1>(v));   // quad_perm [1,0,3,2]
  v = op(v, dpp<0x4E>(v));   // quad_perm [2,3,0,1]
  v = op(v, dpp<0x141>(v));  // row_half_mirror
  return op(v, dpp<0x140>(v));  // row_mirror
}
__device__ __forceinline__ uint32_t row_max16u(uint32_t v) {
  return uint32_t(row16(int(v), [](int a, int b) { return int(max(uint32_t(a), uint32_t(b))); }));
}
__device__ __forceinline__ float row_max16f(float v) {
  return __int_as_float(row16(__float_as_int(v), [](int a, int b) {
    return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
  }));
}
__device__ __forceinline__ float row_sum16f(float v) {
  return __int_as_float(row16(__float_as_int(v), [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}
__device__ __forceinline__ double row_max16(double v) {
#pragma unroll
  for (int d = 8; d; d >>= 1) v = fmax(v, __shfl_xor(v, d, 16));
  return v;
}
__device__ __forceinline__ double row_sum16(double v) {
#pragma unroll
  for (int d = 8; d; d >>= 1) v += __shfl_xor(v, d, 16);
  return v;
}

// RUN consecutive elements from index i, of which the first `held` count;
// -infinity behind them.
template <int RUN>
__device__ __forceinline__ void load_run(const void* p, int dtype, int64_t i, int held, float (&x)[RUN]) {
  if (held == RUN && RUN % 8 == 0) {
#pragma unroll
    for (int j = 0; j < RUN; j += 8) load8(p, dtype, i + j, &x[j]);
  } else if (held == RUN && RUN == 4 && dtype == RS_F32) {
    const ou32x4 v = *reinterpret_cast<const ou32x4_2*>(static_cast<const float*>(p) + i);
#pragma unroll
    for (int j = 0; j < RUN; ++j) x[j] = __uint_as_float(v[j & 3]);
  } else {
#pragma unroll
    for (int j = 0; j < RUN; ++j) x[j] = j < held ? load1(p, dtype, i + j) : -INFINITY;
  }
}
template <int RUN>
__device__ __forceinline__ void nan_to_lowest(float (&x)[RUN]) {
#pragma unroll
  for (int j = 0; j < RUN; ++j) x[j] = x[j] == x[j] ? x[j] : -INFINITY;
}
// Whether any lane of the wave holds an infinity or NaN.
template <int RUN>
__device__ __forceinline__ bool any_special(const float (&x)[RUN]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < RUN; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
  return __ballot(top >= 0x7F800000u) != 0;
}

// exp(x - m) of one logit against its token's largest, in double precision
// (0 for NaN and -infinity; infinite logits share the token's weight).
__device__ __forceinline__ double exp64(double x, double m) {
  return !(x > -INFINITY) ? 0.0 : x == m ? 1.0 : exp(x - m);
}
__device__ __forceinline__ double score64(double x, double m, double z, bool sigmoid) {
  if (!(x > -INFINITY)) return 0.0;
  return sigmoid ? 1.0 / (1.0 + exp(-x)) : exp64(x, m) / z;
}

// The choice in double precision, for tokens that float32 leaves open.
template <int RUN>
__device__ __forceinline__ void choose64(const RouteArgs& p, int64_t t, int lane, int group, int first, int held,
                                         int32_t (&slot)[2]) {
  float x[RUN];
  load_run<RUN>(p.logits, p.dtype, t * p.stride + first, held, x);
  nan_to_lowest(x);
  double m = -INFINITY, z = 1.0;
  if (!p.sigmoid) {
#pragma unroll
    for (int j = 0; j < RUN; ++j) m = fmax(m, double(x[j]));
    m = row_max16(m);
    z = 0.0;
#pragma unroll
    for (int j = 0; j < RUN; ++j) z += exp64(x[j], m);
    z = row_sum16(z);
  }
  double v[RUN];
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    if (!(x[j] > -INFINITY)) v[j] = -INFINITY;
    else if (p.by_logit) v[j] = !p.sigmoid && m == INFINITY && x[j] < m ? 0.0 : double(x[j]);
    else v[j] = score64(x[j], m, z, p.sigmoid) + (p.bias ? double(p.bias[first + j]) : 0.0);
    if (v[j] != v[j]) v[j] = -INFINITY;  // the bias is NaN
  }
  if (p.n_groups > 1) {
    double a = -INFINITY, b = -INFINITY;  // the two largest values of the group
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      b = fmax(b, fmin(a, v[j]));
      a = fmax(a, v[j]);
    }
    for (int d = 1; d < 1 << p.lanes_shift; d <<= 1) {
      const double oa = __shfl_xor(a, d, 16), ob = __shfl_xor(b, d, 16);
      b = fmax(fmin(a, oa), fmax(b, ob));
      a = fmax(a, oa);
    }
    const double gs = p.group_top == 2 && p.group_size > 1 ? a + b : a;
    int before = 0;
    for (int g = 0; g < p.n_groups; ++g) {
      const double o = __shfl(gs, g << p.lanes_shift, 16);
      before += o > gs || (o == gs && g < group);
    }
    if (before >= p.top_groups) {
#pragma unroll
      for (int j = 0; j < RUN; ++j) v[j] = -INFINITY;
    }
  }
  slot[0] = slot[1] = -1;
  for (int i = 0; i < p.top_k; ++i) {
    double best = -INFINITY;
    int e = kMaxExperts;
#pragma unroll
    for (int j = 0; j < RUN; ++j)
      if (v[j] > best) best = v[j], e = first + j;
#pragma unroll
    for (int d = 8; d; d >>= 1) {
      const double o = __shfl_xor(best, d, 16);
      const int oe = __shfl_xor(e, d, 16);
      if (o > best || (o == best && oe < e)) best = o, e = oe;
    }
    if (e == kMaxExperts) break;
    if (lane == (i & 15)) slot[i >> 4] = e;
#pragma unroll
    for (int j = 0; j < RUN; ++j)
      if (first + j == e) v[j] = -INFINITY;
  }
}

__device__ __forceinline__ uint32_t key_of(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return __uint_as_float(k ^ (uint32_t(int32_t(~k) >> 31) | 0x80000000u));
}

// How far the float32 value v = s + bias may be from the exact one, in units
// of 2^-24.  Softmax, with d the logit's distance from the largest: exp(-d) is
// off by 2.3 d + 2 (the difference and its product with log2 e rounded, that
// constant's own error, one step of the instruction), the sum by 11 from its
// terms (their errors weighted by themselves, of 1024 at the most), by RUN - 1
// from a lane's additions, each of which may round the same way, and by 4 from
// the lanes', quotient and product by 2, and d is at most -log s: below
// s (RUN + 18 + 2.3 (-log s)).  Sigmoid: exp as before, but only s (1 - s) of it
// arrives, below 0.8; the addition and the reciprocal (one step of the
// instruction) leave below 0.8 + 3 s.  And v's own rounding; what the
// instruction makes 0 lies below 2^-126.
template <int RUN>
__device__ __forceinline__ float error_of(float s, float v, bool sigmoid) {
  constexpr float kSum = RUN <= 16 ? 17.0f : (RUN + 18) * 0.5f;
  const float f = sigmoid ? 0.5f + 1.5f * s : s * (kSum - 1.2f * __logf(s + 0x1p-126f));
  return fmaf(0x1p-23f, f + fabsf(v), 0x1p-125f);
}

// The sigmoid and what is left of it to 1, both to a few units of themselves.
struct Sigmoid {
  float s, rest;
};
__device__ __forceinline__ Sigmoid sigmoid32(float x) {
  const float e = expf(-fabsf(x)), r = 1.0f / (1.0f + e);
  return x < 0.0f ? Sigmoid{e * r, r} : Sigmoid{r, e * r};
}

__device__ __forceinline__ float score32(float x, float m, float rz, bool sigmoid) {
  if (!(x > -INFINITY)) return 0.0f;
  return sigmoid ? sigmoid32(x).s : (x == m ? 1.0f : expf(x - m)) * rz;
}

// Renormalised weights where a slot's score lies near 2^-126 or below: the
// scores are taken relative to the largest slot's, so that their quotients keep
// their digits.  `top` is the largest of the slots' logits, m the token's
// largest (softmax).  kZero: where double precision has 0 for every score, all
// weights are 0.
struct Share {
  float base;
  bool none;
};
__device__ __forceinline__ Share share_base(float top, float m, bool sigmoid) {
  constexpr float kZero = 745.0f;  // e^-745.13 is half of the smallest number
  if (sigmoid) return Share{fminf(top, 0.0f), !(top >= -kZero)};
  return Share{top, !(top > -INFINITY) || (top != m && !(m - top <= kZero))};
}
__device__ __forceinline__ float share32(float x, const Share& b, bool sigmoid) {
  if (b.none || !(x > -INFINITY)) return 0.0f;
  const float e = x == b.base ? 1.0f : expf(x - b.base);
  if (!sigmoid) return e;
  return x < 0.0f ? e / (1.0f + expf(x)) : 1.0f / (1.0f + expf(-x));
}

template <int RUN>
__global__ __launch_bounds__(256) void rs_route_kernel(RouteArgs p) {
  constexpr uint32_t kPlace = RUN - 1;  // the key bits that hold the place in the run
  constexpr int kPlaceBits = RUN > 64 ? 7 : 6;
  constexpr uint32_t kExpert = (16u << kPlaceBits) - 1;  // those that hold lane and place
  const int lane = threadIdx.x & 15;
  const int64_t t = int64_t(blockIdx.x) * 16 + (threadIdx.x >> 4);
  const bool live = t < p.n_tokens && !(p.mask && !p.mask[t]);
  const int group = lane >> p.lanes_shift;
  const int in_group = (lane & ((1 << p.lanes_shift) - 1)) * p.run;  // first expert of the run within its group
  const int first = group * p.group_size + in_group;
  const int held = group < p.n_groups && live ? max(0, min(p.run, p.group_size - in_group)) : 0;

  float x[RUN];
  load_run<RUN>(p.logits, p.dtype, t * p.stride + first, held, x);
  const bool special = any_special(x);  // ordinary logits need no care for infinities and NaN
  if (special) nan_to_lowest(x);
  float m = 0.0f, rz = 1.0f;
  float v[RUN];
  if (!p.sigmoid) {
    m = x[0];
#pragma unroll
    for (int j = 1; j < RUN; ++j) m = fmaxf(m, x[j]);
    m = row_max16f(m);
    float z = 0.0f;
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      v[j] = x[j] > -INFINITY ? (x[j] == m ? 1.0f : __expf(x[j] - m)) : 0.0f;
      z += v[j];
    }
    z = row_sum16f(z);
    rz = z > 0.0f ? 1.0f / z : 0.0f;
#pragma unroll
    for (int j = 0; j < RUN; ++j) v[j] *= rz;
  } else if (!p.by_logit) {
#pragma unroll
    for (int j = 0; j < RUN; ++j) v[j] = __builtin_amdgcn_rcpf(1.0f + __expf(-x[j]));
  }
  float reach = 0.0f;
  if (p.by_logit) {
#pragma unroll
    for (int j = 0; j < RUN; ++j)  // next to an infinite logit the finite ones score 0, all alike
      v[j] = !p.sigmoid && m == INFINITY && x[j] < m && x[j] > -INFINITY ? 0.0f : x[j] + 0.0f;  // -0 is 0
  } else if (p.bias) {
    float b[RUN];
    load_run<RUN>(p.bias, RS_F32, first, held, b);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      if (special) b[j] = j < held ? b[j] : 0.0f;
      top = max(top, __float_as_uint(b[j]) & 0x7FFFFFFFu);
      v[j] += b[j];
    }
    reach = __uint_as_float(top);
    if (__ballot(top > 0x7F800000u)) {  // a NaN among them: |bias| is at most |v| + 1
      reach = 0.0f;
#pragma unroll
      for (int j = 0; j < RUN; ++j) {
        reach = fmaxf(reach, fabsf(v[j]) + 1.0f);
        v[j] = v[j] == v[j] ? v[j] : -INFINITY;
      }
    }
    reach = row_max16f(reach);
  }
  if (special) {
#pragma unroll
    for (int j = 0; j < RUN; ++j) v[j] = x[j] > -INFINITY ? v[j] : -INFINITY;
  }

  bool sure = true;
  bool on = true;
  if (p.n_groups > 1) {
    float a = v[0], b = -INFINITY;  // the two largest values of the group
#pragma unroll
    for (int j = 1; j < RUN; ++j) {
      b = fmaxf(b, fminf(a, v[j]));
      a = fmaxf(a, v[j]);
    }
    for (int d = 1; d < 1 << p.lanes_shift; d <<= 1) {
      const float oa = __shfl_xor(a, d, 16), ob = __shfl_xor(b, d, 16);
      b = fmaxf(fminf(a, oa), fmaxf(b, ob));
      a = fmaxf(a, oa);
    }
    const bool two = p.group_top == 2 && p.group_size > 1;
    const float gs = two ? a + b : a;
    int before = 0;  // groups that come before this one
    for (int g = 0; g < p.n_groups; ++g) {
      const float o = __shfl(gs, g << p.lanes_shift, 16);
      before += o > gs || (o == gs && g < group);
    }
    on = before < p.top_groups;
    if (!p.by_logit) {
      // the scores lie within what v and the largest |bias| allow; the error grows with them
      const auto off = [&](float v) { return error_of<RUN>(fminf(1.0f, fabsf(v) + reach), v, p.sigmoid); };
      const float err = gs > -INFINITY ? off(a) + (two ? off(b) : 0.0f) + 0x1p-23f * fabsf(gs) : 0.0f;
      const float low = row_max16f(on || group >= p.n_groups ? -INFINITY : gs + err);        // the best group left out
      const float high = -row_max16f(on && group < p.n_groups ? err - gs : -INFINITY);       // the last one kept
      sure = high > low || low == -INFINITY;
    }
  }

  // Keys; those up to kNone, -infinity's, are no candidates.
  constexpr uint32_t kNone = 0x007FFFFFu;
  bool whole = false;  // logits of at most 13 (12) mantissa bits: room for the lane too
  if (p.by_logit) {
    uint32_t low = 0;
#pragma unroll
    for (int j = 0; j < RUN; ++j) low |= __float_as_uint(v[j]) & kExpert;
    whole = row_max16u(low) == 0;
  }
  uint32_t key[RUN];
  const uint32_t keep = !on ? 0u : whole ? ~kExpert : ~kPlace;
  const uint32_t tag = whole ? uint32_t(15 - lane) << kPlaceBits : 0u;
#pragma unroll
  for (int j = 0; j < RUN; ++j) key[j] = (key_of(v[j]) & keep) | (kPlace - j);
  if (p.by_logit) {
#pragma unroll
    for (int j = 0; j < RUN; ++j) key[j] |= tag;
  }
  // Slot i in lane i % 16; one slot more than asked for, to compare the last.
  uint32_t chosen[3] = {0, 0, 0}, winner[3] = {0, 0, 0};
  uint32_t best = 0;
  bool left = true;
  const auto pick = [&](int i, uint32_t& key_at, uint32_t& won_at) {
    uint32_t mine = 0;
#pragma unroll
    for (int j = 0; j < RUN; ++j) mine = max(mine, key[j] - best);
    const uint32_t far = row_max16u(mine);
    best = left ? best + far : 0;
    left = best > kNone;
    const uint64_t won = __ballot(mine == far);
    if (__popcll(won) > 4) {  // more than one lane in some token: equal keys
      const uint32_t at = uint32_t(won >> (threadIdx.x & 48)) & 0xFFFFu;
      if (left && (at & (at - 1))) sure = false;
    }
    if (lane == i) {
      key_at = left ? best : 0;
      won_at = threadIdx.x & 32 ? uint32_t(won >> 32) : uint32_t(won);
    }
  };
  const auto expert_of = [&](uint32_t key_at, uint32_t won_at) {
    if (!key_at) return -1;
    const int place = int(kPlace - (key_at & kPlace)), from = __ffs(int(won_at >> (threadIdx.x & 16) & 0xFFFFu)) - 1;
    return (from >> p.lanes_shift) * p.group_size + (from & ((1 << p.lanes_shift) - 1)) * p.run + place;
  };
  const auto logit_of = [&](int e) { return e < 0 ? -INFINITY : load1(p.logits, p.dtype, t * p.stride + e); };
  // The most that a slot's value can exactly be (a key's value is short of
  // the float32 one by less than RUN steps), and the least.
  const auto most = [&](uint32_t k, float score) {
    const float v = value_of(k | kPlace);
    return !k ? -INFINITY : p.by_logit ? v : v + error_of<RUN>(score, v, p.sigmoid);
  };
  const auto least = [&](uint32_t k, float score) {
    const float v = value_of(k & ~kPlace);
    return p.by_logit ? v : v - error_of<RUN>(score, v, p.sigmoid);
  };
#pragma unroll
  for (int h = 0; h < 3; ++h)
    for (int i = 0; i < 16 && h * 16 + i <= p.top_k; ++i) pick(i, chosen[h], winner[h]);
  // Expert and score of each lane's slots, the one beyond the last among them.
  int32_t slot[3] = {-1, -1, -1};
  float logit[3] = {-INFINITY, -INFINITY, -INFINITY}, s[3] = {0.0f, 0.0f, 0.0f};
  const auto take = [&](int h, int e) {
    slot[h] = e;
    logit[h] = logit_of(e);
    s[h] = score32(logit[h], m, rz, p.sigmoid);
  };
#pragma unroll
  for (int h = 0; h < 3; ++h) {
    if (h * 16 > p.top_k) continue;
    take(h, expert_of(chosen[h], winner[h]));
  }
  // Each slot against the next: in order if the values lie further apart than
  // both can be off.
  bool near = false;
  if (!whole) {
    float high[3];
#pragma unroll
    for (int h = 0; h < 3; ++h) high[h] = h * 16 > p.top_k ? -INFINITY : most(chosen[h], s[h]);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h * 16 >= p.top_k) continue;
      const float ahead = __shfl(high[h], (lane + 1) & 15, 16), wrap = __shfl(high[h + 1], 0, 16);
      if (h * 16 + lane < p.top_k && chosen[h] && !(least(chosen[h], s[h]) > (lane == 15 ? wrap : ahead))) near = true;
    }
  }
  // Of a token's sixteen lanes, those with b.
  const auto row_any = [&](bool b) { return uint32_t(__ballot(b) >> (threadIdx.x & 48)) & 0xFFFFu; };
  bool close = live && row_any(near);
  bool open = live && row_any(!sure);
  if (p.top_k <= 12 && __ballot(close && !open)) {
    // Neighbours too near: sixteen slots are taken and put in order by their
    // values in double precision.  Whatever was not taken is at most the
    // sixteenth; if that may reach the last slot, the token stays open.
    for (int i = p.top_k + 1; i < 16; ++i) pick(i, chosen[0], winner[0]);
    const int e = expert_of(chosen[0], winner[0]);
    const float l = logit_of(e);
    double v64 = -INFINITY;
    if (p.by_logit) {
      if (e >= 0) v64 = !p.sigmoid && m == INFINITY && l < m ? 0.0 : double(l);
    } else {
      double z = 1.0;
      if (!p.sigmoid) {
        float again[RUN];
        load_run<RUN>(p.logits, p.dtype, t * p.stride + first, held, again);
        nan_to_lowest(again);
        z = 0.0;
#pragma unroll
        for (int j = 0; j < RUN; ++j) z += exp64(again[j], m);
        z = row_sum16(z);
      }
      if (e >= 0) v64 = score64(l, m, z, p.sigmoid) + (p.bias ? double(p.bias[e]) : 0.0);
    }
    const float beyond = __shfl(most(chosen[0], score32(l, m, rz, p.sigmoid)), 15, 16);
    int rank = 0;
    for (int j = 0; j < 16; ++j) {
      const double o = __shfl(v64, j, 16);
      const int oe = __shfl(e, j, 16);
      rank += o > v64 || (o == v64 && oe < e);
    }
    const bool held_off = !row_any(rank < p.top_k && e >= 0 && !(v64 > double(beyond)));
    int sorted = -1;
    for (int j = 0; j < 16; ++j) {
      const int oe = __shfl(e, j, 16);
      if (__shfl(rank, j, 16) == lane && oe >= 0) sorted = oe;
    }
    if (close && row_any(!sure)) open = true;
    if (close && held_off && !open) {
      take(0, sorted);
      close = false;
    }
  }
  open = open || close;
  if (open) {
    int32_t again[2];
    choose64<RUN>(p, t, lane, group, first, held, again);
#pragma unroll
    for (int h = 0; h < 2; ++h) take(h, again[h]);
  }

  if (t >= p.n_tokens) return;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (h * 16 + lane >= p.top_k) slot[h] = -1, logit[h] = -INFINITY, s[h] = 0.0f;
  if (p.renormalise) {
    // (65,536 tokens of 128 experts: 19.1 us if every token takes the shares, 18.3 so.)
    if (row_any((slot[0] >= 0 && s[0] < 0x1p-120f) || (slot[1] >= 0 && s[1] < 0x1p-120f))) {
      const Share base = share_base(row_max16f(fmaxf(logit[0], logit[1])), m, p.sigmoid);
#pragma unroll
      for (int h = 0; h < 2; ++h) s[h] = share32(logit[h], base, p.sigmoid);
    }
    const float sum = row_sum16f(s[0] + s[1]);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (h * 16 < p.top_k) s[h] = sum > 0.0f ? s[h] / sum : 0.0f;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int i = h * 16 + lane;
    if (i < p.top_k) {
      p.ids[t * p.top_k + i] = slot[h];
      p.weights[t * p.top_k + i] = s[h] * p.scale;
    }
  }
}

// Gradient of the weights, with g_j = scale * dweights_j and p_j = s at slot
// j.  dl_e = s_e (H_e - sum_j g_j p_j) for the softmax and s_e (1 - s_e) H_e
// for the sigmoid, H_e being the sum of g_j over the slots that name e.
// Renormalised weights, with their shares r_j = p_j / sum p: dl_e is the sum of
// r_j (g_j - sum g r) over the slots that name e (the softmax's sum over all
// slots is 0), times 1 - s_e for the sigmoid.  The expert with the largest
// score, whose own part of such a sum may be next to all of it, takes the
// others' instead: H_e (1 - s_e) - sum over the others, 1 - s_e being their
// scores' sum.  Sixteen lanes a token, a run of
// experts and one or two slots a lane; H (what is not the softmax's own, with
// its factors: dl_e itself) goes through LDS, each expert written by the first
// slot that names it with the sum of all that do, in slot order.
struct RouteGradArgs {
  const void* logits;
  const int32_t* ids;
  const float* dweights;
  void* dlogits;
  int64_t n_tokens, stride, dstride;
  int32_t n_experts, top_k, renormalise, sigmoid, dtype, run;
  float scale;
};

template <int RUN>
__global__ __launch_bounds__(RUN > 16 ? 64 : 256) void rs_route_grad_kernel(RouteGradArgs p) {
  constexpr int kTokens = RUN > 16 ? 4 : 16;
  constexpr int kPitch = RUN * 16 + 16;
  __shared__ __attribute__((aligned(16))) float turn[kTokens * kPitch];
  const int lane = threadIdx.x & 15;
  const int64_t t = int64_t(blockIdx.x) * kTokens + (threadIdx.x >> 4);
  const bool live = t < p.n_tokens;
  const int64_t row = live ? t * p.stride : 0;
  const int first = lane * p.run;
  const int held = live ? max(0, min(p.run, p.n_experts - first)) : 0;
  float s[RUN];
  float m = 0.0f, z = 1.0f, rest = 0.0f;  // rest: what a score above a half leaves to the others
  if (!p.sigmoid) {
    float x[RUN];
    load_run<RUN>(p.logits, p.dtype, row + first, held, x);
    nan_to_lowest(x);
    m = x[0];
#pragma unroll
    for (int j = 1; j < RUN; ++j) m = fmaxf(m, x[j]);
    m = row_max16f(m);
    z = 0.0f;
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      s[j] = x[j] > -INFINITY ? (x[j] == m ? 1.0f : expf(x[j] - m)) : 0.0f;
      z += s[j];
    }
    z = row_sum16f(z);
    const float rz = z > 0.0f ? 1.0f / z : 0.0f;
#pragma unroll
    for (int j = 0; j < RUN; ++j) {
      s[j] *= rz;
      rest += s[j] > 0.5f ? 0.0f : s[j];
    }
    rest = row_sum16f(rest);
    z = rz;
  }
  int32_t id[2];
  float l[2], q[2], h[2];
#pragma unroll
  for (int a = 0; a < 2; ++a) {
    const int i = a * 16 + lane;
    id[a] = live && i < p.top_k ? p.ids[t * p.top_k + i] : -1;
    if (id[a] < 0 || id[a] >= p.n_experts) id[a] = -1;
    l[a] = id[a] < 0 ? -INFINITY : load1(p.logits, p.dtype, row + id[a]);
    l[a] = l[a] == l[a] ? l[a] : -INFINITY;
    // a score that is 0 for good takes no gradient, whatever dweights holds there
    h[a] = l[a] > -INFINITY ? p.scale * p.dweights[t * p.top_k + i] : 0.0f;
  }
  float mean = 0.0f, others = 0.0f;
  if (p.renormalise) {
    const float top = row_max16f(fmaxf(l[0], l[1]));
    const Share base = share_base(top, m, p.sigmoid);
    const int first_of_all = int(row_max16u(max(l[0] == top ? uint32_t(id[0] + 1) : 0u, l[1] == top ? uint32_t(id[1] + 1) : 0u))) - 1;
#pragma unroll
    for (int a = 0; a < 2; ++a) q[a] = share32(l[a], base, p.sigmoid);
    const float sum = row_sum16f(q[0] + q[1]);
#pragma unroll
    for (int a = 0; a < 2; ++a) q[a] = sum > 0.0f ? q[a] / sum : 0.0f;
    const bool large[2] = {id[0] == first_of_all, id[1] == first_of_all};
    const float left = row_sum16f((large[0] ? 0.0f : q[0]) + (large[1] ? 0.0f : q[1]));
    others = row_sum16f((large[0] ? 0.0f : h[0] * q[0]) + (large[1] ? 0.0f : h[1] * q[1]));
    mean = others + row_sum16f((large[0] ? h[0] * q[0] : 0.0f) + (large[1] ? h[1] * q[1] : 0.0f));
#pragma unroll
    for (int a = 0; a < 2; ++a) h[a] = q[a] * (large[a] ? h[a] * left - others : h[a] - mean);
  } else {
#pragma unroll
    for (int a = 0; a < 2; ++a) q[a] = score32(l[a], m, z, p.sigmoid);
    if (!p.sigmoid) {
      mean = row_sum16f(h[0] * q[0] + h[1] * q[1]);
      others = row_sum16f((q[0] > 0.5f ? 0.0f : h[0] * q[0]) + (q[1] > 0.5f ? 0.0f : h[1] * q[1]));
    } else {
      h[0] *= q[0], h[1] *= q[1];
    }
  }
  if (p.sigmoid) {
#pragma unroll
    for (int a = 0; a < 2; ++a) h[a] = l[a] > -INFINITY ? h[a] * sigmoid32(l[a]).rest : 0.0f;
  }
  float* mine = turn + (threadIdx.x >> 4) * kPitch;
#pragma unroll
  for (int j = 0; j < RUN; ++j) mine[lane + 16 * j] = 0.0f;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  float sum[2] = {0.0f, 0.0f};
  bool head[2] = {true, true};  // no slot before names the same expert
  for (int i = 0; i < p.top_k; ++i) {
    const int oi = __shfl(i < 16 ? id[0] : id[1], i & 15, 16);
    const float oh = __shfl(i < 16 ? h[0] : h[1], i & 15, 16);
#pragma unroll
    for (int a = 0; a < 2; ++a) {
      if (oi == id[a]) {
        sum[a] += oh;
        if (i < a * 16 + lane) head[a] = false;
      }
    }
  }
#pragma unroll
  for (int a = 0; a < 2; ++a)
    if (id[a] >= 0 && head[a]) mine[id[a] / p.run * RUN + id[a] % p.run] = sum[a];
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
  for (int j = 0; j < RUN; ++j) {
    const float H = mine[lane * RUN + j];
    const float d = s[j] > 0.5f ? H * rest - others : H - mean;
    s[j] = p.sigmoid || p.renormalise ? H : s[j] > 0.0f ? s[j] * d : 0.0f;
  }
  const int64_t to = t * p.dstride + first;
  if (RUN % 8 == 0 && held == RUN) {
    // Pieces of runs longer than 32 bytes meet in the caches (65,536 tokens,
    // float32: 1024 experts 122 us, 567 by non-temporal stores, 256 28 and 75;
    // bf16, 256 experts, 32 bytes: 28.9 and 27.2).
    const bool streamed = RUN * dtype_size(p.dtype) <= 32;
#pragma unroll
    for (int j = 0; j < RUN; j += 8) {
      if (streamed) store8(p.dlogits, p.dtype, to + j, 8, &s[j]);
      else store8<false>(p.dlogits, p.dtype, to + j, 8, &s[j]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < RUN; ++j)
      if (j < held) store1(p.dlogits, p.dtype, to + j, s[j]);
  }
}

// --------------------------------------------------------------------------
// Slots in expert order: a stable counting sort without atomics on global
// memory, so the order never varies.  Chunks of 2048 slots; one alone takes one
// launch (64 tokens x 8: 4 us on the device), more take a launch for the
// chunks' counts and one that places (32,768 x 8: 3.7 and 9.4 us, the time of
// dependent loads and of ballots over an expert number's bits), many a launch
// for running totals between them.
// --------------------------------------------------------------------------

struct SortArgs {
  const int32_t* ids;
  int32_t* offsets;
  int32_t* tokens;
  int32_t* positions;
  int32_t* hist;  // [chunks][n_experts]
  int64_t n_slots;
  int32_t top_k, first, n_experts, chunks;
};

constexpr int kSortThreads = 512;
constexpr int kSortWaves = kSortThreads / 64;

__device__ __forceinline__ int local_expert(const SortArgs& p, int64_t i) {
  if (i >= p.n_slots) return -1;
  const int32_t id = p.ids[i];
  const int64_t e = int64_t(id) - p.first;
  return id >= 0 && e >= 0 && e < p.n_experts ? int(e) : -1;
}

// Slots per expert of each chunk.
__global__ __launch_bounds__(kSortThreads) void rs_sort_count_kernel(SortArgs p) {
  __shared__ int32_t cnt[kMaxExperts];
  const int64_t base = int64_t(blockIdx.x) * kSortChunk;
  int e[kSortChunk / kSortThreads];
#pragma unroll
  for (int k = 0; k < kSortChunk / kSortThreads; ++k) e[k] = local_expert(p, base + k * kSortThreads + threadIdx.x);
  for (int i = threadIdx.x; i < p.n_experts; i += kSortThreads) cnt[i] = 0;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kSortChunk / kSortThreads; ++k)
    if (e[k] >= 0) atomicAdd(&cnt[e[k]], 1);
  __syncthreads();
  for (int i = threadIdx.x; i < p.n_experts; i += kSortThreads)
    p.hist[int64_t(blockIdx.x) * p.n_experts + i] = cnt[i];
}

// Running totals over the chunks, in place: sixteen experts a workgroup, whose
// sixty-four parts take a run of chunks each.
__global__ __launch_bounds__(1024) void rs_sort_total_kernel(SortArgs p) {
  __shared__ int32_t sums[64][16];
  const int e = int(blockIdx.x) * 16 + (threadIdx.x & 15), part = threadIdx.x >> 4;
  const int each = (p.chunks + 63) / 64, from = part * each, to = e < p.n_experts ? min(p.chunks, from + each) : 0;
  const auto walk = [&](auto with) {
    for (int c0 = from; c0 < to; c0 += 16) {
      int32_t h[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) h[u] = c0 + u < to ? p.hist[int64_t(c0 + u) * p.n_experts + e] : 0;
#pragma unroll
      for (int u = 0; u < 16; ++u) with(c0 + u, h[u]);
    }
  };
  int sum = 0;
  walk([&](int, int32_t h) { sum += h; });
  sums[part][threadIdx.x & 15] = sum;
  __syncthreads();
  sum = 0;
  for (int i = 0; i < part; ++i) sum += sums[i][threadIdx.x & 15];
  walk([&](int c, int32_t h) {
    sum += h;
    if (c < to) p.hist[int64_t(c) * p.n_experts + e] = sum;
  });
}

// Where the counts before a chunk come from: there is one chunk; the chunks'
// counts, added up by every workgroup; or running totals.
enum SortForm { kSortOne, kSortCounts, kSortTotals };

// Where the slots of every expert begin in this chunk, then their ranks.
// Wave w takes the chunk's w-th eighth, 64 slots at a time.
template <SortForm FORM>
__global__ __launch_bounds__(kSortThreads) void rs_sort_place_kernel(SortArgs p) {
  constexpr bool ONE = FORM == kSortOne;
  constexpr int kEach = kSortChunk / kSortWaves, kTurns = kEach / 64;
  __shared__ int32_t next[kSortWaves][kMaxExperts];
  __shared__ int32_t start[kMaxExperts];
  __shared__ int32_t before[kMaxExperts];
  __shared__ int32_t wave_sum[kSortWaves];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t base = int64_t(blockIdx.x) * kSortChunk + wave * kEach;
  int mine[kTurns];
#pragma unroll
  for (int k = 0; k < kTurns; ++k) mine[k] = local_expert(p, base + k * 64 + lane);
  for (int i = tid; i < p.n_experts; i += kSortThreads) {
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) next[w][i] = 0;
    start[i] = before[i] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kTurns; ++k)
    if (mine[k] >= 0) atomicAdd(&next[wave][mine[k]], 1);
  if (FORM == kSortTotals) {
    __syncthreads();
    for (int i = tid; i < p.n_experts; i += kSortThreads) {
      int own = 0;
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) own += next[w][i];
      start[i] = p.hist[int64_t(p.chunks - 1) * p.n_experts + i];
      before[i] = p.hist[int64_t(blockIdx.x) * p.n_experts + i] - own;
    }
  }
  if (FORM == kSortCounts) {
    // All slots of an expert, and those of the chunks before this one: the
    // threads share out the chunks, sixteen loads under way in each.
    const int lanes = kSortThreads / p.n_experts > 0 ? kSortThreads / p.n_experts : 1;  // threads an expert
    for (int i = tid; i < p.n_experts * lanes; i += kSortThreads) {
      const int e = i % p.n_experts, part = i / p.n_experts;
      int total = 0, below = 0;
      for (int c0 = part; c0 < p.chunks; c0 += lanes * 16) {
        int h[16];
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          const int c = c0 + u * lanes;
          h[u] = c < p.chunks ? p.hist[int64_t(c) * p.n_experts + e] : 0;
        }
#pragma unroll
        for (int u = 0; u < 16; ++u) {
          total += h[u];
          below += c0 + u * lanes < int(blockIdx.x) ? h[u] : 0;
        }
      }
      atomicAdd(&start[e], total);
      atomicAdd(&before[e], below);
    }
  }
  __syncthreads();
  // Exclusive scan of the totals, two experts a thread.
  int a = 0, b = 0;
  if (2 * tid < p.n_experts) {
    if (ONE) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) a += next[w][2 * tid];
    } else {
      a = start[2 * tid];
    }
  }
  if (2 * tid + 1 < p.n_experts) {
    if (ONE) {
#pragma unroll
      for (int w = 0; w < kSortWaves; ++w) b += next[w][2 * tid + 1];
    } else {
      b = start[2 * tid + 1];
    }
  }
  int sum = a + b;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(sum, d, 64);
    if (lane >= d) sum += o;
  }
  if (lane == 63) wave_sum[wave] = sum;
  __syncthreads();
  int ahead = 0, rows = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) {
    ahead += w < wave ? wave_sum[w] : 0;
    rows += wave_sum[w];
  }
  const int begin = ahead + sum - a - b;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = 2 * tid + i;
    if (e >= p.n_experts) continue;
    const int from = i ? begin + a : begin;
    if (blockIdx.x == 0) p.offsets[e] = from;
    // from counts to the waves' own beginnings
    int at = from + before[e];
#pragma unroll
    for (int w = 0; w < kSortWaves; ++w) {
      const int n = next[w][e];
      next[w][e] = at;
      at += n;
    }
  }
  if (blockIdx.x == 0 && tid == 0) p.offsets[p.n_experts] = rows;
  __syncthreads();
  const int bits = 32 - __clz(p.n_experts);  // an expert number's
#pragma unroll
  for (int k = 0; k < kTurns; ++k) {
    const int64_t i = base + k * 64 + lane;
    if (i - lane >= p.n_slots) break;
    const int e = mine[k];
    uint64_t same = __ballot(e >= 0);  // lanes with this lane's expert
    for (int bit = 0; bit < bits; ++bit) {
      const uint64_t on = __ballot((e >> bit) & 1);
      same &= (e >> bit) & 1 ? on : ~on;
    }
    int row = -1;
    if (e >= 0) {
      row = next[wave][e] + __popcll(same & ((uint64_t(1) << lane) - 1));
      p.tokens[row] = int32_t(uint32_t(i) / uint32_t(p.top_k));
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (e >= 0 && !(same >> lane >> 1)) next[wave][e] = row + 1;  // the last of its expert
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (i < p.n_slots) {
      p.positions[i] = row;
      if (i >= rows) p.tokens[i] = -1;  // entries behind the last row
    }
  }
}

__global__ void rs_sort_empty_kernel(int32_t* offsets, int n) {
  for (int e = threadIdx.x; e < n; e += blockDim.x) offsets[e] = 0;
}

// --------------------------------------------------------------------------
// Combination of the experts' rows.
// --------------------------------------------------------------------------

struct CombineArgs {
  const void* y;
  const int32_t* positions;
  const float* weights;
  void* out;
  int64_t n_tokens, hidden, n_rows, y_stride, out_stride;
  int32_t top_k;
};

constexpr int kSlots = 8;  // slots whose loads are under way together

// 2048 columns of a token per workgroup, eight a lane (8192 tokens of 7168
// columns: 189 us; 194 with 4096 columns a workgroup, 197 with 512).  A
// token's positions are the same for the whole workgroup, so a slot without a
// row costs no load.
template <int YT, int OT>
__global__ __launch_bounds__(256) void rs_combine_kernel(CombineArgs p) {
  const int64_t t = blockIdx.x;
  for (int64_t c = (int64_t(blockIdx.y) * blockDim.x + threadIdx.x) * 8; c < p.hidden; c += int64_t(blockDim.x) * gridDim.y * 8) {
    const int n = int(min(int64_t(8), p.hidden - c));
    float acc[8] = {};
    for (int j0 = 0; j0 < p.top_k; j0 += kSlots) {
      Raw8<YT> v[kSlots];
      float w[kSlots];
      bool on[kSlots];
#pragma unroll
      for (int j = 0; j < kSlots; ++j) {
        const int64_t at = t * p.top_k + j0 + j;
        const int64_t r = j0 + j < p.top_k ? p.positions[at] : -1;
        on[j] = r >= 0 && r < p.n_rows;
        w[j] = on[j] && p.weights ? p.weights[at] : 1.0f;
        if (on[j]) v[j].load(p.y, r * p.y_stride + c, n);
      }
#pragma unroll
      for (int j = 0; j < kSlots; ++j)
        if (on[j]) {
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] += w[j] * v[j].get(i);
        }
    }
    store8(p.out, OT, t * p.out_stride + c, n, acc);
  }
}

struct CombineGradArgs {
  const void* dout;
  const void* y;
  const int32_t* positions;
  const float* weights;
  void* dy;
  float* dweights;
  int64_t n_tokens, hidden, n_rows, y_stride, out_stride;
  int32_t top_k;
};

// A wave per slot, four of its 512-column pieces under way at a time.  The
// slots of a token are neighbours, so dout's row comes from memory once and
// from the caches after that; a slot without a row costs next to nothing.
// (A workgroup per token with dout in registers took 158 us where this takes
// less: fewer waves fit, and they wait for each other.)
constexpr int kPieces = 4;

template <int YT, int OT>
__global__ __launch_bounds__(256) void rs_combine_grad_kernel(CombineGradArgs p) {
  const int lane = threadIdx.x & 63;
  const int64_t slot = int64_t(blockIdx.x) * 4 + __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  if (slot >= p.n_tokens * p.top_k) return;
  const int64_t r = p.positions[slot];
  if (r < 0 || r >= p.n_rows) {
    if (p.dweights && lane == 0) p.dweights[slot] = 0.0f;
    return;
  }
  const int64_t from = slot / p.top_k * p.out_stride, row = r * p.y_stride;
  const float w = p.weights ? p.weights[slot] : 1.0f;
  float dot = 0.0f;
  for (int64_t c0 = lane * 8; c0 < p.hidden; c0 += 512 * kPieces) {
    Raw8<OT> d[kPieces];
    Raw8<YT> v[kPieces];
    int n[kPieces];
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      const int64_t c = c0 + u * 512;
      n[u] = int(max(int64_t(0), min(int64_t(8), p.hidden - c)));
      if (n[u] == 0) continue;
      d[u].template load<false>(p.dout, from + c, n[u]);
      if (p.dweights) v[u].load(p.y, row + c, n[u]);
    }
#pragma unroll
    for (int u = 0; u < kPieces; ++u) {
      if (n[u] == 0) continue;
      if (p.dweights) {
#pragma unroll
        for (int i = 0; i < 8; ++i) dot += d[u].get(i) * v[u].get(i);
      }
      if (p.dy) {
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i] = w * d[u].get(i);
        store8(p.dy, YT, row + c0 + u * 512, n[u], o);
      }
    }
  }
  if (p.dweights) {
#pragma unroll
    for (int s = 32; s; s >>= 1) dot += __shfl_xor(dot, s, 64);
    if (lane == 0) p.dweights[slot] = dot;
  }
}

}  // namespace

// The lanes that one of n_groups groups takes, as a power of two.
constexpr int route_lanes_shift(int n_groups) {
  int shift = 4;
  for (int slots = 1; slots < n_groups; slots <<= 1) --shift;
  return shift;
}
// The most experts that a lane can hold: 113, of 1,017 in nine groups.  (Runs
// above 64, which take large groups whose number is no power of two, keep part
// of their values in scratch memory: 65,536 tokens of 1,000 experts in ten
// groups 650 us, of 1,024 in eight 153.)
constexpr int longest_run() {
  int most = 0;
  for (int g = 1; g <= kMaxRouteGroups; ++g) {
    const int size = kMaxExperts / g, run = (size + (1 << route_lanes_shift(g)) - 1) >> route_lanes_shift(g);
    if (run > most) most = run;
  }
  return most;
}
static_assert(longest_run() <= 128, "a kernel for every router");

hipError_t launch_route(const rs_router& r, int64_t n_tokens, const void* logits, int64_t stride,
                        const float* bias, const uint8_t* mask, int32_t* ids, float* weights,
                        hipStream_t stream) {
  RouteArgs p{logits, bias, mask, ids, weights, n_tokens, stride, r.n_experts, r.top_k, r.n_groups,
              r.top_groups, r.group_top, r.renormalise, r.score == RS_SCORE_SIGMOID, r.logits_dtype,
              r.n_experts / r.n_groups, route_lanes_shift(r.n_groups), 0, 0, r.scale};
  p.run = (p.group_size + (1 << p.lanes_shift) - 1) >> p.lanes_shift;
  p.by_logit = !bias && (r.n_groups == 1 || r.group_top == 1 || p.group_size == 1);
  const dim3 grid(uint32_t((n_tokens + 15) / 16));
  if (p.run <= 4) rs_route_kernel<4><<<grid, 256, 0, stream>>>(p);
  else if (p.run <= 8) rs_route_kernel<8><<<grid, 256, 0, stream>>>(p);
  else if (p.run <= 16) rs_route_kernel<16><<<grid, 256, 0, stream>>>(p);
  else if (p.run <= 32) rs_route_kernel<32><<<grid, 256, 0, stream>>>(p);
  else if (p.run <= 64) rs_route_kernel<64><<<grid, 256, 0, stream>>>(p);
  else rs_route_kernel<128><<<grid, 256, 0, stream>>>(p);
  return hipGetLastError();
}

template <int RUN>
void route_grad(const RouteGradArgs& p, hipStream_t stream) {
  constexpr int kTokens = RUN > 16 ? 4 : 16;
  rs_route_grad_kernel<RUN><<<dim3(uint32_t((p.n_tokens + kTokens - 1) / kTokens)), kTokens * 16, 0, stream>>>(p);
}

hipError_t launch_route_grad(const rs_router& r, int64_t n_tokens, const void* logits, int64_t stride,
                             const int32_t* ids, const float* dweights, void* dlogits, int64_t dstride,
                             hipStream_t stream) {
  RouteGradArgs p{logits, ids, dweights, dlogits, n_tokens, stride, dstride, r.n_experts, r.top_k,
                  r.renormalise, r.score == RS_SCORE_SIGMOID, r.logits_dtype, (r.n_experts + 15) / 16, r.scale};
  if (p.run <= 4) route_grad<4>(p, stream);
  else if (p.run <= 8) route_grad<8>(p, stream);
  else if (p.run <= 16) route_grad<16>(p, stream);
  else if (p.run <= 32) route_grad<32>(p, stream);
  else route_grad<64>(p, stream);
  return hipGetLastError();
}

hipError_t launch_sort(const int32_t* ids, int64_t n_slots, int32_t top_k, int32_t first, int32_t n_experts,
                       int32_t* offsets, int32_t* tokens, int32_t* positions, int32_t* workspace,
                       hipStream_t stream) {
  if (n_slots == 0) {
    rs_sort_empty_kernel<<<1, 256, 0, stream>>>(offsets, n_experts + 1);
    return hipGetLastError();
  }
  const int32_t chunks = int32_t((n_slots + kSortChunk - 1) / kSortChunk);
  const SortArgs p{ids, offsets, tokens, positions, workspace, n_slots, top_k, first, n_experts, chunks};
  if (chunks == 1) {
    rs_sort_place_kernel<kSortOne><<<1, kSortThreads, 0, stream>>>(p);
    return hipGetLastError();
  }
  rs_sort_count_kernel<<<chunks, kSortThreads, 0, stream>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  // Counts that every workgroup reads whole cost less than a third launch while
  // they are few (us, counts against running totals): 32,768 tokens x 8 over 256
  // experts 13.3 and 14.5, 49,152 15.6 and 15.1, 131,072 33 and 19, 1,048,576
  // 959 and 85; over 64 experts 65,536 x 8 11.8 and 14.5, 131,072 x 8 16.9 and 16.6.
  if (chunks < 512 && int64_t(chunks) * n_experts <= 40000) {
    rs_sort_place_kernel<kSortCounts><<<chunks, kSortThreads, 0, stream>>>(p);
    return hipGetLastError();
  }
  rs_sort_total_kernel<<<(n_experts + 15) / 16, 1024, 0, stream>>>(p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  rs_sort_place_kernel<kSortTotals><<<chunks, kSortThreads, 0, stream>>>(p);
  return hipGetLastError();
}

// One kernel per pair of types.
#define RS_BY_TYPES(kernel, grid, threads, args)                                                              \
  do {                                                                                                        \
    const int pair = c.y_dtype << 8 | c.out_dtype;                                                            \
    if (pair == (RS_BF16 << 8 | RS_BF16)) kernel<RS_BF16, RS_BF16><<<grid, threads, 0, stream>>>(args);       \
    else if (pair == (RS_BF16 << 8 | RS_F16)) kernel<RS_BF16, RS_F16><<<grid, threads, 0, stream>>>(args);    \
    else if (pair == (RS_BF16 << 8 | RS_F32)) kernel<RS_BF16, RS_F32><<<grid, threads, 0, stream>>>(args);    \
    else if (pair == (RS_F16 << 8 | RS_BF16)) kernel<RS_F16, RS_BF16><<<grid, threads, 0, stream>>>(args);    \
    else if (pair == (RS_F16 << 8 | RS_F16)) kernel<RS_F16, RS_F16><<<grid, threads, 0, stream>>>(args);      \
    else if (pair == (RS_F16 << 8 | RS_F32)) kernel<RS_F16, RS_F32><<<grid, threads, 0, stream>>>(args);      \
    else if (pair == (RS_F32 << 8 | RS_BF16)) kernel<RS_F32, RS_BF16><<<grid, threads, 0, stream>>>(args);    \
    else if (pair == (RS_F32 << 8 | RS_F16)) kernel<RS_F32, RS_F16><<<grid, threads, 0, stream>>>(args);      \
    else kernel<RS_F32, RS_F32><<<grid, threads, 0, stream>>>(args);                                          \
  } while (0)

hipError_t launch_combine(const rs_moe_combine& c, const void* y, const int32_t* positions,
                          const float* weights, void* out, hipStream_t stream) {
  const CombineArgs p{y, positions, weights, out, c.n_tokens, c.hidden, c.n_rows, c.y_stride, c.out_stride, c.top_k};
  const int64_t lanes = (c.hidden + 7) / 8, parts = (lanes + 255) / 256;
  const uint32_t threads = lanes >= 256 ? 256 : uint32_t((lanes + 63) / 64 * 64);
  const dim3 grid(uint32_t(c.n_tokens), uint32_t(parts < 65535 ? parts : 65535));
  RS_BY_TYPES(rs_combine_kernel, grid, threads, p);
  return hipGetLastError();
}

hipError_t launch_combine_grad(const rs_moe_combine& c, const void* dout, const void* y,
                               const int32_t* positions, const float* weights, void* dy, float* dweights,
                               hipStream_t stream) {
  const CombineGradArgs p{dout, y, positions, weights, dy, dweights, c.n_tokens, c.hidden, c.n_rows, c.y_stride,
                          c.out_stride, c.top_k};
  const dim3 grid(uint32_t((c.n_tokens * c.top_k + 3) / 4));
  RS_BY_TYPES(rs_combine_grad_kernel, grid, 256, p);
  return hipGetLastError();
}
#undef RS_BY_TYPES

}  // namespace rs
