// The router by scores: experts chosen by score plus bias, from the best
// groups of experts, weighted by the scores alone.
//
//   s_i    = 1 / (1 + exp(-l_i)), or the softmax of the open logits
//   r_i    = s_i + bias_i, or without a bias l_i (which orders alike)
//   v_g    = the largest r of a group, or the sum of its two largest (without
//            a bias of the scores' two largest)
//   ids    = the k largest r of the groups with the largest v; ties to the
//            lowest group, then the lowest expert
//   w_j    = scale * s, divided by the chosen scores' sum when renormalised
//
// The choice is that of r and v computed in 64 bits.  They are computed in 32
// first, with bounds on the error: where two neighbours of the order that
// matter (the chosen ones and the next ones; the last group kept and the first
// left out) lie closer than the bounds, and are not the same logit and bias,
// these alone are computed in 64 bits, an expert to a lane: by the bounds, for
// 8 of 256 by sigmoid with ranks some 2^-8 apart, in a few tokens in a
// thousand.  64-bit exponentials for all 16.8 million scores would take about a
// millisecond.  A softmax's sum stays the one in 32 bits there, as a common
// factor of the scores it decides few orders; where it may, and where more
// experts are close than a token's lanes list, the whole token is computed in
// 64 bits.
//
// As in moe_route.cu a group of L lanes takes a token.  A group of experts has
// lanes of its own (a power of two), so that its two largest are found in the
// sorted lists' heads and exchanges among these lanes; places of the lanes
// past a group's experts stay empty.  Chunks, bits and places are shared
// with moe_route.cu.
// The compares and selects bound it (issue slots 75% busy, some 900
// instructions a token of 256 experts): 65536 tokens, 8 of 256 in 4 of 8
// groups, 80 us for the choices, where the logits' 67 MB take 10.
#include <mutex>
#include <type_traits>

#include "route.cuh"

namespace bra {
namespace {

using namespace route;

constexpr uint32_t kAll = 0xffffffffu;

struct ScoreParams {
  RouteParams r;
  const float* bias;   // [E], or nullptr
  float scale;
  int sigmoid;
  int groups, top_groups, best;   // groups 1: no restriction
  int size;            // experts of a group
  int lanes;           // lanes of a group, a power of two
  int per;             // experts of a lane, a multiple of four, at most V
  int bias_vec;        // bias is read four at a time
};

// The two largest of (a1 >= a2) and (b1 >= b2).
template <typename F>
__device__ __forceinline__ void best_two(F& a1, F& a2, F b1, F b2) {
  const F low = a1 < b1 ? a1 : b1, next = a2 > b2 ? a2 : b2;
  a1 = a1 < b1 ? b1 : a1;
  a2 = low > next ? low : next;
}

// A sigmoid for the choice, of four instructions: within 2^-21.8 (the two
// approximations' units of 2^-23, the exponent's rounding times s (1 - s) |l|,
// and the sum's).
__device__ __forceinline__ float score_of(float l) {
  float e, s;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(l * -1.44269504f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}

// Where a lane's experts are.
struct Place {
  uint32_t group;      // this token's lanes
  int gl, g, first, own;
  template <int L>
  __device__ __forceinline__ static Place of(const ScoreParams& p, int lane) {
    Place a;
    a.group = L == 32 ? kAll : ((1u << (L & 31)) - 1u) << (lane & ~(L - 1));
    a.gl = lane % L;
    a.g = a.gl / p.lanes;
    const int off = (a.gl - a.g * p.lanes) * p.per;
    a.first = a.g * p.size + off;
    a.own = a.g < p.groups ? max(0, min(p.per, p.size - off)) : 0;
    return a;
  }
};

// The paths below run for few tokens, and mostly on an SM that has not run them:
// loops stay loops and the 64-bit functions are there once, as fetching the
// instructions takes most of their time (1518 tokens, 9 of 22, one of them
// settled: 16 us with unrolled loops, 8 without the token).

// A score in 64 bits; of a softmax with the largest logit m.
__device__ __noinline__ double score64(float l, float m, double sum, int sigmoid) {
  const double e = exp(sigmoid ? -(double)l : (double)l - (double)m);
  return (sigmoid ? 1.0 : e) / (sigmoid ? 1.0 + e : sum);
}
// Whether a softmax's sum that is off by up to 2^-18 leaves the order of two
// ranks as it is: x and y with the scores sx and sy in them.
__device__ __forceinline__ bool apart(double x, double sx, double y, double sy) {
  return (x == y && sx == sy) || fabs(x - y) > 0x1p-17 * fabs(sx - sy) + 0x1p-48 * fabs(x);
}

// The choice in 64 bits: the ids of one token, by the lanes of `at.group`.
// open: whether its groups are chosen again too; else those of lanes with
// `kept` are, and experts whose rank in 32 bits lies below `floor` are out.
template <typename T, int L, int V>
__device__ __noinline__ void choose_exact(const ScoreParams& p, int t, int lane, bool open, bool kept,
                                          float floor) {
  const Place at = Place::of<L>(p, lane);
  const T* row = static_cast<const T*>(p.r.logits) + (int64_t)t * p.r.E + at.first;
  const double inf = INFINITY;
  float m = -INFINITY;
  double sum = p.sigmoid ? 1.0 : 0.0;
  if (!p.sigmoid) {
#pragma unroll 1
    for (int i = 0; i < at.own; ++i) m = fmaxf(m, logit(row + i));         // NaN is passed over
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(at.group, m, d));
#pragma unroll 1
    for (int i = 0; i < at.own; ++i) {
      const float v = logit(row + i);
      if (v >= -kLargest) sum += score64(v, m, 1.0, 0);
    }
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) sum += __shfl_xor_sync(at.group, sum, d);
  }
  double r[V], f1 = -inf, f2 = -inf;
  const float inv = (float)(1.0 / sum);
  uint32_t live = 0u;
#pragma unroll 1
  for (int i = 0; i < V; ++i) {
    r[i] = -inf;
    const float v = i < at.own ? logit(row + i) : -INFINITY;
    if (!(v >= -kLargest) || !(open || kept)) continue;
    float x = v;
    if (p.bias) x = (p.sigmoid ? score_of(v) : expf(v - m) * inv) + p.bias[at.first + i];
    if (open || !(x < floor)) live |= 1u << i;
  }
  // each lane's next one, so that the slow 64-bit functions run as few times as can be
  while (__any_sync(at.group, live != 0u)) {
    if (live == 0u) continue;
    const int i = __ffs(live) - 1;
    live &= live - 1u;
    const float v = logit(row + i);
    const double s = score64(v, m, sum, p.sigmoid);
    double x = p.bias ? s + (double)p.bias[at.first + i] : (double)v;
    if (!(x > -inf)) x = -inf;
    r[i] = x < 1e300 ? x : 1e300;
    best_two(f1, f2, p.bias || p.best == 1 ? r[i] : s, -inf);
  }
  if (open) {
    for (int d = 1; d < p.lanes; d <<= 1) {
      const double b1 = __shfl_xor_sync(at.group, f1, d), b2 = __shfl_xor_sync(at.group, f2, d);
      best_two(f1, f2, b1, b2);
    }
    const double v = p.best == 2 && f2 > -inf ? f1 + f2 : f1;
    int better = 0;
    for (int g = 0; g < p.groups; ++g) {
      const double o = __shfl_sync(at.group, v, g * p.lanes, L);
      better += o > v || (o == v && g < at.g) ? 1 : 0;
    }
    if (better >= p.top_groups)
#pragma unroll 1
      for (int i = 0; i < V; ++i) r[i] = -inf;
  }
  for (int j = 0; j < p.r.k; ++j) {
    double most = -inf;
    int mine = 0;
#pragma unroll 1
    for (int i = 0; i < V; ++i)
      if (r[i] > most) most = r[i], mine = i;
    double top = most;
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) {
      const double o = __shfl_xor_sync(at.group, top, d);
      top = o > top ? o : top;
    }
    const int win = __ffs(__ballot_sync(at.group, most == top)) - 1;
    const int id = __shfl_sync(at.group, at.first + mine, win);
    if (lane == win) r[mine] = -inf;
    if (at.gl == j % L) p.r.ids[(int64_t)t * p.r.k + j] = top > -inf ? id : -1;
  }
}

// The best experts of a token in the order of their 32-bit ranks, at least all
// that can be among the k chosen: the o-th of lane gl is number o * L + gl.
template <int KEEP>
struct Listed {
  int id[KEEP];        // -1: none
  uint32_t close;      // bit o: the neighbours' ranks are too close to tell
};

// The choice from a list, by the lanes of a token: ranks that are too close are
// computed in 64 bits, and their experts' places are those of their ranks among
// them; the other places stand.  A softmax's sum is the one in 32 bits; false:
// it decides an order.
template <typename T, int L, int KEEP>
__device__ __noinline__ bool settle(const ScoreParams& p, int t, int lane, Listed<KEEP> of, float m,
                                    float sum) {
  const uint32_t group = L == 32 ? kAll : ((1u << (L & 31)) - 1u) << (lane & ~(L - 1));
  const int gl = lane % L;
  const T* row = static_cast<const T*>(p.r.logits) + (int64_t)t * p.r.E;
  double r[KEEP], score[KEEP];
  int place[KEEP];
#pragma unroll 1
  for (int o = 0; o < KEEP; ++o) {
    place[o] = o * L + gl;
    r[o] = score[o] = 0.0;
    if (of.close >> o & 1u) {
      const float l = logit(row + of.id[o]);
      if (p.bias) score[o] = score64(l, m, sum, p.sigmoid);
      const double x = p.bias ? score[o] + (double)p.bias[of.id[o]] : (double)l;
      r[o] = x < 1e300 ? x : 1e300;
    }
  }
  bool sure = true;
#pragma unroll 1
  for (int from = 0; from < KEEP; ++from) {
    uint32_t left = __ballot_sync(group, of.close >> from & 1u) & group;
#pragma unroll 1
    while (left) {
      const int src = __ffs(left) - 1, at = from * L + src % L;
      left &= left - 1u;
      const double x = __shfl_sync(group, r[from], src), sx = __shfl_sync(group, score[from], src);
      const int id = __shfl_sync(group, of.id[from], src);
#pragma unroll 1
      for (int o = 0; o < KEEP; ++o)
        if (of.close >> o & 1u) {
          place[o] += (x > r[o] || (x == r[o] && id < of.id[o]) ? 1 : 0) - (at < o * L + gl ? 1 : 0);
          sure = sure && (!p.bias || p.sigmoid || apart(x, sx, r[o], score[o]));
        }
    }
  }
  if (__any_sync(group, !sure)) return false;
#pragma unroll 1
  for (int o = 0; o < KEEP; ++o)
    if (place[o] < p.r.k) p.r.ids[(int64_t)t * p.r.k + place[o]] = of.id[o];
  return true;
}

// How many groups of experts of a token come before this lane's, by the lanes
// of the token: the values of groups with `near` in 64 bits, from their experts
// whose ranks in 32 bits are `floor` or more; the other values are v.  -1: a
// softmax's sum in 32 bits decides an order.
template <typename T, int L, int V>
__device__ __noinline__ int settle_groups(const ScoreParams& p, int t, int lane, float v, bool near,
                                          float floor, float m, float sum) {
  const Place at = Place::of<L>(p, lane);
  const T* row = static_cast<const T*>(p.r.logits) + (int64_t)t * p.r.E + at.first;
  const double inf = INFINITY;
  const float inv = 1.f / sum;
  double f1 = -inf, f2 = -inf, s1 = 0.0, s2 = 0.0;
  auto put = [&](double x, double s) {          // among the two largest
    if (x > f1) {
      f2 = f1, s2 = s1;
      f1 = x, s1 = s;
    } else if (x > f2) {
      f2 = x, s2 = s;
    }
  };
#pragma unroll 1
  for (int i = 0; i < at.own && near; ++i) {
    const float l = logit(row + i), b = p.bias ? p.bias[at.first + i] : 0.f;
    float x = l;
    if (p.bias) x = (p.sigmoid ? score_of(l) : expf(l - m) * inv) + fminf(b, kLargest);
    if (!(l >= -kLargest) || !(b >= -kLargest) || x < floor) continue;
    const double s = p.bias || p.best == 2 ? score64(l, m, sum, p.sigmoid) : (double)l;
    const double r = p.bias ? s + (double)b : s;
    put(r < 1e300 ? r : 1e300, s);
  }
#pragma unroll 1
  for (int d = 1; d < p.lanes; d <<= 1) {
    const double a1 = __shfl_xor_sync(at.group, f1, d), b1 = __shfl_xor_sync(at.group, s1, d);
    const double a2 = __shfl_xor_sync(at.group, f2, d), b2 = __shfl_xor_sync(at.group, s2, d);
    put(a1, b1);
    put(a2, b2);
  }
  const bool two = p.best == 2 && f2 > -inf;
  const double value = near ? two ? f1 + f2 : f1 : (double)v, of = two ? s1 + s2 : s1;
  int better = 0;
  bool sure = true;
#pragma unroll 1
  for (int g = 0; g < p.groups; ++g) {
    const double x = __shfl_sync(at.group, value, g * p.lanes, L);
    const double sx = __shfl_sync(at.group, of, g * p.lanes, L);
    const bool too = __shfl_sync(at.group, (int)near, g * p.lanes, L) != 0;
    better += x > value || (x == value && g < at.g) ? 1 : 0;
    if (p.bias && !p.sigmoid && near && too) sure = sure && apart(x, sx, value, of);
  }
  return __any_sync(at.group, !sure) ? -1 : better;
}

// The experts of one token to each group of L lanes (t < 0: none): as choose
// of moe_route.cu.  Whole warps.
template <typename T, int L, int V>
__device__ __forceinline__ void choose_scored(const ScoreParams& p, const Place& at, int t, int lane,
                                              const float* bias, uint32_t* bits, int stride, int word,
                                              uint32_t bit) {
  constexpr int OWN = (BRA_MAX_CHOICES + L - 1) / L;   // choices a lane keeps
  constexpr int NL = V / 8;
  const T* row = static_cast<const T*>(p.r.logits) + (int64_t)t * p.r.E;
  // Groups before this lane's where 64 bits had to tell (-1: they did not,
  // -2: not asked).  The choice then begins anew, so that nothing is kept in
  // registers over that call.
  int before = -2;
begin:
  float l[V];
#pragma unroll
  for (int i = 0; i < V; i += 4) {
    T raw[4];
    if (t >= 0 && p.r.vec && i + 4 <= at.own) {
      if constexpr (sizeof(T) == 4)
        *reinterpret_cast<uint4*>(raw) = *reinterpret_cast<const uint4*>(row + at.first + i);
      else
        *reinterpret_cast<uint2*>(raw) = *reinterpret_cast<const uint2*>(row + at.first + i);
    } else {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        raw[c] = t >= 0 && i + c < at.own ? row[at.first + i + c] : T(-INFINITY);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) l[i + c] = logit(&raw[c]);
  }
  const bool limited = p.top_groups < p.groups, ranked = p.bias != nullptr;
  // softmax: the largest logit and the sum, where scores are needed
  float m = 0.f, sum = 1.f;
  if (!p.sigmoid && (ranked || !p.r.renorm || (limited && p.best == 2))) {
    m = -INFINITY;
#pragma unroll
    for (int i = 0; i < V; ++i) m = fmaxf(m, l[i]);
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, d));
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i)
      if (l[i] >= -kLargest) sum += expf(l[i] - m);
    sum = group_sum(sum, L);
  }
  const float inv = p.sigmoid ? 1.f : 1.f / sum;          // the largest score there can be
  auto score = [&](float v) { return p.sigmoid ? score_of(v) : expf(v - m) * inv; };
  // The least distance at which 32 bits decide: two scores' errors (softmax:
  // also the sum's, one unit of 2^-24 a term of a lane and level), two sums'
  // roundings, two keys' low bits.
  const float slack = ranked ? (p.sigmoid ? 0x1p-20f : 0x1p-18f) * inv : 0.f;
  constexpr float part = 0x1p-22f + V * 0x1p-23f;
  auto distance = [&](float a, float b) { return slack + fmaxf(fabsf(a), fabsf(b)) * part; };
  // 16-bit logits leave their keys' low bits free
  const bool exact = !ranked && sizeof(T) == 2;

  float rank[V];
#pragma unroll
  for (int i = 0; i < V; ++i) rank[i] = l[i];
  if (ranked && p.sigmoid) {
#pragma unroll
    for (int i = 0; i < V; ++i) rank[i] = score_of(l[i]) + bias[i];
  } else if (ranked) {
#pragma unroll
    for (int i = 0; i < V; ++i) rank[i] = expf(l[i] - m) * inv + bias[i];
  }
  // Keys, one word each: the rank, its low bits the place in the lane, the
  // first the largest; lists of eight, sorted (Batcher's odd-even merge sort).
  uint32_t key[NL][8];
#pragma unroll
  for (int n = 0; n < NL; ++n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = rank[n * 8 + i];
      const bool open = l[n * 8 + i] >= -kLargest;
      const uint32_t u = __float_as_uint(x);
      const uint32_t k = u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
      key[n][i] = open && x >= -kLargest ? (k & ~(uint32_t)(V - 1)) | (uint32_t)(V - 1 - n * 8 - i) : 0u;
    }
    auto put = [&](int a, int b) {
      const uint32_t hi = max(key[n][a], key[n][b]), lo = min(key[n][a], key[n][b]);
      key[n][a] = hi, key[n][b] = lo;
    };
    put(0, 1), put(2, 3), put(4, 5), put(6, 7);
    put(0, 2), put(1, 3), put(4, 6), put(5, 7);
    put(1, 2), put(5, 6);
    put(0, 4), put(1, 5), put(2, 6), put(3, 7);
    put(2, 4), put(3, 5);
    put(1, 2), put(3, 4), put(5, 6);
  }
  // what a key says of its rank: at most V - 1 units of it off
  auto rank_of = [&](uint32_t k) { return value_of(k & ~(uint32_t)(V - 1)); };

  bool open = false, kept = true;                // open: 32 bits do not decide the groups
  if (limited) {
    uint32_t k1 = key[0][0], k2 = key[0][1];
#pragma unroll
    for (int n = 1; n < NL; ++n) best_two(k1, k2, key[n][0], key[n][1]);
    for (int d = 1; d < p.lanes; d <<= 1) {
      const uint32_t b1 = __shfl_xor_sync(kAll, k1, d), b2 = __shfl_xor_sync(kAll, k2, d);
      best_two(k1, k2, b1, b2);
    }
    float v = k1 ? rank_of(k1) : -INFINITY;
    if (p.best == 2 && k1) {
      float w = k2 ? rank_of(k2) : 0.f;
      if (!ranked) {
        v = score(v);
        if (k2) w = score(w);
      }
      v = fmaxf(fminf(v + w, kLargest), -kLargest);
    }
    int better = 0;
    for (int g = 0; g < p.groups; ++g) {
      const float o = __shfl_sync(kAll, v, g * p.lanes, L);
      better += o > v || (o == v && g < at.g) ? 1 : 0;
    }
    if (!exact || p.best == 2) {
      // the last group kept and the first left out; a score from a logit whose
      // low bits are gone errs by |l| s (1 - s) V units more (sigmoid: at most
      // V / 4), or by |l| s V (softmax: (|m| + 0.4) V at most)
      const bool head = at.g < p.groups && at.gl == at.g * p.lanes;
      const uint32_t in = __ballot_sync(kAll, head && better == p.top_groups - 1) & at.group;
      const uint32_t out = __ballot_sync(kAll, head && better == p.top_groups) & at.group;
      const float vi = __shfl_sync(kAll, v, __ffs(in) - 1), vo = __shfl_sync(kAll, v, __ffs(out) - 1);
      float off = slack;
      if (!ranked && p.best == 2)
        off = (p.sigmoid ? 0x1p-20f + V * 0x1p-23f
                         : 0x1p-18f + V * 0x1p-23f * (exact ? 1.f : 1.f + fabsf(m))) * inv;
      auto tight = [&](float a, float b) {
        return fabsf(a - b) <= 2.f * (off + fmaxf(fabsf(a), fabsf(b)) * part);
      };
      open = before == -2 && vo > -INFINITY && tight(vi, vo);
      if (__any_sync(kAll, open)) {
        if (open) {                              // the same for all lanes of a token
          const uint32_t least = p.best == 2 ? k2 : k1;
          const float x = least ? rank_of(least) : -INFINITY;
          const bool near =
              v > -INFINITY && (v <= vi || tight(v, vi)) && (v >= vo || tight(v, vo));
          before = settle_groups<T, L, V>(p, t, lane, v, near, x - 2.f * distance(x, x), m, sum);
        } else {
          before = better;
        }
        __syncwarp();
        goto begin;
      }
      if (before >= 0) better = before;
      open = before == -1;
    }
    kept = better < p.top_groups;
    if (!kept) {
#pragma unroll
      for (int n = 0; n < NL; ++n)
#pragma unroll
        for (int i = 0; i < 8; ++i) key[n][i] = 0u;
    }
  }
  // Takes the largest of the lanes' heads from the lists of the tokens with
  // `on`: its key, and the lane that had it.  Whole warps.
  auto take = [&](bool on, int* lane_of) {
    uint32_t head = key[0][0];
#pragma unroll
    for (int n = 1; n < NL; ++n) head = max(head, key[n][0]);
    // without the places: equal ranks go to the lowest lane
    const uint32_t part_of = head & ~(uint32_t)(V - 1);
    uint32_t most = part_of;
    if constexpr (L == 32) {
      most = __reduce_max_sync(kAll, part_of);
    } else {
#pragma unroll
      for (int d = L / 2; d > 0; d >>= 1) most = max(most, __shfl_xor_sync(kAll, most, d));
    }
    const int win = __ffs(__ballot_sync(kAll, part_of == most) & at.group) - 1;
    // the winner drops its head (with most = 0 there is nothing to drop)
#pragma unroll
    for (int n = 0; n < NL; ++n) {
      const bool drop = on && lane == win && key[n][0] == head;
#pragma unroll
      for (int i = 0; i + 1 < 8; ++i) key[n][i] = drop ? key[n][i + 1] : key[n][i];
      key[n][7] = drop ? 0u : key[n][7];
    }
    *lane_of = win;
    return __shfl_sync(kAll, head, win);
  };
  // Whether two experts' order is open in 32 bits: too close, unless equal
  // logits and equal biases make them a tie in any precision.
  auto too_close = [&](uint32_t ka, uint32_t kb) {
    const float hi = rank_of(ka), lo = rank_of(kb);
    return ka && kb && hi - lo <= distance(hi, lo);
  };
  auto same = [&](int a, int b) {
    return logit(row + a) == logit(row + b) && (!ranked || p.bias[a] == p.bias[b]);
  };

  // the largest of the lanes' heads, k times, and the best one left out
  constexpr int KEEP = (BRA_MAX_CHOICES + L) / L;        // of k + 1
  uint32_t my_key[KEEP];
  int my_lane[KEEP];
#pragma unroll
  for (int o = 0; o < KEEP; ++o) {
    my_key[o] = 0u;
    my_lane[o] = 0;
    for (int j = o * L; j < min(p.r.k + 1, (o + 1) * L); ++j) {
      int win;
      const uint32_t best = take(true, &win);
      const bool mine = at.gl == j - o * L;
      my_key[o] = mine ? best : my_key[o];
      my_lane[o] = mine ? win : my_lane[o];
    }
  }
  // Neighbours in the order: too close, and no tie, is an order that 32 bits
  // do not decide.
  Listed<KEEP> list;
  list.close = 0u;
  int id_before = 0;
  uint32_t key_before = 0u;
  bool unsure = false, border = false;           // border: the first left out is close
#pragma unroll
  for (int o = 0; o < KEEP; ++o) {
    const int first = __shfl_sync(kAll, at.first, my_lane[o]);
    list.id[o] = my_key[o] ? first + (V - 1) - (int)(my_key[o] & (uint32_t)(V - 1)) : -1;
    if (!exact) {
      uint32_t kb = __shfl_up_sync(kAll, my_key[o], 1, L);
      int ib = __shfl_up_sync(kAll, list.id[o], 1, L);
      if (at.gl == 0) kb = key_before, ib = id_before;
      key_before = __shfl_sync(kAll, my_key[o], L - 1, L);
      id_before = __shfl_sync(kAll, list.id[o], L - 1, L);
      const bool near = too_close(kb, my_key[o]);
      const uint32_t pairs = __ballot_sync(kAll, near) & at.group;
      const uint32_t open_pairs = __ballot_sync(kAll, near && !same(ib, list.id[o])) & at.group;
      unsure |= open_pairs != 0u;
      // this one and the one behind it
      const uint32_t own = pairs >> (lane & ~(L - 1));
      list.close |= (own >> at.gl & 1u) << o;
      if (at.gl < L - 1) list.close |= (own >> (at.gl + 1) & 1u) << o;
      if (o > 0 && at.gl == L - 1) list.close |= (own & 1u) << (o - 1);
      if (o == p.r.k / L) border = (own >> (p.r.k % L) & 1u) != 0u;
    }
  }
  int n = p.r.k + 1;                             // experts in the list
  bool full = false;
  float low = 0.f;                               // the least rank that can be chosen
  if (!exact) {
    uint32_t last = 0u, out_key = 0u;            // the last chosen, the first left out
    int out_id = 0;
#pragma unroll
    for (int o = 0; o < KEEP; ++o) {
      const uint32_t a = __shfl_sync(kAll, my_key[o], (p.r.k - 1) % L, L);
      const uint32_t b = __shfl_sync(kAll, my_key[o], p.r.k % L, L);
      const int c = __shfl_sync(kAll, list.id[o], p.r.k % L, L);
      if (o == (p.r.k - 1) / L) last = a;
      if (o == p.r.k / L) out_key = b, out_id = c;
    }
    // Whoever is close to the last chosen may stand above it: the order is
    // followed until it leaves its neighbourhood.
    bool on = border;
    while (__any_sync(kAll, on)) {
      int win;
      const uint32_t next = take(on, &win);
      const int id = __shfl_sync(kAll, at.first, win) + (V - 1) - (int)(next & (uint32_t)(V - 1));
      on = on && too_close(last, next);
      if (on) {
        unsure |= !same(out_id, id);
        full |= n >= L * KEEP;
#pragma unroll
        for (int o = 0; o < KEEP; ++o)
          if (o * L + at.gl == n) {
            my_key[o] = next;
            list.id[o] = id;
            list.close |= 1u << o;
          }
        ++n;
      }
    }
    const float least = out_key ? rank_of(out_key) : -INFINITY;
    low = least - 2.f * distance(least, least);
  }
  int my_id[OWN];
#pragma unroll
  for (int o = 0; o < OWN; ++o) my_id[o] = o * L + at.gl < p.r.k ? list.id[o] : -1;
  const int64_t out = (int64_t)t * p.r.k;
  if (open || unsure) {                          // the same for all lanes of a token
    bool done = false;
    if (!open && !full) done = settle<T, L, KEEP>(p, t, lane, list, m, sum);
    if (!done) choose_exact<T, L, V>(p, t, lane, open, kept, low);
    __syncwarp(at.group);                        // the ids, by other lanes of this token
#pragma unroll
    for (int o = 0; o < OWN; ++o)
      my_id[o] = o * L + at.gl < p.r.k ? p.r.ids[out + o * L + at.gl] : -1;
  }
  __syncwarp();
  // the weights, from the chosen logits
  float w[OWN], total = 0.f, peak = -INFINITY;
#pragma unroll
  for (int o = 0; o < OWN; ++o) {
    w[o] = my_id[o] >= 0 && o * L + at.gl < p.r.k ? logit(row + my_id[o]) : -INFINITY;
    peak = fmaxf(peak, w[o]);
  }
  if (!p.sigmoid && p.r.renorm) {
#pragma unroll
    for (int d = L / 2; d > 0; d >>= 1) peak = fmaxf(peak, __shfl_xor_sync(kAll, peak, d));
  }
#pragma unroll
  for (int o = 0; o < OWN; ++o) {
    if (w[o] < -kLargest) w[o] = 0.f;            // no choice
    else if (p.sigmoid) w[o] = 1.f / (1.f + expf(-w[o]));
    else w[o] = expf(w[o] - (p.r.renorm ? peak : m));
    total += w[o];
  }
  if (p.r.renorm) {
    total = group_sum(total, L);
    if (p.sigmoid) total += 1e-20f;
  } else {
    total = sum;
  }
#pragma unroll
  for (int o = 0; o < OWN; ++o)
    if (t >= 0 && o * L + at.gl < p.r.k) {
      p.r.ids[out + o * L + at.gl] = my_id[o];
      p.r.weights[out + o * L + at.gl] = my_id[o] >= 0 ? w[o] / total * p.scale : 0.f;
      if (my_id[o] >= 0) atomicOr(&bits[my_id[o] * stride + word], bit);
    }
}

template <typename T, int L, int V>
__global__ void __launch_bounds__(kThreads)
    route_scored_kernel(const __grid_constant__ ScoreParams p) {
  extern __shared__ uint32_t bits[];                    // [E][stride]
  const Place at = Place::of<L>(p, threadIdx.x & 31);
  clear_bits(bits, p.r.E * bit_stride(p.r.chunk));
  __syncthreads();
  grid_wait();
  grid_go();
  float bias[V];                          // the same for every token
  auto load_bias = [&] {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      if (p.bias && p.bias_vec && i + 4 <= at.own) {
        const float4 b = *reinterpret_cast<const float4*>(p.bias + at.first + i);
        bias[i] = b.x, bias[i + 1] = b.y, bias[i + 2] = b.z, bias[i + 3] = b.w;
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          bias[i + c] = p.bias && i + c < at.own ? p.bias[at.first + i + c] : 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < V; ++i) bias[i] = bias[i] > kLargest ? kLargest : bias[i];   // NaN stays
  };
  if (V == 8) load_bias();
  route_chunk_of<L>(p.r, bits, [&](int t, int lane, int stride, int word, uint32_t bit) {
    if (V > 8) load_bias();               // too many to keep: from L1
    choose_scored<T, L, V>(p, at, t, lane, bias, bits, stride, word, bit);
  });
}

// f for the lanes of a token and the experts of a lane.
template <typename F>
cudaError_t by_shape(int L, int V, F&& f) {
  using std::integral_constant;
  if (V == 8) {
    if (L == 4) return f(integral_constant<int, 4>{}, integral_constant<int, 8>{});
    if (L == 8) return f(integral_constant<int, 8>{}, integral_constant<int, 8>{});
    if (L == 16) return f(integral_constant<int, 16>{}, integral_constant<int, 8>{});
    return f(integral_constant<int, 32>{}, integral_constant<int, 8>{});
  }
  if (V == 16) return f(integral_constant<int, 32>{}, integral_constant<int, 16>{});
  return f(integral_constant<int, 32>{}, integral_constant<int, 32>{});
}

// The kernel with the shared memory of its largest call, once a device (as in
// moe_route.cu: the limit belongs to the kernel, not to a call).
template <typename T, int L, int V>
cudaError_t scored_ready() {
  constexpr int most = (L * V < kMaxGroups ? L * V : kMaxGroups) * bit_stride(kMostChunk) * 4;
  static std::mutex mu;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  std::lock_guard<std::mutex> lk(mu);
  if (!ready[dev & 63]) {
    e = cudaFuncSetAttribute(route_scored_kernel<T, L, V>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    ready[dev & 63] = true;
  }
  return cudaSuccess;
}

}  // namespace

ScoreShape score_shape(int E, int groups) {
  int g = 1;
  while (g < groups) g <<= 1;
  const int size = E / groups;
  for (int i = 0;; ++i) {
    const int L = i < 4 ? 4 << i : 32, V = i < 4 ? 8 : i == 4 ? 16 : 32;
    if (L < g) continue;
    const int lanes = L / g, per = ((size + lanes - 1) / lanes + 3) / 4 * 4;
    if (per <= V || i == 5) return {L, V, lanes, per};
  }
}

cudaError_t launch_route_scored(const RouteCall& r, const ScoreCall& s, cudaStream_t st) {
  // without a restriction the experts are one group
  const int groups = s.top_groups < s.groups ? s.groups : 1;
  const ScoreShape shape = score_shape(r.E, groups);
  if (shape.per > shape.V) return cudaErrorInvalidValue;
  ScoreParams p = {};
  p.r = {r.logits, r.ids, r.weights, r.counts, r.slots, r.tokens, r.hist, (int)r.T,
         r.E,      r.k,   r.renorm,  0,        0,       0,        0};
  p.bias = s.bias;
  p.scale = s.scale;
  p.sigmoid = s.sigmoid;
  p.groups = groups;
  p.top_groups = groups > 1 ? s.top_groups : 1;
  p.best = s.best;
  p.size = r.E / groups;
  p.lanes = shape.lanes;
  p.per = shape.per;
  const bool fours = p.size % 4 == 0;
  p.r.vec = fours && rows_vec(r.logits, r.E, r.dtype);
  p.bias_vec = fours && (reinterpret_cast<uintptr_t>(s.bias) & 15u) == 0;
  route_chunks(&p.r);
  const int smem = r.E * bit_stride(p.r.chunk) * 4;
  auto run = [&](auto* type) {
    using T = std::remove_pointer_t<decltype(type)>;
    return by_shape(shape.L, shape.V, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, V = decltype(v)::value;
      const cudaError_t a = scored_ready<T, L, V>();
      if (a != cudaSuccess) return a;
      return launch_clusters(route_scored_kernel<T, L, V>, 1, (unsigned)p.r.chunks, kThreads, smem,
                             st, p);
    });
  };
  const cudaError_t e = r.dtype == BRA_FP32   ? run((float*)nullptr)
                        : r.dtype == BRA_BF16 ? run((__nv_bfloat16*)nullptr)
                                              : run((__half*)nullptr);
  return e != cudaSuccess ? e : launch_route_places(p.r, st);
}

}  // namespace bra
