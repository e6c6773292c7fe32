// route.cu -- routing of tokens to experts: scores, groups, top-k, weights
// (include/a4w4.h, a4w4_moe_route).
//
// A warp takes one token.  Its E logits become 32-bit keys in shared memory whose
// unsigned order is the order of what is compared (the logits themselves where there is
// no bias: both score functions are increasing; score + bias otherwise).  The k-th
// largest of the 32 lanes' maxima is a lower bound of the k-th largest key, so only the
// few keys at or above it (22 of 896 for k = 16) are looked at again: each one's rank is
// the number of keys above it, no sort and no k passes over the row.
//
// Every loop over the row is short in code: with the keys in registers, and so the
// loops written out, a third of the time went to fetching instructions.  4096 x 896
// experts, sigmoid with a bias, 16 of them chosen: 12.0 us (1.2 TB/s; what bounds it is
// the instructions on each logit and the chain of steps after a row's last one, not
// memory); 1000 x 256 in 8 groups 4.6; one token of 896 3.3, most of it the latency of
// a launch and of that chain.
//
// Choosing as exact scores would: score + bias is known to about 2^-20 of the
// largest score.  Where two neighbours of the chosen order (or a kept and a
// dropped group) are nearer than that and do not come from the same inputs, the
// candidates are compared again as sums of two floats (2^-44), and what then still is
// open, or groups, the row over in 64 bits, of which an SM has few units (some 65 us
// for 896 experts).  Rows with more than 256 candidates go that way too, whatever they are
// compared by: such as tie widely, of ordinary ones none.  4096 rows of equal logits take
// 350 us for 896 experts, 130 for 257, 65 for 256; 256 in 8 groups of equal strength 180.
#include <cfloat>

#include "device.cuh"
#include "kv.cuh"
#include "launch.h"

namespace a4w4 {

namespace {

constexpr int kRouteWarps = 4;
constexpr int kCand = 256;            // candidates that are ranked in shared memory; rows with more are ordered in 64 bits
constexpr unsigned kAll = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ (static_cast<uint32_t>(static_cast<int32_t>(b) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t u) {
  return __uint_as_float(u ^ ((u >> 31) - 1u | 0x80000000u));
}

// What a logit counts as: NaN as -infinity, +infinity as the largest float, -0 as 0.  (Of a NaN
// and a number fmaxf gives the number.)
__device__ __forceinline__ float clean_logit(float x) { return fminf(fmaxf(x, -INFINITY), FLT_MAX) + 0.f; }
__device__ __forceinline__ float clean_bias(float b) { return fmaxf(b, -INFINITY) + 0.f; }

template <bool BF16>
__device__ __forceinline__ float logit(const RouteArgs& p, int t, int e) {
  const long long at = t * p.stride + e;
  return clean_logit(BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p.logits)[at]) << 16)
                          : static_cast<const float*>(p.logits)[at]);
}
__device__ __forceinline__ float bias_of(const RouteArgs& p, int e) { return clean_bias(p.bias[e]); }

// To 2^-21.7 of itself (weights: chosen experts only).
__device__ __forceinline__ float sigmoid(float x) {
  // exp of what is not positive: no overflow, and small scores keep their bits
  const float z = expf(-fabsf(x)), r = __fdividef(1.f, 1.f + z);
  return x >= 0.f ? r : z * r;
}
// The same in fewer instructions, to 2^-21.7 and |x| 2^-23.4 of itself where x < 0: for comparing.
__device__ __forceinline__ float sigmoid_near(float x) {
  const float z = ex2(-1.4426950408889634f * fabsf(x));
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + z));
  return x >= 0.f ? r : z * r;
}
__device__ __forceinline__ double sigmoid_64(double x) { return 1.0 / (1.0 + exp(-x)); }

// (of no NaN)
__device__ __forceinline__ float warp_max(float v) { return from_ordered(__reduce_max_sync(kAll, ordered(v))); }
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ double warp_sum_64(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}

// The k-th largest (k = 1: the largest) of the lanes' values: the largest one that k lanes reach.
// One pass over 32 words instead of the 15 exchanges of a sort over the warp.
__device__ __forceinline__ uint32_t warp_kth(uint32_t v, int k, uint32_t* s_lane, int lane) {
  s_lane[lane] = v;
  __syncwarp();
  int reached = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint4 u = reinterpret_cast<const uint4*>(s_lane)[j];
    reached += (u.x >= v) + (u.y >= v) + (u.z >= v) + (u.w >= v);
  }
  return __reduce_max_sync(kAll, reached >= k ? v : 0u);
}

// ---------------------------------------------------------------------------
// Unevaluated sums of two floats (the error-free sums of Knuth and Dekker, products by fma):
// 2^-46 of the value and more for some ten fp32 instructions, where 64-bit ones wait 100 cycles
// for each other.
struct Pair { float h, l; };
__device__ __forceinline__ Pair fast_two_sum(float a, float b) {      // |a| >= |b|
  const float s = a + b;
  return {s, b - (s - a)};
}
__device__ __forceinline__ Pair two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  const Pair s = two_sum(a.h, b.h);
  return fast_two_sum(s.h, s.l + (a.l + b.l));
}
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  const float p = a.h * b.h;
  return fast_two_sum(p, fmaf(a.h, b.l, fmaf(a.l, b.h, fmaf(a.h, b.h, -p))));
}
__device__ __forceinline__ Pair reciprocal(Pair s) {
  const float r = 1.f / s.h;
  return fast_two_sum(r, r * (fmaf(-s.h, r, 1.f) - s.l * r));
}
__device__ __forceinline__ constexpr Pair as_pair(double v) {
  return {static_cast<float>(v), static_cast<float>(v - static_cast<double>(static_cast<float>(v)))};
}
// exp(d), d <= 0: d = n ln 2 + r, |r| <= 0.35, Taylor's series; 0 below 2^-120.
__device__ __forceinline__ Pair exp_pair(Pair d) {
  constexpr double kLn2 = 0.69314718055994530942;
  constexpr float kA = 0x1.62e4p-1f;                 // 16 bits: n times it is exact
  constexpr Pair kB = as_pair(kLn2 - static_cast<double>(kA));
  if (!(d.h > -83.f)) return {0.f, 0.f};
  const float n = rintf(d.h * 1.44269504f), p = n * kB.h;
  const Pair r = add(add(two_sum(d.h, -n * kA), {d.l, 0.f}), {-p, -fmaf(n, kB.l, fmaf(n, kB.h, -p))});
  constexpr double c8 = 1.0 / 40320, c9 = c8 / 9, c10 = c9 / 10, c11 = c10 / 11, c12 = c11 / 12;
  const float q = fmaf(r.h, fmaf(r.h, fmaf(r.h, fmaf(r.h, float(c12), float(c11)), float(c10)), float(c9)), float(c8));
  Pair e = add(as_pair(1.0 / 5040), mul(r, {q, 0.f}));
  e = add(as_pair(1.0 / 720), mul(r, e));
  e = add(as_pair(1.0 / 120), mul(r, e));
  e = add(as_pair(1.0 / 24), mul(r, e));
  e = add(as_pair(1.0 / 6), mul(r, e));
  e = add({0.5f, 0.f}, mul(r, e));
  e = add({1.f, 0.f}, mul(r, e));
  e = add({1.f, 0.f}, mul(r, e));
  const float scale = pow2i_normal(static_cast<int>(n));
  return {e.h * scale, e.l * scale};
}
__device__ __forceinline__ Pair sigmoid_pair(float x) {
  const Pair z = exp_pair({-fabsf(x), 0.f}), r = reciprocal(add({1.f, 0.f}, z));
  return x >= 0.f ? r : mul(z, r);
}
__device__ __forceinline__ Pair warp_sum(Pair v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = add(v, {__shfl_xor_sync(kAll, v.h, o), __shfl_xor_sync(kAll, v.l, o)});
  return v;
}
// exp(x - top), x <= top, with the difference unrounded: rounded it would be off by 2^-24 of itself, as much
// as the result by 2^-17.7 at a distance of 80.  (Of infinities fmaxf leaves 0.)
__device__ __forceinline__ float exp_of(float x, float top) {
  const Pair d = two_sum(x, -top);
  const float e = expf(d.h);
  return fmaf(e, fmaxf(d.l, -1.f), e);
}
// A key of the same order.  (Infinite biases: nothing is left of the smaller term.)
__device__ __forceinline__ unsigned long long ordered(Pair v) {
  if (!(fabsf(v.h) < INFINITY)) v.l = 0.f;
  return static_cast<unsigned long long>(ordered(v.h + 0.f)) << 32 | ordered(v.l + 0.f);
}

// A group's strength, from its two largest.  (Opposite infinities of a bias: as if it had none.)
template <typename Real>
__device__ __forceinline__ Real strength_of(const RouteArgs& p, Real a, Real b) {
  const Real s = p.group_top == 2 ? a + b : a;
  return s == s ? s : static_cast<Real>(-INFINITY);
}

// Groups whose strength is among the p.top_groups best (ties: the lower index),
// as a mask; lane g < groups holds group g's strength.
template <typename Real>
__device__ __forceinline__ uint32_t best_groups(const RouteArgs& p, Real mine, int lane) {
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) {
    const Real other = __shfl_sync(kAll, mine, g);
    rank += other > mine || (other == mine && g < lane);
  }
  return __ballot_sync(kAll, lane < p.groups && rank < p.top_groups);
}

// The whole choice in 64 bits.  Lane r < topk gets the r-th expert.  For what the rest leaves
// open (see above), and rows with more than kCand keys that tie.  Bound by the few 64-bit
// units of an SM and their latency, so that four exponentials are kept in flight.
template <bool BF16>
__device__ __noinline__ int route_in_64(const RouteArgs& p, int t, int lane) {
  const int E = p.E, per = E / p.groups, n = (E - lane + 31) / 32;
  double c[kRouteMaxExperts / 32];                    // of expert lane + 32 i; NaN: not to be chosen
  if (p.softmax) {
    float m = -INFINITY;
    for (int e = lane; e < E; e += 32) m = fmaxf(m, logit<BF16>(p, t, e));
    m = warp_max(m);
    const double top = m == -INFINITY ? 0.0 : static_cast<double>(m);
    double sum = 0.0;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      c[i] = exp(static_cast<double>(logit<BF16>(p, t, lane + 32 * i)) - top);
      sum += c[i];
    }
    sum = warp_sum_64(sum);
    const double inv = sum > 0.0 ? 1.0 / sum : 0.0;
    for (int i = 0; i < n; ++i) c[i] *= inv;
  } else {
#pragma unroll 4
    for (int i = 0; i < n; ++i) c[i] = sigmoid_64(logit<BF16>(p, t, lane + 32 * i));
  }
  if (p.bias != nullptr)
    for (int i = 0; i < n; ++i) c[i] += static_cast<double>(bias_of(p, lane + 32 * i));
  if (p.groups > 1) {
    double mine = 0.0;
    for (int g = 0; g < p.groups; ++g) {
      double a = -INFINITY, b = -INFINITY;            // the two largest
      for (int i = (g * per - lane + 31) / 32; i < n && lane + 32 * i < (g + 1) * per; ++i) {
        b = fmax(b, fmin(a, c[i]));
        a = fmax(a, c[i]);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const double a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
        b = fmax(fmax(b, b2), fmin(a, a2));
        a = fmax(a, a2);
      }
      if (lane == g) mine = strength_of(p, a, b);
    }
    const uint32_t kept = best_groups<double>(p, mine, lane);
    for (int i = 0; i < n; ++i)
      if ((kept >> ((lane + 32 * i) / per) & 1u) == 0u) c[i] = NAN;
  }
  if (p.bias == nullptr)                               // the logits' own order: scores may have run into 0 or 1
    for (int i = 0; i < n; ++i)
      if (c[i] == c[i]) c[i] = logit<BF16>(p, t, lane + 32 * i);
  int id = 0;
  for (int k = 0; k < p.topk; ++k) {
    double best = 0.0;
    int at = -1;
    for (int i = 0; i < n; ++i) {
      if (c[i] == c[i] && (at < 0 || c[i] > best)) {
        best = c[i];
        at = lane + 32 * i;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const double b2 = __shfl_xor_sync(kAll, best, o);
      const int a2 = __shfl_xor_sync(kAll, at, o);
      if (a2 >= 0 && (at < 0 || b2 > best || (b2 == best && a2 < at))) {
        best = b2;
        at = a2;
      }
    }
    if (lane == (at & 31)) c[at >> 5] = NAN;          // topk <= the kept groups' experts: at >= 0
    if (lane == k) id = at;
  }
  return id;
}

// Four logits of a row from expert e on; -infinity behind the last.
template <bool BF16>
__device__ __forceinline__ float4 raw_logits(const RouteArgs& p, long long row, int e) {
  float x[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
  const long long at = row + e;
  if (p.vectors) {                                    // E and the rows' starts are multiples of four values
    if (e < p.E) {
      if (BF16) {
        const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.logits) + at);
        x[0] = __uint_as_float(w.x << 16); x[1] = __uint_as_float(w.x & 0xFFFF0000u);
        x[2] = __uint_as_float(w.y << 16); x[3] = __uint_as_float(w.y & 0xFFFF0000u);
      } else {
        const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + at);
        x[0] = w.x; x[1] = w.y; x[2] = w.z; x[3] = w.w;
      }
    }
  } else {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (e + u < p.E)
        x[u] = BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p.logits)[at + u]) << 16)
                    : static_cast<const float*>(p.logits)[at + u];
  }
  return make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ float4 clean(float4 x) {
  return make_float4(clean_logit(x.x), clean_logit(x.y), clean_logit(x.z), clean_logit(x.w));
}
template <bool BF16>
__device__ __forceinline__ float4 four_logits(const RouteArgs& p, long long row, int e) {
  return clean(raw_logits<BF16>(p, row, e));
}
__device__ __forceinline__ float4 four_biases(const RouteArgs& p, int e) {
  if (p.bias_vectors) {
    const float4 w = e < p.E ? *reinterpret_cast<const float4*>(p.bias + e) : make_float4(0.f, 0.f, 0.f, 0.f);
    return make_float4(clean_bias(w.x), clean_bias(w.y), clean_bias(w.z), clean_bias(w.w));
  }
  float b[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int u = 0; u < 4; ++u)
    if (e + u < p.E) b[u] = bias_of(p, e + u);
  return make_float4(b[0], b[1], b[2], b[3]);
}
// Keys of experts e .. e + 3; 0 behind the last, below every other.
__device__ __forceinline__ uint4 four_keys(float4 c, int e, int E) {
  return make_uint4(ordered(c.x), e + 1 < E ? ordered(c.y) : 0u, e + 2 < E ? ordered(c.z) : 0u, e + 3 < E ? ordered(c.w) : 0u);
}
__device__ __forceinline__ float4 four_sums(float4 a, float4 b) { return make_float4(a.x + b.x, a.y + b.y, a.z + b.z, a.w + b.w); }

// Two candidates a >= b, by the upper words of their keys: may their exact scores lie the other way around?
// (Infinite ones, of a bias, are equal.)
__device__ __forceinline__ bool scores_near(unsigned long long a, unsigned long long b, float margin) {
  const float va = from_ordered(static_cast<uint32_t>(a >> 32)), vb = from_ordered(static_cast<uint32_t>(b >> 32));
  return !(va - vb > margin + fmaxf(fabsf(va), fabsf(vb)) * 0x1p-22f) && (va != vb || fabsf(va) < INFINITY);
}
// The same of sums of two floats.
__device__ __forceinline__ bool sums_near(unsigned long long a, unsigned long long b, float margin) {
  const float ah = from_ordered(static_cast<uint32_t>(a >> 32)), bh = from_ordered(static_cast<uint32_t>(b >> 32));
  const float gap = (ah - bh) + (from_ordered(static_cast<uint32_t>(a)) - from_ordered(static_cast<uint32_t>(b)));
  const float open = (margin + fmaxf(fabsf(ah), fabsf(bh)) * 0x1p-22f) * 0x1p-20f;
  return !(gap > open) && (ah != bh || fabsf(ah) < INFINITY);
}
// Do experts a and b have the same score, whatever its last bits?
template <bool BF16>
__device__ __forceinline__ bool same_inputs(const RouteArgs& p, int t, int a, int b) {
  return logit<BF16>(p, t, a) == logit<BF16>(p, t, b) && bias_of(p, a) == bias_of(p, b);
}

template <bool BF16>
__global__ void __launch_bounds__(32 * kRouteWarps, 8) moe_route_kernel(const RouteArgs p) {
  __shared__ alignas(16) unsigned long long s_key[kRouteWarps][kCand + 4];
  __shared__ uint16_t s_at[kRouteWarps][kCand];
  __shared__ unsigned long long s_top[kRouteWarps][34];   // the best in order, one more than can be asked for
  __shared__ alignas(16) uint32_t s_lane[kRouteWarps][32];
  extern __shared__ uint4 s_row[];                          // [kRouteWarps][row_quads]: the row's keys (or logits)
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + warp, E = p.E, topk = p.topk;
  if (t >= p.T) return;
  const int count = p.count != nullptr ? *p.count : p.T;    // (looked at when the logits are on their way)
  const long long row = t * p.stride;
  uint4* quad = s_row + warp * p.row_quads;             // quad q: experts 4 q .. + 3, of lane q % 32
  const uint32_t* keys = reinterpret_cast<const uint32_t*>(quad);

  // scores where they are compared: with a bias, or as sums of two
  const bool by_score = p.bias != nullptr, by_sum = p.groups > 1 && (by_score || p.group_top == 2);
  const bool summed = p.softmax && (by_score || by_sum || !p.renorm);      // the row's sum is needed
  float top = -INFINITY;
  uint32_t most = 0u;                                   // the lane's largest key
  constexpr int kAhead = 4;                             // quads of a lane on their way
  for (int q0 = lane; 4 * q0 < E; q0 += 32 * kAhead) {
    float4 raw[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) raw[i] = raw_logits<BF16>(p, row, 4 * (q0 + 32 * i));
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const int q = q0 + 32 * i;
      if (4 * q >= E) break;
      const float4 x = clean(raw[i]);
      top = fmaxf(fmaxf(top, fmaxf(x.x, x.y)), fmaxf(x.z, x.w));
      if (summed) {
        reinterpret_cast<float4*>(quad)[q] = x;
      } else {
        const float4 c = by_score ? four_sums(make_float4(sigmoid_near(x.x), sigmoid_near(x.y), sigmoid_near(x.z), sigmoid_near(x.w)),
                                              four_biases(p, 4 * q))
                                  : x;
        const uint4 k = four_keys(c, 4 * q, E);
        quad[q] = k;
        most = max(max(most, max(k.x, k.y)), max(k.z, k.w));
      }
    }
  }
  int32_t* ids = p.ids + static_cast<long long>(t) * topk;
  float* weights = p.weights + static_cast<long long>(t) * topk;
  if (t >= count) {
    if (lane < topk) {
      ids[lane] = -1;
      weights[lane] = 0.f;
    }
    return;
  }

  // `margin` bounds how far apart two scores may be and still change places
  float inv = 0.f, margin = 0.f;
  if (summed || by_score || by_sum) top = warp_max(top);
  if (summed) {
    if (top == -INFINITY) top = 0.f;
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = lane; 4 * q < E; q += 32) {
      const float4 x = reinterpret_cast<const float4*>(quad)[q];
      sum = four_sums(sum, make_float4(expf(x.x - top), expf(x.y - top), expf(x.z - top), expf(x.w - top)));
    }
    const float z = warp_sum((sum.x + sum.y) + (sum.z + sum.w));
    inv = z > 0.f ? 1.f / z : 0.f;
    margin = inv * 0x1p-18f;        // the sum's 23 roundings, and the exponentials'
    for (int q = lane; 4 * q < E; q += 32) {
      const float4 x = reinterpret_cast<const float4*>(quad)[q];
      const float4 c = by_score ? four_sums(make_float4(expf(x.x - top) * inv, expf(x.y - top) * inv, expf(x.z - top) * inv,
                                                        expf(x.w - top) * inv),
                                            four_biases(p, 4 * q))
                                : x;
      const uint4 k = four_keys(c, 4 * q, E);
      quad[q] = k;
      most = max(max(most, max(k.x, k.y)), max(k.z, k.w));
    }
  } else if (by_score || by_sum) {
    margin = sigmoid_near(top) * (0x1p-19f + fmaxf(-top, 0.f) * 0x1p-21f);
    if (top >= 0.f) margin *= 0.5f;
    if (top == -INFINITY) margin = 0.f;
  }
  margin += 0x1p-120f;              // scores so small that they have lost bits

  bool in_64 = false;
  if (p.groups > 1) {
    __syncwarp();
    // L lanes take a group; groups begin with different places of theirs, which lie on different banks
    const int L = p.group_lanes, g = lane / L, per = E / p.groups, n = (per + L - 1) / L;
    float a = -INFINITY, b = -INFINITY;              // the two largest
    if (g < p.groups) {
      int j = g % n;
      for (int i = 0; i < n; ++i) {
        const int at = j * L + (lane & (L - 1));
        if (at < per) {
          float c = from_ordered(keys[g * per + at]);
          if (by_sum && !by_score) c = p.softmax ? expf(c - top) * inv : sigmoid_near(c);
          b = fmaxf(b, fminf(a, c));
          a = fmaxf(a, c);
        }
        if (++j == n) j = 0;
      }
    }
    for (int o = L >> 1; o > 0; o >>= 1) {
      const float a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
      b = fmaxf(fmaxf(b, b2), fminf(a, a2));
      a = fmaxf(a, a2);
    }
    const float strength = __shfl_sync(kAll, strength_of(p, a, b), lane * L & 31);
    // logits are compared as they are; of a sum of two the error is twice a score's and the roundings of c and of the sum
    float largest = fmaxf(fabsf(a), p.group_top == 2 ? fabsf(b) : 0.f);
    largest = warp_max(largest < INFINITY ? largest : 0.f);
    const uint32_t kept = best_groups<float>(p, strength, lane);
    if (by_sum && p.top_groups < p.groups) {          // do the weakest kept and the strongest dropped group lie too near?
      const bool in = lane < p.groups, mine = kept >> lane & 1u;
      const float least = from_ordered(__reduce_min_sync(kAll, mine ? ordered(strength + 0.f) : kAll));
      const float next = from_ordered(__reduce_max_sync(kAll, in && !mine ? ordered(strength + 0.f) : 0u));
      in_64 = !(least - next > 2.f * margin + largest * 0x1p-21f);
    }
    most = 0u;
    for (int q = lane; 4 * q < E; q += 32) {
      uint4 k = quad[q];
      const auto drop = [&](uint32_t v, int e) { return kept >> (__umulhi(static_cast<unsigned>(e), p.per_recip) & 31u) & 1u ? v : 0u; };
      k = make_uint4(drop(k.x, 4 * q), drop(k.y, 4 * q + 1), drop(k.z, 4 * q + 2), drop(k.w, 4 * q + 3));
      quad[q] = k;
      most = max(max(most, max(k.x, k.y)), max(k.z, k.w));
    }
  }

  int id = 0;
  float xi = -INFINITY;                               // lane r < topk: the r-th expert and its logit
  if (!in_64) {
    uint32_t floor_key = max(warp_kth(most, topk, s_lane[warp], lane), 1u);
    const float f = from_ordered(floor_key);
    if (by_score && fabsf(f) < INFINITY)             // (no such key: NaN)
      floor_key = max(ordered(f - (margin + fabsf(f) * 0x1p-22f)), 1u);
    int before = 0;
    for (int q = lane; 4 * q < E; q += 32) {
      const uint4 k = quad[q];
      before += (k.x >= floor_key) + (k.y >= floor_key) + (k.z >= floor_key) + (k.w >= floor_key);
    }
    const int mine = before;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(kAll, before, o);
      if (lane >= o) before += u;
    }
    const int n = __shfl_sync(kAll, before, 31);
    before -= mine;
    in_64 = n > kCand;
    if (!in_64) {
      unsigned long long* cand = s_key[warp];
      unsigned long long* best = s_top[warp];
      if (mine > 0) {
        for (int q = lane; 4 * q < E; q += 32) {
          const uint4 k = quad[q];
          const uint32_t v[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (v[u] >= floor_key)
              cand[before++] = static_cast<unsigned long long>(v[u]) << 32 | (kAll - (4 * q + u));   // of equals the lower first
        }
      }
      if (lane < 4) cand[n + lane] = 0ull;            // below every key: the ranks are counted four at a time
      __syncwarp();
      for (int i = lane; i < n; i += 32) {
        const unsigned long long c = cand[i];
        int rank = 0;
#pragma unroll 2
        for (int j = 0; j < n; j += 4) {
          const ulonglong2 u = *reinterpret_cast<const ulonglong2*>(cand + j);
          const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(cand + j + 2);
          rank += (u.x > c) + (u.y > c) + (v.x > c) + (v.y > c);
        }
        if (rank <= topk) best[rank] = c;
      }
      __syncwarp();
      const unsigned long long c = best[lane < n && lane < topk ? lane : 0];
      id = static_cast<int>(kAll - static_cast<uint32_t>(c));
      xi = by_score ? logit<BF16>(p, t, id) : from_ordered(static_cast<uint32_t>(c >> 32));
      bool near = false, twin = false;
      if (by_score && lane < topk && lane + 1 < n) {
        const unsigned long long d = best[lane + 1];
        if (scores_near(c, d, margin)) {
          near = !same_inputs<BF16>(p, t, id, static_cast<int>(kAll - static_cast<uint32_t>(d)));
          twin = !near && lane + 1 == topk;
        }
      }
      bool open = __any_sync(kAll, near || twin);
      if (open && __any_sync(kAll, twin)) {
        // The last one chosen and the first one left have the same inputs: behind them may lie others,
        // as near, whose inputs differ.
        const unsigned long long last = best[topk - 1];
        const int e = static_cast<int>(kAll - static_cast<uint32_t>(last));
        for (int i = lane; i < n; i += 32)
          near |= cand[i] < last && scores_near(last, cand[i], margin) &&
                  !same_inputs<BF16>(p, t, e, static_cast<int>(kAll - static_cast<uint32_t>(cand[i])));
        open = __any_sync(kAll, near);
      }
      if (open) {
        Pair share = {1.f, 0.f};                      // a softmax's 1 / sum
        if (p.softmax) {
          Pair sum = {0.f, 0.f};
          for (int q = lane; 4 * q < E; q += 32) {
            const float4 x = four_logits<BF16>(p, row, 4 * q);
            sum = add(sum, add(add(exp_pair(two_sum(x.x, -top)), exp_pair(two_sum(x.y, -top))),
                               add(exp_pair(two_sum(x.z, -top)), exp_pair(two_sum(x.w, -top)))));
          }
          share = reciprocal(warp_sum(sum));
        }
        for (int i = lane; i < n; i += 32) {
          const int e = static_cast<int>(kAll - static_cast<uint32_t>(cand[i]));
          const float x = logit<BF16>(p, t, e);
          const Pair score = p.softmax ? mul(exp_pair(two_sum(x, -top)), share) : sigmoid_pair(x);
          s_at[warp][i] = static_cast<uint16_t>(e);
          cand[i] = ordered(add(score, {bias_of(p, e), 0.f}));
        }
        __syncwarp();
        for (int i = lane; i < n; i += 32) {
          const unsigned long long v = cand[i];
          const int e = s_at[warp][i];
          int rank = 0;
          for (int j = 0; j < n; ++j) rank += cand[j] > v || (cand[j] == v && s_at[warp][j] < e);
          if (rank <= topk) best[rank] = static_cast<unsigned>(i);
        }
        __syncwarp();
        const int i = static_cast<int>(best[lane < topk ? lane : 0]);
        id = s_at[warp][i];
        xi = logit<BF16>(p, t, id);
        near = twin = false;
        if (lane < topk && lane + 1 < n) {
          const int j = static_cast<int>(best[lane + 1]);
          if (sums_near(cand[i], cand[j], margin)) {
            near = !same_inputs<BF16>(p, t, id, s_at[warp][j]);
            twin = !near && lane + 1 == topk;
          }
        }
        if (__any_sync(kAll, twin)) {
          const int l = static_cast<int>(best[topk - 1]), e = s_at[warp][l];
          const unsigned long long last = cand[l];
          for (int j = lane; j < n; j += 32) {
            const int other = s_at[warp][j];
            near |= (cand[j] < last || (cand[j] == last && other > e)) && sums_near(last, cand[j], margin) &&
                    !same_inputs<BF16>(p, t, e, other);
          }
        }
        in_64 = __any_sync(kAll, near);
      }
    }
  }
  if (in_64) {
    id = route_in_64<BF16>(p, t, lane);
    xi = logit<BF16>(p, t, id);
  }

  // weights: scores of the chosen ones, with the largest of them brought near 1 where they are divided by their sum
  const bool mine = lane < topk;
  if (!mine) xi = -INFINITY;
  float m = top;
  if (p.renorm) m = by_score ? warp_max(xi) : __shfl_sync(kAll, xi, 0);
  float w;
  if (p.softmax || (p.renorm && m < 0.f)) {           // (below 0 a sigmoid may run out of fp32)
    w = exp_of(xi, m);
    if (!p.softmax) w = __fdividef(w, 1.f + expf(xi));
  } else {
    w = sigmoid(xi);
  }
  if (p.renorm) {
    w = mine ? w : 0.f;
    w = __fdividef(w, warp_sum(w));
    if (m == -INFINITY) w = 0.f;                      // nothing to share
  } else if (p.softmax) {
    w *= inv;
  }
  if (mine) {
    ids[lane] = id;
    weights[lane] = w * p.scale;
  }
}

}  // namespace

int launch_moe_route(RouteArgs p, int bf16, cudaStream_t st) {
  const int per = p.E / p.groups;
  // 16 bytes (8 in BF16) at a time
  p.vectors = p.E % 4 == 0 && p.stride % 4 == 0 && reinterpret_cast<uintptr_t>(p.logits) % (bf16 ? 8 : 16) == 0;
  p.bias_vectors = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.bias) % 16 == 0;
  p.per_recip = p.groups > 1 ? static_cast<unsigned>((0x100000000ull + per - 1) / per) : 0u;   // per >= 2
  p.group_lanes = 1;
  while (2 * p.group_lanes * p.groups <= 32) p.group_lanes *= 2;
  p.row_quads = (p.E + 3) / 4;
  return launch_pdl_smem(bf16 ? moe_route_kernel<true> : moe_route_kernel<false>, (p.T + kRouteWarps - 1) / kRouteWarps,
                         32 * kRouteWarps, sizeof(uint4) * kRouteWarps * p.row_quads, st, p);
}

}  // namespace a4w4
