// route.cu -- routing of tokens to experts: scores, groups, top-k, weights
// (include/a4w4.h, a4w4_moe_route).
//
// A warp takes one token.  Its E logits stay in registers as 32-bit keys whose
// unsigned order is the order of what is compared (the logits themselves where
// there is no bias: both score functions are increasing; score + bias
// otherwise).  The k-th largest of the 32 lanes' maxima is a lower bound of the
// k-th largest key, so only the few keys at or above it (22 of 896 for k = 16)
// go to shared memory, where each one's rank is the number of keys above it: no
// sort and no k passes over the row.
//
// Choosing as exact scores would: score + bias is known to about 2^-21 of the
// largest score.  Where two neighbours of the chosen order (or a kept and a
// dropped group) are nearer than that and do not come from the same inputs, 64
// bits decide: for the candidates alone (sigmoid), or for the row.
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
  const float z = expf(-fabsf(x)), r = __frcp_rn(1.f + z);
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

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
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
// Fewer trips than sorting over the warp: T = 1 x 896 experts SORT_TIME us.
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

// A group's strength, from its two largest.  (Opposite infinities of a bias: as if it had none.)
template <typename Real>
__device__ __forceinline__ Real strength_of(const RouteArgs& p, Real a, Real b) {
  const Real s = p.group_top == 2 ? a + b : a;
  return s == s ? s : static_cast<Real>(-INFINITY);
}

// Groups whose strength is among the p.top_groups best (ties: the lower index),
// as a mask; lane g < groups holds group g's strength.  *near: a kept and a
// dropped group lie within `margin` of each other.
template <typename Real>
__device__ __forceinline__ uint32_t best_groups(const RouteArgs& p, Real mine, int lane, Real margin, bool* near) {
  int rank = 0;
  for (int g = 0; g < p.groups; ++g) {
    const Real other = __shfl_sync(kAll, mine, g);
    rank += other > mine || (other == mine && g < lane);
  }
  const bool in = lane < p.groups, kept = in && rank < p.top_groups;
  const uint32_t mask = __ballot_sync(kAll, kept);
  if (near != nullptr) {
    bool close = false;
    for (int g = 0; g < p.groups; ++g) {
      const Real other = __shfl_sync(kAll, mine, g);
      close |= kept && (mask >> g & 1u) == 0u && !(mine - other > margin);
    }
    *near = __any_sync(kAll, close);
  }
  return mask;
}

// The whole choice in 64 bits.  Lane r < topk gets the r-th expert.  Rare (see
// above), or rows with more than kCand keys that tie.  Bound by the few 64-bit units of
// an SM and their latency, so that four exponentials are kept in flight.
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
    const uint32_t kept = best_groups<double>(p, mine, lane, 0.0, nullptr);
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

// NV: keys per lane, four consecutive experts each (expert 4 (32 i + lane) + u).
template <int NV, bool BF16>
__global__ void __launch_bounds__(32 * kRouteWarps, NV <= 32 ? 7 : 3) moe_route_kernel(const RouteArgs p) {
  __shared__ alignas(16) unsigned long long s_key[kRouteWarps][kCand + 4];
  __shared__ uint16_t s_at[kRouteWarps][kCand];
  __shared__ unsigned long long s_top[kRouteWarps][34];   // the best in order, one more than can be asked for
  __shared__ alignas(16) uint32_t s_lane[kRouteWarps][32];
  extern __shared__ float s_val[];                          // with groups: [kRouteWarps][E + groups * 32]
  griddep_wait();
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = blockIdx.x * kRouteWarps + warp, E = p.E, topk = p.topk;
  if (t >= p.T) return;
  const int count = p.count != nullptr ? *p.count : p.T;    // (looked at when the logits are on their way)

  float x[NV];
#pragma unroll
  for (int i = 0; i < NV; i += 4) {
    const int e = 4 * (i / 4 * 32 + lane);
    const long long at = t * p.stride + e;
    x[i] = x[i + 1] = x[i + 2] = x[i + 3] = -INFINITY;
    if (p.vectors) {                                  // E and the rows' starts are multiples of four values
      if (e < E) {
        if (BF16) {
          const uint2 w = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p.logits) + at);
          x[i] = __uint_as_float(w.x << 16); x[i + 1] = __uint_as_float(w.x & 0xFFFF0000u);
          x[i + 2] = __uint_as_float(w.y << 16); x[i + 3] = __uint_as_float(w.y & 0xFFFF0000u);
        } else {
          const float4 w = *reinterpret_cast<const float4*>(static_cast<const float*>(p.logits) + at);
          x[i] = w.x; x[i + 1] = w.y; x[i + 2] = w.z; x[i + 3] = w.w;
        }
      }
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (e + u < E)
          x[i + u] = BF16 ? __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(p.logits)[at + u]) << 16)
                          : static_cast<const float*>(p.logits)[at + u];
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
#pragma unroll
  for (int i = 0; i < NV; ++i) x[i] = clean_logit(x[i]);

  // scores where they are compared; `margin` bounds how far apart two of them may be and still change places
  const bool by_score = p.bias != nullptr, by_sum = p.groups > 1 && (by_score || p.group_top == 2);
  float top = -INFINITY, inv = 0.f, margin = 0.f;
  if (by_score || by_sum || (p.softmax && !p.renorm)) {
#pragma unroll
    for (int i = 0; i < NV; ++i) top = fmaxf(top, x[i]);
    top = warp_max(top);
    if (p.softmax) {
      if (top == -INFINITY) top = 0.f;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) sum[i & 3] += expf(x[i] - top);
      const float z = warp_sum((sum[0] + sum[1]) + (sum[2] + sum[3]));
      inv = z > 0.f ? 1.f / z : 0.f;
      margin = inv * 0x1p-18f;      // the sum's 23 roundings, and the exponentials'
    } else {
      margin = sigmoid(top) * (0x1p-19f + fmaxf(-top, 0.f) * 0x1p-21f);
      if (top >= 0.f) margin *= 0.5f;
      if (top == -INFINITY) margin = 0.f;
    }
    margin += 0x1p-120f;            // scores so small that they have lost bits
  }
  uint32_t key[NV];
  if (by_score || by_sum) {
    float* val = s_val + warp * p.val_stride;
#pragma unroll
    for (int i = 0; i < NV; i += 4) {
      const int e = 4 * (i / 4 * 32 + lane);
      float b[4] = {0.f, 0.f, 0.f, 0.f};
      if (by_score) {
        if (p.bias_vectors) {
          if (e < E) {
            const float4 w = *reinterpret_cast<const float4*>(p.bias + e);
            b[0] = clean_bias(w.x); b[1] = clean_bias(w.y); b[2] = clean_bias(w.z); b[3] = clean_bias(w.w);
          }
        } else {
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (e + u < E) b[u] = bias_of(p, e + u);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float c = (p.softmax ? expf(x[i + u] - top) * inv : sigmoid_near(x[i + u])) + b[u];
        key[i + u] = e + u < E ? ordered(by_score ? c : x[i + u]) : 0u;
        if (by_sum && e + u < E) val[e + u + __umulhi(static_cast<unsigned>(e + u), p.per_recip) * p.skew] = c;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = 4 * (i / 4 * 32 + lane) + (i & 3);
      key[i] = e < E ? ordered(x[i]) : 0u;
      if (p.groups > 1 && e < E)
        s_val[warp * p.val_stride + e + __umulhi(static_cast<unsigned>(e), p.per_recip) * p.skew] = x[i];
    }
  }

  bool in_64 = false;
  if (p.groups > 1) {
    // `skew` lanes take a group; groups start that many banks apart
    __syncwarp();
    const int L = p.skew, g = lane / L, per = E / p.groups;
    float a = -INFINITY, b = -INFINITY;              // the two largest
    if (g < p.groups) {
      const float* val = s_val + warp * p.val_stride + g * (per + L);
      for (int j = lane & (L - 1); j < per; j += L) {
        const float c = val[j];
        b = fmaxf(b, fminf(a, c));
        a = fmaxf(a, c);
      }
    }
    for (int o = L >> 1; o > 0; o >>= 1) {
      const float a2 = __shfl_xor_sync(kAll, a, o), b2 = __shfl_xor_sync(kAll, b, o);
      b = fmaxf(fmaxf(b, b2), fminf(a, a2));
      a = fmaxf(a, a2);
    }
    const float strength = __shfl_sync(kAll, strength_of(p, a, b), lane * L & 31);
    // logits are compared as they are; of a sum of two the error is twice a score's and the roundings of c and of the sum
    float most = fmaxf(fabsf(a), p.group_top == 2 ? fabsf(b) : 0.f);
    most = warp_max(most < INFINITY ? most : 0.f);
    const uint32_t kept = best_groups<float>(p, strength, lane, 2.f * margin + most * 0x1p-21f, by_sum ? &in_64 : nullptr);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = 4 * (i / 4 * 32 + lane) + (i & 3);
      const int ge = __umulhi(static_cast<unsigned>(e), p.per_recip);
      if (e < E && (kept >> (ge & 31) & 1u) == 0u) key[i] = 0u;
    }
  }

  int id = 0;
  float xi = -INFINITY;                               // lane r < topk: the r-th expert and its logit
  if (!in_64) {
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < NV; ++i) most = max(most, key[i]);
    uint32_t floor_key = max(warp_kth(most, topk, s_lane[warp], lane), 1u);
    const float f = from_ordered(floor_key);
    if (by_score && fabsf(f) < INFINITY)             // (no such key: NaN)
      floor_key = max(ordered(f - (margin + fabsf(f) * 0x1p-22f)), 1u);
    int mine = 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) mine += key[i] >= floor_key;
    int before = mine;
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
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (key[i] >= floor_key) {
          const unsigned e = 4 * (i / 4 * 32 + lane) + (i & 3);
          cand[before++] = static_cast<unsigned long long>(key[i]) << 32 | (kAll - e);   // of equals the lower comes first
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
      bool near = false;
      if (by_score && lane < topk && lane + 1 < n) {
        const unsigned long long d = best[lane + 1];
        const float vc = from_ordered(static_cast<uint32_t>(c >> 32)), vd = from_ordered(static_cast<uint32_t>(d >> 32));
        if (!(vc - vd > margin + fmaxf(fabsf(vc), fabsf(vd)) * 0x1p-22f) && (vc != vd || fabsf(vc) < INFINITY)) {
          const int other = static_cast<int>(kAll - static_cast<uint32_t>(d));
          near = xi != logit<BF16>(p, t, other) || bias_of(p, id) != bias_of(p, other);
        }
      }
      if (__any_sync(kAll, near)) {
        if (p.softmax) {
          in_64 = true;                               // the row's sum has to be known better too
        } else {
          for (int i = lane; i < n; i += 32) {
            const int e = static_cast<int>(kAll - static_cast<uint32_t>(cand[i]));
            const double v = sigmoid_64(logit<BF16>(p, t, e)) + static_cast<double>(bias_of(p, e)) + 0.0;
            const long long b = __double_as_longlong(v);
            s_at[warp][i] = static_cast<uint16_t>(e);
            cand[i] = static_cast<unsigned long long>(b ^ (b >> 63 | static_cast<long long>(1ull << 63)));
          }
          __syncwarp();
          for (int i = lane; i < n; i += 32) {
            const unsigned long long v = cand[i];
            const int e = s_at[warp][i];
            int rank = 0;
            for (int j = 0; j < n; ++j) rank += cand[j] > v || (cand[j] == v && s_at[warp][j] < e);
            if (rank < topk) best[rank] = static_cast<unsigned>(e);
          }
          __syncwarp();
          id = static_cast<int>(best[lane < topk ? lane : 0]);
          xi = logit<BF16>(p, t, id);
        }
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
  float w;
  if (p.renorm) {
    const float m = by_score ? warp_max(xi) : __shfl_sync(kAll, xi, 0);
    if (m == -INFINITY) {
      w = 0.f;                                        // nothing to share
    } else {
      if (p.softmax) {
        w = expf(xi - m);
      } else {
        const float base = fminf(m, 0.f);
        w = xi >= 0.f ? sigmoid(xi) : expf(xi - base) / (1.f + expf(xi));
      }
      w = mine ? w : 0.f;
      w /= warp_sum(w);
    }
  } else {
    w = p.softmax ? expf(xi - top) * inv : sigmoid(xi);
  }
  if (mine) {
    ids[lane] = id;
    weights[lane] = w * p.scale;
  }
}

template <bool BF16>
int launch_route_type(const RouteArgs& p, cudaStream_t st) {
  const int grid = (p.T + kRouteWarps - 1) / kRouteWarps;
  const size_t smem = p.groups > 1 ? sizeof(float) * kRouteWarps * p.val_stride : 0;
  auto kern = p.E <= 128   ? moe_route_kernel<4, BF16>
              : p.E <= 256 ? moe_route_kernel<8, BF16>
              : p.E <= 512 ? moe_route_kernel<16, BF16>
              : p.E <= 1024 ? moe_route_kernel<32, BF16>
                            : moe_route_kernel<64, BF16>;
  return launch_pdl_smem(kern, grid, 32 * kRouteWarps, smem, st, p);
}

}  // namespace

int launch_moe_route(RouteArgs p, int bf16, cudaStream_t st) {
  const int per = p.E / p.groups;
  // 16 bytes (8 in BF16) at a time
  p.vectors = p.E % 4 == 0 && p.stride % 4 == 0 && reinterpret_cast<uintptr_t>(p.logits) % (bf16 ? 8 : 16) == 0;
  p.bias_vectors = p.E % 4 == 0 && reinterpret_cast<uintptr_t>(p.bias) % 16 == 0;
  p.per_recip = p.groups > 1 ? static_cast<unsigned>((0x100000000ull + per - 1) / per) : 0u;   // per >= 2
  p.skew = 1;
  while (2 * p.skew * p.groups <= 32) p.skew *= 2;
  p.val_stride = p.E + p.groups * p.skew;
  return bf16 ? launch_route_type<true>(p, st) : launch_route_type<false>(p, st);
}

}  // namespace a4w4
