// rope.cu -- norms of query and key heads and their rotation by position, to BF16
// (a4w4_qk_norm_rope), or with the keys and the values to the paged MXFP4 cache
// (a4w4_kv_append_rope).  Formulas: include/a4w4.h.
//
// A thread block takes one token (or, of few tokens, a part of one).  A thread holds
// eight dimensions of a head (16 bytes), D / 8 threads a head, a warp 256 / D heads (a
// unit) at a time.  With y = r w x (r the reciprocal of the root mean square, w
// the norm's weight) dimension i and its partner p of a pair become A_i (r x_i) + B_i (r x_p),
// A_i = w_i cos, B_i = +-w_p sin: the token's coefficients are formed once, in shared
// memory, while its heads are on their way to registers.  r comes first, so that nothing
// on the way passes fp32's range that the result does not.
//
// Angles: position times frequency as turns, in 64-bit integers modulo one turn
// (F = f / 2 pi as a 96-bit binary fraction, position * F wraps): within 2^-63 turns at
// any position.  Quarter turns are taken off in integers, so that what is left keeps
// its bits wherever a sine or cosine comes near zero.
#include <algorithm>
#include <atomic>

#include "device.cuh"
#include "kv.cuh"
#include "kv_walk.cuh"
#include "launch.h"

namespace a4w4 {

namespace {

constexpr int kRopeWarps = 4;
// Blocks on an SM.  More of them do not pay for the registers that they take from each other:
// 8191 x 40 heads of 128 with 5 29.7 us, 6 30.0, 7 34.7; to the cache (and read) with 3 57.4, 4 53.9, 5 67.3.
template <bool CACHE>
constexpr int kRopeBlocks = CACHE ? 4 : 5;
constexpr int kRopeBatch = 4;          // units whose norms go through one reduction
constexpr int kRopeUnits = 32;         // of a part of a token: 16 KB a stage
constexpr unsigned kAll = 0xFFFFFFFFu;

// A frequency in turns per position, modulo 1: hi 2^-64 + lo 2^-96.
struct Turns {
  unsigned long long hi;
  uint32_t lo;
  // position times it, in units of 2^-64 turns (cut by 1.5 of them at most)
  __device__ __forceinline__ unsigned long long at(int position) const {
    const int32_t low = static_cast<int32_t>(__umulhi(static_cast<uint32_t>(position), lo) - (position < 0 ? lo : 0u));
    return static_cast<unsigned long long>(static_cast<long long>(position)) * hi + static_cast<unsigned long long>(static_cast<long long>(low));
  }
};

// f / (2 pi) modulo 1: the 24-bit significand times 128 binary places of 1 / (2 pi) (a quarter
// of the first 130 of 2 / pi).
__device__ __forceinline__ Turns turns_per_position(float f) {
  constexpr unsigned long long kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;
  const uint32_t b = __float_as_uint(f), ex = b >> 23 & 255u;
  const unsigned long long m = (b & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
  const int down = max(150 - static_cast<int>(ex ? ex : 1u), 0);     // f = m 2^-down, below 2^24
  // m (kHi : kLo), 152 bits
  const unsigned long long p0 = m * kLo;
  unsigned long long p1 = m * kHi;
  const unsigned long long c = __umul64hi(m, kLo);
  unsigned long long p2 = __umul64hi(m, kHi);
  p1 += c;
  p2 += p1 < c;
  // shifted down, whole words first
  const int words = down >> 6, bits = down & 63;
  const unsigned long long w0 = words == 0 ? p0 : words == 1 ? p1 : words == 2 ? p2 : 0ull;
  const unsigned long long w1 = words == 0 ? p1 : words == 1 ? p2 : 0ull, w2 = words == 0 ? p2 : 0ull;
  unsigned long long hi = w1 >> bits | (w2 << 1) << (63 - bits);
  uint32_t lo = static_cast<uint32_t>((w0 >> bits | (w1 << 1) << (63 - bits)) >> 32);
  if (b >> 31) {
    lo = 0u - lo;
    hi = ~hi + (lo == 0u);
  }
  return {hi, lo};
}

// An angle less its nearest quarter turns: an eighth of a turn at most, in units of 2^-64 turns.
__device__ __forceinline__ long long off_quarter(unsigned long long turn, uint32_t* quarters) {
  const uint32_t up = static_cast<uint32_t>(turn >> 32);
  *quarters = (up + (1u << 29)) >> 30;
  return static_cast<long long>(static_cast<unsigned long long>(up - (*quarters << 30)) << 32 | (turn & 0xFFFFFFFFull));
}
// Sine and cosine of an angle so many quarter turns further.
template <typename Real>
__device__ __forceinline__ void turn_quarters(uint32_t quarters, Real* s, Real* c) {
  const Real s0 = *s, c0 = *c;
  if (quarters & 1u) {
    *s = c0;
    *c = -s0;
  }
  if (quarters & 2u) {
    *s = -*s;
    *c = -*c;
  }
}

__device__ __forceinline__ Two two_of_bf16(uint32_t w) {
  return pack2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ Two swapped(Two v) { return pack2(hi_of(v), lo_of(v)); }

// E2M1 code (with its sign) of a 64-bit value: rounded towards zero to fp32, with the last bit set
// where something was lost, which no border of E2M1 has.
__device__ __forceinline__ uint32_t e2m1_of(double y) {
  float f = __double2float_rz(y);
  if (static_cast<double>(f) != y) f = __uint_as_float(__float_as_uint(f) | 1u);
  return cvt_e2m1x8(f, f, f, f, f, f, f, f) & 15u;
}

__device__ __forceinline__ float bf16_of(const uint4& x, int u) {
  const uint32_t w = u < 4 ? (u < 2 ? x.x : x.y) : (u < 6 ? x.z : x.w);
  return __uint_as_float(u & 1 ? w & 0xFFFF0000u : w << 16);
}

// Sum of the squares of a thread's eight dimensions (five roundings).
__device__ __forceinline__ float squares_of(const uint4& v) {
  const Two a = two_of_bf16(v.x), b = two_of_bf16(v.y), c = two_of_bf16(v.z), d = two_of_bf16(v.w);
  const Two s = fma2(a, a, fma2(b, b, fma2(c, c, mul2(d, d))));
  return lo_of(s) + hi_of(s);
}

// Is a mean square (with eps) one that fp32 sums are good for?  Above, squares may have passed its range;
// below, lost bits.
__device__ __forceinline__ bool in_range(float v) { return v > 0x1p-100f && v < 0x1p119f; }

// What follows runs seldom.  It stands apart and takes values: a member function that is called
// would keep its object in memory, which the loops would then read again and again.

// Reciprocal of the root mean square of a head (LPH threads) in 64 bits.
template <int LPH>
__device__ __noinline__ double norm_64(uint4 x, float eps) {
  double ssq = 0.0;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const double a = bf16_of(x, u);
    ssq = fma(a, a, ssq);
  }
  // the warp as a whole is here
#pragma unroll
  for (int o = LPH / 2; o > 0; o >>= 1) ssq += __shfl_xor_sync(kAll, ssq, o);
  return rsqrt(ssq * (1.0 / (8 * LPH)) + static_cast<double>(eps));
}

// The values of a unit of keys that fp32 leaves open (a bit each in `open`) in 64 bits: their
// codes in `code` with the scale 1 / unit, or, where `unit` is negative, whether one of them
// reaches -unit in magnitude.  turns: per position, of each pair; eps 0: no norm.  One value
// costs its warp some 3 us, for the latency of the few 64-bit units.
template <int D>
__device__ __noinline__ uint32_t keys_64(const float* w, const Turns* turns, float eps, int rot, int pairs,
                                         int position, uint4 x, uint4 y, uint32_t open, uint32_t code, double unit) {
  constexpr int LPH = D / 8;
  const int d0 = 8 * ((threadIdx.x & 31) % LPH), half = rot / 2;
  const bool second = !pairs && d0 >= half;
  const double r = eps > 0.f ? norm_64<LPH>(x, eps) : 1.0;
  uint32_t reached = 0u;
#pragma unroll 1
  for (; open != 0u; open &= open - 1u) {
    const int u = __ffs(open) - 1, d = d0 + u;
    double o = bf16_of(x, u) * static_cast<double>(w[d]);
    if (d0 < rot) {
      const int other = pairs ? d ^ 1 : second ? d - half : d + half;
      double s, c;
      uint32_t quarters;
      sincospi(static_cast<double>(off_quarter(turns[pairs ? d / 2 : second ? other : d].at(position), &quarters)) * 0x1p-63, &s, &c);
      turn_quarters(quarters, &s, &c);
      const double par = bf16_of(y, u) * static_cast<double>(w[other]);
      o = o * c + par * ((pairs ? (u & 1) != 0 : second) ? s : -s);
    }
    o *= r;
    reached |= fabs(o) >= -unit;
    code = (code & ~(15u << (4 * u))) | e2m1_of(o * unit) << (4 * u);
  }
  return unit < 0.0 ? reached : code;
}

// A token's coefficients, of queries and of keys.
template <int D>
struct RopeCoef {
  float a[2][D], b[2][D];
};

// What forms them: thread i of a block's first D / 2 has pair i; where fewer pairs turn,
// two dimensions that stay.
template <int D, bool PAIRS>
struct RopePair {
  bool mine, turns;
  int u, w;                                              // dimensions
  Turns per_position;

  __device__ __forceinline__ explicit RopePair(const RopeArgs& p) {
    const int i = threadIdx.x, half = p.rot / 2;
    mine = i < D / 2;
    turns = i < half;
    u = !PAIRS && turns ? i : 2 * i;
    w = !PAIRS && turns ? i + half : 2 * i + 1;
    per_position = turns ? turns_per_position(p.inv_freq[i]) : Turns{0ull, 0u};
  }
  __device__ __forceinline__ void form(int position, const float (*weight)[D], RopeCoef<D>& out) const {
    if (!mine) return;
    float c = 1.f, s = 0.f;
    if (turns) {
      // at most a quarter of a half turn, rounded to 24 bits of itself: sine and cosine are within 2^-22.7
      // of themselves (of every float there sincospif's results were within 2^-23.4)
      uint32_t quarters;
      sincospif(__ll2float_rn(off_quarter(per_position.at(position), &quarters)) * 0x1p-63f, &s, &c);
      turn_quarters(quarters, &s, &c);
    }
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
      const float wu = weight[kind][u], ww = weight[kind][w];
      out.a[kind][u] = wu * c;
      out.a[kind][w] = ww * c;
      // (-0: what does not turn adds -0, which leaves a zero its sign)
      out.b[kind][u] = turns ? -ww * s : -0.f;
      out.b[kind][w] = turns ? wu * s : -0.f;
    }
  }
};

// Keys and values to the cache: a thread holds eight consecutive dimensions of a head, and a
// partner's eight come from another thread where halves are paired.
template <int D>
struct RopeCells {
  static constexpr int LPH = D / 8, HPW = 32 / LPH;      // threads per head, heads of a unit
  const RopeArgs& p;
  const int lane, d0, sub;                               // first dimension of this thread, head of the HPW
  int partner;                                           // thread with the pairs' other halves (half split)
  bool rotated, second;                                  // whether d0 .. d0 + 7 turn; are second halves of their pairs
  float lost;                                            // what a key may be off by besides `rel`, for subnormal numbers on the way

  // weight: of keys.  In 2^-150: r x is off by 1 if it is subnormal, A times that, a subnormal A by 1, r |x| <= sqrt(D) times
  // that, each of two terms; their products by 1 each, `off`'s own terms too: 2 max |w| + 2 sqrt(D) + 6.
  __device__ __forceinline__ RopeCells(const RopeArgs& args, const float* weight)
      : p(args), lane(threadIdx.x & 31), d0(8 * (lane % LPH)), sub(lane / LPH) {
    uint32_t most = 0u;
#pragma unroll
    for (int i = 0; i < D; i += 32) most = max(most, __float_as_uint(fabsf(weight[i + lane])));
    lost = fmaf(__uint_as_float(__reduce_max_sync(kAll, most)), 0x1p-149f, 0x1p-145f);
    const int half = p.rot / 2;
    rotated = d0 < p.rot;
    second = !p.interleaved && d0 >= half;
    partner = !rotated || p.interleaved ? lane : second ? lane - half / 8 : lane + half / 8;
  }

  // Reciprocal of the root mean square of a head (over the LPH threads that hold it), to 2^-21.4:
  // nine roundings of what is under the root, halved, and those of the last step.
  __device__ __forceinline__ float norm(const uint4& x) const {
    float ssq = squares_of(x);
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ssq += __shfl_xor_sync(kAll, ssq, o);
    const float v = fmaf(ssq, 1.f / D, p.eps), r = rsqrtf(v);
    if (__any_sync(kAll, !in_range(v))) return static_cast<float>(norm_64<LPH>(x, p.eps));
    return fmaf(0.5f * r, fmaf(-v * r, r, 1.f), r);
  }

  __device__ __forceinline__ uint4 partners(const uint4& x) const {
    uint4 y;
    if (p.interleaved) {
      y.x = x.x << 16 | x.x >> 16; y.y = x.y << 16 | x.y >> 16;
      y.z = x.z << 16 | x.z >> 16; y.w = x.w << 16 | x.w >> 16;
    } else {
      y.x = __shfl_sync(kAll, x.x, partner); y.y = __shfl_sync(kAll, x.y, partner);
      y.z = __shfl_sync(kAll, x.z, partner); y.w = __shfl_sync(kAll, x.w, partner);
    }
    return rotated ? y : make_uint4(0u, 0u, 0u, 0u);      // what stays as it is takes nothing from a neighbour
  }

  // o = A (r x) + B (r y), and what it may be off by (nothing where it is x).
  __device__ __forceinline__ void rotate(const RopeCoef<D>& coef, const uint4& x, const uint4& y, float r, float* o,
                                         float* off) const {
    constexpr float rel = 0x1.dp-21f;
    const bool exact = !rotated && p.k_weight == nullptr;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int u = 0; u < 8; u += 4) {
      const float4 A = *reinterpret_cast<const float4*>(coef.a[1] + d0 + u), B = *reinterpret_cast<const float4*>(coef.b[1] + d0 + u);
      const float a[4] = {A.x, A.y, A.z, A.w}, b[4] = {B.x, B.y, B.z, B.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t wi = w[(u + i) / 2], vi = v[(u + i) / 2];
        const float m = a[i] * (r * __uint_as_float(i & 1 ? wi & 0xFFFF0000u : wi << 16));
        const float n = b[i] * (r * __uint_as_float(i & 1 ? vi & 0xFFFF0000u : vi << 16));
        o[u + i] = m + n;
        off[u + i] = exact ? 0.f : fmaf(fabsf(m), rel, fmaf(fabsf(n), rel, lost));
      }
    }
  }

  static __device__ __forceinline__ uint32_t codes_of(const Two* y) {
    return cvt_e2m1x8(lo_of(y[0]), hi_of(y[0]), lo_of(y[1]), hi_of(y[1]), lo_of(y[2]), hi_of(y[2]), lo_of(y[3]), hi_of(y[3]));
  }

  __device__ __forceinline__ uint8_t* chunk_of(int slot, int h) const {
    const int chunks = 1 << (p.page_lg - 4);
    return p.cache + kv_chunk_offset<D>(slot >> p.page_lg, h, (slot >> 4) & (chunks - 1), p.Hkv, chunks);
  }

  // Keys to the cache, quantised from the fp32 value o = A (r x) + B (r y).  What is known of it: r to
  // 2^-21.4 of itself, sine and cosine to 2^-22.7 of themselves, the weight's product, those with r and
  // with a coefficient and the sum a rounding each: in all within 2^-20.4 of |A r x| + |B r y| and, with
  // a rounding of the ends of the range that this leaves, 2^-20.1 (and `lost`); without norm or
  // rotation o is x.  Where that leaves a code or the scale open, 64 bits decide (some 5 codes of a
  // million).  (A NaN has no part in the scale, as in a4w4_kv_append.)
  __device__ __forceinline__ void key_cell(const RopeCoef<D>& coef, const float* weight, const Turns* turns,
                                           const uint4& v, int n, int slot, int position) const {
    using Ch = KvChunk<D>;
    const bool normed = p.k_weight != nullptr;
    const float r = normed ? norm(v) : 1.f;
    const uint4 y = partners(v);
    float o[8], off[8];
    rotate(coef, v, y, r, o, off);
    float least = 0.f, most = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      least = fmaxf(least, fabsf(o[u]) - off[u]);
      most = fmaxf(most, fabsf(o[u]) + off[u]);
    }
    least = fmaxf(least, __shfl_xor_sync(kAll, least, 1));
    most = fmaxf(most, __shfl_xor_sync(kAll, most, 1));
    least = fmaxf(least, __shfl_xor_sync(kAll, least, 2));
    most = fmaxf(most, __shfl_xor_sync(kAll, most, 2));
    uint32_t eb = __float_as_uint(most) >> 23;
    if (__any_sync(kAll, __float_as_uint(least) >> 23 != eb || eb == 255u)) {
      // does the largest magnitude reach the power of two that `most` has passed?  (2^128: the
      // values that fp32 has no number for tell)
      const bool beyond = eb == 255u;
      const float power = __uint_as_float(eb << 23);
      uint32_t open = 0u;
#pragma unroll
      for (int u = 0; u < 8; ++u) open |= (least < power || beyond) && fabsf(o[u]) + off[u] >= power ? 1u << u : 0u;
      uint32_t reached = keys_64<D>(weight, turns, normed ? p.eps : 0.f, p.rot, p.interleaved, position, v, y, open, 0u,
                                    beyond ? -0x1p128 : -static_cast<double>(power));      // (the warp as a whole)
      reached |= least >= power && !beyond;
      reached |= __shfl_xor_sync(kAll, reached, 1);
      reached |= __shfl_xor_sync(kAll, reached, 2);
      if (reached == 0u) --eb;
    }
    const uint32_t e = eb > 2u ? eb - 2u : 0u;
    const float inv = __uint_as_float((254u - e) << 23);
    const Two i2 = pack2(inv, inv), j2 = pack2(-inv, -inv);
    Two lo[4], hi[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const Two m = mul2(pack2(o[2 * u], o[2 * u + 1]), i2), d = pack2(off[2 * u], off[2 * u + 1]);
      lo[u] = fma2(d, j2, m);
      hi[u] = fma2(d, i2, m);
    }
    uint32_t code = codes_of(lo);
    const uint32_t diff = code ^ codes_of(hi);
    if (__any_sync(kAll, diff != 0u || eb == 255u)) {
      // (of zeros nothing is lost: they have the code of o)
      const uint32_t in[4] = {v.x | y.x, v.y | y.y, v.z | y.z, v.w | y.w};
      uint32_t open = 0u, zeros = 0u;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool zero = (in[u / 2] & (u & 1 ? 0x7FFF0000u : 0x7FFFu)) == 0u;
        zeros |= zero ? 15u << (4 * u) : 0u;
        open |= !zero && ((diff >> (4 * u) & 15u) != 0u || (eb == 255u && !(fabsf(o[u]) < INFINITY))) ? 1u << u : 0u;
      }
      const Two mid[4] = {mul2(pack2(o[0], o[1]), i2), mul2(pack2(o[2], o[3]), i2), mul2(pack2(o[4], o[5]), i2), mul2(pack2(o[6], o[7]), i2)};
      code = (code & ~zeros) | (codes_of(mid) & zeros);
      if (__any_sync(kAll, open != 0u)) code = keys_64<D>(weight, turns, normed ? p.eps : 0.f, p.rot, p.interleaved, position, v, y, open, code, inv);
    }
    const int h = n * HPW + sub;
    if (h < p.Hkv) {
      uint8_t* chunk = chunk_of(slot, h);
      const int row = slot & 15;
      *reinterpret_cast<uint32_t*>(chunk + Ch::key_word(row, d0 / 32, d0 % 32 / 8)) = code;
      if (d0 % 32 == 0) chunk[Ch::kKeyScales + row * Ch::J + d0 / 32] = static_cast<uint8_t>(e);
    }
  }

  __device__ __forceinline__ void value_cell(const uint4& v, int n, int slot) const {
    using Ch = KvChunk<D>;
    uint32_t m = max_abs_bf16x2(max_abs_bf16x2(v.x, v.y), max_abs_bf16x2(v.z, v.w));
    m = max_abs_bf16x2(m, __shfl_xor_sync(kAll, m, 1));
    m = max_abs_bf16x2(m, __shfl_xor_sync(kAll, m, 2)) & 0x7FFF7FFFu;
    const uint32_t eb = max(m & 0xFFFFu, m >> 16) >> 7, e = eb > 2u ? eb - 2u : 0u;
    const float inv = __uint_as_float((254u - e) << 23);
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      f[2 * u] = __uint_as_float(w[u] << 16) * inv;
      f[2 * u + 1] = __uint_as_float(w[u] & 0xFFFF0000u) * inv;
    }
    const uint32_t code = cvt_e2m1x8(f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]);
    // Thread l has the bytes of runs 4 (l % 2) .. + 3 at place i = l / 2; it writes four
    // places of one run: i0 .. i0 + 3 of run `run`.
    const int l = lane % LPH, run = D == 128 ? l / 2 : l, i0 = D == 128 ? 4 * (l & 1) : 0;
    uint32_t word = 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = __shfl_sync(kAll, code, sub * LPH + 2 * (i0 + i) + run / 4);
      word |= (c >> (8 * (run & 3)) & 255u) << (8 * i);
    }
    const int h = n * HPW + sub;
    if (h < p.Hkv) {
      uint8_t* chunk = chunk_of(slot, h);
      const int row = slot & 15;
      *reinterpret_cast<uint32_t*>(chunk + Ch::value_run(row, run) + i0) = word;
      if (d0 % 32 == 0) chunk[Ch::kValueScales + row * Ch::J + d0 / 32] = static_cast<uint8_t>(e);
    }
  }
};

// Heads to BF16 rows: a thread holds two runs of four dimensions of a head, which are each
// other's partners where halves are paired, so that nothing crosses threads but the sums of
// squares; those of four units go through one reduction.
template <int D, bool PAIRS>
struct RopeRows {
  static constexpr int LPH = D / 8, HPW = 32 / LPH;
  const RopeArgs& p;
  const int lane, sub;
  int da, db;                                            // first dimensions of the runs
  bool rotated;
  Two Aa[2], Ab[2], Ba[2], Bb[2];

  __device__ __forceinline__ explicit RopeRows(const RopeArgs& args)
      : p(args), lane(threadIdx.x & 31), sub(lane / LPH) {
    const int j = lane % LPH, h = PAIRS ? 0 : p.rot / 8;  // threads of a head that hold two halves
    da = j < h ? 4 * j : 8 * j;
    db = j < h ? 4 * (j + h) : 8 * j + 4;
    rotated = da < p.rot;
  }
  __device__ __forceinline__ void coefficients(const RopeCoef<D>& c, int kind) {
    const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(c.a[kind] + da), y = *reinterpret_cast<const ulonglong2*>(c.a[kind] + db);
    const ulonglong2 z = *reinterpret_cast<const ulonglong2*>(c.b[kind] + da), w = *reinterpret_cast<const ulonglong2*>(c.b[kind] + db);
    Aa[0] = x.x; Aa[1] = x.y; Ab[0] = y.x; Ab[1] = y.y;
    Ba[0] = z.x; Ba[1] = z.y; Bb[0] = w.x; Bb[1] = w.y;
  }
  // x: this thread's head of the unit.
  __device__ __forceinline__ uint4 load(const uint16_t* x) const {
    const uint2 a = *reinterpret_cast<const uint2*>(x + da), b = *reinterpret_cast<const uint2*>(x + db);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
  __device__ __forceinline__ float norm(const uint4& v) const {
    float s = squares_of(v);
#pragma unroll
    for (int o = 1; o < LPH; o <<= 1) s += __shfl_xor_sync(kAll, s, o);
    const float mean = s * (1.f / D) + p.eps;
    return __any_sync(kAll, !in_range(mean)) ? static_cast<float>(norm_64<LPH>(v, p.eps)) : rsqrtf(mean);
  }
  // The same for four units.
  __device__ __forceinline__ void norms(const uint4* v, float* r) const {
    const float s0 = squares_of(v[0]), s1 = squares_of(v[1]), s2 = squares_of(v[2]), s3 = squares_of(v[3]);
    const bool odd = lane & 1, upper = lane & 2;
    // lane l ends up with unit l % 4's sum
    const float a = (odd ? s1 : s0) + __shfl_xor_sync(kAll, odd ? s0 : s1, 1);
    const float b = (odd ? s3 : s2) + __shfl_xor_sync(kAll, odd ? s2 : s3, 1);
    float s = (upper ? b : a) + __shfl_xor_sync(kAll, upper ? a : b, 2);
#pragma unroll
    for (int o = 4; o < LPH; o <<= 1) s += __shfl_xor_sync(kAll, s, o);
    const float mean = s * (1.f / D) + p.eps, q = rsqrtf(mean);
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = __shfl_sync(kAll, q, (lane & ~3) | i);
    if (__any_sync(kAll, !in_range(mean))) {
#pragma unroll
      for (int i = 0; i < 4; ++i) r[i] = static_cast<float>(norm_64<LPH>(v[i], p.eps));
    }
  }
  __device__ __forceinline__ void store(const uint4& v, float r, uint16_t* x) const {
    const Two r2 = pack2(r, r);
    const Two a[2] = {mul2(r2, two_of_bf16(v.x)), mul2(r2, two_of_bf16(v.y))};
    const Two b[2] = {mul2(r2, two_of_bf16(v.z)), mul2(r2, two_of_bf16(v.w))};
    const bool stays = p.rot < D && !rotated;            // what stays as it is takes nothing from a neighbour
    uint32_t o[4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      Two pa = PAIRS ? swapped(a[u]) : b[u], pb = PAIRS ? swapped(b[u]) : a[u];
      if (stays) pa = pb = 0ull;
      const Two x = fma2(Aa[u], a[u], mul2(Ba[u], pa)), y = fma2(Ab[u], b[u], mul2(Bb[u], pb));
      o[u] = pack_bf16(lo_of(x), hi_of(x));
      o[2 + u] = pack_bf16(lo_of(y), hi_of(y));
    }
    *reinterpret_cast<uint2*>(x + da) = make_uint2(o[0], o[1]);
    *reinterpret_cast<uint2*>(x + db) = make_uint2(o[2], o[3]);
  }
  // Units n .. e - 1 (this warp's), of which this thread has a head in those below m: from rows in
  // shared memory to rows `out` (both: this thread's head of unit 0).
  __device__ __forceinline__ void run(const uint16_t* x, uint16_t* out, const float* w, int n, int e, int m) const {
    const uint4 none = make_uint4(0u, 0u, 0u, 0u);
    for (; n + 1 < e; n += kRopeBatch) {
      uint4 v[kRopeBatch];
#pragma unroll
      for (int i = 0; i < kRopeBatch; ++i) v[i] = n + i < m ? load(x + (n + i) * 256) : none;
      float r[kRopeBatch] = {1.f, 1.f, 1.f, 1.f};
      if (w != nullptr) norms(v, r);
#pragma unroll
      for (int i = 0; i < kRopeBatch; ++i)
        if (n + i < m) store(v[i], r[i], out + (n + i) * 256);
    }
    if (n < e) {
      const uint4 v = n < m ? load(x + n * 256) : none;
      const float r = w != nullptr ? norm(v) : 1.f;
      if (n < m) store(v, r, out + n * 256);
    }
  }
};

// What a warp does of a part of a token: units first .. end - 1, of which this thread has a head in
// those below `mine`.  The part's n units from u0 go to the warps in runs, warp `start` the first.
struct RopeRun {
  int first, end, mine;
  __device__ __forceinline__ RopeRun(int u0, int n, int start, int heads_end) {
    const int run = (n + kRopeWarps - 1) / kRopeWarps, w = ((threadIdx.x >> 5) - start) & (kRopeWarps - 1);
    first = u0 + min(w * run, n);
    end = u0 + min((w + 1) * run, n);
    mine = min(end, heads_end);
  }
};

// A block walks over tokens (or over one part of the heads of each: of few tokens, or of tokens
// with very many heads).  One thread copies the next token's heads to shared memory while
// the block works on this one's; the next token's coefficients go to the other buffer too.
// 8191 tokens x 40 heads of 128 with norms: 29.7 us, 5.6 TB/s.
template <int D, bool CACHE, bool PAIRS>
__global__ void __launch_bounds__(32 * kRopeWarps, kRopeBlocks<CACHE>) kv_rope_kernel(const RopeArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];         // two stages of heads, two sets of coefficients
  __shared__ alignas(8) unsigned long long s_bar[2];
  __shared__ int s_flags[2];
  __shared__ Turns s_turns[CACHE ? D / 2 : 1];   // per position, of each pair
  __shared__ float s_weight[2][D];                       // the norms' (1 without), of queries and of keys
  using Rows = RopeRows<D, PAIRS>;
  constexpr int HPW = Rows::HPW;
  const uint32_t bar = smem_u32(s_bar);
  volatile int *abort_flag = s_flags, *never = s_flags + 1;
  if (threadIdx.x == 0) {
    mbar_init(bar, 1);
    mbar_init(bar + 8u, 1);
    s_flags[0] = s_flags[1] = 0;
    fence_barrier_init();
  }
  const int part = p.split > 1 ? blockIdx.x % p.split : 0, stride = gridDim.x / p.split;
  const int uq = (p.Hq + HPW - 1) / HPW, uk = (p.Hkv + HPW - 1) / HPW;
  // this part's units
  const int q0 = part * p.part_q, q1 = min(q0 + p.part_q, uq), k0 = part * p.part_kv, k1 = min(k0 + p.part_kv, uk);
  const int nq = max(q1 - q0, 0), nk = max(k1 - k0, 0);
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();

  RopeCoef<D>* coef = reinterpret_cast<RopeCoef<D>*>(smem + 2 * p.stage_bytes);
  const int off_k = p.part_q * 512, off_v = off_k + p.part_kv * 512;       // within a stage
  auto issue = [&](long long t, int slot, int s) {                          // thread 0
    const uint32_t fb = bar + 8u * s, dst = smem_u32(smem) + s * p.stage_bytes;
    if (CACHE && static_cast<unsigned>(slot) >= static_cast<unsigned>(p.slots)) {
      mbar_arrive(fb);                                    // nothing to be done, nothing to be fetched
      return;
    }
    const int bq = (min(q1 * HPW, p.Hq) - q0 * HPW) * D * 2, bk = (min(k1 * HPW, p.Hkv) - k0 * HPW) * D * 2;
    mbar_arrive_expect_tx(fb, (nq > 0 ? bq : 0) + (nk > 0 ? (CACHE ? 2 : 1) * bk : 0));
    const uint64_t pol = policy_evict_first();
    if (nq > 0) bulk_g2s(dst, p.q + t * p.q_stride + q0 * 256, bq, fb, pol);
    if (nk > 0) bulk_g2s(dst + off_k, p.k + t * p.k_stride + k0 * 256, bk, fb, pol);
    if (CACHE && nk > 0) bulk_g2s(dst + off_v, p.v + t * p.v_stride + k0 * 256, bk, fb, pol);
  };
  long long t = blockIdx.x / p.split;                     // below T
  int slot = 0, next_slot = 0, issued = 0, done = 0;
  if (CACHE) {
    slot = p.slot_map[t];
    next_slot = t + stride < p.T ? p.slot_map[t + stride] : -1;
  }
  if (threadIdx.x == 0) {
    issue(t, slot, 0);
    if (t + stride < p.T) issue(t + stride, next_slot, 1);
    issued = t + stride < p.T ? 2 : 1;
  }
  if (threadIdx.x < D) {
    s_weight[0][threadIdx.x] = p.q_weight != nullptr ? p.q_weight[threadIdx.x] : 1.f;
    s_weight[1][threadIdx.x] = p.k_weight != nullptr ? p.k_weight[threadIdx.x] : 1.f;
  }
  __syncthreads();
  Rows rows(p);
  const RopeCells<D> cells(p, s_weight[1]);
  const RopePair<D, PAIRS> pair(p);
  if (CACHE && pair.turns) s_turns[threadIdx.x] = pair.per_position;
  // queries, keys and values begin with the warp after the last one of those before
  const int with_q = nq > 0 ? (nq - 1) / ((nq + kRopeWarps - 1) / kRopeWarps) + 1 : 0;
  const int with_k = nk > 0 ? (nk - 1) / ((nk + kRopeWarps - 1) / kRopeWarps) + 1 : 0;
  const RopeRun rq(q0, nq, 0, (p.Hq - rows.sub + HPW - 1) / HPW);
  const RopeRun rk(k0, nk, with_q, (p.Hkv - rows.sub + HPW - 1) / HPW);
  const RopeRun rv(k0, nk, with_q + with_k, (p.Hkv - rows.sub + HPW - 1) / HPW);
  int position = p.rot > 0 ? p.positions[t] : 0;
  pair.form(position, s_weight, coef[0]);
  __syncthreads();
  for (int s = 0;; s ^= 1) {
    const bool more = t + stride < p.T;
    const int next_position = more && p.rot > 0 ? p.positions[t + stride] : 0;
    const int ahead_slot = CACHE && t + 2 * stride < p.T ? p.slot_map[t + 2 * stride] : -1;
    const bool ok = __all_sync(kAll, kv_wait(bar + 8u * s, (done >> 1) & 1, abort_flag, p.wait_ns, p.status));
    done += ok;
    const uint16_t* stage = reinterpret_cast<const uint16_t*>(smem + s * p.stage_bytes);
    const RopeCoef<D>& now = coef[s];
    if (ok && (!CACHE || static_cast<unsigned>(slot) < static_cast<unsigned>(p.slots))) {
      if (rq.first < rq.end) {
        rows.coefficients(now, 0);
        rows.run(stage + rows.sub * D - q0 * 256, p.q_out + t * p.q_out_stride + rows.sub * D, p.q_weight, rq.first, rq.end,
                 rq.mine);
      }
      const uint16_t *k = stage + off_k / 2 - k0 * 256, *v = stage + off_v / 2 - k0 * 256;
      if (CACHE) {
        const uint4 none = make_uint4(0u, 0u, 0u, 0u);
        for (int n = rk.first; n < rk.end; ++n)
          cells.key_cell(now, s_weight[1], s_turns, n < rk.mine ? *reinterpret_cast<const uint4*>(k + n * 256 + cells.lane * 8) : none, n, slot, position);
        for (int n = rv.first; n < rv.end; ++n)
          cells.value_cell(n < rv.mine ? *reinterpret_cast<const uint4*>(v + n * 256 + cells.lane * 8) : none, n, slot);
      } else if (rk.first < rk.end) {
        rows.coefficients(now, 1);
        rows.run(k + rows.sub * D, p.k_out + t * p.k_out_stride + rows.sub * D, p.k_weight, rk.first, rk.end, rk.mine);
      }
    }
    if (!more) break;
    pair.form(next_position, s_weight, coef[s ^ 1]);
    if (__syncthreads_or(!ok)) break;
    if (threadIdx.x == 0 && t + 2 * stride < p.T) {
      issue(t + 2 * stride, ahead_slot, s);
      ++issued;
    }
    t += stride;
    position = next_position;
    slot = next_slot;
    next_slot = ahead_slot;
  }
  // every copy issued lands before the shared memory is released
  if (threadIdx.x == 0) {
    const unsigned long long drain_ns = p.wait_ns > 100000000ull ? p.wait_ns : 100000000ull;
    for (; done < issued; ++done) mbar_wait(bar + 8u * (done & 1), (done >> 1) & 1, never, drain_ns, p.status);
  }
}

template <int D, bool CACHE, bool PAIRS>
int launch_rope_kind(RopeArgs p, cudaStream_t st, int sms) {
  auto kern = kv_rope_kernel<D, CACHE, PAIRS>;
  const int smem = 2 * p.stage_bytes + 2 * static_cast<int>(sizeof(RopeCoef<D>));
  static std::atomic<unsigned long long> attr_devs{0};   // bit d: attribute set on device d
  if (ensure_func_attrs(attr_devs, [&] {
        return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                    2 * kRopeUnits * 512 + 2 * static_cast<int>(sizeof(RopeCoef<D>))) == cudaSuccess;
      }) != 0)
    return -4;
  // as many blocks as stay on the SMs at once
  int fit = 233472 / (smem + 2304 + 1024);                // with what the kernel and the system hold of it
  if (fit > kRopeBlocks<CACHE>) fit = kRopeBlocks<CACHE>;
  const long long items = static_cast<long long>(p.T) * p.split, most = static_cast<long long>(fit) * sms / p.split * p.split;
  return launch_pdl_smem(kern, static_cast<int>(items < most ? items : most), 32 * kRopeWarps, smem, st, p);
}

template <int D, bool CACHE>
int launch_rope_d(const RopeArgs& p, cudaStream_t st, int sms) {
  return p.interleaved ? launch_rope_kind<D, CACHE, true>(p, st, sms) : launch_rope_kind<D, CACHE, false>(p, st, sms);
}

}  // namespace

int launch_kv_rope(RopeArgs p, int D, cudaStream_t st, int sms) {
  const bool cache = p.cache != nullptr;
  const int per = 256 / D, uq = (p.Hq + per - 1) / per, uk = (p.Hkv + per - 1) / per, kinds = cache ? 2 : 1;
  // parts of a token: what a stage holds (69 at most: 4096 heads); of few tokens so many that there
  // are four blocks on every SM, with a unit for each warp, but no more than SMs
  int split = 1;
  const auto units = [&](int n) { return (uq + n - 1) / n + kinds * ((uk + n - 1) / n); };
  while (units(split) > kRopeUnits) ++split;
  const long long want = std::min<long long>((4ll * sms + p.T - 1) / p.T, sms);
  while (split < want && units(split) > kRopeWarps) ++split;
  p.split = split;
  p.part_q = (uq + split - 1) / split;
  p.part_kv = (uk + split - 1) / split;
  p.stage_bytes = units(split) * 512;
  return D == 64 ? (cache ? launch_rope_d<64, true>(p, st, sms) : launch_rope_d<64, false>(p, st, sms))
                 : (cache ? launch_rope_d<128, true>(p, st, sms) : launch_rope_d<128, false>(p, st, sms));
}

}  // namespace a4w4
