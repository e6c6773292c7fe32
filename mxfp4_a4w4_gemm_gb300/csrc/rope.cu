// rope.cu -- norms of query and key heads and their rotation by position, to BF16
// (a4w4_qk_norm_rope), or with the keys and the values to the paged MXFP4 cache
// (a4w4_kv_append_rope).  Formulas: include/a4w4.h.
//
// A thread holds eight consecutive dimensions of a head (16 bytes), D / 8 threads
// a head, a warp 256 / D heads of one token at a time.  With y = r w x (r the
// reciprocal of the root mean square, w the norm's weight) dimension i and its
// partner p of a pair become r (A_i x_i + B_i x_p), A_i = w_i cos, B_i = +-w_p sin:
// sixteen coefficients in registers for all heads of a token, and four shuffles of
// packed BF16 where the partner is another thread's.
//
// Angles: position times frequency as turns, in 64-bit integers modulo one turn
// (F = f / 2 pi as a 64-bit binary fraction, position * F wraps): exact to 2^-33
// turns at position 2^31, so that 32 bits are enough for what is left.
#include "device.cuh"
#include "kv.cuh"
#include "launch.h"

namespace a4w4 {

namespace {

constexpr int kRopeWarps = 4;
constexpr unsigned kAll = 0xFFFFFFFFu;

// f / (2 pi) modulo 1 as a 64-bit binary fraction: the 24-bit significand times
// 128 binary places of 1 / (2 pi) (a quarter of the first 130 of 2 / pi).
__device__ __forceinline__ unsigned long long turns_per_position(float f) {
  constexpr unsigned long long kHi = 0x28BE60DB9391054Aull, kLo = 0x7F09D5F47D4D3770ull;
  const uint32_t b = __float_as_uint(f), ex = b >> 23 & 255u;
  const unsigned long long m = (b & 0x7FFFFFu) | (ex ? 0x800000u : 0u);
  const int sh = static_cast<int>(ex ? ex : 1u) - 150;               // f = m 2^sh
  // m (kHi : kLo), 152 bits
  const unsigned long long p0 = m * kLo;
  unsigned long long p1 = m * kHi;
  const unsigned long long c = __umul64hi(m, kLo);
  unsigned long long p2 = __umul64hi(m, kHi);
  p1 += c;
  p2 += p1 < c;
  unsigned long long F;
  if (sh <= -128) F = 0ull;
  else if (sh <= -64) F = p2 >> (-sh - 64);
  else if (sh < 0) F = p1 >> -sh | p2 << (64 + sh);
  else if (sh == 0) F = p1;
  else if (sh < 64) F = p1 << sh | p0 >> (64 - sh);
  else F = sh < 128 ? p0 << (sh - 64) : 0ull;
  return b >> 31 ? 0ull - F : F;
}

struct Pair { float c, s; };

// E2M1 codes 0..7 of |y|, ties to the even code, in 64 bits.
__device__ __forceinline__ uint32_t e2m1_of(double y) {
  return (y > 0.25) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0);
}

// One warp's share of a token.
template <int D>
struct RopeWarp {
  static constexpr int LPH = D / 8, HPW = 32 / LPH;      // threads per head, heads at a time
  const RopeArgs& p;
  const int lane, d0, sub;                               // first dimension of this thread, head of the HPW
  const long long t;
  const Pair* s_pair;                                    // cos, sin of each pair's angle
  int partner;                                           // thread with the pairs' other halves (half split)
  bool rotated, second;                                  // whether d0 .. d0 + 7 turn; are second halves of their pairs

  __device__ __forceinline__ RopeWarp(const RopeArgs& args, long long token, const Pair* pairs)
      : p(args), lane(threadIdx.x & 31), d0(8 * (lane % LPH)), sub(lane / LPH), t(token), s_pair(pairs) {
    const int half = p.rot / 2;
    rotated = d0 < p.rot;
    second = !p.interleaved && d0 >= half;
    partner = !rotated || p.interleaved ? lane : second ? lane - half / 8 : lane + half / 8;
  }

  // Pair of dimension d0 + u.
  __device__ __forceinline__ int pair_of(int u) const {
    return p.interleaved ? (d0 + u) / 2 : second ? d0 + u - p.rot / 2 : d0 + u;
  }

  // A, B and the largest |w| of this thread's dimensions and of their partners'.
  __device__ __forceinline__ void coefficients(const float* w, float* A, float* B, float* wmax, float* pmax) const {
    *wmax = *pmax = 1.f;
    float own[8];
#pragma unroll
    for (int u = 0; u < 8; u += 4) {
      const float4 v = w != nullptr ? *reinterpret_cast<const float4*>(w + d0 + u) : make_float4(1.f, 1.f, 1.f, 1.f);
      own[u] = v.x; own[u + 1] = v.y; own[u + 2] = v.z; own[u + 3] = v.w;
    }
    const int other = second ? d0 - p.rot / 2 : d0 + p.rot / 2;       // half split only
    float pm = 0.f, om = 0.f;
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      float c = 1.f, s = 0.f, wp = 0.f;
      if (rotated) {
        const Pair a = s_pair[pair_of(u)];
        c = a.c;
        s = (p.interleaved ? (u & 1) != 0 : second) ? a.s : -a.s;
        wp = p.interleaved ? own[u ^ 1] : w != nullptr ? w[other + u] : 1.f;
      }
      A[u] = own[u] * c;
      B[u] = wp * s;
      om = fmaxf(om, fabsf(own[u]));
      pm = fmaxf(pm, fabsf(wp));
    }
    *wmax = om;
    *pmax = pm;
  }

  // Reciprocal of the root mean square of a head (over the LPH threads that hold it).
  __device__ __forceinline__ float norm(const uint4& x) const {
    float ssq = 0.f;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const float a = __uint_as_float(w[u] << 16), b = __uint_as_float(w[u] & 0xFFFF0000u);
      ssq = fmaf(a, a, fmaf(b, b, ssq));
    }
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ssq += __shfl_xor_sync(kAll, ssq, o);
    if (!(ssq < 1e38f)) return static_cast<float>(norm_64(x));   // the squares may have passed fp32's range
    return rsqrtf(ssq * (1.f / D) + p.eps);
  }
  // (a head's threads come here together)
  __device__ __noinline__ double norm_64(const uint4& x) const {
    const unsigned mask = LPH == 32 ? kAll : ((1u << LPH) - 1u) << (sub * LPH);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    double ssq = 0.0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const double a = __uint_as_float(w[u] << 16), b = __uint_as_float(w[u] & 0xFFFF0000u);
      ssq += a * a + b * b;
    }
#pragma unroll
    for (int o = LPH / 2; o > 0; o >>= 1) ssq += __shfl_xor_sync(mask, ssq, o);
    return 1.0 / sqrt(ssq / D + static_cast<double>(p.eps));
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

  __device__ __forceinline__ void rotate(const uint4& x, const uint4& y, const float* A, const float* B, float r,
                                         float* out) const {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w}, v[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      out[2 * u] = r * fmaf(A[2 * u], __uint_as_float(w[u] << 16), B[2 * u] * __uint_as_float(v[u] << 16));
      out[2 * u + 1] = r * fmaf(A[2 * u + 1], __uint_as_float(w[u] & 0xFFFF0000u),
                                B[2 * u + 1] * __uint_as_float(v[u] & 0xFFFF0000u));
    }
  }

  // Heads first, first + step, ... (in units of HPW) of H heads in x: to BF16 rows.
  __device__ __forceinline__ void to_rows(const uint16_t* x, uint16_t* out, int H, const float* w, int first, int step) const {
    if (first * HPW >= H) return;
    float A[8], B[8], wm, pm;
    coefficients(w, A, B, &wm, &pm);
    for (int g = first; g * HPW < H; g += step) {
      const int h = g * HPW + sub;
      const bool in = h < H;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (in) v = *reinterpret_cast<const uint4*>(x + h * D + d0);
      const float r = w != nullptr ? norm(v) : 1.f;
      const uint4 y = partners(v);
      float o[8];
      rotate(v, y, A, B, r, o);
      if (in)
        *reinterpret_cast<uint4*>(out + h * D + d0) =
            make_uint4(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]), pack_bf16(o[4], o[5]), pack_bf16(o[6], o[7]));
    }
  }

  // Codes and scale of a key head in 64 bits.
  __device__ __noinline__ uint32_t key_cells_64(const uint4& x, const uint4& y, const float* w, int position,
                                                uint32_t* code) const {
    const double r = w != nullptr ? norm_64(x) : 1.0;
    const uint32_t a[4] = {x.x, x.y, x.z, x.w}, b[4] = {y.x, y.y, y.z, y.w};
    double o[8], amax = 0.0;
    for (int u = 0; u < 8; ++u) {
      const double own = __uint_as_float(u & 1 ? a[u / 2] & 0xFFFF0000u : a[u / 2] << 16) * (w != nullptr ? w[d0 + u] : 1.0);
      o[u] = own;
      if (rotated) {
        const int other = p.interleaved ? d0 + (u ^ 1) : second ? d0 + u - p.rot / 2 : d0 + u + p.rot / 2;
        const double par = __uint_as_float(u & 1 ? b[u / 2] & 0xFFFF0000u : b[u / 2] << 16) * (w != nullptr ? w[other] : 1.0);
        const unsigned long long turn = static_cast<unsigned long long>(static_cast<long long>(position)) *
                                        turns_per_position(p.inv_freq[pair_of(u)]);
        double s, c;
        sincospi(static_cast<double>(static_cast<long long>(turn)) * 0x1p-63, &s, &c);
        o[u] = own * c + par * ((p.interleaved ? (u & 1) != 0 : second) ? s : -s);
      }
      o[u] *= r;
      amax = fmax(amax, fabs(o[u]));
    }
    const unsigned mask = LPH == 32 ? kAll : ((1u << LPH) - 1u) << (sub * LPH);
    amax = fmax(amax, __shfl_xor_sync(mask, amax, 1));
    amax = fmax(amax, __shfl_xor_sync(mask, amax, 2));
    // 2^(e - 127), e = floor(log2 amax) - 2 + 127, at least 0 and at most what an infinity gives
    const int ex = static_cast<int>(__double_as_longlong(amax) >> 52 & 2047) - 1023;
    const int e = min(max(ex - 2 + 127, 0), 253);
    const double unit = __longlong_as_double(static_cast<long long>(1023 + 127 - e) << 52);
    uint32_t c = 0u;
    for (int u = 0; u < 8; ++u) c |= (e2m1_of(fabs(o[u]) * unit) | (signbit(o[u]) ? 8u : 0u)) << (4 * u);
    *code = c;
    return static_cast<uint32_t>(e);
  }

  __device__ __forceinline__ uint8_t* chunk_of(int slot, int h) const {
    const int chunks = 1 << (p.page_lg - 4);
    return p.cache + kv_chunk_offset<D>(slot >> p.page_lg, h, (slot >> 4) & (chunks - 1), p.Hkv, chunks);
  }

  // The keys to the cache: quantised from the fp32 value.  Each value is known to
  // 2^-19 r (|w x| + |w_p x_p|) (2^-21.6 from the coefficients and products, 2^-20.7 from r,
  // two roundings); where that leaves a code or the scale open, 64 bits decide.
  __device__ __forceinline__ void keys_to_cache(const uint16_t* x, int slot, int position, int first, int step) const {
    using Ch = KvChunk<D>;
    if (first * HPW >= p.Hkv) return;
    float A[8], B[8], wm, pm;
    coefficients(p.k_weight, A, B, &wm, &pm);
    for (int g = first; g * HPW < p.Hkv; g += step) {
      const int h = g * HPW + sub;
      const bool in = h < p.Hkv;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (in) v = *reinterpret_cast<const uint4*>(x + h * D + d0);
      const float r = p.k_weight != nullptr ? norm(v) : 1.f;
      const uint4 y = partners(v);
      float o[8];
      rotate(v, y, A, B, r, o);
      float amax = 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) amax = fmaxf(amax, fabsf(o[u]));
      uint32_t mx = max_abs_bf16x2(max_abs_bf16x2(v.x, v.y), max_abs_bf16x2(v.z, v.w)) & 0x7FFF7FFFu;
      uint32_t my = max_abs_bf16x2(max_abs_bf16x2(y.x, y.y), max_abs_bf16x2(y.z, y.w)) & 0x7FFF7FFFu;
      const float bx = fmaxf(__uint_as_float(mx << 16), __uint_as_float(mx & 0xFFFF0000u));
      const float by = fmaxf(__uint_as_float(my << 16), __uint_as_float(my & 0xFFFF0000u));
      const bool zero = bx == 0.f && by == 0.f;
      float off = r * (bx * wm + by * pm) * 0x1p-19f + (zero ? 0.f : 0x1p-147f);
      amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 1));
      off = fmaxf(off, __shfl_xor_sync(kAll, off, 1));
      amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 2));
      off = fmaxf(off, __shfl_xor_sync(kAll, off, 2));
      const uint32_t eb = __float_as_uint(amax) >> 23;
      uint32_t e = eb > 2u ? eb - 2u : 0u;
      const float inv = __uint_as_float((254u - e) << 23), slack = off * inv;
      float lo[8], hi[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        lo[u] = fmaf(o[u], inv, -slack);
        hi[u] = fmaf(o[u], inv, slack);
      }
      uint32_t code = cvt_e2m1x8(lo[0], lo[1], lo[2], lo[3], lo[4], lo[5], lo[6], lo[7]);
      const uint32_t code_hi = cvt_e2m1x8(hi[0], hi[1], hi[2], hi[3], hi[4], hi[5], hi[6], hi[7]);
      const bool open = code != code_hi || __float_as_uint(amax - off) >> 23 != eb || __float_as_uint(amax + off) >> 23 != eb;
      if (__any_sync(kAll, open && off > 0.f)) e = key_cells_64(v, y, p.k_weight, position, &code);
      if (in) {
        uint8_t* chunk = chunk_of(slot, h);
        const int row = slot & 15;
        *reinterpret_cast<uint32_t*>(chunk + Ch::key_word(row, d0 / 32, d0 % 32 / 8)) = code;
        if (d0 % 32 == 0) chunk[Ch::kKeyScales + row * Ch::J + d0 / 32] = static_cast<uint8_t>(e);
      }
    }
  }

  __device__ __forceinline__ void values_to_cache(const uint16_t* x, int slot, int first, int step) const {
    using Ch = KvChunk<D>;
    for (int g = first; g * HPW < p.Hkv; g += step) {
      const int h = g * HPW + sub;
      const bool in = h < p.Hkv;
      uint4 v = make_uint4(0u, 0u, 0u, 0u);
      if (in) v = *reinterpret_cast<const uint4*>(x + h * D + d0);
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
      // Thread l has the bytes of run g = 4 (l % 2) .. + 3 at place i = l / 2; it writes four
      // places of one run: i0 .. i0 + 3 of run `run`.
      const int l = lane % LPH, run = D == 128 ? l / 2 : l, i0 = D == 128 ? 4 * (l & 1) : 0;
      uint32_t word = 0u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t c = __shfl_sync(kAll, code, sub * LPH + 2 * (i0 + i) + run / 4);
        word |= (c >> (8 * (run & 3)) & 255u) << (8 * i);
      }
      if (in) {
        uint8_t* chunk = chunk_of(slot, h);
        const int row = slot & 15;
        *reinterpret_cast<uint32_t*>(chunk + Ch::value_run(row, run) + i0) = word;
        if (d0 % 32 == 0) chunk[Ch::kValueScales + row * Ch::J + d0 / 32] = static_cast<uint8_t>(e);
      }
    }
  }
};

// A warp takes every `split`-th unit (256 / D heads) of one token: queries, keys, values one after the other.
template <int D, bool CACHE>
__global__ void __launch_bounds__(32 * kRopeWarps) kv_rope_kernel(const RopeArgs p) {
  __shared__ Pair s_pair[kRopeWarps][D / 2];
  griddep_wait();
  griddep_launch_dependents();
  constexpr int HPW = RopeWarp<D>::HPW;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long item = static_cast<long long>(blockIdx.x) * kRopeWarps + warp;
  const long long t = item / p.split;
  const int s = static_cast<int>(item - t * p.split);
  if (t >= p.T) return;
  int slot = 0;
  if (CACHE) {
    slot = p.slot_map[t];
    if (static_cast<unsigned>(slot) >= static_cast<unsigned>(p.slots)) return;
  }
  const int position = p.rot > 0 ? p.positions[t] : 0;
  for (int i = lane; i < p.rot / 2; i += 32) {
    const unsigned long long turn =
        static_cast<unsigned long long>(static_cast<long long>(position)) * turns_per_position(p.inv_freq[i]);
    // the upper half as a signed fraction of half a turn, [-1, 1)
    const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;
    Pair a;
    sincospif(x, &a.s, &a.c);
    s_pair[warp][i] = a;
  }
  __syncwarp();
  const RopeWarp<D> rw(p, t, s_pair[warp]);
  const int uq = (p.Hq + HPW - 1) / HPW, uk = (p.Hkv + HPW - 1) / HPW;
  // first unit of each kind that falls to this warp
  const int fk = ((s - uq) % p.split + p.split) % p.split, fv = ((s - uq - uk) % p.split + p.split) % p.split;
  rw.to_rows(p.q + t * p.q_stride, p.q_out + t * p.q_out_stride, p.Hq, p.q_weight, s, p.split);
  if (CACHE) {
    rw.keys_to_cache(p.k + t * p.k_stride, slot, position, fk, p.split);
    rw.values_to_cache(p.v + t * p.v_stride, slot, fv, p.split);
  } else {
    rw.to_rows(p.k + t * p.k_stride, p.k_out + t * p.k_out_stride, p.Hkv, p.k_weight, fk, p.split);
  }
}

}  // namespace

int launch_kv_rope(RopeArgs p, int D, cudaStream_t st, int sms) {
  const bool cache = p.cache != nullptr;
  const int per = 256 / D, units = (p.Hq + per - 1) / per + (cache ? 2 : 1) * ((p.Hkv + per - 1) / per);
  // warps enough for 16 on every SM, each with whole units
  const long long want = (16ll * sms + p.T - 1) / p.T;
  p.split = static_cast<int>(want < 1 ? 1 : want > units ? units : want);
  const long long grid = (static_cast<long long>(p.T) * p.split + kRopeWarps - 1) / kRopeWarps;
  if (grid > INT32_MAX) return -1;
  auto kern = D == 64 ? (cache ? kv_rope_kernel<64, true> : kv_rope_kernel<64, false>)
                      : (cache ? kv_rope_kernel<128, true> : kv_rope_kernel<128, false>);
  return launch_pdl(kern, static_cast<int>(grid), 32 * kRopeWarps, st, p);
}

}  // namespace a4w4
