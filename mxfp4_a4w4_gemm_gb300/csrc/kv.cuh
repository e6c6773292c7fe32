// kv.cuh -- byte layout of the paged MXFP4 key/value cache (include/a4w4.h), and the
// conversions and short operations that its kernels share.
#pragma once

#include <cstdint>

namespace a4w4 {

// One chunk: 16 tokens of one key/value head.  kBytes is a multiple of 16 and
// every part starts on a 16-byte boundary, so a run of chunks is one bulk copy.
template <int D>
struct KvChunk {
  static_assert(D == 64 || D == 128, "head size");
  static constexpr int J = D / 32;             // 32-blocks of a row
  static constexpr int kKeyScales = 8 * D;
  static constexpr int kValues = kKeyScales + 16 * J;
  static constexpr int kValueScales = kValues + 8 * D;
  static constexpr int kBytes = 17 * D;
  static_assert(kValueScales + 16 * J == kBytes && kBytes % 16 == 0 && kValues % 16 == 0, "chunk");

  // word t (dimensions 32 j + 8 t ..+7) of key block j of token r
  __host__ __device__ static constexpr int key_word(int r, int j, int t) { return r * (D / 2) + (t * J + j) * 4; }
  // the D / 16 bytes of token r's dimensions 16 i + 2 g, 16 i + 2 g + 1, i = 0 .. D / 16 - 1
  __host__ __device__ static constexpr int value_run(int r, int g) {
    return kValues + (r / 8) * 4 * D + (g * 4 + r % 8 / 2) * (D / 8) + (r % 2) * (D / 16);
  }
};

// First byte of chunk `c` of head `h` of page `p`.
template <int D>
__host__ __device__ __forceinline__ long long kv_chunk_offset(long long p, int h, int c, int Hkv, int chunks) {
  return ((p * Hkv + h) * chunks + c) * KvChunk<D>::kBytes;
}

constexpr float kNoMax = -3.0e38f;            // running maximum before the first key

__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The four bytes of w, each two E2M1 codes, as FP16x2 (low nibble in the low half).
__device__ __forceinline__ void e2m1x8_to_f16x2(uint32_t w, uint32_t* o) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]) : "r"(w));
}
// 2^k as a float, k in [-149, 127] (zero below).
__device__ __forceinline__ float pow2i(int k) {
  return k >= -126 ? __uint_as_float(static_cast<uint32_t>(k + 127) << 23)
                   : k >= -149 ? __uint_as_float(1u << (k + 149)) : 0.f;
}
// 2^k as a float, k in [-126, 127] only: one instruction less in a loop
__device__ __forceinline__ float pow2i_normal(int k) { return __uint_as_float(static_cast<uint32_t>(k + 127) << 23); }

}  // namespace a4w4
