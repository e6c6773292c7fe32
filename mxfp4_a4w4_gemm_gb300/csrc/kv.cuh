// kv.cuh -- byte layout of the paged MXFP4 key/value cache (include/a4w4.h).
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

}  // namespace a4w4
