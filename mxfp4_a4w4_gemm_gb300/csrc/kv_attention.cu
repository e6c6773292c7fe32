// kv_attention.cu -- causal attention of the newest tokens over the paged MXFP4
// cache (include/a4w4.h).
#include "device.cuh"
#include "kv.cuh"
#include "kv_walk.cuh"
#include "launch.h"

#include <cmath>

namespace a4w4 {

namespace {

// E2M1 magnitude bits and sign of nibble n (0..15) as float.
__device__ __forceinline__ float e2m1(uint32_t n) {
  constexpr float kMag[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
  const float m = kMag[n & 7u];
  return n & 8u ? -m : m;
}
__device__ __forceinline__ float e8m0(uint32_t e) {
  return e == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23);
}

// One CTA of 128 threads per query row and head: 128 keys at a time, a key per
// thread for the scores, a dimension per thread for the output.
template <int D>
__global__ void __launch_bounds__(128) kv_attention_rows_kernel(const KvAttentionArgs p) {
  using Ch = KvChunk<D>;
  __shared__ float s_q[D], s_p[128], s_red[4];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, b = blockIdx.z, hq = blockIdx.y, i = blockIdx.x;
  const KvRequest rq = kv_request(p, b);
  if (i >= rq.rows) return;
  const long long row = static_cast<long long>(rq.row0) + i;
  const int seen = max(0, rq.len - rq.all + i + 1);
  const int h = hq / (p.Hq / p.Hkv);
  for (int d = tid; d < D; d += 128)
    s_q[d] = __uint_as_float(static_cast<uint32_t>(p.q[row * p.q_stride + hq * D + d]) << 16) * p.sm_scale;
  float m = -INFINITY, l = 0.f, o = 0.f;
  for (int k0 = 0; k0 < seen; k0 += 128) {
    __syncthreads();
    const int tok = k0 + tid;
    float x = -INFINITY;
    if (tok < seen) {
      const int page = max(0, min(p.block_table[static_cast<long long>(b) * p.max_pages + tok / p.page_size], p.num_pages - 1));
      const uint8_t* ch = p.cache + kv_chunk_offset<D>(page, h, tok % p.page_size / 16, p.Hkv, p.page_size / 16);
      x = 0.f;
      for (int j = 0; j < Ch::J; ++j) {
        float a = 0.f;
        for (int t = 0; t < 4; ++t) {
          const uint32_t w = *reinterpret_cast<const uint32_t*>(ch + Ch::key_word(tok % 16, j, t));
          for (int u = 0; u < 8; ++u) a += s_q[32 * j + 8 * t + u] * e2m1(w >> (4 * u));
        }
        x += a * e8m0(ch[Ch::kKeyScales + tok % 16 * Ch::J + j]);
      }
    }
    float mx = x;
    for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, s));
    if (tid % 32 == 0) s_red[tid / 32] = mx;
    __syncthreads();
    mx = fmaxf(m, fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3])));
    const float pr = expf(x - mx);
    s_p[tid] = pr;
    const float f = expf(m - mx);
    m = mx;
    float sum = pr;
    for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
    __syncthreads();
    if (tid % 32 == 0) s_red[tid / 32] = sum;
    __syncthreads();
    l = l * f + s_red[0] + s_red[1] + s_red[2] + s_red[3];
    o *= f;
    if (tid < D) {
      for (int u = 0; u < min(128, seen - k0); ++u) {
        const int tk = k0 + u;
        const int page = max(0, min(p.block_table[static_cast<long long>(b) * p.max_pages + tk / p.page_size], p.num_pages - 1));
        const uint8_t* ch = p.cache + kv_chunk_offset<D>(page, h, tk % p.page_size / 16, p.Hkv, p.page_size / 16);
        const uint32_t byte = ch[Ch::value_run(tk % 16, tid % 16 / 2) + tid / 16];
        o += s_p[u] * e2m1(byte >> (tid % 2 * 4)) * e8m0(ch[Ch::kValueScales + tk % 16 * Ch::J + tid / 32]);
      }
    }
  }
  if (tid < D) {
    const float y = l > 0.f ? o / l : l == 0.f ? 0.f : l;
    p.out[(row * p.Hq + hq) * D + tid] = __bfloat16_as_ushort(__float2bfloat16_rn(y));
  }
  if (tid == 0 && p.lse != nullptr) p.lse[row * p.Hq + hq] = l == 0.f ? -INFINITY : m + logf(l);
}

}  // namespace

size_t kv_attention_ws_bytes(int max_q, int group, int D, int sms) {
  return kv_decode_ws_bytes(max_q <= 16 / group ? max_q * group : 16, D, sms);
}

int launch_kv_attention(const KvAttentionArgs& p, int D, cudaStream_t st, int sms) {
  if (p.max_q <= 16 / (p.Hq / p.Hkv)) return launch_kv_decode(p, D, st, sms);
  const dim3 grid(p.max_q, p.Hq, p.B);
  if (D == 64) kv_attention_rows_kernel<64><<<grid, 128, 0, st>>>(p);
  else kv_attention_rows_kernel<128><<<grid, 128, 0, st>>>(p);
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace a4w4
