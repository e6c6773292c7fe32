// kv.cu -- the paged MXFP4 key/value cache: the step's block tables and slots
// (kv_plan_kernel), the cache's writer (kv_append_kernel) and reader
// (kv_read_kernel).  Layout and rules: include/a4w4.h.
#include "device.cuh"
#include "kv.cuh"
#include "launch.h"

namespace a4w4 {

namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxB = 4096;
constexpr int kPlanPer = kPlanMaxB / kPlanThreads;   // requests per thread of the scan

struct PlanArgs {
  const int32_t *past_lens, *new_lens;
  int B, page_size, max_pages, ring_size, max_tokens;
  int32_t *block_table, *free_ring;
  const int32_t* ring_state;
  int32_t *ring_state_out, *kv_lens, *cu_new, *slot_map, *positions, *refused;
};

// Number of entries of a[0 .. n-1] (non-decreasing) that are <= x, minus one:
// the request whose run of a prefix sum holds x.
__device__ __forceinline__ int run_of(const int* a, int n, int x) {
  int lo = 0, hi = n;                       // a[lo] <= x < a[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x) lo = mid; else hi = mid;
  }
  return lo;
}

__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xFFFFFFFFu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

// Three prefix sums over the requests (tokens wanted, pages needed, pages given
// back) decide everything; the rest is one independent lookup per output.  Every
// CTA forms the sums for itself (B <= 4096: at most 32 KB from L2), which costs
// less than a second launch or a grid-wide wait, and then writes its share of
// the outputs.  No output is read: table entries of held pages and ring entries
// of free pages are not written by this call.
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanArgs p) {
  __shared__ int s_tok[kPlanMaxB + 1], s_page[kPlanMaxB + 1], s_back[kPlanMaxB + 1];
  __shared__ long long s_warp[3][kPlanThreads / 32];
  __shared__ int s_last[2], s_refused;
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = p.B, ps = p.page_size;
  const int head = p.ring_state[0], count = p.ring_state[1];
  if (tid < 2) s_last[tid] = 0;
  if (tid == 2) s_refused = 0;
  const int per = (B + kPlanThreads - 1) / kPlanThreads;
  const long long room = static_cast<long long>(p.max_pages) * ps;
  long long tok[kPlanPer], page[kPlanPer], back[kPlanPer];   // inclusive within the thread
  long long at = 0, ap = 0, ab = 0;
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    const int b = tid * per + i;
    if (i < per && b < B) {
      const long long past = p.past_lens[b], nw = p.new_lens[b];
      const long long want = nw > 0 && past + nw <= room ? nw : 0;
      const long long held = (past + ps - 1) / ps;
      at += want;
      ap += (past + want + ps - 1) / ps - held;
      ab += nw < 0 ? held : 0;
    }
    tok[i] = at; page[i] = ap; back[i] = ab;
  }
  const long long wt = warp_scan(at, lane), wp = warp_scan(ap, lane), wb = warp_scan(ab, lane);
  if (lane == 31) { s_warp[0][warp] = wt; s_warp[1][warp] = wp; s_warp[2][warp] = wb; }
  __syncthreads();
  long long bt = wt - at, bp = wp - ap, bb = wb - ab;
  for (int w = 0; w < warp; ++w) { bt += s_warp[0][w]; bp += s_warp[1][w]; bb += s_warp[2][w]; }
  // the sums only grow, so the requests that fit are those before the first that does not
  int last_t = 0, last_p = 0;
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    if (i < per && tid * per + i < B && bt + tok[i] <= p.max_tokens && bp + page[i] <= count) {
      last_t = static_cast<int>(bt + tok[i]);
      last_p = static_cast<int>(bp + page[i]);
    }
  }
  if (last_t > 0) atomicMax(&s_last[0], last_t);
  if (last_p > 0) atomicMax(&s_last[1], last_p);
  __syncthreads();
  const int T = s_last[0], N = s_last[1];
  int refused = 0;
#pragma unroll
  for (int i = 0; i < kPlanPer; ++i) {
    const int b = tid * per + i;
    if (i < per && b < B) {
      const bool fits = bt + tok[i] <= p.max_tokens && bp + page[i] <= count;
      s_tok[b + 1] = fits ? static_cast<int>(bt + tok[i]) : T;
      s_page[b + 1] = fits ? static_cast<int>(bp + page[i]) : N;
      s_back[b + 1] = static_cast<int>(bb + back[i]);
      const long long before = i > 0 ? tok[i - 1] : 0;
      if (p.new_lens[b] > 0 && (!fits || tok[i] == before)) ++refused;
    }
  }
  if (tid == 0) { s_tok[0] = 0; s_page[0] = 0; s_back[0] = 0; }
  if (refused > 0) atomicAdd(&s_refused, refused);
  __syncthreads();
  const int R = s_back[B];
  if (blockIdx.x == 0 && tid == 0) {
    p.ring_state_out[0] = static_cast<int>((static_cast<long long>(head) + N) % p.ring_size);
    p.ring_state_out[1] = count - N + R;
    p.refused[0] = s_refused;
    p.cu_new[0] = 0;
  }
  const int step = gridDim.x * kPlanThreads, first = blockIdx.x * kPlanThreads + tid;
  for (int b = first; b < B; b += step) {
    p.cu_new[b + 1] = s_tok[b + 1];
    p.kv_lens[b] = p.new_lens[b] < 0 ? 0 : p.past_lens[b] + s_tok[b + 1] - s_tok[b];
  }
  for (int i = first; i < N; i += step) {             // pages taken from the ring
    const int b = run_of(s_page, B, i);
    const int held = (p.past_lens[b] + ps - 1) / ps;
    p.block_table[static_cast<long long>(b) * p.max_pages + held + i - s_page[b]] =
        p.free_ring[(static_cast<long long>(head) + i) % p.ring_size];
  }
  for (int i = first; i < R; i += step) {             // pages given back
    const int b = run_of(s_back, B, i);
    p.free_ring[(static_cast<long long>(head) + count + i) % p.ring_size] =
        p.block_table[static_cast<long long>(b) * p.max_pages + i - s_back[b]];
  }
  for (int i = first; i < p.max_tokens; i += step) {
    int slot = -1, pos = 0;
    if (i < T) {
      const int b = run_of(s_tok, B, i);
      const int past = p.past_lens[b], held = (past + ps - 1) / ps;
      pos = past + i - s_tok[b];
      const int pg = pos / ps;
      const int id = pg < held ? p.block_table[static_cast<long long>(b) * p.max_pages + pg]
                               : p.free_ring[(static_cast<long long>(head) + s_page[b] + pg - held) % p.ring_size];
      slot = id * ps + pos % ps;
    }
    p.slot_map[i] = slot;
    p.positions[i] = pos;
  }
}

// One thread per 32-block of one token and head.
template <int D>
__global__ void __launch_bounds__(256) kv_append_kernel(const uint16_t* __restrict__ k, long long k_stride,
                                                        const uint16_t* __restrict__ v, long long v_stride,
                                                        const int32_t* __restrict__ slot_map, int T, int Hkv,
                                                        uint8_t* __restrict__ cache, int slots, int page_size) {
  using Ch = KvChunk<D>;
  griddep_wait();
  griddep_launch_dependents();
  const int blocks = Hkv * Ch::J;                     // per token, for keys and again for values
  const long long total = 2ll * T * blocks;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
    const long long row = i / blocks;
    const int hj = static_cast<int>(i - row * blocks), h = hj / Ch::J, j = hj % Ch::J;
    const bool is_v = row >= T;
    const long long t = is_v ? row - T : row;
    const int slot = slot_map[t];
    if (static_cast<unsigned>(slot) >= static_cast<unsigned>(slots)) continue;
    const uint16_t* src = (is_v ? v + t * v_stride : k + t * k_stride) + hj * 32;
    uint32_t w[16], c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint4 x = ld_global_nc_v4(src + 8 * u);
      w[4 * u] = x.x; w[4 * u + 1] = x.y; w[4 * u + 2] = x.z; w[4 * u + 3] = x.w;
    }
    const uint32_t e = quant32_bf16(w, c);
    const int page = slot / page_size, r = slot % 16, ch = slot % page_size / 16;
    uint8_t* chunk = cache + kv_chunk_offset<D>(page, h, ch, Hkv, page_size / 16);
    if (!is_v) {
#pragma unroll
      for (int u = 0; u < 4; ++u) *reinterpret_cast<uint32_t*>(chunk + Ch::key_word(r, j, u)) = c[u];
      chunk[Ch::kKeyScales + r * Ch::J + j] = static_cast<uint8_t>(e);
    } else {
      // byte g of each half block 16 i belongs to run g, at i
#pragma unroll
      for (int g = 0; g < 8; ++g) {
        const uint32_t lo = c[g / 4] >> (8 * (g % 4)) & 0xFFu, hi = c[2 + g / 4] >> (8 * (g % 4)) & 0xFFu;
        *reinterpret_cast<uint16_t*>(chunk + Ch::value_run(r, g) + 2 * j) = static_cast<uint16_t>(lo | hi << 8);
      }
      chunk[Ch::kValueScales + r * Ch::J + j] = static_cast<uint8_t>(e);
    }
  }
}

// Two E2M1 codes of a byte times 2^(e - 127), as BF16x2 (exact).
__device__ __forceinline__ uint32_t e2m1x2_to_bf16x2(uint32_t byte, uint32_t e) {
  constexpr float kMag[8] = {0.f, 0.5f, 1.f, 1.5f, 2.f, 3.f, 4.f, 6.f};
  const float s = e == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(e << 23);
  const float a = kMag[byte & 7u] * s, b = kMag[byte >> 4 & 7u] * s;
  const uint32_t ua = __float_as_uint(a) | (byte & 8u) << 28, ub = __float_as_uint(b) | (byte & 0x80u) << 24;
  return ua >> 16 | (ub & 0xFFFF0000u);
}

// One thread per 32-block of one token and head.
template <int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const uint8_t* __restrict__ cache, int slots, int page_size,
                                                      const int32_t* __restrict__ slot_map, int T, int Hkv,
                                                      uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  using Ch = KvChunk<D>;
  griddep_wait();
  griddep_launch_dependents();
  const int blocks = Hkv * Ch::J;
  const long long total = 2ll * T * blocks;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += stride) {
    const long long row = i / blocks;
    const int hj = static_cast<int>(i - row * blocks), h = hj / Ch::J, j = hj % Ch::J;
    const bool is_v = row >= T;
    const long long t = is_v ? row - T : row;
    const int slot = slot_map[t];
    uint32_t o[16];
#pragma unroll
    for (int u = 0; u < 16; ++u) o[u] = 0u;
    if (static_cast<unsigned>(slot) < static_cast<unsigned>(slots)) {
      const int page = slot / page_size, r = slot % 16, ch = slot % page_size / 16;
      const uint8_t* chunk = cache + kv_chunk_offset<D>(page, h, ch, Hkv, page_size / 16);
      const uint32_t e = chunk[(is_v ? Ch::kValueScales : Ch::kKeyScales) + r * Ch::J + j];
#pragma unroll
      for (int u = 0; u < 16; ++u) {
        const uint32_t byte = is_v ? chunk[Ch::value_run(r, u % 8) + 2 * j + u / 8] : chunk[Ch::key_word(r, j, u / 4) + u % 4];
        o[u] = e2m1x2_to_bf16x2(byte, e);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>((is_v ? v : k) + t * blocks * 32 + hj * 32);
#pragma unroll
    for (int u = 0; u < 4; ++u) dst[u] = make_uint4(o[4 * u], o[4 * u + 1], o[4 * u + 2], o[4 * u + 3]);
  }
}

int grid_for(long long items, int per_cta, int most) {
  const long long g = (items + per_cta - 1) / per_cta;
  return static_cast<int>(g < 1 ? 1 : g > most ? most : g);
}

}  // namespace

int launch_kv_plan(const int32_t* past_lens, const int32_t* new_lens, int B, int page_size, int32_t* block_table,
                   int max_pages, int32_t* free_ring, int ring_size, const int32_t* ring_state,
                   int32_t* ring_state_out, int32_t* kv_lens, int32_t* cu_new, int32_t* slot_map, int32_t* positions,
                   int max_tokens, int32_t* refused, cudaStream_t st, int sms) {
  const PlanArgs p{past_lens, new_lens, B, page_size, max_pages, ring_size, max_tokens, block_table, free_ring,
                   ring_state, ring_state_out, kv_lens, cu_new, slot_map, positions, refused};
  const int grid = grid_for(static_cast<long long>(max_tokens) + 2ll * B, 2 * kPlanThreads, sms);
  return launch_pdl(kv_plan_kernel, grid, kPlanThreads, st, p);
}

int launch_kv_append(const void* k, long long k_stride, const void* v, long long v_stride, const int32_t* slot_map,
                     int T, int Hkv, int D, void* cache, int num_pages, int page_size, cudaStream_t st, int sms) {
  const int grid = grid_for(2ll * T * Hkv * (D / 32), 256, sms * 8);
  return launch_pdl(D == 64 ? kv_append_kernel<64> : kv_append_kernel<128>, grid, 256, st,
                    static_cast<const uint16_t*>(k), k_stride, static_cast<const uint16_t*>(v), v_stride, slot_map, T,
                    Hkv, static_cast<uint8_t*>(cache), num_pages * page_size, page_size);
}

int launch_kv_read(const void* cache, int num_pages, int page_size, const int32_t* slot_map, int T, int Hkv, int D,
                   void* k, void* v, cudaStream_t st, int sms) {
  const int grid = grid_for(2ll * T * Hkv * (D / 32), 256, sms * 8);
  return launch_pdl(D == 64 ? kv_read_kernel<64> : kv_read_kernel<128>, grid, 256, st,
                    static_cast<const uint8_t*>(cache), num_pages * page_size, page_size, slot_map, T, Hkv,
                    static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
}

}  // namespace a4w4
