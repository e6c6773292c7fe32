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
// of free pages are not written by this call.  Bound by latency: lengths, sums,
// search, page number, one after the other: 8 requests 3.9 us.  2000 requests with
// 128000 tokens 7.9 us: to the same trips come the arithmetic of four requests and two
// tokens a thread (64-bit sums, of which 20 bytes spill, divisions by page_size and
// ring_size), which was not timed apart (one token per thread in twice the CTAs 9.1 where
// two took 7.5, CTAs of 1024 threads 8.3).
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
      ab += nw < 0 ? min(held, static_cast<long long>(p.max_pages)) : 0;   // a row holds no more
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
  for (uint32_t u = first; u < static_cast<uint32_t>(p.max_tokens); u += step) {   // the last stride may pass 2^31
    const int i = static_cast<int>(u);
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

// Thread -> (token, head, 32-block) of the append and read kernels: a warp takes
// one head of 32 / J consecutive tokens.  New tokens mostly follow one another
// in a page, so that the warp's pieces of a chunk lie side by side (32 / J tokens
// x 2 J bytes of every value run) while each token's BF16 row is still touched in
// runs of 64 J bytes.
template <int D>
struct RowItem {
  static constexpr int J = D / 32, TOK = 32 / J;
  int t, h, j;
  __device__ __forceinline__ RowItem(int Hkv) {
    const int lane = threadIdx.x & 31;
    const long long wid = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
    const int group = static_cast<int>(wid / Hkv);
    h = static_cast<int>(wid - static_cast<long long>(group) * Hkv);
    j = lane % J;
    t = group * TOK + lane / J;
  }
};

// A warp's rows as 128 pieces of 16 bytes: piece o belongs to lane o / 4's
// 32-block and lies at 4 l + (o ^ l / 2) % 4, without bank conflicts whether lanes
// take pieces in order (whole rows, as global memory wants them) or four of their own.
__device__ __forceinline__ int row_piece(int l, int u) { return 4 * l + (u ^ (l >> 1 & 3)); }

// 16 bytes, global -> shared memory.
__device__ __forceinline__ void copy16(uint4* dst, const uint16_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" :: "r"(smem_u32(dst)), "l"(src) : "memory");
}

// Quantises one 32-block of a token's keys and the same one of its values: 128
// bytes read, 34 written.  8191 tokens x 8 heads of 128: 8.4 us alone, with buffers
// beyond L2 in turn (5.1 TB/s, 75% of the copy rate), 33.3 for 40000 tokens (6.2 TB/s,
// 92%): 32 KB of shared memory let six CTAs on an SM, so that the 1024 CTAs of 8191
// tokens are a wave and an eighth.  With the reader after it 16.3 us; over the same
// buffers again and again, whose cells the reader then finds in L2, 12.0 (there 15.0 when
// the rows reach shared memory by way of registers, 16.9 when every thread loads its own
// 64 bytes).
template <int D>
__global__ void __launch_bounds__(256) kv_append_kernel(const uint16_t* __restrict__ k, long long k_stride,
                                                        const uint16_t* __restrict__ v, long long v_stride,
                                                        const int32_t* __restrict__ slot_map, int T, int Hkv,
                                                        uint8_t* __restrict__ cache, int slots, int page_lg) {
  using Ch = KvChunk<D>;
  __shared__ uint4 s_row[8][2][128];
  griddep_wait();
  griddep_launch_dependents();
  const RowItem<D> it(Hkv);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = it.j;
  const int slot = it.t < T ? slot_map[it.t] : -1;
  const int t0 = it.t - lane / RowItem<D>::J;                 // the warp's first token
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int o = s * 32 + lane, l = o >> 2, t = t0 + l / RowItem<D>::J;
    if (t >= T) break;
    const int at = it.h * D + 32 * (l % RowItem<D>::J) + 8 * (o & 3);
    copy16(&s_row[warp][0][row_piece(l, o & 3)], k + t * k_stride + at);
    copy16(&s_row[warp][1][row_piece(l, o & 3)], v + t * v_stride + at);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  if (static_cast<unsigned>(slot) >= static_cast<unsigned>(slots)) return;
  uint32_t w[16], c[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint4 x = s_row[warp][0][row_piece(lane, u)];
    w[4 * u] = x.x; w[4 * u + 1] = x.y; w[4 * u + 2] = x.z; w[4 * u + 3] = x.w;
  }
  const int r = slot & 15, chunks = 1 << (page_lg - 4);
  uint8_t* chunk = cache + kv_chunk_offset<D>(slot >> page_lg, it.h, (slot >> 4) & (chunks - 1), Hkv, chunks);
  const uint32_t ek = quant32_bf16(w, c);
#pragma unroll
  for (int u = 0; u < 4; ++u) *reinterpret_cast<uint32_t*>(chunk + Ch::key_word(r, j, u)) = c[u];
  chunk[Ch::kKeyScales + r * Ch::J + j] = static_cast<uint8_t>(ek);
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const uint4 x = s_row[warp][1][row_piece(lane, u)];
    w[4 * u] = x.x; w[4 * u + 1] = x.y; w[4 * u + 2] = x.z; w[4 * u + 3] = x.w;
  }
  const uint32_t ev = quant32_bf16(w, c);
  // byte g of each half block 16 i belongs to run g, at i = 2 j, 2 j + 1
#pragma unroll
  for (int g = 0; g < 8; ++g)
    *reinterpret_cast<uint16_t*>(chunk + Ch::value_run(r, g) + 2 * j) =
        static_cast<uint16_t>(__byte_perm(c[g / 4], c[2 + g / 4], (g % 4) | (4 + g % 4) << 4));
  chunk[Ch::kValueScales + r * Ch::J + j] = static_cast<uint8_t>(ev);
}

// Eight E2M1 codes (nibble n of w) times 2^(e - 127) -> eight BF16, exact:
// magnitude bits placed at 6..8 of a BF16 and the sign at 15 read as the value
// times 2^-126; the scale follows in two multiplies by powers of two.
__device__ __forceinline__ uint4 e2m1x8_to_bf16x8(uint32_t w, uint32_t e) {
  constexpr uint32_t kMag = 0x01C001C0u, kSign = 0x80008000u;
  const uint32_t f = max(e << 7, 0x40u) * 0x00010001u;                // 2^(e - 127)
  uint32_t o[4];                                                       // elements (n, n + 4)
  o[0] = ((w << 6) & kMag) | ((w << 12) & kSign);
  o[1] = ((w << 2) & kMag) | ((w << 8) & kSign);
  o[2] = ((w >> 2) & kMag) | ((w << 4) & kSign);
  o[3] = ((w >> 6) & kMag) | (w & kSign);
#pragma unroll
  for (int n = 0; n < 4; ++n) o[n] = mul_bf16x2(mul_bf16x2(o[n], 0x7E807E80u), f);
  return make_uint4(__byte_perm(o[0], o[1], 0x5410), __byte_perm(o[2], o[3], 0x5410), __byte_perm(o[0], o[1], 0x7632),
                    __byte_perm(o[2], o[3], 0x7632));
}

// The inverse: 34 bytes read, 128 written.  Bound by HBM in long runs.  A thread's 64 bytes of a row
// go out by way of shared memory, so that a warp's stores write whole rows (16-byte
// stores 64 bytes apart touch every 32-byte sector twice): 40000 tokens x 8 heads of
// 128 36.6 us, 5.7 TB/s; stored directly 55.5.
template <int D>
__global__ void __launch_bounds__(256) kv_read_kernel(const uint8_t* __restrict__ cache, int slots, int page_lg,
                                                      const int32_t* __restrict__ slot_map, int T, int Hkv,
                                                      uint16_t* __restrict__ k, uint16_t* __restrict__ v) {
  using Ch = KvChunk<D>;
  __shared__ uint4 s_row[8][2][128];
  griddep_wait();
  griddep_launch_dependents();
  const RowItem<D> it(Hkv);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, j = it.j;
  const int slot = it.t < T ? slot_map[it.t] : -1;
  uint32_t wk[4] = {0u, 0u, 0u, 0u}, wv[4] = {0u, 0u, 0u, 0u}, ek = 0u, ev = 0u;
  if (static_cast<unsigned>(slot) < static_cast<unsigned>(slots)) {
    const int r = slot & 15, chunks = 1 << (page_lg - 4);
    const uint8_t* chunk = cache + kv_chunk_offset<D>(slot >> page_lg, it.h, (slot >> 4) & (chunks - 1), Hkv, chunks);
    uint32_t b[8];
#pragma unroll
    for (int u = 0; u < 4; ++u) wk[u] = *reinterpret_cast<const uint32_t*>(chunk + Ch::key_word(r, j, u));
#pragma unroll
    for (int g = 0; g < 8; ++g) b[g] = *reinterpret_cast<const uint16_t*>(chunk + Ch::value_run(r, g) + 2 * j);
    ek = chunk[Ch::kKeyScales + r * Ch::J + j];
    ev = chunk[Ch::kValueScales + r * Ch::J + j];
    // low bytes: dimensions 0..15 of the block, high bytes: 16..31
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const uint32_t p01 = __byte_perm(b[4 * q], b[4 * q + 1], 0x5140), p23 = __byte_perm(b[4 * q + 2], b[4 * q + 3], 0x5140);
      wv[q] = __byte_perm(p01, p23, 0x5410);
      wv[2 + q] = __byte_perm(p01, p23, 0x7632);
    }
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    s_row[warp][0][row_piece(lane, u)] = e2m1x8_to_bf16x8(wk[u], ek);
    s_row[warp][1][row_piece(lane, u)] = e2m1x8_to_bf16x8(wv[u], ev);
  }
  __syncwarp();
  const int t0 = it.t - lane / RowItem<D>::J;                 // the warp's first token
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int o = s * 32 + lane, l = o >> 2, t = t0 + l / RowItem<D>::J;
    if (t >= T) break;
    const long long at = (static_cast<long long>(t) * Hkv + it.h) * D + 32 * (l % RowItem<D>::J) + 8 * (o & 3);
    *reinterpret_cast<uint4*>(k + at) = s_row[warp][0][row_piece(l, o & 3)];
    *reinterpret_cast<uint4*>(v + at) = s_row[warp][1][row_piece(l, o & 3)];
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

namespace {

// CTAs of 256 threads for T tokens, Hkv heads, J blocks (RowItem); -1: too many.
int row_grid(int T, int Hkv, int D) {
  const int tok = 32 / (D / 32);
  const long long warps = (static_cast<long long>(T) + tok - 1) / tok * Hkv;
  const long long g = (warps + 7) / 8;
  return g > INT32_MAX ? -1 : static_cast<int>(g);
}

int log2_of(int page_size) { return page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7; }

}  // namespace

int launch_kv_append(const void* k, long long k_stride, const void* v, long long v_stride, const int32_t* slot_map,
                     int T, int Hkv, int D, void* cache, int num_pages, int page_size, cudaStream_t st) {
  const int grid = row_grid(T, Hkv, D);
  if (grid < 0) return -1;
  return launch_pdl(D == 64 ? kv_append_kernel<64> : kv_append_kernel<128>, grid, 256, st,
                    static_cast<const uint16_t*>(k), k_stride, static_cast<const uint16_t*>(v), v_stride, slot_map, T,
                    Hkv, static_cast<uint8_t*>(cache), num_pages * page_size, log2_of(page_size));
}

int launch_kv_read(const void* cache, int num_pages, int page_size, const int32_t* slot_map, int T, int Hkv, int D,
                   void* k, void* v, cudaStream_t st) {
  const int grid = row_grid(T, Hkv, D);
  if (grid < 0) return -1;
  return launch_pdl(D == 64 ? kv_read_kernel<64> : kv_read_kernel<128>, grid, 256, st,
                    static_cast<const uint8_t*>(cache), num_pages * page_size, log2_of(page_size), slot_map, T, Hkv,
                    static_cast<uint16_t*>(k), static_cast<uint16_t*>(v));
}

}  // namespace a4w4
