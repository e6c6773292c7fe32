// kv_decode.cu -- attention over the paged MXFP4 cache for few query rows per
// key/value head (single tokens, short drafts): R = new tokens x (Hq / Hkv) rows,
// 8 or 16 at a time.
//
//   O[r, :] = sum_k 2^(x_rk - m_r) v_k / sum_k 2^(x_rk - m_r),
//   x_rk = log2(e) sm_scale q_r . k_k
//
// One pass over the cache with running maximum and sum: a key and a value cost
// 17/16 D bytes and 4 R D flops, so memory is the floor.  A warp takes 32 tokens
// at a time, streamed by bulk copies into its own ring, and keeps everything
// else in registers; the tensor instruction is the warp-level one
// (m16n8k16, FP16 in, fp32 sums), because its operands come straight from the
// registers that decode the codes: a tcgen05 product would have every decoded
// value written to shared or tensor memory first, four times the bytes that
// the copy brought, which is more than that memory passes in the time.
//
// What bounds it then are the instructions that decode, some 650 a step of 32
// tokens and 8 rows at D = 128: 64 ragged requests of up to 8192 keys 70 us (4.1
// TB/s), 2 x 131000 keys x 16 rows 56 us (2.5 TB/s; a step of 16 rows has a fifth
// more instructions than one of 8, but 255 registers leave 8 warps to hide each
// other's latencies), one request of 1000 keys 8.4 us, most of it latency: launch,
// lengths, page numbers and cells one after the other, then the joins.
//
// Keys and values are the M side, query rows the N side (8 per tile), so that
// small groups waste little:
//   S^T[token, r] = K[token, :] Q^T     A = codes as FP16, exact
//   O^T[dim, r]  += V^T[dim, token] P^T
// * Keys: a thread's fragments are 8 consecutive dimensions of one token per
//   32-block, one word.  Each block's product is taken with the bare codes and
//   multiplied by the block's scale in fp32: exact for every scale below 2^104,
//   beyond which the sums may overflow.
// * Queries become FP16 times a power of two per row that puts the row's
//   largest element at 2^14: exact for elements down to 2^-28 of it.
// * Values need pairs of tokens in one word: two words of codes of neighbouring
//   tokens are merged nibble by nibble (4 logic operations for 16 values)
//   before the conversion, which then gives pairs of tokens.
// * The value scales depend on the token (the summed axis), so they multiply P:
//   one factor per token and 32-block, 2^(e - R + 9) with R the largest
//   exponent the warp has met, in FP16 down to 2^-24; O is rescaled when R
//   grows, as it is when the maximum does.  P is 2^(x - m + 6): FP16 holds it
//   to 11 bits down to 2^-20 of the row's largest, and the sum of a row's P is
//   taken in fp32 before that rounding.  A step with a P below that (or a value
//   scale far below R) takes BF16 products with P in two terms, 16 bits: 64 x 4096
//   keys with one dominant key per row 84 us, 68 without (one term, 8 bits: 78 and
//   67; the second term as a second pass over the values: 113 and 80).
// A warp is a worker of kv_walk.cuh: it walks its own run of 32-token steps, unit
// after unit, and writes the units that lie in it whole.  Parts of cut units stay
// in shared memory; when all warps are through, the CTA joins them, and units
// that reach into other CTAs are joined by the last of these to arrive.
#include "kv_walk.cuh"
#include "kv.cuh"

#include <cuda_fp16.h>

#include <atomic>
#include <cmath>

namespace a4w4 {

namespace {

constexpr int kStep = 32;                     // tokens of a step
// Steps of a worker, at least (2: one request x 1000 keys 2.5 us more), and workers of
// a CTA, at least (1: 100 keys, cut, 0.6 us more; alike from 1000 on).
constexpr uint32_t kLeast = 1;
constexpr int kFew = 4;
// What a unit costs beside its steps, in steps: so many places of the line before its
// first step hold no work.  1, 2, 3: 64 ragged requests x 8192 keys 71.9, 69.9, 71.5
// us (0: 12 us more), 24 ragged x 5 tokens x 3001 21.0, 20.6, 20.9.
constexpr int kUnitCost = 2;
constexpr int kWhole = 64;                    // places of the longest unit that a CTA may take whole
constexpr int kMaxParts = 256;                // CTAs of a launch, and so parts of a cut unit

template <int D, int NT>
struct DecCfg {
  using Ch = KvChunk<D>;
  // As many warps as the registers allow, nearly: at D = 128 the compiler reports 52 bytes of spill stores and 104 of
  // loads (8 rows, 128 registers) and 12 and 28 (16 rows, 255); at D = 64 none.  8, 12, 14, 16 warps, 64 ragged requests
  // x 8192 keys, D = 128, 8 rows: 79.8, 74.3, 80.3, 71.1 us; 16 rows with 12 warps 75.6 us where 8 took 57.4 (2 x 131000).
  static constexpr int WARPS = NT == 1 ? 16 : D == 64 ? 12 : 8;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int ROWS = 8 * NT;
  static constexpr int J = D / 32, I = D / 16;
  static constexpr int STAGE = 2 * Ch::kBytes;
  static constexpr int STAGES = D == 64 ? 4 : 2;
  static constexpr int KS = kStep * J * 4, VS = kStep * J * 2;    // per-warp scale factors
  static constexpr int PITCH = D + 8;                            // floats per row of a staged partial
  static constexpr int OFF_KS = WARPS * STAGES * STAGE;
  static constexpr int OFF_VS = OFF_KS + WARPS * KS;
  static constexpr int OFF_O = OFF_VS + WARPS * VS;
  static constexpr int OFF_ML = OFF_O + WARPS * ROWS * PITCH * 4;   // maxima and sums: [tail or head][warp][row]
  static constexpr int OFF_BAR = OFF_ML + 2 * WARPS * ROWS * 8;
  static constexpr int OFF_OPEN = OFF_BAR + WARPS * STAGES * 8;
  static constexpr int OFF_MISC = OFF_OPEN + (WARPS + 1) * 24;
  static constexpr int OFF_SCAN = OFF_MISC + 16;                 // the cut's scratch: slow warps read it while fast ones work
  static constexpr int OFF_SHARE = OFF_SCAN + (THREADS + 32) * 4;       // each warp's copy of the cut: registers are short
  static constexpr int SMEM = OFF_SHARE + WARPS * static_cast<int>(sizeof(KvShare));
  static constexpr int PART = ROWS * (D + 2);                    // floats of a stored part: O, then m and l
  static_assert(STAGE % 16 == 0 && OFF_KS % 16 == 0 && OFF_VS % 16 == 0 && OFF_O % 16 == 0, "alignment");
  static_assert(kMaxParts <= kTickets && PART % 4 == 0, "join");
  static_assert(ROWS * PITCH * 4 <= STAGES * STAGE, "a part fits in the warp's drained ring");
  static_assert(OFF_OPEN % 4 == 0 && OFF_SCAN % 4 == 0, "alignment");
  static_assert(OFF_BAR % 8 == 0 && SMEM <= 232448, "shared memory");
};

__device__ __forceinline__ void mma_f16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// c = a b
__device__ __forceinline__ void mma_f16_first(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ void mma_bf16(float* c, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Four E2M1 codes in each half of w (nibble k of both halves to o[k]) as BF16x2: the code's magnitude bits at 6..8
// of a BF16 read as the value times 2^-126, which one exact multiply puts right.
__device__ __forceinline__ void e2m1x4_to_bf16x2(uint32_t w, uint32_t* o) {
  constexpr uint32_t kMag = 0x01C001C0u, kSign = 0x80008000u, kUp = 0x7E807E80u;
  o[0] = mul_bf16x2(((w << 6) & kMag) | ((w << 12) & kSign), kUp);
  o[1] = mul_bf16x2(((w << 2) & kMag) | ((w << 8) & kSign), kUp);
  o[2] = mul_bf16x2(((w >> 2) & kMag) | ((w << 4) & kSign), kUp);
  o[3] = mul_bf16x2(((w >> 6) & kMag) | (w & kSign), kUp);
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t v) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(v));
  return d;
}

// The bytes of a chunk's value codes that lane 4 g + t needs: tokens 2t, 2t+1 of both halves.
template <int D>
__device__ __forceinline__ void load_runs(const uint8_t* codes, int lane, uint32_t (&run)[2][2][D / 64]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if constexpr (D == 128) {
      const uint4 v = *reinterpret_cast<const uint4*>(codes + h * 4 * D + lane * 16);
      run[h][0][0] = v.x; run[h][0][1] = v.y; run[h][1][0] = v.z; run[h][1][1] = v.w;
    } else {
      const uint2 v = *reinterpret_cast<const uint2*>(codes + h * 4 * D + lane * 8);
      run[h][0][0] = v.x; run[h][1][0] = v.y;
    }
  }
}

// A unit of which a part waits in this CTA's shared memory.
struct Open {
  int row0, h, r0, rows;      // first row of the request, head, first row of the block, rows to join; rows == 0: none
  uint32_t v0, v1;            // the workers that hold its first and its last step
};

// A walk along the worker's run: one piece (a run of one unit's steps) at a time.
struct Walk {
  int b, h, k, t, n;          // request, head, block of rows, first step of the piece, steps of the unit
  int len, rows, all, row0;   // rows: the request's, all its heads'
  int left;                   // places of the run from the piece's first step on
  __device__ __forceinline__ void load(const KvRequest& r, int G) {
    len = r.len; rows = r.rows * G; all = r.all; row0 = r.row0;
    n = rows > 0 ? max(1, (len + kStep - 1) / kStep) : 0;
  }
  __device__ __forceinline__ int steps() const { return min(left, n - t); }
  // the token where the piece ends
  __device__ __forceinline__ int end() const { return min(len, (t + steps()) * kStep); }
  template <int ROWS>
  __device__ __forceinline__ void next(const KvAttentionArgs& p, int G) {
    left -= steps();
    t = 0;
    if (left <= 0) return;
    left -= kUnitCost;
    if (++k * ROWS < rows) return;
    k = 0;
    if (++h < p.Hkv) return;
    h = 0;
    do { load(kv_request(p, ++b), G); } while (n == 0);    // a run ends in a request that has steps
  }
};

template <int D, int NT>
__global__ void __launch_bounds__(DecCfg<D, NT>::THREADS, 1) a4w4_kv_decode_kernel(const KvAttentionArgs p) {
  using Cf = DecCfg<D, NT>;
  using Ch = KvChunk<D>;
  constexpr int J = Cf::J, I = Cf::I, W = Cf::WARPS, S = Cf::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cf::OFF_MISC);
  volatile int* never = abort_flag + 1;
  volatile int* last_flag = abort_flag + 2;
  Open* open = reinterpret_cast<Open*>(smem + Cf::OFF_OPEN);
  const uint32_t sbase = smem_u32(smem);
  auto full = [&](int s) { return sbase + Cf::OFF_BAR + 8u * (warp * S + s); };
  if (tid == 0) { *abort_flag = 0; *never = 0; }
  if (tid <= W) open[tid].rows = 0;
  if (lane == 0)
    for (int s = 0; s < S; ++s) mbar_init(full(s), 1);
  fence_barrier_init();
  __syncthreads();                               // flags and list are set before anything is put in them
  const int G = p.Hq / p.Hkv;
  griddep_wait();
  griddep_launch_dependents();

  KvShare share;
  KvStart start;
  auto unit = [&](const KvRequest& r) -> uint32_t { return max(1, (r.len + kStep - 1) / kStep) + kUnitCost; };
  auto places = [&](const KvRequest& r) -> uint32_t {
    return r.rows > 0 ? unit(r) * p.Hkv * ((r.rows * G + Cf::ROWS - 1) / Cf::ROWS) : 0;
  };
  if (!kv_locate<Cf::THREADS, W, kWhole>(p, places, unit, kUnitCost, [](uint32_t) { return kLeast; }, kFew,
                                         reinterpret_cast<uint32_t*>(smem + Cf::OFF_SCAN), share, start))
    return;
  const uint32_t per = share.per, me = blockIdx.x * per + warp;
  KvShare* cut = reinterpret_cast<KvShare*>(smem + Cf::OFF_SHARE) + warp;
  if (lane == 0) *cut = share;

  Walk cw;
  cw.left = 0;
  if (warp < per && me < share.workers) {
    cw.b = start.b;
    cw.load(start.req, G);
    const int blocks = (cw.rows + Cf::ROWS - 1) / Cf::ROWS, unit = start.rest / (cw.n + kUnitCost);
    const int at = start.rest - unit * (cw.n + kUnitCost);
    cw.h = unit / blocks;
    cw.k = unit - cw.h * blocks;
    cw.t = max(0, at - kUnitCost);
    cw.left = static_cast<int>(share.first(me + 1) - share.first(me)) - max(0, kUnitCost - at);
  }

  const int lg = 31 - __clz(p.page_size), chunks = p.page_size >> 4;     // page_size is a power of two
  const long long page_bytes = static_cast<long long>(p.Hkv) * chunks * Ch::kBytes;
  uint8_t* ring = smem + warp * S * Cf::STAGE;
  float* ks = reinterpret_cast<float*>(smem + Cf::OFF_KS + warp * Cf::KS);
  uint8_t* vs = smem + Cf::OFF_VS + warp * Cf::VS;

  // ---- the warp's copies: the same steps as the loop below, S ahead of it ----
  Walk pw = cw;
  int ptok = 0, pend = 0;                      // first token of the next step, and where its piece ends
  if (pw.left > 0) { ptok = pw.t * kStep; pend = pw.end(); }
  int pi = 0;                                  // step of the piece
  int page0 = 0, page1 = 0;                    // lane i: pages of step (pi & ~31) + i
  int issued = 0, waited = 0;
  const uint64_t pol = policy_evict_first();
  auto issue = [&]() {
    while (ptok >= pend) {
      if (pw.left <= 0) return;
      pw.template next<Cf::ROWS>(p, G);
      ptok = 0;
      pend = pw.left > 0 ? pw.end() : 0;
      pi = 0;
    }
    if ((pi & 31) == 0) {
      const int ahead = lane * kStep, rest = pw.len - ptok;    // compared like this, since ptok + ahead may pass 2^31
      page0 = ahead < rest ? kv_page(p, pw.b, (ptok + ahead) >> lg) : 0;
      if (lg == 4) page1 = ahead + 16 < rest ? kv_page(p, pw.b, (ptok + ahead + 16) >> 4) : 0;
    }
    const int id0 = __shfl_sync(0xFFFFFFFFu, page0, pi & 31);
    const int id1 = lg == 4 ? __shfl_sync(0xFFFFFFFFu, page1, pi & 31) : 0;
    if (lane == 0) {
      const int slot = issued % S;
      const bool two = pw.len - ptok > 16;
      const uint32_t bar = full(slot), dst = sbase + (warp * S + slot) * Cf::STAGE;
      const uint8_t* head = p.cache + pw.h * (chunks * Ch::kBytes);
      mbar_arrive_expect_tx(bar, two ? 2 * Ch::kBytes : Ch::kBytes);
      if (lg > 4) {
        bulk_g2s(dst, head + id0 * page_bytes + ((ptok >> 4) & (chunks - 1)) * Ch::kBytes,
                 two ? 2 * Ch::kBytes : Ch::kBytes, bar, pol);
      } else {
        bulk_g2s(dst, head + id0 * page_bytes, Ch::kBytes, bar, pol);
        if (two) bulk_g2s(dst + Ch::kBytes, head + id1 * page_bytes, Ch::kBytes, bar, pol);
      }
    }
    ++issued;
    ++pi;
    ptok += kStep;
  };
  // ---- queries: the lane's words of row nt * 8 + g, 8 dimensions per 32-block ----
  uint32_t qf[NT][J][4];
  auto load_queries = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int r = cw.k * Cf::ROWS + nt * 8 + g, qi = p.row_of(r);
      const uint16_t* src = p.q + (static_cast<long long>(cw.row0) + qi) * p.q_stride + (cw.h * G + r - qi * G) * D + 8 * t;
#pragma unroll
      for (int j = 0; j < J; ++j) {
        const uint4 x = r < cw.rows ? ld_global_nc_v4(src + 32 * j) : make_uint4(0u, 0u, 0u, 0u);
        qf[nt][j][0] = x.x; qf[nt][j][1] = x.y; qf[nt][j][2] = x.z; qf[nt][j][3] = x.w;
      }
    }
  };
  if (cw.left > 0) load_queries();               // on their way while the first pages are looked up
  __syncwarp();
  for (int s = 0; s < S; ++s) issue();

  bool ok = true, first_piece = true;
  while (cw.left > 0) {
    const int h = cw.h, len = cw.len;
    const int r0 = cw.k * Cf::ROWS, R = min(cw.rows - r0, Cf::ROWS);
    if (!first_piece) load_queries();
    first_piece = false;
    float fcol[NT][2];                         // raw score -> log2 units, per column
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) top = max_abs_bf16x2(top, qf[nt][j][u]);
      top &= 0x7FFF7FFFu;
      uint32_t e = max(top & 0xFFFFu, top >> 16) >> 7;
      e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 1));
      e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 2));
      const int k = min(141 - static_cast<int>(e), 127);       // largest element to [2^14, 2^15)
      const float f = pow2i(k);
#pragma unroll
      for (int j = 0; j < J; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u)
          qf[nt][j][u] = pack_f16(__uint_as_float(qf[nt][j][u] << 16) * f, __uint_as_float(qf[nt][j][u] & 0xFFFF0000u) * f);
      // positive: a masked score stays -infinity when multiplied
      const float back = fmaxf(p.sm_scale * 1.4426950408889634f * pow2i(-k), 1e-44f);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        fcol[nt][u] = __shfl_sync(0xFFFFFFFFu, back, (2 * t + u) * 4);
      }
    }
    const int all_seen = len - cw.all + 1;                     // keys that every row sees

    float o[I][NT][4];
    float m[NT][2], off[NT][2], l[NT][2];      // raw running maximum, 6 - m f, sum
#pragma unroll
    for (int i = 0; i < I; ++i)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 4; ++u) o[i][nt][u] = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int u = 0; u < 2; ++u) { m[nt][u] = kNoMax; off[nt][u] = 3.0e38f; l[nt][u] = 0.f; }
    int ref = 0;                                               // largest value scale met

    const int end = cw.end();
    for (int tok0 = cw.t * kStep; tok0 < end; tok0 += kStep) {
      const int slot = waited % S;
      if (ok) {
        ok = kv_wait(full(slot), (waited / S) & 1u, abort_flag, p.wait_ns, p.status);
        ok = __all_sync(0xFFFFFFFFu, ok);
      }
      if (!ok) continue;
      ++waited;
      const uint8_t* st = ring + slot * Cf::STAGE;

      // ---- scale factors, lane = token; the value factor of a cell beyond the length is finite ----
      uint32_t vw;
      bool vlow;                                               // a value factor that FP16 does not hold
      int nref;
      {
        const uint8_t* c = st + (lane >> 4) * Ch::kBytes + (lane & 15) * J;
        uint32_t kw;
        if constexpr (J == 4) {
          kw = *reinterpret_cast<const uint32_t*>(c + Ch::kKeyScales);
          vw = *reinterpret_cast<const uint32_t*>(c + Ch::kValueScales);
        } else {
          kw = *reinterpret_cast<const uint16_t*>(c + Ch::kKeyScales);
          vw = *reinterpret_cast<const uint16_t*>(c + Ch::kValueScales);
        }
        if (tok0 + lane >= len) vw = 0u;                       // such a cell holds anything
        uint32_t kf[J];                                        // 2^(e - 127)
#pragma unroll
        for (int j = 0; j < J; ++j)
          kf[j] = max((j < 3 ? kw << (23 - 8 * j) : kw >> 1) & 0x7F800000u, 0x00400000u);
        if constexpr (J == 4) *reinterpret_cast<uint4*>(ks + lane * 4) = make_uint4(kf[0], kf[1], kf[2], kf[3]);
        else *reinterpret_cast<uint2*>(ks + lane * 2) = make_uint2(kf[0], kf[1]);
        // value scales, two blocks to a word
        uint32_t e2[J / 2], top = 0u, least = 0xFFFFFFFFu;     // least: smallest e - 1, zero blocks left out
#pragma unroll
        for (int q = 0; q < J / 2; ++q) {
          e2[q] = __byte_perm(vw, 0u, q ? 0x4342 : 0x4140);
          top = __vmaxu2(top, e2[q]);
          least = __viaddmin_u16x2(e2[q], 0xFFFFFFFFu, least);
        }
        nref = max(ref, static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16))));
        vlow = static_cast<int>(min(least & 0xFFFFu, least >> 16)) < nref - 10;
        uint8_t* dst = vs + (lane >> 1 & 3) * 16 + (lane >> 4) * 8 + (lane >> 3 & 1) * 4 + (lane & 1) * 2;
        const uint32_t up = (24u - static_cast<uint32_t>(nref) & 0xFFFFu) * 0x00010001u;
#pragma unroll
        for (int q = 0; q < J / 2; ++q) {
          const uint32_t f2 = __viaddmax_s16x2_relu(e2[q], up, 0u) << 10;      // 2^(e - nref + 9), exponent field >= 0
          *reinterpret_cast<uint16_t*>(dst + q * 128) = static_cast<uint16_t>(f2);
          *reinterpret_cast<uint16_t*>(dst + q * 128 + 64) = static_cast<uint16_t>(f2 >> 16);
        }
      }
      __syncwarp();

      // ---- raw scores ----
      float x[2][NT][4];
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const uint8_t* cp = st + c * Ch::kBytes;
        uint32_t wa[J], wb[J];
        float sa[J], sb[J];
        if constexpr (J == 4) {
          const uint4 a = *reinterpret_cast<const uint4*>(cp + g * (D / 2) + t * 16);
          const uint4 bb = *reinterpret_cast<const uint4*>(cp + (g + 8) * (D / 2) + t * 16);
          wa[0] = a.x; wa[1] = a.y; wa[2] = a.z; wa[3] = a.w;
          wb[0] = bb.x; wb[1] = bb.y; wb[2] = bb.z; wb[3] = bb.w;
          const float4 fa = *reinterpret_cast<const float4*>(ks + (c * 16 + g) * 4);
          const float4 fb = *reinterpret_cast<const float4*>(ks + (c * 16 + g + 8) * 4);
          sa[0] = fa.x; sa[1] = fa.y; sa[2] = fa.z; sa[3] = fa.w;
          sb[0] = fb.x; sb[1] = fb.y; sb[2] = fb.z; sb[3] = fb.w;
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(cp + g * (D / 2) + t * 8);
          const uint2 bb = *reinterpret_cast<const uint2*>(cp + (g + 8) * (D / 2) + t * 8);
          wa[0] = a.x; wa[1] = a.y; wb[0] = bb.x; wb[1] = bb.y;
          const float2 fa = *reinterpret_cast<const float2*>(ks + (c * 16 + g) * 2);
          const float2 fb = *reinterpret_cast<const float2*>(ks + (c * 16 + g + 8) * 2);
          sa[0] = fa.x; sa[1] = fa.y; sb[0] = fb.x; sb[1] = fb.y;
        }
#pragma unroll
        for (int j = 0; j < J; ++j) {
          uint32_t fa[4], fb[4];
          e2m1x8_to_f16x2(wa[j], fa);
          e2m1x8_to_f16x2(wb[j], fb);
          const uint32_t a0[4] = {fa[0], fb[0], fa[1], fb[1]}, a1[4] = {fa[2], fb[2], fa[3], fb[3]};
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float acc[4];
            mma_f16_first(acc, a0, qf[nt][j][0], qf[nt][j][1]);
            mma_f16(acc, a1, qf[nt][j][2], qf[nt][j][3]);
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const float s = u < 2 ? sa[j] : sb[j];
              x[c][nt][u] = j == 0 ? acc[u] * s : fmaf(acc[u], s, x[c][nt][u]);
            }
          }
        }
      }
      if (tok0 + kStep > all_seen) {
        asm volatile("" ::: "memory");                         // a branch, not selects in every step
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            // keys that the column's row sees, from the step's first on
            const int lim = all_seen + p.row_of(r0 + nt * 8 + 2 * t + (u & 1)) - tok0 - g - (u >> 1) * 8;
            if (0 >= lim) x[0][nt][u] = -INFINITY;
            if (16 >= lim) x[1][nt][u] = -INFINITY;
          }
      }

      // ---- running maximum and value reference ----
      float mx[NT][2];
      bool grow = nref > ref;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          mx[nt][u] = fmaxf(fmaxf(x[0][nt][u], x[0][nt][u + 2]), fmaxf(x[1][nt][u], x[1][nt][u + 2]));
          grow |= mx[nt][u] > m[nt][u];
        }
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float fr = pow2i(ref - nref);
        ref = nref;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          float fo[2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            float y = mx[nt][u];
            y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 4));
            y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 8));
            y = fmaxf(y, __shfl_xor_sync(0xFFFFFFFFu, y, 16));
            y = fmaxf(m[nt][u], y);
            const float a = ex2((m[nt][u] - y) * fcol[nt][u]);
            m[nt][u] = y;
            off[nt][u] = fminf(fmaf(-y, fcol[nt][u], 6.f), 3.0e38f);
            l[nt][u] *= a;
            fo[u] = a * fr;
          }
#pragma unroll
          for (int i = 0; i < I; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) o[i][nt][u] *= fo[u & 1];
        }
      }

      // ---- probabilities times 2^6 ----
      bool low = vlow;                                         // something that FP16 holds to fewer than 11 bits
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < 4; ++u) x[c][nt][u] = fmaf(x[c][nt][u], fcol[nt][u & 1], off[nt][u & 1]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float mn = fminf(x[0][nt][0], x[1][nt][0]);
#pragma unroll
        for (int u = 1; u < 4; ++u) mn = fminf(mn, fminf(x[0][nt][u], x[1][nt][u]));
        low |= mn < -14.f;
      }
      if (tok0 + kStep > all_seen) {                           // masked keys are none of these: their zeros are exact
        asm volatile("" ::: "memory");
        low = vlow;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int u = 0; u < 4; ++u) low |= x[c][nt][u] < -14.f && x[c][nt][u] > -INFINITY;
      }
#pragma unroll
      for (int c = 0; c < 2; ++c)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            x[c][nt][u] = ex2(x[c][nt][u]);
            l[nt][u & 1] += x[c][nt][u];
          }

      // ---- output ----
      if (!__any_sync(0xFFFFFFFFu, low)) {
        uint32_t pb[2][NT][2];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            pb[c][nt][0] = movmatrix_trans(pack_f16(x[c][nt][0], x[c][nt][1]));
            pb[c][nt][1] = movmatrix_trans(pack_f16(x[c][nt][2], x[c][nt][3]));
          }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t run[2][2][I / 4];                           // [half][token of the pair][word]
          load_runs<D>(st + c * Ch::kBytes + Ch::kValues, lane, run);
#pragma unroll
          for (int q4 = 0; q4 < I / 4; ++q4) {
            uint32_t lo[2][4], hi[2][4];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
              const uint32_t va = run[hh][0][q4], vb = run[hh][1][q4];
              e2m1x8_to_f16x2((va & 0x0F0F0F0Fu) | ((vb << 4) & 0xF0F0F0F0u), lo[hh]);
              e2m1x8_to_f16x2(((va >> 4) & 0x0F0F0F0Fu) | (vb & 0xF0F0F0F0u), hi[hh]);
            }
#pragma unroll
            for (int jj = 0; jj < 2; ++jj) {
              const int j = q4 * 2 + jj;
              const uint2 f = *reinterpret_cast<const uint2*>(vs + j * 64 + t * 16 + c * 8);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint32_t b0 = mul_f16x2(pb[c][nt][0], f.x), b1 = mul_f16x2(pb[c][nt][1], f.y);
#pragma unroll
                for (int ii = 2 * jj; ii < 2 * jj + 2; ++ii) {
                  const uint32_t a[4] = {lo[0][ii], hi[0][ii], lo[1][ii], hi[1][ii]};
                  mma_f16(o[q4 * 4 + ii][nt], a, b0, b1);
                }
              }
            }
          }
        }
      } else {
        // the same in BF16, whose exponents reach, P in two terms: its rounding and what that leaves
        uint32_t pb[2][NT][2], rest[2][NT][2];
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              const float y0 = x[c][nt][2 * u], y1 = x[c][nt][2 * u + 1];
              const uint32_t w = pack_bf16(y0, y1);
              pb[c][nt][u] = movmatrix_trans(w);
              rest[c][nt][u] = movmatrix_trans(pack_bf16(y0 - __uint_as_float(w << 16), y1 - __uint_as_float(w & 0xFFFF0000u)));
            }
        __syncwarp();
        uint8_t* dst = vs + (lane >> 1 & 3) * 16 + (lane >> 4) * 8 + (lane >> 3 & 1) * 4 + (lane & 1) * 2;
#pragma unroll
        for (int j = 0; j < J; ++j) {
          const int k = static_cast<int>(vw >> (8 * j) & 0xFFu) - ref + 9;
          *reinterpret_cast<uint16_t*>(dst + j * 64) = static_cast<uint16_t>(max(k + 127, 0) << 7);
        }
        __syncwarp();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t run[2][2][I / 4];
          load_runs<D>(st + c * Ch::kBytes + Ch::kValues, lane, run);
#pragma unroll
          for (int j = 0; j < J; ++j) {                        // 32-block j: row tiles 2j and 2j + 1
            const uint2 f = *reinterpret_cast<const uint2*>(vs + j * 64 + t * 16 + c * 8);
            uint32_t v[2][4];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
              e2m1x4_to_bf16x2(__byte_perm(run[hh][0][j / 2], run[hh][1][j / 2], j & 1 ? 0x7632 : 0x5410), v[hh]);
            const uint32_t a0[4] = {v[0][0], v[0][1], v[1][0], v[1][1]}, a1[4] = {v[0][2], v[0][3], v[1][2], v[1][3]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t* q = k ? (c ? rest[1][nt] : rest[0][nt]) : c ? pb[1][nt] : pb[0][nt];
                const uint32_t b0 = mul_bf16x2(q[0], f.x), b1 = mul_bf16x2(q[1], f.y);
                mma_bf16(o[2 * j][nt], a0, b0, b1);
                mma_bf16(o[2 * j + 1][nt], a1, b0, b1);
              }
          }
        }
      }
      __syncwarp();                                            // the slot and the scale factors are free again
      issue();
    }

    // ---- the unit's output, or the part of it ----
    // O = o 2^(ref - 127 - 9 - 6) relative to the maximum, in two exact steps
    const int k = ref - 142, ka = k / 2;
    const float fa = pow2i(ka), fb = pow2i(k - ka);
    const bool front = cw.t > 0, back = cw.t + cw.steps() < cw.n;
    float* po = back ? reinterpret_cast<float*>(ring) : reinterpret_cast<float*>(smem + Cf::OFF_O) + warp * Cf::ROWS * Cf::PITCH;
    float2* ml = reinterpret_cast<float2*>(smem + Cf::OFF_ML) + ((back ? 0 : W) + warp) * Cf::ROWS;
    if (!ok) {                                                   // copies may still arrive in the ring
      const unsigned long long drain_ns = p.wait_ns > 100000000ull ? p.wait_ns : 100000000ull;
      for (; waited < issued; ++waited) kv_wait(full(waited % S), (waited / S) & 1u, never, drain_ns, p.status);
      __syncwarp();
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int col = nt * 8 + 2 * t + u;
        float s = l[nt][u];
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 4);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 8);
        s += __shfl_xor_sync(0xFFFFFFFFu, s, 16);
        s *= 0.015625f;
        const float mm = fmaxf(m[nt][u] * fcol[nt][u], kNoMax);
        if (front || back) {
          if (g == 0) ml[col] = make_float2(mm, s);
#pragma unroll
          for (int i = 0; i < I; ++i)
            *reinterpret_cast<float2*>(po + col * Cf::PITCH + 16 * i + 2 * g) =
                make_float2(o[i][nt][u] * fa * fb, o[i][nt][u + 2] * fa * fb);
        } else if (col < R) {
          const int qi = p.row_of(r0 + col), hq = h * G + r0 + col - qi * G;
          const long long row = static_cast<long long>(cw.row0) + qi;
          const float inv = s == 0.f ? 0.f : 1.f / s;
#pragma unroll
          for (int i = 0; i < I; ++i)
            *reinterpret_cast<uint32_t*>(p.out + (row * p.Hq + hq) * D + 16 * i + 2 * g) =
                pack_bf16(o[i][nt][u] * fa * fb * inv, o[i][nt][u + 2] * fa * fb * inv);
          if (g == 0 && p.lse != nullptr)
            p.lse[row * p.Hq + hq] = s == 0.f ? -INFINITY : fmaf(mm, 0.6931471805599453f, logf(s));
        }
      }
    // the CTA's list of cut units: by the warp that holds their beginning, or by
    // the first warp if that lies in an earlier CTA
    if (lane == 0 && ((back && !front) || (front && warp == 0))) {
      const uint32_t u0 = cut->first(me + 1) - cw.left - cw.t;   // the unit's first step on the line
      open[front ? 0 : warp + 1] = Open{cw.row0, h, r0, R, cut->holder(u0), cut->holder(u0 + cw.n - 1)};
    }
    cw.template next<Cf::ROWS>(p, G);
  }
  __syncthreads();

  // ---- join the parts in this CTA: a warp per row of a cut unit ----
  const uint32_t cta = blockIdx.x;
  const float2* mls = reinterpret_cast<const float2*>(smem + Cf::OFF_ML);
  float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + kTickets * 4);
  const uint32_t opened = __ballot_sync(0xFFFFFFFFu, lane <= W && open[min(lane, W)].rows != 0);
  uint32_t outside = 0;                                          // the units that reach into other CTAs: two at most
  int turn = 0;                                                  // rows are dealt to the warps in turn
  for (uint32_t left = opened; left != 0; left &= left - 1) {
    const Open un = open[__ffs(left) - 1];
    const int R = un.rows;
    const uint32_t v0 = un.v0, v1 = un.v1;
    const uint32_t mine0 = cta * per, mine1 = mine0 + per;         // this CTA's workers
    const int w0 = v0 < mine0 ? 0 : v0 - mine0, w1 = v1 >= mine1 ? per - 1 : v1 - mine0;
    const bool whole = v0 >= mine0 && v1 < mine1;
    if (!whole) outside |= left & -left;
    // all parts are tails but the one with the unit's end
    const int head = v1 < mine1 ? w1 : W;
    // two places per CTA outside: for a unit that began before it, and for one that goes on after it
    float* mine = parts + (2 * cta + (v0 < mine0 ? 0 : 1)) * Cf::PART;
    const int np = w1 - w0 + 1;
    for (int r = (warp - turn % W + W) % W; r < R; r += W) {
      const int w = w0 + lane;                                   // lane: a part
      const float2 q = lane < np ? mls[((w == head ? W : 0) + w) * Cf::ROWS + r] : make_float2(kNoMax, 0.f);
      float mm = q.x;
#pragma unroll
      for (int s = 8; s > 0; s >>= 1) mm = fmaxf(mm, __shfl_xor_sync(0xFFFFFFFFu, mm, s));
      const float a = ex2(q.x - mm);
      float ll = q.y * a;
#pragma unroll
      for (int s = 8; s > 0; s >>= 1) ll += __shfl_xor_sync(0xFFFFFFFFu, ll, s);
      mm = __shfl_sync(0xFFFFFFFFu, mm, 0);
      ll = __shfl_sync(0xFFFFFFFFu, ll, 0);
      float y[D / 32];
#pragma unroll
      for (int u = 0; u < D / 32; ++u) y[u] = 0.f;
#pragma unroll 4
      for (int k = 0; k < np; ++k) {
        const float ak = __shfl_sync(0xFFFFFFFFu, a, k);
        const uint8_t* src = w0 + k == head ? smem + Cf::OFF_O + head * (Cf::ROWS * Cf::PITCH * 4)
                                            : smem + (w0 + k) * (S * Cf::STAGE);
        const float* v = reinterpret_cast<const float*>(src) + r * Cf::PITCH + lane * (D / 32);
#pragma unroll
        for (int u = 0; u < D / 32; u += 2) {
          const float2 x = *reinterpret_cast<const float2*>(v + u);
          y[u] = fmaf(x.x, ak, y[u]);
          y[u + 1] = fmaf(x.y, ak, y[u + 1]);
        }
      }
      if (whole) {
        const int qi = p.row_of(un.r0 + r), hq = un.h * G + un.r0 + r - qi * G;
        const long long row = static_cast<long long>(un.row0) + qi;
        const float inv = ll == 0.f ? 0.f : 1.f / ll;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (row * p.Hq + hq) * D + lane * (D / 32));
#pragma unroll
        for (int u = 0; u < D / 32; u += 2) dst[u / 2] = pack_bf16(y[u] * inv, y[u + 1] * inv);
        if (lane == 0 && p.lse != nullptr)
          p.lse[row * p.Hq + hq] = ll == 0.f ? -INFINITY : fmaf(mm, 0.6931471805599453f, logf(ll));
      } else {
        float2* dst = reinterpret_cast<float2*>(mine + r * D + lane * (D / 32));
#pragma unroll
        for (int u = 0; u < D / 32; u += 2) dst[u / 2] = make_float2(y[u], y[u + 1]);
        if (lane == 0) *reinterpret_cast<float2*>(mine + Cf::ROWS * D + 2 * r) = make_float2(mm, ll);
      }
    }
    turn += R;
  }
  if (!outside) return;

  // ---- units that reach into other CTAs: the last to arrive joins ----
  __syncthreads();
  if (warp == 0) {                                               // a lane per unit draws its ticket
    const bool mine = (outside >> lane & 1u) != 0;
    bool last = false;
    if (mine) {
      const int c0 = open[lane].v0 / per, np = open[lane].v1 / per - c0 + 1;
      last = draw_ticket(static_cast<int*>(p.ws) + c0) == np - 1;
    }
    const uint32_t lasts = __ballot_sync(0xFFFFFFFFu, last);
    if (lane == 0) *last_flag = static_cast<int>(lasts);
  }
  __syncthreads();
  for (uint32_t left = static_cast<uint32_t>(*last_flag); left != 0; left &= left - 1) {
    const Open un = open[__ffs(left) - 1];
    const int c0 = un.v0 / per, np = un.v1 / per - c0 + 1, R = un.rows;
    auto part = [&](int k) { return parts + (2 * (c0 + k) + (k == 0 ? 1 : 0)) * Cf::PART; };
    // 16 bytes of a row per thread, every thread with its own copy of the row's maximum and sum: one trip to memory
    // for 12 parts (one request x 1000 keys 8.7 us; with a trip and a barrier for the statistics first, 9.6)
    constexpr int AT = 12;
    for (int it = tid; it < R * (D / 4); it += Cf::THREADS) {
      const int r = it / (D / 4), d = it % (D / 4) * 4;
      float mm = kNoMax, ll = 0.f;
      float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int k0 = 0; k0 < np; k0 += AT) {
        float2 q[AT];
        float4 v[AT];
#pragma unroll
        for (int k = 0; k < AT; ++k) {
          const float* src = part(min(k0 + k, np - 1));
          q[k] = __ldcg(reinterpret_cast<const float2*>(src + Cf::ROWS * D + 2 * r));
          v[k] = __ldcg(reinterpret_cast<const float4*>(src + r * D + d));
        }
        float top = mm;
#pragma unroll
        for (int k = 0; k < AT; ++k) top = fmaxf(top, q[k].x);
        const float f = ex2(mm - top);
        mm = top;
        ll *= f;
        y.x *= f; y.y *= f; y.z *= f; y.w *= f;
#pragma unroll
        for (int k = 0; k < AT; ++k) {
          const float a = k0 + k < np ? ex2(q[k].x - mm) : 0.f;
          ll = fmaf(q[k].y, a, ll);
          y.x = fmaf(v[k].x, a, y.x); y.y = fmaf(v[k].y, a, y.y); y.z = fmaf(v[k].z, a, y.z); y.w = fmaf(v[k].w, a, y.w);
        }
      }
      const float inv = ll == 0.f ? 0.f : 1.f / ll;
      const int qi = p.row_of(un.r0 + r), hq = un.h * G + un.r0 + r - qi * G;
      const long long row = static_cast<long long>(un.row0) + qi;
      *reinterpret_cast<uint2*>(p.out + (row * p.Hq + hq) * D + d) =
          make_uint2(pack_bf16(y.x * inv, y.y * inv), pack_bf16(y.z * inv, y.w * inv));
      if (d == 0 && p.lse != nullptr)
        p.lse[row * p.Hq + hq] = ll == 0.f ? -INFINITY : fmaf(mm, 0.6931471805599453f, logf(ll));
    }
    if (tid == 0) static_cast<int*>(p.ws)[c0] = 0;
  }
}

}  // namespace

size_t kv_decode_ws_bytes(int rows, int D, int sms) {
  const int ctas = sms < kMaxParts ? sms : kMaxParts;
  return kTickets * 4 + 2ull * ctas * ((rows + 7) / 8 % 2 ? 8 : 16) * (D + 2) * 4;
}

namespace {

template <int D, int NT>
int launch_one(const KvAttentionArgs& p, int grid, cudaStream_t st) {
  using Cf = DecCfg<D, NT>;
  static std::atomic<unsigned long long> attr_done{0};
  const int rc = ensure_func_attrs(attr_done, [] {
    return cudaFuncSetAttribute(a4w4_kv_decode_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM) ==
           cudaSuccess;
  });
  if (rc != 0) return rc;
  return launch_pdl_smem(a4w4_kv_decode_kernel<D, NT>, grid, Cf::THREADS, Cf::SMEM, st, p);
}

}  // namespace

int launch_kv_decode(const KvAttentionArgs& p, int D, cudaStream_t st, int sms) {
  const int rows = p.max_q * (p.Hq / p.Hkv);
  // 16 rows at a time, but an odd number of 8-row blocks would waste half of one.  In blocks of 8 and of 16: 24 ragged
  // requests x 20 rows 20.5 and 22.5 us (D = 64), 4 x 16384 keys x 24 rows 54.1 and 55.9 (D = 128), 2 x 131000 keys x
  // 16 rows 59.2 and 55.6 (D = 128), 43.0 and 35.8 (D = 64)
  const bool two = (rows + 7) / 8 % 2 == 0;
  // as many CTAs as there can be work for, one per SM at most
  const double units = static_cast<double>(p.B) * p.Hkv * ((rows + (two ? 15 : 7)) / (two ? 16 : 8));
  const double unit = static_cast<double>(p.max_pages) * p.page_size / kStep + 1 + kUnitCost, places = unit * units;
  if (unit * most_units(p, two ? 16 : 8) >= kTooMany) return -1;
  const int most = sms < kMaxParts ? sms : kMaxParts;
  const double ctas = fmax(units, places / (kLeast * kFew) + 1);
  const int grid = ctas < most ? static_cast<int>(ctas) : most;
  if (D == 64) return two ? launch_one<64, 2>(p, grid, st) : launch_one<64, 1>(p, grid, st);
  return two ? launch_one<128, 2>(p, grid, st) : launch_one<128, 1>(p, grid, st);
}

}  // namespace a4w4
