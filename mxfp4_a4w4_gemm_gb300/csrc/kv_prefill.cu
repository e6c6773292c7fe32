// kv_prefill.cu -- attention over the paged MXFP4 cache for many query rows per
// key/value head (prompt chunks, longer drafts, large groups): tcgen05.
//
// Rows are packed: the G query heads of a key/value head times the new tokens
// are the rows of one matrix, so keys are decoded once for all of them.  A unit
// is 256 such rows (two tiles of 128) against the keys that the last of them
// sees, a step is 128 keys.  Per step and tile
//   S = Q K^T   [128 x 128], FP16 operands in shared memory, fp32 in TMEM
//   P = 2^(S f - m), BF16, written over S in TMEM
//   O += P V    [128 x D], BF16, A = P from TMEM, B = V as it lies (tokens x D)
// The two tiles take turns: while one's scores go through the softmax the other's
// products run.  Beside the products and the softmax the decoding counts (a third
// of the instructions), hence two forms:
// * Keys become FP16 by the hardware's conversion, times 2^(e - ref + 13) with ref
//   the largest scale of the step: exact for scales down to 2^-36 of it.  Queries
//   become FP16 times a power of two per row (largest element at 2^14).  Both
//   powers go back in the factor f of the row and step.
// * Values become BF16, since P wants its exponents: E2M1 magnitude bits placed in
//   a BF16 read as the value times 2^-126, and one or two exact multiplies by
//   powers of two apply the scale.
// So the only roundings are P's to BF16 and the fp32 sums.  A row that sees few keys
// (kRestKeys) has no others for their roundings to average out with: in its unit
// (REST) P has a second BF16 term, what the rounding left, and its products are added.
// The running maximum follows with slack: O is rescaled only when a row's maximum
// has grown by more than 2^8, P staying below 2^8 meanwhile.
//
// A step does 512 R D flops for R rows and brings 136 D bytes: operations are the
// floor.  4096 tokens x 16384 keys, 32 heads over 8 of 128: 683 us, 1408 TFLOP/s
// (1911 measured for a plain BF16 product).  A step takes 1.8 us, of which the
// products 58%; the rest is the chain scores -> softmax -> P of either tile, slowed by
// the decoders, with which it shares the issue slots (64% of them taken).  Short
// prompts pay for units beside their steps: 12 ragged requests of up to 700 tokens x
// 1500 keys 33.8 us, 128 tokens x 128 keys 12.0.
//
//   warps 0-3, 4-7   softmax of tile 0, 1 (a thread per row): stage Q, scores ->
//                    probabilities, output
//   warps 8-15       decoders: codes -> FP16 key and BF16 value tiles, two slots each
//   warp 16          TMEM owner and MMA issuer
//   warp 17          copies of the cache chunks, two slots
#include "kv_walk.cuh"
#include "kv.cuh"

#include <atomic>
#include <cmath>
#include <type_traits>

namespace a4w4 {

namespace {

constexpr int kKeys = 128;                    // keys of a step
constexpr int kRows = 256;                    // rows of a unit
// Steps of a worker, at least.  2 and 4: 128 tokens x 128 keys 12.0 and 20.4 us, 8 ragged
// x 100 x 1000 19.6 and 30.4; 1 is like 2 (11.6, 19.7).
constexpr uint32_t kLeastSteps = 2;
// What a part adds to a join, in steps (128 KB through one SM).  A unit of n steps in runs of s takes s + 0.7 n / s
// steps, so runs have sqrt(0.7 n) steps at least.  0, 0.4, 0.7, 1.2: 64 tokens x 8192 keys 48.0, 45.2, 37.9, 42.2 us;
// where there is work for more than that (128 x 8192, 50 x 50000) it makes no difference.
constexpr float kJoinCost = 0.7f;
// What a unit costs beside its steps (queries, output), in steps: so many places of
// the line before its first step hold no work.  1, 2, 3: 12 ragged prompts x 700
// tokens 38.3, 33.8, 35.3 us, 4 x 512 x 512 39.1, 36.9, 38.4, 3 ragged x 3205 52.1,
// 41.6, 41.1 (0, with slower joins: 12 ragged prompts 46.8 where 2 took 39.0).
constexpr int kUnitCost = 2;
constexpr int kMaxCtas = 512;
// Keys that a unit's first row sees, up to which P has two terms: a step's, so that the
// answers hang on what a row sees and not on the table's width.  None, 128, 512: 12
// ragged prompts 32.3, 33.8, 39.5 us, 4096 tokens x 4096 keys 162, 168, 186, 3 ragged x
// 3205 39.0, 41.3, 45.6 (their steps take up to 1.4 times as long, which the cut does
// not know); 4 x 512 x 512 36.9 with 128, 38.9 with 512.
constexpr int kRestKeys = 128;

template <int D>
struct PreCfg {
  using Ch = KvChunk<D>;
  static constexpr int DEC_WARPS = 8;
  static constexpr int THREADS = 32 * (8 + DEC_WARPS + 4);         // five warpgroups, the last one half used
  // registers a thread, by warpgroup: softmax, decoders, the rest; together what the CTA was launched with.  The compiler
  // reports 324 bytes of spill stores and 488 of loads at D = 128, 332 and 476 at D = 64 (all roles together)
  static constexpr int REGS = 96, REGS_SOFTMAX = 160, REGS_DECODE = 56, REGS_REST = 48;
  static_assert(256 * REGS_SOFTMAX + 256 * REGS_DECODE + 128 * REGS_REST <= THREADS * REGS, "register split");
  static constexpr int ATOM = 128 * 128;                         // 128 rows x 64 BF16, 128-byte swizzle
  static constexpr int ATOMS = D / 64;
  static constexpr int TILE = ATOMS * ATOM;                      // 128 rows x D
  static constexpr int RAW = 8 * Ch::kBytes;                     // a step's chunks
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_K = OFF_Q + 2 * TILE;
  static constexpr int OFF_V = OFF_K + 2 * TILE;
  static constexpr int OFF_RAW = OFF_V + 2 * TILE;
  static constexpr int OFF_BAR = OFF_RAW + 2 * RAW;
  // raw full, empty x 2; K full, empty x 2; V full, empty x 2; Q full, S full, P half, P full, O full per tile; drain
  static constexpr int NBAR = 12 + 10 + 1;
  static constexpr int OFF_MISC = OFF_BAR + NBAR * 8;
  static constexpr int SMEM = OFF_MISC + 64 + 48;
  static constexpr int SCOL = 0, OCOL = 256;                     // TMEM columns: S of the tiles, then O
  static constexpr int TMEM_COLS = 512;
  static constexpr int PART = kRows * (D + 2);                   // floats of a stored part: O, then m and l
  static_assert(SMEM <= 232448 && OFF_RAW % 16 == 0 && OFF_BAR % 8 == 0, "shared memory");
};

// 32 columns of this warp's lanes; the values may be used after tmem_wait_ld() on them.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}
// Orders the uses of r[0..15] after the wait.
__device__ __forceinline__ void tmem_landed16(uint32_t* r) {
  asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                    "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
template <int N>
__device__ __forceinline__ void tmem_wait_ld(uint32_t* r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < N; i += 16) tmem_landed16(r + i);
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}
// Two fp32 operations at a time.
__device__ __forceinline__ uint64_t pair_f32(uint32_t lo, uint32_t hi) {
  return static_cast<uint64_t>(hi) << 32 | lo;
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(N));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};"
      :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]),
         "r"(v[8]), "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* v) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void st_global_v8(void* at, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                             uint32_t g, uint32_t h) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
               :: "l"(at), "r"(a), "r"(b), "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h) : "memory");
}

// D (TMEM) (+)= A B, descriptors as their two words.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a_lo, uint32_t a_hi, uint32_t b_lo, uint32_t b_hi,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\tsetp.ne.b32 p, %6, 0;\n\t"
      "mov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}"
      :: "r"(d), "r"(a_lo), "r"(a_hi), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b_lo, uint32_t b_hi, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\tsetp.ne.b32 p, %5, 0;\n\t"
      "mov.b64 b, {%2, %3};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}"
      :: "r"(d), "r"(a), "r"(b_lo), "r"(b_hi), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
// Shared-memory descriptor of a B operand stored K x N with N contiguous
// (MN-major, 128-byte swizzle): blocks of 64 N elements `lead` bytes apart,
// groups of 8 K rows 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr, uint32_t lead) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(lead >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}
// FP16 A and B, both K-major (idesc_bf16's with the formats 0).
__device__ __forceinline__ uint32_t idesc_f16(uint32_t n) { return idesc_bf16(n) & ~(1u << 7 | 1u << 10); }
constexpr uint32_t kIdescBMajorN = 1u << 16;   // instruction descriptor: B is MN-major

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
// Eight E2M1 codes (nibble k of w) -> BF16x2 words of elements (k, k + 4), k = 0..3, times 2^-126: magnitude bits
// to 6..8 of a BF16, sign to 15.
__device__ __forceinline__ uint4 e2m1x8_to_bf16x2(uint32_t w) {
  constexpr uint32_t kMag = 0x01C001C0u, kSign = 0x80008000u;
  return make_uint4(((w << 6) & kMag) | ((w << 12) & kSign), ((w << 2) & kMag) | ((w << 8) & kSign),
                    ((w >> 2) & kMag) | ((w << 4) & kSign), ((w >> 6) & kMag) | (w & kSign));
}
__device__ __forceinline__ uint4 mul_bf16x8(uint4 o, uint32_t f) {
  return make_uint4(mul_bf16x2(o.x, f), mul_bf16x2(o.y, f), mul_bf16x2(o.z, f), mul_bf16x2(o.w, f));
}

// sum over k = 0 .. n - 1 of floor((a k + b) / M) modulo 2^32; a n + b < 2^32
template <uint32_t M>
__device__ __forceinline__ uint32_t floor_sum(uint32_t n, uint32_t a, uint32_t b) {
  if (n == 0) return 0;
  // the first round, whose divisor is a constant, apart: the others divide slowly
  uint32_t s = (n & 1 ? (n - 1) / 2 * n : n / 2 * (n - 1)) * (a / M) + n * (b / M), m = a % M;
  const uint32_t y0 = m * n + b % M;
  if (y0 < M) return s;
  n = y0 / M;
  b = y0 % M;
  a = M;
  while (n > 0) {
    const uint32_t qa = a / m, qb = b / m;
    s += (n & 1 ? (n - 1) / 2 * n : n / 2 * (n - 1)) * qa + n * qb;
    a -= qa * m;
    b -= qb * m;
    const uint32_t y = a * n + b;
    if (y < m) break;
    n = y / m;
    b = y - n * m;
    const uint32_t x = m;
    m = a;
    a = x;
  }
  return s;
}

// A request's units: blocks of `tq` new tokens (all their group's rows), each
// with the keys that its last token sees.
struct Blocks {
  int len, all, rows, row0, tq, n;             // n: blocks
  __device__ __forceinline__ Blocks() {}
  __device__ __forceinline__ Blocks(const KvRequest& r, int tq_) {
    len = r.len; all = r.all; rows = r.rows; row0 = r.row0;
    tq = tq_;
    n = (rows + tq - 1) / tq;
  }
  __device__ __forceinline__ int steps(int k) const {
    const int seen = len - all + min((k + 1) * tq, rows);
    return max(1, (seen + kKeys - 1) / kKeys);
  }
  // places of blocks 0 .. k - 1 on the line, k < n
  __device__ __forceinline__ uint32_t before(int k) const {
    const int base = len - all;
    // the first blocks may see nothing: one empty step each
    const int none = base < 0 ? min(k, -base / tq) : 0;
    return k * kUnitCost + none + floor_sum<kKeys>(k - none, tq, static_cast<uint32_t>(base + (none + 1) * tq + kKeys - 1));
  }
  __device__ __forceinline__ uint32_t total() const { return n > 0 ? before(n - 1) + kUnitCost + steps(n - 1) : 0u; }
};

// A walk along the CTA's run: one piece (a run of one unit's steps) at a time.
struct PreWalk {
  Blocks q;
  int b, h, k, t, n;                           // request, head, block, first step of the piece, steps of the unit
  int left;                                    // places of the run from the piece's first step on
  __device__ __forceinline__ int steps() const { return min(left, n - t); }
  __device__ __forceinline__ void next(const KvAttentionArgs& p) {
    left -= steps();
    t = 0;
    if (left <= 0) return;
    if (++k == q.n) {
      k = 0;
      if (++h == p.Hkv) {
        h = 0;
        do { q = Blocks(kv_request(p, ++b), q.tq); } while (q.n == 0);
      }
    }
    n = q.steps(k);
    left -= kUnitCost;
  }
  // whether the unit's first row, and so some row, sees few keys: then P has two terms
  __device__ __forceinline__ bool few_keys() const { return q.len - q.all + k * q.tq < kRestKeys; }
  // rows of the unit
  __device__ __forceinline__ int rows(int G) const { return min(q.tq, q.rows - k * q.tq) * G; }
};

template <int D>
__global__ void __launch_bounds__(PreCfg<D>::THREADS, 1) a4w4_kv_prefill_kernel(const KvAttentionArgs p) {
  using Cf = PreCfg<D>;
  using Ch = KvChunk<D>;
  constexpr int J = Ch::J;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t base = smem_u32(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t bar0 = base + Cf::OFF_BAR;
  auto raw_full = [&](int s) { return bar0 + 8u * s; };
  auto raw_empty = [&](int s) { return bar0 + 8u * (2 + s); };
  auto k_full = [&](int s) { return bar0 + 8u * (4 + s); };
  auto k_empty = [&](int s) { return bar0 + 8u * (6 + s); };
  auto v_full = [&](int s) { return bar0 + 8u * (8 + s); };
  auto v_empty = [&](int s) { return bar0 + 8u * (10 + s); };
  auto q_full = [&](int w) { return bar0 + 8u * (12 + w); };
  auto s_full = [&](int w) { return bar0 + 8u * (14 + w); };
  auto p_full = [&](int w) { return bar0 + 8u * (16 + w); };
  auto o_full = [&](int w) { return bar0 + 8u * (18 + w); };
  auto p_half = [&](int w) { return bar0 + 8u * (20 + w); };
  const uint32_t drain = bar0 + 8u * 22;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cf::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cf::OFF_MISC + 8);
  volatile int* never = abort_flag + 1;
  volatile int* last_flag = abort_flag + 2;
  PreWalk* start_at = reinterpret_cast<PreWalk*>(smem + Cf::OFF_MISC + 64);
  static_assert(sizeof(PreWalk) == 48 && Cf::SMEM <= 232448, "shared memory");
  // largest key scale of a step; a slot is used again four steps later, when its readers are past the step after
  int* key_ref = reinterpret_cast<int*>(smem + Cf::OFF_MISC + 40);
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(raw_full(s), 1);
      mbar_init(raw_empty(s), Cf::DEC_WARPS);
      mbar_init(k_full(s), Cf::DEC_WARPS);
      mbar_init(k_empty(s), 1);
      mbar_init(v_full(s), Cf::DEC_WARPS);
      mbar_init(v_empty(s), 1);
      mbar_init(q_full(s), 4);
      mbar_init(s_full(s), 1);
      mbar_init(p_half(s), 4);
      mbar_init(p_full(s), 4);
      mbar_init(o_full(s), 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never = 0;
    fence_barrier_init();
    if ((base & 1023u) != 0) {                 // the swizzled tiles need it
      *abort_flag = 1;
      atomicOr(p.status, kStatusTimeout);
    }
  }
  const int G = p.Hq / p.Hkv, tq = kRows / G;
  griddep_wait();
  griddep_launch_dependents();

  KvShare share;
  KvStart start;
  auto places = [&](const KvRequest& r) -> uint32_t { return Blocks(r, tq).total() * p.Hkv; };
  auto longest_unit = [&](const KvRequest& r) -> uint32_t { const Blocks q(r, tq); return q.steps(q.n - 1); };
  auto least = [](uint32_t steps) { return max(kLeastSteps, static_cast<uint32_t>(sqrtf(kJoinCost * steps))); };
  if (!kv_locate<Cf::THREADS, 1, 0>(p, places, longest_unit, 0, least, 1, reinterpret_cast<uint32_t*>(smem + Cf::OFF_Q),
                                    share, start))
    return;
  const uint32_t cta = blockIdx.x;
  if (warp == 0) {
    const Blocks q(start.req, tq);
    const uint32_t per = start.places / p.Hkv;                   // q.total()
    const int h = start.rest / per;
    const uint32_t rest = start.rest - h * per;
    // the block that holds step `rest`: 32 candidates at a time
    int lo = 0, hi = q.n;                      // before(lo) <= rest, and before(hi) > rest or hi == n
    uint32_t lo_at = 0;                        // before(lo)
    while (hi - lo > 1) {
      const int stride = (hi - lo + 31) / 32;
      const int c = lo + stride * lane;
      const uint32_t at = q.before(min(c, q.n - 1));
      const uint32_t in = __ballot_sync(0xFFFFFFFFu, c < hi && at <= rest);
      const int top = 31 - __clz(in);          // lane 0 is always in
      lo += stride * top;
      lo_at = __shfl_sync(0xFFFFFFFFu, at, top);
      hi = min(hi, lo + stride);
    }
    if (lane == 0) {
      const int place = rest - lo_at;
      PreWalk w;
      w.b = start.b;
      w.q = q;
      w.h = h;
      w.k = lo;
      w.n = q.steps(lo);
      w.t = max(0, place - kUnitCost);
      w.left = static_cast<int>(share.first(cta + 1) - share.first(cta)) - max(0, kUnitCost - place);
      *start_at = w;
    }
  }
  if (warp == 16) {
    tmem_alloc(smem_u32(tmem_slot), Cf::TMEM_COLS);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PreWalk w = *start_at;
  const unsigned long long drain_ns = p.wait_ns > 100000000ull ? p.wait_ns : 100000000ull;
  auto wait = [&](uint32_t bar, uint32_t parity) { return mbar_wait(bar, parity, abort_flag, p.wait_ns, p.status); };

  if (warp < 8) {
    // ---------------- softmax ----------------
    regs_up<Cf::REGS_SOFTMAX>();
    const int tile = warp >> 2, quad = warp & 3, r = tile * 128 + quad * 32 + lane;
    const uint32_t lane_base = static_cast<uint32_t>(quad * 32) << 16;
    const uint32_t s_col = tmem + lane_base + Cf::SCOL + tile * 128, o_col = tmem + lane_base + Cf::OCOL + tile * D;
    uint32_t it = 0;                           // steps so far
    float* parts = reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + kTickets * 4);
    uint32_t s_phase = 0, o_phase = 0;
    // output in whole sectors, with half the stores: 128 tokens x 128 keys 12.9 -> 12.3 us, 16 x 64 x 512 37.5 -> 36.7;
    // at D = 64 12 ragged prompts take 33.1 instead of 32.4
    const bool wide_out = D == 128 && (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
    int q_pow = 0;                             // the power of two of this thread's row of Q
    // ---- the warp's 32 rows of a unit's Q tile: C lanes to a row, 32 / C rows at a time; a piece ahead of the rest,
    // while the last products run ----
    auto stage_queries = [&](const PreWalk& u) {
      const int R = u.rows(G), first_tok = u.k * tq;
      if (tile * 128 >= R) return;
      constexpr int C = D / 8, AT = 32 / C, BATCH = 32 / AT;
      const int c = lane % C;
#pragma unroll 1
      for (int j0 = 0; j0 < 32 / AT; j0 += BATCH) {
        uint4 v[BATCH];
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          const int rt = tile * 128 + quad * 32 + (j0 + j) * AT + lane / C, qj = p.row_of(rt);
          v[j] = rt < R ? ld_global_nc_v4(p.q + (static_cast<long long>(u.q.row0) + first_tok + qj) * p.q_stride +
                                          (u.h * G + rt - qj * G) * D + c * 8)
                        : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int j = 0; j < BATCH; ++j) {
          uint32_t top = max_abs_bf16x2(max_abs_bf16x2(v[j].x, v[j].y), max_abs_bf16x2(v[j].z, v[j].w)) & 0x7FFF7FFFu;
          uint32_t e = max(top & 0xFFFFu, top >> 16) >> 7;
#pragma unroll
          for (int s = C / 2; s > 0; s >>= 1) e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, s));
          const int k = min(141 - static_cast<int>(e), 127);
          const float fk = pow2i_normal(k);
          auto two = [&](uint32_t b) { return pack_f16(__uint_as_float(b << 16) * fk, __uint_as_float(b & 0xFFFF0000u) * fk); };
          const int rr = quad * 32 + (j0 + j) * AT + lane / C;
          *reinterpret_cast<uint4*>(smem + Cf::OFF_Q + tile * Cf::TILE + (c >> 3) * Cf::ATOM + rr * 128 +
                                    (((c & 7) ^ (rr & 7)) << 4)) = make_uint4(two(v[j].x), two(v[j].y), two(v[j].z), two(v[j].w));
          const int mine = __shfl_sync(0xFFFFFFFFu, k, (lane % AT) * C);
          if (lane / AT == j0 + j) q_pow = mine;               // this thread's own row
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(q_full(tile));
    };
    if (w.left > 0) stage_queries(w);
    bool ok = true;                            // a warp that gave up goes on through the joins, for their barriers
    for (; w.left > 0; w.next(p)) {
      const int R = w.rows(G);
      const bool active = tile * 128 < R;
      const int first_tok = w.k * tq, qi = p.row_of(r), hq = w.h * G + r - qi * G;
      const long long row = static_cast<long long>(w.q.row0) + first_tok + qi;
      float m = kNoMax, off = 3.0e38f, l = 0.f;   // running maximum in log2 units, -m, sum
      const int row_pow = q_pow;
      if (active && ok) {
        const int seen = r < R ? w.q.len - w.q.all + first_tok + qi + 1 : 0;
        const int n = w.steps();
        auto softmax = [&](auto two_terms) {
          constexpr bool REST = decltype(two_terms)::value;
          for (int i = 0; i < n; ++i) {
            ok = __all_sync(0xFFFFFFFFu, wait(s_full(tile), s_phase));
            if (!ok) break;
            s_phase ^= 1;
            tc_fence_after();
            const int k0 = (w.t + i) * kKeys;
            // score -> log2 units; positive, so that a masked score stays -infinity
            const int ref = *reinterpret_cast<volatile int*>(key_ref + ((it + i) & 3));
            const float f = fmaxf(p.sm_scale * 1.4426950408889634f * pow2i_normal(max(-126, min(127, ref - 140 - row_pow))), 1e-44f);
            const bool edge = __any_sync(0xFFFFFFFFu, k0 + kKeys > seen);
            uint32_t x[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld32(s_col + 32 * c, x + 32 * c);
            tmem_wait_ld<128>(x);
            if (edge) {
              const int k1 = seen - k0;                             // columns that the row sees
#pragma unroll
              for (int u = 0; u < 128; ++u)
                if (u >= k1) x[u] = 0xFF800000u;                    // -infinity
            }
            float top[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              top[c] = max3(__uint_as_float(x[c]), __uint_as_float(x[c + 4]), __uint_as_float(x[c + 8]));
#pragma unroll
              for (int u = c + 12; u < 124; u += 8) top[c] = max3(top[c], __uint_as_float(x[u]), __uint_as_float(x[u + 4]));
              top[c] = fmaxf(top[c], __uint_as_float(x[c + 124]));
            }
            const float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * f;
            // the maximum follows once it is 2^8 ahead
            const bool grow = m == kNoMax ? mx > m : mx - m > 8.f;
            float a = 1.f;
            if (grow) {
              a = ex2(m - mx);
              m = mx;
              off = -m;
              l *= a;
            }
            if (i > 0 && __any_sync(0xFFFFFFFFu, grow)) {
#pragma unroll 1
              for (int c = 0; c < D / 16; ++c) {
                uint32_t y[16];
                tmem_ld16(o_col + 16 * c, y);
                tmem_wait_ld<16>(y);
#pragma unroll
                for (int u = 0; u < 16; ++u) y[u] = __float_as_uint(__uint_as_float(y[u]) * a);
                tmem_st16(o_col + 16 * c, y);
              }
            }
            const uint64_t f2 = pair_f32(__float_as_uint(f), __float_as_uint(f));
            const uint64_t off2 = pair_f32(__float_as_uint(off), __float_as_uint(off));
            uint64_t sum0 = 0, sum1 = 0;                            // two pairs of partial sums
#pragma unroll
            for (int c = 0; c < 8; ++c) {
              uint32_t y[8], rest[8];
#pragma unroll
              for (int u = 0; u < 8; ++u) {
                const uint64_t z = fma_f32x2(pair_f32(x[16 * c + 2 * u], x[16 * c + 2 * u + 1]), f2, off2);
                const float e0 = ex2(__uint_as_float(static_cast<uint32_t>(z)));
                const float e1 = ex2(__uint_as_float(static_cast<uint32_t>(z >> 32)));
                const uint64_t e = pair_f32(__float_as_uint(e0), __float_as_uint(e1));
                if (u & 1) sum1 = add_f32x2(sum1, e); else sum0 = add_f32x2(sum0, e);
                y[u] = pack_bf16(e0, e1);
                if constexpr (REST) rest[u] = pack_bf16(e0 - __uint_as_float(y[u] << 16), e1 - __uint_as_float(y[u] & 0xFFFF0000u));
              }
              tmem_st8(s_col + 8 * c, y);
              if constexpr (REST) tmem_st8(s_col + 64 + 8 * c, rest);
              if (c == 3) {                                         // the products of the first 64 keys may start
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_half(tile));
              }
            }
            sum0 = add_f32x2(sum0, sum1);
            l += __uint_as_float(static_cast<uint32_t>(sum0)) + __uint_as_float(static_cast<uint32_t>(sum0 >> 32));
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(p_full(tile));
          }
        };
        if (w.few_keys()) softmax(std::true_type{}); else softmax(std::false_type{});
      }
      // the unit's scores are done, so Q's place is free for the next one's
      {
        PreWalk ahead = w;
        ahead.next(p);
        if (ok && ahead.left > 0) stage_queries(ahead);
      }
      if (active && ok) {
        ok = __all_sync(0xFFFFFFFFu, wait(o_full(tile), o_phase));
        o_phase ^= 1;
        tc_fence_after();
      }
      it += w.steps();
      // ---- the unit's output, or the part of it ----
      const bool whole = w.t == 0 && w.steps() == w.n;
      const uint32_t u0 = share.first(cta + 1) - w.left - w.t;    // the unit's first step on the line
      float* mine = parts + static_cast<size_t>(2 * cta + (share.first(cta) < u0 ? 1 : 0)) * Cf::PART;
      // dimensions 64 a .. + 63 of the thread's row, times `by`; column g * 8 + e of the block (x) is dimension
      // 64 a + 2 g + {0, 32, 1, 33, 16, 48, 17, 49}[e]
      auto write_out = [&](int a, const uint32_t* x, float by) {
        auto at = [&](int n) {
          return by * __uint_as_float(x[n % 16 / 2 * 8 + (n / 16 == 0 ? 0 : n / 16 == 2 ? 1 : n / 16 == 1 ? 4 : 5) + 2 * (n % 2)]);
        };
        uint16_t* dst = p.out + (row * p.Hq + hq) * D + 64 * a;
        auto two = [&](int n) { return pack_bf16(at(n), at(n + 1)); };
#pragma unroll
        for (int n = 0; n < 64; n += 16) {
          if (wide_out) {
            st_global_v8(dst + n, two(n), two(n + 2), two(n + 4), two(n + 6), two(n + 8), two(n + 10), two(n + 12), two(n + 14));
          } else {
            *reinterpret_cast<uint4*>(dst + n) = make_uint4(two(n), two(n + 2), two(n + 4), two(n + 6));
            *reinterpret_cast<uint4*>(dst + n + 8) = make_uint4(two(n + 8), two(n + 10), two(n + 12), two(n + 14));
          }
        }
      };
      auto write_lse = [&](float mm, float ll) {
        if (p.lse != nullptr) p.lse[row * p.Hq + hq] = ll == 0.f ? -INFINITY : fmaf(mm, 0.6931471805599453f, logf(ll));
      };
      if (active) {
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int a = 0; a < D / 64; ++a) {
          uint32_t x[64];
          tmem_ld32(o_col + 64 * a, x);
          tmem_ld32(o_col + 64 * a + 32, x + 32);
          tmem_wait_ld<64>(x);
          if (r < R) {
            if (whole) {
              write_out(a, x, inv);
            } else {
              // a part: pieces of 4 columns, the rows' side by side, so that a warp writes 512 bytes in a run
              uint4* dst = reinterpret_cast<uint4*>(mine) + a * 16 * kRows + r;
#pragma unroll
              for (int u = 0; u < 16; ++u) dst[u * kRows] = make_uint4(x[4 * u], x[4 * u + 1], x[4 * u + 2], x[4 * u + 3]);
            }
          }
        }
        if (r < R) {
          const float mm = fmaxf(m, kNoMax);
          if (whole) write_lse(mm, l);
          else *reinterpret_cast<float2*>(mine + kRows * D + 2 * r) = make_float2(mm, l);
        }
      }
      if (!whole) {
        // ---- the last part to arrive joins a cut unit (softmax warps only), a thread per row ----
        const int c0 = share.holder(u0), np = share.holder(u0 + w.n - 1) - c0 + 1;
        named_bar_sync(1, 256);
        int* ticket = static_cast<int*>(p.ws) + c0;
        if (tid == 0) *last_flag = draw_ticket(ticket) == np - 1;
        named_bar_sync(1, 256);
        if (*last_flag && active) {            // whole warps, the lanes beyond the rows go along
          const size_t head = share.first(c0) < u0 ? Cf::PART : 0;
          const int own = cta - c0, rr = min(r, R - 1);
#pragma unroll 1
          for (int a = 0; a < D / 64; ++a) {
            float mm = kNoMax, ll = 0.f;
            float y[64];
#pragma unroll
            for (int u = 0; u < 64; ++u) y[u] = 0.f;
#pragma unroll 1
            for (int k = 0; k < np; ++k) {                        // in the parts' order, whoever joins
              uint32_t x[64];
              float2 q;
              if (k == own) {                                     // still in TMEM
                tmem_ld32(o_col + 64 * a, x);
                tmem_ld32(o_col + 64 * a + 32, x + 32);
                tmem_wait_ld<64>(x);
                q = make_float2(fmaxf(m, kNoMax), l);
              } else {
                const float* src = parts + static_cast<size_t>(2 * (c0 + k)) * Cf::PART + (k == 0 ? head : 0);
                q = __ldcg(reinterpret_cast<const float2*>(src + kRows * D) + rr);
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                  const uint4 v = __ldcg(reinterpret_cast<const uint4*>(src) + (a * 16 + u) * kRows + rr);
                  x[4 * u] = v.x; x[4 * u + 1] = v.y; x[4 * u + 2] = v.z; x[4 * u + 3] = v.w;
                }
              }
              const float top = fmaxf(mm, q.x), f = ex2(mm - top), e = ex2(q.x - top);
              mm = top;
              ll = fmaf(q.y, e, ll * f);
#pragma unroll
              for (int u = 0; u < 64; ++u) y[u] = fmaf(__uint_as_float(x[u]), e, y[u] * f);
            }
            if (r < R) {
              uint32_t x[64];
#pragma unroll
              for (int u = 0; u < 64; ++u) x[u] = __float_as_uint(y[u]);
              write_out(a, x, ll == 0.f ? 0.f : 1.f / ll);
              if (a == 0) write_lse(mm, ll);
            }
          }
        }
        if (*last_flag) {
          if (tid == 0) *ticket = 0;
        }
        named_bar_sync(1, 256);                // the flag is free again
      }
    }
  } else if (warp < 16) {
    // ---------------- decoders ----------------
    regs_down<Cf::REGS_DECODE>();
    const int dw = warp - 8;                   // chunk of the step
    uint32_t it = 0;                           // steps so far
    // the first cells: a wait that a limit shorter than the hardware's suspension of a waiting warp ends too (in the
    // loops this form of waiting costs 3%)
    bool ok = w.left <= 0 || __all_sync(0xFFFFFFFFu, kv_wait(raw_full(0), 0, abort_flag, p.wait_ns, p.status));
    for (; w.left > 0 && ok; w.next(p)) {
      const int n = w.steps();
      for (int i = 0; i < n; ++i, ++it) {
        const int s = it & 1;
        const uint32_t ph = it >> 1 & 1;
        if (!(ok = __all_sync(0xFFFFFFFFu, wait(raw_full(s), ph)))) break;
        if (!(ok = __all_sync(0xFFFFFFFFu, wait(k_empty(s), ph ^ 1)))) break;
        const uint8_t* raw = smem + Cf::OFF_RAW + s * Cf::RAW;
        const uint8_t* ch = raw + dw * Ch::kBytes;
        const int tok0 = (w.t + i) * kKeys;
        // the step's largest key scale: 4 bytes a time, lanes over the 8 chunks
        uint32_t top = 0;
#pragma unroll
        for (int u = 0; u < J; ++u) {
          const int word = u * 32 + lane, r16 = word / (4 * J), at = word % (4 * J) * 4;      // chunk, byte of its scales
          const uint32_t x = *reinterpret_cast<const uint32_t*>(raw + r16 * Ch::kBytes + Ch::kKeyScales + at);
          const int tok = tok0 + r16 * 16 + at / J;
#pragma unroll
          for (int bb = 0; bb < 4; ++bb) {
            const uint32_t e = x >> (8 * bb) & 0xFFu;
            if (tok + bb / J < w.q.len) top = max(top, e);
          }
        }
        const int ref = static_cast<int>(__reduce_max_sync(0xFFFFFFFFu, top));
        if (dw == 0 && lane == 0) *reinterpret_cast<volatile int*>(key_ref + (it & 3)) = ref;
        // keys: lane = piece t of tokens r, r + 8; a quarter of the warp holds rows x and x + 4, which the swizzle
        // spreads over all banks
        {
          uint8_t* kt = smem + Cf::OFF_K + s * Cf::TILE;
          const int t = lane & 3, r8 = (lane >> 2 & 1) * 4 + (lane >> 3);
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            const int r = r8 + 8 * hh, row = dw * 16 + r;
            uint32_t wd[J], sc;
            if constexpr (J == 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(ch + Ch::key_word(r, 0, t));
              wd[0] = v.x; wd[1] = v.y; wd[2] = v.z; wd[3] = v.w;
              sc = *reinterpret_cast<const uint32_t*>(ch + Ch::kKeyScales + r * J);
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(ch + Ch::key_word(r, 0, t));
              wd[0] = v.x; wd[1] = v.y;
              sc = *reinterpret_cast<const uint16_t*>(ch + Ch::kKeyScales + r * J);
            }
#pragma unroll
            for (int j = 0; j < J; ++j) {
              // 2^(e - ref + 13), in FP16 down to 2^-24 (cells beyond the length: anything)
              const int k = static_cast<int>(sc >> (8 * j) & 0xFFu) - ref + 140;
              const float fk = __uint_as_float(static_cast<uint32_t>(max(k, 0)) << 23);
              const uint32_t f2 = pack_f16(fk, fk);
              uint32_t x[4];
              e2m1x8_to_f16x2(wd[j], x);
              *reinterpret_cast<uint4*>(kt + (j >> 1) * Cf::ATOM + row * 128 + ((((j & 1) * 4 + t) ^ (row & 7)) << 4)) =
                  make_uint4(mul_f16x2(x[0], f2), mul_f16x2(x[1], f2), mul_f16x2(x[2], f2), mul_f16x2(x[3], f2));
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(k_full(s));
        if (!(ok = __all_sync(0xFFFFFFFFu, wait(v_empty(s), ph ^ 1)))) break;
        // values: lane 4 g + t = 16-byte piece g of tokens 2t, 2t + 1 of each half; tokens beyond the length are zero
        {
          uint8_t* vt = smem + Cf::OFF_V + s * Cf::TILE;
          const int g = lane >> 2, t = lane & 3;
#pragma unroll
          for (int hh = 0; hh < 2; ++hh) {
            uint32_t run[2][J / 2];
            if constexpr (J == 4) {
              const uint4 v = *reinterpret_cast<const uint4*>(ch + Ch::kValues + hh * 4 * D + lane * 16);
              run[0][0] = v.x; run[0][1] = v.y; run[1][0] = v.z; run[1][1] = v.w;
            } else {
              const uint2 v = *reinterpret_cast<const uint2*>(ch + Ch::kValues + hh * 4 * D + lane * 8);
              run[0][0] = v.x; run[1][0] = v.y;
            }
#pragma unroll
            for (int o = 0; o < 2; ++o) {
              const int r = hh * 8 + 2 * t + o, row = dw * 16 + r;
              uint32_t sc;
              if constexpr (J == 4) sc = *reinterpret_cast<const uint32_t*>(ch + Ch::kValueScales + r * J);
              else sc = *reinterpret_cast<const uint16_t*>(ch + Ch::kValueScales + r * J);
              if (tok0 + dw * 16 + r >= w.q.len) {
                sc = 0u;
#pragma unroll
                for (int q4 = 0; q4 < J / 2; ++q4) run[o][q4] = 0u;
              }
              uint4 y[J / 2];
#pragma unroll
              for (int q4 = 0; q4 < J / 2; ++q4) y[q4] = e2m1x8_to_bf16x2(run[o][q4]);
              // word q4: bytes of row tiles 4 q4 ..+3: 32-blocks 2 q4 (low halves) and 2 q4 + 1 (high halves), so the
              // factor's halves are the two blocks' 2^(e - 1); for e > 127 2^126 first, then 2^(e - 127)
              uint32_t plus = 0x3F003F00u;
              if ((sc & 0x80808080u) != 0u) {
#pragma unroll
                for (int q4 = 0; q4 < J / 2; ++q4) y[q4] = mul_bf16x8(y[q4], 0x7E807E80u);
                plus = 0u;
              }
#pragma unroll
              for (int q4 = 0; q4 < J / 2; ++q4) {
                uint32_t f2 = __byte_perm(sc, 0u, q4 ? 0x4342 : 0x4140) * 128u + plus;
                if (plus == 0u) f2 = max(f2 & 0xFFFFu, 0x40u) | max(f2 >> 16, 0x40u) << 16;    // 2^-127 for e = 0
                *reinterpret_cast<uint4*>(vt + q4 * Cf::ATOM + row * 128 + ((g ^ (row & 7)) << 4)) = mul_bf16x8(y[q4], f2);
              }
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(v_full(s));
          mbar_arrive(raw_empty(s));
        }
      }
    }
  } else {
   regs_down<Cf::REGS_REST>();
   if (warp == 16) {
    // ---------------- MMA issuer: the whole warp walks, so that addresses stay in uniform registers ----------------
    const uint32_t id_s = idesc_f16(kKeys), id_o = idesc_bf16(D) | kIdescBMajorN;
    const uint64_t qd = sdesc_sw128(base + Cf::OFF_Q), kd = sdesc_sw128(base + Cf::OFF_K);
    const uint64_t vd = sdesc_mn_sw128(base + Cf::OFF_V, Cf::ATOM);
    const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
    uint32_t it = 0, q_phase = 0, p_phase = 0;                   // a phase bit per tile
    bool ok = true;
    auto sure = [&](uint32_t bar, uint32_t parity) {
      ok = __all_sync(0xFFFFFFFFu, wait(bar, parity));
      return ok;
    };
    auto scores = [&](int tile, int s) {
      const uint32_t q_lo = static_cast<uint32_t>(qd) + tile * (Cf::TILE >> 4), q_hi = static_cast<uint32_t>(qd >> 32);
      const uint32_t k_lo = static_cast<uint32_t>(kd) + s * (Cf::TILE >> 4), k_hi = static_cast<uint32_t>(kd >> 32);
      const uint32_t d = tm + Cf::SCOL + tile * 128;
      if (elect_one()) {
#pragma unroll
        for (int a = 0; a < Cf::ATOMS; ++a)
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ss(d, q_lo + (a * Cf::ATOM >> 4) + 2 * kk, q_hi, k_lo + (a * Cf::ATOM >> 4) + 2 * kk, k_hi, id_s,
                   (a | kk) ? 1u : 0u);
        mma_commit(s_full(tile));
      }
      __syncwarp();
    };
    // the products with keys 64 part .. + 63 of the step
    auto outputs = [&](int tile, int s, int part, bool rest, bool first, bool last_step, bool last_tile) {
      const uint32_t v_lo = static_cast<uint32_t>(vd) + s * (Cf::TILE >> 4), v_hi = static_cast<uint32_t>(vd >> 32);
      const uint32_t d = tm + Cf::OCOL + tile * D, a = tm + Cf::SCOL + tile * 128;
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts(d, a + 32 * part + 8 * kk, v_lo + ((4 * part + kk) * 2048 >> 4), v_hi, id_o, kk == 0 && first ? 0u : 1u);
        if (rest) {
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            mma_ts(d, a + 64 + 32 * part + 8 * kk, v_lo + ((4 * part + kk) * 2048 >> 4), v_hi, id_o, 1u);
        }
        if (last_step) mma_commit(o_full(tile));
        if (last_tile) mma_commit(v_empty(s));
      }
      __syncwarp();
    };
    for (; w.left > 0 && ok; w.next(p)) {
      const int n = w.steps(), tiles = w.rows(G) > 128 ? 2 : 1;
      const bool rest = w.few_keys();
      for (int i = 0; i <= n && ok; ++i) {
        // products of step i - 1 and scores of step i, tile after tile
        const int s = it & 1, sp = (it - 1) & 1;
        const uint32_t ph = it >> 1 & 1, php = (it - 1) >> 1 & 1;
        for (int tile = 0; tile < tiles; ++tile) {
          if (i > 0) {
            if (tile == 0 && !sure(v_full(sp), php)) break;
            if (!sure(p_half(tile), p_phase >> tile & 1)) break;
            tc_fence_after();
            outputs(tile, sp, 0, rest, i == 1, false, false);
            if (!sure(p_full(tile), p_phase >> tile & 1)) break;
            p_phase ^= 1u << tile;
            tc_fence_after();
            outputs(tile, sp, 1, rest, false, i == n, tile == tiles - 1);
          }
          if (i < n) {
            if (i == 0) {
              if (!sure(q_full(tile), q_phase >> tile & 1)) break;
              q_phase ^= 1u << tile;
            }
            if (tile == 0 && !sure(k_full(s), ph)) break;
            tc_fence_after();
            scores(tile, s);
            if (tile == tiles - 1) {
              if (elect_one()) mma_commit(k_empty(s));
              __syncwarp();
            }
          }
        }
        if (i < n) ++it;
      }
    }
    // TMEM is not released while products may still run, whoever gave up
    if (elect_one()) mma_commit(drain);
    __syncwarp();
    mbar_wait(drain, 0, never, drain_ns, p.status);
   } else if (warp == 17) {
    // ---------------- copies ----------------
    const int lg = 31 - __clz(p.page_size), chunks = p.page_size >> 4;
    const int run = min(chunks, 8);                       // chunks of a copy
    const uint64_t pol = policy_evict_last();             // other units read the same pages
    uint32_t it = 0;
    for (; w.left > 0; w.next(p)) {
      const int n = w.steps();
      bool ok = true;
      for (int i = 0; i < n; ++i, ++it) {
        const int s = it & 1;
        const int tok0 = (w.t + i) * kKeys;
        const int live = min(8, max(0, (w.q.len - tok0 + 15) >> 4));      // chunks that hold tokens
        const int c = lane * run;
        const int mine = c < live ? min(run, live - c) : 0;
        const int page = mine > 0 ? kv_page(p, w.b, (tok0 + c * 16) >> lg) : 0;
        ok = wait(raw_empty(s), (it >> 1 & 1) ^ 1);
        ok = __all_sync(0xFFFFFFFFu, ok);
        if (!ok) break;
        if (lane == 0) mbar_arrive_expect_tx(raw_full(s), live * Ch::kBytes);
        __syncwarp();
        if (mine > 0)
          bulk_g2s(base + Cf::OFF_RAW + s * Cf::RAW + c * Ch::kBytes,
                   p.cache + kv_chunk_offset<D>(page, w.h, ((tok0 >> 4) + c) & (chunks - 1), p.Hkv, chunks),
                   mine * Ch::kBytes, raw_full(s), pol);
      }
      if (!ok) break;
    }
    // every copy issued lands before the CTA's shared memory is released
    if (lane == 0)
      for (uint32_t j = it > 2 ? it - 2 : 0; j < it; ++j) mbar_wait(raw_full(j & 1), j >> 1 & 1, never, drain_ns, p.status);
   }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, Cf::TMEM_COLS);
  }
}

}  // namespace

size_t kv_prefill_ws_bytes(int D, int sms) {
  const int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  return kTickets * 4 + 2ull * ctas * kRows * (D + 2) * 4;
}

namespace {

template <int D>
int launch_one(const KvAttentionArgs& p, int grid, cudaStream_t st) {
  using Cf = PreCfg<D>;
  static std::atomic<unsigned long long> attr_done{0};
  const int rc = ensure_func_attrs(attr_done, [] {
    return cudaFuncSetAttribute(a4w4_kv_prefill_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM) ==
           cudaSuccess;
  });
  if (rc != 0) return rc;
  return launch_pdl_smem(a4w4_kv_prefill_kernel<D>, grid, Cf::THREADS, Cf::SMEM, st, p);
}

}  // namespace

int launch_kv_prefill(const KvAttentionArgs& p, int D, cudaStream_t st, int sms) {
  const int G = p.Hq / p.Hkv;
  const double unit = static_cast<double>(p.max_pages) * p.page_size / kKeys + 1 + kUnitCost;
  if (unit * most_units(p, kRows / G * G) >= kTooMany) return -1;
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  return D == 64 ? launch_one<64>(p, grid, st) : launch_one<128>(p, grid, st);
}

}  // namespace a4w4
