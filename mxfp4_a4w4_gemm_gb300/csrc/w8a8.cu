// w8a8.cu -- 8-bit product with a scale for each block of 128 (include/a4w4.h,
// a4w4_gemm_w8a8): BF16 activations quantised to E4M3 with a power-of-two scale per
// row and 128 k's, E4M3 weights with a float scale per 128 x 128 block, BF16 output.
//
//   C[m, n] = sum over b of  2^e[m,b] ws[n/128, b]  sum over k in block b of a~[m,k] w[n,k]
//
// The inner sums are tcgen05.mma.kind::f8f6f4 products of 128 k's (four MMAs of K = 32)
// into a fresh TMEM accumulator; since the weights' scales are any floats, each block's
// sum is read back, scaled and added in fp32 registers while the next block's MMAs run
// into the other accumulator.  Two kernels:
//
//   small  few tokens: 128 weight rows are the MMA's M side, 16 or 32 tokens its N
//          side, K split over the thread blocks of a cluster; activations are quantised
//          in the kernel.  Bound by latencies one after another (below).
//   large  128 tokens x 256 weight rows per tile, one persistent thread block per SM,
//          activations quantised once beforehand into tiles in the workspace; few tiles
//          run as halves whose K is shared by a cluster.
//
// Small, call after call with the weights in L2 / over a ring of weights larger than L2, so
// that they come from memory: 1 x 7168 x 4224 7.2 / 9.0 us (30 MB at a copy's rate: 4.5; the
// rest is the launch, the first block's latency and the exchange of sums, which memory's
// latency lengthens), 1 x 8448 x 7168 10.0 / 12.9, 32 x 1536 x 7168 7.5 / 7.9: set-up 0.8,
// first quantisation 1.4, products and sums of a share's four blocks 1.9, exchange 1.0,
// output 0.4.  Large:
// 2048 x 8448 x 7168 115 us, 2.15 PFLOP/s: bound by the operands' way into the SM (48 KB
// per block of K at about 64 bytes a clock) and by the loop from an accumulator read
// to the MMAs that write it again.  A pair of SMs on one tile, more accumulators,
// more and smaller stages, operands multicast to two blocks: none was faster.
#include <cfloat>

#include "device.cuh"
#include "launch.h"

namespace a4w4 {

namespace {

constexpr int kTile = 16384;                       // 128 rows x 128 bytes
constexpr int kActTile = kTile + 512;              // activation tile: codes, then 128 row scales

// ---------------------------------------------------------------------------
// E4M3

// 16 floats, already scaled -> 16 codes (round to nearest even, saturating).
__device__ __forceinline__ uint4 cvt_e4m3x16(const float* y) {
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    asm("{\n\t.reg .b16 lo, hi;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
        "mov.b32 %0, {lo, hi};\n\t}"
        : "=r"(w[q]) : "f"(y[4 * q]), "f"(y[4 * q + 1]), "f"(y[4 * q + 2]), "f"(y[4 * q + 3]));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint32_t max_abs_of(const uint4& a, const uint4& b) {
  const uint32_t m = max_abs_bf16x2(max_abs_bf16x2(max_abs_bf16x2(a.x, a.y), max_abs_bf16x2(a.z, a.w)),
                                    max_abs_bf16x2(max_abs_bf16x2(b.x, b.y), max_abs_bf16x2(b.z, b.w)));
  return m & 0x7FFF7FFFu;
}

__device__ __forceinline__ void unpack16(const uint4& a, const uint4& b, float f, float* y) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    y[2 * u] = __uint_as_float(w[u] << 16) * f;
    y[2 * u + 1] = __uint_as_float(w[u] & 0xFFFF0000u) * f;
  }
}

// One row's block of 128 over eight neighbouring lanes (16 BF16 each, a and b):
// amax 2^-e <= 448 with the smallest such e >= -126; codes of x 2^-e and the scale 2^e.
// E4M3 is a floating type, so a power of two costs no precision against amax / 448, and
// the scaling is exact.  An infinity in the block, or nothing but NaN, makes the scale NaN; a
// NaN beside numbers has no part in it and goes on as a code.
__device__ __forceinline__ uint4 quant128(const uint4& a, const uint4& b, float* scale) {
  uint32_t m = max_abs_of(a, b);
  uint32_t amax = max(m & 0xFFFFu, m >> 16);
#pragma unroll
  for (int o = 1; o < 8; o <<= 1) amax = max(amax, __shfl_xor_sync(0xFFFFFFFFu, amax, o));
  // amax = 1.f 2^(E - 127), 448 = 1.75 2^8
  const int e = max(static_cast<int>(amax >> 7) - 135 + ((amax & 0x7Fu) > 0x60u ? 1 : 0), -126);
  float y[16];
  unpack16(a, b, __uint_as_float(static_cast<uint32_t>(127 - e) << 23), y);
  *scale = (amax >> 7) == 255u ? __uint_as_float(0x7FC00000u) : __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
  return cvt_e4m3x16(y);
}

// Place of 16-byte piece c of row r in a tile of 128-byte rows, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_piece(int r, int c) {
  return static_cast<uint32_t>((r >> 3) * 1024 + (r & 7) * 128 + ((c ^ (r & 7)) << 4));
}

// Checkpoint codes [N, K] -> tiles (nt, kt) at (nt * KT + kt) * 16384.  One 16-byte piece a thread.
__global__ void __launch_bounds__(256) w8_shuffle_kernel(const uint8_t* __restrict__ w, int K, int KT, long long pieces,
                                                         uint8_t* __restrict__ w8) {
  griddep_wait();
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  const int per_row = K / 16;
  for (long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; i < pieces; i += stride) {
    const long long n = i / per_row;
    const int c = static_cast<int>(i - n * per_row);
    const uint4 v = ld_global_nc_v4(w + i * 16);
    const long long tile = (n >> 7) * KT + (c >> 3);
    *reinterpret_cast<uint4*>(w8 + tile * kTile + tile_piece(static_cast<int>(n & 127), c & 7)) = v;
  }
}

// BF16 weights: one thread block per 128 x 128 block: scale amax / 448, codes of w / scale.
__global__ void __launch_bounds__(256) w8_prepare_kernel(const uint16_t* __restrict__ w, int K, int KT,
                                                         uint8_t* __restrict__ w8, float* __restrict__ ws) {
  __shared__ uint32_t s_max[8];
  griddep_wait();
  const long long tile = blockIdx.x;
  const long long nt = tile / KT;
  const int kt = static_cast<int>(tile - nt * KT);
  uint4 v[4][2];
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 32 + (threadIdx.x >> 3), c = threadIdx.x & 7;
    const uint16_t* src = w + (nt * 128 + r) * K + kt * 128 + c * 16;
    v[i][0] = ld_global_nc_v4(src);
    v[i][1] = ld_global_nc_v4(src + 8);
    const uint32_t x = max_abs_of(v[i][0], v[i][1]);
    m = max(m, max(x & 0xFFFFu, x >> 16));
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, s_max[i]);
  const float scale = __fdiv_rn(__uint_as_float(m << 16), 448.f);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 32 + (threadIdx.x >> 3), c = threadIdx.x & 7;
    float y[16];
    unpack16(v[i][0], v[i][1], 1.f, y);
#pragma unroll
    for (int u = 0; u < 16; ++u) y[u] = scale > 0.f ? __fdiv_rn(y[u], scale) : 0.f;
    *reinterpret_cast<uint4*>(w8 + tile * kTile + tile_piece(r, c)) = cvt_e4m3x16(y);
  }
  if (threadIdx.x == 0) ws[tile] = scale;
}

// Activations -> tiles (x, kt) of 128 rows at (x * KT + kt) * kActTile; rows from M on are zero.
// Eight lanes a block of 128, so a warp reads 1 KB of one row.
__global__ void __launch_bounds__(256) w8_quant_tiles_kernel(const uint16_t* __restrict__ a, int M, int K, int KT,
                                                             long long blocks, uint8_t* __restrict__ aq) {
  griddep_wait();
  griddep_launch_dependents();
  const long long i = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x;
  const long long blk = i >> 3;
  const int c = static_cast<int>(i & 7);
  const long long row = blk / KT;
  const int kt = static_cast<int>(blk - row * KT);
  uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
  if (blk < blocks && row < M) {
    const uint16_t* src = a + row * K + kt * 128 + c * 16;
    v0 = ld_global_nc_v4(src);
    v1 = ld_global_nc_v4(src + 8);
  }
  float scale;
  const uint4 code = quant128(v0, v1, &scale);
  if (blk >= blocks) return;
  const int r = static_cast<int>(row & 127);
  uint8_t* tile = aq + ((row >> 7) * KT + kt) * kActTile;
  *reinterpret_cast<uint4*>(tile + tile_piece(r, c)) = code;
  if (c == 0) *reinterpret_cast<float*>(tile + kTile + 4 * r) = row < M ? scale : 0.f;
}

// ---------------------------------------------------------------------------
// Tensor core

// E4M3 x E4M3, both K-major, fp32 D, M = 128, K = 32: formats 0 at bits 7 and 10.
__device__ __forceinline__ uint32_t idesc_e4m3(uint32_t n) { return (1u << 4) | ((n >> 3) << 17) | ((128u >> 4) << 24); }

__device__ __forceinline__ void mma_e4m3(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate) : "memory");
}

// 64 consecutive fp32 columns of this thread's TMEM lane, in one load.
__device__ __forceinline__ void tmem_ld64_now(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,"
      "%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,"
      "%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
      "}, [%64];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr));
  // the registers are named so that nothing uses them earlier
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]),
                 "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]),
                 "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]),
                 "+r"(r[29]), "+r"(r[30]), "+r"(r[31]), "+r"(r[32]), "+r"(r[33]), "+r"(r[34]), "+r"(r[35]),
                 "+r"(r[36]), "+r"(r[37]), "+r"(r[38]), "+r"(r[39]), "+r"(r[40]), "+r"(r[41]), "+r"(r[42]),
                 "+r"(r[43]), "+r"(r[44]), "+r"(r[45]), "+r"(r[46]), "+r"(r[47]), "+r"(r[48]), "+r"(r[49]),
                 "+r"(r[50]), "+r"(r[51]), "+r"(r[52]), "+r"(r[53]), "+r"(r[54]), "+r"(r[55]), "+r"(r[56]),
                 "+r"(r[57]), "+r"(r[58]), "+r"(r[59]), "+r"(r[60]), "+r"(r[61]), "+r"(r[62]), "+r"(r[63])
               :: "memory");
}

__device__ __forceinline__ uint32_t bf16x2_of(Two v) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo_of(v), hi_of(v));
  return *reinterpret_cast<const uint32_t*>(&h);
}

// ---------------------------------------------------------------------------
// Large

struct W8LargeArgs {
  const uint8_t* Aq;        // activation tiles
  const uint8_t* W8;        // weight tiles
  const float* Ws;          // [N / 128, KT]
  uint16_t* C;              // [M, N] BF16
  int M, N, KT;
  int wide;                 // tiles of 256 weight rows per tile of tokens
  int full_units;           // tiles 0 .. full_units - 1 (x-major) run whole
  int split_units;          // then this many halves of the other wide tiles
  int units;                // and the narrow tiles at the end of an odd N / 128
  int shares;               // of a unit's K, each a thread block's of a cluster (1: no clusters)
  unsigned long long wait_ns;
  unsigned int* status;
};

constexpr int kMaxW8Shares = 6;

// SHARED: K is shared by a cluster; halves and narrow tiles only.
template <bool SHARED>
struct W8L {
  static constexpr int EPI_WARPS = 8, EPI_FIRST = 4;   // the first warpgroup: producer, MMA issuer, two that only help out
  static constexpr int THREADS = 32 * (EPI_FIRST + EPI_WARPS);
  // a thread of the epilogue holds 128 sums and 64 columns: the registers of the launch (384 x
  // 168) go to the two warpgroups that need them (128 x 40 + 256 x 232)
  static constexpr int REGS_FEW = 40, REGS_MANY = 232;
  static_assert(128 * REGS_FEW + 32 * EPI_WARPS * REGS_MANY <= THREADS * 168, "registers");
  static constexpr int STAGES = 4;
  static constexpr int STAGE = (SHARED ? 2 : 3) * kTile;
  static constexpr int STG_PITCH = 80;                 // 32 BF16 columns and 16 bytes: 16-byte rows on different banks
  static constexpr int OFF_STG = STAGES * STAGE;
  // SHARED: in place of the output's rows everyone's sums of this block's rows
  static constexpr int OFF_BAR = OFF_STG + (SHARED ? (128 + kMaxW8Shares - 1) * 512 : EPI_WARPS * 32 * STG_PITCH);
  static constexpr int NBAR = 2 * STAGES + 6;          // full, empty; accumulators' full and empty; drain; sums
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int SMEM_BYTES = OFF_MISC + 32 + 1024;
  static_assert(SMEM_BYTES <= 232448, "shared memory");
};

struct W8Unit { int x, w, n; };                        // token tile, first 128-row weight tile, how many of them

__device__ __forceinline__ W8Unit w8_unit(const W8LargeArgs& p, int u) {
  if (u < p.full_units) return {u / p.wide, 2 * (u % p.wide), 2};
  u -= p.full_units;
  if (u < p.split_units) {
    const int tile = p.full_units + (u >> 1);
    return {tile / p.wide, 2 * (tile % p.wide) + (u & 1), 1};
  }
  return {u - p.split_units, 2 * p.wide, 1};
}

// One unit's blocks of K: COLS columns of this thread's row.  False: a wait gave up.
template <int COLS>
__device__ __forceinline__ bool w8_promote(const W8LargeArgs& p, uint32_t tmem, uint32_t acc_full, uint32_t acc_empty,
                                           const uint8_t* row_scale, const float* block_scale, int nk, int& g,
                                           Two* acc, volatile int* abort_flag) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < COLS / 2; ++i) acc[i] = 0ull;
  float sa = *reinterpret_cast<const float*>(row_scale), sw = block_scale[0];
  for (int kt = 0; kt < nk; ++kt, ++g) {
    const uint32_t s = __float_as_uint(sa * sw);       // exact above 2^-126: sa is a power of two
    const Two s2 = pack2(s, s);
    if (kt + 1 < nk) {
      sa = *reinterpret_cast<const float*>(row_scale + static_cast<long long>(kt + 1) * kActTile);
      sw = block_scale[kt + 1];
    }
    const int b = g & 1;
    if (!__all_sync(0xFFFFFFFFu, mbar_wait(acc_full + 8u * b, static_cast<uint32_t>(g >> 1) & 1u, abort_flag, p.wait_ns, p.status)))
      return false;
    tc_fence_after();
    // few and large loads: the two warps of a scheduler load and add in turn
    static_assert(COLS % 64 == 0, "columns");
    constexpr int W = 64;
#pragma unroll
    for (int c = 0; c < COLS; c += W) {
      uint32_t t[W];
      tmem_ld64_now(tmem + b * 256 + c, t);
      if (c + W == COLS) {                               // everything is read: the accumulator may be written again
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + 8u * b);
      }
#pragma unroll
      for (int i = 0; i < W / 2; ++i) acc[c / 2 + i] = fma2(pack2(t[2 * i], t[2 * i + 1]), s2, acc[c / 2 + i]);
    }
  }
  return true;
}

template <int COLS>
__device__ __forceinline__ void w8_store(const W8LargeArgs& p, const Two* acc, uint8_t* stg, int row0, int col0) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < COLS; c += 32) {
    constexpr int PITCH = W8L<false>::STG_PITCH;
    uint4* mine = reinterpret_cast<uint4*>(stg + lane * PITCH);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mine[i] = make_uint4(bf16x2_of(acc[c / 2 + 4 * i]), bf16x2_of(acc[c / 2 + 4 * i + 1]),
                           bf16x2_of(acc[c / 2 + 4 * i + 2]), bf16x2_of(acc[c / 2 + 4 * i + 3]));
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = i * 8 + (lane >> 2), seg = lane & 3;
      const uint4 v = *reinterpret_cast<const uint4*>(stg + r * PITCH + seg * 16);
      if (row0 + r < p.M)
        *reinterpret_cast<uint4*>(p.C + static_cast<long long>(row0 + r) * p.N + col0 + c + seg * 8) = v;
    }
    __syncwarp();
  }
}

//   warp 0      producer: per block of K one activation tile and two (one) weight tiles;
//   warp 1      TMEM owner and MMA issuer: two accumulators of 256 columns in turn;
//   warps 4-11  two per TMEM lane quadrant, a thread per token row and half of the
//               columns: scale and add each block's sums, then BF16 rows.
// SHARED (one unit per cluster, few of them): every rank has its share of K; of the sums rank r
// owns rows 128 r / S .., the others send their sums there, the owner adds all in rank order.
template <bool SHARED>
__global__ void __launch_bounds__(W8L<SHARED>::THREADS, 1) a4w4_w8a8_large_kernel(const W8LargeArgs p) {
  using Cf = W8L<SHARED>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int S = SHARED ? p.shares : 1, rank = SHARED ? static_cast<int>(cluster_ctarank()) : 0;
  const int G = SHARED ? p.units : gridDim.x, u0 = SHARED ? blockIdx.x / S : blockIdx.x;      // units u0, u0 + G ..
  const int k0 = SHARED ? rank * p.KT / S : 0, nk = (SHARED ? (rank + 1) * p.KT / S : p.KT) - k0;
  const int own0 = rank * 128 / S, own1 = (rank + 1) * 128 / S, slot = (127 + S) / S;
  const unsigned long long drain_ns = p.wait_ns > 100000000ull ? p.wait_ns : 100000000ull;

  const uint32_t full = base + Cf::OFF_BAR, empty = full + 8u * Cf::STAGES;
  const uint32_t acc_full = empty + 8u * Cf::STAGES, acc_empty = acc_full + 16u, drain = acc_empty + 16u;
  const uint32_t sums = drain + 8u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cf::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cf::OFF_MISC + 8);
  volatile int* never = reinterpret_cast<volatile int*>(smem + Cf::OFF_MISC + 16);
  volatile int* owner_ready = reinterpret_cast<volatile int*>(smem + Cf::OFF_MISC + 24);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * Cf::STAGES + 2; ++s) mbar_init(full + 8u * s, 1);   // full, empty, acc_full
    mbar_init(acc_empty, Cf::EPI_WARPS);
    mbar_init(acc_empty + 8u, Cf::EPI_WARPS);
    mbar_init(drain, 1);
    mbar_init(sums, 1);
    *abort_flag = 0;
    *never = 0;
    *owner_ready = 0;
    fence_barrier_init();
    if (SHARED) mbar_arrive_expect_tx(sums, static_cast<uint32_t>((S - 1) * (own1 - own0) * 512));
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tc_fence_before();
  }
  __syncthreads();
  if (SHARED) cluster_arrive_relaxed();                 // this block's barriers exist; waited for before the first sums are sent
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();                                       // the activation tiles come from the kernel before
  griddep_launch_dependents();

  if (warp < Cf::EPI_FIRST) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(Cf::REGS_FEW));
    if (warp == 0) {
      if (lane == 0) {
        const uint64_t pol = policy_evict_last();         // operands are read again by other tiles, from L2
        int g = 0;
        bool ok = true;
        for (int u = u0; u < p.units && ok; u += G) {
          const W8Unit t = w8_unit(p, u);
          const uint8_t* a = p.Aq + (static_cast<long long>(t.x) * p.KT + k0) * kActTile;
          const uint8_t* w = p.W8 + (static_cast<long long>(t.w) * p.KT + k0) * kTile;
          for (int kt = 0; kt < nk; ++kt, ++g) {
            const int s = g % Cf::STAGES;
            if (!mbar_wait(empty + 8u * s, ((g / Cf::STAGES) & 1) ^ 1u, abort_flag, p.wait_ns, p.status)) {
              ok = false;
              break;
            }
            const uint32_t fb = full + 8u * s, dst = base + s * Cf::STAGE;
            mbar_arrive_expect_tx(fb, (1 + t.n) * kTile);
            bulk_g2s(dst, a + static_cast<long long>(kt) * kActTile, kTile, fb, pol);
            bulk_g2s(dst + kTile, w + static_cast<long long>(kt) * kTile, kTile, fb, pol);
            if (!SHARED && t.n == 2) bulk_g2s(dst + 2 * kTile, w + static_cast<long long>(p.KT + kt) * kTile, kTile, fb, pol);
          }
        }
        // every copy issued lands before the shared memory is released
        for (int j = (g > Cf::STAGES ? g - Cf::STAGES : 0); j < g; ++j)
          mbar_wait(full + 8u * (j % Cf::STAGES), (j / Cf::STAGES) & 1u, never, drain_ns, p.status);
      }
    } else if (warp == 1) {
      // (One thread's path from "read" to the next MMAs is part of every block of K: it waits for
      // the operands first, for the accumulator last, and commits the accumulator first.)
      if (elect_one()) {
        const uint64_t adesc0 = sdesc_sw128(base), bdesc0 = sdesc_sw128(base + kTile);
        int s = 0, g = 0;
        uint32_t ph = 0;
        bool ok = true;
        for (int u = u0; u < p.units && ok; u += G) {
          const uint32_t idesc = idesc_e4m3(128u * w8_unit(p, u).n);
          for (int kt = 0; kt < nk; ++kt, ++g) {
            const uint32_t b = g & 1, af = acc_full + 8u * b, d = tmem + b * 256, off = static_cast<uint32_t>(s * Cf::STAGE) >> 4;
            const uint64_t ad = adesc0 + off, bd = bdesc0 + off;
            if (!mbar_wait(full + 8u * s, ph, abort_flag, p.wait_ns, p.status) ||
                // the accumulator's sums of two blocks ago have been read
                (g >= 2 && !mbar_wait(af + 16u, static_cast<uint32_t>((g >> 1) - 1) & 1u, abort_flag, p.wait_ns, p.status))) {
              ok = false;
              break;
            }
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks) mma_e4m3(d, ad + 2 * ks, bd + 2 * ks, idesc, ks > 0 ? 1u : 0u);
            mma_commit(af);
            mma_commit(empty + 8u * s);
            if (++s == Cf::STAGES) {
              s = 0;
              ph ^= 1u;
            }
          }
        }
        // TMEM is released only after every MMA issued has completed
        mma_commit(drain);
        mbar_wait(drain, 0, never, drain_ns, p.status);
      }
    }
    __syncwarp();
    if (SHARED) {
      cluster_wait();
      cluster_arrive_relaxed();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(Cf::REGS_MANY));
    const int q = warp & 3, half = (warp - Cf::EPI_FIRST) >> 2;
    const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
    uint8_t* stg = smem + Cf::OFF_STG + (warp - Cf::EPI_FIRST) * 32 * Cf::STG_PITCH;
    Two acc[64];
    int g = 0;
    for (int u = u0; u < p.units; u += G) {
      const W8Unit t = w8_unit(p, u);
      const uint8_t* sa = p.Aq + (static_cast<long long>(t.x) * p.KT + k0) * kActTile + kTile + 4 * (q * 32 + lane);
      const int row0 = t.x * 128 + q * 32;
      if (SHARED) {
        const bool ok = w8_promote<64>(p, tq + half * 64, acc_full, acc_empty, sa, p.Ws + static_cast<long long>(t.w) * p.KT + k0,
                                       nk, g, acc, abort_flag);
        if (!ok) *abort_flag = 1;
        // The sums by rows over the drained ring, a row's four-column pieces in an order that changes
        // with the row, for the banks; each owner's rows leave in one bulk copy (asynchronous
        // stores of 16 bytes, each counted on the owner's barrier: +2 us).
        float4* mine = reinterpret_cast<float4*>(smem + (q * 32 + lane) * 512);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          mine[(half * 16 + i) ^ lane] = make_float4(lo_of(acc[2 * i]), hi_of(acc[2 * i]), lo_of(acc[2 * i + 1]), hi_of(acc[2 * i + 1]));
        const int et = threadIdx.x - 32 * Cf::EPI_FIRST;
        fence_proxy_async_smem();
        named_bar_sync(3, 32 * Cf::EPI_WARPS);
        cluster_wait();
        // sent whatever happened before, so that every owner's count of bytes completes
        if (warp == Cf::EPI_FIRST && lane < S && lane != rank) {
          const int r0 = lane * 128 / S, rows = (lane + 1) * 128 / S - r0;
          bulk_s2peer(cluster_map_shared(base + Cf::OFF_STG + rank * slot * 512, lane), base + r0 * 512, rows * 512,
                      cluster_map_shared(sums, lane));
        }
        __syncwarp();
        if (et == 0) *owner_ready = mbar_wait_cluster(sums, 0, 32ull * drain_ns, p.status) && !*abort_flag ? 1 : 0;
        named_bar_sync(3, 32 * Cf::EPI_WARPS);
        cluster_arrive_relaxed();                       // what came for this block is here; waited for before any leaves
        if (*owner_ready) {
          constexpr int ROWS = 4;                       // of a warp, in flight
          for (int row0 = own0 + (et >> 5); row0 < own1; row0 += ROWS * Cf::EPI_WARPS) {
            float4 sum[ROWS] = {};
            for (int c = 0; c < S; ++c) {
              const uint8_t* of = c == rank ? smem : smem + Cf::OFF_STG + (c * slot - own0) * 512;
#pragma unroll
              for (int i = 0; i < ROWS; ++i) {
                const int row = min(row0 + i * Cf::EPI_WARPS, own1 - 1);
                const float4 v = reinterpret_cast<const float4*>(of + row * 512)[lane ^ (row & 31)];
                sum[i].x += v.x; sum[i].y += v.y; sum[i].z += v.z; sum[i].w += v.w;
              }
            }
#pragma unroll
            for (int i = 0; i < ROWS; ++i) {
              const int row = row0 + i * Cf::EPI_WARPS;
              const __nv_bfloat162 lo = __floats2bfloat162_rn(sum[i].x, sum[i].y), hi = __floats2bfloat162_rn(sum[i].z, sum[i].w);
              const uint2 v = make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
              if (row < own1 && t.x * 128 + row < p.M)
                *reinterpret_cast<uint2*>(p.C + static_cast<long long>(t.x * 128 + row) * p.N + t.w * 128 + lane * 4) = v;
            }
          }
        }
      } else if (t.n == 2) {
        if (!w8_promote<128>(p, tq + half * 128, acc_full, acc_empty, sa,
                             p.Ws + static_cast<long long>(t.w + half) * p.KT, nk, g, acc, abort_flag))
          break;
        w8_store<128>(p, acc, stg, row0, (t.w + half) * 128);
      } else {
        if (!w8_promote<64>(p, tq + half * 64, acc_full, acc_empty, sa, p.Ws + static_cast<long long>(t.w) * p.KT, nk,
                            g, acc, abort_flag))
          break;
        w8_store<64>(p, acc, stg, row0, t.w * 128 + half * 64);
      }
    }
  }

  if (SHARED) cluster_wait();                           // the peers have read this block's sums
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// Small

struct W8SmallArgs {
  const uint16_t* A;        // [M, K] BF16
  const uint8_t* W8;
  const float* Ws;
  uint16_t* C;
  int M, N, K, KT, splits;
  int prefetch_w;           // 1: weights may be read before the previous grid on the stream completes
  unsigned long long wait_ns;
  unsigned int* status;
};

template <int NX>
struct W8S {
  static constexpr int RING = 4;                       // tiles in flight, of weights and of activations
  static constexpr int ACCS = 4;                       // accumulators
  static constexpr int THREADS = 64 + 128 + 128;       // two single warps, producers, promoters
  static constexpr int X_STAGE = NX * 128;
  static constexpr int OFF_X = RING * kTile;
  static constexpr int OFF_SCALE = OFF_X + RING * X_STAGE;
  // up to 16 senders' shares of this block's slice of the sums ((G + S) groups of 16 bytes, G = 32 NX);
  // this block's own sums are staged over the drained weight ring
  static constexpr int OFF_PUSH = OFF_SCALE + 2 * RING * NX * 4;
  static constexpr int OFF_BAR = OFF_PUSH + NX * 512 + 256;
  static constexpr int NBAR = 5 * RING + 2 * ACCS + 2; // full_w, empty, full_x, scales x 2; accumulators' full and empty; red; drain
  static constexpr int OFF_MISC = OFF_BAR + 8 * NBAR;
  static constexpr int SMEM_BYTES = OFF_MISC + 32 + 1024;
  static constexpr int ACC_COLS = NX;
  static constexpr int TMEM_COLS = ACCS * NX;
  static_assert(ACCS <= RING, "a scale's place is written again after its block was added");
  static_assert(NX * 512 <= RING * kTile, "the sums fit the weight ring");
  static_assert(2 * (SMEM_BYTES + 1024) <= 233472, "two thread blocks on an SM");
};

//   warp 0      weight producer;
//   warp 1      TMEM owner and MMA issuer (accumulators of NX columns in turn);
//   warps 2-5   activations: every fourth block of K each, eight lanes a row, into the ring's place
//               for it; scales have places for two turns of the ring, since they are read after
//               the MMAs that free the codes';
//   warps 6-9   a thread per weight row: scale and add each block's NX sums.
// Then warps 2-9 reduce over the cluster: slice r of the 128 x NX sums belongs to rank r, everyone
// sends its share there as soon as it has it, the owner adds in rank order.
template <int NX>
__global__ void __launch_bounds__(W8S<NX>::THREADS, 2) a4w4_w8a8_small_kernel(const W8SmallArgs p) {
  using Cf = W8S<NX>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int w_tile = blockIdx.x, split = blockIdx.z;
  const int kt0 = static_cast<int>(static_cast<long long>(split) * p.KT / p.splits);
  const int kt1 = static_cast<int>(static_cast<long long>(split + 1) * p.KT / p.splits);
  const int nk = kt1 - kt0;
  const int m0 = blockIdx.y * NX, mvalid = min(NX, p.M - m0);      // this block's tokens
  const unsigned long long drain_ns = p.wait_ns > 100000000ull ? p.wait_ns : 100000000ull;

  const uint32_t full_w = base + Cf::OFF_BAR, empty = full_w + 8u * Cf::RING;
  const uint32_t full_x = empty + 8u * Cf::RING, scales = full_x + 8u * Cf::RING;
  const uint32_t acc_full = scales + 16u * Cf::RING, acc_empty = acc_full + 8u * Cf::ACCS;
  const uint32_t red_bar = acc_empty + 8u * Cf::ACCS, drain = red_bar + 8u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + Cf::OFF_MISC);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + Cf::OFF_MISC + 8);
  volatile int* never = reinterpret_cast<volatile int*>(smem + Cf::OFF_MISC + 16);
  volatile int* owner_ready = reinterpret_cast<volatile int*>(smem + Cf::OFF_MISC + 24);

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * Cf::RING; ++s) mbar_init(full_w + 8u * s, 1);    // full_w, empty
    for (int s = 0; s < 3 * Cf::RING; ++s) mbar_init(full_x + 8u * s, 64);   // full_x, scales: two warps, or one twice
    for (int s = 0; s < Cf::ACCS; ++s) {
      mbar_init(acc_full + 8u * s, 1);
      mbar_init(acc_empty + 8u * s, 4);
    }
    mbar_init(red_bar, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *never = 0;
    *owner_ready = 0;
    fence_barrier_init();
    if (p.splits > 1) {
      const int S = p.splits, G = mvalid * 32, rank = static_cast<int>(cluster_ctarank());
      const int g0 = static_cast<int>(static_cast<long long>(rank) * G / S);
      const int g1 = static_cast<int>(static_cast<long long>(rank + 1) * G / S);
      mbar_arrive_expect_tx(red_bar, static_cast<uint32_t>(S * (g1 - g0) * 16));
    }
  }
  // rows of tokens that do not exist: codes and scales zero, never written again
  for (int i = threadIdx.x; i < (Cf::OFF_PUSH - Cf::OFF_X) / 16; i += Cf::THREADS)
    reinterpret_cast<uint4*>(smem + Cf::OFF_X)[i] = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), Cf::TMEM_COLS);
    tc_fence_before();
  }
  __syncthreads();
  if (p.splits > 1) cluster_arrive_relaxed();          // this block's barriers exist; waited for before the first share is sent
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  griddep_launch_dependents();                         // (the next grid waits for the whole of this one)
  if (warp == 0) {
    if (lane == 0) {
      if (!p.prefetch_w) griddep_wait();
      const uint64_t pol = policy_evict_first();       // every weight byte is read once (per tile of tokens)
      const uint8_t* w = p.W8 + (static_cast<long long>(w_tile) * p.KT + kt0) * kTile;
      int i = 0;
      for (; i < nk; ++i) {
        const int s = i % Cf::RING;
        if (!mbar_wait(empty + 8u * s, ((i / Cf::RING) & 1) ^ 1u, abort_flag, p.wait_ns, p.status)) break;
        mbar_arrive_expect_tx(full_w + 8u * s, kTile);
        bulk_g2s(base + s * kTile, w + static_cast<long long>(i) * kTile, kTile, full_w + 8u * s, pol);
      }
      for (int j = (i > Cf::RING ? i - Cf::RING : 0); j < i; ++j)
        mbar_wait(full_w + 8u * (j % Cf::RING), (j / Cf::RING) & 1u, never, drain_ns, p.status);
    }
    __syncwarp();
    griddep_wait();
  } else if (warp == 1) {
    if (lane == 0) {
      const uint64_t adesc0 = sdesc_sw128(base), bdesc0 = sdesc_sw128(base + Cf::OFF_X);
      const uint32_t idesc = idesc_e4m3(NX);
      bool ok = true;
      for (int i = 0; i < nk && ok; ++i) {
        const int s = i % Cf::RING, b = i % Cf::ACCS;
        ok = mbar_wait(full_x + 8u * s, static_cast<uint32_t>(i / Cf::RING) & 1u, abort_flag, p.wait_ns, p.status);
        ok = ok && (i < Cf::ACCS || mbar_wait(acc_empty + 8u * b, static_cast<uint32_t>(i / Cf::ACCS - 1) & 1u, abort_flag, p.wait_ns, p.status));
        ok = ok && mbar_wait(full_w + 8u * s, (i / Cf::RING) & 1u, abort_flag, p.wait_ns, p.status);
        if (!ok) break;
        tc_fence_after();
        const uint64_t ad = adesc0 + ((s * kTile) >> 4), bd = bdesc0 + ((s * Cf::X_STAGE) >> 4);
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) mma_e4m3(tmem + b * Cf::ACC_COLS, ad + 2 * ks, bd + 2 * ks, idesc, ks > 0 ? 1u : 0u);
        mma_commit(acc_full + 8u * b);
        mma_commit(empty + 8u * s);
      }
      mma_commit(drain);
      mbar_wait(drain, 0, never, drain_ns, p.status);
    }
    __syncwarp();
    griddep_wait();
  } else {
    griddep_wait();                                    // A is written by the previous grid
    int ready = nk > 0;
    // ---------------- activations ----------------
    // Warps 2-5 take every fourth block of K; the promoters, with nothing to add yet, take half of the
    // rows of the first RING blocks.
    {
      constexpr int CH = 4;                            // rows in flight per eight lanes
      const bool helper = warp >= 6;
      const int c = lane & 7, half = (mvalid + 7) / 8 * 4;
      float* s_scale = reinterpret_cast<float*>(smem + Cf::OFF_SCALE);
      bool stop = false;
      for (int i = (warp - 2) & 3; i < nk && !stop; i += 4) {
        const int s = i % Cf::RING, turn = i % (2 * Cf::RING);
        const bool shared = i < Cf::RING;
        const int end = shared && !helper ? min(half, mvalid) : mvalid;
        bool waited = shared;
        for (int r0 = helper ? half : 0; r0 < end; r0 += 4 * CH) {
          uint4 v[CH][2];
#pragma unroll
          for (int h = 0; h < CH; ++h) {
            const int r = r0 + 4 * h + (lane >> 3);
            v[h][0] = v[h][1] = make_uint4(0u, 0u, 0u, 0u);
            if (r < end) {
              const uint16_t* src = p.A + static_cast<long long>(m0 + r) * p.K + (kt0 + i) * 128 + c * 16;
              v[h][0] = ld_global_nc_v4(src);
              v[h][1] = ld_global_nc_v4(src + 8);
            }
          }
          if (!waited) {                               // the MMAs of the block that had this place have run
            waited = true;
            int got = 1;
            if (lane == 0) got = mbar_wait(empty + 8u * s, static_cast<uint32_t>(i / Cf::RING - 1) & 1u, abort_flag, p.wait_ns, p.status);
            stop = __shfl_sync(0xFFFFFFFFu, got, 0) == 0;
            if (stop) break;
          }
#pragma unroll
          for (int h = 0; h < CH; ++h) {
            if (r0 + 4 * h >= end) break;
            const int r = r0 + 4 * h + (lane >> 3);
            float scale;
            const uint4 code = quant128(v[h][0], v[h][1], &scale);
            if (r < end) {
              *reinterpret_cast<uint4*>(smem + Cf::OFF_X + s * Cf::X_STAGE + tile_piece(r, c)) = code;
              if (c == 0) s_scale[turn * NX + r] = scale;
            }
          }
        }
        if (!stop) {
          fence_proxy_async_smem();
          mbar_arrive_n(full_x + 8u * s, shared ? 1 : 2);
          mbar_arrive_n(scales + 8u * turn, shared ? 1 : 2);
        }
        if (helper) break;
      }
      ready = ready && !stop;
    }
    if (warp >= 6) {
      // ---------------- promotion ----------------
      const int q = warp & 3;
      const uint32_t tq = tmem + (static_cast<uint32_t>(q * 32) << 16);
      const float* block_scale = p.Ws + static_cast<long long>(w_tile) * p.KT + kt0;
      Two acc[NX / 2];
#pragma unroll
      for (int i = 0; i < NX / 2; ++i) acc[i] = 0ull;
      for (int i = 0; i < nk; ++i) {
        const int turn = i % (2 * Cf::RING), b = i % Cf::ACCS;
        const uint32_t sw = __float_as_uint(block_scale[i]);
        const Two sw2 = pack2(sw, sw);
        const bool ok = mbar_wait(scales + 8u * turn, static_cast<uint32_t>(i / (2 * Cf::RING)) & 1u, abort_flag, p.wait_ns, p.status) &&
                        mbar_wait(acc_full + 8u * b, static_cast<uint32_t>(i / Cf::ACCS) & 1u, abort_flag, p.wait_ns, p.status);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ready = 0;
          break;
        }
        tc_fence_after();
        const ulonglong2* sa = reinterpret_cast<const ulonglong2*>(smem + Cf::OFF_SCALE + turn * NX * 4);
#pragma unroll
        for (int c = 0; c < NX; c += 16) {
          float t[16];
          tmem_ld16(tq + b * Cf::ACC_COLS + c, t);
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const ulonglong2 s2 = sa[c / 4 + u];       // four tokens' scales
            acc[c / 2 + 2 * u] = fma2(pack2(__float_as_uint(t[4 * u]), __float_as_uint(t[4 * u + 1])), mul2(s2.x, sw2),
                                      acc[c / 2 + 2 * u]);
            acc[c / 2 + 2 * u + 1] = fma2(pack2(__float_as_uint(t[4 * u + 2]), __float_as_uint(t[4 * u + 3])),
                                          mul2(s2.y, sw2), acc[c / 2 + 2 * u + 1]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acc_empty + 8u * b);
      }
      // weight row q * 32 + lane of every token: partial [token][weight row] over the drained ring,
      // or, where nothing is to be reduced, BF16 (a warp writes 64 bytes of a token's row)
      const int lrow = q * 32 + lane;
      if (ready && p.splits == 1) {
#pragma unroll
        for (int i = 0; i < NX; ++i)
          if (i < mvalid)
            p.C[static_cast<long long>(m0 + i) * p.N + w_tile * 128 + lrow] =
                __bfloat16_as_ushort(__float2bfloat16_rn(i & 1 ? hi_of(acc[i / 2]) : lo_of(acc[i / 2])));
      } else if (ready) {
        float* red = reinterpret_cast<float*>(smem);
#pragma unroll
        for (int i = 0; i < NX; ++i)
          if (i < mvalid) red[i * 128 + lrow] = i & 1 ? hi_of(acc[i / 2]) : lo_of(acc[i / 2]);
      }
    }
    if (p.splits > 1 && !ready) *abort_flag = 1;       // this block's sums are not whole
  }

  if (p.splits > 1) {
    if (warp >= 2) {
      constexpr int P = 256;
      const int et = threadIdx.x - 64;
      const int S = p.splits, G = mvalid * 32, slot = (G + S - 1) / S;
      const uint32_t rank = cluster_ctarank();
      const float4* red4 = reinterpret_cast<const float4*>(smem);
      named_bar_sync(3, P);                            // the sums are staged
      cluster_wait();
      // group g (four weight rows of a token) belongs to o = max{o : floor(o G / S) <= g}; sent
      // whatever happened before, so that every owner's byte count completes
      for (int g = et; g < G; g += P) {
        const int o = static_cast<int>((static_cast<long long>(g + 1) * S - 1) / G);
        const int og0 = static_cast<int>(static_cast<long long>(o) * G / S);
        const uint32_t dst = cluster_map_shared(
            base + Cf::OFF_PUSH + static_cast<uint32_t>((static_cast<int>(rank) * slot + (g - og0)) * 16), static_cast<uint32_t>(o));
        st_async_v4(dst, red4[g], cluster_map_shared(red_bar, static_cast<uint32_t>(o)));
      }
      if (et == 0) {
        const unsigned long long lim = 32ull * drain_ns;
        *owner_ready = mbar_wait_cluster(red_bar, 0, lim, p.status) && !*abort_flag ? 1 : 0;
      }
      named_bar_sync(3, P);
      if (*owner_ready) {
        const int g0 = static_cast<int>(static_cast<long long>(rank) * G / S);
        const int g1 = static_cast<int>(static_cast<long long>(rank + 1) * G / S);
        const float4* push = reinterpret_cast<const float4*>(smem + Cf::OFF_PUSH);
        for (int g = g0 + et; g < g1; g += P) {
          float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
          for (int c = 0; c < S; ++c) {
            const float4 v = push[c * slot + (g - g0)];
            sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
          }
          const __nv_bfloat162 lo = __floats2bfloat162_rn(sum.x, sum.y), hi = __floats2bfloat162_rn(sum.z, sum.w);
          uint2 o;
          o.x = *reinterpret_cast<const uint32_t*>(&lo);
          o.y = *reinterpret_cast<const uint32_t*>(&hi);
          *reinterpret_cast<uint2*>(p.C + static_cast<long long>(m0 + (g >> 5)) * p.N + w_tile * 128 + (g & 31) * 4) = o;
        }
      }
    } else {
      cluster_wait();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, Cf::TMEM_COLS);
  }
}

constexpr int kMaxW8Splits = 16;
constexpr int kMaxDevices = 64;

template <int NX>
int small_attrs() {
  auto kern = a4w4_w8a8_small_kernel<NX>;
  static std::atomic<unsigned long long> attr_devs{0};   // bit d: attributes set on device d
  return ensure_func_attrs(attr_devs, [&] {
    // clusters of up to 16 thread blocks (more than the portable 8)
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, W8S<NX>::SMEM_BYTES) == cudaSuccess &&
           cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
  });
}
template <bool SHARED>
int large_attrs() {
  static std::atomic<unsigned long long> attr_devs{0};   // bit d: attribute set on device d
  return ensure_func_attrs(attr_devs, [&] {
    return cudaFuncSetAttribute(a4w4_w8a8_large_kernel<SHARED>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                W8L<SHARED>::SMEM_BYTES) == cudaSuccess;
  });
}

int this_device() {
  int dev = -1;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    cudaGetLastError();
    return -1;
  }
  return dev;
}

// Clusters of n thread blocks that the device holds at once (0: not to be had), per kernel; its
// attributes are set.
int clusters_at_once(int dev, int kind, const void* kern, int threads, int smem, int n) {
  static std::atomic<int> cache[kMaxDevices][3][kMaxW8Splits + 1];     // filled on first use (0: not known yet)
  std::atomic<int>* known = dev >= 0 && dev < kMaxDevices ? &cache[dev][kind][n] : nullptr;
  int count = known != nullptr ? known->load(std::memory_order_relaxed) : 0;
  if (count > 0) return count;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(n), 1, 1);
  cfg.blockDim = dim3(static_cast<unsigned>(threads), 1, 1);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = static_cast<unsigned>(n);
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaOccupancyMaxActiveClusters(&count, kern, &cfg) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  if (count > 0 && known != nullptr) known->store(count, std::memory_order_relaxed);
  return count;
}

// What a kernel takes with K in so many shares, in eighths of a block of K (of its own; 0: not known).
struct W8Cost {
  int shares;
  long long cost;
};

// Shares of K: those that take least time if a wave of clusters costs the blocks of its longest share
// and six more, and a share an eighth of a block (2048 k's, us: 14 to 36 tiles with 2 shares 6.4, with 4
// 4.7, with 8 3.9 to 5.1; 14 tiles with 16 4.3; 40 tiles with 8, a second wave, 8.0).
// A cluster stays within a GPC, so that fewer fit than the SMs' number says: 32 x 4224 x 1536 with
// 9 shares (297 thread blocks of 304, but 33 clusters are a second wave) 11.5 us, with 6 6.5.
// Shares that do not shorten the longest one only add to the sums: 4 x 1536 x 4224 with 16 5.0, with 11 4.6.
// (All with the weights in L2; not fitted with weights that come from memory.)
template <int NX>
W8Cost small_cost(long long tiles, int kt) {
  W8Cost best{1, 0};
  const int dev = this_device();
  for (int s = 1; s <= kt && s <= kMaxW8Splits; ++s) {
    // (the count is for one thread block on an SM, two fit)
    const long long at_once = 2ll * clusters_at_once(dev, NX == 32, reinterpret_cast<const void*>(a4w4_w8a8_small_kernel<NX>),
                                                     W8S<NX>::THREADS, W8S<NX>::SMEM_BYTES, s);
    if (at_once <= 0) continue;
    const long long cost = (tiles + at_once - 1) / at_once * ((kt + s - 1) / s + 6) * 8 + s;
    if (best.cost == 0 || cost < best.cost) best = {s, cost};
  }
  return best;
}

template <int NX>
int launch_small(const W8SmallArgs& a, int w_tiles, cudaStream_t st) {
  using Cf = W8S<NX>;
  auto kern = a4w4_w8a8_small_kernel<NX>;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(w_tiles, (a.M + NX - 1) / NX, static_cast<unsigned>(a.splits));
  cfg.blockDim = dim3(Cf::THREADS, 1, 1);
  cfg.dynamicSmemBytes = Cf::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = 1;
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = static_cast<unsigned>(a.splits);
  cfg.attrs = attrs;
  cfg.numAttrs = a.splits > 1 ? 2 : 1;
  if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) return -4;
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

constexpr int kMaxSmallM = 1024;

// What the tiles of 128 x 256 take, in blocks of K of a half of one: 0.29 us each and 12 of them before
// the first (3.6 us).  Few of them, one wave of halves, share K as long as a cluster for each is there at once:
// 7 blocks' time for the exchange of sums, and one for each share (a rank takes in (S - 1) / S of 64 KB;
// 32 KB from a peer took 1.3 us).  Us with 1, 2, 4, 6 shares (8 are never better):
//   64 x 1536 x 7168  20.0  13.9  10.7  10.0    513 x 1536 x 4224  14.8  12.3 (60 units: no more fit)
//   64 x  256 x 4224  13.3  10.5   8.4   8.1     64 x 4224 x 1536   7.3   7.7   8.1
// Where 32 tokens x 128 weight rows, 2.4 times as much for each of their blocks (small_cost), come to
// less, they are taken; 32 and fewer tokens always are, for the sake of the workspace.  These / those:
//   64 x 1536 x 7168  10.0 /  9.6    128 x 1536 x 7168  10.0 / 13.4     64 x   256 x 4224   8.1 /  6.1
//   64 x 7168 x 4224  11.1 / 16.8     96 x 8448 x 7168  15.4 / 44.0     32 x 18944 x 3584  13.3 / 15.7
long long full_units(const W8Plan& pl) { return static_cast<long long>(pl.x_tiles) * (pl.w_tiles / 2) - pl.half_tiles; }
long long half_units(const W8Plan& pl) { return 2ll * pl.half_tiles + (pl.w_tiles % 2 ? pl.x_tiles : 0); }

W8Cost large_cost(const W8Plan& pl, int sms) {
  const long long full = full_units(pl), halves = half_units(pl);
  W8Cost best{1, 8 * (pl.kt * (2 * ((full + sms - 1) / sms) + (halves + sms - 1) / sms) + 12)};
  if (full > 0 || 2 * halves > sms) return best;
  const int dev = this_device();
  for (int s = 2; s <= pl.kt && s <= kMaxW8Shares; ++s) {
    const long long cost = 8ll * ((pl.kt + s - 1) / s + 19 + s);
    if (cost < best.cost && halves <= clusters_at_once(dev, 2, reinterpret_cast<const void*>(a4w4_w8a8_large_kernel<true>),
                                                       W8L<true>::THREADS, W8L<true>::SMEM_BYTES, s))
      best = {s, cost};
  }
  return best;
}

int launch_large(const W8LargeArgs& a, int sms, cudaStream_t st) {
  if (a.shares == 1) {
    if (large_attrs<false>() != 0) return -4;
    return launch_pdl_smem(a4w4_w8a8_large_kernel<false>, a.units < sms ? a.units : sms, W8L<false>::THREADS,
                           W8L<false>::SMEM_BYTES, st, a);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.units * a.shares), 1, 1);
  cfg.blockDim = dim3(W8L<true>::THREADS, 1, 1);
  cfg.dynamicSmemBytes = W8L<true>::SMEM_BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attrs[2];
  attrs[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attrs[0].val.programmaticStreamSerializationAllowed = 1;
  attrs[1].id = cudaLaunchAttributeClusterDimension;
  attrs[1].val.clusterDim.x = static_cast<unsigned>(a.shares);
  attrs[1].val.clusterDim.y = 1;
  attrs[1].val.clusterDim.z = 1;
  cfg.attrs = attrs;
  cfg.numAttrs = 2;
  if (cudaLaunchKernelEx(&cfg, a4w4_w8a8_large_kernel<true>, a) != cudaSuccess) return -4;
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

}  // namespace

W8Plan plan_w8a8(int M, int N, int K, int sms) {
  W8Plan pl{};
  pl.kt = K / 128;
  pl.w_tiles = N / 128;
  pl.x_tiles = M / 128 + (M % 128 != 0);
  if (M > 32) {
    const long long tiles = static_cast<long long>(pl.x_tiles) * (pl.w_tiles / 2), rest = tiles % sms;
    // the last, partial wave's tiles run as halves where they then still are one wave
    pl.half_tiles = 2 * rest <= sms ? static_cast<int>(rest) : 0;
    pl.ws_bytes = static_cast<size_t>(pl.x_tiles) * pl.kt * kActTile;
  }
  return pl;
}

int launch_w8a8(const W8Plan& pl, const void* A, int M, int K, const void* W8, const float* Ws, int N, void* C,
                void* ws, cudaStream_t st, unsigned long long wait_ns, unsigned int* status, int prefetch_w, int sms) {
  W8Cost large{1, 0};
  if (M > 32) {
    if (large_attrs<true>() != 0) return -4;
    large = large_cost(pl, sms);
  }
  if (M <= kMaxSmallM) {
    W8SmallArgs a{};
    a.A = static_cast<const uint16_t*>(A);
    a.W8 = static_cast<const uint8_t*>(W8);
    a.Ws = Ws;
    a.C = static_cast<uint16_t*>(C);
    a.M = M; a.N = N; a.K = K; a.KT = pl.kt;
    a.prefetch_w = prefetch_w;
    a.wait_ns = wait_ns;
    a.status = status;
    if (M <= 16) {
      if (small_attrs<16>() != 0) return -4;
      a.splits = small_cost<16>(pl.w_tiles, pl.kt).shares;
      return launch_small<16>(a, pl.w_tiles, st);
    }
    if (small_attrs<32>() != 0) return -4;
    const W8Cost small = small_cost<32>(static_cast<long long>(pl.w_tiles) * ((M + 31) / 32), pl.kt);
    if (M <= 32 || (small.cost > 0 && 12 * small.cost < 5 * large.cost)) {
      a.splits = small.shares;
      return launch_small<32>(a, pl.w_tiles, st);
    }
  }
  const long long blocks = static_cast<long long>(pl.x_tiles) * 128 * pl.kt;
  const long long grid = (blocks * 8 + 255) / 256, full = full_units(pl), halves = half_units(pl);
  if (grid > INT32_MAX || full + halves > INT32_MAX) return -1;
  int rc = launch_pdl(w8_quant_tiles_kernel, static_cast<int>(grid), 256, st, static_cast<const uint16_t*>(A), M, K,
                      pl.kt, blocks, static_cast<uint8_t*>(ws));
  if (rc != 0) return rc;
  W8LargeArgs a{};
  a.Aq = static_cast<const uint8_t*>(ws);
  a.W8 = static_cast<const uint8_t*>(W8);
  a.Ws = Ws;
  a.C = static_cast<uint16_t*>(C);
  a.M = M; a.N = N; a.KT = pl.kt;
  a.wide = pl.w_tiles / 2;
  a.full_units = static_cast<int>(full);
  a.split_units = 2 * pl.half_tiles;
  a.units = static_cast<int>(full + halves);
  a.wait_ns = wait_ns;
  a.status = status;
  a.shares = large.shares;
  return launch_large(a, sms, st);
}

int launch_prepare_w8(const void* w_bf16, int N, int K, void* w8, float* ws, cudaStream_t st) {
  const long long tiles = static_cast<long long>(N / 128) * (K / 128);
  if (tiles > INT32_MAX) return -1;
  return launch_pdl(w8_prepare_kernel, static_cast<int>(tiles), 256, st, static_cast<const uint16_t*>(w_bf16), K, K / 128,
                    static_cast<uint8_t*>(w8), ws);
}

int launch_shuffle_w8(const void* w_e4m3, int N, int K, void* w8, cudaStream_t st, int sms) {
  const long long pieces = static_cast<long long>(N) * (K / 16);
  const long long most = static_cast<long long>(sms) * 8, want = (pieces + 255) / 256;
  return launch_pdl(w8_shuffle_kernel, static_cast<int>(want < most ? want : most), 256, st,
                    static_cast<const uint8_t*>(w_e4m3), K, K / 128, pieces, static_cast<uint8_t*>(w8));
}

}  // namespace a4w4
