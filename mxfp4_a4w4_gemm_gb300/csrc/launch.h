// launch.h -- host-side launchers behind the C ABI (internal).
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace a4w4 {

// Tile plan of one dense GEMM call: a pure function of (M, N, K, SM count),
// shared by a4w4_gemm and a4w4_gemm_workspace_bytes.
struct GemmPlan {
  int swap_ab;      // 1: weights are the MMA's M side (small M)
  int decode;       // 1: the decode kernel (decode.cu): M <= 16, and some M <= 32 (plan_gemm)
  int prequant;     // 1: activations quantised once into tiles first (M > 128; M > 64 when N >= 4096)
  int persistent;   // 1 (every prequant plan): the persistent large-M kernel (large.cu)
  int half_tiles;   // persistent: tiles of the last partial wave run as two 128-column halves
  size_t aq_bytes;  // workspace bytes of the quantised activation tiles (codes + scales)
  int nx;           // activation rows per CTA
  int w_tiles;      // weight-row tiles (N / 128 or N / 256)
  int x_tiles;      // activation-row tiles
  int splits;       // K splits
  int ring;         // decode kernel: weight ring depth (K tiles in flight per CTA)
  int cluster_reduce;     // 1: the splits of a tile form a cluster and reduce over DSMEM
  int kt;           // 256-wide K tiles
  size_t ws_bytes;        // workspace: the activation tiles (aq_bytes), or 0
};

GemmPlan plan_gemm(int M, int N, int K, int sms);

// Kernel function attributes (dynamic shared memory size, non-portable
// cluster sizes) belong to the current device's context.  A launcher keeps
// one bit per device in `done` and runs `set` only where that bit is clear
// (devices beyond 63 run it on every launch).  Returns 0, or -4 when the
// device cannot be read or `set` reports a failed attribute call.
template <typename SetFn>
int ensure_func_attrs(std::atomic<unsigned long long>& done, SetFn set) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return -4;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0ull;
  if (bit != 0 && (done.load(std::memory_order_acquire) & bit) != 0) return 0;
  if (!set()) return -4;
  if (bit != 0) done.fetch_or(bit, std::memory_order_release);
  return 0;
}

// Launch `kern` on a 1-D grid with programmatic stream serialisation (the
// kernels launched this way order their global reads after
// griddepcontrol.wait, so they may start while the previous grid finishes).
// Returns 0 or -4.
template <typename... Params, typename... Args>
int launch_pdl_smem(void (*kern)(Params...), int grid, int block, size_t smem, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(block, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, args...) != cudaSuccess) return -4;
  return cudaGetLastError() == cudaSuccess ? 0 : -4;
}

template <typename... Params, typename... Args>
int launch_pdl(void (*kern)(Params...), int grid, int block, cudaStream_t st, Args... args) {
  return launch_pdl_smem(kern, grid, block, 0, st, args...);
}

// Shared by the C ABI entry points (defined in api.cu): SM count of the
// current device if it is a compute capability 10.3 GPU, else a negative
// A4W4 error code; device address of the status word; the current wait limit.
int device_sms();
unsigned int* device_status_ptr();
unsigned long long wait_limit_ns();

// Test hook (a4w4_debug.h): where the activation producers of the CTAs of
// weight tile 0 also store the MXFP4 operand tiles they build in shared
// memory.  Atom a = x_tile * KT + kt: codes at codes + a * (rows per tile *
// 128) in the swizzled tile layout, scales at scales + a * 1024 in the
// scale-atom layout.  codes == nullptr: off (every product call).
struct ActDump {
  uint8_t* codes;
  uint8_t* scales;
};

int launch_mxfp4_quant(const void* x, long long rows, int cols, void* q, void* s, cudaStream_t st, int sms);
int launch_prepare_weight(const void* w, int rows, int K, int experts, int pair_I, void* wq, void* ws,
                          cudaStream_t st, int sms);
// A [M, K] -> MXFP4 tiles of 128 rows x 256 K (rows padded to 128 with zeros),
// atom x*KT + kt at aq + atom*17408: 16 KB of codes in the weight tile layout,
// then its 1 KB of scales.
int launch_quant_activation_tiles(const void* a, int M, int K, void* aq, cudaStream_t st, int sms);
// prefetch_w: weights may be read before the previous grid on the stream
// completes (the caller guarantees that grid does not write them).
int launch_gemm(const GemmPlan& plan, const void* A, int M, int K, const void* Wq, const void* Ws, int N,
                void* C, void* ws, cudaStream_t st, unsigned long long wait_ns, unsigned int* status,
                int prefetch_w, ActDump dump);
// A16WFP4 (BF16 activations x MXFP4 weights): swap-AB tiles of 16 or 32
// tokens, split-K reduced inside clusters; no workspace.
GemmPlan plan_a16w4(int M, int N, int K, int sms);
int launch_a16w4(const GemmPlan& plan, const void* A, int M, int K, const void* Wq, const void* Ws, int N, void* C,
                 cudaStream_t st, unsigned long long wait_ns, unsigned int* status, int prefetch_w);
// plan.persistent: one CTA per SM (at most `sms`) walking the 128 x 256 tiles
// of the activation tiles already quantised into `Aq`, the last
// plan.half_tiles of them as two 128-column halves each (large.cu).
int launch_large(const GemmPlan& plan, const uint8_t* Aq, int M, const void* Wq, const void* Ws, int N, void* C,
                 cudaStream_t st, unsigned long long wait_ns, unsigned int* status, int sms);
// plan.decode: the decode kernel (decode.cu); no workspace.
int launch_decode(const GemmPlan& plan, const void* A, int M, int K, const void* Wq, const void* Ws, int N,
                  void* C, cudaStream_t st, unsigned long long wait_ns, unsigned int* status, int prefetch_w,
                  ActDump dump);
// act: 0 SwiGLU (W1[e] = [2I, D] paired gate/up layout), 1 SiLU (W1[e] =
// [I, D] dense layout); out_tiles: 1 = sorted-slot operand tiles.
int launch_moe_gemm1(const void* X, int T, int D, const int32_t* sorted_rows, const int32_t* block_expert,
                     const int32_t* num_blocks, int max_blocks, int topk, const void* W1q, const void* W1s,
                     int E, int I, int act, int out_tiles, void* out_q, void* out_s, void* xq_ws, cudaStream_t st,
                     unsigned long long wait_ns, unsigned int* status, int sms, ActDump dump);
// MoE GEMM2: GEMM1's sorted-slot tiles x W2[e] ([D, I] dense layout per
// expert, I <= 1024) -> top-k weighted fp32 rows partial[T*topk, D]: one
// persistent CTA per SM walking a contiguous run of (block, 256-column tile)
// units with each block's activation tiles resident (moe2.cu).
int launch_moe_gemm2_persistent(const void* Aq, const void* As, int T, int I, const int32_t* sorted_rows,
                                const int32_t* block_expert, const int32_t* num_blocks, int max_blocks, int topk,
                                const float* topk_w, const void* W2q, const void* W2s, int E, int D, float* partial,
                                cudaStream_t st, unsigned long long wait_ns, unsigned int* status, int sms);
// Y[t, :] (BF16) = sum over k = 0..topk-1, in that order, of partial[t*topk + k, :].
int launch_moe_sum(const float* partial, int T, int topk, int D, void* Y, cudaStream_t st, int sms);
int launch_moe_sort(const int32_t* topk_ids, int T, int topk, int E, int block_m, int32_t* sorted_rows,
                    int32_t* block_expert, int32_t* num_blocks, void* ws, cudaStream_t st);
size_t moe_sort_ws_bytes(int T, int topk, int E);
// Single-launch sort with gather/scatter arrays (cooperative; E <= 4096,
// T*topk <= sms * 32768).  Workspace: histograms + 2 barrier words, zeroed once.
int launch_moe_sort_aux(const int32_t* ids, int T, int topk, int E, int bm, int32_t* sorted_rows,
                        int32_t* block_expert, int32_t* num_blocks, int32_t* sorted_tokens, int32_t* row_slot,
                        void* ws, cudaStream_t st, int sms, unsigned long long wait_ns, unsigned int* status);
size_t moe_sort_aux_ws_bytes(int T, int topk, int E, int sms);

// Routing of tokens to experts (route.cu).
constexpr int kRouteMaxExperts = 2048;
struct RouteArgs {
  const void* logits;           // row t at t * stride
  long long stride;
  const int32_t* count;         // rows from *count on get no experts; nullptr: none
  int T, E;
  const float* bias;            // [E] or nullptr
  int softmax, groups, group_top, top_groups, topk, renorm;
  float scale;
  int32_t* ids;                 // [T, topk]
  float* weights;               // [T, topk]
  // set by the launcher: rows, the bias can be read four values at a time; ceil(2^32 / (E / groups));
  // lanes per group; ceil(E / 4)
  int vectors, bias_vectors;
  unsigned int per_recip;
  int group_lanes, row_quads;
};
int launch_moe_route(RouteArgs p, int bf16, cudaStream_t st);

// Norms and rotation of heads, to rows or to the cache (rope.cu).
struct RopeArgs {
  const uint16_t *q, *k, *v;
  long long q_stride, k_stride, v_stride;
  const int32_t *positions, *slot_map;
  int T, Hq, Hkv;
  const float *q_weight, *k_weight;      // [D] or nullptr: no norm
  float eps;
  const float* inv_freq;                 // [rot / 2]
  int rot, interleaved;
  uint16_t *q_out, *k_out;
  long long q_out_stride, k_out_stride;
  uint8_t* cache;                        // nullptr: keys go to k_out
  int slots, page_lg;
  unsigned long long wait_ns;
  unsigned int* status;
  // set by the launcher: parts of a token, each a block's; units (256 / D heads) of a part, of queries
  // and of keys; bytes of a part's heads
  int split, part_q, part_kv, stage_bytes;
};
int launch_kv_rope(RopeArgs p, int D, cudaStream_t st, int sms);

// 8-bit block-scaled product (w8a8.cu).
struct W8Plan {
  int x_tiles, w_tiles;   // of 128 tokens and of 128 weight rows
  int kt;                 // 128-wide blocks of K
  int half_tiles;         // tiles of 128 x 256 of the last partial wave, run as halves
  size_t ws_bytes;        // of quantised activations: more than 32 tokens
};
W8Plan plan_w8a8(int M, int N, int K, int sms);
int launch_w8a8(const W8Plan& plan, const void* A, int M, int K, const void* W8, const float* Ws, int N, void* C,
                void* ws, cudaStream_t st, unsigned long long wait_ns, unsigned int* status, int prefetch_w, int sms);
int launch_prepare_w8(const void* w_bf16, int N, int K, void* w8, float* ws, cudaStream_t st);
int launch_shuffle_w8(const void* w_e4m3, int N, int K, void* w8, cudaStream_t st, int sms);

// Paged MXFP4 key/value cache (kv.cu) and attention over it (kv_attention.cu).
int launch_kv_plan(const int32_t* past_lens, const int32_t* new_lens, int B, int page_size, int32_t* block_table,
                   int max_pages, int32_t* free_ring, int ring_size, const int32_t* ring_state,
                   int32_t* ring_state_out, int32_t* kv_lens, int32_t* cu_new, int32_t* slot_map, int32_t* positions,
                   int max_tokens, int32_t* refused, cudaStream_t st, int sms);
int launch_kv_append(const void* k, long long k_stride, const void* v, long long v_stride, const int32_t* slot_map,
                     int T, int Hkv, int D, void* cache, int num_pages, int page_size, cudaStream_t st);
int launch_kv_read(const void* cache, int num_pages, int page_size, const int32_t* slot_map, int T, int Hkv, int D,
                   void* k, void* v, cudaStream_t st);

struct KvAttentionArgs {
  const uint16_t* q;            // row t, head h at q + t * q_stride + h * D
  long long q_stride;
  const int32_t* cu_q;          // [B + 1]
  const int32_t* kv_lens;       // [B]
  const int32_t* block_table;   // [B, max_pages]
  const uint8_t* cache;
  uint16_t* out;                // [total_q, Hq, D]
  float* lse;                   // [total_q, Hq] or nullptr
  void* ws;
  int B, total_q, max_q, max_pages, num_pages, page_size, Hq, Hkv;
  float sm_scale;
  unsigned int group_recip;     // ceil(65536 / G), G = Hq / Hkv
  unsigned long long wait_ns;
  unsigned int* status;
#ifdef __CUDACC__
  // new token of row r of a key/value head's rows (r < 256, G <= 256: exact)
  __device__ __forceinline__ int row_of(int r) const { return static_cast<int>(r * group_recip >> 16); }
#endif
};
size_t kv_attention_ws_bytes(int max_q, int group, int D, int sms);
int launch_kv_attention(const KvAttentionArgs& p, int D, cudaStream_t st, int sms);
// Few query rows (max_q * Hq / Hkv) per key/value head (kv_decode.cu).  -1: more work than it counts.
size_t kv_decode_ws_bytes(int rows, int D, int sms);
int launch_kv_decode(const KvAttentionArgs& p, int D, cudaStream_t st, int sms);
// Any number of rows, Hq / Hkv <= 256 (kv_prefill.cu).  -1: more work than it counts.
size_t kv_prefill_ws_bytes(int D, int sms);
int launch_kv_prefill(const KvAttentionArgs& p, int D, cudaStream_t st, int sms);

}  // namespace a4w4
