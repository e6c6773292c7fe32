/*
 * a4w4.h -- C ABI of the GB300 (sm_103a) MXFP4 A4W4 GEMM library (liba4w4.so).
 *
 * What it computes
 *   "[gfx950][FlyDSL] Add direct dense A4W4 MXFP4 GEMM", Summary and
 *   Implementation: BF16 activations are quantised inline to MXFP4 (E2M1 codes,
 *   one E8M0 power-of-two scale per 32 consecutive K elements) and multiplied
 *   against MXFP4 weights that the caller quantised and preshuffled once, with
 *   fp32 accumulation and BF16 output.  "[gfx1250] Fuse A4W4 stage1 FP4
 *   quantization", Summary: the grouped-MoE GEMM1 variant applies SwiGLU and
 *   emits MXFP4 codes and E8M0 scales directly.
 *
 *   Quantisation rule (OCP MX v1.0; the pages do not state one): per 32-block,
 *   e = floor(log2(max|x|)) - 2 clamped to [-127, 127] (-127 for an all-zero
 *   block), E8M0 code = e + 127, element code = sign << 3 | E2M1 index of
 *   |x| / 2^e rounded to nearest, ties to even, saturating at 6.
 *
 * Conventions for every call
 *   - Pointers named *_bf16 / Wq / Ws / q / scales / out_* are DEVICE pointers
 *     to caller-owned memory, 16-byte aligned, contiguous, row-major.  The
 *     library allocates no device memory and keeps no pointer after a call.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Work is
 *     only enqueued; no call synchronises except a4w4_get_device_status().
 *   - Packed E2M1: element 2j in the low nibble of byte j, 2j+1 in the high one.
 *   - Return codes: A4W4_OK or a negative A4W4_ERR_* (a4w4_strerror names it).
 *     Argument errors are detected before anything is enqueued.
 *   - Every kernel bounds its waits; a wait that runs out records
 *     A4W4_ERR_TIMEOUT in a device status word and the kernel returns early.
 *
 * Thread safety: calls may be issued from several host threads; calls that run
 * concurrently on the GPU must not share output buffers or a workspace.
 */
#ifndef A4W4_H_
#define A4W4_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

enum {
  A4W4_OK = 0,
  A4W4_ERR_ARG = -1,        /* null/misaligned pointer, or a shape outside the contract */
  A4W4_ERR_DEVICE = -2,     /* current device is not compute capability 10.3 (GB300) */
  A4W4_ERR_WORKSPACE = -3,  /* workspace smaller than a4w4_*_workspace_bytes() */
  A4W4_ERR_LAUNCH = -4,     /* a CUDA launch or API call failed */
  A4W4_ERR_TIMEOUT = -5     /* a bounded in-kernel wait expired (read by get_device_status) */
};

/* ------------------------------------------------------------------------ */
/* Weights: quantise + preshuffle once.
 * "[gfx950][FlyDSL] Add direct dense A4W4 MXFP4 GEMM", Implementation ("one-time
 * packed E2M1 weight and E8M0 scale preshuffle") and Scope ("N divisible by 256;
 * K divisible by 128"; "preshuffled once by the caller").
 *
 * Preshuffled layout (GB300 tensor-core operand tiles; KP = K rounded up to a
 * multiple of 256, KT = KP / 256, row tiles of 128 rows, nt = n / 128,
 * kt = k / 256, r = n % 128, atom = ((nt / 2) * KT + kt) * 2 + nt % 2: the two
 * 128-row atoms of a 256-row tile and one K tile are adjacent, so a GEMM tile
 * fetches them with one bulk copy):
 *   Wq: atom-major tiles of 16384 bytes.  Byte b (0..127) of row r of a tile
 *       holds the codes of k = kt*256 + 2b (low nibble) and 2b+1 (high nibble)
 *       at offset  atom*16384 + (r/8)*1024 + (r%8)*128 + ((b/16) ^ (r%8))*16 + b%16
 *       (the 128-byte swizzle of the tensor core's K-major shared-memory tiles).
 *   Ws: tiles of 1024 bytes.  The E8M0 scale of 32-block j (0..7) of tile
 *       (nt, kt) for row r is at  atom*1024 + (j/4)*512 + (r%32)*16 + (r/32)*4 + j%4.
 *   Codes and scales for k >= K are zero.
 */
size_t a4w4_weight_codes_bytes(int N, int K);   /* N * KP / 2  */
size_t a4w4_weight_scales_bytes(int N, int K);  /* N * KP / 32 */

/* W_bf16 [N, K] -> Wq, Ws (sizes above).  N % 256 == 0, K % 128 == 0, N,K > 0. */
int a4w4_prepare_gemm_weight(const void* W_bf16, int N, int K, void* Wq, void* Ws,
                             void* stream);

/* ------------------------------------------------------------------------ */
/* Dense A4W4 GEMM:  C[M, N] (BF16) = MXFP4(A)[M, K] x MXFP4(W)[N, K]^T.
 * "[gfx950][FlyDSL] Add direct dense A4W4 MXFP4 GEMM", Summary, Implementation
 * (inline activation quant, BF16 direct output, M-tail masking), Scope.
 *   A_bf16 [M, K] row-major; Wq, Ws from a4w4_prepare_gemm_weight(N, K);
 *   C_bf16 [M, N] row-major, rows >= M are never touched.
 *   M >= 1, N % 256 == 0, K % 128 == 0.
 * Small M uses weights-as-rows tiles (swap-AB) with split-K over the SMs,
 * reduced inside thread-block clusters (no workspace).  Larger M (M > 128;
 * M > 64 when N >= 4096) quantises the activations once into tiles, held in
 * `workspace`, and runs whole 128 x 256 output tiles (no split-K).  The
 * workspace must hold at least a4w4_gemm_workspace_bytes(M, N, K) bytes
 * (a4w4_workspace_init may zero it; its contents are overwritten before they
 * are read).  When that size is 0 the workspace may be NULL.  Every reduction
 * order is fixed, so results are bitwise deterministic. */
size_t a4w4_gemm_workspace_bytes(int M, int N, int K);
int a4w4_workspace_init(void* workspace, size_t ws_bytes, void* stream);
/* Name of the kernel instantiation a4w4_gemm(M, N, K) launches on the current
 * device (planned for GB300's 152 SMs when no device is visible), e.g.
 * "a4w4_decode_kernel<16,3>" (tokens per CTA, weight ring depth) or
 * "a4w4_gemm_kernel<swap,32>" / "a4w4_large_kernel<prequant,persistent>";
 * the quantise-once plans also launch the activation pre-pass.  Host-only, no
 * device work.  Writes a NUL-terminated string of at most n bytes (truncated)
 * into buf.  Returns A4W4_OK, or A4W4_ERR_ARG for a shape a4w4_gemm rejects,
 * a NULL buf or n == 0. */
int a4w4_gemm_kernel_name(int M, int N, int K, char* buf, size_t n);
int a4w4_gemm(const void* A_bf16, int M, int K, const void* Wq, const void* Ws, int N,
              void* C_bf16, void* workspace, size_t ws_bytes, void* stream);

/* a4w4_gemm with per-call options; a4w4_gemm(...) is a4w4_gemm_ex(..., 0, stream).
 * Flags (unknown bits give A4W4_ERR_ARG):
 *   A4W4_GEMM_WEIGHT_PREFETCH -- the GEMM is launched with programmatic
 *     dependent launch like every GEMM here (it may start while the previous
 *     kernel on `stream` still runs, and waits for that kernel before it
 *     touches A, C or the workspace); with this flag it also starts streaming
 *     Wq/Ws before that wait, hiding the weight fetch behind the previous
 *     kernel.  Set it only when the kernel issued just before this call on
 *     the same stream does not write Wq or Ws (weights prepared earlier and
 *     left unchanged, as in inference).  The promise covers this call alone. */
enum { A4W4_GEMM_WEIGHT_PREFETCH = 1 };
int a4w4_gemm_ex(const void* A_bf16, int M, int K, const void* Wq, const void* Ws, int N,
                 void* C_bf16, void* workspace, size_t ws_bytes, unsigned int flags, void* stream);

/* ------------------------------------------------------------------------ */
/* A16WFP4 GEMM:  C[M, N] (BF16) = A[M, K] (BF16, not quantised) x MXFP4(W)^T.
 * "[gfx950][FlyDSL] Add direct dense A4W4 MXFP4 GEMM", Summary (the #4772
 * bullet: BF16 activation x decoded MXFP4 weight).  Same arguments, layouts
 * and shape contract as a4w4_gemm_ex with the same preshuffled Wq/Ws; no
 * workspace.  Each weight tile is decoded to BF16 on chip (exact for E8M0
 * scales from 2^-127 to 2^125, i.e. weight blocks whose largest magnitude is
 * below 2^127) and multiplied in BF16 with fp32 accumulation; split-K is
 * reduced inside thread-block clusters in a fixed order (deterministic).
 * flags: A4W4_GEMM_WEIGHT_PREFETCH as for a4w4_gemm_ex. */
int a4w4_gemm_a16w4(const void* A_bf16, int M, int K, const void* Wq, const void* Ws, int N,
                    void* C_bf16, unsigned int flags, void* stream);

/* ------------------------------------------------------------------------ */
/* 8-bit GEMM with a scale for each block of 128:  C[M, N] (BF16) = A[M, K] x W[N, K]^T
 * (no counterpart on the source pages: the projections that a model with 4-bit experts
 * keeps in 8 bits).
 *   Weights: E4M3 codes with a float scale for each 128 x 128 block, Ws [N/128, K/128].
 *   Activations: BF16, quantised here to E4M3 with a power-of-two scale for each row and
 *   128 k's: 2^e with the smallest e >= -126 such that the block's largest magnitude is
 *   at most 448 * 2^e; the code is x * 2^-e (exact) rounded to nearest, ties to even.  An
 *   infinity or NaN makes its row of C NaN (an infinity by its block's scale, a NaN by its code).
 *   C[m, n] = sum over blocks b of 2^e[m,b] * Ws[n/128, b] * (sum over b's k's of the
 *   codes' products), every sum and 2^e * Ws in fp32 (what lies below 2^-126 loses bits), in
 *   an order fixed by the sizes and the device: bitwise deterministic.
 * N % 128 == 0, K % 128 == 0, M >= 1; rows >= M of C are never touched.  A checkpoint's
 * other N: pad its codes with rows of zeros to a multiple of 128 (its last blocks' scales
 * stay); C then has that many columns, the padding's zero.  Other K: columns of zeros, of A too.
 *
 * Weight tiles: tile (nt, kt) = rows 128 nt .., k's 128 kt .. at byte (nt * (K/128) + kt) *
 * 16384; byte b of row r at (r/8)*1024 + (r%8)*128 + ((b/16) ^ (r%8))*16 + b%16.
 * a4w4_shuffle_w8_weight lays out a checkpoint's codes [N, K] (its scales are used as they
 * are; W8 is not W_e4m3); a4w4_prepare_w8_weight quantises BF16 weights, Ws = largest
 * magnitude / 448, code = w / Ws rounded to nearest. */
size_t a4w4_w8_weight_bytes(int N, int K);   /* N * K */
int a4w4_prepare_w8_weight(const void* W_bf16, int N, int K, void* W8, float* Ws, void* stream);
int a4w4_shuffle_w8_weight(const void* W_e4m3, int N, int K, void* W8, void* stream);
/* M > 32 may quantise the activations once into tiles in `workspace` (at least
 * a4w4_gemm_w8a8_workspace_bytes(M, N, K), which grows with M; 16-byte aligned,
 * overwritten before it is read); where that size is 0 it may be NULL.  flags:
 * A4W4_GEMM_WEIGHT_PREFETCH as for a4w4_gemm_ex (of W8 alone). */
size_t a4w4_gemm_w8a8_workspace_bytes(int M, int N, int K);
int a4w4_gemm_w8a8(const void* A_bf16, int M, int K, const void* W8, const float* Ws, int N, void* C_bf16,
                   void* workspace, size_t ws_bytes, unsigned int flags, void* stream);

/* ------------------------------------------------------------------------ */
/* Standalone MXFP4 quantisation (plain layout).
 * "[gfx1250] Fuse A4W4 stage1 FP4 quantization", Summary (the standalone quant
 * kept as the fallback path).
 *   X_bf16 [rows, cols] -> q [rows, cols/2] packed codes, scales [rows, cols/32]
 *   E8M0 bytes, both row-major.  rows >= 1, cols % 32 == 0. */
int a4w4_mxfp4_quant(const void* X_bf16, int rows, int cols, void* q, void* scales,
                     void* stream);

/* ------------------------------------------------------------------------ */
/* Grouped MoE GEMM1 (gate+up projection, SwiGLU, MXFP4 requant).
 * "[gfx1250] Fuse A4W4 stage1 FP4 quantization", Summary and Performance;
 * "[HIP] [CK] [FlyDSL] [Kernel] Extend MXFP4 GEMM1 replacement to A4W4", Summary
 * (auxiliary sort of routed rows into per-expert blocks).
 *
 * Expert weights W1_bf16 [E, 2I, D]: rows 0..I-1 are the gate projection,
 * rows I..2I-1 the up projection.  a4w4_moe_prepare_w1 writes, per expert, the
 * dense preshuffled layout above of the row-reordered matrix whose 256-row
 * tile j holds gate rows 128j..128j+127 followed by up rows 128j..128j+127
 * (so one accumulator tile holds matching gate/up columns).  Expert e starts
 * at e * a4w4_weight_codes_bytes(2I, D) in W1q and e * a4w4_weight_scales_bytes(2I, D)
 * in W1s.  I % 128 == 0, D % 128 == 0. */
size_t a4w4_moe_w1_codes_bytes(int E, int two_I, int D);
size_t a4w4_moe_w1_scales_bytes(int E, int two_I, int D);
int a4w4_moe_prepare_w1(const void* W1_bf16, int E, int two_I, int D, void* W1q, void* W1s,
                        void* stream);

/* Sort of routed rows.  Routed row r = t * topk + k sends token t to expert
 * topk_ids[t, k] (int32 [T, topk], values in [0, E)).  Output: for experts
 * e = 0..E-1 in order, the rows routed to e in increasing r, padded with the
 * sentinel T*topk to a multiple of block_m (16, 32, 64 or 128);
 * sorted_rows[b*block_m + i] lists block b, block_expert[b] is its expert,
 * *num_blocks the block count (all on the device, no host synchronisation).
 * Buffers: sorted_rows >= a4w4_moe_max_blocks(T, topk, E, block_m) * block_m
 * entries, block_expert >= a4w4_moe_max_blocks(...) entries, num_blocks 1 entry,
 * ws >= a4w4_moe_sort_workspace_bytes(T, topk, E). */
int a4w4_moe_max_blocks(int T, int topk, int E, int block_m);
size_t a4w4_moe_sort_workspace_bytes(int T, int topk, int E);
int a4w4_moe_sort(const int32_t* topk_ids, int T, int topk, int E, int block_m,
                  int32_t* sorted_rows, int32_t* block_expert, int32_t* num_blocks,
                  void* ws, size_t ws_bytes, void* stream);

/* Experts of each token and their weights from a router's logits, as a4w4_moe_sort
 * and a4w4_moe_gemm2 take them (no counterpart on the source pages, which begin
 * with the routed rows).
 *   logits   row t holds E values at element t * stride: float (A4W4_F32) or BF16
 *            (A4W4_BF16), aligned to its elements; stride >= E when T > 1
 *   score    s = softmax over the E logits, or sigmoid of each
 *   bias [E] float or NULL; c = s + bias decides who is chosen, s alone is the weight
 *   groups   of E / groups consecutive experts; the strength of a group is the sum
 *            of its group_top (1 or 2) largest c, and the top_groups strongest take
 *            part.  groups = 1: no groups (group_top, top_groups are 1 or any others
 *            that the limits allow)
 *   topk_ids [T, topk], topk_weights [T, topk]  the topk largest c, largest first;
 *            weights s * scale, or with renormalise = 1 s / (sum of the topk s) * scale
 *   num_tokens [1] or NULL: on the device, rows from *num_tokens on get ids -1 and
 *            weights 0 (rows of padding of a captured step; the sorts leave them out,
 *            and what a4w4_moe_gemm2 writes to those rows of Y is not defined)
 * Ties go to the lower index.  What is chosen, and the order, are those of the exact
 * c (to about 2^-50 of the largest score): fp32 first, then sums of two floats for the
 * candidates of a row whose order that leaves open (near ties of scores with a bias or
 * of group strengths: some 1% of rows), then 64 bits.  A NaN logit counts as -infinity, a
 * logit of +infinity as the largest float, a NaN bias as -infinity; a row whose logits
 * are all -infinity has scores 0, and weights whose sum is 0 are 0.  The weights are
 * fp32, each within 2^-18.7 of itself (some 2^-21 in practice) however far the logits
 * lie apart, above 2^-126.
 * 1 <= E <= 2048, groups <= 32, E % groups == 0, two experts to a group at least
 * where there are several, 1 <= topk <= 32, topk <= top_groups * E / groups, scale
 * finite, T >= 0, T * topk <= 2^30. */
enum { A4W4_F32 = 0, A4W4_BF16 = 1 };
enum { A4W4_MOE_SCORE_SOFTMAX = 0, A4W4_MOE_SCORE_SIGMOID = 1 };
int a4w4_moe_route(const void* logits, int logits_type, long long stride, const int32_t* num_tokens, int T, int E,
                   int score, const float* bias, int groups, int group_top, int top_groups, int topk, int renormalise,
                   float scale, int32_t* topk_ids, float* topk_weights, void* stream);

/* The same sort, with the auxiliary gather/scatter arrays, in one launch for
 * up to 2048 routed rows and two beyond.
 * "[HIP] [CK] [FlyDSL] [Kernel] Extend MXFP4 GEMM1 replacement to A4W4",
 * Summary (the adaptive MoE auxiliary sort; its review names the aux arrays
 * the sort emits for A4W4).  sorted_rows, block_expert and num_blocks are
 * identical to a4w4_moe_sort's; in addition sorted_tokens[s] is the token
 * (r / topk) of sorted slot s, or T for a padding slot (same length as
 * sorted_rows), and row_slot[r] is the slot that holds routed row r (int32
 * [T*topk]).  Up to 2048 routed rows (a decode batch) one CTA does the whole
 * sort; beyond, up to one CTA per SM each counts a run of rows, the last to
 * finish scans the counts, and a second launch places the rows.  E <= 4096,
 * T*topk <= 32768 x the SM count.  ws >= a4w4_moe_sort_aux_workspace_bytes(T,
 * topk, E) bytes, 16-byte aligned, zeroed once with a4w4_workspace_init (it
 * ends with a ticket counter that the last counting CTA resets). */
size_t a4w4_moe_sort_aux_workspace_bytes(int T, int topk, int E);
int a4w4_moe_sort_aux(const int32_t* topk_ids, int T, int topk, int E, int block_m,
                      int32_t* sorted_rows, int32_t* block_expert, int32_t* num_blocks,
                      int32_t* sorted_tokens, int32_t* row_slot, void* ws, size_t ws_bytes,
                      void* stream);

/* GEMM1 over sorted rows (block_m must be 128).  For every routed row r listed
 * by the sort: g = MXFP4(X[t]) . MXFP4(W1[e, gate rows]), u = ... (up rows),
 * h = silu(g) * u in fp32 (silu(g) = g / (1 + exp(-g)); no clamp, no bias,
 * top-k weights not applied), and h is requantised with the rule above:
 * out_q [T*topk, I/2] packed codes and out_s [T*topk, I/32] E8M0 bytes, row r.
 * X_bf16 [T, D]; W1q/W1s from a4w4_moe_prepare_w1.
 * Activation quantisation: with ws == NULL and ws_bytes == 0 each GEMM tile
 * quantises its gathered rows inline (as on the source pages).  Given a
 * workspace of at least a4w4_moe_gemm1_workspace_bytes(T, D) bytes, the tokens
 * are quantised once into it (codes [T, D/2] then scales [T, D/32]) and the
 * tiles gather those rows: each token feeds topk rows times I/128 tiles, so
 * this is the faster choice once T reaches a few tokens.  Same results. */
size_t a4w4_moe_gemm1_workspace_bytes(int T, int D);
int a4w4_moe_gemm1(const void* X_bf16, int T, int D, const int32_t* sorted_rows,
                   const int32_t* block_expert, const int32_t* num_blocks, int topk,
                   const void* W1q, const void* W1s, int E, int I, void* out_q, void* out_s,
                   void* ws, size_t ws_bytes, void* stream);

/* GEMM1 with a choice of activation and output layout; a4w4_moe_gemm1(...) is
 * a4w4_moe_gemm1_ex(..., A4W4_MOE_ACT_SWIGLU, A4W4_MOE_OUT_ROWS, ...).
 * "[gfx1250] Fuse A4W4 stage1 FP4 quantization", Summary: the epilogue emits
 * packed MXFP4 payloads and preshuffled E8M0 scales after SiLU or SwiGLU.
 *   activation:
 *     A4W4_MOE_ACT_SWIGLU  W1 prepared by a4w4_moe_prepare_w1 from [E, 2I, D]
 *                          (gate rows then up rows); h = silu(gate) * up.
 *     A4W4_MOE_ACT_SILU    the ungated form: W1[e] is [I, D], prepared as one
 *                          dense matrix [E*I, D] by a4w4_prepare_gemm_weight
 *                          (expert e starts at e * a4w4_weight_codes_bytes(I, D)
 *                          in W1q, e * a4w4_weight_scales_bytes(I, D) in W1s);
 *                          h = silu(x . w).  I % 256 == 0.
 *   out_layout:
 *     A4W4_MOE_OUT_ROWS    out_q [T*topk, I/2], out_s [T*topk, I/32], row r =
 *                          routed row r (as a4w4_moe_gemm1).
 *     A4W4_MOE_OUT_TILES   the operand layout a4w4_moe_gemm2 reads: for sorted
 *                          block b (128 slots) and K tile kt (256 of the I
 *                          columns; KT = I/256), atom a = b*KT + kt holds the
 *                          codes of slot b*128 + r at out_q + a*16384 in the Wq
 *                          tile layout above (row r, byte b') and its E8M0 scales
 *                          at out_s + a*1024 in the Ws layout; padding slots
 *                          hold zeros.  Sizes a4w4_moe_tiles_codes_bytes /
 *                          _scales_bytes; tiles of blocks at or beyond
 *                          *num_blocks are not written.  I % 256 == 0. */
enum { A4W4_MOE_ACT_SWIGLU = 0, A4W4_MOE_ACT_SILU = 1 };
enum { A4W4_MOE_OUT_ROWS = 0, A4W4_MOE_OUT_TILES = 1 };
size_t a4w4_moe_tiles_codes_bytes(int T, int topk, int E, int I);
size_t a4w4_moe_tiles_scales_bytes(int T, int topk, int E, int I);
int a4w4_moe_gemm1_ex(const void* X_bf16, int T, int D, const int32_t* sorted_rows,
                      const int32_t* block_expert, const int32_t* num_blocks, int topk,
                      const void* W1q, const void* W1s, int E, int I, int activation, int out_layout,
                      void* out_q, void* out_s, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Grouped MoE GEMM2 (down projection) with the top-k weighted per-token sum.
 * "[HIP] [CK] [FlyDSL] [Kernel] Extend MXFP4 GEMM1 replacement to A4W4",
 * Summary (stage-2 paths that consume stage 1's layout) and GEMM2 scope.
 *   Y[t, :] = sum_k topk_weights[t, k] * MXFP4(W2[e_tk]) . a~_(t*topk+k)
 * with a~ GEMM1's MXFP4 output in A4W4_MOE_OUT_TILES layout (A_q, A_s; I
 * columns), the same sort as GEMM1 (sorted_rows, block_expert, num_blocks,
 * block_m 128), topk_weights float32 [T, topk] (4-byte aligned), W2q/W2s the
 * dense preshuffled layout of the stacked [E*D, I] matrix
 * (a4w4_prepare_gemm_weight; expert e at e * a4w4_weight_codes_bytes(D, I) and
 * e * a4w4_weight_scales_bytes(D, I)), Y_bf16 [T, D].
 * Each routed row's product is scaled by its weight in fp32 and stored as an
 * fp32 row of the workspace ([T*topk, D], a4w4_moe_gemm2_workspace_bytes);
 * a second kernel adds a token's rows in k order (bitwise deterministic) and
 * rounds to BF16.  I % 256 == 0, I <= 1024, D % 256 == 0. */
size_t a4w4_moe_gemm2_workspace_bytes(int T, int topk, int D);
int a4w4_moe_gemm2(const void* A_q, const void* A_s, int T, int I, const int32_t* sorted_rows,
                   const int32_t* block_expert, const int32_t* num_blocks, int topk,
                   const float* topk_weights, const void* W2q, const void* W2s, int E, int D,
                   void* Y_bf16, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Dense A4W4 GEMM that allocates nothing (no counterpart on the source pages:
 * it exists for callers of this library).  Same arguments and result as
 * a4w4_gemm() minus the workspace: the same plan, kernels and reduction order,
 * so the output is bit-identical.  For callers that cannot allocate device
 * memory where they call the GEMM -- code under a framework allocator that
 * owns all device memory, or a latency-critical path that cannot afford
 * cudaMalloc's implicit synchronisation -- and so cannot hand a4w4_gemm() the
 * workspace its plan needs for M > 64: the activations quantised once into
 * MXFP4 tiles (64 < M <= 128 when N >= 4096, every M > 128).  Smaller M uses
 * no scratch.
 *   Scratch: a fixed 16 MiB array inside the library's device image.  It comes
 *   into being on a device with the first a4w4_gemm_noalloc call there (the
 *   CUDA runtime loads the library's device code lazily), which also looks up
 *   its device address, whatever the shape; make that first call before any
 *   stream capture.  It stays until the process exits.  No call allocates.
 *   A plan needing more than 16 MiB (a4w4_gemm_workspace_bytes(M, N, K) >
 *   16 MiB: at K = 7168, M above about 4,400 rows) is refused with
 *   A4W4_ERR_WORKSPACE.  All calls on a GPU share the array and it keeps the
 *   last call's contents (overwritten before they are read); calls that may
 *   run at the same time on one GPU (different streams) race on it --
 *   serialise them. */
int a4w4_gemm_noalloc(const void* A_bf16, int M, int K, const void* Wq, const void* Ws, int N,
                      void* C_bf16, void* stream);

/* ------------------------------------------------------------------------ */
/* Paged key/value cache in MXFP4, and attention over it (no counterpart on the
 * source pages: the attention side of a decoder whose GEMMs are the ones above,
 * with the same E2M1 / E8M0 rule).
 *
 * Cache layout.  Pages of page_size tokens (16, 32, 64 or 128), each page_size /
 * 16 chunks of 16 tokens per key/value head.  Chunk c (of page_size / 16) of
 * head h of page p starts at byte ((p * Hkv + h) * (page_size / 16) + c) * 17 * D
 * and holds, for tokens r = 0..15 of the chunk (D = 64 or 128, J = D / 32):
 *   key codes     8*D bytes   the byte of dimensions n, n+1 (n even) of token r
 *                             at r*(D/2) + (t*J + j)*4 + b, with j = n / 32,
 *                             t = n % 32 / 8, b = n % 8 / 2
 *   key scales    D/2 bytes   E8M0 of 32-block j of token r at r*J + j
 *   value codes   8*D bytes   the byte of dimensions n, n+1 of token r at
 *                             (r/8)*4*D + (g*4 + r%8/2)*(D/8) + (r%2)*(D/16) + i,
 *                             with i = n / 16, g = n % 16 / 2
 *   value scales  D/2 bytes   as the key scales
 * (code of dimension n in the low nibble).  A thread of the attention kernels
 * finds the codes of its tensor-core fragments in one run of bytes: keys in
 * blocks of 8 dimensions, values in pairs of tokens.  Slot s is token
 * s % page_size of page s / page_size. */
size_t a4w4_kv_cache_bytes(int num_pages, int page_size, int Hkv, int D);

/* Block tables, slot map and positions of one serving step, from the requests'
 * lengths, on the device.
 *   past_lens [B]  tokens that each request already has in the cache
 *   new_lens [B]   tokens it appends in this step (0: none); negative: the
 *                  request is finished and gives its pages back
 *   block_table [B, max_pages]  in/out: entry j of row b is the page of request
 *                  b's tokens j*page_size ..; entries of new pages are written
 *   free_ring [ring_size], ring_state [2] = {head, count}: the free pages, oldest
 *                  first, at free_ring[(head + i) % ring_size], i < count
 * Requests are served in order: a request needs ceil((past + new) / page_size) -
 * ceil(past / page_size) pages, taken from the head of the ring.  The first one
 * whose pages (or whose tokens, of max_tokens) do not suffice, and every later
 * one, appends nothing in this step; a request whose past + new exceeds
 * max_pages * page_size appends nothing and holds nobody up.  Pages of finished
 * requests go to the ring's end in request order (ring_size >= all pages) and
 * are taken from the next step on.
 *   ring_state_out [2]  the new {head, count}  (not ring_state itself)
 *   kv_lens [B]         tokens after this step (0 for a finished request; not
 *                       past_lens itself)
 *   cu_new [B + 1]      prefix sums of the tokens appended per request
 *   slot_map [max_tokens], positions [max_tokens]  slot and position of each
 *                       appended token, requests in order; -1 and 0 beyond
 *                       cu_new[B]
 *   refused [1]         requests with new_lens > 0 that append nothing
 * All arrays int32 on the device.  1 <= B <= 4096, page_size 16, 32, 64 or 128,
 * max_pages, ring_size >= 1, max_tokens >= 0, max_pages * page_size < 2^31.  A
 * call that is repeated on its own outputs (same past_lens, new_lens and
 * ring_state) gives the same ones.  A finished request longer than its row of the
 * table gives back max_pages pages.  Precondition: 0 <= past_lens, 0 <= head <
 * ring_size, 0 <= count, table entries of held pages and ring entries are page
 * numbers below 2^31 / page_size. */
int a4w4_kv_plan(const int32_t* past_lens, const int32_t* new_lens, int B, int page_size, int32_t* block_table,
                 int max_pages, int32_t* free_ring, int ring_size, const int32_t* ring_state,
                 int32_t* ring_state_out, int32_t* kv_lens, int32_t* cu_new, int32_t* slot_map,
                 int32_t* positions, int max_tokens, int32_t* refused, void* stream);

/* Quantises T new tokens' keys and values (BF16; the quantisation rule above)
 * into the cache.  Token t's Hkv x D keys start at element t * k_stride of
 * k_bf16 and are contiguous; values likewise (so both may be slices of one fused
 * projection); 16-byte aligned, strides multiples of 8 and at least Hkv * D when
 * T > 1.  A token whose slot is outside [0, num_pages * page_size) is skipped;
 * two tokens with one slot leave either one's bytes.  T >= 0,
 * num_pages * page_size < 2^31. */
int a4w4_kv_append(const void* k_bf16, long long k_stride, const void* v_bf16, long long v_stride,
                   const int32_t* slot_map, int T, int Hkv, int D, void* cache, int num_pages, int page_size,
                   void* stream);

/* Norms of query and key heads and their rotation by position, in one pass.
 * For a head x of D dimensions (BF16):
 *   y = x / sqrt(mean(x^2) + eps) * w      (w = q_weight or k_weight, float [D],
 *                                           16-byte aligned; NULL: y = x)
 *   the first rot_dim dimensions turn by the angles a_i = position * inv_freq[i],
 *   i < rot_dim / 2: pairs (y[i], y[i + rot_dim/2]), or with interleaved = 1 the
 *   neighbours (y[2i], y[2i+1]):  (u, v) -> (u cos a - v sin a, v cos a + u sin a)
 * and the result is rounded to BF16 once.  Token t's Hq heads of queries start at
 * element t * q_stride and are contiguous, its Hkv heads of keys likewise, and the
 * results (all 16-byte aligned, strides multiples of 8 and at least the row when
 * T > 1; all may be slices of one fused projection).  A result may take the place of
 * its input (the same address and stride); else they must not overlap.
 *   positions [T] int32; inv_freq [rot_dim / 2] float, finite, below 2^24 in
 *   magnitude.  Angles are those of exact products to 2^-63 turns, reduced before they
 *   are rounded, so that sines and cosines near zero keep their bits.
 * D 64 or 128, rot_dim a multiple of 16, 0 (norms only; positions and inv_freq may be
 * NULL) to D; Hq, Hkv >= 0 (0: no such heads, its pointers may be NULL),
 * Hq + 2 Hkv <= 4096; eps finite and > 0 where there is a norm; T >= 0. */
int a4w4_qk_norm_rope(const void* q_bf16, long long q_stride, const void* k_bf16, long long k_stride,
                      const int32_t* positions, int T, int Hq, int Hkv, int D, const float* q_weight,
                      const float* k_weight, float eps, const float* inv_freq, int rot_dim, int interleaved,
                      void* q_out_bf16, long long q_out_stride, void* k_out_bf16, long long k_out_stride,
                      void* stream);

/* The same for the queries, with the normed and rotated keys and the values
 * quantised into the cache: a4w4_qk_norm_rope and a4w4_kv_append in one pass, with one
 * rounding fewer: keys are quantised from the unrounded result (their codes and
 * scales are those of the exact value, which is below 2^129 in magnitude unless a
 * weight is enormous; where fp32 leaves open which, 64 bits decide),
 * values as a4w4_kv_append does.  Values are rows like the keys.  A token whose slot is
 * outside [0, num_pages * page_size) is skipped: neither its cells nor its row of
 * q_out are written.  Two tokens with one slot leave either one's bytes.  positions
 * and slot_map are what a4w4_kv_plan writes.  Hq may be 0, Hkv not; the rest as above
 * and as in a4w4_kv_append. */
int a4w4_kv_append_rope(const void* q_bf16, long long q_stride, const void* k_bf16, long long k_stride,
                        const void* v_bf16, long long v_stride, const int32_t* positions, const int32_t* slot_map,
                        int T, int Hq, int Hkv, int D, const float* q_weight, const float* k_weight, float eps,
                        const float* inv_freq, int rot_dim, int interleaved, void* q_out_bf16, long long q_out_stride,
                        void* cache, int num_pages, int page_size, void* stream);

/* The BF16 values (exact) of the cache rows at T slots: k_out, v_out [T, Hkv, D],
 * zeros where the slot is outside [0, num_pages * page_size).  For handing a
 * prefix to other code and for looking at what is cached. */
int a4w4_kv_read(const void* cache, int num_pages, int page_size, const int32_t* slot_map, int T, int Hkv, int D,
                 void* k_out_bf16, void* v_out_bf16, void* stream);

/* Causal attention of the newest tokens of B requests over their cached keys and
 * values (the new tokens' own included: append first).
 *   q_bf16     row t (a new token) holds Hq x D at element t * q_stride
 *              (16-byte aligned, stride a multiple of 8, >= Hq * D)
 *   cu_q [B+1] rows of request b are cu_q[b] .. cu_q[b+1] - 1; at most max_q each
 *              and total_q in all (rows beyond are not computed)
 *   kv_lens [B], block_table [B, max_pages]  as a4w4_kv_plan writes them
 * Query i of the n rows of request b sees the keys at positions 0 .. kv_lens[b] -
 * n + i; query head h reads key/value head h / (Hq / Hkv).
 *   out_bf16 [total_q, Hq, D] = softmax(sm_scale q k^T) v
 *   lse [total_q, Hq] float, or NULL: log sum exp of the scaled scores
 * A row that sees no key (empty request, more queries than keys) gives zeros and
 * lse = -infinity.  Queries, keys and values enter as the values they stand for,
 * but query elements below 2^-28 of their row's largest lose bits, and so do, in
 * larger calls with over 48 rows of a key/value head, key blocks of a scale below
 * 2^-36 of the largest of 128 keys; keys or values of 2^104 and more may overflow
 * the sums.  Sums, softmax statistics and the output accumulator are fp32.
 * Probabilities enter the products in FP16 (11 bits) or, where their range asks
 * for it, in two BF16 terms (16 bits); in the larger calls in BF16 (8 bits; 16 for
 * rows that see up to 128 keys).  Which calls are larger depends on the arguments,
 * the table's width (max_pages) among them; the reduction order on the arguments
 * and the lengths alone: results are bitwise deterministic.
 * Hq % Hkv == 0, Hq / Hkv <= 256, D 64 or 128, sm_scale finite and > 0, B >= 1, total_q >= 0,
 * max_q >= 1, max_pages >= 1, max_pages * page_size < 2^31 - 255, num_pages * page_size < 2^31,
 * total_q * Hq < 2^31, with max_q > total_q also B * max_q * Hq < 2^31, and the work of the largest
 * call that the arguments allow (steps of 32 keys of the table's width for each 8 rows of a key/value
 * head, or of 128 keys for each 256 rows, and up to 4 more for each; as many rows as B * max_q or as
 * total_q and a block more for each request) below 2^31.  Row lists that overlap (cu_q not
 * non-decreasing) stay inside the buffers too, but what is then written is not defined.
 * Lengths are clamped to the table's width and page numbers to [0, num_pages):
 * nothing outside the cache is read.  Workspace: a4w4_kv_attention_workspace_bytes
 * bytes, 16-byte aligned, zeroed once with a4w4_workspace_init (it begins with
 * ticket counters that each call leaves at zero; zero it again after
 * A4W4_ERR_TIMEOUT); calls of any sizes may share one workspace one after
 * another. */
size_t a4w4_kv_attention_workspace_bytes(int B, int max_q, int Hq, int Hkv, int D);
int a4w4_kv_attention(const void* q_bf16, long long q_stride, const int32_t* cu_q, int B, int total_q, int max_q,
                      const int32_t* kv_lens, const int32_t* block_table, int max_pages, const void* cache,
                      int num_pages, int page_size, int Hq, int Hkv, int D, float sm_scale, void* out_bf16,
                      float* lse, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Synchronises `stream`, then returns and clears the device status word:
 * A4W4_OK, A4W4_ERR_TIMEOUT, or A4W4_ERR_LAUNCH if the stream reported an error. */
int a4w4_get_device_status(void* stream);

/* Static, human-readable name of a return code. */
const char* a4w4_strerror(int code);

/* Override the in-kernel wait limit in nanoseconds (0 restores the default of
 * 2e8 ns).  Applies to launches issued after the call; used to test that an
 * expired wait is reported rather than hanging. */
void a4w4_set_wait_limit_ns(unsigned long long ns);

#ifdef __cplusplus
}
#endif

#endif /* A4W4_H_ */
