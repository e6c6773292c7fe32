// kv_attention.cu -- which kernel a call of a4w4_kv_attention runs.
#include "launch.h"

namespace a4w4 {

namespace {

// Rows per key/value head up to which the decode kernel runs.  It goes over the keys
// once per 8 or 16 rows, the tcgen05 kernel once per 256 at the price of a whole
// unit.  4 requests x 16384 keys x 8 heads, rows: decode and prompt kernel, D = 128:
// 16: 34 and 75 us, 32: 57 and 73, 48: 80 and 74, 64: 106 and 73; D = 64: 32: 37 and
// 56, 48: 52 and 56, 64: 68 and 55; 16 x 1000 keys, D = 128: 48: 29 and 35, 64: 37
// and 34.
constexpr int kFewRows = 48;
bool few_rows(int max_q, int group) { return max_q <= kFewRows / group; }

// More rows than that, but so little work (as the table and max_q bound it) that time
// goes into starting and joining, where the decode kernel is faster: steps of 16 rows
// x 32 keys for each of 8 warps per SM.  Steps: decode and prompt kernel, 8 heads of
// 128 unless said otherwise: 0.7 (60 tokens x 200 keys): 8.3 and 12.8 us, 1.7 (2 x 16
// x 1000): 13.5 and 17.8, 3.4 (8 x 16 x 500): 15.3 and 17.5, 4.1 (20 x 4000): 20.4 and
// 25.6, 5.0 (4 ragged x 17 x 1214, D = 64): 12.2 and 13.8, 5.2 (5 ragged x 11 x 3370,
// 16 heads over 2): 13.4 and 26.0, 6.3 (4 x 60 x 500): 23.8 and 19.0, 6.7 (8 x 32 x
// 500): 24.8 and 18.0.
constexpr int kSmallRows = 240;
constexpr int kSmallSteps = 6;
bool small_work(const KvAttentionArgs& p, int group, int sms) {
  if (p.max_q > kSmallRows / group) return false;
  const double steps = static_cast<double>(p.B) * p.Hkv * ((p.max_q * group + 15) / 16) * p.max_pages * p.page_size / 32;
  return steps <= 8.0 * kSmallSteps * sms;
}

}  // namespace

size_t kv_attention_ws_bytes(int max_q, int group, int D, int sms) {
  // the prompt kernel's is larger, so it serves both
  return few_rows(max_q, group) ? kv_decode_ws_bytes(max_q * group, D, sms) : kv_prefill_ws_bytes(D, sms);
}

int launch_kv_attention(const KvAttentionArgs& p, int D, cudaStream_t st, int sms) {
  const int group = p.Hq / p.Hkv;
  return few_rows(p.max_q, group) || small_work(p, group, sms) ? launch_kv_decode(p, D, st, sms)
                                                               : launch_kv_prefill(p, D, st, sms);
}

}  // namespace a4w4
