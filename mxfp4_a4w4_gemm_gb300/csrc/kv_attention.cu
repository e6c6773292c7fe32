// kv_attention.cu -- which kernel a call of a4w4_kv_attention runs.
#include "launch.h"

namespace a4w4 {

namespace {

// Rows per key/value head up to which the decode kernel runs.  It goes over the keys
// once per 8 or 16 rows, the tcgen05 kernel once per 256 at the price of a whole
// unit.  4 requests x 16384 keys x 8 heads, rows: decode and prompt kernel, D = 128:
// 16: 36 and 69 us, 32: 56 and 69, 48: 78 and 71, 64: 100 and 71; D = 64: 32: 38 and
// 56, 48: 51 and 56, 64: 64 and 55; 16 x 1000 keys, D = 128: 48: 34 and 35, 64: 40
// and 36.
constexpr int kFewRows = 48;
bool few_rows(int max_q, int group) { return max_q <= kFewRows / group; }

}  // namespace

size_t kv_attention_ws_bytes(int max_q, int group, int D, int sms) {
  return few_rows(max_q, group) ? kv_decode_ws_bytes(max_q * group, D, sms) : kv_prefill_ws_bytes(D, sms);
}

int launch_kv_attention(const KvAttentionArgs& p, int D, cudaStream_t st, int sms) {
  return few_rows(p.max_q, p.Hq / p.Hkv) ? launch_kv_decode(p, D, st, sms) : launch_kv_prefill(p, D, st, sms);
}

}  // namespace a4w4
