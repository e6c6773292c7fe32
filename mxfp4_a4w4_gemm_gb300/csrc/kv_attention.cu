// kv_attention.cu -- which kernel a call of a4w4_kv_attention runs.
#include "launch.h"

namespace a4w4 {

namespace {

// The decode kernel holds up to 16 query rows per key/value head; from there on
// the tcgen05 kernel, whose 256-row units decode a key once for all their rows,
// takes over.
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
