// kv_walk.cuh -- how the attention kernels share out ragged work.
//
// A unit is what one softmax runs over for one block of query rows: request b,
// key/value head h (and block of rows).  Its keys are cut into steps; the steps
// of all units, in order, form one line, which is cut into equal runs, one per
// worker: every worker gets the same work to within one step whatever the
// lengths are, and units that are cut are joined afterwards.  What a unit costs
// beside its steps counts as places without work before them.  The cut depends on
// the lengths alone.
#pragma once

#include <cmath>
#include <cstdint>

#include "device.cuh"
#include "launch.h"

namespace a4w4 {

// The first kTickets 32-bit words of the workspace count the CTAs that have
// stored their part of a cut unit (indexed by the unit's first CTA, of which a
// cut unit is the last one); the last to arrive joins the parts and puts the
// counter back to zero.
constexpr int kTickets = 4096;

// Draws a ticket: what the CTA's threads stored before the barrier before this is
// visible to whoever draws later, and what earlier drawers stored is to this CTA
// after its next barrier.
__device__ __forceinline__ int draw_ticket(int* at) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(at) : "memory");
  return old;
}

// mbar_wait for limits of any size: try_wait may suspend the thread for longer than
// these kernels' waits take, so below 100 us the barrier is only tested.
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool kv_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint64_t limit_ns,
                                        unsigned int* status) {
  if (mbar_test(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    if (limit_ns >= 100000ull ? mbar_try_wait(bar, parity) : mbar_test(bar, parity)) return true;
    if (*abort) return false;
    if (global_timer_ns() - t0 > limit_ns) {
      *abort = 1;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
}

// Lengths of request b as the kernels use them: clamped, so that nothing in the
// arrays can lead outside the buffers.
struct KvRequest {
  int row0, rows;   // new tokens: first row, and rows to compute
  int all;          // new tokens as cu_q has them: row i sees the keys below len - all + i + 1
  int len;          // keys
};
__device__ __forceinline__ KvRequest kv_request(const KvAttentionArgs& p, int b) {
  KvRequest r;
  const int c0 = __ldg(p.cu_q + b), c1 = __ldg(p.cu_q + b + 1);
  const int cap = p.max_pages * p.page_size;
  r.row0 = c0;
  r.all = c0 < 0 ? 0 : max(0, c1 - c0);
  r.rows = min(r.all, max(0, min(p.total_q - c0, p.max_q)));
  r.len = max(0, min(__ldg(p.kv_lens + b), cap));
  return r;
}

// Entry i of request b's row of the block table.
__device__ __forceinline__ int kv_page(const KvAttentionArgs& p, int b, int i) {
  const int id = __ldg(p.block_table + static_cast<long long>(b) * p.max_pages + i);
  return min(max(id, 0), p.num_pages - 1);
}

// The cut of the line, or of this CTA's stretch of it: workers v0 .. workers - 1 share
// the places from `base` on, the first `more` of them each + 1, the others `each`.
struct KvShare {
  uint32_t base, v0, workers;
  uint32_t each, more;
  uint32_t per;             // workers of a CTA
  __device__ __forceinline__ void cut(uint32_t from, uint32_t total, uint32_t first_worker, uint32_t n) {
    base = from; v0 = first_worker; workers = first_worker + n;
    each = total / n;
    more = total - each * n;
  }
  __device__ __forceinline__ uint32_t first(uint32_t v) const { return base + (v - v0) * each + min(v - v0, more); }
  // the worker that holds place f
  __device__ __forceinline__ uint32_t holder(uint32_t f) const {
    const uint32_t wide = more * (each + 1), at = f - base;
    return v0 + (at < wide ? at / (each + 1) : more + (at - wide) / each);
  }
};

// Where a worker's run starts: request b, `rest` places after its first.
struct KvStart {
  uint32_t b, rest, places; // places: all of the request's
  KvRequest req;            // request b's lengths
};

__device__ __forceinline__ KvRequest shfl_request(const KvRequest& r, int lane) {
  KvRequest o;
  o.row0 = __shfl_sync(0xFFFFFFFFu, r.row0, lane);
  o.rows = __shfl_sync(0xFFFFFFFFu, r.rows, lane);
  o.all = __shfl_sync(0xFFFFFFFFu, r.all, lane);
  o.len = __shfl_sync(0xFFFFFFFFu, r.len, lane);
  return o;
}

// The line's places are counted in 32 bits.  The launchers see to it that lists of rows (cu_q) that do not overlap give
// fewer than kTooMany; sums stop there, and a line of so many is not walked.
constexpr uint32_t kTooMany = 0x7FFFFFFFu;
__device__ __forceinline__ uint32_t add_places(uint32_t a, uint32_t b) { return min(a + b, kTooMany); }

// Units of B requests (blocks of `rows` of a head's rows), as many as there can be: every request max_q tokens, or
// total_q tokens in all, with one block more for each request that has any.
inline double most_units(const KvAttentionArgs& p, int rows) {
  const int G = p.Hq / p.Hkv;
  const double each = std::ceil(static_cast<double>(p.max_q) * G / rows) * p.B;
  const double all = static_cast<double>(p.total_q) * G / rows + (p.B < p.total_q ? p.B : p.total_q);
  return (each < all ? each : all) * p.Hkv;
}

// Cuts the line (places(r) places for the units of a request with lengths r) for at most gridDim.x * PER workers of at least
// least(the longest unit's) places, at least `few` of them to a CTA; warp w learns the start of worker
// blockIdx.x * per + w, if there is one.  Every thread of the CTA calls it; with
// up to 32 requests each warp finds out for itself, with more they sum together
// (scratch: THREADS + 32 words of shared memory, in use until every warp has
// returned).  Returns false if the CTA has nothing to do.  For few requests, without
// and with the sums of all warps (a barrier): one token over 1000 keys 9.4 and 10.0
// us, 24 requests x 5 tokens 22.0 and 23.2 (both faster since, by their joins).
//
// Short units (unit(r) places each, `cost` of them without work; WHOLE at most) go to
// CTAs whole, those that begin in its equal stretch of the line, which its own warps
// then cut: a join between CTAs takes some 3 us, about as long as a CTA takes for 21
// places more than the others.  Whole and cut, one token, 8 heads of 128: 1 request
// x 100 keys 6.6 and 8.3 us, 8 x 300 7.4 and 8.9, 8 x 1000 10.1 and 11.1, 64 x 300
// 12.9 and 13.9, 256 ragged x 600 29.2 and 31.8; over the limits 1 x 800 9.6 and 8.6,
// 1 x 1000 10.2 and 8.7, 1 x 2000 13.6 and 9.9.
template <int THREADS, int PER, int WHOLE, typename Places, typename Unit, typename Least>
__device__ __forceinline__ bool kv_locate(const KvAttentionArgs& p, Places places, Unit unit, uint32_t cost, Least least,
                                          uint32_t few, uint32_t* scratch, KvShare& share, KvStart& start) {
  constexpr int W = THREADS / 32;
  static_assert(W <= 32 && PER <= W, "a search per warp");
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const bool small = p.B <= 32;
  const int per = small ? 1 : (p.B + THREADS - 1) / THREADS;     // requests per thread
  const int b0 = (small ? lane : tid) * per, b1 = min(p.B, b0 + per);
  KvRequest mine = {0, 0, 0, 0};
  uint32_t sum = 0;
  uint32_t longest = 0;                                          // places of the longest unit
  for (int b = b0; b < b1; ++b) {
    mine = kv_request(p, b);
    const uint32_t n = places(mine);
    sum = add_places(sum, n);
    if (n > 0) longest = max(longest, unit(mine));
  }
  uint32_t inc = sum;                                            // inclusive, within the warp
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, inc, o);
    if (lane >= o) inc = add_places(inc, u);
  }
  uint32_t wsum = 0, total;
  if (small) {
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    total = __shfl_sync(0xFFFFFFFFu, inc, 31);
  } else {
    longest = __reduce_max_sync(0xFFFFFFFFu, longest);
    scratch[tid] = inc;
    if (lane == 0) scratch[THREADS + warp] = longest;
    __syncthreads();
    longest = __reduce_max_sync(0xFFFFFFFFu, lane < W ? scratch[THREADS + lane] : 0u);
    wsum = lane < W ? scratch[lane * 32 + 31] : 0u;              // the warps' sums, scanned by every warp
#pragma unroll
    for (int o = 1; o < W; o <<= 1) {
      const uint32_t u = __shfl_up_sync(0xFFFFFFFFu, wsum, o);
      if (lane >= o) wsum = add_places(wsum, u);
    }
    total = __shfl_sync(0xFFFFFFFFu, wsum, W - 1);
  }
  // the request that holds place f < total: the warp's run of requests, then the thread's, then one by one
  auto find = [&](uint32_t f) {
    uint32_t lo = 0, ti = inc;
    int base = 0;
    if (!small) {
      const int wi = __popc(__ballot_sync(0xFFFFFFFFu, lane < W && wsum <= f));
      const uint32_t wlo = __shfl_sync(0xFFFFFFFFu, wsum, wi > 0 ? wi - 1 : 0);
      lo = wi > 0 ? wlo : 0u;
      ti = scratch[wi * 32 + lane];
      base = wi * 32;
    }
    const int li = __popc(__ballot_sync(0xFFFFFFFFu, lo + ti <= f));
    const uint32_t tlo = __shfl_sync(0xFFFFFFFFu, ti, li > 0 ? li - 1 : 0);
    lo += li > 0 ? tlo : 0u;
    int b = (base + li) * per;
    if (small) {
      start.req = shfl_request(mine, li);
      start.places = __shfl_sync(0xFFFFFFFFu, sum, li);
    } else {
      start.req = kv_request(p, b);
      for (start.places = places(start.req); f >= lo + start.places; start.places = places(start.req)) {
        lo += start.places;
        start.req = kv_request(p, ++b);
      }
    }
    start.b = b;
    start.rest = f - lo;
  };
  if (total == 0 || total == kTooMany) return false;
  if (WHOLE > 0 && longest <= min(static_cast<uint32_t>(WHOLE), 21u + total / gridDim.x)) {
    KvShare even;
    even.cut(0, total, 0, gridDim.x);
    // the first unit that begins at place f or after it
    auto next_unit = [&](uint32_t f) {
      if (f >= total) return total;
      find(f);
      const uint32_t u = unit(start.req);
      return f - start.rest + (start.rest + u - 1) / u * u;
    };
    const uint32_t from = next_unit(even.first(blockIdx.x)), to = next_unit(even.first(blockIdx.x + 1));
    if (from == to) return false;
    // the CTA's first places without work are left out
    share.cut(from + cost, to - from - cost, blockIdx.x * PER, min(static_cast<uint32_t>(PER), to - from - cost));
    share.per = PER;
  } else {
    const uint32_t fewest = least(longest);
    const uint32_t workers = min(static_cast<uint32_t>(gridDim.x) * PER, (total + fewest - 1) / fewest);
    share.cut(0, total, 0, workers);
    share.per = max(few, (workers + gridDim.x - 1) / gridDim.x);
  }
  const uint32_t v = blockIdx.x * share.per;
  if (v >= share.workers) return false;
  if (warp < share.per && v + warp < share.workers) find(share.first(v + warp));
  return true;
}

}  // namespace a4w4
