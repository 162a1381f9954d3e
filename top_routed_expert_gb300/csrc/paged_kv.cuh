// Shared parts of the paged 8-bit key/value cache (include/paged_kv.h).
#pragma once

#include <cmath>

#include "common.cuh"
#include "../../include/paged_kv.h"

namespace moe {

moe_status_t current_device(unsigned** status, int* num_sms);

constexpr int kMaxBatch = 4096;

inline bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

// The cache's geometry and pointers (everything but the page table's contents).
inline bool kv_cache_shape_ok(const moe_kv_cache_t* c) {
  if (!c) return false;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return false;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return false;
  if (c->n_pages < 1 || c->max_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 1024) return false;
  // positions are 32-bit
  if (static_cast<int64_t>(c->max_pages) * c->page_size > (int64_t(1) << 30)) return false;
  const int64_t s[3] = {c->page_stride, c->head_stride, c->token_stride};
  for (int64_t v : s)
    if (v < c->head_dim || v % 16 != 0) return false;
  return true;
}

inline bool kv_cache_pointers_ok(const moe_kv_cache_t* c) {
  return c->k && c->v && c->k_scale && c->v_scale && c->page_table && aligned_to(c->k, 16) && aligned_to(c->v, 16) &&
         aligned_to(c->k_scale, 4) && aligned_to(c->v_scale, 4) && aligned_to(c->page_table, 4);
}

// A request of the ragged batch: its rows [row0, row0 + n) and the positions
// [start, end) they take.  ok = false: offsets that decrease or leave [0, T].
struct Request {
  int row0, n, start, end;
  bool ok;
};

__device__ __forceinline__ Request load_request(const int32_t* __restrict__ cu, const int32_t* __restrict__ kv_len,
                                                int b, int T) {
  Request r;
  const int lo = cu[b], hi = cu[b + 1];
  r.row0 = lo;
  r.end = max(kv_len[b], 0);
  r.ok = lo >= 0 && hi >= lo && hi <= T;
  r.n = r.ok ? hi - lo : 0;
  r.start = r.end - r.n;
  return r;
}

// The last b in [0, B) with cu[b] * mul / div + b * add <= x, for a
// non-decreasing sequence with cu[0] = 0; the warp looks at 32 places at a
// time, so 4096 requests take three dependent loads.  Every lane gets b.
__device__ __forceinline__ int warp_find_request(const int32_t* __restrict__ cu, int B, int64_t x, int mul, int div,
                                                 int add) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = B;   // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = lo + lane * step;
    const bool below = lane * step < n && static_cast<int64_t>(cu[at]) * mul / div + static_cast<int64_t>(at) * add <= x;
    const unsigned m = __ballot_sync(0xffffffffu, below);
    const int last = m ? 31 - __clz(m) : 0;
    lo += last * step;
    n = min(step, n - last * step);
  }
  return lo;
}

}  // namespace moe
