// Shared parts of the paged 4-bit key/value cache (include/block_kv.h).
#pragma once

#include "paged_kv.cuh"
#include "../../include/block_kv.h"

namespace moe {

constexpr int kMaxBlockBatch = 1 << 20;

// A power of two from 2^-60 to 2^60.
inline bool gscale_ok(float g) {
  int e;
  return std::isfinite(g) && std::frexp(g, &e) == 0.5f && e >= -59 && e <= 61;
}

// The cache's geometry (everything but its pointers and the page table's contents).
inline bool blockkv_shape_ok(const moe_blockkv_cache_t* c) {
  if (!c) return false;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128) return false;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return false;
  if (c->n_pages < 1 || c->max_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 1024) return false;
  // positions are 32-bit
  if (static_cast<int64_t>(c->max_pages) * c->page_size > (int64_t(1) << 30)) return false;
  const int64_t s[3] = {c->page_stride, c->head_stride, c->token_stride};
  for (int64_t v : s)
    if (v < c->head_dim / 2 || v % 16 != 0) return false;
  const int64_t row = c->head_dim / 16, b[3] = {c->scale_page_stride, c->scale_head_stride, c->scale_token_stride};
  for (int64_t v : b)
    if (v < row || v % row != 0) return false;
  // offsets of pages are counted in 32 bits, in units of 16 bytes and of a row of scales
  const int64_t most = (int64_t(1) << 32) - 1, pages = c->n_pages;
  if (c->page_stride / 16 > most / pages || c->scale_page_stride / row > most / pages) return false;
  return gscale_ok(c->k_gscale) && gscale_ok(c->v_gscale);
}

inline bool blockkv_pointers_ok(const moe_blockkv_cache_t* c) {
  const size_t row = c->head_dim / 16;
  return c->k && c->v && c->k_scale && c->v_scale && c->page_table && aligned_to(c->k, 16) && aligned_to(c->v, 16) &&
         aligned_to(c->k_scale, row) && aligned_to(c->v_scale, row) && aligned_to(c->page_table, 4);
}

// The groups of 16 slots that an append writes or a read takes are dealt to blocks:
// request b's start at item cu[b]/16 + 2b, as its n new tokens touch at most n/16 + 2
// of them.  The group that `item` stands for, counted from position 0; -1: none.
// (Counted in groups: a length may be anything up to 2^31 - 1, and the position behind
// the last group would not fit.)
constexpr int kSlots = 16;
__device__ __forceinline__ int slot_group(const Request& r, int b, int item) {
  const int at = item - (r.row0 / kSlots + 2 * b), group = r.start / kSlots + at;
  return r.n > 0 && at >= 0 && group <= (r.end - 1) / kSlots ? group : -1;
}

}  // namespace moe
