// What the attention kernels over the paged cache share: the call's
// arguments, which cached tokens a request's rows see, and the row store.
#pragma once

#include "paged_kv.cuh"

namespace moe {

// A row tile whose partial sums several CTAs left: rows (0: none), where they
// lie, the first CTA's slot and the last CTA.
struct JoinTile {
  int rows, token0, row0, kvh, slot, last;
};

// The row blocks of paged_attn_tc.cuh: part `part` of `parts` of block `blk` of
// request `b`; the parts of a cut block, for key head h, leave their sums in
// slots (slot + part) n_kv_heads + h.
struct TcList {
  int entries, taken, joins, slots;
};
struct TcEntry {
  int b, blk, part, parts, slot;
};
struct TcJoin {
  int b, blk, parts, slot;
};

struct PaArgs {
  static constexpr bool kBlocks = false;   // a scale for a page and head (paged_kv.h)
  const uint16_t* q;
  uint16_t* out;
  float* lse;
  const int32_t* cu;
  const int32_t* kv_len;
  float* part;          // workspace: partial sums,
  JoinTile* joins;      // the row tile that each CTA leaves to others to finish,
  TcList* tc;           // and for paged_attn_tc.cuh the list of its row blocks
  TcEntry* tc_entries;
  TcJoin* tc_joins;     // ... those cut along the cached tokens,
  float* tc_part;       // and their partial sums: rows of D outputs, then (reference, sum) pairs
  moe_kv_cache_t c;
  unsigned* status;
  int64_t qs, os;
  int T, B, group, window, n_sink;
  int tc_rows;          // requests with more rows (tokens x heads of the group) go to paged_attn_tc.cuh
  int tc_ctas;          // its CTAs
  bool tc_split;        // whether row blocks may be cut
  float sm_scale;
};

// A cache in 4 bits (block_kv.h): c holds its codes, page table and sizes.
struct BlockPaArgs : PaArgs {
  static constexpr bool kBlocks = true;    // ... for a token, head and 16 elements
  const uint8_t* k_scales;
  const uint8_t* v_scales;
  uint32_t page16, page_s;   // page strides in units of 16 bytes, and of D / 16
  int64_t scale_page, scale_head, scale_token;   // strides of the scales
  float kg, vg;                                  // factors of keys and values
  bool whole_tiles;                              // row tiles are not cut, and nothing is joined
};

// What a row's outputs are multiplied by: 1 / sum, and the values' factor.
template <class Args> __device__ __forceinline__ float out_factor(const Args& a, float sum) {
  if constexpr (Args::kBlocks) return sum == 0.f ? 0.f : a.vg / sum;   // 0: nothing visible (a NaN sum is not)
  else return sum == 0.f ? 0.f : 1.0f / sum;
}

constexpr int kTcItemRows = 256;   // rows of an item of paged_attn_tc.cuh
constexpr int kTcStep = 128;       // cached tokens of its steps

// The most CTAs, and the most slots of cut row blocks: a part is at least 3/4 of
// 1/tc_ctas of the work, so that all parts are at most 4/3 of the CTAs.
constexpr int kMaxSms = 160, kTcSlots = kMaxSms * 4 / 3 + 1;

// The most row blocks that the requests of a launch can have, for one key head.
__host__ __device__ inline int64_t tc_places(const PaArgs& a) {
  return static_cast<int64_t>(a.T) * a.group / kTcItemRows + (a.B < kMaxBatch ? a.B : kMaxBatch);
}

// Cached tokens that the new tokens of a request can see, in blocks of `unit`
// tokens: the blocks with the first visible positions of a window's sinks,
// then those from the first windowed position to the end.
struct Span {
  int end, lo, window, n_sink;   // positions [lo, end) and [0, n_sink)
  int sink_blocks, lo_block, units;
  __device__ __forceinline__ int block_of(int u) const { return u < sink_blocks ? u : lo_block + u - sink_blocks; }
  // any row of the request
  __device__ __forceinline__ bool seen(int j) const { return j < end && (j >= lo || j < n_sink); }
  // ... and any position of [j0, j1]
  __device__ __forceinline__ bool any_seen(int j0, int j1) const { return j0 < end && (j1 >= lo || j0 < n_sink); }
  // ... and all of them
  __device__ __forceinline__ bool all_seen(int j0, int j1) const { return j1 < end && (j0 >= lo || j1 < n_sink); }
  // the row at position p
  __device__ __forceinline__ bool sees(int p, int j) const {
    return j <= p && (window == 0 || j > p - window || j < n_sink);
  }
  // every row at positions [p0, p1] sees all of [j0, j1]
  __device__ __forceinline__ bool all_see(int j0, int j1, int p0, int p1) const {
    return j1 <= p0 && (window == 0 || j0 > p1 - window || j1 < n_sink);
  }
};

// p0, p1: positions of the first and last row that the span is for.
__device__ __forceinline__ Span span_for(const PaArgs& a, int p0, int p1, int unit) {
  Span s;
  s.window = a.window;
  s.n_sink = a.window ? a.n_sink : 0;
  s.end = min(max(p1 + 1, 0), a.c.max_pages * a.c.page_size);   // what the page table can hold
  s.lo = a.window ? max(0, p0 - a.window + 1) : 0;
  s.lo_block = min(s.lo, s.end) / unit;
  s.sink_blocks = min(ceil_div(min(s.n_sink, s.end), unit), s.lo_block);
  s.units = max(1, s.sink_blocks + ceil_div(s.end, unit) - s.lo_block);   // at least one: its rows are written
  return s;
}

__device__ __forceinline__ Span span_of(const PaArgs& a, const Request& r, int unit) {
  return span_for(a, r.start, r.end - 1, unit);
}

// Units of a request: all its key heads and row tiles of `rows` rows, each with
// `cost` units more than its tokens make.
__device__ __forceinline__ int64_t units_of(const PaArgs& a, const Request& r, int rows, int unit, int cost) {
  if (r.n * a.group > a.tc_rows) return 0;
  return static_cast<int64_t>(a.c.n_kv_heads) * ceil_div(r.n * a.group, rows) * (span_of(a, r, unit).units + cost);
}

// Units of the call, request by request: start[b] units come before request
// b, start[B] in all.  The whole block calls; `status` records offsets that
// are out of order and lengths past the page table.
template <int ROWS, int UNIT, int COST>
__device__ __forceinline__ void build_unit_table(const PaArgs& a, int64_t* start, unsigned* status) {
  __shared__ int64_t s_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int64_t n = 0;
    if (b < a.B) {
      const Request r = load_request(a.cu, a.kv_len, b, a.T);
      if (!r.ok || r.end > a.c.max_pages * a.c.page_size) set_status(status, MOE_ERR_DEVICE_BOUNDS);
      n = units_of(a, r, ROWS, UNIT, COST);
    }
    int64_t sum = n;   // inclusive prefix over the warp, then over the warps
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += x;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int64_t all = 0, below = 0;
    for (int w = 0; w < warps; ++w) {
      all += s_warp[w];
      below += w < warp ? s_warp[w] : 0;
    }
    if (b < a.B) start[b] = base + below + sum - n;
    base += all;
    __syncthreads();
  }
  if (threadIdx.x == 0) start[a.B] = base;
  __syncthreads();
}

// The request that unit x belongs to (requests without units are skipped).
__device__ __forceinline__ int find_entry(const int64_t* start, int B, int64_t x) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// Units of one CTA's piece of the line.
__device__ __forceinline__ int64_t piece_of(int64_t total, int ctas) {
  return max(int64_t(2), (total + ctas - 1) / ctas);
}

// 2^(m - top) for the join of partial maxima; m = -infinity: an empty part.
__device__ __forceinline__ float ex2_from(float m, float top) { return m == -INFINITY ? 0.f : exp2f(m - top); }

// A row's reference lies kRefBelow (base 2) under the maximum that it is taken
// from.  Weights are f16, 11 bits from 2^-14 on and steps of 2^-24 below, so one
// keeps its 11 bits down to 2^-22 of the row's largest and is off by up to 2^-33 of
// it below that; with the maximum itself as reference these would be 2^-14 and
// 2^-25, and the losses of 65536 tokens 2^-9.  A reference moves when weights (16 of
// a group, or a lane's two) sum to over kMostSum, so that none is over f16's 65504.
// A move costs a step most of its time again, which is why it is 8: 32 x 256
// tokens take 264 us with 0, 266 with 8, 273 with 9, 297 with 10; ragged prompts
// 174, 179, 188, 196.
constexpr float kRefBelow = 8.0f, kMostSum = 65504.0f;

// A key scale times a row's factor, kept above 0: a masked score is -infinity
// and has to stay so (a product that small leaves no score to speak of).
__device__ __forceinline__ float score_factor(float k_scale, float rf) { return fmaxf(k_scale * rf, 1e-37f); }

// The two codes of each of a word's four bytes -> two f16 (the low four bits in the low half).
__device__ __forceinline__ void f16x2_of_e2m1(uint32_t w, uint32_t (&r)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(w));
}
// Codes of elements 0, 2, 4, 6 (even) and 1, 3, 5, 7 (odd) of two tokens, a token's code in each half of a byte.
__device__ __forceinline__ uint32_t even_codes(uint32_t a, uint32_t b) { return (a & 0x0f0f0f0fu) | (b << 4 & 0xf0f0f0f0u); }
__device__ __forceinline__ uint32_t odd_codes(uint32_t a, uint32_t b) { return (a >> 4 & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u); }
// Two E4M3 scales (the low 16 bits) -> two f16, exact.
__device__ __forceinline__ uint32_t f16x2_of_scales(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 t, u;\n mov.b32 {t, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
// A code times its scale: six significant bits, 2^-10 to 2688, exact in f16.
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t x, uint32_t y) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(x), "r"(y));
  return r;
}
// One half of two in both places (the multiplication takes it from where it is).
__device__ __forceinline__ uint32_t low_twice(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n mov.b32 %0, {l, l};\n}\n" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t high_twice(uint32_t x) {
  uint32_t r;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %1;\n mov.b32 %0, {h, h};\n}\n" : "=r"(r) : "r"(x));
  return r;
}

// Factor that brings a head's largest |q| into [2^14, 2^15), a power of two;
// NaN when the head holds a non-finite element (its row becomes NaN).
__device__ __forceinline__ float q_factor(float amax, bool finite) {
  if (!finite) return __uint_as_float(0x7fc00000u);
  if (amax == 0.f) return 1.f;
  const int e = static_cast<int>(__float_as_uint(amax) >> 23) - 127;   // subnormal: -127, near enough
  const int f = min(max(14 - e, -126), 126);
  return __uint_as_float(static_cast<uint32_t>(f + 127) << 23);
}

__device__ __forceinline__ void store_lse(const PaArgs& a, int row, int head, float m, float sum) {
  a.lse[static_cast<int64_t>(row) * (a.group * a.c.n_kv_heads) + head] =
      sum == 0.f ? -INFINITY : (m + log2f(sum)) * 0.6931471805599453f;
}

// Four columns of a finished row: outputs `acc` and the weights' sum, both
// relative to 2^m.
template <class Args>
__device__ __forceinline__ void store_row4(const Args& a, int row, int head, int D, int d, const float4& acc, float m,
                                           float sum) {
  const float f = out_factor(a, sum);
  const __nv_bfloat162 x = __floats2bfloat162_rn(acc.x * f, acc.y * f), y = __floats2bfloat162_rn(acc.z * f, acc.w * f);
  *reinterpret_cast<uint2*>(a.out + static_cast<int64_t>(row) * a.os + static_cast<int64_t>(head) * D + d) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&x), *reinterpret_cast<const uint32_t*>(&y));
  if (a.lse && d == 0) store_lse(a, row, head, m, sum);
}

}  // namespace moe
