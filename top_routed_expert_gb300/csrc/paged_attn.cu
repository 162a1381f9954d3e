// Attention over the paged 8-bit cache (include/paged_kv.h,
// moe_paged_attention) for few query rows per request and key head: the
// single-token form, small drafts, and every shape that paged_attn_tc.cu does
// not take.
//
// The rows of one (request, key head) are its new tokens times the query
// heads of the group, row r = token r / group, head r % group; 8 or 16 rows make
// a row tile.  The work of a row tile is cut into units of 64 cached tokens.
// All units of the call stand in one line (request, key head, row tile,
// token), and the persistent CTAs take equal pieces of that line, so a batch
// of mixed lengths keeps every SM busy to the end.  A piece may end inside a
// row tile; then all its CTAs leave partial sums and paged_attn_join adds them
// in order (a fixed order: the same bits every time).
//
// A CTA has four warps; in a unit each has 16 tokens of its own, fetched by
// cp.async into a ring that only this warp uses (no block barrier in the
// loop).  Both products run on the tensor cores as m16n8k16 with f16 operands
// and the rows as N, so that the eight heads of a group fill it:
//   S^T = K Q^T (M = 16 tokens),  O^T = V^T P^T (M = 16 elements of the head)
// The codes are the A operands, converted exactly to f16 in registers, straight
// from the stored rows:
//  - the order of the head's elements inside the first product's K is free if q
//    uses the same: a lane takes 16 consecutive codes of a key and calls them
//    its elements of four K steps;
//  - so is the order of the elements in the second product's M: a lane takes 16
//    consecutive codes of four tokens, and one byte permutation pairs two
//    tokens' codes for the conversion;
//  - the weights become the second product's B operand by a transposition of
//    8x8 blocks between the lanes.
// Sums and references are kept per warp and joined at the end.  Page scales: a
// key's scale multiplies its score; a value's scale goes into the exponent of
// its weight, and the weights' sum takes it out again.  A row's weights are
// relative to 2^-8 of the maximum of the first tile that it sees something in
// (kRefBelow); that reference moves only when weights outgrow f16 (65504), so the
// ordinary tile takes no maximum and rescales nothing.
//
// What each row computes, with p its position and w the window:
//   z_j = sm_scale q . (k_scale_j k_j),  j <= p and (j > p - w or j < n_sink)
//   out = sum 2^(z_j log2 e - m) v_scale_j v_j / sum 2^(z_j log2 e - m)
// The weights are rounded to f16 for the second product (2^-11, under the
// output's bf16 rounding, 2^-9; weights under 2^-22 of the largest by up to 2^-33 of
// it); scores, sums, references and outputs are fp32.
//
// Measured (key heads x query heads of a group x D): 12 requests at 49157 to 65536
// tokens, 4 x 8 x 128, 705 MB in 114 us = 6.2 TB/s, bound by memory; 64 at 17
// to 3712, 123 MB in 32.4 us = 3.8 TB/s, of which the join and the two launches
// are 7; one at 3585 13 us, two launches and eight dependent loads; 48 drafts of
// up to 4 tokens in a window of 1024, 8 x 4 x 64, 49 MB in 29 us, bound by the
// issue of instructions (conversion and weights) and the row tiles' starts; 64 at
// 3584, 4 x 8 x 256, 470 MB in 93 us = 5.0 TB/s.
// Registers spilled (bytes stored, D / blocks of rows): 64/1 60, 64/2 48, 128/2 92,
// 256/1 76, outside the loop over the units; 128/1 none.
#include <climits>

#include "paged_kv.cuh"
#include "tc_ptx.cuh"
#include "paged_attn.cuh"

namespace moe {

bool paged_attn_tc_supported(int D);
cudaError_t launch_paged_attn_tc(const PaArgs& a, cudaStream_t s);

namespace {

constexpr int kWarps = 4;
constexpr int kUnit = 64;        // tokens of a unit
// What a row tile costs beside its units (finding it, q, the join of the
// warps), in units.
constexpr int kTileCost = 4;
constexpr float kLog2e = 1.4426950408889634f;

// D: elements of a head, NB: blocks of eight rows in a row tile.
template <int D, int NB> struct Shape {
  static constexpr int kRows = 8 * NB;
  static constexpr int kTile = 16 * D;                  // bytes of 16 tokens' keys (or values)
  // CTAs on an SM, by registers (O takes D NB / 4 of a thread's, q D NB / 8),
  // and the stages of the ring that fit then
  static constexpr int kCtas = D * NB == 64 ? 5 : D * NB == 128 ? 4 : D * NB == 256 ? 3 : 2;
  static constexpr int kStages = D == 256 ? 2 : D * NB == 128 && D == 128 ? 3 : 4;
  static constexpr int kRing = kStages * 2 * kTile;     // per warp
  static constexpr int kPart = kRows * D + 2 * kRows;   // floats of a partial: outputs, references, sums
};

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros when !valid (the source is not read then).
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Two E4M3 codes (the low 16 bits) -> two f16, exact.
__device__ __forceinline__ uint32_t f16x2_of(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 t, u;\n mov.b32 {t, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_of_hi(uint32_t two) {
  uint32_t r;
  asm("{\n .reg .b16 t, u;\n mov.b32 {t, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, u;\n}\n" : "=r"(r) : "r"(two));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8x8 block of f16, a row in four lanes (two columns each), transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Where a 16-byte chunk of token `row` lies in a tile: no bank conflicts for
// the copies (whole rows), the key reads (two neighbouring rows, 64 bytes of
// each) and the value reads (four rows two apart, one or two chunks of each).
template <int D> __device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
  if (D == 64) {
    const int slot = (row & ~1) | ((row ^ (row >> 1)) & 1);
    return slot * 64 + ((chunk ^ (((row >> 2) & 1) << 1)) << 4);
  }
  return row * D + ((chunk ^ (((row >> 1) & 3) << 1) ^ ((row & 1) << 2)) << 4);
}

// Lists the row blocks of the requests that go to paged_attn_tc.cu, the longest
// first (a counting sort by 256 classes of length; the order inside a class
// does not matter to the results).  Where that is allowed, a block longer than
// 1.5 times a CTA's share of the work is cut along the cached tokens into parts
// of at least 3/4 of that share.  One thread block; `first`: B + 1 ints, `scratch`: the
// block's other shared memory.
__device__ __noinline__ void list_tc_items(const PaArgs& a, int* first, char* scratch) {
  int* bins = reinterpret_cast<int*>(scratch);            // [256]
  int* s_max = bins + 256;
  unsigned long long* s_sum = reinterpret_cast<unsigned long long*>(bins + 258);
  TcList* s_list = reinterpret_cast<TcList*>(bins + 260);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int s_warp[32];
  for (int i = threadIdx.x; i < 256; i += blockDim.x) bins[i] = 0;
  if (threadIdx.x == 0) {
    *s_max = 0;
    *s_sum = 0;
    *s_list = TcList{};
  }
  __syncthreads();
  auto blocks_of = [&](const Request& r) { return r.n * a.group > a.tc_rows ? ceil_div(r.n * a.group, kTcItemRows) : 0; };
  auto length = [&](const Request& r, int blk) {
    const int row0 = blk * kTcItemRows, row1 = min(row0 + kTcItemRows, r.n * a.group) - 1;
    return span_for(a, r.start + row0 / a.group, r.start + row1 / a.group, kTcStep).units;
  };
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < a.B) {
      const Request r = load_request(a.cu, a.kv_len, b, a.T);
      if (!r.ok || r.end > a.c.max_pages * a.c.page_size) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      n = blocks_of(r);
      if (n > 0) atomicMax(s_max, length(r, n - 1));
    }
    int sum = n;
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += x;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int all = 0, below = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x / 32); ++w) {
      all += s_warp[w];
      below += w < warp ? s_warp[w] : 0;
    }
    if (b < a.B) first[b] = static_cast<int>(min(base + below + sum - n, static_cast<int64_t>(INT_MAX)));
    base += all;
    __syncthreads();
  }
  // offsets out of order can name rows twice; the list has room for them once
  const int total = static_cast<int>(min(base, tc_places(a)));
  const int64_t widest = *s_max + 1;
  auto look = [&](int i, int& b, int& blk) {   // the i-th block; its length
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= i) lo = mid; else hi = mid - 1;
    }
    b = lo;
    blk = i - first[lo];
    return length(load_request(a.cu, a.kv_len, b, a.T), blk);
  };
  int b, blk;
  int64_t share = INT_MAX;   // steps of a part
  if (a.tc_split) {
    unsigned long long sum = 0;
    for (int i = threadIdx.x; i < total; i += blockDim.x) sum += look(i, b, blk);
    atomicAdd(s_sum, sum);
    __syncthreads();
    share = max(int64_t(4), static_cast<int64_t>(*s_sum * a.c.n_kv_heads + a.tc_ctas - 1) / a.tc_ctas);
  }
  // rounded down: with equal blocks, the parts then are no more than the CTAs
  auto parts_of = [&](int units) {
    return 2 * int64_t(units) <= 3 * share ? 1 : max(2, static_cast<int>(units / share));
  };
  auto class_of = [&](int units, int parts) {
    return 255 - static_cast<int>(min(static_cast<int64_t>(255), static_cast<int64_t>(units / parts) * 256 / widest));
  };
  for (int i = threadIdx.x; i < total; i += blockDim.x) {
    const int units = look(i, b, blk), parts = parts_of(units);
    atomicAdd(&bins[class_of(units, parts)], parts);
  }
  __syncthreads();
  if (warp == 0) {   // exclusive prefix over the classes
    int sum = 0, mine[8];
    for (int i = 0; i < 8; ++i) {
      mine[i] = sum;
      sum += bins[lane * 8 + i];
    }
    int before = sum;
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, before, off);
      if (lane >= off) before += x;
    }
    before -= sum;
    for (int i = 0; i < 8; ++i) bins[lane * 8 + i] = before + mine[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += blockDim.x) {
    const int units = look(i, b, blk), parts = parts_of(units);
    const int at = atomicAdd(&bins[class_of(units, parts)], parts);
    atomicAdd(&s_list->entries, parts);
    int slot = -1;
    if (parts > 1) {
      slot = atomicAdd(&s_list->slots, parts);
      a.tc_joins[atomicAdd(&s_list->joins, 1)] = TcJoin{b, blk, parts, slot};
    }
    for (int k = 0; k < parts; ++k) a.tc_entries[at + k] = TcEntry{b, blk, k, parts, slot};
  }
  __syncthreads();
  if (threadIdx.x == 0) *a.tc = *s_list;
  __syncthreads();
}

// The list alone, for a batch that has no small requests.
__global__ void __launch_bounds__(512) list_kernel(PaArgs a) {
  extern __shared__ __align__(128) char smem[];
  pdl_enter();
  list_tc_items(a, reinterpret_cast<int*>(smem + 2048), smem);
}

template <int D, int NB>
__global__ void __launch_bounds__(kWarps * 32, Shape<D, NB>::kCtas) paged_attn_kernel(PaArgs a) {
  using S = Shape<D, NB>;
  constexpr int KC = D / 64;      // 64-element chunks of a head
  constexpr int MT = D / 16;      // 16-element tiles of the output
  constexpr int kStages = S::kStages, kRows = S::kRows;
  extern __shared__ __align__(128) char smem[];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ float s_scale[kWarps][kStages][4];
  int64_t* s_start = reinterpret_cast<int64_t*>(smem + kWarps * S::kRing);
  pdl_enter();
  // the last CTA has the least to do here, often nothing
  if (a.tc_rows < INT_MAX && blockIdx.x == gridDim.x - 1) list_tc_items(a, reinterpret_cast<int*>(s_start), smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  build_unit_table<kRows, kUnit, kTileCost>(a, s_start, blockIdx.x == 0 ? a.status : nullptr);
  const int64_t total = s_start[a.B];
  const int64_t piece = piece_of(total, gridDim.x);
  const int64_t first = piece * blockIdx.x, last = min(total, first + piece);
  const uint32_t ring = ptx::smem_u32(smem) + warp * S::kRing;
  const int ps = a.c.page_size, ps_log = 31 - __clz(ps);
  const int64_t ts = a.c.token_stride;
  // this lane's 16-byte chunks of a tile: token (+ RSTEP each) and chunk
  constexpr int CPR = D / 16, RSTEP = 32 / CPR, COPIES = 16 / RSTEP;
  const int crow = lane / CPR, cchunk = lane % CPR;
  const int64_t lane_off = crow * ts + cchunk * 16;
  JoinTile cut = {};   // the row tile that this CTA begins and others go on with

  int b = -1;
  Request rq = {};
  for (int64_t at = first; at < last;) {
    // the row tile at `at`, and the piece of it that is this CTA's
    const int b_now = find_entry(s_start, a.B, at);
    if (b_now != b) {
      b = b_now;
      rq = load_request(a.cu, a.kv_len, b, a.T);
    }
    const Span sp = span_of(a, rq, kUnit);
    const int64_t in_b = at - s_start[b];
    const int width = sp.units + kTileCost;
    int tile;   // (key head, row tile)
    if (in_b <= 0x7fffffff) tile = static_cast<int>(in_b) / width;
    else tile = static_cast<int>(in_b / width);
    const int v0 = static_cast<int>(in_b - static_cast<int64_t>(tile) * width);
    const int v1 = static_cast<int>(min(static_cast<int64_t>(width), v0 + (last - at)));
    const int u0 = max(v0 - kTileCost, 0), u1 = v1 - kTileCost;
    const int64_t tile_end = at + (width - v0);
    const int slot = at == first ? 0 : 1;
    at += v1 - v0;
    if (u1 <= u0) continue;   // the next CTA begins it
    const int rts = ceil_div(rq.n * a.group, kRows);
    const int kvh = tile / rts, row0 = (tile - kvh * rts) * kRows;
    const int rows = min(kRows, rq.n * a.group - row0);
    const bool whole = u0 == 0 && u1 == sp.units;
    if (u0 == 0 && !whole) cut = JoinTile{rows, rq.row0, row0, kvh, slot, static_cast<int>((tile_end - 1) / piece)};

    // q of this lane's row g of each block, on its way while the rest starts
    uint4 raw[NB][KC][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const int r = row0 + 8 * n + g;
      const bool live = 8 * n + g < rows;
      const uint16_t* src = a.q + static_cast<int64_t>(rq.row0 + (live ? r / a.group : 0)) * a.qs +
                            static_cast<int64_t>(kvh * a.group + (live ? r % a.group : 0)) * D + t * 16;
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          raw[n][c][i] = live ? __ldg(reinterpret_cast<const uint4*>(src + c * 64 + i * 8)) : make_uint4(0, 0, 0, 0);
    }

    const uint8_t* kbase = static_cast<const uint8_t*>(a.c.k) + kvh * a.c.head_stride;
    const int64_t v_minus_k = static_cast<const uint8_t*>(a.c.v) - static_cast<const uint8_t*>(a.c.k);
    const int32_t* table = a.c.page_table + static_cast<int64_t>(b) * a.c.max_pages;
    auto tile_base = [&](int u) { return sp.block_of(u) * kUnit + warp * 16; };
    // Page ids are asked for a tile ahead of the copies and looked at there.  A
    // table may hold kNothing's value too: then the tile tells which it is.
    constexpr int kNothing = INT_MIN;
    auto needed = [&](int u) {
      const int j = tile_base(u);
      return u < u1 && sp.any_seen(j, j + 15);
    };
    auto page_id = [&](int u) -> int { return needed(u) ? __ldg(table + (tile_base(u) >> ps_log)) : kNothing; };
    auto issue = [&](int u, int pid, int stage) {
      float* sc = s_scale[warp][stage];
      if (pid == kNothing) {
        if (lane == 0 && needed(u)) {
          sc[2] = 0.f;
          set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
        }
        return;
      }
      const int j0 = tile_base(u);
      const bool ok = static_cast<unsigned>(pid) < static_cast<unsigned>(a.c.n_pages);
      if (lane == 0) sc[2] = ok ? 1.f : 0.f;
      if (!ok) {
        if (lane == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
        return;
      }
      if (lane < 2)
        cp4(ptx::smem_u32(sc + lane), (lane ? a.c.v_scale : a.c.k_scale) + static_cast<int64_t>(pid) * a.c.n_kv_heads + kvh);
      const uint8_t* src = kbase + (pid * a.c.page_stride + (j0 & (ps - 1)) * ts + lane_off);
      const uint32_t kd = ring + stage * 2 * S::kTile, vd = kd + S::kTile;
      if (sp.all_seen(j0, j0 + 15)) {
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          const uint32_t d = chunk_at<D>(i * RSTEP + crow, cchunk);
          cp16(kd + d, src);
          cp16(vd + d, src + v_minus_k);
          src += RSTEP * ts;
        }
      } else {
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          const uint32_t d = chunk_at<D>(i * RSTEP + crow, cchunk);
          const bool seen = sp.seen(j0 + i * RSTEP + crow);
          cp16_or_zero(kd + d, seen ? src : kbase, seen);
          cp16_or_zero(vd + d, seen ? src + v_minus_k : kbase, seen);
          src += RSTEP * ts;
        }
      }
    };

    int pid = page_id(u0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      const int next = page_id(u0 + i + 1);
      issue(u0 + i, pid, i);
      cp_commit();
      pid = next;
    }

    // q as f16, each head scaled by a power of two; the lane's score columns are
    // rows 2t and 2t+1 of each block
    uint32_t qf[NB][KC][4][2];
    float rf[NB][2], m[NB][2], l[NB][2];
    int pos[NB][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      uint32_t top = 0;   // the largest size as bits: a NaN's are above infinity's
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint4 w = raw[n][c][i];
          top = __vmaxu2(top, __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu));
          top = __vmaxu2(top, __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
        }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float f = q_factor(__uint_as_float(top << 16), top < 0x7f80u);
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w[4] = {raw[n][c][i].x, raw[n][c][i].y, raw[n][c][i].z, raw[n][c][i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            qf[n][c][2 * i + (e >> 1)][e & 1] =
                pack_f16(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
        }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * n + 2 * t + h;
        rf[n][h] = a.sm_scale * kLog2e / __shfl_sync(0xffffffffu, f, (2 * t + h) * 4);
        pos[n][h] = r < rows ? rq.start + (row0 + r) / a.group : -1;
        // a row that sees nothing at all needs no reference
        m[n][h] = pos[n][h] >= 0 ? -INFINITY : 0.f;
        l[n][h] = 0.f;
      }
    }
    const int pos_min = rq.start + row0 / a.group, pos_max = rq.start + (row0 + rows - 1) / a.group;

    float o[NB][MT][4];
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int i = 0; i < MT; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][i][e] = 0.f;

#pragma unroll 1
    for (int u = u0, stage = 0; u < u1; ++u, stage = stage + 1 == kStages ? 0 : stage + 1) {
      cp_wait<kStages - 2>();
      __syncwarp();
      const int j0 = tile_base(u);
      const float* sc = s_scale[warp][stage];
      if (sp.any_seen(j0, j0 + 15) && sc[2] != 0.f) {
        const uint32_t kd = ring + stage * 2 * S::kTile, vd = kd + S::kTile;
        // scores: tokens g and g+8 (e >> 1) by rows 2t and 2t+1 (e & 1)
        float s[NB][4] = {};
#pragma unroll
        for (int c = 0; c < KC; ++c) {
          const uint4 klo = lds128(kd + chunk_at<D>(g, 4 * c + t)), khi = lds128(kd + chunk_at<D>(g + 8, 4 * c + t));
          const uint32_t lo[4] = {klo.x, klo.y, klo.z, klo.w}, hi[4] = {khi.x, khi.y, khi.z, khi.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t ka[4] = {f16x2_of(lo[e]), f16x2_of(hi[e]), f16x2_of_hi(lo[e]), f16x2_of_hi(hi[e])};
#pragma unroll
            for (int n = 0; n < NB; ++n) mma16816(s[n], ka, qf[n][c][e][0], qf[n][c][e][1]);
          }
        }
        const float ks = sc[0], lvs = __log2f(sc[1]), ivs = __frcp_rn(sc[1]);
        if (!sp.all_see(j0, j0 + 15, pos_min, pos_max)) {
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!sp.sees(pos[n][e & 1], j0 + g + 8 * (e >> 1))) s[n][e] = -INFINITY;
        }
        // weights relative to the reference so far
        float w[NB][4];
        bool move = false;
        auto weigh = [&](int n, int h) {
          const float f = score_factor(ks, rf[n][h]), shift = lvs - (m[n][h] == -INFINITY ? 0.f : m[n][h]);
          w[n][h] = ex2(fmaf(s[n][h], f, shift));
          w[n][2 + h] = ex2(fmaf(s[n][2 + h], f, shift));
          return m[n][h] == -INFINITY || w[n][h] + w[n][2 + h] > kMostSum;
        };
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) move |= weigh(n, h);
        if (__any_sync(0xffffffffu, move)) {
          // rows whose weights are too large for f16, or that have no reference
          // yet, take their maximum
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const unsigned of_row = __ballot_sync(0xffffffffu, weigh(n, h)) & (0x11111111u << t);
              float top = fmaf(fmaxf(s[n][h], s[n][2 + h]), score_factor(ks, rf[n][h]), lvs);
#pragma unroll
              for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
              if (of_row) {
                const float to = fmaxf(m[n][h], top - kRefBelow), f = m[n][h] == -INFINITY ? 0.f : ex2(m[n][h] - to);
                m[n][h] = to;
                l[n][h] *= f;
#pragma unroll
                for (int i = 0; i < MT; ++i) {
                  o[n][i][h] *= f;
                  o[n][i][2 + h] *= f;
                }
                weigh(n, h);
              }
            }
        }
        uint32_t p[NB][2];
#pragma unroll
        for (int n = 0; n < NB; ++n) {
#pragma unroll
          for (int h = 0; h < 2; ++h) l[n][h] = fmaf(w[n][h] + w[n][2 + h], ivs, l[n][h]);
          p[n][0] = transpose8x8(pack_f16(w[n][0], w[n][1]));
          p[n][1] = transpose8x8(pack_f16(w[n][2], w[n][3]));
        }
        // values: words of tokens 2t, 2t+1 | 2t+8, 2t+9
        constexpr int VW = D >= 128 ? 4 : 2;     // words of a lane's run of codes
#pragma unroll
        for (int c = 0; c < (D + 127) / 128; ++c) {
          uint32_t vw[4][VW];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int row = 2 * t + (i & 1) + 8 * (i >> 1);
            if (D == 64) {
              const uint2 x = lds64(vd + chunk_at<D>(row, g >> 1) + (g & 1) * 8);
              vw[i][0] = x.x;
              vw[i][1] = x.y;
            } else {
              const uint4 x = lds128(vd + chunk_at<D>(row, 8 * c + g));
              vw[i][0] = x.x;
              vw[i][1] = x.y;
              vw[i][VW - 2] = x.z;
              vw[i][VW - 1] = x.w;
            }
          }
#pragma unroll
          for (int i = 0; i < VW; ++i) {
            const uint32_t a01 = __byte_perm(vw[0][i], vw[1][i], 0x5140), a23 = __byte_perm(vw[0][i], vw[1][i], 0x7362);
            const uint32_t b01 = __byte_perm(vw[2][i], vw[3][i], 0x5140), b23 = __byte_perm(vw[2][i], vw[3][i], 0x7362);
            const uint32_t lo[4] = {f16x2_of(a01), f16x2_of_hi(a01), f16x2_of(b01), f16x2_of_hi(b01)};
            const uint32_t hi[4] = {f16x2_of(a23), f16x2_of_hi(a23), f16x2_of(b23), f16x2_of_hi(b23)};
#pragma unroll
            for (int n = 0; n < NB; ++n) {
              mma16816(o[n][c * 8 + 2 * i], lo, p[n][0], p[n][1]);
              mma16816(o[n][c * 8 + 2 * i + 1], hi, p[n][0], p[n][1]);
            }
          }
        }
      }
      __syncwarp();
      const int next = page_id(u + kStages);
      issue(u + kStages - 1, pid, stage == 0 ? kStages - 1 : stage - 1);
      cp_commit();
      pid = next;
    }
    cp_wait<0>();
    __syncthreads();   // every warp is done with its ring

    // join the four warps' sums
    float* mine = reinterpret_cast<float*>(smem) + warp * (S::kRing / 4);
#pragma unroll
    for (int n = 0; n < NB; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int r = 8 * n + 2 * t + h;
#pragma unroll
        for (int off = 4; off < 32; off <<= 1) l[n][h] += __shfl_xor_sync(0xffffffffu, l[n][h], off);
        if (g == 0) {
          s_m[warp][r] = m[n][h];
          s_l[warp][r] = l[n][h];
        }
        // the lane's columns: tiles 2i and 2i+1 of a 128-element chunk have
        // elements 4i, 4i+1 and 4i+2, 4i+3 of its run of codes
        constexpr int RUN = D >= 128 ? 16 : 8;
#pragma unroll
        for (int i = 0; i < MT / 2; ++i) {
          const int col = D == 64 ? RUN * g + 4 * i : i / 4 * 128 + RUN * g + i % 4 * 4;
          *reinterpret_cast<float4*>(mine + r * D + (col ^ ((r & 7) << 2))) =
              make_float4(o[n][2 * i][h], o[n][2 * i][2 + h], o[n][2 * i + 1][h], o[n][2 * i + 1][2 + h]);
        }
      }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (D / 4); i += kWarps * 32) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float mm = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w][r]);
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2_from(s_m[w][r], mm);
        sum += s_l[w][r] * f;
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + w * (S::kRing / 4) + r * D +
                                                          (d ^ ((r & 7) << 2)));
        acc.x += x.x * f;
        acc.y += x.y * f;
        acc.z += x.z * f;
        acc.w += x.w * f;
      }
      if (whole) {
        const int tok = (row0 + r) / a.group, head = kvh * a.group + (row0 + r) % a.group;
        store_row4(a, rq.row0 + tok, head, D, d, acc, mm, sum);
      } else {
        float* part = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * S::kPart;
        *reinterpret_cast<float4*>(part + r * D + d) = acc;
        if (d == 0) {
          part[kRows * D + r] = mm;
          part[kRows * D + kRows + r] = sum;
        }
      }
    }
    __syncthreads();   // the ring is free again
  }
  if (threadIdx.x == 0) a.joins[blockIdx.x] = cut;
}

// Joins the partial sums of the row tiles that more than one CTA worked on.  The
// rows to join are dealt to all blocks (one on an SM) and their warps; where that
// leaves warps over, several share a row's parts.  The kernel is a chain of
// latencies, so what a row needs is under way at once: eight parts' columns, and
// their references and sums, one part a lane.
constexpr int kJoinWarps = 32;
// The workspace is sized for kMaxSms SMs, so that its size needs no device.
constexpr int kMaxCtas = kMaxSms * 5;

template <int D, int NB>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_attn_join(PaArgs a, int n_ctas) {
  using S = Shape<D, NB>;
  constexpr int kRows = S::kRows;
  constexpr int VEC = D / 64;   // pairs of columns of a lane
  __shared__ int s_first[kJoinWarps * 32];   // rows to join before CTA i's
  __shared__ JoinTile s_tile[kMaxCtas];
  __shared__ int s_warp[kJoinWarps];
  __shared__ float2 s_acc[kJoinWarps][VEC][32];
  __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int rows = 0;
  if (threadIdx.x < n_ctas) {
    const JoinTile tile = a.joins[threadIdx.x];
    rows = tile.rows;
    s_tile[threadIdx.x] = tile;
  }
  int before = rows;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, before, off);
    if (lane >= off) before += v;
  }
  if (lane == 31) s_warp[warp] = before;
  __syncthreads();
  int in_warps = s_warp[lane];
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, in_warps, off);
    if (lane >= off) in_warps += v;
  }
  const int total = __shfl_sync(0xffffffffu, in_warps, 31);
  const int prior = __shfl_sync(0xffffffffu, in_warps, max(warp - 1, 0));
  s_first[threadIdx.x] = before - rows + (warp > 0 ? prior : 0);
  __syncthreads();
  const int items = (total - static_cast<int>(blockIdx.x) + gridDim.x - 1) / gridDim.x;   // this block's rows
  if (items <= 0) return;
  int shares = 1;
  while (shares * 2 * items <= kJoinWarps) shares *= 2;
  const int share = warp % shares;
#pragma unroll 1
  for (int base = 0; base < items; base += kJoinWarps / shares) {
    const int item = base + warp / shares;
    const bool live = item < items;
    // the CTA that began the row's tile: the last that has no more rows before it
    const int at = blockIdx.x + (live ? item : 0) * gridDim.x;
    int c0 = 0;
#pragma unroll
    for (int step = kJoinWarps * 16; step > 0; step >>= 1)
      if (c0 + step < n_ctas && s_first[c0 + step] <= at) c0 += step;
    const int r = at - s_first[c0];
    const JoinTile tile = s_tile[c0];
    auto part_of = [&](int c) { return a.part + (static_cast<int64_t>(c) * 2 + (c == c0 ? tile.slot : 0)) * S::kPart; };
    float m = -INFINITY, sum = 0.f;
    float2 acc[VEC] = {};
    // this share's parts
    constexpr int BATCH = D == 256 ? 4 : 8;
#pragma unroll 1
    for (int c = c0 + share; live && c <= tile.last; c += BATCH * shares) {
      float2 v[BATCH][VEC];
      float pm = -INFINITY, pl = 0.f;
      if (lane < BATCH && c + lane * shares <= tile.last) {
        const float* p = part_of(c + lane * shares) + kRows * D + r;
        pm = p[0];
        pl = p[kRows];
      }
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const float2* p = reinterpret_cast<const float2*>(part_of(c + i * shares) + r * D) + lane;
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[i][e] = c + i * shares <= tile.last ? p[e * 32] : make_float2(0.f, 0.f);
      }
      float to = fmaxf(m, pm);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, off));
      const float old = ex2_from(m, to), w = ex2_from(pm, to);
      m = to;
      pl *= w;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) pl += __shfl_xor_sync(0xffffffffu, pl, off);
      sum = sum * old + pl;
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = make_float2(acc[e].x * old, acc[e].y * old);
#pragma unroll
      for (int i = 0; i < BATCH; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          acc[e].x += v[i][e].x * wi;
          acc[e].y += v[i][e].y * wi;
        }
      }
    }
    if (shares > 1) {
      if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = sum;
      }
#pragma unroll
      for (int e = 0; e < VEC; ++e) s_acc[warp][e][lane] = acc[e];
      __syncthreads();
      if (share == 0) {
        const float pm = lane < shares ? s_m[warp + lane] : -INFINITY;
        float to = pm;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, off));
        const float w = ex2_from(pm, to);
        m = to;
        sum = lane < shares ? s_l[warp + lane] * w : 0.f;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
#pragma unroll
        for (int e = 0; e < VEC; ++e) acc[e] = make_float2(0.f, 0.f);
#pragma unroll 4
        for (int i = 0; i < shares; ++i) {
          const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float2 v = s_acc[warp + i][e][lane];
            acc[e].x += v.x * wi;
            acc[e].y += v.y * wi;
          }
        }
      }
      __syncthreads();
    }
    if (live && share == 0) {
      const int tok = (tile.row0 + r) / a.group, head = tile.kvh * a.group + (tile.row0 + r) % a.group;
      const float f = sum == 0.f ? 0.f : 1.0f / sum;   // nothing visible (a NaN sum is not)
      __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(a.out + static_cast<int64_t>(tile.token0 + tok) * a.os +
                                                              static_cast<int64_t>(head) * D);
#pragma unroll
      for (int e = 0; e < VEC; ++e) out[e * 32 + lane] = __floats2bfloat162_rn(acc[e].x * f, acc[e].y * f);
      if (a.lse && lane == 0) store_lse(a, tile.token0 + tok, head, m, sum);
    }
  }
}

// Persistent CTAs: what the SMs hold at once.
template <int D, int NB> int ctas_for(int num_sms) { return std::min(num_sms, kMaxSms) * Shape<D, NB>::kCtas; }

template <int D, int NB>
cudaError_t launch(const PaArgs& a, int num_sms, cudaStream_t s) {
  using S = Shape<D, NB>;
  const size_t smem = kWarps * S::kRing + sizeof(int64_t) * (a.B + 1);
  cudaError_t err = ensure_kernel_attrs(reinterpret_cast<const void*>(paged_attn_kernel<D, NB>), static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  const int ctas = ctas_for<D, NB>(num_sms);
  count_launches(2);
  err = launch_pdl(paged_attn_kernel<D, NB>, ctas, kWarps * 32, smem, s, a);
  if (err != cudaSuccess) return err;
  static_assert(kMaxSms * Shape<D, NB>::kCtas <= kMaxCtas && kMaxCtas <= kJoinWarps * 32, "a thread of the join for each CTA");
  return launch_pdl(paged_attn_join<D, NB>, ctas / Shape<D, NB>::kCtas, kJoinWarps * 32, 0, s, a, ctas);
}

// Row tiles of eight where no request has more rows: half the registers, more
// warps (eight rows, tiles of eight / sixteen: 64 requests at 17 to 3712 tokens
// 33 / 41 us, 12 at about 57000 115 / 150 us).  With more rows, tiles of sixteen
// convert the codes half as often (64 requests of 32 rows at 3584 117 / 92 us).
template <int D>
cudaError_t launch(const PaArgs& a, int64_t most_rows, int num_sms, cudaStream_t s) {
  if (D == 256 || most_rows <= 8) return launch<D, 1>(a, num_sms, s);
  return launch<D == 256 ? 128 : D, 2>(a, num_sms, s);
}

template <int D, int NB> size_t part_bytes() {
  return static_cast<size_t>(ctas_for<D, NB>(kMaxSms)) * 2 * Shape<D, NB>::kPart * sizeof(float);
}

}  // namespace

size_t paged_attn_part_bytes(int D) {
  switch (D) {
    case 64: return std::max(part_bytes<64, 1>(), part_bytes<64, 2>());
    case 128: return std::max(part_bytes<128, 1>(), part_bytes<128, 2>());
    default: return part_bytes<256, 1>();
  }
}

// Which kernels a call takes, from what the host knows.
struct Path {
  bool tc;      // the tcgen05 kernel, for requests with more than kTcRows rows
  bool alone;   // ... and it alone
  bool split;   // ... which may cut row blocks along the cached tokens
};

// The few-row kernel reads a request's tokens once for every 16 rows (8 where D =
// 256), the tcgen05 kernel once for 256, but takes longer to start and to join: with heads of 128
// about 13 us + 3.1 us for a million pairs of a row and a token (a row tile's
// start counting as kTileCost units of tokens) against 29 us + 0.6 us.
// Measured (us, few-row / tcgen05): one request of 1024 rows (of all key heads)
// at 3584 tokens 25 / 33, at 8192 40 / 37, at 16384 65 / 44, at 65536 221 / 67; of
// 512 rows at 8192 27 / 34, at 65536 118 / 63; of 256 rows at 65536 66 / 63; 2048 rows
// of 1 / 8 requests at 3584 37 / 34 and 31 / 37; 64 requests of 32 rows each (8192)
// at 1792 to 3584 94 / 115, of 64 rows 167 / 113; 125 prompts of up to 26 tokens, 8
// x 7 heads, at 40 to 49 tokens 112 / 69.  These are with page tables as wide as
// the longest request.
//
// The host does not know the lengths: the page table's width stands for them, up
// to kTcTokens, since a wide table may be a short one's.  With a table of 131072
// tokens (us, few-row / tcgen05; *: the rule takes the slower), 4 x 8 heads: 32 new
// tokens at 512 18 / 34*, at 2048 25 / 38*, at 4096 31 / 41*; 64 new tokens at 512
// 23 / 34*, at 4096 45 / 40; 16 at 4096 25 / 38*; 4 x 32 at 1024 33 / 40*; and where
// the table is as long as it is wide: 8 new tokens at 131072 122* / 100, 10 150* / 100,
// 12 172 / 100, 16 224 / 101.  A lower limit would trade the first against these.
//
// Cutting row blocks along the tokens adds a launch for their join and pays where
// one block is longer than a CTA's share of the work.  Measured (us, not cut / cut;
// 4 x 8 x 128; places: row blocks and requests, times key heads):
//   512 new tokens at 4096 (68 places) 81 / 69, 1024 (132) 82 / 87, 2048 (260) 119 /
//   126; 512 at 32768 beside 8 x 256 at 512 (356) 520 / 308; 256 at 65536 beside 16 x
//   256 at 512 (612) 978 / 314, at 16384 266 / 153, at 8192 147 / 122; equal requests
//   8 x 512 at 3584 (544) 242 / 251, 16 x 256 (576) 254 / 263;
//   above the limit: 18 x 256 at 256 to 3584 (648) 159 / 169, 32 x 256 (1152) 266 / 280,
//   but 256 at 16384 beside 24 x 256 (900) 271 / 179, at 65536 beside 40 (1476) 1000 /
//   426.
// A call that gains nothing loses up to 10 us, one long request among short ones
// gains several times that; more places make the second rarer, so that cutting is
// allowed up to 4 kMaxSms of them.  The device then cuts what is longer than 1.5
// shares (2 instead of 1.5: the same times to 1 us, with 8 x 512 at 3584, 4 x 1024 at
// 32768, 2 x 2048 at 4096 to 65536, 3 x 512 at 2048 to 16384).
constexpr int kTcRows = 48;                  // of a request and key head
constexpr int kTcTokens = 16384;
constexpr int64_t kTcWork = int64_t(6) << 20;   // pairs

Path path_of(const PaArgs& a, int max_q_len) {
  const int64_t most = static_cast<int64_t>(max_q_len > 0 ? std::min(max_q_len, a.T) : a.T) * a.group;
  Path p;
  const int64_t rows = static_cast<int64_t>(a.T) * a.group * a.c.n_kv_heads;
  const int64_t tokens = std::min<int64_t>(static_cast<int64_t>(a.c.max_pages) * a.c.page_size, kTcTokens);
  p.tc = most > kTcRows && rows * (tokens + kTileCost * kUnit) >= kTcWork && paged_attn_tc_supported(a.c.head_dim);
  // As many rows as if every request had max_q_len of them: they all do (or the
  // hint is wrong, and the tcgen05 kernel takes small ones too).
  p.alone = p.tc && static_cast<int64_t>(max_q_len) * a.B == a.T;
  p.split = p.tc && tc_places(a) * a.c.n_kv_heads <= 4 * kMaxSms;
  return p;
}

cudaError_t launch_paged_attn(PaArgs a, int max_q_len, int num_sms, cudaStream_t s) {
  const Path path = path_of(a, max_q_len);
  const int64_t most = static_cast<int64_t>(max_q_len > 0 ? std::min(max_q_len, a.T) : a.T) * a.group;
  a.tc_rows = path.alone ? 0 : path.tc ? kTcRows : INT_MAX;
  a.tc_ctas = std::min(num_sms, kMaxSms);
  a.tc_split = path.split;
  cudaError_t err;
  if (path.alone) {
    count_launches(1);
    err = launch_pdl(list_kernel, 1, 512, 2048 + sizeof(int) * (a.B + 1), s, a);
  } else {
    switch (a.c.head_dim) {
      case 64: err = launch<64>(a, std::min<int64_t>(most, a.tc_rows), num_sms, s); break;
      case 128: err = launch<128>(a, std::min<int64_t>(most, a.tc_rows), num_sms, s); break;
      default: err = launch<256>(a, most, num_sms, s); break;
    }
  }
  return err == cudaSuccess && path.tc ? launch_paged_attn_tc(a, s) : err;
}

namespace {

// Workspace: partial sums and the row tiles to join, then what the tcgen05
// kernel needs where a call can take it (cut blocks or not, alone or not, so
// that a smaller call never needs more).
struct Workspace {
  size_t joins, tc, tc_entries, tc_joins, tc_part, total;
};

Workspace plan_workspace(const PaArgs& a, int max_q_len) {
  const int D = a.c.head_dim;
  const Path path = path_of(a, max_q_len);
  Workspace w;
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t from = at; at += align_up(bytes, 256); return from; };
  take(paged_attn_part_bytes(D));
  w.joins = take(kMaxCtas * sizeof(JoinTile));
  w.tc = take(sizeof(TcList));
  w.tc_entries = take(path.tc ? (tc_places(a) + kTcSlots) * sizeof(TcEntry) : 0);
  w.tc_joins = take(path.tc ? kTcSlots * sizeof(TcJoin) : 0);
  w.tc_part = take(path.tc ? static_cast<size_t>(kTcSlots) * kTcItemRows * (D + 2) * sizeof(float) : 0);
  w.total = at;
  return w;
}

bool attention_config_ok(const moe_paged_attention_config_t* c, const moe_kv_cache_t* cache) {
  if (!c || !kv_cache_shape_ok(cache)) return false;
  if (c->T < 0 || c->T > (1 << 28) || c->batch < 1 || c->batch > kMaxBatch || c->max_q_len < 0) return false;
  if (c->n_q_heads < 1 || c->n_q_heads % cache->n_kv_heads != 0 || c->n_q_heads / cache->n_kv_heads > 256) return false;
  // row and item counts are 32-bit
  const int64_t rows = static_cast<int64_t>(c->T) * (c->n_q_heads / cache->n_kv_heads);
  if (rows > (int64_t(1) << 30) || (rows / kTcItemRows + c->batch) * cache->n_kv_heads > (int64_t(1) << 30)) return false;
  if (c->window < 0 || c->window > (1 << 30) || c->n_sink < 0 || c->n_sink > (1 << 30)) return false;
  if (!(c->sm_scale > 0.f) || !std::isfinite(c->sm_scale)) return false;
  const int64_t width = static_cast<int64_t>(c->n_q_heads) * cache->head_dim;
  return c->q_stride >= width && c->out_stride >= width && c->q_stride % 8 == 0 && c->out_stride % 8 == 0;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_paged_attention_ws_bytes(const moe_paged_attention_config_t* cfg, const moe_kv_cache_t* cache) {
  using namespace moe;
  if (!attention_config_ok(cfg, cache)) return 0;
  PaArgs a;
  a.T = cfg->T;
  a.B = cfg->batch;
  a.c = *cache;
  a.group = cfg->n_q_heads / cache->n_kv_heads;
  return plan_workspace(a, cfg->max_q_len).total;
}

extern "C" moe_status_t moe_paged_attention(const moe_paged_attention_config_t* cfg, const moe_kv_cache_t* cache,
                                            const void* q, const int32_t* cu, const int32_t* kv_len, void* out,
                                            float* lse, void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  if (!attention_config_ok(cfg, cache)) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!q || !cu || !kv_len || !out || !kv_cache_pointers_ok(cache)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(cu, 4) || !aligned_to(kv_len, 4) ||
      (lse && !aligned_to(lse, 4)))
    return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < moe_paged_attention_ws_bytes(cfg, cache)) return MOE_ERR_WORKSPACE;
  if (!aligned_to(ws, 256)) return MOE_ERR_INVALID_ARG;
  unsigned* status = nullptr;
  int sms = 0;
  const moe_status_t st = current_device(&status, &sms);
  if (st != MOE_OK) return st;
  PaArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.cu = cu;
  a.kv_len = kv_len;
  a.c = *cache;
  a.status = status;
  a.qs = cfg->q_stride;
  a.os = cfg->out_stride;
  a.T = cfg->T;
  a.B = cfg->batch;
  a.group = cfg->n_q_heads / cache->n_kv_heads;
  a.window = cfg->window;
  a.n_sink = cfg->n_sink;
  a.sm_scale = cfg->sm_scale;
  const Workspace w = plan_workspace(a, cfg->max_q_len);
  char* base = static_cast<char*>(ws);
  a.part = reinterpret_cast<float*>(base);
  a.joins = reinterpret_cast<JoinTile*>(base + w.joins);
  a.tc = reinterpret_cast<TcList*>(base + w.tc);
  a.tc_entries = reinterpret_cast<TcEntry*>(base + w.tc_entries);
  a.tc_joins = reinterpret_cast<TcJoin*>(base + w.tc_joins);
  a.tc_part = reinterpret_cast<float*>(base + w.tc_part);
  return launch_paged_attn(a, cfg->max_q_len, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
