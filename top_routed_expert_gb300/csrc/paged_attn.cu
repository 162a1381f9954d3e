// Attention over the paged 8-bit cache (include/paged_kv.h,
// moe_paged_attention) for few query rows per request and key head: the
// single-token form, small drafts, and every shape that paged_attn_tc.cu does
// not take.
//
// The rows of one (request, key head) are its new tokens times the query
// heads of the group, row r = token r / group, head r % group; 16 rows make a
// row tile.  The work of a row tile is cut into units of 64 cached tokens.
// All units of the call stand in one line (request, key head, row tile,
// token), and the persistent CTAs take equal pieces of that line, so a batch
// of mixed lengths keeps every SM busy to the end.  A piece may end inside a
// row tile; then both CTAs leave partial sums and paged_attn_join adds them in
// order (a fixed order: the same bits every time).
//
// A CTA has four warps; in a unit each has 16 tokens of its own, fetched by
// cp.async into a ring that only this warp uses (no block barrier in the
// loop).  Both products run on the tensor cores as m16n8k16 with f16 operands:
// the 16 rows are M, so the codes, converted exactly to f16 in registers, are
// the B operand of both, loaded straight from the stored rows:
//  - the order of the head's elements inside a product's K is free if q uses
//    the same: a lane takes 16 consecutive codes of a key and calls them its
//    elements of four K steps;
//  - so is the order of the tokens in the second product: a lane takes 16
//    consecutive codes of four tokens, and one byte permutation pairs two
//    tokens' codes for the conversion;
//  - the first product's result registers are the second's A operand.
// Sums and references are kept per warp and joined at the end.  Page scales: a
// key's scale multiplies its score; a value's scale goes into the exponent of
// its weight, and the weights' sum takes it out again.  A row's weights are
// relative to the maximum of the first tile that it sees something in; that
// reference moves only when weights grow over 2^15 (f16 holds 65504), so the
// ordinary tile takes no maximum and rescales nothing.
#include <climits>

#include "paged_kv.cuh"
#include "tc_ptx.cuh"
#include "paged_attn.cuh"

namespace moe {

bool paged_attn_tc_supported(int D);
cudaError_t launch_paged_attn_tc(const PaArgs& a, int num_sms, cudaStream_t s);

namespace {

constexpr int kWarps = 4;
constexpr int kRows = 16;
constexpr int kUnit = 64;        // tokens of a unit
constexpr int kJoinThreads = 512, kJoinRows = 4;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMostSum = 32768.0f;   // sum of a lane's four weights that moves the reference: f16 holds 65504

template <int D> struct Shape {
  static constexpr int kTile = 16 * D;                  // bytes of 16 tokens' keys (or values)
  static constexpr int kStages = D == 256 ? 3 : 4;      // what lets two or three CTAs share an SM
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

// Token of a 16-token tile that column n of score tile j stands for: lanes t
// then read tokens t, t+4, t+8, t+12 as values.
__device__ __forceinline__ int token_of(int j, int n) { return (n >> 1) + 4 * (n & 1) + 8 * j; }

// Where a 16-byte chunk of token `row` lies in a tile: no bank conflicts for
// the copies (whole rows), the key reads (rows r and r+4, chunks of 64 bytes)
// and the value reads (rows r..r+3, one or two chunks).
template <int D> __device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
  if (D == 64) {
    const int slot = (row & ~1) | ((row ^ (row >> 2)) & 1);
    return slot * 64 + ((chunk ^ (((row >> 1) & 1) << 1)) << 4);
  }
  return row * D + ((chunk ^ ((row & 3) << 1) ^ (((row >> 2) & 1) << 2)) << 4);
}

// Lists the row blocks of the requests that go to paged_attn_tc.cu, the longest
// first (a counting sort by 256 classes of length; the order inside a class
// does not matter to the results).  One block; `first`: B + 1 ints, `scratch`:
// the block's other shared memory.
__device__ __noinline__ void list_tc_items(const PaArgs& a, int* first, char* scratch) {
  int* bins = reinterpret_cast<int*>(scratch);            // [256]
  int* s_max = bins + 256;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int s_warp[kWarps];
  for (int i = threadIdx.x; i < 256; i += kWarps * 32) bins[i] = 0;
  if (threadIdx.x == 0) *s_max = 0;
  __syncthreads();
  auto blocks_of = [&](const Request& r) { return r.n * a.group > a.tc_rows ? ceil_div(r.n * a.group, kTcItemRows) : 0; };
  auto length = [&](const Request& r, int blk) {
    const int row0 = blk * kTcItemRows, row1 = min(row0 + kTcItemRows, r.n * a.group) - 1;
    return span_for(a, r.start + row0 / a.group, r.start + row1 / a.group, kTcStep).units;
  };
  int base = 0;
  for (int b0 = 0; b0 < a.B; b0 += kWarps * 32) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < a.B) {
      const Request r = load_request(a.cu, a.kv_len, b, a.T);
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
    for (int w = 0; w < kWarps; ++w) {
      all += s_warp[w];
      below += w < warp ? s_warp[w] : 0;
    }
    if (b < a.B) first[b] = base + below + sum - n;
    base += all;
    __syncthreads();
  }
  const int total = base;
  const int64_t widest = *s_max + 1;
  auto look = [&](int i, int2& e) {   // the i-th block and its class
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= i) lo = mid; else hi = mid - 1;
    }
    e = make_int2(lo, i - first[lo]);
    const int units = length(load_request(a.cu, a.kv_len, lo, a.T), e.y);
    return 255 - static_cast<int>(min(static_cast<int64_t>(255), units * 256 / widest));
  };
  int2 e;
  for (int i = threadIdx.x; i < total; i += kWarps * 32) atomicAdd(&bins[look(i, e)], 1);
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
  for (int i = threadIdx.x; i < total; i += kWarps * 32) {
    const int at = atomicAdd(&bins[look(i, e)], 1);
    a.tc_list[1 + at] = e;
  }
  if (threadIdx.x == 0) a.tc_list[0] = make_int2(total, 0);
  __syncthreads();
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, D == 256 ? 2 : 3) paged_attn_kernel(PaArgs a) {
  using S = Shape<D>;
  constexpr int KC = D / 64;      // 64-element chunks of a head
  constexpr int NT = D / 8;       // column tiles of the output
  constexpr int kStages = S::kStages;
  extern __shared__ __align__(128) char smem[];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ float s_scale[kWarps][kStages][4];
  int64_t* s_start = reinterpret_cast<int64_t*>(smem + kWarps * S::kRing);
  pdl_enter();
  // the last CTA has the least to do here, often nothing
  if (a.tc_rows < INT_MAX && blockIdx.x == gridDim.x - 1) list_tc_items(a, reinterpret_cast<int*>(s_start), smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  build_unit_table<kRows, kUnit>(a, s_start, blockIdx.x == 0 ? a.status : nullptr);
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= a.B; i += kWarps * 32) a.starts[i] = s_start[i];
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

  for (int64_t at = first; at < last;) {
    // the row tile at `at`, and the piece of it that is this CTA's
    const int b = find_entry(s_start, a.B, at);
    const Request rq = load_request(a.cu, a.kv_len, b, a.T);
    const Span sp = span_of(a, rq, kUnit);
    const int64_t in_b = at - s_start[b];
    const int tile = static_cast<int>(in_b / sp.units);      // (key head, row tile)
    const int u0 = static_cast<int>(in_b - static_cast<int64_t>(tile) * sp.units);
    const int u1 = static_cast<int>(min(static_cast<int64_t>(sp.units), u0 + (last - at)));
    const int rts = ceil_div(rq.n * a.group, kRows);
    const int kvh = tile / rts, row0 = (tile - kvh * rts) * kRows;
    const int rows = min(kRows, rq.n * a.group - row0);
    const bool whole = u0 == 0 && u1 == sp.units;
    const int slot = at == first ? 0 : 1;
    at += u1 - u0;

    const uint8_t* kbase = static_cast<const uint8_t*>(a.c.k) + kvh * a.c.head_stride;
    const int64_t v_minus_k = static_cast<const uint8_t*>(a.c.v) - static_cast<const uint8_t*>(a.c.k);
    const int32_t* table = a.c.page_table + static_cast<int64_t>(b) * a.c.max_pages;
    auto tile_base = [&](int u) { return sp.block_of(u) * kUnit + warp * 16; };
    // Page ids are asked for a tile ahead of the copies and looked at there.
    constexpr int kNothing = INT_MIN;
    auto page_id = [&](int u) -> int {
      const int j = tile_base(u);
      return u < u1 && sp.any_seen(j, j + 15) ? __ldg(table + (j >> ps_log)) : kNothing;
    };
    auto issue = [&](int u, int pid, int stage) {
      if (pid == kNothing) return;
      const int j0 = tile_base(u);
      float* sc = s_scale[warp][stage];
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

    // this lane's rows g and g+8: position, q as f16 scaled by a power of two
    uint32_t qf[KC][4][4];
    float rf[2];
    int pos[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = row0 + g + 8 * h;
      const bool live = g + 8 * h < rows;
      const int tok = live ? r / a.group : 0, head = kvh * a.group + (live ? r % a.group : 0);
      pos[h] = live ? rq.start + tok : -1;
      const uint16_t* src = a.q + static_cast<int64_t>(rq.row0 + tok) * a.qs + static_cast<int64_t>(head) * D;
      uint4 raw[KC][2];
      uint32_t top = 0;   // the largest size as bits: a NaN's are above infinity's
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          raw[c][i] = live ? __ldg(reinterpret_cast<const uint4*>(src + c * 64 + t * 16 + i * 8)) : make_uint4(0, 0, 0, 0);
          top = __vmaxu2(top, __vmaxu2(raw[c][i].x & 0x7fff7fffu, raw[c][i].y & 0x7fff7fffu));
          top = __vmaxu2(top, __vmaxu2(raw[c][i].z & 0x7fff7fffu, raw[c][i].w & 0x7fff7fffu));
        }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float f = q_factor(__uint_as_float(top << 16), top < 0x7f80u);
      rf[h] = a.sm_scale * kLog2e / f;
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t w[4] = {raw[c][i].x, raw[c][i].y, raw[c][i].z, raw[c][i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            qf[c][2 * i + (e >> 1)][h + 2 * (e & 1)] =
                pack_f16(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
        }
    }
    const int pos_min = rq.start + row0 / a.group, pos_max = rq.start + (row0 + rows - 1) / a.group;
    const bool low_only = rows <= 8;   // rows 8..15 are not there

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    // a row that sees nothing at all needs no reference
    float m[2] = {pos[0] >= 0 ? -INFINITY : 0.f, pos[1] >= 0 ? -INFINITY : 0.f}, l[2] = {0.f, 0.f};

#pragma unroll 1
    for (int u = u0, stage = 0; u < u1; ++u, stage = stage + 1 == kStages ? 0 : stage + 1) {
      cp_wait<kStages - 2>();
      __syncwarp();
      const int j0 = tile_base(u);
      const float* sc = s_scale[warp][stage];
      if (sp.any_seen(j0, j0 + 15) && sc[2] != 0.f) {
        const uint32_t kd = ring + stage * 2 * S::kTile, vd = kd + S::kTile;
        float s[2][4] = {};
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int row = token_of(j, g);
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const uint4 kw = lds128(kd + chunk_at<D>(row, 4 * c + t));
            const uint32_t w[4] = {kw.x, kw.y, kw.z, kw.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) mma16816(s[j], qf[c][e], f16x2_of(w[e]), f16x2_of_hi(w[e]));
          }
        }
        const float ks = sc[0], lvs = __log2f(sc[1]), ivs = __frcp_rn(sc[1]);
        if (!sp.all_see(j0, j0 + 15, pos_min, pos_max)) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!sp.sees(pos[e >> 1], j0 + token_of(j, 2 * t + (e & 1)))) s[j][e] = -INFINITY;
        }
        // weights relative to the reference so far; a sum too large for f16, or
        // a row without a reference, takes the row's maximum first
        float e[2][4], sum[2];
        auto weigh = [&](int h) {
          const float f = score_factor(ks, rf[h]), shift = lvs - (m[h] == -INFINITY ? 0.f : m[h]);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            e[j][2 * h] = ex2(fmaf(s[j][2 * h], f, shift));
            e[j][2 * h + 1] = ex2(fmaf(s[j][2 * h + 1], f, shift));
          }
          sum[h] = (e[0][2 * h] + e[0][2 * h + 1]) + (e[1][2 * h] + e[1][2 * h + 1]);
        };
        weigh(0);
        if (low_only) {
          sum[1] = e[0][2] = e[0][3] = e[1][2] = e[1][3] = 0.f;
        } else {
          weigh(1);
        }
        if (__any_sync(0xffffffffu, m[0] == -INFINITY || m[1] == -INFINITY || sum[0] > kMostSum || sum[1] > kMostSum)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float top = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
            top = fmaf(top, score_factor(ks, rf[h]), lvs);
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            const float to = fmaxf(m[h], top), f = m[h] == -INFINITY ? 0.f : ex2(m[h] - to);
            m[h] = to;
            l[h] *= f;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
              o[i][2 * h] *= f;
              o[i][2 * h + 1] *= f;
            }
            weigh(h);
          }
        }
        uint32_t p[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          l[h] = fmaf(sum[h], ivs, l[h]);
          p[h] = pack_f16(e[0][2 * h], e[0][2 * h + 1]);
          p[2 + h] = pack_f16(e[1][2 * h], e[1][2 * h + 1]);
        }
        // values: words of tokens t, t+4 | t+8, t+12
        constexpr int VW = D >= 128 ? 4 : 2;     // words of a lane's run of codes
#pragma unroll
        for (int c = 0; c < (D + 127) / 128; ++c) {
          uint32_t vw[4][VW];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (D == 64) {
              const uint2 x = lds64(vd + chunk_at<D>(t + 4 * i, g >> 1) + (g & 1) * 8);
              vw[i][0] = x.x;
              vw[i][1] = x.y;
            } else {
              const uint4 x = lds128(vd + chunk_at<D>(t + 4 * i, 8 * c + g));
              vw[i][0] = x.x;
              vw[i][1] = x.y;
              vw[i][VW - 2] = x.z;
              vw[i][VW - 1] = x.w;
            }
          }
#pragma unroll
          for (int w = 0; w < VW; ++w) {
            const uint32_t a01 = __byte_perm(vw[0][w], vw[1][w], 0x5140), a23 = __byte_perm(vw[0][w], vw[1][w], 0x7362);
            const uint32_t b01 = __byte_perm(vw[2][w], vw[3][w], 0x5140), b23 = __byte_perm(vw[2][w], vw[3][w], 0x7362);
            float(*oc)[4] = &o[c * 16 + 4 * w];
            mma16816(oc[0], p, f16x2_of(a01), f16x2_of(b01));
            mma16816(oc[1], p, f16x2_of_hi(a01), f16x2_of_hi(b01));
            mma16816(oc[2], p, f16x2_of(a23), f16x2_of(b23));
            mma16816(oc[3], p, f16x2_of_hi(a23), f16x2_of_hi(b23));
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
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
      if (t == 0) {
        s_m[warp][g + 8 * h] = m[h];
        s_l[warp][g + 8 * h] = l[h];
      }
    }
    // the lane's columns: D = 128c + 16 (2t + (e & 1)) + i for tile 16c + i (D = 64: 8 (2t + (e & 1)) + i)
    float* mine = reinterpret_cast<float*>(smem) + warp * (S::kRing / 4);
    constexpr int RUN = D >= 128 ? 16 : 8;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (h == 0 || !low_only) {
#pragma unroll
        for (int i = 0; i < NT; i += 4)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int col = D == 64 ? RUN * (2 * t + e) + i : i / 16 * 128 + RUN * (2 * t + e) + i % 16;
            *reinterpret_cast<float4*>(mine + (g + 8 * h) * D + col) =
                make_float4(o[i][2 * h + e], o[i + 1][2 * h + e], o[i + 2][2 * h + e], o[i + 3][2 * h + e]);
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
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + w * (S::kRing / 4) + r * D + d);
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
}

// Joins the partial sums of the row tiles that more than one CTA worked on: a
// block for the end of each CTA's piece (but the last) and each group of rows.
// A tile with several ends inside belongs to the first of them.
template <int D>
__global__ void __launch_bounds__(kJoinThreads) paged_attn_join(PaArgs a, int n_ctas) {
  using S = Shape<D>;
  constexpr int LANES = D / 4;                          // threads of a row, four columns each
  constexpr int SHARES = kJoinThreads / (kJoinRows * LANES);   // threads that share a row's parts
  __shared__ float4 s_acc[SHARES][kJoinRows][LANES];
  __shared__ float s_sum[SHARES][kJoinRows];
  __shared__ int s_b;
  pdl_enter();
  const int64_t total = a.starts[a.B], piece = piece_of(total, n_ctas);
  const int64_t end = piece * (blockIdx.x + 1);         // the piece's end: this CTA's last unit is end - 1
  if (end >= total) return;
  // the request that unit end - 1 belongs to
  for (int i = threadIdx.x; i < a.B; i += kJoinThreads)
    if (a.starts[i] <= end - 1 && end - 1 < a.starts[i + 1]) s_b = i;
  __syncthreads();
  const int b = s_b;
  const Request rq = load_request(a.cu, a.kv_len, b, a.T);
  const int units = span_of(a, rq, kUnit).units;
  const int64_t base = a.starts[b];
  const int64_t tile = (end - 1 - base) / units, begin = base + tile * units, stop = begin + units;
  // not split here, or an earlier end inside it has it
  if (stop == end || (begin < end - piece && blockIdx.x > 0)) return;
  const int rts = ceil_div(rq.n * a.group, kRows);
  const int kvh = static_cast<int>(tile / rts), row0 = static_cast<int>(tile - static_cast<int64_t>(kvh) * rts) * kRows;
  const int rows = min(kRows, rq.n * a.group - row0);
  const int c0 = blockIdx.x, c1 = static_cast<int>((stop - 1) / piece);
  const int lane = threadIdx.x % LANES, rl = threadIdx.x / LANES % kJoinRows, share = threadIdx.x / (LANES * kJoinRows);
  const int r = blockIdx.y * kJoinRows + rl;
  if (blockIdx.y * kJoinRows >= rows) return;
  auto part_of = [&](int c) {
    const int slot = (c == c0 && begin != c0 * piece) ? 1 : 0;
    return a.part + (static_cast<int64_t>(c) * 2 + slot) * S::kPart;
  };
  float m = -INFINITY;
  if (r < rows)
    for (int c = c0; c <= c1; ++c) m = fmaxf(m, part_of(c)[kRows * D + r]);
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (r < rows)
#pragma unroll 4
    for (int c = c0 + share; c <= c1; c += SHARES) {
      const float* p = part_of(c);
      const float f = ex2_from(p[kRows * D + r], m);
      const float4 x = *reinterpret_cast<const float4*>(p + r * D + lane * 4);
      sum += p[kRows * D + kRows + r] * f;
      acc.x += x.x * f;
      acc.y += x.y * f;
      acc.z += x.z * f;
      acc.w += x.w * f;
    }
  s_acc[share][rl][lane] = acc;
  if (lane == 0) s_sum[share][rl] = sum;
  __syncthreads();
  if (share > 0 || r >= rows) return;
#pragma unroll
  for (int i = 1; i < SHARES; ++i) {
    const float4 x = s_acc[i][rl][lane];
    acc.x += x.x;
    acc.y += x.y;
    acc.z += x.z;
    acc.w += x.w;
  }
  sum = s_sum[0][rl];
#pragma unroll
  for (int i = 1; i < SHARES; ++i) sum += s_sum[i][rl];
  const int tok = (row0 + r) / a.group, head = kvh * a.group + (row0 + r) % a.group;
  store_row4(a, rq.row0 + tok, head, D, lane * 4, acc, m, sum);
}

// Persistent CTAs: what the SMs hold at once (registers and ring).  The
// workspace is sized for kMaxSms SMs, so that its size needs no device.
constexpr int kMaxSms = 160;
int ctas_for(int D, int num_sms) { return std::min(num_sms, kMaxSms) * (D == 256 ? 2 : 3); }

template <int D>
cudaError_t launch(const PaArgs& a, int num_sms, cudaStream_t s) {
  using S = Shape<D>;
  const size_t smem = kWarps * S::kRing + sizeof(int64_t) * (a.B + 1);
  cudaError_t err = ensure_kernel_attrs(reinterpret_cast<const void*>(paged_attn_kernel<D>), static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  const int ctas = ctas_for(D, num_sms);
  count_launches(2);
  err = launch_pdl(paged_attn_kernel<D>, ctas, kWarps * 32, smem, s, a);
  if (err != cudaSuccess) return err;
  return launch_pdl(paged_attn_join<D>, dim3(std::max(1, ctas - 1), kRows / kJoinRows), kJoinThreads, 0, s, a, ctas);
}

}  // namespace

size_t paged_attn_ws_bytes(int D) {
  const size_t part = (static_cast<size_t>(kRows) * D + 2 * kRows) * sizeof(float);
  return static_cast<size_t>(ctas_for(D, kMaxSms)) * 2 * part;
}

// Requests with more rows than this go to the tcgen05 kernel.
constexpr int kTcRows = 64;

cudaError_t launch_paged_attn(PaArgs a, int max_q_len, int num_sms, cudaStream_t s) {
  const int64_t most = static_cast<int64_t>(max_q_len > 0 ? std::min(max_q_len, a.T) : a.T) * a.group;
  const bool tc = most > kTcRows && paged_attn_tc_supported(a.c.head_dim);
  a.tc_rows = tc ? kTcRows : INT_MAX;
  cudaError_t err;
  switch (a.c.head_dim) {
    case 64: err = launch<64>(a, num_sms, s); break;
    case 128: err = launch<128>(a, num_sms, s); break;
    default: err = launch<256>(a, num_sms, s); break;
  }
  return err == cudaSuccess && tc ? launch_paged_attn_tc(a, num_sms, s) : err;
}

namespace {

// Workspace: partial sums, the requests' first units, the list of row blocks.
struct Workspace {
  size_t starts, tc_list, total;
};

Workspace plan_workspace(const PaArgs& a, int D) {
  Workspace w;
  w.starts = align_up(paged_attn_ws_bytes(D), 256);
  w.tc_list = w.starts + align_up((a.B + 1) * sizeof(int64_t), 256);
  w.total = w.tc_list + align_up((tc_places(a) + 1) * sizeof(int2), 256);
  return w;
}

bool attention_config_ok(const moe_paged_attention_config_t* c, const moe_kv_cache_t* cache) {
  if (!c || !kv_cache_shape_ok(cache)) return false;
  if (c->T < 0 || c->T > (1 << 28) || c->batch < 1 || c->batch > kMaxBatch || c->max_q_len < 0) return false;
  if (c->n_q_heads < 1 || c->n_q_heads % cache->n_kv_heads != 0 || c->n_q_heads / cache->n_kv_heads > 256) return false;
  // row counts are 32-bit
  if (static_cast<int64_t>(c->T) * (c->n_q_heads / cache->n_kv_heads) > (int64_t(1) << 30)) return false;
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
  a.group = cfg->n_q_heads / cache->n_kv_heads;
  return plan_workspace(a, cache->head_dim).total;
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
  const Workspace w = plan_workspace(a, cache->head_dim);
  a.part = static_cast<float*>(ws);
  a.starts = reinterpret_cast<int64_t*>(static_cast<char*>(ws) + w.starts);
  a.tc_list = reinterpret_cast<int2*>(static_cast<char*>(ws) + w.tc_list);
  return launch_paged_attn(a, cfg->max_q_len, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
