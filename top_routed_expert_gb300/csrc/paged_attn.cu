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
// The row maximum and sum are kept per warp and joined at the end.  Page
// scales: a key's scale multiplies its score; a value's scale goes into the
// exponent of its weight, with a running maximum of its own, so that the
// weights rounded to f16 stay at most 1 whatever the scales are.
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
constexpr float kLog2e = 1.4426950408889634f;

template <int D> struct Shape {
  static constexpr int kTile = 16 * D;                  // bytes of 16 tokens' keys (or values)
  static constexpr int kStages = D == 256 ? 3 : 4;      // what lets two or three CTAs share an SM
  static constexpr int kRing = kStages * 2 * kTile;     // per warp
  static constexpr int kPart = kRows * D + 3 * kRows;   // floats of a partial: sums, m, m', l
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
// 16 bytes, or zeros when !valid (the source is not read then).
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool valid) {
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
  __shared__ float s_m[kWarps][kRows], s_m2[kWarps][kRows], s_l[kWarps][kRows];
  __shared__ float s_scale[kWarps][kStages][4];
  int64_t* s_start = reinterpret_cast<int64_t*>(smem + kWarps * S::kRing);
  pdl_enter();
  // the last CTA has the least to do here, often nothing
  if (a.tc_rows < INT_MAX && blockIdx.x == gridDim.x - 1) list_tc_items(a, reinterpret_cast<int*>(s_start), smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  build_unit_table<kRows, kUnit>(a, s_start, blockIdx.x == 0 ? a.status : nullptr);
  const int64_t total = s_start[a.B];
  const int64_t piece = piece_of(total, gridDim.x);
  const int64_t first = piece * blockIdx.x, last = min(total, first + piece);
  const uint32_t ring = ptx::smem_u32(smem) + warp * S::kRing;
  const int ps = a.c.page_size;

  for (int64_t at = first; at < last;) {
    // the row tile at `at`, and the piece of it that is this CTA's
    const int b = find_entry(s_start, a.B, at);
    const Request rq = load_request(a.cu, a.kv_len, b, a.T);
    const Span sp = span_of(a, rq, kUnit);
    const int64_t in_b = at - s_start[b];
    const int tile = static_cast<int>(in_b / sp.units);      // (key head, row tile)
    const int u0 = static_cast<int>(in_b % sp.units);
    const int u1 = static_cast<int>(min(static_cast<int64_t>(sp.units), u0 + (last - at)));
    const int rts = ceil_div(rq.n * a.group, kRows);
    const int kvh = tile / rts, row0 = tile % rts * kRows;
    const int rows = min(kRows, rq.n * a.group - row0);
    const bool whole = u0 == 0 && u1 == sp.units;
    const int slot = at == first ? 0 : 1;
    at += u1 - u0;

    const uint8_t* kbase = static_cast<const uint8_t*>(a.c.k) + kvh * a.c.head_stride;
    const uint8_t* vbase = static_cast<const uint8_t*>(a.c.v) + kvh * a.c.head_stride;
    const int32_t* table = a.c.page_table + static_cast<int64_t>(b) * a.c.max_pages;
    auto tile_base = [&](int u) { return sp.block_of(u) * kUnit + warp * 16; };
    auto page_id = [&](int u) -> int {
      const int j = tile_base(u);
      if (u >= u1 || !sp.any_seen(j, j + 15)) return -2;      // nothing to fetch
      const int p = j / ps;
      return p < a.c.max_pages ? table[p] : -1;
    };
    auto issue = [&](int u, int pid, int stage) {
      const uint32_t kd = ring + stage * 2 * S::kTile, vd = kd + S::kTile;
      float* sc = s_scale[warp][stage];
      if (pid == -2) return;
      const int j0 = tile_base(u);
      const bool ok = pid >= 0 && pid < a.c.n_pages;
      if (!ok && lane == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      if (lane == 0) sc[2] = ok ? 1.f : 0.f;
      const int64_t page = ok ? pid : 0;
      if (lane < 2) {
        const float* src = (lane ? a.c.v_scale : a.c.k_scale) + page * a.c.n_kv_heads + kvh;
        cp4(ptx::smem_u32(sc + lane), src);
      }
      const int64_t off = page * a.c.page_stride + (j0 % ps) * a.c.token_stride;
      constexpr int CPR = D / 16;   // chunks of a token
#pragma unroll
      for (int i = 0; i < 16 * CPR / 32; ++i) {
        const int c = i * 32 + lane, row = c / CPR, chunk = c % CPR;
        const bool valid = ok && sp.seen(j0 + row);
        const int64_t o = off + row * a.c.token_stride + chunk * 16;
        cp16(kd + chunk_at<D>(row, chunk), valid ? kbase + o : kbase, valid);
        cp16(vd + chunk_at<D>(row, chunk), valid ? vbase + o : vbase, valid);
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
      float amax = 0.f;
      bool fin = true;
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          raw[c][i] = live ? *reinterpret_cast<const uint4*>(src + c * 64 + t * 16 + i * 8) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {raw[c][i].x, raw[c][i].y, raw[c][i].z, raw[c][i].w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float lo = fabsf(__uint_as_float(w[e] << 16)), hi = fabsf(__uint_as_float(w[e] & 0xffff0000u));
            fin = fin && lo < INFINITY && hi < INFINITY;
            amax = fmaxf(amax, fmaxf(lo, hi));
          }
        }
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
      amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
      fin = ((__ballot_sync(0xffffffffu, fin) >> (lane & ~3)) & 0xfu) == 0xfu;
      const float f = q_factor(amax, fin);
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

    float o[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, m2[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

    for (int u = u0; u < u1; ++u) {
      const int stage = (u - u0) % kStages;
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
        const float ks = sc[0], lvs = log2f(sc[1]);
        const bool full = sp.all_see(j0, j0 + 15, pos_min, pos_max);
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int h = e >> 1;
            s[j][e] *= ks * rf[h];
            if (!full && !sp.sees(pos[h], j0 + token_of(j, 2 * t + (e & 1)))) s[j][e] = -INFINITY;
            top[h] = fmaxf(top[h], s[j][e]);
          }
        bool grew = false;
        float drop[2] = {1.f, 1.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
          if (top[h] > m[h]) {
            l[h] *= ex2(m[h] - top[h]);
            m[h] = top[h];
          }
          const float top2 = top[h] + lvs;
          if (top2 > m2[h]) {
            drop[h] = ex2(m2[h] - top2);
            m2[h] = top2;
            grew = true;
          }
        }
        if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
          for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][e] *= drop[e >> 1];
        }
        uint32_t p[4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float ms = m[h] == -INFINITY ? 0.f : m[h];
          const float shift = m2[h] == -INFINITY ? -INFINITY : lvs - m2[h];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float s0 = s[j][2 * h], s1 = s[j][2 * h + 1];
            l[h] += ex2(s0 - ms) + ex2(s1 - ms);
            p[2 * j + h] = pack_f16(ex2(s0 + shift), ex2(s1 + shift));
          }
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
      issue(u + kStages - 1, pid, (stage + kStages - 1) % kStages);
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
        s_m2[warp][g + 8 * h] = m2[h];
        s_l[warp][g + 8 * h] = l[h];
      }
    }
    // the lane's columns: D = 128c + 16 (2t + (e & 1)) + i for tile 16c + i (D = 64: 8 (2t + (e & 1)) + i)
    float* mine = reinterpret_cast<float*>(smem) + warp * (S::kRing / 4);
    constexpr int RUN = D >= 128 ? 16 : 8;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < NT; i += 4)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int col = i / 16 * 128 + RUN * (2 * t + e) + i % 16;
          *reinterpret_cast<float4*>(mine + (g + 8 * h) * D + (D == 64 ? RUN * (2 * t + e) + i : col)) =
              make_float4(o[i][2 * h + e], o[i + 1][2 * h + e], o[i + 2][2 * h + e], o[i + 3][2 * h + e]);
        }
    __syncthreads();
    for (int i = threadIdx.x; i < rows * (D / 4); i += kWarps * 32) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float mm = -INFINITY, mm2 = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        mm = fmaxf(mm, s_m[w][r]);
        mm2 = fmaxf(mm2, s_m2[w][r]);
      }
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        sum += s_l[w][r] * ex2_from(s_m[w][r], mm);
        const float f = ex2_from(s_m2[w][r], mm2);
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + w * (S::kRing / 4) + r * D + d);
        acc.x += x.x * f;
        acc.y += x.y * f;
        acc.z += x.z * f;
        acc.w += x.w * f;
      }
      if (whole) {
        const int tok = (row0 + r) / a.group, head = kvh * a.group + (row0 + r) % a.group;
        store_row4(a, rq.row0 + tok, head, D, d, acc, mm, mm2, sum);
      } else {
        float* part = a.part + (static_cast<int64_t>(blockIdx.x) * 2 + slot) * S::kPart;
        *reinterpret_cast<float4*>(part + r * D + d) = acc;
        if (d == 0) {
          part[kRows * D + r] = mm;
          part[kRows * D + kRows + r] = mm2;
          part[kRows * D + 2 * kRows + r] = sum;
        }
      }
    }
    __syncthreads();   // the ring is free again
  }
}

// Joins the partial sums of the row tiles that more than one CTA worked on.
// One block per key head, place of a row tile and row (all rows beside the
// tcgen05 kernel, where few requests or none are left for it); the places of a ragged
// batch are found as moe_kv_append finds its pages: request b's row tiles
// start at cu[b] group / 16 + b; where a request has at most rt_max of them
// (rt_max > 0) they start at b rt_max.
template <int D>
__global__ void __launch_bounds__(128) paged_attn_join(PaArgs a, int n_ctas, int rt_max) {
  using S = Shape<D>;
  __shared__ int64_t s_red[2][4];
  __shared__ float s_acc[4][D], s_st[4][3];
  pdl_enter();
  const int kvh = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = rt_max ? blockIdx.x / rt_max : warp_find_request(a.cu, a.B, blockIdx.x, a.group, kRows, 1);
  const Request rq = load_request(a.cu, a.kv_len, b, a.T);
  const int rt = rt_max ? blockIdx.x % rt_max
                        : blockIdx.x - static_cast<int>(static_cast<int64_t>(rq.row0) * a.group / kRows + b);
  const int rts = ceil_div(rq.n * a.group, kRows);
  if (!rq.ok || rq.n * a.group > a.tc_rows || rt < 0 || rt >= rts) return;
  const int rows = min(kRows, rq.n * a.group - rt * kRows);
  // units before request b, and in all
  int64_t before = 0, total = 0;
  for (int i = threadIdx.x; i < a.B; i += blockDim.x) {
    const Request x = load_request(a.cu, a.kv_len, i, a.T);
    const int64_t n = units_of(a, x, kRows, kUnit);
    total += n;
    before += i < b ? n : 0;
  }
  for (int off = 16; off > 0; off >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, off);
    total += __shfl_xor_sync(0xffffffffu, total, off);
  }
  if (lane == 0) {
    s_red[0][warp] = before;
    s_red[1][warp] = total;
  }
  __syncthreads();
  before = s_red[0][0] + s_red[0][1] + s_red[0][2] + s_red[0][3];
  total = s_red[1][0] + s_red[1][1] + s_red[1][2] + s_red[1][3];
  const int64_t piece = piece_of(total, n_ctas);
  const int units = span_of(a, rq, kUnit).units;
  const int64_t start = before + (static_cast<int64_t>(kvh) * rts + rt) * units, end = start + units;
  const int c0 = static_cast<int>(start / piece), c1 = static_cast<int>((end - 1) / piece);
  if (c0 == c1) return;   // one CTA did all of it
  auto part_of = [&](int c) {
    const int slot = (c == c0 && start != c0 * piece) ? 1 : 0;
    return a.part + (static_cast<int64_t>(c) * 2 + slot) * S::kPart;
  };
  for (int r = blockIdx.z; r < rows; r += gridDim.z) {
    float m = -INFINITY, m2 = -INFINITY;
    for (int c = c0; c <= c1; ++c) {
      const float* p = part_of(c) + kRows * D + r;
      m = fmaxf(m, p[0]);
      m2 = fmaxf(m2, p[kRows]);
    }
    float sum = 0.f;
    constexpr int PER = D / 32;   // columns of a lane
    float acc[PER] = {};
    for (int c = c0 + warp; c <= c1; c += 4) {
      const float* p = part_of(c);
      sum += p[kRows * D + 2 * kRows + r] * ex2_from(p[kRows * D + r], m);
      const float f = ex2_from(p[kRows * D + kRows + r], m2);
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] += p[r * D + lane + 32 * i] * f;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) s_acc[warp][lane + 32 * i] = acc[i];
    if (lane == 0) s_st[warp][0] = sum;
    __syncthreads();
    sum = s_st[0][0] + s_st[1][0] + s_st[2][0] + s_st[3][0];
    const int row = rt * kRows + r, tok = row / a.group, head = kvh * a.group + row % a.group;
    const int d = threadIdx.x * 4;
    if (d < D) {
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        x.x += s_acc[w][d];
        x.y += s_acc[w][d + 1];
        x.z += s_acc[w][d + 2];
        x.w += s_acc[w][d + 3];
      }
      store_row4(a, rq.row0 + tok, head, D, d, x, m, m2, sum);
    }
    __syncthreads();
  }
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
  const int rt_max = a.tc_rows < INT_MAX ? ceil_div(a.tc_rows, kRows) : 0;
  const int64_t places = rt_max ? static_cast<int64_t>(rt_max) * a.B : static_cast<int64_t>(a.T) * a.group / kRows + a.B;
  if (places > 0x7fffffff) return cudaErrorInvalidConfiguration;
  return launch_pdl(paged_attn_join<D>, dim3(static_cast<unsigned>(places), a.c.n_kv_heads, rt_max ? 1 : kRows),
                    128, 0, s, a, ctas, rt_max);
}

}  // namespace

size_t paged_attn_ws_bytes(int D) {
  const size_t part = (static_cast<size_t>(kRows) * D + 3 * kRows) * sizeof(float);
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
  return align_up(paged_attn_ws_bytes(cache->head_dim), 256) + align_up((tc_places(a) + 1) * sizeof(int2), 256);
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
  a.part = static_cast<float*>(ws);
  a.tc_list = reinterpret_cast<int2*>(static_cast<char*>(ws) + align_up(paged_attn_ws_bytes(cache->head_dim), 256));
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
  return launch_paged_attn(a, cfg->max_q_len, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
