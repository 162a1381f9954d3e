// Attention over the paged 4-bit cache (include/block_kv.h,
// moe_blockkv_attention): entry points and the kernel for few query rows per
// request and key head (the single-token form, small drafts, and every shape
// that paged_attn_tc.cuh does not take).  The work is cut as paged_attn_rows.cuh
// says.
//
// A CTA has four warps; in a unit of 128 tokens each has a step of 32 (two tiles of
// 16), fetched by cp.async into a ring that only this warp uses.  Both products run
// on the tensor cores as m16n8k16 with f16 operands and the rows as N:
//   S^T = K Q^T (M = 16 tokens),  O^T = V^T P^T (M = 16 elements of the head)
// The codes are the A operands.  A code times its block's E4M3 scale has six
// significant bits and lies between 2^-10 and 2688, so f16 holds it exactly: two
// codes are converted by one instruction and multiplied by one more.
//  - Keys: a lane takes the 16 codes of one block and calls them its elements of
//    four K steps, so it needs one scale for them.
//  - Values: a lane takes 16 codes of one block from four tokens (D = 64: 8, half
//    a block); the codes of two tokens are interleaved by four bits before the
//    conversion, and one multiplication applies both tokens' scales.
//
// With p a row's position and w the window:
//   z_j = sm_scale kg q . K_j,  j <= p and (j > p - w or j < n_sink)
//   out = vg sum 2^(z_j log2 e - m) V_j / sum 2^(z_j log2 e - m)
// A row's reference m lies 2^-8 under the maximum of the first tile that it sees
// something in and moves only when weights outgrow f16 (kRefBelow); the weights
// are rounded to f16 for the second product, all else is fp32.
//
// Bound by the issue of instructions: 4.5 bits an element leave half the time of
// the 8-bit cache for the same conversions and products, 64 conversions (at half
// the issue rate) and 64 multiplications a tile and warp.  So a step has two tiles
// (one: 105 us where two take 85), the units that all rows of the tile see in full,
// nearly all of a long context, take a path without masks or limits, and registers
// come before CTAs on an SM (D = 128: four with 128 of them 84 us, three with 168
// 78, two 84).
//
// Measured (key heads x query heads of a group x D): 12 requests at 49157 to 65536
// tokens, 4 x 8 x 128, 397 MB in 77 us = 5.1 TB/s, of which 3 are the join and about 7
// what every call has; each further request of 57000 tokens takes 6.1 us, 0.81 of
// the rate of memory.  64 at 17 to 3712, 70 MB in 25.5 us; one at 3585 10.3 us; 48 drafts
// of up to 4 tokens in a window of 1024, 8 x 4 x 64, 22.8 us; 64 at 3584, 4 x 8 x 256, 56 us.
// A row tile that is short and new costs about 2300 instructions of a warp beside
// its steps: 256 requests of 4 x 8 rows at 40 tokens (2048 row tiles) take 45 us, 36 %
// of the issue slots (loading the next row tile's request, q, pages and first codes
// during the join of the last one: 47).  No registers are spilled but 12 bytes at
// D = 64 with 16 rows.
#include "block_kv.cuh"
#include "paged_attn_rows.cuh"

namespace moe {
namespace {

// Where a 16-byte chunk of token `row` lies in a tile: no bank conflicts for the
// copies (whole rows), the key reads (32 bytes of four neighbouring rows at a
// time) and the value reads (32 bytes of rows 0, 2, 4, 6 or 1, 3, 5, 7; D = 64: words
// of them).  Bits 0 + 2 and 1 of the row's number tell the rows of either apart.
template <int D> __device__ __forceinline__ uint32_t chunk_at(int row, int chunk) {
  if (D == 64) return (row ^ (row >> 2 & 1)) * 32 + (chunk << 4);
  if (D == 128) return (row ^ (row >> 2 & 1)) * 64 + ((chunk ^ (row & 2)) << 4);
  return row * 128 + ((chunk ^ (((row ^ row >> 2) & 1) << 2) ^ (row & 2)) << 4);
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// What is added to a row's scores, minus its reference; kNone: it has none yet
// (any score's weight then is infinite, a masked one's still 0).
constexpr float kNone = 1e30f;

template <int D, int NB>
__global__ void __launch_bounds__(kWarps * 32, Shape<D, NB, true>::kCtas) block_attn_kernel(BlockPaArgs a) {
  using S = Shape<D, NB, true>;
  constexpr int KC = D / 64;      // 64-element chunks of a head
  constexpr int MT = D / 16;      // 16-element tiles of the output
  constexpr int kUnit = S::kUnit, kTileCost = S::kTileCost, kStages = S::kStages, kRows = S::kRows;
  constexpr int SB = D / 16, kStep = kUnit / kWarps;   // bytes of a token's scales, tokens of a warp's step
  extern __shared__ __align__(128) char smem[];
  __shared__ float s_m[kWarps][kRows], s_l[kWarps][kRows];
  int64_t* s_start = reinterpret_cast<int64_t*>(smem + kWarps * S::kRing);
  pdl_enter();
  // the last CTA has the least to do here, often nothing
  if (a.tc_rows < INT_MAX && blockIdx.x == gridDim.x - 1) list_tc_items(a, reinterpret_cast<int*>(s_start), smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, t = lane & 3;
  build_unit_table<kRows, kUnit, kTileCost>(a, s_start, blockIdx.x == 0 ? a.status : nullptr);
  const int64_t total = s_start[a.B];
  // As many pieces as CTAs or units, which differ by a unit at most; unit x is in
  // piece ((x + 1) pieces - 1) / total.
  const int64_t pieces = min(total, static_cast<int64_t>(gridDim.x)), me = min(pieces, static_cast<int64_t>(blockIdx.x));
  const int64_t first = pieces ? total * me / pieces : 0, last = me < pieces ? total * (me + 1) / pieces : total;
  const uint32_t ring = ptx::smem_u32(smem) + warp * S::kRing;
  const int ps = a.c.page_size, ps_log = 31 - __clz(ps);
  const int64_t ts = a.c.token_stride;
  // x / group is (x per_group) >> 20 for x < group + 16 <= 272: 272 * 255 < 2^20
  const int per_group = ((1 << 20) + a.group - 1) / a.group;
  // this lane's 16-byte chunks of a tile: token (+ RSTEP each) and chunk
  constexpr int CPR = D / 32, RSTEP = 32 / CPR, COPIES = 16 / RSTEP;
  const int crow = lane / CPR, cchunk = lane % CPR;
  // What the lane reads and writes of a tile, as offsets: rows eight apart are so
  // in memory, the other chunks and the neighbouring row an exclusive or away.
  const uint32_t first_copy = chunk_at<D>(crow, cchunk);
  auto copy_to = [&](int i) { return (D == 256 && (i & 1) ? first_copy ^ 64u : first_copy) + i * RSTEP * (D / 2); };
  const uint32_t to_key = chunk_at<D>(g, t >> 1) + (t & 1) * 8;
  const uint32_t to_value = D == 64 ? chunk_at<D>(2 * t, g >> 2) + (g & 3) * 4 : chunk_at<D>(2 * t, g >> 1) + (g & 1) * 8;
  const uint32_t to_kscale = g * SB + t, to_vscale = 2 * t * SB + (D == 64 ? g >> 1 : g);
  // the first slot in its page of a step's tiles: pages divide the units
  const int slot0 = (warp * kStep) & (ps - 1), slot1 = (warp * kStep + 16) & (ps - 1);
  JoinTile cut = {};   // the row tile that this CTA begins and others go on with

  int b = -1;
  Request rq = {};
  Span sp = {};
  for (int64_t at = first; at < last;) {
    // the row tile at `at`, and the piece of it that is this CTA's
    if (b < 0 || at >= s_start[b + 1]) {
      b = find_entry(s_start, a.B, at);
      rq = load_request(a.cu, a.kv_len, b, a.T);
      sp = span_of(a, rq, kUnit);
    }
    const int64_t in_b = at - s_start[b];
    const int width = sp.units + kTileCost;
    int tile;   // (key head, row tile)
    if (in_b <= 0x7fffffff) tile = static_cast<int>(in_b) / width;
    else tile = static_cast<int>(in_b / width);
    const int v0 = static_cast<int>(in_b - static_cast<int64_t>(tile) * width);
    // a row tile that is not cut is the CTA's in whose piece it begins
    const int v1 = a.whole_tiles ? width : static_cast<int>(min(static_cast<int64_t>(width), v0 + (last - at)));
    const int u0 = max(v0 - kTileCost, 0), u1 = v1 - kTileCost;
    const int64_t tile_end = at + (width - v0);
    const int slot = at == first ? 0 : 1;
    at += v1 - v0;
    if (u1 <= u0 || (a.whole_tiles && v0 > 0)) continue;   // the next CTA begins it, or the one before has it
    const int rts = ceil_div(rq.n * a.group, kRows);
    const int kvh = tile / rts, row0 = (tile - kvh * rts) * kRows;
    const int rows = min(kRows, rq.n * a.group - row0);
    const int tok0 = row0 / a.group, head0 = row0 - tok0 * a.group;
    auto tok_of = [&](int r) { return ((head0 + r) * per_group) >> 20; };   // row r's token, from tok0 on
    const bool whole = u0 == 0 && u1 == sp.units;
    if (u0 == 0 && !whole) cut = JoinTile{rows, rq.row0, row0, kvh, slot, static_cast<int>((tile_end * pieces - 1) / total)};

    // q of this lane's row g of each block, on its way while the rest starts
    uint4 raw[NB][KC][2];
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      const bool live = 8 * n + g < rows;
      const int r = live ? 8 * n + g : 0, tok = tok_of(r);
      const uint16_t* src = a.q + static_cast<int64_t>(rq.row0 + tok0 + tok) * a.qs +
                            static_cast<int64_t>(kvh * a.group + (head0 + r - tok * a.group)) * D + t * 16;
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          raw[n][c][i] = live ? __ldg(reinterpret_cast<const uint4*>(src + c * 64 + i * 8)) : make_uint4(0, 0, 0, 0);
    }

    const int pos_min = rq.start + tok0, pos_max = pos_min + tok_of(rows - 1);
    // units [ua, ub): the tile's rows all see all of them
    const int from = sp.window && pos_max >= sp.window ? (pos_max - sp.window) / kUnit + 1 : 0;
    const int ua = sp.sink_blocks + max(from - sp.lo_block, 0);
    const int ub = max(ua, min(u1, sp.sink_blocks + max(min(pos_min + 1, sp.end), 0) / kUnit - sp.lo_block));

    // the lane's chunks of the step's first tile in page 0, and its token's scales:
    // the keys' in lanes 0 to 15, the values' in 16 to 31
    const uint8_t* codes = static_cast<const uint8_t*>(a.c.k) + kvh * a.c.head_stride + (slot0 + crow) * ts + cchunk * 16;
    const int64_t v_minus_k = static_cast<const uint8_t*>(a.c.v) - static_cast<const uint8_t*>(a.c.k);
    const uint8_t* scales = (lane < 16 ? a.k_scales : a.v_scales) + kvh * a.scale_head + (slot0 + (lane & 15)) * a.scale_token;
    const int32_t* table = a.c.page_table + static_cast<int64_t>(b) * a.c.max_pages;
    const int64_t next_tile = (slot1 - slot0) * ts, next_tile_s = (slot1 - slot0) * a.scale_token;   // within a page
    auto step_base = [&](int u) { return sp.block_of(u) * kUnit + warp * kStep; };
    auto plain = [&](int u) { return static_cast<unsigned>(u - ua) < static_cast<unsigned>(ub - ua); };
    auto needed = [&](int u, int x) {
      const int j = step_base(u) + 16 * x;
      return plain(u) || (u < u1 && sp.any_seen(j, j + 15));
    };
    // Page ids of a step's two tiles are asked for a step ahead of the copies and
    // looked at there.
    auto page_ids = [&](int u, int& pid0, int& pid1) {
      const int32_t* at = table + (step_base(u) >> ps_log);
      pid0 = needed(u, 0) ? __ldg(at) : -1;
      pid1 = needed(u, 1) ? __ldg(at + (ps == 16)) : -1;
    };
    uint32_t there = 0;   // two bits for each step, the last one's the lowest: which tiles hold something to weigh
    auto issue = [&](int u, int pid0, int pid1, int stage) {
      const bool ok0 = static_cast<unsigned>(pid0) < static_cast<unsigned>(a.c.n_pages);
      const bool ok1 = static_cast<unsigned>(pid1) < static_cast<unsigned>(a.c.n_pages);
      there = there << 2 | ok1 << 1 | ok0;
      const uint32_t at_stage = ring + stage * S::kStage;
      if (plain(u) && ok0 && ok1) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t pid = x ? pid1 : pid0;
          const uint8_t* src = codes + static_cast<uint64_t>(pid * a.page16) * 16u + (x ? next_tile : 0);
#pragma unroll
          for (int i = 0; i < COPIES; ++i) {
            const uint32_t d = copy_to(i) + at_stage + x * 2 * S::kTile;
            cp16(d, src);
            cp16(d + S::kTile, src + v_minus_k);
            if (i + 1 < COPIES) src += RSTEP * ts;
          }
          cp_or_zero<SB>(at_stage + 4 * S::kTile + (x * 32 + lane) * SB,
                         scales + static_cast<uint64_t>(pid * a.page_s) * SB + (x ? next_tile_s : 0), true);
        }
        return;
      }
      if (lane == 0 && ((!ok0 && needed(u, 0)) || (!ok1 && needed(u, 1)))) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      if (!ok0 && !ok1) return;
      // zeros where no row sees anything, or a page is missing
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const bool ok = x ? ok1 : ok0;
        const uint32_t pid = ok ? (x ? pid1 : pid0) : 0;
        const int j0 = step_base(u) + 16 * x;
        const uint8_t* src = codes + static_cast<uint64_t>(pid * a.page16) * 16u + (x ? next_tile : 0);
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          const uint32_t d = copy_to(i) + at_stage + x * 2 * S::kTile;
          const bool seen = ok && sp.seen(j0 + i * RSTEP + crow);
          cp16_or_zero(d, seen ? src : codes, seen);
          cp16_or_zero(d + S::kTile, seen ? src + v_minus_k : codes, seen);
          src += RSTEP * ts;
        }
        const bool seen = ok && sp.seen(j0 + (lane & 15));
        cp_or_zero<SB>(at_stage + 4 * S::kTile + (x * 32 + lane) * SB,
                       seen ? scales + static_cast<uint64_t>(pid * a.page_s) * SB + (x ? next_tile_s : 0) : scales, seen);
      }
    };

    int pid0, pid1;
    page_ids(u0, pid0, pid1);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) {
      int next0, next1;
      page_ids(u0 + i + 1, next0, next1);
      issue(u0 + i, pid0, pid1, i);
      cp_commit();
      pid0 = next0;
      pid1 = next1;
    }

    // q as f16, each head scaled by a power of two; the lane's score columns are
    // rows 2t and 2t+1 of each block
    uint32_t qf[NB][KC][4][2];
    float rf[NB][2], shift[NB][2], l[NB][2];
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
        rf[n][h] = score_factor(a.kg, a.sm_scale * kLog2e / __shfl_sync(0xffffffffu, f, (2 * t + h) * 4));
        pos[n][h] = r < rows ? pos_min + tok_of(r) : -1;
        // a row that sees nothing at all needs no reference
        shift[n][h] = pos[n][h] >= 0 ? kNone : 0.f;
        l[n][h] = 0.f;
      }
    }

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
      __syncwarp();   // also: the step before has been read, its stage is free
      const uint32_t have = there >> (2 * (kStages - 2)) & 3u;
      int next0, next1;
      page_ids(u + kStages, next0, next1);
      issue(u + kStages - 1, pid0, pid1, stage == 0 ? kStages - 1 : stage - 1);
      cp_commit();
      pid0 = next0;
      pid1 = next1;
      if (have == 0) continue;
      const uint32_t at_stage = ring + stage * S::kStage;
      // scores: tile x, tokens g and g+8 (e >> 1) by rows 2t and 2t+1 (e & 1)
      float s[2][NB][4] = {};
      const uint32_t key_at = at_stage + to_key, kscale_at = at_stage + 4 * S::kTile + to_kscale;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const uint32_t at_key = (key_at ^ (c << 5)) + x * 2 * S::kTile;
          const uint2 klo = lds64(at_key), khi = lds64(at_key + 8 * (D / 2));
          const uint32_t at_scale = kscale_at + x * 32 * SB + 4 * c;
          const uint32_t both = f16x2_of_scales(__byte_perm(lds8(at_scale), lds8(at_scale + 8 * SB), 0x0040));
          const uint32_t slo = low_twice(both), shi = high_twice(both);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            uint32_t lo[4], hi[4];
            f16x2_of_e2m1(w ? klo.y : klo.x, lo);
            f16x2_of_e2m1(w ? khi.y : khi.x, hi);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const uint32_t a0 = mul_f16x2(lo[2 * e], slo), a1 = mul_f16x2(hi[2 * e], shi);
              const uint32_t a2 = mul_f16x2(lo[2 * e + 1], slo), a3 = mul_f16x2(hi[2 * e + 1], shi);
#pragma unroll
              for (int n = 0; n < NB; ++n) mma(s[x][n], a0, a1, a2, a3, qf[n][c][2 * w + e][0], qf[n][c][2 * w + e][1]);
            }
          }
        }
      }
      if (!plain(u) || have != 3u) {
        const int j0 = step_base(u) + g;
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (!(have >> x & 1) || !sp.sees(pos[n][e & 1], j0 + 16 * x + 8 * (e >> 1))) s[x][n][e] = -INFINITY;
      }
      // weights relative to the reference so far
      float w[2][NB][4];
      bool move = false;
      auto weigh = [&](int n, int h) {
        float sum = 0.f;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          w[x][n][h] = ex2(fmaf(s[x][n][h], rf[n][h], shift[n][h]));
          w[x][n][2 + h] = ex2(fmaf(s[x][n][2 + h], rf[n][h], shift[n][h]));
          sum += w[x][n][h] + w[x][n][2 + h];
        }
        return sum;
      };
      float sum[NB][2];
#pragma unroll
      for (int n = 0; n < NB; ++n)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          sum[n][h] = weigh(n, h);
          move |= sum[n][h] > kMostSum;
        }
      if (__any_sync(0xffffffffu, move)) {
        // rows whose weights are too large for f16, or that have no reference
        // yet, take their maximum
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const unsigned of_row = __ballot_sync(0xffffffffu, sum[n][h] > kMostSum) & (0x11111111u << t);
            float top = fmaxf(fmaxf(s[0][n][h], s[0][n][2 + h]), fmaxf(s[1][n][h], s[1][n][2 + h])) * rf[n][h];
#pragma unroll
            for (int off = 4; off < 32; off <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
            if (of_row) {
              const bool none = shift[n][h] == kNone;
              const float to = none ? kRefBelow - top : fminf(shift[n][h], kRefBelow - top);
              const float f = none ? 0.f : ex2(to - shift[n][h]);
              shift[n][h] = to;
              l[n][h] *= f;
#pragma unroll
              for (int i = 0; i < MT; ++i) {
                o[n][i][h] *= f;
                o[n][i][2 + h] *= f;
              }
              sum[n][h] = weigh(n, h);
            }
          }
      }
      uint32_t p[2][NB][2];
#pragma unroll
      for (int n = 0; n < NB; ++n) {
#pragma unroll
        for (int h = 0; h < 2; ++h) l[n][h] += sum[n][h];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          p[x][n][0] = transpose8x8(pack_f16(w[x][n][0], w[x][n][1]));
          p[x][n][1] = transpose8x8(pack_f16(w[x][n][2], w[x][n][3]));
        }
      }
      // values: the lane's run of codes of tokens 2t, 2t+1 | 2t+8, 2t+9
      constexpr int RW = D >= 128 ? 2 : 1;   // words of the run
      const uint32_t value_at = at_stage + to_value + S::kTile, vscale_at = at_stage + 4 * S::kTile + 16 * SB + to_vscale;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
#pragma unroll
        for (int c = 0; c < (D + 127) / 128; ++c) {
          uint32_t vw[4][RW], scale[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t row = value_at ^ (c << 6);
            const uint32_t from_row = (i & 1 ? (D == 256 ? (row + 128) ^ 64u : row ^ (D / 2)) : row) + (i >> 1) * 8 * (D / 2) +
                                      x * 2 * S::kTile;
            if constexpr (D == 64) {
              vw[i][0] = lds32(from_row);
            } else {
              const uint2 y = lds64(from_row);
              vw[i][0] = y.x;
              vw[i][RW - 1] = y.y;
            }
            scale[i] = lds8(vscale_at + (x * 32 + (i & 1) + 8 * (i >> 1)) * SB + 8 * c);
          }
          const uint32_t sa = f16x2_of_scales(__byte_perm(scale[0], scale[1], 0x0040));
          const uint32_t sb = f16x2_of_scales(__byte_perm(scale[2], scale[3], 0x0040));
#pragma unroll
          for (int y = 0; y < RW; ++y) {
            uint32_t ae[4], ao[4], be[4], bo[4];   // elements 0, 2, 4, 6 and 1, 3, 5, 7 of tokens 2t, 2t+1 and 2t+8, 2t+9
            f16x2_of_e2m1(even_codes(vw[0][y], vw[1][y]), ae);
            f16x2_of_e2m1(odd_codes(vw[0][y], vw[1][y]), ao);
            f16x2_of_e2m1(even_codes(vw[2][y], vw[3][y]), be);
            f16x2_of_e2m1(odd_codes(vw[2][y], vw[3][y]), bo);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t a0 = mul_f16x2(ae[e], sa), a1 = mul_f16x2(ao[e], sa);
              const uint32_t a2 = mul_f16x2(be[e], sb), a3 = mul_f16x2(bo[e], sb);
#pragma unroll
              for (int n = 0; n < NB; ++n) mma(o[n][c * 8 + 4 * y + e], a0, a1, a2, a3, p[x][n][0], p[x][n][1]);
            }
          }
        }
      }
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
          s_m[warp][r] = shift[n][h] == kNone ? -INFINITY : -shift[n][h];
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
      const float ref = mm == -INFINITY ? 0.f : mm;   // no weights at all: each factor is 0
      float sum = 0.f;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float f = ex2(s_m[w][r] - ref);
        sum += s_l[w][r] * f;
        const float4 x = *reinterpret_cast<const float4*>(reinterpret_cast<float*>(smem) + w * (S::kRing / 4) + r * D +
                                                          (d ^ ((r & 7) << 2)));
        acc.x += x.x * f;
        acc.y += x.y * f;
        acc.z += x.z * f;
        acc.w += x.w * f;
      }
      if (whole) {
        const int tok = tok_of(r), head = kvh * a.group + (head0 + r - tok * a.group);
        store_row4(a, rq.row0 + tok0 + tok, head, D, d, acc, mm, sum);
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

// Joins the partial sums of the row tiles that more than one CTA worked on: a block
// for each CTA that may have begun one, a warp for a row, the parts in order.  Small
// blocks find room as soon as the first CTAs of the kernel before are gone, and
// nothing but the tile has to be looked up (a block on each SM, to which the rows
// are dealt, took 4.5 us beside the kernel, these 3.2).  Several parts' columns are on
// their way at once, to shared memory.
template <int D, int NB> struct JoinShape {
  static constexpr int kBatch = 16 / NB / (D == 256 ? 2 : 1);   // parts
  static constexpr int kSmem = 8 * NB * kBatch * D * 4;
};

template <int D, int NB>
__global__ void __launch_bounds__(8 * NB * 32) block_attn_join(BlockPaArgs a) {
  using S = Shape<D, NB, true>;
  constexpr int kRows = S::kRows, VEC = D / 64, BATCH = JoinShape<D, NB>::kBatch;   // VEC: pairs of columns of a lane
  extern __shared__ __align__(128) char smem[];
  pdl_enter();
  const int lane = threadIdx.x & 31, r = threadIdx.x >> 5, c0 = blockIdx.x;
  const JoinTile tile = a.joins[c0];
  if (r >= tile.rows) return;
  float* mine = reinterpret_cast<float*>(smem) + r * (BATCH * D);
  auto part_of = [&](int c) { return a.part + (static_cast<int64_t>(c) * 2 + (c == c0 ? tile.slot : 0)) * S::kPart; };
  float m = -INFINITY, sum = 0.f;
  float2 acc[VEC] = {};
#pragma unroll 1
  for (int c = c0; c <= tile.last; c += BATCH) {
    const int n = min(BATCH, tile.last + 1 - c);
    float pm = -INFINITY, pl = 0.f;
    if (lane < n) {
      const float* p = part_of(c + lane) + kRows * D + r;
      pm = p[0];
      pl = p[kRows];
    }
#pragma unroll
    for (int i = 0; i < BATCH * D / 128; ++i) {
      const int x = i * 32 + lane, part = x / (D / 4), col = x % (D / 4) * 4;
      if (part < n) cp16(ptx::smem_u32(mine + part * D + col), part_of(c + part) + r * D + col);
    }
    cp_commit();
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
    cp_wait<0>();
    __syncwarp();
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const float2 v = *reinterpret_cast<const float2*>(mine + i * D + (e * 32 + lane) * 2);
        acc[e].x += v.x * wi;
        acc[e].y += v.y * wi;
      }
    }
    __syncwarp();   // the columns have been read
  }
  const int tok = (tile.row0 + r) / a.group, head = tile.kvh * a.group + (tile.row0 + r) % a.group;
  const float f = out_factor(a, sum);
  __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(a.out + static_cast<int64_t>(tile.token0 + tok) * a.os +
                                                          static_cast<int64_t>(head) * D);
#pragma unroll
  for (int e = 0; e < VEC; ++e) out[e * 32 + lane] = __floats2bfloat162_rn(acc[e].x * f, acc[e].y * f);
  if (a.lse && lane == 0) store_lse(a, tile.token0 + tok, head, m, sum);
}

struct Kernels {
  template <int D, int NB> static constexpr auto of() { return &block_attn_kernel<D, NB>; }
  template <int D, int NB> static cudaError_t join(const BlockPaArgs& a, int ctas, cudaStream_t s) {
    constexpr int smem = JoinShape<D, NB>::kSmem;
    const cudaError_t err = ensure_kernel_attrs(reinterpret_cast<const void*>(block_attn_join<D, NB>), smem);
    if (err != cudaSuccess) return err;
    return launch_pdl(block_attn_join<D, NB>, ctas, 8 * NB * 32, smem, s, a);
  }
};

bool config_ok(const moe_paged_attention_config_t* cfg, const moe_blockkv_cache_t* cache) {
  return cfg && blockkv_shape_ok(cache) && attention_config_ok(cfg, kMaxBlockBatch, cache->n_kv_heads, cache->head_dim);
}

BlockPaArgs args_of(const moe_blockkv_cache_t* cache) {
  BlockPaArgs a;
  a.c.k = cache->k;
  a.c.v = cache->v;
  a.c.k_scale = a.c.v_scale = nullptr;
  a.c.page_table = cache->page_table;
  a.c.n_pages = cache->n_pages;
  a.c.page_size = cache->page_size;
  a.c.n_kv_heads = cache->n_kv_heads;
  a.c.head_dim = cache->head_dim;
  a.c.max_pages = cache->max_pages;
  a.c.page_stride = cache->page_stride;
  a.c.head_stride = cache->head_stride;
  a.c.token_stride = cache->token_stride;
  a.k_scales = static_cast<const uint8_t*>(cache->k_scale);
  a.v_scales = static_cast<const uint8_t*>(cache->v_scale);
  a.page16 = static_cast<uint32_t>(cache->page_stride / 16);
  a.page_s = static_cast<uint32_t>(cache->scale_page_stride / (cache->head_dim / 16));
  a.scale_page = cache->scale_page_stride;
  a.scale_head = cache->scale_head_stride;
  a.scale_token = cache->scale_token_stride;
  a.kg = cache->k_gscale;
  a.vg = cache->v_gscale;
  return a;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_blockkv_attention_ws_bytes(const moe_paged_attention_config_t* cfg,
                                                 const moe_blockkv_cache_t* cache) {
  using namespace moe;
  return config_ok(cfg, cache) ? attention_ws_bytes(args_of(cache), cfg) : 0;
}

extern "C" moe_status_t moe_blockkv_attention(const moe_paged_attention_config_t* cfg, const moe_blockkv_cache_t* cache,
                                              const void* q, const int32_t* cu, const int32_t* kv_len, void* out,
                                              float* lse, void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  if (!config_ok(cfg, cache)) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!blockkv_pointers_ok(cache)) return MOE_ERR_INVALID_ARG;
  return attention_call<Kernels>(args_of(cache), cfg, q, cu, kv_len, out, lse, ws, ws_bytes, stream);
}
