// Attention over the paged 8-bit cache (include/paged_kv.h,
// moe_paged_attention) for few query rows per request and key head: the
// single-token form, small drafts, and every shape that paged_attn_tc.cuh does
// not take.
//
// The work is cut as paged_attn_rows.cuh says.
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
// 128/1 24, 256/1 76, outside the loop over the units.
#include "paged_attn_rows.cuh"

namespace moe {
namespace {

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

template <int D, int NB>
__global__ void __launch_bounds__(kWarps * 32, Shape<D, NB, false>::kCtas) paged_attn_kernel(PaArgs a) {
  using S = Shape<D, NB, false>;
  constexpr int kUnit = S::kUnit, kTileCost = S::kTileCost;
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
template <int D, int NB>
__global__ void __launch_bounds__(kJoinWarps * 32) paged_attn_join(PaArgs a, int n_ctas) {
  using S = Shape<D, NB, false>;
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
      const float f = out_factor(a, sum);
      __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(a.out + static_cast<int64_t>(tile.token0 + tok) * a.os +
                                                              static_cast<int64_t>(head) * D);
#pragma unroll
      for (int e = 0; e < VEC; ++e) out[e * 32 + lane] = __floats2bfloat162_rn(acc[e].x * f, acc[e].y * f);
      if (a.lse && lane == 0) store_lse(a, tile.token0 + tok, head, m, sum);
    }
  }
}

struct Kernels {
  template <int D, int NB> static constexpr auto of() { return &paged_attn_kernel<D, NB>; }
  template <int D, int NB> static cudaError_t join(const PaArgs& a, int ctas, cudaStream_t s) {
    constexpr int on_sm = Shape<D, NB, false>::kCtas;
    static_assert(kMaxSms * on_sm <= kMaxCtas && kMaxCtas <= kJoinWarps * 32, "a thread of the join for each CTA");
    return launch_pdl(paged_attn_join<D, NB>, ctas / on_sm, kJoinWarps * 32, 0, s, a, ctas);
  }
};

bool config_ok(const moe_paged_attention_config_t* cfg, const moe_kv_cache_t* cache) {
  return cfg && kv_cache_shape_ok(cache) && attention_config_ok(cfg, kMaxBatch, cache->n_kv_heads, cache->head_dim);
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_paged_attention_ws_bytes(const moe_paged_attention_config_t* cfg, const moe_kv_cache_t* cache) {
  using namespace moe;
  if (!config_ok(cfg, cache)) return 0;
  PaArgs a;
  a.c = *cache;
  return attention_ws_bytes(a, cfg);
}

extern "C" moe_status_t moe_paged_attention(const moe_paged_attention_config_t* cfg, const moe_kv_cache_t* cache,
                                            const void* q, const int32_t* cu, const int32_t* kv_len, void* out,
                                            float* lse, void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  if (!config_ok(cfg, cache)) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!kv_cache_pointers_ok(cache)) return MOE_ERR_INVALID_ARG;
  PaArgs a;
  a.c = *cache;
  return attention_call<Kernels>(a, cfg, q, cu, kv_len, out, lse, ws, ws_bytes, stream);
}
