// Append to the paged 4-bit cache (include/block_kv.h, moe_blockkv_append): QK
// norm, rotation, block scales and E2M1 codes in one launch.
//
// With y = norm(x) rotated and s the smallest E4M3 value that holds the largest
// |y| of 16 elements in E2M1's 6 g s, a code is y / (s g) rounded once;
// everything before it is fp32 in the order that the header fixes, so that a
// code next to a border is the same whoever computes it.
//
// A block's scale belongs to its token, so the rows of keys and values are
// independent: no reduction over a page, no second look at what it held.  Cache
// blocks own 16 slots of a page, for keys or for values, and share their rows with
// others, a round each: that many blocks hide each other's look-ups.  A thread has
// one block of 16 elements, several rows of it under way.  In the half layout it
// has four keys and their partners instead, which belong to other blocks of 16
// than its neighbours' do; the sizes of all fours of a row go through shared
// memory then.  Query blocks are those of kv_rows.cuh.
//
// Measured: 32 x 256 tokens of 32 + 4 heads of 128, norm and rotation, 156 MB in 32.0 us
// = 4.9 TB/s (the queries are 134 MB of that; 71 % of the issue slots, the first stall
// that a warp is not selected, and look-ups before the rows); ragged prompts up to 1999
// tokens of 16 + 16 heads of 64, 214 MB in 48.5 us = 4.4 TB/s, at 64 % of the issue slots
// and with waits for loads (with IEEE divisions and eight elements a thread 72 us); 64
// single tokens 3.7 us in a graph.  The interleaved layout spills 144 to 152 bytes of 72
// registers with four heads a thread; with two heads it spills 16 and takes 51.8 us,
// with 80 registers and six blocks on an SM 4 us more as well.
#include "block_kv.cuh"
#include "kv_rows.cuh"

namespace moe {
namespace {

constexpr int kThreads = kQueryThreads;

// Two heads a thread for few tokens (64 single ones: 3.7 us, one head 4.0, four 4.7), else
// four (32 x 256: 32 us, two 34).  Measured in a graph (us, two / four; *: the rule takes
// the slower), 32 + 4 heads of 128: 128 single tokens 4.7 / 5.2, 192 6.0 / 5.9*, 256 7.2 / 6.5*,
// 384 9.7 / 8.7, 1024 23.1 / 17.7; a prompt of 512 3.9 / 5.0*, two of 1000 8.6 / 8.2; 16 + 16 of
// 64, interleaved, 128 5.9 / 6.0, 256 8.7 / 7.9*, 1024 27 / 21; a prompt of 512 4.0 / 5.4*, two of
// 1000 6.8 / 8.7*; 8 + 8 of 128, 64 5.1 / 4.9*, 256 11.7 / 8.9*, 384 16.2 / 11.9; 16 + 2 of 256 (two key
// heads, so that four have nothing to do) 256 7.3 / 8.5, 4096 100 / 113*.
constexpr int kFewTokens = 256;

struct BaArgs : RowArgs {
  moe_blockkv_cache_t c;
  int work;   // blocks but those that check offsets
  int items, key_parts, parts;   // groups of slots that the requests can touch; blocks of one for keys, and in all
  uint32_t chunks, per_chunk;    // a token's heads by the number that a thread has under way; 2^32 / chunks, rounded up
  uint32_t page16, page_s;       // page strides in units of 16 bytes, and of D / 16
};

// The heads that a thread works on: `heads` of `token`'s from `head` on, none for
// threads without work.  i counts tokens and chunks of U heads.
struct Rows {
  int token, head, heads;
};
template <int U>
__device__ __forceinline__ Rows rows_of(const BaArgs& a, int tokens, int i) {
  Rows r;
  r.token = a.chunks == 1 ? i : __umulhi(i, a.per_chunk);
  r.head = (i - r.token * static_cast<int>(a.chunks)) * U;
  r.heads = r.token < tokens ? min(U, a.c.n_kv_heads - r.head) : 0;
  return r;
}

__device__ __forceinline__ float square_of_four(const float* x) {
  return __fadd_rn(__fadd_rn(__fmul_rn(x[0], x[0]), __fmul_rn(x[1], x[1])),
                   __fadd_rn(__fmul_rn(x[2], x[2]), __fmul_rn(x[3], x[3])));
}

// 1 / sqrt(mean + eps) from the thread's share of a row's sum of squares: a tree
// over the row's TPR threads, in the header's order.
template <int D, int TPR>
__device__ __forceinline__ float rstd_of(float ss, float eps) {
#pragma unroll
  for (int off = 1; off < TPR; off <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, off));
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fmul_rn(ss, 1.0f / D), eps)));
}

__device__ __forceinline__ void rotate(float& a, float& b, const float2& cs) {
  const float x = a, y = b;
  a = __fsub_rn(__fmul_rn(x, cs.x), __fmul_rn(y, cs.y));
  b = __fadd_rn(__fmul_rn(y, cs.x), __fmul_rn(x, cs.y));
}

// Largest finite size of N elements, NaN if one of them is; bad: one is not finite.
template <int N>
__device__ __forceinline__ float largest_of(const float* x, bool& bad) {
  float top = fabsf(x[0]);
#pragma unroll
  for (int e = 1; e < N; ++e) top = max_or_nan(top, fabsf(x[e]));
  if (top < INFINITY) return top;
  bad = true;
  if (top != top) return top;
  float t = 0.f;
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (fabsf(x[e]) < INFINITY) t = fmaxf(t, fabsf(x[e]));
  return t;
}

// The smallest E4M3 value s from 2^-9 on with top <= 6 s (448 where there is none):
// top / 6, rounded down, is rounded up to E4M3's three bits by the addition of a
// number whose last place is theirs; where the first rounding took that below s,
// which 6 s < top tells exactly, the next value is s.  (Sizes beyond the largest scale
// need no more than to stay there: the number added to 2^108 would be infinite.)
__device__ __forceinline__ float block_scale(float top) {
  if (top != top) return top;
  const float t = fminf(__fmul_rd(top, 0.16666666f), 512.f);   // below 1 / 6
  const float magic = __uint_as_float(max(__float_as_uint(t) & 0x7f800000u, 0x3c800000u) + 0x0a000000u);   // 2^20 times t's, or 2^-6
  float s = fminf(fmaxf(__fadd_ru(t, magic) - magic, 0.001953125f), 448.f);
  if (6.f * s < top) {
    const float place = __uint_as_float(max(__float_as_uint(s) & 0x7f800000u, 0x3c800000u) - 0x01800000u);   // 2^-3 times s's, or 2^-6
    s = fminf(s + place, 448.f);
  }
  return s;
}

// A scale as its code (NaN: E4M3's).
__device__ __forceinline__ uint8_t scale_code(float s) {
  return static_cast<uint8_t>(__nv_cvt_float_to_fp8(s, __NV_SATFINITE, __NV_E4M3));
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// N quotients x / sg, near enough to give every code as the exact ones would.
// They are x inv (inv: 1 / sg to a unit of the last place) corrected by their
// remainders, which are exact: sg has four significant bits and a border m between
// two codes three, so x (24 bits) either is m sg, and then the corrected quotient
// is m (it is off by 2^-45 before its rounding), or lies a unit of its last place
// away, and then x / sg is over half a unit of m's from m.
// fine: x is finite and none is over 6 sg; else what is larger, whose product with
// inv may overflow, becomes 6 sg, the same code.  (A NaN's sg is NaN, and so are its
// quotients.)
template <int N>
__device__ __forceinline__ void quotients(float (&q)[N], float* x, float sg, float inv, bool fine) {
  if (!fine) {
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = fminf(fmaxf(x[i], -6.f * sg), 6.f * sg);
  }
  const uint64_t sg2 = pair(-sg, -sg), inv2 = pair(inv, inv);
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const uint64_t x2 = pair(x[i], x[i + 1]), q2 = mul2(x2, inv2);
    unpair(fma2(fma2(q2, sg2, x2), inv2, q2), q[i], q[i + 1]);
  }
}

// Codes of the nearest values, ties to even, element 0 in the low four bits.
__device__ __forceinline__ uint32_t codes4(const float* q) {
  uint32_t r;
  asm("{\n .reg .b8 a, b;\n .reg .b16 c;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " mov.b16 c, {a, b};\n cvt.u32.u16 %0, c;\n}\n"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]));
  return r;
}
__device__ __forceinline__ uint32_t codes8(const float* q) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(q[0]), "f"(q[1]), "f"(q[2]), "f"(q[3]), "f"(q[4]), "f"(q[5]), "f"(q[6]), "f"(q[7]));
  return r;
}

__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The 16 elements of a block, whose largest size is `top`, to their place.
__device__ __forceinline__ void store_block(uint8_t* codes, uint8_t* scale, float (&x)[16], float top, bool odd, float g,
                                            float inv_g) {
  const float s = block_scale(top * inv_g), sg = s * g, inv = reciprocal(sg);
  float q[16];
  quotients(q, x, sg, inv, !odd && top <= 6.f * sg);
  *reinterpret_cast<uint2*>(codes) = make_uint2(codes8(q), codes8(q + 8));
  *scale = scale_code(s);
}

// 16 slots of a page and the tokens among them that are new: `tokens` from
// position `first` on, whose rows begin at row0.
struct Slots {
  int64_t row0;
  int first, tokens, pid;   // pid: outside the cache is recorded where it is met
};

// False: nothing to do (or wrong offsets or a length past the page table, which are
// recorded).
__device__ __forceinline__ bool find_slots(const BaArgs& a, int item, Slots& s) {
  const int b = warp_find_request(a.cu, a.B, item, 1, kSlots, 2);
  const Request r = load_request(a.cu, a.kv_len, b, a.T);
  if (!r.ok || r.start < 0) {
    if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return false;
  }
  const int group = slot_group(r, b, item);
  if (group < 0) return false;
  const int page = group >> (27 - __clz(a.c.page_size));   // of page_size / 16 groups
  if (page >= a.c.max_pages) {   // past the page table, and maybe past what the next lines can count
    if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return false;
  }
  const int base = group * kSlots;
  s.first = max(base, r.start);
  s.tokens = min(base + kSlots, r.end) - s.first;
  s.row0 = r.row0 + (s.first - r.start);
  s.pid = a.c.page_table[static_cast<int64_t>(b) * a.c.max_pages + page];
  return true;
}

__device__ __forceinline__ bool has_page(const BaArgs& a, const Slots& s) {
  const bool there = static_cast<unsigned>(s.pid) < static_cast<unsigned>(a.c.n_pages);
  if (!there && threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
  return there;
}

// The cache's codes and scales of a token's key (or value) head.
struct Target {
  uint8_t *codes, *scales;
};
template <int D>
__device__ __forceinline__ Target target_of(const BaArgs& a, const Slots& s, const Rows& r, bool key) {
  const int slot = (s.first + r.token) & (a.c.page_size - 1);
  const uint64_t page = static_cast<uint64_t>(s.pid * a.page16) * 16u, page_s = static_cast<uint64_t>(s.pid * a.page_s) * (D / 16);
  return Target{static_cast<uint8_t*>(key ? a.c.k : a.c.v) + page + (r.head * a.c.head_stride + slot * a.c.token_stride),
                static_cast<uint8_t*>(key ? a.c.k_scale : a.c.v_scale) + page_s +
                    (r.head * a.c.scale_head_stride + slot * a.c.scale_token_stride)};
}

// The frequency table's row of a token, -1 (recorded) outside it; 0 without a rotation.
__device__ __forceinline__ int angle_row(const BaArgs& a, const Slots& s, int token) {
  if (a.rot == 0) return 0;
  const int f = table_row(a, static_cast<int>(s.row0) + token, s.first + token);
  if (f < 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
  return f;
}

// Share `part` of the values: U heads of a token a thread.
template <int D, int U>
__device__ __forceinline__ void append_values(const BaArgs& a, const Slots& s, int part) {
  constexpr int TPR = D / 16, GROUPS = kThreads / TPR;
  const int lr = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  Rows r = rows_of<U>(a, s.tokens, part * GROUPS + grp);
  const uint4* from =
      reinterpret_cast<const uint4*>(a.v + (s.row0 + r.token) * a.vs + static_cast<int64_t>(r.head) * D + lr * 16);
  uint4 raw[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (u < r.heads) {
      raw[u][0] = from[u * (D / 8)];
      raw[u][1] = from[u * (D / 8) + 1];
    }
  if (r.heads && angle_row(a, s, r.token) < 0) r.heads = 0;
  if (!has_page(a, s)) return;
  const float g = a.c.v_gscale, inv_g = 1.f / g;   // powers of two
  Target to = target_of<D>(a, s, r, false);
  to.codes += lr * 8;
  to.scales += lr;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (u >= r.heads) break;
    const uint32_t w[8] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w, raw[u][1].x, raw[u][1].y, raw[u][1].z, raw[u][1].w};
    float x[16];
    uint32_t bits = 0;   // the largest size as bf16 bits: a NaN's are above infinity's
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      bits = __vmaxu2(bits, w[e] & 0x7fff7fffu);
    }
    bits = max(bits & 0xffffu, bits >> 16);
    float top = __uint_as_float(bits << 16);
    bool odd = false;
    if (bits >= 0x7f80u) {
      top = largest_of<16>(x, odd);
      set_status(a.status, MOE_ERR_DEVICE_NONFINITE);
    }
    store_block(to.codes, to.scales, x, top, odd, g, inv_g);
    to.codes += a.c.head_stride;
    to.scales += a.c.scale_head_stride;
  }
}

// Share `part` of the keys, the interleaved layout: U heads of a token a thread.
template <int D, int U>
__device__ __forceinline__ void append_keys_interleaved(const BaArgs& a, const Slots& s, int part) {
  constexpr int TPR = D / 16, GROUPS = kThreads / TPR;
  const int lr = threadIdx.x % TPR, grp = threadIdx.x / TPR, o = lr * 16;
  Rows r = rows_of<U>(a, s.tokens, part * GROUPS + grp);
  const uint4* from = reinterpret_cast<const uint4*>(a.k + (s.row0 + r.token) * a.ks + static_cast<int64_t>(r.head) * D + o);
  uint4 raw[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
    if (u >= r.heads) continue;
    raw[u][0] = from[u * (D / 8)];
    raw[u][1] = from[u * (D / 8) + 1];
  }
  // of the block's two halves, as rotations end at a multiple of 8
  const bool turns[2] = {o < a.rot, o + 8 < a.rot};
  float4 cs[2][2];
  const int f = r.heads ? angle_row(a, s, r.token) : 0;
  if (f < 0) r.heads = 0;
  const float4* angles = reinterpret_cast<const float4*>(a.cos_sin + static_cast<int64_t>(f) * (a.rot / 2) + lr * 8);
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (r.heads && turns[h]) {
      cs[h][0] = __ldg(angles + 2 * h);
      cs[h][1] = __ldg(angles + 2 * h + 1);
    }
  const bool norm = a.gamma_k;
  float gamma[16];
  if (norm) {
#pragma unroll
    for (int e = 0; e < 16; e += 4) *reinterpret_cast<float4*>(gamma + e) = __ldg(reinterpret_cast<const float4*>(a.gamma_k + o + e));
  }
  if (!has_page(a, s)) return;
  const float g = a.c.k_gscale, inv_g = 1.f / g;   // powers of two
  Target to = target_of<D>(a, s, r, true);
  to.codes += lr * 8;
  to.scales += lr;
  bool bad = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const uint32_t w[8] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w, raw[u][1].x, raw[u][1].y, raw[u][1].z, raw[u][1].w};
    float x[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      x[2 * e] = __uint_as_float(w[e] << 16);
      x[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    }
    if (norm) {
      const float ss = __fadd_rn(__fadd_rn(square_of_four(x), square_of_four(x + 4)),
                                 __fadd_rn(square_of_four(x + 8), square_of_four(x + 12)));
      const float rstd = rstd_of<D, TPR>(ss, a.eps);
#pragma unroll
      for (int e = 0; e < 16; ++e) x[e] = __fmul_rn(__fmul_rn(x[e], rstd), gamma[e]);
    }
    if (u >= r.heads) continue;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (turns[h])
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          rotate(x[8 * h + 4 * e], x[8 * h + 4 * e + 1], make_float2(cs[h][e].x, cs[h][e].y));
          rotate(x[8 * h + 4 * e + 2], x[8 * h + 4 * e + 3], make_float2(cs[h][e].z, cs[h][e].w));
        }
    bool odd = false;
    const float top = largest_of<16>(x, odd);
    bad |= odd;
    store_block(to.codes, to.scales, x, top, odd, g, inv_g);
    to.codes += a.c.head_stride;
    to.scales += a.c.scale_head_stride;
  }
  if (bad) set_status(a.status, MOE_ERR_DEVICE_NONFINITE);
}

// ... and the half layout.
template <int D, int U>
__device__ __forceinline__ void append_keys_half(const BaArgs& a, const Slots& s, int part) {
  constexpr int TPR = D / 8, GROUPS = kThreads / TPR;
  __shared__ float4 s_top[2][GROUPS][D / 16];   // sizes of a row's fours, in turn
  const int lr = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  Rows r = rows_of<U>(a, s.tokens, part * GROUPS + grp);
  const Place p = place_of<true>(lr, a.rot);
  const uint16_t* from = a.k + (s.row0 + r.token) * a.ks + static_cast<int64_t>(r.head) * D;
  Raw raw[U];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    raw[u] = Raw{make_uint2(0, 0), make_uint2(0, 0)};
    if (u < r.heads) raw[u] = load_raw<true>(from + u * D, p);
  }
  const int f = r.heads ? angle_row(a, s, r.token) : 0;
  if (f < 0) r.heads = 0;
  float2 cs[4];
  if (r.heads && p.rotates) load_cs<true>(a.cos_sin + static_cast<int64_t>(f) * (a.rot / 2), p, cs);
  const bool norm = a.gamma_k;
  Gamma gamma = {};
  if (norm) gamma = load_gamma(a.gamma_k, p);
  if (!has_page(a, s)) return;
  const float g = a.c.k_gscale, inv_g = 1.f / g;   // powers of two
  Target to = target_of<D>(a, s, r, true);
  bool bad = false;
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float x[8];
    unpack4(raw[u].a, x);
    unpack4(raw[u].b, x + 4);
    if (norm) {
      const float rstd = rstd_of<D, TPR>(__fadd_rn(square_of_four(x), square_of_four(x + 4)), a.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(__fmul_rn(x[e], rstd), gamma.g[e]);
    }
    const bool stored = u < r.heads;
    if (stored && p.rotates) {
#pragma unroll
      for (int e = 0; e < 4; ++e) rotate(x[e], x[4 + e], cs[e]);
    }
    bool odd[2] = {false, false};
    const float top[2] = {largest_of<4>(x, odd[0]), largest_of<4>(x + 4, odd[1])};
    bad |= (odd[0] || odd[1]) && stored;
    float* fours = reinterpret_cast<float*>(s_top[u & 1][grp]);
    fours[p.oa / 4] = top[0];
    fours[p.ob / 4] = top[1];
    __syncwarp();   // (what the other buffer held has been read)
    if (stored) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int o = h ? p.ob : p.oa;
        const float4 t = s_top[u & 1][grp][o / 16];
        const float sc = block_scale(max_or_nan(max_or_nan(t.x, t.y), max_or_nan(t.z, t.w)) * inv_g), sg = sc * g;
        float q[4];
        quotients(q, x + 4 * h, sg, reciprocal(sg), !odd[h] && top[h] <= 6.f * sg);
        *reinterpret_cast<uint16_t*>(to.codes + o / 2) = static_cast<uint16_t>(codes4(q));
        if (o % 16 == 0) to.scales[o / 16] = scale_code(sc);
      }
    }
    to.codes += a.c.head_stride;
    to.scales += a.c.scale_head_stride;
  }
  if (bad) set_status(a.status, MOE_ERR_DEVICE_NONFINITE);
}

// Blocks [0, parts items): cache blocks; then query blocks; from `work` on a few that
// check offsets.  U: heads that a thread has under way.
template <int D, bool HALF, int U>
__global__ void __launch_bounds__(kThreads, 7) blockkv_append_kernel(BaArgs a) {
  pdl_enter();
  const int n_cache = a.parts * a.items, i = blockIdx.x;
  if (i >= a.work) {
    check_offsets(a.cu, a.B, a.T, i - a.work, a.status);
    return;
  }
  if (i < n_cache) {
    const int item = i / a.parts, part = i - item * a.parts;
    Slots s;
    if (!find_slots(a, item, s)) return;
    if (part >= a.key_parts) append_values<D, U>(a, s, part - a.key_parts);
    else if (HALF) append_keys_half<D, U>(a, s, part);
    else append_keys_interleaved<D, U>(a, s, part);
    return;
  }
  const int q = i - n_cache;
  switch (query_tokens<D>(a.Hq, kThreads)) {
    case 4: query_block<D, HALF, 4>(a, 4 * q); break;
    case 2: query_block<D, HALF, 2>(a, 2 * q); break;
    default: query_block<D, HALF, 1>(a, q); break;
  }
}

template <int D, int U>
cudaError_t launch(BaArgs a, cudaStream_t s) {
  // a round of rows for each block
  const int groups = kThreads / (D / 16);   // of threads, one for a row
  a.chunks = ceil_div(a.c.n_kv_heads, U);
  a.per_chunk = static_cast<uint32_t>(((uint64_t(1) << 32) + a.chunks - 1) / a.chunks);   // exact below 16 chunks
  const int rounds = std::min(kSlots, a.T) * a.chunks;
  a.key_parts = ceil_div(rounds, a.half ? groups / 2 : groups);
  a.parts = a.key_parts + ceil_div(rounds, groups);
  int64_t blocks = static_cast<int64_t>(a.parts) * a.items;
  if (a.q) blocks += ceil_div(a.T, query_tokens<D>(a.Hq, kThreads));
  a.work = static_cast<int>(std::min<int64_t>(blocks, 0x7fffffff));
  blocks += ceil_div(a.B, kThreads);
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  count_launches(1);
  return launch_pdl(a.half ? blockkv_append_kernel<D, true, U> : blockkv_append_kernel<D, false, U>,
                    static_cast<unsigned>(blocks), kThreads, 0, s, a);
}

template <int D>
cudaError_t launch(const BaArgs& a, cudaStream_t s) {
  return a.T <= kFewTokens ? launch<D, 2>(a, s) : launch<D, 4>(a, s);
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_blockkv_append(const moe_kv_append_config_t* cfg, const moe_blockkv_cache_t* cache,
                                           const void* q, const void* k, const void* v, const float* gamma_q,
                                           const float* gamma_k, const float* cos_sin, const int32_t* positions,
                                           const int32_t* cu, const int32_t* kv_len, void* q_out, moe_stream_t stream) {
  using namespace moe;
  if (!cfg || !blockkv_shape_ok(cache)) return MOE_ERR_INVALID_ARG;
  const int D = cache->head_dim;
  if (!append_config_ok(cfg, kMaxBlockBatch, cache->n_kv_heads, D, q, gamma_q, q_out)) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!blockkv_pointers_ok(cache) || !append_pointers_ok(cfg, k, v, gamma_k, cos_sin, positions, cu, kv_len))
    return MOE_ERR_INVALID_ARG;
  unsigned* status = nullptr;
  int sms = 0;
  const moe_status_t st = current_device(&status, &sms);
  if (st != MOE_OK) return st;
  BaArgs a;
  fill_rows(a, cfg, q, k, v, gamma_q, gamma_k, cos_sin, positions, cu, kv_len, q_out, status);
  a.c = *cache;
  a.page16 = static_cast<uint32_t>(cache->page_stride / 16);
  a.page_s = static_cast<uint32_t>(cache->scale_page_stride / (D / 16));
  a.items = cfg->T / kSlots + 2 * cfg->batch;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  switch (D) {
    case 64: err = launch<64>(a, s); break;
    case 128: err = launch<128>(a, s); break;
    default: err = launch<256>(a, s); break;
  }
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
