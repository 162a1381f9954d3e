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
// blocks own 16 slots of a page (or a share of their rows), which costs them one
// look-up of request and page; D / 8 threads work on a row, eight elements each.
// In the half layout a thread holds four elements and their partners, which
// belong to other blocks of 16 than its neighbours' do; the sizes of all fours
// of a row go through shared memory then.  Query blocks are those of
// kv_rows.cuh.
//
// A request of n new tokens touches at most n/16 + 2 groups of 16 slots, so
// request b's blocks start at cu[b]/16 + 2b, as in kv_append.cu.
#include "block_kv.cuh"
#include "kv_rows.cuh"

namespace moe {
namespace {

constexpr int kSlots = 16;       // of a cache block
constexpr int kThreads = kQueryThreads;
constexpr int kHeads = 4;        // of a token, that a thread has under way

struct BaArgs : RowArgs {
  moe_blockkv_cache_t c;
  int items, parts;   // groups of slots that the requests can touch; blocks for one
  int chunks;         // kHeads heads of a token
};

// The row's sum of squares, in the header's order: the thread's two fours, then a
// tree over the row's TPR threads.
template <int TPR>
__device__ __forceinline__ float sum_of_squares(const float (&x)[8]) {
  auto four = [&](int i) {
    return __fadd_rn(__fadd_rn(__fmul_rn(x[i], x[i]), __fmul_rn(x[i + 1], x[i + 1])),
                     __fadd_rn(__fmul_rn(x[i + 2], x[i + 2]), __fmul_rn(x[i + 3], x[i + 3])));
  };
  float ss = __fadd_rn(four(0), four(4));
#pragma unroll
  for (int off = 1; off < TPR; off <<= 1) ss = __fadd_rn(ss, __shfl_xor_sync(0xffffffffu, ss, off));
  return ss;
}

template <bool HALF>
__device__ __forceinline__ void rotate(float (&x)[8], const float2 (&cs)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int ia = HALF ? i : 2 * i, ib = HALF ? i + 4 : 2 * i + 1;
    const float a = x[ia], b = x[ib];
    x[ia] = __fsub_rn(__fmul_rn(a, cs[i].x), __fmul_rn(b, cs[i].y));
    x[ib] = __fadd_rn(__fmul_rn(b, cs[i].x), __fmul_rn(a, cs[i].y));
  }
}

// Largest finite size of four elements, NaN if one of them is; bad: one is not finite.
__device__ __forceinline__ float largest4(const float* x, bool& bad) {
  const float top = max_or_nan(max_or_nan(fabsf(x[0]), fabsf(x[1])), max_or_nan(fabsf(x[2]), fabsf(x[3])));
  if (top < INFINITY) return top;
  bad = true;
  if (top != top) return top;
  float t = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (fabsf(x[e]) < INFINITY) t = fmaxf(t, fabsf(x[e]));
  return t;
}

// The block's scale as an E4M3 code, and its value times g (inv_6g: 1 / (6 g)).
// The conversion rounds to nearest; where that came out too small the next code
// is the one (sizes of E4M3 order like their codes), and 6 s g is exact.
__device__ __forceinline__ uint32_t scale_code(float top, float g, float inv_6g, float& sg) {
  if (top != top) {
    sg = 1.f;
    return 0x7fu;
  }
  uint32_t code = max(1u, static_cast<uint32_t>(__nv_cvt_float_to_fp8(top * inv_6g, __NV_SATFINITE, __NV_E4M3)));
  sg = e4m3_to_float(static_cast<uint8_t>(code)) * g;
  if (6.f * sg < top && code < 0x7eu) sg = e4m3_to_float(static_cast<uint8_t>(++code)) * g;
  return code;
}

// Four codes, element 0 in the low four bits.
__device__ __forceinline__ uint32_t codes_of(const float* x, float sg) {
  uint32_t r;
  asm("{\n .reg .b8 a, b;\n .reg .b16 c, d;\n cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " mov.b16 c, {a, b};\n cvt.u32.u16 %0, c;\n}\n"
      : "=r"(r)
      : "f"(__fdiv_rn(x[0], sg)), "f"(__fdiv_rn(x[1], sg)), "f"(__fdiv_rn(x[2], sg)), "f"(__fdiv_rn(x[3], sg)));
  return r;
}

// Share `part` of the rows of 16 slots: for keys, then for values, every token and
// kHeads of its heads at a time.
template <int D, bool HALF>
__device__ __forceinline__ void append_slots(const BaArgs& a, int item, int part) {
  constexpr int TPR = D / 8, GROUPS = kThreads / TPR, U = kHeads;
  __shared__ float4 s_top[2][GROUPS][D / 16];   // sizes of a row's fours, in turn
  const int ps = a.c.page_size, ps_log = 31 - __clz(ps), Hkv = a.c.n_kv_heads;
  const int b = warp_find_request(a.cu, a.B, item, 1, kSlots, 2);
  const Request r = load_request(a.cu, a.kv_len, b, a.T);
  if (!r.ok || r.start < 0) {
    if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  if (r.n == 0) return;
  const int at = item - (r.row0 / kSlots + 2 * b);
  const int base = (r.start / kSlots + at) * kSlots;
  if (at < 0 || base >= r.end) return;   // one block too many, or before the first request
  const int first = max(base, r.start), tokens = min(base + kSlots, r.end) - first;
  const int n = tokens * a.chunks;       // of keys; as many of values behind them
  if (part * GROUPS >= 2 * n) return;
  const int page = base >> ps_log;
  int pid = -1;
  if (page < a.c.max_pages) pid = a.c.page_table[static_cast<int64_t>(b) * a.c.max_pages + page];
  const int lr = threadIdx.x % TPR, grp = threadIdx.x / TPR;
  const Place pk = place_of<HALF>(lr, a.rot), pv = place_of<false>(lr, 0);
  const bool norm = a.gamma_k;
  Gamma gamma = {};
  if (norm) gamma = load_gamma(a.gamma_k, pk);
  int buffer = 0;
#pragma unroll 1
  for (int i0 = part * GROUPS; i0 < 2 * n; i0 += a.parts * GROUPS) {
    const int i = i0 + grp;
    const bool key = i < n;
    bool live = i < 2 * n;
    const int j = key ? i : i - n, token = live ? j / a.chunks : 0, h0 = live ? (j - token * a.chunks) * U : 0;
    const int64_t row = r.row0 + (first - r.start) + token;
    const Place p = key ? pk : pv;
    Raw raw[U];
    const uint16_t* from = key ? a.k + row * a.ks : a.v + row * a.vs;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      raw[u] = Raw{make_uint2(0, 0), make_uint2(0, 0)};
      if (live && h0 + u < Hkv) raw[u] = load_raw<HALF>(from + static_cast<int64_t>(h0 + u) * D, p);
    }
    float2 cs[4];
    if (a.rot > 0 && live) {
      const int f = table_row(a, static_cast<int>(row), first + token);
      live = f >= 0;
      if (f < 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      else if (key && p.rotates) load_cs<HALF>(a.cos_sin + static_cast<int64_t>(f) * (a.rot / 2), p, cs);
    }
    if (pid < 0 || pid >= a.c.n_pages) {
      if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      return;
    }
    const float g = key ? a.c.k_gscale : a.c.v_gscale, inv_6g = 1.f / (6.f * g);
    const int64_t slot = (first + token) & (ps - 1);
    uint8_t* codes = static_cast<uint8_t*>(key ? a.c.k : a.c.v) + pid * a.c.page_stride + h0 * a.c.head_stride +
                     slot * a.c.token_stride;
    uint8_t* scales = static_cast<uint8_t*>(key ? a.c.k_scale : a.c.v_scale) + pid * a.c.scale_page_stride +
                      h0 * a.c.scale_head_stride + slot * a.c.scale_token_stride;
    bool bad = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float x[8], top[2];
      unpack4(raw[u].a, x);
      unpack4(raw[u].b, x + 4);
      if (norm) {
        const float mean = __fmul_rn(sum_of_squares<TPR>(x), 1.0f / D);
        const float rstd = __frcp_rn(__fsqrt_rn(__fadd_rn(mean, a.eps)));
        if (key)
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = __fmul_rn(__fmul_rn(x[e], rstd), gamma.g[e]);
      }
      const bool stored = live && h0 + u < Hkv;
      if (live && key && p.rotates) rotate<HALF>(x, cs);
      bool not_finite = false;
      top[0] = largest4(x, not_finite);
      top[1] = largest4(x + 4, not_finite);
      bad |= not_finite && stored;
      if (HALF) {
        float* fours = reinterpret_cast<float*>(s_top[buffer][grp]);
        fours[p.oa / 4] = top[0];
        fours[p.ob / 4] = top[1];
        __syncwarp();   // (what the other buffer held has been read)
        if (stored) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int o = h ? p.ob : p.oa;
            const float4 t = s_top[buffer][grp][o / 16];
            float sg;
            const uint32_t sc = scale_code(max_or_nan(max_or_nan(t.x, t.y), max_or_nan(t.z, t.w)), g, inv_6g, sg);
            *reinterpret_cast<uint16_t*>(codes + o / 2) = static_cast<uint16_t>(codes_of(x + 4 * h, sg));
            if (o % 16 == 0) scales[o / 16] = static_cast<uint8_t>(sc);
          }
        }
        buffer ^= 1;
      } else {
        top[0] = max_or_nan(top[0], top[1]);
        top[0] = max_or_nan(top[0], __shfl_xor_sync(0xffffffffu, top[0], 1));
        if (stored) {
          float sg;
          const uint32_t sc = scale_code(top[0], g, inv_6g, sg);
          *reinterpret_cast<uint32_t*>(codes + lr * 4) = codes_of(x, sg) | codes_of(x + 4, sg) << 16;
          if (lr % 2 == 0) scales[lr / 2] = static_cast<uint8_t>(sc);
        }
      }
      codes += a.c.head_stride;
      scales += a.c.scale_head_stride;
    }
    if (bad) set_status(a.status, MOE_ERR_DEVICE_NONFINITE);
  }
}

// Blocks [0, parts items): cache blocks; the rest: query blocks.
template <int D, bool HALF>
__global__ void __launch_bounds__(kThreads, 7) blockkv_append_kernel(BaArgs a) {
  pdl_enter();
  const int n_cache = a.parts * a.items, i = blockIdx.x;
  if (i < n_cache) {
    const int item = i / a.parts;
    append_slots<D, HALF>(a, item, i - item * a.parts);
    return;
  }
  const int q = i - n_cache;
  switch (query_tokens<D>(a.Hq, kThreads)) {
    case 4: query_block<D, HALF, 4>(a, 4 * q); break;
    case 2: query_block<D, HALF, 2>(a, 2 * q); break;
    default: query_block<D, HALF, 1>(a, q); break;
  }
}

template <int D>
cudaError_t launch(BaArgs a, cudaStream_t s) {
  // a round of rows for each block
  a.chunks = ceil_div(a.c.n_kv_heads, kHeads);
  a.parts = ceil_div(2 * kSlots * a.chunks, kThreads / (D / 8));
  int64_t blocks = static_cast<int64_t>(a.parts) * a.items;
  if (a.q) blocks += ceil_div(a.T, query_tokens<D>(a.Hq, kThreads));
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  count_launches(1);
  return launch_pdl(a.half ? blockkv_append_kernel<D, true> : blockkv_append_kernel<D, false>,
                    static_cast<unsigned>(blocks), kThreads, 0, s, a);
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
  if (!append_config_ok(cfg, cache->n_kv_heads, D, q, gamma_q, q_out)) return MOE_ERR_INVALID_ARG;
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
