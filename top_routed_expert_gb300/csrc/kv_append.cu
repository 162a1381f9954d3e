// Append to the paged 8-bit cache (include/paged_kv.h, moe_kv_append): QK
// norm, rotation, page scale and E4M3 codes in one launch.
//
// Two kinds of blocks.  A cache block owns one page of one request for one
// head, keys or values: all new tokens of the page pass through its
// registers, so the page's scale is one block reduction and every code is
// written once.  A query block owns one token and turns all its query heads.
//
// Which pages a ragged batch touches is known on the device only.  A request
// of n new tokens touches at most n/page + 2 pages, so request b's blocks
// start at cu[b]/page + 2b, the grid has T/page + 2B of them, and a block
// finds its request by a search over cu; the few blocks too many leave.
#include "paged_kv.cuh"

namespace moe {
namespace {

constexpr float kMinScale = 9.094947017729282e-13f;   // 2^-40
constexpr int kQueryThreads = 128;

struct KaArgs {
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  const float* gamma_q;
  const float* gamma_k;
  const float2* cos_sin;
  const int32_t* positions;
  const int32_t* cu;
  const int32_t* kv_len;
  uint16_t* q_out;
  moe_kv_cache_t c;
  unsigned* status;
  int64_t qs, ks, vs, qos;
  int T, B, Hq, rot, n_pos, items;   // items: page blocks per head, keys or values
  float eps;
  bool half;
};

__device__ __forceinline__ void unpack4(const uint2& v, float* x) {
  x[0] = __uint_as_float(v.x << 16);
  x[1] = __uint_as_float(v.x & 0xffff0000u);
  x[2] = __uint_as_float(v.y << 16);
  x[3] = __uint_as_float(v.y & 0xffff0000u);
}

__device__ __forceinline__ uint2 pack4(const float* x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]);
  const __nv_bfloat162 b = __floats2bfloat162_rn(x[2], x[3]);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

__device__ __forceinline__ uint32_t codes4(const float* x, float inv) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0] * inv, x[1] * inv), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2] * inv, x[3] * inv), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

// Four codes times a power of two at most 1, rounded to codes again.
__device__ __forceinline__ uint32_t rescale4(uint32_t w, float f) {
  float x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) x[i] = e4m3_to_float(static_cast<uint8_t>(w >> (8 * i)));
  return codes4(x, f);
}

// A head is worked on by D/8 threads, eight elements each: the elements
// oa..oa+3 and ob..ob+3.  In the half layout's rotated part the second four
// are the partners of the first, elsewhere they are the next four.
struct Place {
  int oa, ob;
  bool rotates;
};

template <bool HALF>
__device__ __forceinline__ Place place_of(int lane_in_row, int rot) {
  Place p;
  p.rotates = lane_in_row * 8 < rot;
  if (HALF && p.rotates) {
    p.oa = lane_in_row * 4;
    p.ob = rot / 2 + p.oa;
  } else {
    p.oa = lane_in_row * 8;
    p.ob = p.oa + 4;
  }
  return p;
}

struct Raw {
  uint2 a, b;
};

// (Plain loads: the queries may be turned in place.)
__device__ __forceinline__ Raw load_raw(const uint16_t* row, const Place& p) {
  return Raw{*reinterpret_cast<const uint2*>(row + p.oa), *reinterpret_cast<const uint2*>(row + p.ob)};
}

// (cos, sin) of the thread's four pairs: frequencies oa..oa+3 of the half
// layout, (oa/2, oa/2+1, ob/2, ob/2+1) of the interleaved one; both are four
// consecutive table entries.
template <bool HALF>
__device__ __forceinline__ void load_cs(const float2* __restrict__ row, const Place& p, float2 (&cs)[4]) {
  const float4* f = reinterpret_cast<const float4*>(row + (HALF ? p.oa : p.oa / 2));
  const float4 x = __ldg(f), y = __ldg(f + 1);
  cs[0] = make_float2(x.x, x.y);
  cs[1] = make_float2(x.z, x.w);
  cs[2] = make_float2(y.x, y.y);
  cs[3] = make_float2(y.z, y.w);
}

struct Gamma {
  float g[8];
};

__device__ __forceinline__ Gamma load_gamma(const float* __restrict__ gamma, const Place& p) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(gamma + p.oa)), b = __ldg(reinterpret_cast<const float4*>(gamma + p.ob));
  return Gamma{{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w}};
}

// Norm and rotation of the thread's eight elements, in place.  TPR = D/8
// threads of a row, all of them call.
template <int TPR, bool HALF>
__device__ __forceinline__ void norm_rotate(float (&x)[8], bool norm, const Gamma& gamma, const Place& p,
                                            const float2 (&cs)[4], float eps) {
  if (norm) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int off = TPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
    const float rstd = rsqrtf(ss * (1.0f / static_cast<float>(TPR * 8)) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = x[i] * rstd * gamma.g[i];
  }
  if (!p.rotates) return;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    constexpr int step = HALF ? 1 : 2;
    const int ia = i * step, ib = HALF ? i + 4 : 2 * i + 1;
    const float a = x[ia], b = x[ib];
    x[ia] = fmaf(a, cs[i].x, -b * cs[i].y);
    x[ib] = fmaf(b, cs[i].x, a * cs[i].y);
  }
}

// The smallest power of two s >= 2^-40 with amax <= 448 s = 1.75 * 2^8 s.
__device__ __forceinline__ float scale_for(float amax) {
  if (!(amax > 448.f * kMinScale)) return kMinScale;
  const uint32_t u = __float_as_uint(amax);
  const uint32_t e = (u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1u : 0u);
  return __uint_as_float(e << 23);
}

// The larger of two sizes, NaN if either is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Row of the frequency table of a token, or -1.
__device__ __forceinline__ int table_row(const KaArgs& a, int t, int pos) {
  const int p = a.positions ? a.positions[t] : pos;
  return (p >= 0 && p < a.n_pos) ? p : -1;
}

// One page, one head, keys or values.  PASSES rows per thread group; the
// block covers the page's slots in PASSES rounds of blockDim / TPR rows.
template <int D, int PASSES, bool HALF, bool IS_V>
__device__ __forceinline__ void append_block(const KaArgs& a, int item, int head) {
  constexpr int TPR = D / 8;
  __shared__ float s_amax[32];
  const int ps = a.c.page_size, ps_log = 31 - __clz(ps);
  const int b = warp_find_request(a.cu, a.B, item, 1, ps, 2);
  const Request r = load_request(a.cu, a.kv_len, b, a.T);
  if (!r.ok || r.start < 0) {
    if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  if (r.n == 0) return;
  const int at = item - ((r.row0 >> ps_log) + 2 * b);
  const int page = (r.start >> ps_log) + at;
  const int base = page << ps_log;
  if (at < 0 || base >= r.end) return;   // one block too many, or before the first request
  int pid = -1;
  if (page < a.c.max_pages) pid = a.c.page_table[static_cast<int64_t>(b) * a.c.max_pages + page];
  const int lr = threadIdx.x % TPR, grp = threadIdx.x / TPR, rows = blockDim.x / TPR;
  const bool rotates = !IS_V && a.rot > 0, norm = !IS_V && a.gamma_k;
  const Place p = place_of<HALF>(lr, IS_V ? 0 : a.rot);
  const uint16_t* src = (IS_V ? a.v : a.k) + static_cast<int64_t>(head) * D;
  const int64_t stride = IS_V ? a.vs : a.ks;
  const int t0 = r.row0 - r.start;         // row of position 0
  Gamma gamma = {};
  if (norm) gamma = load_gamma(a.gamma_k, p);
  Raw raw[PASSES];
  float2 cs[PASSES][4];
  bool take[PASSES], outside = false;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int j = base + i * rows + grp;
    take[i] = j >= r.start && j < r.end && j < base + ps;
    raw[i] = Raw{make_uint2(0, 0), make_uint2(0, 0)};
    if (take[i]) raw[i] = load_raw(src + (t0 + j) * stride, p);
  }
  if (rotates) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int j = base + i * rows + grp;
      if (!take[i]) continue;
      const int f = table_row(a, t0 + j, j);
      if (f < 0) {
        outside = true;
        take[i] = false;
      } else if (p.rotates) {
        load_cs<HALF>(a.cos_sin + static_cast<int64_t>(f) * (a.rot / 2), p, cs[i]);
      }
    }
  }
  if (pid < 0 || pid >= a.c.n_pages) {
    if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  float* scale_at = (IS_V ? a.c.v_scale : a.c.k_scale) + static_cast<int64_t>(pid) * a.c.n_kv_heads + head;
  const bool had = r.start > base;
  const float old = had ? *scale_at : 0.f;
  float x[PASSES][8], amax = 0.f;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    unpack4(raw[i].a, x[i]);
    unpack4(raw[i].b, x[i] + 4);
    if (!IS_V) norm_rotate<TPR, HALF>(x[i], norm, gamma, p, cs[i], a.eps);
    float top = 0.f;   // a NaN or an infinity makes it one of them
#pragma unroll
    for (int e = 0; e < 8; ++e) top = max_or_nan(top, fabsf(x[i][e]));
    if (!take[i]) continue;
    if (top < INFINITY) {
      amax = fmaxf(amax, top);
    } else {
      bad = true;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (fabsf(x[i][e]) < INFINITY) amax = fmaxf(amax, fabsf(x[i][e]));
    }
  }
  if (bad) set_status(a.status, MOE_ERR_DEVICE_NONFINITE);
  if (outside && lr == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
  // sizes order like their bits
  amax = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(amax)));
  if ((threadIdx.x & 31) == 0) s_amax[threadIdx.x >> 5] = amax;
  __syncthreads();   // also: every thread has read the old scale
  for (int w = 0; w < static_cast<int>(blockDim.x / 32); ++w) amax = fmaxf(amax, s_amax[w]);
  const float scale = fmaxf(scale_for(amax), old);
  if (threadIdx.x == 0) *scale_at = scale;
  const float inv = 1.0f / scale;
  uint8_t* codes = static_cast<uint8_t*>(IS_V ? a.c.v : a.c.k) + pid * a.c.page_stride + head * a.c.head_stride;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int j = base + i * rows + grp;
    uint8_t* row = codes + (j - base) * a.c.token_stride;
    if (take[i]) {
      const uint32_t lo = codes4(x[i], inv), hi = codes4(x[i] + 4, inv);
      if (p.ob == p.oa + 4) {
        *reinterpret_cast<uint2*>(row + p.oa) = make_uint2(lo, hi);
      } else {
        *reinterpret_cast<uint32_t*>(row + p.oa) = lo;
        *reinterpret_cast<uint32_t*>(row + p.ob) = hi;
      }
    } else if (had && scale > old && j < r.start) {
      uint32_t* wa = reinterpret_cast<uint32_t*>(row + p.oa);
      uint32_t* wb = reinterpret_cast<uint32_t*>(row + p.ob);
      *wa = rescale4(*wa, old * inv);
      *wb = rescale4(*wb, old * inv);
    }
  }
}

// All query heads of one token.  The first rows are on their way while the
// token's request, position and angles are looked up.
template <int D, bool HALF>
__device__ __forceinline__ void query_block(const KaArgs& a, int t) {
  constexpr int TPR = D / 8, ILP = 4;
  const int lr = threadIdx.x % TPR, grp = threadIdx.x / TPR, groups = blockDim.x / TPR;
  const Place p = place_of<HALF>(lr, a.rot);
  const uint16_t* src = a.q + t * a.qs;
  uint16_t* dst = a.q_out + t * a.qos;
  Raw raw[ILP];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < ILP; ++i) {
      const int h = h0 + i * groups + grp;
      raw[i] = Raw{make_uint2(0, 0), make_uint2(0, 0)};
      if (h < a.Hq) raw[i] = load_raw(src + h * D, p);
    }
  };
  load(0);
  const bool norm = a.gamma_q;
  Gamma gamma = {};
  if (norm) gamma = load_gamma(a.gamma_q, p);
  float2 cs[4] = {};
  const int b = warp_find_request(a.cu, a.B, t, 1, 1, 0);
  const Request r = load_request(a.cu, a.kv_len, b, a.T);
  if (!r.ok || r.start < 0 || t < r.row0 || t >= r.row0 + r.n) return;   // recorded by the cache blocks, or no request's row
  if (a.rot > 0) {
    const int f = table_row(a, t, r.start + (t - r.row0));
    if (f < 0) {
      if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      return;
    }
    if (p.rotates) load_cs<HALF>(a.cos_sin + static_cast<int64_t>(f) * (a.rot / 2), p, cs);
  }
  // every thread makes the same number of rounds: the norm's shuffles need all lanes
  for (int h0 = 0; h0 < a.Hq; h0 += ILP * groups) {
    if (h0 > 0) load(h0);
#pragma unroll
    for (int i = 0; i < ILP; ++i) {
      const int h = h0 + i * groups + grp;
      float x[8];
      unpack4(raw[i].a, x);
      unpack4(raw[i].b, x + 4);
      norm_rotate<TPR, HALF>(x, norm, gamma, p, cs, a.eps);
      if (h < a.Hq) {
        *reinterpret_cast<uint2*>(dst + h * D + p.oa) = pack4(x);
        *reinterpret_cast<uint2*>(dst + h * D + p.ob) = pack4(x + 4);
      }
    }
  }
}

// Blocks [0, 2 Hkv items): cache blocks; the rest: one query block per token.
template <int D, int PASSES, bool HALF, int THREADS>
__global__ void __launch_bounds__(THREADS) kv_append_kernel(KaArgs a) {
  pdl_enter();
  const int n_cache = 2 * a.c.n_kv_heads * a.items;
  int i = blockIdx.x;
  if (i < n_cache) {
    const bool is_v = i & 1;
    i >>= 1;
    const int item = i / a.c.n_kv_heads, head = i - item * a.c.n_kv_heads;
    if (is_v) append_block<D, PASSES, HALF, true>(a, item, head);
    else append_block<D, PASSES, HALF, false>(a, item, head);
  } else {
    query_block<D, HALF>(a, i - n_cache);
  }
}

template <int D, int PASSES, int THREADS>
cudaError_t launch(const KaArgs& a, int threads, cudaStream_t s) {
  const int64_t blocks = int64_t(2) * a.c.n_kv_heads * a.items + (a.q ? a.T : 0);
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  count_launches(1);
  const unsigned n = static_cast<unsigned>(blocks);
  return a.half ? launch_pdl(kv_append_kernel<D, PASSES, true, THREADS>, n, threads, 0, s, a)
                : launch_pdl(kv_append_kernel<D, PASSES, false, THREADS>, n, threads, 0, s, a);
}

template <int D>
cudaError_t launch_d(const KaArgs& a, cudaStream_t s) {
  // rows of eight elements a thread, at most four a thread
  const int work = a.c.page_size * (D / 8), threads = std::max(kQueryThreads, work / 4);
  if (work <= kQueryThreads) return launch<D, 1, kQueryThreads>(a, kQueryThreads, s);
  if (work <= 2 * kQueryThreads) return launch<D, 2, kQueryThreads>(a, kQueryThreads, s);
  if (threads <= 256) return launch<D, 4, 256>(a, threads, s);
  return launch<D, 4, D == 256 ? 1024 : 512>(a, threads, s);
}

bool stride_ok(int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0; }

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_kv_append(const moe_kv_append_config_t* cfg, const moe_kv_cache_t* cache, const void* q,
                                      const void* k, const void* v, const float* gamma_q, const float* gamma_k,
                                      const float* cos_sin, const int32_t* positions, const int32_t* cu,
                                      const int32_t* kv_len, void* q_out, moe_stream_t stream) {
  using namespace moe;
  if (!cfg || !kv_cache_shape_ok(cache)) return MOE_ERR_INVALID_ARG;
  const int D = cache->head_dim;
  if (cfg->T < 0 || cfg->T > (1 << 28) || cfg->batch < 1 || cfg->batch > kMaxBatch) return MOE_ERR_INVALID_ARG;
  if (cfg->rot_dim < 0 || cfg->rot_dim > D || cfg->rot_dim % 8 != 0) return MOE_ERR_INVALID_ARG;
  if (cfg->rope_layout != MOE_ROPE_HALF && cfg->rope_layout != MOE_ROPE_INTERLEAVED) return MOE_ERR_INVALID_ARG;
  if (cfg->rot_dim > 0 && cfg->n_pos < 1) return MOE_ERR_INVALID_ARG;
  if (!(cfg->eps > 0.f) || !std::isfinite(cfg->eps)) return MOE_ERR_INVALID_ARG;
  const int64_t kv_width = static_cast<int64_t>(cache->n_kv_heads) * D;
  if (!stride_ok(cfg->k_stride, kv_width) || !stride_ok(cfg->v_stride, kv_width)) return MOE_ERR_INVALID_ARG;
  if (q) {
    const int64_t q_width = static_cast<int64_t>(cfg->n_q_heads) * D;
    if (cfg->n_q_heads < 1 || cfg->n_q_heads > 4096 || !stride_ok(cfg->q_stride, q_width) ||
        !stride_ok(cfg->q_out_stride, q_width))
      return MOE_ERR_INVALID_ARG;
    if (!q_out || !aligned_to(q, 16) || !aligned_to(q_out, 16) || (gamma_q && !aligned_to(gamma_q, 16)))
      return MOE_ERR_INVALID_ARG;
  }
  if (cfg->T == 0) return MOE_OK;
  if (!k || !v || !cu || !kv_len || !kv_cache_pointers_ok(cache)) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(k, 16) || !aligned_to(v, 16) || !aligned_to(cu, 4) || !aligned_to(kv_len, 4) ||
      (gamma_k && !aligned_to(gamma_k, 16)) || (positions && !aligned_to(positions, 4)))
    return MOE_ERR_INVALID_ARG;
  if (cfg->rot_dim > 0 && (!cos_sin || !aligned_to(cos_sin, 16))) return MOE_ERR_INVALID_ARG;
  unsigned* status = nullptr;
  int sms = 0;
  const moe_status_t st = current_device(&status, &sms);
  if (st != MOE_OK) return st;
  KaArgs a;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.gamma_q = gamma_q;
  a.gamma_k = gamma_k;
  a.cos_sin = reinterpret_cast<const float2*>(cos_sin);
  a.positions = positions;
  a.cu = cu;
  a.kv_len = kv_len;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.c = *cache;
  a.status = status;
  a.qs = cfg->q_stride;
  a.ks = cfg->k_stride;
  a.vs = cfg->v_stride;
  a.qos = cfg->q_out_stride;
  a.T = cfg->T;
  a.B = cfg->batch;
  a.Hq = cfg->n_q_heads;
  a.rot = cfg->rot_dim;
  a.n_pos = cfg->n_pos;
  a.items = cfg->T / cache->page_size + 2 * cfg->batch;
  a.eps = cfg->eps;
  a.half = cfg->rope_layout == MOE_ROPE_HALF;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  switch (D) {
    case 64: err = launch_d<64>(a, s); break;
    case 128: err = launch_d<128>(a, s); break;
    default: err = launch_d<256>(a, s); break;
  }
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
