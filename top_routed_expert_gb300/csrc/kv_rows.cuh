// What the appends to the paged caches share (kv_append.cu, block_append.cu):
// the call's rows, their norm and rotation, and the blocks that turn the
// queries.
#pragma once

#include "paged_kv.cuh"

namespace moe {

constexpr int kQueryThreads = 128;

struct RowArgs {
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
  unsigned* status;
  int64_t qs, ks, vs, qos;
  int T, B, Hq, rot, n_pos;
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

// (Plain loads: the queries may be turned in place.  The interleaved layout's
// eight elements are one piece.)
template <bool HALF>
__device__ __forceinline__ Raw load_raw(const uint16_t* row, const Place& p) {
  if (HALF) return Raw{*reinterpret_cast<const uint2*>(row + p.oa), *reinterpret_cast<const uint2*>(row + p.ob)};
  const uint4 w = *reinterpret_cast<const uint4*>(row + p.oa);
  return Raw{make_uint2(w.x, w.y), make_uint2(w.z, w.w)};
}
template <bool HALF>
__device__ __forceinline__ void store_row(uint16_t* row, const Place& p, const float (&x)[8]) {
  const uint2 a = pack4(x), b = pack4(x + 4);
  if (HALF) {
    *reinterpret_cast<uint2*>(row + p.oa) = a;
    *reinterpret_cast<uint2*>(row + p.ob) = b;
  } else {
    *reinterpret_cast<uint4*>(row + p.oa) = make_uint4(a.x, a.y, b.x, b.y);
  }
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

// The larger of two sizes, NaN if either is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// Row of the frequency table of a token, or -1.
__device__ __forceinline__ int table_row(const RowArgs& a, int t, int pos) {
  const int p = a.positions ? a.positions[t] : pos;
  return (p >= 0 && p < a.n_pos) ? p : -1;
}

// Largest finite size of eight elements; bad: one of them is not finite.
__device__ __forceinline__ float largest(const float (&x)[8], bool& bad) {
  float top = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max_or_nan(top, fabsf(x[e]));
  if (top < INFINITY) return top;
  bad = true;
  top = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (fabsf(x[e]) < INFINITY) top = fmaxf(top, fabsf(x[e]));
  return top;
}

__device__ __forceinline__ void copy_async(void* to, const void* from, int bytes) {
  const uint32_t at = static_cast<uint32_t>(__cvta_generic_to_shared(to));
  if (bytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(at), "l"(from) : "memory");
}

// All query heads of TOKENS tokens from t on.  The first rows are on their way
// while the tokens' requests, positions and angles are looked up.
template <int D, bool HALF, int TOKENS>
__device__ __forceinline__ void query_block(const RowArgs& a, int t) {
  constexpr int TPR = D / 8, HEADS = 4 / TOKENS;   // heads that a thread has under way for each token
  const int lr = threadIdx.x % TPR, grp = threadIdx.x / TPR, groups = blockDim.x / TPR;
  const Place p = place_of<HALF>(lr, a.rot);
  Raw raw[TOKENS][HEADS];
  auto load = [&](int h0) {
#pragma unroll
    for (int n = 0; n < TOKENS; ++n)
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        const int h = h0 + i * groups + grp;
        raw[n][i] = Raw{make_uint2(0, 0), make_uint2(0, 0)};
        if (h < a.Hq && t + n < a.T) raw[n][i] = load_raw<HALF>(a.q + (t + n) * a.qs + h * D, p);
      }
  };
  load(0);
  const bool norm = a.gamma_q;
  Gamma gamma = {};
  if (norm) gamma = load_gamma(a.gamma_q, p);
  float2 cs[TOKENS][4] = {};
  bool live[TOKENS];
  int b = warp_find_request(a.cu, a.B, t, 1, 1, 0);
  Request r = load_request(a.cu, a.kv_len, b, a.T);
#pragma unroll
  for (int n = 0; n < TOKENS; ++n) {
    while (TOKENS > 1 && r.ok && t + n >= r.row0 + r.n && b + 1 < a.B) r = load_request(a.cu, a.kv_len, ++b, a.T);
    // not live: recorded by the cache blocks, or no request's row
    live[n] = r.ok && r.start >= 0 && t + n >= r.row0 && t + n < r.row0 + r.n;
    if (live[n] && a.rot > 0) {
      const int f = table_row(a, t + n, r.start + (t + n - r.row0));
      live[n] = f >= 0;
      if (f < 0 && threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      if (f >= 0 && p.rotates) load_cs<HALF>(a.cos_sin + static_cast<int64_t>(f) * (a.rot / 2), p, cs[n]);
    }
  }
  // every thread makes the same number of rounds: the norm's shuffles need all lanes
  for (int h0 = 0; h0 < a.Hq; h0 += HEADS * groups) {
    if (h0 > 0) load(h0);
#pragma unroll
    for (int n = 0; n < TOKENS; ++n)
#pragma unroll
      for (int i = 0; i < HEADS; ++i) {
        const int h = h0 + i * groups + grp;
        float x[8];
        unpack4(raw[n][i].a, x);
        unpack4(raw[n][i].b, x + 4);
        norm_rotate<TPR, HALF>(x, norm, gamma, p, cs[n], a.eps);
        if (h < a.Hq && live[n]) {
          uint16_t* dst = a.q_out + (t + n) * a.qos + h * D;
          store_row<HALF>(dst, p, x);
        }
      }
  }
}

// Tokens of a query block: four heads a thread in all.
template <int D> __host__ __device__ __forceinline__ int query_tokens(int Hq, int threads) {
  const int groups = threads / (D / 8);
  return Hq <= groups ? 4 : Hq <= 2 * groups ? 2 : 1;
}

// What a call has to fulfil before anything is launched: the configuration and
// q's arguments, then (T > 0) the pointers.
inline bool append_config_ok(const moe_kv_append_config_t* cfg, int max_batch, int heads, int D, const void* q,
                             const float* gamma_q, const void* q_out) {
  auto stride_ok = [](int64_t stride, int64_t width) { return stride >= width && stride % 8 == 0; };
  if (cfg->T < 0 || cfg->T > (1 << 28) || cfg->batch < 1 || cfg->batch > max_batch) return false;
  if (cfg->rot_dim < 0 || cfg->rot_dim > D || cfg->rot_dim % 8 != 0) return false;
  if (cfg->rope_layout != MOE_ROPE_HALF && cfg->rope_layout != MOE_ROPE_INTERLEAVED) return false;
  if (cfg->rot_dim > 0 && cfg->n_pos < 1) return false;
  if (!(cfg->eps > 0.f) || !std::isfinite(cfg->eps)) return false;
  const int64_t kv_width = static_cast<int64_t>(heads) * D;
  if (!stride_ok(cfg->k_stride, kv_width) || !stride_ok(cfg->v_stride, kv_width)) return false;
  if (!q) return true;
  const int64_t q_width = static_cast<int64_t>(cfg->n_q_heads) * D;
  return cfg->n_q_heads >= 1 && cfg->n_q_heads <= 4096 && stride_ok(cfg->q_stride, q_width) &&
         stride_ok(cfg->q_out_stride, q_width) && q_out && aligned_to(q, 16) && aligned_to(q_out, 16) &&
         (!gamma_q || aligned_to(gamma_q, 16));
}

inline bool append_pointers_ok(const moe_kv_append_config_t* cfg, const void* k, const void* v, const float* gamma_k,
                               const float* cos_sin, const int32_t* positions, const int32_t* cu, const int32_t* kv_len) {
  return k && v && cu && kv_len && aligned_to(k, 16) && aligned_to(v, 16) && aligned_to(cu, 4) && aligned_to(kv_len, 4) &&
         (!gamma_k || aligned_to(gamma_k, 16)) && (!positions || aligned_to(positions, 4)) &&
         (cfg->rot_dim == 0 || (cos_sin && aligned_to(cos_sin, 16)));
}

inline void fill_rows(RowArgs& a, const moe_kv_append_config_t* cfg, const void* q, const void* k, const void* v,
                      const float* gamma_q, const float* gamma_k, const float* cos_sin, const int32_t* positions,
                      const int32_t* cu, const int32_t* kv_len, void* q_out, unsigned* status) {
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
  a.eps = cfg->eps;
  a.half = cfg->rope_layout == MOE_ROPE_HALF;
}

}  // namespace moe
