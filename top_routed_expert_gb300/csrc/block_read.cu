// Rows of the paged 4-bit cache as bf16 or fp32 (include/block_kv.h,
// moe_blockkv_read).
//
// A block owns 16 slots of a page, keys and values of all heads: one look-up of
// request and page, then a thread takes eight codes (four bytes) and their
// scale at a time and writes eight elements, so that neighbouring threads write
// neighbouring 16 bytes.  Bound by memory: 0.56 bytes read and 2 (or 4) written
// an element.  Request b's blocks start at cu[b]/16 + 2b, as in kv_append.cu.
#include "block_kv.cuh"
#include "paged_attn.cuh"

namespace moe {
namespace {

constexpr int kSlots = 16, kThreads = 256, kAtOnce = 4;

struct BrArgs {
  moe_blockkv_cache_t c;
  const int32_t* cu;
  const int32_t* kv_len;
  void* k_out;
  void* v_out;
  unsigned* status;
  int64_t ks, vs;
  int T, B;
};

__device__ __forceinline__ float2 halves(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

template <int D, bool F32>
__global__ void __launch_bounds__(kThreads) blockkv_read_kernel(BrArgs a) {
  constexpr int WORDS = D / 8;   // of a row
  pdl_enter();
  const int item = blockIdx.x, ps = a.c.page_size, ps_log = 31 - __clz(ps);
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
  const int page = base >> ps_log;
  int pid = -1;
  if (page < a.c.max_pages) pid = a.c.page_table[static_cast<int64_t>(b) * a.c.max_pages + page];
  if (pid < 0 || pid >= a.c.n_pages) {
    if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  const int cols = a.c.n_kv_heads * WORDS, n = tokens * cols;   // words of keys; as many of values
  const int64_t row0 = r.row0 + (first - r.start), slot0 = first & (ps - 1);
  auto copy = [&](const void* codes_at, const void* scales_at, float g, void* out, int64_t stride) {
    const uint8_t* codes = static_cast<const uint8_t*>(codes_at) + pid * a.c.page_stride + slot0 * a.c.token_stride;
    const uint8_t* scales =
        static_cast<const uint8_t*>(scales_at) + pid * a.c.scale_page_stride + slot0 * a.c.scale_token_stride;
#pragma unroll 1
    for (int i0 = threadIdx.x; i0 < n; i0 += kAtOnce * kThreads) {
      uint32_t w[kAtOnce], sc[kAtOnce];
      int64_t to[kAtOnce];
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        const int i = i0 + u * kThreads;
        to[u] = -1;
        if (i >= n) continue;
        const int token = i / cols, col = i - token * cols, head = col / WORDS, word = col % WORDS;
        w[u] = __ldg(reinterpret_cast<const uint32_t*>(codes + token * a.c.token_stride + head * a.c.head_stride + word * 4));
        sc[u] = __ldg(scales + token * a.c.scale_token_stride + head * a.c.scale_head_stride + word / 2);
        to[u] = (row0 + token) * stride + static_cast<int64_t>(col) * 8;
      }
#pragma unroll
      for (int u = 0; u < kAtOnce; ++u) {
        if (to[u] < 0) continue;
        uint32_t x[4];
        f16x2_of_e2m1(w[u], x);
        const float f = e4m3_to_float(static_cast<uint8_t>(sc[u])) * g;
        float2 y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 h = halves(x[e]);
          y[e] = make_float2(h.x * f, h.y * f);
        }
        if (F32) {
          float4* dst = reinterpret_cast<float4*>(static_cast<float*>(out) + to[u]);
          dst[0] = make_float4(y[0].x, y[0].y, y[1].x, y[1].y);
          dst[1] = make_float4(y[2].x, y[2].y, y[3].x, y[3].y);
        } else {
          uint32_t p[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 z = __floats2bfloat162_rn(y[e].x, y[e].y);
            p[e] = *reinterpret_cast<const uint32_t*>(&z);
          }
          *reinterpret_cast<uint4*>(static_cast<uint16_t*>(out) + to[u]) = make_uint4(p[0], p[1], p[2], p[3]);
        }
      }
    }
  };
  if (a.k_out) copy(a.c.k, a.c.k_scale, a.c.k_gscale, a.k_out, a.ks);
  if (a.v_out) copy(a.c.v, a.c.v_scale, a.c.v_gscale, a.v_out, a.vs);
}

template <int D>
cudaError_t launch(const BrArgs& a, bool f32, cudaStream_t s) {
  count_launches(1);
  return launch_pdl(f32 ? blockkv_read_kernel<D, true> : blockkv_read_kernel<D, false>, a.T / kSlots + 2 * a.B, kThreads, 0,
                    s, a);
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_blockkv_read(const moe_blockkv_read_config_t* cfg, const moe_blockkv_cache_t* cache,
                                         const int32_t* cu, const int32_t* kv_len, void* k_out, void* v_out,
                                         moe_stream_t stream) {
  using namespace moe;
  if (!cfg || !blockkv_shape_ok(cache)) return MOE_ERR_INVALID_ARG;
  if (cfg->T < 0 || cfg->T > (1 << 28) || cfg->batch < 1 || cfg->batch > kMaxBatch) return MOE_ERR_INVALID_ARG;
  if (cfg->out_dtype != MOE_BF16 && cfg->out_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  const int64_t width = static_cast<int64_t>(cache->n_kv_heads) * cache->head_dim;
  if (k_out && (cfg->k_stride < width || cfg->k_stride % 8 != 0 || !aligned_to(k_out, 16))) return MOE_ERR_INVALID_ARG;
  if (v_out && (cfg->v_stride < width || cfg->v_stride % 8 != 0 || !aligned_to(v_out, 16))) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0 || (!k_out && !v_out)) return MOE_OK;
  if (!cu || !kv_len || !aligned_to(cu, 4) || !aligned_to(kv_len, 4) || !blockkv_pointers_ok(cache))
    return MOE_ERR_INVALID_ARG;
  unsigned* status = nullptr;
  int sms = 0;
  const moe_status_t st = current_device(&status, &sms);
  if (st != MOE_OK) return st;
  BrArgs a;
  a.c = *cache;
  a.cu = cu;
  a.kv_len = kv_len;
  a.k_out = k_out;
  a.v_out = v_out;
  a.status = status;
  a.ks = cfg->k_stride;
  a.vs = cfg->v_stride;
  a.T = cfg->T;
  a.B = cfg->batch;
  const bool f32 = cfg->out_dtype == MOE_F32;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  switch (cache->head_dim) {
    case 64: err = launch<64>(a, f32, s); break;
    case 128: err = launch<128>(a, f32, s); break;
    default: err = launch<256>(a, f32, s); break;
  }
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
