// Rows of the paged 4-bit cache as bf16 or fp32 (include/block_kv.h,
// moe_blockkv_read).
//
// A block owns 16 slots of a page, keys and values of all heads: one look-up of
// request and page, then a thread takes the codes of 16 elements (eight bytes)
// and their scale at a time and writes 32 bytes (fp32: 64), so that neighbouring
// threads write beside each other; what it reads of keys and values is on its way
// together.  Bound by memory: 0.56 bytes read and 2 (or 4) written an element; 64
// requests of up to 3712 tokens, 4 heads of 128, 312 MB in 49.5 us = 6.3 TB/s (16 bytes an
// access, keys before values: 72 us).
#include "block_kv.cuh"
#include "paged_attn.cuh"

namespace moe {
namespace {

constexpr int kThreads = 256, kAtOnce = 4;   // blocks of elements that a thread has under way

struct BrArgs {
  moe_blockkv_cache_t c;
  const int32_t* cu;
  const int32_t* kv_len;
  void* k_out;
  void* v_out;
  unsigned* status;
  int64_t ks, vs;
  uint32_t per_row;   // 2^32 / blocks of a token's keys, rounded up
  int T, B;
};

__device__ __forceinline__ float2 halves(uint32_t x) { return __half22float2(*reinterpret_cast<const __half2*>(&x)); }

__device__ __forceinline__ void store32(void* p, const uint32_t (&v)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]),
               "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}

// 32 bytes: in one access where the rows are aligned to that.
template <bool WIDE> __device__ __forceinline__ void put(void* p, const uint32_t (&v)[8]) {
  if (WIDE) {
    store32(p, v);
  } else {
    static_cast<uint4*>(p)[0] = make_uint4(v[0], v[1], v[2], v[3]);
    static_cast<uint4*>(p)[1] = make_uint4(v[4], v[5], v[6], v[7]);
  }
}

template <int D, bool F32, bool WIDE>
__global__ void __launch_bounds__(kThreads) blockkv_read_kernel(BrArgs a) {
  constexpr int BLOCKS = D / 16;   // of a row
  pdl_enter();
  const int items = a.T / kSlots + 2 * a.B;
  if (static_cast<int>(blockIdx.x) >= items) {   // the last blocks
    check_offsets(a.cu, a.B, a.T, blockIdx.x - items, a.status);
    return;
  }
  const int item = blockIdx.x, ps = a.c.page_size, ps_log = 31 - __clz(ps);
  const int b = warp_find_request(a.cu, a.B, item, 1, kSlots, 2);
  const Request r = load_request(a.cu, a.kv_len, b, a.T);
  if (!r.ok || r.start < 0) {
    if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  const int group = slot_group(r, b, item);
  if (group < 0) return;
  const int page = group >> (ps_log - 4);   // of page_size / 16 groups
  int pid = -1;
  if (page < a.c.max_pages) pid = a.c.page_table[static_cast<int64_t>(b) * a.c.max_pages + page];
  if (pid < 0 || pid >= a.c.n_pages) {
    if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  const int base = group * kSlots, first = max(base, r.start), tokens = min(base + kSlots, r.end) - first;
  const int cols = a.c.n_kv_heads * BLOCKS, n = tokens * cols;   // blocks of keys; as many of values
  const int64_t row0 = r.row0 + (first - r.start), slot0 = first & (ps - 1);
  const int64_t codes0 = pid * a.c.page_stride + slot0 * a.c.token_stride;
  const int64_t scales0 = pid * a.c.scale_page_stride + slot0 * a.c.scale_token_stride;
  const int lo = a.k_out ? 0 : n, hi = a.v_out ? 2 * n : n;
#pragma unroll 1
  for (int i0 = lo + threadIdx.x; i0 < hi; i0 += kAtOnce * kThreads) {
    uint2 w[kAtOnce];
    uint32_t sc[kAtOnce];
    int64_t to[kAtOnce];
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      const int i = i0 + u * kThreads;
      to[u] = -1;
      if (i >= hi) continue;
      const bool value = i >= n;
      const int j = value ? i - n : i;
      const int token = __umulhi(j, a.per_row), col = j - token * cols, head = col / BLOCKS, block = col % BLOCKS;
      const uint8_t* codes = static_cast<const uint8_t*>(value ? a.c.v : a.c.k) + codes0;
      const uint8_t* scales = static_cast<const uint8_t*>(value ? a.c.v_scale : a.c.k_scale) + scales0;
      w[u] = __ldg(reinterpret_cast<const uint2*>(codes + token * a.c.token_stride + head * a.c.head_stride + block * 8));
      sc[u] = __ldg(scales + token * a.c.scale_token_stride + head * a.c.scale_head_stride + block);
      to[u] = (row0 + token) * (value ? a.vs : a.ks) + static_cast<int64_t>(col) * 16;
    }
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
      if (to[u] < 0) continue;
      const bool value = i0 + u * kThreads >= n;
      void* out = value ? a.v_out : a.k_out;
      const float f = e4m3_to_float(static_cast<uint8_t>(sc[u])) * (value ? a.c.v_gscale : a.c.k_gscale);
      uint32_t x[8];
      {
        uint32_t y[4];
        f16x2_of_e2m1(w[u].x, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[e] = y[e];
        f16x2_of_e2m1(w[u].y, y);
#pragma unroll
        for (int e = 0; e < 4; ++e) x[4 + e] = y[e];
      }
      if (F32) {
        float* dst = static_cast<float*>(out) + to[u];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 y = halves(x[4 * h + e]);
            p[2 * e] = __float_as_uint(y.x * f);
            p[2 * e + 1] = __float_as_uint(y.y * f);
          }
          put<WIDE>(dst + 8 * h, p);
        }
      } else {
        uint32_t p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float2 y = halves(x[e]);
          const __nv_bfloat162 z = __floats2bfloat162_rn(y.x * f, y.y * f);
          p[e] = *reinterpret_cast<const uint32_t*>(&z);
        }
        put<WIDE>(static_cast<uint16_t*>(out) + to[u], p);
      }
    }
  }
}

template <int D>
cudaError_t launch(BrArgs a, bool f32, cudaStream_t s) {
  const uint32_t cols = a.c.n_kv_heads * (D / 16);
  a.per_row = static_cast<uint32_t>(((uint64_t(1) << 32) + cols - 1) / cols);   // exact below 16 cols
  // 32-byte accesses need rows at 32 bytes
  const int per32 = f32 ? 8 : 16;
  const bool wide = (!a.k_out || (aligned_to(a.k_out, 32) && a.ks % per32 == 0)) &&
                    (!a.v_out || (aligned_to(a.v_out, 32) && a.vs % per32 == 0));
  count_launches(1);
  auto go = [&](auto kernel) { return launch_pdl(kernel, a.T / kSlots + 2 * a.B + ceil_div(a.B, kThreads), kThreads, 0, s, a); };
  if (f32) return wide ? go(blockkv_read_kernel<D, true, true>) : go(blockkv_read_kernel<D, true, false>);
  return wide ? go(blockkv_read_kernel<D, false, true>) : go(blockkv_read_kernel<D, false, false>);
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_blockkv_read(const moe_blockkv_read_config_t* cfg, const moe_blockkv_cache_t* cache,
                                         const int32_t* cu, const int32_t* kv_len, void* k_out, void* v_out,
                                         moe_stream_t stream) {
  using namespace moe;
  if (!cfg || !blockkv_shape_ok(cache)) return MOE_ERR_INVALID_ARG;
  if (cfg->T < 0 || cfg->T > (1 << 28) || cfg->batch < 1 || cfg->batch > kMaxBlockBatch) return MOE_ERR_INVALID_ARG;
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
