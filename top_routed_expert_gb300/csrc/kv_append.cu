// Append to the paged 8-bit cache (include/paged_kv.h, moe_kv_append): QK
// norm, rotation, page scale and E4M3 codes in one launch.
//
// Two kinds of blocks.  A cache block owns one page of one request for one
// head or several, keys and values: a head's new tokens of the page all pass
// through its registers, so the page's scales are one block reduction and every
// code is written once.  A query block owns a token, or a few where a token has
// few heads, and turns all query heads.
//
// With y = norm(x) rotated and s the smallest power of two that holds the page's
// largest |y| in E4M3's 448, a code is y / s rounded once; everything before it
// is fp32.  A page that already holds tokens keeps the larger of its scales, and
// its old codes are halved as often as that grew.
//
// Bound by memory, and by how many bytes the look-ups before them let be on
// their way: q is read and written once (bf16), k and v are read, their codes
// written.  Measured: 32 x 256 tokens of 32 + 4 heads of 128, norm and rotation,
// 164 MB in 32.4 us = 5.1 TB/s; ragged prompts up to 1999 tokens of 16 + 16 heads
// of 64, 238 MB in 54 us = 4.4 TB/s; 64 single tokens 4.0 us in a graph, a launch and
// four dependent loads.
//
// Which pages a ragged batch touches is known on the device only.  A request
// of n new tokens touches at most n/page + 2 pages, so request b's blocks
// start at cu[b]/page + 2b, the grid has T/page + 2B of them, and a block
// finds its request by a search over cu; the few blocks too many leave.
#include "kv_rows.cuh"

namespace moe {
namespace {

constexpr float kMinScale = 9.094947017729282e-13f;   // 2^-40
constexpr int kMaxHeads = 8;   // of a cache block

struct KaArgs : RowArgs {
  moe_kv_cache_t c;
  int work;                 // blocks but those that check offsets
  int items;                // pages that the requests can touch
  int heads, head_blocks;   // heads of a cache block; its blocks for a page
};

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

// The smallest power of two s >= 2^-40 with amax <= 448 s = 1.75 * 2^8 s.
__device__ __forceinline__ float scale_for(float amax) {
  if (!(amax > 448.f * kMinScale)) return kMinScale;
  const uint32_t u = __float_as_uint(amax);
  const uint32_t e = (u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1u : 0u);
  return __uint_as_float(e << 23);
}

// The new codes of a thread's eight elements, or the old ones rounded to a scale
// that has grown.
template <bool HALF>
__device__ __forceinline__ void store_codes(uint8_t* row, const Place& p, const float (&x)[8], float inv) {
  const uint32_t lo = codes4(x, inv), hi = codes4(x + 4, inv);
  if (!HALF || p.ob == p.oa + 4) {
    *reinterpret_cast<uint2*>(row + p.oa) = make_uint2(lo, hi);
  } else {
    *reinterpret_cast<uint32_t*>(row + p.oa) = lo;
    *reinterpret_cast<uint32_t*>(row + p.ob) = hi;
  }
}
__device__ __forceinline__ void rescale_codes(uint8_t* row, const Place& p, float f) {
  uint32_t* wa = reinterpret_cast<uint32_t*>(row + p.oa);
  uint32_t* wb = reinterpret_cast<uint32_t*>(row + p.ob);
  *wa = rescale4(*wa, f);
  *wb = rescale4(*wb, f);
}

// Heads that a cache block has under way at a time: two where they fit.
__host__ __device__ constexpr int append_stages(int passes, int threads) { return passes * threads <= 512 ? 2 : 1; }
constexpr size_t append_smem(int passes, int threads) {
  return static_cast<size_t>(append_stages(passes, threads)) * passes * threads * 2 * sizeof(uint4);
}

// One page, heads [head0, head1).  PASSES rows per thread group; the block
// covers the page's slots in PASSES rounds of blockDim / TPR rows.  A thread
// fetches its own elements of the next head (asynchronously, so they cost no
// registers and no barrier) while it works on this one.
template <int D, int PASSES, bool HALF, int THREADS>
__device__ __forceinline__ void append_block(const KaArgs& a, int item, int head0, int head1) {
  constexpr int TPR = D / 8, STAGES = append_stages(PASSES, THREADS);
  __shared__ float s_amax[2][2][32];
  extern __shared__ __align__(16) uint4 s_rows[];   // [STAGES][PASSES][key, value][THREADS]
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
  if (at < 0 || page > (r.end - 1) >> ps_log) return;   // one block too many, or before the first request
  if (page >= a.c.max_pages) {   // past the page table, and maybe past what positions can count (a length may be 2^31 - 1)
    if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    return;
  }
  const int base = page << ps_log;
  const int lr = threadIdx.x % TPR, grp = threadIdx.x / TPR, rows = blockDim.x / TPR;
  const bool norm = a.gamma_k;
  const Place p = place_of<HALF>(lr, a.rot), pv = place_of<false>(lr, 0);
  const int t0 = r.row0 - r.start;         // row of position 0
  bool take[PASSES];
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int j = base + i * rows + grp;
    take[i] = j >= r.start && j < r.end && j < base + ps;
  }
  auto slot = [&](int head, int i, int kv) {
    return s_rows + (((head - head0) % STAGES * PASSES + i) * 2 + kv) * THREADS + threadIdx.x;
  };
  auto fetch = [&](int head) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      if (!take[i]) continue;
      const int64_t row = t0 + base + i * rows + grp;
      const uint16_t* k = a.k + row * a.ks + static_cast<int64_t>(head) * D;
      uint4* to = slot(head, i, 0);
      if (HALF) {
        copy_async(to, k + p.oa, 8);
        copy_async(reinterpret_cast<uint2*>(to) + 1, k + p.ob, 8);
      } else {
        copy_async(to, k + p.oa, 16);
      }
      copy_async(slot(head, i, 1), a.v + row * a.vs + static_cast<int64_t>(head) * D + pv.oa, 16);
    }
  };
  int next = head0;   // the next head to fetch
  auto fetch_next = [&] {
    if (next < head1) fetch(next);
    ++next;
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  fetch_next();
  if (STAGES > 1) fetch_next();
  const int pid = a.c.page_table[static_cast<int64_t>(b) * a.c.max_pages + page];
  Gamma gamma = {};
  if (norm) gamma = load_gamma(a.gamma_k, p);
  float2 cs[PASSES][4];
  bool outside = false;
  if (a.rot > 0) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int j = base + i * rows + grp;
      if (!take[i]) continue;
      const int f = table_row(a, t0 + j, j);
      if (f < 0) outside = true;
      if (f < 0) take[i] = false;   // what is on its way goes unread
      else if (p.rotates) load_cs<HALF>(a.cos_sin + static_cast<int64_t>(f) * (a.rot / 2), p, cs[i]);
    }
  }
  if (outside && lr == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
  if (pid < 0 || pid >= a.c.n_pages) {
    if (threadIdx.x == 0) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  const bool had = r.start > base;
#pragma unroll 1
  for (int head = head0; head < head1; ++head) {
    const int64_t scale_at = static_cast<int64_t>(pid) * a.c.n_kv_heads + head;
    const float old_k = had ? a.c.k_scale[scale_at] : 0.f, old_v = had ? a.c.v_scale[scale_at] : 0.f;
    asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
    float x[PASSES][8], top_k = 0.f;
    uint4 rv[PASSES];
    uint32_t bits_v = 0;   // the largest size among the values as bf16 bits
    bool bad = false;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const uint4 zero = make_uint4(0, 0, 0, 0), rk = take[i] ? *slot(head, i, 0) : zero;
      rv[i] = take[i] ? *slot(head, i, 1) : zero;
      unpack4(make_uint2(rk.x, rk.y), x[i]);
      unpack4(make_uint2(rk.z, rk.w), x[i] + 4);
    }
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      norm_rotate<TPR, HALF>(x[i], norm, gamma, p, cs[i], a.eps);
      if (take[i]) top_k = fmaxf(top_k, largest(x[i], bad));
      const uint32_t w = __vmaxu2(__vmaxu2(rv[i].x & 0x7fff7fffu, rv[i].y & 0x7fff7fffu),
                                  __vmaxu2(rv[i].z & 0x7fff7fffu, rv[i].w & 0x7fff7fffu));
      bits_v = __vmaxu2(bits_v, w);
    }
    bits_v = max(bits_v & 0xffffu, bits_v >> 16);
    float top_v = __uint_as_float(bits_v << 16);
    if (bits_v >= 0x7f80u) {   // an infinity or a NaN among them
      top_v = 0.f;
#pragma unroll
      for (int i = 0; i < PASSES; ++i) {
        float y[8];
        unpack4(make_uint2(rv[i].x, rv[i].y), y);
        unpack4(make_uint2(rv[i].z, rv[i].w), y + 4);
        top_v = fmaxf(top_v, largest(y, bad));
      }
    }
    if (bad) set_status(a.status, MOE_ERR_DEVICE_NONFINITE);
    // sizes order like their bits
    top_k = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top_k)));
    top_v = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(top_v)));
    float(&amax)[2][32] = s_amax[head & 1];   // in turn: one barrier for a head
    if ((threadIdx.x & 31) == 0) {
      amax[0][threadIdx.x >> 5] = top_k;
      amax[1][threadIdx.x >> 5] = top_v;
    }
    __syncthreads();   // also: every thread has read the old scales
    fetch_next();      // over what was read above
    for (int w = 0; w < static_cast<int>(blockDim.x / 32); ++w) {
      top_k = fmaxf(top_k, amax[0][w]);
      top_v = fmaxf(top_v, amax[1][w]);
    }
    const float sk = fmaxf(scale_for(top_k), old_k), sv = fmaxf(scale_for(top_v), old_v);
    if (threadIdx.x == 0) {
      a.c.k_scale[scale_at] = sk;
      a.c.v_scale[scale_at] = sv;
    }
    const float inv_k = 1.0f / sk, inv_v = 1.0f / sv;
    const int64_t page_at = pid * a.c.page_stride + head * a.c.head_stride;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      const int j = base + i * rows + grp;
      const int64_t row = page_at + (j - base) * a.c.token_stride;
      uint8_t* kc = static_cast<uint8_t*>(a.c.k) + row;
      uint8_t* vc = static_cast<uint8_t*>(a.c.v) + row;
      if (take[i]) {
        store_codes<HALF>(kc, p, x[i], inv_k);
        float y[8];
        unpack4(make_uint2(rv[i].x, rv[i].y), y);
        unpack4(make_uint2(rv[i].z, rv[i].w), y + 4);
        store_codes<false>(vc, pv, y, inv_v);
      } else if (had && j < r.start) {
        if (sk > old_k) rescale_codes(kc, p, old_k * inv_k);
        if (sv > old_v) rescale_codes(vc, pv, old_v * inv_v);
      }
    }
  }
}

// Blocks on an SM that the registers are cut for: more of them hide more of the
// look-ups' latency (before a block took several heads: prefill of 32 x 256
// tokens, two rows a thread, 37.4 us with the compiler's choice of 5, 32.6 us
// with 7; ragged prompts, four rows a thread, 67.6 and 58.7 us).  With four rows a
// thread that costs spills: 96 to 104 bytes of 80 registers (their angles, 32 of
// them, are held over all heads), 328 to 368 of 64 where D = 256 and pages of 128
// tokens need 1024 threads.
template <int PASSES, int THREADS> constexpr int blocks_on_sm() {
  return THREADS == 128 ? (PASSES < 4 ? 7 : 6) : THREADS == 256 ? 3 : 1;
}

// Blocks [0, head_blocks items): cache blocks; then query blocks; from `work` on a few that check offsets.
template <int D, int PASSES, bool HALF, int THREADS>
__global__ void __launch_bounds__(THREADS, blocks_on_sm<PASSES, THREADS>()) kv_append_kernel(KaArgs a) {
  pdl_enter();
  const int n_cache = a.head_blocks * a.items, i = blockIdx.x;
  if (i >= a.work) {
    check_offsets(a.cu, a.B, a.T, i - a.work, a.status);
    return;
  }
  if (i < n_cache) {
    const int item = i / a.head_blocks, head0 = (i - item * a.head_blocks) * a.heads;
    append_block<D, PASSES, HALF, THREADS>(a, item, head0, min(head0 + a.heads, a.c.n_kv_heads));
    return;
  }
  const int q = i - n_cache;
  switch (query_tokens<D>(a.Hq, blockDim.x)) {
    case 4: query_block<D, HALF, 4>(a, 4 * q); break;
    case 2: query_block<D, HALF, 2>(a, 2 * q); break;
    default: query_block<D, HALF, 1>(a, q); break;
  }
}

template <int D, int PASSES, int THREADS>
cudaError_t launch(KaArgs a, int threads, int sms, cudaStream_t s) {
  // A block takes several heads of a page where there are more pages and heads
  // than blocks at a time: look-ups and angles then serve them all, and the next
  // head's rows come while one is worked on (16 heads, 64 tokens a page: 68 us
  // with a head a block, 57 with four, 54 with six; fewer blocks than fit at
  // once would leave SMs idle).
  const int64_t at_once = static_cast<int64_t>(sms) * blocks_on_sm<PASSES, THREADS>();
  const int64_t pages = a.T / a.c.page_size + std::min<int64_t>(a.B, a.T);
  a.heads = static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(kMaxHeads, pages * a.c.n_kv_heads / at_once)));
  a.head_blocks = ceil_div(a.c.n_kv_heads, a.heads);
  int64_t blocks = static_cast<int64_t>(a.head_blocks) * a.items;
  if (a.q) blocks += ceil_div(a.T, query_tokens<D>(a.Hq, threads));
  a.work = static_cast<int>(std::min<int64_t>(blocks, 0x7fffffff));
  blocks += ceil_div(a.B, threads);
  if (blocks > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned n = static_cast<unsigned>(blocks);
  const auto kernel = a.half ? kv_append_kernel<D, PASSES, true, THREADS> : kv_append_kernel<D, PASSES, false, THREADS>;
  constexpr size_t smem = append_smem(PASSES, THREADS);
  const cudaError_t err = ensure_kernel_attrs(reinterpret_cast<const void*>(kernel), static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  count_launches(1);
  return launch_pdl(kernel, n, threads, smem, s, a);
}

template <int D>
cudaError_t launch_d(const KaArgs& a, int sms, cudaStream_t s) {
  // rows of eight elements a thread, at most four a thread
  const int work = a.c.page_size * (D / 8), threads = std::max(kQueryThreads, work / 4);
  if (work <= kQueryThreads) return launch<D, 1, kQueryThreads>(a, kQueryThreads, sms, s);
  if (work <= 2 * kQueryThreads) return launch<D, 2, kQueryThreads>(a, kQueryThreads, sms, s);
  if (threads <= kQueryThreads) return launch<D, 4, kQueryThreads>(a, threads, sms, s);
  if (threads <= 256) return launch<D, 4, 256>(a, threads, sms, s);
  return launch<D, 4, D == 256 ? 1024 : 512>(a, threads, sms, s);
}

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_kv_append(const moe_kv_append_config_t* cfg, const moe_kv_cache_t* cache, const void* q,
                                      const void* k, const void* v, const float* gamma_q, const float* gamma_k,
                                      const float* cos_sin, const int32_t* positions, const int32_t* cu,
                                      const int32_t* kv_len, void* q_out, moe_stream_t stream) {
  using namespace moe;
  if (!cfg || !kv_cache_shape_ok(cache)) return MOE_ERR_INVALID_ARG;
  const int D = cache->head_dim;
  if (!append_config_ok(cfg, kMaxBatch, cache->n_kv_heads, D, q, gamma_q, q_out)) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!kv_cache_pointers_ok(cache) || !append_pointers_ok(cfg, k, v, gamma_k, cos_sin, positions, cu, kv_len))
    return MOE_ERR_INVALID_ARG;
  unsigned* status = nullptr;
  int sms = 0;
  const moe_status_t st = current_device(&status, &sms);
  if (st != MOE_OK) return st;
  KaArgs a;
  fill_rows(a, cfg, q, k, v, gamma_q, gamma_k, cos_sin, positions, cu, kv_len, q_out, status);
  a.c = *cache;
  a.items = cfg->T / cache->page_size + 2 * cfg->batch;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  switch (D) {
    case 64: err = launch_d<64>(a, sms, s); break;
    case 128: err = launch_d<128>(a, sms, s); break;
    default: err = launch_d<256>(a, sms, s); break;
  }
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
