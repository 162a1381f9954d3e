// Expert selection from given logits (include/route_scores.h): scores, bias,
// groups, top-k and weights of one token in one warp; a warp takes tokens in
// turn and keeps the bias in registers.
//
// Lane l holds the EPL consecutive experts l*EPL .. l*EPL+EPL-1, so a token's
// logits are one vector load per lane, a group of experts is a run of lanes,
// and among lanes with equal values the lowest lane has the lowest expert.
//
// The choice is bound by instructions, not by bytes (a token of 256 experts is
// 512 or 1024 bytes), so it is made of few:
//  - each lane sorts its keys once (19 compare-exchanges of eight keys, each a
//    minimum and a maximum; no index travels with them);
//  - a round of the top-k is one warp maximum of the lanes' heads and one
//    ballot; the lowest lane that holds it goes on to its next key, which waits
//    in shared memory (moving a list up in registers took a third of a round);
//  - which expert a key belongs to is looked up at the end, for the chosen ones
//    alone, by the lane of their slot.
//
// score s = sigmoid(L) or softmax(L); choice c = s + bias (without a bias the
// order of L is that of s, and c = L); a group's value is the sum of its `rank`
// largest c; k experts of the best groups by c, ties to the lowest; weights
// scale s / sum of the chosen s.
//
// Measured: 65519 tokens of 256 experts (8 groups, bias, sigmoid, bf16, k = 8)
// 49.5 us, 675 warp instructions a token at three quarters of the issue
// slots, 0.76 TB/s; one token of 128 experts 1.7 us in a graph, a launch.  A token for half
// a warp would halve the rounds' cost but double the sort's and leaves the
// scores' as it is.
#include <cmath>

#include "common.cuh"
#include "../../include/route_scores.h"

namespace moe {

moe_status_t current_device(unsigned** status, int* num_sms);

namespace {

constexpr int kRsWarps = 4;
constexpr float kMasked = -INFINITY;

// Order-preserving key of a value that is finite or -infinity, and not -0.
// -infinity maps to 0x007fffff, so 0 is free to mark "not available".
__device__ __forceinline__ uint32_t value_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return u ^ (static_cast<uint32_t>(static_cast<int32_t>(u) >> 31) | 0x80000000u);
}
constexpr uint32_t kMaskedKey = 0x007fffffu;

struct RsArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* w;
  unsigned* status;
  int64_t stride;
  int T, E, k, G, tg, rank;
  float scale;
  bool sigmoid, renorm, vectors;   // vectors: rows can be read EPL elements at a time
};

// The two largest of two (largest, second largest) pairs.
struct Top2 {
  float first, second;
};
__device__ __forceinline__ Top2 merge(const Top2& a, const Top2& b) {
  return Top2{fmaxf(a.first, b.first), fmaxf(fmaxf(fminf(a.first, b.first), a.second), b.second)};
}
// The two largest of N values (N a power of two).
template <int N>
__device__ __forceinline__ Top2 top2_of(const float (&v)[N]) {
  Top2 t[N];
#pragma unroll
  for (int i = 0; i < N; ++i) t[i] = Top2{v[i], kMasked};
#pragma unroll
  for (int n = N / 2; n > 0; n /= 2)
#pragma unroll
    for (int i = 0; i < n; ++i) t[i] = merge(t[i], t[i + n]);
  return t[0];
}

// The larger of two values, NaN if either is.
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// N words of a lane into shared memory, 16 bytes at a time where there are as many.
template <int N>
__device__ __forceinline__ void put(uint32_t* to, const uint32_t (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) *reinterpret_cast<uint4*>(to + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) to[i] = v[i];
  }
}

template <int N>
__device__ __forceinline__ void get(const uint32_t* from, uint32_t (&v)[N]) {
  if constexpr (N % 4 == 0) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(from + i);
      v[i] = x.x;
      v[i + 1] = x.y;
      v[i + 2] = x.z;
      v[i + 3] = x.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = from[i];
  }
}

// Descending order of N keys (N a power of two): Batcher's odd-even merge sort.
template <int N>
__device__ __forceinline__ void sort_descending(uint32_t (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int q = p; q > 0; q /= 2)
#pragma unroll
      for (int j = q % p; j + q < N; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i)
          if (i + j + q < N && (i + j) / (2 * p) == (i + j + q) / (2 * p)) {
            const uint32_t a = k[i + j], b = k[i + j + q];
            k[i + j] = max(a, b);
            k[i + j + q] = min(a, b);
          }
}

// The lane's EPL logits of a token as they lie in memory.
template <int EPL, bool BF16> struct RawLogits {
  static constexpr int kWords = BF16 ? (EPL + 1) / 2 : EPL;
  uint32_t w[kWords];
};

template <int EPL, bool BF16>
__device__ __forceinline__ RawLogits<EPL, BF16> load_logits(const RsArgs& a, int t, int lane) {
  RawLogits<EPL, BF16> r;
  constexpr int N = RawLogits<EPL, BF16>::kWords;
  if (a.vectors) {
    const uint32_t* p = static_cast<const uint32_t*>(a.logits) + (BF16 ? t * a.stride / 2 : t * a.stride) + lane * N;
    if constexpr (N % 4 == 0) {
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p + i));
        r.w[i] = v.x;
        r.w[i + 1] = v.y;
        r.w[i + 2] = v.z;
        r.w[i + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) r.w[i] = __ldg(p + i);
    }
  } else {
    constexpr uint32_t none = BF16 ? 0xff80u : 0xff800000u;   // -infinity behind the last expert
#pragma unroll
    for (int i = 0; i < N; ++i) r.w[i] = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane * EPL + i;
      const int64_t at = t * a.stride + e;
      if (BF16) r.w[i / 2] |= static_cast<uint32_t>(e < a.E ? __ldg(static_cast<const uint16_t*>(a.logits) + at) : none) << (16 * (i & 1));
      else r.w[i] = e < a.E ? __ldg(static_cast<const uint32_t*>(a.logits) + at) : none;
    }
  }
  return r;
}

// Blocks on an SM (48 registers a thread); a long batch's warps take several
// tokens each (65519 tokens of 256 experts, 8 groups, 8 / 10 blocks: sigmoid 49.4 to
// 50.6 / 48.2 to 50.1 us, softmax 57.0 to 58.9 / 57.0 to 58.6; softmax without a bias
// spills 12 to 16 bytes with ten, f32 57.0 / 58.0, bf16 57.6 / 57.0).
constexpr int kRsBlocks = 10;

template <int EPL, bool BF16, bool SIGMOID, bool BIAS>
__global__ void __launch_bounds__(kRsWarps * 32, kRsBlocks) route_scores_kernel(RsArgs a) {
  // per warp: a token's keys (first the values that rank groups) and scores
  __shared__ __align__(16) uint32_t s_key[kRsWarps][32 * EPL];
  __shared__ __align__(16) float s_score[kRsWarps][32 * EPL];
  constexpr int kList = EPL % 4 == 0 ? 12 : EPL + 1;   // words of a lane's list: 16-byte stores without conflicts
  __shared__ __align__(16) uint32_t s_sorted[kRsWarps][32 * kList];   // each lane's keys in order, 0 behind the last
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = gridDim.x * kRsWarps;
  int t = blockIdx.x * kRsWarps + warp;
  if (t >= a.T) return;
  RawLogits<EPL, BF16> raw = load_logits<EPL, BF16>(a, t, lane);
  float bias[EPL];
  bool bad_bias = false;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    bias[i] = BIAS && e < a.E ? a.bias[e] : 0.f;
    if (!(bias[i] < INFINITY)) {   // NaN or +infinity: a mask
      bad_bias = true;
      bias[i] = kMasked;
    }
  }
  const int gs = a.E / a.G;
  // groups that are a power of two of whole lanes are ranked by shuffles
  const int lpg = gs / EPL;
  const bool by_lanes = gs == lpg * EPL && (lpg & (lpg - 1)) == 0;
  const int lpg_log = by_lanes ? 31 - __clz(lpg) : 0, my_group = lane >> lpg_log;
  uint32_t* list = s_sorted[warp] + lane * kList;
  list[EPL] = 0u;

  while (true) {
    float L[EPL], s[EPL], c[EPL];
    bool bad = bad_bias;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (BF16) L[i] = __uint_as_float(i & 1 ? raw.w[i / 2] & 0xffff0000u : raw.w[i / 2] << 16);
      else L[i] = __uint_as_float(raw.w[i]);
    }
    float top = L[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) top = max_or_nan(top, L[i]);
    if (!(top < INFINITY)) {   // a NaN or +infinity among them: a mask
      bad = true;
      top = kMasked;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if (!(L[i] < INFINITY)) L[i] = kMasked;
        top = fmaxf(top, L[i]);
      }
    }
    const int next = t + warps;
    if (next < a.T) raw = load_logits<EPL, BF16>(a, next, lane);
    // scores; numer keeps the softmax numerators
    float numer[EPL];
    if (SIGMOID) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) numer[i] = s[i] = __frcp_rn(1.0f + expf(-L[i]));
    } else {
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
      if (top == kMasked) top = 0.f;   // every expert masked
      // The denominator is a compensated sum (a two-term fp32 value, about 2^-45
      // relative), so that its rounding, and with it the order of nearly equal
      // biased scores, does not depend on the order of the addition.
      float hi = 0.f, lo = 0.f;
      auto add = [&](float x, float xlo) {
        const float y = __fadd_rn(hi, x);
        const float z = __fsub_rn(y, hi);
        lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(y, z)), __fsub_rn(x, z)) + xlo;
        hi = y;
      };
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        numer[i] = expf(L[i] - top);
        add(numer[i], 0.f);
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1)
        add(__shfl_xor_sync(0xffffffffu, hi, off), __shfl_xor_sync(0xffffffffu, lo, off));
      const float Z = hi + lo;
#pragma unroll
      for (int i = 0; i < EPL; ++i) s[i] = Z > 0.f ? __fdiv_rn(numer[i], Z) : 0.f;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) c[i] = !BIAS ? L[i] : L[i] > kMasked ? __fadd_rn(s[i], bias[i]) : kMasked;
    // groups
    bool kept = true;              // by_lanes: this lane's group
    uint32_t keep = 0xffffffffu;   // else a bit for each of the lane's experts
    if (a.tg < a.G) {
      // what ranks the groups: the values, or without a bias the scores where two are added
      float v[EPL];
#pragma unroll
      for (int i = 0; i < EPL; ++i) v[i] = !BIAS && a.rank == 2 ? numer[i] : c[i];
      if (by_lanes) {
        Top2 two = top2_of<EPL>(v);
        for (int off = 1; off < lpg; off <<= 1)
          two = merge(two, Top2{__shfl_xor_sync(0xffffffffu, two.first, off), __shfl_xor_sync(0xffffffffu, two.second, off)});
        const float value = (a.rank == 2 && gs > 1) ? two.first + two.second : two.first;
        // the best group that is left, the lowest among equals, tg times
        uint32_t left = my_group < a.G ? value_key(value + 0.0f) : 0u;
        kept = false;
        for (int j = 0; j < a.tg; ++j) {
          const uint32_t best = __reduce_max_sync(0xffffffffu, left);
          const int src = __ffs(__ballot_sync(0xffffffffu, left == best)) - 1;
          if (my_group == src >> lpg_log) {
            kept = true;
            left = 0u;
          }
        }
      } else {
        float* val = s_score[warp];
#pragma unroll
        for (int i = 0; i < EPL; ++i) val[lane * EPL + i] = v[i];
        __syncwarp();
        Top2 two = {kMasked, kMasked};
        if (lane < a.G)
          for (int i = 0; i < gs; ++i) two = merge(two, Top2{val[lane * gs + i], kMasked});
        const float value = (a.rank == 2 && gs > 1) ? two.first + two.second : two.first;
        int better = 0;
        for (int g = 0; g < a.G; ++g) {
          const float u = __shfl_sync(0xffffffffu, value, g);
          better += (u > value || (u == value && g < lane)) ? 1 : 0;
        }
        const unsigned bits = __ballot_sync(0xffffffffu, lane < a.G && better < a.tg);
        keep = 0u;
#pragma unroll
        for (int i = 0; i < EPL; ++i) keep |= ((bits >> ((lane * EPL + i) / gs)) & 1u) << i;
        __syncwarp();
      }
    }
    // keys; lanes behind the last expert hold masked ones, which no slot reaches
    uint32_t key[EPL], score_bits[EPL];
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      key[i] = value_key(BIAS ? c[i] : c[i] + 0.0f);   // s + bias is never -0
      score_bits[i] = __float_as_uint(s[i]);
    }
    if (!by_lanes && a.tg < a.G) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = (keep >> i) & 1u ? key[i] : 0u;
    }
    put(s_key[warp] + lane * EPL, key);
    put(reinterpret_cast<uint32_t*>(s_score[warp]) + lane * EPL, score_bits);
    // k rounds: the warp's largest key, from the lowest lane that holds it
    sort_descending<EPL>(key);
    put(list, key);
    uint32_t head = kept ? key[0] : 0u, my_key = 0u;
    const uint32_t* rest = list;
    int my_src = 0;
    for (int j = 0; j < a.k; ++j) {
      const uint32_t wk = __reduce_max_sync(0xffffffffu, head);
      const int src = __ffs(__ballot_sync(0xffffffffu, head == wk)) - 1;
      if (lane == src) head = *++rest;
      if (lane == j) {
        my_key = wk;
        my_src = src;
      }
    }
    // The expert of slot `lane`: the lane that gave the key gives equal ones one
    // after the other, lowest expert first.
    const uint32_t before_key = __shfl_up_sync(0xffffffffu, my_key, 1);
    const int before_src = __shfl_up_sync(0xffffffffu, my_src, 1);
    const unsigned starts = __ballot_sync(0xffffffffu, lane == 0 || before_key != my_key || before_src != my_src);
    int nth = lane - (31 - __clz(starts & (0xffffffffu >> (31 - lane))));
    __syncwarp();
    get(s_key[warp] + my_src * EPL, key);
    uint32_t hits = 0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) hits |= key[i] == my_key ? 1u << i : 0u;
    for (nth = lane < a.k ? nth : 0; nth > 0; --nth) hits &= hits - 1;
    const int my_e = my_src * EPL + __ffs(hits) - 1;
    float my_s = lane < a.k && my_key > kMaskedKey ? s_score[warp][my_e] : 0.f;
    float sum = my_s;
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);   // k <= 16 slots
    if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(a.status, MOE_ERR_DEVICE_NONFINITE);
    if (lane < a.k) {
      if (a.renorm) my_s = sum > 0.f ? my_s / sum : 0.f;
      a.ids[static_cast<int64_t>(t) * a.k + lane] = my_e;
      a.w[static_cast<int64_t>(t) * a.k + lane] = my_s * a.scale;
    }
    if (next >= a.T) return;
    t = next;
    __syncwarp();   // the token's keys and scores have been read
  }
}

template <int EPL, bool BF16>
cudaError_t launch(const RsArgs& a, int blocks, cudaStream_t s) {
  if (a.sigmoid)
    return a.bias ? launch_pdl(route_scores_kernel<EPL, BF16, true, true>, blocks, kRsWarps * 32, 0, s, a)
                  : launch_pdl(route_scores_kernel<EPL, BF16, true, false>, blocks, kRsWarps * 32, 0, s, a);
  return a.bias ? launch_pdl(route_scores_kernel<EPL, BF16, false, true>, blocks, kRsWarps * 32, 0, s, a)
                : launch_pdl(route_scores_kernel<EPL, BF16, false, false>, blocks, kRsWarps * 32, 0, s, a);
}

template <int EPL>
cudaError_t launch(RsArgs a, bool bf16, int num_sms, cudaStream_t s) {
  const uintptr_t base = reinterpret_cast<uintptr_t>(a.logits);
  const int row_bytes = EPL * (bf16 ? 2 : 4);   // a lane's
  const size_t align = row_bytes >= 16 ? 16 : 4;
  a.vectors = a.E == 32 * EPL && row_bytes % 4 == 0 && base % align == 0 && a.stride * (bf16 ? 2 : 4) % align == 0;
  const int blocks = std::min(ceil_div(a.T, kRsWarps), num_sms * kRsBlocks);
  count_launches(1);
  return bf16 ? launch<EPL, true>(a, blocks, s) : launch<EPL, false>(a, blocks, s);
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_route_scores(const moe_route_scores_config_t* c, const void* logits, const float* bias,
                                         int32_t* topk_ids, float* topk_w, moe_stream_t stream) {
  using namespace moe;
  if (!c || c->T < 0 || c->n_experts < 1 || c->n_experts > kMaxExperts || c->n_groups < 1 || c->n_groups > 32 ||
      c->n_experts % c->n_groups != 0 || c->top_groups < 1 || c->top_groups > c->n_groups)
    return MOE_ERR_INVALID_ARG;
  if (c->top_k < 1 || c->top_k > 16 || c->top_k > c->top_groups * (c->n_experts / c->n_groups))
    return MOE_ERR_INVALID_ARG;
  if ((c->group_rank != 1 && c->group_rank != 2) || (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) ||
      (c->logit_dtype != MOE_F32 && c->logit_dtype != MOE_BF16) || (c->renormalise != 0 && c->renormalise != 1))
    return MOE_ERR_INVALID_ARG;
  if (!(c->scale > 0.f) || !std::isfinite(c->scale) || c->logit_stride < c->n_experts) return MOE_ERR_INVALID_ARG;
  if (c->T > (1 << 30) / 16) return MOE_ERR_INVALID_ARG;
  if (c->T == 0) return MOE_OK;
  const size_t esz = c->logit_dtype == MOE_F32 ? 4 : 2;
  if (!logits || !topk_ids || !topk_w || !aligned_to(logits, esz) || !aligned_to(topk_ids, 4) ||
      !aligned_to(topk_w, 4) || (bias && !aligned_to(bias, 4)))
    return MOE_ERR_INVALID_ARG;
  unsigned* status = nullptr;
  int sms = 0;
  const moe_status_t st = current_device(&status, &sms);
  if (st != MOE_OK) return st;
  RsArgs a;
  a.logits = logits;
  a.bias = bias;
  a.ids = topk_ids;
  a.w = topk_w;
  a.status = status;
  a.stride = c->logit_stride;
  a.T = c->T;
  a.E = c->n_experts;
  a.k = c->top_k;
  a.G = c->n_groups;
  a.tg = c->top_groups;
  a.rank = c->group_rank;
  a.scale = c->scale;
  a.sigmoid = c->score == MOE_SCORE_SIGMOID;
  a.renorm = c->renormalise != 0;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool bf16 = c->logit_dtype == MOE_BF16;
  cudaError_t err;
  if (a.E <= 32) err = launch<1>(a, bf16, sms, s);
  else if (a.E <= 64) err = launch<2>(a, bf16, sms, s);
  else if (a.E <= 128) err = launch<4>(a, bf16, sms, s);
  else err = launch<8>(a, bf16, sms, s);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
