// Expert selection from given logits (include/route_scores.h): scores, bias,
// groups, top-k and weights of one token in one warp.
//
// Lane l holds the EPL consecutive experts l*EPL .. l*EPL+EPL-1, so a token's
// logits are one vector load per lane, a group of experts is a run of lanes,
// and among lanes with equal values the lowest lane has the lowest expert.
#include <cmath>

#include "common.cuh"
#include "../../include/route_scores.h"

namespace moe {

moe_status_t current_device(unsigned** status, int* num_sms);

namespace {

constexpr int kRsWarps = 4;
constexpr float kMasked = -INFINITY;

// Order-preserving key of a value that is finite or -infinity (-0 folded onto
// +0).  -infinity maps to 0x007fffff, so 0 is free to mark "not available".
__device__ __forceinline__ uint32_t value_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
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
  bool bf16, sigmoid, renorm;
};

__device__ __forceinline__ float load_logit(const RsArgs& a, int64_t i) {
  return a.bf16 ? bf16_bits_to_float(static_cast<const uint16_t*>(a.logits)[i]) : static_cast<const float*>(a.logits)[i];
}

// Larger of two (largest, second largest) pairs' union.
__device__ __forceinline__ void merge_top2(float& t1, float& t2, float u1, float u2) {
  t2 = fmaxf(fminf(t1, u1), fmaxf(t2, u2));
  t1 = fmaxf(t1, u1);
}

template <int EPL>
__global__ void __launch_bounds__(kRsWarps * 32) route_scores_kernel(RsArgs a) {
  __shared__ float sval[kRsWarps][32 * EPL];
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x * kRsWarps + warp;
  if (t >= a.T) return;
  float L[EPL], s[EPL], c[EPL];
  bool bad = false;
  float top = kMasked;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    L[i] = e < a.E ? load_logit(a, t * a.stride + e) : kMasked;
    if (!(L[i] < INFINITY)) { bad = true; L[i] = kMasked; }   // NaN or +infinity
    top = fmaxf(top, L[i]);
  }
  // scores; numer keeps the softmax numerators
  float numer[EPL];
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) numer[i] = s[i] = 1.0f / (1.0f + expf(-L[i]));
  } else {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (top == kMasked) top = 0.f;   // every expert masked
#pragma unroll
    for (int i = 0; i < EPL; ++i) numer[i] = expf(L[i] - top);
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
    for (int i = 0; i < EPL; ++i) add(numer[i], 0.f);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) add(__shfl_xor_sync(0xffffffffu, hi, off), __shfl_xor_sync(0xffffffffu, lo, off));
    const float Z = hi + lo;
#pragma unroll
    for (int i = 0; i < EPL; ++i) s[i] = Z > 0.f ? numer[i] / Z : 0.f;
  }
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    if (a.bias && e < a.E) {
      const float b = a.bias[e];
      if (!(b < INFINITY)) bad = true;
      c[i] = (b < INFINITY && L[i] > kMasked) ? __fadd_rn(s[i], b) : kMasked;
    } else {
      c[i] = L[i];
    }
  }
  // groups
  uint32_t keep = 0xffffffffu;
  const int gs = a.E / a.G;
  if (a.tg < a.G) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) sval[warp][lane * EPL + i] = (!a.bias && a.rank == 2) ? numer[i] : c[i];
    __syncwarp();
    float value = kMasked;
    if (lane < a.G) {
      float t1 = kMasked, t2 = kMasked;
      for (int i = 0; i < gs; ++i) merge_top2(t1, t2, sval[warp][lane * gs + i], kMasked);
      value = (a.rank == 2 && gs > 1) ? t1 + t2 : t1;
    }
    int better = 0;
    for (int g = 0; g < a.G; ++g) {
      const float v = __shfl_sync(0xffffffffu, value, g);
      better += (v > value || (v == value && g < lane)) ? 1 : 0;
    }
    keep = __ballot_sync(0xffffffffu, lane < a.G && better < a.tg);
  }
  uint32_t key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane * EPL + i;
    key[i] = (e < a.E && ((keep >> (e / gs)) & 1u)) ? value_key(c[i]) : 0u;
  }
  // k rounds: the warp's largest key, the lowest expert that holds it
  float my_s = 0.f, sum = 0.f;
  int my_e = 0;
  for (int j = 0; j < a.k; ++j) {
    uint32_t bk = 0u;
    int bi = 0;
    float bs = 0.f;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const bool better = key[i] > bk;
      bk = better ? key[i] : bk;
      bi = better ? i : bi;
      bs = better ? s[i] : bs;
    }
    const uint32_t wk = __reduce_max_sync(0xffffffffu, bk);
    const int src = __ffs(__ballot_sync(0xffffffffu, bk == wk)) - 1;
    const int e = src * EPL + __shfl_sync(0xffffffffu, bi, src);
    float v = __shfl_sync(0xffffffffu, bs, src);
    if (wk <= kMaskedKey) v = 0.f;
    if (lane == src) {
#pragma unroll
      for (int i = 0; i < EPL; ++i) key[i] = i == bi ? 0u : key[i];
    }
    sum += v;
    if (lane == j) { my_s = v; my_e = e; }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) set_status(a.status, MOE_ERR_DEVICE_NONFINITE);
  if (lane < a.k) {
    const float w = a.renorm ? (sum > 0.f ? my_s / sum : 0.f) : my_s;
    a.ids[static_cast<int64_t>(t) * a.k + lane] = my_e;
    a.w[static_cast<int64_t>(t) * a.k + lane] = w * a.scale;
  }
}

template <int EPL>
cudaError_t launch(const RsArgs& a, cudaStream_t s) {
  count_launches(1);
  return launch_pdl(route_scores_kernel<EPL>, ceil_div(a.T, kRsWarps), kRsWarps * 32, 0, s, a);
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
  const RsArgs a = {logits,  bias,      topk_ids,        topk_w,          status,   c->logit_stride,
                    c->T,    c->n_experts, c->top_k,     c->n_groups,     c->top_groups, c->group_rank,
                    c->scale, esz == 2,  c->score == MOE_SCORE_SIGMOID, c->renormalise != 0};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  if (a.E <= 32) err = launch<1>(a, s);
  else if (a.E <= 64) err = launch<2>(a, s);
  else if (a.E <= 128) err = launch<4>(a, s);
  else err = launch<8>(a, s);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
