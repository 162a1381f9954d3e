// The residual's addition and the RMS norm behind it (include/add_rms_norm.h,
// moe_add_rms_norm), with an E4M3 copy and its scales where that is asked for.
//
// Bound by memory: every input is read once and every output written once.  A
// block owns a row and keeps it in registers between the sum of squares and the
// outputs, eight consecutive elements a thread and pass, so that every access is
// 16 bytes (fp32: 32) beside its neighbours'.  A group's largest size is taken
// by the 2 to 32 lanes that hold the group, a row's by the block.
#include "common.cuh"
#include "../../include/add_rms_norm.h"

namespace moe {

moe_status_t current_device(unsigned** status, int* num_sms);

namespace {

constexpr float kMinScale = 9.094947017729282e-13f;   // 2^-40

struct NormArgs {
  const void* x;
  const void* res;
  const float* gamma;
  void* out;
  uint8_t* out8;
  float* scale8;
  void* sum;
  int64_t xs, rs, ss, os;
  int d, group;
  float eps;
  bool x_f32, res_f32, out_f32;
};

__device__ __forceinline__ void load8(const void* base, bool f32, int64_t at, float (&x)[8]) {
  if (f32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + at);
    const float4 a = p[0], b = p[1];
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  } else {
    const uint4 w = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(base) + at);
    const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
}

// Rounds to the stored type and stores; x is left as what was stored.
__device__ __forceinline__ void round8(bool f32, float (&x)[8]) {
  if (f32) return;
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = __bfloat162float(__float2bfloat16_rn(x[i]));
}
__device__ __forceinline__ void store8(void* base, bool f32, int64_t at, const float (&x)[8]) {
  if (f32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    uint32_t v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      v[i] = *reinterpret_cast<const uint32_t*>(&y);
    }
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = make_uint4(v[0], v[1], v[2], v[3]);
  }
}

// PASSES: pieces of eight elements of a thread.
template <int THREADS, int PASSES>
__global__ void __launch_bounds__(THREADS) add_rms_norm_kernel(NormArgs a) {
  constexpr int WARPS = THREADS / 32;
  __shared__ float s_sum[WARPS], s_top[WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pieces = a.d / 8;
  const int64_t row = blockIdx.x;
  float gamma[PASSES][8], h[PASSES][8];
  pdl_enter();
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int p = threadIdx.x + i * THREADS;
    if (p >= pieces) continue;
    load8(a.x, a.x_f32, row * a.xs + p * 8, h[i]);
    float r[8];
    if (a.res) load8(a.res, a.res_f32, row * a.rs + p * 8, r);
    load8(a.gamma, true, p * 8, gamma[i]);
    if (a.res) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] += r[e];
      round8(a.res_f32, h[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) sum = fmaf(h[i][e], h[i][e], sum);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane == 0) s_sum[warp] = sum;
  __syncthreads();   // also: the whole row has been read, outputs may lie over it
  sum = 0.f;
#pragma unroll
  for (int w = 0; w < WARPS; ++w) sum += s_sum[w];
  const float rstd = 1.0f / sqrtf(sum / static_cast<float>(a.d) + a.eps);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int p = threadIdx.x + i * THREADS;
    const bool live = p < pieces;
    if (live && a.sum) store8(a.sum, a.res_f32, row * a.ss + p * 8, h[i]);
    float t = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[i][e] = live ? h[i][e] * rstd * gamma[i][e] : 0.f;
      t = fmaxf(t, fabsf(h[i][e]));   // a NaN is left out
    }
    if (live && a.out) store8(a.out, a.out_f32, row * a.os + p * 8, h[i]);
    if (!a.out8) continue;
    if (a.group == 0) {
      top = fmaxf(top, t);
      continue;
    }
    for (int off = 1; off < a.group / 8; off <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
    const float s = fmaxf(t / 448.f, kMinScale), inv = 1.0f / s;
    if (!live) continue;
    if (p * 8 % a.group == 0) a.scale8[row * (a.d / a.group) + p * 8 / a.group] = s;
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      c[e / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(h[i][e] * inv, h[i][e + 1] * inv),
                                                                 __NV_SATFINITE, __NV_E4M3))
                  << (8 * (e % 4));
    *reinterpret_cast<uint2*>(a.out8 + row * a.d + p * 8) = make_uint2(c[0], c[1]);
  }
  if (!a.out8 || a.group != 0) return;
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
  if (lane == 0) s_top[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < WARPS; ++w) top = fmaxf(top, s_top[w]);
  const float s = fmaxf(top / 448.f, kMinScale), inv = 1.0f / s;
  if (threadIdx.x == 0) a.scale8[row] = s;
#pragma unroll
  for (int i = 0; i < PASSES; ++i) {
    const int p = threadIdx.x + i * THREADS;
    if (p >= pieces) continue;
    uint32_t c[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      c[e / 4] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(h[i][e] * inv, h[i][e + 1] * inv),
                                                                 __NV_SATFINITE, __NV_E4M3))
                  << (8 * (e % 4));
    *reinterpret_cast<uint2*>(a.out8 + row * a.d + p * 8) = make_uint2(c[0], c[1]);
  }
}

template <int THREADS, int PASSES>
cudaError_t launch(const NormArgs& a, int T, cudaStream_t s) {
  count_launches(1);
  return launch_pdl(add_rms_norm_kernel<THREADS, PASSES>, T, THREADS, 0, s, a);
}

bool al(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
bool float_type(int32_t t) { return t == MOE_BF16 || t == MOE_F32; }

}  // namespace
}  // namespace moe

extern "C" moe_status_t moe_add_rms_norm(const moe_add_norm_config_t* cfg, const void* x, const void* residual,
                                         const float* gamma, void* out, void* out8, float* out8_scale, void* sum,
                                         moe_stream_t stream) {
  using namespace moe;
  if (!cfg || cfg->T < 0 || cfg->T > (1 << 28) || cfg->d < 8 || cfg->d > 16384 || cfg->d % 8 != 0 || !(cfg->eps > 0.f) ||
      !(cfg->eps < INFINITY))
    return MOE_ERR_INVALID_ARG;
  auto stride_ok = [&](int64_t s) { return s >= cfg->d && s % 8 == 0; };
  if (!float_type(cfg->x_dtype) || !stride_ok(cfg->x_stride)) return MOE_ERR_INVALID_ARG;
  if (residual && (!float_type(cfg->res_dtype) || !stride_ok(cfg->res_stride))) return MOE_ERR_INVALID_ARG;
  if (sum && (!residual || !stride_ok(cfg->sum_stride))) return MOE_ERR_INVALID_ARG;
  if (out && (!float_type(cfg->out_dtype) || !stride_ok(cfg->out_stride))) return MOE_ERR_INVALID_ARG;
  if (!out && !out8) return MOE_ERR_INVALID_ARG;
  if (out8) {
    const int g = cfg->group;
    if (g != 0 && g != 16 && g != 32 && g != 64 && g != 128 && g != 256) return MOE_ERR_INVALID_ARG;
    if (g != 0 && cfg->d % g != 0) return MOE_ERR_INVALID_ARG;
  }
  if (cfg->T == 0) return MOE_OK;
  if (!x || !gamma || (out8 && !out8_scale)) return MOE_ERR_INVALID_ARG;
  if (!al(x, 16) || !al(residual, 16) || !al(gamma, 16) || !al(out, 16) || !al(out8, 8) || !al(out8_scale, 4) || !al(sum, 16))
    return MOE_ERR_INVALID_ARG;
  unsigned* status = nullptr;
  int sms = 0;
  const moe_status_t st = current_device(&status, &sms);
  if (st != MOE_OK) return st;
  NormArgs a;
  a.x = x;
  a.res = residual;
  a.gamma = gamma;
  a.out = out;
  a.out8 = static_cast<uint8_t*>(out8);
  a.scale8 = out8_scale;
  a.sum = sum;
  a.xs = cfg->x_stride;
  a.rs = cfg->res_stride;
  a.ss = cfg->sum_stride;
  a.os = cfg->out_stride;
  a.d = cfg->d;
  a.group = cfg->group;
  a.eps = cfg->eps;
  a.x_f32 = cfg->x_dtype == MOE_F32;
  a.res_f32 = residual && cfg->res_dtype == MOE_F32;
  a.out_f32 = cfg->out_dtype == MOE_F32;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int pieces = cfg->d / 8;
  cudaError_t err;
  if (pieces <= 128) err = launch<128, 1>(a, cfg->T, s);
  else if (pieces <= 256) err = launch<256, 1>(a, cfg->T, s);
  else if (pieces <= 512) err = launch<512, 1>(a, cfg->T, s);
  else if (pieces <= 1024) err = launch<512, 2>(a, cfg->T, s);
  else err = launch<512, 4>(a, cfg->T, s);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
