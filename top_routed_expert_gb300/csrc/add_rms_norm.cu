// The residual's addition and the RMS norm behind it (include/add_rms_norm.h,
// moe_add_rms_norm), with an E4M3 copy and its scales where that is asked for.
//
// Bound by memory: every input is read once and every output written once.  A
// block works on one row after the other: it keeps gamma in registers, and the
// next row's elements are on their way while a row's squares are summed and its
// outputs leave.  A thread has eight consecutive elements a pass, 16 bytes (fp32:
// 32) beside its neighbours', reads and writes no others (so outputs may lie over
// inputs), and one barrier a row joins the sums.  A group's largest size is taken
// by the 2 to 32 lanes that hold the group, a row's by the block.  Measured: 8192 x
// 4096 bf16 with a residual and E4M3 groups of 128, 303 MB in 49 us = 6.2 TB/s, 0.93 of the
// copy rate (a block a row, with IEEE divisions: 69 us); 64 x 4096 1.8 us in a graph.
#include "common.cuh"
#include "../../include/add_rms_norm.h"

namespace moe {

moe_status_t current_device(unsigned** status, int* num_sms);

namespace {

constexpr float kMinScale = 9.094947017729282e-13f;   // 2^-40
constexpr float k448th = 1.0f / 448.0f;

struct NormArgs {
  const void* x;
  const void* res;
  const float* gamma;
  void* out;
  uint8_t* out8;
  float* scale8;
  void* sum;
  int64_t xs, rs, ss, os;
  int T, d, group, group_log, groups;   // groups: of a row
  float inv_d, eps;
  bool x_f32, out_f32;
};

// Eight elements as they lie in memory.
template <bool F32> struct Raw8 {
  uint4 w[F32 ? 2 : 1];
};

template <bool F32>
__device__ __forceinline__ Raw8<F32> load8(const void* base, int64_t at) {
  Raw8<F32> r;
  const uint4* p = reinterpret_cast<const uint4*>(static_cast<const char*>(base) + at * (F32 ? 4 : 2));
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) r.w[i] = p[i];
  return r;
}
template <bool F32>
__device__ __forceinline__ void unpack8(const Raw8<F32>& r, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < (F32 ? 2 : 1); ++i) {
    const uint32_t v[4] = {r.w[i].x, r.w[i].y, r.w[i].z, r.w[i].w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (F32) {
        x[4 * i + e] = __uint_as_float(v[e]);
      } else {
        x[2 * e] = __uint_as_float(v[e] << 16);
        x[2 * e + 1] = __uint_as_float(v[e] & 0xffff0000u);
      }
    }
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 y = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
    v[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
__device__ __forceinline__ void store8(void* base, bool f32, int64_t at, const float (&x)[8]) {
  if (f32) {
    float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + at);
    p[0] = make_float4(x[0], x[1], x[2], x[3]);
    p[1] = make_float4(x[4], x[5], x[6], x[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + at) = pack8(x);
  }
}
// 1 / x to a unit of the last place.
__device__ __forceinline__ float reciprocal(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Eight elements times `inv` as E4M3 codes.
__device__ __forceinline__ uint2 codes8(const float (&x)[8], float inv) {
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int e = 0; e < 8; e += 2)
    c[e / 4] |= static_cast<uint32_t>(
                    __nv_cvt_float2_to_fp8x2(make_float2(x[e] * inv, x[e + 1] * inv), __NV_SATFINITE, __NV_E4M3))
                << (8 * (e % 4));
  return make_uint2(c[0], c[1]);
}

// Blocks on an SM that the registers are cut for.
template <int THREADS, int PASSES> constexpr int blocks_on_sm() { return (PASSES < 4 ? 1024 : 512) / THREADS; }

// PASSES: pieces of eight elements of a thread.  RES: residual 0 none, 1 bf16, 2 fp32.
template <int THREADS, int PASSES, bool XF32, int RES>
__global__ void __launch_bounds__(THREADS, blocks_on_sm<THREADS, PASSES>()) add_rms_norm_kernel(NormArgs a) {
  constexpr int WARPS = THREADS / 32;
  __shared__ float s_sum[2][WARPS], s_top[2][WARPS];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, pieces = a.d / 8;
  auto live = [&](int i) { return static_cast<int>(threadIdx.x) + i * THREADS < pieces; };
  auto at = [&](int i) { return (static_cast<int>(threadIdx.x) + i * THREADS) * 8; };
  pdl_enter();
  float gamma[PASSES][8];
  Raw8<XF32> x[PASSES];
  Raw8<RES == 2> r[PASSES];
  auto load = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      if (!live(i)) continue;
      x[i] = load8<XF32>(a.x, row * a.xs + at(i));
      if (RES) r[i] = load8<RES == 2>(a.res, row * a.rs + at(i));
    }
  };
  load(blockIdx.x);
#pragma unroll
  for (int i = 0; i < PASSES; ++i)
    if (live(i)) unpack8<true>(load8<true>(a.gamma, at(i)), gamma[i]);
  int odd = 0;   // in turn: one barrier a row
#pragma unroll 1
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, odd ^= 1) {
    float h[PASSES][8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
#pragma unroll
      for (int e = 0; e < 8; ++e) h[i][e] = 0.f;
      if (!live(i)) continue;
      unpack8<XF32>(x[i], h[i]);
      if (RES) {
        float y[8];
        unpack8<RES == 2>(r[i], y);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[i][e] += y[e];
        if (RES == 1) {   // the norm is that of the rounded sum
          Raw8<false> rounded;
          rounded.w[0] = pack8(h[i]);
          if (a.sum) *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.sum) + row * a.ss + at(i)) = rounded.w[0];
          unpack8<false>(rounded, h[i]);
        } else if (a.sum) {
          store8(a.sum, true, row * a.ss + at(i), h[i]);
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum = fmaf(h[i][e], h[i][e], sum);
    }
    if (row + gridDim.x < a.T) load(row + gridDim.x);
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    if (lane == 0) s_sum[odd][warp] = sum;
    __syncthreads();
    sum = 0.f;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) sum += s_sum[odd][w];
    const float rstd = rsqrtf(fmaf(sum, a.inv_d, a.eps));
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < PASSES; ++i) {
      float t = 0.f;
      if (live(i)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          h[i][e] = h[i][e] * rstd * gamma[i][e];
          t = fmaxf(t, fabsf(h[i][e]));   // a NaN is left out
        }
        if (a.out) store8(a.out, a.out_f32, row * a.os + at(i), h[i]);
      }
      if (!a.out8) continue;
      if (a.group == 0) {
        top = fmaxf(top, t);
        continue;
      }
      for (int off = 1; off < a.group / 8; off <<= 1) t = fmaxf(t, __shfl_xor_sync(0xffffffffu, t, off));
      if (!live(i)) continue;
      const float s = fmaxf(t * k448th, kMinScale);
      if (at(i) % a.group == 0) a.scale8[row * a.groups + (at(i) >> a.group_log)] = s;
      *reinterpret_cast<uint2*>(a.out8 + row * a.d + at(i)) = codes8(h[i], reciprocal(s));
    }
    if (!a.out8 || a.group != 0) continue;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if (lane == 0) s_top[odd][warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) top = fmaxf(top, s_top[odd][w]);
    const float s = fmaxf(top * k448th, kMinScale), inv = reciprocal(s);
    if (threadIdx.x == 0) a.scale8[row] = s;
#pragma unroll
    for (int i = 0; i < PASSES; ++i)
      if (live(i)) *reinterpret_cast<uint2*>(a.out8 + row * a.d + at(i)) = codes8(h[i], inv);
  }
}

template <int THREADS, int PASSES>
cudaError_t launch(const NormArgs& a, int res, int sms, cudaStream_t s) {
  count_launches(1);
  const int blocks = std::min(a.T, sms * blocks_on_sm<THREADS, PASSES>());
  auto go = [&](auto kernel) { return launch_pdl(kernel, blocks, THREADS, 0, s, a); };
  if (a.x_f32) {
    if (res == 0) return go(add_rms_norm_kernel<THREADS, PASSES, true, 0>);
    return res == 1 ? go(add_rms_norm_kernel<THREADS, PASSES, true, 1>) : go(add_rms_norm_kernel<THREADS, PASSES, true, 2>);
  }
  if (res == 0) return go(add_rms_norm_kernel<THREADS, PASSES, false, 0>);
  return res == 1 ? go(add_rms_norm_kernel<THREADS, PASSES, false, 1>) : go(add_rms_norm_kernel<THREADS, PASSES, false, 2>);
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
  a.T = cfg->T;
  a.d = cfg->d;
  a.group = cfg->group;
  a.group_log = 0;
  while (cfg->group >> a.group_log > 1) ++a.group_log;
  a.groups = out8 && cfg->group ? cfg->d / cfg->group : 1;
  a.inv_d = 1.0f / static_cast<float>(cfg->d);
  a.eps = cfg->eps;
  a.x_f32 = cfg->x_dtype == MOE_F32;
  a.out_f32 = cfg->out_dtype == MOE_F32;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int pieces = cfg->d / 8, res = !residual ? 0 : cfg->res_dtype == MOE_F32 ? 2 : 1;
  cudaError_t err;
  // a pass where that gives a block 512 threads or fewer (8192 x 4096: 512 threads 52 us,
  // 256 with two passes 58, 128 with four 59; 65536 x 512: 64 threads 48, 128 65).  More
  // passes cost spills of gamma and the next row: bytes stored with x / residual bf16 / bf16,
  // f32 / bf16, bf16 / f32, f32 / f32 and f32 / none 16, 48, 48, 72, 16 with two passes, 0, 32, 32,
  // 80, 0 with four.  The rate falls little: as many bytes at d = 4096, 8192, 16384 (bf16, bf16,
  // groups of 128) 48.5, 49.5, 52.2 us.
  if (pieces <= 32) err = launch<32, 1>(a, res, sms, s);
  else if (pieces <= 64) err = launch<64, 1>(a, res, sms, s);
  else if (pieces <= 128) err = launch<128, 1>(a, res, sms, s);
  else if (pieces <= 256) err = launch<256, 1>(a, res, sms, s);
  else if (pieces <= 512) err = launch<512, 1>(a, res, sms, s);
  else if (pieces <= 1024) err = launch<512, 2>(a, res, sms, s);
  else err = launch<512, 4>(a, res, sms, s);
  return err == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
