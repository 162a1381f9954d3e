// Attention over the paged 8-bit cache for many query rows (prompts and
// their chunks) on the 5th-generation tensor cores.
//
// The rows of one (request, key head) are its new tokens times the query
// heads of the group (row r = token r / group, head r % group); an item is 256
// of them, two tiles of 128, and walks the cached tokens that any of them sees
// in steps of 128:
//   S = Q K^T   (kind::f16, M = 128 rows, N = 128 tokens, both from shared
//               memory)
//   P = 2^(S k_scale .. - m), f16, written over S in tensor memory
//   O += P V    (A = P from tensor memory, B = V^T from shared memory)
// Warps 0-3 and 4-7 are the softmax of tile 0 and 1 (one thread a row), warps
// 8-11 convert keys and 12-15 values, warp 16 issues the MMAs, warp 17 looks up
// pages and scales some steps ahead (18 and 19 only lend registers): while one
// tile's softmax runs, the tensor core works on the other's products.  The CTAs
// are persistent, one on an SM, and take items from a list that paged_attn.cu
// has sorted by length; steps of the next item start beside the last of this.
//
// The cache's codes become f16 exactly on the way to shared memory (E4M3 fits
// f16), one conversion for the 256 rows; the values are transposed there by
// byte permutations before the conversion, so both products read K-major
// operands.  Page scales stay out of the products: a score is multiplied by
// its 16-token group's key scale, and the value scale is added to the
// exponent (its logarithm), so that P V needs no scaling and the sum of the
// weights is the group sums divided by the same scale.
//
// A row's weights are taken relative to 2^-8 of the maximum of the first step that
// it sees something in (kRefBelow), and that reference moves only when a group of
// 16 weights sums to over 65504: until then they fit f16, and the quotient is the
// same.  So the scores are read once, no maximum is taken in the ordinary
// step, and the accumulator is almost never rescaled.
//
// Few items would leave SMs idle, so long ones are cut along the tokens
// (paged_attn.cu) and paged_attn_tc_join adds the parts up in order.
//
// Measured: 32 x 256 tokens of 4 x 8 heads of 128 behind up to 3328 others, 241
// GFLOP in 266 us = 906 TFLOP/s, the tensor pipe active 41 % of the time; one
// prompt of 8192, 550 GFLOP in 478 us = 1151 TFLOP/s.  A step of 128 tokens takes
// about 2.2 us.  Its 32 MMAs of 128 x 128 x 16 take about 104 cycles each, 1.75 us
// (one of 128 x 256 x 16 takes 135, but two tiles' scores and outputs fill the
// tensor memory); the rest is the hand-over between scores, weights and products.
// What holds an MMA to 104 cycles is not known: shared memory is at 51 % of its
// rate (30 % operands of the MMAs, 21 % the other warps), so not its bandwidth
// alone.  An item's start and end (its q, the first reference, its output) cost
// two to three steps more, which is what the short prompts lose.  Of 128 registers
// the softmax warps spill 88 bytes (D = 64: 40).
#include <climits>

#include "paged_attn.cuh"
#include "tc_ptx.cuh"

namespace moe {

using namespace ptx;

namespace {

constexpr int kRowTile = 128;
static_assert(kTcItemRows == 2 * kRowTile, "two row tiles");
constexpr int kTok = kTcStep;            // tokens of a step
constexpr int kGroups = kTok / 16;       // scale groups of a step
constexpr int kThreads = 20 * 32;
// Registers of a thread, by warpgroup: two of softmax, two of conversion, one
// that plans and issues.  The launch has 96 for each of the 640 threads;
// 256 x 128 + 256 x 72 + 128 x 80 are the same 61440.
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 128, kConvRegs = 72, kIssueRegs = 80;
static_assert(2 * kSoftmaxRegs + 2 * kConvRegs + kIssueRegs <= 5 * kLaunchRegs, "setmaxnreg would wait forever");
constexpr int kConvThreads = 128;
constexpr int kSlots = 8;              // steps that are planned ahead, at most
constexpr int kItems = 16;             // items that are announced ahead; more than kSlots, as an item has a step or more
constexpr float kLog2e = 1.4426950408889634f;
constexpr long long kWaitCycles = 3000000000ll;
constexpr uint64_t kDrainNs = 200000000ull;

// A row block's work, or a part of it: up to 256 rows of one request and key
// head, over `steps` steps from step u0 on; rows = 0: there is no more.
struct Item {
  int b, kvh, token0, n, end, row0, rows;   // token0, n, end: the request's rows and length
  int u0, steps, slot;                      // slot: where a part leaves its sums; -1: the whole block
  __device__ __forceinline__ Span span(const PaArgs& a) const {
    const int start = end - n;
    return span_for(a, start + row0 / a.group, start + (row0 + rows - 1) / a.group, kTok);
  }
};

struct Ctrl {
  // s_full[tile][step & 1] is the one signal that the MMA warp gives in a step:
  // it says that the tile's scores are there and, the products running in
  // order, that everything issued before them is done.  The converters take
  // their free stages from tile 1's.  (Two barriers in turn, so that none can
  // run a phase ahead of a waiter; a signal of its own for each stage made the
  // issuing warp the bottleneck.)  Steps are counted through all items.
  uint64_t q_full, k_full[2], v_full[2], s_full[2][2], p_full[2], o_full[2], plan_full[kSlots], plan_free[kSlots],
      item_full[kItems], drain;
  // of a step's eight 16-token groups: key scale, log2 of the value scale, 1 /
  // value scale, first token (an integer's bits); byte offset in the cache, -1: none
  float4 scale[kSlots][kGroups];
  int64_t place[kSlots][kGroups];
  Item item[kItems];
  uint32_t tmem_base;
  int abort;
};

template <int D> struct Tc {
  static constexpr int kQ = kRowTile * D * 2;    // bytes of a row tile
  static constexpr int kK = kTok * D * 2;        // of a step's keys, or values
  static constexpr int kSmem = 2 * kQ + 4 * kK + 1024 + static_cast<int>(sizeof(Ctrl));
  // tensor memory columns: two score tiles, two outputs
  static constexpr int kS = 0, kO = 2 * kTok;
};

// Instruction descriptor of kind::f16 with f16 operands, both K-major, fp32
// accumulator: D format [4,6) = 1, N >> 3 in [17,23), M >> 4 in [24,29).
constexpr uint32_t idesc_f16(int M, int N) {
  return (1u << 4) | (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

// The upper half of desc_sw128's descriptors; the lower half holds the address.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);

// ACC 0: D = A B, 1: D += A B, 2: by `accumulate`.
template <int ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 da, db;\n setp.ne.b32 p, %4, 0;\n mov.b64 da, {%1, %5};\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n}\n" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(ACC == 2 ? accumulate : static_cast<uint32_t>(ACC)), "n"(kDescHigh)
      : "memory");
}

// A from tensor memory: row i in lane i, two f16 of consecutive K in a column.
template <int ACC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a_tmem, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 db;\n setp.ne.b32 p, %4, 0;\n mov.b64 db, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n}\n" ::"r"(d),
      "r"(a_tmem), "r"(b), "r"(idesc), "r"(ACC == 2 ? accumulate : static_cast<uint32_t>(ACC)), "n"(kDescHigh)
      : "memory");
}

// 16 consecutive fp32 columns of this thread's lane.  The values may be used
// after the wait; it names them, so that no use moves before it.
__device__ __forceinline__ void tmem_ld16_issue(uint32_t taddr, float (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld16_wait(float (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15])
               :
               : "memory");
}
// 32 consecutive fp32 columns of this thread's lane.  The values may be used
// after the wait; it names them, so that no use moves before it.
__device__ __forceinline__ void tmem_ld32_issue(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, "
      "%20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32_wait(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                 "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
                 "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
                 "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31])
               :
               : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const float (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20,"
      " %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]),
      "f"(v[8]), "f"(v[9]), "f"(v[10]), "f"(v[11]), "f"(v[12]), "f"(v[13]), "f"(v[14]), "f"(v[15]),
      "f"(v[16]), "f"(v[17]), "f"(v[18]), "f"(v[19]), "f"(v[20]), "f"(v[21]), "f"(v[22]), "f"(v[23]),
      "f"(v[24]), "f"(v[25]), "f"(v[26]), "f"(v[27]), "f"(v[28]), "f"(v[29]), "f"(v[30]), "f"(v[31])
      : "memory");
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// True in one lane of the (converged) warp, always the same one.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n" : "=r"(r));
  return r != 0;
}
template <int N> __device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N> __device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

__device__ __forceinline__ uint32_t f16x2_lo(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 t, u;\n mov.b32 {t, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t f16x2_hi(uint32_t w) {
  uint32_t r;
  asm("{\n .reg .b16 t, u;\n mov.b32 {t, u}, %1;\n cvt.rn.f16x2.e4m3x2 %0, u;\n}\n" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one instruction.
__device__ __forceinline__ uint64_t pair(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t v, float& x, float& y) { asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Weights 2^(score - m) of a 16-token group as f16 (s: its scales); their sum
// goes into the largest so far and, divided by the value scale, to `l`.
__device__ __forceinline__ float weigh(const float (&x)[16], const float4& s, float rf, float m, float* p, float& most,
                                       float l) {
  const float f = score_factor(s.x, rf), shift = s.y - m;
  const uint64_t f2 = pair(f, f), shift2 = pair(shift, shift);
  uint64_t sum = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float e0, e1;
    unpair(fma2(pair(x[2 * i], x[2 * i + 1]), f2, shift2), e0, e1);
    e0 = ex2(e0);
    e1 = ex2(e1);
    sum = add2(sum, pair(e0, e1));
    p[i] = __uint_as_float(pack_f16(e0, e1));
  }
  float sum0, sum1;
  unpair(sum, sum0, sum1);
  sum0 += sum1;
  most = fmaxf(most, sum0);
  return fmaf(sum0, s.z, l);
}

// The lowest n bits (n may be negative or over 32).
__device__ __forceinline__ uint32_t first_bits(int n) {
  return n <= 0 ? 0u : n >= 32 ? 0xffffffffu : (1u << n) - 1u;
}

// Waits for the phase of `bar` with the given parity, bounded like mbar_wait.
// A hand-over between two warps is on the critical path here, and a read of
// the wall clock takes longer than one: the limit is in cycles (about a second
// and a half) and is looked at now and then.
__device__ __forceinline__ bool wait_phase(uint64_t* bar, uint32_t parity, volatile int* abort) {
  const uint32_t at = smem_u32(bar);
  if (mbar_try_wait(at, parity)) return true;
  const long long t0 = clock64();
  for (uint32_t i = 1;; ++i) {
    if (mbar_try_wait(at, parity)) return true;
    if ((i & 63) == 0) {
      if (*abort) return false;
      if (clock64() - t0 > kWaitCycles) {
        *abort = 1;
        return false;
      }
    }
  }
}

// 16-byte chunk c of row r in a 128-byte-swizzled tile of 128-byte rows.
__device__ __forceinline__ uint32_t sw128(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

template <int D>
__global__ void __launch_bounds__(kThreads, 1) paged_attn_tc_kernel(PaArgs a) {
  using L = Tc<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Ctrl* c = reinterpret_cast<Ctrl*>(smem + 2 * L::kQ + 4 * L::kK);
  const uint32_t s_q = smem_u32(smem), s_k = s_q + 2 * L::kQ, s_v = s_k + 2 * L::kK;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort = &c->abort;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&c->q_full), 2 * kRowTile);
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&c->k_full[i]), kConvThreads);
      mbar_init(smem_u32(&c->v_full[i]), kConvThreads);
      mbar_init(smem_u32(&c->s_full[i][0]), 1);
      mbar_init(smem_u32(&c->s_full[i][1]), 1);
      mbar_init(smem_u32(&c->p_full[i]), kRowTile);
      mbar_init(smem_u32(&c->o_full[i]), 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&c->plan_full[i]), kGroups);
      mbar_init(smem_u32(&c->plan_free[i]), 1);
    }
    for (int i = 0; i < kItems; ++i) mbar_init(smem_u32(&c->item_full[i]), 1);
    mbar_init(smem_u32(&c->drain), 1);
    c->abort = 0;
    fence_barrier_init();
  }
  if (warp == 16) {
    tmem_alloc(smem_u32(&c->tmem_base), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  pdl_enter();
  const uint32_t tmem = c->tmem_base;
  // item k, once the planning warp has announced it
  auto next_item = [&](int k) { return wait_phase(&c->item_full[k % kItems], (k / kItems) & 1, abort); };

  if (warp < 8) {
    // ---------------------------------------------------------- softmax
    regs_up<kSoftmaxRegs>();
    const int tile = warp >> 2;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + lanes + L::kS + tile * kTok, t_o = tmem + lanes + L::kO + tile * D;
    // q travels in whole rows: D/8 neighbouring lanes have one, 16 bytes each
    constexpr int LPR = D / 8, RPI = 32 / LPR;   // lanes of a row, rows at a time
    const int lr = lane % LPR, lq = lane / LPR;
    // Rows of item `it` into the tile's q as f16, each scaled by a power of two;
    // returns this thread's row's factor for the scores.
    auto load_q = [&](const Item& it) {
      const int r = it.row0 + tile * kRowTile + (threadIdx.x & 127);
      int64_t mine = -1;   // element of this thread's row
      if (r < it.row0 + it.rows)
        mine = (it.token0 + r / a.group) * a.qs + static_cast<int64_t>(it.kvh * a.group + r % a.group) * D;
      static_assert(32 / RPI == LPR, "as many rows for a lane as lanes for a row");
      uint4 raw[LPR];
#pragma unroll
      for (int i = 0; i < LPR; ++i) {
        const int64_t at = __shfl_sync(0xffffffffu, mine, i * RPI + lq);
        raw[i] = at >= 0 ? __ldg(reinterpret_cast<const uint4*>(a.q + at + lr * 8)) : make_uint4(0, 0, 0, 0);
      }
      // The largest size of each row as bits (a NaN's are above infinity's).
      // LPR rows in LPR lanes: each exchange halves the rows that a lane keeps,
      // until lane lr has the maximum of its group's row lr.
      uint32_t top[LPR];
#pragma unroll
      for (int i = 0; i < LPR; ++i) {
        uint32_t x = __vmaxu2(raw[i].x & 0x7fff7fffu, raw[i].y & 0x7fff7fffu);
        x = __vmaxu2(x, __vmaxu2(raw[i].z & 0x7fff7fffu, raw[i].w & 0x7fff7fffu));
        top[i] = max(x & 0xffffu, x >> 16);
      }
#pragma unroll
      for (int half = LPR / 2; half > 0; half >>= 1) {
        const bool upper = lr & half;
#pragma unroll
        for (int i = 0; i < half; ++i) {
          const uint32_t keep = upper ? top[i + half] : top[i], give = upper ? top[i] : top[i + half];
          top[i] = max(keep, __shfl_xor_sync(0xffffffffu, give, half));
        }
      }
      const float factor = q_factor(__uint_as_float(top[0] << 16), top[0] < 0x7f80u);   // of row lr * RPI + lq
#pragma unroll
      for (int i = 0; i < LPR; ++i) {
        const float f = __shfl_sync(0xffffffffu, factor, lq * LPR + i);
        const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t h[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          h[e] = pack_f16(__uint_as_float(w[e] << 16) * f, __uint_as_float(w[e] & 0xffff0000u) * f);
        const int row = (warp & 3) * 32 + i * RPI + lq;
        sts128(s_q + tile * L::kQ + (lr / 8) * (kRowTile * 128) + sw128(row, lr % 8), h[0], h[1], h[2], h[3]);
      }
      const float rf = a.sm_scale * kLog2e / __shfl_sync(0xffffffffu, factor, (lane % RPI) * LPR + lane / RPI);
      fence_async();
      mbar_arrive(smem_u32(&c->q_full));
      return rf;
    };
    int g = 0;   // step, over all items
    bool ok = __all_sync(0xffffffffu, next_item(0));
    float rf = ok && c->item[0].rows > 0 ? load_q(c->item[0]) : 0.f;
#pragma unroll 1
    for (int k = 0; ok; ++k) {
      const Item& it = c->item[k % kItems];
      if (it.rows == 0) break;
      const Span sp = it.span(a);
      const int steps = it.steps, start = it.end - it.n;
      // this thread's row, and the first and last position of the warp's live rows
      const int w0 = it.row0 + tile * kRowTile + (warp & 3) * 32, r = w0 + lane;
      const int w1 = min(w0 + 31, it.row0 + it.rows - 1);
      const bool live = r <= w1;
      const int pos = live ? start + r / a.group : -1;
      const int pos_min = start + w0 / a.group, pos_max = start + max(w1, 0) / a.group;
      // a row that sees nothing at all needs no reference
      float m = pos >= 0 ? -INFINITY : 0.f, l = 0.f;
#pragma unroll 1
      for (int j = 0; j < steps; ++j, ++g) {
        const int slot = g % kSlots;
        ok = wait_phase(&c->s_full[tile][g & 1], (g >> 1) & 1, abort) &&
             wait_phase(&c->plan_full[slot], (g / kSlots) & 1, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const float4* sc = c->scale[slot];
        const int j0 = __float_as_int(sc[0].w);
        if (!sp.all_see(j0, j0 + kTok - 1, pos_min, pos_max)) {
          // scores that the row does not see become -infinity, in place: what
          // follows needs no mask
          const int hi = pos - j0, lo = sp.window ? hi - sp.window : INT_MIN, sink = sp.n_sink - j0;
#pragma unroll 1
          for (int q = 0; q < kTok; q += 32) {
            if (sp.all_see(j0 + q, j0 + q + 31, pos_min, pos_max)) continue;   // the same for the whole warp
            const uint32_t see = first_bits(hi + 1 - q) & (~first_bits(lo == INT_MIN ? 0 : lo + 1 - q) | first_bits(sink - q));
            float v[32];
            tmem_ld32_issue(t_s + q, v);
            tmem_ld32_wait(v);
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (!(see & (1u << i))) v[i] = -INFINITY;
            tmem_st32(t_s + q, v);
          }
          tmem_st_wait();
        }
        // Weights relative to the maximum so far, the scores read once.  A sum
        // that grows too large for f16, or a row without a maximum yet, takes the
        // maximum first and moves the accumulator to it.
        float p[2][32];   // f16 pairs: the first and the last 64 tokens
        float lnew = l;
        bool move = m == -INFINITY;
#pragma unroll 1
        for (int look = 0; look < 2; ++look) {
          if (__any_sync(0xffffffffu, move)) {
            float top = -INFINITY;
#pragma unroll 1
            for (int q = 0; q < kTok; q += 32) {
              float v[32];
              tmem_ld32_issue(t_s + q, v);
              tmem_ld32_wait(v);
              // one positive factor for a group: its largest product has the largest score
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                float u = fmaxf(v[16 * h], v[16 * h + 1]);
#pragma unroll
                for (int i = 2; i < 16; i += 2) u = fmaxf(u, fmaxf(v[16 * h + i], v[16 * h + i + 1]));
                const float4 s = sc[q / 16 + h];
                top = fmaxf(top, fmaf(u, score_factor(s.x, rf), s.y));
              }
            }
            const float to = move ? fmaxf(m, top - kRefBelow) : m, f = m == -INFINITY ? 0.f : ex2(m - to);
            m = to;
            l *= f;
            if (j > 0) {
              // the scores came after the product before: the accumulator is at rest
#pragma unroll 1
              for (int i = 0; i < D; i += 32) {
                float v[32];
                tmem_ld32_issue(t_o + i, v);
                tmem_ld32_wait(v);
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] *= f;
                tmem_st32(t_o + i, v);
              }
            }
          }
          lnew = l;
          const float ms = m == -INFINITY ? 0.f : m;
          float most = 0.f;
          float v[2][16];
          tmem_ld16_issue(t_s, v[0]);
          tmem_ld16_wait(v[0]);
#pragma unroll
          for (int h = 0; h < kGroups; ++h) {
            if (h + 1 < kGroups) tmem_ld16_issue(t_s + (h + 1) * 16, v[(h + 1) & 1]);
            lnew = weigh(v[h & 1], sc[h], rf, ms, p[h >> 2] + (h & 3) * 8, most, lnew);
            if (h + 1 < kGroups) tmem_ld16_wait(v[(h + 1) & 1]);
          }
          move = most > kMostSum;
          if (!__any_sync(0xffffffffu, move)) break;
        }
        l = lnew;
        tmem_st32(t_s, p[0]);
        tmem_st32(t_s + 32, p[1]);
        tmem_st_wait();
        tc_fence_before();
        mbar_arrive(smem_u32(&c->p_full[tile]));
      }
      if (!ok) break;
      // The next item's q goes in while the last product runs (the tile's q is
      // free: its last scores are there), so that its first scores are computed
      // beside this item's output.
      ok = __all_sync(0xffffffffu, next_item(k + 1));
      if (!ok) break;
      float rf_next = 0.f;
      if (c->item[(k + 1) % kItems].rows > 0) rf_next = load_q(c->item[(k + 1) % kItems]);
      ok = __all_sync(0xffffffffu, wait_phase(&c->o_full[tile], k & 1, abort));
      if (!ok) break;
      tc_fence_after();
      const bool cut = it.slot >= 0;
      const float f = cut ? 1.0f : l == 0.f ? 0.f : 1.0f / l;   // 0: nothing visible (a NaN sum is not)
      const int head = it.kvh * a.group + r % a.group, token = it.token0 + r / a.group;
      uint16_t* dst = a.out + static_cast<int64_t>(token) * a.os + static_cast<int64_t>(head) * D;
      float* part = a.tc_part + static_cast<int64_t>(it.slot) * (kTcItemRows * (D + 2));
      const int row = tile * kRowTile + (threadIdx.x & 127);
#pragma unroll 1
      for (int i = 0; i < D; i += 32) {
        float v[32];
        tmem_ld32_issue(t_o + i, v);
        tmem_ld32_wait(v);
        if (live && cut) {
#pragma unroll
          for (int q = 0; q < 32; q += 4)
            *reinterpret_cast<float4*>(part + row * D + i + q) = make_float4(v[q], v[q + 1], v[q + 2], v[q + 3]);
        } else if (live) {
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 y = __floats2bfloat162_rn(v[8 * q + 2 * e] * f, v[8 * q + 2 * e + 1] * f);
              w[e] = *reinterpret_cast<const uint32_t*>(&y);
            }
            *reinterpret_cast<uint4*>(dst + i + q * 8) = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (live && cut) *reinterpret_cast<float2*>(part + kTcItemRows * D + 2 * row) = make_float2(m, l);
      else if (live && a.lse) store_lse(a, token, head, m, l);
      tc_fence_before();
      rf = rf_next;
    }
  } else if (warp < 16) {
    // ---------------------------------------------------------- conversion
    regs_down<kConvRegs>();
    const int t = threadIdx.x & 127;
    const int64_t ts = a.c.token_stride;
    // walks the steps of all items; false: there are no more
    int k = -1, j = 0, g = -1, steps = 0, j0 = 0;
    bool all = false;
    Span sp = {};
    int64_t head_at = 0;
    auto next_step = [&] {
      ++g;
      if (++j >= steps) {
        if (!next_item(++k)) return false;
        const Item& it = c->item[k % kItems];
        if (it.rows == 0) return false;
        sp = it.span(a);
        steps = it.steps;
        head_at = it.kvh * a.c.head_stride;
        j = 0;
      }
      if (!wait_phase(&c->plan_full[g % kSlots], (g / kSlots) & 1, abort)) return false;
      j0 = __float_as_int(c->scale[g % kSlots][0].w);
      // every token of the step is seen by some row
      all = j0 + kTok <= sp.end && (j0 >= sp.lo || j0 + kTok <= sp.n_sink);
      return true;
    };
    if (warp < 12) {
      // keys: token (+ i KSTEP) and 16-byte chunk; eight neighbouring lanes have
      // four chunks of two rows, which the swizzle puts in eight banks
      constexpr int CPT = D / 16, KN = kTok * CPT / kConvThreads, KSTEP = kConvThreads / CPT;
      const int kc = D == 128 ? (t & 3) | ((t >> 1) & 4) : t & 3;
      const int kr = D == 128 ? ((t >> 2) & 1) | (t >> 4 << 1) : t >> 2;
      const uint8_t* mine = static_cast<const uint8_t*>(a.c.k) + (kr & 15) * ts + kc * 16;
      uint4 kw[KN];
      auto load = [&] {
        const uint8_t* from = mine + head_at;
#pragma unroll
        for (int i = 0; i < KN; ++i) {
          const int x = i * KSTEP + kr;
          const int64_t off = c->place[g % kSlots][x >> 4];
          kw[i] = make_uint4(0, 0, 0, 0);
          if (off >= 0 && (all || sp.seen(j0 + x))) kw[i] = __ldg(reinterpret_cast<const uint4*>(from + off));
        }
      };
      bool more = next_step();
      if (more) load();
#pragma unroll 1
      while (more) {
        // the stage is free when the scores of two steps before are there
        const int st = g & 1;
        if (g >= 2 && !wait_phase(&c->s_full[1][st], ((g - 2) >> 1) & 1, abort)) break;
        const uint32_t base = s_k + st * L::kK + (kc >> 2) * (kTok * 128);
#pragma unroll
        for (int i = 0; i < KN; ++i) {
          const int row = i * KSTEP + kr, c0 = (kc & 3) * 2;
          const uint4 w = kw[i];
          sts128(base + sw128(row, c0), f16x2_lo(w.x), f16x2_hi(w.x), f16x2_lo(w.y), f16x2_hi(w.y));
          sts128(base + sw128(row, c0 + 1), f16x2_lo(w.z), f16x2_hi(w.z), f16x2_lo(w.w), f16x2_hi(w.w));
        }
        fence_async();
        mbar_arrive(smem_u32(&c->k_full[st]));
        more = next_step();
        if (more) load();
      }
    } else {
      // values: 8 tokens (an octet of the warp's 32) by 4 elements; the lane's
      // bits are dealt so that eight neighbouring lanes store to eight banks
      constexpr int VN = D / 32;   // 32-byte column blocks
      const int vx = (lane & 1) | ((lane >> 3) << 1), vt = (warp & 3) * 32 + ((lane >> 1) & 3) * 8;
      const uint8_t* mine = static_cast<const uint8_t*>(a.c.v) + (vt & 15) * ts + vx * 4;
      uint32_t vw[VN][8];
      auto load = [&] {
        const int64_t off = c->place[g % kSlots][vt >> 4];
        const uint8_t* row = mine + head_at + off;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const bool there = off >= 0 && (all || sp.seen(j0 + vt + i));
#pragma unroll
          for (int d = 0; d < VN; ++d) {
            vw[d][i] = 0u;
            if (there) vw[d][i] = __ldg(reinterpret_cast<const uint32_t*>(row + d * 32));
          }
          row += ts;
        }
      };
      bool more = next_step();
      if (more) load();
#pragma unroll 1
      while (more) {
        // the stage is free when the products of two steps before are done, which
        // the scores of one step before say; both softmax tiles are past that
        // step then, and its plan is free
        const int st = g & 1;
        if (g >= 2) {
          if (!wait_phase(&c->s_full[1][st ^ 1], ((g - 1) >> 1) & 1, abort)) break;
          if (t == 0) mbar_arrive(smem_u32(&c->plan_free[(g - 2) % kSlots]));
        }
        const uint32_t base = s_v + st * L::kK + (vt >> 6) * (D * 128);
        const int ch = (vt & 63) >> 3;
#pragma unroll
        for (int d = 0; d < VN; ++d) {
          uint32_t lo[4], hi[4];   // token pairs of elements 0,1 and 2,3
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            lo[i] = __byte_perm(vw[d][2 * i], vw[d][2 * i + 1], 0x5140);
            hi[i] = __byte_perm(vw[d][2 * i], vw[d][2 * i + 1], 0x7362);
          }
          const int row = d * 32 + vx * 4;
          sts128(base + sw128(row, ch), f16x2_lo(lo[0]), f16x2_lo(lo[1]), f16x2_lo(lo[2]), f16x2_lo(lo[3]));
          sts128(base + sw128(row + 1, ch), f16x2_hi(lo[0]), f16x2_hi(lo[1]), f16x2_hi(lo[2]), f16x2_hi(lo[3]));
          sts128(base + sw128(row + 2, ch), f16x2_lo(hi[0]), f16x2_lo(hi[1]), f16x2_lo(hi[2]), f16x2_lo(hi[3]));
          sts128(base + sw128(row + 3, ch), f16x2_hi(hi[0]), f16x2_hi(hi[1]), f16x2_hi(hi[2]), f16x2_hi(hi[3]));
        }
        fence_async();
        mbar_arrive(smem_u32(&c->v_full[st]));
        more = next_step();
        if (more) load();
      }
    }
  } else {
    regs_down<kIssueRegs>();
    if (warp == 17) {
      // -------------------------------------------------------- planning
      // Takes items from the list as they come (the longest first; which CTA
      // works on one does not matter to its results), announces them, and looks
      // up their steps: four at a time, a lane for each 16-token group: page id,
      // place in the cache, scales.
      constexpr int kNotSeen = INT_MIN;
      const int ps = a.c.page_size, ps_log = 31 - __clz(ps), grp = lane & 7;
      const int total = a.tc->entries * a.c.n_kv_heads;
      bool ok = true;
      int g = 0;
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        int at = lane == 0 ? atomicAdd(&a.tc->taken, 1) : 0;
        at = __shfl_sync(0xffffffffu, at, 0);
        Item it = {};
        if (at < total) {
          const TcEntry e = a.tc_entries[at / a.c.n_kv_heads];
          const Request rq = load_request(a.cu, a.kv_len, e.b, a.T);
          it.b = e.b;
          it.kvh = at % a.c.n_kv_heads;
          it.token0 = rq.row0;
          it.n = rq.n;
          it.end = rq.end;
          it.row0 = e.blk * kTcItemRows;
          it.rows = min(kTcItemRows, rq.n * a.group - it.row0);
          const int64_t units = it.span(a).units;
          it.u0 = static_cast<int>(units * e.part / e.parts);
          it.steps = static_cast<int>(units * (e.part + 1) / e.parts) - it.u0;
          it.slot = e.parts > 1 ? (e.slot + e.part) * a.c.n_kv_heads + it.kvh : -1;
        }
        if (lane == 0) {
          c->item[k % kItems] = it;
          mbar_arrive(smem_u32(&c->item_full[k % kItems]));
        }
        if (it.rows == 0) break;
        const Span sp = it.span(a);
        const int32_t* table = a.c.page_table + static_cast<int64_t>(it.b) * a.c.max_pages;
#pragma unroll 1
        for (int jb = 0; ok && jb < it.steps; jb += 4) {
          const int j = jb + (lane >> 3), s = g + j, slot = s % kSlots;
          const bool mine = j < it.steps;
          const int x = mine ? sp.block_of(it.u0 + j) * kTok + grp * 16 : 0;
          // any negative id as -1: the table may hold kNotSeen's value
          const int gp = mine && sp.any_seen(x, x + 15) ? max(__ldg(table + (x >> ps_log)), -1) : kNotSeen;
          const bool have = static_cast<unsigned>(gp) < static_cast<unsigned>(a.c.n_pages);
          if (!have && gp != kNotSeen) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
          float ks = 0.f, vs = 1.f;
          if (have) {
            const int64_t sa = static_cast<int64_t>(gp) * a.c.n_kv_heads + it.kvh;
            ks = __ldg(a.c.k_scale + sa);
            vs = __ldg(a.c.v_scale + sa);
          }
          if (mine && s >= kSlots) ok = wait_phase(&c->plan_free[slot], ((s / kSlots) - 1) & 1, abort);
          ok = __all_sync(0xffffffffu, ok);
          if (mine && ok) {
            // a group without a page masks itself
            c->place[slot][grp] = have ? gp * a.c.page_stride + (x & (ps - 1)) * a.c.token_stride : -1;
            c->scale[slot][grp] = have ? make_float4(ks, __log2f(vs), __frcp_rn(vs), __int_as_float(x))
                                       : make_float4(1.f, -INFINITY, 0.f, __int_as_float(x));
            mbar_arrive(smem_u32(&c->plan_full[slot]));
          }
        }
        g += it.steps;
      }
    }
    // ---------------------------------------------------------- MMA issue
    // The whole warp walks the loop, so that descriptors stay in uniform
    // registers (per-thread ones cost an MMA's time to move); one lane issues.
    if (warp == 16) {
      constexpr uint32_t is = idesc_f16(kRowTile, kTok), io = idesc_f16(kRowTile, D);
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
      // descriptors of the first tile and stage; the others lie a multiple of
      // the operand's size (in 16-byte units) behind
      auto low = [](uint32_t saddr) { return static_cast<uint32_t>(desc_sw128(saddr)); };
      const uint32_t dq = low(s_q), dk = low(s_k), dv = low(s_v);
      auto wait = [&](uint64_t* bar, uint32_t parity) {
        return __all_sync(0xffffffffu, wait_phase(bar, parity, abort)) != 0;
      };
      auto scores = [&](int tile, int st) {   // st: step & 1
        const uint32_t da = dq + tile * (L::kQ >> 4), db = dk + st * (L::kK >> 4);
        const uint32_t d = tm + L::kS + tile * kTok;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < D / 16; ++i) {
            const int o = (i >> 2) * (kRowTile * 128 >> 4) + 2 * (i & 3);   // 128-byte column block, 32-byte step
            if (i == 0) mma_ss<0>(d, da + o, db + o, is, 0);
            else mma_ss<1>(d, da + o, db + o, is, 1);
          }
          mma_commit(smem_u32(&c->s_full[tile][st]));
        }
        __syncwarp();
      };
      auto output = [&](int tile, int st, bool first) {
        const uint32_t db = dv + st * (L::kK >> 4);
        const uint32_t d = tm + L::kO + tile * D, p = tm + L::kS + tile * kTok;
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < kTok / 16; ++i) {
            const int o = (i >> 2) * (D * 128 >> 4) + 2 * (i & 3);
            if (i == 0) mma_ts<2>(d, p, db + o, io, !first);
            else mma_ts<1>(d, p + i * 8, db + o, io, 1);
          }
        }
        __syncwarp();
      };
      auto commit = [&](uint64_t* bar) {
        if (elect_one()) mma_commit(smem_u32(bar));
        __syncwarp();
      };
      int g = 0;   // step, over all items
      bool ok = true;
#pragma unroll 1
      for (int k = 0; ok; ++k) {
        if (!(ok = __all_sync(0xffffffffu, next_item(k)))) break;
        const Item& it = c->item[k % kItems];
        if (it.rows == 0) break;
        const int steps = it.steps;
        if (!(ok = wait(&c->q_full, k & 1) && wait(&c->k_full[g & 1], (g >> 1) & 1))) break;
        tc_fence_after();
        scores(0, g & 1);
        scores(1, g & 1);
#pragma unroll 1
        for (int j = 0; j < steps; ++j, ++g) {
          const int st = g & 1, nst = st ^ 1;
          const bool more = j + 1 < steps;
          if (!(ok = wait(&c->v_full[st], (g >> 1) & 1))) break;
#pragma unroll 1
          for (int tile = 0; tile < 2; ++tile) {
            if (!(ok = wait(&c->p_full[tile], g & 1))) break;
            tc_fence_after();
            output(tile, st, j == 0);
            if (!more) {
              commit(&c->o_full[tile]);
            } else {
              if (tile == 0 && !(ok = wait(&c->k_full[nst], ((g + 1) >> 1) & 1))) break;
              tc_fence_after();
              scores(tile, nst);
            }
          }
          if (!ok) break;
        }
      }
      // nothing is in flight when the tensor memory goes back
      commit(&c->drain);
      int no_abort = 0;
      mbar_wait(smem_u32(&c->drain), 0, &no_abort, kDrainNs);
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (threadIdx.x == 0 && c->abort) set_status(a.status, MOE_ERR_DEVICE_TIMEOUT);
  if (warp == 16) tmem_dealloc(tmem, 512);
}

// Joins the parts of cut row blocks, a warp for each row, in the parts' order.
template <int D>
__global__ void __launch_bounds__(256) paged_attn_tc_join(PaArgs a) {
  constexpr int VEC = D / 64;   // pairs of columns of a lane
  pdl_enter();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t groups = static_cast<int64_t>(a.tc->joins) * a.c.n_kv_heads * (kTcItemRows / 8);
  for (int64_t x = blockIdx.x; x < groups; x += gridDim.x) {
    const int row = static_cast<int>(x % (kTcItemRows / 8)) * 8 + warp;
    const int kvh = static_cast<int>(x / (kTcItemRows / 8) % a.c.n_kv_heads);
    const TcJoin jn = a.tc_joins[x / (kTcItemRows / 8) / a.c.n_kv_heads];
    const Request rq = load_request(a.cu, a.kv_len, jn.b, a.T);
    const int r = jn.blk * kTcItemRows + row;
    if (r >= rq.n * a.group) continue;
    auto part_of = [&](int k) {
      return a.tc_part + (static_cast<int64_t>(jn.slot + k) * a.c.n_kv_heads + kvh) * (kTcItemRows * (D + 2));
    };
    float m = -INFINITY, sum = 0.f;
    float2 acc[VEC] = {};
    for (int k0 = 0; k0 < jn.parts; k0 += 32) {
      float2 ml = make_float2(-INFINITY, 0.f);
      if (k0 + lane < jn.parts) ml = *reinterpret_cast<const float2*>(part_of(k0 + lane) + kTcItemRows * D + 2 * row);
      float to = fmaxf(m, ml.x);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) to = fmaxf(to, __shfl_xor_sync(0xffffffffu, to, off));
      const float old = ex2_from(m, to), w = ex2_from(ml.x, to);
      m = to;
      float l = ml.y * w;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) l += __shfl_xor_sync(0xffffffffu, l, off);
      sum = sum * old + l;
#pragma unroll
      for (int e = 0; e < VEC; ++e) acc[e] = make_float2(acc[e].x * old, acc[e].y * old);
#pragma unroll 4
      for (int k = k0; k < min(jn.parts, k0 + 32); ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k - k0);
        const float2* p = reinterpret_cast<const float2*>(part_of(k) + row * D) + lane;
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float2 v = p[e * 32];
          acc[e].x += v.x * wk;
          acc[e].y += v.y * wk;
        }
      }
    }
    const int token = rq.row0 + r / a.group, head = kvh * a.group + r % a.group;
    const float f = sum == 0.f ? 0.f : 1.0f / sum;   // nothing visible (a NaN sum is not)
    __nv_bfloat162* out =
        reinterpret_cast<__nv_bfloat162*>(a.out + static_cast<int64_t>(token) * a.os + static_cast<int64_t>(head) * D);
#pragma unroll
    for (int e = 0; e < VEC; ++e) out[e * 32 + lane] = __floats2bfloat162_rn(acc[e].x * f, acc[e].y * f);
    if (a.lse && lane == 0) store_lse(a, token, head, m, sum);
  }
}

template <int D>
cudaError_t launch(const PaArgs& a, cudaStream_t s) {
  cudaError_t err = ensure_kernel_attrs(reinterpret_cast<const void*>(paged_attn_tc_kernel<D>), Tc<D>::kSmem);
  if (err != cudaSuccess) return err;
  count_launches(a.tc_split ? 2 : 1);
  err = launch_pdl(paged_attn_tc_kernel<D>, a.tc_ctas, kThreads, Tc<D>::kSmem, s, a);
  if (err != cudaSuccess || !a.tc_split) return err;
  return launch_pdl(paged_attn_tc_join<D>, 4 * a.tc_ctas, 256, 0, s, a);
}

}  // namespace

bool paged_attn_tc_supported(int D) { return D == 64 || D == 128; }

cudaError_t launch_paged_attn_tc(const PaArgs& a, cudaStream_t s) {
  return a.c.head_dim == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace moe
