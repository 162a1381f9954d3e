// What the attention kernels for few query rows share, over the paged caches of
// 8 bits (paged_attn.cu) and of 4 (block_attn.cu): the cut of the work into
// pieces, the list of the row blocks that go to paged_attn_tc.cuh, the join of
// partial sums, the choice of kernels and the call.
//
// The rows of one (request, key head) are its new tokens times the query
// heads of the group, row r = token r / group, head r % group; 8 or 16 rows make
// a row tile.  The work of a row tile is cut into units of cached tokens, 64 over the
// 8-bit cache and 128 over the other.  All units of the call stand in one line
// (request, key head, row tile, token), and the persistent CTAs take equal pieces of
// that line, so a batch of mixed lengths keeps every SM busy to the end.  A piece
// may end inside a row tile; then all its CTAs leave partial sums, which
// paged_attn_join or block_attn_join adds in order (a fixed order: the same bits
// every time).  Over the 4-bit cache row tiles of short contexts are not cut
// (kWholeTokens): a CTA has those that begin in its piece, and nothing is joined.
#pragma once

#include <climits>

#include "paged_kv.cuh"
#include "tc_ptx.cuh"
#include "paged_attn.cuh"

namespace moe {

bool paged_attn_tc_supported(int D);
cudaError_t launch_paged_attn_tc(const PaArgs& a, cudaStream_t s);
cudaError_t launch_paged_attn_tc(const BlockPaArgs& a, cudaStream_t s);

namespace {

constexpr int kWarps = 4;
constexpr float kLog2e = 1.4426950408889634f;

// D: elements of a head, NB: blocks of eight rows in a row tile.  A stage of a
// warp's ring holds one tile of 16 tokens, with codes of four bits (BLOCKS) two.
template <int D, int NB, bool BLOCKS> struct Shape {
  static constexpr int kRows = 8 * NB;
  static constexpr int kUnit = BLOCKS ? 128 : 64;         // tokens of a unit, in equal parts for the four warps
  // What a row tile costs beside its units (finding it, q, the join of the
  // warps), in units.
  static constexpr int kTileCost = 4;
  static constexpr int kTile = BLOCKS ? 8 * D : 16 * D;   // bytes of 16 tokens' keys (or values)
  static constexpr int kStage = BLOCKS ? 4 * kTile + 4 * D : 2 * kTile;
  // CTAs on an SM, by registers (O takes D NB / 4 of a thread's, q D NB / 8),
  // and the stages of the ring that fit then
  static constexpr int kCtas = BLOCKS ? (D * NB == 64 ? 4 : D * NB == 128 ? 3 : 2)
                                      : D * NB == 64 ? 5 : D * NB == 128 ? 4 : D * NB == 256 ? 3 : 2;
  static constexpr int kStages = BLOCKS ? 2 : D == 256 ? 2 : D * NB == 128 && D == 128 ? 3 : 4;
  static constexpr int kRing = kStages * kStage;        // per warp
  static constexpr int kPart = kRows * D + 2 * kRows;   // floats of a partial: outputs, references, sums
  static_assert(kRing >= kRows * D * 4, "a warp's outputs are joined in its ring");
};

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes, or zeros when !valid (the source is not read then).
__device__ __forceinline__ void cp16_or_zero(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? 16 : 0;
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void cp4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
// N bytes (4, 8 or 16), or zeros when !valid.
template <int N> __device__ __forceinline__ void cp_or_zero(uint32_t dst, const void* src, bool valid) {
  const int n = valid ? N : 0;
  if constexpr (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(N) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

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
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// An 8x8 block of f16, a row in four lanes (two columns each), transposed.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// Lists the row blocks of the requests that go to paged_attn_tc.cuh, the longest
// first (a counting sort by 256 classes of length; the order inside a class
// does not matter to the results).  Where that is allowed, a block longer than
// 1.5 times a CTA's share of the work is cut along the cached tokens into parts
// of at least 3/4 of that share.  One thread block; `first`: B + 1 ints, `scratch`: the
// block's other shared memory.
__device__ __noinline__ void list_tc_items(const PaArgs& a, int* first, char* scratch) {
  int* bins = reinterpret_cast<int*>(scratch);            // [256]
  int* s_max = bins + 256;
  unsigned long long* s_sum = reinterpret_cast<unsigned long long*>(bins + 258);
  TcList* s_list = reinterpret_cast<TcList*>(bins + 260);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __shared__ int s_warp[32];
  for (int i = threadIdx.x; i < 256; i += blockDim.x) bins[i] = 0;
  if (threadIdx.x == 0) {
    *s_max = 0;
    *s_sum = 0;
    *s_list = TcList{};
  }
  __syncthreads();
  auto blocks_of = [&](const Request& r) { return r.n * a.group > a.tc_rows ? ceil_div(r.n * a.group, kTcItemRows) : 0; };
  auto length = [&](const Request& r, int blk) {
    const int row0 = blk * kTcItemRows, row1 = min(row0 + kTcItemRows, r.n * a.group) - 1;
    return span_for(a, r.start + row0 / a.group, r.start + row1 / a.group, kTcStep).units;
  };
  int64_t base = 0;
  for (int b0 = 0; b0 < a.B; b0 += blockDim.x) {
    const int b = b0 + threadIdx.x;
    int n = 0;
    if (b < a.B) {
      const Request r = load_request(a.cu, a.kv_len, b, a.T);
      if (!r.ok || r.end > a.c.max_pages * a.c.page_size) set_status(a.status, MOE_ERR_DEVICE_BOUNDS);
      n = blocks_of(r);
      if (n > 0) atomicMax(s_max, length(r, n - 1));
    }
    int sum = n;
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, sum, off);
      if (lane >= off) sum += x;
    }
    if (lane == 31) s_warp[warp] = sum;
    __syncthreads();
    int all = 0, below = 0;
    for (int w = 0; w < static_cast<int>(blockDim.x / 32); ++w) {
      all += s_warp[w];
      below += w < warp ? s_warp[w] : 0;
    }
    if (b < a.B) first[b] = static_cast<int>(min(base + below + sum - n, static_cast<int64_t>(INT_MAX)));
    base += all;
    __syncthreads();
  }
  // offsets out of order can name rows twice; the list has room for them once
  const int total = static_cast<int>(min(base, tc_places(a)));
  const int64_t widest = *s_max + 1;
  auto look = [&](int i, int& b, int& blk) {   // the i-th block; its length
    int lo = 0, hi = a.B - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (first[mid] <= i) lo = mid; else hi = mid - 1;
    }
    b = lo;
    blk = i - first[lo];
    return length(load_request(a.cu, a.kv_len, b, a.T), blk);
  };
  int b, blk;
  int64_t share = INT_MAX;   // steps of a part
  if (a.tc_split) {
    unsigned long long sum = 0;
    for (int i = threadIdx.x; i < total; i += blockDim.x) sum += look(i, b, blk);
    atomicAdd(s_sum, sum);
    __syncthreads();
    share = max(int64_t(4), static_cast<int64_t>(*s_sum * a.c.n_kv_heads + a.tc_ctas - 1) / a.tc_ctas);
  }
  // rounded down: with equal blocks, the parts then are no more than the CTAs
  auto parts_of = [&](int units) {
    return 2 * int64_t(units) <= 3 * share ? 1 : max(2, static_cast<int>(units / share));
  };
  auto class_of = [&](int units, int parts) {
    return 255 - static_cast<int>(min(static_cast<int64_t>(255), static_cast<int64_t>(units / parts) * 256 / widest));
  };
  for (int i = threadIdx.x; i < total; i += blockDim.x) {
    const int units = look(i, b, blk), parts = parts_of(units);
    atomicAdd(&bins[class_of(units, parts)], parts);
  }
  __syncthreads();
  if (warp == 0) {   // exclusive prefix over the classes
    int sum = 0, mine[8];
    for (int i = 0; i < 8; ++i) {
      mine[i] = sum;
      sum += bins[lane * 8 + i];
    }
    int before = sum;
    for (int off = 1; off < 32; off <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, before, off);
      if (lane >= off) before += x;
    }
    before -= sum;
    for (int i = 0; i < 8; ++i) bins[lane * 8 + i] = before + mine[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < total; i += blockDim.x) {
    const int units = look(i, b, blk), parts = parts_of(units);
    const int at = atomicAdd(&bins[class_of(units, parts)], parts);
    atomicAdd(&s_list->entries, parts);
    int slot = -1;
    if (parts > 1) {
      slot = atomicAdd(&s_list->slots, parts);
      a.tc_joins[atomicAdd(&s_list->joins, 1)] = TcJoin{b, blk, parts, slot};
    }
    for (int k = 0; k < parts; ++k) a.tc_entries[at + k] = TcEntry{b, blk, k, parts, slot};
  }
  __syncthreads();
  if (threadIdx.x == 0) *a.tc = *s_list;
  __syncthreads();
}

// The list alone, for a batch that has no small requests.
__global__ void __launch_bounds__(512) list_kernel(PaArgs a) {
  extern __shared__ __align__(128) char smem[];
  pdl_enter();
  list_tc_items(a, reinterpret_cast<int*>(smem + 2048), smem);
}

// The workspace is sized for kMaxSms SMs, so that its size needs no device.
constexpr int kMaxCtas = kMaxSms * 5;

// Persistent CTAs: what the SMs hold at once.
template <int D, int NB, bool BLOCKS> int ctas_for(int num_sms) {
  return std::min(num_sms, kMaxSms) * Shape<D, NB, BLOCKS>::kCtas;
}

// Kernels: a type whose of<D, NB>() is the few-row kernel, and whose join<D, NB>()
// launches the join of what its CTAs leave.
template <int D, int NB, class Kernels, class Args>
cudaError_t launch(const Args& a, int num_sms, cudaStream_t s) {
  using S = Shape<D, NB, Args::kBlocks>;
  const size_t smem = kWarps * S::kRing + sizeof(int64_t) * (a.B + 1);
  const auto kernel = Kernels::template of<D, NB>();
  cudaError_t err = ensure_kernel_attrs(reinterpret_cast<const void*>(kernel), static_cast<int>(smem));
  if (err != cudaSuccess) return err;
  const int ctas = ctas_for<D, NB, Args::kBlocks>(num_sms);
  bool join = true;
  if constexpr (Args::kBlocks) join = !a.whole_tiles;
  count_launches(1 + join);
  err = launch_pdl(kernel, ctas, kWarps * 32, smem, s, a);
  if (err != cudaSuccess || !join) return err;
  return Kernels::template join<D, NB>(a, ctas, s);
}

// Row tiles of eight where no request has more rows: half the registers, more
// warps (eight rows, tiles of eight / sixteen: 64 requests at 17 to 3712 tokens
// 33 / 41 us, 12 at about 57000 115 / 150 us).  With more rows, tiles of sixteen
// convert the codes half as often (64 requests of 32 rows at 3584 117 / 92 us).
template <int D, class Kernels, class Args>
cudaError_t launch(const Args& a, int64_t most_rows, int num_sms, cudaStream_t s) {
  if constexpr (D < 256) {
    if (most_rows > 8) return launch<D, 2, Kernels>(a, num_sms, s);
  }
  return launch<D, 1, Kernels>(a, num_sms, s);
}

template <int D, int NB, bool BLOCKS> size_t part_bytes() {
  return static_cast<size_t>(ctas_for<D, NB, BLOCKS>(kMaxSms)) * 2 * Shape<D, NB, BLOCKS>::kPart * sizeof(float);
}

template <bool BLOCKS> size_t part_bytes_of(int D) {
  switch (D) {
    case 64: return std::max(part_bytes<64, 1, BLOCKS>(), part_bytes<64, 2, BLOCKS>());
    case 128: return std::max(part_bytes<128, 1, BLOCKS>(), part_bytes<128, 2, BLOCKS>());
    default: return part_bytes<256, 1, BLOCKS>();
  }
}

// Which kernels a call takes, from what the host knows.
struct Path {
  bool tc;      // the tcgen05 kernel, for requests with more than kTcRows rows
  bool alone;   // ... and it alone
  bool split;   // ... which may cut row blocks along the cached tokens
};

// The few-row kernel reads a request's tokens once for every 16 rows (8 where D =
// 256), the tcgen05 kernel once for 256, but takes longer to start and to join: with heads of 128
// about 13 us + 3.1 us for a million pairs of a row and a token (a row tile's
// start counting as kTileTokens tokens) against 29 us + 0.6 us.
// Measured (us, few-row / tcgen05): one request of 1024 rows (of all key heads)
// at 3584 tokens 25 / 33, at 8192 40 / 37, at 16384 65 / 44, at 65536 221 / 67; of
// 512 rows at 8192 27 / 34, at 65536 118 / 63; of 256 rows at 65536 66 / 63; 2048 rows
// of 1 / 8 requests at 3584 37 / 34 and 31 / 37; 64 requests of 32 rows each (8192)
// at 1792 to 3584 94 / 115, of 64 rows 167 / 113; 125 prompts of up to 26 tokens, 8
// x 7 heads, at 40 to 49 tokens 112 / 69.  These are with page tables as wide as
// the longest request.
//
// The host does not know the lengths: the page table's width stands for them, up
// to kTcTokens, since a wide table may be a short one's.  With a table of 131072
// tokens (us, few-row / tcgen05; *: the rule takes the slower), 4 x 8 heads: 32 new
// tokens at 512 18 / 34*, at 2048 25 / 38*, at 4096 31 / 41*; 64 new tokens at 512
// 23 / 34*, at 4096 45 / 40; 16 at 4096 25 / 38*; 4 x 32 at 1024 33 / 40*; and where
// the table is as long as it is wide: 8 new tokens at 131072 122* / 100, 10 150* / 100,
// 12 172 / 100, 16 224 / 101.  A lower limit would trade the first against these.
//
// Cutting row blocks along the tokens adds a launch for their join and pays where
// one block is longer than a CTA's share of the work.  Measured (us, not cut / cut;
// 4 x 8 x 128; places: row blocks and requests, times key heads):
//   512 new tokens at 4096 (68 places) 81 / 69, 1024 (132) 82 / 87, 2048 (260) 119 /
//   126; 512 at 32768 beside 8 x 256 at 512 (356) 520 / 308; 256 at 65536 beside 16 x
//   256 at 512 (612) 978 / 314, at 16384 266 / 153, at 8192 147 / 122; equal requests
//   8 x 512 at 3584 (544) 242 / 251, 16 x 256 (576) 254 / 263;
//   above the limit: 18 x 256 at 256 to 3584 (648) 159 / 169, 32 x 256 (1152) 266 / 280,
//   but 256 at 16384 beside 24 x 256 (900) 271 / 179, at 65536 beside 40 (1476) 1000 /
//   426.
// A call that gains nothing loses up to 10 us, one long request among short ones
// gains several times that; more places make the second rarer, so that cutting is
// allowed up to 4 kMaxSms of them.  The device then cuts what is longer than 1.5
// shares (2 instead of 1.5: the same times to 1 us, with 8 x 512 at 3584, 4 x 1024 at
// 32768, 2 x 2048 at 4096 to 65536, 3 x 512 at 2048 to 16384).
//
// Over the cache in 4 bits the few-row kernel is faster by what it reads less.
// Measured (us, few-row / tcgen05; 4 x 8 x 128): 32 new tokens at 3584 20.7 / 32.1, at
// 8192 (8.2 million pairs) 30.7 / 36.3, at 16384 47.2 / 43.1, at 65536 147 / 72; 64 at 3584
// (7.5) 29.4 / 33.0; 256 at 1024 (10) 38.5 / 34.8; 16 x 16 at 3584 79.8 / 61.5; 64
// requests of 64 rows each at 3584 151 / 159, at 1024 66 / 61; 256 of 64 rows at 40 108 /
// 62, at 300 146 / 103; 8 x 1 x 128: 256 of 40 rows at 60 127 / 134, 64 of 20 at 1000 60 / 110.
constexpr int kTileTokens = 256;
constexpr int kTcRows = 48;   // of a request and key head
template <bool BLOCKS> constexpr int64_t kTcWork = BLOCKS ? int64_t(9) << 20 : int64_t(6) << 20;   // pairs
constexpr int kTcTokens = 16384;

// Over the cache in 4 bits the few-row kernel cuts no row tiles where its rows see
// at most kWholeTokens, as far as the host knows: cutting spreads a few units over
// more CTAs, but the join is a launch.  Measured (us, cut / whole, queued; one new
// token, 4 x 8 x 128): 1 request at up to 128 7.4 / 5.3, at 512 7.8 / 7.7, at 1024 8.0 / 10.8;
// 100 at 64 to 128 9.8 / 8.6, at 256 13.7 / 9.9, at 512 16.0 / 12.5, at 1024 20.3 / 20.8, at
// 2048 28.4 / 31.6; 128 (512 row tiles for 456 CTAs) 12.8 / 12.2, 16.3 / 14.4, 19.1 / 18.3, 23.7 /
// 25.0, 34.1 / 41.1.
// The better side depends on the number of row tiles too, which the rule does not
// look at: with few, or a little over what the CTAs take at once, cutting gains from
// 256 tokens on.  Measured in a window (us, cut / whole, in a graph; *: the rule takes
// the slower): one new token, 8 x 4 x 64, 32 tiles in 128 tokens 8.3 / 8.0, 256 8.2 / 8.7*,
// 512 8.8 / 9.8*, 1024 9.3 / 12.9; 384 tiles 12.5 / 10.2, 13.5 / 11.3, 15.3 / 13.4, 18.5 / 18.2*;
// 768 tiles 17.1 / 15.9, 18.8 / 17.9, 21.8 / 22.1*, 27.5 / 30.5; four (16 rows), 384 tiles
// 15.3 / 11.7, 17.0 / 12.7, 19.1 / 15.0, 22.9 / 19.5*; one, 4 x 8 x 128, 16 tiles 8.6 / 8.7*,
// 8.4 / 9.4*, 8.9 / 11.1*, 9.3 / 14.3; 192 tiles 12.9 / 10.7, 14.1 / 12.0, 15.3 / 14.6, 17.4 /
// 20.2; 2 x 8 x 256, 8 tiles 9.6 / 10.3*, 9.4 / 11.6*, 9.8 / 13.9*, 10.7 / 18.5; 192 tiles
// 15.3 / 12.6, 16.8 / 14.3, 19.9 / 17.6, 24.3 / 24.4.
constexpr int kWholeTokens = 512;

// Cached tokens that a request's rows can see, as far as the host knows.
inline int64_t most_tokens(const PaArgs& a, int max_q_len) {
  const int64_t all = static_cast<int64_t>(a.c.max_pages) * a.c.page_size;
  const int64_t n = max_q_len > 0 ? std::min(max_q_len, a.T) : a.T;
  return a.window ? std::min(all, n + a.window + a.n_sink) : all;
}

template <bool BLOCKS>
Path path_of(const PaArgs& a, int max_q_len) {
  const int64_t most = static_cast<int64_t>(max_q_len > 0 ? std::min(max_q_len, a.T) : a.T) * a.group;
  Path p;
  const int64_t rows = static_cast<int64_t>(a.T) * a.group * a.c.n_kv_heads;
  const int64_t tokens = std::min<int64_t>(static_cast<int64_t>(a.c.max_pages) * a.c.page_size, kTcTokens);
  p.tc = most > kTcRows && rows * (tokens + kTileTokens) >= kTcWork<BLOCKS> && paged_attn_tc_supported(a.c.head_dim);
  // As many rows as if every request had max_q_len of them: they all do (or the
  // hint is wrong, and the tcgen05 kernel takes small ones too).
  p.alone = p.tc && static_cast<int64_t>(max_q_len) * a.B == a.T;
  p.split = p.tc && tc_places(a) * a.c.n_kv_heads <= 4 * kMaxSms;
  return p;
}

// At most kMaxBatch requests: the tables of the requests are in shared memory.
template <class Kernels, class Args>
cudaError_t launch_requests(const Args& a, const Path& path, int max_q_len, int num_sms, cudaStream_t s) {
  const int64_t most = static_cast<int64_t>(max_q_len > 0 ? std::min(max_q_len, a.T) : a.T) * a.group;
  cudaError_t err;
  if (path.alone) {
    count_launches(1);
    err = launch_pdl(list_kernel, 1, 512, 2048 + sizeof(int) * (a.B + 1), s, static_cast<const PaArgs&>(a));
  } else {
    switch (a.c.head_dim) {
      case 64: err = launch<64, Kernels>(a, std::min<int64_t>(most, a.tc_rows), num_sms, s); break;
      case 128: err = launch<128, Kernels>(a, std::min<int64_t>(most, a.tc_rows), num_sms, s); break;
      default: err = launch<256, Kernels>(a, most, num_sms, s); break;
    }
  }
  return err == cudaSuccess && path.tc ? launch_paged_attn_tc(a, s) : err;
}

// Larger batches in slices of kMaxBatch requests, one after the other (the rows
// of a request are where cu says, so that only the requests' arrays move on).
template <class Kernels, class Args>
cudaError_t launch_paged_attn(Args a, int max_q_len, int num_sms, cudaStream_t s) {
  const Path path = path_of<Args::kBlocks>(a, max_q_len);
  a.tc_rows = path.alone ? 0 : path.tc ? kTcRows : INT_MAX;
  a.tc_ctas = std::min(num_sms, kMaxSms);
  a.tc_split = path.split;
  if constexpr (Args::kBlocks) a.whole_tiles = most_tokens(a, max_q_len) <= kWholeTokens;
  cudaError_t err = cudaSuccess;
  for (int left = a.B; left > 0 && err == cudaSuccess; left -= kMaxBatch) {
    a.B = std::min(left, kMaxBatch);
    err = launch_requests<Kernels>(a, path, max_q_len, num_sms, s);
    a.cu += a.B;
    a.kv_len += a.B;
    a.c.page_table += static_cast<int64_t>(a.B) * a.c.max_pages;
  }
  return err;
}

// Workspace: partial sums and the row tiles to join, then what the tcgen05
// kernel needs where a call can take it (cut blocks or not, alone or not, so
// that a smaller call never needs more).  A larger batch's slices share it.
struct Workspace {
  size_t joins, tc, tc_entries, tc_joins, tc_part, total;
};

template <class Args>
Workspace plan_workspace(const Args& a, int max_q_len) {
  const int D = a.c.head_dim;
  const Path path = path_of<Args::kBlocks>(a, max_q_len);
  Workspace w;
  size_t at = 0;
  auto take = [&](size_t bytes) { const size_t from = at; at += align_up(bytes, 256); return from; };
  take(part_bytes_of<Args::kBlocks>(D));
  w.joins = take(kMaxCtas * sizeof(JoinTile));
  w.tc = take(sizeof(TcList));
  w.tc_entries = take(path.tc ? (tc_places(a) + kTcSlots) * sizeof(TcEntry) : 0);
  w.tc_joins = take(path.tc ? kTcSlots * sizeof(TcJoin) : 0);
  w.tc_part = take(path.tc ? static_cast<size_t>(kTcSlots) * kTcItemRows * (D + 2) * sizeof(float) : 0);
  w.total = at;
  return w;
}

bool attention_config_ok(const moe_paged_attention_config_t* c, int max_batch, int n_kv_heads, int head_dim) {
  if (c->T < 0 || c->T > (1 << 28) || c->batch < 1 || c->batch > max_batch || c->max_q_len < 0) return false;
  if (c->n_q_heads < 1 || c->n_q_heads % n_kv_heads != 0 || c->n_q_heads / n_kv_heads > 256) return false;
  // row and item counts are 32-bit
  const int64_t rows = static_cast<int64_t>(c->T) * (c->n_q_heads / n_kv_heads);
  if (rows > (int64_t(1) << 30) || (rows / kTcItemRows + c->batch) * n_kv_heads > (int64_t(1) << 30)) return false;
  if (c->window < 0 || c->window > (1 << 30) || c->n_sink < 0 || c->n_sink > (1 << 30)) return false;
  if (!(c->sm_scale > 0.f) || !std::isfinite(c->sm_scale)) return false;
  const int64_t width = static_cast<int64_t>(c->n_q_heads) * head_dim;
  return c->q_stride >= width && c->out_stride >= width && c->q_stride % 8 == 0 && c->out_stride % 8 == 0;
}

// Workspace bytes of a call with the geometry that `a` has in c.
template <class Args>
size_t attention_ws_bytes(Args a, const moe_paged_attention_config_t* cfg) {
  a.T = cfg->T;
  a.B = cfg->batch;
  a.group = cfg->n_q_heads / a.c.n_kv_heads;
  return plan_workspace(a, cfg->max_q_len).total;
}

// The call, the configuration and the cache's pointers having been looked at;
// `a` comes with the cache.
template <class Kernels, class Args>
moe_status_t attention_call(Args a, const moe_paged_attention_config_t* cfg, const void* q, const int32_t* cu,
                            const int32_t* kv_len, void* out, float* lse, void* ws, size_t ws_bytes, moe_stream_t stream) {
  if (!q || !cu || !kv_len || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned_to(q, 16) || !aligned_to(out, 16) || !aligned_to(cu, 4) || !aligned_to(kv_len, 4) ||
      (lse && !aligned_to(lse, 4)))
    return MOE_ERR_INVALID_ARG;
  if (!ws || ws_bytes < attention_ws_bytes(a, cfg)) return MOE_ERR_WORKSPACE;
  if (!aligned_to(ws, 256)) return MOE_ERR_INVALID_ARG;
  unsigned* status = nullptr;
  int sms = 0;
  const moe_status_t st = current_device(&status, &sms);
  if (st != MOE_OK) return st;
  a.q = static_cast<const uint16_t*>(q);
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.cu = cu;
  a.kv_len = kv_len;
  a.status = status;
  a.qs = cfg->q_stride;
  a.os = cfg->out_stride;
  a.T = cfg->T;
  a.B = cfg->batch;
  a.group = cfg->n_q_heads / a.c.n_kv_heads;
  a.window = cfg->window;
  a.n_sink = cfg->n_sink;
  a.sm_scale = cfg->sm_scale;
  const Workspace w = plan_workspace(a, cfg->max_q_len);
  char* base = static_cast<char*>(ws);
  a.part = reinterpret_cast<float*>(base);
  a.joins = reinterpret_cast<JoinTile*>(base + w.joins);
  a.tc = reinterpret_cast<TcList*>(base + w.tc);
  a.tc_entries = reinterpret_cast<TcEntry*>(base + w.tc_entries);
  a.tc_joins = reinterpret_cast<TcJoin*>(base + w.tc_joins);
  a.tc_part = reinterpret_cast<float*>(base + w.tc_part);
  return launch_paged_attn<Kernels>(a, cfg->max_q_len, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace
}  // namespace moe
