// Attention over the paged 8-bit cache: the tcgen05 kernel.
#include "paged_attn_tc.cuh"

namespace moe {

bool paged_attn_tc_supported(int D) { return D == 64 || D == 128; }

cudaError_t launch_paged_attn_tc(const PaArgs& a, cudaStream_t s) {
  return a.c.head_dim == 64 ? launch_tc<64>(a, s) : launch_tc<128>(a, s);
}

}  // namespace moe
