// Attention over the paged 8-bit cache (include/paged_kv.h): entry points and
// the few-row kernels.
#include "paged_attn_rows.cuh"

namespace moe {
namespace {

bool config_ok(const moe_paged_attention_config_t* cfg, const moe_kv_cache_t* cache) {
  return cfg && kv_cache_shape_ok(cache) && attention_config_ok(cfg, cache->n_kv_heads, cache->head_dim);
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_paged_attention_ws_bytes(const moe_paged_attention_config_t* cfg, const moe_kv_cache_t* cache) {
  using namespace moe;
  if (!config_ok(cfg, cache)) return 0;
  PaArgs a;
  a.c = *cache;
  return attention_ws_bytes(a, cfg);
}

extern "C" moe_status_t moe_paged_attention(const moe_paged_attention_config_t* cfg, const moe_kv_cache_t* cache,
                                            const void* q, const int32_t* cu, const int32_t* kv_len, void* out,
                                            float* lse, void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  if (!config_ok(cfg, cache)) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!kv_cache_pointers_ok(cache)) return MOE_ERR_INVALID_ARG;
  PaArgs a;
  a.c = *cache;
  return attention_call(a, cfg, q, cu, kv_len, out, lse, ws, ws_bytes, stream);
}
