// Attention over the paged 4-bit cache (include/block_kv.h): entry points and
// the few-row kernels.
#include "block_kv.cuh"
#include "paged_attn_rows.cuh"

namespace moe {
namespace {

bool config_ok(const moe_paged_attention_config_t* cfg, const moe_blockkv_cache_t* cache) {
  return cfg && blockkv_shape_ok(cache) && attention_config_ok(cfg, cache->n_kv_heads, cache->head_dim);
}

BlockPaArgs args_of(const moe_blockkv_cache_t* cache) {
  BlockPaArgs a;
  a.c.k = cache->k;
  a.c.v = cache->v;
  a.c.k_scale = a.c.v_scale = nullptr;
  a.c.page_table = cache->page_table;
  a.c.n_pages = cache->n_pages;
  a.c.page_size = cache->page_size;
  a.c.n_kv_heads = cache->n_kv_heads;
  a.c.head_dim = cache->head_dim;
  a.c.max_pages = cache->max_pages;
  a.c.page_stride = cache->page_stride;
  a.c.head_stride = cache->head_stride;
  a.c.token_stride = cache->token_stride;
  a.k_scales = static_cast<const uint8_t*>(cache->k_scale);
  a.v_scales = static_cast<const uint8_t*>(cache->v_scale);
  a.scale_page = cache->scale_page_stride;
  a.scale_head = cache->scale_head_stride;
  a.scale_token = cache->scale_token_stride;
  a.kg = cache->k_gscale;
  a.vg = cache->v_gscale;
  return a;
}

}  // namespace
}  // namespace moe

extern "C" size_t moe_blockkv_attention_ws_bytes(const moe_paged_attention_config_t* cfg,
                                                 const moe_blockkv_cache_t* cache) {
  using namespace moe;
  return config_ok(cfg, cache) ? attention_ws_bytes(args_of(cache), cfg) : 0;
}

extern "C" moe_status_t moe_blockkv_attention(const moe_paged_attention_config_t* cfg, const moe_blockkv_cache_t* cache,
                                              const void* q, const int32_t* cu, const int32_t* kv_len, void* out,
                                              float* lse, void* ws, size_t ws_bytes, moe_stream_t stream) {
  using namespace moe;
  if (!config_ok(cfg, cache)) return MOE_ERR_INVALID_ARG;
  if (cfg->T == 0) return MOE_OK;
  if (!blockkv_pointers_ok(cache)) return MOE_ERR_INVALID_ARG;
  return attention_call(args_of(cache), cfg, q, cu, kv_len, out, lse, ws, ws_bytes, stream);
}
