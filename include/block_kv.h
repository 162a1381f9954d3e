/*
 * block_kv.h -- C ABI of a paged key/value cache in 4 bits, the attention that
 * reads it and the way back (libmoe_gb300.so; status codes, element types and
 * stream type from moe_gb300.h, append and attention configurations from
 * paged_kv.h; the calls of this header take up to 2^20 requests).
 *
 * The cache holds, for every token and key head, D values as E2M1 codes with
 * one E4M3 scale for every 16 consecutive elements and a factor g for the
 * whole cache, one for keys and one for values:
 *   value = e2m1(code) * e4m3(scale) * g
 * which is 4.5 bits an element.  The scales belong to a token, so nothing that
 * is in the cache changes when a later token is appended.  Requests own pages
 * through a page table, and a ragged batch is given by cu and kv_len, both as
 * in paged_kv.h: token j of request b sits in slot j % page_size of page
 * page_table[b][j / page_size]; new token i of request b is row cu[b] + i and
 * has position kv_len[b] - n_b + i, n_b = cu[b+1] - cu[b].  All of that is read
 * on the device; no call synchronises.
 */
#ifndef BLOCK_KV_H
#define BLOCK_KV_H

#include "paged_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  void* k;                    /* E2M1 codes of the keys, page 0: two to a byte, element */
                              /*   2i in the low four bits                          */
  void* v;                    /* ... of the values, same strides                    */
  void* k_scale;              /* E4M3 scales (0 to 448) of the keys, a byte for 16   */
                              /*   elements                                         */
  void* v_scale;              /* ... of the values, same strides                    */
  const int32_t* page_table;  /* [batch][max_pages]                                 */
  int32_t n_pages;            /* pages in the cache, >= 1                           */
  int32_t page_size;          /* tokens in a page: 16, 32, 64 or 128                */
  int32_t n_kv_heads;         /* key heads, 1..1024                                 */
  int32_t head_dim;           /* D: 64, 128 or 256                                  */
  int32_t max_pages;          /* width of the page table, >= 1, <= 2^30 / page_size  */
  float k_gscale;             /* g of the keys and of the values: powers of two,     */
  float v_gscale;             /*   2^-60 to 2^60                                    */
  int64_t page_stride;        /* bytes of codes between pages, heads and tokens:     */
  int64_t head_stride;        /*   positive multiples of 16, at least D / 2, in any  */
  int64_t token_stride;       /*   order; a token's D / 2 bytes are contiguous;      */
                              /*   n_pages page_stride below 2^36 (64 GB)            */
  int64_t scale_page_stride;  /* bytes of scales between pages, heads and tokens:    */
  int64_t scale_head_stride;  /*   positive multiples of D / 16, in any order; a     */
  int64_t scale_token_stride; /*   token's D / 16 bytes are contiguous; n_pages      */
                              /*   scale_page_stride below 2^32 D / 16               */
} moe_blockkv_cache_t;

/*
 * Normalises and rotates new queries and keys as moe_kv_append does, and
 * appends the keys and values to the cache.
 *
 * All of it in fp32; q_out is rounded once to bf16.  For every 16 elements of a
 * key or value row the scale is the smallest E4M3 value s from 2^-9 on with
 * |x| <= 6 s g for all of them (448 where there is none: larger elements
 * become +-6 s g), and a code is the E2M1 value nearest to the fp32 quotient
 * x / (s g), ties to the even code.  An element that is infinite becomes
 * +-6 s g and is left out of s; one that is NaN makes the scale E4M3's NaN, so
 * that its 16 elements read as NaN; both record MOE_ERR_DEVICE_NONFINITE.
 *
 * So that equal inputs give equal codes on any machine, a key's fp32 operations
 * are fixed: squares are summed four neighbours at a time, (0 + 1) + (2 + 3),
 * then these sums in a tree of neighbours (with MOE_ROPE_HALF the quads i and
 * rot_dim / 8 + i, which rotate together, come first and side by side); the
 * norm is x * (1 / sqrt(sum / D + eps)) * gamma, each product rounded; and the
 * two products of a rotated element are each rounded before they are added.
 *
 * Arguments, alignment, the rows that are left alone and the faults recorded
 * (and what of a call they leave unwritten) are those of moe_kv_append; a
 * slot's codes and scales are written together.  Codes and pointers are
 * 16-byte aligned, scales D / 16 bytes.  A call writes only the slots of its
 * new tokens, so requests may share pages as long as no slot is written by one
 * call twice.
 */
moe_status_t moe_blockkv_append(const moe_kv_append_config_t* cfg, const moe_blockkv_cache_t* cache, const void* q,
                                const void* k, const void* v, const float* gamma_q, const float* gamma_k,
                                const float* cos_sin, const int32_t* positions, const int32_t* cu,
                                const int32_t* kv_len, void* q_out, moe_stream_t stream);

/* Workspace bytes of moe_blockkv_attention; 0 for an invalid configuration.
 * They never shrink when T, batch or max_q_len grow (0 counts as T). */
size_t moe_blockkv_attention_ws_bytes(const moe_paged_attention_config_t* cfg, const moe_blockkv_cache_t* cache);

/*
 * Causal attention of the new tokens over the cache: moe_paged_attention's
 * formulas, masks, arguments, workspace rules and faults.
 *
 * A key or value becomes e2m1(code) * e4m3(scale) exactly in f16 and q is
 * scaled by a power of two per head to f16 (exact but for elements 2^-28 below
 * the head's largest), so the products' operands are exact; scores, maxima,
 * sums and outputs are accumulated in fp32, parts of a row joined by factors
 * good to 2^-22; the softmax weights w_j are rounded to f16 for the product with
 * V, to 11 bits down to 2^-22 of the row's largest, smaller ones by up to 2^-33
 * of it.  g enters the scores' and the outputs' factor.  Results do not depend
 * on scheduling.  A NaN scale in a position that a request's new tokens can see
 * makes NaN of the rows that see it and may make NaN of other rows of the same
 * request and key head; what none of them sees may hold anything.
 */
moe_status_t moe_blockkv_attention(const moe_paged_attention_config_t* cfg, const moe_blockkv_cache_t* cache,
                                   const void* q, const int32_t* cu, const int32_t* kv_len, void* out, float* lse,
                                   void* ws, size_t ws_bytes, moe_stream_t stream);

typedef struct {
  int32_t T;            /* rows of k_out and v_out, 0..2^28 (0 is a no-op)           */
  int32_t batch;        /* requests, 1..2^20                                        */
  int32_t out_dtype;    /* MOE_BF16 or MOE_F32                                      */
  int64_t k_stride;     /* elements between rows of k_out and of v_out (multiples of */
  int64_t v_stride;     /*   8; heads of a row are contiguous)                      */
} moe_blockkv_read_config_t;

/*
 * Reads the last n_b = cu[b+1] - cu[b] tokens of each request back: row cu[b] + i
 * of k_out and v_out [T][n_kv_heads][D] becomes the keys and values at position
 * kv_len[b] - n_b + i.  Values are exact in fp32 and rounded once to bf16
 * (exact as well: six bits).  Either output may be NULL.  After an append with
 * the same cu and kv_len it returns what was stored.
 *
 * k_out, v_out 16-byte aligned.  A page outside the cache, a position past the
 * page table, offsets that decrease or leave [0, T] and kv_len[b] < n_b record
 * MOE_ERR_DEVICE_BOUNDS; the rows of such a page or position, or all rows of
 * such a request, are left as they were, like rows of no request (after offsets
 * that decrease other requests' rows may be too, and rows that two requests
 * name then hold either's tokens).
 */
moe_status_t moe_blockkv_read(const moe_blockkv_read_config_t* cfg, const moe_blockkv_cache_t* cache,
                              const int32_t* cu, const int32_t* kv_len, void* k_out, void* v_out,
                              moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* BLOCK_KV_H */
