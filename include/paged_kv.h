/*
 * paged_kv.h -- C ABI of a paged key/value cache in 8 bits and the attention
 * that reads it (libmoe_gb300.so; status codes, element types and stream type
 * from moe_gb300.h).
 *
 * The cache holds, for every token and key head, D values as E4M3 codes
 * (value = e4m3(code) * scale), with one fp32 scale for each page and head,
 * for keys and for values.  Requests own pages through a page table: token j
 * of request b sits in slot j % page_size of page
 * page_table[b][j / page_size].
 *
 * Both calls take a ragged batch: cu[b] .. cu[b+1]-1 are the rows of request
 * b's new tokens, and kv_len[b] the tokens that its cache holds with them, so
 * that new token i of request b has position kv_len[b] - n_b + i,
 * n_b = cu[b+1] - cu[b].  The same two arrays serve moe_kv_append and the
 * moe_paged_attention after it.  They are read on the device; no call
 * synchronises.
 */
#ifndef PAGED_KV_H
#define PAGED_KV_H

#include "moe_gb300.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  void* k;                   /* E4M3 codes of the keys, page 0                    */
  void* v;                   /* E4M3 codes of the values, same strides            */
  float* k_scale;            /* [n_pages][n_kv_heads], 2^-100 to 2^100            */
  float* v_scale;            /* [n_pages][n_kv_heads], 2^-80 to 2^80, those of    */
                             /*   one request and head within 2^80 of each other  */
  const int32_t* page_table; /* [batch][max_pages]                                */
  int32_t n_pages;           /* pages in the cache, >= 1                          */
  int32_t page_size;         /* tokens in a page: 16, 32, 64 or 128               */
  int32_t n_kv_heads;        /* key heads, 1..1024                                */
  int32_t head_dim;          /* D: 64, 128 or 256                                 */
  int32_t max_pages;         /* width of the page table, >= 1, <= 2^30 / page_size */
  int64_t page_stride;       /* bytes between pages, heads and tokens: positive   */
  int64_t head_stride;       /*   multiples of 16; a token's D codes are          */
  int64_t token_stride;      /*   contiguous.  Any order of the three: pages of   */
                             /*   [head][token][D] and of [token][head][D] alike  */
} moe_kv_cache_t;

enum { MOE_ROPE_HALF = 0, MOE_ROPE_INTERLEAVED = 1 };

typedef struct {
  int32_t T;              /* rows of q, k and v (new tokens), >= 0 (0 is a no-op) */
  int32_t batch;          /* requests, 1..4096                                    */
  int32_t n_q_heads;      /* query heads, 1..4096 (ignored when q is NULL)        */
  int32_t rot_dim;        /* elements of a head that rotate: 0 or a multiple of 8, */
                          /*   at most D (0: no rotation, no table)               */
  int32_t rope_layout;    /* MOE_ROPE_HALF or MOE_ROPE_INTERLEAVED                */
  int32_t n_pos;          /* rows of the cos_sin table, >= 1 with a rotation      */
  float eps;              /* epsilon of the norm: > 0, finite                     */
  int64_t q_stride;       /* elements between the rows of q, k, v and q_out       */
  int64_t k_stride;       /*   (multiples of 8; heads of a row are contiguous,    */
  int64_t v_stride;       /*   so slices of one joint projection can be passed)   */
  int64_t q_out_stride;
} moe_kv_append_config_t;

/*
 * Normalises and rotates new queries and keys, and appends the keys and
 * values to the cache.
 *
 *   y = x                                           (gamma NULL)
 *   y = x / sqrt(mean(x^2) + eps) * gamma           (RMS norm over the head)
 *   with (c, s) = cos_sin[pos][i], i < rot_dim/2, r = rot_dim/2:
 *     HALF:        (y_i, y_{i+r})   -> (y_i c - y_{i+r} s,  y_{i+r} c + y_i s)
 *     INTERLEAVED: (y_2i, y_{2i+1}) -> (y_2i c - y_{2i+1} s, y_{2i+1} c + y_2i s)
 *   elements from rot_dim on stay as they are; values are stored unchanged.
 *
 * All of it in fp32; q_out is rounded once to bf16, keys and values once to
 * E4M3 (nearest, ties to even).  A page and head's scale, for keys and for
 * values, is the smallest power of two s >= 2^-40 for which no element the
 * call writes there is over 448 s in size; where the page already holds
 * earlier tokens of its request (new tokens not starting at its slot 0), the
 * larger of that and the old scale, and if that is larger than the old one
 * the earlier tokens' codes are rounded to it (exact but for codes that fall
 * below E4M3's normal range).  A power of two costs E4M3 no precision, keeps
 * this re-rounding exact and the appended values independent of how a prompt
 * was cut into calls, down to that range.  A page that a call fills from slot
 * 0 takes nothing from what it held, so pages need no clearing.
 * A NaN element is stored as the NaN code; an infinite one as +-448 s; both
 * are left out of the page's scale and record MOE_ERR_DEVICE_NONFINITE.
 *
 * q          [T][n_q_heads][D] bf16 or NULL; q_out likewise (q_out may be q)
 * k, v       [T][n_kv_heads][D] bf16
 * gamma_q/_k [D] float, or NULL for no norm (gamma_q without q is ignored)
 * cos_sin    [n_pos][rot_dim/2][2] float (NULL allowed with rot_dim = 0)
 * positions  [T] int32 rows of cos_sin, or NULL: the token's position
 * cu, kv_len [batch+1], [batch] int32, see above
 * k, v, q, q_out, gamma, cos_sin and the cache's k and v are 16-byte aligned.
 * A table row outside [0, n_pos), a page outside the cache, a position past
 * the page table, offsets that decrease or leave [0, T], and kv_len[b] < n_b
 * record MOE_ERR_DEVICE_BOUNDS; the tokens concerned are not written: by a bad
 * page or position past the page table their keys and values (q_out is), by a
 * bad table row that token's q_out as well, by wrong offsets or a wrong length
 * nothing of the request (after offsets that decrease, other requests' tokens
 * may stay unwritten too).
 * Rows of no request (before cu[0], from cu[batch] on) are left alone.
 * Requests of one call must not share a page that either writes.
 */
moe_status_t moe_kv_append(const moe_kv_append_config_t* cfg, const moe_kv_cache_t* cache, const void* q,
                           const void* k, const void* v, const float* gamma_q, const float* gamma_k,
                           const float* cos_sin, const int32_t* positions, const int32_t* cu, const int32_t* kv_len,
                           void* q_out, moe_stream_t stream);

typedef struct {
  int32_t T;              /* query rows, >= 0 (0 is a no-op)                      */
  int32_t batch;          /* requests, 1..4096                                    */
  int32_t n_q_heads;      /* a multiple of n_kv_heads, at most 256 times it; head */
                          /*   h reads key head h / (n_q_heads / n_kv_heads)      */
  int32_t max_q_len;      /* the most new tokens of a request, as far as the host */
                          /*   knows; 0 = unknown.  Chooses kernels, not results: */
                          /*   requests over it are computed too, only slower     */
  int32_t window;         /* 0: none; W: a token sees the last W positions, its   */
                          /*   own among them (at most 2^30, like n_sink)         */
  int32_t n_sink;         /* with a window: the first n_sink positions stay       */
                          /*   visible, >= 0                                      */
  float sm_scale;         /* factor of the scores, finite and > 0                 */
  int64_t q_stride;       /* elements between rows of q and of out, multiples of 8 */
  int64_t out_stride;
} moe_paged_attention_config_t;

/* Workspace bytes of moe_paged_attention; 0 for an invalid configuration.  They
 * never shrink when T, batch or max_q_len grow (0 counts as T), so a workspace
 * for the largest call serves the smaller ones too. */
size_t moe_paged_attention_ws_bytes(const moe_paged_attention_config_t* cfg, const moe_kv_cache_t* cache);

/*
 * Causal attention of the new tokens over the cache (which holds their own
 * keys and values already).  The token at position p sees the positions
 * j <= p, with a window only those with j > p - window or j < n_sink:
 *   z_j = sm_scale * q . K_j,  out = sum_j softmax(z)_j V_j,
 *   lse = log(sum_j exp(z_j))
 * over the visible j.  A token that sees nothing (its position is negative)
 * gets out = 0 and lse = -infinity.  What lies behind a request's length, or
 * is visible to none of its new tokens, is not used and may hold anything,
 * NaN included.
 *
 * q, out      [T][n_q_heads][D] bf16, 16-byte aligned; out must not overlap q
 * cu, kv_len  [batch+1], [batch] int32
 * lse         [T][n_q_heads] float out, or NULL
 * ws          workspace, 256-byte aligned, no state between calls
 * The products take the codes exactly (E4M3 fits f16) and q scaled by a power
 * of two per head to f16, which is exact but for elements 2^-28 below the
 * head's largest; scores, maxima, sums and outputs are accumulated in fp32;
 * the weights w_j, the softmax times the page's value scale, are rounded to f16
 * for the product with V: to 11 bits down to 2^-22 of the row's largest, smaller
 * ones by up to 2^-33 of it, which can move an output by up to
 * 448 (tokens) 2^-33 max_j w_j.  Results do not depend on scheduling: the same
 * call gives the same bits.  A NaN or infinite q makes its own head's row NaN.
 * A NaN code in a position that a request's new tokens can see makes NaN of the
 * rows that see it and may make NaN of other rows of the same request and key
 * head.
 * A page outside the cache or a position past the page table records
 * MOE_ERR_DEVICE_BOUNDS and is treated as not visible; a request whose
 * offsets decrease or leave [0, T] records it too and its rows stay
 * unwritten.  kv_len[b] < n_b is allowed (the first tokens see nothing);
 * kv_len[b] < 0 counts as 0.
 */
moe_status_t moe_paged_attention(const moe_paged_attention_config_t* cfg, const moe_kv_cache_t* cache, const void* q,
                                 const int32_t* cu, const int32_t* kv_len, void* out, float* lse, void* ws,
                                 size_t ws_bytes, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* PAGED_KV_H */
