/*
 * add_rms_norm.h -- C ABI of the residual's addition and the RMS norm behind
 * it (libmoe_gb300.so; status codes, element types and stream type from
 * moe_gb300.h).
 *
 * For every row t of d elements:
 *   h = x + r                  rounded to the type of r (r NULL: h = x)
 *   y = h / sqrt(mean(h^2) + eps) * gamma
 * The addition, the mean and y are fp32.  h goes to `sum`; y to `out`, rounded
 * once to its type, and to `out8` as E4M3 codes with one scale for a row or
 * for every `group` elements:
 *   s = max(max |y| / 448, 2^-40) over the group,  code = e4m3(y / s)
 * (nearest, ties to even; y / s as y times the reciprocal of s, which like s is
 * exact to a few units of fp32's last place).  A NaN or
 * infinite element of h makes NaN of its row's norm: y is NaN, or 0 where
 * finite elements meet an infinite mean, as the formula has it.  NaN elements
 * become the NaN code and are left out of their group's maximum; other rows
 * are not affected.
 */
#ifndef ADD_RMS_NORM_H
#define ADD_RMS_NORM_H

#include "moe_gb300.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct {
  int32_t T;            /* rows, 0..2^28 (0 is a no-op)                              */
  int32_t d;            /* elements of a row: a multiple of 8, 8..16384              */
  int32_t x_dtype;      /* MOE_BF16 or MOE_F32, each                                 */
  int32_t res_dtype;    /*   of residual and sum (ignored when residual is NULL)     */
  int32_t out_dtype;    /*   (ignored when out is NULL)                              */
  int32_t group;        /* elements that share a scale of out8: 16, 32, 64, 128 or   */
                        /*   256, dividing d; 0: the row (ignored when out8 is NULL) */
  float eps;            /* > 0, finite                                               */
  int64_t x_stride;     /* elements between rows, multiples of 8; out8 and out8_scale */
  int64_t res_stride;   /*   are contiguous                                          */
  int64_t sum_stride;
  int64_t out_stride;
} moe_add_norm_config_t;

/*
 * x           [T][d]
 * residual    [T][d] or NULL
 * gamma       [d] float
 * out         [T][d] or NULL
 * out8        [T][d] E4M3 codes or NULL; at least one of out and out8
 * out8_scale  [T][d / group] float ([T] for group 0), with out8
 * sum         [T][d] of the residual's type or NULL (it needs a residual); it
 *             may be the residual itself, or x where their types and strides
 *             agree; out may be x or residual on the same terms.  Outputs may
 *             not overlap otherwise.
 * All but out8_scale 16-byte aligned (out8: 8).
 */
moe_status_t moe_add_rms_norm(const moe_add_norm_config_t* cfg, const void* x, const void* residual,
                              const float* gamma, void* out, void* out8, float* out8_scale, void* sum,
                              moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* ADD_RMS_NORM_H */
