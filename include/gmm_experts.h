/*
 * gmm_experts.h - what follows the soft assignment: the lists of the
 * components, the rows of the points there and back, and one linear model per
 * component.
 *
 * gmm_assign names the m most responsible components of every point and their
 * responsibilities ([Flash-GMM] Deployment: the coarse quantiser of an IVF
 * index lists each vector in several lists).  Here
 *
 *   gmm_route      turns that assignment into the lists;
 *   gmm_dispatch   lays the points' rows out list by list;
 *   gmm_linear     applies component k's linear model to every row of list k;
 *   gmm_combine    brings the rows back to their points, weighted and summed;
 *   gmm_linear4    does all of it at once for a few points, on 4-bit weights;
 *
 * and the first four have their gradients, so that the components' models (a
 * mixture of linear experts gated by the mixture) can be trained.
 *
 * Terms.  Entry e = point * m + column, 0 <= e < n * m, of the assignment.  List k holds
 * the entries whose idx is k, in increasing e; the slots offsets[k] ..
 * offsets[k + 1] are list k's, entry[s] is the entry in slot s and slot[e] the
 * slot of entry e.  An entry whose idx is not in [0, k) (gmm_assign writes -1
 * for a column without a component) is in no list: its slot is -1.  The
 * T = offsets[k] listed entries fill the slots 0 .. T - 1; entry[s] is -1 for
 * s >= T.  A point may list one component twice; both entries count.
 *
 * Conventions as in gmm.h: device pointers unless "host" is said, caller-owned
 * buffers and stream, asynchronous, no allocation, argument errors before any
 * launch; two calls that share a workspace must not overlap.  "Rows by slot" are
 * arrays [n * m] rows long; their rows from T on belong to no list: they are
 * neither read nor written.  Row strides (ld) are in elements.  Rows are stored in
 * `dtype` (gmm_dtype); products, sums and softmax weights are fp32, each result is
 * rounded once.  Inputs and outputs must not overlap.  Results are bitwise
 * reproducible.  Fastest when base pointers, row strides and widths are multiples of
 * 16 bytes; any other layout goes through slower loads of the same pieces.
 *
 * Limits: 1 <= m <= GMM_MAX_TOPM, 1 <= k <= GMM_MAX_LISTS, 0 <= n with
 * n * m <= 2^30, 1 <= widths <= 2^20, strides <= 2^22, and products of no more than 2^24
 * 128 x 128 tiles; outside them GMM_E_ARG.
 */
#ifndef GMM_EXPERTS_H
#define GMM_EXPERTS_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#include "gmm.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Largest number of lists. */
#define GMM_MAX_LISTS 4096

/* The lists of an assignment (the struct is a host object, its arrays are
 * device int32). */
typedef struct {
    int64_t n;              /* points */
    int32_t m;              /* columns of the assignment */
    int32_t k;              /* lists */
    const int32_t* offsets; /* [k + 1] */
    const int32_t* entry;   /* [n * m] */
    const int32_t* slot;    /* [n * m] */
} gmm_routes;

/* Bytes of device workspace gmm_route needs (0 where the whole assignment is
 * sorted by one workgroup). */
gmm_status gmm_route_workspace_bytes(int64_t n, int32_t m, int32_t k, size_t* bytes /* host */);

/* The lists of idx [n * m] (device int32, as gmm_assign writes it): offsets
 * [k + 1], entry [n * m], slot [n * m], written whole.  ws may be NULL when
 * gmm_route_workspace_bytes says 0, else it is 256-byte aligned. */
gmm_status gmm_route(int64_t n, int32_t m, int32_t k, const int32_t* idx, void* ws, size_t ws_bytes,
                     int32_t* offsets, int32_t* entry, int32_t* slot, hipStream_t stream);

/* y[slot[p * m + i]] = x[p] for every listed column i of every point p: the
 * points' rows [n, d] (stride ldx) as rows by slot (stride ldy). */
gmm_status gmm_dispatch(const gmm_routes* routes, int64_t d, int32_t dtype, const void* x, int64_t ldx,
                        void* y, int64_t ldy, hipStream_t stream);

/* Gradient of gmm_dispatch: dx[p] = sum over the listed columns i, in order,
 * of dy[slot[p * m + i]]; zero for a point in no list. */
gmm_status gmm_dispatch_backward(const gmm_routes* routes, int64_t d, int32_t dtype, const void* dy,
                                 int64_t lddy, void* dx, int64_t lddx, hipStream_t stream);

/* out[p] = sum over the listed columns i, in order, of gamma[p * m + i] *
 * z[slot[p * m + i]]; zero for a point in no list.  gamma: fp32 [n * m]; the
 * weight of an unlisted column is not used. */
gmm_status gmm_combine(const gmm_routes* routes, int64_t d, int32_t dtype, const void* z, int64_t ldz,
                       const float* gamma, void* out, int64_t ldo, hipStream_t stream);

/* Gradients of gmm_combine: dz[slot[e]] = gamma[e] * dout[e / m] (rows by
 * slot, stride lddz) and dgamma[e] = <dout[e / m], z[slot[e]]> (fp32 [n * m],
 * 0 for an unlisted column).  Either may be NULL; z is not read without
 * dgamma and may then be NULL. */
gmm_status gmm_combine_backward(const gmm_routes* routes, int64_t d, int32_t dtype, const void* dout,
                                int64_t lddo, const void* z, int64_t ldz, const float* gamma, void* dz,
                                int64_t lddz, float* dgamma, hipStream_t stream);

/* One linear model per component, y = W_k x + b_k. */
typedef struct {
    int64_t d_in;
    int64_t d_out;
    int64_t ldx;         /* row stride of x */
    int64_t ldy;         /* row stride of y, dy */
    int64_t lddx;        /* row stride of dx (gmm_linear_backward) */
    int32_t dtype;       /* gmm_dtype of x, w, y, dy, dx */
    int32_t sorted_rows; /* 0: x holds the points' rows [n], row s of list k is x[entry[s] / m];
                            1: x holds rows by slot */
} gmm_linear_desc;

/* y[s] = W_k x_s + b_k for every slot s of every list k.  w [k, d_out, d_in],
 * bias fp32 [k, d_out] or NULL, y rows by slot. */
gmm_status gmm_linear(const gmm_routes* routes, const gmm_linear_desc* desc, const void* x, const void* w,
                      const float* bias, void* y, hipStream_t stream);

/* Bytes of device workspace gmm_linear_backward needs. */
gmm_status gmm_linear_backward_workspace_bytes(int64_t n, int32_t m, int32_t k, const gmm_linear_desc* desc,
                                               size_t* bytes /* host */);

/* Gradients of gmm_linear for the rows dy by slot: dx[s] = W_k^T dy[s] (rows by slot,
 * stride lddx; gmm_dispatch_backward sums them at the points), dw[k] = sum over
 * list k of dy[s] x_s^T (fp32 [k, d_out, d_in]) and db[k] = sum dy[s] (fp32 [k,
 * d_out]); zero for an empty list.  Each of dx, dw, db may be NULL, and db needs
 * dw; w is read for dx alone, x for dw alone, and may be NULL without them.
 * Without dw the workspace is not used. */
gmm_status gmm_linear_backward(const gmm_routes* routes, const gmm_linear_desc* desc, const void* dy,
                               const void* x, const void* w, void* dx, float* dw, float* db, void* ws,
                               size_t ws_bytes, hipStream_t stream);

/* 4-bit weights.  Row r of w [rows, d_in] is cut into groups of `group` columns
 * (32, 64 or 128; the last may be shorter).  A group's scale is its largest
 * magnitude / 7, rounded to bf16; a weight's code is
 * round-to-nearest-even(w / scale), clamped to [-8, 7], plus 8 (0 / 0 in an all-zero group counts as 0).
 * codes [rows, (d_in + 1) / 2] bytes: column j in the low half (j even) or the high half (j
 * odd) of byte j / 2, the unused half of an odd row's last byte 8; scales bf16 [rows,
 * ceil(d_in / group)].  A group with a non-finite weight gets a non-finite scale, and every
 * product with it is NaN or infinite. */
gmm_status gmm_quantize4(int64_t rows, int64_t d_in, int32_t group, int32_t dtype, const void* w,
                         uint8_t* codes, void* scales, hipStream_t stream);

/* The single-point form, straight from the assignment: out[p] = sum over the
 * columns i with 0 <= idx[p * m + i] < k, in order, of gamma[p * m + i] * (W_k x[p] + b_k),
 * k = idx[p * m + i], W_k = (code - 8) * scale; zero for a point in no list.  For a few points:
 * every 16 of them read the weights of the components they list once.  codes [k * d_out rows] and scales as
 * gmm_quantize4 writes them, bias fp32 [k, d_out] or NULL; x [n, d_in] (stride ldx) and out
 * [n, d_out] (stride ldo) in dtype.  n <= GMM_LINEAR4_MAX_N.  An infinity in x[p] makes the
 * outputs of point p NaN or infinite. */
#define GMM_LINEAR4_MAX_N 1024
gmm_status gmm_linear4(int64_t n, int32_t m, int32_t k, int64_t d_in, int64_t d_out, int32_t group,
                       int32_t dtype, const void* x, int64_t ldx, const int32_t* idx, const float* gamma,
                       const uint8_t* codes, const void* scales, const float* bias, void* out, int64_t ldo,
                       hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* GMM_EXPERTS_H */
