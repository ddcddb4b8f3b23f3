/*
 * experts.h -- the operators of a mixture-of-experts layer for AMD Instinct
 * MI355X (gfx950). C ABI, part of libpca_hist.so.
 *
 * A router gives each of `tokens` tokens top_k expert ids. A (token, choice)
 * pair i = t * top_k + j is one row of work. The operators:
 *
 *   experts_group           a histogram of the ids by expert, its exclusive
 *                           sum, and the stable sort of the pairs by expert
 *   experts_matmul          y[p] = x[token(p)] w[e(p)]^T for the sorted pairs p
 *   experts_matmul_dx       dx[p] = dy[p] w[e(p)]
 *   experts_matmul_dw       dw[e] = sum over e's pairs p of dy[p]^T x[token(p)]
 *   experts_combine         out[t] = sum_j weights[t,j] y[place[t,j]]
 *   experts_combine_backward  its gradients for y and for the weights
 *   experts_quantize_rows   8-bit rows with one scale each
 *   experts_int8_matmul     the product of 8-bit rows and 8-bit weights, by
 *                           expert or dense
 *   experts_quantize_mx4    4-bit rows, a power of two for 32 values
 *   experts_mx4_matmul      the product of 4-bit rows and 4-bit weights, by
 *                           expert or dense
 *   experts_rms_norm        the norm before the layer, with the residual's
 *                           addition, in 16 bits or (experts_rms_norm_int8) in
 *                           8 as experts_int8_matmul takes them
 *   experts_rms_norm_backward  its gradients
 *   experts_few_tokens      the whole layer for up to EXPERTS_MAX_FEW tokens
 *
 * Pairs are numbered twice: i in the order of the tokens, p in the order of
 * the experts. order[p] = i and place[i] = p. A pair whose id lies outside
 * [0, experts) is dropped: place[i] = -1, and with `kept` pairs left, order[p]
 * = -1 for p >= kept = offsets[experts]. Rows p >= kept of a sorted result are
 * zero.
 *
 * Types: 16-bit elements are EXPERTS_BF16 or EXPERTS_FP16; sums are held in 32
 * bits and rounded once, to nearest even, when the result is stored. (The 8-bit
 * product's are whole numbers; as 32-bit floats they are multiplied by the two
 * scales, three roundings of 2^-24 each, before that.) Leading dimensions (ld*) are in elements, rows have
 * unit stride; any alignment of the element type works (rows of 16-byte
 * aligned addresses and leading dimensions load fastest).
 *
 * Memory, streams and errors follow hist.h: every buffer is the caller's, the
 * calls only queue kernels on `stream` (no allocation, memset or
 * synchronisation, so they can be captured into a HIP graph), inputs and
 * outputs must not overlap, statuses are hist_status_t and come before any
 * work is queued. Products whose launch would take 2^32 threads or more (some
 * 2^37 results) give HIST_ERR_UNSUPPORTED. Device-side indexes (offsets, order, place) are clamped or
 * skipped when out of range; they never lead outside the buffers.
 */
#ifndef PCA_EXPERTS_H
#define PCA_EXPERTS_H

#include "hist.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    EXPERTS_BF16 = 0,
    EXPERTS_FP16 = 1
} experts_dtype_t;

#define EXPERTS_MAX_EXPERTS 1024u
#define EXPERTS_MAX_TOP_K 64u
/* Pairs, and widths n and k of the products. */
#define EXPERTS_MAX_ROWS ((uint64_t)1 << 30)
#define EXPERTS_MAX_WIDTH ((uint32_t)1 << 17)

/* Bytes of workspace experts_group needs (0 for small inputs). */
hist_status_t experts_group_workspace_size(uint64_t tokens, uint32_t top_k, uint32_t experts,
                                           uint64_t *bytes);

/* ids: int32 (id_bits 32) or int64 (id_bits 64) [tokens][top_k].
 * counts[experts], offsets[experts + 1], order[tokens * top_k],
 * place[tokens * top_k]. workspace: 16-byte aligned. */
hist_status_t experts_group(const void *ids, int32_t id_bits, uint64_t tokens, uint32_t top_k,
                            uint32_t experts, int32_t *counts, int32_t *offsets, int32_t *order,
                            int32_t *place, void *workspace, uint64_t workspace_bytes,
                            hipStream_t stream);

/* y [rows][n] from w [experts][n][k] (w_stride elements from one expert to
 * the next). order == NULL: x is [rows][k], already sorted (x_rows == rows).
 * Otherwise x is [x_rows][k] and row p reads x[order[p] / top_k]. */
hist_status_t experts_matmul(void *y, int64_t ldy, const void *x, int64_t ldx, uint64_t x_rows,
                             const void *w, int64_t ldw, int64_t w_stride, const int32_t *offsets,
                             const int32_t *order, uint64_t rows, uint32_t top_k,
                             uint32_t experts, uint32_t n, uint32_t k, int32_t dtype,
                             hipStream_t stream);

/* dx [rows][k] from dy [rows][n] and w [experts][n][k]. */
hist_status_t experts_matmul_dx(void *dx, int64_t lddx, const void *dy, int64_t lddy,
                                const void *w, int64_t ldw, int64_t w_stride,
                                const int32_t *offsets, uint64_t rows, uint32_t experts,
                                uint32_t n, uint32_t k, int32_t dtype, hipStream_t stream);

/* dw [experts][n][k], contiguous, from dy [rows][n] and x as experts_matmul
 * takes it. An expert without rows gets zeros. */
hist_status_t experts_matmul_dw(void *dw, const void *dy, int64_t lddy, const void *x, int64_t ldx,
                                uint64_t x_rows, const int32_t *offsets, const int32_t *order,
                                uint64_t rows, uint32_t top_k, uint32_t experts, uint32_t n,
                                uint32_t k, int32_t dtype, hipStream_t stream);

/* out [tokens][n] from y [rows][n], place [tokens][top_k] and weights
 * [tokens][top_k] (32-bit floats; NULL: all one). The sum runs over j in
 * ascending order. */
hist_status_t experts_combine(void *out, int64_t ldo, const void *y, int64_t ldy, uint64_t rows,
                              const int32_t *place, const float *weights, uint64_t tokens,
                              uint32_t top_k, uint32_t n, int32_t dtype, hipStream_t stream);

/* dy [tokens * top_k][n] and dweights [tokens][top_k] from dout [tokens][n]:
 * dy[place[t,j]] = weights[t,j] dout[t], dweights[t,j] = <dout[t], y[place[t,j]]>,
 * zero where the pair was dropped. */
hist_status_t experts_combine_backward(void *dy, int64_t lddy, float *dweights, const void *dout,
                                       int64_t lddout, const void *y, int64_t ldy,
                                       const int32_t *order, const int32_t *place,
                                       const float *weights, uint64_t tokens, uint32_t top_k,
                                       uint32_t n, int32_t dtype, hipStream_t stream);

/* sx[r] = max |x[r]| / 127 rounded to 32 bits; xq[r] = x[r] / sx[r] rounded
 * to the nearest whole number, ties to even, and clamped to [-127, 127]; a row of
 * zeros has scale 0 and values 0. A row with an infinity or a NaN gets that
 * as its scale (and values 0), so that its products are NaN. */
hist_status_t experts_quantize_rows(int8_t *xq, int64_t ldq, float *sx, const void *x, int64_t ldx,
                                    uint64_t rows, uint32_t k, int32_t dtype, hipStream_t stream);

/* y [rows][n] = (xq wq^T) sx sw. wq [experts][n][k] (contiguous rows with
 * leading dimension ldw, w_stride from one expert to the next), sw
 * [experts][n]. offsets == NULL: dense, one weight [n][k] for all rows
 * (experts must be 1, order NULL). xq and sx are gathered like x in
 * experts_matmul. The whole-number sums are exact for k <= EXPERTS_MAX_WIDTH. */
hist_status_t experts_int8_matmul(void *y, int64_t ldy, const int8_t *xq, int64_t ldq,
                                  uint64_t x_rows, const float *sx, const int8_t *wq, int64_t ldw,
                                  int64_t w_stride, const float *sw, const int32_t *offsets,
                                  const int32_t *order, uint64_t rows, uint32_t top_k,
                                  uint32_t experts, uint32_t n, uint32_t k, int32_t dtype,
                                  hipStream_t stream);

/* 4-bit rows: blocks of 32 values with a power of two each, ceil(k / 32) blocks
 * a row. A block's power is 2^(floor(log2 max |x|) - 2), at least 2^-127,
 * stored as the exponent plus 127 in a byte of xs [rows][blocks]. A value is x
 * divided by it, to the nearest of 0, 0.5, 1, 1.5, 2, 3, 4 and 6 with its sign
 * (ties to the even code, beyond 6 it is 6): a 4-bit code of one sign, two
 * exponent and one fraction bit. xq [rows][16 blocks] holds two codes a byte,
 * the first one in the lower half; past k they are 0. A block with an infinity
 * or a NaN has power 255 and codes 0, and its products are NaN. */
hist_status_t experts_quantize_mx4(uint8_t *xq, int64_t ldq, uint8_t *xs, int64_t ldxs,
                                   const void *x, int64_t ldx, uint64_t rows, uint32_t k,
                                   int32_t dtype, hipStream_t stream);

/* y [rows][n] = xq wq^T, each value times its block's power. wq [experts][n][16
 * blocks] and ws [experts][n][blocks] (w_stride and ws_stride bytes from one
 * expert to the next); all leading dimensions but ldy in bytes. offsets, order
 * and the rows of xq and xs as in experts_int8_matmul. The products are exact,
 * sums are held in 32 bits. Powers whose rows start at multiples of 4 bytes load
 * fastest. */
hist_status_t experts_mx4_matmul(void *y, int64_t ldy, const uint8_t *xq, int64_t ldq,
                                 const uint8_t *xs, int64_t ldxs, uint64_t x_rows,
                                 const uint8_t *wq, int64_t ldw, int64_t w_stride,
                                 const uint8_t *ws, int64_t ldws, int64_t ws_stride,
                                 const int32_t *offsets, const int32_t *order, uint64_t rows,
                                 uint32_t top_k, uint32_t experts, uint32_t n, uint32_t blocks,
                                 int32_t dtype, hipStream_t stream);

/* h = x + residual, rounded to the type (residual NULL: h is x, and the argument
 * h is not used), and y = h (mean h^2 + eps)^-1/2 weight, row by row, in 32 bits
 * and rounded once. x, residual, h, y [rows][n], weight [n]. eps: 1e-30 or
 * more. */
hist_status_t experts_rms_norm(void *y, int64_t ldy, void *h, int64_t ldh, const void *x,
                               int64_t ldx, const void *residual, int64_t ldr,
                               const void *weight, uint64_t rows, uint32_t n, float eps,
                               int32_t dtype, hipStream_t stream);

/* The same with y as 32-bit values rounded to 8 bits: sx[r] = max |y[r]| / 127,
 * xq[r] = y[r] / sx[r] to the nearest whole number. Rows of zeros, infinities
 * and NaN as in experts_quantize_rows. */
hist_status_t experts_rms_norm_int8(int8_t *xq, int64_t ldq, float *sx, void *h, int64_t ldh,
                                    const void *x, int64_t ldx, const void *residual,
                                    int64_t ldr, const void *weight, uint64_t rows, uint32_t n,
                                    float eps, int32_t dtype, hipStream_t stream);

/* Bytes of workspace experts_rms_norm_backward needs. */
hist_status_t experts_rms_norm_backward_workspace_size(uint64_t rows, uint32_t n,
                                                       uint64_t *bytes);

/* dx [rows][n], the gradient of x and of the residual alike, and dweight [n],
 * from dy, the gradient of y, and dh, that of h beyond its part in y (NULL:
 * none). Sums in 32 bits and in a fixed order, rounded once. workspace: 16-byte
 * aligned, not read before it is written. */
hist_status_t experts_rms_norm_backward(void *dx, int64_t lddx, void *dweight, const void *dy,
                                        int64_t lddy, const void *h, int64_t ldh, const void *dh,
                                        int64_t lddh, const void *weight, uint64_t rows,
                                        uint32_t n, float eps, int32_t dtype, void *workspace,
                                        uint64_t workspace_bytes, hipStream_t stream);

/* Experts' weights [experts][rows][k]: 16-bit elements of the tokens' type, or
 * 8-bit whole numbers with scales (float [experts][rows]), or 4-bit codes with
 * powers of two as experts_quantize_mx4 makes them. Leading dimensions, and
 * strides from one expert to the next, are in elements (of codes: bytes). */
typedef enum {
    EXPERTS_WEIGHT_16 = 0,
    EXPERTS_WEIGHT_INT8 = 1,
    EXPERTS_WEIGHT_MX4 = 2
} experts_weight_kind_t;

typedef struct {
    const void *data;
    int64_t ld, stride;
    const void *scales;    /* NULL for EXPERTS_WEIGHT_16 */
    int64_t ld_scales;     /* of powers of two; not used otherwise */
    int64_t scales_stride; /* of scales or powers */
    int32_t kind;
} experts_weight_t;

/* Tokens that experts_few_tokens takes. */
#define EXPERTS_MAX_FEW 64u

/* Bytes of workspace experts_few_tokens needs; down_kind: of the second weight. */
hist_status_t experts_few_tokens_workspace_size(uint64_t tokens, uint32_t top_k,
                                                uint32_t experts, uint32_t hidden, uint32_t n,
                                                int32_t down_kind, uint64_t *bytes);

/* A whole expert layer for a few tokens. out [tokens][n], x [tokens][width]:
 *   out[t] = sum_j weights[t][j] h down[e]^T, e = ids[t][j], a = x[t] up[e]^T,
 *   h = silu(a) (gated 0), or (gated 1) silu of a's first half times its second.
 * up [experts][hidden or 2 hidden][width], down [experts][n][hidden]. ids: int32
 * or int64 (id_bits) [tokens][top_k]; an id outside [0, experts) adds nothing.
 * silu(a) = a / (1 + e^-a). Sums and h are held in 32 bits, and the result is
 * rounded once. Weights of an expert without a token are not read.
 * width and hidden are 8 or more, 16 for 8-bit weights; 64 of x's rows, and an
 * expert's rows of powers of two, lie within 2^31 bytes, and the weights' leading
 * dimensions are 2^25 at most (HIST_ERR_UNSUPPORTED otherwise).
 * workspace: 16-byte aligned, not read before it is written; calls that may run
 * at one time need one each. */
hist_status_t experts_few_tokens(void *out, int64_t ldo, const void *x, int64_t ldx,
                                 const experts_weight_t *up, const experts_weight_t *down,
                                 const void *ids, int32_t id_bits, const float *weights,
                                 uint64_t tokens, uint32_t top_k, uint32_t experts,
                                 uint32_t width, uint32_t hidden, uint32_t n, int32_t gated,
                                 int32_t dtype, void *workspace, uint64_t workspace_bytes,
                                 hipStream_t stream);

typedef enum {
    EXPERTS_MATMUL = 0,
    EXPERTS_MATMUL_DX = 1,
    EXPERTS_MATMUL_DW = 2,
    EXPERTS_INT8_MATMUL = 3,
    EXPERTS_MX4_MATMUL = 4
} experts_product_t;

typedef struct {
    uint32_t rows, cols; /* of the results that one workgroup computes */
    uint32_t threads;    /* of a workgroup */
    uint32_t stages;     /* steps of the reduction in LDS; 0: operands in registers, and the
                            reduction divided among the workgroup's waves */
    uint32_t per_cu;     /* workgroups on a CU at one time (0 where stages is) */
    uint32_t direct;     /* 1: operands go straight from memory to LDS */
} experts_kernel_t;

/* The kernel that a product of these sizes takes, computed on the host with no
 * device present, for tests of the rules. x_rows: rows of a gathered x, 0 if
 * order is NULL. experts 0: the dense 8-bit or 4-bit product. lda, ldb: the leading
 * dimensions of x and w (matmul, int8_matmul), dy and w (dx), dy and x (dw), in
 * elements; of the codes in bytes (mx4_matmul, whose powers of two start each row
 * at a multiple of 16 bytes from the first one). k: elements.
 * alignment: of the operands' addresses in bytes, a power of two; the experts'
 * weights follow one another. rows must be positive. */
hist_status_t experts_product_preview(int32_t product, uint64_t rows, uint64_t x_rows,
                                      uint32_t experts, uint32_t n, uint32_t k, int64_t lda,
                                      int64_t ldb, uint32_t alignment, experts_kernel_t *kernel);

#ifdef __cplusplus
}
#endif

#endif /* PCA_EXPERTS_H */
