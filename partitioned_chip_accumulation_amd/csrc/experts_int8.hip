// experts_int8.hip -- rows in 8 bits and their product with 8-bit weights (declared in
// experts.h).
#include "experts_product.hpp"

namespace pca_experts {

// ---------------------------------------------------------------------------
// One wave a row of x; its pieces stay in registers between the maximum and the
// rounding where the row is short enough, and come from the cache otherwise.
template <class T>
__global__ void __launch_bounds__(256)
    k_quantize(int8_t *__restrict__ xq, int64_t ldq, float *__restrict__ sx,
               const T *__restrict__ x, int64_t ldx, uint32_t rows, uint32_t k)
{
    typedef typename Vec8<T>::type V;
    const uint32_t r = blockIdx.x * 4 + threadIdx.x / 64, lane = threadIdx.x % 64;
    if (r >= rows) return;
    const T *from = x + (int64_t)r * ldx;
    int8_t *to = xq + (int64_t)r * ldq;
    // As whole numbers, magnitudes order like floats, infinity and then NaN above all.
    uint32_t top = 0;
    for (uint32_t c = lane * 8; c < k; c += 512) {
        const V v = load8(from + c, (int)(k - c));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t m = __float_as_uint((float)v[i]) & 0x7fffffffu;
            top = top > m ? top : m;
        }
    }
#pragma unroll
    for (int m = 32; m; m >>= 1) {
        const uint32_t o = __shfl_xor(top, m, 64);
        top = top > o ? top : o;
    }
    const float scale = __uint_as_float(top) / 127.0f;
    const bool finite = top < 0x7f800000u && scale > 0.f;
    if (lane == 0) sx[r] = scale;
    for (uint32_t c = lane * 8; c < k; c += 512) {
        const int left = (int)(k - c);
        const V v = load8(from + c, left);
        typedef int8_t i8x8 __attribute__((ext_vector_type(8)));
        i8x8 q;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = (float)v[i];
            float n = finite ? rintf(f / scale) : 0.f;
            // The rounded quotient can fall on the wrong side of a half. What n leaves
            // of f is exact in 32 bits, so comparing it with half the scale decides.
            const float rest = __builtin_fmaf(-n, scale, f);
            const float twice = 2.f * fabsf(rest);
            const bool odd = ((int)n & 1) != 0;
            if (finite && (twice > scale || (twice == scale && odd)))
                n += rest > 0.f ? 1.f : -1.f;
            n = fminf(fmaxf(n, -127.f), 127.f);
            q[i] = (int8_t)(int)n;
        }
        if (left >= 8) {
            store_any(to + c, q);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) to[c + i] = q[i];
        }
    }
}

}  // namespace pca_experts

using namespace pca_experts;

extern "C" hist_status_t experts_quantize_rows(int8_t *xq, int64_t ldq, float *sx, const void *x,
                                               int64_t ldx, uint64_t rows, uint32_t k,
                                               int32_t dtype, hipStream_t stream)
{
    hist_status_t st = check_sizes(rows, rows, 1, 1, 1, k);
    if (st != HIST_OK) return st;
    if (!dtype_ok(dtype) || bad_matrix(xq, ldq, k, rows, 1) || bad_matrix(x, ldx, k, rows, 2) ||
        (rows && !sx) || misaligned(sx, 4))
        return HIST_ERR_INVALID_ARG;
    st = device_status();
    if (st != HIST_OK || rows == 0) return st;
    const uint32_t blocks = (uint32_t)((rows + 3) / 4);
    if (dtype == EXPERTS_BF16)
        k_quantize<__bf16><<<blocks, 256, 0, stream>>>(xq, ldq, sx, (const __bf16 *)x, ldx,
                                                       (uint32_t)rows, k);
    else
        k_quantize<_Float16><<<blocks, 256, 0, stream>>>(xq, ldq, sx, (const _Float16 *)x, ldx,
                                                         (uint32_t)rows, k);
    return launch_status();
}

extern "C" hist_status_t experts_int8_matmul(void *y, int64_t ldy, const int8_t *xq, int64_t ldq,
                                             uint64_t x_rows, const float *sx, const int8_t *wq,
                                             int64_t ldw, int64_t w_stride, const float *sw,
                                             const int32_t *offsets, const int32_t *order,
                                             uint64_t rows, uint32_t top_k, uint32_t experts,
                                             uint32_t n, uint32_t k, int32_t dtype,
                                             hipStream_t stream)
{
    hist_status_t st = check_sizes(rows, x_rows, top_k, experts, n, k);
    if (st != HIST_OK) return st;
    if (!dtype_ok(dtype) || misaligned(offsets, 4) || misaligned(order, 4) ||
        bad_matrix(y, ldy, n, rows, 2) || bad_matrix(xq, ldq, k, rows, 1) ||
        bad_matrix(wq, ldw, k, rows, 1) || w_stride < 0 || (!order && x_rows != rows) ||
        (rows && (!x_rows || !sx || !sw)) || misaligned(sx, 4) || misaligned(sw, 4) ||
        (!offsets && (order || experts != 1)))
        return HIST_ERR_INVALID_ARG;
    st = device_status();
    if (st != HIST_OK || rows == 0) return st;
    RowsArgs g = {(char *)y, (const char *)xq, (const char *)wq, ldy * 2, ldq, ldw, w_stride,
                  offsets, order, sx, sw, (uint32_t)rows, (uint32_t)x_rows, experts, n, k,
                  0, 0, Divide::by(top_k)};
    return dtype == EXPERTS_BF16
               ? launch_rows<int8_t, __bf16, false>(g, stream)
               : launch_rows<int8_t, _Float16, false>(g, stream);
}
