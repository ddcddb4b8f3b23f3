// experts_int8.hip -- rows in 8 bits and their product with 8-bit weights (declared in
// experts.h).
#include "experts_product.hpp"

namespace pca_experts {

// ---------------------------------------------------------------------------
// THREADS lanes a row of x. What of it a lane holds in registers (KEPT pieces of 16 bytes)
// is read once; the rest of a longer row is read again, from the cache.
template <class T, int THREADS, int KEPT>
__global__ void __launch_bounds__(256)
    k_quantize(int8_t *__restrict__ xq, int64_t ldq, float *__restrict__ sx,
               const T *__restrict__ x, int64_t ldx, uint32_t rows, uint32_t k)
{
    typedef typename Vec8<T>::type V;
    typedef int8_t i8x8 __attribute__((ext_vector_type(8)));
    __shared__ uint32_t tops[4];
    const uint32_t r = blockIdx.x * (256 / THREADS) + threadIdx.x / THREADS;
    const uint32_t lane = threadIdx.x % THREADS;
    if (r >= rows) return;  // a row is a wave's or the workgroup's
    const T *from = x + (int64_t)r * ldx;
    int8_t *to = xq + (int64_t)r * ldq;
    V kept[KEPT];
    // As whole numbers, magnitudes order like floats, infinity and then NaN above all.
    uint32_t top = 0;
    auto widen = [&](const V &v) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t m = __float_as_uint((float)v[i]) & 0x7fffffffu;
            top = top > m ? top : m;
        }
    };
#pragma unroll
    for (int s = 0; s < KEPT; ++s) {
        const uint32_t c = (s * THREADS + lane) * 8;
        kept[s] = c < k ? load8(from + c, (int)(k - c)) : V{};
    }
#pragma unroll
    for (int s = 0; s < KEPT; ++s) widen(kept[s]);
    for (uint32_t c = (KEPT * THREADS + lane) * 8; c < k; c += THREADS * 8)
        widen(load8(from + c, (int)(k - c)));
#pragma unroll
    for (int m = 32; m; m >>= 1) {
        const uint32_t o = __shfl_xor(top, m, 64);
        top = top > o ? top : o;
    }
    if constexpr (THREADS > 64) {
        if (lane % 64 == 0) tops[threadIdx.x / 64] = top;
        __syncthreads();
        top = tops[0];
#pragma unroll
        for (int w = 1; w < 4; ++w) top = top > tops[w] ? top : tops[w];
    }
    const float scale = __uint_as_float(top) / 127.0f;
    const bool finite = top < 0x7f800000u && scale > 0.f;
    if (lane == 0) sx[r] = scale;
    // The quotient by the reciprocal is within 127 * 2^-23 of the real one, so its rounding is
    // right unless it lies next to a half; only pieces with such a value, and rows whose scale has no
    // normal reciprocal, take the way that decides exactly (done for every value, the kernel was
    // bound by its arithmetic: 8192 x 4096 in 30 us).
    const bool normal = scale > 1e-37f && scale < 1e37f;
    const float inverse = normal ? 1.0f / scale : 0.f;
    auto quantize = [&](const V &v, uint32_t c) {
        const int left = (int)(k - c);
        i8x8 q = {};
        if (finite) {
            float n[8];
            bool near_half = !normal;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float t = (float)v[i] * inverse;
                n[i] = rintf(t);
                near_half |= fabsf(t - n[i]) > 0.4999f;
            }
            if (near_half) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float f = (float)v[i];
                    float m = rintf(f / scale);
                    // what m leaves of f is exact in 32 bits: comparing it with half the scale
                    // decides
                    const float rest = __builtin_fmaf(-m, scale, f);
                    const float twice = 2.f * fabsf(rest);
                    const bool odd = ((int)m & 1) != 0;
                    if (twice > scale || (twice == scale && odd)) m += rest > 0.f ? 1.f : -1.f;
                    n[i] = fminf(fmaxf(m, -127.f), 127.f);
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) q[i] = (int8_t)(int)n[i];
        }
        if (left >= 8) {
            store_any(to + c, q);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                if (i < left) to[c + i] = q[i];
        }
    };
#pragma unroll
    for (int s = 0; s < KEPT; ++s) {
        const uint32_t c = (s * THREADS + lane) * 8;
        if (c < k) quantize(kept[s], c);
    }
    for (uint32_t c = (KEPT * THREADS + lane) * 8; c < k; c += THREADS * 8)
        quantize(load8(from + c, (int)(k - c)), c);
}

// A wave a row up to 1024 columns (two pieces a lane); the workgroup otherwise (8192 x 4096: 28 us,
// 3.6 TB/s; a wave a row with eight pieces a lane 33 us).
template <class T>
hist_status_t launch_quantize(int8_t *xq, int64_t ldq, float *sx, const void *x, int64_t ldx,
                              uint32_t rows, uint32_t k, hipStream_t stream)
{
    const bool narrow = k <= 1024;
    const uint64_t most = most_of(narrow ? 4 : 1, 256);
    hist_status_t st = HIST_OK;
    for (uint64_t r = 0; r < rows && st == HIST_OK; r += most) {
        const uint32_t high = (uint32_t)(rows - r < most ? rows - r : most);
        int8_t *to = xq + r * ldq;
        const T *from = (const T *)x + r * ldx;
        st = narrow ? launch(k_quantize<T, 64, 2>, (high + 3) / 4, 256, 0, stream, to, ldq, sx + r,
                             from, ldx, high, k)
                    : launch(k_quantize<T, 256, 4>, high, 256, 0, stream, to, ldq, sx + r, from,
                             ldx, high, k);
    }
    return st;
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
    return (dtype == EXPERTS_BF16 ? launch_quantize<__bf16> : launch_quantize<_Float16>)(
        xq, ldq, sx, x, ldx, (uint32_t)rows, k, stream);
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
