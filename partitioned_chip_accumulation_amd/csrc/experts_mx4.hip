// experts_mx4.hip -- rows in 4 bits, a power of two for each block of 32 of their values, and their
// product with weights in the same form (declared in experts.h). The product is that of
// experts_product.hpp: steps of 128 bytes are 256 values, and the powers of two go to LDS beside the codes,
// 8 bytes of a row a step, for the matrix instruction that multiplies by them. 8192 rows, 8192 x 4096: 152-155 us,
// 3.6 PFLOP/s, the matrix cores busy 47% of the cycles and LDS for about as long (reads 31%, conflicts 6%, what
// is loaded 12% by count), not always at one time, beside the starts and ends of tiles of 16 steps; one row: 8 us,
// 2.2 TB/s of weights, in 128 workgroups.
#include "experts_product.hpp"

namespace pca_experts {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));

// Two values, divided by scale, as 4-bit codes in byte `at` of old: to nearest, ties to the even code,
// magnitudes past 6 become 6 (the instruction agrees with that rule on every finite 16-bit value).
template <int at>
__device__ __forceinline__ uint32_t two_codes(uint32_t old, bf16x2 v, float scale)
{
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, v, scale, at);
}
template <int at>
__device__ __forceinline__ uint32_t two_codes(uint32_t old, f16x2 v, float scale)
{
    return __builtin_amdgcn_cvt_scalef32_pk_fp4_f16(old, v, scale, at);
}

// A lane takes 8 values, four lanes a block. Bound by memory: 8192 rows of 4096 in 17-18 us, 4.7-5.0 TB/s.
template <class T>
__global__ void __launch_bounds__(256)
    k_quantize_mx4(uint8_t *__restrict__ xq, int64_t ldq, uint8_t *__restrict__ xs, int64_t lds,
                   const T *__restrict__ x, int64_t ldx, uint32_t rows, uint32_t k,
                   uint32_t parts)
{
    typedef typename Vec8<T>::type V;
    typedef T T2 __attribute__((ext_vector_type(2)));
    const uint32_t r = blockIdx.x / parts, c = (blockIdx.x % parts * 256 + threadIdx.x) * 8;
    const uint32_t block = c / 32;
    const V v = c < k ? load8(x + (int64_t)r * ldx + c, (int)(k - c)) : V{};
    // As whole numbers, magnitudes order like floats, infinity and then NaN above all.
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t m = __float_as_uint((float)v[i]) & 0x7fffffffu;
        top = top > m ? top : m;
    }
    uint32_t o = __shfl_xor(top, 1, 64);
    top = top > o ? top : o;
    o = __shfl_xor(top, 2, 64);
    top = top > o ? top : o;
    if (block * 32 >= k) return;
    // Its exponent less 2, so that the largest value lies in [4, 8). Below 2^-126 the exponent's
    // bits are 0, and the power is the least one, 2^-127: what a block of such values needs.
    const uint32_t exponent = top >> 23;
    const bool finite = exponent < 255;
    const uint32_t power = finite ? (exponent > 2 ? exponent - 2 : 0) : 255;
    const float scale = __uint_as_float(power ? power << 23 : 1u << 22);
    uint32_t codes = 0;
    if (finite) {
        codes = two_codes<0>(codes, T2{v[0], v[1]}, scale);
        codes = two_codes<1>(codes, T2{v[2], v[3]}, scale);
        codes = two_codes<2>(codes, T2{v[4], v[5]}, scale);
        codes = two_codes<3>(codes, T2{v[6], v[7]}, scale);
    }
    store_any(xq + (int64_t)r * ldq + c / 2, codes);
    if (threadIdx.x % 4 == 0) xs[(int64_t)r * lds + block] = (uint8_t)power;
}

template <class T>
hist_status_t launch_quantize_mx4(uint8_t *xq, int64_t ldq, uint8_t *xs, int64_t lds, const void *x,
                                  int64_t ldx, uint32_t rows, uint32_t k, hipStream_t stream)
{
    const uint32_t parts = ((k + 31) / 32 * 4 + 255) / 256;
    const uint64_t most = most_of(1, 256) / parts;
    hist_status_t st = HIST_OK;
    for (uint64_t r = 0; r < rows && st == HIST_OK; r += most) {
        const uint32_t high = (uint32_t)(rows - r < most ? rows - r : most);
        st = launch(k_quantize_mx4<T>, (uint64_t)high * parts, 256, 0, stream, xq + r * ldq, ldq,
                    xs + r * lds, lds, (const T *)x + r * ldx, ldx, high, k, parts);
    }
    return st;
}

}  // namespace pca_experts

using namespace pca_experts;

extern "C" hist_status_t experts_quantize_mx4(uint8_t *xq, int64_t ldq, uint8_t *xs, int64_t lds,
                                              const void *x, int64_t ldx, uint64_t rows,
                                              uint32_t k, int32_t dtype, hipStream_t stream)
{
    hist_status_t st = check_sizes(rows, rows, 1, 1, 1, k);
    if (st != HIST_OK) return st;
    const uint64_t blocks = (k + 31) / 32;
    if (!dtype_ok(dtype) || bad_matrix(xq, ldq, blocks * 16, rows, 1) ||
        bad_matrix(xs, lds, blocks, rows, 1) || bad_matrix(x, ldx, k, rows, 2))
        return HIST_ERR_INVALID_ARG;
    st = device_status();
    if (st != HIST_OK || rows == 0) return st;
    return (dtype == EXPERTS_BF16 ? launch_quantize_mx4<__bf16> : launch_quantize_mx4<_Float16>)(
        xq, ldq, xs, lds, x, ldx, (uint32_t)rows, k, stream);
}

extern "C" hist_status_t experts_mx4_matmul(void *y, int64_t ldy, const uint8_t *xq, int64_t ldq,
                                            const uint8_t *xs, int64_t ldxs, uint64_t x_rows,
                                            const uint8_t *wq, int64_t ldw, int64_t w_stride,
                                            const uint8_t *ws, int64_t ldws, int64_t ws_stride,
                                            const int32_t *offsets, const int32_t *order,
                                            uint64_t rows, uint32_t top_k, uint32_t experts,
                                            uint32_t n, uint32_t blocks, int32_t dtype,
                                            hipStream_t stream)
{
    if (blocks > EXPERTS_MAX_WIDTH / 32) return HIST_ERR_UNSUPPORTED;
    hist_status_t st = check_sizes(rows, x_rows, top_k, experts, n, blocks);
    if (st != HIST_OK) return st;
    if (!dtype_ok(dtype) || misaligned(offsets, 4) || misaligned(order, 4) ||
        bad_matrix(y, ldy, n, rows, 2) || bad_matrix(xq, ldq, (uint64_t)blocks * 16, rows, 1) ||
        bad_matrix(xs, ldxs, blocks, rows, 1) ||
        bad_matrix(wq, ldw, (uint64_t)blocks * 16, rows, 1) ||
        bad_matrix(ws, ldws, blocks, rows, 1) || w_stride < 0 || ws_stride < 0 ||
        (!order && x_rows != rows) || (rows && !x_rows) || (!offsets && (order || experts != 1)))
        return HIST_ERR_INVALID_ARG;
    st = device_status();
    if (st != HIST_OK || rows == 0) return st;
    RowsArgs g = {(char *)y, (const char *)xq, (const char *)wq, ldy * 2, ldq, ldw, w_stride,
                  offsets, order, nullptr, nullptr, (uint32_t)rows, (uint32_t)x_rows, experts, n,
                  blocks * 16, 0, 0, Divide::by(top_k), xs, ws, ldxs, ldws, ws_stride};
    return dtype == EXPERTS_BF16 ? launch_rows<Mx4, __bf16, false>(g, stream)
                                 : launch_rows<Mx4, _Float16, false>(g, stream);
}
