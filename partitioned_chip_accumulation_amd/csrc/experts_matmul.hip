// experts_matmul.hip -- rows times their experts' weights, and the gradient of the rows (declared in
// experts.h).
#include "experts_product.hpp"

using namespace pca_experts;

extern "C" hist_status_t experts_matmul(void *y, int64_t ldy, const void *x, int64_t ldx,
                                        uint64_t x_rows, const void *w, int64_t ldw,
                                        int64_t w_stride, const int32_t *offsets,
                                        const int32_t *order, uint64_t rows, uint32_t top_k,
                                        uint32_t experts, uint32_t n, uint32_t k, int32_t dtype,
                                        hipStream_t stream)
{
    hist_status_t st = check_sizes(rows, x_rows, top_k, experts, n, k);
    if (st != HIST_OK) return st;
    if (!dtype_ok(dtype) || !offsets || misaligned(offsets, 4) || misaligned(order, 4) ||
        bad_matrix(y, ldy, n, rows, 2) || bad_matrix(x, ldx, k, rows, 2) ||
        bad_matrix(w, ldw, k, rows, 2) || w_stride < 0 || (!order && x_rows != rows) ||
        (rows && !x_rows))
        return HIST_ERR_INVALID_ARG;
    st = device_status();
    if (st != HIST_OK || rows == 0) return st;
    RowsArgs g = {(char *)y, (const char *)x, (const char *)w, ldy * 2, ldx * 2, ldw * 2,
                  w_stride * 2, offsets, order, nullptr, nullptr, (uint32_t)rows,
                  (uint32_t)x_rows, experts, n, k * 2, 0, 0, Divide::by(top_k)};
    return dtype == EXPERTS_BF16
               ? launch_rows<__bf16, __bf16, false>(g, stream)
               : launch_rows<_Float16, _Float16, false>(g, stream);
}

extern "C" hist_status_t experts_matmul_dx(void *dx, int64_t lddx, const void *dy, int64_t lddy,
                                           const void *w, int64_t ldw, int64_t w_stride,
                                           const int32_t *offsets, uint64_t rows,
                                           uint32_t experts, uint32_t n, uint32_t k,
                                           int32_t dtype, hipStream_t stream)
{
    hist_status_t st = check_sizes(rows, rows, 1, experts, n, k);
    if (st != HIST_OK) return st;
    if (!dtype_ok(dtype) || !offsets || misaligned(offsets, 4) ||
        bad_matrix(dx, lddx, k, rows, 2) || bad_matrix(dy, lddy, n, rows, 2) ||
        bad_matrix(w, ldw, k, rows, 2) || w_stride < 0)
        return HIST_ERR_INVALID_ARG;
    st = device_status();
    if (st != HIST_OK || rows == 0) return st;
    RowsArgs g = {(char *)dx, (const char *)dy, (const char *)w, lddx * 2, lddy * 2, ldw * 2,
                  w_stride * 2, offsets, nullptr, nullptr, nullptr, (uint32_t)rows,
                  (uint32_t)rows, experts, k, n * 2, 0, 0, Divide::by(1)};
    return dtype == EXPERTS_BF16
               ? launch_rows<__bf16, __bf16, true>(g, stream)
               : launch_rows<_Float16, _Float16, true>(g, stream);
}

// The rules read the operands' addresses, so the preview makes up addresses as aligned as it is told.
extern "C" hist_status_t experts_product_preview(int32_t product, uint64_t rows, uint64_t x_rows,
                                                 uint32_t experts, uint32_t n, uint32_t k,
                                                 int64_t lda, int64_t ldb, uint32_t alignment,
                                                 experts_kernel_t *kernel)
{
    const bool mx4 = product == EXPERTS_MX4_MATMUL;
    const bool dense = (product == EXPERTS_INT8_MATMUL || mx4) && experts == 0, gather = x_rows != 0;
    if (!kernel || product < EXPERTS_MATMUL || product > EXPERTS_MX4_MATMUL || alignment == 0 ||
        (alignment & (alignment - 1)) || (gather && (dense || product == EXPERTS_MATMUL_DX)))
        return HIST_ERR_INVALID_ARG;
    const uint32_t groups = dense ? 1 : experts;
    const hist_status_t st = check_sizes(rows, x_rows, 1, groups, n, k);
    if (st != HIST_OK) return st;
    const bool dx = product == EXPERTS_MATMUL_DX, dw = product == EXPERTS_MATMUL_DW;
    const uint32_t blocks = (k + 31) / 32, width = mx4 ? blocks * 16 : k;
    if (lda < (int64_t)(dx || dw ? n : width) || ldb < (int64_t)width || rows == 0)
        return HIST_ERR_INVALID_ARG;
    char *const at = (char *)(uintptr_t)alignment;
    const int32_t *const list = (const int32_t *)at;  // not read here
    const int64_t size = product == EXPERTS_INT8_MATMUL || mx4 ? 1 : 2;
    const uint32_t a_rows = (uint32_t)(gather ? x_rows : rows);
    if (dw) {
        const DwArgs g = {at, at, at, lda * size, ldb * size, list, gather ? list : nullptr,
                          (uint32_t)rows, a_rows, groups, n, k, 0, 0, 0, Divide::by(1)};
        return with_dw_kernel(dw_kernel(g), DescribeKernel{kernel});
    }
    const uint32_t reduction = dx ? n : width;
    RowsArgs g = {at, at, at, 0, lda * size, ldb * size, ldb * size * n,
                        dense ? nullptr : list, gather ? list : nullptr, nullptr, nullptr,
                        (uint32_t)rows, a_rows, groups, dx ? k : n, (uint32_t)(reduction * size), 0,
                        0, Divide::by(1)};
    if (mx4) {
        g.pa = g.pb = (const uint8_t *)at;
        g.ldpa = g.ldpb = (blocks + 15) / 16 * 16;
        g.pb_stride = g.ldpb * n;
        return with_rows_kernel<false, true>(rows_kernel<false, true>(g), DescribeKernel{kernel});
    }
    return dx ? with_rows_kernel<true>(rows_kernel<true>(g), DescribeKernel{kernel})
              : with_rows_kernel<false>(rows_kernel<false>(g), DescribeKernel{kernel});
}
