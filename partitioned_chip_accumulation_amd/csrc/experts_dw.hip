// experts_dw.hip -- the gradient of the experts' weights (declared in
// experts.h).
#include "experts_product.hpp"

using namespace pca_experts;

extern "C" hist_status_t experts_matmul_dw(void *dw, const void *dy, int64_t lddy, const void *x,
                                           int64_t ldx, uint64_t x_rows, const int32_t *offsets,
                                           const int32_t *order, uint64_t rows, uint32_t top_k,
                                           uint32_t experts, uint32_t n, uint32_t k,
                                           int32_t dtype, hipStream_t stream)
{
    hist_status_t st = check_sizes(rows, x_rows, top_k, experts, n, k);
    if (st != HIST_OK) return st;
    if (!dtype_ok(dtype) || !offsets || misaligned(offsets, 4) || misaligned(order, 4) ||
        bad_matrix(dw, k, k, true, 2) || bad_matrix(dy, lddy, n, rows, 2) ||
        bad_matrix(x, ldx, k, rows, 2) || (!order && x_rows != rows) || (rows && !x_rows))
        return HIST_ERR_INVALID_ARG;
    st = device_status();
    if (st != HIST_OK) return st;
    DwArgs g = {(char *)dw, (const char *)dy, (const char *)x, lddy * 2, ldx * 2, offsets, order,
                (uint32_t)rows, (uint32_t)x_rows, experts, n, k, 0, 0, 0, Divide::by(top_k)};
    return dtype == EXPERTS_BF16 ? launch_dw<__bf16>(g, stream) : launch_dw<_Float16>(g, stream);
}
