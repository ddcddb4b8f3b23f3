// experts_combine.hip -- expert outputs back to their tokens, and the
// gradients of that sum (declared in experts.h). Both are bound by memory: each
// row is read or written once, 16 bytes a lane. 16384 tokens of 4 choices, 4096 columns: 132 us, 5.1
// TB/s; the gradients of 8191 tokens of 8, 2048 columns: 116 us, 4.9 TB/s (a copy of
// 1 GiB reaches 5.25 TB/s).
#include "experts_common.hpp"

namespace pca_experts {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kCols = 8;  // elements of one lane's access

// A group of 2^lanes_log2 lanes takes one token's next 8 << lanes_log2 columns
// and reads the rows of four choices before it adds the first, so that their
// latencies overlap.
template <class T>
__global__ void __launch_bounds__(kThreads)
    k_combine(T *__restrict__ out, int64_t ldo, const T *__restrict__ y, int64_t ldy,
              uint32_t rows, const int32_t *__restrict__ place,
              const float *__restrict__ weights, uint32_t tokens, uint32_t top_k, uint32_t n,
              uint32_t lanes_log2, uint32_t parts)
{
    typedef typename Vec8<T>::type V;
    const uint64_t group = ((uint64_t)blockIdx.x * kThreads + threadIdx.x) >> lanes_log2;
    const uint32_t lane = threadIdx.x & ((1u << lanes_log2) - 1);
    const uint64_t token = group / parts;
    if (token >= tokens) return;
    const uint32_t col = ((uint32_t)(group % parts) << lanes_log2) * kCols + lane * kCols;
    if (col >= n) return;
    const int left = (int)(n - col);
    const int32_t *places = place + token * top_k;
    const float *weight = weights ? weights + token * top_k : nullptr;
    float sum[kCols] = {};
    for (uint32_t j0 = 0; j0 < top_k; j0 += 4) {
        V v[4];
        float w[4];
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            v[j] = V{};
            w[j] = 0.f;
            if (j0 + j < top_k) {
                const uint32_t p = (uint32_t)places[j0 + j];
                if (p < rows) {
                    w[j] = weight ? weight[j0 + j] : 1.f;
                    v[j] = load8(y + (int64_t)p * ldy + col, left);
                }
            }
        }
#pragma unroll
        for (uint32_t j = 0; j < 4; ++j) {
            if (j0 + j < top_k && (uint32_t)places[j0 + j] < rows)
#pragma unroll
                for (uint32_t c = 0; c < kCols; ++c)
                    sum[c] = __builtin_fmaf(w[j], (float)v[j][c], sum[c]);
        }
    }
    V r;
#pragma unroll
    for (uint32_t c = 0; c < kCols; ++c) r[c] = (T)sum[c];
    store8(out + (int64_t)token * ldo + col, r, left);
}

// One wave a pair i: dy's row place[i] and the weight's gradient, whose sum
// has a fixed order. The waves of a token's choices are neighbours, so its row
// of dout comes from the cache after the first. Wave i also clears row i of dy
// where that lies past the last kept pair.
template <class T>
__global__ void __launch_bounds__(kThreads)
    k_combine_backward(T *__restrict__ dy, int64_t lddy, float *__restrict__ dweights,
                       const T *__restrict__ dout, int64_t lddout, const T *__restrict__ y,
                       int64_t ldy, const int32_t *__restrict__ order,
                       const int32_t *__restrict__ place, const float *__restrict__ weights,
                       uint32_t first, uint32_t pairs, uint32_t top_k, uint32_t n)
{
    typedef typename Vec8<T>::type V;
    const uint32_t i = first + __builtin_amdgcn_readfirstlane(blockIdx.x * (kThreads / 64) +
                                                              threadIdx.x / 64);
    if (i >= pairs) return;
    const uint32_t lane = threadIdx.x % 64;
    if ((uint32_t)order[i] >= pairs) {
        T *row = dy + (int64_t)i * lddy;
        for (uint32_t col = lane * kCols; col < n; col += 64 * kCols)
            store8(row + col, V{}, (int)(n - col));
    }
    const uint32_t p = (uint32_t)place[i];
    if (p >= pairs) {
        if (lane == 0) dweights[i] = 0.f;
        return;
    }
    const float w = weights[i];
    const T *d = dout + (int64_t)(i / top_k) * lddout;
    const T *from = y + (int64_t)p * ldy;
    T *to = dy + (int64_t)p * lddy;
    float dot = 0.f;
    for (uint32_t col = lane * kCols; col < n; col += 64 * kCols) {
        const int left = (int)(n - col);
        const V a = load8(d + col, left), b = load8(from + col, left);
        V r;
#pragma unroll
        for (uint32_t c = 0; c < kCols; ++c) {
            dot = __builtin_fmaf((float)a[c], (float)b[c], dot);
            r[c] = (T)(w * (float)a[c]);
        }
        store8(to + col, r, left);
    }
    dot = wave_sum_f(dot);
    if (lane == 0) dweights[i] = dot;
}

}  // namespace pca_experts

using namespace pca_experts;

template <class T>
static hist_status_t launch_combine(void *out, int64_t ldo, const void *y, int64_t ldy,
                                    uint32_t rows, const int32_t *place, const float *weights,
                                    uint64_t tokens, uint32_t top_k, uint32_t n,
                                    hipStream_t stream)
{
    uint32_t lanes_log2 = 4;
    while (lanes_log2 < 6 && (kCols << lanes_log2) < n) ++lanes_log2;
    const uint32_t parts = (n + (kCols << lanes_log2) - 1) / (kCols << lanes_log2);
    const uint64_t most = (most_of(kThreads, kThreads) >> lanes_log2) / parts;
    hist_status_t st = HIST_OK;
    for (uint64_t t = 0; t < tokens && st == HIST_OK; t += most) {
        const uint64_t some = tokens - t < most ? tokens - t : most;
        const uint64_t blocks = (((some * parts) << lanes_log2) + kThreads - 1) / kThreads;
        st = launch(k_combine<T>, blocks, kThreads, 0, stream, (T *)out + t * ldo, ldo,
                    (const T *)y, ldy, rows, place + t * top_k,
                    weights ? weights + t * top_k : nullptr, (uint32_t)some, top_k, n, lanes_log2,
                    parts);
    }
    return st;
}

template <class T>
static hist_status_t launch_combine_backward(void *dy, int64_t lddy, float *dweights,
                                             const void *dout, int64_t lddout, const void *y,
                                             int64_t ldy, const int32_t *order,
                                             const int32_t *place, const float *weights,
                                             uint32_t pairs, uint32_t top_k, uint32_t n,
                                             hipStream_t stream)
{
    constexpr uint32_t kEach = kThreads / 64;
    const uint64_t most = most_of(kEach, kThreads);
    hist_status_t st = HIST_OK;
    for (uint64_t first = 0; first < pairs && st == HIST_OK; first += most) {
        const uint64_t some = pairs - first < most ? pairs - first : most;
        st = launch(k_combine_backward<T>, (some + kEach - 1) / kEach, kThreads, 0, stream, (T *)dy,
                    lddy, dweights, (const T *)dout, lddout, (const T *)y, ldy, order, place,
                    weights, (uint32_t)first, pairs, top_k, n);
    }
    return st;
}

static hist_status_t check_rows(uint64_t tokens, uint32_t top_k, uint32_t n, int32_t dtype)
{
    if (!dtype_ok(dtype) || top_k == 0 || n == 0) return HIST_ERR_INVALID_ARG;
    if (top_k > EXPERTS_MAX_TOP_K || n > EXPERTS_MAX_WIDTH || tokens > EXPERTS_MAX_ROWS / top_k)
        return HIST_ERR_UNSUPPORTED;
    return HIST_OK;
}

extern "C" hist_status_t experts_combine(void *out, int64_t ldo, const void *y, int64_t ldy,
                                         uint64_t rows, const int32_t *place,
                                         const float *weights, uint64_t tokens, uint32_t top_k,
                                         uint32_t n, int32_t dtype, hipStream_t stream)
{
    hist_status_t st = check_rows(tokens, top_k, n, dtype);
    if (st != HIST_OK) return st;
    if (rows > EXPERTS_MAX_ROWS) return HIST_ERR_UNSUPPORTED;
    if (tokens && (!out || !place)) return HIST_ERR_INVALID_ARG;
    if (rows && tokens && !y) return HIST_ERR_INVALID_ARG;
    if (ldo < (int64_t)n || ldy < (int64_t)n || misaligned(out, 2) || misaligned(y, 2) ||
        misaligned(place, 4) || misaligned(weights, 4))
        return HIST_ERR_INVALID_ARG;
    st = device_status();
    if (st != HIST_OK || tokens == 0) return st;
    return (dtype == EXPERTS_BF16 ? launch_combine<__bf16> : launch_combine<_Float16>)(
        out, ldo, y, ldy, (uint32_t)rows, place, weights, tokens, top_k, n, stream);
}

extern "C" hist_status_t experts_combine_backward(void *dy, int64_t lddy, float *dweights,
                                                  const void *dout, int64_t lddout, const void *y,
                                                  int64_t ldy, const int32_t *order,
                                                  const int32_t *place, const float *weights,
                                                  uint64_t tokens, uint32_t top_k, uint32_t n,
                                                  int32_t dtype, hipStream_t stream)
{
    hist_status_t st = check_rows(tokens, top_k, n, dtype);
    if (st != HIST_OK) return st;
    if (tokens && (!dy || !dweights || !dout || !y || !order || !place || !weights))
        return HIST_ERR_INVALID_ARG;
    if (lddy < (int64_t)n || lddout < (int64_t)n || ldy < (int64_t)n || misaligned(dy, 2) ||
        misaligned(dout, 2) || misaligned(y, 2) || misaligned(dweights, 4) ||
        misaligned(order, 4) || misaligned(place, 4) || misaligned(weights, 4))
        return HIST_ERR_INVALID_ARG;
    st = device_status();
    if (st != HIST_OK || tokens == 0) return st;
    return (dtype == EXPERTS_BF16 ? launch_combine_backward<__bf16>
                                  : launch_combine_backward<_Float16>)(
        dy, lddy, dweights, dout, lddout, y, ldy, order, place, weights,
        (uint32_t)(tokens * top_k), top_k, n, stream);
}
