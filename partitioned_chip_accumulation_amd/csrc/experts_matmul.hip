// experts_matmul.hip -- the products of an expert layer (declared in
// experts.h): rows times weights, the two gradients, and the 8-bit product.
#include "experts_tile.hpp"

namespace pca_experts {

// The tile: 128 x 128 results by four waves of 64 x 64 each.
constexpr int kTile = 128;
constexpr int kThreads = 256;
constexpr int kPart = 64;         // rows and columns of one wave
constexpr int kFrags = kPart / 16;

struct RowsArgs {
    char *out;
    const char *a;
    const char *b;
    int64_t ldo, lda, ldb, b_stride;  // bytes
    const int32_t *offsets;           // nullptr: one group
    const int32_t *order;             // nullptr: row p of a belongs to row p
    const float *sa, *sb;             // 8-bit operands' scales
    uint32_t rows, a_rows, top_k, experts;
    uint32_t cols;   // of the result
    uint32_t bytes;  // of the reduction
    uint32_t n_tiles, span;
};

// The row of a that sorted row p reads; a bad index reads row 0 (the row's
// place in the result is still its own).
__device__ __forceinline__ uint32_t source_row(const RowsArgs &g, uint32_t p)
{
    if (!g.order) return p;
    const uint32_t t = (uint32_t)g.order[p] / g.top_k;
    return t < g.a_rows ? t : 0;
}

template <class O>
__device__ __forceinline__ void store4(O *p, const float *v, int left)
{
    typedef O O4 __attribute__((ext_vector_type(4)));
    const O4 r = {(O)v[0], (O)v[1], (O)v[2], (O)v[3]};
    if (left >= 4) {
        store_any(p, r);
    } else {
#pragma unroll
        for (int i = 0; i < 3; ++i)
            if (i < left) p[i] = r[i];
    }
}

// T: element of the operands; O: of the result; B: how the weights are staged.
template <class T, class O, class B>
__global__ void __launch_bounds__(kThreads) k_rows(RowsArgs g)
{
    typedef Along<T, kTile, kThreads> A;
    typedef typename Mma<T>::Acc Acc;
    __shared__ __align__(16) char lds[2][A::kBytes + B::kBytes];
    const Tile t = find_tile(tile_of_block(blockIdx.x, g.span), g.offsets, g.experts, g.rows, 7,
                             g.n_tiles);
    if (t.group > g.experts) return;
    const uint32_t m0 = t.begin + t.m * kTile, n0 = t.n * kTile;
    const uint32_t high = t.end - m0 < kTile ? t.end - m0 : kTile;
    const uint32_t wide = g.cols - n0 < kTile ? g.cols - n0 : kTile;
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const uint32_t wm = wave / 2 * kPart, wn = wave % 2 * kPart;
    Acc acc[kFrags][kFrags] = {};

    if (!g.offsets || t.group < g.experts) {
        A a;
        B b;
        a.init([&](uint32_t r) {
            return g.a + (int64_t)source_row(g, m0 + (r < high ? r : high - 1)) * g.lda;
        });
        const char *w = g.b + (int64_t)t.group * g.b_stride;
        if constexpr (B::kAcross) b.init((int)wide);
        else b.init([&](uint32_t r) { return w + (int64_t)(n0 + (r < wide ? r : wide - 1)) * g.ldb; });
        const uint32_t steps = (g.bytes + kStepBytes - 1) / kStepBytes;
        auto fetch = [&](uint32_t step) {
            a.fetch(step, g.bytes);
            if constexpr (B::kAcross)
                b.fetch([&](uint32_t r) -> const char * {
                    const uint32_t at = step * B::kRows + r;
                    return at * 2 < g.bytes ? w + (int64_t)at * g.ldb + n0 * 2 : nullptr;
                });
            else b.fetch(step, g.bytes);
        };
        fetch(0);
        for (uint32_t step = 0; step < steps; ++step) {
            char *la = lds[step & 1], *lb = la + A::kBytes;
            a.store(la);
            b.store(lb);
            __syncthreads();  // every wave is then past the other half's reads
            if (step + 1 < steps) fetch(step + 1);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                typename Mma<T>::Frag fa[kFrags], fb[kFrags];
#pragma unroll
                for (int i = 0; i < kFrags; ++i) {
                    fa[i] = A::frag(la, wm + i * 16, kk);
                    fb[i] = B::frag(lb, wn + i * 16, kk);
                }
#pragma unroll
                for (int i = 0; i < kFrags; ++i)
#pragma unroll
                    for (int j = 0; j < kFrags; ++j)
                        acc[i][j] = Mma<T>::run(fb[j], fa[i], acc[i][j]);
            }
        }
    }

    const uint32_t c0 = wn + lane / 16 * 4;
#pragma unroll
    for (int i = 0; i < kFrags; ++i) {
        const uint32_t r = wm + i * 16 + lane % 16;
        if (r >= high) continue;
        O *out = (O *)(g.out + (int64_t)(m0 + r) * g.ldo) + n0;
        float s = 1.f;
        if constexpr (sizeof(T) == 1)
            s = !g.offsets || t.group < g.experts ? g.sa[source_row(g, m0 + r)] : 0.f;
#pragma unroll
        for (int j = 0; j < kFrags; ++j) {
            const uint32_t c = c0 + j * 16;
            const int left = (int)wide - (int)c;
            if (left <= 0) continue;
            float v[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                v[q] = (float)acc[i][j][q];
                if constexpr (sizeof(T) == 1)
                    if (t.group < g.experts || !g.offsets)
                        v[q] = v[q] * s *
                               g.sb[(uint64_t)t.group * g.cols + n0 + c + (q < left ? q : 0)];
            }
            store4(out + c, v, left);
        }
    }
}

struct DwArgs {
    char *out;
    const char *dy;
    const char *x;
    int64_t lddy, ldx;  // bytes
    const int32_t *offsets;
    const int32_t *order;
    uint32_t rows, x_rows, top_k, experts, n, k;
    uint32_t n_tiles, k_tiles, span;
};

template <class T>
__global__ void __launch_bounds__(kThreads) k_dw(DwArgs g)
{
    typedef Across<T, kTile, kThreads> A;
    typedef typename Mma<T>::Acc Acc;
    __shared__ __align__(16) char lds[2][2 * A::kBytes];
    const uint32_t tile = tile_of_block(blockIdx.x, g.span);
    const uint32_t each = g.n_tiles * g.k_tiles, e = tile / each;
    if (e >= g.experts) return;
    const uint32_t in = tile - e * each;
    const uint32_t n0 = in % g.n_tiles * kTile, k0 = in / g.n_tiles * kTile;
    const uint32_t high = g.n - n0 < kTile ? g.n - n0 : kTile;
    const uint32_t wide = g.k - k0 < kTile ? g.k - k0 : kTile;
    uint32_t end = (uint32_t)g.offsets[e + 1], begin = (uint32_t)g.offsets[e];
    end = end > g.rows ? g.rows : end;
    begin = begin > end ? end : begin;
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const uint32_t wm = wave / 2 * kPart, wn = wave % 2 * kPart;
    Acc acc[kFrags][kFrags] = {};
    A a, b;
    a.init((int)high);
    b.init((int)wide);
    auto fetch = [&](uint32_t p0) {
        a.fetch([&](uint32_t r) -> const char * {
            const uint32_t p = p0 + r;
            return p < end ? g.dy + (int64_t)p * g.lddy + n0 * 2 : nullptr;
        });
        b.fetch([&](uint32_t r) -> const char * {
            const uint32_t p = p0 + r;
            if (p >= end) return nullptr;
            const uint32_t s = g.order ? (uint32_t)g.order[p] / g.top_k : p;
            return s < g.x_rows ? g.x + (int64_t)s * g.ldx + k0 * 2 : nullptr;
        });
    };
    if (begin < end) fetch(begin);
    uint32_t half = 0;
    for (uint32_t p0 = begin; p0 < end; p0 += A::kRows, half ^= 1) {
        char *la = lds[half], *lb = la + A::kBytes;
        a.store(la);
        b.store(lb);
        __syncthreads();
        if (p0 + A::kRows < end) fetch(p0 + A::kRows);
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            typename Mma<T>::Frag fa[kFrags], fb[kFrags];
#pragma unroll
            for (int i = 0; i < kFrags; ++i) {
                fa[i] = A::frag(la, wm + i * 16, kk);
                fb[i] = A::frag(lb, wn + i * 16, kk);
            }
#pragma unroll
            for (int i = 0; i < kFrags; ++i)
#pragma unroll
                for (int j = 0; j < kFrags; ++j)
                    acc[i][j] = Mma<T>::run(fb[j], fa[i], acc[i][j]);
        }
    }
#pragma unroll
    for (int i = 0; i < kFrags; ++i) {
        const uint32_t r = wm + i * 16 + lane % 16;
        if (r >= high) continue;
        T *out = (T *)g.out + ((int64_t)e * g.n + n0 + r) * g.k + k0;
#pragma unroll
        for (int j = 0; j < kFrags; ++j) {
            const uint32_t c = wn + lane / 16 * 4 + j * 16;
            if (c >= wide) continue;
            const float v[4] = {acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3]};
            store4(out + c, v, (int)(wide - c));
        }
    }
}

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

// Row tiles there can be: a group of c rows has ceil(c / tile), over the
// experts and the rows past the last kept one.
inline uint64_t most_row_tiles(uint64_t rows, uint64_t groups, uint32_t tile)
{
    const uint64_t m = (rows + groups * (tile - 1)) / tile;
    return m < rows ? m : rows;
}

inline uint32_t span_of(uint64_t tiles)
{
    const uint64_t s = tiles / 8;
    return s < 1 ? 1 : s > 32 ? 32 : (uint32_t)s;
}

template <class T, class O, class B>
hist_status_t launch_rows(RowsArgs g, hipStream_t stream)
{
    g.n_tiles = (g.cols + kTile - 1) / kTile;
    const uint64_t tiles =
        most_row_tiles(g.rows, g.offsets ? g.experts + 1 : 1, kTile) * g.n_tiles;
    g.span = span_of(tiles);
    const uint64_t blocks = (tiles + 8 * g.span - 1) / (8 * g.span) * (8 * g.span);
    if (blocks > INT32_MAX) return HIST_ERR_UNSUPPORTED;
    if (blocks) k_rows<T, O, B><<<(uint32_t)blocks, kThreads, 0, stream>>>(g);
    return launch_status();
}

// Checks that the products share. `unit`: bytes of an element of the result
// of a leading dimension.
inline bool bad_matrix(const void *p, int64_t ld, uint64_t width, bool used, uintptr_t align)
{
    return (used && !p) || ld < (int64_t)width || misaligned(p, align);
}

inline hist_status_t check_sizes(uint64_t rows, uint64_t x_rows, uint32_t top_k, uint32_t experts,
                                 uint32_t n, uint32_t k)
{
    if (experts == 0 || n == 0 || k == 0 || top_k == 0) return HIST_ERR_INVALID_ARG;
    if (experts > EXPERTS_MAX_EXPERTS || n > EXPERTS_MAX_WIDTH || k > EXPERTS_MAX_WIDTH ||
        rows > EXPERTS_MAX_ROWS || x_rows > EXPERTS_MAX_ROWS)
        return HIST_ERR_UNSUPPORTED;
    return HIST_OK;
}

}  // namespace pca_experts

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
                  (uint32_t)x_rows, top_k, experts, n, k * 2, 0, 0};
    return dtype == EXPERTS_BF16
               ? launch_rows<__bf16, __bf16, Along<__bf16, kTile, kThreads>>(g, stream)
               : launch_rows<_Float16, _Float16, Along<_Float16, kTile, kThreads>>(g, stream);
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
                  (uint32_t)rows, 1, experts, k, n * 2, 0, 0};
    return dtype == EXPERTS_BF16
               ? launch_rows<__bf16, __bf16, Across<__bf16, kTile, kThreads>>(g, stream)
               : launch_rows<_Float16, _Float16, Across<_Float16, kTile, kThreads>>(g, stream);
}

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
                (uint32_t)rows, (uint32_t)x_rows, top_k, experts, n, k, (n + kTile - 1) / kTile,
                (k + kTile - 1) / kTile, 0};
    const uint64_t tiles = (uint64_t)g.n_tiles * g.k_tiles * experts;
    g.span = span_of(tiles);
    const uint64_t blocks = (tiles + 8 * g.span - 1) / (8 * g.span) * (8 * g.span);
    if (blocks > INT32_MAX) return HIST_ERR_UNSUPPORTED;
    if (dtype == EXPERTS_BF16) k_dw<__bf16><<<(uint32_t)blocks, kThreads, 0, stream>>>(g);
    else k_dw<_Float16><<<(uint32_t)blocks, kThreads, 0, stream>>>(g);
    return launch_status();
}

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
                  offsets, order, sx, sw, (uint32_t)rows, (uint32_t)x_rows, top_k, experts, n, k,
                  0, 0};
    return dtype == EXPERTS_BF16
               ? launch_rows<int8_t, __bf16, Along<int8_t, kTile, kThreads>>(g, stream)
               : launch_rows<int8_t, _Float16, Along<int8_t, kTile, kThreads>>(g, stream);
}
