// experts_norm.hip -- the root-mean-square norm before an expert layer, with the residual's
// addition, in 16 or 8 bits, and its gradients (declared in experts.h).
//
//   h = x + residual, r = (mean h^2 + eps)^-1/2, y = h r weight
//   dn = dy weight, u = h r:  dx = r (dn - u mean(dn u)) + dh, dweight = sum over rows of dy u
//
// All are bound by memory: each row is read once and kept in registers between its sums and its
// results. 16384 rows of 4096 in bf16, with the residual and h: 93-98 us, 5.5-5.8 TB/s (a large copy runs at
// 5.1); 8192 of them to 8 bits: 45 us, 5.3 TB/s; the gradients of 8191 rows of 2048: 27-29 us, 4.6-5.0 TB/s,
// and 4 for the groups' sums; 32 rows of 4096: 5.4-6 us, the launch and a row's latency. Rows of fewer than 512
// columns leave lanes of their wave without work: 67 MB of rows of 512, 256, 128 and 64 columns with the residual
// and h take 42, 53, 90 and 164 us, their gradients 58, 93, 165 and 310.
#include "experts_common.hpp"

namespace pca_experts {

constexpr uint32_t kCols = 8;  // elements of one lane's access
constexpr uint32_t kBlock = 256;

template <class T> using V8 = typename Vec8<T>::type;

// A row whose squares overflow (values past 2^55 or so) is summed again, each value 2^80 times
// smaller; what that loses is below the last bit of the sum. Only a row that holds an infinity or a
// NaN has no finite sum then.
constexpr float kSmaller = 0x1p-80f;

// Sums over the THREADS lanes of a row, in a fixed order; every lane gets them. lds: a row's own
// kN * THREADS / 64 floats, used once between two barriers.
template <int THREADS, int kN>
__device__ __forceinline__ void row_sums(float (&v)[kN], float *lds)
{
#pragma unroll
    for (int i = 0; i < kN; ++i) v[i] = wave_sum_f(v[i]);
    if constexpr (THREADS > 64) {
        constexpr int kWaves = THREADS / 64;
        __syncthreads();  // the sums before these have been read
        if (threadIdx.x % 64 == 0)
#pragma unroll
            for (int i = 0; i < kN; ++i) lds[i * kWaves + threadIdx.x / 64] = v[i];
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kN; ++i) {
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) s += lds[i * kWaves + w];
            v[i] = s;
        }
    }
}

template <int THREADS>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t *lds)
{
#pragma unroll
    for (int m = 32; m; m >>= 1) {
        const uint32_t o = __shfl_xor(v, m, 64);
        v = v > o ? v : o;
    }
    if constexpr (THREADS > 64) {
        constexpr int kWaves = THREADS / 64;
        __syncthreads();
        if (threadIdx.x % 64 == 0) lds[threadIdx.x / 64] = v;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v = v > lds[w] ? v : lds[w];
    }
    return v;
}

struct NormArgs {
    void *y, *h;         // y: T, or int8_t with the rows' scales in sx
    float *sx;
    const void *x, *residual, *weight;
    int64_t ldy, ldh, ldx, ldr;  // elements
    uint32_t rows, n;
    float eps;
};

// THREADS lanes a row, KEPT pieces of 16 bytes of it in registers; what a longer row has beyond
// them is read again (from h, which this lane wrote, where there is a residual). With a residual h
// is stored in T, and the norm is that of the stored values: the backward pass and the
// next residual see the same ones.
template <class T, int THREADS, int KEPT, bool RESIDUAL, bool INT8>
__global__ void __launch_bounds__(THREADS > kBlock ? THREADS : kBlock) k_norm(NormArgs g)
{
    constexpr uint32_t kRows = THREADS > kBlock ? 1 : kBlock / THREADS;
    __shared__ float sums[THREADS / 64];
    const uint32_t r = blockIdx.x * kRows + (kRows > 1 ? threadIdx.x / THREADS : 0);
    const uint32_t lane = kRows > 1 ? threadIdx.x % THREADS : threadIdx.x;
    if (r >= g.rows) return;  // a row is a wave's or the workgroup's
    const T *x = (const T *)g.x + (int64_t)r * g.ldx;
    const T *residual = (const T *)g.residual + (int64_t)r * g.ldr;
    T *h = (T *)g.h + (int64_t)r * g.ldh;
    const T *weight = (const T *)g.weight;
    const uint32_t n = g.n;
    constexpr uint32_t kFirst = KEPT * THREADS * kCols;  // columns in registers

    auto read = [&](uint32_t c) {
        V8<T> v = load8(x + c, (int)(n - c));
        if constexpr (RESIDUAL) {
            const V8<T> o = load8(residual + c, (int)(n - c));
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = (T)((float)v[i] + (float)o[i]);
        }
        return v;
    };
    auto again = [&](uint32_t c) { return load8((RESIDUAL ? h : x) + c, (int)(n - c)); };
    auto squares = [&](const V8<T> &v, float by, float sum) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float f = (float)v[i] * by;
            sum = __builtin_fmaf(f, f, sum);
        }
        return sum;
    };

    V8<T> kept[KEPT];
#pragma unroll
    for (int s = 0; s < KEPT; ++s) {
        const uint32_t c = (s * THREADS + lane) * kCols;
        kept[s] = c < n ? read(c) : V8<T>{};
    }
    float sum[1] = {0.f};
#pragma unroll
    for (int s = 0; s < KEPT; ++s) {
        const uint32_t c = (s * THREADS + lane) * kCols;
        if (RESIDUAL && c < n) store8(h + c, kept[s], (int)(n - c));
        sum[0] = squares(kept[s], 1.f, sum[0]);
    }
    for (uint32_t c = kFirst + lane * kCols; c < n; c += THREADS * kCols) {
        const V8<T> v = read(c);
        if (RESIDUAL) store8(h + c, v, (int)(n - c));
        sum[0] = squares(v, 1.f, sum[0]);
    }
    row_sums<THREADS>(sum, sums);
    float by = 1.f;
    if (!(sum[0] < __builtin_inff())) {  // the same for all of the row's lanes
        by = kSmaller;
        sum[0] = 0.f;
#pragma unroll
        for (int s = 0; s < KEPT; ++s) sum[0] = squares(kept[s], by, sum[0]);
        for (uint32_t c = kFirst + lane * kCols; c < n; c += THREADS * kCols)
            sum[0] = squares(again(c), by, sum[0]);
        row_sums<THREADS>(sum, sums);
    }
    float inverse = by / sqrtf(sum[0] / (float)n + g.eps * by * by);

    auto normed = [&](const V8<T> &v, uint32_t c, float (&out)[8]) {
        const V8<T> w = load8(weight + c, (int)(n - c));
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = (float)v[i] * inverse * (float)w[i];
    };
    if constexpr (!INT8) {
        T *y = (T *)g.y + (int64_t)r * g.ldy;
        auto put = [&](const V8<T> &v, uint32_t c) {
            float f[8];
            normed(v, c, f);
            V8<T> o;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = (T)f[i];
            store8(y + c, o, (int)(n - c));
        };
#pragma unroll
        for (int s = 0; s < KEPT; ++s) {
            const uint32_t c = (s * THREADS + lane) * kCols;
            if (c < n) put(kept[s], c);
        }
        for (uint32_t c = kFirst + lane * kCols; c < n; c += THREADS * kCols) put(again(c), c);
    } else {
        int8_t *y = (int8_t *)g.y + (int64_t)r * g.ldy;
        // As whole numbers, magnitudes order like floats, infinity and then NaN above all.
        uint32_t top = 0;
        auto widen = [&](const float (&f)[8]) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const uint32_t m = __float_as_uint(f[i]) & 0x7fffffffu;
                top = top > m ? top : m;
            }
        };
#pragma unroll
        for (int s = 0; s < KEPT; ++s) {
            const uint32_t c = (s * THREADS + lane) * kCols;
            float o[8];
            if (c < n) {
                normed(kept[s], c, o);
                widen(o);
            }
        }
        for (uint32_t c = kFirst + lane * kCols; c < n; c += THREADS * kCols) {
            float o[8];
            normed(again(c), c, o);
            widen(o);
        }
        top = row_max<THREADS>(top, (uint32_t *)sums);
        // y is computed again rather than kept: twice the registers of h, and the compiler spilled
        asm volatile("" : "+v"(inverse));
        const float scale = __uint_as_float(top) / 127.0f;
        if (lane == 0) g.sx[r] = scale;
        const bool finite = top < 0x7f800000u && scale > 0.f;
        const Steps steps(scale);
        auto put = [&](const float (&o)[8], uint32_t c) {
            i8x8 q = {};
            if (finite) q = steps(o);
            store8(y + c, q, (int)(n - c));
        };
#pragma unroll
        for (int s = 0; s < KEPT; ++s) {
            const uint32_t c = (s * THREADS + lane) * kCols;
            float o[8];
            if (c < n) {
                normed(kept[s], c, o);
                put(o, c);
            }
        }
        for (uint32_t c = kFirst + lane * kCols; c < n; c += THREADS * kCols) {
            float o[8];
            normed(again(c), c, o);
            put(o, c);
        }
    }
}

struct NormBackwardArgs {
    void *dx;
    float *partial;  // [groups][n]: each group of rows' sum of dy u
    float *inverse;  // [rows], for rows too wide for registers
    const void *dy, *h, *dh, *weight;
    int64_t lddx, lddy, ldh, lddh;  // elements
    uint32_t rows, n, groups;
    float eps;
};

// THREADS lanes a row and every groups-th row to one group of lanes, which holds KEPT pieces of 16
// bytes of h, dy and the weight and its sums for the weight's gradient in registers. Both sums of a
// row (h^2 and dn h) are taken together, so that a row is read once.
template <class T, int THREADS, int KEPT, bool DH>
__global__ void __launch_bounds__(THREADS > kBlock ? THREADS : kBlock)
    k_norm_backward(NormBackwardArgs g)
{
    constexpr uint32_t kRows = THREADS > kBlock ? 1 : kBlock / THREADS;
    __shared__ float lds[2 * THREADS / 64];
    const uint32_t group = blockIdx.x * kRows + (kRows > 1 ? threadIdx.x / THREADS : 0);
    const uint32_t lane = kRows > 1 ? threadIdx.x % THREADS : threadIdx.x;
    if (group >= g.groups) return;
    const uint32_t n = g.n;
    V8<T> weight[KEPT];
    float dweight[KEPT][8] = {};
#pragma unroll
    for (int s = 0; s < KEPT; ++s) {
        const uint32_t c = (s * THREADS + lane) * kCols;
        weight[s] = c < n ? load8((const T *)g.weight + c, (int)(n - c)) : V8<T>{};
    }
    for (uint32_t r = group; r < g.rows; r += g.groups) {
        const T *from_h = (const T *)g.h + (int64_t)r * g.ldh;
        const T *from_dy = (const T *)g.dy + (int64_t)r * g.lddy;
        V8<T> h[KEPT], dy[KEPT], dh[KEPT];
#pragma unroll
        for (int s = 0; s < KEPT; ++s) {
            const uint32_t c = (s * THREADS + lane) * kCols;
            const int left = (int)(n - c);
            h[s] = c < n ? load8(from_h + c, left) : V8<T>{};
            dy[s] = c < n ? load8(from_dy + c, left) : V8<T>{};
            if constexpr (DH)
                dh[s] = c < n ? load8((const T *)g.dh + (int64_t)r * g.lddh + c, left) : V8<T>{};
        }
        float sum[2], by = 1.f;
        auto both = [&] {
            sum[0] = sum[1] = 0.f;
#pragma unroll
            for (int s = 0; s < KEPT; ++s)
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float f = (float)h[s][i] * by;
                    sum[0] = __builtin_fmaf(f, f, sum[0]);
                    sum[1] = __builtin_fmaf((float)dy[s][i] * (float)weight[s][i], f, sum[1]);
                }
            row_sums<THREADS>(sum, lds);
        };
        both();
        if (!(sum[0] < __builtin_inff())) {
            by = kSmaller;
            both();
        }
        const float unit = 1.f / sqrtf(sum[0] / (float)n + g.eps * by * by);
        const float inverse = unit * by, along = sum[1] * unit / (float)n;
        T *dx = (T *)g.dx + (int64_t)r * g.lddx;
#pragma unroll
        for (int s = 0; s < KEPT; ++s) {
            const uint32_t c = (s * THREADS + lane) * kCols;
            V8<T> o;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float u = (float)h[s][i] * inverse, d = (float)dy[s][i];
                dweight[s][i] = __builtin_fmaf(d, u, dweight[s][i]);
                float v = inverse * __builtin_fmaf(-u, along, d * (float)weight[s][i]);
                if constexpr (DH) v += (float)dh[s][i];
                o[i] = (T)v;
            }
            if (c < n) store8(dx + c, o, (int)(n - c));
        }
    }
    float *to = g.partial + (uint64_t)group * n;
#pragma unroll
    for (int s = 0; s < KEPT; ++s) {
        const uint32_t c = (s * THREADS + lane) * kCols;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < n) to[c + i] = dweight[s][i];
    }
}

// Rows too wide for registers: dx, and each row's r for the weight's gradient. A row is read twice.
template <class T>
__global__ void __launch_bounds__(1024) k_norm_backward_wide(NormBackwardArgs g)
{
    __shared__ float lds[2 * 1024 / 64];
    const uint32_t r = blockIdx.x, n = g.n;
    const T *h = (const T *)g.h + (int64_t)r * g.ldh;
    const T *dy = (const T *)g.dy + (int64_t)r * g.lddy;
    const T *dh = g.dh ? (const T *)g.dh + (int64_t)r * g.lddh : nullptr;
    const T *weight = (const T *)g.weight;
    float sum[2], by = 1.f;
    auto both = [&] {
        sum[0] = sum[1] = 0.f;
        for (uint32_t c = threadIdx.x * kCols; c < n; c += 1024 * kCols) {
            const int left = (int)(n - c);
            const V8<T> a = load8(h + c, left), d = load8(dy + c, left);
            const V8<T> w = load8(weight + c, left);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float f = (float)a[i] * by;
                sum[0] = __builtin_fmaf(f, f, sum[0]);
                sum[1] = __builtin_fmaf((float)d[i] * (float)w[i], f, sum[1]);
            }
        }
        row_sums<1024>(sum, lds);
    };
    both();
    if (!(sum[0] < __builtin_inff())) {
        by = kSmaller;
        both();
    }
    const float unit = 1.f / sqrtf(sum[0] / (float)n + g.eps * by * by);
    const float inverse = unit * by, along = sum[1] * unit / (float)n;
    if (threadIdx.x == 0) g.inverse[r] = inverse;
    T *dx = (T *)g.dx + (int64_t)r * g.lddx;
    for (uint32_t c = threadIdx.x * kCols; c < n; c += 1024 * kCols) {
        const int left = (int)(n - c);
        const V8<T> a = load8(h + c, left), d = load8(dy + c, left), w = load8(weight + c, left);
        const V8<T> e = dh ? load8(dh + c, left) : V8<T>{};
        V8<T> o;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float v = inverse * __builtin_fmaf(-((float)a[i] * inverse), along,
                                               (float)d[i] * (float)w[i]);
            if (dh) v += (float)e[i];
            o[i] = (T)v;
        }
        store8(dx + c, o, left);
    }
}

// Their weight's gradient: a wave takes 512 columns of every groups-th row.
template <class T>
__global__ void __launch_bounds__(64) k_norm_dweight_wide(NormBackwardArgs g, uint32_t parts)
{
    const uint32_t group = blockIdx.x / parts, c = (blockIdx.x % parts * 64 + threadIdx.x) * kCols;
    if (c >= g.n) return;
    const int left = (int)(g.n - c);
    float sum[8] = {};
    for (uint32_t r = group; r < g.rows; r += g.groups) {
        const V8<T> h = load8((const T *)g.h + (int64_t)r * g.ldh + c, left);
        const V8<T> dy = load8((const T *)g.dy + (int64_t)r * g.lddy + c, left);
        const float inverse = g.inverse[r];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            sum[i] = __builtin_fmaf((float)dy[i], (float)h[i] * inverse, sum[i]);
    }
    float *to = g.partial + (uint64_t)group * g.n + c;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) to[i] = sum[i];
}

// The groups' sums added up in a fixed order: 32 columns a workgroup, 32 lanes a column.
constexpr uint32_t kSumColumns = 32;
template <class T>
__global__ void __launch_bounds__(1024)
    k_norm_dweight(T *__restrict__ dweight, const float *__restrict__ partial, uint32_t groups,
                   uint32_t n)
{
    __shared__ float sums[32][kSumColumns + 1];
    const uint32_t col = threadIdx.x % kSumColumns, lane = threadIdx.x / kSumColumns;
    const uint32_t c = blockIdx.x * kSumColumns + col;
    float s = 0.f;
    if (c < n)
#pragma unroll 8
        for (uint32_t i = lane; i < groups; i += 32) s += partial[(uint64_t)i * n + c];
    sums[lane][col] = s;
    __syncthreads();
    for (uint32_t half = 16; half; half /= 2) {
        if (lane < half) sums[lane][col] += sums[lane + half][col];
        __syncthreads();
    }
    if (lane == 0 && c < n) dweight[c] = (T)sums[0][col];
}

// Lanes and pieces for a row: a wave where its lanes hold it with four pieces each, then a workgroup
// of 256, then of 1024.
template <class T, bool RESIDUAL, bool INT8>
hist_status_t launch_norm(NormArgs g, hipStream_t stream)
{
    constexpr uint32_t kOut = INT8 ? 1 : sizeof(T);
    const uint32_t rows = g.rows, each = g.n <= 2048 ? 4 : 1;
    const uint64_t most = most_of(each, g.n <= 8192 ? kBlock : 1024);
    hist_status_t st = HIST_OK;
    for (uint64_t r = 0; r < rows && st == HIST_OK; r += most) {
        NormArgs a = g;
        a.rows = (uint32_t)(rows - r < most ? rows - r : most);
        a.y = (char *)g.y + (int64_t)r * g.ldy * kOut;
        a.h = (T *)g.h + (RESIDUAL ? (int64_t)r * g.ldh : 0);
        a.sx = INT8 ? g.sx + r : nullptr;
        a.x = (const T *)g.x + (int64_t)r * g.ldx;
        a.residual = (const T *)g.residual + (RESIDUAL ? (int64_t)r * g.ldr : 0);
        const uint64_t blocks = (a.rows + each - 1) / each;
        if (g.n <= 1024)
            st = launch(k_norm<T, 64, 2, RESIDUAL, INT8>, blocks, kBlock, 0, stream, a);
        else if (g.n <= 2048)
            st = launch(k_norm<T, 64, 4, RESIDUAL, INT8>, blocks, kBlock, 0, stream, a);
        else if (g.n <= 4096)
            st = launch(k_norm<T, 256, 2, RESIDUAL, INT8>, blocks, kBlock, 0, stream, a);
        else if (g.n <= 8192)
            st = launch(k_norm<T, 256, 4, RESIDUAL, INT8>, blocks, kBlock, 0, stream, a);
        else
            st = launch(k_norm<T, 1024, 4, RESIDUAL, INT8>, blocks, 1024, 0, stream, a);
    }
    return st;
}

template <class T>
hist_status_t launch_norm_any(const NormArgs &g, bool int8, hipStream_t stream)
{
    if (int8)
        return g.residual ? launch_norm<T, true, true>(g, stream)
                          : launch_norm<T, false, true>(g, stream);
    return g.residual ? launch_norm<T, true, false>(g, stream)
                      : launch_norm<T, false, false>(g, stream);
}

// The widest rows whose backward pass keeps them in registers.
constexpr uint32_t kWidest = 1024 * 2 * kCols;

// Lanes of a row in the backward pass.
inline uint32_t backward_threads(uint32_t n)
{
    return n <= 1024 ? 64 : n <= 4096 ? 256 : n <= 8192 ? 512 : 1024;
}

// Groups of rows, each with its own sums for the weight's gradient, which are written and read again. us
// with 8, 12 and 16 waves a CU: 8191 x 2048 35.9, 32.7, 34.9; 16384 x 4096 106, 111, 115; 16384 x 1024 35.8,
// 40.8, 44.5; 4096 x 8192 62.2, 61.3, 64.5; 2048 x 16384 83.8, 71.1, 68.7.
inline uint32_t backward_groups(uint64_t rows, uint32_t n)
{
    const uint64_t most = n > kWidest ? 64
                          : n <= 1024 ? 2048
                          : n <= 2048 ? 768
                          : n <= 4096 ? 512
                          : n <= 8192 ? 384
                                      : 256;
    return (uint32_t)(rows < most ? rows : most);
}

inline uint64_t backward_bytes(uint64_t rows, uint32_t n)
{
    return 4 * ((uint64_t)backward_groups(rows, n) * n + (n > kWidest ? rows : 0));
}

template <class T, bool DH>
hist_status_t launch_norm_rows(const NormBackwardArgs &g, hipStream_t stream)
{
    const uint32_t threads = backward_threads(g.n);
    const uint64_t blocks = threads == 64 ? (g.groups + 3) / 4 : g.groups;
    if (g.n <= 512)
        return launch(k_norm_backward<T, 64, 1, DH>, blocks, kBlock, 0, stream, g);
    if (g.n <= 1024)
        return launch(k_norm_backward<T, 64, 2, DH>, blocks, kBlock, 0, stream, g);
    if (g.n <= 2048)
        return launch(k_norm_backward<T, 256, 1, DH>, blocks, kBlock, 0, stream, g);
    if (g.n <= 4096)
        return launch(k_norm_backward<T, 256, 2, DH>, blocks, kBlock, 0, stream, g);
    if (g.n <= 8192)
        return launch(k_norm_backward<T, 512, 2, DH>, blocks, 512, 0, stream, g);
    return launch(k_norm_backward<T, 1024, 2, DH>, blocks, 1024, 0, stream, g);
}

template <class T>
hist_status_t launch_norm_backward(const NormBackwardArgs &g, void *dweight, hipStream_t stream)
{
    hist_status_t st = HIST_OK;
    if (g.n > kWidest && g.rows) {
        const uint64_t most = most_of(1, 1024);
        for (uint64_t r = 0; r < g.rows && st == HIST_OK; r += most) {
            NormBackwardArgs a = g;
            a.dx = (T *)g.dx + (int64_t)r * g.lddx;
            a.dy = (const T *)g.dy + (int64_t)r * g.lddy;
            a.h = (const T *)g.h + (int64_t)r * g.ldh;
            a.dh = g.dh ? (const T *)g.dh + (int64_t)r * g.lddh : nullptr;
            a.inverse = g.inverse + r;
            st = launch(k_norm_backward_wide<T>, g.rows - r < most ? g.rows - r : most, 1024, 0,
                        stream, a);
        }
        const uint32_t parts = (g.n + 64 * kCols - 1) / (64 * kCols);
        if (st == HIST_OK)
            st = launch(k_norm_dweight_wide<T>, (uint64_t)g.groups * parts, 64, 0, stream, g,
                        parts);
    } else if (g.rows) {  // (without rows the weight's gradient is zero)
        st = g.dh ? launch_norm_rows<T, true>(g, stream) : launch_norm_rows<T, false>(g, stream);
    }
    if (st != HIST_OK) return st;
    return launch(k_norm_dweight<T>, (g.n + kSumColumns - 1) / kSumColumns, 1024, 0, stream, (T *)dweight,
                  (const float *)g.partial, g.groups, g.n);
}

// Below this eps squares that underflow could count beside it.
constexpr float kLeastEps = 1e-30f;

inline hist_status_t check_norm(uint64_t rows, uint32_t n, float eps, int32_t dtype)
{
    if (!dtype_ok(dtype) || n == 0 || !(eps >= kLeastEps && eps < __builtin_inff()))
        return HIST_ERR_INVALID_ARG;
    if (rows > EXPERTS_MAX_ROWS || n > EXPERTS_MAX_WIDTH) return HIST_ERR_UNSUPPORTED;
    return HIST_OK;
}

inline bool bad_rows(const void *p, int64_t ld, uint32_t n, bool used, uintptr_t align)
{
    return used && (!p || ld < (int64_t)n || misaligned(p, align));
}

}  // namespace pca_experts

using namespace pca_experts;

static hist_status_t norm(void *y, int64_t ldy, float *sx, void *h, int64_t ldh, const void *x,
                          int64_t ldx, const void *residual, int64_t ldr, const void *weight,
                          uint64_t rows, uint32_t n, float eps, int32_t dtype, bool int8,
                          hipStream_t stream)
{
    hist_status_t st = check_norm(rows, n, eps, dtype);
    if (st != HIST_OK) return st;
    if (bad_rows(y, ldy, n, rows, int8 ? 1 : 2) || bad_rows(x, ldx, n, rows, 2) ||
        bad_rows(residual, ldr, n, rows && residual, 2) || bad_rows(h, ldh, n, rows && residual, 2) ||
        (rows && !weight) || misaligned(weight, 2) || (int8 && ((rows && !sx) || misaligned(sx, 4))))
        return HIST_ERR_INVALID_ARG;
    st = device_status();
    if (st != HIST_OK || rows == 0) return st;
    const NormArgs g = {y, h, sx, x, residual, weight, ldy, ldh, ldx, ldr, (uint32_t)rows, n, eps};
    return dtype == EXPERTS_BF16 ? launch_norm_any<__bf16>(g, int8, stream)
                                 : launch_norm_any<_Float16>(g, int8, stream);
}

extern "C" hist_status_t experts_rms_norm(void *y, int64_t ldy, void *h, int64_t ldh,
                                          const void *x, int64_t ldx, const void *residual,
                                          int64_t ldr, const void *weight, uint64_t rows,
                                          uint32_t n, float eps, int32_t dtype,
                                          hipStream_t stream)
{
    return norm(y, ldy, nullptr, h, ldh, x, ldx, residual, ldr, weight, rows, n, eps, dtype, false,
                stream);
}

extern "C" hist_status_t experts_rms_norm_int8(int8_t *xq, int64_t ldq, float *sx, void *h,
                                               int64_t ldh, const void *x, int64_t ldx,
                                               const void *residual, int64_t ldr,
                                               const void *weight, uint64_t rows, uint32_t n,
                                               float eps, int32_t dtype, hipStream_t stream)
{
    return norm(xq, ldq, sx, h, ldh, x, ldx, residual, ldr, weight, rows, n, eps, dtype, true,
                stream);
}

extern "C" hist_status_t experts_rms_norm_backward_workspace_size(uint64_t rows, uint32_t n,
                                                                  uint64_t *bytes)
{
    if (!bytes || n == 0) return HIST_ERR_INVALID_ARG;
    if (rows > EXPERTS_MAX_ROWS || n > EXPERTS_MAX_WIDTH) return HIST_ERR_UNSUPPORTED;
    *bytes = backward_bytes(rows, n);
    return HIST_OK;
}

extern "C" hist_status_t experts_rms_norm_backward(void *dx, int64_t lddx, void *dweight,
                                                   const void *dy, int64_t lddy, const void *h,
                                                   int64_t ldh, const void *dh, int64_t lddh,
                                                   const void *weight, uint64_t rows, uint32_t n,
                                                   float eps, int32_t dtype, void *workspace,
                                                   uint64_t workspace_bytes, hipStream_t stream)
{
    hist_status_t st = check_norm(rows, n, eps, dtype);
    if (st != HIST_OK) return st;
    if (bad_rows(dx, lddx, n, rows, 2) || bad_rows(dy, lddy, n, rows, 2) ||
        bad_rows(h, ldh, n, rows, 2) || bad_rows(dh, lddh, n, rows && dh, 2) || !dweight ||
        misaligned(dweight, 2) || (rows && !weight) || misaligned(weight, 2))
        return HIST_ERR_INVALID_ARG;
    if (rows && (!workspace || misaligned(workspace, 16) ||
                 workspace_bytes < backward_bytes(rows, n)))
        return HIST_ERR_WORKSPACE;
    st = device_status();
    if (st != HIST_OK) return st;
    const uint32_t groups = backward_groups(rows, n);
    const NormBackwardArgs g = {dx, (float *)workspace, (float *)workspace + (uint64_t)groups * n,
                                dy, h, dh, weight, lddx, lddy, ldh, lddh, (uint32_t)rows, n, groups,
                                eps};
    return (dtype == EXPERTS_BF16 ? launch_norm_backward<__bf16>
                                  : launch_norm_backward<_Float16>)(g, dweight, stream);
}
