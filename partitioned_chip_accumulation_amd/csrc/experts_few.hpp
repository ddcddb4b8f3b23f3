// experts_few.hpp -- a whole expert layer for a few tokens: the kernels of experts_few_tokens and how
// they are launched. Part of libpca_hist.so.
//
//   h[t, e] = act(x[t] up[e]^T),  out[t] = sum over t's experts e of weight[t, e] h[t, e] down[e]^T
//
// Bound by reading the weights of the experts that have a token, once each. Two kernels: the first
// takes an expert's 16 FN columns of h a workgroup, the second 16 FN columns of the result, with the
// products of all experts added up in registers. Both find the experts from the ids by themselves, so
// nothing is sorted, counted or copied before, and the host needs to know nothing of the routing.
//
// The fragments of the matrix instructions come from memory to registers: a lane's 16 bytes of a
// weight's row, 8, 16 or 32 values, are widened to the tokens' type there (exact: 8-bit whole numbers
// and 4-bit values times a power of two have 8 bits at most), so that what is read is what the weights
// take.
#pragma once

#include "experts_tile.hpp"

namespace pca_experts {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

constexpr uint32_t kMostFew = EXPERTS_MAX_FEW;  // tokens
constexpr uint32_t kTurn = 64;                  // bytes of a row that a wave takes in one step

struct FewWeight {
    const char *data;
    const char *scales;  // float [experts][rows], or powers of two
    int64_t ld, stride, ld_scales, scales_stride;  // bytes
};

struct FewArgs {
    char *out;
    const char *x;
    char *h;            // [pairs][ldh]: row t * top_k + j, j the first of t's choices of its expert
    uint32_t *arrived;  // [tiles of the result]
    uint32_t *partial;
    FewWeight up, down;
    const void *ids;
    const float *by;
    int64_t ldo, ldx, ldh;  // bytes
    uint32_t ids64, gated, tokens, top_k, experts, width, hidden, n;
    uint32_t tiles, splits;
};

// How weights of type W go with tokens of type T: C fragments of a lane's 16 bytes.
template <class T, class W> struct Widen;
template <class T> struct Widen<T, T> {
    static constexpr int C = 1;
    typedef typename Vec8<T>::type Frag;
    static __device__ __forceinline__ Frag frag(u32x4 v, int, uint32_t)
    {
        return __builtin_bit_cast(Frag, v);
    }
    static __device__ __forceinline__ void add(Frag w, u32x4 a, f32x4 &acc)
    {
        acc = Mma<T>::run(w, __builtin_bit_cast(Frag, a), acc);
    }
};
template <class T> struct Widen<T, int8_t> {
    static constexpr int C = 2;
    typedef typename Vec8<T>::type Frag;
    static __device__ __forceinline__ Frag frag(u32x4 v, int c, uint32_t)
    {
        Frag f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = (T)(float)(int8_t)(v[c * 2 + i / 4] >> i % 4 * 8);
        return f;
    }
    static __device__ __forceinline__ void add(Frag w, u32x4 a, f32x4 &acc)
    {
        acc = Mma<T>::run(w, __builtin_bit_cast(Frag, a), acc);
    }
};
// A block's values as bfloat16, whose exponents reach as far as the powers of two.
template <class T> struct Widen<T, Mx4> {
    static constexpr int C = 4;
    typedef bf16x8 Frag;
    static __device__ __forceinline__ Frag frag(u32x4 v, int c, uint32_t power)
    {
        // (2^-127 is no normal number; 255 makes every value a NaN)
        const float scale = __uint_as_float(power ? power << 23 : 1u << 22);
        Frag f;
        const bf16x2 v0 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[c], scale, 0);
        const bf16x2 v1 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[c], scale, 1);
        const bf16x2 v2 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[c], scale, 2);
        const bf16x2 v3 = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(v[c], scale, 3);
        f = Frag{v0[0], v0[1], v1[0], v1[1], v2[0], v2[1], v3[0], v3[1]};
        return f;
    }
    // A float16 value is the sum of two bfloat16 ones (11 bits, of 8 and 3), so two products have it
    // whole; float16 weights could not hold every power of two.
    static __device__ __forceinline__ void add(Frag w, u32x4 a, f32x4 &acc)
    {
        if constexpr (std::is_same<T, __bf16>::value) {
            acc = Mma<__bf16>::run(w, __builtin_bit_cast(bf16x8, a), acc);
        } else {
            const f16x8 v = __builtin_bit_cast(f16x8, a);
            bf16x8 high, low;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                high[i] = (__bf16)(float)v[i];
                const float rest = (float)v[i] - (float)high[i];
                low[i] = (__bf16)(rest == rest ? rest : 0.f);  // (of an infinity nothing is left)
            }
            acc = Mma<__bf16>::run(w, high, acc);
            acc = Mma<__bf16>::run(w, low, acc);
        }
    }
};

// Bytes of a row of k values.
template <class W>
__device__ __host__ __forceinline__ uint32_t row_bytes(uint32_t k)
{
    if constexpr (std::is_same<W, Mx4>::value) return (k + 31) / 32 * 16;
    else return k * sizeof(W);
}

// ---------------------------------------------------------------------------
// The routing in LDS: the ids, and the experts that have a token in the order of their numbers.
struct Routes {
    uint32_t mask[EXPERTS_MAX_EXPERTS / 32];
    uint32_t count;
    int16_t list[EXPERTS_MAX_EXPERTS];
};
extern __shared__ __align__(16) char few_lds[];  // int16_t ids[pairs], float by[pairs]

__device__ __forceinline__ int16_t *lds_ids() { return (int16_t *)few_lds; }
__device__ __forceinline__ float *lds_by(uint32_t pairs)
{
    return (float *)(few_lds + (pairs * 2 + 15) / 16 * 16);
}

template <bool BY>
__device__ __forceinline__ void find_routes(const FewArgs &g, Routes &routes)
{
    const uint32_t pairs = g.tokens * g.top_k;
    if (threadIdx.x < EXPERTS_MAX_EXPERTS / 32) routes.mask[threadIdx.x] = 0;
    __syncthreads();
    for (uint32_t i = threadIdx.x; i < pairs; i += blockDim.x) {
        const int64_t id = g.ids64 ? ((const int64_t *)g.ids)[i] : ((const int32_t *)g.ids)[i];
        const bool valid = (uint64_t)id < g.experts;
        lds_ids()[i] = valid ? (int16_t)id : -1;
        if constexpr (BY) lds_by(pairs)[i] = g.by[i];
        if (valid)
            __hip_atomic_fetch_or(&routes.mask[id / 32], 1u << id % 32, __ATOMIC_RELAXED,
                                  __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
    if (threadIdx.x < 64) {
        uint32_t bits = threadIdx.x < EXPERTS_MAX_EXPERTS / 32 ? routes.mask[threadIdx.x] : 0;
        const uint32_t mine = __builtin_popcount(bits), upto = wave_inclusive_scan(mine);
        uint32_t at = upto - mine;
        for (; bits; bits &= bits - 1)
            routes.list[at++] = (int16_t)(threadIdx.x * 32 + __builtin_ctz(bits));
        if (threadIdx.x == 63) routes.count = upto;
    }
    __syncthreads();
}

// ---------------------------------------------------------------------------
// What one step of a wave multiplies: 64 bytes of each of 16 FB rows of a weight, and what goes with
// them of 16 RM rows of tokens. At a row's ragged end the 16 bytes that end with it are loaded, and
// shifted only when they are multiplied, so that no load is waited for before its turn.
template <class T, class W, int RM, int FB>
struct Piece {
    typedef Widen<T, W> By;
    static constexpr int C = By::C;
    static constexpr uint32_t kValues = kTurn / 16 * C * 8;  // of a row
    static constexpr bool kPowers = std::is_same<W, Mx4>::value;
    u32x4 b[FB], a[RM][C];
    uint32_t power[kPowers ? FB : 1];
    uint32_t step;

    static __device__ __forceinline__ u32x4 one(const char *p, int left, uint32_t row)
    {
        if (row < 16) return load16<uint8_t>(p, left, false);
        return load_any<u32x4>(p + (left < 16 ? left : 16) - 16);
    }
    static __device__ __forceinline__ int left_b(uint32_t step, uint32_t k)
    {
        return (int)row_bytes<W>(k) - (int)(step * kTurn + threadIdx.x % 64 / 16 * 16);
    }
    static __device__ __forceinline__ int left_a(uint32_t step, uint32_t k, int c)
    {
        return ((int)k - (int)(step * kValues + threadIdx.x % 64 / 16 * C * 8 + c * 8)) * 2;
    }

    // from_a, from_b: this lane's rows, at the 8 C values and the 16 bytes that are its own in the
    // first step; powers: its row's first one. k: values of a row.
    __device__ __forceinline__ void fetch(const char *const (&from_a)[RM],
                                          const char *const (&from_b)[FB],
                                          const char *const (&powers)[FB], uint32_t which, uint32_t k)
    {
        step = which;
        const int in_b = left_b(step, k);
#pragma unroll
        for (int j = 0; j < FB; ++j) {
            b[j] = one(from_b[j] + step * kTurn, in_b, row_bytes<W>(k));
            if constexpr (kPowers) {  // (past the row's end: that of the last block, of zeros)
                const uint32_t block = step * 4 + threadIdx.x % 64 / 16;
                power[j] = (uint8_t)powers[j][block * 16 < row_bytes<W>(k) ? block : 0];
            }
        }
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int in_a = left_a(step, k, c);
#pragma unroll
            for (int i = 0; i < RM; ++i)
                a[i][c] = one(from_a[i] + step * kValues * 2 + c * 16, in_a, k * 2);
        }
    }

    __device__ __forceinline__ void multiply(f32x4 (&acc)[RM][FB], uint32_t k)
    {
        if (step * kTurn + kTurn > row_bytes<W>(k) || step * kValues + kValues > k) {
            const int in_b = left_b(step, k);
#pragma unroll
            for (int j = 0; j < FB; ++j) {
                if (row_bytes<W>(k) >= 16) b[j] = drop16(b[j], in_b);
                if constexpr (kPowers) power[j] = in_b > 0 ? power[j] : 127;
            }
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int in_a = left_a(step, k, c);
#pragma unroll
                for (int i = 0; i < RM; ++i)
                    if (k * 2 >= 16) a[i][c] = drop16(a[i][c], in_a);
            }
        }
#pragma unroll
        for (int j = 0; j < FB; ++j)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const auto w = By::frag(b[j], c, power[kPowers ? j : 0]);
#pragma unroll
                for (int i = 0; i < RM; ++i) By::add(w, a[i][c], acc[i][j]);
            }
    }
};

// `mine` pieces (one or more), DEEP of them on their way while the ones before are multiplied. fetch
// stays at the last piece when it is asked for more: loads that come from the cache, in place of
// branches around loads, at which the compiler would wait for all of them.
template <int DEEP, class P, class F, class M>
__device__ __forceinline__ void pipeline(uint32_t mine, P (&p)[DEEP], F fetch, M multiply)
{
#pragma unroll
    for (int d = 0; d < DEEP; ++d) fetch(p[d]);
    uint32_t left = mine;
    for (; left > DEEP; left -= DEEP)
#pragma unroll
        for (int d = 0; d < DEEP; ++d) {
            multiply(p[d]);
            fetch(p[d]);
        }
#pragma unroll
    for (int d = 0; d < DEEP; ++d)
        if ((uint32_t)d < left) multiply(p[d]);
}

// Pieces with numbers first, first + turn, ... below count.
__device__ __forceinline__ uint32_t pieces(uint32_t count, uint32_t first, uint32_t turn)
{
    return count > first ? (count - first + turn - 1) / turn : 0;
}

// ---------------------------------------------------------------------------
// Columns of h for one expert, 16 FN of them with a gate (FN fragments of its rows, then FN of the
// others) and 32 FN without, its tokens 16 RM at a time; the four waves divide the reduction.
template <class T, class W, int RM, int FN, int DEEP>
__device__ __forceinline__ void up_rows(const FewArgs &g, uint32_t e, uint32_t n0,
                                        const uint16_t *rows, uint32_t count, f32x4 *sums)
{
    constexpr int FB = 2 * FN;
    typedef Piece<T, W, RM, FB> P;
    const uint32_t lane = threadIdx.x % 64, at = lane / 16;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const char *a[RM], *b[FB], *powers[FB];
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const uint32_t r = i * 16 + lane % 16;
        const uint32_t token = rows[r < count ? r : count - 1] / g.top_k;
        a[i] = g.x + (int64_t)token * g.ldx + at * P::C * 16;
    }
#pragma unroll
    for (int j = 0; j < FB; ++j) {
        uint32_t c = n0 + (g.gated ? j % FN : j) * 16 + lane % 16;
        c = (c < g.hidden ? c : g.hidden - 1) + (g.gated ? j / FN * g.hidden : 0);
        b[j] = g.up.data + (int64_t)e * g.up.stride + (int64_t)c * g.up.ld + at * 16;
        powers[j] = nullptr;
        if constexpr (P::kPowers)
            powers[j] = g.up.scales + (int64_t)e * g.up.scales_stride + (int64_t)c * g.up.ld_scales;
    }
    f32x4 acc[RM][FB] = {};
    const uint32_t steps = (row_bytes<W>(g.width) + kTurn - 1) / kTurn;
    const uint32_t mine = pieces(steps, wave, 4);
    if (mine) {
        P p[DEEP];
        uint32_t next = wave;
        const uint32_t end = wave + (mine - 1) * 4;
        pipeline(mine, p,
                 [&](P &q) {
                     q.fetch(a, b, powers, next, g.width);
                     next = next < end ? next + 4 : end;
                 },
                 [&](P &q) { q.multiply(acc, g.width); });
    }
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) sums[(wave * RM * FB + i * FB + j) * 64 + lane] = acc[i][j];
    __syncthreads();
    const uint32_t columns = g.gated ? FN : FB;  // fragments of results
    for (uint32_t f = wave; f < RM * columns; f += 4) {
        const uint32_t i = f / columns, j = f % columns;
        const uint32_t r = i * 16 + lane % 16, c = n0 + j * 16 + at * 4;
        if (r >= count || c >= g.hidden) continue;
        auto sum = [&](uint32_t j, uint32_t row) {
            f32x4 v = sums[(i * FB + j) * 64 + lane];
#pragma unroll
            for (int w = 1; w < 4; ++w) v += sums[(w * RM * FB + i * FB + j) * 64 + lane];
            if constexpr (std::is_same<W, int8_t>::value) {
                const float *scales =
                    (const float *)(g.up.scales + (int64_t)e * g.up.scales_stride) + row;
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] *= c + q < g.hidden ? scales[q] : 0.f;
            }
            return v;
        };
        f32x4 v = sum(j, c);
#pragma unroll
        for (int q = 0; q < 4; ++q) v[q] = v[q] / (1.f + expf(-v[q]));
        if (g.gated) v *= sum(FN + j, g.hidden + c);
        // h is rounded to the tokens' type here, as the rows between two separate products are.
        T *to = (T *)(g.h + rows[r] * g.ldh) + c;
        typedef T T4 __attribute__((ext_vector_type(4)));
        const T4 o = {(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
        if (c + 4 <= g.hidden) {
            store_any(to, o);
        } else {
#pragma unroll
            for (int q = 0; q < 3; ++q)
                if (c + q < g.hidden) to[q] = o[q];
        }
    }
}

// RM: the most rows of 16 that the tokens fill. Most experts have no more than 16 of 64 tokens, so
// larger tiles have the smallest one beside theirs.
template <class T, class W, int RM, int FN, int DEEP>
__global__ void __launch_bounds__(256) k_few_up(FewArgs g)
{
    __shared__ Routes routes;
    __shared__ uint16_t rows[kMostFew];
    __shared__ __align__(16) f32x4 sums[4 * RM * 2 * FN * 64];
    if (blockIdx.x == 0)
        for (uint32_t i = threadIdx.x; i < g.tiles; i += 256) g.arrived[i] = 0;
    find_routes<false>(g, routes);
    const uint32_t each = g.gated ? 16 * FN : 32 * FN;
    const uint32_t tiles = (g.hidden + each - 1) / each;
    const uint32_t slot = blockIdx.x / tiles, n0 = blockIdx.x % tiles * each;
    if (slot >= __builtin_amdgcn_readfirstlane(routes.count)) return;
    const uint32_t e = __builtin_amdgcn_readfirstlane((uint32_t)routes.list[slot]);
    // the pairs of the expert's tokens: of a token that has it twice, the first
    const uint32_t lane = threadIdx.x % 64;
    int pair = -1;
    if (lane < g.tokens)
        for (uint32_t j = g.top_k; j-- > 0;)
            if (lds_ids()[lane * g.top_k + j] == (int)e) pair = (int)(lane * g.top_k + j);
    const uint64_t mask = __ballot(pair >= 0);
    if (threadIdx.x < 64 && pair >= 0)
        rows[__popcll(mask & ((1ull << lane) - 1))] = (uint16_t)pair;
    __syncthreads();
    const uint32_t count = (uint32_t)__popcll(mask);
    if (RM == 1 || count <= 16) up_rows<T, W, 1, FN, DEEP>(g, e, n0, rows, count, sums);
    else up_rows<T, W, RM, FN, DEEP / 2>(g, e, n0, rows, count, sums);
}

// ---------------------------------------------------------------------------
// 16 FN columns of the result. The steps of all experts, one expert's after another's, go to the waves
// of `splits` workgroups in turn; each adds up its own, a step's product times the token's weight for
// the expert (and the column's scale), the workgroup's last one to arrive adds the workgroups' sums in
// their order.
// Lane l holds the scale of column l % 16; a result's column is at * 4 + c.
__device__ __forceinline__ float column_scale(float scale, int c)
{
    return __shfl(scale, threadIdx.x % 64 / 16 * 4 + c, 64);
}

template <class T, class W, int RM, int FN, int DEEP>
__global__ void __launch_bounds__(256) k_few_down(FewArgs g)
{
    constexpr bool kScales = std::is_same<W, int8_t>::value;
    typedef Piece<T, W, RM, FN> Loads;
    struct P : Loads {
        float by[RM];
        uint32_t has;  // bit i: the token of row i has the expert
        float scale[kScales ? FN : 1];  // of column lane % 16
    };
    __shared__ Routes routes;
    __shared__ __align__(16) f32x4 sums[4 * RM * FN * 64];
    __shared__ uint32_t last;
    find_routes<true>(g, routes);
    const uint32_t lane = threadIdx.x % 64, at = lane / 16;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t tile = blockIdx.x % g.tiles, split = blockIdx.x / g.tiles;
    const uint32_t n0 = tile * 16 * FN, pairs = g.tokens * g.top_k;
    const uint32_t steps = (row_bytes<W>(g.hidden) + kTurn - 1) / kTurn;
    const uint32_t turn = g.splits * 4;
    const uint32_t mine = pieces(__builtin_amdgcn_readfirstlane(routes.count) * steps,
                                 split * 4 + wave, turn);

    // where the next piece is fetched from
    uint32_t slot = 0, step = split * 4 + wave;
    const char *a[RM], *b[FN], *powers[FN];
    const char *scales = nullptr;
    uint32_t columns[FN];
    float by[RM];
    uint32_t has = 0;
    auto enter = [&] {
        const uint32_t e = __builtin_amdgcn_readfirstlane((uint32_t)routes.list[slot]);
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            uint32_t c = n0 + j * 16 + lane % 16;
            c = c < g.n ? c : g.n - 1;
            b[j] = g.down.data + (int64_t)e * g.down.stride + (int64_t)c * g.down.ld + at * 16;
            powers[j] = nullptr;
            if constexpr (P::kPowers)
                powers[j] = g.down.scales + (int64_t)e * g.down.scales_stride +
                            (int64_t)c * g.down.ld_scales;
            columns[j] = c * 4;
        }
        if constexpr (kScales) scales = g.down.scales + (int64_t)e * g.down.scales_stride;
        int pair[RM], any = 0;
        has = 0;
#pragma unroll
        for (int i = 0; i < RM; ++i) {
            const uint32_t t = i * 16 + lane % 16;
            pair[i] = -1;
            by[i] = 0.f;
            if (t < g.tokens)
                for (uint32_t j = 0; j < g.top_k; ++j)
                    if (lds_ids()[t * g.top_k + j] == (int)e) {
                        pair[i] = pair[i] < 0 ? (int)(t * g.top_k + j) : pair[i];
                        by[i] += lds_by(pairs)[t * g.top_k + j];
                    }
            const uint64_t found = __ballot(pair[i] >= 0);
            if (found) any = __builtin_amdgcn_readlane(pair[i], __builtin_ctzll(found));
            has |= pair[i] >= 0 ? 1u << i : 0;
        }
        // a token without the expert reads the row of one that has it, and leaves the product out
#pragma unroll
        for (int i = 0; i < RM; ++i)
            a[i] = g.h + (int64_t)(pair[i] >= 0 ? pair[i] : any) * g.ldh + at * Loads::C * 16;
    };
    auto find = [&] {  // the step's expert
        if (step < steps) return;
        do {
            step -= steps;
            ++slot;
        } while (step >= steps);
        enter();
    };
    f32x4 total[RM][FN] = {};
    if (mine) {
        P p[DEEP];
        uint32_t left = mine;
        enter();
        find();
        pipeline(mine, p,
                 [&](P &q) {
                     q.fetch(a, b, powers, step, g.hidden);
#pragma unroll
                     for (int i = 0; i < RM; ++i) q.by[i] = by[i];
                     q.has = has;
                     if constexpr (kScales)
#pragma unroll
                         for (int j = 0; j < FN; ++j)
                             q.scale[j] = *(const float *)(scales + columns[j]);
                     if (left > 1) {
                         --left;
                         step += turn;
                         find();
                     }
                 },
                 [&](P &q) {
                     f32x4 acc[RM][FN] = {};
                     q.multiply(acc, g.hidden);
#pragma unroll
                     for (int i = 0; i < RM; ++i)
#pragma unroll
                         for (int j = 0; j < FN; ++j)
#pragma unroll
                             for (int c = 0; c < 4; ++c) {
                                 float v = acc[i][j][c] * q.by[i];
                                 if constexpr (kScales) v *= column_scale(q.scale[j], c);
                                 total[i][j][c] += q.has >> i & 1 ? v : 0.f;
                             }
                 });
    }
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) sums[(wave * RM * FN + i * FN + j) * 64 + lane] = total[i][j];
    __syncthreads();
    auto store = [&](uint32_t f, f32x4 v) {
        const uint32_t t = f / FN * 16 + lane % 16, c = n0 + f % FN * 16 + at * 4;
        if (t >= g.tokens || c >= g.n) return;
        typedef T T4 __attribute__((ext_vector_type(4)));
        T *to = (T *)(g.out + t * g.ldo) + c;
        const T4 o = {(T)v[0], (T)v[1], (T)v[2], (T)v[3]};
        if (c + 4 <= g.n) {
            store_any(to, o);
        } else {
#pragma unroll
            for (int q = 0; q < 3; ++q)
                if (c + q < g.n) to[q] = o[q];
        }
    };
    uint32_t *const parts = g.partial + (uint64_t)tile * g.splits * (RM * FN * 256);
    for (uint32_t f = wave; f < RM * FN; f += 4) {
        f32x4 v = sums[f * 64 + lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) v += sums[(w * RM * FN + f) * 64 + lane];
        if (g.splits == 1) {
            store(f, v);
        } else {
            // written through to where every XCD sees it
            uint32_t *to = parts + (split * RM * FN + f) * 256 + lane;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                __hip_atomic_store(to + q * 64, __float_as_uint(v[q]), __ATOMIC_RELAXED,
                                   __HIP_MEMORY_SCOPE_AGENT);
        }
    }
    if (g.splits == 1) return;
    asm volatile("s_waitcnt vmcnt(0)" : : : "memory");  // this wave's sums are there
    __syncthreads();
    if (threadIdx.x == 0)
        last = __hip_atomic_fetch_add(g.arrived + tile, 1u, __ATOMIC_RELAXED,
                                      __HIP_MEMORY_SCOPE_AGENT) == g.splits - 1;
    __syncthreads();
    if (!last) return;
    for (uint32_t f = wave; f < RM * FN; f += 4) {
        f32x4 v = {};
        for (uint32_t s = 0; s < g.splits; ++s) {
            const uint32_t *from = parts + (s * RM * FN + f) * 256 + lane;
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[q] += __uint_as_float(__hip_atomic_load(from + q * 64, __ATOMIC_RELAXED,
                                                          __HIP_MEMORY_SCOPE_AGENT));
        }
        store(f, v);
    }
}

// ---------------------------------------------------------------------------
// Fragments of columns of a workgroup (FN): two where the weights are narrower than the tokens, whose
// rows then count for more of what is loaded, if there are no more than 16 of them.
template <class W, int RM> constexpr int few_columns() { return sizeof(W) == 2 || RM > 1 ? 1 : 2; }
inline uint32_t columns_of(int32_t kind, uint32_t rows)
{
    return kind == EXPERTS_WEIGHT_16 || rows > 1 ? 1 : 2;
}

inline uint32_t rows_of_16(uint64_t tokens) { return tokens <= 16 ? 1 : tokens <= 32 ? 2 : 4; }

struct FewPlan {
    uint32_t rows, tiles, splits;  // of the result
    uint64_t h, arrived, partial, bytes;  // offsets in the workspace, and its size
};

inline FewPlan few_plan(uint64_t tokens, uint32_t top_k, uint32_t experts, uint32_t hidden, uint32_t n,
                        int32_t down_kind)
{
    FewPlan p;
    p.rows = rows_of_16(tokens);
    const uint32_t fn = columns_of(down_kind, p.rows);
    p.tiles = (n + 16 * fn - 1) / (16 * fn);
    const uint64_t pairs = tokens * top_k, slots = pairs < experts ? pairs : experts;
    const uint32_t bytes = down_kind == EXPERTS_WEIGHT_16     ? hidden * 2
                           : down_kind == EXPERTS_WEIGHT_INT8 ? hidden
                                                              : (hidden + 31) / 32 * 16;
    // workgroups for 4 on each CU, if there are steps for them: 4 for each wave
    const uint64_t steps = slots * ((bytes + kTurn - 1) / kTurn);
    uint64_t splits = (1024 + p.tiles - 1) / p.tiles;
    if (splits > steps / 16) splits = steps / 16;
    p.splits = (uint32_t)(splits < 1 ? 1 : splits > 64 ? 64 : splits);
    auto up = [](uint64_t b) { return (b + 255) / 256 * 256; };
    p.h = 0;
    p.arrived = up(pairs * ((hidden + 7) / 8 * 16));
    p.partial = p.arrived + up((uint64_t)p.tiles * 4);
    p.bytes = p.partial + (p.splits > 1 ? (uint64_t)p.tiles * p.splits * p.rows * fn * 1024 : 0);
    return p;
}

template <class T, class W, int RM>
hist_status_t launch_up(const FewArgs &g, uint64_t slots, hipStream_t stream)
{
    constexpr int FN = few_columns<W, RM>(), DEEP = sizeof(W) == 2 ? 8 : 4;
    const uint32_t each = g.gated ? 16 * FN : 32 * FN;
    return launch(k_few_up<T, W, RM, FN, DEEP>, slots * ((g.hidden + each - 1) / each), 256,
                  (g.tokens * g.top_k * 2 + 15) / 16 * 16, stream, g);
}

template <class T, class W>
hist_status_t launch_up_any(const FewArgs &g, uint64_t slots, hipStream_t stream)
{
    return g.tokens <= 16 ? launch_up<T, W, 1>(g, slots, stream)
                          : launch_up<T, W, 4>(g, slots, stream);
}

template <class T, class W, int RM>
hist_status_t launch_down(const FewArgs &g, hipStream_t stream)
{
    constexpr int FN = few_columns<W, RM>(), DEEP = (sizeof(W) == 2 ? 8 : 4) / (RM == 1 ? 1 : 2);
    const uint32_t pairs = g.tokens * g.top_k;
    return launch(k_few_down<T, W, RM, FN, DEEP>, (uint64_t)g.tiles * g.splits, 256,
                  (pairs * 2 + 15) / 16 * 16 + pairs * 4, stream, g);
}

template <class T, class W>
hist_status_t launch_down_any(const FewArgs &g, uint32_t rows, hipStream_t stream)
{
    return rows == 1   ? launch_down<T, W, 1>(g, stream)
           : rows == 2 ? launch_down<T, W, 2>(g, stream)
                       : launch_down<T, W, 4>(g, stream);
}

template <class T>
hist_status_t launch_few(const FewArgs &g, const FewPlan &p, int32_t up_kind, int32_t down_kind,
                         hipStream_t stream)
{
    const uint64_t pairs = (uint64_t)g.tokens * g.top_k;
    const uint64_t slots = pairs < g.experts ? pairs : g.experts;
    const hist_status_t st =
        up_kind == EXPERTS_WEIGHT_16     ? launch_up_any<T, T>(g, slots, stream)
        : up_kind == EXPERTS_WEIGHT_INT8 ? launch_up_any<T, int8_t>(g, slots, stream)
                                         : launch_up_any<T, Mx4>(g, slots, stream);
    if (st != HIST_OK) return st;
    return down_kind == EXPERTS_WEIGHT_16     ? launch_down_any<T, T>(g, p.rows, stream)
           : down_kind == EXPERTS_WEIGHT_INT8 ? launch_down_any<T, int8_t>(g, p.rows, stream)
                                              : launch_down_any<T, Mx4>(g, p.rows, stream);
}

// Defined in a source of their own each, so that they compile at one time.
hist_status_t launch_few_bf16(const FewArgs &g, const FewPlan &p, int32_t up_kind,
                              int32_t down_kind, hipStream_t stream);
hist_status_t launch_few_fp16(const FewArgs &g, const FewPlan &p, int32_t up_kind,
                              int32_t down_kind, hipStream_t stream);

}  // namespace pca_experts
