// experts_product.hpp -- the kernels of the expert layer's matrix products and how
// they are launched. Part of libpca_hist.so.
#pragma once

#include "experts_tile.hpp"

#include <type_traits>

namespace pca_experts {

constexpr uint32_t kCus = 256;           // of the device
constexpr uint32_t kLdsOfCu = 160 << 10;  // bytes

struct RowsArgs {
    char *out;
    const char *a;
    const char *b;
    int64_t ldo, lda, ldb, b_stride;  // bytes
    const int32_t *offsets;           // nullptr: one group
    const int32_t *order;             // nullptr: row p of a belongs to row p
    const float *sa, *sb;             // 8-bit operands' scales
    uint32_t rows, a_rows, experts;
    uint32_t cols;   // of the result
    uint32_t bytes;  // of the reduction
    uint32_t n_tiles, span;
    Divide divide;  // by top_k
};

// The row of a that sorted row p reads; a bad index reads row 0 (the row's
// place in the result is still its own).
__device__ __forceinline__ uint32_t source_row(const RowsArgs &g, uint32_t p)
{
    if (!g.order) return p;
    const uint32_t t = g.divide((uint32_t)g.order[p]);
    return t < g.a_rows ? t : 0;
}

// A wave's fragments, FM x FN of 16 x 16 results, to memory: through LDS, so that
// whole rows of the wave's part leave together, 16 bytes a lane (stored as they
// lie in registers, 8 bytes a lane, a store touched 16 pieces of 32 bytes).
// value(i, j): the four results of fragment (i, j) in this lane, columns lane / 16 * 4
// + 0..3 of row lane % 16. out: the part's first element, `high` rows and `wide`
// columns of it exist. lds: the wave's own FM * FN * 512 bytes.
template <class O, int FM, int FN, class F>
__device__ __forceinline__ void store_part(char *lds, O *out, int64_t ld_bytes, int high, int wide,
                                           F value)
{
    typedef O O4 __attribute__((ext_vector_type(4)));
    constexpr uint32_t kRow = FN * 32, kPieces = FN * 2;  // bytes and 16-byte pieces of a row
    const uint32_t lane = threadIdx.x % 64;
#pragma unroll
    for (int i = 0; i < FM; ++i) {
        const uint32_t r = i * 16 + lane % 16;
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const f32x4 v = value(i, j);
            const uint32_t c = j * 16 + lane / 16 * 4;
            *(O4 *)(lds + r * kRow + ((c / 8) ^ (r % kPieces)) * 16 + c % 8 * 2) =
                O4{(O)v[0], (O)v[1], (O)v[2], (O)v[3]};
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int s = 0; s < FM * 16 * (int)kPieces / 64; ++s) {
        const uint32_t r = (s * 64 + lane) / kPieces, p = lane % kPieces;
        const auto v = *(const typename Vec8<O>::type *)(lds + r * kRow + (p ^ (r % kPieces)) * 16);
        const int left = wide - (int)p * 8;
        if ((int)r < high && left > 0) store8((O *)((char *)out + r * ld_bytes) + p * 8, v, left);
    }
}

// A row's scale of the 8-bit product. A whole-number sum times the scale can pass the range of 32 bits
// where the column's scale would bring it back (a row with 3e38 in it), so a large scale is taken 2^64
// times smaller, and the result 2^64 times larger again. Both are exact, and nothing between them is too
// small: sum * scale is 2^32 or more (or 0), times the least column's scale 2^-117.
struct RowScale {
    float by, back;
    static __device__ __forceinline__ RowScale of(float s)
    {
        const bool large = fabsf(s) >= 0x1p96f;
        return {large ? s * 0x1p-64f : s, large ? 0x1p64f : 1.f};
    }
    __device__ __forceinline__ float operator()(int32_t sum, float column) const
    {
        return (float)sum * by * column * back;
    }
};

// The widest reduction, EXPERTS_MAX_WIDTH products of -128 and -128, sums to 2^31 and wraps to
// -2^31, which is no other sum: the least real one is 2^17 * -128 * 127. 2^31 - 1 becomes 2^31 as a float.
__device__ __forceinline__ void unwrap(s32x4 &sums)
{
#pragma unroll
    for (int q = 0; q < 4; ++q) sums[q] = sums[q] == INT32_MIN ? INT32_MAX : sums[q];
}

__device__ __forceinline__ f32x4 plus(f32x4 a, f32x4 b) { return a + b; }
__device__ __forceinline__ s32x4 plus(s32x4 a, s32x4 b)  // wraps, see unwrap()
{
    return __builtin_bit_cast(s32x4,
                              __builtin_bit_cast(u32x4, a) + __builtin_bit_cast(u32x4, b));
}

// The part of a product of rows: `real` is false for rows past the last kept one.
template <class T, class O, int FM, int FN, class Acc>
__device__ __forceinline__ void store_rows(const RowsArgs &g, char *lds, const Tile &t,
                                           Acc (&acc)[FM][FN], bool real, uint32_t row,
                                           uint32_t col, int high, int wide)
{
    O *out = (O *)(g.out + (int64_t)row * g.ldo) + col;
    if constexpr (sizeof(T) == 1) {
        const uint32_t lane = threadIdx.x % 64;
        f32x4 sb[FN] = {};
        RowScale sa[FM] = {};
        if (real) {
            const float *from = g.sb + (uint64_t)t.group * g.cols + col;
#pragma unroll
            for (int j = 0; j < FN; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int c = j * 16 + lane / 16 * 4 + q;
                    sb[j][q] = c < wide ? from[c] : 0.f;
                }
#pragma unroll
            for (int i = 0; i < FM; ++i) {
                const int r = i * 16 + lane % 16;
                sa[i] = RowScale::of(r < high ? g.sa[source_row(g, row + r)] : 0.f);
            }
        }
        if (g.bytes == EXPERTS_MAX_WIDTH)
#pragma unroll
            for (int i = 0; i < FM; ++i)
#pragma unroll
                for (int j = 0; j < FN; ++j) unwrap(acc[i][j]);
        store_part<O, FM, FN>(lds, out, g.ldo, high, wide, [&](int i, int j) {
            f32x4 v;
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = sa[i](acc[i][j][q], sb[j][q]);
            return v;
        });
    } else {
        store_part<O, FM, FN>(lds, out, g.ldo, high, wide, [&](int i, int j) { return acc[i][j]; });
    }
}

struct DwArgs {
    char *out;
    const char *dy;
    const char *x;
    int64_t lddy, ldx;  // bytes
    const int32_t *offsets;
    const int32_t *order;
    uint32_t rows, x_rows, experts, n, k;
    uint32_t n_tiles, k_tiles, span;
    Divide divide;  // by top_k
};

// ---------------------------------------------------------------------------
// The pipelined products.

// BM x BN results by WM x WN waves, PER_CU workgroups on a CU, STAGES steps in LDS.
template <int BM_, int BN_, int WM_, int WN_, int PER_CU_, int STAGES_ = 2>
struct Shape {
    static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_;
    static constexpr int THREADS = WM * WN * 64, PER_CU = PER_CU_, STAGES = STAGES_;
    static constexpr int FM = BM / WM / 16, FN = BN / WN / 16;  // fragments of a wave
    static constexpr int WAVES_PER_SIMD = THREADS / 256 * PER_CU;
};

extern __shared__ __align__(16) char pipe_lds[];

// The loop over the steps. load(fast, parity, step, lds, i) queues piece i of LOADS of a step
// (fast: a whole one, of which there are `whole`; parity: the step's). Where it is not
// DIRECT, it puts the piece, which is in registers by then, and fetches that of two steps later,
// and first(parity, i) fetches those of steps 0 and 1.
// frag_a and frag_b read the fragments of half a step.
//
// A step is two halves. At its top the first half's fragments are in registers (or
// on their way), and the next step's pieces are. While the first half is multiplied
// the second half's fragments are read; then the stage is free, and while the second
// half is multiplied the pieces of the step after the next go there, and the next step's
// first fragments are read. So there is one barrier a step, loads have a step to
// arrive, and all reads and loads are issued between products.
template <class T, class S, bool DIRECT, int LOADS, uint32_t STAGE, class F, class L, class FA,
          class FB>
__device__ __forceinline__ void run_steps(uint32_t steps, uint32_t whole,
                                          typename Mma<T>::Acc (&acc)[S::FM][S::FN], F first, L load,
                                          FA frag_a, FB frag_b)
{
    constexpr int FM = S::FM, FN = S::FN;
    constexpr int N = S::STAGES;
    static_assert(DIRECT || N == 2, "pieces in registers alternate");
    constexpr uint32_t kAhead = DIRECT ? N : 4;  // steps from a step to what it fetches
    struct Frags {
        typename Mma<T>::Frag a[FM], b[FN];
    };
    constexpr int kReads = FM + FN;
    constexpr int kParts = FM * 3 / 4 > 0 ? FM * 3 / 4 : 1;
    // reads after a product, over the first three quarters of the rows; loads over all of them
    constexpr int kSlots = kParts * FN, kReadsEach = (kReads + kSlots - 1) / kSlots;
    constexpr int kReadGap = kSlots / kReads > 0 ? kSlots / kReads : 1;
    constexpr int kLoadsEach = (LOADS + FM * FN - 1) / (FM * FN);
    constexpr int kLoadGap = FM * FN / LOADS > 0 ? FM * FN / LOADS : 1;
    auto read = [&](const char *lds, Frags &f, int kk, int r) {
        if (r < FN) f.b[r] = frag_b(lds, r, kk);
        else f.a[r - FN] = frag_a(lds, r - FN, kk);
    };
    auto half = [&](auto with_loads, auto fast, auto stage, const Frags &now, Frags &then,
                    const char *lds, int kk, uint32_t step, uint32_t to) {
#pragma unroll
        for (int i = 0; i < FM; ++i) {
#pragma unroll
            for (int j = 0; j < FN; ++j) {
                acc[i][j] = Mma<T>::run(now.b[j], now.a[i], acc[i][j]);
                const int slot = i * FN + j;
                if (slot % kReadGap == 0)
#pragma unroll
                    for (int q = 0; q < kReadsEach; ++q)
                        if (slot / kReadGap * kReadsEach + q < kReads)
                            read(lds, then, kk, slot / kReadGap * kReadsEach + q);
                if constexpr (decltype(with_loads)::value)
                    if (slot % kLoadGap == 0)
#pragma unroll
                        for (int q = 0; q < kLoadsEach; ++q)
                            if (slot / kLoadGap * kLoadsEach + q < LOADS)
                                load(fast, stage, step, to, slot / kLoadGap * kLoadsEach + q);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)pipe_lds;
    Frags f[2];
    auto step = [&](auto fast, auto stage, uint32_t k) {
        constexpr uint32_t kHere = decltype(stage)::value * STAGE;
        constexpr uint32_t kThere = (decltype(stage)::value + 1) % N * STAGE;
        half(std::false_type(), fast, stage, f[0], f[1], pipe_lds + kHere, 1, 0, 0);
        __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave has left the stage
        if constexpr (DIRECT) {  // the next step's pieces are here
            if (N == 2 || (!decltype(fast)::value && k + N - 1 >= steps)) wait_loads<0>();
            else wait_loads<LOADS *(N - 2)>();
        }
        block_barrier();
        half(std::true_type(), fast, stage, f[1], f[0], pipe_lds + kThere, 0, k + N, base + kHere);
    };
    typedef std::integral_constant<int, 0> Even;
    typedef std::integral_constant<int, 1> Odd;
    if constexpr (!DIRECT) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) first(Even(), i);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) first(Odd(), i);
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load(std::false_type(), Even(), 0, base, i);
#pragma unroll
    for (int s = 1; s < N; ++s)
        if ((uint32_t)s < steps)
#pragma unroll
            for (int i = 0; i < LOADS; ++i) load(std::false_type(), Odd(), s, base + s * STAGE, i);
    if constexpr (DIRECT) {
        if (steps >= N) wait_loads<LOADS *(N - 1)>();
        else wait_loads<0>();
    } else {
        __builtin_amdgcn_s_waitcnt(0xc07f);
    }
    block_barrier();
#pragma unroll
    for (int r = 0; r < kReads; ++r) read(pipe_lds, f[0], 0, r);
    uint32_t k = 0;
    typedef std::integral_constant<int, 2 % N> Third;
    typedef std::integral_constant<int, 3 % N> Fourth;
    for (; k + kAhead + N - 1 < whole; k += N) {
        step(std::true_type(), Even(), k);
        step(std::true_type(), Odd(), k + 1);
        if constexpr (N > 2) step(std::true_type(), Third(), k + 2);
        if constexpr (N > 3) step(std::true_type(), Fourth(), k + 3);
    }
    for (; k < steps; k += N) {
        step(std::false_type(), Even(), k);
        if (k + 1 < steps) step(std::false_type(), Odd(), k + 1);
        if constexpr (N > 2)
            if (k + 2 < steps) step(std::false_type(), Third(), k + 2);
        if constexpr (N > 3)
            if (k + 3 < steps) step(std::false_type(), Fourth(), k + 3);
    }
    block_barrier();
}

// The same where two sets of fragments do not fit beside the sums, as with two
// operands across the reduction: a fragment of A takes the registers of the one that has just
// been used up (those of B alternate), so the reads of the second half end with the first
// half's products, and the barrier comes a few rows of products into the second. look(step)
// asks for what the loads of that step need (row numbers), turn(step) makes addresses of it.
template <class T, class S, bool DIRECT, int LOADS, uint32_t STAGE, class F, class L, class FA,
          class FB, class K, class U>
__device__ __forceinline__ void run_steps_sharing(uint32_t steps, uint32_t whole,
                                          typename Mma<T>::Acc (&acc)[S::FM][S::FN], F first, L load,
                                          FA frag_a, FB frag_b, K look, U turn)
{
    constexpr int FM = S::FM, FN = S::FN;
    constexpr uint32_t kAhead = DIRECT ? 2 : 4;  // steps from a step to what it fetches
    constexpr int kWait = FM / 4;  // rows of the second half before the barrier
    constexpr int kReads = (FM + FN + FM - kWait - 1) / (FM - kWait);
    constexpr int kLoads = (LOADS + FM - kWait - 1) / (FM - kWait);
    static_assert(kWait > 0 && FN <= FM, "rows to spread the reads over");
    constexpr bool kUsedUp = [] {  // a fragment of A is only read after its row's products
        for (int i = kWait; i < FM; ++i) {
            const int past = (i - kWait + 1) * kReads;
            if ((past < FM + FN ? past : FM + FN) - 1 - FN > i) return false;
        }
        return true;
    }();
    static_assert(kUsedUp, "reads that are not ahead of the products");
    typename Mma<T>::Frag a[FM], b[2][FN];
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)pipe_lds;
    auto products = [&](int i, const typename Mma<T>::Frag (&with)[FN]) {
#pragma unroll
        for (int j = 0; j < FN; ++j) Mma<T>::add(with[j], a[i], acc[i][j]);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto step = [&](auto fast, auto stage, uint32_t k) {
        constexpr uint32_t kHere = decltype(stage)::value * STAGE;
        constexpr uint32_t kThere = STAGE - kHere;
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            products(i, b[0]);
            if (i < FN) b[1][i] = frag_b(pipe_lds + kHere, i, 1);
            a[i] = frag_a(pipe_lds + kHere, i, 1);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < FM; ++i) {
            products(i, b[1]);
            if (i == kWait - 1) {
                __builtin_amdgcn_s_waitcnt(0xc07f);  // lgkmcnt(0): this wave has left the stage
                if constexpr (DIRECT) wait_loads<0>();
                turn(k + kAhead);  // what it looked up has arrived with the pieces
                look(k + kAhead + 1);
                block_barrier();
            } else if (i >= kWait) {
#pragma unroll
                for (int r = (i - kWait) * kReads; r < (i - kWait + 1) * kReads; ++r) {
                    if (r < FN) b[0][r] = frag_b(pipe_lds + kThere, r, 0);
                    else if (r < FM + FN) a[r - FN] = frag_a(pipe_lds + kThere, r - FN, 0);
                }
#pragma unroll
                for (int p = (i - kWait) * kLoads; p < (i - kWait + 1) * kLoads; ++p)
                    if (p < LOADS) load(fast, stage, k + 2, base + kHere, p);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    typedef std::integral_constant<int, 0> Even;
    typedef std::integral_constant<int, 1> Odd;
    look(0);
    turn(0);
    if constexpr (!DIRECT) {
#pragma unroll
        for (int i = 0; i < LOADS; ++i) first(Even(), i);
        look(1);
        turn(1);
#pragma unroll
        for (int i = 0; i < LOADS; ++i) first(Odd(), i);
        look(2);
        turn(2);
    }
#pragma unroll
    for (int i = 0; i < LOADS; ++i) load(std::false_type(), Even(), 0, base, i);
    look(kAhead - 1);
    turn(kAhead - 1);
    if (steps > 1)
#pragma unroll
        for (int i = 0; i < LOADS; ++i) load(std::false_type(), Odd(), 1, base + STAGE, i);
    if constexpr (DIRECT) {
        if (steps > 1) wait_loads<LOADS>();
        else wait_loads<0>();
    } else {
        __builtin_amdgcn_s_waitcnt(0xc07f);
    }
    look(kAhead);
    block_barrier();
#pragma unroll
    for (int j = 0; j < FN; ++j) b[0][j] = frag_b(pipe_lds, j, 0);
#pragma unroll
    for (int i = 0; i < FM; ++i) a[i] = frag_a(pipe_lds, i, 0);
    uint32_t k = 0;
    for (; k + kAhead + 1 < whole; k += 2) {
        step(std::true_type(), Even(), k);
        step(std::true_type(), Odd(), k + 1);
    }
    for (; k < steps; k += 2) {
        step(std::false_type(), Even(), k);
        if (k + 1 < steps) step(std::false_type(), Odd(), k + 1);
    }
    sums_done(acc);
    block_barrier();
}

// The loads and barriers of either loop, for a wave whose rows a short tile does not have.
template <int LOADS, uint32_t STAGE, class L>
__device__ __forceinline__ void run_steps_idle(uint32_t steps, L load)
{
    typedef std::integral_constant<int, 0> Any;
    const uint32_t base = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char *)pipe_lds;
    for (uint32_t s = 0; s < 2 && s < steps; ++s)
#pragma unroll
        for (int i = 0; i < LOADS; ++i) load(std::false_type(), Any(), s, base + s * STAGE, i);
    if (steps > 1) wait_loads<LOADS>();
    else wait_loads<0>();
    block_barrier();
    for (uint32_t k = 0; k < steps; ++k) {
        wait_loads<0>();
        block_barrier();
#pragma unroll
        for (int i = 0; i < LOADS; ++i)
            load(std::false_type(), Any(), k + 2, base + (k & 1) * STAGE, i);
    }
    block_barrier();
}

// How the operands of a product of rows, and of the weights' gradient, are staged.
template <class T, class S, bool ACROSS>
struct RowsParts {
    static_assert(!ACROSS || S::BN / S::WN % 64 == 0, "a wave's fragments across start at 64 columns");
    typedef Along<T, S::BM, S::THREADS> A;
    typedef typename std::conditional<ACROSS, Across<T, S::BN, S::THREADS>,
                                      Along<T, S::BN, S::THREADS>>::type B;
    static constexpr uint32_t STAGE = A::kBytes + B::kBytes;
};
template <class T, class S>
struct DwParts {
    static_assert(S::BM / S::WM % 64 == 0 && S::BN / S::WN % 64 == 0, "as in RowsParts");
    typedef Across<T, S::BM, S::THREADS> A;
    typedef Across<T, S::BN, S::THREADS> B;
    static constexpr uint32_t STAGE = A::kBytes + B::kBytes;
};

// Rows times their experts' weights, or the gradient of the rows. Bound by the matrix cores
// where groups are long: 32768 pairs, 4096 x 4096, bf16 in 256 x 256 tiles take 880-925 us, 1.19 to 1.25
// PFLOP/s, with the matrix cores busy 70% of the cycles (a dense product of the
// same rows 824 us, the library's 735); by reading the weights where they are short
// (launch_rows has the figures).
// T: element of the operands; O: of the result; ACROSS: the weights lie across the
// reduction; DIRECT: every row at a multiple of 16 bytes, and all rows that a tile can take within
// 32-bit offsets of one address.
template <class T, class O, class S, bool ACROSS, bool DIRECT>
__global__ void __launch_bounds__(S::THREADS)
    __attribute__((amdgpu_waves_per_eu(S::WAVES_PER_SIMD, S::WAVES_PER_SIMD))) k_rows(RowsArgs g)
{
    typedef RowsParts<T, S, ACROSS> P;
    typedef typename P::A A;
    typedef typename P::B B;
    constexpr int kLog2 = __builtin_ctz(S::BM);
    uint32_t tile = tile_of_block(blockIdx.x, g.span), part = 0, parts = 1;
    if constexpr (S::BM == 256) {
        // A workgroup fills a CU. Where the last round of tiles is at most half full, two
        // workgroups take half the rows of each of them.
        const uint32_t all =
            count_row_tiles(g.offsets, g.experts, g.rows, kLog2) * g.n_tiles;
        const uint32_t last = all % kCus, first = all - last;
        if (last <= kCus / 2 && tile >= first) {
            if (tile < first + 2 * last) {
                parts = 2;
                part = (tile - first) % 2;
                tile = first + (tile - first) / 2;
            } else {
                tile -= last;
            }
        }
    }
    const Tile t = find_tile(tile, g.offsets, g.experts, g.rows, kLog2, g.n_tiles);
    if (t.group > g.experts) return;
    const uint32_t rows_each = S::BM / parts;
    const uint32_t m0 = t.begin + t.m * S::BM + part * rows_each;
    if (m0 >= t.end) return;
    // (a last tile across that passes through registers starts where it ends with the last column:
    // no piece then reaches past a row, and the columns that two tiles share get the same bits)
    const bool full = ACROSS && !DIRECT && g.cols >= S::BN;
    const uint32_t n0 = full && g.cols - t.n * S::BN < S::BN ? g.cols - S::BN : t.n * S::BN;
    const uint32_t high = t.end - m0 < rows_each ? t.end - m0 : rows_each;
    const uint32_t wide = g.cols - n0 < S::BN ? g.cols - n0 : S::BN;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t wm = wave / S::WN * (S::BM / S::WM), wn = wave % S::WN * (S::BN / S::WN);
    const bool real = !g.offsets || t.group < g.experts;
    typename Mma<T>::Acc acc[S::FM][S::FN] = {};

    if (real) {
        // rows past the tile's last one read that one: their results are not stored
        const char *rows = g.order ? g.a : g.a + (int64_t)m0 * g.lda;
        auto row_a = [&](int i) {
            const uint32_t r = A::row_of(i) < high ? A::row_of(i) : high - 1;
            return g.order ? source_row(g, m0 + r) : r;
        };
        const char *w = g.b + (int64_t)t.group * g.b_stride +
                        (ACROSS ? (int64_t)n0 * sizeof(T) : (int64_t)n0 * g.ldb);
        auto row_b = [&](int i) { return B::row_of(i) < wide ? B::row_of(i) : wide - 1; };
        const uint32_t steps = (g.bytes + kStepBytes - 1) / kStepBytes;
        // steps that need no check: all but the reduction's ragged end
        const uint32_t whole = ACROSS && !DIRECT && !full ? 0 : g.bytes / kStepBytes;
        auto fa = [&](const char *lds, int i, int kk) { return A::frag(lds, wm, i, kk); };
        auto fb = [&](const char *lds, int j, int kk) {
            return B::frag(lds + A::kBytes, wn, j, kk);
        };
        const uint32_t byte_a = A::byte(), byte_b = B::byte();
        if constexpr (DIRECT) {
            uint32_t at_a[A::kLoads], at_b[ACROSS ? 1 : B::kLoads];
#pragma unroll
            for (int i = 0; i < A::kLoads; ++i) at_a[i] = row_a(i) * (uint32_t)g.lda + byte_a;
            if constexpr (ACROSS) {
                // a piece past the last column reads the first one
                at_b[0] = B::row_of(0) * (uint32_t)g.ldb + (byte_b < wide * 2 ? byte_b : 0);
            } else {
#pragma unroll
                for (int i = 0; i < B::kLoads; ++i) at_b[i] = row_b(i) * (uint32_t)g.ldb + byte_b;
            }
            auto load = [&](auto fast, auto parity, uint32_t step, uint32_t lds, int i) {
                if (!decltype(fast)::value && step >= steps) return;
                const uint32_t from = step * kStepBytes;
                const char *base;
                uint32_t at;
                bool in = true;
                if (i < A::kLoads) {
                    base = rows + from, at = at_a[i], lds += A::place_of(i, wave);
                    if constexpr (!decltype(fast)::value) in = from + byte_a < g.bytes;
                } else {
                    i -= A::kLoads;
                    lds += A::kBytes + B::place_of(i, wave);
                    if constexpr (ACROSS) {
                        const uint32_t r = step * B::kRows + i * B::kRowsEach;
                        base = w + (int64_t)r * g.ldb, at = at_b[0];
                        if constexpr (!decltype(fast)::value)
                            in = (step * B::kRows + B::row_of(i)) * 2 < g.bytes;
                    } else {
                        base = w + from, at = at_b[i];
                        if constexpr (!decltype(fast)::value) in = from + byte_b < g.bytes;
                    }
                }
                if constexpr (decltype(fast)::value) load_to_lds(base, at, lds);
                else load_to_lds(in ? base + at : (const char *)&kZeros, lds);
            };
            if (S::BM == 256 && wm >= high)
                run_steps_idle<A::kLoads + B::kLoads, P::STAGE>(steps, load);
            else
                run_steps<T, S, true, A::kLoads + B::kLoads, P::STAGE>(
                    steps, whole, acc, [](auto, int) {}, load, fa, fb);
        } else {
            const char *from_a[A::kLoads], *from_b[ACROSS ? 1 : B::kLoads];
            u32x4 kept_a[2][A::kLoads], kept_b[2][B::kLoads];
#pragma unroll
            for (int i = 0; i < A::kLoads; ++i) from_a[i] = rows + (int64_t)row_a(i) * g.lda + byte_a;
            if constexpr (ACROSS) {
                from_b[0] = w + (int64_t)B::row_of(0) * g.ldb + byte_b;
            } else {
#pragma unroll
                for (int i = 0; i < B::kLoads; ++i)
                    from_b[i] = w + (int64_t)row_b(i) * g.ldb + byte_b;
            }
            const int left_b = (int)(g.cols - n0) * 2 - (int)byte_b;  // ACROSS: of a row
            const uint32_t reduction = g.bytes / sizeof(T);
            auto fetch = [&](auto fast, auto parity, uint32_t step, int i) {
                constexpr int kTo = decltype(parity)::value;
                if (!decltype(fast)::value && step >= steps) return;
                const uint32_t from = step * kStepBytes;
                const bool whole_step = decltype(fast)::value || step < whole;
                if (i < A::kLoads) {
                    if (whole_step) kept_a[kTo][i] = load_any<u32x4>(from_a[i] + from);
                    else
                        kept_a[kTo][i] = load16<T>(
                            from_a[i] + from, (int)g.bytes - (int)(from + byte_a), g.bytes >= 16);
                } else {
                    i -= A::kLoads;
                    if constexpr (ACROSS) {
                        // a row past the last one reads that one (and counts as 0 below)
                        const int r = (int)(step * B::kRows) + i * B::kRowsEach;
                        const int most = (int)reduction - 1 - (int)B::row_of(0);
                        const char *p =
                            from_b[0] + (int64_t)(whole_step || r <= most ? r : most) * g.ldb;
                        if (whole_step || full) kept_b[kTo][i] = load_any<u32x4>(p);
                        else kept_b[kTo][i] = load16<T>(p, left_b, g.cols >= 8);
                    } else if (whole_step) {
                        kept_b[kTo][i] = load_any<u32x4>(from_b[i] + from);
                    } else {
                        kept_b[kTo][i] = load16<T>(
                            from_b[i] + from, (int)g.bytes - (int)(from + byte_b), g.bytes >= 16);
                    }
                }
            };
            auto load = [&](auto fast, auto parity, uint32_t step, uint32_t lds, int i) {
                if (!decltype(fast)::value && step >= steps) return;
                if (i < A::kLoads) {
                    put_in_lds(kept_a[decltype(parity)::value][i], lds + A::place_of(i, wave));
                } else {
                    const int j = i - A::kLoads;
                    u32x4 v = kept_b[decltype(parity)::value][j];
                    if constexpr (ACROSS)
                        if (!decltype(fast)::value && step * B::kRows + B::row_of(j) >= reduction)
                            v = u32x4{0, 0, 0, 0};
                    put_in_lds(v, lds + A::kBytes + B::place_of(j, wave));
                }
                fetch(fast, parity, step + 2, i);
            };
            auto first = [&](auto parity, int i) {
                fetch(std::false_type(), parity, decltype(parity)::value, i);
            };
            if constexpr (S::FM >= 4)
                run_steps_sharing<T, S, false, A::kLoads + B::kLoads, P::STAGE>(
                    steps, whole, acc, first, load, fa, fb, [](uint32_t) {}, [](uint32_t) {});
            else
                run_steps<T, S, false, A::kLoads + B::kLoads, P::STAGE>(
                    steps, whole, acc, first, load, fa, fb);
        }
    }
    store_rows<T, O>(g, pipe_lds + wave * (S::FM * S::FN * 512), t, acc, real, m0 + wm, n0 + wn,
                     (int)high - (int)wm, (int)wide - (int)wn);
}

// The gradient of the weights: a tile of one expert's, its rows the reduction. 16384 pairs of 32
// skewed experts, 2560 x 2048, fp16: 264-287 us, 0.60 to 0.64 PFLOP/s and 1.6-1.7 TB/s; the steps are few (8 of 64 rows
// on average), so the time is half tile starts and the 128 KiB that each tile stores; with 2048 rows
// an expert it reaches 1.02 PFLOP/s.
template <class T, class S, bool DIRECT>
__global__ void __launch_bounds__(S::THREADS)
    __attribute__((amdgpu_waves_per_eu(S::WAVES_PER_SIMD, S::WAVES_PER_SIMD))) k_dw(DwArgs g)
{
    typedef DwParts<T, S> P;
    typedef typename P::A A;
    typedef typename P::B B;
    const uint32_t tile = tile_of_block(blockIdx.x, g.span);
    const uint32_t each = g.n_tiles * g.k_tiles, rank = tile / each;
    if (rank >= g.experts) return;
    const uint32_t e = g.experts <= 64    ? expert_of_rank<1>(g.offsets, g.experts, g.rows, rank)
                       : g.experts <= 256 ? expert_of_rank<4>(g.offsets, g.experts, g.rows, rank)
                                          : expert_of_rank<EXPERTS_MAX_EXPERTS / 64>(
                                                g.offsets, g.experts, g.rows, rank);
    const uint32_t in = tile - rank * each;
    uint32_t n0 = in % g.n_tiles * S::BM, k0 = in / g.n_tiles * S::BN;
    // (last tiles that pass through registers start where they end with the last column)
    const bool full = !DIRECT && g.n >= S::BM && g.k >= S::BN;
    if (full) {
        n0 = g.n - n0 < S::BM ? g.n - S::BM : n0;
        k0 = g.k - k0 < S::BN ? g.k - S::BN : k0;
    }
    const uint32_t high = g.n - n0 < S::BM ? g.n - n0 : S::BM;
    const uint32_t wide = g.k - k0 < S::BN ? g.k - k0 : S::BN;
    uint32_t end = __builtin_amdgcn_readfirstlane(g.offsets[e + 1]);
    uint32_t begin = __builtin_amdgcn_readfirstlane(g.offsets[e]);
    end = end > g.rows ? g.rows : end;
    begin = begin > end ? end : begin;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t wm = wave / S::WN * (S::BM / S::WM), wn = wave % S::WN * (S::BN / S::WN);
    typename Mma<T>::Acc acc[S::FM][S::FN] = {};
    if (begin < end) {
        const char *dy = g.dy + (int64_t)begin * g.lddy + n0 * 2;
        const char *x = g.x + k0 * 2 + (g.order ? 0 : (int64_t)begin * g.ldx);
        const uint32_t byte_a = A::byte(), byte_b = B::byte();
        const uint32_t count = end - begin, steps = (count + A::kRows - 1) / A::kRows;
        const uint32_t whole = !DIRECT && !full ? 0 : count / A::kRows;
        uint32_t pair[B::kLoads], row_x[B::kLoads];  // of this lane's pieces of x
        auto row_in = [&](uint32_t step, int i) {
            const uint32_t r = step * A::kRows + B::row_of(i);
            return r < count ? r : count - 1;
        };
        auto look = [&](uint32_t step) {
            if (g.order)
#pragma unroll
                for (int i = 0; i < B::kLoads; ++i)
                    pair[i] = (uint32_t)g.order[begin + row_in(step, i)];
        };
        auto turn = [&](uint32_t step) {
#pragma unroll
            for (int i = 0; i < B::kLoads; ++i) {
                uint32_t s;
                if (g.order) {
                    s = g.divide(pair[i]);
                    s = s < g.x_rows ? s : g.x_rows - 1;
                } else {
                    s = row_in(step, i);
                }
                row_x[i] = DIRECT ? s * (uint32_t)g.ldx : s;
            }
        };
        auto fa = [&](const char *lds, int i, int kk) { return A::frag(lds, wm, i, kk); };
        auto fb = [&](const char *lds, int j, int kk) {
            return B::frag(lds + A::kBytes, wn, j, kk);
        };
        if constexpr (DIRECT) {
            // a piece past the last column reads the first one: its results are not stored
            const uint32_t at_a =
                A::row_of(0) * (uint32_t)g.lddy + (byte_a < high * 2 ? byte_a : 0);
            const uint32_t at_b = byte_b < wide * 2 ? byte_b : 0;
            auto load = [&](auto fast, auto parity, uint32_t step, uint32_t lds, int i) {
                if (!decltype(fast)::value && step >= steps) return;
                const char *base = x;
                uint32_t at, row;
                if (i < A::kLoads) {
                    base = dy + (int64_t)(step * A::kRows + i * A::kRowsEach) * g.lddy;
                    at = at_a, row = A::row_of(i), lds += A::place_of(i, wave);
                } else {
                    i -= A::kLoads;
                    at = row_x[i] + at_b, row = B::row_of(i);
                    lds += A::kBytes + B::place_of(i, wave);
                }
                if constexpr (decltype(fast)::value) load_to_lds(base, at, lds);
                else
                    load_to_lds(step * A::kRows + row < count ? base + at : (const char *)&kZeros,
                                lds);
            };
            run_steps_sharing<T, S, true, A::kLoads + B::kLoads, P::STAGE>(
                steps, whole, acc, [](auto, int) {}, load, fa, fb, look, turn);
        } else {
            u32x4 kept_a[2][A::kLoads], kept_b[2][B::kLoads];
            const int left_a = (int)(g.n - n0) * 2 - (int)byte_a;
            const int left_b = (int)(g.k - k0) * 2 - (int)byte_b;
            const char *from_a = dy + (int64_t)A::row_of(0) * g.lddy + byte_a, *from_b = x + byte_b;
            // rows past the last one read that one (and count as 0 below)
            const int most_a = (int)count - 1 - (int)A::row_of(0);
            auto fetch = [&](auto fast, auto parity, uint32_t step, int i) {
                constexpr int kTo = decltype(parity)::value;
                if (!decltype(fast)::value && step >= steps) return;
                if (i < A::kLoads) {
                    const int r = (int)(step * A::kRows) + i * A::kRowsEach;
                    const int row = decltype(fast)::value || r <= most_a ? r : most_a;
                    const char *p = from_a + (int64_t)row * g.lddy;
                    if (decltype(fast)::value || full) kept_a[kTo][i] = load_any<u32x4>(p);
                    else kept_a[kTo][i] = load16<T>(p, left_a, g.n >= 8);
                } else {
                    i -= A::kLoads;
                    const char *p = from_b + (int64_t)row_x[i] * g.ldx;
                    if (decltype(fast)::value || full) kept_b[kTo][i] = load_any<u32x4>(p);
                    else kept_b[kTo][i] = load16<T>(p, left_b, g.k >= 8);
                }
            };
            auto load = [&](auto fast, auto parity, uint32_t step, uint32_t lds, int i) {
                if (!decltype(fast)::value && step >= steps) return;
                const int j = i < A::kLoads ? i : i - A::kLoads;
                u32x4 v = i < A::kLoads ? kept_a[decltype(parity)::value][j % A::kLoads]
                                        : kept_b[decltype(parity)::value][j % B::kLoads];
                const uint32_t row = i < A::kLoads ? A::row_of(j) : B::row_of(j);
                if (!decltype(fast)::value && step * A::kRows + row >= count) v = u32x4{0, 0, 0, 0};
                put_in_lds(v, lds + (i < A::kLoads ? A::place_of(j, wave)
                                                   : A::kBytes + B::place_of(j, wave)));
                fetch(fast, parity, step + 2, i);
            };
            run_steps_sharing<T, S, false, A::kLoads + B::kLoads, P::STAGE>(
                steps, whole, acc,
                [&](auto parity, int i) {
                    fetch(std::false_type(), parity, decltype(parity)::value, i);
                },
                load, fa, fb, look, turn);
        }
    }
    store_part<T, S::FM, S::FN>(pipe_lds + wave * (S::FM * S::FN * 512),
                                (T *)g.out + ((int64_t)e * g.n + n0 + wm) * g.k + k0 + wn,
                                (int64_t)g.k * 2, (int)high - (int)wm, (int)wide - (int)wn,
                                [&](int i, int j) { return acc[i][j]; });
}

// ---------------------------------------------------------------------------
// Few rows: the time goes into reading the weights once, so what counts is how many bytes are
// in flight. A workgroup takes 16 * FN columns and 16 * RM rows; its four waves
// divide the reduction, 128 bytes of it in turn, and add their sums through LDS at the
// end, in the order of the waves. The fragments come from memory to registers as the
// matrix instruction wants them (a lane's 16 bytes are consecutive in a row), with no LDS
// between, `DEEP` pieces of 128 bytes ahead. Any alignment. 4 tokens of 8 choices, 64
// experts of 2560 x 2048: 46 us, 6 TB/s.
template <class T, class O, int RM, int FN, int DEEP>
__global__ void __launch_bounds__(256) k_rows_thin(RowsArgs g)
{
    typedef typename Mma<T>::Acc Acc;
    typedef typename Mma<T>::Frag Frag;
    __shared__ __align__(16) Acc sums[4][RM * FN][64];
    const Tile t = find_tile(tile_of_block(blockIdx.x, g.span), g.offsets, g.experts, g.rows,
                                    4 + __builtin_ctz(RM), g.n_tiles);
    if (t.group > g.experts) return;
    const uint32_t m0 = t.begin + t.m * 16 * RM, n0 = t.n * 16 * FN;
    const uint32_t high = t.end - m0 < 16 * RM ? t.end - m0 : 16 * RM;
    const uint32_t wide = g.cols - n0 < 16 * FN ? g.cols - n0 : 16 * FN;
    const uint32_t lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const bool real = !g.offsets || t.group < g.experts;
    Acc acc[RM][FN] = {};
    if (real) {
        const char *a[RM], *b[FN];
        const uint32_t at = lane / 16 * 16;
#pragma unroll
        for (int i = 0; i < RM; ++i) {
            const uint32_t r = i * 16 + lane % 16;
            a[i] = g.a + (int64_t)source_row(g, m0 + (r < high ? r : high - 1)) * g.lda + at;
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) {
            const uint32_t c = j * 16 + lane % 16;
            b[j] = g.b + (int64_t)t.group * g.b_stride +
                   (int64_t)(n0 + (c < wide ? c : wide - 1)) * g.ldb + at;
        }
        struct Piece {
            u32x4 a[RM][2], b[FN][2];
        };
        // whole: the piece's 128 bytes lie in the rows
        auto fetch = [&](Piece &p, uint32_t from, auto whole) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t f = from + h * 64;
                const int left = (int)g.bytes - (int)(f + at);
                auto one = [&](const char *q) {
                    if constexpr (decltype(whole)::value) return load_any<u32x4>(q);
                    else return load16<T>(q, left, g.bytes >= 16);
                };
#pragma unroll
                for (int j = 0; j < FN; ++j) p.b[j][h] = one(b[j] + f);
#pragma unroll
                for (int i = 0; i < RM; ++i) p.a[i][h] = one(a[i] + f);
            }
        };
        auto multiply = [&](const Piece &p) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < RM; ++i)
#pragma unroll
                    for (int j = 0; j < FN; ++j)
                        acc[i][j] = Mma<T>::run(__builtin_bit_cast(Frag, p.b[j][h]),
                                                __builtin_bit_cast(Frag, p.a[i][h]), acc[i][j]);
        };
        constexpr uint32_t kTurn = 4 * kStepBytes;
        uint32_t from = wave * kStepBytes;
        // DEEP pieces in flight while the DEEP before them are multiplied
        const uint32_t mine = g.bytes > from ? (g.bytes - from + kTurn - kStepBytes) / kTurn : 0;
        uint32_t left = mine / DEEP * DEEP;  // whole pieces of this wave, in groups
        Piece p[DEEP];
        if (left) {
#pragma unroll
            for (int d = 0; d < DEEP; ++d) fetch(p[d], from + d * kTurn, std::true_type());
            from += DEEP * kTurn;
            for (left -= DEEP; left; left -= DEEP) {
#pragma unroll
                for (int d = 0; d < DEEP; ++d) {
                    multiply(p[d]);
                    fetch(p[d], from + d * kTurn, std::true_type());
                }
                from += DEEP * kTurn;
            }
#pragma unroll
            for (int d = 0; d < DEEP; ++d) multiply(p[d]);
        }
        for (; from < g.bytes; from += kTurn) {
            fetch(p[0], from, std::false_type());
            multiply(p[0]);
        }
    }
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) sums[wave][i * FN + j][lane] = acc[i][j];
    __syncthreads();
    for (uint32_t f = wave; f < RM * FN; f += 4) {
        Acc s = sums[0][f][lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) s = plus(s, sums[w][f][lane]);
        const uint32_t r = f / FN * 16 + lane % 16, c = f % FN * 16 + lane / 16 * 4;
        if (r >= high || c >= wide) continue;
        const int left = (int)(wide - c);
        typedef O O4 __attribute__((ext_vector_type(4)));
        float v[4];
        if constexpr (sizeof(T) == 1) {
            const RowScale sa = RowScale::of(real ? g.sa[source_row(g, m0 + r)] : 0.f);
            if (g.bytes == EXPERTS_MAX_WIDTH) unwrap(s);
#pragma unroll
            for (int q = 0; q < 4; ++q)
                v[q] = real && q < left
                           ? sa(s[q], g.sb[(uint64_t)t.group * g.cols + n0 + c + q])
                           : 0.f;
        } else {
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] = s[q];
        }
        O *out = (O *)(g.out + (int64_t)(m0 + r) * g.ldo) + n0 + c;
        const O4 o = {(O)v[0], (O)v[1], (O)v[2], (O)v[3]};
        if (left >= 4) {
            store_any(out, o);
        } else {
#pragma unroll
            for (int q = 0; q < 3; ++q)
                if (q < left) out[q] = o[q];
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

// Blocks for `tiles` tiles, in runs of 8 * span, and the span.
inline uint64_t blocks_for(uint64_t tiles, uint32_t *span)
{
    *span = span_of(tiles);
    return (tiles + 8 * *span - 1) / (8 * *span) * (8 * *span);
}

inline bool aligned16(const void *p, int64_t ld_bytes)
{
    return !misaligned(p, 16) && ld_bytes % 16 == 0;
}

template <class T, class O, bool ACROSS, bool DIRECT, class S>
hist_status_t launch_tiles(RowsArgs g, hipStream_t stream)
{
    constexpr uint32_t kLds = S::STAGES * RowsParts<T, S, ACROSS>::STAGE;
    static_assert(S::PER_CU * kLds <= kLdsOfCu, "workgroups that a CU holds at one time");
    static_assert(S::BM * S::BN * sizeof(O) <= kLds, "results on their way to memory");
    g.n_tiles = (g.cols + S::BN - 1) / S::BN;
    const uint64_t tiles =
        most_row_tiles(g.rows, g.offsets ? g.experts + 1 : 1, S::BM) * g.n_tiles;
    // (and a workgroup more for each tile of a last round that is at most half full)
    const uint64_t blocks = blocks_for(tiles + (S::BM == 256 ? kCus / 2 : 0), &g.span);
    return launch(k_rows<T, O, S, ACROSS, DIRECT>, blocks, S::THREADS, kLds, stream, g);
}

// Whether `rows` rows from one base lie within 32-bit offsets.
inline bool near(uint64_t rows, int64_t ld_bytes)
{
    return rows * (uint64_t)ld_bytes < ((uint64_t)1 << 32) - 256;
}

template <class T, class O, int RM, int FN, int DEEP>
hist_status_t launch_thin(RowsArgs g, hipStream_t stream)
{
    g.n_tiles = (g.cols + 16 * FN - 1) / (16 * FN);
    const uint64_t tiles =
        most_row_tiles(g.rows, g.offsets ? g.experts + 1 : 1, 16 * RM) * g.n_tiles;
    const uint64_t blocks = blocks_for(tiles, &g.span);
    return launch(k_rows_thin<T, O, RM, FN, DEEP>, blocks, 256, 0, stream, g);
}

// The kernel for a product of rows. What decides is the rows of an expert on average (the
// host knows no more) and whether the tiles are enough for 256 CUs. Measured with 32 experts of
// 2560 x 2048 whose weights come from memory (bf16, us; thin 16 x 16, then tiles with the
// stages and workgroups that are used):
//              thin   32x128  64x128 128x128 128x256 256x256
//   rows   2   47.8     62.7    63.5    76.6            91.9
//   rows   8   72.3     73.0    73.4    93.0             112
//   rows  16    107     71.7    76.4    93.8    91.5     107
//   rows  32    179     73.6    76.5    94.9    92.5     108
//   rows  64    313     90.4    80.9     102    94.9     115
//   rows 128    593      128     103     101    94.1     113
//   rows 192    873      170     125     124     113     119
//   rows 256   1145      210     154     144     136     125
// The tiles below 256 x 256 are for groups whose time is the reading of the weights: more
// stages, so that more of it is in flight (64 rows, 64 x 128: 97 us with two stages and three
// workgroups a CU). Few tiles, a dense weight of 8192 x 4096 in 8 bits (64x64, 64x128, 128x128,
// 256x256): rows 256: 20.0, 19.3, 27.6, 38.8; rows 512: 32.5, 28.7, 30.1, 40.0; rows 1024: 54.8,
// 47.9, 40.0, 43.5; and thin 32 x 64 against 64 x 64: rows 32: 18.6, 20.5; rows 64: 18.9, 20.8.
enum class RowsKernel {
    kThin16, kThin32,                                                           // divided reduction
    k256x256, k128x256, k128x128Alone, k128x128, k64x128, k32x128, k32x128Short, k64x64,  // direct
    kVia256x128, kVia128x128, kVia64x64, kVia32x128                             // through registers
};

template <bool ACROSS>
RowsKernel rows_kernel(const RowsArgs &g)
{
    typedef RowsKernel K;
    const uint64_t groups = g.offsets ? g.experts : 1, each = g.rows / groups;
    // about so many: half a tile of each group is empty
    auto tiles = [&](uint32_t bm, uint32_t bn) {
        const uint64_t m = groups == 1 ? (each + bm - 1) / bm : g.rows / bm + (groups + 1) / 2;
        return (m < g.rows ? m : g.rows) * ((g.cols + bn - 1) / bn);
    };
    // The thin kernels divide the reduction among waves, the others do not, so the choice between
    // them does not depend on alignment: a product's bits are the same at every address.
    if (!ACROSS) {
        if (each <= 6) return K::kThin16;
        if (tiles(64, 64) < (each <= 64 ? 256 : 128)) return K::kThin32;
    }
    if (aligned16(g.a, g.lda) && aligned16(g.b, g.ldb) && g.b_stride % 16 == 0 &&
        g.bytes % 16 == 0 && (!ACROSS || g.cols % 8 == 0) &&
        near(g.order ? g.a_rows : 256, g.lda) && near(256, g.ldb)) {
        // a short reduction has no use for stages, but for workgroups beside it (16384 rows, 8 experts,
        // 256 -> 2048: 31 us in 128 x 128, 37 in 256 x 256; 1024 -> 2048: 78 and 80)
        const bool brief = g.bytes <= 8 * kStepBytes;
        if (!brief && each >= 224 && g.cols > 128 && tiles(256, 256) >= 256) return K::k256x256;
        if (!brief && each >= 80 && g.cols > 128 && tiles(128, 256) >= 384) return K::k128x256;
        // a workgroup on each CU at most: stages instead of a second one (8 bits, 8192 x 4096, 512
        // rows: 25 us, with two stages 30)
        const uint64_t small = tiles(128, 128), large = tiles(256, 256);
        if (each >= 80 && small >= 128 && small <= 256) return K::k128x128Alone;
        // A few tiles more than the 512 that run at one time take as long as a round of them (the
        // count is an estimate, hence 528): large tiles, if one round of those fills most CUs. 16
        // experts, 175 rows each, 2688 x 4096: 111 us, with small tiles 147; 32 experts, 138 rows
        // each, 1344 x 2048: 60 and 75 us, but with 128 rows each, in one round, 59 and 53. (The host
        // does not know the routing, so sizes near the edge fall on either side of a round.)
        if (each >= 80 && small > 528 && small % 512 < 128 && large >= 160 && large <= 256 && !brief)
            return K::k256x256;
        if (each >= 80 && small >= 256) return K::k128x128;
        if (each > 40 && (ACROSS || tiles(64, 128) >= 256)) return K::k64x128;
        if (ACROSS || (each <= 40 && tiles(32, 128) >= 256))
            return brief ? K::k32x128Short : K::k32x128;
        return K::k64x64;
    }
    // Through registers. A load that is not aligned takes the CU's path to its cache twice, so a tile
    // that loads less for its products counts for more: 16 experts of 1024 rows on average, 2560 x
    // 2053, 256 x 128 against 128 x 128: 286 and 302 us, the gradient of the rows 231 and 267.
    if (each >= 192 && tiles(256, 128) >= 256) return K::kVia256x128;
    if (each >= 80 && tiles(128, 128) >= 256) return K::kVia128x128;
    return ACROSS ? K::kVia32x128 : K::kVia64x64;
}

// What a kernel is made for: a shape of tiles, or the thin kernel's parameters.
template <class S, bool DIRECT> struct Tiles {};
template <int RM, int FN, int DEEP> struct Thin {};

// Calls f with what the kernel is made for.
template <bool ACROSS, class F>
hist_status_t with_rows_kernel(RowsKernel kernel, const F &f)
{
    typedef RowsKernel K;
    // A stage with weights across the reduction takes 21 KiB of LDS, along it 20, so the gradient of
    // the rows has a stage, or a workgroup, less (32 experts, 2560 -> 2048: 2 to 32 rows an expert
    // 62-64 us, 5.2-5.4 TB/s of weights, 40 rows 78; a fourth stage, which leaves one workgroup on
    // a CU, 62-66 and 82; 1344 -> 2048: 33-34 and 34-36. 64 rows, 64 x 128: 67 us).
    typedef typename std::conditional<ACROSS, Shape<32, 128, 2, 2, 2, 3>,
                                      Shape<32, 128, 1, 4, 2, 4>>::type Lowest;
    typedef typename std::conditional<ACROSS, Shape<32, 128, 2, 2, 3>,
                                      Shape<32, 128, 1, 4, 4>>::type LowestShort;
    switch (kernel) {
    case K::k256x256: return f(Tiles<Shape<256, 256, 2, 4, 1>, true>());
    case K::k128x256: return f(Tiles<Shape<128, 256, 2, 4, 1, 3>, true>());
    case K::k128x128Alone: return f(Tiles<Shape<128, 128, 4, 2, 1, 4>, true>());
    case K::k128x128: return f(Tiles<Shape<128, 128, 2, 2, 2>, true>());
    case K::k64x128: return f(Tiles<Shape<64, 128, 2, 2, 2, 3>, true>());
    case K::k32x128: return f(Tiles<Lowest, true>());
    case K::k32x128Short: return f(Tiles<LowestShort, true>());
    case K::kVia256x128: return f(Tiles<Shape<256, 128, 4, 2, 1>, false>());
    case K::kVia128x128: return f(Tiles<Shape<128, 128, 2, 2, 2>, false>());
    default: break;
    }
    if constexpr (ACROSS) {
        return f(Tiles<Shape<32, 128, 2, 2, 3>, false>());
    } else {
        switch (kernel) {
        case K::kThin16: return f(Thin<1, 1, 4>());
        case K::kThin32: return f(Thin<2, 4, 2>());
        case K::k64x64: return f(Tiles<Shape<64, 64, 2, 2, 3, 3>, true>());
        default: return f(Tiles<Shape<64, 64, 2, 2, 3>, false>());
        }
    }
}

template <class T, class O, bool ACROSS>
struct LaunchRows {
    const RowsArgs &g;
    hipStream_t stream;
    template <class S, bool DIRECT>
    hist_status_t operator()(Tiles<S, DIRECT>) const
    {
        return launch_tiles<T, O, ACROSS, DIRECT, S>(g, stream);
    }
    template <int RM, int FN, int DEEP>
    hist_status_t operator()(Thin<RM, FN, DEEP>) const
    {
        return launch_thin<T, O, RM, FN, DEEP>(g, stream);
    }
};

template <class T, class O, bool ACROSS>
hist_status_t launch_rows(const RowsArgs &g, hipStream_t stream)
{
    return with_rows_kernel<ACROSS>(rows_kernel<ACROSS>(g), LaunchRows<T, O, ACROSS>{g, stream});
}

template <class T, bool DIRECT, class S>
hist_status_t launch_dw_tiles(DwArgs g, hipStream_t stream)
{
    constexpr uint32_t kLds = 2 * DwParts<T, S>::STAGE;
    static_assert(S::PER_CU * kLds <= kLdsOfCu, "workgroups that a CU holds at one time");
    static_assert(S::BM * S::BN * sizeof(T) <= kLds, "results on their way to memory");
    g.n_tiles = (g.n + S::BM - 1) / S::BM;
    g.k_tiles = (g.k + S::BN - 1) / S::BN;
    const uint64_t blocks = blocks_for((uint64_t)g.n_tiles * g.k_tiles * g.experts, &g.span);
    return launch(k_dw<T, S, DIRECT>, blocks, S::THREADS, kLds, stream, g);
}

enum class DwKernel { k256x256, k128x128, kVia256x128, kVia128x128 };

inline DwKernel dw_kernel(const DwArgs &g)
{
    typedef DwKernel K;
    auto tiles = [&](uint32_t bm, uint32_t bn) {
        return (uint64_t)g.experts * ((g.n + bm - 1) / bm) * ((g.k + bn - 1) / bn);
    };
    if (aligned16(g.dy, g.lddy) && aligned16(g.x, g.ldx) && g.n % 8 == 0 && g.k % 8 == 0 &&
        near(64, g.lddy) && near(g.x_rows, g.ldx)) {
        // Large tiles, if they are enough for most of 256 CUs and not much larger than the weight,
        // whatever the rows an expert, for which there are no measurements (32
        // experts, 1024 rows each, 528 x 288: 53 us, in small ones 34; 1024 x 1024: 98 and 111).
        const uint64_t area = tiles(256, 256) * 256 * 256;
        return tiles(256, 256) >= 176 && area * 4 <= tiles(128, 128) * 128 * 128 * 5 ? K::k256x256
                                                                                    : K::k128x128;
    }
    // (the same sizes: 404 and 516 us)
    return tiles(256, 128) >= 256 ? K::kVia256x128 : K::kVia128x128;
}

template <class F>
hist_status_t with_dw_kernel(DwKernel kernel, const F &f)
{
    switch (kernel) {
    case DwKernel::k256x256: return f(Tiles<Shape<256, 256, 2, 4, 1>, true>());
    case DwKernel::k128x128: return f(Tiles<Shape<128, 128, 2, 2, 2>, true>());
    case DwKernel::kVia256x128: return f(Tiles<Shape<256, 128, 4, 2, 1>, false>());
    default: return f(Tiles<Shape<128, 128, 2, 2, 2>, false>());
    }
}

template <class T>
struct LaunchDw {
    const DwArgs &g;
    hipStream_t stream;
    template <class S, bool DIRECT>
    hist_status_t operator()(Tiles<S, DIRECT>) const
    {
        return launch_dw_tiles<T, DIRECT, S>(g, stream);
    }
};

template <class T>
hist_status_t launch_dw(const DwArgs &g, hipStream_t stream)
{
    return with_dw_kernel(dw_kernel(g), LaunchDw<T>{g, stream});
}

// Fills in the answer of experts_product_preview.
struct DescribeKernel {
    experts_kernel_t *kernel;
    template <class S, bool DIRECT>
    hist_status_t operator()(Tiles<S, DIRECT>) const
    {
        *kernel = {S::BM, S::BN, S::THREADS, S::STAGES, S::PER_CU, DIRECT};
        return HIST_OK;
    }
    template <int RM, int FN, int DEEP>
    hist_status_t operator()(Thin<RM, FN, DEEP>) const
    {
        *kernel = {16 * RM, 16 * FN, 256, 0, 0, 0};
        return HIST_OK;
    }
};

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
    if (experts > EXPERTS_MAX_EXPERTS || top_k > EXPERTS_MAX_TOP_K || n > EXPERTS_MAX_WIDTH ||
        k > EXPERTS_MAX_WIDTH || rows > EXPERTS_MAX_ROWS || x_rows > EXPERTS_MAX_ROWS)
        return HIST_ERR_UNSUPPORTED;
    return HIST_OK;
}

}  // namespace pca_experts
