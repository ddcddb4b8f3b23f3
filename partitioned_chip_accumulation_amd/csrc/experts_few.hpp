// experts_few.hpp -- a whole expert layer for a few tokens: the kernels of experts_few_tokens and how
// they are launched. Part of libpca_hist.so.
//
//   h[t, e] = act(x[t] up[e]^T),  out[t] = sum over t's experts e of weight[t, e] h[t, e] down[e]^T
//
// Bound by reading the weights of the experts that have a token, once each: one token, 8 experts of 2048 and
// 2 x 1280 columns in bf16 (126 MB) 34.5 us, the kernels' medians 21.6 and 15.9 (traced); four in 8 bits 51; 16
// tokens, 4 of 32 experts of 2048 and 2 x 2560 in 4 bits 71; 63 tokens, 2 of 32 experts of 2048 and 1344 in fp16
// 80 (of 2050 and 1337, rows at odd addresses, 107). Two kernels: the first takes an expert's 16 FN columns of h
// a workgroup, the second 16 FN columns of the result, with the products of all experts added up in registers.
// Both find the experts from the ids by themselves, so nothing is sorted, counted or copied before, and the host
// needs to know nothing of the routing.
//
// The fragments of the matrix instructions come from memory to registers: a lane's 16 bytes of a
// weight's row, 8, 16 or 32 values, are widened to the tokens' type there (exact: 8-bit whole numbers
// and 4-bit values times a power of two have 8 bits at most), so that what is read is what the weights
// take. h is held in 32 bits between the two products, whatever the types, and all 24 of its bits are multiplied.
#pragma once

#include "experts_tile.hpp"

namespace pca_experts {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kHalf = 64;  // bytes of a row that one load of a wave takes
constexpr uint32_t kStep = 2 * kHalf;  // what the second kernel's waves share out

struct FewWeight {
    const char *data;
    const char *scales;  // float [experts][rows], or powers of two
    int64_t ld, stride, ld_scales, scales_stride;  // bytes
    uint32_t window;                               // bytes of an expert's powers of two
};

struct FewArgs {
    char *out;
    const char *x;
    char *h;            // (see Rows)
    uint32_t *arrived;  // [tiles of the result]
    uint32_t *partial;
    FewWeight up, down;
    const void *ids;
    const float *by;
    int64_t ldo, ldx, ldh;  // bytes
    uint32_t ids64, gated, h_shift, tokens, top_k, experts, width, hidden, n;
    uint32_t tiles, groups, parts;  // of the result; workgroups, and the most of them that share a tile
    // (a kernel's first loads wait for its divisions)
    Divide by_top_k, by_up_tiles, by_tiles, by_groups, by_waves, by_steps;
};

// The upper halves of values of 32 bits, two in a word.
template <int N>
__device__ __forceinline__ uint32_t __attribute__((ext_vector_type(N / 2)))
upper(float __attribute__((ext_vector_type(N))) v)
{
    uint32_t __attribute__((ext_vector_type(N / 2))) two;
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
        two[i] = __builtin_amdgcn_perm(__float_as_uint(v[2 * i + 1]), __float_as_uint(v[2 * i]), 0x07060302);
    return two;
}

// How weights of type W go with tokens of type T, C fragments of a lane's 16 bytes, and with h, which is in
// 32 bits: kParts if they are bfloat16 values exactly (part), which meet the three parts of h; float16 ones are
// widened (wide) for the matrix instruction of 32-bit values, a sixteenth as fast. us in parts and that way: four
// tokens in 8 bits 57 and 61, sixteen in 4 bits 74 and 94, in bf16 89 and 92. (float16 weights in two parts of
// their own: 78 instead of 81 for 63 tokens of 2048 and 1344 columns, 111 instead of 107 of 2050 and 1337.)
template <class T, class W> struct Widen;
template <class T> struct Widen<T, T> {
    static constexpr int C = 1;
    static constexpr bool kParts = std::is_same<T, __bf16>::value;
    typedef typename Vec8<T>::type Frag;
    static __device__ __forceinline__ Frag frag(u32x4 v, int, uint32_t)
    {
        return __builtin_bit_cast(Frag, v);
    }
    static __device__ __forceinline__ void add(Frag w, u32x4 a, f32x4 &acc)
    {
        acc = Mma<T>::run(w, __builtin_bit_cast(Frag, a), acc);
    }
    static __device__ __forceinline__ bf16x8 part(u32x4 v, int, uint32_t)
    {
        return __builtin_bit_cast(bf16x8, v);
    }
    static __device__ __forceinline__ f32x8 wide(u32x4 v, int)
    {
        const Frag w = __builtin_bit_cast(Frag, v);
        f32x8 f;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = (float)w[i];
        return f;
    }
};
template <class T> struct Widen<T, int8_t> {
    static constexpr int C = 2;
    static constexpr bool kParts = true;
    typedef typename Vec8<T>::type Frag;
    static __device__ __forceinline__ Frag frag(u32x4 v, int c, uint32_t)
    {
        const f32x8 w = wide(v, c);
        if constexpr (std::is_same<T, __bf16>::value) {
            return __builtin_bit_cast(Frag, upper<8>(w));  // (8 bits: exact)
        } else {
            Frag f;
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = (T)w[i];
            return f;
        }
    }
    static __device__ __forceinline__ void add(Frag w, u32x4 a, f32x4 &acc)
    {
        acc = Mma<T>::run(w, __builtin_bit_cast(Frag, a), acc);
    }
    static __device__ __forceinline__ bf16x8 part(u32x4 v, int c, uint32_t power)
    {
        return Widen<__bf16, int8_t>::frag(v, c, power);
    }
    static __device__ __forceinline__ f32x8 wide(u32x4 v, int c)
    {
        f32x8 f;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = (float)((int32_t)(v[c * 2 + i / 4] << (24 - i % 4 * 8)) >> 24);
        return f;
    }
};
// A block's values as bfloat16, whose exponents reach as far as the powers of two.
template <class T> struct Widen<T, Mx4> {
    static constexpr int C = 4;
    static constexpr bool kParts = true;
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
    static __device__ __forceinline__ bf16x8 part(u32x4 v, int c, uint32_t power)
    {
        return frag(v, c, power);
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

// A value of 32 bits is the sum of three bfloat16 ones: its upper 16 bits, those of what is left, and what
// is left then (8 of the 24 bits each). An infinity leaves NaN: its first part alone counts.
template <int N>
struct Parts {
    typedef __bf16 Part __attribute__((ext_vector_type(N)));
    Part part[3];
    __device__ __forceinline__ Parts(float __attribute__((ext_vector_type(N))) v)
    {
#pragma unroll
        for (int p = 0; p < 3; ++p) {
            part[p] = __builtin_bit_cast(Part, upper<N>(v));
#pragma unroll
            for (int i = 0; i < N; ++i)
                v[i] -= __uint_as_float(__float_as_uint(v[i]) & 0xffff0000u);
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
// The routing. A slot is what there is to do for one expert and up to kRows pairs of it, in their order.
// Up to 64 pairs are a wave's registers: every wave finds its slots by itself, without LDS and barriers,
// in the order of the experts' first pairs. More pairs go through LDS, where the slots come in the order of
// the experts' numbers.
struct Routes {
    uint32_t many[EXPERTS_MAX_EXPERTS];  // pairs of each expert; then of those before it
    uint32_t count;
    // expert, and which kRows of its pairs << 16 (there are as many as experts, and one more for each 16 of
    // the other pairs)
    uint32_t list[EXPERTS_MAX_EXPERTS + EXPERTS_MAX_FEW * EXPERTS_MAX_TOP_K / 16];
};
extern __shared__ __align__(16) char few_lds[];  // int16_t ids[pairs], float by[pairs], then the sums

__device__ __host__ __forceinline__ uint32_t ids_bytes(uint32_t pairs)
{
    return (pairs * 2 + 15) / 16 * 16;
}
__device__ __host__ __forceinline__ uint32_t by_bytes(uint32_t pairs)
{
    return (pairs * 4 + 15) / 16 * 16;
}

template <uint32_t kRows, bool BY>
struct Router {
    Routes &routes;
    const uint32_t pairs;
    uint32_t count;  // slots
    // of pair number lane, of up to 64
    int id;
    float by;
    uint32_t rank;    // pairs of the expert before it
    uint64_t same;    // its pairs
    uint64_t starts;  // the lanes that a slot begins with, the same for all

    __device__ __forceinline__ int16_t *lds_ids() const { return (int16_t *)few_lds; }
    __device__ __forceinline__ float *lds_by() const { return (float *)(few_lds + ids_bytes(pairs)); }

    __device__ __forceinline__ Router(const FewArgs &g, Routes &r)
        : routes(r), pairs(g.tokens * g.top_k)
    {
        auto id_of = [&](uint32_t i) {
            const int64_t id = g.ids64 ? ((const int64_t *)g.ids)[i] : ((const int32_t *)g.ids)[i];
            return (uint64_t)id < g.experts ? (int)id : -1;
        };
        const uint32_t lane = threadIdx.x % 64;
        if (pairs <= 64) {
            id = lane < pairs ? id_of(lane) : -1;
            by = BY && lane < pairs ? g.by[lane] : 0.f;
            same = __ballot(id >= 0);
#pragma unroll
            for (int bit = 0; (1u << bit) < EXPERTS_MAX_EXPERTS; ++bit) {
                const uint64_t set = __ballot(id >> bit & 1);
                same &= id >> bit & 1 ? set : ~set;
            }
            rank = (uint32_t)__popcll(same & ((1ull << lane) - 1));
            starts = __ballot(id >= 0 && rank % kRows == 0);
            count = (uint32_t)__popcll(starts);
            return;
        }
        for (uint32_t e = threadIdx.x; e < g.experts; e += blockDim.x) routes.many[e] = 0;
        __syncthreads();
        for (uint32_t i = threadIdx.x; i < pairs; i += blockDim.x) {
            const int e = id_of(i);
            lds_ids()[i] = (int16_t)e;
            if constexpr (BY) lds_by()[i] = g.by[i];
            if (e >= 0) lds_add(routes.many, (uint32_t)e, 1);
        }
        __syncthreads();
        if (threadIdx.x < 64) {
            const uint32_t each = (g.experts + 63) / 64, first = lane * each;
            uint32_t mine = 0, of = 0;
            for (uint32_t e = first; e < first + each && e < g.experts; ++e) {
                mine += (routes.many[e] + kRows - 1) / kRows;
                of += routes.many[e];
            }
            const uint32_t upto = wave_inclusive_scan(mine);
            uint32_t at = upto - mine, before = wave_inclusive_scan(of) - of;
            for (uint32_t e = first; e < first + each && e < g.experts; ++e) {
                const uint32_t many = routes.many[e];
                for (uint32_t q = 0; q * kRows < many; ++q) routes.list[at++] = e | q << 16;
                routes.many[e] = before;
                before += many;
            }
            if (lane == 63) routes.count = upto;
        }
        __syncthreads();
        count = __builtin_amdgcn_readfirstlane(routes.count);
    }

    // The expert of a slot, its pairs to `rows` (the wave's own kRows places) and how many pairs the experts
    // and slots before it have; returns how many it has.
    __device__ __forceinline__ uint32_t find(uint32_t slot, uint16_t *rows, uint32_t &expert,
                                             uint32_t &before) const
    {
        const uint32_t lane = threadIdx.x % 64;
        const uint64_t below = (1ull << lane) - 1;
        uint32_t seen = 0;
        if (pairs <= 64) {
            const bool here = starts >> lane & 1 && (uint32_t)__popcll(starts & below) == slot;
            const int at = __builtin_ctzll(__ballot(here));
            expert = __builtin_amdgcn_readlane(id, at);
            const uint32_t first = __builtin_amdgcn_readlane(rank, at);
            const bool mine = id == (int)expert && rank - first < kRows;
            if (mine) rows[rank - first] = (uint16_t)lane;
            seen = (uint32_t)__popcll(__ballot(mine));
            // (the experts' order is that of their first pairs)
            const int own = __builtin_ctzll(same | 1ull << 63);
            before = first + (uint32_t)__popcll(
                                 __ballot(id >= 0 && own < __builtin_amdgcn_readlane(own, at)));
        } else {
            const uint32_t what = __builtin_amdgcn_readfirstlane(routes.list[slot]);
            const uint32_t skip = (what >> 16) * kRows;
            expert = what & 0xffff;
            before = __builtin_amdgcn_readfirstlane(routes.many[expert]) + skip;
            for (uint32_t i = 0; i < pairs && seen < skip + kRows; i += 64) {
                const bool here = i + lane < pairs && lds_ids()[i + lane] == (int)expert;
                const uint64_t mask = __ballot(here);
                const uint32_t at = seen + (uint32_t)__popcll(mask & below) - skip;
                if (here && at < kRows) rows[at] = (uint16_t)(i + lane);
                seen += (uint32_t)__popcll(mask);
            }
            seen -= skip;
            seen = seen < kRows ? seen : kRows;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        return seen;
    }

    // The weight of a pair; of lanes that are all active.
    __device__ __forceinline__ float weight(uint32_t pair) const
    {
        if (pairs <= 64) return __shfl(by, pair, 64);
        return lds_by()[pair];
    }
};

// ---------------------------------------------------------------------------
// Memory that a kernel reads through a descriptor: at a lane's place, plus the wave's. Of a lane whose own
// place lies past the end nothing is loaded, and it gets zeros. kNowhere plus any place in a row is past
// every end.
struct Window {
    __amdgpu_buffer_rsrc_t rsrc;
    static constexpr uint32_t kNowhere = 1u << 31, kMost = kNowhere - 1;
    __device__ __forceinline__ Window(const char *base, uint32_t bytes)
        : rsrc(__builtin_amdgcn_make_buffer_rsrc((void *)base, 0, bytes, 0x00027000))
    {
    }
    // The rows of a matrix from one on: `rows` of them, `bytes` each.
    static __device__ __forceinline__ Window rows(const char *base, int64_t ld, uint32_t rows,
                                                  uint32_t bytes)
    {
        const int64_t all = (int64_t)(rows - 1) * ld + bytes;
        return Window(base, all < kMost ? (uint32_t)all : kMost);
    }
    __device__ __forceinline__ u32x4 load16(uint32_t place, uint32_t wave) const
    {
        return __builtin_bit_cast(
            u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, (int)place, (int)wave, 0));
    }
    template <int BYTES>
    __device__ __forceinline__ uint64_t load(uint32_t place, uint32_t wave) const
    {
        if constexpr (BYTES == 4)
            return (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(rsrc, (int)place, (int)wave, 0);
        else
            return __builtin_bit_cast(
                uint64_t, __builtin_amdgcn_raw_buffer_load_b64(rsrc, (int)place, (int)wave, 0));
    }
};

// What one step of a wave multiplies: kHalves times 64 bytes of each of 16 FB rows of a weight, and
// what goes with them of 16 RM rows of tokens. (Two halves are whole cache lines; with one, each line is
// asked for twice.)
//
// Neighbouring lanes hold neighbouring rows, so every lane is an access of its own to the CU's cache,
// which takes one a cycle: the 64 for each KB of weights leave room for 40 more at 5.5 TB/s. So lanes of
// rows without a token load nothing (with their rows loaded like others, 4-bit weights, four loads of tokens
// for one of theirs, were read at 3.0 TB/s), and 16 lanes load a step's powers of two for all.
//
// No load of a weight leaves its row: at the row's end a lane's 16 bytes are the last ones of the row,
// to be shifted (mend) before they are multiplied. The code is kept short: a pass over other experts' weights
// leaves none of it in the caches, and kernels of 50 KB took 8 us for next to no work.
//
// The tokens' rows can be those of h, which lie as Rows has them: the 32 bytes of a row that go with a fragment
// are two words of a lane, or (kFolded) words of two lanes, so that one load has those of up to 8 pairs, the
// second ones in the rows after the first ones. Then each matrix instruction takes all rows with half of a
// fragment, and its sums count in the rows that this half belongs to (four tokens in 8 bits 54 us instead of 57,
// one in 16 bits 34.6 instead of 35.5).
enum Tokens { kOfX, kOfH, kFolded };
template <class T, class W, int RM, int FB, Tokens OF = kOfX>
struct Piece {
    typedef Widen<T, W> By;
    static constexpr int C = By::C;
    static constexpr int kWords = OF == kOfH ? 2 : 1;  // 16-byte words of a lane that go with a fragment
    static constexpr int kHalves = RM * C * kWords > 4 ? 1 : 2;  // (as registers allow)
    // Sums of the words' products; in parts, those of the first part and then those of the others.
    static constexpr int kOfWords = OF == kFolded ? 2 : 1;
    static constexpr int kSums = OF != kOfX && By::kParts ? 2 * kOfWords : kOfWords;
    static constexpr uint32_t kBytes = kHalf * kHalves, kValues = kBytes / 16 * C * 8;  // of a row
    static constexpr bool kPowers = std::is_same<W, Mx4>::value;
    static constexpr uint32_t kStepPowers = kBytes / 16;
    u32x4 b[FB][kHalves], a[RM][kHalves][C][kWords];
    uint64_t power[kPowers ? FB : 1];  // of a step's blocks, in lanes below 16

    static __device__ __host__ __forceinline__ uint32_t steps(uint32_t k)
    {
        return (row_bytes<W>(k) + kBytes - 1) / kBytes;
    }
    // Whether the rows end within their last step.
    static __device__ __forceinline__ bool ragged(uint32_t k) { return k % kValues != 0; }
    // The places in a row of this lane's 16 bytes of b, and of its values c of a.
    static __device__ __forceinline__ uint32_t place_b(uint32_t step, int h)
    {
        return step * kBytes + h * kHalf + threadIdx.x % 64 / 16 * 16;
    }
    static __device__ __forceinline__ uint32_t place_a(uint32_t step, int h, int c)
    {
        return (step * kValues + (h * 4 + threadIdx.x % 64 / 16) * C * 8 + c * 8) * 2;
    }
    // The place of a step's powers; those of the last step end with the row.
    static __device__ __forceinline__ uint32_t place_p(uint32_t step, uint32_t blocks)
    {
        const uint32_t most = blocks < kStepPowers ? 0 : blocks - kStepPowers;
        return step * kStepPowers < most ? step * kStepPowers : most;
    }

    // What the pieces of a wave are loaded from: windows, and this lane's places in them.
    struct Source {
        const Window &tokens, &first, &second;  // b's fragments below FB / 2 (or 1) lie in the first
        const Window &powers;
        uint32_t a[RM], b[FB], p[FB];  // of rows; kNowhere: none
        uint32_t unit;                 // of h: bytes of the words of all its rows
        __device__ __forceinline__ const Window &of(int j) const
        {
            return j < (FB + 1) / 2 ? first : second;
        }
    };

    __device__ __forceinline__ void fetch(const Source &s, uint32_t step)
    {
        const uint32_t lane = threadIdx.x % 64 / 16;
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int j = 0; j < FB; ++j)
                b[j][h] = s.of(j).load16(s.b[j] + lane * 16 + h * kHalf, step * kBytes);
        if constexpr (kPowers)
#pragma unroll
            for (int j = 0; j < FB; ++j)
                power[j] = s.powers.template load<kStepPowers>(s.p[j], step * kStepPowers);
        if constexpr (OF != kOfX) return fetch_h(s, step);
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < RM; ++i)
                    a[i][h][c][0] = s.tokens.load16(
                        s.a[i] + lane * C * 16 + (h * 4 * C + c) * 16, step * kValues * 2);
    }
    __device__ __forceinline__ void fetch_h(const Source &s, uint32_t step)
    {
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < RM; ++i)
#pragma unroll
                    for (int q = 0; q < kWords; ++q)
                        a[i][h][c][q] = s.tokens.load16(
                            s.a[i], (((step * kHalves + h) * C + c) * kWords + q) * s.unit);
    }
    // The last step, of rows of k values.
    __device__ __forceinline__ void fetch_last(const Source &s, uint32_t step, uint32_t k)
    {
        const uint32_t bytes = row_bytes<W>(k);
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            const uint32_t at = place_b(step, h), in = at < bytes - 16 ? at : bytes - 16;
#pragma unroll
            for (int j = 0; j < FB; ++j) b[j][h] = s.of(j).load16(s.b[j] + in, 0);
        }
        if constexpr (kPowers)
#pragma unroll
            for (int j = 0; j < FB; ++j)
                power[j] = s.powers.template load<kStepPowers>(s.p[j] + place_p(step, bytes / 16), 0);
        if constexpr (OF != kOfX) return fetch_h(s, step);
        const uint32_t room = k * 2;
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const uint32_t at = place_a(step, h, c), in = at < room - 16 ? at : room - 16;
#pragma unroll
                for (int i = 0; i < RM; ++i) a[i][h][c][0] = s.tokens.load16(s.a[i] + in, 0);
            }
    }

    // Puts zeros for what lies past the rows' ends; step: the last one.
    __device__ __forceinline__ void mend_b(uint32_t step, uint32_t k, const char *powers,
                                           const uint32_t (&from_p)[FB])
    {
        const uint32_t bytes = row_bytes<W>(k), blocks = bytes / 16;
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            const int left = (int)bytes - (int)place_b(step, h);
#pragma unroll
            for (int j = 0; j < FB; ++j) {
                if constexpr (kPowers) b[j][h] = left > 0 ? b[j][h] : u32x4{};  // whole blocks
                else b[j][h] = drop16(b[j][h], left);
            }
        }
        if constexpr (kPowers)
#pragma unroll
            for (int j = 0; j < FB; ++j) {
                if (blocks >= kStepPowers) {
                    power[j] >>= (step * kStepPowers - place_p(step, blocks)) * 8;
                } else if (from_p[j] != Window::kNowhere) {  // a row of fewer than a step's
                    power[j] = 0;
#pragma unroll 1
                    for (uint32_t q = step * kStepPowers; q < blocks; ++q)
                        power[j] |= (uint64_t)(uint8_t)powers[from_p[j] + q]
                                    << (q - step * kStepPowers) * 8;
                }
            }
    }
    __device__ __forceinline__ void mend_a(uint32_t step, uint32_t room)
    {
#pragma unroll
        for (int h = 0; h < kHalves; ++h)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                const int left = (int)room - (int)place_a(step, h, c);
#pragma unroll
                for (int i = 0; i < RM; ++i) a[i][h][c][0] = drop16(a[i][h][c][0], left);
            }
    }

    // The power of this lane's block of b's fragment j.
    __device__ __forceinline__ uint32_t own_power(int j, int h) const
    {
        if constexpr (!kPowers) return 0;
        else {
            const uint32_t lane = threadIdx.x % 64;
            return __shfl((uint32_t)(power[j] >> h * 32), lane % 16, 64) >> lane / 16 * 8 & 0xff;
        }
    }
    __device__ __forceinline__ void multiply(f32x4 (&acc)[kSums][RM][FB]) const
    {
        if constexpr (OF != kOfX) return multiply_h(acc);
#pragma unroll
        for (int j = 0; j < FB; ++j)
#pragma unroll
            for (int h = 0; h < kHalves; ++h) {
                const uint32_t own = own_power(j, h);
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const auto w = By::frag(b[j][h], c, own);
#pragma unroll
                    for (int i = 0; i < RM; ++i) By::add(w, a[i][h][c][0], acc[0][i][j]);
                }
            }
    }
    __device__ __forceinline__ void multiply_h(f32x4 (&acc)[kSums][RM][FB]) const
    {
#pragma unroll
        for (int h = 0; h < kHalves; ++h) {
            uint32_t own[FB];
#pragma unroll
            for (int j = 0; j < FB; ++j) own[j] = own_power(j, h);
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int i = 0; i < RM; ++i) {
                    const auto v = words(i, h, c);
                    if constexpr (By::kParts) {
                        const Parts<4 * kWords> parts(v);
#pragma unroll
                        for (int j = 0; j < FB; ++j) {
                            const bf16x8 w = By::part(b[j][h], c, own[j]);
#pragma unroll
                            for (int p = 0; p < 3; ++p)
#pragma unroll
                                for (int q = 0; q < kOfWords; ++q) {
                                    f32x4 &to = acc[(p ? kOfWords : 0) + q][i][j];
                                    if constexpr (OF == kFolded)
                                        to = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(
                                            __builtin_bit_cast(s16x4, four(w, q)),
                                            __builtin_bit_cast(s16x4, parts.part[p]), to, 0, 0, 0);
                                    else
                                        to = Mma<__bf16>::run(w, parts.part[p], to);
                                }
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < FB; ++j) {
                            const f32x8 w = By::wide(b[j][h], c);
#pragma unroll
                            for (int q = 0; q < 8; ++q) {
                                f32x4 &to = acc[q / 4 * (kOfWords - 1)][i][j];
                                to = __builtin_amdgcn_mfma_f32_16x16x4f32(w[q], v[q % (4 * kWords)], to, 0, 0,
                                                                          0);
                            }
                        }
                    }
                }
        }
    }
    // What this lane has of h for a fragment.
    typedef float Words __attribute__((ext_vector_type(4 * kWords)));
    __device__ __forceinline__ Words words(int i, int h, int c) const
    {
        struct {
            u32x4 word[kWords];
        } v;
#pragma unroll
        for (int q = 0; q < kWords; ++q) v.word[q] = a[i][h][c][q];
        return __builtin_bit_cast(Words, v);
    }
    static __device__ __forceinline__ bf16x4 four(bf16x8 w, int q)
    {
        return q ? __builtin_shufflevector(w, w, 4, 5, 6, 7) : __builtin_shufflevector(w, w, 0, 1, 2, 3);
    }
};

// `mine` pieces (one or more), DEEP of them on their way while the ones before are multiplied. first
// fetches the first piece, and start is called for it when it is multiplied. fetch stays at the last one when
// it is asked for more: loads that come from the cache (or, of a ragged step, end with the window), in place
// of branches around loads, at which the compiler would wait for all of them.
template <int DEEP, class P, class O, class F, class S, class M>
__device__ __forceinline__ void pipeline(uint32_t mine, P (&p)[DEEP], O first, F fetch, S start,
                                         M multiply)
{
    first(p[0]);
#pragma unroll
    for (int d = 1; d < DEEP; ++d) fetch(p[d]);
    start(p[0]);
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

// Of `count` steps in a row, share number `at` of `of` (2^15 at most) begins here.
__device__ __forceinline__ uint32_t share(uint32_t count, uint32_t at, uint32_t of, Divide by)
{
    const uint32_t whole = by(count);
    return whole * at + by((count - whole * of) * at);
}

// h of a slot, in 32 bits. It lies in the order in which the second kernel's lanes take it: for each 64 bytes of
// a weight's row (32 columns, or 64 and 128 of narrower weights) and each 8 columns that a lane's 16 bytes of
// them go with, first four columns of each, the 16 bytes of every row for lanes 0 to 15, those for lanes 16 to
// 31, and so on, then the other four likewise: 16 rows are 1 KB in one piece, 16 accesses instead of 64.
struct Rows {
    char *const base;
    const uint32_t count, shift;  // 2^shift fragments of columns go with 16 bytes of a weight
    __device__ __forceinline__ Rows(const FewArgs &g, uint32_t before, uint32_t count)
        : base(g.h + (int64_t)before * g.ldh), count(count), shift(g.h_shift)
    {
    }
    // Few pairs are folded (see Piece): one after another, first all pairs' first four columns, then the others.
    __device__ __forceinline__ bool folded() const { return count <= 8; }
    __device__ __forceinline__ uint32_t unit() const { return count * (folded() ? 128 : 64); }
    // The place of a column of a pair.
    __device__ __forceinline__ float *at(uint32_t row, uint32_t c) const
    {
        const uint32_t fragment = (c >> (5 + shift) << shift) + (c >> 3 & ((1u << shift) - 1));
        const uint32_t lanes = c >> (3 + shift) & 3;
        const uint32_t word = c >> 2 & 1;
        const uint32_t in = folded() ? (lanes * 2 + word) * count + row : (word * 4 + lanes) * count + row;
        return (float *)(base + (fragment * 8 * count + in) * 16) + c % 4;
    }
    // Four columns, of which `left` exist.
    __device__ __forceinline__ void store(uint32_t row, uint32_t c, f32x4 v, uint32_t left) const
    {
        float *const to = at(row, c);
        if (left >= 4) {
            *(f32x4 *)to = v;
        } else {
#pragma unroll
            for (uint32_t q = 0; q < 3; ++q)
                if (q < left) to[q] = v[q];
        }
    }
    // The second kernel reads whole steps: what the rows have from column `hidden` to `end` is 0.
    __device__ __forceinline__ void clear(uint32_t hidden, uint32_t end) const
    {
        const uint32_t wide = end - hidden;
        for (uint32_t i = threadIdx.x; i < count * wide; i += blockDim.x)
            *at(i / wide, hidden + i % wide) = 0.f;
    }
};

// ---------------------------------------------------------------------------
// Columns of h for one expert, 16 FN of them with a gate (FN fragments of its rows, then FN of the
// others) and 32 FN without, its tokens 16 RM at a time. The four waves divide the reduction, they take
// the steps in turn (a wave for each 16 FN columns alone: 35 us instead of 33 for one token in 16 bits, 54
// instead of 49 for four in 8).
template <class T, class W, int RM, int FN, int DEEP>
__device__ __forceinline__ void up_rows(const FewArgs &g, uint32_t e, uint32_t n0,
                                        const uint16_t *rows, const Rows &h, f32x4 *sums)
{
    constexpr int FB = 2 * FN;
    typedef Piece<T, W, RM, FB> P;
    const uint32_t count = h.count;
    const uint32_t lane = threadIdx.x % 64, at = lane / 16;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const char *const base = g.up.data + (int64_t)e * g.up.stride + (int64_t)n0 * g.up.ld;
    const char *const scales = g.up.scales + (int64_t)e * g.up.scales_stride;
    const Window tokens(g.x, (g.tokens - 1) * (uint32_t)g.ldx + g.width * 2), powers(scales, g.up.window);
    // (a gate's rows, and those of the other half)
    const uint32_t others = g.gated ? g.hidden : 0, bytes = row_bytes<W>(g.width);
    const Window first = Window::rows(base, g.up.ld, g.hidden + others - n0, bytes);
    const Window second =
        Window::rows(base + (int64_t)others * g.up.ld, g.up.ld, g.hidden - n0, bytes);
    typename P::Source from = {tokens, first, second, powers, {}, {}, {}, 0};
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const uint32_t r = i * 16 + lane % 16;
        from.a[i] = r < count ? g.by_top_k(rows[r]) * (uint32_t)g.ldx : Window::kNowhere;
    }
#pragma unroll
    for (int j = 0; j < FB; ++j) {
        uint32_t c = n0 + (g.gated ? j % FN : j) * 16 + lane % 16;
        c = c < g.hidden ? c : g.hidden - 1;
        from.b[j] = (c - n0) * (uint32_t)g.up.ld;
        c += g.gated ? j / FN * g.hidden : 0;
        from.p[j] = lane < 16 ? c * (uint32_t)g.up.ld_scales : Window::kNowhere;
    }
    f32x4 acc[1][RM][FB] = {};
    // the last step first: it may be ragged
    const uint32_t steps = P::steps(g.width);
    if (steps > wave) {
        P p[DEEP];
        const bool ragged = wave == 0 && P::ragged(g.width);
        uint32_t next = steps - 1 - wave;
        auto fetch = [&](P &q) {
            q.fetch(from, next);
            next = next < 4 ? next : next - 4;
        };
        pipeline((steps - wave + 3) / 4, p,
                 [&](P &q) {
                     if (!ragged) return fetch(q);
                     q.fetch_last(from, next, g.width);
                     next = next < 4 ? next : next - 4;
                 },
                 fetch,
                 [&](P &q) {
                     if (!ragged) return;
                     q.mend_a(steps - 1, g.width * 2);
                     q.mend_b(steps - 1, g.width, scales, from.p);
                 },
                 [&](P &q) { q.multiply(acc); });
    }
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < FB; ++j) sums[(wave * RM * FB + i * FB + j) * 64 + lane] = acc[0][i][j];
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
        h.store(r, c, v, g.hidden - c);
    }
}

// 16 RM pairs at a time; where there are more than 16 tokens, few experts have that many of them, so the
// smallest tile stands beside the larger one.
template <class T, class W, int RM, int FN, int DEEP>
__global__ void __launch_bounds__(256) k_few_up(FewArgs g)
{
    __shared__ Routes routes;
    __shared__ uint16_t rows[4][16 * RM];
    __shared__ __align__(16) f32x4 sums[4 * RM * 2 * FN * 64];
    if (blockIdx.x == 0)
        for (uint32_t i = threadIdx.x; i < g.tiles; i += 256) g.arrived[i] = 0;
    const Router<16 * RM, false> router(g, routes);
    const uint32_t each = g.gated ? 16 * FN : 32 * FN, tiles = (g.hidden + each - 1) / each;
    const uint32_t slot = g.by_up_tiles(blockIdx.x), n0 = (blockIdx.x - slot * tiles) * each;
    if (slot >= router.count) return;
    uint16_t *const mine = rows[__builtin_amdgcn_readfirstlane(threadIdx.x / 64)];
    uint32_t e, before;
    const uint32_t count = router.find(slot, mine, e, before);
    const Rows h(g, before, count);
    if (n0 == 0 && (uint32_t)(g.ldh / 4) > g.hidden) h.clear(g.hidden, (uint32_t)(g.ldh / 4));
    if (RM == 1 || count <= 16) up_rows<T, W, 1, FN, DEEP>(g, e, n0, mine, h, sums);
    else up_rows<T, W, RM, FN, DEEP>(g, e, n0, mine, h, sums);
}

// ---------------------------------------------------------------------------
// Tiles of 16 FN columns of the result. The workgroups take equal shares of all tiles, so that one
// has a part of a tile, or of several. A part is of the steps of all experts, one expert's after another's; the
// waves have a run of them each, so that a wave meets few experts. When it leaves one, it
// adds the rows' products times their weights (and the columns' scales) to its own sums of the tokens in
// LDS. The workgroup that arrives last at a tile adds the workgroups' sums in their order.

// Lane l holds the scale of column l % 16; a result's column is 4 (l / 16) + c.
__device__ __forceinline__ float column_scale(float scale, int c)
{
    return __shfl(scale, threadIdx.x % 64 / 16 * 4 + c, 64);
}

// Some steps of one slot, the last one first: it may be ragged.
template <class T, class W, int RM, int FN, int DEEP, Tokens OF, class O>
__device__ __forceinline__ void down_rows(const FewArgs &g, const O &router, uint32_t e, uint32_t n0,
                                          uint32_t from, uint32_t some, const uint16_t *rows,
                                          const Rows &h, f32x4 *total)
{
    constexpr bool kScales = std::is_same<W, int8_t>::value;
    typedef Piece<T, W, RM, FN, OF> P;
    constexpr uint32_t kEach = P::kOfWords;  // rows of a pair
    // (the steps that are shared out are two of a piece of one half)
    const uint32_t steps = P::steps(g.hidden);
    if constexpr (P::kHalves == 1) {
        from *= 2;
        some = 2 * some < steps - from ? 2 * some : steps - from;
    }
    const uint32_t lane = threadIdx.x % 64, at = lane / 16, count = h.count;
    const Window tokens(h.base, count * (uint32_t)g.ldh);
    const char *const scales = g.down.scales + (int64_t)e * g.down.scales_stride;
    const Window powers(scales, g.down.window);
    const Window columns =
        Window::rows(g.down.data + (int64_t)e * g.down.stride + (int64_t)n0 * g.down.ld, g.down.ld,
                     g.n - n0, row_bytes<W>(g.hidden));
    typename P::Source source = {tokens, columns, columns, powers, {}, {}, {}, h.unit()};
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const uint32_t r = i * 16 + lane % 16;
        source.a[i] = r < kEach * count ? (at * kEach * count + r) * 16 : Window::kNowhere;
    }
    float scale[kScales ? FN : 1];  // of column lane % 16
#pragma unroll
    for (int j = 0; j < FN; ++j) {
        uint32_t c = n0 + j * 16 + lane % 16;
        c = c < g.n ? c : g.n - 1;
        source.b[j] = (c - n0) * (uint32_t)g.down.ld;
        source.p[j] = lane < 16 ? c * (uint32_t)g.down.ld_scales : Window::kNowhere;
        if constexpr (kScales) scale[j] = ((const float *)scales)[c];
    }
    f32x4 acc[P::kSums][RM][FN] = {};
    P p[DEEP];
    const bool ragged = P::ragged(g.hidden) && from + some == steps;
    uint32_t next = from + some - 1;
    auto fetch = [&](P &q) {
        q.fetch(source, next);
        next = next > from ? next - 1 : from;
    };
    pipeline(some, p,
             [&](P &q) {
                 if (!ragged) return fetch(q);
                 q.fetch_last(source, next, g.hidden);
                 next = next > from ? next - 1 : from;
             },
             fetch,
             [&](P &q) {
                 if (ragged) q.mend_b(steps - 1, g.hidden, scales, source.p);
             },
             [&](P &q) { q.multiply(acc); });
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const uint32_t r = i * 16 + lane % 16, pair = r < count ? rows[r] : 0, token = g.by_top_k(pair);
        const float by = router.weight(pair);
        f32x4 v[FN];
#pragma unroll
        for (int j = 0; j < FN; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                // of an infinite h the first part counts; a folded pair's second word is in a row after its own
                auto sum = [&](int s) {
                    float v = acc[s * P::kOfWords][i][j][c];
                    if constexpr (OF == kFolded)
                        v += __shfl(acc[s * 2 + 1][i][j][c], (int)(lane / 16 * 16 + (lane + count) % 16), 64);
                    return v;
                };
                v[j][c] = sum(0);
                if constexpr (P::kSums > P::kOfWords) {
                    const float rest = sum(1);
                    if (__builtin_isfinite(v[j][c])) v[j][c] += rest;
                }
                v[j][c] *= by;
                if constexpr (kScales) v[j][c] *= column_scale(scale[j], c);
            }
        f32x4 *const to = total + (token / 16 * FN * 4 + at) * 16 + token % 16;
        auto add = [&] {
#pragma unroll
            for (int j = 0; j < FN; ++j) to[j * 64] += v[j];
        };
        // a token that has the expert twice is in two rows: these go one after another
        const uint32_t before = (uint32_t)__shfl_up((int)token, 1, 64);
        const bool twice = lane % 16 != 0 && r < count && before == token;
        if (__ballot(twice) == 0) {
            if (r < count) add();
        } else {
            for (uint32_t q = 0; q < 16; ++q) {
                if (lane % 16 == q && r < count) add();
                __builtin_amdgcn_wave_barrier();
            }
        }
        __builtin_amdgcn_wave_barrier();
    }
}

template <class T, class W, int RM, int FN, int DEEP, int WAVES>
__global__ void __launch_bounds__(WAVES * 64) k_few_down(FewArgs g)
{
    __shared__ Routes routes;
    __shared__ uint16_t rows[WAVES][16 * RM];
    __shared__ uint32_t last;
    const Router<16 * RM, true> router(g, routes);
    const uint32_t lane = threadIdx.x % 64, at = lane / 16;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const uint32_t pairs = g.tokens * g.top_k;
    const uint32_t steps = (row_bytes<W>(g.hidden) + kStep - 1) / kStep;
    const uint32_t all = router.count * steps;
    // the sums of each wave: [tokens, in 16s][FN][16], a row's four columns of a lane together
    const uint32_t high = (g.tokens + 15) / 16;
    f32x4 *const sums = (f32x4 *)(few_lds + ids_bytes(pairs) + by_bytes(pairs));
    f32x4 *const total = sums + wave * high * FN * 64;

    // (in units of 1 / groups of a tile)
    uint32_t until;
    for (uint32_t from_tile = blockIdx.x * g.tiles; from_tile < (blockIdx.x + 1) * g.tiles;
         from_tile = until) {
        const uint32_t tile = g.by_groups(from_tile), n0 = tile * 16 * FN;
        until = (tile + 1) * g.groups;
        if (until > (blockIdx.x + 1) * g.tiles) until = (blockIdx.x + 1) * g.tiles;
        const uint32_t begin = (from_tile - tile * g.groups) * WAVES + wave * (until - from_tile);
        const uint32_t first = share(all, begin, g.groups * WAVES, g.by_waves);
        const uint32_t mine = share(all, begin + until - from_tile, g.groups * WAVES, g.by_waves) - first;
        const uint32_t leader = g.by_tiles(tile * g.groups);  // the first workgroup that has a part of it
        const uint32_t sharing = g.by_tiles((tile + 1) * g.groups - 1) - leader + 1;
        const uint32_t own = blockIdx.x - leader;
        if (from_tile != blockIdx.x * g.tiles) __syncthreads();  // the sums before these have been read
        for (uint32_t i = lane; i < high * FN * 64; i += 64) total[i] = f32x4{};

        for (uint32_t done = 0, some; done < mine; done += some) {
            // some steps of one expert, the last one first: it may be ragged
            const uint32_t slot = g.by_steps(first + done), from = first + done - slot * steps;
            some = steps - from < mine - done ? steps - from : mine - done;
            uint32_t e, before;
            const uint32_t count = router.find(slot, rows[wave], e, before);
            const Rows h(g, before, count);
            if (h.folded())
                down_rows<T, W, 1, FN, DEEP, kFolded>(g, router, e, n0, from, some, rows[wave], h, total);
            else if (RM == 1 || count <= 16)
                down_rows<T, W, 1, FN, DEEP, kOfH>(g, router, e, n0, from, some, rows[wave], h, total);
            else down_rows<T, W, RM, FN, DEEP, kOfH>(g, router, e, n0, from, some, rows[wave], h, total);
        }
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
        uint32_t *const parts = g.partial + (uint64_t)tile * g.parts * (high * FN * 256);
        for (uint32_t f = wave; f < high * FN; f += WAVES) {
            f32x4 v = sums[f * 64 + lane];
#pragma unroll
            for (int w = 1; w < WAVES; ++w) v += sums[(w * high * FN + f) * 64 + lane];
            if (sharing == 1) {
                store(f, v);
            } else {
                // written through to where every XCD sees it
                uint32_t *to = parts + (own * high * FN + f) * 256 + lane;
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    __hip_atomic_store(to + q * 64, __float_as_uint(v[q]), __ATOMIC_RELAXED,
                                       __HIP_MEMORY_SCOPE_AGENT);
            }
        }
        if (sharing == 1) continue;
        asm volatile("s_waitcnt vmcnt(0)" : : : "memory");  // this wave's sums are there
        __syncthreads();
        if (threadIdx.x == 0)
            last = __hip_atomic_fetch_add(g.arrived + tile, 1u, __ATOMIC_RELAXED,
                                          __HIP_MEMORY_SCOPE_AGENT) == sharing - 1;
        __syncthreads();
        if (!last) continue;
        // eight workgroups' sums on their way at one time
        for (uint32_t i = threadIdx.x; i < high * FN * 256; i += WAVES * 64) {
            float v = 0.f;
            for (uint32_t s = 0; s < sharing; s += 8) {
                uint32_t part[8];
#pragma unroll
                for (uint32_t q = 0; q < 8; ++q)
                    part[q] = __hip_atomic_load(
                        parts + (uint64_t)(s + q < sharing ? s + q : s) * high * FN * 256 + i,
                        __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
#pragma unroll
                for (uint32_t q = 0; q < 8; ++q)
                    if (s + q < sharing) v += __uint_as_float(part[q]);
            }
            ((float *)sums)[(i / 256 * 64 + i % 64) * 4 + i / 64 % 4] = v;
        }
        __syncthreads();
        for (uint32_t f = wave; f < high * FN; f += WAVES) store(f, sums[f * 64 + lane]);
    }
}

// ---------------------------------------------------------------------------
// Steps that a wave has on their way (four: 35.7 us instead of 34.5 for one token in 16 bits, 56.5 instead of 51
// for four in 8).
constexpr int kDeep = 2;
constexpr int kDownWaves = 8;  // of a workgroup of the second kernel

// Fragments of columns of a workgroup (FN): two for 4-bit weights, whose tokens' rows count for more of what
// is loaded, if there are no more than 16 of them (71 us instead of 73.5 for 16 tokens; 55 instead of 51 for
// four tokens in 8 bits).
template <class W, int RM> constexpr int few_columns()
{
    return std::is_same<W, Mx4>::value && RM == 1 ? 2 : 1;
}
inline uint32_t columns_of(int32_t kind, uint32_t rows)
{
    return kind == EXPERTS_WEIGHT_MX4 && rows == 1 ? 2 : 1;
}

// 16 pairs of an expert at a time for up to 16 tokens, 32 for more.
inline uint32_t rows_of_16(uint64_t tokens) { return tokens <= 16 ? 1 : 2; }

// Entries of the list that there can be.
inline uint64_t most_slots(uint64_t pairs, uint32_t experts, uint32_t rows)
{
    const uint64_t some = pairs < experts ? pairs : experts;
    return some + (pairs - some) / (16 * rows);
}

// Bytes of a row of h: whole steps of the second kernel.
inline int64_t h_bytes(uint32_t hidden, int32_t down_kind)
{
    const uint32_t values = kStep / 2 << down_kind;  // (16, 8 and 4 bits)
    return ((int64_t)hidden + values - 1) / values * values * 4;
}

struct FewPlan {
    uint32_t rows, tiles, groups, parts;  // of the result (see FewArgs)
    uint64_t h, arrived, partial, bytes;  // offsets in the workspace, and its size
};

inline FewPlan few_plan(uint64_t tokens, uint32_t top_k, uint32_t experts, uint32_t hidden, uint32_t n,
                        int32_t down_kind)
{
    FewPlan p;
    p.rows = rows_of_16(tokens);
    const uint32_t fn = columns_of(down_kind, p.rows);
    p.tiles = (n + 16 * fn - 1) / (16 * fn);
    const uint64_t pairs = tokens * top_k, slots = most_slots(pairs, experts, p.rows);
    const uint32_t bytes = down_kind == EXPERTS_WEIGHT_16     ? hidden * 2
                           : down_kind == EXPERTS_WEIGHT_INT8 ? hidden
                                                              : (hidden + 31) / 32 * 16;
    // Either a tile for `sharing` whole workgroups, or 256 workgroups with equal shares of all tiles. What
    // a workgroup does once a part costs it as much as reading 64 KB or so. us with whole ones and with equal
    // shares: 129 tiles of 0.8 MB 68 and 63, 224 83 and 87, 320 155 and 121, 512 175 and 174; 65 of 0.3 MB 26
    // and 30. Two steps of 128 bytes for each wave are the least.
    constexpr uint64_t kOnce = 65536;
    const uint64_t tile = slots * bytes * 16 * fn, steps = slots * ((bytes + 127) / 128) / (2 * kDownWaves);
    const uint64_t most = steps < 1 ? 1 : steps < 64 ? steps : 64;
    uint64_t best = UINT64_MAX;
    for (uint64_t sharing = 1; sharing <= most && (sharing == 1 || p.tiles * sharing <= 4096); ++sharing) {
        const uint64_t cost = (p.tiles * sharing + kCus - 1) / kCus * (tile / sharing + kOnce);
        if (cost < best) best = cost, p.groups = (uint32_t)(p.tiles * sharing);
    }
    if (p.tiles > 4096) best = UINT64_MAX;  // (share() has 32 bits)
    if (p.tiles * most > kCus && p.tiles * tile / kCus + ((p.tiles + kCus - 1) / kCus + 1) * kOnce < best)
        p.groups = kCus;
    // (where neither is a multiple of the other, a tile's ends lie within workgroups' shares)
    p.parts = (p.groups + p.tiles - 1) / p.tiles + (p.groups % p.tiles && p.tiles % p.groups);
    auto up = [](uint64_t b) { return (b + 255) / 256 * 256; };
    p.h = 0;
    p.arrived = up(pairs * h_bytes(hidden, down_kind));
    p.partial = p.arrived + up((uint64_t)p.tiles * 4);
    p.bytes = p.partial + (p.parts > 1 ? (uint64_t)p.tiles * p.parts * ((tokens + 15) / 16) * fn * 1024 : 0);
    return p;
}

template <class T, class W, int RM>
hist_status_t launch_up(FewArgs g, uint64_t slots, hipStream_t stream)
{
    constexpr int FN = few_columns<W, RM>();
    const uint32_t each = g.gated ? 16 * FN : 32 * FN, tiles = (g.hidden + each - 1) / each;
    g.by_up_tiles = Divide::by(tiles);
    return launch(k_few_up<T, W, RM, FN, kDeep>, slots * tiles, 256, ids_bytes(g.tokens * g.top_k),
                  stream, g);
}

template <class T, class W>
hist_status_t launch_up_any(const FewArgs &g, uint64_t slots, hipStream_t stream)
{
    return g.tokens <= 16 ? launch_up<T, W, 1>(g, slots, stream)
                          : launch_up<T, W, 2>(g, slots, stream);
}

template <class T, class W, int RM, int WAVES>
hist_status_t launch_down(const FewArgs &g, hipStream_t stream)
{
    constexpr int FN = few_columns<W, RM>();
    const uint32_t pairs = g.tokens * g.top_k;
    return launch(k_few_down<T, W, RM, FN, kDeep, WAVES>, g.groups, WAVES * 64,
                  ids_bytes(pairs) + by_bytes(pairs) + WAVES * ((g.tokens + 15) / 16) * FN * 1024,
                  stream, g);
}

template <class T, class W>
hist_status_t launch_down_any(const FewArgs &g, hipStream_t stream)
{
    return g.tokens <= 16 ? launch_down<T, W, 1, kDownWaves>(g, stream)
                          : launch_down<T, W, 2, kDownWaves>(g, stream);
}

template <class T>
hist_status_t launch_few(const FewArgs &g, const FewPlan &p, int32_t up_kind, int32_t down_kind,
                         hipStream_t stream)
{
    const uint64_t slots = most_slots((uint64_t)g.tokens * g.top_k, g.experts, p.rows);
    const hist_status_t st =
        up_kind == EXPERTS_WEIGHT_16     ? launch_up_any<T, T>(g, slots, stream)
        : up_kind == EXPERTS_WEIGHT_INT8 ? launch_up_any<T, int8_t>(g, slots, stream)
                                         : launch_up_any<T, Mx4>(g, slots, stream);
    if (st != HIST_OK) return st;
    return down_kind == EXPERTS_WEIGHT_16     ? launch_down_any<T, T>(g, stream)
           : down_kind == EXPERTS_WEIGHT_INT8 ? launch_down_any<T, int8_t>(g, stream)
                                              : launch_down_any<T, Mx4>(g, stream);
}

// Defined in a source of their own each, so that they compile at one time.
hist_status_t launch_few_bf16(const FewArgs &g, const FewPlan &p, int32_t up_kind,
                              int32_t down_kind, hipStream_t stream);
hist_status_t launch_few_fp16(const FewArgs &g, const FewPlan &p, int32_t up_kind,
                              int32_t down_kind, hipStream_t stream);

}  // namespace pca_experts
