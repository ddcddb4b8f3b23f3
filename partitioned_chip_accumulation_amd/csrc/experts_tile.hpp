// experts_tile.hpp -- one tile of a matrix product on the matrix cores: staging
// of its operands in LDS, the fragments read from there, and the tile's place
// in the ragged list of the experts' rows.
//
// A tile is D[m][n] = sum_r A[m][r] B[n][r]. An operand lies in memory either
// along the reduction (Along: a row of memory is one m or n, its elements
// consecutive r) or across it (Across: a row of memory is one r, its
// elements consecutive m or n). Both are staged in steps of 128 bytes of
// reduction (64 16-bit elements, 128 8-bit ones):
//
//   Along   [rows][128 bytes]; a lane's fragment is one 16-byte read.
//   Across  [64][columns]; a lane's fragment is two transposing 8-byte reads.
//
// The fragments go to the matrix instruction with B first, so that a lane
// holds four consecutive columns n of one row m of the result.
//
// 4-bit operands (Mx4) lie along the reduction, two elements a byte, and are loaded and read like 8-bit
// ones: a lane's 16 bytes are one block of 32 elements, which has a power of two of its own. Those
// of a step, 8 bytes a row, follow the operands in LDS.
#pragma once

#include "experts_common.hpp"

#include <type_traits>

namespace pca_experts {

constexpr uint32_t kCus = 256;  // of the device

constexpr uint32_t kStepBytes = 128;
constexpr uint32_t kStepPowers = kStepBytes / 16;  // bytes of powers of two that go with them

// What one matrix instruction takes and gives, by element type. add() keeps the sum
// in its registers: the compiler's own form names other ones for the result, and in the
// pipelined kernels, whose sums take half of all registers, it spilled. The compiler does not
// see what such an instruction needs around it: s_nop 1 stands between it and a
// move into its operands, and sums_done() must come before the sums are read.
template <class T> struct Mma;
template <> struct Mma<__bf16> {
    typedef bf16x8 Frag;
    typedef f32x4 Acc;
    static __device__ __forceinline__ Acc run(Frag a, Frag b, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ void add(Frag a, Frag b, Acc &c)
    {
        asm("s_nop 1\n\tv_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
    }
};
template <> struct Mma<_Float16> {
    typedef f16x8 Frag;
    typedef f32x4 Acc;
    static __device__ __forceinline__ Acc run(Frag a, Frag b, Acc c)
    {
        return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ void add(Frag a, Frag b, Acc &c)
    {
        asm("s_nop 1\n\tv_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
    }
};
template <> struct Mma<int8_t> {
    typedef s32x4 Frag;
    typedef s32x4 Acc;
    static __device__ __forceinline__ Acc run(Frag a, Frag b, Acc c)
    {
        return __builtin_amdgcn_mfma_i32_16x16x64_i8(a, b, c, 0, 0, 0);
    }
    static __device__ __forceinline__ void add(Frag a, Frag b, Acc &c)
    {
        asm("s_nop 1\n\tv_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+v"(c) : "v"(a), "v"(b));
    }
};

struct Mx4 {
    uint8_t two;
};
template <> struct Mma<Mx4> {
    typedef s32x4 Frag;
    typedef f32x4 Acc;
    // Byte A of pa and byte B of pb: the exponents plus 127 (255: NaN) of the lane's blocks.
    // (4: four bits, of one sign, two exponent and one fraction bit)
    template <int A, int B>
    static __device__ __forceinline__ void add(Frag a, Frag b, Acc &c, uint32_t pa, uint32_t pb)
    {
        asm("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 "
            "op_sel:[%5,%6,0] op_sel_hi:[%7,%8,0] cbsz:4 blgp:4"
            : "+v"(c)
            : "v"(a), "v"(b), "v"(pa), "v"(pb), "n"(A & 1), "n"(B & 1), "n"(A >> 1), "n"(B >> 1));
    }
    // With bytes that the compiler knows once it has unrolled the loops around.
    template <int A>
    static __device__ __forceinline__ void add(Frag a, Frag b, Acc &c, uint32_t pa, uint32_t pb,
                                               int at_b)
    {
        if (at_b == 0) add<A, 0>(a, b, c, pa, pb);
        else if (at_b == 1) add<A, 1>(a, b, c, pa, pb);
        else if (at_b == 2) add<A, 2>(a, b, c, pa, pb);
        else add<A, 3>(a, b, c, pa, pb);
    }
    static __device__ __forceinline__ void add(Frag a, Frag b, Acc &c, uint32_t pa, uint32_t pb,
                                               int at_a, int at_b)
    {
        if (at_a == 0) add<0>(a, b, c, pa, pb, at_b);
        else if (at_a == 1) add<1>(a, b, c, pa, pb, at_b);
        else if (at_a == 2) add<2>(a, b, c, pa, pb, at_b);
        else add<3>(a, b, c, pa, pb, at_b);
    }
};

template <class Acc, int FM, int FN>
__device__ __forceinline__ void sums_done(Acc (&acc)[FM][FN])
{
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(acc[i][j]));
    // the longest matrix instruction here is followed by 19 cycles in which its result
    // must not be read
    asm volatile("s_nop 15\n\ts_nop 15");
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) asm volatile("" : "+v"(acc[i][j]));
}

// Of 16 bytes that end with a row, the last `left` (any number), followed by zeros.
__device__ __forceinline__ u32x4 drop16(u32x4 v, int left)
{
    const uint32_t s = left >= 16 ? 0 : left > 0 ? 16 - left : 16;  // bytes to drop
    const bool eight = s & 8, four = s & 4;
    const uint32_t a0 = eight ? v[2] : v[0], a1 = eight ? v[3] : v[1];
    const uint32_t a2 = eight ? 0 : v[2], a3 = eight ? 0 : v[3];
    const uint32_t b0 = four ? a1 : a0, b1 = four ? a2 : a1, b2 = four ? a3 : a2;
    const uint32_t b3 = four ? 0 : a3;
    const u32x4 r = {__builtin_amdgcn_alignbyte(b1, b0, s), __builtin_amdgcn_alignbyte(b2, b1, s),
                     __builtin_amdgcn_alignbyte(b3, b2, s), __builtin_amdgcn_alignbyte(0, b3, s)};
    return s == 16 ? u32x4{0, 0, 0, 0} : r;
}

// 16 bytes at p, of which only the first `left` (any number) belong to the row; the others
// read 0. Any alignment of T. Where the row has 16 bytes (`roomy`, the same for the wave), the 16 that
// end with it are read and shifted (a product of 16384 rows and 2048 columns with a reduction of
// 133: 56 us; element by element 66).
template <class T>
__device__ __forceinline__ u32x4 load16(const char *p, int left, bool roomy)
{
    if (roomy) return drop16(load_any<u32x4>(p + (left < 16 ? left : 16) - 16), left);
    u32x4 v = {0, 0, 0, 0};
    constexpr int kEach = 16 / sizeof(T);
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
        if (i * (int)sizeof(T) < left) {
            uint32_t e;
            if constexpr (sizeof(T) == 1) e = *(const uint8_t *)(p + i);
            else e = load_any<uint16_t>(p + i * 2);
            v[i * sizeof(T) / 4] |= e << (i * sizeof(T) * 8 % 32);
        }
    }
    return v;
}

// ---------------------------------------------------------------------------
// How an operand lies in LDS. A thread moves kLoads 16-byte pieces of it per step; the pieces of
// one load of a wave lie together, in the order of the lanes, and the place in the
// row that a piece comes from is permuted so that the fragments' reads meet no bank twice.

// Along the reduction: ROWS rows of 128 bytes. Eight pieces a row, piece s of row r holding
// the row's bytes 16 * (s ^ (r >> 1) % 8). (A 16-byte read serves 16 lanes at a time: 0-3, 12-15
// and 20-27 first, then 4-11, 16-19 and 28-31, and so in the upper half.)
template <class T, int ROWS, int THREADS>
struct Along {
    static constexpr bool kAcross = false;
    static constexpr int kLoads = ROWS * 8 / THREADS;
    static constexpr uint32_t kBytes = ROWS * kStepBytes;
    static_assert(ROWS * 8 % THREADS == 0 && THREADS / 8 % 16 == 0, "pieces of one permutation");

    static __device__ __forceinline__ uint32_t row_of(int i)
    {
        return i * (THREADS / 8) + threadIdx.x / 8;
    }
    // This thread's byte within a row's step, and the place of its wave's load i.
    static __device__ __forceinline__ uint32_t byte()
    {
        return ((threadIdx.x % 8) ^ ((threadIdx.x / 16) & 7)) * 16;
    }
    static __device__ __forceinline__ uint32_t place_of(int i, uint32_t wave)
    {
        return (i * (THREADS / 64) + wave) * 1024;
    }
    // Fragment i of the part that starts at row first, half kk (64 bytes) of the step.
    static __device__ __forceinline__ typename Mma<T>::Frag frag(const char *lds, uint32_t first,
                                                                 int i, int kk)
    {
        const uint32_t lane = threadIdx.x % 64, r = first + i * 16 + lane % 16;
        const uint32_t piece = (lane / 16 + 4 * kk) ^ ((r >> 1) & 7);
        return *(const typename Mma<T>::Frag *)(lds + r * kStepBytes + piece * 16);
    }
};

// The powers of two of 4-bit operands in LDS: 8 bytes a row and step, four for each half. Those of
// rows r, r + 16, r + 32 and r + 48 lie together, so that one read of a lane has what four
// fragments need, and one register takes it. A load of a wave is 32 rows: its lane is four bytes of row
// row_of(load), half half_of().
struct Powers {
    static __device__ __forceinline__ uint32_t row_of(uint32_t load)
    {
        const uint32_t lane = threadIdx.x % 64;
        return load / 2 * 64 + lane % 4 * 16 + load % 2 * 8 + lane / 8;
    }
    static __device__ __forceinline__ uint32_t half_of() { return threadIdx.x / 4 % 2; }
    // Byte i: the power of this lane's block of fragment i, N of them (2 or 4) from row first on.
    template <int N>
    static __device__ __forceinline__ uint32_t read(const char *lds, uint32_t first, int kk)
    {
        const uint32_t lane = threadIdx.x % 64, at = lane / 16;
        const char *p = lds + first / 64 * 512 + lane % 16 * 32 + kk * 16 + first / 16 % 4 * 4;
        if constexpr (N == 2) {
            typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
            const u32x2 v = *(const u32x2 *)p;
            return __builtin_amdgcn_perm(v[1], v[0], at | (at + 4) << 8);
        } else {
            const u32x4 v = *(const u32x4 *)p;
            const uint32_t pick = at | (at + 4) << 8;
            const uint32_t low = __builtin_amdgcn_perm(v[1], v[0], pick);
            const uint32_t high = __builtin_amdgcn_perm(v[3], v[2], pick);
            return __builtin_amdgcn_perm(high, low, 0x05040100);
        }
    }
};

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

// Across the reduction. One load of a wave holds kTogether whole rows (1024 bytes), so
// they lie together in LDS; 64 bytes follow them, and 128 more follow each four loads
// of two rows. Within a row the 32-byte parts are permuted by part ^ r % kTogether.
// The eight rows that half a wave takes 32 bytes of in one transposing read, r0 to r0 + 3 and r0 + 8
// to r0 + 11, then meet all 64 banks once, and the fragments of one operand need
// only kTogether addresses in registers (with a permutation of all of a row's parts by
// the row each fragment needed its own, and they did not fit).
template <class T, int COLS, int THREADS>
struct Across {
    static constexpr bool kAcross = true;
    static constexpr int kRows = kStepBytes / 2;
    static constexpr int kPieces = COLS / 8;
    static constexpr int kLoads = kRows * kPieces / THREADS;
    static constexpr int kRowsEach = THREADS / kPieces;
    static constexpr int kTogether = 64 / kPieces;
    static_assert(kRows * kPieces % THREADS == 0 && (kTogether == 2 || kTogether == 4),
                  "rows of 128 or 256 columns");

    // Where load number l of a step (a wave's) lies.
    static constexpr __device__ uint32_t place(uint32_t l)
    {
        return l * 1088 + (kTogether == 2 ? l / 4 * 128 : 0);
    }
    static constexpr uint32_t kBytes = kRows / kTogether * 1088 +
                                       (kTogether == 2 ? kRows / kTogether / 4 * 128 : 0);
    // The place of this wave's load i.
    static __device__ __forceinline__ uint32_t place_of(int i, uint32_t wave)
    {
        return place(i * (THREADS / 64) + wave);
    }
    static __device__ __forceinline__ uint32_t row_of(int i)
    {
        return i * kRowsEach + threadIdx.x / kPieces;
    }
    // The byte in a row of this thread's pieces.
    static __device__ __forceinline__ uint32_t byte()
    {
        return ((threadIdx.x % kPieces) ^ (threadIdx.x / kPieces % kTogether << 1)) * 16;
    }
    // Fragment i of the part that starts at column first (a multiple of 64), half kk.
    static __device__ __forceinline__ typename Mma<T>::Frag frag(const char *lds, uint32_t first,
                                                                 int i, int kk)
    {
        const uint32_t lane = threadIdx.x % 64, q = lane % 16, r = lane / 16 * 8 + q / 4;
        const uint32_t part = (i % kTogether) ^ (r % kTogether);
        const char *p = lds + place(r / kTogether) + r % kTogether * (COLS * 2) + first * 2 +
                        part * 32 + q % 4 * 8;
        p += place(kk * 32 / kTogether) + i / kTogether * kTogether * 32;
        union {
            s16x4 half[2];
            typename Mma<T>::Frag whole;
        } f;
        f.half[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)p);
        f.half[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)(p + place(4 / kTogether)));
        return f.whole;
    }
};

// ---------------------------------------------------------------------------
// Rows at 16-byte multiples go straight from memory to LDS, a lane's piece at a time; others
// pass through registers.

// What a piece outside the operand reads.
static __device__ const u32x4 kZeros = {0, 0, 0, 0};

// 16 bytes from each lane's address to LDS at lds + 16 * lane (lds: byte offset, the
// same for the wave; m0 carries it, which no other instruction here uses). The
// instruction has no result register, so nothing that the compiler allocates can
// be overwritten while it is in flight; wait_loads orders it before the reads.
__device__ __forceinline__ void load_to_lds(const char *p, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off"
                 :
                 : "s"(lds), "v"(p));
}

// The same from base + each lane's offset; base is the wave's.
__device__ __forceinline__ void load_to_lds(const char *base, uint32_t offset, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
                 :
                 : "s"(lds), "v"(offset), "s"(base));
}

// Four bytes a lane, to LDS at lds + 4 * lane; of lanes that are not active, nothing.
__device__ __forceinline__ void load4_to_lds(const char *p, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
                 :
                 : "s"(lds), "v"(p));
}
__device__ __forceinline__ void load4_to_lds(const char *base, uint32_t offset, uint32_t lds)
{
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2"
                 :
                 : "s"(lds), "v"(offset), "s"(base));
}

// The way through registers: a lane's piece to LDS.
template <class V>
__device__ __forceinline__ void put_in_lds(V v, uint32_t lds)
{
    typedef __attribute__((address_space(3))) V Piece;
    *(Piece *)(uintptr_t)(lds + threadIdx.x % 64 * sizeof(V)) = v;
}

// Until at most N of the wave's loads are in flight.
template <int N>
__device__ __forceinline__ void wait_loads()
{
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

__device__ __forceinline__ void block_barrier()
{
    asm volatile("" : : : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" : : : "memory");
}

// n / d for n < 2^30 and 1 <= d < 2^31: mul = ceil(2^(31 + s) / d) with s =
// floor(log2 d) is at most 2^31 and exceeds the real quotient by less than 1, which
// moves n * mul by less than 2^30 < 2^(31 + s) / d (as d < 2^(s + 1)), so the floor
// is exact.
struct Divide {
    uint32_t mul, shift;
    static Divide by(uint32_t d)
    {
        uint32_t s = 0;
        while (d >> (s + 1)) ++s;
        return {(uint32_t)(((1ull << (31 + s)) + d - 1) / d), s};
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t n) const
    {
        return __umulhi(2 * n, mul) >> shift;
    }
};

// ---------------------------------------------------------------------------
// The list of tiles. Group g of the sorted rows is expert g's, g = experts the
// rows past the last kept one (their results are zero). The tiles of one
// group come together, its row tiles within 8 of them fastest, so that tiles
// that run at one time share rows and weights in the L2.
struct Tile {
    uint32_t group;  // > experts: no such tile
    uint32_t begin;  // the group's rows are [begin, end)
    uint32_t end;
    uint32_t m;      // row tile within the group
    uint32_t n;      // column tile
};

// Workgroups go to the 8 XCDs in turn: `span` consecutive tiles go to one.
__device__ __forceinline__ uint32_t tile_of_block(uint32_t block, uint32_t span)
{
    const uint32_t xcd = block % 8, i = block / 8;
    return (i / span * 8 + xcd) * span + i % span;
}

// offsets == nullptr: one group of all rows. Every wave finds the tile by
// itself: 64 groups at a time, the scan of their row tiles, and a ballot.
__device__ __forceinline__ Tile find_tile(uint32_t tile, const int32_t *__restrict__ offsets,
                                          uint32_t experts, uint32_t rows, uint32_t rows_log2,
                                          uint32_t n_tiles)
{
    Tile t;
    uint32_t m_tiles = 0, before = 0;
    const uint32_t want = tile / n_tiles;  // row tiles before, over all groups
    if (!offsets) {
        t.group = 0;
        t.begin = 0;
        t.end = rows;
        m_tiles = (rows + (1u << rows_log2) - 1) >> rows_log2;
        if (want >= m_tiles) t.group = experts + 1;
    } else {
        const uint32_t lane = threadIdx.x % 64;
        t.group = experts + 1;
        t.begin = t.end = 0;
        for (uint32_t g0 = 0; g0 <= experts; g0 += 64) {
            const uint32_t g = g0 + lane;
            uint32_t b = 0, e = 0;
            if (g <= experts) {
                b = (uint32_t)offsets[g];
                e = g < experts ? (uint32_t)offsets[g + 1] : rows;
                e = e > rows ? rows : e;
                b = b > e ? e : b;
            }
            const uint32_t mine = (e - b + (1u << rows_log2) - 1) >> rows_log2;
            const uint32_t upto = wave_inclusive_scan(mine);
            const uint64_t past = __ballot(before + upto > want);
            if (past) {
                const int at = __builtin_ctzll(past);
                t.group = g0 + at;
                t.begin = __builtin_amdgcn_readlane(b, at);
                t.end = __builtin_amdgcn_readlane(e, at);
                m_tiles = __builtin_amdgcn_readlane(mine, at);
                before += __builtin_amdgcn_readlane(upto, at) - m_tiles;
                break;
            }
            before += __builtin_amdgcn_readlane(upto, 63);
        }
    }
    if (t.group <= experts) {
        const uint32_t i = tile - before * n_tiles;
        const uint32_t eight = i / (8 * n_tiles), r = i - eight * 8 * n_tiles;
        const uint32_t high = m_tiles - eight * 8 < 8 ? m_tiles - eight * 8 : 8;
        t.m = eight * 8 + r % high;
        t.n = r / high;
    }
    return t;
}

// Row tiles of all experts (without the rows past the last kept one).
__device__ __forceinline__ uint32_t count_row_tiles(const int32_t *__restrict__ offsets,
                                                    uint32_t experts, uint32_t rows,
                                                    uint32_t rows_log2)
{
    const uint32_t past_one = (1u << rows_log2) - 1;
    if (!offsets) return (rows + past_one) >> rows_log2;
    uint32_t all = 0;
    for (uint32_t g0 = 0; g0 < experts; g0 += 64) {
        const uint32_t g = g0 + threadIdx.x % 64;
        uint32_t b = 0, e = 0;
        if (g < experts) {
            b = (uint32_t)offsets[g];
            e = (uint32_t)offsets[g + 1];
            e = e > rows ? rows : e;
            b = b > e ? e : b;
        }
        all += __builtin_amdgcn_readlane(wave_inclusive_scan((e - b + past_one) >> rows_log2), 63);
    }
    return all;
}

// The expert with the rank-th most rows (0: the most; equals in the order of their numbers), so
// that the workgroups with the most steps start first. The rank-th largest count is
// found bit by bit: a bit stays set if more than `rank` experts have at least so many
// rows, which a ballot of the wave counts.
template <uint32_t kMost>  // 64 experts each
__device__ __forceinline__ uint32_t expert_of_rank(const int32_t *__restrict__ offsets,
                                                   uint32_t experts, uint32_t rows, uint32_t rank)
{
    const uint32_t lane = threadIdx.x % 64;
    uint32_t count[kMost];  // of experts g * 64 + lane, plus 1; 0: no such expert
#pragma unroll
    for (uint32_t g = 0; g < kMost; ++g) {
        count[g] = 0;
        if (g * 64 + lane < experts) {
            uint32_t e = (uint32_t)offsets[g * 64 + lane + 1], b = (uint32_t)offsets[g * 64 + lane];
            e = e > rows ? rows : e;
            count[g] = e > b ? e - b + 1 : 1;
        }
    }
    auto at_least = [&](uint32_t c) {
        uint32_t n = 0;
#pragma unroll
        for (uint32_t g = 0; g < kMost; ++g)
            n += (uint32_t)__popcll(__ballot(count[g] >= c));
        return n;
    };
    uint32_t value = 0;
    for (uint32_t bit = 1u << (31 - __builtin_clz(rows + 1)); bit; bit >>= 1)
        if (at_least(value | bit) > rank) value |= bit;
    uint32_t left = rank - at_least(value + 1), found = 0;  // how many equals come before it
    bool done = false;
#pragma unroll
    for (uint32_t g = 0; g < kMost; ++g) {
        if (!done) {
            const uint64_t equal = __ballot(count[g] == value);
            const uint32_t n = (uint32_t)__popcll(equal);
            const bool here = (equal >> lane & 1) &&
                              (uint32_t)__popcll(equal & ((1ull << lane) - 1)) == left;
            const uint64_t mine = __ballot(here);
            if (mine) {
                found = g * 64 + (uint32_t)__builtin_ctzll(mine);
                done = true;
            }
            left -= n;
        }
    }
    return found;
}

}  // namespace pca_experts
