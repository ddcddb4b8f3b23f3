// experts_group.hip -- pairs counted and sorted by expert (declared in
// experts.h).
//
// The sort is a histogram with ranks: place[i] = offsets[e] + #{i' < i : id
// i' = e} for e = ids[i]. The pairs are cut into chunks of consecutive
// ones, one workgroup each; within a chunk each of the 16 waves owns 1/16 of
// it, in order. Ranks therefore do not depend on the order of any atomic:
//   1. k_group_count: one LDS histogram per chunk, written as a row of the
//      workspace (left out when there is one chunk);
//   2. k_group_place: each workgroup sums the rows before its own (its starts)
//      and all rows (the totals, whose scan is the offsets), counts its waves'
//      ids in LDS, and ranks 64 pairs of a wave at a time: the lanes with
//      the same id are found by one ballot for each bit of the id.
// Bound by latency: 256 pairs take 3.3 us, 524,168 pairs of 256 experts 4.8 and 13.0 us (6.3 MB
// read or written). One workgroup up to 8192 pairs saves the first kernel and its gap.
#include "experts_common.hpp"

namespace pca_experts {

constexpr uint32_t kThreads = 1024;
constexpr uint32_t kWaves = kThreads / 64;
constexpr uint32_t kOneChunk = 8 * kThreads;  // up to here one workgroup does it all
constexpr uint32_t kGroups = 16;              // of lanes, that read the chunks' rows
constexpr uint32_t kMostChunks = 512;         // each workgroup reads every chunk's row

// Pairs of one workgroup.
inline uint32_t chunk_size(uint32_t pairs)
{
    const uint32_t rounds = (pairs + kThreads - 1) / kThreads;
    if (pairs <= kOneChunk) return kThreads * (rounds ? rounds : 1);
    const uint32_t least = (rounds + kMostChunks - 1) / kMostChunks;
    return kThreads * (least > 2 ? least : 2);
}

// Words of a chunk's row: a multiple of 16 bytes (what lies past the last expert is never used).
__host__ __device__ inline uint32_t row_words(uint32_t experts) { return (experts + 3) / 4 * 4; }

// The id of pair i, `experts` for one outside the range.
template <class I>
__device__ __forceinline__ uint32_t expert_of(const I *ids, uint32_t i, uint32_t experts)
{
    const I v = ids[i];
    return v >= 0 && v < (I)experts ? (uint32_t)v : experts;
}

template <class I>
__global__ void __launch_bounds__(kThreads) k_group_count(const I *__restrict__ ids,
                                                          uint32_t pairs, uint32_t experts,
                                                          uint32_t chunk,
                                                          uint32_t *__restrict__ rows)
{
    __shared__ uint32_t hist[EXPERTS_MAX_EXPERTS];
    for (uint32_t e = threadIdx.x; e < experts; e += kThreads) hist[e] = 0;
    __syncthreads();
    for (uint32_t r = 0; r < chunk; r += kThreads) {
        const uint32_t i = blockIdx.x * chunk + r + threadIdx.x;
        if (i < pairs) {
            const uint32_t e = expert_of(ids, i, experts);
            if (e < experts) lds_add(hist, e, 1u);
        }
    }
    __syncthreads();
    for (uint32_t e = threadIdx.x; e < experts; e += kThreads)
        rows[blockIdx.x * row_words(experts) + e] = hist[e];
}

// rows == nullptr: the grid is one workgroup, which takes all pairs.
// Dynamic LDS: kWaves rows of `experts` counters, then (with rows) 2 * kGroups rows of partial sums.
template <class I>
__global__ void __launch_bounds__(kThreads)
    k_group_place(const I *__restrict__ ids, uint32_t pairs, uint32_t experts, uint32_t id_bits,
                  uint32_t chunk, uint32_t chunks, const uint32_t *__restrict__ rows,
                  int32_t *__restrict__ counts, int32_t *__restrict__ offsets,
                  int32_t *__restrict__ order, int32_t *__restrict__ place)
{
    extern __shared__ __align__(16) uint32_t wave_at[];
    __shared__ uint32_t wave_total[kWaves];
    const uint32_t wave = threadIdx.x / 64, lane = threadIdx.x % 64;
    const uint32_t own = chunk / kWaves;  // pairs of one wave
    const uint32_t first = blockIdx.x * chunk + wave * own;

    for (uint32_t s = threadIdx.x; s < kWaves * experts; s += kThreads) wave_at[s] = 0;
    __syncthreads();
    uint32_t *mine = wave_at + wave * experts;
    for (uint32_t r = 0; r < own; r += 64) {
        const uint32_t i = first + r + lane;
        if (i < pairs) {
            const uint32_t e = expert_of(ids, i, experts);
            if (e < experts) lds_add(mine, e, 1u);
        }
    }
    __syncthreads();

    // The experts' pairs in earlier chunks and in all. The rows are read four experts a
    // lane, by as many groups of lanes as there are (at most kGroups), all loads of a lane in flight.
    const uint32_t e = threadIdx.x;
    uint32_t before = 0, total = 0;
    if (rows) {
        uint32_t *part = wave_at + kWaves * experts;
        const uint32_t quads = row_words(experts) / 4;
        const uint32_t most = kThreads / quads, groups = most < kGroups ? most : kGroups;
        const uint32_t quad = threadIdx.x % quads, group = threadIdx.x / quads;
        if (group < groups) {
            u32x4 early = {0, 0, 0, 0}, late = {0, 0, 0, 0};
#pragma unroll 8
            for (uint32_t c = group; c < chunks; c += groups) {
                const u32x4 v = ((const u32x4 *)rows)[c * quads + quad];
                if (c < blockIdx.x) early += v;
                else late += v;
            }
            ((u32x4 *)part)[group * quads + quad] = early;
            ((u32x4 *)part)[(groups + group) * quads + quad] = late;
        }
        __syncthreads();
        if (e < experts) {
            for (uint32_t c = 0; c < groups; ++c) {
                before += part[c * quads * 4 + e];
                total += part[(groups + c) * quads * 4 + e];
            }
            total += before;
        }
    } else if (e < experts) {
        for (uint32_t w = 0; w < kWaves; ++w) total += wave_at[w * experts + e];
    }
    const uint32_t inclusive = wave_inclusive_scan(total);
    if (lane == 63) wave_total[wave] = inclusive;
    __syncthreads();
    uint32_t start = inclusive - total, kept = 0;
    for (uint32_t w = 0; w < kWaves; ++w) {
        if (w < wave) start += wave_total[w];
        kept += wave_total[w];
    }
    if (e < experts) {
        if (blockIdx.x == 0) {
            counts[e] = (int32_t)total;
            offsets[e] = (int32_t)start;
        }
        uint32_t at = start + before;
        for (uint32_t w = 0; w < kWaves; ++w) {
            const uint32_t c = wave_at[w * experts + e];
            wave_at[w * experts + e] = at;
            at += c;
        }
    }
    if (blockIdx.x == 0 && threadIdx.x == 0) offsets[experts] = (int32_t)kept;
    __syncthreads();

    for (uint32_t r = 0; r < own; r += 64) {
        const uint32_t i = first + r + lane;
        const uint32_t v = i < pairs ? expert_of(ids, i, experts) : experts;
        uint64_t same = __ballot(v < experts);
        for (uint32_t b = 0; b < id_bits; ++b) {
            const uint64_t set = __ballot((v >> b) & 1u);
            same &= (v >> b) & 1u ? set : ~set;
        }
        const uint64_t below = same & ((1ull << lane) - 1);
        uint32_t at = 0;
        if (v < experts) at = mine[v] + (uint32_t)__popcll(below);
        // every lane has read its start before the last of each id moves it on;
        // the wave's LDS operations complete in order
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (v < experts && (same >> lane) == 1ull) mine[v] = at + 1;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (i < pairs) {
            place[i] = v < experts ? (int32_t)at : -1;
            if (v < experts) order[at] = (int32_t)i;
            if (i >= kept) order[i] = -1;
        }
    }
}

template <class I>
hist_status_t launch_group(const void *ids, uint32_t pairs, uint32_t experts, int32_t *counts,
                  int32_t *offsets, int32_t *order, int32_t *place, uint32_t *rows,
                  hipStream_t stream)
{
    uint32_t bits = 0;
    while ((experts - 1) >> bits) ++bits;
    const bool one = pairs <= kOneChunk;
    const uint32_t chunk = chunk_size(pairs);
    const uint32_t chunks = one ? 1 : (pairs + chunk - 1) / chunk;
    // the partial sums start at a multiple of 16 bytes: kWaves rows do
    const uint32_t quads = row_words(experts) / 4;
    const uint32_t groups = kThreads / quads < kGroups ? kThreads / quads : kGroups;
    const uint32_t lds = kWaves * experts * 4 + (one ? 0 : 2 * groups * quads * 16);
    if (!one) {
        const hist_status_t st = launch(k_group_count<I>, chunks, kThreads, 0, stream,
                                        (const I *)ids, pairs, experts, chunk, rows);
        if (st != HIST_OK) return st;
    }
    return launch(k_group_place<I>, chunks, kThreads, lds, stream, (const I *)ids, pairs, experts,
                  bits, chunk, chunks, one ? nullptr : rows, counts, offsets, order, place);
}

}  // namespace pca_experts

using namespace pca_experts;

extern "C" hist_status_t experts_group_workspace_size(uint64_t tokens, uint32_t top_k,
                                                      uint32_t experts, uint64_t *bytes)
{
    if (!bytes || top_k == 0 || experts == 0) return HIST_ERR_INVALID_ARG;
    if (experts > EXPERTS_MAX_EXPERTS || top_k > EXPERTS_MAX_TOP_K ||
        tokens > EXPERTS_MAX_ROWS / top_k)
        return HIST_ERR_UNSUPPORTED;
    const uint32_t pairs = (uint32_t)(tokens * top_k), chunk = chunk_size(pairs);
    *bytes = pairs <= kOneChunk ? 0 : (uint64_t)((pairs + chunk - 1) / chunk) * row_words(experts) * 4;
    return HIST_OK;
}

extern "C" hist_status_t experts_group(const void *ids, int32_t id_bits, uint64_t tokens,
                                       uint32_t top_k, uint32_t experts, int32_t *counts,
                                       int32_t *offsets, int32_t *order, int32_t *place,
                                       void *workspace, uint64_t workspace_bytes,
                                       hipStream_t stream)
{
    uint64_t need = 0;
    hist_status_t st = experts_group_workspace_size(tokens, top_k, experts, &need);
    if (st != HIST_OK) return st;
    if (id_bits != 32 && id_bits != 64) return HIST_ERR_INVALID_ARG;
    if (!counts || !offsets || (tokens && (!ids || !order || !place))) return HIST_ERR_INVALID_ARG;
    if (misaligned(ids, id_bits / 8) || misaligned(counts, 4) || misaligned(offsets, 4) ||
        misaligned(order, 4) || misaligned(place, 4))
        return HIST_ERR_INVALID_ARG;
    if (need && (!workspace || misaligned(workspace, 16) || workspace_bytes < need))
        return HIST_ERR_WORKSPACE;
    st = device_status();
    if (st != HIST_OK) return st;
    return (id_bits == 32 ? launch_group<int32_t> : launch_group<int64_t>)(
        ids, (uint32_t)(tokens * top_k), experts, counts, offsets, order, place,
        (uint32_t *)workspace, stream);
}
