// experts_few.hip -- a whole expert layer for a few tokens (declared in experts.h): the checks and the
// kernels for float16 tokens.
#include "experts_few.hpp"

namespace pca_experts {

inline hist_status_t check_few(uint64_t tokens, uint32_t top_k, uint32_t experts, uint32_t hidden,
                               uint32_t n, int32_t down_kind)
{
    if (top_k == 0 || experts == 0 || hidden == 0 || n == 0 || down_kind < EXPERTS_WEIGHT_16 ||
        down_kind > EXPERTS_WEIGHT_MX4)
        return HIST_ERR_INVALID_ARG;
    if (tokens > EXPERTS_MAX_FEW || top_k > EXPERTS_MAX_TOP_K || experts > EXPERTS_MAX_EXPERTS ||
        hidden > EXPERTS_MAX_WIDTH || n > EXPERTS_MAX_WIDTH)
        return HIST_ERR_UNSUPPORTED;
    return HIST_OK;
}

// A weight [experts][rows][k] of a kind, in bytes; false if it cannot be one.
inline bool few_weight(FewWeight &w, const experts_weight_t *from, uint32_t rows, uint32_t k)
{
    if (!from || from->kind < EXPERTS_WEIGHT_16 || from->kind > EXPERTS_WEIGHT_MX4 || !from->data ||
        from->stride < 0)
        return false;
    const bool wide = from->kind == EXPERTS_WEIGHT_16, mx4 = from->kind == EXPERTS_WEIGHT_MX4;
    const int64_t size = wide ? 2 : 1, scale = mx4 ? 1 : 4;
    const int64_t blocks = (k + 31) / 32;
    w = {(const char *)from->data, (const char *)from->scales, from->ld * size, from->stride * size,
         mx4 ? from->ld_scales : 0, from->scales_stride * scale,
         mx4 ? (uint32_t)((rows - 1) * from->ld_scales + blocks) : 0};
    if (from->ld < (mx4 ? blocks * 16 : (int64_t)k) || misaligned(w.data, size)) return false;
    if (wide) return true;
    return w.scales && from->scales_stride >= 0 && !misaligned(w.scales, scale) &&
           (!mx4 || from->ld_scales >= blocks);
}

hist_status_t launch_few_fp16(const FewArgs &g, const FewPlan &p, int32_t up_kind,
                              int32_t down_kind, hipStream_t stream)
{
    return launch_few<_Float16>(g, p, up_kind, down_kind, stream);
}

}  // namespace pca_experts

using namespace pca_experts;

extern "C" hist_status_t experts_few_tokens_workspace_size(uint64_t tokens, uint32_t top_k,
                                                           uint32_t experts, uint32_t hidden,
                                                           uint32_t n, int32_t down_kind,
                                                           uint64_t *bytes)
{
    if (!bytes) return HIST_ERR_INVALID_ARG;
    const hist_status_t st = check_few(tokens, top_k, experts, hidden, n, down_kind);
    if (st != HIST_OK) return st;
    *bytes = tokens ? few_plan(tokens, top_k, experts, hidden, n, down_kind).bytes : 0;
    return HIST_OK;
}

extern "C" hist_status_t experts_few_tokens(void *out, int64_t ldo, const void *x, int64_t ldx,
                                            const experts_weight_t *up,
                                            const experts_weight_t *down, const void *ids,
                                            int32_t id_bits, const float *weights, uint64_t tokens,
                                            uint32_t top_k, uint32_t experts, uint32_t width,
                                            uint32_t hidden, uint32_t n, int32_t gated,
                                            int32_t dtype, void *workspace,
                                            uint64_t workspace_bytes, hipStream_t stream)
{
    if (!down || !up || !dtype_ok(dtype) || width == 0 || (id_bits != 32 && id_bits != 64) ||
        (gated != 0 && gated != 1))
        return HIST_ERR_INVALID_ARG;
    hist_status_t st = check_few(tokens, top_k, experts, hidden, n, down->kind);
    if (st != HIST_OK) return st;
    // (rows of 16 bytes: no load is shorter)
    if (width > EXPERTS_MAX_WIDTH || width < (up->kind == EXPERTS_WEIGHT_INT8 ? 16u : 8u) ||
        hidden < (down->kind == EXPERTS_WEIGHT_INT8 ? 16u : 8u))
        return HIST_ERR_UNSUPPORTED;
    FewArgs g = {};
    const uint32_t up_rows = gated ? 2 * hidden : hidden;
    if (!few_weight(g.up, up, up_rows, width) || !few_weight(g.down, down, n, hidden) || ldo < (int64_t)n ||
        ldx < (int64_t)width || misaligned(out, 2) || misaligned(x, 2) ||
        misaligned(ids, id_bits / 8) || misaligned(weights, 4) ||
        (tokens && (!out || !x || !ids || !weights)))
        return HIST_ERR_INVALID_ARG;
    // (32-bit places in x, in h, in 32 rows of a weight and in an expert's powers of two)
    auto near = [](uint64_t rows, int64_t ld) { return rows * ld <= Window::kMost; };
    if (ldx > (1 << 30) || !near(EXPERTS_MAX_FEW, ldx * 2) || up->ld > (1 << 25) ||
        down->ld > (1 << 25) ||
        (up->kind == EXPERTS_WEIGHT_MX4 &&
         (up->ld_scales > (1 << 30) || !near(up_rows, up->ld_scales))) ||
        (down->kind == EXPERTS_WEIGHT_MX4 &&
         (down->ld_scales > (1 << 30) || !near(n, down->ld_scales))))
        return HIST_ERR_UNSUPPORTED;
    const FewPlan p = few_plan(tokens ? tokens : 1, top_k, experts, hidden, n, down->kind);
    if (tokens && (!workspace || misaligned(workspace, 16) || workspace_bytes < p.bytes))
        return HIST_ERR_WORKSPACE;
    st = device_status();
    if (st != HIST_OK || tokens == 0) return st;
    g.out = (char *)out;
    g.x = (const char *)x;
    g.h = (char *)workspace + p.h;
    g.arrived = (uint32_t *)((char *)workspace + p.arrived);
    g.partial = (uint32_t *)((char *)workspace + p.partial);
    g.ids = ids;
    g.by = weights;
    g.ldo = ldo * 2;
    g.ldx = ldx * 2;
    g.ldh = h_bytes(hidden, down->kind);
    g.ids64 = id_bits == 64;
    g.tokens = (uint32_t)tokens;
    g.top_k = top_k;
    g.experts = experts;
    g.width = width;
    g.hidden = hidden;
    g.n = n;
    g.tiles = p.tiles;
    g.groups = p.groups;
    g.parts = p.parts;
    g.by_top_k = Divide::by(top_k);
    g.by_tiles = Divide::by(p.tiles);
    g.by_groups = Divide::by(p.groups);
    g.by_waves = Divide::by(p.groups * kDownWaves);
    g.by_steps = Divide::by((uint32_t)(g.ldh / 4 / (kStep / 2 << down->kind)));
    g.gated = (uint32_t)gated;
    g.h_shift = (uint32_t)down->kind;  // (of 16, 8 and 4 bits: 0, 1, 2)
    return (dtype == EXPERTS_BF16 ? launch_few_bf16 : launch_few_fp16)(g, p, up->kind, down->kind,
                                                                      stream);
}
