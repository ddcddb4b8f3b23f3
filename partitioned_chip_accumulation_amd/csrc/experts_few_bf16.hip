// experts_few_bf16.hip -- a whole expert layer for a few bfloat16 tokens (declared in experts.h).
#include "experts_few.hpp"

namespace pca_experts {

hist_status_t launch_few_bf16(const FewArgs &g, const FewPlan &p, int32_t up_kind,
                              int32_t down_kind, hipStream_t stream)
{
    return launch_few<__bf16>(g, p, up_kind, down_kind, stream);
}

}  // namespace pca_experts
