// Instantiations of the experts' gradient product for the rows.
#include "expert_gemm.cuh"

namespace pts {

template <int KIND>
static ExpertOps pick(int cg)
{
    return cg == 2 ? ExpertInst<KIND, EXPERT_DGRAD, 2, kExpertTileN>::ops()
                   : ExpertInst<KIND, EXPERT_DGRAD, 1, kExpertTileN>::ops();
}

ExpertOps expert_ops_dgrad(int kind, int cg) { return kind == 0 ? pick<0>(cg) : pick<1>(cg); }

}  // namespace pts
