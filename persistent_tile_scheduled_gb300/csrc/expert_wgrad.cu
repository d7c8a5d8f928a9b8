// Instantiations of the experts' gradient product for the weights.
#include "expert_gemm.cuh"

namespace pts {

template <int KIND>
static ExpertOps pick(int cg)
{
    return cg == 2 ? ExpertInst<KIND, EXPERT_WGRAD, 2, kExpertTileN>::ops()
                   : ExpertInst<KIND, EXPERT_WGRAD, 1, kExpertTileN>::ops();
}

ExpertOps expert_ops_wgrad(int kind, int cg) { return kind == 0 ? pick<0>(cg) : pick<1>(cg); }

}  // namespace pts
