// Instantiations of the experts' forward product.
#include "expert_gemm.cuh"

namespace pts {

template <int KIND>
static ExpertOps pick(int cg, int bn)
{
    if (bn == kExpertTileNFew) return ExpertInst<KIND, EXPERT_FWD, 1, kExpertTileNFew>::ops();
    return cg == 2 ? ExpertInst<KIND, EXPERT_FWD, 2, kExpertTileN>::ops()
                   : ExpertInst<KIND, EXPERT_FWD, 1, kExpertTileN>::ops();
}

ExpertOps expert_ops_fwd(int kind, int cg, int bn)
{
    return kind == 0 ? pick<0>(cg, bn) : (kind == 1 ? pick<1>(cg, bn) : pick<2>(cg, bn));
}

}  // namespace pts
