// Instantiations of the forward product with an epilogue, for one type: the
// including file names the type (PTS_LINEAR_KIND) and the function.
#include "expert_gemm.cuh"

namespace pts {

template <int EPI>
static ExpertOps pick(int cg, int bn)
{
    if (bn == kExpertTileNFew) return ExpertInst<PTS_LINEAR_KIND, EXPERT_FWD, 1, kExpertTileNFew, EPI>::ops();
    return cg == 2 ? ExpertInst<PTS_LINEAR_KIND, EXPERT_FWD, 2, kExpertTileN, EPI>::ops()
                   : ExpertInst<PTS_LINEAR_KIND, EXPERT_FWD, 1, kExpertTileN, EPI>::ops();
}

ExpertOps PTS_LINEAR_OPS(bool gated, int cg, int bn) { return gated ? pick<EPI_GATED>(cg, bn) : pick<EPI_LINEAR>(cg, bn); }

}  // namespace pts
