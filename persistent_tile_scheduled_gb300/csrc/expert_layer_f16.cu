#include "expert_layer.cuh"

namespace pts {
cudaError_t launch_layer_f16(const LayerParams &p, const RowsRoom &room, cudaStream_t stream, bool overlap) { return launch_layer<0>(p, room, stream, overlap); }
}  // namespace pts
