#include "expert_layer.cuh"

namespace pts {
cudaError_t launch_layer_bf16(const LayerParams &p, const RowsRoom &room, cudaStream_t stream, bool overlap) { return launch_layer<1>(p, room, stream, overlap); }
}  // namespace pts
