// The forward product with an epilogue, bf16 operands.
#define PTS_LINEAR_KIND 1
#define PTS_LINEAR_OPS linear_ops_bf16
#include "linear_inst.cuh"
