// The forward product with an epilogue, fp16 operands.
#define PTS_LINEAR_KIND 0
#define PTS_LINEAR_OPS linear_ops_f16
#include "linear_inst.cuh"
