// The forward product with an epilogue, e4m3 operands.
#define PTS_LINEAR_KIND 2
#define PTS_LINEAR_OPS linear_ops_e4m3
#include "linear_inst.cuh"
