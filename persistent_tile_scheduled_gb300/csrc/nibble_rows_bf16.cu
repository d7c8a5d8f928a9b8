// More rows times 4-bit weights, bf16 rows.
#define PTS_NIBBLE_KIND 1
#define PTS_NIBBLE_ROWS_LAUNCH launch_nibble_rows_bf16
#include "nibble_rows.cuh"
