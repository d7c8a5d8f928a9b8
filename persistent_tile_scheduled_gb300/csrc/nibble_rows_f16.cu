// More rows times 4-bit weights, fp16 rows.
#define PTS_NIBBLE_KIND 0
#define PTS_NIBBLE_ROWS_LAUNCH launch_nibble_rows_f16
#include "nibble_rows.cuh"
