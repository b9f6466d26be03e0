// experts_tile128.hip -- experts' products in tiles of 128 rows by 256 weight
// rows.
#define Q4_GEMM_BM 128
#define Q4_EXPERTS_LAUNCH launch_experts_tile128
#include "experts_tile.hpp"
