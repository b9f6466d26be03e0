// experts_tile256.hip -- experts' products in tiles of up to 256 rows by 256
// weight rows, as the prefill GEMM's.
#define Q4_EXPERTS_MF 16
#define Q4_EXPERTS_WAVES_PER_SIMD 2
#define Q4_EXPERTS_LAUNCH launch_experts_tile256
#include "experts_tile.hpp"
