// experts_tile128.hip -- experts' products in tiles of up to 128 rows by 128
// weight rows, by workgroups of 4 waves, several of which share a compute unit.
#define Q4_GEMM_BN 128
#define Q4_GEMM_WAVES 4
#define Q4_EXPERTS_MF 8
#define Q4_EXPERTS_WAVES_PER_SIMD 3
#define Q4_EXPERTS_LAUNCH launch_experts_tile128
#include "experts_tile.hpp"
