// experts_tile64.hip -- experts' products in tiles of up to 64 rows by 128
// weight rows, where larger ones are too few to fill the card.
#define Q4_GEMM_BN 128
#define Q4_GEMM_WAVES 4
#define Q4_EXPERTS_MF 4
#define Q4_EXPERTS_WAVES_PER_SIMD 3
#define Q4_EXPERTS_LAUNCH launch_experts_tile64
#include "experts_tile.hpp"
