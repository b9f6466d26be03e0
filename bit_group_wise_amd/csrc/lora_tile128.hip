// lora_tile128.hip -- the product with adapters in tiles of 256 rows by 128
// weight rows, for middle numbers of rows (as gemm_bn128.hip).
#define Q4_GEMM_BN 128
#define Q4_GEMM_WAVES 4
#define Q4_LORA_LAUNCH launch_lora_tile128
#include "lora_tile.hpp"
