// lora_tile64.hip -- the product with adapters in tiles of 64 rows by 128
// weight rows, where larger ones are too few to fill the card.
#define Q4_GEMM_BN 128
#define Q4_GEMM_WAVES 4
#define Q4_LORA_MF 4
#define Q4_LORA_LAUNCH launch_lora_tile64
#include "lora_tile.hpp"
