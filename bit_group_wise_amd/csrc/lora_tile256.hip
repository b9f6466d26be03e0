// lora_tile256.hip -- the product with adapters in 256 x 256 tiles.
#define Q4_LORA_LAUNCH launch_lora_tile256
#include "lora_tile.hpp"
