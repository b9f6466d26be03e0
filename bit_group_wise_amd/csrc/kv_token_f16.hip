// kv_token_f16.hip -- the few-row attention of kv_token.hip for fp16 outputs,
// which have as many bits as one fp16 weight: weights enter the second product
// in two parts, so that the output's own rounding is all that shows.
#define Q4_KV_TOKEN_TWO 1
#define launch_kv_token launch_kv_token_f16
#include "kv_token.hip"
