// k_attn_q8_0.cu -- qattn_decode over a q8_0 cache.
#define QMM_ATTN_FMT QMM_KV_Q8_0
#include "attn_launch.cuh"
