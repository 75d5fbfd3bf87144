// k_attn_f16.cu -- qattn_decode over a f16 cache.
#define QMM_ATTN_FMT QMM_KV_F16
#include "attn_launch.cuh"
