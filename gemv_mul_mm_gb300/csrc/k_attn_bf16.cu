// k_attn_bf16.cu -- qattn_decode over a bf16 cache.
#define QMM_ATTN_FMT QMM_KV_BF16
#include "attn_launch.cuh"
