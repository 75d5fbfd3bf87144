// k_attn_q4_0.cu -- qattn_decode over a q4_0 cache.
#include "attn_q4_kernel.cuh"
#define QMM_ATTN_FMT QMM_KV_Q4_0
#define QMM_ATTN_Q4
#include "attn_launch.cuh"
