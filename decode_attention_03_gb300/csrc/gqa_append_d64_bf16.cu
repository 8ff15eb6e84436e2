// Filling a paged cache, d_head 64, bfloat16.
#include "gqa_append_inst.cuh"

GQA_APPEND_INSTANCE(64, true)
