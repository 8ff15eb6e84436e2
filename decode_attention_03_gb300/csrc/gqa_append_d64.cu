// Filling a paged cache, d_head 64, binary16.
#include "gqa_append_inst.cuh"

GQA_APPEND_INSTANCE(64, false)
