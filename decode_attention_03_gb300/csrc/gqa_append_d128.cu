// Filling a paged cache, d_head 128, binary16.
#include "gqa_append_inst.cuh"

GQA_APPEND_INSTANCE(128, false)
