// Decode attention over the 4-bit cache, d_head 64, bfloat16.
#include "gqa_win_inst.cuh"

GQA_WIN_INSTANCE(64, true, true)
