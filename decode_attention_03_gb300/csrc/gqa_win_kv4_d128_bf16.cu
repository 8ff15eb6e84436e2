// Decode attention over the 4-bit cache, d_head 128, bfloat16.
#include "gqa_win_inst.cuh"

GQA_WIN_INSTANCE(128, true, true)
