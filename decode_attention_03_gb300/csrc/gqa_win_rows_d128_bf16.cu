// Decode attention over 16-bit pools with a sliding window, d_head 128, bfloat16.
#include "gqa_win_inst.cuh"

GQA_WIN_INSTANCE(128, false, true)
