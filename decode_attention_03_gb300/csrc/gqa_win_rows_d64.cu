// Decode attention over 16-bit pools with a sliding window, d_head 64, binary16.
#include "gqa_win_inst.cuh"

GQA_WIN_INSTANCE(64, false, false)
