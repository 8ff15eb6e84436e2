// The launches of the append kernel for one d_head and type; a translation unit for each instantiates them.
#pragma once
#include "../../include/gqa_decode.h"
#include "gqa_host.cuh"
#include "gqa_kv8.cuh"

namespace gqa {

// Heads of a warp, in groups of HPW: as many as four where the tokens then still fill the GPU's resident warps,
// so that a token's cosines, sines and weights are loaded once for them; else one, the shortest chain.
// Measured (us, groups 1 / 2 / 4): 16384 tokens, 64 + 8 + 8 heads of 128: 117.0 / 105.6 / 105.4; 8192 tokens, 32 + 8 + 8
// heads into the 8-bit cache, with a read-back: 61.9 / 58.1 / 57.2; but 64 tokens with theirs, before the rule 4.5 / 4.8 / 5.6.
template <int D, bool BF16, int CW, bool PAIRS, int LAYOUT, bool AXES>
cudaError_t append_launch(AppendParams p, int sms, cudaStream_t st) {
  constexpr int HPW = 32 / (D / (2 * CW));
  const int qg = (p.h_q + HPW - 1) / HPW, kg = (p.h_kv + HPW - 1) / HPW;
  int sets = 0;
  for (p.iters = kAppendIters;; p.iters /= 2) {
    p.q_sets = (qg + p.iters - 1) / p.iters;
    p.k_sets = (kg + p.iters - 1) / p.iters;
    sets = p.q_sets + 2 * p.k_sets;
    if (p.iters == 1 || (int64_t)p.num_tokens * sets >= (int64_t)sms * 4 * (kAppendThreads / 32)) break;
  }
  const unsigned per = kAppendThreads / 32;
  // as many tokens of a warp as leave two rounds of CTAs.  Measured (us, at least 1 / 2 / 3 / 4 rounds): 8192 tokens of
  // 32 + 8 + 8 heads of 128 with the read-back 58.8 / 57.2 / 57.2 / 60.7; of 8 + 2 + 2 heads of 64 10.1 / 9.8 / 11.4 / 11.3.
  const int64_t round = (int64_t)sms * kAppendCtas * per;
  for (p.run = 1; p.run < kAppendRun && (int64_t)p.num_tokens * sets >= 4 * p.run * round;) p.run *= 2;
  const dim3 grid(((unsigned)p.num_tokens + per * p.run - 1) / (per * p.run), (unsigned)sets);
  return launch_pdl_smem(gqa_append_kernel<D, BF16, CW, PAIRS, LAYOUT, AXES>, grid, kAppendThreads, 0, st, 1, p);
}

template <int D, bool BF16, int CW, bool PAIRS, int LAYOUT>
cudaError_t append_axes(const AppendParams& p, int sms, cudaStream_t st) {
  if (p.cos_sin != nullptr && p.pair_axes != nullptr) return append_launch<D, BF16, CW, PAIRS, LAYOUT, true>(p, sms, st);
  return append_launch<D, BF16, CW, PAIRS, LAYOUT, false>(p, sms, st);
}

template <int D, bool BF16, int CW, bool PAIRS>
cudaError_t append_layout(const AppendParams& p, int layout, int sms, cudaStream_t st) {
  switch (layout) {
    case GQA_CACHE_ROWS: return append_axes<D, BF16, CW, PAIRS, GQA_CACHE_ROWS>(p, sms, st);
    case GQA_CACHE_VLLM: return append_axes<D, BF16, CW, PAIRS, GQA_CACHE_VLLM>(p, sms, st);
    case GQA_CACHE_KV8: return append_axes<D, BF16, CW, PAIRS, GQA_CACHE_KV8>(p, sms, st);
    default: return append_axes<D, BF16, CW, PAIRS, GQA_CACHE_KV4>(p, sms, st);
  }
}

}  // namespace gqa

#define GQA_APPEND_INSTANCE(D, BF16)                                                                                \
  namespace gqa {                                                                                                   \
  template <>                                                                                                       \
  cudaError_t append_run<D, BF16>(const AppendParams& p, int layout, int sms, cudaStream_t st) {                    \
    const bool pairs = p.cos_sin != nullptr && p.interleaved;                                                       \
    if (p.cos_sin != nullptr && p.rot_dim % 16 != 0)                                                                \
      return pairs ? append_layout<D, BF16, 4, true>(p, layout, sms, st)                                            \
                   : append_layout<D, BF16, 4, false>(p, layout, sms, st);                                          \
    return pairs ? append_layout<D, BF16, 8, true>(p, layout, sms, st)                                              \
                 : append_layout<D, BF16, 8, false>(p, layout, sms, st);                                            \
  }                                                                                                                 \
  }
