// Host helpers that the cache operators share: checks of shapes, kernel classes, the plan of the merge and the workspace.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/gqa_decode.h"
#include "gqa_host.cuh"
#include "gqa_kv8_decode.cuh"

namespace gqa {

inline bool block_size_ok(int bs) { return bs == 8 || bs == 16 || bs == 32 || bs == 64; }

inline int log2_of(int block_size) { return block_size == 8 ? 3 : (block_size == 16 ? 4 : (block_size == 32 ? 5 : 6)); }

inline bool aligned_to(const void* p, uintptr_t n) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

inline gqa_status cuda_status(cudaError_t e) { return e == cudaSuccess ? GQA_OK : GQA_ERR_CUDA; }

inline gqa_status check_kv8(int N, int h_kv, int D, int max_blocks, int num_blocks, int block_size) {
  if (N < 0 || N > 65535 || h_kv < 1 || h_kv > 65535 || max_blocks < 1 || num_blocks < 0) return GQA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return GQA_ERR_UNSUPPORTED;
  if (!block_size_ok(block_size)) return GQA_ERR_INVALID_ARG;
  if ((int64_t)max_blocks * block_size >= (int64_t(1) << 31)) return GQA_ERR_INVALID_ARG;
  if ((int64_t)num_blocks * block_size >= (int64_t(1) << 31)) return GQA_ERR_INVALID_ARG;
  return GQA_OK;
}

inline gqa_status check_rows(int N, int T_q, int h_q, int h_kv, int D) {
  if (N < 0 || N > 65535 || T_q < 1 || h_q < 1 || h_kv < 1 || h_kv > 65535 || h_q % h_kv != 0)
    return GQA_ERR_INVALID_ARG;
  if (D != 64 && D != 128) return GQA_ERR_UNSUPPORTED;
  if ((int64_t)(h_q / h_kv) * T_q > 64) return GQA_ERR_UNSUPPORTED;
  return GQA_OK;
}

// ---------------------------------------------------------------- decode
// Kernel shapes: up to 8, 16, 24 or 32 query rows for one warp, 48 or 64 for two warps that share a ring.
// 24 and 48 beside 32 and 64, measured (us, with / without): 131071 keys, 24 rows, d 128 56.6 / 67.7, in f16 65.5 / 85.3; 10
// sequences of 5000-53000, 35 rows 136 / 175; 43 of 50-1460, 24 rows, d 64 27.8 / 31.4.
inline int kv8_class(int rows) { return rows <= 32 ? (rows + 7) / 8 - 1 : (rows <= 48 ? 4 : 5); }
inline int kv8_groups(int cls) { return cls < 4 ? kKv8Warps : kKv8Warps / 2; }

// Workers for each unit from which the merge gives 32 columns of a row a CTA instead of a whole row a warp, as long as those
// are no more than kMergeCtas.  Measured (us, columns a CTA / rows a warp; CTAs in brackets): 9 pieces, 16 sequences of
// 250-500 keys, 8 KV heads 15.5 / 12.4; 19 pieces, 8 of 8000-16000 38.7 / 40.4 [1024], 64 of 16000-32000 with one KV head of
// 4 query heads 67.3 / 69.4 [1024], of 16 79.2 / 75.3 [4096]; 38 pieces, 4 of 8000-16000 23.8 / 30.9 [512]; 64 rows of 30 of
// 8000-16000, d 64, 54.2 / 51.6 [3840].
constexpr int kManyPieces = 16;
constexpr int kMergeCtas = 2048;

// CTAs of a unit in the short kernel, a cluster of 1, 2, 4 or 8: the fewest that give each worker one tile, as far as all
// units' clusters fit on three quarters of the SMs at once (a cluster lies in one GPC).  0: the general kernel, where a
// worker would have more than kKv8Short tiles, or more than two above what the general kernel, which uses every SM,
// gives one.  Measured (us of a replayed call, short / general; tiles of a worker in brackets): 8 KV heads of 128: one
// sequence of 300 keys 5.3 / 7.6 [1, 1], 2000 5.7 / 7.6 [1, 1], 8000 8.9 / 8.9 [4, 2], 16000 13.1 / 11.0 [8, 4]; 4 of 500-1000
// 6.5 / 9.6 [1, 1]; 16 of 1000-2000 13.0 / 17.0 [8, 7]; 2 KV heads of 64: 4096 keys 5.5 / 6.6 [2, 1], 16384 10.2 / 8.3 [8, 1].
inline int kv8_short_ctas(int64_t units, int64_t seq_tiles, int sms, int groups) {
  int ctas = 1;
  while (ctas < 8 && ctas * groups < seq_tiles && units * ctas * 2 <= sms * 3 / 4) ctas *= 2;
  const int64_t here = (seq_tiles + ctas * groups - 1) / (ctas * groups);
  const int64_t there = (units * seq_tiles + sms * groups - 1) / (sms * groups);
  if (units * ctas > sms || here > kKv8Short || here > there + 2) return 0;
  return ctas;
}

struct Kv8Layout {
  size_t splits, m, l, o, total;
};

// workspace: the status header, the units that are cut and two partials for each worker
inline Kv8Layout kv8_layout(int workers, int rows, int D) {
  Kv8Layout L;
  const size_t n = 2 * (size_t)workers * rows;
  L.splits = kHeaderBytes;
  L.m = L.splits + align256((size_t)workers * sizeof(int4));
  L.l = L.m + align256(n * 4);
  L.o = L.l + align256(n * 4);
  L.total = L.o + align256(n * D * 4);
  return L;
}

}  // namespace gqa
