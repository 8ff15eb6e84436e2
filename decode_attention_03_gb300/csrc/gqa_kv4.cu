// Host side of gqa_decode_kv4, gqa_decode_window and gqa_kv4_read, and the kernel of the last.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/gqa_decode.h"
#include "gqa_cache_host.cuh"
#include "gqa_win.cuh"

namespace gqa {
namespace {

// ---------------------------------------------------------------- per-device state
struct WinDevice {
  int sms = 0;
  bool ready[2][2][6][2] = {};   // [cache][d index][row class][bf16]: the kernels' shared memory is allowed
};
constexpr int kMaxDevices = 64;
std::mutex g_mu;
WinDevice g_win[kMaxDevices];

template <int D, bool KV4>
cudaError_t win_prepare_type(int cls, bool bf16) {
  return bf16 ? win_prepare<D, KV4, true>(cls) : win_prepare<D, KV4, false>(cls);
}

// SMs of the current device; the kernels of (cache, D, cls, bf16) are ready to launch on it
gqa_status win_device(bool kv4, int D, int cls, bool bf16, int* sms) {
  std::lock_guard<std::mutex> lock(g_mu);
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return GQA_ERR_CUDA;
  WinDevice& d = g_win[dev];
  if (d.sms == 0 && cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    d.sms = 0;
    return GQA_ERR_CUDA;
  }
  bool& ready = d.ready[kv4][D == 64 ? 0 : 1][cls][bf16];
  if (!ready) {
    const cudaError_t e = kv4 ? (D == 64 ? win_prepare_type<64, true>(cls, bf16) : win_prepare_type<128, true>(cls, bf16))
                              : (D == 64 ? win_prepare_type<64, false>(cls, bf16) : win_prepare_type<128, false>(cls, bf16));
    if (e != cudaSuccess) return GQA_ERR_CUDA;
    ready = true;
  }
  *sms = d.sms;
  return GQA_OK;
}

// ---------------------------------------------------------------- decode
int win_groups(bool kv4, int D, int cls) {
  if (D == 64) return kv4 ? win_workers<true, 64>(cls) : win_workers<false, 64>(cls);
  return kv4 ? win_workers<true, 128>(cls) : win_workers<false, 128>(cls);
}

template <int D, bool KV4, bool BF16>
cudaError_t win_decode(const WinParams& p, int cls, unsigned grid, bool cut, bool many_pieces, cudaStream_t st) {
  const cudaError_t e = win_launch<D, KV4, BF16>(p, cls, grid, st);
  if (e != cudaSuccess || !cut) return e;
  const Kv8Params& m = p;
  if (many_pieces)
    return launch_pdl(gqa_kv8_merge_kernel<D, BF16, true>, (unsigned)((int64_t)p.N * p.T_q * p.h_q * (D / 32)),
                      kMergeThreads, st, m);
  const int64_t tasks = (int64_t)p.workers * p.rows, warps = kMergeThreads / 32;
  return launch_pdl(gqa_kv8_merge_kernel<D, BF16, false>, (unsigned)((tasks + warps - 1) / warps), kMergeThreads, st, m);
}

template <int D, bool KV4>
cudaError_t win_decode_type(const WinParams& p, int cls, bool bf16, unsigned grid, bool cut, bool many, cudaStream_t st) {
  return bf16 ? win_decode<D, KV4, true>(p, cls, grid, cut, many, st) : win_decode<D, KV4, false>(p, cls, grid, cut, many, st);
}

// Tiles of a sequence that can be visible: what the table holds, or the sinks' and those that a stretch of the window and the
// other new tokens' places can touch.
int64_t most_tiles(int64_t keys, int tile, int window, int sink_tiles, int new_tokens) {
  const int64_t all = (keys + tile - 1) / tile;
  if (window == 0) return all;
  const int64_t some = sink_tiles + ((int64_t)window + new_tokens - 1 + tile - 2) / tile + 1;
  return some < all ? some : all;
}

// CTAs of a unit in the short kernel, as kv8_short_ctas: a cluster of 1, 2, 4 or 8, the fewest that give every second worker one
// tile; at most `most` tiles a worker.  0: the general kernel.  The tiles go evenly to a unit's CTAs (window
// 1024 + 4, 8 KV heads of 128, f16, a call 6.9 us with the first CTAs full, 6.2 now).  Measured (us of a replayed call, a tile for
// each worker / every second / third): that one 5.8 / 5.4 / 5.4; window 128 + 4 4.1 / 4.2 / 4.7; 300 keys over the 4-bit cache
// 5.2 / 5.3 / 5.7.
int win_short_ctas(int64_t units, int64_t seq_tiles, int sms, int groups, int most) {
  int ctas = 1;
  while (ctas < 8 && ctas * (groups / 2) < seq_tiles && units * ctas * 2 <= sms * 3 / 4) ctas *= 2;
  const int64_t here = (seq_tiles + ctas * groups - 1) / (ctas * groups);
  const int64_t there = (units * seq_tiles + sms * groups - 1) / (sms * groups);
  if (units * ctas > sms || here > most || here > there + 2) return 0;
  return ctas;
}

struct WinCall {
  const uint16_t* q;
  const void *cache, *k_pool, *v_pool;    // the 4-bit cache, or the pools
  const int32_t *tables, *lens;
  uint16_t* o;
  int N, T_q, max_blocks, num_blocks, block_size, h_q, h_kv, D;
  float scale;
  int window, sinks;
  void* ws;
  size_t ws_bytes;
  void *status, *stream;
};

gqa_status decode_impl(const WinCall& c, const gqa_options* opt_in) {
  const gqa_options opt = opt_in ? *opt_in : gqa_default_options();
  const bool kv4 = c.k_pool == nullptr && c.v_pool == nullptr, bf16 = opt.bf16 != 0;
  gqa_status s = check_rows(c.N, c.T_q, c.h_q, c.h_kv, c.D);
  if (s == GQA_OK) s = check_kv8(c.N, c.h_kv, c.D, c.max_blocks, c.num_blocks, c.block_size);
  if (s != GQA_OK) return s;
  if (!std::isfinite(c.scale) || c.window < 0 || c.sinks < 0) return GQA_ERR_INVALID_ARG;
  if ((int64_t)(c.N < kWinSeqs ? c.N : kWinSeqs) * c.T_q * c.h_q >= (int64_t(1) << 31)) return GQA_ERR_INVALID_ARG;
  if (c.N == 0) return GQA_OK;
  void* status = c.status != nullptr ? c.status : c.ws;
  if (!aligned16(c.q) || !aligned16(c.o) || !aligned16(c.ws) || !aligned16(status) || !aligned_to(c.tables, 4) ||
      !aligned_to(c.lens, 4) || (kv4 ? !aligned16(c.cache) : !aligned16(c.k_pool) || !aligned16(c.v_pool)))
    return GQA_ERR_INVALID_ARG;
  if (c.ws_bytes < kHeaderBytes) return GQA_ERR_WORKSPACE;
  const int rows = c.h_q / c.h_kv * c.T_q, cls = kv8_class(rows), groups = win_groups(kv4, c.D, cls);
  const int tile = kv4 ? win_tile_keys<true>(cls) : win_tile_keys<false>(cls);
  int sms = 0;
  if ((s = win_device(kv4, c.D, cls, bf16, &sms)) != GQA_OK) return s;
  const Kv8Layout lay = kv8_layout(sms * groups, rows, c.D);
  if (c.ws_bytes < lay.total) return GQA_ERR_WORKSPACE;
  uint8_t* wsb = static_cast<uint8_t*>(c.ws);
  WinParams p = {};
  p.cache = static_cast<const uint8_t*>(c.cache);
  p.k_pool = static_cast<const uint16_t*>(c.k_pool);
  p.v_pool = static_cast<const uint16_t*>(c.v_pool);
  p.status = static_cast<uint32_t*>(status);
  p.splits = reinterpret_cast<int4*>(wsb + lay.splits);
  p.ws_m = reinterpret_cast<float*>(wsb + lay.m);
  p.ws_l = reinterpret_cast<float*>(wsb + lay.l);
  p.ws_o = reinterpret_cast<float*>(wsb + lay.o);
  p.T_q = c.T_q; p.h_q = c.h_q; p.h_kv = c.h_kv; p.G = c.h_q / c.h_kv; p.rows = rows;
  p.max_blocks = c.max_blocks; p.num_blocks = c.num_blocks; p.block_size = c.block_size;
  p.bs_log = log2_of(c.block_size);
  p.ids_log = c.block_size < tile ? log2_of(tile) - p.bs_log : 0;
  p.causal = opt.causal ? 1 : 0;
  p.stall = opt.test_stall_cta;
  p.scale_log2 = c.scale * kLog2e;
  p.timeout_ns = wait_limit_ns(opt.timeout_us);
  // a window of all that the table holds hides nothing
  const int64_t keys = (int64_t)c.max_blocks * c.block_size;
  p.window = c.window < keys ? c.window : 0;
  p.sinks = p.window == 0 ? 0 : c.sinks;
  p.sink_tiles = (int)(((int64_t)p.sinks + tile - 1) / tile);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(c.stream);
  const int64_t seq_tiles = most_tiles(keys, tile, p.window, p.sink_tiles, p.causal ? c.T_q : 1);
  std::lock_guard<std::mutex> turn(turn_of(c.ws));
  for (int b0 = 0; b0 < c.N; b0 += kWinSeqs) {
    p.N = c.N - b0 < kWinSeqs ? c.N - b0 : kWinSeqs;
    p.q = c.q + (int64_t)b0 * c.T_q * c.h_q * c.D;
    p.o = c.o + (int64_t)b0 * c.T_q * c.h_q * c.D;
    p.block_tables = c.tables + (int64_t)b0 * c.max_blocks;
    p.seq_lens = c.lens + b0;
    // as many CTAs as there can be tiles, at most one on each SM
    const int64_t units = (int64_t)p.N * c.h_kv;
    unsigned grid = units * seq_tiles < sms ? (unsigned)(units * seq_tiles) : (unsigned)sms;
    if (units * seq_tiles / ((int64_t)grid * groups) >= (int64_t(1) << 31)) return GQA_ERR_INVALID_ARG;   // tiles of a worker
    // few units of few tiles a worker: one launch of clusters
    p.ctas = win_short_ctas(units, seq_tiles, sms, groups, kKv8Short < 32 >> p.ids_log ? kKv8Short : 32 >> p.ids_log);
    if (p.ctas > 0) grid = (unsigned)(units * p.ctas);
    p.workers = (int)grid * groups;
    const bool many = p.workers / units >= kManyPieces && units * rows * (c.D / 32) <= kMergeCtas;
    const bool cut = seq_tiles > 1 && p.ctas == 0;   // (a unit of one tile is never cut)
    p.sliced = many ? 1 : 0;
    const cudaError_t e = kv4 ? (c.D == 64 ? win_decode_type<64, true>(p, cls, bf16, grid, cut, many, st)
                                           : win_decode_type<128, true>(p, cls, bf16, grid, cut, many, st))
                              : (c.D == 64 ? win_decode_type<64, false>(p, cls, bf16, grid, cut, many, st)
                                           : win_decode_type<128, false>(p, cls, bf16, grid, cut, many, st));
    if (e != cudaSuccess) return GQA_ERR_CUDA;
  }
  return GQA_OK;
}

// ---------------------------------------------------------------- read
struct Kv4ReadParams {
  const uint8_t* cache;
  const int32_t *block_tables, *seq_lens, *begins;
  uint16_t *k_out, *v_out;
  uint32_t* status;
  int64_t out_len, most;   // rows of an output sequence, and how many of them there can be tokens for
  int num_seqs, max_blocks, num_blocks, block_size, bs_log, h_kv;
};

// One warp for 4 * RPP tokens of one head, as the kernel that reads the 8-bit cache: a lane has the 16 elements of a group
// (8 bytes of codes, one scale, 32 bytes of output), the loads of K and V of all its rows first.  Bound by its bytes, of
// which the output is four fifths.
template <int D, bool BF16>
__global__ void __launch_bounds__(kReadThreads)
gqa_kv4_read_kernel(const Kv4ReadParams a) {
  constexpr int LPR = ReadCfg<D>::LPR, RPP = ReadCfg<D>::RPP, P = ReadCfg<D>::P;
  ptx::grid_dependency_wait();
  const int lane = threadIdx.x & 31, c = lane % LPR;
  const uint32_t w = blockIdx.x * (kReadThreads / 32) + (threadIdx.x >> 5), group = w / (uint32_t)a.h_kv;
  const int g = (int)(w - group * (uint32_t)a.h_kv);
  const int64_t b = blockIdx.y, i0 = (int64_t)group * ReadCfg<D>::TOKENS;
  if (i0 >= a.most) return;
  const int cap = a.max_blocks * a.block_size;
  int len = a.seq_lens[b];
  const int begin = a.begins != nullptr ? a.begins[b] : 0;
  if (len < 0 || len > cap || begin < 0) {
    if (lane == 0) atomicOr(a.status, kDevBadInput);
    len = len > cap ? cap : len;
  }
  if (begin < 0 || begin + i0 >= len) return;
  const int bb = kv4_block_bytes(a.block_size, D), v_codes = a.block_size * (D / 2), v_scales = a.block_size * (D / 16);
  uint2 codes[2][P];
  uint32_t scale[2][P];
  bool have[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int64_t i = i0 + p * RPP + lane / LPR, tok = begin + i;
    have[p] = false;
    if (i < a.out_len && tok < len) {
      const int j = (int)((uint32_t)tok >> a.bs_log), row = (int)tok & (a.block_size - 1);
      const int id = __ldg(a.block_tables + b * a.max_blocks + j);
      have[p] = id >= 0 && id < a.num_blocks;
      if (!have[p]) atomicOr(a.status, kDevBadInput);
      const uint8_t* at = a.cache + ((int64_t)id * a.h_kv + g) * bb;
#pragma unroll
      for (int kv = 0; kv < 2; ++kv)
        if (have[p] && (kv ? a.v_out : a.k_out) != nullptr) {
          codes[kv][p] = __ldcs(reinterpret_cast<const uint2*>(at + kv * v_codes + kv4_chunk<D>(row, c >> 1) + (c & 1) * 8));
          scale[kv][p] = __ldg(at + 2 * v_codes + kv * v_scales + row * (D / 16) + c);
        }
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint16_t* out = kv ? a.v_out : a.k_out;
    if (out == nullptr) continue;
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (!have[p]) continue;
      const uint32_t s = kv4_scales(scale[kv][p], scale[kv][p], kv4_pick(0, 0));
      uint32_t y[8];
      kv4_unpack(codes[kv][p].x, *reinterpret_cast<uint32_t(*)[4]>(y));
      kv4_unpack(codes[kv][p].y, *reinterpret_cast<uint32_t(*)[4]>(y + 4));
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        y[q] = kv4_mul(y[q], s);
        if constexpr (BF16) {
          const float2 f = half2_floats(y[q]);
          y[q] = ptx::pack_bf162(f.x, f.y);
        }
      }
      const int64_t at = ((b * a.out_len + i0 + p * RPP + lane / LPR) * a.h_kv + g) * D + c * 16;
      if (!idx_ok(at + 15, a.num_seqs * a.out_len * a.h_kv * D, a.status)) continue;
      if (reinterpret_cast<uintptr_t>(out) & 31) {
        *reinterpret_cast<uint4*>(out + at) = make_uint4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<uint4*>(out + at + 8) = make_uint4(y[4], y[5], y[6], y[7]);
      } else {   // a lane's 32 bytes in one store: whole sectors
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(out + at), "r"(y[0]), "r"(y[1]),
                     "r"(y[2]), "r"(y[3]), "r"(y[4]), "r"(y[5]), "r"(y[6]), "r"(y[7])
                     : "memory");
      }
    }
  }
}

template <int D, bool BF16>
cudaError_t read_launch(const Kv4ReadParams& p, cudaStream_t st) {
  const int64_t groups = (p.most + ReadCfg<D>::TOKENS - 1) / ReadCfg<D>::TOKENS, per = kReadThreads / 32;
  const int64_t blocks = (groups * p.h_kv + per - 1) / per;
  return launch_pdl_smem(gqa_kv4_read_kernel<D, BF16>, dim3((unsigned)blocks, (unsigned)p.num_seqs), kReadThreads, 0, st, 1, p);
}

gqa_status read_impl(const void* cache, const int32_t* tables, const int32_t* lens, const int32_t* begins, uint16_t* k_out,
                     uint16_t* v_out, int N, int64_t out_len, int max_blocks, int num_blocks, int block_size, int h_kv, int D,
                     void* ws, size_t ws_bytes, void* stream, const gqa_options* opt) {
  gqa_status s = check_kv8(N, h_kv, D, max_blocks, num_blocks, block_size);
  if (s != GQA_OK) return s;
  if (out_len < 0 || out_len >= (int64_t(1) << 31)) return GQA_ERR_INVALID_ARG;
  const int64_t most = out_len < (int64_t)max_blocks * block_size ? out_len : (int64_t)max_blocks * block_size;
  if ((most / 16 + 1) * h_kv >= (int64_t(1) << 30)) return GQA_ERR_INVALID_ARG;   // warps of a sequence
  if (N == 0 || out_len == 0) return GQA_OK;
  if (k_out == nullptr && v_out == nullptr) return GQA_ERR_INVALID_ARG;
  if (!aligned16(cache) || (k_out != nullptr && !aligned16(k_out)) || (v_out != nullptr && !aligned16(v_out)) ||
      !aligned16(ws) || !aligned_to(tables, 4) || !aligned_to(lens, 4) || (begins != nullptr && !aligned_to(begins, 4)))
    return GQA_ERR_INVALID_ARG;
  if (ws_bytes < kHeaderBytes) return GQA_ERR_WORKSPACE;
  Kv4ReadParams p = {};
  p.cache = static_cast<const uint8_t*>(cache);
  p.block_tables = tables; p.seq_lens = lens; p.begins = begins;
  p.k_out = k_out; p.v_out = v_out; p.status = static_cast<uint32_t*>(ws);
  p.out_len = out_len;
  p.most = most;      // tokens past the table exist in no sequence: no warps for them
  p.num_seqs = N; p.max_blocks = max_blocks; p.num_blocks = num_blocks; p.block_size = block_size;
  p.bs_log = log2_of(block_size); p.h_kv = h_kv;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = opt != nullptr && opt->bf16;
  if (D == 64) return cuda_status(bf16 ? read_launch<64, true>(p, st) : read_launch<64, false>(p, st));
  return cuda_status(bf16 ? read_launch<128, true>(p, st) : read_launch<128, false>(p, st));
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

size_t gqa_kv4_block_bytes(int block_size, int d_head) {
  if (!block_size_ok(block_size) || (d_head != 64 && d_head != 128)) return 0;
  return (size_t)kv4_block_bytes(block_size, d_head);
}

size_t gqa_decode_window_workspace_size(int num_seqs, int T_q, int h_q, int h_kv, int d_head, int cache_layout) {
  try {
    if (cache_layout != GQA_CACHE_ROWS && cache_layout != GQA_CACHE_KV4) return 0;
    if (check_rows(num_seqs, T_q, h_q, h_kv, d_head) != GQA_OK) return 0;
    const bool kv4 = cache_layout == GQA_CACHE_KV4;
    const int rows = h_q / h_kv * T_q, cls = kv8_class(rows);
    int sms = 0;
    if (win_device(kv4, d_head, cls, false, &sms) != GQA_OK) return 0;
    return kv8_layout(sms * win_groups(kv4, d_head, cls), rows, d_head).total;
  } catch (...) {
    return 0;
  }
}

gqa_status gqa_decode_kv4(const uint16_t* q, const void* cache, const int32_t* block_tables, const int32_t* seq_lens,
                          uint16_t* o, int num_seqs, int T_q, int max_blocks_per_seq, int num_blocks, int block_size, int h_q,
                          int h_kv, int d_head, float scale, int window, int sinks, void* workspace, size_t ws_bytes,
                          void* status, void* stream, const gqa_options* opt) {
  try {
    return decode_impl({q, cache, nullptr, nullptr, block_tables, seq_lens, o, num_seqs, T_q, max_blocks_per_seq, num_blocks,
                        block_size, h_q, h_kv, d_head, scale, window, sinks, workspace, ws_bytes, status, stream}, opt);
  } catch (...) {
    return GQA_ERR_CUDA;
  }
}

gqa_status gqa_decode_window(const uint16_t* q, const uint16_t* k_pool, const uint16_t* v_pool, const int32_t* block_tables,
                             const int32_t* seq_lens, uint16_t* o, int num_seqs, int T_q, int max_blocks_per_seq,
                             int num_blocks, int block_size, int h_q, int h_kv, int d_head, float scale, int window, int sinks,
                             void* workspace, size_t ws_bytes, void* status, void* stream, const gqa_options* opt) {
  try {
    if (num_seqs > 0 && (k_pool == nullptr || v_pool == nullptr)) return GQA_ERR_INVALID_ARG;
    return decode_impl({q, nullptr, k_pool, v_pool, block_tables, seq_lens, o, num_seqs, T_q, max_blocks_per_seq, num_blocks,
                        block_size, h_q, h_kv, d_head, scale, window, sinks, workspace, ws_bytes, status, stream}, opt);
  } catch (...) {
    return GQA_ERR_CUDA;
  }
}

gqa_status gqa_kv4_read(const void* cache, const int32_t* block_tables, const int32_t* seq_lens, const int32_t* begins,
                        uint16_t* k_out, uint16_t* v_out, int num_seqs, int64_t out_len, int max_blocks_per_seq, int num_blocks,
                        int block_size, int h_kv, int d_head, void* workspace, size_t ws_bytes, void* stream,
                        const gqa_options* opt) {
  try {
    return read_impl(cache, block_tables, seq_lens, begins, k_out, v_out, num_seqs, out_len, max_blocks_per_seq, num_blocks,
                     block_size, h_kv, d_head, workspace, ws_bytes, stream, opt);
  } catch (...) {
    return GQA_ERR_CUDA;
  }
}

}  // extern "C"
