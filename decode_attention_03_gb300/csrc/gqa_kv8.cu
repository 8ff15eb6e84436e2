// Host side of gqa_append, gqa_decode_kv8 and gqa_kv8_read.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>
#include <mutex>

#include "../../include/gqa_decode.h"
#include "gqa_cache_host.cuh"
#include "gqa_kv8.cuh"
#include "gqa_kv8_decode.cuh"

namespace gqa {
namespace {

// ---------------------------------------------------------------- per-device state
struct Kv8Device {
  int sms = 0;
  void* status = nullptr;     // g_status on this device
  bool ready[2][6][2] = {};   // [d index][row class][bf16]: the kernel's shared memory is allowed
};
constexpr int kMaxDevices = 64;
__device__ __align__(256) unsigned char g_status[kHeaderBytes];   // the library's own status word, zero from the start
std::mutex g_mu;
Kv8Device g_kv8[kMaxDevices];

// SMs of the current device, with g_mu held by the caller
gqa_status device_locked(Kv8Device** out) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return GQA_ERR_CUDA;
  Kv8Device& d = g_kv8[dev];
  if (d.sms == 0 && cudaDeviceGetAttribute(&d.sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
    d.sms = 0;
    return GQA_ERR_CUDA;
  }
  *out = &d;
  return GQA_OK;
}

// Address of the current device's g_status.  The lookup is no work on a stream, but may load the module: allowed while this
// thread captures a graph.
void* device_status() {
  std::lock_guard<std::mutex> lock(g_mu);
  Kv8Device* d = nullptr;
  if (device_locked(&d) != GQA_OK) return nullptr;
  if (d->status == nullptr) {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return nullptr;
    void* p = nullptr;
    if (cudaGetSymbolAddress(&p, g_status) == cudaSuccess) d->status = p;
    if (cudaThreadExchangeStreamCaptureMode(&mode) != cudaSuccess) return nullptr;
  }
  return d->status;
}

// ---------------------------------------------------------------- append
gqa_status append_impl(const gqa_append_args& a, const uint8_t* pair_axes, int num_axes, void* ws, size_t ws_bytes,
                       void* stream) {
  if (num_axes < 1 || num_axes > kAppendAxes || (num_axes > 1 && pair_axes == nullptr)) return GQA_ERR_INVALID_ARG;
  if (a.num_tokens < 0 || a.h_q < 0 || a.h_kv < 1 || a.num_blocks < 0) return GQA_ERR_INVALID_ARG;
  if (a.h_q > 32767 || a.h_kv > 16383 || a.h_q % a.h_kv != 0) return GQA_ERR_INVALID_ARG;   // sets fit a grid's y
  if (a.d_head != 64 && a.d_head != 128) return GQA_ERR_UNSUPPORTED;
  if (!block_size_ok(a.block_size) || (int64_t)a.num_blocks * a.block_size >= (int64_t(1) << 31))
    return GQA_ERR_INVALID_ARG;
  if ((a.cache_layout < GQA_CACHE_ROWS || a.cache_layout > GQA_CACHE_KV8) && a.cache_layout != GQA_CACHE_KV4) return GQA_ERR_INVALID_ARG;
  if (!std::isfinite(a.eps) || a.eps < 0.f) return GQA_ERR_INVALID_ARG;
  if (a.cos_sin != nullptr &&
      (a.rot_dim < 8 || a.rot_dim > a.d_head || a.rot_dim % 8 != 0 || a.max_position < 1 || !aligned16(a.cos_sin) ||
       !aligned_to(a.positions, 4)))
    return GQA_ERR_INVALID_ARG;
  const int64_t qn = (int64_t)a.h_q * a.d_head, kn = (int64_t)a.h_kv * a.d_head;
  if (a.num_tokens > 0) {
    if (a.k_stride < kn || a.v_stride < kn || a.k_stride % 8 || a.v_stride % 8) return GQA_ERR_INVALID_ARG;
    if (a.h_q > 0 && (a.q_stride < qn || a.q_out_stride < qn || a.q_stride % 8 || a.q_out_stride % 8 ||
                      !aligned16(a.q) || !aligned16(a.q_out)))
      return GQA_ERR_INVALID_ARG;
    if (!aligned16(a.k) || !aligned16(a.v) || !aligned_to(a.slots, 8) || !aligned16(a.k_cache) ||
        (a.cache_layout < GQA_CACHE_KV8 && !aligned16(a.v_cache)))
      return GQA_ERR_INVALID_ARG;
    if ((a.q_weight != nullptr && !aligned16(a.q_weight)) || (a.k_weight != nullptr && !aligned16(a.k_weight)))
      return GQA_ERR_INVALID_ARG;
    if (!aligned16(ws)) return GQA_ERR_INVALID_ARG;
    if (ws_bytes < kHeaderBytes) return GQA_ERR_WORKSPACE;
  }
  if (a.num_tokens == 0) return GQA_OK;
  int sms = 0;
  {
    std::lock_guard<std::mutex> lock(g_mu);
    Kv8Device* dev = nullptr;
    const gqa_status s = device_locked(&dev);
    if (s != GQA_OK) return s;
    sms = dev->sms;
  }
  AppendParams p = {};
  p.q = a.q; p.k = a.k; p.v = a.v; p.q_out = a.q_out;
  p.q_stride = a.q_stride; p.k_stride = a.k_stride; p.v_stride = a.v_stride; p.q_out_stride = a.q_out_stride;
  p.q_weight = a.q_weight; p.k_weight = a.k_weight;
  p.cos_sin = a.cos_sin; p.positions = a.positions; p.slots = a.slots;
  p.k_cache = a.k_cache; p.v_cache = a.v_cache;
  p.status = static_cast<uint32_t*>(ws);
  p.num_tokens = a.num_tokens; p.h_q = a.h_q; p.h_kv = a.h_kv;
  p.max_position = a.max_position; p.rot_dim = a.rot_dim; p.interleaved = a.interleaved ? 1 : 0;
  p.num_blocks = a.num_blocks; p.block_size = a.block_size; p.bs_log = log2_of(a.block_size);
  p.eps = a.eps;
  p.pair_axes = pair_axes; p.num_axes = num_axes;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a.d_head == 64)
    return cuda_status(a.bf16 ? append_run<64, true>(p, a.cache_layout, sms, st) : append_run<64, false>(p, a.cache_layout, sms, st));
  return cuda_status(a.bf16 ? append_run<128, true>(p, a.cache_layout, sms, st) : append_run<128, false>(p, a.cache_layout, sms, st));
}

// ---------------------------------------------------------------- decode
template <int D, int NT, int RG, bool BF16>
cudaError_t kv8_prepare() {
  constexpr int bytes = Kv8Cfg<D, NT, RG>::SMEM;
  const cudaError_t e = cudaFuncSetAttribute(gqa_decode_kv8_kernel<D, NT, RG, BF16>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(gqa_decode_kv8_short_kernel<D, NT, RG, BF16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              bytes);
}

template <int D, bool BF16>
cudaError_t kv8_prepare_class(int cls) {
  switch (cls) {
    case 0: return kv8_prepare<D, 1, 1, BF16>();
    case 1: return kv8_prepare<D, 2, 1, BF16>();
    case 2: return kv8_prepare<D, 3, 1, BF16>();
    case 3: return kv8_prepare<D, 4, 1, BF16>();
    case 4: return kv8_prepare<D, 3, 2, BF16>();
    default: return kv8_prepare<D, 4, 2, BF16>();
  }
}

// SMs of the current device; the kernel of (D, cls, bf16) is ready to launch on it
gqa_status kv8_device(int D, int cls, int bf16, int* sms) {
  std::lock_guard<std::mutex> lock(g_mu);
  Kv8Device* dev = nullptr;
  const gqa_status s = device_locked(&dev);
  if (s != GQA_OK) return s;
  bool& ready = dev->ready[D == 64 ? 0 : 1][cls][bf16];
  if (!ready) {
    const cudaError_t e = D == 64 ? (bf16 ? kv8_prepare_class<64, true>(cls) : kv8_prepare_class<64, false>(cls))
                                  : (bf16 ? kv8_prepare_class<128, true>(cls) : kv8_prepare_class<128, false>(cls));
    if (e != cudaSuccess) return GQA_ERR_CUDA;
    ready = true;
  }
  *sms = dev->sms;
  return GQA_OK;
}

template <int D, int NT, int RG, bool BF16>
cudaError_t kv8_launch(const Kv8Params& p, unsigned grid, cudaStream_t st) {
  constexpr int bytes = Kv8Cfg<D, NT, RG>::SMEM;
  if (p.ctas > 0)
    return launch_pdl_smem(gqa_decode_kv8_short_kernel<D, NT, RG, BF16>, grid, kKv8Threads, bytes, st, p.ctas, p);
  return launch_pdl_smem(gqa_decode_kv8_kernel<D, NT, RG, BF16>, grid, kKv8Threads, bytes, st, 1, p);
}

template <int D, bool BF16>
cudaError_t kv8_decode(const Kv8Params& p, int cls, unsigned grid, bool cut, bool many_pieces, cudaStream_t st) {
  cudaError_t e;
  switch (cls) {
    case 0: e = kv8_launch<D, 1, 1, BF16>(p, grid, st); break;
    case 1: e = kv8_launch<D, 2, 1, BF16>(p, grid, st); break;
    case 2: e = kv8_launch<D, 3, 1, BF16>(p, grid, st); break;
    case 3: e = kv8_launch<D, 4, 1, BF16>(p, grid, st); break;
    case 4: e = kv8_launch<D, 3, 2, BF16>(p, grid, st); break;
    default: e = kv8_launch<D, 4, 2, BF16>(p, grid, st); break;
  }
  if (e != cudaSuccess || !cut) return e;
  if (many_pieces)
    return launch_pdl(gqa_kv8_merge_kernel<D, BF16, true>, (unsigned)((int64_t)p.N * p.T_q * p.h_q * (D / 32)),
                      kMergeThreads, st, p);
  const int64_t tasks = (int64_t)p.workers * p.rows, warps = kMergeThreads / 32;
  return launch_pdl(gqa_kv8_merge_kernel<D, BF16, false>, (unsigned)((tasks + warps - 1) / warps), kMergeThreads, st, p);
}

gqa_status decode_kv8_impl(const uint16_t* q, const void* cache, const int32_t* tables, const int32_t* lens,
                           uint16_t* o, int N, int T_q, int max_blocks, int num_blocks, int block_size, int h_q,
                           int h_kv, int D, float scale, void* ws, size_t ws_bytes, void* status, void* stream,
                           const gqa_options* opt_in) {
  const gqa_options opt = opt_in ? *opt_in : gqa_default_options();
  gqa_status s = check_rows(N, T_q, h_q, h_kv, D);
  if (s == GQA_OK) s = check_kv8(N, h_kv, D, max_blocks, num_blocks, block_size);
  if (s != GQA_OK) return s;
  if (!std::isfinite(scale)) return GQA_ERR_INVALID_ARG;
  if ((int64_t)(N < kKv8Seqs ? N : kKv8Seqs) * T_q * h_q >= (int64_t(1) << 31)) return GQA_ERR_INVALID_ARG;
  if (N == 0) return GQA_OK;
  if (!aligned16(q) || !aligned16(cache) || !aligned16(o) || !aligned16(ws) || !aligned16(status) ||
      !aligned_to(tables, 4) || !aligned_to(lens, 4))
    return GQA_ERR_INVALID_ARG;
  if (ws_bytes < kHeaderBytes) return GQA_ERR_WORKSPACE;
  const int rows = h_q / h_kv * T_q, cls = kv8_class(rows), bf16 = opt.bf16 ? 1 : 0;
  int sms = 0;
  if ((s = kv8_device(D, cls, bf16, &sms)) != GQA_OK) return s;
  const Kv8Layout lay = kv8_layout(sms * kv8_groups(cls), rows, D);
  if (ws_bytes < lay.total) return GQA_ERR_WORKSPACE;
  uint8_t* wsb = static_cast<uint8_t*>(ws);
  Kv8Params p = {};
  p.cache = static_cast<const uint8_t*>(cache);
  p.status = static_cast<uint32_t*>(status);
  p.splits = reinterpret_cast<int4*>(wsb + lay.splits);
  p.ws_m = reinterpret_cast<float*>(wsb + lay.m);
  p.ws_l = reinterpret_cast<float*>(wsb + lay.l);
  p.ws_o = reinterpret_cast<float*>(wsb + lay.o);
  p.T_q = T_q; p.h_q = h_q; p.h_kv = h_kv; p.G = h_q / h_kv; p.rows = rows;
  p.max_blocks = max_blocks; p.num_blocks = num_blocks; p.block_size = block_size;
  p.bs_log = log2_of(block_size);
  p.causal = opt.causal ? 1 : 0;
  p.stall = opt.test_stall_cta;
  p.scale_log2 = scale * kLog2e;
  p.timeout_ns = wait_limit_ns(opt.timeout_us);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int64_t seq_tiles = ((int64_t)max_blocks * block_size + kKv8Keys - 1) / kKv8Keys;
  std::lock_guard<std::mutex> turn(turn_of(ws));
  for (int b0 = 0; b0 < N; b0 += kKv8Seqs) {
    p.N = N - b0 < kKv8Seqs ? N - b0 : kKv8Seqs;
    p.q = q + (int64_t)b0 * T_q * h_q * D;
    p.o = o + (int64_t)b0 * T_q * h_q * D;
    p.block_tables = tables + (int64_t)b0 * max_blocks;
    p.seq_lens = lens + b0;
    // as many CTAs as there can be tiles, at most one on each SM
    const int64_t units = (int64_t)p.N * h_kv;
    unsigned grid = units * seq_tiles < sms ? (unsigned)(units * seq_tiles) : (unsigned)sms;
    if (units * seq_tiles / ((int64_t)grid * kv8_groups(cls)) >= (int64_t(1) << 31)) return GQA_ERR_INVALID_ARG;   // tiles of a worker
    // few units that the table bounds to kKv8Short tiles a worker: one launch of clusters
    p.ctas = kv8_short_ctas(units, seq_tiles, sms, kv8_groups(cls));
    if (p.ctas > 0) grid = (unsigned)(units * p.ctas);
    p.workers = (int)grid * kv8_groups(cls);
    // pieces of a unit: about workers / units + 1 when the sequences are alike
    const bool many = p.workers / units >= kManyPieces && units * rows * (D / 32) <= kMergeCtas;
    const bool cut = seq_tiles > 1 && p.ctas == 0;   // (a unit of one tile is never cut)
    p.sliced = many ? 1 : 0;
    const cudaError_t e = D == 64 ? (bf16 ? kv8_decode<64, true>(p, cls, grid, cut, many, st)
                                          : kv8_decode<64, false>(p, cls, grid, cut, many, st))
                                  : (bf16 ? kv8_decode<128, true>(p, cls, grid, cut, many, st)
                                          : kv8_decode<128, false>(p, cls, grid, cut, many, st));
    if (e != cudaSuccess) return GQA_ERR_CUDA;
  }
  return GQA_OK;
}

// ---------------------------------------------------------------- read
template <int D, bool BF16>
cudaError_t read_launch(const Kv8ReadParams& p, cudaStream_t st) {
  const int64_t groups = (p.most + ReadCfg<D>::TOKENS - 1) / ReadCfg<D>::TOKENS, per = kReadThreads / 32;
  const int64_t blocks = (groups * p.h_kv + per - 1) / per;
  return launch_pdl_smem(gqa_kv8_read_kernel<D, BF16>, dim3((unsigned)blocks, (unsigned)p.num_seqs), kReadThreads, 0, st,
                         1, p);
}

gqa_status read_impl(const void* cache, const int32_t* tables, const int32_t* lens, const int32_t* begins,
                     uint16_t* k_out, uint16_t* v_out, int N, int64_t out_len, int max_blocks, int num_blocks,
                     int block_size, int h_kv, int D, void* ws, size_t ws_bytes, void* stream,
                     const gqa_options* opt) {
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
  Kv8ReadParams p = {};
  p.cache = static_cast<const uint8_t*>(cache);
  p.block_tables = tables; p.seq_lens = lens; p.begins = begins;
  p.k_out = k_out; p.v_out = v_out; p.status = static_cast<uint32_t*>(ws);
  p.out_len = out_len;
  p.num_seqs = N; p.max_blocks = max_blocks; p.num_blocks = num_blocks; p.block_size = block_size;
  p.bs_log = log2_of(block_size); p.h_kv = h_kv;
  // tokens past the table exist in no sequence: no warps for them
  p.most = most;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const bool bf16 = opt != nullptr && opt->bf16;
  if (D == 64) return cuda_status(bf16 ? read_launch<64, true>(p, st) : read_launch<64, false>(p, st));
  return cuda_status(bf16 ? read_launch<128, true>(p, st) : read_launch<128, false>(p, st));
}

}  // namespace
}  // namespace gqa

using namespace gqa;

extern "C" {

size_t gqa_kv8_block_bytes(int block_size, int d_head) {
  if (!block_size_ok(block_size) || (d_head != 64 && d_head != 128)) return 0;
  return (size_t)kv8_block_bytes(block_size, d_head);
}

gqa_status gqa_append(const gqa_append_args* args, void* workspace, size_t ws_bytes, void* stream) {
  try {
    if (args == nullptr) return GQA_ERR_INVALID_ARG;
    return append_impl(*args, nullptr, 1, workspace, ws_bytes, stream);
  } catch (...) {
    return GQA_ERR_CUDA;
  }
}

gqa_status gqa_append_axes(const gqa_append_args* args, const uint8_t* pair_axes, int num_axes, void* workspace,
                           size_t ws_bytes, void* stream) {
  try {
    if (args == nullptr) return GQA_ERR_INVALID_ARG;
    return append_impl(*args, pair_axes, num_axes, workspace, ws_bytes, stream);
  } catch (...) {
    return GQA_ERR_CUDA;
  }
}

size_t gqa_decode_kv8_workspace_size(int num_seqs, int T_q, int h_q, int h_kv, int d_head) {
  try {
    if (check_rows(num_seqs, T_q, h_q, h_kv, d_head) != GQA_OK) return 0;
    const int rows = h_q / h_kv * T_q, cls = kv8_class(rows);
    int sms = 0;
    if (kv8_device(d_head, cls, 0, &sms) != GQA_OK) return 0;
    return kv8_layout(sms * kv8_groups(cls), rows, d_head).total;
  } catch (...) {
    return 0;
  }
}

gqa_status gqa_decode_kv8(const uint16_t* q, const void* cache, const int32_t* block_tables, const int32_t* seq_lens,
                          uint16_t* o, int num_seqs, int T_q, int max_blocks_per_seq, int num_blocks, int block_size,
                          int h_q, int h_kv, int d_head, float scale, void* workspace, size_t ws_bytes, void* stream,
                          const gqa_options* opt) {
  try {
    return decode_kv8_impl(q, cache, block_tables, seq_lens, o, num_seqs, T_q, max_blocks_per_seq, num_blocks,
                           block_size, h_q, h_kv, d_head, scale, workspace, ws_bytes, workspace, stream, opt);
  } catch (...) {
    return GQA_ERR_CUDA;
  }
}

gqa_status gqa_decode_kv8_status(const uint16_t* q, const void* cache, const int32_t* block_tables,
                                 const int32_t* seq_lens, uint16_t* o, int num_seqs, int T_q, int max_blocks_per_seq,
                                 int num_blocks, int block_size, int h_q, int h_kv, int d_head, float scale,
                                 void* workspace, size_t ws_bytes, void* status, void* stream, const gqa_options* opt) {
  try {
    return decode_kv8_impl(q, cache, block_tables, seq_lens, o, num_seqs, T_q, max_blocks_per_seq, num_blocks,
                           block_size, h_q, h_kv, d_head, scale, workspace, ws_bytes, status, stream, opt);
  } catch (...) {
    return GQA_ERR_CUDA;
  }
}

void* gqa_device_status(void) {
  try {
    return device_status();
  } catch (...) {
    return nullptr;
  }
}

gqa_status gqa_kv8_read(const void* cache, const int32_t* block_tables, const int32_t* seq_lens, const int32_t* begins,
                        uint16_t* k_out, uint16_t* v_out, int num_seqs, int64_t out_len, int max_blocks_per_seq,
                        int num_blocks, int block_size, int h_kv, int d_head, void* workspace, size_t ws_bytes,
                        void* stream, const gqa_options* opt) {
  try {
    return read_impl(cache, block_tables, seq_lens, begins, k_out, v_out, num_seqs, out_len, max_blocks_per_seq,
                     num_blocks, block_size, h_kv, d_head, workspace, ws_bytes, stream, opt);
  } catch (...) {
    return GQA_ERR_CUDA;
  }
}

}  // extern "C"
