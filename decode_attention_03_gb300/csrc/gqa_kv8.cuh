// The 8-bit cache (kv8) and the kernels that fill a cache and read this one back.
//
// A (block, head) of the cache is one contiguous stretch of block_size * (2 D + 2) bytes (a multiple
// of 16): K codes, V codes, K exponents, V exponents.  So one plain bulk copy brings everything that
// attention needs of a block's head into shared memory, and because the 16-byte chunks of a row are
// stored where the bank swizzle wants them, the copy lands ready for conflict-free ldmatrix.
// Scales are powers of two, one byte for each row: an e4m3 code has its own exponent, so a finer scale
// would not make it more exact, and multiplying by a power of two rounds nothing in either direction.
#pragma once
#include <cuda_fp8.h>

#include "gqa_kernels.cuh"
#include "gqa_kv4.cuh"

namespace gqa {

constexpr int kAppendThreads = 256;
constexpr int kAppendCtas = 4;    // on an SM
constexpr int kAppendIters = 4;   // groups of heads of a warp at most
constexpr int kAppendRun = 4;     // tokens of a warp at most
constexpr int kAppendAxes = 32;   // position axes at most: a lane each
constexpr int kVllmShift = 16;    // tokens from which a CTA looks where its eights begin (fewer: a load's time is not worth it)
constexpr int kReadThreads = 256;

__host__ __device__ constexpr int kv8_block_bytes(int block_size, int D) { return block_size * (2 * D + 2); }

// byte offset, among a (block, head)'s K or V codes, of 16-byte chunk c of row r
template <int D>
__host__ __device__ constexpr int kv8_chunk(int r, int c) {
  return r * D + ((c ^ (D == 128 ? (r & 7) : ((r >> 1) & 3))) << 4);
}

// 2^(e - 127) of an exponent byte (1..254)
__device__ __forceinline__ float kv8_scale(uint32_t e) { return __uint_as_float(e << 23); }

// exponent byte of a row with max|x| = amax: k + 127, k the smallest integer with amax <= 448 * 2^k.
// 448 = 1.75 * 2^8, so amax = 1.m * 2^E needs k = E - 8, and one more where 1.m > 1.75.
__device__ __forceinline__ int kv8_exponent(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = (int)(b >> 23) - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < 1 ? 1 : e;
}

// four codes of x[0..3] * inv, nearest even (|x| * inv <= 448; infinities become 448, NaN stays)
__device__ __forceinline__ uint32_t kv8_codes(const float* x, float inv) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1] * inv), "f"(x[0] * inv));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3] * inv), "f"(x[2] * inv));
  return (uint32_t)lo | ((uint32_t)hi << 16);
}

// two codes as exact f16 values
__device__ __forceinline__ uint32_t kv8_halves(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return h;
}

__device__ __forceinline__ float2 half2_floats(uint32_t h) { return __half22float2(*reinterpret_cast<__half2*>(&h)); }

// two fp32 operations in one instruction
struct Two {
  uint64_t v;
};
__device__ __forceinline__ Two two(float lo, float hi) {
  Two t;
  asm("mov.b64 %0, {%1, %2};" : "=l"(t.v) : "f"(lo), "f"(hi));
  return t;
}
__device__ __forceinline__ float2 split(Two t) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(t.v));
  return f;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d.v) : "l"(a.v), "l"(b.v));
  return d;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return d;
}

template <bool BF16>
__device__ __forceinline__ void unpack4(uint2 r, float* x) {
  if constexpr (BF16) {
    x[0] = __uint_as_float(r.x << 16);
    x[1] = __uint_as_float(r.x & 0xffff0000u);
    x[2] = __uint_as_float(r.y << 16);
    x[3] = __uint_as_float(r.y & 0xffff0000u);
  } else {
    const float2 a = half2_floats(r.x), b = half2_floats(r.y);
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
  }
}

// =====================================================================================
// new tokens into a paged cache
// =====================================================================================
struct AppendParams {
  const uint16_t *q, *k, *v;
  uint16_t* q_out;
  int64_t q_stride, k_stride, v_stride, q_out_stride;
  const uint16_t *q_weight, *k_weight;
  const float* cos_sin;
  const int32_t* positions;
  const int64_t* slots;
  void *k_cache, *v_cache;
  uint32_t* status;
  int num_tokens, h_q, h_kv, max_position, rot_dim, interleaved, num_blocks, block_size, bs_log, q_sets, k_sets, iters, run;
  float eps;
  const uint8_t* pair_axes;   // the axis of each of the rot_dim / 2 pairs, or NULL: all on axis 0
  int num_axes;               // rows of positions
};

// CW neighbouring 16-bit elements: one 8- or 16-byte access
template <int CW>
struct Chunk {
  uint32_t w[CW / 2];
};

template <int CW>
__device__ __forceinline__ Chunk<CW> load_chunk(const uint16_t* p) {
  Chunk<CW> c;
  if constexpr (CW == 8) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    c.w[0] = v.x; c.w[1] = v.y; c.w[2] = v.z; c.w[3] = v.w;
  } else {
    const uint2 v = *reinterpret_cast<const uint2*>(p);
    c.w[0] = v.x; c.w[1] = v.y;
  }
  return c;
}

// the same into shared memory, asynchronously
template <int CW>
__device__ __forceinline__ void copy_chunk(Chunk<CW>* to, const uint16_t* from) {
  if constexpr (CW == 8)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(to)), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(ptx::smem_u32(to)), "l"(from) : "memory");
}

// all groups of copies but the last n - 1 are there
__device__ __forceinline__ void wait_copies(int n) {
  switch (n) {
    case 1: asm volatile("cp.async.wait_group 0;" ::: "memory"); break;
    case 2: asm volatile("cp.async.wait_group 1;" ::: "memory"); break;
    case 3: asm volatile("cp.async.wait_group 2;" ::: "memory"); break;
    default: asm volatile("cp.async.wait_group 3;" ::: "memory"); break;
  }
}

template <int CW>
__device__ __forceinline__ void store_chunk(uint16_t* p, const Chunk<CW>& c) {
  if constexpr (CW == 8) *reinterpret_cast<uint4*>(p) = make_uint4(c.w[0], c.w[1], c.w[2], c.w[3]);
  else *reinterpret_cast<uint2*>(p) = make_uint2(c.w[0], c.w[1]);
}

template <bool BF16, int CW>
__device__ __forceinline__ void unpack_chunk(const Chunk<CW>& c, float* x) {
#pragma unroll
  for (int i = 0; i < CW / 2; i += 2) unpack4<BF16>(make_uint2(c.w[i], c.w[i + 1]), x + 2 * i);
}

template <bool BF16, int CW>
__device__ __forceinline__ Chunk<CW> pack_chunk(const float* x) {
  Chunk<CW> c;
#pragma unroll
  for (int i = 0; i < CW / 2; ++i) c.w[i] = Elem<BF16>::pack(x[2 * i], x[2 * i + 1]);
  return c;
}

// n consecutive floats of shared memory, aligned to 8 n bytes or 16
template <int n>
__device__ __forceinline__ void shared_floats(float* x, const float* p) {
  if constexpr (n % 4 == 0) {
#pragma unroll
    for (int i = 0; i < n; i += 4) {
      const float4 v = *reinterpret_cast<const float4*>(p + i);
      x[i] = v.x; x[i + 1] = v.y; x[i + 2] = v.z; x[i + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < n; i += 2) {
      const float2 v = *reinterpret_cast<const float2*>(p + i);
      x[i] = v.x; x[i + 1] = v.y;
    }
  }
}

// The values of a CTA's tokens into vLLM's value cache, where a token's elements lie block_size apart: a warp takes 64
// columns of a head of eight tokens, which mostly fill eight neighbouring rows of a block, so that a column's eight are one
// 16-byte store.  Where a prompt begins inside such rows the eights are shifted to them; those that reach over the CTA's
// tokens are then written by its neighbour too, with the same bytes.  8192 tokens of 32 + 8 + 8 heads of 128, block 16: 38.2 us
// instead of 118.5 with a store for each element; from row 3 on 41.6, without the shift 87.3.
template <int D, int HPW>
__device__ __forceinline__ void append_vllm_values(const AppendParams& a, int set) {
  constexpr int WARPS = kAppendThreads / 32, PARTS = D / 64;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h0 = set * (a.iters * HPW), heads = min(a.iters * HPW, a.h_kv - h0);
  if (a.cos_sin != nullptr && a.pair_axes != nullptr) {      // a pair on an axis that is none: no token is taken
    bool bad = false;
    for (int i = lane; i < a.rot_dim / 2; i += 32) bad |= a.pair_axes[i] >= (uint32_t)a.num_axes;
    if (__any_sync(0xffffffffu, bad)) {
      if (threadIdx.x == 0) atomicOr(a.status, kDevBadInput);
      return;
    }
  }
  const int64_t first = (int64_t)blockIdx.x * (8 * a.run);
  const int64_t end = min(first + 8 * a.run, (int64_t)a.num_tokens);       // the CTA's tokens
  int shift = 0;
  if (end - first >= 2 && a.num_tokens >= kVllmShift) {
    const int64_t s0 = a.slots[first];
    if (s0 >= 0 && a.slots[first + 1] == s0 + 1) shift = (int)(s0 & 7);
  }
  const int octets = (int)((end - first + shift + 7) / 8), per = heads * PARTS;
  const int64_t rows = (int64_t)a.num_blocks * a.block_size, size = rows * a.h_kv * D;
  uint16_t* cache = reinterpret_cast<uint16_t*>(a.v_cache);
  for (int i = warp; i < octets * per; i += WARPS) {
    const int oct = i / per, part = i - oct * per, h = h0 + part / PARTS, d = part % PARTS * 64 + 2 * lane;
    const int64_t t0 = first - shift + 8 * oct;
    uint32_t x[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      x[j] = t0 + j >= 0 && t0 + j < a.num_tokens
                 ? __ldg(reinterpret_cast<const uint32_t*>(a.v + (t0 + j) * a.v_stride + h * D + d)) : 0u;
    // lane j < 8: where token j goes, or -1
    const bool there = lane < 8 && t0 + lane >= 0 && t0 + lane < a.num_tokens;
    int64_t slot = there ? a.slots[t0 + lane] : -1;
    bool bad = slot >= rows;
    if (a.cos_sin != nullptr && there)
      for (int axis = 0; axis < a.num_axes; ++axis) {
        const int pos = a.positions[(int64_t)axis * a.num_tokens + t0 + lane];
        bad |= pos < 0 || pos >= a.max_position;
      }
    if (bad) {
      atomicOr(a.status, kDevBadInput);
      slot = -1;
    }
    const int s = slot < 0 ? -1 : (int)slot, s0 = __shfl_sync(0xffffffffu, s, 0);
    const uint32_t follow = __ballot_sync(0xffffffffu, s >= 0 && s == s0 + lane);
    if ((follow & 0xffu) == 0xffu && (s0 & 7) == 0) {
      const int64_t at = (((int64_t)(s0 >> a.bs_log) * a.h_kv + h) * D + d) * a.block_size + (s0 & (a.block_size - 1));
      if (!idx_ok(at + a.block_size + 7, size, a.status)) continue;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t pick = k == 0 ? 0x5410 : 0x7632;
        *reinterpret_cast<uint4*>(cache + at + k * a.block_size) =
            make_uint4(__byte_perm(x[0], x[1], pick), __byte_perm(x[2], x[3], pick), __byte_perm(x[4], x[5], pick),
                       __byte_perm(x[6], x[7], pick));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int sj = __shfl_sync(0xffffffffu, s, j);
        const int64_t at = (((int64_t)(sj >> a.bs_log) * a.h_kv + h) * D + d) * a.block_size + (sj & (a.block_size - 1));
        if (sj < 0 || t0 + j < first || t0 + j >= end || !idx_ok(at + a.block_size, size, a.status)) continue;
        cache[at] = (uint16_t)x[j];
        cache[at + a.block_size] = (uint16_t)(x[j] >> 16);
      }
    }
  }
}

// Where the CW elements of a head from element e on are: (lane of the head's D/(2 CW) << 1) | which of its two chunks.
template <int D, int CW>
__device__ __forceinline__ int append_holder(int e, int rot) {
  const bool turned = e < rot;
  const int half = turned ? rot / 2 : (D - rot) / 2;
  const int i = turned ? e : e - rot, j = i >= half;
  return (((turned ? 0 : rot / 2) + i - j * half) / CW << 1) | j;
}

// A head's D elements lie on D/(2 CW) lanes, each with two chunks of CW: elements CW s.. and rot/2 + CW s.. for
// the lanes s < rot/(2 CW) that rotate, so that both elements of every rotated pair (i, i + rot/2) are in one
// thread and the rotation needs no exchange; the rest of the head (rot..D) is cut the same way.  A warp takes
// heads of one kind (queries, keys or values): 32/(D/(2 CW)) at a time, up to a.iters times for each of a.run tokens.
// Heads are copied to the threads' own places in shared memory a token ahead, a token's cosines and sines with
// its first group, so that the next token is on its way while this one is worked on.  Bound by its bytes, the
// heads read and written once, when there are many tokens; the sums of squares and maxima go through log2 of
// the lanes' number of shuffles.  CW = 8 (16-byte accesses) where rot/2 is a multiple of 8, else 4.
// 16384 tokens of 64 + 8 + 8 heads of 128 take 105.3 us (6.45 TB/s; a copy 6.69); 110.5 with one token a warp,
// 117.9 with five CTAs an SM (48 registers) instead of four (64).
// AXES: pairs turned by positions of several axes, a.pair_axes: 16384 tokens of text and pictures 103.3 us.
// Into the 4-bit cache (LAYOUT 4) a lane's chunks find the other elements of their sixteen by shuffles; three CTAs an SM, as
// four have too few registers for it (8192 tokens of 32 + 8 + 8 heads, with a read-back: 59.3 us instead of 61.3).
template <int D, bool BF16, int CW, bool PAIRS, int LAYOUT, bool AXES>
__global__ void __launch_bounds__(kAppendThreads, LAYOUT == 4 ? 3 : kAppendCtas)
gqa_append_kernel(const AppendParams a) {
  constexpr int LPH = D / (2 * CW), HPW = 32 / LPH, WARPS = kAppendThreads / 32;
  __shared__ __align__(16) Chunk<CW> stage[kAppendIters][2][kAppendThreads];   // a thread's own places
  __shared__ __align__(16) float turn_rows[WARPS][2][D];                       // a warp's: cosines and sines of two tokens
  __shared__ __align__(16) uint16_t weights[WARPS][D];
  ptx::grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, sub = lane % LPH;
  // a CTA has one set of heads of WARPS * a.run tokens, a warp every WARPS-th of them
  int set = blockIdx.y;
  const int kind = set < a.q_sets ? 0 : (set < a.q_sets + a.k_sets ? 1 : 2);
  set -= kind == 0 ? 0 : (kind == 1 ? a.q_sets : a.q_sets + a.k_sets);
  if (LAYOUT == 1 && kind == 2) {
    append_vllm_values<D, HPW>(a, set);
    return;
  }
  int64_t t = (int64_t)blockIdx.x * (WARPS * a.run) + warp;
  if (t >= a.num_tokens) return;
  int left = min(a.run, (a.num_tokens - 1 - (int)t) / WARPS + 1);   // tokens of this warp
  const int heads = kind == 0 ? a.h_q : a.h_kv;
  const int h0 = set * (a.iters * HPW) + lane / LPH;
  const int iters = min(a.iters, (heads - set * (a.iters * HPW) + HPW - 1) / HPW);   // groups of this warp
  const int rot = a.cos_sin != nullptr ? a.rot_dim : 0;
  const bool turns = 2 * CW * sub < rot;
  int off[2];
  off[0] = turns ? CW * sub : rot + CW * (sub - rot / (2 * CW));
  off[1] = off[0] + (turns ? rot / 2 : (D - rot) / 2);
  const int64_t stride = kind == 0 ? a.q_stride : (kind == 1 ? a.k_stride : a.v_stride);
  const uint16_t* src = (kind == 0 ? a.q : (kind == 1 ? a.k : a.v)) + t * stride + h0 * D;

  // where a lane's four cosines or sines lie: as in the table, but where eight threads read eight each (SPLIT) the first fours
  // of all and then the second ones, free of bank conflicts (1024 tokens of 64 + 8 + 8 heads 8.4 -> 7.8 us)
  constexpr bool SPLIT = D == 128 && CW == 8 && !PAIRS;
  const int quarter = rot / 8, q4 = lane < quarter ? lane : lane - quarter;
  const int place = SPLIT ? 4 * ((lane - q4) + (q4 >> 1) + (q4 & 1) * (quarter >> 1)) : 4 * lane;
  auto copy_heads = [&](int it) {       // the heads of group `it` of src's token
    if (h0 + it * HPW < heads) {
#pragma unroll
      for (int j = 0; j < 2; ++j) copy_chunk<CW>(&stage[it][j][threadIdx.x], src + it * (HPW * D) + off[j]);
    }
  };
  // AXES: the axes of this lane's four pairs, a byte each; kNoAxis: some pair's axis is none of them.  A token's position on
  // axis i is read by lane i (the others: on axis 0).
  constexpr uint32_t kNoAxis = 0xffffffffu;
  uint32_t pair_axes = 0;
  if (AXES && rot) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t axis = 4 * lane < rot ? a.pair_axes[4 * lane % (rot / 2) + i] : 0;
      bad |= axis >= (uint32_t)a.num_axes;
      pair_axes |= (axis & 31u) << (8 * i);
    }
    if (__any_sync(0xffffffffu, bad)) pair_axes = kNoAxis;
  }
  auto position = [&](int64_t token) {
    return a.positions[AXES ? (int64_t)(lane < a.num_axes ? lane : 0) * a.num_tokens + token : token];
  };
  auto copy_turn = [&](int pos, int at) {   // the cosines and sines of a position; false: it is not in the table
    bool in = pos >= 0 && pos < a.max_position;
    if (AXES) in = __all_sync(0xffffffffu, in) && pair_axes != kNoAxis;
    if (in) {
      if constexpr (AXES) {
        int p[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __shfl_sync(0xffffffffu, pos, pair_axes >> (8 * i));
        if (kind < 2 && 4 * lane < rot) {
          const float* from = a.cos_sin + 4 * lane;
          float* to = &turn_rows[warp][at][place];
          if (pair_axes == (pair_axes & 0xffu) * 0x01010101u) {
            copy_chunk<8>(reinterpret_cast<Chunk<8>*>(to), reinterpret_cast<const uint16_t*>(from + (int64_t)p[0] * rot));
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(ptx::smem_u32(to + i)), "l"(from + (int64_t)p[i] * rot + i)
                           : "memory");
          }
        }
      } else if (kind < 2 && 4 * lane < rot) {
        copy_chunk<8>(reinterpret_cast<Chunk<8>*>(&turn_rows[warp][at][place]),
                      reinterpret_cast<const uint16_t*>(a.cos_sin + (int64_t)pos * rot + 4 * lane));
      }
      return true;
    }
    if (lane == 0) atomicOr(a.status, kDevBadInput);
    return false;
  };
  // the 4-bit cache: where the other elements of the sixteen of each chunk are, (lane << 1) | chunk
  constexpr int OTHERS = 16 / CW - 1;
  int holder[LAYOUT == 4 ? 2 : 1][OTHERS];
  if constexpr (LAYOUT == 4) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int i = 0; i < OTHERS; ++i) holder[j][i] = append_holder<D, CW>(off[j] ^ ((i + 1) * CW), rot) + 2 * (lane - sub);
  }
  // the first token
  int64_t next_slot = kind != 0 ? a.slots[t] : -1;
  int pos = rot ? position(t) : 0, next_pos = rot && left > 1 ? position(t + WARPS) : 0;
#pragma unroll
  for (int it = 0; it < kAppendIters; ++it)
    if (it < iters) copy_heads(it);
  const uint16_t* weight = kind == 0 ? a.q_weight : (kind == 1 ? a.k_weight : nullptr);
  if (weight != nullptr && 8 * lane < D)
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16;"     // (through L1: every warp of the GPU reads these bytes)
                 ::"r"(ptx::smem_u32(&weights[warp][8 * lane])), "l"(weight + 8 * lane)
                 : "memory");
  bool next_ok = rot ? copy_turn(pos, 0) : true;
  asm volatile("cp.async.commit_group;" ::: "memory");
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  int flip = 0;
#pragma unroll 1
  for (;; --left, t += WARPS, flip ^= 1) {
    const bool ok = next_ok;
    int64_t slot = next_slot;
    if (slot >= (int64_t)a.num_blocks * a.block_size) {
      if (lane == 0) atomicOr(a.status, kDevBadInput);
      slot = -1;
    }
    const int64_t blk = (uint32_t)slot >> a.bs_log;
    const int row = (int)slot & (a.block_size - 1);
    if (kind != 0 && left > 1) next_slot = a.slots[t + WARPS];
    src += WARPS * stride;
    int h = h0;
#pragma unroll 1
    for (int it = 0; it < iters; ++it, h += HPW) {
      float x[2][CW];
      wait_copies(iters);
      if (it == 0) __syncwarp();     // the warp's cosines, sines and weights; and all lanes have read those of the last token
      unpack_chunk<BF16, CW>(stage[it][0][threadIdx.x], x[0]);
      unpack_chunk<BF16, CW>(stage[it][1][threadIdx.x], x[1]);
      if (left > 1) {
        copy_heads(it);
        if (it == 0 && rot) {
          next_ok = copy_turn(next_pos, flip ^ 1);
          if (left > 2) next_pos = position(t + 2 * WARPS);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (!ok || (kind != 0 && slot < 0)) continue;
      if (weight != nullptr) {
        Two sq[2] = {two(0.f, 0.f), two(0.f, 0.f)};
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < CW; i += 2) {
            const Two v = two(x[j][i], x[j][i + 1]);
            sq[j] = fma2(v, v, sq[j]);
          }
        const float2 sums = split(add2(sq[0], sq[1]));
        float ss = sums.x + sums.y;
#pragma unroll
        for (int m = LPH / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float g[CW];
          unpack_chunk<BF16, CW>(load_chunk<CW>(&weights[warp][off[j]]), g);
#pragma unroll
          for (int i = 0; i < CW; i += 2) {
            const float2 v = split(mul2(mul2(two(x[j][i], x[j][i + 1]), two(r, r)), two(g[i], g[i + 1])));
            x[j][i] = v.x;
            x[j][i + 1] = v.y;
          }
        }
      }
      if (turns && kind < 2) {
        const float* c = turn_rows[warp][flip];
        float cs[2][CW];          // cosines and sines of this lane's pairs
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if constexpr (SPLIT) {
            shared_floats<4>(cs[k], c + k * (rot / 2) + off[0] / 2);
            shared_floats<4>(cs[k] + 4, c + k * (rot / 2) + rot / 4 + off[0] / 2);
          } else if constexpr (PAIRS) {
            shared_floats<CW / 2>(cs[k], c + k * (rot / 2) + off[0] / 2);
            shared_floats<CW / 2>(cs[k] + CW / 2, c + k * (rot / 2) + off[1] / 2);
          } else {
            shared_floats<CW>(cs[k], c + k * (rot / 2) + off[0]);
          }
        }
#pragma unroll
        for (int i = 0; i < CW; ++i) {
          // pair i of the lane: (x[0][i], x[1][i]), or neighbours of chunk i / (CW/2)
          float& p = PAIRS ? x[i / (CW / 2)][2 * (i % (CW / 2))] : x[0][i];
          float& n = PAIRS ? x[i / (CW / 2)][2 * (i % (CW / 2)) + 1] : x[1][i];
          const float y = p * cs[0][i] - n * cs[1][i];
          n = n * cs[0][i] + p * cs[1][i];
          p = y;
        }
      }
      if (kind == 0) {
        if (h < heads) {
          uint16_t* to = a.q_out + t * a.q_out_stride + h * D;
          store_chunk<CW>(to + off[0], pack_chunk<BF16, CW>(x[0]));
          store_chunk<CW>(to + off[1], pack_chunk<BF16, CW>(x[1]));
        }
      } else if constexpr (LAYOUT == 2) {
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < CW; ++i) top = fmaxf(top, fmaxf(fabsf(x[0][i]), fabsf(x[1][i])));
#pragma unroll
        for (int m = LPH / 2; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
        const int e = kv8_exponent(top);
        const int bb = kv8_block_bytes(a.block_size, D);
        const int64_t at = (blk * a.h_kv + h) * bb;
        if (h < heads && idx_ok(at + bb - 1, (int64_t)a.num_blocks * a.h_kv * bb, a.status)) {
          uint8_t* base = reinterpret_cast<uint8_t*>(a.k_cache) + at;
          uint8_t* codes = base + (kind - 1) * a.block_size * D;
          const float inv = kv8_scale(254 - e);   // 2^-k
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint8_t* to = codes + kv8_chunk<D>(row, off[j] >> 4) + (off[j] & 15);
            if constexpr (CW == 8) *reinterpret_cast<uint2*>(to) = make_uint2(kv8_codes(x[j], inv), kv8_codes(x[j] + 4, inv));
            else *reinterpret_cast<uint32_t*>(to) = kv8_codes(x[j], inv);
          }
          if (sub == 0) base[2 * a.block_size * D + (kind - 1) * a.block_size + row] = (uint8_t)e;
        }
      } else if constexpr (LAYOUT == 4) {
        uint32_t own[2], top[2];     // largest magnitudes, as bits: a NaN is the largest of all
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float m = fabsf(x[j][0]);
#pragma unroll
          for (int i = 1; i < CW; ++i) asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(m), "f"(fabsf(x[j][i])));
          top[j] = own[j] = __float_as_uint(m);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < OTHERS; ++i) {
            const uint32_t p = __shfl_sync(0xffffffffu, own[0], holder[j][i] >> 1);
            const uint32_t n = __shfl_sync(0xffffffffu, own[1], holder[j][i] >> 1);
            top[j] = max(top[j], holder[j][i] & 1 ? n : p);
          }
        const int bb = kv4_block_bytes(a.block_size, D);
        const int64_t at = (blk * a.h_kv + h) * bb;
        if (h < heads && idx_ok(at + bb - 1, (int64_t)a.num_blocks * a.h_kv * bb, a.status)) {
          uint8_t* base = reinterpret_cast<uint8_t*>(a.k_cache) + at;
          uint8_t* codes = base + (kind - 1) * a.block_size * (D / 2);
          uint8_t* scales = base + a.block_size * D + ((kind - 1) * a.block_size + row) * (D / 16);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t byte = kv4_scale_byte(top[j]);
            const float s = byte == 0 ? 1.f : kv4_scale(byte), inv = kv4_inverse(s);   // (0: elements far below a half)
            uint8_t* to = codes + kv4_chunk<D>(row, off[j] >> 5) + ((off[j] & 31) >> 1);
            if constexpr (CW == 8) *reinterpret_cast<uint32_t*>(to) = kv4_codes(x[j], s, inv) | (kv4_codes(x[j] + 4, s, inv) << 16);
            else *reinterpret_cast<uint16_t*>(to) = (uint16_t)kv4_codes(x[j], s, inv);
            if (off[j] % 16 == 0) scales[off[j] / 16] = (uint8_t)byte;
          }
        }
      } else if (h < heads) {
        uint16_t* pool = reinterpret_cast<uint16_t*>(kind == 1 ? a.k_cache : a.v_cache);
        const int64_t size = (int64_t)a.num_blocks * a.block_size * a.h_kv * D;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const Chunk<CW> y = pack_chunk<BF16, CW>(x[j]);
          const int64_t at = LAYOUT == 0
                                 ? (slot * a.h_kv + h) * D + off[j]
                                 : (((blk * a.h_kv + h) * (D / 8) + off[j] / 8) * a.block_size + row) * 8 + off[j] % 8;
          if (idx_ok(at + CW - 1, size, a.status)) store_chunk<CW>(pool + at, y);
        }
      }
    }
    if (left == 1) return;
  }
}

// the launch, a translation unit for each d_head and type (gqa_append_inst.cuh)
template <int D, bool BF16>
cudaError_t append_run(const AppendParams& p, int layout, int sms, cudaStream_t st);

// =====================================================================================
// the 8-bit cache back to 16 bits
// =====================================================================================
struct Kv8ReadParams {
  const uint8_t* cache;
  const int32_t *block_tables, *seq_lens, *begins;
  uint16_t *k_out, *v_out;
  uint32_t* status;
  int64_t out_len, most;   // rows of an output sequence, and how many of them there can be tokens for
  int num_seqs, max_blocks, num_blocks, block_size, bs_log, h_kv;
};

// One warp for 4 * RPP tokens of one head: D/16 lanes a row, 16 codes a lane, the loads of K and V of all
// its rows first.  Warps of a CTA take the heads of the same tokens, whose blocks lie side by side in the
// cache and whose output rows touch.  Bound by its bytes.
template <int D>
struct ReadCfg {
  static constexpr int LPR = D / 16, RPP = 32 / LPR, P = 4, TOKENS = P * RPP;
};

template <int D, bool BF16>
__global__ void __launch_bounds__(kReadThreads)
gqa_kv8_read_kernel(const Kv8ReadParams a) {
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
  const int bb = kv8_block_bytes(a.block_size, D), v_off = a.block_size * D;
  uint4 codes[2][P];
  uint32_t e[2][P];
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
          codes[kv][p] = __ldcs(reinterpret_cast<const uint4*>(at + kv * v_off + kv8_chunk<D>(row, c)));
          e[kv][p] = __ldg(at + 2 * v_off + kv * a.block_size + row);
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
      const float s = kv8_scale(e[kv][p]);
      const uint32_t word[4] = {codes[kv][p].x, codes[kv][p].y, codes[kv][p].z, codes[kv][p].w};
      uint32_t y[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        const float2 f = half2_floats(kv8_halves((uint16_t)(word[q >> 1] >> (16 * (q & 1)))));
        y[q] = Elem<BF16>::pack(f.x * s, f.y * s);
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

}  // namespace gqa
