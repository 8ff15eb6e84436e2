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

namespace gqa {

constexpr int kAppendThreads = 256;
constexpr int kReadThreads = 256;
constexpr int kReadTokens = 16;   // tokens of one warp of the read kernel

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
__device__ __forceinline__ uint32_t kv8_codes(const float (&x)[4], float inv) {
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
  int num_tokens, h_q, h_kv, max_position, rot_dim, interleaved, num_blocks, block_size, layout, sets;
  float eps;
};

// A head's D elements lie on D/8 lanes, each with two groups of four: elements 4s.. and rot/2 + 4s.. for
// the lanes s < rot/8 that rotate, so that both elements of every rotated pair (i, i + rot/2) are in one
// thread and the rotation needs no exchange; the rest of the head (rot..D) is cut the same way.  A warp takes U
// times 32/(D/8) heads of one token and issues all their loads before it uses one.  Bound by its bytes:
// the heads read and written once; the sums of squares and maxima go through log2(D/8) shuffles.
template <int D, bool BF16, int U>
__global__ void __launch_bounds__(kAppendThreads)
gqa_append_kernel(const AppendParams a) {
  constexpr int LPH = D / 8, HPW = 32 / LPH;
  ptx::grid_dependency_wait();
  const int lane = threadIdx.x & 31, sub = lane % LPH;
  const int64_t w = ((int64_t)blockIdx.x * kAppendThreads + threadIdx.x) >> 5;
  const int64_t t = w / a.sets;
  if (t >= a.num_tokens) return;
  const int h0 = (int)(w - t * a.sets) * (U * HPW) + lane / LPH;
  const int heads = a.h_q + 2 * a.h_kv;
  const bool turns = a.cos_sin != nullptr && sub < a.rot_dim / 8;
  const int rot = a.cos_sin != nullptr ? a.rot_dim : 0;
  int off[2];
  off[0] = turns ? 4 * sub : rot + 4 * (sub - rot / 8);
  off[1] = turns ? rot / 2 + 4 * sub : rot + (D - rot) / 2 + 4 * (sub - rot / 8);

  uint2 raw[U][2];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * HPW;
    const uint16_t* src = nullptr;
    if (h < a.h_q) src = a.q + t * a.q_stride + h * D;
    else if (h < a.h_q + a.h_kv) src = a.k + t * a.k_stride + (h - a.h_q) * D;
    else if (h < heads) src = a.v + t * a.v_stride + (h - a.h_q - a.h_kv) * D;
#pragma unroll
    for (int j = 0; j < 2; ++j)
      raw[u][j] = src != nullptr ? *reinterpret_cast<const uint2*>(src + off[j]) : make_uint2(0u, 0u);
  }
  const int64_t slot = a.slots[t];
  const int64_t n_slots = (int64_t)a.num_blocks * a.block_size;
  if (slot >= n_slots && lane == 0) atomicOr(a.status, kDevBadInput);
  const bool stored = slot >= 0 && slot < n_slots;
  const int64_t blk = stored ? slot / a.block_size : 0;
  const int row = stored ? (int)(slot - blk * a.block_size) : 0;
  float cs[8];   // cosines and sines of this lane's four pairs
  if (a.cos_sin != nullptr) {
    const int p = a.positions[t];
    if (p < 0 || p >= a.max_position) {
      if (lane == 0) atomicOr(a.status, kDevBadInput);
      return;
    }
    if (turns) {
      const float* c = a.cos_sin + (int64_t)p * a.rot_dim;
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float2 x = *reinterpret_cast<const float2*>(c + off[j] / 2);
          const float2 y = *reinterpret_cast<const float2*>(c + rot / 2 + off[j] / 2);
          cs[2 * j] = x.x; cs[2 * j + 1] = x.y; cs[4 + 2 * j] = y.x; cs[5 + 2 * j] = y.y;
        }
      } else {
        const float4 x = *reinterpret_cast<const float4*>(c + 4 * sub);
        const float4 y = *reinterpret_cast<const float4*>(c + rot / 2 + 4 * sub);
        cs[0] = x.x; cs[1] = x.y; cs[2] = x.z; cs[3] = x.w;
        cs[4] = y.x; cs[5] = y.y; cs[6] = y.z; cs[7] = y.w;
      }
    }
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int h = h0 + u * HPW;
    float x[2][4];
    unpack4<BF16>(raw[u][0], x[0]);
    unpack4<BF16>(raw[u][1], x[1]);
    const bool is_q = h < a.h_q, is_k = !is_q && h < a.h_q + a.h_kv;
    // ---- norm of the head
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) ss += x[0][i] * x[0][i] + x[1][i] * x[1][i];
#pragma unroll
    for (int m = LPH / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
    const uint16_t* wt = is_q ? a.q_weight : (is_k ? a.k_weight : nullptr);
    if (wt != nullptr) {
      const float r = 1.f / sqrtf(ss * (1.f / D) + a.eps);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float g[4];
        unpack4<BF16>(*reinterpret_cast<const uint2*>(wt + off[j]), g);
#pragma unroll
        for (int i = 0; i < 4; ++i) x[j][i] = x[j][i] * r * g[i];
      }
    }
    // ---- rotation of its pairs
    if (turns && (is_q || is_k)) {
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const float c = cs[2 * j + i / 2], s = cs[4 + 2 * j + i / 2], p = x[j][i], n = x[j][i + 1];
            x[j][i] = p * c - n * s;
            x[j][i + 1] = n * c + p * s;
          }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float c = cs[i], s = cs[4 + i], p = x[0][i], n = x[1][i];
          x[0][i] = p * c - n * s;
          x[1][i] = n * c + p * s;
        }
      }
    }
    // ---- the row's exponent (kv8)
    int e = 0;
    if (a.layout == 2) {
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, fmaxf(fabsf(x[0][i]), fabsf(x[1][i])));
#pragma unroll
      for (int m = LPH / 2; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
      e = kv8_exponent(top);
    }
    if (h >= heads) continue;
    if (is_q) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<uint2*>(a.q_out + t * a.q_out_stride + h * D + off[j]) =
            make_uint2(Elem<BF16>::pack(x[j][0], x[j][1]), Elem<BF16>::pack(x[j][2], x[j][3]));
      continue;
    }
    if (!stored) continue;
    const int g = is_k ? h - a.h_q : h - a.h_q - a.h_kv;
    if (a.layout == 2) {
      const int bb = kv8_block_bytes(a.block_size, D);
      const int64_t at = (blk * a.h_kv + g) * bb;
      if (!idx_ok(at + bb - 1, (int64_t)a.num_blocks * a.h_kv * bb, a.status)) continue;
      uint8_t* base = reinterpret_cast<uint8_t*>(a.k_cache) + at;
      uint8_t* codes = base + (is_k ? 0 : a.block_size * D);
      const float inv = kv8_scale(254 - e);   // 2^-k
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<uint32_t*>(codes + kv8_chunk<D>(row, off[j] >> 4) + (off[j] & 15)) = kv8_codes(x[j], inv);
      if (sub == 0) base[2 * a.block_size * D + (is_k ? 0 : a.block_size) + row] = (uint8_t)e;
    } else {
      uint16_t* pool = reinterpret_cast<uint16_t*>(is_k ? a.k_cache : a.v_cache);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint2 y = make_uint2(Elem<BF16>::pack(x[j][0], x[j][1]), Elem<BF16>::pack(x[j][2], x[j][3]));
        if (a.layout == 0 || is_k) {
          const int64_t at =
              a.layout == 0 ? ((blk * a.block_size + row) * a.h_kv + g) * D + off[j]
                            : (((blk * a.h_kv + g) * (D / 8) + off[j] / 8) * a.block_size + row) * 8 + off[j] % 8;
          if (idx_ok(at + 3, n_slots * a.h_kv * D, a.status)) *reinterpret_cast<uint2*>(pool + at) = y;
        } else {
          const int64_t at = ((blk * a.h_kv + g) * D + off[j]) * a.block_size + row;
          if (!idx_ok(at + 3 * a.block_size, n_slots * a.h_kv * D, a.status)) continue;
          pool[at] = (uint16_t)y.x;
          pool[at + a.block_size] = (uint16_t)(y.x >> 16);
          pool[at + 2 * a.block_size] = (uint16_t)y.y;
          pool[at + 3 * a.block_size] = (uint16_t)(y.y >> 16);
        }
      }
    }
  }
}

// =====================================================================================
// the 8-bit cache back to 16 bits
// =====================================================================================
struct Kv8ReadParams {
  const uint8_t* cache;
  const int32_t *block_tables, *seq_lens, *begins;
  uint16_t *k_out, *v_out;
  uint32_t* status;
  int64_t out_len, groups;   // token groups of a sequence
  int num_seqs, max_blocks, num_blocks, block_size, h_kv;
};

// One warp for kReadTokens tokens of one head: D/8 lanes a row, 8 codes a lane, all loads of the warp's
// rows first.  Warps of a CTA take the heads of the same tokens, whose blocks lie side by side in the
// cache and whose output rows touch.  Bound by its bytes.
template <int D, bool BF16>
__global__ void __launch_bounds__(kReadThreads)
gqa_kv8_read_kernel(const Kv8ReadParams a) {
  constexpr int LPR = D / 8, RPP = 32 / LPR, P = kReadTokens / RPP;
  ptx::grid_dependency_wait();
  const int lane = threadIdx.x & 31, c8 = lane % LPR;
  int64_t w = ((int64_t)blockIdx.x * kReadThreads + threadIdx.x) >> 5;
  if (w >= (int64_t)a.num_seqs * a.groups * a.h_kv) return;
  const int g = (int)(w % a.h_kv);
  w /= a.h_kv;
  const int64_t b = w / a.groups, i0 = (w - b * a.groups) * kReadTokens;
  const int cap = a.max_blocks * a.block_size;
  int len = a.seq_lens[b];
  const int begin = a.begins != nullptr ? a.begins[b] : 0;
  if (len < 0 || len > cap || begin < 0) {
    if (lane == 0) atomicOr(a.status, kDevBadInput);
    len = len > cap ? cap : len;
  }
  if (begin < 0 || begin + i0 >= len) return;
  const int bb = kv8_block_bytes(a.block_size, D);
  int64_t base[P];
  int rows[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const int64_t i = i0 + p * RPP + lane / LPR, tok = begin + i;
    base[p] = -1;
    rows[p] = 0;
    if (i < a.out_len && tok < len) {
      const int64_t j = tok / a.block_size;
      const int id = a.block_tables[b * a.max_blocks + j];
      rows[p] = (int)(tok - j * a.block_size);
      if (id >= 0 && id < a.num_blocks) base[p] = ((int64_t)id * a.h_kv + g) * bb;
      else atomicOr(a.status, kDevBadInput);
    }
  }
#pragma unroll
  for (int kv = 0; kv < 2; ++kv) {
    uint16_t* out = kv ? a.v_out : a.k_out;
    if (out == nullptr) continue;
    uint2 codes[P];
    uint32_t e[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      codes[p] = make_uint2(0u, 0u);
      e[p] = 127;
      if (base[p] >= 0) {
        const uint8_t* at = a.cache + base[p];
        codes[p] = __ldcs(reinterpret_cast<const uint2*>(at + kv * a.block_size * D + kv8_chunk<D>(rows[p], c8 >> 1) +
                                                         (c8 & 1) * 8));
        e[p] = at[2 * a.block_size * D + kv * a.block_size + rows[p]];
      }
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (base[p] < 0) continue;
      const float s = kv8_scale(e[p]);
      uint4 y;
      uint32_t* yw = reinterpret_cast<uint32_t*>(&y);
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t word = q < 2 ? codes[p].x : codes[p].y;
        const float2 f = half2_floats(kv8_halves((uint16_t)(word >> (16 * (q & 1)))));
        yw[q] = Elem<BF16>::pack(f.x * s, f.y * s);
      }
      const int64_t at = ((b * a.out_len + i0 + p * RPP + lane / LPR) * a.h_kv + g) * D + c8 * 8;
      if (idx_ok(at + 7, a.num_seqs * a.out_len * a.h_kv * D, a.status)) *reinterpret_cast<uint4*>(out + at) = y;
    }
  }
}

}  // namespace gqa
