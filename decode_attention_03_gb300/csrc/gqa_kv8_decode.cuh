// Decode attention over the 8-bit cache.
#pragma once
#include "gqa_kv8.cuh"

namespace gqa {

struct Kv8Params {
  const uint16_t* q;
  uint16_t* o;
  const uint8_t* cache;
  const int32_t *block_tables, *seq_lens;
  uint32_t* status;
  int N, T_q, h_q, h_kv, G, rows, max_blocks, num_blocks, block_size, causal;
  float scale_log2;
};

constexpr int kKv8Warps = 4;

// One CTA per (sequence, query token, query head), its warps taking every fourth key: the running
// maximum, sum and O of each warp in registers, folded through shared memory.
template <int D, bool BF16>
__global__ void __launch_bounds__(kKv8Warps * 32)
gqa_decode_kv8_kernel(const Kv8Params a) {
  constexpr int PER = D / 32;
  __shared__ float sm[kKv8Warps][D + 2];
  ptx::grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t r = blockIdx.x;
  const int h = (int)(r % a.h_q), t = (int)(r / a.h_q % a.T_q);
  const int64_t b = r / ((int64_t)a.h_q * a.T_q);
  const int g = h / a.G, cap = a.max_blocks * a.block_size, bb = kv8_block_bytes(a.block_size, D);
  int len = a.seq_lens[b];
  if (len < 0 || len > cap) {
    if (threadIdx.x == 0) atomicOr(a.status, kDevBadInput);
    len = len < 0 ? 0 : cap;
  }
  const int end = a.causal ? len - a.T_q + t + 1 : len;
  float q[PER], acc[PER], m = -CUDART_INF_F, l = 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const uint16_t x = a.q[r * D + lane * PER + i];
    q[i] = BF16 ? __uint_as_float((uint32_t)x << 16) : __half2float(__ushort_as_half(x));
    acc[i] = 0.f;
  }
  for (int j = warp; j < end; j += kKv8Warps) {
    const int id = a.block_tables[b * a.max_blocks + j / a.block_size], row = j % a.block_size;
    if (id < 0 || id >= a.num_blocks) {
      if (lane == 0) atomicOr(a.status, kDevBadInput);
      continue;
    }
    const uint8_t* at = a.cache + ((int64_t)id * a.h_kv + g) * bb;
    const int off = kv8_chunk<D>(row, lane * PER / 16) + lane * PER % 16;
    float s = 0.f, v[PER];
#pragma unroll
    for (int i = 0; i < PER; i += 2) {
      const float2 x = half2_floats(kv8_halves(*reinterpret_cast<const uint16_t*>(at + off + i)));
      const float2 y = half2_floats(kv8_halves(*reinterpret_cast<const uint16_t*>(at + a.block_size * D + off + i)));
      s += q[i] * x.x + q[i + 1] * x.y;
      v[i] = y.x;
      v[i + 1] = y.y;
    }
#pragma unroll
    for (int k = 16; k > 0; k >>= 1) s += __shfl_xor_sync(0xffffffffu, s, k);
    s *= kv8_scale(at[2 * a.block_size * D + row]) * a.scale_log2;
    const float m_new = fmaxf(m, s), m_use = m_new == -CUDART_INF_F ? 0.f : m_new;
    const float alpha = ptx::ex2(m - m_use), p = ptx::ex2(s - m_use);
    const float pv = p * kv8_scale(at[2 * a.block_size * D + a.block_size + row]);
    m = m_new;
    l = l * alpha + p;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = acc[i] * alpha + pv * v[i];
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) sm[warp][lane * PER + i] = acc[i];
  if (lane == 0) {
    sm[warp][D] = m;
    sm[warp][D + 1] = l;
  }
  __syncthreads();
  if (warp != 0) return;
  float M = -CUDART_INF_F, L = 0.f;
#pragma unroll
  for (int k = 0; k < kKv8Warps; ++k) M = fmaxf(M, sm[k][D]);
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll
  for (int k = 0; k < kKv8Warps; ++k) {
    const float f = M == -CUDART_INF_F ? 0.f : ptx::ex2(sm[k][D] - M);
    L += f * sm[k][D + 1];
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] += f * sm[k][lane * PER + i];
  }
  const float inv = L > 0.f ? 1.f / L : 0.f;
#pragma unroll
  for (int i = 0; i < PER; ++i)
    Elem<BF16>::store(reinterpret_cast<__half*>(a.o), r * D + lane * PER + i, acc[i] * inv);
}

}  // namespace gqa
