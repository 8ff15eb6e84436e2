// Decode attention over the 8-bit cache.
//
// Work: every (sequence, KV head) is a row of 32-key tiles; all tiles of a launch lie on one axis, which is
// cut into equal shares, one for each worker (a worker is RG warps, GROUPS of them on a CTA, one CTA on an
// SM).  The cut does not look at sequences: a share may hold many short ones or a part of a long one, so
// every worker streams the same bytes whatever the lengths are, and nothing is claimed or counted at run
// time.  A (sequence, head) that lies inside one share is finished by its worker; the others leave partials
// (m, l, O) that a merge kernel folds in the order of the keys: the same bits every time.
//
// Few units that their table bounds to few tiles take another kernel, without a merge: see the short kernel below.
//
// A worker streams its tiles through a ring of its own in shared memory: one plain bulk copy for each block
// (32 keys are 32/block_size of them), K, V and scales together.  No warp waits for another worker's.
//
// Arithmetic of a warp, for its 8 NT query rows and 32 keys.  S^T = K Q^T with keys on the MMA's M side and
// query rows on its N side (n = 8: with 4 query heads a KV head only half of the tile is idle).  K codes come
// by ldmatrix -- a thread's 4 bytes are the elements 16j + 4c .. +3 of one key, and since the order of the
// summed index is free, Q is laid out to match -- and become f16 by one conversion for two codes, exactly.
// The K scale multiplies the fp32 score, the V scale multiplies the weight: P = p 2^(ev - e + 11), e the largest V
// exponent so far (O is rescaled when e grows, together with the running maximum), so that P <= 2^15.  f16 holds a
// weight with all its bits down to 2^-25 of the running maximum's, and nothing below 2^-36; as long as the V exponents seen
// lie within 10 of one another, that is at most 2^-26 of the row's largest term.  Where they lie further apart (a row of
// zeros, an infinity, an outlier), a weight of 1 may belong to the smallest terms of its row, and the worker goes on with
// the wide form of a tile's products (kv8_wide), which has a reference of its own for every tile, row and range of
// exponents.  V codes come by transposing ldmatrix as byte pairs of two d for each of two keys, one byte permutation turns
// them into pairs of keys, the MMA's A operand of O^T += V^T P^T.
// bfloat16 queries are brought into f16's range by a power of two for each row (8 bits of fraction fit into
// 11: nothing is rounded that fp32 sums would keep); O, m and l are fp32.
// The running maximum is only moved when a score exceeds it by 2^4: the weights stay below 2^4 and the
// common tile needs no cross-lane maximum and no rescaling.
#pragma once
#include "gqa_kv8.cuh"
#include "gqa_merge.cuh"   // kMergeThreads, kMergeChunk
#include "kv8_notes.h"

namespace gqa {

constexpr int kKv8Keys = 32;                   // keys of a tile
constexpr int kKv8Seqs = 1024;                 // sequences of a launch (the host splits larger batches)
constexpr int kKv8Warps = 8;
constexpr int kKv8Short = 8;                   // tiles of a worker of the short kernel: 32 blocks of 8 keys
constexpr int kKv8Threads = 32 * kKv8Warps;
// log2 of the largest weight.  8 leaves a lift of 7 bits instead of 11, and a weight of 2^-26 none of its bits; fewer moves
// of the maximum then (131071 keys, 32 rows 71.9 us instead of 73.5, one n-tile the same).
constexpr float kKv8Slack = 4.f;
constexpr int kKv8Lift = 11;                   // P in f16 is the weight times 2^this: at most 2^15
constexpr int kKv8Spread = 10;                 // V exponents further apart than this: the wide form
constexpr int kKv8Wide = 1024;                 // Kv8Warp::lo of a worker that has gone over to it, above every exponent
constexpr int kKv8ByToken = 1025;              // the same, and a row is not to meet the values that it does not see
constexpr int kKv8ToToken = 1026;              // that, from the next products on
constexpr int kKv8WideUnit = 16;               // log2 of the unit of its O: sums of many values of 448 * 2^120 fit

// What is copied where the cache has no block: zeros, as many as one copy brings at most.  (An exponent byte of 0 stands for
// the scale 0.)
__device__ const uint4 kKv8Zeros[kv8_block_bytes(kKv8Keys, 128) / 16] = {};

struct Kv8Params {
  const uint16_t* q;
  uint16_t* o;
  const uint8_t* cache;
  const int32_t *block_tables, *seq_lens;
  uint32_t* status;
  int4* splits;          // the units that are cut, for the merge (Kv8Note); [workers], sliced: [units]
  float *ws_m, *ws_l;    // [2 * workers][rows]   m in log2 units
  float* ws_o;           // [2 * workers][rows][D]
  int N, T_q, h_q, h_kv, G, rows, max_blocks, num_blocks, block_size, bs_log, causal, workers, stall;
  int sliced;            // few units of many pieces: splits has one entry for each unit
  int ctas;              // short kernel: CTAs of a unit, one cluster
  float scale_log2;
  uint64_t timeout_ns;
};

// The slots of partials: worker w's first piece 2w, a later piece that it does not finish 2w + 1.
template <int D, int NT, int RG>
struct Kv8Cfg {
  static constexpr int GROUPS = kKv8Warps / RG;
  static constexpr int TILE = kKv8Keys * (2 * D + 2);
  static constexpr bool Q_SMEM = NT > 2;                    // query fragments in shared memory, else in registers
  static constexpr int QUERIES = Q_SMEM ? 8 * NT * (D * 2 + 4) : 0;   // of a warp, and its rows' factors
  static constexpr int PREFIX_OFF = 0;
  static constexpr int LENS_OFF = (kKv8Seqs + 2) * 8;
  static constexpr int SUMS_OFF = LENS_OFF + kKv8Seqs * 4;
  static constexpr int FLAG_OFF = SUMS_OFF + kKv8Warps * 8;
  static constexpr int BAR_OFF = FLAG_OFF + 16;
  // 2 x 8.25 KB in flight for each warp.  Three entries at d_head 128: 64 sequences of 1K-16K keys 168 us instead of
  // 157, 2^20 keys 340 instead of 320: the fuller the memory's queues, the more unevenly it serves the SMs, and the
  // shares are equal (last worker done 22 us after the median instead of 10).
  static constexpr int STAGES = (D == 128 ? 2 : 4) * RG;
  static constexpr int Q_OFF = (BAR_OFF + GROUPS * STAGES * 16 + 127) & ~127;
  static constexpr int ML_OFF = Q_OFF + kKv8Warps * QUERIES;    // m and l of a warp's rows, where a CTA folds its warps'
  static constexpr int RING_OFF = (ML_OFF + kKv8Warps * 8 * NT * 8 + 127) & ~127;
  static constexpr int SMEM = RING_OFF + GROUPS * STAGES * TILE;
  static constexpr int AREA = STAGES * TILE / RG;               // a warp's part of the ring: holds its O there
  static_assert(GROUPS * STAGES <= kKv8Threads && SMEM <= 232448 && AREA >= 8 * NT * D * 4 && AREA % 16 == 0, "ring");
};

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;"
      ::"r"(dst), "l"(src), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}

// the four e4m3 codes of a word as two pairs of f16
__device__ __forceinline__ void kv8_unpack(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// The MMA and the 8x8 transpose as ptx:: has them, but free to be scheduled among the shared-memory reads.
__device__ __forceinline__ void kv8_mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ uint32_t kv8_transpose(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// 2^d for d <= 127, 0 below 2^-126
__device__ __forceinline__ float kv8_ratio(int d) { return __uint_as_float((uint32_t)max(d + 127, 0) << 23); }

// A place on the axis of tiles: tile t of the `tiles` tiles of head g of sequence b.
struct Kv8Place {
  int b, g, t, tiles;
};

__device__ __forceinline__ void kv8_next_unit(Kv8Place& p, const int64_t* prefix, int N, int h_kv) {
  p.t = 0;
  if (++p.g < h_kv) return;
  p.g = 0;
  do {
    ++p.b;
  } while (p.b < N && prefix[p.b + 1] == prefix[p.b]);
  p.tiles = p.b < N ? (int)(prefix[p.b + 1] - prefix[p.b]) : 0;
}

__device__ __forceinline__ Kv8Place kv8_find(int64_t f, const int64_t* prefix, int N, int h_kv) {
  int lo = 0, hi = N - 1;   // the first sequence that ends after f
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (prefix[mid + 1] * h_kv > f) hi = mid; else lo = mid + 1;
  }
  Kv8Place p;
  p.b = lo;
  p.tiles = (int)(prefix[lo + 1] - prefix[lo]);
  const int64_t rem = f - prefix[lo] * h_kv;
  p.g = (int)(rem / p.tiles);
  p.t = (int)(rem - (int64_t)p.g * p.tiles);
  return p;
}

// Tiles (of one head) before each sequence of the launch, in shared memory.
__device__ __forceinline__ void kv8_prefix(const Kv8Params& a, int64_t* prefix, int* lens, int64_t* sums) {
  constexpr int PER = kKv8Seqs / kKv8Threads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t cap = (int64_t)a.max_blocks * a.block_size;
  int64_t v[PER], run = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = threadIdx.x * PER + i;
    int len = b < a.N ? a.seq_lens[b] : 0;
    if (len < 0 || len > cap) {
      if (blockIdx.x == 0) atomicOr(a.status, kDevBadInput);
      len = len < 0 ? 0 : (int)cap;
    }
    lens[b] = len;
    run += ((int64_t)len + kKv8Keys - 1) / kKv8Keys;
    v[i] = run;
  }
  int64_t incl = run;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, incl, off);
    if (lane >= off) incl += x;
  }
  if (lane == 31) sums[warp] = incl;
  __syncthreads();
  int64_t before = incl - run;
  for (int w = 0; w < warp; ++w) before += sums[w];
  if (threadIdx.x == 0) prefix[0] = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int b = threadIdx.x * PER + i;
    if (b < a.N) prefix[b + 1] = before + v[i];
  }
  __syncthreads();
}

// Rows of sequences without keys: zeros, each sequence by one CTA.
template <int D>
__device__ __forceinline__ void kv8_empty_rows(const Kv8Params& a, const int* lens) {
  const int64_t words = (int64_t)a.T_q * a.h_q * D / 8;
  for (int b = blockIdx.x; b < a.N; b += gridDim.x)
    if (lens[b] == 0) {
      for (int64_t i = threadIdx.x; i < words; i += kKv8Threads)
        reinterpret_cast<uint4*>(a.o)[b * words + i] = make_uint4(0u, 0u, 0u, 0u);
      if (a.sliced)
        for (int g = threadIdx.x; g < a.h_kv; g += kKv8Threads) a.splits[b * a.h_kv + g] = make_int4(0, 0, 0, 0);
    }
}

// The copying side of a worker: block ids of the next tiles, one for each lane (-1: no block, or a bad id), and what
// this lane copies of a tile.
struct Kv8Stream {
  Kv8Place at;       // next tile to copy
  Kv8Place ahead;    // first tile after the current window
  int id, id_next;   // this lane's block id in the current window and the one after it
  int t_end;         // tile of at's unit where the current window ends
  int k;             // lane of the window that holds at's first block
  const uint8_t* head;     // head at.g of block 0
  // the same for every tile: lanes 0 .. n - 1 copy `size` bytes from `off` of a (block, head) to `to` of the tile,
  // + step in the second half of a block of 64
  int n;
  uint32_t size, to, off, step, stride;   // stride: bytes of a block
};

template <int D>
__device__ __forceinline__ void kv8_stream_setup(Kv8Stream& s, const Kv8Params& a, int lane) {
  const int bs = a.block_size, bb = kv8_block_bytes(bs, D);
  s.stride = (uint32_t)a.h_kv * (uint32_t)bb;
  if (bs <= kKv8Keys) {        // whole blocks
    s.n = kKv8Keys >> a.bs_log;
    s.size = bb;
    s.to = lane * bb;
    s.off = s.step = 0;
  } else {                     // half a block: K, V, K exponents, V exponents
    s.n = 4;
    s.size = lane < 2 ? kKv8Keys * D : kKv8Keys;
    s.to = lane < 2 ? lane * kKv8Keys * D : 2 * kKv8Keys * D + (lane - 2) * kKv8Keys;
    s.off = lane < 2 ? lane * bs * D : 2 * bs * D + (lane - 2) * bs;
    s.step = lane < 2 ? kKv8Keys * D : kKv8Keys;
  }
}

// blocks of a sequence, the block that holds a tile's first key, and the tile where the window of 32 blocks
// that starts at p ends
__device__ __forceinline__ int kv8_blocks(const Kv8Params& a, int len) {
  return (int)(((uint32_t)len + (uint32_t)a.block_size - 1) >> a.bs_log);
}
__device__ __forceinline__ int kv8_first_block(const Kv8Params& a, int t) {
  return (int)(((uint32_t)t * (uint32_t)kKv8Keys) >> a.bs_log);
}
__device__ __forceinline__ int kv8_window_end(const Kv8Params& a, const Kv8Place& p) {
  const int n = a.block_size > kKv8Keys ? a.block_size - (p.t & 1) : a.block_size;   // 32 blocks in tiles
  return p.tiles - p.t < n ? p.tiles : p.t + n;
}

// this lane's block id of the window that starts at p
__device__ __forceinline__ int kv8_window(const Kv8Params& a, const Kv8Place& p, int len, int lane) {
  const int j = kv8_first_block(a, p.t) + lane;
  if (j >= kv8_blocks(a, len) || !idx_ok((int64_t)p.b * a.max_blocks + j, (int64_t)a.N * a.max_blocks, a.status))
    return -1;
  return __ldg(a.block_tables + (int64_t)p.b * a.max_blocks + j);
}

template <int D>
__device__ __forceinline__ void kv8_window_begin(Kv8Stream& s, const Kv8Params& a, int len, int lane) {
  const int j = kv8_first_block(a, s.at.t) + lane;
  if (j < kv8_blocks(a, len) && (s.id < 0 || s.id >= a.num_blocks)) {
    atomicOr(a.status, kDevBadInput);
    s.id = -1;
  }
  s.k = 0;
  s.head = a.cache + (int64_t)s.at.g * kv8_block_bytes(a.block_size, D);
}

// Enters the window at s.at, whose ids are in s.id: reports bad ids, finds where the next window begins and starts
// loading its ids.
template <int D>
__device__ __forceinline__ void kv8_enter(Kv8Stream& s, const Kv8Params& a, const int64_t* prefix, const int* lens,
                                          int lane) {
  kv8_window_begin<D>(s, a, lens[s.at.b], lane);
  s.t_end = kv8_window_end(a, s.at);
  s.ahead = s.at;
  s.ahead.t = s.t_end;
  if (s.t_end >= s.at.tiles) {
    kv8_next_unit(s.ahead, prefix, a.N, a.h_kv);
    // the next unit's queries into L2 (its rows lie together for each token)
    const uint32_t bytes = (uint32_t)a.G * D * 2;
    if (s.ahead.b < a.N)
      for (uint32_t i = lane * 128; i < bytes; i += 32 * 128)
        for (int t = 0; t < a.T_q; ++t)
          asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t*>(
              a.q + (((int64_t)s.ahead.b * a.T_q + t) * a.h_q + (int64_t)s.ahead.g * a.G) * D) + i));
  }
  s.id_next = s.ahead.b < a.N ? kv8_window(a, s.ahead, lens[s.ahead.b], lane) : -1;
}

// Copies the stream's next tile to `dst`; on to the next tile of the window (true: the window ends).  Every lane of the
// warp calls this.
template <int D>
__device__ __forceinline__ bool kv8_issue(Kv8Stream& s, const Kv8Params& a, uint32_t dst, uint32_t bar, uint64_t policy,
                                          int lane, const Win& ring) {
  const bool half = a.block_size > kKv8Keys;
  const int id = __shfl_sync(0xffffffffu, s.id, (s.k + (half ? 0 : lane)) & 31);
  if (lane == 0) ptx::mbar_arrive_expect_tx(bar, kKv8Keys * (2 * D + 2));
  if (lane < s.n) {
    const uint32_t off = s.off + (s.at.t & 1) * s.step;
    const uint8_t* src = s.head + (uint64_t)(uint32_t)id * s.stride + off;
    if (id < 0) src = reinterpret_cast<const uint8_t*>(kKv8Zeros);       // no block, or one with a bad id
    if ((id < 0 || idx_ok(src + s.size - 1 - a.cache, (int64_t)a.num_blocks * s.stride, a.status)) &&
        smem_ok(dst + s.to, s.size, ring.lo, ring.hi, ring.status))
      bulk_load(dst + s.to, src, s.size, bar, policy);
  }
  if (++s.at.t == s.t_end) return true;
  s.k += half ? 1 - (s.at.t & 1) : s.n;
  return false;
}

// the same, and on to the next window
template <int D>
__device__ __forceinline__ void kv8_copy(Kv8Stream& s, const Kv8Params& a, const int64_t* prefix, const int* lens,
                                         uint32_t dst, uint32_t bar, uint64_t policy, int lane, const Win& ring) {
  if (!kv8_issue<D>(s, a, dst, bar, policy, lane, ring)) return;
  s.at = s.ahead;
  s.id = s.id_next;
  if (s.at.b < a.N) kv8_enter<D>(s, a, prefix, lens, lane);
}

// RG warps share a ring (RG = 2: more than 32 rows), each with NT n-tiles of 8 query rows.
template <int D, int NT, int RG>
struct Kv8Warp {
  static constexpr int KD = D / 16;
  static constexpr bool Q_SMEM = NT > 2;
  uint32_t qf[Q_SMEM ? 1 : NT][Q_SMEM ? 1 : KD][2];   // Q^T fragments, or, in shared memory at q_at, [KD][NT][lane] ...
  float qs[Q_SMEM ? 1 : NT][2];                       // ... followed by the rows' factors
  uint32_t q_at;
  float acc[KD][NT][4];
  float m[NT][2], l[NT][2];
  int e, lo;            // largest and smallest V exponent byte so far; lo = kKv8Wide: the wide form
  // the same for every unit and tile
  uint32_t rows[2];     // byte offset in a tile of this lane's ldmatrix row, keys 16p + lane % 16
  uint32_t ex[4];       // and of the K exponent of key 8o + lane / 4
  uint32_t turn;        // chunk swizzle of that row, and which of two chunks this lane addresses
};

template <int D, int NT, int RG>
__device__ __forceinline__ void kv8_setup(Kv8Warp<D, NT, RG>& w, const Kv8Params& a, uint32_t q_at, int lane) {
  w.q_at = q_at;
  const int r = lane >> 2;
  const int eb = min(a.block_size, kKv8Keys), bb = kv8_block_bytes(eb, D);
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    const int key = 16 * p + (lane & 15);
    w.rows[p] = key / eb * bb + key % eb * D;
  }
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    const int key = 8 * o + r;
    w.ex[o] = key / eb * bb + 2 * eb * D + key % eb;
  }
  w.turn = (uint32_t)((lane >> 4) ^ (D == 128 ? (lane & 7) : ((lane >> 1) & 3))) << 4;
}

// A piece begins: its queries are loaded, ...
template <int D, int NT, int RG>
__device__ __forceinline__ void kv8_load_q(uint2 (&raw)[NT][D / 16], const Kv8Params& a, int b, int g, int rg, int lane) {
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = (rg * NT + nt) * 8 + r, t = row / a.G;
    const int64_t at = (((int64_t)b * a.T_q + t) * a.h_q + (int64_t)g * a.G + (row - t * a.G)) * D + 4 * c;
    const bool ok = row < a.rows && idx_ok(at + D - 1 - 4 * c, (int64_t)a.N * a.T_q * a.h_q * D, a.status);
#pragma unroll
    for (int j = 0; j < D / 16; ++j)
      raw[nt][j] = ok ? __ldg(reinterpret_cast<const uint2*>(a.q + at + 16 * j)) : make_uint2(0u, 0u);
  }
}

// ... brought into the MMA's form, and the state is emptied.
template <int D, int NT, int RG, bool BF16>
__device__ __forceinline__ void kv8_begin(Kv8Warp<D, NT, RG>& w, uint2 (&raw)[NT][D / 16], const Kv8Params& a, int len,
                                          int lane) {
  using W = Kv8Warp<D, NT, RG>;
  constexpr int KD = W::KD;
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float qs = fabsf(a.scale_log2);
    if (a.scale_log2 < 0.f) {    // the factor of a row is kept >= 0, so that the largest y is the largest logit
#pragma unroll
      for (int j = 0; j < KD; ++j) raw[nt][j] = make_uint2(raw[nt][j].x ^ 0x80008000u, raw[nt][j].y ^ 0x80008000u);
    }
    if constexpr (BF16) {
      uint32_t top = 0;
#pragma unroll
      for (int j = 0; j < KD; ++j)
        top = max(max(top, max(raw[nt][j].x & 0x7fffu, (raw[nt][j].x >> 16) & 0x7fffu)),
                  max(raw[nt][j].y & 0x7fffu, (raw[nt][j].y >> 16) & 0x7fffu));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const uint32_t e = max(top >> 7, 15u);                    // the row's largest value becomes 2^14 .. 2^15
      const float up = __uint_as_float((268u - e) << 23);
      qs *= __uint_as_float((e - 14u) << 23);
#pragma unroll
      for (int j = 0; j < KD; ++j) {
        float x[4];
        unpack4<true>(raw[nt][j], x);
        raw[nt][j] = make_uint2(ptx::pack_half2(x[0] * up, x[1] * up), ptx::pack_half2(x[2] * up, x[3] * up));
      }
    }
    if constexpr (W::Q_SMEM) {
#pragma unroll
      for (int j = 0; j < KD; ++j)
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(w.q_at + ((j * NT + nt) * 32 + lane) * 8), "r"(raw[nt][j].x),
                     "r"(raw[nt][j].y)
                     : "memory");
      if (c == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(w.q_at + KD * NT * 256 + (nt * 8 + r) * 4), "f"(qs) : "memory");
    } else {
#pragma unroll
      for (int j = 0; j < KD; ++j) {
        w.qf[nt][j][0] = raw[nt][j].x;
        w.qf[nt][j][1] = raw[nt][j].y;
      }
#pragma unroll
      for (int i = 0; i < 2; ++i) w.qs[nt][i] = __shfl_sync(0xffffffffu, qs, (2 * c + i) * 4);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      w.m[nt][i] = -CUDART_INF_F;
      w.l[nt][i] = 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < KD; ++j)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 4; ++i) w.acc[j][nt][i] = 0.f;
  w.e = 1;
  w.lo = 255;
  if constexpr (W::Q_SMEM) __syncwarp();
}

// O += the products of a tile whose V exponents, or those before it, lie far apart.  y + off: a key's weight in log2
// units, -inf where it is hidden.  The keys go by ranges of 11 exponents from the largest on, and a row's weights in a
// range are relative to its largest one there: a product too small for f16 is at most 2^-29 of the largest of its tile,
// row and range.  The sums of a range start from zero and are added to O in fp32, whose unit is 2^kKv8WideUnit.
// Values below 2^-88 beside much larger ones, and terms below 2^-110, are not kept.  Rare: each n-tile reads V again, and
// it is a call with its arrays in local memory, so that the common form keeps its registers.  Measured (us; no V row of
// zeros / the first row of every sequence / one row of 64): 64 sequences of 8000-16000 keys, 4 rows 228 / 346 / 452; 131071
// keys, 32 rows 73.6 / 205 / 385; 4096 keys, d 64 7.3 / 8.9 / 10.1.
template <int D, int NT>
struct Kv8WideTile {
  float acc[D / 16][NT][4];
  float2 x[4][NT];          // log2 of the weights of keys 8o + lane / 4
  int ev[4];                // and their V exponents
  uint32_t v[2], turn;      // this lane's rows of V for ldmatrix, and its chunk swizzle
  Win ring;
  // tokens > 0: the rows of each of so many query tokens by themselves, with only the values that the token sees.
  // last: the last key of the newest one, row0: this lane's first row, G: rows of a token
  int tokens, last, row0, G;
};

template <int D, int NT, bool FINE>
__device__ __noinline__ void kv8_wide(Kv8WideTile<D, NT>& w) {
  constexpr int KD = D / 16, kUp = 14;
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
  int token = w.tokens - 1, lim = w.tokens > 0 ? w.last : kKv8Keys - 1;   // the last key of this pass
#pragma unroll 1
  for (int hi = 255;;) {
    int top = 0;       // this range: exponents top - kKv8Spread .. top
#pragma unroll
    for (int o = 0; o < 4; ++o)
      if (w.ev[o] <= hi && 8 * o + r <= lim) top = max(top, w.ev[o]);
    top = __reduce_max_sync(0xffffffffu, top);
    if (top == 0) {    // no more keys; an older token sees one key less
      if (--token < 0 || --lim < 0) return;
      hi = 255;
      continue;
    }
    hi = top - kKv8Spread - 1;
    const float back = kv8_ratio(top - 127 - kUp - kKv8WideUnit);
    uint32_t keep[2][2];   // bytes of the pairs of keys 16p + 8i + 2c, + 1
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int key = 16 * p + 8 * i + 2 * c;
        keep[p][i] = (key <= lim ? 0x00ff00ffu : 0u) | (key < lim ? 0xff00ff00u : 0u);
      }
#pragma unroll 1
    for (int nt = 0; nt < NT; ++nt) {
      float2 x[4];
      float m[2] = {-CUDART_INF_F, -CUDART_INF_F};
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        const bool in = w.ev[o] <= top && w.ev[o] > hi;
        x[o] = in ? w.x[o][nt] : make_float2(-CUDART_INF_F, -CUDART_INF_F);
        m[0] = fmaxf(m[0], x[o].x);
        m[1] = fmaxf(m[1], x[o].y);
      }
      float up[2], base[2];
      bool mine[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 4));
        m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 8));
        m[i] = fmaxf(m[i], __shfl_xor_sync(0xffffffffu, m[i], 16));
        base[i] = m[i] == -CUDART_INF_F ? 0.f : m[i];
        up[i] = ptx::ex2(base[i]);
        // a row without keys in this range meets none of its NaN
        mine[i] = m[i] != -CUDART_INF_F && (w.tokens == 0 || (w.row0 + 8 * nt + i) / w.G == token);
      }
      uint32_t pf[2][2], pl[2][2];
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        const float v = w.ev[o] <= top && w.ev[o] > hi ? kv8_ratio(w.ev[o] - top + kUp) : 0.f;
        const float2 p = make_float2(ptx::ex2(x[o].x - base[0]) * v, ptx::ex2(x[o].y - base[1]) * v);
        const uint32_t h = ptx::pack_half2(p.x, p.y);
        pf[o >> 1][o & 1] = kv8_transpose(h);
        if constexpr (FINE) {
          const float2 f = half2_floats(h);
          pl[o >> 1][o & 1] = kv8_transpose(ptx::pack_half2(p.x - f.x, p.y - f.y));
        }
      }
#pragma unroll
      for (int j = 0; j < KD; j += 2) {
        float sum[2][4] = {};
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint32_t v[4], f[2][4];
          ptx::ldmatrix_x4_trans(v, smem_clamp(w.v[p] + ((uint32_t)(j << 4) ^ w.turn), 16, w.ring.lo, w.ring.hi,
                                               w.ring.status));
#pragma unroll
          for (int i = 0; i < 4; ++i)
            kv8_unpack(__byte_perm(v[i], 0, 0x3120) & keep[p][i & 1], f[i >> 1][(i & 1) * 2], f[i >> 1][(i & 1) * 2 + 1]);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            kv8_mma(sum[k], f[k], pf[p]);
            if constexpr (FINE) kv8_mma(sum[k], f[k], pl[p]);
          }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (mine[i & 1]) w.acc[j + k][nt][i] = fmaf(sum[k][i] * up[i & 1], back, w.acc[j + k][nt][i]);
      }
    }
  }
}

// Whether a value of the keys first .. valid - 1 is NaN: some token does not see them, and a weight of 0 is not enough.
template <int D>
__device__ __noinline__ bool kv8_hidden_nan(uint32_t st, int eb, int first, int valid, const Win& ring) {
  bool nan = false;
  for (int i = threadIdx.x & 31; i < (valid - first) * (D / 16); i += 32) {
    const int key = first + i / (D / 16);
    const uint32_t at = st + key / eb * kv8_block_bytes(eb, D) + (eb + key % eb) * D + i % (D / 16) * 16;
    uint32_t v[4];
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                 : "r"(smem_clamp(at, 16, ring.lo, ring.hi, ring.status)));
#pragma unroll
    for (int k = 0; k < 4; ++k) nan |= __vcmpeq4(v[k] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0;
  }
  return __any_sync(0xffffffffu, nan);
}

// One tile of `valid` keys, `st` its place in the ring; last: the sequence's last key, counted from the tile's first;
// masked: some key of it is hidden from some row.
// FINE: the weights as two f16 numbers, the rounded one and what was lost.  A weight rounded to f16 is off by as much as
// an f16 output is (64 sequences, against 64 bits: 2.9e-4 instead of 2.1e-4, 1.41 times), so f16 calls take the
// second product; the rounding of a bf16 output is eight times as coarse (1 % more error with one number), and there it
// costs time.  Measured (us, bf16 calls, one number / two): up to 8 rows: 384 sequences of 1000-2000 keys 190.3 / 189.6, 23 of
// 2000-3900 15.2 / 15.6, 16 of 1000-2000 11.5 / 12.4; 16 rows: 64 of 16000-32000 72.6 / 78.7, 64 of 4000-8000 126.3 / 136.1.
template <int D, int NT, int RG, bool FINE>
__device__ __forceinline__ void kv8_tile(Kv8Warp<D, NT, RG>& w, const Kv8Params& a, uint32_t st, int eb, int valid,
                                         int last, bool masked, int rg, int lane, const Win& ring) {
  using W = Kv8Warp<D, NT, RG>;
  constexpr int KD = Kv8Warp<D, NT, RG>::KD;
  const int r = lane >> 2;
  if (masked) {
    if (a.causal && a.T_q > 1 && kv8_hidden_nan<D>(st, eb, max(last - (a.T_q - 1) + 1, 0), valid, ring))
      w.lo = w.lo < kKv8Wide ? kKv8ToToken : kKv8ByToken;
    // V rows that hold no key (there are some in every last tile that is not full): zeros, so that a weight of 0 meets no
    // NaN, and the exponent of the first key, which spreads nothing.  Then the writes are ordered before the next copy
    // into this place.
    for (int i = lane; i < (kKv8Keys - valid) * KD; i += 32) {
      const int key = valid + i / KD;
      const uint32_t to = st + key / eb * kv8_block_bytes(eb, D) + (eb + key % eb) * D + i % KD * 16;
      if (smem_ok(to, 16, ring.lo, ring.hi, ring.status))
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(to), "r"(0) : "memory");
    }
    const uint32_t v_exp = st + 2 * eb * D + eb;
    uint32_t first;
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(first) : "r"(smem_clamp(v_exp, 1, ring.lo, ring.hi, ring.status)));
    if (lane >= valid) {
      const uint32_t to = v_exp + lane / eb * kv8_block_bytes(eb, D) + lane % eb;
      if (smem_ok(to, 1, ring.lo, ring.hi, ring.status)) asm volatile("st.shared.u8 [%0], %1;" ::"r"(to), "r"(first) : "memory");
    }
    ptx::fence_proxy_async_smem();
    __syncwarp();
  }
  // ---- exponents of this lane's keys 8o + r
  int ek[4], ev[4];
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    uint32_t x, y;
    const uint32_t at = smem_clamp(st + w.ex[o], 1, ring.lo, ring.hi, ring.status);
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(at));
    asm volatile("ld.shared.u8 %0, [%1];" : "=r"(y) : "r"(smem_clamp(st + w.ex[o] + eb, 1, ring.lo, ring.hi, ring.status)));
    ek[o] = (int)x;
    ev[o] = (int)y;
  }
  // ---- S^T = K Q^T
  float s[2][NT][4];
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[p][nt][0] = s[p][nt][1] = s[p][nt][2] = s[p][nt][3] = 0.f;
#pragma unroll
  for (int j = 0; j < KD; j += 2) {
    uint32_t q[2][NT][2], x[2][4];
#pragma unroll
    for (int p = 0; p < 2; ++p)
      ptx::ldmatrix_x4(x[p], smem_clamp(st + w.rows[p] + ((uint32_t)(j << 4) ^ w.turn), 16, ring.lo, ring.hi, ring.status));
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if constexpr (W::Q_SMEM) {
          asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                       : "=r"(q[k][nt][0]), "=r"(q[k][nt][1])
                       : "r"(w.q_at + (((j + k) * NT + nt) * 32 + lane) * 8));
        } else {
          q[k][nt][0] = w.qf[nt][j + k][0];
          q[k][nt][1] = w.qf[nt][j + k][1];
        }
      }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint32_t f[2][4];
      kv8_unpack(x[p][0], f[0][0], f[0][2]);
      kv8_unpack(x[p][1], f[0][1], f[0][3]);
      kv8_unpack(x[p][2], f[1][0], f[1][2]);
      kv8_unpack(x[p][3], f[1][1], f[1][3]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) kv8_mma(s[p][nt], f[0], q[0][nt]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) kv8_mma(s[p][nt], f[1], q[1][nt]);
    }
  }
  // ---- y: the logits in log2 units, the scores by the K scales and their row's factor, rounded here once: the weight of a
  // row's largest is 2^0 to 2^kKv8Slack then, however large the logits are.  (An exponent fma(score, factor, -m) would be what
  // rounding the maximum left: from 2^27 on more than f16's weights have room for.)
  // s[p][nt][i]: key 16p + 8 (i / 2) + r, row 2c + i % 2 of n-tile nt
  // over: a score far above the running maximum, or a V exponent outside of what has been seen
  bool over = max(max(ev[0], ev[1]), max(ev[2], ev[3])) > w.e || min(min(ev[0], ev[1]), min(ev[2], ev[3])) < w.lo;
  float mx[NT][2];
  Two y[4][NT], qs[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    if constexpr (W::Q_SMEM) {
      float2 f;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];"
                   : "=f"(f.x), "=f"(f.y)
                   : "r"(w.q_at + KD * NT * 256 + (nt * 8 + 2 * (lane & 3)) * 4));
      qs[nt] = two(f.x, f.y);
    } else {
      qs[nt] = two(w.qs[nt][0], w.qs[nt][1]);
    }
  }
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    const float k = kv8_scale((uint32_t)ek[o]);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) y[o][nt] = mul2(mul2(two(s[o >> 1][nt][(o & 1) * 2], s[o >> 1][nt][(o & 1) * 2 + 1]), two(k, k)), qs[nt]);
  }
  if (masked) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      // the last key that each row sees: token row / G of T_q
      int lim[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = (rg * NT + nt) * 8 + 2 * (lane & 3) + i;
        lim[i] = last - (a.causal ? max(a.T_q - 1 - row / a.G, 0) : 0);
      }
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        const float2 f = split(y[o][nt]);
        y[o][nt] = two(8 * o + r > lim[0] ? -CUDART_INF_F : f.x, 8 * o + r > lim[1] ? -CUDART_INF_F : f.y);
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float2 f0 = split(y[0][nt]), f1 = split(y[1][nt]), f2 = split(y[2][nt]), f3 = split(y[3][nt]);
    mx[nt][0] = fmaxf(fmaxf(f0.x, f1.x), fmaxf(f2.x, f3.x));
    mx[nt][1] = fmaxf(fmaxf(f0.y, f1.y), fmaxf(f2.y, f3.y));
    over |= mx[nt][0] - w.m[nt][0] > kKv8Slack || mx[nt][1] - w.m[nt][1] > kKv8Slack;
  }
  bool wide = false;
  if (__any_sync(0xffffffffu, over)) {
    float fe = 1.f;
    if (w.lo < kKv8Wide || w.lo == kKv8ToToken) {
      int top = w.e, low = w.lo;
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        top = max(top, ev[o]);
        low = min(low, ev[o]);
      }
      top = __reduce_max_sync(0xffffffffu, top);
      low = __reduce_min_sync(0xffffffffu, low);
      if (top - low > kKv8Spread || w.lo == kKv8ToToken) {
        const float f = kv8_ratio(w.e - 127 - kKv8Lift - kKv8WideUnit);
#pragma unroll
        for (int j = 0; j < KD; ++j)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) w.acc[j][nt][i] *= f;
        w.lo = w.lo == kKv8ToToken ? kKv8ByToken : kKv8Wide;
      } else {
        fe = kv8_ratio(w.e - top);
        w.e = top;
        w.lo = low;
      }
    }
    wide = w.lo >= kKv8Wide;
    float f[NT][2];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float x = mx[nt][i];
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
        x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
        x = fmaxf(x, w.m[nt][i]);
        f[nt][i] = ptx::ex2(w.m[nt][i] - (x == -CUDART_INF_F ? 0.f : x));
        w.m[nt][i] = x;
        w.l[nt][i] *= f[nt][i];
        f[nt][i] *= fe;
      }
#pragma unroll
    for (int j = 0; j < KD; ++j)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) w.acc[j][nt][i] *= f[nt][i & 1];
  }
  // ---- weights, and P as the B operand
  Two off[NT], sum[NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    off[nt] = two(w.m[nt][0] == -CUDART_INF_F ? 0.f : -w.m[nt][0], w.m[nt][1] == -CUDART_INF_F ? 0.f : -w.m[nt][1]);
    sum[nt] = two(w.l[nt][0], w.l[nt][1]);
  }
  if (wide) {
    Kv8WideTile<D, NT> t;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        const float2 x = split(add2(y[o][nt], off[nt]));
        sum[nt] = add2(sum[nt], two(ptx::ex2(x.x), ptx::ex2(x.y)));
        t.x[o][nt] = x;
      }
      const float2 f = split(sum[nt]);
      w.l[nt][0] = f.x;
      w.l[nt][1] = f.y;
    }
#pragma unroll
    for (int o = 0; o < 4; ++o) t.ev[o] = ev[o];
#pragma unroll
    for (int p = 0; p < 2; ++p) t.v[p] = st + w.rows[p] + eb * D;
    t.turn = w.turn;
    t.ring = ring;
    t.tokens = w.lo == kKv8ByToken ? a.T_q : 0;
    t.last = last;
    t.row0 = rg * NT * 8 + 2 * (lane & 3);
    t.G = a.G;
#pragma unroll
    for (int j = 0; j < KD; ++j)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) t.acc[j][nt][i] = w.acc[j][nt][i];
    kv8_wide<D, NT, FINE>(t);
#pragma unroll
    for (int j = 0; j < KD; ++j)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) w.acc[j][nt][i] = t.acc[j][nt][i];
    return;
  }
  uint32_t pf[2][NT][2], pl[2][NT][2];
#pragma unroll
  for (int o = 0; o < 4; ++o) {
    const float v = kv8_ratio(ev[o] - w.e + kKv8Lift);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const float2 x = split(add2(y[o][nt], off[nt]));
      const Two p = two(ptx::ex2(x.x), ptx::ex2(x.y));
      sum[nt] = add2(sum[nt], p);
      const float2 pv = split(mul2(p, two(v, v)));
      const uint32_t h = ptx::pack_half2(pv.x, pv.y);
      pf[o >> 1][nt][o & 1] = kv8_transpose(h);
      if constexpr (FINE) {
        const float2 f = half2_floats(h);
        pl[o >> 1][nt][o & 1] = kv8_transpose(ptx::pack_half2(pv.x - f.x, pv.y - f.y));
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const float2 f = split(sum[nt]);
    w.l[nt][0] = f.x;
    w.l[nt][1] = f.y;
  }
  // ---- O^T += V^T P^T; accumulator rows r, r + 8 of tile j: d = 16j + 2r, 16j + 2r + 1
#pragma unroll
  for (int p = 0; p < 2; ++p)
#pragma unroll
    for (int j = 0; j < KD; j += 2) {
      uint32_t x[4], f[2][4];
      ptx::ldmatrix_x4_trans(x, smem_clamp(st + w.rows[p] + eb * D + ((uint32_t)(j << 4) ^ w.turn), 16, ring.lo, ring.hi,
                                           ring.status));
#pragma unroll
      for (int i = 0; i < 4; ++i) kv8_unpack(__byte_perm(x[i], 0, 0x3120), f[i >> 1][(i & 1) * 2], f[i >> 1][(i & 1) * 2 + 1]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        kv8_mma(w.acc[j][nt], f[0], pf[p][nt]);
        kv8_mma(w.acc[j + 1][nt], f[1], pf[p][nt]);
        if constexpr (FINE) {
          kv8_mma(w.acc[j][nt], f[0], pl[p][nt]);
          kv8_mma(w.acc[j + 1][nt], f[1], pl[p][nt]);
        }
      }
    }
}

// A state as it leaves the worker: m + shift, l times `l` = 2^-shift and O times `o` stand for m, l and O.  The shift
// keeps sums of the largest values, and of the smallest, in float's range.  Where it would be lost in m (logits of 2^24 and
// more) a row leaves without it.
template <int D, int NT, int RG>
struct Kv8Units {
  float shift, l, o, far;      // far: what O is multiplied by without the shift
  __device__ __forceinline__ explicit Kv8Units(const Kv8Warp<D, NT, RG>& w) {
    const int s = w.lo >= kKv8Wide || w.e >= 192 ? kKv8WideUnit : (w.e < 64 ? -64 : 0);
    shift = (float)s;
    l = kv8_ratio(-s);
    o = w.lo >= kKv8Wide ? 1.f : kv8_ratio(w.e - 127 - kKv8Lift - s);
    far = kv8_ratio((w.lo >= kKv8Wide ? 0 : w.e - 127 - kKv8Lift - s) + s);
  }
  // a row's m, its l and the factor of its O, as they leave
  __device__ __forceinline__ void leave(float& m, float& sum, float& unit) const {
    const bool apart = fabsf(m) >= 16777216.f;
    m = apart ? m : m + shift;
    sum = apart ? sum : sum * l;
    unit = apart ? far : o;
  }
};

// The end of a piece: the whole unit's output, or the partial of slot >= 0.
template <int D, int NT, int RG, bool BF16>
__device__ __forceinline__ void kv8_end(Kv8Warp<D, NT, RG>& w, const Kv8Params& a, int b, int g, int64_t slot, int rg,
                                        int lane) {
  constexpr int KD = Kv8Warp<D, NT, RG>::KD;
  const int r = lane >> 2, c = lane & 3;
  const Kv8Units<D, NT, RG> u(w);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float l = w.l[nt][i];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      float m = w.m[nt][i], unit;
      u.leave(m, l, unit);
      const int row = (rg * NT + nt) * 8 + 2 * c + i;
      if (row >= a.rows) continue;
      if (slot < 0) {
        const int t = row / a.G;
        const int64_t at = (((int64_t)b * a.T_q + t) * a.h_q + (int64_t)g * a.G + (row - t * a.G)) * D;
        if (!idx_ok(at + D - 1, (int64_t)a.N * a.T_q * a.h_q * D, a.status)) continue;
        const float f = l > 0.f ? 1.f / l : l;      // (0, or NaN)
#pragma unroll
        for (int j = 0; j < KD; ++j)
          Elem<BF16>::store2(reinterpret_cast<__half*>(a.o), at + 16 * j + 2 * r, w.acc[j][nt][i] * f * unit,
                             w.acc[j][nt][2 + i] * f * unit);
      } else {
        const int64_t at = slot * a.rows + row;
        if (!idx_ok(at, 2 * (int64_t)a.workers * a.rows, a.status)) continue;
#pragma unroll
        for (int j = 0; j < KD; ++j)
          *reinterpret_cast<float2*>(a.ws_o + at * D + 16 * j + 2 * r) =
              make_float2(w.acc[j][nt][i] * unit, w.acc[j][nt][2 + i] * unit);
        if (r == 0) {
          a.ws_m[at] = l == l ? m : 0.f;   // NaN scores move no maximum: not to be taken for an empty piece
          a.ws_l[at] = l;
        }
      }
    }
}

// Waits, bounded, for a phase of a barrier; the warp's lanes give up together (a lane that went on alone would wait for the
// others in the next shuffle).  The vote costs 0.8 % of a long call over the 4-bit cache.
__device__ __forceinline__ bool kv8_wait(uint32_t bar, uint32_t phase, uint64_t timeout_ns, const volatile int* abort) {
  return __all_sync(0xffffffffu, ptx::mbar_wait_bounded(bar, phase, timeout_ns, abort));
}

template <int D, int NT, int RG, bool BF16>
__global__ void __launch_bounds__(kKv8Threads, 1)
gqa_decode_kv8_kernel(const Kv8Params a) {
  using C = Kv8Cfg<D, NT, RG>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  int64_t* prefix = reinterpret_cast<int64_t*>(smem + C::PREFIX_OFF);
  int* lens = reinterpret_cast<int*>(smem + C::LENS_OFF);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::FLAG_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / RG, rg = warp % RG;
  const uint32_t full = ptx::smem_u32(smem + C::BAR_OFF) + grp * STAGES * 16, empty = full + STAGES * 8;
  if (threadIdx.x < C::GROUPS * STAGES) {
    const uint32_t f = ptx::smem_u32(smem + C::BAR_OFF) + threadIdx.x / STAGES * STAGES * 16 + threadIdx.x % STAGES * 8;
    ptx::mbar_init(f, 1);
    ptx::mbar_init(f + STAGES * 8, RG);
  }
  if (threadIdx.x == 0) *abort = 0;
  ptx::fence_mbar_init();
  ptx::grid_dependency_wait();
  kv8_prefix(a, prefix, lens, reinterpret_cast<int64_t*>(smem + C::SUMS_OFF));
  if (threadIdx.x == 0) ptx::grid_launch_dependents();
  kv8_empty_rows<D>(a, lens);

  const int64_t total = prefix[a.N] * a.h_kv;
  const int64_t share = (total + a.workers - 1) / a.workers;
  const int64_t wk = (int64_t)grp * gridDim.x + blockIdx.x;
  const int64_t f0 = wk * share, f1 = f0 + share < total ? f0 + share : total;
  if (f0 >= f1) {
    if (lane == 0 && rg == 0 && !a.sliced) a.splits[wk] = make_int4(0, 0, 0, 0);
    return;
  }
  const int n = (int)(f1 - f0);
  Kv8Place at = kv8_find(f0, prefix, a.N, a.h_kv);
  if (lane == 0 && rg == 0) {
    // this range begins inside a unit, and it is the first that does: the unit's pieces are those of the range
    // before (its slot 0 if the unit begins with that range, else 1), this one and as many more as the unit has tiles
    const bool first_cut = at.t > 0 && at.t <= share;
    const int64_t pieces = first_cut ? 1 + (at.tiles - at.t + share - 1) / share : 0;
    const int first = 2 * ((int)wk - 1) + (at.t < share ? 1 : 0);
    if (!a.sliced) a.splits[wk] = make_int4((int)pieces, first, at.b, at.g);
    else if (first_cut) a.splits[at.b * a.h_kv + at.g] = make_int4((int)pieces, first, at.b, at.g);
  }
  const uint32_t ring0 = ptx::smem_u32(smem + C::RING_OFF) + grp * STAGES * C::TILE;
  const Win ring = {ring0, ring0 + STAGES * C::TILE, a.status};
  const uint64_t policy = ptx::policy_evict_first();
  const int eb = min(a.block_size, kKv8Keys);
  uint2 raw[NT][D / 16];
  kv8_load_q<D, NT, RG>(raw, a, at.b, at.g, rg, lane);
  Kv8Stream str;
  int issued = 0;
  if (rg == 0) {
    str.at = at;
    kv8_stream_setup<D>(str, a, lane);
    str.id = kv8_window(a, at, lens[at.b], lane);
    kv8_enter<D>(str, a, prefix, lens, lane);
    for (; issued < n && issued < STAGES; ++issued)
      if (!(issued == 1 && wk == a.stall))
        kv8_copy<D>(str, a, prefix, lens, ring0 + issued * C::TILE, full + issued * 8, policy, lane, ring);
  }
  Kv8Warp<D, NT, RG> w;
  kv8_setup(w, a, ptx::smem_u32(smem + C::Q_OFF) + warp * C::QUERIES, lane);
  int len = lens[at.b];
  kv8_begin<D, NT, RG, BF16>(w, raw, a, len, lane);
  bool fresh = at.t == 0;        // this piece begins with its unit
  int64_t slot = 2 * wk;         // where it goes when it is not the whole unit
  int i = 0, stage = 0, phase = 0;
  for (; i < n; ++i) {
    if (!kv8_wait(full + stage * 8, phase, a.timeout_ns, abort)) break;
    const int key0 = at.t * kKv8Keys;
    const int valid = min(len - key0, kKv8Keys);
    const int sees = a.causal ? len - a.T_q : len - 1;       // the fewest keys that a row sees
    kv8_tile<D, NT, RG, !BF16>(w, a, ring0 + stage * C::TILE, eb, valid, len - 1 - key0, kKv8Keys - 1 > sees - key0, rg, lane, ring);
    __syncwarp();
    if (RG > 1 && lane == 0) ptx::mbar_arrive(empty + stage * 8);
    if (rg == 0 && i + STAGES < n) {
      if (RG > 1 && !kv8_wait(empty + stage * 8, phase, a.timeout_ns, abort)) {
        ++i;
        break;
      }
      kv8_copy<D>(str, a, prefix, lens, ring0 + stage * C::TILE, full + stage * 8, policy, lane, ring);
      ++issued;
    }
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1;
    }
    if (++at.t == at.tiles || i + 1 == n) {
      const bool whole = fresh && at.t == at.tiles;
      if (whole && a.sliced && lane == 0 && rg == 0) a.splits[at.b * a.h_kv + at.g] = make_int4(0, 0, 0, 0);
      kv8_end<D, NT, RG, BF16>(w, a, at.b, at.g, whole ? -1 : slot, rg, lane);
      if (i + 1 < n) {
        kv8_next_unit(at, prefix, a.N, a.h_kv);
        len = lens[at.b];
        kv8_load_q<D, NT, RG>(raw, a, at.b, at.g, rg, lane);
        kv8_begin<D, NT, RG, BF16>(w, raw, a, len, lane);
        fresh = true;
        slot = 2 * wk + 1;
      }
    }
  }
  if (i < n) {
    // a wait gave up: tell the others and wait (bounded) for this worker's copies in flight
    if (lane == 0) {
      atomicOr(a.status, kDevTimeout);
      *abort = 1;
    }
    if (rg == 0)
      for (int k = i; k < issued; ++k)
        ptx::mbar_wait_bounded(full + k % STAGES * 8, k / STAGES & 1, a.timeout_ns, nullptr);
  }
}

// Short kernel: the warps of a CTA leave their states in shared memory (their parts of the drained ring).
template <int D, int NT, int RG>
__device__ __forceinline__ void kv8_leave(Kv8Warp<D, NT, RG>& w, float2* ml, float* o, int lane) {
  constexpr int KD = Kv8Warp<D, NT, RG>::KD;
  const int r = lane >> 2, c = lane & 3;
  const Kv8Units<D, NT, RG> u(w);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float l = w.l[nt][i];
      l += __shfl_xor_sync(0xffffffffu, l, 4);
      l += __shfl_xor_sync(0xffffffffu, l, 8);
      l += __shfl_xor_sync(0xffffffffu, l, 16);
      float m = w.m[nt][i], unit;
      u.leave(m, l, unit);
      const int row = nt * 8 + 2 * c + i;
      if (r == 0) ml[row] = make_float2(m, l);
#pragma unroll
      for (int j = 0; j < KD; ++j)
        *reinterpret_cast<float2*>(o + row * D + 16 * j + 2 * r) =
            make_float2(w.acc[j][nt][i] * unit, w.acc[j][nt][2 + i] * unit);
    }
}

// One row's four columns of n <= 8 states, folded in the order of the keys: state i has its m and l at ml(i), its O at o(i).
template <typename ML, typename O>
__device__ __forceinline__ void kv8_fold(int n, ML ml, O o, float& m, float& l, float4& acc) {
  float2 s[8];
  float4 v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    s[i] = i < n ? ml(i) : make_float2(-CUDART_INF_F, 0.f);
    v[i] = i < n ? o(i) : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  m = -CUDART_INF_F;
  l = 0.f;
  acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int i = 0; i < 8; ++i) m = fmaxf(m, s[i].x);
  const float base = m == -CUDART_INF_F ? 0.f : m;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float f = ptx::ex2(s[i].x - base);
    l += f * s[i].y;      // (NaN scores move no maximum, but their sum is NaN)
    acc.x += f * v[i].x;
    acc.y += f * v[i].y;
    acc.z += f * v[i].z;
    acc.w += f * v[i].w;
  }
}

template <bool BF16>
__device__ __forceinline__ void kv8_store4(const Kv8Params& a, int b, int g, int row, int d, int D, float l, float4 v) {
  const int t = row / a.G;
  const int64_t at = (((int64_t)b * a.T_q + t) * a.h_q + (int64_t)g * a.G + (row - t * a.G)) * D + d;
  if (!idx_ok(at + 3, (int64_t)a.N * a.T_q * a.h_q * D, a.status)) return;
  const float f = l > 0.f ? 1.f / l : l;
  Elem<BF16>::store2(reinterpret_cast<__half*>(a.o), at, v.x * f, v.y * f);
  Elem<BF16>::store2(reinterpret_cast<__half*>(a.o), at + 2, v.z * f, v.w * f);
}

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
  return v;
}

__device__ __forceinline__ float2 ld_cluster_v2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
  return v;
}

// Decode of few, short units in one launch: a cluster of a.ctas CTAs for each (sequence, head), its tiles cut evenly over
// their workers (at most kKv8Short tiles each, so that one window of block ids serves a worker).  There is nothing to
// search: a CTA needs one length.  The warps of a CTA fold their states in shared memory, the CTAs of the cluster
// theirs through distributed shared memory, each a part of the columns, both in the order of the keys.
// Bound by latency: one sequence of 4096 keys, 8 + 2 heads of 64, 5.5 us replayed (1.1 MB, 0.2 us of HBM) against 6.6 of the
// general kernel and its merge.
template <int D, int NT, int RG, bool BF16>
__global__ void __launch_bounds__(kKv8Threads, 1)
gqa_decode_kv8_short_kernel(const Kv8Params a) {
  using C = Kv8Cfg<D, NT, RG>;
  constexpr int STAGES = C::STAGES;
  extern __shared__ __align__(128) uint8_t smem[];
  volatile int* flags = reinterpret_cast<volatile int*>(smem + C::FLAG_OFF);   // [0] abort
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / RG, rg = warp % RG;
  const int unit = blockIdx.x / a.ctas, c = blockIdx.x - unit * a.ctas, b = unit / a.h_kv, g = unit - b * a.h_kv;
  const uint32_t full = ptx::smem_u32(smem + C::BAR_OFF) + grp * STAGES * 16, empty = full + STAGES * 8;
  if (threadIdx.x < C::GROUPS * STAGES) {
    const uint32_t f = ptx::smem_u32(smem + C::BAR_OFF) + threadIdx.x / STAGES * STAGES * 16 + threadIdx.x % STAGES * 8;
    ptx::mbar_init(f, 1);
    ptx::mbar_init(f + STAGES * 8, RG);
  }
  if (threadIdx.x == 0) flags[0] = 0;
  ptx::fence_mbar_init();
  __syncthreads();
  ptx::grid_dependency_wait();
  if (threadIdx.x == 0) ptx::grid_launch_dependents();
  int len = __ldg(a.seq_lens + b);
  const int64_t cap = (int64_t)a.max_blocks * a.block_size;
  if (len < 0 || len > cap) {
    if (threadIdx.x == 0) atomicOr(a.status, kDevBadInput);
    len = len < 0 ? 0 : (int)cap;
  }
  const int tiles = (int)(((int64_t)len + kKv8Keys - 1) / kKv8Keys);
  const int per = max((tiles + a.ctas * C::GROUPS - 1) / (a.ctas * C::GROUPS), 1);
  const int busy_ctas = (tiles + per * C::GROUPS - 1) / (per * C::GROUPS);
  // workers of this CTA that have tiles
  const int busy = max(min((tiles - c * C::GROUPS * per + per - 1) / per, C::GROUPS), 0);
  const int wk = c * C::GROUPS + grp, t0 = wk * per, n = grp < busy ? min(per, tiles - t0) : 0;
  const uint32_t ring0 = ptx::smem_u32(smem + C::RING_OFF) + grp * STAGES * C::TILE;
  const Win ring = {ring0, ring0 + STAGES * C::TILE, a.status};
  const uint64_t policy = ptx::policy_evict_first();
  const int eb = min(a.block_size, kKv8Keys);
  const bool stalled = a.stall >= 0 && a.stall == (int)blockIdx.x * C::GROUPS + grp;
  float2* ml = reinterpret_cast<float2*>(smem + C::ML_OFF);
  bool good = true;
  if (n > 0) {
    Kv8Stream str;
    int issued = 0;
    if (rg == 0) {
      str.at = {b, g, t0, tiles};
      kv8_stream_setup<D>(str, a, lane);
      str.id = kv8_window(a, str.at, len, lane);
    }
    uint2 raw[NT][D / 16];
    kv8_load_q<D, NT, RG>(raw, a, b, g, rg, lane);
    if (rg == 0) {
      kv8_window_begin<D>(str, a, len, lane);
      str.t_end = t0 + n;
      for (; issued < n && issued < STAGES; ++issued)
        if (!(stalled && issued == 1))
          kv8_issue<D>(str, a, ring0 + issued * C::TILE, full + issued * 8, policy, lane, ring);
    }
    Kv8Warp<D, NT, RG> w;
    kv8_setup(w, a, ptx::smem_u32(smem + C::Q_OFF) + warp * C::QUERIES, lane);
    kv8_begin<D, NT, RG, BF16>(w, raw, a, len, lane);
    const int sees = a.causal ? len - a.T_q : len - 1;       // the fewest keys that a row sees
    int i = 0, stage = 0, phase = 0;
    for (; i < n; ++i) {
      good = kv8_wait(full + stage * 8, phase, a.timeout_ns, flags);
      if (!good) break;
      const int key0 = (t0 + i) * kKv8Keys;
      kv8_tile<D, NT, RG, !BF16>(w, a, ring0 + stage * C::TILE, eb, min(len - key0, kKv8Keys), len - 1 - key0,
                                 kKv8Keys - 1 > sees - key0, rg, lane, ring);
      __syncwarp();
      if (RG > 1 && lane == 0) ptx::mbar_arrive(empty + stage * 8);
      if (rg == 0 && i + STAGES < n) {
        if (RG > 1) {
          good = kv8_wait(empty + stage * 8, phase, a.timeout_ns, flags);
          if (!good) break;
        }
        kv8_issue<D>(str, a, ring0 + stage * C::TILE, full + stage * 8, policy, lane, ring);
        ++issued;
      }
      if (++stage == STAGES) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (!good) {
      // a wait gave up: tell the others and wait (bounded) for this worker's copies in flight
      if (lane == 0) {
        atomicOr(a.status, kDevTimeout);
        flags[0] = 1;
      }
      if (rg == 0)
        for (int k = i; k < issued; ++k)
          ptx::mbar_wait_bounded(full + k % STAGES * 8, k / STAGES & 1, a.timeout_ns, nullptr);
    }
    if (RG > 1) __syncwarp();
    if (RG > 1) ptx::named_bar_sync(1 + grp, 32 * RG);   // the other warp of the ring has read its last tile
    if (good) kv8_leave<D, NT, RG>(w, ml + warp * 8 * NT, reinterpret_cast<float*>(smem + C::RING_OFF + warp * C::AREA), lane);
  }
  __syncthreads();
  // ---- the CTA's state: m and l where the general kernel has its prefix sums, O in the first worker's areas (an item is
  // read and written by one thread); the output itself when this CTA has the whole unit
  float2* cta_ml = reinterpret_cast<float2*>(smem + C::PREFIX_OFF);
  uint8_t* areas = smem + C::RING_OFF;
  const bool alone = a.ctas == 1 || tiles == 0;
  if (flags[0] == 0)
    for (int i = threadIdx.x; i < a.rows * (D / 4); i += kKv8Threads) {
      const int row = i / (D / 4), d = i % (D / 4) * 4, part = row / (8 * NT), wrow = row % (8 * NT);
      float m, l;
      float4 v;
      kv8_fold(busy, [&](int k) { return ml[(k * RG + part) * 8 * NT + wrow]; },
               [&](int k) {
                 return *reinterpret_cast<const float4*>(areas + (k * RG + part) * C::AREA + (wrow * D + d) * 4);
               }, m, l, v);
      if (alone) {
        if (c == 0) kv8_store4<BF16>(a, b, g, row, d, D, l, v);
        continue;
      }
      *reinterpret_cast<float4*>(areas + part * C::AREA + (wrow * D + d) * 4) = v;
      if (d == 0) cta_ml[row] = make_float2(m, l);
    }
  if (a.ctas == 1) return;
  // ---- the cluster's fold (every CTA comes here, also one that gave up or has no tiles)
  ptx::cluster_sync();
  if (!alone) {
    const uint32_t ml_at = ptx::smem_u32(cta_ml), o_at = ptx::smem_u32(areas);
    for (int i = c * kKv8Threads + threadIdx.x; i < a.rows * (D / 4); i += a.ctas * kKv8Threads) {
      const int row = i / (D / 4), d = i % (D / 4) * 4, part = row / (8 * NT), wrow = row % (8 * NT);
      float m, l;
      float4 v;
      kv8_fold(busy_ctas, [&](int k) { return ld_cluster_v2(ptx::mapa(ml_at + row * 8, k)); },
               [&](int k) { return ld_cluster_v4(ptx::mapa(o_at + part * C::AREA + (wrow * D + d) * 4, k)); }, m, l, v);
      kv8_store4<BF16>(a, b, g, row, d, D, l, v);
    }
  }
  ptx::cluster_sync();       // no CTA leaves while another reads its shared memory
}

// Folds the pieces of every unit that more than one worker streamed, in the order of its keys.
// SLICED = false, for batches whose units have a few pieces each: a warp for each worker's range (whose first cut
// unit the worker has noted: no search, no division) and row, all D columns.
// SLICED = true, for few units of many pieces: a CTA for 32 columns of one row of a unit, 8 lanes for each piece.
template <int D, bool BF16, bool SLICED>
__global__ void __launch_bounds__(kMergeThreads)
gqa_kv8_merge_kernel(const Kv8Params a) {
  constexpr int WARPS = kMergeThreads / 32;
  constexpr int LANES = SLICED ? 8 : 32;                 // lanes of a piece
  constexpr int PER = (SLICED ? 32 : D) / LANES;         // columns of a lane
  constexpr int SUBS = 32 / LANES, STEP = SLICED ? WARPS * SUBS : 1;
  // pieces of a lane in flight: 4 / 6 / 8 for whole rows 25.1 / 24.1 / 24.6 us (16 sequences of 2000-4000 keys, 8 KV heads)
  constexpr int LOADS = SLICED ? 4 : 6;
  if (threadIdx.x == 0) ptx::grid_launch_dependents();
  ptx::grid_dependency_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int4 noted;    // pieces, first slot, sequence, head
  int row, col = lane % LANES * PER;
  if constexpr (SLICED) {
    const uint32_t r = blockIdx.x / (D / 32), u = r / (uint32_t)a.rows;
    col += (int)(blockIdx.x % (D / 32)) * 32;
    noted = __ldcg(a.splits + u);
    noted.z = (int)(u / (uint32_t)a.h_kv);
    noted.w = (int)(u - (uint32_t)noted.z * (uint32_t)a.h_kv);
    row = (int)(r - u * (uint32_t)a.rows);
  } else {
    const uint32_t i = blockIdx.x * WARPS + warp, w = i / (uint32_t)a.rows;
    if (w >= (uint32_t)a.workers) return;
    noted = __ldcg(a.splits + w);
    row = (int)(i - w * (uint32_t)a.rows);
  }
  const Kv8Note unit = {noted.x, noted.y, noted.z, noted.w};
  if (!kv8_note_ok(unit, a.workers, a.N, a.h_kv)) return;
  const int t = row / a.G;
  const int64_t out = (((int64_t)unit.b * a.T_q + t) * a.h_q + (int64_t)unit.g * a.G + (row - t * a.G)) * D;
  if (!idx_ok(out + D - 1, (int64_t)a.N * a.T_q * a.h_q * D, a.status)) return;
  float M = -CUDART_INF_F, L = 0.f, acc[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) acc[i] = 0.f;
  for (int s0 = SLICED ? warp * SUBS + lane / LANES : 0; s0 < unit.pieces; s0 += LOADS * STEP) {
    float mj[LOADS], lj[LOADS], oj[LOADS][PER];
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int s = s0 + j * STEP;
      const int64_t at = (int64_t)kv8_slot(unit, s) * a.rows + row;
      const bool have = s < unit.pieces && idx_ok(at, 2 * (int64_t)a.workers * a.rows, a.status);
      mj[j] = have ? __ldcg(a.ws_m + at) : -CUDART_INF_F;
      lj[j] = have ? __ldcg(a.ws_l + at) : 0.f;
      const float* src = a.ws_o + at * D + col;
      if constexpr (PER == 4) {
        const float4 v = have ? __ldcg(reinterpret_cast<const float4*>(src)) : make_float4(0.f, 0.f, 0.f, 0.f);
        oj[j][0] = v.x; oj[j][1] = v.y; oj[j][2] = v.z; oj[j][3] = v.w;
      } else {
        const float2 v = have ? __ldcg(reinterpret_cast<const float2*>(src)) : make_float2(0.f, 0.f);
        oj[j][0] = v.x; oj[j][1] = v.y;
      }
    }
    float Mc = M;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) Mc = fmaxf(Mc, mj[j]);
    if (Mc == -CUDART_INF_F) continue;
    const float so = ptx::ex2(M - Mc);
    L *= so;
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] *= so;
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const float f = ptx::ex2(mj[j] - Mc);
      L += f * lj[j];
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] += f * oj[j][i];
    }
    M = Mc;
  }
  if constexpr (SLICED) {
    // the groups of a warp, then the warps
    __shared__ float sm[WARPS][32 + 2];
    float Mt = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, 8));
    Mt = fmaxf(Mt, __shfl_xor_sync(0xffffffffu, Mt, 16));
    const float f = M == -CUDART_INF_F ? 0.f : ptx::ex2(M - Mt);
    L *= f;
    L += __shfl_xor_sync(0xffffffffu, L, 8);
    L += __shfl_xor_sync(0xffffffffu, L, 16);
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      acc[i] *= f;
      acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 8);
      acc[i] += __shfl_xor_sync(0xffffffffu, acc[i], 16);
      if (lane < LANES) sm[warp][lane * PER + i] = acc[i];
    }
    if (lane == 0) {
      sm[warp][32] = Mt;
      sm[warp][33] = L;
    }
    __syncthreads();
    if (threadIdx.x >= LANES) return;
    M = -CUDART_INF_F;
    L = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) M = fmaxf(M, sm[k][32]);
#pragma unroll
    for (int i = 0; i < PER; ++i) acc[i] = 0.f;
#pragma unroll
    for (int k = 0; k < WARPS; ++k) {
      const float g = sm[k][32] == -CUDART_INF_F ? 0.f : ptx::ex2(sm[k][32] - M);
      L += g * sm[k][33];
#pragma unroll
      for (int i = 0; i < PER; ++i) acc[i] += g * sm[k][lane * PER + i];
    }
  }
  const float inv = L > 0.f ? 1.f / L : L;
#pragma unroll
  for (int i = 0; i < PER; i += 2)
    Elem<BF16>::store2(reinterpret_cast<__half*>(a.o), out + col + i, acc[i] * inv, acc[i + 1] * inv);
}

}  // namespace gqa
