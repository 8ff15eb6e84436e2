// Decode attention over paged caches with a sliding window and a few first tokens that stay visible: the 4-bit cache, and
// 16-bit pools (num_blocks, block_size, h_kv * D).
//
// Query token t of T_q newest has the place p = len - T_q + t (causal; else len - 1) and sees key j <= p if j > p - window or
// j < sinks.  A row of keys with a window is a short row: the tiles that no token of it sees are left out, and what remains,
// the sinks' tiles and those from the oldest visible key on, is numbered through; blocks that no token sees are neither copied
// nor looked up, so that their pages may be gone.  All tiles of a launch then lie on one axis that is cut into equal shares,
// one for each worker, as in the kernels of the 8-bit cache, whose plan, partials and merge these kernels share: the cut looks
// at no sequence, and the same call gives the same bits.
//
// A worker is one warp, or two that share a ring (more than 32 query rows; over the 4-bit cache more than 24), with a ring of
// its own in shared memory, filled by one bulk copy for each block of the 4-bit cache, and by 16-byte asynchronous copies from
// the 16-bit pools, whose rows of a head lie apart: a bulk copy for each row costs its lane's turn in a loop over the lanes
// (four warps on an SM: 322 us instead of 206 for 64 sequences under a window of 4096).  Two warps of a ring both convert all
// of its tiles' codes, each for its own query rows.
//
// Measured: 64 sequences of 1K-16K keys, 32 + 8 heads of 128, over the 4-bit cache 100 us (5.6 TB/s of a copy's 6.69;
// bound by issue slots and the ALU's conversions); 64 of 1K-32K over 16 bits under a window of 4096 160 us (6.4 TB/s; DRAM).
//
// Arithmetic of a warp, for its 8 NT query rows and the keys of a tile: S^T = K Q^T and O^T += V^T P^T by mma.sync, keys
// and columns on the M side, query rows on the N side.  kv4: a code becomes f16 by one conversion for two of them, and is
// multiplied by its scale there, exactly; with K, lane c of a row's four holds the elements 32c .. 32c + 31 (D = 128), two
// whole groups, and since the order of the summed index is free, Q is laid out to match; with V, a transposing ldmatrix
// gives four codes of each of two keys, which change places by nibbles so that a byte is the two keys' code of one column.
// The weights are rounded to f16 with 2^kWinLift of headroom below the largest, or kept as two 16-bit numbers (FINE).
// The running maximum is only moved when a score exceeds it by 2^kKv8Slack.
#pragma once
#include "gqa_kv4.cuh"
#include "gqa_kv8_decode.cuh"

namespace gqa {

constexpr int kWinSeqs = 768;      // sequences of a launch (the host splits larger batches): what the rings leave room for

// What is copied where the 4-bit cache has no block: zeros, as many as one copy brings at most.
__device__ const uint4 kWinZeros[kv4_block_bytes(32, 128) / 16] = {};

struct WinParams : Kv8Params {
  const uint16_t *k_pool, *v_pool;   // 16-bit pools; the 4-bit cache is `cache`
  int window;                        // 0: none
  int sinks, sink_tiles;             // first keys that stay visible (0 without a window)
  int ids_log;                       // log2 of the block ids of a tile
};

// Keys of a tile: 64 where the registers allow it (two independent halves, and half the work around a tile: 12 warps with
// two tiles of 64 keys 100.8 us instead of 119 for 64 sequences of 1K-16K keys over the 4-bit cache, 16 query rows of 64
// sequences 164 instead of 182), 32 otherwise, and for 16 bits, whose rows fill the ring (d_head 64: no faster with 64).
template <bool KV4, int NT>
constexpr int win_keys = KV4 && NT <= 2 ? 64 : 32;

template <int D, int NT, int RG, bool KV4>
struct WinCfg {
  // 16 rows of 64 elements leave the registers for twelve warps too (64 sequences of 1K-16K keys 104 us instead of 115); of
  // 128 they do not (spills: 194 us instead of 164)
  static constexpr int WARPS = NT == 1 || (KV4 && NT == 2 && D == 64) ? 12 : 8;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int GROUPS = WARPS / RG;
  static constexpr int KEYS = win_keys<KV4, NT>;                   // of a tile: one or two of 32, laid out one after the other
  static constexpr int TILE = KEYS * (KV4 ? D + D / 8 : 4 * D);
  static constexpr bool Q_SMEM = NT > 2 || (KV4 && NT == 2);          // query fragments in shared memory, else in registers
  static constexpr int QUERIES = Q_SMEM ? 8 * NT * (D * 2 + 4) : 0;   // of a warp, and its rows' factors
  static constexpr int PREFIX_OFF = 0;
  static constexpr int LENS_OFF = (kWinSeqs + 2) * 8;
  static constexpr int SUMS_OFF = LENS_OFF + kWinSeqs * 4;
  static constexpr int FLAG_OFF = SUMS_OFF + WARPS * 8;
  static constexpr int BAR_OFF = FLAG_OFF + 16;
  // Tiles of a warp in the ring.  The 4-bit cache takes two (NT > 2: four, of 32 keys).  16 bits: one, and the other warps
  // compute while it comes (12 warps with one tile of 32 keys 160 us instead of 206 with 4 warps and three, 64 sequences
  // under a window of 4096).
  static constexpr int DEPTH = KV4 ? (NT > 2 ? 4 : 2) * (NT == 2 ? 1 : 128 / D) : 128 / D;
  static constexpr int STAGES = DEPTH * RG;
  static constexpr int Q_OFF = (BAR_OFF + GROUPS * STAGES * 16 + 127) & ~127;
  static constexpr int ML_OFF = Q_OFF + WARPS * QUERIES;
  static constexpr int RING_OFF = (ML_OFF + WARPS * 8 * NT * 8 + 127) & ~127;
  static constexpr int SMEM = RING_OFF + GROUPS * STAGES * TILE;
  static constexpr int AREA = STAGES * TILE / RG;                     // a warp's part of the ring: holds its O there
  static_assert(GROUPS * STAGES <= THREADS && SMEM <= 232448 && AREA >= 8 * NT * D * 4 && AREA % 16 == 0, "ring");
  static constexpr int FULL = KV4 ? 1 : 32;                           // arrivals at a full barrier: the lane that expects, or all
  static constexpr int FOLD = GROUPS > 8 ? GROUPS : 8;                // states that one fold takes: a CTA's workers, a cluster's CTAs
};

// log2 of what a weight is multiplied by: its f16 is at most 2^15
template <bool KV4, bool BF16>
constexpr int kWinLift = KV4 || !BF16 ? 11 : 0;

// The visible part of a sequence of len keys: the first key behind the sinks that some token sees, the tiles that are left out
// between the sinks' and those, and the number of the others.
struct WinSpan {
  int first, skip, tiles;
};

template <int K>
__device__ __forceinline__ WinSpan win_span(const WinParams& a, int len) {
  WinSpan s = {0, 0, (int)(((int64_t)len + K - 1) / K)};
  if (a.window > 0) {
    const int64_t first = (int64_t)len - (a.causal ? a.T_q : 1) - a.window + 1;
    if (first > 0) {
      s.first = (int)first;
      s.skip = max(s.first / K - a.sink_tiles, 0);
      s.tiles -= s.skip;
    }
  }
  return s;
}

// The tiles [from, from + count) of a unit, as it numbers them, of which every token sees every key.
struct WinClear {
  int from;
  uint32_t count;
  __device__ __forceinline__ bool has(int t) const { return (uint32_t)(t - from) < count; }
};

template <int K>
__device__ __forceinline__ WinClear win_clear_tiles(const WinParams& a, int len, int skip) {
  const int last = a.causal ? len - a.T_q : len - 1;         // the oldest token's place
  const int end = last >= 0 ? (int)(((int64_t)last + 1) / K) : 0;
  int from = 0;
  if (a.window > 0 && len > a.window && len - a.window > a.sinks)   // the newest token's oldest key
    from = (int)(((int64_t)len - a.window + K - 1) / K);
  return {from - skip, (uint32_t)max(end - from, 0)};
}

__device__ __forceinline__ int win_tile_of(const WinParams& a, int skip, int t) { return t < a.sink_tiles ? t : t + skip; }

// Tiles (of one head) before each sequence of the launch, in shared memory.
template <int K, int THREADS>
__device__ __forceinline__ void win_prefix(const WinParams& a, int64_t* prefix, int* lens, int64_t* sums) {
  constexpr int PER = (kWinSeqs + THREADS - 1) / THREADS;
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
    if (b < kWinSeqs) lens[b] = len;
    run += win_span<K>(a, len).tiles;
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
template <int D, int THREADS>
__device__ __forceinline__ void win_empty_rows(const WinParams& a, const int* lens) {
  const int64_t words = (int64_t)a.T_q * a.h_q * D / 8;
  for (int b = blockIdx.x; b < a.N; b += gridDim.x)
    if (lens[b] == 0) {
      for (int64_t i = threadIdx.x; i < words; i += THREADS)
        reinterpret_cast<uint4*>(a.o)[b * words + i] = make_uint4(0u, 0u, 0u, 0u);
      if (a.sliced)
        for (int g = threadIdx.x; g < a.h_kv; g += THREADS) a.splits[b * a.h_kv + g] = make_int4(0, 0, 0, 0);
    }
}

// ---------------------------------------------------------------- the copying side of a worker
// Block ids go by windows of 32, one for each lane: of the 32 >> ids_log tiles from one on.
struct WinStream {
  Kv8Place at;       // next tile to copy
  Kv8Place ahead;    // first tile after the current window
  int id, id_next;   // this lane's block id in the current window and the one after it (-1: no block, or a bad id)
  bool want, want_next;   // the lane has a block that some token sees
  int len, skip, first;   // of at's sequence
  int t_end;         // tile of at's unit where the current window ends
  int k;             // at's place in the window
  // kv4, the same for every tile: lanes 0 .. n - 1 copy `size` bytes from `off` of a (block, head) to `to` of the tile,
  // + step in the second half of a block of 64; `head` is `off` in head at.g of block 0, `stride` the bytes of a block
  const uint8_t* head;
  int n;
  uint32_t size, to, off, step, stride;
};

template <int D, bool KV4, int K>
__device__ __forceinline__ void win_stream_setup(WinStream& s, const WinParams& a, int lane) {
  s.off = 0;
  if constexpr (KV4) {
    const int bs = a.block_size, bb = kv4_block_bytes(bs, D);
    s.stride = (uint32_t)a.h_kv * (uint32_t)bb;
    if (bs <= 32) {              // whole blocks
      s.n = K >> a.bs_log;
      s.size = bb;
      s.to = lane * bb;
      s.off = s.step = 0;
    } else {                     // half a block, or each half: K codes, V codes, K scales, V scales
      const int part = lane & 3, h = lane >> 2;
      const bool codes = part < 2;
      s.n = K / 8;
      s.size = s.step = 32 * (codes ? D / 2 : D / 16);
      s.to = h * 32 * (D + D / 8) + (codes ? part * s.size : 32 * D + (part - 2) * s.size);
      s.off = (codes ? part * bs * (D / 2) : bs * D + (part - 2) * bs * (D / 16)) + h * s.size;
    }
  }
}

// this lane's block id of the window that starts at p
template <int K>
__device__ __forceinline__ int win_ids(const WinParams& a, const Kv8Place& p, int len, bool& want, int lane) {
  const WinSpan span = win_span<K>(a, len);
  const int t = p.t + (lane >> a.ids_log), tile = win_tile_of(a, span.skip, t);
  const int64_t j = a.block_size <= K ? ((int64_t)tile << a.ids_log) + (lane & ((1 << a.ids_log) - 1)) : tile >> 1;
  const int64_t key = j << a.bs_log, end = key + a.block_size;
  want = t < p.tiles && key < len && (key < a.sinks || end > span.first) &&
         idx_ok((int64_t)p.b * a.max_blocks + j, (int64_t)a.N * a.max_blocks, a.status);
  return want ? __ldg(a.block_tables + (int64_t)p.b * a.max_blocks + j) : -1;
}

template <int D>
__device__ __forceinline__ void win_ids_check(WinStream& s, const WinParams& a) {
  s.head = a.cache + (int64_t)s.at.g * kv4_block_bytes(a.block_size, D) + s.off;
  if (s.want && (s.id < 0 || s.id >= a.num_blocks)) {
    atomicOr(a.status, kDevBadInput);
    s.id = -1;
  }
  s.k = 0;
}

// Enters the window at s.at, whose ids are in s.id: reports bad ids, finds where the next window begins and starts
// loading its ids.
template <int D, int K>
__device__ __forceinline__ void win_enter(WinStream& s, const WinParams& a, const int64_t* prefix, const int* lens, int lane) {
  s.len = lens[s.at.b];
  const WinSpan span = win_span<K>(a, s.len);
  s.skip = span.skip;
  s.first = span.first;
  win_ids_check<D>(s, a);
  s.t_end = min(s.at.tiles, s.at.t + (32 >> a.ids_log));
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
  s.want_next = false;
  s.id_next = s.ahead.b < a.N ? win_ids<K>(a, s.ahead, lens[s.ahead.b], s.want_next, lane) : -1;
}

// bits 0 .. n - 1
__device__ __forceinline__ uint32_t win_below(int n) { return n <= 0 ? 0u : (n >= 32 ? ~0u : (1u << n) - 1); }

// Copies the stream's next tile to `dst`; on to the next tile of the window (true: the window ends).  Every lane of the
// warp calls this.
template <int D, bool KV4, int K>
__device__ __forceinline__ bool win_issue(WinStream& s, const WinParams& a, uint32_t dst, uint32_t bar, uint64_t policy,
                                          int lane, const Win& ring) {
  const bool half = a.block_size > 32;       // the 32 rows of a copy are a part of a block
  const int tile = win_tile_of(a, s.skip, s.at.t);
  if constexpr (KV4) {
    const int id = __shfl_sync(0xffffffffu, s.id, ((s.k << a.ids_log) + (half ? 0 : lane)) & 31);
    if (lane == 0) ptx::mbar_arrive_expect_tx(bar, K * (D + D / 8));
    if (lane < s.n) {
      const uint8_t* src = s.head + (uint64_t)(uint32_t)id * s.stride + (K == 32 ? (tile & 1) * s.step : 0u);
      if (id < 0) src = reinterpret_cast<const uint8_t*>(kWinZeros);       // no block, or one with a bad id
      if ((id < 0 || idx_ok(src + s.size - 1 - a.cache, (int64_t)a.num_blocks * s.stride, a.status)) &&
          smem_ok(dst + s.to, s.size, ring.lo, ring.hi, ring.status))
        bulk_load(dst + s.to, src, s.size, bar, policy);
    }
  } else {
    // Every lane copies as often as every other: rows that no token sees, or of a block with a bad id, are zeros, so that a
    // weight of 0 meets no NaN there.  No branch, and no cache hint, which would take two more instructions a copy.
    static_assert(K == 32, "a key for each bit of a register");
    constexpr int CH = D / 8, KEYS = 32 / CH;     // chunks of a row; keys that the lanes copy at once
    const int key0 = tile * K, first = a.block_size > K ? (tile & 1) * K : 0, c = lane % CH;
    const uint32_t seen = (win_below(s.len - key0) & (~win_below(s.first - key0) | win_below(a.sinks - key0))) >> (lane / CH);
    const int64_t row = (int64_t)a.h_kv * D, apart = a.v_pool - a.k_pool;
    const uint32_t to = dst + lane / CH * (2 * D);
#pragma unroll
    for (int o = 0; o < K / 8; ++o) {       // eight keys lie in one block
      const int id = __shfl_sync(0xffffffffu, s.id, ((s.k << a.ids_log) + (8 * o >> a.bs_log)) & 31);
      const int r = lane / CH + ((first + 8 * o) & (a.block_size - 1));
      const uint16_t* from = a.k_pool + ((int64_t)max(id, 0) * a.block_size + r) * row + s.at.g * D + 8 * c;
      const uint32_t some = id < 0 ? 0u : seen >> (8 * o);
#pragma unroll
      for (int i = 0; i < 8 / KEYS; ++i, from += KEYS * row) {
        const uint32_t at = to + (8 * o + i * KEYS) * (2 * D) + ((c ^ ((i * KEYS + lane / CH) & 7)) << 4);
        uint32_t bytes = (some >> (i * KEYS) & 1) << 4;
        if (!idx_ok(from + 7 - a.k_pool, (int64_t)a.num_blocks * a.block_size * row, a.status)) bytes = 0;
        if (smem_ok(at, K * 2 * D + 16, ring.lo, ring.hi, ring.status)) {
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at), "l"(from), "r"(bytes) : "memory");
          asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(at + K * 2 * D), "l"(from + apart), "r"(bytes) : "memory");
        }
      }
    }
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
  }
  if (++s.at.t == s.t_end) return true;
  ++s.k;
  return false;
}

// the same, and on to the next window
template <int D, bool KV4, int K>
__device__ __forceinline__ void win_copy(WinStream& s, const WinParams& a, const int64_t* prefix, const int* lens, uint32_t dst,
                                         uint32_t bar, uint64_t policy, int lane, const Win& ring) {
  if (!win_issue<D, KV4, K>(s, a, dst, bar, policy, lane, ring)) return;
  s.at = s.ahead;
  s.id = s.id_next;
  s.want = s.want_next;
  if (s.at.b < a.N) win_enter<D, K>(s, a, prefix, lens, lane);
}

// ---------------------------------------------------------------- the computing side
// RG warps share a ring, each with NT n-tiles of 8 query rows.
template <int D, int NT, int RG, bool KV4>
struct WinWarp {
  static constexpr int KD = D / 16;
  static constexpr bool Q_SMEM = WinCfg<D, NT, RG, KV4>::Q_SMEM;
  uint32_t qf[Q_SMEM ? 1 : NT][Q_SMEM ? 1 : KD][2];   // Q^T fragments, or, in shared memory at q_at, [KD][NT][lane] ...
  float qs[Q_SMEM ? 1 : NT][2];                       // ... followed by the rows' factors
  uint32_t q_at;
  float acc[KD][NT][4];
  float m[NT][2], l[NT][2];
  // the same for every unit and tile
  // byte offsets in a tile.  kv4: this lane's part of the K rows 8o + lane / 4 and their scales, from which the scales of
  // the V rows 8o + 2 (lane % 4) are v_scale away, and its rows of V for ldmatrix (without the swizzled chunk); 16 bits:
  // k_at[0] and v_at[0], of the first sixteen keys
  uint32_t k_at[KV4 ? 4 : 1], k_scale[KV4 ? 4 : 1], v_at[KV4 ? 2 : 1], v_scale;
  uint32_t k_turn, v_turn;
  uint32_t pick[2];
};

// a value that stays in its register
__device__ __forceinline__ void win_keep(uint32_t& x) { asm volatile("" : "+r"(x)); }

template <int D, int NT, int RG, bool KV4>
__device__ __forceinline__ void win_setup(WinWarp<D, NT, RG, KV4>& w, const WinParams& a, uint32_t q_at, int lane) {
  w.q_at = q_at + lane * 8;
  const int r = lane >> 2, c = lane & 3, q = lane >> 3, i = lane & 7;
  if constexpr (KV4) {
    const int eb = min(a.block_size, 32), bb = kv4_block_bytes(eb, D);
    const int part = D == 128 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : r * 32 + (((c >> 1) ^ ((r >> 2) & 1)) << 4) + (c & 1) * 8;
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      const int block = 8 * o / eb * bb, row = 8 * o % eb;
      w.k_at[o] = block + row * (D / 2) + part;
      w.k_scale[o] = block + eb * D + (row + r) * (D / 16) + (D / 64) * c;
    }
    w.v_scale = eb * (D / 16) + (2 * c - r) * (D / 16) - (D / 64) * c;
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      const int key = 16 * p + 8 * (q & 1) + i;
      w.v_at[p] = key / eb * bb + (eb + key % eb) * (D / 2);
    }
    w.v_turn = ((q >> 1) ^ (D == 128 ? ((i >> 1) & 3) : ((i >> 2) & 1))) << 4;
    w.pick[0] = kv4_pick(r >> 2, r >> 2);
    w.pick[1] = kv4_pick(2 + (r >> 2), 2 + (r >> 2));
    // Worked out once: without this the compiler does it again for every tile.
    win_keep(w.q_at);
    win_keep(w.v_scale);
    win_keep(w.v_turn);
#pragma unroll
    for (int o = 0; o < 4; ++o) {
      win_keep(w.k_at[o]);
      win_keep(w.k_scale[o]);
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      win_keep(w.v_at[p]);
      win_keep(w.pick[p]);
    }
  } else {
    w.k_at[0] = (8 * (q & 1) + i) * (2 * D);
    w.k_turn = ((q >> 1) ^ i) << 4;
    w.v_at[0] = win_keys<KV4, NT> * 2 * D + (8 * (q >> 1) + i) * (2 * D);
    w.v_turn = ((q & 1) ^ i) << 4;
  }
}

// column of accumulator row r (half 0) or r + 8 (half 1) of m-tile j
template <bool KV4>
__device__ __forceinline__ int win_column(int j, int half, int r) {
  return KV4 ? 32 * (j >> 1) + 4 * r + 2 * (j & 1) + half : 16 * j + 8 * half + r;
}

// A piece begins: its queries are loaded, ...
template <int D, int NT, int RG, bool KV4>
__device__ __forceinline__ void win_load_q(uint2 (&raw)[NT][D / 16], const WinParams& a, int b, int g, int rg, int lane) {
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int row = (rg * NT + nt) * 8 + r, t = row / a.G;
    const int64_t at = (((int64_t)b * a.T_q + t) * a.h_q + (int64_t)g * a.G + (row - t * a.G)) * D;
    const bool ok = row < a.rows && idx_ok(at + D - 1, (int64_t)a.N * a.T_q * a.h_q * D, a.status);
#pragma unroll
    for (int j = 0; j < D / 16; ++j) {
      raw[nt][j] = make_uint2(0u, 0u);
      if (ok) {
        if constexpr (KV4) {       // (the four elements of step j of lane c's part of a K row)
          raw[nt][j] = __ldg(reinterpret_cast<const uint2*>(a.q + at + (D / 4) * c + 4 * j));
        } else {
          raw[nt][j].x = __ldg(reinterpret_cast<const uint32_t*>(a.q + at + 16 * j + 2 * c));
          raw[nt][j].y = __ldg(reinterpret_cast<const uint32_t*>(a.q + at + 16 * j + 8 + 2 * c));
        }
      }
    }
  }
}

// ... brought into the MMA's form, and the state is emptied.
template <int D, int NT, int RG, bool KV4, bool BF16>
__device__ __forceinline__ void win_begin(WinWarp<D, NT, RG, KV4>& w, uint2 (&raw)[NT][D / 16], const WinParams& a, int lane) {
  using W = WinWarp<D, NT, RG, KV4>;
  constexpr int KD = W::KD;
  const int r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float qs = fabsf(a.scale_log2);
    if (a.scale_log2 < 0.f) {    // the factor of a row is kept >= 0, so that the largest y is the largest logit
#pragma unroll
      for (int j = 0; j < KD; ++j) raw[nt][j] = make_uint2(raw[nt][j].x ^ 0x80008000u, raw[nt][j].y ^ 0x80008000u);
    }
    if constexpr (KV4 && BF16) {       // bf16 queries into f16's range by a power of two for each row
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
        asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(w.q_at + (j * NT + nt) * 256), "r"(raw[nt][j].x),
                     "r"(raw[nt][j].y)
                     : "memory");
      if (c == 0) asm volatile("st.shared.f32 [%0], %1;" ::"r"(w.q_at - lane * 8 + KD * NT * 256 + (nt * 8 + r) * 4), "f"(qs) : "memory");
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
  if constexpr (W::Q_SMEM) __syncwarp();
}

template <bool BF16>
__device__ __forceinline__ void win_mma(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
  if constexpr (BF16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
  else
    kv8_mma(d, a, b);
}

// Which keys of a tile a query token sees; places are counted from the tile's first key.
struct WinMask {
  int last, lo;        // the newest token's place, and the oldest key in its window (or one far before the tile)
  int sinks;           // keys below stay visible
  int back;            // the oldest token's distance from the newest
  // seen by the token `back` places before the newest
  __device__ __forceinline__ bool sees(int key, int behind) const {
    return key <= last - behind && (key < sinks || key >= lo - behind);
  }
  // seen by some token, and by every one
  __device__ __forceinline__ bool any(int key) const { return key <= last && (key < sinks || key >= lo - back); }
  __device__ __forceinline__ bool all(int key) const { return key <= last - back && (key < sinks || key >= lo); }
};

__device__ __forceinline__ WinMask win_mask(const WinParams& a, int len, int key0) {
  WinMask k;
  k.last = len - 1 - key0;
  k.lo = a.window > 0 ? max(k.last - (a.window - 1), -(1 << 20)) : -(1 << 20);
  k.sinks = a.sinks - key0;
  k.back = a.causal ? a.T_q - 1 : 0;
  return k;
}

// byte offsets in a tile of the V scales of a key (kv4)
template <int D>
__device__ __forceinline__ uint32_t win_v_scales(int key, int eb) {
  return key / eb * kv4_block_bytes(eb, D) + eb * (D + D / 16) + key % eb * (D / 16);
}

// Values of keys that no token sees: zeros, by their scales, so that a weight of 0 meets no NaN.  (Rows of 16 bits come as
// zeros.)
template <int D, int K>
__device__ __forceinline__ void win_clear(const WinMask& k, uint32_t st, int eb, int lane, const Win& ring) {
#pragma unroll
  for (int key = lane; key < K; key += 32) {
    const uint32_t to = st + win_v_scales<D>(key, eb);
    if (!k.any(key) && smem_ok(to, D / 16, ring.lo, ring.hi, ring.status)) {
      if constexpr (D == 128) asm volatile("st.shared.v2.b32 [%0], {%1, %1};" ::"r"(to), "r"(0) : "memory");
      else asm volatile("st.shared.b32 [%0], %1;" ::"r"(to), "r"(0) : "memory");
    }
  }
  ptx::fence_proxy_async_smem();     // before the next bulk copy into this place
  __syncwarp();
}

template <bool BF16>
__device__ __forceinline__ bool win_infinite(uint32_t x) {     // one of two 16-bit values
  constexpr uint32_t E = BF16 ? 0x7f80u : 0x7c00u;
  return (x & E) == E || (x >> 16 & E) == E;
}

// Whether a value of a key that some token sees and another does not is not finite: then a weight of 0 is not enough.
template <int D, bool KV4, bool BF16, int K>
__device__ __noinline__ bool win_hidden_infinite(WinMask k, uint32_t st, int eb, Win ring) {
  const int lane = threadIdx.x & 31;
  bool bad = false;
  if constexpr (KV4) {
    for (int key = lane; key < K; key += 32) {
      if (!k.any(key) || k.all(key)) continue;
      const uint32_t at = smem_clamp(st + win_v_scales<D>(key, eb), D / 16, ring.lo, ring.hi, ring.status);
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        uint32_t s;
        asm volatile("ld.shared.u8 %0, [%1];" : "=r"(s) : "r"(at + i));
        bad |= s >= kKv4Infinite;
      }
    }
  } else {
    for (uint32_t some = __ballot_sync(0xffffffffu, k.any(lane) && !k.all(lane)); some != 0; some &= some - 1) {
      uint32_t v[D / 64];
      const uint32_t at = smem_clamp(st + (K + __ffs(some) - 1) * (2 * D) + lane * (D / 16), D / 16, ring.lo,
                                     ring.hi, ring.status);
#pragma unroll
      for (int j = 0; j < D / 64; ++j) {
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[j]) : "r"(at + 4 * j));
        bad |= win_infinite<BF16>(v[j]);
      }
    }
  }
  return __any_sync(0xffffffffu, bad);
}

// O += the values of such a tile, each by the rows that see its key.  Rare: one key and column after the other, and a call
// with its arrays in local memory, so that the common form keeps its registers.
template <int D, int NT, int K>
struct WinSlow {
  float acc[D / 16][NT][4];
  float2 p[K / 8][NT];      // weights of keys 8o + lane / 4
  int behind[NT][2];        // this lane's rows: distance of their token from the newest one
  WinMask mask;
  uint32_t st;
  int eb;
  Win ring;
};

template <int D, int NT, bool KV4, bool BF16, int K>
__device__ __noinline__ void win_slow_values(WinSlow<D, NT, K>& w) {
  constexpr int KD = D / 16;
  const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
#pragma unroll 1
  for (int key = 0; key < K; ++key) {
    if (!w.mask.any(key)) continue;
#pragma unroll 1
    for (int j = 0; j < KD; ++j)
#pragma unroll 1
      for (int half = 0; half < 2; ++half) {
        const int d = win_column<KV4>(j, half, r);
        float v;
        if constexpr (KV4) {
          const int row = key % w.eb;
          const uint32_t at = w.st + key / w.eb * kv4_block_bytes(w.eb, D) + w.eb * (D / 2) + kv4_chunk<D>(row, d / 32) + d % 32 / 2;
          const uint32_t sat = w.st + win_v_scales<D>(key, w.eb) + d / 16;
          uint32_t x, s, h[4];
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(x) : "r"(smem_clamp(at, 1, w.ring.lo, w.ring.hi, w.ring.status)));
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(s) : "r"(smem_clamp(sat, 1, w.ring.lo, w.ring.hi, w.ring.status)));
          kv4_unpack(x >> (d % 2 * 4), h);
          v = s >= kKv4Infinite ? CUDART_NAN_F : half2_floats(h[0]).x * kv4_scale(s);
        } else {
          uint16_t x;
          const uint32_t at = w.st + (K + key) * (2 * D) + (((d >> 3) ^ (key & 7)) << 4) + (d & 7) * 2;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(smem_clamp(at, 2, w.ring.lo, w.ring.hi, w.ring.status)));
          v = BF16 ? __uint_as_float((uint32_t)x << 16) : __half2float(*reinterpret_cast<const __half*>(&x));
        }
#pragma unroll 1
        for (int nt = 0; nt < NT; ++nt) {
          const float2 mine = w.p[key >> 3][nt];
          const float2 p = make_float2(__shfl_sync(0xffffffffu, mine.x, (key & 7) * 4 + c),
                                       __shfl_sync(0xffffffffu, mine.y, (key & 7) * 4 + c));
          if (w.mask.sees(key, w.behind[nt][0])) w.acc[j][nt][2 * half] += p.x * v;
          if (w.mask.sees(key, w.behind[nt][1])) w.acc[j][nt][2 * half + 1] += p.y * v;
        }
      }
  }
}

// the shared-memory reads of a tile, free to be scheduled among the products
__device__ __forceinline__ uint4 win_lds4(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ uint2 win_lds2(uint32_t at) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
  return v;
}

// the low four bits of a's bytes, the high ones of b's
__device__ __forceinline__ uint32_t win_low_nibbles(uint32_t a, uint32_t b) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, 0x0f0f0f0f, 0xe4;" : "=r"(y) : "r"(a), "r"(b));
  return y;
}

// One tile of keys key0 ..; masked: some token may not see some key of it.  FINE: the weights as two 16-bit numbers, the rounded one and what was lost.
template <int D, int NT, int RG, bool KV4, bool BF16, bool FINE>
__device__ __forceinline__ void win_tile(WinWarp<D, NT, RG, KV4>& w, const WinParams& a, uint32_t st, int eb, int len, int key0,
                                         bool masked, int rg, int lane, const Win& ring) {
  using W = WinWarp<D, NT, RG, KV4>;
  constexpr int KD = W::KD, K = win_keys<KV4, NT>, OCTETS = K / 8, SUB = 32 * (D + D / 8);   // SUB: bytes of 32 keys (kv4)
  constexpr bool B = !KV4 && BF16;      // bf16 products
  const int r = lane >> 2, c = lane & 3;
  const bool apart = masked && a.causal && a.T_q > 1;     // tokens see different keys
  bool infinite = false;
  if (masked) {
    const WinMask mask = win_mask(a, len, key0);
    if (apart) infinite = win_hidden_infinite<D, KV4, BF16, K>(mask, st, eb, ring);
    if constexpr (KV4) win_clear<D, K>(mask, st, eb, lane, ring);
  }
  // ---- S^T = K Q^T
  float s[K / 16][NT][4];
#pragma unroll
  for (int p = 0; p < K / 16; ++p)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) s[p][nt][0] = s[p][nt][1] = s[p][nt][2] = s[p][nt][3] = 0.f;
  auto query = [&](uint32_t (&q)[NT][2], int j) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      if constexpr (W::Q_SMEM) {
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];"
                     : "=r"(q[nt][0]), "=r"(q[nt][1])
                     : "r"(w.q_at + (j * NT + nt) * 256));
      } else {
        q[nt][0] = w.qf[nt][j][0];
        q[nt][1] = w.qf[nt][j][1];
      }
    }
  };
  if constexpr (KV4) {
    constexpr int WORDS = D / 32;
#pragma unroll
    for (int h = 0; h < K / 32; ++h) {
      uint32_t x[4][WORDS], sc[4][WORDS / 2];
#pragma unroll
      for (int o = 0; o < 4; ++o) {
        const uint32_t at = smem_clamp(st + w.k_at[o] + h * SUB, D / 8, ring.lo, ring.hi, ring.status);
        const uint32_t sat = smem_clamp(st + w.k_scale[o] + h * SUB, D / 64, ring.lo, ring.hi, ring.status);
        if constexpr (D == 128) {
          const uint4 v = win_lds4(at);
          x[o][0] = v.x; x[o][1] = v.y; x[o][2] = v.z; x[o][3] = v.w;
          uint16_t two;
          asm volatile("ld.shared.u16 %0, [%1];" : "=h"(two) : "r"(sat));
          sc[o][0] = kv4_scales(two, two, kv4_pick(0, 0));
          sc[o][1] = kv4_scales(two, two, kv4_pick(1, 1));
        } else {
          const uint2 v = win_lds2(at);
          x[o][0] = v.x; x[o][1] = v.y;
          uint32_t one;
          asm volatile("ld.shared.u8 %0, [%1];" : "=r"(one) : "r"(sat));
          sc[o][0] = kv4_scales(one, one, kv4_pick(0, 0));
        }
      }
#pragma unroll
      for (int i = 0; i < WORDS; ++i) {
        uint32_t q[2][NT][2];
        query(q[0], 2 * i);
        query(q[1], 2 * i + 1);
#pragma unroll
        for (int p = 0; p < 2; ++p) {
          uint32_t lo[4], hi[4];
          kv4_unpack(x[2 * p][i], lo);
          kv4_unpack(x[2 * p + 1][i], hi);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t f[4] = {kv4_mul(lo[2 * k], sc[2 * p][i / 2]), kv4_mul(hi[2 * k], sc[2 * p + 1][i / 2]),
                                   kv4_mul(lo[2 * k + 1], sc[2 * p][i / 2]), kv4_mul(hi[2 * k + 1], sc[2 * p + 1][i / 2])};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) kv8_mma(s[2 * h + p][nt], f, q[k][nt]);
          }
        }
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < KD; ++j) {
      uint32_t q[NT][2];
      query(q, j);
#pragma unroll
      for (int p = 0; p < K / 16; ++p) {
        uint32_t f[4];
        ptx::ldmatrix_x4(f, smem_clamp(st + p * 16 * (2 * D) + w.k_at[0] + ((uint32_t)(j << 5) ^ w.k_turn), 16, ring.lo, ring.hi,
                                       ring.status));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) win_mma<B>(s[p][nt], f, q[nt]);
      }
    }
  }
  // ---- y: the logits in log2 units, the scores by their row's factor, rounded here once: the weight of a row's largest is
  // 2^0 to 2^kKv8Slack then, however large the logits are.  (An exponent fma(score, factor, -m) would be what rounding the maximum left: from
  // 2^27 on more than f16's weights have room for.)
  // s[p][nt][i]: key 16p + 8 (i / 2) + r, row 2c + i % 2 of n-tile nt
  bool over = false;     // a score far above the running maximum
  float mx[NT][2];
  Two y[OCTETS][NT];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    Two qs;
    if constexpr (W::Q_SMEM) {
      float2 f;
      asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(f.x), "=f"(f.y) : "r"(w.q_at - lane * 8 + KD * NT * 256 + (nt * 8 + 2 * c) * 4));
      qs = two(f.x, f.y);
    } else {
      qs = two(w.qs[nt][0], w.qs[nt][1]);
    }
#pragma unroll
    for (int o = 0; o < OCTETS; ++o) y[o][nt] = mul2(two(s[o >> 1][nt][(o & 1) * 2], s[o >> 1][nt][(o & 1) * 2 + 1]), qs);
  }
  // rows beyond the last (padding of the n-tile) are taken for the newest token's
  auto behind = [&](int nt, int i) {
    const int row = (rg * NT + nt) * 8 + 2 * c + i;
    return a.causal ? max(a.T_q - 1 - row / a.G, 0) : 0;
  };
  if (masked) {
    const WinMask mask = win_mask(a, len, key0);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const int b0 = behind(nt, 0), b1 = behind(nt, 1);
#pragma unroll
      for (int o = 0; o < OCTETS; ++o) {
        const float2 f = split(y[o][nt]);
        y[o][nt] = two(mask.sees(8 * o + r, b0) ? f.x : -CUDART_INF_F, mask.sees(8 * o + r, b1) ? f.y : -CUDART_INF_F);
      }
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    float2 top = split(y[0][nt]);
#pragma unroll
    for (int o = 1; o < OCTETS; ++o) {
      const float2 f = split(y[o][nt]);
      top = make_float2(fmaxf(top.x, f.x), fmaxf(top.y, f.y));
    }
    mx[nt][0] = top.x;
    mx[nt][1] = top.y;
    over |= top.x - w.m[nt][0] > kKv8Slack || top.y - w.m[nt][1] > kKv8Slack;      // (m + slack would be rounded)
  }
  if (__any_sync(0xffffffffu, over)) {
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
      }
#pragma unroll
    for (int j = 0; j < KD; ++j)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) w.acc[j][nt][i] *= f[nt][i & 1];
  }
  // ---- weights, and P as the B operand
  uint32_t pf[K / 16][NT][2], pl[K / 16][NT][2];
  constexpr float kUp = (float)(1 << kWinLift<KV4, BF16>);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const Two off = two(w.m[nt][0] == -CUDART_INF_F ? 0.f : -w.m[nt][0], w.m[nt][1] == -CUDART_INF_F ? 0.f : -w.m[nt][1]);
    Two sum = two(w.l[nt][0], w.l[nt][1]);
#pragma unroll
    for (int o = 0; o < OCTETS; ++o) {
      const float2 x = split(add2(y[o][nt], off));
      const Two p = two(ptx::ex2(x.x), ptx::ex2(x.y));
      sum = add2(sum, p);
      const Two up = mul2(p, two(kUp, kUp));
      y[o][nt] = up;
      const float2 pv = split(up);
      const uint32_t h = Elem<B>::pack(pv.x, pv.y);
      pf[o >> 1][nt][o & 1] = kv8_transpose(h);
      if constexpr (FINE) {
        const float2 f = B ? make_float2(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u)) : half2_floats(h);
        pl[o >> 1][nt][o & 1] = kv8_transpose(Elem<B>::pack(pv.x - f.x, pv.y - f.y));
      }
    }
    const float2 f = split(sum);
    w.l[nt][0] = f.x;
    w.l[nt][1] = f.y;
  }
  if (infinite) {
    WinSlow<D, NT, K> t;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int o = 0; o < OCTETS; ++o) t.p[o][nt] = split(y[o][nt]);
      t.behind[nt][0] = behind(nt, 0);
      t.behind[nt][1] = behind(nt, 1);
#pragma unroll
      for (int j = 0; j < KD; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) t.acc[j][nt][i] = w.acc[j][nt][i];
    }
    t.mask = win_mask(a, len, key0);
    t.st = st;
    t.eb = eb;
    t.ring = ring;
    win_slow_values<D, NT, KV4, BF16, K>(t);
#pragma unroll
    for (int j = 0; j < KD; ++j)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) w.acc[j][nt][i] = t.acc[j][nt][i];
    return;
  }
  // ---- O^T += V^T P^T
  auto product = [&](int j, int p, const uint32_t (&f)[4]) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      win_mma<B>(w.acc[j][nt], f, pf[p][nt]);
      if constexpr (FINE) win_mma<B>(w.acc[j][nt], f, pl[p][nt]);
    }
  };
  if constexpr (KV4) {
    constexpr int CHUNKS = D / 32;
#pragma unroll
    for (int p = 0; p < K / 16; ++p) {
      uint32_t sc[2][CHUNKS];       // scales of keys 16p + 8h + 2c, + 1 for this lane's columns of chunk mt
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int o = 2 * (p & 1) + h;
        const uint32_t at = smem_clamp(st + w.k_scale[o] + w.v_scale + p / 2 * SUB, D / 8, ring.lo, ring.hi, ring.status);
        if constexpr (D == 128) {
          const uint4 v = win_lds4(at);
          sc[h][0] = kv4_scales(v.x, v.z, w.pick[0]);
          sc[h][1] = kv4_scales(v.x, v.z, w.pick[1]);
          sc[h][2] = kv4_scales(v.y, v.w, w.pick[0]);
          sc[h][3] = kv4_scales(v.y, v.w, w.pick[1]);
        } else {
          const uint2 v = win_lds2(at);
          sc[h][0] = kv4_scales(v.x, v.y, w.pick[0]);
          sc[h][1] = kv4_scales(v.x, v.y, w.pick[1]);
        }
      }
#pragma unroll
      for (int mt = 0; mt < CHUNKS; mt += 2) {
        uint32_t x[4];     // chunk mt of the first and second eight keys, chunk mt + 1
        ptx::ldmatrix_x4_trans(x, smem_clamp(st + w.v_at[p & 1] + ((uint32_t)(mt << 4) ^ w.v_turn) + p / 2 * SUB, 16, ring.lo, ring.hi, ring.status));
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          // a word: columns 4r .. 4r + 3 of key 2c in the lower half, of key 2c + 1 in the upper one
          const uint32_t k0 = __byte_perm(x[2 * h], x[2 * h + 1], 0x5410), k1 = __byte_perm(x[2 * h], x[2 * h + 1], 0x7632);
          uint32_t even[4], odd[4];    // columns 0 and 2 of the first eight keys, of the second; 1 and 3
          kv4_unpack(win_low_nibbles(k0, k1 << 4), even);
          kv4_unpack(win_low_nibbles(k0 >> 4, k1), odd);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const uint32_t f[4] = {kv4_mul(even[k], sc[0][mt + h]), kv4_mul(odd[k], sc[0][mt + h]),
                                   kv4_mul(even[2 + k], sc[1][mt + h]), kv4_mul(odd[2 + k], sc[1][mt + h])};
            product(2 * (mt + h) + k, p, f);
          }
        }
      }
    }
  } else {
#pragma unroll
    for (int p = 0; p < K / 16; ++p)
#pragma unroll
      for (int j = 0; j < KD; ++j) {
        uint32_t f[4];
        ptx::ldmatrix_x4_trans(f, smem_clamp(st + p * 16 * (2 * D) + w.v_at[0] + ((uint32_t)(j << 5) ^ w.v_turn), 16, ring.lo,
                                             ring.hi, ring.status));
        product(j, p, f);
      }
  }
}

// ---------------------------------------------------------------- the end of a piece
// l of the rows of this lane's accumulators, summed over the lanes that share them
__device__ __forceinline__ float win_sum(float l) {
  l += __shfl_xor_sync(0xffffffffu, l, 4);
  l += __shfl_xor_sync(0xffffffffu, l, 8);
  return l + __shfl_xor_sync(0xffffffffu, l, 16);
}

template <bool KV4, bool BF16>
__device__ __forceinline__ float win_unit() { return 1.f / (float)(1 << kWinLift<KV4, BF16>); }

// The whole unit's output, or the partial of slot >= 0.
template <int D, int NT, int RG, bool KV4, bool BF16>
__device__ __forceinline__ void win_end(WinWarp<D, NT, RG, KV4>& w, const WinParams& a, int b, int g, int64_t slot, int rg,
                                        int lane) {
  constexpr int KD = D / 16;
  const int r = lane >> 2, c = lane & 3;
  const float unit = win_unit<KV4, BF16>();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float l = win_sum(w.l[nt][i]);
      const int row = (rg * NT + nt) * 8 + 2 * c + i;
      if (row >= a.rows) continue;
      if (slot < 0) {
        const int t = row / a.G;
        const int64_t at = (((int64_t)b * a.T_q + t) * a.h_q + (int64_t)g * a.G + (row - t * a.G)) * D;
        if (!idx_ok(at + D - 1, (int64_t)a.N * a.T_q * a.h_q * D, a.status)) continue;
        const float f = (l > 0.f ? 1.f / l : l) * unit;      // (0, or NaN)
        __half* o = reinterpret_cast<__half*>(a.o);
#pragma unroll
        for (int j = 0; j < KD; ++j) {
          if constexpr (KV4) {
            Elem<BF16>::store2(o, at + win_column<true>(j, 0, r), w.acc[j][nt][i] * f, w.acc[j][nt][2 + i] * f);
          } else {
            Elem<BF16>::store(o, at + win_column<false>(j, 0, r), w.acc[j][nt][i] * f);
            Elem<BF16>::store(o, at + win_column<false>(j, 1, r), w.acc[j][nt][2 + i] * f);
          }
        }
      } else {
        const int64_t at = slot * a.rows + row;
        if (!idx_ok(at, 2 * (int64_t)a.workers * a.rows, a.status)) continue;
#pragma unroll
        for (int j = 0; j < KD; ++j)
#pragma unroll
          for (int half = 0; half < 2; ++half)
            a.ws_o[at * D + win_column<KV4>(j, half, r)] = w.acc[j][nt][2 * half + i] * unit;
        if (r == 0) {
          a.ws_m[at] = l == l ? w.m[nt][i] : 0.f;   // NaN scores move no maximum: not to be taken for an empty piece
          a.ws_l[at] = l;
        }
      }
    }
}

// Short kernel: the warps of a CTA leave their states in shared memory (their parts of the drained ring).
template <int D, int NT, int RG, bool KV4, bool BF16>
__device__ __forceinline__ void win_leave(WinWarp<D, NT, RG, KV4>& w, float2* ml, float* o, int lane) {
  constexpr int KD = D / 16;
  const int r = lane >> 2, c = lane & 3;
  const float unit = win_unit<KV4, BF16>();
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float l = win_sum(w.l[nt][i]);
      const int row = nt * 8 + 2 * c + i;
      if (r == 0) ml[row] = make_float2(w.m[nt][i], l);
#pragma unroll
      for (int j = 0; j < KD; ++j)
#pragma unroll
        for (int half = 0; half < 2; ++half) o[row * D + win_column<KV4>(j, half, r)] = w.acc[j][nt][2 * half + i] * unit;
    }
}

// One row's four columns of n <= MOST states, folded in the order of the keys: state i has its m and l at ml(i), its O at o(i).
template <int MOST, typename ML, typename O>
__device__ __forceinline__ void win_fold(int n, ML ml, O o, float& m, float& l, float4& acc) {
  if constexpr (MOST <= 8) {
    kv8_fold(n, ml, o, m, l, acc);
  } else {
    m = -CUDART_INF_F;
    l = 0.f;
    acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i = 0; i < n; i += 8) {
      float mi, li;
      float4 v;
      kv8_fold(n - i, [&](int k) { return ml(i + k); }, [&](int k) { return o(i + k); }, mi, li, v);
      const float top = fmaxf(m, mi), base = top == -CUDART_INF_F ? 0.f : top;
      const float f = ptx::ex2(m - base), g = ptx::ex2(mi - base);
      m = top;
      l = l * f + li * g;
      acc = make_float4(acc.x * f + v.x * g, acc.y * f + v.y * g, acc.z * f + v.z * g, acc.w * f + v.w * g);
    }
  }
}

// ---------------------------------------------------------------- kernels
template <int D, int NT, int RG, bool KV4, bool BF16>
__global__ void __launch_bounds__(WinCfg<D, NT, RG, KV4>::THREADS, 1)
gqa_win_kernel(const WinParams a) {
  using C = WinCfg<D, NT, RG, KV4>;
  constexpr int STAGES = C::STAGES;
  constexpr bool FINE = !(KV4 && BF16);
  extern __shared__ __align__(128) uint8_t smem[];
  int64_t* prefix = reinterpret_cast<int64_t*>(smem + C::PREFIX_OFF);
  int* lens = reinterpret_cast<int*>(smem + C::LENS_OFF);
  volatile int* abort = reinterpret_cast<volatile int*>(smem + C::FLAG_OFF);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / RG, rg = warp % RG;
  const uint32_t full = ptx::smem_u32(smem + C::BAR_OFF) + grp * STAGES * 16, empty = full + STAGES * 8;
  if (threadIdx.x < C::GROUPS * STAGES) {
    const uint32_t f = ptx::smem_u32(smem + C::BAR_OFF) + threadIdx.x / STAGES * STAGES * 16 + threadIdx.x % STAGES * 8;
    ptx::mbar_init(f, C::FULL);
    ptx::mbar_init(f + STAGES * 8, RG);
  }
  if (threadIdx.x == 0) *abort = 0;
  ptx::fence_mbar_init();
  ptx::grid_dependency_wait();
  win_prefix<C::KEYS, C::THREADS>(a, prefix, lens, reinterpret_cast<int64_t*>(smem + C::SUMS_OFF));
  if (threadIdx.x == 0) ptx::grid_launch_dependents();
  win_empty_rows<D, C::THREADS>(a, lens);

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
    // as in the kernel of the 8-bit cache: this range begins inside a unit, and it is the first that does
    const bool first_cut = at.t > 0 && at.t <= share;
    const int64_t pieces = first_cut ? 1 + (at.tiles - at.t + share - 1) / share : 0;
    const int first = 2 * ((int)wk - 1) + (at.t < share ? 1 : 0);
    if (!a.sliced) a.splits[wk] = make_int4((int)pieces, first, at.b, at.g);
    else if (first_cut) a.splits[at.b * a.h_kv + at.g] = make_int4((int)pieces, first, at.b, at.g);
  }
  const uint32_t ring0 = ptx::smem_u32(smem + C::RING_OFF) + grp * STAGES * C::TILE;
  const Win ring = {ring0, ring0 + STAGES * C::TILE, a.status};
  const uint64_t policy = KV4 ? ptx::policy_evict_first() : 0;       // (of bulk copies)
  const int eb = min(a.block_size, 32);
  uint2 raw[NT][D / 16];
  win_load_q<D, NT, RG, KV4>(raw, a, at.b, at.g, rg, lane);
  WinStream str;
  int issued = 0;
  if (rg == 0) {
    str.at = at;
    win_stream_setup<D, KV4, C::KEYS>(str, a, lane);
    str.id = win_ids<C::KEYS>(a, at, lens[at.b], str.want, lane);
    win_enter<D, C::KEYS>(str, a, prefix, lens, lane);
    for (; issued < n && issued < STAGES; ++issued)
      if (!(issued == 1 && wk == a.stall))
        win_copy<D, KV4, C::KEYS>(str, a, prefix, lens, ring0 + issued * C::TILE, full + issued * 8, policy, lane, ring);
  }
  WinWarp<D, NT, RG, KV4> w;
  win_setup(w, a, ptx::smem_u32(smem + C::Q_OFF) + warp * C::QUERIES, lane);
  int len = lens[at.b], skip = win_span<C::KEYS>(a, len).skip;
  WinClear clear = win_clear_tiles<C::KEYS>(a, len, skip);
  win_begin<D, NT, RG, KV4, BF16>(w, raw, a, lane);
  bool fresh = at.t == 0;        // this piece begins with its unit
  int64_t slot = 2 * wk;         // where it goes when it is not the whole unit
  int i = 0, stage = 0, phase = 0;
  for (; i < n; ++i) {
    if (!kv8_wait(full + stage * 8, phase, a.timeout_ns, abort)) break;
    win_tile<D, NT, RG, KV4, BF16, FINE>(w, a, ring0 + stage * C::TILE, eb, len, win_tile_of(a, skip, at.t) * C::KEYS,
                                         !clear.has(at.t), rg, lane, ring);
    __syncwarp();
    if (RG > 1 && lane == 0) ptx::mbar_arrive(empty + stage * 8);
    if (rg == 0 && i + STAGES < n) {
      if (RG > 1 && !kv8_wait(empty + stage * 8, phase, a.timeout_ns, abort)) {
        ++i;
        break;
      }
      if (!(STAGES == 1 && i == 0 && wk == a.stall))
        win_copy<D, KV4, C::KEYS>(str, a, prefix, lens, ring0 + stage * C::TILE, full + stage * 8, policy, lane, ring);
      ++issued;
    }
    if (++stage == STAGES) {
      stage = 0;
      phase ^= 1;
    }
    if (++at.t == at.tiles || i + 1 == n) {
      const bool whole = fresh && at.t == at.tiles;
      if (whole && a.sliced && lane == 0 && rg == 0) a.splits[at.b * a.h_kv + at.g] = make_int4(0, 0, 0, 0);
      win_end<D, NT, RG, KV4, BF16>(w, a, at.b, at.g, whole ? -1 : slot, rg, lane);
      if (i + 1 < n) {
        kv8_next_unit(at, prefix, a.N, a.h_kv);
        len = lens[at.b];
        skip = win_span<C::KEYS>(a, len).skip;
        clear = win_clear_tiles<C::KEYS>(a, len, skip);
        win_load_q<D, NT, RG, KV4>(raw, a, at.b, at.g, rg, lane);
        win_begin<D, NT, RG, KV4, BF16>(w, raw, a, lane);
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

// Few, short units in one launch, as the short kernel of the 8-bit cache: a cluster of a.ctas CTAs for each (sequence,
// head), its tiles cut evenly over their workers (at most kKv8Short each, so that one window of block ids serves a
// worker), the states folded in shared memory and then through distributed shared memory, in the order of the keys.
template <int D, int NT, int RG, bool KV4, bool BF16>
__global__ void __launch_bounds__(WinCfg<D, NT, RG, KV4>::THREADS, 1)
gqa_win_short_kernel(const WinParams a) {
  using C = WinCfg<D, NT, RG, KV4>;
  constexpr int STAGES = C::STAGES;
  constexpr bool FINE = !(KV4 && BF16);
  extern __shared__ __align__(128) uint8_t smem[];
  volatile int* flags = reinterpret_cast<volatile int*>(smem + C::FLAG_OFF);   // [0] abort
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int grp = warp / RG, rg = warp % RG;
  const int unit = blockIdx.x / a.ctas, c = blockIdx.x - unit * a.ctas, b = unit / a.h_kv, g = unit - b * a.h_kv;
  const uint32_t full = ptx::smem_u32(smem + C::BAR_OFF) + grp * STAGES * 16, empty = full + STAGES * 8;
  if (threadIdx.x < C::GROUPS * STAGES) {
    const uint32_t f = ptx::smem_u32(smem + C::BAR_OFF) + threadIdx.x / STAGES * STAGES * 16 + threadIdx.x % STAGES * 8;
    ptx::mbar_init(f, C::FULL);
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
  const WinSpan span = win_span<C::KEYS>(a, len);
  const int tiles = span.tiles;
  // the tiles go evenly to the CTAs, and a CTA's in runs of `per` to its workers
  const int share = max((tiles + a.ctas - 1) / a.ctas, 1), per = (share + C::GROUPS - 1) / C::GROUPS;
  const int busy_ctas = (tiles + share - 1) / share;
  const int mine = max(min(tiles - c * share, share), 0);
  const int busy = (mine + per - 1) / per;       // workers of this CTA that have tiles
  const int t0 = c * share + grp * per, n = grp < busy ? min(per, mine - grp * per) : 0;
  const uint32_t ring0 = ptx::smem_u32(smem + C::RING_OFF) + grp * STAGES * C::TILE;
  const Win ring = {ring0, ring0 + STAGES * C::TILE, a.status};
  const uint64_t policy = KV4 ? ptx::policy_evict_first() : 0;       // (of bulk copies)
  const int eb = min(a.block_size, 32);
  const bool stalled = a.stall >= 0 && a.stall == (int)blockIdx.x * C::GROUPS + grp;
  float2* ml = reinterpret_cast<float2*>(smem + C::ML_OFF);
  bool good = true;
  if (n > 0) {
    WinStream str;
    int issued = 0;
    if (rg == 0) {
      str.at = {b, g, t0, tiles};
      str.len = len;
      str.skip = span.skip;
      str.first = span.first;
      win_stream_setup<D, KV4, C::KEYS>(str, a, lane);
      str.id = win_ids<C::KEYS>(a, str.at, len, str.want, lane);
    }
    uint2 raw[NT][D / 16];
    win_load_q<D, NT, RG, KV4>(raw, a, b, g, rg, lane);
    if (rg == 0) {
      win_ids_check<D>(str, a);
      str.t_end = t0 + n;
      for (; issued < n && issued < STAGES; ++issued)
        if (!(stalled && issued == 1))
          win_issue<D, KV4, C::KEYS>(str, a, ring0 + issued * C::TILE, full + issued * 8, policy, lane, ring);
    }
    WinWarp<D, NT, RG, KV4> w;
    win_setup(w, a, ptx::smem_u32(smem + C::Q_OFF) + warp * C::QUERIES, lane);
    win_begin<D, NT, RG, KV4, BF16>(w, raw, a, lane);
    const WinClear clear = win_clear_tiles<C::KEYS>(a, len, span.skip);
    int i = 0, stage = 0, phase = 0;
    for (; i < n; ++i) {
      good = kv8_wait(full + stage * 8, phase, a.timeout_ns, flags);
      if (!good) break;
      win_tile<D, NT, RG, KV4, BF16, FINE>(w, a, ring0 + stage * C::TILE, eb, len, win_tile_of(a, span.skip, t0 + i) * C::KEYS,
                                           !clear.has(t0 + i), rg, lane, ring);
      __syncwarp();
      if (RG > 1 && lane == 0) ptx::mbar_arrive(empty + stage * 8);
      if (rg == 0 && i + STAGES < n) {
        if (RG > 1) {
          good = kv8_wait(empty + stage * 8, phase, a.timeout_ns, flags);
          if (!good) break;
        }
        if (!(STAGES == 1 && i == 0 && stalled))
          win_issue<D, KV4, C::KEYS>(str, a, ring0 + stage * C::TILE, full + stage * 8, policy, lane, ring);
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
    if (good)
      win_leave<D, NT, RG, KV4, BF16>(w, ml + warp * 8 * NT, reinterpret_cast<float*>(smem + C::RING_OFF + warp * C::AREA), lane);
  }
  __syncthreads();
  // ---- the CTA's state: m and l where the general kernel has its prefix sums, O in the first worker's areas (an item is
  // read and written by one thread); the output itself when this CTA has the whole unit
  float2* cta_ml = reinterpret_cast<float2*>(smem + C::PREFIX_OFF);
  uint8_t* areas = smem + C::RING_OFF;
  const bool alone = a.ctas == 1 || tiles == 0;
  if (flags[0] == 0)
    for (int i = threadIdx.x; i < a.rows * (D / 4); i += C::THREADS) {
      const int row = i / (D / 4), d = i % (D / 4) * 4, part = row / (8 * NT), wrow = row % (8 * NT);
      float m, l;
      float4 v;
      win_fold<C::FOLD>(busy, [&](int k) { return ml[(k * RG + part) * 8 * NT + wrow]; },
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
    for (int i = c * C::THREADS + threadIdx.x; i < a.rows * (D / 4); i += a.ctas * C::THREADS) {
      const int row = i / (D / 4), d = i % (D / 4) * 4, part = row / (8 * NT), wrow = row % (8 * NT);
      float m, l;
      float4 v;
      win_fold<8>(busy_ctas, [&](int k) { return ld_cluster_v2(ptx::mapa(ml_at + row * 8, k)); },
               [&](int k) { return ld_cluster_v4(ptx::mapa(o_at + part * C::AREA + (wrow * D + d) * 4, k)); }, m, l, v);
      kv8_store4<BF16>(a, b, g, row, d, D, l, v);
    }
  }
  ptx::cluster_sync();       // no CTA leaves while another reads its shared memory
}

// ---------------------------------------------------------------- launches, one translation unit for each cache, d_head and type (gqa_win_inst.cuh)
// Kernel shapes as those of the 8-bit cache: up to 8, 16, 24 or 32 query rows for one warp, 48 or 64 for two.
template <int D, bool KV4, bool BF16>
cudaError_t win_prepare(int cls);
template <int D, bool KV4, bool BF16>
cudaError_t win_launch(const WinParams& p, int cls, unsigned grid, cudaStream_t st);

// The n-tiles of a warp and the warps of a ring for a class of query rows (8, 16, 24, 32, 48, 64).  32 rows over the 4-bit
// cache: two warps of 16 rows and tiles of 64 keys (131071 keys 88 us instead of 95; four such warps for 64 rows 227 us instead
// of 221).
template <bool KV4>
constexpr int win_rows_nt(int cls) {
  return cls < 2 ? cls + 1 : (cls == 2 || cls == 4 ? 3 : (KV4 && cls == 3 ? 2 : 4));
}
template <bool KV4>
constexpr int win_rows_rg(int cls) {
  return cls < 3 ? 1 : (cls == 3 && !KV4 ? 1 : 2);
}

// keys of a tile and workers of a CTA for a class of query rows
template <bool KV4>
constexpr int win_tile_keys(int cls) { return win_rows_nt<KV4>(cls) <= 2 ? win_keys<KV4, 2> : win_keys<KV4, 3>; }
template <bool KV4, int D>
constexpr int win_workers(int cls) {
  const int nt = win_rows_nt<KV4>(cls);
  return (nt == 1 ? WinCfg<D, 1, 1, KV4>::WARPS : (nt == 2 ? WinCfg<D, 2, 1, KV4>::WARPS : WinCfg<D, 3, 1, KV4>::WARPS)) /
         win_rows_rg<KV4>(cls);
}

}  // namespace gqa
