// Attention of a chunk's rows over a paged cache on tcgen05, and the attention weight that each
// cached token gathers.
//
// Rows of one KV head's group of G query heads are packed into tiles of 128: row r of a tile is
// token r / G, head r % G (128 / G whole tokens, loaded by one TMA box of G heads), so K and V are
// read once for the group. A unit of work is 256 rows (two tiles) of one stream and KV head; where a
// stream brings no more than 128 rows the two softmax warpgroups instead take every second key
// tile of the one query tile and merge at the end.
//
// Lengths differ and are known on the device only, and 148 SMs take 264 equal units in two waves of which
// the second is three quarters full. So one thread block per SM stays, and the blocks share the batch's
// key tiles evenly: a small kernel (paged_plan_kernel) lists the units, counts their tiles and says how
// they are shared (PagedWork), and units that are shared leave partial rows that paged_join_kernel adds up.
// Lengths that differ are shared in a row, tile by tile. Units of nearly one size are shared in
// step: then all blocks of a head read the same keys at the same time, from L2. (In a row, 24 heads of
// 18480 tokens read their K and V from HBM eleven times over: 760 us, against 672 us for one thread
// block per unit, although an eighth less of the machine idles.)
//
// Attention, structure of one block (as the rolling-window kernel's, rkv_attention.cu):
//   warps 0-3, 4-7  softmax of query tile 0 / 1 (or of the even / odd key tiles)
//   warp 8          TMA producer: queries once, K and V tiles of 128 tokens into two stages each, one
//                   box per page and 64-column half, a lane per box
//   warp 9          TMEM allocator and tcgen05.mma issuer (one thread)
// TMEM: S0 | S1 | O0 | O1, 128 fp32 columns each; P (bf16) overwrites its S.
//
// What is masked: keys a row does not see become -infinity before the softmax, whatever stale
// bytes the tile holds there; V rows past the last visible token are left out of the product in
// steps of 16 tokens, and zeroed within the last step, since 0 times a stale NaN would be NaN.
// Every wait is bounded; on expiry the block reports, drains what it issued and returns.
//
// A wait names its phase by parity, so no barrier may complete a phase more than one ahead of any warp that waits
// at it, however long that warp is held up. Nearly always the next phase needs something of every such warp; the
// two waits that see to it elsewhere say so (tests/test_chunk_barriers.py models the protocol).
#include <algorithm>
#include <mutex>

#include "attention_tile.cuh"
#include "paged.cuh"
#include "ptx_warp.cuh"

namespace rkv {
namespace {

constexpr int kBM = 128;  // rows per query tile
constexpr int kBN = 128;  // tokens per key tile
constexpr int kThreads = 320;
constexpr int kSmemQ = 0;
constexpr int kSmemK = 2 * kTile;
constexpr int kSmemV = 4 * kTile;
constexpr int kSmemChain = 6 * kTile;
constexpr int kSmemBar = kSmemChain + 2 * 128 * 16;
constexpr int kSmemBytes = kSmemBar + 256 + 1024;
constexpr unsigned long long kDrainNs = 2000000000ull;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoKey = -1e30f;        // reference (log2) of a row that has seen no key
constexpr float kLazyRescale = 8.0f;    // exact path: the reference follows a maximum past 2^8
constexpr float kLazySum = 256.0f;      // one-pass path: the reference follows a tile sum past 2^8
constexpr float kSumSlack = 18446744073709551616.0f;  // 2^64: largest accepted one-pass tile sum

enum : int {
  kBarQ = 0,
  kBarKFull = 1,   // +stage
  kBarKEmpty = 3,  // +stage
  kBarVFull = 5,   // +stage
  kBarVEmpty = 7,  // +stage
  kBarSFull = 9,   // +softmax warpgroup
  kBarPFull = 11,  // +softmax warpgroup
  kBarODone = 13,
  kBarDrain = 14,
  kBarVFix = 15,   // a unit's last tile's stale V rows were zeroed
  kBarQEmpty = 16,  // every score product of a unit completed: its query buffer is free
  kNumBars = 17
};

__device__ __forceinline__ constexpr uint32_t col_s(int t) { return static_cast<uint32_t>(t) * 128u; }
__device__ __forceinline__ constexpr uint32_t col_o(int t) { return 256u + static_cast<uint32_t>(t) * 128u; }
constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(kBM, kBN, false);
constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kBM, kHeadDim, true);

// ---------------------------------------------------------------- the plan
constexpr int kPlanNear = 1024;  // streams, and blocks of rows, that the plan holds in shared memory

// Exclusive sum over the thread block, and its total.
template <int kPlanThreads>
__device__ __forceinline__ int plan_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[wp] = inc;
  __syncthreads();
  const int v = lane < kPlanThreads / 32 ? warp_sums[lane] : 0;
  total = __reduce_add_sync(0xffffffffu, v);
  return inc - x + __reduce_add_sync(0xffffffffu, lane < wp ? v : 0);
}

// The last of n rising values that is at most y: in shared memory if they fit there, else in `far`.
__device__ __forceinline__ int last_at_most(const int* near, const int* far, int stride, int n, int y) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    const int v = n <= kPlanNear ? near[m] : far[static_cast<long long>(m) * stride];
    if (v <= y) lo = m; else hi = m;
  }
  return lo;
}

// One thread block: the units of the batch and their key tiles, from the lengths on the device, and how
// they are shared. 256 threads, unless there are more streams or blocks: its time is that of some ten barriers, and the
// more warps the longer each takes (5 units of one tile: 16.1 us with 1024, 15.3 with 256).
template <int kPlanThreads>
__global__ void __launch_bounds__(kPlanThreads) paged_plan_kernel(const __grid_constant__ PagedAttnParams p) {
  constexpr int kPlanWarps = kPlanThreads / 32;
  __shared__ int warp_sums[kPlanWarps];
  __shared__ int sizes[2][kPlanWarps];
  __shared__ int near_seq[kPlanNear];    // first block of every stream, if there are that few
  __shared__ int near_start[kPlanNear];  // first tile of every block, if there are that few
  __shared__ int2 near_rows[kPlanNear];  // its first row and tokens
  __shared__ int near_rest[kSmCount + 2];
  ptx::let_next_launch();
  ptx::wait_previous();
  const PagedView& w = p.view;
  const int t = threadIdx.x;
  int blocks = 0;
  bool falls = false;
  for (int base = 0; base < w.n_seqs; base += kPlanThreads) {
    const int s = base + t;
    int c = 0;
    if (s < w.n_seqs) {
      const PagedSeq q = paged_seq(w, s);
      falls |= q.falls;
      if (q.ok)
        c = (q.n_q + p.block_tokens - 1) / p.block_tokens;
      else
        paged_report(w, kStatusLength);
    }
    int total;
    const int first = blocks + plan_scan<kPlanThreads>(c, warp_sums, total);
    if (s < w.n_seqs) p.seq_first[s] = first;
    if (s < kPlanNear) near_seq[s] = first;
    blocks += total;
  }
  // row ranges that overlap (q_start decreases: reported above) may need more blocks than the list holds, or than
  // 31 bits count: then there is no work
  if (__syncthreads_or(falls)) blocks = 0;
  // for the weights: the streams with the longest chunks first, so that the last key tiles drawn are short work
  if (p.order != nullptr) {
    auto length = [&](int s) { return (s + 1 < w.n_seqs ? near_seq[s + 1] : blocks) - near_seq[s]; };
    for (int i = t; i < w.n_seqs; i += kPlanThreads) {
      const int mine = length(i);
      int rank = 0;
      for (int s = 0; s < w.n_seqs; ++s) {
        const int x = length(s);
        rank += x > mine || (x == mine && s < i);
      }
      p.order[rank] = i;
    }
  }
  int tiles = 0, most = 0, least = 1 << 30;
  for (int base = 0; base < blocks; base += kPlanThreads) {
    const int b = base + t;
    PagedBlock k = {};
    if (b < blocks) {
      const int s = last_at_most(near_seq, p.seq_first, 1, w.n_seqs, b);
      const PagedSeq q = paged_seq(w, s);
      const int i0 = (b - (w.n_seqs <= kPlanNear ? near_seq[s] : p.seq_first[s])) * p.block_tokens;
      k.row0 = q.q0 + i0;
      k.cnt = min(p.block_tokens, q.n_q - i0);
      k.keys = p.causal ? max(0, q.kv - q.n_q + i0 + k.cnt) : q.kv;
      k.place0 = q.kv - q.n_q + i0;
      k.seq = s;
      k.tiles = max(1, (k.keys + kBN - 1) / kBN);
      most = max(most, k.tiles);
      least = min(least, k.tiles);
    }
    int total;
    k.start = tiles + plan_scan<kPlanThreads>(k.tiles, warp_sums, total);
    if (b < blocks) p.blocks[b] = k;
    if (b < blocks && b < kPlanNear) {
      near_start[b] = k.start;
      near_rows[b] = make_int2(k.row0, k.cnt);
    }
    tiles += total;
  }
  // the whole thread block's largest and smallest
  most = __reduce_max_sync(0xffffffffu, most);
  least = __reduce_min_sync(0xffffffffu, least);
  if ((t & 31) == 0) {
    sizes[0][t >> 5] = most;
    sizes[1][t >> 5] = least;
  }
  __syncthreads();
  most = __reduce_max_sync(0xffffffffu, sizes[0][t % kPlanWarps]);
  least = __reduce_min_sync(0xffffffffu, sizes[1][t % kPlanWarps]);
  auto tiles_of = [&](int b) {
    return blocks <= kPlanNear ? (b + 1 < blocks ? near_start[b + 1] : tiles) - near_start[b] : p.blocks[b].tiles;
  };
  auto start_of = [&](int b) { return blocks <= kPlanNear ? near_start[b] : p.blocks[b].start; };

  const long long units = static_cast<long long>(blocks) * w.kv_heads;
  const long long all = static_cast<long long>(tiles) * w.kv_heads;
  PagedWork* out = p.work;
  const int waves = static_cast<int>(units / kSmCount), n_tail = static_cast<int>(units - static_cast<long long>(waves) * kSmCount);
  const long long first = static_cast<long long>(waves) * kSmCount;  // the first of the last units
  int n = 0;  // thread i < n_tail: tiles of the i-th of them
  if (t < n_tail) n = tiles_of(static_cast<int>(first + t - quotient(first + t, blocks) * blocks));
  int tail_tiles;
  plan_scan<kPlanThreads>(n, warp_sums, tail_tiles);
  const int quota = (tail_tiles + kSmCount - 1) / kSmCount;
  // in step: sizes within an eighth of each other
  const bool in_step = blocks > 0 && least >= most - most / 8;
  int rest_tiles;
  const int rest = plan_scan<kPlanThreads>(max(0, n - quota), warp_sums, rest_tiles);
  if (t <= n_tail) out->rest[t] = near_rest[t] = rest;
  if (t == 0) *p.ticket = 0;
  // in a row: shares down to one tile, since idle SMs cost more than the merge (6 units of 8 to 11 tiles: 16 us; 25
  // with four tiles at least)
  PagedShares row;
  row.split(all, kSmCount);
  const int n_ctas = in_step ? kSmCount : row.n;
  if (t == 0) {
    out->n_blocks = blocks;
    out->n_ctas = n_ctas;
    out->in_step = in_step;
    out->waves = waves;
    out->n_tail = n_tail;
    out->quota = quota;
  }
  __syncthreads();
  if (t >= kSmCount) return;
  PagedShare mine = {};
  PagedJoin join = {};
  int joined = 0;  // its block
  if (in_step) {
    const int helpers = kSmCount - n_tail;
    if (t < n_tail) {
      mine.left = quota;
      const int r0 = near_rest[t], r1 = near_rest[t + 1];
      if (r1 > r0) {
        const int j0 = min(helpers - 1, r0 / quota), j1 = min(helpers - 1, (r1 - 1) / quota);
        join.h = static_cast<int>(quotient(first + t, blocks));
        joined = static_cast<int>(first + t - static_cast<long long>(join.h) * blocks);
        join.slot0 = 2 * t + j0;
        join.step = 1;
        join.parts = j1 - j0 + 2;
      }
    } else {
      mine.pos = min(rest_tiles, (t - n_tail) * quota);
      mine.left = (t == kSmCount - 1 ? rest_tiles : min(rest_tiles, mine.pos + quota)) - mine.pos;
      int hi = n_tail;  // the last unit whose leftover begins at or before pos
      while (hi - mine.i > 1) {
        const int m = (mine.i + hi) >> 1;
        if (near_rest[m] <= mine.pos) mine.i = m; else hi = m;
      }
    }
  } else if (t < n_ctas) {
    const long long x = row.start(t);
    mine.left = row.start(t + 1) - x;
    mine.h = static_cast<int>(quotient(x, tiles));
    const int y = static_cast<int>(x - static_cast<long long>(mine.h) * tiles);
    mine.b = last_at_most(near_start, &p.blocks[0].start, sizeof(PagedBlock) / 4, blocks, y);
    mine.t = y - start_of(mine.b);
    // the unit that this share's start cuts, if it is the first border inside it
    const long long begin = x - mine.t;
    if (mine.t > 0 && row.start(t - 1) <= begin) {
      joined = mine.b;
      join.h = mine.h;
      join.slot0 = 2 * t - 1;
      join.step = 2;
      join.parts = row.owner(begin + tiles_of(mine.b) - 1) - t + 2;
    }
  }
  if (join.parts > 0) {
    join.row0 = blocks <= kPlanNear ? near_rows[joined].x : p.blocks[joined].row0;
    join.cnt = blocks <= kPlanNear ? near_rows[joined].y : p.blocks[joined].cnt;
  }
  out->share[t] = mine;
  p.joins[t] = join;
}

// In step: the thread block (of those past n_tail, counted from 0) that takes leftover tile y.
__device__ __forceinline__ int helper_of(const PagedWork& r, int y) {
  return min(kSmCount - r.n_tail - 1, y / r.quota);
}

// A unit, or the part of one, that a thread block works on.
struct PagedUnit {
  PagedBlock k;
  int h;
  int t0, t1;  // its key tiles
  int slot;    // of a part: where its rows go
  bool two;    // two query tiles
  int j0, n_tiles, last_valid;  // first key, tiles, visible keys of the last tile
};

// The units of one thread block's share, in order; every role of the block walks them by itself.
struct PagedWalk {
  const PagedBlock* blocks;
  const PagedWork* work;
  int n_blocks, tpt, cta;
  bool in_step;
  int wave;        // in step: whole units taken
  long long left;  // tiles of the share still to take (in step: of the last units)
  int h, b, t;     // the next unit's head, block and first tile
  int i, pos;      // in step, of a helper: the last unit it is at, and the next leftover tile

  __device__ __forceinline__ void take(PagedUnit& u, long long most) {
    const int4* src = reinterpret_cast<const int4*>(blocks + b);
    const int4 x = src[0], y = src[1];
    u.k.row0 = x.x;
    u.k.cnt = x.y;
    u.k.keys = x.z;
    u.k.place0 = x.w;
    u.k.seq = y.x;
    u.k.start = y.y;
    u.k.tiles = y.z;
    u.h = h;
    u.t0 = t;
    u.t1 = static_cast<int>(min(static_cast<long long>(u.k.tiles), t + most));
    u.two = u.k.cnt > tpt;
    u.j0 = t * kBN;
    u.n_tiles = u.t1 - t;
    u.last_valid = min(kBN, u.k.keys - (u.t1 - 1) * kBN);
  }
  __device__ __forceinline__ void at_unit(long long n) {
    h = static_cast<int>(quotient(n, n_blocks));
    b = static_cast<int>(n - static_cast<long long>(h) * n_blocks);
  }
  __device__ __forceinline__ bool next(PagedUnit& u) {
    if (!in_step) {
      if (left <= 0) return false;
      take(u, left);
      // this thread block's first slot if the unit began before its share, else its second
      u.slot = 2 * cta + (t == 0 ? 1 : 0);
      left -= u.n_tiles;
      t = 0;
      if (++b == n_blocks) {
        b = 0;
        ++h;
      }
      return true;
    }
    t = 0;
    if (wave < work->waves) {
      at_unit(cta + static_cast<long long>(wave) * kSmCount);
      take(u, 1 << 30);
      ++wave;
      return true;
    }
    const long long first = static_cast<long long>(work->waves) * kSmCount;
    const int n_tail = work->n_tail;
    if (cta < n_tail) {
      if (left <= 0) return false;
      left = 0;
      at_unit(first + cta);
      take(u, work->quota);
      u.slot = 2 * cta + helper_of(*work, work->rest[cta]);
      return true;
    }
    // a helper: leftover tiles [pos, pos + left) in a row
    while (left > 0) {
      const int begin = work->rest[i], end = work->rest[i + 1];
      if (pos >= end) {
        ++i;
        continue;
      }
      at_unit(first + i);
      t = work->quota + pos - begin;
      take(u, left);
      u.slot = 2 * i + cta - n_tail + 1;
      pos += u.n_tiles;
      left -= u.n_tiles;
      return true;
    }
    return false;
  }
};

// 64 numerators 2^(s sl2 - m) of one row, packed to bf16 pairs (the operand type of the product
// with V; half a step, 2^-8, of each), their unrounded sum in acc. All on the special-function unit: a
// polynomial for two pairs in eight, as in the rolling-window kernel, made the kernel 3 % slower (1046 us
// against 1010 us, 2048 rows of 32 heads, the last of 32768 tokens), its own degree 4 instead of 3 (a row sum
// has to hold fp32) costing more issue slots than the unit gains.
__device__ __forceinline__ void numerators(const uint32_t* sh, uint64_t c2, uint64_t nm2, uint32_t* pk,
                                           uint64_t (&acc)[4]) {
#pragma unroll
  for (int k = 0; k < kBN / 4; ++k) {
    const uint64_t x = ptx::f2_fma(ptx::f2_pack(__uint_as_float(sh[2 * k]), __uint_as_float(sh[2 * k + 1])), c2, nm2);
    float a, b;
    ptx::f2_unpack(x, a, b);
    a = ptx::ex2(a);
    b = ptx::ex2(b);
    acc[k & 3] = ptx::f2_add(acc[k & 3], ptx::f2_pack(a, b));
    pk[k] = pack_bf16x2(a, b);
  }
}

__device__ __forceinline__ float sum_of(const uint64_t (&acc)[4]) {
  float rs[4];
  ptx::f2_unpack(ptx::f2_add(acc[0], acc[1]), rs[0], rs[1]);
  ptx::f2_unpack(ptx::f2_add(acc[2], acc[3]), rs[2], rs[3]);
  return (rs[0] + rs[1]) + (rs[2] + rs[3]);
}

// One key tile of this thread's row, `valid` of its keys visible (any number; 128 and above: all).
// m_used: the reference (log2) of the numerators; l: their sum in its scale; pend: a change of
// reference decided on this tile, applied to O and l at the next. After the first tile the numerators are
// formed in one pass against the running reference; the tile's sum bounds its largest one, so a
// sum past 2^8 moves the reference, and a sum past 2^64 (or NaN) takes the exact path, which
// finds the row's maximum first.
__device__ __forceinline__ void softmax_tile(bool first, int valid, uint32_t tS, uint32_t tO, float sl2, uint64_t c2,
                                             float& m_used, float& l, float& pend) {
  if (__any_sync(0xffffffffu, pend != 1.0f)) scale_o(tO, pend);
  l *= pend;
  pend = 1.0f;
  const bool whole = __all_sync(0xffffffffu, valid >= kBN);
  bool stored = false;
  if (!first) {
    const uint64_t nm2 = ptx::f2_pack(-m_used, -m_used);
    uint64_t acc[4] = {0, 0, 0, 0};
    uint32_t pk[kBN / 2];
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {
      uint32_t sh[kBN / 2];
      ptx::tmem_ld64(tS + 64 * hh, sh);
      if (whole) {
        numerators(sh, c2, nm2, pk + 32 * hh, acc);
      } else {
#pragma unroll
        for (int i = 0; i < kBN / 2; ++i)
          if (64 * hh + i >= valid) sh[i] = 0xff800000u;
        numerators(sh, c2, nm2, pk + 32 * hh, acc);
      }
    }
    const float lt = sum_of(acc);
    if (!__any_sync(0xffffffffu, !(lt <= kSumSlack))) {
      l += lt;
      if (lt > kLazySum) {
        const float up = lg2_approx(lt);
        pend = ptx::ex2(-up);
        m_used += up;
      }
      ptx::tmem_st64(tS, pk);
      stored = true;
    }
  }
  if (!stored) {
    float m_tile;
    {
      uint32_t sr[kBN];
      ptx::tmem_ld128(tS, sr);
      if (!whole) {
#pragma unroll
        for (int i = 0; i < kBN; ++i)
          if (i >= valid) sr[i] = 0xff800000u;
      }
      float mq[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const uint32_t* t = sr + 32 * c;
        float m = ptx::fmax3(__uint_as_float(t[0]), __uint_as_float(t[1]), __uint_as_float(t[2]));
#pragma unroll
        for (int i = 3; i < 31; i += 2) m = ptx::fmax3(m, __uint_as_float(t[i]), __uint_as_float(t[i + 1]));
        mq[c] = fmaxf(m, __uint_as_float(t[31]));
      }
      m_tile = ptx::fmax3(mq[0], mq[1], fmaxf(mq[2], mq[3])) * sl2;
    }
    const bool need = m_tile > m_used + kLazyRescale;
    float alpha = 1.0f;
    if (need) {
      alpha = ptx::ex2(m_used - m_tile);
      m_used = m_tile;
    }
    l *= alpha;
    if (!first && __any_sync(0xffffffffu, need)) scale_o(tO, alpha);
    const uint64_t nm2 = ptx::f2_pack(-m_used, -m_used);
    uint64_t acc[4] = {0, 0, 0, 0};
#pragma unroll
    for (int hh = 0; hh < 2; ++hh) {  // P of the first half overwrites S columns 0..31, already read
      uint32_t sh[kBN / 2], pk[kBN / 4];
      ptx::tmem_ld64(tS + 64 * hh, sh);
      if (whole) {
        numerators(sh, c2, nm2, pk, acc);
      } else {
#pragma unroll
        for (int i = 0; i < kBN / 2; ++i)
          if (64 * hh + i >= valid) sh[i] = 0xff800000u;
        numerators(sh, c2, nm2, pk, acc);
      }
      ptx::tmem_st32(tS + 32 * hh, pk);
    }
    l += sum_of(acc);
  }
}

// a[v] of lane q of four becomes a[q] of lane v.
__device__ __forceinline__ void swap_lanes(uint4& a, uint4& b, int bit, bool upper) {
  uint4 x = upper ? a : b;
  x.x = __shfl_xor_sync(0xffffffffu, x.x, bit);
  x.y = __shfl_xor_sync(0xffffffffu, x.y, bit);
  x.z = __shfl_xor_sync(0xffffffffu, x.z, bit);
  x.w = __shfl_xor_sync(0xffffffffu, x.w, bit);
  a = upper ? x : a;
  b = upper ? b : x;
}
__device__ __forceinline__ void transpose4(uint4 (&a)[4], int lane) {
  swap_lanes(a[0], a[1], 1, lane & 1);
  swap_lanes(a[2], a[3], 1, lane & 1);
  swap_lanes(a[0], a[2], 2, lane & 2);
  swap_lanes(a[1], a[3], 2, lane & 2);
}

__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float4* chain = reinterpret_cast<float4*>(smem + kSmemChain);  // [2][128]: reference, sum, pending factor
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kSmemBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  const PagedView& w = p.view;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned long long limit = p.wait_limit_ns;

  ptx::let_next_launch();
  ptx::wait_previous();
  const PagedWork& work = *p.work;
  const int cta = blockIdx.x;
  if (cta >= work.n_ctas) return;
  const int G = p.group;
  const int tpt = kBM / G;  // tokens of a query tile
  PagedWalk walk;
  walk.blocks = p.blocks;
  walk.work = &work;
  walk.n_blocks = work.n_blocks;
  walk.tpt = tpt;
  walk.cta = cta;
  walk.in_step = work.in_step != 0;
  walk.wave = 0;
  const PagedShare& share = work.share[cta];
  walk.left = share.left;
  walk.h = share.h;
  walk.b = share.b;
  walk.t = share.t;
  walk.i = share.i;
  walk.pos = share.pos;
  if (threadIdx.x == 32) {
    ptx::mbar_init(&bars[kBarQ], 1);
    ptx::mbar_init(&bars[kBarQEmpty], 1);
    for (int i = 0; i < 2; ++i) {
      ptx::mbar_init(&bars[kBarKFull + i], 1);
      ptx::mbar_init(&bars[kBarKEmpty + i], 1);
      ptx::mbar_init(&bars[kBarVFull + i], 1);
      ptx::mbar_init(&bars[kBarVEmpty + i], 1);
      ptx::mbar_init(&bars[kBarSFull + i], 1);
      ptx::mbar_init(&bars[kBarPFull + i], kBM);
    }
    ptx::mbar_init(&bars[kBarODone], 1);
    ptx::mbar_init(&bars[kBarDrain], 1);
    ptx::mbar_init(&bars[kBarVFix], 1);
    ptx::fence_mbar_init();
  } else if (warp == 9) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  // rows of the query tiles that no box fills (128 is no multiple of G) are zeros
  const int pad = kBM - tpt * G;
  for (int i = threadIdx.x; i < pad * 32; i += kThreads) {
    const int r = tpt * G + i / 32, c = i & 31;  // 32 16-byte pieces: two tiles, two halves, eight each
    *reinterpret_cast<uint4*>(smem + kSmemQ + (c >> 3) * kSlab + r * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
  }
  if (pad) ptx::fence_proxy_async_smem();
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  PagedUnit u;

  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    const int box = min(1 << w.page_shift, kBN);  // tokens per copy
    const int n_box = kBN / box;
    const int b = lane % n_box, c = (lane / n_box) & 1;
    const bool is_v = (lane / n_box) & 2, mine = lane < 4 * n_box;
    const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
    uint8_t* dst = smem + (is_v ? kSmemV : kSmemK) + c * kSlab + b * box * 128;
    if (lane == 0) {
      ptx::prefetch_tmap(&tm_q);
      ptx::prefetch_tmap(&tm_k);
      ptx::prefetch_tmap(&tm_v);
    }
    bool ok = true;
    int nq = 0, nk = 0, nv = 0;  // units' queries, K and V tiles issued
    while (ok && walk.next(u)) {
      if (nq > 0) {
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kBarQEmpty], (nq - 1) & 1, limit));
        if (!ok) break;
      }
      if (lane == 0) {
        ptx::mbar_arrive_expect_tx(&bars[kBarQ], (u.two ? 2 : 1) * 2 * 128 * tpt * G);
        for (int t = 0; t < (u.two ? 2 : 1); ++t)
          for (int cc = 0; cc < 2; ++cc)
            ptx::tma_load_3d(smem + kSmemQ + t * kTile + cc * kSlab, &tm_q, &bars[kBarQ], cc * 64, u.h * G,
                             u.k.row0 + t * tpt);
      }
      ++nq;
      const int j1 = min(u.k.keys, u.t1 * kBN);
      int id = -1;
      if (mine && u.j0 + b * box < j1) id = paged_id(w, u.k.seq, (u.j0 + b * box) >> w.page_shift);
      for (int t = 0; t < u.n_tiles; ++t) {
        const int st = nk & 1;
        const int j = u.j0 + t * kBN + b * box;
        const int page = max(id, 0);
        if (mine && j + kBN < j1) id = paged_id(w, u.k.seq, (j + kBN) >> w.page_shift);
        const int bytes = (max(0, min(kBN, j1 - u.j0 - t * kBN)) + box - 1) / box * box * 256;
        const int row = (u.h << w.page_shift) + (j & ((1 << w.page_shift) - 1));
        if (nk >= 2) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kBarKEmpty + st], ((nk - 2) >> 1) & 1, limit));
          if (!ok) break;
        }
        if (lane == 0) ptx::mbar_arrive_expect_tx(&bars[kBarKFull + st], bytes);
        __syncwarp();
        if (mine && !is_v && j < j1) ptx::tma_load_3d(dst + st * kTile, tm, &bars[kBarKFull + st], c * 64, row, page);
        ++nk;
        if (nv >= 2) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kBarVEmpty + st], ((nv - 2) >> 1) & 1, limit));
          if (!ok) break;
        }
        if (lane == 0) ptx::mbar_arrive_expect_tx(&bars[kBarVFull + st], bytes);
        __syncwarp();
        if (mine && is_v && j < j1) ptx::tma_load_3d(dst + st * kTile, tm, &bars[kBarVFull + st], c * 64, row, page);
        ++nv;
      }
      // the last tile's V rows from the last visible token to the end of its step of 16
      if (ok && (u.last_valid & 15)) {
        const int st = (nv - 1) & 1;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kBarVFull + st], ((nv - 1) >> 1) & 1, limit));
        // The value product before this tile's was issued, so the issuer has seen the kBarVFix of the unit before: of
        // two phases completed in a row it would wait for the one that has the first one's parity again.
        if (ok && nv >= 2)
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kBarVEmpty + (st ^ 1)], ((nv - 2) >> 1) & 1, limit));
        if (ok) {
          const int end = (u.last_valid + 15) & ~15;
          for (int i = lane; i < (end - u.last_valid) * 16; i += 32)
            *reinterpret_cast<uint4*>(smem + kSmemV + st * kTile + ((i >> 3) & 1) * kSlab +
                                      (u.last_valid + (i >> 4)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bars[kBarVFix]);
        }
      }
    }
    if (lane == 0) {
      if (!ok) paged_report(w, kStatusTimeout);
      // every copy issued must land before the thread block may exit
      if (nq > 0) ptx::mbar_wait(&bars[kBarQ], (nq - 1) & 1, kDrainNs);
      for (int t = max(0, nk - 2); t < nk; ++t) ptx::mbar_wait(&bars[kBarKFull + (t & 1)], (t >> 1) & 1, kDrainNs);
      for (int t = max(0, nv - 2); t < nv; ++t) ptx::mbar_wait(&bars[kBarVFull + (t & 1)], (t >> 1) & 1, kDrainNs);
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0) {
      const uint32_t k_addr = ptx::smem_u32(smem + kSmemK);
      const uint32_t v_addr = ptx::smem_u32(smem + kSmemV);
      bool ok = true;
      int g0 = 0;                 // tiles of the units before this one
      int used[2] = {0, 0};       // P tiles that each accumulator took before this unit
      int n_unit = 0, n_fix = 0;  // units, and those whose last V tile was mended
      while (ok && walk.next(u)) {
        const uint32_t q_addr[2] = {ptx::smem_u32(smem + kSmemQ), ptx::smem_u32(smem + kSmemQ + (u.two ? kTile : 0))};
        const bool fix = (u.last_valid & 15) != 0;
        auto issue_s = [&](int t, uint32_t kt) {
#pragma unroll
          for (int kk = 0; kk < kHeadDim / 16; ++kk)
            ptx::mma_ss(tmem + col_s(t), desc_kmajor(q_addr[t], kk), desc_kmajor(kt, kk), kIdescS, kk > 0 ? 1u : 0u);
        };
        auto wait_k = [&](int j) {
          return ptx::mbar_wait(&bars[kBarKFull + ((g0 + j) & 1)], ((g0 + j) >> 1) & 1, limit);
        };
        // V of tile j observed, the unit's last one's stale rows zeroed
        auto wait_v = [&](int j) -> bool {
          if (!ptx::mbar_wait(&bars[kBarVFull + ((g0 + j) & 1)], ((g0 + j) >> 1) & 1, limit)) return false;
          return j + 1 < u.n_tiles || !fix || ptx::mbar_wait(&bars[kBarVFix], n_fix & 1, limit);
        };
        // O_t += P_t V(j), the use-th of the unit into this accumulator; V(j) already observed
        auto issue_pv = [&](int t, int j, int use, bool frees_v) -> bool {
          if (!ptx::mbar_wait(&bars[kBarPFull + t], (used[t] + use) & 1, limit)) return false;
          ptx::tc_fence_after();
          const uint32_t vt = v_addr + ((g0 + j) & 1) * kTile;
          const int steps = j + 1 < u.n_tiles ? kBN / 16 : (u.last_valid + 15) >> 4;
#pragma unroll
          for (int kk = 0; kk < kBN / 16; ++kk)
            if (kk < steps)
              ptx::mma_ts(tmem + col_o(t), tmem + col_s(t) + kk * 8, desc_v(vt, kk), kIdescPV,
                          (use > 0 || kk > 0) ? 1u : 0u);
          if (frees_v) ptx::mma_commit(&bars[kBarVEmpty + ((g0 + j) & 1)]);
          return true;
        };
        if (!ptx::mbar_wait(&bars[kBarQ], n_unit & 1, limit)) { ok = false; break; }
        if (u.two) {
          // S0(j), PV1(j-1), S1(j), PV0(j): one warpgroup's softmax beside the other tile's products;
          // the waits on V(j) and K(j+1) are taken before the wait for P0(j), where this thread idles
          bool k_ready = wait_k(0);
          if (!k_ready) ok = false;
          for (int j = 0; ok && j < u.n_tiles; ++j) {
            if (!k_ready && !wait_k(j)) { ok = false; break; }
            ptx::tc_fence_after();
            const uint32_t kt = k_addr + ((g0 + j) & 1) * kTile;
            issue_s(0, kt);
            ptx::mma_commit(&bars[kBarSFull + 0]);
            if (j > 0 && !issue_pv(1, j - 1, j - 1, true)) { ok = false; break; }
            issue_s(1, kt);
            ptx::mma_commit(&bars[kBarSFull + 1]);
            ptx::mma_commit(&bars[kBarKEmpty + ((g0 + j) & 1)]);
            if (j + 1 == u.n_tiles) ptx::mma_commit(&bars[kBarQEmpty]);
            if (!wait_v(j)) { ok = false; break; }
            k_ready = j + 1 < u.n_tiles && ptx::mbar_try_wait(&bars[kBarKFull + ((g0 + j + 1) & 1)], ((g0 + j + 1) >> 1) & 1);
            if (!issue_pv(0, j, j, false)) { ok = false; break; }
          }
          if (ok && !issue_pv(1, u.n_tiles - 1, u.n_tiles - 1, true)) ok = false;
          used[0] += u.n_tiles;
          used[1] += u.n_tiles;
        } else {
          // two chains over the one query tile: S(j) into buffer j & 1 while the other's softmax runs
          for (int j = 0; ok && j < u.n_tiles; ++j) {
            if (!wait_k(j)) { ok = false; break; }
            ptx::tc_fence_after();
            issue_s(j & 1, k_addr + ((g0 + j) & 1) * kTile);
            ptx::mma_commit(&bars[kBarSFull + (j & 1)]);
            ptx::mma_commit(&bars[kBarKEmpty + ((g0 + j) & 1)]);
            if (j + 1 == u.n_tiles) ptx::mma_commit(&bars[kBarQEmpty]);
            if (j > 0 && !(wait_v(j - 1) && issue_pv((j - 1) & 1, j - 1, (j - 1) >> 1, true))) ok = false;
          }
          const int j = u.n_tiles - 1;
          if (ok && !(wait_v(j) && issue_pv(j & 1, j, j >> 1, true))) ok = false;
          used[0] += (u.n_tiles + 1) >> 1;
          used[1] += u.n_tiles >> 1;
        }
        if (ok) ptx::mma_commit(&bars[kBarODone]);
        g0 += u.n_tiles;
        n_fix += fix;
        ++n_unit;
      }
      if (!ok) paged_report(w, kStatusTimeout);
      // everything issued must complete before TMEM is released
      ptx::mma_commit(&bars[kBarDrain]);
      ptx::mbar_wait(&bars[kBarDrain], 0, kDrainNs);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax warpgroups
    const int wg = warp >> 2;
    const int r = threadIdx.x & 127;
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t tS = lane_base + col_s(wg), tO = lane_base + col_o(wg);
    const float sl2 = p.scale_log2;
    const uint64_t c2 = ptx::f2_pack(sl2, sl2);
    const int tok = r / G;
    // After an expired wait a warp skips further waits and work but still passes the named barriers.
    bool ok = true;
    int n_s = 0, n_unit = 0;  // score tiles and units taken
    while (walk.next(u)) {
      const int tile0 = u.two ? wg * tpt : 0;  // this query tile's first token in the unit
      const bool live = r < min(tpt, u.k.cnt - tile0) * G;
      // how many of the part's keys this row sees; rows of no token see what the unit sees, so that
      // they hold no whole warp on the masked path
      const int seen = min(u.k.keys, p.causal && live ? u.k.place0 + tile0 + tok + 1 : u.k.keys) - u.j0;
      const int n_mine = u.two ? u.n_tiles : (u.n_tiles + 1 - wg) >> 1;
      float m_used = kNoKey, l = 0.f, pend = 1.0f;
      // A unit of one score tile takes nothing from the second warpgroup before its end: it may not complete kBarODone
      // while a warp there still waits for that of the unit before, which has the other parity. (This and the wait
      // before kBarVFix: 3000 streams of 1 to 20 tokens 204 us, 199 without; long units the same.)
      if (!u.two && u.n_tiles == 1) {
        if (wg == 0)
          ptx::named_bar_sync(2, 256);
        else
          ptx::named_bar_arrive(2, 256);
      }
      for (int i = 0; i < n_mine; ++i, ++n_s) {
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kBarSFull + wg], n_s & 1, limit));
        if (!ok) continue;
        ptx::tc_fence_after();
        softmax_tile(i == 0, seen - (u.two ? i : 2 * i + wg) * kBN, tS, tO, sl2, c2, m_used, l, pend);
        ptx::tmem_st_wait();
        ptx::tc_fence_before();
        ptx::mbar_arrive(&bars[kBarPFull + wg]);
      }
      if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kBarODone], n_unit & 1, limit));
      ++n_unit;
      ptx::tc_fence_after();
      l *= pend;
      float f0 = pend, f1 = 0.f;  // factors of the row's accumulator, and of the other chain's
      bool has1 = false;
      if (!u.two) {
        // join the chains: both warpgroups see both accumulators, and take half of the columns each
        chain[wg * kBM + r] = make_float4(m_used, l, pend, 0.f);
        ptx::named_bar_sync(1, 256);
        const float4 a = chain[r], e = chain[kBM + r];
        const float m = fmaxf(a.x, e.x);
        const float fa = ptx::ex2(a.x - m), fe = ptx::ex2(e.x - m);
        f0 = a.z * fa;
        f1 = e.z * fe;
        l = a.y * fa + e.y * fe;
        m_used = m;
        has1 = u.n_tiles > 1;
      }
      const long long row = u.k.row0 + tile0 + tok;
      const int head = u.h * G + r - tok * G;
      const bool whole = u.t0 == 0 && u.t1 == u.k.tiles;
      const float inv = l == 0.f ? 0.f : 1.0f / l;  // a row that saw nothing: its accumulator may hold anything
      const int part_row = (u.two ? wg * kBM : 0) + r;
      float4* part = reinterpret_cast<float4*>(p.part) + static_cast<long long>(u.slot) * kPagedPartRows * (kHeadDim / 4);
      // where this lane writes its 16 bytes of each of the rows of its group of four lanes
      uint16_t* to[4];
      const unsigned live_rows = __ballot_sync(0xffffffffu, live) >> (lane & ~3);
      {
        const unsigned long long mine = reinterpret_cast<unsigned long long>(p.out + row * p.out_stride + head * kHeadDim);
#pragma unroll
        for (int v = 0; v < 4; ++v)
          to[v] = reinterpret_cast<uint16_t*>(__shfl_sync(0xffffffffu, mine, (lane & ~3) + v)) + (lane & 3) * 8;
      }
#pragma unroll 1
      for (int c = u.two ? 0 : 2 * wg; ok && c < (u.two ? 4 : 2 * wg + 2); ++c) {
        uint32_t rr[32];
        ptx::tmem_ld32(lane_base + col_o(u.two ? wg : 0) + 32 * c, rr);
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(rr[i]) * f0;
        if (has1) {
          ptx::tmem_ld32(lane_base + col_o(1) + 32 * c, rr);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] += __uint_as_float(rr[i]) * f1;
        }
        if (whole) {
          uint4 ob[4];
          uint32_t* o32 = reinterpret_cast<uint32_t*>(ob);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            o32[i] = l != 0.f ? pack_bf16x2(x[2 * i] * inv, x[2 * i + 1] * inv) : 0u;
          // a row's 64 bytes by four lanes at once instead of by one lane piece after piece (3000 streams of 1 to 20
          // tokens 6 us less; the code costs the long units' loop up to a hundredth)
          transpose4(ob, lane);
#pragma unroll
          for (int v = 0; v < 4; ++v)
            if (live_rows >> v & 1u) *reinterpret_cast<uint4*>(to[v] + 32 * c) = ob[v];
        } else if (live) {
          // whole lines: 512 bytes of one row per thread, the rows' one after the other, made this 6 us of a unit
#pragma unroll
          for (int v = 0; v < 8; ++v)
            part[paged_part_place(part_row, 8 * c + v)] = make_float4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
        }
      }
      if (ok && live && (u.two || wg == 0)) {
        if (!whole) {
          p.part_ml[static_cast<long long>(u.slot) * kPagedPartRows + part_row] = make_float2(m_used, l);
        } else {
          const float z = l > 0.f ? m_used + log2f(l) : l == 0.f ? -INFINITY : l;
          const long long rh = row * p.q_heads + head;
          if (p.lse != nullptr) p.lse[rh] = z * kLn2;
          if (p.lse2 != nullptr) p.lse2[rh] = z;
        }
      }
      // neither chain's next product may overwrite an accumulator that the other still reads
      if (!u.two) {
        ptx::tc_fence_before();
        ptx::named_bar_sync(1, 256);
      }
    }
    if (!ok && lane == 0) paged_report(w, kStatusTimeout);
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 9) ptx::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------------------------
// Attention weight of chunks. With z the rows' log-sum-exp from the attention before, key j of KV
// head h gathers sum over the group's rows i that see it of 2^(s_ij - z_i). The product is
// taken transposed, S^T = K Q^T: a thread block owns 128 keys (the TMEM lanes) and walks the query tiles
// (128 columns), so that a key's sum stays in one thread's registers: no atomics, a fixed order.
//   warps 0-7: two warpgroups, one key per thread, every second query tile each (their sums are added
//   up at the end); warp 8: TMA producer (the K tile once, query tiles into two stages); warp 9: TMEM
//   allocator and MMA issuer, one S buffer per warpgroup.
// The exponentials bound it (128 x 128 per tile against 8 MMA steps: 1024 clocks at 16 a clock). Each is
// one of a chain of short dependent instructions, so two thread blocks per SM take turns, sixteen such
// warps; and a key tile needs some 6000 clocks besides (K and first query tile, end), which the other covers.
// The thread blocks stay and draw key tiles from a counter, since their costs differ with the chunks'
// lengths. (One thread block per key tile of the longest stream: 105 us for four chunks of 128 to 512 tokens over
// 1024 to 8192, their slots held by empty ones for a third of the time.)
constexpr int kWGroups = 2;
constexpr int kWThreads = kWGroups * 128 + 64;
constexpr int kWSmemQ = kTile;
constexpr int kWSmemLse = kWSmemQ + kWGroups * kTile;  // [group][2][128] floats: -z per row, two tiles
constexpr int kWSmemSum = kWSmemLse + kWGroups * 2 * kBM * 4;  // [group - 1][128]: the other groups' sums
constexpr int kWSmemBar = kWSmemSum + (kWGroups - 1) * kBM * 4;
constexpr int kWSmemBytes = kWSmemBar + 256 + 1024;

enum : int {
  kWbK = 0,
  kWbQFull = 1,                        // +stage
  kWbQEmpty = kWbQFull + kWGroups,     // +stage
  kWbSFull = kWbQEmpty + kWGroups,     // +buffer
  kWbSEmpty = kWbSFull + kWGroups,     // +buffer
  kWbDrain = kWbSEmpty + kWGroups,
  kWbCount
};

// One query tile's weights of this thread's key, added to acc; rows outside [lo, hi) do not count.
template <bool kWhole>
__device__ __forceinline__ void weigh_tile(uint32_t tS, const float* z, uint64_t c2, int lo, int hi, uint64_t* s_empty,
                                           uint64_t (&acc)[4]) {
#pragma unroll
  for (int part = 0; part < 4; ++part) {
    uint32_t sv[32];
    ptx::tmem_ld32(tS + part * 32, sv);
    if (part == 3) {
      ptx::tc_fence_before();
      ptx::mbar_arrive(s_empty);
    }
    const ulonglong2* zz = reinterpret_cast<const ulonglong2*>(z + part * 32);
#pragma unroll
    for (int k = 0; k < 16; k += 2) {
      const ulonglong2 z2 = zz[k >> 1];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint64_t v = ptx::f2_fma(
            ptx::f2_pack(__uint_as_float(sv[2 * (k + e)]), __uint_as_float(sv[2 * (k + e) + 1])), c2, e ? z2.y : z2.x);
        float a, b;
        ptx::f2_unpack(v, a, b);
        a = ptx::ex2(a);
        b = ptx::ex2(b);
        if (!kWhole) {
          const int i = part * 32 + 2 * (k + e);
          a = i >= lo && i < hi ? a : 0.f;
          b = i + 1 >= lo && i + 1 < hi ? b : 0.f;
        }
        acc[(k + e) & 3] = ptx::f2_add(acc[(k + e) & 3], ptx::f2_pack(a, b));
      }
    }
  }
}

__global__ void __launch_bounds__(kWThreads, 2)
    paged_weight_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ PagedAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* nz = reinterpret_cast<float*>(smem + kWSmemLse);
  float* sums = reinterpret_cast<float*>(smem + kWSmemSum);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWSmemBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kWbCount);
  const PagedView& w = p.view;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned long long limit = p.wait_limit_ns;
  int* ticket = reinterpret_cast<int*>(bars + kWbCount + 1);
  ptx::let_next_launch();
  ptx::wait_previous();
  if (p.work != nullptr && p.work->n_blocks == 0) return;  // the plan found nothing to do
  PagedTiles<kBN> place;
  place.order = p.order;
  place.count(w, false);  // a bad length was reported by the attention
  if (static_cast<int>(blockIdx.x) >= place.all) return;
  const int G = p.group;
  const int tpt = kBM / G;
  if (threadIdx.x == 0) {
    ptx::mbar_init(&bars[kWbK], 1);
    for (int i = 0; i < kWGroups; ++i) {
      ptx::mbar_init(&bars[kWbQFull + i], 1);
      ptx::mbar_init(&bars[kWbQEmpty + i], 1);
      ptx::mbar_init(&bars[kWbSFull + i], 1);
      ptx::mbar_init(&bars[kWbSEmpty + i], kBM);
    }
    ptx::mbar_init(&bars[kWbDrain], 1);
    ptx::fence_mbar_init();
  }
  if (warp == kWGroups * 4 + 1) {
    ptx::tmem_alloc(tmem_slot, kWGroups * 128);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  long long x = blockIdx.x;  // this thread block's unit; the next one is drawn while it is worked on
  int n_k = 0, g0 = 0;       // units with work done, and their query tiles
  bool ok = true;            // no wait of this thread's warp has expired
  while (x < place.all) {
    unsigned drawn = 0;
    if (threadIdx.x == 0) drawn = atomicAdd(p.ticket, 1u);
    place.go_to(w, x);
    const PagedSeq& q = place.q;
    const int s = place.s, h = place.h, j0 = place.t * kBN;
    const int first_place = q.kv - q.n_q;  // place of the chunk's first token
    // query tiles from the first with a row that sees this tile's first key (none if nothing is cached)
    const int qt0 = p.causal ? max(0, j0 - first_place) / tpt : 0;
    const int n_qt = j0 < q.kv ? (q.n_q + tpt - 1) / tpt - qt0 : 0;

    if (warp == kWGroups * 4) {
      // ---------------------------------------------------------- TMA producer
      const int box = min(1 << w.page_shift, kBN);
      const int n_box = kBN / box;
      const int b = lane % n_box, c = lane / n_box;
      const int j = j0 + b * box;
      if (n_qt > 0) {
        if (lane == 0) ptx::mbar_arrive_expect_tx(&bars[kWbK], (min(kBN, q.kv - j0) + box - 1) / box * box * 256);
        __syncwarp();
        if (c < 2 && j < q.kv)
          ptx::tma_load_3d(smem + c * kSlab + b * box * 128, &tm_k, &bars[kWbK], c * 64,
                           (h << w.page_shift) + (j & ((1 << w.page_shift) - 1)),
                           max(0, paged_id(w, s, j >> w.page_shift)));
        __syncwarp();
        if (lane == 0) {
          for (int t = 0; ok && t < n_qt; ++t) {
            const int g = g0 + t, st = g % kWGroups;
            if (g >= kWGroups) ok = ptx::mbar_wait(&bars[kWbQEmpty + st], (g / kWGroups - 1) & 1, limit);
            if (!ok) break;
            ptx::mbar_arrive_expect_tx(&bars[kWbQFull + st], 2 * 128 * tpt * G);
            for (int cc = 0; cc < 2; ++cc)
              ptx::tma_load_3d(smem + kWSmemQ + st * kTile + cc * kSlab, &tm_q, &bars[kWbQFull + st], cc * 64, h * G,
                               q.q0 + (qt0 + t) * tpt);
          }
          // every copy issued lands before the K tile's memory, or the thread block, is given up
          ptx::mbar_wait(&bars[kWbK], n_k & 1, kDrainNs);
        }
      }
      __syncwarp();
    } else if (warp == kWGroups * 4 + 1) {
      // ---------------------------------------------------------- MMA issuer
      if (lane == 0 && n_qt > 0) {
        const uint32_t ka = ptx::smem_u32(smem);
        if (ok) ok = ptx::mbar_wait(&bars[kWbK], n_k & 1, limit);
        for (int t = 0; ok && t < n_qt; ++t) {
          const int g = g0 + t, st = g % kWGroups;  // the query stage, the S buffer and the warpgroup
          ok = ptx::mbar_wait(&bars[kWbQFull + st], (g / kWGroups) & 1, limit) &&
               (g < kWGroups || ptx::mbar_wait(&bars[kWbSEmpty + st], (g / kWGroups - 1) & 1, limit));
          if (!ok) break;
          ptx::tc_fence_after();
          const uint32_t qa = ptx::smem_u32(smem + kWSmemQ + st * kTile);
#pragma unroll
          for (int kk = 0; kk < kHeadDim / 16; ++kk)
            ptx::mma_ss(tmem + st * 128, desc_kmajor(ka, kk), desc_kmajor(qa, kk), kIdescS, kk > 0 ? 1u : 0u);
          ptx::mma_commit(&bars[kWbSFull + st]);
          ptx::mma_commit(&bars[kWbQEmpty + st]);
        }
      }
      __syncwarp();
    } else if (n_qt > 0) {
      const int wg = warp >> 2;
      const int r = threadIdx.x & 127;  // key of the tile, and the query row whose z this thread fetches
      const uint32_t tS = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + wg * 128;
      const uint64_t c2 = ptx::f2_pack(p.scale_log2, p.scale_log2);
      const int my_tok = r / G;
      const float* z_of = p.lse2 + static_cast<long long>(q.q0) * p.q_heads + h * G + r - my_tok * G;
      // -z of row r of query tile t; what rows of no token get is masked below
      auto fetch = [&](int t) -> float {
        const int tok = (qt0 + t) * tpt + my_tok;
        if (t >= n_qt || my_tok >= tpt || tok >= q.n_q) return 0.f;
        return -*(z_of + static_cast<long long>(tok) * p.q_heads);
      };
      const int t0 = (wg - g0) & (kWGroups - 1);  // this warpgroup's first tile of the unit
      float next = fetch(t0);
      float* to = p.weight + (static_cast<long long>(s) * w.kv_heads + h) * p.weight_stride + j0 + r;
      const float old = wg == 0 && j0 + r < first_place ? *to : 0.f;  // the chunk's own keys start from zero
      uint64_t acc[4] = {0, 0, 0, 0};
      for (int t = t0; t < n_qt; t += kWGroups) {
        const int n = (g0 + t) / kWGroups;  // tiles that this warpgroup took before
        float* z = nz + (wg * 2 + (n & 1)) * kBM;
        z[r] = next;
        next = fetch(t + kWGroups);
        // rows [lo, hi) of this tile are of the chunk and see this thread's key
        const int tok0 = (qt0 + t) * tpt;
        const int hi = min(tpt, q.n_q - tok0) * G;
        const int lo = p.causal ? max(0, j0 + r - first_place - tok0) * G : 0;
        const bool whole = __all_sync(0xffffffffu, lo == 0 && hi == kBM);
        if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kWbSFull + wg], n & 1, limit));
        ptx::named_bar_sync(1 + wg, kBM);  // every row's z is in place; the readers of two tiles ago are past it
        if (!ok) continue;
        ptx::tc_fence_after();
        // two copies, so that whole tiles pay nothing for the mask (its compares and selects were three
        // fifths of all instructions)
        if (whole)
          weigh_tile<true>(tS, z, c2, lo, hi, &bars[kWbSEmpty + wg], acc);
        else
          weigh_tile<false>(tS, z, c2, lo, hi, &bars[kWbSEmpty + wg], acc);
      }
      // the warpgroups' sums of a key, in order
      if (wg != 0) sums[(wg - 1) * kBM + r] = sum_of(acc);
      ptx::named_bar_sync(1 + kWGroups, kWGroups * kBM);
      if (wg == 0 && ok && j0 + r < q.kv) {
        float sum = sum_of(acc);
        for (int i = 0; i < kWGroups - 1; ++i) sum += sums[i * kBM + r];
        *to = old + sum;
      }
    }
    g0 += n_qt;
    n_k += n_qt > 0;
    if (threadIdx.x == 0) *ticket = static_cast<int>(min(drawn, 0x7fffffffu - gridDim.x));
    __syncthreads();
    x = static_cast<long long>(gridDim.x) + *ticket;
    __syncthreads();
  }
  if (!ok && lane == 0) paged_report(w, kStatusTimeout);
  if (warp == kWGroups * 4 && lane == 0)  // the last query tiles' copies
    for (int g = max(0, g0 - kWGroups); g < g0; ++g) ptx::mbar_wait(&bars[kWbQFull + g % kWGroups], (g / kWGroups) & 1, kDrainNs);
  if (warp == kWGroups * 4 + 1 && lane == 0) {
    // everything issued must complete before TMEM is released
    ptx::mma_commit(&bars[kWbDrain]);
    ptx::mbar_wait(&bars[kWbDrain], 0, kDrainNs);
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == kWGroups * 4 + 1) ptx::tmem_dealloc(tmem, kWGroups * 128);
}

// the dynamic shared-memory limit is a per-device setting: raised once on every device this process
// launches on
cudaError_t configure() {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static bool configured[kMaxDevices] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (configured[dev]) return cudaSuccess;
  err = cudaFuncSetAttribute(paged_chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (err == cudaSuccess)
    err = cudaFuncSetAttribute(paged_weight_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kWSmemBytes);
  if (err == cudaSuccess) configured[dev] = true;
  return err;
}

}  // namespace

cudaError_t launch_paged_chunk(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                               const PagedAttnParams& p, cudaStream_t stream) {
  cudaError_t err = configure();
  if (err != cudaSuccess) return err;
  const bool small = std::max(p.view.n_seqs, p.n_blocks) <= 256;
  err = launch_after(small ? paged_plan_kernel<256> : paged_plan_kernel<1024>, 1, small ? 256 : 1024, 0, stream, p);
  if (err == cudaSuccess)
    err = launch_after(paged_chunk_kernel, kSmCount, kThreads, kSmemBytes, stream, tm_q, tm_k, tm_v, p);
  return err;
}

cudaError_t launch_paged_weight(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const PagedAttnParams& p,
                                cudaStream_t stream) {
  const cudaError_t err = configure();
  if (err != cudaSuccess) return err;
  return launch_after(paged_weight_kernel, 2 * kSmCount, kWThreads, kWSmemBytes, stream, tm_q, tm_k, p);
}

}  // namespace rkv
