// Device helpers shared by the paged-cache kernels: which stream a chunk row belongs to, the
// checked lengths of a stream, the address of a cached token.
#pragma once

#include <utility>

#include "paged_internal.h"

namespace rkv {

// Launch a kernel that may be set up while the stream's previous one still runs; it waits for that one
// itself (ptx::wait_previous, in every thread block, before it touches memory).
// What it reads may still be written while it is resident, so no load of it may be one of read-only data
// (__ldg, which holds for memory that no one writes during the whole kernel): plain loads, after the wait.
template <typename... P, typename... A>
cudaError_t launch_after(void (*kernel)(P...), dim3 grid, unsigned block, size_t smem, cudaStream_t stream,
                         A&&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, std::forward<A>(args)...);
}

__device__ __forceinline__ void paged_report(const PagedView& w, unsigned bits) {
  if (w.status != nullptr) atomicOr(w.status, bits);
}

// The stream of chunk row `row` (the last one whose rows start at or before it), or -1. A whole
// warp calls it with the same row: 32 starts are probed at a time, so 1024 streams take two
// dependent loads instead of ten.
__device__ __forceinline__ int paged_seq_of_row(const PagedView& w, int row) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = w.n_seqs + 1;  // starts [lo, hi) are undecided; the answer counts those <= row
  while (hi > lo) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const bool le = i < hi && w.q_start[i] <= row;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    if (c == 0) {
      hi = lo;
    } else {
      const int nlo = lo + (c - 1) * step + 1;
      hi = min(hi, lo + c * step);
      lo = nlo;
    }
  }
  const int s = lo - 1;
  return s < w.n_seqs ? s : -1;
}

struct PagedSeq {
  int q0, n_q, kv;  // first chunk row, chunk rows (if ok), cached tokens
  bool ok;
  bool falls;  // its row range ends before it begins
};

// The lengths of stream s, checked against the batch's bounds.
__device__ __forceinline__ PagedSeq paged_seq(const PagedView& w, int s) {
  PagedSeq r;
  r.q0 = w.q_start[s];
  const int q1 = w.q_start[s + 1];
  r.kv = w.kv_len[s];
  r.ok = r.q0 >= 0 && q1 >= r.q0 && q1 <= w.n_rows && q1 - r.q0 <= w.max_q && r.kv >= 0 && r.kv <= w.max_kv;
  r.falls = q1 < r.q0;
  r.n_q = r.ok ? q1 - r.q0 : 0;  // the difference of any two ints may not fit one
  return r;
}

// Page id at place `i` of stream s's list, or -1 (reported) if it is not a page of the pool.
__device__ __forceinline__ int paged_id(const PagedView& w, int s, int i) {
  const int id = w.table[static_cast<long long>(s) * w.table_stride + i];
  if (static_cast<unsigned>(id) < static_cast<unsigned>(w.n_pages)) return id;
  paged_report(w, kStatusPage);
  return -1;
}

// Element offset of token `slot` (place within the page) of KV head h in page `id`.
__device__ __forceinline__ long long paged_offset(const PagedView& w, int id, int h, int slot) {
  return static_cast<long long>(id) * w.page_stride +
         (static_cast<long long>(h) * (1 << w.page_shift) + slot) * kHeadDim;
}

// A part of the chunk form: float4 number `col` (of 32) of row `row`. Eight rows lie side by side, so that a thread per
// row writes, and a thread per row and float4 reads, whole lines.
__device__ __forceinline__ int paged_part_place(int row, int col) { return ((row >> 3) * 32 + col) * 8 + (row & 7); }

// x / y where both nearly always fit 32 bits (a 64-bit division is some 100 instructions).
__device__ __forceinline__ long long quotient(long long x, long long y) {
  return ((x | y) >> 32) == 0 ? static_cast<long long>(static_cast<unsigned>(x) / static_cast<unsigned>(y)) : x / y;
}

// Tiles shared evenly by n thread blocks, at least one each: share c is tiles [start(c), start(c + 1)). Those with one
// tile more lie spread among the others (all in front: 42 us instead of 41 for drafts of 1 to 7 tokens).
struct PagedShares {
  long long all;
  int n;

  __device__ __forceinline__ void split(long long tiles, int most) {
    all = tiles;
    n = static_cast<int>(min(static_cast<long long>(most), tiles));
  }
  __device__ __forceinline__ long long start(int c) const { return quotient(all * c, n); }
  // the share that tile x is in: the last c with floor(all c / n) <= x
  __device__ __forceinline__ int owner(long long x) const { return static_cast<int>(quotient(n * (x + 1) - 1, all)); }
};

// Tiles of kTokens cached tokens of one KV head of a stream: none without rows, one (all masked) if nothing is
// cached.
template <int kTokens>
__device__ __forceinline__ int paged_seq_tiles(const PagedSeq& q) {
  return q.ok && q.n_q > 0 ? max(1, (q.kv + kTokens - 1) / kTokens) : 0;
}

// All tiles of the batch, stream after stream (in the order of `order`, if it is set) and head after head, and a
// place among them. Whole warps call these.
template <int kTokens>
struct PagedTiles {
  const int* order = nullptr;
  long long all;
  int s, h, t;  // the place: stream, head, tile
  PagedSeq q;   // its stream
  int tiles;    // and that stream's tiles of one head
  int q0, n_q, kv, mine;  // lane l: stream l of the first 32, and its tiles

  __device__ __forceinline__ int nth(int i) const { return order != nullptr ? order[i] : i; }
  __device__ __forceinline__ void count(const PagedView& w, bool report) {
    const int lane = threadIdx.x & 31;
    all = 0;
    mine = 0;
    for (int base = 0; base < w.n_seqs; base += 32) {
      int x = 0;
      if (base + lane < w.n_seqs) {
        const PagedSeq y = paged_seq(w, nth(base + lane));
        if (!y.ok && report) paged_report(w, kStatusLength);
        x = paged_seq_tiles<kTokens>(y);
        if (base == 0) {
          q0 = y.q0;
          n_q = y.n_q;
          kv = y.kv;
          mine = x;
        }
      }
      all += __reduce_add_sync(0xffffffffu, x);
    }
    all *= w.kv_heads;
  }
  // to tile x < all
  __device__ __forceinline__ void go_to(const PagedView& w, long long x) {
    const int lane = threadIdx.x & 31;
    long long before = 0;
    for (int base = 0; base < w.n_seqs; base += 32) {
      const int c = base == 0 ? mine : base + lane < w.n_seqs ? paged_seq_tiles<kTokens>(paged_seq(w, nth(base + lane))) : 0;
      int inc = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
      }
      const unsigned hit = __ballot_sync(0xffffffffu, (before + inc) * w.kv_heads > x);
      if (hit) {
        const int l = __ffs(hit) - 1;
        s = nth(base + l);
        before += __shfl_sync(0xffffffffu, inc - c, l);
        tiles = __shfl_sync(0xffffffffu, c, l);
        if (base == 0) {
          q.q0 = __shfl_sync(0xffffffffu, q0, l);
          q.n_q = __shfl_sync(0xffffffffu, n_q, l);
          q.kv = __shfl_sync(0xffffffffu, kv, l);
          q.ok = true;
        } else {
          q = paged_seq(w, s);
        }
        break;
      }
      before += __shfl_sync(0xffffffffu, inc, 31);
    }
    const long long in = x - before * w.kv_heads;
    h = static_cast<int>(quotient(in, tiles));
    t = static_cast<int>(in - static_cast<long long>(h) * tiles);
  }
};

}  // namespace rkv
