// The paged cache's data movement: the write of a chunk into pages and eviction by weight.
#include <algorithm>

#include "paged.cuh"

namespace rkv {
namespace {

// ---------------------------------------------------------------- write
// One warp per chunk row; 16 lanes move one head vector of K and V (16 bytes each).
constexpr int kWriteWarps = 4;

__global__ void __launch_bounds__(kWriteWarps * 32) paged_write_kernel(const __grid_constant__ PagedWriteParams p) {
  const PagedView& w = p.view;
  const int row = blockIdx.x * kWriteWarps + (threadIdx.x >> 5);
  if (row >= w.n_rows) return;
  const int s = paged_seq_of_row(w, row);
  if (s < 0) return;
  const PagedSeq q = paged_seq(w, s);
  const int lane = threadIdx.x & 31;
  const int pos = q.kv - q.n_q + (row - q.q0);
  if (!q.ok || pos < 0) {
    if (lane == 0) paged_report(w, kStatusLength);
    return;
  }
  const int id = paged_id(w, s, pos >> w.page_shift);
  if (id < 0) return;
  const int slot = pos & ((1 << w.page_shift) - 1);
  const int c = (lane & 15) * 8;
  for (int h = lane >> 4; h < w.kv_heads; h += 2) {
    const uint4 kx = __ldg(reinterpret_cast<const uint4*>(p.k + row * p.k_stride + h * kHeadDim + c));
    const uint4 vx = __ldg(reinterpret_cast<const uint4*>(p.v + row * p.v_stride + h * kHeadDim + c));
    const long long to = paged_offset(w, id, h, slot) + c;
    *reinterpret_cast<uint4*>(w.k + to) = kx;
    *reinterpret_cast<uint4*>(w.v + to) = vx;
  }
}

// ---------------------------------------------------------------- eviction: the choice
// Weights as unsigned numbers of the same order: NaN lowest, -0 equal to +0.
__device__ __forceinline__ unsigned weight_key(float x) {
  if (x != x) return 0u;
  const unsigned u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

constexpr int kSelThreads = 1024;
constexpr int kSelWarps = kSelThreads / 32;

// Sum over the block's threads before this one (exclusive), and the block's total.
__device__ __forceinline__ int block_scan(int x, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, wp = threadIdx.x >> 5;
  int inc = x;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += y;
  }
  if (lane == 31) warp_sums[wp] = inc;
  __syncthreads();
  int before = 0, all = 0;
  for (int i = 0; i < kSelWarps; ++i) {
    if (i == wp) before = all;
    all += warp_sums[i];
  }
  __syncthreads();
  total = all;
  return before + inc - x;
}

// One block per (stream, KV head). The weight of rank `need` among the middle tokens is found
// digit by digit (11, 11 and 10 bits of the ordered key: the first digit holds the exponent
// and two bits of the fraction, so that equal digits, which collide in shared memory, are
// few); then one ordered pass lists the kept places and moves their weights.
__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(const __grid_constant__ PagedEvictParams p) {
  __shared__ int hist[2048];
  __shared__ int warp_sums[kSelWarps];
  __shared__ int found[2];
  const PagedView& w = p.view;
  const int s = blockIdx.x / w.kv_heads;
  const int n = __ldg(w.kv_len + s);
  int* kept = p.kept + static_cast<long long>(blockIdx.x) * p.keep;
  if (n < 0 || n > w.max_kv) {
    if (threadIdx.x == 0) paged_report(w, kStatusLength);
    for (int i = threadIdx.x; i < p.keep; i += kSelThreads) kept[i] = -1;
    return;
  }
  if (n <= p.keep) {
    for (int i = threadIdx.x; i < p.keep; i += kSelThreads) kept[i] = i < n ? i : -1;
    return;
  }
  float* wt = p.weight + static_cast<long long>(blockIdx.x) * p.weight_stride;
  const int a = p.sinks, b = n - p.recent;  // the middle: sinks + recent <= keep < n
  const int need = p.keep - p.sinks - p.recent;
  unsigned prefix = 0, mask = 0;
  int rem = need;
  for (int pass = 0; pass < 3 && need > 0; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bins = pass == 2 ? 1024 : 2048;
    for (int i = threadIdx.x; i < bins; i += kSelThreads) hist[i] = 0;
    __syncthreads();
    for (int i = a + threadIdx.x; i < b; i += kSelThreads) {
      const unsigned u = weight_key(wt[i]);
      if ((u & mask) == prefix) atomicAdd(&hist[(u >> shift) & (bins - 1)], 1);
    }
    __syncthreads();
    // bins from the top: thread t owns the pair of bins bins - 2 - 2t, bins - 1 - 2t
    const int hi = bins - 1 - 2 * static_cast<int>(threadIdx.x);
    const int c1 = hi > 0 ? hist[hi] : 0, c0 = hi > 0 ? hist[hi - 1] : 0;
    int total;
    const int above = block_scan(c0 + c1, warp_sums, total);
    if (above < rem && rem <= above + c1) {
      found[0] = hi;
      found[1] = rem - above;
    } else if (above + c1 < rem && rem <= above + c1 + c0) {
      found[0] = hi - 1;
      found[1] = rem - above - c1;
    }
    __syncthreads();
    prefix |= static_cast<unsigned>(found[0]) << shift;
    mask |= static_cast<unsigned>(bins - 1) << shift;
    rem = found[1];
    __syncthreads();
  }
  // ordered list: every key above the rank's, the first `rem` of its equals
  int done = 0, ties = 0;
  for (int base = 0; base < n; base += kSelThreads) {
    const int i = base + threadIdx.x;
    const float x = i < n ? wt[i] : 0.f;
    const unsigned u = weight_key(x);
    const bool mid = i >= a && i < b;
    const bool tie = mid && need > 0 && u == prefix;
    bool take = i < n && (!mid || (need > 0 && u > prefix));
    int total;
    const int rank = block_scan(tie ? 1 : 0, warp_sums, total);
    if (tie && ties + rank < rem) take = true;
    ties += total;
    const int at = done + block_scan(take ? 1 : 0, warp_sums, total);
    if (take) {
      kept[at] = i;
      wt[at] = x;  // at <= i, and this tile's weights were read before the barriers above
    }
    done += total;
  }
}

// ---------------------------------------------------------------- eviction: the move
// Kept token i moves from place kept[i] >= i to place i, in order, within the same pages. A
// block owns 16 / kMoveParts of the 16-byte columns of one (stream, KV head)'s K or V and walks
// the list in tiles: a tile's sources are read before its places are written, and a later
// tile's sources lie behind them.
constexpr int kMoveThreads = 256;
constexpr int kMoveParts = 8;
constexpr int kMoveLanes = 16 / kMoveParts;            // lanes of one token
constexpr int kMoveTokens = kMoveThreads / kMoveLanes;  // tokens per step
constexpr int kMoveSteps = 8;

__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(const __grid_constant__ PagedEvictParams p) {
  const PagedView& w = p.view;
  int b = blockIdx.x;
  const int part = b % kMoveParts;
  b /= kMoveParts;
  const bool is_v = b & 1;
  b >>= 1;
  const int h = b % w.kv_heads, s = b / w.kv_heads;
  const int* kept = p.kept + static_cast<long long>(b) * p.keep;
  // tokens kept, and the first that moves: kept[i] - i never decreases, -1 only at the end
  int lo = 0, hi = p.keep;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (kept[m] >= 0) lo = m + 1; else hi = m;
  }
  const int count = lo;
  if (part == 0 && !is_v && h == 0 && threadIdx.x == 0) p.kv_len_out[s] = count;
  lo = 0;
  hi = count;
  while (lo < hi) {
    const int m = (lo + hi) >> 1;
    if (kept[m] == m) lo = m + 1; else hi = m;
  }
  const int first = lo;
  uint16_t* base = is_v ? w.v : w.k;
  const int lane = threadIdx.x % kMoveLanes, tok = threadIdx.x / kMoveLanes;
  const int c = (part * kMoveLanes + lane) * 8;
  const int pm = (1 << w.page_shift) - 1;
  for (int i0 = first; i0 < count; i0 += kMoveTokens * kMoveSteps) {
    uint4 x[kMoveSteps];
    bool have[kMoveSteps];
#pragma unroll
    for (int t = 0; t < kMoveSteps; ++t) {
      const int i = i0 + t * kMoveTokens + tok;
      have[t] = i < count;
      if (have[t]) {
        const int from = kept[i];
        const int id = paged_id(w, s, from >> w.page_shift);
        have[t] = id >= 0;
        if (id >= 0) x[t] = *reinterpret_cast<const uint4*>(base + paged_offset(w, id, h, from & pm) + c);
      }
    }
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kMoveSteps; ++t) {
      const int i = i0 + t * kMoveTokens + tok;
      if (have[t]) {
        const int id = paged_id(w, s, i >> w.page_shift);
        if (id >= 0) *reinterpret_cast<uint4*>(base + paged_offset(w, id, h, i & pm) + c) = x[t];
      }
    }
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_paged_write(const PagedWriteParams& p, cudaStream_t stream) {
  const int grid = (p.view.n_rows + kWriteWarps - 1) / kWriteWarps;
  paged_write_kernel<<<grid, kWriteWarps * 32, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_paged_evict(const PagedEvictParams& p, cudaStream_t stream) {
  const unsigned heads = static_cast<unsigned>(p.view.n_seqs) * p.view.kv_heads;
  paged_select_kernel<<<heads, kSelThreads, 0, stream>>>(p);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  paged_move_kernel<<<heads * 2 * kMoveParts, kMoveThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace rkv
