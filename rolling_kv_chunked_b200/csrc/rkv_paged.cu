// The paged cache's data movement: the write of a chunk into pages and eviction by weight.
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>

#include "paged.cuh"
#include "ptx_warp.cuh"

namespace rkv {
namespace {

// ---------------------------------------------------------------- write
// One warp per chunk row; 16 lanes move one head vector of K and V (16 bytes each), four pairs of heads on
// their way at once.
constexpr int kWriteWarps = 4;
constexpr int kWriteBatch = 4;

__global__ void __launch_bounds__(kWriteWarps * 32) paged_write_kernel(const __grid_constant__ PagedWriteParams p) {
  const PagedView& w = p.view;
  ptx::let_next_launch();
  ptx::wait_previous();
  const int row = blockIdx.x * kWriteWarps + (threadIdx.x >> 5);
  if (row >= w.n_rows) return;
  const int s = paged_seq_of_row(w, row);
  if (s < 0) return;
  const PagedSeq q = paged_seq(w, s);
  const int lane = threadIdx.x & 31;
  const int at = row - q.q0;  // the search finds another stream's range where q_start decreases
  const int pos = q.kv - q.n_q + at;
  if (!q.ok || at < 0 || at >= q.n_q) {
    if (lane == 0) paged_report(w, kStatusLength);
    return;
  }
  if (pos < 0) return;  // a chunk longer than its stream: this row has no place
  const int id = paged_id(w, s, pos >> w.page_shift);
  if (id < 0) return;
  const int slot = pos & ((1 << w.page_shift) - 1);
  const int c = (lane & 15) * 8;
  for (int h0 = lane >> 4; h0 < w.kv_heads; h0 += 2 * kWriteBatch) {
    uint4 kx[kWriteBatch], vx[kWriteBatch];
#pragma unroll
    for (int i = 0; i < kWriteBatch; ++i) {
      const int h = h0 + 2 * i;
      if (h < w.kv_heads) {
        kx[i] = *reinterpret_cast<const uint4*>(p.k + row * p.k_stride + h * kHeadDim + c);
        vx[i] = *reinterpret_cast<const uint4*>(p.v + row * p.v_stride + h * kHeadDim + c);
      }
    }
#pragma unroll
    for (int i = 0; i < kWriteBatch; ++i) {
      const int h = h0 + 2 * i;
      if (h < w.kv_heads) {
        const long long to = paged_offset(w, id, h, slot) + c;
        *reinterpret_cast<uint4*>(w.k + to) = kx[i];
        *reinterpret_cast<uint4*>(w.v + to) = vx[i];
      }
    }
  }
}

// ---------------------------------------------------------------- eviction: the choice
// Weights as unsigned numbers of the same order: NaN lowest, -0 equal to +0.
__device__ __forceinline__ unsigned weight_key(float x) {
  if (x != x) return 0u;
  const unsigned u = __float_as_uint(x + 0.0f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// A cluster of up to eight blocks chooses for one (stream, KV head). The weights are cut into equal runs,
// one per warp of the cluster, in order; a lane holds its keys in registers (up to kHeldKeys; longer
// streams are read from L2 again in every pass). The weight of rank `need` among the middle tokens is
// found digit by digit (11, 11 and 10 bits of the ordered key: the first digit holds the exponent and
// two bits of the fraction, so that equal digits, which collide in shared memory, are few): each block
// counts its digits, after one cluster barrier every block adds up the histograms through
// distributed shared memory and finds the digit for itself. Then each warp counts its kept tokens,
// one more exchange gives every warp its place in the list, and the warps write their parts without
// meeting again.
// Measured, one stream of 65536 tokens and eight heads: 154 us with one block per head; in cycles of the
// cluster form, per digit: counting 1000, the barrier 1650, the histograms 2100 (16 bytes a clock through
// distributed shared memory: the held form therefore packs two counts to a word), finding 600.
// Blocks have 1024 threads; many heads of short streams (to 4096 tokens) take 256, eight to an SM.
constexpr int kSelCluster = 8;  // blocks of a cluster at most
constexpr int kHeldKeys = 16;
constexpr int kDigits = 2048;

// kHeld: every warp's run has at most 32 * kHeldKeys tokens, a block's then less than 65536.
template <int kSelThreads, bool kHeld>
__global__ void __launch_bounds__(kSelThreads) paged_select_kernel(const __grid_constant__ PagedEvictParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  // counts of the digits, by pass (a neighbour may still read the last pass's): two digits to a word if held,
  // else one; a thread looks at kOwn of them in a row
  constexpr int kSelWarps = kSelThreads / 32;
  constexpr int kOwn = kDigits / kSelThreads;
  constexpr int kWords = kHeld ? kOwn / 2 : kOwn;
  struct __align__(4 * kWords) Own {
    unsigned x[kWords];
  };
  __shared__ Own hist[3][kSelThreads];
  __shared__ int warp_sums[kSelWarps];
  __shared__ int found[2];
  __shared__ int2 counts[kSelWarps];  // kept above the rank's weight (or fixed), and its equals, by warp
  __shared__ int2 block_counts;
  const PagedView& w = p.view;
  const int size = static_cast<int>(cluster.num_blocks());
  const int rank = blockIdx.x % size, sh = blockIdx.x / size;
  const int s = sh / w.kv_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ptx::wait_previous();
  const int n = w.kv_len[s];
  int* kept = p.kept + static_cast<long long>(sh) * p.keep;
  const bool bad = n < 0 || n > w.max_kv;
  if (bad || n <= p.keep) {  // the same in the whole cluster
    if (bad && rank == 0 && threadIdx.x == 0) paged_report(w, kStatusLength);
    for (int i = rank * kSelThreads + threadIdx.x; i < p.keep; i += size * kSelThreads)
      kept[i] = !bad && i < n ? i : -1;
    return;
  }
  const float* wt = p.weight + static_cast<long long>(sh) * p.weight_stride;
  const int a = p.sinks, b = n - p.recent;  // the middle: sinks + recent <= keep < n
  const int need = p.keep - p.sinks - p.recent;
  // this warp's run of tokens
  const int run = ((n + size * kSelWarps - 1) / (size * kSelWarps) + 31) / 32 * 32;
  const int i0 = min(n, (rank * kSelWarps + warp) * run), i1 = min(n, i0 + run);

  unsigned held[kHeldKeys];
  if (kHeld) {
#pragma unroll
    for (int k = 0; k < kHeldKeys; ++k) {
      const int i = i0 + 32 * k + lane;
      held[k] = i < i1 ? weight_key(wt[i]) : 0u;
    }
  }
  // f(token, its key) for this lane's tokens, 32 tokens of the run at a time, in order
  auto each = [&](auto f) {
    if (kHeld) {
#pragma unroll
      for (int k = 0; k < kHeldKeys; ++k) {
        if (i0 + 32 * k >= i1) break;
        f(i0 + 32 * k + lane, held[k]);
      }
    } else {
#pragma unroll 8
      for (int i = i0; i < i1; i += 32) f(i + lane, i + lane < i1 ? weight_key(wt[i + lane]) : 0u);
    }
  };
  unsigned prefix = 0, mask = 0;
  int rem = need;
  for (int i = 0; i < 3; ++i)
    for (int k = 0; k < kWords; ++k) hist[i][threadIdx.x].x[k] = 0u;
  __syncthreads();
  if (need > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const unsigned top = pass == 2 ? 1023u : 2047u;
      unsigned* mine = hist[pass][0].x;
      each([&](int i, unsigned u) {
        if (i < i1 && i >= a && i < b && (u & mask) == prefix) {
          const unsigned digit = (u >> shift) & top;
          if (kHeld)
            atomicAdd(&mine[digit >> 1], (digit & 1) ? 0x10000u : 1u);
          else
            atomicAdd(&mine[digit], 1u);
        }
      });
      cluster.sync();
      // thread t's digits, counted from the top: kOwn (kSelThreads - 1 - t) and those above it
      const int own = kSelThreads - 1 - static_cast<int>(threadIdx.x);
      Own part[kSelCluster];
#pragma unroll
      for (int r = 0; r < kSelCluster; ++r)  // all on their way at once; a smaller cluster reads some twice
        part[r] = cluster.map_shared_rank(hist[pass], min(r, size - 1))[own];
      int bins[kOwn], sum = 0;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        bins[i] = 0;
#pragma unroll
        for (int r = 0; r < kSelCluster; ++r) {
          const unsigned v = kHeld ? (i & 1 ? part[r].x[i / 2] >> 16 : part[r].x[i / 2] & 0xffffu) : part[r].x[i % kWords];
          bins[i] += r < size ? static_cast<int>(v) : 0;
        }
        sum += bins[i];
      }
      int inc = sum;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += y;
      }
      if (lane == 31) warp_sums[warp] = inc;
      __syncthreads();
      int above = inc - sum + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sums[lane] : 0);
#pragma unroll
      for (int i = kOwn - 1; i >= 0; --i) {
        if (above < rem && rem <= above + bins[i]) {
          found[0] = kOwn * own + i;
          found[1] = rem - above;
        }
        above += bins[i];
      }
      __syncthreads();
      prefix |= static_cast<unsigned>(found[0]) << shift;
      mask |= top << shift;
      rem = found[1];
    }
  }
  // every key above the rank's is kept, and the first `rem` of its equals
  auto look = [&](int i, unsigned u, bool& take, bool& tie) {
    const bool mid = i >= a && i < b;
    take = i < i1 && (!mid || (need > 0 && u > prefix));
    tie = i < i1 && mid && need > 0 && u == prefix;
  };
  int n_take = 0, n_tie = 0;
  each([&](int i, unsigned u) {
    bool take, tie;
    look(i, u, take, tie);
    n_take += take;
    n_tie += tie;
  });
  n_take = __reduce_add_sync(0xffffffffu, n_take);
  n_tie = __reduce_add_sync(0xffffffffu, n_tie);
  if (lane == 0) counts[warp] = make_int2(n_take, n_tie);
  __syncthreads();
  const int2 mine = lane < kSelWarps ? counts[lane] : make_int2(0, 0);
  int2 before;
  before.x = __reduce_add_sync(0xffffffffu, lane < warp ? mine.x : 0);
  before.y = __reduce_add_sync(0xffffffffu, lane < warp ? mine.y : 0);
  if (warp == 0) {
    const int all_x = __reduce_add_sync(0xffffffffu, mine.x), all_y = __reduce_add_sync(0xffffffffu, mine.y);
    if (lane == 0) block_counts = make_int2(all_x, all_y);
  }
  cluster.sync();
  int2 neighbour = make_int2(0, 0);  // lane r: the counts of block r, if it comes before this one
  if (lane < rank) neighbour = *cluster.map_shared_rank(&block_counts, lane);
  cluster.barrier_arrive();  // no block leaves while a neighbour may read its counts
  before.x += __reduce_add_sync(0xffffffffu, neighbour.x);
  before.y += __reduce_add_sync(0xffffffffu, neighbour.y);
  // only now: the next kernel's blocks would settle on the SMs that this one leaves free, and a few heads'
  // move would stay there (one stream, eight heads, its pages in L2: 56 us instead of 50)
  ptx::let_next_launch();
  int ties = before.y;                       // equals of the rank's weight before this token
  int at = before.x + min(before.y, rem);    // kept before this token
  const unsigned below = (1u << lane) - 1u;
  each([&](int i, unsigned u) {
    bool take, tie;
    look(i, u, take, tie);
    const unsigned tied = __ballot_sync(0xffffffffu, tie);
    if (tie && ties + __popc(tied & below) < rem) take = true;
    ties += __popc(tied);
    const unsigned taken = __ballot_sync(0xffffffffu, take);
    if (take) kept[at + __popc(taken & below)] = i;
    at += __popc(taken);
  });
  cluster.barrier_wait();
}

// ---------------------------------------------------------------- eviction: the move
// Kept token i moves from place kept[i] >= i to place i, in order, within the same pages: a stable
// compaction in place. The 256 bytes of a token are cut into two columns that never meet (128 bytes, a
// line: columns of 32 bytes were bound by the lines that a warp's access touches), so
// (stream, KV head, K or V, column) are independent blocks, each walking the list in tiles: a tile's
// sources have been read by all before its places are written, and later tiles' sources lie behind
// them, so two more tiles are on their way (cp.async into shared memory, each thread's 16 bytes its
// own) while one is written. A cluster of blocks shares a tile's tokens where there are few heads. List entries and page ids are fetched ahead in registers: with a tile's
// three dependent loads (entry, page id, data) in one row a tile took 3.6 us. One more block per
// (stream, KV head) moves the weights.
// On pages that are not in L2 the move takes 57 us for 65536 tokens of eight heads to 16384 and for 16 streams of
// eight heads to 4096 each alike (134 and 201 MB, 20 and 31 us of HBM): bound by the tiles' turns, each a wait of the
// whole cluster for its slowest load.
constexpr int kMoveThreads = 256;
constexpr int kMoveSteps = 4;   // 16-byte pieces of a tile per thread
constexpr int kMoveAhead = 2;   // tiles in flight beside the one written
constexpr int kMoveSmem = (kMoveAhead + 1) * kMoveSteps * kMoveThreads * 16;

struct MoveList {
  int first, count;
};

// Tokens kept, and the first that moves: kept[i] - i never decreases, -1 stands only at the end. The whole
// block probes at once: two rounds for lists up to 262144, where a search by halves waits
// for 2 log2(keep) loads in a row (10 us of the kernel's time at 16384).
__device__ __forceinline__ MoveList move_list(const int* kept, int keep) {
  int lo0 = 0, hi0 = keep, lo1 = 0, hi1 = keep;  // the count, the first that moves: in [lo, hi]
  const int t = threadIdx.x;
  while (lo0 < hi0 || lo1 < hi1) {
    const int step0 = (hi0 - lo0 + kMoveThreads - 1) / kMoveThreads, step1 = (hi1 - lo1 + kMoveThreads - 1) / kMoveThreads;
    const int i0 = lo0 + t * step0, i1 = lo1 + t * step1;
    const bool there = step0 > 0 && i0 < hi0 && kept[i0] >= 0;
    const bool stays = step1 > 0 && i1 < hi1 && kept[i1] == i1;
    const int c0 = __syncthreads_count(there), c1 = __syncthreads_count(stays);
    // c probes hold: the border lies behind the last of them, up to the next probe
    hi0 = c0 == 0 ? lo0 : min(hi0, lo0 + c0 * step0);
    lo0 = c0 == 0 ? lo0 : lo0 + (c0 - 1) * step0 + 1;
    hi1 = c1 == 0 ? lo1 : min(hi1, lo1 + c1 * step1);
    lo1 = c1 == 0 ? lo1 : lo1 + (c1 - 1) * step1 + 1;
  }
  MoveList r;
  r.count = lo0;
  r.first = min(lo1, lo0);
  return r;
}

constexpr int kMoveParts = 2;                          // columns of a token
constexpr int kMoveLanes = 16 / kMoveParts;             // lanes of one token, 16 bytes each
constexpr int kMoveTokens = kMoveThreads / kMoveLanes;  // tokens per step
constexpr int kMoveCluster = 8;                         // blocks of a cluster at most

__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(const __grid_constant__ PagedEvictParams p) {
  namespace cg = cooperative_groups;
  cg::cluster_group cluster = cg::this_cluster();
  const int size = static_cast<int>(cluster.num_blocks()), rank = blockIdx.x % size;
  const PagedView& w = p.view;
  const int heads = w.n_seqs * w.kv_heads;
  const int task = blockIdx.x / size / heads, b = blockIdx.x / size % heads;
  const int h = b % w.kv_heads, s = b / w.kv_heads;
  const int* kept = p.kept + static_cast<long long>(b) * p.keep;
  ptx::wait_previous();
  const MoveList m = move_list(kept, p.keep);
  if (task == 2 * kMoveParts) {
    if (rank != 0) return;
    if (h == 0 && threadIdx.x == 0) p.kv_len_out[s] = m.count;
    float* wt = p.weight + static_cast<long long>(b) * p.weight_stride;
    for (int i0 = m.first; i0 < m.count; i0 += kMoveThreads * 8) {
      float x[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int i = i0 + t * kMoveThreads + threadIdx.x;
        if (i < m.count) x[t] = wt[kept[i]];
      }
      __syncthreads();
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int i = i0 + t * kMoveThreads + threadIdx.x;
        if (i < m.count) wt[i] = x[t];
      }
      __syncthreads();
    }
    return;
  }
  extern __shared__ uint4 pieces[];  // [tile][step][thread]
  uint16_t* base = task >= kMoveParts ? w.v : w.k;
  const int tok = threadIdx.x / kMoveLanes;
  const int c = ((task % kMoveParts) * kMoveLanes + threadIdx.x % kMoveLanes) * 8;
  const int pm = (1 << w.page_shift) - 1;
  constexpr int kTileTokens = kMoveTokens * kMoveSteps;  // this block's share of a tile
  const int n_tiles = (m.count - m.first + size * kTileTokens - 1) / (size * kTileTokens);
  if (n_tiles == 0) return;
  auto place = [&](int tile, int t) {
    return m.first + (tile * size + rank) * kTileTokens + t * kMoveTokens + tok;
  };
  auto entry = [&](int tile, int t) {
    const int i = place(tile, t);
    return i < m.count ? kept[i] : -1;
  };
  // the list's raw entry (-1 where there is no token): checked where it is used, a whole tile after
  // its load was issued
  const int* table = w.table + static_cast<long long>(s) * w.table_stride;
  auto page = [&](int j) { return j >= 0 ? table[j >> w.page_shift] : -1; };
  auto checked = [&](int id, bool live) {
    if (static_cast<unsigned>(id) < static_cast<unsigned>(w.n_pages)) return id;
    if (live) paged_report(w, kStatusPage);
    return -1;
  };
  // a tile is written where its source page and its own page are pages of the pool
  unsigned good = 0;  // bit tile % 8 * 4 + step: fetched
  auto mark = [&](int tile, int t, bool ok) {
    const unsigned bit = 1u << ((tile & 7) * kMoveSteps + t);
    good = ok ? good | bit : good & ~bit;
  };
  auto fetch = [&](int tile, int t, int raw, int from) {
    const int id = checked(raw, from >= 0);
    mark(tile, t, id >= 0);
    if (id >= 0)
      ptx::cp_async16(ptx::smem_u32(pieces + ((tile % (kMoveAhead + 1)) * kMoveSteps + t) * kMoveThreads + threadIdx.x),
                      base + paged_offset(w, id, h, from & pm) + c);
  };
#pragma unroll
  for (int tile = 0; tile < kMoveAhead; ++tile) {
#pragma unroll
    for (int t = 0; t < kMoveSteps; ++t) {
      const int from = entry(tile, t);
      fetch(tile, t, page(from), from);
    }
    ptx::cp_async_commit();
  }
  int ahead[kMoveSteps], from[kMoveSteps], src[kMoveSteps], dst[kMoveSteps];
#pragma unroll
  for (int t = 0; t < kMoveSteps; ++t) {
    from[t] = entry(kMoveAhead, t);
    src[t] = page(from[t]);
    ahead[t] = entry(kMoveAhead + 1, t);
    dst[t] = page(place(0, t) < m.count ? place(0, t) : -1);
  }
  ptx::cp_async_wait<kMoveAhead - 1>();
  cluster.barrier_arrive();  // this block has read its share of tile 0
  for (int tile = 0; tile < n_tiles; ++tile) {
    int to[kMoveSteps];
#pragma unroll
    for (int t = 0; t < kMoveSteps; ++t) {
      fetch(tile + kMoveAhead, t, src[t], from[t]);
      from[t] = ahead[t];
      src[t] = page(from[t]);
      ahead[t] = entry(tile + kMoveAhead + 2, t);
      to[t] = dst[t];
      const int i = place(tile + 1, t);
      dst[t] = page(i < m.count ? i : -1);
    }
    ptx::cp_async_commit();
    cluster.barrier_wait();  // the tile was read by all
#pragma unroll
    for (int t = 0; t < kMoveSteps; ++t) {
      const bool got = good >> ((tile & 7) * kMoveSteps + t) & 1u;
      const int id = checked(to[t], got);
      if (got && id >= 0)
        *reinterpret_cast<uint4*>(base + paged_offset(w, id, h, place(tile, t) & pm) + c) =
            pieces[((tile % (kMoveAhead + 1)) * kMoveSteps + t) * kMoveThreads + threadIdx.x];
    }
    ptx::cp_async_wait<kMoveAhead - 1>();
    cluster.barrier_arrive();  // the next one's share was read
  }
  cluster.barrier_wait();
  ptx::cp_async_wait<0>();
}

// the dynamic shared-memory limit is a per-device setting, made once on every device this process
// launches on
cudaError_t configure() {
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static bool done[kMaxDevices] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev]) return cudaSuccess;
  err = cudaFuncSetAttribute(paged_move_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoveSmem);
  if (err == cudaSuccess) done[dev] = true;
  return err;
}

}  // namespace

cudaError_t launch_paged_write(const PagedWriteParams& p, cudaStream_t stream) {
  const int grid = (p.view.n_rows + kWriteWarps - 1) / kWriteWarps;
  return launch_after(paged_write_kernel, grid, kWriteWarps * 32, 0, stream, p);
}

cudaError_t launch_paged_evict(const PagedEvictParams& p, cudaStream_t stream) {
  const unsigned heads = static_cast<unsigned>(p.view.n_seqs) * p.view.kv_heads;
  // Blocks per cluster: as many as keep one block of 1024 threads to an SM, each with at least 2048 tokens of the
  // longest stream. Where one block already has less than that and there are more heads than SMs, 256 threads
  // (440 heads of 556 tokens: 17 us with 1024, three waves).
  const bool small = heads > kSmCount && p.view.max_kv <= 256 * kHeldKeys;
  unsigned size = kSelCluster;
  while (size > 1 && (heads * size > kSmCount || static_cast<unsigned>(p.view.max_kv) < 2048u * size)) size /= 2;
  const int threads = small ? 256 : 1024;
  const long long piece = static_cast<long long>(size) * (threads / 32);
  const bool held = (p.view.max_kv + piece - 1) / piece <= 32 * kHeldKeys;
  cudaError_t err = configure();
  if (err != cudaSuccess) return err;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(heads * size);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  err = cudaLaunchKernelEx(&cfg, small ? paged_select_kernel<256, true> : held ? paged_select_kernel<1024, true>
                                                                               : paged_select_kernel<1024, false>, p);
  if (err != cudaSuccess) return err;
  // blocks that share a column: up to eight, while the grid stays near three blocks to an SM
  size = kMoveCluster;
  while (size > 1 && heads * 2 * kMoveParts * size > 1024) size /= 2;
  attr[0].val.clusterDim.x = size;
  cfg.gridDim = dim3(heads * (2 * kMoveParts + 1) * size);
  cfg.blockDim = dim3(kMoveThreads);
  // no more tiles in shared memory than the longest list has
  const long long tiles = (p.keep + static_cast<long long>(size) * kMoveTokens * kMoveSteps - 1) / (size * kMoveTokens * kMoveSteps);
  cfg.dynamicSmemBytes = static_cast<size_t>(std::min<long long>(tiles, kMoveAhead + 1)) * kMoveSteps * kMoveThreads * 16;
  return cudaLaunchKernelEx(&cfg, paged_move_kernel, p);
}

}  // namespace rkv
