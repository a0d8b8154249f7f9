// Attention of a chunk's rows over a paged cache on tcgen05, and the attention weight that each
// cached token gathers.
//
// Rows of one KV head's group of G query heads are packed into tiles of 128: row r of a tile is
// token r / G, head r % G (128 / G whole tokens, loaded by one TMA box of G heads), so K and V are
// read once for the group. A block takes 256 rows (two tiles) of one stream and KV head and walks the
// pages; where a stream brings no more than 128 rows the two softmax warpgroups instead take
// every second key tile of the one query tile and merge at the end.
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
#include <mutex>

#include "attention_tile.cuh"
#include "paged.cuh"

namespace rkv {
namespace {

constexpr int kBM = 128;  // rows per query tile
constexpr int kBN = 128;  // tokens per key tile
constexpr int kThreads = 320;
constexpr int kSmemQ = 0;
constexpr int kSmemK = 2 * kTile;
constexpr int kSmemV = 4 * kTile;
constexpr int kSmemBar = 6 * kTile;
constexpr int kSmemBytes = 6 * kTile + 256 + 1024;
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
  kBarVFix = 15,   // the last tile's stale V rows were zeroed
  kNumBars = 16
};

__device__ __forceinline__ constexpr uint32_t col_s(int t) { return static_cast<uint32_t>(t) * 128u; }
__device__ __forceinline__ constexpr uint32_t col_o(int t) { return 256u + static_cast<uint32_t>(t) * 128u; }
constexpr uint32_t kIdescS = ptx::idesc_bf16_f32(kBM, kBN, false);
constexpr uint32_t kIdescPV = ptx::idesc_bf16_f32(kBM, kHeadDim, true);

// The block of chunk tokens that index b names, counted from the batch's last stream and its last
// block down (under a causal mask a stream's last block sees most keys, so the long ones start
// first). A whole warp calls it; returns false past the last block.
__device__ __forceinline__ bool find_block(const PagedView& w, int b, int block_tokens, int& s, int& blk) {
  const int lane = threadIdx.x & 31;
  int before = 0;
  for (int base = w.n_seqs - 1; base >= 0; base -= 32) {
    const int i = base - lane;
    int c = 0;
    if (i >= 0) {
      const PagedSeq q = paged_seq(w, i);
      if (q.ok) c = (q.n_q + block_tokens - 1) / block_tokens;
      else paged_report(w, kStatusLength);
    }
    int inc = c;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, before + inc > b);
    if (hit) {
      const int l = __ffs(hit) - 1;
      s = base - l;
      blk = __shfl_sync(0xffffffffu, before + inc, l) - 1 - b;
      return true;
    }
    before += __shfl_sync(0xffffffffu, inc, 31);
  }
  return false;
}

// 2^x on the FMA pipe for two lanes: r = round(x) by adding 1.5 * 2^23, f = x - r in [-1/2, 1/2], a
// polynomial for 2^f fitted for least relative error (tests/exp2_poly.py; degree 4: 2.7e-6, mean
// 4e-8, which keeps a row sum within fp32's own rounding; degree 5: 2.3e-7), r added to the exponent.
// x is clamped to [-125, 126].
template <int kDegree>
__device__ __forceinline__ void exp2_poly(uint64_t x2, float& y0, float& y1) {
  float x0, x1;
  ptx::f2_unpack(x2, x0, x1);
  const uint64_t x = ptx::f2_pack(fminf(fmaxf(x0, -125.0f), 126.0f), fminf(fmaxf(x1, -125.0f), 126.0f));
  const uint64_t t = ptx::f2_add(x, ptx::f2_pack(12582912.0f, 12582912.0f));
  const uint64_t r = ptx::f2_add(t, ptx::f2_pack(-12582912.0f, -12582912.0f));
  const uint64_t f = ptx::f2_fma(r, ptx::f2_pack(-1.0f, -1.0f), x);
  auto two = [](float c) { return ptx::f2_pack(c, c); };
  uint64_t q;
  if (kDegree == 5) {
    q = ptx::f2_fma(two(0.0013276471519076234f), f, two(0.00967554133066553f));
    q = ptx::f2_fma(q, f, two(0.05550713274962234f));
    q = ptx::f2_fma(q, f, two(0.24022119723934193f));
    q = ptx::f2_fma(q, f, two(0.693146967063863f));
    q = ptx::f2_fma(q, f, two(1.000000071654653f));
  } else {
    q = ptx::f2_fma(two(0.009570101434034835f), f, two(0.055917860281963716f));
    q = ptx::f2_fma(q, f, two(0.2402474483964632f));
    q = ptx::f2_fma(q, f, two(0.6931218147436669f));
    q = ptx::f2_fma(q, f, two(0.9999992614421643f));
  }
  float t0, t1, q0, q1;
  ptx::f2_unpack(t, t0, t1);
  ptx::f2_unpack(q, q0, q1);
  y0 = __uint_as_float((__float_as_uint(t0) << 23) + __float_as_uint(q0));
  y1 = __uint_as_float((__float_as_uint(t1) << 23) + __float_as_uint(q1));
}

constexpr int kPolyPairs = 2;  // of every 8 pairs of an unmasked tile

// 64 numerators 2^(s sl2 - m) of one row, packed to bf16 pairs (the operand type of the product
// with V; half a step, 2^-8, of each), their unrounded sum in acc.
template <bool kPoly>
__device__ __forceinline__ void numerators(const uint32_t* sh, uint64_t c2, uint64_t nm2, uint32_t* pk,
                                           uint64_t (&acc)[4]) {
#pragma unroll
  for (int k = 0; k < kBN / 4; ++k) {
    const uint64_t x = ptx::f2_fma(ptx::f2_pack(__uint_as_float(sh[2 * k]), __uint_as_float(sh[2 * k + 1])), c2, nm2);
    float a, b;
    if (kPoly && (k & 7) < kPolyPairs) {
      exp2_poly<4>(x, a, b);
    } else {
      float x0, x1;
      ptx::f2_unpack(x, x0, x1);
      a = ptx::ex2(x0);
      b = ptx::ex2(x1);
    }
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
        numerators<true>(sh, c2, nm2, pk + 32 * hh, acc);
      } else {
#pragma unroll
        for (int i = 0; i < kBN / 2; ++i)
          if (64 * hh + i >= valid) sh[i] = 0xff800000u;
        numerators<false>(sh, c2, nm2, pk + 32 * hh, acc);
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
        numerators<true>(sh, c2, nm2, pk, acc);
      } else {
#pragma unroll
        for (int i = 0; i < kBN / 2; ++i)
          if (64 * hh + i >= valid) sh[i] = 0xff800000u;
        numerators<false>(sh, c2, nm2, pk, acc);
      }
      ptx::tmem_st32(tS + 32 * hh, pk);
    }
    l += sum_of(acc);
  }
}

__global__ void __launch_bounds__(kThreads, 1)
    paged_chunk_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ PagedAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kSmemBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kNumBars);
  int* found = reinterpret_cast<int*>(bars + kNumBars + 1);
  const PagedView& w = p.view;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned long long limit = p.wait_limit_ns;

  const int sp = blockIdx.x % p.n_split;
  const int u = blockIdx.x / p.n_split;
  const int h = u / p.n_blocks;
  if (warp == 0) {
    int s = -1, blk = 0;
    if (!find_block(w, u - h * p.n_blocks, p.block_tokens, s, blk)) s = -1;
    if (lane == 0) {
      found[0] = s;
      found[1] = blk;
    }
  } else if (threadIdx.x == 32) {
    ptx::mbar_init(&bars[kBarQ], 1);
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
  }
  __syncthreads();
  const int s = found[0], blk = found[1];
  if (s < 0) return;
  const PagedSeq q = paged_seq(w, s);
  const int G = p.group;
  const int tpt = kBM / G;                 // tokens of a query tile
  const int i0 = blk * p.block_tokens;     // the block's first chunk token
  const int cnt = min(p.block_tokens, q.n_q - i0);
  const bool two = cnt > tpt;
  const int keys = p.causal ? max(0, q.kv - q.n_q + i0 + cnt) : q.kv;  // seen by the block's last row
  const int j0 = sp * p.split_keys;
  if (j0 >= keys && (sp > 0 || p.n_split > 1)) return;
  const int j1 = min(keys, j0 + p.split_keys);
  const int n_tiles = (j1 - j0 + kBN - 1) / kBN;  // 0 only when the rows see nothing at all
  const int last_valid = j1 - j0 - (n_tiles - 1) * kBN;

  if (warp == 9) {
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

  if (warp == 8) {
    // ------------------------------------------------------------ TMA producer
    bool ok = true;
    int nk = 0, nv = 0;
    if (n_tiles > 0) {
      const int box = min(1 << w.page_shift, kBN);  // tokens per copy
      const int n_box = kBN / box;
      const int b = lane % n_box, c = (lane / n_box) & 1;
      const bool is_v = (lane / n_box) & 2, mine = lane < 4 * n_box;
      const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
      uint8_t* dst = smem + (is_v ? kSmemV : kSmemK) + c * kSlab + b * box * 128;
      if (lane == 0) {
        ptx::prefetch_tmap(&tm_k);
        ptx::prefetch_tmap(&tm_v);
        ptx::mbar_arrive_expect_tx(&bars[kBarQ], (two ? 2 : 1) * 2 * 128 * tpt * G);
        for (int t = 0; t < (two ? 2 : 1); ++t)
          for (int cc = 0; cc < 2; ++cc)
            ptx::tma_load_3d(smem + kSmemQ + t * kTile + cc * kSlab, &tm_q, &bars[kBarQ], cc * 64, h * G,
                             q.q0 + i0 + t * tpt);
      }
      int id = -1;
      if (mine && j0 + b * box < j1) id = paged_id(w, s, (j0 + b * box) >> w.page_shift);
      for (int t = 0; t < n_tiles; ++t) {
        const int st = t & 1;
        const int j = j0 + t * kBN + b * box;
        const int page = max(id, 0);
        if (mine && j + kBN < j1) id = paged_id(w, s, (j + kBN) >> w.page_shift);
        const int bytes = (min(kBN, j1 - j0 - t * kBN) + box - 1) / box * box * 256;
        const int row = (h << w.page_shift) + (j & ((1 << w.page_shift) - 1));
        if (t >= 2) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kBarKEmpty + st], ((t - 2) >> 1) & 1, limit));
          if (!ok) break;
        }
        if (lane == 0) ptx::mbar_arrive_expect_tx(&bars[kBarKFull + st], bytes);
        __syncwarp();
        if (mine && !is_v && j < j1) ptx::tma_load_3d(dst + st * kTile, tm, &bars[kBarKFull + st], c * 64, row, page);
        nk = t + 1;
        if (t >= 2) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kBarVEmpty + st], ((t - 2) >> 1) & 1, limit));
          if (!ok) break;
        }
        if (lane == 0) ptx::mbar_arrive_expect_tx(&bars[kBarVFull + st], bytes);
        __syncwarp();
        if (mine && is_v && j < j1) ptx::tma_load_3d(dst + st * kTile, tm, &bars[kBarVFull + st], c * 64, row, page);
        nv = t + 1;
      }
      // the last tile's V rows from the last visible token to the end of its step of 16
      if (ok && (last_valid & 15)) {
        const int t = n_tiles - 1;
        ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kBarVFull + (t & 1)], (t >> 1) & 1, limit));
        if (ok) {
          const int end = (last_valid + 15) & ~15;
          for (int i = lane; i < (end - last_valid) * 16; i += 32)
            *reinterpret_cast<uint4*>(smem + kSmemV + (t & 1) * kTile + ((i >> 3) & 1) * kSlab +
                                      (last_valid + (i >> 4)) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
          ptx::fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(&bars[kBarVFix]);
        }
      }
      if (lane == 0) {
        if (!ok) paged_report(w, kStatusTimeout);
        // every copy issued must land before the block may exit
        ptx::mbar_wait(&bars[kBarQ], 0, kDrainNs);
        for (int t = max(0, nk - 2); t < nk; ++t) ptx::mbar_wait(&bars[kBarKFull + (t & 1)], (t >> 1) & 1, kDrainNs);
        for (int t = max(0, nv - 2); t < nv; ++t) ptx::mbar_wait(&bars[kBarVFull + (t & 1)], (t >> 1) & 1, kDrainNs);
      }
    }
    __syncwarp();
  } else if (warp == 9) {
    // ------------------------------------------------------------ MMA issuer
    if (lane == 0 && n_tiles > 0) {
      const uint32_t q_addr[2] = {ptx::smem_u32(smem + kSmemQ), ptx::smem_u32(smem + kSmemQ + (two ? kTile : 0))};
      const uint32_t k_addr = ptx::smem_u32(smem + kSmemK);
      const uint32_t v_addr = ptx::smem_u32(smem + kSmemV);
      bool ok = ptx::mbar_wait(&bars[kBarQ], 0, limit);
      auto issue_s = [&](int t, uint32_t kt) {
#pragma unroll
        for (int kk = 0; kk < kHeadDim / 16; ++kk)
          ptx::mma_ss(tmem + col_s(t), desc_kmajor(q_addr[t], kk), desc_kmajor(kt, kk), kIdescS, kk > 0 ? 1u : 0u);
      };
      // V of tile j observed, the last one's stale rows zeroed
      auto wait_v = [&](int j) -> bool {
        if (!ptx::mbar_wait(&bars[kBarVFull + (j & 1)], (j >> 1) & 1, limit)) return false;
        return j + 1 < n_tiles || (last_valid & 15) == 0 || ptx::mbar_wait(&bars[kBarVFix], 0, limit);
      };
      // O_t += P_t V(j), the use-th of its accumulator; V(j) already observed
      auto issue_pv = [&](int t, int j, int use, bool frees_v) -> bool {
        if (!ptx::mbar_wait(&bars[kBarPFull + t], use & 1, limit)) return false;
        ptx::tc_fence_after();
        const uint32_t vt = v_addr + (j & 1) * kTile;
        const int steps = j + 1 < n_tiles ? kBN / 16 : (last_valid + 15) >> 4;
#pragma unroll
        for (int kk = 0; kk < kBN / 16; ++kk)
          if (kk < steps)
            ptx::mma_ts(tmem + col_o(t), tmem + col_s(t) + kk * 8, desc_v(vt, kk), kIdescPV,
                        (use > 0 || kk > 0) ? 1u : 0u);
        if (frees_v) ptx::mma_commit(&bars[kBarVEmpty + (j & 1)]);
        return true;
      };
      if (two) {
        // S0(j), PV1(j-1), S1(j), PV0(j): one warpgroup's softmax beside the other tile's products;
        // the waits on V(j) and K(j+1) are taken before the wait for P0(j), where this thread idles
        bool k_ready = ok && ptx::mbar_wait(&bars[kBarKFull], 0, limit);
        if (!k_ready) ok = false;
        for (int j = 0; ok && j < n_tiles; ++j) {
          const int st = j & 1;
          if (!k_ready && !ptx::mbar_wait(&bars[kBarKFull + st], (j >> 1) & 1, limit)) { ok = false; break; }
          ptx::tc_fence_after();
          const uint32_t kt = k_addr + st * kTile;
          issue_s(0, kt);
          ptx::mma_commit(&bars[kBarSFull + 0]);
          if (j > 0 && !issue_pv(1, j - 1, j - 1, true)) { ok = false; break; }
          issue_s(1, kt);
          ptx::mma_commit(&bars[kBarSFull + 1]);
          ptx::mma_commit(&bars[kBarKEmpty + st]);
          if (!wait_v(j)) { ok = false; break; }
          k_ready = j + 1 < n_tiles && ptx::mbar_try_wait(&bars[kBarKFull + (st ^ 1)], ((j + 1) >> 1) & 1);
          if (!issue_pv(0, j, j, false)) { ok = false; break; }
        }
        if (ok && !issue_pv(1, n_tiles - 1, n_tiles - 1, true)) ok = false;
      } else {
        // two chains over the one query tile: S(j) into buffer j & 1 while the other's softmax runs
        for (int j = 0; ok && j < n_tiles; ++j) {
          if (!ptx::mbar_wait(&bars[kBarKFull + (j & 1)], (j >> 1) & 1, limit)) { ok = false; break; }
          ptx::tc_fence_after();
          issue_s(j & 1, k_addr + (j & 1) * kTile);
          ptx::mma_commit(&bars[kBarSFull + (j & 1)]);
          ptx::mma_commit(&bars[kBarKEmpty + (j & 1)]);
          if (j > 0 && !(wait_v(j - 1) && issue_pv((j - 1) & 1, j - 1, (j - 1) >> 1, true))) ok = false;
        }
        if (ok && !(wait_v(n_tiles - 1) && issue_pv((n_tiles - 1) & 1, n_tiles - 1, (n_tiles - 1) >> 1, true))) ok = false;
      }
      if (ok) ptx::mma_commit(&bars[kBarODone]);
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
    const int tile0 = two ? wg * tpt : 0;  // this query tile's first token in the block
    const int tok = r / G;
    const bool live = r < min(tpt, cnt - tile0) * G;
    // the last place this row sees; rows of no token see what the block sees, so that they
    // hold no whole warp on the masked path
    const int last = p.causal && live ? q.kv - q.n_q + i0 + tile0 + tok : keys - 1;
    const int n_mine = two ? n_tiles : (n_tiles + 1 - wg) >> 1;
    float m_used = kNoKey, l = 0.f, pend = 1.0f;
    bool ok = true;
    for (int i = 0; i < n_mine; ++i) {
      const int t = two ? i : 2 * i + wg;
      ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kBarSFull + wg], i & 1, limit));
      if (!ok) break;
      ptx::tc_fence_after();
      softmax_tile(i == 0, min(j1, last + 1) - j0 - t * kBN, tS, tO, sl2, c2, m_used, l, pend);
      ptx::tmem_st_wait();
      ptx::tc_fence_before();
      ptx::mbar_arrive(&bars[kBarPFull + wg]);
    }
    if (ok && n_tiles > 0) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kBarODone], 0, limit));
    if (!ok && lane == 0) paged_report(w, kStatusTimeout);
    ptx::tc_fence_after();
    l *= pend;
    float f = pend, fo = 0.f;  // factors of this warpgroup's O and of the other's
    float* other = reinterpret_cast<float*>(smem) + r * kPartRow;
    if (!two) {
      // join the chains: the odd tiles' row goes through shared memory, free by now
      if (wg == 1) {
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t rr[32];
          ptx::tmem_ld32(tO + 32 * c, rr);
#pragma unroll
          for (int v = 0; v < 8; ++v)
            reinterpret_cast<float4*>(other + 32 * c)[v] =
                n_mine == 0 ? make_float4(0.f, 0.f, 0.f, 0.f)
                            : make_float4(__uint_as_float(rr[4 * v]), __uint_as_float(rr[4 * v + 1]),
                                          __uint_as_float(rr[4 * v + 2]), __uint_as_float(rr[4 * v + 3]));
        }
        reinterpret_cast<float4*>(other + 128)[0] = make_float4(m_used, l, pend, 0.f);
      }
      ptx::named_bar_sync(1, 256);
      if (wg == 0) {
        const float4 e = reinterpret_cast<const float4*>(other + 128)[0];
        const float m = fmaxf(m_used, e.x);
        const float fa = ptx::ex2(m_used - m), fb = ptx::ex2(e.x - m);
        f = pend * fa;
        fo = e.z * fb;
        l = l * fa + e.y * fb;
        m_used = m;
      }
    }
    if (ok && (two || wg == 0)) {
      const long long row = q.q0 + i0 + tile0 + tok;
      const int head = h * G + r - tok * G;
      const long long rh = row * p.q_heads + head;
      const bool parts = p.n_split > 1;
      const float inv = parts ? 1.0f : (l > 0.f ? 1.0f / l : 0.f);
      const long long at = static_cast<long long>(sp) * w.n_rows * p.q_heads + rh;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t rr[32];
        ptx::tmem_ld32(tO + 32 * c, rr);
        float x[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = n_tiles > 0 ? __uint_as_float(rr[i]) * f : 0.f;
        if (!two) {
#pragma unroll
          for (int v = 0; v < 8; ++v) {
            const float4 y = reinterpret_cast<const float4*>(other + 32 * c)[v];
            x[4 * v] += y.x * fo;
            x[4 * v + 1] += y.y * fo;
            x[4 * v + 2] += y.z * fo;
            x[4 * v + 3] += y.w * fo;
          }
        }
        if (!live) continue;
        if (parts) {
          float4* dst = reinterpret_cast<float4*>(p.part + at * kHeadDim + 32 * c);
#pragma unroll
          for (int v = 0; v < 8; ++v) dst[v] = make_float4(x[4 * v], x[4 * v + 1], x[4 * v + 2], x[4 * v + 3]);
        } else {
          uint32_t ob[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) ob[i] = pack_bf16x2(x[2 * i] * inv, x[2 * i + 1] * inv);
          uint4* dst = reinterpret_cast<uint4*>(p.out + row * p.out_stride + head * kHeadDim + 32 * c);
#pragma unroll
          for (int v = 0; v < 4; ++v) dst[v] = make_uint4(ob[4 * v], ob[4 * v + 1], ob[4 * v + 2], ob[4 * v + 3]);
        }
      }
      if (live && parts) {
        p.part_ml[at] = make_float2(m_used, l);
      } else if (live) {
        const float z = l > 0.f ? m_used + log2f(l) : -INFINITY;
        if (p.lse != nullptr) p.lse[rh] = z * kLn2;
        if (p.lse2 != nullptr) p.lse2[rh] = z;
      }
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 9) ptx::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------------------------
// Attention weight of chunks. With z the rows' log-sum-exp from the attention before, key j of KV
// head h gathers sum over the group's rows i that see it of 2^(s_ij - z_i). The product is
// taken transposed, S^T = K Q^T: a block owns 128 keys (the TMEM lanes) and walks the query tiles
// (128 columns), so that a key's sum stays in one thread's registers: no atomics, a fixed order. The
// two warpgroups take every second query tile and are added up at the end.
//   warp 8: TMA producer (the K tile once, query tiles into four stages), warp 9: MMA issuer;
//   four S buffers fill the TMEM, two per warpgroup, so the next product runs beside the exponentials,
//   which bound the kernel: 128 x 128 of them per tile against 8 MMA steps.
constexpr int kWStages = 4;
constexpr int kWSmemQ = kTile;
constexpr int kWSmemLse = kWSmemQ + kWStages * kTile;  // [4][128] floats: -z per row, by S buffer
constexpr int kWSmemBar = kWSmemLse + kWStages * kBM * 4;
constexpr int kWSmemBytes = kWSmemBar + 256 + 1024;
constexpr int kWPolyPairs = 2;

enum : int {
  kWbK = 0,
  kWbQFull = 1,    // +stage
  kWbQEmpty = 5,   // +stage
  kWbSFull = 9,    // +buffer
  kWbSEmpty = 13,  // +buffer
  kWbDrain = 17,
  kWbCount = 18
};

__global__ void __launch_bounds__(kThreads, 1)
    paged_weight_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                        const __grid_constant__ PagedAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* nz = reinterpret_cast<float*>(smem + kWSmemLse);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kWSmemBar);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + kWbCount);
  const PagedView& w = p.view;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned long long limit = p.wait_limit_ns;
  const int n_kt = (w.max_kv + kBN - 1) / kBN;
  const int kt = blockIdx.x % n_kt, sh = blockIdx.x / n_kt;
  const int h = sh % w.kv_heads, s = sh / w.kv_heads;
  const PagedSeq q = paged_seq(w, s);
  const int j0 = kt * kBN;
  if (!q.ok || q.n_q == 0 || j0 >= q.kv) return;  // a bad length was reported by the attention
  const int G = p.group;
  const int tpt = kBM / G;
  const int first_place = q.kv - q.n_q;  // place of the chunk's first token
  // query tiles from the first with a row that sees this tile's first key
  const int qt0 = p.causal ? max(0, j0 - first_place) / tpt : 0;
  const int n_qt = (q.n_q + tpt - 1) / tpt - qt0;

  if (threadIdx.x == 0) {
    ptx::mbar_init(&bars[kWbK], 1);
    for (int i = 0; i < kWStages; ++i) {
      ptx::mbar_init(&bars[kWbQFull + i], 1);
      ptx::mbar_init(&bars[kWbQEmpty + i], 1);
      ptx::mbar_init(&bars[kWbSFull + i], 1);
      ptx::mbar_init(&bars[kWbSEmpty + i], kBM);
    }
    ptx::mbar_init(&bars[kWbDrain], 1);
    ptx::fence_mbar_init();
  }
  if (warp == 9) {
    ptx::tmem_alloc(tmem_slot, 512);
    ptx::tmem_relinquish();
  }
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 8) {
    const int box = min(1 << w.page_shift, kBN);
    const int n_box = kBN / box;
    const int b = lane % n_box, c = lane / n_box;
    const int j = j0 + b * box;
    if (lane == 0) {
      ptx::prefetch_tmap(&tm_q);
      const int boxes = (min(kBN, q.kv - j0) + box - 1) / box;
      ptx::mbar_arrive_expect_tx(&bars[kWbK], boxes * box * 256);
    }
    __syncwarp();
    if (c < 2 && j < q.kv)
      ptx::tma_load_3d(smem + c * kSlab + b * box * 128, &tm_k, &bars[kWbK], c * 64,
                       (h << w.page_shift) + (j & ((1 << w.page_shift) - 1)),
                       max(0, paged_id(w, s, j >> w.page_shift)));
    __syncwarp();
    if (lane == 0) {
      bool ok = true;
      int nq = 0;
      for (int t = 0; t < n_qt; ++t) {
        const int st = t % kWStages;
        if (t >= kWStages && !ptx::mbar_wait(&bars[kWbQEmpty + st], (t / kWStages - 1) & 1, limit)) { ok = false; break; }
        ptx::mbar_arrive_expect_tx(&bars[kWbQFull + st], 2 * 128 * tpt * G);
        for (int cc = 0; cc < 2; ++cc)
          ptx::tma_load_3d(smem + kWSmemQ + st * kTile + cc * kSlab, &tm_q, &bars[kWbQFull + st], cc * 64, h * G,
                           q.q0 + (qt0 + t) * tpt);
        nq = t + 1;
      }
      if (!ok) paged_report(w, kStatusTimeout);
      ptx::mbar_wait(&bars[kWbK], 0, kDrainNs);
      for (int t = max(0, nq - kWStages); t < nq; ++t)
        ptx::mbar_wait(&bars[kWbQFull + t % kWStages], (t / kWStages) & 1, kDrainNs);
    }
    __syncwarp();
  } else if (warp == 9) {
    if (lane == 0) {
      const uint32_t ka = ptx::smem_u32(smem);
      bool ok = ptx::mbar_wait(&bars[kWbK], 0, limit);
      for (int t = 0; ok && t < n_qt; ++t) {
        const int st = t % kWStages;  // the query stage and the S buffer
        if (!ptx::mbar_wait(&bars[kWbQFull + st], (t / kWStages) & 1, limit)) { ok = false; break; }
        if (t >= kWStages && !ptx::mbar_wait(&bars[kWbSEmpty + st], (t / kWStages - 1) & 1, limit)) { ok = false; break; }
        ptx::tc_fence_after();
        const uint32_t qa = ptx::smem_u32(smem + kWSmemQ + st * kTile);
#pragma unroll
        for (int kk = 0; kk < kHeadDim / 16; ++kk)
          ptx::mma_ss(tmem + st * 128, desc_kmajor(ka, kk), desc_kmajor(qa, kk), kIdescS, kk > 0 ? 1u : 0u);
        ptx::mma_commit(&bars[kWbSFull + st]);
        ptx::mma_commit(&bars[kWbQEmpty + st]);
      }
      if (!ok) paged_report(w, kStatusTimeout);
      ptx::mma_commit(&bars[kWbDrain]);
      ptx::mbar_wait(&bars[kWbDrain], 0, kDrainNs);
    }
    __syncwarp();
  } else {
    const int wg = warp >> 2;
    const int r = threadIdx.x & 127;  // key of the tile, and the query row whose z this thread fetches
    const uint32_t lane_base = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint64_t c2 = ptx::f2_pack(p.scale_log2, p.scale_log2);
    // -z of row r of query tile t; rows of no token get -infinity, which makes their weight 0
    // (their scores are finite or are masked below)
    auto fetch = [&](int t) -> float {
      const int tok = (qt0 + t) * tpt + r / G;
      if (t >= n_qt || r >= tpt * G || tok >= q.n_q) return -INFINITY;
      return -p.lse2[static_cast<long long>(q.q0 + tok) * p.q_heads + h * G + r % G];
    };
    float next = fetch(wg);
    uint64_t acc[4] = {0, 0, 0, 0};
    bool ok = true;
    for (int t = wg; t < n_qt; t += 2) {
      const int st = t % kWStages;
      float* z = nz + st * kBM;
      z[r] = next;
      next = fetch(t + 2);
      // rows [lo, hi) of this tile are of the chunk and see this thread's key
      const int tok0 = (qt0 + t) * tpt;
      const int hi = min(tpt, q.n_q - tok0) * G;
      const int lo = p.causal ? max(0, j0 + r - first_place - tok0) * G : 0;
      const bool whole = __all_sync(0xffffffffu, lo == 0 && hi == kBM);
      if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&bars[kWbSFull + st], (t / kWStages) & 1, limit));
      ptx::named_bar_sync(1 + wg, kBM);  // the warpgroup's z are in place (and the buffer before last was read)
      if (!ok) continue;
      ptx::tc_fence_after();
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        uint32_t sh_[64];
        ptx::tmem_ld64(lane_base + st * 128 + hh * 64, sh_);
        if (hh == 1) {
          ptx::tc_fence_before();
          ptx::mbar_arrive(&bars[kWbSEmpty + st]);
        }
        const uint64_t* zz = reinterpret_cast<const uint64_t*>(z + hh * 64);
        if (whole) {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const uint64_t x = ptx::f2_fma(
                ptx::f2_pack(__uint_as_float(sh_[2 * k]), __uint_as_float(sh_[2 * k + 1])), c2, zz[k]);
            float a, e;
            if ((k & 7) < kWPolyPairs) {
              exp2_poly<5>(x, a, e);
            } else {
              ptx::f2_unpack(x, a, e);
              a = ptx::ex2(a);
              e = ptx::ex2(e);
            }
            acc[k & 3] = ptx::f2_add(acc[k & 3], ptx::f2_pack(a, e));
          }
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            const int i = hh * 64 + 2 * k;
            float a, e;
            ptx::f2_unpack(ptx::f2_fma(ptx::f2_pack(__uint_as_float(sh_[2 * k]), __uint_as_float(sh_[2 * k + 1])), c2,
                                       zz[k]), a, e);
            a = i >= lo && i < hi ? ptx::ex2(a) : 0.f;
            e = i + 1 >= lo && i + 1 < hi ? ptx::ex2(e) : 0.f;
            acc[k & 3] = ptx::f2_add(acc[k & 3], ptx::f2_pack(a, e));
          }
        }
      }
    }
    if (!ok && lane == 0) paged_report(w, kStatusTimeout);
    const float sum = sum_of(acc);
    float* half = nz;  // the z of every tile have been read once both warpgroups are here
    ptx::named_bar_sync(3, 256);
    if (wg == 1) half[r] = sum;
    ptx::named_bar_sync(3, 256);
    const int j = j0 + r;
    if (wg == 0 && ok && j < q.kv) {
      float* to = p.weight + (static_cast<long long>(s) * w.kv_heads + h) * p.weight_stride + j;
      *to = (j < first_place ? *to : 0.f) + (sum + half[r]);
    }
  }

  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  if (warp == 9) ptx::tmem_dealloc(tmem, 512);
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
  const cudaError_t err = configure();
  if (err != cudaSuccess) return err;
  const unsigned grid = static_cast<unsigned>(p.n_blocks) * p.view.kv_heads * p.n_split;
  paged_chunk_kernel<<<grid, kThreads, kSmemBytes, stream>>>(tm_q, tm_k, tm_v, p);
  return cudaGetLastError();
}

cudaError_t launch_paged_weight(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const PagedAttnParams& p,
                                cudaStream_t stream) {
  const cudaError_t err = configure();
  if (err != cudaSuccess) return err;
  const unsigned n_kt = (p.view.max_kv + kBN - 1) / kBN;
  const unsigned grid = n_kt * p.view.n_seqs * p.view.kv_heads;
  paged_weight_kernel<<<grid, kThreads, kWSmemBytes, stream>>>(tm_q, tm_k, p);
  return cudaGetLastError();
}

}  // namespace rkv
