// Attention over a paged cache when a stream brings few rows: at most 32 per KV head (a single token of
// grouped heads, a few drafted tokens).
//
// With R rows per KV head a cached token costs 512 bytes of K and V and 256 R multiply-adds: at 16 rows 16 flops
// a byte, which the warp-level matrix instructions (mma.sync m16n8k16, 16 rows at a time; one in 32 clocks
// per SM quarter here, 144 TFLOP/s in all) still outrun: the kernel is bound by HBM, and everything serves to
// keep loads in flight. (At 32 rows they are the bound, at 64 the kernel took 40 us where the tcgen05 kernel
// of rkv_paged_attention.cu takes 35: so far this form goes.) One warp issues TMA copies of 64-token tiles (K and V, one box per page and 64-column
// half) into three stages; four warps share a tile: kRowTiles of 16 rows times 4 / kRowTiles runs of tokens.
// Each runs its own softmax in registers, without meeting the others until the unit's end, where the runs'
// partial results are merged through shared memory. Two thread blocks fit an SM: six stages of 32 KB
// in flight.
//
// A unit of work is one stream and KV head. Lengths differ, so all units' tiles, stream after stream and head
// after head, are shared evenly by the 296 thread blocks that fit the card at once, each walking its share
// without a pause at unit borders; units that a border cuts are left as partial rows for
// paged_join_kernel. (Parts of a fixed length, a thread block each: 238 us for 48 streams of 49 to
// 16384 tokens and 101 us for one of 131071 at the length that suits both, 221 and 91 us at the one that
// suits each; shares of four tiles at least: 11 us for 1590 tokens where single tiles take 8.) Every thread block counts the tiles for itself: one probe of 32 lengths per warp step.
#include <mutex>

#include "numeric.cuh"
#include "paged.cuh"
#include "ptx_warp.cuh"

namespace rkv {
namespace {

constexpr int kTileKeys = kPagedDecodeTile;
constexpr int kHalf = kTileKeys * 128;  // bytes of one 64-column half of a tile
constexpr int kStageBytes = 4 * kHalf;  // K halves, V halves
constexpr int kStages = 3;
constexpr int kWarps = 4;               // consumer warps, 16 tokens of a tile each
constexpr int kDecodeThreads = (kWarps + 1) * 32;
constexpr int kMergeRows = kWarps;      // rows merged at a time, a warp each
constexpr int kSmemMerge = kStages * kStageBytes;                              // [warp][row][128] floats
constexpr int kSmemMl = kSmemMerge + kWarps * kMergeRows * kHeadDim * 4;       // [warp][row]: reference, sum
constexpr int kSmemDecodeBar = kSmemMl + 128 * 8;
constexpr int kDecodeSmem = kSmemDecodeBar + 128 + 1024;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;  // log2: the running reference follows a maximum only past this
constexpr float kNoKey = -1e30f;  // reference (log2) of a row that has seen no key
constexpr unsigned long long kDrainNs = 2000000000ull;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// A unit, or the part of one, of a thread block's share.
struct TokenUnit {
  PagedSeq q;
  int s, h;
  int t0, t1, tiles;  // its tiles, and the unit's
};

// The shares of all units' tiles, and one thread block's way through its own. Whole warps call these.
struct TokenWalk : PagedTiles<kTileKeys> {
  long long left;  // tiles still to walk
  PagedShares of;

  __device__ __forceinline__ void share(const PagedView& w) {
    count(w, blockIdx.x == 0);
    of.split(all, 2 * kSmCount);
  }
  // What the join has to do where share c starts: nothing unless this is the first border inside a unit.
  __device__ __forceinline__ PagedJoin join(int c) const {
    PagedJoin r = {};
    const long long first = of.start(c) - t;
    if (t == 0 || of.start(c - 1) > first) return r;
    r.row0 = q.q0;
    r.cnt = q.n_q;
    r.h = h;
    // the second slot of thread block c - 1, then the first slots of c, c + 1, ... as far as the unit goes
    r.slot0 = 2 * c - 1;
    r.step = 2;
    r.parts = of.owner(first + tiles - 1) - c + 2;
    return r;
  }
  __device__ __forceinline__ bool next(const PagedView& w, TokenUnit& u) {
    if (left <= 0) return false;
    u.q = q;
    u.s = s;
    u.h = h;
    u.t0 = t;
    u.t1 = static_cast<int>(min(static_cast<long long>(tiles), t + left));
    u.tiles = tiles;
    left -= u.t1 - t;
    t = 0;
    if (++h == w.kv_heads && left > 0) {
      h = 0;
      do {
        q = paged_seq(w, ++s);
        tiles = paged_seq_tiles<kTileKeys>(q);
      } while (tiles == 0);
    }
    return true;
  }
};

// One unit (or part) of a thread block's share, by the four consumer warps: kRowTiles tiles of 16 rows times
// 4 / kRowTiles runs of each tile's tokens. g: tiles consumed before it; ok: no wait has expired (a warp whose
// wait expires skips further work but still passes the barriers).
template <int kRowTiles>
__device__ __forceinline__ void token_unit(const PagedAttnParams& p, const TokenUnit& u, uint8_t* smem, uint64_t* full,
                                           uint64_t* empty, int& g, bool& ok) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kRuns = kWarps / kRowTiles;       // warps that share a row tile
  constexpr int kRun = kTileKeys / kRuns;         // tokens of a tile per warp
  const int row_tile = warp % kRowTiles, run0 = warp / kRowTiles * kRun;
  const int ra = row_tile * 16 + (lane >> 2), rb = ra + 8;  // this lane's two rows
  const int cq = (lane & 3) * 2;                            // and its pair of columns within 8
  const int tok_a = ra / p.group, tok_b = rb / p.group;
  // ldmatrix rows: K by token (lanes 8-15: the next 8 columns, 16-31: the next 8 tokens), V by token
  // (lanes 8-15: the next 8 tokens, 16-31: the next 8 columns)
  const int krow = run0 + (lane >> 4) * 8 + (lane & 7), kcol = (lane >> 3) & 1;
  const int vrow = run0 + ((lane >> 3) & 1) * 8 + (lane & 7), vcol = lane >> 4;
  const uint32_t sbase = ptx::smem_u32(smem);
  float* mo = reinterpret_cast<float*>(smem + kSmemMerge);
  float2* ml = reinterpret_cast<float2*>(smem + kSmemMl);
  const PagedSeq& q = u.q;
  const int rows = q.n_q * p.group;
  uint32_t qa[8][4];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = e ? rb : ra, tok = e ? tok_b : tok_a;
    const bool live = r < rows;
    const uint16_t* src = p.q + (q.q0 + (live ? tok : 0)) * p.q_stride + (u.h * p.group + r - tok * p.group) * kHeadDim;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      qa[kk][e] = live ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + cq) : 0u;
      qa[kk][2 + e] = live ? *reinterpret_cast<const uint32_t*>(src + kk * 16 + 8 + cq) : 0u;
    }
  }
  // the last place each row sees
  const int last_a = p.causal ? q.kv - q.n_q + tok_a : q.kv - 1;
  const int last_b = p.causal ? q.kv - q.n_q + tok_b : q.kv - 1;
  const int last_all = p.causal ? q.kv - q.n_q : q.kv - 1;
  // where their scores go (a pair of places each), if they are kept
  const long long score_a = (static_cast<long long>(q.q0 + tok_a) * p.q_heads + u.h * p.group + ra - tok_a * p.group) * p.score_stride + cq;
  const long long score_b = (static_cast<long long>(q.q0 + tok_b) * p.q_heads + u.h * p.group + rb - tok_b * p.group) * p.score_stride + cq;
  float o[16][4];
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  float ma = kNoKey, mb = kNoKey, la = 0.f, lb = 0.f;  // references (log2) and this lane's sums
  for (int t = u.t0; t < u.t1; ++t, ++g) {
    const int st = g % kStages;
    if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(&full[st], (g / kStages) & 1, p.wait_limit_ns));
    if (!ok) continue;
    const uint32_t kt = sbase + st * kStageBytes, vt = kt + 2 * kHalf;
    const int jw = t * kTileKeys + run0;  // this warp's first token
    if (jw < q.kv && row_tile * 16 < rows) {
      float sc[2 * kRowTiles][4];
#pragma unroll
      for (int i = 0; i < 2 * kRowTiles; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[i][c] = 0.f;
      if (kRowTiles == 1) {
        // four chains of four products instead of two of eight: half the latency
        float sd[2][4];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) sd[i][c] = 0.f;
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const int chunk = kk * 2 + kcol;  // 16-byte chunk of the row; 128-byte swizzle within a half
          uint32_t b[4];
          ptx::ldsm4(kt + (chunk >> 3) * kHalf + krow * 128 + (((chunk & 7) ^ (krow & 7)) << 4), b);
          ptx::mma16816(kk & 1 ? sd[0] : sc[0], qa[kk], b[0], b[1]);
          ptx::mma16816(kk & 1 ? sd[1] : sc[1], qa[kk], b[2], b[3]);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[i][c] += sd[i][c];
      } else {
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const int chunk = kk * 2 + kcol;
#pragma unroll
          for (int i = 0; i < kRowTiles; ++i) {
            uint32_t b[4];
            ptx::ldsm4(kt + (chunk >> 3) * kHalf + (krow + 16 * i) * 128 + (((chunk & 7) ^ (krow & 7)) << 4), b);
            ptx::mma16816(sc[2 * i], qa[kk], b[0], b[1]);
            ptx::mma16816(sc[2 * i + 1], qa[kk], b[2], b[3]);
          }
        }
      }
      float xa = -INFINITY, xb = -INFINITY;
      const bool ragged = jw + kRun - 1 > last_all;
#pragma unroll
      for (int i = 0; i < 2 * kRowTiles; ++i) {
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[i][c] *= p.scale_log2;
        if (ragged) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (jw + i * 8 + cq + (c & 1) > (c < 2 ? last_a : last_b)) sc[i][c] = -INFINITY;
        }
        xa = ptx::fmax3(xa, sc[i][0], sc[i][1]);
        xb = ptx::fmax3(xb, sc[i][2], sc[i][3]);
      }
      if (kRowTiles == 1 && p.scores != nullptr) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (ra < rows)
            *reinterpret_cast<float2*>(p.scores + score_a + jw + i * 8) = make_float2(sc[i][0], sc[i][1]);
          if (rb < rows)
            *reinterpret_cast<float2*>(p.scores + score_b + jw + i * 8) = make_float2(sc[i][2], sc[i][3]);
        }
      }
      xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 1));
      xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 1));
      xa = fmaxf(xa, __shfl_xor_sync(0xffffffffu, xa, 2));
      xb = fmaxf(xb, __shfl_xor_sync(0xffffffffu, xb, 2));
      if (__any_sync(0xffffffffu, xa > ma + kRescale || xb > mb + kRescale)) {
        const float na = fmaxf(ma, xa), nb = fmaxf(mb, xb);
        const float fa = ptx::ex2(ma - na), fb = ptx::ex2(mb - nb);
        ma = na;
        mb = nb;
        la *= fa;
        lb *= fb;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          o[i][0] *= fa;
          o[i][1] *= fa;
          o[i][2] *= fb;
          o[i][3] *= fb;
        }
      }
      const bool cut = jw + kRun > q.kv;
#pragma unroll
      for (int i = 0; i < kRowTiles; ++i) {
        // p in fp32 for the sum; rounded to bf16 for the product with V, the operand type of the
        // matrix instruction (half a step, 2^-8, of each weight: the size of the output's own rounding)
        float (&x)[4] = sc[2 * i];
        float (&y)[4] = sc[2 * i + 1];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          x[c] = ptx::ex2(x[c] - (c < 2 ? ma : mb));
          y[c] = ptx::ex2(y[c] - (c < 2 ? ma : mb));
        }
        la += (x[0] + x[1]) + (y[0] + y[1]);
        lb += (x[2] + x[3]) + (y[2] + y[3]);
        const uint32_t pa[4] = {pack2(x[0], x[1]), pack2(x[2], x[3]), pack2(y[0], y[1]), pack2(y[2], y[3])};
        // tokens past the end have p = 0, but their V may be anything: zero it
        uint32_t k0 = 0xffffffffu, k1 = 0xffffffffu;
        if (cut) {
          const int v = q.kv - jw - 16 * i;
          k0 = (cq < v ? 0xffffu : 0u) | (cq + 1 < v ? 0xffff0000u : 0u);
          k1 = (cq + 8 < v ? 0xffffu : 0u) | (cq + 9 < v ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int np = 0; np < 8; ++np) {
          const int chunk = np * 2 + vcol;
          uint32_t b[4];
          ptx::ldsm4_t(vt + (chunk >> 3) * kHalf + (vrow + 16 * i) * 128 + (((chunk & 7) ^ (vrow & 7)) << 4), b);
          if (cut) {
            b[0] &= k0;
            b[1] &= k1;
            b[2] &= k0;
            b[3] &= k1;
          }
          ptx::mma16816(o[2 * np], pa, b[0], b[1]);
          ptx::mma16816(o[2 * np + 1], pa, b[2], b[3]);
        }
      }
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&empty[st]);
  }

  // ------------------------------------------------------------ merge of the runs
  la += __shfl_xor_sync(0xffffffffu, la, 1);
  lb += __shfl_xor_sync(0xffffffffu, lb, 1);
  la += __shfl_xor_sync(0xffffffffu, la, 2);
  lb += __shfl_xor_sync(0xffffffffu, lb, 2);
  const bool whole = u.t0 == 0 && u.t1 == u.tiles;
  // a part: this thread block's first slot if the unit began before its share, else its second
  const long long slot = (2LL * blockIdx.x + (u.t0 == 0 ? 1 : 0)) * p.slot_rows;
  if (kRowTiles == 2) {
    // the second run's warp holds the same rows and columns lane by lane: half of them at a time
    float2* far = reinterpret_cast<float2*>(mo) + row_tile * 16 * 32 + lane;
    if (warp >= kRowTiles) {
      ml[row_tile * 64 + lane] = make_float2(ma, la);
      ml[row_tile * 64 + 32 + lane] = make_float2(mb, lb);
    }
    float ga = 0.f, gb = 0.f;
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      if (warp >= kRowTiles) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          far[(2 * i) * 32] = make_float2(o[half * 8 + i][0], o[half * 8 + i][1]);
          far[(2 * i + 1) * 32] = make_float2(o[half * 8 + i][2], o[half * 8 + i][3]);
        }
      }
      ptx::named_bar_sync(1, kWarps * 32);
      if (warp < kRowTiles) {
        if (half == 0) {
          const float2 ea = ml[row_tile * 64 + lane], eb = ml[row_tile * 64 + 32 + lane];
          const float na = fmaxf(ma, ea.x), nb = fmaxf(mb, eb.x);
          const float fa = ptx::ex2(ma - na), fb = ptx::ex2(mb - nb);
          ga = ptx::ex2(ea.x - na);
          gb = ptx::ex2(eb.x - nb);
          ma = na;
          mb = nb;
          la = la * fa + ea.y * ga;
          lb = lb * fb + eb.y * gb;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            o[i][0] *= fa;
            o[i][1] *= fa;
            o[i][2] *= fb;
            o[i][3] *= fb;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float2 x = far[(2 * i) * 32], y = far[(2 * i + 1) * 32];
          o[half * 8 + i][0] += x.x * ga;
          o[half * 8 + i][1] += x.y * ga;
          o[half * 8 + i][2] += y.x * gb;
          o[half * 8 + i][3] += y.y * gb;
        }
      }
      ptx::named_bar_sync(1, kWarps * 32);
    }
    if (ok && warp < kRowTiles) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int r = e ? rb : ra, tok = e ? tok_b : tok_a;
        if (r >= rows) continue;
        const float m = e ? mb : ma, l = e ? lb : la;
        if (whole) {
          const long long row = q.q0 + tok;
          const int head = u.h * p.group + r - tok * p.group;
          const float inv = l == 0.f ? 0.f : 1.0f / l;
          uint16_t* to = p.out + row * p.out_stride + head * kHeadDim + cq;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            *reinterpret_cast<uint32_t*>(to + i * 8) = pack2(o[i][2 * e] * inv, o[i][2 * e + 1] * inv);
          if (cq == 0) {
            const float z = l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : l;
            const long long rh = row * p.q_heads + head;
            if (p.lse != nullptr) p.lse[rh] = z * kLn2;
            if (p.lse2 != nullptr) p.lse2[rh] = z;
          }
        } else {
          float* to = p.part + (slot + r) * kHeadDim + cq;
#pragma unroll
          for (int i = 0; i < 16; ++i)
            *reinterpret_cast<float2*>(to + i * 8) = make_float2(o[i][2 * e], o[i][2 * e + 1]);
          if (cq == 0) p.part_ml[slot + r] = make_float2(m, l);
        }
      }
    }
    return;
  }
  if ((lane & 3) == 0) {
    ml[warp * 16 + ra] = make_float2(ma, la);
    ml[warp * 16 + rb] = make_float2(mb, lb);
  }
#pragma unroll
  for (int rg = 0; rg < 16 / kMergeRows; ++rg) {
    if (rg * kMergeRows >= rows) break;
    // lanes 16 (rg & 1) .. + 15 hold these rows, in their first or second half
    if ((lane >> 4) == (rg & 1)) {
      float* to = mo + (warp * kMergeRows + (ra & (kMergeRows - 1))) * kHeadDim + cq;
#pragma unroll
      for (int i = 0; i < 16; ++i)
        *reinterpret_cast<float2*>(to + i * 8) = make_float2(o[i][rg & 2], o[i][(rg & 2) + 1]);
    }
    ptx::named_bar_sync(1, kWarps * 32);
    const int r = rg * kMergeRows + warp, c = lane * 4;  // a warp per row
    if (ok && r < rows) {
      float m = kNoKey;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) m = fmaxf(m, ml[i * 16 + r].x);
      float l = 0.f;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float2 e = ml[i * 16 + r];
        const float f = ptx::ex2(e.x - m);
        const float4 y = *reinterpret_cast<const float4*>(mo + (i * kMergeRows + warp) * kHeadDim + c);
        l += e.y * f;
        x.x += y.x * f;
        x.y += y.y * f;
        x.z += y.z * f;
        x.w += y.w * f;
      }
      if (whole) {
        const int tok = r / p.group;
        const long long row = q.q0 + tok;
        const int head = u.h * p.group + r - tok * p.group;
        const float inv = l == 0.f ? 0.f : 1.0f / l;
        *reinterpret_cast<uint2*>(p.out + row * p.out_stride + head * kHeadDim + c) =
            make_uint2(pack2(x.x * inv, x.y * inv), pack2(x.z * inv, x.w * inv));
        if (lane == 0) {
          const float z = l > 0.f ? m + log2f(l) : l == 0.f ? -INFINITY : l;
          const long long rh = row * p.q_heads + head;
          if (p.lse != nullptr) p.lse[rh] = z * kLn2;
          if (p.lse2 != nullptr) p.lse2[rh] = z;
        }
      } else {
        *reinterpret_cast<float4*>(p.part + (slot + r) * kHeadDim + c) = x;
        if (lane == 0) p.part_ml[slot + r] = make_float2(m, l);
      }
    }
    ptx::named_bar_sync(1, kWarps * 32);
  }
}

template <int kMaxRowTiles>
__global__ void __launch_bounds__(kDecodeThreads, 2)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ PagedAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kSmemDecodeBar);
  uint64_t* empty = full + kStages;
  ptx::let_next_launch();
  const PagedView& w = p.view;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], kWarps);
    }
    ptx::fence_mbar_init();
  }
  __syncthreads();  // the last one: from here on every warp finds its way by itself
  ptx::wait_previous();
  if (cta == 0 && threadIdx.x == 0) *p.ticket = 0;
  TokenWalk walk;
  walk.share(w);
  if (cta >= walk.of.n) {
    if (threadIdx.x == 0) p.joins[cta] = PagedJoin{};
    return;
  }
  walk.left = walk.of.start(cta + 1) - walk.of.start(cta);
  walk.go_to(w, walk.of.start(cta));
  TokenUnit u;

  if (warp == kWarps) {
    // ------------------------------------------------------------ TMA producer
    const int box = min(1 << w.page_shift, kTileKeys);  // tokens per copy
    const int n_box = kTileKeys / box;
    const int b = lane % n_box, c = (lane / n_box) & 1;
    const bool is_v = (lane / n_box) & 2;
    const bool mine = lane < 4 * n_box;
    const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
    uint8_t* dst = smem + (is_v ? 2 : 0) * kHalf + c * kHalf + b * box * 128;
    if (mine && b == 0 && c == 0) ptx::prefetch_tmap(tm);
    bool ok = true;
    int g = 0;  // tiles issued
    while (ok && walk.next(w, u)) {
      const int kv = u.q.kv;
      int id = -1;
      if (mine && u.t0 * kTileKeys + b * box < kv) id = paged_id(w, u.s, (u.t0 * kTileKeys + b * box) >> w.page_shift);
      for (int t = u.t0; t < u.t1; ++t) {
        const int st = g % kStages;
        const int j = t * kTileKeys + b * box;
        const int page = max(id, 0);
        // the next tile's page, on its way while this tile's stage is waited for
        if (mine && t + 1 < u.t1 && j + kTileKeys < kv) id = paged_id(w, u.s, (j + kTileKeys) >> w.page_shift);
        if (g >= kStages) {
          ok = __all_sync(0xffffffffu, ptx::mbar_wait(&empty[st], ((g / kStages) - 1) & 1, p.wait_limit_ns));
          if (!ok) break;
        }
        if (lane == 0) {
          const int boxes = (max(0, min(kv - t * kTileKeys, kTileKeys)) + box - 1) / box;
          ptx::mbar_arrive_expect_tx(&full[st], boxes * box * 128 * 4);
        }
        __syncwarp();
        if (mine && j < kv)
          ptx::tma_load_3d(dst + st * kStageBytes, tm, &full[st], c * 64,
                           (u.h << w.page_shift) + (j & ((1 << w.page_shift) - 1)), page);
        ++g;
      }
    }
    if (!ok && lane == 0) paged_report(w, kStatusTimeout);
    // every copy issued must land before the thread block may exit
    if (lane == 0)
      for (int t = max(0, g - kStages); t < g; ++t) ptx::mbar_wait(&full[t % kStages], (t / kStages) & 1, kDrainNs);
    return;
  }

  // -------------------------------------------------------------- consumers
  // a unit takes the fewest row tiles that hold its rows: with few rows all four warps share the tokens
  if (threadIdx.x == 0) p.joins[cta] = walk.join(cta);
  bool ok = true;
  int g = 0;
  while (walk.next(w, u)) {
    const int rows = u.q.n_q * p.group;
    if (kMaxRowTiles == 1 || rows <= 16)
      token_unit<1>(p, u, smem, full, empty, g, ok);
    else
      token_unit<2>(p, u, smem, full, empty, g, ok);
  }
  if (!ok && lane == 0) paged_report(w, kStatusTimeout);
}

// ---------------------------------------------------------------- attention weight of single tokens
// The scores that the attention kept (masked ones -infinity) and the rows' log-sum-exp: a key gathers
// the sum over the stream's at most 16 rows of 2^(score - z). Keeping a score costs 8
// bytes of traffic per row and key; reading K again would cost 256 for all rows.
constexpr int kTokenWeightThreads = 256;
constexpr int kTokenWeightKeys = 4;  // per thread
constexpr int kTokenWeightTile = kTokenWeightThreads * kTokenWeightKeys;

__global__ void __launch_bounds__(kTokenWeightThreads)
    paged_token_weight_kernel(const __grid_constant__ PagedAttnParams p) {
  const PagedView& w = p.view;
  const int n_kt = (w.max_kv + kTokenWeightTile - 1) / kTokenWeightTile;
  const int sh = blockIdx.x / n_kt;
  const int h = sh % w.kv_heads, s = sh / w.kv_heads;
  const int j0 = (blockIdx.x - sh * n_kt) * kTokenWeightTile + threadIdx.x;
  ptx::wait_previous();  // before the lengths too: the kernels before this one let it start before they have waited
  const PagedSeq q = paged_seq(w, s);
  float* to = p.weight + (static_cast<long long>(s) * w.kv_heads + h) * p.weight_stride;
  const int fresh = q.kv - q.n_q;  // the chunk's own keys start from zero
  if (!q.ok || q.n_q == 0 || j0 >= q.kv) return;
  float old[kTokenWeightKeys], sum[kTokenWeightKeys];
#pragma unroll
  for (int k = 0; k < kTokenWeightKeys; ++k) {
    const int j = j0 + k * kTokenWeightThreads;
    old[k] = j < fresh ? to[j] : 0.f;
    sum[k] = 0.f;
  }
  for (int t = 0; t < q.n_q; ++t) {
    const long long rh = static_cast<long long>(q.q0 + t) * p.q_heads + h * p.group;
#pragma unroll 4
    for (int g = 0; g < p.group; ++g) {
      // a row that sees no key has z = -infinity and nothing but scores of -infinity: +infinity gives its keys 0
      const float lse = p.lse2[rh + g], z = lse == -INFINITY ? INFINITY : lse;
      const float* sc = p.scores + (rh + g) * p.score_stride;
#pragma unroll
      for (int k = 0; k < kTokenWeightKeys; ++k) {
        const int j = j0 + k * kTokenWeightThreads;
        if (j < q.kv) sum[k] += ptx::ex2(sc[j] - z);
      }
    }
  }
#pragma unroll
  for (int k = 0; k < kTokenWeightKeys; ++k) {
    const int j = j0 + k * kTokenWeightThreads;
    if (j < q.kv) to[j] = old[k] + sum[k];
  }
}

}  // namespace

cudaError_t launch_paged_token_weight(const PagedAttnParams& p, cudaStream_t stream) {
  const unsigned n_kt = (p.view.max_kv + kTokenWeightTile - 1) / kTokenWeightTile;
  return launch_after(paged_token_weight_kernel, n_kt * p.view.n_seqs * p.view.kv_heads, kTokenWeightThreads, 0, stream, p);
}

cudaError_t launch_paged_decode(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const PagedAttnParams& p,
                                cudaStream_t stream) {
  // a per-device setting, made once on every device this process launches on
  constexpr int kMaxDevices = 64;
  static std::mutex mu;
  static bool configured[kMaxDevices] = {};
  int dev = 0;
  cudaError_t err = cudaGetDevice(&dev);
  if (err != cudaSuccess) return err;
  if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
  {
    std::lock_guard<std::mutex> lock(mu);
    if (!configured[dev]) {
      constexpr auto kAttr = cudaFuncAttributeMaxDynamicSharedMemorySize;
      err = cudaFuncSetAttribute(paged_decode_kernel<1>, kAttr, kDecodeSmem);
      if (err == cudaSuccess) err = cudaFuncSetAttribute(paged_decode_kernel<2>, kAttr, kDecodeSmem);
      if (err != cudaSuccess) return err;
      configured[dev] = true;
    }
  }
  const auto kernel = p.slot_rows == 16 ? paged_decode_kernel<1> : paged_decode_kernel<2>;
  return launch_after(kernel, 2 * kSmCount, kDecodeThreads, kDecodeSmem, stream, tm_k, tm_v, p);
}

}  // namespace rkv
