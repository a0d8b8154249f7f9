// Attention over a paged cache when a stream brings few rows: at most 16 per KV head (a single
// token of up to 16 grouped heads, a few drafted tokens of fewer). And the combine of parts, for
// every form.
//
// With R rows per KV head a cached token costs 512 bytes of K and V and 512 R multiply-adds, so
// at 16 rows the memory asks for 16 flops a byte, a fraction of what even the warp-level matrix
// instructions (mma.sync m16n8k16, whose 16 rows fit exactly) give: the kernel is bound by
// HBM, and everything serves to keep loads in flight. A block takes one (stream, KV head, part
// of the key stream); one warp issues TMA copies of 64-token tiles (K and V, one box per page and
// 64-column half) into three stages, four warps own 16 tokens of each tile and run their own
// softmax in registers, without meeting each other until the part's end, where the four partial
// results are merged in shared memory. Two blocks fit an SM: six stages of 32 KB in flight.
#include <mutex>

#include "numeric.cuh"
#include "paged.cuh"
#include "ptx_sm100.cuh"

namespace rkv {
namespace {

constexpr int kTileKeys = kPagedDecodeTile;
constexpr int kHalf = kTileKeys * 128;  // bytes of one 64-column half of a tile
constexpr int kStageBytes = 4 * kHalf;  // K halves, V halves
constexpr int kStages = 3;
constexpr int kWarps = 4;               // consumer warps, 16 tokens of a tile each
constexpr int kDecodeThreads = (kWarps + 1) * 32;
constexpr int kDecodeSmem = kStages * kStageBytes + 128 + 1024;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescale = 8.0f;  // log2: the running reference follows a maximum only past this
constexpr float kNoKey = -1e30f;  // reference (log2) of a row that has seen no key
constexpr unsigned long long kDrainNs = 2000000000ull;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__global__ void __launch_bounds__(kDecodeThreads, 2)
    paged_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const __grid_constant__ PagedAttnParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  ptx::let_next_launch();
  const PagedView& w = p.view;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // blocks of one stream and head next to each other: they share pages' neighbourhoods in L2
  const int sp = blockIdx.x % p.n_split;
  const int sh = blockIdx.x / p.n_split;
  const int h = sh % w.kv_heads, s = sh / w.kv_heads;
  const PagedSeq q = paged_seq(w, s);
  if (!q.ok) {
    if (threadIdx.x == 0) paged_report(w, kStatusLength);
    return;
  }
  const int rows = q.n_q * p.group;
  const int j0 = sp * p.split_keys;
  if (rows == 0 || (j0 >= q.kv && (sp > 0 || p.n_split > 1))) return;
  const int j1 = min(q.kv, j0 + p.split_keys);
  const int n_tiles = (j1 - j0 + kTileKeys - 1) / kTileKeys;  // 0 only when kv == 0

  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      ptx::mbar_init(&full[i], 1);
      ptx::mbar_init(&empty[i], kWarps);
    }
    ptx::fence_mbar_init();
  }
  __syncthreads();

  if (warp == kWarps) {
    // ------------------------------------------------------------ TMA producer
    const int box = min(1 << w.page_shift, kTileKeys);  // tokens per copy
    const int n_box = kTileKeys / box;
    const int b = lane % n_box, c = (lane / n_box) & 1;
    const bool is_v = (lane / n_box) & 2;
    const bool mine = lane < 4 * n_box;
    const CUtensorMap* tm = is_v ? &tm_v : &tm_k;
    const int dst = (is_v ? 2 : 0) * kHalf + c * kHalf + b * box * 128;
    if (mine && b == 0 && c == 0) ptx::prefetch_tmap(tm);
    bool ok = true;
    int issued = 0;
    int id = -1;
    if (mine && j0 + b * box < j1) id = paged_id(w, s, (j0 + b * box) >> w.page_shift);
    for (int t = 0; t < n_tiles; ++t) {
      const int st = t % kStages;
      const int j = j0 + t * kTileKeys + b * box;
      const int page = id;
      // the next tile's page, on its way while this tile's stage is waited for
      if (mine && j + kTileKeys < j1) id = paged_id(w, s, (j + kTileKeys) >> w.page_shift);
      if (t >= kStages) {
        ok = ptx::mbar_wait(&empty[st], ((t / kStages) - 1) & 1, p.wait_limit_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
      }
      if (lane == 0) {
        const int boxes = (min(j1 - (j0 + t * kTileKeys), kTileKeys) + box - 1) / box;
        ptx::mbar_arrive_expect_tx(&full[st], boxes * box * 128 * 4);
      }
      __syncwarp();
      if (mine && j < j1)
        ptx::tma_load_3d(smem + st * kStageBytes + dst, tm, &full[st], c * 64,
                         (h << w.page_shift) + (j & ((1 << w.page_shift) - 1)), max(page, 0));
      issued = t + 1;
    }
    if (!ok && lane == 0) paged_report(w, kStatusTimeout);
    // every copy issued must land before the block may exit
    if (lane == 0)
      for (int t = max(0, issued - kStages); t < issued; ++t)
        ptx::mbar_wait(&full[t % kStages], (t / kStages) & 1, kDrainNs);
    return;
  }

  // -------------------------------------------------------------- consumers
  const int ra = lane >> 2, rb = ra + 8;  // this lane's two rows
  const int cq = (lane & 3) * 2;          // and its pair of columns within 8
  uint32_t qa[8][4];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int r = e ? rb : ra;
    const int tok = r / p.group;
    const bool live = r < rows;
    const uint16_t* src = p.q + (q.q0 + (live ? tok : 0)) * p.q_stride + (h * p.group + r - tok * p.group) * kHeadDim;
#pragma unroll
    for (int kk = 0; kk < 8; ++kk) {
      qa[kk][e] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + cq)) : 0u;
      qa[kk][2 + e] = live ? __ldg(reinterpret_cast<const uint32_t*>(src + kk * 16 + 8 + cq)) : 0u;
    }
  }
  // the last place each row sees
  const int last_a = p.causal ? q.kv - q.n_q + ra / p.group : q.kv - 1;
  const int last_b = p.causal ? q.kv - q.n_q + rb / p.group : q.kv - 1;
  const int last_all = p.causal ? q.kv - q.n_q : q.kv - 1;
  // where their scores go (a pair of places each), if they are kept
  auto score_row = [&](int r) {
    return (static_cast<long long>(q.q0 + r / p.group) * p.q_heads + h * p.group + r % p.group) * p.score_stride + cq;
  };
  const long long score_a = score_row(ra), score_b = score_row(rb);
  float o[16][4];
#pragma unroll
  for (int i = 0; i < 16; ++i)
#pragma unroll
    for (int c = 0; c < 4; ++c) o[i][c] = 0.f;
  float ma = kNoKey, mb = kNoKey, la = 0.f, lb = 0.f;  // references (log2) and this lane's sums
  // ldmatrix rows: K by token (lanes 8-15: the next 8 columns, 16-31: the next 8 tokens), V by token
  // (lanes 8-15: the next 8 tokens, 16-31: the next 8 columns)
  const int krow = warp * 16 + (lane >> 4) * 8 + (lane & 7), kcol = (lane >> 3) & 1;
  const int vrow = warp * 16 + ((lane >> 3) & 1) * 8 + (lane & 7), vcol = lane >> 4;
  const uint32_t sbase = ptx::smem_u32(smem);
  bool ok = true;
  for (int t = 0; t < n_tiles; ++t) {
    const int st = t % kStages;
    ok = ptx::mbar_wait(&full[st], (t / kStages) & 1, p.wait_limit_ns);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) break;
    const uint32_t kt = sbase + st * kStageBytes, vt = kt + 2 * kHalf;
    const int jw = j0 + t * kTileKeys + warp * 16;  // this warp's first token
    if (jw < j1) {
      float sc[2][4];
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[i][c] = 0.f;
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const int chunk = kk * 2 + kcol;  // 16-byte chunk of the row; 128-byte swizzle within a half
        uint32_t b[4];
        ptx::ldsm4(kt + (chunk >> 3) * kHalf + krow * 128 + (((chunk & 7) ^ (krow & 7)) << 4), b);
        ptx::mma16816(sc[0], qa[kk], b[0], b[1]);
        ptx::mma16816(sc[1], qa[kk], b[2], b[3]);
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[i][c] *= p.scale_log2;
      const bool ragged = jw + 15 > last_all;
      if (ragged) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (jw + i * 8 + cq + (c & 1) > (c < 2 ? last_a : last_b)) sc[i][c] = -INFINITY;
      }
      if (p.scores != nullptr) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (ra < rows)
            *reinterpret_cast<float2*>(p.scores + score_a + jw + i * 8) = make_float2(sc[i][0], sc[i][1]);
          if (rb < rows)
            *reinterpret_cast<float2*>(p.scores + score_b + jw + i * 8) = make_float2(sc[i][2], sc[i][3]);
        }
      }
      float xa = fmaxf(fmaxf(sc[0][0], sc[0][1]), fmaxf(sc[1][0], sc[1][1]));
      float xb = fmaxf(fmaxf(sc[0][2], sc[0][3]), fmaxf(sc[1][2], sc[1][3]));
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
      // p in fp32 for the sum; rounded to bf16 for the product with V, the operand type of the
      // matrix instruction (half a step, 2^-8, of each weight: the size of the output's own rounding)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        sc[i][0] = ptx::ex2(sc[i][0] - ma);
        sc[i][1] = ptx::ex2(sc[i][1] - ma);
        sc[i][2] = ptx::ex2(sc[i][2] - mb);
        sc[i][3] = ptx::ex2(sc[i][3] - mb);
        la += sc[i][0] + sc[i][1];
        lb += sc[i][2] + sc[i][3];
      }
      const uint32_t pa[4] = {pack2(sc[0][0], sc[0][1]), pack2(sc[0][2], sc[0][3]), pack2(sc[1][0], sc[1][1]),
                              pack2(sc[1][2], sc[1][3])};
      // tokens past the end have p = 0, but their V may be anything: zero it
      uint32_t k0 = 0xffffffffu, k1 = 0xffffffffu;
      const bool cut = jw + 16 > j1;
      if (cut) {
        const int v = j1 - jw;
        k0 = (cq < v ? 0xffffu : 0u) | (cq + 1 < v ? 0xffff0000u : 0u);
        k1 = (cq + 8 < v ? 0xffffu : 0u) | (cq + 9 < v ? 0xffff0000u : 0u);
      }
#pragma unroll
      for (int np = 0; np < 8; ++np) {
        const int chunk = np * 2 + vcol;
        uint32_t b[4];
        ptx::ldsm4_t(vt + (chunk >> 3) * kHalf + vrow * 128 + (((chunk & 7) ^ (vrow & 7)) << 4), b);
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
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(&empty[st]);
  }
  if (!ok && lane == 0) paged_report(w, kStatusTimeout);

  // -------------------------------------------------------------- merge of the four warps
  la += __shfl_xor_sync(0xffffffffu, la, 1);
  lb += __shfl_xor_sync(0xffffffffu, lb, 1);
  la += __shfl_xor_sync(0xffffffffu, la, 2);
  lb += __shfl_xor_sync(0xffffffffu, lb, 2);
  ptx::named_bar_sync(1, kWarps * 32);  // every tile was read: the stages' memory is free
  float* mo = reinterpret_cast<float*>(smem);                                  // [warp][row][128]
  float2* ml = reinterpret_cast<float2*>(smem + kWarps * 16 * kHeadDim * 4);  // [warp][row]
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    *reinterpret_cast<float2*>(mo + (warp * 16 + ra) * kHeadDim + i * 8 + cq) = make_float2(o[i][0], o[i][1]);
    *reinterpret_cast<float2*>(mo + (warp * 16 + rb) * kHeadDim + i * 8 + cq) = make_float2(o[i][2], o[i][3]);
  }
  if ((lane & 3) == 0) {
    ml[warp * 16 + ra] = make_float2(ma, la);
    ml[warp * 16 + rb] = make_float2(mb, lb);
  }
  ptx::named_bar_sync(1, kWarps * 32);
  if (!ok) return;
  // one row at a time per warp, four columns per lane
  for (int r = warp; r < rows; r += kWarps) {
    float m = kNoKey;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) m = fmaxf(m, ml[i * 16 + r].x);
    float l = 0.f;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      const float2 e = ml[i * 16 + r];
      const float f = ptx::ex2(e.x - m);
      const float4 y = *reinterpret_cast<const float4*>(mo + (i * 16 + r) * kHeadDim + lane * 4);
      l += e.y * f;
      x.x += y.x * f;
      x.y += y.y * f;
      x.z += y.z * f;
      x.w += y.w * f;
    }
    const int tok = r / p.group;
    const long long row = q.q0 + tok;
    const int head = h * p.group + r - tok * p.group;
    const long long rh = row * p.q_heads + head;
    if (p.n_split > 1) {
      const long long at = static_cast<long long>(sp) * w.n_rows * p.q_heads + rh;
      *reinterpret_cast<float4*>(p.part + at * kHeadDim + lane * 4) = x;
      if (lane == 0) p.part_ml[at] = make_float2(m, l);
    } else {
      const float inv = l > 0.f ? 1.0f / l : 0.f;
      *reinterpret_cast<uint2*>(p.out + row * p.out_stride + head * kHeadDim + lane * 4) =
          make_uint2(pack2(x.x * inv, x.y * inv), pack2(x.z * inv, x.w * inv));
      if (lane == 0) {
        const float z = l > 0.f ? m + log2f(l) : -INFINITY;
        if (p.lse != nullptr) p.lse[rh] = z * kLn2;
        if (p.lse2 != nullptr) p.lse2[rh] = z;
      }
    }
  }
}

// ---------------------------------------------------------------- combine of parts
// With parts i of a row, references m_i, sums l_i and unnormalised outputs o_i:
//   m = max m_i, out = sum_i o_i 2^(m_i - m) / sum_i l_i 2^(m_i - m).
// One block per (row, query head); its four warps take every fourth part.
constexpr int kCombineThreads = 128;

__global__ void __launch_bounds__(kCombineThreads) paged_combine_kernel(const __grid_constant__ PagedAttnParams p) {
  __shared__ float factor[kPagedMaxSplit];
  __shared__ float red[2][4];
  __shared__ float4 acc[4][32];
  const PagedView& w = p.view;
  const int head = blockIdx.x % p.q_heads, row = blockIdx.x / p.q_heads;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ptx::let_next_launch();
  const int s = paged_seq_of_row(w, row);
  PagedSeq q = {};
  if (s >= 0) q = paged_seq(w, s);
  ptx::wait_previous();  // in every thread block, so that the kernel after this one may rely on it
  if (s < 0 || !q.ok) return;
  // keys that the row's block of tokens sees, and so the parts that were written
  const int last_tok = min(q.n_q, ((row - q.q0) / p.block_tokens + 1) * p.block_tokens) - 1;
  const int keys = p.causal ? max(0, q.kv - q.n_q + last_tok + 1) : q.kv;
  const int n = (keys + p.split_keys - 1) / p.split_keys;
  const long long rh = static_cast<long long>(row) * p.q_heads + head;
  const long long step = static_cast<long long>(w.n_rows) * p.q_heads;
  float m = kNoKey;
  for (int i = threadIdx.x; i < n; i += kCombineThreads) m = fmaxf(m, p.part_ml[i * step + rh].x);
  for (int d = 16; d; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if (lane == 0) red[0][warp] = m;
  __syncthreads();
  m = fmaxf(fmaxf(red[0][0], red[0][1]), fmaxf(red[0][2], red[0][3]));
  float l = 0.f;
  for (int i = threadIdx.x; i < n; i += kCombineThreads) {
    const float2 e = p.part_ml[i * step + rh];
    const float f = ptx::ex2(e.x - m);
    factor[i] = f;
    l += e.y * f;
  }
  for (int d = 16; d; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  if (lane == 0) red[1][warp] = l;
  __syncthreads();
  l = (red[1][0] + red[1][1]) + (red[1][2] + red[1][3]);
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int i = warp; i < n; i += 4) {
    const float4 y = *reinterpret_cast<const float4*>(p.part + (i * step + rh) * kHeadDim + lane * 4);
    const float f = factor[i];
    x.x += y.x * f;
    x.y += y.y * f;
    x.z += y.z * f;
    x.w += y.w * f;
  }
  acc[warp][lane] = x;
  __syncthreads();
  if (warp != 0) return;
  float4 y = acc[0][lane];
  for (int i = 1; i < 4; ++i) {
    y.x += acc[i][lane].x;
    y.y += acc[i][lane].y;
    y.z += acc[i][lane].z;
    y.w += acc[i][lane].w;
  }
  const float inv = l > 0.f ? 1.0f / l : 0.f;
  *reinterpret_cast<uint2*>(p.out + row * p.out_stride + head * kHeadDim + lane * 4) =
      make_uint2(pack2(y.x * inv, y.y * inv), pack2(y.z * inv, y.w * inv));
  if (lane == 0) {
    const float z = l > 0.f ? m + log2f(l) : -INFINITY;
    if (p.lse != nullptr) p.lse[rh] = z * kLn2;
    if (p.lse2 != nullptr) p.lse2[rh] = z;
  }
}

// ---------------------------------------------------------------- attention weight of single tokens
// The scores that the attention kept (masked ones -infinity) and the rows' log-sum-exp: a key gathers
// the sum over the stream's at most 16 rows of 2^(score - z). One thread per key. Keeping a score costs 8
// bytes of traffic per row and key; reading K again would cost 256 for all rows.
constexpr int kTokenWeightThreads = 256;

__global__ void __launch_bounds__(kTokenWeightThreads)
    paged_token_weight_kernel(const __grid_constant__ PagedAttnParams p) {
  const PagedView& w = p.view;
  const int n_kt = (w.max_kv + kTokenWeightThreads - 1) / kTokenWeightThreads;
  const int sh = blockIdx.x / n_kt;
  const int h = sh % w.kv_heads, s = sh / w.kv_heads;
  const int j = (blockIdx.x - sh * n_kt) * kTokenWeightThreads + threadIdx.x;
  const PagedSeq q = paged_seq(w, s);
  ptx::wait_previous();
  if (!q.ok || q.n_q == 0 || j >= q.kv) return;
  float sum = 0.f;
  for (int t = 0; t < q.n_q; ++t) {
    const long long rh = static_cast<long long>(q.q0 + t) * p.q_heads + h * p.group;
#pragma unroll 4
    for (int g = 0; g < p.group; ++g)
      sum += ptx::ex2(p.scores[(rh + g) * p.score_stride + j] - p.lse2[rh + g]);
  }
  float* to = p.weight + (static_cast<long long>(s) * w.kv_heads + h) * p.weight_stride + j;
  *to = (j < q.kv - q.n_q ? *to : 0.f) + sum;
}

}  // namespace

cudaError_t launch_paged_token_weight(const PagedAttnParams& p, cudaStream_t stream) {
  const unsigned n_kt = (p.view.max_kv + kTokenWeightThreads - 1) / kTokenWeightThreads;
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
      err = cudaFuncSetAttribute(paged_decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDecodeSmem);
      if (err != cudaSuccess) return err;
      configured[dev] = true;
    }
  }
  const unsigned grid = static_cast<unsigned>(p.view.n_seqs) * p.view.kv_heads * p.n_split;
  paged_decode_kernel<<<grid, kDecodeThreads, kDecodeSmem, stream>>>(tm_k, tm_v, p);
  return cudaGetLastError();
}

cudaError_t launch_paged_combine(const PagedAttnParams& p, cudaStream_t stream) {
  return launch_after(paged_combine_kernel, static_cast<unsigned>(p.view.n_rows) * p.q_heads, kCombineThreads, 0, stream, p);
}

}  // namespace rkv
