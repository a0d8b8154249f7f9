// Units of the paged attention that several thread blocks shared: their parts are added up. With references m_i
// (log2), sums l_i and unnormalised outputs o_i of the parts
//   m = max m_i, out = sum_i o_i 2^(m_i - m) / sum_i l_i 2^(m_i - m), in a fixed order.
//
// There may be hundreds of shared units with two parts each, or one with hundreds, of 1 to 256 rows.
//   Many units, so few parts each: thread blocks for every place of the list, most of which are empty; eight rows by half
// the columns (single-token form) or by all (chunk form).
//   Few units (by the host's bound): the thread blocks first gather the units from the list, and cut the columns as finely,
// down to an eighth, as gives each of them work.
// The lanes that a row's columns leave over, and the warps that the rows leave over, read further parts at the
// same time (not in the chunk form of the first). All of a step's loads leave together; a part past the last weighs nothing.
// The time is that of a few loads in a row: 1 us to start, 2 to 3 us for up to 40 parts. Measured, attention and join,
// few units' way and many units': one stream of 20000 tokens, 16 heads to one KV head (296 parts), 20 and 31 us; 30
// tokens of 8 heads to one (148 parts of 240 rows), 29 and 56; 8 KV heads of 64 rows (18 parts), 28 and 35; of 4 rows
// (37 parts), 10.5 and 9.5; 24 streams of 8 KV heads with their weights, 72 and 70.5.
#include <algorithm>

#include "attention_tile.cuh"
#include "paged.cuh"
#include "ptx_warp.cuh"

namespace rkv {
namespace {

constexpr int kWarps = 8;  // rows of an item
constexpr int kTokenBatch = 5, kChunkBatch = 4, kFewBatch = 4;  // parts on their way per lane
constexpr int kRows = 128;  // rows of a query tile of the chunk form
constexpr int kBlocks = 4 * kSmCount;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kNoKey = -1e30f;  // reference (log2) of a row that has seen no key

struct Sum {  // of some parts of a row: reference, sum of p, four columns of the sum of p v
  float m, l;
  float4 o;

  __device__ __forceinline__ void add(float em, float el, float4 y) {
    const float mn = fmaxf(m, em);
    const float f = ptx::ex2(m - mn), f2 = ptx::ex2(em - mn);
    m = mn;
    l = l * f + el * f2;
    o.x = o.x * f + y.x * f2;
    o.y = o.y * f + y.y * f2;
    o.z = o.z * f + y.z * f2;
    o.w = o.w * f + y.w * f2;
  }
};

__device__ __forceinline__ long long slot_of(const PagedJoin& j, int i) {
  return i == 0 ? j.slot0 : j.slot0 + 1 + (i - 1) * j.step;
}

// Four columns of a row, and with the first ones its log-sum-exp.
__device__ __forceinline__ void store(const PagedAttnParams& p, const Sum& s, long long row, int head, int col) {
  const float inv = s.l == 0.f ? 0.f : 1.0f / s.l;
  *reinterpret_cast<uint2*>(p.out + row * p.out_stride + head * kHeadDim + col) =
      make_uint2(pack_bf16x2(s.o.x * inv, s.o.y * inv), pack_bf16x2(s.o.z * inv, s.o.w * inv));
  if (col == 0) {
    const float z = s.l > 0.f ? s.m + log2f(s.l) : s.l == 0.f ? -INFINITY : s.l;
    const long long rh = row * p.q_heads + head;
    if (p.lse != nullptr) p.lse[rh] = z * kLn2;
    if (p.lse2 != nullptr) p.lse2[rh] = z;
  }
}

// Rows [row0, row0 + 8) of unit j, column block cb of 2^cut; kBatch parts on their way per lane. Whole thread blocks
// call it. per_token: 1 / G in 16 bits after the point, rounded up (exact for the quotients of 256 rows). kChunk: the
// parts are the chunk form's.
template <int kBatch, bool kChunk>
__device__ __forceinline__ void join_rows(const PagedAttnParams& p, const PagedJoin& j, int row0, int cut, int cb, int tpt, int per_token) {
  __shared__ float4 sum_o[kWarps][32];
  __shared__ float2 sum_ml[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.group;
  const int rows = min(kWarps, (j.cnt <= tpt ? j.cnt * G : 2 * kRows) - row0);
  if (rows <= 0) return;
  const int lanes = 32 >> cut, sub = lane >> (5 - cut), subs = 1 << cut;
  const int col = cb * (kHeadDim >> cut) + (lane & (lanes - 1)) * 4;
  int teams = 0, team = -1;  // kWarps / rows, warp / rows
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    teams += (i + 1) * rows <= kWarps;
    team += i * rows <= warp;
  }
  const int rr = row0 + warp - team * rows, r = rr % kRows, t = r * per_token >> 16;
  const int tok = rr / kRows * tpt + t;
  const bool live = team < teams && t < tpt && tok < j.cnt;
  Sum s = {kNoKey, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  if (live) {
    const int step = teams * subs;
    for (int i0 = team * subs + sub; i0 < j.parts; i0 += kBatch * step) {
      float2 e[kBatch];
      float4 y[kBatch];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = i0 + k * step;
        const long long slot = slot_of(j, i) * p.part_rows;
        e[k] = make_float2(kNoKey, 0.f);
        y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (i < j.parts) {
          e[k] = p.part_ml[slot + rr];
          y[k] = reinterpret_cast<const float4*>(p.part)[slot * 32 + (kChunk ? paged_part_place(rr, col / 4) : rr * 32 + col / 4)];
        }
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) s.add(e[k].x, e[k].y, y[k]);
    }
  }
  for (int d = lanes; d < 32; d <<= 1) {
    const float em = __shfl_down_sync(0xffffffffu, s.m, d), el = __shfl_down_sync(0xffffffffu, s.l, d);
    float4 y;
    y.x = __shfl_down_sync(0xffffffffu, s.o.x, d);
    y.y = __shfl_down_sync(0xffffffffu, s.o.y, d);
    y.z = __shfl_down_sync(0xffffffffu, s.o.z, d);
    y.w = __shfl_down_sync(0xffffffffu, s.o.w, d);
    s.add(em, el, y);
  }
  if (teams > 1) {
    if (sub == 0) sum_o[warp][lane] = s.o;
    if (lane == 0) sum_ml[warp] = make_float2(s.m, s.l);
    __syncthreads();
    if (team == 0 && sub == 0)
      for (int i = 1; i < teams; ++i) s.add(sum_ml[i * rows + warp].x, sum_ml[i * rows + warp].y, sum_o[i * rows + warp][lane]);
    __syncthreads();  // before the next item's sums
  }
  if (!live || team != 0 || sub != 0) return;
  store(p, s, j.row0 + tok, j.h * G + r - t * G, col);
}

__host__ __device__ __forceinline__ int row_blocks(const PagedAttnParams& p) { return (p.join_rows + kWarps - 1) / kWarps; }

// The single-token form's: two blocks of columns.
__global__ void __launch_bounds__(kWarps * 32, 4) paged_join_kernel(const __grid_constant__ PagedAttnParams p) {
  ptx::let_next_launch();
  const int tpt = kRows / p.group, per_token = (65535 + p.group) / p.group;
  ptx::wait_previous();  // in every thread block, so that the kernel after this one may rely on it
  const PagedJoin j = p.joins[blockIdx.y];
  if (j.parts > 0)
    join_rows<kTokenBatch, false>(p, j, (blockIdx.x >> 1) * kWarps, 1, blockIdx.x & 1, tpt, per_token);
}

// The chunk form's: a thread has four columns of one of eight rows.
__global__ void __launch_bounds__(256) paged_join_chunk_kernel(const __grid_constant__ PagedAttnParams p) {
  ptx::let_next_launch();
  const int tpt = kRows / p.group, per_token = (65535 + p.group) / p.group;
  ptx::wait_previous();
  const PagedJoin j = p.joins[blockIdx.y];
  const int rr = blockIdx.x * 8 + (threadIdx.x & 7), r = rr % kRows, t = r * per_token >> 16;
  const int tok = rr / kRows * tpt + t;
  if (t >= tpt || tok >= j.cnt) return;  // no parts: no tokens
  Sum s = {kNoKey, 0.f, make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int i0 = 0; i0 < j.parts; i0 += kChunkBatch) {
    float2 x[kChunkBatch];
    float4 y[kChunkBatch];
#pragma unroll
    for (int k = 0; k < kChunkBatch; ++k) {
      const long long slot = slot_of(j, i0 + k) * kPagedPartRows;
      x[k] = make_float2(kNoKey, 0.f);
      y[k] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i0 + k < j.parts) {
        x[k] = p.part_ml[slot + rr];
        y[k] = reinterpret_cast<const float4*>(p.part)[slot * 32 + paged_part_place(rr, threadIdx.x >> 3)];
      }
    }
#pragma unroll
    for (int k = 0; k < kChunkBatch; ++k) s.add(x[k].x, x[k].y, y[k]);
  }
  store(p, s, j.row0 + tok, j.h * p.group + r - t * p.group, (threadIdx.x >> 3) * 4);
}

template <bool kChunk>
__global__ void __launch_bounds__(kWarps * 32, 4) paged_join_few_kernel(const __grid_constant__ PagedAttnParams p) {
  __shared__ PagedJoin list[2 * kSmCount];
  __shared__ int counts[kWarps];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  ptx::let_next_launch();
  const int tpt = kRows / p.group, per_token = (65535 + p.group) / p.group;
  ptx::wait_previous();
  const int per = (p.n_joins + kWarps - 1) / kWarps;  // places of a warp: at most 37
  PagedJoin mine[2];
  unsigned has[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int i = e * 32 + lane, c = warp * per + i;
    mine[e].parts = 0;
    if (i < per && c < p.n_joins) mine[e] = p.joins[c];
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) has[e] = __ballot_sync(0xffffffffu, mine[e].parts > 0);
  if (lane == 0) counts[warp] = __popc(has[0]) + __popc(has[1]);
  __syncthreads();
  const int v = lane < kWarps ? counts[lane] : 0;
  const int total = __reduce_add_sync(0xffffffffu, v);
  const int before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
  const unsigned below = (1u << lane) - 1u;
  if (mine[0].parts > 0) list[before + __popc(has[0] & below)] = mine[0];
  if (mine[1].parts > 0) list[before + __popc(has[0]) + __popc(has[1] & below)] = mine[1];
  __syncthreads();
  const int blocks = row_blocks(p);
  int cut = 0;
  while (cut < 3 && (total * blocks << (cut + 1)) <= kBlocks) ++cut;
  for (int item = blockIdx.x; item < total * blocks << cut; item += gridDim.x) {
    const int x = item >> cut, n = x / blocks;
    join_rows<kFewBatch, kChunk>(p, list[n], (x - n * blocks) * kWarps, cut, item & ((1 << cut) - 1), tpt, per_token);
  }
}

}  // namespace

cudaError_t launch_paged_join(const PagedAttnParams& p, cudaStream_t stream) {
  const bool token = p.slot_rows > 0;
  const int blocks = std::max(1, row_blocks(p));
  // few: a unit's parts, if all thread blocks share the units, would take the usual kernel two steps (chunk form) or four
  // (the figures above)
  if (p.max_units * (token ? 8 * kTokenBatch : 2 * kChunkBatch) <= p.n_joins) {
    const int items = static_cast<int>(p.max_units) * blocks * 8;
    return launch_after(token ? paged_join_few_kernel<false> : paged_join_few_kernel<true>, std::min(kBlocks, std::max(1, items)),
                        kWarps * 32, 0, stream, p);
  }
  const unsigned n = static_cast<unsigned>(p.n_joins);
  if (token) return launch_after(paged_join_kernel, dim3(2 * blocks, n), kWarps * 32, 0, stream, p);
  return launch_after(paged_join_chunk_kernel, dim3(blocks, n), 256, 0, stream, p);
}

}  // namespace rkv
