// Attention of chunk rows over a paged cache, and the attention weight that each cached token
// gathers.
#include "numeric.cuh"
#include "paged.cuh"

namespace rkv {
namespace {

constexpr float kLn2 = 0.6931471805599453f;

// One warp per (chunk row, query head), four elements of d per lane, one key at a time with a
// running maximum and sum.
__global__ void __launch_bounds__(128) paged_attention_kernel(const __grid_constant__ PagedAttnParams p) {
  const PagedView& w = p.view;
  const long long gw = (static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x) >> 5;
  const int row = static_cast<int>(gw / p.q_heads), head = static_cast<int>(gw % p.q_heads);
  if (row >= w.n_rows) return;
  const int s = paged_seq_of_row(w, row);
  if (s < 0) return;
  const PagedSeq q = paged_seq(w, s);
  const int lane = threadIdx.x & 31;
  if (!q.ok) {
    if (lane == 0) paged_report(w, kStatusLength);
    return;
  }
  const int h = head / p.group;
  const int last = p.causal ? q.kv - q.n_q + (row - q.q0) : q.kv - 1;
  const uint2 qx = *reinterpret_cast<const uint2*>(p.q + row * p.q_stride + head * kHeadDim + lane * 4);
  const float q0 = bf16_to_f32(qx.x & 0xffff), q1 = bf16_to_f32(qx.x >> 16), q2 = bf16_to_f32(qx.y & 0xffff),
              q3 = bf16_to_f32(qx.y >> 16);
  float m = -INFINITY, l = 0.f, o0 = 0.f, o1 = 0.f, o2 = 0.f, o3 = 0.f;
  for (int j = 0; j <= last; ++j) {
    const int id = max(0, paged_id(w, s, j >> w.page_shift));
    const long long at = paged_offset(w, id, h, j & ((1 << w.page_shift) - 1)) + lane * 4;
    const uint2 kx = *reinterpret_cast<const uint2*>(w.k + at);
    const uint2 vx = *reinterpret_cast<const uint2*>(w.v + at);
    float x = q0 * bf16_to_f32(kx.x & 0xffff) + q1 * bf16_to_f32(kx.x >> 16) + q2 * bf16_to_f32(kx.y & 0xffff) +
              q3 * bf16_to_f32(kx.y >> 16);
    for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    x *= p.scale_log2;
    const float mn = fmaxf(m, x);
    const float f = exp2f(m - mn), e = exp2f(x - mn);
    m = mn;
    l = l * f + e;
    o0 = o0 * f + e * bf16_to_f32(vx.x & 0xffff);
    o1 = o1 * f + e * bf16_to_f32(vx.x >> 16);
    o2 = o2 * f + e * bf16_to_f32(vx.y & 0xffff);
    o3 = o3 * f + e * bf16_to_f32(vx.y >> 16);
  }
  const float inv = l > 0.f ? 1.0f / l : 0.f;
  uint2 o;
  o.x = f32_to_bf16_rne(o0 * inv) | (static_cast<uint32_t>(f32_to_bf16_rne(o1 * inv)) << 16);
  o.y = f32_to_bf16_rne(o2 * inv) | (static_cast<uint32_t>(f32_to_bf16_rne(o3 * inv)) << 16);
  *reinterpret_cast<uint2*>(p.out + row * p.out_stride + head * kHeadDim + lane * 4) = o;
  if (lane == 0) {
    const float z = l > 0.f ? m + log2f(l) : -INFINITY;
    if (p.lse != nullptr) p.lse[static_cast<long long>(row) * p.q_heads + head] = z * kLn2;
    if (p.lse2 != nullptr) p.lse2[static_cast<long long>(row) * p.q_heads + head] = z;
  }
}

// One warp per (stream, KV head, key): the key's weight over the rows that see it.
__global__ void __launch_bounds__(128) paged_weight_kernel(const __grid_constant__ PagedAttnParams p) {
  const PagedView& w = p.view;
  const int j = blockIdx.x * 4 + (threadIdx.x >> 5);
  const int s = blockIdx.y / w.kv_heads, h = blockIdx.y % w.kv_heads;
  const PagedSeq q = paged_seq(w, s);
  if (!q.ok || q.n_q == 0 || j >= q.kv) return;
  const int lane = threadIdx.x & 31;
  const int id = max(0, paged_id(w, s, j >> w.page_shift));
  const long long at = paged_offset(w, id, h, j & ((1 << w.page_shift) - 1)) + lane * 4;
  const uint2 kx = *reinterpret_cast<const uint2*>(w.k + at);
  const float k0 = bf16_to_f32(kx.x & 0xffff), k1 = bf16_to_f32(kx.x >> 16), k2 = bf16_to_f32(kx.y & 0xffff),
              k3 = bf16_to_f32(kx.y >> 16);
  float sum = 0.f;
  for (int i = p.causal ? max(0, j - (q.kv - q.n_q)) : 0; i < q.n_q; ++i)
    for (int g = 0; g < p.group; ++g) {
      const long long row = q.q0 + i;
      const int head = h * p.group + g;
      const uint2 qx = *reinterpret_cast<const uint2*>(p.q + row * p.q_stride + head * kHeadDim + lane * 4);
      float x = k0 * bf16_to_f32(qx.x & 0xffff) + k1 * bf16_to_f32(qx.x >> 16) + k2 * bf16_to_f32(qx.y & 0xffff) +
                k3 * bf16_to_f32(qx.y >> 16);
      for (int d = 16; d; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      sum += exp2f(x * p.scale_log2 - p.lse2[row * p.q_heads + head]);
    }
  if (lane == 0) {
    float* to = p.weight + (static_cast<long long>(s) * w.kv_heads + h) * p.weight_stride + j;
    *to = (j < q.kv - q.n_q ? *to : 0.f) + sum;
  }
}

}  // namespace

cudaError_t launch_paged_attention(const PagedAttnParams& p, cudaStream_t stream) {
  const long long warps = static_cast<long long>(p.view.n_rows) * p.q_heads;
  paged_attention_kernel<<<static_cast<unsigned>((warps + 3) / 4), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_paged_weight(const PagedAttnParams& p, cudaStream_t stream) {
  paged_weight_kernel<<<dim3((p.view.max_kv + 3) / 4, p.view.n_seqs * p.view.kv_heads), 128, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace rkv
