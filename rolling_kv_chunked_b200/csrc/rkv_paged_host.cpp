// Host side of the paged caches: argument checks and launches. Every exported function is
// declared and documented in include/rkv.h.
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/rkv.h"
#include "paged_internal.h"

#define RKV_API extern "C" __attribute__((visibility("default")))

using rkv::kHeadDim;
using rkv::PagedView;

namespace {

constexpr int kMaxSeqs = 1 << 16;
constexpr unsigned long long kWaitNs = 2000000000ull;  // cap on each device wait
constexpr long long kMaxScores = 1LL << 32;  // bytes of scores that a call keeps at most (in its workspace)
constexpr int kMaxGroup = 128;  // query heads of one KV head: one tile of query rows holds a token's

bool aligned16(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return p != nullptr && (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
// A failure is reported here and cleared: the rolling window's calls ask for the last error after their launches.
int cuda_rc(cudaError_t e) {
  if (e == cudaSuccess) return RKV_OK;
  cudaGetLastError();
  return RKV_ERR_CUDA;
}

// Host values of the pool and the batch (what rkv_paged_workspace looks at, no pointers).
int check_sizes(const rkv_page_pool* pool, const rkv_paged_batch* b, int n_rows) {
  if (pool == nullptr || b == nullptr || n_rows < 0) return RKV_ERR_ARG;
  if (pool->n_pages < 1 || pool->kv_heads < 1 || pool->page_tokens < 1 || b->n_seqs < 0 || b->max_q < 0 ||
      b->max_kv < 0 || b->table_stride < 0)
    return RKV_ERR_ARG;
  const int p = pool->page_tokens;
  if (p != 16 && p != 32 && p != 64 && p != 128) return RKV_ERR_UNSUPPORTED;
  const long long page = static_cast<long long>(pool->kv_heads) * p * kHeadDim;
  if (pool->page_stride < page || pool->page_stride % 8 != 0) return RKV_ERR_ARG;
  if (static_cast<long long>(b->table_stride) * p < b->max_kv) return RKV_ERR_ARG;
  // a tensor map's stride and extents; the launch grids
  if (pool->page_stride >= (1LL << 38) || static_cast<long long>(pool->kv_heads) * p >= (1LL << 31) ||
      b->n_seqs > kMaxSeqs || static_cast<long long>(b->n_seqs) * pool->kv_heads >= (1LL << 24) ||
      b->max_kv > (1 << 30) ||
      static_cast<long long>(b->n_seqs) * pool->kv_heads * ((b->max_kv + 127LL) / 128) >= (1LL << 30))
    return RKV_ERR_UNSUPPORTED;
  return RKV_OK;
}

int check_batch(const rkv_page_pool* pool, const rkv_paged_batch* b, int n_rows, bool rows) {
  const int rc = check_sizes(pool, b, n_rows);
  if (rc) return rc;
  if (!aligned16(pool->k) || !aligned16(pool->v)) return RKV_ERR_ARG;
  if (b->status != nullptr && !aligned4(b->status)) return RKV_ERR_ARG;
  if (b->n_seqs > 0 && (!aligned4(b->page_table) || !aligned4(b->kv_len))) return RKV_ERR_ARG;
  if (b->n_seqs > 0 && rows && !aligned4(b->q_start)) return RKV_ERR_ARG;
  return RKV_OK;
}

bool row_stride_ok(long long stride, int heads) {
  return stride % 8 == 0 && stride >= static_cast<long long>(heads) * kHeadDim && stride < (1LL << 38);
}

PagedView view_of(const rkv_page_pool* pool, const rkv_paged_batch* b, int n_rows) {
  PagedView w;
  std::memset(&w, 0, sizeof(w));
  w.k = static_cast<uint16_t*>(pool->k);
  w.v = static_cast<uint16_t*>(pool->v);
  w.page_stride = pool->page_stride;
  w.n_pages = pool->n_pages;
  w.kv_heads = pool->kv_heads;
  while ((1 << w.page_shift) < pool->page_tokens) ++w.page_shift;
  w.table = b->page_table;
  w.kv_len = b->kv_len;
  w.q_start = b->q_start;
  w.status = b->status;
  w.table_stride = b->table_stride;
  w.n_seqs = b->n_seqs;
  w.n_rows = n_rows;
  w.max_q = b->max_q;
  w.max_kv = b->max_kv;
  return w;
}

int check_heads(const rkv_page_pool* pool, int q_heads, int n_rows) {
  if (q_heads < 1 || q_heads % pool->kv_heads != 0) return RKV_ERR_ARG;
  if (q_heads / pool->kv_heads > kMaxGroup || static_cast<long long>(n_rows) * q_heads >= (1LL << 31))
    return RKV_ERR_UNSUPPORTED;
  return RKV_OK;
}

// Which form a call takes, and its workspace. The single-token form (warp-level matrix instructions, bound by
// HBM) serves up to 32 rows per stream and KV head; above that the chunk form's tiles of 128 rows are the
// better use (the measurements stand in rkv_paged_decode.cu).
rkv::PagedPlan plan_of(const rkv_page_pool* pool, const rkv_paged_batch* b, int q_heads, int n_rows, bool weight) {
  rkv::PagedPlan p;
  std::memset(&p, 0, sizeof(p));
  const int group = q_heads / pool->kv_heads;
  const long long most = static_cast<long long>(b->max_q) * group;
  if (most <= rkv::kPagedRows) {
    p.slot_rows = most <= 16 ? 16 : 32;
  } else {
    p.block_tokens = 2 * (rkv::kQueryBox / group);
    const long long per_seq = (static_cast<long long>(b->max_q) + p.block_tokens - 1) / p.block_tokens;
    p.n_blocks = static_cast<int>(std::min(static_cast<long long>(n_rows) / p.block_tokens + b->n_seqs,
                                           static_cast<long long>(b->n_seqs) * per_seq));
    // key tiles of one head are counted in 31 bits
    if (static_cast<long long>(p.n_blocks) * (b->max_kv / rkv::kKeyBox + 1LL) >= (1LL << 31)) {
      p.total = -1;
      return p;
    }
  }
  const long long heads = static_cast<long long>(n_rows) * q_heads;
  auto take = [&p](long long bytes) {
    const long long at = p.total;
    p.total += (bytes + 255) / 256 * 256;
    return at;
  };
  p.lse = weight ? take(4 * heads) : -1;
  p.blocks = p.work = p.seq_first = p.order = -1;
  p.n_joins = p.slot_rows ? 2 * rkv::kSmCount : rkv::kSmCount;  // thread blocks of the attention
  p.part_rows = p.slot_rows ? p.slot_rows : rkv::kPagedPartRows;
  // the rows of one tile, or two
  p.join_rows = b->max_q <= rkv::kQueryBox / group ? static_cast<int>(most) : rkv::kPagedPartRows;
  p.max_units = static_cast<long long>(p.slot_rows ? b->n_seqs : p.n_blocks) * pool->kv_heads;
  const long long rows = 2LL * p.n_joins * p.part_rows;
  p.part = take(4 * rows * kHeadDim);
  p.part_ml = take(8 * rows);
  p.ticket = take(4);
  p.joins = take(static_cast<long long>(sizeof(rkv::PagedJoin)) * p.n_joins);
  if (!p.slot_rows) {
    p.blocks = take(static_cast<long long>(sizeof(rkv::PagedBlock)) * p.n_blocks);
    p.work = take(sizeof(rkv::PagedWork));
    p.seq_first = take(4LL * b->n_seqs);
    if (weight && b->n_seqs <= rkv::kPagedMaxOrder) p.order = take(4LL * b->n_seqs);
  }
  p.score_stride = (b->max_kv + 63LL) / 64 * 64;
  // Scores are kept for at most 16 rows (8 bytes of traffic for each, where reading K again takes 256 for all of them),
  // but not past kMaxScores: their size goes by max_kv, which a captured step sets to the longest stream it may ever
  // see. The weights are then formed from K again, as for more rows. The limit is high, since that takes longer: 64
  // streams of 131072 tokens, 32 heads on 8 (1 GiB of scores), 5.8 ms with them and 13.7 without; of 4096 tokens,
  // 257 and 471 us; 24 of 8192 tokens, 169 and 353 us.
  p.scores = -1;
  if (weight && p.slot_rows == 16) {
    if (p.score_stride > 0 && heads > (1LL << 48) / p.score_stride)
      p.total = -1;  // pairs of rows and places are counted in 48 bits
    else if (4 * heads * p.score_stride <= kMaxScores)
      p.scores = take(4 * heads * p.score_stride);
  }
  return p;
}

// The pages as a tensor of 64-column boxes of min(page_tokens, tile) tokens.
bool encode_pages(CUtensorMap* m, const void* base, const rkv_page_pool* pool, int tile) {
  return rkv::encode_map(m, base, static_cast<uint64_t>(pool->kv_heads) * pool->page_tokens, pool->n_pages,
                         kHeadDim * 2, static_cast<uint64_t>(pool->page_stride) * 2,
                         std::min(pool->page_tokens, tile), 1);
}

// whether two row tensors of n rows share a byte range
bool overlap(const void* a, long long stride_a, const void* b, long long stride_b, int n, int heads) {
  const long long row = static_cast<long long>(heads) * kHeadDim;
  const char* a0 = static_cast<const char*>(a);
  const char* b0 = static_cast<const char*>(b);
  return a0 < b0 + 2 * ((n - 1) * stride_b + row) && b0 < a0 + 2 * ((n - 1) * stride_a + row);
}

}  // namespace

RKV_API int rkv_paged_write(const rkv_page_pool* pool, const rkv_paged_batch* batch, const void* k, const void* v,
                            int n_rows, long long k_stride, long long v_stride, void* stream) {
  const int rc = check_batch(pool, batch, n_rows, true);
  if (rc) return rc;
  if (static_cast<long long>(n_rows) * pool->kv_heads >= (1LL << 31)) return RKV_ERR_UNSUPPORTED;
  if (n_rows == 0 || batch->n_seqs == 0) return RKV_OK;
  if (!aligned16(k) || !aligned16(v) || !row_stride_ok(k_stride, pool->kv_heads) ||
      !row_stride_ok(v_stride, pool->kv_heads))
    return RKV_ERR_ARG;
  rkv::PagedWriteParams p;
  std::memset(&p, 0, sizeof(p));
  p.view = view_of(pool, batch, n_rows);
  p.k = static_cast<const uint16_t*>(k);
  p.v = static_cast<const uint16_t*>(v);
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  return cuda_rc(rkv::launch_paged_write(p, static_cast<cudaStream_t>(stream)));
}

RKV_API int rkv_paged_workspace(const rkv_page_pool* pool, const rkv_paged_batch* batch, int q_heads, int n_rows,
                                int with_weight, long long* bytes) {
  int rc = check_sizes(pool, batch, n_rows);
  if (rc) return rc;
  if (bytes == nullptr) return RKV_ERR_ARG;
  rc = check_heads(pool, q_heads, n_rows);
  if (rc) return rc;
  const long long total = plan_of(pool, batch, q_heads, n_rows, with_weight != 0).total;
  if (total < 0) return RKV_ERR_UNSUPPORTED;
  *bytes = total;
  return RKV_OK;
}

RKV_API int rkv_paged_attention(const rkv_page_pool* pool, const rkv_paged_batch* batch, const void* q, int q_heads,
                                int n_rows, long long q_stride, void* out, long long out_stride, int causal,
                                float* lse, float* weight, long long weight_stride, void* workspace,
                                long long workspace_bytes, void* stream) {
  int rc = check_batch(pool, batch, n_rows, true);
  if (rc) return rc;
  rc = check_heads(pool, q_heads, n_rows);
  if (rc) return rc;
  if (lse != nullptr && !aligned4(lse)) return RKV_ERR_ARG;
  if (weight != nullptr && (!aligned4(weight) || weight_stride < batch->max_kv)) return RKV_ERR_ARG;
  if (n_rows == 0 || batch->n_seqs == 0) return RKV_OK;
  if (!aligned16(q) || !aligned16(out) || !row_stride_ok(q_stride, q_heads) || !row_stride_ok(out_stride, q_heads) ||
      overlap(q, q_stride, out, out_stride, n_rows, q_heads))
    return RKV_ERR_ARG;
  const rkv::PagedPlan plan = plan_of(pool, batch, q_heads, n_rows, weight != nullptr);
  if (plan.total < 0) return RKV_ERR_UNSUPPORTED;
  if (workspace_bytes < plan.total) return RKV_ERR_CAPACITY;
  if (plan.total > 0 && !aligned16(workspace)) return RKV_ERR_ARG;
  rkv::PagedAttnParams p;
  std::memset(&p, 0, sizeof(p));
  p.view = view_of(pool, batch, n_rows);
  p.q = static_cast<const uint16_t*>(q);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.weight = weight;
  p.q_stride = q_stride;
  p.out_stride = out_stride;
  p.weight_stride = weight_stride;
  p.q_heads = q_heads;
  p.group = q_heads / pool->kv_heads;
  p.causal = causal != 0;
  p.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(kHeadDim)));
  char* ws = static_cast<char*>(workspace);
  if (plan.lse >= 0) p.lse2 = reinterpret_cast<float*>(ws + plan.lse);
  p.part = reinterpret_cast<float*>(ws + plan.part);
  p.part_ml = reinterpret_cast<float2*>(ws + plan.part_ml);
  p.ticket = reinterpret_cast<unsigned*>(ws + plan.ticket);
  p.joins = reinterpret_cast<rkv::PagedJoin*>(ws + plan.joins);
  p.n_joins = plan.n_joins;
  p.part_rows = plan.part_rows;
  p.join_rows = plan.join_rows;
  p.max_units = plan.max_units;
  if (plan.blocks >= 0) {
    p.blocks = reinterpret_cast<rkv::PagedBlock*>(ws + plan.blocks);
    p.work = reinterpret_cast<rkv::PagedWork*>(ws + plan.work);
    p.seq_first = reinterpret_cast<int*>(ws + plan.seq_first);
    if (plan.order >= 0) p.order = reinterpret_cast<int*>(ws + plan.order);
  }
  if (plan.scores >= 0) p.scores = reinterpret_cast<float*>(ws + plan.scores);
  p.score_stride = plan.score_stride;
  p.slot_rows = plan.slot_rows;
  p.block_tokens = plan.block_tokens;
  p.n_blocks = plan.n_blocks;
  p.wait_limit_ns = kWaitNs;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t err;
  CUtensorMap tm_q, tm_k, tm_v;
  const int tile = plan.slot_rows ? rkv::kPagedDecodeTile : rkv::kKeyBox;
  const bool weigh = weight != nullptr && batch->max_kv > 0, from_scores = plan.scores >= 0;
  if (!encode_pages(&tm_k, pool->k, pool, tile) || !encode_pages(&tm_v, pool->v, pool, tile)) return RKV_ERR_CUDA;
  if (!plan.slot_rows || (weigh && !from_scores)) {
    if (!rkv::encode_map(&tm_q, q, q_heads, n_rows, kHeadDim * 2, static_cast<uint64_t>(q_stride) * 2, p.group,
                         rkv::kQueryBox / p.group))
      return RKV_ERR_CUDA;
  }
  err = plan.slot_rows ? rkv::launch_paged_decode(tm_k, tm_v, p, st) : rkv::launch_paged_chunk(tm_q, tm_k, tm_v, p, st);
  if (err == cudaSuccess) err = rkv::launch_paged_join(p, st);
  if (err == cudaSuccess && weigh) {
    if (from_scores) {
      err = rkv::launch_paged_token_weight(p, st);
    } else {
      if (plan.slot_rows && !encode_pages(&tm_k, pool->k, pool, rkv::kKeyBox)) return RKV_ERR_CUDA;
      err = rkv::launch_paged_weight(tm_q, tm_k, p, st);
    }
  }
  return cuda_rc(err);
}

RKV_API int rkv_paged_evict(const rkv_page_pool* pool, const rkv_paged_batch* batch, float* weight,
                            long long weight_stride, int keep, int sinks, int recent, int* kept, int* kv_len_out,
                            void* stream) {
  const int rc = check_batch(pool, batch, 0, false);
  if (rc) return rc;
  if (keep < 1 || sinks < 0 || recent < 0 || static_cast<long long>(sinks) + recent > keep) return RKV_ERR_ARG;
  if (keep > (1 << 30)) return RKV_ERR_UNSUPPORTED;
  if (batch->n_seqs == 0) return RKV_OK;
  if (!aligned4(weight) || weight_stride < batch->max_kv || !aligned4(kept) || !aligned4(kv_len_out))
    return RKV_ERR_ARG;
  rkv::PagedEvictParams p;
  std::memset(&p, 0, sizeof(p));
  p.view = view_of(pool, batch, 0);
  p.weight = weight;
  p.weight_stride = weight_stride;
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  p.kept = kept;
  p.kv_len_out = kv_len_out;
  return cuda_rc(rkv::launch_paged_evict(p, static_cast<cudaStream_t>(stream)));
}

RKV_API int rkv_paged_poll_status(unsigned* status, void* stream) {
  if (!aligned4(status)) return RKV_ERR_ARG;
  // all in the stream's order: a clear on another stream could wipe out what this one's next kernel reports
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  unsigned word = 0;
  cudaError_t err = cudaMemcpyAsync(&word, status, sizeof(word), cudaMemcpyDeviceToHost, st);
  if (err == cudaSuccess) err = cudaStreamSynchronize(st);
  if (err == cudaSuccess && word != 0) err = cudaMemsetAsync(status, 0, sizeof(word), st);
  if (err != cudaSuccess) return cuda_rc(err);
  if (word & rkv::kStatusTimeout) return RKV_ERR_TIMEOUT;
  return (word & (rkv::kStatusPage | rkv::kStatusLength)) ? RKV_ERR_PAGE : RKV_OK;
}
