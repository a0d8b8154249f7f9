// Internal interface between the paged caches' host side (rkv_paged_host.cpp) and their kernels
// (rkv_paged.cu, rkv_paged_decode.cu, rkv_paged_attention.cu, rkv_paged_join.cu). Not installed.
#pragma once

#include "rkv_internal.h"
#include "tensor_map.h"

namespace rkv {

// Device status word bits, beside kStatusTimeout.
constexpr unsigned kStatusPage = 2u;    // a page id outside the pool
constexpr unsigned kStatusLength = 4u;  // a length or row range outside its bound

// What every paged kernel needs of the pool and the batch (include/rkv.h, rkv_page_pool and
// rkv_paged_batch).
struct PagedView {
  uint16_t* k;
  uint16_t* v;
  long long page_stride;
  const int* table;
  const int* kv_len;
  const int* q_start;
  unsigned* status;
  int n_pages, kv_heads, page_shift;  // page_tokens = 1 << page_shift
  int table_stride, n_seqs, n_rows, max_q, max_kv;
};

constexpr int kSmCount = 148;

struct PagedWriteParams {
  PagedView view;
  const uint16_t* k;
  const uint16_t* v;
  long long k_stride, v_stride;
};

// How a call is cut up (a host rule on the batch's host values; workspace offsets in bytes).
struct PagedPlan {
  int slot_rows;     // single-token form: rows of a stream and KV head, rounded up to 16 or 32; 0: chunk form
  int block_tokens;  // chunk form: tokens of one unit of rows
  int n_blocks;      // and such units of one KV head in the batch at most
  long long lse, part, part_ml, scores, joins, blocks, work, seq_first, order, ticket, total;  // -1: not used
  long long score_stride;
  int n_joins, part_rows, join_rows;
  long long max_units;  // units of work at most
};

constexpr int kPagedRows = 32;  // rows of the single-token form at most

// Work of the chunk form, laid out on the device by a small kernel from the lengths of the moment
// (workspace). A block of up to block_tokens chunk tokens of one stream, for every KV head the same:
struct PagedBlock {
  int row0, cnt;  // first row of the chunk tensors, tokens
  int keys;       // cached tokens that its last row sees
  int place0;     // the last place that its first row sees
  int seq;
  int start;      // key tiles of the blocks before it (one KV head)
  int tiles;      // key tiles, at least 1
  int unused;
};
// How the thread blocks share them. In a row: block c of n_ctas walks an even share (PagedShares) of
// all heads' tiles. In step (units of nearly one size): every thread block takes `waves` whole units; of the
// last n_tail, thread block i < n_tail takes the first `quota` tiles of unit i, and the others share
// what is left of them, `quota` tiles each, in a row.
struct PagedShare {  // one thread block's
  long long left;  // tiles (in step: of the last units)
  int h, b, t;     // in a row: head, block and tile of its first
  int i, pos;      // in step, sharing leftovers: the last unit it begins in, and its first leftover tile
  int unused;
};
// A unit that thread blocks shared: parts in slots slot0, slot0 + 1, slot0 + 1 + step, ... (parts 0: none)
struct __align__(16) PagedJoin {
  int row0, cnt, h;  // its first row of the chunk tensors, tokens, head
  int slot0, step, parts;
  int unused[2];
};
struct PagedWork {
  int n_blocks;
  int n_ctas;
  int in_step;
  int waves, n_tail, quota;
  int rest[kSmCount + 2];  // in step: tiles left of the last units before unit i
  PagedShare share[kSmCount];
};
constexpr int kPagedMaxOrder = 1024;  // streams that the plan puts in order at most
constexpr int kPagedPartRows = 256;  // rows of a partial result of the chunk form

struct PagedAttnParams {
  PagedView view;
  const uint16_t* q;
  uint16_t* out;
  float* lse;     // [n_rows][q_heads], natural log; null: not wanted
  float* weight;  // [n_seqs][kv_heads][weight_stride]; null: not wanted
  long long q_stride, out_stride, weight_stride;
  int q_heads, group, causal;
  float scale_log2;  // log2(e) / sqrt(d)
  // workspace
  float* lse2;      // [n_rows][q_heads], log2; null when no weight is wanted
  float* part;      // unnormalised sums of p v of cut units: [4 * kSmCount][slot_rows][128] (single-token
                    // form) or [2 * kSmCount][kPagedPartRows * 128] (paged_part_place)
  float2* part_ml;  // the same rows: reference (log2) and sum of p
  PagedJoin* joins;    // [n_joins], an entry per thread block of the attention
  PagedBlock* blocks;  // chunk form: [n_blocks]
  PagedWork* work;
  unsigned* ticket;    // units that the chunks' weight kernel has drawn
  int* seq_first;      // chunk form: [n_seqs], the stream's first block
  int* order;          // chunk form: [n_seqs], the streams by falling chunk length; null: as they come
  float* scores;    // [n_rows][q_heads][score_stride]: log2 scores of the single-token form; null: not kept
  long long score_stride;
  int n_joins, part_rows, join_rows;  // join_rows: rows of a part that are used at most
  long long max_units;
  int slot_rows;                // single-token form
  int block_tokens, n_blocks;  // chunk form
  unsigned long long wait_limit_ns;
};

struct PagedEvictParams {
  PagedView view;
  float* weight;
  long long weight_stride;
  int keep, sinks, recent;
  int* kept;
  int* kv_len_out;
};

cudaError_t launch_paged_write(const PagedWriteParams& p, cudaStream_t stream);
// tm_k, tm_v: boxes of min(page_tokens, kPagedDecodeTile) tokens, 64 columns.
constexpr int kPagedDecodeTile = 64;
cudaError_t launch_paged_decode(const CUtensorMap& tm_k, const CUtensorMap& tm_v, const PagedAttnParams& p,
                                cudaStream_t stream);
// tm_q: boxes of 64 columns, the group's heads and floor(128 / group) tokens; tm_k, tm_v: boxes of
// min(page_tokens, kKeyBox) tokens.
cudaError_t launch_paged_chunk(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const CUtensorMap& tm_v,
                               const PagedAttnParams& p, cudaStream_t stream);
// adds up what the thread blocks of either left in parts
cudaError_t launch_paged_join(const PagedAttnParams& p, cudaStream_t stream);
cudaError_t launch_paged_weight(const CUtensorMap& tm_q, const CUtensorMap& tm_k, const PagedAttnParams& p,
                                cudaStream_t stream);
cudaError_t launch_paged_token_weight(const PagedAttnParams& p, cudaStream_t stream);
cudaError_t launch_paged_evict(const PagedEvictParams& p, cudaStream_t stream);

}  // namespace rkv
