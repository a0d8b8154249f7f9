// Device helpers shared by the paged-cache kernels: which stream a chunk row belongs to, the
// checked lengths of a stream, the address of a cached token.
#pragma once

#include <utility>

#include "rkv_internal.h"

namespace rkv {

// Launch a kernel that may be set up while the stream's previous one still runs; it waits for that one
// itself (ptx::wait_previous, in every thread block, before it touches memory).
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
    const bool le = i < hi && __ldg(w.q_start + i) <= row;
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
  int q0, n_q, kv;  // first chunk row, chunk rows, cached tokens
  bool ok;
};

// The lengths of stream s, checked against the batch's bounds.
__device__ __forceinline__ PagedSeq paged_seq(const PagedView& w, int s) {
  PagedSeq r;
  r.q0 = __ldg(w.q_start + s);
  const int q1 = __ldg(w.q_start + s + 1);
  r.kv = __ldg(w.kv_len + s);
  r.ok = r.q0 >= 0 && q1 >= r.q0 && q1 <= w.n_rows && q1 - r.q0 <= w.max_q && r.kv >= 0 && r.kv <= w.max_kv;
  r.n_q = q1 - r.q0;
  return r;
}

// Page id at place `i` of stream s's list, or -1 (reported) if it is not a page of the pool.
__device__ __forceinline__ int paged_id(const PagedView& w, int s, int i) {
  const int id = __ldg(w.table + static_cast<long long>(s) * w.table_stride + i);
  if (static_cast<unsigned>(id) < static_cast<unsigned>(w.n_pages)) return id;
  paged_report(w, kStatusPage);
  return -1;
}

// Element offset of token `slot` (place within the page) of KV head h in page `id`.
__device__ __forceinline__ long long paged_offset(const PagedView& w, int id, int h, int slot) {
  return static_cast<long long>(id) * w.page_stride +
         (static_cast<long long>(h) * (1 << w.page_shift) + slot) * kHeadDim;
}

}  // namespace rkv
