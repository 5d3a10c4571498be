// Device-side walk over a ragged batch and its page table, shared by the paged
// cache's kernels.
#pragma once

#include "common.cuh"
#include "kernels_serving.h"
#include "paged_math.h"

namespace flexq {

// The new tokens of one sequence: rows row0 .. row0 + n - 1 of the token
// buffers, positions len - n .. len - 1.
struct Span {
  int row0, n, len;
};

// Span of sequence i; n = 0 when it brings nothing or breaks the batch's
// bounds (then the device error word is set).
__device__ __forceinline__ Span ragged_span(const RaggedView& r, int i, uint32_t* err) {
  Span s;
  s.row0 = r.row_start[i];
  s.n = r.row_start[i + 1] - s.row0;
  s.len = r.kv_len[i];
  if (s.n == 0) return s;
  if (!span_ok(s.row0, s.n, s.len, r.rows, r.max_new, r.max_len)) {
    set_error(err, DEV_BAD_ARGUMENT);
    s.n = 0;
  }
  return s;
}

// Looks at every sequence, by one warp: a start table that decreases gives some of them no unit,
// and they are to be reported all the same.
__device__ __forceinline__ void check_spans(const RaggedView& r, uint32_t* err) {
  for (int i = static_cast<int>(lane_id()); i < r.b; i += 32) ragged_span(r, i, err);
}

// First unit of 2^shift rows of sequence i.
__device__ __forceinline__ long long unit_base(const RaggedView& r, int i, int shift, int extra) {
  return unit_base_at(r.row_start[i], i, 1, shift, extra);
}

// Sequence that owns unit u: the last i in 0 .. b-1 with unit_base(i) <= u,
// found 32 probes at a time by the whole warp.  -1: none.
__device__ __forceinline__ int find_unit_owner(const RaggedView& r, long long u, int shift, int extra) {
  const int lane = static_cast<int>(lane_id());
  int lo = 0, hi = r.b;  // the owner, if any, is in [lo, hi)
  while (hi - lo > 32) {
    const int step = (hi - lo + 31) / 32;
    const int p = lo + lane * step;
    const bool le = p < hi && unit_base(r, p, shift, extra) <= u;
    const int cnt = __popc(__ballot_sync(0xffffffffu, le));
    if (cnt == 0) return -1;
    lo += (cnt - 1) * step;
    hi = min(hi, lo + step);
  }
  const int p = lo + lane;
  const bool le = p < hi && unit_base(r, p, shift, extra) <= u;
  const int cnt = __popc(__ballot_sync(0xffffffffu, le));
  return cnt == 0 ? -1 : lo + cnt - 1;
}

// Page of position `pos` of sequence i, or -1 (error word set) when the
// table names a page outside the pool.
__device__ __forceinline__ int page_of(const PagedView& kv, int i, int pos, uint32_t* err) {
  const int p = kv.table[static_cast<size_t>(i) * kv.table_ld + (pos >> kv.page_shift)];
  if (page_ok(p, kv.num_pages)) return p;
  set_error(err, DEV_BAD_ARGUMENT);
  return -1;
}

// Slot index of the pool's [num_pages][kv_heads][page_size] order.
__device__ __forceinline__ size_t pool_slot(const PagedView& kv, int page, int head, int pos) {
  return ((static_cast<size_t>(page) * kv.kv_heads + head) << kv.page_shift) +
         (pos & ((1 << kv.page_shift) - 1));
}

}  // namespace flexq
