// Index arithmetic of the paged cache's kernels that needs no GPU: which
// sequences and pages a kernel accepts, and how a ragged batch is cut into
// units.  (Plain C++, so that it can be checked on the host.)
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define FQ_HD __host__ __device__ __forceinline__
#else
#define FQ_HD inline
#endif

namespace flexq {

// Whether a sequence of n > 0 new tokens in rows row0 .. row0 + n - 1 and of
// length len keeps the batch's bounds: then its rows lie in the token buffers and
// its positions in its table row.
FQ_HD bool span_ok(int row0, int n, int len, int rows, int max_new, int max_len) {
  return row0 >= 0 && n > 0 && n <= max_new && n <= rows && row0 <= rows - n && len >= n && len <= max_len;
}

FQ_HD bool page_ok(int page, int num_pages) { return page >= 0 && page < num_pages; }

// Work on a ragged batch is cut into units of 2^shift of the sequence's
// (rows * scale) items.  Sequence i owns the unit numbers from
// floor(scale * row_start[i] / 2^shift) + extra * i up to the next sequence's
// first: enough for its items whatever their phase (floor(a + b) - floor(a) >=
// floor(b)), known without a prefix sum, and at most scale * rows / 2^shift +
// extra * b numbers in all; a few at a sequence's end stay empty.
FQ_HD long long unit_base_at(int row_start_i, int i, int scale, int shift, int extra) {
  return ((static_cast<long long>(row_start_i) * scale) >> shift) + static_cast<long long>(extra) * i;
}

FQ_HD long long unit_total(int rows, int b, int scale, int shift, int extra) {
  return ((static_cast<long long>(rows) * scale) >> shift) + static_cast<long long>(extra) * b;
}

}  // namespace flexq
