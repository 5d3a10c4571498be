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

// The chunk kernel's units: kUnitRows consecutive query rows of a sequence and key/value head (rows = n
// new tokens times `group` query heads, at most 2^30), and the key tiles that they see.
// `first` is the position of the first new token.
constexpr int kUnitRowShift = 8;
constexpr int kUnitRows = 1 << kUnitRowShift;
constexpr int kKeyTile = 128;

FQ_HD int row_units(int rows) { return (rows + kUnitRows - 1) / kUnitRows; }

// Rows of the unit that starts at row c0.
FQ_HD int unit_rows(int rows, int c0) { return rows - c0 < kUnitRows ? rows - c0 : kUnitRows; }

// Key tiles that its last row sees.
FQ_HD int unit_tiles(int first, int group, int c0, int rows) { return (first + (c0 + rows - 1) / group + kKeyTile) / kKeyTile; }

// How many of the `units` of a sequence of n new tokens (no units: it is not the kernel's) see at
// least `tiles` (> 0) tiles: its last ones, from the row on whose token is at or behind `need`.
FQ_HD int long_units(int first, int n, int group, int units, int tiles) {
  const int need = kKeyTile * (tiles - 1) - first;
  return units == 0 || need >= n ? 0 : need <= 0 ? units : units - need * group / kUnitRows;
}

// How many of `tiles` tiles fall to CTA `rank` of a cluster of `splits`: rank, rank + splits, ..
FQ_HD int share_tiles(int tiles, int rank, int splits) { return tiles > rank ? (tiles - rank + splits - 1) / splits : 0; }

}  // namespace flexq
