// Launch entry points of the serving kernels: paged cache, ragged attention,
// few-row product.
#pragma once

#include "kernels.h"

namespace flexq {

// Paged cache (page_size = 1 << page_shift slots) and ragged batch, as
// include/flexq.h describes them.
struct PagedView {
  void *k, *v, *k_meta, *v_meta;
  int kv_heads, num_pages, page_shift;
  const int32_t* table;
  int table_ld;
};
struct RaggedView {
  int b, rows, max_new, max_len;
  const int32_t* row_start;
  const int32_t* kv_len;
};
struct RopeView {
  const float* cos_sin;  // NULL: no rotation
  int max_pos, rot_dim, interleaved;
};
cudaError_t launch_paged_append(const PagedView& kv, const RaggedView& batch, const RopeView& rope, int heads, int d,
                                int kv_bits, const __half* k, const __half* v, int ld, const __half* q, int ldq,
                                __half* q_out, int ldqo, cudaStream_t s);
cudaError_t launch_paged_read(const PagedView& kv, const RaggedView& batch, int d, int kv_bits, __half* k_out,
                              __half* v_out, int ld, cudaStream_t s);
cudaError_t launch_attn_paged(const PagedView& kv, const RaggedView& batch, int heads, int d, int kv_bits,
                              const __half* q, int ldq, __half* out, int ldo, cudaStream_t s);
// Its sequences with at least min_rows query rows to a key/value head.
cudaError_t launch_attn_paged_chunks(const PagedView& kv, const RaggedView& batch, int heads, int d, int kv_bits,
                                     int min_rows, const __half* q, int ldq, __half* out, int ldo, cudaStream_t s);

// Few-row product with a 4-bit tiled weight.
constexpr int kGemvMaxRows = 16;
cudaError_t launch_gemv_q4(const __half* x, int ldx, const uint8_t* w, int m, int n, int k, const __half* bias,
                           const __half* residual, int ld_res, int epi, void* y, int ldy, cudaStream_t s);

}  // namespace flexq
