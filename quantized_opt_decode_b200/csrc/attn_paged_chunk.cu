// Attention of a ragged batch of new tokens over the paged cache:
// o = softmax(q K^T / sqrt(d)) V over positions 0..p for the row at position p.
//
// One warp per (row, query head): d/32 dimensions per lane, one token at a time
// with a running maximum and sum.
#include <math.h>

#include "paged.cuh"

namespace flexq {
namespace {

constexpr int kWarps = 4;

struct PagedAttnArgs {
  PagedView kv;
  RaggedView batch;
  int heads, group;
  int min_rows;
  const __half* q;
  int ldq;
  __half* out;
  int ldo;
  float scale_log2;
  uint32_t* err;
};

__device__ __forceinline__ float dq(uint32_t code, __half2 ms) {
  const float2 m = __half22float2(ms);
  return __half2float(__float2half_rn(__fadd_rn(__fmul_rn(static_cast<float>(code), m.y), m.x)));
}

template <int D, bool Q4>
__global__ void __launch_bounds__(kWarps * 32) attn_paged_rows_kernel(const PagedAttnArgs a) {
  constexpr int VEC = D / 32;
  pdl_wait();
  const int lane = static_cast<int>(lane_id());
  const long long w = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (w >= static_cast<long long>(a.batch.rows) * a.heads) return;
  const int row = static_cast<int>(w / a.heads), head = static_cast<int>(w % a.heads);
  const int i = find_unit_owner(a.batch, row, 1, 0, 0);
  if (i < 0) return;
  const Span sp = ragged_span(a.batch, i, a.err);
  if (sp.n * a.group < a.min_rows) return;
  if (row >= sp.row0 + sp.n) return;
  const int pos = sp.len - sp.n + row - sp.row0;
  const int j = head / a.group;
  const int e0 = lane * VEC;
  float q[VEC], o[VEC], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    q[e] = __half2float(a.q[static_cast<size_t>(row) * a.ldq + head * D + e0 + e]) * a.scale_log2;
    o[e] = 0.f;
  }
  for (int p = 0; p <= pos; ++p) {
    const int page = page_of(a.kv, i, p, a.err);
    if (page < 0) return;
    const size_t slot = pool_slot(a.kv, page, j, p);
    float k[VEC], v[VEC];
    if (Q4) {
      const __half2 km = static_cast<const __half2*>(a.kv.k_meta)[slot * (D / 64) + e0 / 64];
      const __half2 vm = static_cast<const __half2*>(a.kv.v_meta)[slot * (D / 64) + e0 / 64];
      const uint8_t* kc = static_cast<const uint8_t*>(a.kv.k) + slot * (D / 2) + e0 / 2;
      const uint32_t* vw = static_cast<const uint32_t*>(a.kv.v) + (slot >> 3) * D + e0;
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        k[e] = dq((kc[e / 2] >> (4 * (e & 1))) & 0xFu, km);
        v[e] = dq((vw[e] >> (4 * (p & 7))) & 0xFu, vm);
      }
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        k[e] = __half2float(static_cast<const __half*>(a.kv.k)[slot * D + e0 + e]);
        v[e] = __half2float(static_cast<const __half*>(a.kv.v)[slot * D + e0 + e]);
      }
    }
    float s = 0.f;
#pragma unroll
    for (int e = 0; e < VEC; ++e) s += q[e] * k[e];
    s = warp_sum(s);
    const float mn = fmaxf(m, s);
    const float al = exp2f(m - mn), pr = exp2f(s - mn);
    l = l * al + pr;
#pragma unroll
    for (int e = 0; e < VEC; ++e) o[e] = o[e] * al + pr * v[e];
    m = mn;
  }
  const float inv = 1.f / l;
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    a.out[static_cast<size_t>(row) * a.ldo + head * D + e0 + e] = __float2half_rn(o[e] * inv);
}

}  // namespace

cudaError_t launch_attn_paged_chunks(const PagedView& kv, const RaggedView& batch, int heads, int d, int kv_bits, int min_rows,
                              const __half* q, int ldq, __half* out, int ldo, cudaStream_t s) {
  PagedAttnArgs a{kv,  batch, heads, heads / kv.kv_heads, min_rows, q, ldq,
                  out, ldo,   1.4426950408889634f / sqrtf(static_cast<float>(d)), runtime().err};
  const long long warps = static_cast<long long>(batch.rows) * heads;
  const dim3 grid(static_cast<unsigned>((warps + kWarps - 1) / kWarps));
  if (kv_bits == 4)
    return d == 128 ? launch_pdl(attn_paged_rows_kernel<128, true>, grid, kWarps * 32, 0, s, a)
                    : launch_pdl(attn_paged_rows_kernel<64, true>, grid, kWarps * 32, 0, s, a);
  return d == 128 ? launch_pdl(attn_paged_rows_kernel<128, false>, grid, kWarps * 32, 0, s, a)
                  : launch_pdl(attn_paged_rows_kernel<64, false>, grid, kWarps * 32, 0, s, a);
}

}  // namespace flexq
