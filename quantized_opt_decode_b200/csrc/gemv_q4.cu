// Few-row linear layer with a 4-bit weight in the tiled layout:
// Y[m][n] = epilogue(X[m][k] W^T), m <= 16, w = fp16(fp32(code * scale) + min).
//
// One warp per output feature: the lanes share out the 8-code words of the
// feature's row, each word dequantized once and used for every row of X.
#include "common.cuh"
#include "kernels.h"

namespace flexq {
namespace {

constexpr int kWarps = 4;

struct GemvArgs {
  const __half* x;
  int ldx;
  const uint8_t* w;
  int m, n, k;
  const __half* bias;
  const __half* residual;
  int ld_res;
  int epi;
  void* y;
  int ldy;
};

__device__ __forceinline__ void store_out(const GemvArgs& a, int row, int col, float v) {
  if (a.epi & EPI_BIAS) v += __half2float(a.bias[col]);
  if (a.epi & EPI_GELU) v = 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
  if (a.epi & EPI_RESIDUAL) v += __half2float(a.residual[static_cast<size_t>(row) * a.ld_res + col]);
  if (a.epi & EPI_F32_OUT)
    static_cast<float*>(a.y)[static_cast<size_t>(row) * a.ldy + col] = v;
  else
    static_cast<__half*>(a.y)[static_cast<size_t>(row) * a.ldy + col] = __float2half_rn(v);
}

__global__ void __launch_bounds__(kWarps * 32) gemv_rows_kernel(const GemvArgs a) {
  pdl_wait();
  const int lane = static_cast<int>(lane_id());
  const int f = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (f >= a.n) return;
  const int kb = a.k / 64;
  const uint8_t* tile = a.w + static_cast<size_t>(f / kTileRows) * kb * kTileBytes;
  const int r = f % kTileRows;
  float acc[kGemvMaxRows];
#pragma unroll
  for (int t = 0; t < kGemvMaxRows; ++t) acc[t] = 0.f;
  for (int wd = lane; wd < a.k / 8; wd += 32) {
    const uint8_t* blk = tile + static_cast<size_t>(wd / 8) * kTileBytes;
    const uint32_t word = reinterpret_cast<const uint32_t*>(blk)[r * 8 + (wd & 7)];
    const float2 ms = __half22float2(reinterpret_cast<const __half2*>(blk + kTileCodeBytes)[r]);
    float w[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float c = static_cast<float>((word >> (4 * ((e >> 1) + 4 * (e & 1)))) & 0xFu);
      w[e] = __half2float(__float2half_rn(__fadd_rn(__fmul_rn(c, ms.y), ms.x)));
    }
#pragma unroll
    for (int t = 0; t < kGemvMaxRows; ++t) {
      if (t >= a.m) break;
      const uint4 raw = *reinterpret_cast<const uint4*>(a.x + static_cast<size_t>(t) * a.ldx + wd * 8);
      const __half2* h = reinterpret_cast<const __half2*>(&raw);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 x = __half22float2(h[e]);
        acc[t] += w[2 * e] * x.x + w[2 * e + 1] * x.y;
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kGemvMaxRows; ++t) {
    if (t >= a.m) break;
    const float v = warp_sum(acc[t]);
    if (lane == 0) store_out(a, t, f, v);
  }
}

}  // namespace

cudaError_t launch_gemv_q4(const __half* x, int ldx, const uint8_t* w, int m, int n, int k, const __half* bias,
                           const __half* residual, int ld_res, int epi, void* y, int ldy, cudaStream_t s) {
  const GemvArgs a{x, ldx, w, m, n, k, bias, residual, ld_res, epi, y, ldy};
  return launch_pdl(gemv_rows_kernel, dim3((n + kWarps - 1) / kWarps), kWarps * 32, 0, s, a);
}

}  // namespace flexq
