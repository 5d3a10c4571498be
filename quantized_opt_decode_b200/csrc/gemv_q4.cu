// Few-row linear layer with a 4-bit weight in the tiled layout:
// Y[m][n] = epilogue(X[m][k] W^T), m <= 16, w = code * scale + min rounded once
// to fp16, fp32 sums.
//
// The weight is read once (n k / 2 bytes of codes and n k / 16 of pairs) and that
// is the bound; the rows of X are the B operand of mma.sync (8 columns an
// instruction, one or two of them), so the arithmetic does not grow with m.  A CTA owns 16 MT
// features; its warps share out the K axis in steps of two 64-wide k-blocks, each
// through its own ring of asynchronous 16-byte copies (codes, pairs and the rows'
// 128 columns), so no warp waits for another before the end, where the warps'
// sums are joined in a fixed order.
#include "warp_mma.cuh"

namespace flexq {
namespace {

constexpr int kStages = 4;

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
  int stage_bytes;
};

// Stage of one K step (128 columns): codes [2 blocks][16 MT rows][32 B] with
// the second block's 16-byte units XORed by 4, pairs [2][16 MT] (rows of
// kMetaStride bytes), rows of X [m][256 B] with unit u of row i at u ^ (u/8*2) ^ (i%2):
// each eight lanes of a 16-byte read then touch eight different bank groups.
template <int MT>
struct Stage {
  static constexpr int codes = 2 * MT * 16 * 32;
  static constexpr int meta_stride = MT * 16 * 4 + 16;
  static constexpr int x0 = codes + 2 * meta_stride;
  static int bytes(int m) { return x0 + m * 256; }
};

template <int MT>
__device__ __forceinline__ void load_step(const GemvArgs& a, const uint8_t* tile, int rb, int sb, uint32_t st, int lane) {
  using S = Stage<MT>;
  const int kb0 = sb * 2, kbs = a.k / 64;
#pragma unroll
  for (int i = 0; i < 2 * MT; ++i) {
    constexpr int U = MT * 32;  // 16-byte units of a block's rows
    const int idx = lane + 32 * i, b = idx / U, u = idx % U;
    const bool ok = kb0 + b < kbs;
    const uint8_t* src = tile + static_cast<size_t>(ok ? kb0 + b : 0) * kTileBytes + rb * 32 + u * 16;
    cp_async16(st + b * U * 16 + ((u ^ (b << 2)) * 16), src, ok);
  }
  if (lane < 8 * MT) {
    const int b = lane / (4 * MT), c = lane % (4 * MT);
    const bool ok = kb0 + b < kbs;
    const uint8_t* src = tile + static_cast<size_t>(ok ? kb0 + b : 0) * kTileBytes + kTileCodeBytes + rb * 4 + c * 16;
    cp_async16(st + S::codes + b * S::meta_stride + c * 16, src, ok);
  }
  for (int idx = lane; idx < a.m * 16; idx += 32) {
    const int i = idx >> 4, u = idx & 15;
    const int col = sb * 128 + u * 8;
    const bool ok = col < a.k;
    cp_async16(st + S::x0 + i * 256 + ((u ^ ((u >> 3) << 1) ^ (i & 1)) * 16),
               a.x + static_cast<size_t>(i) * a.ldx + (ok ? col : 0), ok);
  }
}

template <int MT, int NT>
__global__ void __launch_bounds__(512) gemv_q4_kernel(const GemvArgs a) {
  using S = Stage<MT>;
  extern __shared__ __align__(16) uint8_t smem[];
  pdl_wait();
  const int lane = static_cast<int>(lane_id()), warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int r = lane >> 2, j = lane & 3;
  const int f0 = blockIdx.x * 16 * MT;
  const uint8_t* tile = a.w + static_cast<size_t>(f0 / kTileRows) * (a.k / 64) * kTileBytes;
  const int rb = f0 % kTileRows;
  const int steps = (a.k + 127) / 128;
  const uint32_t ring = smem_u32(smem) + warp * kStages * a.stage_bytes;

  float acc[MT][NT][4];
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;

  int sb_load = warp;
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) {
    if (sb_load < steps) load_step<MT>(a, tile, rb, sb_load, ring + s * a.stage_bytes, lane);
    cp_commit();
    sb_load += warps;
  }
  int slot = 0;
  for (int sb = warp; sb < steps; sb += warps) {
    cp_wait<kStages - 2>();
    __syncwarp();
    {
      int to = slot + kStages - 1;
      to = to >= kStages ? to - kStages : to;
      if (sb_load < steps) load_step<MT>(a, tile, rb, sb_load, ring + to * a.stage_bytes, lane);
      cp_commit();
      sb_load += warps;
    }
    const uint32_t st = ring + slot * a.stage_bytes;
    slot = slot + 1 == kStages ? 0 : slot + 1;
    // lane (r, j): 32 columns 32j .. 32j + 31 of the step, for rows r and r + 8 of
    // each 16 features and for rows r (and r + 8) of X
    const int b = j >> 1;
    uint4 cw[MT][2];
    __half2 sc[MT][2], mn[MT][2];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int row = mt * 16 + h * 8 + r;
        cw[mt][h] = lds128(st + b * MT * 512 + (((row * 2 + (j & 1)) ^ (b << 2)) * 16));
        const uint32_t ms = lds32(st + S::codes + b * S::meta_stride + row * 4);
        const __half2 p = *reinterpret_cast<const __half2*>(&ms);
        mn[mt][h] = __low2half2(p);
        sc[mt][h] = __high2half2(p);
      }
#pragma unroll
    for (int wd = 0; wd < 4; ++wd) {
      uint4 x[NT];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int i = nt * 8 + r, u = 4 * j + wd;
        // rows past m are columns of the product that nobody reads
        x[nt] = i < a.m ? lds128(st + S::x0 + i * 256 + ((u ^ ((u >> 3) << 1) ^ (i & 1)) * 16)) : make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t lo[4], hi[4];
        const uint32_t w0 = wd == 0 ? cw[mt][0].x : wd == 1 ? cw[mt][0].y : wd == 2 ? cw[mt][0].z : cw[mt][0].w;
        const uint32_t w1 = wd == 0 ? cw[mt][1].x : wd == 1 ? cw[mt][1].y : wd == 2 ? cw[mt][1].z : cw[mt][1].w;
        dequant_word(w0, sc[mt][0], mn[mt][0], lo);
        dequant_word(w1, sc[mt][1], mn[mt][1], hi);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          mma_16816(acc[mt][nt], lo[0], hi[0], lo[1], hi[1], x[nt].x, x[nt].y);
          mma_16816(acc[mt][nt], lo[2], hi[2], lo[3], hi[3], x[nt].z, x[nt].w);
        }
      }
    }
  }
  cp_wait<0>();
  __syncthreads();
  pdl_trigger();
  // sums of the warps: [warp][8 NT rows][16 MT features + 1]
  constexpr int F = 16 * MT, LD = F + 1;
  float* red = reinterpret_cast<float*>(smem);
  {
    float* mine = red + warp * 8 * NT * LD;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          mine[(nt * 8 + 2 * j + (e & 1)) * LD + mt * 16 + (e >> 1) * 8 + r] = acc[mt][nt][e];
  }
  __syncthreads();
  for (int o = threadIdx.x; o < a.m * F; o += blockDim.x) {
    const int row = o / F, f = o % F;
    const int col = f0 + f;
    if (col >= a.n) continue;
    float v = 0.f;
    for (int w = 0; w < warps; ++w) v += red[(w * 8 * NT + row) * LD + f];
    if (a.epi & EPI_BIAS) v += __half2float(a.bias[col]);
    if (a.epi & EPI_GELU) v = 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    if (a.epi & EPI_RESIDUAL) v += __half2float(a.residual[static_cast<size_t>(row) * a.ld_res + col]);
    if (a.epi & EPI_F32_OUT)
      static_cast<float*>(a.y)[static_cast<size_t>(row) * a.ldy + col] = v;
    else
      static_cast<__half*>(a.y)[static_cast<size_t>(row) * a.ldy + col] = __float2half_rn(v);
  }
}

template <int MT, int NT>
cudaError_t launch_gemv(GemvArgs a, int warps, cudaStream_t s) {
  a.stage_bytes = Stage<MT>::bytes(a.m);
  const int red = warps * 8 * NT * (16 * MT + 1) * 4;
  const int smem = max(warps * kStages * a.stage_bytes, red);
  const cudaError_t e = allow_smem<gemv_q4_kernel<MT, NT>>(227 * 1024);
  if (e != cudaSuccess) return e;
  return launch_pdl(gemv_q4_kernel<MT, NT>, dim3((a.n + 16 * MT - 1) / (16 * MT)), warps * 32, smem, s, a);
}

}  // namespace

cudaError_t launch_gemv_q4(const __half* x, int ldx, const uint8_t* w, int m, int n, int k, const __half* bias,
                           const __half* residual, int ld_res, int epi, void* y, int ldy, cudaStream_t s) {
  const GemvArgs a{x, ldx, w, m, n, k, bias, residual, ld_res, epi, y, ldy, 0};
  const int sms = runtime().num_sms;
  // 32 features a CTA (X read once for them) unless that leaves SMs without work
  const bool wide = (n + 31) / 32 >= 2 * sms;
  const int ctas = wide ? (n + 31) / 32 : (n + 15) / 16;
  const int steps = (k + 127) / 128;
  int warps = 4;  // more warps to a CTA's K axis while the grid leaves room for them
  if (ctas < 2 * sms && steps >= 8) warps = 8;
  if (wide) return m <= 8 ? launch_gemv<2, 1>(a, warps, s) : launch_gemv<2, 2>(a, warps, s);
  return m <= 8 ? launch_gemv<1, 1>(a, warps, s) : launch_gemv<1, 2>(a, warps, s);
}

}  // namespace flexq
