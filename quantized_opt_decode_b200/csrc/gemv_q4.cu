// Few-row linear layer with a 4-bit weight in the tiled layout:
// Y[m][n] = epilogue(X[m][k] W^T), m <= 16, w = code * scale + min rounded once
// to fp16, fp32 sums.
//
// The weight is read once (n k / 2 bytes of codes and n k / 16 of pairs) and that
// is the bound; the rows of X are the B operand of mma.sync (8 columns an
// instruction, one or two of them), so the arithmetic does not grow with m.  A CTA
// owns one 128-feature tile of the weight, whose k-blocks are contiguous: a ninth warp
// streams them through a ring, one bulk copy a stage of four blocks, with X's columns of
// the stage beside them (16-byte copies that arrive on the same barrier); eight warps
// take 32 features of every other block each and dequantize their rows' words into A
// fragments.  Where there are fewer tiles than SMs the K axis is shared out over a
// cluster, whose sums are joined over distributed shared memory in a fixed order.
//
// With one warp a K slice and 32 features, each with its own ring of 16-byte copies, the
// same sums took 41 us (5 rows, 28672 x 7168) and 50 us (16 rows, 50272 x 4096): 600
// instructions a warp for 2304 bytes, more than half of them addresses and copies of X.
#include <cooperative_groups.h>

#include "warp_mma.cuh"

namespace flexq {
namespace {

namespace cg = cooperative_groups;

constexpr int kWarps = 8;  // 32 features each, of the even or the odd k-blocks
constexpr int kHalves = 2;
constexpr int kMT = 2;  // 16-feature tiles of a warp
constexpr int kThreads = (kWarps + 1) * 32;
constexpr int kBlocks = 4;  // k-blocks of a stage
constexpr int kWBytes = kBlocks * kTileBytes;
constexpr int kXRow = kBlocks * 128 + 16;  // a row of X in a stage; the pad keeps fragment reads free of bank conflicts
constexpr int kMaxCluster = 8;
constexpr uint64_t kDrainNs = 2000000000ull;

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
  uint64_t limit_ns;
  uint32_t* err;
};

__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Stages of the ring: two or three CTAs' worth of 18 KB weight copies in flight on an SM.
template <int NT>
struct Ring {
  static constexpr int stages = NT == 1 ? 3 : 2;
  static constexpr int stage_bytes = kWBytes + 8 * NT * kXRow;
  static constexpr int smem = stages * stage_bytes;
};

template <int NT>
__global__ void __launch_bounds__(kThreads, 3) gemv_q4_kernel(const GemvArgs a) {
  constexpr int LD = kTileRows + 4;  // floats of a row of sums
  constexpr int kStages = Ring<NT>::stages, kStageBytes = Ring<NT>::stage_bytes;
  static_assert(kHalves * 8 * NT * LD * 4 <= Ring<NT>::smem, "the sums lie over the ring");
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kStages], empty[kStages];
  __shared__ int s_fail;
  const int lane = static_cast<int>(lane_id()), warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1 + 32);
      mbar_init(&empty[s], kWarps);
    }
    s_fail = 0;
    mbar_fence_init();
  }
  __syncthreads();
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int splits = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int tile = blockIdx.x / splits;
  const int kbs = a.k / 64;
  const int per = (kbs + splits - 1) / splits;
  const int kb0 = min(rank * per, kbs), kb1 = min(kb0 + per, kbs);
  const int steps = (kb1 - kb0 + kBlocks - 1) / kBlocks;
  const int r = lane >> 2, j = lane & 3;
  auto wait = [&](uint64_t* b, uint32_t parity, uint32_t code) {
    if (mbar_wait(b, parity, a.limit_ns)) return true;
    set_error(a.err, code);
    atomicExch(&s_fail, 1);
    return false;
  };

  float acc[kMT][NT][4];
#pragma unroll
  for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[mt][nt][e] = 0.f;
  const int feat = (warp & 3) * 32, half = warp >> 2;

  if (warp == kWarps) {
    const uint8_t* src = a.w + (static_cast<size_t>(tile) * kbs + kb0) * kTileBytes;
    const uint64_t policy = policy_evict_first();
    int s = 0;
    for (; s < steps; ++s) {
      const int slot = s % kStages;
      if (!__all_sync(0xffffffffu, wait(&empty[slot], ((s / kStages) & 1) ^ 1, DEV_TIMEOUT_PRODUCER))) break;
      uint8_t* st = smem + slot * kStageBytes;
      const int nb = min(kBlocks, kb1 - kb0 - s * kBlocks);
      if (lane == 0) {
        mbar_arrive_expect_tx(&full[slot], static_cast<uint32_t>(nb) * kTileBytes);
        bulk_load(st, src + static_cast<size_t>(s) * kWBytes, static_cast<uint32_t>(nb) * kTileBytes, &full[slot], policy);
      }
      if (lane < nb * 8) {
        const __half* xs = a.x + (kb0 + s * kBlocks) * 64 + lane * 8;
        const uint32_t to = smem_u32(st + kWBytes + lane * 16);
#pragma unroll
        for (int i = 0; i < 8 * NT; ++i)
          if (i < a.m) cp_async16(to + i * kXRow, xs + static_cast<size_t>(i) * a.ldx, true);
      }
      cp_async_arrive(&full[slot]);
    }
    // no copy is in flight when the CTA lets go of its shared memory
    for (int d = max(0, s - kStages); d < s; ++d)
      if (!mbar_wait(&full[d % kStages], (d / kStages) & 1, kDrainNs)) set_error(a.err, DEV_TIMEOUT_PRODUCER);
  } else {
    // lane (r, j): features feat + r, + 8, + 16, + 24, columns 16 j .. 16 j + 15 of a k-block,
    // rows r (and r + 8) of X; what stands in rows past m are columns of the product that
    // nobody reads
    const uint8_t* codes = smem + (feat + r) * 32 + j * 8 + half * kTileBytes;
    const uint8_t* pairs = smem + kTileCodeBytes + (feat + r) * 4 + half * kTileBytes;
    const uint8_t* xcols = smem + kWBytes + r * kXRow + j * 32 + half * 128;
    auto block = [&](int slot, int b) {
      const int at = slot * kStageBytes + b * kTileBytes, xat = slot * kStageBytes + b * 128;
      uint4 x[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        x[nt][0] = lds128(xcols + xat + nt * 8 * kXRow);
        x[nt][1] = lds128(xcols + xat + nt * 8 * kXRow + 16);
      }
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        const uint2 c0 = lds64(codes + at + mt * 512), c1 = lds64(codes + at + mt * 512 + 256);
        const uint32_t p0 = lds32(pairs + at + mt * 64), p1 = lds32(pairs + at + mt * 64 + 32);
        const __half2 h0 = *reinterpret_cast<const __half2*>(&p0), h1 = *reinterpret_cast<const __half2*>(&p1);
        const __half2 m0 = __low2half2(h0), s0 = __high2half2(h0), m1 = __low2half2(h1), s1 = __high2half2(h1);
#pragma unroll
        for (int wd = 0; wd < 2; ++wd) {
          uint32_t lo[4], hi[4];
          dequant_word(wd ? c0.y : c0.x, s0, m0, lo);
          dequant_word(wd ? c1.y : c1.x, s1, m1, hi);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16816(acc[mt][nt], lo[0], hi[0], lo[1], hi[1], x[nt][wd].x, x[nt][wd].y);
            mma_16816(acc[mt][nt], lo[2], hi[2], lo[3], hi[3], x[nt][wd].z, x[nt][wd].w);
          }
        }
      }
    };
    bool ok = true;
    int slot = 0, parity = 0;
    for (int s = 0; s < steps; ++s) {
      ok = __all_sync(0xffffffffu, wait(&full[slot], parity, DEV_TIMEOUT_CONSUMER));
      if (!ok) break;
      const int nb = kb1 - kb0 - s * kBlocks - half;  // blocks from the warp's first of the stage on
      if (nb > kHalves) {
        block(slot, 0);
        block(slot, kHalves);
      } else if (nb > 0) {
        block(slot, 0);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[slot]);
      if (++slot == kStages) {
        slot = 0;
        parity ^= 1;
      }
    }
  }
  __syncwarp();
  __syncthreads();
  pdl_trigger();

  // the tile's sums [half][rows of X][128 features] over the ring
  float* sums = reinterpret_cast<float*>(smem);
  if (warp < kWarps) {
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sums[(half * 8 * NT + nt * 8 + 2 * j + (e & 1)) * LD + feat + mt * 16 + (e >> 1) * 8 + r] = acc[mt][nt][e];
  }
  bool fine = true;
  if (splits == 1) {
    __syncthreads();
    fine = s_fail == 0;
  } else {
    cluster.sync();
    for (int c = 0; c < splits; ++c) fine &= *cluster.map_shared_rank(&s_fail, c) == 0;
  }
  for (int o = rank * kThreads + threadIdx.x; fine && o < a.m * kTileRows; o += splits * kThreads) {
    const int row = o / kTileRows, f = o % kTileRows;
    const int col = tile * kTileRows + f;
    if (col >= a.n) continue;
    float v = 0.f;
    if (splits == 1) {
      v = sums[row * LD + f] + sums[(8 * NT + row) * LD + f];
    } else {
      float part[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        const float* s0 = cluster.map_shared_rank(sums, c < splits ? c : 0) + row * LD + f;
        part[c] = c < splits ? s0[0] + s0[8 * NT * LD] : 0.f;
      }
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) v += part[c];
    }
    if (a.epi & EPI_BIAS) v += __half2float(a.bias[col]);
    if (a.epi & EPI_GELU) v = 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
    if (a.epi & EPI_RESIDUAL) v += __half2float(a.residual[static_cast<size_t>(row) * a.ld_res + col]);
    if (a.epi & EPI_F32_OUT)
      static_cast<float*>(a.y)[static_cast<size_t>(row) * a.ldy + col] = v;
    else
      static_cast<__half*>(a.y)[static_cast<size_t>(row) * a.ldy + col] = __float2half_rn(v);
  }
  if (splits > 1) {
    __syncwarp();
    cluster.sync();  // nobody leaves while another reads its shared memory
  }
}

template <int NT>
cudaError_t launch_gemv(const GemvArgs& a, cudaStream_t s) {
  cudaError_t e = allow_smem<gemv_q4_kernel<NT>>(Ring<NT>::smem);
  if (e != cudaSuccess) return e;
  const int tiles = (a.n + kTileRows - 1) / kTileRows, kbs = a.k / 64;
  // the K axis over a cluster while SMs would have nothing to do and each CTA keeps a stage's half
  int splits = 1;
  while (splits < kMaxCluster && tiles * splits < runtime().num_sms && kbs >= 2 * splits * (kBlocks / 2)) splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles) * splits);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Ring<NT>::smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = runtime().pdl ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, gemv_q4_kernel<NT>, a);
  return e != cudaSuccess ? e : launched();
}

}  // namespace

cudaError_t launch_gemv_q4(const __half* x, int ldx, const uint8_t* w, int m, int n, int k, const __half* bias,
                           const __half* residual, int ld_res, int epi, void* y, int ldy, cudaStream_t s) {
  const GemvArgs a{x, ldx, w, m, n, k, bias, residual, ld_res, epi, y, ldy, runtime().wait_limit_ns, runtime().err};
  return m <= 8 ? launch_gemv<1>(a, s) : launch_gemv<2>(a, s);
}

}  // namespace flexq
