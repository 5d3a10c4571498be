// Few-row linear layer with a 4-bit weight in the tiled layout:
// Y[m][n] = epilogue(X[m][k] W^T), m <= 16, w = code * scale + min rounded once
// to fp16, fp32 sums.
//
// The weight is read once (n k / 2 bytes of codes and n k / 16 of pairs) and that
// is the bound; the rows of X are the B operand of mma.sync (8 columns an
// instruction, one or two of them), so the arithmetic does not grow with m.  A CTA
// owns one 128-feature tile of the weight, whose k-blocks are contiguous: one warp
// streams them through a ring, one bulk copy a stage, with X's columns of
// the stage beside them (16-byte copies that arrive on the same barrier); each of the other warps
// takes 32 features and two blocks of a stage and dequantizes its rows' words into A
// fragments.  Where there are fewer tiles than SMs the K axis is shared out over a
// cluster, whose sums are joined over distributed shared memory in a fixed order.
//
// Measured (B200): 5 rows, 28672 x 7168: 37 us for 116 MB, 0.47 of the copy rate; 16 rows, 50272 x 4096:
// 41 us for 119 MB; one row, 2048 x 2048: 5.0 us, the launch (flexq_linear: 64, 62 and 19 us).  The
// half-precision pipe that the dequantizer's multiply-adds and mma.sync share is busy for 190 of the 290
// cycles that four warps take for a k-block, which would allow the copy rate; lost are the other
// 100, a ring that starts empty in every CTA, and 224 tiles on 148 SMs: two on some, one on others.  Sharing K out more finely cost
// more than it evened out (38 us with two parts, 51 with eight), and so did CTAs of 64 or 32 features
// (41 and 44 us; 53 and 51 for the larger).  Tried: a warp a K slice with its own ring of
// 16-byte copies (41 and 50 us: 600 instructions for 2304 bytes, half of them addresses and copies
// of X); X through the L1 cache (36 and 47 us); the dequantized rows in tensor memory and the products on
// tcgen05 (42 and 38 us, 6.3 instead of 5.0 us for the small one: the hand-offs between the
// warps cost what the products had).
#include <cooperative_groups.h>

#include "warp_mma.cuh"

namespace flexq {
namespace {

namespace cg = cooperative_groups;

constexpr int kMT = 2;     // 16-feature tiles of a warp: four warps side by side cover a block
constexpr int kParts = 2;  // fours of warps, which take a stage's k-blocks by turns
constexpr int kFold = 4;   // stages (of two k-blocks a warp) between two foldings of the accumulator
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

// NT column tiles of 8 rows of X.  (Sixteen warps where one or two CTAs have an SM to
// themselves measured 35.3 against 36.0 us at 5 rows, 28672 x 7168: not kept.)
template <int NT>
struct Shape {
  static constexpr int warps = 4 * kParts, threads = (warps + 1) * 32;
  static constexpr int blocks = 2 * kParts;  // k-blocks of a stage
  static constexpr int w_bytes = blocks * kTileBytes;
  static constexpr int x_row = blocks * 128 + 16;  // (the pad keeps fragment reads free of bank conflicts)
  static constexpr int stages = NT == 1 ? 3 : 2;
  static constexpr int stage_bytes = w_bytes + 8 * NT * x_row;
  static constexpr int smem = stages * stage_bytes;
};

template <int NT>
__global__ void __launch_bounds__(Shape<NT>::threads, 3) gemv_q4_kernel(const GemvArgs a) {
  using Sh = Shape<NT>;
  constexpr int LD = kTileRows + 4;  // floats of a row of sums
  constexpr int kWarps = Sh::warps, kThreads = Sh::threads, kBlocks = Sh::blocks, kStages = Sh::stages;
  constexpr int kStageBytes = Sh::stage_bytes;
  static_assert(kParts * 8 * NT * LD * 4 <= Sh::smem, "the sums lie over the ring");
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
    if (wait_phase(b, parity, a.limit_ns)) return true;
    set_error(a.err, code);
    atomicExch(&s_fail, 1);
    return false;
  };

  // The tensor core truncates when it adds to its accumulator.  Every few stages what it
  // has is added, with rounding, to sums of our own and it starts from zero again, so that the error
  // does not grow with k (fp32 logits at k = 4096: 2.5e-6 without, below 1e-6 with it).
  float acc[kMT][NT][4], total[kMT][NT][4];
  auto fold = [&](bool first) {
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          total[mt][nt][e] = first ? 0.f : total[mt][nt][e] + acc[mt][nt][e];
          acc[mt][nt][e] = 0.f;
        }
  };
  fold(true);
  const int feat = (warp & 3) * 32, part = warp >> 2;

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
        bulk_load(st, src + static_cast<size_t>(s) * Sh::w_bytes, static_cast<uint32_t>(nb) * kTileBytes, &full[slot], policy);
      }
      for (int u = lane; u < nb * 8; u += 32) {
        const __half* xs = a.x + (kb0 + s * kBlocks) * 64 + u * 8;
        const uint32_t to = smem_u32(st + Sh::w_bytes + u * 16);
#pragma unroll
        for (int i = 0; i < 8 * NT; ++i)
          if (i < a.m) cp_async16(to + i * Sh::x_row, xs + static_cast<size_t>(i) * a.ldx, true);
      }
      cp_async_arrive(&full[slot]);
    }
    // no copy is in flight when the CTA lets go of its shared memory
    for (int d = max(0, s - kStages); d < s; ++d)
      if (!wait_phase(&full[d % kStages], (d / kStages) & 1, kDrainNs)) set_error(a.err, DEV_TIMEOUT_PRODUCER);
  } else {
    // lane (r, j): features feat + r, + 8, + 16, + 24, columns 16 j .. 16 j + 15 of a k-block,
    // rows r (and r + 8) of X; what stands in rows past m are columns of the product that
    // nobody reads
    const uint8_t* codes = smem + (feat + r) * 32 + j * 8 + part * kTileBytes;
    const uint8_t* pairs = smem + kTileCodeBytes + (feat + r) * 4 + part * kTileBytes;
    const uint8_t* xcols = smem + Sh::w_bytes + r * Sh::x_row + j * 32 + part * 128;
    auto block = [&](int slot, int b) {
      const int at = slot * kStageBytes + b * kTileBytes, xat = slot * kStageBytes + b * 128;
      uint4 x[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        x[nt][0] = lds128(xcols + xat + nt * 8 * Sh::x_row);
        x[nt][1] = lds128(xcols + xat + nt * 8 * Sh::x_row + 16);
      }
#pragma unroll
      for (int mt = 0; mt < kMT; ++mt) {
        const uint2 c0 = lds64(codes + at + mt * 512), c1 = lds64(codes + at + mt * 512 + 256);
        const uint32_t p0 = lds32(pairs + at + mt * 64), p1 = lds32(pairs + at + mt * 64 + 32);
        const __half2 m0 = dup_half(p0, 0), s0 = dup_half(p0, 1), m1 = dup_half(p1, 0), s1 = dup_half(p1, 1);
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
      const int nb = kb1 - kb0 - s * kBlocks - part;  // blocks from the warp's first of the stage on
      if (nb > kParts) {
        block(slot, 0);
        block(slot, kParts);
      } else if (nb > 0) {
        block(slot, 0);
      }
      if (s % kFold == kFold - 1) fold(false);
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

  // the tile's sums [part][rows of X][128 features] over the ring
  float* sums = reinterpret_cast<float*>(smem);
  if (warp < kWarps) {
#pragma unroll
    for (int mt = 0; mt < kMT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          sums[(part * 8 * NT + nt * 8 + 2 * j + (e & 1)) * LD + feat + mt * 16 + (e >> 1) * 8 + r] = total[mt][nt][e] + acc[mt][nt][e];
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
#pragma unroll
      for (int q = 0; q < kParts; ++q) v += sums[(q * 8 * NT + row) * LD + f];
    } else {
      float sum[kMaxCluster];
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) {
        const float* from = cluster.map_shared_rank(sums, c < splits ? c : 0) + row * LD + f;
        sum[c] = 0.f;
#pragma unroll
        for (int q = 0; q < kParts; ++q) sum[c] += c < splits ? from[q * 8 * NT * LD] : 0.f;
      }
#pragma unroll
      for (int c = 0; c < kMaxCluster; ++c) v += sum[c];
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
  using Sh = Shape<NT>;
  cudaError_t e = allow_smem<gemv_q4_kernel<NT>>(Sh::smem);
  if (e != cudaSuccess) return e;
  const int tiles = (a.n + kTileRows - 1) / kTileRows, kbs = a.k / 64;
  // the K axis over a cluster while SMs would have nothing to do and each CTA keeps two blocks
  int splits = 1;
  while (splits < kMaxCluster && tiles * splits < runtime().num_sms && kbs >= 4 * splits) splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(tiles) * splits);
  cfg.blockDim = dim3(Sh::threads);
  cfg.dynamicSmemBytes = Sh::smem;
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
