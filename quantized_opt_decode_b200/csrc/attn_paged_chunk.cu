// Attention of chunks of new tokens over the paged cache (the sequences of a
// ragged batch with many query rows; attn_paged.cu has the few-row form).
//
// The n new tokens x heads/kv_heads query heads that share a key/value head are the rows of
// two 128-row tiles of a CTA; per 128 cached keys, on tcgen05 with accumulators in
// tensor memory,
//   S_m = Q_m K^T  (both operands in shared memory),
//   O_m += P_m V   (P in tensor memory, over S; V^T in shared memory),
// so 2 x 4 * 128 * 128 * d flops stand against one pass over the tile's codes.  Roles:
//   warps 0-3, 4-7   softmax of row tile 0, 1: a thread owns a row (a TMEM lane), so the
//                    running maximum and sum need no exchange.  The maximum used as
//                    exponent base only moves when a row outgrows it by 2^8: P then stays
//                    below 2^8 in fp16 (a relative rounding, so the base does not
//                    matter), and O is rescaled rarely;
//   warps 8-15       bring K and V: pages looked up, codes fetched a tile ahead
//                    into registers, dequantized (rounded once to fp16, as the codec's
//                    values) and stored in the 128-byte-swizzled layout; a
//                    word of codes is one 16-byte store, since the orders of the head's
//                    dimensions in Q K^T, of the keys in P V and of O's columns are
//                    free: pairs (e, e + 4) of Q are swapped into place when Q is
//                    loaded, keys y, y + 4 of a block lie side by side, and O's columns
//                    are unscrambled when they are stored.  V of an fp16 cache is
//                    transposed 8 x 8 in registers;
//   warp 16          issues the products: while row tile 0 is in its softmax,
//                    row tile 1's products run.
// A long history of few units is shared out over a cluster of CTAs, whose
// (maximum, sum, O) are joined over distributed shared memory in a fixed order.
// Every wait is bounded; on expiry the error word is set and the CTA unwinds.
#include <cooperative_groups.h>
#include <math.h>

#include "paged.cuh"
#include "warp_mma.cuh"

namespace flexq {
namespace {

namespace cg = cooperative_groups;

constexpr int kRowShift = 8;  // 256 query rows of a unit
constexpr int kRows = 1 << kRowShift;
constexpr int kKeys = 128;
constexpr int kStages = 2;
constexpr int kSoftmaxWarps = 8, kLoadWarps = 8;
constexpr int kMmaWarp = kSoftmaxWarps + kLoadWarps;
constexpr int kThreads = (kMmaWarp + 1) * 32;
constexpr int kMaxCluster = 8;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kDrainNs = 2000000000ull;

struct ChunkArgs {
  PagedView kv;
  RaggedView batch;
  int heads, group;
  int min_rows;
  const __half* q;
  int ldq;
  __half* out;
  int ldo;
  float scale_log2;
  uint64_t limit_ns;
  uint32_t* err;
};

template <int D>
struct Layout {
  static constexpr int q_tile = 128 * D * 2;  // one row tile
  static constexpr int k_stage = kKeys * D * 2;
  static constexpr int v_stage = kKeys * D * 2;
  static constexpr int k0 = 2 * q_tile, v0 = k0 + kStages * k_stage;
  static constexpr int bytes = v0 + kStages * v_stage;
  static_assert(bytes - k0 >= kRows * D * 4, "the joined output lies over the K and V stages");
  static constexpr int smem = bytes + 1024;  // room to align the base
};

struct Barriers {
  uint64_t q_full, k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages], s_full[2], p_full[2], done;
  uint32_t tmem;
};

__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

// Waits for the loads issued so far; naming the registers keeps their uses behind it.
__device__ __forceinline__ void tmem_wait_x32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])::"memory");
}

// One asm of load and wait for eight columns.
__device__ __forceinline__ void tmem_read_x8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}

__device__ __forceinline__ uint4 ldg128(const void* p) { return __ldcg(reinterpret_cast<const uint4*>(p)); }
__device__ __forceinline__ uint32_t ldg32(const void* p) { return __ldcg(reinterpret_cast<const unsigned int*>(p)); }
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

// Byte offset of 16-byte chunk c (0..7) of a row of a 128-byte-swizzled tile.
__device__ __forceinline__ uint32_t sw128(int row, int c) {
  return static_cast<uint32_t>((row >> 3) * 1024 + (row & 7) * 128 + ((c ^ (row & 7)) << 4));
}

// What a loading lane holds of one tile: its part of up to two 8-token blocks.
template <int D, bool Q4>
struct Loader;

template <int D>
struct Loader<D, true> {
  static constexpr int lanes = D / 4;           // lanes of a block: 16 bytes of its codes each
  static constexpr int per_warp = 32 / lanes;   // blocks a warp covers at once
  static constexpr int NQ = kKeys / 8 / (kLoadWarps * per_warp);
  static constexpr int units = D / 32;          // 16-byte units of a key
  uint4 k[NQ], v[NQ];
  uint32_t km[NQ], vm[NQ];
  int page[NQ];
  int warp, lane, sub, len;

  __device__ __forceinline__ int block(int q) const { return (q * kLoadWarps + warp) * per_warp + lane / lanes; }
  __device__ __forceinline__ void look_up(const ChunkArgs& a, int i, int t) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int p = t * kKeys + block(q) * 8;
      page[q] = p < len ? page_of(a.kv, i, p, a.err) : -1;
    }
  }
  __device__ __forceinline__ void fetch_k(const ChunkArgs& a, int head, int t) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      k[q] = make_uint4(0u, 0u, 0u, 0u);
      km[q] = 0u;
      if (page[q] < 0) continue;
      const size_t slot = pool_slot(a.kv, page[q], head, t * kKeys + block(q) * 8);
      k[q] = ldg128(static_cast<const char*>(a.kv.k) + slot * (D / 2) + sub * 16);
      km[q] = ldg32(static_cast<const char*>(a.kv.k_meta) + (slot + sub / units) * (D / 64) * 4 +
                    (D == 128 ? ((sub % units) >> 1) * 4 : 0));
    }
  }
  __device__ __forceinline__ void fetch_v(const ChunkArgs& a, int head, int t) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      v[q] = make_uint4(0u, 0u, 0u, 0u);
      vm[q] = 0u;
      if (page[q] < 0) continue;
      const int p = t * kKeys + block(q) * 8;
      const size_t slot = pool_slot(a.kv, page[q], head, p);
      v[q] = ldg128(static_cast<const char*>(a.kv.v) + slot * (D / 2) + sub * 16);
      // one pair a lane, in order; tokens behind the end read as zero (their
      // weights are zero, and 0 times an old NaN is not)
      if (sub < 8 * (D / 64) && p + sub / (D / 64) < len)
        vm[q] = ldg32(static_cast<const char*>(a.kv.v_meta) + slot * (D / 64) * 4 + sub * 4);
    }
  }
  __device__ __forceinline__ void store_k(uint32_t st) const {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int y = sub / units, u = sub % units;
      const int row = block(q) * 8 + (y < 4 ? 2 * y : 2 * y - 7);
      const __half2 mn = __low2half2(as_half2(km[q])), sc = __high2half2(as_half2(km[q]));
      // words in pairwise swapped order for half the units: eight lanes then hit
      // eight bank groups
      const bool swap = D == 128 && (u & 2);
      const uint32_t w[4] = {swap ? k[q].y : k[q].x, swap ? k[q].x : k[q].y, swap ? k[q].w : k[q].z,
                             swap ? k[q].z : k[q].w};
      const uint32_t base = st + (u >> 1) * (kKeys * 128);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t o[4];
        dequant_word(w[e], sc, mn, o);
        sts128(base + sw128(row, (u & 1) * 4 + (e ^ (swap ? 1 : 0))), o[0], o[1], o[2], o[3]);
      }
    }
  }
  __device__ __forceinline__ void store_v(uint32_t st) const {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int blk = block(q);
      __half2 sc[4], mn[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const int from = (lane / lanes) * lanes + (D == 128 ? 2 * y + (sub >> 4) : y);
        const uint32_t lo = __shfl_sync(0xffffffffu, vm[q], from);
        const uint32_t hi = __shfl_sync(0xffffffffu, vm[q], from + 4 * (D / 64));
        mn[y] = as_half2(__byte_perm(lo, hi, 0x5410));
        sc[y] = as_half2(__byte_perm(lo, hi, 0x7632));
      }
      const uint32_t w[4] = {v[q].x, v[q].y, v[q].z, v[q].w};
      const uint32_t base = st + (blk >> 3) * (D * 128);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        uint32_t o[4];
        dequant_word(w[e], sc[0], mn[0], sc[1], mn[1], sc[2], mn[2], sc[3], mn[3], o);
        sts128(base + sw128((D / 4) * e + sub, blk & 7), o[0], o[1], o[2], o[3]);  // dimension 4 sub + e
      }
    }
  }
};

template <int D>
struct Loader<D, false> {
  static constexpr int lanes = D / 8;  // lanes of a block: 16 bytes of each of its eight keys
  static constexpr int per_warp = 32 / lanes;
  uint4 k[8], v[8];
  int page;
  int warp, lane, sub, len;

  __device__ __forceinline__ int block() const { return warp * per_warp + lane / lanes; }
  __device__ __forceinline__ bool mine() const { return block() < kKeys / 8; }
  __device__ __forceinline__ void look_up(const ChunkArgs& a, int i, int t) {
    const int p = t * kKeys + block() * 8;
    page = mine() && p < len ? page_of(a.kv, i, p, a.err) : -1;
  }
  __device__ __forceinline__ void fetch(const ChunkArgs& a, const void* pool, int head, int t, uint4 (&x)[8]) const {
    const int p = t * kKeys + block() * 8;
    const size_t slot = page >= 0 ? pool_slot(a.kv, page, head, p) : 0;
#pragma unroll
    for (int y = 0; y < 8; ++y) {
      x[y] = make_uint4(0u, 0u, 0u, 0u);
      if (page >= 0 && p + y < len) x[y] = ldg128(static_cast<const char*>(pool) + (slot + y) * (D * 2) + sub * 16);
    }
  }
  __device__ __forceinline__ void fetch_k(const ChunkArgs& a, int head, int t) { fetch(a, a.kv.k, head, t, k); }
  __device__ __forceinline__ void fetch_v(const ChunkArgs& a, int head, int t) { fetch(a, a.kv.v, head, t, v); }
  __device__ __forceinline__ void store_k(uint32_t st) const {
    if (!mine()) return;
#pragma unroll
    for (int y = 0; y < 8; ++y)
      sts128(st + (sub >> 3) * (kKeys * 128) + sw128(block() * 8 + y, sub & 7), k[y].x, k[y].y, k[y].z, k[y].w);
  }
  __device__ __forceinline__ void store_v(uint32_t st) const {
    if (!mine()) return;
    const int blk = block();
    const uint32_t base = st + (blk >> 3) * (D * 128);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t o[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        const uint4 &lo = v[2 * y], &hi = v[2 * y + 1];
        const uint32_t x0 = e < 2 ? lo.x : e < 4 ? lo.y : e < 6 ? lo.z : lo.w;
        const uint32_t x1 = e < 2 ? hi.x : e < 4 ? hi.y : e < 6 ? hi.z : hi.w;
        o[y] = __byte_perm(x0, x1, (e & 1) ? 0x7632 : 0x5410);
      }
      sts128(base + sw128((D / 8) * e + sub, blk & 7), o[0], o[1], o[2], o[3]);  // dimension 8 sub + e
    }
  }
};

template <int D, bool Q4>
__global__ void __launch_bounds__(kThreads, 1) attn_paged_chunk_kernel(const ChunkArgs a) {
  using L = Layout<D>;
  constexpr int W = Q4 ? 4 : 8;  // O's column (D / W) e + u is dimension W u + e
  extern __shared__ uint8_t raw_smem[];
  __shared__ Barriers bar;
  __shared__ float s_m[kRows], s_l[kRows];
  __shared__ int s_fail;
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int splits = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int lane = static_cast<int>(lane_id()), warp = threadIdx.x >> 5;

  // the unit: 256 query rows of one sequence and key/value head, the later rows first
  const int work = blockIdx.x / splits;
  const int head = work % a.kv.kv_heads, u = work / a.kv.kv_heads;
  const int g = a.group;
  const int i = find_unit_owner(a.batch, u, g, kRowShift, 1);
  if (i < 0) return;
  const Span sp = ragged_span(a.batch, i, a.err);
  const int total = sp.n * g;  // at most max_new * group, checked by the launcher
  const int rel = u - static_cast<int>(unit_base(a.batch, i, g, kRowShift, 1));
  const int units = (total + kRows - 1) / kRows;
  if (sp.n == 0 || total < a.min_rows || rel < 0 || rel >= units) return;  // (all CTAs of a cluster alike)
  const int c0 = (units - 1 - rel) * kRows;
  const int rows = min(kRows, total - c0);
  const int mtiles = rows > 128 ? 2 : 1;
  const int first = sp.len - sp.n;
  const int keys = first + (c0 + rows - 1) / g + 1;  // keys that some row of the unit sees
  const int all = (keys + kKeys - 1) / kKeys;
  const int mine = all > rank ? (all - rank + splits - 1) / splits : 0;  // tiles rank, rank + splits, ..

  uint8_t* smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  if (threadIdx.x == 0) {
    mbar_init(&bar.q_full, kSoftmaxWarps);
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar.k_full[s], kLoadWarps);
      mbar_init(&bar.v_full[s], kLoadWarps);
      mbar_init(&bar.k_empty[s], 1);
      mbar_init(&bar.v_empty[s], 1);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&bar.s_full[m], 1);
      mbar_init(&bar.p_full[m], 4);
    }
    mbar_init(&bar.done, 1);
    s_fail = 0;
    mbar_fence_init();
  }
  if (warp == kMmaWarp) {
    tmem_alloc(&bar.tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar.tmem;
  auto wait = [&](uint64_t* b, uint32_t parity, uint32_t code) {
    if (mbar_wait(b, parity, a.limit_ns)) return true;
    set_error(a.err, code);
    atomicExch(&s_fail, 1);
    return false;
  };

  if (warp < kSoftmaxWarps) {
    // --- softmax of one row -------------------------------------------------------
    const int m = warp >> 2, row = threadIdx.x;  // row of the unit: lane row % 128 of tile m
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + m * 128, o_col = tmem + lanes + 256 + m * D;
    const bool live = row < rows;
    const int c = c0 + (live ? row : 0);
    {
      const __half* src = a.q + static_cast<size_t>(sp.row0 + c / g) * a.ldq + (head * g + c % g) * D;
      const uint32_t dst = sbase + m * L::q_tile;
#pragma unroll
      for (int ch = 0; ch < D / 8; ++ch) {
        const uint4 x = live ? *reinterpret_cast<const uint4*>(src + ch * 8) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t at = dst + (ch >> 3) * (128 * 128) + sw128(row & 127, ch & 7);
        if (Q4)  // (e, e + 4)
          sts128(at, __byte_perm(x.x, x.z, 0x5410), __byte_perm(x.x, x.z, 0x7632), __byte_perm(x.y, x.w, 0x5410),
                 __byte_perm(x.y, x.w, 0x7632));
        else
          sts128(at, x.x, x.y, x.z, x.w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_full);
    }
    const int pos = live ? first + c / g : keys - 1;
    float base = -INFINITY, sum = 0.f;  // base: exponent base in units of the raw scores
    const float slack = 8.f / a.scale_log2;
    bool ok = true;
    if (m < mtiles) {
      for (int it = 0; it < mine; ++it) {
        if (!(ok = __all_sync(0xffffffffu, wait(&bar.s_full[m], it & 1, DEV_TIMEOUT_EPILOGUE)))) break;
        tc_fence_after();
        const int p0 = (rank + it * splits) * kKeys;
        const int lim = pos - p0;  // tokens 0 .. lim of the tile count
        const bool masked = __any_sync(0xffffffffu, lim < kKeys - 1);
        float top = -INFINITY;
        uint32_t s[2][32];
        tmem_ld_x32(s_col, s[0]);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          tmem_wait_x32(s[ch & 1]);
          if (ch < 3) tmem_ld_x32(s_col + 32 * (ch + 1), s[(ch + 1) & 1]);
          if (masked) {
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int tok = 32 * ch + (Q4 ? (e & ~7) + ((e & 7) >> 1) + 4 * (e & 1) : e);
              if (tok <= lim) top = fmaxf(top, __uint_as_float(s[ch & 1][e]));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(s[ch & 1][e]));
          }
        }
        const bool move = top > base + slack;  // (from -inf: any finite score)
        if (__any_sync(0xffffffffu, move)) {
          const float nb = move ? top : base;
          const float alpha = base == -INFINITY ? 0.f : exp2_approx((base - nb) * a.scale_log2);
          base = nb;
          sum *= alpha;
          if (it > 0) {
            const float f = alpha;
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
              tmem_ld_x32(o_col + 32 * ch, s[0]);
              tmem_wait_x32(s[0]);
#pragma unroll
              for (int e = 0; e < 32; ++e) s[0][e] = __float_as_uint(__uint_as_float(s[0][e]) * f);
              tmem_st_x32(o_col + 32 * ch, s[0]);
            }
          }
        }
        const float off = base == -INFINITY ? 0.f : -base * a.scale_log2;
        tmem_ld_x32(s_col, s[0]);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          tmem_wait_x32(s[ch & 1]);
          if (ch < 3) tmem_ld_x32(s_col + 32 * (ch + 1), s[(ch + 1) & 1]);
          uint32_t p[16];
          float add[2] = {0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0 = fmaf(__uint_as_float(s[ch & 1][e]), a.scale_log2, off);
            float x1 = fmaf(__uint_as_float(s[ch & 1][e + 1]), a.scale_log2, off);
            if (masked) {
              const int t0 = 32 * ch + (Q4 ? (e & ~7) + ((e & 7) >> 1) : e);
              if (t0 > lim) x0 = -INFINITY;
              if (t0 + (Q4 ? 4 : 1) > lim) x1 = -INFINITY;
            }
            x0 = exp2_approx(x0);
            x1 = exp2_approx(x1);
            add[0] += x0;
            add[1] += x1;
            p[e / 2] = pack_half2(x0, x1);
          }
          sum += add[0] + add[1];
          // over S's columns 16 ch .. 16 ch + 15, which are read already (the load
          // in flight is of columns 32 (ch + 1) and up)
          tmem_st_x16(s_col + 16 * ch, p);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[m]);
      }
    }
    ok = ok && __all_sync(0xffffffffu, wait(&bar.done, 0, DEV_TIMEOUT_EPILOGUE));
    tc_fence_after();
    if (ok && m < mtiles) {
      if (splits == 1) {
        const float inv = 1.f / sum;
        __half* dst = a.out + static_cast<size_t>(sp.row0 + c / g) * a.ldo + (head * g + c % g) * D;
#pragma unroll 1
        for (int u0 = 0; u0 < D / W; u0 += 8) {
          uint32_t o[W][8];
#pragma unroll
          for (int e = 0; e < W; ++e) tmem_read_x8(o_col + (D / W) * e + u0, o[e]);
          if (live) {
#pragma unroll
            for (int x = 0; x < 8 * W; x += 8) {
              uint32_t h[4];
#pragma unroll
              for (int e = 0; e < 8; e += 2)
                h[e / 2] = pack_half2(__uint_as_float(o[(x + e) % W][(x + e) / W]) * inv,
                                      __uint_as_float(o[(x + e + 1) % W][(x + e + 1) / W]) * inv);
              *reinterpret_cast<uint4*>(dst + W * u0 + x) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          }
        }
      } else {
        s_m[row] = base;
        s_l[row] = sum;
        // column order, 16-byte units XORed by the row: over the K and V stages, which
        // no product reads any more
#pragma unroll 1
        for (int q = 0; q < D; q += 8) {
          uint32_t o[8];
          if (mine > 0) {
            tmem_read_x8(o_col + q, o);
          } else {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = 0u;
          }
          const uint32_t at = sbase + L::k0 + row * (D * 4);
          sts128(at + (((q >> 2) ^ (row & 7)) << 4), o[0], o[1], o[2], o[3]);
          sts128(at + ((((q >> 2) + 1) ^ (row & 7)) << 4), o[4], o[5], o[6], o[7]);
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // --- K and V ------------------------------------------------------------------
    Loader<D, Q4> ld;
    ld.warp = warp - kSoftmaxWarps;
    ld.lane = lane;
    ld.sub = lane % Loader<D, Q4>::lanes;
    ld.len = sp.len;
    if (mine > 0) {
      ld.look_up(a, i, rank);
      ld.fetch_k(a, head, rank);
      ld.fetch_v(a, head, rank);
    }
    for (int it = 0; it < mine; ++it) {
      const int st = it % kStages, next = rank + (it + 1) * splits;
      const uint32_t free_parity = ((it / kStages) & 1) ^ 1;
      if (!__all_sync(0xffffffffu, wait(&bar.k_empty[st], free_parity, DEV_TIMEOUT_PRODUCER))) break;
      if (it + 1 < mine) ld.look_up(a, i, next);
      ld.store_k(sbase + L::k0 + st * L::k_stage);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.k_full[st]);
      if (it + 1 < mine) ld.fetch_k(a, head, next);
      if (!__all_sync(0xffffffffu, wait(&bar.v_empty[st], free_parity, DEV_TIMEOUT_PRODUCER))) break;
      ld.store_v(sbase + L::v0 + st * L::v_stage);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.v_full[st]);
      if (it + 1 < mine) ld.fetch_v(a, head, next);
    }
  } else if (lane == 0) {
    // --- products -----------------------------------------------------------------
    const uint32_t id_s = idesc_f16_m128(kKeys), id_o = idesc_f16_m128(D);
    auto issue_s = [&](int m, int st) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * (128 * 128) + (kk & 3) * 32;
        mma_f16_ss(tmem + m * 128, sw128_kmajor_desc(sbase + m * L::q_tile + off),
                   sw128_kmajor_desc(sbase + L::k0 + st * L::k_stage + off), id_s, kk > 0);
      }
      mma_commit(&bar.s_full[m]);
    };
    bool ok = wait(&bar.q_full, 0, DEV_TIMEOUT_MMA);
    if (ok && mine > 0) {
      ok = wait(&bar.k_full[0], 0, DEV_TIMEOUT_MMA);
      if (ok) {
        tc_fence_after();
        for (int m = 0; m < mtiles; ++m) issue_s(m, 0);
        mma_commit(&bar.k_empty[0]);
      }
    }
    for (int it = 0; ok && it < mine; ++it) {
      const int st = it % kStages, ns = (it + 1) % kStages;
      for (int m = 0; ok && m < mtiles; ++m) {
        if (m == 0) ok = wait(&bar.v_full[st], (it / kStages) & 1, DEV_TIMEOUT_MMA);
        ok = ok && wait(&bar.p_full[m], it & 1, DEV_TIMEOUT_MMA);
        if (!ok) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < kKeys / 16; ++kk)
          mma_f16_ts(tmem + 256 + m * D, tmem + m * 128 + kk * 8,
                     sw128_kmajor_desc(sbase + L::v0 + st * L::v_stage + (kk >> 2) * (D * 128) + (kk & 3) * 32), id_o,
                     it > 0 || kk > 0);
        if (m == mtiles - 1) mma_commit(&bar.v_empty[st]);
        if (it + 1 < mine) {
          if (m == 0) {
            ok = wait(&bar.k_full[ns], ((it + 1) / kStages) & 1, DEV_TIMEOUT_MMA);
            if (!ok) break;
            tc_fence_after();
          }
          issue_s(m, ns);  // over P: the products run in the order of issue
          if (m == mtiles - 1) mma_commit(&bar.k_empty[ns]);
        }
      }
    }
    mma_commit(&bar.done);
    // the products in flight have read shared and tensor memory before the CTA lets go of
    // them, whatever the waits' limit
    if (!mbar_wait(&bar.done, 0, kDrainNs)) set_error(a.err, DEV_TIMEOUT_MMA);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
  if (splits == 1) return;

  // join the cluster's parts: CTA `rank` takes every splits-th group of four columns
  cluster.sync();
  bool fine = true;
  for (int k = 0; k < splits; ++k) fine &= *cluster.map_shared_rank(&s_fail, k) == 0;
  constexpr int C4 = D / 4;
  // (an aligned base is at the same offset in every CTA of the launch)
  const float4* parts = reinterpret_cast<const float4*>(smem + L::k0);
  for (int x = rank * kThreads + threadIdx.x; fine && x < rows * C4; x += splits * kThreads) {
    const int row = x / C4, c4 = x % C4;
    float top = -INFINITY, mk[kMaxCluster], lk[kMaxCluster];
    float4 pk[kMaxCluster];
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k)
      if (k < splits) {
        mk[k] = *cluster.map_shared_rank(&s_m[row], k);
        lk[k] = *cluster.map_shared_rank(&s_l[row], k);
        pk[k] = *cluster.map_shared_rank(parts + row * C4 + (c4 ^ (row & 7)), k);
        top = fmaxf(top, mk[k]);
      }
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float den = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k)
      if (k < splits && mk[k] != -INFINITY) {
        const float f = exp2_approx((mk[k] - top) * a.scale_log2);
        den += f * lk[k];
        acc.x += f * pk[k].x;
        acc.y += f * pk[k].y;
        acc.z += f * pk[k].z;
        acc.w += f * pk[k].w;
      }
    const float inv = 1.f / den;
    const int c = c0 + row;
    __half* dst = a.out + static_cast<size_t>(sp.row0 + c / g) * a.ldo + (head * g + c % g) * D;
    const float o[4] = {acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int col = c4 * 4 + e;
      dst[W * (col % (D / W)) + col / (D / W)] = __float2half_rn(o[e]);
    }
  }
  __syncwarp();
  cluster.sync();  // nobody leaves while another reads its shared memory
}

template <int D, bool Q4>
cudaError_t launch_d(const ChunkArgs& a, cudaStream_t s) {
  cudaError_t e = allow_smem<attn_paged_chunk_kernel<D, Q4>>(Layout<D>::smem);
  if (e != cudaSuccess) return e;
  const int sms = runtime().num_sms;
  const long long works = unit_total(a.batch.rows, a.batch.b, a.group, kRowShift, 1) * a.kv.kv_heads;
  // units that the batch's rows fill; a history is shared out while that leaves SMs idle
  // and every CTA keeps two tiles of keys
  const long long full =
      ((static_cast<long long>(a.batch.rows) * a.group + kRows - 1) / kRows) * a.kv.kv_heads;
  int splits = 1;
  while (splits < kMaxCluster && full * splits * 2 <= sms && a.batch.max_len > splits * 2 * 2 * kKeys) splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(works * splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = Layout<D>::smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = runtime().pdl ? 2 : 1;
  e = cudaLaunchKernelEx(&cfg, attn_paged_chunk_kernel<D, Q4>, a);
  return e != cudaSuccess ? e : launched();
}

}  // namespace

cudaError_t launch_attn_paged_chunks(const PagedView& kv, const RaggedView& batch, int heads, int d, int kv_bits,
                                     int min_rows, const __half* q, int ldq, __half* out, int ldo, cudaStream_t s) {
  const ChunkArgs a{kv, batch, heads, heads / kv.kv_heads, min_rows, q, ldq, out, ldo,
                    1.4426950408889634f / sqrtf(static_cast<float>(d)), runtime().wait_limit_ns, runtime().err};
  if (kv_bits == 4) return d == 128 ? launch_d<128, true>(a, s) : launch_d<64, true>(a, s);
  return d == 128 ? launch_d<128, false>(a, s) : launch_d<64, false>(a, s);
}

}  // namespace flexq
