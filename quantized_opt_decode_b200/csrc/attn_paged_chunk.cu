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
//                    running maximum and sum need no exchange.  The exponent base is a whole
//                    power of two that only moves when a score outgrows it by 2^7; a tile's scores
//                    are read once, 32 columns at a time, and where the base moves, the factor
//                    for O and for the P already stored is exact (kWeightBias: what P is in fp16);
//   warps 8-15       bring K and V: pages looked up two tiles ahead, codes fetched one
//                    tile ahead into registers (of an fp16 cache only once its stage is free: 363 us
//                    where the 4-bit form takes 395), dequantized (code * scale + min rounded
//                    once to fp16) and stored in the 128-byte-swizzled layout; a
//                    word of codes is one 16-byte store, since the orders of the head's
//                    dimensions in Q K^T, of the keys in P V and of O's columns are
//                    free: pairs (e, e + 4) of Q are swapped into place when Q is
//                    loaded, keys y, y + 4 of a block lie side by side, and O's columns
//                    are unscrambled when they are stored.  V of an fp16 cache is
//                    transposed 8 x 8 in registers;
//   warp 16          issues the products, row tile 0's and row tile 1's by turns: while
//                    one is in its softmax, the other's run.
// One CTA an SM walks the units (256 query rows of a sequence and key/value head) that fall to it:
// every role runs on into the next unit on its own, so the stores of one unit overlap the
// products of the next.  Where the bounds allow few units, or long ones, the launch is one of clusters: each
// shares out the units of many tiles that fall to it, whose (maximum, sum, O) are joined over
// distributed shared memory in a fixed order; then its CTAs walk the shorter ones alone.  The bounds may be
// far above the batch (a captured graph), so clusters are as many as are resident at once and not one a
// possible unit (32 sequences, four of them chunks, 56 heads, under a bound of 32768 keys: 173 us against 146
// under their own; 776 with a cluster a unit).
// Every wait is bounded; on expiry the error word is set and the CTA unwinds.
//
// Measured (B200; two sequences of 1900 to 2048 new tokens over 5600 to 6100 keys, 32 heads, d = 128,
// 4 bit): 392 to 400 us = 808 to 824 TFLOP/s, 0.49 to 0.50 of the library product's rate.  A pair of row tiles
// takes some 4400 cycles a key tile against 2100 of products: scores, softmax, P and products are one chain
// per row tile, of which the 16-lane exponential unit (2048 cycles a pair) and the issue slots
// (9500 instructions, 3700 of them the dequantizer's) make up the most.  Tried, at the
// same sizes (the last three where the kept form took 417): scores of 64 keys, twice, so that the next are there when a softmax ends (464 us: twice
// the hand-offs); one thread a row tile issuing the products (547 us against 451: both softmaxes
// then run at the same time); a quarter of the exponentials as polynomials (446 us: issue slots);
// loops rolled up for the instruction cache (519 us); four loading warps (446 us); the largest score of the
// whole tile first, P then handed over in halves (447 us: scores are read twice); two key tiles at once
// for units of one row tile (434 us); pages' entries looked at a step after their load (423 us).  The softmax
// keeps more than its registers hold: 156 to 260 bytes of spill stores a thread without clusters, 900 to
// 1050 with them.  The roles' waits are inlined: a function call would tie the roles to one register count.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "paged.cuh"
#include "per_device.h"
#include "warp_mma.cuh"

namespace flexq {
namespace {

namespace cg = cooperative_groups;

constexpr int kRows = kUnitRows;  // 256 query rows of a unit
constexpr int kKeys = kKeyTile;
constexpr int kStages = 2;
constexpr int kSoftmaxWarps = 8, kLoadWarps = 8;
constexpr int kMmaWarp = kSoftmaxWarps + kLoadWarps;
constexpr int kThreads = (kMmaWarp + 4) * 32;  // whole warpgroups, which share a register count
// Registers a thread by role, out of the launch's 640 * 96 (136, 72 and 64: 405 us where this takes 395).
constexpr int kLaunchRegs = 96, kSoftmaxRegs = 128, kLoadRegs = 80, kMmaRegs = 64;
static_assert(256 * kSoftmaxRegs + 256 * kLoadRegs + 128 * kMmaRegs <= kThreads * kLaunchRegs,
              "a split above the launch's registers would wait for ever");
constexpr int kMaxCluster = 8;
// Key tiles that one accumulator takes.  The tensor core truncates, always towards zero, when it
// adds to it: 1024 additions of at most 2^-23 each are a quarter of the output's own rounding, 2^-13
// (measured over 16384 keys of values of one sign: 1.0e-4, and 3.8e-4 over 65536).  Where a CTA's share may
// be longer, what has come together is put aside after every so many tiles and added up with rounding.
constexpr int kShareTiles = 128;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kDrainNs = 2000000000ull;

struct ChunkArgs {
  PagedView kv;
  RaggedView batch;
  int group;
  int min_rows;
  int joint_tiles;  // tiles from which on a unit is shared out
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
  // joined output of a unit's pieces so far: 16 dimensions of a row a thread, its maximum and sum
  static constexpr int kept = kRows * (16 + 2) * 4;
};

struct Barriers {
  uint64_t k_full[kStages], k_empty[kStages], v_full[kStages], v_empty[kStages];
  uint64_t q_full[2], s_full[2], p_full[2], o_full[2], o_free[2];  // by row tile
  uint64_t done;
  uint32_t tmem;
};

// 256 query rows of one sequence and key/value head.
struct Unit {
  int i, head, row0, first, len, c0, rows;
  int t0, tiles;  // key tiles t0 .. tiles - 1: the unit's, or the next piece of a shared-out one
  int all;        // key tiles that some row of the unit sees
  bool joint;     // shared out over the cluster
};

// The units of CTA (or cluster) `id` of `stride`, in order: one of each `stride` units, from the front
// and from the back by turns (a sequence's later rows, which see more keys, come first).  A warp
// counts the units of 32 sequences at a time, a lane each, as it comes to them; sequences that have none cost
// nothing more.  In a launch of clusters first the cluster's units, those of joint_tiles tiles and
// more, piece by piece, then the CTA's own, the shorter ones.
template <bool J, bool P>
struct UnitWalk {
  int id, stride, total;  // total: more units than a batch of sound spans has (any other ends there)
  int most;               // tiles of a piece
  bool joint;
  int k, i0, before;      // units taken; the 32 sequences' first; units of the sequences before them
  int row0, n, len;       // the lane's sequence
  int through, shift;     // units of the sequences up to and with it; minus the first one's number

  __device__ __forceinline__ void start(const ChunkArgs& a, int splits) {
    total = static_cast<int>(unit_total(a.batch.rows, a.batch.b, a.group, kUnitRowShift, 1));
    joint = J;
    most = J && P ? kShareTiles * splits : 1 << 30;
    id = static_cast<int>(blockIdx.x) / splits;
    stride = static_cast<int>(gridDim.x) / splits;
    k = i0 = before = 0;
    count(a);
  }
  __device__ __forceinline__ void count(const ChunkArgs& a) {
    const int lane = static_cast<int>(lane_id()), i = i0 + lane;
    Span sp{0, 0, 0};
    if (i < a.batch.b) sp = ragged_span(a.batch, i, a.err);
    row0 = sp.row0;
    n = sp.n;
    len = sp.len;
    const int rows = n * a.group;  // at most max_new * group, which the entry point bounds
    const int units = n > 0 && rows >= a.min_rows ? row_units(rows) : 0;
    int mine = units, skipped = 0;
    if (J) {
      const int longs = long_units(len - n, n, a.group, units, a.joint_tiles);
      mine = joint ? longs : units - longs;
      skipped = joint ? 0 : longs;
    }
    through = mine;
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int x = __shfl_up_sync(0xffffffffu, through, o);
      if (lane >= o) through += x;
    }
    shift = skipped - (through - mine);
  }
  // Every lane of the warp calls this, with the unit it got last, and gets the same unit; false: no more.
  __device__ __forceinline__ bool next(const ChunkArgs& a, Unit& out) {
    if (J && P && out.joint && out.tiles < out.all) {
      out.t0 = out.tiles;
      out.tiles = min(out.all, out.t0 + most);
      return true;
    }
    int w, u;
    for (;;) {
      w = k * stride + (k & 1 ? stride - 1 - id : id);
      u = w / a.kv.kv_heads;
      while (u < total) {
        const int here = __shfl_sync(0xffffffffu, through, 31);
        if (u < before + here) break;
        if (i0 + 32 >= a.batch.b) {
          u = total;
        } else {
          before += here;
          i0 += 32;
          count(a);
        }
      }
      if (u < total) break;
      if (!J || !joint) return false;
      joint = false;
      id = static_cast<int>(blockIdx.x);
      stride = static_cast<int>(gridDim.x);
      k = i0 = before = 0;
      count(a);
    }
    ++k;
    const int from = __ffs(__ballot_sync(0xffffffffu, u - before < through)) - 1;
    const int g = a.group;
    out.i = i0 + from;
    out.head = w - u * a.kv.kv_heads;
    out.row0 = __shfl_sync(0xffffffffu, row0, from);
    out.len = __shfl_sync(0xffffffffu, len, from);
    const int tokens = __shfl_sync(0xffffffffu, n, from);
    const int behind = u - before + __shfl_sync(0xffffffffu, shift, from);  // units of later rows
    out.first = out.len - tokens;
    out.c0 = (row_units(tokens * g) - 1 - behind) * kRows;
    out.rows = unit_rows(tokens * g, out.c0);
    out.all = unit_tiles(out.first, g, out.c0, out.rows);
    out.joint = J && joint;
    out.t0 = 0;
    out.tiles = J && P && out.joint ? min(out.all, most) : out.all;
    return true;
  }
};

__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "
      "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
        "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
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
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_read_x16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_st_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// Load and wait in one statement.
__device__ __forceinline__ void tmem_read_x32(uint32_t taddr, uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {"
      "%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, "
      "%21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]),
        "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]),
        "=r"(r[30]), "=r"(r[31])
      : "r"(taddr)
      : "memory");
}

__device__ __forceinline__ void tmem_read_x8(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}

// One lane of the converged warp, always the same; the compiler then keeps the
// descriptors of the products it issues in uniform registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}

__device__ __forceinline__ float max3(float x, float y, float z) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(x), "f"(y), "f"(z));
  return m;
}

// Pairs of fp32 in one instruction.
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) {
  uint64_t x;
  asm("mov.b64 %0, {%1, %2};" : "=l"(x) : "r"(lo), "r"(hi));
  return x;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ void unpair(uint64_t x, float& lo, float& hi) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x));
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

// One key tile of a unit; t < 0: none.  ends: shared-out units before its own, twice, plus one if its own is.
struct TileRef {
  int i, head, t, len, ends;
};

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
  int warp, lane, sub;

  __device__ __forceinline__ int block(int q) const { return (q * kLoadWarps + warp) * per_warp + lane / lanes; }
  __device__ __forceinline__ void look_up(const ChunkArgs& a, const TileRef& x, int (&page)[NQ]) const {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int p = x.t * kKeys + block(q) * 8;
      page[q] = x.t >= 0 && p < x.len ? page_of(a.kv, x.i, p, a.err) : -1;
    }
  }
  __device__ __forceinline__ void fetch_k(const ChunkArgs& a, const TileRef& x, const int (&page)[NQ]) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      k[q] = make_uint4(0u, 0u, 0u, 0u);
      km[q] = 0u;
      if (page[q] < 0) continue;
      const size_t slot = pool_slot(a.kv, page[q], x.head, x.t * kKeys + block(q) * 8);
      k[q] = ldg128(static_cast<const char*>(a.kv.k) + slot * (D / 2) + sub * 16);
      km[q] = ldg32(static_cast<const char*>(a.kv.k_meta) + (slot + sub / units) * (D / 64) * 4 +
                    (D == 128 ? ((sub % units) >> 1) * 4 : 0));
    }
  }
  __device__ __forceinline__ void fetch_v(const ChunkArgs& a, const TileRef& x, const int (&page)[NQ]) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      v[q] = make_uint4(0u, 0u, 0u, 0u);
      vm[q] = 0u;
      if (page[q] < 0) continue;
      const int p = x.t * kKeys + block(q) * 8;
      const size_t slot = pool_slot(a.kv, page[q], x.head, p);
      v[q] = ldg128(static_cast<const char*>(a.kv.v) + slot * (D / 2) + sub * 16);
      // one pair a lane, in order; tokens behind the end read as zero (their
      // weights are zero, and 0 times an old NaN is not)
      if (sub < 8 * (D / 64) && p + sub / (D / 64) < x.len)
        vm[q] = ldg32(static_cast<const char*>(a.kv.v_meta) + slot * (D / 64) * 4 + sub * 4);
    }
  }
  __device__ __forceinline__ void store_k(uint32_t st) const {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int y = sub / units, u = sub % units;
      const int row = block(q) * 8 + (y < 4 ? 2 * y : 2 * y - 7);
      const __half2 mn = dup_half(km[q], 0), sc = dup_half(km[q], 1);
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
  static constexpr int NQ = 1;  // (head width 64: half the warps have no block)
  static_assert(kLoadWarps * per_warp >= kKeys / 8, "one turn of the warps covers a tile");
  uint4 v[NQ][8];
  int warp, lane, sub;

  __device__ __forceinline__ int block(int q) const { return (q * kLoadWarps + warp) * per_warp + lane / lanes; }
  __device__ __forceinline__ void look_up(const ChunkArgs& a, const TileRef& x, int (&page)[NQ]) const {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int p = x.t * kKeys + block(q) * 8;
      page[q] = block(q) < kKeys / 8 && x.t >= 0 && p < x.len ? page_of(a.kv, x.i, p, a.err) : -1;
    }
  }
  // K straight into its swizzled place; rows behind the end are zeros.
  __device__ __forceinline__ void copy_k(const ChunkArgs& a, const TileRef& x, const int (&page)[NQ], uint32_t st) const {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int p = x.t * kKeys + block(q) * 8;
      const size_t slot = page[q] >= 0 ? pool_slot(a.kv, page[q], x.head, p) : 0;
      if (block(q) >= kKeys / 8) continue;
#pragma unroll
      for (int y = 0; y < 8; ++y)
        cp_async16(st + (sub >> 3) * (kKeys * 128) + sw128(block(q) * 8 + y, sub & 7),
                   static_cast<const char*>(a.kv.k) + (slot + y) * (D * 2) + sub * 16, page[q] >= 0 && p + y < x.len);
    }
    cp_commit();
  }
  __device__ __forceinline__ void fetch_v(const ChunkArgs& a, const TileRef& x, const int (&page)[NQ]) {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int p = x.t * kKeys + block(q) * 8;
      const size_t slot = page[q] >= 0 ? pool_slot(a.kv, page[q], x.head, p) : 0;
#pragma unroll
      for (int y = 0; y < 8; ++y) {
        v[q][y] = make_uint4(0u, 0u, 0u, 0u);
        if (page[q] >= 0 && p + y < x.len)
          v[q][y] = ldg128(static_cast<const char*>(a.kv.v) + (slot + y) * (D * 2) + sub * 16);
      }
    }
  }
  __device__ __forceinline__ void store_v(uint32_t st) const {
#pragma unroll
    for (int q = 0; q < NQ; ++q) {
      const int blk = block(q);
      if (blk >= kKeys / 8) continue;
      const uint32_t base = st + (blk >> 3) * (D * 128);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t o[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          const uint4 &lo = v[q][2 * y], &hi = v[q][2 * y + 1];
          const uint32_t x0 = e < 2 ? lo.x : e < 4 ? lo.y : e < 6 ? lo.z : lo.w;
          const uint32_t x1 = e < 2 ? hi.x : e < 4 ? hi.y : e < 6 ? hi.z : hi.w;
          o[y] = __byte_perm(x0, x1, (e & 1) ? 0x7632 : 0x5410);
        }
        sts128(base + sw128((D / 8) * e + sub, blk & 7), o[0], o[1], o[2], o[3]);  // dimension 8 sub + e
      }
    }
  }
};

// J: in clusters, which share out long units.  P: shares may be longer than kShareTiles.  A cluster then
// takes a unit piece by piece and keeps the pieces' joined output; a CTA alone puts the bulk of O aside in the unit's
// own rows of `out`, as fp16, and goes on with the remainder, which loses nothing.  (Forms of their own: what
// they keep costs the softmax registers, 3240 us instead of 2850 for 148 chunks of 700 tokens over
// 32768 keys shared out.)
template <int D, bool Q4, bool J, bool P>
__global__ void __launch_bounds__(kThreads, 1) attn_paged_chunk_kernel(const ChunkArgs a) {
  using L = Layout<D>;
  constexpr int W = Q4 ? 4 : 8;  // O's column (D / W) e + u is dimension W u + e
  extern __shared__ uint8_t raw_smem[];
  __shared__ Barriers bar;
  __shared__ float s_m[kRows], s_l[kRows];
  __shared__ int s_fail;
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int splits = J ? static_cast<int>(cluster.num_blocks()) : 1, rank = J ? static_cast<int>(cluster.block_rank()) : 0;
  const int lane = static_cast<int>(lane_id());
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);  // (uniform to the compiler)
  const int g = a.group;
  UnitWalk<J, P> walk;
  Unit un{};
  walk.start(a, splits);
  const bool any = walk.next(a, un);
  if (blockIdx.x == 0 && warp == kMmaWarp + 1) check_spans(a.batch, a.err);
  if (!any) return;  // (every warp of the CTA alike; of the cluster, if it has a shared-out unit)

  uint8_t* smem = raw_smem + ((1024 - (smem_u32(raw_smem) & 1023)) & 1023);
  const uint32_t sbase = smem_u32(smem);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&bar.k_full[s], kLoadWarps);
      mbar_init(&bar.v_full[s], kLoadWarps);
      mbar_init(&bar.k_empty[s], 1);
      mbar_init(&bar.v_empty[s], 1);
    }
    for (int m = 0; m < 2; ++m) {
      mbar_init(&bar.q_full[m], 4);
      mbar_init(&bar.s_full[m], 1);
      mbar_init(&bar.p_full[m], 4);
      mbar_init(&bar.o_full[m], 1);
      mbar_init(&bar.o_free[m], 4);
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
  const uint32_t tmem = __shfl_sync(0xffffffffu, bar.tmem, 0);
  auto wait = [&](uint64_t* b, uint32_t parity, uint32_t code) {
    if (wait_phase(b, parity, a.limit_ns)) return true;
    set_error(a.err, code);
    atomicExch(&s_fail, 1);
    return false;
  };
  // key tiles of this CTA: all, or rank, rank + splits, ..
  auto start_of = [&](const Unit& x) { return J && P ? x.t0 : 0; };
  auto first_of = [&](const Unit& x) { return J && x.joint ? start_of(x) + rank : 0; };
  auto step_of = [&](const Unit& x) { return J && x.joint ? splits : 1; };
  auto tiles_of = [&](const Unit& x) {
    return !J || !x.joint ? x.tiles : share_tiles(x.tiles - start_of(x), rank, splits);
  };
  // A shared-out unit ends with two barriers of the whole cluster, which every warp passes whatever
  // became of its waits: parts are written before the first and read before the second.  No wait of a
  // role falls between them, so all see the same failures and leave together.
  auto cluster_sync = [&]() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  };
  auto cluster_fine = [&]() {
    bool fine = true;
#pragma unroll 1
    for (int k = 0; k < splits; ++k) fine &= *cluster.map_shared_rank(&s_fail, k) == 0;
    return __all_sync(0xffffffffu, fine) != 0;
  };
  auto unit_end = [&]() {  // (false: no further unit)
    cluster_sync();
    const bool fine = cluster_fine();
    cluster_sync();
    return fine;
  };

  if (warp < kSoftmaxWarps) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
    // --- softmax of one row -------------------------------------------------------
    const int m = warp >> 2, row = threadIdx.x;  // row of the unit: TMEM lane row % 128 of row tile m
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + m * 128, o_col = tmem + lanes + 256 + m * D;
    const float inv_scale = 1.f / a.scale_log2;
    // Q's row into its swizzled place (every product that read the last one has completed)
    auto load_q = [&](const Unit& x) {
      const bool live = row < x.rows;
      const int c = x.c0 + (live ? row : 0), tok = c / g;
      const __half* src = a.q + static_cast<size_t>(x.row0 + tok) * a.ldq + (x.head * g + c - tok * g) * D;
      const uint32_t dst = sbase + m * L::q_tile;
#pragma unroll
      for (int ch = 0; ch < D / 8; ++ch) {
        const uint4 v = live ? *reinterpret_cast<const uint4*>(src + ch * 8) : make_uint4(0u, 0u, 0u, 0u);
        const uint32_t at = dst + (ch >> 3) * (128 * 128) + sw128(row & 127, ch & 7);
        if (Q4)  // (e, e + 4)
          sts128(at, __byte_perm(v.x, v.z, 0x5410), __byte_perm(v.x, v.z, 0x7632), __byte_perm(v.y, v.w, 0x5410),
                 __byte_perm(v.y, v.w, 0x7632));
        else
          sts128(at, v.x, v.y, v.z, v.w);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.q_full[m]);
    };
    bool more = true, ok = true;
    // row tile 1: units that have one (of a shared-out unit, the join alone)
    while (more && !(J && un.joint) && m * 128 >= un.rows) more = walk.next(a, un);
    if (more && m * 128 < un.rows) load_q(un);
    uint32_t s_phase = 0, o_phase = 0;  // o_phase: bit m row tile m's
    while (more) {
      const Unit cur = un;
      const bool has = !J || m * 128 < cur.rows;
      const bool live = row < cur.rows;
      const int c = cur.c0 + (live ? row : 0), tok = c / g;
      const int pos = live ? cur.first + tok : cur.len;
      const int mine = has ? tiles_of(cur) : 0;
      float base = -INFINITY;   // exponent base: log2 of the weights' unit, a whole number
      float limit = -INFINITY;  // the raw score that moves it
      uint64_t sum = 0;        // sums of the even and the odd columns' weights
      int lim = pos - first_of(cur) * kKeys;  // tokens 0 .. lim of the tile count
      __half* dst = a.out + static_cast<size_t>(cur.row0 + tok) * a.ldo + (cur.head * g + c - tok * g) * D;
      float unit = 0.f;   // of what is put aside in dst: O's columns (D / W) e + u0 .. + 7 at W u0 + 8 e .. + 7
      float aside = 0.f;  // the weights' sum put aside with it
      auto put_aside = [&]() {
        // |O| is at most the weights' sum times 65504 (and 2^-11 of that): with twice the sum's power of two
        // as the unit it is in fp16's range.  Read, add, round, keep the remainder: all exact but the addition.
        float s0, s1;
        unpair(sum, s0, s1);
        aside += s0 + s1;
        sum = 0;
        const int ex = (__float_as_int(aside) >> 23) - 127 + 2;
        const float next = __int_as_float((ex + 127) << 23), inv = __int_as_float((127 - ex) << 23);
#pragma unroll 1
        for (int x0 = 0; x0 < D; x0 += 32) {  // 16-byte pieces of dst, four at a time
          uint4 was[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            was[i] = make_uint4(0u, 0u, 0u, 0u);
            if (live && unit != 0.f) was[i] = *reinterpret_cast<const uint4*>(dst + x0 + 8 * i);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int x = x0 + 8 * i, col = (D / W) * (x / 8 % W) + x / (8 * W) * 8;
            uint32_t o[8];
            tmem_read_x8(o_col + col, o);
            const uint32_t t[4] = {was[i].x, was[i].y, was[i].z, was[i].w};
            uint32_t to[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 w = __half22float2(as_half2(t[k]));
              const float y0 = fmaf(w.x, unit, __uint_as_float(o[2 * k])), y1 = fmaf(w.y, unit, __uint_as_float(o[2 * k + 1]));
              to[k] = pack_half2(y0 * inv, y1 * inv);
              const float2 n = __half22float2(as_half2(to[k]));
              o[2 * k] = __float_as_uint(fmaf(-n.x, next, y0));
              o[2 * k + 1] = __float_as_uint(fmaf(-n.y, next, y1));
            }
            if (live) *reinterpret_cast<uint4*>(dst + x) = make_uint4(to[0], to[1], to[2], to[3]);
            tmem_st_x8(o_col + col, o);
          }
        }
        unit = next;
        tmem_st_wait();
      };
      for (int it = 0; it < mine; ++it, lim -= step_of(cur) * kKeys) {
        if (!(ok = __all_sync(0xffffffffu, wait(&bar.s_full[m], s_phase, DEV_TIMEOUT_EPILOGUE)))) break;
        s_phase ^= 1;
        tc_fence_after();
        if (!J && P && it > 0 && it % kShareTiles == 0) put_aside();
        if (__any_sync(0xffffffffu, lim < kKeys - 1)) {
          // the scores behind the row's position leave S here
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t s[32];
            tmem_read_x32(s_col + 32 * ch, s);
            const int here = lim - 32 * ch;
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              const int t = Q4 ? (e & ~7) + ((e & 7) >> 1) + 4 * (e & 1) : e;
              if (t > here) s[e] = 0xff800000u;
            }
            tmem_st_x32(s_col + 32 * ch, s);
          }
          tmem_st_wait();
        }
        uint64_t sums[4] = {sum, 0, 0, 0};  // (17 roundings a tile: 2^-13 over kShareTiles at the most)
        uint32_t s[2][32];
        tmem_ld_x32(s_col, s[0]);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t(&x)[32] = s[ch & 1];
          tmem_wait_x32(x);
          if (ch < 3) tmem_ld_x32(s_col + 32 * (ch + 1), s[(ch + 1) & 1]);
          float top = -INFINITY, top1 = -INFINITY;
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            top = max3(top, __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
            top1 = max3(top1, __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
          }
          top = fmaxf(top, top1);
          if (__any_sync(0xffffffffu, top > limit)) {  // (from -inf: any finite score)
            // P of the columns before, and O after an earlier move in this tile, were stored by this
            // thread and are read back here: only the wait orders the two
            tmem_st_wait();
            const float nb = top > limit ? ceilf(top * a.scale_log2) : base;
            const float alpha = base == -INFINITY ? 0.f : exp2_approx(base - nb);
            base = nb;
            if (!J && P) {
              unit *= alpha;
              aside *= alpha;
            }
            limit = (nb + kWeightSlack) * inv_scale;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float s0, s1;
              unpair(sums[k], s0, s1);
              sums[k] = pair(__float_as_uint(s0 * alpha), __float_as_uint(s1 * alpha));
            }
#pragma unroll 1
            for (int q = 0; q < ch; ++q) {
              uint32_t o[16];
              tmem_read_x16(s_col + 16 * q, o);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                // (in fp32: the factor itself may lie below fp16's range)
                const float2 y = __half22float2(as_half2(o[e]));
                o[e] = pack_half2(y.x * alpha, y.y * alpha);
              }
              tmem_st_x16(s_col + 16 * q, o);
            }
            if (it > 0) {
#pragma unroll 1
              for (int q = 0; q < D / 16; ++q) {
                uint32_t o[16];
                tmem_read_x16(o_col + 16 * q, o);
#pragma unroll
                for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st_x16(o_col + 16 * q, o);
              }
            }
          }
          const uint32_t off = __float_as_uint(base == -INFINITY ? 0.f : kWeightBias - base);
          const uint64_t off2 = pair(off, off), scale2 = pair(__float_as_uint(a.scale_log2), __float_as_uint(a.scale_log2));
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float x0, x1;
            unpair(fma2(pair(x[e], x[e + 1]), scale2, off2), x0, x1);
            x0 = exp2_approx(x0);
            x1 = exp2_approx(x1);
            sums[(e / 2) & 3] = add2(sums[(e / 2) & 3], pair(__float_as_uint(x0), __float_as_uint(x1)));
            p[e / 2] = pack_half2(x0, x1);
          }
          tmem_st_x16(s_col + 16 * ch, p);  // over columns of S that are read
        }
        sum = add2(add2(sums[0], sums[1]), add2(sums[2], sums[3]));
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.p_full[m]);
      }
      float s0, s1;
      unpair(sum, s0, s1);
      if (!J || !cur.joint) {
        if (!ok) break;
        do more = walk.next(a, un);
        while (more && m * 128 >= un.rows);
        if (more) load_q(un);

        if (!(ok = __all_sync(0xffffffffu, wait(&bar.o_full[m], (o_phase >> m) & 1, DEV_TIMEOUT_EPILOGUE)))) break;
        tc_fence_after();
        const float inv = 1.f / (s0 + s1 + aside);
#pragma unroll 1
        for (int u0 = 0; u0 < D / W; u0 += 8) {
          uint32_t o[W][8];
#pragma unroll
          for (int e = 0; e < W; ++e) tmem_read_x8(o_col + (D / W) * e + u0, o[e]);
          if (live) {
            if (!J && P && cur.all > kShareTiles) {
#pragma unroll
              for (int e = 0; e < W; ++e) {
                const uint4 was = *reinterpret_cast<const uint4*>(dst + W * u0 + 8 * e);
                const uint32_t* t = reinterpret_cast<const uint32_t*>(&was);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                  const float2 w = __half22float2(as_half2(t[i]));
                  o[e][2 * i] = __float_as_uint(fmaf(w.x, unit, __uint_as_float(o[e][2 * i])));
                  o[e][2 * i + 1] = __float_as_uint(fmaf(w.y, unit, __uint_as_float(o[e][2 * i + 1])));
                }
              }
            }
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
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.o_free[m]);
      } else {
        if (ok && has) ok = __all_sync(0xffffffffu, wait(&bar.o_full[m], (o_phase >> m) & 1, DEV_TIMEOUT_EPILOGUE));
        if (ok && has && cur.rows > 128)  // the parts are laid over K and V: wait for both row tiles
          ok = __all_sync(0xffffffffu, wait(&bar.o_full[m ^ 1], (o_phase >> (m ^ 1)) & 1, DEV_TIMEOUT_EPILOGUE));
        if (ok && has) {
          tc_fence_after();
          s_m[row] = base;
          s_l[row] = s0 + s1;
          // in O's column order, 16-byte units XORed by the row
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
          tc_fence_before();
          __syncwarp();
          if (lane == 0 && mine > 0) mbar_arrive(&bar.o_free[m]);
        }
        cluster_sync();
        const bool fine = cluster_fine();
        // join the cluster's parts, N dimensions of a row at a time: C columns of each of O's W
        // stretches.  Where the unit goes on, the thread keeps what it has and takes it up again: pieces
        // are only of clusters of eight, where nobody has more than one item.
        constexpr int C = P ? 16 / W : 4, N = C * W, items = D / N;
        static_assert(!P || items <= kMaxCluster, "one item a thread");
        using Cols = typename std::conditional<C == 4, float4, float2>::type;
        // (an aligned base is at the same offset in every CTA of the launch)
        const float* parts = reinterpret_cast<const float*>(smem + L::k0);
        float4* kept = reinterpret_cast<float4*>(smem + L::bytes) + threadIdx.x;
        float* kept_m = reinterpret_cast<float*>(smem + L::bytes + kRows * 64) + threadIdx.x;
        const bool goes_on = P && cur.tiles < cur.all, resumed = P && cur.t0 > 0;
#pragma unroll 1
        for (int x = rank * kRows + static_cast<int>(threadIdx.x); fine && x < items * kRows; x += splits * kRows) {
          const int jr = x % kRows, u = x / kRows;
          if (jr >= cur.rows) break;
          float f[kMaxCluster], top = -INFINITY, den = 0.f, back = 0.f;
#pragma unroll
          for (int k = 0; k < kMaxCluster; ++k) {
            f[k] = k < splits ? *cluster.map_shared_rank(&s_m[jr], k) : -INFINITY;
            top = fmaxf(top, f[k]);
          }
          if (resumed) {
            const float m0 = kept_m[0];  // (finite: every row sees the first tile)
            top = fmaxf(top, m0);
            back = exp2_approx(m0 - top);
            den = back * kept_m[kRows];
          }
#pragma unroll
          for (int k = 0; k < kMaxCluster; ++k) {
            f[k] = f[k] == -INFINITY ? 0.f : exp2_approx(f[k] - top);
            if (k < splits) den += f[k] * *cluster.map_shared_rank(&s_l[jr], k);
          }
          float o[N];
#pragma unroll
          for (int q = 0; q < N / 4; ++q) {
            const float4 was = resumed ? kept[q * kRows] : make_float4(0.f, 0.f, 0.f, 0.f);
            o[4 * q] = back * was.x;
            o[4 * q + 1] = back * was.y;
            o[4 * q + 2] = back * was.z;
            o[4 * q + 3] = back * was.w;
          }
#pragma unroll
          for (int q = 0; q < W; ++q) {
            const float* at = parts + jr * D + ((((q * (D / W) + C * u) >> 2) ^ (jr & 7)) << 2) + ((C * u) & 3);
#pragma unroll
            for (int k = 0; k < kMaxCluster; ++k) {
              if (k >= splits) continue;
              const Cols pk = *reinterpret_cast<const Cols*>(cluster.map_shared_rank(at, k));
              const float* e = reinterpret_cast<const float*>(&pk);
#pragma unroll
              for (int c = 0; c < C; ++c) o[q * C + c] += f[k] * e[c];
            }
          }
          if (goes_on) {
            kept_m[0] = top;
            kept_m[kRows] = den;
#pragma unroll
            for (int q = 0; q < N / 4; ++q) kept[q * kRows] = make_float4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
            continue;
          }
          const float inv = 1.f / den;
          const int jc = cur.c0 + jr;
          __half* dst = a.out + static_cast<size_t>(cur.row0 + jc / g) * a.ldo + (cur.head * g + jc % g) * D + u * N;
#pragma unroll
          for (int e = 0; e < N; e += 8) {  // dimension e of these: stretch e % W, column e / W
            uint32_t h[4];
#pragma unroll
            for (int i = 0; i < 8; i += 2)
              h[i / 2] = pack_half2(o[(e + i) % W * C + (e + i) / W] * inv, o[(e + i + 1) % W * C + (e + i + 1) / W] * inv);
            *reinterpret_cast<uint4*>(dst + e) = make_uint4(h[0], h[1], h[2], h[3]);
          }
        }
        cluster_sync();  // nobody writes, or leaves, while another reads its shared memory
        if (!fine) break;
        do more = walk.next(a, un);
        while (more && !(J && un.joint) && m * 128 >= un.rows);
        if (more && m * 128 < un.rows) load_q(un);
      }
      o_phase ^= cur.rows > 128 ? 3u : 1u;
    }
  } else if (warp < kMmaWarp) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    // --- K and V ------------------------------------------------------------------
    using Ld = Loader<D, Q4>;
    Ld ld;
    ld.warp = warp - kSoftmaxWarps;
    ld.lane = lane;
    ld.sub = lane % Ld::lanes;
    bool more = true;
    int it = 0, mine = tiles_of(un), units = 0;
    auto advance = [&]() {  // the CTA's next tile
      while (more && it == mine) {
        units += un.joint;
        more = walk.next(a, un);
        it = 0;
        mine = more ? tiles_of(un) : 0;
      }
      TileRef x{un.i, un.head, -1, un.len, 2 * units + un.joint};
      if (more) x.t = first_of(un) + it++ * step_of(un);
      return x;
    };
    TileRef cur = advance(), next = advance();
    int page[Ld::NQ], next_page[Ld::NQ];
    ld.look_up(a, cur, page);
    ld.look_up(a, next, next_page);
    if constexpr (Q4) ld.fetch_k(a, cur, page);
    if constexpr (Q4) ld.fetch_v(a, cur, page);
    int ended = 0;  // shared-out units behind this warp
    bool fine = true;
    auto end_units = [&](int count) {
      for (; J && fine && ended < count; ++ended) fine = unit_end();
    };
    for (int n = 0; cur.t >= 0; ++n) {
      end_units(cur.ends >> 1);  // (their parts lie over the stages)
      if (!fine) break;
      const int st = n % kStages;
      const uint32_t free_parity = ((n / kStages) & 1) ^ 1;
      const uint32_t ks = sbase + L::k0 + st * L::k_stage, vs = sbase + L::v0 + st * L::v_stage;
      if (!__all_sync(0xffffffffu, wait(&bar.k_empty[st], free_parity, DEV_TIMEOUT_PRODUCER))) {
        units = (cur.ends + 1) >> 1;
        break;
      }
      if constexpr (Q4) {
        ld.store_k(ks);
      } else {
        ld.copy_k(a, cur, page, ks);
        ld.fetch_v(a, cur, page);
        cp_wait<0>();
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.k_full[st]);
      if constexpr (Q4) ld.fetch_k(a, next, next_page);
      if (!__all_sync(0xffffffffu, wait(&bar.v_empty[st], free_parity, DEV_TIMEOUT_PRODUCER))) {
        units = (cur.ends + 1) >> 1;
        break;
      }
      ld.store_v(vs);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar.v_full[st]);
      if constexpr (Q4) ld.fetch_v(a, next, next_page);
      cur = next;
      next = advance();
#pragma unroll
      for (int q = 0; q < Ld::NQ; ++q) page[q] = next_page[q];
      ld.look_up(a, next, next_page);
    }
    end_units(units);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kMmaRegs));
    if (warp == kMmaWarp) {
      // --- products: one lane issues them ---------------------------------------------
      const uint32_t id_s = idesc_f16_m128(kKeys), id_o = idesc_f16_m128(D);
      auto issue_s = [&](int m, int st, bool last) {
        const uint64_t q_desc = sw128_kmajor_desc(sbase + m * L::q_tile);
        const uint64_t k_desc = sw128_kmajor_desc(sbase + L::k0 + st * L::k_stage);
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * (128 * 128) + (kk & 3) * 32) >> 4;  // (addresses are in units of 16 bytes)
          mma_f16_ss(tmem + m * 128, q_desc + off, k_desc + off, id_s, kk > 0);
        }
        mma_commit(&bar.s_full[m]);
        if (last) mma_commit(&bar.k_empty[st]);
      };
      auto ready = [&](uint64_t* b, uint32_t parity) { return wait(b, parity, DEV_TIMEOUT_MMA); };
      bool ok = true, more = true;
      int n0 = 0;  // tiles of the units before
      uint32_t q_phase = 0, p_phase = 0, o_phase = 3;  // bit m: row tile m's
      while (ok && more) {
        const int mtiles = un.rows > 128 ? 2 : 1, mine = tiles_of(un);
        if (elect_one()) {
          if (mine > 0) ok = ready(&bar.k_full[n0 % kStages], (n0 / kStages) & 1);
          for (int m = 0; ok && m < mtiles; ++m) {
            ok = ready(&bar.q_full[m], (q_phase >> m) & 1);
            tc_fence_after();
            if (ok && mine > 0) issue_s(m, n0 % kStages, m == mtiles - 1);
            if (ok && mine == 0) mma_commit(&bar.o_full[m]);  // a share of no tiles: nothing to add
          }
          uint32_t p_par = p_phase;
          for (int it = 0; ok && it < mine; ++it, p_par ^= 3) {
            const int n = n0 + it, st = n % kStages, ns = (n + 1) % kStages;
            const uint64_t v_desc = sw128_kmajor_desc(sbase + L::v0 + st * L::v_stage);
            ok = ready(&bar.v_full[st], (n / kStages) & 1);
            for (int m = 0; ok && m < mtiles; ++m) {
              if (it == 0) ok = ready(&bar.o_free[m], (o_phase >> m) & 1);  // the last unit's output has been read
              ok = ok && ready(&bar.p_full[m], (p_par >> m) & 1);
              if (!ok) break;
              tc_fence_after();
#pragma unroll
              for (int kk = 0; kk < kKeys / 16; ++kk)
                mma_f16_ts(tmem + 256 + m * D, tmem + m * 128 + kk * 8,
                           v_desc + (((kk >> 2) * (D * 128) + (kk & 3) * 32) >> 4), id_o, it > 0 || kk > 0);
              if (it + 1 == mine) mma_commit(&bar.o_full[m]);
              if (m == mtiles - 1) mma_commit(&bar.v_empty[st]);
              if (it + 1 < mine) {
                if (m == 0) ok = ready(&bar.k_full[ns], ((n + 1) / kStages) & 1);
                if (!ok) break;
                tc_fence_after();
                issue_s(m, ns, m == mtiles - 1);  // over P: the products run in the order of issue
              }
            }
          }
        }
        ok = __all_sync(0xffffffffu, ok) != 0;
        const uint32_t used = mtiles == 2 ? 3 : 1;
        n0 += mine;
        q_phase ^= used;
        if (mine > 0) o_phase ^= used;
        if (mine & 1) p_phase ^= used;
        if (J && un.joint) more = unit_end();  // (not ok: nor is it fine)
        if (ok && more) more = walk.next(a, un);
      }
      __syncwarp();
      if (elect_one()) {
        mma_commit(&bar.done);
        // the products in flight have read shared and tensor memory before the CTA lets go of
        // them, whatever the waits' limit
        if (!wait_phase(&bar.done, 0, kDrainNs)) set_error(a.err, DEV_TIMEOUT_MMA);
      }
    } else {
      for (bool more = J; more && un.joint;) more = unit_end() && walk.next(a, un);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  pdl_trigger();
  if (warp == kMmaWarp) tmem_dealloc(tmem, kTmemCols);
}

template <int D, bool Q4, bool J, bool P>
cudaError_t launch_j(const ChunkArgs& a, long long works, int splits, cudaStream_t s) {
  constexpr int smem = Layout<D>::smem + (J && P ? Layout<D>::kept : 0);
  cudaError_t e = allow_smem<attn_paged_chunk_kernel<D, Q4, J, P>>(smem);
  if (e != cudaSuccess) return e;
  int dev = 0, regs = 0;
  if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
  // the split of the registers counts on the launch having them
  static PerDevice registers;
  e = registers.get(dev, &regs, [](int* n) {
    cudaFuncAttributes f{};
    const cudaError_t err = cudaFuncGetAttributes(&f, attn_paged_chunk_kernel<D, Q4, J, P>);
    *n = f.numRegs;
    return err;
  });
  if (e != cudaSuccess) return e;
  if (regs < kLaunchRegs) return cudaErrorInvalidConfiguration;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(splits));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = runtime().pdl ? 2 : 1;
  // one CTA an SM, or as many clusters as are resident at once
  static PerDevice resident[kMaxCluster + 1];
  int clusters = runtime().num_sms;
  if (J) {
    e = resident[splits].get(dev, &clusters, [&cfg](int* n) {
      const cudaError_t err = cudaOccupancyMaxActiveClusters(n, attn_paged_chunk_kernel<D, Q4, J, P>, &cfg);
      *n = std::max(*n, 1);
      return err;
    });
    if (e != cudaSuccess) return e;
  }
  cfg.gridDim = dim3(static_cast<unsigned>(std::min<long long>(works, clusters) * splits));
  e = cudaLaunchKernelEx(&cfg, attn_paged_chunk_kernel<D, Q4, J, P>, a);
  return e != cudaSuccess ? e : launched();
}

template <int D, bool Q4>
cudaError_t launch_d(const ChunkArgs& args, cudaStream_t s) {
  const int sms = runtime().num_sms;
  const long long works = unit_total(args.batch.rows, args.batch.b, args.group, kUnitRowShift, 1) * args.kv.kv_heads;
  // Units that the batch's rows fill.  Histories are shared out while that leaves SMs idle and every
  // CTA keeps two tiles of keys; and, while an SM has few units, very long ones too, into shares
  // of 32 tiles and more: the longest unit's CTA would work on alone (12 sequences of up to 24000 keys,
  // 16 heads: 538 us in one piece)
  const long long full =
      ((static_cast<long long>(args.batch.rows) * args.group + kRows - 1) / kRows) * args.kv.kv_heads;
  int splits = 1;
  while (splits < kMaxCluster && full * splits * 2 <= sms && args.batch.max_len > splits * 2 * 2 * kKeys) splits *= 2;
  ChunkArgs a = args;
  a.joint_tiles = splits > 1 ? 2 * splits : 48;
  while (splits < kMaxCluster && full < 4ll * sms && args.batch.max_len / (2 * splits) >= 32 * kKeys) splits *= 2;
  // (clusters: no share longer than an accumulator takes, as far as their size goes)
  while (splits > 1 && splits < kMaxCluster && args.batch.max_len > splits * kShareTiles * kKeys) splits *= 2;
  const bool pieces = args.batch.max_len > splits * kShareTiles * kKeys;
  if (splits == 1) return pieces ? launch_j<D, Q4, false, true>(a, works, 1, s) : launch_j<D, Q4, false, false>(a, works, 1, s);
  return pieces ? launch_j<D, Q4, true, true>(a, works, splits, s) : launch_j<D, Q4, true, false>(a, works, splits, s);
}

}  // namespace

cudaError_t launch_attn_paged_chunks(const PagedView& kv, const RaggedView& batch, int heads, int d, int kv_bits,
                                     int min_rows, const __half* q, int ldq, __half* out, int ldo, cudaStream_t s) {
  const ChunkArgs a{kv, batch, heads / kv.kv_heads, min_rows, 0, q, ldq, out, ldo,
                    1.4426950408889634f / sqrtf(static_cast<float>(d)), runtime().wait_limit_ns, runtime().err};
  if (kv_bits == 4) return d == 128 ? launch_d<128, true>(a, s) : launch_d<64, true>(a, s);
  return d == 128 ? launch_d<128, false>(a, s) : launch_d<64, false>(a, s);
}

}  // namespace flexq
