// Attention of a ragged batch of new tokens over the paged cache:
// o = softmax(q K^T / sqrt(d)) V over positions 0..p for the row at position p.
//
// This file: sequences with few query rows (n new tokens x heads/kv_heads query heads
// of one key/value head at most 8 NT), the decode step.  Reading the cache once
// is the bound: its bytes are used by all the rows that share a head.  The rows are
// the 8 (or 16) columns of mma.sync with K and V as the wide operand:
//   S^T [keys x rows] = K [keys x d] Q^T,   O^T [d x rows] = V^T [d x keys] P^T,
// so a lane keeps the running maximum and sum of the same two rows in both products, and
// the weights pass from one to the other by one 8x8 transpose a block of 8 keys.
// The order of keys and dimensions inside the products is free, and is chosen so that a
// lane's codes sit in 16-byte reads and come out as the fp16 pairs that the fragments want:
// the 4-bit words are dequantized in registers, never stored as fp16.
//
// A warp walks tiles of 32 keys (16 of an fp16 cache) through its own ring of
// asynchronous 16-byte copies; the warps of a CTA, and the CTAs of a cluster
// where one unit's history is shared out, take tiles in turn.  Their (maximum, sum,
// output) are joined in a fixed order: in shared memory, then over the cluster's
// distributed shared memory, so the call needs no workspace.
//
// Measured (B200): 144 sequences of 300 to 1040 keys, 56 heads, d = 128, 4 bit: 200 to 214 us from box to
// box for 788 MB, 0.57 to 0.60 of the copy rate; five of 18900 to 32700 keys, 8 key/value heads: 58 to 61 us for
// 149 MB (the clusters are alike, the histories are not: the longest is 1.3 times the mean); one fp16
// sequence of 902 keys, 32 heads, d = 64: 5.8 us, the launch.  The 4-bit form has no unit at its
// roof.  Closest is the half-precision pipe that the dequantizer's eight multiply-adds and the mma.sync of
// a word share: 23 cycles a word and scheduler alone in a loop, 750 cycles a tile of the 1150 that it takes,
// and by itself it would allow nearly the copy rate.  The rest is what a warp does in sequence (dequantize K,
// products, maximum, exponentials, transpose, dequantize V, products) with 13 warps an SM to overlap it.
// Three quarters of the registers (18 warps an SM) gained nothing (214 us), nor did two stages instead of
// three.  An fp16 cache has no dequantizer: 64 sequences of 528 keys, 32 heads, d = 128, read at 6.2 TB/s.
#include <cooperative_groups.h>
#include <math.h>

#include <algorithm>

#include "paged.cuh"
#include "warp_mma.cuh"

namespace flexq {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxWarps = 8;
constexpr int kMaxCluster = 8;

struct PagedAttnArgs {
  PagedView kv;
  RaggedView batch;
  int heads, group;
  const __half* q;
  int ldq;
  __half* out;
  int ldo;
  float scale_log2;
  float slack;        // kWeightSlack / scale_log2
  uint32_t by_group;  // c / group = (c * by_group) >> 16 for the columns c < 16
  uint32_t* err;
};

template <int D, bool Q4>
struct Tile {
  static constexpr int keys = Q4 ? 32 : 16;
  static constexpr int blocks = keys / 8;         // 8-token blocks; a block never crosses a page
  static constexpr int lanes = 32 / blocks;       // lanes that copy a block
  static constexpr int row = Q4 ? D / 2 : D * 2;  // bytes of a key's codes (values)
  static constexpr int side = keys * row;         // bytes of K, and of V
  static constexpr int meta = Q4 ? keys * (D / 64) * 4 : 0;
  static constexpr int bytes = 2 * side + 2 * meta;
  static constexpr int stages = 3;
  static constexpr int chunks = 8 * row / 16;  // 16-byte units of a block's K (and V)
};

// Copies tile t of sequence i (key/value head base `head`) into a stage.  A lane
// copies parts of one 8-token block, whose page it is given (-1: behind
// the end, or refused; zeros then).
template <int D, bool Q4>
__device__ __forceinline__ void load_tile(const PagedView& kv, int head, int t, int page, uint32_t st, int lane) {
  using T = Tile<D, Q4>;
  const int blk = lane / T::lanes, m = lane % T::lanes;
  const bool ok = page >= 0;
  const size_t slot = pool_slot(kv, ok ? page : 0, head, ok ? t * T::keys + blk * 8 : 0);
  const char* k = static_cast<const char*>(kv.k) + slot * T::row;
  const char* v = static_cast<const char*>(kv.v) + slot * T::row;
  const uint32_t ks = st + blk * 8 * T::row, vs = ks + T::side;
#pragma unroll
  for (int c0 = 0; c0 < T::chunks; c0 += T::lanes) {
    const int c = c0 + m;
    int ck, cv;
    if (Q4) {
      // K: keys 4.. of a block (and, with two units a key, every other block) XORed to
      // other bank groups; V: the unit XORed by the block
      constexpr int U = D / 32;
      ck = c ^ (((c / U) >> 2) * (D == 128 ? 4 : 2)) ^ (D == 64 ? (blk & 1) * 4 : 0);
      cv = c ^ (2 * blk);
    } else {
      constexpr int U = D / 8;
      const int y = c / U, u = c % U;
      ck = y * U + (D == 128 ? u ^ ((u >> 3) << 1) ^ (y & 1) : u ^ (y & 1));
      cv = y * U + (u ^ y);
    }
    cp_async16(ks + ck * 16, k + c * 16, ok);
    cp_async16(vs + cv * 16, v + c * 16, ok);
  }
  if (Q4) {
    constexpr int MC = 8 * (D / 64) * 4 / 16;  // units of a block's pairs: 4 (d 128) or 2
    if ((m & 3) < MC) {
      const void* src = (m & 4) ? kv.v_meta : kv.k_meta;
      cp_async16(st + 2 * T::side + ((m & 4) ? T::meta : 0) + blk * MC * 16 + (m & 3) * 16,
                 static_cast<const char*>(src) + slot * (D / 64) * 4 + (m & 3) * 16, ok);
    }
  }
}

// Makes the tokens of the stage's tile at and behind `len` zeros of V: their
// weights are zero, but 0 times a slot's old NaN is not.
template <int D, bool Q4>
__device__ __forceinline__ void clear_tail(uint32_t st, int t, int len, int lane) {
  using T = Tile<D, Q4>;
  if (Q4) {
    if (t * 32 + lane >= len) {
      const uint32_t a = st + 2 * T::side + T::meta + lane * (D / 64) * 4;
      asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(0u) : "memory");
      if (D == 128) asm volatile("st.shared.b32 [%0], %1;" ::"r"(a + 4), "r"(0u) : "memory");
    }
  } else {
    for (int y = max(0, len - t * T::keys); y < T::keys; ++y)
      for (int u = lane; u < D / 8; u += 32)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(st + T::side + y * T::row + u * 16), "r"(0u) : "memory");
  }
  __syncwarp();
}

__device__ __forceinline__ uint32_t word_of(const uint4& v, int i) {
  return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w;
}
__device__ __forceinline__ __half2 as_half2(uint32_t x) { return *reinterpret_cast<__half2*>(&x); }

// The tensor core truncates, always towards zero, when it adds to its accumulator: O lost 3e-5 of
// its size over 128 tiles a warp, and 8e-4 over 4096 (262144 keys of values of one sign).  Fold: a
// tile's products start from zero and are added to O with rounding, which over n tiles is at most
// n 2^-25 off and has no direction of its own (4e-5 over 4096).  It costs 4 % (4736 histories of 262144
// keys, one head: 37.9 ms with it, 36.5 without), so shares of up to kPlainTiles tiles, whose 512 additions of at most 2^-23
// each cannot come to more than a quarter of the output's own rounding, 2^-13, are added up in the accumulator.
constexpr int kPlainTiles = 256;

template <int D, bool Q4, int NT, bool Fold>
__global__ void __maxnreg__(NT == 1 ? 128 : 168) attn_paged_rows_kernel(const PagedAttnArgs a) {
  using T = Tile<D, Q4>;
  constexpr int NC = 8 * NT;       // columns: query rows
  constexpr int DL = D / 4;        // dimensions of Q and K that a lane holds
  constexpr int WL = DL / 8;       // ... in words of eight
  constexpr int MT = D / 16;       // 16-dimension tiles of the output
  constexpr int KM = T::keys / 16; // 16-key tiles
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float s_m[kMaxWarps][NC], s_l[kMaxWarps][NC];
  __shared__ float c_m[NC], c_l[NC];
  pdl_wait();
  cg::cluster_group cluster = cg::this_cluster();
  const int splits = static_cast<int>(cluster.num_blocks()), rank = static_cast<int>(cluster.block_rank());
  const int lane = static_cast<int>(lane_id()), warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
  const int r = lane >> 2, j = lane & 3;
  const int unit = blockIdx.x / splits;
  const int i = unit / a.kv.kv_heads, head = unit % a.kv.kv_heads;
  const Span sp = ragged_span(a.batch, i, a.err);
  const int g = a.group;
  const int cols = sp.n * g;
  if (sp.n == 0 || cols > NC) return;  // (every CTA of the cluster alike)
  const int tiles = (sp.len + T::keys - 1) / T::keys;
  const int first = sp.len - sp.n;  // position of the first new token
  const int step = splits * warps;
  auto token_of = [&](int c) { return static_cast<int>((c * a.by_group) >> 16); };
  uint8_t* ring = smem + warp * T::stages * T::bytes;

  // the lane's page of tile t (looked up one tile before its copies start)
  const int my_blk = (lane / T::lanes) * 8;
  auto page_for = [&](int t) {
    const int p = t * T::keys + my_blk;
    return p < sp.len ? page_of(a.kv, i, p, a.err) : -1;
  };
  int t_load = rank * warps + warp;
#pragma unroll
  for (int s = 0; s < T::stages - 1; ++s) {
    if (t_load < tiles) load_tile<D, Q4>(a.kv, head, t_load, page_for(t_load), smem_u32(ring + s * T::bytes), lane);
    cp_commit();
    t_load += step;
  }
  int next_page = t_load < tiles ? page_for(t_load) : -1;

  // Q: column nt * 8 + r, dimensions DL j .., pairs in the order of K's
  uint32_t qf[NT][WL][4];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int c = nt * 8 + r;
    const bool live = c < cols;
    const int tok = live ? token_of(c) : 0, hq = live ? c - tok * g : 0;
    const __half* src = a.q + static_cast<size_t>(sp.row0 + tok) * a.ldq + (head * g + hq) * D + j * DL;
#pragma unroll
    for (int w = 0; w < WL; ++w) {
      uint4 v = *reinterpret_cast<const uint4*>(src + w * 8);
      if (!live) v = make_uint4(0u, 0u, 0u, 0u);
      if (Q4) {  // (e, e + 4)
        qf[nt][w][0] = __byte_perm(v.x, v.z, 0x5410);
        qf[nt][w][1] = __byte_perm(v.x, v.z, 0x7632);
        qf[nt][w][2] = __byte_perm(v.y, v.w, 0x5410);
        qf[nt][w][3] = __byte_perm(v.y, v.w, 0x7632);
      } else {
        qf[nt][w][0] = v.x;
        qf[nt][w][1] = v.y;
        qf[nt][w][2] = v.z;
        qf[nt][w][3] = v.w;
      }
    }
  }

  float o[MT][NT][4];
  float mx[NT][2], off[NT][2], sum[NT][2];  // base of the exponents (raw score), bias - base * scale, sum of weights
  int last[NT][2];  // position of the lane's two rows of each column tile
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[mt][nt][e] = 0.f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      mx[nt][e] = -INFINITY;
      off[nt][e] = 0.f;
      sum[nt][e] = 0.f;
      last[nt][e] = first + min(token_of(nt * 8 + 2 * j + e), sp.n - 1);
    }
  }

  int slot = 0;
  for (int t = rank * warps + warp; t < tiles; t += step) {
    cp_wait<T::stages - 2>();
    __syncwarp();
    {
      int to = slot + T::stages - 1;
      to = to >= T::stages ? to - T::stages : to;
      if (t_load < tiles) load_tile<D, Q4>(a.kv, head, t_load, next_page, smem_u32(ring + to * T::bytes), lane);
      cp_commit();
      t_load += step;
      next_page = t_load < tiles ? page_for(t_load) : -1;
    }
    const uint8_t* st = ring + slot * T::bytes;
    slot = slot + 1 == T::stages ? 0 : slot + 1;
    if (t * T::keys + T::keys > sp.len) clear_tail<D, Q4>(smem_u32(st), t, sp.len, lane);

    // S^T: 16-key tile km holds blocks 2 km (rows r) and 2 km + 1 (rows r + 8)
    float s[KM][NT][4];
#pragma unroll
    for (int km = 0; km < KM; ++km)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) s[km][nt][e] = 0.f;
#pragma unroll
    for (int km = 0; km < KM; ++km) {
      if (Q4) {
        // row r of block x is token 8 (r / 2) + x + 4 (r % 2): the transposed weights then
        // pair up tokens (x, x + 4) of block j, as V's words hold them
        uint4 cw[2];
        __half2 sc[2], mn[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int x = 2 * km + h, y = x + 4 * (r & 1);  // y: token in its block
          const uint8_t* kb = st + (r >> 1) * 8 * T::row;
          const uint32_t ms = lds32(st + 2 * T::side + ((r >> 1) * 8 + y) * (D / 64) * 4 + (D == 128 ? (j >> 1) * 4 : 0));
          mn[h] = dup_half(ms, 0);
          sc[h] = dup_half(ms, 1);
          if (D == 128) {
            cw[h] = lds128(kb + ((y * 4 + j) ^ ((r & 1) * 4)) * 16);
          } else {
            const int u = y * 2 + (j >> 1);
            const uint2 v = lds64(kb + (u ^ ((r & 1) * 2) ^ ((r & 2) * 2)) * 16 + (j & 1) * 8);
            cw[h] = make_uint4(v.x, v.y, 0u, 0u);
          }
        }
#pragma unroll
        for (int w = 0; w < WL; ++w) {
          uint32_t lo[4], hi[4];
          dequant_word(word_of(cw[0], w), sc[0], mn[0], lo);
          dequant_word(word_of(cw[1], w), sc[1], mn[1], hi);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16816(s[km][nt], lo[0], hi[0], lo[1], hi[1], qf[nt][w][0], qf[nt][w][1]);
            mma_16816(s[km][nt], lo[2], hi[2], lo[3], hi[3], qf[nt][w][2], qf[nt][w][3]);
          }
        }
      } else {
#pragma unroll
        for (int w = 0; w < WL; ++w) {
          uint4 kv2[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int u = WL * j + w;
            const uint32_t us = D == 128 ? u ^ ((u >> 3) << 1) ^ (r & 1) : u ^ (r & 1);
            kv2[h] = lds128(st + (16 * km + 8 * h + r) * T::row + us * 16);
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_16816(s[km][nt], kv2[0].x, kv2[1].x, kv2[0].y, kv2[1].y, qf[nt][w][0], qf[nt][w][1]);
            mma_16816(s[km][nt], kv2[0].z, kv2[1].z, kv2[0].w, kv2[1].w, qf[nt][w][2], qf[nt][w][3]);
          }
        }
      }
    }

    // running maximum and weights
    if (t * T::keys + T::keys - 1 > first) {
#pragma unroll
      for (int km = 0; km < KM; ++km)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int x = 2 * km + (e >> 1);
          const int p = t * T::keys + (Q4 ? 8 * (r >> 1) + x + 4 * (r & 1) : 8 * x + r);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            if (p > last[nt][e & 1]) s[km][nt][e] = -INFINITY;
        }
    }
    // The exponent base of a row only moves when a score outgrows it by 2^7, so that O is
    // rarely rescaled (kWeightBias: what the weights are in fp16).
    uint32_t pt[NT][2 * KM];
    float tm[NT][2];
    bool grew = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float m = -INFINITY;
#pragma unroll
        for (int km = 0; km < KM; ++km) m = fmaxf(m, fmaxf(s[km][nt][e], s[km][nt][e + 2]));
        tm[nt][e] = m;
        grew |= m > mx[nt][e] + a.slack;  // (from -inf: any finite score)
      }
    if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float alpha[2];
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float m = tm[nt][e];
#pragma unroll
          for (int x = 4; x < 32; x <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, x));
          m = m > mx[nt][e] + a.slack ? m : mx[nt][e];
          alpha[e] = m == -INFINITY ? 1.f : exp2_approx((mx[nt][e] - m) * a.scale_log2);
          mx[nt][e] = m;
          off[nt][e] = m == -INFINITY ? 0.f : fmaf(-m, a.scale_log2, kWeightBias);  // no key of the row so far: 0
          sum[nt][e] *= alpha[e];
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[mt][nt][e] *= alpha[e & 1];
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int km = 0; km < KM; ++km) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[km][nt][e] = exp2_approx(fmaf(s[km][nt][e], a.scale_log2, off[nt][e & 1]));
        pt[nt][2 * km] = movmatrix_trans(pack_half2(s[km][nt][0], s[km][nt][1]));
        pt[nt][2 * km + 1] = movmatrix_trans(pack_half2(s[km][nt][2], s[km][nt][3]));
      }

#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float l = s[0][nt][e] + s[0][nt][e + 2];
        if (KM == 2) l += s[KM - 1][nt][e] + s[KM - 1][nt][e + 2];
        sum[nt][e] += l;
      }

    // O^T += V^T P^T
    if (Q4) {
      // lane (r, j): block j's words of dimensions 32 q + 4 r + {0..3}; 16-dimension
      // tile 2q + h is dimensions 32q + 4r + 2h (rows r) and + 1 (rows r + 8)
      const uint8_t* vb = st + T::side + j * 8 * T::row;
      const uint8_t* vm = st + 2 * T::side + T::meta + j * 8 * (D / 64) * 4;
#pragma unroll
      for (int gd = 0; gd < D / 64; ++gd) {
        __half2 sc[4], mn[4];
        if (D == 128) {
          // pairs [token][2 groups]: tokens y and y + 4 of group gd
#pragma unroll
          for (int y = 0; y < 4; y += 2) {
            const uint4 lo = lds128(vm + y * 8), hi = lds128(vm + (y + 4) * 8);
            const uint32_t a0 = gd ? lo.y : lo.x, a1 = gd ? lo.w : lo.z;
            const uint32_t b0 = gd ? hi.y : hi.x, b1 = gd ? hi.w : hi.z;
            mn[y] = as_half2(__byte_perm(a0, b0, 0x5410));
            sc[y] = as_half2(__byte_perm(a0, b0, 0x7632));
            mn[y + 1] = as_half2(__byte_perm(a1, b1, 0x5410));
            sc[y + 1] = as_half2(__byte_perm(a1, b1, 0x7632));
          }
        } else {
          const uint4 lo = lds128(vm), hi = lds128(vm + 16);
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            mn[y] = as_half2(__byte_perm(word_of(lo, y), word_of(hi, y), 0x5410));
            sc[y] = as_half2(__byte_perm(word_of(lo, y), word_of(hi, y), 0x7632));
          }
        }
#pragma unroll
        for (int q2 = 0; q2 < 2; ++q2) {
          const int q = 2 * gd + q2;
          const uint4 w = lds128(vb + ((8 * q + r) ^ (2 * j)) * 16);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t lo[4], hi[4];
            dequant_word(word_of(w, 2 * h), sc[0], mn[0], sc[1], mn[1], sc[2], mn[2], sc[3], mn[3], lo);
            dequant_word(word_of(w, 2 * h + 1), sc[0], mn[0], sc[1], mn[1], sc[2], mn[2], sc[3], mn[3], hi);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float(&to)[4] = o[2 * q + h][nt];
              if (Fold) {
                float part[4];
                mma_16816_first(part, lo[0], hi[0], lo[1], hi[1], pt[nt][0], pt[nt][1]);
                mma_16816(part, lo[2], hi[2], lo[3], hi[3], pt[nt][2 * KM - 2], pt[nt][2 * KM - 1]);
#pragma unroll
                for (int e = 0; e < 4; ++e) to[e] += part[e];
              } else {
                mma_16816(to, lo[0], hi[0], lo[1], hi[1], pt[nt][0], pt[nt][1]);
                mma_16816(to, lo[2], hi[2], lo[3], hi[3], pt[nt][2 * KM - 2], pt[nt][2 * KM - 1]);
              }
            }
          }
        }
      }
    } else {
      // matrices (keys 0-7, dimensions 0-7), (keys 0-7, 8-15), (keys 8-15, 0-7), (8-15, 8-15)
      const int y = (lane >> 4) * 8 + (lane & 7);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        uint32_t f[4];
        const int u = 2 * mt + ((lane >> 3) & 1);
        ldmatrix4_trans(smem_u32(st + T::side + y * T::row + ((u ^ (y & 7)) * 16)), f);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (Fold) {
            float part[4];
            mma_16816_first(part, f[0], f[1], f[2], f[3], pt[nt][0], pt[nt][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[mt][nt][e] += part[e];
          } else {
            mma_16816(o[mt][nt], f[0], f[1], f[2], f[3], pt[nt][0], pt[nt][1]);
          }
        }
      }
    }
  }
  cp_wait<0>();
  __syncwarp();
  pdl_trigger();

  // join the warps: O as [column][D] in the warp's own ring
  float* mine = reinterpret_cast<float*>(smem + warp * T::stages * T::bytes);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int c = nt * 8 + 2 * j + e;
      float l = sum[nt][e];
#pragma unroll
      for (int x = 4; x < 32; x <<= 1) l += __shfl_xor_sync(0xffffffffu, l, x);
      if (r == 0) {
        s_m[warp][c] = mx[nt][e];
        s_l[warp][c] = l;
      }
      if (c < cols) {
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          if (Q4) {
            *reinterpret_cast<float2*>(mine + c * D + 32 * (mt >> 1) + 4 * r + 2 * (mt & 1)) =
                make_float2(o[mt][nt][e], o[mt][nt][e + 2]);
          } else {
            mine[c * D + 16 * mt + r] = o[mt][nt][e];
            mine[c * D + 16 * mt + 8 + r] = o[mt][nt][e + 2];
          }
        }
      }
    }
  __syncthreads();
  auto weight = [&](float m, float top) { return m == -INFINITY ? 0.f : exp2_approx((m - top) * a.scale_log2); };
  float* joined = reinterpret_cast<float*>(smem);  // over the first warp's part, element by element
  for (int x = threadIdx.x; x < cols * D; x += warps * 32) {
    const int c = x / D, e = x % D;
    float top = s_m[0][c];
    for (int w = 1; w < warps; ++w) top = fmaxf(top, s_m[w][c]);
    float acc = 0.f, l = 0.f;
    for (int w = 0; w < warps; ++w) {
      const float f = weight(s_m[w][c], top);
      acc += f * reinterpret_cast<const float*>(smem + w * T::stages * T::bytes)[x];
      l += f * s_l[w][c];
    }
    if (splits == 1) {
      a.out[static_cast<size_t>(sp.row0 + token_of(c)) * a.ldo + (head * g + c - token_of(c) * g) * D + e] = __float2half_rn(acc / l);
    } else {
      joined[x] = acc;
      if (e == 0) {
        c_m[c] = top;
        c_l[c] = l;
      }
    }
  }
  if (splits == 1) return;
  __syncwarp();
  cluster.sync();
  for (int x = rank * warps * 32 + threadIdx.x; x < cols * D; x += splits * warps * 32) {
    const int c = x / D, e = x % D;
    float top = -INFINITY, part[kMaxCluster], m[kMaxCluster], l[kMaxCluster];
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k)
      if (k < splits) {
        m[k] = *cluster.map_shared_rank(&c_m[c], k);
        l[k] = *cluster.map_shared_rank(&c_l[c], k);
        part[k] = *cluster.map_shared_rank(joined + x, k);
        top = fmaxf(top, m[k]);
      }
    float acc = 0.f, den = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k)
      if (k < splits) {
        const float f = weight(m[k], top);
        acc += f * part[k];
        den += f * l[k];
      }
    a.out[static_cast<size_t>(sp.row0 + token_of(c)) * a.ldo + (head * g + c - token_of(c) * g) * D + e] = __float2half_rn(acc / den);
  }
  __syncwarp();
  cluster.sync();  // nobody leaves while another reads its shared memory
}

// How a unit's history is dealt out: warps of a CTA and CTAs of a cluster (its tiles go round
// them all).  The plan counts on 16 warps an SM, which is what eight columns of a 4-bit cache, or of fp16 with
// d = 64, have; with sixteen columns 12 warps fit (registers), with fp16 and d = 128 nine (rings), and a launch that
// is meant to be resident at once then takes two rounds.  Very many units: two warps each, so that the fixed cost of a
// unit is shared by few (8064 units of 300 to 1040 keys: 205 us with two, 211 with four, 231 with one).  Few
// units: the largest number of warps that is resident at once, by that count.  Where that leaves a fifth of the SMs'
// room empty and histories are long, four-warp CTAs in at least two and a half rounds, down to
// 512 keys a CTA (320 units of 8000 keys: 118 us in one round of 320 CTAs).
struct Plan {
  int warps, splits;
};
long long tiles_of(int max_len, int tile) { return (static_cast<long long>(max_len) + tile - 1) / tile; }
Plan plan_balanced(long long units, int max_len, int tile, int sms) {
  const long long tiles = tiles_of(max_len, tile);
  if (tiles <= 2) return {static_cast<int>(tiles), 1};  // no warp without a tile
  if (units >= 32ll * sms) return {2, 1};
  Plan best{4, 1};
  long long resident = 0;
  for (const int warps : {4, 8}) {
    if (warps > 4 && tiles < warps) continue;
    const long long room = 16 / warps * sms;  // CTAs at once
    const long long splits = std::min({static_cast<long long>(kMaxCluster), room / units, std::max(1ll, tiles / warps)});
    if (splits >= 1 && units * splits * warps > resident) {
      resident = units * splits * warps;
      best = {warps, static_cast<int>(splits)};
    }
  }
  if (resident >= 13ll * sms) return best;
  const long long rounds = (10ll * sms + units - 1) / units;  // splits for 2.5 rounds of 4 CTAs an SM
  const long long splits = std::min({static_cast<long long>(kMaxCluster), rounds, static_cast<long long>(max_len / 512)});
  return splits > 1 && units * splits >= 5ll * sms ? Plan{4, static_cast<int>(splits)} : best;
}
// The same, but no warp's share of a history longer than 4096 tiles (as far as 64 warps a history
// go): a sum of more roundings could, all in one direction, reach 2^-12.
Plan plan_rows(long long units, int max_len, int tile, int sms) {
  Plan p = plan_balanced(units, max_len, tile, sms);
  const long long tiles = tiles_of(max_len, tile);
  while (p.warps < kMaxWarps && tiles > 4096ll * p.warps * p.splits) p.warps *= 2;
  while (p.splits < kMaxCluster && tiles > 4096ll * p.warps * p.splits) p.splits = std::min(2 * p.splits, kMaxCluster);
  return p;
}

template <int D, bool Q4, int NT, bool Fold>
cudaError_t launch_plan(const PagedAttnArgs& a, const Plan& plan, cudaStream_t s) {
  using T = Tile<D, Q4>;
  static_assert(T::stages * T::bytes >= 8 * NT * D * 4, "a warp's ring holds its partial output");
  cudaError_t e = allow_smem<attn_paged_rows_kernel<D, Q4, NT, Fold>>(kMaxWarps * T::stages * T::bytes);
  if (e != cudaSuccess) return e;
  const int warps = plan.warps, splits = plan.splits;
  const long long units = static_cast<long long>(a.batch.b) * a.kv.kv_heads;
  const int smem = warps * T::stages * T::bytes;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(units * splits));
  cfg.blockDim = dim3(warps * 32);
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
  e = cudaLaunchKernelEx(&cfg, attn_paged_rows_kernel<D, Q4, NT, Fold>, a);
  return e != cudaSuccess ? e : launched();
}

template <int D, bool Q4, int NT>
cudaError_t launch_rows(const PagedAttnArgs& a, cudaStream_t s) {
  const long long units = static_cast<long long>(a.batch.b) * a.kv.kv_heads;
  const Plan plan = plan_rows(units, a.batch.max_len, Tile<D, Q4>::keys, runtime().num_sms);
  const bool plain = tiles_of(a.batch.max_len, Tile<D, Q4>::keys) <= static_cast<long long>(kPlainTiles) * plan.warps * plan.splits;
  return plain ? launch_plan<D, Q4, NT, false>(a, plan, s) : launch_plan<D, Q4, NT, true>(a, plan, s);
}

template <int D, bool Q4>
cudaError_t launch_d(const PagedAttnArgs& a, cudaStream_t s) {
  // columns of the few-row kernel; sequences with more rows take the chunk kernel
  const long long most = static_cast<long long>(a.group) * a.batch.max_new;
  const int cols = most <= 8 || (most > 16 && a.group <= 8) ? 8 : 16;
  if (a.group <= cols) {
    const cudaError_t e = cols == 8 ? launch_rows<D, Q4, 1>(a, s) : launch_rows<D, Q4, 2>(a, s);
    if (e != cudaSuccess || most <= cols) return e;
  }
  return launch_attn_paged_chunks(a.kv, a.batch, a.heads, D, Q4 ? 4 : 16, a.group <= cols ? cols + 1 : 1, a.q, a.ldq, a.out,
                                  a.ldo, s);
}

}  // namespace

cudaError_t launch_attn_paged(const PagedView& kv, const RaggedView& batch, int heads, int d, int kv_bits,
                              const __half* q, int ldq, __half* out, int ldo, cudaStream_t s) {
  const float scale_log2 = 1.4426950408889634f / sqrtf(static_cast<float>(d));
  const int group = heads / kv.kv_heads;
  // ceil(2^16 / group): exact quotients for c < 16, group <= 16 (the error c * group / 2^16 stays below 1 / group)
  const PagedAttnArgs a{kv,  batch, heads,      group,           q,
                        ldq, out,   ldo,        scale_log2,      kWeightSlack / scale_log2,
                        static_cast<uint32_t>((65536 + group - 1) / group), runtime().err};
  if (kv_bits == 4) return d == 128 ? launch_d<128, true>(a, s) : launch_d<64, true>(a, s);
  return d == 128 ? launch_d<128, false>(a, s) : launch_d<64, false>(a, s);
}

}  // namespace flexq
