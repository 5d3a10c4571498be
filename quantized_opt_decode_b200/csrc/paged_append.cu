// Paged KV cache: append (position rotation, quantization and page lookup in
// one pass) and read-back of a ragged batch of tokens.
//
// A warp takes one 8-token block of one sequence and a few neighbouring heads of K,
// of V or (rotation only) of Q.  The 8-token block is the unit in which the 4-bit V codes are
// interleaved, so the warp owns the words it writes: a block that the new tokens
// cover only in part is read, merged and written back without atomics, and slots before
// and behind the new tokens keep their codes.  A lane holds 16 dimensions of one head as
// two 16-byte chunks: the two halves of its rotation pairs, so that no value is loaded
// twice and a token's cosines and sines (64 bytes a lane) serve all the heads of the warp; past the
// rotated dimensions, and in V, 16 neighbouring ones.  A 64-element group is then
// spread over the 8 (d = 128) or 4 lanes of the head: its minimum and maximum are one
// shuffle ladder a group on the pair (min x, -max x) in two fp16 halves.
//
// Memory is the floor of both kernels: rows in, codes and pairs out, and for Q rows in and
// out.  Measured (B200): 8345 rows of 8 key/value and 32 query heads, d = 128, rotated, to 4 bit:
// 43 us for 175 MB, 0.62 of the copy rate: warps wait for their loads (3.8 of them at each issue, a third
// of the warps that an SM could hold, 56 % of the issue slots taken); prefetched rows, or
// more or fewer warps an SM, changed nothing (with a check of each code against the reciprocal's
// error instead of the corrected quotient 46 us); 2055 rows to fp16, d = 64: 12.5 us for
// 51 MB; reading 19085 tokens of 32 heads back: 68.5 us for 401 MB, 0.89 of the copy rate (82 us with a
// lane's two chunks side by side, which its stores then half fill).
//
// The codes are exactly those of flexq_quantize on the (rotated) fp16 rows:
// rotation multiplies and adds in fp32 without contraction and rounds once to
// fp16, then the shared group rule applies.
#include <math.h>

#include "paged.cuh"
#include "quant_common.cuh"

namespace flexq {
namespace {

constexpr int kWarps = 4;
constexpr int kUnitShift = 3;  // units of 8 tokens
constexpr int kUnitExtra = 2;  // n tokens at any phase touch at most floor(n / 8) + 2 blocks

constexpr int kQHeads = 4;  // heads of Q that a lane takes in turn
constexpr int kQParts = 4;  // jobs that share a block's tokens of Q

// Elements of a 16-byte chunk.
__device__ __forceinline__ void unpack(const uint4& raw, float (&x)[8]) {
  const __half2* h = reinterpret_cast<const __half2*>(&raw);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = __half22float2(h[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 pack16(const float (&x)[8]) {
  uint4 raw;
  __half2* h = reinterpret_cast<__half2*>(&raw);
#pragma unroll
  for (int e = 0; e < 4; ++e) h[e] = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
  return raw;
}

// The two chunks of lane p of a head: dimensions ea .. ea + 7 and eb .. eb + 7.  Without
// rotation they lie half a head apart, so that eight lanes' chunks are 128 bytes in a row.
struct Slot {
  int ea, eb;
  bool turned;
};
template <int D>
__device__ __forceinline__ Slot slot_of(int p, int rot, bool interleaved) {
  Slot s;
  if (rot == 0) {
    s.turned = false;
    s.ea = 8 * p;
    s.eb = D / 2 + 8 * p;
    return s;
  }
  s.turned = p < rot / 16;
  s.ea = s.turned && !interleaved ? 8 * p : 16 * p;
  s.eb = s.turned && !interleaved ? rot / 2 + 8 * p : 16 * p + 8;
  return s;
}

// Cosines and sines of the lane's eight pairs at position pos.
struct Turn {
  float c[8], s[8];
};
__device__ __forceinline__ void load_turn(const RopeView& rope, int pos, int p, Turn& t) {
  const float* row = rope.cos_sin + static_cast<size_t>(pos) * rope.rot_dim + 8 * p;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    *reinterpret_cast<float4*>(&t.c[4 * h]) = __ldg(reinterpret_cast<const float4*>(row) + h);
    *reinterpret_cast<float4*>(&t.s[4 * h]) = __ldg(reinterpret_cast<const float4*>(row + rope.rot_dim / 2) + h);
  }
}

// a' = a cos - b sin, b' = b cos + a sin, every operation rounded.
__device__ __forceinline__ void turn_chunks(uint4& ra, uint4& rb, const Turn& t, bool interleaved) {
  float x[8], y[8], u[8], v[8];
  unpack(ra, x);
  unpack(rb, y);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // pair i: (x[i], y[i]), or elements 2i and 2i + 1 of the 16
    const float a = interleaved ? (i < 4 ? x[2 * (i & 3)] : y[2 * (i & 3)]) : x[i];
    const float b = interleaved ? (i < 4 ? x[2 * (i & 3) + 1] : y[2 * (i & 3) + 1]) : y[i];
    u[i] = __fsub_rn(__fmul_rn(a, t.c[i]), __fmul_rn(b, t.s[i]));
    v[i] = __fadd_rn(__fmul_rn(b, t.c[i]), __fmul_rn(a, t.s[i]));
  }
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = u[i];
      x[2 * i + 1] = v[i];
      y[2 * i] = u[4 + i];
      y[2 * i + 1] = v[4 + i];
    }
    ra = pack16(x);
    rb = pack16(y);
  } else {
    ra = pack16(u);
    rb = pack16(v);
  }
}

// (min, -max) of a chunk as two fp16 halves.
__device__ __forceinline__ uint32_t chunk_range(const uint4& raw) {
  const __half2* h = reinterpret_cast<const __half2*>(&raw);
  const __half2 lo = __hmin2(__hmin2(h[0], h[1]), __hmin2(h[2], h[3]));
  const __half2 hi = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
  const __half l = __hmin(__low2half(lo), __high2half(lo)), m = __hmax(__low2half(hi), __high2half(hi));
  return __half_as_ushort(l) | (static_cast<uint32_t>(__half_as_ushort(m) ^ 0x8000u) << 16);
}
__device__ __forceinline__ uint32_t min2(uint32_t x, uint32_t y) {
  const __half2 m = __hmin2(*reinterpret_cast<const __half2*>(&x), *reinterpret_cast<const __half2*>(&y));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// x / 15 correctly rounded: the product with the rounded reciprocal is within an
// ulp, its remainder is exact in one multiply-add, and one more with the reciprocal
// rounds to the quotient (Markstein, 1990).  x: a difference of fp16 values, so
// nothing underflows; the remainder of an infinity is NaN and is left out.
__device__ __forceinline__ float fifteenth(float x) {
  constexpr float y = 1.0f / 15.0f;
  const float q = __fmul_rn(x, y);
  return fabsf(x) == INFINITY ? x : fmaf(fmaf(-15.0f, q, x), y, q);
}

struct Group {
  __half2 pair;  // (min, scale) as stored
  float mn, sc, inv;
};
__device__ __forceinline__ Group group_of(uint32_t range) {
  const float lo = __fadd_rn(__half2float(__ushort_as_half(range & 0xffffu)), 0.0f);  // -0 -> +0
  const float hi = __fadd_rn(__half2float(__ushort_as_half((range >> 16) ^ 0x8000u)), 0.0f);
  const __half s16 = __float2half_rn(fifteenth(__fsub_rn(hi, lo)));
  const __half m16 = __float2half_rn(lo);
  Group g;
  g.pair = __halves2half2(m16, s16);
  g.mn = __half2float(m16);
  g.sc = __half2float(s16);
  g.inv = g.sc != 0.0f ? __frcp_rn(g.sc) : 0.0f;
  return g;
}

// Codes of a chunk, rint(a / s) of a = x - min, as the bits of 1.5 * 2^23 + code (0x4B400000 +
// code): adding that number rounds to the nearest integer, half to even.  The quotient is the
// correctly rounded one without a division, by the correction step of fifteenth(): with y the rounded
// reciprocal, q + (a - q s) y is within 1.5 ulp * 2^-24 of a / s.  A midpoint of two fp32 numbers
// has 25 bits and s has 11, so a / s, unless it is one, is at least 2^-11 of half an ulp away from every
// midpoint; and it never is one, since the product of an odd 25-bit number with s does not fit a's
// 24 bits.  x >= min, so codes are never negative; only a subnormal scale can have been rounded down
// so far that a quotient exceeds 15.5.  NaN (of a value, or of a group with an infinity: 0 * inf) takes
// code 0, as in the codec; left as it is, its bits would carry into the word's other codes.
constexpr uint32_t kCodeBias = 0x4B400000u;
__device__ __forceinline__ void chunk_codes(const uint4& raw, const Group& g, uint32_t (&c)[8]) {
  float x[8];
  unpack(raw, x);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float d = __fsub_rn(x[e], g.mn);
    const float q = __fmul_rn(d, g.inv);
    c[e] = __float_as_uint(__fadd_rn(fmaxf(fmaf(fmaf(-g.sc, q, d), g.inv, q), 0.0f), 12582912.0f));
  }
  if (g.sc < 0x1p-14f) {
#pragma unroll
    for (int e = 0; e < 8; ++e) c[e] = min(c[e], kCodeBias + 15);
  }
}

// Eight such codes as a word, element e in nibble e: the biases add up to a constant.
__device__ __forceinline__ uint32_t pack_codes(const uint32_t (&c)[8]) {
  uint32_t w = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) w += (c[e] << (4 * e));
  constexpr uint32_t bias = kCodeBias * 0x11111111u;
  return w - bias;
}

// The lane's two chunks quantized with their head's groups; every lane of the warp
// calls this.  The lane p < d/64 of a head stores the pair of group p.
template <int D>
__device__ __forceinline__ void quantize(const uint4& ra, const uint4& rb, const Slot& s, int p, bool live, __half2* meta,
                                         uint32_t (&ca)[8], uint32_t (&cb)[8]) {
  uint32_t a = chunk_range(ra), b = chunk_range(rb);
  if (D == 64) {
    a = min2(a, b);
#pragma unroll
    for (int o = 2; o > 0; o >>= 1) a = min2(a, __shfl_xor_sync(0xffffffffu, a, o));
    const Group g = group_of(a);
    if (p == 0 && live) meta[0] = g.pair;
    chunk_codes(ra, g, ca);
    chunk_codes(rb, g, cb);
  } else {
    constexpr uint32_t kNone = 0x7fff7fffu;  // NaN twice, which the minimum passes over
    uint32_t r0 = min2(s.ea < 64 ? a : kNone, s.eb < 64 ? b : kNone);
    uint32_t r1 = min2(s.ea < 64 ? kNone : a, s.eb < 64 ? kNone : b);
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) {
      r0 = min2(r0, __shfl_xor_sync(0xffffffffu, r0, o));
      r1 = min2(r1, __shfl_xor_sync(0xffffffffu, r1, o));
    }
    const Group g0 = group_of(r0), g1 = group_of(r1);
    if (p < 2 && live) meta[p] = p == 0 ? g0.pair : g1.pair;
    chunk_codes(ra, s.ea < 64 ? g0 : g1, ca);
    chunk_codes(rb, s.eb < 64 ? g0 : g1, cb);
  }
}

// A unit's sequence and block: tokens t0 .. t1-1 (positions) of sequence i.
struct Unit {
  int i, t0, t1, row;  // row = token buffer row of position 0 (row of position p is row + p)
};

__device__ __forceinline__ bool find_unit(const RaggedView& batch, int u, Unit& w, uint32_t* err) {
  int blk_rel = 0;
  if (batch.max_new == 1) {  // one block per sequence
    w.i = u;
  } else {
    w.i = find_unit_owner(batch, u, kUnitShift, kUnitExtra);
    if (w.i < 0) return false;
    blk_rel = u - static_cast<int>(unit_base(batch, w.i, kUnitShift, kUnitExtra));
  }
  const Span sp = ragged_span(batch, w.i, err);
  if (sp.n == 0) return false;
  const int p0 = sp.len - sp.n;
  const int blk = (p0 >> 3) + blk_rel;
  w.t0 = max(p0, blk * 8);
  w.t1 = min(sp.len, blk * 8 + 8);
  w.row = sp.row0 - p0;
  return w.t0 < w.t1;
}

long long unit_count(const RaggedView& batch) {
  return batch.max_new == 1 ? batch.b : unit_total(batch.rows, batch.b, 1, kUnitShift, kUnitExtra);
}

struct AppendArgs {
  PagedView kv;
  RaggedView batch;
  RopeView rope;
  int heads;
  const __half *k, *v;
  int ld;
  const __half* q;
  int ldq;
  __half* q_out;
  int ldqo;
  int kv_jobs, jobs;  // of a block: K's (and V's), and all with Q's
  long long total;
  uint32_t* err;
};

// kind of a job: K, V or Q of a block and a warp's heads
enum Kind { kK, kV, kQ };

template <int D, bool Q4>
__global__ void __launch_bounds__(kWarps * 32, 6) paged_append_kernel(const AppendArgs a) {
  constexpr int LH = D / 16;     // lanes of a head
  constexpr int HW = 32 / LH;    // heads of a warp at once
  constexpr int G = D / 64;
  pdl_wait();
  const long long widx = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (widx == 0 && a.batch.max_new > 1) check_spans(a.batch, a.err);
  if (widx >= a.total) return;
  const int lane = static_cast<int>(lane_id());
  Unit un;
  if (!find_unit(a.batch, static_cast<int>(widx / a.jobs), un, a.err)) return;
  int job = static_cast<int>(widx % a.jobs);
  const int kvh = a.kv.kv_heads;
  const Kind kind = job < a.kv_jobs ? kK : job < 2 * a.kv_jobs ? kV : kQ;
  job -= kind * a.kv_jobs;
  const int p = lane % LH;
  const bool turn = a.rope.cos_sin != nullptr && kind != kV;
  const bool inter = a.rope.interleaved != 0;
  if (turn && un.t1 > a.rope.max_pos) {
    if (lane == 0) set_error(a.err, DEV_BAD_ARGUMENT);
    return;
  }
  const Slot sl = slot_of<D>(p, turn ? a.rope.rot_dim : 0, inter);

  if (kind == kQ) {
    const int h0 = job / kQParts * HW * kQHeads + lane / LH;
    const int first = (un.t0 & ~7) + job % kQParts * (8 / kQParts);
    for (int t = max(un.t0, first); t < min(un.t1, first + 8 / kQParts); ++t) {
      const size_t row = static_cast<size_t>(un.row + t);
      uint4 ra[kQHeads], rb[kQHeads];
#pragma unroll
      for (int i = 0; i < kQHeads; ++i) {
        const int h = h0 + i * HW;
        if (h >= a.heads) continue;
        const __half* src = a.q + row * a.ldq + h * D;
        ra[i] = *reinterpret_cast<const uint4*>(src + sl.ea);
        rb[i] = *reinterpret_cast<const uint4*>(src + sl.eb);
      }
      if (sl.turned) {
        Turn tn;
        load_turn(a.rope, t, p, tn);
#pragma unroll
        for (int i = 0; i < kQHeads; ++i) turn_chunks(ra[i], rb[i], tn, inter);
      }
      // (in place: a lane writes the chunks that it alone has read)
#pragma unroll
      for (int i = 0; i < kQHeads; ++i) {
        const int h = h0 + i * HW;
        if (h >= a.heads) continue;
        __half* dst = a.q_out + row * a.ldqo + h * D;
        *reinterpret_cast<uint4*>(dst + sl.ea) = ra[i];
        *reinterpret_cast<uint4*>(dst + sl.eb) = rb[i];
      }
    }
    return;
  }

  const int head = job * HW + lane / LH;
  const bool live = head < kvh;
  const int base = un.t0 & ~7;
  const int page = page_of(a.kv, un.i, base, a.err);
  if (page < 0) return;
  const size_t slot0 = pool_slot(a.kv, page, live ? head : 0, base);
  const __half* src = (kind == kK ? a.k : a.v) + (live ? head : 0) * D;
  // V's words of 16 dimensions; where the new tokens cover the block only in part, the
  // others' codes are merged in at the end (loaded here, so that the rows' loads overlap)
  uint32_t w[16];
  uint4 old[4];
  uint32_t* block = static_cast<uint32_t*>(a.kv.v) + (slot0 >> 3) * D;
  auto word4 = [&](int q) { return reinterpret_cast<uint4*>(block + (q < 2 ? sl.ea + 4 * q : sl.eb + 4 * (q - 2))); };
  const bool merge = Q4 && kind == kV && un.t1 - un.t0 < 8;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    old[q] = make_uint4(0u, 0u, 0u, 0u);
    if (merge) old[q] = *word4(q);
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) w[e] = 0u;
  uint32_t places = 0;  // of the tokens in the words: the codes' biases come off at the end
  constexpr int B = Q4 ? 1 : 2;  // tokens in flight (4-bit: more warps instead, by the registers)
  for (int t = un.t0; t < un.t1; t += B) {
    uint4 ra[B], rb[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const __half* row = src + static_cast<size_t>(un.row + min(t + i, un.t1 - 1)) * a.ld;
      ra[i] = *reinterpret_cast<const uint4*>(row + sl.ea);
      rb[i] = *reinterpret_cast<const uint4*>(row + sl.eb);
    }
    if (sl.turned) {
#pragma unroll
      for (int i = 0; i < B; ++i) {
        Turn tn;
        load_turn(a.rope, min(t + i, un.t1 - 1), p, tn);
        turn_chunks(ra[i], rb[i], tn, inter);
      }
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (t + i >= un.t1) break;
      const size_t slot = slot0 + (t + i - base);
      if (!Q4) {
        __half* dst = static_cast<__half*>(kind == kK ? a.kv.k : a.kv.v) + slot * D;
        if (live) {
          *reinterpret_cast<uint4*>(dst + sl.ea) = ra[i];
          *reinterpret_cast<uint4*>(dst + sl.eb) = rb[i];
        }
        continue;
      }
      uint32_t ca[8], cb[8];
      __half2* meta = static_cast<__half2*>(kind == kK ? a.kv.k_meta : a.kv.v_meta) + slot * G;
      quantize<D>(ra[i], rb[i], sl, p, live, meta, ca, cb);
      if (kind == kK) {
        if (live) {
          uint8_t* dst = static_cast<uint8_t*>(a.kv.k) + slot * (D / 2);
          *reinterpret_cast<uint32_t*>(dst + sl.ea / 2) = pack_codes(ca);
          *reinterpret_cast<uint32_t*>(dst + sl.eb / 2) = pack_codes(cb);
        }
      } else {
        const uint32_t place = 1u << (4 * (t + i - base));
        places += place;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          w[e] += ca[e] * place;
          w[8 + e] += cb[e] * place;
        }
      }
    }
  }
  if (Q4 && kind == kV && live) {
    const uint32_t kept = ~static_cast<uint32_t>(((1ull << (4 * (un.t1 - un.t0))) - 1) << (4 * (un.t0 - base)));
#pragma unroll
    for (int e = 0; e < 16; ++e) w[e] -= places * kCodeBias;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      *word4(q) = make_uint4(w[4 * q] | (old[q].x & kept), w[4 * q + 1] | (old[q].y & kept),
                             w[4 * q + 2] | (old[q].z & kept), w[4 * q + 3] | (old[q].w & kept));
  }
}

struct ReadArgs {
  PagedView kv;
  RaggedView batch;
  __half *k_out, *v_out;
  int ld;
  int kv_jobs;
  long long total;
  uint32_t* err;
};

// Eight codes of a word (element e in nibble e) as the codec's fp16 values: the
// product with the scale is exact in fp32, so one multiply-add rounds as the codec's two
// operations do.  c[e]: 0x4B000000 + code, the fp32 value 2^23 + code.
__device__ __forceinline__ uint4 dequant_chunk(const uint32_t (&c)[8], float2 ms) {
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = fmaf(__uint_as_float(c[e]) - 8388608.0f, ms.y, ms.x);
  return pack16(x);
}
// Byte i of a word of single codes, as such a value.
__device__ __forceinline__ uint32_t byte_value(uint32_t codes, int i) {
  return __byte_perm(codes, 0x4B000000u, 0x7440 | i);
}
constexpr uint32_t kLow = 0x0F0F0F0Fu;

template <int D, bool Q4>
__global__ void __launch_bounds__(kWarps * 32) paged_read_kernel(const ReadArgs a) {
  constexpr int LH = D / 16, HW = 32 / LH, G = D / 64;
  pdl_wait();
  const long long widx = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (widx == 0 && a.batch.max_new > 1) check_spans(a.batch, a.err);
  if (widx >= a.total) return;
  const int lane = static_cast<int>(lane_id());
  const int jobs = 2 * a.kv_jobs;
  Unit un;
  if (!find_unit(a.batch, static_cast<int>(widx / jobs), un, a.err)) return;
  int job = static_cast<int>(widx % jobs);
  const bool is_k = job < a.kv_jobs;
  if (!is_k) job -= a.kv_jobs;
  const int p = lane % LH, head = job * HW + lane / LH;
  const int base = un.t0 & ~7;
  const int page = page_of(a.kv, un.i, base, a.err);
  if (page < 0 || head >= a.kv.kv_heads) return;
  const size_t slot0 = pool_slot(a.kv, page, head, base);
  const int first = un.t0 - base, last = un.t1 - base;
  // the lane's two chunks lie half a head apart: eight lanes store 128 bytes in a row, and with
  // d = 128 the second chunk is in the second group
  __half* dst = (is_k ? a.k_out : a.v_out) + static_cast<long long>(un.row + base) * a.ld + head * D + 8 * p;
  uint4 w[4];     // V: the block's words of 16 dimensions
  uint2 code[8];  // K: 16 codes of each token
  uint2 ms[8];    // (min, scale) of the two chunks
  if (Q4) {
    const char* meta = static_cast<const char*>(is_k ? a.kv.k_meta : a.kv.v_meta) + slot0 * G * 4;
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (t >= first && t < last) {
        if (G == 2) {
          ms[t] = __ldcg(reinterpret_cast<const uint2*>(meta + t * 8));
        } else {
          ms[t].x = __ldcg(reinterpret_cast<const unsigned int*>(meta + t * 4));
          ms[t].y = ms[t].x;
        }
      }
    if (is_k) {
      const char* src = static_cast<const char*>(a.kv.k) + slot0 * (D / 2) + 4 * p;
#pragma unroll
      for (int t = 0; t < 8; ++t)
        if (t >= first && t < last) {
          code[t].x = __ldcg(reinterpret_cast<const unsigned int*>(src + t * (D / 2)));
          code[t].y = __ldcg(reinterpret_cast<const unsigned int*>(src + t * (D / 2) + D / 4));
        }
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint32_t*>(a.kv.v) + (slot0 >> 3) * D + 8 * p);
#pragma unroll
      for (int q = 0; q < 4; ++q) w[q] = __ldcg(src + (q < 2 ? q : D / 8 + q - 2));
    }
  }
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    if (t < first || t >= last) continue;
    uint4 lo, hi;
    if (Q4) {
      uint32_t ca[8], cb[8];
      if (is_k) {
        const uint32_t a0 = code[t].x & kLow, a1 = (code[t].x >> 4) & kLow;
        const uint32_t b0 = code[t].y & kLow, b1 = (code[t].y >> 4) & kLow;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ca[e] = byte_value(e & 1 ? a1 : a0, e / 2);
          cb[e] = byte_value(e & 1 ? b1 : b0, e / 2);
        }
      } else {
        const uint32_t* words = reinterpret_cast<const uint32_t*>(w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ca[e] = ((words[e] >> (4 * t)) & 0xFu) | 0x4B000000u;
          cb[e] = ((words[8 + e] >> (4 * t)) & 0xFu) | 0x4B000000u;
        }
      }
      lo = dequant_chunk(ca, __half22float2(*reinterpret_cast<const __half2*>(&ms[t].x)));
      hi = dequant_chunk(cb, __half22float2(*reinterpret_cast<const __half2*>(&ms[t].y)));
    } else {
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const __half*>(is_k ? a.kv.k : a.kv.v) +
                                                        (slot0 + t) * D + 8 * p);
      lo = __ldcg(src);
      hi = __ldcg(src + D / 16);
    }
    uint4* to = reinterpret_cast<uint4*>(dst + static_cast<size_t>(t) * a.ld);
    to[0] = lo;
    to[D / 16] = hi;
  }
}

// Jobs of a block's K (and of its V): a warp's heads each.
int kv_jobs_of(int kv_heads, int d) { return (kv_heads * (d / 16) + 31) / 32; }

unsigned ctas(long long warps) { return static_cast<unsigned>((warps + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_paged_append(const PagedView& kv, const RaggedView& batch, const RopeView& rope, int heads, int d,
                                int kv_bits, const __half* k, const __half* v, int ld, const __half* q, int ldq,
                                __half* q_out, int ldqo, cudaStream_t s) {
  AppendArgs a{kv, batch, rope, heads, k, v, ld, q, ldq, q_out, ldqo, kv_jobs_of(kv.kv_heads, d), 0, 0, runtime().err};
  const int q_heads = 32 / (d / 16) * kQHeads;
  a.jobs = 2 * a.kv_jobs + (q != nullptr ? (heads + q_heads - 1) / q_heads * kQParts : 0);
  a.total = unit_count(batch) * a.jobs;
  const dim3 grid(ctas(a.total));
  if (kv_bits == 4)
    return d == 128 ? launch_pdl(paged_append_kernel<128, true>, grid, kWarps * 32, 0, s, a)
                    : launch_pdl(paged_append_kernel<64, true>, grid, kWarps * 32, 0, s, a);
  return d == 128 ? launch_pdl(paged_append_kernel<128, false>, grid, kWarps * 32, 0, s, a)
                  : launch_pdl(paged_append_kernel<64, false>, grid, kWarps * 32, 0, s, a);
}

cudaError_t launch_paged_read(const PagedView& kv, const RaggedView& batch, int d, int kv_bits, __half* k_out,
                              __half* v_out, int ld, cudaStream_t s) {
  ReadArgs a{kv, batch, k_out, v_out, ld, kv_jobs_of(kv.kv_heads, d), 0, runtime().err};
  a.total = unit_count(batch) * 2 * a.kv_jobs;
  const dim3 grid(ctas(a.total));
  if (kv_bits == 4)
    return d == 128 ? launch_pdl(paged_read_kernel<128, true>, grid, kWarps * 32, 0, s, a)
                    : launch_pdl(paged_read_kernel<64, true>, grid, kWarps * 32, 0, s, a);
  return d == 128 ? launch_pdl(paged_read_kernel<128, false>, grid, kWarps * 32, 0, s, a)
                  : launch_pdl(paged_read_kernel<64, false>, grid, kWarps * 32, 0, s, a);
}

}  // namespace flexq
