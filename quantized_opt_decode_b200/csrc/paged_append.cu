// Paged KV cache: append (position rotation, quantization and page lookup in
// one pass) and read-back of a ragged batch of tokens.
//
// One warp takes one 8-token block of one sequence and one head of K, of V or
// (rotation only) of Q.  The 8-token block is the unit in which the 4-bit V
// codes are interleaved, so the warp owns the words it writes: a block that the
// new tokens cover only in part is read, merged and written back without atomics,
// and slots before and behind the new tokens keep their codes.  A lane holds d/32
// neighbouring dimensions of up to 8 tokens, so a 64-element group is 16 (d =
// 128) or 32 (d = 64) lanes and its min and max are one shuffle ladder on the pair
// (min x, -max x) in two fp16 halves.
//
// The codes are exactly those of flexq_quantize on the (rotated) fp16 rows:
// rotation multiplies and adds in fp32 without contraction and rounds once to
// fp16, then the shared group rule applies.
#include "paged.cuh"
#include "quant_common.cuh"

namespace flexq {
namespace {

constexpr int kWarps = 8;
constexpr int kUnitShift = 3;  // units of 8 tokens
constexpr int kUnitExtra = 2;  // n tokens at any phase touch at most floor(n / 8) + 2 blocks

template <int VEC>
struct Vec;
template <>
struct Vec<4> {
  using T = uint2;
};
template <>
struct Vec<2> {
  using T = uint32_t;
};

template <int VEC>
__device__ __forceinline__ void unpack(const typename Vec<VEC>::T& raw, float (&x)[VEC]) {
  const __half2* h = reinterpret_cast<const __half2*>(&raw);
#pragma unroll
  for (int e = 0; e < VEC / 2; ++e) {
    const float2 f = __half22float2(h[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}

template <int VEC>
__device__ __forceinline__ typename Vec<VEC>::T pack16(const float (&x)[VEC]) {
  typename Vec<VEC>::T raw;
  __half2* h = reinterpret_cast<__half2*>(&raw);
#pragma unroll
  for (int e = 0; e < VEC / 2; ++e) h[e] = __floats2half2_rn(x[2 * e], x[2 * e + 1]);
  return raw;
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
    w.i = find_unit_owner(batch, u, 1, kUnitShift, kUnitExtra);
    if (w.i < 0) return false;
    blk_rel = u - static_cast<int>(unit_base(batch, w.i, 1, kUnitShift, kUnitExtra));
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
  int jobs;  // K heads, V heads, Q heads of a unit
  long long total;
  uint32_t* err;
};

template <int D, bool Q4>
__global__ void __launch_bounds__(kWarps * 32) paged_append_kernel(const AppendArgs a) {
  constexpr int VEC = D / 32;
  using V = typename Vec<VEC>::T;
  pdl_wait();
  const long long widx = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (widx >= a.total) return;
  const int lane = static_cast<int>(lane_id());
  Unit un;
  if (!find_unit(a.batch, static_cast<int>(widx / a.jobs), un, a.err)) return;
  const int job = static_cast<int>(widx % a.jobs);
  const int kvh = a.kv.kv_heads;
  const bool is_k = job < kvh, is_v = !is_k && job < 2 * kvh, is_q = !is_k && !is_v;
  const int head = is_k ? job : (is_v ? job - kvh : job - 2 * kvh);
  const __half* src = is_k ? a.k : (is_v ? a.v : a.q);
  const int lds = is_q ? a.ldq : a.ld;
  const int e0 = lane * VEC;
  const int base = un.t0 & ~7;

  // the lane's dimensions of the block's tokens, all loads in flight at once
  V raw[8];
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const int p = base + t;
    raw[t] = V{};
    if (p >= un.t0 && p < un.t1)
      raw[t] = *reinterpret_cast<const V*>(src + static_cast<size_t>(un.row + p) * lds + head * D + e0);
  }
  if (a.rope.cos_sin != nullptr && !is_v) {
    if (un.t1 > a.rope.max_pos) {
      if (lane == 0) set_error(a.err, DEV_BAD_ARGUMENT);
      return;
    }
    const int rot = a.rope.rot_dim, half_rot = rot / 2;
    const bool turned = e0 < rot;
    const bool upper = !a.rope.interleaved && e0 >= half_rot;  // the lane holds the pairs' second elements
    if (turned) {
      V other[8];
      if (!a.rope.interleaved) {
        const int eo = upper ? e0 - half_rot : e0 + half_rot;
#pragma unroll
        for (int t = 0; t < 8; ++t) {
          const int p = base + t;
          other[t] = V{};
          if (p >= un.t0 && p < un.t1)
            other[t] = *reinterpret_cast<const V*>(src + static_cast<size_t>(un.row + p) * lds + head * D + eo);
        }
      }
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const int p = base + t;
        if (p < un.t0 || p >= un.t1) continue;
        const float* cs = a.rope.cos_sin + static_cast<size_t>(p) * rot;
        float x[VEC], y[VEC];
        unpack<VEC>(raw[t], x);
        if (a.rope.interleaved) {
#pragma unroll
          for (int e = 0; e < VEC; e += 2) {
            const float c = cs[(e0 + e) / 2], s = cs[half_rot + (e0 + e) / 2];
            y[e] = __fsub_rn(__fmul_rn(x[e], c), __fmul_rn(x[e + 1], s));
            y[e + 1] = __fadd_rn(__fmul_rn(x[e + 1], c), __fmul_rn(x[e], s));
          }
        } else {
          float z[VEC];
          unpack<VEC>(other[t], z);
          const int a0 = upper ? e0 - half_rot : e0;
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float c = cs[a0 + e], s = cs[half_rot + a0 + e];
            const float xs = __fmul_rn(z[e], s);
            y[e] = upper ? __fadd_rn(__fmul_rn(x[e], c), xs) : __fsub_rn(__fmul_rn(x[e], c), xs);
          }
        }
        raw[t] = pack16<VEC>(y);
      }
    }
    __syncwarp();  // in place: every lane has read its pairs before any lane writes
  }
  if (is_q) {
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int p = base + t;
      if (p >= un.t0 && p < un.t1)
        *reinterpret_cast<V*>(a.q_out + static_cast<size_t>(un.row + p) * a.ldqo + head * D + e0) = raw[t];
    }
    return;
  }
  const int page = page_of(a.kv, un.i, base, a.err);
  if (page < 0) return;
  const size_t slot0 = pool_slot(a.kv, page, head, base);
  if (!Q4) {
    __half* dst = static_cast<__half*>(is_k ? a.kv.k : a.kv.v);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int p = base + t;
      if (p >= un.t0 && p < un.t1) *reinterpret_cast<V*>(dst + (slot0 + t) * D + e0) = raw[t];
    }
    return;
  }
  constexpr int G = D / 64;
  constexpr int kGroupLanes = 64 / VEC;
  uint32_t* words = static_cast<uint32_t*>(a.kv.v) + (slot0 >> 3) * D + e0;
  const bool whole = un.t1 - un.t0 == 8;
  uint32_t w[VEC];
#pragma unroll
  for (int e = 0; e < VEC; ++e) w[e] = 0u;
  if (is_v && !whole) {
    uint32_t kept = 0xffffffffu;
#pragma unroll
    for (int t = 0; t < 8; ++t)
      if (base + t >= un.t0 && base + t < un.t1) kept &= ~(0xFu << (4 * t));
#pragma unroll
    for (int e = 0; e < VEC; ++e) w[e] = words[e] & kept;
  }
  __half2* meta = static_cast<__half2*>(is_k ? a.kv.k_meta : a.kv.v_meta);
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const int p = base + t;
    if (p < un.t0 || p >= un.t1) continue;
    float x[VEC];
    unpack<VEC>(raw[t], x);
    const __half2* h = reinterpret_cast<const __half2*>(&raw[t]);
    // (min x, -max x) of the lane's values, then of the group
    __half2 lo2 = h[0], hi2 = h[0];
    if (VEC == 4) {
      lo2 = __hmin2(lo2, h[VEC / 2 - 1]);
      hi2 = __hmax2(hi2, h[VEC / 2 - 1]);
    }
    const __half lo1 = __hmin(__low2half(lo2), __high2half(lo2)), hi1 = __hmax(__low2half(hi2), __high2half(hi2));
    uint32_t mm = __half_as_ushort(lo1) | (static_cast<uint32_t>(__half_as_ushort(hi1) ^ 0x8000u) << 16);
#pragma unroll
    for (int o = kGroupLanes / 2; o > 0; o >>= 1) {
      const uint32_t r = __shfl_xor_sync(0xffffffffu, mm, o);
      const __half2 m2 = __hmin2(*reinterpret_cast<const __half2*>(&mm), *reinterpret_cast<const __half2*>(&r));
      mm = *reinterpret_cast<const uint32_t*>(&m2);
    }
    const float lo = __fadd_rn(__half2float(__ushort_as_half(mm & 0xffffu)), 0.0f);  // -0 -> +0
    const float hi = __fadd_rn(__half2float(__ushort_as_half((mm >> 16) ^ 0x8000u)), 0.0f);
    const __half s16 = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const __half m16 = __float2half_rn(lo);
    const float sc = __half2float(s16), mn = __half2float(m16);
    const float inv = sc != 0.0f ? __frcp_rn(sc) : 0.0f;
    uint32_t c[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) c[e] = sc != 0.0f ? q64_code(__fsub_rn(x[e], mn), sc, inv) : 0u;
    if (lane % kGroupLanes == 0) meta[(slot0 + t) * G + lane / kGroupLanes] = __halves2half2(m16, s16);
    if (is_k) {
      uint8_t* dst = static_cast<uint8_t*>(a.kv.k) + (slot0 + t) * (D / 2) + e0 / 2;
      if (VEC == 4)
        *reinterpret_cast<uint16_t*>(dst) =
            static_cast<uint16_t>(c[0] | (c[1] << 4) | (c[VEC - 2] << 8) | (c[VEC - 1] << 12));
      else
        *dst = static_cast<uint8_t>(c[0] | (c[1] << 4));
    } else {
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] |= c[e] << (4 * t);
    }
  }
  if (is_v) {
    if (VEC == 4)
      *reinterpret_cast<uint4*>(words) = make_uint4(w[0], w[1], w[VEC - 2], w[VEC - 1]);
    else
      *reinterpret_cast<uint2*>(words) = make_uint2(w[0], w[1]);
  }
}

struct ReadArgs {
  PagedView kv;
  RaggedView batch;
  __half *k_out, *v_out;
  int ld;
  long long total;
  uint32_t* err;
};

template <int D, bool Q4>
__global__ void __launch_bounds__(kWarps * 32) paged_read_kernel(const ReadArgs a) {
  constexpr int VEC = D / 32;
  using V = typename Vec<VEC>::T;
  pdl_wait();
  const long long widx = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  if (widx >= a.total) return;
  const int lane = static_cast<int>(lane_id());
  const int kvh = a.kv.kv_heads;
  Unit un;
  if (!find_unit(a.batch, static_cast<int>(widx / (2 * kvh)), un, a.err)) return;
  const int job = static_cast<int>(widx % (2 * kvh));
  const bool is_k = job < kvh;
  const int head = is_k ? job : job - kvh;
  const int e0 = lane * VEC;
  const int base = un.t0 & ~7;
  const int page = page_of(a.kv, un.i, base, a.err);
  if (page < 0) return;
  const size_t slot0 = pool_slot(a.kv, page, head, base);
  V val[8];
  if (!Q4) {
    const __half* src = static_cast<const __half*>(is_k ? a.kv.k : a.kv.v);
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int p = base + t;
      val[t] = V{};
      if (p >= un.t0 && p < un.t1) val[t] = *reinterpret_cast<const V*>(src + (slot0 + t) * D + e0);
    }
  } else {
    constexpr int G = D / 64;
    const __half2* meta = static_cast<const __half2*>(is_k ? a.kv.k_meta : a.kv.v_meta) + slot0 * G + e0 / 64;
    uint32_t code[8];  // K: token t's VEC codes
    uint32_t w[VEC];   // V: 8 tokens' codes per dimension
    __half2 ms[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int p = base + t;
      ms[t] = __half2{};
      code[t] = 0u;
      if (p < un.t0 || p >= un.t1) continue;
      ms[t] = meta[t * G];
      if (is_k) {
        const uint8_t* src = static_cast<const uint8_t*>(a.kv.k) + (slot0 + t) * (D / 2) + e0 / 2;
        code[t] = VEC == 4 ? *reinterpret_cast<const uint16_t*>(src) : *src;
      }
    }
    if (!is_k) {
      const uint32_t* src = static_cast<const uint32_t*>(a.kv.v) + (slot0 >> 3) * D + e0;
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] = src[e];
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const float2 m = __half22float2(ms[t]);  // (min, scale)
      float x[VEC];
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        const uint32_t c = (is_k ? code[t] >> (4 * e) : w[e] >> (4 * t)) & 0xFu;
        x[e] = __fadd_rn(__fmul_rn(static_cast<float>(c), m.y), m.x);
      }
      val[t] = pack16<VEC>(x);
    }
  }
  __half* dst = is_k ? a.k_out : a.v_out;
#pragma unroll
  for (int t = 0; t < 8; ++t) {
    const int p = base + t;
    if (p >= un.t0 && p < un.t1)
      *reinterpret_cast<V*>(dst + static_cast<size_t>(un.row + p) * a.ld + head * D + e0) = val[t];
  }
}

unsigned ctas(long long warps) { return static_cast<unsigned>((warps + kWarps - 1) / kWarps); }

}  // namespace

cudaError_t launch_paged_append(const PagedView& kv, const RaggedView& batch, const RopeView& rope, int heads, int d,
                                int kv_bits, const __half* k, const __half* v, int ld, const __half* q, int ldq,
                                __half* q_out, int ldqo, cudaStream_t s) {
  AppendArgs a{kv, batch, rope, heads, k, v, ld, q, ldq, q_out, ldqo, 0, 0, runtime().err};
  a.jobs = 2 * kv.kv_heads + (q != nullptr ? heads : 0);
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
  ReadArgs a{kv, batch, k_out, v_out, ld, 0, runtime().err};
  a.total = unit_count(batch) * 2 * kv.kv_heads;
  const dim3 grid(ctas(a.total));
  if (kv_bits == 4)
    return d == 128 ? launch_pdl(paged_read_kernel<128, true>, grid, kWarps * 32, 0, s, a)
                    : launch_pdl(paged_read_kernel<64, true>, grid, kWarps * 32, 0, s, a);
  return d == 128 ? launch_pdl(paged_read_kernel<128, false>, grid, kWarps * 32, 0, s, a)
                  : launch_pdl(paged_read_kernel<64, false>, grid, kWarps * 32, 0, s, a);
}

}  // namespace flexq
