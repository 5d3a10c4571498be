// Warp-level building blocks of the kernels that stream 4-bit or fp16 data
// through per-warp shared-memory rings into mma.sync: asynchronous 16-byte copies,
// the m16n8k16 product, fragment loads, and the codec's dequantizer on the
// bit positions in which the codes are stored.
#pragma once

#include <atomic>

#include "common.cuh"
#include "kernels_serving.h"

namespace flexq {

// 16 bytes global -> shared (L2 only); zeros when !valid (src is not read).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Reads through pointers into the kernel's shared array: the compiler may move them between
// products, which inline assembly in program order would not let it.
__device__ __forceinline__ uint4 lds128(const uint8_t* p) { return *reinterpret_cast<const uint4*>(p); }
__device__ __forceinline__ uint2 lds64(const uint8_t* p) { return *reinterpret_cast<const uint2*>(p); }
__device__ __forceinline__ uint32_t lds32(const uint8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }

// Four transposed 8x8 fp16 matrices; lane l names row l % 8 of matrix l / 8.
__device__ __forceinline__ void ldmatrix4_trans(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}

// Transpose of one 8x8 fp16 matrix held as a fragment (row lane/4, columns 2(lane%4)..).
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// D[16][8] += A[16][16] B[16][8], fp16 in, fp32 accumulate.  Lane (r = lane/4,
// j = lane%4): a0 rows r, a1 rows r + 8 of k = 2j, 2j+1; a2, a3 the same of k + 8;
// b0, b1 column r of the same k; c0, c1 row r, columns 2j, 2j+1; c2, c3 row r + 8.
__device__ __forceinline__ void mma_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                          uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// D = A B: the same product from zero.
__device__ __forceinline__ void mma_16816_first(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%10, %10, %10, %10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The softmax's weights enter the product with V in fp16 as 2^(x + bias), x the base-2 exponent
// above the row's running base, which is moved once a score outgrows it by `slack`.  They then
// stay at or below 2^14 (2^15 and a little for scores of 2^22, whose exponents are off by up to 1); from
// 2^-14 on the rounding is 2^-11 relative, and below, a multiple of 2^-24 is at most 2^-32 of the base's
// unit off.  The largest weight of a row is at least half that unit (the base is a maximum, or its exponent
// rounded up).  Without the bias all the weights below 2^-25 of the base were lost to the product but
// not to the sum: 0.3 % of a flat history of 131072 keys behind one that outweighs each of them by 2^25.
constexpr float kWeightBias = 7.f, kWeightSlack = 7.f;

// The low (0) or high (1) half of a pair, twice.
__device__ __forceinline__ __half2 dup_half(uint32_t x, int which) {
  const uint32_t y = __byte_perm(x, x, which ? 0x3232 : 0x1010);
  return *reinterpret_cast<const __half2*>(&y);
}

// The eight codes of a word as four fp16 pairs (code i, code i + 4), i = 0..3,
// dequantized: code * scale + min rounded once to fp16 (the codec rounds the
// product, exact in fp32, plus min to fp32 and then to fp16: the same value
// except where the first rounding lands on the second's tie).  (w & 15) | 0x6400 is the fp16
// value 1024 + code, and a code four bits higher reads 1024 + 16 code: one
// multiply-add by 1/16 brings it down exactly.
__device__ __forceinline__ void dequant_word(uint32_t w, __half2 s0, __half2 m0, __half2 s1, __half2 m1, __half2 s2,
                                             __half2 m2, __half2 s3, __half2 m3, uint32_t (&out)[4]) {
  const __half2 k1024 = __half2half2(__ushort_as_half(0x6400));
  const __half2 k16th = __half2half2(__ushort_as_half(0x2C00));  // 1/16
  const __half2 km64 = __half2half2(__ushort_as_half(0xD400));   // -64
  auto magic = [](uint32_t x, uint32_t mask) {
    uint32_t y;
    asm("lop3.b32 %0, %1, %2, 0x64006400, 0xEA;" : "=r"(y) : "r"(x), "r"(mask));  // (x & mask) | 0x64006400
    return *reinterpret_cast<__half2*>(&y);
  };
  const uint32_t v = w >> 8;
  const __half2 c0 = __hsub2(magic(w, 0x000F000Fu), k1024);
  const __half2 c1 = __hfma2(magic(w, 0x00F000F0u), k16th, km64);
  const __half2 c2 = __hsub2(magic(v, 0x000F000Fu), k1024);
  const __half2 c3 = __hfma2(magic(v, 0x00F000F0u), k16th, km64);
  const __half2 x0 = __hfma2(c0, s0, m0), x1 = __hfma2(c1, s1, m1);
  const __half2 x2 = __hfma2(c2, s2, m2), x3 = __hfma2(c3, s3, m3);
  out[0] = *reinterpret_cast<const uint32_t*>(&x0);
  out[1] = *reinterpret_cast<const uint32_t*>(&x1);
  out[2] = *reinterpret_cast<const uint32_t*>(&x2);
  out[3] = *reinterpret_cast<const uint32_t*>(&x3);
}

// One scale and min for the whole word.
__device__ __forceinline__ void dequant_word(uint32_t w, __half2 s, __half2 m, uint32_t (&out)[4]) {
  dequant_word(w, s, m, s, m, s, m, s, m, out);
}

// mbar_wait without a call: registers stay where they are, and roles that
// differ in their register counts can share it.
__device__ __forceinline__ bool wait_phase(uint64_t* b, uint32_t parity, uint64_t limit_ns) {
  if (mbar_test(b, parity)) return true;
  if (limit_ns < 1000) return false;  // (a test's limit: the first probe decides)
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_try_wait(b, parity))
    if (globaltimer_ns() - t0 > limit_ns) return false;
  return true;
}

// Opts a kernel in to `bytes` of dynamic shared memory, once per device
// (host side; the attribute belongs to the device's context).
template <auto kKernel>
cudaError_t allow_smem(int bytes) {
  static std::atomic<int> allowed[64];
  int dev = 0;
  const cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 64 && allowed[dev].load(std::memory_order_relaxed) >= bytes) return cudaSuccess;
  const cudaError_t s = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (s == cudaSuccess && dev < 64) allowed[dev].store(bytes, std::memory_order_relaxed);
  return s;
}

}  // namespace flexq
