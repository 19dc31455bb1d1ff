// Building blocks of the tensor-core kernels of linear attention with a decay
// for each head (decay_tc.cu, decay_pipe.cu): chunks of 64 tokens, head_dim 128.
#pragma once

#include <cuda.h>

#include "decay_common.cuh"
#include "tc_common.cuh"

namespace gdn {

constexpr int kTc = 64;  // tokens per chunk
constexpr int kTd = 128;

// Descriptor of a tile [k][mn] of 16-bit elements read with k as the
// contraction (MN-major, 128-byte swizzle): boxes of 64 mn columns 8 KB apart,
// eight k rows in 1024 bytes, so that 16 of k advance it by 2048.
__device__ __forceinline__ uint64_t sdesc_mn128(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= (uint64_t)((smem_addr & 0x3FFFF) >> 4);
  d |= (uint64_t)(8192 >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}
constexpr uint32_t kTransA = 1u << 15, kTransB = 1u << 16;

// 16 lanes x 32 columns: thread lane holds rows lane/4 and lane/4 + 8,
// columns 8 c + 2 (lane % 4) and the next, at v[4 c], v[4 c + 1] and
// v[4 c + 2], v[4 c + 3]
__device__ __forceinline__ void tmem_ld_16x32(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x4.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}

// Four 8 x 8 blocks of 16-bit elements between shared memory and registers,
// transposed: lane l gives the address of row l % 8 of block l / 8, and its
// register m holds elements (2 (l % 4), l / 4) and (2 (l % 4) + 1, l / 4) of
// block m as (shared row, shared column).
__device__ __forceinline__ void ldmatrix_t4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stmatrix_t4(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3])
               : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// two floats to packed bf16 (x in the low half)
__device__ __forceinline__ uint32_t pack2(float2 a) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(a.y), "f"(a.x));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint32_t r) {
  return make_float2(__uint_as_float(r << 16), __uint_as_float(r & 0xffff0000u));
}
// the same, leaving in a what the rounding dropped
__device__ __forceinline__ uint32_t split2(float2& a) {
  const uint32_t r = pack2(a);
  a = fma2(unpack2(r), make_float2(-1.f, -1.f), a);
  return r;
}
// the same with the hi part cut off instead of rounded: no conversion, and
// what is left is exact too
__device__ __forceinline__ uint32_t cut2(float2& a) {
  const uint32_t x = __float_as_uint(a.x), y = __float_as_uint(a.y);
  a = fma2(make_float2(__uint_as_float(x & 0xffff0000u), __uint_as_float(y & 0xffff0000u)), make_float2(-1.f, -1.f), a);
  return __byte_perm(x, y, 0x7632);
}
__device__ __forceinline__ float2 mul2(float2 a, float b) { return fma2(a, make_float2(b, b), make_float2(-0.f, -0.f)); }

// a + b as two floats
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two add2(Two a, Two b) {
  const float s = a.hi + b.hi;
  const float t = s - a.hi;
  const float e = (a.hi - (s - t)) + (b.hi - t);
  const float l = e + (a.lo + b.lo);
  const float h = s + l;
  return Two{h, l - (h - s)};
}
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr float kLog2eLo = 1.9259629911e-8f;  // log2(e) less its fp32 rounding
__device__ __forceinline__ Two to_log2(float g) {
  const float h = g * kLog2e;
  return Two{h, fmaf(g, kLog2e, -h) + g * kLog2eLo};
}

}  // namespace gdn
