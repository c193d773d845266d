// Warp-level helpers of the decode-block kernels: m16n8k16 products, matrix loads from shared
// memory, asynchronous 16-byte copies and warp sums.
//
// The products here have few columns (up to 64 tokens of a decode step, up to 16 query heads that share
// a key head) against a stream of weights or keys that is read once, so memory or the conversions bound
// them up to some 16 columns; the warp-level product takes its operands from registers, where the
// conversions leave them, with no trip through tensor memory.
#pragma once

#include <cstdint>

#include "ftmoe_device.cuh"

namespace ftmoe {

// D += A B, m16n8k16. A (row-major): a0 (row l/4, k 2(l%4)..+1), a1 (row + 8), a2 (k + 8),
// a3 (row + 8, k + 8); B: b0 (k 2(l%4)..+1, column l/4), b1 (k + 8); D: d0, d1 (row l/4, columns
// 2(l%4)..+1), d2, d3 (row + 8).
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Four 8 x 8 matrices of 16-bit elements; lane l gives the address of row l % 8 of matrix l / 8.
// Register i: row l/4 of matrix i, elements 2(l%4)..+1; transposed: rows 2(l%4)..+1, element l/4.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

// 16 bytes from global to shared memory, past L1; zeros (and no access) when !valid.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(valid ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {   // all but the newest N groups are complete
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
  return v;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
// (lo, hi) rounded to the nearest bf16 / f16, packed.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ float f16_lo(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)w)); }
__device__ __forceinline__ float f16_hi(uint32_t w) { return f16_lo(w >> 16); }

__device__ __forceinline__ uint4 ld16(const void* p) {   // 16 bytes, read once
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p)
               : "memory");
  return v;
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&f)[8]) {   // 8 bf16, read once
  const uint4 v = ld16(p);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    f[2 * j] = bf16_lo(w[j]);
    f[2 * j + 1] = bf16_hi(w[j]);
  }
}
__device__ __forceinline__ void load8(const float* p, float (&f)[8]) {
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];"
      : "=f"(f[0]), "=f"(f[1]), "=f"(f[2]), "=f"(f[3])
      : "l"(p)
      : "memory");
  asm volatile("ld.global.L1::no_allocate.v4.f32 {%0,%1,%2,%3}, [%4];"
      : "=f"(f[4]), "=f"(f[5]), "=f"(f[6]), "=f"(f[7])
      : "l"(p + 4)
      : "memory");
}
__device__ __forceinline__ void store8(uint16_t* p, const float (&f)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                            pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&f)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}

// Largest finite magnitude among four bf16 (two packed words).
__device__ __forceinline__ float finite_top(uint32_t a, uint32_t b) {
  const uint32_t v[4] = {(a << 16) & 0x7FFF0000u, a & 0x7FFF0000u, (b << 16) & 0x7FFF0000u,
                         b & 0x7FFF0000u};
  uint32_t top = 0;   // magnitudes compare as integers
#pragma unroll
  for (int i = 0; i < 4; ++i) top = v[i] < 0x7F800000u && v[i] > top ? v[i] : top;
  return __uint_as_float(top);
}

// A power of two that brings values up to `top` (finite, >= 0) below 2^15, and its inverse: a bf16
// times it is an f16 exactly, down to 2^-29 of `top`.
__device__ __forceinline__ void f16_scale(float top, float& up, float& down) {
  int e = (int)(__float_as_uint(top) >> 23) - 127;        // floor(log2 top); subnormal, 0: -127
  e = e < -112 ? -112 : e;                                // keeps both factors normal
  up = __uint_as_float((uint32_t)(14 - e + 127) << 23);   // 2^(14 - e)
  down = __uint_as_float((uint32_t)(e - 14 + 127) << 23);
}

// a b c of positive factors, where the product of two may lie outside the floats although all three's does not: the
// largest and the smallest are multiplied first.
__device__ __forceinline__ float product3(float a, float b, float c) {
  const float lo = fminf(a, b), hi = fmaxf(a, b);
  return fmaxf(hi, c) * fminf(lo, c) * fmaxf(lo, fminf(hi, c));
}

}  // namespace ftmoe
