// mma16.cuh -- warp-level 16-bit matrix products (m16n8k16, fp16 operands,
// fp32 accumulators) and the moves between their register layouts and shared
// memory.
//
// Register layouts, with g = lane / 4 and c = lane % 4:
//   accumulator 16 x 8:  d[0], d[1] = (g, 2c), (g, 2c+1); d[2], d[3] = rows g + 8
//   A 16 x 16 (4 words): (g, 2c..), (g+8, 2c..), (g, 2c+8..), (g+8, 2c+8..)
//   B 16 x 8 (2 words):  (k = 2c.., n = g), (k = 2c+8.., n = g)
// So two neighbouring accumulator tiles, rounded, are the A operand of the
// next product: a chain of products needs no trip through shared memory.
//
// Shared tiles are rows of 16-byte chunks, chunk j of row r at j ^ (r % 8), so
// that the eight rows of a fragment load fall into different banks.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace mma16 {

__device__ __forceinline__ uint32_t smem_at(const void *p) { return static_cast<uint32_t>(__cvta_generic_to_shared(p)); }

// Byte offset of 16-byte chunk j of row r in a tile whose rows have `bytes` (a multiple of 128).
__host__ __device__ __forceinline__ uint32_t swz(uint32_t r, uint32_t j, uint32_t bytes) {
  return r * bytes + ((j ^ (r & 7u)) << 4);
}

__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void stsm4t(uint32_t addr, const uint32_t (&r)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}

__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}
__device__ __forceinline__ float2 unpack(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2 *>(&v)); }
__device__ __forceinline__ float2 unpack_bf16(uint32_t v) {
  return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// (a, b) as fp16 plus, with kTerms 2, the fp16 of what the first rounding
// left over: 11 or 22 bits of the value.
template <int kTerms>
__device__ __forceinline__ void split(float a, float b, uint32_t (&out)[kTerms]) {
  out[0] = pack(a, b);
  if constexpr (kTerms == 2) {
    const float2 h = unpack(out[0]);
    out[1] = pack(a - h.x, b - h.y);
  }
}

// Power of two 2^e with 2^(e-1) <= m < 2^e, e held to +-100; 1 for m = 0 and for what is not finite.
__device__ __forceinline__ float pow2_above(float m) {
  const uint32_t u = __float_as_uint(m);
  int e = int((u >> 23) & 255u) - 126;
  if (m == 0.f || e > 128) return 1.f;
  e = max(-100, min(100, e));
  return __uint_as_float(uint32_t(e + 127) << 23);
}
// 1 / s of a power of two s = 2^e, |e| <= 126, exactly.
__device__ __forceinline__ float pow2_inv(float s) { return __uint_as_float(0x7F000000u - __float_as_uint(s)); }

// Address of this lane's row in a four-matrix load of B operands: matrices
// (n0, k0), (n0, k0+8), (n0+8, k0), (n0+8, k0+8) of a tile [n][k], giving b0,
// b1 of the n-tile at n0 and b0, b1 of the one at n0 + 8.
__device__ __forceinline__ uint32_t b_addr(uint32_t tile, int n0, int k0, int bytes, int lane) {
  return tile + swz(n0 + (lane & 7) + ((lane >> 4) << 3), (k0 >> 3) + ((lane >> 3) & 1), bytes);
}
// A operand 16 x 16 at (m0, k0) of a tile [m][k].
__device__ __forceinline__ uint32_t a_addr(uint32_t tile, int m0, int k0, int bytes, int lane) {
  return tile + swz(m0 + (lane & 7) + (((lane >> 3) & 1) << 3), (k0 >> 3) + (lane >> 4), bytes);
}
// A operand 16 x 16 at (m0, k0) of a tile [k][m] (transposing load).
__device__ __forceinline__ uint32_t at_addr(uint32_t tile, int m0, int k0, int bytes, int lane) {
  return tile + swz(k0 + (lane & 7) + ((lane >> 4) << 3), (m0 >> 3) + ((lane >> 3) & 1), bytes);
}

}  // namespace mma16
