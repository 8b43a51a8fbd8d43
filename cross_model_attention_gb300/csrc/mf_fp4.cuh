// mf_fp4.cuh — the 4-bit form of a paged cache: conversions and where a
// token's bytes are.
//
// 16 neighbouring dimensions of a token's head share a scale s in e4m3, a value
// is an e2m1 number times s times a scale g of its head.  An e2m1 number has at
// most two significant bits and an e4m3 number four, so their product is exact
// in fp16 (from 2^-10 to 2688) and in anything wider.
//
// 16 tokens of a head are 18 d bytes, so that any multiple of 16 tokens is one
// contiguous piece and a page of any such size needs no other layout:
//   keys' codes   [16 tokens][d/2]                    at 0
//   values' codes [2][d/16 blocks][8 tokens][8]       at 8 d
//   keys' scales  [16 tokens][d/16]                   at 16 d
//   values' scales [d/16][16 tokens]                  at 17 d
// Keys meet the product with q along their dimensions, values theirs with the
// weights along the tokens: the order is that in which the operands of both
// matrix products lie in a warp's lanes, 16 bytes to a lane and no two lanes of
// a quarter warp in one bank.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>

namespace mf {

constexpr int kFp4Block = 16;  // dimensions that share a scale, and tokens of a piece
__host__ __device__ constexpr int fp4_piece(int d) { return 18 * d; }

// Two e2m1 codes (byte I of w, the first in the low bits) as fp16.
template <int I>
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t w) {
  uint32_t r;
  if (I == 0) asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, a;}" : "=r"(r) : "r"(w));
  if (I == 1) asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, b;}" : "=r"(r) : "r"(w));
  if (I == 2) asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, c;}" : "=r"(r) : "r"(w));
  if (I == 3) asm("{.reg .b8 a, b, c, d; mov.b32 {a, b, c, d}, %1; cvt.rn.f16x2.e2m1x2 %0, d;}" : "=r"(r) : "r"(w));
  return r;
}
// Two e4m3 scales as fp16.
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two)));
  return r;
}
__device__ __forceinline__ float e4m3_f32(uint32_t byte) {
  const uint32_t r = e4m3x2_f16x2(byte & 0xffu);
  return __half2float(__ushort_as_half(static_cast<unsigned short>(r & 0xffffu)));
}
// Eight numbers as e2m1 codes, to the nearest, ties to even, at most 6.
__device__ __forceinline__ uint32_t f32x8_e2m1(const float* t) {
  uint32_t r;
  asm("{.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};}"
      : "=r"(r)
      : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
  return r;
}
// Two numbers as e4m3 (lo in the low byte), to the nearest, ties to even, at most 448.
__device__ __forceinline__ uint32_t f32x2_e4m3(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %2, %1;" : "=h"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 32 bytes at a 32-byte aligned address: a lane's whole sector.
struct Sector {
  uint32_t w[8];
};
__device__ __forceinline__ void st_sector(void* p, const Sector& s) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(s.w[0]), "r"(s.w[1]), "r"(s.w[2]),
               "r"(s.w[3]), "r"(s.w[4]), "r"(s.w[5]), "r"(s.w[6]), "r"(s.w[7])
               : "memory");
}
__device__ __forceinline__ Sector ld_sector(const void* p) {
  Sector s;
  asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(s.w[0]), "=r"(s.w[1]), "=r"(s.w[2]), "=r"(s.w[3]), "=r"(s.w[4]), "=r"(s.w[5]), "=r"(s.w[6]), "=r"(s.w[7])
               : "l"(p));
  return s;
}

}  // namespace mf
