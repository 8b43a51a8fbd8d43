// mf_ff.cuh — arithmetic in two fp32 numbers (a high part and what it lacks),
// good to 2^-43.6 (sine and cosine of a turn; sums and products to 2^-45).
//
// GB300 has a sixty-fourth of its fp32 rate in fp64: a row of 128 normed, rotated
// and rounded dimensions took a warp 28 us in it, in this 5, and two blocks of 16
// dimensions 1.3.  The sums and products are the error-free ones of Dekker (1971)
// and Knuth, with an fma for a product's rest.
//
// A host compiler takes it too, for the tests that compare it with wider numbers.
#pragma once
#include <cmath>
#include <cstdint>

#ifdef __CUDACC__
#define MF_FF __device__ __forceinline__
#else
#define MF_FF inline
#endif

namespace mf {

struct ff {
  float h, l;
};

// (never contracted into an fma: the rest of a sum is what its rounding lost)
MF_FF float mul_rn(float a, float b) {
#ifdef __CUDACC__
  return __fmul_rn(a, b);
#else
  const volatile float r = a * b;
  return r;
#endif
}
MF_FF float add_rn(float a, float b) {
#ifdef __CUDACC__
  return __fadd_rn(a, b);
#else
  const volatile float r = a + b;
  return r;
#endif
}
MF_FF ff ff_fast_sum(float a, float b) {  // |a| >= |b|
  const float s = add_rn(a, b);
  return {s, add_rn(b, -add_rn(s, -a))};
}
MF_FF ff ff_sum(float a, float b) {
  const float s = add_rn(a, b), bb = add_rn(s, -a);
  return {s, add_rn(add_rn(a, -add_rn(s, -bb)), add_rn(b, -bb))};
}
MF_FF ff ff_add(ff a, ff b) {
  const ff s = ff_sum(a.h, b.h);
  return ff_fast_sum(s.h, add_rn(s.l, add_rn(a.l, b.l)));
}
MF_FF ff ff_mul(ff a, ff b) {
  const float p = mul_rn(a.h, b.h);
  return ff_fast_sum(p, fmaf(a.l, b.h, fmaf(a.h, b.l, fmaf(a.h, b.h, -p))));
}
MF_FF ff ff_mul(ff a, float b) {
  const float p = mul_rn(a.h, b);
  return ff_fast_sum(p, fmaf(a.l, b, fmaf(a.h, b, -p)));
}
MF_FF ff ff_neg(ff a) { return {-a.h, -a.l}; }

// cosine and sine of j / 64 of a turn, each in two parts
#ifdef __CUDACC__
__device__
#endif
const float kFfTurn[9][4] = {
    {1.f, 0.f, 0.f, 0.f},
    {0.99518472f, 7.10966619e-09f, 0.0980171412f, -8.93393193e-10f},
    {0.980785251f, 2.97394731e-08f, 0.195090324f, -1.67047143e-09f},
    {0.956940353f, -1.7184508e-08f, 0.290284663f, 1.38156651e-08f},
    {0.923879504f, 2.83074897e-08f, 0.382683426f, 6.22335072e-09f},
    {0.881921291f, -2.70029634e-08f, 0.471396744f, -7.42525375e-09f},
    {0.831469595f, 1.68702634e-08f, 0.555570245f, -1.17695214e-08f},
    {0.773010433f, 2.06425526e-08f, 0.634393275f, 9.37955758e-09f},
    {0.707106769f, 1.21016175e-08f, 0.707106769f, 1.21016175e-08f},
};

// Cosine and sine of `turn` 2^-64ths of a turn: the nearest quarter turn, then
// the nearest 64th, whose values are added to those of the rest (at most 0.05
// radians), of which three terms of the series suffice.
MF_FF void ff_sincos(uint64_t turn, ff* sn, ff* cn) {
  const unsigned quarter = static_cast<unsigned>((turn + (1ull << 61)) >> 62) & 3u;
  const int64_t r = static_cast<int64_t>(turn - (static_cast<uint64_t>(quarter) << 62));
  const uint64_t a = r < 0 ? 0ull - static_cast<uint64_t>(r) : static_cast<uint64_t>(r);
  const unsigned j = static_cast<unsigned>((a + (1ull << 57)) >> 58);
  const int64_t s = static_cast<int64_t>(a - (static_cast<uint64_t>(j) << 58));
  const float sh = static_cast<float>(s), sl = static_cast<float>(s - static_cast<int64_t>(sh));
  const ff d = ff_mul(ff{mul_rn(sh, 5.42101086e-20f), mul_rn(sl, 5.42101086e-20f)}, ff{6.28318548f, -1.74845553e-07f});  // 2^-64, 2 pi
  const ff d2 = ff_mul(d, d);
  const float x = d2.h;
  // sin d = d + d p, cos d = 1 + c
  ff p = ff_mul(d2, ff{-0.166666672f, 4.96705388e-09f});
  p = ff_fast_sum(p.h, add_rn(p.l, mul_rn(mul_rn(x, x), fmaf(x, -1.f / 5040.f, 1.f / 120.f))));
  ff c = {-0.5f * d2.h, -0.5f * d2.l};
  c = ff_fast_sum(c.h, add_rn(c.l, mul_rn(mul_rn(x, x), fmaf(x, -1.f / 720.f, 1.f / 24.f))));
  const ff sd = ff_add(d, ff_mul(d, p));
  const float* t = kFfTurn[j];
  const ff C = {t[0], t[1]}, S = {t[2], t[3]};
  const ff co = ff_add(C, ff_add(ff_mul(C, c), ff_neg(ff_mul(S, sd))));
  ff si = ff_add(S, ff_add(ff_mul(S, c), ff_mul(C, sd)));
  if (r < 0) si = ff_neg(si);
  *cn = quarter == 0 ? co : quarter == 1 ? ff_neg(si) : quarter == 2 ? ff_neg(co) : si;
  *sn = quarter == 0 ? si : quarter == 1 ? co : quarter == 2 ? ff_neg(si) : ff_neg(co);
}

}  // namespace mf
#undef MF_FF
