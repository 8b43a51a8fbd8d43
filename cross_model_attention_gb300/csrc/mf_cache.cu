// mf_cache.cu — a paged cache of keys and values: tokens appended to it
// (mf_cache_append) and read back as bf16 rows (mf_cache_read), sm_103a.
//
// Appending, for each head of a token: the key's norm and rotary embedding as
// mf_qk_norm_rope has them,
//   y = x (mean(x^2) + eps)^(-1/2) w,   (y_a, y_b) <- gain (y_a cos t - y_b sin t, ...),
// then, in 4 bits, for 16 neighbouring dimensions and a scale g of the head
//   s = e4m3(max |y| / (6 g)),   code = e2m1(y / (s g)),
// both to the nearest, ties to even, at most 448 and 6.  Values are held as
// they come.  A block with a value that is not finite is held as NaN (s is NaN).
//
// Which code a value gets is a step, and a rounding of fp32 on the wrong side
// of it is an error of a whole code.  Codes are therefore those of the exact
// values, whatever the order of sums.  In units of 2^-24 of a pair's |a| + |b|, fp32
// is good to 7 for angle, sine, cosine and the products with them, 5 for the
// quotient and 7.1 for the norm's sum and root: 20 with the norm and 16
// without are counted, and blocks with a value that near to a step (in one row of
// 150) are done again in twice that precision, by the warp that finds them, once its
// rows are done (mf_ff.cuh: 2^-43, which leaves one value in 10^11 undecided).  What
// is exact in fp32 (values, keys that are neither normed nor rotated) often lies on
// a step itself: its quotient is corrected by its residue, which finds those exactly,
// and what only rounds to a step goes back to its side.
//
// Bound: HBM for bf16 rows (4099 tokens of 40 heads of 128 put in their places in
// 30 us, 5.6 TB/s, 82 % of the copy rate) and reading (32000 tokens of 8 heads 29 us,
// 5.8 TB/s).  For 4 bits (16384 tokens of 8 heads 33 us, 2.6 TB/s) instructions and
// their latency, 57 % of the issue slots used by 16 warps an SM, and the ends of warps
// that do blocks again (26 us where none is).
//
// Lanes as in the rotary kernel: d / 16 lanes to a head's row, each with two chunks
// of 8 dimensions that hold both halves of its pairs, sines and cosines kept over a
// token's heads.  A value's 4-bit codes lie by block, then
// token: the lanes of a warp, which hold neighbouring tokens, exchange them so
// that neighbouring lanes write neighbouring bytes.
#include <cstdint>

#include <cuda_bf16.h>

#include "mf_ff.cuh"
#include "mf_fp4.cuh"
#include "mf_internal.cuh"
#include "mf_ptx.cuh"

namespace mf {
namespace {

constexpr int kThreads = 128;
constexpr unsigned kFull = 0xffffffffu;

__device__ __forceinline__ void unpack8(const uint4& w, float* f) {
  f[0] = bf16lo(w.x), f[1] = bf16hi(w.x), f[2] = bf16lo(w.y), f[3] = bf16hi(w.y);
  f[4] = bf16lo(w.z), f[5] = bf16hi(w.z), f[6] = bf16lo(w.w), f[7] = bf16hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}

// How a lane's two chunks of 8 map to dimensions (rot: rotated ones).
enum { kHalf = 0, kPairs = 1, kAny = 2 };
// kHalf: pairs (i, i + rot/2), rot a multiple of 32 (a pair of lanes then holds
//   whole blocks): chunks l and l + rot/16, past the rotated part 2l and 2l + 1
// kPairs: chunks 2l and 2l + 1, pairs (2i, 2i + 1) or none
// kAny: chunks 2l and 2l + 1, a pair's other element is read again

// The page's number and the place in it of token t's row; false where there is none.
__device__ __forceinline__ bool place_of(const CacheParams& p, long long t, long long& page, int& o) {
  const int s = p.seq[t], at = p.at[t];
  if (static_cast<unsigned>(s) >= static_cast<unsigned>(p.n_seqs) || at < 0) return false;
  const int i = at / p.ps;
  if (i >= p.max_pages) return false;
  o = at - i * p.ps;
  page = p.table[s * p.ld_table + i];
  return page >= 0 && page < p.n_pages;
}
// The token of a unit (of shares of a token's heads).
__device__ __forceinline__ long long token_of(const CacheParams& p, long long unit) {
  if (p.shares == 1) return unit;
  return p.n_units <= 0x7fffffff ? static_cast<int>(unit) / p.shares : unit / p.shares;
}
template <int D>
__device__ __forceinline__ uint8_t* piece_of(const CacheParams& p, long long page, int o, int h) {
  return p.pages + ((page * p.H + h) * (p.ps / kFp4Block) + o / kFp4Block) * fp4_piece(D);
}

// -------------------------------------------------------------- the steps --
// The largest magnitude's bits: NaN is above infinity, which is above the rest.
__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t kInf = 0x7f800000u;
constexpr uint32_t kNanScale = 0x7f;

__device__ __forceinline__ float rcp(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The larger magnitude, NaN where one is.
__device__ __forceinline__ float most(float m, float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(fabsf(a)), "f"(fabsf(b)));
  return r;
}

// A head's scale, NaN where it is out of its range (NaN makes every block's scale NaN):
// there a block's, or its reciprocal, would leave fp32's normal numbers.
__device__ __forceinline__ float head_scale(const float* g, int h) {
  constexpr uint32_t kLeast = 0x1f800000u, kMost = 0x5f800000u;  // 2^-64, 2^64
  const uint32_t x = __float_as_uint(g[h]);
  return x - kLeast <= kMost - kLeast ? __uint_as_float(x) : NAN;
}
struct Scale {
  uint32_t byte;
  float sg, lo, r;  // s g in two parts and the reciprocal of it, 0 where s is 0
};
__device__ __forceinline__ Scale scale_of(uint32_t byte, float g) {
  Scale s;
  const float f = byte == kNanScale ? 0.f : e4m3_f32(byte);
  s.byte = byte;
  s.sg = f * g;
  s.lo = fmaf(f, g, -s.sg);
  s.r = s.sg > 0.f ? rcp(s.sg) : 0.f;
  return s;
}
// Of a block with the largest magnitude `top`, off by at most `off`; near: whether
// another scale is as likely.  (inv_g6 = 1 / (6 g) to a unit in the last place,
// which `off` counts.)
__device__ __forceinline__ uint32_t scale_about(float top, float off, float inv_g6, bool& near) {
  const uint32_t two = f32x2_e4m3(fmaf(top, inv_g6, -off * inv_g6), fmaf(top, inv_g6, off * inv_g6));
  near |= (two & 0xffu) != (two >> 8);
  return top < INFINITY ? two >> 8 : kNanScale;
}
// Where it is exact: of the two scales within 2^-21 of the quotient, if they are not
// the same, that on the side of their middle where top / (6 g) lies; a tie to the
// even one.
__device__ __forceinline__ uint32_t scale_exactly(float top, float g) {
  const float g6 = mul_rn(6.f, g), q = top * rcp(g6);
  const uint32_t two = f32x2_e4m3(q * (1.f - 4.76837158203125e-07f), q * (1.f + 4.76837158203125e-07f));
  const uint32_t a = two & 0xffu, b = two >> 8;
  uint32_t s = a;
  if (a != b) {
    const float border = 0.5f * (e4m3_f32(a) + e4m3_f32(b));
    const float d = add_rn(fmaf(-border, g6, top), -border * fmaf(6.f, g, -g6));
    s = d > 0.f || (d == 0.f && (a & 1)) ? b : a;
  }
  return top < INFINITY ? s : kNanScale;
}
// y / (s g): a product with the reciprocal, corrected by its residue, so that a
// quotient of few bits comes out exactly.
__device__ __forceinline__ float quotient(float y, const Scale& s) {
  const float t = y * s.r;
  return fmaf(fmaf(-t, s.lo, fmaf(-t, s.sg, y)), s.r, t);
}
// Codes of 8 values, each exact in fp32.  A quotient rounded to fp32 is on the right
// side of a border, unless it is the border (its last 21 bits are zero) and was not
// before: then it goes back to the side that its residue says (one value in 10^6; where
// the quotient is the border, the even code is the right one).  Residues are looked at
// where a lane has a quotient on a border at all: without head scales that is often (16384
// tokens of 8 heads 37.3 us, with all residues 36.0), with them hardly ever (33.2, 36.1).
__device__ __forceinline__ uint32_t codes_exactly(const float* y, const Scale& s) {
  float t[8];
  bool odd = false;
  auto on_border = [](float c) { return (__float_as_uint(c) & 0x1fffffu) == 0; };
  if (s.byte == 0x7e) {  // the largest scale: quotients may be of any size
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      t[i] = fabsf(y[i] * s.r) < 8.f ? quotient(y[i], s) : y[i] * s.r;
      odd |= on_border(t[i]);
    }
  } else {
    const float2 r = make_float2(s.r, s.r), sg = make_float2(-s.sg, -s.sg), lo = make_float2(-s.lo, -s.lo);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 v = make_float2(y[i], y[i + 1]), q = fmul2(v, r);
      const float2 c = ffma2(ffma2(q, lo, ffma2(q, sg, v)), r, q);
      t[i] = c.x;
      t[i + 1] = c.y;
      odd |= on_border(c.x) || on_border(c.y);
    }
  }
  if (odd) {  // (mostly quotients that are a border)
    float rest[8];
    odd = false;
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 c = make_float2(t[i], t[i + 1]), sg = make_float2(-s.sg, -s.sg), lo = make_float2(-s.lo, -s.lo);
      const float2 x = ffma2(c, lo, ffma2(c, sg, make_float2(y[i], y[i + 1])));
      rest[i] = x.x;
      rest[i + 1] = x.y;
      odd |= (on_border(c.x) && x.x != 0.f) || (on_border(c.y) && x.y != 0.f);
    }
    if (odd) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float c = t[i];
        if (on_border(c) && rest[i] != 0.f && c != 0.f && fabsf(c) < 8.f)
          t[i] = __int_as_float(__float_as_int(c) + ((rest[i] > 0.f) == (c > 0.f) ? 1 : -1));
      }
    }
  }
  return f32x8_e2m1(t);
}
// Codes of 8 values times r that are off by at most e (which counts the product's
// own rounding); near: whether one of them has another code as likely.  (A zero's sign
// says nothing.  Any other's is certain unless e itself passes the first border, as
// beside values 2^19 times as large.)
__device__ __forceinline__ uint32_t codes_about(const float* y, float r, float e, bool& near) {
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const float2 v = make_float2(y[i], y[i + 1]), f = make_float2(r, r);
    const float2 a = ffma2(v, f, make_float2(-e, -e)), b = ffma2(v, f, make_float2(e, e));
    lo[i] = a.x, lo[i + 1] = a.y;
    hi[i] = b.x, hi[i + 1] = b.y;
  }
  const uint32_t a = f32x8_e2m1(lo), b = f32x8_e2m1(hi);
  near |= ((a ^ b) & 0x77777777u) != 0 || e > 0.25f;
  return b;
}

// The same in two fp32 numbers, of a value and a scale g.
__device__ __forceinline__ uint32_t scale_ff(ff top, float g) {
  if (!(top.h < INFINITY)) return kNanScale;
  const float g6 = mul_rn(6.f, g), q = top.h / g6;
  const uint32_t two = f32x2_e4m3(q * (1.f - 4.76837158203125e-07f), q * (1.f + 4.76837158203125e-07f));
  const uint32_t a = two & 0xffu, b = two >> 8;
  if (a == b) return a;
  const float border = 0.5f * (e4m3_f32(a) + e4m3_f32(b));  // between neighbours: exact
  const float d = add_rn(fmaf(-border, g6, top.h), fmaf(-border, fmaf(6.f, g, -g6), top.l));
  return d > 0.f || (d == 0.f && (a & 1)) ? b : a;
}
__device__ __forceinline__ uint32_t code_ff(ff y, float sg, float lo) {
  const bool minus = y.h < 0.f;
  if (minus) y = ff_neg(y);
  // past the border x (a half between codes goes to the even one)
  auto past = [&](float x, bool even) {
    const float d = add_rn(fmaf(-x, sg, y.h), fmaf(-x, lo, y.l));
    return d > 0.f || (even && d == 0.f) ? 1u : 0u;
  };
  const uint32_t c = past(0.25f, false) + past(0.75f, true) + past(1.25f, false) + past(1.75f, true) + past(2.5f, false) +
                     past(3.5f, true) + past(5.f, false);
  return sg > 0.f ? c | (minus ? 8u : 0u) : 0u;
}
__device__ __forceinline__ ff larger(ff a, ff b) { return a.h > b.h || (a.h == b.h && a.l >= b.l) ? a : b; }
__device__ __forceinline__ ff from_lane(ff a, int mask) {
  return {__shfl_xor_sync(kFull, a.h, mask), __shfl_xor_sync(kFull, a.l, mask)};
}

// Two blocks of a row (or one, b0 = b1) in twice fp32's precision, by a whole warp:
// a dimension to a lane.  (All 128 of them, four to a lane, took 9000 cycles, and a
// warp that finds two or three such rows holds up the rest.)
template <int D>
__device__ __forceinline__ void exact_blocks(const CacheParams& p, const __nv_bfloat16* row, long long pos, float g, int b0,
                                             int b1, uint8_t* codes, uint8_t* scales) {
  constexpr int N = D / 32;
  const int lane = threadIdx.x & 31, half = p.rot >> 1;
  const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p.weight);
  const int block = lane < 16 ? b0 : b1, d = block * 16 + (lane & 15);
  const bool turned = d < p.rot, first = p.layout == 1 ? (d & 1) == 0 : d < half;
  const int other = !turned ? d : p.layout == 1 ? d ^ 1 : first ? d + half : d - half;
  const float xd = __bfloat162float(row[d]), xo = __bfloat162float(row[other]);
  float x[N];
  uint32_t top = 0;
#pragma unroll
  for (int e = 0; e < N; ++e) {
    x[e] = __bfloat162float(row[lane * N + e]);
    top = max(top, mag(x[e]));
  }
  ff cn = {1.f, 0.f}, sn = {0.f, 0.f};
  if (turned) ff_sincos(static_cast<uint64_t>(pos) * p.freq[p.layout == 1 ? d >> 1 : first ? d : other], &sn, &cn);
  top = __reduce_max_sync(kFull, top);
  // rows of huge values are brought into range, with what they are compared with (a
  // little, for sums of two: a small head scale has to stay a normal number); to be
  // normed, further (what the norm gives is in range), and rows of tiny ones under a
  // tiny eps too
  const int ex = static_cast<int>(top >> 23) - 127;
  float down = ex > 100 ? 0.00390625f : 1.f;
  if (p.norm) {
    down = ex > 30 ? __int_as_float((127 - min(ex, 127) + 30) << 23) : 1.f;
    const int e = max(ex, (static_cast<int>(__float_as_uint(p.eps) >> 23) - 127) / 2);
    if (e < -30) down = __int_as_float((127 - e) << 23);
  }
  if (!p.norm) g *= down;
  ff r = {1.f, 0.f};
  if (p.norm) {
    ff ss = {0.f, 0.f};
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const ff t = ff_sum(ss.h, mul_rn(x[e] * down, x[e] * down));  // (a square of 8 bits is exact)
      ss = {t.h, add_rn(ss.l, t.l)};
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) ss = ff_add(ss, from_lane(ss, off));
    const ff m = ff_add(ff{ss.h * (1.f / D), ss.l * (1.f / D)}, ff{p.eps * down * down, 0.f});
    const float r0 = rsqrtf(m.h);
    const ff q = ff_mul(m, ff_mul(ff{r0, 0.f}, r0));
    r = ff_fast_sum(r0, mul_rn(0.5f * r0, add_rn(add_rn(1.f, -q.h), -q.l)));  // one step of Newton's
    if (top >= kInf) r = {top > kInf ? NAN : 0.f, 0.f};  // (an infinity's row: 0 but for it)
  }
  auto normed = [&](float v, int i) {
    v *= down;
    if (w) v = mul_rn(v, __bfloat162float(w[i]));  // (16 bits)
    return p.norm ? ff_mul(r, v) : ff{v, 0.f};
  };
  ff y = normed(xd, d);
  if (turned) {
    const ff t = ff_mul(normed(xo, other), ff_mul(sn, p.gain));
    y = ff_add(ff_mul(y, ff_mul(cn, p.gain)), first ? ff_neg(t) : t);
  }
  ff most = !(fabsf(y.h) < INFINITY) ? ff{INFINITY, 0.f} : y.h < 0.f ? ff_neg(y) : y;
#pragma unroll
  for (int off = 1; off < 16; off <<= 1) most = larger(most, from_lane(most, off));
  const uint32_t s = scale_ff(most, g);
  const float f = s == kNanScale ? 0.f : e4m3_f32(s), sg = mul_rn(f, g), lo = fmaf(f, g, -sg);
  uint32_t c = code_ff(y, sg, lo);
  c |= __shfl_down_sync(kFull, c, 1) << 4;
  if (lane < 16 || b0 != b1) {
    if ((lane & 1) == 0) codes[d >> 1] = static_cast<uint8_t>(c);
    if ((lane & 15) == 0) scales[block] = static_cast<uint8_t>(s);
  }
}

// 16 values of one block, rounded once.
__device__ __forceinline__ Sector block_values(uint2 codes, uint32_t scale, float g) {
  const uint32_t s = e4m3x2_f16x2(scale | scale << 8);
  auto two = [&](uint32_t f16x2) {
    const __half2 x = *reinterpret_cast<const __half2*>(&f16x2);
    return pack_bf16x2(__low2float(x) * g, __high2float(x) * g);
  };
  return {two(mul_f16x2(e2m1x2_f16x2<0>(codes.x), s)), two(mul_f16x2(e2m1x2_f16x2<1>(codes.x), s)),
          two(mul_f16x2(e2m1x2_f16x2<2>(codes.x), s)), two(mul_f16x2(e2m1x2_f16x2<3>(codes.x), s)),
          two(mul_f16x2(e2m1x2_f16x2<0>(codes.y), s)), two(mul_f16x2(e2m1x2_f16x2<1>(codes.y), s)),
          two(mul_f16x2(e2m1x2_f16x2<2>(codes.y), s)), two(mul_f16x2(e2m1x2_f16x2<3>(codes.y), s))};
}
// A lane's 16 values to or from memory that is 16-byte aligned: whole sectors
// where `even` says that all the rows' lie so.
__device__ __forceinline__ void put16(__nv_bfloat16* to, const Sector& x, bool even) {
  if (even) {
    st_sector(to, x);
  } else {
    reinterpret_cast<uint4*>(to)[0] = make_uint4(x.w[0], x.w[1], x.w[2], x.w[3]);
    reinterpret_cast<uint4*>(to)[1] = make_uint4(x.w[4], x.w[5], x.w[6], x.w[7]);
  }
}
__device__ __forceinline__ Sector get16(const __nv_bfloat16* from, bool even) {
  if (even) return ld_sector(from);
  const uint4 a = reinterpret_cast<const uint4*>(from)[0], b = reinterpret_cast<const uint4*>(from)[1];
  return {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// ------------------------------------------------------------------ append --
// (Four CTAs to an SM: 16384 tokens of 8 heads 33.2 us; three 36.9, five, which
// spill, 38.1.  At four kAny spills as well, most for rows of bf16:
// 4099 tokens of 40 heads 49 us, the others 30.)
template <int D, int LAYOUT, bool FP4>
__global__ void __launch_bounds__(kThreads, 4) append_kernel(const CacheParams p) {
  constexpr int LPR = D / 16;            // lanes to a row
  constexpr int kGroups = kThreads / LPR;
  constexpr int kPerWarp = 32 / LPR;     // rows to a warp
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // what comes after may be set up
  asm volatile("griddepcontrol.wait;" ::: "memory");               // what came before may still run
  const int half = p.rot >> 1, lane = threadIdx.x & 31;
  const int l = threadIdx.x % LPR;
  const long long unit = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / LPR;
  // (a group without a token stores nothing, but joins the shuffles)
  const long long tok = unit < p.n_units ? token_of(p, unit) : 0;
  const int h_begin = static_cast<int>(unit - tok * p.shares) * p.heads_per_unit;
  long long page = 0;
  int o = 0;
  const bool here = unit < p.n_units && place_of(p, tok, page, o);
  const int n = here ? min(p.heads_per_unit, p.H - h_begin) : 0;
  const long long at = static_cast<long long>(h_begin) * D;
  const __nv_bfloat16* ksrc = static_cast<const __nv_bfloat16*>(p.k_in) + tok * p.ld_kin + at;
  const __nv_bfloat16* vsrc = static_cast<const __nv_bfloat16*>(p.v_in) + tok * p.ld_vin + at;

  const int hc = half / 8;
  const bool turned = LAYOUT == kHalf && l < hc;
  const int c0 = turned ? l : 2 * l, c1 = turned ? l + hc : 2 * l + 1;

  // heads on their way ahead of the one worked on
  constexpr int kAhead = FP4 ? 1 : 2;
  uint4 ka[kAhead], kb[kAhead];
  Sector vw[kAhead];
  auto load = [&](int i, int j) {
    if (i < n) {
      ka[j] = *reinterpret_cast<const uint4*>(ksrc + i * D + c0 * 8);
      kb[j] = *reinterpret_cast<const uint4*>(ksrc + i * D + c1 * 8);
      vw[j] = get16(vsrc + i * D + l * 16, p.even);
    }
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    ka[j] = kb[j] = make_uint4(0u, 0u, 0u, 0u);
    vw[j] = Sector{{0u, 0u, 0u, 0u, 0u, 0u, 0u, 0u}};
    load(j, j);
  }

  // A lane's 16 outputs are its inputs times `own` and their partners (the pair's
  // other half) times `other`: cosines and sines with the weights in them.
  const long long pos = p.rot ? p.positions[tok] : 0;
  const __nv_bfloat16* weight = static_cast<const __nv_bfloat16*>(p.weight);
  // (normed rows of bf16: weights times 2^-40, the norm's factor times 2^40, so that no
  // product with a weight passes fp32's range before a factor of 0 makes the row 0.
  // The factor first, as in the rotary layer, costs kAny 2 of 54 us.)
  constexpr float kDown = FP4 ? 1.f : 9.094947017729282e-13f, kUp = FP4 ? 1.f : 1099511627776.f;
  const float down = p.norm ? kDown : 1.f;
  auto weight_of = [&](int d) { return weight ? __bfloat162float(weight[d]) * down : down; };
  float own[16], other[16], heaviest = 0.f;
  auto turn_of = [&](int f, float& sn, float& cs) {
    const unsigned long long turn = static_cast<unsigned long long>(pos) * p.freq[f];
    sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &sn, &cs);  // 2^-31
    cs *= p.gain;
    sn *= p.gain;
  };
#pragma unroll
  for (int e = 0; e < 16; ++e) own[e] = down, other[e] = FP4 ? 0.f : -0.f;  // (kAny: 0 times -0 leaves a row's -0 too)
  if (weight) {
    unpack8(*reinterpret_cast<const uint4*>(weight + c0 * 8), own);
    unpack8(*reinterpret_cast<const uint4*>(weight + c1 * 8), own + 8);
#pragma unroll
    for (int e = 0; e < 16; ++e) own[e] *= down;
  }
#pragma unroll
  for (int e = 0; e < 16; ++e) heaviest = fmaxf(heaviest, fabsf(own[e]));
  if (LAYOUT == kHalf) {
    if (turned) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float sn, cs;
        turn_of(c0 * 8 + e, sn, cs);
        const float a = own[e], b = own[8 + e];
        own[e] = a * cs;
        own[8 + e] = b * cs;
        other[e] = -b * sn;
        other[8 + e] = a * sn;
      }
    }
  } else if (LAYOUT == kPairs) {
#pragma unroll
    for (int e = 0; e < 16; e += 2) {
      if (c0 * 8 + e < p.rot) {
        float sn, cs;
        turn_of(c0 * 4 + (e >> 1), sn, cs);
        const float a = own[e], b = own[e + 1];
        own[e] = a * cs;
        own[e + 1] = b * cs;
        other[e] = -b * sn;
        other[e + 1] = a * sn;
      }
    }
  } else {
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const int d = c0 * 8 + e;
      if (d < p.rot) {
        float sn, cs;
        const int q = d < half ? d + half : d - half;
        turn_of(d < half ? d : q, sn, cs);
        const float b = weight_of(q);
        own[e] *= cs;
        other[e] = d < half ? -b * sn : b * sn;
        heaviest = fmaxf(heaviest, fabsf(b));
      }
    }
  }
  // Whether the lane's values are not exact in fp32, and how far they may be off,
  // of |a| + |b| (kAny and kPairs: where only some are, the rest is taken to be so too).
  // At position 0 they are: a prompt's first token would have most of its blocks done
  // again by one warp, 12 us after the others of 16384.  (So it is with keys that are
  // neither normed nor scaled where they are hardly turned, for as many tokens as there
  // are: 64 tokens at position 1 take 6.8 us, at 0 4.0 and at 100 4.5; 16384 at once
  // 65, 37 and 35, and at position 1 of angles stretched by 64 114.)
  const bool loose = p.norm || ((LAYOUT == kHalf ? turned : c0 * 8 < p.rot) && (pos != 0 || p.gain != 1.f));
  const float err = (p.norm ? 20.f : 16.f) * 5.9604644775390625e-08f * fmaxf(1.f, fabsf(p.gain));  // 2^-24

  // where the rows go
  uint8_t *kdst = nullptr, *ksdst = nullptr, *vdst = nullptr, *vsdst = nullptr;
  __nv_bfloat16 *kout = nullptr, *vout = nullptr;
  const long long hstride = static_cast<long long>(p.ps / kFp4Block) * fp4_piece(D);  // between heads of a page
  const int i16 = o % kFp4Block;
  const int vsrc_lane = (lane % kPerWarp) * LPR + lane / kPerWarp;  // whose value codes this lane stores
  int vn = 0;
  if (FP4) {
    uint8_t* base = here ? piece_of<D>(p, page, o, h_begin) : nullptr;
    kdst = base + i16 * (D / 2);
    ksdst = base + 16 * D + i16 * (D / 16);
    uint8_t* vbase = reinterpret_cast<uint8_t*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(base), vsrc_lane));
    const int vi = __shfl_sync(kFull, i16, vsrc_lane), b = lane / kPerWarp;
    vn = __shfl_sync(kFull, n, vsrc_lane);
    vdst = vbase + 8 * D + (vi / 8) * (4 * D) + b * 64 + (vi % 8) * 8;
    vsdst = vbase + 17 * D + b * 16 + vi;
  } else if (here) {
    const long long row = page * p.ps + o;
    kout = static_cast<__nv_bfloat16*>(p.k) + row * p.ld_k + at;
    vout = static_cast<__nv_bfloat16*>(p.v) + row * p.ld_v + at;
  }

  float gk_next = FP4 && here && p.k_scale ? head_scale(p.k_scale, h_begin) : 1.f;
  float gv_next = FP4 && here && p.v_scale ? head_scale(p.v_scale, h_begin) : 1.f;
  unsigned again = 0;  // of 32 heads: those with blocks to be done more exactly
#pragma unroll 1
  for (int ib = 0; ib < p.heads_per_unit; ib += kAhead)
#pragma unroll
  for (int ja = 0; ja < kAhead; ++ja) {
    const int i = ib + ja;  // (past the last: a row that is not live)
    float a[16], y[16];
    unpack8(ka[ja], a);
    unpack8(kb[ja], a + 8);
    const bool live = i < n;
    bool near = false;  // whether the lane's blocks are to be done more exactly
    const Sector v = vw[ja];
    load(i + kAhead, ja);
    float r = 1.f;  // the norm's factor
    if (p.norm) {
      float2 s0 = make_float2(0.f, 0.f), s1 = s0;  // (four short sums: a small error)
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float2 x = make_float2(a[e], a[e + 1]), z = make_float2(a[8 + e], a[9 + e]);
        s0 = ffma2(x, x, s0);
        s1 = ffma2(z, z, s1);
      }
      float ss = (s0.x + s0.y) + (s1.x + s1.y);
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(kFull, ss, off);
      const float m = fmaf(ss, 1.f / D, p.eps);
      near = !(ss < 1e36f && m > 1e-30f);  // (bf16 squares pass fp32's range at either end)
      asm("rsqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(m));  // (m may be a subnormal number)
      r *= kUp;
    }
    float sum = 0.f;  // kAny: a bound of |a| + |b|
    if (LAYOUT == kAny) {
      float ma = 0.f, mb = 0.f;
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int d = c0 * 8 + e;
        const float b = live && d < p.rot ? __bfloat162float(ksrc[i * D + (d < half ? d + half : d - half)]) : 0.f;
        y[e] = fmaf(b, other[e], a[e] * own[e]);
        ma = fmaxf(ma, fabsf(a[e]));
        mb = fmaxf(mb, fabsf(b));
      }
      sum = (ma + mb) * heaviest;
    } else {
#pragma unroll
      for (int e = 0; e < 16; e += 2) {
        const float2 x = make_float2(a[e], a[e + 1]);
        const float2 z = LAYOUT == kHalf ? make_float2(a[e ^ 8], a[(e ^ 8) + 1]) : make_float2(x.y, x.x);
        float2 v = fmul2(x, make_float2(own[e], own[e + 1]));
        // (rows of bf16: 0 times what is not finite is not 0.  A 4-bit block of it is NaN as a whole)
        if (FP4 || (LAYOUT == kHalf ? turned : c0 * 8 + e < p.rot)) v = ffma2(z, make_float2(other[e], other[e + 1]), v);
        y[e] = v.x;
        y[e + 1] = v.y;
      }
    }
    if (!FP4) {
      if (live) {
#pragma unroll
        for (int e = 0; e < 16; ++e) y[e] *= r;
        *reinterpret_cast<uint4*>(kout + i * D + c0 * 8) = pack8(y);
        *reinterpret_cast<uint4*>(kout + i * D + c1 * 8) = pack8(y + 8);
        put16(vout + i * D + l * 16, v, p.even);
      }
      continue;
    }
    // the key's blocks: a lane's two chunks, or one chunk of each of two lanes
    float t0 = 0.f, t1 = 0.f;
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      t0 = most(t0, y[e], y[e + 1]);
      t1 = most(t1, y[8 + e], y[9 + e]);
    }
    if (LAYOUT == kHalf) {
      const float o0 = __shfl_xor_sync(kFull, t0, 1), o1 = __shfl_xor_sync(kFull, t1, 1);
      t0 = most(t0, turned ? o0 : t1, 0.f);
      t1 = turned ? most(t1, o1, 0.f) : t0;
    } else {
      t0 = t1 = most(t0, t1, 0.f);
    }
    const float gk = gk_next, gv = gv_next;
    if (i + 1 < n) {
      if (p.k_scale) gk_next = head_scale(p.k_scale, h_begin + i + 1);
      if (p.v_scale) gv_next = head_scale(p.v_scale, h_begin + i + 1);
    }
    {
      uint32_t w0, w1, b0, b1;
      const float inv = rcp(6.f * gk);
      if (loose) {
        // (|a| + |b| is at most 2 max(|y_a|, |y_b|) of the rotated pair, both of
        // which are in these blocks)
        const float off = (LAYOUT == kAny ? sum : 2.f * fmaxf(t0, t1)) * r * err;
        b0 = scale_about(t0 * r, off, inv, near);
        const Scale s0 = scale_of(b0, gk);
        w0 = codes_about(y, r * s0.r, off * s0.r, near);
        b1 = b0;
        float r1 = s0.r;
        if (LAYOUT == kHalf) {
          b1 = scale_about(t1 * r, off, inv, near);
          r1 = scale_of(b1, gk).r;
        }
        w1 = codes_about(y + 8, r * r1, off * r1, near);
      } else {
        b0 = scale_exactly(t0, gk);
        const Scale s0 = scale_of(b0, gk);
        w0 = codes_exactly(y, s0);
        b1 = b0;
        Scale s1 = s0;
        if (LAYOUT == kHalf && turned) {
          b1 = scale_exactly(t1, gk);
          s1 = scale_of(b1, gk);
        }
        w1 = codes_exactly(y + 8, s1);
      }
      if (live) {
        uint8_t* dst = kdst + i * hstride;
        uint8_t* sdst = ksdst + i * hstride;
        if (turned) {
          *reinterpret_cast<uint32_t*>(dst + c0 * 4) = w0;
          *reinterpret_cast<uint32_t*>(dst + c1 * 4) = w1;
          if ((l & 1) == 0) {
            sdst[c0 >> 1] = static_cast<uint8_t>(b0);
            sdst[c1 >> 1] = static_cast<uint8_t>(b1);
          }
        } else {
          *reinterpret_cast<uint2*>(dst + l * 8) = make_uint2(w0, w1);
          sdst[l] = static_cast<uint8_t>(b0);
        }
      }
      if (near && live) again |= 1u << (i & 31);
    }
    // the value's block
#pragma unroll
    for (int e = 0; e < 8; ++e) y[2 * e] = bf16lo(v.w[e]), y[2 * e + 1] = bf16hi(v.w[e]);
    float tv = 0.f;
#pragma unroll
    for (int e = 0; e < 16; e += 2) tv = most(tv, y[e], y[e + 1]);
    const Scale sv = scale_of(scale_exactly(tv, gv), gv);
    const uint32_t d0 = __shfl_sync(kFull, codes_exactly(y, sv), vsrc_lane);
    const uint32_t d1 = __shfl_sync(kFull, codes_exactly(y + 8, sv), vsrc_lane);
    const uint32_t ds = __shfl_sync(kFull, sv.byte, vsrc_lane);
    if (i < vn) {
      *reinterpret_cast<uint2*>(vdst + i * hstride) = make_uint2(d0, d1);
      vsdst[i * hstride] = static_cast<uint8_t>(ds);
    }
    if ((i & 31) == 31 || i + 1 == p.heads_per_unit) {
      __syncwarp();  // (what is written again was written by other lanes)
      for (unsigned rest = __reduce_or_sync(kFull, again); rest; rest &= rest - 1) {
        const int b = __ffs(rest) - 1, j = (i & ~31) + b;
        for (unsigned lanes = __ballot_sync(kFull, again >> b & 1); lanes;) {
          // the blocks that this lane had a part of, and its neighbour where it has one too
          const int from = __ffs(lanes) - 1, fl = from % LPR;
          const bool two = LAYOUT == kHalf && fl < hc;
          lanes &= ~(two ? 3u << (from & ~1) : 1u << from);
          auto of = [&](auto* x) {
            return reinterpret_cast<decltype(x)>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(x), from));
          };
          const int hj = __shfl_sync(kFull, h_begin, from) + j;
          exact_blocks<D>(p, of(ksrc) + j * D, __shfl_sync(kFull, pos, from), p.k_scale ? head_scale(p.k_scale, hj) : 1.f,
                          two ? fl >> 1 : fl, two ? (fl + hc) >> 1 : fl, of(kdst) + j * hstride, of(ksdst) + j * hstride);
        }
      }
      again = 0;
    }
  }
}

// -------------------------------------------------------------------- read --
template <int D, bool FP4>
__global__ void __launch_bounds__(kThreads) read_kernel(const CacheParams p) {
  constexpr int LPR = D / 16;
  constexpr int kGroups = kThreads / LPR;
  constexpr int kPerWarp = 32 / LPR;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, l = threadIdx.x % LPR;
  const long long unit = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / LPR;
  const long long tok = unit < p.n_units ? token_of(p, unit) : 0;
  const int h_begin = static_cast<int>(unit - tok * p.shares) * p.heads_per_unit;
  long long page = 0;
  int o = 0;
  const bool here = unit < p.n_units && place_of(p, tok, page, o);
  const int n = here ? min(p.heads_per_unit, p.H - h_begin) : 0;
  const long long at = static_cast<long long>(h_begin) * D;
  __nv_bfloat16* kout = static_cast<__nv_bfloat16*>(p.k_out) + tok * p.ld_kin + at + l * 16;
  if (!FP4) {
    const long long row = page * p.ps + o;
    const __nv_bfloat16* ks = static_cast<const __nv_bfloat16*>(p.k) + row * p.ld_k + at + l * 16;
    const __nv_bfloat16* vs = static_cast<const __nv_bfloat16*>(p.v) + row * p.ld_v + at + l * 16;
    __nv_bfloat16* vout = static_cast<__nv_bfloat16*>(p.v_out) + tok * p.ld_vin + at + l * 16;
    constexpr int kAhead = 4;
    for (int i0 = 0; i0 < n; i0 += kAhead) {
      Sector a[kAhead], b[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i0 + j < n) {
          a[j] = get16(ks + (i0 + j) * D, p.even);
          b[j] = get16(vs + (i0 + j) * D, p.even);
        }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (i0 + j < n) {
          put16(kout + (i0 + j) * D, a[j], p.even);
          put16(vout + (i0 + j) * D, b[j], p.even);
        }
    }
    return;
  }
  const long long hstride = static_cast<long long>(p.ps / kFp4Block) * fp4_piece(D);
  const uint8_t* base = here ? piece_of<D>(p, page, o, h_begin) : nullptr;
  const int i16 = o % kFp4Block;
  const uint8_t* kc = base + i16 * (D / 2) + l * 8;
  const uint8_t* ks = base + 16 * D + i16 * (D / 16) + l;
  // a value's codes lie by block, then token: lanes take them in that order
  const int src = (lane % kPerWarp) * LPR + lane / kPerWarp, b = lane / kPerWarp;
  const uint8_t* vbase = reinterpret_cast<const uint8_t*>(__shfl_sync(kFull, reinterpret_cast<unsigned long long>(base), src));
  const int vi = __shfl_sync(kFull, i16, src), vn = __shfl_sync(kFull, n, src);
  const long long vtok = __shfl_sync(kFull, tok, src);
  const int vh = __shfl_sync(kFull, h_begin, src);
  const uint8_t* vc = vbase + 8 * D + (vi / 8) * (4 * D) + b * 64 + (vi % 8) * 8;
  const uint8_t* vs = vbase + 17 * D + b * 16 + vi;
  __nv_bfloat16* vout = static_cast<__nv_bfloat16*>(p.v_out) + vtok * p.ld_vin + static_cast<long long>(vh) * D + b * 16;
  constexpr int kAhead = 4;
  for (int i0 = 0; i0 < p.heads_per_unit; i0 += kAhead) {
    uint2 kw[kAhead], vw[kAhead];
    uint32_t kq[kAhead], vq[kAhead];
    float gk[kAhead], gv[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j;
      kw[j] = vw[j] = make_uint2(0u, 0u);
      kq[j] = vq[j] = 0;
      gk[j] = gv[j] = 1.f;
      if (i < n) {
        kw[j] = *reinterpret_cast<const uint2*>(kc + i * hstride);
        kq[j] = ks[i * hstride];
        if (p.k_scale) gk[j] = p.k_scale[h_begin + i];
      }
      if (i < vn) {
        vw[j] = *reinterpret_cast<const uint2*>(vc + i * hstride);
        vq[j] = vs[i * hstride];
        if (p.v_scale) gv[j] = p.v_scale[vh + i];
      }
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int i = i0 + j;
      if (i < n) put16(kout + i * D, block_values(kw[j], kq[j], gk[j]), p.even);
      if (i < vn) put16(vout + i * D, block_values(vw[j], vq[j], gv[j]), p.even);
    }
  }
}

// A token's heads in shares: all of them to one group of lanes where that
// leaves every SM about `rounds` rounds, else spread.  (Appending, whose groups
// begin with sines and cosines, two: 16384 tokens of 8 heads 33.2 us, with eight
// 35.6; 4099 of 40 heads in bf16 29.9, with one 34.1 and with four 31.5.  Reading
// eight: the same 16384 15.8 us, with two 16.4.)
template <typename F>
cudaError_t spread(CacheParams p, long long T, int D, int rounds, F&& go) {
  const int groups = kThreads / (D / 16);
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const long long all = static_cast<long long>(sms) * groups * rounds;
  long long hpu = (T * p.H + all - 1) / all;
  if (hpu > p.H) hpu = p.H;
  p.shares = static_cast<int>((p.H + hpu - 1) / hpu);
  p.heads_per_unit = (p.H + p.shares - 1) / p.shares;
  p.shares = (p.H + p.heads_per_unit - 1) / p.heads_per_unit;
  p.n_units = T * p.shares;
  const long long grid = (p.n_units + groups - 1) / groups;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  return go(p, dim3(static_cast<unsigned>(grid)));
}

bool even32(const void* a, long long ld) { return !a || ((reinterpret_cast<uintptr_t>(a) & 31) == 0 && ld % 16 == 0); }

template <int D, bool FP4>
cudaError_t append_t(const CacheParams& p, long long T, cudaStream_t s) {
  return spread(p, T, D, 2, [&](const CacheParams& q, dim3 grid) {
    const bool pairs = q.rot == 0 || q.layout == 1;
    auto* kernel = pairs ? append_kernel<D, kPairs, FP4> : q.rot % 32 == 0 ? append_kernel<D, kHalf, FP4> : append_kernel<D, kAny, FP4>;
    return launch_early(kernel, grid, kThreads, 0, s, q);
  });
}
template <int D, bool FP4>
cudaError_t read_t(const CacheParams& p, long long T, cudaStream_t s) {
  return spread(p, T, D, 8, [&](const CacheParams& q, dim3 grid) { return launch_early(read_kernel<D, FP4>, grid, kThreads, 0, s, q); });
}

}  // namespace

cudaError_t launch_cache_append(const CacheParams& c, long long T, int d, cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  CacheParams p = c;
  p.even = even32(p.v_in, p.ld_vin) && even32(p.v, p.ld_v);
  if (p.pages) return d == 128 ? append_t<128, true>(p, T, s) : append_t<64, true>(p, T, s);
  return d == 128 ? append_t<128, false>(p, T, s) : append_t<64, false>(p, T, s);
}
cudaError_t launch_cache_read(const CacheParams& c, long long T, int d, cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  CacheParams p = c;
  p.even = even32(p.k_out, p.ld_kin) && even32(p.v_out, p.ld_vin) && even32(p.k, p.ld_k) && even32(p.v, p.ld_v);
  if (p.pages) return d == 128 ? read_t<128, true>(p, T, s) : read_t<64, true>(p, T, s);
  return d == 128 ? read_t<128, false>(p, T, s) : read_t<64, false>(p, T, s);
}

}  // namespace mf
