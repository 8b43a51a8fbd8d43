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
// values, whatever the order of sums: fp32 is good to 2^-19 (with the norm; 2^-21
// without: angle, sine and cosine 2^-22 together, products and sum 2^-24 each,
// the norm's sum and root 2^-20) of a pair's |a| + |b|, a row with a value that
// near to a step (one in some hundred) is done again in fp64, by the warp that
// finds it.  What is exact in fp32 (values, keys that are neither normed nor
// rotated) often lies on a step itself: its quotient is corrected by its residue,
// which finds those exactly.
//
// Bound: HBM.  Lanes as in the rotary kernel: d / 16 lanes to a head's row, each
// with two chunks of 8 dimensions that hold both halves of its pairs, sines and
// cosines kept over a token's heads.  A value's 4-bit codes lie by block, then
// token: the lanes of a warp, which hold neighbouring tokens, exchange them so
// that neighbouring lanes write neighbouring bytes.
#include <cstdint>

#include <cuda_bf16.h>

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
template <int D>
__device__ __forceinline__ uint8_t* piece_of(const CacheParams& p, long long page, int o, int h) {
  return p.pages + ((page * p.H + h) * (p.ps / kFp4Block) + o / kFp4Block) * fp4_piece(D);
}

// -------------------------------------------------------------- the steps --
// The largest magnitude's bits: NaN is above infinity, which is above the rest.
__device__ __forceinline__ uint32_t mag(float x) { return __float_as_uint(x) & 0x7fffffffu; }
constexpr uint32_t kInf = 0x7f800000u;
constexpr uint32_t kNanScale = 0x7f;

struct Scale {
  uint32_t byte;
  float sg, lo, r;  // s g in two parts and the reciprocal of it, 0 where s is 0
};
// Of a block with the largest magnitude `top` (its bits), off by at most `off`;
// near: whether another scale is as likely.
__device__ __forceinline__ Scale scale_of(uint32_t top, float off, float g, bool& near) {
  Scale s;
  const float g6 = 6.f * g, q = __uint_as_float(top) / g6, e = off / g6;
  const uint32_t two = f32x2_e4m3(q - e, q + e);
  near |= (two & 0xffu) != (two >> 8);
  s.byte = top >= kInf ? kNanScale : two >> 8;
  const float f = top >= kInf ? 0.f : e4m3_f32(s.byte);
  s.sg = f * g;
  s.lo = fmaf(f, g, -s.sg);
  s.r = s.sg > 0.f ? 1.f / s.sg : 0.f;
  return s;
}
// y / (s g): a product with the reciprocal, corrected by its residue, so that a
// quotient of few bits comes out exactly.
__device__ __forceinline__ float quotient(float y, const Scale& s) {
  const float t = y * s.r;
  const float rest = fmaf(-t, s.lo, fmaf(-t, s.sg, y));
  return fabsf(t) < 8.f ? fmaf(rest, s.r, t) : t;
}
// Codes of 8 values that are off by at most off[e] or `off`; near: whether
// one of them has another code as likely (a zero's sign says nothing).
__device__ __forceinline__ uint32_t codes_of(const float* y, const Scale& s, float off, unsigned loose, bool& near) {
  float lo[8], hi[8];
  const float e = off * s.r;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float t = quotient(y[i], s), ei = (loose >> i) & 1 ? e : 0.f;
    lo[i] = t - ei;
    hi[i] = t + ei;
  }
  const uint32_t a = f32x8_e2m1(lo), b = f32x8_e2m1(hi);
  near |= ((a ^ b) & 0x77777777u) != 0;
  return b;
}
__device__ __forceinline__ uint32_t codes_exactly(const float* y, const Scale& s) {
  float t[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) t[i] = quotient(y[i], s);
  return f32x8_e2m1(t);
}

// The same in fp64.
__device__ __forceinline__ uint32_t scale64(double top, double g) {
  if (!(top < 1e300)) return kNanScale;
  return f32x2_e4m3(static_cast<float>(fmin(top / (6.0 * g), 448.0)), 0.f) & 0xffu;
}
__device__ __forceinline__ uint32_t codes64(const double* y, uint32_t byte, double g) {
  const double sg = byte == kNanScale ? 0.0 : static_cast<double>(e4m3_f32(byte)) * g;
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double t = sg > 0.0 ? fabs(y[i]) / sg : 0.0;
    const uint32_t c = (t > 0.25) + (t >= 0.75) + (t > 1.25) + (t >= 1.75) + (t > 2.5) + (t >= 3.5) + (t > 5.0);
    w |= (c | (y[i] < 0.0 ? 8u : 0u)) << (4 * i);
  }
  return w;
}

struct Held {
  uint32_t c0, c1;  // codes of the two chunks
  uint32_t s0, s1;  // the scales of their blocks
};

// One row in fp64, by the lanes that have it (the whole warp comes here; rows
// without keys bring `row` = nullptr).
template <int D, int LAYOUT>
__device__ __noinline__ Held exact_row(const CacheParams& p, const __nv_bfloat16* row, long long pos, int c0, int c1,
                                       bool turned, float g) {
  constexpr int LPR = D / 16;
  const int half = p.rot >> 1;
  const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p.weight);
  auto x_of = [&](int d) { return row ? static_cast<double>(__bfloat162float(row[d])) : 0.0; };
  double y[16];
  double ss = 0.0;
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    y[e] = x_of((e < 8 ? c0 * 8 : c1 * 8 - 8) + e);
    ss += y[e] * y[e];
  }
#pragma unroll
  for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(kFull, ss, off);
  const double r = p.norm ? 1.0 / sqrt(ss / D + static_cast<double>(p.eps)) : 1.0;
  auto normed = [&](double x, int d) { return x * r * (w ? static_cast<double>(__bfloat162float(w[d])) : 1.0); };
  auto turn = [&](int f, double& cn, double& sn) {
    const unsigned long long t = static_cast<unsigned long long>(pos) * p.freq[f];
    sincospi(static_cast<double>(static_cast<long long>(t)) * 1.0842021724855044e-19, &sn, &cn);  // 2^-63
    cn *= static_cast<double>(p.gain);
    sn *= static_cast<double>(p.gain);
  };
#pragma unroll
  for (int e = 0; e < 16; ++e) y[e] = normed(y[e], (e < 8 ? c0 * 8 : c1 * 8 - 8) + e);
  double cn, sn;
  if (LAYOUT == kHalf) {
    if (turned) {
#pragma unroll 1
      for (int e = 0; e < 8; ++e) {
        turn(c0 * 8 + e, cn, sn);
#pragma unroll
        for (int i = 0; i < 8; ++i)  // (registers, not an array in memory)
          if (i == e) {
            const double a = y[i], b = y[8 + i];
            y[i] = a * cn - b * sn;
            y[8 + i] = b * cn + a * sn;
          }
      }
    }
  } else {
#pragma unroll 1
    for (int e = 0; e < 16; e += LAYOUT == kPairs ? 2 : 1) {
      const int d = c0 * 8 + e;
      if (d >= p.rot) break;
      if (LAYOUT == kPairs) {
        turn(d >> 1, cn, sn);
#pragma unroll
        for (int i = 0; i < 16; i += 2)
          if (i == e) {
            const double a = y[i], b = y[i + 1];
            y[i] = a * cn - b * sn;
            y[i + 1] = b * cn + a * sn;
          }
      } else {
        const int other = d < half ? d + half : d - half;
        const double z = normed(x_of(other), other);
        turn(d < half ? d : other, cn, sn);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (i == e) y[i] = d < half ? y[i] * cn - z * sn : y[i] * cn + z * sn;
      }
    }
  }
  constexpr double kBad = 1e308;  // above everything that a row of bf16 can come to
  auto size = [](double v) { return fabs(v) < kBad ? fabs(v) : kBad; };
  double t0 = 0.0, t1 = 0.0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    t0 = fmax(t0, size(y[e]));
    t1 = fmax(t1, size(y[8 + e]));
  }
  if (LAYOUT == kHalf) {
    const double o0 = __shfl_xor_sync(kFull, t0, 1), o1 = __shfl_xor_sync(kFull, t1, 1);
    t0 = turned ? fmax(t0, o0) : fmax(t0, t1);
    t1 = turned ? fmax(t1, o1) : t0;
  } else {
    t0 = t1 = fmax(t0, t1);
  }
  Held h;
  h.s0 = scale64(t0, g);
  h.s1 = scale64(t1, g);
  h.c0 = codes64(y, h.s0, g);
  h.c1 = codes64(y + 8, h.s1, g);
  return h;
}

// ------------------------------------------------------------------ append --
template <int D, int LAYOUT, bool FP4>
__global__ void __launch_bounds__(kThreads) append_kernel(const CacheParams p) {
  constexpr int LPR = D / 16;            // lanes to a row
  constexpr int kGroups = kThreads / LPR;
  constexpr int kPerWarp = 32 / LPR;     // rows to a warp
  const int half = p.rot >> 1, lane = threadIdx.x & 31;
  const int l = threadIdx.x % LPR;
  const long long unit = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / LPR;
  // (a group without a token stores nothing, but joins the shuffles)
  const long long tok = unit < p.n_units ? unit / p.shares : 0;
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

  uint4 ka = make_uint4(0u, 0u, 0u, 0u), kb = ka, va = ka, vb = ka;
  auto load = [&](int i) {
    if (i < n) {
      ka = *reinterpret_cast<const uint4*>(ksrc + i * D + c0 * 8);
      kb = *reinterpret_cast<const uint4*>(ksrc + i * D + c1 * 8);
      va = *reinterpret_cast<const uint4*>(vsrc + i * D + l * 16);
      vb = *reinterpret_cast<const uint4*>(vsrc + i * D + l * 16 + 8);
    }
  };
  load(0);

  const long long pos = p.rot ? p.positions[tok] : 0;
  constexpr int kTurns = LAYOUT == kAny ? 16 : 8;
  float cs[kTurns], sn[kTurns];
#pragma unroll
  for (int e = 0; e < kTurns; ++e) {
    int f;  // the pair
    if (LAYOUT == kHalf) {
      f = turned ? c0 * 8 + e : -1;
    } else if (LAYOUT == kPairs) {
      f = c0 * 4 + e;
      if (f >= half) f = -1;
    } else {
      const int d = c0 * 8 + e;
      f = d < half ? d : d < p.rot ? d - half : -1;
    }
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (f >= 0) {
      const unsigned long long turn = static_cast<unsigned long long>(pos) * p.freq[f];
      sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &sn[e], &cs[e]);  // 2^-31
      cs[e] *= p.gain;
      sn[e] *= p.gain;
    }
  }
  float ga[8], gb[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) ga[e] = gb[e] = 1.f;
  if (p.weight) {
    const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p.weight);
    unpack8(*reinterpret_cast<const uint4*>(w + c0 * 8), ga);
    unpack8(*reinterpret_cast<const uint4*>(w + c1 * 8), gb);
  }
  // which of the lane's dimensions are not exact in fp32, and by how much of
  // |a| + |b| they are off
  unsigned loose = p.norm || turned ? 0xffffu : 0u;
  if (LAYOUT != kHalf && !p.norm && c0 * 8 < p.rot) loose = p.rot - c0 * 8 >= 16 ? 0xffffu : (1u << (p.rot - c0 * 8)) - 1u;
  const float err = (p.norm ? 1.9073486328125e-06f : 4.76837158203125e-07f) * fmaxf(1.f, p.gain);

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

  for (int i = 0; i < p.heads_per_unit; ++i) {
    float a[8], b[8], x[8], z[8];
    unpack8(ka, a);
    unpack8(kb, b);
    const bool live = i < n;
    const uint4 v0 = va, v1 = vb;
    load(i + 1);
    const __nv_bfloat16* row = ksrc + i * D;
    bool near = false;  // whether the row is to be done in fp64
    float oa[8], ob[8];  // kAny: each element's partner, normed
    if (LAYOUT == kAny) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int da = c0 * 8 + e, db = c1 * 8 + e;
        oa[e] = live && da < p.rot ? __bfloat162float(row[da < half ? da + half : da - half]) : 0.f;
        ob[e] = live && db < p.rot ? __bfloat162float(row[db < half ? db + half : db - half]) : 0.f;
      }
    }
    if (p.norm) {
      float ss = 0.f;  // (in the rotary kernel's order)
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(kFull, ss, off);
      near = !(ss < 1e36f);  // (bf16 squares pass fp32's range)
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] *= r * ga[e];
        b[e] *= r * gb[e];
      }
      if (LAYOUT == kAny) {
        const __nv_bfloat16* w = static_cast<const __nv_bfloat16*>(p.weight);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int da = c0 * 8 + e, db = c1 * 8 + e;
          oa[e] *= r * (w && da < p.rot ? __bfloat162float(w[da < half ? da + half : da - half]) : 1.f);
          ob[e] *= r * (w && db < p.rot ? __bfloat162float(w[db < half ? db + half : db - half]) : 1.f);
        }
      }
    }
    float off = 0.f;  // the largest |a| + |b|
    if (LAYOUT == kHalf) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        x[e] = turned ? a[e] * cs[e] - b[e] * sn[e] : a[e];
        z[e] = turned ? b[e] * cs[e] + a[e] * sn[e] : b[e];
        off = fmaxf(off, fabsf(a[e]) + fabsf(b[e]));
      }
    } else if (LAYOUT == kPairs) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        x[e] = a[e] * cs[e >> 1] - a[e + 1] * sn[e >> 1];
        x[e + 1] = a[e + 1] * cs[e >> 1] + a[e] * sn[e >> 1];
        z[e] = b[e] * cs[4 + (e >> 1)] - b[e + 1] * sn[4 + (e >> 1)];
        z[e + 1] = b[e + 1] * cs[4 + (e >> 1)] + b[e] * sn[4 + (e >> 1)];
        off = fmaxf(off, fmaxf(fabsf(a[e]) + fabsf(a[e + 1]), fabsf(b[e]) + fabsf(b[e + 1])));
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int da = c0 * 8 + e, db = c1 * 8 + e;
        x[e] = da < p.rot ? a[e] * cs[e] + (da < half ? -oa[e] : oa[e]) * sn[e] : a[e];
        z[e] = db < p.rot ? b[e] * cs[8 + e] + (db < half ? -ob[e] : ob[e]) * sn[8 + e] : b[e];
        off = fmaxf(off, fmaxf(fabsf(a[e]) + fabsf(oa[e]), fabsf(b[e]) + fabsf(ob[e])));
      }
    }
    if (!FP4) {
      if (live) {
        *reinterpret_cast<uint4*>(kout + i * D + c0 * 8) = pack8(x);
        *reinterpret_cast<uint4*>(kout + i * D + c1 * 8) = pack8(z);
        *reinterpret_cast<uint4*>(vout + i * D + l * 16) = v0;
        *reinterpret_cast<uint4*>(vout + i * D + l * 16 + 8) = v1;
      }
      continue;
    }
    // the key's blocks: a lane's two chunks, or one chunk of each of two lanes
    off = loose ? off * err : 0.f;
    uint32_t t0 = 0, t1 = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      t0 = max(t0, mag(x[e]));
      t1 = max(t1, mag(z[e]));
    }
    if (LAYOUT == kHalf) {
      const uint32_t o0 = __shfl_xor_sync(kFull, t0, 1), o1 = __shfl_xor_sync(kFull, t1, 1);
      const float oo = __shfl_xor_sync(kFull, off, 1);
      if (turned) off = fmaxf(off, oo);
      t0 = turned ? max(t0, o0) : max(t0, t1);
      t1 = turned ? max(t1, o1) : t0;
    } else {
      t0 = t1 = max(t0, t1);
    }
    const int h = live ? h_begin + i : 0;
    const float gk = p.k_scale ? p.k_scale[h] : 1.f;
    Held kh;
    {
      const Scale s0 = scale_of(t0, off, gk, near);
      kh.s0 = s0.byte;
      kh.c0 = codes_of(x, s0, off, loose & 0xffu, near);
      const Scale s1 = LAYOUT == kHalf ? scale_of(t1, off, gk, near) : s0;
      kh.s1 = s1.byte;
      kh.c1 = codes_of(z, s1, off, loose >> 8, near);
    }
    if (__any_sync(kFull, near && live)) kh = exact_row<D, LAYOUT>(p, live ? row : nullptr, pos, c0, c1, turned, gk);
    if (live) {
      uint8_t* dst = kdst + i * hstride;
      uint8_t* sdst = ksdst + i * hstride;
      if (turned) {
        *reinterpret_cast<uint32_t*>(dst + c0 * 4) = kh.c0;
        *reinterpret_cast<uint32_t*>(dst + c1 * 4) = kh.c1;
        if ((l & 1) == 0) {
          sdst[c0 >> 1] = static_cast<uint8_t>(kh.s0);
          sdst[c1 >> 1] = static_cast<uint8_t>(kh.s1);
        }
      } else {
        *reinterpret_cast<uint2*>(dst + l * 8) = make_uint2(kh.c0, kh.c1);
        sdst[l] = static_cast<uint8_t>(kh.s0);
      }
    }
    // the value's block
    unpack8(v0, x);
    unpack8(v1, z);
    uint32_t tv = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) tv = max(tv, max(mag(x[e]), mag(z[e])));
    bool none = false;
    const Scale sv = scale_of(tv, 0.f, p.v_scale ? p.v_scale[h] : 1.f, none);
    const uint32_t d0 = __shfl_sync(kFull, codes_exactly(x, sv), vsrc_lane);
    const uint32_t d1 = __shfl_sync(kFull, codes_exactly(z, sv), vsrc_lane);
    const uint32_t ds = __shfl_sync(kFull, sv.byte, vsrc_lane);
    if (i < vn) {
      *reinterpret_cast<uint2*>(vdst + i * hstride) = make_uint2(d0, d1);
      vsdst[i * hstride] = static_cast<uint8_t>(ds);
    }
  }
}

// -------------------------------------------------------------------- read --
// 16 values of one block, rounded once.
__device__ __forceinline__ void block_values(uint2 codes, uint32_t scale, float g, uint4* out) {
  const uint32_t s = e4m3x2_f16x2(scale | scale << 8);
  auto two = [&](uint32_t f16x2) {
    const __half2 x = *reinterpret_cast<const __half2*>(&f16x2);
    return pack_bf16x2(__low2float(x) * g, __high2float(x) * g);
  };
  out[0] = make_uint4(two(mul_f16x2(e2m1x2_f16x2<0>(codes.x), s)), two(mul_f16x2(e2m1x2_f16x2<1>(codes.x), s)),
                      two(mul_f16x2(e2m1x2_f16x2<2>(codes.x), s)), two(mul_f16x2(e2m1x2_f16x2<3>(codes.x), s)));
  out[1] = make_uint4(two(mul_f16x2(e2m1x2_f16x2<0>(codes.y), s)), two(mul_f16x2(e2m1x2_f16x2<1>(codes.y), s)),
                      two(mul_f16x2(e2m1x2_f16x2<2>(codes.y), s)), two(mul_f16x2(e2m1x2_f16x2<3>(codes.y), s)));
}

template <int D, bool FP4>
__global__ void __launch_bounds__(kThreads) read_kernel(const CacheParams p) {
  constexpr int LPR = D / 16;
  constexpr int kGroups = kThreads / LPR;
  constexpr int kPerWarp = 32 / LPR;
  const int lane = threadIdx.x & 31, l = threadIdx.x % LPR;
  const long long unit = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / LPR;
  const long long tok = unit < p.n_units ? unit / p.shares : 0;
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
#pragma unroll 2
    for (int i = 0; i < n; ++i) {
      const uint4* k4 = reinterpret_cast<const uint4*>(ks + i * D);
      const uint4* v4 = reinterpret_cast<const uint4*>(vs + i * D);
      const uint4 a = k4[0], b = k4[1], c = v4[0], d = v4[1];
      uint4* ko = reinterpret_cast<uint4*>(kout + i * D);
      uint4* vo = reinterpret_cast<uint4*>(vout + i * D);
      ko[0] = a, ko[1] = b;
      vo[0] = c, vo[1] = d;
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
      uint4 w[2];
      if (i < n) {
        block_values(kw[j], kq[j], gk[j], w);
        uint4* to = reinterpret_cast<uint4*>(kout + i * D);
        to[0] = w[0], to[1] = w[1];
      }
      if (i < vn) {
        block_values(vw[j], vq[j], gv[j], w);
        uint4* to = reinterpret_cast<uint4*>(vout + i * D);
        to[0] = w[0], to[1] = w[1];
      }
    }
  }
}

// A token's heads in shares: all of them to one group of lanes where that
// leaves every SM about eight rounds, else spread.
template <typename F>
cudaError_t spread(CacheParams p, long long T, int D, F&& go) {
  const int groups = kThreads / (D / 16);
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  const long long rounds = static_cast<long long>(sms) * groups * 8;
  long long hpu = (T * p.H + rounds - 1) / rounds;
  if (hpu > p.H) hpu = p.H;
  p.shares = static_cast<int>((p.H + hpu - 1) / hpu);
  p.heads_per_unit = (p.H + p.shares - 1) / p.shares;
  p.shares = (p.H + p.heads_per_unit - 1) / p.heads_per_unit;
  p.n_units = T * p.shares;
  const long long grid = (p.n_units + groups - 1) / groups;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  go(p, static_cast<unsigned>(grid));
  return cudaGetLastError();
}

template <int D, bool FP4>
cudaError_t append_t(const CacheParams& p, long long T, cudaStream_t s) {
  return spread(p, T, D, [&](const CacheParams& q, unsigned grid) {
    if (q.rot == 0 || q.layout == 1) append_kernel<D, kPairs, FP4><<<grid, kThreads, 0, s>>>(q);
    else if (q.rot % 32 == 0) append_kernel<D, kHalf, FP4><<<grid, kThreads, 0, s>>>(q);
    else append_kernel<D, kAny, FP4><<<grid, kThreads, 0, s>>>(q);
  });
}
template <int D, bool FP4>
cudaError_t read_t(const CacheParams& p, long long T, cudaStream_t s) {
  return spread(p, T, D, [&](const CacheParams& q, unsigned grid) { read_kernel<D, FP4><<<grid, kThreads, 0, s>>>(q); });
}

}  // namespace

cudaError_t launch_cache_append(const CacheParams& p, long long T, int d, cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  if (p.pages) return d == 128 ? append_t<128, true>(p, T, s) : append_t<64, true>(p, T, s);
  return d == 128 ? append_t<128, false>(p, T, s) : append_t<64, false>(p, T, s);
}
cudaError_t launch_cache_read(const CacheParams& p, long long T, int d, cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  if (p.pages) return d == 128 ? read_t<128, true>(p, T, s) : read_t<64, true>(p, T, s);
  return d == 128 ? read_t<128, false>(p, T, s) : read_t<64, false>(p, T, s);
}

}  // namespace mf
