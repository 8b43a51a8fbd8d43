// mf_rope.cu — per-head RMS norm of queries and keys with the rotary position
// embedding in the same pass (mf_qk_norm_rope), sm_103a.
//
// For each row x (one head of one token):
//   y = x * (mean(x^2) + eps)^(-1/2) * w                     (norm, optional)
//   (y_a, y_b) <- gain * (y_a cos t - y_b sin t, y_b cos t + y_a sin t)
// for the rot/2 pairs (a, b) of the first rot dimensions, t = position * f_i;
// the other dimensions keep y.  Everything is fp32 and rounded once on the
// way out.
//
// Angles: position * f_i is far larger than a turn for far positions, and its
// fp32 product would lose the angle (2^-24 of 10^6 radians is 0.06).  The
// table therefore holds f_i / 2 pi as a 64-bit binary fraction of a turn, whose
// integer product with the position, taken modulo 2^64, is the fraction of a turn
// without a further rounding (the entry has that of its fp64 computation: at
// positions up to 2^27 less than fp32's own, 2^-24); its top 32 bits go to
// sincospif.
//
// Bound: HBM (each row read once, written once).  A group of d * size / 32
// lanes takes a token's heads one after another: a lane holds two 16-byte
// chunks of the row that have both halves of its pairs, so that the rotation
// needs no exchange and the norm only a few shuffles, and its pairs' sines and
// cosines and its weights stay in registers for all of the group's heads.
// (From shared memory for every row, their reads, at four-way bank conflicts,
// bound the kernel: 143 us for 16384 tokens of 40 + 40 heads of 128 in bf16.)
// A group's share of a token is as many heads as leave every SM about eight
// rounds of groups; a single token's heads all go to groups of their own.
// Measured on that prompt: 104.8 us (6.4 TB/s, 94 % of the copy rate) with two
// heads on their way ahead of the one worked on and six CTAs of 128 threads
// per SM (one head ahead: 116-121 us; three, or 256 threads: 107-114).
#include <cstdint>

#include <cuda_bf16.h>

#include "mf_internal.cuh"
#include "mf_ptx.cuh"

namespace mf {
namespace {

constexpr int kThreads = 128;
constexpr int kCtasPerSm = 6;

template <typename T>
struct Vec;  // one 16-byte chunk as floats
template <>
struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& w, float* f) {
    f[0] = bf16lo(w.x), f[1] = bf16hi(w.x), f[2] = bf16lo(w.y), f[3] = bf16hi(w.y);
    f[4] = bf16lo(w.z), f[5] = bf16hi(w.z), f[6] = bf16lo(w.w), f[7] = bf16hi(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
  static __device__ __forceinline__ float load(const __nv_bfloat16* p) { return __bfloat162float(*p); }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& w, float* f) {
    f[0] = __uint_as_float(w.x), f[1] = __uint_as_float(w.y);
    f[2] = __uint_as_float(w.z), f[3] = __uint_as_float(w.w);
  }
  static __device__ __forceinline__ uint4 pack(const float* f) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                      __float_as_uint(f[3]));
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
};

// How a lane's two chunks map to dimensions.
enum { kHalf = 0, kPairs = 1, kHalfOdd = 2 };
// kHalf: chunks c and c + rot/2/N of the rotated part (needs rot/2 % N == 0),
//   then consecutive chunks of the rest
// kPairs: two consecutive chunks, pairs inside a chunk
// kHalfOdd: two consecutive chunks; a pair's other element is read from
//   global memory again (rot/2 not a multiple of a chunk)

template <typename T, int D, int LAYOUT>
__global__ void __launch_bounds__(kThreads, LAYOUT == kHalfOdd ? 2 : kCtasPerSm) rope_kernel(const RopeParams p) {
  constexpr int N = Vec<T>::N;
  constexpr int LPR = D / (2 * N);       // lanes per group
  constexpr int kGroups = kThreads / LPR;
  const int half = p.rot >> 1;
  const int l = threadIdx.x % LPR;
  const long long unit = static_cast<long long>(blockIdx.x) * kGroups + threadIdx.x / LPR;
  // (a group past the end works on the last unit and stores nothing, so that
  // every lane joins the shuffles)
  const bool here = unit < p.n_units;
  const long long u = here ? unit : p.n_units - 1;
  const int chunks = p.q_chunks + p.k_chunks;
  const long long tok = u / chunks;
  int c = static_cast<int>(u - tok * chunks);
  const bool is_q = c < p.q_chunks;
  if (!is_q) c -= p.q_chunks;
  const int h_begin = c * p.heads_per_unit;
  const int n = here ? min(p.heads_per_unit, (is_q ? p.H_q : p.H_k) - h_begin) : 0;
  const long long at = static_cast<long long>(h_begin) * D;
  const T* src = is_q ? static_cast<const T*>(p.q) + tok * p.ld_q + at : static_cast<const T*>(p.k) + tok * p.ld_k + at;
  T* dst = is_q ? static_cast<T*>(p.q_out) + tok * p.ld_qo + at : static_cast<T*>(p.k_out) + tok * p.ld_ko + at;

  const int hc = half / N;  // kHalf: chunks of half the rotated part
  const bool turned = LAYOUT != kHalf || l < hc;  // kHalf: whether this lane's chunks are rotated
  const int c0 = LAYOUT == kHalf && turned ? l : 2 * l;  // (2 hc + 2 (l - hc) = 2 l)
  const int c1 = LAYOUT == kHalf && turned ? l + hc : 2 * l + 1;
  // the next two heads are on their way while one is worked on
  constexpr int kAhead = 2;
  uint4 wa[kAhead], wb[kAhead];
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    wa[j] = wb[j] = make_uint4(0u, 0u, 0u, 0u);
    if (j < n) {
      wa[j] = *reinterpret_cast<const uint4*>(src + j * D + c0 * N);
      wb[j] = *reinterpret_cast<const uint4*>(src + j * D + c1 * N);
    }
  }

  // sines and cosines of this lane's pairs
  const long long pos = p.positions[tok];
  auto turn_of = [&](int f, float& cn, float& sn) {
    const unsigned long long turn = static_cast<unsigned long long>(pos) * p.freq[f];
    // top 32 bits as a signed fraction of a turn; sincospif takes half turns
    sincospif(static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f, &sn, &cn);  // 2^-31
    cn *= p.gain;
    sn *= p.gain;
  };
  constexpr int kTurns = LAYOUT == kHalfOdd ? 2 * N : N;
  float cs[kTurns], sn[kTurns];
#pragma unroll
  for (int e = 0; e < kTurns; ++e) {
    int f;  // the pair
    if (LAYOUT == kHalf) {
      f = turned ? c0 * N + e : -1;
    } else if (LAYOUT == kPairs) {
      f = e < N / 2 ? c0 * (N / 2) + e : c1 * (N / 2) + e - N / 2;
      if (f >= half) f = -1;
    } else {
      const int d = e < N ? c0 * N + e : c1 * N + e - N;
      f = d < half ? d : d < p.rot ? d - half : -1;
    }
    cs[e] = 1.f;
    sn[e] = 0.f;
    if (f >= 0) turn_of(f, cs[e], sn[e]);
  }
  float ga[N], gb[N];  // weights
#pragma unroll
  for (int e = 0; e < N; ++e) ga[e] = gb[e] = 1.f;
  if (p.norm) {
    const T* w = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
    if (w) {
      Vec<T>::unpack(*reinterpret_cast<const uint4*>(w + c0 * N), ga);
      Vec<T>::unpack(*reinterpret_cast<const uint4*>(w + c1 * N), gb);
    }
  }

  for (int i0 = 0; i0 < p.heads_per_unit; i0 += kAhead)
#pragma unroll
  for (int j = 0; j < kAhead; ++j) {
    const int i = i0 + j;
    float a[N], b[N];
    Vec<T>::unpack(wa[j], a);
    Vec<T>::unpack(wb[j], b);
    const bool live = i < n;
    if (i + kAhead < n) {
      wa[j] = *reinterpret_cast<const uint4*>(src + (i + kAhead) * D + c0 * N);
      wb[j] = *reinterpret_cast<const uint4*>(src + (i + kAhead) * D + c1 * N);
    }
    float oa[N], ob[N];  // kHalfOdd: each element's partner, normed
    if (LAYOUT == kHalfOdd) {
      const T* row = src + i * D;
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int da = c0 * N + e, db = c1 * N + e;
        const int pa = da < half ? da + half : da - half, pb = db < half ? db + half : db - half;
        oa[e] = live && da < p.rot ? Vec<T>::load(row + pa) : 0.f;
        ob[e] = live && db < p.rot ? Vec<T>::load(row + pb) : 0.f;
      }
    }
    if (p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        a[e] *= r * ga[e];
        b[e] *= r * gb[e];
      }
      if (LAYOUT == kHalfOdd) {
        const T* w = static_cast<const T*>(is_q ? p.q_weight : p.k_weight);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int da = c0 * N + e, db = c1 * N + e;
          const int pa = da < half ? da + half : da - half, pb = db < half ? db + half : db - half;
          oa[e] *= r * (w && da < p.rot ? Vec<T>::load(w + pa) : 1.f);
          ob[e] *= r * (w && db < p.rot ? Vec<T>::load(w + pb) : 1.f);
        }
      }
    }
    if (LAYOUT == kHalf) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float x = a[e], y = b[e];
        if (turned) {
          a[e] = x * cs[e] - y * sn[e];
          b[e] = y * cs[e] + x * sn[e];
        }
      }
    } else if (LAYOUT == kPairs) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const float x = a[e], y = a[e + 1], z = b[e], w = b[e + 1];
        const int i0 = e >> 1, i1 = (N + e) >> 1;
        if (2 * (c0 * (N / 2) + i0) < p.rot) {
          a[e] = x * cs[i0] - y * sn[i0];
          a[e + 1] = y * cs[i0] + x * sn[i0];
        }
        if (2 * (c1 * (N / 2) + i0) < p.rot) {
          b[e] = z * cs[i1] - w * sn[i1];
          b[e + 1] = w * cs[i1] + z * sn[i1];
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int da = c0 * N + e, db = c1 * N + e;
        if (da < p.rot) a[e] = a[e] * cs[e] + (da < half ? -oa[e] : oa[e]) * sn[e];
        if (db < p.rot) b[e] = b[e] * cs[N + e] + (db < half ? -ob[e] : ob[e]) * sn[N + e];
      }
      // in place: every lane of the row has read it before any lane writes it
      __syncwarp();
    }
    if (live) {
      *reinterpret_cast<uint4*>(dst + i * D + c0 * N) = Vec<T>::pack(a);
      *reinterpret_cast<uint4*>(dst + i * D + c1 * N) = Vec<T>::pack(b);
    }
  }
}

template <typename T, int D>
cudaError_t launch_t(RopeParams p, long long T_, cudaStream_t s) {
  constexpr int kGroups = kThreads / (D / (2 * Vec<T>::N));
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // heads per group: one while that leaves less than eight rounds of CTAs,
  // else what does; shares of a token as even as they go
  const long long rounds = static_cast<long long>(sms) * kCtasPerSm * kGroups * 8;
  const int most = p.H_q > p.H_k ? p.H_q : p.H_k;
  long long hpu = (T_ * (p.H_q + p.H_k) + rounds - 1) / rounds;
  if (hpu > most) hpu = most;
  const int shares = static_cast<int>((most + hpu - 1) / hpu);
  p.heads_per_unit = (most + shares - 1) / shares;
  p.q_chunks = (p.H_q + p.heads_per_unit - 1) / p.heads_per_unit;
  p.k_chunks = (p.H_k + p.heads_per_unit - 1) / p.heads_per_unit;
  p.n_units = T_ * (p.q_chunks + p.k_chunks);
  const long long grid = (p.n_units + kGroups - 1) / kGroups;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  auto go = [&](auto kern) -> cudaError_t {
    kern<<<static_cast<unsigned>(grid), kThreads, 0, s>>>(p);
    return cudaGetLastError();
  };
  if (p.layout == 1) return go(rope_kernel<T, D, kPairs>);
  if (p.rot / 2 % Vec<T>::N == 0) return go(rope_kernel<T, D, kHalf>);
  return go(rope_kernel<T, D, kHalfOdd>);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, long long T, int f32, int d, cudaStream_t s) {
  if (T <= 0) return cudaSuccess;
  if (f32) return d == 128 ? launch_t<float, 128>(p, T, s) : launch_t<float, 64>(p, T, s);
  return d == 128 ? launch_t<__nv_bfloat16, 128>(p, T, s) : launch_t<__nv_bfloat16, 64>(p, T, s);
}

}  // namespace mf
