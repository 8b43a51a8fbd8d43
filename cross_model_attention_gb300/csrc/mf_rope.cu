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
// table therefore holds f_i / 2 pi as a 64-bit binary fraction of a turn, so
// the integer product with the position, taken modulo 2^64, IS the exact
// fraction of a turn; its top 32 bits go to sincospif.
//
// Bound: HBM (each row read once, written once).  A lane takes two 16-byte
// chunks of a row that hold both halves of its pairs, so the rotation needs
// no exchange and the norm only log2(lanes per row) shuffles.  A CTA walks a
// run of consecutive (token, head) rows and computes the sines and cosines of
// its few tokens once, in shared memory, for all of their heads.
#include <cstdint>

#include <cuda_bf16.h>

#include "mf_internal.cuh"
#include "mf_ptx.cuh"

namespace mf {
namespace {

constexpr int kThreads = 256;

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
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  constexpr int N = Vec<T>::N;
  constexpr int LPR = D / (2 * N);       // lanes per row
  constexpr int kRowsPerPass = kThreads / LPR;
  extern __shared__ float smem[];        // [2][D] weights, then [span][rot/2] (cos, sin)
  float* wsm = smem;
  float2* cs = reinterpret_cast<float2*>(smem + 2 * D);
  const int half = p.rot >> 1;
  const int H = p.H_q + p.H_k;
  const long long row0 = static_cast<long long>(blockIdx.x) * p.rows_per_cta;
  const long long row_end = min(row0 + p.rows_per_cta, p.n_rows);
  const int t0 = static_cast<int>(row0 / H);
  const int h0 = static_cast<int>(row0 - static_cast<long long>(t0) * H);
  const int n_here = static_cast<int>(row_end - row0);
  const int span = (h0 + n_here - 1) / H + 1;

  if (p.norm) {
    for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
      const T* w = static_cast<const T*>(i < D ? p.q_weight : p.k_weight);
      wsm[i] = w ? Vec<T>::load(w + (i < D ? i : i - D)) : 1.f;
    }
  }
  for (int i = threadIdx.x; i < span * half; i += kThreads) {
    const int t = i / half, f = i - t * half;
    const unsigned long long turn =
        static_cast<unsigned long long>(static_cast<long long>(p.positions[t0 + t])) * p.freq[f];
    // top 32 bits as a signed fraction of a turn; sincospif takes half turns
    const float x = static_cast<float>(static_cast<int>(turn >> 32)) * 4.656612873077393e-10f;  // 2^-31
    float sn, cn;
    sincospif(x, &sn, &cn);
    cs[i] = make_float2(cn * p.gain, sn * p.gain);
  }
  __syncthreads();

  const int lane_row = threadIdx.x / LPR, l = threadIdx.x % LPR;
  const int hc = half / N;  // kHalf: chunks of half the rotated part
  int c0, c1;
  bool turned = true;       // kHalf: whether this lane's chunks are rotated
  if (LAYOUT == kHalf) {
    turned = l < hc;
    c0 = turned ? l : 2 * l;              // 2 hc + 2 (l - hc) = 2 l
    c1 = turned ? l + hc : 2 * l + 1;
  } else {
    c0 = 2 * l;
    c1 = 2 * l + 1;
  }
  // Lanes of one row are in one warp; a row past the end is computed on the
  // last row's data and not stored, so that every lane joins the shuffles.
  for (int base = 0; base < n_here; base += kRowsPerPass) {
    const int i = base + lane_row;
    const bool live = i < n_here;
    const int j = h0 + (live ? i : n_here - 1);
    const int tt = j / H, h = j - tt * H;
    const bool is_q = h < p.H_q;
    const long long tok = t0 + tt;
    const T* src = is_q ? static_cast<const T*>(p.q) + tok * p.ld_q + static_cast<long long>(h) * D
                        : static_cast<const T*>(p.k) + tok * p.ld_k + static_cast<long long>(h - p.H_q) * D;
    T* dst = is_q ? static_cast<T*>(p.q_out) + tok * p.ld_qo + static_cast<long long>(h) * D
                  : static_cast<T*>(p.k_out) + tok * p.ld_ko + static_cast<long long>(h - p.H_q) * D;
    float a[N], b[N];
    Vec<T>::unpack(*reinterpret_cast<const uint4*>(src + c0 * N), a);
    Vec<T>::unpack(*reinterpret_cast<const uint4*>(src + c1 * N), b);
    float oa[N], ob[N];  // kHalfOdd: each element's partner
    if (LAYOUT == kHalfOdd) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int da = c0 * N + e, db = c1 * N + e;
        oa[e] = da < p.rot ? Vec<T>::load(src + (da < half ? da + half : da - half)) : 0.f;
        ob[e] = db < p.rot ? Vec<T>::load(src + (db < half ? db + half : db - half)) : 0.f;
      }
    }
    if (p.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < N; ++e) ss = fmaf(a[e], a[e], fmaf(b[e], b[e], ss));
#pragma unroll
      for (int off = LPR / 2; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
      const float* w = wsm + (is_q ? 0 : D);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        a[e] *= r * w[c0 * N + e];
        b[e] *= r * w[c1 * N + e];
      }
      if (LAYOUT == kHalfOdd) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const int da = c0 * N + e, db = c1 * N + e;
          if (da < p.rot) oa[e] *= r * w[da < half ? da + half : da - half];
          if (db < p.rot) ob[e] *= r * w[db < half ? db + half : db - half];
        }
      }
    }
    const float2* ct = cs + tt * half;
    if (LAYOUT == kHalf) {
      if (turned) {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          const float2 c = ct[c0 * N + e];
          const float x = a[e], y = b[e];
          a[e] = x * c.x - y * c.y;
          b[e] = y * c.x + x * c.y;
        }
      }
    } else if (LAYOUT == kPairs) {
#pragma unroll
      for (int e = 0; e < N; e += 2) {
        const int ia = (c0 * N + e) >> 1, ib = (c1 * N + e) >> 1;
        if (ia < half) {
          const float2 c = ct[ia];
          const float x = a[e], y = a[e + 1];
          a[e] = x * c.x - y * c.y;
          a[e + 1] = y * c.x + x * c.y;
        }
        if (ib < half) {
          const float2 c = ct[ib];
          const float x = b[e], y = b[e + 1];
          b[e] = x * c.x - y * c.y;
          b[e + 1] = y * c.x + x * c.y;
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int da = c0 * N + e, db = c1 * N + e;
        if (da < p.rot) {
          const float2 c = ct[da < half ? da : da - half];
          a[e] = a[e] * c.x + (da < half ? -oa[e] : oa[e]) * c.y;
        }
        if (db < p.rot) {
          const float2 c = ct[db < half ? db : db - half];
          b[e] = b[e] * c.x + (db < half ? -ob[e] : ob[e]) * c.y;
        }
      }
    }
    // in place: every lane of the row has read it before any lane writes it
    // (a dead lane re-reads a live row of the same warp or of an earlier one)
    if (LAYOUT == kHalfOdd) __syncwarp();
    if (live) {
      *reinterpret_cast<uint4*>(dst + c0 * N) = Vec<T>::pack(a);
      *reinterpret_cast<uint4*>(dst + c1 * N) = Vec<T>::pack(b);
    }
  }
}

template <typename T, int D>
cudaError_t launch_t(RopeParams p, cudaStream_t s) {
  constexpr int kRowsPerPass = kThreads / (D / (2 * Vec<T>::N));
  const int H = p.H_q + p.H_k;
  int sms = 0;
  cudaError_t e = sm_count(&sms);
  if (e != cudaSuccess) return e;
  // passes per CTA: enough CTAs for eight per SM first, then more rows per
  // CTA so that a token's angles serve more of its heads; several passes only
  // while they span at most 34 tokens, and one pass spans at most 64 (the
  // shared memory for their angles)
  long long passes = p.n_rows / (static_cast<long long>(kRowsPerPass) * sms * 8);
  if (passes > 8) passes = 8;
  if (passes > 32ll * H / kRowsPerPass) passes = 32ll * H / kRowsPerPass;
  if (passes < 1) passes = 1;
  p.rows_per_cta = static_cast<int>(passes) * kRowsPerPass;
  const int half = p.rot / 2;
  const int span = (p.rows_per_cta + H - 2) / H + 1;  // most tokens that rows_per_cta rows touch
  const size_t smem = (2 * D) * sizeof(float) + static_cast<size_t>(span) * half * sizeof(float2);
  const long long grid = (p.n_rows + p.rows_per_cta - 1) / p.rows_per_cta;
  if (grid > 0x7fffffffll) return cudaErrorInvalidValue;
  auto go = [&](auto kern) -> cudaError_t {
    if (smem > 48 * 1024) {
      cudaError_t a = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
      if (a != cudaSuccess) return a;
    }
    kern<<<static_cast<unsigned>(grid), kThreads, smem, s>>>(p);
    return cudaGetLastError();
  };
  if (p.layout == 1) return go(rope_kernel<T, D, kPairs>);
  if (half % Vec<T>::N == 0) return go(rope_kernel<T, D, kHalf>);
  return go(rope_kernel<T, D, kHalfOdd>);
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int f32, int d, cudaStream_t s) {
  if (p.n_rows <= 0) return cudaSuccess;
  if (f32) return d == 128 ? launch_t<float, 128>(p, s) : launch_t<float, 64>(p, s);
  return d == 128 ? launch_t<__nv_bfloat16, 128>(p, s) : launch_t<__nv_bfloat16, 64>(p, s);
}

}  // namespace mf
