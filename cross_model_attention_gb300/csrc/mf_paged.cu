// mf_paged.cu — decoding attention over a paged cache held in 4 bits
// (mf_attn_paged), sm_103a.
//
// For new token t of a request with len keys, at position i = len - Lq + t, over
// the keys j <= i with i - j < window or j < sinks:
//   s_j = scale q.k_j,  cap tanh(s_j / cap) where scores are capped,
//   less slope (i - j) where there is a bias by distance,
//   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  lse = m + log(sum_j exp(s_j - m)).
//
// What bounds it: a key and a value of one head are 9 d / 8 bytes (144 at d =
// 128), which an SM's share of memory brings every 6 cycles, but 2 d numbers that
// have to become operands of a matrix product.  They do so in registers: a warp
// takes 16 keys at a time as the A operand of 16 x 8 x 16 products, K against q
// and V (transposed) against the weights, whose rows are few in decoding (8 to a
// product, the query heads of a KV head and its new tokens).  Through shared
// memory, as tcgen05 takes its operands, the 512 bytes of a key and value
// unpacked to fp16 would be written once and read once: 8 cycles at 128 bytes a
// cycle, more than memory needs to bring them.
//
// An e2m1 code times its e4m3 scale is exact in fp16, so K and V meet the
// products as they are held; q goes there scaled by a power of two per row (its
// bf16 values then are exact in fp16 within 2^-32 of the row's largest), weights
// scaled by 2^7 (off by 2^-11, or 2^-32 of the row's largest).  Sums, the
// softmax's statistics and o are fp32.
//
// One pass over the keys: a row's reference m moves (and o and the sum are
// rescaled) only where a score exceeds it by 2^8.
//
// Work: tiles of 32 or 64 keys of all (request, head) pairs laid end to end, cut
// into equal spans, one per warp; a warp has a ring of tiles of its own in shared
// memory, filled by cp.async, and waits for no other warp until the end.  Pieces
// of a pair that warps of a CTA share are joined in shared memory, those that
// CTAs share through the workspace, by a second kernel; both in a fixed order.
//
// Measured in back-to-back graph replays, 32 requests, 32q/8kv heads of 128: 35 us
// over 4096 keys each, 106 over 16384, 200 over 32768: 6.4 TB/s (95 % of the copy
// rate) from key to key, and 12 us besides, for the lengths and the table (4), the
// first tiles (3), joining in the CTA (2) and the second kernel (3).  From 9 rows on
// the instructions of 12 warps are the bound: 142 us over 16384 keys with 9 to 16
// rows, as much again for every further 16.  So they are with heads of 64, whose keys
// have half the bytes but the same softmax (69 us over 16384 keys, 4.4 TB/s), with
// capped scores (124 us) and a bias by distance (113).
#include <algorithm>
#include <cmath>
#include <cstdint>
#include <mutex>
#include <type_traits>

#include <cuda_bf16.h>

#include "mf_fp4.cuh"
#include "mf_internal.cuh"
#include "mf_ptx.cuh"

namespace mf {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kRingBytes = 221184;   // of a CTA
constexpr int kCost = 1;             // a pair's start and end, in tiles
constexpr int kMinSpan = 4;          // least work of a CTA, in tiles (8 requests of 300 keys 9.1 us, with 2 10.2; one of 1000 8.6, 8.9)
constexpr int kLensHere = 900;       // requests whose lengths are kept in shared memory
constexpr float kLift = 7.f;         // weights are held times 2^7
constexpr float kNoRef = 1e30f;      // kLift less the reference of a row that has seen no key
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// D dimensions, NT times 8 rows to a unit of work.  Measured with 32 requests of
// 16384 keys (and 200 of up to 2000): heads of 128 with one to 8 rows take 105 us (56)
// with 12 warps and tiles of 64 keys, 105 (59) with 16 and 32 (12 and 32 reach 5.5 TB/s
// from key to key, not 6.4); heads of 64 69 us with 16 and 64, 72 with 12 and 128, 74
// with 24 and 32.  More rows leave registers and a ring for 12 warps; tiles of 64 do not
// fit it twice with heads of 128.
template <int D, int NT>
struct Cfg {
  static constexpr int W = NT == 1 && D == 64 ? 16 : 12;   // warps
  static constexpr int NB = NT > 1 && D == 128 ? 2 : 4;  // 16-key blocks of a tile
  static constexpr int TK = NB * 16;
  static constexpr int kPiece = fp4_piece(D);
  static constexpr int kStage = NB * kPiece;
  static constexpr bool kQShared = NT > 1;               // q's operands in shared memory, not in registers
  static constexpr int kQBytes = kQShared ? D / 16 * NT * 256 : 0;  // of a warp
  static constexpr int kRing = (kRingBytes / W - kQBytes) & ~15;
  static constexpr int S = kRing / kStage;
  static constexpr int R = 8 * NT;
  static constexpr int kThreads = 32 * W;
  static constexpr int kQueue = S < 4 ? 4 : 8;           // parts of a warp: one in work, those in the ring, the next
  static constexpr int kQ = W * kRing;
  static constexpr int kPrefix = kQ + W * kQBytes;       // [threads + 4] int
  static constexpr int kSums = kPrefix + 4 * (kThreads + 4);  // [16] int
  static constexpr int kLens = kSums + 64;               // [kLensHere]
  static constexpr int kParts = kLens + 4 * kLensHere;
  static constexpr int kPieces = kParts + 32 * W * kQueue;
  static constexpr int kWalk = kPieces + 16 * 2 * W;
  static constexpr int kRows = kWalk + 48 * W;           // [R] slope and position of each row
  static constexpr int kBytes = kRows + 8 * R * W;
  static_assert(kBytes <= 232448, "shared memory");
  static_assert(R * D * 4 + R * 8 <= kRing, "a partial result in a warp's ring");
  static_assert(S >= 2 && S + 1 <= kQueue && 32 % NB == 0 && S * NB <= 32, "ring");
};

// A part of a warp's span: tiles i0 .. i1 of a unit.
struct alignas(16) Part {
  int r, u, len, i0, i1, flags, ta, tb;  // flags: and from bit 8 on the last CTA with tiles of the unit
};
enum { kBegins = 1, kEnds = 2, kHere = 4 };
// Where a warp's walk over its span is: the unit whose line begins at `at`.
struct alignas(16) Walk {
  int r, u, at, f0, f1, len, ta, tb, nt, pad[3];
};
// A partial result of a warp.
struct alignas(16) Piece {
  int r, u, flags, end;  // end: the last CTA with tiles of the unit
};

__device__ __forceinline__ void cp16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// D (16 x 8, fp32) += A (16 x 16) B (16 x 8), fp16.
__device__ __forceinline__ void mma(float* c, uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %2, %1;" : "=r"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// tanh: by its series below 0.3, above by the exponential, 1 - 2 / (1 + e^2a); off
// by 2^-20 of it.  (With tanhf 32 requests of 16384 keys with capped scores took 158
// us, with this 138, and 121 where a tile's are taken together; two by two in packed
// arithmetic 2 more.)
__device__ __forceinline__ float tanh_of(float x) {
  const float a = fabsf(x), q = x * x;
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + ex2(2.f * kLog2e * a)));
  const float far = copysignf(fmaf(-2.f, r, 1.f), x);
  const float near = x * fmaf(q, fmaf(q, fmaf(q, fmaf(q, 62.f / 2835.f, -17.f / 315.f), 2.f / 15.f), -1.f / 3.f), 1.f);
  return a < 0.3f ? near : far;
}
// Bits of x where m has ones, of y elsewhere.
__device__ __forceinline__ uint32_t select(uint32_t m, uint32_t x, uint32_t y) { return (m & x) | (~m & y); }

// The tiles of a request: [0, ta) and [tb, tb + nt - ta) of its keys.
struct Tiles {
  int len, ta, tb, nt;
};
template <int TK>
__device__ __forceinline__ Tiles tiles_of(const PagedParams& p, int len) {
  Tiles t;
  t.len = min(max(len, 0), p.max_pages * p.ps);
  const int b0 = max(0, t.len - p.Lq - p.window + 1);
  t.tb = b0 / TK;
  t.ta = min(t.tb, (min(p.n_sink, t.len) + TK - 1) / TK);
  t.nt = t.ta + (t.len + TK - 1) / TK - t.tb;
  return t;
}
// The line of one of a request's units.
__device__ __forceinline__ int line_of(const Tiles& t) { return t.nt > 0 ? kCost + t.nt : 0; }

// Where row `row` of unit u of request r is in q and o, its head; false past the last row.
struct Row {
  long long tok;
  int head;
};
__device__ __forceinline__ bool row_of(const PagedParams& p, int r, int u, int row, int R, Row& x) {
  const int rg = p.Lq * p.G <= R ? 0 : u / p.H_kv, h = u - rg * p.H_kv, rr = rg * R + row;
  const int t = static_cast<int>(static_cast<unsigned>(rr) * p.inv_G >> 16);
  x.head = h * p.G + rr - t * p.G;
  x.tok = static_cast<long long>(r) * p.Lq + t;
  return rr < p.Lq * p.G;
}
// Of a reference (in base 2, less kLift) and a sum of weights beside it.
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2; }
// A piece's weight beside others under the common reference M.
__device__ __forceinline__ float weight_of(float m, float l, float M) {
  return m == -INFINITY ? (l == 0.f ? 0.f : 1.f) : ex2(m - M);  // (a sum without a reference is NaN)
}

// A warp's D / 32 values of a joined row.
template <int D>
__device__ __forceinline__ void store_row(const PagedParams& p, int r, int u, int row, int R, float M, float L, const float* acc) {
  Row x;
  if (!row_of(p, r, u, row, R, x)) return;
  const int lane = threadIdx.x & 31;
  const float inv = L == 0.f ? 0.f : 1.f / L;
  __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + x.tok * p.ld_o + x.head * D + lane * (D / 32);
  uint32_t w[D / 64];
#pragma unroll
  for (int i = 0; i < D / 64; ++i) w[i] = L == 0.f ? 0u : pack_bf16x2(acc[2 * i] * inv, acc[2 * i + 1] * inv);
  if (D == 128) *reinterpret_cast<uint2*>(o) = make_uint2(w[0], w[D / 64 - 1]);
  else *reinterpret_cast<uint32_t*>(o) = w[0];
  if (p.lse && lane == 0) p.lse[x.tok * (p.H_kv * p.G) + x.head] = lse_of(M, L);
}

// SPECIAL: scores are capped or there is a bias by distance.  (In one kernel with the
// rest 9 to 16 rows over 16384 keys took 148 us, not 143, and one to 8 rows 108.6.)
template <int D, int NT, bool SPECIAL>
__global__ void __launch_bounds__(Cfg<D, NT>::kThreads, 1) paged_kernel(const PagedParams p) {
  using C = Cfg<D, NT>;
  constexpr int W = C::W, NB = C::NB, TK = C::TK, S = C::S, T = C::kThreads;
  extern __shared__ __align__(16) uint8_t smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  int* prefix = reinterpret_cast<int*>(smem + C::kPrefix);
  int* lens_s = reinterpret_cast<int*>(smem + C::kLens);
  Part* parts = reinterpret_cast<Part*>(smem + C::kParts) + warp * C::kQueue;
  Piece* pieces = reinterpret_cast<Piece*>(smem + C::kPieces);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // what comes after may be set up
  // What came before may still run.  Meanwhile q, the lengths and the table come
  // as far as L2, which has the newest of what is still being written: a line to a
  // thread.  (32 requests with a window of 4096 keys 33.6 us, without this 34.1.)
  {
    const long long x = static_cast<long long>(threadIdx.x) * gridDim.x + blockIdx.x;
    auto ask = [&](const void* base, long long rows, long long ld, unsigned lines) {
      if (x >= rows * lines) return;
      const unsigned y = static_cast<unsigned>(x) / lines;
      asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(base) + y * ld + (static_cast<unsigned>(x) - y * lines) * 128u));
    };
    ask(p.q, static_cast<long long>(p.n) * p.Lq, p.ld_q * 2, p.H_kv * p.G * D / 64);
    ask(p.lens, 1, 0, (p.n + 31) / 32);
    ask(p.table, p.n, p.ld_table * 4, (p.max_pages + 31) / 32);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // ---- the lines: a thread sums those of consecutive requests
  const int share = (p.n + T - 1) / T;
  const int groups = (p.Lq * p.G + C::R - 1) / C::R, units = p.H_kv * groups;
  int all;  // the lines of one unit of every request
  {
    int* sums = reinterpret_cast<int*>(smem + C::kSums);
    const int busy = (p.n + 32 * share - 1) / (32 * share);  // warps with a request
    int inc = 0;
    if (warp < busy) {
      for (int j = 0; j < share; ++j) {
        const int r = threadIdx.x * share + j;
        if (r >= p.n) break;
        const int len = p.lens[r];
        if (p.n <= kLensHere) lens_s[r] = len;
        inc += line_of(tiles_of<TK>(p, len));
      }
      __syncwarp();
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(kFull, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) sums[warp] = inc;
    }
    if (lane < 2) pieces[2 * warp + lane].flags = 0;
    __syncthreads();
    const int of_warp = lane < busy ? sums[lane] : 0;
    all = __reduce_add_sync(kFull, of_warp);
    prefix[threadIdx.x + 1] = inc + __reduce_add_sync(kFull, lane < warp ? of_warp : 0);
    if (threadIdx.x == 0) prefix[0] = 0;
    __syncthreads();
  }
  auto len_of = [&](int r) { return p.n <= kLensHere ? lens_s[r] : p.lens[r]; };
  const long long total = static_cast<long long>(all) * units;
  // (rounded up: all spans together are never short)
  const int per = max(kMinSpan, __float2int_ru(__fmul_ru(__ll2float_ru(total), p.inv_grid)));
  // this CTA's span, from here on in places from its start, and this warp's
  const long long cta0 = min(total, static_cast<long long>(per) * blockIdx.x);
  const int cta1 = static_cast<int>(min(total - cta0, static_cast<long long>(per)));
  const int f0 = cta1 / W * warp + cta1 % W * warp / W, f1 = cta1 / W * (warp + 1) + cta1 % W * (warp + 1) / W;

  // ---- the walk over this warp's span
  int wr = p.n, wu = 0, at = 0;  // request and unit of the line that begins at `at`
  Tiles wt{0, 0, 0, 0};
  if (f0 < f1) {
    // the thread whose requests' lines f0 lies in, then the request
    constexpr int kStep = T / 32;
    const long long f = cta0 + f0;
    auto begins = [&](int line) { return static_cast<long long>(line) * units; };
    const int hi = 31 - __clz(__ballot_sync(kFull, begins(prefix[lane * kStep]) <= f));
    const int j = hi * kStep + 31 - __clz(__ballot_sync(kFull, lane < kStep && begins(prefix[hi * kStep + min(lane, kStep - 1)]) <= f));
    int line = prefix[j];
    wr = j;
    if (share > 1) {
      wr = p.n;
      for (int r0 = j * share; r0 < p.n; r0 += 32) {
        const int r = r0 + lane;
        const int mine = line_of(tiles_of<TK>(p, r < p.n ? len_of(r) : 0));
        int inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(kFull, inc, o);
          if (lane >= o) inc += y;
        }
        const unsigned hit = __ballot_sync(kFull, begins(line + inc) > f);
        if (hit) {
          const int k = __ffs(hit) - 1;
          wr = r0 + k;
          line += __shfl_sync(kFull, inc - mine, k);
          break;
        }
        line += __shfl_sync(kFull, inc, 31);
      }
    }
    if (wr < p.n) {
      wt = tiles_of<TK>(p, len_of(wr));
      // (a request's lines may be 2^31 and more long, a unit's are not)
      const long long in = f - begins(line);
      wu = in < 0x7fffffff ? static_cast<int>(in) / (kCost + wt.nt) : static_cast<int>(in / (kCost + wt.nt));
      at = static_cast<int>(begins(line) + static_cast<long long>(wu) * (kCost + wt.nt) - cta0);
    }
  }
  Walk* walk = reinterpret_cast<Walk*>(smem + C::kWalk) + warp;
  if (lane == 0) *walk = Walk{wr, wu, at, f0, f1, wt.len, wt.ta, wt.tb, wt.nt, {0, 0, 0}};
  __syncwarp();
  // The producer's part: tiles i .. i1 of it are to be asked for.  The next one,
  // onto the queue; false after the last.
  int i = 0, i1 = 0, pushed = 0, popped = 0;
  auto next_part = [&]() {
    Walk x = *walk;
    bool some = false;
    while (!some && x.at < x.f1 && x.r < p.n) {
      if (x.u == units) {  // to the next request with keys
        x.u = 0;
        int r0 = x.r + 1;
        x.r = p.n;
        for (; r0 < p.n; r0 += 32) {
          const int r = r0 + lane;
          const unsigned full = __ballot_sync(kFull, r < p.n && tiles_of<TK>(p, len_of(min(r, p.n - 1))).nt > 0);
          if (full) {
            x.r = r0 + __ffs(full) - 1;
            break;
          }
        }
        if (x.r >= p.n) break;
        const Tiles y = tiles_of<TK>(p, len_of(x.r));
        x.len = y.len, x.ta = y.ta, x.tb = y.tb, x.nt = y.nt;
      }
      const int b = x.at + kCost;
      const int lo = max(0, x.f0 - b), hi = min(x.nt, x.f1 - b);
      x.at = b + x.nt;
      const int u = x.u++;
      if (lo < hi) {
        some = true;
        i = lo;
        i1 = hi;
        // (its tiles past this CTA's span are the next CTAs')
        const int end = hi == x.nt ? 0 : static_cast<int>(blockIdx.x + (static_cast<unsigned>(x.at - cta1) + per - 1) / static_cast<unsigned>(per));
        if (lane == 0)
          parts[pushed & (C::kQueue - 1)] = Part{x.r, u, x.len, lo, hi, (lo == 0 ? kBegins : 0) | (hi == x.nt ? kEnds : 0) | end << 8, x.ta, x.tb};
        ++pushed;
      }
    }
    __syncwarp();
    if (lane == 0) *walk = x;
    __syncwarp();
    return some;
  };

  // Row rr of a unit's head: its token and its head within the group.
  auto split = [&](int rr, int& tt, int& gg) {
    tt = static_cast<int>(static_cast<unsigned>(rr) * p.inv_G >> 16);
    gg = rr - tt * p.G;
    return rr < p.Lq * p.G;
  };
  auto head_of = [&](int u, int& rg) {  // (and its group of rows)
    rg = groups == 1 ? 0 : u / p.H_kv;
    return u - rg * p.H_kv;
  };

  // ---- q of a part: loads, then fp16
  constexpr int NQ = C::kQShared ? 1 : NT;
  uint4 qw[NQ][D / 32];
  float kscale = 1.f, vscale = 1.f;
  auto load_rows = [&](int r, int h, int rg, int nt, uint4* w) {
    int tt, gg;
    const bool ok = split(rg * C::R + nt * 8 + g, tt, gg);
    const __nv_bfloat16* src = static_cast<const __nv_bfloat16*>(p.q) + (static_cast<long long>(r) * p.Lq + tt) * p.ld_q +
                               (h * p.G + gg) * D + t * (D / 4);
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      w[c] = make_uint4(0u, 0u, 0u, 0u);
      if (ok) w[c] = reinterpret_cast<const uint4*>(src)[c];
    }
  };
  auto load_q = [&](int r, int u) {
    int rg;
    const int h = head_of(u, rg);
    if (p.k_scale) kscale = p.k_scale[h];
    if (p.v_scale) vscale = p.v_scale[h];
    if (!C::kQShared) {
#pragma unroll
      for (int nt = 0; nt < NQ; ++nt) load_rows(r, h, rg, nt, qw[nt]);
    }
  };

  bool have = next_part();
  if (have) load_q(parts[0].r, parts[0].u);  // (before the first tiles: what is asked for first comes first)

  // The tile that is the n-th of a part.  Under a bias by distance scores rise towards
  // the newest key: from there back the reference stays where the first tile puts it.
  // (32 requests of 16384 keys with slopes 114 us, from the oldest on 126; 9 to 16 rows
  // that are capped too 185 and 218.)
  auto nth = [](const Part& x, int n) { return SPECIAL ? x.i0 + x.i1 - 1 - n : n; };

  int fill = 0;            // the ring's next slot
  unsigned bad = 0;        // of the ring's blocks: those on no page, NB bits to a slot
  long long offs = 0;      // of the lane's block of 32: its bytes' place, or -1
  int at_block = 32;       // the next of them
  const long long hstride = static_cast<long long>(p.ps / kFp4Block) * C::kPiece;
  const uint32_t ring = smem_u32(smem) + warp * C::kRing;
  auto issue = [&]() {
    if (have) {
      if (at_block == 32) {
        at_block = 0;
        const Part& x = parts[(pushed - 1) & (C::kQueue - 1)];
        const int at = i + lane / NB, b = lane % NB;
        const int ii = nth(x, at), tile = ii < x.ta ? ii : x.tb + ii - x.ta;
        const int key = (tile * NB + b) * kFp4Block;
        offs = -1;
        if (at < i1 && key < x.len) {
          const int page = key / p.ps;
          const int id = p.table[x.r * p.ld_table + page];
          int rg;
          const int h = head_of(x.u, rg);
          if (id >= 0 && id < p.n_pages)
            offs = (static_cast<long long>(id) * p.H_kv + h) * hstride + (key - page * p.ps) / kFp4Block * C::kPiece;
        }
      }
      const uint32_t dst = ring + fill * C::kStage + lane * 16;
      unsigned miss = 0;
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const long long off = __shfl_sync(kFull, offs, at_block + b);
        if (off < 0) {
          miss |= 1u << b;
        } else {
          const uint8_t* src = p.pages + off + lane * 16;
#pragma unroll
          for (int c = 0; c < C::kPiece / 16; c += 32)
            if (c + 32 <= C::kPiece / 16 || lane < C::kPiece / 16 - c) cp16(dst + b * C::kPiece + c * 16, src + c * 16);
        }
      }
      bad = (bad & ~(((1u << NB) - 1u) << (fill * NB))) | miss << (fill * NB);
      at_block += NB;
      if (++i == i1) {
        have = next_part();
        at_block = 32;
      }
      if (++fill == S) fill = 0;
    }
    cp_commit();
  };
#pragma unroll 1
  for (int s = 0; s < S - 1; ++s) issue();

  // ---- requests without keys
  for (int r = blockIdx.x + gridDim.x * warp; r < p.n; r += gridDim.x * W) {
    if (tiles_of<TK>(p, len_of(r)).nt > 0) continue;
    const int H = p.H_kv * p.G;
#pragma unroll 1
    for (int x = lane; x < p.Lq * H * (D / 8); x += 32) {
      const int tt = x / (H * (D / 8)), y = x - tt * (H * (D / 8));
      reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.o) + (static_cast<long long>(r) * p.Lq + tt) * p.ld_o)[y] =
          make_uint4(0u, 0u, 0u, 0u);
    }
    if (p.lse)
#pragma unroll 1
      for (int x = lane; x < p.Lq * H; x += 32) p.lse[static_cast<long long>(r) * p.Lq * H + x] = -INFINITY;
  }

  // ---- parts and their tiles
  int slot = 0;
  bool q_here = have || pushed > 0;
  __syncwarp();
#pragma unroll 1
  while (popped != pushed) {
    // (its place in the queue is not used again before it is done)
    const Part& d = parts[popped & (C::kQueue - 1)];
    ++popped;
    if (!q_here) load_q(d.r, d.u);
    q_here = false;
    const float vs = vscale;
    uint32_t qf[NQ][D / 16][2];
    uint2* qs = reinterpret_cast<uint2*>(smem + C::kQ + warp * C::kQBytes) + lane;  // [D / 16][NT][32], where they are shared
    float acc[D / 16][NT][4], lift[NT][2], l[NT][2], coef[NT][2];  // lift: kLift less the reference
    int rg0;
    const int h0 = head_of(d.u, rg0);
    uint4 qn[C::kQShared ? NT : 1][D / 32];
    if (C::kQShared) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) load_rows(d.r, h0, rg0, nt, qn[C::kQShared ? nt : 0]);
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const uint4* w = C::kQShared ? qn[C::kQShared ? nt : 0] : qw[C::kQShared ? 0 : nt];
      uint32_t top = 0;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        const uint32_t v[4] = {w[c].x, w[c].y, w[c].z, w[c].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) top = __vmaxu2(top, v[e] & 0x7fff7fffu);
      }
      top = max(top & 0xffffu, top >> 16);
      top = max(top, __shfl_xor_sync(kFull, top, 1));
      top = max(top, __shfl_xor_sync(kFull, top, 2));
      // 2^e brings the row's largest to [2^14, 2^15)
      const int ex = static_cast<int>(top >> 7);
      const bool fine = ex < 255;
      const int e = top == 0 || !fine ? 0 : min(120, 141 - ex);
      const float up = __int_as_float((e + 127) << 23);
      float c = p.scale * kscale * __int_as_float((127 - e) << 23);
      c *= SPECIAL && p.cap > 0.f ? 1.f / p.cap : kLog2e;
      if (!fine) c = NAN;
#pragma unroll
      for (int k = 0; k < D / 32; ++k) {
        const uint32_t v[4] = {w[k].x, w[k].y, w[k].z, w[k].w};
        uint32_t f[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = pack_f16x2(bf16lo(v[j]) * up, bf16hi(v[j]) * up);
        if (C::kQShared) {
          qs[(2 * k * NT + nt) * 32] = make_uint2(f[0], f[1]);
          qs[((2 * k + 1) * NT + nt) * 32] = make_uint2(f[2], f[3]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) qf[C::kQShared ? 0 : nt][2 * k + (j >> 1)][j & 1] = f[j];
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        coef[nt][j] = __shfl_sync(kFull, c, (2 * t + j) * 4);
        lift[nt][j] = kNoRef;
        l[nt][j] = 0.f;
      }
    }
#pragma unroll
    for (int a = 0; a < D / 16; ++a)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[a][nt][e] = 0.f;

    const int len = d.len, last_tile = d.i1, ta = d.ta, skip = d.tb - d.ta;
    float2* rows_s = reinterpret_cast<float2*>(smem + C::kRows) + warp * C::R;
    if (SPECIAL) {
      __syncwarp();
      if (lane < C::R) {
        int tt, gg;
        const bool is = split(rg0 * C::R + lane, tt, gg);
        rows_s[lane] = make_float2(is && p.slopes ? p.slopes[h0 * p.G + gg] * kLog2e : 0.f, __int_as_float(is ? len - p.Lq + tt : -1));
      }
      __syncwarp();
    }
#pragma unroll 1
    for (int ci = d.i0; ci < last_tile; ++ci) {
      cp_wait<S - 2>();
      __syncwarp();
      issue();
      const uint8_t* st = smem + warp * C::kRing + slot * C::kStage;
      const unsigned gone = bad >> (slot * NB) & ((1u << NB) - 1u);
      if (++slot == S) slot = 0;
      const int ii = nth(d, ci), key0 = (ii < ta ? ii : ii + skip) * TK;
      const bool whole = key0 + TK - 1 <= len - p.Lq && gone == 0 && (len - 1 - key0 < p.window || key0 + TK <= p.n_sink);

      // S = K q^T: rows are keys, columns the unit's rows
      float x[NB][NT][4];
      uint32_t k0[NB][D / 32], k1[NB][D / 32];  // a lane's codes of keys g and g + 8
      uint32_t s0[NB], s1[NB];                  // their scales, one or two
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint8_t* base = st + b * C::kPiece;
        if (D == 128) {
          const uint4 a = *reinterpret_cast<const uint4*>(base + g * 64 + t * 16);
          const uint4 c = *reinterpret_cast<const uint4*>(base + (g + 8) * 64 + t * 16);
          k0[b][0] = a.x, k0[b][1] = a.y, k0[b][D / 32 - 2] = a.z, k0[b][D / 32 - 1] = a.w;
          k1[b][0] = c.x, k1[b][1] = c.y, k1[b][D / 32 - 2] = c.z, k1[b][D / 32 - 1] = c.w;
          s0[b] = e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(base + 16 * D + g * 8 + t * 2));
          s1[b] = e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(base + 16 * D + (g + 8) * 8 + t * 2));
        } else {
          const uint2 a = *reinterpret_cast<const uint2*>(base + g * 32 + t * 8);
          const uint2 c = *reinterpret_cast<const uint2*>(base + (g + 8) * 32 + t * 8);
          k0[b][0] = a.x, k0[b][1] = a.y;
          k1[b][0] = c.x, k1[b][1] = c.y;
          s0[b] = e4m3x2_f16x2(base[16 * D + g * 4 + t]);
          s1[b] = e4m3x2_f16x2(base[16 * D + (g + 8) * 4 + t]);
        }
      }
      // (blocks inside words where q comes from shared memory, which is then read once
      // a tile; words inside blocks where it does not, for fewer registers)
      constexpr int kOuter = C::kQShared ? D / 32 : NB, kInner = C::kQShared ? NB : D / 32;
#pragma unroll
      for (int io = 0; io < kOuter; ++io) {
        uint2 qa[C::kQShared ? NT : 1], qb[C::kQShared ? NT : 1];
        if (C::kQShared) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            qa[C::kQShared ? nt : 0] = qs[(2 * io * NT + nt) * 32];
            qb[C::kQShared ? nt : 0] = qs[((2 * io + 1) * NT + nt) * 32];
          }
        }
#pragma unroll
        for (int ii = 0; ii < kInner; ++ii) {
          const int w = C::kQShared ? io : ii, b = C::kQShared ? ii : io;
          const bool second = D == 128 && w >= 2;  // of the lane's two blocks of 16
          const uint32_t fa = __byte_perm(s0[b], 0, second ? 0x3232 : 0x1010);
          const uint32_t fb = __byte_perm(s1[b], 0, second ? 0x3232 : 0x1010);
          const uint32_t a0 = mul_f16x2(e2m1x2_f16x2<0>(k0[b][w]), fa), a1 = mul_f16x2(e2m1x2_f16x2<0>(k1[b][w]), fb);
          const uint32_t a2 = mul_f16x2(e2m1x2_f16x2<1>(k0[b][w]), fa), a3 = mul_f16x2(e2m1x2_f16x2<1>(k1[b][w]), fb);
          const uint32_t c0 = mul_f16x2(e2m1x2_f16x2<2>(k0[b][w]), fa), c1 = mul_f16x2(e2m1x2_f16x2<2>(k1[b][w]), fb);
          const uint32_t c2 = mul_f16x2(e2m1x2_f16x2<3>(k0[b][w]), fa), c3 = mul_f16x2(e2m1x2_f16x2<3>(k1[b][w]), fb);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const uint2 q0 = C::kQShared ? qa[C::kQShared ? nt : 0] : make_uint2(qf[C::kQShared ? 0 : nt][2 * w][0], qf[C::kQShared ? 0 : nt][2 * w][1]);
            const uint2 q1 = C::kQShared ? qb[C::kQShared ? nt : 0] : make_uint2(qf[C::kQShared ? 0 : nt][2 * w + 1][0], qf[C::kQShared ? 0 : nt][2 * w + 1][1]);
            if (w == 0) x[b][nt][0] = x[b][nt][1] = x[b][nt][2] = x[b][nt][3] = 0.f;
            mma(x[b][nt], a0, a1, a2, a3, q0.x, q0.y);
            mma(x[b][nt], c0, c1, c2, c3, q1.x, q1.y);
          }
        }
      }

      // scores in base 2: x times its factor
      float by[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) by[nt][j] = coef[nt][j];
      if (SPECIAL && p.cap > 0.f) {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[b][nt][e] = tanh_of(x[b][nt][e] * coef[nt][e & 1]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) by[nt][0] = by[nt][1] = p.cap * kLog2e;
      }
      if (SPECIAL && p.slopes) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const float4 two = *reinterpret_cast<const float4*>(rows_s + nt * 8 + 2 * t);
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float slope = k ? two.z : two.x;
            const float bias = slope * static_cast<float>(key0 + g - __float_as_int(k ? two.w : two.y));
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int e = k; e < 4; e += 2)
                x[b][nt][e] = fmaf(x[b][nt][e], by[nt][k], fmaf(slope, static_cast<float>(16 * b + (e & 2) * 4), bias));
            by[nt][k] = 1.f;
          }
        }
      }
      if (!whole) {
        int rg;
        if (!SPECIAL) head_of(d.u, rg);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            int row;
            if (SPECIAL) {
              row = __float_as_int(rows_s[nt * 8 + 2 * t + k].y);
            } else {
              int tt, gg;
              row = split(rg * C::R + nt * 8 + 2 * t + k, tt, gg) ? len - p.Lq + tt : -1;
            }
            const int far0 = row - key0 - g;  // to the lane's first key
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
              for (int e = k; e < 4; e += 2) {
                const int far = far0 - (16 * b + (e & 2) * 4);
                const bool seen = far >= 0 && (far < p.window || row - far < p.n_sink) && !(gone >> b & 1);
                x[b][nt][e] = seen ? x[b][nt][e] * by[nt][k] : -INFINITY;
              }
            by[nt][k] = 1.f;
          }
        }
      }

      // exponents, and the rows' references
      float y[NB][NT][4];
      auto exponents = [&]() {
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[b][nt][e] = fmaf(x[b][nt][e], by[nt][e & 1], lift[nt][e & 1]);
      };
      exponents();
      {
        float top[NT][2];
        bool up = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            top[nt][j] = fmaxf(y[0][nt][j], y[0][nt][2 + j]);
#pragma unroll
            for (int b = 1; b < NB; ++b) top[nt][j] = fmaxf(top[nt][j], fmaxf(y[b][nt][j], y[b][nt][2 + j]));
            up |= top[nt][j] > kLift + 8.f;
          }
        if (__any_sync(kFull, up)) {
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              // (without a reference, kNoRef hides the scores: theirs is to be taken)
              float s = -INFINITY;
#pragma unroll
              for (int b = 0; b < NB; ++b) s = fmaxf(s, fmaxf(x[b][nt][j], x[b][nt][2 + j]) * by[nt][j]);
#pragma unroll
              for (int o = 4; o < 32; o <<= 1) s = fmaxf(s, __shfl_xor_sync(kFull, s, o));
              const float old = lift[nt][j];
              const bool move = s + old > kLift + 8.f;
              if (move) lift[nt][j] = kLift - s;
              const float f = !move ? 1.f : old == kNoRef ? 0.f : ex2(lift[nt][j] - old);
              l[nt][j] *= f;
#pragma unroll
              for (int a = 0; a < D / 16; ++a) {
                acc[a][nt][j] *= f;
                acc[a][nt][2 + j] *= f;
              }
            }
          exponents();
        }
      }
      // weights, and as the B operand: keys by rows
      uint32_t pf[NB][NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          float w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = ex2(y[b][nt][e]);
          l[nt][0] += w[0] + w[2];
          l[nt][1] += w[1] + w[3];
          pf[b][nt][0] = transpose8x8(pack_f16x2(w[0], w[1]));
          pf[b][nt][1] = transpose8x8(pack_f16x2(w[2], w[3]));
        }
      }

      // O^T += V^T P^T: rows are dimensions
#pragma unroll
      for (int b = 0; b < NB; ++b) {
        const uint8_t* base = st + b * C::kPiece;
        constexpr int NW = D / 64;  // words (8 dimensions) of a lane
        uint32_t va[2][NW], vb[2][NW], sc[2];  // keys 2t and 2t + 1 of each half
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          if (D == 128) {
            const uint4 v = *reinterpret_cast<const uint4*>(base + 8 * D + hf * 512 + g * 64 + t * 16);
            va[hf][0] = v.x, va[hf][NW - 1] = v.y;
            vb[hf][0] = v.z, vb[hf][NW - 1] = v.w;
            sc[hf] = e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(base + 17 * D + g * 16 + hf * 8 + t * 2));
          } else {
            const uint8_t* from = base + 8 * D + hf * 256 + (g >> 1) * 64 + t * 16 + (g & 1) * 4;
            va[hf][0] = *reinterpret_cast<const uint32_t*>(from);
            vb[hf][0] = *reinterpret_cast<const uint32_t*>(from + 8);
            sc[hf] = e4m3x2_f16x2(*reinterpret_cast<const uint16_t*>(base + 17 * D + (g >> 1) * 16 + hf * 8 + t * 2));
          }
          if (!whole) {  // what no row sees may be anything
            const int b0 = len - p.Lq - p.window + 1;
            uint32_t keep = 0;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const int key = key0 + 16 * b + 8 * hf + 2 * t + j;
              const bool dead = key >= len || (key < b0 && key >= p.n_sink) || (gone >> b & 1);
              keep |= dead ? 0u : 0xffffu << (16 * j);
            }
            sc[hf] &= keep;
          }
        }
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          // codes of both keys to each dimension: even ones and odd ones
          uint32_t ev[2], od[2];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            ev[hf] = select(0x0f0f0f0fu, va[hf][w], vb[hf][w] << 4);
            od[hf] = select(0x0f0f0f0fu, va[hf][w] >> 4, vb[hf][w]);
          }
          auto four = [&](auto I) {
            constexpr int kI = decltype(I)::value;
            const uint32_t a0 = mul_f16x2(e2m1x2_f16x2<kI>(ev[0]), sc[0]), a1 = mul_f16x2(e2m1x2_f16x2<kI>(od[0]), sc[0]);
            const uint32_t a2 = mul_f16x2(e2m1x2_f16x2<kI>(ev[1]), sc[1]), a3 = mul_f16x2(e2m1x2_f16x2<kI>(od[1]), sc[1]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma(acc[4 * w + kI][nt], a0, a1, a2, a3, pf[b][nt][0], pf[b][nt][1]);
          };
          four(std::integral_constant<int, 0>());
          four(std::integral_constant<int, 1>());
          four(std::integral_constant<int, 2>());
          four(std::integral_constant<int, 3>());
        }
      }
    }

    // ---- the part's end
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) l[nt][j] += __shfl_xor_sync(kFull, l[nt][j], o);
    const bool done = (d.flags & (kBegins | kEnds)) == (kBegins | kEnds);
    const bool more = popped != pushed;
    // a whole unit's rows, or a partial result: in the ring, which is empty
    // then, or in the workspace where the warp goes on
    const long long spot = 2ll * gridDim.x + static_cast<long long>(blockIdx.x) * W + warp;
    float* po = more ? p.part_o + spot * p.rows * D : reinterpret_cast<float*>(smem + warp * C::kRing);
    float2* pm = more ? p.part_ml + spot * p.rows : reinterpret_cast<float2*>(smem + warp * C::kRing + C::R * D * 4);
    int rg;
    const int h = head_of(d.u, rg);
    __syncwarp();
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int row = nt * 8 + 2 * t + j;
        int tt, gg;
        if (!split(rg * C::R + row, tt, gg)) continue;
        const float L = l[nt][j];
        if (done) {
          const float inv = L == 0.f ? 0.f : vs / L;
          const long long tok = static_cast<long long>(d.r) * p.Lq + tt;
          const int head = h * p.G + gg;
          __nv_bfloat16* o = static_cast<__nv_bfloat16*>(p.o) + tok * p.ld_o + head * D + g * (D / 8);
#pragma unroll
          for (int c = 0; c < D / 64; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = L == 0.f ? 0u : pack_bf16x2(acc[4 * c + e][nt][j] * inv, acc[4 * c + e][nt][2 + j] * inv);
            reinterpret_cast<uint4*>(o)[c] = make_uint4(w[0], w[1], w[2], w[3]);
          }
          if (p.lse && g == 0) p.lse[tok * (p.H_kv * p.G) + head] = lse_of(-lift[nt][j], L);
        } else {
          float* to = po + row * D + g * (D / 8);
#pragma unroll
          for (int c = 0; c < D / 32; ++c)
            reinterpret_cast<float4*>(to)[c] = make_float4(acc[2 * c][nt][j] * vs, acc[2 * c][nt][2 + j] * vs,
                                                           acc[2 * c + 1][nt][j] * vs, acc[2 * c + 1][nt][2 + j] * vs);
          if (g == 0) pm[row] = make_float2(lift[nt][j] == kNoRef ? -INFINITY : -lift[nt][j], L);
        }
      }
    if (!done && lane == 0) pieces[2 * warp + (more ? 0 : 1)] = Piece{d.r, d.u, kHere | (d.flags & 0xff), d.flags >> 8};
  }

  // ---- the CTA's pieces: those of one unit follow each other, all but perhaps
  // the last of them in shared memory
  __syncthreads();
  Piece mine{0, 0, 0, 0};
  if (lane < 2 * W) mine = pieces[lane];
  const unsigned present = __ballot_sync(kFull, (mine.flags & kHere) != 0);
  const unsigned lower = present & ((1u << lane) - 1u);
  const int prev = lower ? 31 - __clz(lower) : lane;
  const int prev_r = __shfl_sync(kFull, mine.r, prev), prev_u = __shfl_sync(kFull, mine.u, prev);
  const bool leads = (mine.flags & kHere) && (!lower || prev_r != mine.r || prev_u != mine.u);
  const unsigned leaders = __ballot_sync(kFull, leads);
  // (group, row) by warp; a group's last piece has the CTA's tail
  const int n_groups = __popc(leaders), rank = __popc(leaders & ((1u << lane) - 1u));
  constexpr int E = D / 32;
  auto take = [&](const float* from, float* v) {
    if (D == 128) {
      const float4 x = *reinterpret_cast<const float4*>(from);
      v[0] = x.x, v[1] = x.y, v[E - 2] = x.z, v[E - 1] = x.w;
    } else {
      const float2 x = *reinterpret_cast<const float2*>(from);
      v[0] = x.x, v[1] = x.y;
    }
  };
  // (16 rows four at a time, so that a CTA with many short units has enough loads in
  // flight: 64 rows of 8 requests of 500 to 7500 keys 57.1 us with two, 54.2 with four)
  constexpr int RI = NT == 1 ? 1 : 4;
  const int row_items = (p.rows + RI - 1) / RI;
  for (int item = warp; item < n_groups * row_items; item += W) {
    const int at_group = item / row_items, row0 = (item - at_group * row_items) * RI;
    const int first = __ffs(__ballot_sync(kFull, leads && rank == at_group)) - 1;
    const unsigned after = leaders & ~((2u << first) - 1u);
    const unsigned group = present & ~((1u << first) - 1u) & (after ? (1u << (__ffs(after) - 1)) - 1u : kFull);
    const int last = 31 - __clz(group);
    const Piece a = pieces[first], z = pieces[last];
    const bool begins = a.flags & kBegins, ends = z.flags & kEnds;
    const bool far = !(last & 1);  // the last piece is in the workspace
    const int w0 = first >> 1, w1 = (last >> 1) + (far ? 0 : 1);  // warps with a piece in shared memory
    // (rows past the last are the last again, and not stored)
    int row[RI];
    float out[RI][E], add[RI][E], M[RI], L[RI];
    float2 ml_far[RI];
    const long long spot_far = 2ll * gridDim.x + static_cast<long long>(blockIdx.x) * W + (last >> 1);
#pragma unroll
    for (int x = 0; x < RI; ++x) {
      row[x] = min(row0 + x, p.rows - 1);
      M[x] = -INFINITY;
      L[x] = 0.f;
      ml_far[x] = make_float2(-INFINITY, 0.f);
#pragma unroll
      for (int e = 0; e < E; ++e) out[x][e] = add[x][e] = 0.f;
      if (far) {
        take(p.part_o + (spot_far * p.rows + row[x]) * D + lane * E, add[x]);
        ml_far[x] = p.part_ml[spot_far * p.rows + row[x]];
      }
    }
    // (short spans leave warps without tiles)
    auto ml_of = [&](int w, int x) {
      return group >> (2 * w + 1) & 1 ? reinterpret_cast<const float2*>(smem + w * C::kRing + C::R * D * 4)[row[x]] : make_float2(-INFINITY, 0.f);
    };
    constexpr int kAtOnce = 4 / RI;
    for (int w = w0; w < w1; w += kAtOnce)
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
        for (int x = 0; x < RI; ++x) M[x] = fmaxf(M[x], w + j < w1 ? ml_of(w + j, x).x : -INFINITY);
#pragma unroll
    for (int x = 0; x < RI; ++x) M[x] = fmaxf(M[x], ml_far[x].x);
    for (int w = w0; w < w1; w += kAtOnce) {
      float2 ml[kAtOnce][RI];
      float v[kAtOnce][RI][E];
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
        for (int x = 0; x < RI; ++x) {
          ml[j][x] = make_float2(-INFINITY, 0.f);
#pragma unroll
          for (int e = 0; e < E; ++e) v[j][x][e] = 0.f;
          if (w + j < w1 && (group >> (2 * (w + j) + 1) & 1)) {
            ml[j][x] = ml_of(w + j, x);
            take(reinterpret_cast<const float*>(smem + (w + j) * C::kRing) + row[x] * D + lane * E, v[j][x]);
          }
        }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j)
#pragma unroll
        for (int x = 0; x < RI; ++x) {
          const float f = weight_of(ml[j][x].x, ml[j][x].y, M[x]);
          L[x] = fmaf(f, ml[j][x].y, L[x]);
#pragma unroll
          for (int e = 0; e < E; ++e) out[x][e] = fmaf(f, v[j][x][e], out[x][e]);
        }
    }
#pragma unroll
    for (int x = 0; x < RI; ++x) {
      if (row0 + x >= p.rows) continue;
      if (far) {
        const float f = weight_of(ml_far[x].x, ml_far[x].y, M[x]);
        L[x] = fmaf(f, ml_far[x].y, L[x]);
#pragma unroll
        for (int e = 0; e < E; ++e) out[x][e] = fmaf(f, add[x][e], out[x][e]);
      }
      if (begins && ends) {
        store_row<D>(p, a.r, a.u, row[x], C::R, M[x], L[x], out[x]);
      } else {
        const long long spot = 2ll * blockIdx.x + (begins ? 1 : 0);
        float* to = p.part_o + (spot * p.rows + row[x]) * D + lane * E;
        if (D == 128) *reinterpret_cast<float4*>(to) = make_float4(out[x][0], out[x][1], out[x][E - 2], out[x][E - 1]);
        else *reinterpret_cast<float2*>(to) = make_float2(out[x][0], out[x][1]);
        if (lane == 0) p.part_ml[spot * p.rows + row[x]] = make_float2(M[x], L[x]);
      }
    }
  }
  if (warp == 0) {  // for the join: a unit that begins here and ends in another CTA
    const int last = present ? 31 - __clz(present) : 0, head = leaders ? 31 - __clz(leaders) : 0;
    if (lane == 0) {
      const Piece a = pieces[head], z = pieces[last];
      p.cuts[blockIdx.x] = present && (a.flags & kBegins) && !(z.flags & kEnds) ? make_int4(z.r, z.u, z.end, 0) : make_int4(-1, 0, 0, 0);
    }
  }
}

// The units that several CTAs share: a warp to a row, the results of CTA c's
// last unit and of the following CTAs' first.
template <int D, int NT>
__global__ void __launch_bounds__(32) join_kernel(const PagedParams p) {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x, row = blockIdx.y, lane = threadIdx.x;
  auto spot = [&](int k) { return (k == 0 ? 2ll * c + 1 : 2ll * (c + k)) * p.rows + row; };
  // Two results are asked for before it is known which there are, then 16 or 8 at a
  // time.  (Four, each replaced as it is added: one request of 16000 keys, in 19
  // CTAs to a head, 16.5 us for 13.2; 1000 keys 12.2 for 9.3.)
  constexpr int kAhead = 2, E = D / 32;
  const int4 cut = p.cuts[c];
  float v[kAhead][E];
  float2 ml[kAhead];
  auto take = [&](int k, float* x, float2& m) {
    m = p.part_ml[spot(k)];
    const float* s = p.part_o + spot(k) * D + lane * E;
    if (D == 128) {
      const float4 y = *reinterpret_cast<const float4*>(s);
      x[0] = y.x, x[1] = y.y, x[E - 2] = y.z, x[E - 1] = y.w;
    } else {
      const float2 y = *reinterpret_cast<const float2*>(s);
      x[0] = y.x, x[1] = y.y;
    }
  };
  const int most = gridDim.x - c;
#pragma unroll
  for (int j = 0; j < kAhead; ++j) take(min(j, most - 1), v[j], ml[j]);
  if (cut.x < 0) return;
  const int n = cut.z - c + 1;
  constexpr int kMore = 16 / NT;
  float w[kMore][E];
  float2 wl[kMore];
  auto ask = [&](int k0) {
#pragma unroll
    for (int j = 0; j < kMore; ++j)
      if (k0 + j < n) take(k0 + j, w[j], wl[j]);
  };
  ask(kAhead);
  float M = -INFINITY, L = 0.f;
  for (int k = lane; k < n; k += 32) M = fmaxf(M, p.part_ml[spot(k)].x);
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  float out[E];
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = 0.f;
  auto add = [&](const float2 m, const float* x) {
    const float f = weight_of(m.x, m.y, M);
    L = fmaf(f, m.y, L);
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] = fmaf(f, x[e], out[e]);
  };
#pragma unroll
  for (int j = 0; j < kAhead; ++j)
    if (j < n) add(ml[j], v[j]);
  for (int k0 = kAhead; k0 < n; k0 += kMore) {
    if (k0 > kAhead) ask(k0);
#pragma unroll
    for (int j = 0; j < kMore; ++j)
      if (k0 + j < n) add(wl[j], w[j]);
  }
  store_row<D>(p, cut.x, cut.y, row, 8 * NT, M, L, out);
}

template <int D, int NT, bool SPECIAL>
cudaError_t launch_t(PagedParams p, cudaStream_t s) {
  using C = Cfg<D, NT>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(paged_kernel<D, NT, SPECIAL>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  });
  if (e != cudaSuccess) return e;
  int sms = 0;
  if ((e = sm_count(&sms)) != cudaSuccess) return e;
  p.inv_grid = std::nextafterf(1.f / sms, 1.f);
  if ((e = launch_early(paged_kernel<D, NT, SPECIAL>, dim3(sms), C::kThreads, C::kBytes, s, p)) != cudaSuccess) return e;
  return launch_early(join_kernel<D, NT>, dim3(sms, p.rows), 32, 0, s, p);
}

}  // namespace

// Rows to a unit: 8 where there are no more, else 16 and as many units to a head as
// it takes.  (Units of 32 rows, whose products alone fill 255 registers of 8 warps: 64
// rows over 32 requests of 16384 keys 488 us, not 531; but of 4096 152, not 150, and over
// 8 requests of 4000 keys on average 65, not 53.)
namespace {
int row_tiles(int rows) { return rows <= 8 ? 1 : 2; }
}  // namespace

void paged_shape(int Lq, int G, int sms, int* grid, int* parts, int* rows) {
  const int nt = row_tiles(Lq * G);
  *grid = sms;
  *parts = sms * (2 + (nt == 1 ? std::max(Cfg<128, 1>::W, Cfg<64, 1>::W) : std::max(Cfg<128, 2>::W, Cfg<64, 2>::W)));
  *rows = Lq * G < 8 * nt ? Lq * G : 8 * nt;
}

cudaError_t launch_paged(const PagedParams& p, int d, cudaStream_t s) {
  if (p.n <= 0) return cudaSuccess;
  // a call's two launches follow each other, so that calls of several threads on one stream may share a workspace
  static std::mutex mutex;
  const std::lock_guard<std::mutex> lock(mutex);
  auto launch = [&](auto special) {
    constexpr bool kSpecial = decltype(special)::value;
    if (row_tiles(p.Lq * p.G) == 1) return d == 128 ? launch_t<128, 1, kSpecial>(p, s) : launch_t<64, 1, kSpecial>(p, s);
    return d == 128 ? launch_t<128, 2, kSpecial>(p, s) : launch_t<64, 2, kSpecial>(p, s);
  };
  return p.cap > 0.f || p.slopes ? launch(std::true_type()) : launch(std::false_type());
}

}  // namespace mf
