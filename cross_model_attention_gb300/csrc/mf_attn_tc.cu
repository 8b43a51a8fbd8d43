// mf_attn_tc.cu — attention with a sliding window, sinks and shared prefixes
// on the fifth-generation tensor cores, bf16, sm_103a.
//
// For a query row at position i of its sequence, over the keys j it sees
// (j <= i, and i - j < window or j < sinks):
//   o = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),  s_j = scale q.k_j,
//   lse = m + log(sum_j exp(s_j - m)).
// The softmax runs in one pass over the keys: m is a running reference, moved
// (and o, the sum rescaled) only when a block's maximum exceeds it by 2^8, so
// that exp2 arguments stay below 8 and the rescaling is rare.  Sums and o are
// fp32; P is rounded to bf16 for the second product (at most 2^-8 of each
// weight, the same size as the rounding of the output): the tensor cores take
// both its operands in one type, and V is bf16.
//
// Rows of a tile: (token, query head of one KV group), TQ = 128 / G tokens of
// all G heads, so that the heads of a group share every key that is read.
// A CTA (one per SM, persistent) runs two streams, each 128 rows with its own
// softmax warpgroup and TMEM (S 128 columns in two halves of 64 keys, each
// half's P over it, O d columns).  The halves decouple a stream's softmax from
// its products: while one half is exponentiated, the other's P V and its next
// Q K run.  Pair runs give the streams two neighbouring row tiles that share
// each key block (K and V come through L2 at ~160 GB/s per SM, which one
// 128-row tile would outrun); single-tile runs (few rows, many keys) give
// them alternate key blocks of one tile and two partial results.  While one
// stream's warps exponentiate, the other's products run.
// Warps 0-3 and 4-7: softmax of stream 0 and 1 (thread = row).  Warps 8 and
// 10: the streams' products (one issuing warp for both spent 2.7 us on a
// block pair whose products take 1.3).  Warp 9: TMA loads, K and V blocks of
// 128 keys through one ring.  Warp 11: the planner, which finds the CTA's runs
// and lays them before the others.
//
// What bounds it.  A prompt: the tensor cores in principle; 8192 causal tokens
// of 32q/8kv heads of 128 take 369 us back to back, 1.49 PFLOP/s of the 1.92
// that a large matrix product reaches (the tensor pipes 66 % busy; what is left
// is the chain S -> softmax -> P of the two streams at a time that the registers
// hold, and a run's start and end).  Decoding: memory; 32 requests of up to 4100
// visible keys read 0.47 GB in 85 us, 5.5 TB/s of 6.8 (the kernel alone 80 us;
// four ring stages 90 us, three 107).  A prefix for many rows: both, 200
// requests with two tokens each over 32767 keys and caches of up to 700 in 194
// us, of them about 130 the prefix's products and 50 the caches' loads.
//
// Masked keys: a row's hidden scores are replaced by -inf before anything is
// done with them, and V rows that no row may see (past a range's end, where
// the box still reads) are zeroed in shared memory or left out of the
// product, so what lies there, NaN included, reaches nothing.  A key that some
// row of a tile pair sees is multiplied by all its rows, by weight 0 where it is
// hidden: a value that is not finite makes those NaN too.
#include <cstdint>
#include <type_traits>

#include "mf_internal.cuh"
#include "mf_ptx.cuh"

namespace mf {
namespace {

constexpr int kRows = 128;
constexpr int kKeys = 128;   // keys per block
constexpr int kHalf = 64;    // keys that the softmax takes at a time
constexpr int kThreads = 384;
constexpr int kRunSlots = 4;  // runs that the planner may be ahead

template <int D>
struct Lay {
  static constexpr int kChunk = 128 * 128;           // 128 rows x 64 bf16
  static constexpr int kTile = (D / 64) * kChunk;    // Q tile, K block or V block
  static constexpr int kStages = D == 128 ? 5 : 10;
  static constexpr int kQ = 0;
  static constexpr int kRing = 2 * kTile;
  static constexpr int kBar = kRing + kStages * kTile;
  static constexpr int kMisc = kBar + 8 * (16 + 2 * kStages + 2 * kRunSlots);
  static constexpr int kRuns = kMisc + 32;            // the planner's runs
  static constexpr int kFull = kRuns + 64 * kRunSlots;  // cache form: map of requests with keys
  static constexpr int kBytes = kFull + kAttnSlotBits / 8 + 1024;
};
static_assert(Lay<128>::kBytes <= 232448 && Lay<64>::kBytes <= 232448, "shared memory");

// misc words: [0] TMEM address, [1] abort; from byte 16 on two barriers
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColS = 0, kColO = 256;  // + 128 * stream each

// ------------------------------------------------------------ PTX not in mf_ptx
// D (+)= A[tmem] * B[smem]^T, kind::f16.
__device__ __forceinline__ void tc_mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc,
                                          uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// 32 bytes to a 32-byte aligned address: a lane's whole sector.
__device__ __forceinline__ void st_global_v8(void* ptr, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(ptr), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ int uniform(int x) { return __shfl_sync(0xffffffffu, x, 0); }
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
      "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]),
      "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,"
      "%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Q tile: 64 columns of G heads of one group, of consecutive tokens.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z,
                                            int w, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(bar)
      : "memory");
}

// Waits of a whole, converged warp; false (in every lane) after the time limit
// or where another role has given up.  The roles' loops share the instruction
// caches, so what is rare stays out of them.
__device__ __noinline__ bool warp_wait_on(uint32_t bar, uint32_t parity, int* err, const volatile int* misc) {
  const unsigned long long t0 = globaltimer();
  for (uint32_t it = 1;; ++it) {
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
    if ((it & 63u) == 0) {
      const bool late = globaltimer() - t0 > kWaitLimitNs;
      if (__any_sync(0xffffffffu, late || misc[1] != 0)) {
        if (late) set_error(err, kDevErrTimeout);
        return false;
      }
    }
  }
}

__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity, int* err, const volatile int* misc) {
  if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
  return warp_wait_on(bar, parity, err, misc);
}
// V rows past the block's last key, up to the next multiple of 16, become
// zero: their weights are zero, but what the box read there may be NaN.  By a
// warp; both streams' may do so to a shared block: they write the same.
template <int D>
__device__ __noinline__ void trim(uint8_t* stage, int valid) {
  const int n = (((valid + 15) & ~15) - valid) * 8;
  for (int i = threadIdx.x & 31; i < n * (D / 64); i += 32) {
    const int c = i / n, x = i - c * n;
    *reinterpret_cast<uint4*>(stage + c * Lay<D>::kChunk + valid * 128 + x * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
  fence_async_smem();
  __syncwarp();
}

// -------------------------------------------------------------------- runs --
// What one run of key blocks is, for every role.
struct alignas(16) Run {
  int q_row, n_tok0, n_tok1;  // tokens of the tile(s); n_tok1 = 0: one tile
  int alt;                    // one tile, key blocks alternate between the streams
  int pos;                    // position of the first token
  int k_row0, a1, b0, b1;
  int nb;                     // key blocks of a head
  int blk0, blk1;             // this run's: block j is block j % nb of head j / nb
  int head, heads;            // first KV head, KV heads of the tile
  int kind;                   // kOwn, kPrefix (K and V are the shared ones), kCache, kEnd
  int part;                   // first partial index, or -1
};
enum { kOwn = 0, kPrefix = 1, kCache = 2, kEnd = 3 };
static_assert(sizeof(Run) == 64, "a slot of the planner's");

// Block j of a run: its head (of the tile's), first key and how many count.
__device__ __forceinline__ void block_at(const Run& r, int j, int& hh, int& j0, int& valid) {
  hh = 0;
  if (r.kind == kCache) {
    hh = j / r.nb;
    j -= hh * r.nb;
  }
  const int na = (r.a1 + kKeys - 1) / kKeys;
  const bool in_a = j < na;
  j0 = in_a ? j * kKeys : r.b0 + (j - na) * kKeys;
  valid = min(kKeys, (in_a ? r.a1 : r.b1) - j0);
}

struct NoRuns {
  __device__ NoRuns(const AttnParams&, volatile uint8_t*) {}
  __device__ bool next(Run&) { return false; }
};

// The runs of this CTA in order, packed form: from the plan's table.
struct PackedRuns {
  static constexpr int kUnrollHalves = 1;
  static constexpr bool kPlanned = false;
  const AttnParams& p;
  int i, end;
  AttnSeg nxt;
  __device__ PackedRuns(const AttnParams& p_, volatile uint8_t*) : p(p_) {
    i = p.cta_segs[blockIdx.x];
    end = p.cta_segs[blockIdx.x + 1];
    if (i < end) nxt = p.segs[i];
  }
  __device__ bool next(Run& r) {
    if (i >= end) return false;
    const AttnSeg s = nxt;
    if (++i < end) nxt = p.segs[i];  // in flight while this run is worked on
    r.q_row = s.q_row;
    r.n_tok0 = min(s.n_tok, p.TQ);
    r.n_tok1 = s.n_tok - r.n_tok0;
    r.alt = r.n_tok1 == 0 && s.part >= 0;
    r.pos = s.pos;
    r.k_row0 = s.k_row0;
    r.a1 = s.a1;
    r.b0 = s.b0;
    r.b1 = s.b1;
    r.blk0 = s.blk0;
    r.blk1 = s.blk1;
    r.nb = 0;
    r.head = s.head;
    r.heads = 1;
    r.kind = kOwn;
    r.part = s.part;
    return true;
  }
};

// Cache form.  The prefix's units are (tile pair, KV head); a cache's are
// (request, group of as many KV heads as have their rows in one tile): all
// heads' rows are one Q tile, and a block of head h gives weights to h's rows
// only, so that a run takes a request's heads one after another without
// starting anew.  Each unit is a line: what a run costs to start and end, then
// its blocks.  The prefix's lines laid end to end are cut into equal spans,
// one per CTA, and the caches' lines likewise, so that uneven lengths balance
// and a unit is cut only where a span ends; a block belongs to the span in
// which it begins.  Every second CTA takes its caches' span first: the
// prefix's products and the caches' loads then overlap.  Where a CTA's share
// of both is at most kApart blocks, a second run's start and end can cost more
// than that brings: the spans are then as long as the shares together, and
// prefix and caches meet from the two ends of the CTAs.  32q/8kv heads of 128,
// lengths from 1 to the one named, spans of both together against apart, us:
//   share 3   16 requests of 200 over 4096    17.6 / 21.9
//        11   64 of 512 over 4096             31.8 / 35.2
//        16   64 of 512 over 16384            45.1 / 44.1
//        17   16 of 3000 over 16384           37.2 / 44.2
//        25   128 of 512 over 8192            63.5 / 60.4
//        26   300 of 100 over 4096            67.5 / 60.0
//        34   16 of 6000 over 32768           58.4 / 65.8
//        36   64 of 1500 over 32768           78.3 / 73.1
//        56   300 of 600 over 4096            121 / 104
//       130   200 with two new tokens of 700 over 32768  257 / 239
// Together wins up to about 15 blocks, and where requests are few (16) past 34;
// where they are many, apart wins from about 16 blocks on.  32 lies between: the
// rule takes the slower side of some shares from 16 to 34, by at most 13 % in
// these.
struct Unit {
  int a1, b0, b1, nb;  // key ranges of a request's cache, in blocks
};
__device__ __forceinline__ Unit cache_unit(const AttnParams& p, int len) {
  len = min(max(len, 0), p.cap);
  Unit u;
  u.b1 = len;
  u.b0 = max(0, len - p.Lq - p.window + 1);
  u.a1 = 0;
  if (p.n_sink >= u.b0) u.b0 = 0;
  else u.a1 = p.n_sink;
  u.nb = (u.a1 + kKeys - 1) / kKeys + (u.b1 - u.b0 + kKeys - 1) / kKeys;
  return u;
}
constexpr int kCostPre = kAttnCostPre, kCostCache = kAttnCostCache;  // a run's start and end, in blocks
// the lines of a request's units
__device__ __forceinline__ int cache_line(const AttnParams& p, int nb) {
  return nb > 0 ? p.groups * kCostCache + nb * p.H_kv : 0;
}
constexpr int kApart = 32;
__device__ __forceinline__ int pre_lines(const AttnParams& p) {
  return p.pre_pairs * p.H_kv * (kCostPre + p.pre_blocks);
}
// length of the spans of the prefix's lines or of the caches' (`suffix` long)
__device__ __forceinline__ int span_of(const AttnParams& p, bool pre, int suffix) {
  const int grid = static_cast<int>(gridDim.x), first = pre_lines(p);
  const int both = (first + suffix + grid - 1) / grid;
  const int own = ((pre ? first : suffix) + grid - 1) / grid;
  return max(p.min_span, both <= kApart ? both : own);
}

struct CacheRuns {
  static constexpr int kUnrollHalves = 2;
  static constexpr bool kPlanned = true;
  const AttnParams& p;
  const volatile uint8_t* full;  // bit per 2^slot_shift requests, one where a cache has a unit
  int todo;                      // parts left: 2, 1, 0
  bool pre;                      // the part at hand is the prefix
  int f0, f1, per;               // this CTA's span of it
  int at;                        // start of the unit's line
  int who, head;                 // tile pair or request, (first) KV head
  // all requests' lines, the request in which this CTA's span of them begins
  // and the lines before it
  int suffix, first, before;
  // (by a whole warp)
  __device__ CacheRuns(const AttnParams& p_, volatile uint8_t* full_) : p(p_), full(full_) {
    find(full_);
    todo = 2;
    pre = (blockIdx.x & 1) == 0;
    begin();
  }
  __device__ void find(volatile uint8_t* bits);
  __device__ int pre_line() const { return kCostPre + p.pre_blocks; }
  __device__ void begin() {
    const int total = pre ? pre_lines(p) : suffix;
    per = span_of(p, pre, suffix);
    // (from the other end of the CTAs: two short lists meet late)
    f0 = min(total, per * static_cast<int>(pre ? blockIdx.x : gridDim.x - 1 - blockIdx.x));
    f1 = min(total, f0 + per);
    if (pre) {
      const int unit = f0 / pre_line();
      who = unit / p.H_kv;
      head = unit - who * p.H_kv;
      at = unit * pre_line();
    } else {
      who = first;
      head = 0;
      at = before;
    }
  }
  // to the next request with a key, or (more than 8192 requests) the next group
  // with one: a batch's unused slots cost next to nothing.  (One after another by
  // their lengths, 246 of them between the first three and the last seven of 256
  // requests of 900 keys cost a call 72 us where it takes 18, and 99403 between 597
  // requests of 600 keys 22 ms where it takes 0.26.)
  __device__ void skip_empty() {
    while (who < p.n) {
      const int g = who >> p.slot_shift;
      // (bytes that nobody wrote are those of requests past the last)
      const uint32_t w = reinterpret_cast<const volatile uint32_t*>(full)[g >> 5] >> (g & 31);
      if (w) {
        who = max(who, (g + __ffs(static_cast<int>(w)) - 1) << p.slot_shift);
        return;
      }
      who = ((g | 31) + 1) << p.slot_shift;
    }
  }
  __device__ bool next(Run& o) {
    for (;;) {
      if (at >= f1) {
        if (--todo <= 0) return false;
        pre = !pre;
        begin();
        continue;
      }
      // the unit at `at` (at < f1: a request is there)
      Unit u{};
      if (!pre) u = cache_unit(p, p.lens[min(who, p.n - 1)]);
      const int heads = pre ? 1 : min(p.HG, p.H_kv - head);
      const int nb = pre ? p.pre_blocks : u.nb * heads;
      const int begins = at + (pre ? kCostPre : kCostCache);
      o.blk0 = max(0, f0 - begins);
      o.blk1 = min(nb, f1 - begins);
      const bool some = o.blk0 < o.blk1;
      if (some) {
        o.head = head;
        o.heads = heads;
        int unit;
        if (pre) {
          const int tok0 = who * 2 * p.TQ, n_tok = p.n * p.Lq - tok0;
          o.kind = kPrefix;
          o.q_row = tok0;
          o.n_tok0 = min(n_tok, p.TQ);
          o.n_tok1 = min(n_tok - o.n_tok0, p.TQ);
          o.alt = o.n_tok1 == 0;
          o.pos = kAttnFar;
          o.k_row0 = 0;
          o.a1 = 0;
          o.b0 = 0;
          o.b1 = p.P;
          o.nb = nb;
          unit = who * p.H_kv + head;
        } else {
          o.kind = kCache;
          o.q_row = who * p.Lq;
          o.n_tok0 = p.Lq;
          o.n_tok1 = 0;
          o.alt = 1;
          o.pos = u.b1 - p.Lq;
          o.k_row0 = who * p.cap;
          o.a1 = u.a1;
          o.b0 = u.b0;
          o.b1 = u.b1;
          o.nb = u.nb;
          unit = who * p.groups + head / p.HG;
        }
        // Along the lines neither unit nor span goes down and one of them goes
        // up from run to run, so their sum tells the runs' results apart.
        o.part = 2 * (unit + f0 / per);
        // for the join: block j of the unit is in span (x + j) / y
        if (o.blk1 == nb)
          p.cuts[pre ? unit : p.pre_pairs * p.H_kv + unit] = make_int2(begins, per);
      }
      // the next unit
      if (nb > 0) at = begins + nb;
      head += nb > 0 ? heads : p.H_kv;  // an empty cache has no units
      if (head >= p.H_kv) {
        head = 0;
        ++who;
        if (!pre) skip_empty();
        if (pre ? who >= p.pre_pairs : who >= p.n) at = f1;  // past the last
      }
      if (some) return true;
    }
  }
};

// The length of all requests' lines, and the request in which this CTA's span
// begins with the length before it.  A lane sums the lines of consecutive
// requests, eight lengths asked for at a time, and the lanes' sums tell in whose
// part the span begins.
__device__ __forceinline__ void CacheRuns::find(volatile uint8_t* bits) {
  const int lane = threadIdx.x & 31;
  const int byte = 8 << p.slot_shift;  // requests to a byte of the map; a lane's share is whole bytes
  const int share = max(byte, ((p.n + 31) / 32 + byte - 1) & ~(byte - 1)), mine = lane * share;
  int sum = 0;
  uint32_t bit8 = 0;
#pragma unroll 2
  for (int r = mine; r < min(p.n, mine + share); r += 8) {
    int len[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) len[i] = r + i < p.n ? __ldg(p.lens + r + i) : 0;
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int line = cache_line(p, cache_unit(p, len[i]).nb);
      sum += line;
      m |= line > 0 ? 1u << i : 0u;
    }
    if (p.slot_shift == 0) {
      bits[r >> 3] = static_cast<uint8_t>(m);
    } else {
      bit8 |= (m ? 1u : 0u) << ((r >> p.slot_shift) & 7);
      if (((r + 8) & (byte - 1)) == 0 || r + 8 >= min(p.n, mine + share)) {
        bits[r >> (p.slot_shift + 3)] = static_cast<uint8_t>(bit8);
        bit8 = 0;
      }
    }
  }
  __syncwarp();
  suffix = __reduce_add_sync(0xffffffffu, sum);
  const int f = min(suffix, span_of(p, false, suffix) * static_cast<int>(gridDim.x - 1 - blockIdx.x));
  first = p.n;
  before = suffix;
  if (f >= suffix) return;
  // of 32 values that begin at `run`: the lane whose value f falls in, or -1
  // where all lie before it; run moves to that lane's beginning, or past them
  auto among = [&](int value, int& run) {
    int inc = value;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc += y;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, f < run + inc);
    const int l = hit ? __ffs(static_cast<int>(hit)) - 1 : -1;
    run += hit ? __shfl_sync(0xffffffffu, inc - value, l) : __shfl_sync(0xffffffffu, inc, 31);
    return l;
  };
  int run = 0;
  const int part = among(sum, run) * share;
  for (int r = part; first == p.n; r += 32) {  // (f lies in this part)
    const int at_r = r + lane;
    const bool in = at_r < min(p.n, part + share);
    const int l = among(in ? cache_line(p, cache_unit(p, __ldg(p.lens + at_r)).nb) : 0, run);
    if (l >= 0) {
      first = r + l;
      before = run;
    } else if (r - part >= share) {
      break;  // not reached
    }
  }
}

// ----------------------------------------------------------------- softmax --
// bits [lo, hi) of the 32 columns from c0 on
__device__ __forceinline__ uint32_t span_bits(int lo, int hi, int c0) {
  lo = min(max(lo - c0, 0), 32);
  hi = min(max(hi - c0, 0), 32);
  if (hi <= lo) return 0u;
  const uint32_t upto = hi == 32 ? 0xffffffffu : (1u << hi) - 1u;
  return upto & ~((1u << lo) - 1u);  // lo < 32 here
}

template <int D, typename Runs>
__global__ void __launch_bounds__(kThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tkp,
                const __grid_constant__ CUtensorMap tvp, const __grid_constant__ CUtensorMap tqc,
                const AttnParams p, const bool cached) {
  using L = Lay<D>;
  constexpr int NS = L::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~uintptr_t(1023));
  const uint32_t sb = smem_u32(smem);
  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  volatile int* misc = reinterpret_cast<volatile int*>(smem + L::kMisc);

  auto barQFull = [&](int t) { return sb + L::kBar + 8u * t; };
  auto barQEmpty = [&](int t) { return sb + L::kBar + 16 + 8u * t; };
  auto barS = [&](int s, int h) { return sb + L::kBar + 32 + 8u * (2 * s + h); };
  auto barP = [&](int s, int h) { return sb + L::kBar + 64 + 8u * (2 * s + h); };
  // (a run's last products have barriers of their own: the next run's first S
  // may be there before a softmax warp looks, and it must not miss a phase)
  auto barO = [&](int s, int h) { return sb + L::kBar + 96 + 8u * (2 * s + h); };
  auto barFull = [&](int i) { return sb + L::kBar + 128 + 8u * i; };
  auto barEmpty = [&](int i) { return sb + L::kBar + 128 + 8u * (NS + i); };
  auto barRun = [&](int i) { return sb + L::kBar + 128 + 8u * (2 * NS + i); };
  auto barRunFree = [&](int i) { return sb + L::kBar + 128 + 8u * (2 * NS + kRunSlots + i); };

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");  // the join may be set up
  if (threadIdx.x == 9 * 32) {
    prefetch_tmap(&tk);
    prefetch_tmap(&tv);
    prefetch_tmap(&tq);
    if (cached) {
      prefetch_tmap(&tqc);
      if (p.P > 0) {
        prefetch_tmap(&tkp);
        prefetch_tmap(&tvp);
      }
    }
  }
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(barQFull(t), 1);
      mbar_init(barQEmpty(t), 2);  // both streams' MMA warps
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(barS(i >> 1, i & 1), 1);
      mbar_init(barO(i >> 1, i & 1), 1);
      mbar_init(barP(i >> 1, i & 1), 4);
    }
    for (int i = 0; i < NS; ++i) {
      mbar_init(barFull(i), 1);
      mbar_init(barEmpty(i), 2);
    }
    for (int i = 0; i < kRunSlots; ++i) {
      mbar_init(barRun(i), 1);
      mbar_init(barRunFree(i), 11);  // all other warps
    }
    fence_mbar_init();
    misc[1] = 0;
  }
  if (warp == 8) tmem_alloc(sb + L::kMisc, kTmemCols);
  // rows of the Q tiles that no load fills (G does not divide 128)
  {
    const int filled = p.G * p.TQ, spare = (kRows - filled) * 8;
    for (int i = threadIdx.x; i < spare * 2 * (D / 64); i += kThreads)
      *reinterpret_cast<uint4*>(smem + L::kQ + (i / spare) * L::kChunk + filled * 128 + (i % spare) * 16) =
          make_uint4(0u, 0u, 0u, 0u);
    fence_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = static_cast<uint32_t>(uniform(misc[0]));
  // The CTA's runs.  The packed form's come from a table and each warp reads
  // them for itself, from addresses that the compiler knows to be the same in
  // all lanes (through the planner a causal 8192-token prompt takes 450 us, not
  // 369); the cache form's are worked out by the planner, which is ahead of the
  // others (each warp for itself: a 4096-key window for 32 requests 88 us, not
  // 86, 1024 requests of 200 keys 5 us more).
  Run r{};
  using Own = typename std::conditional<Runs::kPlanned, NoRuns, Runs>::type;
  Own own(p, nullptr);
  int run_slot = 0;
  uint32_t run_ph = 0;
  // The next run, for a warp or (one) its first lane alone; false after the last
  // or when something has given up.
  auto next_run = [&](auto one) {
    if (!Runs::kPlanned) return own.next(r);
    if (one.value) {
      if (misc[1] || !mbar_wait(barRun(run_slot), run_ph, p.err)) return false;
    } else {
      if (!warp_wait(barRun(run_slot), run_ph, p.err, misc)) return false;
    }
    r = *reinterpret_cast<const Run*>(smem + L::kRuns + 64 * run_slot);
    if (!one.value) __syncwarp();
    if (lane == 0) mbar_arrive(barRunFree(run_slot));
    if (++run_slot == kRunSlots) {
      run_slot = 0;
      run_ph ^= 1;
    }
    return r.kind != kEnd;
  };
  // Who waits for the ring.  A barrier's phase is told from the one before it
  // only, so no use of a stage may pass unseen: both streams' MMA warps see
  // every use in turn, the other stream's too, and a stage is free when both
  // have said so.

  if (warp == 9) {
    // ------------------------------------------------------------- loader
    if (lane == 0) {
      int g = 0, nq0 = 0, nq1 = 0, slot = 0;  // ring uses, uses of the Q slots, next slot
      bool ok = true;
      auto load = [&](const CUtensorMap* map, int i) {
        const int st = g % NS;
        int hh, j0, valid;
        block_at(r, r.blk0 + i, hh, j0, valid);
        if (misc[1] || !mbar_wait(barEmpty(st), ((g / NS) & 1) ^ 1, p.err)) {
          ok = false;
          return;
        }
        mbar_arrive_tx(barFull(st), L::kTile);
#pragma unroll
        for (int c = 0; c < D / 64; ++c)
          tma_load_2d(sb + L::kRing + st * L::kTile + c * L::kChunk, map, (r.head + hh) * D + c * 64,
                      r.k_row0 + j0, barFull(st));
        ++g;
      };
      while (ok && next_run(std::true_type())) {
        const CUtensorMap* mk = r.kind == kPrefix ? &tkp : &tk;
        const CUtensorMap* mv = r.kind == kPrefix ? &tvp : &tv;
        const CUtensorMap* mq = r.kind == kCache ? &tqc : &tq;
        const int q_bytes = (D / 64) * 128 * p.G * (r.kind == kCache ? p.HG * p.Lq : p.TQ);
        const int nb = r.blk1 - r.blk0, ahead = r.alt ? 2 : 1;
        // Q tile t into a slot, once the products of the slot's last run are done
        auto load_q = [&](int to, int t) {
          int& nq = to ? nq1 : nq0;
          if (!ok || misc[1] || !mbar_wait(barQEmpty(to), (nq & 1) ^ 1, p.err)) {
            ok = false;
            return;
          }
          ++nq;
          mbar_arrive_tx(barQFull(to), q_bytes);
#pragma unroll
          for (int c = 0; c < D / 64; ++c)
            tma_load_4d(sb + L::kQ + to * L::kTile + c * L::kChunk, mq, c * 64, 0, r.head, r.q_row + t * p.TQ,
                        barQFull(to));
        };
        // one-tile runs alternate between the slots: the next run's Q comes
        // while this one's is in use
        const bool two = r.n_tok1 > 0;
        if (!two) {
          load_q(slot, 0);
          slot ^= 1;
        }
        for (int i = 0; ok && i < min(ahead, nb); ++i) load(mk, i);
        if (two) {
          load_q(0, 0);
          load_q(1, 1);
        }
        for (int i = 0; ok && i < nb; ++i) {
          load(mv, i);
          if (ok && i + ahead < nb) load(mk, i + ahead);
        }
      }
      if (!ok) misc[1] = 1;
      // drain what is in flight before the CTA may end
      for (int u = max(0, g - NS); u < g; ++u) mbar_wait(barFull(u % NS), (u / NS) & 1, nullptr);
      if (nq0 > 0) mbar_wait(barQFull(0), (nq0 - 1) & 1, nullptr);
      if (nq1 > 0) mbar_wait(barQFull(1), (nq1 - 1) & 1, nullptr);
    }
  } else if (warp == 8 || warp == 10) {
    // ------------------------------------------- MMA, one warp per stream
    const int s = warp == 8 ? 0 : 1;
    // (code of the issuing loop, one half after the other or both laid out: a
    // causal 8192-token prompt 370 / 399 us, 200 requests over a 32k prefix 207 /
    // 196 us)
    constexpr int kUnrollHalves = Runs::kUnrollHalves;
    constexpr uint32_t idS = idesc_bf16_f32(kRows, kHalf, false, false);
    constexpr uint32_t idO = idesc_bf16_f32(kRows, D, false, true);
    const uint64_t q_desc = sdesc_sw128(sb + L::kQ, 16, 1024);             // K-major
    const uint64_t k_desc = sdesc_sw128(sb + L::kRing, 16, 1024);
    const uint64_t v_desc = sdesc_sw128(sb + L::kRing, L::kChunk, 1024);   // MN-major
    int stage = 0;                    // of the ring's next block
    uint32_t ring_ph = 0, q_ph = 0, p_ph = 0;  // q_ph: bit per Q slot; p_ph: both halves of P
    int slot = 0;
    bool ok = true;
    auto pass = [&]() {  // the ring's next block's stage
      const int st = stage;
      if (++stage == NS) {
        stage = 0;
        ring_ph ^= 1;
      }
      return st;
    };
    // S of one half of a key block
    auto qk = [&](int h, int tile, int st) {
      const uint64_t qd = q_desc + (uint32_t)(tile * (L::kTile >> 4));
      const uint64_t kd = k_desc + (uint32_t)(st * (L::kTile >> 4) + h * (kHalf * 128 >> 4));
      constexpr uint32_t kC = L::kChunk >> 4;
      const uint32_t dst = tmem + kColS + 128 * s + kHalf * h;
      if (lane == 0) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma(dst, qd + ((k >> 2) * kC + (k & 3) * 2), kd + ((k >> 2) * kC + (k & 3) * 2), idS, k > 0 ? 1u : 0u);
      }
    };
    // O += P V over the first `steps` groups of 16 keys of half h
    auto pv = [&](int h, int st, int steps, uint32_t fresh) {
      if (!warp_wait(barP(s, h), p_ph, p.err, misc)) {
        ok = false;
        return;
      }
      tc_fence_after();
      const uint64_t vd = v_desc + (uint32_t)(st * (L::kTile >> 4) + h * (kHalf * 128 >> 4));
      const uint32_t dst = tmem + kColO + 128 * s, src = tmem + kColS + 128 * s + kHalf * h;
      if (lane == 0) {
        if (steps == 4) {
#pragma unroll
          for (int k = 0; k < 4; ++k) tc_mma_ts(dst, src + k * 8, vd + k * 128, idO, k > 0 ? 1u : fresh ^ 1u);
        } else {
          for (int k = 0; k < steps; ++k) tc_mma_ts(dst, src + k * 8, vd + k * 128, idO, k > 0 ? 1u : fresh ^ 1u);
        }
      }
    };
    while (ok && uniform(next_run(std::false_type()))) {
      const int nb = uniform(r.blk1 - r.blk0);
      const int alt = uniform(r.alt), two = uniform(r.n_tok1 > 0);
      const int ahead = alt ? 2 : 1;
      const bool on = alt || s == 0 || two;  // whether this stream works in this run
      const int tile = two ? s : slot;       // the Q slot it reads, or that is free without it
      if (!two) slot ^= 1;
      auto wait_q = [&](int t) {
        if (!ok || !warp_wait(barQFull(t), (q_ph >> t) & 1u, p.err, misc)) ok = false;
        q_ph ^= 1u << t;
      };
      wait_q(tile);
      if (!ok) break;
      tc_fence_after();
      auto mine = [&](int i) { return on && (!alt || (i & 1) == s); };
      // the last block whose S this stream makes
      const int last = !on ? -1 : alt ? nb - 1 - ((nb - 1 - s) & 1) : nb - 1;
      // a Q slot or stage this stream has issued its products of, or does not use
      auto leave = [&](uint32_t bar, bool used) {
        if (lane == 0) {
          if (used) tc_commit(bar);
          else mbar_arrive(bar);
        }
      };
      if (last < 0) leave(barQEmpty(tile), false);
      // the stream's first S
      for (int i = 0; ok && i < min(ahead, nb); ++i) {
        const uint32_t kph = ring_ph;
        const int kst = pass();
        if (!warp_wait(barFull(kst), kph, p.err, misc)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (mine(i)) {
#pragma unroll 1
          for (int h = 0; h < 2; ++h) {
            qk(h, tile, kst);
            if (lane == 0) tc_commit(barS(s, h));
          }
        }
        leave(barEmpty(kst), mine(i));
        if (i == last) leave(barQEmpty(tile), true);
        __syncwarp();
      }
      // the other stream's Q: this one only says that it does not read it
      if (ok && two) {
        wait_q(s ^ 1);
        if (ok) leave(barQEmpty(s ^ 1), false);
        __syncwarp();
      }
      for (int i = 0; ok && i < nb; ++i) {
        const uint32_t vph = ring_ph;
        const int vst = pass();
        const bool more = i + ahead < nb;
        const uint32_t kph = ring_ph;
        const int kst = more ? pass() : 0;
        if (!warp_wait(barFull(vst), vph, p.err, misc)) {
          ok = false;
          break;
        }
        if (!mine(i)) {
          leave(barEmpty(vst), false);
          if (more) {
            if (!warp_wait(barFull(kst), kph, p.err, misc)) {
              ok = false;
              break;
            }
            leave(barEmpty(kst), false);
          }
          __syncwarp();
          continue;
        }
        int hh, j0, valid;
        block_at(r, r.blk0 + i, hh, j0, valid);
        valid = uniform(valid);
        if (valid & 15) trim<D>(smem + L::kRing + vst * L::kTile, valid);
        const int steps = (valid + 15) >> 4;
#pragma unroll kUnrollHalves
        for (int h = 0; h < 2; ++h) {
          pv(h, vst, min(4, max(0, steps - 4 * h)), i < ahead && h == 0);
          if (!ok) break;
          if (more && h == 0 && !warp_wait(barFull(kst), kph, p.err, misc)) {
            ok = false;
            break;
          }
          if (more) qk(h, tile, kst);
          if (lane == 0) {
            tc_commit(more ? barS(s, h) : barO(s, h));  // O so far, and the next S
            if (h == 1 && more && i + ahead == last) tc_commit(barQEmpty(tile));
          }
          __syncwarp();
        }
        if (!ok) break;
        leave(barEmpty(vst), true);
        if (more) leave(barEmpty(kst), true);
        __syncwarp();
        p_ph ^= 1;
      }
    }
    if (!ok) misc[1] = 1;
    // everything issued is done before TMEM is freed and the CTA ends
    if (lane == 0) {
      const uint32_t done = sb + L::kMisc + 16 + 8 * s;
      mbar_init(done, 1);
      fence_mbar_init();
      tc_commit(done);
      mbar_wait(done, 0, nullptr);
    }
    __syncwarp();
  } else if (warp == 11) {
    // ------------------------------------------------------------ planner
    if constexpr (Runs::kPlanned) {
      Runs runs(p, smem + L::kFull);
      if (lane == 0) {
        for (bool more = true; more;) {
          Run x{};
          more = runs.next(x);
          if (!more) x.kind = kEnd;
          if (misc[1] || !mbar_wait(barRunFree(run_slot), run_ph ^ 1, p.err)) {
            misc[1] = 1;
            break;
          }
          *reinterpret_cast<Run*>(smem + L::kRuns + 64 * run_slot) = x;
          mbar_arrive(barRun(run_slot));
          if (++run_slot == kRunSlots) {
            run_slot = 0;
            run_ph ^= 1;
          }
        }
      }
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int s = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t colS = lanes + kColS + 128 * s, colO = lanes + kColO + 128 * s;
    // the row's token, KV head of the tile and query head of the group, in a
    // tile of one KV head and in a tile of a cache's HG
    const int tok_1 = row / p.G, hg_1 = row - tok_1 * p.G;
    const int tok_c = tok_1 / p.HG, hh_c = tok_1 - tok_c * p.HG;
    const float sc = p.scale * 1.4426950408889634f;
    const float slack = 8.f / sc;
    const bool wide = ((reinterpret_cast<uintptr_t>(p.o) | static_cast<uintptr_t>(p.ld_o * 2)) & 31) == 0;
    uint32_t ph = 0, o_ph = 0;  // phases of both halves' S, and of the runs' last products
    bool ok = true;
    while (ok && next_run(std::false_type())) {
      const int tile = r.alt ? 0 : s;
      if (!r.alt && s == 1 && r.n_tok1 == 0) continue;
      const int n_tok = tile ? r.n_tok1 : r.n_tok0;
      const bool cache = r.kind == kCache, prefix = r.kind == kPrefix;
      const int tok = cache ? tok_c : tok_1, my_hh = cache ? hh_c : 0;
      const int pos0 = r.pos + (prefix ? 0 : tile * p.TQ);
      const int step = r.alt ? 2 : 1;
      const int first = r.blk0 + (r.alt ? s : 0);
      const int pos = prefix ? kAttnFar : pos0 + tok;
      const int pos_last = prefix ? kAttnFar : pos0 + n_tok - 1;
      // a warp none of whose rows is a query leaves its P as it finds it: rows
      // of a product do not mix
      const bool idle = (warp & 3) * 32 >= n_tok * p.G * (cache ? p.HG : 1);
      float m = -INFINITY, l = 0.f;  // reference (raw scores), sum
      for (int b = first; ok && b < r.blk1; b += step) {
        int hh, j0, valid;
        block_at(r, b, hh, j0, valid);
        const bool mine = hh == my_hh && (!cache || tok < n_tok);  // whether the row takes part
        const bool none = !__any_sync(0xffffffffu, mine);
        // blocks that every row of the tile sees whole need no mask
        const bool whole = !cache && valid == kKeys && j0 + kKeys - 1 <= pos0 &&
                           (j0 > pos_last - p.window || j0 + kKeys <= p.n_sink);
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          if (!warp_wait(barS(s, h), ph, p.err, misc)) {
            ok = false;
            break;
          }
          if (idle || kHalf * h >= valid) {  // (or a half without keys: it has no product)
            if (lane == 0) mbar_arrive(barP(s, h));
            continue;
          }
          tc_fence_after();
          const uint32_t col = colS + kHalf * h;
          if (none) {  // another head's block: no weight for these rows
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = 0u;
            tmem_st32(col, w);
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(barP(s, h));
            continue;
          }
          float x[kHalf];
          {
            uint32_t* w = reinterpret_cast<uint32_t*>(x);
            tmem_ld32(col, w);
            tmem_ld32(col + 32, w + 32);
          }
          tc_wait_ld();
          if (!whole) {
            const int c0 = j0 + kHalf * h;  // position of the half's first key
            const int hi = mine ? min(valid - kHalf * h, pos + 1 - c0) : 0, lo = pos - p.window + 1 - c0;
            const int sink = min(hi, p.n_sink - c0);
#pragma unroll
            for (int c = 0; c < kHalf; c += 32) {
              const uint32_t seen = span_bits(lo, hi, c) | span_bits(0, sink, c);
#pragma unroll
              for (int e = 0; e < 32; ++e) x[c + e] = (seen >> e) & 1u ? x[c + e] : -INFINITY;
            }
          }
          float mx[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            mx[q] = fmaxf(x[q * 16], x[q * 16 + 1]);
#pragma unroll
            for (int e = 2; e < 16; e += 2) mx[q] = fmax3(mx[q], x[q * 16 + e], x[q * 16 + e + 1]);
          }
          const float top = fmaxf(fmax3(mx[0], mx[1], mx[2]), mx[3]);
          // a row's first visible key sets its reference; later only a maximum
          // 2^8 above it moves it.  (The maximum passes over NaN; the sum does
          // not, and tells a row that saw only such scores from one that saw
          // none.)
          const bool move = m == -INFINITY ? top > -INFINITY : top > m + slack;
          // (a row that starts has weight zero in O so far: nothing to rescale)
          const bool rescale = move && m > -INFINITY;
          float f = 1.f;
          if (move) {
            f = rescale ? ex2((m - top) * sc) : 0.f;
            m = top;
            l *= f;
          }
          if (__any_sync(0xffffffffu, rescale)) {
            // O must hold every product so far: those of the other half's last
            // P are covered by that half's next S, or are the run's last
            const bool end = h == 1 && b + step >= r.blk1;
            if (!warp_wait(end ? barO(s, 0) : barS(s, h ^ 1), end ? o_ph : h == 0 ? ph : ph ^ 1, p.err, misc)) {
              ok = false;
              break;
            }
            tc_fence_after();
            if (!rescale) f = 1.f;
            // (rolled up: rare, and the loop it sits in has to stay small in the
            // instruction cache; unrolled, a causal 8192-token prompt takes 15 us
            // more)
#pragma unroll 1
            for (int c = 0; c < D; c += 16) {
              uint32_t w[16];
              tmem_ld16(colO + c, w);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(__uint_as_float(w[e]) * f);
              tmem_st16(colO + c, w);
            }
          }
          const float ref = m == -INFINITY ? 0.f : m * sc;
          const float2 sc2 = make_float2(sc, sc), nr = make_float2(-ref, -ref);
          float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < kHalf; e += 2) {
            float2 t = ffma2(make_float2(x[e], x[e + 1]), sc2, nr);
            t.x = ex2(t.x);
            t.y = ex2(t.y);
            acc[(e >> 1) & 1] = fadd2(acc[(e >> 1) & 1], t);
            w[e >> 1] = pack_bf16x2(t.x, t.y);
          }
          tmem_st32(col, w);
          const float2 a = fadd2(acc[0], acc[1]);
          l += a.x + a.y;
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(barP(s, h));
        }
        ph ^= 1;
      }
      if (!ok) break;
      // ----------------------------------------------------------- epilogue
      const bool any = first < r.blk1;
      if (any) {
        if (!warp_wait(barO(s, 0), o_ph, p.err, misc) || !warp_wait(barO(s, 1), o_ph, p.err, misc)) {
          ok = false;
          break;
        }
        o_ph ^= 1;
        tc_fence_after();
      }
      const bool mine = tok < n_tok && my_hh < r.heads;
      const long long q_tok = r.q_row + tile * p.TQ + tok;
      const int head = (r.head + my_hh) * p.G + hg_1;
      if (r.part < 0) {
        const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
        __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + q_tok * p.ld_o + static_cast<long long>(head) * D;
#pragma unroll
        for (int c = 0; c < D; c += 32) {
          uint32_t w[32];
          tmem_ld32(colO + c, w);
          tc_wait_ld();
          uint32_t y[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2)
            y[e / 2] = inv == 0.f ? 0u : pack_bf16x2(__uint_as_float(w[e]) * inv, __uint_as_float(w[e + 1]) * inv);
          if (mine) {
            // (a lane writes its own row: whole sectors where the rows allow it)
            if (wide) {
              st_global_v8(dst + c, y);
              st_global_v8(dst + c + 16, y + 8);
            } else {
#pragma unroll
              for (int e = 0; e < 16; e += 4)
                *reinterpret_cast<uint4*>(dst + c + 2 * e) = make_uint4(y[e], y[e + 1], y[e + 2], y[e + 3]);
            }
          }
        }
        if (mine && p.lse) p.lse[q_tok * p.H_q + head] = l == 0.f ? -INFINITY : m * p.scale + logf(l);
      } else {
        const long long part = r.part + s;
        const long long at = cache ? p.suf_base + part * p.suf_rows + row : part * kRows + row;
        float* dst = p.part_o + at * D;
        if (mine) p.part_ml[at] = make_float2(m == -INFINITY ? -INFINITY : m * sc, l);
        if (any) {
#pragma unroll
          for (int c = 0; c < D; c += 32) {
            uint32_t w[32];
            tmem_ld32(colO + c, w);
            tc_wait_ld();
            if (mine) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) st_global_v8(dst + c + e, w + e);
            }
          }
        }
      }
      tc_fence_before();
    }
    if (!ok) misc[1] = 1;
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// -------------------------------------------------------------------- join --
// o = sum_p 2^(m_p - m) o_p / sum_p 2^(m_p - m) l_p over a row's partial
// results, in their order (the same result every time); a row without any
// visible key gets 0 and lse = -inf.  A warp takes RW rows, 32 / RW lanes over d
// each.
template <int D, bool CACHED, int RW>
__global__ void __launch_bounds__(256) join_kernel(const AttnParams p, const AttnJoin* joins, int n_joins) {
  constexpr int LPR = 32 / RW;   // lanes of a row
  constexpr int V = D / LPR;     // values per lane, in vectors LPR vectors apart
  using Vec = typename std::conditional<V == 2, float2, float4>::type;
  constexpr int NW = sizeof(Vec) / 4, NV = V / NW;
  const int lane = threadIdx.x % LPR;
  // (at most 2^31 rows; 64-bit divisions would take as long as the rest)
  const unsigned w = blockIdx.x * (blockDim.x / LPR) + threadIdx.x / LPR;
  // A row's partial results: n0 of the prefix or of a packed tile, then n1 of
  // its cache.  Result i: part first + i * step (in halves of a slot), rows
  // apart by the tile's.
  long long at0 = 0, at1 = 0, step0 = 0;
  int q_tok = 0, head = 0, n0 = 0, n1 = 0;
  bool live = true;  // (four rows to a warp: a last warp's rows may be past the end)
  // Launched while the attention kernel still runs; its results are there after
  // this.  (What it does not write is looked at before: the lengths.)
  auto wait = []() { asm volatile("griddepcontrol.wait;" ::: "memory"); };
  if (CACHED) {
    live = w < static_cast<unsigned>(p.n * p.Lq) * p.H_q;
    const int len = live ? __ldg(p.lens + w / p.H_q / p.Lq) : 0;
    const int nb = cache_unit(p, len).nb;
    wait();
    if (live) {
      q_tok = static_cast<int>(w / p.H_q);
      head = static_cast<int>(w - static_cast<unsigned>(q_tok) * p.H_q);
      const int kv = head / p.G, hg = head - kv * p.G, req = q_tok / p.Lq;
      const int grid = p.grid;
      // (slots are held to what the buffers have, whatever a failed run left)
      auto slots = [&](int unit, int2 cut, int b0, int b1, int& slot) {
        const int c0 = min(max((cut.x + b0) / cut.y, 0), grid - 1);
        const int c1 = min(max((cut.x + b1) / cut.y, c0), grid - 1);
        slot = unit + c0;
        return c1 - c0 + 1;
      };
      if (p.pre_pairs > 0) {
        const int tile = q_tok / p.TQ, pair = tile >> 1, unit = pair * p.H_kv + kv;
        int slot;
        n0 = slots(unit, p.cuts[unit], 0, p.pre_blocks - 1, slot);
        // a pair's tiles have a stream each; a lone last tile ran on both
        const bool lone = (2 * pair + 1) * p.TQ >= p.n * p.Lq;
        step0 = (lone ? 1 : 2) * kRows;
        at0 = static_cast<long long>(2 * slot + (lone ? 0 : tile & 1)) * kRows + (q_tok - tile * p.TQ) * p.G + hg;
        if (lone) n0 *= 2;
      }
      if (nb > 0) {  // the pieces with blocks of the row's head
        const int hh = kv % p.HG, unit = req * p.groups + kv / p.HG;
        int slot;
        n1 = 2 * slots(unit, p.cuts[p.pre_pairs * p.H_kv + unit], hh * nb, hh * nb + nb - 1, slot);
        at1 = p.suf_base + 2ll * slot * p.suf_rows + ((q_tok - req * p.Lq) * p.HG + hh) * p.G + hg;
      }
    }
  } else {
    wait();
    const unsigned j = w / kRows;
    if (j >= static_cast<unsigned>(n_joins)) return;  // (a whole warp)
    const AttnJoin jn = joins[j];
    const int row = static_cast<int>(w - j * kRows), tok = row / p.G;
    if (tok >= jn.n_tok) return;
    q_tok = jn.q_row + tok;
    head = jn.head * p.G + row - tok * p.G;
    n0 = jn.n_part;
    at0 = static_cast<long long>(jn.part0) * kRows + row;
    step0 = static_cast<long long>(jn.step) * kRows;
  }
  auto at = [&](int i) { return i < n0 ? at0 + i * step0 : at1 + static_cast<long long>(i - n0) * p.suf_rows; };
  const int n = n0 + n1, n_warp = RW == 1 ? n : __reduce_max_sync(0xffffffffu, n);
  float top = -INFINITY, l = 0.f, acc[V] = {};
  // results of o asked for together, before their weights are known
  constexpr int kAtOnce = RW == 1 ? 16 : 64 / V < LPR ? 64 / V : LPR;
  for (int b = 0; b < n_warp; b += kAtOnce) {
    const int m = min(kAtOnce, n - b);
    const float2 ml = lane < m ? p.part_ml[at(b + lane)] : make_float2(-INFINITY, 0.f);
    Vec v[kAtOnce][NV];
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i)
      if (i < m) {
#pragma unroll
        for (int c = 0; c < NV; ++c)
          v[i][c] = *reinterpret_cast<const Vec*>(p.part_o + at(b + i) * D + (c * LPR + lane) * NW);
      }
    float mx = ml.x;
#pragma unroll
    for (int o = kAtOnce / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o, kAtOnce));
    mx = __shfl_sync(0xffffffffu, mx, 0, LPR);
    const float was = top;
    top = fmaxf(top, mx);
    const float f = was == -INFINITY ? 0.f : ex2(was - top);
    const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
    l *= f;
#pragma unroll
    for (int e = 0; e < V; ++e) acc[e] *= f;
#pragma unroll
    for (int i = 0; i < kAtOnce; ++i) {
      const float wi = __shfl_sync(0xffffffffu, w, i, LPR), li = __shfl_sync(0xffffffffu, ml.y, i, LPR);
      // (one that saw nothing has sum 0, and its o was perhaps not written; a sum
      // that is NaN comes through with weight 0 too)
      if (i < m && li != 0.f) {
        l += wi * li;
        const float* x = reinterpret_cast<const float*>(v[i]);
#pragma unroll
        for (int e = 0; e < V; ++e) acc[e] += wi * x[e];
      }
    }
  }
  const bool none = l == 0.f;
  const float inv = none ? 0.f : 1.f / l;
  if (!live) return;
  __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.o) + q_tok * p.ld_o + head * D + lane * NW;
#pragma unroll
  for (int c = 0; c < NV; ++c) {
    const float* x = acc + c * NW;
    if (NW == 4)
      *reinterpret_cast<uint2*>(dst + c * LPR * NW) =
          make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[NW - 2] * inv, x[NW - 1] * inv));
    else
      *reinterpret_cast<uint32_t*>(dst + c * LPR * NW) = pack_bf16x2(x[0] * inv, x[1] * inv);
  }
  if (p.lse && lane == 0)
    p.lse[static_cast<long long>(q_tok) * p.H_q + head] = none ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
}

// The join kernel may be set up while the attention kernel before it in the
// stream runs (it waits for its end on the device).
template <int D, bool CACHED, int RW>
cudaError_t launch_dependent(int grid, cudaStream_t s,
                             const AttnParams& p, const AttnJoin* joins, int n_joins) {
  cudaLaunchAttribute at{};
  // (the attention kernel takes nearly all of an SM's memory as shared memory;
  // a kernel that wants another split beside it makes the SMs change over, twice
  // per call)
  auto kern = join_kernel<D, CACHED, RW>;
  static std::atomic<unsigned long long> done{0};
  const cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributePreferredSharedMemoryCarveout, cudaSharedmemCarveoutMaxShared);
  });
  if (e != cudaSuccess) return e;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p, joins, n_joins);
}

template <int D, typename Runs>
cudaError_t launch_main(const AttnParams& p, int grid, const CUtensorMap& tq, const CUtensorMap& tk,
                        const CUtensorMap& tv, const CUtensorMap& tkp, const CUtensorMap& tvp,
                        const CUtensorMap& tqc, bool cached, cudaStream_t s) {
  auto kern = attn_kernel<D, Runs>;
  static std::atomic<unsigned long long> done{0};
  cudaError_t e = once_per_device(done, [&] {
    return cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Lay<D>::kBytes);
  });
  if (e != cudaSuccess) return e;
  kern<<<grid, kThreads, Lay<D>::kBytes, s>>>(tq, tk, tv, tkp, tvp, tqc, p, cached);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_attn_packed(const AttnParams& p, int d, int grid, const CUtensorMap& tq,
                               const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s) {
  return d == 128 ? launch_main<128, PackedRuns>(p, grid, tq, tk, tv, tk, tv, tq, false, s)
                  : launch_main<64, PackedRuns>(p, grid, tq, tk, tv, tk, tv, tq, false, s);
}

cudaError_t launch_attn_join(const AttnParams& p, int d, const AttnJoin* joins, int n_joins, cudaStream_t s) {
  if (n_joins <= 0) return cudaSuccess;
  const int grid = n_joins * (kRows / 8);
  return d == 128 ? launch_dependent<128, false, 1>(grid, s, p, joins, n_joins)
                  : launch_dependent<64, false, 1>(grid, s, p, joins, n_joins);
}

cudaError_t launch_attn_cache(const AttnParams& p, int d, int grid, const CUtensorMap& tq,
                              const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tkp,
                              const CUtensorMap& tvp, const CUtensorMap& tqc, cudaStream_t s) {
  cudaError_t e = d == 128 ? launch_main<128, CacheRuns>(p, grid, tq, tk, tv, tkp, tvp, tqc, true, s)
                           : launch_main<64, CacheRuns>(p, grid, tq, tk, tv, tkp, tvp, tqc, true, s);
  if (e != cudaSuccess) return e;
  // More rows than the SMs take at once: four to a warp of the join.  (One /
  // four: 64 requests of 512 over a 16384-token prefix 46.5 / 50.0 us, 256 of
  // 500 104 / 97 us, 1024 of 200 215 / 191 us.)
  const long long rows = static_cast<long long>(p.n) * p.Lq * p.H_q;
  const bool many = rows > 32ll * grid;
  const long long blocks = many ? (rows + 31) / 32 : (rows + 7) / 8;
  if (blocks > 0x7fffffffll) return cudaErrorInvalidValue;
  const int g = static_cast<int>(blocks);
  if (many) return d == 128 ? launch_dependent<128, true, 4>(g, s, p, nullptr, 0) : launch_dependent<64, true, 4>(g, s, p, nullptr, 0);
  return d == 128 ? launch_dependent<128, true, 1>(g, s, p, nullptr, 0) : launch_dependent<64, true, 1>(g, s, p, nullptr, 0);
}

}  // namespace mf
