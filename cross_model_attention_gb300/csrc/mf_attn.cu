// mf_attn.cu — host side of the rotary and attention entry points of
// include/mapflow.h: argument checks, the packed form's work plan, workspace
// sizes, tensor maps and launches.
#include <cuda.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>
#include <functional>
#include <new>
#include <queue>
#include <vector>

#include "../../include/mapflow.h"
#include "mf_handle.h"
#include "mf_internal.cuh"

using namespace mf;

struct mf_attn_s {
  bool cached = false;
  int device = 0;               // where the tables are and the calls run
  int H_q = 0, H_kv = 0, d = 0, G = 0, TQ = 0;
  int window = kAttnNoWindow, n_sink = 0;
  int grid = 0;
  // packed form
  int rows = 0;                 // rows of q, k, v and o that the sequences cover
  int n_segs = 0, n_joins = 0, n_slots = 0;
  AttnSeg* segs_d = nullptr;
  int* cta_d = nullptr;
  AttnJoin* joins_d = nullptr;
  // cache form
  int n_max = 0, Lq = 0, cap = 0, P = 0, HG = 1, groups = 1;
  int* err_d = nullptr;
  int* host_err = nullptr;      // pinned
  mf_alloc_fn alloc = nullptr;
  mf_free_fn dealloc = nullptr;
  void* ctx = nullptr;
};

namespace {

constexpr int kBlock = 128;     // keys per block of the kernel
// Cache form: least key blocks per CTA, one for each stream.  (One request of
// 1024 keys with at least 1 / 2 / 4 blocks 12.6 / 12.4 / 13.5 us; two requests
// over a prefix of 1000 13.8 / 12.6 / 14.5 us.)
constexpr int kMinSpan = 2;
constexpr int kMaxTokens = kAttnFar;
// One sequence's, cache's or prefix's keys: a run over them takes about a
// second, and the kernel's waits give up after two.
constexpr int kMaxKeys = 1 << 26;
// Of a packed plan: its table takes up to 0.8 GB on the device, and twice that
// and some 0.3 GB of lists on the host while the plan is made.
constexpr long long kMaxRuns = 1ll << 24;

void* h_alloc(mf_attn_t h, size_t bytes) {
  if (h->alloc) return h->alloc(bytes, h->ctx, nullptr);
  void* p = nullptr;
  if (cudaMallocAsync(&p, bytes, nullptr) != cudaSuccess) {
    cudaGetLastError();
    return nullptr;
  }
  return p;
}
void h_free(mf_attn_t h, void* p) {
  if (!p) return;
  if (h->dealloc) h->dealloc(p, h->ctx, nullptr);
  else cudaFreeAsync(p, nullptr);
}

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

int check_heads(int H_q, int H_kv, int d, int window, int n_sink) {
  if (H_q < 1 || H_kv < 1 || H_q % H_kv != 0) return fail(MF_ERR_ARG, "H_q %% H_kv != 0");
  if (d != 64 && d != 128) return fail(MF_ERR_UNSUPPORTED, "d = %d (supported: 64, 128)", d);
  if (H_q / H_kv > 128) return fail(MF_ERR_UNSUPPORTED, "H_q / H_kv = %d > 128", H_q / H_kv);
  if (H_q > 1024) return fail(MF_ERR_UNSUPPORTED, "H_q = %d > 1024", H_q);
  if (window < 0) return fail(MF_ERR_ARG, "window must be >= 0 (0: none)");
  if (n_sink < 0) return fail(MF_ERR_ARG, "n_sink must be >= 0");
  return MF_OK;
}

// A tensor of `heads` x d values per token, ld values apart.
int check_rows(const char* name, const void* p, int64_t ld, int64_t heads, int d, int esz) {
  if (!p) return fail(MF_ERR_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & 15) return fail(MF_ERR_ARG, "%s must be 16-byte aligned", name);
  if (ld < heads * d) return fail(MF_ERR_ARG, "%s: %lld values between tokens, a token has %lld", name, (long long)ld, (long long)heads * d);
  if ((ld * esz) % 16 != 0) return fail(MF_ERR_ARG, "%s: tokens must be a multiple of 16 bytes apart", name);
  if (ld > (1ll << 32)) return fail(MF_ERR_UNSUPPORTED, "%s: tokens are too far apart", name);
  return MF_OK;
}

// A vector of the caller's, of values of `size` bytes.
int check_aligned(const char* name, const void* p, size_t size) {
  if (reinterpret_cast<uintptr_t>(p) & (size - 1)) return fail(MF_ERR_ARG, "%s must be %zu-byte aligned", name, size);
  return MF_OK;
}

// Whether any value of one strided tensor shares memory with the other's.
bool overlap(const void* a, int64_t lda, int64_t wa, int64_t na, const void* b, int64_t ldb, int64_t wb,
             int64_t nb, int esz) {
  if (na < 1 || nb < 1) return false;
  const int64_t a0 = (int64_t)reinterpret_cast<uintptr_t>(a), b0 = (int64_t)reinterpret_cast<uintptr_t>(b);
  const int64_t a1 = a0 + ((na - 1) * lda + wa) * esz, b1 = b0 + ((nb - 1) * ldb + wb) * esz;
  if (a1 <= b0 || b1 <= a0) return false;
  if (lda != ldb) return true;  // interleaved with different strides: refuse
  const int64_t ld = lda * esz;
  const int64_t off = (((b0 - a0) % ld) + ld) % ld;  // b's row start within a's row
  return off < wa * esz || off + wb * esz > ld;
}

// Keys that the rows at positions pos .. pos + n - 1 see: [0, a1) and [b0, b1).
void key_ranges(int pos, int n, int window, int n_sink, int* a1, int* b0, int* b1) {
  *b1 = pos + n;
  *b0 = std::max(0, pos - window + 1);
  *a1 = 0;
  if (n_sink >= *b0) *b0 = 0;
  else *a1 = n_sink;
}
int blocks_of(int a1, int b0, int b1) { return (a1 + kBlock - 1) / kBlock + (b1 - b0 + kBlock - 1) / kBlock; }

int finish_handle(mf_attn_t h, mf_attn_t* out, const std::vector<AttnSeg>& segs, const std::vector<int>& cta,
                  const std::vector<AttnJoin>& joins) {
  int rc = MF_OK;
  auto put = [&](void** dst, const void* src, size_t bytes) {
    if (rc != MF_OK || bytes == 0) return;
    *dst = h_alloc(h, bytes);
    if (!*dst) {
      rc = fail(MF_ERR_OOM, "allocation of %zu bytes failed", bytes);
      return;
    }
    cudaError_t e = src ? cudaMemcpy(*dst, src, bytes, cudaMemcpyHostToDevice) : cudaMemset(*dst, 0, bytes);
    if (e != cudaSuccess) rc = cuda_fail(e, "attention plan tables");
  };
  put((void**)&h->err_d, nullptr, sizeof(int));
  put((void**)&h->segs_d, segs.data(), segs.size() * sizeof(AttnSeg));
  put((void**)&h->cta_d, cta.data(), cta.size() * sizeof(int));
  put((void**)&h->joins_d, joins.data(), joins.size() * sizeof(AttnJoin));
  if (rc == MF_OK) {
    cudaError_t e = cudaMallocHost((void**)&h->host_err, sizeof(int));
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    if (e != cudaSuccess) rc = cuda_fail(e, "attention plan setup");
  }
  if (rc != MF_OK) {
    char msg[512];
    std::snprintf(msg, sizeof(msg), "%s", mf_last_error());
    mf_attn_destroy(h);
    return fail(rc, "%s", msg);
  }
  *out = h;
  return MF_OK;
}

// Cache form: the workspace's parts.  A line of units cut into one span per
// CTA has fewer than units + CTAs runs.
struct CacheLayout {
  int pairs, nbp, suf_rows;
  long long suf_base;
  size_t ml, o, bytes;  // (the cuts of the units come first)
};
CacheLayout cache_layout(const mf_attn_s* h, int n) {
  CacheLayout c{};
  const long long toks = (long long)n * h->Lq, tiles = (toks + h->TQ - 1) / h->TQ;
  c.pairs = h->P > 0 ? (int)((tiles + 1) / 2) : 0;
  c.nbp = (h->P + kBlock - 1) / kBlock;
  c.suf_rows = h->Lq * h->HG * h->G;
  const long long pre_units = (long long)c.pairs * h->H_kv, suf_units = (long long)n * h->groups;
  c.suf_base = pre_units > 0 ? 2 * (pre_units + h->grid) * kBlock : 0;
  const size_t rows = (size_t)(c.suf_base + 2 * (suf_units + h->grid) * c.suf_rows);
  c.ml = up256((size_t)(pre_units + suf_units) * sizeof(int2));
  c.o = c.ml + up256(rows * sizeof(float2));
  c.bytes = c.o + up256(rows * h->d * sizeof(float));
  return c;
}

// Q tiles of `heads` KV heads' queries and `toks` tokens.
int make_q_map(const mf_attn_s* h, CUtensorMap* m, const void* q, int64_t ld, int64_t rows, int heads, int toks) {
  const uint64_t dims[4] = {(uint64_t)h->d, (uint64_t)h->G, (uint64_t)h->H_kv, (uint64_t)rows};
  const uint64_t st[3] = {(uint64_t)h->d * 2, (uint64_t)h->G * h->d * 2, (uint64_t)ld * 2};
  const uint32_t box[4] = {64, (uint32_t)h->G, (uint32_t)heads, (uint32_t)toks};
  return make_map4(m, q, dims, st, box);
}

int check_device(const mf_attn_s* h) {
  int dev = -1;
  MF_CUDA(cudaGetDevice(&dev), "device query");
  if (dev != h->device) return fail(MF_ERR_ARG, "the plan is on device %d, the current device is %d", h->device, dev);
  return MF_OK;
}

int check_scale(float scale) {
  if (!(scale > 1e-30f && scale < 1e30f)) return fail(MF_ERR_ARG, "scale must be positive and finite");
  return MF_OK;
}

}  // namespace

extern "C" {

// ------------------------------------------------------------------ rotary --
int mf_rope_frequencies(int rot_dim, double base, int scaling, double factor, int original_length,
                        double beta_fast, double beta_slow, uint64_t* turns_out, float* gain_out) {
  if (!turns_out || !gain_out) return fail(MF_ERR_ARG, "NULL pointer argument");
  if (rot_dim < 2 || rot_dim % 2 != 0) return fail(MF_ERR_ARG, "rot_dim = %d must be even and >= 2", rot_dim);
  if (!(base > 1.0) || !std::isfinite(base)) return fail(MF_ERR_ARG, "base must be finite and > 1");
  if (scaling < MF_ROPE_NONE || scaling > MF_ROPE_YARN) return fail(MF_ERR_ARG, "unknown scaling %d", scaling);
  if (scaling != MF_ROPE_NONE && !(factor >= 1.0 && std::isfinite(factor)))
    return fail(MF_ERR_ARG, "factor must be finite and >= 1");
  if (scaling == MF_ROPE_YARN &&
      !(original_length >= 1 && beta_fast > 0 && beta_slow > 0 && beta_fast >= beta_slow && std::isfinite(beta_fast)))
    return fail(MF_ERR_ARG, "by-parts scaling needs original_length >= 1 and beta_fast >= beta_slow > 0");
  const double pi = 3.14159265358979323846;
  double b = base;
  if (scaling == MF_ROPE_NTK && rot_dim > 2) b = base * std::pow(factor, rot_dim / (rot_dim - 2.0));
  double low = 0, high = 0;
  if (scaling == MF_ROPE_YARN) {
    auto dim_of = [&](double turns) {
      return rot_dim * std::log(original_length / (turns * 2.0 * pi)) / (2.0 * std::log(base));
    };
    low = std::max(std::floor(dim_of(beta_fast)), 0.0);
    high = std::min(std::ceil(dim_of(beta_slow)), rot_dim - 1.0);
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double f = std::pow(b, -2.0 * i / rot_dim);
    if (scaling == MF_ROPE_LINEAR) f /= factor;
    if (scaling == MF_ROPE_YARN) {
      const double r = std::min(1.0, std::max(0.0, (i - low) / std::max(high - low, 1e-3)));
      f = f / factor * r + f * (1.0 - r);
    }
    // f <= 1 radian, so its fraction of a turn is below 2^-2
    turns_out[i] = (uint64_t)std::llrint(std::ldexp(f / (2.0 * pi), 64));
  }
  *gain_out = scaling == MF_ROPE_YARN ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
  return MF_OK;
}

int mf_qk_norm_rope(const void* q, int64_t ld_q, void* q_out, int64_t ld_qo, const void* k, int64_t ld_k,
                    void* k_out, int64_t ld_ko, const void* q_weight, const void* k_weight, int norm, float eps,
                    const int32_t* positions, const uint64_t* turns, int rot_dim, int layout, float gain,
                    int dtype, int T, int H_q, int H_k, int d, void* stream) {
  if (dtype != MF_DTYPE_BF16 && dtype != MF_DTYPE_F32) return fail(MF_ERR_ARG, "unknown dtype");
  if (d != 64 && d != 128) return fail(MF_ERR_UNSUPPORTED, "d = %d (supported: 64, 128)", d);
  if (T < 0 || H_q < 1 || H_k < 0 || H_q > 4096 || H_k > 4096)
    return fail(MF_ERR_ARG, "T >= 0, 1 <= H_q <= 4096 and 0 <= H_k <= 4096 expected");
  if (rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > d)
    return fail(MF_ERR_ARG, "rot_dim = %d must be even and in [2, %d]", rot_dim, d);
  if (layout != MF_ROPE_HALF && layout != MF_ROPE_INTERLEAVED) return fail(MF_ERR_ARG, "unknown layout %d", layout);
  if (norm != 0 && norm != 1) return fail(MF_ERR_ARG, "norm must be 0 or 1");
  if (norm && !(eps > 0.f && std::isfinite(eps))) return fail(MF_ERR_ARG, "eps must be positive and finite");
  if (!norm && (q_weight || k_weight)) return fail(MF_ERR_ARG, "weights without a norm");
  if ((reinterpret_cast<uintptr_t>(q_weight) & 15) || (reinterpret_cast<uintptr_t>(k_weight) & 15))
    return fail(MF_ERR_ARG, "weights must be 16-byte aligned");
  if (!std::isfinite(gain)) return fail(MF_ERR_ARG, "gain must be finite");
  if (T == 0) return MF_OK;
  if (!positions || !turns) return fail(MF_ERR_ARG, "positions and turns must be non-NULL");
  const int esz = dtype == MF_DTYPE_F32 ? 4 : 2;
  int rc;
  if ((rc = check_aligned("positions", positions, 4)) != MF_OK) return rc;
  if ((rc = check_aligned("turns", turns, 8)) != MF_OK) return rc;
  if ((rc = check_rows("q", q, ld_q, H_q, d, esz)) != MF_OK) return rc;
  if ((rc = check_rows("q_out", q_out, ld_qo, H_q, d, esz)) != MF_OK) return rc;
  if (H_k > 0) {
    if ((rc = check_rows("k", k, ld_k, H_k, d, esz)) != MF_OK) return rc;
    if ((rc = check_rows("k_out", k_out, ld_ko, H_k, d, esz)) != MF_OK) return rc;
  }
  const int64_t wq = (int64_t)H_q * d, wk = (int64_t)H_k * d;
  auto same = [](const void* a, int64_t lda, const void* b, int64_t ldb) { return a == b && lda == ldb; };
  if (!same(q, ld_q, q_out, ld_qo) && overlap(q, ld_q, wq, T, q_out, ld_qo, wq, T, esz))
    return fail(MF_ERR_ARG, "q_out must be q itself or apart from it");
  if (H_k > 0) {
    if (!same(k, ld_k, k_out, ld_ko) && overlap(k, ld_k, wk, T, k_out, ld_ko, wk, T, esz))
      return fail(MF_ERR_ARG, "k_out must be k itself or apart from it");
    if (overlap(q_out, ld_qo, wq, T, k_out, ld_ko, wk, T, esz) || overlap(q_out, ld_qo, wq, T, k, ld_k, wk, T, esz) ||
        overlap(q, ld_q, wq, T, k_out, ld_ko, wk, T, esz))
      return fail(MF_ERR_ARG, "the outputs share memory with each other or with the other input");
  }
  RopeParams p{};
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.ld_q = ld_q;
  p.ld_k = ld_k;
  p.ld_qo = ld_qo;
  p.ld_ko = ld_ko;
  p.q_weight = q_weight;
  p.k_weight = k_weight;
  p.positions = positions;
  p.freq = reinterpret_cast<const unsigned long long*>(turns);
  p.H_q = H_q;
  p.H_k = H_k;
  p.rot = rot_dim;
  p.layout = layout;
  p.norm = norm;
  p.eps = eps;
  p.gain = gain;
  MF_CUDA(launch_rope(p, T, dtype == MF_DTYPE_F32, d, static_cast<cudaStream_t>(stream)), "norm and rotary kernel");
  return MF_OK;
}

// --------------------------------------------------------------- attention --
int mf_attn_create_packed(mf_attn_t* out, const int32_t* cu_seqlens_host, const int32_t* q_begin_host, int n_seqs,
                          int H_q, int H_kv, int d, int window, int n_sink, mf_alloc_fn alloc_fn,
                          mf_free_fn free_fn, void* alloc_ctx) {
  if (!out) return fail(MF_ERR_ARG, "out is NULL");
  *out = nullptr;
  if (n_seqs < 1 || !cu_seqlens_host) return fail(MF_ERR_ARG, "n_seqs must be >= 1 and cu_seqlens non-NULL");
  if ((alloc_fn == nullptr) != (free_fn == nullptr))
    return fail(MF_ERR_ARG, "alloc_fn and free_fn must both be set or both be NULL");
  int rc = check_heads(H_q, H_kv, d, window, n_sink);
  if (rc != MF_OK) return rc;
  if (cu_seqlens_host[0] != 0) return fail(MF_ERR_ARG, "cu_seqlens[0] must be 0");
  long long q_rows = 0, runs = 0;
  for (int s = 0; s < n_seqs; ++s) {
    const long long len = (long long)cu_seqlens_host[s + 1] - cu_seqlens_host[s];
    if (len < 0) return fail(MF_ERR_ARG, "cu_seqlens must be non-decreasing (sequence %d)", s);
    const int qb = q_begin_host ? q_begin_host[s] : 0;
    if (len > kMaxKeys) return fail(MF_ERR_UNSUPPORTED, "sequence %d has more than 2^26 tokens", s);
    if (qb < 0 || qb > len) return fail(MF_ERR_ARG, "q_begin[%d] = %d must be in [0, %lld]", s, qb, len);
    q_rows += len - qb;
    const int pair = 2 * (kBlock / (H_q / H_kv));
    runs += (len - qb + pair - 1) / pair;
  }
  if (cu_seqlens_host[n_seqs] > kMaxTokens) return fail(MF_ERR_UNSUPPORTED, "more than 2^29 tokens");
  if (q_rows == 0) return fail(MF_ERR_ARG, "the sequences hold no query rows");
  if (runs * H_kv > kMaxRuns) return fail(MF_ERR_UNSUPPORTED, "%lld query tiles of %d heads are too many for one plan", 2 * runs, H_kv);

  mf_attn_t h = new (std::nothrow) mf_attn_s();
  if (!h) return fail(MF_ERR_OOM, "host memory");
  h->H_q = H_q;
  h->H_kv = H_kv;
  h->d = d;
  h->G = H_q / H_kv;
  h->TQ = kBlock / h->G;
  h->window = window == 0 || window > kAttnFar ? kAttnNoWindow : window;
  h->n_sink = std::min(n_sink, kAttnFar);
  h->rows = cu_seqlens_host[n_seqs];
  h->alloc = alloc_fn;
  h->dealloc = free_fn;
  h->ctx = alloc_ctx;
  cudaError_t ce = cudaGetDevice(&h->device);
  if (ce == cudaSuccess) ce = sm_count(&h->grid);
  if (ce != cudaSuccess) {
    delete h;
    return cuda_fail(ce, "device query");
  }
  std::vector<AttnSeg> items, segs;
  std::vector<int> cta;
  std::vector<AttnJoin> joins;
  try {
    cta.assign(h->grid + 1, 0);
    items.reserve(runs * H_kv);
    segs.reserve(runs * H_kv + h->grid);  // (cut, the runs are at most that many)
    for (int s = 0; s < n_seqs; ++s) {
      const int start = cu_seqlens_host[s], len = cu_seqlens_host[s + 1] - start;
      for (int head = 0; head < H_kv; ++head)
        for (int t = q_begin_host ? q_begin_host[s] : 0; t < len; t += 2 * h->TQ) {
          AttnSeg a{};
          a.q_row = start + t;
          a.n_tok = std::min(2 * h->TQ, len - t);
          a.pos = t;
          a.k_row0 = start;
          key_ranges(t, a.n_tok, h->window, h->n_sink, &a.a1, &a.b0, &a.b1);
          a.blk0 = 0;
          a.blk1 = blocks_of(a.a1, a.b0, a.b1);
          a.head = head;
          a.part = -1;
          items.push_back(a);
        }
    }
    // Whole runs, the longest first, each to the CTA with the least work so
    // far; a run costs its blocks and about two more for its start and end.
    // Where that leaves CTAs uneven (few query rows over many keys), the runs
    // are laid end to end instead and cut into equal spans; a cut run's pieces
    // write partial results that a second kernel joins, which costs about as
    // much as five blocks.  (32q/8kv heads of 128, whole against cut: one row
    // over 1000 keys 14.6 / 10.0 us, 64 rows over 700 14.8 / 16.1, 128 rows over
    // 1500 24.3 / 18.9, 256 over 4096 54 / 31, a 1024-token prompt 18.8 / 32.5.)
    const int n = (int)items.size(), grid = h->grid;
    constexpr int kRun = 2, kJoin = 5;
    std::vector<int> order(n);
    long long total = 0;
    for (int i = 0; i < n; ++i) {
      order[i] = i;
      total += items[i].blk1 + kRun;
    }
    std::stable_sort(order.begin(), order.end(), [&](int a, int b) { return items[a].blk1 > items[b].blk1; });
    using Slot = std::pair<long long, int>;
    std::priority_queue<Slot, std::vector<Slot>, std::greater<Slot>> least;
    for (int c = 0; c < grid; ++c) least.push({0, c});
    std::vector<std::vector<int>> mine(grid);
    long long makespan = 0;
    for (int i : order) {
      Slot x = least.top();
      least.pop();
      mine[x.second].push_back(i);
      x.first += items[i].blk1 + kRun;
      makespan = std::max(makespan, x.first);
      least.push(x);
    }
    const long long span = std::max<long long>(kRun + 2, (total + grid - 1) / grid);
    if (makespan <= span + kJoin) {
      for (int c = 0; c < grid; ++c) {
        cta[c] = (int)segs.size();
        for (int i : mine[c]) segs.push_back(items[i]);
      }
      cta[grid] = (int)segs.size();
    } else {
      // block b of an item lies at place at + kRun + b, in CTA place / span
      long long at = 0;
      int c = 0;
      for (int i = 0; i < n; ++i) {
        const int nb = items[i].blk1;
        const long long begin = at + kRun;
        const bool cut = begin / span != (begin + nb - 1) / span;
        const int slot0 = h->n_slots;
        int pieces = 0;
        for (long long b = 0; b < nb;) {
          const long long who = (begin + b) / span;
          const long long upto = std::min<long long>(nb, (who + 1) * span - begin);
          while (c < who) cta[++c] = (int)segs.size();
          AttnSeg a = items[i];
          a.blk0 = (int)b;
          a.blk1 = (int)upto;
          a.part = cut ? 2 * (slot0 + pieces) : -1;
          segs.push_back(a);
          ++pieces;
          b = upto;
        }
        if (cut) {
          h->n_slots += pieces;
          const AttnSeg& a = items[i];
          const int n0 = std::min(a.n_tok, h->TQ), n1 = a.n_tok - n0;
          if (n1 > 0) {
            joins.push_back(AttnJoin{a.q_row, n0, a.head, 2 * slot0, pieces, 2});
            joins.push_back(AttnJoin{a.q_row + n0, n1, a.head, 2 * slot0 + 1, pieces, 2});
          } else {
            joins.push_back(AttnJoin{a.q_row, n0, a.head, 2 * slot0, 2 * pieces, 1});
          }
        }
        at = begin + nb;
      }
      while (c < grid) cta[++c] = (int)segs.size();
    }
    h->n_segs = (int)segs.size();
    h->n_joins = (int)joins.size();
  } catch (const std::exception&) {
    delete h;
    return fail(MF_ERR_OOM, "host memory for the plan");
  }
  return finish_handle(h, out, segs, cta, joins);
}

int mf_attn_create_cache(mf_attn_t* out, int n_max, int Lq, int capacity, int prefix_len, int H_q, int H_kv, int d,
                         int window, int n_sink, mf_alloc_fn alloc_fn, mf_free_fn free_fn, void* alloc_ctx) {
  if (!out) return fail(MF_ERR_ARG, "out is NULL");
  *out = nullptr;
  if (n_max < 1 || Lq < 1 || capacity < 1 || prefix_len < 0)
    return fail(MF_ERR_ARG, "n_max, Lq and capacity must be >= 1 and prefix_len >= 0");
  if ((alloc_fn == nullptr) != (free_fn == nullptr))
    return fail(MF_ERR_ARG, "alloc_fn and free_fn must both be set or both be NULL");
  int rc = check_heads(H_q, H_kv, d, window, n_sink);
  if (rc != MF_OK) return rc;
  if (prefix_len > 0 && (window != 0 || n_sink != 0))
    return fail(MF_ERR_UNSUPPORTED, "a shared prefix with a window");
  if ((long long)Lq * (H_q / H_kv) > kBlock)
    return fail(MF_ERR_UNSUPPORTED, "Lq * H_q / H_kv = %lld > 128 (use the packed form)", (long long)Lq * (H_q / H_kv));
  if (capacity > kMaxKeys || prefix_len > kMaxKeys) return fail(MF_ERR_UNSUPPORTED, "more than 2^26 keys");
  if ((long long)n_max * capacity > 0x7fffffffll || (long long)n_max * Lq > 0x7fffffffll / 1024)
    return fail(MF_ERR_UNSUPPORTED, "n_max = %d is too large", n_max);
  {  // the kernel lays all work end to end in 32 bits
    const long long tiles = ((long long)n_max * Lq + kBlock / (H_q / H_kv) - 1) / (kBlock / (H_q / H_kv));
    const long long lines = (tiles + 1) / 2 * (kAttnCostPre + (prefix_len + kBlock - 1ll) / kBlock) +
                            n_max * (kAttnCostCache + (capacity + kBlock - 1ll) / kBlock + 1);
    if (lines * H_kv > (1ll << 30)) return fail(MF_ERR_UNSUPPORTED, "n_max = %d, capacity = %d and prefix_len = %d are too much work for one call", n_max, capacity, prefix_len);
  }
  mf_attn_t h = new (std::nothrow) mf_attn_s();
  if (!h) return fail(MF_ERR_OOM, "host memory");
  h->cached = true;
  h->H_q = H_q;
  h->H_kv = H_kv;
  h->d = d;
  h->G = H_q / H_kv;
  h->TQ = kBlock / h->G;
  h->window = window == 0 || window > kAttnFar ? kAttnNoWindow : window;
  h->n_sink = std::min(n_sink, kAttnFar);
  h->n_max = n_max;
  h->Lq = Lq;
  h->cap = capacity;
  h->P = prefix_len;
  h->HG = std::min(H_kv, kBlock / (Lq * h->G));
  h->groups = (H_kv + h->HG - 1) / h->HG;
  h->alloc = alloc_fn;
  h->dealloc = free_fn;
  h->ctx = alloc_ctx;
  cudaError_t ce = cudaGetDevice(&h->device);
  if (ce == cudaSuccess) ce = sm_count(&h->grid);
  if (ce != cudaSuccess) {
    delete h;
    return cuda_fail(ce, "device query");
  }
  return finish_handle(h, out, {}, {}, {});
}

void mf_attn_destroy(mf_attn_t h) {
  if (!h) return;
  DeviceScope scope(h->device);
  if (capture_refused(cudaDeviceSynchronize())) {
    cudaGetLastError();  // kernels may still read the tables: they stay allocated
  } else {
    h_free(h, h->segs_d);
    h_free(h, h->cta_d);
    h_free(h, h->joins_d);
    h_free(h, h->err_d);
    if (h->host_err) cudaFreeHost(h->host_err);
  }
  delete h;
}

int mf_attn_workspace(mf_attn_t h, int n, int64_t* bytes) {
  if (!h || !bytes) return fail(MF_ERR_ARG, "NULL argument");
  if (h->cached) {
    if (n < 1 || n > h->n_max) return fail(MF_ERR_ARG, "n = %d is not in [1, %d]", n, h->n_max);
    *bytes = (int64_t)cache_layout(h, n).bytes;
  } else {
    const size_t rows = (size_t)h->n_slots * 2 * kBlock;
    *bytes = h->n_slots ? (int64_t)(up256(rows * sizeof(float2)) + rows * h->d * sizeof(float)) : 0;
  }
  return MF_OK;
}

int mf_attn_packed(mf_attn_t h, const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                   int64_t ld_v, void* o, int64_t ld_o, float* lse, int dtype, float scale, void* workspace,
                   int64_t workspace_bytes, void* stream) {
  if (!h) return fail(MF_ERR_ARG, "handle is NULL");
  if (h->cached) return fail(MF_ERR_ARG, "the plan is of the cache form");
  if (dtype != MF_DTYPE_BF16) return fail(MF_ERR_UNSUPPORTED, "attention is built for bf16");
  int rc = check_device(h);
  if (rc != MF_OK) return rc;
  if ((rc = check_rows("q", q, ld_q, h->H_q, h->d, 2)) != MF_OK) return rc;
  if ((rc = check_rows("k", k, ld_k, h->H_kv, h->d, 2)) != MF_OK) return rc;
  if ((rc = check_rows("v", v, ld_v, h->H_kv, h->d, 2)) != MF_OK) return rc;
  if ((rc = check_rows("o", o, ld_o, h->H_q, h->d, 2)) != MF_OK) return rc;
  if ((rc = check_aligned("lse", lse, 4)) != MF_OK) return rc;
  if ((rc = check_scale(scale)) != MF_OK) return rc;
  const int64_t wq = (int64_t)h->H_q * h->d, wk = (int64_t)h->H_kv * h->d, T = h->rows;
  if (overlap(q, ld_q, wq, T, o, ld_o, wq, T, 2) || overlap(k, ld_k, wk, T, o, ld_o, wq, T, 2) ||
      overlap(v, ld_v, wk, T, o, ld_o, wq, T, 2))
    return fail(MF_ERR_ARG, "o shares memory with an input");
  int64_t need = 0;
  mf_attn_workspace(h, 1, &need);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(MF_ERR_ARG, "the workspace has %lld bytes, %lld are needed", (long long)workspace_bytes, (long long)need);
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(MF_ERR_ARG, "the workspace must be 256-byte aligned");
  CUtensorMap tq, tk, tv;
  if ((rc = make_q_map(h, &tq, q, ld_q, T, 1, h->TQ)) != MF_OK) return rc;
  if ((rc = make_map(&tk, k, (uint64_t)wk, (uint64_t)T, (uint64_t)ld_k * 2, 64, kBlock)) != MF_OK) return rc;
  if ((rc = make_map(&tv, v, (uint64_t)wk, (uint64_t)T, (uint64_t)ld_v * 2, 64, kBlock)) != MF_OK) return rc;
  AttnParams p{};
  p.H_q = h->H_q;
  p.H_kv = h->H_kv;
  p.G = h->G;
  p.TQ = h->TQ;
  p.scale = scale;
  p.window = h->window;
  p.n_sink = h->n_sink;
  p.o = o;
  p.ld_o = ld_o;
  p.lse = lse;
  p.HG = 1;
  p.segs = h->segs_d;
  p.cta_segs = h->cta_d;
  const size_t rows = (size_t)h->n_slots * 2 * kBlock;
  p.part_ml = static_cast<float2*>(workspace);
  p.part_o = reinterpret_cast<float*>(static_cast<char*>(workspace) + up256(rows * sizeof(float2)));
  p.err = h->err_d;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  MF_CUDA(launch_attn_packed(p, h->d, h->grid, tq, tk, tv, s), "attention kernel");
  MF_CUDA(launch_attn_join(p, h->d, h->joins_d, h->n_joins, s), "attention join kernel");
  return MF_OK;
}

int mf_attn_cached(mf_attn_t h, int n, const void* q, int64_t ld_q, const void* k_cache, int64_t ld_k,
                   const void* v_cache, int64_t ld_v, const int32_t* lens, const void* k_prefix, int64_t ld_kp,
                   const void* v_prefix, int64_t ld_vp, void* o, int64_t ld_o, float* lse, int dtype, float scale,
                   void* workspace, int64_t workspace_bytes, void* stream) {
  if (!h) return fail(MF_ERR_ARG, "handle is NULL");
  if (!h->cached) return fail(MF_ERR_ARG, "the plan is of the packed form");
  if (n < 1 || n > h->n_max) return fail(MF_ERR_ARG, "n = %d is not in [1, %d]", n, h->n_max);
  if (dtype != MF_DTYPE_BF16) return fail(MF_ERR_UNSUPPORTED, "attention is built for bf16");
  if (!lens) return fail(MF_ERR_ARG, "lens is NULL");
  int rc = check_device(h);
  if (rc != MF_OK) return rc;
  if ((rc = check_aligned("lens", lens, 4)) != MF_OK) return rc;
  if ((rc = check_aligned("lse", lse, 4)) != MF_OK) return rc;
  if ((rc = check_rows("q", q, ld_q, h->H_q, h->d, 2)) != MF_OK) return rc;
  if ((rc = check_rows("k_cache", k_cache, ld_k, h->H_kv, h->d, 2)) != MF_OK) return rc;
  if ((rc = check_rows("v_cache", v_cache, ld_v, h->H_kv, h->d, 2)) != MF_OK) return rc;
  if ((rc = check_rows("o", o, ld_o, h->H_q, h->d, 2)) != MF_OK) return rc;
  if (h->P > 0) {
    if ((rc = check_rows("k_prefix", k_prefix, ld_kp, h->H_kv, h->d, 2)) != MF_OK) return rc;
    if ((rc = check_rows("v_prefix", v_prefix, ld_vp, h->H_kv, h->d, 2)) != MF_OK) return rc;
  } else if (k_prefix || v_prefix) {
    return fail(MF_ERR_ARG, "the plan has no prefix");
  }
  if ((rc = check_scale(scale)) != MF_OK) return rc;
  const int64_t wq = (int64_t)h->H_q * h->d, wk = (int64_t)h->H_kv * h->d;
  const int64_t rows = (int64_t)n * h->Lq, kr = (int64_t)n * h->cap;
  if (overlap(q, ld_q, wq, rows, o, ld_o, wq, rows, 2) || overlap(k_cache, ld_k, wk, kr, o, ld_o, wq, rows, 2) ||
      overlap(v_cache, ld_v, wk, kr, o, ld_o, wq, rows, 2) ||
      (h->P > 0 && (overlap(k_prefix, ld_kp, wk, h->P, o, ld_o, wq, rows, 2) ||
                    overlap(v_prefix, ld_vp, wk, h->P, o, ld_o, wq, rows, 2))))
    return fail(MF_ERR_ARG, "o shares memory with an input");
  const CacheLayout c = cache_layout(h, n);
  if (!workspace || workspace_bytes < (int64_t)c.bytes)
    return fail(MF_ERR_ARG, "the workspace has %lld bytes, %zu are needed", (long long)workspace_bytes, c.bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return fail(MF_ERR_ARG, "the workspace must be 256-byte aligned");
  CUtensorMap tq, tqc, tk, tv, tkp, tvp;
  if ((rc = make_q_map(h, &tqc, q, ld_q, rows, h->HG, h->Lq)) != MF_OK) return rc;
  if ((rc = make_map(&tk, k_cache, (uint64_t)wk, (uint64_t)kr, (uint64_t)ld_k * 2, 64, kBlock)) != MF_OK) return rc;
  if ((rc = make_map(&tv, v_cache, (uint64_t)wk, (uint64_t)kr, (uint64_t)ld_v * 2, 64, kBlock)) != MF_OK) return rc;
  tq = tqc;
  tkp = tk;
  tvp = tv;
  if (h->P > 0) {
    if ((rc = make_q_map(h, &tq, q, ld_q, rows, 1, h->TQ)) != MF_OK) return rc;
    if ((rc = make_map(&tkp, k_prefix, (uint64_t)wk, (uint64_t)h->P, (uint64_t)ld_kp * 2, 64, kBlock)) != MF_OK) return rc;
    if ((rc = make_map(&tvp, v_prefix, (uint64_t)wk, (uint64_t)h->P, (uint64_t)ld_vp * 2, 64, kBlock)) != MF_OK) return rc;
  }
  AttnParams p{};
  p.H_q = h->H_q;
  p.H_kv = h->H_kv;
  p.G = h->G;
  p.TQ = h->TQ;
  p.scale = scale;
  p.window = h->window;
  p.n_sink = h->n_sink;
  p.o = o;
  p.ld_o = ld_o;
  p.lse = lse;
  p.lens = lens;
  p.n = n;
  p.Lq = h->Lq;
  p.cap = h->cap;
  p.P = h->P;
  p.pre_pairs = c.pairs;
  p.pre_blocks = c.nbp;
  p.HG = h->HG;
  p.groups = h->groups;
  p.grid = h->grid;
  p.suf_base = c.suf_base;
  p.suf_rows = c.suf_rows;
  p.min_span = kMinSpan;
  if (n > kAttnSlotBits)  // (the kernel sums eight requests at a time: 0 or at least 3)
    for (p.slot_shift = 3; n > kAttnSlotBits << p.slot_shift;) ++p.slot_shift;
  char* ws = static_cast<char*>(workspace);
  p.cuts = reinterpret_cast<int2*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + c.ml);
  p.part_o = reinterpret_cast<float*>(ws + c.o);
  p.err = h->err_d;
  MF_CUDA(launch_attn_cache(p, h->d, h->grid, tq, tk, tv, tkp, tvp, tqc, static_cast<cudaStream_t>(stream)),
          "cache attention kernels");
  return MF_OK;
}

int mf_attn_status(mf_attn_t h, void* stream) {
  if (!h) return fail(MF_ERR_ARG, "handle is NULL");
  const int rc = check_device(h);
  if (rc != MF_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  MF_CUDA(cudaMemcpyAsync(h->host_err, h->err_d, sizeof(int), cudaMemcpyDeviceToHost, s), "error word copy");
  MF_CUDA(cudaStreamSynchronize(s), "attention status");
  if (*h->host_err == 0) return MF_OK;
  MF_CUDA(cudaMemsetAsync(h->err_d, 0, sizeof(int), s), "error word reset");
  return fail(MF_ERR_TIMEOUT, "a device-side wait timed out in the attention kernel");
}

}  // extern "C"
