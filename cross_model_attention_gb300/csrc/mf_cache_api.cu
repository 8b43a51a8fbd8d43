// mf_cache_api.cu — host side of the paged cache's entry points of
// include/mapflow.h: argument checks, the workspace's parts and launches.
#include <cuda_runtime.h>

#include <cmath>

#include "../../include/mapflow.h"
#include "mf_fp4.cuh"
#include "mf_handle.h"
#include "mf_internal.cuh"

using namespace mf;

namespace {

// A sequence's tokens: tiles and distances stay in int (as fp32, for a bias by
// distance, they are off by 2^-24 of themselves at most).
constexpr long long kMaxKeys = 1ll << 26;

size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

int check_aligned(const char* name, const void* p, size_t size) {
  if (!p) return fail(MF_ERR_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) & (size - 1)) return fail(MF_ERR_ARG, "%s must be %zu-byte aligned", name, size);
  return MF_OK;
}
// A tensor of `heads` x d bf16 values per token, ld values apart.
int check_rows(const char* name, const void* p, int64_t ld, int64_t heads, int d) {
  int rc = check_aligned(name, p, 16);
  if (rc != MF_OK) return rc;
  if (ld < heads * d) return fail(MF_ERR_ARG, "%s: %lld values between tokens, a token has %lld", name, (long long)ld, (long long)heads * d);
  if (ld % 8 != 0) return fail(MF_ERR_ARG, "%s: tokens must be a multiple of 16 bytes apart", name);
  if (ld > (1ll << 32)) return fail(MF_ERR_UNSUPPORTED, "%s: tokens are too far apart", name);
  return MF_OK;
}

int check_cache(const mf_cache_t* c) {
  if (!c) return fail(MF_ERR_ARG, "cache is NULL");
  if (c->format != MF_CACHE_BF16 && c->format != MF_CACHE_FP4) return fail(MF_ERR_ARG, "unknown cache format %d", c->format);
  if (c->d != 64 && c->d != 128) return fail(MF_ERR_UNSUPPORTED, "d = %d (supported: 64, 128)", c->d);
  if (c->H < 1 || c->H > 1024) return fail(MF_ERR_ARG, "H = %d must be in [1, 1024]", c->H);
  if (c->page_size < 1) return fail(MF_ERR_ARG, "page_size must be >= 1");
  if (c->n_pages < 1 || c->n_pages > 0x7fffffffll) return fail(MF_ERR_ARG, "n_pages must be in [1, 2^31 - 1]");
  int rc;
  if (c->format == MF_CACHE_FP4) {
    if (c->page_size % kFp4Block != 0) return fail(MF_ERR_ARG, "page_size = %d must be a multiple of 16", c->page_size);
    if (c->v) return fail(MF_ERR_ARG, "4-bit pages hold keys and values: v must be NULL");
    if ((rc = check_aligned("the cache's pages", c->k, 16)) != MF_OK) return rc;
    if (c->k_scale && (rc = check_aligned("k_scale", c->k_scale, 4)) != MF_OK) return rc;
    if (c->v_scale && (rc = check_aligned("v_scale", c->v_scale, 4)) != MF_OK) return rc;
    return MF_OK;
  }
  if (c->k_scale || c->v_scale) return fail(MF_ERR_ARG, "a bf16 cache has no scales");
  if ((rc = check_rows("the cache's k", c->k, c->ld_k, c->H, c->d)) != MF_OK) return rc;
  return check_rows("the cache's v", c->v, c->ld_v, c->H, c->d);
}

int check_table(const mf_cache_t* c, const int32_t* table, int64_t ld_table, int rows, int max_pages) {
  if (max_pages < 1) return fail(MF_ERR_ARG, "max_pages must be >= 1");
  if (ld_table < max_pages) return fail(MF_ERR_ARG, "table: rows of %d numbers are %lld apart", max_pages, (long long)ld_table);
  if (ld_table > (1ll << 32)) return fail(MF_ERR_UNSUPPORTED, "table: rows are too far apart");
  if ((long long)max_pages * c->page_size > kMaxKeys)
    return fail(MF_ERR_UNSUPPORTED, "%d pages of %d tokens: more than 2^26 tokens a sequence", max_pages, c->page_size);
  if (rows < 1) return fail(MF_ERR_ARG, "the table has no rows");
  return check_aligned("table", table, 4);
}

// The bytes from a tensor's first value to its last.
struct Span {
  uintptr_t a, b;
};
Span rows_span(const void* p, int64_t ld, int64_t width, int64_t rows) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, rows < 1 ? a : a + ((rows - 1) * ld + width) * 2};
}
bool apart(Span x, Span y) { return x.b <= y.a || y.b <= x.a; }
// Whether rows of a and b share memory: in one span, rows may still lie beside each other.
bool rows_apart(const void* a, int64_t lda, int64_t wa, int64_t na, const void* b, int64_t ldb, int64_t wb, int64_t nb) {
  if (na < 1 || nb < 1 || apart(rows_span(a, lda, wa, na), rows_span(b, ldb, wb, nb))) return true;
  if (lda != ldb) return false;
  const int64_t ld = lda * 2, off = (int64_t)(reinterpret_cast<uintptr_t>(b) - reinterpret_cast<uintptr_t>(a));
  const int64_t in = ((off % ld) + ld) % ld;  // b's rows' start in a's
  return in >= wa * 2 && in + wb * 2 <= ld;
}
int shared(const char* a, const char* b) { return fail(MF_ERR_ARG, "%s shares memory with %s", a, b); }
// What a call reads besides rows of heads, NULL where there is none.
struct Read {
  const char* name;
  const void* p;
  int64_t bytes;
};
template <int N>
int check_apart(const char* name, Span out, const Read (&in)[N]) {
  for (const Read& r : in) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(r.p);
    if (r.p && !apart(out, {a, a + r.bytes})) return shared(name, r.name);
  }
  return MF_OK;
}
Span pages_span(const mf_cache_t* c) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(c->k);
  return {a, a + (uintptr_t)(c->n_pages * c->page_size / kFp4Block) * c->H * fp4_piece(c->d)};
}
int64_t table_bytes(int64_t ld, int rows, int max_pages) { return (int64_t)(((uint64_t)(rows - 1) * (uint64_t)ld + max_pages) * 4); }
// Whether a tensor of T rows shares no memory with the cache.
bool clear_of(const mf_cache_t* c, const void* p, int64_t ld, int T) {
  const int64_t w = (int64_t)c->H * c->d, rows = c->n_pages * c->page_size;
  if (c->format == MF_CACHE_FP4) return apart(pages_span(c), rows_span(p, ld, w, T));
  return rows_apart(c->k, c->ld_k, w, rows, p, ld, w, T) && rows_apart(c->v, c->ld_v, w, rows, p, ld, w, T);
}

void fill(CacheParams* p, const mf_cache_t* c, const int32_t* seq, const int32_t* at, const int32_t* table,
          int64_t ld_table, int n_seqs, int max_pages) {
  const bool fp4 = c->format == MF_CACHE_FP4;
  p->pages = fp4 ? static_cast<uint8_t*>(c->k) : nullptr;
  p->k = fp4 ? nullptr : c->k;
  p->v = fp4 ? nullptr : c->v;
  p->ld_k = c->ld_k;
  p->ld_v = c->ld_v;
  p->k_scale = c->k_scale;
  p->v_scale = c->v_scale;
  p->n_pages = c->n_pages;
  p->ps = c->page_size;
  p->H = c->H;
  p->seq = seq;
  p->at = at;
  p->table = table;
  p->ld_table = ld_table;
  p->n_seqs = n_seqs;
  p->max_pages = max_pages;
}

struct PagedLayout {
  int rows;
  size_t ml, cuts, bytes;  // (the partial results come first)
};
int check_shape(int Lq, int H_q, int H_kv, int d) {
  if (d != 64 && d != 128) return fail(MF_ERR_UNSUPPORTED, "d = %d (supported: 64, 128)", d);
  if (Lq < 1 || H_q < 1 || H_kv < 1 || H_q % H_kv != 0) return fail(MF_ERR_ARG, "Lq >= 1 and H_q %% H_kv == 0 expected");
  if (H_q > 1024) return fail(MF_ERR_UNSUPPORTED, "H_q = %d > 1024", H_q);
  if ((long long)Lq * (H_q / H_kv) > 128) return fail(MF_ERR_UNSUPPORTED, "Lq * H_q / H_kv = %lld > 128", (long long)Lq * (H_q / H_kv));
  return MF_OK;
}
int paged_layout(int Lq, int H_q, int H_kv, int d, PagedLayout* l) {
  int sms = 0, grid = 0, parts = 0;
  MF_CUDA(sm_count(&sms), "device query");
  paged_shape(Lq, H_q / H_kv, sms, &grid, &parts, &l->rows);
  const size_t rows = (size_t)parts * l->rows;
  l->ml = up256(rows * d * sizeof(float));
  l->cuts = l->ml + up256(rows * sizeof(float2));
  l->bytes = l->cuts + up256((size_t)grid * sizeof(int4));
  return MF_OK;
}

}  // namespace

extern "C" {

int mf_cache_append(const mf_cache_t* cache, const void* k, int64_t ld_k_in, const void* v, int64_t ld_v_in, int T,
                    const int32_t* seq, const int32_t* at, const int32_t* table, int64_t ld_table, int n_seqs,
                    int max_pages, const int32_t* positions, const uint64_t* turns, int rot_dim, int layout,
                    float gain, const void* k_weight, int norm, float eps, void* stream) {
  int rc = check_cache(cache);
  if (rc != MF_OK) return rc;
  const int d = cache->d;
  if (T < 0) return fail(MF_ERR_ARG, "T must be >= 0");
  if (rot_dim < 0 || rot_dim % 2 != 0 || rot_dim > d) return fail(MF_ERR_ARG, "rot_dim = %d must be even and in [0, %d]", rot_dim, d);
  if (layout != MF_ROPE_HALF && layout != MF_ROPE_INTERLEAVED) return fail(MF_ERR_ARG, "unknown layout %d", layout);
  if (norm != 0 && norm != 1) return fail(MF_ERR_ARG, "norm must be 0 or 1");
  if (norm && !(eps > 0.f && std::isfinite(eps))) return fail(MF_ERR_ARG, "eps must be positive and finite");
  if (!norm && k_weight) return fail(MF_ERR_ARG, "a weight without a norm");
  if (reinterpret_cast<uintptr_t>(k_weight) & 15) return fail(MF_ERR_ARG, "k_weight must be 16-byte aligned");
  if (rot_dim && !std::isfinite(gain)) return fail(MF_ERR_ARG, "gain must be finite");
  if (T == 0) return MF_OK;
  if ((rc = check_table(cache, table, ld_table, n_seqs, max_pages)) != MF_OK) return rc;
  if ((rc = check_aligned("seq", seq, 4)) != MF_OK) return rc;
  if ((rc = check_aligned("at", at, 4)) != MF_OK) return rc;
  if (positions && (rc = check_aligned("positions", positions, 4)) != MF_OK) return rc;
  if (rot_dim && (rc = check_aligned("turns", turns, 8)) != MF_OK) return rc;
  if ((rc = check_rows("k", k, ld_k_in, cache->H, d)) != MF_OK) return rc;
  if ((rc = check_rows("v", v, ld_v_in, cache->H, d)) != MF_OK) return rc;
  if (!clear_of(cache, k, ld_k_in, T) || !clear_of(cache, v, ld_v_in, T))
    return fail(MF_ERR_ARG, "k or v shares memory with the cache");
  if (cache->format == MF_CACHE_BF16 &&
      !rows_apart(cache->k, cache->ld_k, (int64_t)cache->H * d, cache->n_pages * cache->page_size, cache->v, cache->ld_v,
                  (int64_t)cache->H * d, cache->n_pages * cache->page_size))
    return fail(MF_ERR_ARG, "the cache's k and v share memory");
  const Read in[] = {{"seq", seq, T * 4ll}, {"at", at, T * 4ll}, {"table", table, table_bytes(ld_table, n_seqs, max_pages)},
                     {"positions", positions, T * 4ll}, {"turns", rot_dim ? turns : nullptr, rot_dim * 4ll},
                     {"k_weight", k_weight, d * 2ll}, {"k_scale", cache->k_scale, cache->H * 4ll},
                     {"v_scale", cache->v_scale, cache->H * 4ll}};
  if (cache->format == MF_CACHE_FP4) {
    if ((rc = check_apart("the cache", pages_span(cache), in)) != MF_OK) return rc;
  } else {
    const int64_t w = (int64_t)cache->H * d, rows = cache->n_pages * cache->page_size;
    if ((rc = check_apart("the cache's k", rows_span(cache->k, cache->ld_k, w, rows), in)) != MF_OK) return rc;
    if ((rc = check_apart("the cache's v", rows_span(cache->v, cache->ld_v, w, rows), in)) != MF_OK) return rc;
  }
  CacheParams p{};
  fill(&p, cache, seq, at, table, ld_table, n_seqs, max_pages);
  p.k_in = k;
  p.v_in = v;
  p.ld_kin = ld_k_in;
  p.ld_vin = ld_v_in;
  p.positions = positions ? positions : at;
  p.freq = reinterpret_cast<const unsigned long long*>(turns);
  p.rot = rot_dim;
  p.layout = layout;
  p.norm = norm;
  p.eps = eps;
  p.gain = gain;
  p.weight = k_weight;
  MF_CUDA(launch_cache_append(p, T, d, static_cast<cudaStream_t>(stream)), "cache append kernel");
  return MF_OK;
}

int mf_cache_read(const mf_cache_t* cache, int T, const int32_t* seq, const int32_t* at, const int32_t* table,
                  int64_t ld_table, int n_seqs, int max_pages, void* k_out, int64_t ld_k_out, void* v_out,
                  int64_t ld_v_out, void* stream) {
  int rc = check_cache(cache);
  if (rc != MF_OK) return rc;
  if (T < 0) return fail(MF_ERR_ARG, "T must be >= 0");
  if (T == 0) return MF_OK;
  if ((rc = check_table(cache, table, ld_table, n_seqs, max_pages)) != MF_OK) return rc;
  if ((rc = check_aligned("seq", seq, 4)) != MF_OK) return rc;
  if ((rc = check_aligned("at", at, 4)) != MF_OK) return rc;
  if ((rc = check_rows("k_out", k_out, ld_k_out, cache->H, cache->d)) != MF_OK) return rc;
  if ((rc = check_rows("v_out", v_out, ld_v_out, cache->H, cache->d)) != MF_OK) return rc;
  if (!clear_of(cache, k_out, ld_k_out, T) || !clear_of(cache, v_out, ld_v_out, T))
    return fail(MF_ERR_ARG, "k_out or v_out shares memory with the cache");
  const int64_t w = (int64_t)cache->H * cache->d;
  if (!rows_apart(k_out, ld_k_out, w, T, v_out, ld_v_out, w, T)) return fail(MF_ERR_ARG, "k_out and v_out share memory");
  const Read in[] = {{"seq", seq, T * 4ll}, {"at", at, T * 4ll}, {"table", table, table_bytes(ld_table, n_seqs, max_pages)},
                     {"k_scale", cache->k_scale, cache->H * 4ll}, {"v_scale", cache->v_scale, cache->H * 4ll}};
  if ((rc = check_apart("k_out", rows_span(k_out, ld_k_out, w, T), in)) != MF_OK) return rc;
  if ((rc = check_apart("v_out", rows_span(v_out, ld_v_out, w, T), in)) != MF_OK) return rc;
  CacheParams p{};
  fill(&p, cache, seq, at, table, ld_table, n_seqs, max_pages);
  p.k_out = k_out;
  p.v_out = v_out;
  p.ld_kin = ld_k_out;
  p.ld_vin = ld_v_out;
  MF_CUDA(launch_cache_read(p, T, cache->d, static_cast<cudaStream_t>(stream)), "cache read kernel");
  return MF_OK;
}

int mf_attn_paged_workspace(int Lq, int H_q, int H_kv, int d, int64_t* bytes) {
  if (!bytes) return fail(MF_ERR_ARG, "bytes is NULL");
  int rc = check_shape(Lq, H_q, H_kv, d);
  if (rc != MF_OK) return rc;
  PagedLayout l;
  if ((rc = paged_layout(Lq, H_q, H_kv, d, &l)) != MF_OK) return rc;
  *bytes = (int64_t)l.bytes;
  return MF_OK;
}

int mf_attn_paged(const mf_cache_t* cache, int n, int Lq, int H_q, const void* q, int64_t ld_q, const int32_t* table,
                  int64_t ld_table, int max_pages, const int32_t* lens, void* o, int64_t ld_o, float* lse,
                  const float* slopes, float softcap, int window, int n_sink, float scale, void* workspace,
                  int64_t workspace_bytes, void* stream) {
  int rc = check_cache(cache);
  if (rc != MF_OK) return rc;
  if (cache->format != MF_CACHE_FP4)
    return fail(MF_ERR_UNSUPPORTED, "attention over pages takes a 4-bit cache (over bf16 caches: mf_attn_cached)");
  if (n < 0) return fail(MF_ERR_ARG, "n must be >= 0");
  if (n > 1 << 20) return fail(MF_ERR_UNSUPPORTED, "more than 2^20 requests");
  if (window < 0) return fail(MF_ERR_ARG, "window must be >= 0 (0: none)");
  if (n_sink < 0) return fail(MF_ERR_ARG, "n_sink must be >= 0");
  if (!(scale > 1e-30f && scale < 1e30f)) return fail(MF_ERR_ARG, "scale must be positive and finite");
  if (!(softcap >= 0.f && softcap < 1e30f) || (softcap > 0.f && softcap < 1e-30f)) return fail(MF_ERR_ARG, "softcap must be positive and finite (0: none)");
  if (softcap > 0.f && !(scale / softcap > 1e-30f && scale / softcap < 1e30f)) return fail(MF_ERR_ARG, "scale / softcap is out of range");
  const int H = cache->H, d = cache->d;
  if ((rc = check_shape(Lq, H_q, H, d)) != MF_OK) return rc;
  if (n == 0) return MF_OK;
  if ((rc = check_table(cache, table, ld_table, n, max_pages)) != MF_OK) return rc;
  // (the kernel counts tiles of 32 keys, of one head in 32 bits)
  const long long lines = (long long)n * ((long long)max_pages * cache->page_size / 32 + 2);
  if (lines >= 1ll << 31 || lines * H * ((Lq * (H_q / H) + 15) / 16) >= 1ll << 37)
    return fail(MF_ERR_UNSUPPORTED, "%d requests of up to %lld keys: too many keys for one call", n, (long long)max_pages * cache->page_size);
  if ((rc = check_aligned("lens", lens, 4)) != MF_OK) return rc;
  if (lse && (rc = check_aligned("lse", lse, 4)) != MF_OK) return rc;
  if (slopes && (rc = check_aligned("slopes", slopes, 4)) != MF_OK) return rc;
  if ((rc = check_rows("q", q, ld_q, H_q, d)) != MF_OK) return rc;
  if ((rc = check_rows("o", o, ld_o, H_q, d)) != MF_OK) return rc;
  const int64_t w = (int64_t)H_q * d, rows = (int64_t)n * Lq;
  if (!rows_apart(q, ld_q, w, rows, o, ld_o, w, rows)) return shared("o", "q");
  if ((rc = check_aligned("workspace", workspace, 256)) != MF_OK) return rc;
  PagedLayout l;
  if ((rc = paged_layout(Lq, H_q, H, d, &l)) != MF_OK) return rc;
  if (workspace_bytes < (int64_t)l.bytes)
    return fail(MF_ERR_ARG, "workspace of %lld bytes, %lld are needed", (long long)workspace_bytes, (long long)l.bytes);
  const Span pages = pages_span(cache), qs = rows_span(q, ld_q, w, rows), os = rows_span(o, ld_o, w, rows);
  const Read in[] = {{"the cache", cache->k, (int64_t)(pages.b - pages.a)}, {"lens", lens, n * 4ll},
                     {"table", table, table_bytes(ld_table, n, max_pages)}, {"slopes", slopes, H_q * 4ll},
                     {"k_scale", cache->k_scale, H * 4ll}, {"v_scale", cache->v_scale, H * 4ll}};
  if ((rc = check_apart("o", os, in)) != MF_OK) return rc;
  const uintptr_t ls = reinterpret_cast<uintptr_t>(lse), wsp = reinterpret_cast<uintptr_t>(workspace);
  const Span lse_s = {ls, lse ? ls + rows * H_q * 4 : ls}, ws_s = {wsp, wsp + l.bytes};
  if ((rc = check_apart("workspace", ws_s, in)) != MF_OK) return rc;
  if (!apart(ws_s, qs)) return shared("workspace", "q");
  if (!apart(ws_s, os)) return shared("workspace", "o");
  if (lse) {
    if ((rc = check_apart("lse", lse_s, in)) != MF_OK) return rc;
    if (!apart(lse_s, qs)) return shared("lse", "q");
    if (!apart(lse_s, os)) return shared("lse", "o");
    if (!apart(lse_s, ws_s)) return shared("lse", "workspace");
  }
  PagedParams p{};
  p.pages = static_cast<const uint8_t*>(cache->k);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.n_pages = cache->n_pages;
  p.ps = cache->page_size;
  p.H_kv = H;
  p.G = H_q / H;
  p.inv_G = (65536 + p.G - 1) / p.G;
  p.table = table;
  p.ld_table = ld_table;
  p.max_pages = max_pages;
  p.lens = lens;
  p.slopes = slopes;
  p.q = q;
  p.o = o;
  p.ld_q = ld_q;
  p.ld_o = ld_o;
  p.lse = lse;
  p.n = n;
  p.Lq = Lq;
  p.window = window == 0 || window > kAttnNoWindow ? kAttnNoWindow : window;
  p.n_sink = n_sink > kAttnFar ? kAttnFar : n_sink;
  p.scale = scale;
  p.cap = softcap;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.part_o = reinterpret_cast<float*>(ws);
  p.part_ml = reinterpret_cast<float2*>(ws + l.ml);
  p.cuts = reinterpret_cast<int4*>(ws + l.cuts);
  p.rows = l.rows;
  MF_CUDA(launch_paged(p, d, static_cast<cudaStream_t>(stream)), "paged attention kernel");
  return MF_OK;
}

int mf_cache_append_args(const mf_cache_append_args_t* a) {
  if (!a) return fail(MF_ERR_ARG, "args is NULL");
  return mf_cache_append(a->cache, a->k, a->ld_k_in, a->v, a->ld_v_in, a->T, a->seq, a->at, a->table, a->ld_table, a->n_seqs,
                         a->max_pages, a->positions, a->turns, a->rot_dim, a->layout, static_cast<float>(a->gain),
                         a->k_weight, a->norm, static_cast<float>(a->eps), a->stream);
}

int mf_cache_read_args(const mf_cache_read_args_t* a) {
  if (!a) return fail(MF_ERR_ARG, "args is NULL");
  return mf_cache_read(a->cache, a->T, a->seq, a->at, a->table, a->ld_table, a->n_seqs, a->max_pages, a->k_out, a->ld_k_out,
                       a->v_out, a->ld_v_out, a->stream);
}

int mf_attn_paged_args(const mf_attn_paged_args_t* a) {
  if (!a) return fail(MF_ERR_ARG, "args is NULL");
  return mf_attn_paged(a->cache, a->n, a->Lq, a->H_q, a->q, a->ld_q, a->table, a->ld_table, a->max_pages, a->lens, a->o,
                       a->ld_o, a->lse, a->slopes, static_cast<float>(a->softcap), a->window, a->n_sink,
                       static_cast<float>(a->scale), a->workspace, a->workspace_bytes, a->stream);
}

}  // extern "C"
