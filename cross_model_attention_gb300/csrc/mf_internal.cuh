// mf_internal.cuh — shared host/device structures and kernel launchers of
// libmapflow (not part of the public ABI).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <atomic>
#include <cstdint>

namespace mf {

// One global block-row (a B-row block of one packed sequence).
struct RowBlock {
  int seq_start;  // first token of the sequence in the packed batch
  int L;          // sequence length
  int bi;         // block-row index within the sequence
  int cand_off;   // offset of this block-row's candidates in a head's mass row
};

// One 128-query-row tile of a sequence (the compressor's CTA unit).
struct RowTile {
  int seq_start;
  int L;
  int tl;   // tile index within the sequence (rows 128*tl .. 128*tl+127)
  int rb0;  // global block-row of the tile's first block-row
};

// One 64-row slab of a block-row (the retrieval's CTA unit).
struct RowSlab {
  int rb;    // global block-row
  int half;  // 0 for B = 64; 0/1 for B = 128
};

struct CompressParams {
  const RowBlock* rbs;
  const RowTile* tiles;
  int n_tiles;
  const int* items;  // pack order: [n_tiles * H_s] tile index << 8 | head, or null (tile-major)
  const int* stats_items;  // the two-CTA statistics kernel's order, same form, or null
  int T, H_s, H_ks, d, B, causal;
  int R;            // block-rows
  int C;            // candidates per head
  int max_cand;     // most candidates of one block-row
  float scale_log2; // log2(e) / sqrt(d)
  float p;
  // outputs / intermediates
  float* mass;      // [H_s][C]
  float* row_max;   // [H_s][T]  natural-log units
  float* row_sum;   // [H_s][T]
  int* kcount;      // [H_s*R]
  int* keptcols;    // [H_s][C]  per row: kept block columns, ascending
  int* row_ptr;     // [H_s*R + 1]
  int* col_idx;     // [nnz]
  int* tile_of;     // [C][H_s]  tile index of (block-row cand, head) or -1
  int* union_cnt;   // [R]
  int* union_list;  // [C]
  int* utile;       // [C][H_s]  tile_of in union order: row cand_off + j is union column j
  long long* nnz_out;  // device scalar
  int* pack_ctr;    // device scalar: the pack kernel's next item (reset by the selection kernel)
  int* sel_done;    // device scalar: selection CTAs finished (reset by the statistics kernel)
  uint16_t* zero_tile;  // the all-zero tile after the kept ones (bf16 pack writes it), or null
  uint32_t* kmask;  // [H_s*R][8] kept columns of each BSR row as bit masks (bf16 path), or null
  int union_in_pack;  // 1: the bf16 pack kernel writes union_cnt / union_list / utile
  int* err;
};

struct RetrieveParams {
  const RowBlock* rbs;
  const RowSlab* slabs;
  int n_slabs;
  int T, H_s, H_r, H_kv, d, B;
  int R, C;
  const int* tile_of;     // [C][H_s]
  const int* union_cnt;   // [R]
  const int* union_list;  // [C]
  const int* utile;       // [C][H_s] tile_of in union order
  const int* team_slabs;  // team retrieval: [n_teams][team_stride] slab indices, -1 padded
  int team_stride;
  const float* W;         // [H_r][H_s] of this receiver layer
  int zero_tile;          // index of an all-zero tile (= nnz)
  const uint16_t* values; // [nnz+1][B][B] bf16 tiles
  int* err;
};

// SM count of the current device, queried once per device.
inline cudaError_t sm_count(int* out) {
  static std::atomic<int> cache[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  int v = cache[dev].load(std::memory_order_relaxed);
  if (v == 0) {
    e = cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return e;
    cache[dev].store(v, std::memory_order_relaxed);
  }
  *out = v;
  return cudaSuccess;
}

// Calls `set` (a kernel's attribute) once per device; `done` is a static of
// the caller, one per kernel.
template <typename F>
cudaError_t once_per_device(std::atomic<unsigned long long>& done, F&& set) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (done.load(std::memory_order_acquire) >> dev & 1ull) return cudaSuccess;
  e = set();
  if (e == cudaSuccess) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

// Launches a kernel that may be set up while the one before it still runs: it loads
// and stores nothing before griddepcontrol.wait.  (Prefetches into L2 may come before:
// they bring no value, and L2 has what is still being written.)
template <typename P>
cudaError_t launch_early(void (*kernel)(P), dim3 grid, int threads, size_t smem, cudaStream_t s, const P& p) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// -------------------------------------------------------------- launchers --
// All return cudaError_t of the launch (cudaSuccess when enqueued).
// Head-map calibration: Gram matrix of the stacked head maps of two BSR
// layers over one block grid (rows 0..H_s-1 sender heads, then receiver heads).
constexpr int kCalibRows = 96;
struct CalibParams {
  const int* s_tile_of;      // sender [C][H_s] kept tile index or -1
  const uint16_t* s_values;  // sender tiles [.][B][B] bf16
  const int* r_tile_of;      // receiver [C][H_r]
  const uint16_t* r_values;
  int C, H_s, H_r, B;
  float* partial;            // [grid][kCalibRows][kCalibRows] per-CTA sums
  int* err;                  // device error word (bounded waits)
};
// CTAs for C candidate blocks (two per SM at most, none idle).
int calib_grid(int C);
// The Gram kernel, then the fixed-order fp64 sum of its partials into
// G [n][n], n = H_s + H_r.
cudaError_t launch_calib_gram(const CalibParams& p, int grid, double* G, cudaStream_t s);

// Statistics with two CTAs per SM (64-key S tiles) for rows of at most 128
// candidate blocks; tk64 boxes are 64 keys high.
bool stats2_supported(int max_cand);
cudaError_t launch_stats2_bf16(const CompressParams& p, const CUtensorMap& tq,
                               const CUtensorMap& tk64, cudaStream_t s);
cudaError_t launch_stats_bf16(const CompressParams& p, const CUtensorMap& tq,
                              const CUtensorMap& tk, cudaStream_t s);
cudaError_t launch_stats_f32(const CompressParams& p, const float* q, const float* k,
                             cudaStream_t s);
// Selection and, in its last CTA, the row_ptr scan.
cudaError_t launch_select(const CompressParams& p, cudaStream_t s);
cudaError_t launch_pack_bf16(const CompressParams& p, const CUtensorMap& tq,
                             const CUtensorMap& tk, const CUtensorMap& tvals,
                             cudaStream_t s);
cudaError_t launch_pack_f32(const CompressParams& p, const float* q, const float* k,
                            uint16_t* values, cudaStream_t s);
cudaError_t launch_union(const CompressParams& p, cudaStream_t s);
cudaError_t launch_retrieve_bf16(const RetrieveParams& p, const CUtensorMap& tp,
                                 const CUtensorMap& tv, void* o, cudaStream_t s);
// Team retrieval: persistent cooperative kernel, teams of 8 CTAs exchanging
// the combined maps through a ring in global memory (`ring` of
// retrieve_team_ring_bytes, `flags` of retrieve_team_flag_bytes, zeroed
// once: every launch leaves them at zero; `ta` maps the ring as
// retrieve_team_ring_rows x 64 bf16
// with boxes of 64 x retrieve_team_ring_box_rows).
bool retrieve_team_supported(int H_s, int H_r, int H_kv, int d, int B);
int retrieve_team_count(int n_slabs, int sms);
size_t retrieve_team_ring_bytes(int n_teams);
size_t retrieve_team_flag_bytes(int n_teams);
int retrieve_team_ring_box_rows(int H_r);
int retrieve_team_ring_rows(int n_teams);
cudaError_t launch_retrieve_team(const RetrieveParams& p, const CUtensorMap& ta,
                                 const CUtensorMap& tv, void* o, void* ring, uint32_t* flags,
                                 int n_teams, cudaStream_t s);
cudaError_t launch_retrieve_f32(const RetrieveParams& p, const uint16_t* values, const float* v,
                                float* o, cudaStream_t s);

// No-allocation selection (scratch in a static device array; mf_noalloc.cu).
size_t noalloc_scratch_bytes();
size_t noalloc_needed_bytes(long long R, long long H_s, long long C);
cudaError_t launch_select_noalloc(const RowBlock* rbs_host, int R, int C, int H_s, int B,
                                  int causal, float p, const float* mass, int* row_ptr,
                                  int* col_idx, long long* nnz, cudaStream_t s);

// Per-head norm of queries and keys with the rotary embedding (mf_rope.cu).
struct RopeParams {
  const void* q;
  const void* k;
  void* q_out;
  void* k_out;
  long long ld_q, ld_k, ld_qo, ld_ko;  // elements between tokens
  const void* q_weight;                // [d] or null (ones)
  const void* k_weight;
  const int* positions;                // [T]
  const unsigned long long* freq;      // [rot/2] turns per position, 64-bit fractions
  int H_q, H_k, rot;
  int layout;                          // 0: pairs (i, i + rot/2), 1: pairs (2i, 2i+1)
  int norm;
  float eps, gain;
  // set by the launcher: a token's heads in shares of heads_per_unit
  long long n_units;
  int heads_per_unit, q_chunks, k_chunks;
};
cudaError_t launch_rope(const RopeParams& p, long long T, int f32, int d, cudaStream_t s);

// Attention over packed sequences or caches (mf_attn_tc.cu).
constexpr int kAttnNoWindow = 1 << 30;  // a window that hides nothing
constexpr int kAttnCostPre = 1, kAttnCostCache = 2;  // a run's start and end, in key blocks
constexpr int kAttnSlotBits = 8192;     // of the map of requests with keys
constexpr int kAttnFar = 1 << 29;       // a row position past every key, and the most keys

// One run of key blocks of one query tile pair (packed form): what a CTA does
// between two loads of Q.  Keys are positions [0, a1) and [b0, b1) of a
// sequence, cut into blocks of 128 from each range's start.
struct alignas(16) AttnSeg {
  int q_row;       // first token's row in q and o
  int n_tok;       // tokens of the (one or two) tiles
  int pos;         // position of the first token in its sequence
  int k_row0;      // the sequence's first row in k and v
  int a1, b0, b1;
  int blk0, blk1;  // this run's blocks
  int head;        // KV head
  int part;        // partial result index, or -1: the run is whole and writes o
  int pad;
};
// One tile whose runs wrote partial results (packed form).
struct AttnJoin {
  int q_row, n_tok, head;
  int part0, n_part, step;
};

struct AttnParams {
  int H_q, H_kv, G, TQ;      // heads, heads per group, tokens per 128-row tile
  float scale;               // of the scores
  int window, n_sink;
  void* o;
  long long ld_o;
  float* lse;                // [rows of q][H_q] or null
  // packed form
  const AttnSeg* segs;
  const int* cta_segs;       // [grid + 1]
  // cache form
  const int* lens;           // [n] device
  int n, Lq, cap, P;
  int pre_pairs, pre_blocks; // prefix: pairs of row tiles (0: no prefix), key blocks
  int HG, groups;            // caches: KV heads per tile, tiles per request
  int grid;                  // CTAs of the launch
  int min_span;              // least work per CTA, in blocks
  int slot_shift;            // a bit of the map of requests with keys stands for 2^this of them
  int2* cuts;                // [units] how a unit's blocks are cut, written by its last run
  // partial results
  float* part_o;             // [row][d], not normalised
  float2* part_ml;           // [row]: reference (log2 units), sum
  // a run's results: slot part/2, each of its two streams 128 rows; those of a
  // cache's run from row suf_base on, suf_rows each
  long long suf_base;
  int suf_rows;
  int* err;
};
cudaError_t launch_attn_packed(const AttnParams& p, int d, int grid, const CUtensorMap& tq,
                               const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t s);
cudaError_t launch_attn_join(const AttnParams& p, int d, const AttnJoin* joins, int n_joins, cudaStream_t s);
cudaError_t launch_attn_cache(const AttnParams& p, int d, int grid, const CUtensorMap& tq,
                              const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tkp,
                              const CUtensorMap& tvp, const CUtensorMap& tqc, cudaStream_t s);

// A paged cache and the tokens that go in or come out (mf_cache.cu).
struct CacheParams {
  // the cache: 4-bit pages, or (pages null) bf16 rows of heads
  uint8_t* pages;
  void* k;
  void* v;
  long long ld_k, ld_v;        // elements between tokens
  const float* k_scale;        // [H] or null (ones)
  const float* v_scale;
  long long n_pages;
  int ps, H;                   // tokens of a page, heads
  // where the tokens are
  const int* seq;              // [T]
  const int* at;               // [T]
  const int* table;            // [n_seqs][max_pages], ld_table apart
  long long ld_table;
  int n_seqs, max_pages;
  // append
  const void* k_in;
  const void* v_in;
  long long ld_kin, ld_vin;    // (read: of k_out and v_out)
  const int* positions;        // [T]
  const unsigned long long* freq;
  int rot, layout, norm;
  float eps, gain;
  const void* weight;          // [d] or null (ones)
  // read
  void* k_out;
  void* v_out;
  // set by the launcher
  long long n_units;
  int heads_per_unit, shares;
  int even;                    // whether rows lie at multiples of 32 bytes
};
cudaError_t launch_cache_append(const CacheParams& p, long long T, int d, cudaStream_t s);
cudaError_t launch_cache_read(const CacheParams& p, long long T, int d, cudaStream_t s);

// Decoding attention over a paged cache in 4 bits (mf_paged.cu).
struct PagedParams {
  const uint8_t* pages;
  const float* k_scale;        // [H_kv] or null
  const float* v_scale;
  long long n_pages;
  int ps, H_kv, G;
  const int* table;            // [n][max_pages], ld_table apart
  long long ld_table;
  int max_pages;
  const int* lens;             // [n]
  const float* slopes;         // [H_q] or null
  const void* q;               // [n * Lq][H_q][d] bf16
  void* o;
  long long ld_q, ld_o;
  float* lse;                  // [n * Lq][H_q] or null
  int n, Lq, window, n_sink;
  unsigned inv_G;              // rr * inv_G >> 16 = rr / G for rr < 128
  float scale, cap;            // cap 0: none
  // workspace: a CTA's two partial results and a warp's one
  float* part_o;               // [grid * (2 + warps)][rows][d]
  float2* part_ml;             // [grid * (2 + warps)][rows]
  int4* cuts;                  // [grid]
  int rows;                    // of a partial result
  float inv_grid;              // set by the launcher: 1 / CTAs, rounded up
};
// What a launch takes: CTAs, partial results and rows of one.
void paged_shape(int Lq, int G, int sms, int* grid, int* parts, int* rows);
cudaError_t launch_paged(const PagedParams& p, int d, cudaStream_t s);
cudaError_t launch_selftest_wait(int* err, unsigned long long limit_ns, cudaStream_t s);

}  // namespace mf
