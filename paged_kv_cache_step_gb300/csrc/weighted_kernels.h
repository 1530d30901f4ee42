// Internal interface between the host side of the accumulated-weight
// operators (weighted.cpp) and their kernels (k_append.cu, k_weights.cu,
// k_chunk.cu, k_chunk_tc.cu, k_evict.cu).  Plain structs of device pointers
// and sizes; no torch types.
//
// The accumulated weights are the caller's: fp32 [L][M][Hkv][cap], by request
// slot and logical token, cap = max_pages_per_req * 256.
#pragma once

#include "gp_kernels.h"

namespace gp {

// ---- new tokens into the cache (RoPE, pages, weights cleared) ---------------
struct AppendReq {
  int64_t pos;     // RoPE position of the first new token
  int64_t row0;    // its row in the packed inputs
  int32_t cached;  // its logical slot
  int32_t nnew;    // tokens, at least one
  int32_t slot;    // request slot (row of the weights)
  int32_t bt_off;  // pages of the logical blocks cached / 256, ...
};

struct AppendArgs {
  void* k_cache;
  void* v_cache;
  int kv_f32, q_f32;
  int num_pages_total;
  int layer, Hq, Hkv, D, M;
  int64_t cap;               // tokens of a row of the weights
  const AppendReq* reqs;     // [n], row0 ascending; null: `few`
  const int32_t* bt;
  int n;
  int rows;                  // packed rows
  const void* q;             // [rows][Hq][D] or null
  const void* k;             // [rows][Hkv][D]
  const void* v;             // [rows][Hkv][D]
  void* q_rot;               // [rows][Hq][D], may be q
  float* weights;            // or null
  const double* inv_freq;    // [D / 2]
  int* err;
  // the descriptors of a small call travel with the launch: no copy before it,
  // and constant-bank reads instead of dependent trips to L2.  One token each of 1,
  // 8, 32 and 64 requests, 32 and 8 heads of 128: 7.6, 8.1, 10.5 and 13.0 us a call,
  // 12.4, 13.2, 15.5 and 18.1 with the copy.  The launch's parameters grow with the
  // limit, whatever the call: room for 256 requests takes 65 to 256 of them from
  // 18.1 - 32.5 to 13.7 - 28.8 us, and adds up to 0.6 us to the others.
  static constexpr int FEW_REQS = 64, FEW_PAGES = 128;
  AppendReq few[FEW_REQS];
  int32_t few_bt[FEW_PAGES];
};
cudaError_t launch_append(const AppendArgs& a, cudaStream_t s);

// ---- one decode step's weights from the logits the attention kernel kept ----
struct WeightReq {
  int64_t logit_off;  // float offset of the request's logits [Hkv][pages * 256][G]
  int32_t page0;      // pages of the requests before it
  int32_t ntok;
  int32_t slot;
  int32_t pad;
};
static_assert(sizeof(WeightReq) == 24, "uploaded as it is");

struct WeightArgs {
  const WeightReq* reqs;  // [n], page0 ascending
  int n;
  int pages;              // of all requests
  int layer, Hq, Hkv, G, M;
  int64_t cap;
  const float* logits;    // base 2
  const float2* stat;     // [n][Hq] (maximum, 1 / sum)
  float* weights;
  int* err;
};
cudaError_t launch_decode_weights(const WeightArgs& a, cudaStream_t s);

// ---- eviction by accumulated weight -----------------------------------------
struct EvictReq {
  int32_t slot;
  int32_t T, keep, recent;  // tokens, tokens kept, of them the most recent
  int32_t bt_off;
  int32_t items;            // move items of a unit: ceil(keep / rows of an item), 0 when T <= keep
  int32_t idx_pitch;        // keep, rounded up to 8
  int64_t idx_off;          // offset of the kept slots [units][idx_pitch]
  int64_t item0;            // items of the requests before it (all units)
  int64_t pre_off;          // offset of the kept-slot counts [units][items + 1]
};

struct EvictArgs {
  void* k_cache;
  void* v_cache;
  int num_pages_total;
  int L, Hkv, M, row_bytes;
  int64_t cap;
  const EvictReq* reqs;       // [n]
  int n;
  const int32_t* old_bt;
  const int32_t* new_bt;
  float* weights;
  uint16_t* idx;              // kept slot of each rank
  int32_t* pre;               // kept slots below every item's first slot
  unsigned* flags;            // [items of all units], 1: the item's rows are read
  unsigned long long* ticket; // next item
  int64_t items;              // of all requests
  int longest;                // most tokens of a request that evicts
  int sms;
  unsigned long long* moved;
  int* err;
  long long wait_limit;
};
// Rows of a move item: K rows of 8 KB.
__host__ __device__ constexpr int evict_rows(int row_bytes) { return 8192 / row_bytes; }
cudaError_t launch_evict_select(const EvictArgs& a, cudaStream_t s);
cudaError_t launch_evict_move(const EvictArgs& a, cudaStream_t s);

// ---- causal attention of several new tokens a request -----------------------
struct ChunkReq {
  int64_t row0;    // packed row of the first new token
  int32_t cached;  // tokens before it
  int32_t nnew;
  int32_t slot;
  int32_t bt_off;
};

// CUDA-core kernels: a tile of 64 query rows (64 / G tokens of the G heads of
// a KV head), a tile of 64 keys.  An item is a query tile and key tiles
// [from, to) of it, or (weights) a key tile and query tiles [from, to).
struct ChunkTile {
  int32_t r, h, first;  // request, KV head, first token of the rows (or first key)
  int32_t from, to;
  int32_t part;         // partial, -1: the result directly
  int32_t pad[2];
};
struct ChunkTileJoin {
  int32_t r, h, first;  // as above
  int32_t part, n;      // its partials
  int32_t pad[3];
};
constexpr int CHUNK_ROWS = 64, CHUNK_KEYS = 64;

struct ChunkArgs {
  const void* k_cache;
  const void* v_cache;
  int kv_f32, q_f32;
  int num_pages_total;
  int layer, Hq, Hkv, D, G, M;
  int64_t cap;
  const ChunkReq* reqs;
  int n;
  const int32_t* bt;
  const ChunkTile* tiles;   // of the attention
  int n_tiles;
  const ChunkTileJoin* joins;
  int n_joins;
  const ChunkTile* wtiles;  // of the weights
  int n_wtiles;
  const ChunkTileJoin* wjoins;
  int n_wjoins;
  float* part;              // partial outputs [64][D], 64 maxima, 64 sums each
  float* wpart;             // partial weights [64] each
  const void* q;            // [rows][Hq][D], rotated
  void* out;                // [rows][Hq][D] in q's type
  float2* stat;             // [rows][Hq] (maximum, 1 / sum) of the base-2 logits
  float* weights;           // or null
  int* err;
};
__host__ __device__ constexpr size_t chunk_tile_part_floats(int D) { return (size_t)CHUNK_ROWS * (D + 2); }
cudaError_t launch_chunk(const ChunkArgs& a, cudaStream_t s);
cudaError_t launch_chunk_weights(const ChunkArgs& a, cudaStream_t s);

// Tensor-core kernels (bf16 caches and queries).  A query tile is 128 rows,
// 128 / G tokens of the G heads; a key tile 128 slots.
//
// Attention: an item is a range of key tiles for either two query tiles that
// follow each other (the second may be missing), or (kitems) one query tile
// whose even key tiles go to the first softmax group and the odd ones to the
// second.
struct ChunkItem {
  int32_t r, h, t0;      // request, KV head, first token
  int32_t alone;         // of a pair: there is no second query tile
  int32_t kb, ke;        // key tiles
  int32_t part_a, part_b;// partial of each group, -1: its output directly
};
static_assert(sizeof(ChunkItem) == 32, "two 16-byte loads");
// A query tile whose partials are joined.
struct ChunkJoin {
  int32_t r, h, t0, first, n, pad[3];
};
// Weights: an item is one or more pages (256 keys each), one after the other,
// against a range of query tiles.
struct WeightItem {
  int32_t r, h, page, pages;
  int32_t qb, qe;        // query tiles
  int32_t part;          // partial (of a single page), -1: added to the weights directly
  int32_t pad;
};
struct WeightJoin {
  int32_t r, h, page, first, n, pad[3];
};

struct ChunkTcArgs {
  CUtensorMap kmap, vmap;  // caches as [rows][D], box 64 x 128, 128-byte swizzle
  CUtensorMap qmap;        // queries as [rows][Hq][D], box 64 x G x 128 / G
  int num_pages_total;
  int layer, Hq, Hkv, D, G, M;
  int64_t cap;
  const ChunkReq* reqs;
  const int32_t* bt;
  const ChunkItem* items;      // CTA c takes [begin[c], begin[c + 1])
  const int32_t* begin;
  int grid;
  const ChunkItem* kitems;     // the same of the items of one query tile
  const int32_t* kbegin;
  int kgrid;
  const ChunkJoin* joins;
  int n_joins;
  const WeightItem* witems;
  const int32_t* wbegin;
  int wgrid;
  const WeightJoin* wjoins;
  int n_wjoins;
  void* out;                   // [rows][Hq][D] bf16
  float* lse;                  // [rows][Hq] base-2 log of the softmax's sum, or null
  float* weights;
  float* part;                 // partial outputs, chunk_part_floats(D) each
  float* wpart;                // partial weights, 256 each
  int* err;
  long long wait_limit;        // clock cycles
};
// A partial: outputs [D / 4][128 rows][4], then 128 maxima, then 128 sums.
__host__ __device__ constexpr size_t chunk_part_floats(int D) { return (size_t)128 * (D + 2); }
inline bool chunk_tc_shape(int D, int G) { return (D == 64 || D == 128) && (G == 2 || G == 4); }
cudaError_t launch_chunk_tc(const ChunkTcArgs& a, cudaStream_t s);
cudaError_t launch_chunk_weights_tc(const ChunkTcArgs& a, cudaStream_t s);

}  // namespace gp
