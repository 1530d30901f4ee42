// Internal interface between the host side of the calls over a step's device
// arrays (sparse.cpp) and their kernels (k_tables.cu, k_mapped.cu, k_bounds.cu,
// k_block_select.cu, k_sparse.cu, k_sparse_mma.cu, k_sparse_tc.cu).  Plain structs of device pointers and sizes;
// no torch types.
#pragma once

#include <cuda.h>

#include "gp_kernels.h"

namespace gp {

// The arrays of a step (gp_step) and the sizes that the kernels hold them to:
// what they find there is checked on the device, nothing of it is known here.
struct StepArgs {
  int n, max_rows;
  const int32_t* slots;      // [n]
  const int32_t* cached;     // [n]
  const int32_t* row0;       // [n + 1]
  const int32_t* row_req;    // [max_rows], -1: no row
  const int32_t* tables;     // [M][maxp]
  int M, maxp;
  int num_pages_total;
  int* err;
};

// ---- block tables, slot map and positions ------------------------------------
constexpr int kStepMaxRequests = 4096;  // the scans' arrays stay in shared memory
constexpr int kStepMaxSlots = 1 << 18;  // two bits a slot there
struct TablesArgs {
  int n, max_rows, num_free, M, maxp, num_pages_total;
  const int32_t *slots, *cached, *fresh;
  const int64_t* pos;
  const int32_t* held;       // [M]
  const int32_t* free_pages; // [num_free]
  const int32_t* taken_in;   // [1] or null
  int32_t *tables, *num_pages, *row0, *row_req, *state, *taken;
  int64_t *slot_map, *positions;
  int* err;
  bool apart;                // num_pages is not held, taken not taken_in
};

// ---- rotary forms, through the slot map ----------------------------------------
struct MappedArgs {
  int rows;                  // of the buffers
  const int64_t* slot_map;
  const int64_t* positions;
  void *k_cache, *v_cache;
  int kv_f32, q_f32;
  int num_pages_total, layer, Hq, Hkv, D;
  const void *q, *k, *v;     // rows of heads, `*_row` elements apart
  int64_t q_row, k_row, v_row;
  void* q_rot;               // [rows][Hq][D], may be q when that is packed
  int rotary_dim;            // of a head, a multiple of 16
  int interleaved;
  float amplitude;           // of cosine and sine
  int* err;
  double inv_freq[64];       // [rotary_dim / 2]
};

// ---- bounds of the blocks -------------------------------------------------------
struct BoundsArgs {
  StepArgs s;
  const void* k_cache;
  int kv_f32, layer, Hkv, D, block;
  int8_t* bounds;            // [L][pages][Hkv][256 / block][2][D]
  float* scales;             // [L][pages][Hkv][256 / block]
};

// ---- blocks by score --------------------------------------------------------------
struct SelectBlocksArgs {
  StepArgs s;
  int layer, Hq, Hkv, D, q_f32, block, top, sink, recent;
  const void* q;             // [max_rows][Hq][D]
  const int8_t* bounds;
  const float* scales;
  int32_t* blocks;           // [max_rows][Hkv][top]
  int rows;                  // of a tile: 8, or 16 while their scores fit kSelectShared
  int splits;                // CTAs of a cluster that share a tile's blocks
};
constexpr int kSelectShared = 64 * 1024;

// ---- attention over listed blocks ---------------------------------------------------
struct SparseArgs {
  StepArgs s;
  const void *k_cache, *v_cache;
  int kv_f32, q_f32;
  int layer, Hq, Hkv, D, block, top;
  const void* q;             // [max_rows][Hq][D]
  const int32_t* blocks;     // [max_rows][Hkv][top]
  void* out;                 // [max_rows][Hq][D], q's type
  int splits;                // CTAs of a cluster that share the blocks of a row or piece
  long long wait_limit;      // clock cycles a wait may take before the CTA gives up
};

cudaError_t launch_tables(const TablesArgs& a, cudaStream_t s);
cudaError_t launch_mapped(const MappedArgs& a, cudaStream_t s);
cudaError_t launch_bounds(const BoundsArgs& a, cudaStream_t s);
cudaError_t launch_select_blocks(const SelectBlocksArgs& a, cudaStream_t s);
// Pieces of T rows that a launch has room for (step.cuh).
inline int sparse_pieces(const StepArgs& s, int T) { return s.max_rows / T + s.n; }

// K and V as 2-D tensors of key rows, boxes of 64 dimensions by a block (64 rows of
// one that is larger).
struct SparseMaps {
  CUtensorMap k, v;
};
cudaError_t launch_sparse(const SparseArgs& a, cudaStream_t s);
// bf16 caches and queries: a few rows of a request at a time, and many
cudaError_t launch_sparse_mma(const SparseArgs& a, const SparseMaps& maps, cudaStream_t s);
cudaError_t launch_sparse_tc(const SparseArgs& a, const SparseMaps& maps, const CUtensorMap& qmap, cudaStream_t s);
constexpr int kSparseMmaRows = 16;  // of the products: 16 / G rows of a request
constexpr int kSparseTcRows = 128;  // qmap's box: 64 dimensions of G heads of 128 / G rows

}  // namespace gp
