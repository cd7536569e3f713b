// Launch entries of the key/value cache and its attention.
#pragma once

#include <cstddef>

#include "kv_layout.hpp"
#include "launch.hpp"

namespace nvfp4 {

// kvcache.hip: rotate q and k, quantize k and v, write them to their cache slots
// (rows without a slot are skipped), and read rows back as values.
struct KvAppendArgs {
  const void* q;               // n_q_heads == 0: none
  const void* k;
  const void* v;
  int64_t ldq, ldk, ldv, ldqo, T;
  int32_t n_q_heads;
  const float* cos;
  const float* sin;
  int64_t n_pos;
  int32_t rot_dim;
  int32_t interleaved;
  const int32_t* positions;
  const int64_t* slots;
  uint8_t* cache;
  KvGeom geom;
  const float* k_gscale;
  const float* v_gscale;
  void* q_out;
};
hipError_t launch_rope_append(const KvAppendArgs& a, InType t, int32_t D, hipStream_t s);

struct KvGatherArgs {
  const uint8_t* cache;
  KvGeom geom;
  const int64_t* slots;
  int64_t T;
  const float* k_gscale;
  const float* v_gscale;
  void* k_out;
  void* v_out;
  int64_t ldk, ldv;
};
hipError_t launch_kv_gather(const KvGatherArgs& a, InType t, int32_t D, hipStream_t s);

// kvevict.hip: rows that move within a sequence's pages.
struct KvPages {
  const int32_t* table;
  int64_t max_pages, ld_table; // table row: max_pages entries, ld_table apart
  KvGeom geom;
  int32_t batch;
};
constexpr int kKvMoveThreads = 1024;
constexpr int kKvMostAccepted = 256;
struct KvAcceptArgs {
  uint8_t* cache;
  KvPages pages;
  const int32_t* kv_len;
  const int32_t* cu_q;         // NULL: one query token per sequence
  const int32_t* accepted;     // [batch][ld_accepted]
  int64_t ld_accepted;
  int32_t max_accepted;
  const int32_t* n_accepted;
  int32_t* kv_len_out;
};
hipError_t launch_kv_accept(const KvAcceptArgs& a, int32_t D, hipStream_t s);

struct KvEvictArgs {
  uint8_t* cache;
  KvPages pages;
  const int32_t* kv_len;
  const float* weights;        // [n_pages][n_kv_heads][page_size]
  float* weights_out;          // optional; may be weights
  int32_t budget, first, last;
  int32_t* kept;               // optional [batch][n_kv_heads][budget]
  int32_t* kv_len_out;
  int32_t* lists;              // [rows][2][budget]: what moves, and where to (workspace)
  int32_t* moving;             // [rows]: entries of the lists (workspace)
  void* counts;                // of the rows, and of their parts (workspace)
  // the plan
  int32_t rows;                // batch * n_kv_heads
  int32_t lengths;             // whether the kernels write the lengths
  int32_t parts;               // of a row; 0: a workgroup does a whole one
  int32_t move_parts;          // for what moves; 0: the same workgroup moves it
};
constexpr int kKvEvictMostParts = 64;              // of a row
constexpr int kKvEvictRowBytes = 20736;            // that a row's parts count
constexpr int kKvEvictPartBytes = 8448;            // and each of them
struct KvEvictPlan {
  int32_t parts;
  int64_t moving_at, counts_at;   // byte offsets in the workspace
  int64_t workspace;           // bytes
};
KvEvictPlan kv_evict_plan(int32_t batch, int32_t n_kv_heads, int64_t budget, int64_t max_kv_len);
hipError_t launch_kv_evict(KvEvictArgs a, int32_t D, const KvEvictPlan& p, int64_t max_kv_len, void* workspace, hipStream_t s);

// kvattn.hip: attention over the cache.
struct KvAttnArgs {
  const void* q;
  int64_t ldq, T;
  int32_t n_q_heads, batch;
  const int32_t* cu_q;         // NULL: one token per sequence
  const int32_t* kv_len;
  const int32_t* table;
  int64_t max_pages, ld_table; // table row: max_pages entries, ld_table apart
  const uint8_t* cache;
  KvGeom geom;
  const float* k_gscale;
  const float* v_gscale;
  float scale;
  int32_t window;              // 0 = none
  void* o;
  int64_t ldo;
  float* lse;                  // optional
  float* part;                 // partial results (workspace)
  // the plan
  void* pieces;                // [blocks] items done in pieces
  int32_t n_workers;           // 0: one workgroup per item; else items are cut into pieces
  int32_t blocks;              // workgroups
  int32_t min_steps;           // of a piece
  int32_t tile_cols;           // query columns of an item
  int32_t col_tiles;           // items per sequence and kv head
  FastDiv by_group, by_heads, by_tile_cols, by_col_tiles, by_pairs;   // pairs: sequence, kv head
  // Last, so that what causal calls read lies in 256 bytes, four lines of the kernel's arguments (with a fifth,
  // 1 x 257 keys 6.7 us, not 6.5)
  const uint64_t* tree;        // NULL: causal; else the query rows' bits over their sequence's query tokens
  int64_t ld_tree;             // words from row to row
  int32_t tree_words;
};
static_assert(offsetof(KvAttnArgs, tree) <= 256, "causal calls' arguments: four lines");
constexpr int kItemPiecesBytes = 32;
constexpr int kMaxTreeWords = 64;
struct KvAttnPlan {
  int32_t n_workers, blocks, min_steps, tile_cols, col_tiles, nq;
  bool prefill;                // kvprefill.hip
  int64_t pieces_at;           // byte offset in the workspace
  int64_t workspace;           // bytes
};
KvAttnPlan kv_attn_plan(InType t, int64_t T, int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t D,
                        int64_t max_q_len, int64_t max_kv_len, int64_t window, bool tree);
// bytes for a call of these sizes, of a tree or not, with any window
int64_t kv_attn_workspace(InType t, int64_t T, int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t D,
                          int64_t max_q_len, int64_t max_kv_len);
hipError_t launch_kv_attn(KvAttnArgs a, const KvAttnPlan& p, InType t, int32_t D, hipStream_t s);

// kvweights.hip: the attention weight of cached tokens
struct KvWeightsArgs {
  const float* lse;            // [T][n_q_heads]
  float* weights;              // [n_pages][n_kv_heads][page_size]
  float decay;
  // the plan
  int32_t tiles;               // workgroups per sequence and kv head
  int32_t steps;               // few query columns: 64 tokens each, of a wave's run
  int32_t split;               // many: log2 of the waves that share tokens; few: minus the
                               // blocks of 16 columns that a wave holds
  FastDiv by_tiles;
  // last, so that the tree's fields are behind all that is read (3 x 37 to 300 new fp32 tokens 17.9 us, 17.5)
  KvAttnArgs a;                // its queries, pages and scale; o, lse, plan unused
};
constexpr int64_t kKvWeightsMostLd = 1 << 23;      // elements between query rows: a tile's offsets have 32 bits
hipError_t launch_kv_weights(KvWeightsArgs w, InType t, int32_t D, int64_t max_q_len, int64_t max_kv_len, hipStream_t s);

// joins the pieces that either kernel left
hipError_t launch_kv_join(const KvAttnArgs& a, InType t, int32_t D, hipStream_t s);

// kvprefill.hip: bf16, items of kv_prefill_cols() query columns, a workgroup of
// kv_prefill_threads() each.
int32_t kv_prefill_cols();
int32_t kv_tree_cols(int32_t D);   // columns from which drafted trees go there, 128 at a time up to 128
int32_t kv_prefill_threads();
hipError_t launch_kv_prefill(const KvAttnArgs& a, int32_t D, hipStream_t s);

}  // namespace nvfp4
