// Launch entries of the key/value cache and its attention.
#pragma once

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
  const uint64_t* tree;        // NULL: causal; else the query rows' bits over their sequence's query tokens
  int64_t ld_tree;             // words from row to row
  int32_t tree_words;
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
};
constexpr int kItemPiecesBytes = 32;
constexpr int kMaxTreeWords = 64;
struct KvAttnPlan {
  int32_t n_workers, blocks, min_steps, tile_cols, col_tiles, nq;
  bool prefill;                // kvprefill.hip
  int64_t pieces_at;           // byte offset in the workspace
  int64_t workspace;           // bytes
};
KvAttnPlan kv_attn_plan(InType t, int64_t T, int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t D,
                        int64_t max_q_len, int64_t max_kv_len, int64_t window);
hipError_t launch_kv_attn(KvAttnArgs a, const KvAttnPlan& p, InType t, int32_t D, hipStream_t s);

// joins the pieces that either kernel left
hipError_t launch_kv_join(const KvAttnArgs& a, InType t, int32_t D, hipStream_t s);

// kvprefill.hip: bf16, items of kv_prefill_cols() query columns, a workgroup of
// kv_prefill_threads() each.
int32_t kv_prefill_cols();
int32_t kv_prefill_threads();
hipError_t launch_kv_prefill(const KvAttnArgs& a, int32_t D, hipStream_t s);

}  // namespace nvfp4
