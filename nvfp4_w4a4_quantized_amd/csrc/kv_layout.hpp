// Layout of the paged NVFP4 key/value cache, shared by the kernels that write and
// read it.
//
// A page holds page_size tokens (a power of two, at least 16) of every kv head as
// [head][page_size / 16] granules of 16 tokens; a granule is 18 D bytes:
//   K codes   [16 tokens][D/2]              at 0
//   K scales  [16 tokens][D/16]             at 8 D
//   V codes   [4 quads][16][4 tokens][D/32] at 9 D   (a token's D/2 bytes in 16 parts)
//   V scales  [4 quads][D/16][4 tokens]     at 17 D
// The order is the one in which the matrix instructions take their operands, so that
// every load of the attention kernels is a whole contiguous piece of a granule: lane
// (g = lane / 16, r = lane % 16) of a 16-row MFMA reads key row r at its g-th quarter
// of the elements, and for the values (transposed: rows are elements, the K axis is
// tokens) part r of the four tokens of quad g, 16 bytes at D = 128.  Each code byte
// holds two elements of ONE token, and each token has its own scale bytes, so that
// appending a token writes whole bytes and never touches its neighbours'.
#pragma once

#include <stdint.h>

namespace nvfp4 {

constexpr int kv_granule_bytes(int D) { return 18 * D; }

// Division of n in [0, 2^31) by a divisor known on the host: n m >> (31 + L) with L =
// ceil(log2 d), m = floor(2^(31+L) / d) + 1 (the product exceeds n / d by less than 2^-L <= 1 / d).
// On the device a division costs some 30 dependent instructions, and a single-token call
// makes ten before its first load.
struct FastDiv {
  uint32_t d, m, s;
};

inline FastDiv fast_div(uint32_t d) {
  uint32_t l = 0;
  while ((1ull << l) < d) ++l;
  return FastDiv{d, (uint32_t)((1ull << (31 + l)) / d + 1), 31 + l};
}

#ifdef __HIPCC__
__host__ __device__
#endif
inline int32_t operator/(int32_t n, const FastDiv& f) {
  return (int32_t)(((uint64_t)(uint32_t)n * f.m) >> f.s);
}

struct KvGeom {
  int32_t n_kv_heads;
  int32_t page_shift;      // log2(page_size)
  int64_t page_bytes;      // n_kv_heads * page_size * D * 9 / 8
  int64_t n_pages;
};

inline bool kv_shape_ok(int32_t D, int32_t page_size) {
  return (D == 64 || D == 128 || D == 256) && page_size >= 16 && page_size <= 4096 &&
         (page_size & (page_size - 1)) == 0;
}

inline int64_t kv_page_bytes(int32_t n_kv_heads, int32_t page_size, int32_t D) {
  return (int64_t)n_kv_heads * page_size * D * 9 / 8;
}

// Workgroups of `threads` that one launch may have: HIP counts a grid's threads in 32 bits and
// refuses more.
inline int64_t kv_most_blocks(int32_t threads) { return 0xFFFFFFFFll / threads; }

// Workgroups (256 threads) that append or read `heads` rows of each of T tokens: a wave takes
// 64 / (D / 16) tokens of one head.
constexpr int kKvRowThreads = 256;
inline int64_t kv_row_blocks(int64_t T, int64_t heads, int32_t D) {
  const int64_t per_wave = 64 / (D / 16), per_block = kKvRowThreads / 64;
  return ((T + per_wave - 1) / per_wave * heads + per_block - 1) / per_block;
}

// Column tiles that the attention's grid has for each of `pairs` (sequence, kv head), at most
// 2^22 of them, where the bounds on the lengths ask for `tiles`.  Any number is right (the kernels
// take further tiles with the planned ones), and bounds far above the lengths ask for too many.
inline int32_t kv_planned_tiles(int64_t tiles, int64_t pairs, int32_t threads) {
  const int64_t most = kv_most_blocks(threads) / pairs;
  return (int32_t)(tiles < most ? tiles : most);
}

}  // namespace nvfp4
