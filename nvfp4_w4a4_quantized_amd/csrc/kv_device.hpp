// Device helpers of the attention kernels over the NVFP4 key/value cache.
#pragma once

#include "kernel_common.hpp"
#include "kv_launch.hpp"

namespace nvfp4 {
namespace {

constexpr float kNegBig = -3.402823466e38f;   // reference M of a row that has seen nothing: the lowest fp32
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Joined with the lane 32 (16) away, by a swap of the halves (of the rows of 16) with itself
__device__ __forceinline__ float max_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float max_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __builtin_fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ __forceinline__ float sum_xor32(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float sum_xor16(float x) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Largest of the results of one MFMA, or of N of them, by v_max3_f32 (fmaxf gets a canonicalizing
// max per value).  The compiler does not count the wait states between an MFMA and an asm that
// reads its result, so the asm takes its first operand from ordinary maxima that read a result of
// every one of the MFMAs: those wait, and what an MFMA writes is all there when any of it is.
__device__ __forceinline__ float max_of(const f32x16& x) {
  float m = __builtin_fmaxf(x[0], x[15]);
#pragma unroll
  for (int i = 1; i + 1 < 16; i += 2) asm("v_max3_f32 %0, %0, %1, %2" : "+v"(m) : "v"(x[i]), "v"(x[i + 1]));
  return m;
}
template <int N>
__device__ __forceinline__ float max_of(const f32x4 (&x)[N]) {
  static_assert(N % 2 == 0, "pairs");
  float m = __builtin_fmaxf(x[0][0], x[1][0]);
#pragma unroll
  for (int u = 2; u < N; ++u) m = __builtin_fmaxf(m, x[u][0]);
#pragma unroll
  for (int u = 0; u < N; u += 2)
#pragma unroll
    for (int i = 1; i < 4; ++i) asm("v_max3_f32 %0, %0, %1, %2" : "+v"(m) : "v"(x[u][i]), "v"(x[u + 1][i]));
  return m;
}

// Two fp32 -> two f16, round to nearest even
__device__ __forceinline__ f16x2 to_f16(float a, float b) { return f16x2{(_Float16)a, (_Float16)b}; }

// Query rows enter the f16 product scaled by 2^(14 - e), amax of the row in [2^e, 2^(e+1)), and
// their scores are scaled back; rows below 2^-100 stay near zero.
__device__ __forceinline__ int query_exponent(float amax) {
  const int e = (int)((__float_as_uint(amax) >> 23) & 255u) - 127;
  return e < -100 ? -100 : e;
}
__device__ __forceinline__ float query_up(float amax) {
  return __uint_as_float((uint32_t)(14 - query_exponent(amax) + 127) << 23);
}
// What a product of the scaled query (negated where the scale is negative) and a stored key
// counts in a base-2 exponent: positive, so that the largest product is the largest score and
// a product masked with -inf stays masked.
__device__ __forceinline__ float score_factor(float scale, float kg, float amax) {
  const float down = __uint_as_float((uint32_t)(query_exponent(amax) - 14 + 127) << 23);
  return __builtin_fmaxf(__builtin_fabsf(scale) * kLog2e * kg * down, 0x1p-120f);
}

// The exponent fma(product, factor, -M) is exact but for M, which is the largest score, rounded:
// off by 1 where scores reach 2^24 (then weights pass f16's range), by anything beyond.  Products
// stay below 2^15 * 2688 * 256 < 2^35, so columns whose factor is at most this one have scores
// below 2^23; a wave that holds another ("wide") multiplies its products by their factors first
// and goes on with a factor of 1, so that scores and M round alike.
constexpr float kWideFactor = 0x1p-12f;

// What a workgroup needs of its sequence
struct SeqInfo {
  int32_t q0;              // first query token (row of q)
  int32_t m;               // query tokens
  int32_t n;               // cached tokens
};

__device__ __forceinline__ SeqInfo seq_info(const KvAttnArgs& a, int b) {
  SeqInfo s;
  int64_t q0 = b, q1 = b + 1;
  if (a.cu_q) {
    q0 = a.cu_q[b];
    q1 = a.cu_q[b + 1];
  }
  q0 = q0 < 0 ? 0 : (q0 > a.T ? a.T : q0);
  q1 = q1 < q0 ? q0 : (q1 > a.T ? a.T : q1);
  s.q0 = (int32_t)q0;
  s.m = (int32_t)(q1 - q0);
  const int64_t most = a.max_pages << a.geom.page_shift;
  const int64_t n = a.kv_len[b];
  s.n = (int32_t)(n < 0 ? 0 : (n > most ? most : n));
  return s;
}

// The tokens that query columns [col0, col1) of a sequence attend to, as one range
struct Span {
  int32_t lo, hi;          // [lo, hi)
  int32_t all_lo, all_hi;  // tokens that every one of these columns attends to
};

__device__ __forceinline__ Span span_of(const SeqInfo& s, int32_t col0, int32_t col1, const FastDiv& group, int window) {
  const int32_t first = s.n - s.m + col0 / group, last = s.n - s.m + (col1 - 1) / group;
  Span r;
  r.hi = last + 1 > 0 ? last + 1 : 0;
  r.all_hi = first + 1 > 0 ? first + 1 : 0;
  r.lo = window && first - window + 1 > 0 ? first - window + 1 : 0;
  r.all_lo = window && last - window + 1 > 0 ? last - window + 1 : 0;
  return r;
}

// The scales (a byte each) of four tokens from `first` on, those outside [lo, hi) cleared:
// nothing attends to these tokens, but their bytes may never have been written, and a weight of
// zero times a NaN would reach the sums.
__device__ __forceinline__ uint32_t live_scales(uint32_t x, int32_t first, int32_t lo, int32_t hi) {
  asm volatile("" : "+v"(first));          // rare: nothing of it is kept in registers through a loop
  const int32_t skip = lo - first, left = hi - first;
  const uint32_t from = skip <= 0 ? ~0u : (skip >= 4 ? 0u : ~0u << (8 * skip));
  const uint32_t upto = left >= 4 ? ~0u : (left <= 0 ? 0u : (1u << (8 * left)) - 1u);
  return x & from & upto;
}

__device__ __forceinline__ int64_t uniform64(int64_t x) {
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
  return (int64_t)(((uint64_t)hi << 32) | lo);
}

// The sequences of a call, one per lane where there are at most 64.
struct SeqTable {
  SeqInfo mine;
  bool held;

  __device__ __forceinline__ SeqTable(const KvAttnArgs& a, int lane) : mine{0, 0, 0}, held(a.batch <= 64) {
    if (held && lane < a.batch) mine = seq_info(a, lane);
  }
  // sequence b (wave-uniform)
  __device__ __forceinline__ SeqInfo at(const KvAttnArgs& a, int b) const {
    if (!held) return seq_info(a, b);
    SeqInfo s;
    s.q0 = __builtin_amdgcn_readlane(mine.q0, b);
    s.m = __builtin_amdgcn_readlane(mine.m, b);
    s.n = __builtin_amdgcn_readlane(mine.n, b);
    return s;
  }
};

// What the first worker of an item done in pieces leaves for the join: the item's query
// columns.  The other pieces are those of the workers after it.
struct alignas(16) ItemPieces {
  int32_t cols;            // columns of the item; 0: this worker began none
  int32_t pieces;
  int32_t q0, first_col, kh, pad[3];
};
static_assert(sizeof(ItemPieces) == kItemPiecesBytes, "launch.hpp");

// Partial results of column c: [maximum, sum, -, -, output D] floats
__device__ __forceinline__ float* piece_at(const KvAttnArgs& a, int D, int32_t worker, int32_t c) {
  return a.part + ((int64_t)worker * a.tile_cols + c) * (D + 4);
}

// A granule as a buffer: its address in scalar registers, the lanes' 32-bit offsets in one
// register each for all granules.
template <int D>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t granule_buffer(const KvAttnArgs& a, int32_t page, int32_t in_page) {
  const uint8_t* p = a.cache + uniform64((int64_t)page * a.geom.page_bytes + (int64_t)in_page * kv_granule_bytes(D));
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<uint8_t*>(p), (short)0, kv_granule_bytes(D), 0x00020000);
}

constexpr int kStream = 2;         // cache policy of loads: non-temporal

template <int N, int POLICY>
__device__ __forceinline__ void load_dwords(__amdgpu_buffer_rsrc_t r, uint32_t off, uint32_t* d) {
  if constexpr (N == 2) {
    const auto x = __builtin_amdgcn_raw_buffer_load_b64(r, off, 0, POLICY);
    d[0] = x[0];
    d[1] = x[1];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const auto x = __builtin_amdgcn_raw_buffer_load_b128(r, off + 4 * i, 0, POLICY);
#pragma unroll
      for (int e = 0; e < 4; ++e) d[i + e] = x[e];
    }
  }
}

// Nibbles of four tokens' code bytes re-paired by token: byte i of lo[0] holds element 2 i
// of tokens (0, 1), of hi[0] element 2 i + 1, and lo[1], hi[1] those of tokens (2, 3); w = the
// dword (4 bytes) of each token.
__device__ __forceinline__ void pair_tokens(const uint32_t w[4], uint32_t lo[2], uint32_t hi[2]) {
  constexpr uint32_t M = 0x0F0F0F0Fu;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t x = w[2 * i], y = w[2 * i + 1];
    lo[i] = (x & M) | ((y << 4) & ~M);
    hi[i] = ((x >> 4) & M) | (y & ~M);
  }
}

template <int SEL>
__device__ __forceinline__ f16x2 cvt_fp4(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, SEL);
}

// The four tokens' code bytes of dword `part` (8 elements) of a value granule
template <int D>
__device__ __forceinline__ void value_words(const uint32_t v[D / 32], int part, uint32_t w[4]) {
  if constexpr (D == 64) {               // 2 bytes per token
    w[0] = v[0];
    w[1] = v[0] >> 16;
    w[2] = v[1];
    w[3] = v[1] >> 16;
  } else if constexpr (D == 128) {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = v[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = v[2 * e + part];
  }
}

template <bool F32>
__device__ __forceinline__ void load8(const void* base, int64_t off, float v[8]) {
  if constexpr (F32) {
    const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(base) + off);
    const f32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = a[i];
      v[4 + i] = b[i];
    }
  } else {
    const u32x4 a = *reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  }
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return f32_to_bf16_bits(a) | (f32_to_bf16_bits(b) << 16);
}

}  // namespace
}  // namespace nvfp4
