// Attention over the paged NVFP4 key/value cache (layout: kv_layout.hpp).
//
// For query head h of token i of a sequence with m query tokens and n cached tokens
// (the query tokens are the last m of the n), kv head h / G, position p = n - m + i:
//   S_t = scale * <q, k_t>,  o = sum_t e^{S_t - M} v_t / sum_t e^{S_t - M},
//   lse = M + log sum_t e^{S_t - M}   over max(0, p - window + 1) <= t <= p,
// o = 0 and lse = -inf where that range is empty.
//
// Numerics.  Cached values e2m1 * s are exact in f16, so both products run on the f16
// MFMA with fp32 accumulation; the global scales multiply the score and the output.
// Query rows are scaled by a power of two so that their largest element is in
// [2^14, 2^15): bf16 queries are then exact in f16 (elements 2^-29 below the row's
// largest lose bits), and fp32 queries go as two f16 terms q = hi + lo.  The weights
// p = 2^(s - M) (base 2, log2 e folded into the scale) are rounded to f16 for the second
// product where the output is bf16 (11 bits against the output's 8), and go as two f16
// terms where it is fp32; their sum is taken of the unrounded fp32 values.  Weights are
// 2^(s - M) with M 7 below the running maximum when it was last moved, and M moves only when a
// tile's largest weight would pass 2^15: f16 has that range, most tiles leave the output
// accumulators alone, and weights 2^-21 below the largest are still normal f16 numbers.
//
// One pass over the cache.  S^T = K q^T: keys are the A operand's rows (tokens), query
// columns (query token x head of the group, 16 per block) the B operand's; a lane's
// scores are then all of one column, the softmax needs two cross-lane steps per tile,
// and the scores of two 16-token granules are, in place, the B operand of O^T = V^T P^T
// (the K axis, tokens, in the order quads g of both granules; V^T is read in the same
// order).  Codes go from HBM to registers in whole 16-byte pieces and are decoded there.
#include "kernel_common.hpp"
#include "kv_layout.hpp"

namespace nvfp4 {

namespace {

constexpr float kNegBig = -1.0e30f;      // reference M of a row that has seen nothing
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float xor16(float x) { return __shfl_xor(x, 16); }
__device__ __forceinline__ float xor32(float x) { return __shfl_xor(x, 32); }

// What a workgroup needs of its sequence
struct SeqInfo {
  int64_t q0;              // first query token (row of q)
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
  s.q0 = q0;
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

__device__ __forceinline__ Span span_of(const SeqInfo& s, int64_t col0, int64_t col1, int group, int window) {
  const int32_t first = s.n - s.m + (int32_t)col0 / group, last = s.n - s.m + ((int32_t)col1 - 1) / group;
  Span r;
  r.hi = last + 1 > 0 ? last + 1 : 0;
  r.all_hi = first + 1 > 0 ? first + 1 : 0;
  r.lo = window && first - window + 1 > 0 ? first - window + 1 : 0;
  r.all_lo = window && last - window + 1 > 0 ? last - window + 1 : 0;
  return r;
}

// One granule as a lane of the 16-row MFMAs holds it.
template <int D>
struct Granule {
  static constexpr int KD = D / 32;        // dwords of key codes, and of value codes
  static constexpr int KS = D == 256 ? 2 : 1;
  uint32_t k[KD], ks[KS], v[KD], vs;
};

template <int N>
__device__ __forceinline__ void load_dwords(const uint8_t* p, uint32_t* d) {
  if constexpr (N == 2) {
    const u32x2 x = *reinterpret_cast<const u32x2*>(p);
    d[0] = x[0];
    d[1] = x[1];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const u32x4 x = *reinterpret_cast<const u32x4*>(p + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) d[i + e] = x[e];
    }
  }
}

// Keys: lane (g, r) holds token r, elements 32 g + 8 m + j (D = 128), 128 c + 32 g + 8 m + j
// (D = 256), 16 g + 8 m + j (D = 64); values: tokens 4 g + e, elements (D / 16) r + j.
template <int D>
__device__ __forceinline__ void load_granule(const uint8_t* p, int lane, Granule<D>& x) {
  const int g = lane >> 4, r = lane & 15;
  if constexpr (D == 64) {
    load_dwords<2>(p + r * 32 + g * 8, x.k);
    x.ks[0] = p[8 * D + r * 4 + g];
  } else if constexpr (D == 128) {
    load_dwords<4>(p + r * 64 + g * 16, x.k);
    x.ks[0] = *reinterpret_cast<const uint16_t*>(p + 8 * D + r * 8 + 2 * g);
  } else {
    load_dwords<4>(p + r * 128 + g * 16, x.k);
    load_dwords<4>(p + r * 128 + 64 + g * 16, x.k + 4);
    x.ks[0] = *reinterpret_cast<const uint16_t*>(p + 8 * D + r * 16 + 2 * g);
    x.ks[1] = *reinterpret_cast<const uint16_t*>(p + 8 * D + r * 16 + 8 + 2 * g);
  }
  load_dwords<D / 32>(p + 9 * D + (g * 16 + r) * (D / 8), x.v);
  x.vs = *reinterpret_cast<const uint32_t*>(p + 17 * D + (g * (D / 16) + r * D / 256) * 4);
}

// A operand of key chunk i (8 elements of token r): codes k[i] under their block's scale
template <int D>
__device__ __forceinline__ f16x8 key_frag(const Granule<D>& x, int i) {
  if constexpr (D == 64) {
    return decode8_f16(x.k[i], bcast(scale_pair_f16(x.ks[0]), 0));
  } else {
    return decode8_f16(x.k[i], bcast(scale_pair_f16(x.ks[i / 4]), (i >> 1) & 1));
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
__device__ __forceinline__ void value_words(const Granule<D>& x, int part, uint32_t w[4]) {
  if constexpr (D == 64) {               // 2 bytes per token
    w[0] = x.v[0];
    w[1] = x.v[0] >> 16;
    w[2] = x.v[1];
    w[3] = x.v[1] >> 16;
  } else if constexpr (D == 128) {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = x.v[e];
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = x.v[2 * e + part];
  }
}

__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f16x8 join(f16x2 a, f16x2 b, f16x2 c, f16x2 d) {
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Two fp32 -> two f16, round to nearest even
__device__ __forceinline__ f16x2 to_f16(float a, float b) { return f16x2{(_Float16)a, (_Float16)b}; }

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

// One workgroup = W waves = (sequence, kv head, 16 NQ query columns, split of the key
// axis); each wave takes a contiguous piece of the split's tokens, NG granules at a time,
// with the next ones' loads in flight; the waves' (maximum, sum, output) are joined in
// LDS.  With one split the result goes out, else it goes to the partials for k_kv_join.
constexpr int kAttnWaves = 4;

template <int D, int NQ, bool F32>
__global__ __launch_bounds__(64 * kAttnWaves, 2) void k_kv_attn(KvAttnArgs a) {
  constexpr int W = kAttnWaves;
  constexpr int NG = D == 256 ? 2 : 4;             // granules per step
  constexpr int TOK = 16 * NG;
  constexpr int KC = D / 32;                       // 32-element chunks of the first product
  constexpr int NJ = D / 16;                       // 16-row blocks of the second
  constexpr int TERMS = F32 ? 2 : 1;
  constexpr int LDO = D + 4;                       // LDS row of a column's output: 16-byte aligned, banks spread
  __shared__ float s_o[W][16 * LDO];
  __shared__ float s_m[W][16 * NQ], s_l[W][16 * NQ];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int hkv = a.geom.n_kv_heads, group = a.n_q_heads / hkv;
  int bid = blockIdx.x;
  const int split = bid % a.n_splits;
  bid /= a.n_splits;
  const int tile = bid % a.col_tiles;
  bid /= a.col_tiles;
  const int kh = bid % hkv, b = bid / hkv;
  const SeqInfo seq = seq_info(a, b);
  const int64_t cols = (int64_t)seq.m * group;
  const float kg = a.k_gscale[kh], vg = a.v_gscale[kh];
  const int32_t last_page = (seq.n - 1) >> a.geom.page_shift;
  const int per_head = 1 << (a.geom.page_shift - 4);

  for (int64_t col0 = (int64_t)tile * 16 * NQ; col0 < cols; col0 += (int64_t)a.col_tiles * 16 * NQ) {
    const int64_t col1 = col0 + 16 * NQ < cols ? col0 + 16 * NQ : cols;
    const Span sp = span_of(seq, col0, col1, group, a.window);
    // this split's tokens, in whole steps from a granule-aligned start; the split
    // length is the plan's, or longer where the plan's bound was too low
    const int32_t begin = sp.lo & ~15;
    const int32_t steps = (sp.hi - begin + TOK - 1) / TOK;
    int32_t per = (steps + a.n_splits - 1) / a.n_splits;
    const int32_t planned = a.split_tokens / TOK;
    per = per > planned ? per : planned;
    const int32_t s0 = split * per, s1 = s0 + per < steps ? s0 + per : steps;
    const int32_t pw = s1 > s0 ? (s1 - s0 + W - 1) / W : 0;
    const int32_t w0 = s0 + wave * pw, w1 = w0 + pw < s1 ? w0 + pw : s1;

    // query columns: lane (g, r) holds column r of every block, the chunks' elements
    f16x8 qf[TERMS][NQ][KC];
    float csc[NQ], m[NQ], l[NQ];
    int32_t limit[NQ], floor_[NQ];                 // the column attends to floor_ <= t < limit
    f32x4 acc[NQ][NJ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      int64_t col = col0 + 16 * n + r;
      if (col >= cols) col = cols - 1;             // computed, never written
      const int32_t qi = (int32_t)col / group;
      const int head = kh * group + ((int32_t)col - qi * group);
      const int64_t off = (seq.q0 + qi) * a.ldq + (int64_t)head * D;
      float v[KC][8];
      float amax = 0.0f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const int d0 = D == 64 ? 16 * g + 8 * c : 128 * (c / 4) + 32 * g + 8 * (c % 4);
        load8<F32>(a.q, off + d0, v[c]);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = __builtin_fmaxf(amax, __builtin_fabsf(v[c][e]));
      }
      amax = __builtin_fmaxf(amax, xor16(amax));
      amax = __builtin_fmaxf(amax, xor32(amax));
      // 2^(14 - e) for amax in [2^e, 2^(e+1)); zero and tiny rows are left near zero
      int e = (int)((__float_as_uint(amax) >> 23) & 255u) - 127;
      e = e < -100 ? -100 : e;
      const float up = __uint_as_float((uint32_t)(14 - e + 127) << 23);
      csc[n] = a.scale * kLog2e * kg * __uint_as_float((uint32_t)(e - 14 + 127) << 23);
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = v[c][i] * up;
          const _Float16 hi = (_Float16)x;
          qf[0][n][c][i] = hi;
          if constexpr (F32) qf[TERMS - 1][n][c][i] = (_Float16)(x - (float)hi);
        }
      const int32_t pos = seq.n - seq.m + qi;
      limit[n] = pos + 1;
      floor_[n] = a.window ? pos - a.window + 1 : 0;
      m[n] = kNegBig;
      l[n] = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[n][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    if (w0 < w1) {
      // page of token tb + 16 lane, held by the lane, for 1024 tokens and the 1024 after
      auto load_pages = [&](int32_t t) -> int32_t {
        int32_t pg = (t + 16 * lane) >> a.geom.page_shift;
        pg = pg < last_page ? pg : last_page;
        int32_t id = a.table[(int64_t)b * a.ld_table + pg];
        return id < 0 ? 0 : (id >= a.geom.n_pages ? (int32_t)a.geom.n_pages - 1 : id);
      };
      constexpr int SPB = 64 / NG;                 // steps per 64 granules
      int32_t pages = load_pages(begin + w0 * TOK), pages_next = load_pages(begin + (w0 + SPB) * TOK);
      const int32_t last_granule = (seq.n - 1) >> 4;
      auto issue = [&](int32_t s, Granule<D> x[NG]) {
        const int32_t i = (s - w0) % SPB;
#pragma unroll
        for (int u = 0; u < NG; ++u) {
          const int32_t id = __builtin_amdgcn_readlane(pages, i * NG + u);
          int32_t gr = (begin + s * TOK) / 16 + u;
          gr = gr < last_granule ? gr : last_granule;   // past the end: the last granule again
          const uint8_t* p = a.cache + (int64_t)id * a.geom.page_bytes +
                             (int64_t)(kh * per_head + (gr & (per_head - 1))) * kv_granule_bytes(D);
          load_granule<D>(p, lane, x[u]);
        }
        if (i == SPB - 1) {
          pages = pages_next;
          pages_next = load_pages(begin + (s + 1 + SPB) * TOK);
        }
      };

      Granule<D> cur[NG], nxt[NG];
      issue(w0, nxt);
      for (int32_t s = w0; s < w1; ++s) {
#pragma unroll
        for (int u = 0; u < NG; ++u) cur[u] = nxt[u];
        if (s + 1 < w1) issue(s + 1, nxt);
        const int32_t t0 = begin + s * TOK;
        const bool edge = t0 < sp.all_lo || t0 + TOK > sp.all_hi;

        // S^T: rows = tokens 16 u + 4 g + i
        f32x4 sc[NQ][NG];
#pragma unroll
        for (int u = 0; u < NG; ++u) {
#pragma unroll
          for (int n = 0; n < NQ; ++n) sc[n][u] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int c = 0; c < KC; ++c) {
            const f16x8 kf = key_frag<D>(cur[u], c);
#pragma unroll
            for (int n = 0; n < NQ; ++n)
#pragma unroll
              for (int t = 0; t < TERMS; ++t) sc[n][u] = mfma16(kf, qf[t][n][c], sc[n][u]);
          }
        }

        // weights, in the layout of the second product's B operand
        f16x8 pf[TERMS][NQ][NG / 2];
#pragma unroll
        for (int n = 0; n < NQ; ++n) {
          float x[NG][4], top = -__builtin_inff();
#pragma unroll
          for (int u = 0; u < NG; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) x[u][i] = sc[n][u][i] * csc[n];
          if (edge) {
#pragma unroll
            for (int u = 0; u < NG; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int32_t t = t0 + 16 * u + 4 * g + i;
                if (t >= limit[n] || t < floor_[n]) x[u][i] = -__builtin_inff();
              }
          }
#pragma unroll
          for (int u = 0; u < NG; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = __builtin_fmaxf(top, x[u][i]);
          top = __builtin_fmaxf(top, xor16(top));
          top = __builtin_fmaxf(top, xor32(top));
          if (__builtin_amdgcn_ballot_w64(top > m[n] + 15.0f)) {
            const float m1 = __builtin_fmaxf(m[n], top - 7.0f);
            const float f = __builtin_amdgcn_exp2f(m[n] - m1);
            m[n] = m1;
            l[n] *= f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[n][j] *= f;
          }
          float p[NG][4];
#pragma unroll
          for (int u = 0; u < NG; ++u)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              p[u][i] = __builtin_amdgcn_exp2f(x[u][i] - m[n]);
              l[n] += p[u][i];
            }
#pragma unroll
          for (int k = 0; k < NG / 2; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float v = p[2 * k + i / 4][i % 4];
              const _Float16 hi = (_Float16)v;
              pf[0][n][k][i] = hi;
              if constexpr (F32) pf[TERMS - 1][n][k][i] = (_Float16)(v - (float)hi);
            }
        }

        // O^T += V^T P^T: rows = elements NJ r + j.  The scales of tokens past the end
        // are cleared: their bytes may hold anything, and 0 * NaN would reach the sums.
        if (t0 + TOK > seq.n) {
#pragma unroll
          for (int u = 0; u < NG; ++u) {
            const int32_t left = seq.n - (t0 + 16 * u + 4 * g);    // live tokens from this quad's first on
            cur[u].vs = left <= 0 ? 0u : (left >= 4 ? cur[u].vs : cur[u].vs & ((1u << (8 * left)) - 1u));
          }
        }
#pragma unroll
        for (int k = 0; k < NG / 2; ++k) {
          f16x2 vs[2][2];
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            vs[u][0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(cur[2 * k + u].vs, 1.0f, false);
            vs[u][1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(cur[2 * k + u].vs, 1.0f, true);
          }
#pragma unroll
          for (int part = 0; part < (NJ + 7) / 8; ++part) {
            uint32_t lo[2][2], hi[2][2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t w[4];
              value_words<D>(cur[2 * k + u], part, w);
              pair_tokens(w, lo[u], hi[u]);
            }
            auto rows = [&](int j, f16x2 (&x)[2][2]) {
#pragma unroll
              for (int n = 0; n < NQ; ++n)
#pragma unroll
                for (int t = 0; t < TERMS; ++t)
                  acc[n][8 * part + j] = mfma16(join(x[0][0], x[0][1], x[1][0], x[1][1]), pf[t][n][k],
                                                acc[n][8 * part + j]);
            };
#define NVFP4_VROWS(SEL)                                                       \
  if constexpr (2 * (SEL) < NJ) {                                              \
    f16x2 x[2][2], y[2][2];                                                    \
    _Pragma("unroll") for (int u = 0; u < 2; ++u)                              \
        _Pragma("unroll") for (int e = 0; e < 2; ++e) {                        \
      x[u][e] = cvt_fp4<SEL>(lo[u][e]) * vs[u][e];                             \
      y[u][e] = cvt_fp4<SEL>(hi[u][e]) * vs[u][e];                             \
    }                                                                          \
    rows(2 * (SEL), x);                                                        \
    rows(2 * (SEL) + 1, y);                                                    \
  }
            NVFP4_VROWS(0)
            NVFP4_VROWS(1)
            NVFP4_VROWS(2)
            NVFP4_VROWS(3)
#undef NVFP4_VROWS
          }
        }
      }
    }

    // join the waves
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      l[n] += xor16(l[n]);
      l[n] += xor32(l[n]);
      if (g == 0) {
        s_m[wave][16 * n + r] = m[n];
        s_l[wave][16 * n + r] = l[n];
      }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float top = s_m[0][16 * n + r];
#pragma unroll
      for (int w = 1; w < W; ++w) top = __builtin_fmaxf(top, s_m[w][16 * n + r]);
      const float f = __builtin_amdgcn_exp2f(m[n] - top);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float* dst = &s_o[wave][r * LDO + NJ * (4 * g + i)];
#pragma unroll
        for (int j = 0; j < NJ; j += 4)
          *reinterpret_cast<f32x4*>(dst + j) =
              f32x4{acc[n][j][i] * f, acc[n][j + 1][i] * f, acc[n][j + 2][i] * f, acc[n][j + 3][i] * f};
      }
      __syncthreads();
      // thread = (column, D / 16 elements)
      const int c = threadIdx.x >> 4, part = threadIdx.x & 15;
      const int64_t col = col0 + 16 * n + c;
      if (col < cols) {
        float top_c = s_m[0][16 * n + c], sum = 0.0f;
#pragma unroll
        for (int w = 1; w < W; ++w) top_c = __builtin_fmaxf(top_c, s_m[w][16 * n + c]);
#pragma unroll
        for (int w = 0; w < W; ++w) sum += s_l[w][16 * n + c] * __builtin_amdgcn_exp2f(s_m[w][16 * n + c] - top_c);
        float out[NJ];
#pragma unroll
        for (int j = 0; j < NJ; j += 4) {
          f32x4 x = *reinterpret_cast<const f32x4*>(&s_o[0][c * LDO + part * NJ + j]);
#pragma unroll
          for (int w = 1; w < W; ++w) x += *reinterpret_cast<const f32x4*>(&s_o[w][c * LDO + part * NJ + j]);
#pragma unroll
          for (int e = 0; e < 4; ++e) out[j + e] = x[e];
        }
        const int32_t qi = (int32_t)col / group;
        const int head = kh * group + ((int32_t)col - qi * group);
        const int64_t row = (seq.q0 + qi) * a.n_q_heads + head;
        if (a.n_splits == 1) {
          const float f = sum > 0.0f ? vg / sum : 0.0f;
          const int64_t off = (seq.q0 + qi) * a.ldo + (int64_t)head * D + part * NJ;
          if constexpr (F32) {
#pragma unroll
            for (int j = 0; j < NJ; j += 4)
              *reinterpret_cast<f32x4*>(reinterpret_cast<float*>(a.o) + off + j) =
                  f32x4{out[j] * f, out[j + 1] * f, out[j + 2] * f, out[j + 3] * f};
          } else {
#pragma unroll
            for (int j = 0; j < NJ; j += 4)
              *reinterpret_cast<u32x2*>(reinterpret_cast<uint16_t*>(a.o) + off + j) =
                  u32x2{pack_bf16(out[j] * f, out[j + 1] * f), pack_bf16(out[j + 2] * f, out[j + 3] * f)};
          }
          if (a.lse && part == 0)
            a.lse[row] = sum > 0.0f ? (top_c + __builtin_log2f(sum)) * kLn2 : -__builtin_inff();
        } else {
          float* dst = a.part + (row * a.n_splits + split) * (D + 4);
#pragma unroll
          for (int j = 0; j < NJ; j += 4)
            *reinterpret_cast<f32x4*>(dst + 4 + part * NJ + j) = f32x4{out[j], out[j + 1], out[j + 2], out[j + 3]};
          if (part == 0) {
            dst[0] = top_c;
            dst[1] = sum;
          }
        }
      }
      __syncthreads();
    }
  }
}

// Join the splits of an output row: one wave per row, lane = D / 64 elements.
template <int D, bool F32>
__global__ __launch_bounds__(256) void k_kv_join(KvAttnArgs a) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 63;
  const int64_t row = (int64_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  if (row >= a.T * a.n_q_heads) return;
  const float* src = a.part + row * a.n_splits * (D + 4);
  float top = kNegBig;
  for (int s = 0; s < a.n_splits; ++s) top = __builtin_fmaxf(top, src[s * (D + 4)]);
  float sum = 0.0f, out[E];
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = 0.0f;
  for (int s = 0; s < a.n_splits; ++s) {
    const float* p = src + s * (D + 4);
    const float f = __builtin_amdgcn_exp2f(p[0] - top);
    sum += p[1] * f;
#pragma unroll
    for (int e = 0; e < E; ++e) out[e] += p[4 + lane * E + e] * f;
  }
  const int64_t tok = row / a.n_q_heads;
  const int head = (int)(row - tok * a.n_q_heads);
  const float f = sum > 0.0f ? a.v_gscale[head / (a.n_q_heads / a.geom.n_kv_heads)] / sum : 0.0f;
  const int64_t off = tok * a.ldo + (int64_t)head * D + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) {
    if constexpr (F32) reinterpret_cast<float*>(a.o)[off + e] = out[e] * f;
    else reinterpret_cast<uint16_t*>(a.o)[off + e] = (uint16_t)f32_to_bf16_bits(out[e] * f);
  }
  if (a.lse && lane == 0) a.lse[row] = sum > 0.0f ? (top + __builtin_log2f(sum)) * kLn2 : -__builtin_inff();
}

template <int D, int NQ, bool F32>
hipError_t launch(const KvAttnArgs& a, hipStream_t s) {
  const int64_t blocks = (int64_t)a.batch * a.geom.n_kv_heads * a.col_tiles * a.n_splits;
  hipLaunchKernelGGL((k_kv_attn<D, NQ, F32>), dim3((unsigned)blocks), dim3(64 * kAttnWaves), 0, s, a);
  hipError_t e = hipGetLastError();
  if (e == hipSuccess && a.n_splits > 1) {
    hipLaunchKernelGGL((k_kv_join<D, F32>), dim3((unsigned)((a.T * a.n_q_heads + 3) / 4)), dim3(256), 0, s, a);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace

KvAttnPlan kv_attn_plan(InType t, int64_t T, int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t D,
                        int64_t max_q_len, int64_t max_kv_len) {
  KvAttnPlan p{};
  const int64_t cols = max_q_len * (n_q_heads / n_kv_heads);
  // two column blocks share a decoded granule where their registers fit
  p.nq = cols > 16 && (D == 64 || (D == 128 && t == InType::BF16)) ? 2 : 1;
  int64_t tiles = (cols + 16 * p.nq - 1) / (16 * p.nq);
  // the kernel walks the tiles with the grid's stride: any number of them is right
  const int64_t most_tiles = ((int64_t)1 << 30) / ((int64_t)batch * n_kv_heads * 64);
  if (tiles > most_tiles) tiles = most_tiles < 1 ? 1 : most_tiles;
  p.col_tiles = (int32_t)tiles;
  const int64_t wgs = (int64_t)batch * n_kv_heads * tiles;
  const int64_t chunk = 256;                            // fewest tokens of a split
  int64_t splits = (512 + wgs - 1) / wgs;
  const int64_t most = (max_kv_len + chunk - 1) / chunk;
  if (splits > most) splits = most;
  if (splits > 64) splits = 64;
  if (splits < 1) splits = 1;
  p.n_splits = (int32_t)splits;
  const int64_t per = (max_kv_len + splits - 1) / splits;
  p.split_tokens = (int32_t)((per + 255) / 256 * 256);
  p.workspace = splits > 1 ? T * n_q_heads * splits * (D + 4) * (int64_t)sizeof(float) : 0;
  return p;
}

hipError_t launch_kv_attn(KvAttnArgs a, const KvAttnPlan& p, InType t, int32_t D, hipStream_t s) {
  a.n_splits = p.n_splits;
  a.split_tokens = p.split_tokens;
  a.col_tiles = p.col_tiles;
  const bool f32 = t == InType::F32;
  if (D == 64) {
    if (p.nq == 2) return f32 ? launch<64, 2, true>(a, s) : launch<64, 2, false>(a, s);
    return f32 ? launch<64, 1, true>(a, s) : launch<64, 1, false>(a, s);
  }
  if (D == 128) {
    if (p.nq == 2) return launch<128, 2, false>(a, s);
    return f32 ? launch<128, 1, true>(a, s) : launch<128, 1, false>(a, s);
  }
  return f32 ? launch<256, 1, true>(a, s) : launch<256, 1, false>(a, s);
}

}  // namespace nvfp4
