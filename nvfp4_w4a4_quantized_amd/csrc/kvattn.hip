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
// [2^14, 2^15): bf16 queries are then exact in f16 (elements below 2^-28 of the row's
// largest may lose bits), and fp32 queries go as two f16 terms q = hi + lo.  The weights
// p = 2^(s - M) (base 2, log2 e folded into the scale) are rounded to f16 for the second
// product where the output is bf16 (11 bits against the output's 8), and go as two f16
// terms where it is fp32; their sum is taken of the unrounded fp32 values.  Weights are
// 2^(s - M) with M 7 below the running maximum when it was last moved, and M moves only when a
// tile's largest weight would pass 2^15: f16 has that range, most tiles leave the output
// accumulators alone, and weights 2^-21 below the largest are still normal f16 numbers.  Scores
// may be of any size that fp32 holds (kWideFactor).
//
// One pass over the cache.  S^T = K q^T: keys are the A operand's rows (tokens), query
// columns (query token x head of the group, 16 per block) the B operand's; a lane's
// scores are then all of one column, the softmax needs two cross-lane steps per tile,
// and the scores of two 16-token granules are, in place, the B operand of O^T = V^T P^T
// (the K axis, tokens, in the order quads g of both granules; V^T is read in the same
// order).  Codes go from HBM to registers in whole 16-byte pieces and are decoded there.
//
// What bounds it: the cache's bytes.  32 sequences of 1024 to 8192 tokens, 32 / 8 heads of 128: 174 MB
// in 39 us and 4.6 us for the join, 4.4 TB/s (a kernel of these loads alone 44 us before they were
// non-temporal; a 1 GiB copy moves 5.2); 2 of 131072: 266 MB in 49 us, 5.4 TB/s, and 4.7 us; head
// dimension 256, 16 of 32768: 226 MB in 49 us, 4.6 TB/s, and 5 us.  One sequence of 257 tokens takes
// 6.4 us, latency.  Drafted tokens are bound by no unit: 24 sequences of 1 to 6 tokens of 48 / 8 heads
// take 44 us, 97 MB at 2.2 TB/s with the vector unit 34 % busy, the matrix unit 9 %, and 35 % of the
// waves' time waiting; of a wave's 4043 vector instructions some 1500 are a piece's own, around
// about five steps of 450 (64 tokens each, most of it decoding), and 36 columns take a second column
// group that decodes every key again.  Two blocks of 16 columns share a decoded granule (9 or 14
// registers spilled, one access of them in the loop over the steps; fp32 at head dimension 256
// spills 20 or 23); three spilled 180.  Granules two steps ahead (62 us instead of 49 then) and two
// steps a turn without the register copies between them (no change; drafts 57 us instead of 47) did
// not pay.
#include "kv_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kMaxWorkers = 512;         // two workgroups per compute unit
constexpr int kMostPieces = kMaxWorkers; // of one item (S is at least its share of all steps)

// One granule as a lane of the 16-row MFMAs holds it.
template <int D>
struct Granule {
  static constexpr int KD = D / 32;        // dwords of key codes, and of value codes
  static constexpr int KS = D == 256 ? 2 : 1;
  uint32_t k[KD], ks[KS], v[KD], vs;
};

// Keys: lane (g, r) holds token r, elements 32 g + 8 m + j (D = 128), 128 c + 32 g + 8 m + j
// (D = 256), 16 g + 8 m + j (D = 64); values: tokens 4 g + e, elements (D / 16) r + j.
// Non-temporal: a cache is read once, or by the column groups of one workgroup at a time (2 x
// 131072 keys 63.4 -> 56.1 us).
template <int D>
__device__ __forceinline__ void load_granule(__amdgpu_buffer_rsrc_t p, uint32_t lane, Granule<D>& x) {
  const uint32_t g = lane >> 4, r = lane & 15;
  if constexpr (D == 64) {
    load_dwords<2, kStream>(p, r * 32 + g * 8, x.k);
    x.ks[0] = (uint8_t)__builtin_amdgcn_raw_buffer_load_b8(p, r * 4 + g, 8 * D, kStream);
  } else if constexpr (D == 128) {
    load_dwords<4, kStream>(p, r * 64 + g * 16, x.k);
    x.ks[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(p, r * 8 + 2 * g, 8 * D, kStream);
  } else {
    load_dwords<4, kStream>(p, r * 128 + g * 16, x.k);
    load_dwords<4, kStream>(p, r * 128 + g * 16 + 64, x.k + 4);
    x.ks[0] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(p, r * 16 + 2 * g, 8 * D, kStream);
    x.ks[1] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(p, r * 16 + 2 * g + 8, 8 * D, kStream);
  }
  load_dwords<D / 32, kStream>(p, lane * (D / 8) + 9 * D, x.v);
  x.vs = __builtin_amdgcn_raw_buffer_load_b32(p, (g * (D / 16) + r * D / 256) * 4, 17 * D, kStream);
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

__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ f16x8 join(f16x2 a, f16x2 b, f16x2 c, f16x2 d) {
  return f16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// Work of a call: items (sequence, kv head, tile of tile_cols query columns), each a run of
// steps of NG granules along its keys.  With whole items (n_workers == 0) a workgroup takes
// one.  Otherwise an item is cut into the fewest equal pieces of at most S steps, a workgroup
// each, where S is all steps of the call by n_workers; there are at most n_workers + items
// pieces, and as many workgroups.  Pieces of one item leave partial results for k_kv_join.
// (Equal runs of all steps, one per workgroup whatever items they cross, were slower: the
// second item of a workgroup costs 5 us of latency, more than the better balance gives.)
//
// Inside a workgroup, waves are groups of 16 NQ columns (1, 2 or 4, what the item has) by pieces
// of the piece's tokens, joined in LDS.
constexpr int kAttnWaves = 4;

// Steps of one item of sequence b, and its items
struct SeqWork {
  SeqInfo seq;
  int32_t cols, tiles, begin, steps;    // begin: first token, granule-aligned
};

template <int TOK>
__device__ __forceinline__ SeqWork seq_work(const KvAttnArgs& a, const SeqInfo& seq) {
  SeqWork w;
  w.seq = seq;
  w.cols = w.seq.m * (int32_t)a.by_group.d;
  w.tiles = 0;
  w.begin = w.steps = 0;
  if (w.cols > 0) {
    const Span sp = span_of(w.seq, 0, w.cols, a.by_group, a.window);
    const int32_t tiles = (w.cols + a.tile_cols - 1) / a.by_tile_cols;
    w.tiles = tiles < a.col_tiles ? tiles : a.col_tiles;   // further ones go with the first tiles' items
    w.begin = sp.lo & ~15;
    w.steps = (sp.hi - w.begin + TOK - 1) / TOK;
    w.steps = w.steps < 1 ? 1 : w.steps;                   // an empty item still writes its zeros
  }
  return w;
}

template <int D, int NQ, bool GROUPS, bool F32>
__global__ __launch_bounds__(64 * kAttnWaves, 2) void k_kv_attn(KvAttnArgs a) {
  constexpr int W = kAttnWaves;
  constexpr int NG = D == 256 ? 2 : 4;             // granules per step
  constexpr int TOK = 16 * NG;
  constexpr int KC = D / 32;                       // 32-element chunks of the first product
  constexpr int NJ = D / 16;                       // 16-row blocks of the second
  constexpr int TERMS = F32 ? 2 : 1;
  constexpr int LDO = D + 4;                       // LDS row of a column's output: 16-byte aligned, banks spread
  __shared__ float s_o[W][16 * LDO];
  __shared__ float s_m[W][16 * NQ], s_l[W][16 * NQ], s_c[W][16 * NQ];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int hkv = a.geom.n_kv_heads, group = (int)a.by_group.d;
  const int per_head = 1 << (a.geom.page_shift - 4);

  // this workgroup's item and its steps [s_first, s_last) of it
  int b, kh, tile0;
  int32_t s_first, s_last;
  SeqWork sw;
  if (a.n_workers == 0) {
    const int item = (int)blockIdx.x / a.by_col_tiles;
    b = item / a.by_heads;
    kh = item - b * hkv;
    tile0 = (int)blockIdx.x - item * a.col_tiles;
    sw = seq_work<TOK>(a, seq_info(a, b));
    if (tile0 >= sw.tiles) return;
    s_first = 0;
    s_last = sw.steps;
  } else {
    // each lane counts the steps, then the pieces, of `each` consecutive sequences
    const SeqTable seqs(a, lane);
    const int each = (a.batch + 63) / 64;
    auto steps_of = [&](int i, int32_t& items) {
      const int bb = lane * each + i;
      items = 0;
      if (bb >= a.batch) return 0;
      const SeqWork x = seq_work<TOK>(a, seqs.held ? seqs.mine : seq_info(a, bb));
      items = x.tiles * hkv;
      return x.steps;
    };
    float total = 0.0f;
    for (int i = 0; i < each; ++i) {
      int32_t items;
      const int32_t steps = steps_of(i, items);
      total += (float)items * (float)steps;
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) total += __shfl_xor(total, off);
    // rounded up, past the rounding of the sum
    int32_t S = (int32_t)(total * 1.0001f / (float)a.n_workers) + 1;
    S = S < a.min_steps ? a.min_steps : S;
    int32_t own = 0;
    for (int i = 0; i < each; ++i) {
      int32_t items;
      const int32_t steps = steps_of(i, items);
      if (items) own += items * (int32_t)((uint32_t)(steps + S - 1) / (uint32_t)S);
    }
    int32_t upto = own;
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) {
      const int32_t x = __shfl_up(upto, off);
      if (lane >= off) upto += x;
    }
    const uint64_t past = __builtin_amdgcn_ballot_w64(upto > (int32_t)blockIdx.x);
    if (past == 0) {
      if (threadIdx.x == 0) static_cast<ItemPieces*>(a.pieces)[blockIdx.x].cols = 0;
      return;
    }
    const int first = __builtin_ctzll(past);
    int32_t in_seq = (int32_t)blockIdx.x - __builtin_amdgcn_readlane(upto - own, first), pieces;
    for (b = first * each;; ++b) {
      sw = seq_work<TOK>(a, seqs.at(a, b));
      pieces = (int32_t)((uint32_t)(sw.steps + S - 1) / (uint32_t)S);
      if (in_seq < sw.tiles * hkv * pieces) break;
      in_seq -= sw.tiles * hkv * pieces;
    }
    const int32_t item = pieces == 1 ? in_seq : (int32_t)((uint32_t)in_seq / (uint32_t)pieces);
    const int32_t piece = in_seq - item * pieces;
    kh = sw.tiles == 1 ? item : (int32_t)((uint32_t)item / (uint32_t)sw.tiles);
    tile0 = item - kh * sw.tiles;
    const int32_t q = pieces == 1 ? sw.steps : (int32_t)((uint32_t)sw.steps / (uint32_t)pieces);
    const int32_t rest = sw.steps - q * pieces;
    s_first = piece * q + (piece < rest ? piece : rest);
    s_last = s_first + q + (piece < rest);
    if (threadIdx.x == 0) {
      const int32_t fc = tile0 * a.tile_cols, left = sw.cols - fc;
      ItemPieces* const p = static_cast<ItemPieces*>(a.pieces) + blockIdx.x;
      p->cols = piece == 0 && pieces > 1 ? (left < a.tile_cols ? left : a.tile_cols) : 0;
      p->pieces = pieces;
      p->q0 = sw.seq.q0;
      p->first_col = fc;
      p->kh = kh;
    }
  }

  {
    const SeqInfo& seq = sw.seq;
    const float kg = a.k_gscale[kh], vg = a.v_gscale[kh];
    const int32_t last_page = (seq.n - 1) >> a.geom.page_shift;

    // tiles past the planned ones are done whole, with the item's first piece
    for (int32_t tile = tile0; (int64_t)tile * a.tile_cols < sw.cols; tile += a.col_tiles) {
    if (tile != tile0 && s_first > 0) break;
    const int32_t col_first = tile * a.tile_cols;
    const int32_t cols = col_first + a.tile_cols < sw.cols ? col_first + a.tile_cols : sw.cols;   // end of the tile
    Span sp = span_of(seq, col_first, cols, a.by_group, a.window);
    int32_t begin = sw.begin, s0 = s_first, s1 = s_last;
    bool whole = s0 == 0 && s1 == sw.steps;
    if (a.n_workers == 0 || tile != tile0) {       // the tile's own keys
      begin = sp.lo & ~15;
      s0 = 0;
      s1 = (sp.hi - begin + TOK - 1) / TOK;
      whole = true;
    }
    if (seq.n <= 0) s1 = s0;
    // column groups of this item: 2^cs of them, by W >> cs pieces of tokens
    const int cs = !GROUPS || cols - col_first <= 16 * NQ ? 0 : (cols - col_first <= 32 * NQ ? 1 : 2);
    const int cg = wave & ((1 << cs) - 1), tg = wave >> cs, tw = W >> cs;
    const int32_t col0 = col_first + cg * 16 * NQ;
    const int32_t pw = s1 > s0 && col0 < cols ? (s1 - s0 + tw - 1) >> (2 - cs) : 0;
    const int32_t w0 = s0 + tg * pw, w1 = w0 + pw < s1 ? w0 + pw : s1;

    // page of token tb + 16 lane, held by the lane, for 1024 tokens and the 1024 after
    auto load_pages = [&](int32_t t) -> int32_t {
      int32_t pg = (t + 16 * lane) >> a.geom.page_shift;
      pg = pg < last_page ? pg : last_page;
      const int32_t id = a.table[(int64_t)b * a.ld_table + pg];
      return id < 0 ? 0 : (id >= a.geom.n_pages ? (int32_t)a.geom.n_pages - 1 : id);
    };
    constexpr int SPB = 64 / NG;                   // steps per 64 granules
    const int32_t last_granule = (seq.n - 1) >> 4;
    int32_t pages = 0, pages_next = 0;
    auto issue = [&](int32_t s, Granule<D> x[NG]) {
      const int32_t i = (s - w0) % SPB;
#pragma unroll
      for (int u = 0; u < NG; ++u) {
        const int32_t id = __builtin_amdgcn_readlane(pages, i * NG + u);
        int32_t gr = (begin + s * TOK) / 16 + u;
        gr = gr < last_granule ? gr : last_granule;     // past the end: the last granule again
        load_granule<D>(granule_buffer<D>(a, id, kh * per_head + (gr & (per_head - 1))), lane, x[u]);
      }
      if (i == SPB - 1) {
        pages = pages_next;
        pages_next = load_pages(begin + (s + 1 + SPB) * TOK);
      }
    };
    if (w0 < w1) {
      pages = load_pages(begin + w0 * TOK);
      pages_next = load_pages(begin + (w0 + SPB) * TOK);
    }

    // query columns: lane (g, r) holds column r of every block, the chunks' elements
    f16x8 qf[TERMS][NQ][KC];
    float csc[NQ], m[NQ], l[NQ];
    int32_t limit[NQ], floor_[NQ];                 // the column attends to floor_ <= t < limit
    f32x4 acc[NQ][NJ];
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      const int32_t col = col0 + 16 * n + r < cols ? col0 + 16 * n + r : cols - 1;   // past the end: never written
      const int32_t qi = col / a.by_group, pos = seq.n - seq.m + qi;
      const int64_t off = (seq.q0 + qi) * a.ldq + (int64_t)(kh * group + (col - qi * group)) * D;
      float v[KC][8];
      float amax = 0.0f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        const int d0 = D == 64 ? 16 * g + 8 * c : 128 * (c / 4) + 32 * g + 8 * (c % 4);
        load8<F32>(a.q, off + d0, v[c]);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = __builtin_fmaxf(amax, __builtin_fabsf(v[c][e]));
      }
      amax = max_xor32(max_xor16(amax));
      const float up = a.scale < 0.0f ? -query_up(amax) : query_up(amax);
      csc[n] = score_factor(a.scale, kg, amax);
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float x = v[c][i] * up;
          const _Float16 hi = (_Float16)x;
          qf[0][n][c][i] = hi;
          if constexpr (F32) qf[TERMS - 1][n][c][i] = (_Float16)(x - (float)hi);
        }
      limit[n] = pos + 1;
      floor_[n] = a.window ? pos - a.window + 1 : 0;
      m[n] = kNegBig;
      l[n] = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) acc[n][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    bool wide = false;
#pragma unroll
    for (int n = 0; n < NQ; ++n) wide |= __builtin_amdgcn_ballot_w64(csc[n] > kWideFactor) != 0;
    if (wide) {
#pragma unroll
      for (int n = 0; n < NQ; ++n) {
        s_c[wave][16 * n + r] = csc[n];            // each lane reads what it wrote
        csc[n] = 1.0f;
      }
    }
    const int32_t all_lo = wide ? INT32_MAX : sp.all_lo;   // wide: every step takes the slower way

    if (w0 < w1) {
      Granule<D> cur[NG], nxt[NG];
      issue(w0, nxt);
      for (int32_t s = w0; s < w1; ++s) {
#pragma unroll
        for (int u = 0; u < NG; ++u) cur[u] = nxt[u];
        if (s + 1 < w1) issue(s + 1, nxt);
        const int32_t t0 = begin + s * TOK;
        const bool edge = t0 < all_lo || t0 + TOK > sp.all_hi;

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
          if (edge) {
            const int32_t upto = limit[n] - t0 - 4 * g, from = floor_[n] - t0 - 4 * g;
#pragma unroll
            for (int u = 0; u < NG; ++u)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (16 * u + i >= upto || 16 * u + i < from) sc[n][u][i] = -__builtin_inff();
            if (wide) {
              const float factor = s_c[wave][16 * n + r];
#pragma unroll
              for (int u = 0; u < NG; ++u) sc[n][u] *= factor;
            }
          }
          const float top = max_xor32(max_xor16(max_of(sc[n]))) * csc[n];
          if (__builtin_amdgcn_ballot_w64(top - m[n] > 15.0f)) {
            const float m1 = __builtin_fmaxf(m[n], top - 7.0f);
            const float f = __builtin_amdgcn_exp2f(m[n] - m1);
            m[n] = m1;
            l[n] *= f;
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[n][j] *= f;
          }
#pragma unroll
          for (int k = 0; k < NG / 2; ++k)
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
              const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][2 * k + i / 4][i % 4], csc[n], -m[n]));
              const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[n][2 * k + i / 4][i % 4 + 1], csc[n], -m[n]));
              l[n] += x + y;
              const f16x2 hi = to_f16(x, y);
              pf[0][n][k][i] = hi[0];
              pf[0][n][k][i + 1] = hi[1];
              if constexpr (F32) {
                const f16x2 lo = to_f16(x - (float)hi[0], y - (float)hi[1]);
                pf[TERMS - 1][n][k][i] = lo[0];
                pf[TERMS - 1][n][k][i + 1] = lo[1];
              }
            }
        }

        // O^T += V^T P^T: rows = elements NJ r + j
        if (t0 < sp.lo || t0 + TOK > seq.n) {
#pragma unroll
          for (int u = 0; u < NG; ++u) cur[u].vs = live_scales(cur[u].vs, t0 + 16 * u + 4 * g, sp.lo, seq.n);
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
              value_words<D>(cur[2 * k + u].v, part, w);
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

    // join the waves of each column group
    __syncthreads();                               // s_m, s_l, s_o of the work before are read
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      l[n] = sum_xor32(sum_xor16(l[n]));
      if (g == 0) {
        s_m[wave][16 * n + r] = m[n];
        s_l[wave][16 * n + r] = l[n];
      }
    }
    __syncthreads();
#pragma unroll
    for (int n = 0; n < NQ; ++n) {
      float top = m[n];
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float x = s_m[w][16 * n + r];
        if ((w & ((1 << cs) - 1)) == cg) top = __builtin_fmaxf(top, x);
      }
      const float f = __builtin_amdgcn_exp2f(m[n] - top);
      if (n) __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float* dst = &s_o[wave][r * LDO + NJ * (4 * g + i)];
#pragma unroll
        for (int j = 0; j < NJ; j += 4)
          *reinterpret_cast<f32x4*>(dst + j) =
              f32x4{acc[n][j][i] * f, acc[n][j + 1][i] * f, acc[n][j + 2][i] * f, acc[n][j + 3][i] * f};
      }
      __syncthreads();
      // thread = (column, D / 16 elements) of each column group in turn
      const int c = threadIdx.x >> 4, part = threadIdx.x & 15;
      for (int h = 0; h < 1 << cs; ++h) {
        const int32_t col = col_first + h * 16 * NQ + 16 * n + c;
        if (col >= cols) break;
        float top_c = kNegBig, sum = 0.0f, out[NJ] = {};
        auto add = [&](int w) {
          sum += s_l[w][16 * n + c] * __builtin_amdgcn_exp2f(s_m[w][16 * n + c] - top_c);
#pragma unroll
          for (int j = 0; j < NJ; j += 4) {
            const f32x4 x = *reinterpret_cast<const f32x4*>(&s_o[w][c * LDO + part * NJ + j]);
#pragma unroll
            for (int e = 0; e < 4; ++e) out[j + e] += x[e];
          }
        };
        if (cs == 0) {                             // the usual case, its reads side by side
#pragma unroll
          for (int w = 0; w < W; ++w) top_c = __builtin_fmaxf(top_c, s_m[w][16 * n + c]);
#pragma unroll
          for (int w = 0; w < W; ++w) add(w);
        } else {
          for (int w = h; w < W; w += 1 << cs) top_c = __builtin_fmaxf(top_c, s_m[w][16 * n + c]);
          for (int w = h; w < W; w += 1 << cs) add(w);
        }
        if (whole) {
          const int32_t qi = col / a.by_group;
          const int head = kh * group + (col - qi * group);
          const float f = sum == 0.0f ? 0.0f : vg / sum;
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
            a.lse[(seq.q0 + qi) * a.n_q_heads + head] =
                sum == 0.0f ? -__builtin_inff() : (top_c + __builtin_log2f(sum)) * kLn2;
        } else {
          float* dst = piece_at(a, D, blockIdx.x, col - col_first);
#pragma unroll
          for (int j = 0; j < NJ; j += 4)
            *reinterpret_cast<f32x4*>(dst + 4 + part * NJ + j) = f32x4{out[j], out[j + 1], out[j + 2], out[j + 3]};
          if (part == 0) {
            dst[0] = top_c;
            dst[1] = sum;
          }
        }
      }
    }
    }
  }
}

// The joined row of column c of an item: o = sum_i 2^(M_i - M) O_i / sum_i 2^(M_i - M) l_i
template <int D, bool F32, int E>
__device__ __forceinline__ void store_joined(const KvAttnArgs& a, const ItemPieces& item, int32_t c, int first,
                                             const float (&x)[E], float top, float sum) {
  const int32_t col = item.first_col + c, qi = col / a.by_group, tok = item.q0 + qi;
  const int head = item.kh * (int)a.by_group.d + col - qi * (int)a.by_group.d;
  const float g = sum == 0.0f ? 0.0f : a.v_gscale[item.kh] / sum;
  const int64_t off = (int64_t)tok * a.ldo + (int64_t)head * D + first;
  if constexpr (F32) {
#pragma unroll
    for (int e = 0; e < E; ++e) reinterpret_cast<float*>(a.o)[off + e] = x[e] * g;
  } else if constexpr (E == 1) {
    reinterpret_cast<uint16_t*>(a.o)[off] = (uint16_t)f32_to_bf16_bits(x[0] * g);
  } else {
#pragma unroll
    for (int e = 0; e < E; e += 2)
      *reinterpret_cast<uint32_t*>(reinterpret_cast<uint16_t*>(a.o) + off + e) = pack_bf16(x[e] * g, x[e + 1] * g);
  }
  if (a.lse && first == 0)
    a.lse[(int64_t)tok * a.n_q_heads + head] = sum == 0.0f ? -__builtin_inff() : (top + __builtin_log2f(sum)) * kLn2;
}

// Join the pieces of the item that a worker began, few pieces: a wave per query column, a
// lane D / 64 elements, four pieces' loads at a time.
template <int D, bool F32>
__global__ __launch_bounds__(256) void k_kv_join(KvAttnArgs a) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 63;
  const int32_t id = (int32_t)blockIdx.x * 4 + __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int32_t worker = id / a.by_tile_cols, c = id - worker * a.tile_cols;
  if (worker >= a.blocks) return;
  const ItemPieces item = static_cast<const ItemPieces*>(a.pieces)[worker];
  if (c >= item.cols) return;
  const int32_t n = item.pieces;
  float top = kNegBig, sum = 0.0f, x[E] = {};
  for (int32_t i0 = 0; i0 < n; i0 += 4) {
    float m[4], l[4], v[4][E];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int32_t k = i0 + i < n ? i0 + i : n - 1;
      const float* p = piece_at(a, D, worker + k, c);
      m[i] = p[0];
      l[i] = p[1];
#pragma unroll
      for (int e = 0; e < E; ++e) v[i][e] = p[4 + lane * E + e];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i0 + i >= n) break;
      const float t = __builtin_fmaxf(top, m[i]);
      const float f = __builtin_amdgcn_exp2f(top - t), g = __builtin_amdgcn_exp2f(m[i] - t);
      top = t;
      sum = sum * f + l[i] * g;
#pragma unroll
      for (int e = 0; e < E; ++e) x[e] = x[e] * f + v[i][e] * g;
    }
  }
  store_joined<D, F32>(a, item, c, lane * E, x, top, sum);
}

// The same for many pieces: a workgroup per query column.  The pieces' factors go to LDS
// first, then D / 4 threads take four elements of a piece each, 1024 / D pieces at a time,
// with no load depending on another.
template <int D, bool F32>
__global__ __launch_bounds__(256) void k_kv_join_many(KvAttnArgs a) {
  constexpr int TPS = D / 4, LANES = 256 / TPS;      // threads per piece, pieces side by side
  __shared__ float s_f[kMostPieces], s_red[4], s_sum[4];
  __shared__ f32x4 s_x[LANES][TPS];
  const int tid = threadIdx.x;
  const int32_t worker = (int32_t)blockIdx.x / a.by_tile_cols, c = (int32_t)blockIdx.x - worker * a.tile_cols;
  const ItemPieces item = static_cast<const ItemPieces*>(a.pieces)[worker];
  if (c >= item.cols) return;
  const int32_t n = item.pieces;
  auto piece = [&](int i) { return piece_at(a, D, worker + i, c); };
  float m[kMostPieces / 256], l[kMostPieces / 256], top = kNegBig;
#pragma unroll
  for (int i = 0; i < kMostPieces / 256; ++i) {
    m[i] = kNegBig;
    l[i] = 0.0f;
    if (tid + 256 * i < n) {
      const f32x4 ml = *reinterpret_cast<const f32x4*>(piece(tid + 256 * i));
      m[i] = ml[0];
      l[i] = ml[1];
    }
    top = __builtin_fmaxf(top, m[i]);
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off));
  if ((tid & 63) == 0) s_red[tid >> 6] = top;
  __syncthreads();
  top = __builtin_fmaxf(__builtin_fmaxf(s_red[0], s_red[1]), __builtin_fmaxf(s_red[2], s_red[3]));
  float sum = 0.0f;
#pragma unroll
  for (int i = 0; i < kMostPieces / 256; ++i) {
    const float f = __builtin_amdgcn_exp2f(m[i] - top);
    s_f[tid + 256 * i] = f;
    sum += l[i] * f;
  }
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
  if ((tid & 63) == 0) s_sum[tid >> 6] = sum;
  __syncthreads();
  sum = (s_sum[0] + s_sum[1]) + (s_sum[2] + s_sum[3]);
  const int part = tid % TPS, lane = tid / TPS;
  f32x4 x = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int i = lane; i < n; i += LANES) x += *reinterpret_cast<const f32x4*>(piece(i) + 4 + 4 * part) * s_f[i];
  s_x[lane][part] = x;
  __syncthreads();
  if (tid >= TPS) return;
#pragma unroll
  for (int i = 1; i < LANES; ++i) x += s_x[i][part];
  const float out[4] = {x[0], x[1], x[2], x[3]};
  store_joined<D, F32>(a, item, c, 4 * part, out, top, sum);
}

template <int D, int NQ, bool F32>
hipError_t launch(const KvAttnArgs& a, hipStream_t s) {
  const int64_t blocks = a.blocks;
  if (a.tile_cols > 16 * NQ)
    hipLaunchKernelGGL((k_kv_attn<D, NQ, true, F32>), dim3((unsigned)blocks), dim3(64 * kAttnWaves), 0, s, a);
  else
    hipLaunchKernelGGL((k_kv_attn<D, NQ, false, F32>), dim3((unsigned)blocks), dim3(64 * kAttnWaves), 0, s, a);
  const hipError_t e = hipGetLastError();
  return e == hipSuccess && a.n_workers ? launch_kv_join(a, F32 ? InType::F32 : InType::BF16, D, s) : e;
}

template <int D, bool F32>
hipError_t join(const KvAttnArgs& a, hipStream_t s) {
  const unsigned columns = (unsigned)a.blocks * a.tile_cols;
  if (a.n_workers > 8 * (a.blocks - a.n_workers))             // more than 8 pieces an item
    hipLaunchKernelGGL((k_kv_join_many<D, F32>), dim3(columns), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((k_kv_join<D, F32>), dim3((columns + 3) / 4), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_join(const KvAttnArgs& a, InType t, int32_t D, hipStream_t s) {
  const bool f32 = t == InType::F32;
  if (D == 64) return f32 ? join<64, true>(a, s) : join<64, false>(a, s);
  if (D == 128) return f32 ? join<128, true>(a, s) : join<128, false>(a, s);
  return f32 ? join<256, true>(a, s) : join<256, false>(a, s);
}

KvAttnPlan kv_attn_plan(InType t, int64_t T, int32_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t D,
                        int64_t max_q_len, int64_t max_kv_len, int64_t window) {
  KvAttnPlan p{};
  const int64_t cols = (max_q_len < T ? max_q_len : T) * (n_q_heads / n_kv_heads);
  // From one full tile of query columns on, decoding a key once for all of them pays.  This
  // kernel / kvprefill.hip, us: 1 x 16384 keys and 256 columns 64 / 53, 1024 columns 123 / 93; 8 x
  // 4096 and 256 columns 81 / 66, but 128 columns 56 / 58; 32 x 4096 and 256 columns 245 / 175, but 128
  // columns 127 / 146; head dimension 256, 1 x 16384, 512 columns 81 / 61; 64, 2 x 4096, 512 columns 44 / 35.
  if (t == InType::BF16 && cols >= kv_prefill_cols()) {
    p.prefill = true;
    p.tile_cols = kv_prefill_cols();
    const int64_t pairs = (int64_t)batch * n_kv_heads, tiles = (cols + p.tile_cols - 1) / p.tile_cols;
    p.col_tiles = kv_planned_tiles(tiles, pairs, kv_prefill_threads());
    const int64_t items = pairs * p.col_tiles;
    p.blocks = (int32_t)items;
    // Fewer items than compute units: cut along the keys, one workgroup a compute unit.
    // Whole / cut: 8 items of 16384 keys 452 / 53 us, 128 items of 4096 keys
    // 123 / 101.  (A lane of the kernel looks up a sequence: at most 64.)
    const bool few = items <= 160;
    // So are the items of sequences of unlike lengths, which n_tokens shows, where the longest
    // run far longer than the others (all timed before later steps): 3 x up to 2048 new tokens of up
    // to 16384 (head dimension 256) 1337 / 903 us, 4 x 1024 of 16384 814 / 587, 2 x 2048 of 8192 387 / 312.  Equal lengths lose by it, 4 x
    // 1024 of 16384 974 / 1004 us, 1 x 2048 of 8192 245 / 286, and short ones, 16 x 1024 of 4096 (64) 131 / 148.
    const bool unlike = 8 * T <= 7 * (int64_t)batch * max_q_len && items <= 512 && max_kv_len >= 64 * (D == 256 ? 64 : 128);
    if ((few || unlike) && batch <= 64) {
      p.n_workers = (int32_t)(few ? 256 - items / 2 : 384);
      p.blocks = (int32_t)(p.n_workers + items);
      p.min_steps = 2;
      p.pieces_at = (int64_t)p.blocks * p.tile_cols * (D + 4) * (int64_t)sizeof(float);
      p.workspace = p.pieces_at + (int64_t)p.blocks * kItemPiecesBytes;
    }
    return p;
  }
  // two column blocks share a decoded granule where their registers fit, or nearly (head dimension
  // 128: 9 to 14 spill)
  p.nq = cols > 16 && (D == 64 || (D == 128 && t == InType::BF16)) ? 2 : 1;
  const int64_t blk = 16 * p.nq;
  p.tile_cols = (int32_t)(cols < blk * kAttnWaves ? cols : blk * kAttnWaves);
  const int64_t pairs = (int64_t)batch * n_kv_heads;
  p.col_tiles = kv_planned_tiles((cols + p.tile_cols - 1) / p.tile_cols, pairs, 64 * kAttnWaves);
  const int64_t items = pairs * p.col_tiles;
  p.blocks = (int32_t)items;
  const int64_t tok = D == 256 ? 32 : 64, waves = cols <= blk ? 4 : (cols <= 2 * blk ? 2 : 1);
  // keys that a tile attends to, at most
  const int64_t span = window > 0 && window + max_q_len < max_kv_len ? window + max_q_len : max_kv_len;
  const int64_t steps = (span + tok - 1) / tok;
  // Whole items where a wave's part of one is short: cutting costs the join's launch and
  // latency (4.5 us) and pays where it brings idle compute units to work.  Measured, whole
  // / cut: 256 items of up to 64 steps 29.7 / 32.8 us, 128 of 32 15.8 / 20.2 and of 64 26.7 / 22.0,
  // 64 of 32 15.1 / 18.8, 32 of 32 15.5 / 11.3.
  const int64_t alone = items >= 256 ? 16 : (items >= 64 ? 8 : 4);
  if (items >= 1024 || steps <= alone * waves) return p;
  p.min_steps = (int32_t)waves;                           // a step for each wave
  // about as many pieces as run at once: rounding up adds half a piece to an item
  p.n_workers = (int32_t)(items > kMaxWorkers ? kMaxWorkers / 2 : kMaxWorkers - items / 2);
  p.blocks = (int32_t)(p.n_workers + items);
  p.pieces_at = (int64_t)p.blocks * p.tile_cols * (D + 4) * (int64_t)sizeof(float);
  p.workspace = p.pieces_at + (int64_t)p.blocks * kItemPiecesBytes;
  return p;
}

hipError_t launch_kv_attn(KvAttnArgs a, const KvAttnPlan& p, InType t, int32_t D, hipStream_t s) {
  a.n_workers = p.n_workers;
  a.blocks = p.blocks;
  a.min_steps = p.min_steps;
  a.tile_cols = p.tile_cols;
  a.col_tiles = p.col_tiles;
  a.by_group = fast_div((uint32_t)(a.n_q_heads / a.geom.n_kv_heads));
  a.by_heads = fast_div((uint32_t)a.geom.n_kv_heads);
  a.by_tile_cols = fast_div((uint32_t)a.tile_cols);
  a.by_col_tiles = fast_div((uint32_t)a.col_tiles);
  a.by_pairs = fast_div((uint32_t)a.batch * (uint32_t)a.geom.n_kv_heads);
  a.pieces = reinterpret_cast<uint8_t*>(a.part) + p.pieces_at;
  if (p.prefill) return launch_kv_prefill(a, D, s);
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
