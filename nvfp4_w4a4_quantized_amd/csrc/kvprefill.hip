// Attention of many query columns over the paged NVFP4 cache (bf16): prompts and chunks.
// The mathematics and numerics are those of kvattn.hip; what differs is the work split.
//
// Here the two matrix products bound the kernel, so keys and values are decoded once per
// workgroup: eight waves share tiles of tokens, decoded to f16 (exactly) into LDS, and each
// wave takes 32 query columns through them with MFMA 32x32x16.  S^T = K q^T leaves a lane with
// scores of one column, 16 of every 32 tokens (tokens 8 (i / 4) + 4 h + i % 4, h = lane / 32), which
// are in place the B operand of O^T = V^T P^T when its K axis takes the tokens of a granule in
// the order quads 0, 2, 1, 3; V^T is written to LDS in that order, so the weights never leave
// the registers.
//
// Where the registers allow (D <= 128) a wave works on three blocks of 32 tokens at once: the
// scores of block j + 1 and the output of block j - 1 on the matrix unit beside the softmax of
// block j on the vector unit, neither waiting for the other.
//
// LDS, two decoded tiles of each (a tile is decoded while the one before is used; one barrier
// per tile):
//   K   [tokens][D], V^T [D][tokens], each row one 16-byte chunk longer than its data
// so that a wave's 16-byte reads of 16 rows meet every bank once, and every address is one base
// plus a constant (with exclusive-or swizzles instead: 14 more vector instructions on the 100 of a
// block of 32 tokens, prompts of 8192 tokens 572 us against 543).  Row 16 i + p of V^T is dimension
// p D/16 + i, so that the 16 parts of a quad are decoded into 16 neighbouring rows.
// D <= 128: tiles of 128 tokens, wave w loads and decodes granule w.  D = 256: 64 tokens (what LDS
// holds), wave w granule w % 4, keys (w < 4) or values.
//
// A workgroup has one item (256 query columns of a kv head and sequence).  Where these are
// fewer than the compute units, or of unlike lengths, items are cut along the keys into equal pieces, one per
// workgroup, which k_kv_join puts together, as in kvattn.hip: 256 columns of 16384 keys in 53 us
// instead of 452.
//
// What bounds it: matrix and vector instructions of two waves per SIMD that only partly overlap.  8192
// tokens, 32 / 8 heads of 128: 527 to 617 us by card, 890 to 1043 TFLOP/s (a large f16 matrix product
// reaches 1095 to 1193 there, at the clock that its power leaves); the matrix unit is busy 47 % of the
// cycles, the vector unit 54 %, LDS 36 %, and waves wait 32 %.  Head dimension 256, whose accumulators leave no
// registers for the pipeline (20 or 26 spill, four or five accesses of them in the loop over the
// tiles): 3 sequences of 300 to 2048 new tokens of up to 16384 862 to 952 us, 879 to 971 TFLOP/s, the
// matrix unit 42 % busy, waves waiting 45 %.  64 columns a wave at one wave per SIMD (512 registers)
// took 845 us where this took 606.
#include <type_traits>

#include "kv_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kPrefillWaves = 8;
constexpr int kPrefillCols = 32 * kPrefillWaves;
template <int D>
constexpr int kTok = D == 256 ? 64 : 128;          // tokens of a tile

__device__ __forceinline__ f32x16 mfma32(f16x8 a, f16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

// Places in the decoded tiles: rows of 16-byte chunks, one chunk longer than their data.
template <int D>
constexpr int kKRow = 2 * D + 16;
template <int D>
constexpr int kVRow = 2 * kTok<D> + 16;
template <int D>
constexpr int kKTile = kTok<D> * kKRow<D>;
template <int D>
constexpr int kVTile = D * kVRow<D>;
// after the tiles: the columns' score factors where a wave's are wide
template <int D>
constexpr int kFactors = 2 * (kKTile<D> + kVTile<D>);

template <typename T>
__device__ __forceinline__ __attribute__((address_space(3))) T& lds_at(uint32_t at) {
  return *reinterpret_cast<__attribute__((address_space(3))) T*>(at);
}

__device__ __forceinline__ f32x16 zeros16() {
  f32x16 x;
#pragma unroll
  for (int e = 0; e < 16; ++e) x[e] = 0.0f;
  return x;
}

// Plain loads of a granule's pieces (buffer loads, whose descriptors take scalar registers, were
// slower here: head dimension 256 1376 us against 1322 us)
template <int N>
__device__ __forceinline__ void read_dwords(const uint8_t* p, uint32_t* d) {
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

// A tile of query columns: the keys it attends to, the first of them, and `steps` tiles of tokens
// from granule-aligned `begin` on
struct TileSpan {
  int32_t lo, begin, steps;
};
template <int D>
__device__ __forceinline__ TileSpan tile_span(const KvAttnArgs& a, const SeqInfo& seq, int32_t tile, int group) {
  const int32_t cols = seq.m * group, first = tile * kPrefillCols;
  const Span s = span_of(seq, first, first + kPrefillCols < cols ? first + kPrefillCols : cols, a.by_group, a.window);
  TileSpan t;
  t.lo = s.lo;
  t.begin = s.lo & ~15;
  t.steps = seq.n > 0 ? (s.hi - t.begin + kTok<D> - 1) / kTok<D> : 0;
  return t;
}
__device__ __forceinline__ int32_t tiles_of(const SeqInfo& seq, int group) {
  return (seq.m * group + kPrefillCols - 1) / kPrefillCols;
}
__device__ __forceinline__ int32_t planned_tiles(const KvAttnArgs& a, const SeqInfo& seq, int group) {
  const int32_t t = tiles_of(seq, group);
  return t < a.col_tiles ? t : a.col_tiles;
}

// SPLIT: workgroups have pieces of items instead of items (a template parameter: its
// registers cost the other form 2 to 5 %)
template <int D, bool SPLIT>
__global__ __launch_bounds__(64 * kPrefillWaves, 2) void k_kv_prefill(KvAttnArgs a) {
  constexpr bool PIPE = D <= 128;
  constexpr int TOK = kTok<D>;
  constexpr int KD = D / 32;                       // dwords of codes a lane decodes, keys and values each
  constexpr int NB = D / 32;                       // 32-row blocks of O^T
  constexpr int KS = D / 16;                       // K steps of the first product
  extern __shared__ __attribute__((aligned(256))) uint8_t shared[];
  // LDS addresses as numbers: one register each, offsets in the instruction
  const uint32_t lds = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) uint8_t*)shared;

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hkv = a.geom.n_kv_heads, group = (int)a.by_group.d;
  // this workgroup's item, and its steps [s_first, s_last) of it (s_last < 0: all)
  int b, kh, tile0;
  int32_t s_first = 0, s_last = -1;
  SeqInfo seq;
  if constexpr (!SPLIT) {
    // the longest spans (last tiles) start first; workgroups side by side differ in the head
    const int turn = (int)blockIdx.x / a.by_pairs, pair = (int)blockIdx.x - turn * (int)a.by_pairs.d;
    b = pair / a.by_heads;
    kh = pair - b * hkv;
    seq = seq_info(a, b);
    const int32_t tiles = tiles_of(seq, group);
    tile0 = (tiles < a.col_tiles ? tiles : a.col_tiles) - 1 - turn;
    if (tile0 < 0) return;
  } else {
    // Few items: each is cut into equal pieces of at most S steps (tokens of a tile), S all
    // steps of the call by n_workers, as in kvattn.hip; a lane counts every 64th tile.
    const SeqTable seqs(a, lane);
    float total = 0.0f;
    for (b = 0; b < a.batch; ++b) {
      seq = seqs.at(a, b);
      const int32_t tiles = planned_tiles(a, seq, group);
      for (int32_t t = lane; t < tiles; t += 64) total += (float)tile_span<D>(a, seq, t, group).steps;
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) total += __shfl_xor(total, off);
    int32_t S = (int32_t)(total * (float)hkv * 1.0001f / (float)a.n_workers) + 1;
    S = S < a.min_steps ? a.min_steps : S;
    auto pieces_of = [&](int32_t steps) {
      return steps <= S ? 1 : (int32_t)((uint32_t)(steps + S - 1) / (uint32_t)S);
    };
    int32_t rest = (int32_t)blockIdx.x, tiles = 0, of_head = 0;
    for (b = 0; b < a.batch; ++b) {
      seq = seqs.at(a, b);
      tiles = planned_tiles(a, seq, group);
      of_head = 0;
      for (int32_t t = lane; t < tiles; t += 64) of_head += pieces_of(tile_span<D>(a, seq, t, group).steps);
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) of_head += __shfl_xor(of_head, off);
      of_head = __builtin_amdgcn_readfirstlane(of_head);
      if (rest < of_head * hkv) break;
      rest -= of_head * hkv;
    }
    if (b == a.batch) {
      if (threadIdx.x == 0) static_cast<ItemPieces*>(a.pieces)[blockIdx.x].cols = 0;
      return;
    }
    kh = (int32_t)((uint32_t)rest / (uint32_t)of_head);
    rest -= kh * of_head;
    int32_t pieces = 1;
    for (int32_t t0 = 0;; t0 += 64) {
      const int32_t own = t0 + lane < tiles ? pieces_of(tile_span<D>(a, seq, t0 + lane, group).steps) : 0;
      int32_t upto = own;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int32_t x = __shfl_up(upto, off);
        if (lane >= off) upto += x;
      }
      const uint64_t past = __builtin_amdgcn_ballot_w64(upto > rest);
      if (past) {
        const int first = __builtin_ctzll(past);
        tile0 = t0 + first;
        pieces = __builtin_amdgcn_readlane(own, first);
        rest -= __builtin_amdgcn_readlane(upto - own, first);
        break;
      }
      rest -= __builtin_amdgcn_readlane(upto, 63);
    }
    const int32_t steps = tile_span<D>(a, seq, tile0, group).steps;
    if (pieces > 1) {
      const int32_t q = (int32_t)((uint32_t)steps / (uint32_t)pieces), more = steps - q * pieces;
      s_first = rest * q + (rest < more ? rest : more);
      s_last = s_first + q + (rest < more);
    }
    if (threadIdx.x == 0) {
      const int32_t fc = tile0 * kPrefillCols, left = seq.m * group - fc;
      ItemPieces* const p = static_cast<ItemPieces*>(a.pieces) + blockIdx.x;
      p->cols = pieces > 1 && rest == 0 ? (left < kPrefillCols ? left : kPrefillCols) : 0;
      p->pieces = pieces;
      p->q0 = seq.q0;
      p->first_col = fc;
      p->kh = kh;
    }
  }
  const int32_t cols = seq.m * group;
  const int32_t last_page = (seq.n - 1) >> a.geom.page_shift, last_granule = (seq.n - 1) >> 4;
  const int per_head = 1 << (a.geom.page_shift - 4);
  const float kg = a.k_gscale[kh], vg = a.v_gscale[kh];
  const int h = lane >> 5, c32 = lane & 31;
  const int gran = D == 256 ? wave & 3 : wave;      // this wave's granule of a tile

  // tiles past the planned ones are done whole, with the first piece of one of those
  for (int32_t tile = tile0; (int64_t)tile * kPrefillCols < cols; tile += a.col_tiles) {
    const bool whole = !SPLIT || s_last < 0 || tile != tile0;
    if (SPLIT && tile != tile0 && s_first > 0) break;
    const int32_t col_first = tile * kPrefillCols;
    const int32_t col_end = col_first + kPrefillCols < cols ? col_first + kPrefillCols : cols;
    const TileSpan span = tile_span<D>(a, seq, tile, group);
    const int32_t begin = whole ? span.begin : span.begin + s_first * TOK;
    const int32_t steps = whole ? span.steps : s_last - s_first;

    // this wave's columns (past the tile's end: its last one again, never written)
    const int32_t col0 = col_first + 32 * wave;
    const int32_t w0 = col0 < col_end ? col0 : col_end - 1;
    const int32_t w1 = col0 + 32 < col_end ? col0 + 32 : col_end;
    const Span sp = span_of(seq, w0, w1, a.by_group, a.window);

    // loads of tile s: this wave's granule, its page id known one tile ahead
    auto page_of = [&](int32_t s) -> int32_t {
      int32_t pg = (begin + s * TOK + 16 * gran) >> a.geom.page_shift;
      pg = pg < last_page ? pg : last_page;
      const int32_t id = a.table[(int64_t)b * a.ld_table + pg];
      return id < 0 ? 0 : (id >= a.geom.n_pages ? (int32_t)a.geom.n_pages - 1 : id);
    };
    auto granule = [&](int32_t s, int32_t id) {
      int32_t gr = (begin + s * TOK) / 16 + gran;
      gr = gr < last_granule ? gr : last_granule;
      return a.cache + (int64_t)id * a.geom.page_bytes +
             (int64_t)(kh * per_head + (gr & (per_head - 1))) * kv_granule_bytes(D);
    };
    // the quad of tokens and part of a granule's values that this lane decodes
    const int quad = lane >> 4, part = lane & 15;
    // (D = 256: a wave holds either)
    uint32_t rk[KD] = {}, rv_[D == 256 ? 1 : KD] = {}, ksc = 0, vsc_ = 0;
    uint32_t* const rv = D == 256 ? rk : rv_;
    uint32_t& vsc = D == 256 ? ksc : vsc_;
    auto load_k = [&](int32_t s, int32_t id) {
      const uint8_t* p = granule(s, id);
      if constexpr (D == 256) {          // a quarter of either half of a token's row
        const uint8_t *c = p + (lane >> 2) * 128 + (lane & 3) * 16, *f = p + 8 * D + (lane >> 2) * 16 + (lane & 3) * 2;
        read_dwords<4>(c, rk);
        read_dwords<4>(c + 64, rk + 4);
        ksc = *reinterpret_cast<const uint16_t*>(f) | (uint32_t)*reinterpret_cast<const uint16_t*>(f + 8) << 16;
      } else {                           // a quarter of a token's row
        read_dwords<KD>(p + lane * (D / 8), rk);
        ksc = D == 64 ? p[8 * D + lane] : *reinterpret_cast<const uint16_t*>(p + 8 * D + 2 * lane);
      }
    };
    auto load_v = [&](int32_t s, int32_t id) {
      const uint8_t* p = granule(s, id);
      read_dwords<KD>(p + 9 * D + (16 * quad + part) * (D / 8), rv);
      vsc = *reinterpret_cast<const uint32_t*>(p + 17 * D + (quad * (D / 16) + part * D / 256) * 4);
      const int32_t first = begin + s * TOK + 16 * gran;
      if (first < span.lo || first + 16 > seq.n) vsc = live_scales(vsc, first + 4 * quad, span.lo, seq.n);
    };
    // decode dword i of the loaded keys: a 16-byte chunk of a token's row
    auto decode_k = [&](uint32_t kb, int i) {               // kb: the lane's first chunk in the tile
      const f16x2 sc = bcast(scale_pair_f16(D == 256 ? ksc >> (16 * (i / 4)) : ksc), D == 64 ? 0 : (i >> 1) & 1);
      lds_at<f16x8>(kb + 16 * i + (i < 4 ? 0 : 192)) = decode8_f16(rk[i], sc);
    };
    // decode byte i of the four tokens' words of the loaded values: elements 2 i and 2 i + 1
    auto decode_v = [&](uint32_t vb, int i) {               // vb: the lane's first element in the tile
      f16x2 sc[2];
      sc[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(vsc, 1.0f, false);
      sc[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(vsc, 1.0f, true);
      uint32_t w[4], lo[2], hi[2];
      value_words<D>(rv, i / 4, w);
      pair_tokens(w, lo, hi);
      typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
      auto put = [&](int j, f16x2 x, f16x2 y) {
        lds_at<f16x4>(vb + j * 16 * kVRow<D>) = f16x4{x[0], x[1], y[0], y[1]};
      };
      auto two = [&](auto sel) {
        constexpr int SEL = decltype(sel)::value;
        put(2 * i, cvt_fp4<SEL>(lo[0]) * sc[0], cvt_fp4<SEL>(lo[1]) * sc[1]);
        put(2 * i + 1, cvt_fp4<SEL>(hi[0]) * sc[0], cvt_fp4<SEL>(hi[1]) * sc[1]);
      };
      if (i % 4 == 0) two(std::integral_constant<int, 0>{});
      else if (i % 4 == 1) two(std::integral_constant<int, 1>{});
      else if (i % 4 == 2) two(std::integral_constant<int, 2>{});
      else two(std::integral_constant<int, 3>{});
    };
    const int kwbase = (16 * gran + lane / 4) * kKRow<D> + (lane % 4) * (D == 256 ? 4 : KD) * 16;
    const int vwbase = part * kVRow<D> + 32 * gran + 16 * (quad & 1) + 8 * (quad >> 1);

    int32_t id_next = 0;
    __syncthreads();                               // the tile before is done with LDS
    if (steps > 0) {
      const int32_t id = page_of(0);
      if (D != 256 || wave < 4) load_k(0, id);
      if (D != 256 || wave >= 4) load_v(0, id);
      id_next = page_of(1);
    }

    // query columns: B operand of K step k: elements 16 k + 8 h + j of column c32
    f16x8 qf[KS];
    int32_t col = col0 + c32;
    col = col < col_end ? col : col_end - 1;
    const int32_t qi = col / a.by_group;
    const int head = kh * group + (col - qi * group);
    float amax = 0.0f;
    {
      u32x4 raw[KS];
      const uint16_t* src = reinterpret_cast<const uint16_t*>(a.q) + (seq.q0 + qi) * a.ldq + (int64_t)head * D + 8 * h;
#pragma unroll
      for (int k = 0; k < KS; ++k) raw[k] = *reinterpret_cast<const u32x4*>(src + 16 * k);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          amax = __builtin_fmaxf(amax, __builtin_fabsf(__uint_as_float(raw[k][e] << 16)));
          amax = __builtin_fmaxf(amax, __builtin_fabsf(__uint_as_float(raw[k][e] & 0xFFFF0000u)));
        }
      amax = max_xor32(amax);
      const float up = a.scale < 0.0f ? -query_up(amax) : query_up(amax);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const f16x2 x = to_f16(__uint_as_float(raw[k][e] << 16) * up, __uint_as_float(raw[k][e] & 0xFFFF0000u) * up);
          qf[k][2 * e] = x[0];
          qf[k][2 * e + 1] = x[1];
        }
    }
    float csc = score_factor(a.scale, kg, amax);
    const bool wide = __builtin_amdgcn_ballot_w64(csc > kWideFactor) != 0;
    if (wide) {
      lds_at<float>(lds + kFactors<D> + 4 * (32 * wave + c32)) = csc;   // each lane reads what it wrote
      csc = 1.0f;
    }
    const int32_t all_lo = wide ? INT32_MAX : sp.all_lo;   // wide: every block takes the slower way
    const int32_t pos = seq.n - seq.m + qi;
    const int32_t limit = pos + 1, floor_ = a.window ? pos - a.window + 1 : 0;
    float m = kNegBig, l = 0.0f;
    f32x16 acc[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) acc[i] = zeros16();

    // The parts of a block of 32 tokens, cut into KS pieces that the pipeline deals out: piece
    // i of the scores is K step i, piece i of the output one value operand, both read from LDS
    // PF pieces ahead.
    constexpr int PF = D == 256 ? 2 : 3;
    f16x8 kf[PF + 1], vf_[D == 256 ? 1 : PF + 1];
    f16x8* const vf = D == 256 ? kf : vf_;           // one at a time there
    const int kbase = c32 * kKRow<D> + 16 * h, vbase = c32 * kVRow<D> + 16 * h;
    auto read_k = [&](uint32_t kb, int b, int i) {          // kb: kbase in the tile
      kf[i % (PF + 1)] = lds_at<f16x8>(kb + 32 * kKRow<D> * b + 32 * i);
    };
    auto read_v = [&](uint32_t vb, int b, int i) {
      vf[i % (PF + 1)] = lds_at<f16x8>(vb + 32 * kVRow<D> * (i % NB) + 32 * (2 * b + i / NB));
    };
    auto score_piece = [&](f32x16& sc, int i) { sc = mfma32(kf[i % (PF + 1)], qf[i], sc); };
    auto output_piece = [&](const f16x8 p[2], int i) { acc[i % NB] = mfma32(vf[i % (PF + 1)], p[i / NB], acc[i % NB]); };
    // moves the reference M for the block from token t0 on; returns what the earlier sums are
    // scaled by
    auto reference = [&](int32_t t0, f32x16& sc) {
      if (t0 < all_lo || t0 + 32 > sp.all_hi) {
        const int32_t upto = limit - t0 - 4 * h, from = floor_ - t0 - 4 * h;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int32_t t = 8 * (e / 4) + e % 4;
          if (t >= upto || t < from) sc[e] = -__builtin_inff();
        }
        if (wide) {
          const float factor = lds_at<float>(lds + kFactors<D> + 4 * (32 * wave + c32));
#pragma unroll
          for (int e = 0; e < 16; ++e) sc[e] *= factor;
        }
        // masked in place (as two versions, the scores were copied in every block)
        asm volatile("" : "+v"(sc));
      }
      const float top = max_xor32(max_of(sc)) * csc;
      const float m1 = top - m > 15.0f ? __builtin_fmaxf(m, top - 7.0f) : m;
      const float f = __builtin_amdgcn_exp2f(m - m1);
      l *= f;
      m = m1;
      return f;
    };
    // weights of scores 2 i and 2 i + 1
    auto weight_pair = [&](const f32x16& sc, f16x8 p[2], int i) {
      const float x = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[2 * i], csc, -m));
      const float y = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[2 * i + 1], csc, -m));
      l += x + y;
      const f16x2 w = to_f16(x, y);
      p[i / 4][2 * (i % 4)] = w[0];
      p[i / 4][2 * (i % 4) + 1] = w[1];
    };
    auto rescale = [&](float f) {
      if (__builtin_amdgcn_ballot_w64(f != 1.0f)) {
#pragma unroll
        for (int i = 0; i < NB; ++i) acc[i] *= f;
      }
    };
    auto k_tile = [&](int32_t s) { return lds + (uint32_t)((s & 1) * kKTile<D>); };
    auto v_tile = [&](int32_t s) { return lds + (uint32_t)(2 * kKTile<D> + (s & 1) * kVTile<D>); };
    // an address that the compiler does not take out of the loop: with every chunk's address
    // in a register of its own the kernel spills
    auto fresh = [](uint32_t x) {
      asm volatile("" : "+v"(x));
      return x;
    };

    if (steps > 0) {
      if (D != 256 || wave < 4) {
#pragma unroll
        for (int i = 0; i < KD; ++i) decode_k(k_tile(0) + kwbase, i);
      }
      if (D != 256 || wave >= 4) {
#pragma unroll
        for (int i = 0; i < KS / 2; ++i) decode_v(v_tile(0) + vwbase, i);
      }
      if (steps > 1) {
        if (D != 256 || wave < 4) load_k(1, id_next);
        if (D != 256 || wave >= 4) load_v(1, id_next);
        id_next = page_of(2);
      }
      if constexpr (PIPE) {
        // the values "before" tile 0 meet weights of zero: they must not be NaN
#pragma unroll
        for (int at = 16 * threadIdx.x; at < kVTile<D>; at += 16 * 64 * kPrefillWaves)
          lds_at<u32x4>(v_tile(1) + at) = u32x4{0, 0, 0, 0};
      }
      __syncthreads();
      if constexpr (PIPE) {
        // one stage: scores of a block (kb, bk) into `next`, the weights of the block before it
        // (scores `now`, from token t0 on) into `w`, the output of the one before that (vb, bv;
        // weights `old`); pieces of the next tile's decoding in between
        auto stage = [&](uint32_t kt, int bk, uint32_t vt, int bv, int32_t t0, f32x16& next, f32x16& now,
                         f16x8 (&w)[2], const f16x8 (&old)[2], auto decode_piece) {
          float f = 1.0f;
          const uint32_t kb = fresh(kbase + kt), vb = fresh(vbase + vt);
          next = zeros16();
#pragma unroll
          for (int i = 0; i < PF; ++i) {
            read_k(kb, bk, i);
            read_v(vb, bv, i);
          }
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            __builtin_amdgcn_sched_barrier(0);
            if (i + PF < KS) {
              read_k(kb, bk, i + PF);
              read_v(vb, bv, i + PF);
            }
            score_piece(next, i);
            output_piece(old, i);
            if (i == 0) f = reference(t0, now);
            // 8 pairs over the pieces after the first
#pragma unroll
            for (int x = 0; x < 8; ++x)
              if (x >= (i - 1) * 8 / (KS - 1) && x < i * 8 / (KS - 1)) weight_pair(now, w, x);
            decode_piece(i);
          }
          // the weights and their sum are due here, not where they are used
          asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(l));
          __builtin_amdgcn_sched_barrier(0);
          rescale(f);
        };
        auto nothing = [](int) {};
        f32x16 sa = zeros16(), sb;
        f16x8 pa[2], pb[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 8; ++e) pb[k][e] = (_Float16)0.0f;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          read_k(k_tile(0) + kbase, 0, i);
          score_piece(sa, i);
        }
        // Past the last tile the decoder writes, from stale registers, what nothing reads unmasked.
        // The next keys are written after the reads of the tile before them and are due after the
        // second barrier, the next values after the second and due after the first.
        for (int32_t s = 0; s < steps; ++s) {
          const int32_t t0 = begin + s * TOK;
          stage(k_tile(s), 1, v_tile(s + 1), 3, t0, sb, sa, pa, pb, nothing);
          __syncthreads();
          const uint32_t kw = fresh(k_tile(s + 1) + kwbase);
          stage(k_tile(s), 2, v_tile(s), 0, t0 + 32, sa, sb, pb, pa, [&](int i) {
            if (i < KD) decode_k(kw, i);
          });
          if (s + 2 < steps) load_k(s + 2, id_next);
          stage(k_tile(s), 3, v_tile(s), 1, t0 + 64, sb, sa, pa, pb, nothing);
          __syncthreads();
          const uint32_t vw = fresh(v_tile(s + 1) + vwbase);
          stage(k_tile(s + 1), 0, v_tile(s), 2, t0 + 96, sa, sb, pb, pa, [&](int i) {
            if (i < KS / 2) decode_v(vw, i);
          });
          if (s + 2 < steps) {
            load_v(s + 2, id_next);
            id_next = page_of(s + 3);
          }
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          read_v(v_tile(steps - 1) + vbase, 3, i);
          output_piece(pb, i);
        }
      } else {
        for (int32_t s = 0; s < steps; ++s) {
          const uint32_t kw = fresh(k_tile(s + 1) + kwbase), vw = fresh(v_tile(s + 1) + vwbase);
          if (wave < 4) {
#pragma unroll
            for (int i = 0; i < KD; ++i) decode_k(kw, i);
          } else {
#pragma unroll
            for (int i = 0; i < KS / 2; ++i) decode_v(vw, i);
          }
          if (s + 2 < steps) {
            if (wave < 4) load_k(s + 2, id_next);
            else load_v(s + 2, id_next);
            id_next = page_of(s + 3);
          }
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            f32x16 sc = zeros16();
            f16x8 w[2];
            const uint32_t kb = fresh(k_tile(s) + kbase), vb = fresh(v_tile(s) + vbase);
#pragma unroll
            for (int i = 0; i < PF; ++i) read_k(kb, b, i);
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              __builtin_amdgcn_sched_barrier(0);
              if (i + PF < KS) read_k(kb, b, i + PF);
              score_piece(sc, i);
            }
            __builtin_amdgcn_sched_barrier(0);
            const float f = reference(begin + s * TOK + 32 * b, sc);
#pragma unroll
            for (int x = 0; x < 8; ++x) weight_pair(sc, w, x);
            asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(l));
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int i = 0; i < PF; ++i) read_v(vb, b, i);
            rescale(f);
#pragma unroll
            for (int i = 0; i < KS; ++i) {
              __builtin_amdgcn_sched_barrier(0);
              if (i + PF < KS) read_v(vb, b, i + PF);
              output_piece(w, i);
            }
            __builtin_amdgcn_sched_barrier(0);
          }
          __syncthreads();
        }
      }
    }

    // elements g and g + 8 of the blocks: consecutive dimensions, those of a part of the granule
    l = sum_xor32(l);
    if (col0 + c32 < col_end) {
      auto first_of = [&](int g) { return ((g & 4) * 2 + 4 * h + (g & 3)) * (D / 16); };
      if (whole) {
        const float f = l == 0.0f ? 0.0f : vg / l;
        uint16_t* dst = reinterpret_cast<uint16_t*>(a.o) + (seq.q0 + qi) * a.ldo + (int64_t)head * D;
#pragma unroll
        for (int g = 0; g < 8; ++g)
#pragma unroll
          for (int i = 0; i < NB; i += 2)
            *reinterpret_cast<u32x2*>(dst + first_of(g) + 2 * i) =
                u32x2{pack_bf16(acc[i][g] * f, acc[i][g + 8] * f), pack_bf16(acc[i + 1][g] * f, acc[i + 1][g + 8] * f)};
        if (a.lse && h == 0)
          a.lse[(seq.q0 + qi) * a.n_q_heads + head] = l == 0.0f ? -__builtin_inff() : (m + __builtin_log2f(l)) * kLn2;
      } else {
        float* dst = piece_at(a, D, blockIdx.x, col0 + c32 - col_first);
#pragma unroll
        for (int g = 0; g < 8; ++g)
#pragma unroll
          for (int i = 0; i < NB; i += 2)
            *reinterpret_cast<f32x4*>(dst + 4 + first_of(g) + 2 * i) =
                f32x4{acc[i][g], acc[i][g + 8], acc[i + 1][g], acc[i + 1][g + 8]};
        if (h == 0) {
          dst[0] = m;
          dst[1] = l;
        }
      }
    }
  }
}

template <int D, bool SPLIT>
hipError_t launch(const KvAttnArgs& a, hipStream_t s) {
  constexpr int bytes = kFactors<D> + 4 * kPrefillCols;
  const hipError_t e = lds_limit_once<k_kv_prefill<D, SPLIT>>(bytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_kv_prefill<D, SPLIT>), dim3((unsigned)a.blocks), dim3(64 * kPrefillWaves), bytes, s, a);
  const hipError_t launched = hipGetLastError();
  return SPLIT && launched == hipSuccess ? launch_kv_join(a, InType::BF16, D, s) : launched;
}

template <int D>
hipError_t launch(const KvAttnArgs& a, hipStream_t s) {
  return a.n_workers ? launch<D, true>(a, s) : launch<D, false>(a, s);
}

}  // namespace

int32_t kv_prefill_cols() { return kPrefillCols; }
int32_t kv_prefill_threads() { return 64 * kPrefillWaves; }

hipError_t launch_kv_prefill(const KvAttnArgs& a, int32_t D, hipStream_t s) {
  if (D == 64) return launch<64>(a, s);
  if (D == 128) return launch<128>(a, s);
  return launch<256>(a, s);
}

}  // namespace nvfp4
