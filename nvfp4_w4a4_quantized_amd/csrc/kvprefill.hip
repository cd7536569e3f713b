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
// tokens, 32 / 8 heads of 128: 519 to 551 us by card, 998 to 1060 TFLOP/s (a large f16
// matrix product reaches 1095 to 1193, at the clock that its power leaves); the matrix unit is busy 49 % of the
// cycles, the vector unit 56 %, LDS 37 %, and waves wait 29 %.  Head dimension 256, whose accumulators leave no
// registers for the pipeline (11 or 16 spill, outside of the products): 3 sequences of 300 to 2048 new
// tokens of up to 16384 764 to 811 us, 1032 to 1096 TFLOP/s, the matrix unit 51 % busy, waves waiting 39 %.  What a
// tile's loads return is looked at only when the tile is decoded: the check of a page id and the halves of a row
// of scales, put together right after their loads, made every wave wait for these (826 us where it takes 764, 894 / 811
// on another card).  Drafted trees spill 28 or 32 registers at head dimension 256, and 39 to 67 scalar ones at
// every head dimension (causal items 0 to 11): 8 trees of 64 to 128 nodes over up to 16384 tokens 206 to 208 us, 769
// TFLOP/s, the matrix unit 42 % busy.  64 columns a wave at one wave per SIMD (512 registers)
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
// of trees with D = 256, then the last of each lane's query operands: the masks' code leaves no registers
// for it, and read back from scratch memory it waited for the loads of the next tile (8 trees of 64 to 128
// nodes over up to 16384 tokens 243 / 229 us)
template <int D>
constexpr int kLdsQ = D == 256 ? 1 : 0;
template <int D>
constexpr int kQueries = kFactors<D> + 4 * kPrefillCols;
// after those, of a tree's tile: the first token that any column attends to, and the bits of the
// tree's tokens that any column attends to
template <int D>
constexpr int kTreeFirst = kQueries<D> + kLdsQ<D> * 16 * 64 * kPrefillWaves;
template <int D>
constexpr int kTreeAny = kTreeFirst<D> + 16;
// and its rows' windows' first tokens and, where they are not too many, their words
template <int D>
constexpr int kTreeFloor = kTreeAny<D> + 8 * kMaxTreeWords;
template <int D>
constexpr int kTreeBits = kTreeFloor<D> + 4 * kPrefillCols;
template <int D>
constexpr int kTreeStaged = D == 256 ? 1024 : 2048;
template <int D, bool TREE>
constexpr int kLdsBytes = TREE ? kTreeBits<D> + 8 * kTreeStaged<D> : kQueries<D>;

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
template <int D, int COLS, bool TREE>
__device__ __forceinline__ TileSpan tile_span(const KvAttnArgs& a, const SeqInfo& seq, int32_t tile, int group) {
  const int32_t cols = seq.m * group, first = tile * COLS;
  const Span s = span_of<TREE>(seq, first, first + COLS < cols ? first + COLS : cols, a.by_group, a.window);
  TileSpan t;
  t.lo = s.lo;
  t.begin = s.lo & ~15;
  t.steps = seq.n > 0 ? (s.hi - t.begin + kTok<D> - 1) / kTok<D> : 0;
  return t;
}
template <int COLS>
__device__ __forceinline__ int32_t tiles_of(const SeqInfo& seq, int group) {
  return (seq.m * group + COLS - 1) / COLS;
}
template <int COLS>
__device__ __forceinline__ int32_t planned_tiles(const KvAttnArgs& a, const SeqInfo& seq, int group) {
  const int32_t t = tiles_of<COLS>(seq, group);
  return t < a.col_tiles ? t : a.col_tiles;
}

// SPLIT: workgroups have pieces of items instead of items (a template parameter: its
// registers cost the other form 2 to 5 %)
// TG: groups of waves that have the same 256 / TG query columns and share the blocks of every tile, for
// items of 128 columns (TG 2), whose results are joined in LDS.
template <int D, bool SPLIT, bool TREE, int TG>
__global__ __launch_bounds__(64 * kPrefillWaves, 2) void k_kv_prefill(KvAttnArgs a) {
  constexpr bool PIPE = D <= 128;
  static_assert(TG == 1 || (TG == 2 && PIPE), "a group has two blocks of a tile");
  constexpr int COLS = kPrefillCols / TG, CW = kPrefillWaves / TG;
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
    const int32_t tiles = tiles_of<COLS>(seq, group);
    tile0 = (tiles < a.col_tiles ? tiles : a.col_tiles) - 1 - turn;
    if (tile0 < 0) return;
  } else {
    // Few items: each is cut into equal pieces of at most S steps (tokens of a tile), S all
    // steps of the call by n_workers, as in kvattn.hip; a lane counts every 64th tile.
    const SeqTable seqs(a, lane);
    float total = 0.0f;
    if constexpr (TREE) {
      // every tile of a sequence has the same keys: a lane counts a sequence
      total = (float)planned_tiles<COLS>(a, seqs.mine, group) * (float)tile_span<D, COLS, TREE>(a, seqs.mine, 0, group).steps;
    } else
    for (b = 0; b < a.batch; ++b) {
      seq = seqs.at(a, b);
      const int32_t tiles = planned_tiles<COLS>(a, seq, group);
      for (int32_t t = lane; t < tiles; t += 64) total += (float)tile_span<D, COLS, TREE>(a, seq, t, group).steps;
    }
#pragma unroll
    for (int off = 1; off < 64; off <<= 1) total += __shfl_xor(total, off);
    int32_t S = (int32_t)(total * (float)hkv * 1.0001f / (float)a.n_workers) + 1;
    S = S < a.min_steps ? a.min_steps : S;
    auto pieces_of = [&](int32_t steps) {
      return steps <= S ? 1 : (int32_t)((uint32_t)(steps + S - 1) / (uint32_t)S);
    };
    int32_t rest = (int32_t)blockIdx.x, tiles = 0, of_head = 0, pieces = 1;
    if constexpr (TREE) {
      const int32_t each = pieces_of(tile_span<D, COLS, TREE>(a, seqs.mine, 0, group).steps);
      const int32_t own = planned_tiles<COLS>(a, seqs.mine, group) * each;
      int32_t upto = own * hkv;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int32_t x = __shfl_up(upto, off);
        if (lane >= off) upto += x;
      }
      const uint64_t past = __builtin_amdgcn_ballot_w64(upto > rest);
      b = past ? __builtin_ctzll(past) : a.batch;
      if (past) {
        seq = seqs.at(a, b);
        of_head = __builtin_amdgcn_readlane(own, b);
        pieces = __builtin_amdgcn_readlane(each, b);
        rest -= __builtin_amdgcn_readlane(upto, b) - of_head * hkv;
      }
    } else
    for (b = 0; b < a.batch; ++b) {
      seq = seqs.at(a, b);
      tiles = planned_tiles<COLS>(a, seq, group);
      of_head = 0;
      for (int32_t t = lane; t < tiles; t += 64) of_head += pieces_of(tile_span<D, COLS, TREE>(a, seq, t, group).steps);
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
    if constexpr (TREE) {
      tile0 = (int32_t)((uint32_t)rest / (uint32_t)pieces);
      rest -= tile0 * pieces;
    } else
    for (int32_t t0 = 0;; t0 += 64) {
      const int32_t own = t0 + lane < tiles ? pieces_of(tile_span<D, COLS, TREE>(a, seq, t0 + lane, group).steps) : 0;
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
    const int32_t steps = tile_span<D, COLS, TREE>(a, seq, tile0, group).steps;
    if (pieces > 1) {
      const int32_t q = (int32_t)((uint32_t)steps / (uint32_t)pieces), more = steps - q * pieces;
      s_first = rest * q + (rest < more ? rest : more);
      s_last = s_first + q + (rest < more);
    }
    if (threadIdx.x == 0) {
      const int32_t fc = tile0 * COLS, left = seq.m * group - fc;
      ItemPieces* const p = static_cast<ItemPieces*>(a.pieces) + blockIdx.x;
      p->cols = pieces > 1 && rest == 0 ? (left < COLS ? left : COLS) : 0;
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
  for (int32_t tile = tile0; (int64_t)tile * COLS < cols; tile += a.col_tiles) {
    const bool whole = !SPLIT || s_last < 0 || tile != tile0;
    if (SPLIT && tile != tile0 && s_first > 0) break;
    const int32_t col_first = tile * COLS;
    const int32_t col_end = col_first + COLS < cols ? col_first + COLS : cols;
    const TileSpan span = tile_span<D, COLS, TREE>(a, seq, tile, group);
    const int32_t begin = whole ? span.begin : span.begin + s_first * TOK;
    const int32_t steps = whole ? span.steps : s_last - s_first;

    // this wave's columns (past the tile's end: its last one again, never written)
    const int cw = wave % CW, tg = wave / CW;
    const int32_t col0 = col_first + 32 * cw;
    const int32_t w0 = col0 < col_end ? col0 : col_end - 1;
    const int32_t w1 = col0 + 32 < col_end ? col0 + 32 : col_end;
    const Span sp = span_of<TREE>(seq, w0, w1, a.by_group, a.window);

    // an address that the compiler does not take out of the loop: with every chunk's address
    // in a register of its own the kernel spills
    auto fresh = [](uint32_t x) {
      asm volatile("" : "+v"(x));
      return x;
    };

    // loads of tile s: this wave's granule, its page id known one tile ahead (as the table has it: looked
    // at only when it is used, it is not waited for here, and with it the loads before it)
    auto page_of = [&](int32_t s) -> int32_t {
      int32_t pg = (begin + s * TOK + 16 * gran) >> a.geom.page_shift;
      pg = pg < last_page ? pg : last_page;
      return a.table[(int64_t)b * a.ld_table + pg];
    };
    auto granule = [&](int32_t s, int32_t id) {
      id = __builtin_amdgcn_readfirstlane(id);
      id = id < 0 ? 0 : (id >= a.geom.n_pages ? (int32_t)a.geom.n_pages - 1 : id);
      int32_t gr = (begin + s * TOK) / 16 + gran;
      gr = gr < last_granule ? gr : last_granule;
      return a.cache + (int64_t)id * a.geom.page_bytes +
             (int64_t)(kh * per_head + (gr & (per_head - 1))) * kv_granule_bytes(D);
    };
    // the quad of tokens and part of a granule's values that this lane decodes
    const int quad = lane >> 4, part = lane & 15;
    // (D = 256: a wave holds either)
    uint32_t rk[KD] = {}, rv_[D == 256 ? 1 : KD] = {}, ksc = 0, ksc_far = 0, vsc_ = 0;
    uint32_t* const rv = D == 256 ? rk : rv_;
    uint32_t& vsc = D == 256 ? ksc : vsc_;
    auto load_k = [&](int32_t s, int32_t id) {
      const uint8_t* p = granule(s, id);
      if constexpr (D == 256) {          // a quarter of either half of a token's row
        const uint32_t i = fresh(lane);
        const uint8_t *c = p + ((i >> 2) * 128 + (i & 3) * 16), *f = p + 8 * D + ((i >> 2) * 16 + (i & 3) * 2);
        read_dwords<4>(c, rk);
        read_dwords<4>(c + 64, rk + 4);
        ksc = *reinterpret_cast<const uint16_t*>(f);
        ksc_far = *reinterpret_cast<const uint16_t*>(f + 8);   // (put together here, they were waited for)
      } else {                           // a quarter of a token's row
        read_dwords<KD>(p + lane * (D / 8), rk);
        ksc = D == 64 ? p[8 * D + lane] : *reinterpret_cast<const uint16_t*>(p + 8 * D + 2 * lane);
      }
    };
    auto load_v = [&](int32_t s, int32_t id) {
      const uint8_t* p = granule(s, id);
      const uint32_t i = D == 256 ? fresh(lane) : lane;
      read_dwords<KD>(p + 9 * D + i * (D / 8), rv);
      vsc = *reinterpret_cast<const uint32_t*>(p + 17 * D + ((i >> 4) * (D / 16) + (i & 15) * D / 256) * 4);
      const int32_t first = begin + s * TOK + 16 * gran;
      if (!TREE && (first < span.lo || first + 16 > seq.n)) vsc = live_scales(vsc, first + 4 * quad, span.lo, seq.n);
    };
    // (TREE: when they are decoded, so that the load is not waited for)
    auto mask_v = [&](int32_t s) {
      if constexpr (TREE) {
        const int32_t first = begin + s * TOK + 16 * gran;
        const int32_t c0 = seq.n - seq.m, from = lds_at<int32_t>(lds + kTreeFirst<D>);
        if (first < from || first + 16 > c0) {
          uint32_t any = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int32_t t = first + 4 * quad + e, j = t - c0;
            const bool node = j >= 0 && j < seq.m && j < 64 * a.tree_words;
            const bool sees = node ? (lds_at<uint32_t>(lds + kTreeAny<D> + 4 * (j >> 5)) >> (j & 31)) & 1 : j < 0 && t >= from;
            any |= (uint32_t)sees << e;
          }
          vsc &= bytes_of_bits(any);
        }
      }
    };
    // decode dword i of the loaded keys: a 16-byte chunk of a token's row
    auto decode_k = [&](uint32_t kb, int i) {               // kb: the lane's first chunk in the tile
      const f16x2 sc = bcast(scale_pair_f16(D == 256 && i >= 4 ? ksc_far : ksc), D == 64 ? 0 : (i >> 1) & 1);
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

    // TREE: the rows' words and windows, and what of the tree any of them attends to
    const int32_t row_first = col_first / a.by_group, words = TREE ? tree_words(a, seq) : 0;
    const int32_t rows = (col_end - 1) / a.by_group - row_first + 1;
    const bool staged = TREE && rows * words <= kTreeStaged<D>;
    auto bits_of = [&](int32_t row, int32_t w) -> uint64_t {
      if (staged) return w >= 0 && w < words ? lds_at<uint64_t>(lds + kTreeBits<D> + 8 * (row * words + w)) : 0;
      return tree_word(a, seq, seq.q0 + row_first + row, w);
    };
    auto stage_tree = [&] {
      if constexpr (!TREE) return;
      if (threadIdx.x < 2 * kMaxTreeWords) lds_at<uint32_t>(lds + kTreeAny<D> + 4 * threadIdx.x) = 0;
      if (threadIdx.x == 0) lds_at<int32_t>(lds + kTreeFirst<D>) = INT32_MAX;
      if (staged)
        for (int32_t i = threadIdx.x; i < rows * words; i += 64 * kPrefillWaves) {
          const int32_t row = words == 1 ? i : (int32_t)((uint32_t)i / (uint32_t)words);
          lds_at<uint64_t>(lds + kTreeBits<D> + 8 * i) = tree_word(a, seq, seq.q0 + row_first + row, i - row * words);
        }
      lds_sync();                                  // (loads of keys and queries stay on their way)
      for (int32_t i = threadIdx.x; i < rows; i += 64 * kPrefillWaves) {
        const int32_t from = a.window ? tree_floor(a, seq, [&](int32_t w) { return bits_of(i, w); }) : 0;
        lds_at<int32_t>(lds + kTreeFloor<D> + 4 * i) = from;
        atomicMin((int32_t*)(shared + kTreeFirst<D>), from);
        for (int32_t w = 0; w < words; ++w) {
          uint64_t x = bits_of(i, w);
          const int32_t skip = from - (seq.n - seq.m) - 64 * w;
          if (skip > 0) x &= skip >= 64 ? 0 : ~0ull << skip;
          if ((uint32_t)x) atomicOr((uint32_t*)(shared + kTreeAny<D>) + 2 * w, (uint32_t)x);
          if ((uint32_t)(x >> 32)) atomicOr((uint32_t*)(shared + kTreeAny<D>) + 2 * w + 1, (uint32_t)(x >> 32));
        }
      }
      lds_sync();
    };
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
      stage_tree();
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
    const int32_t limit = pos + 1;
    const int32_t floor_ = TREE ? lds_at<int32_t>(lds + kTreeFloor<D> + 4 * (qi - row_first)) : (a.window ? pos - a.window + 1 : 0);
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
    auto query = [&](int i) { return lds + kQueries<D> + 16 * (threadIdx.x + 64 * kPrefillWaves * (KS - 1 - i)); };
    constexpr int QL = TREE ? kLdsQ<D> : 0;
    if constexpr (QL > 0) {
#pragma unroll
      for (int i = KS - QL; i < KS; ++i) lds_at<f16x8>(query(i)) = qf[i];   // each lane reads what it wrote
    }
    auto score_piece = [&](f32x16& sc, int i) {
      sc = mfma32(kf[i % (PF + 1)], i < KS - QL ? qf[i] : lds_at<f16x8>(query(i)), sc);
    };
    auto output_piece = [&](const f16x8 p[2], int i) { acc[i % NB] = mfma32(vf[i % (PF + 1)], p[i / NB], acc[i % NB]); };
    // moves the reference M for the block from token t0 on; returns what the earlier sums are
    // scaled by
    auto reference = [&](int32_t t0, f32x16& sc) {
      if (t0 < all_lo || t0 + 32 > sp.all_hi) {
        if constexpr (TREE) {
          const uint32_t sees = (uint32_t)tree_sees(seq, floor_, t0, [&](int32_t w) { return bits_of(qi - row_first, w); }) >> (4 * h);
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (!((sees >> (8 * (e / 4) + e % 4)) & 1)) sc[e] = -__builtin_inff();
        } else {
          const int32_t upto = limit - t0 - 4 * h, from = floor_ - t0 - 4 * h;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int32_t t = 8 * (e / 4) + e % 4;
            if (t >= upto || t < from) sc[e] = -__builtin_inff();
          }
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

    if (steps > 0) {
      if (D != 256 || wave < 4) {
#pragma unroll
        for (int i = 0; i < KD; ++i) decode_k(k_tile(0) + kwbase, i);
      }
      if (D != 256 || wave >= 4) {
        mask_v(0);
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
          read_k(k_tile(0) + kbase, TG == 1 ? 0 : 2 * tg, i);
          score_piece(sa, i);
        }
        if constexpr (TG == 1) {
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
            mask_v(s + 1);
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
          // Blocks 2 tg and 2 tg + 1 of a tile.  The next keys are written before the barrier and due after it,
          // into the place of the tile before this one, whose keys were read before the last barrier; the
          // next values after the barrier and due after the next one, over those that were read before it.
          const int b0 = 2 * tg, b1 = b0 + 1;
          for (int32_t s = 0; s < steps; ++s) {
            const int32_t t0 = begin + s * TOK + 32 * b0;
            const uint32_t kw = fresh(k_tile(s + 1) + kwbase);
            stage(k_tile(s), b1, v_tile(s + 1), b1, t0, sb, sa, pa, pb, [&](int i) {
              if (i < KD) decode_k(kw, i);
            });
            if (s + 2 < steps) load_k(s + 2, id_next);
            __syncthreads();
            mask_v(s + 1);
            const uint32_t vw = fresh(v_tile(s + 1) + vwbase);
            stage(k_tile(s + 1), b0, v_tile(s), b0, t0 + 32, sa, sb, pb, pa, [&](int i) {
              if (i < KS / 2) decode_v(vw, i);
            });
            if (s + 2 < steps) {
              load_v(s + 2, id_next);
              id_next = page_of(s + 3);
            }
          }
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            read_v(v_tile(steps - 1) + vbase, b1, i);
            output_piece(pb, i);
          }
        }
      } else {
        for (int32_t s = 0; s < steps; ++s) {
          const uint32_t kw = fresh(k_tile(s + 1) + kwbase), vw = fresh(v_tile(s + 1) + vwbase);
          if (wave < 4) {
#pragma unroll
            for (int i = 0; i < KD; ++i) decode_k(kw, i);
          } else {
            mask_v(s + 1);
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

    l = sum_xor32(l);
    if constexpr (TG == 2) {
      // the second group's results to the first one's: a lane's registers to the lane that has the same
      // column and elements
      const uint32_t slot = lds + (uint32_t)(cw * (16 * NB + 2)) * 256 + 4 * lane;
      __syncthreads();                             // the tiles are read
      if (tg == 1) {
        lds_at<float>(slot) = m;
        lds_at<float>(slot + 256) = l;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) lds_at<float>(slot + 256 * (2 + 16 * i + e)) = acc[i][e];
      }
      __syncthreads();
      if (tg == 0) {
        const float m1 = lds_at<float>(slot), top = __builtin_fmaxf(m, m1);
        const float f = __builtin_amdgcn_exp2f(m - top), f1 = __builtin_amdgcn_exp2f(m1 - top);
        l = l * f + lds_at<float>(slot + 256) * f1;
        m = top;
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) acc[i][e] = acc[i][e] * f + lds_at<float>(slot + 256 * (2 + 16 * i + e)) * f1;
      }
    }
    // elements g and g + 8 of the blocks: consecutive dimensions, those of a part of the granule
    if (tg == 0 && col0 + c32 < col_end) {
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

template <int D, bool SPLIT, bool TREE, int TG>
hipError_t launch(const KvAttnArgs& a, hipStream_t s) {
  constexpr int bytes = kLdsBytes<D, TREE>;
  const hipError_t e = lds_limit_once<k_kv_prefill<D, SPLIT, TREE, TG>>(bytes);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_kv_prefill<D, SPLIT, TREE, TG>), dim3((unsigned)a.blocks), dim3(64 * kPrefillWaves), bytes, s, a);
  const hipError_t launched = hipGetLastError();
  return SPLIT && launched == hipSuccess ? launch_kv_join(a, InType::BF16, D, s) : launched;
}

template <int D, bool TREE, int TG>
hipError_t launch(const KvAttnArgs& a, hipStream_t s) {
  return a.n_workers ? launch<D, true, TREE, TG>(a, s) : launch<D, false, TREE, TG>(a, s);
}

template <int D>
hipError_t launch(const KvAttnArgs& a, hipStream_t s) {
  if (!a.tree) return launch<D, false, 1>(a, s);
  if (a.tile_cols == kPrefillCols) return launch<D, true, 1>(a, s);
  if constexpr (D == 256) return launch<D, true, 1>(a, s);
  else return launch<D, true, 2>(a, s);
}

}  // namespace

int32_t kv_prefill_cols() { return kPrefillCols; }
// kvattn.hip / here, us: 8 x 4096, 32 / 8 heads, 16 nodes (64 columns) 40 / 42, 32 nodes 56 / 50; 32 x 2048, 16 nodes 42 / 41,
// 32 nodes 83 / 53, 60 nodes 128 / 86; head dimension 64, 32 nodes 43 / 41; 256 (16 / 2 heads, 8 x 8192), 16 nodes 66 / 67, 30
// nodes 97 / 95.
int32_t kv_tree_cols(int32_t D) { return D == 256 ? kPrefillCols / 2 + 1 : kPrefillCols / 4 + 1; }
int32_t kv_prefill_threads() { return 64 * kPrefillWaves; }

hipError_t launch_kv_prefill(const KvAttnArgs& a, int32_t D, hipStream_t s) {
  if (D == 64) return launch<64>(a, s);
  if (D == 128) return launch<128>(a, s);
  return launch<256>(a, s);
}

}  // namespace nvfp4
