// The attention weight that cached tokens receive, summed over query tokens and the heads of a
// group, from the queries' log-sums:
//   W_t <- decay W_t [t < n - m] + sum_{i, h} e^{scale <q_ih, k_t> - lse_ih}  over the i that attend to t
//
// Both kernels take query columns (query token x head) as the rows of a matrix product and tokens as
// its columns, so that a lane has scores of one token and sums its weights in place; a token's
// sum is in one wave's registers, or eight waves' that are joined in a fixed order: a call of
// the same sizes and bounds gives the same bits every time.  Exponents, weights and sums are fp32.
#include <type_traits>

#include "kv_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kWeightWaves = 4;
constexpr int kWaveTokens = 64;

__device__ __forceinline__ f32x4 mfma16(f16x8 a, f16x8 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

// Chunk i (8 elements) of key r of a granule, for lane (g, r): elements 32 g + 8 m + j (D = 128),
// 128 c + 32 g + 8 m + j (D = 256), 16 g + 8 m + j (D = 64)
template <int D>
struct Keys {
  uint32_t k[D / 32];
  uint16_t ks[D == 256 ? 2 : 1];         // (widened where it is loaded, it was waited for)
};

template <int D>
__device__ __forceinline__ void load_keys(__amdgpu_buffer_rsrc_t p, uint32_t lane, Keys<D>& x) {
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
}

template <int D>
__device__ __forceinline__ f16x8 key_frag(const Keys<D>& x, int i) {
  if constexpr (D == 64) return decode8_f16(x.k[i], bcast(scale_pair_f16(x.ks[0]), 0));
  else return decode8_f16(x.k[i], bcast(scale_pair_f16(x.ks[i / 4]), (i >> 1) & 1));
}

// Query tokens [first, end) of a sequence that attend to any of the tokens [t0, t0 + count)
struct QueryRange {
  int32_t first, end;
};
__device__ __forceinline__ QueryRange queries_of(const SeqInfo& s, int32_t t0, int32_t count, int window) {
  const int32_t c0 = s.n - s.m;
  QueryRange r;
  r.first = t0 > c0 ? t0 - c0 : 0;
  r.end = s.m;
  if (window) {
    const int64_t end = (int64_t)t0 + count - 1 - c0 + window;   // p - window < t
    r.end = end < s.m ? (end > 0 ? (int32_t)end : 0) : s.m;
  }
  return r;
}

// Few query columns: one token a sequence, or a path of a few.  Bound by the keys' bytes, so a wave goes through
// a run of tokens, 64 at a time, with the next 64 tokens' codes in flight; S on the f16 MFMA
// 16x16x32 with the numerics of kvattn.hip, up to NB blocks of 16 query columns, which stay in registers (more of
// them, which the bounds did not announce, are prepared again for every step).  32 sequences of up to 8192 tokens, 32 / 8
// heads of 128: 27 us, 3.6 TB/s (unlike lengths: the longest runs last); of 32768 124 to 128 us, 5.2 TB/s, as fast
// as a copy.
template <int D, bool F32, int NB>
__global__ __launch_bounds__(64 * kWeightWaves, D == 256 || NB == 4 ? 2 : (NB == 2 ? 3 : 4)) void k_kv_weights(KvWeightsArgs w) {
  constexpr int KC = D / 32, TERMS = F32 ? 2 : 1, NG = kWaveTokens / 16;
  const KvAttnArgs& a = w.a;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g = lane >> 4, r = lane & 15;
  const int hkv = a.geom.n_kv_heads, group = (int)a.by_group.d;
  const int per_head = 1 << (a.geom.page_shift - 4);
  const int item = (int)blockIdx.x / w.by_tiles;
  const int b = item / a.by_heads, kh = item - b * hkv;
  const SeqInfo seq = seq_info(a, b);
  if (seq.m == 0) return;
  const int32_t c0 = seq.n - seq.m, cols = seq.m * group;
  const float kg = a.k_gscale[kh];
  const int32_t run = w.steps * kWaveTokens;

  // the blocks of columns in registers: A operand, row r; results' rows 4 g + i
  f16x8 qf[NB][TERMS][KC];
  float csc[NB][4], sub[NB][4];
  int32_t pos[NB][4];
  auto prepare = [&](int32_t col0, int nb) {
    int32_t col = col0 + r;
    const bool past = col >= cols;
    col = past ? cols - 1 : col;
    const int32_t qi = col / a.by_group, head = kh * group + (col - qi * group);
    const int64_t off = (seq.q0 + qi) * a.ldq + (int64_t)head * D;
    const float lse = w.lse[(seq.q0 + qi) * a.n_q_heads + head];
    float v[KC][8];
    float amax = 0.0f;
#pragma unroll
    for (int c = 0; c < KC; ++c) load8<F32>(a.q, off + (D == 64 ? 16 * g + 8 * c : 128 * (c / 4) + 32 * g + 8 * (c % 4)), v[c]);
    // A row that attends to nothing, is taken out or is not there has no weights: e^(0 - inf).  Its query may hold anything,
    // and a NaN or an infinity would stay a NaN.
    const bool none = past || lse == -__builtin_inff();
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[c][e] = none ? 0.0f : v[c][e];
        amax = __builtin_fmaxf(amax, __builtin_fabsf(v[c][e]));
      }
    amax = max_xor32(max_xor16(amax));
    const float up = a.scale < 0.0f ? -query_up(amax) : query_up(amax);
    const float csc_r = score_factor(a.scale, kg, amax);
    const float sub_r = none ? __builtin_inff() : lse * kLog2e;
#pragma unroll
    for (int c = 0; c < KC; ++c)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = v[c][e] * up;
        const _Float16 hi = (_Float16)x;
        qf[nb][0][c][e] = hi;
        if constexpr (F32) qf[nb][TERMS - 1][c][e] = (_Float16)(x - (float)hi);
      }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      csc[nb][i] = __shfl(csc_r, 4 * g + i);
      sub[nb][i] = __shfl(sub_r, 4 * g + i);
      pos[nb][i] = c0 + __shfl(qi, 4 * g + i);
    }
  };

  // runs past the planned ones go with the first ones' waves
  for (int64_t at = (int64_t)((int)blockIdx.x - item * w.tiles) * kWeightWaves + wave; at * run < seq.n;
       at += (int64_t)w.tiles * kWeightWaves) {
    const int32_t begin = (int32_t)(at * run), end = begin + run < seq.n ? begin + run : seq.n;
    const int32_t last_granule = (end - 1) >> 4;
    // page of token begin + 16 lane (a run is at most 1024 tokens)
    int32_t t_page = begin + 16 * lane;
    t_page = t_page < seq.n ? t_page : seq.n - 1;
    const int32_t id = a.table[(int64_t)b * a.ld_table + (t_page >> a.geom.page_shift)];
    const int32_t pages = id < 0 ? 0 : (id >= a.geom.n_pages ? (int32_t)a.geom.n_pages - 1 : id);
    // the lane's own token of a step, 16 g + r, and its weight
    float* own = nullptr;
    float old = 0.0f;
    auto issue_old = [&](int32_t t0) {
      const int32_t t = t0 + lane, i = ((t0 - begin) >> 4) + g;
      const int32_t page = __shfl(id, i < 63 ? i : 63);
      const bool there = t < end && page >= 0 && page < a.geom.n_pages;
      const uint32_t slot = (uint32_t)t & ((1u << a.geom.page_shift) - 1);
      own = w.weights + (there ? (((int64_t)page * hkv + kh) << a.geom.page_shift) + slot : 0);
      old = *own;
      own = there ? own : nullptr;
    };
    auto put = [&](int32_t t0, float total) {
      if (own) *own = t0 + lane < c0 && w.decay != 0.0f ? __builtin_fmaf(w.decay, old, total) : total;
    };
    // where no query attends to anything of the run, no key is read, but weights fade
    const QueryRange all = queries_of(seq, begin, end - begin, a.window);
    if (all.first >= all.end) {
      if (w.decay != 1.0f)
        for (int32_t t0 = begin; t0 < end; t0 += kWaveTokens) {
          issue_old(t0);
          put(t0, 0.0f);
        }
      continue;
    }
    Keys<D> key[NG];
    auto issue = [&](int32_t t0, int u) {
      int32_t gr = (t0 >> 4) + u;
      gr = gr < last_granule ? gr : last_granule;         // past the end: the last granule again
      const int32_t page = __builtin_amdgcn_readlane(pages, gr - (begin >> 4));
      load_keys<D>(granule_buffer<D>(a, page, kh * per_head + (gr & (per_head - 1))), lane, key[u]);
    };
    auto go = [&](auto once) {
      for (int32_t t0 = begin; t0 < end; t0 += kWaveTokens) {
        const QueryRange q = queries_of(seq, t0, kWaveTokens, a.window);
        // every query token attends to every token of the step
        const bool full = t0 + kWaveTokens - 1 <= c0 && (!a.window || t0 > seq.n - 1 - a.window);
        float total = 0.0f;
#pragma unroll
        for (int u = 0; u < NG; ++u) {
          f16x8 kf[KC];
          if (!decltype(once)::value) issue(t0, u);
#pragma unroll
          for (int c = 0; c < KC; ++c) kf[c] = key_frag<D>(key[u], c);
          // decoded here, so that the next step's keys come into the registers that these leave: with a copy of
          // them at the step's end, that waits for them
#pragma unroll
          for (int c = 0; c < KC; ++c) asm volatile("" : "+v"(kf[c]));
          __builtin_amdgcn_sched_barrier(0);
          if (decltype(once)::value) issue(t0 + kWaveTokens, u);
          const int32_t t = t0 + 16 * u + r;
          float sum = 0.0f;
          auto add = [&](int nb) {
            f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
            for (int c = 0; c < KC; ++c)
#pragma unroll
              for (int e = 0; e < TERMS; ++e) s = mfma16(qf[nb][e][c], kf[c], s);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float x = __builtin_fmaf(s[i], csc[nb][i], -sub[nb][i]);
              if (!full) x = t <= pos[nb][i] && (!a.window || t > pos[nb][i] - a.window) ? x : -__builtin_inff();
              sum += __builtin_amdgcn_exp2f(x);
            }
          };
          if constexpr (decltype(once)::value) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              if (nb == 0 || 16 * nb < cols) add(nb);
          } else {
            for (int32_t col0 = q.first * group; col0 < q.end * group; col0 += 16) {
              prepare(col0, 0);
              add(0);
            }
          }
          sum = sum_xor32(sum_xor16(sum));
          if (g == u) total = sum;
        }
        if (q.first < q.end || w.decay != 1.0f) put(t0, total);
        issue_old(t0 + kWaveTokens);
      }
    };
    if (cols <= 16 * NB) {
#pragma unroll
      for (int u = 0; u < NG; ++u) issue(begin, u);
      issue_old(begin);
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) prepare(16 * nb, nb);
      go(std::true_type{});
    } else {
      issue_old(begin);
      go(std::false_type{});
    }
  }
}

// Many query columns: the matrix product and the exponentials bound it.  A wave keeps TB blocks of 32
// tokens decoded in registers, as B operands of the bf16 MFMA 32x32x16 (e2m1 * s has 6 significant
// bits, and bf16 queries go in as they are), and takes tiles of 32 query columns past them; the
// waves of a workgroup have different tokens, or every qs-th tile of the same ones, whose sums
// are joined in LDS at the end.  Tiles go from memory to LDS by asynchronous loads, each wave's its own,
// one ahead: no barrier in the loop.  fp32 queries go as three bf16 terms, which hold all their bits.
//
// 8192 tokens, 32 / 8 heads of 128: 274 to 291 us by card, 945 to 1002 TFLOP/s (a large bf16 matrix product reaches
// 1188); 256, 3 sequences of 300 to 2048 new tokens of up to 16384 478 to 494 us, 847 to 875; fp32, 4096 tokens 220 to
// 228 us, 302 to 312, a third of the products' terms.
//
// A tile is whole query tokens, as many as 32 rows hold (heads 32 s .. of one token where the
// group has more), so that its rows' places are the same in every tile.
constexpr int kManyWaves = 8;
constexpr int kTileRows = 32;
constexpr int kRingBytes = 8192;                   // of each of the two places of a wave's ring

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

template <int D, bool F32>
struct Many {
  static constexpr int SIZE = F32 ? 4 : 2;
  static constexpr int TB = D == 256 || (F32 && D == 128) ? 2 : 4;
  static constexpr int KS = D / 16;                          // K steps: elements (D / 2) h + 8 k + j
  static constexpr int CHUNK = F32 ? 64 : (D < 128 ? D : 128);   // elements of a row that are loaded at once
  static constexpr int NCH = D / CHUNK;
  static constexpr int KSC = CHUNK / 16;
  static constexpr int UNITS = CHUNK * SIZE / 16;            // 16-byte units of a row
  static constexpr int LOADS = kTileRows * UNITS / 64;
  // a unit's place in its row: 16 lanes that read a unit of 16 rows meet every bank once
  static __device__ __forceinline__ int swizzle(int row) { return UNITS == 16 ? row & 15 : (row >> 1) & 7; }
};

__device__ __forceinline__ f32x16 mfma32(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

__device__ __forceinline__ uint32_t high_halves(float lo, float hi) {
  return __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
}

// 8 codes under their block's scale: exact in bf16
__device__ __forceinline__ bf16x8 decode8_bf16(uint32_t codes, float s) {
  u32x4 x;
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 0);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 1);
  const auto c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 2);
  const auto d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, 1.0f, 3);
  x[0] = high_halves(a[0] * s, a[1] * s);
  x[1] = high_halves(b[0] * s, b[1] * s);
  x[2] = high_halves(c[0] * s, c[1] * s);
  x[3] = high_halves(d[0] * s, d[1] * s);
  return __builtin_bit_cast(bf16x8, x);
}

__device__ __forceinline__ void to_lds16(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 16, off, 0, 0, 0);
}
__device__ __forceinline__ void to_lds4(__amdgpu_buffer_rsrc_t r, uint8_t* lds, uint32_t off) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)lds, 4, off, 0, 0, 0);
}

// `bytes` from p on as a buffer (what lies past them reads as 0)
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void* p, int64_t bytes) {
  const int32_t n = bytes < 0 ? 0 : (bytes > 0x7FFFFFFF ? 0x7FFFFFFF : (int32_t)bytes);
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(reinterpret_cast<const void*>(uniform64((int64_t)p))), (short)0,
                                           __builtin_amdgcn_readfirstlane(n), 0x00020000);
}

// SLICED: more heads in a group than a tile has rows
template <int D, bool F32, bool SLICED>
__global__ __launch_bounds__(64 * kManyWaves, 2) void k_kv_weights_many(KvWeightsArgs w) {
  using M = Many<D, F32>;
  constexpr int TB = M::TB, KS = M::KS;
  extern __shared__ __attribute__((aligned(256))) uint8_t shared[];
  const KvAttnArgs& a = w.a;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int h = lane >> 5, r = lane & 31;
  uint8_t* const ring = shared + wave * 2 * kRingBytes;
  float* const s_lse = reinterpret_cast<float*>(shared + kManyWaves * 2 * kRingBytes) + wave * 3 * kTileRows;
  float* const s_sub = s_lse + 2 * kTileRows;
  float* const s_sum = reinterpret_cast<float*>(shared + kManyWaves * (2 * kRingBytes + 3 * kTileRows * 4));
  uint32_t* const s_off = reinterpret_cast<uint32_t*>(s_sum + kManyWaves * 4 * 32);

  const int hkv = a.geom.n_kv_heads, group = (int)a.by_group.d;
  const int per_head = 1 << (a.geom.page_shift - 4);
  // the tiles that the most queries attend to first; workgroups side by side differ in the head
  const int turn = (int)blockIdx.x / a.by_pairs, item = (int)blockIdx.x - turn * (int)a.by_pairs.d;
  const int b = item / a.by_heads, kh = item - b * hkv;
  const SeqInfo seq = seq_info(a, b);
  if (seq.m == 0) return;
  const int32_t c0 = seq.n - seq.m;
  const float csc = (float)((double)a.scale * 1.4426950408889634 * (double)a.k_gscale[kh]);
  const int qs = 1 << w.split, ql = wave & (qs - 1), tg = wave >> w.split;
  const int32_t wg_tokens = (kManyWaves >> w.split) * TB * 32;

  const int32_t per_tile = SLICED ? 1 : kTileRows / group;                      // query tokens of a tile
  const int32_t slices = SLICED ? (group + kTileRows - 1) / kTileRows : 1;      // tiles of a query token
  const int32_t rows = SLICED ? kTileRows : per_tile * group;

  // a lane's bytes of a tile's rows, the same for every wave: load i of the tile
  for (int i = wave; i <= M::LOADS; i += kManyWaves) {
    const int place = i < M::LOADS ? i * (64 / M::UNITS) + lane / M::UNITS : r;
    const int row = place < rows ? place : rows - 1;
    const int unit = (lane % M::UNITS) ^ M::swizzle(place);
    const int tok = SLICED ? 0 : row / a.by_group, hd = row - tok * group;
    s_off[i * 64 + lane] =
        i < M::LOADS ? (uint32_t)(((int64_t)tok * a.ldq + hd * D + (unit / (M::UNITS / 2)) * (D / 2)) * M::SIZE +
                                  (unit % (M::UNITS / 2)) * 16)
                     : (uint32_t)(tok * a.n_q_heads + hd) * 4;                  // the log-sum of row r
  }
  __syncthreads();

  for (int64_t tile = turn; tile * wg_tokens < seq.n; tile += w.tiles) {
    const int32_t t0 = (int32_t)(tile * wg_tokens) + tg * TB * 32;
    const QueryRange q = queries_of(seq, t0, TB * 32, a.window);
    float sum[TB] = {};
    if (t0 < seq.n && q.first < q.end) {
      // keys
      bf16x8 kf[TB][KS];
#pragma unroll
      for (int tb = 0; tb < TB; ++tb) {
        int32_t t = t0 + 32 * tb + r;
        t = t < seq.n ? t : seq.n - 1;
        int32_t id = a.table[(int64_t)b * a.ld_table + (t >> a.geom.page_shift)];
        id = id < 0 ? 0 : (id >= a.geom.n_pages ? (int32_t)a.geom.n_pages - 1 : id);
        const uint8_t* p = a.cache + (int64_t)id * a.geom.page_bytes +
                           (int64_t)(kh * per_head + ((t >> 4) & (per_head - 1))) * kv_granule_bytes(D);
        const uint8_t* codes = p + (t & 15) * (D / 2) + h * (D / 4);
        const uint8_t* scales = p + 8 * D + (t & 15) * (D / 16) + h * (D / 32);
        uint32_t c[KS], sc[D == 256 ? 2 : 1];
#pragma unroll
        for (int i = 0; i < KS; i += 4) {
          const u32x4 x = *reinterpret_cast<const u32x4*>(codes + 4 * i);
#pragma unroll
          for (int e = 0; e < 4; ++e) c[i + e] = x[e];
        }
        if constexpr (D == 64) sc[0] = *reinterpret_cast<const uint16_t*>(scales);
        else if constexpr (D == 128) sc[0] = *reinterpret_cast<const uint32_t*>(scales);
        else {
          sc[0] = *reinterpret_cast<const uint32_t*>(scales);
          sc[1] = *reinterpret_cast<const uint32_t*>(scales + 4);
        }
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          float s;
          const int blk = i / 2;
          if (blk % 4 == 0) s = __builtin_amdgcn_cvt_f32_fp8(sc[blk / 4], 0);
          else if (blk % 4 == 1) s = __builtin_amdgcn_cvt_f32_fp8(sc[blk / 4], 1);
          else if (blk % 4 == 2) s = __builtin_amdgcn_cvt_f32_fp8(sc[blk / 4], 2);
          else s = __builtin_amdgcn_cvt_f32_fp8(sc[blk / 4], 3);
          kf[tb][i] = decode8_bf16(c[i], s);
        }
      }

      // the query tokens' tiles from the last on, every qs-th of them
      const int32_t first = q.first / per_tile, tiles = ((q.end - 1) / per_tile - first + 1) * slices;
      const int64_t q_end = ((int64_t)(a.T - 1) * a.ldq + (int64_t)a.n_q_heads * D) * M::SIZE;
      const int64_t lse_end = a.T * a.n_q_heads * 4;
      auto issue = [&](int32_t x, int chunk, int place) {
        const int32_t j = first + x / slices, slice = x - (x / slices) * slices;
        const int64_t at = ((int64_t)(seq.q0 + j * per_tile) * a.ldq + (int64_t)(kh * group + slice * kTileRows) * D) * M::SIZE +
                           chunk * (M::CHUNK / 2) * M::SIZE;
        const auto buf = buffer_of(static_cast<const uint8_t*>(a.q) + at, q_end - at);
#pragma unroll
        for (int i = 0; i < M::LOADS; ++i) to_lds16(buf, ring + place * kRingBytes + i * 1024, s_off[i * 64 + lane]);
        if (chunk == 0) {
          const int64_t l = ((int64_t)(seq.q0 + j * per_tile) * a.n_q_heads + kh * group + slice * kTileRows) * 4;
          const auto lbuf = buffer_of(reinterpret_cast<const uint8_t*>(w.lse) + l, lse_end - l);
          if (h == 0) to_lds4(lbuf, reinterpret_cast<uint8_t*>(s_lse + (x >> w.split & 1) * kTileRows), s_off[M::LOADS * 64 + r]);
        }
      };
      int32_t x = tiles - 1 - ql;
      int place = 0;
      if (x >= 0) issue(x, 0, 0);
      for (; x >= 0; x -= qs) {
        const int32_t j = first + x / slices, slice = x - (x / slices) * slices;
        // rows from the tile's first query token on that are there
        const int32_t tok0 = j * per_tile, tok1 = tok0 + per_tile < seq.m ? tok0 + per_tile : seq.m;
        int32_t have = SLICED ? group - slice * kTileRows : (tok1 - tok0) * group;
        have = have < kTileRows ? have : kTileRows;
        // every row is there and attends to every token
        const bool full = have >= rows && t0 + TB * 32 - 1 <= c0 + tok0 && (!a.window || t0 > c0 + tok1 - 1 - a.window);
        // scores' rows: 8 (i / 4) + 4 h + i % 4
        float sub[16];
        auto weight = [&](const f32x16& score, float (&part)[4], int i) {
          part[i % 4] += __builtin_amdgcn_exp2f(__builtin_fmaf(score[i], csc, -sub[i]));
        };
        // rows that attend to a lane's token are neighbours: those of the query tokens from its own place on, before
        // the window leaves it behind
        auto add_some = [&](const f32x16& score, int32_t tmin, float& to) {
          int32_t d = tmin + r - c0 - tok0;        // the tile's query tokens before the token
          d = d < kTileRows ? d : kTileRows;
          int32_t gone = a.window ? d + a.window : kTileRows;
          gone = gone < 0 ? 0 : (gone < kTileRows ? gone : kTileRows);
          d = d < 0 ? 0 : d;
          const int32_t lo = SLICED ? (d ? kTileRows : 0) : d * group, upto = SLICED ? (gone ? kTileRows : 0) : gone * group;
          const int32_t hi = upto < have ? upto : have, row0 = 4 * h - lo;
          const uint32_t count = hi > lo ? hi - lo : 0;
#pragma unroll
          for (int i4 = 0; i4 < 4; ++i4) {
            if (8 * i4 >= have) continue;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = __builtin_fmaf(score[4 * i4 + e], csc, -sub[4 * i4 + e]);
              to += __builtin_amdgcn_exp2f((uint32_t)(row0 + 8 * i4 + e) < count ? y : -__builtin_inff());
            }
          }
        };
        auto landed = [&](int32_t next_x, int next_chunk) {
          wait_vmcnt<0>();                         // this chunk (and the log-sums) are there
          asm volatile("" ::: "memory");           // and nothing is read before
          if (next_x >= 0) issue(next_x, next_chunk, place ^ 1);
        };
        // Rows of log-sum -inf have no weights, e^(0 - inf): their queries are taken as 0, since a NaN or an
        // infinity in one would stay a NaN.  none: whether the lane's row is one; any_none: whether any is (rare).
        bool none = false, any_none = false;
        auto log_sums = [&] {
          const float lse = s_lse[(x >> w.split & 1) * kTileRows + r];
          none = lse == -__builtin_inff();
          any_none = __builtin_amdgcn_ballot_w64(none) != 0;
          if (h == 0) s_sub[r] = r >= rows || none ? __builtin_inff() : lse * kLog2e;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const f32x4 y = *reinterpret_cast<const f32x4*>(s_sub + 8 * i + 4 * h);
#pragma unroll
            for (int e = 0; e < 4; ++e) sub[4 * i + e] = y[e];
          }
        };
        auto unit_at = [&](int unit) {
          return ring + place * kRingBytes + r * (M::UNITS * 16) + ((unit ^ M::swizzle(r)) * 16);
        };
        if constexpr (!F32 && M::NCH == 1) {
          // scores of block i + 1 on the matrix unit beside the weights of block i
          landed(x - qs, 0);
          bf16x8 qf[KS];
#pragma unroll
          for (int k = 0; k < KS; ++k) qf[k] = *reinterpret_cast<const bf16x8*>(unit_at(h * (M::UNITS / 2) + k));
          log_sums();
          if (any_none) {
#pragma unroll
            for (int k = 0; k < KS; ++k) qf[k] = none ? bf16x8{} : qf[k];
          }
          f32x16 acc[2];
#pragma unroll
          for (int k = 0; k < KS; ++k) acc[0] = mfma32(qf[k], kf[0][k], k == 0 ? f32x16{} : acc[0]);
          if (full) {
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
              float part[4] = {};
#pragma unroll
              for (int k = 0; k < KS; ++k) {
                __builtin_amdgcn_sched_barrier(0);
                if (tb + 1 < TB) acc[(tb + 1) & 1] = mfma32(qf[k], kf[tb + 1 < TB ? tb + 1 : 0][k], k == 0 ? f32x16{} : acc[(tb + 1) & 1]);
#pragma unroll
                for (int i = 0; i < 16 / KS; ++i) weight(acc[tb & 1], part, k * (16 / KS) + i);
              }
              sum[tb] += (part[0] + part[1]) + (part[2] + part[3]);
            }
            __builtin_amdgcn_sched_barrier(0);
          } else {
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
              if (tb) {
#pragma unroll
                for (int k = 0; k < KS; ++k) acc[0] = mfma32(qf[k], kf[tb][k], k == 0 ? f32x16{} : acc[0]);
              }
              add_some(acc[0], t0 + 32 * tb, sum[tb]);
            }
          }
          place ^= 1;
        } else {
          f32x16 acc[TB];
#pragma unroll
          for (int chunk = 0; chunk < M::NCH; ++chunk) {
            if (chunk + 1 < M::NCH) landed(x, chunk + 1);
            else landed(x - qs, 0);
            if (chunk == 0) log_sums();
            if (any_none) {
              // the row in LDS, half of it a lane, before any lane reads it
              if (none) {
#pragma unroll
                for (int u = 0; u < M::UNITS / 2; ++u)
                  *reinterpret_cast<u32x4*>(unit_at(h * (M::UNITS / 2) + u)) = u32x4{0, 0, 0, 0};
              }
              asm volatile("" ::: "memory");
            }
#pragma unroll
            for (int k = 0; k < M::KSC; ++k) {
              const int step = chunk * M::KSC + k;
              if constexpr (!F32) {
                const bf16x8 qf = *reinterpret_cast<const bf16x8*>(unit_at(h * (M::UNITS / 2) + k));
#pragma unroll
                for (int i = 0; i < TB; ++i) acc[i] = mfma32(qf, kf[i][step], step == 0 ? f32x16{} : acc[i]);
              } else {
                float v[8];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                  const f32x4 y = *reinterpret_cast<const f32x4*>(unit_at(h * (M::UNITS / 2) + 2 * k + e));
#pragma unroll
                  for (int z = 0; z < 4; ++z) v[4 * e + z] = y[z];
                }
                // each term the upper 16 bits of what is left: three hold every bit
                u32x4 term[3];
#pragma unroll
                for (int t = 0; t < 3; ++t)
#pragma unroll
                  for (int e = 0; e < 4; ++e) {
                    term[t][e] = high_halves(v[2 * e], v[2 * e + 1]);
                    v[2 * e] -= __uint_as_float(__float_as_uint(v[2 * e]) & 0xFFFF0000u);
                    v[2 * e + 1] -= __uint_as_float(__float_as_uint(v[2 * e + 1]) & 0xFFFF0000u);
                  }
#pragma unroll
                for (int t = 2; t >= 0; --t)
#pragma unroll
                  for (int i = 0; i < TB; ++i)
                    acc[i] = mfma32(__builtin_bit_cast(bf16x8, term[t]), kf[i][step], step == 0 && t == 2 ? f32x16{} : acc[i]);
              }
            }
            place ^= 1;
          }
          if (full) {
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) {
              float part[4] = {};
#pragma unroll
              for (int i = 0; i < 16; ++i) weight(acc[tb], part, i);
              sum[tb] += (part[0] + part[1]) + (part[2] + part[3]);
            }
          } else {
#pragma unroll
            for (int tb = 0; tb < TB; ++tb) add_some(acc[tb], t0 + 32 * tb, sum[tb]);
          }
        }
      }
    }
    // the waves' sums: lane (0, r) token r of each block
    __syncthreads();                               // s_sum of the tile before is read
#pragma unroll
    for (int tb = 0; tb < TB; ++tb) {
      const float y = sum_xor32(sum[tb]);
      if (h == 0) s_sum[wave * TB * 32 + 32 * tb + r] = y;
    }
    __syncthreads();
    for (int32_t i = threadIdx.x; i < wg_tokens; i += 64 * kManyWaves) {
      const int32_t t = (int32_t)(tile * wg_tokens) + i;
      if (t >= seq.n) break;
      const int32_t of = i / (TB * 32), lane_at = i % (TB * 32);
      const QueryRange mine = queries_of(seq, (int32_t)(tile * wg_tokens) + of * TB * 32, TB * 32, a.window);
      if (mine.first >= mine.end && w.decay == 1.0f) continue;
      const int32_t id = a.table[(int64_t)b * a.ld_table + (t >> a.geom.page_shift)];
      if (id < 0 || id >= a.geom.n_pages) continue;
      float total = 0.0f;
      for (int s = 0; s < qs; ++s) total += s_sum[((of << w.split) + s) * TB * 32 + lane_at];
      float* const out = w.weights + ((((int64_t)id * hkv + kh) << a.geom.page_shift) + (t & ((1 << a.geom.page_shift) - 1)));
      *out = t < c0 && w.decay != 0.0f ? __builtin_fmaf(w.decay, *out, total) : total;
    }
  }
}

constexpr int kManyLds = kManyWaves * (2 * kRingBytes + 3 * kTileRows * 4) + kManyWaves * 4 * 32 * 4 + 9 * 64 * 4;

template <int D, bool F32, bool SLICED>
hipError_t launch_many(const KvWeightsArgs& w, int64_t blocks, hipStream_t s) {
  const hipError_t e = lds_limit_once<k_kv_weights_many<D, F32, SLICED>>(kManyLds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_kv_weights_many<D, F32, SLICED>), dim3((unsigned)blocks), dim3(64 * kManyWaves), kManyLds, s, w);
  return hipGetLastError();
}

// Blocks of 16 columns of the kernel for few, as far as registers hold them.  Many / few, us, 32 / 8 heads of
// 128: 32 columns, 8 x 4096 11.4 / 10.4, 32 x up to 8192 57 / 39, 1 x 300 7.3 / 5.9; 64 columns, 8 x 4096 14.6 / 16.4,
// 32 x up to 8192 70 / 56; 36 (48 / 8 heads, 24 x up to 6001) 39 / 28; fp32, 32 columns 16.9 / 16.1, head dimension
// 64, 64 columns 13.3 / 11.8; 256, 32 columns 8 x 8192 10.4 / 10.9.  The rule looks at the columns alone, and loses
// 0.5 to 2 us where they are many for the head dimension and the tokens not many (8 x 4096 with 64, the last one).
constexpr int few_blocks(int D, bool F32) { return D == 64 || (D == 128 && !F32) ? 4 : (D == 256 && F32 ? 1 : 2); }

template <int D, bool F32>
hipError_t launch(const KvWeightsArgs& w, int64_t blocks, hipStream_t s) {
  if (w.split < 0) {
    const dim3 grid((unsigned)blocks), threads(64 * kWeightWaves);
    constexpr int MOST = few_blocks(D, F32);
    if (w.split == -1) hipLaunchKernelGGL((k_kv_weights<D, F32, 1>), grid, threads, 0, s, w);
    else if (w.split == -2) hipLaunchKernelGGL((k_kv_weights<D, F32, MOST < 2 ? 1 : 2>), grid, threads, 0, s, w);
    else hipLaunchKernelGGL((k_kv_weights<D, F32, MOST>), grid, threads, 0, s, w);
    return hipGetLastError();
  }
  return w.a.by_group.d > kTileRows ? launch_many<D, F32, true>(w, blocks, s) : launch_many<D, F32, false>(w, blocks, s);
}

template <int D, bool F32>
hipError_t plan(KvWeightsArgs w, int64_t max_q_len, int64_t max_kv_len, hipStream_t s) {
  const int64_t pairs = (int64_t)w.a.batch * w.a.geom.n_kv_heads, group = w.a.by_group.d;
  const int64_t m = max_q_len < w.a.T ? max_q_len : w.a.T;
  const int64_t n = max_kv_len < 1 ? 1 : max_kv_len;
  // keys that a sequence's queries attend to, at most
  const int64_t span = w.a.window && w.a.window + m < n ? w.a.window + m : n;
  if (m * group <= 16 * few_blocks(D, F32)) {
    // Runs so long that about all waves are there at once, four a SIMD; two or one, where a wave's columns are more or
    // longer and it takes longer to bring them.  By 4096 / 2048 / 1024 waves, us: head dimension 128, 32 x up to 8192 27 / 29 / 30,
    // fp32 8 x up to 8192 11 / 11 / 13; 64, 32 x up to 8192 13 / 14 / 19; 256, 16 x up to 32768 36 / 32 / 32, fp32 4 x up
    // to 32768 22 / 14 / 13; 128 with 32 columns 8 x 4096 13 / 10 / 11, with 64 24 / 16 / 17, 24 x up to 6001 with 36
    // 31 / 28 / 45.
    const int64_t steps = pairs * ((span + kWaveTokens - 1) / kWaveTokens);
    const int64_t each = steps / (D == 256 ? 1024 : (m * group > 16 ? 2048 : 4096));
    w.split = m * group <= 16 ? -1 : (m * group <= 32 ? -2 : -4);
    w.steps = (int32_t)(each < 1 ? 1 : (each > 16 ? 16 : each));
    const int64_t tokens = (int64_t)w.steps * kWaveTokens * kWeightWaves;
    w.tiles = kv_planned_tiles((n + tokens - 1) / tokens, pairs, 64 * kWeightWaves);
  } else {
    const int64_t tiles = group <= kTileRows ? (m + kTileRows / group - 1) / (kTileRows / group) : m * ((group + kTileRows - 1) / kTileRows);
    // More waves to the same tokens while workgroups are few (two a compute unit) and each wave has two
    // tiles, or where the tiles are many: the keys are decoded by each of them.  While they are fewer than half the
    // compute units, each wave one: without / with, us, 1 x 300, 40 new, 32 / 8 heads of 128 14.9 / 9.3, 1 x 2000, 100 new, 8 / 2
    // heads 14.9 / 10.8, fp32 1 x 100, 40 new, 4 / 2 heads of 256 17.7 / 11.7.
    w.split = 0;
    constexpr int64_t WG = kManyWaves * Many<D, F32>::TB * 32;
    while (w.split < 3 && ((tiles >= (4 << w.split) && (tiles >= 32 || pairs * ((span * 2 + WG - 1) / (WG >> w.split)) < 1024)) ||
                           (tiles > (1 << w.split) && pairs * ((span + (WG >> w.split) - 1) / (WG >> w.split)) < 128)))
      ++w.split;
    const int64_t tokens = (kManyWaves >> w.split) * Many<D, F32>::TB * 32;
    w.tiles = kv_planned_tiles((n + tokens - 1) / tokens, pairs, 64 * kManyWaves);
  }
  w.by_tiles = fast_div((uint32_t)w.tiles);
  return launch<D, F32>(w, pairs * w.tiles, s);
}

}  // namespace

hipError_t launch_kv_weights(KvWeightsArgs w, InType t, int32_t D, int64_t max_q_len, int64_t max_kv_len, hipStream_t s) {
  w.a.by_group = fast_div((uint32_t)(w.a.n_q_heads / w.a.geom.n_kv_heads));
  w.a.by_heads = fast_div((uint32_t)w.a.geom.n_kv_heads);
  w.a.by_pairs = fast_div((uint32_t)w.a.batch * (uint32_t)w.a.geom.n_kv_heads);
  const bool f32 = t == InType::F32;
  if (D == 64) return f32 ? plan<64, true>(w, max_q_len, max_kv_len, s) : plan<64, false>(w, max_q_len, max_kv_len, s);
  if (D == 128) return f32 ? plan<128, true>(w, max_q_len, max_kv_len, s) : plan<128, false>(w, max_q_len, max_kv_len, s);
  return f32 ? plan<256, true>(w, max_q_len, max_kv_len, s) : plan<256, false>(w, max_q_len, max_kv_len, s);
}

}  // namespace nvfp4
