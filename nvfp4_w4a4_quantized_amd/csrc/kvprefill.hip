// Attention of many query columns over the paged NVFP4 cache (bf16): prompts and chunks.
// The mathematics and numerics are those of kvattn.hip; what differs is the work split.
//
// Here the two matrix products bound the kernel, so keys and values are decoded once per
// workgroup: eight waves share a tile of 64 tokens, decoded to f16 (exactly) into LDS, and
// each wave takes 32 query columns through it with MFMA 32x32x16.  S^T = K q^T leaves a
// lane with scores of one column, 16 of every 32 tokens (tokens 8 (i / 4) + 4 h + i % 4, h =
// lane / 32), which are in place the B operand of O^T = V^T P^T when its K axis takes the
// tokens of a granule in the order quads 0, 2, 1, 3; V^T is written to LDS in that order, so
// the weights never leave the registers.
//
// LDS, twice (a tile is decoded while the one before is used, one barrier per tile):
//   K   [64 tokens][D]: 16-byte chunk c of row t at place c ^ (t mod 16)
//   V^T [D][64 slots]:  16-byte chunk c of row d at place c ^ ((d ^ d/8 ^ d/64) mod 8)
// so that a wave's 16-byte reads of 32 rows, and the decoder's writes, spread over the banks.
// Wave w loads granule w % 4 of the next tile but one, keys (w < 4) or values.
#include "kv_device.hpp"

namespace nvfp4 {

namespace {

constexpr int kPrefillWaves = 8;
constexpr int kPrefillCols = 32 * kPrefillWaves;
constexpr int kTok = 64;

__device__ __forceinline__ f32x16 mfma32(f16x8 a, f16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(a, b, c, 0, 0, 0);
}

template <int D>
__device__ __forceinline__ int k_place(int t, int c) {
  constexpr int M = D == 64 ? 7 : 15;
  return t * 2 * D + ((c ^ (t & M)) << 4);
}

__device__ __forceinline__ int v_place(int d, int c) { return d * 2 * kTok + ((c ^ ((d ^ (d >> 3) ^ (d >> 6)) & 7)) << 4); }

template <int D>
__global__ __launch_bounds__(64 * kPrefillWaves, 2) void k_kv_prefill(KvAttnArgs a) {
  constexpr int KD = D / 32;                       // dwords of codes a lane decodes
  constexpr int NB = D / 32;                       // 32-row blocks of O^T
  constexpr int KS = D / 16;                       // K steps of the first product
  constexpr int SB = D == 256 ? 1 : 2;             // 32-token blocks of scores at a time: what registers hold
  constexpr int KBYTES = kTok * D * 2, BUF = 2 * KBYTES;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];

  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int hkv = a.geom.n_kv_heads, group = a.n_q_heads / hkv;
  const int pairs = a.batch * hkv;
  // the longest spans (last tiles) start first; workgroups side by side differ in the head
  const int pair = blockIdx.x % pairs, kh = pair % hkv;
  const SeqInfo seq = seq_info(a, pair / hkv);
  const int32_t cols = seq.m * group;
  const int32_t tiles = (cols + kPrefillCols - 1) / kPrefillCols;
  const int32_t last_page = (seq.n - 1) >> a.geom.page_shift;
  const int per_head = 1 << (a.geom.page_shift - 4);
  const float kg = a.k_gscale[kh], vg = a.v_gscale[kh];
  const int u = wave & 3, h = lane >> 5, c32 = lane & 31;
  const bool values = wave >= 4;

  for (int32_t tile = tiles - 1 - (int32_t)(blockIdx.x / pairs); tile >= 0; tile -= a.col_tiles) {
    const int32_t col_first = tile * kPrefillCols;
    const int32_t col_end = col_first + kPrefillCols < cols ? col_first + kPrefillCols : cols;
    const Span all = span_of(seq, col_first, col_end, group, a.window);
    const int32_t begin = all.lo & ~15;
    const int32_t steps = seq.n > 0 ? (all.hi - begin + kTok - 1) / kTok : 0;

    // this wave's columns
    const int32_t col0 = col_first + 32 * wave;
    const bool live = col0 < col_end;
    const int32_t col1 = col0 + 32 < col_end ? col0 + 32 : col_end;
    Span sp{0, 0, 0, 0};
    if (live) sp = span_of(seq, col0, col1, group, a.window);
    int32_t col = col0 + c32;
    if (col >= col_end) col = col_end - 1;
    const int32_t qi = col / group;
    const int head = kh * group + (col - qi * group);

    // loads of tile s: this wave's granule, its page id known one tile ahead
    auto page_of = [&](int32_t s) -> int32_t {
      int32_t pg = (begin + s * kTok + 16 * u) >> a.geom.page_shift;
      pg = pg < last_page ? pg : last_page;
      const int32_t id = a.table[(int64_t)(pair / hkv) * a.ld_table + pg];
      return id < 0 ? 0 : (id >= a.geom.n_pages ? (int32_t)a.geom.n_pages - 1 : id);
    };
    uint32_t raw[KD], rs = 0;
    auto load = [&](int32_t s, int32_t id) {
      int32_t gr = (begin + s * kTok) / 16 + u;
      const int32_t last = (seq.n - 1) >> 4;
      gr = gr < last ? gr : last;
      const uint8_t* p = a.cache + (int64_t)id * a.geom.page_bytes +
                         (int64_t)(kh * per_head + (gr & (per_head - 1))) * kv_granule_bytes(D);
      if (!values) {
        load_dwords<KD>(p + lane * (D / 8), raw);
        const uint8_t* ps = p + 8 * D + lane * (D / 64);
        if constexpr (D == 64) rs = *ps;
        else if constexpr (D == 128) rs = *reinterpret_cast<const uint16_t*>(ps);
        else rs = *reinterpret_cast<const uint32_t*>(ps);
      } else {
        load_dwords<KD>(p + 9 * D + lane * (D / 8), raw);
        rs = *reinterpret_cast<const uint32_t*>(p + 17 * D + ((lane >> 4) * (D / 16) + (lane & 15) * D / 256) * 4);
      }
    };
    // decode the loaded granule of tile s into its buffer
    auto decode = [&](int32_t s) {
      uint8_t* buf = lds + (s & 1) * BUF;
      if (!values) {
        const int t = 16 * u + lane / 4, part = lane % 4;
#pragma unroll
        for (int i = 0; i < KD; ++i) {
          const f16x2 sc = bcast(scale_pair_f16(D == 256 ? rs >> (16 * (i / 4)) : rs), D == 64 ? 0 : (i >> 1) & 1);
          *reinterpret_cast<f16x8*>(buf + k_place<D>(t, part * KD + i)) = decode8_f16(raw[i], sc);
        }
      } else {
        const int g = lane >> 4, r = lane & 15;
        const int32_t left = seq.n - (begin + s * kTok + 16 * u + 4 * g);
        const uint32_t sb = left >= 4 ? rs : (left <= 0 ? 0u : rs & ((1u << (8 * left)) - 1u));
        f16x2 sc[2];
        sc[0] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sb, 1.0f, false);
        sc[1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(sb, 1.0f, true);
        const int chunk = 2 * u + (g & 1);
        uint8_t* base = buf + KBYTES + (g >> 1) * 8;
#pragma unroll
        for (int part = 0; part < (KD + 3) / 4; ++part) {
          uint32_t w[4], lo[2], hi[2];
          value_words<D>(raw, part, w);
          pair_tokens(w, lo, hi);
          auto put = [&](int j, f16x2 x, f16x2 y) {
            const int d = r * (D / 16) + 8 * part + j;
            typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));
            *reinterpret_cast<f16x4*>(base + v_place(d, chunk)) = f16x4{x[0], x[1], y[0], y[1]};
          };
#define NVFP4_VROWS(SEL)                                                     \
  if constexpr (2 * (SEL) < D / 16) {                                        \
    put(2 * (SEL), cvt_fp4<SEL>(lo[0]) * sc[0], cvt_fp4<SEL>(lo[1]) * sc[1]); \
    put(2 * (SEL) + 1, cvt_fp4<SEL>(hi[0]) * sc[0], cvt_fp4<SEL>(hi[1]) * sc[1]); \
  }
          NVFP4_VROWS(0)
          NVFP4_VROWS(1)
          NVFP4_VROWS(2)
          NVFP4_VROWS(3)
#undef NVFP4_VROWS
        }
      }
    };

    int32_t id_next = 0;
    __syncthreads();                               // the tile before is done with LDS
    if (steps > 0) {
      load(0, page_of(0));
      id_next = page_of(1);
    }

    // query columns: B operand of K step k: elements 16 k + 8 h + j of column c32
    f16x8 qf[KS];
    float amax = 0.0f;
    {
      float v[KS][8];
      const int64_t off = (seq.q0 + qi) * a.ldq + (int64_t)head * D + 8 * h;
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        load8<false>(a.q, off + 16 * k, v[k]);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = __builtin_fmaxf(amax, __builtin_fabsf(v[k][e]));
      }
      amax = __builtin_fmaxf(amax, xor32(amax));
      const float up = query_up(amax);
#pragma unroll
      for (int k = 0; k < KS; ++k)
#pragma unroll
        for (int e = 0; e < 8; ++e) qf[k][e] = (_Float16)(v[k][e] * up);
    }
    const float csc = a.scale * kLog2e * kg * query_down(amax);
    const int32_t pos = seq.n - seq.m + qi;
    const int32_t limit = pos + 1, floor_ = a.window ? pos - a.window + 1 : 0;
    float m = kNegBig, l = 0.0f;
    f32x16 acc[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][e] = 0.0f;

    if (steps > 0) {
      decode(0);
      if (steps > 1) {
        load(1, id_next);
        id_next = page_of(2);
      }
      __syncthreads();
    }
    for (int32_t s = 0; s < steps; ++s) {
      if (s + 1 < steps) {
        decode(s + 1);
        if (s + 2 < steps) {
          load(s + 2, id_next);
          id_next = page_of(s + 3);
        }
      }
      const int32_t t0 = begin + s * kTok;
      if (live && t0 < sp.hi && t0 + kTok > sp.lo) {
        const uint8_t* kb = lds + (s & 1) * BUF;
        const uint8_t* vb = kb + KBYTES;
#pragma unroll
        for (int pass = 0; pass < 2 / SB; ++pass) {
        f32x16 sc[SB];
#pragma unroll
        for (int i = 0; i < SB; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) sc[i][e] = 0.0f;
#pragma unroll
        for (int k = 0; k < KS; ++k)
#pragma unroll
          for (int i = 0; i < SB; ++i) {
            const f16x8 kf = *reinterpret_cast<const f16x8*>(kb + k_place<D>(32 * (SB * pass + i) + c32, 2 * k + h));
            sc[i] = mfma32(kf, qf[k], sc[i]);
          }
#pragma unroll
        for (int i = 0; i < SB; ++i) sc[i] *= csc;
        if (t0 < sp.all_lo || t0 + kTok > sp.all_hi) {
#pragma unroll
          for (int i = 0; i < SB; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int32_t t = t0 + 32 * (SB * pass + i) + 8 * (e / 4) + 4 * h + e % 4;
              if (t >= limit || t < floor_) sc[i][e] = -__builtin_inff();
            }
        }
        float top = -__builtin_inff();
#pragma unroll
        for (int i = 0; i < SB; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) top = __builtin_fmaxf(top, sc[i][e]);
        top = __builtin_fmaxf(top, xor32(top));
        if (__builtin_amdgcn_ballot_w64(top > m + 15.0f)) {
          const float m1 = __builtin_fmaxf(m, top - 7.0f);
          const float f = __builtin_amdgcn_exp2f(m - m1);
          m = m1;
          l *= f;
#pragma unroll
          for (int i = 0; i < NB; ++i) acc[i] *= f;
        }
        f16x8 pf[2 * SB];
#pragma unroll
        for (int i = 0; i < SB; ++i)
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float p = __builtin_amdgcn_exp2f(sc[i][e] - m);
            l += p;
            pf[2 * i + e / 8][e % 8] = (_Float16)p;
          }
#pragma unroll
        for (int k = 0; k < 2 * SB; ++k)
#pragma unroll
          for (int i = 0; i < NB; ++i) {
            const f16x8 vf = *reinterpret_cast<const f16x8*>(vb + v_place(32 * i + c32, 2 * (2 * SB * pass + k) + h));
            acc[i] = mfma32(vf, pf[k], acc[i]);
          }
        }
      }
      __syncthreads();
    }

    l += xor32(l);
    if (col0 + c32 < col_end) {
      const float f = l > 0.0f ? vg / l : 0.0f;
      uint16_t* dst = reinterpret_cast<uint16_t*>(a.o) + (seq.q0 + qi) * a.ldo + (int64_t)head * D + 4 * h;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int e = 0; e < 16; e += 4)
          *reinterpret_cast<u32x2*>(dst + 32 * i + 2 * e) =
              u32x2{pack_bf16(acc[i][e] * f, acc[i][e + 1] * f), pack_bf16(acc[i][e + 2] * f, acc[i][e + 3] * f)};
      if (a.lse && h == 0)
        a.lse[(seq.q0 + qi) * a.n_q_heads + head] = l > 0.0f ? (m + __builtin_log2f(l)) * kLn2 : -__builtin_inff();
    }
  }
}

template <int D>
hipError_t launch(const KvAttnArgs& a, hipStream_t s) {
  constexpr int bytes = 2 * 2 * kTok * D * 2;
  const hipError_t e = lds_limit_once<k_kv_prefill<D>>(bytes);
  if (e != hipSuccess) return e;
  const int64_t blocks = (int64_t)a.batch * a.geom.n_kv_heads * a.col_tiles;
  hipLaunchKernelGGL((k_kv_prefill<D>), dim3((unsigned)blocks), dim3(64 * kPrefillWaves), bytes, s, a);
  return hipGetLastError();
}

}  // namespace

int32_t kv_prefill_cols() { return kPrefillCols; }

hipError_t launch_kv_prefill(const KvAttnArgs& a, int32_t D, hipStream_t s) {
  if (D == 64) return launch<64>(a, s);
  if (D == 128) return launch<128>(a, s);
  return launch<256>(a, s);
}

}  // namespace nvfp4
