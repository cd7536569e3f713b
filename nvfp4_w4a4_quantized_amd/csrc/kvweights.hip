// The attention weight that cached tokens receive, summed over query tokens and the heads of a
// group, from the queries' log-sums:
//   W_t <- decay W_t [t < n - m] + sum_{i, h} e^{scale <q_ih, k_t> - lse_ih}  over the i that attend to t
//
// S = q K^T on the f16 MFMA 16x16x32: the rows are query columns (query token x head), the columns
// tokens, so that a lane has four query columns of one token and sums in place; over all query
// columns the sum stays in one register a token, in an order that does not depend on the grid.
// Numerics of the product as in kvattn.hip; exponents, weights and sums are fp32.
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
  uint32_t k[D / 32], ks[D == 256 ? 2 : 1];
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

template <int D, bool F32>
__global__ __launch_bounds__(64 * kWeightWaves) void k_kv_weights(KvWeightsArgs w) {
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
  const int32_t c0 = seq.n - seq.m;
  const float kg = a.k_gscale[kh];

  // tokens past the planned ones go with the first tiles
  for (int64_t tile = (int)blockIdx.x - item * w.tiles; tile * (kWeightWaves * kWaveTokens) < seq.n; tile += w.tiles) {
    const int32_t t0 = (int32_t)tile * (kWeightWaves * kWaveTokens) + wave * kWaveTokens;
    if (t0 >= seq.n) break;
    const QueryRange q = queries_of(seq, t0, kWaveTokens, a.window);
    const bool any = q.first < q.end;
    if (!any && w.decay == 1.0f) continue;

    int64_t page[NG];
    f16x8 kf[NG][KC];
#pragma unroll
    for (int u = 0; u < NG; ++u) {
      int32_t t = t0 + 16 * u;
      t = t < seq.n ? t : seq.n - 1;                 // past the end: the last granule again
      const int32_t id = __builtin_amdgcn_readfirstlane(a.table[(int64_t)b * a.ld_table + (t >> a.geom.page_shift)]);
      page[u] = id;
      const int32_t read = id < 0 ? 0 : (id >= a.geom.n_pages ? (int32_t)a.geom.n_pages - 1 : id);
      if (any) {
        Keys<D> x;
        load_keys<D>(granule_buffer<D>(a, read, kh * per_head + ((t >> 4) & (per_head - 1))), lane, x);
#pragma unroll
        for (int c = 0; c < KC; ++c) kf[u][c] = key_frag<D>(x, c);
      }
    }

    float sum[NG] = {};
    for (int32_t col0 = q.first * group; any && col0 < q.end * group; col0 += 16) {
      const int32_t cols = q.end * group;
      // A operand: row r of the block of columns
      int32_t col = col0 + r;
      const bool past = col >= cols;
      col = past ? cols - 1 : col;
      const int32_t qi = col / a.by_group, head = kh * group + (col - qi * group);
      const int64_t off = (seq.q0 + qi) * a.ldq + (int64_t)head * D;
      float v[KC][8];
      float amax = 0.0f;
#pragma unroll
      for (int c = 0; c < KC; ++c) {
        load8<F32>(a.q, off + (D == 64 ? 16 * g + 8 * c : 128 * (c / 4) + 32 * g + 8 * (c % 4)), v[c]);
#pragma unroll
        for (int e = 0; e < 8; ++e) amax = __builtin_fmaxf(amax, __builtin_fabsf(v[c][e]));
      }
      amax = max_xor32(max_xor16(amax));
      const float up = a.scale < 0.0f ? -query_up(amax) : query_up(amax);
      const float csc_r = score_factor(a.scale, kg, amax);
      const float lse = w.lse[(seq.q0 + qi) * a.n_q_heads + head];
      // a row that attends to nothing, or is not there, has no weights
      const float sub_r = past || lse == -__builtin_inff() ? __builtin_inff() : lse * kLog2e;
      f16x8 qf[TERMS][KC];
#pragma unroll
      for (int c = 0; c < KC; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = v[c][e] * up;
          const _Float16 hi = (_Float16)x;
          qf[0][c][e] = hi;
          if constexpr (F32) qf[TERMS - 1][c][e] = (_Float16)(x - (float)hi);
        }
      // the results' rows: 4 g + i
      float csc[4], sub[4];
      int32_t pos[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        csc[i] = __shfl(csc_r, 4 * g + i);
        sub[i] = __shfl(sub_r, 4 * g + i);
        pos[i] = c0 + __shfl(qi, 4 * g + i);
      }
#pragma unroll
      for (int u = 0; u < NG; ++u) {
        f32x4 s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int c = 0; c < KC; ++c)
#pragma unroll
          for (int e = 0; e < TERMS; ++e) s = mfma16(qf[e][c], kf[u][c], s);
        const int32_t t = t0 + 16 * u + r;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const bool sees = t <= pos[i] && (!a.window || t > pos[i] - a.window);
          const float x = sees ? __builtin_fmaf(s[i], csc[i], -sub[i]) : -__builtin_inff();
          sum[u] += __builtin_amdgcn_exp2f(x);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < NG; ++u) {
      const float total = sum_xor32(sum_xor16(sum[u]));
      const int32_t t = t0 + 16 * u + r;
      if (g == 0 && t < seq.n && page[u] >= 0 && page[u] < a.geom.n_pages) {
        float* const at = w.weights + (((page[u] * hkv + kh) << a.geom.page_shift) + (t & ((1 << a.geom.page_shift) - 1)));
        *at = t < c0 && w.decay != 0.0f ? __builtin_fmaf(w.decay, *at, total) : total;
      }
    }
  }
}

template <int D>
hipError_t launch(const KvWeightsArgs& w, InType t, hipStream_t s) {
  const dim3 blocks((unsigned)((int64_t)w.a.batch * w.a.geom.n_kv_heads * w.tiles)), threads(64 * kWeightWaves);
  if (t == InType::F32) hipLaunchKernelGGL((k_kv_weights<D, true>), blocks, threads, 0, s, w);
  else hipLaunchKernelGGL((k_kv_weights<D, false>), blocks, threads, 0, s, w);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_weights(KvWeightsArgs w, InType t, int32_t D, int64_t max_kv_len, hipStream_t s) {
  const int64_t tokens = kWeightWaves * kWaveTokens, pairs = (int64_t)w.a.batch * w.a.geom.n_kv_heads;
  const int64_t tiles = max_kv_len < 1 ? 1 : (max_kv_len + tokens - 1) / tokens;
  w.tiles = kv_planned_tiles(tiles, pairs, 64 * kWeightWaves);
  w.by_tiles = fast_div((uint32_t)w.tiles);
  w.a.by_group = fast_div((uint32_t)(w.a.n_q_heads / w.a.geom.n_kv_heads));
  w.a.by_heads = fast_div((uint32_t)w.a.geom.n_kv_heads);
  if (D == 64) return launch<64>(w, t, s);
  if (D == 128) return launch<128>(w, t, s);
  return launch<256>(w, t, s);
}

}  // namespace nvfp4
