// The paged NVFP4 key/value cache: position rotation, quantization and appending of
// new tokens, and reading rows back as values.  Layout: kv_layout.hpp.
//
// Rotation of a head row x at position p, with c = cos[p], s = sin[p] and R = rot_dim:
//   half-split    y_i = x_i c_i - x_{i+R/2} s_i,  y_{i+R/2} = x_{i+R/2} c_i + x_i s_i   (i < R/2)
//   interleaved   y_{2i} = x_{2i} c_i - x_{2i+1} s_i,  y_{2i+1} = x_{2i+1} c_i + x_{2i} s_i
// elements from R on unchanged; both products and their sum or difference are rounded
// to fp32 separately, so that the codes of the rotated keys are reproducible.  Keys and
// values are then NVFP4 blocks of 16 along the head, quantized from the fp32 values
// (the rotated key is not rounded to the input type first) by the layer's exact
// block-scale and code routines under one calibrated global scale per kv head.
#include "kernel_common.hpp"
#include "kv_launch.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = kKvRowThreads;
constexpr int kWaves = kThreads / 64;

// 16 consecutive elements of a row as fp32
template <InType T>
__device__ __forceinline__ void load16(const void* base, int64_t off, float v[16]) {
  if constexpr (T == InType::BF16) {
    const u32x4* p = reinterpret_cast<const u32x4*>(reinterpret_cast<const uint16_t*>(base) + off);
    const u32x4 a = p[0], b = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
      v[8 + 2 * i] = __uint_as_float(b[i] << 16);
      v[8 + 2 * i + 1] = __uint_as_float(b[i] & 0xFFFF0000u);
    }
  } else {
    const f32x4* p = reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f32x4 a = p[i];
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] = a[e];
    }
  }
}

template <InType T>
__device__ __forceinline__ void store16(void* base, int64_t off, const float v[16]) {
  if constexpr (T == InType::BF16) {
    u32x4* p = reinterpret_cast<u32x4*>(reinterpret_cast<uint16_t*>(base) + off);
    u32x4 a, b;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      a[i] = f32_to_bf16_bits(v[2 * i]) | (f32_to_bf16_bits(v[2 * i + 1]) << 16);
      b[i] = f32_to_bf16_bits(v[8 + 2 * i]) | (f32_to_bf16_bits(v[8 + 2 * i + 1]) << 16);
    }
    p[0] = a;
    p[1] = b;
  } else {
    f32x4* p = reinterpret_cast<f32x4*>(reinterpret_cast<float*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]};
  }
}

__device__ __forceinline__ void load_f32(const float* p, int n4, float* v) {
#pragma unroll
  for (int i = 0; i < n4; ++i) {
    const f32x4 a = reinterpret_cast<const f32x4*>(p)[i];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[4 * i + e] = a[e];
  }
}

// Block b (16 elements) of a head row at x + off, rotated
template <InType T>
__device__ __forceinline__ void load_rotated(const KvAppendArgs& a, const void* x, int64_t off, int b, int64_t pos,
                                             float v[16]) {
  load16<T>(x, off + 16 * b, v);
  const int rb = a.rot_dim >> 4;                     // rotated blocks (even)
  if (b >= rb) return;
  const int64_t row = pos * (a.rot_dim >> 1);
  if (a.interleaved) {
    float c[8], s[8];
    load_f32(a.cos + row + 8 * b, 2, c);
    load_f32(a.sin + row + 8 * b, 2, s);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x0 = v[2 * i], x1 = v[2 * i + 1];
      v[2 * i] = x0 * c[i] - x1 * s[i];
      v[2 * i + 1] = x1 * c[i] + x0 * s[i];
    }
  } else {
    const bool low = b < (rb >> 1);
    const int lb = low ? b : b - (rb >> 1);          // the pair's lower block
    float w[16], c[16], s[16];
    load16<T>(x, off + 16 * (low ? b + (rb >> 1) : lb), w);
    load_f32(a.cos + row + 16 * lb, 4, c);
    load_f32(a.sin + row + 16 * lb, 4, s);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const float t = w[i] * s[i];
      v[i] = v[i] * c[i] + (low ? -t : t);           // x - t and x + (-t) round alike
    }
  }
}

// 16 bytes that are read (written) once: non-temporal where the call's queries exceed the
// caches, so that they do not push out what does get read again
template <bool STREAM, typename V>
__device__ __forceinline__ V load_once(const void* p) {
  if constexpr (STREAM) return __builtin_nontemporal_load(static_cast<const V*>(p));
  else return *static_cast<const V*>(p);
}
template <bool STREAM, typename V>
__device__ __forceinline__ void store_once(V x, void* p) {
  if constexpr (STREAM) __builtin_nontemporal_store(x, static_cast<V*>(p));
  else *static_cast<V*>(p) = x;
}

// 8 consecutive elements as fp32, and back
template <InType T, bool STREAM>
__device__ __forceinline__ void load8_once(const void* base, int64_t off, float v[8]) {
  if constexpr (T == InType::BF16) {
    const u32x4 a = load_once<STREAM, u32x4>(static_cast<const uint16_t*>(base) + off);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(a[i] << 16);
      v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const f32x4 a = load_once<STREAM, f32x4>(static_cast<const float*>(base) + off + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] = a[e];
    }
  }
}

template <InType T, bool STREAM>
__device__ __forceinline__ void store8_once(void* base, int64_t off, const float v[8]) {
  if constexpr (T == InType::BF16) {
    u32x4 a;
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = f32_to_bf16_bits(v[2 * i]) | (f32_to_bf16_bits(v[2 * i + 1]) << 16);
    store_once<STREAM>(a, static_cast<uint16_t*>(base) + off);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      store_once<STREAM>(f32x4{v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]},
                         static_cast<float*>(base) + off + 4 * i);
  }
}

// Part j of D / 16 of a query row: two runs of 8 elements that the rotation pairs up (the
// lower and the upper one of the halves, or 16 consecutive elements), so that the row is read
// once.
template <InType T, bool STREAM>
__device__ __forceinline__ void rotate_query(const KvAppendArgs& a, const void* x, int64_t off, int j, int64_t pos,
                                             void* out, int64_t out_off) {
  const int half = a.rot_dim >> 1;
  const bool rotated = 16 * j < a.rot_dim, split = rotated && !a.interleaved;
  const int lo = split ? 8 * j : 16 * j, hi = split ? 8 * j + half : 16 * j + 8;
  float v[8], w[8];
  load8_once<T, STREAM>(x, off + lo, v);
  load8_once<T, STREAM>(x, off + hi, w);
  if (rotated) {
    float c[8], s[8];
    load_f32(a.cos + pos * half + 8 * j, 2, c);
    load_f32(a.sin + pos * half + 8 * j, 2, s);
    if (!a.interleaved) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float x0 = v[i], x1 = w[i];
        v[i] = x0 * c[i] - x1 * s[i];
        w[i] = x1 * c[i] + x0 * s[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x0 = v[2 * i], x1 = v[2 * i + 1], y0 = w[2 * i], y1 = w[2 * i + 1];
        v[2 * i] = x0 * c[i] - x1 * s[i];
        v[2 * i + 1] = x1 * c[i] + x0 * s[i];
        w[2 * i] = y0 * c[4 + i] - y1 * s[4 + i];
        w[2 * i + 1] = y1 * c[4 + i] + y0 * s[4 + i];
      }
    }
  }
  store8_once<T, STREAM>(out, out_off + lo, v);
  store8_once<T, STREAM>(out, out_off + hi, w);
}

// Byte address of the granule of (head, token slot); the slot is inside the cache
__device__ __forceinline__ int64_t granule_at(const KvGeom& g, int D, int head, int64_t slot) {
  const int64_t page = slot >> g.page_shift;
  const int64_t in_page = slot & (((int64_t)1 << g.page_shift) - 1);
  const int64_t per_head = (int64_t)1 << (g.page_shift - 4);
  return page * g.page_bytes + ((int64_t)head * per_head + (in_page >> 4)) * kv_granule_bytes(D);
}

// A wave takes 64 / (D / 16) consecutive tokens of one head of q, k or v: a lane one
// block of 16 elements, so that its amax needs no cross-lane step, and the wave's code
// stores are whole granule pieces (at D = 128, 8 tokens: 512 contiguous bytes of keys,
// two 256-byte quads of values).  The partner half of a rotated block is read again by
// its own lane (the row is in the L1 then) rather than exchanged.  Which of q, k, v is
// wave-uniform.
// Bound by HBM from a few thousand tokens on: 8192 tokens of 32 / 8 heads of 128 in bf16 read and
// write 180 MB in 38.5 us, 4.7 TB/s (a 1 GiB copy moves 5.2); 96 or fewer tokens take 3.5 us, a
// launch and one round trip to memory.
template <InType T, int D, bool STREAM>
__global__ __launch_bounds__(kThreads) void k_rope_append(KvAppendArgs a) {
  constexpr int BPR = D / 16, TPW = 64 / BPR;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t task = (int64_t)blockIdx.x * kWaves + wave;
  const int heads = a.n_q_heads + 2 * a.geom.n_kv_heads;
  const int64_t group = task / heads;
  const int h = (int)(task - group * heads);
  const int64_t t = group * TPW + lane / BPR;
  const int b = lane % BPR;
  if (t >= a.T) return;
  if (h < a.n_q_heads + a.geom.n_kv_heads) {
    int64_t pos = a.positions[t];
    pos = pos < 0 ? 0 : (pos >= a.n_pos ? a.n_pos - 1 : pos);
    if (h < a.n_q_heads) {
      rotate_query<T, STREAM>(a, a.q, t * a.ldq + (int64_t)h * D, b, pos, a.q_out, t * a.ldqo + (int64_t)h * D);
      return;
    }
    float v[16];
    const int kh = h - a.n_q_heads;
    const int64_t slot = a.slots[t];
    if (slot < 0 || (slot >> a.geom.page_shift) >= a.geom.n_pages) return;
    load_rotated<T>(a, a.k, t * a.ldk + (int64_t)kh * D, b, pos, v);
    const float g = a.k_gscale[kh];
    const uint32_t sb = block_scale_byte(amax_abs<16>(v), g);
    uint32_t w[2];
    quant16(v, sb, g, w);
    uint8_t* p = a.cache + granule_at(a.geom, D, kh, slot);
    const int r = (int)(slot & 15);
    *reinterpret_cast<u32x2*>(p + r * (D / 2) + 8 * b) = u32x2{w[0], w[1]};
    p[8 * D + r * BPR + b] = (uint8_t)sb;
    return;
  }
  const int kh = h - a.n_q_heads - a.geom.n_kv_heads;
  const int64_t slot = a.slots[t];
  if (slot < 0 || (slot >> a.geom.page_shift) >= a.geom.n_pages) return;
  float v[16];
  load16<T>(a.v, t * a.ldv + (int64_t)kh * D + 16 * b, v);
  const float g = a.v_gscale[kh];
  const uint32_t sb = block_scale_byte(amax_abs<16>(v), g);
  uint32_t w[2];
  quant16(v, sb, g, w);
  uint8_t* p = a.cache + granule_at(a.geom, D, kh, slot);
  const int quad = (int)(slot >> 2) & 3, e = (int)slot & 3;
  constexpr int PART = D / 32;                       // bytes of one of the row's 16 parts: 2, 4 or 8
  uint8_t* pv = p + 9 * D + (quad * 16 + (8 / PART) * b) * 4 * PART + e * PART;
  if constexpr (PART == 8) {
    *reinterpret_cast<u32x2*>(pv) = u32x2{w[0], w[1]};
  } else if constexpr (PART == 4) {
    *reinterpret_cast<uint32_t*>(pv) = w[0];
    *reinterpret_cast<uint32_t*>(pv + 16) = w[1];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) *reinterpret_cast<uint16_t*>(pv + 8 * i) = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
  }
  p[17 * D + (quad * BPR + b) * 4 + e] = (uint8_t)sb;
}

// Values of cache rows: a lane decodes one block, e2m1 * s exact in fp32, times g
// rounded once, then once to the output type.  Tokens without a slot give zeros.
// 8192 tokens of 8 heads of 128 take 12.1 us: 44 MB at 3.6 TB/s, 1.4 times what a copy of them
// would, 2.2 us of it the launch, which is all that 96 tokens or fewer take.
template <InType T, int D>
__global__ __launch_bounds__(kThreads) void k_kv_gather(KvGatherArgs a) {
  constexpr int BPR = D / 16, TPW = 64 / BPR;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t task = (int64_t)blockIdx.x * kWaves + wave;
  const int heads = 2 * a.geom.n_kv_heads;
  const int64_t group = task / heads;
  const int h = (int)(task - group * heads);
  const int64_t t = group * TPW + lane / BPR;
  const int b = lane % BPR;
  if (t >= a.T) return;
  const bool values = h >= a.geom.n_kv_heads;
  const int kh = values ? h - a.geom.n_kv_heads : h;
  const int64_t slot = a.slots[t];
  uint32_t w[2] = {0u, 0u}, sb = 0u;
  if (slot >= 0 && (slot >> a.geom.page_shift) < a.geom.n_pages) {
    const uint8_t* p = a.cache + granule_at(a.geom, D, kh, slot);
    if (!values) {
      const int r = (int)(slot & 15);
      const u32x2 x = *reinterpret_cast<const u32x2*>(p + r * (D / 2) + 8 * b);
      w[0] = x[0];
      w[1] = x[1];
      sb = p[8 * D + r * BPR + b];
    } else {
      constexpr int PART = D / 32;
      const int quad = (int)(slot >> 2) & 3, e = (int)slot & 3;
      const uint8_t* pv = p + 9 * D + (quad * 16 + (8 / PART) * b) * 4 * PART + e * PART;
      if constexpr (PART == 8) {
        const u32x2 x = *reinterpret_cast<const u32x2*>(pv);
        w[0] = x[0];
        w[1] = x[1];
      } else if constexpr (PART == 4) {
        w[0] = *reinterpret_cast<const uint32_t*>(pv);
        w[1] = *reinterpret_cast<const uint32_t*>(pv + 16);
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i >> 1] |= (uint32_t)*reinterpret_cast<const uint16_t*>(pv + 8 * i) << (16 * (i & 1));
      }
      sb = p[17 * D + (quad * BPR + b) * 4 + e];
    }
  }
  const float g = (values ? a.v_gscale : a.k_gscale)[kh];
  const f16x2 s2 = scale_f16x2(sb);
  float v[16];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f16x8 x = decode8_f16(w[i], s2);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[8 * i + e] = (float)x[e] * g;
  }
  store16<T>(values ? a.v_out : a.k_out, t * (values ? a.ldv : a.ldk) + (int64_t)kh * D + 16 * b, v);
}

}  // namespace

hipError_t launch_rope_append(const KvAppendArgs& a, InType t, int32_t D, hipStream_t s) {
  const dim3 grid((unsigned)kv_row_blocks(a.T, a.n_q_heads + 2 * (int64_t)a.geom.n_kv_heads, D)), block(kThreads);
  // queries beyond the L2s (32 MiB): 8192 tokens of 32 heads of 128 in bf16 54.3 us with ordinary
  // loads and stores, 50.1 us with non-temporal ones; 1543 fp32 tokens of 15 heads of 64 the other way
  // round, 10.9 and 12.4 us (with the read-back of the rows in both)
  const bool stream = a.T * a.n_q_heads * D * (t == InType::BF16 ? 2 : 4) > (int64_t(32) << 20);
#define NVFP4_APPEND_AS(DD, S)                                                                            \
  if (t == InType::BF16) hipLaunchKernelGGL((k_rope_append<InType::BF16, DD, S>), grid, block, 0, s, a);  \
  else hipLaunchKernelGGL((k_rope_append<InType::F32, DD, S>), grid, block, 0, s, a)
#define NVFP4_APPEND(DD)                    \
  if (stream) { NVFP4_APPEND_AS(DD, true); } \
  else { NVFP4_APPEND_AS(DD, false); }
  if (D == 64) { NVFP4_APPEND(64) }
  else if (D == 128) { NVFP4_APPEND(128) }
  else { NVFP4_APPEND(256) }
#undef NVFP4_APPEND
#undef NVFP4_APPEND_AS
  return hipGetLastError();
}

hipError_t launch_kv_gather(const KvGatherArgs& a, InType t, int32_t D, hipStream_t s) {
  const dim3 grid((unsigned)kv_row_blocks(a.T, 2 * (int64_t)a.geom.n_kv_heads, D)), block(kThreads);
#define NVFP4_GATHER(DD)                                                                            \
  if (t == InType::BF16) hipLaunchKernelGGL((k_kv_gather<InType::BF16, DD>), grid, block, 0, s, a); \
  else hipLaunchKernelGGL((k_kv_gather<InType::F32, DD>), grid, block, 0, s, a)
  if (D == 64) { NVFP4_GATHER(64); }
  else if (D == 128) { NVFP4_GATHER(128); }
  else { NVFP4_GATHER(256); }
#undef NVFP4_GATHER
  return hipGetLastError();
}

}  // namespace nvfp4
