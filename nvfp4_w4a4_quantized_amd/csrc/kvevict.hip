// Rows of the paged NVFP4 key/value cache that move: the accepted path of a drafted tree, and the
// tokens that stay when a sequence is cut to a budget.  Layout: kv_layout.hpp.
//
// A row (one token of one kv head) is 9/8 D bytes in places that its neighbours' lie between:
// D/2 bytes of key codes and D/16 of their scales in one piece each, 16 parts of D/32 bytes of
// value codes, D/16 single bytes of value scales.  16 lanes move a row: a part of the key codes
// and of the value codes each, and a byte of both scales.
#include "kernel_common.hpp"
#include "kv_launch.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = kKvMoveThreads;
constexpr int kWaves = kThreads / 64;
constexpr int kRowLanes = 16;
constexpr int kRows = kThreads / kRowLanes;        // rows that a workgroup moves side by side

template <int D>
struct PartOf { using type = uint32_t; };
template <>
struct PartOf<64> { using type = uint16_t; };
template <>
struct PartOf<256> { using type = uint64_t; };

// What one of its 16 lanes holds of a row
template <int D>
struct RowPart {
  typename PartOf<D>::type k, v;
  uint8_t ks, vs;
};

// A sequence's pages
struct Pages {
  const int32_t* table;
  KvGeom geom;
  int32_t last;                // of the table's entries
  // the page of token t, or -1: an entry outside the cache is never followed
  __device__ __forceinline__ int64_t of(int32_t t) const {
    const int32_t at = t >> geom.page_shift;
    if (t < 0 || at > last) return -1;
    const int32_t id = table[at];
    return id >= 0 && id < geom.n_pages ? id : -1;
  }
  __device__ __forceinline__ int32_t place(int32_t t) const { return t & ((1 << geom.page_shift) - 1); }
  // token t's weight (page: of(t))
  __device__ __forceinline__ int64_t weight_at(int64_t page, int32_t kh, int32_t t) const {
    return ((page * geom.n_kv_heads + kh) << geom.page_shift) + place(t);
  }
};

__device__ __forceinline__ Pages pages_of(const KvPages& p, int b) {
  return Pages{p.table + (int64_t)b * p.ld_table, p.geom, (int32_t)p.max_pages - 1};
}

// Cached tokens of sequence b
__device__ __forceinline__ int32_t length_of(const KvPages& p, const int32_t* kv_len, int b) {
  const int64_t most = p.max_pages << p.geom.page_shift, n = kv_len[b];
  return (int32_t)(n < 0 ? 0 : (n > most ? most : n));
}

template <int D>
__device__ __forceinline__ uint8_t* granule_at(uint8_t* cache, const Pages& p, int64_t page, int32_t kh, int32_t t) {
  return cache + page * p.geom.page_bytes +
         ((int64_t)(kh << (p.geom.page_shift - 4)) + (p.place(t) >> 4)) * kv_granule_bytes(D);
}

template <int D>
__device__ __forceinline__ RowPart<D> load_row(const uint8_t* granule, int32_t t, int l) {
  using P = typename PartOf<D>::type;
  const int r = t & 15;
  RowPart<D> x;
  x.k = *reinterpret_cast<const P*>(granule + r * (D / 2) + l * (D / 32));
  x.v = *reinterpret_cast<const P*>(granule + 9 * D + (r >> 2) * (2 * D) + l * (D / 8) + (r & 3) * (D / 32));
  x.ks = x.vs = 0;
  if (l < D / 16) {
    x.ks = granule[8 * D + r * (D / 16) + l];
    x.vs = granule[17 * D + (r >> 2) * (D / 4) + 4 * l + (r & 3)];
  }
  return x;
}

template <int D>
__device__ __forceinline__ void store_row(uint8_t* granule, int32_t t, int l, const RowPart<D>& x) {
  using P = typename PartOf<D>::type;
  const int r = t & 15;
  *reinterpret_cast<P*>(granule + r * (D / 2) + l * (D / 32)) = x.k;
  *reinterpret_cast<P*>(granule + 9 * D + (r >> 2) * (2 * D) + l * (D / 8) + (r & 3) * (D / 32)) = x.v;
  if (l < D / 16) {
    granule[8 * D + r * (D / 16) + l] = x.ks;
    granule[17 * D + (r >> 2) * (D / 4) + 4 * l + (r & 3)] = x.vs;
  }
}

// Accepted path: a workgroup per sequence, so that the sequence's length may be written where it was
// read.  The rows of whole heads, up to kRows times kHeld at a time, are all read before any is
// written: a path's numbers need not increase.
constexpr int kHeld = kKvMostAccepted / kRows;

template <int D>
__global__ __launch_bounds__(kThreads) void k_kv_accept(KvAcceptArgs a) {
  const int b = blockIdx.x, hkv = a.pages.geom.n_kv_heads;
  const Pages pages = pages_of(a.pages, b);
  const int32_t n = length_of(a.pages, a.kv_len, b);
  int32_t m = 1;
  if (a.cu_q) {
    const int64_t d = (int64_t)a.cu_q[b + 1] - a.cu_q[b];
    m = (int32_t)(d < 0 ? 0 : (d > (1 << 30) ? (1 << 30) : d));
  }
  int32_t count = a.n_accepted[b];
  const int32_t most = m < a.max_accepted ? m : a.max_accepted;
  count = count < 0 ? 0 : (count > most ? most : count);
  const int32_t c0 = n - m;
  const int row = threadIdx.x / kRowLanes, l = threadIdx.x % kRowLanes;
  const int32_t heads = count > 0 ? kHeld * kRows / count : hkv;      // at a time
  for (int32_t h0 = 0; count > 0 && h0 < hkv; h0 += heads) {
    const int32_t rows = (hkv - h0 < heads ? hkv - h0 : heads) * count;
    RowPart<D> x[kHeld];
    uint8_t* to[kHeld];
    int32_t at[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int32_t j = row + i * kRows;
      to[i] = nullptr;
      if (j >= rows) continue;
      const int32_t h = j / count, p = j - h * count;
      int32_t node = a.accepted[(int64_t)b * a.ld_accepted + p];
      node = node < 0 ? 0 : (node >= m ? m - 1 : node);
      const int32_t from = c0 + node;
      at[i] = c0 + p;
      if (from == at[i] || from < 0 || at[i] < 0) continue;
      const int64_t src = pages.of(from), dst = pages.of(at[i]);
      if (src < 0 || dst < 0) continue;
      x[i] = load_row<D>(granule_at<D>(a.cache, pages, src, h0 + h, from), from, l);
      to[i] = granule_at<D>(a.cache, pages, dst, h0 + h, at[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeld; ++i)
      if (to[i]) store_row<D>(to[i], at[i], l, x[i]);
  }
  __syncthreads();                                 // every thread has read the length
  if (threadIdx.x == 0) {
    const int32_t left = c0 + count;
    a.kv_len_out[b] = left < 0 ? 0 : (left > n ? n : left);
  }
}

// Eviction.  A workgroup per sequence and kv head:
//   the weights of the tokens [first, n - last) as 32-bit keys of the same order (in LDS where they
//   fit), the largest kept one by its digits (11, 11 and 10 bits, a histogram each), of the
//   tokens that equal it the lowest ones;
//   kept tokens behind the places of the kept (movers) and free places, ascending, to two lists;
//   mover i to free place i, then the last tokens down, 256 at a time.
constexpr uint32_t kDigits[3] = {21, 10, 0};
constexpr int kBins = 2048;

// Larger weights have larger keys; a NaN counts as -inf, -0 as 0
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t x = __float_as_uint(w == 0.0f ? 0.0f : (w == w ? w : -__builtin_inff()));
  return x & 0x80000000u ? ~x : x | 0x80000000u;
}

// Sum over the threads before this one, and over all (every thread calls it)
__device__ __forceinline__ int32_t sum_before(int32_t x, int32_t* s_waves, int32_t& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int32_t upto = x;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int32_t y = __shfl_up(upto, off);
    if (lane >= off) upto += y;
  }
  __syncthreads();                                 // s_waves of the call before is read
  if (lane == 63) s_waves[wave] = upto;
  __syncthreads();
  int32_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    const int32_t y = s_waves[w];
    before += w < wave ? y : 0;
    all += y;
  }
  return before + upto - x;
}

template <int D>
__global__ __launch_bounds__(kThreads) void k_kv_evict(KvEvictArgs a) {
  extern __shared__ uint32_t s_keys[];
  __shared__ int32_t s_hist[kBins];
  __shared__ int32_t s_waves[kWaves];
  __shared__ int32_t s_found[3];
  const int hkv = a.pages.geom.n_kv_heads;
  const int b = (int)blockIdx.x / hkv, kh = (int)blockIdx.x - b * hkv;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Pages pages = pages_of(a.pages, b);
  const int32_t n = length_of(a.pages, a.kv_len, b), budget = a.budget;
  const bool over = n > budget;
  const int32_t left = over ? budget : n;
  int32_t* const kept = a.kept ? a.kept + (int64_t)blockIdx.x * budget : nullptr;
  // what does not move
  if (kept)
    for (int32_t j = tid; j < budget; j += kThreads) kept[j] = j < left ? j : -1;
  if (a.weights_out && a.weights_out != a.weights)
    for (int32_t j = tid; j < left; j += kThreads) {
      const int64_t page = pages.of(j);
      if (page >= 0) {
        const int64_t at = pages.weight_at(page, kh, j);
        a.weights_out[at] = a.weights[at];
      }
    }
  if (a.lengths && kh == 0 && tid == 0) a.kv_len_out[b] = left;
  if (!over) return;

  const int32_t first = a.first, last = a.last;
  const int32_t rated = n - first - last, keep = budget - first - last, behind = budget - last;
  const bool in_lds = rated <= a.lds_keys;
  auto load_key = [&](int32_t i) {
    const int64_t page = pages.of(first + i);
    return page < 0 ? weight_key(-__builtin_inff()) : weight_key(a.weights[pages.weight_at(page, kh, first + i)]);
  };
  auto key_of = [&](int32_t i) { return in_lds ? s_keys[i] : load_key(i); };
  if (in_lds)
    for (int32_t i = tid; i < rated; i += kThreads) s_keys[i] = load_key(i);

  // the smallest kept key, and how many tokens of it are kept
  uint32_t border = 0, known = 0;
  int32_t wanted = keep, equal = 0;
  if (keep > 0) {
    for (int pass = 0; pass < 3; ++pass) {
      const uint32_t shift = kDigits[pass], mask = pass < 2 ? kBins - 1 : (kBins >> 1) - 1;
      for (int i = tid; i < kBins; i += kThreads) s_hist[i] = 0;
      __syncthreads();
      for (int32_t i = tid; i < rated; i += kThreads) {
        const uint32_t k = key_of(i);
        if ((k & known) == border) atomicAdd(&s_hist[(k >> shift) & mask], 1);
      }
      __syncthreads();
      // bins from the largest digit on, two a thread
      const int hi = kBins - 1 - 2 * tid;
      const int32_t x = s_hist[hi], y = s_hist[hi - 1];
      int32_t all;
      const int32_t before = sum_before(x + y, s_waves, all);
      if (before < wanted && wanted <= before + x + y) {
        const bool upper = wanted <= before + x;
        s_found[0] = upper ? hi : hi - 1;
        s_found[1] = wanted - before - (upper ? 0 : x);
        s_found[2] = upper ? x : y;
      }
      __syncthreads();
      border |= (uint32_t)s_found[0] << shift;
      known |= mask << shift;
      wanted = s_found[1];
      equal = s_found[2];
    }
  }

  // each wave a run of tokens, in order
  const int32_t run = ((rated + kWaves - 1) / kWaves + 63) & ~63;
  const int32_t r0 = wave * run < rated ? wave * run : rated, r1 = r0 + run < rated ? r0 + run : rated;
  const uint64_t below = (1ull << lane) - 1;
  int32_t ties0 = 0;                               // tokens of the border's key before this wave's run
  if (keep > 0 && equal > wanted) {
    int32_t ties = 0;
    for (int32_t i = r0; i < r1; i += 64)
      ties += i + lane < r1 && key_of(i + lane) == border;
    int32_t all;
    // of the waves before: what the first lane has before it
    ties0 = __builtin_amdgcn_readfirstlane(sum_before(ties, s_waves, all));
  }
  // calls f(token, its number among the movers or free places of the run) for each of these
  auto walk = [&](int32_t& movers, int32_t& free_, auto f) {
    int32_t ties = ties0;
    for (int32_t i = r0; i < r1; i += 64) {
      const bool have = i + lane < r1;
      const uint32_t k = have ? key_of(i + lane) : 0;
      const bool tie = have && keep > 0 && k == border;
      const uint64_t tie_lanes = __builtin_amdgcn_ballot_w64(tie);
      const bool stays = have && keep > 0 &&
                         (k > border || (tie && ties + __builtin_popcountll(tie_lanes & below) < wanted));
      ties += __builtin_popcountll(tie_lanes);
      const int32_t t = first + i + lane;
      const bool moves = stays && t >= behind, gap = have && !stays && t < behind;
      const uint64_t mv = __builtin_amdgcn_ballot_w64(moves), gp = __builtin_amdgcn_ballot_w64(gap);
      f(t, moves, movers + __builtin_popcountll(mv & below), gap, free_ + __builtin_popcountll(gp & below));
      movers += __builtin_popcountll(mv);
      free_ += __builtin_popcountll(gp);
    }
  };
  int32_t movers = 0, free_ = 0, moving, gaps;
  walk(movers, free_, [](int32_t, bool, int32_t, bool, int32_t) {});
  const int32_t movers0 = __builtin_amdgcn_readfirstlane(sum_before(lane == 0 ? movers : 0, s_waves, moving));
  const int32_t free0 = __builtin_amdgcn_readfirstlane(sum_before(lane == 0 ? free_ : 0, s_waves, gaps));
  int32_t* const from = a.lists + (int64_t)blockIdx.x * 2 * budget;
  int32_t* const to = from + budget;
  movers = movers0;
  free_ = free0;
  walk(movers, free_, [&](int32_t t, bool moves, int32_t i, bool gap, int32_t j) {
    if (moves) from[i] = t;
    if (gap) to[j] = t;
  });
  __syncthreads();

  const int row = tid / kRowLanes, l = tid % kRowLanes;
  struct Held {
    RowPart<D> x;
    float w;
    uint8_t* to;
    int64_t w_at;
    int32_t t;
  };
  auto read = [&](int32_t old, int32_t place, Held& h) {
    h.to = nullptr;
    const int64_t src = pages.of(old), dst = pages.of(place);
    if (src < 0 || dst < 0) return;
    h.x = load_row<D>(granule_at<D>(a.cache, pages, src, kh, old), old, l);
    h.to = granule_at<D>(a.cache, pages, dst, kh, place);
    h.t = place;
    if (l == 0) {
      if (a.weights_out) {
        h.w = a.weights[pages.weight_at(src, kh, old)];
        h.w_at = pages.weight_at(dst, kh, place);
      }
      if (kept) kept[place] = old;
    }
  };
  auto write = [&](const Held& h) {
    if (!h.to) return;
    store_row<D>(h.to, h.t, l, h.x);
    if (l == 0 && a.weights_out) a.weights_out[h.w_at] = h.w;
  };
  // movers stand behind every free place: nothing that is read here is written
  for (int32_t i = row; i < moving; i += kRows) {
    Held h;
    read(from[i], to[i], h);
    write(h);
  }
  // Down by n - budget: what a chunk overwrites was read by it, by the movers or by chunks before
  for (int32_t j0 = 0; j0 < last; j0 += kHeld * kRows) {
    Held h[kHeld];
#pragma unroll
    for (int i = 0; i < kHeld; ++i) {
      const int32_t j = j0 + i * kRows + row;
      h[i].to = nullptr;
      if (j < last) read(n - last + j, behind + j, h[i]);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHeld; ++i) write(h[i]);
  }
}

// The lengths, where they are written over those that the workgroups read
__global__ __launch_bounds__(256) void k_kv_lengths(KvEvictArgs a) {
  const int b = (int)blockIdx.x * 256 + threadIdx.x;
  if (b >= a.pages.batch) return;
  const int32_t n = length_of(a.pages, a.kv_len, b);
  a.kv_len_out[b] = n < a.budget ? n : a.budget;
}

template <int D>
hipError_t evict(const KvEvictArgs& a, hipStream_t s) {
  const int bytes = a.lds_keys * (int)sizeof(uint32_t);
  const hipError_t e = lds_limit_once<k_kv_evict<D>>(kKvEvictMostKeys * (int)sizeof(uint32_t));
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_kv_evict<D>), dim3((unsigned)(a.pages.batch * a.pages.geom.n_kv_heads)), dim3(kThreads), bytes, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_accept(const KvAcceptArgs& a, int32_t D, hipStream_t s) {
  const dim3 blocks((unsigned)a.pages.batch), threads(kThreads);
  if (D == 64) hipLaunchKernelGGL((k_kv_accept<64>), blocks, threads, 0, s, a);
  else if (D == 128) hipLaunchKernelGGL((k_kv_accept<128>), blocks, threads, 0, s, a);
  else hipLaunchKernelGGL((k_kv_accept<256>), blocks, threads, 0, s, a);
  return hipGetLastError();
}

hipError_t launch_kv_evict(KvEvictArgs a, int32_t D, int64_t max_kv_len, hipStream_t s) {
  const int64_t rated = max_kv_len - a.first - a.last;
  a.lds_keys = (int32_t)(rated < 0 ? 0 : (rated > kKvEvictMostKeys ? 0 : rated));
  a.lengths = a.kv_len_out != a.kv_len;
  const hipError_t e = D == 64 ? evict<64>(a, s) : (D == 128 ? evict<128>(a, s) : evict<256>(a, s));
  if (e != hipSuccess || a.lengths) return e;
  hipLaunchKernelGGL(k_kv_lengths, dim3((unsigned)((a.pages.batch + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace nvfp4
