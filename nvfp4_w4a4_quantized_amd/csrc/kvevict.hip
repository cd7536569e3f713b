// Rows of the paged NVFP4 key/value cache that move: the accepted path of a drafted tree, and the
// tokens that stay when a sequence is cut to a budget.  Layout: kv_layout.hpp.
//
// A row (one token of one kv head) is 9/8 D bytes in places that its neighbours' lie between:
// D/2 bytes of key codes and D/16 of their scales in one piece each, 16 parts of D/32 bytes of
// value codes, D/16 single bytes of value scales.  A wave moves 16 rows: four lanes a row its keys, in a load
// of both (16 bytes a lane at D = 128), then 16 lanes a row the parts of the values, in four, and D/16
// lanes a row their scales.  What counts is the number of such loads and stores, not their bytes (with
// 16 lanes a row for everything, twice as many: 32 x 8 heads of about 4130 tokens to 4096 19 us, not 17).
#include <type_traits>

#include "kernel_common.hpp"
#include "kv_launch.hpp"

namespace nvfp4 {

namespace {

constexpr int kThreads = kKvMoveThreads;
constexpr int kWaves = kThreads / 64;
constexpr int kWaveRows = 16;                      // rows of a wave
constexpr int kRows = kWaves * kWaveRows;          // and of a workgroup

// A sequence's pages
struct Pages {
  const int32_t* table;
  KvGeom geom;
  int32_t last;                // of the table's entries
  // the page of token t, or -1: an entry outside the cache is never followed.  (No branches here and in what
  // follows: loads are counted in order, and a load that waits for another one, or for a branch, holds up all
  // those behind it.)
  __device__ __forceinline__ int32_t of(int32_t t) const {
    const int32_t at = t >> geom.page_shift, id = table[at < 0 ? 0 : (at > last ? last : at)];
    return at >= 0 && at <= last && id >= 0 && id < geom.n_pages ? id : -1;
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

// Where a row is: 16 times the place of its granule in the cache, and its place in the granule
template <int D>
__device__ __forceinline__ int64_t row_at(const Pages& p, int64_t page, int32_t kh, int32_t t) {
  return (page * p.geom.page_bytes + ((int64_t)(kh << (p.geom.page_shift - 4)) + (p.place(t) >> 4)) * kv_granule_bytes(D)) * 16 +
         (t & 15);
}

__device__ __forceinline__ int64_t of_lane(int64_t x, int lane) {
  const uint32_t lo = (uint32_t)__shfl((int)x, lane), hi = (uint32_t)__shfl((int)(x >> 32), lane);
  return (int64_t)((uint64_t)hi << 32 | lo);
}

// What a lane holds of its wave's 16 rows.  Rows are given by four lanes each, lanes 4 i to 4 i + 3 row i;
// every lane of the wave takes part.
template <int D>
struct Rows {
  static constexpr int VS = D / 64, PER = D / 16;  // loads of value scales; lanes a row in them
  uint32_t k[D / 32], ks;
  uint64_t v[4];
  uint8_t vs[VS];

  template <typename F>
  static __device__ __forceinline__ void parts(int64_t row, F f) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t x = of_lane(row, (4 * i + (lane >> 4)) * 4);
      const int r = (int)(x & 15);
      f(i, x, 9 * D + (r >> 2) * (2 * D) + (lane & 15) * (D / 8) + (r & 3) * (D / 32));
    }
  }
  template <typename F>
  static __device__ __forceinline__ void scales(int64_t row, F f) {
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int i = 0; i < VS; ++i) {
      const int64_t x = of_lane(row, (i * (64 / PER) + lane / PER) * 4);
      const int r = (int)(x & 15);
      f(i, x, 17 * D + (r >> 2) * (D / 4) + (lane % PER) * 4 + (r & 3));
    }
  }

  // rows `from` (all of them in the cache)
  __device__ __forceinline__ void load(const uint8_t* cache, int64_t from) {
    const int q = threadIdx.x & 3, r = (int)(from & 15);
    const uint8_t* const p = cache + (from >> 4);
    const uint8_t *kp = p + r * (D / 2) + q * (D / 8), *sp = p + 8 * D + r * (D / 16) + q * (D / 64);
    if constexpr (D == 64) {
      const u32x2 x = *reinterpret_cast<const u32x2*>(kp);
      k[0] = x[0];
      k[1] = x[1];
      ks = *sp;
    } else {
#pragma unroll
      for (int i = 0; i < D / 32; i += 4) {
        const u32x4 x = *reinterpret_cast<const u32x4*>(kp + 4 * i);
#pragma unroll
        for (int e = 0; e < 4; ++e) k[i + e] = x[e];
      }
      ks = D == 128 ? *reinterpret_cast<const uint16_t*>(sp) : *reinterpret_cast<const uint32_t*>(sp);
    }
    parts(from, [&](int i, int64_t x, int at) {
      const uint8_t* const vp = cache + (x >> 4) + at;
      if constexpr (D == 64) v[i] = *reinterpret_cast<const uint16_t*>(vp);
      else if constexpr (D == 128) v[i] = *reinterpret_cast<const uint32_t*>(vp);
      else v[i] = *reinterpret_cast<const uint64_t*>(vp);
    });
    scales(from, [&](int i, int64_t x, int at) { vs[i] = cache[(x >> 4) + at]; });
  }
  // to the rows `to` (-1: nowhere)
  __device__ __forceinline__ void store(uint8_t* cache, int64_t to) const {
    const int q = threadIdx.x & 3, r = (int)(to & 15);
    if (to >= 0) {
      uint8_t* const p = cache + (to >> 4);
      uint8_t *kp = p + r * (D / 2) + q * (D / 8), *sp = p + 8 * D + r * (D / 16) + q * (D / 64);
      if constexpr (D == 64) {
        *reinterpret_cast<u32x2*>(kp) = u32x2{k[0], k[1]};
        *sp = (uint8_t)ks;
      } else {
#pragma unroll
        for (int i = 0; i < D / 32; i += 4) *reinterpret_cast<u32x4*>(kp + 4 * i) = u32x4{k[i], k[i + 1], k[i + 2], k[i + 3]};
        if constexpr (D == 128) *reinterpret_cast<uint16_t*>(sp) = (uint16_t)ks;
        else *reinterpret_cast<uint32_t*>(sp) = ks;
      }
    }
    parts(to, [&](int i, int64_t x, int at) {
      if (x < 0) return;
      uint8_t* const vp = cache + (x >> 4) + at;
      if constexpr (D == 64) *reinterpret_cast<uint16_t*>(vp) = (uint16_t)v[i];
      else if constexpr (D == 128) *reinterpret_cast<uint32_t*>(vp) = (uint32_t)v[i];
      else *reinterpret_cast<uint64_t*>(vp) = v[i];
    });
    scales(to, [&](int i, int64_t x, int at) {
      if (x >= 0) cache[(x >> 4) + at] = vs[i];
    });
  }
};

// Accepted path: a workgroup per sequence, so that the sequence's length may be written where it was
// read.  The rows of whole heads, up to kRows at a time, are all read before any is written: a path's
// numbers need not increase.
static_assert(kKvMostAccepted <= kRows, "a head's rows at a time");

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
  const int row = threadIdx.x / 4;
  const int32_t heads = count > 0 ? kRows / count : hkv;              // at a time
  for (int32_t h0 = 0; count > 0 && h0 < hkv; h0 += heads) {
    const int32_t rows = (hkv - h0 < heads ? hkv - h0 : heads) * count, j = row < rows ? row : rows - 1;
    const bool busy = (row & ~(kWaveRows - 1)) < rows;                // the wave has rows
    Rows<D> x;
    int64_t to = -1;
    if (busy) {
      const int32_t h = j / count, p = j - h * count, at = c0 + p;
      const int32_t node = a.accepted[(int64_t)b * a.ld_accepted + p];
      const int32_t from = c0 + (node < 0 ? 0 : (node >= m ? m - 1 : node));
      const int32_t src = pages.of(from), dst = pages.of(at);
      const bool moves = row < rows && from != at && from >= 0 && at >= 0 && src >= 0 && dst >= 0;
      x.load(a.cache, row_at<D>(pages, src < 0 ? 0 : src, h0 + h, from));
      if (moves) to = row_at<D>(pages, dst, h0 + h, at);
    }
    __syncthreads();
    if (busy) x.store(a.cache, to);
  }
  __syncthreads();                                 // every thread has read the length
  if (threadIdx.x == 0) {
    const int32_t left = c0 + count;
    a.kv_len_out[b] = left < 0 ? 0 : (left > n ? n : left);
  }
}

// Eviction of a row: one kv head of one sequence.
//   the weights of the tokens [first, n - last) as 32-bit keys of the same order, the smallest
//   kept key by its digits (11, 11 and 10 bits, a histogram each), of the tokens that equal it the
//   lowest ones;
//   kept tokens behind the places of the kept (movers) and free places, ascending, to two lists;
//   mover i to free place i, then the last tokens down.
// A workgroup does a whole row of up to 16384 rated tokens, their keys in registers (and moves what moves, or another
// launch does where workgroups are few and that is much); where longer rows are
// announced, they are cut into parts, and each pass over the keys is a launch.  What bounds it: short rows by the latency of
// their steps, each of which waits for the one before (weights, three histograms, lists, rows: 32 x 8 heads
// of about 4130 tokens to 4096 17 us, of which reading the weights and moving about 290 rows a head take 6 at a
// copy's rate); long ones by that of six launches (2 x 8 heads of up to 131072 tokens to 16384 83 us, 38 of
// them before the move) and by the sectors of what moves: a row's bytes lie in 26 pieces at D = 128, and the
// move reads 106 MB for rows of 33, at 3.3 TB/s.
constexpr uint32_t kDigits[3] = {21, 10, 0};
constexpr int kBins = 2048;

// Larger weights have larger keys; a NaN counts as -inf, -0 as 0
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t x = __float_as_uint(w == 0.0f ? 0.0f : (w == w ? w : -__builtin_inff()));
  return x & 0x80000000u ? ~x : x | 0x80000000u;
}

// Sum over the lanes up to this one: within rows of 16, then the rows before
__device__ __forceinline__ int32_t sum_upto(int32_t x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, false);   // the lane 1, 2, 4, 8 before in the row
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, false);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);   // lane 15 (47) to the row after
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);   // lane 31 to the upper half
  return x;
}

// Sum over the threads before this one, and over all (every thread calls it)
__device__ __forceinline__ int32_t sum_before(int32_t x, int32_t* s_waves, int32_t& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int32_t upto = sum_upto(x);
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

// A row and what of it is kept
struct Row {
  Pages pages;
  int32_t kh, n, budget, first, last;
  bool over;
  int32_t left, rated, keep, behind;   // new length; tokens that are rated, and kept of them; places below the last tokens'

  __device__ __forceinline__ Row(const KvEvictArgs& a, int32_t row)
      : pages(pages_of(a.pages, row / a.pages.geom.n_kv_heads)), kh(row % a.pages.geom.n_kv_heads),
        n(length_of(a.pages, a.kv_len, row / a.pages.geom.n_kv_heads)), budget(a.budget), first(a.first), last(a.last),
        over(n > budget), left(over ? budget : n), rated(n - first - last), keep(budget - first - last),
        behind(budget - last) {}

  __device__ __forceinline__ uint32_t key(const KvEvictArgs& a, int32_t i) const {
    const int32_t page = pages.of(first + i);
    return page < 0 ? weight_key(-__builtin_inff()) : weight_key(a.weights[pages.weight_at(page, kh, first + i)]);
  }
};

// Calls f(i, key of rated token i) for i = begin + thread, + count, ... below end, eight tokens' loads side
// by side; COPY: and gives the weights of the tokens that may stay where they are to weights_out
template <bool COPY, typename F>
__device__ __forceinline__ void for_keys(const KvEvictArgs& a, const Row& x, int32_t begin, int32_t end, int32_t thread,
                                         int32_t count, F f) {
  constexpr int N = 8;
  const bool copy = COPY && a.weights_out && a.weights_out != a.weights;
  for (int32_t i0 = begin + thread; i0 < end; i0 += N * count) {
    int64_t at[N];
    float w[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int32_t i = i0 + e * count, t = x.first + (i < end ? i : i0);
      const int32_t page = x.pages.of(t);
      at[e] = page < 0 ? -1 : x.pages.weight_at(page, x.kh, t);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = a.weights[at[e] < 0 ? 0 : at[e]];
#pragma unroll
    for (int e = 0; e < N; ++e) w[e] = at[e] < 0 ? -__builtin_inff() : w[e];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      const int32_t i = i0 + e * count;
      if (i >= end) break;
      if (copy && x.first + i < x.behind && at[e] >= 0) a.weights_out[at[e]] = w[e];
      f(i, weight_key(w[e]));
    }
  }
}

// What does not move, but for the rated tokens' weights (for_keys): `count` threads of a row share it
__device__ __forceinline__ void keep_places(const KvEvictArgs& a, const Row& x, int32_t row, int32_t thread, int32_t count) {
  const int32_t stay = x.over ? x.behind : x.left;
  if (a.kept)
    for (int32_t j = thread; j < (x.over ? x.behind : a.budget); j += count)
      a.kept[(int64_t)row * a.budget + j] = j < stay ? j : -1;
  if (a.weights_out && a.weights_out != a.weights)
    for (int32_t j = thread; j < (x.over ? x.first : x.left); j += count) {
      const int32_t page = x.pages.of(j);
      if (page >= 0) {
        const int64_t at = x.pages.weight_at(page, x.kh, j);
        a.weights_out[at] = a.weights[at];
      }
    }
  if (a.lengths && x.kh == 0 && thread == 0) a.kv_len_out[row / a.pages.geom.n_kv_heads] = x.left;
}

// The digit in which `wanted` keys, from the largest digit on, are reached; `mine`: this thread's
// two bins, kBins - 1 - 2 tid and the one below.  Writes {digit, those wanted of its keys, its keys}.
__device__ __forceinline__ void find_digit(int32_t x, int32_t y, int32_t wanted, int32_t* s_waves, int32_t* s_found) {
  int32_t all;
  const int32_t before = sum_before(x + y, s_waves, all);
  if (before < wanted && wanted <= before + x + y) {
    const bool upper = wanted <= before + x;
    s_found[0] = kBins - 1 - 2 * (int)threadIdx.x - (upper ? 0 : 1);
    s_found[1] = wanted - before - (upper ? 0 : x);
    s_found[2] = upper ? x : y;
  }
  __syncthreads();
}

// Walks the rated tokens [r0, r1) of a wave in order, `ties` tokens of the border's key before them, and
// calls f(token, whether it moves, its number among the movers, whether its place is free, its
// number among those) for 64 at a time
template <typename K, typename F>
__device__ __forceinline__ void walk(const Row& x, int32_t r0, int32_t r1, uint32_t border, int32_t wanted, int32_t ties, K key_of,
                                     int32_t& movers, int32_t& gaps, F f) {
  const int lane = threadIdx.x & 63;
  const uint64_t below = (1ull << lane) - 1;
  for (int32_t i = r0; i < r1; i += 64) {
    const bool have = i + lane < r1;
    const uint32_t k = have ? key_of(i + lane) : 0;
    const bool tie = have && x.keep > 0 && k == border;
    const uint64_t tie_lanes = __builtin_amdgcn_ballot_w64(tie);
    const bool stays = have && x.keep > 0 &&
                       (k > border || (tie && ties + __builtin_popcountll(tie_lanes & below) < wanted));
    ties += __builtin_popcountll(tie_lanes);
    const int32_t t = x.first + i + lane;
    const bool moves = stays && t >= x.behind, gap = have && !stays && t < x.behind;
    const uint64_t mv = __builtin_amdgcn_ballot_w64(moves), gp = __builtin_amdgcn_ballot_w64(gap);
    f(t, moves, movers + __builtin_popcountll(mv & below), gap, gaps + __builtin_popcountll(gp & below));
    movers += __builtin_popcountll(mv);
    gaps += __builtin_popcountll(gp);
  }
}

// 16 N rows of a wave on their way
template <int D, int N>
struct Moving {
  Rows<D> x[N];
  int64_t to[N], w_at[N];
  float w[N];

  // rows e: token old[e] to place[e], where live[e]; none from rows `some` on is (the same number for the wave)
  __device__ __forceinline__ void read(const KvEvictArgs& a, const Row& row, int32_t* kept, const int32_t (&old)[N],
                                       const int32_t (&place)[N], const bool (&live)[N], int some) {
    int32_t src[N], dst[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
      src[e] = dst[e] = 0;
      to[e] = -1;
      if (e >= some) continue;
      src[e] = row.pages.of(old[e]);
      dst[e] = row.pages.of(place[e]);
    }
#pragma unroll
    for (int e = 0; e < N; ++e) {
      if (e >= some) continue;
      const bool moves = live[e] && src[e] >= 0 && dst[e] >= 0;
      const int32_t from = src[e] < 0 ? 0 : src[e];
      x[e].load(a.cache, row_at<D>(row.pages, from, row.kh, old[e]));
      w[e] = a.weights[row.pages.weight_at(from, row.kh, old[e])];
      if (moves) {
        to[e] = row_at<D>(row.pages, dst[e], row.kh, place[e]);
        w_at[e] = row.pages.weight_at(dst[e], row.kh, place[e]);
      }
      // a row that does not move leaves the place as it is
      if (kept && live[e] && (threadIdx.x & 3) == 0) kept[place[e]] = moves ? old[e] : place[e];
    }
  }
  __device__ __forceinline__ void write(const KvEvictArgs& a) const {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (__builtin_amdgcn_ballot_w64(to[e] >= 0)) {
        x[e].store(a.cache, to[e]);
        if (a.weights_out && to[e] >= 0 && (threadIdx.x & 3) == 0) a.weights_out[w_at[e]] = w[e];
      }
  }
};

// The last tokens down by n - budget, kRows at a time from j0 on, in order where old and new places
// overlap: what they overwrite was read with them or before.

// how many of N groups of rows, `side` apart, a wave has where `left` rows are left for its workgroup
__device__ __forceinline__ int groups_of(int32_t left, int side) {
  const int32_t own = left - (int32_t)(threadIdx.x >> 6) * kWaveRows;
  return __builtin_amdgcn_readfirstlane(own <= 0 ? 0 : (own + side - 1) / side);
}

template <int D, int N>
__device__ __forceinline__ void read_last(const KvEvictArgs& a, const Row& x, int32_t* kept, int32_t j0, int32_t rows,
                                          Moving<D, N>& h) {
  int32_t old[N], place[N];
  bool live[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int32_t j = j0 + e * rows + (int32_t)threadIdx.x / 4;
    live[e] = j < x.last;
    old[e] = live[e] ? x.n - x.last + j : x.n - 1;
    place[e] = live[e] ? x.behind + j : 0;
  }
  h.read(a, x, kept, old, place, live, groups_of(x.last - j0, rows));
}

// Rows i0 + thread / 4, + side, ... of the lists (N of them, those below `moving`)
template <int D, int N>
__device__ __forceinline__ void read_listed(const KvEvictArgs& a, const Row& x, int32_t* kept, const int32_t* from, const int32_t* to,
                                            int32_t i0, int side, int32_t moving, Moving<D, N>& m) {
  int32_t old[N], place[N];
  bool live[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    const int32_t i = i0 + e * side + (int32_t)threadIdx.x / 4;
    live[e] = i < moving;
    old[e] = from[live[e] ? i : i0];
    place[e] = to[live[e] ? i : i0];
  }
  m.read(a, x, kept, old, place, live, groups_of(moving - i0, side));
}

// Movers stand behind every free place: nothing that is read here is written
template <int D>
__device__ __forceinline__ void move_listed(const KvEvictArgs& a, const Row& x, int32_t* kept, const int32_t* from,
                                            const int32_t* to, int32_t moving) {
  for (int32_t i0 = 0; i0 < moving; i0 += kRows) {
    Moving<D, 1> m;
    read_listed<D, 1>(a, x, kept, from, to, i0, kRows, moving, m);
    m.write(a);
  }
}

// The last tokens, their first chunk read already
template <int D>
__device__ __forceinline__ void move_last(const KvEvictArgs& a, const Row& x, int32_t* kept, Moving<D, 1>& tail) {
  __syncthreads();                                 // the movers are read
  tail.write(a);
  for (int32_t j0 = kRows; j0 < x.last; j0 += kRows) {
    read_last<D, 1>(a, x, kept, j0, kRows, tail);
    __syncthreads();
    tail.write(a);
  }
}

// A whole row of any length, longer than the bound announced: its keys are read again and again.
// s_hist [kBins]: the histograms.  APART: what moves is listed, and moved by k_kv_evict_move
template <int D, bool APART>
__device__ __forceinline__ void evict_row(const KvEvictArgs& a, const Row& x, int32_t* s_hist, int32_t* s_waves, int32_t* s_found) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int32_t* const kept = a.kept ? a.kept + (int64_t)blockIdx.x * a.budget : nullptr;
  auto key_of = [&](int32_t i) { return x.key(a, i); };
  for_keys<true>(a, x, 0, x.rated, tid, kThreads, [](int32_t, uint32_t) {});
  // the last tokens' first chunk, on its way while the others are chosen
  Moving<D, 1> tail;
  if constexpr (!APART) read_last<D, 1>(a, x, kept, 0, kRows, tail);
  keep_places(a, x, blockIdx.x, tid, kThreads);

  // the smallest kept key, and how many tokens of it are kept
  uint32_t border = 0, known = 0;
  int32_t wanted = x.keep, equal = 0;
  for (int pass = 0; x.keep > 0 && pass < 3; ++pass) {
    const uint32_t shift = kDigits[pass], mask = pass < 2 ? kBins - 1 : (kBins >> 1) - 1;
    for (int i = tid; i < kBins; i += kThreads) s_hist[i] = 0;
    __syncthreads();
    for (int32_t i = tid; i < x.rated; i += kThreads) {
      const uint32_t k = key_of(i);
      if ((k & known) == border) atomicAdd(&s_hist[(k >> shift) & mask], 1);
    }
    __syncthreads();
    find_digit(s_hist[kBins - 1 - 2 * tid], s_hist[kBins - 2 - 2 * tid], wanted, s_waves, s_found);
    border |= (uint32_t)s_found[0] << shift;
    known |= mask << shift;
    wanted = s_found[1];
    equal = s_found[2];
  }

  // each wave a run of tokens, in order
  const int32_t run = ((x.rated + kWaves - 1) / kWaves + 63) & ~63;
  const int32_t r0 = wave * run < x.rated ? wave * run : x.rated, r1 = r0 + run < x.rated ? r0 + run : x.rated;
  int32_t ties0 = 0;                               // tokens of the border's key before this wave's run
  if (x.keep > 0 && equal > wanted) {
    int32_t ties = 0, all;
    for (int32_t i = r0 + lane; i < r1; i += 64) ties += key_of(i) == border;
    ties0 = __builtin_amdgcn_readfirstlane(sum_before(ties, s_waves, all));   // what the first lane has before it
  }
  int32_t movers = 0, gaps = 0, moving, all;
  walk(x, r0, r1, border, wanted, ties0, key_of, movers, gaps, [](int32_t, bool, int32_t, bool, int32_t) {});
  movers = __builtin_amdgcn_readfirstlane(sum_before(lane == 0 ? movers : 0, s_waves, moving));
  gaps = __builtin_amdgcn_readfirstlane(sum_before(lane == 0 ? gaps : 0, s_waves, all));
  int32_t* const from = a.lists + (int64_t)blockIdx.x * 2 * a.budget;
  int32_t* const to = from + a.budget;
  walk(x, r0, r1, border, wanted, ties0, key_of, movers, gaps, [&](int32_t t, bool moves, int32_t i, bool gap, int32_t j) {
    if (moves) from[i] = t;
    if (gap) to[j] = t;
  });
  if constexpr (APART) {
    if (tid == 0) a.moving[blockIdx.x] = moving;
  } else {
    __syncthreads();
    move_listed<D>(a, x, kept, from, to, moving);
    move_last<D>(a, x, kept, tail);
  }
}

// A run of rated tokens whose keys a wave holds, token r0 + 64 e + lane in key[e] (below `end`)
template <int KEYS>
struct Run {
  int32_t r0, end;             // r0: the lane's
  uint32_t key[KEYS];
  uint64_t moves[KEYS], gaps[KEYS];   // lanes whose token moves, or whose place is free

  __device__ __forceinline__ Run(int32_t begin, int32_t upto) {
    const int32_t wave = (int32_t)(threadIdx.x >> 6), run = ((upto - begin + kWaves - 1) / kWaves + 63) & ~63;
    const int32_t first = begin + wave * run;
    r0 = first + (int32_t)(threadIdx.x & 63);
    end = first + run < upto ? first + run : upto;
  }
  __device__ __forceinline__ bool have(int e) const { return r0 + 64 * e < end; }

  // COPY: weights of tokens that may stay where they are go to weights_out
  template <bool COPY>
  __device__ __forceinline__ void load(const KvEvictArgs& a, const Row& x) {
    const bool copy = COPY && a.weights_out && a.weights_out != a.weights;
    constexpr int N = KEYS < 8 ? KEYS : 8;         // tokens whose loads are side by side
#pragma unroll
    for (int e0 = 0; e0 < KEYS; e0 += N) {
      int64_t at[N];
      float w[N];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const int32_t t = have(e0 + e) ? x.first + r0 + 64 * (e0 + e) : x.first;
        const int32_t page = x.pages.of(t);
        at[e] = page < 0 ? -1 : x.pages.weight_at(page, x.kh, t);
      }
#pragma unroll
      for (int e = 0; e < N; ++e) w[e] = a.weights[at[e] < 0 ? 0 : at[e]];
#pragma unroll
      for (int e = 0; e < N; ++e) {
        w[e] = at[e] < 0 ? -__builtin_inff() : w[e];
        if (copy && have(e0 + e) && at[e] >= 0 && x.first + r0 + 64 * (e0 + e) < x.behind) a.weights_out[at[e]] = w[e];
        key[e0 + e] = weight_key(w[e]);
      }
    }
  }
  // the wave's tokens of this key
  __device__ __forceinline__ int32_t equal(uint32_t border) const {
    int32_t n = 0;
#pragma unroll
    for (int e = 0; e < KEYS; ++e) n += __builtin_popcountll(__builtin_amdgcn_ballot_w64(have(e) && key[e] == border));
    return n;
  }
  // which tokens move and whose places are free, `ties` tokens of the border's key before the run; how many
  __device__ __forceinline__ void choose(const Row& x, uint32_t border, int32_t wanted, int32_t ties, int32_t& n_moves, int32_t& n_gaps) {
    const uint64_t below = (1ull << (threadIdx.x & 63)) - 1;
    n_moves = n_gaps = 0;
#pragma unroll
    for (int e = 0; e < KEYS; ++e) {
      const bool tie = have(e) && x.keep > 0 && key[e] == border;
      const uint64_t tie_lanes = __builtin_amdgcn_ballot_w64(tie);
      const bool stays = have(e) && x.keep > 0 &&
                         (key[e] > border || (tie && ties + __builtin_popcountll(tie_lanes & below) < wanted));
      ties += __builtin_popcountll(tie_lanes);
      const int32_t t = x.first + r0 + 64 * e;
      moves[e] = __builtin_amdgcn_ballot_w64(stays && t >= x.behind);
      gaps[e] = __builtin_amdgcn_ballot_w64(have(e) && !stays && t < x.behind);
      n_moves += __builtin_popcountll(moves[e]);
      n_gaps += __builtin_popcountll(gaps[e]);
    }
  }
  // to the lists, the wave's from numbers i and j on
  __device__ __forceinline__ void list(const Row& x, int32_t* from, int32_t* to, int32_t i, int32_t j) const {
    const int lane = threadIdx.x & 63;
    const uint64_t below = (1ull << lane) - 1;
#pragma unroll
    for (int e = 0; e < KEYS; ++e) {
      const int32_t t = x.first + r0 + 64 * e;
      if (moves[e] >> lane & 1) from[i + __builtin_popcountll(moves[e] & below)] = t;
      if (gaps[e] >> lane & 1) to[j + __builtin_popcountll(gaps[e] & below)] = t;
      i += __builtin_popcountll(moves[e]);
      j += __builtin_popcountll(gaps[e]);
    }
  }
};

// Of a number that each wave has, those of the waves before this one, and of all (every thread calls it)
__device__ __forceinline__ uint32_t waves_before(uint32_t x, int32_t* s_waves, uint32_t& all) {
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) s_waves[wave] = (int32_t)x;
  __syncthreads();
  uint32_t before = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    before += w < wave ? (uint32_t)s_waves[w] : 0;
    all += (uint32_t)s_waves[w];
  }
  return before;
}

// A whole row of up to kThreads * KEYS rated tokens, whose keys stay in registers: each wave has a run of
// tokens, 64 at a time.  (Rows that the bound did not announce are longer: evict_row.)  APART: as there
template <int D, int KEYS, bool APART>
__global__ __launch_bounds__(kThreads) void k_kv_evict_held(KvEvictArgs a) {
  __shared__ int32_t s_hist[3][kBins];             // and the lists, where they are short
  __shared__ int32_t s_waves[2][kWaves], s_scan[3][kWaves];
  __shared__ int32_t s_found[3][3];
  constexpr int kListed = 3 * kBins / 2;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Row x(a, blockIdx.x);
  if (!x.over) {
    keep_places(a, x, blockIdx.x, tid, kThreads);
    return;
  }
  if (x.rated > KEYS * kThreads) {
    evict_row<D, APART>(a, x, s_hist[0], s_waves[0], s_found[0]);
    return;
  }
  int32_t* const kept = a.kept ? a.kept + (int64_t)blockIdx.x * a.budget : nullptr;
  Run<KEYS> run(0, x.rated);
  run.template load<true>(a, x);
  // the last tokens' first chunk, on its way while the others are chosen
  Moving<D, 1> tail;
  if constexpr (!APART) read_last<D, 1>(a, x, kept, 0, kRows, tail);
  keep_places(a, x, blockIdx.x, tid, kThreads);
  for (int i = tid; i < 3 * kBins; i += kThreads) s_hist[0][i] = 0;
  __syncthreads();

  // the smallest kept key, and how many tokens of it are kept
  uint32_t border = 0;
  int32_t wanted = x.keep, equal = 0;
  if (x.keep > 0) {
#pragma unroll
    for (int pass = 0; pass < 3; ++pass) {
      const uint32_t shift = kDigits[pass], mask = pass < 2 ? kBins - 1 : (kBins >> 1) - 1, above = shift + (pass < 2 ? 11 : 10);
#pragma unroll
      for (int e = 0; e < KEYS; ++e)
        if (run.have(e) && (pass == 0 || run.key[e] >> above == border >> above))
          atomicAdd(&s_hist[pass][(run.key[e] >> shift) & mask], 1);
      __syncthreads();
      // bins from the largest digit on, two a thread
      const int32_t lo = s_hist[pass][kBins - 2 - 2 * tid], hi = s_hist[pass][kBins - 1 - 2 * tid];
      const int32_t upto = sum_upto(hi + lo);
      if (lane == 63) s_scan[pass][wave] = upto;
      __syncthreads();
      int32_t before = upto - hi - lo;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) before += w < wave ? s_scan[pass][w] : 0;
      if (before < wanted && wanted <= before + hi + lo) {
        const bool upper = wanted <= before + hi;
        s_found[pass][0] = kBins - 1 - 2 * tid - (upper ? 0 : 1);
        s_found[pass][1] = wanted - before - (upper ? 0 : hi);
        s_found[pass][2] = upper ? hi : lo;
      }
      __syncthreads();
      border |= (uint32_t)s_found[pass][0] << shift;
      wanted = s_found[pass][1];
      equal = s_found[pass][2];
    }
  }

  // tokens of the border's key before this wave's run
  uint32_t ties = 0, all;
  if (x.keep > 0 && equal > wanted) ties = waves_before((uint32_t)run.equal(border), s_waves[0], all);
  int32_t movers, gaps;
  run.choose(x, border, wanted, (int32_t)ties, movers, gaps);
  // both are at most kThreads KEYS < 2^16
  const uint32_t before = waves_before((uint32_t)movers << 16 | (uint32_t)gaps, s_waves[1], all);
  const int32_t moving = (int32_t)(all >> 16);
  const bool listed = !APART && moving <= kListed;
  int32_t* const from = listed ? s_hist[0] : a.lists + (int64_t)blockIdx.x * 2 * a.budget;
  int32_t* const to = from + (listed ? kListed : a.budget);
  run.list(x, from, to, (int32_t)(before >> 16), (int32_t)(before & 0xFFFF));
  if constexpr (APART) {
    if (tid == 0) a.moving[blockIdx.x] = moving;
  } else {
    __syncthreads();
    move_listed<D>(a, x, kept, from, to, moving);
    move_last<D>(a, x, kept, tail);
  }
}

// Longer rows in parts: row blockIdx / parts, part blockIdx % parts, of equal runs of the row's rated
// tokens.  Parts add their histograms up; each pass over the keys is a launch.
struct Parts {
  int32_t row, part;
  __device__ __forceinline__ Parts(const KvEvictArgs& a, int32_t block) : row(block / a.parts), part(block % a.parts) {}
  __device__ __forceinline__ int32_t begin(const KvEvictArgs& a, const Row& x, int32_t p) const {
    const int32_t size = ((x.rated + a.parts - 1) / a.parts + kThreads - 1) / kThreads * kThreads;
    const int64_t at = (int64_t)p * size;
    return at < x.rated ? (int32_t)at : x.rated;
  }
};
struct RowCounts {
  int32_t digit[2][kBins], last[kBins / 2];        // the histograms
  // after each launch: the border's digits so far, the tokens wanted of those that have them
  struct {
    uint32_t border;
    int32_t wanted;
  } found[2];
};
// of a part's tokens on kept places (0) and behind them (1): those whose key is at least the border's first two
// digits and third digit i
struct PartCounts {
  int32_t least[2][kBins / 2 + 4];
};
static_assert(sizeof(RowCounts) <= kKvEvictRowBytes && sizeof(PartCounts) <= kKvEvictPartBytes, "kv_launch.hpp");
__device__ __forceinline__ RowCounts* row_counts(const KvEvictArgs& a, int32_t row) {
  return reinterpret_cast<RowCounts*>(static_cast<uint8_t*>(a.counts) + (int64_t)row * kKvEvictRowBytes);
}
__device__ __forceinline__ PartCounts* part_counts(const KvEvictArgs& a, int32_t row, int32_t part) {
  return reinterpret_cast<PartCounts*>(static_cast<uint8_t*>(a.counts) + (int64_t)a.rows * kKvEvictRowBytes +
                                       ((int64_t)row * a.parts + part) * kKvEvictPartBytes);
}

__global__ __launch_bounds__(256) void k_kv_evict_clear(KvEvictArgs a) {
  u32x4* const p = reinterpret_cast<u32x4*>(row_counts(a, blockIdx.x));
  for (int i = threadIdx.x; i < kKvEvictRowBytes / 16; i += 256) p[i] = u32x4{0, 0, 0, 0};
}

// Histogram PASS of a part's keys, those whose digits before are the border's
template <int PASS>
__global__ __launch_bounds__(kThreads) void k_kv_evict_digits(KvEvictArgs a) {
  __shared__ int32_t s_hist[kBins];
  __shared__ int32_t s_waves[kWaves];
  __shared__ int32_t s_found[3];
  __shared__ int32_t s_larger[2], s_near;
  const int tid = threadIdx.x;
  const Parts p(a, blockIdx.x);
  const Row x(a, p.row);
  if constexpr (PASS == 0) keep_places(a, x, p.row, p.part * kThreads + tid, a.parts * kThreads);
  if (!x.over || (PASS > 0 && x.keep == 0)) return;   // the first one copies weights
  RowCounts* const c = row_counts(a, p.row);
  for (int i = tid; i < kBins; i += kThreads) s_hist[i] = 0;
  if (tid < 2) s_larger[tid] = 0;
  uint32_t border = 0;
  if constexpr (PASS > 0) {
    int32_t wanted = x.keep;
    if constexpr (PASS == 2) {
      border = c->found[0].border;
      wanted = c->found[0].wanted;
    }
    const int2 bins = *reinterpret_cast<const int2*>(&c->digit[PASS - 1][kBins - 2 - 2 * tid]);
    find_digit(bins.y, bins.x, wanted, s_waves, s_found);
    border |= (uint32_t)s_found[0] << kDigits[PASS - 1];
    if (p.part == 0 && tid == 0) {
      c->found[PASS - 1].border = border;
      c->found[PASS - 1].wanted = s_found[1];
    }
  }
  __syncthreads();
  const int32_t r0 = p.begin(a, x, p.part), r1 = p.begin(a, x, p.part + 1);
  int32_t larger[2] = {0, 0};
  for_keys<PASS == 0>(a, x, r0, r1, tid, kThreads, [&](int32_t i, uint32_t k) {
    if constexpr (PASS == 0) {
      atomicAdd(&s_hist[k >> 21], 1);
    } else if constexpr (PASS == 1) {
      if (k >> 21 == border >> 21) atomicAdd(&s_hist[(k >> 10) & (kBins - 1)], 1);
    } else {
      const int behind = x.first + i >= x.behind;
      if (k >> 10 == border >> 10) atomicAdd(&s_hist[behind * (kBins / 2) + (k & (kBins / 2 - 1))], 1);
      else if (k >> 10 > border >> 10) ++larger[behind];
    }
  });
  if constexpr (PASS == 2) {
    if (larger[0]) atomicAdd(&s_larger[0], larger[0]);
    if (larger[1]) atomicAdd(&s_larger[1], larger[1]);
  }
  __syncthreads();
  if constexpr (PASS < 2) {
    for (int i = tid; i < kBins; i += kThreads)
      if (s_hist[i]) atomicAdd(&c->digit[PASS][i], s_hist[i]);
  } else {
    static_assert(kThreads == kBins / 2, "a thread per digit, and two digits of one half a thread");
    const int32_t both = s_hist[tid] + s_hist[kBins / 2 + tid];
    if (both) atomicAdd(&c->last[tid], both);
    const int z = tid >> 9, at = kBins / 2 - 2 - 2 * (tid & 511);
    const int32_t lo = s_hist[z * (kBins / 2) + at], hi = s_hist[z * (kBins / 2) + at + 1];
    int32_t all;
    int32_t before = sum_before(lo + hi, s_waves, all);
    if (tid == kThreads / 2) s_near = before;
    __syncthreads();
    before += s_larger[z] - (z ? s_near : 0);
    PartCounts* const out = part_counts(a, p.row, p.part);
    out->least[z][at + 1] = before + hi;
    out->least[z][at] = before + hi + lo;
    if (at + 2 == kBins / 2) out->least[z][kBins / 2] = before;
  }
}

// The lists
__global__ __launch_bounds__(kThreads) void k_kv_evict_lists(KvEvictArgs a) {
  constexpr int KEYS = 8;                              // of a thread, where a part is as long as was announced
  __shared__ int32_t s_waves[3][kWaves];
  __shared__ int32_t s_found[3];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const Parts p(a, blockIdx.x);
  const Row x(a, p.row);
  if (!x.over) return;
  const int32_t r0 = p.begin(a, x, p.part), r1 = p.begin(a, x, p.part + 1);
  const bool held = r1 - r0 <= KEYS * kThreads;
  Run<KEYS> run(r0, r1);
  if (held) run.template load<false>(a, x);
  RowCounts* const c = row_counts(a, p.row);
  uint32_t border = 0;
  int32_t wanted = 0, larger[2] = {0, 0}, equal[2] = {0, 0};
  static_assert(kKvEvictMostParts <= 64, "a lane counts a part");
  if (x.keep > 0) {
    // the third digit has half the bins: threads from kBins / 4 on
    int2 bins = {0, 0};
    if (tid >= kBins / 4) bins = *reinterpret_cast<const int2*>(&c->last[kBins - 2 - 2 * tid]);
    find_digit(bins.y, bins.x, c->found[1].wanted, s_waves[0], s_found);
    const int32_t digit = s_found[0];
    border = c->found[1].border | (uint32_t)digit;
    wanted = s_found[1];
    const PartCounts* const q = part_counts(a, p.row, lane < a.parts ? lane : 0);
#pragma unroll
    for (int z = 0; z < 2; ++z) {
      const int32_t from = q->least[z][digit], more = q->least[z][digit + 1];
      larger[z] = lane < a.parts ? more : 0;
      equal[z] = lane < a.parts ? from - more : 0;
    }
  }
  // What stands before this part, and in all: lane q counts part q.  Of its ties, in order, those that are
  // still wanted stay.
  const int32_t q0 = p.begin(a, x, lane < a.parts ? lane : a.parts), q1 = p.begin(a, x, lane < a.parts ? lane + 1 : a.parts);
  int32_t near = x.behind - x.first - q0;              // its tokens on kept ones' places
  near = near < 0 ? 0 : (near > q1 - q0 ? q1 - q0 : near);
  const int32_t ties_before = sum_upto(equal[0] + equal[1]) - equal[0] - equal[1];
  const int32_t open = wanted - ties_before < 0 ? 0 : wanted - ties_before;
  const int32_t stay0 = equal[0] < open ? equal[0] : open, stay1 = equal[1] < open - stay0 ? equal[1] : open - stay0;
  const int32_t moves = larger[1] + stay1, free_ = near - larger[0] - stay0;
  const int32_t moves_upto = sum_upto(moves), free_upto = sum_upto(free_);
  if (p.part == 0 && tid == 63) a.moving[p.row] = moves_upto;
  const int32_t movers = __builtin_amdgcn_readlane(moves_upto - moves, p.part);
  const int32_t gaps = __builtin_amdgcn_readlane(free_upto - free_, p.part);
  int32_t ties = __builtin_amdgcn_readlane(ties_before, p.part);
  const bool tied = __builtin_amdgcn_readlane(equal[0] + equal[1], p.part) > 0;

  int32_t* const from = a.lists + (int64_t)p.row * 2 * a.budget;
  int32_t* const to = from + a.budget;
  uint32_t all;
  if (held) {
    if (tied) ties += (int32_t)waves_before((uint32_t)run.equal(border), s_waves[1], all);
    int32_t m, g;
    run.choose(x, border, wanted, ties, m, g);
    const uint32_t before = waves_before((uint32_t)m << 16 | (uint32_t)g, s_waves[2], all);
    run.list(x, from, to, movers + (int32_t)(before >> 16), gaps + (int32_t)(before & 0xFFFF));
    return;
  }
  auto key_of = [&](int32_t i) { return x.key(a, i); };
  const int32_t size = ((r1 - r0 + kWaves - 1) / kWaves + 63) & ~63;
  const int32_t w0 = r0 + wave * size < r1 ? r0 + wave * size : r1, w1 = w0 + size < r1 ? w0 + size : r1;
  int32_t own = 0, m = 0, g = 0;
  for (int32_t i = w0 + lane; i < w1; i += 64) own += x.keep > 0 && key_of(i) == border;
  ties += __builtin_amdgcn_readfirstlane(sum_before(own, s_waves[0], own));
  walk(x, w0, w1, border, wanted, ties, key_of, m, g, [](int32_t, bool, int32_t, bool, int32_t) {});
  int32_t sum;
  m = movers + __builtin_amdgcn_readfirstlane(sum_before(lane == 0 ? m : 0, s_waves[0], sum));
  g = gaps + __builtin_amdgcn_readfirstlane(sum_before(lane == 0 ? g : 0, s_waves[0], sum));
  walk(x, w0, w1, border, wanted, ties, key_of, m, g, [&](int32_t t, bool mv, int32_t i, bool gap, int32_t j) {
    if (mv) from[i] = t;
    if (gap) to[j] = t;
  });
}

// Movers, and the last tokens.  The last tokens' new places may hold movers, those below the budget: first
// in the list.  Where old and new places of the last tokens do not overlap, they go in chunks of 64, and the
// workgroup of a chunk moves the movers of its new places before; else the first workgroup moves all of
// these in order, 128 at a time (8 heads of 50000 to 49900, the last 1024: 64 at a time 81 us, 128 71).
constexpr int kMoveThreads = 256, kMoveRows = kMoveThreads / 4, kMoveDeep = 2;

// How many of the movers, which ascend, are below token t: a lane looks at every 64th part of what is left, as
// each look waits for memory (one lane's search, of 14 looks: 2 x 8 heads of up to 131072 87 us, not 83)
__device__ __forceinline__ int32_t movers_below(const int32_t* from, int32_t moving, int32_t t) {
  int32_t lo = 0, left = moving;                     // `lo` of them are, and of the `left` next ones some
  while (left > 0) {
    const int32_t part = (left + 63) >> 6, i = (int32_t)(threadIdx.x & 63) * part;
    // the first of each part
    const bool below = i < left && from[lo + (i < left ? i : 0)] < t;
    const int32_t parts = __builtin_popcountll(__builtin_amdgcn_ballot_w64(below));
    if (parts == 0) break;
    const int32_t skip = (parts - 1) * part + 1;     // the last such one, too
    lo += skip;
    left = part - 1 < left - skip ? part - 1 : left - skip;
  }
  return lo;
}

template <int D>
__global__ __launch_bounds__(kMoveThreads) void k_kv_evict_move(KvEvictArgs a) {
  const Parts p(a, blockIdx.x);
  const Row x(a, p.row);
  if (!x.over) return;
  int32_t* const kept = a.kept ? a.kept + (int64_t)p.row * a.budget : nullptr;
  const int32_t* const from = a.lists + (int64_t)p.row * 2 * a.budget;
  const int32_t* const to = from + a.budget;
  const int32_t moving = a.moving[p.row];
  const bool overlap = x.n - x.budget < x.last;
  auto movers = [&](int32_t i0, int32_t i1, int32_t step) __attribute__((always_inline)) {
    for (; i0 < i1; i0 += step) {
      Moving<D, kMoveDeep> m;
      read_listed<D, kMoveDeep>(a, x, kept, from, to, i0, kMoveRows, i1, m);
      m.write(a);
    }
  };
  auto last = [&](auto deep, int32_t j0, int32_t step) __attribute__((always_inline)) {
    constexpr int N = decltype(deep)::value;
    for (; j0 < x.last; j0 += step) {
      const int32_t place = x.behind + j0, end = place + kMoveRows * N < x.budget ? place + kMoveRows * N : x.budget;
      movers(movers_below(from, moving, place), movers_below(from, moving, end), kMoveRows * kMoveDeep);
      Moving<D, N> m;
      read_last<D, N>(a, x, kept, j0, kMoveRows, m);
      __syncthreads();                             // these movers and tokens are read
      m.write(a);
    }
  };
  if (!overlap) last(std::integral_constant<int, 1>{}, p.part * kMoveRows, a.parts * kMoveRows);
  else if (p.part == 0) last(std::integral_constant<int, kMoveDeep>{}, 0, kMoveRows * kMoveDeep);
  const int32_t rest = movers_below(from, moving, x.budget);
  movers(rest + p.part * kMoveRows * kMoveDeep, moving, a.parts * kMoveRows * kMoveDeep);
}

// The lengths, where they are written over those that the workgroups read
__global__ __launch_bounds__(256) void k_kv_lengths(KvEvictArgs a) {
  const int b = (int)blockIdx.x * 256 + threadIdx.x;
  if (b >= a.pages.batch) return;
  const int32_t n = length_of(a.pages, a.kv_len, b);
  a.kv_len_out[b] = n < a.budget ? n : a.budget;
}

template <int D, bool APART>
void evict_held(const KvEvictArgs& a, bool short_rows, hipStream_t s) {
  const dim3 rows((unsigned)a.rows), threads(kThreads);
  if (short_rows) hipLaunchKernelGGL((k_kv_evict_held<D, 4, APART>), rows, threads, 0, s, a);
  else hipLaunchKernelGGL((k_kv_evict_held<D, 16, APART>), rows, threads, 0, s, a);
}

template <int D>
hipError_t evict(KvEvictArgs a, bool short_rows, hipStream_t s) {
  if (a.parts == 0 && a.move_parts == 0) {
    evict_held<D, false>(a, short_rows, s);
    return hipGetLastError();
  }
  if (a.parts == 0) {
    evict_held<D, true>(a, short_rows, s);
  } else {
    const dim3 rows((unsigned)a.rows), parts((unsigned)(a.rows * a.parts)), threads(kThreads);
    hipLaunchKernelGGL(k_kv_evict_clear, rows, dim3(256), 0, s, a);
    hipLaunchKernelGGL((k_kv_evict_digits<0>), parts, threads, 0, s, a);
    hipLaunchKernelGGL((k_kv_evict_digits<1>), parts, threads, 0, s, a);
    hipLaunchKernelGGL((k_kv_evict_digits<2>), parts, threads, 0, s, a);
    hipLaunchKernelGGL(k_kv_evict_lists, parts, threads, 0, s, a);
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  KvEvictArgs m = a;
  m.parts = a.move_parts;
  hipLaunchKernelGGL((k_kv_evict_move<D>), dim3((unsigned)(m.rows * m.parts)), dim3(kMoveThreads), 0, s, m);
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

KvEvictPlan kv_evict_plan(int32_t batch, int32_t n_kv_heads, int64_t budget, int64_t max_kv_len) {
  KvEvictPlan p{};
  const int64_t rows = (int64_t)batch * n_kv_heads;
  p.moving_at = (rows * 2 * budget * (int64_t)sizeof(int32_t) + 255) & ~255ll;
  p.counts_at = (p.moving_at + rows * (int64_t)sizeof(int32_t) + 255) & ~255ll;
  p.workspace = p.counts_at;
  // Parts of 8192 tokens, where a workgroup's registers do not hold a row's keys, and a launch takes them.  By
  // 4096 / 8192 / 16384, us: 2 x 8 heads of up to 131072 106 / 87 / 104, 1 x 8 of 32768 47 / 50 / 67, 48 x 8 of 20000
  // 324 / 264 / 261.  The lengths are the device's: rows that turn out short are taken in as many parts (32 x 8 heads of
  // about 4130 tokens to 4096, us by bound: 4201 16, 16384 25, 16400 97, 131072 312).
  const int64_t parts = (max_kv_len + 8191) / 8192;
  p.parts = (int32_t)(parts < kKvEvictMostParts ? parts : kKvEvictMostParts);
  if (max_kv_len <= 16 * kThreads) p.parts = 0;
  if (p.parts) p.workspace += rows * (kKvEvictRowBytes + (int64_t)p.parts * kKvEvictPartBytes);
  if (rows * p.parts > kv_most_blocks(kThreads)) p.parts = 0;
  return p;
}

hipError_t launch_kv_evict(KvEvictArgs a, int32_t D, const KvEvictPlan& p, int64_t max_kv_len, void* workspace, hipStream_t s) {
  a.rows = a.pages.batch * a.pages.geom.n_kv_heads;
  a.lengths = a.kv_len_out != a.kv_len;
  a.parts = p.parts;
  a.lists = static_cast<int32_t*>(workspace);
  a.moving = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + p.moving_at);
  a.counts = static_cast<uint8_t*>(workspace) + p.counts_at;
  const int64_t turns = (a.budget + kMoveRows * kMoveDeep - 1) / (kMoveRows * kMoveDeep), most = 2048 / a.rows + 1;
  a.move_parts = (int32_t)(turns < most ? turns : most);
  // What moves is a launch of its own also where whole rows are done by few workgroups and much can move (not
  // where the last tokens' places would overlap: these go in turn).  One workgroup a row / two launches, us, 8 rows:
  // 4100 tokens to 3500 17 / 18, to 2000 22 / 18, 8200 to 2000 36 / 27, 16000 to 6000 73 / 31; 64 rows: 25 / 26
  // (4100 to 2000), 39 / 36, 95 / 61; 128 rows: 27 / 41, 52 / 62, 106 / 103; 8 rows, 4100 to 4000, the last 300: 15 / 27.
  const int64_t keep = a.budget - a.first - a.last, behind = max_kv_len - a.budget;
  if (p.parts == 0 && !(a.rows <= 64 && (keep < behind ? keep : behind) > 768 && behind >= a.last)) a.move_parts = 0;
  const bool short_rows = max_kv_len - a.first - a.last <= 4 * kThreads;
  const hipError_t e = D == 64 ? evict<64>(a, short_rows, s) : (D == 128 ? evict<128>(a, short_rows, s) : evict<256>(a, short_rows, s));
  if (e != hipSuccess || a.lengths) return e;
  hipLaunchKernelGGL(k_kv_lengths, dim3((unsigned)((a.pages.batch + 255) / 256)), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace nvfp4
