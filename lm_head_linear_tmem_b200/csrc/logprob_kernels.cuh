// Kernels of the LM head's scoring operator (flce_logprobs_forward): log
// probabilities of given tokens, entropy and top alternatives of every row's
// distribution softmax(x), x = softcap(hidden . weight^T) / temperature.
//
//   ScoreEpi        epilogue of the tcgen05 GEMM (tc_gemm.cuh): streaming softmax
//                   statistics and the candidates for the largest logits of a row
//   score_simt      the same partial results for float32 inputs (CUDA cores), few rows
//   score_tile      ... and more rows
//   score_finish    joins a row's partial results and evaluates the outputs
#pragma once

#include <math_constants.h>

#include "small_kernels.cuh"

namespace flce {

// Longest list of large logits that a row keeps: top_k (at most kMaxTopK) and
// kTopMargin more, because the lists are ordered by the tensor cores' fp32 logits
// and the final order by the logits in fp64: an alternative is lost only if more
// than kTopMargin others stand between its fp32 rank and top_k.
constexpr int kMaxTopK = 32;
constexpr int kTopMargin = 4;
constexpr int kMaxTopList = kMaxTopK + kTopMargin;
// Without alternatives a list still serves the correction of lse and entropy (see
// score_finish).  2: 671 us at 8192 x 2048 x 32000, against 710 with 4; on rows of 4 equally
// likely tokens at H = 4096 log probabilities are 4e-7 off and entropies 6e-6 (fp32 sums of
// cuBLAS: 5e-6 and 4e-6), with one or more alternatives 7e-8 and 2e-7.
constexpr int kPlainList = 2;

// Order-preserving map of the floats (no NaN) onto unsigned; 0 lies below all.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  if (k == 0u) return -CUDART_INF_F;
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// The largest float below v (not NaN); -inf stays.
__device__ __forceinline__ float nextbelow(float v) {
  return v == -CUDART_INF_F ? v : v == 0.f ? -1.4e-45f : order_value(order_key(v) - 1u);
}

// Statistics of a set of logits L (after the softcap), scale = log2(e) / temperature: m their
// maximum, s = sum 2^((L - m) scale), t = sum 2^((L - m) scale) (L - m) scale.  Then, in log2
// units,
//   lse = m scale + log2 s      entropy = log2 s - t / s
// (t <= 0: the entropy is a sum of two non-negative terms, nothing cancels).
// Differences are taken before they are scaled: the largest term is then 2^0 at any
// temperature.  (A rounded m scale is off by half its step, which passes 2^7 once |m| scale
// passes 2^31, and the largest term would be infinite or 0.)
struct Stats {
  float m, s, t;
};

// Moves (s, t) to the maximum `m1` >= st.m; d = exp2_arg(st.m, m1), e = 2^d.
__device__ __forceinline__ void stats_rebase(Stats& st, float m1, float d, float e) {
  st.t = fmaf(st.s, d, st.t) * e;
  st.s *= e;
  st.m = m1;
}

__device__ __forceinline__ void stats_merge(Stats& a, Stats b, float scale) {
  const float m1 = fmaxf(a.m, b.m);
  const float da = exp2_arg(a.m, m1, scale), db = exp2_arg(b.m, m1, scale);
  stats_rebase(a, m1, da, exp2f(da));
  stats_rebase(b, m1, db, exp2f(db));
  a.s += b.s;
  a.t += b.t;
}

// One entry of a list of large logits: the logit before softcap and temperature
// (both keep the order; > kNoMax) and its vocabulary id.
struct TopEntry {
  float v;
  int id;
};
// The order of alternatives (entries with different ids).
__device__ __forceinline__ bool better(TopEntry a, TopEntry b) {
  return a.v > b.v || (a.v == b.v && a.id < b.id);
}

// ------------------------------------------------------------------ GEMM epilogue
// A CTA works on runs of consecutive column tiles of one row tile, so a thread
// sees one row's logits over a long range of columns and keeps that row's state
// in registers until the run ends: partial results per row and run instead of
// per row and tile.  Candidates for the row's K best are appended to the run's list
// in global memory by stores that nothing waits for.  (The tensor cores and TMA
// keep shared memory and the L1 busy: lists there, or in local memory, cost 1000 to
// 13000 clocks an update, against the 33000 clocks that a 256 x 512 tile's MMAs
// take at H = 2048.)
// What keeps candidates few: `seen` holds, for each row, the maxima of K groups of
// the columns that any CTA has seen (128-column blocks, dealt out in turn); the
// least of them is a lower bound of the row's K-th best.  A logit below it cannot
// be among the K best; equal ones are kept, because a lower id wins.  About
// ln(K + 1) K / n of the columns are candidates after n columns.
// The K best by (logit, lowest id) are in the lists whatever the order in which
// runs are worked on, so the results do not depend on it.

// Entries of a run's list: room for the K best and K new ones (see scan), and some
// more so that this limit seldom counts.
constexpr int top_list_cap(int K) { return 2 * K + 24; }
constexpr int kMaxTopCap = top_list_cap(kMaxTopList);

template <bool kSoftcap>
struct ScoreEpi {
  static constexpr bool kRun = true;
  static constexpr bool kSplit = false;
  static constexpr int kEpiWarps = 8;
  static constexpr int kStagingPerWarp = 32 * 32 * 4;  // 32 columns of 32 rows (see scan)
  __device__ static void init_smem(uint8_t*) {}

  struct Params {
    int N;
    int V;
    float softcap;
    float inv_softcap;
    float scale;      // log2(e) / temperature
    RunMap map;
    int tile_cols;
    int slots;        // 2 * runs per row (the two warps of a row, half a bank each)
    int K;
    float4* part;     // [N][slots]: m, s, t, largest logit of the run (-inf: none)
    int* count;       // [N][slots]: entries of the list
    TopEntry* lists;  // [N][slots][top_list_cap(K)], ids ascending
    uint32_t* seen;   // [K][N] order_key of the groups' maxima; zeroed before the launch
  };

  struct State {
    Stats st;
    float zmax;   // largest logit of the run
    float above;  // candidates are larger than this
    int n;        // entries of the list
  };

  struct Pre {
    float bound;
  };
  __device__ static Pre prepare(const Params& p, int m_base, int q, int lane) {
    const int row = m_base + q * 32 + lane;
    if (row >= p.N) return Pre{CUDART_INF_F};
    uint32_t least = 0xffffffffu;
    const volatile uint32_t* g = p.seen + row;
#pragma unroll 4
    for (int i = 0; i < p.K; ++i) least = min(least, g[static_cast<size_t>(i) * p.N]);
    return Pre{order_value(least)};
  }

  // Bit j: r[j] > b, by the sign of b - r[j] (a NaN has none): no predicates to wait for.
  __device__ static uint32_t larger(const uint32_t (&r)[32], float b) {
    uint32_t h[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int j = 7; j >= 0; --j)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        h[i] = __funnelshift_l(__float_as_uint(b - __uint_as_float(r[8 * i + j])), h[i], 1);
    return h[0] | h[1] << 8 | h[2] << 16 | h[3] << 24;
  }

  // How many of n values are at least x (a NaN counts as large: the alternatives
  // of such a row are not defined).
  template <int n, class F>
  __device__ static int at_least(const F& value, float x) {
    uint32_t below[4] = {0u, 0u, 0u, 0u};  // v < x is the sign of v - x
#pragma unroll
    for (int j = 0; j < n; ++j) below[j & 3] += __float_as_uint(value(j) - x) >> 31;
    return n - static_cast<int>((below[0] + below[1]) + (below[2] + below[3]));
  }

  // The K-th largest of n values none of which exceeds mx (-inf if there are fewer).
  template <int n, class F>
  __device__ static float kth_largest(const F& value, int K, float mx) {
    uint32_t lo = order_key(-CUDART_INF_F), hi = order_key(mx);
    // (32 halvings settle any interval)
    for (int it = 0; it < 32 && __any_sync(0xffffffffu, lo < hi); ++it) {
      const uint32_t mid = lo + (hi - lo + 1u) / 2u;
      if (at_least<n>(value, order_value(mid)) >= K)
        lo = mid;
      else
        hi = mid > lo ? mid - 1u : lo;
    }
    return order_value(lo);
  }

  // A lower bound of the K-th largest of 128 columns (-inf if it finds none) that
  // not many more than K reach.  It starts from the least of the four chunks'
  // maxima, which about nine columns reach, goes down in growing steps while
  // fewer than K reach it, and then halves; the second largest maximum is the
  // upper end, so that one logit far above the others does not stretch the range.
  __device__ static float near_kth(const uint32_t (&r)[4][32], int K, const float (&mx)[4],
                                   float mx_all) {
    const auto value = [&](int j) { return __uint_as_float(r[j / 32][j % 32]); };
    float m[4];  // a chunk past the vocabulary, or masked, says nothing
#pragma unroll
    for (int c = 0; c < 4; ++c) m[c] = mx[c] <= kNoMax ? mx_all : mx[c];
    const float a0 = fminf(m[0], m[1]), a1 = fmaxf(m[0], m[1]);
    const float b0 = fminf(m[2], m[3]), b1 = fmaxf(m[2], m[3]);
    float hi = fmaxf(fminf(a1, b1), fmaxf(a0, b0)), x = fminf(a0, b0);
    float step = hi - x, bound = -CUDART_INF_F;
#pragma unroll 1
    for (int it = 0; it < 8; ++it) {
      const int n = at_least<128>(value, x);
      if (n >= K)
        bound = x;
      else
        hi = x;
      // (NaN bounds, from infinities, end the search where it is)
      const bool done = (n >= K && n <= 2 * K + 4) || !(hi > bound);
      if (__all_sync(0xffffffffu, done)) break;
      if (!done) {
        x = bound > -CUDART_INF_F ? 0.5f * bound + 0.5f * hi : x - step;
        step *= 2.f;
      }
    }
    return bound;
  }

  // Appends the candidates among the 128 columns starting at `col`; mx are the
  // maxima of 32 columns each.  Most often no lane has more than one, which then is
  // its maximum.  Where a list has no room for all of a lane's candidates, the
  // block's own K best will do (there is room for K: tidy() sees to it).
  __device__ static void scan(State& S, TopEntry* list, int K, const uint32_t (&r)[4][32],
                              const float (&mx)[4], float mx_all, int col, float* stage) {
    if (!__any_sync(0xffffffffu, mx_all > S.above)) return;
    uint32_t hits[4];
    const auto find = [&](float above) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        hits[c] = __any_sync(0xffffffffu, mx[c] > above) ? larger(r[c], above) : 0u;
      return (__popc(hits[0]) + __popc(hits[1])) + (__popc(hits[2]) + __popc(hits[3]));
    };
    int n = find(S.above);
    float kth = -CUDART_INF_F;
    if (__any_sync(0xffffffffu, n > 2 * K + 4)) {
      // a run's start, before any CTA has seen enough of the row (or logits that
      // rise with the id): all but the block's own best would be for nothing
      kth = near_kth(r, K, mx, mx_all);
      n = find(fmaxf(S.above, nextbelow(kth)));
    }
    const bool full = n > top_list_cap(K) - S.n;
    if (__any_sync(0xffffffffu, full)) {
      const float x = kth_largest<128>(
          [&](int j) { return __uint_as_float(r[j / 32][j % 32]); }, K, mx_all);
      // those above x, and of those equal to x the first ones up to K
      uint32_t gt[4], eq[4];
      int room = K;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        gt[c] = larger(r[c], x);
        eq[c] = larger(r[c], nextbelow(x)) & ~gt[c];
        room -= __popc(gt[c]);
      }
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        while (__popc(eq[c]) > max(room, 0)) eq[c] &= ~(0x80000000u >> __clz(eq[c]));
        room -= __popc(eq[c]);
        if (full) hits[c] = gt[c] | eq[c];
      }
      if (full) {
        n = __popc(hits[0]) + __popc(hits[1]) + __popc(hits[2]) + __popc(hits[3]);
        S.above = fmaxf(S.above, x);
      }
    }
    if (!__any_sync(0xffffffffu, n > 1)) {
      int j = 0;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (hits[c] != 0u) j = c * 32 + __ffs(hits[c]) - 1;
      if (n > 0) list[S.n++] = TopEntry{mx_all, col + j};
    } else {
      // through shared memory, where a lane can take column j of its own: a short
      // loop, for code that is seldom run waits for its instructions (32 unrolled
      // conditional stores took 10000 clocks)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        if (!__any_sync(0xffffffffu, hits[c] != 0u)) continue;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; ++j) stage[32 * j] = __uint_as_float(r[c][j]);
        __syncwarp();
        for (uint32_t h = hits[c]; h != 0u; h &= h - 1u) {
          const int j = __ffs(h) - 1;
          list[S.n++] = TopEntry{stage[32 * j], col + c * 32 + j};
        }
      }
    }
    S.above = fmaxf(S.above, kth);  // K columns with lower ids reach kth
  }

  // Cuts a list that may have no room for K more down to its own K best.
  __device__ static void tidy(State& S, TopEntry* list, int K) {
    const bool full = S.n > top_list_cap(K) - K;
    if (!__any_sync(0xffffffffu, full)) return;
    float e[kMaxTopCap];
    float top = -CUDART_INF_F;
#pragma unroll
    for (int i = 0; i < kMaxTopCap; ++i) {
      e[i] = i < S.n ? list[i].v : -CUDART_INF_F;
      top = fmaxf(top, e[i]);
    }
    const float x = kth_largest<kMaxTopCap>([&](int i) { return e[i]; }, K, top);
    if (!full) return;
    int room = K;
#pragma unroll
    for (int i = 0; i < kMaxTopCap; ++i) room -= e[i] > x ? 1 : 0;
    int n = 0;
    for (int i = 0; i < S.n; ++i) {
      const TopEntry c = list[i];
      if (c.v > x || (c.v == x && room-- > 0)) list[n++] = c;
    }
    S.n = n;
    S.above = fmaxf(S.above, x);  // later ids that equal x come after K others
  }

  __device__ static float max32(const uint32_t (&r)[32]) {
    float mx[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) mx[j] = fmaxf(__uint_as_float(r[j]), __uint_as_float(r[j + 16]));
#pragma unroll
    for (int w = 8; w >= 1; w /= 2)
#pragma unroll
      for (int j = 0; j < w; ++j) mx[j] = fmaxf(mx[j], mx[j + w]);
    return mx[0];
  }

  __device__ static bool tile(const Params& p, const Pre& pre, int m_base, int col0,
                              uint32_t taddr, int q, int lane, int part, uint8_t* stg,
                              const CUtensorMap*, uint32_t tempty, State& S, bool,
                              const volatile int*, unsigned long long, int) {
    if (col0 >= p.V) {  // the second bank of a 512-column tile past the vocabulary
      release_tmem(tempty, lane);
      return true;
    }
    const int row = m_base + q * 32 + lane;
    const bool row_ok = row < p.N;
    const int run = p.map.of_tile(col0 / p.tile_cols);
    int run_start, run_len;
    p.map.of_run(run, run_start, run_len);
    const bool first = col0 == run_start * p.tile_cols;
    if (first) {
      S.st = Stats{kNoneYet, 0.f, 0.f};
      S.zmax = -CUDART_INF_F;
      S.above = row_ok ? kNoMax : CUDART_INF_F;  // rows past the end take nothing
      S.n = 0;
    }
    const size_t at = static_cast<size_t>(row) * p.slots + run * 2 + part;
    TopEntry* list = p.lists + at * top_list_cap(p.K);
    const int h0 = col0 + part * (BN / 2);  // this warp's first column
    const int ncols = max(0, min(BN / 2, p.V - h0));
    const uint32_t ta = taddr + part * (BN / 2);
    // all 128 columns into registers, the TMEM half released at once
    uint32_t r[4][32];
#pragma unroll
    for (int c = 0; c < 4; ++c) tmem_ld_x32(ta + c * 32, r[c]);
    tmem_ld_wait();
#pragma unroll
    for (int c = 0; c < 4; ++c) reg_fence(r[c]);
    release_tmem(tempty, lane);
    if (ncols < BN / 2) {  // the vocabulary ends inside (or before) these columns
#pragma unroll
      for (int j = 0; j < 128; ++j)
        if (j >= ncols) r[j / 32][j % 32] = __float_as_uint(-CUDART_INF_F);
    }
    if (!kSoftcap && p.scale < kTinyScale) {
#pragma unroll
      for (int j = 0; j < 128; ++j)
        if (__uint_as_float(r[j / 32][j % 32]) <= kNoMax)
          r[j / 32][j % 32] = __float_as_uint(-CUDART_INF_F);
    }
    float mx[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) mx[c] = max32(r[c]);
    float mx_all = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));

    // ---- list
    S.zmax = fmaxf(S.zmax, mx_all);
    S.above = fmaxf(S.above, nextbelow(pre.bound));  // (an equal logit may still count)
    scan(S, list, p.K, r, mx, mx_all, h0, reinterpret_cast<float*>(stg) + lane);
    if (row_ok && mx_all > pre.bound)
      atomicMax(p.seen + static_cast<size_t>(h0 / (BN / 2) % p.K) * p.N + row,
                order_key(mx_all));

    // ---- statistics
    if constexpr (kSoftcap) {
      auto cap = [&](float z) { return cap_logit(p.softcap, tanh_exp2(z * p.inv_softcap)); };
#pragma unroll
      for (int j = 0; j < 128; ++j)
        r[j / 32][j % 32] = __float_as_uint(cap(__uint_as_float(r[j / 32][j % 32])));
      if (ncols < BN / 2) {  // the cap has made columns past the end -softcap
#pragma unroll
        for (int j = 0; j < 128; ++j)
          if (j >= ncols) r[j / 32][j % 32] = __float_as_uint(-CUDART_INF_F);
      }
      // (rounded tanh may swap logits a step apart, and over a tiny temperature a step is much: the
      // maximum is that of the capped ones; -inf: no columns)
#pragma unroll
      for (int c = 0; c < 4; ++c) mx[c] = max32(r[c]);
      mx_all = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
    }
    Stats& st = S.st;
    const float m1 = fmaxf(st.m, mx_all);  // a NaN maximum (all NaN) leaves st.m
    const float d1 = exp2_arg(st.m, m1, p.scale);
    stats_rebase(st, m1, d1, ex2_approx(d1));
    float s4[4] = {0.f, 0.f, 0.f, 0.f}, t4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 128; ++j) {
      const float d = exp2_arg(__uint_as_float(r[j / 32][j % 32]), m1, p.scale);
      const float e = ex2_approx(d);
      s4[j & 3] += e;
      t4[j & 3] = fmaf(e, d, t4[j & 3]);
    }
    st.s += (s4[0] + s4[1]) + (s4[2] + s4[3]);
    st.t += (t4[0] + t4[1]) + (t4[2] + t4[3]);

    const int run_end = min((run_start + run_len) * p.tile_cols, (p.V + BN - 1) / BN * BN);
    if (col0 + BN < run_end) {
      tidy(S, list, p.K);
    } else if (row_ok) {  // the run's last bank
      p.part[at] = make_float4(st.m, st.s, st.t, S.zmax);
      p.count[at] = S.n;
    }
    return true;
  }
};

// ------------------------------------------------------------------ fp32 inputs
// Partial results of kRows rows x kCols columns per block (slot = column
// block): each warp computes the logits of four columns at a time against all
// rows (hidden rows in shared memory, the weight read once per block), then one
// warp per row reduces them.
constexpr int kScoreThreads = 256;

// Sums of n values over the 2 * o lanes that differ in the bits below 2 * o, halving the
// values that a lane holds at each step (31 shuffles for 32 values, where a sum of its
// own for each takes 160): lane l of 32 ends with value l / (32 / n) in v[0].
template <int o, int n, int size>
__device__ __forceinline__ void lane_sums(float (&v)[size], int lane) {
  if constexpr (n > 1) {
    const bool up = (lane & o) != 0;
#pragma unroll
    for (int i = 0; i < n / 2; ++i) {
      const float keep = up ? v[i + n / 2] : v[i], send = up ? v[i] : v[i + n / 2];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
    }
    if constexpr (o > 1) lane_sums<o / 2, n / 2>(v, lane);
  } else {
    v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    if constexpr (o > 1) lane_sums<o / 2, 1>(v, lane);
  }
}

// kVec: 4 where H is a multiple of 4 and hidden and weight are 16-byte aligned (so are their
// rows then), else 1.
template <int kRows, int kCols, int kVec>
__global__ void __launch_bounds__(kScoreThreads)
    score_simt_kernel(const float* __restrict__ hidden, const float* __restrict__ weight, int N,
                      int H, int V, float softcap, float scale, int slots, int K, int cap,
                      float4* __restrict__ part, int* __restrict__ count,
                      TopEntry* __restrict__ lists) {
  extern __shared__ __align__(16) float sh[];
  float* hs = sh;               // [kRows][H]
  float* zs = sh + kRows * H;   // [kRows][kCols]
  const int row0 = blockIdx.y * kRows, v0 = blockIdx.x * kCols;
  const int rows = min(kRows, N - row0), cols = min(kCols, V - v0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll 8
  for (int i = threadIdx.x; i < kRows * H; i += kScoreThreads)
    hs[i] = i < rows * H ? hidden[static_cast<size_t>(row0) * H + i] : 0.f;
  __syncthreads();
  constexpr int kC = 4;
  constexpr int kSums = kRows * kC;
  static_assert(kSums <= 32, "a lane for every sum");
  for (int c0 = warp * kC; c0 < cols; c0 += kScoreThreads / 32 * kC) {
    float acc[kRows][kC];
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int c = 0; c < kC; ++c) acc[r][c] = 0.f;
    const float* w[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c)  // columns past the block's end repeat its last one
      w[c] = weight + static_cast<size_t>(v0 + min(c0 + c, cols - 1)) * H;
#pragma unroll 2
    for (int k = lane * kVec; k < H; k += 32 * kVec) {
      float wv[kC][kVec];
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        if constexpr (kVec == 4)
          *reinterpret_cast<float4*>(wv[c]) = *reinterpret_cast<const float4*>(w[c] + k);
        else
          wv[c][0] = w[c][k];
      }
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        float h[kVec];
        if constexpr (kVec == 4)
          *reinterpret_cast<float4*>(h) = *reinterpret_cast<const float4*>(hs + r * H + k);
        else
          h[0] = hs[r * H + k];
#pragma unroll
        for (int c = 0; c < kC; ++c)
#pragma unroll
          for (int i = 0; i < kVec; ++i) acc[r][c] = fmaf(h[i], wv[c][i], acc[r][c]);
      }
    }
    float v[kSums];
#pragma unroll
    for (int i = 0; i < kSums; ++i) v[i] = acc[i / kC][i % kC];
    lane_sums<16, kSums>(v, lane);
    const int at = lane / (32 / kSums), r = at / kC, c = at % kC;
    if (lane % (32 / kSums) == 0 && c0 + c < cols) zs[r * kCols + c0 + c] = v[0];
  }
  __syncthreads();
  for (int r = warp; r < rows; r += kScoreThreads / 32) {
    float* z = zs + r * kCols;
    const size_t at = static_cast<size_t>(row0 + r) * slots + blockIdx.x;
    Stats st{kNoneYet, 0.f, 0.f};
    for (int c = lane; c < cols; c += 32) st.m = fmaxf(st.m, seen_logit(z[c], softcap));
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) st.m = fmaxf(st.m, __shfl_xor_sync(0xffffffffu, st.m, o));
    for (int c = lane; c < cols; c += 32) {
      const float d = exp2_arg(seen_logit(z[c], softcap), st.m, scale);
      const float e = exp2f(d);
      st.s += e;
      st.t = fmaf(e, d, st.t);
    }
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) {
      st.s += __shfl_xor_sync(0xffffffffu, st.s, o);
      st.t += __shfl_xor_sync(0xffffffffu, st.t, o);
    }
    // the K largest, one after another
    int n = 0;
    float top = -CUDART_INF_F;
    for (; n < K; ++n) {
      float best = kNoMax;
      int id = -1;
      for (int c = lane; c < cols; c += 32)
        if (z[c] > best) {
          best = z[c];
          id = c;
        }
#pragma unroll
      for (int o = 16; o >= 1; o /= 2) {
        const float v = __shfl_xor_sync(0xffffffffu, best, o);
        const int vi = __shfl_xor_sync(0xffffffffu, id, o);
        if (v > best || (v == best && vi >= 0 && (id < 0 || vi < id))) {
          best = v;
          id = vi;
        }
      }
      if (id < 0) break;
      top = fmaxf(top, best);
      if (lane == 0) {
        lists[at * cap + n] = TopEntry{best, v0 + id};
        z[id] = -CUDART_INF_F;
      }
      __syncwarp();
    }
    if (lane == 0) {
      part[at] = make_float4(st.m, st.s, st.t, top);
      count[at] = n;
    }
  }
}

// The same for more rows than a few: kTileRows rows x kTiles * 64 columns a block, as a
// register-tiled product.  Stages of 64 k arrive by cp.async, three ahead; in each, four
// groups of 128 threads take a quarter of the k with 8 x 4 products a thread, so that one
// block keeps 16 warps busy on a 64 x 64 tile.  The groups add their sums one after another
// into zs, from which a warp reduces a row at a time.
// 60 x 4096 x 32000: 0.58 ms (1.50 by score_simt, which reads the weight once per 8 rows);
// 4096 x 1000 x 32000: 8.2 ms, half the rate of the multiply-adds.  The other half goes to
// operands from shared memory and the copies' instructions; groups of 64 threads with 8 x 8
// products, packed multiply-adds, stages of 128 k and 1024 threads were no faster.
constexpr int kTileRows = 64, kTileCols = 64, kTileK = 64, kTileStages = 4;
constexpr int kTileThreads = 512, kTileGroups = 4, kTileTc = 4;  // columns of a thread
constexpr int kTilePitch = kTileK + 4;  // floats; rows then start 4 banks apart

__device__ __forceinline__ void cp_async_16(uint32_t dst, const float* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const float* src, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
template <int kTiles>
constexpr int kTileZPitch = kTiles * kTileCols + 8;
template <int kTiles>
constexpr size_t kTileSmem = sizeof(float) * (kTileStages * (kTileRows + kTileCols) * kTilePitch +
                                              kTileRows * kTileZPitch<kTiles>);

template <int kTiles, int kVec>
__global__ void __launch_bounds__(kTileThreads, 1)
    score_tile_kernel(const float* __restrict__ hidden, const float* __restrict__ weight, int N,
                      int H, int V, float softcap, float scale, int slots, int K, int cap,
                      float4* __restrict__ part, int* __restrict__ count,
                      TopEntry* __restrict__ lists) {
  extern __shared__ __align__(16) float sh[];
  constexpr int kStage = (kTileRows + kTileCols) * kTilePitch;
  constexpr int kZ = kTileZPitch<kTiles>, kCols = kTiles * kTileCols;
  float* zs = sh + kTileStages * kStage;  // [kTileRows][kZ]
  const int row0 = blockIdx.y * kTileRows, v0 = blockIdx.x * kCols;
  const int rows = min(kTileRows, N - row0), cols = min(kCols, V - v0);
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int tiles = (cols + kTileCols - 1) / kTileCols;

  // The next stage to load: k block at lk of column tile lt, zeros past the rows, the columns
  // and H.  A thread's four vectors are at one k of rows 32 apart, so that what is left
  // to do for each is an addition, two selections and the copy (the addresses worked out anew
  // took as many instructions as the products).
  constexpr int kQ = kTileK / 4, kEach = kTileThreads / kQ;
  static_assert(kTileRows == 2 * kEach && kTileCols == 2 * kEach, "vectors of a thread");
  const int lr = t / kQ, lq = 4 * (t % kQ);
  const float* src[4];
  int lim[4];  // k below which there is something to load
  const auto point = [&](int e, const float* base, int row, int end) {
    src[e] = base + (row < end ? static_cast<size_t>(row) * H : 0) + lq;
    lim[e] = row < end ? H - lq : 0;
  };
  const auto point_cols = [&](int c0) {
    point(2, weight, c0 + lr, V);
    point(3, weight, c0 + lr + kEach, V);
  };
  point(0, hidden, row0 + lr, N);
  point(1, hidden, row0 + lr + kEach, N);
  point_cols(v0);
  int lk = 0, lt = 0, ls = 0;
  const uint32_t dst0 = smem_u32(sh + lr * kTilePitch + lq);
  const auto load = [&] {
    if (lt < tiles) {
      const uint32_t dst = dst0 + static_cast<uint32_t>(ls * kStage * 4);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float* from = lk < lim[e] ? src[e] + lk : hidden;
        const uint32_t to = dst + static_cast<uint32_t>(e * kEach * kTilePitch * 4);
        if constexpr (kVec == 4) {
          cp_async_16(to, from, lk < lim[e] ? 16 : 0);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            cp_async_4(to + 4u * j, lk + j < lim[e] ? from + j : hidden, lk + j < lim[e] ? 4 : 0);
        }
      }
      ls = ls + 1 < kTileStages ? ls + 1 : 0;
      lk += kTileK;
      if (lk >= H) {
        lk = 0;
        ++lt;
        point_cols(v0 + lt * kTileCols);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int i = 0; i < kTileStages - 1; ++i) load();

  constexpr int kTx = kTileCols / kTileTc, kGroup = 8 * kTx;
  static_assert(kGroup * kTileGroups == kTileThreads, "threads");
  const int group = t / kGroup, ty = t % kGroup / kTx, tx = t % kTx;
  float acc[8][kTileTc];
  const float* a0 = sh + ty * kTilePitch + group * (kTileK / kTileGroups);
  const float* b0 = sh + (kTileRows + tx) * kTilePitch + group * (kTileK / kTileGroups);
  int stage = 0;
  for (int tile = 0; tile < tiles; ++tile) {
#pragma unroll
    for (int r = 0; r < 8; ++r)
#pragma unroll
      for (int c = 0; c < kTileTc; ++c) acc[r][c] = 0.f;
    for (int k = 0; k < H; k += kTileK) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kTileStages - 2) : "memory");
      __syncthreads();  // this stage is there, and the one before it has been read
      load();
      const float *a = a0 + stage * kStage, *b = b0 + stage * kStage;
      stage = stage + 1 < kTileStages ? stage + 1 : 0;
#pragma unroll
      for (int q = 0; q < kTileK / 4 / kTileGroups; ++q) {
        float4 av[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
          av[r] = *reinterpret_cast<const float4*>(a + r * 8 * kTilePitch + 4 * q);
#pragma unroll
        for (int c = 0; c < kTileTc; ++c) {
          const float4 bv =
              *reinterpret_cast<const float4*>(b + c * kTx * kTilePitch + 4 * q);
#pragma unroll
          for (int r = 0; r < 8; ++r) {
            acc[r][c] = fmaf(av[r].x, bv.x, acc[r][c]);
            acc[r][c] = fmaf(av[r].y, bv.y, acc[r][c]);
            acc[r][c] = fmaf(av[r].z, bv.z, acc[r][c]);
            acc[r][c] = fmaf(av[r].w, bv.w, acc[r][c]);
          }
        }
      }
    }
    float* z = zs + ty * kZ + tile * kTileCols + tx;
    for (int g = 0; g < kTileGroups; ++g) {
      if (group == g)
#pragma unroll
        for (int r = 0; r < 8; ++r)
#pragma unroll
          for (int c = 0; c < kTileTc; ++c) {
            float& o = z[r * 8 * kZ + c * kTx];
            o = g == 0 ? acc[r][c] : o + acc[r][c];
          }
      __syncthreads();
    }
  }

  constexpr int kMine = kCols / 32;  // columns of a lane
  for (int r = warp; r < rows; r += kTileThreads / 32) {
    const size_t at = static_cast<size_t>(row0 + r) * slots + blockIdx.x;
    float z[kMine];
    Stats st{kNoneYet, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < kMine; ++c) {
      z[c] = lane + 32 * c < cols ? zs[r * kZ + lane + 32 * c] : -CUDART_INF_F;
      if (lane + 32 * c < cols) st.m = fmaxf(st.m, seen_logit(z[c], softcap));
    }
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) st.m = fmaxf(st.m, __shfl_xor_sync(0xffffffffu, st.m, o));
    uint32_t key[kMine];
#pragma unroll
    for (int c = 0; c < kMine; ++c) {
      key[c] = z[c] > kNoMax ? order_key(z[c]) : 0u;
      if (lane + 32 * c < cols) {
        const float d = exp2_arg(seen_logit(z[c], softcap), st.m, scale);
        const float e = exp2f(d);
        st.s += e;
        st.t = fmaf(e, d, st.t);
      }
    }
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) {
      st.s += __shfl_xor_sync(0xffffffffu, st.s, o);
      st.t += __shfl_xor_sync(0xffffffffu, st.t, o);
    }
    // the K largest, one after another: the lowest column of the largest key
    int n = 0;
    uint32_t top = 0u;
    for (; n < K; ++n) {
      uint32_t mine = key[0];
#pragma unroll
      for (int c = 1; c < kMine; ++c) mine = max(mine, key[c]);
      const uint32_t best = __reduce_max_sync(0xffffffffu, mine);
      if (best == 0u) break;
      if (n == 0) top = best;
      bool taken = false;
#pragma unroll
      for (int c = 0; c < kMine; ++c) {
        const uint32_t have = __ballot_sync(0xffffffffu, !taken && key[c] == best);
        if (have != 0u && !taken) {
          taken = true;
          if (lane == __ffs(have) - 1) {
            key[c] = 0u;
            lists[at * cap + n] = TopEntry{order_value(best), v0 + 32 * c + lane};
          }
        }
      }
    }
    if (lane == 0) {
      part[at] = make_float4(st.m, st.s, st.t, order_value(top));
      count[at] = n;
    }
  }
}

// ------------------------------------------------------------------ outputs
// One block per (compact) row: merges the slots' statistics in a fixed order,
// picks the K best entries of the lists, computes the logits of those and of
// the row's token again in fp64 (the products of two bf16 are exact in fp32;
// of two fp32, in fp64), orders them by (logit, lowest id) and writes the row's
// outputs at its place in token order.
// The fp64 pass makes the order of near-equal alternatives, and with it the
// ids, independent of how the logits were summed; it reads (K + 1) weight rows
// per token against the V rows of the GEMM.
// It also puts the statistics right where they are large.  The tensor cores cut
// each of the H / 16 partial sums off towards zero, which lowers a logit of 20 at
// H = 4096 by about 1e-4 (measured: 1e-5 of the log probability).  In the bulk of
// the vocabulary that hardly shows (small logits), but a row whose probability
// sits in a few tokens has an lse that is one of their logits.  So the listed
// logits' terms are taken out of (s, t) as the epilogue added them and put back
// with their fp64 values.  The backward recomputes the uncorrected logits L: it gets
// the uncorrected statistics (`saved`), the maximum m and log2 s apart: with
// log2 p = (L - m) scale - log2 s, p of a dominant token is 1 - p to fp32 rounding at any
// temperature (of one fp32 number of the size of L / T, half a step goes into every p: the 1 - p
// of a certain token came out 1e-6 at T = 1 and 3e-4 at 0.01, and is divided by T).
constexpr int kGroups = 64;  // of a row's lists, for the lower bound of the K-th best
constexpr int kMaxHits = 512;
constexpr int kMaxHitSlots = 256;

struct FinishArgs {
  const int64_t* tokens;  // token order; null: none given
  const int* perm;        // compact row -> token row; null: the same
  const long long* n_valid;
  int N, H, V;
  int64_t ignore_index;
  float softcap;
  double inv_temp;   // 1 / temperature
  float scale;       // log2(e) / temperature
  int slots, K, cap, top_k;  // cap: entries between one list's start and the next's
  const float4* part;
  const int* count;
  const TopEntry* lists;
  float* logprobs;   // [N]; null without tokens
  float* entropy;    // [N]
  float* lse;        // [N]
  // of the logits that the backward sees, saved_rows numbers saved_stride apart.  3: their
  // maximum, log2 of their sum s and the entropy; 2: lse and the entropy
  float* saved;
  int saved_rows, saved_stride;
  float* top_logprobs;  // [N, top_k]
  int64_t* top_ids;     // [N, top_k]
  unsigned int* status;
};

// This lane's part of a dot product, in four chains (a double addition's latency,
// not its rate, is what a single one waits for).
__device__ __forceinline__ double dot_part(const __nv_bfloat16* a, const __nv_bfloat16* b, int H,
                                           int lane) {
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
#pragma unroll 8
  for (int k = lane * 8; k < H; k += 256) {  // H is a multiple of 8
    const uint4 x = *reinterpret_cast<const uint4*>(a + k);
    const uint4 y = __ldg(reinterpret_cast<const uint4*>(b + k));
    const __nv_bfloat162* x2 = reinterpret_cast<const __nv_bfloat162*>(&x);
    const __nv_bfloat162* y2 = reinterpret_cast<const __nv_bfloat162*>(&y);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u = __bfloat1622float2(x2[j]), v = __bfloat1622float2(y2[j]);
      acc[j] += static_cast<double>(u.x * v.x);
      acc[j] += static_cast<double>(u.y * v.y);
    }
  }
  return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

__device__ __forceinline__ double dot_part(const float* a, const float* b, int H, int lane) {
  double acc[4] = {0.0, 0.0, 0.0, 0.0};
  int k = lane;
  for (; k + 96 < H; k += 128)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc[j] = fma(static_cast<double>(a[k + 32 * j]), static_cast<double>(b[k + 32 * j]), acc[j]);
  for (; k < H; k += 32) acc[0] = fma(static_cast<double>(a[k]), static_cast<double>(b[k]), acc[0]);
  return (acc[0] + acc[1]) + (acc[2] + acc[3]);
}

// The softcap as the partial results have it.
template <class T>
__device__ __forceinline__ float gemm_softcap(float z, float softcap);
template <>
__device__ __forceinline__ float gemm_softcap<__nv_bfloat16>(float z, float softcap) {
  return cap_logit(softcap, tanh_exp2(z * (1.0f / softcap)));
}
template <>
__device__ __forceinline__ float gemm_softcap<float>(float z, float softcap) {
  return cap_logit(softcap, tanhf(z / softcap));
}

// kFinishThreads: by the rows and the dot products of a row (see run_finish).
template <class T, int kFinishThreads>
__global__ void __launch_bounds__(kFinishThreads)
    score_finish_kernel(const T* __restrict__ hidden, const T* __restrict__ weight,
                        const FinishArgs a) {
  constexpr int kWarps = kFinishThreads / 32;
  __shared__ float wm[kWarps], ws[kWarps], wt[kWarps], bound_sh;
  __shared__ __align__(16) float tmaxs[kFinishThreads];
  __shared__ int n_hits, n_hit_slots;
  __shared__ int hit_slots[kMaxHitSlots];  // slot, and its entries in the top byte
  __shared__ TopEntry hits[kMaxHits], wbest[2][kWarps];
  __shared__ int ids[kMaxTopList + 1];
  __shared__ float za[kMaxTopList];
  __shared__ double zx[kMaxTopList + 1], xe[kMaxTopList + 1];
  __shared__ double max_sh, log_s_sh;  // lse's two parts (their sum may round log s away)
  static_assert(kFinishThreads % kGroups == 0 && kMaxTopList < kGroups, "groups of lists");
  griddep_wait();
  const int j = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int row = a.perm != nullptr ? a.perm[j] : j;
  // After a GEMM that gave up on a wait (only the status word tells) the partial results may
  // be unwritten memory, whose counts and ids must not be followed.
  const bool failed = (*a.status & kStatusTimeout) != 0u;
  bool live = !failed && (a.perm == nullptr || j < *a.n_valid);
  int64_t y = -1;
  if (a.tokens != nullptr) {
    y = a.tokens[row];
    if (a.perm == nullptr && y != a.ignore_index && (y < 0 || y >= a.V) && t == 0)
      atomicOr(a.status, kStatusLabelRange);
    live = live && y != a.ignore_index && y >= 0 && y < a.V;
  }
  if (!live) {
    if (t == 0) {
      if (a.logprobs != nullptr) a.logprobs[row] = 0.f;
      a.entropy[row] = 0.f;
      a.lse[row] = 0.f;
      for (int i = 0; i < a.saved_rows; ++i)
        a.saved[static_cast<size_t>(i) * a.saved_stride + row] = 0.f;
    }
    for (int i = t; i < a.top_k; i += kFinishThreads) {
      a.top_logprobs[static_cast<size_t>(row) * a.top_k + i] = 0.f;
      a.top_ids[static_cast<size_t>(row) * a.top_k + i] = -1;
    }
    return;
  }

  // ---- statistics, and the largest logit of this thread's slots
  const float4* part = a.part + static_cast<size_t>(j) * a.slots;
  const int* count = a.count + static_cast<size_t>(j) * a.slots;
  const TopEntry* lists = a.lists + static_cast<size_t>(j) * a.slots * a.cap;
  Stats st{kNoneYet, 0.f, 0.f};
  float tmax = -CUDART_INF_F;
  for (int i = t; i < a.slots; i += kFinishThreads) {
    const float4 v = part[i];
    stats_merge(st, Stats{v.x, v.y, v.z}, a.scale);
    tmax = fmaxf(tmax, v.w);
  }
  float wmax = st.m;
#pragma unroll
  for (int o = 16; o >= 1; o /= 2) wmax = fmaxf(wmax, __shfl_xor_sync(0xffffffffu, wmax, o));
  if (lane == 0) wm[warp] = wmax;

  // ---- the K best entries.  The K-th largest of the groups' maxima is a lower
  // bound of the K-th best (each is a logit of its own), and about K lists have
  // entries that reach it.  Those entries are ranked against one another; if
  // ties make them more than fit, the K best are taken one by one from all lists.
  tmaxs[t] = tmax;
  if (t == 0) {
    n_hits = n_hit_slots = 0;
    bound_sh = -CUDART_INF_F;
  }
  if (t <= a.K) ids[t] = -1;
  __syncthreads();
  float gmax = tmax;
  if constexpr (kFinishThreads > kGroups) {  // a group's maximum, over its threads
    if (t < kGroups) {
#pragma unroll
      for (int i = kGroups; i < kFinishThreads; i += kGroups) gmax = fmaxf(gmax, tmaxs[t + i]);
      tmaxs[t] = gmax;
    }
    __syncthreads();
  }
  if (t < kGroups) {
    int above = 0, ties = 0;
#pragma unroll
    for (int i = 0; i < kGroups; i += 4) {
      const float4 g = *reinterpret_cast<const float4*>(tmaxs + i);
      above += (g.x > gmax) + (g.y > gmax) + (g.z > gmax) + (g.w > gmax);
      ties += (g.x == gmax) + (g.y == gmax) + (g.z == gmax) + (g.w == gmax);
    }
    if (above < a.K && above + ties >= a.K) bound_sh = gmax;  // one value whoever writes it
  }
  // the row's statistics: all slots' sums at the largest maximum, added in a fixed order
  float M = wm[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) M = fmaxf(M, wm[w]);
  const float d_m = exp2_arg(st.m, M, a.scale);
  stats_rebase(st, M, d_m, exp2f(d_m));
#pragma unroll
  for (int o = 16; o >= 1; o /= 2) {
    st.s += __shfl_xor_sync(0xffffffffu, st.s, o);
    st.t += __shfl_xor_sync(0xffffffffu, st.t, o);
  }
  if (lane == 0) {
    ws[warp] = st.s;
    wt[warp] = st.t;
  }
  __syncthreads();
  const float bound = bound_sh;
  if (tmax >= bound && tmax > -CUDART_INF_F)
    for (int l = t; l < a.slots; l += kFinishThreads)
      if (part[l].w >= bound && count[l] > 0) {
        const int at = atomicAdd(&n_hit_slots, 1);
        if (at < kMaxHitSlots) hit_slots[at] = l | count[l] << 24;
      }
  __syncthreads();
  if (n_hit_slots <= kMaxHitSlots) {
    for (int e = t; e < n_hit_slots * a.cap; e += kFinishThreads) {
      const int h = e / a.cap, i = e - h * a.cap;
      const int l = hit_slots[h] & 0xffffff;
      if (i >= hit_slots[h] >> 24) continue;
      const TopEntry x = lists[static_cast<size_t>(l) * a.cap + i];
      if (x.v >= bound) {
        const int at = atomicAdd(&n_hits, 1);
        if (at < kMaxHits) hits[at] = x;
      }
    }
  }
  __syncthreads();
  if (n_hit_slots <= kMaxHitSlots && n_hits <= kMaxHits) {
    for (int i = t; i < n_hits; i += kFinishThreads) {
      const TopEntry x = hits[i];
      int rank = 0;
      for (int c = 0; c < n_hits && rank < a.K; ++c) rank += better(hits[c], x) ? 1 : 0;
      if (rank < a.K) {
        ids[rank] = x.id;
        za[rank] = x.v;
      }
    }
  } else {
    TopEntry last{CUDART_INF_F, -1};  // taken last: the order's place to go on from
    for (int n = 0; n < a.K; ++n) {
      TopEntry best{-CUDART_INF_F, -1};
      for (int l = t; l < a.slots; l += kFinishThreads) {
        const TopEntry* e = lists + static_cast<size_t>(l) * a.cap;
        for (int i = 0; i < count[l]; ++i) {
          const TopEntry x = e[i];
          if (better(last, x) && (best.id < 0 || better(x, best))) best = x;
        }
      }
      auto take = [&](TopEntry x) {
        if (x.id >= 0 && (best.id < 0 || better(x, best))) best = x;
      };
#pragma unroll
      for (int o = 16; o >= 1; o /= 2)
        take(TopEntry{__shfl_xor_sync(0xffffffffu, best.v, o),
                      __shfl_xor_sync(0xffffffffu, best.id, o)});
      if (lane == 0) wbest[n & 1][warp] = best;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWarps; ++w) take(wbest[n & 1][w]);
      last = best;
      if (t == 0) {
        ids[n] = best.id;
        za[n] = best.v;
      }
    }
  }
  if (t == 0) ids[a.K] = a.tokens != nullptr ? static_cast<int>(y) : -1;
  __syncthreads();

  // ---- their logits in fp64
  const T* h = hidden + static_cast<size_t>(row) * a.H;
  for (int c = warp; c <= a.K; c += kWarps) {
    const int id = ids[c];
    double z = -CUDART_INF;
    if (id >= 0) {
      z = dot_part(h, weight + static_cast<size_t>(id) * a.H, a.H, lane);
#pragma unroll
      for (int o = 16; o >= 1; o /= 2) z += __shfl_xor_sync(0xffffffffu, z, o);
    }
    if (lane == 0) zx[c] = z;
  }
  __syncthreads();

  // ---- outputs.  xe: the listed logits as the softmax sees them
  const double ln2 = 0.693147180559945309417, log2e = 1.442695040888963407360;
  double x = 0.0;
  if (t <= a.K) {
    const double z = zx[t];
    x = (a.softcap > 0.f ? a.softcap * tanh(z / a.softcap)
                         : (z <= kNoMax ? -CUDART_INF : z)) * a.inv_temp;
    xe[t] = x;
  }
  __syncthreads();
  if (warp == 0) {
    st = Stats{M, ws[0], wt[0]};
#pragma unroll
    for (int w = 1; w < kWarps; ++w) {
      st.s += ws[w];
      st.t += wt[w];
    }
    auto sum = [](float v) {
#pragma unroll
      for (int o = 16; o >= 1; o /= 2) v += __shfl_xor_sync(0xffffffffu, v, o);
      return v;
    };
    const double Me = static_cast<double>(st.m) * a.inv_temp;  // the GEMM's maximum
    double m1 = -CUDART_INF;
    float s_rest = 0.f, t_rest = 0.f, z_sum = 0.f, dz_sum = 0.f, z_min = CUDART_INF_F;
    for (int c = lane; c < a.K; c += 32) {
      if (ids[c] < 0) continue;
      z_min = fminf(z_min, za[c]);
      const float L = a.softcap > 0.f ? gemm_softcap<T>(za[c], a.softcap) : za[c];
      const float d = exp2_arg(L, st.m, a.scale);
      const float e = exp2f(d);
      s_rest += e;
      t_rest = fmaf(e, d, t_rest);
      m1 = fmax(m1, xe[c]);
      z_sum += fabsf(za[c]);
      dz_sum += static_cast<float>(fabs(zx[c]) - fabs(static_cast<double>(za[c])));
    }
    // what the listed ones leave (a NaN sum stays NaN)
    s_rest = st.s - sum(s_rest);
    t_rest = st.t - sum(t_rest);
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) m1 = fmax(m1, __shfl_xor_sync(0xffffffffu, m1, o));
    // The token's own logit may not be listed and yet be the largest in fp64, among others that the
    // GEMM's rounding put before it.  It is then taken out of the rest (by what the GEMM can have
    // had for it: its fp64 value, but no more than the least listed one) and put back like those.
    const bool above = ids[a.K] >= 0 && xe[a.K] > m1 && m1 > -CUDART_INF;
    if (above) {
      m1 = xe[a.K];
#pragma unroll
      for (int o = 16; o >= 1; o /= 2)
        z_min = fminf(z_min, __shfl_xor_sync(0xffffffffu, z_min, o));
      const float z = fminf(static_cast<float>(zx[a.K]), z_min);
      const float d = exp2_arg(a.softcap > 0.f ? gemm_softcap<T>(z, a.softcap) : z, st.m, a.scale);
      const float e = exp2f(d);
      s_rest -= e;
      t_rest = fmaf(-e, d, t_rest);
    }
    if (s_rest < 0.f) s_rest = 0.f;
    if (t_rest > 0.f) t_rest = 0.f;
    // those that are put back: the listed ones, and the token's
    const int back_ids = above ? a.K + 1 : a.K;
    // The backward's logits: the same GEMM's, or, fp32, fp64 sums rounded once (simt_logit),
    // whose listed terms take the places of the fp32 sums' here too.
    Stats back = st;
    if constexpr (std::is_same_v<T, float>) {
      float m = -CUDART_INF_F, s = 0.f, e_d = 0.f;
      for (int c = lane; c < back_ids; c += 32)
        if (ids[c] >= 0) m = fmaxf(m, seen_logit(static_cast<float>(zx[c]), a.softcap));
#pragma unroll
      for (int o = 16; o >= 1; o /= 2) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (m == -CUDART_INF_F) m = st.m;
      for (int c = lane; c < back_ids; c += 32) {
        if (ids[c] < 0) continue;
        const float L = seen_logit(static_cast<float>(zx[c]), a.softcap);
        const float d = exp2_arg(L, m, a.scale), e = exp2f(d);
        s += e;
        e_d = fmaf(e, d, e_d);
      }
      const float d = fminf(exp2_arg(st.m, m, a.scale), 1.f), e = exp2f(d);
      back = Stats{m, sum(s) + s_rest * e, sum(e_d) + fmaf(s_rest, d, t_rest) * e};
    }
    // ... and with their fp64 values, at the largest of those (nothing is listed of a row that is
    // all masked, or NaN)
    if (m1 == -CUDART_INF) m1 = Me;
    // The rest is moved to that maximum.  The share that the tensor cores' truncation took of the
    // listed logits it took, on the average, of the others too; their mean (by probability) is
    // known, so their sum is moved by that as well.  An estimate, capped at H 2^-27: H / 16
    // additions, each of which takes half a step of 2^-23 on the average, of sums that grow to the
    // logit.  (fp32 sums are rounded to nearest: their errors say nothing of the others'.)
    float shift = static_cast<float>((Me - m1) * log2e);
    if constexpr (!std::is_same_v<T, float>) {
      z_sum = sum(z_sum);
      dz_sum = sum(dz_sum);
      if (a.softcap == 0.f && s_rest > 0.f && z_sum > 0.f) {
        const float share = fminf(fmaxf(dz_sum / z_sum, 0.f), a.H * 0x1p-27f);
        shift = fmaf(share, static_cast<float>(Me * log2e) + t_rest / s_rest, shift);
      }
    }
    // (At temperatures so low that the error of an fp32 logit divided by them counts, the
    // difference of two maxima says nothing: the rest must not outweigh the listed ones.)
    shift = fminf(fmaxf(shift, kLowExp2), 1.f);
    float s1 = 0.f, t1 = 0.f;
    for (int c = lane; c < back_ids; c += 32) {
      if (ids[c] < 0) continue;
      const float d = fmaxf(static_cast<float>((xe[c] - m1) * log2e), kLowExp2);
      const float e = exp2f(d);
      s1 += e;
      t1 = fmaf(e, d, t1);
    }
    const float down = exp2f(shift);
    s1 = sum(s1) + s_rest * down;
    t1 = sum(t1) + fmaf(s_rest, shift, t_rest) * down;
    if (lane == 0) {
      const float log2_s = log2f(s1), log2_b = log2f(back.s);  // of 0: -inf
      max_sh = m1;
      log_s_sh = ln2 * log2_s;
      a.lse[row] = static_cast<float>(m1 + log_s_sh);
      a.entropy[row] = static_cast<float>(ln2) * (log2_s - t1 / s1);
      if (a.saved_rows == 3) {
        a.saved[row] = back.m;
        a.saved[static_cast<size_t>(a.saved_stride) + row] = log2_b;
      } else {
        a.saved[row] = static_cast<float>(static_cast<double>(back.m) * a.inv_temp + ln2 * log2_b);
      }
      a.saved[static_cast<size_t>(a.saved_rows - 1) * a.saved_stride + row] =
          static_cast<float>(ln2) * (log2_b - back.t / back.s);
    }
  }
  __syncthreads();
  if (t == a.K && a.logprobs != nullptr)
    a.logprobs[row] = static_cast<float>((x - max_sh) - log_s_sh);
  if (t < a.K) {
    const int id = ids[t];
    auto ordered = [](double z) { return z != z ? -CUDART_INF : z; };  // NaN (inf - inf) last
    const double z = ordered(zx[t]);
    int rank = 0;
    for (int c = 0; c < a.K; ++c) {
      const int ic = ids[c];
      const double zc = ordered(zx[c]);
      if (c == t) continue;
      if (id < 0)  // places left empty keep their order, behind the others
        rank += (ic >= 0 || c < t) ? 1 : 0;
      else
        rank += (ic >= 0 && (zc > z || (zc == z && ic < id))) ? 1 : 0;
    }
    if (rank < a.top_k) {
      a.top_logprobs[static_cast<size_t>(row) * a.top_k + rank] =
          id < 0 ? -CUDART_INF_F : static_cast<float>((x - max_sh) - log_s_sh);
      a.top_ids[static_cast<size_t>(row) * a.top_k + rank] = id;
    }
  }
}

}  // namespace flce
