// Kernels of the LM head's scoring operator (flce_logprobs_forward): log
// probabilities of given tokens, entropy and top alternatives of every row's
// distribution softmax(x), x = softcap(hidden . weight^T) / temperature.
//
//   ScoreEpi        epilogue of the tcgen05 GEMM (tc_gemm.cuh): streaming softmax
//                   statistics and a sorted list of the largest logits per row
//   score_simt      the same partial results for float32 inputs (CUDA cores)
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

// A running maximum that nothing has been merged into.  Finite, so that the
// differences of two maxima are never inf - inf.
constexpr float kNoMax = -1e30f;

// Order-preserving map of the floats (no NaN) onto unsigned; 0 lies below all.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float order_value(uint32_t k) {
  if (k == 0u) return -CUDART_INF_F;
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}

// Statistics of a set of values x (in the log2 domain): m their maximum,
// s = sum 2^(x - m), t = sum 2^(x - m) (x - m).  Then, in that domain,
//   lse = m + log2 s      entropy = log2 s - t / s
// (t <= 0: the entropy is a sum of two non-negative terms, nothing cancels).
struct Stats {
  float m, s, t;
};

// Moves (s, t) to the maximum `m1` >= st.m.
__device__ __forceinline__ void stats_rebase(Stats& st, float m1, float scale) {
  st.t = (st.t + st.s * (st.m - m1)) * scale;
  st.s *= scale;
  st.m = m1;
}

__device__ __forceinline__ void stats_merge(Stats& a, Stats b) {
  const float m1 = fmaxf(a.m, b.m);
  stats_rebase(a, m1, exp2f(a.m - m1));
  stats_rebase(b, m1, exp2f(b.m - m1));
  a.s += b.s;
  a.t += b.t;
}

// One entry of a list of large logits: the logit before softcap and temperature
// (both keep the order) and its vocabulary id; id -1: no entry.
struct TopEntry {
  float v;
  int id;
};

// ------------------------------------------------------------------ GEMM epilogue
// A CTA works on runs of consecutive column tiles of one row tile, so a thread
// sees one row's logits over a long range of columns and keeps that row's state
// in registers (statistics) and local memory (list) until the run ends:
// partial results per row and run instead of per row and tile, and a list that
// soon turns nearly every column down with one comparison of the maximum of 32.
// `thr` holds, per row, the largest known K-th best logit of any run (a lower
// bound of the row's K-th best): later runs start from it.  A logit below it
// cannot be among the K best; equal ones are kept, because a lower id wins.
// The K best by (logit, lowest id) are in the lists whatever the order in
// which runs are worked on, so the results do not depend on it.
template <bool kSoftcap, bool kTop>
struct ScoreEpi {
  static constexpr bool kRun = true;
  static constexpr int kEpiWarps = 8;
  static constexpr int kStagingPerWarp = 0;
  __device__ static void init_smem(uint8_t*) {}

  struct Params {
    int N;
    int V;
    float softcap;
    float inv_softcap;
    float scale;      // log2(e) / temperature
    int run_cols;     // columns of a full run
    int slots;        // 2 * runs per row (the two warps of a row, half a bank each)
    int K;            // list length
    float4* part;     // [N][slots]: m, s, t
    TopEntry* lists;  // [N][slots][K], best first
    uint32_t* thr;    // [N] order_key of the bound; zeroed before the launch
  };

  struct State {
    Stats st;
    float kth;        // the list's last value: -inf until it is full
    float told;       // largest bound written to or read from thr
    float lv[kTop ? kMaxTopList : 1];
    int li[kTop ? kMaxTopList : 1];
  };

  struct Pre {
    float thr;
  };
  __device__ static Pre prepare(const Params& p, int m_base, int q, int lane) {
    if constexpr (!kTop) return Pre{0.f};
    const int row = m_base + q * 32 + lane;
    if (row >= p.N) return Pre{CUDART_INF_F};
    return Pre{order_value(*reinterpret_cast<const volatile uint32_t*>(p.thr + row))};
  }

  // Keeps the list sorted by (value descending, id ascending); ids arrive in
  // ascending order, so an equal value goes behind those already there.
  __device__ static void insert(State& S, int K, float v, int id) {
    int i = K - 1;
    for (; i > 0 && S.lv[i - 1] < v; --i) {
      S.lv[i] = S.lv[i - 1];
      S.li[i] = S.li[i - 1];
    }
    S.lv[i] = v;
    S.li[i] = id;
    S.kth = S.lv[K - 1];
  }

  // The candidates among 32 columns starting at `col`, `mx` their maximum.
  __device__ static void scan32(State& S, const Params& p, float thr, const uint32_t (&r)[32],
                                float mx, int col) {
    if (!__any_sync(0xffffffffu, mx > S.kth && mx >= thr)) return;
    float qv[32];
    int qc[32];
    int n = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      const float v = __uint_as_float(r[j]);
      if (v > S.kth && v >= thr) {
        qv[n] = v;
        qc[n] = col + j;
        ++n;
      }
    }
    for (int i = 0; i < n; ++i)
      if (qv[i] > S.kth) insert(S, p.K, qv[i], qc[i]);
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

  // Adds n columns (values x / scale) whose maximum is mx to the statistics.
  template <int n>
  __device__ static void add(Stats& st, float scale, const uint32_t (&r)[n][32], float mx) {
    const float m1 = fmaxf(st.m, mx * scale);  // a NaN maximum (all NaN) leaves st.m
    stats_rebase(st, m1, ex2_approx(st.m - m1));
    float s4[4] = {0.f, 0.f, 0.f, 0.f}, t4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < n * 32; ++j) {
      const float d = max_nan(fmaf(__uint_as_float(r[j / 32][j % 32]), scale, -m1), kLowExp2);
      const float e = ex2_approx(d);
      s4[j & 3] += e;
      t4[j & 3] = fmaf(e, d, t4[j & 3]);
    }
    st.s += (s4[0] + s4[1]) + (s4[2] + s4[3]);
    st.t += (t4[0] + t4[1]) + (t4[2] + t4[3]);
  }

  __device__ static bool tile(const Params& p, const Pre& pre, int m_base, int col0,
                              uint32_t taddr, int q, int lane, int part, uint8_t*,
                              const CUtensorMap*, uint32_t tempty, State& S, bool,
                              const volatile int*, unsigned long long) {
    if (col0 >= p.V) {  // the second bank of a 512-column tile past the vocabulary
      release_tmem(tempty, lane);
      return true;
    }
    const int row = m_base + q * 32 + lane;
    const bool row_ok = row < p.N;
    const int run = col0 / p.run_cols;
    if (col0 == run * p.run_cols) {
      S.st = Stats{kNoMax, 0.f, 0.f};
      if constexpr (kTop) {
        S.kth = row_ok ? -CUDART_INF_F : CUDART_INF_F;  // rows past the end take nothing
        S.told = -CUDART_INF_F;
        for (int i = 0; i < p.K; ++i) {
          S.lv[i] = -CUDART_INF_F;
          S.li[i] = -1;
        }
      }
    }
    const int h0 = col0 + part * (BN / 2);  // this warp's first column
    const int ncols = max(0, min(BN / 2, p.V - h0));
    const uint32_t ta = taddr + part * (BN / 2);
    if constexpr (!kSoftcap) {
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
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) mx[c] = max32(r[c]);
      if constexpr (kTop) {
#pragma unroll
        for (int c = 0; c < 4; ++c) scan32(S, p, pre.thr, r[c], mx[c], h0 + c * 32);
      }
      add<4>(S.st, p.scale, r, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
    } else {
      // softcapped: 32-column chunks, the next chunk's TMEM load in flight; the
      // tanh body is kept rolled to bound code size
      auto chunk = [&](int c, uint32_t(&r)[1][32]) {
        if (c * 32 + 32 > ncols) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (c * 32 + j >= ncols) r[0][j] = __float_as_uint(-CUDART_INF_F);
        }
        if constexpr (kTop) scan32(S, p, pre.thr, r[0], max32(r[0]), h0 + c * 32);
#pragma unroll
        for (int j = 0; j < 32; ++j)
          r[0][j] = __float_as_uint(
              c * 32 + j < ncols
                  ? p.softcap * tanh_exp2(__uint_as_float(r[0][j]) * p.inv_softcap)
                  : -CUDART_INF_F);
        add<1>(S.st, p.scale, r, max32(r[0]));
      };
      constexpr int kChunks = BN / 2 / 32;
      uint32_t b0[1][32], b1[1][32];
      tmem_ld_x32(ta, b0[0]);
      tmem_ld_wait(b0[0]);
#pragma unroll 1
      for (int c = 0; c < kChunks; c += 2) {
        tmem_ld_x32(ta + (c + 1) * 32, b1[0]);
        chunk(c, b0);
        tmem_ld_wait(b1[0]);
        if (c + 2 < kChunks)
          tmem_ld_x32(ta + (c + 2) * 32, b0[0]);
        else
          release_tmem(tempty, lane);  // every column of this half is in registers
        chunk(c + 1, b1);
        if (c + 2 < kChunks) tmem_ld_wait(b0[0]);
      }
    }
    if constexpr (kTop) {
      // tell the other runs of this row
      S.told = fmaxf(S.told, pre.thr);
      if (row_ok && S.kth > S.told) {
        atomicMax(p.thr + row, order_key(S.kth));
        S.told = S.kth;
      }
    }
    const int run_end = min((run + 1) * p.run_cols, (p.V + BN - 1) / BN * BN);
    if (col0 + BN >= run_end && row_ok) {  // the run's last bank
      const size_t at = static_cast<size_t>(row) * p.slots + run * 2 + part;
      p.part[at] = make_float4(S.st.m, S.st.s, S.st.t, 0.f);
      if constexpr (kTop) {
        TopEntry* o = p.lists + at * p.K;
        for (int i = 0; i < p.K; ++i) o[i] = TopEntry{S.lv[i], S.li[i]};
      }
    }
    return true;
  }
};

// ------------------------------------------------------------------ fp32 inputs
// Partial results of kRows rows x kScoreCols columns per block (slot = column
// block): each warp computes the logits of four columns at a time against all
// rows (hidden rows in shared memory, the weight read once per block), then one
// warp per row reduces them.
constexpr int kScoreCols = 256;
constexpr int kScoreThreads = 256;

template <int kRows>
__global__ void __launch_bounds__(kScoreThreads)
    score_simt_kernel(const float* __restrict__ hidden, const float* __restrict__ weight, int N,
                      int H, int V, float softcap, float scale, int slots, int K,
                      float4* __restrict__ part, TopEntry* __restrict__ lists) {
  extern __shared__ float sh[];
  float* hs = sh;               // [kRows][H]
  float* zs = sh + kRows * H;   // [kRows][kScoreCols]
  const int row0 = blockIdx.y * kRows, v0 = blockIdx.x * kScoreCols;
  const int rows = min(kRows, N - row0), cols = min(kScoreCols, V - v0);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kRows * H; i += kScoreThreads)
    hs[i] = i < rows * H ? hidden[static_cast<size_t>(row0) * H + i] : 0.f;
  __syncthreads();
  constexpr int kC = 4;
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
    for (int k = lane; k < H; k += 32) {
      float wv[kC];
#pragma unroll
      for (int c = 0; c < kC; ++c) wv[c] = w[c][k];
#pragma unroll
      for (int r = 0; r < kRows; ++r) {
        const float h = hs[r * H + k];
#pragma unroll
        for (int c = 0; c < kC; ++c) acc[r][c] = fmaf(h, wv[c], acc[r][c]);
      }
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int c = 0; c < kC; ++c) {
        float a = acc[r][c];
#pragma unroll
        for (int o = 16; o >= 1; o /= 2) a += __shfl_xor_sync(0xffffffffu, a, o);
        if (lane == 0 && c0 + c < cols) zs[r * kScoreCols + c0 + c] = a;
      }
  }
  __syncthreads();
  for (int r = warp; r < rows; r += kScoreThreads / 32) {
    float* z = zs + r * kScoreCols;
    const size_t at = static_cast<size_t>(row0 + r) * slots + blockIdx.x;
    Stats st{kNoMax, 0.f, 0.f};
    for (int c = lane; c < cols; c += 32) st.m = fmaxf(st.m, capped(z[c], softcap) * scale);
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) st.m = fmaxf(st.m, __shfl_xor_sync(0xffffffffu, st.m, o));
    for (int c = lane; c < cols; c += 32) {
      const float d = max_nan(fmaf(capped(z[c], softcap), scale, -st.m), kLowExp2);
      const float e = exp2f(d);
      st.s += e;
      st.t = fmaf(e, d, st.t);
    }
#pragma unroll
    for (int o = 16; o >= 1; o /= 2) {
      st.s += __shfl_xor_sync(0xffffffffu, st.s, o);
      st.t += __shfl_xor_sync(0xffffffffu, st.t, o);
    }
    if (lane == 0) part[at] = make_float4(st.m, st.s, st.t, 0.f);
    // the K largest, one after another
    for (int i = 0; i < K; ++i) {
      float best = -CUDART_INF_F;
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
      if (lane == 0) {
        lists[at * K + i] = TopEntry{best, id < 0 ? -1 : v0 + id};
        if (id >= 0) z[id] = -CUDART_INF_F;
      }
      __syncwarp();
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
// ids, independent of how the logits were summed; it reads (top_k + margin + 1)
// weight rows per token against the V rows of the GEMM.
constexpr int kFinishThreads = 128;

struct FinishArgs {
  const int64_t* tokens;  // token order; null: none given
  const int* perm;        // compact row -> token row; null: the same
  const long long* n_valid;
  int N, H, V;
  int64_t ignore_index;
  float softcap;
  double inv_temp;   // 1 / temperature
  double nat;        // 1 / (temperature * ScoreEpi's scale): see the lse below
  int slots, K, top_k;
  const float4* part;
  const TopEntry* lists;
  float* logprobs;   // [N]; null without tokens
  float* entropy;    // [N]
  float* lse;        // [N]
  float* top_logprobs;  // [N, top_k]
  int64_t* top_ids;     // [N, top_k]
  unsigned int* status;
};

__device__ __forceinline__ double dot_part(const __nv_bfloat16* a, const __nv_bfloat16* b, int H,
                                           int lane) {
  double acc = 0.0;
  for (int k = lane * 8; k < H; k += 256) {  // H is a multiple of 8
    const uint4 x = *reinterpret_cast<const uint4*>(a + k);
    const uint4 y = *reinterpret_cast<const uint4*>(b + k);
    const __nv_bfloat162* x2 = reinterpret_cast<const __nv_bfloat162*>(&x);
    const __nv_bfloat162* y2 = reinterpret_cast<const __nv_bfloat162*>(&y);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 u = __bfloat1622float2(x2[j]), v = __bfloat1622float2(y2[j]);
      acc += static_cast<double>(u.x * v.x);
      acc += static_cast<double>(u.y * v.y);
    }
  }
  return acc;
}

__device__ __forceinline__ double dot_part(const float* a, const float* b, int H, int lane) {
  double acc = 0.0;
  for (int k = lane; k < H; k += 32)
    acc = fma(static_cast<double>(a[k]), static_cast<double>(b[k]), acc);
  return acc;
}

template <class T>
__global__ void __launch_bounds__(kFinishThreads)
    score_finish_kernel(const T* __restrict__ hidden, const T* __restrict__ weight,
                        const FinishArgs a) {
  constexpr int kWarps = kFinishThreads / 32;
  __shared__ Stats wst[kWarps];
  __shared__ float bv[2][kWarps];
  __shared__ int bi[2][kWarps], bt[2][kWarps];
  __shared__ int ids[kMaxTopList + 1];
  __shared__ double zx[kMaxTopList + 1];
  griddep_wait();
  const int j = blockIdx.x, t = threadIdx.x, lane = t & 31, warp = t >> 5;
  const int row = a.perm != nullptr ? a.perm[j] : j;
  bool live = a.perm == nullptr || j < *a.n_valid;
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
    }
    for (int i = t; i < a.top_k; i += kFinishThreads) {
      a.top_logprobs[static_cast<size_t>(row) * a.top_k + i] = 0.f;
      a.top_ids[static_cast<size_t>(row) * a.top_k + i] = -1;
    }
    return;
  }

  // ---- statistics
  Stats st{kNoMax, 0.f, 0.f};
  for (int i = t; i < a.slots; i += kFinishThreads) {
    const float4 v = a.part[static_cast<size_t>(j) * a.slots + i];
    stats_merge(st, Stats{v.x, v.y, v.z});
  }
#pragma unroll
  for (int o = 16; o >= 1; o /= 2)
    stats_merge(st, Stats{__shfl_down_sync(0xffffffffu, st.m, o),
                          __shfl_down_sync(0xffffffffu, st.s, o),
                          __shfl_down_sync(0xffffffffu, st.t, o)});
  if (lane == 0) wst[warp] = st;

  // ---- the K best entries: every thread keeps the best head of its lists
  if (a.K > 0) {
    const TopEntry* L = a.lists + static_cast<size_t>(j) * a.slots * a.K;
    // heads of the lists t, t + kFinishThreads, ...: an entry is taken by its
    // thread at most once, in list order, so a position per list would do; the
    // thread's last taken (value, id) says the same for all its lists
    float last_v = CUDART_INF_F;
    int last_id = -1;
    for (int n = 0; n < a.K; ++n) {
      float best = -CUDART_INF_F;
      int id = -1;
      for (int l = t; l < a.slots; l += kFinishThreads) {
        const TopEntry* e = L + static_cast<size_t>(l) * a.K;
        for (int i = 0; i < a.K; ++i) {
          const TopEntry x = e[i];
          if (x.id < 0) break;
          // not taken yet: behind (last_v, last_id) in the order
          if (x.v < last_v || (x.v == last_v && x.id > last_id)) {
            if (id < 0 || x.v > best || (x.v == best && x.id < id)) {
              best = x.v;
              id = x.id;
            }
            break;
          }
        }
      }
      int who = t;
#pragma unroll
      for (int o = 16; o >= 1; o /= 2) {
        const float v = __shfl_xor_sync(0xffffffffu, best, o);
        const int vi = __shfl_xor_sync(0xffffffffu, id, o);
        const int vw = __shfl_xor_sync(0xffffffffu, who, o);
        if (vi >= 0 && (id < 0 || v > best || (v == best && vi < id))) {
          best = v;
          id = vi;
          who = vw;
        }
      }
      if (lane == 0) {
        bv[n & 1][warp] = best;
        bi[n & 1][warp] = id;
        bt[n & 1][warp] = who;
      }
      __syncthreads();
      float gv = bv[n & 1][0];
      int gi = bi[n & 1][0], gw = bt[n & 1][0];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) {
        const float v = bv[n & 1][w];
        const int vi = bi[n & 1][w];
        if (vi >= 0 && (gi < 0 || v > gv || (v == gv && vi < gi))) {
          gv = v;
          gi = vi;
          gw = bt[n & 1][w];
        }
      }
      if (t == gw && gi >= 0) {
        last_v = gv;
        last_id = gi;
      }
      if (t == 0) ids[n] = gi;
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

  // ---- outputs
  st = wst[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) stats_merge(st, wst[w]);
  const double ln2 = 0.693147180559945309417;
  const double log2_s = st.s == 0.f ? -CUDART_INF : log2(static_cast<double>(st.s));
  // the maximum goes back by the fp32 scale that made it, so the rounding of
  // log2(e) / temperature does not reach the lse through it
  const double lse = static_cast<double>(st.m) * a.nat + ln2 * log2_s;
  auto logprob = [&](double z) -> float {
    const double L = a.softcap > 0.f ? a.softcap * tanh(z / a.softcap) : z;
    return static_cast<float>(L * a.inv_temp - lse);
  };
  if (t == 0) {
    a.lse[row] = static_cast<float>(lse);
    a.entropy[row] = static_cast<float>(ln2 * (log2_s - static_cast<double>(st.t) / st.s));
  }
  if (t == 32 && a.logprobs != nullptr) a.logprobs[row] = logprob(zx[a.K]);
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
      a.top_logprobs[static_cast<size_t>(row) * a.top_k + rank] = logprob(zx[t]);
      a.top_ids[static_cast<size_t>(row) * a.top_k + rank] = id;
    }
  }
}

}  // namespace flce
