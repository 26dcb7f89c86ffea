// Ordering of token rows by one block: the embedding's sort, and the row
// compaction and label sort of the loss and the scoring operator.
#pragma once

#include "small_kernels.cuh"

namespace flce {

// Tokens in (id, token) order, those without an id (ignored, or out of range) behind
// the others: a stable radix sort, digits of `digit_bits` bits, by one block in shared
// memory.  Up to kSortMost tokens it does in one launch, of 16 us at 4096 tokens, what the
// kernels of small_kernels.cuh do in one per step of every digit; more tokens
// go through those.
constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kSortMost = 16384;
constexpr int kSortRounds = kSortMost / kSortThreads;  // tokens of a lane
constexpr int kMaxDigits = 256;
// Up to so many tokens each counts those before it, one step where the digits take one (live
// tokens first) to four; its time grows with their square.  Embedding gradients of V = 131072: 12.7
// against 16.7 us for 100 tokens, 14.7 / 16.8 for 256, 20.6 / 17.5 for 400 (V = 500: 12.6 / 14.7,
// 16.5 / 16.6, 20.8 / 16.8); forward of the loss at V = 500: 29.6 / 31.0 for 64 rows, 31.0 / 29.1
// for 200.
constexpr int kCountMost = 256, kCountMostLive = 128;
// Digit counts: a row of a count per warp for each digit, 17 words apart so that
// a warp's lanes, which read the same column of different rows, use all banks.
constexpr int kCntRow = kSortWarps + 2;
// two (key, index) buffers and the digit counts
constexpr size_t kSortSmem =
    2 * kSortMost * (sizeof(uint32_t) + sizeof(uint16_t)) + kMaxDigits * kCntRow * sizeof(uint16_t);

struct SortArgs {
  const int64_t* ids;  // (labels)
  int N;
  int64_t V;
  int64_t ignore_index;
  int passes, digit_bits;  // by_id; else one pass of one bit puts the live tokens first
  int by_id;
  long long* n_valid;
  unsigned int* status;
};

// put(i, key, token, live): the i-th in order, of `live` live ones.
template <class Put>
__device__ __forceinline__ void sort_block(const SortArgs& a, uint8_t* smem, const Put& put) {
  uint32_t* key[2] = {reinterpret_cast<uint32_t*>(smem),
                      reinterpret_cast<uint32_t*>(smem) + kSortMost};
  uint16_t* val[2] = {reinterpret_cast<uint16_t*>(smem + 8 * kSortMost),
                      reinterpret_cast<uint16_t*>(smem + 8 * kSortMost) + kSortMost};
  uint16_t* cnt = reinterpret_cast<uint16_t*>(smem + 12 * kSortMost);  // [digit][kCntRow]
  __shared__ int warp_sum[kSortWarps];
  __shared__ int live_sum;
  const int t = threadIdx.x, lane = t & 31, warp = t >> 5;
  if (t == 0) live_sum = 0;
  __syncthreads();
  // a warp's tokens are consecutive: warp * per_warp + 32 * round + lane
  const int rounds = (a.N + kSortThreads - 1) / kSortThreads;
  const int per_warp = rounds * 32;
  int live = 0;
  int64_t id_of[kSortRounds];  // all loads in flight
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int i = warp * per_warp + r * 32 + lane;
    id_of[r] = r < rounds && i < a.N ? a.ids[i] : a.ignore_index;
  }
#pragma unroll
  for (int r = 0; r < kSortRounds; ++r) {
    const int i = warp * per_warp + r * 32 + lane;
    // tokens left out sort behind the others
    uint32_t k = a.by_id ? static_cast<uint32_t>(a.V) : 1u;
    if (r < rounds && i < a.N) {
      const int64_t id = id_of[r];
      if (id != a.ignore_index) {
        if (id >= 0 && id < a.V) {
          k = a.by_id ? static_cast<uint32_t>(id) : 0u;
          ++live;
        } else {
          atomicOr(a.status, kStatusLabelRange);
        }
      }
      key[0][i] = k;
      val[0][i] = static_cast<uint16_t>(i);
    }
  }
  atomicAdd(&live_sum, live);
  if (a.N <= (a.by_id ? kCountMost : kCountMostLive)) {
    // (a broadcast of four keys at a time)
    static_assert(kCountMost <= kSortThreads && kCountMostLive <= kSortThreads, "a token a thread");
    __syncthreads();
    for (int i = a.N + t; i < (a.N + 3) / 4 * 4; i += kSortThreads) key[0][i] = 0xffffffffu;
    __syncthreads();
    if (t < a.N) {
      const uint32_t k = key[0][t];
      int rank = 0;
      for (int i = 0; i < a.N; i += 4) {
        const uint4 q = *reinterpret_cast<const uint4*>(key[0] + i);
        rank += (q.x < k || (q.x == k && i < t)) + (q.y < k || (q.y == k && i + 1 < t)) +
                (q.z < k || (q.z == k && i + 2 < t)) + (q.w < k || (q.w == k && i + 3 < t));
      }
      put(rank, k, t, live_sum);
    }
    if (t == 0) *a.n_valid = live_sum;
    return;
  }
  const int digits = 1 << a.digit_bits, mask = digits - 1;
  for (int ps = 0; ps < a.passes; ++ps) {
    const int src = ps & 1, shift = ps * a.digit_bits;
    for (int i = t; i < digits * kCntRow / 2; i += kSortThreads)
      reinterpret_cast<uint32_t*>(cnt)[i] = 0u;
    __syncthreads();
    // digits of this warp's tokens, and each one's rank among the warp's equal ones
    uint16_t rank[kSortRounds];
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      if (r >= rounds) break;
      const int i = warp * per_warp + r * 32 + lane;
      const int d = i < a.N ? static_cast<int>((key[src][i] >> shift) & mask) : digits;
      // lanes with the same digit, a ballot for each bit (__match_any_sync took
      // five times as long with 32 warps at it)
      unsigned peers = __ballot_sync(0xffffffffu, d < digits);
      for (int b = 0; b < a.digit_bits; ++b) {
        const bool bit = (d >> b) & 1;
        const unsigned ones = __ballot_sync(0xffffffffu, bit);
        peers &= bit ? ones : ~ones;
      }
      const int before = d < digits ? cnt[d * kCntRow + warp] : 0;
      rank[r] = static_cast<uint16_t>(before + __popc(peers & ((1u << lane) - 1u)));
      __syncwarp();
      if (d < digits && (peers >> lane) == 1u)  // the last of its peers
        cnt[d * kCntRow + warp] = static_cast<uint16_t>(before + __popc(peers));
      __syncwarp();
    }
    __syncthreads();
    // exclusive prefix sum over (digit, warp)
    // (four threads for each digit, eight warps' counts each)
    static_assert(kSortWarps == 32 && kMaxDigits * 4 == kSortThreads, "a thread's counts");
    uint32_t* mine = reinterpret_cast<uint32_t*>(cnt + (t >> 2) * kCntRow + (t & 3) * 8);
    uint32_t c[4] = {0u, 0u, 0u, 0u};
    int sum = 0;
    if (t < digits * 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[i] = mine[i];
        sum += static_cast<int>((c[i] & 0xffffu) + (c[i] >> 16));
      }
    }
    int incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    int before = warp_sum[lane];  // the sums of the warps up to `lane`
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, before, o);
      if (lane >= o) before += y;
    }
    before = __shfl_sync(0xffffffffu, before, (warp + 31) & 31);
    int base = incl - sum + (warp > 0 ? before : 0);
    if (t < digits * 4) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // (offsets stay below N <= 16384)
        const uint32_t first = base, second = base + (c[i] & 0xffffu);
        mine[i] = first | second << 16;
        base = static_cast<int>(second + (c[i] >> 16));
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kSortRounds; ++r) {
      if (r >= rounds) break;
      const int i = warp * per_warp + r * 32 + lane;
      if (i < a.N) {
        const uint32_t k = key[src][i];
        const int to = cnt[((k >> shift) & mask) * kCntRow + warp] + rank[r];
        key[src ^ 1][to] = k;
        val[src ^ 1][to] = val[src][i];
      }
    }
    __syncthreads();
  }
  const int fin = a.passes & 1;
  for (int i = t; i < a.N; i += kSortThreads)
    put(i, key[fin][i], static_cast<int>(val[fin][i]), live_sum);
  if (t == 0) *a.n_valid = live_sum;
}

// The rows that take part in the loss first, in (label, row) or row order, then the
// others: what compact_count, exclusive_scan, compact_scatter, the radix passes and
// apply_label_order do for more rows (perm, labels, lse and count are theirs).
__global__ void __launch_bounds__(kSortThreads)
    order_rows_kernel(const SortArgs a, const float* __restrict__ lse, int* __restrict__ perm,
                      int64_t* __restrict__ labels_c, float* __restrict__ lse_c) {
  extern __shared__ __align__(16) uint8_t smem_dyn[];
  sort_block(a, smem_dyn, [&](int i, uint32_t, int row, int live) {
    perm[i] = row;
    labels_c[i] = i < live ? a.ids[row] : a.ignore_index;
    if (lse_c != nullptr) lse_c[i] = i < live ? lse[row] : 0.f;
  });
}

}  // namespace flce
