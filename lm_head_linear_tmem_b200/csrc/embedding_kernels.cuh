// Kernels of the embedding that shares the LM head's weight: row lookup with a
// scale, and the weight's gradient by sorted tokens.
//   forward   out[i]  = scale * W[ids[i]]
//   backward  dW[v]   = scale * sum over the tokens i with ids[i] = v, in order, of dOut[i]
// (Arrays that an earlier launch of the call writes are read through plain pointers:
// the launches overlap, so they are not constant for a kernel's lifetime.)
// Both move memory and compute next to nothing: the lookup reads and writes N rows,
// the gradient reads N rows and writes all V (overwritten) or those that the tokens
// touch (accumulated).  Sums are fp32, rounded once.
#pragma once

#include "row_order.cuh"

namespace flce {

// ---------------------------------------------------------------- element groups
// kVec consecutive elements of a row: 8 or 4 where rows and pointers allow vector
// accesses of 16 or 8 bytes of bf16 (32 or 16 bytes of fp32), else 1.
template <int kVec>
__device__ __forceinline__ void load_vec(const __nv_bfloat16* p, float (&v)[kVec]) {
  if constexpr (kVec == 1) {
    v[0] = __bfloat162float(*p);
  } else {
    uint32_t w[kVec / 2];
    if constexpr (kVec == 8) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w;
    } else {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x, w[1] = x.y;
    }
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) {
      const float2 f = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]));
      v[2 * i] = f.x;
      v[2 * i + 1] = f.y;
    }
  }
}

template <int kVec>
__device__ __forceinline__ void load_vec(const float* p, float (&v)[kVec]) {
  if constexpr (kVec == 1) {
    v[0] = *p;
  } else {
#pragma unroll
    for (int i = 0; i < kVec / 4; ++i) {
      const float4 x = reinterpret_cast<const float4*>(p)[i];
      v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
    }
  }
}

template <int kVec>
__device__ __forceinline__ void store_vec(__nv_bfloat16* p, const float (&v)[kVec]) {
  if constexpr (kVec == 1) {
    *p = __float2bfloat16_rn(v[0]);
  } else {
    uint32_t w[kVec / 2];
#pragma unroll
    for (int i = 0; i < kVec / 2; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if constexpr (kVec == 8)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

template <int kVec>
__device__ __forceinline__ void store_vec(float* p, const float (&v)[kVec]) {
  if constexpr (kVec == 1) {
    *p = v[0];
  } else {
#pragma unroll
    for (int i = 0; i < kVec / 4; ++i)
      reinterpret_cast<float4*>(p)[i] =
          make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
  }
}

// ---------------------------------------------------------------- lookup
// `group` threads (a power of two) for each row, kLookupThreads / group rows per
// block; each thread has up to four loads in flight.
constexpr int kLookupThreads = 128;

template <class T, int kVec>
__global__ void __launch_bounds__(kLookupThreads)
    embed_lookup_kernel(const T* __restrict__ weight, const int64_t* __restrict__ ids, int N, int H,
                        int64_t V, int64_t ignore_index, float scale, int group,
                        T* __restrict__ out, unsigned int* status) {
  const int t = threadIdx.x & (group - 1);
  const int row = blockIdx.x * (kLookupThreads / group) + threadIdx.x / group;
  if (row >= N) return;
  const int64_t id = ids[row];
  const bool live = id != ignore_index && id >= 0 && id < V;
  if (!live && id != ignore_index && t == 0 && status != nullptr)
    atomicOr(status, kStatusLabelRange);
  const T* src = weight + static_cast<size_t>(live ? id : 0) * H;
  T* dst = out + static_cast<size_t>(row) * H;
  const int chunks = H / kVec;
  for (int c = t; c < chunks; c += 4 * group) {
    float v[4][kVec];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (live && c + i * group < chunks) load_vec<kVec>(src + (c + i * group) * kVec, v[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (c + i * group >= chunks) break;
#pragma unroll
      for (int k = 0; k < kVec; ++k) v[i][k] = live ? v[i][k] * scale : 0.f;
      store_vec<kVec>(dst + (c + i * group) * kVec, v[i]);
    }
  }
}

// ---------------------------------------------------------------- zeros
// The rows that no live token touches (padding_idx counts as untouched) are zeroed in
// chunks of 32 rows, spread over the launches of the call so that stores go on while
// the sort, the sums and the join wait for their loads: chunk c of its range
// belongs to the first launch if c < first, to embed_join if c >= last, else to
// embed_segments.  A range is the chunks that one block of the first launch maps: it
// reads all ids and writes a word of touched rows for each.
struct ZeroPlan {
  uint32_t* touched;  // [chunks]
  int chunks;         // of the weight; 0: nothing is zeroed (accumulating calls)
  int range;          // chunks of a range
  int first, last;
};
constexpr int kZeroWords = 1024;  // of a range's map at a time

// Rows [32 c, 32 c + 32) of d_weight whose bit is not set, a warp per row.  kVec: 16-byte
// stores, where rows are whole multiples of them.
template <class TOut, bool kVec>
__device__ __forceinline__ void zero_chunk(uint32_t touched, int c, int64_t V, int H,
                                           TOut* d_weight, int warps) {
  const int lane = threadIdx.x & 31;
  for (int r = threadIdx.x >> 5; r < 32; r += warps) {
    const int64_t v = static_cast<int64_t>(c) * 32 + r;
    if (v >= V) return;
    if ((touched >> r) & 1u) continue;
    TOut* o = d_weight + static_cast<size_t>(v) * H;
    if constexpr (kVec) {
      const int n = H * static_cast<int>(sizeof(TOut)) / 16;
      for (int k = lane; k < n; k += 32) reinterpret_cast<uint4*>(o)[k] = make_uint4(0, 0, 0, 0);
    } else {
      for (int k = lane; k < H; k += 32) o[k] = TOut(0.f);
    }
  }
}

// Chunk number i of those that belong to [from, to) of every range.
template <class TOut, bool kVec>
__device__ __forceinline__ void zero_share(const ZeroPlan& z, int from, int to, int i, int64_t V,
                                           int H, TOut* d_weight, int threads) {
  const int c = i / (to - from) * z.range + from + i % (to - from);
  if (c < z.chunks) zero_chunk<TOut, kVec>(z.touched[c], c, V, H, d_weight, threads / 32);
}

// Block 0 sorts (if `sort`); the others, or all, map one range each and zero its first share.
template <class TOut, bool kVec>
__global__ void __launch_bounds__(kSortThreads)
    embed_sort_zero_kernel(const SortArgs a, uint32_t* keys, int* vals, int sort, const ZeroPlan z,
                           int64_t padding_idx, int H, TOut* __restrict__ d_weight) {
  extern __shared__ __align__(16) uint8_t smem_dyn[];
  griddep_launch_dependents();
  if (sort && blockIdx.x == 0) {
    sort_block(a, smem_dyn, [&](int i, uint32_t key, int token, int) {
      keys[i] = key;
      vals[i] = token;
    });
    return;
  }
  uint32_t* bits = reinterpret_cast<uint32_t*>(smem_dyn);
  const int64_t begin = static_cast<int64_t>(static_cast<int>(blockIdx.x) - sort) * z.range;
  const int64_t end = min(begin + z.range, static_cast<int64_t>(z.chunks));
  for (int64_t c0 = begin; c0 < end; c0 += kZeroWords) {
    const int words = static_cast<int>(min(end - c0, static_cast<int64_t>(kZeroWords)));
    const int64_t v0 = c0 * 32;
    __syncthreads();
    for (int i = threadIdx.x; i < words; i += kSortThreads) bits[i] = 0u;
    __syncthreads();
    for (int i = threadIdx.x; i < a.N; i += kSortThreads) {
      const int64_t id = a.ids[i];
      if (id >= v0 && id < v0 + static_cast<int64_t>(words) * 32 && id < a.V &&
          id != a.ignore_index && id != padding_idx)
        atomicOr(&bits[(id - v0) >> 5], 1u << ((id - v0) & 31));
    }
    __syncthreads();
    for (int i = threadIdx.x; i < words; i += kSortThreads) z.touched[c0 + i] = bits[i];
    for (int i = 0; i < words && c0 + i - begin < z.first; ++i)
      zero_chunk<TOut, kVec>(bits[i], static_cast<int>(c0 + i), a.V, H, d_weight,
                             kSortThreads / 32);
  }
}

// ---------------------------------------------------------------- sums
// Segments of kEmbedSeg sorted tokens x kEmbedThreads * kVec columns.  A run of one
// id inside a segment is finished there; a run that crosses segments leaves its
// pieces in part[segment][slot] (slot 0: the segment's first run, begun earlier;
// slot 1: its last run, going on), and embed_join adds them in order.  The segment
// where such a run begins enters itself in the list of joins, each a task of its
// own, whatever the list's order.
constexpr int kEmbedSeg = 32;
constexpr int kEmbedThreads = 128;

// scale * sum into row v: stored, or added to what is there.  Into fp32 by
// reductions that return nothing: no thread waits for the old value, and each
// element gets one addition per call, so the result stays reproducible (waiting,
// a segment of 32 different ids took 26 us).  Such a reduction adds the rounded product
// scale * sum and may flush subnormals; the loss's label terms are added to the same
// buffer that way.
template <class TOut, int kVec>
__device__ __forceinline__ void embed_put(TOut* d_weight, uint32_t v, int H, int col,
                                          const float (&sum)[kVec], float scale, int accumulate) {
  TOut* o = d_weight + static_cast<size_t>(v) * H + col;
  float x[kVec];
#pragma unroll
  for (int k = 0; k < kVec; ++k) x[k] = scale * sum[k];
  if (accumulate) {
    if constexpr (std::is_same_v<TOut, float>) {
      if constexpr (kVec == 1) {
        atomicAdd(o, x[0]);
      } else {
#pragma unroll
        for (int i = 0; i < kVec / 4; ++i)
          atomicAdd(reinterpret_cast<float4*>(o) + i,
                    make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]));
      }
      return;
    } else {
      float old[kVec];
      load_vec<kVec>(o, old);
#pragma unroll
      for (int k = 0; k < kVec; ++k) x[k] = fmaf(scale, sum[k], old[k]);
    }
  }
  store_vec<kVec>(o, x);
}

// Blocks 0 .. segs * (column blocks) - 1 add, those behind them zero.
template <class TIn, class TOut, int kVec, bool kZeroVec>
__global__ void __launch_bounds__(kEmbedThreads)
    embed_segments_kernel(int segs, int adders, const ZeroPlan z, int64_t V,
                          const uint32_t* keys, const int* vals,
                          const long long* n_valid, const TIn* __restrict__ d_out,
                          int H, uint32_t padding, float scale, int accumulate, TOut* d_weight,
                          float* part, int* join_count, int* joins) {
  __shared__ uint32_t key[kEmbedSeg + 2];  // with the tokens before and behind
  __shared__ int val[kEmbedSeg];
  griddep_wait();
  griddep_launch_dependents();
  if (static_cast<int>(blockIdx.x) >= adders) {
    zero_share<TOut, kZeroVec>(z, z.first, z.last, static_cast<int>(blockIdx.x) - adders, V, H,
                               d_weight, kEmbedThreads);
    return;
  }
  const int seg_id = static_cast<int>(blockIdx.x) % segs, col_id = static_cast<int>(blockIdx.x) / segs;
  const long long nv = *n_valid;
  const long long s0 = static_cast<long long>(seg_id) * kEmbedSeg;
  if (s0 >= nv) return;
  const int n = static_cast<int>(nv - s0 < kEmbedSeg ? nv - s0 : kEmbedSeg);
  constexpr uint32_t kNone = 0xffffffffu;
  for (int i = threadIdx.x; i < kEmbedSeg + 2; i += kEmbedThreads) {
    const long long j = s0 + i - 1;
    key[i] = (j >= 0 && j < nv) ? keys[j] : kNone;
    if (i < kEmbedSeg) val[i] = vals[s0 + min(i, n - 1)];  // (past the end: the last one again)
  }
  __syncthreads();
  if (col_id == 0 && threadIdx.x == 0) {
    const uint32_t last = key[n];
    const bool whole = key[0] == last && key[1] == last;  // began in an earlier segment
    if (n == kEmbedSeg && key[n + 1] == last && !whole && last != padding)
      joins[atomicAdd(join_count, 1)] = seg_id;
  }
  const int col = (col_id * kEmbedThreads + static_cast<int>(threadIdx.x)) * kVec;
  if (col >= H) return;
  float* seg = part + static_cast<size_t>(seg_id) * 2 * H + col;
  const TIn* src = d_out + col;
  float sum[kVec];
#pragma unroll
  for (int k = 0; k < kVec; ++k) sum[k] = 0.f;
  bool begun_before = key[0] == key[1];
  constexpr int kAhead = 8;  // loads in flight
  for (int b = 0; b < n; b += kAhead) {
    float x[kAhead][kVec];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      load_vec<kVec>(src + static_cast<size_t>(val[b + i]) * H, x[i]);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (b + i >= n) break;
#pragma unroll
      for (int k = 0; k < kVec; ++k) sum[k] += x[i][k];
      const uint32_t id = key[b + i + 1];
      if (id == key[b + i + 2] && b + i + 1 < n) continue;  // the run goes on here
      const bool goes_on = id == key[b + i + 2];            // ... in the next segment
      if (begun_before)
        store_vec<kVec>(seg, sum);
      else if (goes_on)
        store_vec<kVec>(seg + H, sum);
      else if (id != padding)
        embed_put<TOut, kVec>(d_weight, id, H, col, sum, scale, accumulate);
      begun_before = false;
#pragma unroll
      for (int k = 0; k < kVec; ++k) sum[k] = 0.f;
    }
  }
}

// The runs that cross segments: for each entry of the list, kJoinWays groups of
// threads each add a stretch of the run's pieces, and their sums are added in order.
constexpr int kJoinWays = 8;
constexpr int kJoinCols = 32;  // threads along the columns

// Blocks 0 .. adders - 1 (`along` of them along the list) add, those behind them zero.
template <class TOut, int kVec, bool kZeroVec>
__global__ void __launch_bounds__(kJoinWays * kJoinCols)
    embed_join_kernel(int along, int adders, const ZeroPlan z, int64_t V,
                      const uint32_t* keys, const long long* n_valid, int H, float scale,
                      int accumulate, TOut* d_weight, const float* part, const int* join_count,
                      const int* joins) {
  __shared__ float sums[kJoinWays][kJoinCols][kVec + 1];
  griddep_wait();
  if (static_cast<int>(blockIdx.x) >= adders) {
    zero_share<TOut, kZeroVec>(z, z.last, z.range, static_cast<int>(blockIdx.x) - adders, V, H,
                               d_weight, kJoinWays * kJoinCols);
    return;
  }
  const int count = *join_count;
  const long long nv = *n_valid;
  const int t = threadIdx.x, x = t % kJoinCols, y = t / kJoinCols;
  const int col = (static_cast<int>(blockIdx.x) / along * kJoinCols + x) * kVec;
  for (int j = static_cast<int>(blockIdx.x) % along; j < count; j += along) {
    const int seg = joins[j];
    const long long end = static_cast<long long>(seg + 1) * kEmbedSeg;
    const uint32_t id = keys[end - 1];
    // pieces: this segment's slot 1, then slot 0 of every later segment that starts
    // with the id (all threads look at once: a search by halves waits for 14 loads)
    int pieces = 1;
    for (bool more = true; more;) {
      const long long first = end + static_cast<long long>(pieces - 1 + t) * kEmbedSeg;
      const int n = __syncthreads_count(first < nv && keys[first] == id);
      pieces += n;
      more = n == kJoinWays * kJoinCols;
    }
    float sum[kVec];
#pragma unroll
    for (int k = 0; k < kVec; ++k) sum[k] = 0.f;
    if (col < H) {
      const int p0 = static_cast<int>(static_cast<long long>(pieces) * y / kJoinWays);
      const int p1 = static_cast<int>(static_cast<long long>(pieces) * (y + 1) / kJoinWays);
#pragma unroll 4
      for (int p = p0; p < p1; ++p) {
        float v[kVec];
        load_vec<kVec>(part + (static_cast<size_t>(seg + p) * 2 + (p == 0 ? 1 : 0)) * H + col, v);
#pragma unroll
        for (int k = 0; k < kVec; ++k) sum[k] += v[k];
      }
    }
#pragma unroll
    for (int k = 0; k < kVec; ++k) sums[y][x][k] = sum[k];
    __syncthreads();
    if (y == 0 && col < H) {
#pragma unroll
      for (int w = 1; w < kJoinWays; ++w)
#pragma unroll
        for (int k = 0; k < kVec; ++k) sum[k] += sums[w][x][k];
      embed_put<TOut, kVec>(d_weight, id, H, col, sum, scale, accumulate);
    }
    __syncthreads();
  }
}

}  // namespace flce
