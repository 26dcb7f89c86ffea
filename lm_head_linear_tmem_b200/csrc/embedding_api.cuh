// Host side of the embedding (flce_embedding_* in include/flce.h).  Included by
// flce_api.cu, whose helpers it uses.
//
// forward:   embed_lookup
// backward:  sort of the tokens by id, beside the zeros of the rows that no token
//            touches (overwriting calls) -> embed_segments -> embed_join
#pragma once

namespace flce {
namespace {

// Elements that a thread handles together: all rows must start on the vector's
// boundary, which 16-byte-aligned pointers and a multiple of 8 (or 4) elements
// give for bf16 and fp32 alike.
int embed_vec(int64_t H, std::initializer_list<const void*> ptrs) {
  uintptr_t all = 0;
  for (const void* p : ptrs) all |= reinterpret_cast<uintptr_t>(p);
  if (all % 16 != 0) return 1;
  return H % 8 == 0 ? 8 : (H % 4 == 0 ? 4 : 1);
}

bool embed_sizes_ok(int64_t N, int64_t H, int64_t V) {
  return N >= 0 && V >= 1 && H >= 1 && N <= kMaxDim && V <= kMaxDim && H <= (1 << 20);
}

// Workspace: header (status word, number of joins at 4) | sorted ids and tokens, live
// count | joins | touched rows | pieces of runs | and, for
// more tokens than one block sorts, the label sort's arrays.
struct EmbedLayout {
  size_t keys, vals, n_valid, joins, touched, part, keys1, vals1, perm, labels_c, block_valid, hist, end;
};

EmbedLayout embed_layout(int64_t N, int64_t H, int64_t V) {
  EmbedLayout L{};
  const size_t n = static_cast<size_t>(N);
  size_t off = kHeaderBytes;
  const auto take = [&off](size_t bytes) {
    const size_t at = off;
    off = align_up(off + bytes, 256);
    return at;
  };
  L.keys = take(4 * n);
  L.vals = take(4 * n);
  L.n_valid = take(8);
  L.joins = take(4 * ((n + kEmbedSeg - 1) / kEmbedSeg));
  L.touched = take(4 * ((static_cast<size_t>(V) + 31) / 32));
  L.part = take(((n + kEmbedSeg - 1) / kEmbedSeg) * 2 * static_cast<size_t>(H) * sizeof(float));
  if (N > kSortMost) {
    const size_t nblk = (n + kCompactThreads - 1) / kCompactThreads;
    L.keys1 = take(4 * n);
    L.vals1 = take(4 * n);
    L.perm = take(4 * n);
    L.labels_c = take(8 * n);
    L.block_valid = take(4 * nblk);
    L.hist = take(4 * static_cast<size_t>(kRadixBuckets) * nblk);
  }
  L.end = off;
  return L;
}

template <class T>
cudaError_t run_lookup(const void* weight, const int64_t* ids, int N, int H, int64_t V,
                       int64_t ignore_index, float scale, void* out, unsigned int* status,
                       cudaStream_t st) {
  const int vec = embed_vec(H, {weight, out});
  const int chunks = H / vec;
  int group = 8;  // threads of a row: about four chunks each, up to the whole block
  while (group < kLookupThreads && group * 4 < chunks) group *= 2;
  const int per_block = kLookupThreads / group;
  const unsigned grid = static_cast<unsigned>((static_cast<int64_t>(N) + per_block - 1) / per_block);
  const auto k = vec == 8 ? embed_lookup_kernel<T, 8>
                          : (vec == 4 ? embed_lookup_kernel<T, 4> : embed_lookup_kernel<T, 1>);
  return launch(kHelper, st, [&] {
    k<<<grid, kLookupThreads, 0, st>>>(static_cast<const T*>(weight), ids, N, H, V, ignore_index,
                                       scale, group, static_cast<T*>(out), status);
  });
}

// A launch that may start while the one before it drains (it waits by itself).
template <class Kern, class... Args>
cudaError_t launch_dependent(Kern k, dim3 grid, dim3 block, cudaStream_t st, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t le = cudaSuccess;
  const cudaError_t e = launch(kHelper, st, [&] { le = cudaLaunchKernelEx(&cfg, k, args...); });
  return le != cudaSuccess ? le : e;
}

// Blocks of embed_join along its list.
constexpr int kJoinBlocks = 64;

template <class TIn, class TOut, int kVec, bool kZeroVec>
cudaError_t run_sums(const void* d_out, int64_t N, int H, int64_t V, int64_t padding, float scale,
                     int accumulate, void* d_weight, const ZeroPlan& z, char* w,
                     const EmbedLayout& L, cudaStream_t st) {
  const uint32_t* keys = reinterpret_cast<const uint32_t*>(w + L.keys);
  const int* vals = reinterpret_cast<const int*>(w + L.vals);
  const long long* n_valid = reinterpret_cast<const long long*>(w + L.n_valid);
  float* part = reinterpret_cast<float*>(w + L.part);
  int* join_count = reinterpret_cast<int*>(w + 4);
  int* joins = reinterpret_cast<int*>(w + L.joins);
  // an id that no live token has, where there is no padding_idx
  const uint32_t pad = padding >= 0 ? static_cast<uint32_t>(padding) : 0xffffffffu;
  const int segs = static_cast<int>((N + kEmbedSeg - 1) / kEmbedSeg);
  const auto cols = [H](int threads) { return (H + threads * kVec - 1) / (threads * kVec); };
  const int ranges = z.chunks > 0 ? (z.chunks + z.range - 1) / z.range : 0;
  const int adders = segs * cols(kEmbedThreads);
  cudaError_t e = launch_dependent(
      embed_segments_kernel<TIn, TOut, kVec, kZeroVec>,
      dim3(static_cast<unsigned>(adders + ranges * (z.last - z.first))), dim3(kEmbedThreads), st,
      segs, adders, z, V, keys, vals, n_valid, static_cast<const TIn*>(d_out), H, pad, scale,
      accumulate, static_cast<TOut*>(d_weight), part, join_count, joins);
  const int along = segs > 1 ? std::min(segs, kJoinBlocks) : 0;  // (one segment joins nothing)
  const int joiners = along * cols(kJoinCols), zeros = ranges * (z.range - z.last);
  if (e == cudaSuccess && joiners + zeros > 0)
    e = launch_dependent(embed_join_kernel<TOut, kVec, kZeroVec>,
                         dim3(static_cast<unsigned>(joiners + zeros)), dim3(kJoinCols * kJoinWays),
                         st, along, joiners, z, V, keys, n_valid, H, scale, accumulate,
                         static_cast<TOut*>(d_weight), static_cast<const float*>(part),
                         static_cast<const int*>(join_count), static_cast<const int*>(joins));
  return e;
}

// Where the zeros go: about as many bytes beside the sort and the join as are
// written while those run (the sort about 6 us and 3 ns a token, the join 15 us, at
// about 6 TB/s), the rest beside the sums.  All of them with the first launch
// where it does not sort.
// 16384 tokens of a 131072 x 4096 bf16 gradient: 222 us, and 234 with all zeros in the
// first launch.
ZeroPlan zero_plan(int64_t N, int64_t V, int H, size_t elem, int ranges, bool sorts,
                   uint32_t* touched) {
  ZeroPlan z{};
  z.touched = touched;
  z.chunks = static_cast<int>((V + 31) / 32);
  z.range = (z.chunks + ranges - 1) / ranges;
  z.first = z.last = z.range;
  if (!sorts || N == 0) return z;
  const double chunk = 32.0 * H * static_cast<double>(elem) * ranges;  // a chunk of each range
  const auto share = [chunk](double us) { return static_cast<int>(us * 6e6 / chunk) + 1; };
  z.first = std::min(z.range, share(6.0 + 3e-3 * static_cast<double>(N)));
  z.last = std::max(z.first, z.range - share(15.0));
  return z;
}

template <class TOut>
cudaError_t run_embed_backward(DevInfo* d, const void* d_out, bool in_bf16, const SortArgs& a,
                               int H, int64_t padding, float scale, int accumulate,
                               void* d_weight, char* w, const EmbedLayout& L, cudaStream_t st) {
  const bool one_block = a.N <= kSortMost;
  uint32_t* sorted_keys = reinterpret_cast<uint32_t*>(w + L.keys);
  int* sorted_vals = reinterpret_cast<int*>(w + L.vals);
  cudaError_t e = cudaSuccess;
  if (!one_block) {
    const int n = a.N, nblk = (n + kCompactThreads - 1) / kCompactThreads;
    int* perm = reinterpret_cast<int*>(w + L.perm);
    int64_t* labels_c = reinterpret_cast<int64_t*>(w + L.labels_c);
    int* block_valid = reinterpret_cast<int*>(w + L.block_valid);
    int* hist = reinterpret_cast<int*>(w + L.hist);
    uint32_t* keys[2] = {sorted_keys, reinterpret_cast<uint32_t*>(w + L.keys1)};
    int* vals[2] = {sorted_vals, reinterpret_cast<int*>(w + L.vals1)};
    const int passes = (bit_length(static_cast<uint64_t>(a.V - 1)) + 7) / 8;
    const int first = passes & 1;  // so that the last pass ends in sorted_keys
    e = launch(kHelper, st, [&] {
      compact_count_kernel<<<nblk, kCompactThreads, 0, st>>>(a.ids, n, a.ignore_index, a.V,
                                                             a.status, block_valid);
    });
    if (e == cudaSuccess)
      e = launch(kHelper, st, [&] {
        exclusive_scan_kernel<<<1, kCompactThreads, 0, st>>>(block_valid, nblk, a.n_valid);
      });
    if (e == cudaSuccess)
      e = launch(kHelper, st, [&] {
        compact_scatter_kernel<<<nblk, kCompactThreads, 0, st>>>(
            a.ids, nullptr, n, a.ignore_index, block_valid, a.n_valid, perm, labels_c, nullptr,
            a.V, keys[first], vals[first]);
      });
    for (int ps = 0; ps < passes && e == cudaSuccess; ++ps) {
      const int src = (first + ps) & 1, shift = 8 * ps;
      e = launch(kHelper, st, [&] {
        radix_hist_kernel<<<nblk, kCompactThreads, 0, st>>>(keys[src], a.n_valid, shift, nblk,
                                                            hist);
      });
      if (e == cudaSuccess)
        e = launch(kHelper, st, [&] {
          exclusive_scan_kernel<<<1, kCompactThreads, 0, st>>>(hist, kRadixBuckets * nblk,
                                                               nullptr);
        });
      if (e == cudaSuccess)
        e = launch(kHelper, st, [&] {
          radix_scatter_kernel<<<nblk, kCompactThreads, 0, st>>>(
              keys[src], vals[src], keys[src ^ 1], vals[src ^ 1], a.n_valid, shift, nblk, hist);
        });
    }
    if (e != cudaSuccess) return e;
  }
  const bool zvec = reinterpret_cast<uintptr_t>(d_weight) % 16 == 0 &&
                    (static_cast<size_t>(H) * sizeof(TOut)) % 16 == 0;
  ZeroPlan z{};
  if (one_block || !accumulate) {
    const auto k = zvec ? embed_sort_zero_kernel<TOut, true> : embed_sort_zero_kernel<TOut, false>;
    e = set_smem_attr(k, kSortSmem);
    if (e != cudaSuccess) return e;
    const int sort = one_block ? 1 : 0;
    if (!accumulate)
      z = zero_plan(a.N, a.V, H, sizeof(TOut), d->sms - sort, one_block,
                    reinterpret_cast<uint32_t*>(w + L.touched));
    const size_t smem = one_block ? kSortSmem : kZeroWords * sizeof(uint32_t);
    const int grid = accumulate ? 1 : d->sms;
    e = launch(kHelper, st, [&] {
      k<<<grid, kSortThreads, smem, st>>>(a, sorted_keys, sorted_vals, sort, z, padding, H,
                                          static_cast<TOut*>(d_weight));
    });
    if (e != cudaSuccess) return e;
  }
  if (a.N == 0) return cudaSuccess;
  const int vec = embed_vec(H, {d_out, d_weight});
  const auto sums = [&](auto in) {
    using TIn = decltype(in);
    // (vector loads of 8 or 4 elements imply the zeros' 16-byte stores, but for
    // bf16 rows of a multiple of 4)
    const auto run = zvec ? (vec == 8 ? run_sums<TIn, TOut, 8, true>
                                      : (vec == 4 ? run_sums<TIn, TOut, 4, true>
                                                  : run_sums<TIn, TOut, 1, true>))
                          : (vec == 4 ? run_sums<TIn, TOut, 4, false>
                                      : run_sums<TIn, TOut, 1, false>);
    return run(d_out, a.N, H, a.V, padding, scale, accumulate, d_weight, z, w, L, st);
  };
  return in_bf16 ? sums(__nv_bfloat16{}) : sums(float{});
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

flce_status flce_embedding_forward(const void* weight, const int64_t* ids, int64_t N, int64_t H,
                                   int64_t V, int64_t ignore_index, float scale, int32_t dtype,
                                   void* out, uint32_t* status, void* stream) {
  if (dtype != FLCE_BF16 && dtype != FLCE_FP32) return FLCE_ERR_ARG;
  if (!(scale > -INFINITY) || !(scale < INFINITY)) return FLCE_ERR_ARG;
  if (!embed_sizes_ok(N, H, V)) return FLCE_ERR_SHAPE;
  if (weight == nullptr || (N > 0 && (ids == nullptr || out == nullptr))) return FLCE_ERR_ARG;
  const uintptr_t esize = dtype == FLCE_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(weight) % esize != 0 ||
      reinterpret_cast<uintptr_t>(out) % esize != 0 || reinterpret_cast<uintptr_t>(ids) % 8 != 0 ||
      reinterpret_cast<uintptr_t>(status) % 4 != 0)
    return FLCE_ERR_ARG;
  DevInfo* d = nullptr;
  const flce_status s = device_info(&d);
  if (s != FLCE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (status != nullptr) e = cudaMemsetAsync(status, 0, sizeof(uint32_t), st);
  if (e == cudaSuccess && N > 0)
    e = dtype == FLCE_BF16
            ? run_lookup<__nv_bfloat16>(weight, ids, static_cast<int>(N), static_cast<int>(H), V,
                                        ignore_index, scale, out, status, st)
            : run_lookup<float>(weight, ids, static_cast<int>(N), static_cast<int>(H), V,
                                ignore_index, scale, out, status, st);
  return e == cudaSuccess ? FLCE_OK : cuda_fail(e);
}

size_t flce_embedding_workspace_bytes(int64_t N, int64_t H, int64_t V) {
  return embed_sizes_ok(N, H, V) ? embed_layout(N, H, V).end : 0;
}

flce_status flce_embedding_backward(const void* d_out, const int64_t* ids, int64_t N, int64_t H,
                                    int64_t V, int64_t ignore_index, int64_t padding_idx,
                                    float scale, int32_t dtype, void* d_weight, int32_t flags,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (dtype != FLCE_BF16 && dtype != FLCE_FP32) return FLCE_ERR_ARG;
  if ((flags & ~(FLCE_ACCUMULATE_DWEIGHT | FLCE_DWEIGHT_BF16)) != 0) return FLCE_ERR_ARG;
  if (!(scale > -INFINITY) || !(scale < INFINITY)) return FLCE_ERR_ARG;
  if (!embed_sizes_ok(N, H, V)) return FLCE_ERR_SHAPE;
  if (padding_idx >= V) return FLCE_ERR_ARG;
  if (d_weight == nullptr || workspace == nullptr ||
      (N > 0 && (ids == nullptr || d_out == nullptr)))
    return FLCE_ERR_ARG;
  const bool in_bf16 = dtype == FLCE_BF16, out_bf16 = (flags & FLCE_DWEIGHT_BF16) != 0;
  if (reinterpret_cast<uintptr_t>(d_out) % (in_bf16 ? 2 : 4) != 0 ||
      reinterpret_cast<uintptr_t>(d_weight) % (out_bf16 ? 2 : 4) != 0 ||
      reinterpret_cast<uintptr_t>(ids) % 8 != 0 ||
      (reinterpret_cast<uintptr_t>(workspace) & 255u) != 0)
    return FLCE_ERR_ARG;
  const EmbedLayout L = embed_layout(N, H, V);
  if (workspace_bytes < L.end) return FLCE_ERR_WORKSPACE;
  DevInfo* d = nullptr;
  const flce_status s = device_info(&d);
  if (s != FLCE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(workspace);
  cudaError_t e = cudaMemsetAsync(w, 0, 16, st);  // status word, number of joins
  if (e != cudaSuccess) return cuda_fail(e);
  SortArgs a{};
  a.ids = ids;
  a.N = static_cast<int>(N);
  a.V = V;
  a.ignore_index = ignore_index;
  sort_by_id(a);
  a.n_valid = reinterpret_cast<long long*>(w + L.n_valid);
  a.status = ws_status(w);
  const int acc = (flags & FLCE_ACCUMULATE_DWEIGHT) != 0 ? 1 : 0;
  e = out_bf16 ? run_embed_backward<__nv_bfloat16>(d, d_out, in_bf16, a, static_cast<int>(H),
                                                   padding_idx, scale, acc, d_weight, w, L, st)
               : run_embed_backward<float>(d, d_out, in_bf16, a, static_cast<int>(H), padding_idx,
                                           scale, acc, d_weight, w, L, st);
  return e == cudaSuccess ? FLCE_OK : cuda_fail(e);
}

}  // extern "C"
