// Host side of the LM head's scoring operator (flce_logprobs_* in
// include/flce.h): workspace layout, choice of the schedule and launches.
// Included by flce_api.cu, whose helpers it uses.
//
// forward, bf16:  [row compaction] -> tc_gemm<ScoreEpi> -> score_finish
// forward, fp32:  score_simt -> score_finish
// backward:       flce_backward's, with per-row upstream gradients
#pragma once

namespace flce {
namespace {

// A token batch of at most one 128-row tile reads the weight once whatever the
// tile shape; single CTAs then spend half the tensor-core time of a pair on
// the tile's empty rows.
constexpr int kFewRows = BM;
// Longest runs (in tiles).  Longer ones mean fewer partial results, but CTAs that
// share a column tile fall out of step and its weight rows leave L2 before the
// last of them comes: 4096 x 4096 x 131072 took 2.47 ms with runs of 2, 2.54 with
// 4 and 2.65 with 8 (8192 x 2048 x 32000: no difference).  Longer runs all the
// same where the lists would take more than kMaxListBytes.  Where they still take more than
// kChunkListBytes (fp32 lists, which come in one length, too), the call works on its rows in
// chunks that share the lists' memory: 65536 x 131072 with 32 alternatives would keep 4.3 GB of
// them in bf16 and 9.7 GB in fp32.
constexpr int kMaxRun = 2;
constexpr int kLongestRun = 16;
constexpr size_t kMaxListBytes = size_t{512} << 20;
constexpr size_t kChunkListBytes = size_t{1} << 30;

struct ScorePlan {
  int cta_group;   // 1: 128 x 256 tiles of single CTAs, 2: 256-row tiles of pairs
  int bn;          // columns of a tile (fp32: of a block)
  RunMap map;      // runs of column tiles
  int runs;
  int slots;       // partial results per row
  int K;           // large logits kept for each row
  int cap;         // entries of a list
  int64_t rows;    // worked on at a time
  int tiles;       // fp32: column tiles of a score_tile block; 0: score_simt
  bool compact;    // rows without a token are left out of the GEMM
};

// score_simt's blocks: eight rows (two where eight rows of hidden do not fit shared
// memory) x 64 columns (8 x 1000 x 8009: 29 us, and 55 with 256, for which most SMs get no
// block; 8 x 4096 x 131072: 0.873 and 0.879 ms).
constexpr int kScoreRows = 8, kScoreCols = 64;
constexpr size_t kScoreSimtSmem = 200 * 1024;
size_t score_simt_smem(int rows, int64_t H) {
  return sizeof(float) * static_cast<size_t>(rows) * (static_cast<size_t>(H) + kScoreCols);
}
// Rows that are score_simt's; more are score_tile's.  24, or 16 where one block of eight rows fills
// an SM's shared memory (H > 3536, where its loads and products take turns) and where H < 512 makes
// neither long.  V = 32000, 24 rows, score_simt / score_tile: H = 512 68 / 88 us, 1000 140 / 152,
// 2048 224 / 275, 3500 440 / 454; but 3584 583 / 462, 4096 663 / 522, and 256 x 8009 24 / 20.  25 rows
// (a fourth group of eight): 2048 260 / 275, 2048 x 131072 1023 / 948, 3500 523 / 454.
int simt_rows(int64_t H) {
  constexpr size_t kSmSmem = 228 * 1024, kBlockOwn = 1024;  // of an SM, and what a block adds
  return H >= 512 && 2 * (score_simt_smem(kScoreRows, H) + kBlockOwn) <= kSmSmem ? 24 : 16;
}
// Column tiles of a block: 1, or kWideTiles where that still leaves kWideFrom blocks for every
// SM, which means longer lists but fewer of them (4096 x 1000 x 32000, K = 12: 9.7 ms
// with 1, 9.0 with 4; 500 x 1000 x 10007: 0.39 with 1, 0.48 with 4).
constexpr int kWideTiles = 4, kWideFrom = 8;

// Tiles of 256 columns, whose epilogue runs beside the next tile's MMAs, where a
// 512-column tile would expose a long one: with softcap (777 x 3584 x 256000: 1.06 against 1.11
// ms), and with alternatives over short K loops.  There, 256 / 512 columns, timed in turn: top 8,
// 8192 x 1024 x 32000 541 / 595 us, 8192 x 2048 x 32000 833 / 945; top 4, 1024 x 2048 x 131072
// 430 / 486; top 20, 1000 x 2048 x 32000 131 / 202, but top 8, 4096 x 1024 x 131072 1007 / 1002 and top
// 20, 4096 x 2048 x 131072 1896 / 1896; top 4, 4096 x 2560 x 65536 1066 / 1117.  Else as the forward's,
// 512 (top 4, 300 x 4096 x 131072: 0.36 against 0.38 ms; none, 8192 x 2048 x 32000: 0.72 against
// 0.76).
constexpr int64_t kShortH = 2048;

ScorePlan rows_plan(const Opts& o, int64_t N, int64_t H, int64_t V, bool bf16, int top_k,
                    bool softcap) {
  ScorePlan P{};
  P.rows = N;
  P.K = static_cast<int>(std::min<int64_t>(top_k > 0 ? top_k + kTopMargin : kPlainList, V));
  P.cap = bf16 ? top_list_cap(P.K) : P.K;
  if (!bf16 && N > simt_rows(H)) {
    const int64_t blocks = (N + kTileRows - 1) / kTileRows * ((V + kWideTiles * kTileCols - 1) /
                                                              (kWideTiles * kTileCols));
    P.tiles = blocks >= kWideFrom * kPlanSms ? kWideTiles : 1;
    P.bn = P.tiles * kTileCols;
    P.slots = static_cast<int>((V + P.bn - 1) / P.bn);
    return P;
  }
  if (!bf16) {
    P.bn = kScoreCols;
    P.slots = static_cast<int>((V + P.bn - 1) / P.bn);
    return P;
  }
  P.cta_group = (o.cta_group == 1 || N <= kFewRows) ? 1 : 2;
  P.bn = P.cta_group == 1 || softcap || (top_k > 0 && H <= kShortH) ? 256 : o.fwd_bn;
  P.compact = N > kFewRows && o.fwd_compact;
  const int64_t unit_rows = BM * P.cta_group, workers = kPlanSms / P.cta_group;
  const int64_t mt = std::max<int64_t>((N + unit_rows - 1) / unit_rows, 1);
  const int64_t nt = (V + P.bn - 1) / P.bn;
  // run_n: four of the longest runs for every worker at least; run_q (one for every
  // worker) of each smaller length
  const int64_t q = (workers + mt - 1) / mt;
  for (int64_t n = 1;; n *= 2) {
    const int64_t c0 = n == 1 ? nt : std::max<int64_t>(0, (nt - q * (n - 1)) / n);
    P.map = RunMap{static_cast<int>(n), static_cast<int>(c0), static_cast<int>(q)};
    P.runs = P.map.of_tile(static_cast<int>(nt - 1)) + 1;
    const size_t bytes = sizeof(TopEntry) * static_cast<size_t>(N) * 2 * P.runs * P.cap;
    if (n >= kLongestRun || 2 * n * 4 * workers > mt * nt) break;
    if (n >= kMaxRun && bytes <= kMaxListBytes) break;
  }
  P.slots = 2 * P.runs;
  return P;
}

size_t list_bytes(const ScorePlan& P) {
  return sizeof(TopEntry) * static_cast<size_t>(P.rows) * P.slots * P.cap;
}

// The plan of a call: that of all its rows, or of a chunk of them.
ScorePlan score_plan(const Opts& o, int64_t N, int64_t H, int64_t V, bool bf16, int top_k,
                     bool softcap) {
  ScorePlan P = rows_plan(o, N, H, V, bf16, top_k, softcap);
  while (P.rows > 1 && list_bytes(P) > kChunkListBytes) {
    int64_t rows = (P.rows + 1) / 2;
    if (rows > 256) rows = static_cast<int64_t>(align_up(static_cast<size_t>(rows), 256));
    P = rows_plan(o, rows, H, V, bf16, top_k, softcap);
  }
  return P;
}

// Workspace: header | group maxima (zeroed with the header) | statistics | lists |
// row compaction.
struct ScoreLayout {
  size_t seen, part, count, lists, perm, tokens_c, block_valid, n_valid_c, hidden_c, end;
};

ScoreLayout score_layout(const ScorePlan& P, int64_t H) {
  ScoreLayout L{};
  const size_t n = static_cast<size_t>(P.rows);
  size_t off = kHeaderBytes;
  L.seen = off;
  off = align_up(off + 4 * n * P.K, 256);
  L.part = off;
  off = align_up(off + sizeof(float4) * n * P.slots, 256);
  L.count = off;
  off = align_up(off + sizeof(int) * n * P.slots, 256);
  L.lists = off;
  off = align_up(off + sizeof(TopEntry) * n * P.slots * P.cap, 256);
  if (P.compact) {
    L.perm = off;
    off = align_up(off + 4 * n, 256);
    L.tokens_c = off;
    off = align_up(off + 8 * n, 256);
    L.block_valid = off;
    off = align_up(off + 4 * ((n + kCompactThreads - 1) / kCompactThreads), 256);
    L.n_valid_c = off;
    off = align_up(off + 8, 1024);
    L.hidden_c = off;
    off = align_up(off + 2 * n * static_cast<size_t>(H), 256);
  }
  L.end = off;
  return L;
}

// Tile indices and the partial results' row-slot product must stay in int range.
bool score_sizes_ok(int64_t N, int64_t H, int64_t V, int32_t dtype) {
  if (N < 0 || V < 1 || H < 8 || N > kMaxDim || V > kMaxDim || H > kMaxDim) return false;
  if (dtype == FLCE_BF16 ? H % 8 != 0 : H > kSimtMaxH) return false;
  if (((N + BM - 1) / BM) * ((V + BN - 1) / BN) > (int64_t{1} << 26)) return false;
  if ((V + BN - 1) / BN >= (1 << 22)) return false;  // (a row's slots are counted in 24 bits)
  return dtype == FLCE_BF16 || (N + 1) / 2 <= 65535;  // score_simt's grid
}

flce_status check_score(const Opts& o, const void* hidden, const void* weight, int64_t N,
                        int64_t H, int64_t V, float softcap, double temperature, int32_t dtype,
                        const void* ws) {
  (void)o;
  if (dtype != FLCE_BF16 && dtype != FLCE_FP32) return FLCE_ERR_ARG;
  if (!(softcap >= 0.f) || !(softcap < INFINITY)) return FLCE_ERR_ARG;
  // 1 / temperature must be a finite, normal fp32 number
  if (!(temperature >= 1e-30) || !(temperature <= 1e30)) return FLCE_ERR_ARG;
  if (!score_sizes_ok(N, H, V, dtype)) return FLCE_ERR_SHAPE;
  if (N > 0 && hidden == nullptr) return FLCE_ERR_ARG;
  if (weight == nullptr || ws == nullptr) return FLCE_ERR_ARG;
  if (!inputs_aligned(hidden, weight, dtype)) return FLCE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(ws) & 255u) != 0) return FLCE_ERR_ARG;
  return FLCE_OK;
}

// Threads that score_finish gives each row.  Up to kFinishFewRows rows (two for every SM),
// where a row's latency is what counts, 512 (32 rows, K = 24: 55 us with 128), and 1024 where
// 16 warps would take its dot products in two rounds (the same: 33 us with 512, 29 with 1024).
// Of more rows 64, or 128 from kFinishManyDots dot products (8192 rows, K = 4: 70 us with 64, 93
// with 128; 4096 rows, K = 12: 187 against 140).
constexpr int kFinishFewRows = 2 * kPlanSms;
constexpr int kFinishManyDots = 8;

template <class T, int kThreads>
cudaError_t run_finish_with(const void* hidden, const void* weight, const FinishArgs& a,
                       cudaStream_t st) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.N), 1, 1);
  cfg.blockDim = dim3(kThreads, 1, 1);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cudaError_t le = cudaSuccess;
  const cudaError_t e = launch(kFwdMerge, st, [&] {
    le = cudaLaunchKernelEx(&cfg, score_finish_kernel<T, kThreads>, static_cast<const T*>(hidden),
                            static_cast<const T*>(weight), a);
  });
  return le != cudaSuccess ? le : e;
}

template <class T>
cudaError_t run_finish(const void* hidden, const void* weight, const FinishArgs& a,
                       cudaStream_t st) {
  if (a.N <= kFinishFewRows)
    return a.K + 1 > 512 / 32 ? run_finish_with<T, 1024>(hidden, weight, a, st)
                              : run_finish_with<T, 512>(hidden, weight, a, st);
  return a.K + 1 >= kFinishManyDots ? run_finish_with<T, 128>(hidden, weight, a, st)
                                    : run_finish_with<T, 64>(hidden, weight, a, st);
}

flce_status score_bf16(DevInfo* d, Opts o, const ScorePlan& P, const ScoreLayout& L,
                       const void* hidden, const void* weight, const int64_t* tokens,
                       FinishArgs fin, char* w, cudaStream_t st) {
  const int n = fin.N, H = fin.H;
  const void* hid = hidden;
  long long* n_valid_c = nullptr;
  cudaError_t e = cudaSuccess;
  if (P.compact && tokens != nullptr) {
    int* perm = reinterpret_cast<int*>(w + L.perm);
    int64_t* tokens_c = reinterpret_cast<int64_t*>(w + L.tokens_c);
    int* block_valid = reinterpret_cast<int*>(w + L.block_valid);
    n_valid_c = reinterpret_cast<long long*>(w + L.n_valid_c);
    void* hidden_c = w + L.hidden_c;
    e = compact_rows(tokens, n, fin.V, fin.ignore_index, perm, tokens_c, block_valid, n_valid_c,
                     fin.status, st);
    if (e == cudaSuccess)
      e = launch(kHelper, st, [&] {
        gather_rows_kernel<<<n, 256, 0, st>>>(static_cast<const uint4*>(hidden), H / 8, n, perm,
                                              n_valid_c, static_cast<uint4*>(hidden_c), nullptr,
                                              H / 4, 0);
      });
    if (e != cudaSuccess) return cuda_fail(e);
    hid = hidden_c;
    fin.perm = perm;
    fin.n_valid = n_valid_c;
  }

  o.cta_group = P.cta_group;
  CUtensorMap ta, tb;
  if (!make_map(&ta, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, hid, H, n, static_cast<uint64_t>(H) * 2, BK,
                BM) ||
      !make_map(&tb, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, weight, H, fin.V,
                static_cast<uint64_t>(H) * 2, BK, b_box_rows(o)))
    return FLCE_ERR_CUDA;
  GemmArgs g{};
  g.k_blocks = (H + BK - 1) / BK;
  g.group_m = o.fwd_group;
  g.status = fin.status;
  g.timeout_ns = o.timeout_ns;
  g.tile_counter = o.fwd_dynamic ? ws_fwd_counter(w) : nullptr;
  g.run_n = P.map.n;
  g.run_c0 = P.map.c0;
  g.run_q = P.map.q;
  g.runs = P.runs;
  if (n_valid_c != nullptr) {
    g.rows_valid = n_valid_c;
    g.rows_host = n;
    g.rows_dim = kRowsM;
  }
  const GemmProblem prob{&ta, &tb, &ta, n, fin.V, g};
  const auto score = [&](auto epi) {
    using Epi = decltype(epi);
    const typename Epi::Params ep{n,
                                  fin.V,
                                  fin.softcap,
                                  fin.softcap > 0.f ? 1.0f / fin.softcap : 0.f,
                                  fin.scale,
                                  P.map,
                                  P.bn,
                                  P.slots,
                                  P.K,
                                  reinterpret_cast<float4*>(w + L.part),
                                  reinterpret_cast<int*>(w + L.count),
                                  reinterpret_cast<TopEntry*>(w + L.lists),
                                  reinterpret_cast<uint32_t*>(w + L.seen)};
    return run_gemm<Epi, false, false>(d, o, P.bn, kFwdGemm, prob, ep, nullptr, ep, st);
  };
  e = fin.softcap > 0.f ? score(ScoreEpi<true>{}) : score(ScoreEpi<false>{});
  if (e == cudaSuccess) e = run_finish<__nv_bfloat16>(hidden, weight, fin, st);
  return e == cudaSuccess ? FLCE_OK : cuda_fail(e);
}

// Loads of four floats: rows must start on 16-byte boundaries.
bool fp32_vectors(const void* hidden, const void* weight, int H) {
  return H % 4 == 0 && aligned16(hidden) && aligned16(weight);
}

template <int kRows>
cudaError_t run_score_simt(const void* hidden, const void* weight, const FinishArgs& a,
                           float4* part, int* count, TopEntry* lists, cudaStream_t st) {
  static_assert(2 * (kSimtMaxH + kScoreCols) * sizeof(float) <= kScoreSimtSmem, "two rows fit");
  const auto k =
      fp32_vectors(hidden, weight, a.H) ? score_simt_kernel<kRows, kScoreCols, 4>
                                        : score_simt_kernel<kRows, kScoreCols, 1>;
  const cudaError_t e = set_smem_attr(k, kScoreSimtSmem);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.slots), static_cast<unsigned>((a.N + kRows - 1) / kRows));
  return launch(kSimt, st, [&] {
    k<<<grid, kScoreThreads, score_simt_smem(kRows, a.H), st>>>(
        static_cast<const float*>(hidden), static_cast<const float*>(weight), a.N, a.H, a.V,
        a.softcap, a.scale, a.slots, a.K, a.cap, part, count, lists);
  });
}

template <int kTiles>
cudaError_t run_score_tile(const void* hidden, const void* weight, const FinishArgs& a,
                           float4* part, int* count, TopEntry* lists, cudaStream_t st) {
  const auto k = fp32_vectors(hidden, weight, a.H) ? score_tile_kernel<kTiles, 4>
                                                   : score_tile_kernel<kTiles, 1>;
  const cudaError_t e = set_smem_attr(k, kTileSmem<kTiles>);
  if (e != cudaSuccess) return e;
  const dim3 grid(static_cast<unsigned>(a.slots),
                  static_cast<unsigned>((a.N + kTileRows - 1) / kTileRows));
  return launch(kSimt, st, [&] {
    k<<<grid, kTileThreads, kTileSmem<kTiles>, st>>>(
        static_cast<const float*>(hidden), static_cast<const float*>(weight), a.N, a.H, a.V,
        a.softcap, a.scale, a.slots, a.K, a.cap, part, count, lists);
  });
}

flce_status score_fp32(const ScorePlan& P, const ScoreLayout& L, const void* hidden,
                       const void* weight, const FinishArgs& fin, char* w, cudaStream_t st) {
  float4* part = reinterpret_cast<float4*>(w + L.part);
  int* count = reinterpret_cast<int*>(w + L.count);
  TopEntry* lists = reinterpret_cast<TopEntry*>(w + L.lists);
  const bool eight = score_simt_smem(kScoreRows, fin.H) <= kScoreSimtSmem;
  const auto run =
      P.tiles == kWideTiles ? run_score_tile<kWideTiles>
      : P.tiles == 1        ? run_score_tile<1>
      : eight               ? run_score_simt<kScoreRows>
                            : run_score_simt<2>;
  cudaError_t e = run(hidden, weight, fin, part, count, lists, st);
  if (e == cudaSuccess) e = run_finish<float>(hidden, weight, fin, st);
  return e == cudaSuccess ? FLCE_OK : cuda_fail(e);
}

// The body of flce_logprobs_forward(_ex): saved_rows rows of N floats in `saved`.
flce_status score_forward(const void* hidden, const void* weight, const int64_t* tokens, int64_t N,
                          int64_t H, int64_t V, int64_t ignore_index, float softcap,
                          double temperature, int32_t top_k, int32_t dtype, float* logprobs,
                          float* entropy, float* lse, float* saved, int saved_rows,
                          float* top_logprobs, int64_t* top_ids, void* workspace,
                          size_t workspace_bytes, void* stream) {
  static_assert(FLCE_MAX_TOP_K == kMaxTopK, "header and kernels agree");
  const Opts o = opts();
  flce_status s = check_score(o, hidden, weight, N, H, V, softcap, temperature, dtype, workspace);
  if (s != FLCE_OK) return s;
  if (top_k < 0 || top_k > FLCE_MAX_TOP_K || top_k > V) return FLCE_ERR_ARG;
  if ((reinterpret_cast<uintptr_t>(tokens) & 7u) != 0 ||
      (reinterpret_cast<uintptr_t>(top_ids) & 7u) != 0)
    return FLCE_ERR_ARG;
  if (N > 0 && (entropy == nullptr || lse == nullptr || saved == nullptr)) return FLCE_ERR_ARG;
  if (N > 0 && (tokens == nullptr) != (logprobs == nullptr)) return FLCE_ERR_ARG;
  if (N > 0 && top_k > 0 && (top_logprobs == nullptr || top_ids == nullptr)) return FLCE_ERR_ARG;
  const bool bf16 = dtype == FLCE_BF16;
  const ScorePlan P = score_plan(o, N, H, V, bf16, top_k, softcap > 0.f);
  const ScoreLayout L = score_layout(P, H);
  if (workspace_bytes < L.end) return FLCE_ERR_WORKSPACE;
  DevInfo* d = nullptr;
  s = device_info(&d);
  if (s != FLCE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* w = static_cast<char*>(workspace);
  const float scale = static_cast<float>(1.4426950408889634074 / temperature);
  FinishArgs fin{};
  fin.H = static_cast<int>(H);
  fin.V = static_cast<int>(V);
  fin.ignore_index = ignore_index;
  fin.softcap = softcap;
  fin.inv_temp = 1.0 / temperature;
  fin.scale = scale;
  fin.slots = P.slots;
  fin.K = P.K;
  fin.cap = P.cap;
  fin.top_k = top_k;
  fin.part = reinterpret_cast<const float4*>(w + L.part);
  fin.count = reinterpret_cast<const int*>(w + L.count);
  fin.lists = reinterpret_cast<const TopEntry*>(w + L.lists);
  fin.saved_rows = saved_rows;
  fin.saved_stride = static_cast<int>(N);
  fin.status = ws_status(w);
  int64_t row0 = 0;
  do {
    const int64_t n = std::min(P.rows, N - row0);
    // tile counter, and the group maxima behind the header; the status word once
    const size_t keep = row0 == 0 ? 0 : sizeof(unsigned int);
    cudaError_t e = cudaMemsetAsync(
        w + keep, 0, L.seen + (bf16 ? 4 * static_cast<size_t>(n) * P.K : 0) - keep, st);
    if (e != cudaSuccess) return cuda_fail(e);
    if (N == 0) return FLCE_OK;
    fin.N = static_cast<int>(n);
    fin.tokens = tokens != nullptr ? tokens + row0 : nullptr;
    fin.logprobs = logprobs != nullptr ? logprobs + row0 : nullptr;
    fin.entropy = entropy + row0;
    fin.lse = lse + row0;
    fin.saved = saved + row0;
    if (top_k > 0) {
      fin.top_logprobs = top_logprobs + row0 * top_k;
      fin.top_ids = top_ids + row0 * top_k;
    }
    const char* hid = static_cast<const char*>(hidden) + row0 * H * (bf16 ? 2 : 4);
    s = bf16 ? score_bf16(d, o, P, L, hid, weight, fin.tokens, fin, w, st)
             : score_fp32(P, L, hid, weight, fin, w, st);
    if (s != FLCE_OK) return s;
    row0 += n;
  } while (row0 < N);
  return FLCE_OK;
}

// saved: as flce_logprobs_forward (saved_rows 2) or flce_logprobs_forward_ex (3) wrote it.
flce_status score_backward(const void* hidden, const void* weight, const int64_t* tokens,
                           const float* saved, int saved_rows, int64_t N, int64_t H, int64_t V,
                           int64_t ignore_index, float softcap, double temperature, int32_t dtype,
                           const float* d_logprobs, const float* d_entropy, float* d_hidden,
                           float* d_weight, int32_t flags, void* workspace,
                           size_t workspace_bytes, void* stream) {
  if (!(temperature >= 1e-30) || !(temperature <= 1e30)) return FLCE_ERR_ARG;
  RowGrads rg{};
  rg.d_logprobs = d_logprobs;
  rg.d_entropy = d_entropy;
  rg.inv_temp = static_cast<float>(1.0 / temperature);
  rg.scale = static_cast<float>(1.4426950408889634074 / temperature);
  rg.lse_unit = saved_rows == 3 ? 1.0f : kLog2e;
  // (a null saved is refused like a null lse)
  const float* lse = saved;
  if (saved != nullptr && N > 0) {
    rg.entropy = saved + (saved_rows - 1) * N;
    if (saved_rows == 3) {
      rg.row_max = saved;
      lse = saved + N;
    }
  }
  return backward_any(hidden, weight, tokens, lse, N, H, V, ignore_index, softcap, FLCE_SUM, dtype,
                      nullptr, 1.0f, -1, nullptr, d_hidden, d_weight, flags, workspace,
                      workspace_bytes, stream, &rg);
}

}  // namespace
}  // namespace flce

using namespace flce;

extern "C" {

size_t flce_logprobs_workspace_bytes(int64_t N, int64_t H, int64_t V, int32_t dtype,
                                     int32_t top_k) {
  if (dtype != FLCE_BF16 && dtype != FLCE_FP32) return 0;
  if (!score_sizes_ok(N, H, V, dtype)) return 0;
  if (top_k < 0 || top_k > FLCE_MAX_TOP_K || top_k > V) return 0;
  const bool bf16 = dtype == FLCE_BF16;
  const Opts o = opts();
  return std::max(score_layout(score_plan(o, N, H, V, bf16, top_k, false), H).end,
                  score_layout(score_plan(o, N, H, V, bf16, top_k, true), H).end);
}

flce_status flce_logprobs_forward(const void* hidden, const void* weight, const int64_t* tokens,
                                  int64_t N, int64_t H, int64_t V, int64_t ignore_index,
                                  float softcap, double temperature, int32_t top_k,
                                  int32_t dtype, float* logprobs, float* entropy, float* lse,
                                  float* saved, float* top_logprobs, int64_t* top_ids,
                                  void* workspace, size_t workspace_bytes, void* stream) {
  return score_forward(hidden, weight, tokens, N, H, V, ignore_index, softcap, temperature, top_k,
                       dtype, logprobs, entropy, lse, saved, 2, top_logprobs, top_ids, workspace,
                       workspace_bytes, stream);
}

flce_status flce_logprobs_backward(const void* hidden, const void* weight, const int64_t* tokens,
                                   const float* saved, int64_t N, int64_t H, int64_t V,
                                   int64_t ignore_index, float softcap, double temperature,
                                   int32_t dtype, const float* d_logprobs,
                                   const float* d_entropy, float* d_hidden, float* d_weight,
                                   int32_t flags, void* workspace, size_t workspace_bytes,
                                   void* stream) {
  return score_backward(hidden, weight, tokens, saved, 2, N, H, V, ignore_index, softcap,
                        temperature, dtype, d_logprobs, d_entropy, d_hidden, d_weight, flags,
                        workspace, workspace_bytes, stream);
}

flce_status flce_logprobs_forward_ex(const void* hidden, const void* weight, const int64_t* tokens,
                                     int64_t N, int64_t H, int64_t V, int64_t ignore_index,
                                     float softcap, double temperature, int32_t top_k,
                                     int32_t dtype, float* logprobs, float* entropy, float* lse,
                                     float* saved, float* top_logprobs, int64_t* top_ids,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  return score_forward(hidden, weight, tokens, N, H, V, ignore_index, softcap, temperature, top_k,
                       dtype, logprobs, entropy, lse, saved, 3, top_logprobs, top_ids, workspace,
                       workspace_bytes, stream);
}

flce_status flce_logprobs_backward_ex(const void* hidden, const void* weight, const int64_t* tokens,
                                      const float* saved, int64_t N, int64_t H, int64_t V,
                                      int64_t ignore_index, float softcap, double temperature,
                                      int32_t dtype, const float* d_logprobs,
                                      const float* d_entropy, float* d_hidden, float* d_weight,
                                      int32_t flags, void* workspace, size_t workspace_bytes,
                                      void* stream) {
  return score_backward(hidden, weight, tokens, saved, 3, N, H, V, ignore_index, softcap,
                        temperature, dtype, d_logprobs, d_entropy, d_hidden, d_weight, flags,
                        workspace, workspace_bytes, stream);
}

}  // extern "C"
