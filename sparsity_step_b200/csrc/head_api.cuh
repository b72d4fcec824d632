// C ABI of the block-scaled 8-bit float linear and of the linear cross entropy (declared
// in include/bitlinear.h). Part of bitlinear_api.cu, whose checks, error text and TMA
// descriptor helpers it uses.
#pragma once

namespace {

inline int64_t round_up(int64_t v, int64_t m) { return (v + m - 1) / m * m; }

// Launch configuration of the head's kernels: clusters of `cluster` CTAs, set up while the
// kernel before them on the stream still runs (follow_stream() in the kernel).
void head_config(cudaLaunchConfig_t& cfg, cudaLaunchAttribute (&attr)[2], int64_t grid, int threads, size_t smem, int cluster,
                 cudaStream_t st) {
  cfg = cudaLaunchConfig_t{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = static_cast<unsigned>(cluster);
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
}

// A kernel without clusters or dynamic shared memory.
template <class... P, class... A>
bl_status launch_head(const char* what, void (*kern)(P...), int64_t grid, int threads, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  head_config(cfg, attr, grid, threads, 0, 0, st);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args...);
  if (e != cudaSuccess) return cuda_fail(e, what);
  return BL_OK;
}

// Once per device: the kernel's shared-memory limit and how many of its CTA pairs fit.
template <class K>
bl_status pair_setup(PerDeviceSetup& setup, K kern, int threads, size_t smem, int* pairs) {
  if (bl_status s = per_device_setup(setup, pairs, [&](int* r) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(head)");
        cudaLaunchConfig_t probe;
        cudaLaunchAttribute attr[2];
        head_config(probe, attr, 2 * (device_sm_count() / 2), threads, smem, 2, nullptr);
        int n = 0;
        e = cudaOccupancyMaxActiveClusters(&n, kern, &probe);
        if (e != cudaSuccess) return cuda_fail(e, "cudaOccupancyMaxActiveClusters(head)");
        *r = n > 0 ? n : 0;
        return BL_OK;
      }))
    return s;
  if (*pairs <= 0) return fail(BL_ERR_CUDA, "no CTA pair of this kernel fits on this device");
  return BL_OK;
}

// ------------------------------------------------------------------ 8-bit float linear

bl_status check_fp8_format(int f, const char* what) {
  if (f != BL_FP8_E4M3 && f != BL_FP8_E5M2) return fail(BL_ERR_INVALID_ARG, "%s must be BL_FP8_E4M3 or BL_FP8_E5M2", what);
  return BL_OK;
}

template <bool kWeight>
bl_status enqueue_fp8_quant(const bl::Fp8QuantArgs& a, bool e5m2, cudaStream_t st) {
  const int64_t tiles = ((a.rows + 127) / 128) * ((a.cols + 127) / 128);
  if (tiles > INT32_MAX) return fail(BL_ERR_UNSUPPORTED_SHAPE, "too much work in one call");
  auto kern = a.qt ? (e5m2 ? bl::fp8_quant_kernel<kWeight, true, true> : bl::fp8_quant_kernel<kWeight, false, true>)
                   : (e5m2 ? bl::fp8_quant_kernel<kWeight, true, false> : bl::fp8_quant_kernel<kWeight, false, false>);
  return launch_head("fp8 quant launch", kern, tiles, bl::kFp8QuantThreads, st, a);
}

// One operand of the pair product: K-major codes [rows, k] (row stride k) and their scales.
struct Fp8Operand {
  const uint8_t* q;
  const uint8_t* scales;
  int64_t rows;
  int e5m2;
};

// out[m, n] = A B^T with both operands' reduction of length k (codes [rows, k], k % 16 == 0).
struct Fp8Job {
  Fp8Operand A, B;
  int64_t k;
  void* out;
  bool f32;
};

// Tiles of the pair product: one or two accumulators of a multiple of 32 columns, whichever
// has the least modelled time in cycles. Per 128 of K a tile costs the larger of its MMAs (2
// a column) and its operand loads (128 rows of A and half its columns of B, 128 bytes each,
// at about 40 bytes a cycle); besides, a narrow tile costs about 1500 and a wide one, whose
// two accumulators are drained one after the other, 5000; whole waves of tiles over the
// pairs decide. Over 16 shapes (300 to 16384 rows, K 896 to 11008) the choice was within 3%
// of the best of all 14 tiles; the widest tile alone would be up to 1.5 times slower.
// Two products in one launch are taken by their common end (the levels of ce_shares.cuh),
// over the wider tiles: over 12 shapes the choice was within 1.3% of the best of 72 pairs of
// tiles on average (6% at most); the least sum of work, which may leave one deep tile behind,
// within 12% (46%).
struct Fp8Tiles {
  int halves, n_half[bl::kMaxFp8Group];
  int64_t tiles[bl::kMaxFp8Group], cost[bl::kMaxFp8Group];
};
// When `pairs` pairs end that take n0 tiles of cost c0 in turn and then n1 of c1, each on the
// least loaded pair: the least level below which n1 of them fit.
int64_t fp8_common_end(int64_t n0, int64_t c0, int64_t n1, int64_t c1, int64_t pairs) {
  const int64_t above = n0 % pairs, low = n0 / pairs * c0, high = above ? low + c0 : low;   // loads after the first product
  const int64_t alone = low + (n1 + pairs - above - 1) / (pairs - above) * c1;   // on the less loaded pairs
  if (alone < high + c1) return alone > high ? alone : high;
  int64_t level = (n0 * c0 + n1 * c1) / pairs;   // the mean load: no end is earlier
  if (level < high) level = high;
  for (;;) {
    const int64_t l = (level - low) / c1, h = (level - high) / c1;
    if (above * h + (pairs - above) * l >= n1) return level;
    const int64_t next_l = low + (l + 1) * c1, next_h = high + (h + 1) * c1;
    level = next_l < next_h ? next_l : next_h;
  }
}
Fp8Tiles fp8_tiles(const Fp8Job* jobs, int count, int pairs) {
  auto cover = [&](int j, int halves, int w, int64_t* tiles, int64_t* cost) {
    const int64_t cols = int64_t(halves) * w, k_blocks = (jobs[j].k + 127) / 128;
    *tiles = (jobs[j].A.rows + 255) / 256 * ((jobs[j].B.rows + cols - 1) / cols);
    const double mma = 2.0 * cols, load = (128 + cols / 2) * 128.0 / 40.0;
    *cost = static_cast<int64_t>(double(k_blocks) * (mma > load ? mma : load)) + (halves == 2 ? 5000 : 1500);
  };
  Fp8Tiles best{};
  int64_t best_end = INT64_MAX;
  for (int halves = 1; halves <= 2; ++halves)
    for (int w0 = 32; w0 <= bl::kF8MaxN; w0 += 32) {
      Fp8Tiles t{};
      t.halves = halves;
      t.n_half[0] = w0;
      cover(0, halves, w0, &t.tiles[0], &t.cost[0]);
      if (count == 1) {
        const int64_t end = (t.tiles[0] + pairs - 1) / pairs * t.cost[0];
        if (end <= best_end) best = t, best_end = end;
        continue;
      }
      if (w0 < 96 && halves * w0 < jobs[0].B.rows) continue;
      for (int w1 = 32; w1 <= bl::kF8MaxN; w1 += 32) {
        if (w1 < 96 && halves * w1 < jobs[1].B.rows) continue;
        t.n_half[1] = w1;
        cover(1, halves, w1, &t.tiles[1], &t.cost[1]);
        const int64_t end = fp8_common_end(t.tiles[0], t.cost[0], t.tiles[1], t.cost[1], pairs);
        if (end <= best_end) best = t, best_end = end;
      }
    }
  return best;
}

template <int kHalves>
bl_status launch_fp8_gemm(const Fp8Job* jobs, int count, const Fp8Tiles& t, int max_clusters, cudaStream_t st) {
  bl::Fp8Group G{};
  G.count = count;
  int64_t tiles = 0;
  for (int j = 0; j < count; ++j) {
    const Fp8Operand &A = jobs[j].A, &B = jobs[j].B;
    const int64_t k = jobs[j].k;
    const int n_half = t.n_half[j];
    const bool f32 = jobs[j].f32;
    bl::Fp8Problem& P = G.p[j];
    P.sa = reinterpret_cast<const uint32_t*>(A.scales);
    P.sb = reinterpret_cast<const uint32_t*>(B.scales);
    P.M = static_cast<int>(A.rows);
    P.N = static_cast<int>(B.rows);
    P.n_half = n_half;
    P.num_k_blocks = static_cast<int>((k + 127) / 128);
    P.num_m_blocks = static_cast<int>((A.rows + 255) / 256);
    P.num_n_blocks = static_cast<int>((B.rows + kHalves * n_half - 1) / (kHalves * n_half));
    P.a_e5m2 = A.e5m2;
    P.b_e5m2 = B.e5m2;
    P.out_f32 = f32 ? 1 : 0;
    bl::GemmArgs order{};
    set_raster(order, double(A.rows) * double(k), double(B.rows) * double(k));
    P.m_fastest = order.m_fastest;
    if (bl_status s = make_map(&P.tmA, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, A.q, k, A.rows, 128, 128)) return s;
    if (bl_status s = make_map(&P.tmB, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, B.q, k, B.rows, 128, n_half / 2)) return s;
    if (bl_status s = make_map_strided(&P.tmOut, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                                       f32 ? 4 : 2, jobs[j].out, B.rows, A.rows, B.rows, 32, 32,
                                       f32 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B))
      return s;
    tiles += t.tiles[j];
  }
  if (tiles > INT32_MAX) return fail(BL_ERR_UNSUPPORTED_SHAPE, "too much work in one call");
  if (max_clusters > bl::kMaxCePairs) max_clusters = bl::kMaxCePairs;
  const int clusters = static_cast<int>(tiles < max_clusters ? tiles : max_clusters);
  bl::ce_shares(G.share, t.tiles, t.cost, count, clusters);
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  head_config(cfg, attr, 2 * clusters, bl::kF8Threads, bl::gemm_fp8_smem_bytes(), 2, st);
  cudaError_t e = cudaLaunchKernelEx(&cfg, bl::gemm_fp8_kernel<kHalves>, G);
  if (e != cudaSuccess) return cuda_fail(e, "fp8 gemm launch");
  return BL_OK;
}

// One product, or two that share the pairs (the deeper one first).
bl_status enqueue_fp8_gemm(const Fp8Job* jobs, int count, cudaStream_t st) {
  static PerDeviceSetup setup[2];
  int pairs = 0, pairs2 = 0;
  if (bl_status s = pair_setup(setup[0], bl::gemm_fp8_kernel<1>, bl::kF8Threads, bl::gemm_fp8_smem_bytes(), &pairs)) return s;
  if (bl_status s = pair_setup(setup[1], bl::gemm_fp8_kernel<2>, bl::kF8Threads, bl::gemm_fp8_smem_bytes(), &pairs2)) return s;
  const Fp8Tiles tiles = fp8_tiles(jobs, count, pairs);
  return tiles.halves == 2 ? launch_fp8_gemm<2>(jobs, count, tiles, pairs2, st)
                           : launch_fp8_gemm<1>(jobs, count, tiles, pairs, st);
}

size_t fp8_scale_bytes(int64_t rows, int64_t cols) { return static_cast<size_t>((cols + 511) / 512) * 4 * rows; }

// ------------------------------------------------------------------ few tokens

constexpr int64_t kFewFp8Tokens = 4096, kFewCeTokens = 32, kFewQuantised = 16;
constexpr size_t kFewSmemTwo = 113 * 1024;   // two CTAs on an SM
constexpr size_t kFewSmemOne = 226 * 1024;

struct FewPlan {
  int split, stages, tok, part_blocks;
  size_t smem;
};
// How a product of few tokens is spread: K is split over a cluster while row blocks x split
// stays within two CTAs an SM and every CTA keeps two K blocks; then as many stages as fit
// beside the tokens' operand (`kept`: all of its K blocks, quantised in the kernel), two
// CTAs on an SM if that leaves three stages. Beyond 128 tokens only where the 128 x 128 tiles
// are fewer than half the SMs and K is long, so that the pair product's few tiles walk over
// all of K (1024 tokens 11008 -> 1024: 18.5 us here, 38.9 on the pair product; 896 -> 896:
// 11.0 and 7.3). False if it does not fit even when split by 8.
bool few_plan(bool fp8, bool kept, int64_t t, int64_t num_k_blocks, int64_t row_blocks, int sms, FewPlan* p) {
  if (t > (kept ? kFewQuantised : fp8 ? kFewFp8Tokens : kFewCeTokens) || num_k_blocks > 4096) return false;
  const int tok = t <= 16 ? 16 : t <= 32 ? 32 : t <= 64 ? 64 : 128;
  const int64_t blocks_mn = row_blocks * ((t + tok - 1) / tok);
  if (t > 128 && (2 * blocks_mn > sms || num_k_blocks < 32)) return false;
  int split = 1;
  while (split < 8 && blocks_mn * split * 2 <= 2 * int64_t(sms) && num_k_blocks >= 4 * split) split *= 2;
  for (; split <= 8; split *= 2) {
    const int blocks = bl::few_blocks_max(static_cast<int>(num_k_blocks), split);
    int part = 1;
    while (part < bl::kFewPartBlocks && bl::few_parts(fp8, blocks, part) * tok > 256) part *= 2;
    if (bl::few_parts(fp8, blocks, part) * tok > 256) continue;   // TMEM
    for (const size_t room : {kFewSmemTwo, kFewSmemOne}) {
      int stages = bl::kFewMaxStages;
      while (stages >= 3 && bl::few_smem_bytes(fp8, kept, tok, stages, blocks) > room) --stages;
      if (stages < 3) continue;
      *p = {split, stages, tok, part, bl::few_smem_bytes(fp8, kept, tok, stages, blocks)};
      return true;
    }
  }
  return false;
}

template <bool kFp8, int kTok>
bl_status launch_few(const bl::FewMaps& M, bl::FewArgs& a, const FewPlan& p, cudaStream_t st) {
  auto kern = bl::few_tokens_kernel<kFp8, kTok>;
  static PerDeviceSetup setup;
  int unused = 0;
  if (bl_status s = per_device_setup(setup, &unused, [&](int* r) {
        cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kFewSmemOne);
        if (e != cudaSuccess) return cuda_fail(e, "cudaFuncSetAttribute(few tokens)");
        *r = 1;
        return BL_OK;
      }))
    return s;
  a.split = p.split;
  a.stages = p.stages;
  const int blocks = bl::few_blocks_max(a.num_k_blocks, p.split);
  a.part_blocks = p.part_blocks;
  a.parts = bl::few_parts(kFp8, blocks, p.part_blocks);
  const int cols = a.parts * kTok;
  a.bufs = 2 * cols + (kFp8 ? 64 : 0) <= 256 ? 2 : 1;
  a.sf_col0 = static_cast<uint32_t>(a.bufs * cols);
  uint32_t need = a.sf_col0 + (kFp8 ? 64u : 0u);
  a.tmem_cols = 32;
  while (a.tmem_cols < need) a.tmem_cols *= 2;
  int64_t grid = int64_t(a.num_row_blocks) * p.split;
  const int64_t resident = int64_t(device_sm_count()) * (p.smem <= kFewSmemTwo ? 2 : 1);
  if (p.split == 1 && grid > resident) grid = resident;   // several row blocks per CTA
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  head_config(cfg, attr, grid, bl::kFewThreads, p.smem, p.split, st);
  cfg.gridDim.y = static_cast<unsigned>((a.t + kTok - 1) / kTok);
  cudaError_t e = cudaLaunchKernelEx(&cfg, kern, M, a);
  if (e != cudaSuccess) return cuda_fail(e, "few tokens launch");
  return BL_OK;
}

// Whether the product quantises bf16 activations itself: up to 16 tokens, where their codes
// fit whatever n is (a plan for one row block has the largest split, and more row blocks may
// have less of it, but never less than they need). More tokens go through the quantiser:
// every CTA would repeat their work (11008 -> 2048: 16 tokens 11 us either way, 32 tokens
// 25.6 us in the product, 20 through the quantiser).
bool few_quantises(int64_t t, int64_t k_in) {
  FewPlan p;
  return few_plan(true, true, t, (k_in + 127) / 128, 1, 148, &p);
}

// y of few tokens; *done is false (nothing enqueued) where the plan does not fit.
bl_status enqueue_fp8_few(const void* x, bool x_bf16, const uint8_t* x_scales, bool x5, const uint8_t* w_q,
                          const uint8_t* w_scales, bool w5, int64_t t, int64_t k, int64_t n, void* y, bool f32,
                          cudaStream_t st, bool* done) {
  *done = false;
  FewPlan p;
  if (!few_plan(true, x_bf16, t, (k + 127) / 128, (n + 127) / 128, device_sm_count(), &p)) return BL_OK;
  bl::FewMaps M{};
  for (int c = 0; c < 4; ++c)   // weight rows c, c + 4, ... (n % 16 == 0)
    if (bl_status s = make_map_strided(&M.w[c], CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, w_q + c * k, k, n / 4, 4 * k, 128, 32,
                                       CU_TENSOR_MAP_SWIZZLE_128B))
      return s;
  if (!x_bf16)
    if (bl_status s = make_map(&M.x, CU_TENSOR_MAP_DATA_TYPE_UINT8, 1, x, k, t, 128, p.tok)) return s;
  bl::FewArgs a{};
  a.x = x;
  a.xs = reinterpret_cast<const uint32_t*>(x_scales);
  a.x_bf16 = x_bf16 ? 1 : 0;
  a.ws = reinterpret_cast<const uint32_t*>(w_scales);
  a.a_e5m2 = w5;
  a.b_e5m2 = x5;
  a.t = static_cast<int>(t);
  a.k = static_cast<int>(k);
  a.n = static_cast<int>(n);
  a.num_k_blocks = static_cast<int>((k + 127) / 128);
  a.num_row_blocks = static_cast<int>((n + 127) / 128);
  a.y = y;
  a.y_f32 = f32 ? 1 : 0;
  *done = true;
  switch (p.tok) {
    case 16: return launch_few<true, 16>(M, a, p, st);
    case 32: return launch_few<true, 32>(M, a, p, st);
    case 64: return launch_few<true, 64>(M, a, p, st);
    default: return launch_few<true, 128>(M, a, p, st);
  }
}

// ------------------------------------------------------------------ linear cross entropy

// Rows of dl: up to kCeSplitTokens tokens have two, whatever t is.
int64_t ce_dl_rows(int64_t t) { return t >= 2 * bl::kCeSplitTokens ? t : t <= bl::kCeSplitTokens ? 2 * t : 2 * bl::kCeSplitTokens; }

// dl of the whole vocabulary up to kCeWholeBytes, else of a piece of kCePieceBytes at most
// (8192 x 2048 x 65536 backward: pieces of 32 MB 5.13 ms, 64 MB 5.00, 128 MB 4.55, 256 MB
// 4.61; 112 MB keeps the workspace below a third of the logits there).
constexpr int64_t kCeWholeBytes = int64_t(64) << 20, kCePieceBytes = int64_t(112) << 20;
// But never of fewer rows of the vocabulary than these: grad_W's product has a tile for 256 of
// them and 256 columns, each over all tokens, and below four rows of tiles most SMs have none
// (backward, pieces of at least 1024 / 512 / 256 rows: 65536 x 2048 x 1000 0.99 / 1.31 / 2.03
// ms, x 4000 2.87 / 3.51 / 3.52; 131072 x 1024 x 32768 30 / 47 / 89). So a piece of more than
// 57344 tokens exceeds kCePieceBytes, and a vocabulary of up to 1024 is never divided.
constexpr int64_t kCePieceRows = 1024;

// Vocabulary rows per piece of the backward pass: all of them, or a multiple of 256 and, above
// kCePieceRows, a quarter of the vocabulary at most, so that the two pieces held at a time
// stay well below the logits.
int64_t ce_piece(int64_t t, int64_t v) {
  const int64_t all = round_up(v, 256), row = 2 * (t > 0 ? ce_dl_rows(t) : 1);
  if (row * all <= kCeWholeBytes) return all;
  const int64_t fit = kCePieceBytes / row / 256 * 256, quarter = round_up((v + 3) / 4, 256);
  const int64_t p = fit < quarter ? fit : quarter;
  return p >= kCePieceRows ? p : all < kCePieceRows ? all : kCePieceRows;
}

// The few tokens' plan of the forward pass, if it takes that kernel.
bool few_ce_plan(int64_t t, int64_t k_in, int64_t v, FewPlan* p) {
  return few_plan(false, false, t, k_in / 64, (v + 127) / 128, device_sm_count(), p);
}
// Whether the targets' logits of more tokens are dot products too, in both passes, or the
// tensor cores', in which case the backward pass adds them up in the forward's parts, so that
// both passes' agree. Dot products read every token's rows of X and W once more, whatever v is;
// short parts make the product over v longer. Forward and backward of 8192 x 2048, dot
// products / parts: v 1000 184 / 176 us, 4096 424 / 421, 8192 828 / 826, 32768 2.99 / 3.05
// ms; 2047 x 1536 x 32003 580 / 590 us, 65536 x 2048 x 1000 1.38 / 1.20 ms.
bool ce_dots(int64_t v) { return v >= 8192; }

// Shapes of the head's operators: those of every entry point, with tokens up to 2^30 (the
// kernels count padded tiles in 32 bits).
bl_status check_head_shape(int64_t t, int64_t k_in, int64_t n_out) {
  if (t > (int64_t(1) << 30)) return fail(BL_ERR_UNSUPPORTED_SHAPE, "t=%lld out of range", (long long)t);
  return check_shape(t, k_in, n_out);
}

bl_status check_ce(int64_t t, int64_t k_in, int64_t v) {
  if (bl_status s = check_head_shape(t, k_in, 16)) return s;
  if (v < 1 || v > (int64_t(1) << 30)) return fail(BL_ERR_UNSUPPORTED_SHAPE, "v=%lld: need 1 <= v <= 2^30", (long long)v);
  return BL_OK;
}

bl_status launch_ce(bl::CeGroup& G, cudaStream_t st) {
  constexpr size_t smem = bl::gemm2_smem_bytes();
  static PerDeviceSetup setup;
  int max_clusters = 0;
  if (bl_status s = pair_setup(setup, bl::ce_gemm_kernel, bl::kGemmThreads, smem, &max_clusters)) return s;
  constexpr int64_t kTileCost = 4;   // a tile's start and epilogue, in K blocks
  int64_t n[bl::kMaxCeGroup], cost[bl::kMaxCeGroup], tiles = 0;
  for (int j = 0; j < G.count; ++j) {
    n[j] = int64_t(G.p[j].num_m_blocks) * G.p[j].num_n_blocks * G.p[j].splits;
    cost[j] = G.p[j].split_blocks + kTileCost;
    tiles += n[j];
  }
  if (tiles > INT32_MAX) return fail(BL_ERR_UNSUPPORTED_SHAPE, "too much work in one call");
  if (max_clusters > bl::kMaxCePairs) max_clusters = bl::kMaxCePairs;
  bl::ce_shares(G.share, n, cost, G.count, static_cast<int>(tiles < max_clusters ? tiles : max_clusters));
  cudaLaunchConfig_t cfg;
  cudaLaunchAttribute attr[2];
  head_config(cfg, attr, 2 * (tiles < max_clusters ? tiles : max_clusters), bl::kGemmThreads, smem, 2, st);
  cudaError_t e = cudaLaunchKernelEx(&cfg, bl::ce_gemm_kernel, G);
  if (e != cudaSuccess) return cuda_fail(e, "linear ce launch");
  return BL_OK;
}

// A bf16 operand [outer, inner] (row stride `stride` elements) as the product's A or B:
// K-major (inner is the reduction; boxes of 128 rows) or MN-major (outer is).
bl_status ce_operand(CUtensorMap* m, const void* p, int64_t inner, int64_t outer, int64_t stride, bool mn) {
  return make_map_strided(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, p, inner, outer, stride, 64, mn ? 64 : 128,
                          CU_TENSOR_MAP_SWIZZLE_128B);
}
bl_status ce_output(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t stride, bool f32) {
  return make_map_strided(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, f32 ? 4 : 2, p, cols,
                          rows, stride, f32 ? 32 : 64, 32, CU_TENSOR_MAP_SWIZZLE_128B);
}
void ce_shape(bl::CeProblem& P, int mode, int64_t m, int64_t n, int64_t k, bool a_mn, bool b_mn) {
  P.mode = mode;
  P.a_mn = a_mn ? 1 : 0;
  P.b_mn = b_mn ? 1 : 0;
  P.M = static_cast<int>(m);
  P.N = static_cast<int>(n);
  P.num_k_blocks = static_cast<int>((k + 63) / 64);
  P.num_m_blocks = static_cast<int>((m + 255) / 256);
  P.num_n_blocks = static_cast<int>((n + 255) / 256);
  P.splits = 1;
  P.split_blocks = P.num_k_blocks;
  P.live_m = P.live_k = 0;
  P.m_fastest = m <= n ? 1 : 0;   // the smaller operand stays in L2 while the other streams by once
}

// Layout of the workspaces (every part 256-byte aligned).
struct CeFwdSpace {
  size_t strips, target_logit, total;
};
CeFwdSpace ce_fwd_space(int64_t t, int64_t v) {
  CeFwdSpace s{};
  // 128 columns a strip; for few tokens as few as 16, an eighth of a row block
  const size_t per_t = t <= kFewCeTokens ? 8 * static_cast<size_t>((v + 127) / 128) : 2 * static_cast<size_t>((v + 255) / 256);
  const size_t n = per_t * static_cast<size_t>(t) * sizeof(float2);
  s.strips = 0;
  s.target_logit = round256(n);
  s.total = s.target_logit + round256(static_cast<size_t>(t) * sizeof(float));
  return s;
}
// Runs of a piece of the vocabulary that grad_X's product is split into when it has fewer
// tiles than there are CTA pairs (one token: 8 tiles of 2048 columns, each over the whole
// vocabulary); at least 16 K blocks a run. A function of the sizes alone: the order of the
// sums must not depend on the device.
struct CeRuns {
  int splits, blocks;   // runs of a whole piece, K blocks of a run
};
CeRuns ce_grad_x_runs(int64_t t, int64_t k_in, int64_t piece) {
  constexpr int64_t kPairs = 74;
  const int64_t tiles = ((t + 255) / 256) * ((k_in + 255) / 256), blocks = (piece + 63) / 64;
  int64_t s = tiles < kPairs ? kPairs / tiles : 1;
  if (s > blocks / 16) s = blocks / 16;
  if (s < 1) s = 1;
  const int64_t per = (blocks + s - 1) / s;
  return {static_cast<int>((blocks + per - 1) / per), static_cast<int>(per)};
}

struct CeBwdSpace {
  size_t head, place, from, target_dl, target, lse, grad, x, dl[2], acc, total;
};
CeBwdSpace ce_bwd_space(int64_t t, int64_t k_in, int64_t v, bool want_grad_x) {
  CeBwdSpace s{};
  const int64_t piece = ce_piece(t, v);
  const size_t bytes = round256(static_cast<size_t>(ce_dl_rows(t)) * static_cast<size_t>(piece) * 2);
  const size_t rows = static_cast<size_t>(round_up(t, 256));
  s.head = 0;   // the live rows' number, the largest |grad_loss| and the first low half
  s.place = 256;
  s.from = s.place + rows * 4;
  s.target_dl = s.from + rows * 4;
  s.target = s.target_dl + rows * 4;
  s.lse = s.target + rows * 4;
  s.grad = s.lse + rows * 4;
  s.x = s.grad + rows * 4;
  s.dl[0] = s.x + round256(rows * static_cast<size_t>(k_in) * 2);
  s.dl[1] = s.dl[0] + (piece < v ? bytes : 0);   // the next piece's dl is written while this one's is read
  s.acc = s.dl[1] + bytes;
  const size_t splits = static_cast<size_t>(ce_grad_x_runs(t, k_in, piece < v ? piece : v).splits);
  s.total = s.acc + (want_grad_x ? splits * rows * static_cast<size_t>(k_in) * 4 : 0);
  return s;
}

}  // namespace

extern "C" {

bl_status bitlinear_fp8_quant(const uint16_t* x, int64_t t, int64_t cols, int format, uint8_t* q_out, uint8_t* scales_out,
                              uint8_t* qt_out, uint8_t* scales_t_out, void* stream) {
  g_err[0] = 0;
  if (bl_status s = check_fp8_format(format, "format")) return s;
  if ((qt_out == nullptr) != (scales_t_out == nullptr))
    return fail(BL_ERR_INVALID_ARG, "give both qt_out and scales_t_out, or neither");
  if (cols < 16 || cols % 16 || cols > (int64_t(1) << 30))
    return fail(BL_ERR_UNSUPPORTED_SHAPE, "cols=%lld: need cols >= 16, cols %% 16 == 0", (long long)cols);
  if (bl_status s = check_head_shape(t, 64, 16)) return s;
  if (t == 0) return BL_OK;   // empty batch: the arrays may be NULL
  if (!x || !q_out || !scales_out) return fail(BL_ERR_INVALID_ARG, "x, q_out, scales_out are required");
  if (!aligned16(x) || !aligned16(q_out) || !aligned16(scales_out) || (qt_out && (!aligned16(qt_out) || !aligned16(scales_t_out))))
    return fail(BL_ERR_ALIGNMENT, "every pointer must be 16-byte aligned");
  const bl::Fp8QuantArgs a{x, t, cols, round_up(t, 16), q_out, scales_out, qt_out, scales_t_out};
  return enqueue_fp8_quant<false>(a, format == BL_FP8_E5M2, as_stream(stream));
}

bl_status bitlinear_fp8_quant_weight(const float* w, int64_t n_out, int64_t k_in, int format, uint8_t* q_out,
                                     uint8_t* scales_out, uint8_t* qt_out, uint8_t* scales_t_out, void* stream) {
  g_err[0] = 0;
  if (!w || !q_out || !scales_out) return fail(BL_ERR_INVALID_ARG, "w, q_out, scales_out are required");
  if (bl_status s = check_fp8_format(format, "format")) return s;
  if ((qt_out == nullptr) != (scales_t_out == nullptr))
    return fail(BL_ERR_INVALID_ARG, "give both qt_out and scales_t_out, or neither");
  if (bl_status s = check_shape(0, k_in, n_out)) return s;
  if (!aligned16(w) || !aligned16(q_out) || !aligned16(scales_out) || (qt_out && (!aligned16(qt_out) || !aligned16(scales_t_out))))
    return fail(BL_ERR_ALIGNMENT, "every pointer must be 16-byte aligned");
  const bl::Fp8QuantArgs a{w, n_out, k_in, n_out, q_out, scales_out, qt_out, scales_t_out};
  return enqueue_fp8_quant<true>(a, format == BL_FP8_E5M2, as_stream(stream));
}

size_t bitlinear_fp8_fwd_workspace_size(int64_t t, int64_t k_in, int x_type) {
  if (x_type != BL_X_BF16 || t <= 0 || k_in <= 0 || few_quantises(t, k_in)) return 0;
  return round256(static_cast<size_t>(t) * static_cast<size_t>(k_in)) + round256(fp8_scale_bytes(t, k_in));
}

bl_status bitlinear_fp8_fwd(const void* x, int x_type, const uint8_t* x_scales, const uint8_t* w_q, int w_format,
                            const uint8_t* w_scales, int64_t t, int64_t k_in, int64_t n_out, void* y_out, int y_dtype,
                            void* workspace, size_t workspace_bytes, void* stream) {
  g_err[0] = 0;
  if (x_type != BL_X_BF16 && x_type != BL_X_E4M3 && x_type != BL_X_E5M2)
    return fail(BL_ERR_INVALID_ARG, "x_type must be BL_X_BF16, BL_X_E4M3 or BL_X_E5M2");
  if (bl_status s = check_fp8_format(w_format, "w_format")) return s;
  if (y_dtype != BL_OUT_BF16 && y_dtype != BL_OUT_F32) return fail(BL_ERR_INVALID_ARG, "y_dtype must be BL_OUT_BF16 or BL_OUT_F32");
  if (!w_q || !w_scales) return fail(BL_ERR_INVALID_ARG, "w_q and w_scales are required");
  if (bl_status s = check_head_shape(t, k_in, n_out)) return s;
  if (!aligned16(w_q) || !aligned16(w_scales)) return fail(BL_ERR_ALIGNMENT, "every pointer must be 16-byte aligned");
  if (t == 0) return BL_OK;   // empty batch: the t-sized arrays may be NULL
  const bool bf16 = x_type == BL_X_BF16;
  if (!x || !y_out || (!bf16 && !x_scales)) return fail(BL_ERR_INVALID_ARG, "x, y_out and the scales of 8-bit x are required");
  const size_t need = bitlinear_fp8_fwd_workspace_size(t, k_in, x_type);
  if (need && (!workspace || workspace_bytes < need))
    return fail(BL_ERR_WORKSPACE, "workspace too small: %zu < %zu", workspace ? workspace_bytes : size_t(0), need);
  if (!aligned16(x) || !aligned16(y_out) || (!bf16 && !aligned16(x_scales)) || (need && !aligned16(workspace)))
    return fail(BL_ERR_ALIGNMENT, "every pointer must be 16-byte aligned");
  cudaStream_t st = as_stream(stream);
  const bool w5 = w_format == BL_FP8_E5M2, x5 = x_type == BL_X_E5M2, f32 = y_dtype == BL_OUT_F32;
  if (need) {   // codes of bf16 x in the workspace first
    uint8_t* xq = static_cast<uint8_t*>(workspace);
    uint8_t* xs = xq + round256(static_cast<size_t>(t) * static_cast<size_t>(k_in));
    const bl::Fp8QuantArgs a{x, t, k_in, round_up(t, 16), xq, xs, nullptr, nullptr};
    if (bl_status s = enqueue_fp8_quant<false>(a, false, st)) return s;
    x = xq;
    x_scales = xs;
  }
  bool done = false;
  if (bl_status s = enqueue_fp8_few(x, bf16 && !need, x_scales, x5, w_q, w_scales, w5, t, k_in, n_out, y_out, f32, st, &done))
    return s;
  if (done) return BL_OK;
  const Fp8Job job{{static_cast<const uint8_t*>(x), x_scales, t, x5}, {w_q, w_scales, n_out, w5}, k_in, y_out, f32};
  return enqueue_fp8_gemm(&job, 1, st);
}

bl_status bitlinear_fp8_bwd(const uint8_t* dy_q, const uint8_t* dy_scales, const uint8_t* dy_qt, const uint8_t* dy_scales_t,
                            int dy_format, const uint8_t* x_qt, const uint8_t* x_scales_t, int x_format, const uint8_t* w_qt,
                            const uint8_t* w_scales_t, int w_format, int64_t t, int64_t k_in, int64_t n_out, uint16_t* grad_x,
                            void* grad_w, int grad_w_dtype, void* stream) {
  g_err[0] = 0;
  if (!grad_x && !grad_w) return fail(BL_ERR_INVALID_ARG, "request grad_x, grad_w or both");
  if (bl_status s = check_fp8_format(dy_format, "dy_format")) return s;
  if (grad_x)
    if (bl_status s = check_fp8_format(w_format, "w_format")) return s;
  if (grad_w) {
    if (bl_status s = check_fp8_format(x_format, "x_format")) return s;
    if (grad_w_dtype != BL_OUT_BF16 && grad_w_dtype != BL_OUT_F32)
      return fail(BL_ERR_INVALID_ARG, "grad_w_dtype must be BL_OUT_BF16 or BL_OUT_F32");
  }
  if (bl_status s = check_head_shape(t, k_in, n_out)) return s;
  if (grad_x && (!w_qt || !w_scales_t || (t != 0 && (!dy_q || !dy_scales))))
    return fail(BL_ERR_INVALID_ARG, "grad_x needs dy_q, dy_scales, w_qt and w_scales_t");
  if (grad_w && t != 0 && (!dy_qt || !dy_scales_t || !x_qt || !x_scales_t))
    return fail(BL_ERR_INVALID_ARG, "grad_w needs dy_qt, dy_scales_t, x_qt and x_scales_t");
  const void* all[] = {dy_q, dy_scales, dy_qt, dy_scales_t, x_qt, x_scales_t, w_qt, w_scales_t, grad_x, grad_w};
  for (const void* p : all)
    if (p && !aligned16(p)) return fail(BL_ERR_ALIGNMENT, "every pointer must be 16-byte aligned");
  cudaStream_t st = as_stream(stream);
  const int d5 = dy_format == BL_FP8_E5M2;
  if (t == 0) {
    if (grad_w) {
      cudaError_t e = cudaMemsetAsync(grad_w, 0, static_cast<size_t>(n_out) * k_in * (grad_w_dtype == BL_OUT_F32 ? 4 : 2), st);
      if (e != cudaSuccess) return cuda_fail(e, "grad_w zero");
    }
    return BL_OK;
  }
  const bool w5 = w_format == BL_FP8_E5M2;
  bool done = false;   // grad_x of few tokens
  if (grad_x)
    if (bl_status s = enqueue_fp8_few(dy_q, false, dy_scales, d5, w_qt, w_scales_t, w5, t, n_out, k_in, grad_x, false, st, &done))
      return s;
  const Fp8Job x_job{{dy_q, dy_scales, t, d5}, {w_qt, w_scales_t, k_in, w5}, n_out, grad_x, false};
  const Fp8Job w_job{{dy_qt, dy_scales_t, n_out, d5}, {x_qt, x_scales_t, k_in, x_format == BL_FP8_E5M2}, round_up(t, 16), grad_w,
                     grad_w_dtype == BL_OUT_F32};
  Fp8Job jobs[bl::kMaxFp8Group];
  int count = 0;
  const bool x_first = n_out >= t;   // the deeper product's tiles go first
  if (grad_x && !done && x_first) jobs[count++] = x_job;
  if (grad_w) jobs[count++] = w_job;
  if (grad_x && !done && !x_first) jobs[count++] = x_job;
  return count ? enqueue_fp8_gemm(jobs, count, st) : BL_OK;
}

size_t bitlinear_linear_ce_fwd_workspace_size(int64_t t, int64_t v) {
  if (t <= 0 || v <= 0) return 0;
  return ce_fwd_space(t, v).total;
}

bl_status bitlinear_linear_ce_fwd(const uint16_t* x, const uint16_t* w, const int64_t* targets, int64_t t, int64_t k_in,
                                  int64_t v, float* loss_out, float* lse_out, void* workspace, size_t workspace_bytes,
                                  void* stream) {
  g_err[0] = 0;
  if (!w) return fail(BL_ERR_INVALID_ARG, "w is required");
  if (bl_status s = check_ce(t, k_in, v)) return s;
  if (!aligned16(w)) return fail(BL_ERR_ALIGNMENT, "every pointer must be 16-byte aligned");
  if (t == 0) return BL_OK;   // empty batch: the t-sized arrays may be NULL
  if (!x || !targets || !loss_out || !lse_out) return fail(BL_ERR_INVALID_ARG, "x, targets, loss_out, lse_out are required");
  const CeFwdSpace sp = ce_fwd_space(t, v);
  if (!workspace || workspace_bytes < sp.total)
    return fail(BL_ERR_WORKSPACE, "workspace too small: %zu < %zu", workspace ? workspace_bytes : size_t(0), sp.total);
  if (!aligned16(x) || !aligned16(targets) || !aligned16(loss_out) || !aligned16(lse_out) || !aligned16(workspace))
    return fail(BL_ERR_ALIGNMENT, "every pointer must be 16-byte aligned");
  cudaStream_t st = as_stream(stream);
  float2* strips = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + sp.strips);
  float* target_logit = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sp.target_logit);
  int num_strips = 0;
  FewPlan plan;
  if (few_ce_plan(t, k_in, v, &plan)) {
    bl::FewMaps M{};
    if (bl_status s = ce_operand(&M.w[0], w, k_in, v, k_in, false)) return s;
    if (bl_status s = make_map(&M.x, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, x, k_in, t, 64, plan.tok)) return s;
    bl::FewArgs a{};
    a.t = static_cast<int>(t);
    a.k = static_cast<int>(k_in);
    a.n = static_cast<int>(v);
    a.num_k_blocks = static_cast<int>(k_in / 64);
    a.num_row_blocks = static_cast<int>((v + 127) / 128);
    a.x = x;
    a.rows = w;
    a.targets = targets;
    a.strips = strips;
    a.target_logit = target_logit;
    num_strips = a.num_row_blocks * (plan.split > 1 ? plan.split : 4);
    if (bl_status s = plan.tok == 16 ? launch_few<false, 16>(M, a, plan, st) : launch_few<false, 32>(M, a, plan, st)) return s;
  } else {
    bl::CeGroup G{};
    G.count = 1;
    G.v = v;
    G.targets = targets;
    G.strips = strips;
    G.target_logit = target_logit;
    G.x = ce_dots(v) ? reinterpret_cast<const uint4*>(x) : nullptr;
    G.w = reinterpret_cast<const uint4*>(w);
    G.row8 = static_cast<int>(k_in / 8);
    bl::CeProblem& P = G.p[0];
    ce_shape(P, bl::CE_LSE, t, v, k_in, false, false);
    if (bl_status s = ce_operand(&P.tmA, x, k_in, t, k_in, false)) return s;
    if (bl_status s = ce_operand(&P.tmB, w, k_in, v, k_in, false)) return s;
    num_strips = 2 * P.num_n_blocks;
    if (bl_status s = launch_ce(G, st)) return s;
  }
  return launch_head("linear ce join launch", bl::ce_join_kernel, (t + 31) / 32, bl::kCeJoinThreads, st,
                     static_cast<const float2*>(strips), num_strips, t, v, targets, static_cast<const float*>(target_logit),
                     loss_out, lse_out);
}

size_t bitlinear_linear_ce_bwd_workspace_size(int64_t t, int64_t k_in, int64_t v, int want_grad_x) {
  if (t <= 0 || v <= 0 || k_in <= 0) return 0;
  return ce_bwd_space(t, k_in, v, want_grad_x != 0).total;
}

bl_status bitlinear_linear_ce_bwd(const uint16_t* x, const uint16_t* w, const int64_t* targets, const float* lse,
                                  const float* grad_loss, int64_t t, int64_t k_in, int64_t v, uint16_t* grad_x, void* grad_w,
                                  int grad_w_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  g_err[0] = 0;
  if (!grad_x && !grad_w) return fail(BL_ERR_INVALID_ARG, "request grad_x, grad_w or both");
  if (!w) return fail(BL_ERR_INVALID_ARG, "w is required");
  if (grad_w && grad_w_dtype != BL_OUT_BF16 && grad_w_dtype != BL_OUT_F32)
    return fail(BL_ERR_INVALID_ARG, "grad_w_dtype must be BL_OUT_BF16 or BL_OUT_F32");
  if (bl_status s = check_ce(t, k_in, v)) return s;
  if (t != 0 && (!x || !targets || !lse || !grad_loss))
    return fail(BL_ERR_INVALID_ARG, "x, targets, lse, grad_loss are required");
  const void* all[] = {x, w, targets, lse, grad_loss, grad_x, grad_w, workspace};
  for (const void* p : all)
    if (p && !aligned16(p)) return fail(BL_ERR_ALIGNMENT, "every pointer must be 16-byte aligned");
  cudaStream_t st = as_stream(stream);
  const bool w32 = grad_w_dtype == BL_OUT_F32;
  if (t == 0) {
    if (grad_w) {
      cudaError_t e = cudaMemsetAsync(grad_w, 0, static_cast<size_t>(v) * k_in * (w32 ? 4 : 2), st);
      if (e != cudaSuccess) return cuda_fail(e, "grad_w zero");
    }
    return BL_OK;
  }
  const CeBwdSpace sp = ce_bwd_space(t, k_in, v, grad_x != nullptr);
  if (!workspace || workspace_bytes < sp.total)
    return fail(BL_ERR_WORKSPACE, "workspace too small: %zu < %zu", workspace ? workspace_bytes : size_t(0), sp.total);
  uint8_t* space = static_cast<uint8_t*>(workspace);
  int* live = reinterpret_cast<int*>(space + sp.head);
  float* grad_max = reinterpret_cast<float*>(space + sp.head) + 1;
  int* low = live + 2;
  int* place = reinterpret_cast<int*>(space + sp.place);
  int* from = reinterpret_cast<int*>(space + sp.from);
  float* target_dl = reinterpret_cast<float*>(space + sp.target_dl);
  int* row_target = reinterpret_cast<int*>(space + sp.target);
  float* row_lse = reinterpret_cast<float*>(space + sp.lse);
  float* row_grad = reinterpret_cast<float*>(space + sp.grad);
  uint8_t* x_live = space + sp.x;
  float* acc = reinterpret_cast<float*>(space + sp.acc);
  const int64_t rows = round_up(t, 256), dl_rows = ce_dl_rows(t), piece = ce_piece(t, v), pieces = (v + piece - 1) / piece;
  const CeRuns runs = ce_grad_x_runs(t, k_in, piece < v ? piece : v);
  const int row8 = static_cast<int>(k_in / 8);
  const int64_t cap = int64_t(device_sm_count()) * 16;   // blocks of the gather and scatter kernels
  if (bl_status s = launch_head("linear ce live launch", bl::ce_live_kernel, 1, 1024, st, grad_loss, targets, t, v, place, from, live,
                                low, grad_max))
    return s;
  FewPlan plan;
  const bool dots = few_ce_plan(t, k_in, v, &plan) || ce_dots(v);   // as in the forward pass
  const int64_t row_blocks = rows / 8 < cap ? rows / 8 : cap, dot_blocks = !dots ? 0 : (t + 7) / 8 < cap ? (t + 7) / 8 : cap;
  if (bl_status s = launch_head("linear ce gather launch", bl::ce_gather_kernel, row_blocks + dot_blocks, 256, st,
                                reinterpret_cast<const uint4*>(x), reinterpret_cast<const uint4*>(w), targets, lse, grad_loss, t, v,
                                static_cast<int>(row_blocks), static_cast<const int*>(from), static_cast<const int*>(live),
                                static_cast<const int*>(low), static_cast<const float*>(grad_max), row8,
                                reinterpret_cast<uint4*>(x_live), row_target, row_lse, row_grad, target_dl))
    return s;
  bl::CeGroup G{};
  G.v = v;
  G.live = live;
  G.low = low;
  G.row_target = row_target;
  G.row_lse = row_lse;
  G.from = from;
  G.target_dl = dots ? target_dl : nullptr;
  G.row_grad = row_grad;
  G.grad_max = grad_max;
  // launch i: the two products of piece i - 1 and dl of piece i
  for (int64_t i = 0; i <= pieces; ++i) {
    G.count = 0;
    if (i > 0) {
      const int64_t v0 = (i - 1) * piece, n = v - v0 < piece ? v - v0 : piece;
      const uint8_t* dl = space + sp.dl[(i - 1) & 1];
      bl::CeProblem *px = nullptr, *pw = nullptr;
      const bool w_first = t >= 64 * int64_t(runs.blocks);   // the deeper product's tiles go first
      if (grad_w && w_first) pw = &G.p[G.count++];
      if (grad_x) px = &G.p[G.count++];
      if (grad_w && !w_first) pw = &G.p[G.count++];
      if (px) {
        ce_shape(*px, i == 1 ? bl::CE_PART : bl::CE_ADD_PART, dl_rows, k_in, n, false, true);
        px->live_m = 1;
        px->split_blocks = runs.blocks;
        px->splits = (px->num_k_blocks + runs.blocks - 1) / runs.blocks;   // the last piece may have fewer
        if (bl_status s = ce_operand(&px->tmA, dl, n, dl_rows, piece, false)) return s;
        if (bl_status s = ce_operand(&px->tmB, w + v0 * k_in, k_in, n, k_in, true)) return s;
        if (bl_status s = ce_output(&px->tmOut, acc, runs.splits * rows, k_in, k_in, true)) return s;
      }
      if (pw) {
        ce_shape(*pw, w32 ? bl::CE_F32 : bl::CE_BF16, n, k_in, dl_rows, true, true);
        pw->live_k = 1;
        if (bl_status s = ce_operand(&pw->tmA, dl, n, dl_rows, piece, true)) return s;
        if (bl_status s = ce_operand(&pw->tmB, x_live, k_in, rows, k_in, true)) return s;
        if (bl_status s = ce_output(&pw->tmOut, static_cast<uint8_t*>(grad_w) + v0 * k_in * (w32 ? 4 : 2), n, k_in, k_in, w32))
          return s;
      }
    }
    if (i < pieces) {   // dl of the piece [dl_rows, n], row stride `piece`
      const int64_t v0 = i * piece, n = v - v0 < piece ? v - v0 : piece;
      bl::CeProblem& P = G.p[G.count++];
      ce_shape(P, bl::CE_DLOGITS, dl_rows, n, k_in, false, false);
      P.v0 = static_cast<int>(v0);
      P.live_m = 1;
      if (bl_status s = ce_operand(&P.tmA, x_live, k_in, rows, k_in, false)) return s;
      if (bl_status s = ce_operand(&P.tmB, w + v0 * k_in, k_in, n, k_in, false)) return s;
      if (bl_status s = ce_output(&P.tmOut, space + sp.dl[i & 1], dl_rows, n, piece, false)) return s;
    }
    if (bl_status s = launch_ce(G, st)) return s;
  }
  if (grad_x) {
    const int64_t n8 = t * row8, blocks = (n8 + 255) / 256;
    if (bl_status s = launch_head("linear ce scatter launch", bl::ce_scatter_kernel, blocks < cap ? blocks : cap, 256, st,
                                  reinterpret_cast<const float4*>(acc), static_cast<const int*>(place), static_cast<const int*>(low), n8,
                                  row8, runs.splits, rows * k_in / 4, static_cast<const float*>(grad_max), reinterpret_cast<uint4*>(grad_x)))
      return s;
  }
  return BL_OK;
}

}  // extern "C"
