// Block-scaled 8-bit float product on CTA pairs: tcgen05.mma kind::mxf8f6f4.block_scale.
//
//   out[m, n] = sum_k A[m, k] 2^ea(m, k / 128) * B[n, k] 2^eb(n, k / 128)
//
// Both operands are K-major codes with one power-of-two scale per row and 128-wide block
// of K (fp8_quant.cuh; the 128 x 128 blocks of weights repeat their scale over 128 rows).
// The tensor core multiplies each 32-wide slice of K by its two UE8M0 scales, so the
// four MMAs of a 128-byte K step share one scale byte per row and the accumulator in TMEM
// is the finished product in fp32: no rescaling pass over partial sums, which a scale
// that is not a power of two would need after every 128 of K (512 accumulator columns
// read, multiplied and added per 512 MMA cycles). The forward product (tokens x weights),
// the input gradient (dY x W^T's codes) and the weight gradient (dY^T's x X^T's) are all
// this one kernel on different operands.
//
// A cluster of two CTAs computes one tile of 256 rows x kHalves * n_half columns (n_half a
// multiple of 32, at most 224). Why 224 and not the 256 of the other pair kernels: the
// scales live in TMEM beside the accumulators, 2 x 224 + 64 = 512 columns.
//   kHalves = 2 (the wide tile): both accumulators belong to one tile, whose two column
//     halves share every load of A: 44 KB per 128 of K for 896 MMA cycles. With no
//     accumulator to spare, the next tile's first four K blocks run on half 0 alone while
//     the epilogue still drains half 1, then on half 1, so the tensor cores do not wait.
//   kHalves = 1: one accumulator per tile, the other one drained meanwhile; 30 KB per 448
//     MMA cycles. For products with too few wide tiles to fill the SMs evenly, or short K.
// A launch takes up to two products, the two gradients of a backward pass, so that the
// second fills the SMs while the first runs out (ce_shares.cuh): both gradients of 4095 x
// 896 x 4864 took 40.0 us in two launches and take 28.2, of 777 x 1536 x 8960 45.2 and 28.1,
// of 4096 x 11008 x 2048 157 and 140.
// What bounds it: 8192 tokens, 2048 -> 11008 take 133-145 us (2.5-2.8 PFLOP/s), the loads
// alone 84, the MMAs alone 110, and with all-zero operands the whole kernel 126 at full
// clock, while with real ones the card runs into its 1000 W (1432 MHz in a long loop, 168
// us); cuBLAS's 8-bit product of that shape with one scale per tensor: 177 us, 166 in the
// long loop. The int8 pair product, one MMA kind without scales, takes 121.
//
// Scales. A 32-bit word holds a row's bytes of four consecutive K blocks ([K / 512, rows, 4]
// in memory), so one copy serves 16 MMAs per half, which select their byte by the
// instruction descriptor's scale ids. Warps 10 and 11 take turns to gather the words of the
// CTA's 128 rows of A and of the tile's rows of B (both CTAs need all of them) into the order
// that tcgen05.cp.32x128b.warpx4 takes: row r of a 128-row group at 16 (r % 32) + 4 (r / 32).
// One warp's round of waiting for its loads outlasts four K blocks of a narrow tile: with two
// 777 x 8960 -> 1536 takes 18.3 us instead of 22.6 and 4096 x 11008 -> 2048 70.8 instead of
// 74.5; shapes with enough MMAs a block lose 0 to 2%.
// The leader's MMA thread copies them to both CTAs' TMEM in issue order with its MMAs.
//
// Synchronisation as in gemm_tc2.cuh, plus the scale ring:
//   sffull[b] (leader)   : a scale warp of each CTA arrives after filling slot b.
//   sfempty[b] (each CTA): the leader's commit after the copies of slot b (multicast).
// Every wait is bounded. No load uses multicast.
#pragma once

#include "ce_shares.cuh"
#include "pair_issue.cuh"

namespace bl {

constexpr int kF8MaxN = 224;                              // columns of one accumulator
constexpr int kF8ABytes = 128 * 128;                      // one K block (128 bytes) of the CTA's rows
constexpr int kF8BBytes = kF8MaxN / 2 * 128;              // and of its columns of one accumulator
// A stage is one K block: six of 30 KB for narrow tiles, four of 44 KB for wide ones. (With
// two K blocks a stage the refill came too late: the MMAs of two stages do not cover it.)
template <int kHalves>
struct F8Stage {
  static constexpr int kCount = kHalves == 2 ? 4 : 6;
  static constexpr int kBytes = kF8ABytes + kHalves * kF8BBytes;
  static constexpr int kSfGroups = 1 + 2 * kHalves;       // 128-row groups of scales: A, then B by halves
  static constexpr int kSfSlots = kHalves == 2 ? 3 : 4;
};
constexpr int kF8RingBytes = 6 * (kF8ABytes + kF8BBytes);   // 180 KB
constexpr int kF8SfRingBytes = 3 * 5 * 512;
constexpr int kF8EpiWarps = 8;
constexpr int kF8SfWarp = 2 + kF8EpiWarps;
constexpr int kF8SfWarps = 2;
constexpr int kF8Threads = 32 * (kF8SfWarp + kF8SfWarps);   // 384
constexpr int kF8StgBytes = 32 * 128;                     // per epilogue warp: 32 rows x 32 columns fp32, or two of bf16
constexpr uint32_t kF8SfCol0 = 2 * kF8MaxN;               // TMEM: scales after the accumulators
constexpr int kF8BarBytes = 512;
static_assert(kF8ABytes % 1024 == 0 && kF8BBytes % 1024 == 0, "128B-swizzle atoms need 1 KB alignment");
static_assert(F8Stage<1>::kCount * F8Stage<1>::kBytes <= kF8RingBytes && F8Stage<2>::kCount * F8Stage<2>::kBytes <= kF8RingBytes,
              "stages");
static_assert(F8Stage<1>::kSfSlots * F8Stage<1>::kSfGroups * 512 <= kF8SfRingBytes &&
                  F8Stage<2>::kSfSlots * F8Stage<2>::kSfGroups * 512 <= kF8SfRingBytes,
              "scale slots");
static_assert(kF8SfCol0 + 4 * F8Stage<1>::kSfSlots * F8Stage<1>::kSfGroups <= 512 &&
                  kF8SfCol0 + 4 * F8Stage<2>::kSfSlots * F8Stage<2>::kSfGroups <= 512,
              "accumulators and scales exceed the TMEM of a CTA");
constexpr size_t gemm_fp8_smem_bytes() {
  return 1024 + static_cast<size_t>(kF8RingBytes) + kF8EpiWarps * kF8StgBytes + kF8SfRingBytes + kF8BarBytes;
}
static_assert(gemm_fp8_smem_bytes() <= 232448, "fp8 GEMM exceeds the shared memory of a CTA");

struct Fp8Problem {
  CUtensorMap tmA, tmB, tmOut;
  const uint32_t* sa;   // [ceil(K / 512), M] words of A's scale bytes
  const uint32_t* sb;   // [ceil(K / 512), N]
  int M, N;
  int n_half;           // columns of one accumulator: multiple of 32, <= kF8MaxN
  int num_k_blocks;     // ceil(K / 128)
  int num_m_blocks, num_n_blocks;   // 256-row blocks and tiles of kHalves * n_half columns
  int m_fastest;
  int a_e5m2, b_e5m2;
  int out_f32;
};
// The products of one launch, the tiles of each shared out by ce_shares.cuh.
constexpr int kMaxFp8Group = 2;
struct Fp8Group {
  Fp8Problem p[kMaxFp8Group];
  CeShares share[kMaxFp8Group];
  int count;
};

// Instruction descriptor of a block-scaled MMA (kind::mxf8f6f4): b scale id [4,6),
// a format [7,10), b format [10,13) (0 e4m3, 1 e5m2), N >> 3 [17,23), scale type bit 23
// (1 = UE8M0), M >> 4 [24,29), a scale id [29,31). Both operands K-major.
__device__ __forceinline__ uint32_t make_idesc_mxf8(uint32_t a_fmt, uint32_t b_fmt, uint32_t n, uint32_t m, uint32_t sf_id) {
  return (sf_id << 4) | (a_fmt << 7) | (b_fmt << 10) | ((n >> 3) << 17) | (1u << 23) | ((m >> 4) << 24) | (sf_id << 29);
}
__device__ __forceinline__ void tc_mma_mxf8_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                                 uint32_t sfa, uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
      : "memory");
}
// 32 rows x 16 B of shared memory into 4 TMEM columns, repeated over the four lane
// quarters, in each CTA of the pair from its own shared memory.
__device__ __forceinline__ void tc_cp_32x128b_pair(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
__device__ __forceinline__ uint64_t make_sf_desc(uint32_t saddr) {   // 8-row core matrices of 128 B, no swizzle
  return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | static_cast<uint64_t>(1) << 16 |
         static_cast<uint64_t>(128 >> 4) << 32 | static_cast<uint64_t>(1) << 46;
}
__device__ __forceinline__ void fp8_tile_coords(const Fp8Problem& g, int tile, int& mb, int& nb) {
  if (g.m_fastest) {
    mb = tile % g.num_m_blocks;
    nb = tile / g.num_m_blocks;
  } else {
    mb = tile / g.num_n_blocks;
    nb = tile % g.num_n_blocks;
  }
}

template <int kHalves>
__global__ void __launch_bounds__(kF8Threads, 1) gemm_fp8_kernel(const __grid_constant__ Fp8Group G) {
  using S = F8Stage<kHalves>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  // stage s: the CTA's rows of A, then its columns of B for each half
  auto st_a = [&](int s) { return base + static_cast<uint32_t>(s * S::kBytes); };
  auto st_b = [&](int s, int half) { return st_a(s) + static_cast<uint32_t>(kF8ABytes + half * kF8BBytes); };
  constexpr int kOutOff = kF8RingBytes;
  constexpr int kSfOff = kOutOff + kF8EpiWarps * kF8StgBytes;
  const uint32_t sOut = base + kOutOff, sSf = base + kSfOff;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kSfOff + kF8SfRingBytes);
  const uint32_t bar0 = smem_u32(bars);
  // full[S] | empty[S] | sffull[F] | sfempty[F] | tfull[2] | tempty[2] | done
  const uint32_t full0 = bar0, empty0 = full0 + 8u * S::kCount;
  const uint32_t sffull0 = empty0 + 8u * S::kCount, sfempty0 = sffull0 + 8u * S::kSfSlots;
  const uint32_t tfull0 = sfempty0 + 8u * S::kSfSlots, tempty0 = tfull0 + 16u, done_bar = tempty0 + 16u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * S::kCount + 2 * S::kSfSlots + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // warp-uniform
  if (threadIdx.x == 0) {
    for (int s = 0; s < S::kCount; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int s = 0; s < S::kSfSlots; ++s) {
      mbar_init(sffull0 + 8u * s, 2);    // a scale warp of each CTA
      mbar_init(sfempty0 + 8u * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8u * b, 1);
      mbar_init(tempty0 + 8u * b, 2 * kF8EpiWarps);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int j = 0; j < G.count; ++j) {
      tma_prefetch_desc(&G.p[j].tmA);
      tma_prefetch_desc(&G.p[j].tmB);
      tma_prefetch_desc(&G.p[j].tmOut);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_sync();   // barriers of both CTAs initialised, TMEM allocated in both
  tc_fence_after_sync();
  follow_stream();
  const uint32_t tmem_base = __reduce_or_sync(0xffffffffu, *tmem_slot);   // the same in every lane: a uniform register
  const uint32_t peer_abort = map_to_rank(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u);
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------- TMA producer (both CTAs)
    const uint32_t full_leader0 = __reduce_or_sync(0xffffffffu, map_to_rank(full0, 0));
    uint32_t live = 1;   // 0 after a wait gave up: the loops run out without issuing or waiting
    int s = 0;
    uint32_t ph = 0;
    uint32_t issued = 0;
    for (int j = 0; j < G.count; ++j) {
      const Fp8Problem& P = G.p[j];
      const int rounds = G.share[j].count[cluster], pos = G.share[j].pos[cluster];
      const int my_n = P.n_half >> 1;   // columns of each half that this CTA loads
      const uint32_t stage_bytes = 2u * static_cast<uint32_t>(kF8ABytes + kHalves * my_n * 128);   // of both CTAs
      for (int r = 0; r < rounds; ++r) {
        int mb, nb;
        fp8_tile_coords(P, ce_round_tile(G.share[j], nclusters, pos, r), mb, nb);
        const int m0 = mb * 256 + 128 * static_cast<int>(rank);
        const int n0 = nb * kHalves * P.n_half + my_n * static_cast<int>(rank);
        for (int kb = 0; kb < P.num_k_blocks; ++kb) {
          live = wait_live<false>(live, empty0 + 8u * s, ph ^ 1u, abort_flag, peer_abort);
          const uint32_t fb = full_leader0 + 8u * s;
          if (elect_one() && live) {
            if (leader) mbar_arrive_expect_tx(full0 + 8u * s, stage_bytes);
            tma_load_2d_pair(st_a(s), &P.tmA, fb, kb * 128, m0);
#pragma unroll
            for (int half = 0; half < kHalves; ++half)
              tma_load_2d_pair(st_b(s, half), &P.tmB, fb, kb * 128, n0 + half * P.n_half);
          }
          issued += live;
          if (++s == S::kCount) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
    }
    if (!live && elect_one()) {
      atomicOr(&g_device_status, DEV_ST_TIMEOUT_PRODUCER);
      // the leader's full barriers count both CTAs' copies: drain the last ring of them
      if (leader) {
        const uint32_t first = issued > S::kCount ? issued - S::kCount : 0;
        for (uint32_t i = first; i < issued; ++i)
          if (!mbar_wait_plain(full0 + 8u * (i % S::kCount), (i / S::kCount) & 1u)) atomicOr(&g_device_status, DEV_ST_TIMEOUT_DRAIN);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer (leader only)
    if (leader) {
      uint32_t idesc0 = 0;       // of the current product
      bool wide = false;
      uint32_t live = 1;         // 0 after a wait gave up: the loops run out without issuing or waiting
      int s = 0, f = 0;          // next stage and scale slot
      uint32_t ph = 0, fph = 0;
      uint32_t col = 0;          // TMEM column of the current scales
      // scales of the next four K blocks to TMEM
      auto scales = [&]() {
        live = wait_live<true>(live, sffull0 + 8u * f, fph, abort_flag, peer_abort);
        tc_fence_after_sync();
        col = tmem_base + kF8SfCol0 + static_cast<uint32_t>(4 * S::kSfGroups * f);
        const uint32_t src = sSf + static_cast<uint32_t>(f * S::kSfGroups * 512);
        if (elect_one() && live) {
          tc_cp_32x128b_pair(col, make_sf_desc(src));
#pragma unroll
          for (int half = 0; half < kHalves; ++half) {
            tc_cp_32x128b_pair(col + 4u + 8u * half, make_sf_desc(src + 512u + 1024u * half));
            if (wide) tc_cp_32x128b_pair(col + 8u + 8u * half, make_sf_desc(src + 1024u + 1024u * half));
          }
          tc_commit_pair(sfempty0 + 8u * f);
        }
        if (++f == S::kSfSlots) {
          f = 0;
          fph ^= 1u;
        }
      };
      // four MMAs of K block kb, in stage st, on accumulator buf (one lane)
      auto block = [&](int st, int half, int buf, int kb) {
        const uint64_t ad = make_sw128_desc(st_a(st), 16, 1024), bd = make_sw128_desc(st_b(st, half), 16, 1024);
        const uint32_t id = static_cast<uint32_t>(kb & 3);
        const uint32_t idesc = idesc0 | id << 4 | id << 29;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)   // 32 bytes of K further inside the swizzled row: 2 in the address field
          tc_mma_mxf8_pair(tmem_base + static_cast<uint32_t>(buf * kF8MaxN), ad + 2u * kk, bd + 2u * kk, idesc, col,
                           col + 4u + 8u * half, (kb | kk) != 0 ? 1u : 0u);
      };
      auto next_stage = [&]() {
        if (++s == S::kCount) {
          s = 0;
          ph ^= 1u;
        }
      };
      uint32_t tph = 1;   // phase of the accumulators' buffers
      int local = 0;
      for (int j = 0; j < G.count; ++j) {
        const int rounds = G.share[j].count[cluster], num_k_blocks = G.p[j].num_k_blocks;
        idesc0 = __reduce_or_sync(0xffffffffu, make_idesc_mxf8(G.p[j].a_e5m2, G.p[j].b_e5m2, G.p[j].n_half, 256, 0));
        wide = G.p[j].n_half > 128;
        for (int r = 0; r < rounds; ++r, ++local) {
          if constexpr (kHalves == 1) {
            const int buf = local & 1;
            live = wait_live<false>(live, tempty0 + 8u * buf, tph, abort_flag, peer_abort);
            tc_fence_after_sync();
            for (int kb = 0; kb < num_k_blocks; ++kb) {
              if ((kb & 3) == 0) scales();
              live = wait_live<false>(live, full0 + 8u * s, ph, abort_flag, peer_abort);
              tc_fence_after_sync();
              if (elect_one() && live) {
                block(s, 0, buf, kb);
                tc_commit_pair(empty0 + 8u * s);
                if (kb + 1 == num_k_blocks) tc_commit_pair(tfull0 + 8u * buf);
              }
              next_stage();
            }
            tph ^= static_cast<uint32_t>(buf);
          } else {
            // the first K blocks (at most a ring of them, one scale group) on half 0, then on half 1
            const int lead = min(S::kCount, num_k_blocks);
            live = wait_live<false>(live, tempty0, tph, abort_flag, peer_abort);
            scales();
            int st = s;
            uint32_t sph = ph;
            for (int kb = 0; kb < lead; ++kb) {
              live = wait_live<false>(live, full0 + 8u * st, sph, abort_flag, peer_abort);
              tc_fence_after_sync();
              if (elect_one() && live) {
                block(st, 0, 0, kb);
                if (kb == num_k_blocks - 1) tc_commit_pair(tfull0);
              }
              if (++st == S::kCount) {
                st = 0;
                sph ^= 1u;
              }
            }
            live = wait_live<false>(live, tempty0 + 8u, tph, abort_flag, peer_abort);
            tc_fence_after_sync();
            for (int kb = 0; kb < lead; ++kb) {
              if (elect_one() && live) {
                block(s, 1, 1, kb);
                tc_commit_pair(empty0 + 8u * s);
                if (kb == num_k_blocks - 1) tc_commit_pair(tfull0 + 8u);
              }
              next_stage();
            }
            for (int kb = lead; kb < num_k_blocks; ++kb) {
              if ((kb & 3) == 0) scales();
              live = wait_live<false>(live, full0 + 8u * s, ph, abort_flag, peer_abort);
              tc_fence_after_sync();
              if (elect_one() && live) {
                const bool end = kb == num_k_blocks - 1;
                block(s, 0, 0, kb);
                if (end) tc_commit_pair(tfull0);
                block(s, 1, 1, kb);
                tc_commit_pair(empty0 + 8u * s);
                if (end) tc_commit_pair(tfull0 + 8u);
              }
              next_stage();
            }
            tph ^= 1u;
          }
        }
      }
      if (elect_one()) {
        if (!live) atomicOr(&g_device_status, DEV_ST_TIMEOUT_MMA);
        tc_commit_pair_local(done_bar);
        if (!mbar_wait_plain(done_bar, 0)) atomicOr(&g_device_status, DEV_ST_TIMEOUT_DRAIN);
      }
    }
  } else if (warp >= kF8SfWarp) {
    // ------------------------------------------------------------- scale warps (both CTAs)
    const uint32_t sffull_leader0 = map_to_rank(sffull0, 0);
    int f = warp - kF8SfWarp;   // every kF8SfWarps-th scale slot and group of K blocks
    uint32_t fph = 0;
    bool ok = true;
    uint32_t w[4 * S::kSfGroups];
    // The next words' place: coordinates are worked out once a tile. (Worked out for every
    // four K blocks they delayed the scales: 2048 x 11008 -> 2048 took 40.4 us instead of 34.5.)
    const uint32_t *pa = nullptr, *pb = nullptr;
    int M = 0, N = 0, n_half = 0, m0 = 0, n0 = 0;
    int j = 0, r = 0, left = 0;   // product, round, and what the tile has left of four K blocks each
    auto aim = [&]() {            // at the pair's next tile; none: left stays 0
      while (j < G.count && r == G.share[j].count[cluster]) {
        ++j;
        r = 0;
      }
      if (j == G.count) return;
      const Fp8Problem& P = G.p[j];
      int mb, nb;
      fp8_tile_coords(P, ce_round_tile(G.share[j], nclusters, G.share[j].pos[cluster], r), mb, nb);
      m0 = mb * 256 + 128 * static_cast<int>(rank) + lane;
      n0 = nb * kHalves * P.n_half + lane;
      M = P.M;
      N = P.N;
      n_half = P.n_half;
      pa = P.sa + m0;
      pb = P.sb + n0;
      left = (P.num_k_blocks + 3) >> 2;
    };
    auto load = [&]() {   // rows past the operands' ends (zero codes) get scale byte 0
#pragma unroll
      for (int c = 0; c < 4; ++c) w[c] = m0 + 32 * c < M ? ld_plain(pa + 32 * c) : 0u;
#pragma unroll
      for (int c = 0; c < 8 * kHalves; ++c) {
        const int in_half = 32 * (c & 7), at = (c >> 3) * n_half + in_half;
        w[4 + c] = in_half < n_half && n0 + at < N ? ld_plain(pb + at) : 0u;
      }
    };
    auto next = [&](int groups) {   // that many times four K blocks further
      for (; left && groups > 0; --groups) {
        pa += M;
        pb += N;
        if (--left == 0) {
          ++r;
          aim();
        }
      }
    };
    aim();
    next(f);
    if (left) load();
    while (left) {
      const bool got = mbar_wait(sfempty0 + 8u * f, fph ^ 1u, abort_flag);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      const uint32_t dst = sSf + static_cast<uint32_t>(f * S::kSfGroups * 512 + lane * 16);
#pragma unroll
      for (int i = 0; i < S::kSfGroups; ++i)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 512u * i), "r"(w[4 * i]), "r"(w[4 * i + 1]),
                     "r"(w[4 * i + 2]), "r"(w[4 * i + 3])
                     : "memory");
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(sffull_leader0 + 8u * f);
      // after the fence, which would wait for them: the next group's words travel while
      // this warp waits for a free slot
      next(kF8SfWarps);
      if (left) load();
      f += kF8SfWarps;
      if (f >= S::kSfSlots) {
        f -= S::kSfSlots;
        fph ^= 1u;
      }
    }
    if (!ok && lane == 0) {
      pair_abort(abort_flag, peer_abort);
      atomicOr(&g_device_status, DEV_ST_TIMEOUT_PRODUCER);
    }
  } else {
    // ------------------------------------------------------------- epilogue (8 warps, both CTAs)
    // two warps per TMEM lane quarter, each half of an accumulator's 32-column pieces:
    // TMEM -> registers -> staging (swizzled by the store's tensor map) -> TMA store
    const int e = warp - 2;
    const int quad = warp & 3;
    const uint32_t stg0 = sOut + static_cast<uint32_t>(e * kF8StgBytes);
    const uint32_t tempty_leader0 = map_to_rank(tempty0, 0);
    int cnt = 0;
    int unit = 0;   // accumulators so far: unit u is in buffer u & 1
    bool ok = true;
    for (int j = 0; j < G.count && ok; ++j) {
      const Fp8Problem& P = G.p[j];
      const int rounds = G.share[j].count[cluster], pos = G.share[j].pos[cluster];
      const int pieces = P.n_half >> 5;
      const int first = (e >> 2) ? (pieces + 1) >> 1 : 0, last = (e >> 2) ? pieces : (pieces + 1) >> 1;
      if (lane == 0) bulk_wait_group_read<0>();   // the staging buffer's use depends on the output type
      __syncwarp();
      for (int r = 0; r < rounds && ok; ++r) {
        int mb, nb;
        fp8_tile_coords(P, ce_round_tile(G.share[j], nclusters, pos, r), mb, nb);
        const int row0 = mb * 256 + 128 * static_cast<int>(rank) + quad * 32;
#pragma unroll 1
        for (int half = 0; half < kHalves; ++half, ++unit) {
          const int buf = unit & 1;
          const int n0 = (nb * kHalves + half) * P.n_half;
          const bool got = mbar_wait(tfull0 + 8u * buf, static_cast<uint32_t>(unit >> 1) & 1u, abort_flag);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          // all of the warp's columns to registers at once, so that the accumulator is free
          // again after one TMEM latency, not after the conversion and the stores
          const uint32_t t_row = tmem_base + static_cast<uint32_t>(buf * kF8MaxN + first * 32) + (static_cast<uint32_t>(quad * 32) << 16);
          uint32_t v[4][32];
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (first + i < last) tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(i * 32), v[i]);
          tmem_ld_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(tempty_leader0 + 8u * buf);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (first + i >= last) break;
            const int col = n0 + (first + i) * 32;
            if (lane == 0) {   // the buffer's previous store has finished reading it
              if (P.out_f32) bulk_wait_group_read<0>();
              else bulk_wait_group_read<1>();
            }
            __syncwarp();
            const uint32_t stg = P.out_f32 ? stg0 : stg0 + static_cast<uint32_t>((cnt++ & 1) * 2048);
            if (P.out_f32) {   // 128-byte rows, 128B swizzle: chunk j at j ^ (row & 7)
              const uint32_t row_addr = stg + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
              for (int j = 0; j < 8; ++j)
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row_addr + static_cast<uint32_t>((j ^ (lane & 7)) * 16)),
                             "r"(v[i][4 * j]), "r"(v[i][4 * j + 1]), "r"(v[i][4 * j + 2]), "r"(v[i][4 * j + 3])
                             : "memory");
            } else {           // 64-byte rows, 64B swizzle: chunk j at j ^ ((row >> 1) & 3)
              const uint32_t row_addr = stg + static_cast<uint32_t>(lane) * 64u;
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                  w[q] = pack_bf16x2(__uint_as_float(v[i][8 * j + 2 * q]), __uint_as_float(v[i][8 * j + 2 * q + 1]));
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row_addr + static_cast<uint32_t>((j ^ ((lane >> 1) & 3)) * 16)),
                             "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                             : "memory");
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              if (col < P.N) tma_store_2d(&P.tmOut, stg, col, row0);
              bulk_commit_group();
            }
          }
        }
      }
    }
    if (!ok && lane == 0) {
      pair_abort(abort_flag, peer_abort);
      atomicOr(&g_device_status, DEV_ST_TIMEOUT_EPILOGUE);
    }
    if (lane == 0) bulk_wait_group_all();
  }

  __syncthreads();
  tc_fence_before_sync();
  cluster_sync();   // the peer no longer reads this CTA's shared memory or barriers
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

}  // namespace bl
