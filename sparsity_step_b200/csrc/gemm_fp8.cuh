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
// A cluster of two CTAs computes one 256 x n_tile tile (n_tile a multiple of 32, at most
// 224): CTA r loads 128 rows of A and n_tile / 2 rows of B per 128-byte K step, six stages.
// Why 224 and not the 256 of the other pair kernels: the scales live in TMEM beside the
// two accumulators, 2 x 224 + 64 = 512 columns.
//
// Scales. A 32-bit word holds a row's bytes of four consecutive K blocks ([K / 512, rows, 4]
// in memory), so one copy serves 16 MMAs, which select their byte by the instruction
// descriptor's scale ids. Warp 10 gathers the words of the CTA's 128 rows of A and of the
// tile's n_tile rows of B (both CTAs need all of them) into the order that
// tcgen05.cp.32x128b.warpx4 takes: row r of a 128-row group at 16 (r % 32) + 4 (r / 32).
// The leader's MMA thread copies them to both CTAs' TMEM in issue order with its MMAs.
//
// Synchronisation as in gemm_tc2.cuh, plus the scale ring:
//   sffull[b] (leader)   : the scale warps of both CTAs arrive after filling slot b.
//   sfempty[b] (each CTA): the leader's commit after the copies of slot b (multicast).
// Every wait is bounded. No load uses multicast.
#pragma once

#include "gemm_tc2.cuh"

namespace bl {

constexpr int kF8MaxN = 224;
constexpr int kF8Stages = 6;
constexpr int kF8ABytes = 128 * 128;
constexpr int kF8BBytes = kF8MaxN / 2 * 128;
constexpr int kF8StageBytes = kF8ABytes + kF8BBytes;      // 30 KB
constexpr int kF8SfSlots = 4;
constexpr int kF8SfBytes = 3 * 512;                       // A: 128 rows; B: 2 x 128 rows
constexpr int kF8EpiWarps = 8;
constexpr int kF8SfWarp = 2 + kF8EpiWarps;
constexpr int kF8Threads = 32 * (kF8SfWarp + 1);          // 352
constexpr int kF8StgBytes = 32 * 128;                     // per epilogue warp: 32 rows x 32 columns (<= 4 B)
constexpr uint32_t kF8SfCol0 = 2 * kF8MaxN;               // TMEM: scales after the accumulators
constexpr int kF8BarBytes = 512;
static_assert(kF8StageBytes % 1024 == 0 && kF8ABytes % 1024 == 0, "128B-swizzle atoms need 1 KB alignment");
static_assert(kF8SfCol0 + 16 * kF8SfSlots <= 512, "accumulators and scales exceed the TMEM of a CTA");
constexpr size_t gemm_fp8_smem_bytes() {
  return 1024 + static_cast<size_t>(kF8Stages) * kF8StageBytes + kF8EpiWarps * kF8StgBytes + kF8SfSlots * kF8SfBytes +
         kF8BarBytes;
}
static_assert(gemm_fp8_smem_bytes() <= 232448, "fp8 GEMM exceeds the shared memory of a CTA");

struct Fp8GemmArgs {
  const uint32_t* sa;   // [ceil(K / 512), M] words of A's scale bytes
  const uint32_t* sb;   // [ceil(K / 512), N]
  int M, N;
  int n_tile;           // multiple of 32, <= kF8MaxN
  int num_k_blocks;     // ceil(K / 128)
  int num_m_blocks, num_n_blocks;   // 256-row and n_tile-column blocks
  int m_fastest;
  int a_e5m2, b_e5m2;
  int out_f32;
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
// As mbar_wait, for a barrier that the other CTA's threads arrive on too after writing
// what they hand over: acquires at cluster scope.
__device__ __forceinline__ bool mbar_wait_cluster(uint32_t bar, uint32_t parity, const volatile int* abort) {
  const uint64_t t0 = global_timer_ns();
  for (;;) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
    if (*abort || global_timer_ns() - t0 > kWaitTimeoutNs) return false;
  }
}

__device__ __forceinline__ void fp8_tile_coords(const Fp8GemmArgs& g, int tile, int& mb, int& nb) {
  if (g.m_fastest) {
    mb = tile % g.num_m_blocks;
    nb = tile / g.num_m_blocks;
  } else {
    mb = tile / g.num_n_blocks;
    nb = tile % g.num_n_blocks;
  }
}

__global__ void __launch_bounds__(kF8Threads, 1)
    gemm_fp8_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                    const __grid_constant__ CUtensorMap tmOut, const Fp8GemmArgs g) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  auto st_a = [&](int s) { return base + static_cast<uint32_t>(s * kF8StageBytes); };
  auto st_b = [&](int s) { return base + static_cast<uint32_t>(s * kF8StageBytes + kF8ABytes); };
  constexpr int kOutOff = kF8Stages * kF8StageBytes;
  constexpr int kSfOff = kOutOff + kF8EpiWarps * kF8StgBytes;
  const uint32_t sOut = base + kOutOff, sSf = base + kSfOff;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kSfOff + kF8SfSlots * kF8SfBytes);
  const uint32_t bar0 = smem_u32(bars);
  // full[S] | empty[S] | sffull[F] | sfempty[F] | tfull[2] | tempty[2] | done
  const uint32_t full0 = bar0, empty0 = full0 + 8u * kF8Stages;
  const uint32_t sffull0 = empty0 + 8u * kF8Stages, sfempty0 = sffull0 + 8u * kF8SfSlots;
  const uint32_t tfull0 = sfempty0 + 8u * kF8SfSlots, tempty0 = tfull0 + 16u, done_bar = tempty0 + 16u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kF8Stages + 2 * kF8SfSlots + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kF8Stages; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int s = 0; s < kF8SfSlots; ++s) {
      mbar_init(sffull0 + 8u * s, 2);    // the scale warps of both CTAs
      mbar_init(sfempty0 + 8u * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8u * b, 1);
      mbar_init(tempty0 + 8u * b, 2 * kF8EpiWarps);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    tma_prefetch_desc(&tmOut);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), 512);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_sync();   // barriers of both CTAs initialised, TMEM allocated in both
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t peer_abort = map_to_rank(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u);
  const int num_tiles = g.num_m_blocks * g.num_n_blocks;
  const int num_k_groups = (g.num_k_blocks + 3) >> 2;
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------- TMA producer (both CTAs)
    if (lane == 0) {
      const uint32_t full_leader0 = map_to_rank(full0, 0);
      const int half_n = g.n_tile >> 1;
      const uint32_t pair_bytes = 2u * static_cast<uint32_t>(kF8ABytes + half_n * 128);
      int s = 0;
      uint32_t ph = 0;
      long long issued = 0;
      bool ok = true;
      for (int tile = cluster; tile < num_tiles && ok; tile += nclusters) {
        int mb, nb;
        fp8_tile_coords(g, tile, mb, nb);
        const int m0 = mb * 256 + 128 * static_cast<int>(rank);
        const int n0 = nb * g.n_tile + half_n * static_cast<int>(rank);
        for (int kb = 0; kb < g.num_k_blocks; ++kb) {
          if (!mbar_wait(empty0 + 8u * s, ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t fb = full_leader0 + 8u * s;
          if (leader) mbar_arrive_expect_tx(full0 + 8u * s, pair_bytes);
          tma_load_2d_pair(st_a(s), &tmA, fb, kb * 128, m0);
          tma_load_2d_pair(st_b(s), &tmB, fb, kb * 128, n0);
          ++issued;
          if (++s == kF8Stages) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) {
        pair_abort(abort_flag, peer_abort);
        atomicOr(&g_device_status, DEV_ST_TIMEOUT_PRODUCER);
        if (leader) {   // the leader's full barriers count both CTAs' copies: drain them
          const long long first = issued > kF8Stages ? issued - kF8Stages : 0;
          for (long long i = first; i < issued; ++i)
            if (!mbar_wait_plain(full0 + 8u * static_cast<uint32_t>(i % kF8Stages), static_cast<uint32_t>((i / kF8Stages) & 1)))
              atomicOr(&g_device_status, DEV_ST_TIMEOUT_DRAIN);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer (leader only)
    if (lane == 0 && leader) {
      const uint32_t idesc0 = make_idesc_mxf8(g.a_e5m2, g.b_e5m2, g.n_tile, 256, 0);
      int s = 0, f = 0;
      uint32_t ph = 0, fph = 0;
      int local = 0;
      bool ok = true;
      for (int tile = cluster; tile < num_tiles && ok; tile += nclusters, ++local) {
        const int buf = local & 1;
        const uint32_t tph = static_cast<uint32_t>(local >> 1) & 1u;
        if (!mbar_wait(tempty0 + 8u * buf, tph ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * kF8MaxN);
        uint32_t sfa = 0;
        for (int kb = 0; kb < g.num_k_blocks; ++kb) {
          if ((kb & 3) == 0) {   // the scales of the next four K blocks
            if (!mbar_wait_cluster(sffull0 + 8u * f, fph, abort_flag)) {
              ok = false;
              break;
            }
            tc_fence_after_sync();
            sfa = tmem_base + kF8SfCol0 + 16u * static_cast<uint32_t>(f);
            const uint32_t src = sSf + static_cast<uint32_t>(f * kF8SfBytes);
            tc_cp_32x128b_pair(sfa, make_sf_desc(src));
            tc_cp_32x128b_pair(sfa + 4u, make_sf_desc(src + 512u));
            if (g.n_tile > 128) tc_cp_32x128b_pair(sfa + 8u, make_sf_desc(src + 1024u));
            tc_commit_pair(sfempty0 + 8u * f);
            if (++f == kF8SfSlots) {
              f = 0;
              fph ^= 1u;
            }
          }
          if (!mbar_wait(full0 + 8u * s, ph, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a_base = st_a(s), b_base = st_b(s);
          const uint32_t id = static_cast<uint32_t>(kb & 3);
          const uint32_t idesc = idesc0 | id << 4 | id << 29;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_mxf8_pair(d_tmem, make_sw128_desc(a_base + kk * 32, 16, 1024), make_sw128_desc(b_base + kk * 32, 16, 1024),
                             idesc, sfa, sfa + 4u, (kb | kk) != 0 ? 1u : 0u);
          tc_commit_pair(empty0 + 8u * s);
          if (++s == kF8Stages) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit_pair(tfull0 + 8u * buf);
      }
      if (!ok) {
        pair_abort(abort_flag, peer_abort);
        atomicOr(&g_device_status, DEV_ST_TIMEOUT_MMA);
      }
      tc_commit_pair_local(done_bar);
      if (!mbar_wait_plain(done_bar, 0)) atomicOr(&g_device_status, DEV_ST_TIMEOUT_DRAIN);
    }
  } else if (warp == kF8SfWarp) {
    // ------------------------------------------------------------- scale warp (both CTAs)
    const uint32_t sffull_leader0 = map_to_rank(sffull0, 0);
    int f = 0;
    uint32_t fph = 0;
    bool ok = true;
    for (int tile = cluster; tile < num_tiles && ok; tile += nclusters) {
      int mb, nb;
      fp8_tile_coords(g, tile, mb, nb);
      const int m0 = mb * 256 + 128 * static_cast<int>(rank), n0 = nb * g.n_tile;
      for (int kg = 0; kg < num_k_groups; ++kg) {
        const uint32_t* pa = g.sa + static_cast<int64_t>(kg) * g.M;
        const uint32_t* pb = g.sb + static_cast<int64_t>(kg) * g.N;
        uint32_t w[12];
#pragma unroll
        for (int c = 0; c < 12; ++c) {   // rows past the operands' ends (zero codes) get scale byte 0
          const int r = c < 4 ? m0 + 32 * c + lane : n0 + 32 * (c - 4) + lane;
          w[c] = 0;
          if (c < 4 ? r < g.M : (r < g.N && 32 * (c - 4) < g.n_tile)) w[c] = __ldg(c < 4 ? pa + r : pb + r);
        }
        const bool got = mbar_wait(sfempty0 + 8u * f, fph ^ 1u, abort_flag);
        if (!__all_sync(0xffffffffu, got)) {
          ok = false;
          break;
        }
        const uint32_t dst = sSf + static_cast<uint32_t>(f * kF8SfBytes + lane * 16);
#pragma unroll
        for (int j = 0; j < 3; ++j)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + 512u * j), "r"(w[4 * j]), "r"(w[4 * j + 1]),
                       "r"(w[4 * j + 2]), "r"(w[4 * j + 3])
                       : "memory");
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(sffull_leader0 + 8u * f);
        if (++f == kF8SfSlots) {
          f = 0;
          fph ^= 1u;
        }
      }
    }
    if (!ok && lane == 0) {
      pair_abort(abort_flag, peer_abort);
      atomicOr(&g_device_status, DEV_ST_TIMEOUT_PRODUCER);
    }
  } else {
    // ------------------------------------------------------------- epilogue (8 warps, both CTAs)
    // two warps per TMEM lane quarter, each half of the tile's 32-column pieces: TMEM ->
    // registers -> staging (swizzled by the store's tensor map) -> TMA store
    const int e = warp - 2;
    const int quad = warp & 3;
    const int pieces = g.n_tile >> 5;
    const int first = (e >> 2) ? (pieces + 1) >> 1 : 0, last = (e >> 2) ? pieces : (pieces + 1) >> 1;
    const uint32_t stg = sOut + static_cast<uint32_t>(e * kF8StgBytes);
    const uint32_t tempty_leader0 = map_to_rank(tempty0, 0);
    int cnt = 0;
    int local = 0;
    bool ok = true;
    for (int tile = cluster; tile < num_tiles; tile += nclusters, ++local) {
      const int buf = local & 1;
      const uint32_t tph = static_cast<uint32_t>(local >> 1) & 1u;
      int mb, nb;
      fp8_tile_coords(g, tile, mb, nb);
      const int row0 = mb * 256 + 128 * static_cast<int>(rank) + quad * 32, n0 = nb * g.n_tile;
      const bool got = mbar_wait(tfull0 + 8u * buf, tph, abort_flag);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t t_row = tmem_base + static_cast<uint32_t>(buf * kF8MaxN) + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll 1
      for (int c = first; c < last; ++c, ++cnt) {
        uint32_t r[32];
        tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(c * 32), r);
        if (cnt >= 1) {
          if (lane == 0) bulk_wait_group_read<0>();   // the previous store has finished reading the buffer
          __syncwarp();
        }
        tmem_ld_wait();
        if (g.out_f32) {   // 128-byte rows, 128B swizzle: chunk j at j ^ (row & 7)
          const uint32_t row_addr = stg + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
          for (int j = 0; j < 8; ++j)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row_addr + static_cast<uint32_t>((j ^ (lane & 7)) * 16)),
                         "r"(r[4 * j]), "r"(r[4 * j + 1]), "r"(r[4 * j + 2]), "r"(r[4 * j + 3])
                         : "memory");
        } else {           // 64-byte rows, 64B swizzle: chunk j at j ^ ((row >> 1) & 3)
          const uint32_t row_addr = stg + static_cast<uint32_t>(lane) * 64u;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              w[i] = pack_bf16x2(__uint_as_float(r[8 * j + 2 * i]), __uint_as_float(r[8 * j + 2 * i + 1]));
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(row_addr + static_cast<uint32_t>((j ^ ((lane >> 1) & 3)) * 16)),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          tma_store_2d(&tmOut, stg, n0 + c * 32, row0);
          bulk_commit_group();
        }
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(tempty_leader0 + 8u * buf);
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
