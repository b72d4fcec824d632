// Softmax cross entropy of a linear head straight from its inputs, without the logits.
//
//   l[t, v] = sum_k X[t, k] W[v, k]          lse_t = log sum_v exp(l[t, v])
//   loss_t  = lse_t - l[t, y_t]              (0 where y_t is outside [0, V))
//   dl[t, v] = (exp(l[t, v] - lse_t) - [v = y_t]) * g_t     g_t = d(total) / d(loss_t)
//   grad_X = dl W,  grad_W = dl^T X
//
// Forward: one pass of the CTA-pair product of gemm_tc2.cuh whose epilogue reduces each
// 128-column strip of logits in registers to its maximum and its sum of exponentials (fp32,
// the logits never rounded), so a token leaves 8 bytes per 128 columns of the vocabulary
// instead of 512; a small kernel joins the strips in a fixed order.
// Backward, one piece of the vocabulary after another: the logits of the piece are computed
// again, their epilogue writes dl of the piece in bf16 (the operand type of the tensor
// cores: one rounding of at most half a step per factor), and two products consume it,
// grad_W of the piece's rows and the piece's addend of grad_X, summed in fp32. Four
// products of 2 T V K operations in all against three with all logits kept (T x V).
// Bound by the bf16 tensor pipe; W's stream (2 bytes per weight) for few tokens.
//
// The kernel takes up to three products with their own operand orders, depths and
// epilogues in one launch (their tiles numbered consecutively), so that the products of a
// piece fill the SMs together. Synchronisation, stages and TMEM use as in gemm_tc2.cuh.
#pragma once

#include "gemm_tc2.cuh"

namespace bl {

enum CeMode : int {
  CE_LSE = 0,       // strip maxima and sums of exponentials, and the target's logit
  CE_DLOGITS = 1,   // dl in bf16
  CE_BF16 = 2,      // the product, bf16
  CE_F32 = 3,       // the product, fp32
  CE_ADD_F32 = 4,   // the product added to fp32 memory
};

struct CeProblem {
  CUtensorMap tmA, tmB, tmOut;   // tmOut unused by CE_LSE
  int mode;
  int a_mn, b_mn;                // operand order: 0 K-major, 1 MN-major
  int M, N;
  int num_k_blocks;              // ceil(K / 64)
  int num_m_blocks, num_n_blocks;   // 256 x 256 tiles
  int m_fastest;
  int tile_begin;
  int v0;                        // first vocabulary row of the piece (CE_DLOGITS)
};
constexpr int kMaxCeGroup = 3;
struct CeGroup {
  CeProblem p[kMaxCeGroup];
  int count, total_tiles;
  int64_t v;                     // vocabulary size
  const int64_t* targets;        // [T]
  const float* lse;              // [T]  (CE_DLOGITS)
  const float* grad;             // [T]  (CE_DLOGITS)
  float2* strips;                // [2 * n blocks, T] (max, sum)  (CE_LSE)
  float* target_logit;           // [T]  (CE_LSE)
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// fp32 tile added to global memory by the TMA engine (one add per element and launch, so
// the order of additions is the order of launches).
__device__ __forceinline__ void tma_add_2d(const CUtensorMap* map, uint32_t src, int c0, int c1) {
  asm volatile("cp.reduce.async.bulk.tensor.2d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(c0), "r"(c1)
               : "memory");
}
__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ int ce_problem(const CeGroup& G, int tile) {
  int i = 0;
#pragma unroll
  for (int j = 1; j < kMaxCeGroup; ++j) i += (j < G.count && tile >= G.p[j].tile_begin) ? 1 : 0;
  return i;
}
__device__ __forceinline__ void ce_tile(const CeProblem& P, int tile, int& mb, int& nb) {
  if (P.m_fastest) {
    mb = tile % P.num_m_blocks;
    nb = tile / P.num_m_blocks;
  } else {
    mb = tile / P.num_n_blocks;
    nb = tile % P.num_n_blocks;
  }
}

// Epilogue of 32 rows x 128 columns of logits: one strip of one token per thread.
__device__ __forceinline__ void ce_strip(const CeGroup& G, const CeProblem& P, uint32_t t_row, int row, int n0, int strip) {
  float m = -INFINITY, s = 0.f;   // m in units of log2
  const bool row_ok = row < P.M;
  const int64_t rel = row_ok ? G.targets[row] - n0 : -1;
#pragma unroll 1
  for (int c = 0; c < 4; ++c) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(c * 32), r);
    tmem_ld_wait();
    const int left = P.N - n0 - c * 32;   // columns of the vocabulary in this piece
    if (left <= 0) break;
    if (left < 32) {
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j >= left) r[j] = 0xFF800000u;
    }
    const int64_t hit = rel - c * 32;
    if (hit >= 0 && hit < 32 && hit < left) {
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (j == static_cast<int>(hit)) t = __uint_as_float(r[j]);
      G.target_logit[row] = t;
    }
    float cm[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) cm[j] = __uint_as_float(r[j]);
#pragma unroll
    for (int j = 4; j < 32; ++j) cm[j & 3] = fmaxf(cm[j & 3], __uint_as_float(r[j]));
    const float m2 = fmaxf(m, fmaxf(fmaxf(cm[0], cm[1]), fmaxf(cm[2], cm[3])) * kLog2e);
    float a[4] = {s * ex2(m - m2), 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < 32; ++j) a[j & 3] += ex2(fmaf(__uint_as_float(r[j]), kLog2e, -m2));
    s = (a[0] + a[1]) + (a[2] + a[3]);
    m = m2;
  }
  if (row_ok) G.strips[static_cast<int64_t>(strip) * P.M + row] = make_float2(m, s);
}

// Epilogue of 32 rows x 128 columns through shared memory: dl, or the product itself.
__device__ __forceinline__ void ce_store(const CeGroup& G, const CeProblem& P, uint32_t t_row, uint32_t stg, int& cnt, int row0,
                                         int n0, int lane) {
  const bool f32 = P.mode >= CE_F32;
  const int cols = f32 ? 32 : 64;
  float lse2 = 0.f, grad = 0.f;
  int64_t rel = -1;
  if (P.mode == CE_DLOGITS && row0 + lane < P.M) {
    const int64_t y = G.targets[row0 + lane];
    if (y >= 0 && y < G.v) {
      grad = G.grad[row0 + lane];
      lse2 = G.lse[row0 + lane] * kLog2e;
      rel = y - P.v0 - n0;
    }
  }
#pragma unroll 1
  for (int c = 0; c < 128; c += cols, ++cnt) {
    uint32_t w[32];   // the 128 bytes of this thread's row
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (h == 1 && f32) break;
      uint32_t r[32];
      tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(c + 32 * h), r);
      tmem_ld_wait();
      if (P.mode == CE_DLOGITS) {
        const int64_t hit = rel - c - 32 * h;
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(ex2(fmaf(__uint_as_float(r[j]), kLog2e, -lse2)));
        if (hit >= 0 && hit < 32) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (j == static_cast<int>(hit)) r[j] = __float_as_uint(__uint_as_float(r[j]) - 1.f);
        }
        // a token without a loss has no gradient, whatever its logits are
#pragma unroll
        for (int j = 0; j < 32; ++j) r[j] = grad == 0.f ? 0u : __float_as_uint(__uint_as_float(r[j]) * grad);
      }
      if (f32) {
#pragma unroll
        for (int j = 0; j < 32; ++j) w[j] = r[j];
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) w[16 * h + j] = pack_bf16x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
      }
    }
    if (cnt >= 1) {
      if (lane == 0) bulk_wait_group_read<0>();   // the previous store has finished reading the buffer
      __syncwarp();
    }
    const uint32_t row_addr = stg + static_cast<uint32_t>(lane) * 128u;
#pragma unroll
    for (int j = 0; j < 8; ++j)
      st_shared_v4(row_addr + static_cast<uint32_t>((j ^ (lane & 7)) * 16), w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (P.mode == CE_ADD_F32) tma_add_2d(&P.tmOut, stg, n0 + c, row0);
      else tma_store_2d(&P.tmOut, stg, n0 + c, row0);
      bulk_commit_group();
    }
  }
}

__global__ void __launch_bounds__(kGemmThreads, 1) ce_gemm_kernel(const __grid_constant__ CeGroup G) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  const uint32_t sA = base;
  const uint32_t sB = base + kStages2 * kAHalfBytes;
  const uint32_t sOut = base + kStages2 * kStage2Bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages2 * kStage2Bytes + kOutStagingBytes);
  const uint32_t bar0 = smem_u32(bars);
  const uint32_t full0 = bar0, empty0 = bar0 + 8u * kStages2;
  const uint32_t tfull0 = bar0 + 16u * kStages2, tempty0 = tfull0 + 16u, done_bar = tempty0 + 16u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages2 + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages2; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8u * b, 1);
      mbar_init(tempty0 + 8u * b, 2 * kEpiWarps);
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int i = 0; i < G.count; ++i) {
      tma_prefetch_desc(&G.p[i].tmA);
      tma_prefetch_desc(&G.p[i].tmB);
      if (G.p[i].mode != CE_LSE) tma_prefetch_desc(&G.p[i].tmOut);
    }
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_slot), kTmemCols);
    tmem_relinquish_pair();
  }
  tc_fence_before_sync();
  cluster_sync();   // barriers of both CTAs initialised, TMEM allocated in both
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_slot;
  const uint32_t peer_abort = map_to_rank(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u);
  const int num_tiles = G.total_tiles;
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------- TMA producer (both CTAs)
    if (lane == 0) {
      const uint32_t full_leader0 = map_to_rank(full0, 0);
      int s = 0;
      uint32_t ph = 0;
      long long issued = 0;
      bool ok = true;
      int local = 0;
      for (int tile = cluster; tile < num_tiles && ok; tile += nclusters, ++local) {
        const CeProblem& P = G.p[ce_problem(G, tile)];
        int mb, nb;
        ce_tile(P, tile - P.tile_begin, mb, nb);
        const int m0 = mb * 256 + 128 * static_cast<int>(rank);
        const int n0 = nb * 256 + 128 * static_cast<int>(rank);
        for (int kq = 0; kq < P.num_k_blocks; ++kq) {
          const int kb = (local & 1) ? P.num_k_blocks - 1 - kq : kq;   // serpentine K order
          if (!mbar_wait(empty0 + 8u * s, ph ^ 1u, abort_flag)) {
            ok = false;
            break;
          }
          const uint32_t fb = full_leader0 + 8u * s;
          if (leader) mbar_arrive_expect_tx(full0 + 8u * s, 2 * kStage2Bytes);
          const uint32_t a_dst = sA + s * kAHalfBytes, b_dst = sB + s * kBHalfBytes;
          const int kc = kb * 64;
          if (P.a_mn) {
            tma_load_2d_pair(a_dst, &P.tmA, fb, m0, kc);
            tma_load_2d_pair(a_dst + 8192, &P.tmA, fb, m0 + 64, kc);
          } else {
            tma_load_2d_pair(a_dst, &P.tmA, fb, kc, m0);
          }
          if (P.b_mn) {
            tma_load_2d_pair(b_dst, &P.tmB, fb, n0, kc);
            tma_load_2d_pair(b_dst + 8192, &P.tmB, fb, n0 + 64, kc);
          } else {
            tma_load_2d_pair(b_dst, &P.tmB, fb, kc, n0);
          }
          ++issued;
          if (++s == kStages2) {
            s = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok) {
        pair_abort(abort_flag, peer_abort);
        atomicOr(&g_device_status, DEV_ST_TIMEOUT_PRODUCER);
        if (leader) {   // the leader's full barriers count both CTAs' copies: drain them
          const long long first = issued > kStages2 ? issued - kStages2 : 0;
          for (long long i = first; i < issued; ++i)
            if (!mbar_wait_plain(full0 + 8u * static_cast<uint32_t>(i % kStages2), static_cast<uint32_t>((i / kStages2) & 1)))
              atomicOr(&g_device_status, DEV_ST_TIMEOUT_DRAIN);
        }
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer (leader only)
    if (lane == 0 && leader) {
      int s = 0;
      uint32_t ph = 0;
      int local = 0;
      bool ok = true;
      for (int tile = cluster; tile < num_tiles && ok; tile += nclusters, ++local) {
        const CeProblem& P = G.p[ce_problem(G, tile)];
        const uint32_t idesc = make_idesc(1u, 1u, 1u, P.a_mn, P.b_mn, 256, 256);
        // K-major: a K step of 16 is 32 B inside the swizzled row; MN-major: 16 K rows = 2 KB
        const uint32_t a_step = P.a_mn ? 2048u : 32u, b_step = P.b_mn ? 2048u : 32u;
        const uint32_t a_lbo = P.a_mn ? 8192u : 16u, b_lbo = P.b_mn ? 8192u : 16u;
        const int buf = local & 1;
        const uint32_t tph = static_cast<uint32_t>(local >> 1) & 1u;
        if (!mbar_wait(tempty0 + 8u * buf, tph ^ 1u, abort_flag)) {
          ok = false;
          break;
        }
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(buf * kBN);
        const int nk = P.num_k_blocks;
        for (int kb = 0; kb < nk; ++kb) {
          if (!mbar_wait(full0 + 8u * s, ph, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t a_base = sA + s * kAHalfBytes, b_base = sB + s * kBHalfBytes;
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)
            tc_mma_f16_pair(d_tmem, make_sw128_desc(a_base + kk * a_step, a_lbo, 1024),
                            make_sw128_desc(b_base + kk * b_step, b_lbo, 1024), idesc, (kb | kk) != 0 ? 1u : 0u);
          tc_commit_pair(empty0 + 8u * s);   // frees this stage in both CTAs
          if (++s == kStages2) {
            s = 0;
            ph ^= 1u;
          }
        }
        if (!ok) break;
        tc_commit_pair(tfull0 + 8u * buf);   // both CTAs' accumulators complete
      }
      if (!ok) {
        pair_abort(abort_flag, peer_abort);
        atomicOr(&g_device_status, DEV_ST_TIMEOUT_MMA);
      }
      tc_commit_pair_local(done_bar);
      if (!mbar_wait_plain(done_bar, 0)) atomicOr(&g_device_status, DEV_ST_TIMEOUT_DRAIN);
    }
  } else {
    // ------------------------------------------------------------- epilogue (warps 2..9, both CTAs)
    const int e = warp - 2;
    const int quad = warp & 3;
    const int half = e >> 2;   // columns [128 half, 128 half + 128) of the tile
    const uint32_t stg = sOut + static_cast<uint32_t>(e * kStageOutBytes);
    const uint32_t tempty_leader0 = map_to_rank(tempty0, 0);
    int cnt = 0;
    int local = 0;
    bool ok = true;
    for (int tile = cluster; tile < num_tiles; tile += nclusters, ++local) {
      const int buf = local & 1;
      const uint32_t tph = static_cast<uint32_t>(local >> 1) & 1u;
      const CeProblem& P = G.p[ce_problem(G, tile)];
      int mb, nb;
      ce_tile(P, tile - P.tile_begin, mb, nb);
      const int row0 = mb * 256 + 128 * static_cast<int>(rank) + quad * 32;
      const int n0 = nb * 256 + 128 * half;
      const bool got = mbar_wait(tfull0 + 8u * buf, tph, abort_flag);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t t_row = tmem_base + static_cast<uint32_t>(buf * kBN + 128 * half) + (static_cast<uint32_t>(quad * 32) << 16);
      if (P.mode == CE_LSE) ce_strip(G, P, t_row, row0 + lane, n0, nb * 2 + half);
      else ce_store(G, P, t_row, stg, cnt, row0, n0, lane);
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
    tmem_dealloc_pair(tmem_base, kTmemCols);
  }
}

// Joins the strips of each token: 32 tokens x 8 slices of the strips per block, the
// slices' (max, sum) pairs joined in order.
__global__ void __launch_bounds__(256) ce_join_kernel(const float2* strips, int num_strips, int64_t t, int64_t v,
                                                      const int64_t* targets, const float* target_logit, float* loss,
                                                      float* lse) {
  __shared__ float2 s_part[8][32];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  float m = -INFINITY, s = 0.f;
  if (row < t)
    for (int i = slice; i < num_strips; i += 8) {
      const float2 p = strips[static_cast<int64_t>(i) * t + row];
      if (p.y == 0.f) continue;   // a strip past the vocabulary's end
      const float m2 = fmaxf(m, p.x);
      s = s * ex2(m - m2) + p.y * ex2(p.x - m2);
      m = m2;
    }
  s_part[slice][lane] = make_float2(m, s);
  __syncthreads();
  if (slice == 0 && row < t) {
    float mm = s_part[0][lane].x;
#pragma unroll
    for (int i = 1; i < 8; ++i) mm = fmaxf(mm, s_part[i][lane].x);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (s_part[i][lane].y != 0.f) ss += s_part[i][lane].y * ex2(s_part[i][lane].x - mm);
    const float l = mm * 0.6931471805599453f + logf(ss);
    const int64_t y = targets[row];
    lse[row] = l;
    loss[row] = y >= 0 && y < v ? l - target_logit[row] : 0.f;
  }
}

// fp32 -> bf16, 8 elements per thread and step.
__global__ void __launch_bounds__(256) ce_round_kernel(const float4* src, int64_t n8, uint4* dst) {
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n8; i += static_cast<int64_t>(gridDim.x) * 256) {
    const float4 a = __ldg(src + 2 * i), b = __ldg(src + 2 * i + 1);
    dst[i] = make_uint4(pack_bf16x2(a.x, a.y), pack_bf16x2(a.z, a.w), pack_bf16x2(b.x, b.y), pack_bf16x2(b.z, b.w));
  }
}

}  // namespace bl
