// Softmax cross entropy of a linear head straight from its inputs, without the logits.
//
//   l[t, v] = sum_k X[t, k] W[v, k]          lse_t = log sum_v exp(l[t, v])
//   loss_t  = lse_t - l[t, y_t]              (0 where y_t is outside [0, V))
//   dl[t, v] = (exp(l[t, v] - lse_t) - [v = y_t]) * g_t     g_t = d(total) / d(loss_t)
//   grad_X = dl W,  grad_W = dl^T X
//
// Forward: one pass of a CTA-pair product whose epilogue reduces each 128-column strip of
// logits but the target's in registers to its maximum and its sum of exponentials (fp32, the
// logits never rounded), so a token leaves 8 bytes per 128 columns of the vocabulary instead
// of 512; a small kernel joins the strips in a fixed order. The tensor core's accumulator
// drops the bits of an addend below its own last one, always towards zero, half a unit per MMA
// on average: a logit of 18 over K = 2048 came out 4e-5 too small. So the accumulator starts
// afresh every 512 of K and the parts are added in registers, rounded to nearest: 2^-20 of a
// logit at any K.
// Backward, one piece of the vocabulary after another: the logits of the piece are computed
// again, their epilogue writes dl of the piece in bf16 (the operand type of the tensor cores:
// one rounding of at most half a step per factor; few tokens as the sum of two, see
// kCeSplitTokens), and two products consume it, grad_W of the piece's rows and the piece's
// addend of grad_X, summed in fp32. dl of a target is exp(l_y - lse) - 1, of a sure token a
// small difference: l_y has to be off by what it was off by in the forward pass's lse (a
// logit from one accumulation of K = 2048 made dl of one token 4.5e-5 instead of 0.9e-5). So
// both passes take the same dot product, or the same parts (ce_dots). Tokens without a loss
// (padding, prompts) are left out first: the others' rows are gathered to the front, the
// products stop after them, and grad_X is scattered back. Four products of 2 T V K operations
// in all against three with all logits kept (T x V). g is divided by its largest magnitude
// before that rounding and the gradients multiplied by it after: with the usual constant g, dl
// of a target is then p - 1 itself, not a product whose rounding error every token would
// share.
// Bound by the bf16 tensor pipe (and the power it draws).
//
// The kernel takes up to three products with their own operand orders, depths and
// epilogues in one launch, so that the two products of one piece and the logits of the next
// fill the SMs together (ce_shares.cuh).
// Stages, synchronisation and TMEM use as in gemm_tc2.cuh.
#pragma once

#include <cfloat>
#include <climits>

#include "ce_shares.cuh"
#include "gemm_sp2.cuh"
#include "pair_issue.cuh"

namespace bl {

enum CeMode : int {
  CE_LSE = 0,       // strip maxima and sums of exponentials, without the target's
  CE_DLOGITS = 1,   // dl in bf16
  CE_BF16 = 2,      // the product times the largest |g|, bf16
  CE_F32 = 3,       // the product times the largest |g|, fp32
  CE_PART = 4,      // the product, fp32
  CE_ADD_PART = 5,  // the product added to fp32 memory
};

struct CeProblem {
  CUtensorMap tmA, tmB, tmOut;   // tmOut unused by CE_LSE
  int mode;
  int a_mn, b_mn;                // operand order: 0 K-major, 1 MN-major
  int M, N;
  int num_k_blocks;              // ceil(K / 64)
  int num_m_blocks, num_n_blocks;   // 256 x 256 tiles
  // CE_PART, CE_ADD_PART: K in `splits` runs of split_blocks, run i to output rows from
  // i * 256 num_m_blocks on (1 run otherwise)
  int splits, split_blocks;
  int live_m, live_k;            // rows (A's rows) or K blocks end with the live tokens
  int m_fastest;
  int v0;                        // first vocabulary row of the piece (CE_DLOGITS)
};
constexpr int kMaxCeGroup = 3;
struct CeGroup {
  CeProblem p[kMaxCeGroup];
  CeShares share[kMaxCeGroup];
  int count;
  int64_t v;                     // vocabulary size
  // CE_LSE: the targets' logits are dot products of these rows of 8 row8 (x null: the product's)
  const uint4 *x, *w;
  int row8;
  const int64_t* targets;        // [T]  (CE_LSE)
  // backward: the tokens with a loss in order (a few of them a second time, for their low
  // halves), then zeros (target -1) up to 256 rows
  const int* live;               // rows of them, at least 1
  const int* low;                // first of their low halves' rows (INT_MAX: none)
  const int* row_target;
  const float* row_lse;
  const float* row_grad;         // g over the largest |g|
  const float* grad_max;         // the largest finite |g|, or 1
  const int* from;               // the live tokens
  const float* target_dl;        // [T] dl of the targets over g (null: from the product's logits)
  float2* strips;                // [2 * n blocks, T] (max, sum)  (CE_LSE)
  float* target_logit;           // [T]  (CE_LSE)
};

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Maximum of a strip's logits in units of log2, kept finite: with logits of -infinity alone
// its exponentials then add up to 0, with one of +infinity to infinity, never to inf - inf.
__device__ __forceinline__ float strip_max(float m2) { return fminf(fmaxf(m2, -FLT_MAX), FLT_MAX); }
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

__device__ __forceinline__ void st_shared_bf16(uint32_t addr, __nv_bfloat16 v) {
  asm volatile("st.shared.b16 [%0], %1;" ::"r"(addr), "h"(__bfloat16_as_ushort(v)) : "memory");
}

// Blocks of a tile and its run of K blocks [kb0, kb1), empty behind the live tokens.
struct CeTile {
  int mb, nb, split, kb0, kb1;
};
__device__ __forceinline__ CeTile ce_tile(const CeProblem& P, int tile, int live) {
  CeTile T;
  const int per = P.num_m_blocks * P.num_n_blocks;
  T.split = P.splits > 1 ? tile / per : 0;
  tile -= T.split * per;
  if (P.m_fastest) {
    T.mb = tile % P.num_m_blocks;
    T.nb = tile / P.num_m_blocks;
  } else {
    T.mb = tile / P.num_n_blocks;
    T.nb = tile % P.num_n_blocks;
  }
  T.kb0 = T.split * P.split_blocks;
  T.kb1 = min(T.kb0 + P.split_blocks, P.live_k ? min(P.num_k_blocks, (live + 63) >> 6) : P.num_k_blocks);
  if (P.live_m && T.mb * 256 >= live) T.kb1 = T.kb0;
  return T;
}

// K blocks per accumulation of the logits: 512 of K in the forward pass, where the backward
// pass has its targets' logits from them too, and where dl is held as two numbers. Else one
// bf16 number (half a step 2^-8) does not show what 4096 of K lose, 2^-17 of a logit, and
// parts of 512 made the backward pass longer: 8192 x 2048 x 32768 2.28 -> 2.37 ms, 2047 x 1536
// x 32003 440 -> 452 us.
constexpr int kCePartBlocks = 8, kCeLongPartBlocks = 64;
__device__ __forceinline__ int ce_part_blocks(const CeProblem& P, bool short_parts) {
  return P.mode == CE_LSE || (P.mode == CE_DLOGITS && short_parts) ? kCePartBlocks
         : P.mode == CE_DLOGITS                                    ? kCeLongPartBlocks
                                                                   : P.num_k_blocks;
}

// The accumulator's 32 rows x 128 columns of one warp: thread = row, acc[c][j] = column 32 c + j.
using CeAcc = float[4][32];

// One strip of one token per thread.
__device__ __forceinline__ void ce_strip(const CeGroup& G, const CeProblem& P, CeAcc& acc, int row, int n0, int strip) {
  const int left = P.N - n0;   // columns of the vocabulary in the strip
  if (row >= P.M) return;
  const int64_t hit = G.targets[row] - n0;
  if (hit >= 0 && hit < 128 && hit < left) {
    float t = 0.f;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < 32; ++j)
      {   // two selects: a branch around them spills registers
        const bool is = 32 * c + j == static_cast<int>(hit);
        t = is ? acc[c][j] : t;
        acc[c][j] = is ? -INFINITY : acc[c][j];
      }
    if (!G.x) G.target_logit[row] = t;
  }
  if (left < 128) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < 32; ++j)
        if (32 * c + j >= left) acc[c][j] = -INFINITY;
  }
  float m[4], s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    m[c] = acc[c][0];
#pragma unroll
    for (int j = 1; j < 32; ++j) m[c] = fmaxf(m[c], acc[c][j]);
  }
  const float m2 = strip_max(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * kLog2e);
  if (left > 0) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < 32; ++j) s[j & 3] += ex2(fmaf(acc[c][j], kLog2e, -m2));
  }
  G.strips[static_cast<int64_t>(strip) * P.M + row] = make_float2(m2, (s[0] + s[1]) + (s[2] + s[3]));
}

// x . w of one row each, by a warp in fp32: the loss and a target's dl depend on the target's
// logit with nothing to average over, and the tensor core's lost bits left one token's loss
// (2048 x 32768, 40 draws) up to 1.4e-6 off; now 2.1e-7. Every lane returns the sum.
__device__ __forceinline__ float ce_dot(const uint4* x, const uint4* w, int row8, int lane) {
  auto low = [](uint32_t p) { return __uint_as_float(p << 16); };
  auto high = [](uint32_t p) { return __uint_as_float(p & 0xFFFF0000u); };
  float dot = 0.f;
#pragma unroll 4
  for (int j = lane; j < row8; j += 32) {
    const uint4 p = ld_plain(x + j), q = ld_plain(w + j);
    float part = low(p.x) * low(q.x);
    part = fmaf(high(p.x), high(q.x), part);
    part = fmaf(low(p.y), low(q.y), part);
    part = fmaf(high(p.y), high(q.y), part);
    part = fmaf(low(p.z), low(q.z), part);
    part = fmaf(high(p.z), high(q.z), part);
    part = fmaf(low(p.w), low(q.w), part);
    dot += fmaf(high(p.w), high(q.w), part);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
  return dot;
}

// Of the targets of tokens i, i + step, ..., `most` of them at most, by a warp: the logits, or
// with lse their dl over g, exp(l - lse) - 1 (in one: of a sure token it is far below the
// roundings of exp(l - lse)). i is the next token after them.
__device__ __forceinline__ void ce_targets(const uint4* x, const uint4* w, const int64_t* targets, const float* lse, int64_t t, int64_t v,
                                           int row8, int64_t& i, int64_t step, int most, int lane, float* out) {
  for (; i < t && most > 0; i += step, --most) {
    const int64_t y = targets[i];
    if (y < 0 || y >= v) continue;
    const float l = ce_dot(x + i * row8, w + y * row8, row8, lane);
    if (lane == 0) out[i] = lse ? expm1f(l - lse[i]) : l;
  }
}

// dl of a row's target from that of its token.
__device__ __forceinline__ __nv_bfloat16 ce_target_dl(const CeGroup& G, int row) {
  const int first_low = *G.low;
  const bool low = row >= first_low;
  const float g = G.row_grad[row];
  const float dl = g == 0.f ? 0.f : G.target_dl[G.from[low ? row - first_low : row]] * g;
  const __nv_bfloat16 first = __float2bfloat16_rn(dl);
  return low ? __float2bfloat16_rn(dl - __bfloat162float(first)) : first;
}

// 32 rows x 128 columns through shared memory: dl, or the product itself.
__device__ __forceinline__ void ce_store(const CeGroup& G, const CeProblem& P, CeAcc& acc, uint32_t stg, int row0, int n0,
                                         int lane) {
  const int row = row0 + lane;
  int hit = -1;   // the target's column, if it is among these 128
  if (P.mode == CE_DLOGITS) {
    const float lse2 = G.row_lse[row] * kLog2e, g = G.row_grad[row];
    const bool low = row >= *G.low;
    hit = G.row_target[row] - P.v0 - n0;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < 32; ++j) acc[c][j] = ex2(fmaf(acc[c][j], kLog2e, -lse2));
    if (!G.target_dl && hit >= 0 && hit < 128) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 32; ++j)
          if (32 * c + j == hit) acc[c][j] -= 1.f;
    }
    // rows behind the last token: zeros
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < 32; ++j) acc[c][j] = g == 0.f ? 0.f : acc[c][j] * g;
    if (low) {   // what the rounding of the token's first row leaves
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 32; ++j) acc[c][j] -= __bfloat162float(__float2bfloat16_rn(acc[c][j]));
    }
  } else if (P.mode <= CE_F32) {
    const float scale = *G.grad_max;
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < 32; ++j) acc[c][j] *= scale;
  }
  const uint32_t row_addr = stg + static_cast<uint32_t>(lane) * 128u;
  auto put = [&](int j, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {   // 128B swizzle
    st_shared_v4(row_addr + static_cast<uint32_t>((j ^ (lane & 7)) * 16), a, b, c, d);
  };
  auto free_buffer = [&]() {   // the previous store has finished reading the buffer
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  };
  auto store = [&](int col) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      if (n0 + col < P.N) {
        if (P.mode == CE_ADD_PART) tma_add_2d(&P.tmOut, stg, n0 + col, row0);
        else tma_store_2d(&P.tmOut, stg, n0 + col, row0);
      }
      bulk_commit_group();
    }
  };
  if (P.mode >= CE_F32) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      free_buffer();
#pragma unroll
      for (int j = 0; j < 8; ++j)
        put(j, __float_as_uint(acc[c][4 * j]), __float_as_uint(acc[c][4 * j + 1]), __float_as_uint(acc[c][4 * j + 2]),
            __float_as_uint(acc[c][4 * j + 3]));
      store(32 * c);
    }
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      free_buffer();
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float* f = &acc[2 * h + (j >> 2)][8 * (j & 3)];
        put(j, pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
      }
      if (G.target_dl && hit >> 6 == h) {   // the target's dl over the p that is there
        const uint32_t at = row_addr + static_cast<uint32_t>(((hit >> 3 & 7) ^ (lane & 7)) * 16 + (hit & 7) * 2);
        st_shared_bf16(at, ce_target_dl(G, row));
      }
      store(64 * h);
    }
  }
}

__global__ void __launch_bounds__(kGemmThreads, 1) ce_gemm_kernel(const __grid_constant__ CeGroup G) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (base - raw);
  auto st_a = [&](int s) { return base + static_cast<uint32_t>(s * kStage2Bytes); };   // this CTA's 128 rows of A
  auto st_b = [&](int s) { return st_a(s) + kAHalfBytes; };                           // and of B
  const uint32_t sOut = base + kStages2 * kStage2Bytes;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + kStages2 * kStage2Bytes + kOutStagingBytes);
  const uint32_t bar0 = smem_u32(bars);
  const uint32_t full0 = bar0, empty0 = bar0 + 8u * kStages2;
  const uint32_t tfull0 = bar0 + 16u * kStages2, tempty0 = tfull0 + 16u, done_bar = tempty0 + 16u;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + 2 * kStages2 + 5);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const uint32_t rank = cluster_ctarank();
  const bool leader = rank == 0;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // warp-uniform
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
  follow_stream();
  const uint32_t tmem_base = __reduce_or_sync(0xffffffffu, *tmem_slot);   // the same in every lane: a uniform register
  const uint32_t peer_abort = map_to_rank(smem_u32(const_cast<int*>(abort_flag)), rank ^ 1u);
  const int cluster = blockIdx.x >> 1, nclusters = gridDim.x >> 1;
  const bool short_parts =
      G.low && (!G.target_dl || __reduce_min_sync(0xffffffffu, static_cast<unsigned>(ld_plain(G.low))) != INT_MAX);
  const int live_rows = G.live ? static_cast<int>(__reduce_max_sync(0xffffffffu, static_cast<unsigned>(ld_plain(G.live)))) : 0;

  if (warp == 0) {
    // ------------------------------------------------------------- TMA producer (both CTAs)
    const uint32_t full_leader0 = __reduce_or_sync(0xffffffffu, map_to_rank(full0, 0));
    uint32_t live = 1;   // 0 after a wait gave up: the loops run out without issuing or waiting
    int s = 0;
    uint32_t ph = 0;
    uint32_t issued = 0;
    for (int j = 0; j < G.count; ++j) {
      const CeProblem& P = G.p[j];
      const int rounds = G.share[j].count[cluster], pos = G.share[j].pos[cluster];
      for (int r = 0; r < rounds; ++r) {
        const CeTile T = ce_tile(P, ce_round_tile(G.share[j], nclusters, pos, r), live_rows);
        const int m0 = T.mb * 256 + 128 * static_cast<int>(rank);
        const int n0 = T.nb * 256 + 128 * static_cast<int>(rank);
        for (int kb = T.kb0; kb < T.kb1; ++kb) {
          live = wait_live<false>(live, empty0 + 8u * s, ph ^ 1u, abort_flag, peer_abort);
          const uint32_t fb = full_leader0 + 8u * s;
          const int kc = kb * 64;
          if (elect_one() && live) {
            if (leader) mbar_arrive_expect_tx(full0 + 8u * s, 2 * kStage2Bytes);
            if (P.a_mn) {
              tma_load_2d_pair(st_a(s), &P.tmA, fb, m0, kc);
              tma_load_2d_pair(st_a(s) + 8192, &P.tmA, fb, m0 + 64, kc);
            } else {
              tma_load_2d_pair(st_a(s), &P.tmA, fb, kc, m0);
            }
            if (P.b_mn) {
              tma_load_2d_pair(st_b(s), &P.tmB, fb, n0, kc);
              tma_load_2d_pair(st_b(s) + 8192, &P.tmB, fb, n0 + 64, kc);
            } else {
              tma_load_2d_pair(st_b(s), &P.tmB, fb, kc, n0);
            }
          }
          issued += live;
          if (++s == kStages2) {
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
        const uint32_t first = issued > kStages2 ? issued - kStages2 : 0;
        for (uint32_t i = first; i < issued; ++i)
          if (!mbar_wait_plain(full0 + 8u * (i % kStages2), (i / kStages2) & 1u)) atomicOr(&g_device_status, DEV_ST_TIMEOUT_DRAIN);
      }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer (leader only)
    if (leader) {
      uint32_t live = 1;
      int s = 0;
      uint32_t ph = 0;
      uint32_t unit = 0;   // accumulations so far: unit u is in buffer u & 1
      for (int j = 0; j < G.count; ++j) {
        const CeProblem& P = G.p[j];
        const int rounds = G.share[j].count[cluster], pos = G.share[j].pos[cluster];
        const uint32_t idesc = make_idesc(1u, 1u, 1u, P.a_mn, P.b_mn, 256, 256);
        // a K step of 16 in the address field (16-byte units): K-major 32 B inside the
        // swizzled row, MN-major 16 K rows = 2 KB
        const uint64_t a_step = P.a_mn ? 128u : 2u, b_step = P.b_mn ? 128u : 2u;
        const uint32_t a_lbo = P.a_mn ? 8192u : 16u, b_lbo = P.b_mn ? 8192u : 16u;
        const int part = ce_part_blocks(P, short_parts);
        for (int r = 0; r < rounds; ++r) {
          const CeTile T = ce_tile(P, ce_round_tile(G.share[j], nclusters, pos, r), live_rows);
          for (int k0 = T.kb0; k0 < T.kb1; k0 += part, ++unit) {
            const uint32_t buf = unit & 1u;
            const int end = min(k0 + part, T.kb1);
            live = wait_live<false>(live, tempty0 + 8u * buf, ((unit >> 1) & 1u) ^ 1u, abort_flag, peer_abort);
            tc_fence_after_sync();
            const uint32_t d_tmem = tmem_base + buf * kBN;
            for (int kb = k0; kb < end; ++kb) {
              live = wait_live<false>(live, full0 + 8u * s, ph, abort_flag, peer_abort);
              tc_fence_after_sync();
              if (elect_one() && live) {
                const uint64_t ad = make_sw128_desc(st_a(s), a_lbo, 1024), bd = make_sw128_desc(st_b(s), b_lbo, 1024);
#pragma unroll
                for (int kk = 0; kk < 4; ++kk)
                  tc_mma_f16_pair(d_tmem, ad + a_step * kk, bd + b_step * kk, idesc, kb > k0 || kk != 0 ? 1u : 0u);
                tc_commit_pair(empty0 + 8u * s);   // frees this stage in both CTAs
                if (kb + 1 == end) tc_commit_pair(tfull0 + 8u * buf);   // both CTAs' accumulators complete
              }
              if (++s == kStages2) {
                s = 0;
                ph ^= 1u;
              }
            }
          }
        }
      }
      if (elect_one()) {
        if (!live) atomicOr(&g_device_status, DEV_ST_TIMEOUT_MMA);
        tc_commit_pair_local(done_bar);
        if (!mbar_wait_plain(done_bar, 0)) atomicOr(&g_device_status, DEV_ST_TIMEOUT_DRAIN);
      }
    }
  } else {
    // ------------------------------------------------------------- epilogue (warps 2..9, both CTAs)
    const int e = warp - 2;
    const int quad = warp & 3;
    const int half = e >> 2;   // columns [128 half, 128 half + 128) of the tile
    const uint32_t stg = sOut + static_cast<uint32_t>(e * kStageOutBytes);
    const uint32_t tempty_leader0 = map_to_rank(tempty0, 0);
    uint32_t unit = 0;
    bool ok = true;
    // the targets' logits, while tiles are on their way: a few before each, so that no other
    // warp waits long for this one, what is left of them at the end
    int64_t token = static_cast<int64_t>(blockIdx.x) * kEpiWarps + e;
    auto target_logits = [&](int most) {
      ce_targets(G.x, G.w, G.targets, nullptr, G.p[0].M, G.v, G.row8, token, static_cast<int64_t>(gridDim.x) * kEpiWarps, most, lane,
                 G.target_logit);
    };
    for (int j = 0; j < G.count && ok; ++j) {
      const CeProblem& P = G.p[j];
      const int rounds = G.share[j].count[cluster], pos = G.share[j].pos[cluster];
      const int part = ce_part_blocks(P, short_parts);
      for (int r = 0; r < rounds && ok; ++r) {
        const CeTile T = ce_tile(P, ce_round_tile(G.share[j], nclusters, pos, r), live_rows);
        const int row0 = T.mb * 256 + 128 * static_cast<int>(rank) + quad * 32;
        const int n0 = T.nb * 256 + 128 * half;
        if (G.x) target_logits(8);
        CeAcc acc;
#pragma unroll 1
        for (int k0 = T.kb0; k0 < T.kb1; k0 += part, ++unit) {
          const uint32_t buf = unit & 1u;
          const bool got = mbar_wait(tfull0 + 8u * buf, (unit >> 1) & 1u, abort_flag);
          if (!__all_sync(0xffffffffu, got)) {
            ok = false;
            break;
          }
          tc_fence_after_sync();
          const uint32_t t_row = tmem_base + buf * kBN + static_cast<uint32_t>(128 * half) + (static_cast<uint32_t>(quad * 32) << 16);
          if (k0 == T.kb0) {
            uint32_t(&r)[4][32] = reinterpret_cast<uint32_t(&)[4][32]>(acc);
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_32x32b_x32(t_row + static_cast<uint32_t>(c * 32), r[c]);
            tmem_ld_wait();
          } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) {   // 16 columns at a time: with 32 the registers do not last
              uint32_t r[16];
              tmem_ld_32x32b_x16(t_row + static_cast<uint32_t>(c * 16), r);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) acc[c >> 1][16 * (c & 1) + j] += __uint_as_float(r[j]);
            }
          }
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(tempty_leader0 + 8u * buf);   // the accumulator is free again
        }
        if (!ok) break;
        if (T.kb0 >= T.kb1) continue;
        if (P.mode == CE_LSE) ce_strip(G, P, acc, row0 + lane, n0, T.nb * 2 + half);
        else ce_store(G, P, acc, stg, row0 + T.split * P.num_m_blocks * 256, n0, lane);
      }
    }
    if (G.x) target_logits(INT_MAX);
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

// The rounding of dl to bf16 is the same for a whole row of grad_W, so that of one token
// shows in full: one token over 500 to 131072 columns left gradients 3.6e-3 off (rounding
// the outputs alone: 1.7e-3), while over many tokens the errors meet the outputs' rounding
// (2.0e-3 to 2.2e-3). So where there are few tokens dl is carried as the sum of two bf16
// numbers. Up to 32 tokens their 64 rows are one K block of grad_W and part of one tile of
// the other products: 32 x 1536 x 32003 takes 105 us, 33 tokens 95 (up to 128 tokens it cost
// 10 to 20%).
constexpr int kCeSplitTokens = 32;

// The tokens with a loss, in order: place[t] among them (-1 for the others), from[i] the
// i-th one, their number (1 if there is none: its row is zeros then) and the largest finite
// |g| of them (1 if there is none above 0): an infinity or a NaN stays with its own token
// and does not divide the others. Up to kCeSplitTokens of them get a second row each, from
// row `low` on (live counts both). One block, 1024 tokens and 1.4 us a step, in which nothing
// else runs: 14 us for 8192 tokens, 95 for 65536, 1.5 ms for 2^20.
__global__ void __launch_bounds__(1024) ce_live_kernel(const float* grad, const int64_t* targets, int64_t t, int64_t v,
                                                       int* place, int* from, int* live, int* low, float* grad_max) {
  __shared__ uint32_t s_max[32];
  __shared__ int s_count[33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  follow_stream();
  uint32_t m = 0;   // |g| as its bit pattern
  int before = 0;
  for (int64_t t0 = 0; t0 < t; t0 += 1024) {
    const int64_t i = t0 + threadIdx.x;
    bool in = false;
    if (i < t) {
      const int64_t y = targets[i];
      in = y >= 0 && y < v;
    }
    if (in) {
      const uint32_t g = __float_as_uint(grad[i]) & 0x7FFFFFFFu;
      if (g < 0x7F800000u) m = max(m, g);
    }
    const uint32_t votes = __ballot_sync(0xFFFFFFFFu, in);
    if (lane == 0) s_count[warp] = __popc(votes);
    __syncthreads();
    if (warp == 0) {   // exclusive sums over the warps
      int sum = s_count[lane];
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xFFFFFFFFu, sum, off);
        if (lane >= off) sum += o;
      }
      s_count[lane + 1] = sum;   // every lane has read its own count
      if (lane == 0) s_count[0] = 0;
    }
    __syncthreads();
    const int at = before + s_count[warp] + __popc(votes & ((1u << lane) - 1u));
    if (i < t) place[i] = in ? at : -1;
    if (in) from[at] = static_cast<int>(i);
    before += s_count[32];
    __syncthreads();
  }
  m = __reduce_max_sync(0xFFFFFFFFu, m);
  if (lane == 0) s_max[warp] = m;
  __syncthreads();
  if (warp == 0) {
    m = __reduce_max_sync(0xFFFFFFFFu, s_max[lane]);
    if (lane == 0) {
      *grad_max = m ? __uint_as_float(m) : 1.f;
      const bool split = before > 0 && before <= kCeSplitTokens;
      *live = before == 0 ? 1 : split ? 2 * before : before;
      *low = split ? before : INT_MAX;
      if (before == 0) from[0] = -1;
    }
  }
}

// Their rows of X and what dl needs of them, then zeros up to a multiple of 256 rows, by the
// first `row_blocks` blocks, a warp per row. The others, if any, meanwhile take all tokens'
// target_dl: nothing here depends on those, and they on nothing of ce_live_kernel (32 tokens:
// after the rows, or in that kernel, they took 4 us more).
__global__ void __launch_bounds__(256) ce_gather_kernel(const uint4* x, const uint4* w, const int64_t* targets, const float* lse,
                                                        const float* grad, int64_t t, int64_t v, int row_blocks, const int* from,
                                                        const int* live, const int* low_row, const float* grad_max, int row8,
                                                        uint4* x_live, int* row_target, float* row_lse, float* row_grad,
                                                        float* target_dl) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, block = blockIdx.x;
  follow_stream();
  if (block >= row_blocks) {
    int64_t i = static_cast<int64_t>(block - row_blocks) * 8 + warp;
    ce_targets(x, w, targets, lse, t, v, row8, i, static_cast<int64_t>(gridDim.x - row_blocks) * 8, INT_MAX, lane, target_dl);
    return;
  }
  const int n = *live, low = *low_row, end = (n + 255) / 256 * 256;
  for (int r = block * 8 + warp; r < end; r += row_blocks * 8) {
    const int at = r < n ? from[r < low ? r : r - low] : -1;
    uint4* dst = x_live + static_cast<int64_t>(r) * row8;
    const uint4* src = x + static_cast<int64_t>(at < 0 ? 0 : at) * row8;
    for (int i = lane; i < row8; i += 32) dst[i] = at < 0 ? make_uint4(0, 0, 0, 0) : ld_plain(src + i);
    if (lane == 0) {
      const float g = at < 0 ? 0.f : grad[at];
      row_target[r] = at < 0 ? -1 : static_cast<int>(targets[at]);
      row_lse[r] = at < 0 ? 0.f : lse[at];
      row_grad[r] = g == 0.f ? 0.f : __fdiv_rn(g, *grad_max);
    }
  }
}

// Joins the strips of each token, which leave the target's logit out: with the others' sum
// relative to it the loss, log(1 + sum exp(l_v - l_y)), is exact to the logits' error even
// where it is nearly 0 (as lse - l_y a loss of 0.26 at a logit of 12 was 2.4e-6 off). 32
// tokens x 32 slices of the strips per block, the slices' (max, sum) pairs joined in order.
constexpr int kCeJoinThreads = 1024;
__global__ void __launch_bounds__(kCeJoinThreads) ce_join_kernel(const float2* strips, int num_strips, int64_t t, int64_t v,
                                                                 const int64_t* targets, const float* target_logit,
                                                                 float* loss, float* lse) {
  __shared__ float2 s_part[32][32];
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * 32 + lane;
  follow_stream();
  float m = -INFINITY, s = 0.f;
  if (row < t) {
#pragma unroll 4
    for (int i = slice; i < num_strips; i += 32) {
      const float2 p = strips[static_cast<int64_t>(i) * t + row];
      const bool some = p.y != 0.f;   // else a strip past the vocabulary's end or of -infinity alone
      const float m2 = some ? fmaxf(m, p.x) : m;
      s = some ? s * ex2(m - m2) + p.y * ex2(p.x - m2) : s;
      m = m2;
    }
  }
  s_part[slice][lane] = make_float2(m, s);
  __syncthreads();
  if (slice == 0 && row < t) {
    float mm = -INFINITY;
#pragma unroll
    for (int i = 0; i < 32; ++i) mm = fmaxf(mm, s_part[i][lane].x);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (s_part[i][lane].y != 0.f) ss += s_part[i][lane].y * ex2(s_part[i][lane].x - mm);
    // mm (base 2, the others' largest logit) back in logits in two parts; the factor is 1 /
    // kLog2e as rounded
    constexpr float kHigh = static_cast<float>(1.0 / static_cast<double>(kLog2e));
    constexpr float kLow = static_cast<float>(1.0 / static_cast<double>(kLog2e) - static_cast<double>(kHigh));
    const int64_t y = targets[row];
    const bool counts = y >= 0 && y < v;
    float tl = counts ? target_logit[row] : -INFINITY;
    const float t2 = tl * kLog2e;   // infinite from a logit of 2.36e38 on, as in the strips
    if (isinf(t2)) tl = t2;
    if (tl == INFINITY || (tl == -INFINITY && mm == -INFINITY)) {
      // the target's logit beyond all numbers, or no logit above -infinity: log of the sum is
      // that infinity (a NaN among the others stays one), the loss infinity minus itself
      lse[row] = ss != ss ? ss : tl;
      loss[row] = counts ? NAN : 0.f;
      return;
    }
    const float d = fmaf(mm, kHigh, -tl) + mm * kLow;   // by how much it is above the target's
    if (d > 0.f) {
      const float sum = logf(ss + expf(-d));
      lse[row] = fmaf(mm, kHigh, fmaf(mm, kLow, sum));
      loss[row] = counts ? d + sum : 0.f;
    } else {
      const float l = log1pf(ss * expf(d));
      lse[row] = tl + l;
      loss[row] = counts ? l : 0.f;
    }
  }
}

// grad_X: the token's row of the `splits` partial sums (`stride` float4 apart), and its second
// row from `low_row` on, added in order, times the largest |g|, in bf16; zeros for a token
// without a loss. 8 elements per thread and step. With few tokens the runs are many and the
// threads few: one load after the other took 8 us more (33 x 1536 x 32003).
__global__ void __launch_bounds__(256) ce_scatter_kernel(const float4* src, const int* place, const int* low_row, int64_t n8,
                                                         int row8, int splits, int64_t stride, const float* scale, uint4* dst) {
  follow_stream();
  const float f = *scale;
  const int low = *low_row;
  const bool two = low != INT_MAX;   // whether a token has two rows
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const int64_t half = two ? 2 * static_cast<int64_t>(low) * row8 : 0;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; i < n8; i += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t t = i / row8;
    const int p = ld_plain(place + t);
    if (p < 0) {
      dst[i] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const float4* at = src + 2 * (static_cast<int64_t>(p) * row8 + (i - t * row8));
    float4 a = zero, b = zero;
    auto add = [&](const float4& c, const float4& e) {
      a = make_float4(a.x + c.x, a.y + c.y, a.z + c.z, a.w + c.w);
      b = make_float4(b.x + e.x, b.y + e.y, b.z + e.z, b.w + e.w);
    };
    for (int s0 = 0; s0 < splits; s0 += 4) {   // four addends at a time, so that their loads overlap
      float4 c[4][2], d[4][2];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float4* from = at + (s0 + u < splits ? s0 + u : s0) * stride;
        c[u][0] = ld_plain(from);
        c[u][1] = ld_plain(from + 1);
        d[u][0] = two ? ld_plain(from + half) : zero;
        d[u][1] = two ? ld_plain(from + half + 1) : zero;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (s0 + u < splits) {
          add(c[u][0], c[u][1]);
          add(d[u][0], d[u][1]);
        }
    }
    dst[i] = make_uint4(pack_bf16x2(a.x * f, a.y * f), pack_bf16x2(a.z * f, a.w * f), pack_bf16x2(b.x * f, b.y * f),
                        pack_bf16x2(b.z * f, b.w * f));
  }
}

}  // namespace bl
