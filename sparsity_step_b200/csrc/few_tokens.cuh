// Products of few tokens (blocks of up to 128, the logits up to 32) with a large weight matrix,
// on the tensor cores with the weights as the M operand:
//
//   kFp8:  y[t, n]  = sum_k xq[t, k] 2^ex * wq[n, k] 2^ew   (kind::mxf8f6f4, block-scaled)
//   else:  l[t, v]  = sum_k X[t, k] W[v, k]                  (kind::f16), reduced to strips of
//          (maximum, sum of exponentials) without the target for the cross entropy
//
// Bound by HBM: every weight is read once and used for a few multiplications. A CTA takes
// 128 weight rows; its producer streams them through a ring of 16 KB K blocks (128 rows x
// 128 bytes) as far ahead as shared memory allows, and nothing between HBM and the tensor
// core touches them: converting 8-bit codes in registers for warp MMAs (three times the
// instructions) bounded an earlier version at 10.6 us for 22.5 MB against 3.5 of HBM time.
// The tokens' operand has 16 to 128 rows, 128-byte swizzled, and a K block of it comes with
// every K block of weights (from L2), except for bf16 activations of up to 16 tokens (kFp8):
// these are quantised here, once per CTA while the first weights are on their way, and kept
// in shared memory, so that a single token needs one launch.
// Two CTAs fit on an SM, so that the next call's are set up while this one's run.
// Where there are fewer row blocks than SMs, a cluster of up to 8 CTAs splits K and adds its
// partial sums through distributed shared memory in the order of the ranks; else a CTA
// walks over several row blocks with its ring running on.
//
// Scales (kFp8). One 512-byte bulk copy per K block brings the 128 rows' scale words in row
// order, which tcgen05.cp puts at (lane r / 4, column r % 4), while the MMA looks for row i's
// at (lane i % 32, column i / 32). So the rows are permuted instead: four copies of 32 rows
// each, four apart, and MMA row 32 c + l is weight row 4 l + c.
// Every wait is bounded. No load uses multicast.
#pragma once

#include "fp8_quant.cuh"
#include "gemm_fp8.cuh"
#include "gemm_sp2.cuh"
#include "linear_ce.cuh"

namespace bl {

constexpr int kFewThreads = 192;      // producer, MMA, four epilogue warps
constexpr int kFewMaxStages = 8;
constexpr int kFewStageBytes = 128 * 128;
constexpr int kFewSfBytes = 512;
// K blocks (64 of K) per accumulation of logits, at most: as few as fit in TMEM beside each
// other are taken. One token's loss has nobody to average with: with 8, as in linear_ce.cuh,
// it was 1.3e-6 off, with 4 half of that, with 2 a quarter (medians of 40 draws). Where 4 do
// not fit, more CTAs share K.
constexpr int kFewPartBlocks = 4;
__host__ __device__ constexpr int few_parts(bool fp8, int blocks, int part_blocks) {
  return fp8 ? 1 : (blocks + part_blocks - 1) / part_blocks;
}
constexpr int kFewBarBytes = 256;

struct FewMaps {
  CUtensorMap w[4];   // kFp8: rows c, c + 4, c + 8, ...; else w[0]: all rows
  CUtensorMap x;      // bf16 or codes (not x_bf16)
};
struct FewArgs {
  const void* x;              // [t, k] bf16 (x_bf16, cross entropy)
  const uint32_t* xs;         // scale words of codes, [ceil(k / 512), t]
  int x_bf16;                 // kFp8: quantise x here (e4m3)
  const uint32_t* ws;         // kFp8: [ceil(k / 512), n]
  int a_e5m2, b_e5m2;
  int t, k, n;                // t: all tokens; blockIdx.y is the block of kTok (kFp8 codes only, else one)
  int num_k_blocks, num_row_blocks;
  int split;                  // CTAs of the cluster that share a row block
  int stages;
  int part_blocks;            // K blocks per accumulation of logits
  int parts, bufs;            // accumulations per row block and row blocks in TMEM at a time
  uint32_t sf_col0, tmem_cols;
  void* y;                    // kFp8
  int y_f32;
  const void* rows;           // cross entropy: [n, k] bf16
  const int64_t* targets;
  float2* strips;             // [num_row_blocks * (split > 1 ? split : 4), t]
  float* target_logit;
};

// The partial sums of a split K (kTok x 128 fp32) go over the rings once their MMAs are done.
constexpr size_t few_ring_bytes(bool fp8, int tok, int stages) {
  return static_cast<size_t>(stages) * (kFewStageBytes + (fp8 ? kFewSfBytes : 0) + tok * 128);
}
static_assert(few_ring_bytes(true, 128, 3) >= 128 * 128 * 4 && 3 * kFewStageBytes >= 64 * 128 * 4, "exchange over the rings");
// Shared memory: ring of weights | ring of their scales (kFp8) | tokens' operand, a ring too
// or (quantised here) all K blocks of the CTA | its scales (kFp8) | barriers.
__host__ __device__ constexpr int few_blocks_max(int num_k_blocks, int split) { return (num_k_blocks + split - 1) / split; }
__host__ __device__ constexpr size_t few_smem_bytes(bool fp8, bool kept, int tok, int stages, int blocks) {
  return 2048 + static_cast<size_t>(stages) * (kFewStageBytes + (fp8 ? kFewSfBytes : 0)) +
         static_cast<size_t>(kept ? blocks : stages) * tok * 128 + (fp8 ? static_cast<size_t>(blocks / 4 + 2) * kFewSfBytes : 0) +
         kFewBarBytes;
}

__device__ __forceinline__ void tc_mma_mxf8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc, uint32_t sfa,
                                            uint32_t sfb, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %6, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tc_cp_32x128b(uint32_t taddr, uint64_t sdesc) {
  asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(sdesc) : "memory");
}
__device__ __forceinline__ float ld_shared_cluster_f32(uint32_t cluster_addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
  return v;
}
__device__ __forceinline__ float4 ld_shared_cluster_v4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}
template <int kCols>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[kCols]) {
  if constexpr (kCols == 16) tmem_ld_32x32b_x16(taddr, r);
  else tmem_ld_32x32b_x32(taddr, r);
}
__device__ __forceinline__ int lane_id() { return static_cast<int>(threadIdx.x & 31); }
__device__ __forceinline__ void st_shared_u8(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u8 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

// Scales of the tokens' operand of K blocks [kb0, kb1) and, from bf16, its codes, by all
// threads of the CTA.
template <int kTok>
__device__ __forceinline__ void few_fp8_operand(const FewArgs& a, uint32_t sB, uint32_t sSfb, int kb0, int kb1, int tok0) {
  const int blocks = kb1 - kb0, groups = (kb1 - 1) / 4 - kb0 / 4 + 1;
  // scale word of token i of K group g at 512 g + 16 (i % 32) + 4 (i / 32), zero past the last
  for (int i = threadIdx.x; i < groups * 32; i += kFewThreads) {
    uint32_t w[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const int tok = tok0 + 32 * c + (i & 31);
      w[c] = !a.x_bf16 && tok < a.t ? ld_plain(a.xs + static_cast<int64_t>(kb0 / 4 + (i >> 5)) * a.t + tok) : 0u;
    }
    st_shared_v4(sSfb + 16u * static_cast<uint32_t>(i), w[0], w[1], w[2], w[3]);
  }
  if (!a.x_bf16) return;
  auto at = [&](int b, int tok, int j) { return sB + static_cast<uint32_t>((b * kTok + tok) * 128 + ((j ^ (tok & 7)) * 16)); };
  for (int i = threadIdx.x; i < blocks * (kTok - a.t) * 8; i += kFewThreads) {   // rows without a token
    const int r = i >> 3;
    st_shared_v4(at(r / (kTok - a.t), a.t + r % (kTok - a.t), i & 7), 0, 0, 0, 0);
  }
  __syncthreads();   // the scale words are zeros before their bytes are filled in
  // item: 16 codes (chunk j) of token tok in block b, 8 lanes to a block of 128; four items
  // a thread at a time, so that their loads overlap
  const uint4 zero = make_uint4(0, 0, 0, 0);
  const int items = blocks * a.t * 8;
  for (int i0 = static_cast<int>(threadIdx.x); i0 - lane_id() < items; i0 += 4 * kFewThreads) {
    uint4 lo[4], hi[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * kFewThreads, j = i & 7, tok = (i >> 3) % a.t, kb = kb0 + (i >> 3) / a.t;
      const bool in = i < items && kb * 128 + j * 16 < a.k;
      const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.x) + static_cast<int64_t>(tok) * a.k + kb * 128 + j * 16);
      lo[u] = in ? ld_plain(p) : zero;
      hi[u] = in ? ld_plain(p + 1) : zero;
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * kFewThreads, j = i & 7, tok = (i >> 3) % a.t, b = (i >> 3) / a.t, kb = kb0 + b;
      uint32_t m = __vmaxu2(__vmaxu2(__vmaxu2(lo[u].x & 0x7FFF7FFFu, lo[u].y & 0x7FFF7FFFu), __vmaxu2(lo[u].z & 0x7FFF7FFFu, lo[u].w & 0x7FFF7FFFu)),
                            __vmaxu2(__vmaxu2(hi[u].x & 0x7FFF7FFFu, hi[u].y & 0x7FFF7FFFu), __vmaxu2(hi[u].z & 0x7FFF7FFFu, hi[u].w & 0x7FFF7FFFu)));
      m = max(m & 0xFFFFu, m >> 16);
#pragma unroll
      for (int off = 1; off < 8; off <<= 1) m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, off));
      const uint32_t byte = fp8_scale_byte(m << 16, fp8_top_exponent(FP8_E4M3));
      const float inv = fp8_inv_scale(byte);
      auto codes = [&](uint32_t p0, uint32_t p1) {
        return fp8_pack4<false>(__uint_as_float(p0 << 16) * inv, __uint_as_float(p0 & 0xFFFF0000u) * inv,
                                __uint_as_float(p1 << 16) * inv, __uint_as_float(p1 & 0xFFFF0000u) * inv);
      };
      if (i < items) {
        st_shared_v4(at(b, tok, j), codes(lo[u].x, lo[u].y), codes(lo[u].z, lo[u].w), codes(hi[u].x, hi[u].y), codes(hi[u].z, hi[u].w));
        if (j == 0) st_shared_u8(sSfb + static_cast<uint32_t>((kb / 4 - kb0 / 4) * kFewSfBytes + tok * 16 + (kb & 3)), byte);
      }
    }
  }
}

template <bool kFp8, int kTok>
__global__ void __launch_bounds__(kFewThreads) few_tokens_kernel(const __grid_constant__ FewMaps M, const FewArgs a) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  const int max_blocks = few_blocks_max(a.num_k_blocks, a.split);
  const bool kept = kFp8 && a.x_bf16;
  const uint32_t sRing = base, sSfa = sRing + static_cast<uint32_t>(a.stages * kFewStageBytes);
  const uint32_t sB = (sSfa + (kFp8 ? static_cast<uint32_t>(a.stages * kFewSfBytes) : 0u) + 1023u) & ~1023u;
  const uint32_t sSfb = sB + static_cast<uint32_t>((kept ? max_blocks : a.stages) * kTok * 128);
  const uint32_t bar0 = sSfb + (kFp8 ? static_cast<uint32_t>((max_blocks / 4 + 2) * kFewSfBytes) : 0u);
  const uint32_t full0 = bar0, empty0 = bar0 + 8u * kFewMaxStages, tfull0 = empty0 + 8u * kFewMaxStages, tempty0 = tfull0 + 16u;
  const uint32_t done_bar = tempty0 + 16u, slot = done_bar + 8u;
  volatile uint32_t* tmem_slot = reinterpret_cast<volatile uint32_t*>(smem_raw + (slot - raw));
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem_raw + (slot - raw) + 4);

  const int rank = a.split > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // warp-uniform
  const int kb0 = static_cast<int>(static_cast<int64_t>(rank) * a.num_k_blocks / a.split);
  const int kb1 = static_cast<int>(static_cast<int64_t>(rank + 1) * a.num_k_blocks / a.split);
  const int blk0 = blockIdx.x / a.split, blk_step = gridDim.x / a.split;
  const int tok0 = blockIdx.y * kTok, toks = min(kTok, a.t - tok0);   // this CTA's tokens
  if (threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) {
      mbar_init(full0 + 8u * s, 1);
      mbar_init(empty0 + 8u * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(tfull0 + 8u * b, 1);
      mbar_init(tempty0 + 8u * b, 4);   // epilogue warps
    }
    mbar_init(done_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    if (!kept) tma_prefetch_desc(&M.x);
    for (int c = 0; c < (kFp8 ? 4 : 1); ++c) tma_prefetch_desc(&M.w[c]);
  }
  if (warp == 1) {
    tmem_alloc(slot, a.tmem_cols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem_base = __reduce_or_sync(0xffffffffu, *tmem_slot);
  follow_stream();

  uint32_t live = 1;   // producer and MMA warps: 0 after a wait gave up
  int s = 0;
  uint32_t ph = 0, issued = 0;
  const uint32_t own_abort = map_to_rank(slot + 4u, static_cast<uint32_t>(rank));
  auto issue = [&](int blk, int kb) {   // K block kb of row block blk into stage s
    const int row0 = blk * 128;
    const uint32_t sf_bytes = kFp8 ? 4u * static_cast<uint32_t>(min(128, a.n - row0)) : 0u;
    live = wait_live<false>(live, empty0 + 8u * s, ph ^ 1u, abort_flag, own_abort);
    if (elect_one() && live) {
      const uint32_t fb = full0 + 8u * s, dst = sRing + static_cast<uint32_t>(s * kFewStageBytes);
      mbar_arrive_expect_tx(fb, kFewStageBytes + sf_bytes + (kept ? 0u : static_cast<uint32_t>(kTok * 128)));
      if constexpr (kFp8) {
#pragma unroll
        for (int c = 0; c < 4; ++c) tma_load_2d(dst + 4096u * c, &M.w[c], fb, kb * 128, row0 / 4);
        bulk_load_1d(sSfa + static_cast<uint32_t>(s * kFewSfBytes), a.ws + static_cast<int64_t>(kb >> 2) * a.n + row0, sf_bytes, fb);
      } else {
        tma_load_2d(dst, &M.w[0], fb, kb * 64, row0);
      }
      if (!kept) tma_load_2d(sB + static_cast<uint32_t>(s * kTok * 128), &M.x, fb, kb * (kFp8 ? 128 : 64), tok0);
    }
    issued += live;
    if (++s == a.stages) {
      s = 0;
      ph ^= 1u;
    }
  };
  // the first ring of weights is on its way while all warps make the tokens' operand
  const int ahead = kFp8 ? min(a.stages, kb1 - kb0) : 0;
  if constexpr (kFp8) {
    if (warp == 0)
      for (int i = 0; i < ahead; ++i) issue(blk0, kb0 + i);
    few_fp8_operand<kTok>(a, sB, sSfb, kb0, kb1, tok0);
    fence_proxy_async_smem();
    __syncthreads();
  }

  if (warp == 0) {
    // ------------------------------------------------------------- TMA producer
    for (int blk = blk0; blk < a.num_row_blocks; blk += blk_step)
      for (int kb = blk == blk0 ? kb0 + ahead : kb0; kb < kb1; ++kb) issue(blk, kb);
    if (!live && elect_one()) {
      atomicOr(&g_device_status, DEV_ST_TIMEOUT_PRODUCER);
      const uint32_t st = static_cast<uint32_t>(a.stages), first = issued > st ? issued - st : 0;
      for (uint32_t i = first; i < issued; ++i)
        if (!mbar_wait_plain(full0 + 8u * (i % st), (i / st) & 1u)) atomicOr(&g_device_status, DEV_ST_TIMEOUT_DRAIN);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------- MMA issuer
    const uint32_t idesc0 = kFp8 ? make_idesc_mxf8(a.a_e5m2, a.b_e5m2, kTok, 128, 0) : make_idesc(1u, 1u, 1u, 0u, 0u, kTok, 128);
    uint32_t unit = 0, count = 0;
    for (int blk = blk0; blk < a.num_row_blocks; blk += blk_step, ++unit) {
      const uint32_t buf = a.bufs == 2 ? unit & 1u : 0u, uph = a.bufs == 2 ? unit >> 1 : unit;
      live = wait_live<false>(live, tempty0 + 8u * buf, (uph & 1u) ^ 1u, abort_flag, own_abort);
      tc_fence_after_sync();
      for (int kb = kb0; kb < kb1; ++kb, ++count) {
        live = wait_live<false>(live, full0 + 8u * s, ph, abort_flag, own_abort);
        tc_fence_after_sync();
        if (elect_one() && live) {
          const int b = kb - kb0;
          const int part = kFp8 ? 0 : b / a.part_blocks;
          const uint32_t add = (kFp8 ? b == 0 : b % a.part_blocks == 0) ? 0u : 1u;   // first MMA of an accumulation
          const uint32_t d = tmem_base + (buf * a.parts + part) * kTok;
          const uint64_t ad = make_sw128_desc(sRing + static_cast<uint32_t>(s * kFewStageBytes), 16, 1024);
          const uint64_t bd = make_sw128_desc(sB + static_cast<uint32_t>((kept ? b : s) * kTok * 128), 16, 1024);
          if constexpr (kFp8) {
            // eight slots of scale columns: a slot's last user was at least a ring of stages ago
            const uint32_t col = tmem_base + a.sf_col0 + 8u * (count % kFewMaxStages);
            tc_cp_32x128b(col, make_sf_desc(sSfa + static_cast<uint32_t>(s * kFewSfBytes)));
            tc_cp_32x128b(col + 4u, make_sf_desc(sSfb + static_cast<uint32_t>((kb / 4 - kb0 / 4) * kFewSfBytes)));
            const uint32_t id = static_cast<uint32_t>(kb & 3), idesc = idesc0 | id << 4 | id << 29;
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              tc_mma_mxf8(d, ad + 2u * kk, bd + 2u * kk, idesc, col, col + 4u, kk != 0 ? 1u : add);
          } else {
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) tc_mma_f16(d, ad + 2u * kk, bd + 2u * kk, idesc0, kk != 0 ? 1u : add);
          }
          tc_commit(empty0 + 8u * s);
          if (kb + 1 == kb1) tc_commit(tfull0 + 8u * buf);
        }
        if (++s == a.stages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    if (elect_one()) {
      if (!live) atomicOr(&g_device_status, DEV_ST_TIMEOUT_MMA);
      tc_commit(done_bar);   // every MMA issued above has retired once this arrives
      if (!mbar_wait_plain(done_bar, 0)) atomicOr(&g_device_status, DEV_ST_TIMEOUT_DRAIN);
    }
  } else {
    // ------------------------------------------------------------- epilogue (4 warps)
    const int quad = warp & 3;
    if constexpr (!kFp8) {   // the targets' logits, while the weights stream by
      int64_t i = static_cast<int64_t>(blockIdx.x) * 4 + quad;
      ce_targets(static_cast<const uint4*>(a.x), static_cast<const uint4*>(a.rows), a.targets, nullptr, a.t, a.n, a.k / 8, i,
                 static_cast<int64_t>(gridDim.x) * 4, INT_MAX, lane, a.target_logit);
    }
    bool ok = true;
    uint32_t unit = 0;
    for (int blk = blk0; blk < a.num_row_blocks && ok; blk += blk_step, ++unit) {
      const uint32_t buf = a.bufs == 2 ? unit & 1u : 0u, uph = a.bufs == 2 ? unit >> 1 : unit;
      const bool got = mbar_wait(tfull0 + 8u * buf, uph & 1u, abort_flag);
      if (!__all_sync(0xffffffffu, got)) {
        ok = false;
        break;
      }
      tc_fence_after_sync();
      const uint32_t t_row = tmem_base + buf * a.parts * kTok + (static_cast<uint32_t>(quad * 32) << 16);
      const int local = kFp8 ? 4 * lane + quad : quad * 32 + lane;   // the weight row of this thread
      const int row = blk * 128 + local;
      const int parts = few_parts(kFp8, kb1 - kb0, a.part_blocks);
      constexpr int kCols = kTok < 32 ? kTok : 32;
#pragma unroll 1
      for (int c0 = 0; c0 < kTok; c0 += kCols) {   // tokens, 16 or 32 at a time
        uint32_t r[kCols];
        float v[kCols];
        tmem_ld_cols<kCols>(t_row + static_cast<uint32_t>(c0), r);
        tmem_ld_wait();
#pragma unroll
        for (int i = 0; i < kCols; ++i) v[i] = __uint_as_float(r[i]);
        for (int p = 1; p < parts; ++p) {
          tmem_ld_cols<kCols>(t_row + static_cast<uint32_t>(p * kTok + c0), r);
          tmem_ld_wait();
#pragma unroll
          for (int i = 0; i < kCols; ++i) v[i] += __uint_as_float(r[i]);
        }
        if (c0 + kCols == kTok) {   // the accumulators are free again
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(tempty0 + 8u * buf);
        }
        if (a.split > 1) {   // the cluster's only row block: partial sums for the exchange below, in the rings
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            asm volatile("st.shared.f32 [%0], %1;" ::"r"(sRing + static_cast<uint32_t>(((c0 + i) * 128 + local) * 4)), "f"(v[i]) : "memory");
        } else if constexpr (kFp8) {
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            if (c0 + i < toks && row < a.n) {
              const int64_t off = static_cast<int64_t>(tok0 + c0 + i) * a.n + row;
              if (a.y_f32) static_cast<float*>(a.y)[off] = v[i];
              else static_cast<__nv_bfloat16*>(a.y)[off] = __float2bfloat16_rn(v[i]);
            }
        } else {   // one strip of 32 rows per warp
#pragma unroll
          for (int i = 0; i < kCols; ++i)
            if (i < a.t) {
              if (row < a.n && a.targets[i] == row) v[i] = -INFINITY;
              const float l2 = row < a.n ? v[i] * kLog2e : -INFINITY;
              float m = l2;
#pragma unroll
              for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
              m = strip_max(m);
              float e = row < a.n ? ex2(fmaf(v[i], kLog2e, -m)) : 0.f;
#pragma unroll
              for (int off = 16; off > 0; off >>= 1) e += __shfl_xor_sync(0xffffffffu, e, off);
              if (lane == 0) a.strips[static_cast<int64_t>(blk * 4 + quad) * a.t + i] = make_float2(m, e);
            }
        }
      }
    }
    if (!ok && lane == 0) {
      pair_abort(abort_flag, own_abort);
      atomicOr(&g_device_status, DEV_ST_TIMEOUT_EPILOGUE);
    }
  }

  __syncthreads();
  if (a.split > 1) {
    cluster_sync();   // every CTA's partial sums are in its shared memory
    const int per = 128 / a.split, blk = blk0;   // rows of the block that this CTA finishes
    auto at = [&](int i, int local, int c) {   // rank c's partial sum
      return map_to_rank(sRing + static_cast<uint32_t>((i * 128 + local) * 4), static_cast<uint32_t>(c));
    };
    auto total = [&](int i, int local) {   // ranks in order
      float v = 0.f;
      for (int c = 0; c < a.split; ++c) v += ld_shared_cluster_f32(at(i, local, c));
      return v;
    };
    if constexpr (kFp8) {
      const int quads = per / 4;   // four rows at a time (n % 16 == 0)
      for (int e = threadIdx.x; e < toks * quads; e += kFewThreads) {
        const int i = e / quads, local = rank * per + 4 * (e % quads), row = blk * 128 + local;
        if (row < a.n) {
          float4 p[8];
#pragma unroll
          for (int c = 0; c < 8; ++c)
            if (c < a.split) p[c] = ld_shared_cluster_v4(at(i, local, c));
          float4 v = p[0];
#pragma unroll
          for (int c = 1; c < 8; ++c)
            if (c < a.split) v = make_float4(v.x + p[c].x, v.y + p[c].y, v.z + p[c].z, v.w + p[c].w);
          const int64_t off = static_cast<int64_t>(tok0 + i) * a.n + row;
          if (a.y_f32) *reinterpret_cast<float4*>(static_cast<float*>(a.y) + off) = v;
          else *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.y) + off) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        }
      }
    } else {
      for (int i = warp; i < a.t; i += kFewThreads / 32) {   // a warp per token, one strip per CTA
        float l[2], m = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h) {   // per is 16, 32 or 64
          const int local = rank * per + 32 * h + lane, row = blk * 128 + local;
          l[h] = -INFINITY;
          if (32 * h + lane < per && row < a.n) {
            l[h] = total(i, local);
            if (a.targets[i] == row) l[h] = -INFINITY;
          }
          m = fmaxf(m, l[h] * kLog2e);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        m = strip_max(m);
        float e = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (32 * h + lane < per && blk * 128 + rank * per + 32 * h + lane < a.n) e += ex2(fmaf(l[h], kLog2e, -m));
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) e += __shfl_xor_sync(0xffffffffu, e, off);
        if (lane == 0) a.strips[static_cast<int64_t>(blk * a.split + rank) * a.t + i] = make_float2(m, e);
      }
    }
    cluster_sync();   // no CTA leaves while another still reads its partial sums
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after_sync();
    tmem_dealloc(tmem_base, a.tmem_cols);
  }
}

}  // namespace bl
