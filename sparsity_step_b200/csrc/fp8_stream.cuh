// Block-scaled 8-bit float product for few tokens: the weights' codes stream from HBM
// once, straight into warp-MMA fragments.
//
//   y[t, n] = sum_b 2^(ex(t, b) + ew(n, b)) * sum_{k in block b} xq[t, k] * wq[n, k]
//
// A CTA computes 16 weight rows x up to 8 NT tokens; its warps take the 128-wide K blocks
// in turn, so every SM has many independent 2 KB pieces of W in flight, and add their
// partial sums in shared memory in a fixed order. Within a block a lane loads 16
// contiguous bytes of a row (mma.m16n8k32 wants four scattered words; the order of k
// inside a block is free, and W and X use the same one). The four MMAs of a block
// accumulate in fp32 from zero and are then scaled and added, so no scale is rounded.
// With bf16 activations (kXBf16) each warp makes the block's codes itself: 32 values a
// lane, one maximum over four lanes. That repeats the work for every 16 weight rows but
// saves the quantiser's launch, which at one token costs about as much as the product.
// Bound by HBM (1 byte per weight).
#pragma once

#include "fp8_quant.cuh"

namespace bl {

constexpr int kFsMaxWarps = 16;

struct Fp8StreamArgs {
  const void* x;            // bf16 or codes [t, k]
  const uint32_t* xs;       // [ceil(k / 512), t] scale words (codes only)
  const uint8_t* wq;        // [n, k]
  const uint32_t* ws;       // [ceil(k / 512), n] scale words
  void* y;                  // [t, n]
  int t, k, n;
  int y_f32;
};

template <bool kA5, bool kB5>
__device__ __forceinline__ void mma_fp8_16x8x32(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                                uint32_t b0, uint32_t b1) {
#define BL_FP8_MMA(TA, TB)                                                                                           \
  asm volatile("mma.sync.aligned.m16n8k32.row.col.f32." TA "." TB ".f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "        \
               "{%8, %9}, {%0, %1, %2, %3};"                                                                         \
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])                                                       \
               : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1))
  if (kA5 && kB5) BL_FP8_MMA("e5m2", "e5m2");
  else if (kA5) BL_FP8_MMA("e5m2", "e4m3");
  else if (kB5) BL_FP8_MMA("e4m3", "e5m2");
  else BL_FP8_MMA("e4m3", "e4m3");
#undef BL_FP8_MMA
}

// Weight codes of one K block for this lane: rows g and g + 8, 16 bytes of each half.
struct FsBlock {
  uint4 lo[2], hi[2];   // [half]: row g, row g + 8
};
__device__ __forceinline__ uint4 ldg_stream(const uint8_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}
__device__ __forceinline__ uint32_t absmax_bf16x8(uint4 v, uint32_t m) {
  m = __vmaxu2(__vmaxu2(m, v.x & 0x7FFF7FFFu), v.y & 0x7FFF7FFFu);
  return __vmaxu2(__vmaxu2(m, v.z & 0x7FFF7FFFu), v.w & 0x7FFF7FFFu);
}
__device__ __forceinline__ uint32_t codes_bf16x4(uint32_t a, uint32_t b, float inv) {
  return fp8_pack4<false>(__uint_as_float(a << 16) * inv, __uint_as_float(a & 0xFFFF0000u) * inv,
                          __uint_as_float(b << 16) * inv, __uint_as_float(b & 0xFFFF0000u) * inv);
}

template <int NT, bool kXBf16, bool kW5, bool kX5>
__global__ void __launch_bounds__(32 * kFsMaxWarps) fp8_stream_kernel(const Fp8StreamArgs a) {
  __shared__ float s_part[kFsMaxWarps][NT][128];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int g = lane >> 2, q = lane & 3;
  const int row0 = blockIdx.x * 16;
  const int nkb = (a.k + 127) >> 7;
  const uint8_t* w0 = a.wq + static_cast<int64_t>(row0 + g) * a.k + q * 16;
  const uint8_t* w1 = w0 + static_cast<int64_t>(8) * a.k;
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  const uint4 zero = make_uint4(0, 0, 0, 0);

  auto load = [&](FsBlock& b, int kb) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k0 = kb * 128 + h * 64;   // k % 64 == 0: a half is all in or all out
      b.lo[h] = k0 < a.k ? ldg_stream(w0 + k0) : zero;
      b.hi[h] = k0 < a.k ? ldg_stream(w1 + k0) : zero;
    }
  };
  auto block = [&](const FsBlock& b, int kb) {
    const int sh = 8 * (kb & 3);
    const uint32_t* wsrow = a.ws + static_cast<int64_t>(kb >> 2) * a.n + row0 + g;
    const float sw0 = fp8_scale((__ldg(wsrow) >> sh) & 255u), sw1 = fp8_scale((__ldg(wsrow + 8) >> sh) & 255u);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const int tok = i * 8 + g;
      uint4 xc[2];
      uint32_t byte = 0;
      if constexpr (kXBf16) {
        const uint16_t* xr = static_cast<const uint16_t*>(a.x) + static_cast<int64_t>(tok) * a.k + kb * 128 + q * 16;
        uint4 v[4];
        uint32_t m = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const bool in = tok < a.t && kb * 128 + h * 64 < a.k;
          v[2 * h] = in ? __ldg(reinterpret_cast<const uint4*>(xr + 64 * h)) : zero;
          v[2 * h + 1] = in ? __ldg(reinterpret_cast<const uint4*>(xr + 64 * h + 8)) : zero;
          m = absmax_bf16x8(v[2 * h + 1], absmax_bf16x8(v[2 * h], m));
        }
        m = max(m & 0xFFFFu, m >> 16);
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
        m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
        byte = fp8_scale_byte(m << 16, fp8_top_exponent(FP8_E4M3));
        const float inv = fp8_inv_scale(byte);
#pragma unroll
        for (int h = 0; h < 2; ++h)
          xc[h] = make_uint4(codes_bf16x4(v[2 * h].x, v[2 * h].y, inv), codes_bf16x4(v[2 * h].z, v[2 * h].w, inv),
                             codes_bf16x4(v[2 * h + 1].x, v[2 * h + 1].y, inv),
                             codes_bf16x4(v[2 * h + 1].z, v[2 * h + 1].w, inv));
      } else {
        const uint8_t* xr = static_cast<const uint8_t*>(a.x) + static_cast<int64_t>(tok) * a.k + kb * 128 + q * 16;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          xc[h] = tok < a.t && kb * 128 + h * 64 < a.k ? __ldg(reinterpret_cast<const uint4*>(xr + 64 * h)) : zero;
        if (tok < a.t) byte = (__ldg(a.xs + static_cast<int64_t>(kb >> 2) * a.t + tok) >> sh) & 255u;
      }
      float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mma_fp8_16x8x32<kW5, kX5>(d, b.lo[h].x, b.hi[h].x, b.lo[h].y, b.hi[h].y, xc[h].x, xc[h].y);
        mma_fp8_16x8x32<kW5, kX5>(d, b.lo[h].z, b.hi[h].z, b.lo[h].w, b.hi[h].w, xc[h].z, xc[h].w);
      }
      // the accumulator's columns are tokens 2q and 2q + 1, whose scales lanes 8q and 8q + 4 hold
      const float s0 = fp8_scale(__shfl_sync(0xFFFFFFFFu, byte, 8 * q));
      const float s1 = fp8_scale(__shfl_sync(0xFFFFFFFFu, byte, 8 * q + 4));
      acc[i][0] = fmaf(d[0], sw0 * s0, acc[i][0]);
      acc[i][1] = fmaf(d[1], sw0 * s1, acc[i][1]);
      acc[i][2] = fmaf(d[2], sw1 * s0, acc[i][2]);
      acc[i][3] = fmaf(d[3], sw1 * s1, acc[i][3]);
    }
  };
  // two blocks' loads in flight per warp
  for (int kb = warp; kb < nkb; kb += 2 * warps) {
    FsBlock b0, b1;
    load(b0, kb);
    const bool two = kb + warps < nkb;   // warp-uniform
    if (two) load(b1, kb + warps);
    block(b0, kb);
    if (two) block(b1, kb + warps);
  }
#pragma unroll
  for (int i = 0; i < NT; ++i) {   // [token][row] within the 16 x 8 tile
    float* p = s_part[warp][i];
    p[(2 * q) * 16 + g] = acc[i][0];
    p[(2 * q + 1) * 16 + g] = acc[i][1];
    p[(2 * q) * 16 + g + 8] = acc[i][2];
    p[(2 * q + 1) * 16 + g + 8] = acc[i][3];
  }
  __syncthreads();
  for (int o = threadIdx.x; o < NT * 128; o += blockDim.x) {
    const int i = o >> 7, e = o & 127;
    float s = 0.f;
    for (int w = 0; w < warps; ++w) s += s_part[w][i][e];
    const int tok = i * 8 + (e >> 4);
    if (tok < a.t) {
      const int64_t off = static_cast<int64_t>(tok) * a.n + row0 + (e & 15);
      if (a.y_f32) static_cast<float*>(a.y)[off] = s;
      else static_cast<__nv_bfloat16*>(a.y)[off] = __float2bfloat16_rn(s);
    }
  }
}

}  // namespace bl
