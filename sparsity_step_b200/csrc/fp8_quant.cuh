// Block-scaled 8-bit float codes of activations, gradients and weights.
//
// A block of 128 values along the reduction (1 x 128 of activations and gradients,
// 128 x 128 of weights) shares one power-of-two scale 2^e, the smallest that brings the
// block within the format's range (top = 1.75 * 2^P: P = 8 for e4m3, 15 for e5m2):
//   amax = m * 2^E, 1 <= m < 2:  e = E - P + [m > 1.75], not below -127
//   code = round-to-nearest-even(x * 2^-e),  stored scale byte = e + 127 (UE8M0)
// A power of two scales without rounding, so a code is one rounding of its value, every
// output is determined bit for bit, and the tensor cores' block-scaled MMA applies the
// scale by itself. An all-zero block gets byte 0; one with an infinity or a NaN gets byte
// 255 (the scale NaN) and codes 0x7F, so that what it touches comes out as NaN.
//
// One CTA takes one 128 x 128 tile: every element is read once and both outputs are made
// from registers, the codes along the rows and (kT) the transposed copy that the backward
// products reduce along. 256 threads: thread (rg, cv) holds rows [8 rg, 8 rg + 8) of the
// 8 columns at 8 cv, so a half-warp reads one row's 256 contiguous bytes, a row maximum is
// four shuffles over the half-warp, and the eight codes of one column are one 8-byte word
// of the transposed tile in shared memory.
// Bound by HBM: 2 (4 for weights) bytes read, 1 + 1 written per element.
#pragma once

#include "pair_issue.cuh"

namespace bl {

enum : int { FP8_E4M3 = 0, FP8_E5M2 = 1 };

__host__ __device__ constexpr int fp8_top_exponent(int fmt) { return fmt == FP8_E5M2 ? 15 : 8; }

// Scale byte of a block whose largest |value| has the fp32 pattern `bits`: adding
// 0x1FFFFF carries into the exponent exactly when the mantissa is above 0x600000 (1.75).
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t bits, int top) {
  const int e = static_cast<int>((bits + 0x1FFFFFu) >> 23) - top;
  return bits >= 0x7F800000u ? 255u : static_cast<uint32_t>(e > 0 ? e : 0);
}
// 2^-e of a scale byte (exact; byte <= 247 for finite blocks), NaN for byte 255.
__device__ __forceinline__ float fp8_inv_scale(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FFFFFFFu : (254u - byte) << 23);
}
// The same as bf16, in both halves.
__device__ __forceinline__ uint32_t fp8_inv_scale_bf16x2(uint32_t byte) {
  const uint32_t h = byte == 255u ? 0x7FFFu : (254u - byte) << 7;
  return h | h << 16;
}
// Two bf16 times two powers of two: exact down to bf16's subnormals, which are far below
// half of either format's smallest code.
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&r);
}
// Larger magnitudes of two bf16 pairs; a NaN stays one (its pattern is above every number's).
__device__ __forceinline__ uint32_t absmax_bf16x2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 r = __hmax2_nan(__habs2(*reinterpret_cast<const __nv_bfloat162*>(&a)),
                                       __habs2(*reinterpret_cast<const __nv_bfloat162*>(&b)));
  return *reinterpret_cast<const uint32_t*>(&r);
}

// Two codes, `lo` in the low byte.
template <bool kE5M2>
__device__ __forceinline__ uint32_t fp8_pack2(float lo, float hi) {
  uint16_t r;
  if (kE5M2) asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
template <bool kE5M2>
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  return fp8_pack2<kE5M2>(a, b) | fp8_pack2<kE5M2>(c, d) << 16;
}

// Codes of two scaled bf16 pairs.
template <bool kE5M2>
__device__ __forceinline__ uint32_t fp8_codes4(uint32_t a, uint32_t b) {
  return fp8_pack4<kE5M2>(__uint_as_float(a << 16), __uint_as_float(a & 0xFFFF0000u), __uint_as_float(b << 16),
                          __uint_as_float(b & 0xFFFF0000u));
}

struct Fp8QuantArgs {
  const void* src;        // bf16 (activations) or fp32 (weights) [rows, cols]
  int64_t rows, cols;     // cols % 16 == 0
  int64_t rows_pad;       // row stride of qt: rows rounded up to 16
  uint8_t* q;             // [rows, cols]
  uint8_t* scales;        // [ceil(cols / 512), rows, 4]
  uint8_t* qt;            // [cols, rows_pad] (kT)
  uint8_t* scales_t;      // [ceil(rows / 512), cols, 4] (kT)
};

// One scale byte of block b of row r, in a [ceil(blocks / 4), rows, 4] array; the last
// block also clears the bytes behind it, so the whole array is always written.
__device__ __forceinline__ void fp8_put_scale(uint8_t* scales, int64_t rows, int64_t r, int b, int blocks, uint32_t byte) {
  uint8_t* p = scales + ((b >> 2) * rows + r) * 4;
  p[b & 3] = static_cast<uint8_t>(byte);
  if (b == blocks - 1)
    for (int j = (b & 3) + 1; j < 4; ++j) p[j] = 0;
}

constexpr int kFp8QuantThreads = 256;

template <bool kWeight, bool kE5M2, bool kT>
__global__ void __launch_bounds__(kFp8QuantThreads) fp8_quant_kernel(const Fp8QuantArgs a) {
  constexpr int kTop = fp8_top_exponent(kE5M2 ? FP8_E5M2 : FP8_E4M3);
  __shared__ __align__(16) uint32_t s_max[8][64];            // per warp: column maxima (bf16 pairs) or one block maximum
  __shared__ __align__(16) uint32_t s_inv[64];               // column pairs' 2^-e
  __shared__ __align__(16) uint8_t s_t[kT ? 128 * 128 : 16];   // transposed codes
  __shared__ uint8_t s_row[128];                             // row scale bytes
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cv = lane & 15, rg = warp * 2 + (lane >> 4);
  const int col_blocks = static_cast<int>((a.cols + 127) / 128), row_blocks = static_cast<int>((a.rows + 127) / 128);
  // a row of tiles is read in order (32-bit division: tiles are counted in 31 bits)
  const int rb = static_cast<int>(blockIdx.x / static_cast<unsigned>(col_blocks));
  const int cb = static_cast<int>(blockIdx.x - static_cast<unsigned>(rb) * static_cast<unsigned>(col_blocks));
  const int64_t col0 = static_cast<int64_t>(cb) * 128 + cv * 8, row0 = static_cast<int64_t>(rb) * 128 + rg * 8;
  const int64_t at0 = row0 * a.cols + col0;   // this thread's first element
  const int rows_in = row0 < a.rows ? static_cast<int>(a.rows - row0 < 8 ? a.rows - row0 : 8) : 0;
  follow_stream();
  const bool col_ok = col0 < a.cols;   // cols % 8 == 0: a thread's 8 columns are all in or all out

  if constexpr (!kWeight) {
    // ------------------------------------------------ bf16, one scale per row and block
    uint4 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = make_uint4(0, 0, 0, 0);
      if (col_ok && i < rows_in) v[i] = ld_plain(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.src) + at0 + i * a.cols));
    }
    uint32_t rm[4] = {0, 0, 0, 0};   // maxima of row pairs (i, i + 4) as 16-bit |bf16| patterns
    uint32_t cm[4] = {0, 0, 0, 0};   // column pairs
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (kT) {
        cm[0] = absmax_bf16x2(cm[0], v[i].x);
        cm[1] = absmax_bf16x2(cm[1], v[i].y);
        cm[2] = absmax_bf16x2(cm[2], v[i].z);
        cm[3] = absmax_bf16x2(cm[3], v[i].w);
      }
      const uint32_t m2 = absmax_bf16x2(absmax_bf16x2(v[i].x, v[i].y), absmax_bf16x2(v[i].z, v[i].w));
      const uint32_t m = max(m2 & 0xFFFFu, m2 >> 16);
      rm[i & 3] |= i < 4 ? m : m << 16;
    }
#pragma unroll
    for (int off = 1; off < 16; off <<= 1)
#pragma unroll
      for (int j = 0; j < 4; ++j) rm[j] = __vmaxu2(rm[j], __shfl_xor_sync(0xFFFFFFFFu, rm[j], off));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t pat = i < 4 ? rm[i & 3] & 0xFFFFu : rm[i & 3] >> 16;
      const uint32_t byte = fp8_scale_byte(pat << 16, kTop);
      const uint32_t inv2 = fp8_inv_scale_bf16x2(byte);
      if (cv == i) s_row[rg * 8 + i] = static_cast<uint8_t>(byte);
      if (col_ok && i < rows_in)
        *reinterpret_cast<uint2*>(a.q + at0 + i * a.cols) =
            make_uint2(fp8_codes4<kE5M2>(mul_bf16x2(v[i].x, inv2), mul_bf16x2(v[i].y, inv2)),
                       fp8_codes4<kE5M2>(mul_bf16x2(v[i].z, inv2), mul_bf16x2(v[i].w, inv2)));
    }
    if (kT) {
#pragma unroll
      for (int j = 0; j < 4; ++j) cm[j] = __vmaxu2(cm[j], __shfl_xor_sync(0xFFFFFFFFu, cm[j], 16));
      if (lane < 16) *reinterpret_cast<uint4*>(&s_max[warp][cv * 4]) = make_uint4(cm[0], cm[1], cm[2], cm[3]);
    }
    __syncthreads();
    if (threadIdx.x < 128 && static_cast<int64_t>(rb) * 128 + threadIdx.x < a.rows)
      fp8_put_scale(a.scales, a.rows, static_cast<int64_t>(rb) * 128 + threadIdx.x, cb, col_blocks, s_row[threadIdx.x]);
    if constexpr (kT) {
      if (threadIdx.x < 64) {   // scales of a pair of columns
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 8; ++w) m = __vmaxu2(m, s_max[w][threadIdx.x]);
        const uint32_t b0 = fp8_scale_byte(m << 16, kTop), b1 = fp8_scale_byte(m & 0xFFFF0000u, kTop);
        s_inv[threadIdx.x] = (fp8_inv_scale_bf16x2(b0) & 0xFFFFu) | (fp8_inv_scale_bf16x2(b1) & 0xFFFF0000u);
        const int64_t col = static_cast<int64_t>(cb) * 128 + 2 * threadIdx.x;
        if (col < a.cols) {   // an even number of columns: both or none
          fp8_put_scale(a.scales_t, a.cols, col, rb, row_blocks, b0);
          fp8_put_scale(a.scales_t, a.cols, col + 1, rb, row_blocks, b1);
        }
      }
      __syncthreads();
      const uint4 inv4 = *reinterpret_cast<const uint4*>(&s_inv[cv * 4]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        // columns 2 j and 2 j + 1 side by side: one multiplication per row for both
        const uint32_t inv2 = j == 0 ? inv4.x : j == 1 ? inv4.y : j == 2 ? inv4.z : inv4.w;
        uint32_t p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = mul_bf16x2(j == 0 ? v[i].x : j == 1 ? v[i].y : j == 2 ? v[i].z : v[i].w, inv2);
        // 8-byte word rg of a column, its place rotated by the column group: a half-warp's
        // 16 words fall into 16 different bank pairs
        uint8_t* dst = s_t + (cv * 8 + 2 * j) * 128 + ((rg ^ cv) * 8);
        auto even = [&](int i) { return __uint_as_float(p[i] << 16); };
        auto odd = [&](int i) { return __uint_as_float(p[i] & 0xFFFF0000u); };
        *reinterpret_cast<uint2*>(dst) = make_uint2(fp8_pack4<kE5M2>(even(0), even(1), even(2), even(3)),
                                                    fp8_pack4<kE5M2>(even(4), even(5), even(6), even(7)));
        *reinterpret_cast<uint2*>(dst + 128) = make_uint2(fp8_pack4<kE5M2>(odd(0), odd(1), odd(2), odd(3)),
                                                          fp8_pack4<kE5M2>(odd(4), odd(5), odd(6), odd(7)));
      }
    }
  } else {
    // ------------------------------------------------ fp32, one scale per 128 x 128 block
    float4 v[8][2];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i][0] = v[i][1] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (col_ok && i < rows_in) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.src) + at0 + i * a.cols);
        v[i][0] = ld_plain(p);
        v[i][1] = ld_plain(p + 1);
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        m = max(m, max(max(__float_as_uint(v[i][j].x) & 0x7FFFFFFFu, __float_as_uint(v[i][j].y) & 0x7FFFFFFFu),
                       max(__float_as_uint(v[i][j].z) & 0x7FFFFFFFu, __float_as_uint(v[i][j].w) & 0x7FFFFFFFu)));
      }
    m = __reduce_max_sync(0xFFFFFFFFu, m);
    if (lane == 0) s_max[warp][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, s_max[w][0]);
    const uint32_t byte = fp8_scale_byte(m, kTop);
    const float inv = fp8_inv_scale(byte);
    uint2 c[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = make_uint2(fp8_pack4<kE5M2>(v[i][0].x * inv, v[i][0].y * inv, v[i][0].z * inv, v[i][0].w * inv),
                        fp8_pack4<kE5M2>(v[i][1].x * inv, v[i][1].y * inv, v[i][1].z * inv, v[i][1].w * inv));
      if (col_ok && i < rows_in) *reinterpret_cast<uint2*>(a.q + at0 + i * a.cols) = c[i];
    }
    if (threadIdx.x < 128 && static_cast<int64_t>(rb) * 128 + threadIdx.x < a.rows)
      fp8_put_scale(a.scales, a.rows, static_cast<int64_t>(rb) * 128 + threadIdx.x, cb, col_blocks, byte);
    if constexpr (kT) {
      const int64_t col = static_cast<int64_t>(cb) * 128 + (threadIdx.x & 127);
      if (threadIdx.x >= 128 && col < a.cols) fp8_put_scale(a.scales_t, a.cols, col, rb, row_blocks, byte);
      // the same codes transposed: an 8 x 8 byte block per thread by byte permutes
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {   // columns 4 half .. 4 half + 3, rows 4 h .. 4 h + 3
          const uint32_t r0 = half ? c[4 * h].y : c[4 * h].x, r1 = half ? c[4 * h + 1].y : c[4 * h + 1].x;
          const uint32_t r2 = half ? c[4 * h + 2].y : c[4 * h + 2].x, r3 = half ? c[4 * h + 3].y : c[4 * h + 3].x;
          const uint32_t a01 = __byte_perm(r0, r1, 0x5140), b01 = __byte_perm(r0, r1, 0x7362);
          const uint32_t a23 = __byte_perm(r2, r3, 0x5140), b23 = __byte_perm(r2, r3, 0x7362);
          const uint32_t t[4] = {__byte_perm(a01, a23, 0x5410), __byte_perm(a01, a23, 0x7632),
                                 __byte_perm(b01, b23, 0x5410), __byte_perm(b01, b23, 0x7632)};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            *reinterpret_cast<uint32_t*>(s_t + (cv * 8 + 4 * half + j) * 128 + ((rg ^ cv) * 8) + 4 * h) = t[j];
        }
      }
    }
  }
  if constexpr (kT) {
    __syncthreads();
    // 16 bytes (two words) of a column at a time, back in row order
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int idx = it * kFp8QuantThreads + threadIdx.x;
      const int c = idx >> 3, piece = idx & 7;
      const int64_t col = static_cast<int64_t>(cb) * 128 + c, row = static_cast<int64_t>(rb) * 128 + piece * 16;
      if (col < a.cols && row < a.rows_pad) {
        const int g = (c >> 3) & 15;
        const uint2 lo = *reinterpret_cast<const uint2*>(s_t + c * 128 + (((2 * piece) ^ g) * 8));
        const uint2 hi = *reinterpret_cast<const uint2*>(s_t + c * 128 + (((2 * piece + 1) ^ g) * 8));
        *reinterpret_cast<uint4*>(a.qt + col * a.rows_pad + row) = make_uint4(lo.x, lo.y, hi.x, hi.y);
      }
    }
  }
}

}  // namespace bl
