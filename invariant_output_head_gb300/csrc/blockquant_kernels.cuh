// blockquant_kernels.cuh -- float rows (bf16, fp16 or fp32) in e4m3 with a
// scale for each block: 1 x 128 elements (hidden rows) or 128 x 128 (weights).
//
//   scale = 2^e, e >= -126 the smallest with max |x| <= 448 * 2^e
//   q     = x / scale, rounded to nearest even
//
// The scale is dyadic, as the int8 front end's are: dividing by it is exact, so
// every q is one rounding of x itself and has one right value. An empty block's
// scale is 1; a block with a NaN or an infinity has NaN for its scale and all of
// its q, which reaches every logit of the row.
//
// e from the bits of amax = 1.f * 2^k: 448 = 1.75 * 2^8, so e is k - 8, or one
// more where 1.f > 1.75.
//
// One pass: a block's elements stay in registers between its maximum and its
// conversion. Eight elements a lane (16 bytes of a 16-bit row), 16 lanes a row
// of a block. Bound by memory for weights: 128256 x 4096 bf16 in 128 x 128 blocks
// 234 us, 6.73 TB/s (285 with two blocks of threads an SM instead of three: their
// loads are what is on its way); in rows 240 us (292 with 64-bit divisions for a
// block's place). A decode batch of 32 rows is the launch and two latencies.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cstdint>
#include "quant_kernels.cuh"

namespace detlm {

constexpr int kBQThreads = 256;
constexpr int kBQBlock = 128;

struct BlockQuantParams {
  const void* x;
  int64_t B, d;
  int32_t nb;            // blocks of a row
  uint8_t* q;            // [B, d] e4m3
  float* scale;          // [B or ceil(B / 128), nb]
};

// Two floats in e4m3, the first in the low byte (round to nearest even,
// magnitudes above 448 to 448, NaN to NaN).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// Eight elements of a row, as loaded.
template <int FMT>
struct Eight {
  uint4 w[FMT == QF_FP32 ? 2 : 1];
  __device__ __forceinline__ void load(const void* x, size_t at) {
    const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(x) +
                                                    at * (FMT == QF_FP32 ? 4 : 2));
#pragma unroll
    for (int i = 0; i < (FMT == QF_FP32 ? 2 : 1); ++i) w[i] = p[i];
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < (FMT == QF_FP32 ? 2 : 1); ++i) w[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void values(float (&f)[8]) const {
    if constexpr (FMT == QF_FP32) {
      const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i]);
    } else {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (FMT == QF_BF16) {
          f[2 * i] = __uint_as_float(u[i] << 16);
          f[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
        } else {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
          f[2 * i] = v.x;
          f[2 * i + 1] = v.y;
        }
      }
    }
  }
  // largest magnitude as fp32 bits (NaN above infinity above every number)
  __device__ __forceinline__ uint32_t amax() const {
    float f[8];
    values(f);
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(f[i]) & 0x7FFFFFFFu);
    return m;
  }
  __device__ __forceinline__ uint2 convert(float inv) const {
    float f[8];
    values(f);
    uint2 r;
    r.x = e4m3x2(f[0] * inv, f[1] * inv) | (e4m3x2(f[2] * inv, f[3] * inv) << 16);
    r.y = e4m3x2(f[4] * inv, f[5] * inv) | (e4m3x2(f[6] * inv, f[7] * inv) << 16);
    return r;
  }
};

// The scale of a block and its inverse, both powers of two and normal.
struct BlockScale {
  float scale, inv;
  bool ok;
  __device__ __forceinline__ explicit BlockScale(uint32_t amax) {
    ok = amax < 0x7F800000u;
    int e = static_cast<int>(amax >> 23) - 127 - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = max(e, -126);
    if (amax == 0) e = 0;
    scale = ok ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23) : __uint_as_float(0x7FC00000u);
    inv = ok ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) : 0.0f;
  }
};

__device__ __forceinline__ uint32_t max16(uint32_t m) {   // over 16 neighbouring lanes
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// 1 x 128: 16 lanes a block, kBQPer blocks in flight a thread.
constexpr int kBQPer = 4;
template <int FMT>
__global__ void __launch_bounds__(kBQThreads) quantize_blocks_kernel(const BlockQuantParams p) {
  grid_dep_launch();
  grid_dep_wait();
  const uint32_t total = static_cast<uint32_t>(p.B) * static_cast<uint32_t>(p.nb);   // (below 2^31)
  const uint32_t l = threadIdx.x & 15;
  const uint32_t first = blockIdx.x * (kBQPer * (kBQThreads / 16)) + (threadIdx.x >> 4);
  Eight<FMT> x[kBQPer];
  size_t at[kBQPer];
#pragma unroll
  for (int i = 0; i < kBQPer; ++i) {
    const uint32_t b = first + i * (kBQThreads / 16);
    const uint32_t n = b / static_cast<uint32_t>(p.nb);
    const int64_t k = static_cast<int64_t>(b - n * p.nb) * kBQBlock + 8 * l;
    at[i] = b < total && k < p.d ? static_cast<size_t>(n * p.d + k) : SIZE_MAX;
    if (at[i] != SIZE_MAX) x[i].load(p.x, at[i]);
    else x[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kBQPer; ++i) {
    const uint32_t b = first + i * (kBQThreads / 16);
    const BlockScale s(max16(x[i].amax()));
    if (at[i] != SIZE_MAX)
      *reinterpret_cast<uint2*>(p.q + at[i]) =
          s.ok ? x[i].convert(s.inv) : make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
    if (l == 0 && b < total) p.scale[b] = s.scale;
  }
}

// 128 x 128: one block of threads a tile, eight rows of it a thread. (No early
// start for what follows: a head's calls read the weight it writes.)
template <int FMT>
__global__ void __launch_bounds__(kBQThreads, 3) quantize_tiles_kernel(const BlockQuantParams p) {
  grid_dep_wait();
  const uint32_t tile = blockIdx.x;
  const uint32_t ti = tile / static_cast<uint32_t>(p.nb), tj = tile - ti * p.nb;
  const int64_t k = static_cast<int64_t>(tj) * kBQBlock + 8 * (threadIdx.x & 15);
  const int64_t n0 = static_cast<int64_t>(ti) * kBQBlock + (threadIdx.x >> 4);
  constexpr int kRows = kBQBlock * 16 / kBQThreads;
  Eight<FMT> x[kRows];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t n = n0 + i * (kBQThreads / 16);
    if (n < p.B && k < p.d) x[i].load(p.x, static_cast<size_t>(n * p.d + k));
    else x[i].zero();
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) m = max(m, x[i].amax());
  m = __reduce_max_sync(0xffffffffu, m);
  __shared__ uint32_t wmax[kBQThreads / 32];
  if ((threadIdx.x & 31) == 0) wmax[threadIdx.x >> 5] = m;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kBQThreads / 32; ++w) m = max(m, wmax[w]);
  const BlockScale s(m);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t n = n0 + i * (kBQThreads / 16);
    if (n < p.B && k < p.d)
      *reinterpret_cast<uint2*>(p.q + static_cast<size_t>(n * p.d + k)) =
          s.ok ? x[i].convert(s.inv) : make_uint2(0x7F7F7F7Fu, 0x7F7F7F7Fu);
  }
  if (threadIdx.x == 0) p.scale[tile] = s.scale;
}

}  // namespace detlm
