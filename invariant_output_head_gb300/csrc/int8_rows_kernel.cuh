// int8_rows_kernel.cuh -- scaled logits of up to four rows: W streamed through
// registers.
//
// out[n, v] = (sum_k q[n, k] W[v, k]) * (x_scale[n] * w_scale[v])
//
// With this few rows the product is a read of W: 23 bytes per clock and SM at
// the copy bandwidth, which dp4a (four int8 products and their exact int32 sum
// per lane and instruction) takes in with most of its rate to spare. So no
// tensor core, no conversion to fp16 and no shared-memory ring: eight lanes
// share a vocabulary row, 128 bytes of it at a time, four rows a warp, against
// the rows of q in shared memory (the four rows read the same 16 bytes). The
// lanes' sums meet in three shuffles at the end of K. Integer sums are exact
// in any order, so the logits are the wide kernels' bit for bit.
//
// Eight 16-byte loads a lane are in flight, 128 KB an SM at 32 warps, three
// times what latency times bandwidth asks for. Bound: HBM. 1 x 128256 x 4096:
// 73.9 us, 7.1 TB/s (the int8-streaming kernel: 106); 4 rows 86 us.
#pragma once
#include "int8_kernels.cuh"

namespace detlm {

constexpr int kI8RowsThreads = 512;     // two blocks an SM
constexpr int kI8RowsMax = 4;           // rows of q
constexpr int kI8RowsGroup = 4;         // vocabulary rows of a warp at a time
constexpr int kI8RowsAhead = 8;         // 16-byte loads of a lane in flight

struct Int8RowsParams {
  const int8_t* W;          // [V][d]
  const int8_t* q;          // [B][d]
  const float* x_scale;
  const float* w_scale;
  void* out;                // [B][V]
  int32_t V, d, B, type;    // type: OUT_*
};

__device__ __forceinline__ uint4 load_stream(const uint4* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}

template <int NB>
__global__ void __launch_bounds__(kI8RowsThreads, 2) int8_rows_kernel(const Int8RowsParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint4* sq = reinterpret_cast<uint4*>(smem_raw);        // [NB][d / 16]
  const int lane = threadIdx.x & 31;
  const int d16 = p.d >> 4;
  const int warps = gridDim.x * (kI8RowsThreads / 32);
  const int groups = (p.V + kI8RowsGroup - 1) / kI8RowsGroup;
  // groups go round the blocks, so that every SM reads the same share
  const int first = static_cast<int>(blockIdx.x) + (threadIdx.x >> 5) * static_cast<int>(gridDim.x);
  const uint4* W = reinterpret_cast<const uint4*>(p.W);
  grid_dep_launch();
  grid_dep_wait();
  for (int i = threadIdx.x; i < NB * d16; i += kI8RowsThreads) {
    const int n = i / d16;
    sq[i] = n < p.B ? reinterpret_cast<const uint4*>(p.q)[i] : make_uint4(0, 0, 0, 0);
  }
  __syncthreads();
  const int sub = lane & 7;                              // this lane's share of a row
  for (int g = first; g < groups; g += warps) {
    const int v = g * kI8RowsGroup + (lane >> 3);
    const uint4* w = W + static_cast<size_t>(min(v, p.V - 1)) * d16;
    int acc[NB] = {};
    for (int c0 = sub; c0 < d16; c0 += 8 * kI8RowsAhead) {
      uint4 x[kI8RowsAhead];
#pragma unroll
      for (int j = 0; j < kI8RowsAhead; ++j)
        x[j] = c0 + 8 * j < d16 ? load_stream(w + c0 + 8 * j) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < kI8RowsAhead; ++j) {
        if (c0 + 8 * j >= d16) break;
#pragma unroll
        for (int n = 0; n < NB; ++n) {
          const uint4 y = sq[n * d16 + c0 + 8 * j];
          acc[n] = __dp4a(static_cast<int>(x[j].x), static_cast<int>(y.x), acc[n]);
          acc[n] = __dp4a(static_cast<int>(x[j].y), static_cast<int>(y.y), acc[n]);
          acc[n] = __dp4a(static_cast<int>(x[j].z), static_cast<int>(y.z), acc[n]);
          acc[n] = __dp4a(static_cast<int>(x[j].w), static_cast<int>(y.w), acc[n]);
        }
      }
    }
    __syncwarp();
    // lane `sub` = n of each row keeps and writes sum n
    int mine = 0;
#pragma unroll
    for (int n = 0; n < NB; ++n) {
      int s = acc[n];
#pragma unroll
      for (int b = 1; b < 8; b <<= 1) s += __shfl_xor_sync(0xffffffffu, s, b);
      if (sub == n) mine = s;
    }
    if (sub < NB && sub < p.B && v < p.V)
      store_scaled(p.out, static_cast<size_t>(sub) * p.V + v,
                   __fmul_rn(__int2float_rn(mine), __fmul_rn(p.x_scale[sub], p.w_scale[v])), p.type);
  }
}

}  // namespace detlm
