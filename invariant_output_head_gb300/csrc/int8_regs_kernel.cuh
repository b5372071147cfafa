// int8_regs_kernel.cuh -- scaled logits of 5 to 8 rows: W streamed through
// registers into the warp-level tensor-core instruction.
//
// out[n, v] = (sum_k q[n, k] W[v, k]) * (x_scale[n] * w_scale[v])
//
// The product is still a read of W. The int8-streaming kernel, which brings W
// by TMA, converts it to fp16 and hands it to tcgen05.mma through tensor
// memory, reads it at 5.0 TB/s; loads into registers read it at 6.2 here. For
// eight rows the legacy instruction keeps up (mma.sync with fp16 inputs and an
// fp32 accumulator: 594 TFLOP/s measured on GB300, 1029 multiply-adds per clock
// and SM): 8 x 128256 x 4096 in 84.6 us against 106.9. With 16 rows it runs
// 106.9, with 32 161.6: its rate and the conversions of q bind, and those go to
// the streaming kernel. Every int8 value is exact in fp16 and every product at
// most 2^14, so sums over at most 1024 elements of K are exact in fp32; warps'
// sums meet in int32. The logits are the other kernels' bit for bit.
//
// A warp holds 32 vocabulary rows x 64 elements of K a step: lane 4 g + t reads
// 16 bytes, k = 16 t .. 16 t + 15, of rows g, g + 8, g + 16, g + 24. K may be
// taken in any order, as long as q takes the same: the four bytes 4 j .. 4 j + 3
// of each lane are the instruction's k = 2 t, 2 t + 1, 2 t + 8, 2 t + 9 in step
// j, for W and q alike, so no byte moves between lanes. q stays int8 in shared
// memory and is converted where it is used. The block's 16 warps split into wr
// groups of 32 rows times wk shares of K (at most 16 steps each); the shares
// meet in a shared int32 tile (exact in any order), which all threads then
// scale and write. Loads run two steps ahead, over the ends of rounds.
#pragma once
#include "int8_kernels.cuh"
#include "int8_rows_kernel.cuh"

namespace detlm {

constexpr int kI8RegsThreads = 512;
constexpr int kI8RegsMax = 8;           // rows of q (the instruction's N)
constexpr int kI8RegsSums = 16;         // row stride of the shared sums, words

struct Int8RegsParams {
  const int8_t* W;          // [V][d]
  const int8_t* q;          // [B][d]
  const float* x_scale;
  const float* w_scale;
  void* out;                // [B][V]
  int32_t V, d, B, type;    // type: OUT_*
  int32_t steps;            // 64-element steps of K
  int32_t wk;               // shares of K: 1, 2, 4, 8 or 16
};

// Row stride of q in shared memory: whole steps, half a bank row on (two rows
// read at once touch different banks).
__host__ __device__ inline int int8_regs_stride(int steps) { return steps * 64 + ((steps & 1) ? 0 : 64); }
__host__ __device__ inline size_t int8_regs_smem(int steps, int wk) {
  return static_cast<size_t>(kI8RegsMax) * int8_regs_stride(steps) +
         2u * (16 / wk) * 32u * kI8RegsSums * 4u;
}

__device__ __forceinline__ void mma_16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                          uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__global__ void __launch_bounds__(kI8RegsThreads, 1) int8_regs_kernel(const Int8RegsParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const int stride = int8_regs_stride(p.steps);
  const int wr = 16 / p.wk;                      // groups of 32 rows a round
  const int my_r = warp / p.wk, my_k = warp - my_r * p.wk;
  uint8_t* sq = smem_raw;
  int32_t* sums = reinterpret_cast<int32_t*>(smem_raw + kI8RegsMax * stride);
  const int sums_words = wr * 32 * kI8RegsSums;
  const int rows = 32 * wr;                      // vocabulary rows a round
  const int rounds = (p.V + rows - 1) / rows;
  const int mine = (p.steps - my_k + p.wk - 1) / p.wk;   // this warp's steps a round (0 or more)

  // the next step to load: round lr, the li-th of this warp's steps
  int lr = blockIdx.x, li = 0;
  uint4 x[2][4];
  auto load = [&](uint4 (&y)[4]) {
    const int k = 64 * (my_k + li * p.wk) + 16 * t;
    const bool in = lr < rounds && li < mine && k < p.d;
    const int v0 = lr * rows + my_r * 32 + g;
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      y[r] = make_uint4(0, 0, 0, 0);
      if (in)
        y[r] = load_stream(reinterpret_cast<const uint4*>(
            p.W + static_cast<size_t>(min(v0 + 8 * r, p.V - 1)) * p.d + k));
    }
    if (++li >= mine) {
      li = 0;
      lr += gridDim.x;
    }
  };
  // W does not change under a call: its first steps are requested before the
  // previous kernels on the stream are done
  if (mine > 0) {
    load(x[0]);
    load(x[1]);
  }
  for (int i = threadIdx.x; i < 2 * sums_words; i += kI8RegsThreads) sums[i] = 0;
  grid_dep_launch();
  grid_dep_wait();
  for (int i = threadIdx.x; i < kI8RegsMax * (stride / 16); i += kI8RegsThreads) {
    const int n = i / (stride / 16), k = 16 * (i - n * (stride / 16));
    uint4 w = make_uint4(0, 0, 0, 0);
    if (n < p.B && k < p.d)
      w = *reinterpret_cast<const uint4*>(p.q + static_cast<size_t>(n) * p.d + k);
    *reinterpret_cast<uint4*>(sq + n * stride + k) = w;
  }
  __syncthreads();

  int turn = 0;
  for (int round = blockIdx.x; round < rounds; round += gridDim.x, turn ^= 1) {
    float acc[2][4] = {};                        // rows 0-15, 16-31 of the warp's 32
    auto step = [&](uint4 (&y)[4], int i) {
      uint32_t a[4][2][4];                        // [MMA step][rows 0-15, 16-31][fragment]
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t w[4] = {y[r].x, y[r].y, y[r].z, y[r].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) i8x4_to_h2x2(w[j], a[j][r >> 1][r & 1], a[j][r >> 1][2 + (r & 1)]);
      }
      load(y);                                    // two steps ahead
      const uint4 u = *reinterpret_cast<const uint4*>(sq + g * stride + 64 * (my_k + i * p.wk) + 16 * t);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t b0, b1;
        i8x4_to_h2x2(w[j], b0, b1);
        mma_16816(acc[0], a[j][0], b0, b1);
        mma_16816(acc[1], a[j][1], b0, b1);
      }
    };
    // (a warp's steps alternate between the two sets of registers; with an odd
    // number of them the sets swap roles from round to round)
    int i = 0;
    const bool swap = (mine & 1) != 0 && (((round - blockIdx.x) / gridDim.x) & 1) != 0;
    if (swap) {
      for (; i + 1 < mine; i += 2) {
        step(x[1], i);
        step(x[0], i + 1);
      }
      if (i < mine) step(x[1], i);
    } else {
      for (; i + 1 < mine; i += 2) {
        step(x[0], i);
        step(x[1], i + 1);
      }
      if (i < mine) step(x[0], i);
    }
    int32_t* s = sums + turn * sums_words;
    if (mine > 0) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          atomicAdd(&s[(my_r * 32 + m * 16 + g + 8 * (c >> 1)) * kI8RegsSums + 2 * t + (c & 1)],
                    __float2int_rn(acc[m][c]));
    }
    __syncthreads();
    // every thread: vocabulary row by row fastest, so a warp writes 32
    // consecutive entries of a row of out; the tile is left at zero
    const int v0 = round * rows;
    for (int o = threadIdx.x; o < rows * kI8RegsMax; o += kI8RegsThreads) {
      const int n = o / rows, r = o - n * rows;
      int32_t* at = &s[r * kI8RegsSums + n];
      const int32_t sum = *at;
      *at = 0;
      const int v = v0 + r;
      if (n < p.B && v < p.V)
        store_scaled(p.out, static_cast<size_t>(n) * p.V + v,
                     __fmul_rn(__int2float_rn(sum), __fmul_rn(__ldg(p.x_scale + n), __ldg(p.w_scale + v))),
                     p.type);
    }
  }
}

}  // namespace detlm
