// block_kernels.cuh -- the projection of an 8-bit floating-point (e4m3) head
// whose values carry a scale for each block of 128.
//
//   out[n, v] = sum_c xs[n, c] ws[v / 128, c] (sum_{k in c} q[n, k] W[v, k])
//
// c counts the blocks of 128 elements of K. A block's sum is one chunk of the
// tensor core (tcgen05.mma kind::f8f6f4, four K = 32 steps into an accumulator
// that starts from zero): its products are exact and it is held in fp32. The
// epilogue takes it out of tensor memory and adds it, times the product of the
// two scales (rounded once), with one fused multiply-add, blocks in ascending
// order. Every logit's arithmetic is this whatever the number of rows, the
// kernel and the place in a tile, so a row's bits do not depend on its batch.
//
// A 128-byte row of a swizzled shared-memory box holds 128 elements: one box of
// K is one block of the scales, and one drain of tensor memory. That is what
// sets the layout of both kernels: the drains, at half the MMA time per byte of
// the 16-bit heads, have to run beside the MMAs.
//
// block_gemm_kernel: up to 128 rows. A read of W: vocabulary rows are the MMA's
// M axis, hidden rows its N. One CTA per SM takes a contiguous share of the
// vocabulary in groups of 32 rows (whole tiles of 128 would leave the last round
// of V = 32000 a third full): tiles of four groups, the last of fewer, whose
// missing groups are not loaded. A warp's 32 rows lie in one block of w_scale.
// Bound by the stream of W from memory: 32 rows x 128256 x 4096 in 82 us, 6.48
// TB/s of the 6.78 that a copy reaches; one row of 32000 x 2048 in 14.2 us, of
// which some 4.5 are the launch, the first boxes' latency and the last drain. W's
// first boxes are requested before the prologue (2 us more without). Up to 64
// rows a row more costs nothing (86 us); at 96 and 128 (98 and 114) the hidden
// rows' boxes, which every SM reads from L2, are as large as W's.
//
// block_pair_kernel: more rows, on CTA pairs (see pairop_kernels.cuh for the
// pair protocol): 256 hidden rows x 256 vocabulary rows a unit, a thread holds
// one hidden row's 128 logits of one vocabulary tile, so its scales are one
// value of its row and one of the tile a block. Bound by the drains, which run
// nearly after the MMAs instead of beside them: 2048 rows x 128256 x 4096 in 915
// to 925 us, 2.33 PFLOP/s, a block of K every 0.54 us, tensor pipe 45 %, issue
// slots 40 %. The four pairs of MMAs alone take 0.27 us at 1.9 GHz (without
// tensor-memory reads and sums the kernel takes 609 us), a drain's sums, 64 packed
// multiply-adds of each of two warps a scheduler, 256 cycles or 0.135 us: both
// would fit beside each other, but the reads and waits before the sums do not
// hide behind two warps a scheduler. What it took: accumulator slots by vocabulary
// tile, so that the two tiles' warps come one after the other (985 -> 975 us); no
// spilled registers (-> 936; 232 a thread -> 915); two threads issuing (no change).
// Slower: sixteen warps of 64 columns with 104 registers, read 32 at a time (2402:
// they spill; 16 at a time is not tried), row scales loaded four at a time (999 to
// 1047), single multiply-adds (974), the loop unrolled by the two slots (1690:
// spills).
#pragma once
#include "pairop_kernels.cuh"

namespace detlm {

constexpr int kBlockK = 128;               // elements of K a scale covers
constexpr int kBlockMaxD = 16384;          // bounds the row scales in shared memory
constexpr int kBlockGroup = 32;            // vocabulary rows of a group
constexpr int kBlockMaxStages = 12;
constexpr int kBlockMaxSlots = 8;

// D[tmem] (+)= A[smem] * B[smem]^T of e4m3 values, fp32 accumulator.
__device__ __forceinline__ void mma_f8(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                       uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f8_pair(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}"
      :: "r"(d_tmem), "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Instruction descriptor, kind::f8f6f4: fp32 D, A and B e4m3 (format 0), both
// K-major, shape M x N.
__host__ __device__ constexpr uint32_t idesc_e4m3(uint32_t M, uint32_t N) {
  return (1u << 4) | ((N >> 3) << 17) | ((M >> 4) << 24);
}
// The wait for this thread's tensor-memory loads, tied to the registers that
// they fill: nothing that reads those moves above it.
__device__ __forceinline__ void tmem_wait_ld_of(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]),
                 "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]),
                 "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]),
                 "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]),
                 "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :: "memory");
}

struct BlockParams {
  const float* x_scale;     // [B][nk]
  const float* w_scale;     // [ceil(V / 128)][nk]
  void* out;                // [B][V]
  int32_t V, B, nk;         // nk: blocks of K
  int32_t type;             // OUT_*
  uint32_t idesc;
  int32_t stages, slots, stall;
  int32_t n1, units, tma;   // block_pair_kernel: hidden-row tiles, units, whether out has a tensor map
  uint64_t timeout_ns;
  int* err;
};
static_assert(sizeof(BlockParams) <= 128, "kernel parameter struct above 128 bytes");

__device__ __forceinline__ void store_out(void* out, size_t at, float x, int type) {
  if (type == OUT_F32) static_cast<float*>(out)[at] = x;
  else if (type == OUT_BF16) static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
  else static_cast<__half*>(out)[at] = __float2half_rn(x);
}

// ------------------------------------------------------------- up to 128 rows
// K boxes of a stage (and of an accumulator slot): two while a slot ring of
// four fits, which halves the barriers a byte of W passes.
__host__ __device__ constexpr int block_kps(int N) { return N <= 64 ? 2 : 1; }
// Epilogue warps: a warp's drain of more than 64 columns takes longer than W's
// box takes to come (96 rows x 128256 x 4096: 125 us with four, 98 with eight), so two share a quarter's columns there.
__host__ __device__ constexpr int block_warps(int N) { return N <= 64 ? 4 : 8; }
__host__ __device__ constexpr int block_threads(int N) { return 64 + 32 * block_warps(N); }

struct BlockLayout {
  uint32_t stage_bytes, ctrl_off, sx_off, total;
};
// Stage s: kps W boxes [128 rows x 128 B], then kps hidden-row boxes [N x 128
// B]; barriers full[S], empty[S], slot_full[8], slot_empty[8], never, drain, the
// TMEM address holder and the abort flag; the row scales, [nk][N].
__host__ __device__ inline BlockLayout block_layout(int N, int stages, int nk) {
  BlockLayout L;
  L.stage_bytes = static_cast<uint32_t>(block_kps(N)) * (kBM + N) * kRowBytes;
  L.ctrl_off = static_cast<uint32_t>(stages) * L.stage_bytes;
  L.sx_off = L.ctrl_off + (2u * kBlockMaxStages + 2u * kBlockMaxSlots + 2u) * 8u + 16u;
  L.sx_off = (L.sx_off + 127u) & ~127u;
  L.total = L.sx_off + static_cast<uint32_t>(nk) * N * 4u;
  return L;
}

// tmW: box of 128 vocabulary rows; tmG: of one group; tmX: of the hidden rows
// (as many as there are, in whole 8-row swizzle atoms: h_rows).
template <int NBLK>
__global__ void __launch_bounds__(block_threads(16 * NBLK), 1)
block_gemm_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmG,
                  const __grid_constant__ CUtensorMap tmX, const BlockParams p) {
  constexpr int N = 16 * NBLK;
  constexpr int KPS = block_kps(N);
  constexpr int EW = block_warps(N), ET = 32 * EW;
  constexpr int NW = N * 4 / EW;                   // columns of an epilogue warp
  static_assert(NW % 16 == 0, "whole 16-column blocks");
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int S = p.stages, SL = p.slots;
  const BlockLayout L = block_layout(N, S, p.nk);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.ctrl_off);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (kBlockMaxStages + s); };
  auto accf_bar = [&](int b) { return bar0 + 8u * (2 * kBlockMaxStages + b); };
  auto acce_bar = [&](int b) { return bar0 + 8u * (2 * kBlockMaxStages + kBlockMaxSlots + b); };
  const uint32_t never_bar = bar0 + 8u * (2 * kBlockMaxStages + 2 * kBlockMaxSlots);
  const uint32_t drain_bar = never_bar + 8u;
  uint32_t* tmem_holder =
      reinterpret_cast<uint32_t*>(smem + L.ctrl_off + (2 * kBlockMaxStages + 2 * kBlockMaxSlots + 2) * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  float* sx = reinterpret_cast<float*>(smem + L.sx_off);
  const uint32_t smem_base = smem_u32(smem);
  auto sW = [&](int s, int b) {
    return smem_base + static_cast<uint32_t>(s) * L.stage_bytes + static_cast<uint32_t>(b) * (kBM * kRowBytes);
  };
  auto sX = [&](int s, int b) {
    return sW(s, KPS) + static_cast<uint32_t>(b) * (N * kRowBytes);
  };

  const int64_t groups = (static_cast<int64_t>(p.V) + kBlockGroup - 1) / kBlockGroup;
  const int g0 = static_cast<int>(groups * blockIdx.x / gridDim.x);
  const int g1 = static_cast<int>(groups * (blockIdx.x + 1) / gridDim.x);
  const int steps = (p.nk + KPS - 1) / KPS;
  const uint64_t pol_w = policy_evict_first();
  const uint64_t pol_x = policy_evict_last();
  const uint32_t x_bytes = static_cast<uint32_t>((p.B + 7) / 8 * 8) * kRowBytes;
  // boxes of a step: W's (and the bytes that the step's barrier waits for),
  // the hidden rows'
  auto load_w = [&](uint32_t stage, int g, int st) {
    const int ng = min(4, g1 - g), nb = min(KPS, p.nk - st * KPS);
    mbar_expect_tx(full_bar(stage), nb * (static_cast<uint32_t>(ng) * kBlockGroup * kRowBytes + x_bytes));
    for (int b = 0; b < nb; ++b) {
      const int k = (st * KPS + b) * kBlockK;
      if (ng == 4) {
        tma_load_2d(sW(stage, b), &tmW, k, g * kBlockGroup, full_bar(stage), pol_w);
      } else {
        for (int i = 0; i < ng; ++i)
          tma_load_2d(sW(stage, b) + i * (kBlockGroup * kRowBytes), &tmG, k, (g + i) * kBlockGroup,
                      full_bar(stage), pol_w);
      }
    }
  };
  auto load_x = [&](uint32_t stage, int st) {
    const int nb = min(KPS, p.nk - st * KPS);
    for (int b = 0; b < nb; ++b)
      tma_load_2d(sX(stage, b), &tmX, (st * KPS + b) * kBlockK, 0, full_bar(stage), pol_x);
    mbar_arrive(full_bar(stage));
  };
  // W is read-only between announced changes: the first stages' boxes of it are
  // requested before the previous kernels on the stream are done, and before
  // anything else here
  const int pre = min(S, (g1 - g0 + 3) / 4 * steps);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);
      mbar_init(empty_bar(s), 1);
    }
    for (int b = 0; b < SL; ++b) {
      mbar_init(accf_bar(b), 1);
      mbar_init(acce_bar(b), EW);      // the epilogue warps
    }
    mbar_init(never_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
    for (int j = 0; j < pre; ++j) load_w(j, g0 + j / steps * 4, j % steps);
    tma_prefetch_desc(&tmX);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_holder), 512u);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  // the call after this one may start its prologue on SMs that are free
  grid_dep_launch();

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    if (lane == 0) {
      grid_dep_wait();
      uint32_t stage = 0, phase = 0, outstanding = 0, out_par = 0;
      bool ok = true;
      int j = 0;
      for (int g = g0; g < g1 && ok; g += 4) {
        for (int st = 0; st < steps; ++st, ++j) {
          if (j >= pre) {
            if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.timeout_ns)) { ok = false; break; }
            load_w(stage, g, st);
          }
          load_x(stage, st);
          outstanding |= 1u << stage;
          out_par = (out_par & ~(1u << stage)) | (phase << stage);
          if (++stage == static_cast<uint32_t>(S)) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        atomicOr(p.err, ERR_TIMEOUT);
        // loads in flight land before the CTA's shared memory goes away
        const int zero = 0;
        for (int s = 0; s < S; ++s)
          if ((outstanding >> s) & 1u) mbar_wait(full_bar(s), (out_par >> s) & 1u, &zero, p.timeout_ns);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer
    if (lane == 0) {
      uint32_t stage = 0, phase = 0, slot = 0, sph = 0;
      bool ok = true;
      if (p.stall) ok = mbar_wait(never_bar, 0, abort_flag, p.timeout_ns);
      for (int g = g0; g < g1 && ok; g += 4) {
        for (int st = 0; st < steps; ++st) {
          if (!mbar_wait(acce_bar(slot), sph ^ 1u, abort_flag, p.timeout_ns)) { ok = false; break; }
          if (!mbar_wait(full_bar(stage), phase, abort_flag, p.timeout_ns)) { ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int b = 0; b < KPS; ++b) {
            if (st * KPS + b >= p.nk) break;
            const uint32_t d_tmem = tmem_base + (slot * KPS + b) * static_cast<uint32_t>(N);
            const uint64_t da = sdesc_sw128(sW(stage, b));
            const uint64_t db = sdesc_sw128(sX(stage, b));
#pragma unroll
            for (int k = 0; k < 4; ++k)       // K = 32 per MMA: 32 bytes = 2 descriptor units
              mma_f8(d_tmem, da + 2u * k, db + 2u * k, p.idesc, k != 0);
          }
          mma_commit(empty_bar(stage));
          mma_commit(accf_bar(slot));
          if (++stage == static_cast<uint32_t>(S)) { stage = 0; phase ^= 1u; }
          if (++slot == static_cast<uint32_t>(SL)) { slot = 0; sph ^= 1u; }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        atomicOr(p.err, ERR_TIMEOUT);
      }
      mma_commit(drain_bar);
      const int zero = 0;
      mbar_wait(drain_bar, 0, &zero, p.timeout_ns);
    }
    __syncwarp();
  } else {
    // --------------------------------------------------------- epilogue
    const int q = warp & 3;                    // TMEM lane quarter: the tile's group
    const int n_first = (warp - 2) / 4 * NW;   // first column: a hidden row
    const int et = threadIdx.x - 64;
    const uint32_t tlane = static_cast<uint32_t>(q * 32) << 16;
    grid_dep_wait();                           // the scales are the previous kernels' outputs
    for (int i = et; i < p.nk * N; i += ET) {
      const int c = i / N, n = i - (i / N) * N;
      sx[i] = n < p.B ? p.x_scale[static_cast<size_t>(n) * p.nk + c] : 0.0f;
    }
    named_bar_sync(1, ET);
    uint32_t slot = 0, sph = 0;
    bool failed = false;
    for (int g = g0; g < g1; g += 4) {
      const bool mine = g + q < g1;            // this warp's group exists
      const int v = mine ? (g + q) * kBlockGroup + lane : 0;
      const float* ws = p.w_scale + static_cast<size_t>(mine ? (g + q) / (kBM / kBlockGroup) : 0) * p.nk;
      float2 acc[NW / 2];
#pragma unroll
      for (int i = 0; i < NW / 2; ++i) acc[i] = make_float2(0.0f, 0.0f);
      float sw[KPS];
#pragma unroll
      for (int b = 0; b < KPS; ++b) sw[b] = b < p.nk ? ws[b] : 0.0f;
      for (int st = 0; st < steps; ++st) {
        float sw_next[KPS];
#pragma unroll
        for (int b = 0; b < KPS; ++b) {
          const int c = (st + 1) * KPS + b;
          sw_next[b] = c < p.nk ? ws[c] : 0.0f;
        }
        const uint32_t cur = slot, cph = sph;
        if (++slot == static_cast<uint32_t>(SL)) { slot = 0; sph ^= 1u; }
        if (!failed && !mbar_wait(accf_bar(cur), cph, abort_flag, p.timeout_ns)) {
          failed = true;
          *abort_flag = 1;
        }
        if (failed) continue;
        tc_fence_after();
        if (mine) {
#pragma unroll
          for (int b = 0; b < KPS; ++b) {
            const int c = st * KPS + b;
            if (c >= p.nk) break;
            const uint32_t at = tmem_base + tlane + (cur * KPS + b) * static_cast<uint32_t>(N) +
                                static_cast<uint32_t>(n_first);
            const float* s = sx + c * N + n_first;
            const float2 w2 = make_float2(sw[b], sw[b]);
            auto add16 = [&](const uint32_t* r, int n0) {
#pragma unroll
              for (int i = 0; i < 16; i += 4) {
                const float4 x = *reinterpret_cast<const float4*>(s + n0 + i);
                float2* a = &acc[(n0 + i) / 2];
                a[0] = fma2_rn(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])),
                               mul2_rn(make_float2(x.x, x.y), w2), a[0]);
                a[1] = fma2_rn(make_float2(__uint_as_float(r[i + 2]), __uint_as_float(r[i + 3])),
                               mul2_rn(make_float2(x.z, x.w), w2), a[1]);
              }
            };
            if constexpr (NW % 32 != 0) {
              uint32_t r[16];
              tmem_ld16(at + NW - 16, r);
              tmem_wait_ld();
              add16(r, NW - 16);
            }
#pragma unroll
            for (int h = 0; h < NW / 32; ++h) {
              uint32_t r[32];
              tmem_ld32(at + h * 32, r);
              tmem_wait_ld_of(r);
              add16(r, h * 32);
              add16(r + 16, h * 32 + 16);
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(acce_bar(cur));
#pragma unroll
        for (int b = 0; b < KPS; ++b) sw[b] = sw_next[b];
      }
      if (__any_sync(0xffffffffu, failed || *abort_flag)) {
        *abort_flag = 1;
        if (lane == 0) atomicOr(p.err, ERR_TIMEOUT);
        failed = true;
        break;
      }
      if (mine && v < p.V) {
        size_t at = static_cast<size_t>(n_first) * p.V + v;
#pragma unroll
        for (int n = 0; n < NW; ++n, at += p.V)
          if (n_first + n < p.B) store_out(p.out, at, (n & 1) ? acc[n / 2].y : acc[n / 2].x, p.type);
      }
    }
  }
  // every MMA and every tensor-memory load is done
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, 512u);
  }
}

// ------------------------------------------------------------ more than 128 rows
constexpr int kBlockPairMaxStages = 6;

struct BlockPairLayout {
  uint32_t stage_bytes, ctrl_off, xs_off, total;
};
// Stage s: this CTA's 128 hidden rows [128 x 128 B], its 64 rows of either
// vocabulary tile; barriers (full[S], empty[S], slot_full[4], slot_empty[4],
// never, drain[2]), the TMEM address holder and the abort flag; the epilogue
// warps' staging buffers.
__host__ __device__ inline BlockPairLayout block_pair_layout(int stages) {
  BlockPairLayout L;
  L.stage_bytes = 2u * kRowsHalf * kRowBytes;
  L.ctrl_off = static_cast<uint32_t>(stages) * L.stage_bytes;
  L.xs_off = (L.ctrl_off + (2u * stages + 11u) * 8u + 16u + 1023u) & ~1023u;
  L.total = L.xs_off + 8u * kOpXsBytes;
  return L;
}

__global__ void __launch_bounds__(kRowsThreads, 1)
block_pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW,
                  const __grid_constant__ CUtensorMap tmO, const BlockParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int S = p.stages;
  const BlockPairLayout L = block_pair_layout(S);
  const uint32_t rank = cluster_rank();            // 0: leader, 1: peer
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int n_pairs = static_cast<int>(gridDim.x >> 1);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.ctrl_off);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto accf_bar = [&](int b) { return bar0 + 8u * (2 * S + b); };
  auto acce_bar = [&](int b) { return bar0 + 8u * (2 * S + 4 + b); };
  const uint32_t never_bar = bar0 + 8u * (2 * S + 8);
  const uint32_t drain_bar = bar0 + 8u * (2 * S + 9);      // and the next
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L.ctrl_off + (2 * S + 11) * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const uint32_t smem_base = smem_u32(smem);
  auto sX = [&](int s) { return smem_base + static_cast<uint32_t>(s) * L.stage_bytes; };
  auto sW = [&](int s) { return sX(s) + kRowsHalf * kRowBytes; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);       // the leader's arrival (+ both CTAs' loads)
      mbar_init(empty_bar(s), 1);      // the leader's MMA commit
    }
    for (int b = 0; b < 4; ++b) {
      mbar_init(accf_bar(b), 1);       // the leader's MMA commit
      mbar_init(acce_bar(b), 8);       // four epilogue warps of each CTA
    }
    mbar_init(never_bar, 1);
    mbar_init(drain_bar, 1);
    mbar_init(drain_bar + 8u, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tmX);
    tma_prefetch_desc(&tmW);
    if (p.tma) tma_prefetch_desc(&tmO);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(tmem_holder), 512u);
    tmem_relinquish_pair();
  }
  // both CTAs' barriers are initialised before any load or arrival of the
  // other CTA can reach them
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_holder;
  const int half = static_cast<int>(rank) * kRowsHalf;

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRegsWg0Wide));
    if (lane == 0) {
      const uint64_t pol_w = policy_evict_normal();
      const uint64_t pol_x = policy_evict_last();
      const bool leader = rank == 0;
      grid_dep_wait();
      uint32_t stage = 0, phase = 0, outstanding = 0, out_par = 0;
      bool ok = true;
      for (int u = pair; u < p.units && ok; u += n_pairs) {
        const int vt = u / p.n1, rt = u - vt * p.n1;
        const int n0 = rt * 256 + half, v0 = vt * 256 + half / 2;
        // the peer's hidden rows may not exist: its box is not loaded then
        const uint32_t bytes = (2u + (rt * 256 + kRowsHalf < p.B ? 2u : 1u)) * kRowsHalf * kRowBytes;
        for (int c = 0; c < p.nk; ++c) {
          const uint32_t fb = cluster_addr(full_bar(stage), 0);
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.timeout_ns)) { ok = false; break; }
          if (leader) mbar_arrive_expect_tx(full_bar(stage), bytes);
          tma_load_2d_pair(sW(stage), &tmW, c * kBlockK, v0, fb, pol_w);
          tma_load_2d_pair(sW(stage) + 64 * kRowBytes, &tmW, c * kBlockK, v0 + 128, fb, pol_w);
          if (n0 < p.B) tma_load_2d_pair(sX(stage), &tmX, c * kBlockK, n0, fb, pol_x);
          outstanding |= 1u << stage;
          out_par = (out_par & ~(1u << stage)) | (phase << stage);
          if (++stage == static_cast<uint32_t>(S)) { stage = 0; phase ^= 1u; }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        atomicOr(p.err, ERR_TIMEOUT);
        if (leader) {
          // the armed stages complete once both CTAs' loads have landed
          const int zero = 0;
          for (int s = 0; s < S; ++s)
            if ((outstanding >> s) & 1u) mbar_wait(full_bar(s), (out_par >> s) & 1u, &zero, p.timeout_ns);
        } else {
          // the peer's loads complete on the leader's barriers: give the
          // ones in flight time to land before this CTA may leave
          const uint64_t t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < kPairSettleNs) __nanosleep(1000);
        }
      }
    }
    __syncwarp();
  } else if (warp < 3) {
    // ------------------------------------------------------ MMA issuers
    // One thread's waits, MMAs and commits take about 950 cycles a block of K, the
    // MMAs themselves 512: warps 1 and 2 issue every second block, each into its
    // own accumulator slots, one of each vocabulary tile. When a thread comes to
    // block c it has issued c - 2, whose slots were free once c - 4 was drained:
    // blocks are drained in order, so with four stages or more (the host makes no
    // fewer) what was in c's stage before is done, and the stage's parity means c.
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRegsWg0Wide));
    if (lane == 0 && rank == 0) {
      const uint32_t slot = static_cast<uint32_t>(warp - 1);
      uint32_t stage = slot, phase = 0, sph = 0;
      bool ok = true;
      if (p.stall) ok = mbar_wait(never_bar, 0, abort_flag, p.timeout_ns);
      int c = static_cast<int>(slot);            // this thread's block in the unit
      for (int u = pair; u < p.units && ok; u += n_pairs) {
        for (; c < p.nk; c += 2) {
          if (!mbar_wait(full_bar(stage), phase, abort_flag, p.timeout_ns)) { ok = false; break; }
          const uint64_t da = sdesc_sw128(sX(stage));
#pragma unroll
          for (int v = 0; v < 2; ++v) {           // vocabulary tile
            const uint32_t at = 2u * slot + v;
            if (!mbar_wait(acce_bar(at), sph ^ 1u, abort_flag, p.timeout_ns)) { ok = false; break; }
            tc_fence_after();
            const uint64_t db = sdesc_sw128(sW(stage) + v * (64u * kRowBytes));
#pragma unroll
            for (int k = 0; k < 4; ++k)           // K = 32 per MMA
              mma_f8_pair(tmem_base + at * 128u, da + 2u * k, db + 2u * k, p.idesc, k != 0);
            mma_commit_pair(accf_bar(at), 3);
          }
          if (!ok) break;
          mma_commit_pair(empty_bar(stage), 3);
          sph ^= 1u;
          stage += 2;
          if (stage >= static_cast<uint32_t>(S)) { stage -= static_cast<uint32_t>(S); phase ^= 1u; }
        }
        c -= p.nk;                               // blocks alternate over the units' ends
      }
      if (!ok) {
        *abort_flag = 1;
        atomicOr(p.err, ERR_TIMEOUT);
      }
      mma_commit_pair(drain_bar + 8u * slot, 1);
      const int zero = 0;
      mbar_wait(drain_bar + 8u * slot, 0, &zero, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp < 4) {
    // warp 3: no role, fewer registers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kRegsWg0Wide));
  } else {
    // --------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kRegsEpiWide));
    grid_dep_wait();
    const int q = warp & 3;                    // TMEM lane quarter
    const int g = (warp - 4) >> 2;             // vocabulary tile of the unit
    const uint32_t tlane = static_cast<uint32_t>(q * 32) << 16;
    uint32_t slot = 0, sph = 0;
    bool failed = false;
    for (int u = pair; u < p.units; u += n_pairs) {
      const int vt = u / p.n1;
      const int nw0 = (u - vt * p.n1) * 256 + half + q * 32;   // the warp's first row
      const int n = nw0 + lane;                        // this thread's row
      const int vb = vt * 256 + g * 128;               // its first column
      const bool live = nw0 < p.B && vb < p.V;
      // (rows and tiles that do not exist read another's scales)
      const float* xs = p.x_scale + static_cast<size_t>(min(n, p.B - 1)) * p.nk;
      const float* ws = p.w_scale + static_cast<size_t>(min(vb, p.V - 1) >> 7) * p.nk;
      float acc[8][16];
#pragma unroll
      for (int i = 0; i < 128; ++i) acc[i >> 4][i & 15] = 0.0f;
      float sx = xs[0], sw = ws[0];
      for (int c = 0; c < p.nk; ++c) {
        const float s = __fmul_rn(sx, sw);
        if (c + 1 < p.nk) {
          sx = xs[c + 1];
          sw = ws[c + 1];
        }
        const uint32_t cur = 2u * slot + g, cph = sph;
        if (++slot == 2u) { slot = 0; sph ^= 1u; }
        if (!failed && !mbar_wait(accf_bar(cur), cph, abort_flag, p.timeout_ns)) {
          failed = true;
          *abort_flag = 1;
        }
        if (failed) continue;
        tc_fence_after();
        auto add32 = [&](const uint32_t (&r)[32], int b) {
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            float* a = &acc[2 * b + (i >> 4)][i & 15];
            const float2 y = fma2_rn(make_float2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])),
                                     make_float2(s, s), make_float2(a[0], a[1]));
            a[0] = y.x;
            a[1] = y.y;
          }
        };
        const uint32_t at = tmem_base + tlane + cur * 128u;
        uint32_t ra[32], rb[32];
        if (live) {
          tmem_ld32(at, ra);
          tmem_ld32(at + 32, rb);
          tmem_wait_ld_of(ra);
          tmem_wait_ld_of(rb);
          add32(ra, 0);
          add32(rb, 1);
          tmem_ld32(at + 64, ra);
          tmem_ld32(at + 96, rb);
          tmem_wait_ld_of(ra);
          tmem_wait_ld_of(rb);
        }
        // the slot is read: back to the leader's MMA thread, before the sums
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive(acce_bar(cur));
          else mbar_arrive_remote(cluster_addr(acce_bar(cur), 0));
        }
        if (live) {
          add32(ra, 2);
          add32(rb, 3);
        }
      }
      if (__any_sync(0xffffffffu, failed || *abort_flag)) {
        *abort_flag = 1;
        if (lane == 0) atomicOr(p.err, ERR_TIMEOUT);
        break;
      }
      if (live) {
        Staging sg;
        sg.xs = smem + L.xs_off + (warp - 4) * kOpXsBytes;
        sg.xs_u32 = smem_u32(sg.xs);
        const OutRows out{p.out, p.B, p.V, p.type, p.tma};
        store_rows(out, &tmO, sg, lane, n, nw0, vb, min(128, p.V - vb),
                   [&](int j, float (&y)[4]) {
#pragma unroll
                     for (int i = 0; i < 4; ++i) y[i] = acc[(j + i) >> 4][(j + i) & 15];
                   });
      }
    }
    // the stores are complete before the CTA (and its shared memory) goes
    if (lane == 0) bulk_wait_group<0>();
    __syncwarp();
  }

  // neither CTA leaves (or frees its tensor memory) before the leader's MMAs
  // and both CTAs' remote arrivals are done
  tc_fence_before();
  cluster_sync();
  grid_dep_launch();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512u);
  }
}

}  // namespace detlm
