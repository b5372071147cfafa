// pairop_kernels.cuh -- the matrix products of the score call and of its
// gradient, on CTA pairs.
//
// One kernel body, nine products. A unit is a 256 x 256 tile of
// D = A * B^T, computed by a cluster of two CTAs with tcgen05.mma.cta_group::2
// (each CTA holds 128 rows of A and 128 of B per stage and finds its own 128
// rows of D in its tensor memory), with the pair protocol of
// rows_kernels.cuh: the leader issues every MMA, both producers' loads
// complete on the leader's stage barrier, commits arrive on both CTAs, a
// chunk's accumulator slot goes back when the epilogue warps of both CTAs have
// drained it, every wait is bounded.
//
//   OP_SCORE   D[n, v] = h W^T: softmax statistics of each row and 256-entry
//              tile, the target's logit, and the candidates for the row's
//              largest logits; logits are never written.
//   OP_SCOREZ  the same with the logits written to a workspace instead of
//              candidates (few rows, where the candidates' thresholds come too
//              late to thin them out).
//   OP_SELECT  OP_SCORE again, for the 256-row tiles that hold a row
//              whose candidates overflowed: only its candidates, with the
//              exact threshold found meanwhile.
//   OP_DZ      D[n, v] = h W^T again, turned into the gradient with respect
//              to the logits and written in 16 bits, but for the target's
//              entry, which goes to an fp32 word of the row.
//   OP_DH      D[n, k] = sum_v dz[n, v] W[v, k]: A = dz with the contracted
//              axis contiguous, B = W with the free axis contiguous.
//   OP_DW      D[v, k] = sum_n dz[n, v] h[n, k]: both operands with the free
//              axis contiguous. OP_DW_FEW: of at most kFewRows rows.
//   OP_SCALED  D[n, v] = q W^T of int8 values held as fp16, written times a
//              scale of the row and one of the column; OP_SCALED2 where d is
//              at most two chunks (no integer conversions: the rounded sum of
//              two exact integers is the rounding of their exact sum).
//
// The target's entry (g_l (1 - p) - ...) / T of the gradient never passes
// through 16 bits: it is mostly by far the largest of its row, and its rounding
// would be as large as that of the result (as it is where another token holds
// most of the row: the result's error is then up to sqrt(2) of its own rounding). dz holds a zero in its place; its fp32
// value contributes a row of W to dh and a row of h to dW, added in fp32
// (grad_fold_kernel, and this kernel's OP_DW epilogue).
//
// K chunks, each accumulated from zero in a tensor-memory slot and added in
// fp32 (round to nearest, ascending order) by the epilogue: 512 elements for
// the scores (kScoreChunkK); 2048 for the gradient's three products -- 128 MMA
// steps of the tensor core's accumulation, at most about 128 half-ulps of
// fp32 (8e-6) per chunk, far below the 16-bit rounding of dz and of what comes
// out; 1024 for OP_SCALED, whose chunk sums are integers of magnitude at most
// 1024 * 2^14 = 2^24, exact in fp32, added in int32. Longer chunks mean fewer
// drains of tensor memory, which at 128 elements take longer than the MMAs.
//
// Operands with the free axis contiguous ("MN-major") are loaded as boxes of
// 64 free x 64 contracted elements, 128-byte swizzle: 64 rows of 128 bytes,
// the rows running along the contracted axis. Eight rows make a 1024-byte
// atom (the descriptor's stride offset), the next 64 free elements start 8 KB
// on (its leading offset), and a K = 16 step is 16 rows = 2048 bytes.
//
// Why 256 x 256 on a pair: an SM then loads 64 KB of operands for every 128
// x 256 x 128 products, half of what one CTA with the same accumulator loads,
// and two 256-column slots fill the tensor memory, one drained while the other
// is multiplied into. A unit's statistics (5 instructions a logit) run while the
// MMA fills the slots with the next unit's first chunks, which hide them if they
// are long enough.
//
// What bounds them: for thousands of rows the tensor pipe and, on calls of
// milliseconds, the power limit under it: called again and again at 8192 x
// 151936 x 1536 the gradient's products run at 1.71 GHz of 2.07 (1.7 PFLOP/s,
// what a library product sustains), the int8 product of 2048 rows at 1.88, the
// score, whose drains leave the pipe idle longer, at 2.02. Of one launch, with
// cold caches, the pipe is active (2048 x 50176 x 1536 unless said otherwise):
//   OP_SCORE   K = 8, 212 us    63 %    OP_DZ      192 us    70 %
//   OP_DH      186 us           73 %    OP_DW      184 us    76 %
//   OP_SCALED  2048 x 32000 x 4096, 305 us         74 %
// the rest being the drains at a unit's end and the partial last round of
// units. With a few hundred rows the
// operands bound them (units share W tiles and hidden rows through L2, which
// delivers about 15.5 TB/s to the SMs): 301 x 50001 x 1000 scores in 58 us
// where the MMAs of its 512 padded rows need 27. Under 128 rows the gradient's
// products are streams: W read (OP_DZ, OP_DH) or dW written (OP_DW), 28 to 33
// us each at 48 x 32000 x 2048, 131 MB (20 us at the copy bandwidth).
#pragma once
#include "head_kernels.cuh"
#include "int8_kernels.cuh"
#include "rows_kernels.cuh"

namespace detlm {

enum : int { OP_SCORE = 0, OP_SCOREZ = 1, OP_SELECT = 2, OP_DZ = 3, OP_DH = 4, OP_DW = 5,
             OP_SCALED = 6, OP_SCALED2 = 7, OP_DW_FEW = 8 };
__host__ __device__ constexpr bool op_dw(int op) { return op == OP_DW || op == OP_DW_FEW; }
__host__ __device__ constexpr bool op_scaled(int op) { return op == OP_SCALED || op == OP_SCALED2; }

constexpr int kGradChunkBoxes = 32;      // 64-element K boxes per gradient chunk (2048)
constexpr int kScaledChunkBoxes = 16;    // OP_SCALED: 1024
constexpr int kSegChunks = 8;            // gradient chunks per vocabulary segment (16384)
constexpr int kCandFloats = 20;          // a candidate block: 16 logits, its index, padding
constexpr float kLowLogP = -1.0e4f;       // e^ of it is zero in fp32
constexpr int kFewRows = 128;            // OP_DW: rows whose targets a warp holds in registers
constexpr int kRowWords = 4;             // words of a row before its slots
enum : int { RW_COUNT = 0, RW_SEL_M = 1, RW_SEL_T = 2, RW_OVER = 3 };

// Two fp32 values rounded to bf16 or fp16, the first in the low half; and back.
__device__ __forceinline__ uint32_t pack16(float lo, float hi, bool fp16) {
  if (fp16) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
  }
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float2 unpack16(uint32_t w, bool fp16) {
  if (fp16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&w));
}

__host__ __device__ constexpr int row_words(int K) { return kRowWords + ((K + 3) & ~3); }

// MN-major operand tile in the 128-byte swizzle layout written by TMA as
// boxes of 64 (free) x 64 (contracted) 16-bit elements.
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t smem_addr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((smem_addr & 0x3FFFFu) >> 4);   // start address
  d |= static_cast<uint64_t>(8192 >> 4) << 16;               // next 64 free elements
  d |= static_cast<uint64_t>(1024 >> 4) << 32;               // next 8 contracted elements
  d |= static_cast<uint64_t>(1) << 46;                       // descriptor version
  d |= static_cast<uint64_t>(2) << 61;                       // 128-byte swizzle
  return d;
}
// Instruction descriptor bits: operand with the free axis contiguous.
constexpr uint32_t kIdescMnA = 1u << 15, kIdescMnB = 1u << 16;

struct ScoreArgs {
  float* rec;               // [3][rec_part]: m, S, U of each [B][n_vt] tile
  float* zt;                // [B] target logits
  const int32_t* targets;   // optional [B]
  int32_t* words;           // [B][row_words(K)]: candidate count, ..., K slot maxima
  float* cand;              // [B][C][kCandFloats]
  const int32_t* tile_over; // OP_SELECT: whether any tile is marked, then [n_rt] marks
};
struct GradArgs {
  const float* lse;         // [B]
  const float* entropy;     // [B]
  const float* dlogp;       // [B]
  const float* dentropy;    // optional [B]
  const int32_t* targets;   // [B], vocabulary index of the whole head
  const float* scale;       // optional: {power of two dz is held in, its inverse}
};

struct DwArgs {
  const int32_t* targets;   // OP_DW_FEW: [B] (and no runs)
  const int32_t* starts;    // [256 n_vt + 1] where a vocabulary entry's run in the list starts
  const float* sums;        // [list position][d]: the sum of the run that starts there
  const void* h;            // [B][d]
  const float* scale;       // as above
};
struct ScaledArgs {
  const float* x_scale;     // [B]
  const float* w_scale;     // [V]
  void* out;                // [B][V], for rows that the tensor map cannot store
  int32_t type, tma;        // OUT_*; 1: D leaves through the tensor map
};

// 128 bytes or less (see HeadParams).
struct PairOpParams {
  int32_t B, V;             // hidden rows; vocabulary entries (of this pass)
  int32_t n0, n1;           // unit grid (see unit_of)
  int32_t nk;               // K boxes of 64
  int32_t seg;              // K boxes per unit (OP_DH; else nk)
  int32_t units;
  uint8_t stages, stall, a_rows, pad; // a_rows: rows of A's box (K-major A; 128 or fewer)
  uint32_t idesc;
  int32_t K, C;             // score: alternatives wanted, candidate blocks a row can hold;
                            // OP_DH, OP_DW: K is the number of columns of D (d);
                            // OP_DZ: K is the whole head's V
  int32_t t_off;            // gradient: vocabulary index of this pass's first entry
  float c, inv_t;           // score: log2(e) / T; 1 / T
  union {
    int64_t rec_part;       // score: elements between the record arrays
    float* coef;            // OP_DZ: [B] out, OP_DW: in: the target's entry of dz (as scaled)
  };
  uint64_t timeout_ns;
  int* err;
  union {
    ScoreArgs s;
    GradArgs g;
    DwArgs w;
    ScaledArgs q;
  };
};
static_assert(sizeof(PairOpParams) <= 128, "kernel parameter struct above 128 bytes");

// Origins of unit u in the operands: 256 rows of A from a0, 256 of B from b0,
// nkb K boxes from kb0.
//   OP_SCORE, OP_SELECT, OP_DZ: n1 hidden-row tiles, fastest (they share each
//     W tile from L2)
//   OP_DH: n1 tiles of d, fastest, then n0 hidden-row tiles, then segments, the
//     last one first: OP_DZ has left the end of W and of dz in L2 (777 x 50001
//     x 1000: gradient 245.6 -> 240.6 us; 48 x 32000 x 2048: 99.4 -> 96.8;
//     W's loads marked evict-last, without it no gain there)
//   OP_DW: n1 tiles of d, fastest, then vocabulary tiles
struct PairUnit { int a0, b0, kb0, nkb, seg; };

// The units of one pair: u = pair, pair + n_pairs, ..., as (q, r) = (u / n1,
// u % n1) without a division per unit.
struct UnitWalk {
  int u, q, r, du, dq, dr, n1;
  __device__ __forceinline__ UnitWalk(int pair, int n_pairs, int n1_)
      : u(pair), q(pair / n1_), r(pair - (pair / n1_) * n1_), du(n_pairs), dq(n_pairs / n1_),
        dr(n_pairs - (n_pairs / n1_) * n1_), n1(n1_) {}
  __device__ __forceinline__ void next() {
    u += du;
    q += dq;
    r += dr;
    if (r >= n1) {
      r -= n1;
      ++q;
    }
  }
};

template <int OP>
__device__ __forceinline__ PairUnit unit_of(const PairOpParams& p, const UnitWalk& w) {
  PairUnit t;
  t.kb0 = 0;
  t.nkb = p.nk;
  t.seg = 0;
  if constexpr (OP == OP_DH) {
    const int q = w.q / p.n0;
    t.seg = (p.nk - 1) / p.seg - q;
    t.a0 = (w.q - q * p.n0) * 256;
    t.b0 = w.r * 256;
    t.kb0 = t.seg * p.seg;
    t.nkb = min(p.seg, p.nk - t.kb0);
  } else if constexpr (op_dw(OP)) {
    t.a0 = w.q * 256;
    t.b0 = w.r * 256;
  } else {
    t.a0 = w.r * 256;
    t.b0 = w.q * 256;
  }
  return t;
}

// Staging of D: per epilogue warp two buffers of 32 rows x 128 bytes (whole
// cache lines leave; 128-byte swizzle: 16-byte chunk c of row r sits at chunk
// c ^ (r & 7)), each stored by the tensor map's box while the warp goes on.
// (Four buffers and fewer stages measured the same on the shortest K loops.)
constexpr uint32_t kOpStageBuf = 32 * 128;
constexpr uint32_t kOpXsBytes = 2 * kOpStageBuf;
// registers: the producer and the MMA issuer walk the units, which 40 (the
// other pair kernels' share) do not hold
constexpr int kOpRegsWg0 = 56, kOpRegsEpi = 224;
static_assert(128 * kOpRegsWg0 + 256 * kOpRegsEpi == 384 * kRegsLaunchWide,
              "register split must equal the launch budget");
constexpr int kOpMaxStages = 12;

__host__ __device__ constexpr bool op_stores(int op) { return op != OP_SCORE && op != OP_SELECT; }
// Words kept beside the stages: the half-row records [3][128] of the score
// products, each epilogue warp's column scales [8][128] of OP_SCALED.
__host__ __device__ constexpr uint32_t op_words(int op) {
  return op == OP_SCORE || op == OP_SCOREZ ? 384u : op_scaled(op) ? 1024u : 0u;
}

struct OpLayout {
  uint32_t a_bytes, stage_bytes, ctrl_off, red_off, xs_off, total;
};
// Stage s: this CTA's rows of A (128, or as many as its box has), then its 128
// rows of B (128 bytes of K each, or two MN-major boxes of 8 KB each); then
// the barriers (full[S], empty[S],
// slot_full[2], slot_empty[2], never, drain), the TMEM address holder and the
// abort flag; the op's words; the staging buffers.
__host__ __device__ inline OpLayout op_layout(int op, int stages, int a_rows) {
  OpLayout L;
  L.a_bytes = static_cast<uint32_t>(a_rows) * kRowBytes;
  L.stage_bytes = L.a_bytes + kRowsHalf * kRowBytes;
  L.ctrl_off = static_cast<uint32_t>(stages) * L.stage_bytes;
  L.red_off = L.ctrl_off + (2u * stages + 6u) * 8u + 16u;
  L.xs_off = L.red_off + 4u * op_words(op);
  if (op_stores(op)) L.xs_off = (L.xs_off + 1023u) & ~1023u;
  L.total = L.xs_off + (op_stores(op) ? 8u * kOpXsBytes : 0u);
  return L;
}

// A warp's two staging buffers.
struct Staging {
  uint8_t* xs;
  uint32_t xs_u32;
  // both buffers may be written: their previous stores have read them
  __device__ __forceinline__ void claim(int lane) {
    if (lane == 0) bulk_wait_group_read<0>();
    __syncwarp();
  }
  // 32 rows x 128 bytes (lane = row) into buffer b
  __device__ __forceinline__ void put(int b, const uint4 (&w)[8], int lane) {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      *reinterpret_cast<uint4*>(xs + b * kOpStageBuf + lane * 128 + 16 * (k ^ (lane & 7))) = w[k];
  }
  // out to the tensor map's boxes at (c0, row0) and, where two, (c1, row0);
  // asynchronous
  __device__ __forceinline__ void store(const void* tmap, int lane, int c0, int c1, bool two, int row0) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) {
      tma_store_2d(tmap, xs_u32, c0, row0);
      if (two) tma_store_2d(tmap, xs_u32 + kOpStageBuf, c1, row0);
      bulk_commit_group();
    }
  }
};

// 128 fp32 columns of a warp's rows through the staging buffers: columns c0
// on, `cols` of them in the tensor.
__device__ __forceinline__ void store_f32(const float (&acc)[8][16], Staging& sg, const void* tmap,
                                          int lane, int c0, int cols, int row0) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (c0 + 64 * h >= cols) break;
    sg.claim(lane);
#pragma unroll
    for (int b = 0; b < 2; ++b) {
      uint4 w[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float* x = &acc[4 * h + 2 * b + (k >> 2)][4 * (k & 3)];
        w[k] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
      }
      sg.put(b, w, lane);
    }
    sg.store(tmap, lane, c0 + 64 * h, c0 + 64 * h + 32, c0 + 64 * h + 32 < cols, row0);
  }
}

// The score call's epilogue of one half-unit: this thread's row n, 128
// entries from vb (nv of them exist).
//
// Candidates. The row keeps K slots; slot j holds the largest logit of the
// 32-entry groups j, j + K, ... seen so far, so K different entries are at
// least as large as the smallest slot: that value is a threshold no entry
// below which can be among the K largest, however many CTAs add to it and
// however late a reader sees it. Every 16-entry block that reaches the
// threshold is appended whole to the row's list (its place there depends on
// timing, the set of entries above the final threshold does not). About
// K H_K entries stay above the final threshold (H_K the harmonic number), so
// of V / 16 blocks some K H_K log(n_vt) are appended.
template <bool RAGGED, bool CAND>
__device__ __forceinline__ Stat score_tail(const PairOpParams& p, const float (&acc)[8][16], int n,
                                           int vb, int nv, float thr, bool records) {
  float bm[8];
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    bm[b] = -INFINITY;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (!RAGGED || b * 16 + i < nv) bm[b] = fmaxf(bm[b], acc[b][i]);
  }
  uint32_t mask = 0;
  int base = 0;
  int32_t* w = nullptr;
  if constexpr (CAND) w = p.s.words + static_cast<size_t>(n) * row_words(p.K);
  if (CAND && p.K > 0) {
#pragma unroll
    for (int b = 0; b < 8; ++b)
      if (bm[b] >= thr && (!RAGGED || b * 16 < nv)) mask |= 1u << b;
    if (mask != 0) {
      base = atomicAdd(&w[RW_COUNT], __popc(mask));
      if (records) {
        int slot = (vb >> 5) % p.K;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float gm = fmaxf(bm[2 * j], bm[2 * j + 1]);
          if (gm >= thr && (!RAGGED || j * 32 < nv))
            atomicMax(reinterpret_cast<uint32_t*>(w + kRowWords + slot), score_key(gm));
          if (++slot == p.K) slot = 0;
        }
      }
    }
  }
  Stat st{-INFINITY, 0.0f, 0.0f};
  if (records) {
    Stat g[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (RAGGED && j * 32 >= nv) {
        g[j] = Stat{-INFINITY, 0.0f, 0.0f};
      } else {
        g[j] = stat32<RAGGED>(acc[2 * j], acc[2 * j + 1], fmaxf(bm[2 * j], bm[2 * j + 1]), p.c,
                              nv - j * 32);
      }
    }
    st = stat_merge(stat_merge(g[0], g[1], p.c), stat_merge(g[2], g[3], p.c), p.c);
  }
  if (CAND && mask != 0) {
    float* cd = p.s.cand + static_cast<size_t>(n) * p.C * kCandFloats;
#pragma unroll
    for (int b = 0; b < 8; ++b) {
      if (!(mask & (1u << b))) continue;
      if (base < p.C) {
        float* o = cd + static_cast<size_t>(base) * kCandFloats;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float4 v = make_float4(acc[b][4 * k], acc[b][4 * k + 1], acc[b][4 * k + 2],
                                 acc[b][4 * k + 3]);
          reinterpret_cast<float4*>(o)[k] = v;
        }
        o[16] = __int_as_float((vb >> 4) + b);
      }
      ++base;
    }
  }
  return st;
}

// OP_DW_FEW: acc += g h[n][col0 ..], 128 columns or up to d (a multiple of 8).
__device__ __forceinline__ void add_row(const PairOpParams& p, float (&acc)[8][16], int n, float g,
                                        int col0, bool f16) {
  const uint4* h = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p.w.h) +
                                                  static_cast<size_t>(n) * p.K + col0);
#pragma unroll
  for (int b = 0; b < 16; ++b) {
    if (col0 + 8 * b >= p.K) break;
    const uint4 w = __ldg(h + b);
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = unpack16(x[k], f16);
      float* a = &acc[b >> 1][(b & 1) * 8 + 2 * k];
      a[0] = fmaf(g, v.x, a[0]);
      a[1] = fmaf(g, v.y, a[1]);
    }
  }
}

// OP_DW: the targets' entries of the warp's 32 vocabulary rows. The hidden rows
// of one target have been summed (target_sum_kernel: coef_n h[n], ascending,
// so a frequent token costs no thread a walk); `first` is the sum of this
// lane's row, or -1. The warp fetches the sums row by row, through the staging
// buffers (16 rows of 512 bytes, 16-byte chunks swizzled by the row), and
// every lane adds its own.
__device__ __forceinline__ void add_targets(const PairOpParams& p, float (&acc)[8][16], Staging& sg,
                                            int first, int col0, int lane) {
  const uint32_t hits = __ballot_sync(0xffffffffu, first >= 0);
  if (hits == 0) return;
  const bool in = col0 + 4 * lane < p.K;       // d is a multiple of 8
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    uint32_t left = (hits >> (16 * h)) & 0xFFFFu;
    if (left == 0) continue;
    sg.claim(lane);                            // (a warp barrier: earlier reads are done)
    while (left != 0) {
      float4 x[4];
      int row[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        row[j] = left != 0 ? __ffs(left) - 1 : -1;
        left &= left - 1;
        const int f = __shfl_sync(0xffffffffu, first, 16 * h + (row[j] & 15));
        if (row[j] >= 0 && in)
          x[j] = __ldg(reinterpret_cast<const float4*>(p.w.sums + static_cast<size_t>(f) * p.K + col0) +
                       lane);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (row[j] >= 0 && in)
          *reinterpret_cast<float4*>(sg.xs + row[j] * 512 + 16 * (lane ^ (row[j] & 7))) = x[j];
    }
    __syncwarp();
    if ((lane >> 4) == h && first >= 0) {
      const int r = lane & 15;
#pragma unroll
      for (int b = 0; b < 32; ++b) {
        if (col0 + 4 * b >= p.K) break;
        const float4 v = *reinterpret_cast<const float4*>(sg.xs + r * 512 + 16 * (b ^ (r & 7)));
        float* a = &acc[b >> 2][4 * (b & 3)];
        a[0] += v.x;
        a[1] += v.y;
        a[2] += v.z;
        a[3] += v.w;
      }
    }
    __syncwarp();
  }
}

// OP_SCALED: this thread's row n, columns vb .. (lim of them exist): the exact
// int32 sum rounded once to fp32, one rounded product of the two scales, one
// rounded product, and the output's own rounding. Rows that do not start on
// 16-byte boundaries are written from the staging buffer one row at a time, a
// 4-byte word a lane: 16-bit rows of odd origin pair elements (2 l - 1, 2 l).
// acc: the int32 sums, or (OP_SCALED2) the fp32 integers that the tensor core
// left; sw: the warp's 128 column scales in shared memory.
template <typename Acc>
__device__ __forceinline__ void scaled_tail(const PairOpParams& p, const void* tmO,
                                            const Acc (&acc)[8][16], const float* sw, Staging& sg,
                                            int lane, int n, int nw0, int vb, int lim) {
  const int type = p.q.type;
  const float sx = n < p.B ? p.q.x_scale[n] : 0.0f;
  const int rows = min(32, p.B - nw0);
  // fp32 rows that the tensor map cannot store: 32 columns of a row at a time
  auto rows32 = [&](uint32_t off, int c0) {
    const uint8_t* sb = sg.xs + off;
    float* out = static_cast<float*>(p.q.out) + static_cast<size_t>(nw0) * p.V + c0 + lane;
    if (c0 + lane < p.V) {
#pragma unroll 8
      for (int r = 0; r < rows; ++r)
        out[static_cast<size_t>(r) * p.V] = *reinterpret_cast<const float*>(
            sb + r * 128 + 16 * ((lane >> 2) ^ (r & 7)) + 4 * (lane & 3));
    }
  };
  // 16-bit rows that it cannot store. Their owners have staged them as 4-byte
  // words of the row's own alignment (rows at odd elements: elements 2 k - 1
  // and 2 k in word k), so a warp writes a row's words 32 at a time; what
  // shares a word with a neighbour goes element by element.
  auto rows16 = [&]() {
    const uint8_t* sb = sg.xs + 4 * (lane & 3);
    uint16_t* o = static_cast<uint16_t*>(p.q.out) + static_cast<size_t>(nw0) * p.V + vb;
    if (lim >= 128) {
#pragma unroll 4
      for (int r = 0; r < rows; ++r, o += p.V) {
        const uint32_t at = r * 128 + 16 * ((lane >> 2) ^ (r & 7));
        const uint32_t w0 = *reinterpret_cast<const uint32_t*>(sb + at);
        const uint32_t w1 = *reinterpret_cast<const uint32_t*>(sb + kOpStageBuf + at);
        const int odd = static_cast<int>((reinterpret_cast<uintptr_t>(o) >> 1) & 1);
        uint32_t* x = reinterpret_cast<uint32_t*>(o - odd) + lane;
        if (odd && lane == 0) o[0] = static_cast<uint16_t>(w0 >> 16);
        else x[0] = w0;
        x[32] = w1;
      }
    } else {
      for (int r = 0; r < rows; ++r, o += p.V) {
        const int odd = static_cast<int>((reinterpret_cast<uintptr_t>(o) >> 1) & 1);
        for (int e = lane; e < lim; e += 32) {
          const int k = (e + odd) >> 1;
          o[e] = *reinterpret_cast<const uint16_t*>(sg.xs + (k >> 5) * kOpStageBuf + r * 128 +
                                                    16 * (((k >> 2) & 7) ^ (r & 7)) + 4 * (k & 3) +
                                                    2 * ((e + odd) & 1));
        }
      }
    }
  };
  // columns j .. j + 3
  auto values = [&](int j, float (&y)[4]) {
    const float4 w = *reinterpret_cast<const float4*>(sw + j);
    const float s[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i] = __fmul_rn(static_cast<float>(acc[(j + i) >> 4][(j + i) & 15]), __fmul_rn(sx, s[i]));
    }
  };
  uint4 w[8];
  float x[4], y[4];
  if (type == OUT_F32) {
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      if (32 * b >= lim) break;
      if ((b & 1) == 0) sg.claim(lane);        // (and the previous rows' reads are done)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        values(32 * b + 4 * k, x);
        w[k] = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                          __float_as_uint(x[3]));
      }
      sg.put(b & 1, w, lane);
      const bool more = (b & 1) == 0 && 32 * (b + 1) < lim;   // the pair's second box follows
      if (more) continue;
      const int c0 = vb + 32 * (b & ~1);
      if (p.q.tma) {
        sg.store(tmO, lane, c0, c0 + 32, (b & 1) != 0, nw0);
      } else {
        __syncwarp();
        rows32(0, c0);
        if ((b & 1) != 0) rows32(kOpStageBuf, c0 + 32);
      }
    }
  } else {
    const bool f16 = type == OUT_FP16;
    // this row's origin is an odd element (and not the tensor map's to store)
    uint16_t* mine = static_cast<uint16_t*>(p.q.out) + static_cast<size_t>(n) * p.V + vb;
    const uint32_t shift =
        !p.q.tma ? static_cast<uint32_t>((reinterpret_cast<uintptr_t>(mine) >> 1) & 1) * 16u : 0u;
    uint32_t last = 0;
    sg.claim(lane);                            // (and the previous rows' reads are done)
#pragma unroll
    for (int b = 0; b < 2; ++b) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        values(64 * b + 8 * k, x);
        values(64 * b + 8 * k + 4, y);
        const uint32_t e[4] = {pack16(x[0], x[1], f16), pack16(x[2], x[3], f16),
                               pack16(y[0], y[1], f16), pack16(y[2], y[3], f16)};
        w[k] = make_uint4(__funnelshift_l(last, e[0], shift), __funnelshift_l(e[0], e[1], shift),
                          __funnelshift_l(e[1], e[2], shift), __funnelshift_l(e[2], e[3], shift));
        last = e[3];
      }
      sg.put(b, w, lane);
    }
    if (p.q.tma) {
      sg.store(tmO, lane, vb, vb + 64, lim > 64, nw0);
    } else {
      // (the 128th element of a shifted row has no word)
      if (shift != 0 && lim >= 128 && n < p.B) mine[127] = static_cast<uint16_t>(last >> 16);
      __syncwarp();
      rows16();
    }
  }
}

template <int OP>
__global__ void __launch_bounds__(kRowsThreads, 1)
pairop_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmO, const PairOpParams p) {
  constexpr bool kScore = OP == OP_SCORE || OP == OP_SCOREZ || OP == OP_SELECT;
  constexpr bool kLogits = kScore || OP == OP_DZ || op_scaled(OP);     // D = h W^T
  constexpr bool kStore = op_stores(OP);               // D leaves through staging and tmO
  constexpr bool kInt = OP == OP_SCALED;               // integer sums, int32
  constexpr bool kMnA = op_dw(OP), kMnB = OP == OP_DH || op_dw(OP);
  constexpr int kBoxes = kScore ? kScoreChunkK / 64 : op_scaled(OP) ? kScaledChunkBoxes : kGradChunkBoxes;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int S = p.stages;
  const OpLayout L = op_layout(OP, S, p.a_rows);
  const uint32_t rank = cluster_rank();            // 0: leader, 1: peer
  const int pair = static_cast<int>(blockIdx.x >> 1);
  const int n_pairs = static_cast<int>(gridDim.x >> 1);

  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.ctrl_off);
  const uint32_t bar0 = smem_u32(bars);
  auto full_bar = [&](int s) { return bar0 + 8u * s; };
  auto empty_bar = [&](int s) { return bar0 + 8u * (S + s); };
  auto accf_bar = [&](int b) { return bar0 + 8u * (2 * S + b); };
  auto acce_bar = [&](int b) { return bar0 + 8u * (2 * S + 2 + b); };
  const uint32_t never_bar = bar0 + 8u * (2 * S + 4);
  const uint32_t drain_bar = bar0 + 8u * (2 * S + 5);
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + L.ctrl_off + (2 * S + 6) * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  const uint32_t smem_base = smem_u32(smem);
  auto sA = [&](int s) { return smem_base + static_cast<uint32_t>(s) * L.stage_bytes; };
  auto sB = [&](int s) { return sA(s) + L.a_bytes; };

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(full_bar(s), 1);       // the leader's arrival (+ both CTAs' loads)
      mbar_init(empty_bar(s), 1);      // the leader's MMA commit
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(accf_bar(b), 1);       // the leader's MMA commit
      mbar_init(acce_bar(b), 16);      // eight epilogue warps of each CTA
    }
    mbar_init(never_bar, 1);
    mbar_init(drain_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    tma_prefetch_desc(&tmA);
    tma_prefetch_desc(&tmB);
    if (kStore) tma_prefetch_desc(&tmO);
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
  // OP_SELECT computes the units of the marked hidden-row tiles alone (the
  // marks are the previous kernel's, read after the wait by every role)
  auto skip = [&](const UnitWalk& w) {
    if constexpr (OP == OP_SELECT) return p.s.tile_over[1 + w.r] == 0;
    return false;
  };
  const UnitWalk first(pair, n_pairs, p.n1);
  int units = p.units;
  if constexpr (OP == OP_SELECT) {
    grid_dep_wait();
    if (p.s.tile_over[0] == 0) units = 0;   // the usual case: no row overflowed
  }

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOpRegsWg0));
    if (lane == 0) {
      const uint64_t pol_n = policy_evict_normal();
      const uint64_t pol_l = policy_evict_last();
      const bool leader = rank == 0;
      auto load_a = [&](int s, const PairUnit& t, int kb, uint32_t fb) {
        if constexpr (kMnA) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            tma_load_2d_pair(sA(s) + i * 8192, &tmA, t.a0 + half + i * 64, kb * 64, fb, pol_n);
        } else if (t.a0 + half < p.B) {
          tma_load_2d_pair(sA(s), &tmA, kb * 64, t.a0 + half, fb, kLogits ? pol_l : pol_n);
        }
      };
      // bytes of a stage over both CTAs: boxes of rows that do not exist are
      // not loaded (their rows of D are not read)
      auto bytes = [&](const PairUnit& t) {
        if constexpr (kMnA) return 2u * L.stage_bytes;
        return 2u * kRowsHalf * kRowBytes + (t.a0 + kRowsHalf < p.B ? 2u : 1u) * L.a_bytes;
      };
      auto load_b = [&](int s, const PairUnit& t, int kb, uint32_t fb) {
        if constexpr (kMnB) {
#pragma unroll
          for (int i = 0; i < 2; ++i)
            tma_load_2d_pair(sB(s) + i * 8192, &tmB, t.b0 + half + i * 64, kb * 64, fb, pol_l);
        } else {
          tma_load_2d_pair(sB(s), &tmB, kb * 64, t.b0 + half, fb, pol_n);
        }
      };
      // unlike the other projections, no W box is requested before the wait:
      // a trainer updates W on the stream between calls
      grid_dep_wait();
      uint32_t stage = 0, phase = 0, outstanding = 0, out_par = 0;
      bool ok = true;
      for (UnitWalk w = first; w.u < units && ok; w.next()) {
        if (skip(w)) continue;
        const PairUnit t = unit_of<OP>(p, w);
        for (int kb = t.kb0; kb < t.kb0 + t.nkb; ++kb) {
          const uint32_t fb = cluster_addr(full_bar(stage), 0);
          if (!mbar_wait(empty_bar(stage), phase ^ 1u, abort_flag, p.timeout_ns)) { ok = false; break; }
          if (leader) mbar_arrive_expect_tx(full_bar(stage), bytes(t));
          load_b(stage, t, kb, fb);
          load_a(stage, t, kb, fb);
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
  } else if (warp == 1) {
    // ------------------------------------------------------- MMA issuer
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOpRegsWg0));
    if (lane == 0 && rank == 0) {
      uint32_t stage = 0, phase = 0, slot = 0, sph = 0;
      bool ok = true;
      if (p.stall) ok = mbar_wait(never_bar, 0, abort_flag, p.timeout_ns);
      for (UnitWalk w = first; w.u < units && ok; w.next()) {
        if (skip(w)) continue;
        const int nkb = unit_of<OP>(p, w).nkb;
        for (int c0 = 0; c0 < nkb && ok; c0 += kBoxes) {
          if (!mbar_wait(acce_bar(slot), sph ^ 1u, abort_flag, p.timeout_ns)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d_tmem = tmem_base + slot * 256u;
          const int nb = min(kBoxes, nkb - c0);
#pragma unroll 1
          for (int sc = 0; sc < kBoxes; ++sc) {
            if (sc >= nb) break;
            if (!mbar_wait(full_bar(stage), phase, abort_flag, p.timeout_ns)) { ok = false; break; }
            tc_fence_after();
            const uint64_t da = kMnA ? sdesc_mn_sw128(sA(stage)) : sdesc_sw128(sA(stage));
            const uint64_t db = kMnB ? sdesc_mn_sw128(sB(stage)) : sdesc_sw128(sB(stage));
            constexpr uint32_t ka = kMnA ? 128u : 2u, kb = kMnB ? 128u : 2u;   // K = 16 step, 16 B units
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_f16_pair(d_tmem, da + ka * k, db + kb * k, p.idesc, !(sc == 0 && k == 0));
            mma_commit_pair(empty_bar(stage), 3);
            if (++stage == static_cast<uint32_t>(S)) { stage = 0; phase ^= 1u; }
          }
          if (!ok) break;
          mma_commit_pair(accf_bar(slot), 3);
          if (++slot == 2u) { slot = 0; sph ^= 1u; }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        atomicOr(p.err, ERR_TIMEOUT);
      }
      mma_commit_pair(drain_bar, 1);
      const int zero = 0;
      mbar_wait(drain_bar, 0, &zero, p.timeout_ns);
    }
    __syncwarp();
  } else if (warp < 4) {
    // warps 2 and 3: no role, fewer registers
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" :: "n"(kOpRegsWg0));
  } else {
    // --------------------------------------------------------- epilogue
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" :: "n"(kOpRegsEpi));
    grid_dep_wait();          // outputs and records: only after the previous kernels
    const int q = warp & 3;                    // TMEM lane quarter
    const int g = (warp - 4) >> 2;             // column half of the unit
    const int r = q * 32 + lane;               // row within this CTA's half
    const uint32_t tlane = static_cast<uint32_t>(q * 32) << 16;
    Staging sg;
    sg.xs = smem + L.xs_off + (warp - 4) * kOpXsBytes;
    sg.xs_u32 = smem_u32(sg.xs);
    float* red = reinterpret_cast<float*>(smem + L.red_off);  // the op's words
    using Acc = typename std::conditional<kInt, int32_t, float>::type;
    uint32_t slot = 0, sph = 0;
    bool failed = false;
    // OP_DW_FEW: lane l of every warp holds the targets of rows l, l + 32, ...
    int few[kFewRows / 32];
    if constexpr (OP == OP_DW_FEW) {
#pragma unroll
      for (int k = 0; k < kFewRows / 32; ++k) {
        few[k] = -1;
        if (32 * k + lane < p.B) {
          const int v = p.w.targets[32 * k + lane];
          if (v >= p.t_off && v - p.t_off < p.V) few[k] = v - p.t_off;
        }
      }
    }
    for (UnitWalk walk = first; walk.u < units; walk.next()) {
      if (skip(walk)) continue;
      const PairUnit t = unit_of<OP>(p, walk);
      const int nw0 = t.a0 + half + q * 32;    // the warp's first row of D
      const int n = nw0 + lane;                // this thread's row
      const int rows = op_dw(OP) ? p.V : p.B;
      const int vb = t.b0 + g * 128;           // first column of this half
      Acc acc[8][16];
      float thr = -INFINITY;
      if constexpr (op_scaled(OP)) {
        // the unit's column scales, for the warp's own tail
        float* sw = red + (warp - 4) * 128;
        __syncwarp();                          // the previous tail's reads are done
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int v = vb + 32 * k + lane;
          sw[32 * k + lane] = v < p.V ? __ldg(p.q.w_scale + v) : 0.0f;
        }
        __syncwarp();
      }
      int run0 = 0, run1 = 0;                  // OP_DW: this row's run in the list
      if constexpr (OP == OP_DW) {
        run0 = p.w.starts[n];
        run1 = p.w.starts[n + 1];
      }
      const int n_chunks = (t.nkb + kBoxes - 1) / kBoxes;
      for (int c = 0; c < n_chunks; ++c) {
        const uint32_t cur = slot, cph = sph;
        if (++slot == 2u) { slot = 0; sph ^= 1u; }
        if (!failed && !mbar_wait(accf_bar(cur), cph, abort_flag, p.timeout_ns)) {
          failed = true;
          *abort_flag = 1;
        }
        if (failed) continue;
        tc_fence_after();
        if (nw0 < rows) {
          const uint32_t sbase = tmem_base + tlane + cur * 256u + static_cast<uint32_t>(g * 128);
          // two groups of two 32-column loads, one wait each
#pragma unroll
          for (int h4 = 0; h4 < 2; ++h4) {
            uint32_t rw[2][32];
#pragma unroll
            for (int b2 = 0; b2 < 2; ++b2) tmem_ld32(sbase + (h4 * 2 + b2) * 32, rw[b2]);
            tmem_wait_ld();
#pragma unroll
            for (int b4 = 0; b4 < 4; ++b4) {
              const int bb = h4 * 4 + b4;
              const uint32_t* rr = &rw[b4 >> 1][(b4 & 1) * 16];   // this block's 16 columns
              if constexpr (kInt) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                  const int32_t x = __float2int_rn(__uint_as_float(rr[i]));
                  acc[bb][i] = c == 0 ? x : acc[bb][i] + x;
                }
              } else if (c == 0) {
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[bb][i] = __uint_as_float(rr[i]);
              } else {
#pragma unroll
                for (int i = 0; i < 16; i += 2)
                  add2_rn(acc[bb][i], acc[bb][i + 1], __uint_as_float(rr[i]),
                          __uint_as_float(rr[i + 1]));
              }
            }
          }
        }
        tc_fence_before();   // slot fully read: hand it back to the leader's MMA warp
        __syncwarp();
        if (lane == 0) {
          if (rank == 0) mbar_arrive(acce_bar(cur));
          else mbar_arrive_remote(cluster_addr(acce_bar(cur), 0));
        }
        if constexpr (OP == OP_SCORE) {
          // the row's threshold as of now: read here, where the epilogue
          // waits for the tensor core anyway
          if (c == (n_chunks >> 1) && p.K > 0 && n < p.B) {
            const uint4* sl = reinterpret_cast<const uint4*>(
                p.s.words + static_cast<size_t>(n) * row_words(p.K) + kRowWords);
            uint32_t lo = 0xFFFFFFFFu;
            for (int k = 0; k < p.K; k += 4) {
              const uint4 v = __ldcg(sl + (k >> 2));
              lo = min(lo, v.x);
              if (k + 1 < p.K) lo = min(lo, v.y);
              if (k + 2 < p.K) lo = min(lo, v.z);
              if (k + 3 < p.K) lo = min(lo, v.w);
            }
            thr = score_unkey(lo);
          }
        }
      }
      if constexpr (kScore) {
        if (epi_bar_or<256>(failed || *abort_flag)) {
          if (threadIdx.x == 128) { *abort_flag = 1; atomicOr(p.err, ERR_TIMEOUT); }
          break;
        }
      } else if (__any_sync(0xffffffffu, failed || *abort_flag)) {
        // (the other products' warps share nothing: no barrier)
        *abort_flag = 1;
        if (lane == 0) atomicOr(p.err, ERR_TIMEOUT);
        break;
      }
      if constexpr (kScore) {
        const int vt = t.b0 >> 8;
        const int n_vt = p.units / p.n1;
        const int nv = min(128, p.V - vb);      // valid entries in this half (<= 0: none)
        const bool row_ok = n < p.B;
        const size_t o = static_cast<size_t>(n) * n_vt + vt;   // records [B][n_vt]
        Stat st{-INFINITY, 0.0f, 0.0f};
        if constexpr (OP == OP_SCORE || OP == OP_SCOREZ) {
          if constexpr (OP == OP_SCOREZ) {
            if (nw0 < p.B) store_f32(acc, sg, &tmO, lane, vb, p.V, nw0);
          }
          if (row_ok && nv > 0) {
            // the target's logit, if it lies in this half: a select chain
            // over the 16-entry blocks, then over the block
            // (OP_SCOREZ: the merge reads it from the logits)
            const int tl = OP == OP_SCORE && p.s.targets != nullptr ? p.s.targets[n] - vb : -1;
            if (tl >= 0 && tl < 128) {
              const int tb = tl >> 4, ti = tl & 15;
              float sel[16];
#pragma unroll
              for (int i = 0; i < 16; ++i) sel[i] = acc[0][i];
#pragma unroll
              for (int bb = 1; bb < 8; ++bb)
#pragma unroll
                for (int i = 0; i < 16; ++i) sel[i] = bb == tb ? acc[bb][i] : sel[i];
              float z = sel[0];
#pragma unroll
              for (int i = 1; i < 16; ++i) z = i == ti ? sel[i] : z;
              p.s.zt[n] = z;
            }
            constexpr bool cand = OP == OP_SCORE;
            st = nv == 128 ? score_tail<false, cand>(p, acc, n, vb, nv, thr, true)
                           : score_tail<true, cand>(p, acc, n, vb, nv, thr, true);
          }
          // the two halves of a row: the second hands its record to the first
          if (g == 1) {
            red[r] = st.m;
            red[128 + r] = st.S;
            red[256 + r] = st.U;
          }
          named_bar_sync(1, 256);
          if (g == 0 && row_ok) {
            const Stat tot = stat_merge(st, Stat{red[r], red[128 + r], red[256 + r]}, p.c);
            p.s.rec[o] = tot.m;
            p.s.rec[p.rec_part + o] = tot.S;
            p.s.rec[2 * p.rec_part + o] = tot.U;
          }
          named_bar_sync(1, 256);
        } else {
          if (row_ok && nv > 0) {
            // only tiles among the row's K best, by (maximum, lowest index)
            const int32_t* w = p.s.words + static_cast<size_t>(n) * row_words(p.K);
            const float sm = __int_as_float(w[RW_SEL_M]);
            const float m = p.s.rec[o];
            if (w[RW_OVER] != 0 && (m > sm || (m == sm && vt <= w[RW_SEL_T]))) {
              if (nv == 128) score_tail<false, true>(p, acc, n, vb, nv, sm, false);
              else score_tail<true, true>(p, acc, n, vb, nv, sm, false);
            }
          }
        }
      } else if constexpr (op_scaled(OP)) {
        if (vb < p.V && nw0 < p.B) {
          scaled_tail(p, &tmO, acc, red + (warp - 4) * 128, sg, lane, n, nw0, vb, min(128, p.V - vb));
        }
      } else if constexpr (OP == OP_DZ) {
        // dz - (1/T) g_l 1[v = t] = -(1/T) p (g_l + g_H (log p + H)), written
        // as p (a1 log p + a0) with the row's own a1, a0. log p = z/T - lse is
        // one rounding of the difference itself: a rounded lse log2(e), or H -
        // lse, would leave the size of the logits in it. Below kLowLogP, where p
        // is zero, it stays there, so that their product is zero for -inf too.
        float a0 = 0.0f, a1 = 0.0f, lse = 0.0f, gl = 0.0f;
        int tl = -1;                        // the target's place in this half
        if (n < p.B) {
          const int tg = p.g.targets[n];
          const float s = -p.inv_t * (p.g.scale != nullptr ? p.g.scale[0] : 1.0f);
          lse = p.g.lse[n];
          // (no such token: no term)
          if (tg >= 0 && tg < p.K) {
            gl = p.g.dlogp[n] * s;
            tl = tg - p.t_off - vb;
          }
          a0 = gl;
          if (p.g.dentropy != nullptr) {
            a1 = p.g.dentropy[n] * s;
            a0 = fmaf(a1, p.g.entropy[n], a0);
          }
        }
        if (vb < p.V && nw0 < p.B) {
          const bool f16 = (p.idesc & (7u << 7)) == 0;   // the head's format
          sg.claim(lane);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint4 w[8];
#pragma unroll
            for (int hb = 0; hb < 2; ++hb) {
              const int c0 = 64 * b + 32 * hb;             // first of 32 columns
              float x[32];
#pragma unroll
              for (int i = 0; i < 32; i += 2) {
                const float* z = &acc[(c0 + i) >> 4][i & 15];
                float2 lp = fma2_rn(make_float2(z[0], z[1]), make_float2(p.inv_t, p.inv_t),
                                    make_float2(-lse, -lse));
                lp = make_float2(fmax_nan(lp.x, kLowLogP), fmax_nan(lp.y, kLowLogP));
                const float2 e = mul2_rn(lp, make_float2(kLog2eScore, kLog2eScore));
                const float2 y = mul2_rn(make_float2(exp2_approx(e.x), exp2_approx(e.y)),
                                         fma2_rn(lp, make_float2(a1, a1), make_float2(a0, a0)));
                x[i] = y.x;
                x[i + 1] = y.y;
              }
              const bool hit = tl >= c0 && tl < c0 + 32;
              if (__any_sync(0xffffffffu, hit)) {
                float at = 0.0f;
#pragma unroll
                for (int i = 0; i < 32; ++i) {
                  at = tl == c0 + i ? x[i] : at;
                  x[i] = tl == c0 + i ? 0.0f : x[i];
                }
                if (hit) p.coef[n] = at - gl;
              }
#pragma unroll
              for (int k = 0; k < 4; ++k)
                w[4 * hb + k] = make_uint4(
                    pack16(x[8 * k], x[8 * k + 1], f16), pack16(x[8 * k + 2], x[8 * k + 3], f16),
                    pack16(x[8 * k + 4], x[8 * k + 5], f16), pack16(x[8 * k + 6], x[8 * k + 7], f16));
            }
            sg.put(b, w, lane);
          }
          sg.store(&tmO, lane, vb, vb + 64, vb + 64 < p.V, nw0);
        }
      } else if constexpr (OP == OP_DH) {
        // fp32 partial sums of the segment, rows padded to whole tiles
        const int row0 = t.seg * (p.n0 * 256) + nw0;
        if (nw0 < p.B) store_f32(acc, sg, &tmO, lane, vb, p.K, row0);
      } else {
        const bool f16 = (p.idesc & (7u << 7)) == 0;
        if constexpr (OP == OP_DW_FEW) {
          // the warp's vocabulary rows that are targets: mostly none, which is
          // one branch around one copy of the long code
          constexpr int kW = kFewRows / 32;
          uint32_t hits[kW], any = 0;
          int rel[kW];
#pragma unroll
          for (int k = 0; k < kW; ++k) {
            rel[k] = few[k] >= 0 ? few[k] - nw0 : -1;
            hits[k] = __ballot_sync(0xffffffffu, rel[k] >= 0 && rel[k] < 32);
            any |= hits[k];
          }
          while (any != 0) {
            int n = 0, row = 0;
            bool found = false;
            any = 0;
#pragma unroll
            for (int k = 0; k < kW; ++k) {
              const int src = __ffs(hits[k]) - 1;
              const int at = __shfl_sync(0xffffffffu, rel[k], src < 0 ? 0 : src);
              if (!found && src >= 0) {          // the same in every lane
                found = true;
                n = 32 * k + src;
                row = at;
                hits[k] &= hits[k] - 1;
              }
              any |= hits[k];
            }
            if (lane == row) add_row(p, acc, n, p.coef[n], vb, f16);
          }
        } else {
          add_targets(p, acc, sg, run1 > run0 ? run0 : -1, vb, lane);
        }
        __syncwarp();
        const float s = p.w.scale != nullptr ? p.w.scale[1] : 1.0f;
        if (vb < p.K && nw0 < p.V) {
          sg.claim(lane);
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            uint4 w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const float* x = &acc[4 * b + (k >> 1)][(k & 1) * 8];
              w[k] = make_uint4(pack16(x[0] * s, x[1] * s, f16), pack16(x[2] * s, x[3] * s, f16),
                                pack16(x[4] * s, x[5] * s, f16), pack16(x[6] * s, x[7] * s, f16));
            }
            sg.put(b, w, lane);
          }
          sg.store(&tmO, lane, vb, vb + 64, vb + 64 < p.K, nw0);
        }
      }
    }
    if (failed && threadIdx.x == 128) atomicOr(p.err, ERR_TIMEOUT);
    if (kStore) {
      // the stores are complete before the CTA (and its shared memory) goes
      if (lane == 0) bulk_wait_group<0>();
      __syncwarp();
    }
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
