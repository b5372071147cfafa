// score_kernels.cuh -- from the projection's records to the score call's
// outputs, one block of 256 threads per hidden row: warps 0..3 fold the
// softmax statistics in the fixed tree, warps 4..7 meanwhile find the row's K
// largest logits; then every thread ranks candidates.
//
// The K largest, from K disjoint maxima. Any K disjoint sets of entries have
// K maxima; the smallest of those is a value that at least K entries reach.
// With the sets' maxima at hand (tile records, or the slots of the wide
// projection) this threshold costs no search, and only entries at or above it
// -- K H_K of them on average for exchangeable entries, H_K the harmonic
// number: 22 for K = 8, 130 for K = 32 -- need be ranked. A candidate's rank
// is the number of candidates that come before it (larger value, or the same
// value and a lower index), so every output slot has one writer and the
// result does not depend on the order in which candidates were gathered.
//
// Bound: latency. A block makes four dependent rounds of loads (records,
// their tree, the candidates' logits, the target), and a launch of up to ~1200
// rows is one wave of blocks. One launch with cold caches: 1 row of 32000
// 7.5 us (about 4 behind the projection, whose end it overlaps), 301 rows of
// 50001 10 us, 2048 rows of 50176 with candidates 17 us, 4098 rows of 1352
// with logits 30 us.
#pragma once
#include "head_kernels.cuh"
#include "pairop_kernels.cuh"

namespace detlm {

constexpr int kScoreThreads = 256;
constexpr int kTopMax = 32;          // alternatives a row can return
constexpr int kEntryCap = 512;       // candidates ranked in shared memory
constexpr int kTileCap = 512;        // tiles at or above the threshold

struct ScoreMergeParams {
  int32_t V, B, n_vt;       // n_vt: record tiles of a row
  int32_t K, C;
  float c, inv_t;
  const float* rec_m;       // [B][n_vt]
  const float* rec_s;
  const float* rec_u;
  const float* logits;      // in a workspace: [B][ld]
  int64_t ld;
  const float* zt;          // wide: [B] target logits
  const float* cand;        // wide: [B][C][kCandFloats]
  int32_t* words;           // wide: [B][row_words(K)]
  int32_t* tile_over;       // wide: any mark, then [ceil(B / 256)] marks
  const int32_t* targets;   // optional
  float* logp;              // with targets
  float* entropy;           // optional
  float* lse;               // optional
  int32_t* top_token;       // [B][K]
  float* top_logp;          // [B][K]
  int* err;
};

struct ScoreShared {
  Stat part[4];
  Stat tot;
  uint32_t slots[kTopMax];
  int n_tiles, n_entries;
  int32_t tiles[kTileCap];
  unsigned long long entry[kEntryCap];   // order words
  unsigned long long best[kScoreThreads / 32];
};

// Statistics of a row, by 128 threads (warps 0 .. 3). Narrow records are of
// 128-entry halves: a tile is the union of two.
template <bool NARROW>
__device__ __forceinline__ Stat row_stat(const ScoreMergeParams& p, size_t base, int g) {
  const int n_tiles = NARROW ? (p.n_vt + 1) >> 1 : p.n_vt;
  const int t1 = leaf_lo(g + 1, n_tiles);
  Stat acc{-INFINITY, 0.0f, 0.0f};
  auto rec = [&](int i) {
    return i < p.n_vt ? Stat{p.rec_m[base + i], p.rec_s[base + i], p.rec_u[base + i]}
                      : Stat{-INFINITY, 0.0f, 0.0f};
  };
#pragma unroll 2
  for (int t = leaf_lo(g, n_tiles); t < t1; ++t)
    acc = stat_merge(acc, NARROW ? stat_merge(rec(2 * t), rec(2 * t + 1), p.c) : rec(t), p.c);
  return acc;
}

// Order of alternatives as one word: larger value first, then lower index.
__device__ __forceinline__ unsigned long long order_word(uint32_t key, int32_t id) {
  return (static_cast<unsigned long long>(key) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(id));
}

// The entry of the whole block that comes first among those after `last`
// (0: none left). visit(f) calls f(value, id) on this thread's share.
template <typename Visit>
__device__ __forceinline__ unsigned long long next_best(ScoreShared& sh, unsigned long long last,
                                                        Visit visit) {
  unsigned long long b = 0;
  visit([&](float z, int32_t id) {
    if (!(z == z)) return;                            // a NaN is no alternative
    const unsigned long long o = order_word(score_key(z), id);
    if (o < last && o > b) b = o;
  });
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) {
    const unsigned long long x = __shfl_xor_sync(0xffffffffu, b, s);
    b = x > b ? x : b;
  }
  __syncthreads();                                    // the previous round's reads are done
  if ((threadIdx.x & 31) == 0) sh.best[threadIdx.x >> 5] = b;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kScoreThreads / 32; ++w) b = sh.best[w] > b ? sh.best[w] : b;
  return b;
}

// Write the row's alternatives: by rank when the gathered entries fit, else
// (very many equal values) one after the other by rescans.
template <typename Visit>
__device__ __forceinline__ void write_top(const ScoreMergeParams& p, ScoreShared& sh, int n,
                                          Visit visit) {
  const Stat tot = sh.tot;
  const float log_s = logf(tot.S);
  auto put = [&](int k, unsigned long long word) {
    const size_t o = static_cast<size_t>(n) * p.K + k;
    p.top_token[o] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(word));
    p.top_logp[o] = (score_unkey(static_cast<uint32_t>(word >> 32)) - tot.m) * p.inv_t - log_s;
  };
  const int ne = sh.n_entries;
  int found = min(ne, p.K);
  if (ne <= kEntryCap) {
    for (int e = threadIdx.x; e < ne; e += kScoreThreads) {
      const unsigned long long me = sh.entry[e];
      int rank = 0;
#pragma unroll 4
      for (int j = 0; j < ne; ++j) rank += sh.entry[j] > me;
      if (rank < p.K) put(rank, me);
    }
  } else {
    unsigned long long last = ~0ull;
    found = 0;
    for (int k = 0; k < p.K; ++k) {
      last = next_best(sh, last, visit);
      if (last == 0) break;
      found = k + 1;
      if (threadIdx.x == 0) put(k, last);
    }
  }
  // fewer logits than alternatives that are numbers
  for (int k = found + threadIdx.x; k < p.K; k += kScoreThreads) {
    p.top_token[static_cast<size_t>(n) * p.K + k] = -1;
    p.top_logp[static_cast<size_t>(n) * p.K + k] = __int_as_float(0x7fc00000);
  }
}

__device__ __forceinline__ void push_entry(ScoreShared& sh, float z, int32_t id, float thr) {
  if (z >= thr) {
    const int at = atomicAdd(&sh.n_entries, 1);
    if (at < kEntryCap) sh.entry[at] = order_word(score_key(z), id);
  }
}

// The row's statistics from the four warps' partial trees, and its outputs.
__device__ __forceinline__ void write_stats(const ScoreMergeParams& p, ScoreShared& sh, int n,
                                            float zt, int tg) {
  const Stat tot = stat_merge(stat_merge(sh.part[0], sh.part[1], p.c),
                              stat_merge(sh.part[2], sh.part[3], p.c), p.c);
  sh.tot = tot;
  const float log_s = logf(tot.S);
  const float nan = __int_as_float(0x7fc00000);
  const bool some = tot.m > -INFINITY;      // a row without a number has no distribution
  if (p.lse != nullptr) p.lse[n] = some ? fmaf(tot.m, p.inv_t, log_s) : nan;
  if (p.entropy != nullptr) p.entropy[n] = some ? log_s - (tot.U / tot.S) * p.inv_t : nan;
  if (p.targets != nullptr) {
    float lp = (zt - tot.m) * p.inv_t - log_s;
    if (tg == -1) {
      lp = 0.0f;                            // no token to score
    } else if (tg < 0 || tg >= p.V) {
      lp = nan;
      atomicOr(p.err, ERR_TARGET);
    }
    p.logp[n] = lp;
  }
}

// Logits in a workspace, with records of TILE entries: 128 (the one-CTA
// projection) or 256 (OP_SCOREZ).
template <int TILE>
__global__ void __launch_bounds__(kScoreThreads) score_logits_kernel(const ScoreMergeParams p) {
  constexpr int kPer = TILE / 32;
  __shared__ ScoreShared sh;
  grid_dep_launch();   // the next call's projection may start (it prefetches only W)
  const int n = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t base = static_cast<size_t>(n) * p.n_vt;
  const float* z = p.logits + static_cast<size_t>(n) * p.ld;
  const int g = static_cast<int>(threadIdx.x) - 128;
  if (g >= 0 && g < kTopMax) sh.slots[g] = 0;
  if (g == 0) sh.n_tiles = sh.n_entries = 0;
  grid_dep_wait();     // records and logits are complete and visible
  float zt = 0.0f;
  int tg = -1;
  if (threadIdx.x == 0 && p.targets != nullptr) {
    tg = p.targets[n];
    if (tg >= 0 && tg < p.V) zt = z[tg];
  }
  if (warp < 4) {
    Stat x = row_stat<TILE == kBM>(p, base, threadIdx.x);
#pragma unroll
    for (int b = 1; b < 32; b <<= 1) x = stat_merge(x, shfl_xor(x, b), p.c);
    if (lane == 0) sh.part[warp] = x;
  } else if (p.K > 0) {
    // the tiles' maxima, kept in registers up to 1024 tiles (further ones are
    // read again)
    constexpr int kKeep = 8;
    float keep[kKeep];
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const int t = g + 128 * i;
      keep[i] = t < p.n_vt ? p.rec_m[base + t] : __int_as_float(0x7fc00000);
    }
    named_bar_sync(1, 128);                       // slots are zero
#pragma unroll
    for (int i = 0; i < kKeep; ++i)
      if (g + 128 * i < p.n_vt) atomicMax(&sh.slots[(g + 128 * i) % p.K], score_key(keep[i]));
    for (int t = g + 128 * kKeep; t < p.n_vt; t += 128)
      atomicMax(&sh.slots[t % p.K], score_key(p.rec_m[base + t]));
    named_bar_sync(1, 128);
    uint32_t lo = lane < p.K ? sh.slots[lane] : 0xFFFFFFFFu;
    lo = __reduce_min_sync(0xffffffffu, lo);
    const float thr = score_unkey(lo);
    auto want = [&](float m, int t) {
      if (m >= thr) {
        const int at = atomicAdd(&sh.n_tiles, 1);
        if (at < kTileCap) sh.tiles[at] = t;
      }
    };
#pragma unroll
    for (int i = 0; i < kKeep; ++i) want(keep[i], g + 128 * i);
    for (int t = g + 128 * kKeep; t < p.n_vt; t += 128) want(p.rec_m[base + t], t);
    named_bar_sync(1, 128);
    const int nt = sh.n_tiles;
    if (nt > kTileCap) {
      if (g == 0) sh.n_entries = kEntryCap + 1;   // rescans below
    } else {
      // several tiles at a time per warp: 32 loads in flight a lane
      constexpr int kT = 32 / kPer;
      for (int i0 = (warp - 4) * kT; i0 < nt; i0 += 4 * kT) {
        float x[kT][kPer];
        int v0[kT];
#pragma unroll
        for (int i = 0; i < kT; ++i) {
          v0[i] = i0 + i < nt ? sh.tiles[i0 + i] * TILE + lane : p.V;
#pragma unroll
          for (int j = 0; j < kPer; ++j)
            x[i][j] = v0[i] + 32 * j < p.V ? z[v0[i] + 32 * j] : __int_as_float(0x7fc00000);
        }
#pragma unroll
        for (int i = 0; i < kT; ++i)
#pragma unroll
          for (int j = 0; j < kPer; ++j) push_entry(sh, x[i][j], v0[i] + 32 * j, thr);
      }
    }
  }
  __syncthreads();
  if (threadIdx.x == 0) write_stats(p, sh, n, zt, tg);
  if (p.K == 0) return;
  __syncthreads();
  write_top(p, sh, n, [&](auto f) {
    for (int v = threadIdx.x; v < p.V; v += kScoreThreads) f(z[v], v);
  });
}

// The candidates of a wide row at or above thr into shared memory.
__device__ __forceinline__ void gather_blocks(const ScoreMergeParams& p, ScoreShared& sh, int n,
                                              int nb, float thr, int g, int threads) {
  const float* cd = p.cand + static_cast<size_t>(n) * p.C * kCandFloats;
  constexpr int kU = 4;
  for (int i0 = g; i0 < nb * 4; i0 += threads * kU) {
    float4 x[kU];
    int v0[kU];
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      const int i = i0 + k * threads;
      v0[k] = p.V;
      if (i < nb * 4) {
        const float* b = cd + static_cast<size_t>(i >> 2) * kCandFloats;
        x[k] = reinterpret_cast<const float4*>(b)[i & 3];
        v0[k] = __float_as_int(b[16]) * 16 + (i & 3) * 4;
      }
    }
#pragma unroll
    for (int k = 0; k < kU; ++k) {
      if (v0[k] < p.V) push_entry(sh, x[k].x, v0[k], thr);
      if (v0[k] + 1 < p.V) push_entry(sh, x[k].y, v0[k] + 1, thr);
      if (v0[k] + 2 < p.V) push_entry(sh, x[k].z, v0[k] + 2, thr);
      if (v0[k] + 3 < p.V) push_entry(sh, x[k].w, v0[k] + 3, thr);
    }
  }
}

template <typename F>
__device__ __forceinline__ void visit_blocks(const ScoreMergeParams& p, int n, int nb, F f) {
  const float* cd = p.cand + static_cast<size_t>(n) * p.C * kCandFloats;
  for (int i = threadIdx.x; i < nb * 16; i += kScoreThreads) {
    const float* b = cd + static_cast<size_t>(i >> 4) * kCandFloats;
    const int v = __float_as_int(b[16]) * 16 + (i & 15);
    if (v < p.V) f(b[i & 15], v);
  }
}

// More than 128 rows: 256-entry records, slots and candidate blocks. A row
// whose list overflowed gets the exact rule for its K best tiles -- (maximum,
// lowest index) of the K-th -- and its 256-row tile is marked for OP_SELECT,
// which computes the whole tile's product again (rows of all equal logits, say
// of zeros: 8192 x 151936 x 1536, K = 8, none 2327 us, one such row 2744, one in
// every tile 4891).
__global__ void __launch_bounds__(kScoreThreads) score_wide_kernel(const ScoreMergeParams p) {
  __shared__ ScoreShared sh;
  const int n = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t base = static_cast<size_t>(n) * p.n_vt;
  const int g = static_cast<int>(threadIdx.x) - 128;
  if (g == 0) sh.n_entries = 0;
  grid_dep_launch();
  grid_dep_wait();
  int32_t* w = p.words + static_cast<size_t>(n) * row_words(p.K);
  float zt = 0.0f;
  int tg = -1;
  if (threadIdx.x == 0 && p.targets != nullptr) {
    tg = p.targets[n];
    if (tg >= 0 && tg < p.V) zt = p.zt[n];
  }
  const int nb = p.K > 0 ? w[RW_COUNT] : 0;
  const bool over = nb > p.C;
  if (warp < 4) {
    Stat x = row_stat<false>(p, base, threadIdx.x);
#pragma unroll
    for (int b = 1; b < 32; b <<= 1) x = stat_merge(x, shfl_xor(x, b), p.c);
    if (lane == 0) sh.part[warp] = x;
  } else if (p.K > 0 && !over) {
    named_bar_sync(1, 128);                       // the entry count is zero
    uint32_t lo = lane < p.K ? static_cast<uint32_t>(w[kRowWords + lane]) : 0xFFFFFFFFu;
    lo = __reduce_min_sync(0xffffffffu, lo);
    gather_blocks(p, sh, n, nb, score_unkey(lo), g, 128);
  }
  __syncthreads();
  if (threadIdx.x == 0) write_stats(p, sh, n, zt, tg);
  if (p.K == 0) return;
  __syncthreads();
  if (!over) {
    write_top(p, sh, n, [&](auto f) { visit_blocks(p, n, nb, f); });
    return;
  }
  unsigned long long last = ~0ull;
  for (int k = 0; k < p.K; ++k) {
    const unsigned long long b = next_best(sh, last, [&](auto f) {
      for (int t = threadIdx.x; t < p.n_vt; t += kScoreThreads) f(p.rec_m[base + t], t);
    });
    if (b == 0) break;
    last = b;
  }
  if (threadIdx.x == 0) {
    w[RW_COUNT] = 0;
    w[RW_SEL_M] = __float_as_int(score_unkey(static_cast<uint32_t>(last >> 32)));
    w[RW_SEL_T] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(last));
    w[RW_OVER] = 1;
    p.tile_over[0] = 1;
    p.tile_over[1 + (n >> 8)] = 1;
  }
}

// The rows that OP_SELECT served: alternatives from their second lists (K
// tiles of 16 blocks at most, which the list always holds).
__global__ void __launch_bounds__(kScoreThreads) score_select_kernel(const ScoreMergeParams p) {
  __shared__ ScoreShared sh;
  grid_dep_launch();
  grid_dep_wait();
  if (p.tile_over[0] == 0) return;
  for (int n = blockIdx.x; n < p.B; n += gridDim.x) {
    if (p.tile_over[1 + (n >> 8)] == 0) continue;
    const int32_t* w = p.words + static_cast<size_t>(n) * row_words(p.K);
    if (w[RW_OVER] == 0) continue;
    const size_t base = static_cast<size_t>(n) * p.n_vt;
    __syncthreads();
    if (threadIdx.x == 0) sh.n_entries = 0;
    if (threadIdx.x < 128) {
      Stat x = row_stat<false>(p, base, threadIdx.x);
#pragma unroll
      for (int b = 1; b < 32; b <<= 1) x = stat_merge(x, shfl_xor(x, b), p.c);
      if ((threadIdx.x & 31) == 0) sh.part[threadIdx.x >> 5] = x;
    }
    __syncthreads();
    if (threadIdx.x == 0)
      sh.tot = stat_merge(stat_merge(sh.part[0], sh.part[1], p.c),
                          stat_merge(sh.part[2], sh.part[3], p.c), p.c);
    const int nb = min(w[RW_COUNT], p.C);
    gather_blocks(p, sh, n, nb, __int_as_float(w[RW_SEL_M]), threadIdx.x, kScoreThreads);
    __syncthreads();
    write_top(p, sh, n, [&](auto f) { visit_blocks(p, n, nb, f); });
  }
}

// int8 -> fp16 (exact) of the hidden rows, n16 16-byte words, as a dependent
// of the previous kernel on the stream. A copy of a few MB: a launch's latency
// (2.7 us, 205 x 1040) bounds it.
__global__ void __launch_bounds__(256) rows_to_f16_kernel(const uint4* __restrict__ in,
                                                          uint4* __restrict__ out, size_t n16) {
  grid_dep_launch();
  grid_dep_wait();
  for (size_t i = blockIdx.x * size_t{256} + threadIdx.x; i < n16; i += size_t{256} * gridDim.x) {
    const uint4 w = in[i];
    uint4 o0, o1;
    i8x4_to_h2x2(w.x, o0.x, o0.y);
    i8x4_to_h2x2(w.y, o0.z, o0.w);
    i8x4_to_h2x2(w.z, o1.x, o1.y);
    i8x4_to_h2x2(w.w, o1.z, o1.w);
    out[2 * i] = o0;
    out[2 * i + 1] = o1;
  }
}

// Rows of d8 16-byte words into rows of ld8 (the words behind them are left:
// the tensor maps end at d). Bound: for W (once a change of it) the copy, 50001
// x 1000 in 30 us, 6.7 TB/s; for hidden rows a launch's latency, 3 us.
__global__ void __launch_bounds__(256) pad_rows_kernel(const uint4* __restrict__ in,
                                                       uint4* __restrict__ out, int64_t rows, int d8,
                                                       int ld8) {
  grid_dep_launch();
  grid_dep_wait();
  const int64_t n = rows * d8;
  for (int64_t i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
    const int64_t r = i / d8;
    out[r * ld8 + (i - r * d8)] = in[i];
  }
}

// ------------------------------------------------------- gradient helpers
// The power of two that dz of an fp16 head is held in: |dz| is at most
// (|g_l| + |g_H| (1 + log V)) / T, whose largest finite value C over the rows
// goes to [2^13, 2^14). fp16 then keeps every dz of 2^-27 C or more with its
// full 11 bits (its smallest normal is 2^-14), and smaller ones to 2^-38 C (half
// a step of its subnormals). Rows whose gradient is not finite have no say:
// theirs is lost whatever the scale, and a scale of 1 would take small
// gradients of the others with it. (bf16 has fp32's exponents and needs none.)
// One block; the maximum is exact, so the result does not depend on any order.
// A launch's latency, 3.7 us at 777 rows.
__global__ void __launch_bounds__(1024)
grad_scale_kernel(const float* dlogp, const float* dentropy, const int32_t* targets, int B,
                  float inv_t, float h_max, float* scale) {
  __shared__ float wm[32];
  grid_dep_launch();
  grid_dep_wait();
  float m = 0.0f;
  for (int n = threadIdx.x; n < B; n += 1024) {
    float b = targets[n] >= 0 ? fabsf(dlogp[n]) : 0.0f;
    if (dentropy != nullptr) b = fmaf(fabsf(dentropy[n]), h_max, b);
    b *= inv_t;
    if (b < INFINITY) m = fmaxf(m, b);
  }
#pragma unroll
  for (int s = 16; s > 0; s >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, s));
  if ((threadIdx.x & 31) == 0) wm[threadIdx.x >> 5] = m;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < 32; ++w) m = fmaxf(m, wm[w]);
    int e = 0;
    // frexp: m = f 2^e with f in [1/2, 1), so m 2^(14 - e) < 2^14; nothing to
    // scale (all zero): 1
    if (m > 0.0f) frexpf(m, &e);
    int s = m > 0.0f ? 14 - e : 0;
    s = max(-100, min(100, s));
    scale[0] = ldexpf(1.0f, s);
    scale[1] = ldexpf(1.0f, -s);
  }
}

// The hidden rows by their target: list holds the rows whose target lies in
// [v0, v0 + vc), by target, then ascending; starts[v] is where entry v's run
// begins. Block t does the 256 entries of tile t: its threads count, each over
// an ascending share of the rows, the targets of lower tiles and of each of
// its own entries; gather its own rows in order; and place them by entry.
// Every block reads all B targets (from L2). Latency: 196 tiles, 777 rows in 4.2
// us, 2048 rows in 5.0.
struct TargetListParams {
  const int32_t* targets;
  int32_t B, v0, vc;
  int32_t* starts;          // [256 n_vt + 1]
  int32_t* list;            // [B]
};
constexpr int kListWindow = 4096;    // rows of a tile gathered at a time

__global__ void __launch_bounds__(256) target_list_kernel(const TargetListParams p) {
  __shared__ int sums[2][8];
  __shared__ int count[256];           // of the tile's entries
  __shared__ int rows[kListWindow];
  __shared__ uint8_t entries[kListWindow];
  grid_dep_launch();
  const int tile = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  count[threadIdx.x] = 0;
  __syncthreads();
  grid_dep_wait();
  const int share = (p.B + 255) / 256;
  const int n0 = min(p.B, static_cast<int>(threadIdx.x) * share), n1 = min(p.B, n0 + share);
  // the entry of row n's target within this pass, or -1
  auto entry = [&](int n) {
    const int32_t t = p.targets[n];
    return t >= p.v0 && t - p.v0 < p.vc ? t - p.v0 : -1;
  };
  int less = 0, mine = 0;
#pragma unroll 8
  for (int n = n0; n < n1; ++n) {
    const int v = entry(n);
    less += v >= 0 && (v >> 8) < tile;
    if (v >= 0 && (v >> 8) == tile) {
      ++mine;
      atomicAdd(&count[v & 255], 1);
    }
  }
  // exclusive scans over the block: of the shares' rows, of the entries' counts
  int scan = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, scan, s);
    if (lane >= s) scan += x;
  }
  less = __reduce_add_sync(0xffffffffu, less);
  if (lane == 31) sums[0][warp] = scan;
  if (lane == 0) sums[1][warp] = less;
  __syncthreads();
  int before = 0, all = 0;
  less = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) {
    before += w < warp ? sums[0][w] : 0;
    all += sums[0][w];
    less += sums[1][w];
  }
  const int place = before + scan - mine;              // this share's first row in the tile
  const int own = count[threadIdx.x];
  scan = own;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, scan, s);
    if (lane >= s) scan += x;
  }
  __syncthreads();
  if (lane == 31) sums[0][warp] = scan;
  __syncthreads();
  before = 0;
#pragma unroll
  for (int w = 0; w < 8; ++w) before += w < warp ? sums[0][w] : 0;
  const int start = less + before + scan - own;
  p.starts[tile * 256 + threadIdx.x] = start;
  count[threadIdx.x] = start;                          // from here on: the entry's next place
  if (tile == static_cast<int>(gridDim.x) - 1 && threadIdx.x == 255) p.starts[tile * 256 + 256] = less + all;
  for (int w0 = 0; w0 < all; w0 += kListWindow) {
    if (mine > 0) {
      int i = place - w0;
      for (int n = n0; n < n1; ++n) {
        const int v = entry(n);
        if (v < 0 || (v >> 8) != tile) continue;
        if (i >= 0 && i < kListWindow) {
          rows[i] = n;
          entries[i] = static_cast<uint8_t>(v);
        }
        ++i;
      }
    }
    __syncthreads();
    // one warp places them, 32 at a time in order (a barrier per step would
    // cost more than the other warps bring)
    const int here = min(kListWindow, all - w0);
    if (warp == 0) {
      for (int i0 = 0; i0 < here; i0 += 32) {
        const bool in = i0 + lane < here;
        const int e = in ? entries[i0 + lane] : 256 + lane;
        const uint32_t same = __match_any_sync(0xffffffffu, e);
        const int rank = __popc(same & ((1u << lane) - 1u));
        int to = 0;
        if (in) {
          to = count[e];
          p.list[to + rank] = rows[i0 + lane];
        }
        __syncwarp();
        if (in && rank == 0) count[e] = to + __popc(same);
        __syncwarp();
      }
    }
    __syncthreads();
  }
}

// The sums of the list's runs: sums[first][k] = sum coef_n h[n][k], fp32, rows
// in ascending order. Block (i, j): the run that starts at list position i, if
// one does, columns 1024 j on, eight a thread. Bound by latency: 777 x 1000 in
// 5.6 us, 2048 x 1536 in 9.6, with a few rows a run. A run's rows are fetched
// eight at a time, one group after another, so a token that many rows share
// costs about a microsecond for every eight of them: 5928 x 1077 x 296, the
// whole gradient (alone, cold caches) 117 us with uniform targets, 459 with half
// of them equal; rows without a token to score are best given as -1 (107).
struct TargetSumParams {
  const int32_t* targets;
  const int32_t* starts;
  const int32_t* list;
  const float* coef;
  const uint4* h;           // [B][d8]
  float* sums;              // [B][d]
  int32_t n_vt, v0, d8, fp16;
};

__global__ void __launch_bounds__(128) target_sum_kernel(const TargetSumParams p) {
  grid_dep_launch();
  grid_dep_wait();
  const int i = blockIdx.x;
  if (i >= p.starts[p.n_vt * 256]) return;
  const int v = p.targets[p.list[i]] - p.v0;
  const int first = p.starts[v], end = p.starts[v + 1];
  if (first != i) return;
  const int c = blockIdx.y * 128 + threadIdx.x;
  if (c >= p.d8) return;
  float a[8] = {};
  const bool f16 = p.fp16 != 0;
  constexpr int kU = 8;                       // rows in flight
  for (int e0 = first; e0 < end; e0 += kU) {
    uint4 w[kU];
    float g[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      g[j] = 0.0f;
      w[j] = make_uint4(0, 0, 0, 0);
      if (e0 + j < end) {
        const int n = p.list[e0 + j];
        g[j] = p.coef[n];
        w[j] = __ldg(p.h + static_cast<size_t>(n) * p.d8 + c);
      }
    }
#pragma unroll
    for (int j = 0; j < kU; ++j) {
      if (e0 + j >= end) break;
      const uint32_t x[4] = {w[j].x, w[j].y, w[j].z, w[j].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 t = unpack16(x[k], f16);
        a[2 * k] = fmaf(g[j], t.x, a[2 * k]);
        a[2 * k + 1] = fmaf(g[j], t.y, a[2 * k + 1]);
      }
    }
  }
  float4* o = reinterpret_cast<float4*>(p.sums) + (static_cast<size_t>(first) * p.d8 + c) * 2;
  o[0] = make_float4(a[0], a[1], a[2], a[3]);
  o[1] = make_float4(a[4], a[5], a[6], a[7]);
}

// dh from the partial sums [n_part][rows_pad][d] (fp32): partials of a segment
// are added in ascending order (per_seg of them; one when a unit covered the
// whole segment), the segments' sums in ascending order onto the running
// sum -- the same additions however the segments were split over units or
// passes -- and last the target's entry of dz times its row of W.
// Four columns a thread; bound by reading the partials: 777 x 1000, 25 partials
// (78 MB) in 17 us; 2048 x 1536, four of them, in 16.
struct FoldParams {
  const float* part;
  int64_t rows_pad;
  int32_t B, d4;            // d / 4
  int32_t n_part, per_seg;  // per_seg: 1 or kSegChunks
  float* acc;               // running sum [B][d] between passes
  int32_t first, last;      // first pass: start from zero; last: write dh
  int32_t fp16;
  const float* scale;
  const int32_t* targets;
  const float* coef;        // [B] the target's entry of dz
  const void* W;            // [V][d]
  int32_t V;
  uint32_t* out;            // dh [B][d], two elements a word
};

__global__ void __launch_bounds__(256) grad_fold_kernel(const FoldParams p) {
  grid_dep_launch();
  grid_dep_wait();
  const int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x;
  if (i >= static_cast<int64_t>(p.B) * p.d4) return;
  const int64_t step = p.rows_pad * p.d4;               // float4 per partial
  const float4* src = reinterpret_cast<const float4*>(p.part) + i;
  float4* run = reinterpret_cast<float4*>(p.acc) + i;
  // the target's row of W is on its way while the partials are added
  const int n = static_cast<int>(i / p.d4), c = static_cast<int>(i - static_cast<int64_t>(n) * p.d4);
  float g = 0.0f;
  uint2 w = make_uint2(0, 0);
  if (p.last) {
    const int tg = p.targets[n];
    if (tg >= 0 && tg < p.V) {
      g = p.coef[n];
      w = reinterpret_cast<const uint2*>(p.W)[static_cast<size_t>(tg) * p.d4 + c];
    }
  }
  float4 a = p.first ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : *run;
  auto add = [](float4& x, const float4& y) {
    x.x = __fadd_rn(x.x, y.x);
    x.y = __fadd_rn(x.y, y.y);
    x.z = __fadd_rn(x.z, y.z);
    x.w = __fadd_rn(x.w, y.w);
  };
  constexpr int kU = kSegChunks;                        // loads in flight
  for (int s = 0; s < p.n_part; s += kU) {
    float4 v[kU];
#pragma unroll
    for (int j = 0; j < kU; ++j)
      if (s + j < p.n_part) v[j] = __ldcs(src + (s + j) * step);
    if (p.per_seg == 1) {
#pragma unroll
      for (int j = 0; j < kU; ++j)
        if (s + j < p.n_part) add(a, v[j]);
    } else {
#pragma unroll
      for (int j = 1; j < kU; ++j)
        if (s + j < p.n_part) add(v[0], v[j]);
      add(a, v[0]);
    }
  }
  if (!p.last) {
    *run = a;
    return;
  }
  const float s = p.scale != nullptr ? p.scale[1] : 1.0f;
  const bool f16 = p.fp16 != 0;
  if (g != 0.0f) {
    const float2 lo = unpack16(w.x, f16), hi = unpack16(w.y, f16);
    a.x = fmaf(g, lo.x, a.x);
    a.y = fmaf(g, lo.y, a.y);
    a.z = fmaf(g, hi.x, a.z);
    a.w = fmaf(g, hi.y, a.w);
  }
  reinterpret_cast<uint2*>(p.out)[i] =
      make_uint2(pack16(a.x * s, a.y * s, f16), pack16(a.z * s, a.w * s, f16));
}

}  // namespace detlm
