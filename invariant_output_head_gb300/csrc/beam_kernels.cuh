// beam_kernels.cuh -- one step of beam search: the best continuations of a
// sequence's beams, and the beams' states moved to their new places.
//
// Selection. Row r = sequence * beams + beam has logits z_v. A candidate (beam,
// v) scores  s_beam + (z_v - m) / T - log sum_u 2^((z_u - m) log2(e) / T),  m the
// row's maximum. The n_out best of a sequence are found in one pass over its
// logits: within a row all scores move together, so a row's candidates are its
// n_out largest logits, and the row's sum is needed for those alone.
//
// beam_scan_kernel reads the logits, once. Its blocks share the tiles (1024
// logits) of all rows evenly, so the last block ends with the first whatever the
// rows; a row that spans blocks has a part in each. A warp takes a tile a round.
// Each tile leaves its maximum and sum (in an order that its elements' places in
// the row set, so they do not depend on how rows are cut). The part's largest
// logits collect in shared memory: an element is kept if it is above the
// smallest of the M = n_out best at the last cut, and the list is cut to M after
// rounds 2, 4, 8, 16, ...: about M entries a span (16 sequences of 32 beams, M =
// 64: 104 us; cut after 4, 16, 64: 115; the same at M = 16). The first threshold comes from
// the first round itself: the M-th largest of 128 maxima of 64 elements each. An
// element is compared as a 64-bit word: its order as a number, then the lower
// index first. Warps meet at the cuts only.
//
// beam_merge_kernel, a block a sequence: a warp a beam joins the tiles' sums in
// a fixed tree and merges the parts' sorted lists, then the block merges the
// beams' lists by score.
//
// What the scan waits for is the latency of its chains, not memory: 64 sequences
// of 8 beams x 128256 in bf16, n_out = 16, 131 MB: 49 us a call (2.7 TB/s), 55 %
// of the issue slots busy with 24 warps an SM, about 440 instructions a tile of
// 1024: some 130 the exponentials' sum, 180 the loads, maxima and the rest, 130
// the entries and cuts (a lane with an entry takes its warp through the appends).
// Without entries and cuts it would take 31. Tried and slower: tiles of 512 with 32 to 48 warps an SM
// (54 to 64 us: the instructions a tile that do not depend on its size), tiles
// staged three ahead by asynchronous copies (54: more instructions, and loads are
// not what is waited for), whole rows or equal parts of rows for blocks (73: the
// last wave).
#pragma once
#include "quant_kernels.cuh"
#include "score_kernels.cuh"

namespace detlm {

constexpr int kBeamMax = 32;              // beams of a sequence (a lane each in the merge)
constexpr int kBeamOutMax = 64;           // continuations a sequence can ask for
constexpr int kBeamPartsMax = 32;         // parts of a row (a lane each in the merge)
constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanTile = 1024;           // logits of a tile: 32 a lane
constexpr int kScanPer = kScanTile / 32;
constexpr int kScanRound = kScanWarps * kScanTile;
constexpr int kScanCap = 1024;            // entries of the list
constexpr float kFusedMost = 16777216.0f; // largest |maximum| log2(e) / T of a tile summed in fused form
// blocks of an SM (their registers: a tile and the next)
__host__ __device__ constexpr int scan_resident(int fmt) { return fmt == QF_FP32 ? 2 : 3; }

using u64 = unsigned long long;

struct BeamScanParams {
  const void* logits;       // [rows][V]
  const float* score;       // [rows] the beams' scores
  const uint8_t* finished;  // optional [rows]
  float2* tile;             // [rows][n_tiles]: maximum, sum
  u64* best;                // [rows][parts][M], sorted, 0 behind the last
  int64_t tiles;            // of all rows
  int32_t V, n_tiles, parts, M;
  float c;                  // log2(e) / T
};
struct BeamMergeParams {
  const float* score;
  const uint8_t* finished;
  const float2* tile;
  const u64* best;
  int32_t* parent;          // [n_seq][M]
  int32_t* token;
  float* out;
  int64_t tiles;
  int32_t n_tiles, parts, M, beams, end_token;
  int32_t blocks;           // of the scan
  float c, inv_t;
};

// The scan's block b takes tiles [scan_first(b), scan_first(b + 1)) of all rows';
// scan_block is the block that a tile falls to.
__device__ __forceinline__ int64_t scan_first(int64_t tiles, int blocks, int b) { return tiles * b / blocks; }
__device__ __forceinline__ int scan_block(int64_t tiles, int blocks, int64_t t) {
  const uint64_t n = static_cast<uint64_t>(t + 1) * static_cast<uint32_t>(blocks) - 1;
  // (a division of 32 bits is much shorter, and mostly enough)
  if ((n | static_cast<uint64_t>(tiles)) >> 32 == 0) return static_cast<int>(static_cast<uint32_t>(n) / static_cast<uint32_t>(tiles));
  return static_cast<int>(n / static_cast<uint64_t>(tiles));
}

// A beam that proposes continuations of its own.
__device__ __forceinline__ bool beam_open(const float* score, const uint8_t* finished, int64_t r) {
  return isfinite(score[r]) && (finished == nullptr || finished[r] == 0);
}

// The list's n entries (at most kScanCap), sorted and cut to the M largest, all
// different; the threads of the block together. Entries count those above them.
__device__ __forceinline__ int scan_cut(u64* list, int n, int M) {
  constexpr int kMine = kScanCap / kScanThreads;
  u64 mine[kMine];
  int rank[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int at = threadIdx.x + i * kScanThreads;
    mine[i] = at < n ? list[at] : 0;
    rank[i] = 0;
  }
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    if (threadIdx.x + i * kScanThreads >= n) break;
#pragma unroll 8
    for (int j = 0; j < n; ++j) rank[i] += list[j] > mine[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kMine; ++i)
    if (threadIdx.x + i * kScanThreads < n && rank[i] < M) list[rank[i]] = mine[i];
  __syncthreads();
  return min(n, M);
}

// A lane's share of a tile as loaded: 32 numbers of 32 bits, or 16 words of two
// neighbours of 16.
template <int FMT>
struct ScanTile {
  static constexpr int kWords = FMT == QF_FP32 ? kScanPer : kScanPer / 2;
  uint32_t w[kWords];
  // nothing: the type's -inf
  static constexpr uint32_t kNone = FMT == QF_FP32 ? 0xFF800000u : FMT == QF_BF16 ? 0xFF80FF80u : 0xFC00FC00u;
  __device__ __forceinline__ void none() {
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = kNone;
  }
  // Tile `at` of a row of V; `words`: a row of 16-bit numbers starts on a word.
  // (The loads stand alone, so that all are under way together.)
  __device__ __forceinline__ void load(const uint8_t* row, int at, int V, bool words) {
    const int lane = threadIdx.x & 31;
    if (words && at <= V - kScanTile) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + (FMT == QF_FP32 ? at : at / 2) + lane;
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __ldg(p + 32 * i);
    } else if constexpr (FMT == QF_FP32) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(row);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int k = at + 32 * i + lane;
        w[i] = k < V ? __ldg(p + k) : kNone;
      }
    } else {
      const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
      if (at <= V - kScanTile) {           // (between words: element by element)
        p += at + 2 * lane;
        uint16_t lo[kWords], hi[kWords];
#pragma unroll
        for (int i = 0; i < kWords; ++i) {
          lo[i] = __ldg(p + 64 * i);
          hi[i] = __ldg(p + 64 * i + 1);
        }
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = lo[i] | (static_cast<uint32_t>(hi[i]) << 16);
        return;
      }
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int k = at + 64 * i + 2 * lane;
        const uint32_t lo = k < V ? __ldg(p + k) : kNone & 0xFFFFu;
        const uint32_t hi = k + 1 < V ? __ldg(p + k + 1) : kNone & 0xFFFFu;
        w[i] = lo | (hi << 16);
      }
    }
  }
  // elements 2 i and 2 i + 1 of the lane
  __device__ __forceinline__ float2 pair(int i) const {
    if constexpr (FMT == QF_FP32)
      return make_float2(__uint_as_float(w[2 * i]), __uint_as_float(w[2 * i + 1]));
    else
      return unpack16(w[i], FMT == QF_FP16);
  }
  // the largest of each eight elements, NaN aside
  __device__ __forceinline__ void maxima(float (&m)[kScanPer / 8]) const {
#pragma unroll
    for (int g = 0; g < kScanPer / 8; ++g) {
      if constexpr (FMT == QF_FP32) {
        float y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          y[i] = fmaxf(__uint_as_float(w[8 * g + i]), __uint_as_float(w[8 * g + 4 + i]));
        m[g] = fmaxf(fmaxf(y[0], y[1]), fmaxf(y[2], y[3]));
      } else {
        const uint32_t y = max2(max2(w[4 * g], w[4 * g + 1]), max2(w[4 * g + 2], w[4 * g + 3]));
        const float2 v = unpack16(y, FMT == QF_FP16);
        m[g] = fmaxf(v.x, v.y);
      }
    }
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    if constexpr (FMT == QF_BF16) {
      const __nv_bfloat162 m = __hmax2(*reinterpret_cast<__nv_bfloat162*>(&a), *reinterpret_cast<__nv_bfloat162*>(&b));
      return *reinterpret_cast<const uint32_t*>(&m);
    }
    const __half2 m = __hmax2(*reinterpret_cast<__half2*>(&a), *reinterpret_cast<__half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&m);
  }
};
// index in the row of a lane's element i of the tile at `at`
template <int FMT>
__device__ __forceinline__ int scan_index(int at, int i) {
  const int lane = threadIdx.x & 31;
  return FMT == QF_FP32 ? at + 32 * i + lane : at + 64 * (i >> 1) + 2 * lane + (i & 1);
}

// The sum of 2^f over a lane's elements, in a fixed order.
template <int FMT, typename F>
__device__ __forceinline__ float scan_sum(const ScanTile<FMT>& x, F f) {
  float2 e[4];
#pragma unroll
  for (int i = 0; i < kScanPer / 2; ++i) {
    float2 y = f(x.pair(i));
    y = make_float2(exp2_approx(y.x), exp2_approx(y.y));
    if (i < 4) e[i] = y;
    else add2_rn(e[i & 3].x, e[i & 3].y, y.x, y.y);
  }
  add2_rn(e[0].x, e[0].y, e[1].x, e[1].y);
  add2_rn(e[2].x, e[2].y, e[3].x, e[3].y);
  add2_rn(e[0].x, e[0].y, e[2].x, e[2].y);
  return e[0].x + e[0].y;
}

template <int FMT>
__global__ void __launch_bounds__(kScanThreads, scan_resident(FMT)) beam_scan_kernel(const BeamScanParams p) {
  __shared__ u64 list[kScanCap];
  __shared__ __align__(16) uint32_t top[kScanWarps * 128];
  __shared__ int count;
  __shared__ uint32_t level;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t size = FMT == QF_FP32 ? 4 : 2;
  const int blocks = static_cast<int>(gridDim.x);
  const int64_t end = scan_first(p.tiles, blocks, blockIdx.x + 1);
  grid_dep_wait();
  for (int64_t from = scan_first(p.tiles, blocks, blockIdx.x); from < end;) {
    // the block's part of row r: tiles [t0, t1)
    const int64_t r = from / p.n_tiles;
    const int t0 = static_cast<int>(from - r * p.n_tiles);
    const int t1 = static_cast<int>(min(static_cast<int64_t>(p.n_tiles), t0 + end - from));
    from += t1 - t0;
    if (!beam_open(p.score, p.finished, r)) continue;
    const uint8_t* row = static_cast<const uint8_t*>(p.logits) + static_cast<size_t>(r) * p.V * size;
    const bool words = (reinterpret_cast<uintptr_t>(row) & 3) == 0;   // (rows of 32-bit numbers always)
    ScanTile<FMT> next;
    if (t0 + warp < t1) next.load(row, (t0 + warp) * kScanTile, p.V, words);
    u64 last = 0;                         // the M-th best entry at the last cut
    float above = -INFINITY;              // an entry is larger (-inf is none)
    int n = 0;                            // entries before this span
    auto cut = [&]() {
      n = scan_cut(list, count, p.M);
      if (n == p.M) {
        // (what comes later has a higher index: of equal logits it is the lower)
        last = list[p.M - 1];
        above = score_unkey(static_cast<uint32_t>(last >> 32));
      }
      if (threadIdx.x == 0) count = n;
      __syncthreads();
    };
    __syncthreads();                      // the previous part is written
    if (threadIdx.x == 0) {
      count = 0;
      level = 0xFFFFFFFFu;
    }
    __syncthreads();
    const int rounds = (t1 - t0 + kScanWarps - 1) / kScanWarps;
    for (int done = 0; done < rounds;) {
      // a span: rounds 0 and 1, 2 and 3, 4 to 7, ...
      const int stop = min(rounds, max(2, 2 * done));
      bool over = false;
      for (int k = done; k < stop; ++k) {
        const int t = t0 + k * kScanWarps + warp;
        const int at = t * kScanTile;
        ScanTile<FMT> x;
        if (t < t1) x = next;
        else x.none();
        // the next round's tile is on its way during this one
        if (t + kScanWarps < t1) next.load(row, at + kScanRound, p.V, words);
        float g[kScanPer / 8];
        x.maxima(g);
        float m = fmaxf(fmaxf(g[0], g[1]), fmaxf(g[2], g[3]));
        if (k == 0) {
          // the first threshold: the M-th largest of maxima of as few and large
          // groups as hold twice M in the round's tiles: of four lanes, two, one, or
          // of eight elements
          const int tiles = min(t1 - t0, kScanWarps);
          int each = 8;                                  // groups of a tile
          while (each < 128 && tiles * each < 2 * p.M) each = each == 32 ? 128 : 2 * each;
          if (t < t1) {
            if (each == 128) {
#pragma unroll
              for (int j = 0; j < 4; ++j) top[warp * 128 + 4 * lane + j] = score_key(g[j]);
            } else {
              float pm = m;
              if (each < 32) pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 1));
              if (each < 16) pm = fmaxf(pm, __shfl_xor_sync(0xffffffffu, pm, 2));
              const int step = 32 / each;
              if (lane % step == 0) top[warp * each + lane / step] = score_key(pm);
            }
          }
          __syncthreads();
          const int groups = tiles * each;
          for (int i = threadIdx.x; i < (groups + 31) / 32 * 32; i += kScanThreads) {
            const uint32_t me = i < groups ? top[i] : 0u;
            int larger = 0;
#pragma unroll 4
            for (int j = 0; j < groups; j += 4) {
              const uint4 o = *reinterpret_cast<const uint4*>(&top[j]);
              larger += (o.x > me) + (o.y > me) + (o.z > me) + (o.w > me);
            }
            // (the least of those with fewer than M above them)
            const uint32_t least =
                __reduce_min_sync(0xffffffffu, i < groups && larger < p.M ? me : 0xFFFFFFFFu);
            if (lane == 0) atomicMin(&level, least);
          }
          __syncthreads();
          // one step below it, so that its equals are entries (below +0 comes
          // the first negative number: keys know no -0); -inf stays
          const uint32_t key = groups >= p.M ? level : 0u;
          if (key > score_key(-INFINITY)) above = score_unkey(key == 0x80000000u ? key - 2 : key - 1);
        }
        // entries above the threshold
        if (m > above) {
          auto add = [&](float y, int i) {
            const int to = atomicAdd(&count, 1);
            if (to < kScanCap) list[to] = order_word(score_key(y), scan_index<FMT>(at, i));
            else over = true;
          };
#pragma unroll
          for (int j = 0; j < kScanPer / 8; ++j) {
            if (!(g[j] > above)) continue;
#pragma unroll
            for (int i = 4 * j; i < 4 * j + 4; ++i) {
              const float2 v = x.pair(i);
              if (v.x > above) add(v.x, 2 * i);
              if (v.y > above) add(v.y, 2 * i + 1);
            }
          }
        }
        // the tile's sum: 0 where it holds nothing but -inf, NaN with a NaN or +inf.
        // The rounding of base c is at most half a step of it, so up to 2^24 the
        // factor that puts it back is between 2^-1/2 and 2^1/2; from 2^32 on it can
        // be 0 or infinite (a tile masked with -1e10, or with the type's lowest
        // value at T = 2), so large maxima take the difference first.
        m = score_unkey(__reduce_max_sync(0xffffffffu, score_key(m)));
        const float base = m == -INFINITY ? 0.0f : m;
        const float e0 = __fmul_rn(base, p.c);
        float sum;
        if (fabsf(e0) < kFusedMost) {
          // x c - e0 in one rounding; e0 is off base c by what the factor puts back
          sum = scan_sum(x, [&](float2 v) {
            return fma2_rn(v, make_float2(p.c, p.c), make_float2(-e0, -e0));
          }) * exp2_approx(-fmaf(base, p.c, -e0));
        } else {
          sum = scan_sum(x, [&](float2 v) {
            return make_float2(__fmul_rn(v.x - base, p.c), __fmul_rn(v.y - base, p.c));
          });
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (lane == 0 && t < t1) p.tile[static_cast<size_t>(r) * p.n_tiles + t] = make_float2(m, sum);
      }
      // (nobody looks at the count but after this, and then nobody adds to it)
      if (__syncthreads_or(over)) {
        // more than the list holds (long runs of equal or rising logits): the
        // span again, after the n entries before it, one element a thread at a
        // time, cut whenever the next could run over
        if (threadIdx.x == 0) count = n;
        __syncthreads();
        for (int k = done; k < stop; ++k) {
          const int t = t0 + k * kScanWarps + warp;
          ScanTile<FMT> x;
          if (t < t1) x.load(row, t * kScanTile, p.V, words);
          else x.none();
          for (int i = 0; i < kScanPer; ++i) {
            const int now = count;
            __syncthreads();
            if (now > kScanCap - kScanThreads) cut();
            float y = -INFINITY;
#pragma unroll
            for (int j = 0; j < kScanPer / 2; ++j) {
              const float2 v = x.pair(j);
              y = 2 * j == i ? v.x : 2 * j + 1 == i ? v.y : y;
            }
            const u64 word = order_word(score_key(y), scan_index<FMT>(t * kScanTile, i));
            if (y > -INFINITY && word > last) list[atomicAdd(&count, 1)] = word;
            __syncthreads();
          }
        }
      }
      // (a few more than M would not raise the threshold by much)
      const int have = count;
      if (stop == rounds || have > 2 * p.M) {
        cut();
      } else {
        n = have;
        __syncthreads();
      }
      done = stop;
    }
    // the part's best, sorted; nothing behind the last
    const int part = static_cast<int>(blockIdx.x) - scan_block(p.tiles, blocks, r * p.n_tiles);
    u64* out = p.best + (static_cast<size_t>(r) * p.parts + part) * p.M;
    for (int i = threadIdx.x; i < p.M; i += kScanThreads) out[i] = i < n ? list[i] : 0;
  }
  // (only now: blocks of the merge that wait would take the place of blocks that
  // read)
  grid_dep_launch();
}

// (x - m) f for a finite m, by halves: the difference of two numbers may be past
// fp32 where its product is not (+-3e38 at T = 1e38). Otherwise the same bits.
__device__ __forceinline__ float far_times(float x, float m, float f) {
  const float y = __fmul_rn(__fmaf_rn(0.5f, x, __fmul_rn(-0.5f, m)), f);
  return __fadd_rn(y, y);
}

// Two tiles' maximum and sum as one (the same bits in either order).
__device__ __forceinline__ float2 tile_join(float2 a, float2 b, float c) {
  const float m = fmaxf(a.x, b.x);
  const float fa = a.x == m ? 1.0f : exp2_approx(far_times(a.x, m, c));
  const float fb = b.x == m ? 1.0f : exp2_approx(far_times(b.x, m, c));
  return make_float2(m, __fadd_rn(__fmul_rn(a.y, fa), __fmul_rn(b.y, fb)));
}

constexpr int kMergeBeamThreads = 256;

// The block's shared memory: a warp's lists of a beam, for as many warps as have
// one (later the merge's entries, 8 bytes each too); then every beam's candidates
// [beams][M]: scores, tokens, and their number; a number of each warp; one more.
__host__ __device__ inline size_t merge_lists(int beams, int parts, int M) {
  const int warps = beams < kMergeBeamThreads / 32 ? beams : kMergeBeamThreads / 32;
  return static_cast<size_t>(warps * parts > beams ? warps * parts : beams) * M;
}
__host__ __device__ inline size_t merge_smem(int beams, int parts, int M) {
  return merge_lists(beams, parts, M) * sizeof(u64) + static_cast<size_t>(beams) * (M * 8 + 4) +
         (kMergeBeamThreads / 32 + 1) * 4;
}

// Both merges place an entry by counting those before it, once a threshold has
// taken most of the others out. (Taking the best head M times over, or counting
// by bisection in each list, takes longer: every step waits for the one before.)
// Bound by latency: 5 to 7 us for a few beams, of which a few loads and the
// launch are half. As the last step of a sequence's last scan block (one launch,
// a counter a sequence) it saved 1 us for one request and cost 3 to 7 for
// hundreds of rows, whose scan it then holds up.
__global__ void __launch_bounds__(kMergeBeamThreads) beam_merge_kernel(const BeamMergeParams p) {
  grid_dep_launch();
  grid_dep_wait();
  extern __shared__ __align__(16) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t seq = blockIdx.x;
  const int M = p.M;
  u64* list = reinterpret_cast<u64*>(smem_raw) + static_cast<size_t>(warp) * p.parts * M;
  float* score = reinterpret_cast<float*>(reinterpret_cast<u64*>(smem_raw) + merge_lists(p.beams, p.parts, M));
  int32_t* token = reinterpret_cast<int32_t*>(score + p.beams * M);
  int* found = token + p.beams * M;
  int* count = found + p.beams;                // a number of each warp
  int& kept = count[kMergeBeamThreads / 32];
  if (threadIdx.x < p.beams) found[threadIdx.x] = 0;
  __syncthreads();
  for (int b = warp; b < p.beams; b += kMergeBeamThreads / 32) {
    const int64_t r = seq * p.beams + b;
    const float own = p.score[r];
    if (beam_open(p.score, p.finished, r)) {
      // the row's parts
      const int parts = scan_block(p.tiles, p.blocks, (r + 1) * p.n_tiles - 1) -
                        scan_block(p.tiles, p.blocks, r * p.n_tiles) + 1;
      const u64* best = p.best + static_cast<size_t>(r) * p.parts * M;
      const float2* tiles = p.tile + static_cast<size_t>(r) * p.n_tiles;
      const float2 none = make_float2(-INFINITY, 0.0f);
      // (the first loads of both together)
      const float2 first = lane < p.n_tiles ? tiles[lane] : none;
      const u64 word = lane < parts * M ? best[lane] : 0;
      __syncwarp();                            // the beam before has been read
      if (lane < parts * M) list[lane] = word;
#pragma unroll 8
      for (int i = lane + 32; i < parts * M; i += 32) list[i] = best[i];
      float2 t = tile_join(none, first, p.c);
#pragma unroll 4
      for (int i = lane + 32; i < p.n_tiles; i += 32) t = tile_join(t, tiles[i], p.c);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        t = tile_join(t, make_float2(__shfl_xor_sync(0xffffffffu, t.x, o),
                                     __shfl_xor_sync(0xffffffffu, t.y, o)), p.c);
      __syncwarp();
      // a row with a NaN or +inf, or with nothing but -inf, proposes nothing
      if (!(t.y > 0.0f && isfinite(t.y))) continue;
      const float log_s = logf(t.y);
      // entries below either bound are not among the M best: the least of the
      // lists' j-th entries, as j of each make M; the largest M-th entry
      const uint32_t* key = reinterpret_cast<const uint32_t*>(list) + 1;
      const int j = (M + parts - 1) / parts - 1;
      const uint32_t low = __reduce_min_sync(0xffffffffu, lane < parts ? key[2 * (lane * M + j)] : 0xFFFFFFFFu);
      const uint32_t high = __reduce_max_sync(0xffffffffu, lane < parts ? key[2 * (lane * M + M - 1)] : 0u);
      uint32_t least = max(max(low, high), 1u);
      // A short part's entries make the first bound a low one: then the M-th best
      // of all, closed in on by counting in every list until few more than M stay.
      auto at_least = [&](uint32_t v) {
        int a = 0, z = lane < parts ? M : 0;
        while (a < z) {
          const int mid = (a + z) >> 1;
          if (key[2 * (lane * M + mid)] >= v) a = mid + 1;
          else z = mid;
        }
        return static_cast<int>(__reduce_add_sync(0xffffffffu, a));
      };
      if (parts > 2) {
        uint32_t above = __reduce_max_sync(0xffffffffu, lane < parts ? key[2 * lane * M] : 0u) + 1;
        int stay = at_least(least);
        while (stay > 2 * M && above - least > 1) {
          const uint32_t mid = least + ((above - least) >> 1);
          const int c = at_least(mid);
          if (c >= M) {
            least = mid;
            stay = c;
          } else {
            above = mid;
          }
        }
      }
      int n = 0;
      for (int i0 = 0; i0 < parts * M; i0 += 32) {
        const u64 word = i0 + lane < parts * M ? list[i0 + lane] : 0;
        const bool stays = static_cast<uint32_t>(word >> 32) >= least;
        const uint32_t stay = __ballot_sync(0xffffffffu, stays);     // (all have read)
        if (stays) list[n + __popc(stay & ((1u << lane) - 1))] = word;
        n += __popc(stay);
      }
      __syncwarp();
      for (int i = lane; i < n; i += 32) {
        const u64 word = list[i];
        int rank = 0;
#pragma unroll 8
        for (int k = 0; k < n; ++k) rank += list[k] > word;
        if (rank >= M) continue;
        const float z = score_unkey(static_cast<uint32_t>(word >> 32));
        const float s = __fadd_rn(own, __fsub_rn(far_times(z, t.x, p.inv_t), log_s));
        if (!(s > -INFINITY)) continue;        // (and those behind it score no more)
        score[b * M + rank] = s;
        token[b * M + rank] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(word));
        atomicMax(&found[b], rank + 1);
      }
    } else if (isfinite(own) && lane == 0) {   // finished: stays as it is
      score[b * M] = own;
      token[b * M] = p.end_token;
      found[b] = 1;
    }
  }
  __syncthreads();
  // The beams' candidates, each beam's in falling order: score, then beam, then
  // place. The M-th best score by bisection of its bits, where the candidates
  // are many.
  const size_t o = static_cast<size_t>(seq) * M;
  const int all_places = p.beams * M;
  uint32_t least = 1;
  if (all_places > 2 * kMergeBeamThreads) {
    constexpr int kMine = kBeamMax * kBeamOutMax / kMergeBeamThreads;
    uint32_t mine[kMine];
#pragma unroll
    for (int k = 0; k < kMine; ++k) {
      const int i = threadIdx.x + k * kMergeBeamThreads;
      mine[k] = i < all_places && i % M < found[i / M] ? score_key(score[i]) : 0u;
    }
    least = 0;
    for (uint32_t bit = 0x80000000u; bit != 0; bit >>= 1) {
      const uint32_t at = least | bit;
      int n = 0;
#pragma unroll
      for (int k = 0; k < kMine; ++k) n += mine[k] >= at;
      n = __reduce_add_sync(0xffffffffu, n);
      if (lane == 0) count[warp] = n;
      __syncthreads();
      int all = 0;
#pragma unroll
      for (int k = 0; k < kMergeBeamThreads / 32; ++k) all += count[k];
      if (all >= M) least = at;
      __syncthreads();
    }
    least = max(least, 1u);
  }
  // those at least as good, in order of their places
  if (threadIdx.x == 0) kept = 0;
  __syncthreads();
  uint2* entry = reinterpret_cast<uint2*>(smem_raw);      // score, place (the lists are done with)
  for (int i = threadIdx.x; i < all_places; i += kMergeBeamThreads) {
    if (i % M >= found[i / M]) continue;
    const uint32_t x = score_key(score[i]);
    if (x >= least) entry[atomicAdd(&kept, 1)] = make_uint2(x, static_cast<uint32_t>(i));
  }
  __syncthreads();
  const int n = kept;
  for (int i = threadIdx.x; i < n; i += kMergeBeamThreads) {
    const uint2 me = entry[i];
    int rank = 0;
#pragma unroll 8
    for (int k = 0; k < n; ++k) {
      const uint2 x = entry[k];
      rank += x.x > me.x || (x.x == me.x && x.y < me.y);
    }
    if (rank >= M) continue;
    const int place = static_cast<int>(me.y);
    p.parent[o + rank] = place / M;
    p.token[o + rank] = token[place];
    p.out[o + rank] = score[place];
  }
  // places without a candidate
  int all = 0;
  for (int k = 0; k < p.beams; ++k) all += found[k];
  for (int j = all + threadIdx.x; j < M; j += kMergeBeamThreads) {
    p.parent[o + j] = -1;
    p.token[o + j] = -1;
    p.out[o + j] = -INFINITY;
  }
}

// ------------------------------------------------------------------- reorder
// Row n of a state is n_seg pieces of `bytes` contiguous bytes, seg_src (seg_dst)
// bytes apart, rows row_src (row_dst) apart. A sequence's rows take those of
// their parents. A thread takes one column (16 bytes, or as many as every
// address, stride and length of the state is a multiple of) of all the rows of a
// sequence: it has read every row that it overwrites before it writes one, so
// rows can move in place. Bound by memory, each parent read once (L1 has it for
// the rows that share it): the same 32 x 8 beams with parents drawn at random,
// 2.14 GB written and 1.4 GB of distinct parents read, 7.0 TB/s.
struct BeamState {
  const uint8_t* src;
  uint8_t* dst;
  int64_t row_src, row_dst, seg_src, seg_dst;
  uint32_t cols;            // columns of a segment
  uint32_t n_seg;
  uint32_t grain;           // bytes of a column: 16, 8, 4, 2 or 1
  uint32_t block0;          // the state's first block
};
constexpr int kReorderStates = 48;       // of a launch
constexpr int kReorderThreads = 256;
struct ReorderParams {
  const int32_t* parent;    // [n_seq][beams_out]
  int64_t n_seq;
  int32_t n_states, beams_in, beams_out;
  BeamState state[kReorderStates];
};
static_assert(sizeof(ReorderParams) <= 4096, "kernel parameters above 4 KB");

template <typename T, int KB>
__device__ __forceinline__ void reorder_column(const BeamState& s, const int* parent, int64_t seq,
                                               int beams_in, int beams_out, uint32_t col) {
  const uint32_t seg = col / s.cols;
  const int64_t off = static_cast<int64_t>(col - seg * s.cols) * sizeof(T);
  const uint8_t* src = s.src + seg * s.seg_src + off + seq * beams_in * s.row_src;
  uint8_t* dst = s.dst + seg * s.seg_dst + off + seq * beams_out * s.row_dst;
  const bool in_place = s.src == s.dst;
  // rows with no parent, and rows that stay where they are, are left alone
  auto moves = [&](int j) { return parent[j] >= 0 && !(in_place && parent[j] == j); };
  for (int j0 = 0; j0 < beams_out; j0 += KB) {
    T v[KB];
#pragma unroll
    for (int j = 0; j < KB; ++j)
      if (j0 + j < beams_out && moves(j0 + j))
        v[j] = *reinterpret_cast<const T*>(src + parent[j0 + j] * s.row_src);
#pragma unroll
    for (int j = 0; j < KB; ++j)
      if (j0 + j < beams_out && moves(j0 + j))
        *reinterpret_cast<T*>(dst + (j0 + j) * s.row_dst) = v[j];
  }
}

// KB: rows a thread holds; in place at least beams_out. Blocks of an SM: loads and
// stores wait for memory, so the warps count for more than registers that hold
// addresses (32 sequences of 8 beams, rows of 8.4 MB: 616 us with two blocks, 509
// with four; 16 of 4 beams: 160 with four, 132 with six).
__host__ __device__ constexpr int reorder_resident(int kb) { return kb <= 4 ? 6 : kb <= 8 ? 4 : kb <= 16 ? 2 : 1; }
template <int KB>
__global__ void __launch_bounds__(kReorderThreads, reorder_resident(KB))
beam_reorder_kernel(const __grid_constant__ ReorderParams p) {
  grid_dep_launch();
  grid_dep_wait();
  __shared__ int parent[kBeamOutMax];
  int k = 0;
  while (k + 1 < p.n_states && blockIdx.x >= p.state[k + 1].block0) ++k;
  const BeamState& s = p.state[k];
  const uint64_t col = static_cast<uint64_t>(blockIdx.x - s.block0) * kReorderThreads + threadIdx.x;
  const bool mine = col < static_cast<uint64_t>(s.cols) * s.n_seg;
  for (int64_t seq = blockIdx.y; seq < p.n_seq; seq += gridDim.y) {
    __syncthreads();
    if (threadIdx.x < p.beams_out) {
      const int from = p.parent[seq * p.beams_out + threadIdx.x];
      parent[threadIdx.x] = from < p.beams_in ? from : -1;
    }
    __syncthreads();
    if (!mine) continue;
    const uint32_t c = static_cast<uint32_t>(col);
    if (s.grain == 16) reorder_column<uint4, KB>(s, parent, seq, p.beams_in, p.beams_out, c);
    else if (s.grain == 8) reorder_column<uint2, KB>(s, parent, seq, p.beams_in, p.beams_out, c);
    else if (s.grain == 4) reorder_column<uint32_t, KB>(s, parent, seq, p.beams_in, p.beams_out, c);
    else if (s.grain == 2) reorder_column<uint16_t, KB>(s, parent, seq, p.beams_in, p.beams_out, c);
    else reorder_column<uint8_t, KB>(s, parent, seq, p.beams_in, p.beams_out, c);
  }
}

}  // namespace detlm
