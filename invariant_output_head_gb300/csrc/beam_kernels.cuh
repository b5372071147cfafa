// beam_kernels.cuh -- one step of beam search: the best continuations of a
// sequence's beams, and the beams' states moved to their new places.
//
// Selection. Row r = sequence * beams + beam has logits z_v. A candidate (beam,
// v) scores  s_beam + (z_v - m) / T - log sum_u 2^((z_u - m) log2(e) / T),  m the
// row's maximum. The n_out best of a sequence are found in one pass over its
// logits: within a row all scores move together, so a row's candidates are its
// n_out largest logits, and the row's sum is needed for those alone.
//
// beam_scan_kernel reads the logits. A block takes a part of a row in ascending
// order, kScanWarps tiles of kScanTile a round, each element in one register. Each
// tile leaves its maximum and sum (in an order that its elements' places in the
// row set, so they do not depend on how rows are cut into parts). The part's
// largest logits collect in shared memory: an element is kept if it is above the
// smallest of the M = n_out best so far, which after the first round few are
// (about M log(V / 4096) more in the whole row). The first threshold comes from
// the first round itself: the M-th largest of 128 maxima of 32 elements each.
// When the list runs full it is sorted by counting and cut to M. An element is
// compared as a 64-bit word: its order as a number, then the lower index first.
//
// beam_merge_kernel, a block a sequence: a warp a beam folds the tiles' sums in
// ascending order and merges the parts' sorted lists (one lane a list, the best
// head taken each time), then one warp merges the beams' lists by score.
//
// The scan is bound by instruction issue and the exponentials' unit about as
// much as by memory: an element costs a load, its conversion, a maximum, a
// fused multiply-add, an exponential, an addition and a comparison.
#pragma once
#include "score_kernels.cuh"

namespace detlm {

constexpr int kBeamMax = 32;              // beams of a sequence (a lane each in the merge)
constexpr int kBeamOutMax = 64;           // continuations a sequence can ask for
constexpr int kBeamPartsMax = 32;         // parts of a row (a lane each in the merge)
constexpr int kScanThreads = 256;
constexpr int kScanWarps = kScanThreads / 32;
constexpr int kScanTile = 512;            // logits of a tile: 16 a lane
constexpr int kScanPer = kScanTile / 32;
constexpr int kScanRound = kScanWarps * kScanTile;
constexpr int kScanCap = 1024;            // entries of the list

using u64 = unsigned long long;

struct BeamScanParams {
  const void* logits;       // [rows][V]
  const float* score;       // [rows] the beams' scores
  const uint8_t* finished;  // optional [rows]
  float2* tile;             // [rows][n_tiles]: maximum, sum
  u64* best;                // [rows][parts][M], sorted, 0 behind the last
  int64_t rows;
  int32_t V, n_tiles, parts, M;
  int32_t cut;              // entries above which the list is cut before the next round
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
  int32_t n_tiles, parts, M, beams, end_token;
  float c, inv_t;
};

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

// A lane's share of a tile as loaded: 16 numbers of 32 bits, or eight words of
// two neighbours of 16.
template <int FMT>
struct ScanTile {
  static constexpr int kWords = FMT == QF_FP32 ? kScanPer : kScanPer / 2;
  uint32_t w[kWords];
  // Tile `at` of a row of V; `words`: a row of 16-bit numbers starts on a word.
  // (A loop over the whole loads alone, so that all are under way together.)
  __device__ __forceinline__ void load(const uint8_t* row, int at, int V, bool words) {
    const int lane = threadIdx.x & 31;
    if (words && at + kScanTile <= V) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(row) + (FMT == QF_FP32 ? at : at / 2) + lane;
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = __ldg(p + 32 * i);
    } else if constexpr (FMT == QF_FP32) {
      const uint32_t* p = reinterpret_cast<const uint32_t*>(row);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int k = at + 32 * i + lane;
        w[i] = k < V ? __ldg(p + k) : 0xFF800000u;
      }
    } else {
      // (beyond the row's end: the type's -inf)
      constexpr uint32_t kNone = FMT == QF_BF16 ? 0xFF80u : 0xFC00u;
      const uint16_t* p = reinterpret_cast<const uint16_t*>(row);
#pragma unroll
      for (int i = 0; i < kWords; ++i) {
        const int k = at + 64 * i + 2 * lane;
        const uint32_t lo = k < V ? __ldg(p + k) : kNone;
        const uint32_t hi = k + 1 < V ? __ldg(p + k + 1) : kNone;
        w[i] = lo | (hi << 16);
      }
    }
  }
  __device__ __forceinline__ void values(float (&x)[kScanPer]) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      if constexpr (FMT == QF_FP32) {
        x[i] = __uint_as_float(w[i]);
      } else {
        const float2 v = unpack16(w[i], FMT == QF_FP16);
        x[2 * i] = v.x;
        x[2 * i + 1] = v.y;
      }
    }
  }
};
// index in the row of a lane's element i of the tile at `at`
template <int FMT>
__device__ __forceinline__ int scan_index(int at, int i) {
  const int lane = threadIdx.x & 31;
  return FMT == QF_FP32 ? at + 32 * i + lane : at + 64 * (i >> 1) + 2 * lane + (i & 1);
}

template <int FMT>
__global__ void __launch_bounds__(kScanThreads) beam_scan_kernel(const BeamScanParams p) {
  grid_dep_launch();
  grid_dep_wait();
  __shared__ u64 list[kScanCap];
  __shared__ __align__(16) uint32_t top[128];
  __shared__ int count;
  __shared__ uint32_t level;
  const int64_t r = blockIdx.y + static_cast<int64_t>(blockIdx.z) * gridDim.y;
  if (r >= p.rows || !beam_open(p.score, p.finished, r)) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const size_t size = FMT == QF_FP32 ? 4 : 2;
  const uint8_t* row = static_cast<const uint8_t*>(p.logits) + static_cast<size_t>(r) * p.V * size;
  const bool words = (reinterpret_cast<uintptr_t>(row) & 3) == 0;   // (rows of 32-bit numbers always)
  // whole tiles to a part
  const int t0 = static_cast<int>(static_cast<int64_t>(p.n_tiles) * blockIdx.x / p.parts);
  const int t1 = static_cast<int>(static_cast<int64_t>(p.n_tiles) * (blockIdx.x + 1) / p.parts);
  u64 last = 0;                           // the M-th best entry at the last cut
  float above = -INFINITY;                // an entry is larger (-inf is none)
  auto cut = [&](int have) {
    const int n = scan_cut(list, have, p.M);
    if (n == p.M) {
      // (what comes later has a higher index: of equal logits it is the lower)
      last = list[p.M - 1];
      above = score_unkey(static_cast<uint32_t>(last >> 32));
    }
    if (threadIdx.x == 0) count = n;
    __syncthreads();
  };
  if (threadIdx.x == 0) count = 0;
  __syncthreads();
  ScanTile<FMT> next;
  if (t0 + warp < t1) next.load(row, (t0 + warp) * kScanTile, p.V, words);
  for (int tr = t0; tr < t1; tr += kScanWarps) {
    const int t = tr + warp;
    const int at = t * kScanTile;
    float x[kScanPer];
    float m = -INFINITY;
    if (t < t1) {
      next.values(x);
    } else {
#pragma unroll
      for (int i = 0; i < kScanPer; ++i) x[i] = -INFINITY;
    }
    // the next round's tile is on its way during this one
    if (t + kScanWarps < t1) next.load(row, at + kScanRound, p.V, words);
    {
      // (a tree: the maximum's bits are the same in any order)
      float y[kScanPer / 2];
#pragma unroll
      for (int i = 0; i < kScanPer / 2; ++i) y[i] = fmaxf(x[i], x[i + kScanPer / 2]);
#pragma unroll
      for (int o = kScanPer / 4; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < o; ++i) y[i] = fmaxf(y[i], y[i + o]);
      m = y[0];
    }
    const float lane_max = m;             // NaN aside
    if (tr == t0) {
      // the first threshold: the M-th largest maximum of two lanes
      const float pm = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
      if ((lane & 1) == 0) top[warp * 16 + (lane >> 1)] = score_key(pm);
      if (threadIdx.x == 0) level = 0;
      __syncthreads();
      if (threadIdx.x < 128) {
        const uint32_t me = top[threadIdx.x];
        int larger = 0, equal = 0;
#pragma unroll 8
        for (int j = 0; j < 128; j += 4) {
          const uint4 o = *reinterpret_cast<const uint4*>(&top[j]);
          larger += (o.x > me) + (o.y > me) + (o.z > me) + (o.w > me);
          equal += (o.x == me) + (o.y == me) + (o.z == me) + (o.w == me);
        }
        if (larger < p.M && p.M <= larger + equal) level = me;
      }
      __syncthreads();
      // one step below it, so that its equals are entries (below +0 comes the
      // first negative number: keys know no -0); -inf stays
      const uint32_t key = level;
      if (key > score_key(-INFINITY)) above = score_unkey(key == 0x80000000u ? key - 2 : key - 1);
    }
    const float wm = score_unkey(__reduce_max_sync(0xffffffffu, score_key(m)));
    // the tile's sum: 0 where it holds nothing but -inf, NaN with a NaN or +inf
    const float base = wm == -INFINITY ? 0.0f : wm;
    float2 e[kScanPer / 2];
#pragma unroll
    for (int i = 0; i < kScanPer / 2; ++i) {
      float2 y = make_float2(x[2 * i], x[2 * i + 1]);
      add2_rn(y.x, y.y, -base, -base);
      y = mul2_rn(y, make_float2(p.c, p.c));
      e[i] = make_float2(exp2_approx(y.x), exp2_approx(y.y));
    }
#pragma unroll
    for (int o = kScanPer / 4; o > 0; o >>= 1)
#pragma unroll
      for (int i = 0; i < o; ++i) add2_rn(e[i].x, e[i].y, e[i + o].x, e[i + o].y);
    float sum = e[0].x + e[0].y;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0 && t < t1) p.tile[static_cast<size_t>(r) * p.n_tiles + t] = make_float2(wm, sum);

    // entries above the threshold
    bool over = false;
    if (lane_max > above) {
#pragma unroll
      for (int i = 0; i < kScanPer; ++i)
        if (x[i] > above) {
          const int k = atomicAdd(&count, 1);
          if (k < kScanCap) list[k] = order_word(score_key(x[i]), scan_index<FMT>(at, i));
          over |= k >= p.cut;
        }
    }
    // (nobody looks at the count but after this, and then nobody adds to it)
    if (__syncthreads_or(over)) {
      const int have = count;
      if (have <= kScanCap) {
        cut(have);
      } else {
        // more than the list holds (long runs of equal or rising logits): this
        // round again, after the entries of the rounds before it (their indices
        // are lower), one element a thread at a time, cut whenever the next
        // could run over
        u64 kept[kScanCap / kScanThreads];
#pragma unroll
        for (int i = 0; i < kScanCap / kScanThreads; ++i) kept[i] = list[threadIdx.x + i * kScanThreads];
        __syncthreads();
        if (threadIdx.x == 0) count = 0;
        __syncthreads();
        const uint32_t before = 0xFFFFFFFFu - static_cast<uint32_t>(tr * kScanTile);
#pragma unroll
        for (int i = 0; i < kScanCap / kScanThreads; ++i)
          if (static_cast<uint32_t>(kept[i]) > before) list[atomicAdd(&count, 1)] = kept[i];
        __syncthreads();
        for (int i = 0; i < kScanPer; ++i) {
          const int now = count;
          __syncthreads();
          if (now > kScanCap - kScanThreads) cut(now);
          float y = -INFINITY;
#pragma unroll
          for (int k = 0; k < kScanPer; ++k) y = k == i ? x[k] : y;
          const u64 word = order_word(score_key(y), scan_index<FMT>(at, i));
          if (y > -INFINITY && word > last) list[atomicAdd(&count, 1)] = word;
          __syncthreads();
        }
        cut(count);
      }
    }
  }
  // the part's best, sorted; nothing behind the last
  __syncthreads();
  const int n = scan_cut(list, count, p.M);
  u64* out = p.best + (static_cast<size_t>(r) * p.parts + blockIdx.x) * p.M;
  for (int i = threadIdx.x; i < p.M; i += kScanThreads) out[i] = i < n ? list[i] : 0;
}

// Two tiles' maximum and sum as one (the same bits in either order).
__device__ __forceinline__ float2 tile_join(float2 a, float2 b, float c) {
  const float m = fmaxf(a.x, b.x);
  const float fa = a.x == m ? 1.0f : exp2_approx((a.x - m) * c);
  const float fb = b.x == m ? 1.0f : exp2_approx((b.x - m) * c);
  return make_float2(m, __fadd_rn(__fmul_rn(a.y, fa), __fmul_rn(b.y, fb)));
}

constexpr int kMergeBeamThreads = 256;

__global__ void __launch_bounds__(kMergeBeamThreads) beam_merge_kernel(const BeamMergeParams p) {
  grid_dep_launch();
  grid_dep_wait();
  __shared__ float score[kBeamMax][kBeamOutMax];
  __shared__ int32_t token[kBeamMax][kBeamOutMax];
  __shared__ int found[kBeamMax];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t seq = blockIdx.x;
  for (int b = warp; b < p.beams; b += kMergeBeamThreads / 32) {
    const int64_t r = seq * p.beams + b;
    const float own = p.score[r];
    int n = 0;
    if (beam_open(p.score, p.finished, r)) {
      // the first entries of the parts' lists are on their way meanwhile
      const u64* lists = p.best + static_cast<size_t>(r) * p.parts * p.M;
      const u64* mine = lists + static_cast<size_t>(min(lane, p.parts - 1)) * p.M;
      u64 head = lane < p.parts ? mine[0] : 0;
      u64 next = lane < p.parts && p.M > 1 ? mine[1] : 0;
      int at = 2;
      float2 t = make_float2(-INFINITY, 0.0f);
      const float2* tiles = p.tile + static_cast<size_t>(r) * p.n_tiles;
#pragma unroll 4
      for (int i = lane; i < p.n_tiles; i += 32) t = tile_join(t, tiles[i], p.c);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        t = tile_join(t, make_float2(__shfl_xor_sync(0xffffffffu, t.x, o),
                                     __shfl_xor_sync(0xffffffffu, t.y, o)), p.c);
      // a row with a NaN or +inf, or with nothing but -inf, proposes nothing
      const float log_s = logf(t.y);
      if (t.y > 0.0f && isfinite(t.y)) {
        for (int j = 0; j < p.M; ++j) {
          u64 best;
          if (p.parts == 1) {
            best = mine[j];
          } else {
            const uint32_t hi = __reduce_max_sync(0xffffffffu, static_cast<uint32_t>(head >> 32));
            const uint32_t low = static_cast<uint32_t>(head >> 32) == hi ? static_cast<uint32_t>(head) : 0u;
            const uint32_t lo = __reduce_max_sync(0xffffffffu, low);
            best = (static_cast<u64>(hi) << 32) | lo;
            if (head == best && best != 0) {
              head = next;
              next = at < p.M ? mine[at] : 0;
              ++at;
            }
          }
          if (best == 0) break;
          const float z = score_unkey(static_cast<uint32_t>(best >> 32));
          const float s = __fadd_rn(own, __fsub_rn(__fmul_rn(__fsub_rn(z, t.x), p.inv_t), log_s));
          if (!(s > -INFINITY)) break;         // (and those behind it score no more)
          if (lane == 0) {
            score[b][j] = s;
            token[b][j] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
          }
          n = j + 1;
        }
      }
    } else if (isfinite(own)) {                // finished: stays as it is
      if (lane == 0) {
        score[b][0] = own;
        token[b][0] = p.end_token;
      }
      n = 1;
    }
    if (lane == 0) found[b] = n;
  }
  __syncthreads();
  if (warp != 0) return;
  // the beams' lists, each in falling order; of equal scores the lower beam's
  const int mine = lane < p.beams ? found[lane] : 0;
  int at = 0;
  uint32_t head = mine > 0 ? score_key(score[lane][0]) : 0u;
  const size_t o = static_cast<size_t>(seq) * p.M;
  for (int j = 0; j < p.M; ++j) {
    const uint32_t best = __reduce_max_sync(0xffffffffu, head);
    const int who = __ffs(__ballot_sync(0xffffffffu, head == best)) - 1;
    if (best == 0u) {                          // no candidate is left
      for (int k = j + lane; k < p.M; k += 32) {
        p.parent[o + k] = -1;
        p.token[o + k] = -1;
        p.out[o + k] = -INFINITY;
      }
      break;
    }
    if (lane == who) {
      p.parent[o + j] = lane;
      p.token[o + j] = token[lane][at];
      p.out[o + j] = score[lane][at];
      ++at;
      head = at < mine ? score_key(score[lane][at]) : 0u;
    }
  }
}

// ------------------------------------------------------------------- reorder
// Row n of a state is n_seg pieces of `bytes` contiguous bytes, seg_src (seg_dst)
// bytes apart, rows row_src (row_dst) apart. A sequence's rows take those of
// their parents. A thread takes one column (16 bytes, or as many as every
// address, stride and length of the state is a multiple of) of all the rows of a
// sequence: it has read every row that it overwrites before it writes one, so
// rows can move in place. Bound by memory.
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

// KB: rows a thread holds; in place at least beams_out.
template <int KB>
__global__ void __launch_bounds__(kReorderThreads)
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
