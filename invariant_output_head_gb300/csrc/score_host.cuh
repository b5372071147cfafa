// score_host.cuh -- the host side of the score call, its gradient and the
// scaled logits: argument checks, workspaces, tensor maps and launches. Part
// of detlm_head.cu's translation unit (it uses that file's handle and
// helpers).
#pragma once

namespace {

constexpr int kNarrowRows = 128;             // rows of the one-CTA projection at most
// The wide projection writes its logits (OP_SCOREZ) where candidates do not
// pay. Candidates cost some 14 us whatever the size (until a threshold can thin
// them out, every block of the vocabulary is one); logits cost about 3 ns a
// row more in the merge and 0.2 ns per thousand of them. They break even near
// B (15000 + V) = kLogitWork. Logits against candidates, us:
//   256 x 151936 x 1536, K = 8    118 / 134    512 rows    188 / 181
//   1024 rows                     342 / 313    1024 x 50001 x 1000    106 / 106
//   1280 x 32000 x 2048, K = 8    130 / 140    2048 rows   197 / 193
//   2048 x 8192 x 1024, K = 8      53 /  58    4096 rows    93 /  87
//   4098 x 1352 x 384, K = 5       40 /  47    6000 rows    52 /  47
// (The largest exception found: 384 x 151936 x 1536, 181 / 176.)
constexpr int64_t kLogitWork = 68000000;
constexpr int64_t kGradPassBytes = int64_t{8} << 30;   // dz held at once, about
constexpr int64_t kGradSeg = static_cast<int64_t>(kSegChunks) * kGradChunkBoxes * 64;   // entries of a segment

// 2-D tensor map of 16-bit or 32-bit elements: `inner` contiguous, rows of
// `stride` bytes.
bool encode_box(CUtensorMap* m, CUtensorMapDataType type, const void* base, int64_t inner,
                int64_t outer, int64_t stride, uint32_t box_inner, uint32_t box_outer,
                CUtensorMapSwizzle swizzle, bool load) {
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(outer)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(stride)};
  cuuint32_t box[2] = {box_inner, box_outer};
  cuuint32_t estr[2] = {1, 1};
  return g_encode(m, type, 2, const_cast<void*>(base), dims, strides, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                  load ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_NONE,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
CUtensorMapDataType map_type(int dtype) {
  return dtype == DETLM_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

int ensure_buffer(void** buf, size_t* have, size_t need, cudaStream_t stream) {
  if (need <= *have) return DETLM_OK;
  if (*buf != nullptr) {
    cudaError_t e = cudaStreamSynchronize(stream);
    if (e != cudaSuccess) return status_from_cuda(e);
    cudaFree(*buf);
    *buf = nullptr;
    *have = 0;
  }
  cudaError_t e = cudaMalloc(buf, need);
  if (e != cudaSuccess) {
    *buf = nullptr;
    cudaGetLastError();
    return status_from_cuda(e);
  }
  *have = need;
  return DETLM_OK;
}

template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), dim3 grid, unsigned block, cudaStream_t stream,
                             Args... args) {
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

// An ordinary (not programmatic) launch between a change of W on the stream
// and a call whose kernels request W boxes before waiting for the stream: it
// starts when everything before it is complete and visible.
__global__ void weights_fence_kernel() {}
int weights_fence(cudaStream_t stream) {
  weights_fence_kernel<<<1, 32, 0, stream>>>();
  return status_from_cuda(cudaGetLastError());
}

// Rows of 16-bit operands whose length is an odd multiple of 16 bytes start
// in the middle of a 32-byte sector every other time, and a TMA box of them
// moves half as fast (1024 x 50001 x 1000 scored: 105 us, x 1008: 76 us). Such
// heads keep a copy of W with rows on cache lines, made by the first call (or
// reserve) that wants it and again by detlm_head_weights_changed, and the
// pair products copy their hidden rows likewise.
bool needs_padding(const detlm_head* h) { return h->d % 16 != 0; }
int64_t padded_d(const detlm_head* h) { return needs_padding(h) ? (h->d + 63) / 64 * 64 : h->d; }

unsigned copy_grid(const detlm_head* h, int64_t words) {
  const int64_t want = (words + 255) / 256;
  return static_cast<unsigned>(want < 16 * h->num_sms ? want : 16 * h->num_sms);
}
int pad_rows(const detlm_head* h, const void* in, void* out, int64_t rows, cudaStream_t stream) {
  const int d8 = static_cast<int>(h->d / 8), ld8 = static_cast<int>(padded_d(h) / 8);
  return status_from_cuda(launch_dependent(pad_rows_kernel, copy_grid(h, rows * d8), 256, stream,
                                           static_cast<const uint4*>(in), static_cast<uint4*>(out),
                                           rows, d8, ld8));
}

// W for the score and gradient calls: itself, or its copy with padded rows
// (see copy_enqueued).
int padded_weights(detlm_head* h, cudaStream_t stream, const void** W) {
  *W = h->W;
  if (!needs_padding(h)) return DETLM_OK;
  if (h->Wp == nullptr) {
    void* p = nullptr;
    const cudaError_t e = cudaMalloc(&p, static_cast<size_t>(h->V) * padded_d(h) * 2);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return status_from_cuda(e);
    }
    h->Wp = p;
  }
  if (!h->wp_ready) {
    int st = pad_rows(h, h->W, h->Wp, h->V, stream);
    if (st == DETLM_OK) st = weights_fence(stream);
    if (st != DETLM_OK) return st;
    h->wp_ready = copy_enqueued(stream);
  }
  *W = h->Wp;
  return DETLM_OK;
}

int reserve_weights(detlm_head* h) {
  if (!needs_padding(h) || h->wp_ready) return DETLM_OK;
  // the copy is made on no stream of the caller's: whatever writes W first
  cudaError_t e = cudaDeviceSynchronize();
  if (e != cudaSuccess) return status_from_cuda(e);
  const void* W = nullptr;
  const int st = padded_weights(h, nullptr, &W);
  return st == DETLM_OK ? status_from_cuda(cudaStreamSynchronize(nullptr)) : st;
}

// CTA pairs of the pair-product kernels that fit on the GPU at once (they all
// have one shape: 384 threads, the full shared memory).
cudaError_t op_pairs(detlm_head* h, int* pairs) {
  if (h->op_pairs == 0) {
    cudaError_t e = prepare_kernel<pairop_kernel<OP_DZ>>(kRegsLaunchWide);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg;
    std::memset(&cfg, 0, sizeof(cfg));
    cfg.blockDim = dim3(kRowsThreads);
    cfg.dynamicSmemBytes = kSmemLimit;
    cfg.gridDim = dim3(static_cast<unsigned>(h->num_sms & ~1));
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int clusters = 0;
    e = cudaOccupancyMaxActiveClusters(&clusters, pairop_kernel<OP_DZ>, &cfg);
    if (e != cudaSuccess) return e;
    if (clusters <= 0) return cudaErrorInvalidConfiguration;
    h->op_pairs = clusters < h->num_sms / 2 ? clusters : h->num_sms / 2;
  }
  *pairs = h->op_pairs;
  return cudaSuccess;
}

// The stages of a product: as many as fit beside its staging buffers and
// words (with few rows a stage is small, and more of them keep as much of B
// in flight).
template <int OP>
int op_stages(int a_rows) {
  int s = kOpMaxStages;
  while (s > 2 && op_layout(OP, s, a_rows).total + 1024u > kSmemLimit) --s;
  return s;
}
// Rows of the box of a K-major operand of B rows: with fewer than 128 no more
// than there are (whole 8-row swizzle atoms).
uint32_t a_box_rows(int64_t B) { return B < kRowsHalf ? static_cast<uint32_t>((B + 7) / 8 * 8) : kRowsHalf; }

template <int OP>
cudaError_t launch_pairop(detlm_head* h, const CUtensorMap& a, const CUtensorMap& b,
                          const CUtensorMap& o, PairOpParams p, cudaStream_t stream) {
  cudaError_t e = prepare_kernel<pairop_kernel<OP>>(kRegsLaunchWide);
  if (e != cudaSuccess) return e;
  int pairs = 0;
  e = op_pairs(h, &pairs);
  if (e != cudaSuccess) return e;
  p.a_rows = static_cast<uint8_t>(op_dw(OP) ? kRowsHalf : a_box_rows(p.B));
  p.stages = static_cast<uint8_t>(op_stages<OP>(p.a_rows));
  p.stall = static_cast<uint8_t>(h->stall);
  p.err = h->d_err;
  p.timeout_ns = h->timeout_ns;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.blockDim = dim3(kRowsThreads);
  cfg.dynamicSmemBytes = op_layout(OP, p.stages, p.a_rows).total + 1024u;
  cfg.gridDim = dim3(static_cast<unsigned>(2 * (p.units < pairs ? p.units : pairs)));
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, pairop_kernel<OP>, a, b, o, p);
}

bool is_device_memory(const void* p) {
  cudaPointerAttributes a;
  if (cudaPointerGetAttributes(&a, p) != cudaSuccess) {
    cudaGetLastError();   // clear the error the query recorded
    return false;
  }
  return a.type == cudaMemoryTypeDevice;
}

// OUT_* of a header dtype.
bool out_type(int dtype, int* type) {
  if (dtype != DETLM_FP32 && dtype != DETLM_BF16 && dtype != DETLM_FP16) return false;
  *type = dtype == DETLM_FP32 ? OUT_F32 : dtype == DETLM_BF16 ? OUT_BF16 : OUT_FP16;
  return true;
}

// The tensor map of an output [B][V] that the pair products' staging buffers
// leave by: whole 16-byte rows of device memory (false: plain stores).
bool encode_out(CUtensorMap* m, int type, void* out, int64_t V, int64_t B) {
  const CUtensorMapDataType t = type == OUT_F32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                : type == OUT_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                   : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const int size = type == OUT_F32 ? 4 : 2;
  return (V * size) % 16 == 0 && aligned(out, 16) && is_device_memory(out) &&
         encode_box(m, t, out, V, B, V * size, 128u / size, 32, CU_TENSOR_MAP_SWIZZLE_128B, false);
}

void time_start(detlm_head* h, cudaStream_t stream) {
  if (h->t_start) cudaEventRecord(h->t_start, stream);
}
void time_stop(detlm_head* h, cudaStream_t stream) {
  if (h->t_stop) cudaEventRecord(h->t_stop, stream);
  h->t_start = h->t_stop = nullptr;
}

// ------------------------------------------------------------------- score
// Candidate blocks a row's list can hold: those of the tiles that run before
// any threshold can reach them (two rounds of the pairs over n_rt row tiles),
// what passes a threshold of K slots (see score_tail), and room. More is not
// an error: such rows are computed again (OP_SELECT).
int cand_blocks(int pairs, int64_t n_rt, int K) {
  return 64 + 32 * K + 16 * static_cast<int>((pairs + n_rt - 1) / n_rt + 2);
}

// With logits: logits [B][ld] and records [3][B][n_vt]. Without (many rows, or
// no alternatives wanted of more than 128): records, target logits, row words and
// tile marks (cleared together), candidates.
struct ScoreLayout {
  int64_t n_vt, ld;
  size_t rows, logits, rec, rec_part, zt, words, words_bytes, tiles, cand, total;
};
// The most rows whose alternatives come from logits in the workspace.
int64_t logit_rows(const detlm_head* h) { return kLogitWork / (15000 + h->V); }
bool score_has_logits(const detlm_head* h, int64_t B, int K) {
  return B <= kNarrowRows || (K > 0 && B <= logit_rows(h));
}

ScoreLayout score_layout(const detlm_head* h, int64_t B, int K, int pairs) {
  ScoreLayout L;
  std::memset(&L, 0, sizeof(L));
  const bool narrow = B <= kNarrowRows;
  size_t at = 0;
  auto part = [&](size_t bytes) {
    const size_t a = at;
    at += round256(bytes);
    return a;
  };
  L.n_vt = narrow ? h->n_vt : tiles256(h->V);
  L.rec_part = round256(static_cast<size_t>(B) * L.n_vt * 4) / 4;
  L.rec = part(3 * L.rec_part * 4);
  if (!narrow && needs_padding(h)) L.rows = part(static_cast<size_t>(B) * padded_d(h) * 2);
  if (score_has_logits(h, B, K)) {
    L.ld = narrow ? h->V : (h->V + 31) / 32 * 32;
    L.logits = part(static_cast<size_t>(B) * L.ld * 4);
  } else {
    const int64_t n_rt = (B + kRowsM - 1) / kRowsM;
    L.zt = part(static_cast<size_t>(B) * 4);
    L.words_bytes = (static_cast<size_t>(B) * row_words(K) + 1 + n_rt) * 4;
    L.words = part(L.words_bytes);
    L.tiles = L.words + static_cast<size_t>(B) * row_words(K) * 4;
    // an upper bound of B * cand_blocks that grows with B, so that a
    // workspace for B rows serves fewer
    const size_t blocks = static_cast<size_t>(B) * (64 + 32 * K) +
                          static_cast<size_t>(kRowsM) * 16 * (pairs + 3 * n_rt);
    L.cand = part(K > 0 ? blocks * kCandFloats * 4 : 0);
  }
  L.total = at;
  return L;
}

struct ScoreOut {
  float* logp;
  float* entropy;
  float* lse;
  int32_t* top_token;
  float* top_logp;
};

void score_merge_params(ScoreMergeParams* mp, const detlm_head* h, const ScoreLayout& L, int64_t B,
                        int K, float inv_t, const int32_t* targets, const ScoreOut& out) {
  std::memset(mp, 0, sizeof(*mp));
  float* rec = reinterpret_cast<float*>(static_cast<uint8_t*>(h->sws) + L.rec);
  mp->V = static_cast<int32_t>(h->V);
  mp->n_vt = static_cast<int32_t>(L.n_vt);
  mp->logits = reinterpret_cast<const float*>(static_cast<uint8_t*>(h->sws) + L.logits);
  mp->ld = L.ld;
  mp->B = static_cast<int32_t>(B);
  mp->K = K;
  mp->c = kLog2eScore * inv_t;
  mp->inv_t = inv_t;
  mp->rec_m = rec;
  mp->rec_s = rec + L.rec_part;
  mp->rec_u = rec + 2 * L.rec_part;
  mp->targets = targets;
  mp->logp = out.logp;
  mp->entropy = out.entropy;
  mp->lse = out.lse;
  mp->top_token = out.top_token;
  mp->top_logp = out.top_logp;
  mp->err = h->d_err;
}

int score_narrow(detlm_head* h, const void* h_dev, const int32_t* targets, int64_t B, int K,
                 float inv_t, const ScoreOut& out, cudaStream_t stream) {
  const int N = cols_for(B);
  CUtensorMap tmH;
  if (!encode_2d(&tmH, h->dtype, h_dev, h->d, B, static_cast<uint32_t>(N))) return DETLM_EINVAL;
  const ScoreLayout L = score_layout(h, B, K, 0);
  int st = ensure_buffer(&h->sws, &h->sws_bytes, L.total, stream);
  if (st != DETLM_OK) return st;
  const void* W = nullptr;
  st = padded_weights(h, stream, &W);
  if (st != DETLM_OK) return st;
  CUtensorMap tmW;
  if (!encode_box(&tmW, map_type(h->dtype), W, h->d, h->V, padded_d(h) * 2, 64, kBM,
                  CU_TENSOR_MAP_SWIZZLE_128B, true))
    return DETLM_EINVAL;
  uint8_t* ws = static_cast<uint8_t*>(h->sws);
  float* rec = reinterpret_cast<float*>(ws + L.rec);
  HeadParams p;
  std::memset(&p, 0, sizeof(p));
  p.V = static_cast<int32_t>(h->V);
  p.d = static_cast<int32_t>(h->d);
  p.B = static_cast<int32_t>(B);
  p.N = N;
  p.nk = h->nk;
  p.n_chunks = static_cast<int32_t>((h->d + kScoreChunkK - 1) / kScoreChunkK);
  p.n_vt = h->n_vt;
  p.n_nt = 1;
  p.n_slots = slots_for(N);
  p.stages = stages_for(N);
  p.n_issuers = 1;
  p.tmem_cols = tmem_cols_for(p.n_slots * N);
  p.idesc = idesc_f16(h->dtype == DETLM_BF16 ? 1u : 0u, kBM, static_cast<uint32_t>(N));
  p.logits = reinterpret_cast<float*>(ws + L.logits);
  p.rec_m = rec;
  p.rec_s = rec + L.rec_part;
  p.rec_i = reinterpret_cast<int32_t*>(rec + 2 * L.rec_part);
  p.err = h->d_err;
  p.stall = h->stall;
  p.timeout_ns = h->timeout_ns;
  p.temperature = kLog2eScore * inv_t;
  const int grid = p.n_vt < h->num_sms ? p.n_vt : h->num_sms;
  time_start(h, stream);
  cudaError_t e = launch_gemm<MODE_SCORE>(tmW, tmH, p, grid, smem_layout(N, p.stages).total + 1024,
                                          stream);
  time_stop(h, stream);
  if (e != cudaSuccess) return status_from_cuda(e);
  ScoreMergeParams mp;
  score_merge_params(&mp, h, L, B, K, inv_t, targets, out);
  return status_from_cuda(launch_dependent(score_logits_kernel<kBM>, static_cast<unsigned>(B),
                                           kScoreThreads, stream, mp));
}

int score_wide(detlm_head* h, const void* h_dev, const int32_t* targets, int64_t B, int K,
               float inv_t, const ScoreOut& out, cudaStream_t stream) {
  int pairs = 0;
  cudaError_t e = op_pairs(h, &pairs);
  if (e != cudaSuccess) return status_from_cuda(e);
  const ScoreLayout L = score_layout(h, B, K, pairs);
  int st = ensure_buffer(&h->sws, &h->sws_bytes, L.total, stream);
  if (st != DETLM_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(h->sws);
  const void* W = nullptr;
  st = padded_weights(h, stream, &W);
  if (st != DETLM_OK) return st;
  const void* rows = h_dev;
  if (needs_padding(h)) {
    rows = ws + L.rows;
    st = pad_rows(h, h_dev, ws + L.rows, B, stream);
    if (st != DETLM_OK) return st;
  }
  CUtensorMap tmH, tmW;
  const CUtensorMapDataType t16 = map_type(h->dtype);
  if (!encode_box(&tmH, t16, rows, h->d, B, padded_d(h) * 2, 64, kRowsHalf, CU_TENSOR_MAP_SWIZZLE_128B,
                  true) ||
      !encode_box(&tmW, t16, W, h->d, h->V, padded_d(h) * 2, 64, kRowsHalf, CU_TENSOR_MAP_SWIZZLE_128B,
                  true))
    return DETLM_EINVAL;
  const int64_t n_vt = L.n_vt, n_rt = (B + kRowsM - 1) / kRowsM;
  if (n_vt * n_rt >= (int64_t{1} << 31)) return DETLM_EINVAL;
  PairOpParams p;
  std::memset(&p, 0, sizeof(p));
  p.B = static_cast<int32_t>(B);
  p.V = static_cast<int32_t>(h->V);
  p.n1 = static_cast<int32_t>(n_rt);
  p.nk = h->nk;
  p.seg = p.nk;
  p.units = static_cast<int32_t>(n_vt * n_rt);
  p.idesc = idesc_f16(h->dtype == DETLM_BF16 ? 1u : 0u, kRowsM, kRowsN);
  p.K = K;
  p.C = cand_blocks(pairs, n_rt, K);
  p.c = kLog2eScore * inv_t;
  p.inv_t = inv_t;
  p.rec_part = static_cast<int64_t>(L.rec_part);
  p.s.rec = reinterpret_cast<float*>(ws + L.rec);
  p.s.zt = reinterpret_cast<float*>(ws + L.zt);
  p.s.targets = targets;
  p.s.words = reinterpret_cast<int32_t*>(ws + L.words);
  ScoreMergeParams mp;
  score_merge_params(&mp, h, L, B, K, inv_t, targets, out);
  if (score_has_logits(h, B, K)) {
    CUtensorMap zOut;
    if (!encode_box(&zOut, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, ws + L.logits, L.ld, B, L.ld * 4, 32, 32,
                    CU_TENSOR_MAP_SWIZZLE_128B, false))
      return DETLM_EINVAL;
    time_start(h, stream);
    e = launch_pairop<OP_SCOREZ>(h, tmH, tmW, zOut, p, stream);
    time_stop(h, stream);
    if (e != cudaSuccess) return status_from_cuda(e);
    return status_from_cuda(launch_dependent(score_logits_kernel<kRowsN>, static_cast<unsigned>(B),
                                             kScoreThreads, stream, mp));
  }
  p.s.cand = reinterpret_cast<float*>(ws + L.cand);
  p.s.tile_over = reinterpret_cast<const int32_t*>(ws + L.tiles);
  if (K > 0) {
    e = cudaMemsetAsync(ws + L.words, 0, L.words_bytes, stream);
    if (e != cudaSuccess) return status_from_cuda(e);
  }
  time_start(h, stream);
  e = launch_pairop<OP_SCORE>(h, tmH, tmW, tmH, p, stream);
  time_stop(h, stream);
  if (e != cudaSuccess) return status_from_cuda(e);
  mp.C = p.C;
  mp.zt = p.s.zt;
  mp.cand = p.s.cand;
  mp.words = p.s.words;
  mp.tile_over = reinterpret_cast<int32_t*>(ws + L.tiles);
  e = launch_dependent(score_wide_kernel, static_cast<unsigned>(B), kScoreThreads, stream, mp);
  if (e != cudaSuccess) return status_from_cuda(e);
  // a row's list can overflow only where it is shorter than all its blocks
  if (K == 0 || 16 * n_vt <= p.C) return DETLM_OK;
  e = launch_pairop<OP_SELECT>(h, tmH, tmW, tmH, p, stream);
  if (e != cudaSuccess) return status_from_cuda(e);
  const int64_t blocks = (B + 15) / 16 < 2 * h->num_sms ? (B + 15) / 16 : 2 * h->num_sms;
  return status_from_cuda(launch_dependent(score_select_kernel, static_cast<unsigned>(blocks),
                                           kScoreThreads, stream, mp));
}

// ---------------------------------------------------------------- gradient
// The vocabulary is passed over in pieces of whole 16384-entry segments, as
// many as keep dz within kGradPassBytes (one at least).
struct GradLayout {
  int64_t pass;             // vocabulary entries of a pass
  int64_t ld;               // dz row stride, elements
  int64_t rows_pad, n_rt, n_dt;
  size_t scale, coef, rows, starts, list, sums, dz, part, acc, total;
};
GradLayout grad_layout(const detlm_head* h, int64_t B, int pairs) {
  GradLayout L;
  const int64_t segs = (h->V + kGradSeg - 1) / kGradSeg;
  int64_t per = kGradPassBytes / (2 * kGradSeg * B);
  per = per < 1 ? 1 : per > segs ? segs : per;
  L.pass = per * kGradSeg;
  const int64_t entries = L.pass < h->V ? L.pass : h->V;
  L.ld = (entries + 63) / 64 * 64;
  L.n_rt = (B + 255) / 256;
  L.n_dt = (h->d + 255) / 256;
  L.rows_pad = L.n_rt * 256;
  size_t at = 0;
  auto part = [&](size_t bytes) {
    const size_t a = at;
    at += round256(bytes);
    return a;
  };
  L.scale = part(8);
  L.coef = part(static_cast<size_t>(B) * 4);
  if (needs_padding(h)) L.rows = part(static_cast<size_t>(B) * padded_d(h) * 2);
  L.starts = part(static_cast<size_t>((entries + 255) / 256 * 256 + 1) * 4);
  L.list = part(static_cast<size_t>(B) * 4);
  L.sums = part(static_cast<size_t>(B) * h->d * 4);
  L.dz = part(static_cast<size_t>(B) * L.ld * 2);
  // split (few units) or whole segments, whichever is used
  const bool split = per * L.n_rt * L.n_dt < 2 * pairs;
  const int64_t parts = split ? per * kSegChunks : per;
  L.part = part(static_cast<size_t>(parts) * L.rows_pad * h->d * 4);
  L.acc = part(L.pass < h->V ? static_cast<size_t>(B) * h->d * 4 : 0);
  L.total = at;
  return L;
}

// The most that any call of up to max_B rows needs. The layout grows with B but
// for two steps down: behind every multiple of 256 rows (a new tile of rows
// may end the split of segments, and with it seven eighths of the partial
// sums), and where the pass loses a segment.
size_t grad_reserve(const detlm_head* h, int64_t max_B, int pairs) {
  size_t need = 0;
  auto at = [&](int64_t b) {
    const size_t n = grad_layout(h, b, pairs).total;
    if (n > need) need = n;
  };
  for (int64_t b = max_B; b > 0; b = (b - 1) / 256 * 256) at(b);
  const int64_t segs = (h->V + kGradSeg - 1) / kGradSeg;
  for (int64_t per = 1; per <= segs; ++per) {
    const int64_t last = kGradPassBytes / (2 * kGradSeg * per);   // rows of passes of `per` segments
    if (last > 0 && last < max_B) at(last);
  }
  return need;
}

struct GradIn {
  const void* h;
  const int32_t* targets;
  const float *lse, *entropy, *dlogp, *dentropy;
};

int score_backward(detlm_head* h, const GradIn& in, int64_t B, float inv_t, void* dh, void* dW,
                   cudaStream_t stream) {
  int pairs = 0;
  cudaError_t e = op_pairs(h, &pairs);
  if (e != cudaSuccess) return status_from_cuda(e);
  const GradLayout L = grad_layout(h, B, pairs);
  int st = ensure_buffer(&h->gws, &h->gws_bytes, L.total, stream);
  if (st != DETLM_OK) return st;
  uint8_t* ws = static_cast<uint8_t*>(h->gws);
  const void* Wrows = nullptr;
  st = padded_weights(h, stream, &Wrows);
  if (st != DETLM_OK) return st;
  const void* hrows = in.h;
  if (needs_padding(h)) {
    hrows = ws + L.rows;
    st = pad_rows(h, in.h, ws + L.rows, B, stream);
    if (st != DETLM_OK) return st;
  }
  float* scale = h->dtype == DETLM_FP16 ? reinterpret_cast<float*>(ws + L.scale) : nullptr;
  void* dz = ws + L.dz;
  float* part = reinterpret_cast<float*>(ws + L.part);
  const CUtensorMapDataType t16 = map_type(h->dtype);
  const uint32_t idesc = idesc_f16(h->dtype == DETLM_BF16 ? 1u : 0u, 256, 256);
  const int64_t row = h->d * 2, prow = padded_d(h) * 2;   // bytes of a row, and of one loaded

  if (scale != nullptr) {
    const float h_max = 1.0f + std::log(static_cast<float>(h->V));
    e = launch_dependent(grad_scale_kernel, 1, 1024, stream, in.dlogp, in.dentropy, in.targets,
                         static_cast<int>(B), inv_t, h_max, scale);
    if (e != cudaSuccess) return status_from_cuda(e);
  }
  time_start(h, stream);
  for (int64_t v0 = 0; v0 < h->V; v0 += L.pass) {
    const int64_t vc = h->V - v0 < L.pass ? h->V - v0 : L.pass;
    const uint8_t* W = static_cast<const uint8_t*>(Wrows) + v0 * prow;
    const int64_t n_vt = (vc + 255) / 256;
    const int64_t vboxes = (vc + 63) / 64;
    CUtensorMap hK, wK, zOut, zK, wN, pOut, zN, hN, dwOut;
    if (!encode_box(&hK, t16, hrows, h->d, B, prow, 64, a_box_rows(B), CU_TENSOR_MAP_SWIZZLE_128B, true) ||
        !encode_box(&wK, t16, W, h->d, vc, prow, 64, 128, CU_TENSOR_MAP_SWIZZLE_128B, true) ||
        !encode_box(&zOut, t16, dz, vc, B, L.ld * 2, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B, false))
      return DETLM_EINVAL;
    PairOpParams p;
    std::memset(&p, 0, sizeof(p));
    p.B = static_cast<int32_t>(B);
    p.V = static_cast<int32_t>(vc);
    p.n1 = static_cast<int32_t>(L.n_rt);
    p.nk = h->nk;
    p.seg = p.nk;
    p.units = static_cast<int32_t>(n_vt * L.n_rt);
    p.idesc = idesc;
    p.K = static_cast<int32_t>(h->V);
    p.t_off = static_cast<int32_t>(v0);
    p.inv_t = inv_t;
    p.coef = reinterpret_cast<float*>(ws + L.coef);
    p.g.lse = in.lse;
    p.g.entropy = in.entropy;
    p.g.dlogp = in.dlogp;
    p.g.dentropy = in.dentropy;
    p.g.targets = in.targets;
    p.g.scale = scale;
    // the targets' lists while little is in flight, their sums as soon as
    // OP_DZ has the entries (300 x 32000 x 2048: 164.7 -> 161.1 us against both
    // behind the fold)
    TargetListParams tl;
    std::memset(&tl, 0, sizeof(tl));
    TargetSumParams ts;
    std::memset(&ts, 0, sizeof(ts));
    const bool runs = dW != nullptr && B > kFewRows;
    if (runs) {
      tl.targets = in.targets;
      tl.B = p.B;
      tl.v0 = p.t_off;
      tl.vc = p.V;
      tl.starts = reinterpret_cast<int32_t*>(ws + L.starts);
      tl.list = reinterpret_cast<int32_t*>(ws + L.list);
      e = launch_dependent(target_list_kernel, static_cast<unsigned>(n_vt), 256, stream, tl);
      if (e != cudaSuccess) return status_from_cuda(e);
      ts.targets = in.targets;
      ts.starts = tl.starts;
      ts.list = tl.list;
      ts.coef = p.coef;
      ts.h = static_cast<const uint4*>(in.h);
      ts.sums = reinterpret_cast<float*>(ws + L.sums);
      ts.n_vt = static_cast<int32_t>(n_vt);
      ts.v0 = p.t_off;
      ts.d8 = static_cast<int32_t>(h->d / 8);
      ts.fp16 = h->dtype == DETLM_FP16;
    }
    e = launch_pairop<OP_DZ>(h, hK, wK, zOut, p, stream);
    if (e != cudaSuccess) return status_from_cuda(e);
    if (runs) {
      e = launch_dependent(target_sum_kernel,
                           dim3(static_cast<unsigned>(B), static_cast<unsigned>((ts.d8 + 127) / 128)),
                           128, stream, ts);
      if (e != cudaSuccess) return status_from_cuda(e);
    }
    // OP_DH: whole segments per unit, or single chunks where those would leave
    // SMs idle; the fold adds either in the same order
    const int64_t seg_boxes = static_cast<int64_t>(kSegChunks) * kGradChunkBoxes;
    const int64_t segs = (vboxes + seg_boxes - 1) / seg_boxes;
    const bool split = (L.pass * L.n_rt * L.n_dt) / (seg_boxes * 64) < 2 * pairs;
    const int64_t per_part = split ? kGradChunkBoxes : seg_boxes;
    const int64_t parts = split ? (vboxes + per_part - 1) / per_part : segs;
    if (dh != nullptr) {
      if (!encode_box(&zK, t16, dz, vc, B, L.ld * 2, 64, a_box_rows(B), CU_TENSOR_MAP_SWIZZLE_128B, true) ||
          !encode_box(&wN, t16, W, h->d, vc, prow, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B, true) ||
          !encode_box(&pOut, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, part, h->d, parts * L.rows_pad,
                      h->d * 4, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B, false))
        return DETLM_EINVAL;
      PairOpParams q = p;
      q.n0 = static_cast<int32_t>(L.n_rt);
      q.n1 = static_cast<int32_t>(L.n_dt);
      q.nk = static_cast<int32_t>(vboxes);
      q.seg = static_cast<int32_t>(per_part);
      q.units = static_cast<int32_t>(parts * L.n_rt * L.n_dt);
      q.K = static_cast<int32_t>(h->d);
      q.idesc = idesc | kIdescMnB;
      e = launch_pairop<OP_DH>(h, zK, wN, pOut, q, stream);
      if (e != cudaSuccess) return status_from_cuda(e);
      FoldParams f;
      std::memset(&f, 0, sizeof(f));
      f.part = part;
      f.rows_pad = L.rows_pad;
      f.B = static_cast<int32_t>(B);
      f.d4 = static_cast<int32_t>(h->d / 4);
      f.n_part = static_cast<int32_t>(parts);
      f.per_seg = split ? kSegChunks : 1;
      f.acc = reinterpret_cast<float*>(ws + L.acc);
      f.first = v0 == 0;
      f.last = v0 + L.pass >= h->V;
      f.fp16 = h->dtype == DETLM_FP16;
      f.scale = scale;
      f.targets = in.targets;
      f.coef = p.coef;
      f.W = h->W;
      f.V = static_cast<int32_t>(h->V);
      f.out = static_cast<uint32_t*>(dh);
      const int64_t blocks = (B * f.d4 + 255) / 256;
      e = launch_dependent(grad_fold_kernel, static_cast<unsigned>(blocks), 256, stream, f);
      if (e != cudaSuccess) return status_from_cuda(e);
    }
    if (dW != nullptr) {
      uint8_t* out = static_cast<uint8_t*>(dW) + v0 * row;
      if (!encode_box(&zN, t16, dz, vc, B, L.ld * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B, true) ||
          !encode_box(&hN, t16, hrows, h->d, B, prow, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B, true) ||
          !encode_box(&dwOut, t16, out, h->d, vc, row, 64, 32, CU_TENSOR_MAP_SWIZZLE_128B, false))
        return DETLM_EINVAL;
      PairOpParams q = p;
      q.n1 = static_cast<int32_t>(L.n_dt);
      q.nk = static_cast<int32_t>((B + 63) / 64);
      q.seg = q.nk;
      q.units = static_cast<int32_t>(n_vt * L.n_dt);
      q.K = static_cast<int32_t>(h->d);
      q.idesc = idesc | kIdescMnA | kIdescMnB;
      q.w.targets = in.targets;
      q.w.starts = tl.starts;
      q.w.sums = ts.sums;
      q.w.h = in.h;
      q.w.scale = scale;
      e = B > kFewRows ? launch_pairop<OP_DW>(h, zN, hN, dwOut, q, stream)
                       : launch_pairop<OP_DW_FEW>(h, zN, hN, dwOut, q, stream);
      if (e != cudaSuccess) return status_from_cuda(e);
    }
  }
  time_stop(h, stream);
  return DETLM_OK;
}

template <int NB>
cudaError_t launch_int8_rows(const detlm_head* h, const Int8RowsParams& p, cudaStream_t stream) {
  cudaError_t e = prepare_kernel<int8_rows_kernel<NB>>(0);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  const int64_t groups = (h->V + kI8RowsGroup - 1) / kI8RowsGroup;
  cfg.gridDim = dim3(static_cast<unsigned>(groups < 2 * h->num_sms ? groups : 2 * h->num_sms));
  cfg.blockDim = dim3(kI8RowsThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(NB) * h->d;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, int8_rows_kernel<NB>, p);
}

// Shares of K of the register-streaming kernel: at least four steps each (or
// one share), at most sixteen (exact fp32 sums).
int int8_regs_shares(int steps) {
  int wk = 1;
  while (wk < 16 && steps >= 8 * wk) wk *= 2;
  return wk;
}

cudaError_t launch_int8_regs(const detlm_head* h, const Int8RegsParams& p, cudaStream_t stream) {
  cudaError_t e = prepare_kernel<int8_regs_kernel>(0);
  if (e != cudaSuccess) return e;
  const int rows = 32 * (16 / p.wk);
  const int64_t rounds = (h->V + rows - 1) / rows;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>(rounds < h->num_sms ? rounds : h->num_sms));
  cfg.blockDim = dim3(kI8RegsThreads);
  cfg.dynamicSmemBytes = int8_regs_smem(p.steps, p.wk);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, int8_regs_kernel, p);
}

// (log2(e) / T, the larger, scales the differences of logits)
bool bad_temperature(float t) {
  return !(t > 0.0f) || !std::isfinite(t) || !std::isfinite(kLog2eScore * (1.0f / t));
}

}  // namespace

extern "C" {

int detlm_head_weights_changed(detlm_head_t* h, cudaStream_t stream) {
  if (h == nullptr) return DETLM_EINVAL;
  // the copies that calls (and graphs) may already read, in place; a copy that
  // is not filled yet is filled by the call that needs it
  if (h->w16_ready) {
    const cudaError_t e = i8_to_f16(h->W, h->W16, static_cast<size_t>(h->V) * h->d, stream);
    if (e != cudaSuccess) return status_from_cuda(e);
  }
  if (h->wp_ready) {
    const int st = pad_rows(h, h->W, h->Wp, h->V, stream);
    if (st != DETLM_OK) return st;
  }
  return weights_fence(stream);
}

int detlm_head_reserve_score(detlm_head_t* h, int64_t max_B, int top_k) {
  if (h == nullptr || bad_B(max_B) || top_k < 0 || top_k > kTopMax) return DETLM_EINVAL;
  if (h->P > 1 || !is_float(h)) return DETLM_EUNSUPPORTED;
  if (max_B == 0) return DETLM_OK;
  int pairs = 0;
  const cudaError_t e = op_pairs(h, &pairs);
  if (e != cudaSuccess) return status_from_cuda(e);
  // each kind of call's workspace grows with its rows
  size_t need = 0;
  for (const int64_t most : {static_cast<int64_t>(kNarrowRows), logit_rows(h), max_B}) {
    const size_t n = score_layout(h, most < max_B ? most : max_B, top_k, pairs).total;
    if (n > need) need = n;
  }
  const int st = ensure_buffer(&h->sws, &h->sws_bytes, need, nullptr);
  return st == DETLM_OK ? reserve_weights(h) : st;
}

int detlm_head_score(detlm_head_t* h, const void* h_dev, const int32_t* targets_dev, int64_t B,
                     int top_k, float temperature, float* logp_dev, float* entropy_dev,
                     float* lse_dev, int32_t* top_token_dev, float* top_logp_dev,
                     cudaStream_t stream) {
  if (h == nullptr || bad_B(B) || bad_temperature(temperature)) return DETLM_EINVAL;
  if (h->P > 1) return DETLM_EUNSUPPORTED;   // a vocabulary shard: the *_shard calls
  if (!is_float(h)) return DETLM_EUNSUPPORTED;
  if (top_k < 0 || top_k > kTopMax || top_k > h->V) return DETLM_EINVAL;
  if (B == 0) return DETLM_OK;
  if (h_dev == nullptr || !aligned(h_dev, 16)) return DETLM_EINVAL;
  if ((targets_dev == nullptr) != (logp_dev == nullptr)) return DETLM_EINVAL;
  if (!aligned(targets_dev, 4) || !aligned(logp_dev, 4)) return DETLM_EINVAL;
  if (!aligned(entropy_dev, 4) || !aligned(lse_dev, 4)) return DETLM_EINVAL;
  if (top_k > 0 && (top_token_dev == nullptr || top_logp_dev == nullptr ||
                    !aligned(top_token_dev, 4) || !aligned(top_logp_dev, 4)))
    return DETLM_EINVAL;
  const ScoreOut out{logp_dev, entropy_dev, lse_dev, top_token_dev, top_logp_dev};
  const float inv_t = 1.0f / temperature;
  if (B <= kNarrowRows)
    return score_narrow(h, h_dev, targets_dev, B, top_k, inv_t, out, stream);
  return score_wide(h, h_dev, targets_dev, B, top_k, inv_t, out, stream);
}

int detlm_head_reserve_backward(detlm_head_t* h, int64_t max_B) {
  if (h == nullptr || bad_B(max_B)) return DETLM_EINVAL;
  if (h->P > 1 || !is_float(h)) return DETLM_EUNSUPPORTED;
  if (max_B == 0) return DETLM_OK;
  int pairs = 0;
  const cudaError_t e = op_pairs(h, &pairs);
  if (e != cudaSuccess) return status_from_cuda(e);
  const size_t need = grad_reserve(h, max_B, pairs);
  const int st = ensure_buffer(&h->gws, &h->gws_bytes, need, nullptr);
  return st == DETLM_OK ? reserve_weights(h) : st;
}

int detlm_head_score_backward(detlm_head_t* h, const void* h_dev, const int32_t* targets_dev,
                              int64_t B, float temperature, const float* lse_dev,
                              const float* entropy_dev, const float* dlogp_dev,
                              const float* dentropy_dev, void* dh_dev, void* dW_dev,
                              cudaStream_t stream) {
  if (h == nullptr || bad_B(B) || bad_temperature(temperature)) return DETLM_EINVAL;
  if (h->P > 1) return DETLM_EUNSUPPORTED;
  if (!is_float(h)) return DETLM_EUNSUPPORTED;
  if (!aligned(dh_dev, 16) || !aligned(dW_dev, 16)) return DETLM_EINVAL;
  if (B == 0) {   // no rows: the weight's gradient is zero
    if (dW_dev == nullptr) return DETLM_OK;
    return status_from_cuda(cudaMemsetAsync(dW_dev, 0, static_cast<size_t>(h->V) * h->d * 2, stream));
  }
  if (dh_dev == nullptr && dW_dev == nullptr) return DETLM_OK;
  if (h_dev == nullptr || !aligned(h_dev, 16)) return DETLM_EINVAL;
  if (targets_dev == nullptr || !aligned(targets_dev, 4)) return DETLM_EINVAL;
  if (lse_dev == nullptr || !aligned(lse_dev, 4)) return DETLM_EINVAL;
  if (dlogp_dev == nullptr || !aligned(dlogp_dev, 4)) return DETLM_EINVAL;
  if (dentropy_dev != nullptr && (entropy_dev == nullptr || !aligned(entropy_dev, 4) ||
                                  !aligned(dentropy_dev, 4)))
    return DETLM_EINVAL;
  const GradIn in{h_dev, targets_dev, lse_dev, entropy_dev, dlogp_dev, dentropy_dev};
  return score_backward(h, in, B, 1.0f / temperature, dh_dev, dW_dev, stream);
}

int detlm_head_scaled_logits(detlm_head_t* h, const int8_t* q_dev, const float* x_scale_dev,
                             const float* w_scale_dev, int64_t B, int out_dtype, void* out_dev,
                             cudaStream_t stream) {
  if (h == nullptr || bad_B(B)) return DETLM_EINVAL;
  if (h->P > 1) return DETLM_EUNSUPPORTED;   // a vocabulary shard: the *_shard calls
  if (h->dtype != DETLM_INT8) return DETLM_EUNSUPPORTED;
  int type = 0;
  if (!out_type(out_dtype, &type)) return DETLM_EINVAL;
  const int size = type == OUT_F32 ? 4 : 2;
  if (B == 0) return DETLM_OK;
  if (q_dev == nullptr || !aligned(q_dev, 16)) return DETLM_EINVAL;
  if (x_scale_dev == nullptr || !aligned(x_scale_dev, 4)) return DETLM_EINVAL;
  if (w_scale_dev == nullptr || !aligned(w_scale_dev, 4)) return DETLM_EINVAL;
  if (out_dev == nullptr || !aligned(out_dev, static_cast<size_t>(size))) return DETLM_EINVAL;
  cudaError_t e;
  if (B <= kI8RowsMax) {
    Int8RowsParams p;
    p.W = static_cast<const int8_t*>(h->W);
    p.q = q_dev;
    p.x_scale = x_scale_dev;
    p.w_scale = w_scale_dev;
    p.out = out_dev;
    p.V = static_cast<int32_t>(h->V);
    p.d = static_cast<int32_t>(h->d);
    p.B = static_cast<int32_t>(B);
    p.type = type;
    time_start(h, stream);
    e = B == 1   ? launch_int8_rows<1>(h, p, stream)
        : B == 2 ? launch_int8_rows<2>(h, p, stream)
                 : launch_int8_rows<4>(h, p, stream);
    time_stop(h, stream);
    return status_from_cuda(e);
  }
  if (B <= kI8RegsMax) {
    Int8RegsParams p;
    p.W = static_cast<const int8_t*>(h->W);
    p.q = q_dev;
    p.x_scale = x_scale_dev;
    p.w_scale = w_scale_dev;
    p.out = out_dev;
    p.V = static_cast<int32_t>(h->V);
    p.d = static_cast<int32_t>(h->d);
    p.B = static_cast<int32_t>(B);
    p.type = type;
    p.steps = static_cast<int32_t>((h->d + 63) / 64);
    p.wk = int8_regs_shares(p.steps);
    time_start(h, stream);
    e = launch_int8_regs(h, p, stream);
    time_stop(h, stream);
    return status_from_cuda(e);
  }
  if (B < kI8ScaledWideB) {
    const int N = int8_cols_for(B, h->d);
    CUtensorMap tmH;
    if (!encode_2d(&tmH, DETLM_INT8, q_dev, h->d, B, static_cast<uint32_t>(N))) return DETLM_EINVAL;
    Int8Params p;
    if (!int8_params(h, B, N, &p)) return DETLM_EINVAL;
    p.logits = static_cast<int32_t*>(out_dev);
    p.out_type = type;
    p.x_scale = x_scale_dev;
    p.w_scale = w_scale_dev;
    const int64_t units = static_cast<int64_t>(p.n_vt) * p.n_nt;
    const int grid = static_cast<int>(units < h->num_sms ? units : h->num_sms);
    time_start(h, stream);
    e = launch_int8_n<true>(N, h->tmW, tmH, p, grid, int8_layout(N, p.stages).total + 1024, stream);
    time_stop(h, stream);
    return status_from_cuda(e);
  }
  const int st = ensure_wide(h, B, stream);
  if (st != DETLM_OK) return st;
  const size_t words = static_cast<size_t>(B) * h->d / 16;
  e = launch_dependent(rows_to_f16_kernel, copy_grid(h, static_cast<int64_t>(words)), 256, stream,
                       reinterpret_cast<const uint4*>(q_dev), static_cast<uint4*>(h->h16), words);
  if (e != cudaSuccess) return status_from_cuda(e);
  CUtensorMap tmH;
  if (!encode_2d(&tmH, DETLM_FP16, h->h16, h->d, B, a_box_rows(B))) return DETLM_EINVAL;
  int pairs = 0;
  e = op_pairs(h, &pairs);
  if (e != cudaSuccess) return status_from_cuda(e);
  const int64_t n_vt = tiles256(h->V), n_rt = (B + kRowsM - 1) / kRowsM;
  if (n_vt * n_rt >= (int64_t{1} << 31)) return DETLM_EINVAL;
  PairOpParams p;
  std::memset(&p, 0, sizeof(p));
  p.B = static_cast<int32_t>(B);
  p.V = static_cast<int32_t>(h->V);
  p.n1 = static_cast<int32_t>(n_rt);
  p.nk = static_cast<int32_t>((h->d + 63) / 64);
  p.seg = p.nk;
  p.units = static_cast<int32_t>(n_vt * n_rt);
  p.idesc = idesc_f16(0u, kRowsM, kRowsN);
  p.q.x_scale = x_scale_dev;
  p.q.w_scale = w_scale_dev;
  p.q.out = out_dev;
  p.q.type = type;
  CUtensorMap tmO = tmH;   // not read unless it is valid
  p.q.tma = encode_out(&tmO, type, out_dev, h->V, B) ? 1 : 0;
  time_start(h, stream);
  e = p.nk <= 2 * kScaledChunkBoxes ? launch_pairop<OP_SCALED2>(h, tmH, h->tmW16, tmO, p, stream)
                                : launch_pairop<OP_SCALED>(h, tmH, h->tmW16, tmO, p, stream);
  time_stop(h, stream);
  return status_from_cuda(e);
}

}  // extern "C"
