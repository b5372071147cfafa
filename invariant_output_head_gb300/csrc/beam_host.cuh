// beam_host.cuh -- the host side of the beam-search step: argument checks,
// workspace and launches. Part of detlm_head.cu's translation unit.
#pragma once

namespace {

int beam_tiles(const detlm_head* h) { return static_cast<int>((h->V + kScanTile - 1) / kScanTile); }

// The scan's blocks: as many as run at once, with four tiles each at least (a
// block's cuts cost as much as a round) but one for each row, and so few that a
// row has at most kBeamPartsMax parts: G / rows + 2 of G blocks.
constexpr int64_t kScanLeast = 4;
int scan_blocks(const detlm_head* h, int64_t rows, int fmt) {
  const int64_t tiles = rows * beam_tiles(h), slots = static_cast<int64_t>(h->num_sms) * scan_resident(fmt);
  int64_t g = tiles / kScanLeast > rows ? tiles / kScanLeast : rows;
  if (g > slots) g = slots;
  if (g > rows * (kBeamPartsMax - 2)) g = rows * (kBeamPartsMax - 2);
  return static_cast<int>(g);
}
// The tiles' sums and the parts' lists of up to `rows` rows: at most G + 2 rows
// lists.
size_t beam_tile_bytes(const detlm_head* h, int64_t rows) {
  return round256(static_cast<size_t>(rows) * beam_tiles(h) * sizeof(float2));
}
size_t beam_bytes(const detlm_head* h, int64_t rows, int n_out) {
  const int64_t most = static_cast<int64_t>(h->num_sms) * scan_resident(QF_BF16);
  const int64_t lists = (rows * (kBeamPartsMax - 2) < most ? rows * (kBeamPartsMax - 2) : most) + 2 * rows;
  return beam_tile_bytes(h, rows) + static_cast<size_t>(lists) * n_out * sizeof(u64);
}

template <int FMT>
cudaError_t launch_beam_scan(const BeamScanParams& p, int blocks, cudaStream_t stream) {
  return launch_dependent(beam_scan_kernel<FMT>, dim3(static_cast<unsigned>(blocks)), kScanThreads, stream, p);
}

template <int KB>
cudaError_t launch_beam_reorder(const ReorderParams& p, unsigned blocks, cudaStream_t stream) {
  const unsigned y = static_cast<unsigned>(p.n_seq < 65535 ? p.n_seq : 65535);
  return launch_dependent(beam_reorder_kernel<KB>, dim3(blocks, y), kReorderThreads, stream, p);
}

}  // namespace

extern "C" {

int detlm_head_reserve_beams(detlm_head_t* h, int64_t max_rows, int n_out) {
  if (h == nullptr || bad_B(max_rows) || n_out < 1 || n_out > kBeamOutMax) return DETLM_EINVAL;
  if (h->P > 1) return DETLM_EUNSUPPORTED;
  if (max_rows == 0) return DETLM_OK;
  return ensure_buffer(&h->bws, &h->bws_bytes, beam_bytes(h, max_rows, n_out), nullptr);
}

int detlm_head_beam_select(detlm_head_t* h, const void* logits_dev, int logits_dtype,
                           const float* score_dev, const uint8_t* finished_dev, int32_t end_token,
                           int64_t n_seq, int beams, int n_out, float temperature,
                           int32_t* parent_dev, int32_t* token_dev, float* out_score_dev,
                           cudaStream_t stream) {
  if (h == nullptr || bad_B(n_seq) || bad_temperature(temperature)) return DETLM_EINVAL;
  if (h->P > 1) return DETLM_EUNSUPPORTED;   // a vocabulary shard has part of the logits
  if (beams < 1 || beams > kBeamMax || n_out < 1 || n_out > kBeamOutMax) return DETLM_EINVAL;
  if (n_seq * beams >= (int64_t{1} << 31)) return DETLM_EINVAL;
  int type = 0;
  if (!out_type(logits_dtype, &type)) return DETLM_EINVAL;
  if (finished_dev != nullptr && (end_token < 0 || end_token >= h->V)) return DETLM_EINVAL;
  if (n_seq == 0) return DETLM_OK;
  if (logits_dev == nullptr || !aligned(logits_dev, type == OUT_F32 ? 4 : 2)) return DETLM_EINVAL;
  if (score_dev == nullptr || !aligned(score_dev, 4)) return DETLM_EINVAL;
  if (parent_dev == nullptr || !aligned(parent_dev, 4)) return DETLM_EINVAL;
  if (token_dev == nullptr || !aligned(token_dev, 4)) return DETLM_EINVAL;
  if (out_score_dev == nullptr || !aligned(out_score_dev, 4)) return DETLM_EINVAL;
  const int64_t rows = n_seq * beams;
  const int st = ensure_buffer(&h->bws, &h->bws_bytes, beam_bytes(h, rows, n_out), stream);
  if (st != DETLM_OK) return st;
  BeamScanParams p;
  std::memset(&p, 0, sizeof(p));
  p.logits = logits_dev;
  p.score = score_dev;
  p.finished = finished_dev;
  p.tile = static_cast<float2*>(h->bws);
  p.best = reinterpret_cast<u64*>(static_cast<uint8_t*>(h->bws) + beam_tile_bytes(h, rows));
  p.V = static_cast<int32_t>(h->V);
  p.n_tiles = beam_tiles(h);
  p.tiles = rows * p.n_tiles;
  const int fmt = type == OUT_F32 ? QF_FP32 : type == OUT_BF16 ? QF_BF16 : QF_FP16;
  const int blocks = scan_blocks(h, rows, fmt);
  p.parts = static_cast<int32_t>(blocks / rows) + 2;
  p.M = n_out;
  const float inv_t = 1.0f / temperature;
  p.c = kLog2eScore * inv_t;
  cudaError_t e = fmt == QF_FP32   ? launch_beam_scan<QF_FP32>(p, blocks, stream)
                  : fmt == QF_BF16 ? launch_beam_scan<QF_BF16>(p, blocks, stream)
                                   : launch_beam_scan<QF_FP16>(p, blocks, stream);
  if (e != cudaSuccess) return status_from_cuda(e);
  BeamMergeParams m;
  std::memset(&m, 0, sizeof(m));
  m.score = score_dev;
  m.finished = finished_dev;
  m.tile = p.tile;
  m.best = p.best;
  m.parent = parent_dev;
  m.token = token_dev;
  m.out = out_score_dev;
  m.n_tiles = p.n_tiles;
  m.parts = p.parts;
  m.tiles = p.tiles;
  m.blocks = blocks;
  m.M = n_out;
  m.beams = beams;
  m.end_token = end_token;
  m.c = p.c;
  m.inv_t = inv_t;
  e = prepare_kernel<beam_merge_kernel>(0);
  if (e != cudaSuccess) return status_from_cuda(e);
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3(static_cast<unsigned>(n_seq));
  cfg.blockDim = dim3(kMergeBeamThreads);
  cfg.dynamicSmemBytes = merge_smem(beams, p.parts, n_out);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return status_from_cuda(cudaLaunchKernelEx(&cfg, beam_merge_kernel, m));
}

int detlm_beam_reorder(const detlm_beam_state_t* states, int n_states, const int32_t* parent_dev,
                       int64_t n_seq, int beams_in, int beams_out, int64_t used, cudaStream_t stream) {
  if (n_states < 0 || (n_states > 0 && states == nullptr) || bad_B(n_seq)) return DETLM_EINVAL;
  if (beams_in < 1 || beams_in > kBeamMax || beams_out < 1 || beams_out > kBeamMax) return DETLM_EINVAL;
  if (n_seq * beams_in >= (int64_t{1} << 31) || n_seq * beams_out >= (int64_t{1} << 31)) return DETLM_EINVAL;
  bool in_place = false;
  // bytes of each piece that move
  auto moved = [&](const detlm_beam_state_t& s) {
    if (used < 0 || s.position_bytes == 0) return s.seg_bytes;
    return used >= s.seg_bytes / s.position_bytes ? s.seg_bytes : used * s.position_bytes;
  };
  for (int i = 0; i < n_states; ++i) {
    const detlm_beam_state_t& s = states[i];
    if (s.n_seg < 0 || s.seg_bytes < 0 || s.position_bytes < 0) return DETLM_EINVAL;
    if (s.n_seg == 0 || s.seg_bytes == 0) continue;
    if (n_seq > 0 && (s.src == nullptr || s.dst == nullptr)) return DETLM_EINVAL;
    if (s.src == s.dst) {
      if (beams_in != beams_out || s.src_row != s.dst_row || s.src_seg != s.dst_seg) return DETLM_EINVAL;
      in_place = true;
    }
  }
  if (n_seq == 0) return DETLM_OK;
  if (n_states > 0 && (parent_dev == nullptr || !aligned(parent_dev, 4))) return DETLM_EINVAL;
  ReorderParams p;
  std::memset(&p, 0, sizeof(p));
  p.parent = parent_dev;
  p.n_seq = n_seq;
  p.beams_in = beams_in;
  p.beams_out = beams_out;
  uint64_t blocks = 0;
  auto launch = [&]() {
    const unsigned n = static_cast<unsigned>(blocks);
    cudaError_t e;
    if (beams_out <= 4) e = launch_beam_reorder<4>(p, n, stream);
    else if (beams_out <= 8 || !in_place) e = launch_beam_reorder<8>(p, n, stream);
    else if (beams_out <= 16) e = launch_beam_reorder<16>(p, n, stream);
    else e = launch_beam_reorder<32>(p, n, stream);
    p.n_states = 0;
    blocks = 0;
    return e;
  };
  for (int pass = 0; pass < 2; ++pass) {        // checked whole before the first launch
    for (int i = 0; i < n_states; ++i) {
      const detlm_beam_state_t& s = states[i];
      const int64_t bytes = moved(s);
      if (s.n_seg == 0 || bytes == 0) continue;
      // the widest column that every address of the state is a multiple of
      const uint64_t all = static_cast<uint64_t>(bytes) | reinterpret_cast<uintptr_t>(s.src) |
                           reinterpret_cast<uintptr_t>(s.dst) | static_cast<uint64_t>(s.src_row) |
                           static_cast<uint64_t>(s.dst_row) |
                           (s.n_seg > 1 ? static_cast<uint64_t>(s.src_seg) | static_cast<uint64_t>(s.dst_seg) : 0u);
      uint32_t grain = 16;
      while (all % grain != 0) grain /= 2;
      const uint64_t cols = static_cast<uint64_t>(bytes) / grain;
      // (columns are counted in 32 bits)
      if (cols >= (uint64_t{1} << 31) / static_cast<uint64_t>(s.n_seg)) return DETLM_EINVAL;
      if (pass == 0) continue;
      const uint64_t need = (cols * s.n_seg + kReorderThreads - 1) / kReorderThreads;
      if (p.n_states == kReorderStates || blocks + need >= (uint64_t{1} << 31)) {
        const cudaError_t e = launch();
        if (e != cudaSuccess) return status_from_cuda(e);
      }
      BeamState& o = p.state[p.n_states++];
      o.src = static_cast<const uint8_t*>(s.src);
      o.dst = static_cast<uint8_t*>(s.dst);
      o.row_src = s.src_row;
      o.row_dst = s.dst_row;
      o.seg_src = s.src_seg;
      o.seg_dst = s.dst_seg;
      o.cols = static_cast<uint32_t>(cols);
      o.n_seg = static_cast<uint32_t>(s.n_seg);
      o.grain = grain;
      o.block0 = static_cast<uint32_t>(blocks);
      blocks += need;
    }
  }
  return p.n_states > 0 ? status_from_cuda(launch()) : DETLM_OK;
}

}  // extern "C"
