// block_host.cuh -- the host side of the e4m3 head: block quantisation and
// block-scaled logits. Part of detlm_head.cu's translation unit (it uses that
// file's handle and helpers, and score_host.cuh's).
#pragma once

namespace {

// The most rows of the kernel that reads W with vocabulary rows on the MMA's M
// axis (its N is at most 128 hidden rows).
constexpr int64_t kBlockNarrow = 128;

template <int NBLK>
cudaError_t launch_block_gemm(const CUtensorMap& w, const CUtensorMap& g, const CUtensorMap& x,
                              BlockParams p, int sms, cudaStream_t stream) {
  constexpr int N = 16 * NBLK, kps = block_kps(N);
  cudaError_t e = prepare_kernel<block_gemm_kernel<NBLK>>(0);
  if (e != cudaSuccess) return e;
  p.idesc = idesc_e4m3(kBM, N);
  p.slots = 512 / (kps * N) < kBlockMaxSlots ? 512 / (kps * N) : kBlockMaxSlots;
  p.stages = kBlockMaxStages;
  while (p.stages > 2 && block_layout(N, p.stages, p.nk).total + 1024u > kSmemLimit) --p.stages;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  const int64_t groups = (static_cast<int64_t>(p.V) + kBlockGroup - 1) / kBlockGroup;
  cfg.gridDim = dim3(static_cast<unsigned>(groups < sms ? groups : sms));
  cfg.blockDim = dim3(block_threads(N));
  cfg.dynamicSmemBytes = block_layout(N, p.stages, p.nk).total + 1024u;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, block_gemm_kernel<NBLK>, w, g, x, p);
}

cudaError_t launch_block_pair(detlm_head* h, const CUtensorMap& x, const CUtensorMap& w,
                              const CUtensorMap& o, BlockParams p, cudaStream_t stream) {
  cudaError_t e = prepare_kernel<block_pair_kernel>(kRegsLaunchWide);
  if (e != cudaSuccess) return e;
  int pairs = 0;
  e = op_pairs(h, &pairs);
  if (e != cudaSuccess) return e;
  p.idesc = idesc_e4m3(kRowsM, 128);
  p.stages = kBlockPairMaxStages;
  while (p.stages > 4 && block_pair_layout(p.stages).total + 1024u > kSmemLimit) --p.stages;
  cudaLaunchConfig_t cfg;
  std::memset(&cfg, 0, sizeof(cfg));
  cfg.blockDim = dim3(kRowsThreads);
  cfg.dynamicSmemBytes = block_pair_layout(p.stages).total + 1024u;
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
  return cudaLaunchKernelEx(&cfg, block_pair_kernel, x, w, o, p);
}

template <int FMT>
cudaError_t launch_quantize_blocks(const BlockQuantParams& p, int block_rows, cudaStream_t stream) {
  if (block_rows == kBQBlock) {
    const int64_t tiles = (p.B + kBQBlock - 1) / kBQBlock * p.nb;
    const cudaError_t e = launch_dependent(quantize_tiles_kernel<FMT>, dim3(static_cast<unsigned>(tiles)),
                                           kBQThreads, stream, p);
    if (e != cudaSuccess) return e;
    // a weight: calls of a head on it request its boxes before they wait
    weights_fence_kernel<<<1, 32, 0, stream>>>();
    return cudaGetLastError();
  }
  const int64_t per = kBQPer * (kBQThreads / 16);
  return launch_dependent(quantize_blocks_kernel<FMT>,
                          dim3(static_cast<unsigned>((p.B * p.nb + per - 1) / per)), kBQThreads, stream, p);
}

}  // namespace

extern "C" {

int detlm_quantize_blocks(const void* x_dev, int dtype, int64_t B, int64_t d, int block_rows,
                          void* q_dev, float* scale_dev, cudaStream_t stream) {
  if (dtype != DETLM_BF16 && dtype != DETLM_FP16 && dtype != DETLM_FP32) return DETLM_EINVAL;
  if (block_rows != 1 && block_rows != kBQBlock) return DETLM_EINVAL;
  if (bad_B(B) || d < 1 || d >= (int64_t{1} << 31) || d % 16 != 0) return DETLM_EINVAL;
  BlockQuantParams p;
  p.x = x_dev;
  p.B = B;
  p.d = d;
  p.nb = static_cast<int32_t>((d + kBQBlock - 1) / kBQBlock);
  p.q = static_cast<uint8_t*>(q_dev);
  p.scale = scale_dev;
  // (a launch has fewer than 2^31 blocks)
  if ((B + block_rows - 1) / block_rows * p.nb >= (int64_t{1} << 31)) return DETLM_EINVAL;
  if (B == 0) return DETLM_OK;
  if (x_dev == nullptr || !aligned(x_dev, 16)) return DETLM_EINVAL;
  if (q_dev == nullptr || !aligned(q_dev, 16)) return DETLM_EINVAL;
  if (scale_dev == nullptr || !aligned(scale_dev, 4)) return DETLM_EINVAL;
  return status_from_cuda(dtype == DETLM_BF16   ? launch_quantize_blocks<QF_BF16>(p, block_rows, stream)
                          : dtype == DETLM_FP16 ? launch_quantize_blocks<QF_FP16>(p, block_rows, stream)
                                                : launch_quantize_blocks<QF_FP32>(p, block_rows, stream));
}

int detlm_head_block_scaled_logits(detlm_head_t* h, const void* q_dev, const float* x_scale_dev,
                                   const float* w_scale_dev, int64_t B, int out_dtype,
                                   void* out_dev, cudaStream_t stream) {
  if (h == nullptr || bad_B(B)) return DETLM_EINVAL;
  if (h->dtype != DETLM_E4M3) return DETLM_EUNSUPPORTED;
  int type = 0;
  if (!out_type(out_dtype, &type)) return DETLM_EINVAL;
  const int size = type == OUT_F32 ? 4 : 2;
  if (B == 0) return DETLM_OK;
  if (q_dev == nullptr || !aligned(q_dev, 16)) return DETLM_EINVAL;
  if (x_scale_dev == nullptr || !aligned(x_scale_dev, 4)) return DETLM_EINVAL;
  if (w_scale_dev == nullptr || !aligned(w_scale_dev, 4)) return DETLM_EINVAL;
  if (out_dev == nullptr || !aligned(out_dev, static_cast<size_t>(size))) return DETLM_EINVAL;
  BlockParams p;
  std::memset(&p, 0, sizeof(p));
  p.x_scale = x_scale_dev;
  p.w_scale = w_scale_dev;
  p.out = out_dev;
  p.V = static_cast<int32_t>(h->V);
  p.B = static_cast<int32_t>(B);
  p.nk = static_cast<int32_t>((h->d + kBlockK - 1) / kBlockK);
  p.type = type;
  p.stall = h->stall;
  p.timeout_ns = h->timeout_ns;
  p.err = h->d_err;
  CUtensorMap tmX;
  if (!encode_2d(&tmX, DETLM_E4M3, q_dev, h->d, B, a_box_rows(B))) return DETLM_EINVAL;
  cudaError_t e = cudaErrorInvalidValue;
  if (B <= kBlockNarrow) {
    CUtensorMap tmG;
    if (!encode_2d(&tmG, DETLM_E4M3, h->W, h->d, h->V, kBlockGroup)) return DETLM_EINVAL;
    time_start(h, stream);
    switch ((B + 15) / 16) {
      case 1: e = launch_block_gemm<1>(h->tmW, tmG, tmX, p, h->num_sms, stream); break;
      case 2: e = launch_block_gemm<2>(h->tmW, tmG, tmX, p, h->num_sms, stream); break;
      case 3: e = launch_block_gemm<3>(h->tmW, tmG, tmX, p, h->num_sms, stream); break;
      case 4: e = launch_block_gemm<4>(h->tmW, tmG, tmX, p, h->num_sms, stream); break;
      case 5: case 6: e = launch_block_gemm<6>(h->tmW, tmG, tmX, p, h->num_sms, stream); break;
      default: e = launch_block_gemm<8>(h->tmW, tmG, tmX, p, h->num_sms, stream); break;
    }
    time_stop(h, stream);
    return status_from_cuda(e);
  }
  const int64_t n_rt = (B + kRowsM - 1) / kRowsM, units = tiles256(h->V) * n_rt;
  if (units >= (int64_t{1} << 31)) return DETLM_EINVAL;
  p.n1 = static_cast<int32_t>(n_rt);
  p.units = static_cast<int32_t>(units);
  CUtensorMap tmO = tmX;   // not read unless it is valid
  p.tma = encode_out(&tmO, type, out_dev, h->V, B) ? 1 : 0;
  CUtensorMap tmV;         // half a vocabulary tile: what one of the pair's CTAs loads of it
  if (!encode_2d(&tmV, DETLM_E4M3, h->W, h->d, h->V, 64)) return DETLM_EINVAL;
  time_start(h, stream);
  e = launch_block_pair(h, tmX, tmV, tmO, p, stream);
  time_stop(h, stream);
  return status_from_cuda(e);
}

}  // extern "C"
