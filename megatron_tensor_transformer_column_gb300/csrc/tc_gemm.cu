// tc_gemm.cu -- the tensor-core GEMM's kernels, one symbol per launch kind
// (body: tc_gemm_body.cuh; the launches with 8-bit checkpoints:
// tc_gemm_ckpt8.cu), and their launcher.
#include <mutex>

#include "tc_gemm_body.cuh"

namespace tpmlp {

// Launch kinds whose epilogues carry the activation (the column GEMM, the
// dgrad GEMM) also exist with 16 epilogue warps (suffix _w16).  The host
// takes them where the tiles' K is short (tc_epi_warps_for): there the
// epilogue of a tile lasts longer than its main loop and is bound by each
// warp's chain of TMEM load, arithmetic and store, which more warps overlap.
// With longer K the epilogue hides under the next tile's main loop and the
// extra warps only compete with the producer and the MMA issuer for issue
// slots (measured on GB300: C2's column and dgrad launches -7 % and -5 % with
// 16 warps; C3 to C5's +1 to +3 %).
TPMLP_TC_KERNELS(tpmlp_fwd_column_gemm_act, 8, EPIS_ALL)
TPMLP_TC_KERNELS(tpmlp_fwd_column_gemm_act_w16, 16, EPIS_ALL)
TPMLP_TC_KERNELS(tpmlp_fwd_row_gemm_gsum, 8, EPIS_STORE)
TPMLP_TC_KERNELS(tpmlp_bwd_dgrad_act_wgrad2, 8, EPIS_ALL)
TPMLP_TC_KERNELS(tpmlp_bwd_dgrad_act_wgrad2_w16, 16, EPIS_ALL)
TPMLP_TC_KERNELS(tpmlp_bwd_dx_fsum_wgrad1, 8, EPIS_STORE)
TPMLP_TC_KERNELS(tpmlp_attn_qkv_proj, 8, EPIS_ALL)
TPMLP_TC_KERNELS(tpmlp_attn_out_proj_gsum, 8, EPIS_ALL)
TPMLP_TC_KERNELS(tpmlp_attn_out_proj_bwd, 8, EPIS_ALL)
TPMLP_TC_KERNELS(tpmlp_attn_qkv_bwd_dx_fsum, 8, EPIS_ALL)

int tc_gemm_max_smem_bytes() { return kSmemBytes; }

int tc_epi_warps_for(const GemmParams& p, int tag) {
  if (tag != TAG_FWD_COLUMN && tag != TAG_BWD_DGRAD) return 8;
  for (int i = 0; i < p.num_probs; ++i) {
    const Prob& P = p.probs[i];
    if (P.epi != EPI_STORE && P.kblocks > kShortKBlocks) return 8;
  }
  return 16;
}

using KernelFn = TcKernelFn;

KernelFn kernel_for(int tag, bool stream_k, int epi_warps) {
  const bool w16 = epi_warps == 16;
  switch (tag) {
    case TAG_FWD_COLUMN:
      return w16 ? (stream_k ? tpmlp_fwd_column_gemm_act_w16_sk : tpmlp_fwd_column_gemm_act_w16)
                 : (stream_k ? tpmlp_fwd_column_gemm_act_sk : tpmlp_fwd_column_gemm_act);
    case TAG_FWD_ROW: return stream_k ? tpmlp_fwd_row_gemm_gsum_sk : tpmlp_fwd_row_gemm_gsum;
    case TAG_BWD_DGRAD:
      return w16 ? (stream_k ? tpmlp_bwd_dgrad_act_wgrad2_w16_sk : tpmlp_bwd_dgrad_act_wgrad2_w16)
                 : (stream_k ? tpmlp_bwd_dgrad_act_wgrad2_sk : tpmlp_bwd_dgrad_act_wgrad2);
    case TAG_BWD_FSUM: return stream_k ? tpmlp_bwd_dx_fsum_wgrad1_sk : tpmlp_bwd_dx_fsum_wgrad1;
    case TAG_ATTN_QKV: return stream_k ? tpmlp_attn_qkv_proj_sk : tpmlp_attn_qkv_proj;
    case TAG_ATTN_OUT: return stream_k ? tpmlp_attn_out_proj_gsum_sk : tpmlp_attn_out_proj_gsum;
    case TAG_ATTN_OUT_BWD: return stream_k ? tpmlp_attn_out_proj_bwd_sk : tpmlp_attn_out_proj_bwd;
    case TAG_ATTN_QKV_BWD: return stream_k ? tpmlp_attn_qkv_bwd_dx_fsum_sk : tpmlp_attn_qkv_bwd_dx_fsum;
    default: return nullptr;
  }
}

// Pairs (clusters of two CTAs) that can be resident at once on this device
// (every kernel has one CTA per SM: the same shared memory).
int tc_gemm_max_pairs(int tag) {
  static std::mutex mu;
  static int cache[64][kNumKernelTags] = {};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64 || tag < 0 || tag >= kNumKernelTags) return 0;
  std::lock_guard<std::mutex> lk(mu);
  if (cache[dev][tag] > 0) return cache[dev][tag];
  KernelFn k = kernel_for(tag, false, 8);
  if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes) != cudaSuccess) return 0;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2, 1, 1);
  cfg.blockDim = dim3(threads_for(8), 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess || n <= 0) return 0;
  cache[dev][tag] = n;
  return n;
}

int tc_gemm_grid_pairs(const GemmParams& p, int kernel_tag, int max_pairs_hint) {
  int pairs = tc_gemm_max_pairs(kernel_tag);
  if (pairs <= 0) pairs = max_pairs_hint > 0 ? max_pairs_hint : 1;
  return pairs < p.total_tiles ? pairs : p.total_tiles;
}

cudaError_t launch_tc_gemm(const GemmParams& p, int kernel_tag, int epi_warps, int max_pairs_hint,
                           cudaStream_t stream) {
  KernelFn k = p.ckpt8 ? tc_ckpt8_kernel(kernel_tag, p.sk.on != 0, epi_warps)
                       : kernel_for(kernel_tag, p.sk.on != 0, epi_warps);
  if (!k) return cudaErrorInvalidValue;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  // the stream-K ranges were cut for exactly p.sk.pairs pairs
  const int pairs = p.sk.on ? p.sk.pairs : tc_gemm_grid_pairs(p, kernel_tag, max_pairs_hint);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * pairs, 1, 1);
  cfg.blockDim = dim3(threads_for(epi_warps), 1, 1);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k, p);
}

}  // namespace tpmlp
