// tc_gemm_ckpt8.cu -- the tensor-core GEMM's launches that keep their
// pre-activations as 8-bit checkpoints (format: ckpt8.cuh; body:
// tc_gemm_body.cuh): the column GEMM, whose epilogue writes them from the fp32
// accumulators, and the dgrad GEMM, whose epilogue reads them, takes act' of
// the kept values and recomputes H.
//
// Bound by the tensor cores like the launches they stand beside: an epilogue
// moves 1.0625 bytes per pre-activation instead of 2, with plain stores and
// loads of a warp's own block, and does about two instructions more for it.
#include "tc_gemm_body.cuh"

namespace tpmlp {

#define TPMLP_TC_CKPT8_KERNELS(name, EW) TPMLP_TC_KERNEL_PAIR(name, EW, true)

TPMLP_TC_CKPT8_KERNELS(tpmlp_fwd_column_gemm_act_ckpt8, 8)
TPMLP_TC_CKPT8_KERNELS(tpmlp_fwd_column_gemm_act_ckpt8_w16, 16)
TPMLP_TC_CKPT8_KERNELS(tpmlp_bwd_dgrad_act_ckpt8, 8)
TPMLP_TC_CKPT8_KERNELS(tpmlp_bwd_dgrad_act_ckpt8_w16, 16)

TcKernelFn tc_ckpt8_kernel(int tag, bool stream_k, int epi_warps) {
  const bool w16 = epi_warps == 16;
  switch (tag) {
    case TAG_FWD_COLUMN:
      return w16 ? (stream_k ? tpmlp_fwd_column_gemm_act_ckpt8_w16_sk : tpmlp_fwd_column_gemm_act_ckpt8_w16)
                 : (stream_k ? tpmlp_fwd_column_gemm_act_ckpt8_sk : tpmlp_fwd_column_gemm_act_ckpt8);
    case TAG_BWD_DGRAD:
      return w16 ? (stream_k ? tpmlp_bwd_dgrad_act_ckpt8_w16_sk : tpmlp_bwd_dgrad_act_ckpt8_w16)
                 : (stream_k ? tpmlp_bwd_dgrad_act_ckpt8_sk : tpmlp_bwd_dgrad_act_ckpt8);
    default: return nullptr;
  }
}

}  // namespace tpmlp
