// tc_gemm_ckpt8.cu -- the tensor-core GEMM's launches that keep their
// pre-activations as 8-bit checkpoints (format: ckpt8.cuh; body:
// tc_gemm_body.cuh): the column GEMM, whose epilogue writes them from the fp32
// accumulators, and the dgrad GEMM, whose epilogue reads them, takes act' of
// the kept values and recomputes H.
//
// The checkpoint is taken of the fp32 accumulator.  H and the activation
// gradients leave in bf16, as from the launches these stand beside: they are the
// next launch's tensor-core operands.  The weight and bias gradients therefore carry one
// rounding (2^-8) a term more than sums in 32 bits throughout would; against 64
// bits 2.4e-3 of their norm instead of 1.7e-3.
//
// Bound by the tensor cores like the launches they stand beside, or, with short
// K, by the epilogue: it moves 1.0625 bytes per pre-activation instead of 2,
// with plain stores and loads of a warp's own block, and a thread finds its
// row's largest magnitudes, scales and codes in about 35 instructions per 16
// elements.  Measured on GB300 (device time of the launch, against the one with
// bf16 pre-activations and, for dgrad, recomputed H):
//   GeLU, 8192 x 768, 4 x 768:          column 49 against 51 us, dgrad 57 against 68
//   GeLU, 8192 x 2048, 8192 hidden:     column 176 against 176 us, dgrad 190 against 200
//   SwiGLU, 8192 x 4096, 8 x 1376:      column 820 against 849-875 us, dgrad 495 against 554
// Each launch has a body with its own epilogues only (column 53 -> 49 us, dgrad
// 61 -> 57 on the first shape); where the checkpoint's rows lie is worked out
// once per tile; dA and H leave behind one fence.  Fetching a chunk's bytes
// while the one before is worked on was measured equal and is not done.
#include "tc_gemm_body.cuh"

namespace tpmlp {

TPMLP_TC_KERNELS(tpmlp_fwd_column_gemm_act_ckpt8, 8, EPIS_CK8_FWD)
TPMLP_TC_KERNELS(tpmlp_fwd_column_gemm_act_ckpt8_w16, 16, EPIS_CK8_FWD)
TPMLP_TC_KERNELS(tpmlp_bwd_dgrad_act_ckpt8, 8, EPIS_CK8_BWD)
TPMLP_TC_KERNELS(tpmlp_bwd_dgrad_act_ckpt8_w16, 16, EPIS_CK8_BWD)

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
