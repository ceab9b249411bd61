// tc_gemm_ckpt8.cu -- the tensor-core GEMM's launches that keep their
// pre-activations as 8-bit checkpoints (format: ckpt8.cuh; body:
// tc_gemm_body.cuh): the column GEMM, whose epilogue writes them from the fp32
// accumulators, and the dgrad GEMM, whose epilogue reads them, takes act' of
// the kept values and recomputes H.
//
// Bound by the tensor cores like the launches they stand beside, or, with short
// K, by the epilogue: it moves 1.0625 bytes per pre-activation instead of 2,
// with plain stores and loads of a warp's own block, and a thread finds its
// row's largest magnitudes, scales and codes in about 35 instructions per 16
// elements.  Measured on GB300 (device time of the launch, against the one with
// bf16 pre-activations and, for dgrad, recomputed H):
//   GeLU, 8192 x 768, 4 x 768:          column 54 against 51 us, dgrad 61 against 68
//   GeLU, 8192 x 2048, 8192 hidden:     column 176 against 176 us, dgrad 192 against 200
//   SwiGLU, 8192 x 4096, 8 x 1376:      column 820 against 849-875 us, dgrad 499 against 554
// Where the checkpoint's rows lie is worked out once per tile (column of the
// first shape 57 -> 54 us), dA and H leave behind one fence (dgrad 65 -> 63).
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
