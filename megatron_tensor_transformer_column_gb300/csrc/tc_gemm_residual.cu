// tc_gemm_residual.cu -- the row-parallel products with the residual stream
// added in the epilogue (body: tc_gemm_body.cuh): Y = R + sum_i H_i W2_i + b2
// and Z = R + sum_i O_i WO_i.  The sum is taken of the fp32 accumulator and
// rounded once; R is read by the warp that then writes the same 32 x 32 block,
// so that Y may be R itself.
//
// Bound by the tensor cores like the launches without a residual; R's reads
// take their place among the operands' (T d elements to T d_ff + d_ff d) and
// spare the norm behind the product the reading of Y and R and the rounding of
// Y.
#include "tc_gemm_body.cuh"

namespace tpmlp {

TPMLP_TC_KERNELS(tpmlp_fwd_row_gemm_gsum_res, 8, EPIS_RESIDUAL)
TPMLP_TC_KERNELS(tpmlp_attn_out_proj_gsum_res, 8, EPIS_RESIDUAL)

TcKernelFn tc_residual_kernel(int tag, bool stream_k) {
  switch (tag) {
    case TAG_FWD_ROW: return stream_k ? tpmlp_fwd_row_gemm_gsum_res_sk : tpmlp_fwd_row_gemm_gsum_res;
    case TAG_ATTN_OUT: return stream_k ? tpmlp_attn_out_proj_gsum_res_sk : tpmlp_attn_out_proj_gsum_res;
    default: return nullptr;
  }
}

}  // namespace tpmlp
