// tc_gemm_residual.cu -- the row-parallel products with the residual stream
// added in the epilogue (body: tc_gemm_body.cuh): Y = R + sum_i H_i W2_i + b2
// and Z = R + sum_i O_i WO_i.  The sum is taken of the fp32 accumulator and
// rounded once; R is read by the warp that then writes the same 32 x 32 block,
// so that Y may be R itself.
//
// Bound by the tensor cores like the launches without a residual.  R's reads
// come on top of the operands' (T d elements to T d_ff + d_ff d), and spare the
// norm behind the product the reading of two arrays for one, the writing of the
// sum, and a rounding.  A chunk's block of R is fetched while the chunk before is
// worked on, the first one while the accumulator is computed; it passes through
// the block of shared memory that the sum leaves by.  Measured on GB300, against
// the launch without a residual:
//   8192 x 4096 by 4096 (8 shards)     156 against 151 us (0.93 of the burst rate)
//   8192 x 11008 by 4096 (8 shards)    412 against 406 us
//   8192 x 8192 by 2048, unequal       161.5 against 157 us
//   8192 x (4 x 768) by 768            37 against 35 us
//   1 to 64 tokens, 4096 by 4096 (8 shards)    25 against 25 us (weights 5)
//   1 to 64 tokens, 11008 by 4096 (8 shards)   36 against 34 us (weights 13)
// With few tokens 16 tiles of 256 columns are 16 of 76 pairs at work, each going
// through all of K: latency-bound, with or without the residual.
// Fetching a chunk's block when it is due took 161, 421, 165 and 38 us; a
// prefetch of R into L2 made no difference.
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
