// simt_gemm.cu -- fp32 path of the t-sharded MLP block (exact fp32 FFMA,
// fp32 accumulation), for problems stored in fp32.
//
// It runs the same problem lists as the tensor-core path (same segments, so
// the g-sum and the f-sum are K loops into one register accumulator here
// too, and the same epilogues), one 32x32 output tile per CTA.  The
// tensor-core path is bf16-only; fp32 storage with a 1e-4 relative bound
// rules out the tf32 tensor-core kind, whose per-product error is too close
// to that bound.
#include <cuda_runtime.h>

#include "act.cuh"
#include "ckpt8.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int kT = 32;        // tile edge (M and N)
constexpr int kK = 32;        // K chunk
constexpr int kThreads = 256; // 32 columns x 8 row groups of 4 rows

// Element (row, col) of a stored row-major array, or of the launch's striped
// input (token stripes) when `striped`.
__device__ __forceinline__ const float* elem(const GemmParams& p, const void* base, int64_t ld, bool striped,
                                             int64_t row, int64_t col) {
  if (striped) {
    const Stripes& st = p.stripes;
    int j = 0;
    while (j + 1 < st.num && row >= st.row0[j + 1]) ++j;
    return static_cast<const float*>(st.in[j]) + (row - st.row0[j]) * st.in_ld + col;
  }
  return static_cast<const float*>(base) + row * ld + col;
}

constexpr int kLoads = kT * kK / kThreads;  // a thread's elements of a chunk of an operand

// A thread's elements (mn, k) of an operand [K x MN] (MAJOR_MN) or [MN x K], for
// the chunks of one segment: neighbouring lanes along the contiguous dimension.
struct Operand {
  const float* at;   // the thread's first element of the chunk K = 0
  int64_t apart;     // between its elements
  int64_t step;      // from a K to the next
  int mn0, k0;       // its first element; the next ones are 8 further in the other dimension
  bool mn_major;
  __device__ __forceinline__ Operand(const void* base, int64_t ld, int major, int64_t tile0) {
    const int fast = threadIdx.x & 31, slow = threadIdx.x >> 5;
    mn_major = major == MAJOR_MN;
    mn0 = static_cast<int>(tile0) + (mn_major ? fast : slow);
    k0 = mn_major ? slow : fast;
    step = mn_major ? ld : 1;
    apart = (kThreads / 32) * ld;
    at = static_cast<const float*>(base) + (mn_major ? k0 * ld + mn0 : mn0 * ld + k0);
  }
  __device__ __forceinline__ void load(int k, int MN, int K, float (&r)[kLoads]) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int more = i * (kThreads / 32);
      const bool in = mn_major ? mn0 < MN && k + k0 + more < K : mn0 + more < MN && k + k0 < K;
      r[i] = in ? at[k * step + i * apart] : 0.f;
    }
  }
  // of the launch's striped input
  __device__ __forceinline__ void load_striped(const GemmParams& p, int k, int MN, int K, float (&r)[kLoads]) const {
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int more = i * (kThreads / 32);
      const int mn = mn0 + (mn_major ? 0 : more), kk = k + k0 + (mn_major ? more : 0);
      r[i] = mn < MN && kk < K ? *elem(p, nullptr, 0, true, mn_major ? kk : mn, mn_major ? mn : kk) : 0.f;
    }
  }
};

// An operand's chunk into shared memory, [k][mn] with rows of kLd floats.
template <int kLd>
__device__ __forceinline__ void put(float (*s)[kLd], bool mn_major, const float (&r)[kLoads]) {
  const int fast = threadIdx.x & 31, slow = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) {
    const int other = slow + i * (kThreads / 32);
    if (mn_major) s[other][fast] = r[i];
    else s[fast][other] = r[i];
  }
}

// A value of one lane of a row of 32 columns to and from an 8-bit checkpoint:
// the 16 lanes of a group find its largest magnitude by shuffles.
__device__ __forceinline__ int64_t ckpt8_block(const Prob& P, int64_t row, int64_t col) {
  return (row / ck::kRows) * ck::groups(P.N) + col / ck::kGroup;
}

__device__ __forceinline__ void store_ckpt8(void* ckpt, const Prob& P, int64_t row, int64_t col, bool row_ok, float v) {
  uint32_t m = __float_as_uint(col < P.N ? v : 0.0f) & 0x7fffffffu;
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
  const uint32_t b = ck::scale_byte(m);
  const int64_t k = col % ck::kGroup;
  if (!row_ok || col - k >= P.N) return;
  const float w[4] = {col < P.N ? v : 0.0f, 0.0f, 0.0f, 0.0f};
  uint32_t c[1];
  ck::encode<4>(w, b, c);
  const int64_t blk = ckpt8_block(P, row, col);
  uint8_t* base = static_cast<uint8_t*>(ckpt);
  base[blk * ck::kBlockBytes + (row % ck::kRows) * ck::kGroup + k] =
      static_cast<uint8_t>(c[0]);
  if (k == 0) base[ck::scale_offset(P.M, P.N) + blk * ck::kRows + row % ck::kRows] = static_cast<uint8_t>(b);
}

__device__ __forceinline__ float load_ckpt8(const void* ckpt, const Prob& P, int64_t row, int64_t col) {
  const int64_t blk = ckpt8_block(P, row, col);
  const uint8_t* base = static_cast<const uint8_t*>(ckpt);
  float x0, x1;
  ck::decode2(base[blk * ck::kBlockBytes + (row % ck::kRows) * ck::kGroup + col % ck::kGroup],
              ck::scale(base[ck::scale_offset(P.M, P.N) + blk * ck::kRows + row % ck::kRows]), x0, x1);
  return x0;
}

// The activation epilogues with 8-bit checkpoints: rows row0 .. row0 + 3 of
// this thread's column.  Every lane takes part (the groups' shuffles).
__device__ __forceinline__ void ckpt8_epilogue(const Prob& P, int64_t row0, int64_t n0, const float (&acc)[4],
                                               const float (&acc2)[4]) {
  const int64_t col = n0 + (threadIdx.x & 31);
  const bool in = col < P.N;
  for (int i = 0; i < 4; ++i) {
    const int64_t row = row0 + i;
    const bool row_ok = row < P.M;  // the same for the whole warp
    const int64_t o = row * P.ldo + col;
    float v = acc[i];
    switch (P.epi) {
      case EPI_GELU_FWD:
        if (P.aux0 && in) v += static_cast<const float*>(P.aux0)[col];
        store_ckpt8(P.out0, P, row, col, row_ok, v);
        if (row_ok && in) static_cast<float*>(P.out1)[o] = act::gelu(v);
        break;
      case EPI_SWIGLU_FWD: {
        float u = acc2[i];
        if (P.aux0 && in) v += static_cast<const float*>(P.aux0)[col];
        if (P.aux1 && in) u += static_cast<const float*>(P.aux1)[col];
        store_ckpt8(P.out0, P, row, col, row_ok, v);
        store_ckpt8(P.out1, P, row, col, row_ok, u);
        if (row_ok && in) static_cast<float*>(P.out2)[o] = u * act::swish(v);
        break;
      }
      case EPI_GELU_BWD:
        if (row_ok && in) {
          const float a = load_ckpt8(P.aux0, P, row, col);
          static_cast<float*>(P.out0)[o] = v * act::gelu_grad(a);
          static_cast<float*>(P.out1)[o] = act::gelu(a);
        }
        break;
      case EPI_SWIGLU_BWD:
        if (row_ok && in) {
          float dg, du;
          const float gg = load_ckpt8(P.aux0, P, row, col), uu = load_ckpt8(P.aux1, P, row, col);
          act::swiglu_grads(v, gg, uu, dg, du);
          static_cast<float*>(P.out0)[o] = dg;
          static_cast<float*>(P.out1)[o] = du;
          static_cast<float*>(P.out2)[o] = uu * act::swish(gg);
        }
        break;
      default:
        break;
    }
  }
}

__global__ void __launch_bounds__(kThreads) tpmlp_fp32_simt_gemm(const __grid_constant__ GemmParams p) {
  __shared__ __align__(16) float As[kK][kT + 4];  // [k][m], rows of 16 bytes
  __shared__ float Bs[kK][kT + 1];                // [k][n]
  __shared__ float B2s[kK][kT + 1];               // [k][n] (SwiGLU up projection)

  // tile decode (same raster as the tensor-core path, tile_m = 32)
  const int tile = blockIdx.x;
  int g = 0;
  while (g + 1 < p.num_groups && tile >= p.groups[g + 1].tile_start) ++g;
  const Group& G = p.groups[g];
  int mt, n_lin;
  group_tile(G, tile - G.tile_start, mt, n_lin);
  int pi = G.first_prob;
  while (n_lin >= p.probs[pi].tiles_n) {
    n_lin -= p.probs[pi].tiles_n;
    ++pi;
  }
  const Prob& P = p.probs[pi];
  const int64_t m0 = static_cast<int64_t>(mt) * kT;
  const int64_t n0 = static_cast<int64_t>(n_lin) * P.tile_n;
  const bool dual = P.epi == EPI_SWIGLU_FWD;

  const int tx = threadIdx.x & 31;   // output column in tile
  const int ty = threadIdx.x >> 5;   // rows 4*ty .. 4*ty+3
  float acc[4] = {0.f, 0.f, 0.f, 0.f};
  float acc2[4] = {0.f, 0.f, 0.f, 0.f};

  // A chunk of K travels global memory -> registers -> shared memory, the next
  // one's loads on their way while this one is worked on, all of a thread's at
  // once.  (Waiting for each before the next one, 203 x 264 with K = 408 took
  // 47 us; working out every element's address anew 35.)
  const int seg_end = P.seg_begin + P.seg_count;
  for (int sg = P.seg_begin; sg < seg_end; ++sg) {
    const Seg& S = p.segs[sg];
    const int K = S.K;
    const bool a_striped = S.a_striped, b_striped = S.b_striped;
    const Operand A(S.a, S.lda, P.a_major, m0), B(S.b, S.ldb, P.b_major, n0), B2(S.b2, S.ldb, P.b_major, n0);
    float ra[kLoads], rb[kLoads], rb2[kLoads];
    auto fetch = [&](int k) {
      if (a_striped) A.load_striped(p, k, P.M, K, ra);
      else A.load(k, P.M, K, ra);
      if (b_striped) B.load_striped(p, k, P.N, K, rb);
      else B.load(k, P.N, K, rb);
      if (dual) B2.load(k, P.N, K, rb2);
    };
    fetch(0);
    for (int k0 = 0; k0 < K; k0 += kK) {
      put(As, A.mn_major, ra);
      put(Bs, B.mn_major, rb);
      if (dual) put(B2s, B.mn_major, rb2);
      __syncthreads();
      if (k0 + kK < K) fetch(k0 + kK);
      if (dual) {
#pragma unroll 8
        for (int kk = 0; kk < kK; ++kk) {
          const float b = Bs[kk][tx], b2 = B2s[kk][tx];
          const float4 a = *reinterpret_cast<const float4*>(&As[kk][4 * ty]);
          acc[0] = fmaf(a.x, b, acc[0]);
          acc[1] = fmaf(a.y, b, acc[1]);
          acc[2] = fmaf(a.z, b, acc[2]);
          acc[3] = fmaf(a.w, b, acc[3]);
          acc2[0] = fmaf(a.x, b2, acc2[0]);
          acc2[1] = fmaf(a.y, b2, acc2[1]);
          acc2[2] = fmaf(a.z, b2, acc2[2]);
          acc2[3] = fmaf(a.w, b2, acc2[3]);
        }
      } else {
#pragma unroll 8
        for (int kk = 0; kk < kK; ++kk) {
          const float b = Bs[kk][tx];
          const float4 a = *reinterpret_cast<const float4*>(&As[kk][4 * ty]);
          acc[0] = fmaf(a.x, b, acc[0]);
          acc[1] = fmaf(a.y, b, acc[1]);
          acc[2] = fmaf(a.z, b, acc[2]);
          acc[3] = fmaf(a.w, b, acc[3]);
        }
      }
      __syncthreads();
    }
  }

  const int64_t col = n0 + tx;
  if (p.ckpt8) {
    ckpt8_epilogue(P, m0 + 4 * ty, n0, acc, acc2);
    return;
  }
  if (col >= P.N) return;
  for (int i = 0; i < 4; ++i) {
    const int64_t row = m0 + 4 * ty + i;
    if (row >= P.M) continue;
    const int64_t o = row * P.ldo + col;
    float v = acc[i];
    switch (P.epi) {
      case EPI_STORE:
        if (P.aux0) v += static_cast<const float*>(P.aux0)[col];
        if (P.aux1) v += static_cast<const float*>(P.aux1)[o];  // the residual stream
        if (P.out_striped) {  // token stripes of the sequence-parallel layout
          const Stripes& st = p.stripes;
          int j = 0;
          while (j + 1 < st.num && row >= st.row0[j + 1]) ++j;
          static_cast<float*>(st.out[j])[(row - st.row0[j]) * st.out_ld + col] = v;
        } else {
          static_cast<float*>(P.out0)[o] = v;
        }
        break;
      case EPI_GELU_FWD:
        if (P.aux0) v += static_cast<const float*>(P.aux0)[col];
        static_cast<float*>(P.out0)[o] = v;
        static_cast<float*>(P.out1)[o] = act::gelu(v);
        break;
      case EPI_SWIGLU_FWD: {
        float u = acc2[i];
        if (P.aux0) v += static_cast<const float*>(P.aux0)[col];
        if (P.aux1) u += static_cast<const float*>(P.aux1)[col];
        static_cast<float*>(P.out0)[o] = v;
        static_cast<float*>(P.out1)[o] = u;
        static_cast<float*>(P.out2)[o] = u * act::swish(v);
        break;
      }
      case EPI_GELU_BWD: {
        const float a = static_cast<const float*>(P.aux0)[o];
        static_cast<float*>(P.out0)[o] = v * act::gelu_grad(a);
        if (P.out1) static_cast<float*>(P.out1)[o] = act::gelu(a);  // recomputed H
        break;
      }
      case EPI_SWIGLU_BWD: {
        float dg, du;
        const float gg = static_cast<const float*>(P.aux0)[o], uu = static_cast<const float*>(P.aux1)[o];
        act::swiglu_grads(v, gg, uu, dg, du);
        static_cast<float*>(P.out0)[o] = dg;
        static_cast<float*>(P.out1)[o] = du;
        if (P.out2) static_cast<float*>(P.out2)[o] = uu * act::swish(gg);  // recomputed H
        break;
      }
      default:
        break;
    }
  }
}

}  // namespace

cudaError_t launch_simt_gemm(const GemmParams& p, cudaStream_t stream) {
  if (p.total_tiles <= 0) return cudaSuccess;
  tpmlp_fp32_simt_gemm<<<p.total_tiles, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace tpmlp
