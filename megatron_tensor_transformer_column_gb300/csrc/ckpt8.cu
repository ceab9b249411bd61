// ckpt8.cu -- packs a row-major tensor into the 8-bit checkpoint format of
// ckpt8.cuh and unpacks it.
//
// HBM-bound: 2 (bf16) or 4 (fp32) bytes an element on one side, 1.0625 on the
// other, a dozen instructions in between.  A warp owns 32 rows x 128 bytes of
// the tensor, i.e. whole blocks of the checkpoint: 4 groups wide for bf16, 2
// for fp32.  Eight lanes cover the 128 bytes of a row with 16-byte accesses, a
// warp instruction 4 rows, so the tensor's side is read or written in whole
// 128-byte lines, all eight accesses of a lane in flight at once; the
// checkpoint's side gets 64 contiguous bytes per block and instruction.  The
// 2 or 4 lanes of a group find its largest magnitude by shuffles.
//
// Measured on GB300, 8192 x 4096, packed and unpacked again: 30.1 us bf16, 52.8
// us fp32, 1.00 and 0.95 of the copy bandwidth.  Warps of 128-thread CTAs
// start as slots get free: 1531 x 1364 fp32 takes 6.9 us against 7.6 with 256.
// The three-input maximum and paired products took bf16 from 35.2 us.  Loads
// without the streaming hint: 31.3 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "ckpt8.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kSteps = 8;  // 4 rows each

// 16 bytes of the storage type <-> floats
template <typename E>
__device__ __forceinline__ void to_floats(uint4 q, float* v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (sizeof(E) == 2) {
      v[2 * e] = __uint_as_float(w[e] << 16);
      v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
    } else {
      v[e] = __uint_as_float(w[e]);
    }
  }
}

template <typename E>
__device__ __forceinline__ uint4 from_floats(const float* v) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if constexpr (sizeof(E) == 2) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * e], v[2 * e + 1]);
      w[e] = *reinterpret_cast<const uint32_t*>(&h);
    } else {
      w[e] = __float_as_uint(v[e]);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// Where a lane stands: its first column, and its place in the checkpoint for
// row r of the warp's 32.
template <typename E>
struct Place {
  static constexpr int kPer = 16 / sizeof(E);         // elements of a lane
  static constexpr int kLanes = ck::kGroup / kPer;    // lanes of a group
  int64_t row0, col, block;
  int sub;   // this lane's part of its group
  bool on;   // the column is inside the tensor
  __device__ __forceinline__ Place(int64_t rows, int64_t cols, int64_t strips) {
    const int lane = threadIdx.x & 31;
    const int64_t tile = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t rb = tile / strips;
    row0 = rb * ck::kRows;
    col = (tile - rb * strips) * (8 * kPer) + (lane & 7) * kPer;
    block = rb * ck::groups(cols) + col / ck::kGroup;
    sub = (lane & 7) % kLanes;
    on = row0 < rows && col < cols;
  }
};

template <typename E>
__global__ void __launch_bounds__(kThreads)
tpmlp_ckpt8_pack_kernel(int64_t rows, int64_t cols, int64_t strips, const E* src, int64_t ld, uint8_t* ckpt) {
  using P = Place<E>;
  const P p(rows, cols, strips);
  const int lr = (threadIdx.x & 31) >> 3;
  uint4 q[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t r = p.row0 + 4 * i + lr;
    q[i] = p.on && r < rows ? __ldcs(reinterpret_cast<const uint4*>(src + r * ld + p.col)) : make_uint4(0, 0, 0, 0);
  }
  uint8_t* codes = ckpt + p.block * ck::kBlockBytes + p.sub * P::kPer;
  uint8_t* scales = ckpt + ck::scale_offset(rows, cols) + p.block * ck::kRows;
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    float v[P::kPer];
    to_floats<E>(q[i], v);
    uint32_t m = ck::largest<P::kPer>(v);
#pragma unroll
    for (int o = 1; o < P::kLanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
    const uint32_t b = ck::scale_byte(m);
    const int r = 4 * i + lr;
    // A group whose later columns lie past the end: the lane in the tensor
    // writes the zeros of those that are not.
    if (!(p.col - p.sub * P::kPer < cols && p.row0 + r < rows)) continue;
    uint32_t c[P::kPer / 4];
    ck::encode<P::kPer>(v, b, c);
    if constexpr (P::kPer == 8) *reinterpret_cast<uint2*>(codes + r * ck::kGroup) = make_uint2(c[0], c[1]);
    else *reinterpret_cast<uint32_t*>(codes + r * ck::kGroup) = c[0];
    if (p.sub == 0) scales[r] = static_cast<uint8_t>(b);
  }
}

template <typename E>
__global__ void __launch_bounds__(kThreads)
tpmlp_ckpt8_unpack_kernel(int64_t rows, int64_t cols, int64_t strips, const uint8_t* ckpt, E* dst, int64_t ld) {
  using P = Place<E>;
  const P p(rows, cols, strips);
  if (!p.on) return;
  const int lr = (threadIdx.x & 31) >> 3;
  const uint8_t* codes = ckpt + p.block * ck::kBlockBytes + p.sub * P::kPer;
  const uint8_t* scales = ckpt + ck::scale_offset(rows, cols) + p.block * ck::kRows;
  uint2 c[kSteps];
  uint32_t b[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int r = 4 * i + lr;
    c[i] = make_uint2(0, 0);
    b[i] = 127;
    if (p.row0 + r < rows) {
      if constexpr (P::kPer == 8) c[i] = __ldcs(reinterpret_cast<const uint2*>(codes + r * ck::kGroup));
      else c[i].x = __ldcs(reinterpret_cast<const uint32_t*>(codes + r * ck::kGroup));
      b[i] = scales[r];
    }
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int64_t r = p.row0 + 4 * i + lr;
    if (r >= rows) continue;
    float v[8];
    const float s = ck::scale(b[i]);
    ck::decode4(c[i].x, s, v);
    if constexpr (P::kPer == 8) ck::decode4(c[i].y, s, v + 4);
    *reinterpret_cast<uint4*>(dst + r * ld + p.col) = from_floats<E>(v);
  }
}

template <typename E>
int64_t strips_of(int64_t cols) { return (cols + 8 * Place<E>::kPer - 1) / (8 * Place<E>::kPer); }

}  // namespace

cudaError_t launch_ckpt8_pack(bool bf16, int64_t rows, int64_t cols, const void* src, int64_t ld, void* ckpt,
                              cudaStream_t stream) {
  if (rows <= 0 || cols <= 0) return cudaSuccess;
  const int64_t strips = bf16 ? strips_of<__nv_bfloat16>(cols) : strips_of<float>(cols);
  const int64_t ctas = (ck::row_blocks(rows) * strips + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(ctas);
  if (bf16)
    tpmlp_ckpt8_pack_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(
        rows, cols, strips, static_cast<const __nv_bfloat16*>(src), ld, static_cast<uint8_t*>(ckpt));
  else
    tpmlp_ckpt8_pack_kernel<float><<<grid, kThreads, 0, stream>>>(rows, cols, strips, static_cast<const float*>(src),
                                                                  ld, static_cast<uint8_t*>(ckpt));
  return cudaGetLastError();
}

cudaError_t launch_ckpt8_unpack(bool bf16, int64_t rows, int64_t cols, const void* ckpt, void* dst, int64_t ld,
                                cudaStream_t stream) {
  if (rows <= 0 || cols <= 0) return cudaSuccess;
  const int64_t strips = bf16 ? strips_of<__nv_bfloat16>(cols) : strips_of<float>(cols);
  const int64_t ctas = (ck::row_blocks(rows) * strips + kWarps - 1) / kWarps;
  if (ctas > 0x7fffffff) return cudaErrorInvalidConfiguration;
  const unsigned grid = static_cast<unsigned>(ctas);
  if (bf16)
    tpmlp_ckpt8_unpack_kernel<__nv_bfloat16><<<grid, kThreads, 0, stream>>>(
        rows, cols, strips, static_cast<const uint8_t*>(ckpt), static_cast<__nv_bfloat16*>(dst), ld);
  else
    tpmlp_ckpt8_unpack_kernel<float><<<grid, kThreads, 0, stream>>>(
        rows, cols, strips, static_cast<const uint8_t*>(ckpt), static_cast<float*>(dst), ld);
  return cudaGetLastError();
}

}  // namespace tpmlp
