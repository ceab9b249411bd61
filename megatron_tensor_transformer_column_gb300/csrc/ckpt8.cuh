// ckpt8.cuh -- the 8-bit checkpoint of a [rows x cols] tensor: its format and
// the arithmetic of one group, shared by the pack and unpack kernels and the
// GEMM epilogues.
//
// A group is 16 consecutive columns of one row.  With m its largest magnitude,
// its scale is 2^e with the smallest e for which m <= 448 * 2^e (448 is the
// largest e4m3 number), limited to [-117, 120]; an element x is kept as the
// e4m3 number nearest to x 2^-e, ties to even.  A power of two as the scale
// makes the scaling exact, so an element is rounded once: by at most 2^-4 of
// its value while |x| >= 2^-6 2^e, by 2^(e - 10) below.  e >= -117 keeps the
// smallest kept number, 2^-9 2^e, a normal fp32 and bf16 number; with e = 120
// codes stop at 240, so that no finite input comes back as an infinity.  A
// group that holds a NaN or an infinity has the scale byte 255 and comes back
// as NaN throughout: a value that 8 bits do not hold is never replaced by a
// finite one.
//
// Storage: blocks of 32 rows x 16 columns, 512 bytes each, row after row (16
// bytes a row), the blocks of 32 rows side by side; behind the last block one
// byte e + 127 per group, 32 per block, in the blocks' order.  A block is what
// one epilogue warp holds (a row per lane), so that its stores and loads are
// 512 contiguous bytes.  Bytes of rows past the last are neither written nor
// read; columns past the last, within a group, are kept as 0.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#include "act.cuh"
#endif

namespace tpmlp {
namespace ck {

constexpr int kGroup = 16;
constexpr int kRows = 32;
constexpr int kBlockBytes = kGroup * kRows;

__host__ __device__ inline int64_t groups(int64_t cols) { return (cols + kGroup - 1) / kGroup; }
__host__ __device__ inline int64_t row_blocks(int64_t rows) { return (rows + kRows - 1) / kRows; }
__host__ __device__ inline int64_t scale_offset(int64_t rows, int64_t cols) {
  return row_blocks(rows) * groups(cols) * kBlockBytes;
}
__host__ __device__ inline int64_t bytes(int64_t rows, int64_t cols) {
  return row_blocks(rows) * groups(cols) * (kBlockBytes + kRows);
}

#ifdef __CUDACC__

constexpr uint32_t kBadScale = 255;  // scale byte of a group that holds a NaN or an infinity

// The scale byte of a group whose largest magnitude has the bits m (an
// infinity's or a NaN's bits are above every finite number's).
__device__ __forceinline__ uint32_t scale_byte(uint32_t m) {
  // floor(log2 m) - 8, one more if m > 1.75 * 2^floor(log2 m); biased by 127
  const int b = static_cast<int>(m >> 23) - 8 + ((m & 0x7fffffu) > 0x600000u ? 1 : 0);
  return m >= 0x7f800000u ? kBadScale : static_cast<uint32_t>(b < 10 ? 10 : b);
}

// 2^-e and 2^e of a scale byte (2^e: NaN for kBadScale).
__device__ __forceinline__ float inv_scale(uint32_t b) { return __uint_as_float((254u - (b < 254u ? b : 127u)) << 23); }
__device__ __forceinline__ float scale(uint32_t b) {
  return b == kBadScale ? __uint_as_float(0x7fc00000u) : __uint_as_float(b << 23);
}

// Two e4m3 codes: x0 in the low byte.
__device__ __forceinline__ uint32_t encode2(float x0, float x1) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(x1), "f"(x0));
  return r;
}
constexpr uint32_t kTopScale = 247;  // e = 120, whose codes stop at 240
// N / 4 words of codes of x[0 .. N - 1] * inv.
template <int N>
__device__ __forceinline__ void encode(const float* x, uint32_t byte, uint32_t (&c)[N / 4]) {
  const uint64_t inv = act::x2::splat(inv_scale(byte));
  float v[N];
#pragma unroll
  for (int k = 0; k < N; k += 2) act::x2::upk(act::x2::mul2(act::x2::pk(x[k], x[k + 1]), inv), v[k], v[k + 1]);
  if (__builtin_expect(byte == kTopScale, 0)) {
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = fminf(fmaxf(v[k], -240.0f), 240.0f);
  }
#pragma unroll
  for (int k = 0; k < N / 4; ++k)
    c[k] = encode2(v[4 * k], v[4 * k + 1]) | (encode2(v[4 * k + 2], v[4 * k + 3]) << 16);
}

// Two values from the low 16 bits of c (exact: every e4m3 number is an fp16
// number).
__device__ __forceinline__ void decode2(uint32_t c, float s, float& x0, float& x1) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(c)));
  float f0, f1;
  asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.f32.f16 %0, lo;\n cvt.f32.f16 %1, hi;\n}"
      : "=f"(f0), "=f"(f1)
      : "r"(h));
  x0 = f0 * s;
  x1 = f1 * s;
}
__device__ __forceinline__ void decode4(uint32_t c, float s, float* x) {
  decode2(c, s, x[0], x[1]);
  decode2(c >> 16, s, x[2], x[3]);
}

// The bits of the largest magnitude of x[0 .. N - 1] (a NaN's where there is one).
template <int N>
__device__ __forceinline__ uint32_t largest(const float* x) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int k = 1; k + 1 < N; k += 2)
    asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(x[k]), "f"(x[k + 1]));
  if (N % 2 == 0) asm("max.NaN.abs.f32 %0, %0, %1, %1;" : "+f"(m) : "f"(x[N - 1]));
  return __float_as_uint(m) & 0x7fffffffu;
}

// One row of a group, held by one thread: 16 values to 16 codes and the scale
// byte, and back.
__device__ __forceinline__ uint4 encode_row(const float* x, uint32_t& byte) {
  byte = scale_byte(largest<kGroup>(x));
  uint32_t c[kGroup / 4];
  encode<kGroup>(x, byte, c);
  return make_uint4(c[0], c[1], c[2], c[3]);
}
__device__ __forceinline__ void decode_row(uint4 c, uint32_t byte, float* x) {
  const float s = scale(byte);
  decode4(c.x, s, x);
  decode4(c.y, s, x + 4);
  decode4(c.z, s, x + 8);
  decode4(c.w, s, x + 12);
}

#endif  // __CUDACC__

}  // namespace ck
}  // namespace tpmlp
