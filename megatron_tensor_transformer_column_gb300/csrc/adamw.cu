// adamw.cu -- an AdamW step over many tensors at once, moments in 32 or in 8
// bits, and the gradients' global norm that it clips by.
//
// Element p with gradient g (fp32 throughout):
//   f = grad_scale, or max_norm / norm where grad_scale norm > max_norm
//   m = b1 m + (1 - b1) f g,  v = b2 v + (1 - b2) (f g)^2
//   p = p - lr decay p - lr m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps)
// p is the fp32 master where there is one (the bf16 weight is then written
// only), else the weight itself, rounded once.  A norm that is not finite skips
// the step; so does one that grad_scale takes past the range, unless it is clipped.
//
// Moments in 8 bits.  Groups of 256 elements; M a group's largest magnitude, e =
// floor(log2 M), one more where M > 1.875 2^e, at least -90.  A code is a number
// with 3 bits behind its leading one, so (1 + (c % 8) / 8) 2^(c / 8) 2^(e - S),
// 0 for c = 0: 7 bits and the sign for m (S = 15), 8 bits for v (S = 31), whose
// root then spans as much as m.  Rounding is stochastic: a step moves v by
// (1 - b2) of itself, far less than half a code, so the nearest code would hold
// it where it is, rising when a large gradient comes and never falling.  The
// random 16 bits of an element, used for both moments, are a hash of seed, step
// and the element's number.  A v above 0 and below the smallest code is kept as
// that code, since the root of a 0 would divide by eps alone; a small m is
// rounded between 0 and the smallest code like any other.  The step itself uses m
// and v before they are rounded.
//
// The codes are cut out of the fp32 bits: with the group's exponent taken off,
// a magnitude's bits 20.. are its code, and adding 16 random bits at bit 4
// rounds it.  A warp holds one group, 8 elements a lane, and takes four groups
// one after the other, the next one's loads on their way from L2, where the lines
// of all four are asked for at the start (238 -> 222 us on the first shape below).
//
// Bound by HBM with moments in 32 bits (10 to 20 instructions an element of 22 to
// 30 bytes), by the integer pipe and the issue slots with 8 bits (52 instructions
// an element of 10 bytes; 74 and 76 % of them taken before that).  The 72 registers that
// 7 CTAs an SM leave do not hold all of a pass with 8 bits: 32 bytes a thread are
// spilled with bf16 weights and gradients, up to 140 with masters and fp32
// gradients; 6 CTAs take 3 % longer.
//
// Measured on GB300, six tensors of 22.5 M, and share of the copy bandwidth:
//   bf16 weights, fp32 masters, 32 bits 543 us (1.0); without masters 426 (1.0)
//   8 bits: bf16 weights 222 us (0.90), with masters 316 (1.0), fp32 weights 312
//     (1.0); read out as bf16 118 (1.0)
//   the norm of bf16 gradients 44 us (0.90), of fp32 ones 80 (0.99)
// A first version with 82 instructions an element took 435 us.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <type_traits>

#include "act.cuh"
#include "ptx.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

using act::x2::add2;
using act::x2::fma2;
using act::x2::mul2;
using act::x2::pk;
using act::x2::splat;
using act::x2::upk;

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 8;     // elements of a thread and pass
constexpr int kPasses = 4;  // of a CTA: a warp's consecutive groups, whose scale bytes are one word
constexpr int kChunk = kThreads * kPer * kPasses;  // elements of a CTA
constexpr uint32_t kNanScale = 255;
constexpr float kMost = 3.402823466e38f;  // of fp32's finite numbers
static_assert(32 * kPer == kAdamGroup && kPasses == 4, "a warp's pass is a group, its chunk's scales a word");

// Two multiplications with xors of the upper bits; the multipliers are those that
// C. Wellons published in 2018 from a search for 32-bit mixers of low bias.  The
// host works out a step's key with the same function (adam_hash).
__device__ __forceinline__ uint32_t hash32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x7feb352du;
  x = (x ^ (x >> 15)) * 0x846ca68bu;
  return x ^ (x >> 16);
}

// Loads under a predicate (zeros without it), with no branch around them: where
// two paths meet the loaded registers would be copied, and waited for, one load
// after the other.
__device__ __forceinline__ uint4 load16_if(const void* p, uint32_t go) {
  uint4 q;
  asm volatile(
      "{\n .reg .pred go;\n setp.ne.u32 go, %5, 0;\n"
      " mov.u32 %0, 0;\n mov.u32 %1, 0;\n mov.u32 %2, 0;\n mov.u32 %3, 0;\n"
      " @go ld.global.v4.u32 {%0, %1, %2, %3}, [%4];\n}"
      : "=&r"(q.x), "=&r"(q.y), "=&r"(q.z), "=&r"(q.w)
      : "l"(p), "r"(go)
      : "memory");
  return q;
}
__device__ __forceinline__ uint2 load8_if(const void* p, uint32_t go) {
  uint2 q;
  asm volatile(
      "{\n .reg .pred go;\n setp.ne.u32 go, %3, 0;\n mov.u32 %0, 0;\n mov.u32 %1, 0;\n"
      " @go ld.global.v2.u32 {%0, %1}, [%2];\n}"
      : "=&r"(q.x), "=&r"(q.y)
      : "l"(p), "r"(go)
      : "memory");
  return q;
}
// Lines of 128 bytes from p on into L2, one a lane.
__device__ __forceinline__ void prefetch(const void* p, int bytes, int lane) {
  for (int at = lane * 128; at < bytes; at += 32 * 128) ptx::prefetch_l2(static_cast<const char*>(p) + at);
}

// 8 elements as they lie in memory.
template <typename E>
struct Eight {
  static constexpr int kQuads = sizeof(E) / 2;
  uint4 q[kQuads];
  // elements i .. i + 7, all of which the array has; nothing without `go`
  __device__ __forceinline__ void load(const E* p, int64_t i, uint32_t go) {
#pragma unroll
    for (int k = 0; k < kQuads; ++k) q[k] = load16_if(p + i + k * (16 / static_cast<int>(sizeof(E))), go);
  }
  __device__ __forceinline__ void store(E* p, int64_t i) const {
#pragma unroll
    for (int k = 0; k < kQuads; ++k) reinterpret_cast<uint4*>(p + i)[k] = q[k];
  }
  // of an array of n: what lies past its end is 0 and is not touched
  __device__ __forceinline__ void load_tail(const E* p, int64_t i, int64_t n) {
    uint32_t w[8] = {};
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (i + k >= n) continue;
      if constexpr (sizeof(E) == 2)
        w[k / 2] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t*>(p)[i + k]) << (16 * (k & 1));
      else w[k] = reinterpret_cast<const uint32_t*>(p)[i + k];
    }
#pragma unroll
    for (int k = 0; k < kQuads; ++k) q[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  }
  __device__ __forceinline__ void store_tail(E* p, int64_t i, int64_t n) const {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint4 f = q[sizeof(E) == 2 ? 0 : k / 4];
      const int e = sizeof(E) == 2 ? k / 2 : k % 4;
      const uint32_t w = e == 0 ? f.x : e == 1 ? f.y : e == 2 ? f.z : f.w;
      if (i + k >= n) continue;
      if constexpr (sizeof(E) == 2) reinterpret_cast<uint16_t*>(p)[i + k] = static_cast<uint16_t>(w >> (16 * (k & 1)));
      else reinterpret_cast<uint32_t*>(p)[i + k] = w;
    }
  }
  __device__ __forceinline__ void get(uint64_t (&v)[4]) const {
    if constexpr (sizeof(E) == 2) {
      const uint32_t w[4] = {q[0].x, q[0].y, q[0].z, q[0].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = pk(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
    } else {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        v[2 * k] = pk(__uint_as_float(q[k].x), __uint_as_float(q[k].y));
        v[2 * k + 1] = pk(__uint_as_float(q[k].z), __uint_as_float(q[k].w));
      }
    }
  }
  __device__ __forceinline__ void set(const uint64_t (&v)[4]) {
    uint32_t w[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      float lo, hi;
      upk(v[k], lo, hi);
      if constexpr (sizeof(E) == 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      } else {
        w[2 * k] = __float_as_uint(lo);
        w[2 * k + 1] = __float_as_uint(hi);
      }
    }
#pragma unroll
    for (int k = 0; k < static_cast<int>(sizeof(E)) / 2; ++k)
      q[k] = make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
  }
};

// ------------------------------------------------------------------ moments in 8 bits

// 2^(e - S) as fp32 bits: what a code's bits 20.. are added to.
template <bool kSecond>
__device__ __forceinline__ uint32_t scale_bits(uint32_t scale) {
  return (scale + (kSecond ? 96u : 112u) - 91u) << 23;
}

// 8 codes of a group with this scale byte, as floats.  Without a zero code (all
// but a few words) two codes at a time as bf16 numbers: a code's place there is
// bits 4.., the sign's (of m) bit 15, and the scale's exponent is added.
template <bool kSecond>
__device__ __forceinline__ void decode8(uint2 q, uint32_t scale, uint64_t (&x)[4]) {
  constexpr uint32_t kMask = kSecond ? 0xffffffffu : 0x7f7f7f7fu;
  const uint32_t base = scale_bits<kSecond>(scale);
  const uint32_t a = q.x & kMask, b = q.y & kMask;
  if ((((a - 0x01010101u) & ~a) | ((b - 0x01010101u) & ~b)) & 0x80808080u) {  // a zero byte
    const float zero = scale == kNanScale ? __uint_as_float(0x7fffffffu) : 0.0f;
    float v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const uint32_t c = (k < 4 ? q.x : q.y) >> (8 * (k & 3));
      const uint32_t mag = c & (kMask & 0xffu);
      v[k] = mag ? __uint_as_float((mag << 20) + base) : zero;
      if (!kSecond && (c & 0x80u)) v[k] = -v[k];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) x[k] = pk(v[2 * k], v[2 * k + 1]);
  } else {
    const uint32_t base2 = (base >> 16) * 0x10001u;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t w = k < 2 ? q.x : q.y;
      uint32_t h;
      if (kSecond) {
        h = __byte_perm(w, 0, k & 1 ? 0x4342 : 0x4140) * 16u + base2;
      } else {
        const uint32_t c = __byte_perm(w, 0, k & 1 ? 0x3424 : 0x1404);  // the codes in the upper bytes
        h = ((c & 0x80008000u) | ((c >> 4) & 0x07f007f0u)) + base2;
      }
      x[k] = pk(__uint_as_float(h << 16), __uint_as_float(h & 0xffff0000u));
    }
  }
}

__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 8 elements of the warp's group to codes; the scale byte of the group.  h: the
// random bits of elements 2 k (low half) and 2 k + 1.  Multiplied by a power of
// two, the group's numbers have the exponent 128 + c / 8 (m) or 96 + c / 8 (v): so
// bits 20 .. 27 are the code, and shifted up by 4 it is the top byte (what is
// above it falls off), under which the random bits stand at 8 .. 23 to round it.
template <bool kSecond>
__device__ __forceinline__ uint2 encode8(const uint64_t (&pairs)[4], const uint32_t (&h)[4], uint32_t& scale) {
  float x[8], y[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) upk(pairs[k], x[2 * k], x[2 * k + 1]);
  auto mag = [](float v) { return kSecond ? v : fabsf(v); };
  const float most = max3_nan(max3_nan(mag(x[0]), mag(x[1]), mag(x[2])), max3_nan(mag(x[3]), mag(x[4]), mag(x[5])),
                              max3_nan(mag(x[6]), mag(x[7]), mag(x[7])));
  const uint32_t big = __reduce_max_sync(0xffffffffu, __float_as_uint(most) & 0x7fffffffu);
  const int e = max(static_cast<int>((big + 0xfffffu) >> 23) - 127, -90);
  if (big == 0 || e >= 127) {  // nothing; or a NaN, an infinity or a number beyond 2^127: the group is lost
    scale = big ? kNanScale : 0u;
    return make_uint2(0, 0);
  }
  scale = static_cast<uint32_t>(e + 91);
  // 2^16 / 2^e: 2^(e - 15) becomes 2; 1 / 2^e: 2^(e - 31) becomes 2^-31
  const uint64_t up = splat(__uint_as_float(static_cast<uint32_t>((kSecond ? 127 : 143) - e) << 23));
  constexpr float kLeast = kSecond ? 1.125f * 0x1p-31f : 2.25f;  // the smallest code
  uint32_t z[8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    upk(mul2(pairs[k], up), y[2 * k], y[2 * k + 1]);
#pragma unroll
    for (int j = 2 * k; j < 2 * k + 2; ++j) {
      const uint32_t bits = __float_as_uint(y[j]);
      z[j] = bits * 16u + __byte_perm(h[k], 0, j & 1 ? 0x4324 : 0x4104);
      if (!kSecond) z[j] |= bits & 0x80000000u;
    }
  }
  const float least = min3(min3(mag(y[0]), mag(y[1]), mag(y[2])), min3(mag(y[3]), mag(y[4]), mag(y[5])),
                           fminf(mag(y[6]), mag(y[7])));
  if (least < kLeast) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      if (mag(y[k]) >= kLeast) continue;
      uint32_t c;
      if (kSecond) {
        c = x[k] > 0.0f ? 1u : 0u;
      } else {
        const uint32_t r = k & 1 ? h[k >> 1] >> 16 : h[k >> 1] & 0xffffu;
        c = mag(y[k]) * 32768.0f > static_cast<float>(r) * 1.125f ? 1u : 0u;  // y / 2 times 2^16
        c |= (__float_as_uint(x[k]) >> 24) & 0x80u;
      }
      z[k] = c << 24;
    }
  }
  uint2 q;
  q.x = __byte_perm(__byte_perm(z[0], z[1], 0x0073), __byte_perm(z[2], z[3], 0x0073), 0x5410);
  q.y = __byte_perm(__byte_perm(z[4], z[5], 0x0073), __byte_perm(z[6], z[7], 0x0073), 0x5410);
  return q;
}

// ------------------------------------------------------------------ the step

// The tensor of chunk blockIdx.x, and the chunk's first element in it.
__device__ __forceinline__ int find_chunk(const AdamParams& a, int64_t& first) {
  const int c = blockIdx.x;
  int lo = 0, hi = a.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (c < a.t[mid].end) hi = mid;
    else lo = mid + 1;
  }
  first = static_cast<int64_t>(c - (lo ? a.t[lo - 1].end : 0)) * kChunk;
  return lo;
}

// What a thread reads for a pass.  M: the type that the weight is read as.
template <typename M, typename G, bool k8>
struct Pass {
  Eight<G> g;
  Eight<M> p;
  Eight<float> m, v;  // in 32 bits,
  uint2 mc, vc;       // or codes
  __device__ __forceinline__ void load(const AdamTensor& t, const M* src, int64_t i, bool whole, uint32_t go) {
    if (whole) {
      g.load(static_cast<const G*>(t.g), i, go);
      p.load(src, i, go);
    } else {
      g.load_tail(static_cast<const G*>(t.g), i, t.n);
      p.load_tail(src, i, t.n);
    }
    if constexpr (k8) {  // whole groups always
      mc = load8_if(static_cast<const uint8_t*>(t.m) + i, go);
      vc = load8_if(static_cast<const uint8_t*>(t.v) + i, go);
    } else if (whole) {
      m.load(static_cast<const float*>(t.m), i, go);
      v.load(static_cast<const float*>(t.v), i, go);
    } else {
      m.load_tail(static_cast<const float*>(t.m), i, t.n);
      v.load_tail(static_cast<const float*>(t.v), i, t.n);
    }
  }
};

// The scale bytes of a warp's kPasses groups, which are neighbours, as one word
// (n of them where the tensor ends before).  A warp reads and writes them once
// for its whole chunk: with a byte of a group at a time, stores to and loads from
// the same sectors held each other up (135 M weights: 520 us instead of 240).
__device__ __forceinline__ uint32_t load_scales(const uint8_t* p, int n) {
  if (n >= kPasses) return *reinterpret_cast<const uint32_t*>(p);
  uint32_t w = 0;
  for (int k = 0; k < n; ++k) w |= static_cast<uint32_t>(p[k]) << (8 * k);
  return w;
}
__device__ __forceinline__ void store_scales(uint8_t* p, int n, uint32_t w) {
  if (n >= kPasses) {
    *reinterpret_cast<uint32_t*>(p) = w;
  } else {
    for (int k = 0; k < n; ++k) p[k] = static_cast<uint8_t>(w >> (8 * k));
  }
}

template <typename E>
__device__ __forceinline__ void put8(const uint64_t (&x)[4], E* p, int64_t i, int64_t n, bool whole) {
  Eight<E> out;
  out.set(x);
  if (whole) out.store(p, i);
  else out.store_tail(p, i, n);
}

// kFlush: a v below 2^-126 may be taken for 0, as the faster root does.  The
// denominator is then less by 2^-63 (1 - b2^t)^(-1/2) at most, a 2^-25th of itself
// where eps is at least kFlushEps times the first step's correction: half of one
// fp32 rounding.  A smaller eps takes the root that keeps such a v, three
// instructions an element more: with 8 bits 222 -> 236 us for 135 M bf16 weights,
// with 32 bits or masters, which HBM bounds, equal (there always).
template <bool kFlush>
__device__ __forceinline__ void root(float& x) {
  if constexpr (kFlush) asm("sqrt.approx.ftz.f32 %0, %0;" : "+f"(x));
  else asm("sqrt.approx.f32 %0, %0;" : "+f"(x));
}
constexpr double kFlushEps = 0x1p-38;

// kMaster: the fp32 copy is updated, the weight only written.  m and v take one
// rounding for each product and sum as the formulas have them, so that what the
// random bits make of them does not depend on how products and sums are fused:
// the assembler fuses an fp32x2 product with the sum behind it although both are
// .rn, so each product is a sum itself, with a -0 that only the host knows (8 bits,
// 135 M bf16 weights: 222 us, fused 217; elsewhere equal).
template <typename P, typename G, bool k8, bool kMaster, bool kFlush>
__global__ void __launch_bounds__(kThreads, k8 ? 7 : 4) tpmlp_adamw_step_all(const __grid_constant__ AdamParams a) {
  using M = typename std::conditional<kMaster, float, P>::type;
  int64_t first;
  const AdamTensor t = a.t[find_chunk(a, first)];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t codes = (t.n + kAdamGroup - 1) / kAdamGroup * kAdamGroup;
  M* src = kMaster ? reinterpret_cast<M*>(t.master) : static_cast<M*>(t.p);
  int64_t at = first + warp * (kPasses * kAdamGroup);  // this warp's group, the next one on every pass
  Pass<M, G, k8> now;
  now.load(t, src, at + lane * kPer, true, at + kAdamGroup <= t.n);
  if (k8 && at + kPasses * kAdamGroup <= t.n) {  // the warp's other groups on their way into L2
    constexpr int kAll = kPasses * kAdamGroup;
    prefetch(static_cast<const G*>(t.g) + at, kAll * static_cast<int>(sizeof(G)), lane);
    prefetch(src + at, kAll * static_cast<int>(sizeof(M)), lane);
    prefetch((lane & 16 ? static_cast<const uint8_t*>(t.v) : static_cast<const uint8_t*>(t.m)) + at, kAll, lane & 15);
  }
  uint8_t* ms = static_cast<uint8_t*>(t.m) + codes + at / kAdamGroup;
  uint8_t* vs = static_cast<uint8_t*>(t.v) + codes + at / kAdamGroup;
  const int groups = static_cast<int>(min(static_cast<int64_t>(kPasses), max(int64_t{0}, (codes - at) / kAdamGroup)));
  uint32_t m_scales = 0, v_scales = 0, m_new = 0, v_new = 0;
  if (k8) {
    m_scales = load_scales(ms, groups);
    v_scales = load_scales(vs, groups);
  }

  float f = a.grad_scale;
  if (a.norm) {
    const float norm = *a.norm, scaled = norm * a.grad_scale;
    const bool clip = a.max_norm > 0.0f && scaled > a.max_norm, fits = scaled <= kMost;
    if (!(norm <= kMost) || !(clip || fits)) return;  // NaN, an infinity, or scaled to one that nothing clips
    if (clip) f = fits ? f * (a.max_norm * __frcp_rn(scaled)) : __fdiv_rn(a.max_norm, norm);
  }
  const float lr = a.lr_dev ? *a.lr_dev : a.lr;
  float rate = a.rate, c2 = a.c2;
  uint32_t key = a.key;
  if (a.step_dev) {  // corrections and key of the step that the device counts
    const int64_t step = *a.step_dev;
    rate = 1.0f / -expm1f(static_cast<float>(static_cast<double>(step) * a.ln_b1));
    c2 = rsqrtf(-expm1f(static_cast<float>(static_cast<double>(step) * a.ln_b2)));
    key = hash32(hash32(key ^ static_cast<uint32_t>(step)) ^ static_cast<uint32_t>(step >> 32));
  }
  const uint64_t zero = splat(a.minus_zero), f2 = splat(f), b1 = splat(a.b1), b1c = splat(a.b1c), b2 = splat(a.b2), b2c = splat(a.b2c);
  const uint64_t root_scale = splat(c2), eps = splat(a.eps), shrink = splat(-(lr * t.decay)), rate2 = splat(-(lr * rate));
  uint32_t seeds = 0;
  if (k8) {  // lane k: the random bits' start of pass k's group
    const uint64_t q = static_cast<uint64_t>(t.group0 + at / kAdamGroup + lane % kPasses);
    seeds = hash32(hash32(key ^ static_cast<uint32_t>(q)) ^ static_cast<uint32_t>(q >> 32));
  }

  // One pass.  whole: the group is; next: whether the one after it is, and is this warp's, whose loads are on their way
  // while this one is worked on.
  auto one = [&](int pass, bool whole, bool next) {
    const int64_t i = at + lane * kPer;
    uint64_t x[4], p[4], m[4], v[4];
    now.g.get(x);
    now.p.get(p);
    if constexpr (k8) {
      decode8<false>(now.mc, (m_scales >> (8 * pass)) & 0xffu, m);
      decode8<true>(now.vc, (v_scales >> (8 * pass)) & 0xffu, v);
    } else {
      now.m.get(m);
      now.v.get(v);
    }
    if (whole) now.load(t, src, i + kAdamGroup, true, next);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      x[k] = mul2(x[k], f2);
      m[k] = add2(fma2(m[k], b1, zero), fma2(x[k], b1c, zero));
      v[k] = add2(fma2(v[k], b2, zero), fma2(mul2(x[k], b2c), x[k], zero));
      float lo, hi;
      upk(v[k], lo, hi);
      root<kFlush>(lo);
      root<kFlush>(hi);
      upk(fma2(pk(lo, hi), root_scale, eps), lo, hi);
      asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(lo));
      asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(hi));
      p[k] = fma2(mul2(m[k], pk(lo, hi)), rate2, fma2(shrink, p[k], p[k]));
    }
    if (kMaster) put8(p, t.master, i, t.n, whole);
    put8(p, static_cast<P*>(t.p), i, t.n, whole);
    if constexpr (k8) {
      const uint32_t seed = __shfl_sync(0xffffffffu, seeds, pass) + lane * (4 * 0x9e3779b9u);
      uint32_t h[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) h[k] = hash32(seed + k * 0x9e3779b9u);
      uint32_t sm, sv;
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + i) = encode8<false>(m, h, sm);
      *reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + i) = encode8<true>(v, h, sv);
      m_new |= sm << (8 * pass);
      v_new |= sv << (8 * pass);
    } else {
      put8(m, static_cast<float*>(t.m), i, t.n, whole);
      put8(v, static_cast<float*>(t.v), i, t.n, whole);
    }
  };
  int pass = 0;
#pragma unroll 1
  for (; pass < kPasses && at + kAdamGroup <= t.n; ++pass, at += kAdamGroup)
    one(pass, true, pass + 1 < kPasses && at + 2 * kAdamGroup <= t.n);
  if (pass < kPasses && at < t.n) {  // the tensor's last group, where it is not whole
    now.load(t, src, at + lane * kPer, false, 1);
    one(pass, false, false);
  }
  if (k8 && lane == 0) {
    store_scales(ms, groups, m_new);
    store_scales(vs, groups, v_new);
  }
}

// Codes to the values that they stand for, each of which is a bf16 number.
// t.p and t.master: where m and v go.
__global__ void __launch_bounds__(kThreads) tpmlp_adamw8_unpack_all(const __grid_constant__ AdamParams a) {
  int64_t first;
  const AdamTensor t = a.t[find_chunk(a, first)];
  const int64_t codes = (t.n + kAdamGroup - 1) / kAdamGroup * kAdamGroup;
  const uint8_t* src[2] = {static_cast<const uint8_t*>(t.m), static_cast<const uint8_t*>(t.v)};
  __nv_bfloat16* dst[2] = {static_cast<__nv_bfloat16*>(t.p), reinterpret_cast<__nv_bfloat16*>(t.master)};
  const int64_t i0 = first + threadIdx.x * kPer;
  uint2 c[2][kPasses];
  uint32_t s[2][kPasses];
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    const int64_t i = i0 + pass * (kThreads * kPer);
#pragma unroll
    for (int w = 0; w < 2; ++w)
      if (dst[w] && i < t.n) {
        c[w][pass] = *reinterpret_cast<const uint2*>(src[w] + i);
        s[w][pass] = src[w][codes + i / kAdamGroup];
      }
  }
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    const int64_t i = i0 + pass * (kThreads * kPer);
    if (i >= t.n) break;
    uint64_t x[4];
    if (dst[0]) {
      decode8<false>(c[0][pass], s[0][pass], x);
      put8(x, dst[0], i, t.n, i + kPer <= t.n);
    }
    if (dst[1]) {
      decode8<true>(c[1][pass], s[1][pass], x);
      put8(x, dst[1], i, t.n, i + kPer <= t.n);
    }
  }
}

// ------------------------------------------------------------------ the norm
// The sum of squares of all gradients: a thread adds 8 squares in fp32 and keeps
// the running sum in two floats (the second holds what the first lost), a CTA's
// threads and then the CTAs add in 64 bits, in a fixed order; the CTA whose
// ticket is the last does that and puts the counter back to 0.
template <typename G>
__global__ void __launch_bounds__(kThreads) tpmlp_grad_norm_all(const __grid_constant__ AdamParams a, uint32_t* ticket,
                                                                double* partial, float* norm, int chunks) {
  float s = 0.0f, lost = 0.0f;
  int k = 0;
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    while (c >= a.t[k].end) ++k;
    const AdamTensor& t = a.t[k];
    const int64_t i0 = static_cast<int64_t>(c - (k ? a.t[k - 1].end : 0)) * kChunk + threadIdx.x * kPer;
    Eight<G> g[kPasses];
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int64_t i = i0 + pass * (kThreads * kPer);
      g[pass].load(static_cast<const G*>(t.g), i, i + kPer <= t.n);
    }
    if (i0 + (kPasses - 1) * (kThreads * kPer) + kPer > t.n) {  // near the tensor's end
#pragma unroll
      for (int pass = 0; pass < kPasses; ++pass) {
        const int64_t i = i0 + pass * (kThreads * kPer);
        if (i < t.n && i + kPer > t.n) g[pass].load_tail(static_cast<const G*>(t.g), i, t.n);
      }
    }
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      uint64_t x[4], y2 = 0;
      g[pass].get(x);
#pragma unroll
      for (int j = 0; j < 4; ++j) y2 = fma2(x[j], x[j], y2);
      float y, z;
      upk(y2, y, z);
      y += z;
      const float sum = s + y, back = sum - s;
      lost += (s - (sum - back)) + (y - back);
      s = sum;
    }
  }
  double d = static_cast<double>(s);
  if (s <= kMost) d += static_cast<double>(lost);  // an infinite sum loses infinities
  __shared__ double parts[kThreads / 32];
  __shared__ bool last;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = d;
  __syncthreads();
  if (threadIdx.x == 0) {
    d = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) d += parts[w];
    partial[blockIdx.x] = d;
    __threadfence();
    last = atomicInc(ticket, gridDim.x - 1) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!last) return;
  d = 0.0;
  for (int i = threadIdx.x; i < gridDim.x; i += kThreads) d += __ldcg(partial + i);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
  if ((threadIdx.x & 31) == 0) parts[threadIdx.x >> 5] = d;
  __syncthreads();
  if (threadIdx.x == 0) {
    d = 0.0;
    for (int w = 0; w < kThreads / 32; ++w) d += parts[w];
    if (a.more) partial[kAdamNormCtas] = a.first_batch ? d : partial[kAdamNormCtas] + d;
    else *norm = static_cast<float>(sqrt(a.first_batch ? d : partial[kAdamNormCtas] + d));
  }
}

using AdamKernel = void (*)(AdamParams);

template <typename G, bool k8, bool kFlush>
AdamKernel pick(bool bf16, bool master) {
  if (!bf16) return tpmlp_adamw_step_all<float, G, k8, false, kFlush>;
  return master ? tpmlp_adamw_step_all<__nv_bfloat16, G, k8, true, kFlush>
                : tpmlp_adamw_step_all<__nv_bfloat16, G, k8, false, kFlush>;
}

template <typename G>
AdamKernel pick(bool bf16, bool master, bool bits8, bool flush) {
  if (!bits8) return pick<G, false, false>(bf16, master);
  return flush ? pick<G, true, true>(bf16, master) : pick<G, true, false>(bf16, master);
}

// Ends of the tensors' chunks; their number.
int lay_out(AdamParams& a) {
  int64_t c = 0;
  for (int k = 0; k < a.n; ++k) {
    c += (a.t[k].n + kChunk - 1) / kChunk;
    if (c > 0x7fffffff) return -1;
    a.t[k].end = static_cast<int32_t>(c);
  }
  return static_cast<int>(c);
}

}  // namespace

cudaError_t launch_adamw(AdamParams& a, bool bf16, bool grad_bf16, bool bits8, cudaStream_t stream) {
  const int chunks = lay_out(a);
  if (chunks < 0) return cudaErrorInvalidConfiguration;
  if (chunks == 0) return cudaSuccess;
  const bool master = a.t[0].master != nullptr;  // of all tensors or none
  const bool flush = a.eps >= kFlushEps / std::sqrt(-std::expm1(a.ln_b2));
  const AdamKernel k = grad_bf16 ? pick<__nv_bfloat16>(bf16, master, bits8, flush) : pick<float>(bf16, master, bits8, flush);
  k<<<chunks, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_adamw8_unpack(AdamParams& a, cudaStream_t stream) {
  const int chunks = lay_out(a);
  if (chunks < 0) return cudaErrorInvalidConfiguration;
  if (chunks == 0) return cudaSuccess;
  tpmlp_adamw8_unpack_all<<<chunks, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_grad_norm(AdamParams& a, bool grad_bf16, void* workspace, float* norm, int sms,
                             cudaStream_t stream) {
  const int chunks = lay_out(a);
  if (chunks < 0) return cudaErrorInvalidConfiguration;
  const int ctas = std::max(1, std::min(chunks, std::min(8 * sms, kAdamNormCtas)));
  uint32_t* ticket = static_cast<uint32_t*>(workspace);
  double* partial = reinterpret_cast<double*>(static_cast<char*>(workspace) + kStatusBytes);
  if (grad_bf16) tpmlp_grad_norm_all<__nv_bfloat16><<<ctas, kThreads, 0, stream>>>(a, ticket, partial, norm, chunks);
  else tpmlp_grad_norm_all<float><<<ctas, kThreads, 0, stream>>>(a, ticket, partial, norm, chunks);
  return cudaGetLastError();
}

}  // namespace tpmlp
