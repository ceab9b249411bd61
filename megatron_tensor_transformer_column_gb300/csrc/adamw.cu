// adamw.cu -- an AdamW step over many tensors at once, moments in 32 or in 8
// bits, and the gradients' global norm that it clips by.
//
// Element p with gradient g (fp32 throughout):
//   f = grad_scale, or max_norm / norm where grad_scale norm > max_norm
//   m = b1 m + (1 - b1) f g,  v = b2 v + (1 - b2) (f g)^2
//   p = p - lr decay p - lr m / (1 - b1^t) / (sqrt(v / (1 - b2^t)) + eps)
// p is the fp32 master where there is one (the bf16 weight is then written
// only), else the weight itself, rounded once.  A norm that is not finite skips
// the step.
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
// rounds it.  A warp holds one group, 8 elements a lane.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int kThreads = 256;
constexpr int kPer = 8;  // elements of a thread and pass
constexpr int kPasses = 2;
constexpr int kChunk = kThreads * kPer * kPasses;  // elements of a CTA
constexpr uint32_t kNanScale = 255;
static_assert(kChunk % kAdamGroup == 0 && 32 * kPer == kAdamGroup, "a warp's pass is a group");

__device__ __forceinline__ uint32_t hash32(uint32_t x) {
  x = (x ^ (x >> 16)) * 0x7feb352du;
  x = (x ^ (x >> 15)) * 0x846ca68bu;
  return x ^ (x >> 16);
}

// Elements i .. i + 7 of an array of n (those past the end read as 0).
template <typename E>
__device__ __forceinline__ void load8(const E* p, int64_t i, int64_t n, float (&v)[8]) {
  if (i + 8 <= n) {
    if constexpr (sizeof(E) == 2) {
      const uint4 q = *reinterpret_cast<const uint4*>(p + i);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        v[2 * k] = __uint_as_float(w[k] << 16);
        v[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
      }
    } else {
      const float4 a = *reinterpret_cast<const float4*>(p + i), b = *reinterpret_cast<const float4*>(p + i + 4);
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = i + k < n ? static_cast<float>(p[i + k]) : 0.0f;
  }
}

template <typename E>
__device__ __forceinline__ void store8(E* p, int64_t i, int64_t n, const float (&v)[8]) {
  if (i + 8 <= n) {
    if constexpr (sizeof(E) == 2) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[2 * k], v[2 * k + 1]);
        w[k] = *reinterpret_cast<const uint32_t*>(&h);
      }
      *reinterpret_cast<uint4*>(p + i) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
      *reinterpret_cast<float4*>(p + i) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(p + i + 4) = make_float4(v[4], v[5], v[6], v[7]);
    }
  } else {
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (i + k < n) p[i + k] = static_cast<E>(v[k]);
  }
}

// ------------------------------------------------------------------ moments in 8 bits

// 8 codes of a group with this scale byte, as floats.
template <bool kSecond>
__device__ __forceinline__ void decode8(uint2 q, uint32_t scale, float (&x)[8]) {
  constexpr uint32_t kMask = kSecond ? 0xffu : 0x7fu;
  const uint32_t base = (scale + (kSecond ? 96u : 112u) - 91u) << 23;  // 2^(e - S)
  const float zero = scale == kNanScale ? __uint_as_float(0x7fffffffu) : 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t c = (k < 4 ? q.x : q.y) >> (8 * (k & 3));
    const uint32_t mag = c & kMask;
    float v = mag ? __uint_as_float((mag << 20) + base) : zero;
    if (!kSecond) v = __uint_as_float(__float_as_uint(v) | ((c & 0x80u) << 24));
    x[k] = v;
  }
}

// 8 elements of the warp's group to codes; the scale byte of the group.
template <bool kSecond>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], const uint32_t (&r)[8], uint32_t& scale) {
  uint32_t big = 0;
#pragma unroll
  for (int k = 0; k < 8; ++k) big = max(big, __float_as_uint(x[k]) & 0x7fffffffu);
  big = __reduce_max_sync(0xffffffffu, big);
  const int e = max(static_cast<int>((big + 0xfffffu) >> 23) - 127, -90);
  if (e >= 127) {  // a NaN, an infinity or a number beyond 2^127: the group is lost
    scale = kNanScale;
    return make_uint2(0, 0);
  }
  scale = big ? static_cast<uint32_t>(e + 91) : 0u;
  const int base = (e + (kSecond ? 96 : 112)) << 23;
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    const uint32_t bits = __float_as_uint(x[k]);
    const uint32_t a = bits & 0x7fffffffu;
    const int y = static_cast<int>(a) - base;
    uint32_t c = static_cast<uint32_t>(y + static_cast<int>(r[k] << 4)) >> 20;
    if (y < (1 << 20)) {  // below the smallest code, 1.125 2^(e - S)
      if (kSecond) {
        c = a ? 1u : 0u;
      } else {
        const float t = __uint_as_float(a) * __uint_as_float(static_cast<uint32_t>(142 - e) << 23);  // 2^(S - e) |x|
        c = t * 65536.0f > static_cast<float>(r[k]) * 1.125f ? 1u : 0u;
      }
    }
    if (!kSecond) c |= (bits >> 24) & 0x80u;
    w[k >> 2] |= c << (8 * (k & 3));
  }
  return make_uint2(w[0], w[1]);
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

template <typename P, typename G, bool k8>
__global__ void __launch_bounds__(kThreads) tpmlp_adamw_step_all(const __grid_constant__ AdamParams a) {
  int64_t first;
  const AdamTensor& t = a.t[find_chunk(a, first)];
  float f = a.grad_scale;
  if (a.norm) {
    const float norm = *a.norm * a.grad_scale;
    if (!(norm <= 3.402823466e38f)) return;  // NaN or infinity
    if (a.max_norm > 0.0f && norm > a.max_norm) f *= a.max_norm / norm;
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
  const float lr_t = lr * rate;
  const float shrink = lr * t.decay;
#pragma unroll 1
  for (int pass = 0; pass < kPasses; ++pass) {
    const int64_t i = first + (pass * kThreads + threadIdx.x) * kPer;
    if (i - (threadIdx.x & 31) * kPer >= t.n) break;  // the warp's group is past the end
    float g[8], p[8], m[8], v[8];
    load8(static_cast<const G*>(t.g), i, t.n, g);
    if (t.master) load8(t.master, i, t.n, p);
    else load8(static_cast<const P*>(t.p), i, t.n, p);
    const int64_t groups = (t.n + kAdamGroup - 1) / kAdamGroup, q = i / kAdamGroup;
    uint8_t* mc = static_cast<uint8_t*>(t.m);
    uint8_t* vc = static_cast<uint8_t*>(t.v);
    if constexpr (k8) {
      const uint2 cm = *reinterpret_cast<const uint2*>(mc + i), cv = *reinterpret_cast<const uint2*>(vc + i);
      const uint32_t sm = mc[groups * kAdamGroup + q], sv = vc[groups * kAdamGroup + q];
      decode8<false>(cm, sm, m);
      decode8<true>(cv, sv, v);
    } else {
      load8(static_cast<const float*>(t.m), i, t.n, m);
      load8(static_cast<const float*>(t.v), i, t.n, v);
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x = g[k] * f;
      m[k] = fmaf(m[k], a.b1, x * a.b1c);
      v[k] = fmaf(v[k], a.b2, x * a.b2c * x);
      float root;
      asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(root) : "f"(v[k]));
      const float u = __fdividef(m[k] * lr_t, fmaf(root, c2, a.eps));
      p[k] = fmaf(-shrink, p[k], p[k]) - u;
    }
    if (t.master) store8(t.master, i, t.n, p);
    store8(static_cast<P*>(t.p), i, t.n, p);
    if constexpr (k8) {
      const uint64_t number = static_cast<uint64_t>(t.group0 + q);
      const uint32_t h = hash32(hash32(key ^ static_cast<uint32_t>(number)) ^ static_cast<uint32_t>(number >> 32));
      uint32_t r[8];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t x = hash32(h + ((threadIdx.x & 31) * 4 + k) * 0x9e3779b9u);
        r[2 * k] = x & 0xffffu;
        r[2 * k + 1] = x >> 16;
      }
      uint32_t sm, sv;
      const uint2 cm = encode8<false>(m, r, sm), cv = encode8<true>(v, r, sv);
      *reinterpret_cast<uint2*>(mc + i) = cm;
      *reinterpret_cast<uint2*>(vc + i) = cv;
      if ((threadIdx.x & 31) == 0) {
        mc[groups * kAdamGroup + q] = static_cast<uint8_t>(sm);
        vc[groups * kAdamGroup + q] = static_cast<uint8_t>(sv);
      }
    } else {
      store8(static_cast<float*>(t.m), i, t.n, m);
      store8(static_cast<float*>(t.v), i, t.n, v);
    }
  }
}

// Codes to the values that they stand for, each of which is a bf16 number.
// t.p and t.master: where m and v go.
__global__ void __launch_bounds__(kThreads) tpmlp_adamw8_unpack_all(const __grid_constant__ AdamParams a) {
  int64_t first;
  const AdamTensor& t = a.t[find_chunk(a, first)];
  const int64_t groups = (t.n + kAdamGroup - 1) / kAdamGroup;
#pragma unroll
  for (int pass = 0; pass < kPasses; ++pass) {
    const int64_t i = first + (pass * kThreads + threadIdx.x) * kPer;
    if (i >= t.n) break;
    const int64_t q = groups * kAdamGroup + i / kAdamGroup;
    const uint8_t* mc = static_cast<const uint8_t*>(t.m);
    const uint8_t* vc = static_cast<const uint8_t*>(t.v);
    float x[8];
    if (t.p) {
      decode8<false>(*reinterpret_cast<const uint2*>(mc + i), mc[q], x);
      store8(static_cast<__nv_bfloat16*>(t.p), i, t.n, x);
    }
    if (t.master) {
      decode8<true>(*reinterpret_cast<const uint2*>(vc + i), vc[q], x);
      store8(reinterpret_cast<__nv_bfloat16*>(t.master), i, t.n, x);
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
    const int64_t first = static_cast<int64_t>(c - (k ? a.t[k - 1].end : 0)) * kChunk;
#pragma unroll
    for (int pass = 0; pass < kPasses; ++pass) {
      const int64_t i = first + (pass * kThreads + threadIdx.x) * kPer;
      float g[8], y = 0.0f;
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = 0.0f;
      if (i < t.n) load8(static_cast<const G*>(t.g), i, t.n, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) y = fmaf(g[j], g[j], y);
      const float sum = s + y, back = sum - s;
      lost += (s - (sum - back)) + (y - back);
      s = sum;
    }
  }
  double d = static_cast<double>(s);
  if (s <= 3.402823466e38f) d += static_cast<double>(lost);  // an infinite sum loses infinities
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

template <bool k8>
AdamKernel pick(bool bf16, bool gbf16) {
  if (bf16) return gbf16 ? tpmlp_adamw_step_all<__nv_bfloat16, __nv_bfloat16, k8>
                         : tpmlp_adamw_step_all<__nv_bfloat16, float, k8>;
  return gbf16 ? tpmlp_adamw_step_all<float, __nv_bfloat16, k8> : tpmlp_adamw_step_all<float, float, k8>;
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
  const AdamKernel k = bits8 ? pick<true>(bf16, grad_bf16) : pick<false>(bf16, grad_bf16);
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
