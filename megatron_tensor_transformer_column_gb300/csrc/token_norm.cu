// token_norm.cu -- layer norm and RMS norm of the tokens in front of a block,
// with the residual stream's sum, and the backward pass.
//
// One token x of `cols` elements (fp32 throughout, each output rounded once to
// the storage type):
//   s = x + residual            (kept in the storage type; what is kept is normed)
//   mu = mean(s), r = (mean((s - mu)^2) + eps)^(-1/2)      (RMS: mu = 0)
//   n = (s - mu) r,  y = n gain + bias
// Backward, from dy and dsum (the gradient that reaches s past the norm):
//   w = dy gain,  dx = r (w - mean(w) - n mean(w n)) + dsum  (RMS: without mean(w))
//   dgain = sum over tokens of dy n,  dbias = sum over tokens of dy
// Two passes over the values for mu and r (the second sums squares of s - mu), so
// that a mean far larger than the spread costs no digits.
//
// Layout of the work.  HBM-bound: every array is read or written once.  A token
// belongs to a team of W warps, up to 32 elements a thread, always the same
// columns, so that gain, bias and the sums of their gradients stay in registers
// for the whole launch.  Each thread copies its own 16-byte vectors of the next
// tokens into shared memory by itself (asynchronous copies, a queue per thread)
// and reads back only what it copied: no barrier but those of the sums over a
// token, and bytes in flight without registers.  The sums of the gains'
// gradients are added over a CTA's teams, then over the CTAs by a second launch,
// each in a fixed order.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "ptx.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSmem = 227 * 1024;
constexpr int kMaxStages = 6;

template <typename E>
constexpr int kPer = 16 / static_cast<int>(sizeof(E));  // elements of a vector

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

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Waits until at most n of this thread's groups are on their way.
__device__ __forceinline__ void copy_wait_all_but(int n) {
  switch (n) {
    case 0: copy_wait<0>(); break;
    case 1: copy_wait<1>(); break;
    case 2: copy_wait<2>(); break;
    case 3: copy_wait<3>(); break;
    case 4: copy_wait<4>(); break;
    default: copy_wait<5>(); break;
  }
}

// Sums over the threads of a team, in a fixed order.  red: 2 x W float2 of the
// team; the calls alternate between the halves, so that one barrier a call
// suffices: a half is written again only behind the other half's barrier, at
// which everybody has read it.
template <int W>
struct TeamSum {
  float2* red;
  int bar;   // named barrier of the team
  int half;
  __device__ __forceinline__ float2 operator()(float a, float b, int warp_in_team) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xffffffffu, a, o);
      b += __shfl_xor_sync(0xffffffffu, b, o);
    }
    if constexpr (W > 1) {
      float2* mine = red + half * W;
      if ((threadIdx.x & 31) == 0) mine[warp_in_team] = make_float2(a, b);
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(W * 32) : "memory");
      a = b = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) {
        const float2 f = mine[w];
        a += f.x;
        b += f.y;
      }
      half ^= 1;
    }
    return make_float2(a, b);
  }
  __device__ __forceinline__ float operator()(float a, int warp_in_team) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if constexpr (W > 1) {
      float2* mine = red + half * W;
      if ((threadIdx.x & 31) == 0) mine[warp_in_team].x = a;
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(W * 32) : "memory");
      a = 0.0f;
#pragma unroll
      for (int w = 0; w < W; ++w) a += mine[w].x;
      half ^= 1;
    }
    return a;
  }
};

template <typename E, int W, int V>
struct Thread {
  int t, team, warp_in_team;
  int64_t first, step;
  bool on[V];
  __device__ __forceinline__ explicit Thread(int cols) {
    t = threadIdx.x % (W * 32);
    team = threadIdx.x / (W * 32);
    warp_in_team = (threadIdx.x >> 5) % W;
    // tokens are dealt to the CTAs first, then to their teams: few tokens spread over many SMs
    first = static_cast<int64_t>(team) * gridDim.x + blockIdx.x;
    step = static_cast<int64_t>(gridDim.x) * (kWarps / W);
#pragma unroll
    for (int v = 0; v < V; ++v) on[v] = (v * W * 32 + t) * kPer<E> < cols;
  }
  // bytes of vector v from a row's start
  __device__ __forceinline__ int off(int v) const { return 16 * t + v * (W * 32 * 16); }
};

__device__ __forceinline__ uint32_t slot_of(uint32_t base, int arrays, int V, int stage, int array, int v) {
  return base + static_cast<uint32_t>(((stage * arrays + array) * V + v) * kThreads + threadIdx.x) * 16u;
}

template <typename E, int W, int V>
__global__ void __launch_bounds__(kThreads, 1) tpmlp_norm_fwd(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 red[2 * kWarps];
  const uint32_t base = ptx::smem_u32(smem);
  const Thread<E, W, V> th(p.cols);
  TeamSum<W> sum{red + th.team * 2 * W, 1 + th.team, 0};
  const bool add = p.res != nullptr;
  const int arrays = add ? 2 : 1, S = p.stages;

  auto fetch = [&](int64_t row, int stage) {
    if (row < p.rows) {
      const char* x = static_cast<const char*>(p.x) + row * p.ldx;
      const char* r = static_cast<const char*>(p.res) + row * p.ldr;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!th.on[v]) continue;
        copy16(slot_of(base, arrays, V, stage, 0, v), x + th.off(v));
        if (add) copy16(slot_of(base, arrays, V, stage, 1, v), r + th.off(v));
      }
    }
    copy_commit();
  };

  for (int i = 0; i + 1 < S; ++i) fetch(th.first + i * th.step, i);
  uint4 gain[V], bias[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    gain[v] = bias[v] = make_uint4(0, 0, 0, 0);
    if (p.gain && th.on[v]) gain[v] = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.gain) + th.off(v));
    if (p.bias && th.on[v]) bias[v] = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.bias) + th.off(v));
  }
  int stage = 0;
  for (int64_t row = th.first; row < p.rows; row += th.step) {
    fetch(row + (S - 1) * th.step, stage == 0 ? S - 1 : stage - 1);
    copy_wait_all_but(S - 1);
    float x[V][kPer<E>];
    float a = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
#pragma unroll
      for (int e = 0; e < kPer<E>; ++e) x[v][e] = 0.0f;
      if (!th.on[v]) continue;
      to_floats<E>(ptx::ld_shared_v4(slot_of(base, arrays, V, stage, 0, v)), x[v]);
      if (add) {
        float r[kPer<E>];
        to_floats<E>(ptx::ld_shared_v4(slot_of(base, arrays, V, stage, 1, v)), r);
#pragma unroll
        for (int e = 0; e < kPer<E>; ++e) x[v][e] += r[e];
        const uint4 q = from_floats<E>(x[v]);
        *reinterpret_cast<uint4*>(static_cast<char*>(p.sum) + row * p.lds + th.off(v)) = q;
        to_floats<E>(q, x[v]);
      }
    }
    float mu = 0.0f;
    if (!p.rms) {
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < kPer<E>; ++e) a += x[v][e];
      mu = sum(a, th.warp_in_team) * p.inv_cols;
    }
    a = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!th.on[v]) continue;
#pragma unroll
      for (int e = 0; e < kPer<E>; ++e) {
        x[v][e] -= mu;
        a = fmaf(x[v][e], x[v][e], a);
      }
    }
    const float r = rsqrtf(fmaf(sum(a, th.warp_in_team), p.inv_cols, p.eps));
    if (th.t == 0 && p.stats) reinterpret_cast<float2*>(p.stats)[row] = make_float2(mu, r);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!th.on[v]) continue;
      float g[kPer<E>], b[kPer<E>];
      to_floats<E>(bias[v], b);
      if (p.gain) {
        to_floats<E>(gain[v], g);
#pragma unroll
        for (int e = 0; e < kPer<E>; ++e) x[v][e] = fmaf(x[v][e] * r, g[e], b[e]);
      } else {
#pragma unroll
        for (int e = 0; e < kPer<E>; ++e) x[v][e] = fmaf(x[v][e], r, b[e]);
      }
      *reinterpret_cast<uint4*>(static_cast<char*>(p.y) + row * p.ldy + th.off(v)) = from_floats<E>(x[v]);
    }
    stage = stage + 1 == S ? 0 : stage + 1;
  }
  copy_wait<0>();
}

template <typename E, int W, int V>
__global__ void __launch_bounds__(kThreads, 1) tpmlp_norm_bwd(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ float2 red[2 * kWarps];
  const uint32_t base = ptx::smem_u32(smem);
  const Thread<E, W, V> th(p.cols);
  TeamSum<W> sum{red + th.team * 2 * W, 1 + th.team, 0};
  const bool add = p.dsum != nullptr;
  const int arrays = add ? 3 : 2, S = p.stages;

  auto fetch = [&](int64_t row, int stage) {
    if (row < p.rows) {
      const char* x = static_cast<const char*>(p.x) + row * p.ldx;
      const char* dy = static_cast<const char*>(p.dy) + row * p.lddy;
      const char* ds = static_cast<const char*>(p.dsum) + row * p.ldds;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (!th.on[v]) continue;
        copy16(slot_of(base, arrays, V, stage, 0, v), x + th.off(v));
        copy16(slot_of(base, arrays, V, stage, 1, v), dy + th.off(v));
        if (add) copy16(slot_of(base, arrays, V, stage, 2, v), ds + th.off(v));
      }
    }
    copy_commit();
  };

  for (int i = 0; i + 1 < S; ++i) fetch(th.first + i * th.step, i);
  const float2* stats = reinterpret_cast<const float2*>(p.stats);
  float2 next = th.first < p.rows ? stats[th.first] : make_float2(0.0f, 0.0f);
  uint4 gain[V];
  float dg[V][kPer<E>], db[V][kPer<E>];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    gain[v] = make_uint4(0, 0, 0, 0);
    if (p.gain && th.on[v]) gain[v] = *reinterpret_cast<const uint4*>(static_cast<const char*>(p.gain) + th.off(v));
#pragma unroll
    for (int e = 0; e < kPer<E>; ++e) dg[v][e] = db[v][e] = 0.0f;
  }
  int stage = 0;
  for (int64_t row = th.first; row < p.rows; row += th.step) {
    fetch(row + (S - 1) * th.step, stage == 0 ? S - 1 : stage - 1);
    const float mu = next.x, r = next.y;
    if (row + th.step < p.rows) next = stats[row + th.step];
    copy_wait_all_but(S - 1);
    float sw = 0.0f, swn = 0.0f;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!th.on[v]) continue;
      float x[kPer<E>], w[kPer<E>], g[kPer<E>];
      to_floats<E>(ptx::ld_shared_v4(slot_of(base, arrays, V, stage, 0, v)), x);
      to_floats<E>(ptx::ld_shared_v4(slot_of(base, arrays, V, stage, 1, v)), w);
      to_floats<E>(gain[v], g);
#pragma unroll
      for (int e = 0; e < kPer<E>; ++e) {
        const float n = (x[e] - mu) * r;
        dg[v][e] = fmaf(w[e], n, dg[v][e]);
        db[v][e] += w[e];
        if (p.gain) w[e] *= g[e];
        sw += w[e];
        swn = fmaf(w[e], n, swn);
      }
    }
    const float2 m = sum(sw, swn, th.warp_in_team);
    const float c1 = p.rms ? 0.0f : m.x * p.inv_cols, c2 = m.y * p.inv_cols;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      if (!th.on[v]) continue;
      float x[kPer<E>], w[kPer<E>], g[kPer<E>];
      to_floats<E>(ptx::ld_shared_v4(slot_of(base, arrays, V, stage, 0, v)), x);
      to_floats<E>(ptx::ld_shared_v4(slot_of(base, arrays, V, stage, 1, v)), w);
      to_floats<E>(gain[v], g);
#pragma unroll
      for (int e = 0; e < kPer<E>; ++e) {
        const float n = (x[e] - mu) * r;
        if (p.gain) w[e] *= g[e];
        x[e] = r * fmaf(-n, c2, w[e] - c1);
      }
      if (add) {
        to_floats<E>(ptx::ld_shared_v4(slot_of(base, arrays, V, stage, 2, v)), w);
#pragma unroll
        for (int e = 0; e < kPer<E>; ++e) x[e] += w[e];
      }
      *reinterpret_cast<uint4*>(static_cast<char*>(p.dx) + row * p.lddx + th.off(v)) = from_floats<E>(x);
    }
    stage = stage + 1 == S ? 0 : stage + 1;
  }
  copy_wait<0>();
  if (!p.partial) return;

  // This CTA's sums, over its teams in order (the queues' memory is reused).
  constexpr int kWide = W * 32 * V * kPer<E>;
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll 1
  for (int which = 0; which < 2; ++which) {
    if (which && !p.want_bias) break;
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < kPer<E>; ++e)
        sums[th.team * kWide + (v * W * 32 + th.t) * kPer<E> + e] = which ? db[v][e] : dg[v][e];
    __syncthreads();
    float* out = p.partial + (static_cast<int64_t>(which) * gridDim.x + blockIdx.x) * p.cols;
    for (int c = threadIdx.x; c < p.cols; c += kThreads) {
      float s = 0.0f;
#pragma unroll
      for (int k = 0; k < kWarps / W; ++k) s += sums[k * kWide + c];
      out[c] = s;
    }
  }
}

// The CTAs' sums of 32 columns, added in a fixed order: dgain (blockIdx.y = 0)
// and dbias.
template <typename E>
__global__ void __launch_bounds__(1024) tpmlp_norm_gain_grad(const float* partial, int cols, int ctas, E* dgain,
                                                             E* dbias) {
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + c;
  E* dst = blockIdx.y ? dbias : dgain;
  if (!dst) return;
  const float* src = partial + static_cast<int64_t>(blockIdx.y) * ctas * cols;
  float v = 0.0f;
  if (e < cols)
    for (int i = r; i < ctas; i += 32) v += src[static_cast<int64_t>(i) * cols + e];
  s[r][c] = v;
  __syncthreads();
  if (r == 0 && e < cols) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][c];
    if constexpr (sizeof(E) == 2) dst[e] = __float2bfloat16_rn(t);
    else dst[e] = t;
  }
}

using NormKernel = void (*)(NormParams);
struct Pick {
  NormKernel kernel;
  int W, V;
};

// The team and the vectors a thread holds: up to 32 elements a thread, then up
// to 16 warps a token.
template <typename E, int W, int V>
Pick pick_one(bool bwd) {
  return {bwd ? tpmlp_norm_bwd<E, W, V> : tpmlp_norm_fwd<E, W, V>, W, V};
}

template <typename E>
Pick pick(int cols, bool bwd) {
  constexpr int V = 32 / kPer<E>;
  if (cols <= 256) return pick_one<E, 1, V / 4>(bwd);
  if (cols <= 512) return pick_one<E, 1, V / 2>(bwd);
  if (cols <= 1024) return pick_one<E, 1, V>(bwd);
  if (cols <= 2048) return pick_one<E, 2, V>(bwd);
  if (cols <= 4096) return pick_one<E, 4, V>(bwd);
  if (cols <= 8192) return pick_one<E, 8, V>(bwd);
  return pick_one<E, 16, V>(bwd);
}

}  // namespace

cudaError_t launch_norm(NormParams& p, bool bf16, bool bwd, int sms, cudaStream_t stream) {
  if (p.rows <= 0) return cudaSuccess;
  const Pick k = bf16 ? pick<__nv_bfloat16>(p.cols, bwd) : pick<float>(p.cols, bwd);
  const int arrays = bwd ? (p.dsum ? 3 : 2) : (p.res ? 2 : 1);
  const int stage = arrays * k.V * kThreads * 16;
  p.stages = std::max(1, std::min(kMaxStages, (kMaxSmem - 1024) / stage));
  const int sums = bwd ? kThreads * k.V * (bf16 ? 8 : 4) * 4 : 0;
  const int bytes = std::max(p.stages * stage, sums);
  cudaError_t e = cudaFuncSetAttribute(k.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem - 1024);
  if (e != cudaSuccess) return e;
  p.ctas = static_cast<int32_t>(std::min<int64_t>(p.rows, std::min(sms, kNormMaxCtas)));
  k.kernel<<<p.ctas, kThreads, bytes, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_norm_gain_grad(const NormParams& p, bool bf16, void* dgain, void* dbias, cudaStream_t stream) {
  const dim3 grid((p.cols + 31) / 32, dbias ? 2 : 1);
  if (bf16)
    tpmlp_norm_gain_grad<__nv_bfloat16><<<grid, 1024, 0, stream>>>(
        p.partial, p.cols, p.ctas, static_cast<__nv_bfloat16*>(dgain), static_cast<__nv_bfloat16*>(dbias));
  else
    tpmlp_norm_gain_grad<float><<<grid, 1024, 0, stream>>>(p.partial, p.cols, p.ctas, static_cast<float*>(dgain),
                                                           static_cast<float*>(dbias));
  return cudaGetLastError();
}

}  // namespace tpmlp
