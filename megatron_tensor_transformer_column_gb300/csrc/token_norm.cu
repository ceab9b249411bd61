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
// that a mean far larger than the spread costs r no digits.  mu itself is one fp32
// number: what its sum and rounding leave it off by, up to 56 2^-24 mean|s|, shifts
// every n of the token by r times that, in the backward pass too, which takes the
// stored statistics as they are.
//
// Layout of the work.  HBM-bound: every array is read or written once.  A token
// belongs to a team of W warps, up to 32 elements a thread, always the same
// columns, so that the sums of the gain's and the bias's gradients stay in
// registers for the whole launch (two a column: backward there is no room for
// gain or token beside them, both are read twice from shared memory).  Each
// thread copies its own 16-byte vectors of the next tokens into shared memory by
// itself (asynchronous copies, a queue per thread) and reads back only what it
// copied: no barrier but those of the sums over a token, and bytes in flight
// without registers.  One CTA of 512 threads an SM walks the tokens.  The
// gradients' sums are added over a CTA's teams, then over the CTAs by a second
// launch, each in a fixed order.
//
// Measured on GB300, bf16, device time and share of the copy bandwidth:
//   8192 x 16384: forward 84 to 93 us (0.94 to 0.85), with the sum 173 to 180
//     (0.89), backward 132 (0.90), with dsum 161 us (0.98)
//   8192 x 4096:  22 to 24 (0.87), 46 (0.86), 35 (0.84), 45 us (0.88); 32768 x
//     4096: 93 (0.85), 175 (0.90), 129 (0.92), 156 us (1.01)
//   65536 x 256 (layer norm with bias): 18 (0.55), 23 (0.88), 25 (0.60), 31 us
//     (0.64); 16384 x 64: 7 us forward, 10 backward (0.1)
//   fp32, 8192 x 16384: 175 (0.91), 320 (0.99), 259 (0.91), 329 us (0.96); 8192 x
//     4096: 50 (0.80), 93 (0.86), 71 (0.83), 90 us (0.87); 8192 x 2048 (layer norm
//     with bias): 25 (0.80), 50 (0.80), 44 (0.67), 54 us (0.74)
//   8192 x 768 (layer norm with bias): forward with the sum 8.4, backward with dsum
//     12.4 us, 3 of them the second launch; one token of 4096 3.6 and 5.8 us
// A first version, one element an instruction and with a branch around every
// vector, took 188 and 243 us on the first shape: bound by issue (33 instructions
// an element backward, now 22 and half of the issue slots) and by each token's
// chain of sum, barrier and store.  What bounds it now is HBM where tokens are
// many; with the sum, two arrays written for two read; with 8192 x 4096 also the
// launch's ramp and its last round (13.5 tokens a team).  Narrow tokens are a warp's
// each, and 16 warps an SM do not hide a token's chain of wait, sums over the lanes,
// root and store; below 256 columns lanes are idle as well.  fp32 backward, 8
// vectors of x and dy a thread fill shared memory, so that there is one stage and
// a token's loads wait for the token before.  64 elements a thread
// forward (175 us on 8192 x 16384 with the sum, 2 to 10 % slower elsewhere),
// streaming stores and L2 prefetch hints (within 1 %) were measured and not kept.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

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

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSmem = 227 * 1024;
constexpr int kMaxStages = 6;
// Forward, a stage is refilled as soon as it is in registers, and 64 KB on their
// way to an SM are best: with all of shared memory 8192 x 4096 with the sum takes
// 48 us instead of 46, 32768 x 4096 180 instead of 174, one token 4.3 instead of
// 3.6; with less, 65536 x 256 with the sum 29 instead of 22.  Backward a stage is free only
// when its token is done: two of them (one: 30 % slower; three: 0 to 3 %).
constexpr int kFlight = 64 * 1024;

template <typename E>
constexpr int kPer = 16 / static_cast<int>(sizeof(E));  // elements of a vector

// A vector as pairs of floats (one fp32x2 instruction each), and back.
template <typename E>
__device__ __forceinline__ void to_pairs(uint4 q, uint64_t (&v)[kPer<E> / 2]) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  if constexpr (sizeof(E) == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pk(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xffff0000u));
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) v[e] = pk(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
  }
}

template <typename E>
__device__ __forceinline__ uint4 from_pairs(const uint64_t (&v)[kPer<E> / 2]) {
  uint32_t w[4];
  if constexpr (sizeof(E) == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float lo, hi;
      upk(v[e], lo, hi);
      const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
      w[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float lo, hi;
      upk(v[e], lo, hi);
      w[2 * e] = __float_as_uint(lo);
      w[2 * e + 1] = __float_as_uint(hi);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ float both(uint64_t v) {
  float lo, hi;
  upk(v, lo, hi);
  return lo + hi;
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
      for (int w = 0; w < W; w += 2) {
        const float4 f = *reinterpret_cast<const float4*>(mine + w);
        a += f.x;
        b += f.y;
        a += f.z;
        b += f.w;
      }
      half ^= 1;
    } else {
      __syncwarp();  // keeps what follows from being fetched early, into registers that are not there
    }
    return make_float2(a, b);
  }
  __device__ __forceinline__ float operator()(float a, int warp_in_team) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o);
    if constexpr (W > 1) {
      float* mine = reinterpret_cast<float*>(red + half * W);
      if ((threadIdx.x & 31) == 0) mine[warp_in_team] = a;
      asm volatile("bar.sync %0, %1;" ::"r"(bar), "n"(W * 32) : "memory");
      a = 0.0f;
#pragma unroll
      for (int w = 0; w < W; w += 2) {
        const float2 f = *reinterpret_cast<const float2*>(mine + w);
        a += f.x;
        a += f.y;
      }
      half ^= 1;
    }
    return a;
  }
};

// Where a thread stands: vector v of its V is columns (v W 32 + t) kPer on.  A
// vector past the end (on[v] false) is never copied; its slots in the queue hold
// zeros from the start, so that the arithmetic needs no branches.
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
  // Vector v of a parameter, or `none` where there is none or it is past the end.
  __device__ __forceinline__ uint4 param(const void* p, int v, uint32_t none) const {
    if (p && on[v]) return *reinterpret_cast<const uint4*>(static_cast<const char*>(p) + off(v));
    return make_uint4(none, none, none, none);
  }
};

// A thread's queue in shared memory: slots of 16 bytes, [stage][array][vector].
constexpr uint32_t kSlot = kThreads * 16;
template <int V>
__device__ __forceinline__ uint32_t slot(uint32_t stage, int array, int v) {
  return stage + static_cast<uint32_t>(array * V + v) * kSlot;
}

template <typename E>
constexpr bool kGainInSmem = sizeof(E) == 2;
template <typename E>
constexpr uint32_t kOnes = sizeof(E) == 2 ? 0x3f803f80u : 0x3f800000u;

template <typename E, int W, int V>
__global__ void __launch_bounds__(kThreads, 1) tpmlp_norm_fwd(const __grid_constant__ NormParams p) {
  constexpr int P = kPer<E> / 2;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float2 red[2 * kWarps];
  const Thread<E, W, V> th(p.cols);
  TeamSum<W> sum{red + th.team * 2 * W, 1 + th.team, 0};
  const bool add = p.res != nullptr;
  const int S = p.stages;
  // In front of the queue (bf16): the vectors of gain and bias, one copy for all teams.
  constexpr uint32_t kParamBytes = kGainInSmem<E> ? V * W * 32 * 16 : 0;
  const uint32_t gains = ptx::smem_u32(smem) + th.t * 16, biases = gains + kParamBytes;
  const uint32_t base = ptx::smem_u32(smem) + (p.bias ? 2 : 1) * kParamBytes + threadIdx.x * 16;
  const uint32_t stage_bytes = (add ? 2 : 1) * V * kSlot;

  auto fetch = [&](int64_t row, uint32_t stage) {
    if (row < p.rows) {
      const char* x = static_cast<const char*>(p.x) + row * p.ldx;
      const char* r = static_cast<const char*>(p.res) + row * p.ldr;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (th.on[v]) copy16(slot<V>(stage, 0, v), x + th.off(v));
        if (add && th.on[v]) copy16(slot<V>(stage, 1, v), r + th.off(v));
      }
    }
    copy_commit();
  };

  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!th.on[v]) {
        ptx::st_shared_v4(slot<V>(base + i * stage_bytes, 0, v), make_uint4(0, 0, 0, 0));
        if (add) ptx::st_shared_v4(slot<V>(base + i * stage_bytes, 1, v), make_uint4(0, 0, 0, 0));
      }
  for (int i = 0; i < S; ++i) fetch(th.first + i * th.step, base + i * stage_bytes);
  if (kGainInSmem<E>) {
    // every team writes the same: a thread reads back what it wrote, or the same from another
#pragma unroll
    for (int v = 0; v < V; ++v) {
      ptx::st_shared_v4(gains + v * (W * 32 * 16), th.param(p.gain, v, kOnes<E>));
      if (p.bias) ptx::st_shared_v4(biases + v * (W * 32 * 16), th.param(p.bias, v, 0));
    }
  }
  auto param = [&](const void* src, uint32_t at, int v, uint32_t none) {
    return kGainInSmem<E> ? ptx::ld_shared_v4(at + v * (W * 32 * 16)) : th.param(src, v, none);
  };
  int at = 0;
#pragma unroll 1
  for (int64_t row = th.first; row < p.rows; row += th.step) {
    copy_wait_all_but(S - 1);
    const uint32_t stage = base + at * stage_bytes;
    at = at + 1 == S ? 0 : at + 1;
    uint64_t x[V][P];
#pragma unroll
    for (int v = 0; v < V; ++v) to_pairs<E>(ptx::ld_shared_v4(slot<V>(stage, 0, v)), x[v]);
    if (add) {
#pragma unroll
      for (int v = 0; v < V; ++v) {
        uint64_t r[P];
        to_pairs<E>(ptx::ld_shared_v4(slot<V>(stage, 1, v)), r);
#pragma unroll
        for (int e = 0; e < P; ++e) x[v][e] = add2(x[v][e], r[e]);
        const uint4 q = from_pairs<E>(x[v]);
        if (th.on[v]) *reinterpret_cast<uint4*>(static_cast<char*>(p.sum) + row * p.lds + th.off(v)) = q;
        to_pairs<E>(q, x[v]);
      }
    }
    fetch(row + S * th.step, stage);  // what lay there is in registers
    float mu = 0.0f;
    if (!p.rms) {
      uint64_t a = 0;
#pragma unroll
      for (int v = 0; v < V; ++v)
#pragma unroll
        for (int e = 0; e < P; ++e) a = add2(a, x[v][e]);
      mu = sum(both(a), th.warp_in_team) * p.inv_cols;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const uint64_t shift = splat(th.on[v] ? -mu : 0.0f);
#pragma unroll
        for (int e = 0; e < P; ++e) x[v][e] = add2(x[v][e], shift);
      }
    }
    uint64_t a = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < P; ++e) a = fma2(x[v][e], x[v][e], a);
    const float r = rsqrtf(fmaf(sum(both(a), th.warp_in_team), p.inv_cols, p.eps));
    if (th.t == 0 && p.stats) reinterpret_cast<float2*>(p.stats)[row] = make_float2(mu, r);
    const uint64_t r2 = splat(r);
    char* y = static_cast<char*>(p.y) + row * p.ldy;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint64_t g[P];
      to_pairs<E>(param(p.gain, gains, v, kOnes<E>), g);
      if (p.bias) {
        uint64_t b[P];
        to_pairs<E>(param(p.bias, biases, v, 0), b);
#pragma unroll
        for (int e = 0; e < P; ++e) x[v][e] = fma2(mul2(x[v][e], r2), g[e], b[e]);
      } else {
#pragma unroll
        for (int e = 0; e < P; ++e) x[v][e] = mul2(mul2(x[v][e], r2), g[e]);
      }
      if (th.on[v]) *reinterpret_cast<uint4*>(y + th.off(v)) = from_pairs<E>(x[v]);
    }
  }
  copy_wait<0>();
}

// kBias: dbias is summed up as well.
template <typename E, int W, int V, bool kBias>
__global__ void __launch_bounds__(kThreads, 1) tpmlp_norm_bwd(const __grid_constant__ NormParams p) {
  constexpr int P = kPer<E> / 2;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) float2 red[2 * kWarps];
  const Thread<E, W, V> th(p.cols);
  TeamSum<W> sum{red + th.team * 2 * W, 1 + th.team, 0};
  const bool add = p.dsum != nullptr;
  const int S = p.stages;
  // The gain's vectors lie in front of the queue (bf16; fp32 leaves no room for them beside the queue, they come from L2):
  // registers are for the sums.
  const uint32_t gains = ptx::smem_u32(smem) + threadIdx.x * 16, base = gains + (kGainInSmem<E> ? V * kSlot : 0);
  const uint32_t stage_bytes = (add ? 3 : 2) * V * kSlot;

  auto fetch = [&](int64_t row, uint32_t stage) {
    if (row < p.rows) {
      const char* x = static_cast<const char*>(p.x) + row * p.ldx;
      const char* dy = static_cast<const char*>(p.dy) + row * p.lddy;
      const char* ds = static_cast<const char*>(p.dsum) + row * p.ldds;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        if (th.on[v]) copy16(slot<V>(stage, 0, v), x + th.off(v));
        if (th.on[v]) copy16(slot<V>(stage, 1, v), dy + th.off(v));
        if (add && th.on[v]) copy16(slot<V>(stage, 2, v), ds + th.off(v));
      }
    }
    copy_commit();
  };

  for (int i = 0; i < S; ++i)
#pragma unroll
    for (int v = 0; v < V; ++v)
      if (!th.on[v]) {
        ptx::st_shared_v4(slot<V>(base + i * stage_bytes, 0, v), make_uint4(0, 0, 0, 0));
        ptx::st_shared_v4(slot<V>(base + i * stage_bytes, 1, v), make_uint4(0, 0, 0, 0));
      }
  for (int i = 0; i + 1 < S; ++i) fetch(th.first + i * th.step, base + i * stage_bytes);
  const float2* stats = reinterpret_cast<const float2*>(p.stats);
  float2 next = th.first < p.rows ? stats[th.first] : make_float2(0.0f, 0.0f);
  uint64_t dg[V][P], db[V][P];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    if (kGainInSmem<E>) ptx::st_shared_v4(slot<V>(gains, 0, v), th.param(p.gain, v, kOnes<E>));
#pragma unroll
    for (int e = 0; e < P; ++e) dg[v][e] = db[v][e] = 0;
  }
  int at = 0;
#pragma unroll 1
  for (int64_t row = th.first; row < p.rows; row += th.step) {
    fetch(row + (S - 1) * th.step, base + (at == 0 ? S - 1 : at - 1) * stage_bytes);
    const float mu = next.x, r = next.y;
    if (row + th.step < p.rows) next = stats[row + th.step];
    copy_wait_all_but(S - 1);
    const uint32_t stage = base + at * stage_bytes;
    at = at + 1 == S ? 0 : at + 1;
    const uint64_t shift = splat(-mu), r2 = splat(r);
    uint64_t sw = 0, swn = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint64_t x[P], w[P], g[P];
      to_pairs<E>(ptx::ld_shared_v4(slot<V>(stage, 0, v)), x);
      to_pairs<E>(ptx::ld_shared_v4(slot<V>(stage, 1, v)), w);
      to_pairs<E>(kGainInSmem<E> ? ptx::ld_shared_v4(slot<V>(gains, 0, v)) : th.param(p.gain, v, kOnes<E>), g);
#pragma unroll
      for (int e = 0; e < P; ++e) {
        const uint64_t n = mul2(add2(x[e], shift), r2);
        dg[v][e] = fma2(w[e], n, dg[v][e]);
        if (kBias) db[v][e] = add2(db[v][e], w[e]);
        w[e] = mul2(w[e], g[e]);
        sw = add2(sw, w[e]);
        swn = fma2(w[e], n, swn);
      }
    }
    const float2 m = sum(both(sw), both(swn), th.warp_in_team);
    // dx = r w - r mean(w) - (x - mu) r^2 mean(w n)
    const uint64_t c1 = splat(p.rms ? 0.0f : -(r * (m.x * p.inv_cols))), c2 = splat(-(r * r * (m.y * p.inv_cols)));
    char* dx = static_cast<char*>(p.dx) + row * p.lddx;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      uint64_t x[P], w[P], g[P];
      to_pairs<E>(ptx::ld_shared_v4(slot<V>(stage, 0, v)), x);
      to_pairs<E>(ptx::ld_shared_v4(slot<V>(stage, 1, v)), w);
      to_pairs<E>(kGainInSmem<E> ? ptx::ld_shared_v4(slot<V>(gains, 0, v)) : th.param(p.gain, v, kOnes<E>), g);
#pragma unroll
      for (int e = 0; e < P; ++e) x[e] = fma2(add2(x[e], shift), c2, fma2(mul2(w[e], g[e]), r2, c1));
      if (add) {
        to_pairs<E>(ptx::ld_shared_v4(slot<V>(stage, 2, v)), w);
#pragma unroll
        for (int e = 0; e < P; ++e) x[e] = add2(x[e], w[e]);
      }
      if (th.on[v]) *reinterpret_cast<uint4*>(dx + th.off(v)) = from_pairs<E>(x);
    }
  }
  copy_wait<0>();
  if (!p.partial) return;

  // This CTA's sums, over its teams in order (the queues' memory is reused).
  constexpr int kWide = W * 32 * V * kPer<E>;
  float* sums = reinterpret_cast<float*>(smem);
#pragma unroll
  for (int which = 0; which < (kBias ? 2 : 1); ++which) {
    __syncthreads();
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int e = 0; e < P; ++e) {
        float lo, hi;
        upk(which ? db[v][e] : dg[v][e], lo, hi);
        *reinterpret_cast<float2*>(sums + th.team * kWide + (v * W * 32 + th.t) * kPer<E> + 2 * e) =
            make_float2(lo, hi);
      }
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

template <typename E, int W, int V>
Pick pick_one(bool bwd, bool bias) {
  return {!bwd   ? tpmlp_norm_fwd<E, W, V>
          : bias ? tpmlp_norm_bwd<E, W, V, true>
                 : tpmlp_norm_bwd<E, W, V, false>,
          W, V};
}

// 24 or 32 elements a thread, whichever leaves fewer threads idle.
template <typename E, int W>
Pick pick_team(int cols, bool bwd, bool bias) {
  constexpr int V = 32 / kPer<E>;
  return cols <= W * 32 * 24 ? pick_one<E, W, V / 4 * 3>(bwd, bias) : pick_one<E, W, V>(bwd, bias);
}

// The team and the vectors a thread holds: up to 32 elements a thread, then up
// to 16 warps a token.
template <typename E>
Pick pick(int cols, bool bwd, bool bias) {
  constexpr int V = 32 / kPer<E>;
  if (cols <= 256) return pick_one<E, 1, V / 4>(bwd, bias);
  if (cols <= 512) return pick_one<E, 1, V / 2>(bwd, bias);
  if (cols <= 1024) return pick_team<E, 1>(cols, bwd, bias);
  if (cols <= 2048) return pick_team<E, 2>(cols, bwd, bias);
  if (cols <= 4096) return pick_team<E, 4>(cols, bwd, bias);
  if (cols <= 8192) return pick_team<E, 8>(cols, bwd, bias);
  return pick_team<E, 16>(cols, bwd, bias);
}

}  // namespace

cudaError_t launch_norm(NormParams& p, bool bf16, bool bwd, int sms, cudaStream_t stream) {
  if (p.rows <= 0) return cudaSuccess;
  const Pick k = bf16 ? pick<__nv_bfloat16>(p.cols, bwd, p.want_bias) : pick<float>(p.cols, bwd, p.want_bias);
  const int arrays = bwd ? (p.dsum ? 3 : 2) : (p.res ? 2 : 1);
  const int stage = arrays * k.V * kThreads * 16;
  int params = 0;  // gain (and bias) in front of the queue
  if (bf16) params = bwd ? k.V * kThreads * 16 : (p.bias ? 2 : 1) * k.V * k.W * 32 * 16;
  const int fit = (kMaxSmem - 1024 - params) / stage;
  p.stages = std::max(1, std::min(fit, bwd ? 2 : std::min(kMaxStages, kFlight / stage)));
  const int sums = bwd ? kThreads * k.V * (bf16 ? 8 : 4) * 4 : 0;
  const int bytes = std::max(params + p.stages * stage, sums);
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
