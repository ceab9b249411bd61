// qk_norm_rope.cu -- RMS norm of every query and key head and the position
// rotation, in one pass over the shards' fused QKV buffers, and its backward
// pass.
//
// One head x of D elements of the token at position p (fp32 throughout, each
// output rounded once to the storage type):
//   r = (mean(x^2) + eps)^(-1/2),  u = g * x * r          (g: a gain per element)
//   pair j < R/2, phi = p f_j:  a' = u_a cos phi - u_b sin phi,
//                               b' = u_b cos phi + u_a sin phi
//   elements past R are stored as u.  A pair is (j, j + R/2) or (2j, 2j + 1).
// Backward, from dy: w = dy rotated back, n = x r, s = w g:
//   dx = r (s - n mean(s n)),  dg = sum over tokens and heads of w n.
//
// The angle.  f_j is held as a 64-bit fraction of a turn, F_j = 2^64 f_j / 2 pi,
// and p F_j is taken modulo 2^64, which drops whole turns exactly; the top 32
// bits are the angle in units of 2^-32 turn.  Its error is the rounding of
// F_j (below 2^-53 f_j) times p, as that of the product in 64-bit floating
// point, without 64-bit floating-point instructions.
//
// Layout of the work.  HBM-bound: a head is read and written once.  A lane
// holds a unit: V pairs, i.e. two vectors of V elements, both partners of each
// pair, so that the rotation needs no exchange; L lanes (a power of two)
// share a head and add its sum of squares by shuffles; a warp takes 32 / L
// heads at a time, all heads of one kind (queries or keys) of one token, one
// after another, with that token's sines and cosines in registers.  CTAs belong
// to one kind, so that the gains (and, backward, the lane's sums of the gain's
// gradient) stay in registers for the whole launch; the host deals the CTAs
// to the kinds in proportion to their bytes.  With few tokens the heads of a
// token are split over several warps.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;

// V elements of the storage type at p, as floats.
template <typename E, int V>
__device__ __forceinline__ void load_vec(const E* p, float (&v)[V]) {
  if constexpr (sizeof(E) == 2) {
    if constexpr (V == 8) {
      const uint4 q = *reinterpret_cast<const uint4*>(p);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        v[2 * e] = __uint_as_float(w[e] << 16);
        v[2 * e + 1] = __uint_as_float(w[e] & 0xffff0000u);
      }
    } else if constexpr (V == 4) {
      const uint2 q = *reinterpret_cast<const uint2*>(p);
      v[0] = __uint_as_float(q.x << 16);
      v[1] = __uint_as_float(q.x & 0xffff0000u);
      v[2] = __uint_as_float(q.y << 16);
      v[3] = __uint_as_float(q.y & 0xffff0000u);
    } else {
      v[0] = __bfloat162float(*p);
    }
  } else {
    if constexpr (V == 4) {
      const float4 q = *reinterpret_cast<const float4*>(p);
      v[0] = q.x;
      v[1] = q.y;
      v[2] = q.z;
      v[3] = q.w;
    } else {
      v[0] = *p;
    }
  }
}

__device__ __forceinline__ uint32_t pack2(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

template <typename E, int V>
__device__ __forceinline__ void store_vec(E* p, const float (&v)[V]) {
  if constexpr (sizeof(E) == 2) {
    if constexpr (V == 8) {
      *reinterpret_cast<uint4*>(p) =
          make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    } else if constexpr (V == 4) {
      *reinterpret_cast<uint2*>(p) = make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
    } else {
      *p = __float2bfloat16_rn(v[0]);
    }
  } else {
    if constexpr (V == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else {
      *p = v[0];
    }
  }
}

// A unit of V pairs between its two stored vectors and the partners (a, b).
// Halves: vector 0 holds the a's, vector 1 the b's.  Pairs: the 2V elements
// are a0 b0 a1 b1 ...
template <typename E, int V, bool kPairs>
__device__ __forceinline__ void load_unit(const E* row, int o1, int o2, float (&a)[V], float (&b)[V]) {
  float v1[V], v2[V];
  load_vec<E, V>(row + o1, v1);
  load_vec<E, V>(row + o2, v2);
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (kPairs && V > 1) {
      a[k] = 2 * k < V ? v1[(2 * k) % V] : v2[(2 * k) % V];
      b[k] = 2 * k + 1 < V ? v1[(2 * k + 1) % V] : v2[(2 * k + 1) % V];
    } else {
      a[k] = v1[k];
      b[k] = v2[k];
    }
  }
}

template <typename E, int V, bool kPairs>
__device__ __forceinline__ void store_unit(E* row, int o1, int o2, const float (&a)[V], const float (&b)[V]) {
  float v1[V], v2[V];
#pragma unroll
  for (int k = 0; k < V; ++k) {
    if (kPairs && V > 1) {
      v1[k] = k % 2 == 0 ? a[k / 2] : b[k / 2];
      v2[k] = k % 2 == 0 ? a[V / 2 + k / 2] : b[V / 2 + k / 2];
    } else {
      v1[k] = a[k];
      v2[k] = b[k];
    }
  }
  store_vec<E, V>(row + o1, v1);
  store_vec<E, V>(row + o2, v2);
}

// Where unit u of a head lies, and its first pair (-1: not rotated).  Halves:
// the units of the rotated part, then the rest cut into neighbouring vectors.
template <int V, bool kPairs>
__device__ __forceinline__ void unit_at(int u, int R, int& o1, int& o2, int& j0) {
  if (kPairs) {
    o1 = 2 * V * u;
    o2 = o1 + V;
    j0 = V * u;
    return;
  }
  const int ru = R / (2 * V);
  if (u < ru) {
    o1 = V * u;
    o2 = R / 2 + V * u;
    j0 = V * u;
  } else {
    o1 = R + 2 * V * (u - ru);
    o2 = o1 + V;
    j0 = R;  // past the last pair
  }
}

// The shard and the position in it of a kind's head h, counted over shards.
__device__ __forceinline__ int shard_of_head(const QkParams& p, int kind, int h, int from) {
  while (h >= p.head_end[kind][from]) ++from;
  return from;
}

// One kind's heads of a warp's tokens: this warp is w of nw of that kind,
// part w % parts of the heads of tokens w / parts, + nw / parts, ...
template <typename E, int V, int NU, bool kPairs, bool kBwd>
__device__ __forceinline__ void qk_walk(const QkParams& p, int kind, int w, int nw, float (&dga)[NU][V],
                                        float (&dgb)[NU][V]) {
  const int lane = threadIdx.x & 31;
  const int L = p.lanes;
  const int G = 32 / L;  // heads of a warp at a time
  const int grp = lane / L, li = lane % L;
  const int units = p.D / (2 * V);
  const int parts = p.parts[kind];
  const int heads = p.heads[kind];
  const float inv_d = 1.0f / static_cast<float>(p.D);

  int o1[NU], o2[NU];
  bool on[NU];
  float ga[NU][V], gb[NU][V];
  uint64_t F[NU][V];
  const E* g = static_cast<const E*>(p.gain[kind]);
#pragma unroll
  for (int n = 0; n < NU; ++n) {
    const int u = li + n * L;
    on[n] = u < units;
    int j0;
    unit_at<V, kPairs>(on[n] ? u : 0, p.R, o1[n], o2[n], j0);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      ga[n][k] = gb[n][k] = 1.0f;
      F[n][k] = 2 * (j0 + k) < p.R ? p.freq[j0 + k] : 0;  // 0: the rotation by no angle
    }
    if (g && on[n]) load_unit<E, V, kPairs>(g, o1[n], o2[n], ga[n], gb[n]);
  }

  const int rows = nw / parts;  // tokens at a time; warps left over have none
  for (int64_t tok = w < rows * parts ? w / parts : p.T; tok < p.T; tok += rows) {
    const uint64_t pos = p.pos ? static_cast<uint64_t>(p.pos[tok]) : static_cast<uint64_t>(tok);
    float cs[NU][V], sn[NU][V];
#pragma unroll
    for (int n = 0; n < NU; ++n)
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int32_t turn = static_cast<int32_t>((pos * F[n][k]) >> 32);  // in 2^-32 turns
        sincospif(static_cast<float>(turn) * 0x1p-31f, &sn[n][k], &cs[n][k]);
      }
    int sh = 0;
    for (int h0 = (w % parts) * G; h0 < heads; h0 += parts * G) {
      const int h = h0 + grp;
      const bool ok = h < heads;
      sh = shard_of_head(p, kind, ok ? h : heads - 1, sh);
      const QkShard& S = p.shards[sh];
      const int col = S.col[kind] + ((ok ? h : heads - 1) - (sh ? p.head_end[kind][sh - 1] : 0)) * p.D;
      const E* x = static_cast<const E*>(S.x) + tok * S.ldx + col;
      float a[NU][V], b[NU][V], ya[NU][V], yb[NU][V];
      float ss = 0.0f;
#pragma unroll
      for (int n = 0; n < NU; ++n) {
#pragma unroll
        for (int k = 0; k < V; ++k) a[n][k] = b[n][k] = ya[n][k] = yb[n][k] = 0.0f;
        if (ok && on[n]) {
          load_unit<E, V, kPairs>(x, o1[n], o2[n], a[n], b[n]);
          if (kBwd)
            load_unit<E, V, kPairs>(static_cast<const E*>(S.dy) + tok * S.lddy + col, o1[n], o2[n], ya[n], yb[n]);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) ss = fmaf(a[n][k], a[n][k], fmaf(b[n][k], b[n][k], ss));
      }
      float r = 1.0f;
      if (p.norm) {
        for (int o = L >> 1; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
        r = rsqrtf(fmaf(ss, inv_d, p.eps));
      }
      E* out = static_cast<E*>(S.out) + tok * S.ldo + col;
      if (!kBwd) {
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          if (!(ok && on[n])) continue;
          float oa[V], ob[V];
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const float ua = a[n][k] * r * ga[n][k], ub = b[n][k] * r * gb[n][k];
            oa[k] = ua * cs[n][k] - ub * sn[n][k];
            ob[k] = ub * cs[n][k] + ua * sn[n][k];
          }
          store_unit<E, V, kPairs>(out, o1[n], o2[n], oa, ob);
        }
      } else {
        float m = 0.0f;
#pragma unroll
        for (int n = 0; n < NU; ++n)
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const float wa = ya[n][k] * cs[n][k] + yb[n][k] * sn[n][k];
            const float wb = yb[n][k] * cs[n][k] - ya[n][k] * sn[n][k];
            a[n][k] *= r;  // n = x r
            b[n][k] *= r;
            dga[n][k] = fmaf(wa, a[n][k], dga[n][k]);
            dgb[n][k] = fmaf(wb, b[n][k], dgb[n][k]);
            ya[n][k] = wa * ga[n][k];
            yb[n][k] = wb * gb[n][k];
            m = fmaf(ya[n][k], a[n][k], fmaf(yb[n][k], b[n][k], m));
          }
        if (p.norm) {
          for (int o = L >> 1; o > 0; o >>= 1) m += __shfl_xor_sync(0xffffffffu, m, o);
          m *= inv_d;
        } else {
          m = 0.0f;
        }
#pragma unroll
        for (int n = 0; n < NU; ++n) {
          if (!(ok && on[n])) continue;
          float oa[V], ob[V];
#pragma unroll
          for (int k = 0; k < V; ++k) {
            oa[k] = r * (ya[n][k] - a[n][k] * m);
            ob[k] = r * (yb[n][k] - b[n][k] * m);
          }
          store_unit<E, V, kPairs>(out, o1[n], o2[n], oa, ob);
        }
      }
    }
  }
}

// dV into the value columns of dQKV: 16 bytes a lane.
template <typename E>
__device__ __forceinline__ void copy_values(const QkParams& p, int w, int nw) {
  constexpr int V = 16 / sizeof(E);
  const int lane = threadIdx.x & 31;
  for (int64_t tok = w; tok < p.T; tok += nw) {
    for (int s = 0; s < p.t; ++s) {
      const QkShard& S = p.shards[s];
      const uint4* src = reinterpret_cast<const uint4*>(static_cast<const E*>(S.dv) + tok * S.dkv);
      uint4* dst = reinterpret_cast<uint4*>(static_cast<E*>(S.out) + tok * S.ldo + S.vcol);
      for (int c = lane; c < S.dkv / V; c += 32) dst[c] = src[c];
    }
  }
}

template <typename E, int V, int NU, bool kPairs, bool kBwd>
__device__ __forceinline__ void qk_body(const QkParams& p) {
  const int cta = blockIdx.x, warp = threadIdx.x >> 5;
  const int kind = cta < p.cta_end[0] ? 0 : cta < p.cta_end[1] ? 1 : 2;
  const int c0 = kind ? p.cta_end[kind - 1] : 0;
  const int w = (cta - c0) * kWarps + warp, nw = (p.cta_end[kind] - c0) * kWarps;
  if (kind == 2) {
    if (kBwd) copy_values<E>(p, w, nw);
    return;
  }
  float dga[NU][V], dgb[NU][V];
#pragma unroll
  for (int n = 0; n < NU; ++n)
#pragma unroll
    for (int k = 0; k < V; ++k) dga[n][k] = dgb[n][k] = 0.0f;
  qk_walk<E, V, NU, kPairs, kBwd>(p, kind, w, nw, dga, dgb);
  if (!kBwd || !p.partial) return;

  // This CTA's sum of the gain's gradient: over the groups of a warp by
  // shuffles, over the warps in shared memory, in a fixed order.
  __shared__ float sums[kWarps][kMaxHeadDim];
  const int lane = threadIdx.x & 31, L = p.lanes;
#pragma unroll
  for (int n = 0; n < NU; ++n)
#pragma unroll
    for (int k = 0; k < V; ++k)
      for (int o = L; o < 32; o <<= 1) {
        dga[n][k] += __shfl_xor_sync(0xffffffffu, dga[n][k], o);
        dgb[n][k] += __shfl_xor_sync(0xffffffffu, dgb[n][k], o);
      }
  if (lane < L) {
#pragma unroll
    for (int n = 0; n < NU; ++n) {
      const int u = lane + n * L;
      if (u >= p.D / (2 * V)) continue;
      int o1, o2, j0;
      unit_at<V, kPairs>(u, p.R, o1, o2, j0);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int ea = kPairs ? o1 + 2 * k : o1 + k, eb = kPairs ? o1 + 2 * k + 1 : o2 + k;
        sums[warp][ea] = dga[n][k];
        sums[warp][eb] = dgb[n][k];
      }
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.D; e += kThreads) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) s += sums[i][e];
    p.partial[static_cast<int64_t>(cta) * p.D + e] = s;
  }
}

template <typename E, int V, int NU, bool kPairs>
__global__ void __launch_bounds__(kThreads) tpmlp_attn_qk_norm_rope_fwd(const __grid_constant__ QkParams p) {
  qk_body<E, V, NU, kPairs, false>(p);
}

template <typename E, int V, int NU, bool kPairs>
__global__ void __launch_bounds__(kThreads) tpmlp_attn_qk_norm_rope_bwd(const __grid_constant__ QkParams p) {
  qk_body<E, V, NU, kPairs, true>(p);
}

// dg of one kind (blockIdx.y) for 32 elements: the CTAs' sums added in a
// fixed order.
template <typename E>
__global__ void __launch_bounds__(1024) tpmlp_attn_qk_gain_grad(const float* partial, int D, int end0, int end1,
                                                               E* dgq, E* dgk) {
  __shared__ float s[32][33];
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  const int e = blockIdx.x * 32 + c;
  const int first = blockIdx.y ? end0 : 0, last = blockIdx.y ? end1 : end0;
  E* dg = blockIdx.y ? dgk : dgq;
  float v = 0.0f;
  if (e < D)
    for (int i = first + r; i < last; i += 32) v += partial[static_cast<int64_t>(i) * D + e];
  s[r][c] = v;
  __syncthreads();
  if (r == 0 && e < D && dg) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) t += s[i][c];
    if constexpr (sizeof(E) == 2) dg[e] = __float2bfloat16_rn(t);
    else dg[e] = t;
  }
}

using QkKernel = void (*)(QkParams);

template <typename E, int V, int NU>
QkKernel pick(bool pairs, bool bwd) {
  if (bwd) return pairs ? tpmlp_attn_qk_norm_rope_bwd<E, V, NU, true> : tpmlp_attn_qk_norm_rope_bwd<E, V, NU, false>;
  return pairs ? tpmlp_attn_qk_norm_rope_fwd<E, V, NU, true> : tpmlp_attn_qk_norm_rope_fwd<E, V, NU, false>;
}

// The widest vector (in elements) that every part of a head is a whole number
// of: 16 bytes, 8 bytes (bf16), or one element.
int vector_width(bool bf16, int D, int R, bool pairs) {
  const int most = bf16 ? 8 : 4;
  for (int V = most; V >= 4; V /= 2)
    if (D % (2 * V) == 0 && (pairs || R % (2 * V) == 0)) return V;
  return 1;
}

QkKernel kernel_for(bool bf16, int V, bool pairs, bool bwd) {
  if (bf16) {
    if (V == 8) return pick<__nv_bfloat16, 8, 1>(pairs, bwd);
    if (V == 4) return pick<__nv_bfloat16, 4, 1>(pairs, bwd);
    return pick<__nv_bfloat16, 1, 4>(pairs, bwd);
  }
  if (V == 4) return pick<float, 4, 1>(pairs, bwd);
  return pick<float, 1, 4>(pairs, bwd);
}

}  // namespace

// Lays the launch out (lanes, parts, CTAs of each kind) and launches it.
cudaError_t launch_qk_norm_rope(QkParams& p, bool bf16, bool pairs, bool bwd, int sms, cudaStream_t stream) {
  if (p.T <= 0) return cudaSuccess;
  const int V = vector_width(bf16, p.D, p.R, pairs);
  const int units = p.D / (2 * V);
  int L = 1;
  while (L < units && L < 32) L *= 2;
  p.lanes = L;
  const int G = 32 / L;
  const QkKernel k = kernel_for(bf16, V, pairs, bwd);
  static std::atomic<int> resident[2][9][2][2];  // CTAs per SM of each kernel, once known
  std::atomic<int>& known = resident[bf16][V][pairs][bwd];
  int per_sm = known.load(std::memory_order_relaxed);
  if (per_sm == 0) {
    const cudaError_t e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, kThreads, 0);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    known.store(per_sm, std::memory_order_relaxed);
  }
  const int slots = sms * per_sm;
  const int64_t most_warps = int64_t{slots} * kWarps;

  // Heads of a token in parts, so that a launch of few tokens still has a
  // warp for every slot: a part is a whole number of rounds of G heads.
  int rounds[2], most_rounds = 1;
  for (int kind = 0; kind < 2; ++kind) {
    rounds[kind] = (p.heads[kind] + G - 1) / G;
    most_rounds = rounds[kind] > most_rounds ? rounds[kind] : most_rounds;
  }
  int per_part = most_rounds;
  while (per_part > 1 && p.T * ((rounds[0] + per_part - 1) / per_part + (rounds[1] + per_part - 1) / per_part) < most_warps)
    per_part = (per_part + 1) / 2;
  // CTAs of each kind in proportion to its bytes.
  int64_t cost[3], total = 0, want[3];
  for (int kind = 0; kind < 2; ++kind) {
    p.parts[kind] = (rounds[kind] + per_part - 1) / per_part;
    cost[kind] = static_cast<int64_t>(p.heads[kind]) * p.D * (bwd ? 3 : 2);
    want[kind] = (p.T * p.parts[kind] + kWarps - 1) / kWarps;
  }
  cost[2] = bwd && p.values ? p.values * 2 : 0;
  want[2] = cost[2] ? (p.T + kWarps - 1) / kWarps : 0;
  for (int kind = 0; kind < 3; ++kind) total += cost[kind];
  int end = 0;
  for (int kind = 0; kind < 3; ++kind) {
    int64_t n = (cost[kind] * slots + total - 1) / total;
    if (n > want[kind]) n = want[kind];
    if (kind < 2) n = std::max<int64_t>(n, (p.parts[kind] + kWarps - 1) / kWarps);  // a warp for every part
    end += static_cast<int>(n);
    p.cta_end[kind] = end;
  }
  if (end > kQkMaxCtas) return cudaErrorInvalidConfiguration;  // parts < 2 x the slots' warps: not reached
  k<<<end, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

cudaError_t launch_qk_gain_grad(const QkParams& p, bool bf16, void* dgq, void* dgk, cudaStream_t stream) {
  const dim3 grid((p.D + 31) / 32, 2);
  if (bf16)
    tpmlp_attn_qk_gain_grad<__nv_bfloat16><<<grid, 1024, 0, stream>>>(
        p.partial, p.D, p.cta_end[0], p.cta_end[1], static_cast<__nv_bfloat16*>(dgq), static_cast<__nv_bfloat16*>(dgk));
  else
    tpmlp_attn_qk_gain_grad<float><<<grid, 1024, 0, stream>>>(p.partial, p.D, p.cta_end[0], p.cta_end[1],
                                                              static_cast<float*>(dgq), static_cast<float*>(dgk));
  return cudaGetLastError();
}

}  // namespace tpmlp
