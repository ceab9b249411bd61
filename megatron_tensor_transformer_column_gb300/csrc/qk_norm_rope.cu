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
// Without a norm dx = w: that is the forward pass of dy with the angles
// negated, and the kernel without a norm runs both (x is not read).
//
// The angle.  f_j is held as a 64-bit fraction of a turn, F_j = 2^64 f_j / 2 pi,
// and p F_j is taken modulo 2^64, which drops whole turns exactly; the top 32
// bits are the angle in units of 2^-32 turn.  Its error is that of F_j times p:
// |p f_j| 2^-53 turns, as that of the product in 64-bit floating point, and
// |p| 2^-65 for the fraction's last bit (2^-25 turns at p = 2^40), without
// 64-bit floating-point instructions.
//
// Layout of the work.  HBM-bound: a head is read and written once.  A lane
// holds a unit: V pairs, i.e. two vectors of V elements, both partners of each
// pair, so that the rotation needs no exchange.  n lanes share a head and add
// its sums by shuffles; a warp takes 32 / n heads at a time (a round), all
// heads of one kind (queries or keys) of one token, round after round, with
// that token's sines and cosines in registers: they are computed once per
// token by all lanes, a pair each, and read back from shared memory.  Each
// lane's vectors of the next kStages - 1 rounds, of the next tokens too, are
// on their way into shared memory (16-byte asynchronous copies, a queue of
// its own per lane, so that nothing waits but the lane): bytes in flight
// without registers.  CTAs belong to one kind, so that the gains (and,
// backward, the lane's sums of the gain's gradient) stay with the CTA for the
// whole launch; the host deals the CTAs to the kinds by their work.  With few
// tokens the heads of a token are split over several warps.  Every CTA first
// copies its share of dV, eight 16-byte accesses of a lane in flight (CTAs of
// their own for it were the last to finish: 228 against 160 us on 8192 tokens
// of 8 shards of 16 + 1 heads of 128).
//
// Measured on GB300, bf16, device time and share of the copy bandwidth:
//   16384 tokens, 8 shards of 4 + 4 heads of 96:   68 us (0.87), backward 141 us (0.84);
//     without a norm 73 (0.81) and 100 us (0.89)
//   8192 tokens, 8 shards of 16 + 1 heads of 128: 102 us (0.82), backward 158 us (0.83);
//     without a norm 96 (0.88) and 100 us (0.89)
// A first version with the loads in registers and every lane computing its own
// angles took 147 and 359 us on the former: it was bound by instruction issue
// (250 instructions a round forward) and latency.  What bounds it now is issue
// and the latency of a round's chain (load, sum, root, store) together: 55 % of
// the issue slots taken (190 instructions a round, backward 370) with the warps
// an SM that the registers allow: 20 forward (92 registers), 16 backward (128).
// Two heads a lane and round (4 % less time on the former shape, 1 to 30 %
// more on small and 64-wide ones) and queues of four or six rounds (no gain)
// were measured and not kept; a queue of two helps the latter shape (94 us) and
// costs the former 11 %.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "act.cuh"
#include "ptx.cuh"
#include "tpmlp_internal.h"

namespace tpmlp {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxSmem = 227 * 1024;    // dynamic shared memory of a CTA
constexpr int kSmemPerSm = 228 * 1024;  // of an SM, 1 KB of it taken by each CTA

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
    } else if constexpr (V == 2) {
      const uint32_t q = *reinterpret_cast<const uint32_t*>(p);
      v[0] = __uint_as_float(q << 16);
      v[1] = __uint_as_float(q & 0xffff0000u);
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
    } else if constexpr (V == 2) {
      const float2 q = *reinterpret_cast<const float2*>(p);
      v[0] = q.x;
      v[1] = q.y;
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
    } else if constexpr (V == 2) {
      *reinterpret_cast<uint32_t*>(p) = pack2(v[0], v[1]);
    } else {
      *p = __float2bfloat16_rn(v[0]);
    }
  } else {
    if constexpr (V == 4) {
      *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    } else if constexpr (V == 2) {
      *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    } else {
      *p = v[0];
    }
  }
}

constexpr int kStages = 3;  // rounds of a lane's queue: one being worked on, two on their way

// Element-wise operations on V floats, two at a time where V is even.
template <int V>
__device__ __forceinline__ void mul_v(const float (&a)[V], const float (&b)[V], float (&o)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int k = 0; k < V; k += 2)
      act::x2::upk(act::x2::mul2(act::x2::pk(a[k], a[k + 1]), act::x2::pk(b[k], b[k + 1])), o[k], o[k + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = a[k] * b[k];
  }
}
template <int V>
__device__ __forceinline__ void scale_v(const float (&a)[V], float s, float (&o)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int k = 0; k < V; k += 2)
      act::x2::upk(act::x2::mul2(act::x2::pk(a[k], a[k + 1]), act::x2::splat(s)), o[k], o[k + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = a[k] * s;
  }
}
// o = a b + c
template <int V>
__device__ __forceinline__ void fma_v(const float (&a)[V], const float (&b)[V], const float (&c)[V], float (&o)[V]) {
  if constexpr (V % 2 == 0) {
#pragma unroll
    for (int k = 0; k < V; k += 2)
      act::x2::upk(act::x2::fma2(act::x2::pk(a[k], a[k + 1]), act::x2::pk(b[k], b[k + 1]), act::x2::pk(c[k], c[k + 1])),
                   o[k], o[k + 1]);
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = fmaf(a[k], b[k], c[k]);
  }
}
// The sum of a b, two running sums where V is even.
template <int V>
__device__ __forceinline__ float dot_v(const float (&a)[V], const float (&b)[V], const float (&c)[V],
                                       const float (&d)[V]) {
  if constexpr (V % 2 == 0) {
    uint64_t s = 0;
#pragma unroll
    for (int k = 0; k < V; k += 2) {
      s = act::x2::fma2(act::x2::pk(a[k], a[k + 1]), act::x2::pk(b[k], b[k + 1]), s);
      s = act::x2::fma2(act::x2::pk(c[k], c[k + 1]), act::x2::pk(d[k], d[k + 1]), s);
    }
    float s0, s1;
    act::x2::upk(s, s0, s1);
    return s0 + s1;
  } else {
    float s = 0.0f;
#pragma unroll
    for (int k = 0; k < V; ++k) s = fmaf(a[k], b[k], fmaf(c[k], d[k], s));
    return s;
  }
}

// V floats from shared memory.
template <int V>
__device__ __forceinline__ void read_v(const float* p, float (&o)[V]) {
  if constexpr (V % 4 == 0) {
#pragma unroll
    for (int k = 0; k < V; k += 4) {
      const float4 q = *reinterpret_cast<const float4*>(p + k);
      o[k] = q.x;
      o[k + 1] = q.y;
      o[k + 2] = q.z;
      o[k + 3] = q.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) o[k] = p[k];
  }
}

// The partners (a, b) of a unit's V pairs between the registers and its two
// stored vectors v1, v2.  Halves: v1 holds the a's, v2 the b's.  Pairs: the 2V
// elements are a0 b0 a1 b1 ...
template <int V, bool kPairs>
__device__ __forceinline__ void to_partners(const float (&v1)[V], const float (&v2)[V], float (&a)[V], float (&b)[V]) {
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
__device__ __forceinline__ void load_unit(const E* p1, const E* p2, float (&a)[V], float (&b)[V]) {
  float v1[V], v2[V];
  load_vec<E, V>(p1, v1);
  load_vec<E, V>(p2, v2);
  to_partners<V, kPairs>(v1, v2, a, b);
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

// Where unit u of a head lies: two vectors far apart, so that the vectors that
// neighbouring lanes read at once are neighbours too (two next to each other
// made every 32-byte sector travel twice: 127 against 105 us on 8192 tokens
// of 136 heads of 128, neighbouring pairs).  Halves: the units of the rotated part, then those of
// the rest; pairs: the vectors of the head's two halves (whole pairs, V even).
template <int V, bool kPairs>
__device__ __forceinline__ void unit_at(int u, int D, int R, int& o1, int& o2) {
  if (kPairs) {
    o1 = V > 1 ? V * u : 2 * u;
    o2 = V > 1 ? D / 2 + V * u : 2 * u + 1;
    return;
  }
  const int ru = R / (2 * V);
  if (u < ru) {
    o1 = V * u;
    o2 = R / 2 + V * u;
  } else {
    o1 = R + V * (u - ru);
    o2 = R + (D - R) / 2 + V * (u - ru);
  }
}

// A unit's V entries of a per-pair table (an entry per pair; past R / 2 pairs
// that are not rotated, whichever two elements those are).
template <int V, bool kPairs>
__device__ __forceinline__ void read_pairs(const float* table, int u, int D, float (&o)[V]) {
  if constexpr (kPairs && V > 1) {
    float lo[V / 2], hi[V / 2];
    read_v<V / 2>(table + V / 2 * u, lo);
    read_v<V / 2>(table + D / 4 + V / 2 * u, hi);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) {
      o[k] = lo[k];
      o[V / 2 + k] = hi[k];
    }
  } else {
    read_v<V>(table + V * u, o);
  }
}

// The pair in that table of element k of unit u's a's and b's.
template <int V, bool kPairs>
__device__ __forceinline__ int pair_at(int u, int k, int D) {
  if (kPairs && V > 1) return V / 2 * u + (k < V / 2 ? k : D / 4 + k - V / 2);
  return V * u + k;
}

// The sums of s (and t) over the n lanes of a group, to all of them (the same
// bits): a tree to the group's first lane and back for an n that is no power of
// two.  n is the same for the whole warp.
template <bool kTwo>
__device__ __forceinline__ void group_sum(float& s, float& t, int n, int li, int leader) {
  if ((n & (n - 1)) == 0) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o >= n) continue;
      s += __shfl_xor_sync(0xffffffffu, s, o);
      if (kTwo) t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    return;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o >= n) continue;
    const float us = __shfl_down_sync(0xffffffffu, s, o);
    const float ut = kTwo ? __shfl_down_sync(0xffffffffu, t, o) : 0.0f;
    if (li + o < n) {
      s += us;
      t += ut;
    }
  }
  s = __shfl_sync(0xffffffffu, s, leader);
  if (kTwo) t = __shfl_sync(0xffffffffu, t, leader);
}

// B bytes to shared memory, or zeros (src is not read then).
template <int B>
__device__ __forceinline__ void copy_async(uint32_t dst, const void* src, bool ok) {
  const int n = ok ? B : 0;
  if constexpr (B == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(B), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Shared memory of a CTA (bytes from the start of the dynamic part): the
// kind's heads, the frequencies, the gains by unit, each warp's cosines and
// sines, each warp's queue.
// At most kMaxHeads heads of at most kMaxHeadDim elements a kind: a row is
// below 2^22 bytes, a token's offset one 32-bit product.
template <bool kBwd>
struct Head {  // of token 0, and the row strides in bytes
  const char* x;
  char* out;
  uint32_t ldx, ldo;
  uint64_t pad;
};
template <>
struct Head<true> {
  const char* x;
  char* out;
  const char* dy;
  uint32_t ldx, ldo, lddy, pad[3];
};
template <typename P>
__device__ __forceinline__ P row_of(P base, uint32_t tok, uint32_t ld) {
  return base + static_cast<uint64_t>(tok) * ld;
}
template <int V>
constexpr bool kQueue = V > 1;  // single elements are loaded when they are needed
// Units of a lane: heads of up to kMaxHeadDim elements on 32 lanes.
__host__ __device__ constexpr int units_of_lane(int V) { return V >= 4 ? 1 : V == 2 ? 2 : 4; }
// Bytes of a warp's queue.
__host__ __device__ constexpr int queue_bytes(int V, int elem, bool bwd) {
  return V > 1 ? kStages * units_of_lane(V) * (bwd ? 4 : 2) * 32 * V * elem : 0;
}
__host__ __device__ constexpr int round16(int n) { return (n + 15) / 16 * 16; }
struct Place {
  int freq, gain, angle, queue, total;
};
__host__ __device__ inline Place place(int heads, int D, int queue, bool bwd) {
  Place p;
  p.freq = heads * int(bwd ? sizeof(Head<true>) : sizeof(Head<false>));
  p.gain = p.freq + round16(D / 2 * 8);
  p.angle = p.gain + round16(D * 4);
  p.queue = p.angle + kWarps * round16(D * 4);
  p.total = p.queue + kWarps * queue;
  return p;
}

// A position in a warp's sequence of (token, round).
struct Cursor {
  uint32_t tok;
  int h0;
};
__device__ __forceinline__ void cursor_next(Cursor& c, int first, int step, int heads, uint32_t rows) {
  c.h0 += step;
  if (c.h0 >= heads) {
    c.h0 = first;
    c.tok += rows;
  }
}

// What a kernel computes.  Without a norm it is a kernel of its own: as a branch
// of the normed one it took that from 92 to 103 registers, a CTA less an SM.
enum Pass { kNormFwd, kNormBwd, kRotate };

template <typename E, int V, int NU, bool kPairs, Pass kPass>
__device__ __forceinline__ void qk_kind(const QkParams& p, int kind, int w, int nw, uint8_t* smem) {
  constexpr bool kBwd = kPass == kNormBwd, kNorm = kPass != kRotate;
  constexpr int kVecBytes = V * int(sizeof(E));
  constexpr int kQueueBytes = queue_bytes(V, sizeof(E), kBwd);
  constexpr int kUnitVecs = kBwd ? 4 : 2;          // a unit's vectors in the queue
  constexpr int kRoundVecs = NU * kUnitVecs;       // a round's
  static_assert(NU == units_of_lane(V), "units of a lane");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = p.lanes, G = p.groups;  // lanes of a head, heads of a round
  const int grp = lane / n, li = lane - grp * n, leader = grp * n;
  const int units = p.D / (2 * V), heads = p.heads[kind], parts = p.parts[kind];
  const uint32_t T = static_cast<uint32_t>(p.T);
  const Place at = place(max(p.heads[0], p.heads[1]), p.D, kQueueBytes, kBwd);
  Head<kBwd>* head = reinterpret_cast<Head<kBwd>*>(smem);
  uint64_t* freq = reinterpret_cast<uint64_t*>(smem + at.freq);
  float* gains = reinterpret_cast<float*>(smem + at.gain);  // by unit: V a's, V b's
  float* cosines = reinterpret_cast<float*>(smem + at.angle + warp * round16(p.D * 4));
  float* sines = cosines + p.D / 2;

  // The CTA's tables.
  for (int h = threadIdx.x; h < heads; h += kThreads) {
    int s = 0;
    while (h >= p.head_end[kind][s]) ++s;
    const QkShard& S = p.shards[s];
    const int col = S.col[kind] + (h - (s ? p.head_end[kind][s - 1] : 0)) * p.D;
    Head<kBwd> H;
    H.x = reinterpret_cast<const char*>(static_cast<const E*>(S.x) + col);
    H.out = reinterpret_cast<char*>(static_cast<E*>(S.out) + col);
    H.ldx = static_cast<uint32_t>(S.ldx * sizeof(E));
    H.ldo = static_cast<uint32_t>(S.ldo * sizeof(E));
    if constexpr (kBwd) {
      H.dy = reinterpret_cast<const char*>(static_cast<const E*>(S.dy) + col);
      H.lddy = static_cast<uint32_t>(S.lddy * sizeof(E));
    }
    head[h] = H;
  }
  for (int j = threadIdx.x; j < p.R / 2; j += kThreads) freq[j] = p.freq[j];
  const E* g = static_cast<const E*>(p.gain[kind]);
  for (int u = threadIdx.x; u < units; u += kThreads) {
    int o1, o2;
    unit_at<V, kPairs>(u, p.D, p.R, o1, o2);
    float a[V], b[V];
#pragma unroll
    for (int k = 0; k < V; ++k) a[k] = b[k] = 1.0f;
    if (g) load_unit<E, V, kPairs>(g + o1, g + o2, a, b);
#pragma unroll
    for (int k = 0; k < V; ++k) {
      gains[2 * V * u + k] = a[k];
      gains[2 * V * u + V + k] = b[k];
    }
  }
  for (int j = p.R / 2 + lane; j < p.D / 2; j += 32) {  // not rotated
    cosines[j] = 1.0f;
    sines[j] = 0.0f;
  }
  __syncthreads();

  int o1[NU], o2[NU], un[NU];
  bool on[NU];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    const int u = li + i * n;
    on[i] = grp < G && u < units;
    un[i] = on[i] ? u : 0;
    unit_at<V, kPairs>(un[i], p.D, p.R, o1[i], o2[i]);
  }
  float dga[NU][V], dgb[NU][V];
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int k = 0; k < V; ++k) dga[i][k] = dgb[i][k] = 0.0f;

  const uint32_t rows = nw / parts;  // tokens at a time; warps left over have none
  const int first = (w % parts) * G, step = parts * G;
  Cursor get, run;  // what is fetched next, what is worked on next
  run.tok = static_cast<uint32_t>(w) < rows * parts && first < heads ? w / parts : T;
  run.h0 = first;
  get = run;

  // The queue: slot s holds, per vector and lane, this lane's bytes of a round.
  const uint32_t queue = ptx::smem_u32(smem + at.queue + warp * kQueueBytes) + lane * kVecBytes;
  auto fetch = [&](int slot) {
    if constexpr (kQueue<V>) {
      if (get.tok < T) {
        const int h = get.h0 + grp;
        const Head<kBwd>& H = head[h < heads && grp < G ? h : 0];
        const E* x = reinterpret_cast<const E*>(row_of(H.x, get.tok, H.ldx));
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          if (i > 0 && i * n >= units) break;  // no lane has a unit there
          const bool ok = on[i] && h < heads;  // else zeros, which add nothing to any sum
          const uint32_t q = queue + (slot * kRoundVecs + i * kUnitVecs) * 32 * kVecBytes;
          copy_async<kVecBytes>(q, x + o1[i], ok);
          copy_async<kVecBytes>(q + 32 * kVecBytes, x + o2[i], ok);
          if constexpr (kBwd) {
            const E* y = reinterpret_cast<const E*>(row_of(H.dy, get.tok, H.lddy));
            copy_async<kVecBytes>(q + 64 * kVecBytes, y + o1[i], ok);
            copy_async<kVecBytes>(q + 96 * kVecBytes, y + o2[i], ok);
          }
        }
        cursor_next(get, first, step, heads, rows);
      }
      copy_commit();  // one group a round, an empty one past the end
    }
  };
  if constexpr (kQueue<V>) {
#pragma unroll
    for (int s = 0; s < kStages - 1; ++s) fetch(s);
  }
  int slot = 0;
  // The position of the next token is fetched a token ahead.
  auto position = [&](uint32_t tok) {
    return tok < T && p.pos ? static_cast<uint64_t>(p.pos[tok]) : static_cast<uint64_t>(tok);
  };
  uint64_t pos = position(run.tok);

  // Forward: the coefficients of a and b in a' and b'; else the cosines and
  // sines (c3, c4) and, backward, the gains.
  float c1[NU][V], c2[NU][V], c3[NU][V], c4[NU][V];
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    read_v<V>(gains + 2 * V * un[i], c1[i]);
    read_v<V>(gains + 2 * V * un[i] + V, c2[i]);
#pragma unroll
    for (int k = 0; k < V; ++k) c3[i][k] = c4[i][k] = 0.0f;
  }

  // Vector 0 of a round's unit i in the queue.
  auto queued = [&](int slot, int i) {
    return reinterpret_cast<const E*>(smem + at.queue + warp * kQueueBytes +
                                      (slot * kRoundVecs + i * kUnitVecs) * 32 * kVecBytes + lane * kVecBytes);
  };

  // Past R the partner's part is nothing, not 0 times the partner, which is a NaN if that is infinite.  (With a norm an
  // infinity spoils the whole head.)
  auto drop_unrotated = [&](int i, float (&t)[V]) {
    if (p.R == p.D) return;
#pragma unroll
    for (int k = 0; k < V; ++k)
      if (pair_at<V, kPairs>(un[i], k, p.D) >= p.R / 2) t[k] = 0.0f;
  };

  auto forward_head = [&](const Cursor& run, int slot) {
    const int h = run.h0 + grp;
    const bool ok = grp < G && h < heads;
    const Head<kBwd>& H = head[ok ? h : 0];
    float a[NU][V], b[NU][V], ss = 0.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
#pragma unroll
      for (int k = 0; k < V; ++k) a[i][k] = b[i][k] = 0.0f;
      if constexpr (kQueue<V>) {
        if (i == 0 || i * n < units) {
          const E* q = queued(slot, i);
          load_unit<E, V, kPairs>(q, q + 32 * V, a[i], b[i]);
        }
      } else {
        if (ok && on[i]) {
          const E* x = reinterpret_cast<const E*>(row_of(H.x, run.tok, H.ldx));
          load_unit<E, V, kPairs>(x + o1[i], x + o2[i], a[i], b[i]);
        }
      }
      if constexpr (kNorm) ss += dot_v<V>(a[i], a[i], b[i], b[i]);
    }
    float r = 1.0f, none = 0.0f;
    if constexpr (kNorm) {
      group_sum<false>(ss, none, n, li, leader);
      r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
    }
    E* out = reinterpret_cast<E*>(row_of(H.out, run.tok, H.ldo));
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float oa[V], ob[V], t[V];
      if constexpr (kNorm) {
        mul_v<V>(b[i], c2[i], t);
        fma_v<V>(a[i], c1[i], t, oa);
        mul_v<V>(a[i], c4[i], t);
        fma_v<V>(b[i], c3[i], t, ob);
        scale_v<V>(oa, r, oa);
        scale_v<V>(ob, r, ob);
      } else {
        mul_v<V>(b[i], c4[i], t);
        scale_v<V>(t, -1.0f, t);
        drop_unrotated(i, t);
        fma_v<V>(a[i], c3[i], t, oa);
        mul_v<V>(a[i], c4[i], t);
        drop_unrotated(i, t);
        fma_v<V>(b[i], c3[i], t, ob);
      }
      if (ok && on[i]) store_unit<E, V, kPairs>(out, o1[i], o2[i], oa, ob);
    }
  };

  auto backward_head = [&](const Cursor& run, int slot) {
    const int h = run.h0 + grp;
    const bool ok = grp < G && h < heads;
    const Head<kBwd>& H = head[ok ? h : 0];
    float a[NU][V], b[NU][V], wa[NU][V], wb[NU][V];
    float ss = 0.0f, sx = 0.0f;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float ya[V], yb[V], sa[V], sb[V], t[V];
#pragma unroll
      for (int k = 0; k < V; ++k) a[i][k] = b[i][k] = ya[k] = yb[k] = 0.0f;
      if constexpr (kQueue<V>) {
        if (i == 0 || i * n < units) {
          const E* q = queued(slot, i);
          load_unit<E, V, kPairs>(q, q + 32 * V, a[i], b[i]);
          load_unit<E, V, kPairs>(q + 64 * V, q + 96 * V, ya, yb);
        }
      } else {
        if constexpr (kBwd) {
          if (ok && on[i]) {
            const E* x = reinterpret_cast<const E*>(row_of(H.x, run.tok, H.ldx));
            load_unit<E, V, kPairs>(x + o1[i], x + o2[i], a[i], b[i]);
            const E* y = reinterpret_cast<const E*>(row_of(H.dy, run.tok, H.lddy));
            load_unit<E, V, kPairs>(y + o1[i], y + o2[i], ya, yb);
          }
        }
      }
      ss += dot_v<V>(a[i], a[i], b[i], b[i]);
      // w = dy rotated back; the sum of w g x
      mul_v<V>(yb, c4[i], t);
      fma_v<V>(ya, c3[i], t, wa[i]);
      scale_v<V>(ya, -1.0f, t);
      mul_v<V>(t, c4[i], t);
      fma_v<V>(yb, c3[i], t, wb[i]);
      mul_v<V>(wa[i], c1[i], sa);
      mul_v<V>(wb[i], c2[i], sb);
      sx += dot_v<V>(sa, a[i], sb, b[i]);
    }
    group_sum<true>(ss, sx, n, li, leader);
    const float r = rsqrtf(fmaf(ss, p.inv_d, p.eps));
    const float m = -(r * (sx * p.inv_d));  // - mean(s n)
    E* out = reinterpret_cast<E*>(row_of(H.out, run.tok, H.ldo));
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      float oa[V], ob[V], sa[V], sb[V], mm[V];
      scale_v<V>(a[i], r, a[i]);  // n = x r
      scale_v<V>(b[i], r, b[i]);
      fma_v<V>(wa[i], a[i], dga[i], dga[i]);
      fma_v<V>(wb[i], b[i], dgb[i], dgb[i]);
      mul_v<V>(wa[i], c1[i], sa);
      mul_v<V>(wb[i], c2[i], sb);
#pragma unroll
      for (int k = 0; k < V; ++k) mm[k] = m;
      fma_v<V>(a[i], mm, sa, oa);
      fma_v<V>(b[i], mm, sb, ob);
      scale_v<V>(oa, r, oa);
      scale_v<V>(ob, r, ob);
      if (ok && on[i]) store_unit<E, V, kPairs>(out, o1[i], o2[i], oa, ob);
    }
  };

  while (run.tok < T) {
    if (run.h0 == first) {  // a new token
      for (int j = lane; j < p.R / 2; j += 32) {
        const int32_t turn = static_cast<int32_t>((pos * freq[j]) >> 32);  // in 2^-32 turns
        float c, s;
        sincospif(static_cast<float>(turn) * 0x1p-31f, &s, &c);
        cosines[j] = c;
        sines[j] = kNorm ? s : s * p.turn;
      }
      pos = position(run.tok + rows);
      __syncwarp();
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (kPass != kNormFwd) {
          read_pairs<V, kPairs>(cosines, un[i], p.D, c3[i]);
          read_pairs<V, kPairs>(sines, un[i], p.D, c4[i]);
        } else {
          float cs[V], sn[V], ga[V], gb[V];
          read_pairs<V, kPairs>(cosines, un[i], p.D, cs);
          read_pairs<V, kPairs>(sines, un[i], p.D, sn);
          read_v<V>(gains + 2 * V * un[i], ga);
          read_v<V>(gains + 2 * V * un[i] + V, gb);
          mul_v<V>(ga, cs, c1[i]);
          mul_v<V>(gb, sn, c2[i]);
          scale_v<V>(c2[i], -1.0f, c2[i]);
          mul_v<V>(gb, cs, c3[i]);
          mul_v<V>(ga, sn, c4[i]);
        }
      }
      __syncwarp();  // read before the next token's are written
    }
    fetch((slot + kStages - 1) % kStages);
    copy_wait<kQueue<V> ? kStages - 1 : 0>();

    if constexpr (kBwd) backward_head(run, slot);
    else forward_head(run, slot);
    slot = (slot + 1) % kStages;
    cursor_next(run, first, step, heads, rows);
  }
  copy_wait<0>();
  if (!kBwd || !p.partial) return;

  // This CTA's sum of the gain's gradient: over the groups of a warp, then the
  // warps, in a fixed order (the tables' memory is reused).
  __syncthreads();
  float* sums = reinterpret_cast<float*>(smem);  // [warp][group][D]
#pragma unroll
  for (int i = 0; i < NU; ++i) {
    if (!on[i]) continue;
#pragma unroll
    for (int k = 0; k < V; ++k) {
      int ea = o1[i] + k, eb = o2[i] + k;
      if (kPairs && V > 1) {
        ea = 2 * k < V ? o1[i] + 2 * k : o2[i] + 2 * k - V;
        eb = ea + 1;
      }
      sums[(warp * G + grp) * p.D + ea] = dga[i][k];
      sums[(warp * G + grp) * p.D + eb] = dgb[i][k];
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.D; e += kThreads) {
    float s = 0.0f;
    for (int i = 0; i < kWarps * G; ++i) s += sums[i * p.D + e];
    p.partial[static_cast<int64_t>(blockIdx.x) * p.D + e] = s;
  }
}

// dV into the value columns of dQKV: 16 bytes a lane and step, kFlight steps
// (of one token after another) in flight.
template <typename E>
__device__ __forceinline__ void copy_values(const QkParams& p, int w, int nw) {
  constexpr int V = 16 / sizeof(E);
  constexpr int kFlight = 8;
  const int chunks = static_cast<int>(p.values / V);  // of a token, over all shards
  int64_t tok = w;
  int c = threadIdx.x & 31;       // this lane's chunk of the token,
  int s = 0, c0 = 0;              // its shard, and that shard's first chunk
  while (c >= chunks && tok < p.T) {
    c -= chunks;
    tok += nw;
  }
  while (tok < p.T) {
    uint4 q[kFlight];
    uint4* dst[kFlight];
#pragma unroll
    for (int u = 0; u < kFlight; ++u) {
      dst[u] = nullptr;
      if (tok >= p.T) continue;
      while (c - c0 >= p.shards[s].dkv / V) c0 += p.shards[s++].dkv / V;
      const QkShard& S = p.shards[s];
      q[u] = reinterpret_cast<const uint4*>(static_cast<const E*>(S.dv) + tok * S.dkv)[c - c0];
      dst[u] = reinterpret_cast<uint4*>(static_cast<E*>(S.out) + tok * S.ldo + S.vcol) + (c - c0);
      c += 32;
      while (c >= chunks && tok < p.T) {
        c -= chunks;
        tok += nw;
        s = c0 = 0;
      }
    }
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      if (dst[u]) *dst[u] = q[u];
  }
}

template <typename E, int V, int NU, bool kPairs, Pass kPass>
__device__ __forceinline__ void qk_body(const QkParams& p) {
  extern __shared__ __align__(16) uint8_t qk_smem[];
  const int cta = blockIdx.x, warp = threadIdx.x >> 5;
  if (kPass != kNormFwd && p.values) copy_values<E>(p, cta * kWarps + warp, gridDim.x * kWarps);
  const int kind = cta < p.cta_end[0] ? 0 : 1;
  const int c0 = kind ? p.cta_end[0] : 0;
  qk_kind<E, V, NU, kPairs, kPass>(p, kind, (cta - c0) * kWarps + warp, (p.cta_end[kind] - c0) * kWarps, qk_smem);
}

template <typename E, int V, int NU, bool kPairs>
__global__ void __launch_bounds__(kThreads, 4) tpmlp_attn_qk_norm_rope_fwd(const __grid_constant__ QkParams p) {
  qk_body<E, V, NU, kPairs, kNormFwd>(p);
}

template <typename E, int V, int NU, bool kPairs>
__global__ void __launch_bounds__(kThreads, 4) tpmlp_attn_qk_rope(const __grid_constant__ QkParams p) {
  qk_body<E, V, NU, kPairs, kRotate>(p);
}

template <typename E, int V, int NU, bool kPairs>
__global__ void __launch_bounds__(kThreads, 4) tpmlp_attn_qk_norm_rope_bwd(const __grid_constant__ QkParams p) {
  qk_body<E, V, NU, kPairs, kNormBwd>(p);
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

template <typename E, int V>
QkKernel pick(bool pairs, Pass pass) {
  constexpr int NU = units_of_lane(V);
  if (pass == kRotate) return pairs ? tpmlp_attn_qk_rope<E, V, NU, true> : tpmlp_attn_qk_rope<E, V, NU, false>;
  if (pass == kNormBwd)
    return pairs ? tpmlp_attn_qk_norm_rope_bwd<E, V, NU, true> : tpmlp_attn_qk_norm_rope_bwd<E, V, NU, false>;
  return pairs ? tpmlp_attn_qk_norm_rope_fwd<E, V, NU, true> : tpmlp_attn_qk_norm_rope_fwd<E, V, NU, false>;
}

// The widest vector (in elements) that every part of a head is a whole number
// of, up to 16 bytes.  8192 tokens of 32 + 8 heads of 80, bf16, on GB300: 24 us
// in 8-element vectors (all 80 rotated), 26 us in 4 (40), and, before 2 was
// added, 134 us in single elements (20; 71 us with 2).
int vector_width(bool bf16, int D, int R, bool pairs) {
  for (int V = bf16 ? 8 : 4; V >= 2; V /= 2)
    if (D % (2 * V) == 0 && (pairs || R % (2 * V) == 0)) return V;
  return 1;
}

QkKernel kernel_for(bool bf16, int V, bool pairs, Pass pass) {
  if (bf16) {
    if (V == 8) return pick<__nv_bfloat16, 8>(pairs, pass);
    if (V == 4) return pick<__nv_bfloat16, 4>(pairs, pass);
    if (V == 2) return pick<__nv_bfloat16, 2>(pairs, pass);
    return pick<__nv_bfloat16, 1>(pairs, pass);
  }
  if (V == 4) return pick<float, 4>(pairs, pass);
  if (V == 2) return pick<float, 2>(pairs, pass);
  return pick<float, 1>(pairs, pass);
}

}  // namespace

// A token's angles, in rounds of heads, for the deal of the CTAs to the kinds: 2
// and 3 were measured equal to 8 % slower (8 shards of 16 + 1 heads).
constexpr double kAngleWork = 1.0;

// Lays the launch out (lanes, parts, CTAs of each kind) and launches it.
cudaError_t launch_qk_norm_rope(QkParams& p, bool bf16, bool pairs, bool bwd, int sms, cudaStream_t stream) {
  if (p.T <= 0) return cudaSuccess;
  const int V = vector_width(bf16, p.D, p.R, pairs);
  const int units = p.D / (2 * V);
  p.lanes = std::min(units, 32);
  p.groups = 32 / p.lanes;
  const int G = p.groups;
  const Pass pass = !p.norm ? kRotate : bwd ? kNormBwd : kNormFwd;
  const bool sums = pass == kNormBwd;  // of the gain's gradient
  const QkKernel k = kernel_for(bf16, V, pairs, pass);
  int bytes = place(std::max(p.heads[0], p.heads[1]), p.D, queue_bytes(V, bf16 ? 2 : 4, sums), sums).total;
  if (sums) bytes = std::max(bytes, kWarps * G * p.D * 4);
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
  if (e != cudaSuccess) return e;
  // CTAs that an SM holds: by registers (asked once per kernel) and by shared memory.
  static std::atomic<int> by_registers[2][9][2][3];
  std::atomic<int>& known = by_registers[bf16][V][pairs][pass];
  int per_sm = known.load(std::memory_order_relaxed);
  if (per_sm == 0) {
    e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, k, kThreads, 0);
    if (e != cudaSuccess) return e;
    if (per_sm < 1) return cudaErrorInvalidConfiguration;
    known.store(per_sm, std::memory_order_relaxed);
  }
  per_sm = std::max(1, std::min(per_sm, kSmemPerSm / (bytes + 1024)));
  const int slots = sms * per_sm;
  const int64_t most_warps = int64_t{slots} * kWarps;

  // Heads of a token in parts, so that a launch of few tokens still has a
  // warp for every slot: a part is a whole number of rounds of G heads.
  int rounds[2];
  for (int kind = 0; kind < 2; ++kind) rounds[kind] = (p.heads[kind] + G - 1) / G;
  auto parts_of = [&](int kind, int per_part) { return (rounds[kind] + per_part - 1) / per_part; };
  int per_part = std::max(rounds[0], rounds[1]);
  while (per_part > 1 && p.T * (parts_of(0, per_part) + parts_of(1, per_part)) < most_warps) per_part = (per_part + 1) / 2;
  // CTAs of each kind in proportion to its work, in rounds: a token's angles
  // count as one more.  (Every CTA copies an equal share of dV first.)
  double work[2];
  int64_t want[2];
  for (int kind = 0; kind < 2; ++kind) {
    p.parts[kind] = parts_of(kind, per_part);
    work[kind] = rounds[kind] + kAngleWork * p.parts[kind];
    want[kind] = (p.T * p.parts[kind] + kWarps - 1) / kWarps;
  }
  int end = 0;
  for (int kind = 0; kind < 2; ++kind) {
    int64_t c = static_cast<int64_t>(work[kind] / (work[0] + work[1]) * slots + 0.5);
    c = std::min(c, want[kind]);
    c = std::max<int64_t>(c, (p.parts[kind] + kWarps - 1) / kWarps);  // a warp for every part
    end += static_cast<int>(c);
    p.cta_end[kind] = end;
  }
  if (end > kQkMaxCtas) return cudaErrorInvalidConfiguration;  // parts < 2 x the slots' warps: not reached
  k<<<end, kThreads, bytes, stream>>>(p);
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
