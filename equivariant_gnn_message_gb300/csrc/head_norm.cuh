// Norms of queries and keys for each head, with the rotation by a node's
// position in the same pass (sm_103a).
//
//   r = (mean_d x^2 + eps)^-1/2,  u = x r w          over the D values of a head
//   theta[p] = sum_a pos[a] freq[p][a]               p: the pair (2p, 2p+1)
//   y[2p] = u[2p] cos - u[2p+1] sin,  y[2p+1] = u[2p] sin + u[2p+1] cos
// Backward, with g = dL/dy turned back by -theta (b):
//   a = b w,  dx = r (a - x r mean_d(a x r)),  dw = sum b x r
//   dpos[a] = sum_{heads, p} freq[p][a] (b[2p+1] u[2p] - b[2p] u[2p+1])
// (a rotation turns g and y alike, so the last one needs no y).
//
// A warp takes a few nodes: the cosines and sines of their pairs are formed once,
// by all lanes, and kept in shared memory for all heads.  Memory binds: x is read
// once and y written once.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace eqmp {

struct HeadNormArgs {
  const void *q, *k;          // [N][Hq][D], [N][Hk][D]
  const void *gq, *gk;        // backward: dL/d of the outputs
  long long q_ld, k_ld, gq_ld, gk_ld;
  const float *wq, *wk;       // [D] or NULL
  const float *pos, *freq;    // [N][axes], [D/2][axes] or NULL
  void *oq, *ok;              // forward: the outputs; backward: the gradients of q and k
  float* rstd;                // [N][Hq+Hk]
  float *gwq, *gwk, *gpos;
  float* part;                // [parts][2][D]
  float eps;
  int N, Hq, Hk, D, axes;
  int each;  // nodes of a warp at a time
};

constexpr int kHeadWarps = 8;       // of a CTA
constexpr int kHeadAngles = 64;     // pairs of a warp's nodes at a time, or those of one node (at most 128)

// An angle in turns, reduced to half a turn: the frequency in turns is held as
// the sum of two floats, and the product's rounding error is kept, so that a
// position of 10^5 turns has its angle to 10^-7 of a turn.  (In one float the
// product alone would be off by 10^-2.)
struct Turns {
  float hi, lo;
  __device__ __forceinline__ void set(float freq) {
    const double t = (double)freq * 0.15915494309189535;  // 1 / (2 pi)
    hi = (float)t;
    lo = (float)(t - hi);
  }
  __device__ __forceinline__ float of(float pos) const {
    const float t = pos * hi, rest = fmaf(pos, lo, fmaf(pos, hi, -t));
    return t - rintf(t) + rest;
  }
};

// The share of a head's row that a lane holds: NV vectors of V elements, the
// j-th at (j G + l) V.  V = 2: single loads, the last pair may be half.
template <typename T, int V, int G, int NV>
struct HeadShare {
  static constexpr bool WIDE = V * sizeof(T) == 16;
  uint4 raw[WIDE ? NV : 1];
  T one[WIDE ? 1 : NV * V];
  __device__ __forceinline__ void load(const T* row, int l, int D, bool ok) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * G + l) * V;
      if constexpr (WIDE) {
        raw[j] = ok && c < D ? *reinterpret_cast<const uint4*>(row + c) : make_uint4(0u, 0u, 0u, 0u);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i) one[j * V + i] = ok && c + i < D ? row[c + i] : T(0.0f);
      }
    }
  }
  __device__ __forceinline__ void get(float (&f)[NV * V]) const {
    if constexpr (WIDE) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t w[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (V == 4) {
            f[j * V + i] = __uint_as_float(w[i]);
          } else {
            f[j * V + 2 * i] = __uint_as_float(w[i] << 16);
            f[j * V + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV * V; ++i) f[i] = (float)one[i];
    }
  }
  static __device__ __forceinline__ void store(T* row, int l, int D, const float (&f)[NV * V]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = (j * G + l) * V;
      if (c >= D) break;
      if constexpr (V == 4) {
        *reinterpret_cast<float4*>(row + c) = make_float4(f[j * V], f[j * V + 1], f[j * V + 2], f[j * V + 3]);
      } else if constexpr (V == 8) {
        __nv_bfloat162 b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) b[i] = __floats2bfloat162_rn(f[j * V + 2 * i], f[j * V + 2 * i + 1]);
        *reinterpret_cast<uint4*>(row + c) = *reinterpret_cast<const uint4*>(b);
      } else {
#pragma unroll
        for (int i = 0; i < V; ++i)
          if (c + i < D) row[c + i] = T(f[j * V + i]);
      }
    }
  }
};

// The lane's weights of queries and keys; 1 where there are none.
template <int V, int G, int NV>
__device__ __forceinline__ void load_weights(const float* w, int l, int D, float (&f)[NV * V]) {
#pragma unroll
  for (int i = 0; i < NV * V; ++i) {
    const int c = (i / V * G + l) * V + i % V;
    f[i] = w && c < D ? w[c] : 1.0f;
  }
}

// The angles of a warp's nodes.  freq: the pairs' frequencies in turns, [pair][axis]
// (shared by the CTA); turn: the cosines and sines of the warp's nodes,
// [node][pair].

__device__ __forceinline__ void load_freq(const HeadNormArgs& a, Turns* freq) {
  for (int i = threadIdx.x; i < a.D / 2 * a.axes; i += blockDim.x) freq[i].set(a.freq[i]);
}

__device__ __forceinline__ void form_turns(const HeadNormArgs& a, const Turns* freq, float2* turn, int node0, int nodes) {
  const int pairs = a.D / 2;
  __syncwarp();  // the last nodes' have been read
  for (int i = threadIdx.x & 31; i < nodes * pairs; i += 32) {
    const int n = i / pairs, p = i - n * pairs;
    const float* pos = a.pos + (long long)(node0 + n) * a.axes;
    float t = freq[p * a.axes].of(__ldg(pos));
    for (int x = 1; x < a.axes; ++x) t += freq[p * a.axes + x].of(__ldg(pos + x));
    t -= rintf(t);
    float s, c;
    sincospif(2.0f * t, &s, &c);
    turn[i] = make_float2(c, s);
  }
  __syncwarp();
}

// The lane's pairs of a node.
template <int V, int G, int NV>
__device__ __forceinline__ void load_turns(const float2* turn, int pairs, int l, float2 (&t)[NV * V / 2]) {
#pragma unroll
  for (int p = 0; p < NV * V / 2; ++p) {
    const int pair = ((2 * p / V * G + l) * V + 2 * p % V) / 2;
    t[p] = pair < pairs ? turn[pair] : make_float2(1.0f, 0.0f);
  }
}

// A warp's way through its nodes and their heads, U * 32 / G heads at a time.
struct HeadWalk {
  long long node, node0, step;  // the node, the first of its batch of `each`, from batch to batch
  int each, t0, heads, stride;
  __device__ __forceinline__ HeadWalk(const HeadNormArgs& a, int each, int stride)
      : node0(((long long)blockIdx.x * kHeadWarps + (threadIdx.x >> 5)) * each), step((long long)gridDim.x * kHeadWarps * each), each(each),
        t0(0), heads(a.Hq + a.Hk), stride(stride) {
    node = node0;
  }
  __device__ __forceinline__ void next(int N) {
    t0 += stride;
    if (t0 < heads) return;
    t0 = 0;
    ++node;
    if (node - node0 < each && node < N) return;
    node0 += step;
    node = node0;
  }
};

// A step's rows are loaded before its angles are formed, and the first ones before
// anything else.  (Loading a step ahead costs the registers of two steps: 100,000
// nodes, 8 + 8 heads of 32, bf16 68 us for 59, backward fp32 160 for 138.)
template <typename T, int V, int G, int NV, int U>
__global__ void __launch_bounds__(32 * kHeadWarps) k_head_norm(const __grid_constant__ HeadNormArgs a) {
  constexpr int W = NV * V, P = W / 2, AT_ONCE = 32 / G;
  __shared__ Turns freq[128 * 3];
  __shared__ float2 turns[kHeadWarps][128];
  const int lane = threadIdx.x & 31, l = lane % G, heads = a.Hq + a.Hk, pairs = a.D / 2;
  const int each = a.each;
  float2* const turn = turns[threadIdx.x >> 5];
  HeadWalk at(a, each, U * AT_ONCE);
  HeadShare<T, V, G, NV> x[U];
  auto load = [&] {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = at.t0 + lane / G + u * AT_ONCE;
      const bool ok = at.node < a.N && t < heads;
      const long long node = ok ? at.node : 0;
      x[u].load(t < a.Hq ? static_cast<const T*>(a.q) + node * a.q_ld + (long long)t * a.D
                         : static_cast<const T*>(a.k) + node * a.k_ld + (long long)(t - a.Hq) * a.D, l, a.D, ok);
    }
  };
  load();
  bool first = true;
  float wq[W], wk[W];
  load_weights<V, G, NV>(a.wq, l, a.D, wq);
  load_weights<V, G, NV>(a.wk, l, a.D, wk);
  if (a.axes) load_freq(a, freq);
  __syncthreads();
  float2 cs[P];
  for (; at.node < a.N; at.next(a.N)) {
    if (!first) load();
    first = false;
    if (a.axes && at.t0 == 0) {
      if (at.node == at.node0) form_turns(a, freq, turn, (int)at.node0, (int)(a.N - at.node0 < each ? a.N - at.node0 : each));
      load_turns<V, G, NV>(turn + (int)(at.node - at.node0) * pairs, pairs, l, cs);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = at.t0 + lane / G + u * AT_ONCE;
      float f[W], ss = 0.0f;
      x[u].get(f);
#pragma unroll
      for (int i = 0; i < W; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (t >= heads) continue;
      const bool query = t < a.Hq;
      const float r = 1.0f / sqrtf(ss / (float)a.D + a.eps);
      if (a.rstd && l == 0) a.rstd[at.node * heads + t] = r;
#pragma unroll
      for (int i = 0; i < W; ++i) f[i] *= r * (query ? wq[i] : wk[i]);
      if (a.axes)
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const float u0 = f[2 * p], u1 = f[2 * p + 1];
          f[2 * p] = u0 * cs[p].x - u1 * cs[p].y;
          f[2 * p + 1] = u0 * cs[p].y + u1 * cs[p].x;
        }
      T* out = static_cast<T*>(query ? a.oq : a.ok);
      const long long row = query ? at.node * a.Hq + t : at.node * a.Hk + (t - a.Hq);
      if (out) HeadShare<T, V, G, NV>::store(out + row * a.D, l, a.D, f);
    }
  }
}

template <typename T, int V, int G, int NV, int U>
__global__ void __launch_bounds__(32 * kHeadWarps) k_head_norm_bwd(const __grid_constant__ HeadNormArgs a) {
  constexpr int W = NV * V, P = W / 2, AT_ONCE = 32 / G;
  __shared__ Turns freq[128 * 3];
  __shared__ float2 turns[kHeadWarps][128];
  __shared__ float red[kHeadWarps][2 * G * W];
  const int lane = threadIdx.x & 31, l = lane % G, warp = threadIdx.x >> 5, heads = a.Hq + a.Hk, pairs = a.D / 2;
  const int each = a.each;
  float2* const turn = turns[warp];
  HeadWalk at(a, each, U * AT_ONCE);
  HeadShare<T, V, G, NV> x[U], g[U];
  float r[U];
  auto load = [&] {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = at.t0 + lane / G + u * AT_ONCE, hk = t - a.Hq;
      const bool query = t < a.Hq, ok = at.node < a.N && t < heads;
      const long long node = ok ? at.node : 0;
      x[u].load(static_cast<const T*>(query ? a.q : a.k) + (query ? node * a.q_ld + (long long)t * a.D : node * a.k_ld + (long long)hk * a.D),
                l, a.D, ok);
      g[u].load(static_cast<const T*>(query ? a.gq : a.gk) + (query ? node * a.gq_ld + (long long)t * a.D : node * a.gk_ld + (long long)hk * a.D),
                l, a.D, ok);
      r[u] = ok ? __ldg(a.rstd + node * heads + t) : 0.0f;
    }
  };
  load();
  bool first = true;
  float wq[W], wk[W], dwq[W], dwk[W];
  load_weights<V, G, NV>(a.wq, l, a.D, wq);
  load_weights<V, G, NV>(a.wk, l, a.D, wk);
#pragma unroll
  for (int i = 0; i < W; ++i) dwq[i] = dwk[i] = 0.0f;
  if (a.axes) load_freq(a, freq);
  __syncthreads();
  float2 cs[P];
  float turned[P];
  for (; at.node < a.N; at.next(a.N)) {
    if (!first) load();
    first = false;
    if (a.axes && at.t0 == 0) {
      if (at.node == at.node0) form_turns(a, freq, turn, (int)at.node0, (int)(a.N - at.node0 < each ? a.N - at.node0 : each));
      load_turns<V, G, NV>(turn + (int)(at.node - at.node0) * pairs, pairs, l, cs);
#pragma unroll
      for (int p = 0; p < P; ++p) turned[p] = 0.0f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int t = at.t0 + lane / G + u * AT_ONCE;
      const bool query = t < a.Hq, ok = t < heads;
      float h[W], b[W], mean = 0.0f;
      x[u].get(h);
      g[u].get(b);
#pragma unroll
      for (int i = 0; i < W; ++i) h[i] *= r[u];
      if (a.axes)
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const float g0 = b[2 * p], g1 = b[2 * p + 1];
          b[2 * p] = g0 * cs[p].x + g1 * cs[p].y;
          b[2 * p + 1] = g1 * cs[p].x - g0 * cs[p].y;
          const float u0 = h[2 * p] * (query ? wq[2 * p] : wk[2 * p]);
          const float u1 = h[2 * p + 1] * (query ? wq[2 * p + 1] : wk[2 * p + 1]);
          if (ok) turned[p] += b[2 * p + 1] * u0 - b[2 * p] * u1;
        }
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const float d = b[i] * h[i];
        if (ok && query) dwq[i] += d;
        if (ok && !query) dwk[i] += d;
        b[i] *= query ? wq[i] : wk[i];
        mean = fmaf(b[i], h[i], mean);
      }
#pragma unroll
      for (int o = G / 2; o > 0; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
      if (!ok) continue;
      mean /= (float)a.D;
#pragma unroll
      for (int i = 0; i < W; ++i) b[i] = r[u] * fmaf(-h[i], mean, b[i]);
      T* out = static_cast<T*>(query ? a.oq : a.ok);
      const long long row = query ? at.node * a.Hq + t : at.node * a.Hk + (t - a.Hq);
      if (out) HeadShare<T, V, G, NV>::store(out + row * a.D, l, a.D, b);
    }
    if (a.gpos && at.t0 + at.stride >= heads) {
      float d[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int pair = ((2 * p / V * G + l) * V + 2 * p % V) / 2;
#pragma unroll
        for (int x = 0; x < 3; ++x)
          if (pair < pairs && x < a.axes) d[x] = fmaf(turned[p], freq[pair * a.axes + x].hi, d[x]);
      }
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        if (x >= a.axes) break;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d[x] += __shfl_xor_sync(0xffffffffu, d[x], o);
        if (lane == 0) a.gpos[at.node * a.axes + x] = d[x] * 6.2831853071795865f;
      }
    }
  }
  if (!a.part) return;
  // over the groups of a warp, then over the warps, in a fixed order
#pragma unroll
  for (int i = 0; i < W; ++i) {
#pragma unroll
    for (int o = G; o < 32; o <<= 1) {
      dwq[i] += __shfl_xor_sync(0xffffffffu, dwq[i], o);
      dwk[i] += __shfl_xor_sync(0xffffffffu, dwk[i], o);
    }
    if (lane < G) {
      const int c = (i / V * G + l) * V + i % V;
      red[warp][c] = dwq[i];
      red[warp][G * W + c] = dwk[i];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * a.D; i += blockDim.x) {
    const int c = i < a.D ? i : G * W + i - a.D;
    float t = red[0][c];
#pragma unroll
    for (int w = 1; w < kHeadWarps; ++w) t += red[w][c];
    a.part[(long long)blockIdx.x * 2 * a.D + i] = t;
  }
}

// dw: the sums of the CTAs' parts, 8 columns a block.
constexpr int kHeadSumX = 8, kHeadSumY = 32;

static __global__ void __launch_bounds__(kHeadSumX * kHeadSumY) k_head_norm_sum(HeadNormArgs a, int parts) {
  __shared__ float red[kHeadSumY][kHeadSumX];
  const int c = blockIdx.x * kHeadSumX + threadIdx.x;
  float t = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // until the kernel that writes the parts is done
  if (c < 2 * a.D) {
#pragma unroll 8
    for (int p = threadIdx.y; p < parts; p += kHeadSumY) t += a.part[(long long)p * 2 * a.D + c];
  }
  red[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y || c >= 2 * a.D) return;
#pragma unroll
  for (int y = 1; y < kHeadSumY; ++y) t += red[y][threadIdx.x];
  if (c < a.D) {
    if (a.gwq) a.gwq[c] = t;
  } else if (a.gwk) {
    a.gwk[c - a.D] = t;
  }
}

}  // namespace eqmp
