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
// by all lanes, and kept in shared memory for all heads.  x is read once and y
// written once: 100,000 nodes of 16 heads of 32 with three axes, fp32 74 us forward
// (83 % of the copy rate) and 115 backward (80 %), bf16 49 and 111, bound by
// instructions (420 a node forward, 74 % issue).
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
  int each;   // nodes of a warp at a time
  int shift;  // see form_turns
};

constexpr int kHeadWarps = 8;       // of a CTA

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

// 2^shift lanes a node: the least power of two that holds its pairs, at most 32.
__device__ __forceinline__ void form_turns(const HeadNormArgs& a, const Turns* freq, float2* turn, int node0, int nodes) {
  const int pairs = a.D / 2, lane = threadIdx.x & 31, side = 1 << a.shift;
  __syncwarp();  // the last nodes' have been read
  for (int n = lane >> a.shift; n < nodes; n += 32 >> a.shift) {
    const float* pos = a.pos + (long long)(node0 + n) * a.axes;
    float x[3];
#pragma unroll
    for (int i = 0; i < 3; ++i) x[i] = i < a.axes ? __ldg(pos + i) : 0.0f;
    for (int p = lane & (side - 1); p < pairs; p += side) {
      const Turns* f = freq + p * a.axes;
      float t = f[0].of(x[0]);
      if (a.axes > 1) t += f[1].of(x[1]);
      if (a.axes > 2) t += f[2].of(x[2]);
      t -= rintf(t);
      float s, c;
      sincospif(2.0f * t, &s, &c);
      turn[n * pairs + p] = make_float2(c, s);
    }
  }
  __syncwarp();
}

// The lane's pairs of a node.
template <int V, int G, int NV>
__device__ __forceinline__ void load_turns(const float2* turn, int pairs, int l, float2 (&t)[NV * V / 2]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int first = (j * G + l) * (V / 2);
#pragma unroll
    for (int p = 0; p < V / 2; ++p) t[j * V / 2 + p] = make_float2(1.0f, 0.0f);
    if (first < pairs)  // all of a vector's pairs are there, or none
#pragma unroll
      for (int p = 0; p < V / 2; ++p) t[j * V / 2 + p] = turn[first + p];
  }
}

// The U rows of a step: the same 32 / G heads of neighbouring nodes, so that what
// hangs on the heads alone (addresses, weights) is found once for all of them; or,
// where there are few nodes, the next heads of one node.  Either way they are on
// their way together.
template <typename T>
struct HeadStep {
  int t, heads, first, nodes;  // the lane's first head, of how many; their place in rstd; nodes there
  bool key, by_head;
  __device__ __forceinline__ HeadStep(const HeadNormArgs& a, bool key, int t, int nodes)
      : t(t), heads(key ? a.Hk : a.Hq), first(key ? a.Hq : 0), nodes(nodes), key(key), by_head(a.each == 1) {}
  template <int AT_ONCE>
  __device__ __forceinline__ bool has(int u) const {
    return by_head ? nodes > 0 && t + u * AT_ONCE < heads : u < nodes && t < heads;
  }
};

// Where a step's rows lie in an array: the first, and the distance between them.
template <typename T>
struct HeadRows {
  const T* x;
  long long step;
  template <int AT_ONCE>
  static __device__ __forceinline__ HeadRows at(const HeadNormArgs& a, const HeadStep<T>& s, const void* q, long long q_ld, const void* k,
                                                long long k_ld, int node0) {
    const long long ld = s.key ? k_ld : q_ld;
    return HeadRows{static_cast<const T*>(s.key ? k : q) + node0 * ld + s.t * a.D, s.by_head ? (long long)AT_ONCE * a.D : ld};
  }
};

template <typename T, int V, int G, int NV, int U>
__global__ void __launch_bounds__(32 * kHeadWarps, 4) k_head_norm(const __grid_constant__ HeadNormArgs a) {
  constexpr int W = NV * V, P = W / 2, AT_ONCE = 32 / G;
  using Share = HeadShare<T, V, G, NV>;
  __shared__ Turns freq[128 * 3];
  __shared__ __align__(16) float2 turns[kHeadWarps][U * G * W / 2];
  const int lane = threadIdx.x & 31, l = lane % G, all = a.Hq + a.Hk, pairs = a.D / 2;
  float2* const turn = turns[threadIdx.x >> 5];
  const float per_d = 1.0f / (float)a.D;
  bool ready = false;
  for (int node0 = (int)(blockIdx.x * kHeadWarps + (threadIdx.x >> 5)) * a.each;; node0 += gridDim.x * kHeadWarps * a.each) {
    const int nodes = min(a.N - node0, a.each);
    if (nodes <= 0 && ready) break;
    bool fresh = true;
    for (int key = 0; key < (a.Hk ? 2 : 1); ++key) {
      float w[W];
      load_weights<V, G, NV>(key ? a.wk : a.wq, l, a.D, w);
      T* const out = static_cast<T*>(key ? a.ok : a.oq);
      for (int t0 = 0; t0 < (key ? a.Hk : a.Hq); t0 += a.each == 1 ? U * AT_ONCE : AT_ONCE) {
        const HeadStep<T> s(a, key, t0 + lane / G, nodes);
        const HeadRows<T> from = HeadRows<T>::template at<AT_ONCE>(a, s, a.q, a.q_ld, a.k, a.k_ld, node0);
        const int row0 = s.by_head ? AT_ONCE : s.heads, rstd0 = s.by_head ? AT_ONCE : all;  // from one row to the next
        Share x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u].load(from.x + u * from.step, l, a.D, s.template has<AT_ONCE>(u));
        if (fresh) {
          if (!ready) {  // once, behind the first rows' loads
            if (a.axes) load_freq(a, freq);
            __syncthreads();
            ready = true;
          }
          if (a.axes) form_turns(a, freq, turn, node0, nodes);
          fresh = false;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float f[W], ss = 0.0f;
          x[u].get(f);
#pragma unroll
          for (int i = 0; i < W; ++i) ss = fmaf(f[i], f[i], ss);
#pragma unroll
          for (int o = G / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          if (!s.template has<AT_ONCE>(u)) continue;
          const float r = rsqrtf(fmaf(ss, per_d, a.eps));
          if (a.rstd && l == 0) a.rstd[(long long)node0 * all + s.first + s.t + u * rstd0] = r;
#pragma unroll
          for (int i = 0; i < W; ++i) f[i] *= r * w[i];
          if (a.axes) {
            float2 cs[P];
            load_turns<V, G, NV>(turn + (s.by_head ? 0 : u * pairs), pairs, l, cs);
#pragma unroll
            for (int p = 0; p < P; ++p) {
              const float u0 = f[2 * p], u1 = f[2 * p + 1];
              f[2 * p] = u0 * cs[p].x - u1 * cs[p].y;
              f[2 * p + 1] = u0 * cs[p].y + u1 * cs[p].x;
            }
          }
          if (out) Share::store(out + ((long long)node0 * s.heads + s.t + u * row0) * a.D, l, a.D, f);
        }
      }
    }
  }
}

template <typename T, int V, int G, int NV, int U>
__global__ void __launch_bounds__(32 * kHeadWarps, 3) k_head_norm_bwd(const __grid_constant__ HeadNormArgs a) {
  constexpr int W = NV * V, P = W / 2, AT_ONCE = 32 / G;
  using Share = HeadShare<T, V, G, NV>;
  __shared__ Turns freq[128 * 3];
  __shared__ __align__(16) float2 turns[kHeadWarps][U * G * W / 2];
  __shared__ float red[kHeadWarps][2 * G * W];
  const int lane = threadIdx.x & 31, l = lane % G, warp = threadIdx.x >> 5, all = a.Hq + a.Hk, pairs = a.D / 2;
  float2* const turn = turns[warp];
  const float per_d = 1.0f / (float)a.D;
  float dwq[W], dwk[W];
#pragma unroll
  for (int i = 0; i < W; ++i) dwq[i] = dwk[i] = 0.0f;
  if (a.axes) load_freq(a, freq);
  __syncthreads();
  for (int node0 = (int)(blockIdx.x * kHeadWarps + warp) * a.each; node0 < a.N; node0 += gridDim.x * kHeadWarps * a.each) {
    const int nodes = min(a.N - node0, a.each);
    if (a.axes) form_turns(a, freq, turn, node0, nodes);
    float turned[U][P];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int p = 0; p < P; ++p) turned[u][p] = 0.0f;
    auto run = [&](bool key, float (&dw)[W]) {
      float w[W];
      load_weights<V, G, NV>(key ? a.wk : a.wq, l, a.D, w);
      T* const out = static_cast<T*>(key ? a.ok : a.oq);
      for (int t0 = 0; t0 < (key ? a.Hk : a.Hq); t0 += a.each == 1 ? U * AT_ONCE : AT_ONCE) {
        const HeadStep<T> s(a, key, t0 + lane / G, nodes);
        const HeadRows<T> from = HeadRows<T>::template at<AT_ONCE>(a, s, a.q, a.q_ld, a.k, a.k_ld, node0);
        const HeadRows<T> from_g = HeadRows<T>::template at<AT_ONCE>(a, s, a.gq, a.gq_ld, a.gk, a.gk_ld, node0);
        const int row0 = s.by_head ? AT_ONCE : s.heads, rstd0 = s.by_head ? AT_ONCE : all;
        Share x[U], g[U];
        float r[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const bool ok = s.template has<AT_ONCE>(u);
          x[u].load(from.x + u * from.step, l, a.D, ok);
          g[u].load(from_g.x + u * from_g.step, l, a.D, ok);
          r[u] = ok ? __ldg(a.rstd + (long long)node0 * all + s.first + s.t + u * rstd0) : 0.0f;
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {  // rows that are not there are zeros and change no sum
          float h[W], b[W], mean = 0.0f;
          x[u].get(h);
          g[u].get(b);
#pragma unroll
          for (int i = 0; i < W; ++i) h[i] *= r[u];
          if (a.axes) {
            float2 cs[P];
            load_turns<V, G, NV>(turn + (s.by_head || u >= nodes ? 0 : u * pairs), pairs, l, cs);
#pragma unroll
            for (int p = 0; p < P; ++p) {
              const float g0 = b[2 * p], g1 = b[2 * p + 1];
              b[2 * p] = g0 * cs[p].x + g1 * cs[p].y;
              b[2 * p + 1] = g1 * cs[p].x - g0 * cs[p].y;
              if (a.gpos) turned[u][p] += b[2 * p + 1] * (h[2 * p] * w[2 * p]) - b[2 * p] * (h[2 * p + 1] * w[2 * p + 1]);
            }
          }
#pragma unroll
          for (int i = 0; i < W; ++i) {
            dw[i] = fmaf(b[i], h[i], dw[i]);
            b[i] *= w[i];
            mean = fmaf(b[i], h[i], mean);
          }
#pragma unroll
          for (int o = G / 2; o > 0; o >>= 1) mean += __shfl_xor_sync(0xffffffffu, mean, o);
          if (!out || !s.template has<AT_ONCE>(u)) continue;
          mean *= per_d;
#pragma unroll
          for (int i = 0; i < W; ++i) b[i] = r[u] * fmaf(-h[i], mean, b[i]);
          Share::store(out + ((long long)node0 * s.heads + s.t + u * row0) * a.D, l, a.D, b);
        }
      }
    };
    run(false, dwq);
    if (a.Hk) run(true, dwk);
    if (!a.gpos) continue;
    if (a.each == 1)  // one node's heads
#pragma unroll
      for (int u = 1; u < U; ++u)
#pragma unroll
        for (int p = 0; p < P; ++p) turned[0][p] += turned[u][p];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (u >= nodes) break;
      float d[3] = {0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int pair = ((2 * p / V * G + l) * V + 2 * p % V) / 2;
#pragma unroll
        for (int x = 0; x < 3; ++x)
          if (pair < pairs && x < a.axes) d[x] = fmaf(turned[u][p], freq[pair * a.axes + x].hi, d[x]);
      }
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        if (x >= a.axes) break;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) d[x] += __shfl_xor_sync(0xffffffffu, d[x], o);
        if (lane == 0) a.gpos[(long long)(node0 + u) * a.axes + x] = d[x] * 6.2831853071795865f;
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
