// The norms' kernels for rows that fit the registers of one CTA.
//
// A group of G lanes owns one row at a time: `active` of them hold up to NV
// vectors of V values each, lane t the vectors t, t + active, t + 2 active...
// G is a power of two up to 32 (a warp works on 32/G rows, sums by shuffles)
// or a multiple of 32 (sums by shuffles, then through shared memory).  With
// degrees (L > 0), `active` is a multiple of K / gcd(K, V), so the component
// of a lane's i-th value is the same in all of its vectors: what depends on
// the degree (its class, its mean, its deviation) is one value per slot i,
// and a row's sums of squares go to their degrees once per row, not once per
// value.
#pragma once

#include "common.cuh"
#include "launch.h"
#include "norm.cuh"

namespace eqmp {

struct RowShape {
  int lanes;   // G
  int active;  // lanes that hold values
  int groups;  // rows of a CTA at a time
};

// ---------------------------------------------------------------- vectors
// V values of type T as loaded: 16 bytes, or one value.
template <typename T, int V>
struct Pack;

template <>
struct Pack<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void zero() { v = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void get(float (&f)[4]) const {
    f[0] = v.x;
    f[1] = v.y;
    f[2] = v.z;
    f[3] = v.w;
  }
  __device__ __forceinline__ static void store(float* p, const float (&f)[4]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
  }
};

template <>
struct Pack<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = bf16_lo(v.x);
    f[1] = bf16_hi(v.x);
    f[2] = bf16_lo(v.y);
    f[3] = bf16_hi(v.y);
    f[4] = bf16_lo(v.z);
    f[5] = bf16_hi(v.z);
    f[6] = bf16_lo(v.w);
    f[7] = bf16_hi(v.w);
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float (&f)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                              pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
  }
};

template <typename T>
struct Pack<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = T(0.0f); }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = load1(&v); }
  __device__ __forceinline__ static void store(T* p, const float (&f)[1]) { store1(p, f[0]); }
};

// Dropout of V consecutive values of a row from column col (a multiple of V).
template <int V>
__device__ __forceinline__ void drop_values(const Dropper& d, float (&f)[V], uint32_t row, int col) {
  if (V > 1 && d.group == 1) {
    const uint4 w = d.block(row, (uint32_t)col >> 3);
    const bool upper = V == 4 && (col & 4);
    const uint32_t w0 = upper ? w.z : w.x, w1 = upper ? w.w : w.y;
    const uint32_t words[4] = {w0, w1, w.z, w.w};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const uint32_t draw = (i & 1) ? words[i >> 1] >> 16 : words[i >> 1] & 0xffffu;
      f[i] = draw >= d.threshold ? f[i] * d.scale : 0.0f;
    }
    return;
  }
  // the units that the vector touches, one after the other
  uint32_t unit = (uint32_t)col / (uint32_t)d.group;
  int end = (int)((unit + 1) * (uint32_t)d.group) - col;  // of the unit, counted from the vector's start
  uint32_t blk = unit >> 3, keep = 0;
  uint4 w = d.block(row, blk);
#pragma unroll 1
  for (int at = 0;;) {
    if (Dropper::draw(w, unit) >= d.threshold) keep |= (end >= V ? 1u << V : 1u << end) - (1u << at);
    if (end >= V) break;
    at = end;
    end += d.group;
    ++unit;
    if (unit >> 3 != blk) w = d.block(row, blk = unit >> 3);
  }
#pragma unroll
  for (int i = 0; i < V; ++i) f[i] = (keep >> i) & 1 ? f[i] * d.scale : 0.0f;
}

// ---------------------------------------------------------------- sums
// Sums N values over the lanes of each group, in a fixed order.  Groups of
// several warps exchange their warps' sums through red (two halves of
// N floats per warp of the CTA, taken in turn, so that one barrier per sum is
// enough); every thread of the CTA takes part.
template <int N>
struct GroupSum {
  int lanes, warps, first;  // of the group: lanes, warps, its first warp
  float* red;
  int half;
  __device__ __forceinline__ GroupSum(int lanes_, float* red_) : lanes(lanes_), red(red_), half(0) {
    warps = lanes_ >> 5;
    first = warps > 1 ? (int)(threadIdx.x >> 5) / warps * warps : 0;
  }
  template <int M>
  __device__ __forceinline__ void operator()(float (&v)[M]) {
    static_assert(M <= N, "buffer too small");
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o < lanes) {
#pragma unroll
        for (int i = 0; i < M; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
      }
    }
    if (lanes <= 32) return;
    const int all = blockDim.x >> 5;
    float* buf = red + half * all * N;
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int i = 0; i < M; ++i) buf[i * all + (threadIdx.x >> 5)] = v[i];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < M; ++i) {
      float t = buf[i * all + first];
      for (int k = 1; k < warps; ++k) t += buf[i * all + first + k];
      v[i] = t;
    }
    half ^= 1;
  }
};

// What a lane knows of its columns.
template <int L, int V, int NV>
struct Slots {
  static constexpr int K = (L + 1) * (L + 1);
  int lane, col0, stride;  // within the group; of vector 0; between vectors
  int cls[L ? V : 1];      // degree of value i (L > 0)
  uint32_t first;          // bit i: value i is a degree 0 (L > 0)
  __device__ __forceinline__ Slots(const RowShape& sh) {
    lane = threadIdx.x % sh.lanes;
    col0 = lane * V;
    stride = sh.active * V;
    first = 0;
    if (L) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int k = (col0 + i) % K;
        int l = 0;
#pragma unroll
        for (int m = 1; m <= L; ++m) l += k >= m * m;
        cls[i] = l;
        first |= (uint32_t)(l == 0) << i;
      }
    }
  }
  __device__ __forceinline__ bool is0(int i) const { return L == 0 || ((first >> i) & 1); }
  __device__ __forceinline__ int col(int j) const { return col0 + j * stride; }
  // The slots' sums put to their degrees.
  __device__ __forceinline__ void by_degree(const float (&slot)[V], float (&out)[L + 1]) const {
    if (L == 0) {
      float t = slot[0];
#pragma unroll
      for (int i = 1; i < V; ++i) t += slot[i];
      out[0] = t;
    } else {
#pragma unroll
      for (int l = 0; l <= L; ++l) {
        float t = 0.0f;
#pragma unroll
        for (int i = 0; i < V; ++i) t += cls[i] == l ? slot[i] : 0.0f;
        out[l] = t;
      }
    }
  }
  // The degrees' values put to the slots.
  __device__ __forceinline__ void to_slots(const float (&deg)[L + 1], float (&slot)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float t = deg[0];
#pragma unroll
      for (int l = 1; l <= L; ++l) t = cls[L ? i : 0] == l ? deg[l] : t;
      slot[i] = t;
    }
  }
  __device__ __forceinline__ void degree0(float v, float (&slot)[V]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) slot[i] = is0(i) ? v : 0.0f;
  }
};

constexpr int kRowThreads = 256;     // of a CTA, where a group is smaller
constexpr int kMaxRowThreads = 512;  // 128 registers a thread: 16 values of each array with their weights

// ---------------------------------------------------------------- forward
// One pass: each value is loaded once, kept in registers through the mean and
// the centred squares, and stored once.  The next row's vectors are loaded
// before the sums of the current one are formed.  FUSED: with a residual sum
// or dropout in front.
template <typename T, int L, int V, int NV, bool FUSED>
__global__ void __launch_bounds__(kMaxRowThreads) k_norm_rows(NormArgs a, RowShape sh) {
  __shared__ float red[2 * (kMaxRowThreads / 32) * (L + 1)];
  const Slots<L, V, NV> at(sh);
  GroupSum<L + 1> sum(sh.lanes, red);
  Dropper drop(a.drop);
  const T* x = static_cast<const T*>(a.x);
  const T* r = static_cast<const T*>(a.r);
  bool has[NV];
  float w[NV][V], b[NV][V];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    has[j] = at.lane < sh.active && at.col(j) < a.cols;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (at.col(j) + i) / at.K, l = L ? at.cls[L ? i : 0] : 0;
      w[j][i] = has[j] && a.w ? a.w[l * a.C + c] : 1.0f;
      b[j][i] = has[j] && a.b && at.is0(i) ? a.b[c] : 0.0f;
    }
  }
  const float inv = 1.0f / (float)a.C;
  const int stride = gridDim.x * sh.groups;
  Pack<T, V> nx[NV], nr[FUSED ? NV : 1];
  auto fetch = [&](int row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const bool ok = has[j] && row < a.rows;
      if (ok)
        nx[j].load(x + (long long)row * a.x_ld + at.col(j));
      else
        nx[j].zero();
      if (FUSED) {
        if (ok && r)
          nr[FUSED ? j : 0].load(r + (long long)row * a.r_ld + at.col(j));
        else
          nr[FUSED ? j : 0].zero();
      }
    }
  };
  int row = blockIdx.x * sh.groups + threadIdx.x / sh.lanes;
  fetch(row);
  // the same number of rounds for every group of the CTA
  for (int base = blockIdx.x * sh.groups; base < a.rows; base += stride, row += stride) {
    float v[NV][V], slot[V];
#pragma unroll
    for (int j = 0; j < NV; ++j) nx[j].get(v[j]);
    if (FUSED) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (drop.threshold) drop_values<V>(drop, v[j], row, at.col(j));
        float f[V];
        nr[FUSED ? j : 0].get(f);
#pragma unroll
        for (int i = 0; i < V; ++i) v[j][i] += f[i];
      }
    }
    fetch(row + stride);
    const bool live = row < a.rows;
    const long long out = (long long)row * a.cols;
    if (FUSED && a.s && live) {
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (has[j]) Pack<T, V>::store(static_cast<T*>(a.s) + out + at.col(j), v[j]);
    }
    float mean[1] = {0.0f};
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float t = v[0][i];
#pragma unroll
      for (int j = 1; j < NV; ++j) t += v[j][i];
      mean[0] += at.is0(i) ? t : 0.0f;
    }
    sum(mean);
    mean[0] *= inv;
    at.degree0(mean[0], slot);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] = has[j] ? v[j][i] - slot[i] : 0.0f;
    float q[L + 1];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      slot[i] = v[0][i] * v[0][i];
#pragma unroll
      for (int j = 1; j < NV; ++j) slot[i] += v[j][i] * v[j][i];
    }
    at.by_degree(slot, q);
    sum(q);
#pragma unroll
    for (int l = 0; l <= L; ++l) q[l] = 1.0f / sqrtf(q[l] * (inv * (1.0f / (2 * l + 1))) + a.eps);
    if (!live) continue;
    if (a.stats && at.lane == 0) {
      float* st = a.stats + (long long)row * (L + 2);
      st[0] = mean[0];
#pragma unroll
      for (int l = 0; l <= L; ++l) st[1 + l] = q[l];
    }
    if (!a.y) continue;
    at.to_slots(q, slot);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[j][i] = v[j][i] * slot[i] * w[j][i] + b[j][i];
      if (has[j]) Pack<T, V>::store(static_cast<T*>(a.y) + out + at.col(j), v[j]);
    }
  }
}

// ---------------------------------------------------------------- backward
// One pass over g and s (and dL/ds): the row's sums of a and a h, then dL/ds
// and dL/dx from the registers, while each lane adds g h and g of its columns
// over all the rows of its group.  At the end the groups of a CTA are added in
// their order through shared memory, the orders of a degree with them, and
// the CTA's (L+2) C sums go to its part of the workspace.  FUSED: with dL/ds
// of a residual stream, dropout, or both gradients asked for.
template <typename T, int L, int V, int NV, bool FUSED>
__global__ void __launch_bounds__(kMaxRowThreads) k_norm_bwd_rows(NormArgs a, RowShape sh) {
  __shared__ float red[2 * (kMaxRowThreads / 32) * (L + 2)];
  extern __shared__ float colsum[];  // [cols] g h, then [C] g
  const Slots<L, V, NV> at(sh);
  GroupSum<L + 2> sum(sh.lanes, red);
  const Dropper drop(a.drop);
  const T* x = static_cast<const T*>(a.x);
  const T* g = static_cast<const T*>(a.g);
  const T* r = static_cast<const T*>(a.r);
  constexpr int NB = L ? 1 : V;  // degree-0 values of a vector, at most
  constexpr int NQ = L ? V : 1;  // deviations of a lane's slots
  bool has[NV];
  float w[NV][V], dw[NV][V], db[NV][NB];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    has[j] = at.lane < sh.active && at.col(j) < a.cols;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (at.col(j) + i) / at.K, l = L ? at.cls[L ? i : 0] : 0;
      w[j][i] = has[j] && a.w ? a.w[l * a.C + c] : 1.0f;
      dw[j][i] = 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NB; ++i) db[j][i] = 0.0f;
  }
  const float inv = 1.0f / (float)a.C;
  const int stride = gridDim.x * sh.groups;
  Pack<T, V> nx[NV], ng[NV], nr[FUSED ? NV : 1];
  float nmean, nq[NQ];
  auto fetch = [&](int row) {
    const bool live = row < a.rows;
    const float* st = a.stats + (long long)row * (L + 2);
    nmean = live ? st[0] : 0.0f;
#pragma unroll
    for (int i = 0; i < NQ; ++i) nq[i] = live ? st[1 + (L ? at.cls[L ? i : 0] : 0)] : 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (has[j] && live) {
        nx[j].load(x + (long long)row * a.x_ld + at.col(j));
        ng[j].load(g + (long long)row * a.g_ld + at.col(j));
      } else {
        nx[j].zero();
        ng[j].zero();
      }
      if (FUSED) {
        if (has[j] && live && r)
          nr[FUSED ? j : 0].load(r + (long long)row * a.r_ld + at.col(j));
        else
          nr[FUSED ? j : 0].zero();
      }
    }
  };
  int row = blockIdx.x * sh.groups + threadIdx.x / sh.lanes;
  fetch(row);
  for (int base = blockIdx.x * sh.groups; base < a.rows; base += stride, row += stride) {
    float h[NV][V], av[NV][V], slot[V], tot[L + 2], q[NQ];
    Pack<T, V> cr[FUSED ? NV : 1];
#pragma unroll
    for (int i = 0; i < NQ; ++i) q[i] = nq[i];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      nx[j].get(h[j]);
      ng[j].get(av[j]);
      if (FUSED) cr[FUSED ? j : 0] = nr[FUSED ? j : 0];
    }
    const float mean = nmean;
    fetch(row + stride);
    tot[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const bool first = at.is0(i);
      const float mu = first ? mean : 0.0f, qi = q[L ? i : 0];
      slot[i] = 0.0f;
      float sa = 0.0f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        h[j][i] = (h[j][i] - mu) * qi;
        dw[j][i] += av[j][i] * h[j][i];
        if (L == 0)
          db[j][L ? 0 : i] += av[j][i];
        else
          db[j][0] += first ? av[j][i] : 0.0f;
        av[j][i] *= w[j][i];
        sa += av[j][i];
        slot[i] += av[j][i] * h[j][i];
      }
      tot[0] += first ? sa : 0.0f;
    }
    float deg[L + 1];
    at.by_degree(slot, deg);
#pragma unroll
    for (int l = 0; l <= L; ++l) tot[1 + l] = deg[l];
    sum(tot);
    if (row >= a.rows) continue;
    const float m0 = tot[0] * inv;
#pragma unroll
    for (int l = 0; l <= L; ++l) deg[l] = tot[1 + l] * (inv * (1.0f / (2 * l + 1)));
    at.to_slots(deg, slot);
    const long long out = (long long)row * a.cols;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V];
#pragma unroll
      for (int i = 0; i < V; ++i)
        f[i] = (av[j][i] - h[j][i] * slot[i] - (at.is0(i) ? m0 : 0.0f)) * q[L ? i : 0];
      if (FUSED) {
        float s[V];
        cr[FUSED ? j : 0].get(s);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] += s[i];
        if (a.gr && has[j]) Pack<T, V>::store(static_cast<T*>(a.gr) + out + at.col(j), f);
        if (a.gx) {
          if (drop.threshold) drop_values<V>(drop, f, row, at.col(j));
          if (has[j]) Pack<T, V>::store(static_cast<T*>(a.gx) + out + at.col(j), f);
        }
      } else if (has[j]) {
        T* dst = static_cast<T*>(a.gx ? a.gx : a.gr);
        if (dst) Pack<T, V>::store(dst + out + at.col(j), f);
      }
    }
  }
  if (!a.gw && !a.gb) return;
  // the CTA's sums: the groups of a warp by shuffles, the warps (or the
  // groups of several warps) in turn
  if (sh.lanes < 32) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      if (o >= sh.lanes) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
          for (int i = 0; i < V; ++i) dw[j][i] += __shfl_xor_sync(0xffffffffu, dw[j][i], o);
#pragma unroll
          for (int i = 0; i < NB; ++i) db[j][i] += __shfl_xor_sync(0xffffffffu, db[j][i], o);
        }
      }
    }
  }
  const int unit = sh.lanes <= 32 ? 32 : sh.lanes;  // threads that add together
  const int units = (blockDim.x + unit - 1) / unit, mine = threadIdx.x / unit;
  const bool speaks = (int)(threadIdx.x % unit) < sh.lanes;
  for (int u = 0; u < units; ++u) {
    if (u == mine && speaks) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!has[j]) continue;
        const int col = at.col(j);
#pragma unroll
        for (int i = 0; i < V; ++i) {
          colsum[col + i] = u ? colsum[col + i] + dw[j][i] : dw[j][i];
          if (at.is0(i)) {
            float* d = colsum + a.cols + (col + i) / at.K;
            const float v = db[j][L ? 0 : i];
            *d = u ? *d + v : v;
          }
        }
      }
    }
    __syncthreads();
  }
  const int M = (L + 2) * a.C, nw = (L + 1) * a.C;
  float* part = a.parts > 1 ? a.part + (long long)blockIdx.x * M : nullptr;
  for (int m = threadIdx.x; m < M; m += blockDim.x) {
    float t = 0.0f;
    if (L && m < nw) {
      const int l = m / a.C, c = m - l * a.C;
      for (int k = l * l; k < (l + 1) * (l + 1); ++k) t += colsum[c * at.K + k];
    } else {
      t = colsum[L ? a.cols + m - nw : m];
    }
    if (part)
      part[m] = t;
    else if (m < nw) {
      if (a.gw) a.gw[m] = t;
    } else if (a.gb) {
      a.gb[m - nw] = t;
    }
  }
}

// ---------------------------------------------------------------- launch
// Lanes for a row of cols values in vectors of V, NV per lane.
inline RowShape row_shape(int cols, int K, int V, int NV) {
  int period = 1;  // K / gcd(K, V)
  while (period * V % K) ++period;
  const int vectors = cols / V;
  RowShape sh;
  sh.active = ((vectors + NV - 1) / NV + period - 1) / period * period;
  if (sh.active <= 32) {
    sh.lanes = 1;
    while (sh.lanes < sh.active) sh.lanes *= 2;
  } else {
    sh.lanes = (sh.active + 31) / 32 * 32;
  }
  sh.groups = sh.lanes < kRowThreads ? kRowThreads / sh.lanes : 1;
  return sh;
}

constexpr int kMaxColSum = 2 * 16 * kMaxRowThreads * 4;  // bytes of the column sums of the widest row

// dw and db from the parts (norm.cu).
eqmp_status launch_norm_bwd_sum(const NormArgs& a, int L, cudaStream_t st);

// CTAs of a persistent launch: what the device holds at a time, at most one
// per group of rows.
template <typename Kernel>
inline int resident_grid(Kernel kernel, int threads, size_t smem, const DeviceInfo& dev, long long tiles,
                         int (&cache)[64][33]) {
  int d = 0;
  if (cudaGetDevice(&d) != cudaSuccess) return 0;
  int occ = __atomic_load_n(&cache[d & 63][threads / 32], __ATOMIC_RELAXED);
  if (occ == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kernel, threads, smem) != cudaSuccess || occ < 1) return 0;
    __atomic_store_n(&cache[d & 63][threads / 32], occ, __ATOMIC_RELAXED);
  }
  const long long cap = (long long)dev.sms * occ;
  return (int)(tiles < cap ? tiles : cap);
}

template <typename T, int L, int V, int NV, bool FUSED>
static eqmp_status launch_fwd(const NormArgs& a, const RowShape& sh, const DeviceInfo& dev, cudaStream_t st) {
  static int cache[64][33];
  const int threads = sh.lanes * sh.groups;
  auto kern = k_norm_rows<T, L, V, NV, FUSED>;
  const int grid = resident_grid(kern, threads, 0, dev, ((long long)a.rows + sh.groups - 1) / sh.groups, cache);
  if (grid < 1) return EQMP_ERR_CUDA;
  kern<<<grid, threads, 0, st>>>(a, sh);
  return cuda_status(cudaGetLastError());
}

template <typename T, int L, int V, int NV, bool FUSED>
static eqmp_status launch_bwd(NormArgs a, const RowShape& sh, const DeviceInfo& dev, cudaStream_t st) {
  static int cache[64][33];
  const int threads = sh.lanes * sh.groups;
  const size_t smem = a.gw || a.gb ? sizeof(float) * ((size_t)a.cols + a.C) : 0;
  auto kern = k_norm_bwd_rows<T, L, V, NV, FUSED>;
  static unsigned long long attr_done = 0;
  if (ensure_smem_attr(kern, kMaxColSum, &attr_done) != cudaSuccess) return EQMP_ERR_CUDA;
  int grid = resident_grid(kern, threads, smem, dev, ((long long)a.rows + sh.groups - 1) / sh.groups, cache);
  if (grid < 1) return EQMP_ERR_CUDA;
  if (grid > kMaxParts) grid = kMaxParts;
  a.parts = grid;
  kern<<<grid, threads, smem, st>>>(a, sh);
  if (cudaGetLastError() != cudaSuccess) return EQMP_ERR_CUDA;
  if ((!a.gw && !a.gb) || grid == 1) return EQMP_OK;
  return launch_norm_bwd_sum(a, L, st);
}

template <typename T, int L, int V, int NV, bool BACKWARD>
static eqmp_status launch_rows(const NormArgs& a, const RowShape& sh, const DeviceInfo& dev, cudaStream_t st) {
  if constexpr (BACKWARD) {
    const bool fused = a.r || a.drop.threshold || (a.gr && a.gx);
    return fused ? launch_bwd<T, L, V, NV, true>(a, sh, dev, st) : launch_bwd<T, L, V, NV, false>(a, sh, dev, st);
  } else {
    const bool fused = a.r || a.drop.threshold || a.s;
    return fused ? launch_fwd<T, L, V, NV, true>(a, sh, dev, st) : launch_fwd<T, L, V, NV, false>(a, sh, dev, st);
  }
}

// 8 or 16 values a lane.  Forward: whichever leaves fewer places empty; 8
// where both are equal and the row fits a warp (fewer registers, more rows in
// flight).  Backward: 8 where the row fits, since 16 values of every array do
// not fit 128 registers.
template <typename T, int L, int V, bool BACKWARD>
static eqmp_status launch_rows_v(const NormArgs& a, const DeviceInfo& dev, cudaStream_t st, bool* done) {
  constexpr int K = (L + 1) * (L + 1), N8 = 8 / V, N16 = 16 / V;
  const RowShape s8 = row_shape(a.cols, K, V, N8), s16 = row_shape(a.cols, K, V, N16);
  const int p8 = s8.lanes * N8, p16 = s16.lanes * N16;
  const bool take8 = s8.lanes <= kMaxRowThreads && (BACKWARD || p8 < p16 || (p8 == p16 && s8.lanes <= 32));
  *done = take8 || s16.lanes <= kMaxRowThreads;
  if (!*done) return EQMP_OK;
  return take8 ? launch_rows<T, L, V, N8, BACKWARD>(a, s8, dev, st) : launch_rows<T, L, V, N16, BACKWARD>(a, s16, dev, st);
}

inline bool vec16(const void* p, long long ld, int bytes) {
  return !p || (reinterpret_cast<uintptr_t>(p) % 16 == 0 && ld * bytes % 16 == 0);
}

// Runs the pass if the row fits; *done says whether it did.  Vectors of 16
// bytes where every row of every array starts on one.
template <typename T, int L, bool BACKWARD>
static eqmp_status launch_rows_l(const NormArgs& a, const DeviceInfo& dev, cudaStream_t st, bool* done) {
  constexpr int B = sizeof(T);
  const bool vec = vec16(a.x, a.x_ld, B) && vec16(a.r, a.r_ld, B) && vec16(a.g, a.g_ld, B) && vec16(a.s, a.cols, B) &&
                   vec16(a.y, a.cols, B) && vec16(a.gr, a.cols, B) && vec16(a.gx, a.cols, B) && a.cols * B % 16 == 0;
  return vec ? launch_rows_v<T, L, 16 / B, BACKWARD>(a, dev, st, done) : launch_rows_v<T, L, 1, BACKWARD>(a, dev, st, done);
}

template <typename T, bool BACKWARD>
static eqmp_status launch_rows_t(const NormArgs& a, int L, const DeviceInfo& dev, cudaStream_t st, bool* done) {
  switch (L) {
    case 0: return launch_rows_l<T, 0, BACKWARD>(a, dev, st, done);
    case 3: return launch_rows_l<T, 3, BACKWARD>(a, dev, st, done);
    case 4: return launch_rows_l<T, 4, BACKWARD>(a, dev, st, done);
    case 5: return launch_rows_l<T, 5, BACKWARD>(a, dev, st, done);
    case 6: return launch_rows_l<T, 6, BACKWARD>(a, dev, st, done);
  }
  return EQMP_ERR_UNSUPPORTED;
}

eqmp_status launch_norm_rows_f32(const NormArgs& a, int L, const DeviceInfo& dev, cudaStream_t st, bool* done);
eqmp_status launch_norm_rows_bf16(const NormArgs& a, int L, const DeviceInfo& dev, cudaStream_t st, bool* done);
eqmp_status launch_norm_bwd_rows_f32(const NormArgs& a, int L, const DeviceInfo& dev, cudaStream_t st, bool* done);
eqmp_status launch_norm_bwd_rows_bf16(const NormArgs& a, int L, const DeviceInfo& dev, cudaStream_t st, bool* done);

}  // namespace eqmp
