// The norms' kernels for rows that fit the registers of one CTA.
//
// A group of G lanes owns one row at a time: `active` of them hold up to NV
// vectors of V values each, lane t the vectors t, t + active, t + 2 active...
// G is a power of two up to 32 (a warp works on 32/G rows, sums by shuffles)
// or a multiple of 32 (sums by shuffles, then through shared memory).  With
// degrees (L > 0), `active` is a multiple of K / gcd(K, V), so the component
// of a lane's i-th value is the same in all of its vectors: what depends on
// the degree is one value per slot i, and a row's sums go to their degrees
// once per row, not once per value.
//
// The values move from and to HBM once, so these kernels are bound by
// instructions before they are bound by memory: a bf16 value that is read and
// written once may cost about 20 of them.  Hence the arithmetic is on pairs
// (fma.rn.f32x2), and sums of several values are scattered over the lanes as
// they are formed.
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

constexpr int kRowThreads = 256;     // of a CTA, where a group is smaller
constexpr int kMaxRowThreads = 512;  // 128 registers a thread

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// ---------------------------------------------------------------- vectors
// V values of type T as loaded: 16 bytes, or one value.
template <typename T, int V>
struct Pack;

template <>
struct Pack<float, 4> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void zero() { v = make_float4(0.0f, 0.0f, 0.0f, 0.0f); }
  __device__ __forceinline__ void get(float2* f) const {
    f[0] = make_float2(v.x, v.y);
    f[1] = make_float2(v.z, v.w);
  }
  __device__ __forceinline__ static void store(float* p, const float2* f) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  }
};

template <>
struct Pack<__nv_bfloat16, 8> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void get(float2* f) const {
    f[0] = make_float2(bf16_lo(v.x), bf16_hi(v.x));
    f[1] = make_float2(bf16_lo(v.y), bf16_hi(v.y));
    f[2] = make_float2(bf16_lo(v.z), bf16_hi(v.z));
    f[3] = make_float2(bf16_lo(v.w), bf16_hi(v.w));
  }
  __device__ __forceinline__ static void store(__nv_bfloat16* p, const float2* f) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0].x, f[0].y), pack_bf16x2(f[1].x, f[1].y),
                                              pack_bf16x2(f[2].x, f[2].y), pack_bf16x2(f[3].x, f[3].y));
  }
};

template <typename T>
struct Pack<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = T(0.0f); }
};

// The NV vectors of a lane, as pairs of values: two neighbours, or for V = 1
// the values of two vectors.
template <typename T, int V, int NV>
__device__ __forceinline__ void get_pairs(const Pack<T, V> (&v)[NV], float2 (&p)[NV * V / 2]) {
  if constexpr (V == 1) {
#pragma unroll
    for (int k = 0; k < NV / 2; ++k) p[k] = make_float2(load1(&v[2 * k].v), load1(&v[2 * k + 1].v));
  } else {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j].get(p + j * (V / 2));
  }
}

template <typename T, int V, int NV>
__device__ __forceinline__ void put_pairs(T* row, const uint32_t (&col)[NV], const bool (&has)[NV],
                                          const float2 (&p)[NV * V / 2]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!has[j]) continue;
    if constexpr (V == 1)
      store1(row + col[j], j & 1 ? p[j / 2].y : p[j / 2].x);
    else
      Pack<T, V>::store(row + col[j], p + j * (V / 2));
  }
}

// ---------------------------------------------------------------- slots
// What a lane knows of its columns.  Values i = 0..V-1 of a vector fall into
// GROUPS of one degree: all of them (L = 0, or V = 1), the first and the other
// three of each four (K a multiple of 4: degrees begin at l^2 = 0 or 1 mod 4),
// or each by itself.
template <int L, int V, int NV>
struct Slots {
  static constexpr int K = (L + 1) * (L + 1);
  static constexpr bool FOURS = L > 0 && V > 1 && K % 4 == 0;
  static constexpr int GROUPS = L == 0 || V == 1 ? 1 : FOURS ? V / 2 : V;
  static constexpr int PAIRS = V > 1 ? V / 2 : 1;  // pairs of a vector
  uint32_t col[NV];
  bool has[NV];
  int lane;         // within the group
  int cls[GROUPS];  // degree
  float2 first[PAIRS];  // 1 where a value is a degree 0, else 0

  __device__ __forceinline__ Slots(const RowShape& sh, int cols) {
    lane = threadIdx.x % sh.lanes;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      col[j] = (lane + j * sh.active) * V;
      has[j] = lane < sh.active && (int)col[j] < cols;
    }
    if constexpr (L == 0) {
      cls[0] = 0;
    } else {
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const int k = (int)(col[0] + (FOURS ? g / 2 * 4 + g % 2 : g)) % K;
        int l = 0;
#pragma unroll
        for (int m = 1; m <= L; ++m) l += k >= m * m;
        cls[g] = l;
      }
    }
    float f[GROUPS];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) f[g] = cls[g] == 0 ? 1.0f : 0.0f;
    spread(f, first);
  }
  // Whether pair s of a vector may hold a degree 0.
  __device__ __forceinline__ static constexpr bool may0(int s) { return !FOURS || s % 2 == 0; }
  // One value per group put to the pairs of a vector.
  __device__ __forceinline__ static void spread(const float (&g)[GROUPS], float2 (&p)[PAIRS]) {
#pragma unroll
    for (int s = 0; s < PAIRS; ++s) {
      if (GROUPS == 1)
        p[s] = both(g[0]);
      else if (FOURS)
        p[s] = s % 2 ? both(g[s / 2 * 2 + 1]) : make_float2(g[s / 2 * 2], g[s / 2 * 2 + 1]);
      else
        p[s] = make_float2(g[2 * s % GROUPS], g[(2 * s + 1) % GROUPS]);
    }
  }
  // The sums of the pairs put to their degrees, out[FROM + l].
  template <int FROM, int N>
  __device__ __forceinline__ void by_degree(const float2 (&p)[PAIRS], float (&out)[N]) const {
    if constexpr (L == 0) {
      float2 t = p[0];
#pragma unroll
      for (int s = 1; s < PAIRS; ++s) t = __fadd2_rn(t, p[s]);
      out[FROM] = t.x + t.y;
    } else {
      float g[GROUPS];
      if constexpr (V == 1) {
        g[0] = p[0].x + p[0].y;
      } else if constexpr (FOURS) {
#pragma unroll
        for (int k = 0; k < GROUPS; k += 2) {
          g[k] = p[k].x;
          g[k + 1] = p[k].y + (p[k + 1].x + p[k + 1].y);
        }
      } else {
#pragma unroll
        for (int k = 0; k < GROUPS; ++k) g[k] = k % 2 ? p[k / 2].y : p[k / 2].x;
      }
#pragma unroll
      for (int l = 0; l <= L; ++l) {
        float t = cls[0] == l ? g[0] : 0.0f;
#pragma unroll
        for (int k = 1; k < GROUPS; ++k) t += cls[k] == l ? g[k] : 0.0f;
        out[FROM + l] = t;
      }
    }
  }
};

// ---------------------------------------------------------------- dropout
// Which of a lane's values the dropout keeps.  V = 1: the group forms the keep
// bits of its row together, eight columns a byte, in shared memory (form();
// the caller waits until it is visible).  V > 1: each lane draws for its own
// vectors; where a unit is at least as wide as a vector, a vector touches two
// units at most, which are found once (meta: the first unit, and how many of
// the vector's values it has).
constexpr int kKeepBytes = kMaxRowThreads * 16 / 8 + kRowThreads;  // bits of a CTA's rows, a byte each begun

template <int L, int V, int NV>
struct Keeps {
  uint32_t meta[NV];
  uint8_t* bits;  // V = 1: of this row group, two halves taken in turn
  int bytes;
  int half;
  __device__ __forceinline__ Keeps(const Dropper& d, const Slots<L, V, NV>& at, const RowShape& sh, int cols,
                                   uint8_t* smem) {
    if constexpr (V == 1) {
      bytes = (cols + 7) / 8;
      bits = smem + (threadIdx.x / sh.lanes) * bytes;
      half = 0;
    } else {
      const uint32_t group = L ? (uint32_t)at.K : (uint32_t)d.group;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t unit = at.col[j] / group, left = group - (at.col[j] - unit * group);
        meta[j] = unit << 4 | (left < V ? left : V);
      }
    }
  }
  // V = 1: the bits of a row, by all lanes of its group.
  __device__ __forceinline__ void form(const Dropper& d, const Slots<L, V, NV>& at, const RowShape& sh, int row) {
    if constexpr (V == 1) {
      half ^= 1;
      for (int y = at.lane; y < bytes; y += sh.lanes) bits[half * kKeepBytes + y] = (uint8_t)d.keep_bits(row, 8 * y, 8);
    }
  }
  // The values of a row, p, with the dropout applied.
  __device__ __forceinline__ void apply(const Dropper& d, const Slots<L, V, NV>& at, int row,
                                        float2 (&p)[NV * V / 2]) const {
    if constexpr (V == 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float& f = j & 1 ? p[j / 2].y : p[j / 2].x;
        const bool keep = at.has[j] && (bits[half * kKeepBytes + (at.col[j] >> 3)] >> (at.col[j] & 7)) & 1;
        f = keep ? f * d.scale : 0.0f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float2* f = p + j * (V / 2);
        if (L == 0 && d.group == 1) {
          const uint4 w = d.block(row, at.col[j] >> 3);
          const bool upper = V == 4 && (at.col[j] & 4);
          const uint32_t words[4] = {upper ? w.z : w.x, upper ? w.w : w.y, w.z, w.w};
#pragma unroll
          for (int s = 0; s < V / 2; ++s) {
            f[s].x = words[s] << 16 > d.bound ? f[s].x * d.scale : 0.0f;
            f[s].y = words[s] > d.bound ? f[s].y * d.scale : 0.0f;
          }
        } else if (L > 0 || d.group >= V) {
          const uint32_t unit = meta[j] >> 4;
          const int n = meta[j] & 15;
          uint4 w = d.block(row, unit >> 3);
          const bool k0 = d.keeps(w, unit);
          bool k1 = k0;
          if ((L == 0 || at.K % V) && n < V) {
            if ((unit & 7) == 7) w = d.block(row, (unit + 1) >> 3);
            k1 = d.keeps(w, unit + 1);
          }
#pragma unroll
          for (int s = 0; s < V / 2; ++s) {
            f[s].x = (2 * s < n ? k0 : k1) ? f[s].x * d.scale : 0.0f;
            f[s].y = (2 * s + 1 < n ? k0 : k1) ? f[s].y * d.scale : 0.0f;
          }
        } else {
          const uint32_t keep = d.keep_bits(row, at.col[j], V);
#pragma unroll
          for (int s = 0; s < V / 2; ++s) {
            f[s].x = (keep >> (2 * s)) & 1 ? f[s].x * d.scale : 0.0f;
            f[s].y = (keep >> (2 * s + 1)) & 1 ? f[s].y * d.scale : 0.0f;
          }
        }
      }
    }
  }
};

// ---------------------------------------------------------------- sums
// Sums N values over the lanes of each group, in a fixed order, and leaves
// them spread over the lanes: value n is then fetched by a shuffle.  For N > 2
// the values are halved as the lanes are (each lane passes on the half that it
// does not keep), so that N values take about as many shuffles as log2 G + N.
// Groups of several warps exchange their warps' sums through red (two halves,
// taken in turn, so that one barrier per sum is enough; every thread of the
// CTA takes part).  N = 2 needs groups of at least 2 lanes, N > 2 of 8.
template <int N>
struct GroupSum {
  static constexpr int P = N <= 1 ? 1 : N <= 2 ? 2 : N <= 4 ? 4 : 8;  // N rounded up to a power of two
  static constexpr int kRed = 2 * (kMaxRowThreads / 32) * P;          // floats of red
  int lanes, warps, first;  // of the group: lanes, warps, its first warp
  int base;                 // of the group within the warp
  float* red;
  int half;
  float val;  // after sum(): this lane's value
  __device__ __forceinline__ GroupSum(int lanes_, float* red_) : lanes(lanes_), red(red_), half(0), val(0.0f) {
    warps = lanes_ >> 5;
    first = warps > 1 ? (int)(threadIdx.x >> 5) / warps * warps : 0;
    base = lanes_ < 32 ? (int)(threadIdx.x & 31) / lanes_ * lanes_ : 0;
  }
  // The lane that holds value n.
  __device__ __forceinline__ int source(int n) const {
    if (N == 1) return threadIdx.x & 31;
    if (lanes > 32) return n;
    if (N == 2) return base + n * (lanes >> 1);
    int lane = base;
    if (P == 8) lane += (n >> 2 & 1) * (lanes >> 1) + (n >> 1 & 1) * (lanes >> 2) + (n & 1) * (lanes >> 3);
    if (P == 4) lane += (n >> 1 & 1) * (lanes >> 1) + (n & 1) * (lanes >> 2);
    return lane;
  }
  __device__ __forceinline__ float fetch(int source_lane) const {
    return N == 1 ? val : __shfl_sync(0xffffffffu, val, source_lane);
  }
  __device__ __forceinline__ void operator()(const float (&v)[N]) {
    const int in_warp = lanes < 32 ? lanes : 32;
    int o = in_warp >> 1;
    float x[P];
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = i < N ? v[i] : 0.0f;
    int mine = 0;  // the value of this lane
#pragma unroll
    for (int n = P / 2; n > 0; n >>= 1) {
      const bool up = threadIdx.x & o;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float send = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
        x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
      mine += up ? n : 0;
      o >>= 1;
    }
    for (; o > 0; o >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
    val = x[0];
    if (lanes <= 32) return;
    const int lane = threadIdx.x & 31;
    float* buf = red + half * (kRed / 2);
    if (lane % (32 / P) == 0) buf[(threadIdx.x >> 5) * P + mine] = val;
    __syncthreads();
    float t = 0.0f;
    for (int k = lane / P; k < warps; k += 32 / P) t += buf[(first + k) * P + lane % P];
    for (o = P; o < 32 && o < warps * P; o <<= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    val = N == 1 ? __shfl_sync(0xffffffffu, t, 0) : t;
    half ^= 1;
  }
};

// ---------------------------------------------------------------- forward
// One pass: each value is loaded once, kept in registers through the mean and
// the centred squares, and stored once.  The next row's vectors are loaded
// before the sums of the current one are formed.  FUSED: with a residual sum
// or dropout in front.
template <typename T, int L, int V, int NV, bool FUSED>
__global__ void __launch_bounds__(kMaxRowThreads) k_norm_rows(NormArgs a, RowShape sh) {
  using S = Slots<L, V, NV>;
  constexpr int P = NV * V / 2, PV = S::PAIRS, NS = L + 1;
  constexpr bool EACH = L == 0 || V == 1;  // a bias per value; else one per vector, which has at most one degree 0
  __shared__ float red1[GroupSum<1>::kRed], red2[GroupSum<NS>::kRed];
  __shared__ uint8_t bits[FUSED && V == 1 ? 2 * kKeepBytes : 1];
  const S at(sh, a.cols);
  GroupSum<1> sum1(sh.lanes, red1);
  GroupSum<NS> sum2(sh.lanes, red2);
  const Dropper drop(a.drop);
  Keeps<L, V, NV> keeps(drop, at, sh, a.cols, bits);
  float2 w[P], b[EACH ? P : NV], m[V == 1 ? P : NV];  // m: -1 where a value is one of the row's, else 0
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (int)(at.col[j] + i) / S::K;
      int l = 0;
      if (L) {
        l = at.cls[S::GROUPS == 1 ? 0 : S::FOURS ? i / 4 * 2 + (i % 4 > 0) : i];
      }
      const float wi = at.has[j] && a.w ? a.w[l * a.C + c] : 1.0f;
      const float bi = at.has[j] && a.b && l == 0 ? a.b[c] : 0.0f;
      const float mi = at.has[j] ? -1.0f : 0.0f;
      const int e = j * V + i;
      (e & 1 ? w[e / 2].y : w[e / 2].x) = wi;
      if (EACH)
        (e & 1 ? b[e / 2].y : b[e / 2].x) = bi;
      else if (i == 0 || l == 0)
        b[EACH ? 0 : j] = both(bi);
      if (V == 1)
        (e & 1 ? m[e / 2].y : m[e / 2].x) = mi;
      else
        m[V == 1 ? 0 : j] = both(mi);
    }
  }
  const float inv = 1.0f / (float)a.C;
  float scale[S::GROUPS];
  int from[S::GROUPS];
#pragma unroll
  for (int g = 0; g < S::GROUPS; ++g) {
    scale[g] = inv / (float)(2 * at.cls[g] + 1);
    from[g] = sum2.source(at.cls[g]);
  }
  const int stride = gridDim.x * sh.groups;
  int row = blockIdx.x * sh.groups + threadIdx.x / sh.lanes;
  const T* x = static_cast<const T*>(a.x) + (long long)row * a.x_ld;
  const T* r = static_cast<const T*>(a.r) + (long long)row * a.r_ld;
  Pack<T, V> nx[NV], nr[FUSED ? NV : 1];
  auto fetch = [&](bool live) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (at.has[j] && live)
        nx[j].load(x + at.col[j]);
      else
        nx[j].zero();
      if (FUSED) {
        if (at.has[j] && live && a.r)
          nr[FUSED ? j : 0].load(r + at.col[j]);
        else
          nr[FUSED ? j : 0].zero();
      }
    }
  };
  fetch(row < a.rows);
  if (FUSED && V == 1 && drop.on) {
    keeps.form(drop, at, sh, row);
    __syncthreads();
  }
  // the same number of rounds for every group of the CTA
  for (int base = blockIdx.x * sh.groups; base < a.rows; base += stride, row += stride) {
    float2 v[P], acc[PV];
    get_pairs<T, V, NV>(nx, v);
    if constexpr (FUSED) {
      if (drop.on) keeps.apply(drop, at, row, v);
      if (a.r) {
        float2 f[P];
        get_pairs<T, V, NV>(nr, f);
#pragma unroll
        for (int p = 0; p < P; ++p) v[p] = __fadd2_rn(v[p], f[p]);
      }
    }
    x += stride * a.x_ld;
    r += stride * a.r_ld;
    fetch(row + stride < a.rows);
    if (FUSED && V == 1 && drop.on) {  // the next row's, seen after a barrier of this row's sums
      keeps.form(drop, at, sh, row + stride);
      if (sh.lanes <= 32) __syncwarp();
    }
    const bool live = row < a.rows;
    const long long out = (long long)row * a.cols;
    if (FUSED && a.s && live) put_pairs<T, V, NV>(static_cast<T*>(a.s) + out, at.col, at.has, v);
    // the mean of degree 0
#pragma unroll
    for (int s = 0; s < PV; ++s) {
      acc[s] = v[s];
#pragma unroll
      for (int p = s + PV; p < P; p += PV) acc[s] = __fadd2_rn(acc[s], v[p]);
    }
    float part[1] = {0.0f};
#pragma unroll
    for (int s = 0; s < PV; ++s) {
      if (!S::may0(s)) continue;
      if (L) acc[s] = __fmul2_rn(acc[s], at.first[s]);
      part[0] += acc[s].x + acc[s].y;
    }
    sum1(part);
    const float mean = sum1.fetch(0) * inv;
    // centred; what lies outside the row stays 0
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if (!S::may0(p % PV)) continue;
      float2 mu = both(mean);
      if (L) mu = __fmul2_rn(mu, at.first[p % PV]);
      v[p] = __ffma2_rn(mu, m[V == 1 ? p : p / PV], v[p]);
    }
#pragma unroll
    for (int s = 0; s < PV; ++s) {
      acc[s] = __fmul2_rn(v[s], v[s]);
#pragma unroll
      for (int p = s + PV; p < P; p += PV) acc[s] = __ffma2_rn(v[p], v[p], acc[s]);
    }
    float sq[NS];
    at.template by_degree<0>(acc, sq);
    sum2(sq);
    float q[S::GROUPS];
#pragma unroll
    for (int g = 0; g < S::GROUPS; ++g) q[g] = rsqrtf(sum2.fetch(from[g]) * scale[g] + a.eps);
    if (a.stats) {
      float* st = a.stats + (long long)row * (L + 2);
      const int l = at.lane < L ? at.lane : L;
      const float ql = L ? rsqrtf(sum2.fetch(sum2.source(l)) * (inv / (float)(2 * l + 1)) + a.eps) : q[0];
      if (live && at.lane <= L) st[1 + l] = ql;
      if (live && at.lane == 0) st[0] = mean;
    }
    if (!live || !a.y) continue;
    float2 qs[PV];
    S::spread(q, qs);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const float2 h = __fmul2_rn(v[p], qs[p % PV]);
      if (EACH)
        v[p] = __ffma2_rn(h, w[p], b[EACH ? p : 0]);
      else if (S::may0(p % PV))
        v[p] = __ffma2_rn(h, w[p], __fmul2_rn(b[EACH ? 0 : p / PV], at.first[p % PV]));
      else
        v[p] = __fmul2_rn(h, w[p]);
    }
    put_pairs<T, V, NV>(static_cast<T*>(a.y) + out, at.col, at.has, v);
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
  using S = Slots<L, V, NV>;
  constexpr int P = NV * V / 2, PV = S::PAIRS, NS = L + 2;
  constexpr bool EACH = L == 0 || V == 1;  // db per value; else per vector, which has at most one degree 0
  __shared__ float red[GroupSum<NS>::kRed];
  __shared__ uint8_t bits[FUSED && V == 1 ? 2 * kKeepBytes : 1];
  extern __shared__ float colsum[];  // [cols] g h, then [C] g
  const S at(sh, a.cols);
  GroupSum<NS> sum(sh.lanes, red);
  const Dropper drop(a.drop);
  Keeps<L, V, NV> keeps(drop, at, sh, a.cols, bits);
  float2 w[P], dw[P], db[EACH ? P : NV];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (int)(at.col[j] + i) / S::K;
      int l = 0;
      if (L) l = at.cls[S::GROUPS == 1 ? 0 : S::FOURS ? i / 4 * 2 + (i % 4 > 0) : i];
      const float wi = at.has[j] && a.w ? a.w[l * a.C + c] : 1.0f;
      const int e = j * V + i;
      (e & 1 ? w[e / 2].y : w[e / 2].x) = wi;
    }
  }
#pragma unroll
  for (int p = 0; p < P; ++p) dw[p] = both(0.0f);
#pragma unroll
  for (int p = 0; p < (EACH ? P : NV); ++p) db[p] = both(0.0f);
  const float inv = 1.0f / (float)a.C;
  float scale[S::GROUPS];
  int from[S::GROUPS];
#pragma unroll
  for (int g = 0; g < S::GROUPS; ++g) {
    scale[g] = -inv / (float)(2 * at.cls[g] + 1);
    from[g] = sum.source(1 + at.cls[g]);
  }
  const int from0 = sum.source(0);
  const int stride = gridDim.x * sh.groups;
  int row = blockIdx.x * sh.groups + threadIdx.x / sh.lanes;
  const T* x = static_cast<const T*>(a.x) + (long long)row * a.x_ld;
  const T* g = static_cast<const T*>(a.g) + (long long)row * a.g_ld;
  const T* r = static_cast<const T*>(a.r) + (long long)row * a.r_ld;
  const float* st = a.stats + (long long)row * (L + 2);
  Pack<T, V> nx[NV], ng[NV];
  float nmean, nq[S::GROUPS];
  auto fetch = [&](bool live) {
    nmean = live ? st[0] : 0.0f;
#pragma unroll
    for (int k = 0; k < S::GROUPS; ++k) nq[k] = live ? st[1 + at.cls[k]] : 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (at.has[j] && live) {
        nx[j].load(x + at.col[j]);
        ng[j].load(g + at.col[j]);
      } else {
        nx[j].zero();
        ng[j].zero();
      }
    }
  };
  fetch(row < a.rows);
  for (int base = blockIdx.x * sh.groups; base < a.rows; base += stride, row += stride) {
    const bool live = row < a.rows;
    float2 h[P], av[P], qs[PV];
    Pack<T, V> cr[FUSED ? NV : 1];
    float q[S::GROUPS];
    get_pairs<T, V, NV>(nx, h);
    get_pairs<T, V, NV>(ng, av);
#pragma unroll
    for (int k = 0; k < S::GROUPS; ++k) q[k] = nq[k];
    const float2 mu = both(-nmean);
    if constexpr (FUSED) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (at.has[j] && live && a.r)
          cr[j].load(r + at.col[j]);
        else
          cr[j].zero();
      }
    }
    x += stride * a.x_ld;
    g += stride * a.g_ld;
    r += stride * a.r_ld;
    st += (long long)stride * (L + 2);
    fetch(row + stride < a.rows);
    if (FUSED && V == 1 && drop.on) {  // seen after the barrier of this row's sums
      keeps.form(drop, at, sh, row);
      if (sh.lanes <= 32) __syncwarp();
    }
    S::spread(q, qs);
    float2 sa[PV], sah[PV];
#pragma unroll
    for (int s = 0; s < PV; ++s) sa[s] = sah[s] = both(0.0f);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int s = p % PV;
      if (L == 0)
        h[p] = __fadd2_rn(h[p], mu);
      else if (S::may0(s))
        h[p] = __ffma2_rn(mu, at.first[s], h[p]);
      h[p] = __fmul2_rn(h[p], qs[s]);
      dw[p] = __ffma2_rn(av[p], h[p], dw[p]);
      if (EACH)
        db[EACH ? p : 0] = __fadd2_rn(db[EACH ? p : 0], av[p]);
      else if (S::may0(s))
        db[EACH ? 0 : p / PV] = __ffma2_rn(av[p], at.first[s], db[EACH ? 0 : p / PV]);
      av[p] = __fmul2_rn(av[p], w[p]);
      if (S::may0(s)) sa[s] = __fadd2_rn(sa[s], av[p]);
      sah[s] = __ffma2_rn(av[p], h[p], sah[s]);
    }
    float tot[NS];
    tot[0] = 0.0f;
#pragma unroll
    for (int s = 0; s < PV; ++s) {
      if (!S::may0(s)) continue;
      if (L) sa[s] = __fmul2_rn(sa[s], at.first[s]);
      tot[0] += sa[s].x + sa[s].y;
    }
    at.template by_degree<1>(sah, tot);
    sum(tot);
    // r = q a - (q mean(a h)) h - q mean(a) for degree 0
    const float m0 = sum.fetch(from0) * -inv;
    float c[S::GROUPS];
#pragma unroll
    for (int k = 0; k < S::GROUPS; ++k) c[k] = sum.fetch(from[k]) * scale[k] * q[k];
    if (!live) continue;
    float2 cs[PV], c0[PV];
    S::spread(c, cs);
#pragma unroll
    for (int s = 0; s < PV; ++s) c0[s] = L ? __fmul2_rn(__fmul2_rn(qs[s], both(m0)), at.first[s]) : __fmul2_rn(qs[s], both(m0));
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int s = p % PV;
      const float2 t = S::may0(s) ? __ffma2_rn(av[p], qs[s], c0[s]) : __fmul2_rn(av[p], qs[s]);
      av[p] = __ffma2_rn(h[p], cs[s], t);
    }
    const long long out = (long long)row * a.cols;
    if constexpr (FUSED) {
      if (a.r) {
        get_pairs<T, V, NV>(cr, h);
#pragma unroll
        for (int p = 0; p < P; ++p) av[p] = __fadd2_rn(av[p], h[p]);
      }
      if (a.gr) put_pairs<T, V, NV>(static_cast<T*>(a.gr) + out, at.col, at.has, av);
      if (a.gx) {
        if (drop.on) keeps.apply(drop, at, row, av);
        put_pairs<T, V, NV>(static_cast<T*>(a.gx) + out, at.col, at.has, av);
      }
    } else {
      T* dst = static_cast<T*>(a.gx ? a.gx : a.gr);
      if (dst) put_pairs<T, V, NV>(dst + out, at.col, at.has, av);
    }
  }
  if (!a.gw && !a.gb) return;
  // the CTA's sums: the groups of a warp by shuffles, the warps (or the
  // groups of several warps) in turn
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (o >= sh.lanes) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        dw[p].x += __shfl_xor_sync(0xffffffffu, dw[p].x, o);
        dw[p].y += __shfl_xor_sync(0xffffffffu, dw[p].y, o);
      }
#pragma unroll
      for (int p = 0; p < (EACH ? P : NV); ++p) {
        db[p].x += __shfl_xor_sync(0xffffffffu, db[p].x, o);
        db[p].y += __shfl_xor_sync(0xffffffffu, db[p].y, o);
      }
    }
  }
  const int unit = sh.lanes <= 32 ? 32 : sh.lanes;  // threads that add together
  const int units = blockDim.x / unit, mine = threadIdx.x / unit;
  const bool speaks = (int)(threadIdx.x % unit) < sh.lanes;
  for (int u = 0; u < units; ++u) {
    if (u == mine && speaks) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!at.has[j]) continue;
#pragma unroll
        for (int i = 0; i < V; ++i) {
          const int e = j * V + i, col = (int)at.col[j] + i;
          const float t = e & 1 ? dw[e / 2].y : dw[e / 2].x;
          colsum[col] = u ? colsum[col] + t : t;
          if (EACH && col % S::K == 0) {
            const float f = e & 1 ? db[EACH ? e / 2 : 0].y : db[EACH ? e / 2 : 0].x;
            float* d = colsum + a.cols + col / S::K;
            *d = u ? *d + f : f;
          }
        }
        if (!EACH) {
          const int c = (int)(at.col[j] + V - 1) / S::K;  // the channel that begins in the vector, if one does
          if (c * S::K >= (int)at.col[j]) {
            const float f = db[EACH ? 0 : j].x + db[EACH ? 0 : j].y;
            float* d = colsum + a.cols + c;
            *d = u ? *d + f : f;
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
      for (int k = l * l; k < (l + 1) * (l + 1); ++k) t += colsum[c * S::K + k];
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
// Lanes for a row of cols values in vectors of V, NV per lane, at least
// min_lanes (a power of two).
inline RowShape row_shape(int cols, int K, int V, int NV, int min_lanes) {
  int period = 1;  // K / gcd(K, V)
  while (period * V % K) ++period;
  const int vectors = cols / V;
  RowShape sh;
  sh.active = ((vectors + NV - 1) / NV + period - 1) / period * period;
  if (sh.active <= 32) {
    sh.lanes = min_lanes;
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
  constexpr int least = L ? 8 : BACKWARD ? 2 : 1;  // what GroupSum needs
  const RowShape s8 = row_shape(a.cols, K, V, N8, least), s16 = row_shape(a.cols, K, V, N16, least);
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
