// Row norms and dropout between message layers (sm_103a): arguments, the
// dropout's generator and the kernels that take any shape.
//
// A row holds C channels of K = (L+1)^2 values, component k = l*l + l + m of
// degree l.  Each degree of a row is normalised by itself:
//   s = residual + drop(x)
//   l = 0:  mu = mean_c s,  q_0 = (mean_c (s - mu)^2 + eps)^-1/2,  h = (s - mu) q_0
//   l > 0:  q_l = (mean_{c,m} s^2 + eps)^-1/2,                     h = s q_l
//   y = h w[l,c]  (+ b[c] for l = 0)
// With L = 0 (K = 1) that is the layer norm of a row of C values, so one
// template serves both: layer norm at L = 0, the norm by degree at L = 3..6.
// Backward, with a = g w (g = dL/dy):
//   r = dL/ds + q_l (a - h mean(a h) - [l = 0] mean(a)),  dL/dx = drop'(r)
//   dw[l,c] = sum_rows sum_m g h,   db[c] = sum_rows g  (l = 0)
// Statistics and sums are fp32; bf16 is only the storage of x, s, y and of
// their gradients, rounded once on the store.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace eqmp {

// ---------------------------------------------------------------- dropout
// Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as
// easy as 1, 2, 3", SC 2011): counter (c0, c1, c2, c3), key (k0, k1).  One
// block of four words gives eight 16-bit draws; 16 bits resolve p to 1.5e-5,
// halve the generator's work per element and keep the mean exact, because the
// scale is that of the resolved rate.
__device__ __forceinline__ uint4 philox(uint32_t c0, uint32_t c1, uint32_t c2, uint32_t c3, uint32_t k0,
                                        uint32_t k1) {
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const unsigned long long a = (unsigned long long)c0 * 0xD2511F53u, b = (unsigned long long)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c1 = (uint32_t)b;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// The first three rounds take the block index (c0) and the row (c1) apart: of
// their six products two are constant for a column block over all rows, one
// for a row over all blocks, one for a call.  A kernel whose lanes keep their
// columns forms those once and has 15 products a block left of 20.
struct PhiloxRow {
  uint32_t hi, lo;  // of the second round's first product
};
struct PhiloxBlock {
  uint32_t e0, e1, e2, e3;
};
constexpr uint32_t kPhiloxM0 = 0xD2511F53u, kPhiloxM1 = 0xCD9E8D57u, kPhiloxW0 = 0x9E3779B9u, kPhiloxW1 = 0xBB67AE85u;

struct DropArgs {
  unsigned long long seed, offset;
  const unsigned long long* step;  // device, added to offset; may be NULL
  uint32_t threshold;              // 0 (off) .. 65536 (nothing kept)
  float scale;                     // 65536 / (65536 - threshold); 0 when nothing is kept
  int group;                       // consecutive columns that share a draw
};

// The draws of one call: unit u of row r is word (u%8)/2 of block u/8, its
// low half for even u.  A half h of a word is compared in the upper half of a
// register, with what lies below it left standing: h >= t is
// (h, anything) > (t, 0) - 1, and t = 65536 gives a bound that nothing passes.
struct Dropper {
  uint32_t k0, k1, o0, o1, bound;
  float scale;
  int group;
  bool on;
  __device__ __forceinline__ explicit Dropper(const DropArgs& d) {
    on = d.threshold > 0;
    const unsigned long long off = d.offset + (d.step ? *d.step : 0ull);
    k0 = (uint32_t)d.seed;
    k1 = (uint32_t)(d.seed >> 32);
    o0 = (uint32_t)off;
    o1 = (uint32_t)(off >> 32);
    bound = (uint32_t)(((unsigned long long)d.threshold << 16) - 1);
    scale = d.scale;
    group = d.group;
  }
  __device__ __forceinline__ uint4 block(uint32_t row, uint32_t blk) const { return philox(blk, row, o0, o1, k0, k1); }
  __device__ __forceinline__ PhiloxBlock of_block(uint32_t blk) const {
    const uint32_t c2 = __umulhi(blk, kPhiloxM0) ^ o1 ^ k1, lo = o0 * kPhiloxM1;
    const uint32_t c0 = __umulhi(c2, kPhiloxM1) ^ lo ^ (k0 + kPhiloxW0);
    PhiloxBlock b;
    b.e0 = blk * kPhiloxM0 ^ (k1 + kPhiloxW1);
    b.e1 = c2 * kPhiloxM1 ^ (k0 + 2 * kPhiloxW0);
    b.e2 = __umulhi(c0, kPhiloxM0) ^ (k1 + 2 * kPhiloxW1);
    b.e3 = c0 * kPhiloxM0;
    return b;
  }
  __device__ __forceinline__ PhiloxRow of_row(uint32_t row) const {
    const uint32_t c0 = __umulhi(o0, kPhiloxM1) ^ row ^ k0;
    return PhiloxRow{__umulhi(c0, kPhiloxM0), c0 * kPhiloxM0};
  }
  // block(row, blk) from the two.
  __device__ __forceinline__ uint4 block(const PhiloxRow& r, const PhiloxBlock& b) const {
    unsigned long long m = (unsigned long long)(r.hi ^ b.e0) * kPhiloxM1;
    uint32_t c0 = (uint32_t)(m >> 32) ^ b.e1, c1 = (uint32_t)m, c2 = b.e2 ^ r.lo, c3 = b.e3;
#pragma unroll
    for (uint32_t i = 3; i < 10; ++i) {
      const unsigned long long a = (unsigned long long)c0 * kPhiloxM0;
      m = (unsigned long long)c2 * kPhiloxM1;
      c0 = (uint32_t)(m >> 32) ^ c1 ^ (k0 + i * kPhiloxW0);
      c1 = (uint32_t)m;
      c2 = (uint32_t)(a >> 32) ^ c3 ^ (k1 + i * kPhiloxW1);
      c3 = (uint32_t)a;
    }
    return make_uint4(c0, c1, c2, c3);
  }
  __device__ __forceinline__ bool keeps(const uint4& w, uint32_t unit) const {
    const uint32_t a = (unit & 4) ? w.z : w.x, b = (unit & 4) ? w.w : w.y;
    const uint32_t v = (unit & 2) ? b : a;
    return ((unit & 1) ? v : v << 16) > bound;
  }
  // A dropped value is 0 whatever it held, a NaN or an infinity included.
  __device__ __forceinline__ float apply(float v, uint32_t row, int col) const {
    const uint32_t unit = (uint32_t)col / (uint32_t)group;
    return keeps(block(row, unit >> 3), unit) ? v * scale : 0.0f;
  }
  // Bit i: unit i of the block is kept.
  __device__ __forceinline__ uint32_t keep_bits(const uint4& w) const {
    uint32_t keep = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) keep |= (uint32_t)keeps(w, i) << i;
    return keep;
  }
};

// ---------------------------------------------------------------- storage
template <typename T>
__device__ __forceinline__ float load1(const T* p);
template <>
__device__ __forceinline__ float load1<float>(const float* p) {
  return *p;
}
template <>
__device__ __forceinline__ float load1<__nv_bfloat16>(const __nv_bfloat16* p) {
  return __bfloat162float(*p);
}
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

struct NormArgs {
  const void* x;        // forward: x; backward: the stored s
  const void* r;        // forward: residual; backward: dL/ds of the residual stream; may be NULL
  const void* g;        // backward: dL/dy
  void *s, *y;          // forward outputs
  void *gr, *gx;        // backward outputs: dL/ds, dL/dx
  float* stats;         // [rows][L+2]: mean, then q_l; written forward, read backward
  const float *w, *b;   // [L+1][C], [C]; NULL: 1 and 0
  float *gw, *gb;
  float* part;          // partial dw, db: [parts][(L+2)*C]
  long long x_ld, r_ld, g_ld;  // row strides of the inputs, in elements (outputs are packed)
  int rows, cols, C;
  int parts;
  float eps;
  DropArgs drop;
};

constexpr int kWideThreads = 256;

__device__ __forceinline__ int degree_of(int k) {
  int l = 0;
  while ((l + 1) * (l + 1) <= k) ++l;
  return l;
}

// Sums NV values over the CTA; every thread gets the totals.  The order is
// fixed: lanes by halving distance, then the warps in turn.
template <int NV>
__device__ __forceinline__ void cta_sum(float (&v)[NV], float* red) {
  const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  __syncthreads();  // the previous sums have been read
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < NV; ++i) red[warp * NV + i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float t = red[i];
    for (int k = 1; k < warps; ++k) t += red[k * NV + i];
    v[i] = t;
  }
}

// Any shape, forward: one CTA per row, which reads the row three times.  Takes
// the rows that are too wide for the registers of one CTA: over 8192 values, by
// degree over 8192, 8000, 8064 and 7840 at l_max 3 to 6 (whole periods of lanes),
// up to 14 less where rows begin anywhere.  1800 x 16384 fp32 147 us, 24 % of the
// measured copy rate, bound by its single values.
template <typename T, int L>
__global__ void __launch_bounds__(kWideThreads) k_norm_wide(NormArgs a) {
  constexpr int K = (L + 1) * (L + 1);
  __shared__ float red[(kWideThreads / 32) * (L + 1)];
  const Dropper drop(a.drop);
  const bool dropping = drop.on;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + (long long)row * a.x_ld;
    const T* r = a.r ? static_cast<const T*>(a.r) + (long long)row * a.r_ld : nullptr;
    const long long out = (long long)row * a.cols;
    auto value = [&](int col) {
      float v = load1(x + col);
      if (dropping) v = drop.apply(v, row, col);
      return r ? v + load1(r + col) : v;
    };
    float mean[1] = {0.0f};
    for (int col = threadIdx.x; col < a.cols; col += blockDim.x) {
      const float v = value(col);
      if (a.s) store1(static_cast<T*>(a.s) + out + col, v);
      if (col % K == 0) mean[0] += v;
    }
    cta_sum(mean, red);
    mean[0] /= (float)a.C;
    float q[L + 1];
#pragma unroll
    for (int l = 0; l <= L; ++l) q[l] = 0.0f;
    for (int col = threadIdx.x; col < a.cols; col += blockDim.x) {
      const int l = L ? degree_of(col % K) : 0;
      const float v = l ? value(col) : value(col) - mean[0];
#pragma unroll
      for (int k = 0; k <= L; ++k) q[k] += k == l ? v * v : 0.0f;
    }
    cta_sum(q, red);
#pragma unroll
    for (int l = 0; l <= L; ++l) q[l] = 1.0f / sqrtf(q[l] / ((float)(2 * l + 1) * (float)a.C) + a.eps);
    if (a.stats && threadIdx.x == 0) {
      float* st = a.stats + (long long)row * (L + 2);
      st[0] = mean[0];
#pragma unroll
      for (int l = 0; l <= L; ++l) st[1 + l] = q[l];
    }
    if (!a.y) continue;
    for (int col = threadIdx.x; col < a.cols; col += blockDim.x) {
      const int l = L ? degree_of(col % K) : 0, c = col / K;
      float ql = q[0];
#pragma unroll
      for (int k = 1; k <= L; ++k) ql = k == l ? q[k] : ql;
      float h = (l ? value(col) : value(col) - mean[0]) * ql;
      if (a.w) h *= a.w[(long long)l * a.C + c];
      if (a.b && l == 0) h += a.b[c];
      store1(static_cast<T*>(a.y) + out + col, h);
    }
  }
}

// Any shape, backward: dL/ds and dL/dx, one CTA per row.
template <typename T, int L>
__global__ void __launch_bounds__(kWideThreads) k_norm_bwd_wide(NormArgs a) {
  constexpr int K = (L + 1) * (L + 1);
  __shared__ float red[(kWideThreads / 32) * (L + 2)];
  const Dropper drop(a.drop);
  const bool dropping = drop.on;
  for (int row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + (long long)row * a.x_ld;
    const T* g = static_cast<const T*>(a.g) + (long long)row * a.g_ld;
    const T* r = a.r ? static_cast<const T*>(a.r) + (long long)row * a.r_ld : nullptr;
    const float* st = a.stats + (long long)row * (L + 2);
    const long long out = (long long)row * a.cols;
    float sum[L + 2];
#pragma unroll
    for (int l = 0; l < L + 2; ++l) sum[l] = 0.0f;
    auto hat = [&](int col, int l) { return (l ? load1(x + col) : load1(x + col) - st[0]) * st[1 + l]; };
    auto weighted = [&](int col, int l) {
      const float v = load1(g + col);
      return a.w ? v * a.w[(long long)l * a.C + col / K] : v;
    };
    for (int col = threadIdx.x; col < a.cols; col += blockDim.x) {
      const int l = L ? degree_of(col % K) : 0;
      const float v = weighted(col, l), vh = v * hat(col, l);
      sum[0] += l ? 0.0f : v;
#pragma unroll
      for (int k = 0; k <= L; ++k) sum[1 + k] += k == l ? vh : 0.0f;
    }
    cta_sum(sum, red);
    sum[0] /= (float)a.C;
#pragma unroll
    for (int l = 0; l <= L; ++l) sum[1 + l] /= (float)(2 * l + 1) * (float)a.C;
    for (int col = threadIdx.x; col < a.cols; col += blockDim.x) {
      const int l = L ? degree_of(col % K) : 0;
      float m = sum[1];
#pragma unroll
      for (int k = 1; k <= L; ++k) m = k == l ? sum[1 + k] : m;
      float v = (weighted(col, l) - hat(col, l) * m - (l ? 0.0f : sum[0])) * st[1 + l];
      if (r) v += load1(r + col);
      if (a.gr) store1(static_cast<T*>(a.gr) + out + col, v);
      if (a.gx) store1(static_cast<T*>(a.gx) + out + col, dropping ? drop.apply(v, row, col) : v);
    }
  }
}

// Any shape, dw and db: partial sums over a range of rows for 32 channels.
// Part p covers the rows [p rows / parts, (p+1) rows / parts).
constexpr int kWideSumX = 32, kWideSumY = 8;

template <typename T, int L>
__global__ void __launch_bounds__(kWideSumX * kWideSumY) k_norm_bwd_wide_w(NormArgs a) {
  constexpr int K = (L + 1) * (L + 1);
  __shared__ float red[kWideSumY][kWideSumX];
  const int p = blockIdx.y, c = blockIdx.x * kWideSumX + threadIdx.x;
  const int row0 = (int)((long long)a.rows * p / a.parts), row1 = (int)((long long)a.rows * (p + 1) / a.parts);
  float sum[L + 2];
#pragma unroll
  for (int l = 0; l < L + 2; ++l) sum[l] = 0.0f;
  if (c < a.C) {
    for (int row = row0 + threadIdx.y; row < row1; row += kWideSumY) {
      const T* x = static_cast<const T*>(a.x) + (long long)row * a.x_ld + (long long)c * K;
      const T* g = static_cast<const T*>(a.g) + (long long)row * a.g_ld + (long long)c * K;
      const float* st = a.stats + (long long)row * (L + 2);
#pragma unroll
      for (int l = 0; l <= L; ++l) {
        float t = 0.0f;
        for (int k = l * l; k < (l + 1) * (l + 1); ++k) t += load1(g + k) * (l ? load1(x + k) : load1(x + k) - st[0]);
        sum[l] += t * st[1 + l];
      }
      sum[L + 1] += load1(g);
    }
  }
  for (int l = 0; l < L + 2; ++l) {
    __syncthreads();
    red[threadIdx.y][threadIdx.x] = sum[l];
    __syncthreads();
    if (threadIdx.y == 0 && c < a.C) {
      float t = red[0][threadIdx.x];
#pragma unroll
      for (int k = 1; k < kWideSumY; ++k) t += red[k][threadIdx.x];
      a.part[((long long)p * (L + 2) + l) * a.C + c] = t;
    }
  }
}

// dw and db: the parts' sums.  A block takes 8 columns; thread (x, y) adds the
// parts y, y + 64, ... of column x (its loads go out together: the kernel is
// one latency long), then the rows of the block are added in a fixed order.
constexpr int kSumX = 8, kSumY = 64;
constexpr int kMaxParts = 608;  // four CTAs on each of 152 SMs

static __global__ void __launch_bounds__(kSumX * kSumY) k_norm_bwd_sum(NormArgs a, int L) {
  __shared__ float red[kSumX * kSumY / 32][kSumX];
  const long long M = (long long)(L + 2) * a.C, m = (long long)blockIdx.x * kSumX + threadIdx.x;
  float t = 0.0f;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // until the kernel that writes the parts is done
  if (m < M) {
    const float* from = a.part + m;
    constexpr int N = (kMaxParts + kSumY - 1) / kSumY;
    float v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) {
      const int p = threadIdx.y + k * kSumY;
      v[k] = p < a.parts ? from[p * M] : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < N; ++k) t += v[k];
  }
  t += __shfl_xor_sync(0xffffffffu, t, 8);
  t += __shfl_xor_sync(0xffffffffu, t, 16);
  if (threadIdx.y % 4 == 0) red[threadIdx.y / 4][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y || m >= M) return;
#pragma unroll
  for (int k = 1; k < kSumY / 4; ++k) t += red[k][threadIdx.x];
  const long long nw = (long long)(L + 1) * a.C;
  if (m < nw) {
    if (a.gw) a.gw[m] = t;
  } else if (a.gb) {
    a.gb[m - nw] = t;
  }
}

}  // namespace eqmp
