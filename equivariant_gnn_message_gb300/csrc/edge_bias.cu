// A learned bias of each edge and head by the bucket of the edge's length, and
// the gradient of its table (sm_103a).  Contracts are in include/eqmp.h.
//
//   bucket[e] = #{b : borders[b] <= |vec_e|},  bias[e][h] = table[bucket[e]][h]
//   dtable[b][h] = sum of dbias[e][h] over the edges of bucket b
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include "host_args.h"
#include "launch.h"

namespace eqmp {

constexpr int kMaxBuckets = 1024, kMaxBiasHeads = 256;
constexpr int64_t kMaxEdges = 1ll << 30;

struct BiasArgs {
  const float *vec, *borders, *table;
  float* bias;
  int* bucket;
  const float* grad;
  float* gtable;
  float* part;  // [parts][B][H]
  int E, B, H, parts;
};

// ---------------------------------------------------------------- forward
// A CTA finds the buckets of a tile of edges, then writes the tile's rows of the
// table side by side.  The search is made in fp32 on squares, and again in 64
// bits (whose rate is 1/60 of it here) only where a border is near.  1,909,372
// edges, 8 heads, 64 buckets: 19 us with cold caches, 71 % of the copy rate (16 where a
// replayed graph finds part of its inputs in L2), 20.5 a call; 105 with every search
// in 64 bits and rows of single values.
constexpr int kBiasThreads = 256, kBiasEdges = 1024;  // edges of a CTA's tile
constexpr int kTableFloats = 4096;                    // a larger table is read through L1

// Squares of fp32 values are exact in 64 bits, so that a length next to a border
// is decided by one rounding of the sum of three, and the same everywhere.
__device__ __noinline__ int bucket_exact(float vx, float vy, float vz, const float* borders, int n) {
  const double x = vx, y = vy, z = vz;
  const double d = __dadd_rn(__dadd_rn(x * x, y * y), z * z);
  int lo = 0, len = n;  // borders[0..lo) <= |vec|
  while (len > 0) {
    const int half = len / 2;
    const double b = borders[lo + half];
    if (b * b <= d) {
      lo += half + 1;
      len -= half + 1;
    } else {
      len = half;
    }
  }
  return lo;
}

// In fp32 the sum of squares is off by 3 2^-24 of itself at most, and a border's
// square by 2^-24, as long as nothing over- or underflows: a border whose square
// is 2^-20 away or more is on the side that it seems to be on.
__device__ __forceinline__ int bucket_of(float x, float y, float z, const float* borders, const float* squares, int n) {
  const float d = fmaf(x, x, fmaf(y, y, z * z));
  int lo = 0, len = n;
  while (len > 0) {
    const int half = len / 2;
    const bool up = squares[lo + half] <= d;
    lo = up ? lo + half + 1 : lo;
    len = up ? len - half - 1 : half;
  }
  const float below = lo > 0 ? squares[lo - 1] : 0.0f, above = lo < n ? squares[lo] : __int_as_float(0x7f800000);
  const bool clear = d > 1e-30f && d < 1e30f && below <= d * (1.0f - 0x1p-20f) && above >= d * (1.0f + 0x1p-20f);
  return clear ? lo : bucket_exact(x, y, z, borders, n);
}

template <typename F>  // float4 where H is a multiple of 4 and everything lies on 16 bytes, else float
__global__ void __launch_bounds__(kBiasThreads) k_edge_bias(BiasArgs a) {
  constexpr int V = sizeof(F) / 4;
  extern __shared__ __align__(16) float shared[];  // borders, their squares, then the table where it fits
  __shared__ int at[kBiasEdges];
  const int n = a.B - 1, width = a.H / V;
  const bool fits = a.B * a.H <= kTableFloats;
  float *const borders = shared, *const squares = shared + n;
  F* const table = reinterpret_cast<F*>(shared + (2 * n + 3) / 4 * 4);
  for (int i = threadIdx.x; i < n; i += kBiasThreads) {
    const float b = a.borders[i];
    borders[i] = b;
    squares[i] = b * b;
  }
  if (fits && a.bias)
    for (int i = threadIdx.x; i < a.B * width; i += kBiasThreads) table[i] = reinterpret_cast<const F*>(a.table)[i];
  const F* const from = fits ? table : reinterpret_cast<const F*>(a.table);
  // a thread's place in the rows that the CTA writes at a time
  const int lines = kBiasThreads / width, line = threadIdx.x / width, col = threadIdx.x % width;
  for (long long e0 = (long long)blockIdx.x * kBiasEdges; e0 < a.E; e0 += (long long)gridDim.x * kBiasEdges) {
    const int count = a.E - e0 < kBiasEdges ? (int)(a.E - e0) : kBiasEdges;
    const float* vec = a.vec + 3 * e0;
    constexpr int EACH = kBiasEdges / kBiasThreads;
    float v[EACH][3];
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const int i = k * kBiasThreads + threadIdx.x;
#pragma unroll
      for (int x = 0; x < 3; ++x) v[k][x] = i < count ? __ldg(vec + 3 * i + x) : 0.0f;
    }
    __syncthreads();  // borders and table are here; the last tile's buckets have been read
#pragma unroll
    for (int k = 0; k < EACH; ++k) {
      const int i = k * kBiasThreads + threadIdx.x;
      if (i >= count) break;
      const int b = bucket_of(v[k][0], v[k][1], v[k][2], borders, squares, n);
      at[i] = b;
      if (a.bucket) a.bucket[e0 + i] = b;
    }
    __syncthreads();
    if (!a.bias || line >= lines) continue;
    F* out = reinterpret_cast<F*>(a.bias + e0 * a.H) + col;
#pragma unroll 4
    for (int i = line; i < count; i += lines) out[(long long)i * width] = from[at[i] * width + col];
  }
}

// ---------------------------------------------------------------- backward
// A CTA sums a range of edges into copies of the table in shared memory: thread
// (r, h) alone adds to column h of copy r, so the order is fixed and nothing is
// atomic.  The next edges' values are loaded while the last ones are added.  Then
// the copies are added, and k_edge_bias_sum adds the CTAs' parts.  A thread takes
// two heads where it can: 1,909,372 edges, 8 heads, 64 buckets 20 us from a replayed
// graph (22 with cold caches, 24.7 a call), one head 24, four 36 (the copies leave room
// for too few threads).  There are 32 copies of 64 buckets and 8 heads, so half of the
// threads have none and wait at the barrier, the main stall.
constexpr int kGradThreads = 256, kGradAhead = 8;
constexpr int kCopyFloats = 16384;  // of the copies of a CTA: three CTAs an SM

__device__ __forceinline__ void add_to(float& t, float v) { t += v; }
__device__ __forceinline__ void add_to(float2& t, const float2& v) { t.x += v.x, t.y += v.y; }

// Sums the edges [begin, end) into the CTA's copies.
template <typename F>  // float2 or float: heads of a thread
__device__ __forceinline__ void sum_range(const BiasArgs& a, float* copy, int heads, int copies, int begin, int end) {
  constexpr int V = sizeof(F) / 4;
  const int h0 = blockIdx.y * heads, hn = min(heads, a.H - h0), size = a.B * heads, width = heads / V;
  const int h = threadIdx.x % width * V, r = threadIdx.x / width;
  const bool mine = r < copies && h < hn;
  const float* grad = a.grad + h0 + h;
  int b[kGradAhead];
  F g[kGradAhead];
  auto load = [&](int e) {
#pragma unroll
    for (int k = 0; k < kGradAhead; ++k) {
      const int i = e + k * copies;
      b[k] = mine && i < end ? __ldg(a.bucket + i) : -1;
      g[k] = mine && i < end ? __ldg(reinterpret_cast<const F*>(grad + (long long)i * a.H)) : F{};
    }
  };
  load(begin + r);
  for (int i = threadIdx.x; i < copies * size; i += kGradThreads) copy[i] = 0.0f;
  __syncthreads();
  float* const own = copy + r * size + h;
  for (int e = begin + r; mine && e < end; e += kGradAhead * copies) {
    int now_b[kGradAhead];
    F now_g[kGradAhead];
#pragma unroll
    for (int k = 0; k < kGradAhead; ++k) now_b[k] = b[k], now_g[k] = g[k];
    load(e + kGradAhead * copies);
#pragma unroll
    for (int k = 0; k < kGradAhead; ++k)
      if ((unsigned)now_b[k] < (unsigned)a.B) {
        F* const to = reinterpret_cast<F*>(own + now_b[k] * heads);
        F t = *to;
        add_to(t, now_g[k]);
        *to = t;
      }
  }
  __syncthreads();
}

// The sum of a CTA's copies at one place of the table.
__device__ __forceinline__ float sum_copies(const float* copy, int copies, int size, int at) {
  float t = 0.0f;
#pragma unroll 8
  for (int c = 0; c < copies; ++c) t += copy[c * size + at];
  return t;
}

template <typename F>
__global__ void __launch_bounds__(kGradThreads) k_edge_bias_bwd(BiasArgs a, int heads, int copies) {
  extern __shared__ __align__(16) float copy[];  // [copies][B][heads]
  const int h0 = blockIdx.y * heads, hn = min(heads, a.H - h0);
  sum_range<F>(a, copy, heads, copies, (int)((long long)a.E * blockIdx.x / a.parts), (int)((long long)a.E * (blockIdx.x + 1) / a.parts));
  float* const out = a.part + (long long)blockIdx.x * a.B * a.H;
  for (int i = threadIdx.x; i < a.B * hn; i += kGradThreads)
    out[(long long)(i / hn) * a.H + h0 + i % hn] = sum_copies(copy, copies, a.B * heads, i / hn * heads + i % hn);
}

// Few edges: a cluster of CTAs, which adds its sums through distributed shared
// memory, in the order of the CTAs.  One launch in place of two, and no workspace:
// 16,516 edges, 4 heads, 32 buckets 16.5 -> 7.1 us a call, 5.1 on the GPU either way.
constexpr int kGradCluster = 8;
constexpr int64_t kFewEdges = 32768;

template <typename F>
__global__ void __cluster_dims__(kGradCluster, 1, 1) __launch_bounds__(kGradThreads) k_edge_bias_bwd_few(BiasArgs a, int heads, int copies) {
  extern __shared__ __align__(16) float copy[];
  const auto cluster = cooperative_groups::this_cluster();
  const int h0 = blockIdx.y * heads, hn = min(heads, a.H - h0), size = a.B * heads, rank = blockIdx.x;
  sum_range<F>(a, copy, heads, copies, (int)((long long)a.E * rank / kGradCluster), (int)((long long)a.E * (rank + 1) / kGradCluster));
  for (int i = threadIdx.x; i < size; i += kGradThreads) copy[i] = sum_copies(copy, copies, size, i);  // a thread's own place
  cluster.sync();
  for (int i = rank * kGradThreads + threadIdx.x; i < a.B * hn; i += kGradCluster * kGradThreads) {
    const int at = i / hn * heads + i % hn;
    float t = 0.0f;
#pragma unroll
    for (int c = 0; c < kGradCluster; ++c) t += cluster.map_shared_rank(copy, c)[at];
    a.gtable[(long long)(i / hn) * a.H + h0 + i % hn] = t;
  }
  cluster.sync();  // no CTA leaves while its sums are read
}

constexpr int kBiasSumX = 32, kBiasSumY = 16;

__global__ void __launch_bounds__(kBiasSumX * kBiasSumY) k_edge_bias_sum(BiasArgs a) {
  __shared__ float red[kBiasSumY][kBiasSumX];
  const int i = blockIdx.x * kBiasSumX + threadIdx.x, n = a.B * a.H;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // until the kernel that writes the parts is done
  float t = 0.0f;
  if (i < n) {
#pragma unroll 8
    for (int p = threadIdx.y; p < a.parts; p += kBiasSumY) t += a.part[(long long)p * n + i];
  }
  red[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y || i >= n) return;
#pragma unroll
  for (int y = 1; y < kBiasSumY; ++y) t += red[y][threadIdx.x];
  a.gtable[i] = t;
}

// CTAs of the backward pass: three on each of 152 SMs, at least 256 edges each,
// and no more than 64 MB of parts; 0: the cluster of CTAs for few edges.
static int grad_parts(int64_t E, int64_t B, int64_t H) {
  if (E <= kFewEdges) return 0;
  int64_t n = (E + 255) / 256;
  const int64_t most = (16ll << 20) / (B * H);
  if (n > 456) n = 456;
  if (n > most) n = most;
  return n < 1 ? 1 : (int)n;
}

static eqmp_status check(int64_t E, int32_t B, int32_t H) {
  if (E < 0 || B < 1 || H < 1) return EQMP_ERR_INVALID_ARG;
  return E > kMaxEdges || B > kMaxBuckets || H > kMaxBiasHeads ? EQMP_ERR_UNSUPPORTED : EQMP_OK;
}

static int64_t grad_workspace(int64_t E, int64_t B, int64_t H) {
  const int parts = grad_parts(E, B, H);
  return parts * B * H * 4;
}

}  // namespace eqmp

using namespace eqmp;

extern "C" {

eqmp_status eqmp_edge_bias(const float* vec, int64_t E, const float* borders, int32_t B, const float* table, int32_t H,
                           float* bias, int32_t* bucket, eqmp_stream_t stream) {
  const eqmp_status cs = check(E, B, H);
  if (cs != EQMP_OK) return cs;
  if (E == 0 || (!bias && !bucket)) return EQMP_OK;
  if (!vec || (B > 1 && !borders) || (bias && !table)) return EQMP_ERR_INVALID_ARG;
  for (const void* p : {(const void*)vec, (const void*)borders, (const void*)table, (const void*)bias, (const void*)bucket})
    if (!aligned(p, 4)) return EQMP_ERR_INVALID_ARG;
  const Span reads[] = {span(vec, E * 12), span(borders, (B - 1) * 4), span(table, bias ? (int64_t)B * H * 4 : 0)};
  const Span writes[] = {span(bias, E * H * 4), span(bucket, E * 4)};
  if (!outputs_apart(reads, writes)) return EQMP_ERR_INVALID_ARG;
  DeviceInfo dev;
  const eqmp_status ds = device_info(&dev);
  if (ds != EQMP_OK) return ds;
  BiasArgs a{};
  a.vec = vec, a.borders = borders, a.table = table, a.bias = bias, a.bucket = bucket;
  a.E = (int)E, a.B = B, a.H = H;
  const int64_t tiles = (E + kBiasEdges - 1) / kBiasEdges, most = (int64_t)dev.sms * 8;
  const int smem = ((2 * (B - 1) + 3) / 4 * 4 + (B * H <= kTableFloats ? B * H : 0)) * 4;
  const unsigned grid = (unsigned)(tiles < most ? tiles : most);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (H % 4 == 0 && aligned(table, 16) && aligned(bias, 16))
    k_edge_bias<float4><<<grid, kBiasThreads, smem, st>>>(a);
  else
    k_edge_bias<float><<<grid, kBiasThreads, smem, st>>>(a);
  return cuda_status(cudaGetLastError());
}

int64_t eqmp_edge_bias_backward_workspace_size(int64_t E, int32_t B, int32_t H) {
  return check(E, B, H) == EQMP_OK ? grad_workspace(E, B, H) : -1;
}

eqmp_status eqmp_edge_bias_backward(const float* grad_bias, const int32_t* bucket, int64_t E, int32_t B, int32_t H,
                                    float* grad_table, void* workspace, int64_t workspace_bytes, eqmp_stream_t stream) {
  const eqmp_status cs = check(E, B, H);
  if (cs != EQMP_OK) return cs;
  if (!grad_table) return EQMP_OK;
  if (!aligned(grad_bias, 4) || !aligned(bucket, 4) || !aligned(grad_table, 4)) return EQMP_ERR_INVALID_ARG;
  if (E > 0 && (!grad_bias || !bucket)) return EQMP_ERR_INVALID_ARG;
  const int64_t ws = grad_workspace(E, B, H);
  if (ws > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < ws)) return EQMP_ERR_INVALID_ARG;
  const Span reads[] = {span(grad_bias, E * H * 4), span(bucket, E * 4)};
  const Span writes[] = {span(grad_table, (int64_t)B * H * 4), span(workspace, ws)};
  if (!outputs_apart(reads, writes)) return EQMP_ERR_INVALID_ARG;
  BiasArgs a{};
  a.bucket = const_cast<int*>(bucket), a.grad = grad_bias, a.gtable = grad_table, a.part = static_cast<float*>(workspace);
  a.E = (int)E, a.B = B, a.H = H, a.parts = grad_parts(E, B, H);
  // heads of a CTA: all, or as many as one copy of the table has room for
  int heads = H < kCopyFloats / B ? H : kCopyFloats / B;
  const int V = heads % 2 == 0 && H % 2 == 0 && aligned(grad_bias, 8) ? 2 : 1;
  int copies = kGradThreads * V / heads;
  if (copies > kCopyFloats / (B * heads)) copies = kCopyFloats / (B * heads);
  const int smem = copies * B * heads * 4;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const dim3 grid((unsigned)(a.parts ? a.parts : kGradCluster), (unsigned)((H + heads - 1) / heads));
  static unsigned long long done[4] = {0, 0, 0, 0};
  auto run = [&](auto kernel, unsigned long long* mask) {
    if (ensure_smem_attr(kernel, kCopyFloats * 4, mask) != cudaSuccess) return false;
    kernel<<<grid, kGradThreads, smem, st>>>(a, heads, copies);
    return cudaGetLastError() == cudaSuccess;
  };
  if (!a.parts) {
    const bool set = V == 2 ? run(k_edge_bias_bwd_few<float2>, done) : run(k_edge_bias_bwd_few<float>, done + 1);
    return set ? EQMP_OK : EQMP_ERR_CUDA;
  }
  if (!(V == 2 ? run(k_edge_bias_bwd<float2>, done + 2) : run(k_edge_bias_bwd<float>, done + 3))) return EQMP_ERR_CUDA;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((B * H + kBiasSumX - 1) / kBiasSumX));
  cfg.blockDim = dim3(kBiasSumX, kBiasSumY);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, k_edge_bias_sum, a));
}

}  // extern "C"
