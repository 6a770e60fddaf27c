// Entry points of the norms and of dropout: argument checks and dispatch.
// Contracts are in include/eqmp.h, the formulas in norm.cuh.
#include <math.h>

#include "launch.h"
#include "norm.cuh"
#include "norm_rows.cuh"

namespace eqmp {

static bool aligned(const void* p, int dtype_bytes) { return reinterpret_cast<uintptr_t>(p) % dtype_bytes == 0; }

// Checks d for rows of `cols` columns and resolves its rate to 1/65536.
static eqmp_status drop_args(const eqmp_drop& d, long long cols, DropArgs* out) {
  *out = DropArgs{};
  out->group = 1;
  if (!(d.p >= 0.0 && d.p <= 1.0)) return EQMP_ERR_INVALID_ARG;
  if (d.p == 0.0) return EQMP_OK;
  if (d.group < 1 || cols % d.group != 0 || !aligned(d.step, 8)) return EQMP_ERR_INVALID_ARG;
  out->seed = d.seed;
  out->offset = d.offset;
  out->step = reinterpret_cast<const unsigned long long*>(d.step);
  out->threshold = (uint32_t)floor(d.p * 65536.0 + 0.5);
  out->scale = out->threshold < 65536 ? 65536.0f / (float)(65536 - out->threshold) : 0.0f;
  out->group = d.group;
  return EQMP_OK;
}

// One strided matrix: rows of `cols` elements, `ld` elements apart.
struct Plane {
  const void* p;
  long long ld;
};

// The memory of an argument; NULL and empty ones meet nothing.
struct Span {
  uintptr_t begin, end;
};

static Span span(const void* p, long long bytes) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return Span{at, p && bytes > 0 ? at + (uintptr_t)bytes : at};
}

static Span span(const Plane& a, long long rows, long long cols, int bytes) {
  return span(a.p, rows > 0 ? ((rows - 1) * a.ld + cols) * bytes : 0);
}

static Span span(const DropArgs& d) { return span(d.step, sizeof(*d.step)); }

static bool meet(const Span& a, const Span& b) {
  return a.begin < a.end && b.begin < b.end && a.begin < b.end && b.begin < a.end;
}

// Outputs apart from the inputs and from one another.
template <int I, int O>
static bool outputs_apart(const Span (&in)[I], const Span (&out)[O]) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (meet(in[i], out[o])) return false;
    for (int q = 0; q < o; ++q)
      if (meet(out[q], out[o])) return false;
  }
  return true;
}

// A row stride of up to 2^31 elements, so that 2^30 rows stay in 64 bits.
static bool stride_ok(long long ld) { return ld >= 0 && ld <= 1ll << 31; }

// Inputs: aligned, strides that address forward.  Outputs (packed): aligned.
static bool planes_ok(const Plane* in, int n_in, void* const* outs, int n_out, int bytes) {
  for (int i = 0; i < n_in; ++i)
    if (in[i].p && (!aligned(in[i].p, bytes) || !stride_ok(in[i].ld))) return false;
  for (int o = 0; o < n_out; ++o)
    if (!aligned(outs[o], bytes)) return false;
  return true;
}

static int rows_grid(long long rows, const DeviceInfo& dev) {
  const long long cap = (long long)dev.sms * 8;
  return (int)(rows < cap ? rows : cap);
}

eqmp_status launch_norm_bwd_sum(const NormArgs& a, int L, cudaStream_t st) {
  const long long M = (long long)(L + 2) * a.C;
  // launched while the pass before it runs; the kernel waits for its parts
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((M + kSumX - 1) / kSumX));
  cfg.blockDim = dim3(kSumX, kSumY);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, k_norm_bwd_sum, a, L));
}

template <typename T, int L>
static eqmp_status forward_t(const NormArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  k_norm_wide<T, L><<<rows_grid(a.rows, dev), kWideThreads, 0, st>>>(a);
  return cuda_status(cudaGetLastError());
}

template <typename T, int L>
static eqmp_status backward_t(const NormArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  if (a.gr || a.gx) {
    k_norm_bwd_wide<T, L><<<rows_grid(a.rows, dev), kWideThreads, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return EQMP_ERR_CUDA;
  }
  if (!a.gw && !a.gb) return EQMP_OK;
  const dim3 grid((unsigned)((a.C + kWideSumX - 1) / kWideSumX), (unsigned)a.parts);
  k_norm_bwd_wide_w<T, L><<<grid, dim3(kWideSumX, kWideSumY), 0, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return EQMP_ERR_CUDA;
  return launch_norm_bwd_sum(a, L, st);
}

template <int L>
static eqmp_status dispatch_t(const NormArgs& a, bool bf16, bool backward, const DeviceInfo& dev, cudaStream_t st) {
  if (backward) return bf16 ? backward_t<__nv_bfloat16, L>(a, dev, st) : backward_t<float, L>(a, dev, st);
  return bf16 ? forward_t<__nv_bfloat16, L>(a, dev, st) : forward_t<float, L>(a, dev, st);
}

static eqmp_status dispatch(const NormArgs& a, int L, bool bf16, bool backward, cudaStream_t st) {
  DeviceInfo dev;
  const eqmp_status s = device_info(&dev);
  if (s != EQMP_OK) return s;
  bool done = false;
  const auto rows = backward ? (bf16 ? launch_norm_bwd_rows_bf16 : launch_norm_bwd_rows_f32)
                             : (bf16 ? launch_norm_rows_bf16 : launch_norm_rows_f32);
  const eqmp_status rs = rows(a, L, dev, st, &done);
  if (rs != EQMP_OK || done) return rs;
  switch (L) {
    case 0: return dispatch_t<0>(a, bf16, backward, dev, st);
    case 3: return dispatch_t<3>(a, bf16, backward, dev, st);
    case 4: return dispatch_t<4>(a, bf16, backward, dev, st);
    case 5: return dispatch_t<5>(a, bf16, backward, dev, st);
    case 6: return dispatch_t<6>(a, bf16, backward, dev, st);
  }
  return EQMP_ERR_UNSUPPORTED;
}

// Row ranges of the partial weight gradients in the kernels for any shape:
// enough to fill the device, at least 64 rows each, so that the partials stay
// a small part of the traffic.
static int wide_parts(long long rows) {
  const long long want = (rows + 63) / 64;
  return (int)(want < 1 ? 1 : want > 128 ? 128 : want);
}

// At most one part a row, at most kMaxParts.
static int64_t workspace_bytes(int64_t rows, int64_t C, int L) {
  return (rows < kMaxParts ? rows : kMaxParts) * (L + 2) * C * 4;
}

// Up to 2^30 rows of up to 2^30 values, so that a row or column index plus a
// stride of the launch stays an int.
static eqmp_status check_sizes(int64_t rows, int64_t C, int64_t K, eqmp_dtype dtype) {
  if (rows < 0 || C < 1 || (dtype != EQMP_F32 && dtype != EQMP_BF16)) return EQMP_ERR_INVALID_ARG;
  return rows > (1ll << 30) || C > (1ll << 30) / K ? EQMP_ERR_UNSUPPORTED : EQMP_OK;
}

static eqmp_status run_forward(Plane x, Plane r, eqmp_dtype dtype, int64_t rows, int64_t C, int L, eqmp_drop drop,
                               const float* w, const float* b, float eps, void* s, void* y, float* stats,
                               cudaStream_t st) {
  const int64_t K = (L + 1) * (L + 1);
  const eqmp_status zs = check_sizes(rows, C, K, dtype);
  if (zs != EQMP_OK) return zs;
  if (!(eps >= 0.0f) || isinf(eps)) return EQMP_ERR_INVALID_ARG;
  NormArgs a{};
  const eqmp_status ds = drop_args(drop, C * K, &a.drop);
  if (ds != EQMP_OK) return ds;
  if (rows == 0 || (!s && !y && !stats)) return EQMP_OK;
  const bool bf16 = dtype == EQMP_BF16;
  const int bytes = bf16 ? 2 : 4;
  const Plane in[] = {x, r};
  void* const outs[] = {s, y};
  if (!x.p || !planes_ok(in, 2, outs, 2, bytes)) return EQMP_ERR_INVALID_ARG;
  if (!aligned(w, 4) || !aligned(b, 4) || !aligned(stats, 4)) return EQMP_ERR_INVALID_ARG;
  const Span reads[] = {span(x, rows, C * K, bytes), span(r, rows, C * K, bytes), span(w, (L + 1) * C * 4), span(b, C * 4),
                        span(a.drop)};
  const Span writes[] = {span(s, rows * C * K * bytes), span(y, rows * C * K * bytes), span(stats, rows * (L + 2) * 4)};
  if (!outputs_apart(reads, writes)) return EQMP_ERR_INVALID_ARG;
  a.x = x.p;
  a.x_ld = x.ld;
  a.r = r.p;
  a.r_ld = r.ld;
  a.s = s;
  a.y = y;
  a.stats = stats;
  a.w = w;
  a.b = b;
  a.rows = (int)rows;
  a.cols = (int)(C * K);
  a.C = (int)C;
  a.eps = eps;
  return dispatch(a, L, bf16, false, st);
}

static eqmp_status run_backward(Plane g, Plane x, Plane r, eqmp_dtype dtype, int64_t rows, int64_t C, int L,
                                eqmp_drop drop, const float* w, const float* stats, void* gr, void* gx, float* gw,
                                float* gb, void* workspace, int64_t ws_bytes, cudaStream_t st) {
  const int64_t K = (L + 1) * (L + 1);
  const eqmp_status zs = check_sizes(rows, C, K, dtype);
  if (zs != EQMP_OK) return zs;
  NormArgs a{};
  const eqmp_status ds = drop_args(drop, C * K, &a.drop);
  if (ds != EQMP_OK) return ds;
  if (!gr && !gx && !gw && !gb) return EQMP_OK;
  if (!aligned(gw, 4) || !aligned(gb, 4)) return EQMP_ERR_INVALID_ARG;
  const bool bf16 = dtype == EQMP_BF16;
  const int bytes = bf16 ? 2 : 4;
  const Plane in[] = {x, g, r};
  if (rows > 0 && !planes_ok(in, 3, nullptr, 0, bytes)) return EQMP_ERR_INVALID_ARG;
  const Span reads[] = {span(x, rows, C * K, bytes), span(g, rows, C * K, bytes), span(r, rows, C * K, bytes),
                        span(w, (L + 1) * C * 4), span(stats, rows * (L + 2) * 4), span(a.drop)};
  const Span writes[] = {span(gr, rows * C * K * bytes), span(gx, rows * C * K * bytes), span(gw, (L + 1) * C * 4),
                         span(gb, C * 4), span(workspace, gw || gb ? workspace_bytes(rows, C, L) : 0)};
  if (!outputs_apart(reads, writes)) return EQMP_ERR_INVALID_ARG;
  if (rows == 0) {  // no row: the sums are zero
    if (gw && cudaMemsetAsync(gw, 0, (size_t)(L + 1) * C * 4, st) != cudaSuccess) return EQMP_ERR_CUDA;
    if (gb && cudaMemsetAsync(gb, 0, (size_t)C * 4, st) != cudaSuccess) return EQMP_ERR_CUDA;
    return EQMP_OK;
  }
  void* const outs[] = {gr, gx};
  if (!x.p || !g.p || !stats || !planes_ok(nullptr, 0, outs, 2, bytes)) return EQMP_ERR_INVALID_ARG;
  if (!aligned(w, 4) || !aligned(stats, 4)) return EQMP_ERR_INVALID_ARG;
  if ((gw || gb) && (!workspace || !aligned(workspace, 16) || ws_bytes < workspace_bytes(rows, C, L)))
    return EQMP_ERR_INVALID_ARG;
  a.x = x.p;
  a.x_ld = x.ld;
  a.g = g.p;
  a.g_ld = g.ld;
  a.r = r.p;
  a.r_ld = r.ld;
  a.gr = gr;
  a.gx = gx;
  a.gw = gw;
  a.gb = gb;
  a.stats = const_cast<float*>(stats);
  a.w = w;
  a.part = static_cast<float*>(workspace);
  a.parts = wide_parts(rows);
  a.rows = (int)rows;
  a.cols = (int)(C * K);
  a.C = (int)C;
  return dispatch(a, L, bf16, true, st);
}

// ---------------------------------------------------------------- dropout
// A CTA takes `lanes` neighbouring vectors (a segment of the columns) of
// kDropPasses * lines rows; a thread keeps its columns, so that what the
// generator makes of them is formed once, and loads its vectors before it
// draws for them.  Rows that begin on 16 bytes: each vector's draws are formed
// by its thread.  Rows that begin anywhere (SHIFT, or V = 1 where they do not
// begin alike): the CTA forms the keep bits of its rows' units together, since
// neighbours share the generator's blocks, and a vector looks its bits up.
// With SHIFT a CTA's rows are 8 apart, so that all of them begin at the same
// place behind a 16-byte boundary (see norm_rows.cuh).
// 1,909,372 x 64 bf16 by element 71 us (101 % of the measured copy rate; with a
// division and all 20 products of the generator per vector it took 97, bound by
// the multiplier), 500,000 x 131 fp32 89 us (87 %), 1,000,000 x 131 bf16 160 us
// (48 %: seven instructions a value for the bits alone).
constexpr int kDropThreads = 256, kDropPasses = 8;

struct DropShape {
  int lanes, segments, lines;
};

template <typename T, int V, bool SHIFT>
__global__ void __launch_bounds__(kDropThreads) k_drop(const T* x, long long ld, T* out, int rows, int cols,
                                                       DropArgs d, DropShape sh) {
  constexpr bool TABLE = V == 1 || SHIFT;
  constexpr int APART = SHIFT ? 8 : 1;
  const Dropper drop(d);
  extern __shared__ uint8_t bits[];  // TABLE: [row][byte], from the segment's first unit on, rounded down to a byte
  const int lane = threadIdx.x % sh.lanes, line = threadIdx.x / sh.lanes;
  const int seg = blockIdx.x % sh.segments, tile = blockIdx.x / sh.segments;
  const int row0 = tile / APART * (APART * kDropPasses * sh.lines) + tile % APART;
  const int step = APART * sh.lines;  // between a thread's rows
  const int shift = SHIFT ? (int)((uint32_t)row0 * (uint32_t)cols % V) : 0;
  const int seg_col = seg * sh.lanes * V - shift, col = seg_col + lane * V;
  const bool mine = line < sh.lines && col < cols;
  const int first_row = row0 + APART * line;
  const int lo = col < 0 ? -col : 0, n = cols - col < V ? cols - col : V;  // the row's values of the vector
  Pack<T, V> in[kDropPasses];
#pragma unroll
  for (int k = 0; k < kDropPasses; ++k) {
    const int row = first_row + k * step;
    if (SHIFT && (!mine || row >= rows)) break;
    // a whole vector may hold the end of the row before and the beginning of the next one
    if (SHIFT || (mine && row < rows)) {
      if (!SHIFT || n == V || row + 1 < rows)
        in[k].load(x + row * ld + col);
      else
        in[k].load_part(x + row * ld + col, n);
    }
  }
  const uint32_t unit = (uint32_t)(col > 0 ? col : 0) / (uint32_t)drop.group;
  const int left = (int)((unit + 1) * drop.group) - col;  // of the vector's values in its first unit
  if constexpr (TABLE) {
    const int last_col = seg_col + sh.lanes * V - 1 < cols - 1 ? seg_col + sh.lanes * V - 1 : cols - 1;
    const uint32_t first = (uint32_t)(seg_col > 0 ? seg_col : 0) / (uint32_t)drop.group >> 3;
    const int bytes = (int)((uint32_t)last_col / (uint32_t)drop.group >> 3) - (int)first + 1;
    if (drop.on) {
      for (int i = threadIdx.x; i < bytes * kDropPasses * sh.lines; i += blockDim.x)
        bits[i] = (uint8_t)drop.keep_bits(drop.block(row0 + i / bytes * APART, first + i % bytes));
      __syncthreads();
    }
    const uint8_t* b = bits + line * bytes + ((unit >> 3) - first);
#pragma unroll
    for (int k = 0; k < kDropPasses; ++k, b += sh.lines * bytes) {
      const int row = first_row + k * step;
      if (!mine || row >= rows) break;
      T* to = out + (long long)row * cols + col;
      if constexpr (V == 1) {
        float f = load1(&in[k].v);
        if (drop.on) f = *b >> (unit & 7) & 1 ? f * drop.scale : 0.0f;
        store1(to, f);
      } else {
        float2 f[V / 2];
        in[k].get(f);
        if (drop.on) {
          uint32_t keep;
          if (drop.group == 1) {
            keep = (b[0] | (uint32_t)b[1] << 8) >> (unit & 7);
            keep <<= lo;
          } else {  // one unit after the other
            keep = *b >> (unit & 7) & 1 ? (1u << V) - 1 : 0;
            uint32_t u = unit;
#pragma unroll 1
            for (int i = left; i < n; i += drop.group) {
              ++u;
              const uint32_t from = 1u << i, rest = (1u << V) - from;
              keep = b[(u >> 3) - (unit >> 3)] >> (u & 7) & 1 ? keep | rest : keep & ~rest;
            }
          }
#pragma unroll
          for (int s = 0; s < V / 2; ++s) {
            f[s] = __fmul2_rn(f[s], both(drop.scale));
            f[s].x = keep >> (2 * s) & 1 ? f[s].x : 0.0f;
            f[s].y = keep >> (2 * s + 1) & 1 ? f[s].y : 0.0f;
          }
        }
        if (lo == 0 && n == V)
          Pack<T, V>::store(to, f);
        else
          put_part(to, f, lo, n);
      }
    }
  } else {
    const PhiloxBlock pb = drop.of_block(unit >> 3);
#pragma unroll
    for (int k = 0; k < kDropPasses; ++k) {
      const int row = first_row + k * step;
      if (!mine || row >= rows) break;
      float2 f[V / 2];
      in[k].get(f);
      if (drop.on) {
        uint4 w = drop.block(drop.of_row(row), pb);
        if (drop.group == 1) {
          const bool upper = V == 4 && (col & 4);
          const uint32_t words[4] = {upper ? w.z : w.x, upper ? w.w : w.y, w.z, w.w};
#pragma unroll
          for (int s = 0; s < V / 2; ++s) {
            f[s] = __fmul2_rn(f[s], both(drop.scale));
            f[s].x = words[s] << 16 > drop.bound ? f[s].x : 0.0f;
            f[s].y = words[s] > drop.bound ? f[s].y : 0.0f;
          }
        } else {
          uint32_t keep = drop.keeps(w, unit) ? (1u << V) - 1 : 0;
          if (left < V) {  // more units: one after the other
            uint32_t u = unit;
#pragma unroll 1
            for (int i = left; i < V; i += drop.group) {
              if ((++u & 7) == 0) w = drop.block(row, u >> 3);
              const uint32_t from = 1u << i, rest = (1u << V) - from;
              keep = drop.keeps(w, u) ? keep | rest : keep & ~rest;
            }
          }
#pragma unroll
          for (int s = 0; s < V / 2; ++s) {
            f[s] = __fmul2_rn(f[s], both(drop.scale));
            f[s].x = keep >> (2 * s) & 1 ? f[s].x : 0.0f;
            f[s].y = keep >> (2 * s + 1) & 1 ? f[s].y : 0.0f;
          }
        }
      }
      Pack<T, V>::store(out + (long long)row * cols + col, f);
    }
  }
}

template <typename T, int V, bool SHIFT>
static eqmp_status launch_drop(const T* x, long long ld, T* out, int rows, int cols, const DropArgs& d, cudaStream_t st) {
  const int vectors = SHIFT ? (cols + 2 * (V - 1)) / V : cols / V, apart = SHIFT ? 8 : 1;
  DropShape sh;
  sh.segments = (vectors + kDropThreads - 1) / kDropThreads;
  sh.lanes = (vectors + sh.segments - 1) / sh.segments;
  sh.lines = kDropThreads / sh.lanes;
  if (sh.lines > rows / (apart * kDropPasses)) sh.lines = rows / (apart * kDropPasses) > 0 ? rows / (apart * kDropPasses) : 1;
  const int threads = (sh.lanes * sh.lines + 31) / 32 * 32;
  const int tile = kDropPasses * sh.lines;
  const long long grid = ((long long)rows + apart * tile - 1) / (apart * tile) * apart * sh.segments;
  if (grid > INT32_MAX) return EQMP_ERR_UNSUPPORTED;
  // a byte for eight units begun, one more read with the last
  const size_t smem = V == 1 || SHIFT ? (size_t)(sh.lanes * V / 8 + 2) * tile + 1 : 0;
  k_drop<T, V, SHIFT><<<(unsigned)grid, threads, smem, st>>>(x, ld, out, rows, cols, d, sh);
  return cuda_status(cudaGetLastError());
}

template <typename T>
static eqmp_status run_dropout(const void* x, long long ld, void* out, int rows, int cols, const DropArgs& d,
                               cudaStream_t st) {
  constexpr int B = sizeof(T);
  const T* in = static_cast<const T*>(x);
  T* to = static_cast<T*>(out);
  const bool whole = cols * (long long)B % 16 == 0;
  if (whole && on16(x) && on16(out) && ld * B % 16 == 0) return launch_drop<T, 16 / B, false>(in, ld, to, rows, cols, d, st);
  // in place a row's last vector would read what another thread writes
  if (cols >= 4 * (16 / B) && in != to && on16(out) && lies_packed(x, ld, cols, B))
    return launch_drop<T, 16 / B, true>(in, ld, to, rows, cols, d, st);
  return launch_drop<T, 1, false>(in, ld, to, rows, cols, d, st);
}

}  // namespace eqmp

using namespace eqmp;

extern "C" {

eqmp_status eqmp_layer_norm(const void* x, int64_t x_ld, const void* residual, int64_t residual_ld, eqmp_dtype dtype,
                            int64_t rows, int64_t cols, eqmp_drop drop, const float* w, const float* b, float eps,
                            void* s, void* y, float* stats, eqmp_stream_t stream) {
  return run_forward(Plane{x, x_ld}, Plane{residual, residual_ld}, dtype, rows, cols, 0, drop, w, b, eps, s, y, stats,
                     reinterpret_cast<cudaStream_t>(stream));
}

int64_t eqmp_layer_norm_backward_workspace_size(int64_t rows, int64_t cols) {
  return check_sizes(rows, cols, 1, EQMP_F32) == EQMP_OK ? workspace_bytes(rows, cols, 0) : -1;
}

eqmp_status eqmp_layer_norm_backward(const void* grad_y, int64_t grad_y_ld, const void* s, int64_t s_ld,
                                     const void* grad_s, int64_t grad_s_ld, eqmp_dtype dtype, int64_t rows,
                                     int64_t cols, eqmp_drop drop, const float* w, const float* stats, void* grad_r,
                                     void* grad_x, float* grad_w, float* grad_b, void* workspace,
                                     int64_t workspace_bytes, eqmp_stream_t stream) {
  return run_backward(Plane{grad_y, grad_y_ld}, Plane{s, s_ld}, Plane{grad_s, grad_s_ld}, dtype, rows, cols, 0, drop,
                      w, stats, grad_r, grad_x, grad_w, grad_b, workspace, workspace_bytes,
                      reinterpret_cast<cudaStream_t>(stream));
}

static bool degree_ok(int32_t l_max) { return l_max >= 3 && l_max <= 6; }

// A draw covers a whole channel: dropping single components would turn with
// the frame.
static bool whole_channels(const eqmp_drop& d, int32_t l_max) {
  return d.p == 0.0 || d.group == (l_max + 1) * (l_max + 1);
}

eqmp_status eqmp_degree_norm(const void* x, const void* residual, eqmp_dtype dtype, int64_t N, int32_t C,
                             int32_t l_max, eqmp_drop drop, const float* w, const float* b, float eps, void* s,
                             void* y, float* stats, eqmp_stream_t stream) {
  if (!degree_ok(l_max)) return EQMP_ERR_UNSUPPORTED;
  if (!whole_channels(drop, l_max)) return EQMP_ERR_INVALID_ARG;
  const long long ld = (long long)C * (l_max + 1) * (l_max + 1);
  return run_forward(Plane{x, ld}, Plane{residual, ld}, dtype, N, C, l_max, drop, w, b, eps, s, y, stats,
                     reinterpret_cast<cudaStream_t>(stream));
}

int64_t eqmp_degree_norm_backward_workspace_size(int64_t N, int32_t C, int32_t l_max) {
  return degree_ok(l_max) && check_sizes(N, C, (l_max + 1) * (l_max + 1), EQMP_F32) == EQMP_OK ? workspace_bytes(N, C, l_max) : -1;
}

eqmp_status eqmp_degree_norm_backward(const void* grad_y, const void* s, const void* grad_s, eqmp_dtype dtype,
                                      int64_t N, int32_t C, int32_t l_max, eqmp_drop drop, const float* w,
                                      const float* stats, void* grad_r, void* grad_x, float* grad_w, float* grad_b,
                                      void* workspace, int64_t workspace_bytes, eqmp_stream_t stream) {
  if (!degree_ok(l_max)) return EQMP_ERR_UNSUPPORTED;
  if (!whole_channels(drop, l_max)) return EQMP_ERR_INVALID_ARG;
  const long long ld = (long long)C * (l_max + 1) * (l_max + 1);
  return run_backward(Plane{grad_y, ld}, Plane{s, ld}, Plane{grad_s, ld}, dtype, N, C, l_max, drop, w, stats, grad_r,
                      grad_x, grad_w, grad_b, workspace, workspace_bytes, reinterpret_cast<cudaStream_t>(stream));
}

eqmp_status eqmp_dropout(const void* x, int64_t x_ld, eqmp_dtype dtype, int64_t rows, int64_t cols, eqmp_drop drop,
                         void* out, eqmp_stream_t stream) {
  const eqmp_status zs = check_sizes(rows, cols, 1, dtype);
  if (zs != EQMP_OK) return zs;
  DropArgs d;
  const eqmp_status ds = drop_args(drop, cols, &d);
  if (ds != EQMP_OK) return ds;
  if (rows == 0) return EQMP_OK;
  const int bytes = dtype == EQMP_BF16 ? 2 : 4;
  if (!x || !out || !stride_ok(x_ld) || !aligned(x, bytes) || !aligned(out, bytes)) return EQMP_ERR_INVALID_ARG;
  const bool in_place = x == out && (x_ld == cols || rows == 1);  // each element is read before it is written, by one thread
  const Span reads[] = {in_place ? Span{} : span(Plane{x, x_ld}, rows, cols, bytes), span(d)};
  const Span writes[] = {span(out, rows * cols * bytes)};
  if (!outputs_apart(reads, writes)) return EQMP_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == EQMP_BF16 ? run_dropout<__nv_bfloat16>(x, x_ld, out, (int)rows, (int)cols, d, st)
                            : run_dropout<float>(x, x_ld, out, (int)rows, (int)cols, d, st);
}

}  // extern "C"
