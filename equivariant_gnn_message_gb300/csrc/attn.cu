// Entry points of the attention over a receiver's edges: argument checks and
// the choice of the kernels' forms.  Contracts are in include/eqmp.h.
#include <math.h>

#include "attn_launch.cuh"
#include "host_args.h"

namespace eqmp {

constexpr int kMaxDim = 256, kMaxValueDim = 1024, kMaxHeads = 1024;
constexpr int64_t kMaxCount = 1ll << 30;  // nodes and edges: an index plus a stride of the launch stays an int

struct Sizes {
  int64_t N, Ns, E;
  int32_t H, D, Dv;
};

static eqmp_status check_sizes(const Sizes& n, eqmp_dtype dtype, float scale) {
  if (n.N < 0 || n.Ns < 0 || n.E < 0 || n.H < 1 || n.D < 1 || n.Dv < 1) return EQMP_ERR_INVALID_ARG;
  if (dtype != EQMP_F32 && dtype != EQMP_BF16) return EQMP_ERR_INVALID_ARG;
  if (!isfinite(scale)) return EQMP_ERR_INVALID_ARG;
  const bool fits = n.N <= kMaxCount && n.Ns <= kMaxCount && n.E <= kMaxCount && n.H <= kMaxHeads && n.D <= kMaxDim &&
                    n.Dv <= kMaxValueDim;
  return fits ? EQMP_OK : EQMP_ERR_UNSUPPORTED;
}

// Blocks that rows of more than two are cut into: at least 32 edges, at most
// 2048 blocks in all, and fewer of wide heads, so that their parts (`values`
// each, two a block) stay below 64 MB, or are those of 8 blocks.  Graphs of up to kWhole
// edges are not cut: there the launches that join the parts cost more than they
// save (64 atoms, 742 edges: forward 24.5 us a call with them, 19.4 without,
// backward 38 and 34), unless nearly all edges are one node's (1000 edges of one
// receiver: 119 us by one warp a head, 24 in blocks).
constexpr int64_t kWhole = 1024, kPartBytes = 64ll << 20;

static void cut(int64_t E, int64_t values, int* block, int* blocks) {
  int64_t most = kPartBytes / (2 * 4 * values);
  most = most < 8 ? 8 : most > 2048 ? 2048 : most;
  const int64_t want = (E + most - 1) / most;
  *block = (int)(want < 32 ? 32 : (want + 31) / 32 * 32);
  *blocks = E > kWhole ? (int)((E + *block - 1) / *block) : 0;
}

// Values of a part: the row's maximum, sum and result; its sums of p dp, of dp and of edges, and of p dp k and p k; its
// gradients of key and value.
static int64_t forward_values(const Sizes& n) { return (int64_t)n.H * (n.Dv + 2); }
static int64_t recv_values(const Sizes& n) { return (int64_t)n.H * (2 * n.D + 3); }
static int64_t send_values(const Sizes& n) { return (int64_t)n.H * (n.D + n.Dv); }

static int64_t part_bytes(int64_t E, int64_t values) {
  int block, blocks;
  cut(E, values, &block, &blocks);
  return 2ll * blocks * values * 4;
}

static int64_t forward_workspace(const Sizes& n) { return part_bytes(n.E, forward_values(n)); }

struct BackwardSpace {
  int64_t pd, delta, part;
  int64_t total() const { return pd + delta + part; }
};

static BackwardSpace backward_workspace(const Sizes& n, int64_t E_send) {
  const int64_t recv = part_bytes(n.E, recv_values(n)), send = part_bytes(E_send, send_values(n));
  return BackwardSpace{n.E * n.H * 8 + 15 & ~15ll, n.N * n.H * 4 + 15 & ~15ll, recv > send ? recv : send};
}

// What every head of every row begins on, at most 16 bytes: gathered over the
// addresses, row pitches and head sizes of a call.
struct Alignment {
  unsigned long long bits = 16;
  void add(const void* p) { bits |= reinterpret_cast<uintptr_t>(p); }
  void add(const void* p, long long ld, int bytes) {
    if (!p) return;
    add(p);
    bits |= (unsigned long long)(ld * bytes);
    if (ld * bytes >= 1ll << 32) bits |= 1;  // rows too far apart for the rings' 32-bit pitches
  }
  int bytes() const { return (int)(bits & -bits); }
};

// The widest vectors that the alignment allows, and for them the fewest lanes a
// head whose registers hold it; more lanes where there are too few rows to fill
// the device.  Heads that the forms with vectors of 8 or 4 bytes do not hold, and
// bf16 heads that begin anywhere, take the general kernels.
static AttnForm form_of(const Sizes& n, int64_t rows, int64_t gathered, int bytes, int alignment) {
  AttnForm f;
  if (gathered == 0) alignment = 0;  // the rings' copies of nothing need an address that is one
  for (f.VB = alignment < 4 ? 0 : alignment; f.VB >= 4; f.VB /= 2) {
    const int k = (n.D * bytes + f.VB - 1) / f.VB, v = (n.Dv * bytes + f.VB - 1) / f.VB;
    auto fits = [&](int G) { return k <= 2 * G && v <= 8 * G; };
    f.G = 8;
    while (f.G < 32 && (!fits(f.G) || n.H * f.G * 2 <= 32 || rows * ((n.H * f.G + 31) / 32) < 152 * 16)) f.G *= 2;
    if (f.VB < 16 && f.G > 8) f.G = f.VB == 8 ? 16 : 32;
    f.KN = (k + f.G - 1) / f.G;
    f.VN = (v + f.G - 1) / f.G;
    if (fits(f.G)) break;
  }
  if (f.VB < 4) {
    f.VB = 0;
    f.G = n.D <= 32 && n.Dv <= 128 && n.H > 2 && rows * ((n.H + 3) / 4) >= 152 * 16 ? 8 : 32;
    f.KN = (n.D + f.G - 1) / f.G;
    f.VN = (n.Dv + f.G - 1) / f.G;
  }
  // Rows of a warp: up to 4, as long as there are eight warps for each place on the device.  More keep the ring filled across
  // more ends of rows, but neighbouring rows, which share senders, are then further apart in time: 100,000 atoms in cells'
  // order, fp32, forward 780 us with one row, 726 two, 701 four, 711 six, 755 sixteen; 10,000 of 48 edges, bf16, one or two
  // rows 190, four 204.
  const int64_t each = rows * ((n.H * f.G + 31) / 32) / (152 * 8 * 8);
  f.rows_each = (int)(each < 1 ? 1 : each > 4 ? 4 : each);
  return f;
}

}  // namespace eqmp

using namespace eqmp;

extern "C" {

int64_t eqmp_edge_attention_workspace_size(int64_t E, int32_t H, int32_t Dv) {
  const Sizes n{0, 0, E, H, 1, Dv};
  return check_sizes(n, EQMP_F32, 1.0f) == EQMP_OK ? forward_workspace(n) : -1;
}

eqmp_status eqmp_edge_attention(const void* q, int64_t q_ld, const void* k, int64_t k_ld, const void* v, int64_t v_ld,
                                eqmp_dtype dtype, int64_t N, int64_t N_src, int64_t E, int32_t H, int32_t D, int32_t Dv,
                                const int32_t* row_offsets, const int32_t* src, const float* bias, float scale,
                                void* out, float* stats, void* workspace, int64_t workspace_bytes, eqmp_stream_t stream) {
  const Sizes n{N, N_src, E, H, D, Dv};
  const eqmp_status zs = check_sizes(n, dtype, scale);
  if (zs != EQMP_OK) return zs;
  if (N == 0 || (!out && !stats)) return EQMP_OK;
  const int bytes = dtype == EQMP_BF16 ? 2 : 4;
  const Plane in[] = {{q, q_ld}, {k, k_ld}, {v, v_ld}};
  void* const outs[] = {out};
  if (!q || !row_offsets || (E > 0 && (!src || (N_src > 0 && (!k || !v))))) return EQMP_ERR_INVALID_ARG;
  if (!planes_ok(in, 3, outs, 1, bytes) || !aligned(row_offsets, 4) || !aligned(src, 4) || !aligned(bias, 4) ||
      !aligned(stats, 4))
    return EQMP_ERR_INVALID_ARG;
  const int64_t ws = forward_workspace(n);
  if (ws > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < ws)) return EQMP_ERR_INVALID_ARG;
  const int64_t HD = (int64_t)H * D, HV = (int64_t)H * Dv;
  const Span reads[] = {span(in[0], N, HD, bytes), span(in[1], N_src, HD, bytes), span(in[2], N_src, HV, bytes),
                        span(row_offsets, (N + 1) * 4), span(src, E * 4), span(bias, E * H * 4)};
  const Span writes[] = {span(out, N * HV * bytes), span(stats, N * H * 8), span(workspace, ws)};
  if (!outputs_apart(reads, writes)) return EQMP_ERR_INVALID_ARG;
  AttnArgs a{};
  a.q = q, a.q_ld = q_ld, a.k = k, a.k_ld = k_ld, a.v = v, a.v_ld = v_ld;
  a.bias = bias, a.off = row_offsets, a.src = src;
  a.out = out, a.stats = stats, a.part = static_cast<float*>(workspace);
  a.scale = scale;
  a.N = (int)N, a.Ns = (int)N_src, a.E = (int)E, a.H = H, a.D = D, a.Dv = Dv;
  cut(E, forward_values(n), &a.block, &a.blocks);
  Alignment at;
  at.add(q, q_ld, bytes), at.add(k, k_ld, bytes), at.add(v, v_ld, bytes);
  at.add(out);
  at.bits |= (unsigned long long)D * bytes | (unsigned long long)Dv * bytes;
  const AttnForm f = form_of(n, N, N_src, bytes, at.bytes());
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return dtype == EQMP_BF16 ? launch_attn_fwd_bf16(a, f, st) : launch_attn_fwd_f32(a, f, st);
}

int64_t eqmp_edge_attention_backward_workspace_size(int64_t N, int64_t E, int64_t E_send, int32_t H, int32_t D, int32_t Dv) {
  const Sizes n{N, 0, E, H, D, Dv};
  if (check_sizes(n, EQMP_F32, 1.0f) != EQMP_OK || E_send < 0 || E_send > kMaxCount) return -1;
  return backward_workspace(n, E_send).total();
}

eqmp_status eqmp_edge_attention_backward(const void* grad_out, int64_t grad_out_ld, const void* q, int64_t q_ld,
                                         const void* k, int64_t k_ld, const void* v, int64_t v_ld, eqmp_dtype dtype,
                                         int64_t N, int64_t N_src, int64_t E, int32_t H, int32_t D, int32_t Dv,
                                         const int32_t* row_offsets, const int32_t* src, const int32_t* dst,
                                         const int32_t* send_offsets, const int32_t* send_edges, int64_t E_send,
                                         const float* bias, float scale, const float* stats, void* grad_q, void* grad_k,
                                         void* grad_v, float* grad_bias, void* workspace, int64_t workspace_bytes,
                                         eqmp_stream_t stream) {
  const Sizes n{N, N_src, E, H, D, Dv};
  const eqmp_status zs = check_sizes(n, dtype, scale);
  if (zs != EQMP_OK) return zs;
  if (E_send < 0) return EQMP_ERR_INVALID_ARG;
  if (E_send > kMaxCount) return EQMP_ERR_UNSUPPORTED;
  const bool send = (grad_k || grad_v) && N_src > 0;
  if (!grad_q && !send && !grad_bias) return EQMP_OK;
  const int bytes = dtype == EQMP_BF16 ? 2 : 4;
  const Plane in[] = {{q, q_ld}, {k, k_ld}, {v, v_ld}, {grad_out, grad_out_ld}};
  void* const outs[] = {grad_q, grad_k, grad_v};
  if (N > 0 && (!q || !grad_out || !stats || !row_offsets)) return EQMP_ERR_INVALID_ARG;
  if (N > 0 && E > 0 && (!src || (N_src > 0 && (!k || !v)))) return EQMP_ERR_INVALID_ARG;
  if (send && (!send_offsets || (E_send > 0 && (!send_edges || (E > 0 && !dst))))) return EQMP_ERR_INVALID_ARG;
  if (!planes_ok(in, 4, outs, 3, bytes)) return EQMP_ERR_INVALID_ARG;
  for (const void* p : {(const void*)row_offsets, (const void*)src, (const void*)dst, (const void*)send_offsets,
                        (const void*)send_edges, (const void*)bias, (const void*)stats, (const void*)grad_bias})
    if (!aligned(p, 4)) return EQMP_ERR_INVALID_ARG;
  const BackwardSpace ws = backward_workspace(n, E_send);
  if (ws.total() > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < ws.total())) return EQMP_ERR_INVALID_ARG;
  const int64_t HD = (int64_t)H * D, HV = (int64_t)H * Dv;
  const Span reads[] = {span(in[0], N, HD, bytes), span(in[1], N_src, HD, bytes), span(in[2], N_src, HV, bytes),
                        span(in[3], N, HV, bytes), span(row_offsets, (N + 1) * 4), span(src, E * 4), span(dst, E * 4),
                        span(send_offsets, (N_src + 1) * 4), span(send_edges, E_send * 4), span(bias, E * H * 4),
                        span(stats, N * H * 8)};
  const Span writes[] = {span(grad_q, N * HD * bytes), span(grad_k, N_src * HD * bytes), span(grad_v, N_src * HV * bytes),
                         span(grad_bias, E * H * 4), span(workspace, ws.total())};
  if (!outputs_apart(reads, writes)) return EQMP_ERR_INVALID_ARG;
  char* const space = static_cast<char*>(workspace);
  AttnArgs a{};
  a.q = q, a.q_ld = q_ld, a.k = k, a.k_ld = k_ld, a.v = v, a.v_ld = v_ld, a.g = grad_out, a.g_ld = grad_out_ld;
  a.bias = bias, a.off = row_offsets, a.src = src, a.dst = send ? dst : nullptr, a.send_off = send_offsets, a.send_edges = send_edges;
  a.stats = const_cast<float*>(stats);
  a.gq = grad_q, a.gk = grad_k, a.gv = grad_v, a.gbias = grad_bias;
  a.delta = reinterpret_cast<float*>(space + ws.pd);
  a.part = reinterpret_cast<float*>(space + ws.pd + ws.delta);
  a.scale = scale;
  a.N = (int)N, a.Ns = (int)N_src, a.E = (int)E, a.E_send = (int)E_send, a.H = H, a.D = D, a.Dv = Dv;
  a.pd = send || grad_bias ? reinterpret_cast<float2*>(space) : nullptr;
  Alignment at;
  at.add(q, q_ld, bytes), at.add(k, k_ld, bytes), at.add(v, v_ld, bytes), at.add(grad_out, grad_out_ld, bytes);
  at.add(grad_q), at.add(grad_k), at.add(grad_v);
  at.bits |= (unsigned long long)D * bytes | (unsigned long long)Dv * bytes;
  const bool bf16 = dtype == EQMP_BF16;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (N > 0) {
    cut(E, recv_values(n), &a.block, &a.blocks);
    const AttnForm f = form_of(n, N, N_src, bytes, at.bytes());
    const eqmp_status s = bf16 ? launch_attn_recv_bf16(a, f, st) : launch_attn_recv_f32(a, f, st);
    if (s != EQMP_OK) return s;
  }
  if (N == 0 && grad_bias && E > 0) {
    if (cudaMemsetAsync(grad_bias, 0, (size_t)E * H * 4, st) != cudaSuccess) return EQMP_ERR_CUDA;
    a.gbias = nullptr;
  }
  if (!send) return launch_attn_finish<float>(a, 0, st);
  cut(E_send, send_values(n), &a.block, &a.blocks);
  const AttnForm f = form_of(n, N_src, N, bytes, at.bytes());
  return bf16 ? launch_attn_send_bf16(a, f, st) : launch_attn_send_f32(a, f, st);
}

}  // extern "C"
