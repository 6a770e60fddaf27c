// Attention over a receiver's edges (sm_103a): arguments, the split of long rows
// and the kernels.
//
//   s[e,h] = scale q[i,h].k[src_e,h] + bias[e,h]           (e: src_e -> i)
//   m = max_e s,  z = sum_e exp(s - m),  p = exp(s - m) / z
//   out[i,h] = sum_e p v[src_e,h]
// Backward, with g = dL/dout:
//   dp = g[i,h].v[src_e,h],  delta[i,h] = sum_e p dp,  ds = p (dp - delta)
//   dq[i] = scale sum_e ds k,  dk[j] = scale sum_{src_e = j} ds q,
//   dv[j] = sum_{src_e = j} p g,  dbias = ds
// An edge with s = -inf is left out: nothing of its rows enters a sum.  A row
// with no edge left has m = z = 0, zeros as its result and no gradients.  A row
// with one edge left has its value as the result and no gradients but the
// value's: ds is exactly 0, not what rounding leaves of dp - delta.
// Scores, statistics and sums are fp32; bf16 is the storage of q, k, v, out and
// their gradients, rounded once on the store.  delta is summed from the row's
// own p and dp, not from the stored out, whose rounding would reach the fp32
// gradient of the bias.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace eqmp {

struct AttnArgs {
  const void *q, *k, *v, *g;  // [N][H][D], [Ns][H][D], [Ns][H][Dv], [N][H][Dv]
  long long q_ld, k_ld, v_ld, g_ld;
  const float* bias;  // [E][H] or NULL
  const int *off, *src;
  const int *dst, *send_off, *send_edges;  // backward: the sender view
  void* out;                               // [N][H][Dv]
  float* stats;                            // [N][H][2]: m and z, written forward, read backward
  void *gq, *gk, *gv;
  float* gbias;   // [E][H]
  float2* pd;     // backward scratch [E][H]: p and dp of an edge; p = -1: left out
  float* delta;   // backward scratch [N][H]
  float* part;    // partial sums of long rows, [2 * blocks][H][part_width]
  float scale;
  int N, Ns, E, E_send, H, D, Dv;
  int block, blocks;  // edges of a block of a long row, blocks in all (0: rows are not split)
  int rows_each;      // rows of a warp in the kernels of attn_ring.cuh
};

constexpr int kAttnWarps = 4;  // of a CTA, each with its own piece

// ---------------------------------------------------------------- long rows
// A row of more than two blocks is cut where the edge list is cut into blocks
// of `block` edges: its own warp takes the part up to the next multiple, and
// the warp of each block that begins inside the row takes that block.  So a
// node that is linked with all others is spread over the device.  The parts
// lie in slots that no two pieces share: slot c for the block c that begins
// inside a long row, slot blocks + c for the long row that begins inside block
// c (there is at most one, since it is longer than a block).  k_attn_join adds
// them in the order of the edges.
struct Piece {
  int row, e0, e1;
  int slot;  // -1: a whole row
};

struct Rows {
  const int* off;
  int n, E, block, blocks;
};

__device__ __forceinline__ int clamped(int v, int hi) { return min(max(v, 0), hi); }

__device__ __forceinline__ bool is_long(const Rows& r, int e0, int e1) { return r.blocks && e1 - e0 > 2 * r.block; }

// The last row that begins at or before edge x (-1: none), by a warp: each round
// the lanes probe 32 places of what is left.  Ends whatever the offsets hold.
__device__ __forceinline__ int row_of_edge(const Rows& r, int x) {
  int lo = -1, hi = r.n;  // off[lo] <= x < off[hi], in words
  const int lane = threadIdx.x & 31;
  while (hi - lo > 1) {
    const long long d = (long long)hi - lo - 1;
    const int p = lo + 1 + (int)(d * lane / 32);
    const unsigned le = __ballot_sync(0xffffffffu, __ldg(r.off + p) <= x);
    const int n = le ? 32 - __clz(le) : 0;  // the last probe that holds
    const int at = __shfl_sync(0xffffffffu, p, n ? n - 1 : 0), next = __shfl_sync(0xffffffffu, p, n < 32 ? n : 31);
    if (n < 32) hi = next;
    if (n) lo = at;
  }
  return lo;
}

// The piece of worker w: the blocks first, then a row each.  row < 0: nothing.
__device__ __forceinline__ Piece find_piece(const Rows& r, int w) {
  Piece t;
  t.row = -1;
  t.slot = -1;
  t.e0 = t.e1 = 0;
  if (w >= r.blocks) {
    const int row = w - r.blocks;
    if (row >= r.n) return t;
    t.row = row;
    t.e0 = clamped(__ldg(r.off + row), r.E);
    t.e1 = max(t.e0, clamped(__ldg(r.off + row + 1), r.E));
    if (is_long(r, t.e0, t.e1)) {
      t.slot = r.blocks + t.e0 / r.block;
      t.e1 = min(t.e1, (t.e0 / r.block + 1) * r.block);
    }
    return t;
  }
  const int x = w * r.block, row = row_of_edge(r, x);
  if (row < 0) return t;
  const int e0 = clamped(__ldg(r.off + row), r.E), e1 = clamped(__ldg(r.off + row + 1), r.E);
  if (!is_long(r, e0, e1) || e0 >= x || e1 <= x) return t;
  t.row = row;
  t.slot = w;
  t.e0 = x;
  t.e1 = min(e1, x + r.block);
  return t;
}

// ---------------------------------------------------------------- vectors
// V elements of T at a time.
template <typename T, int V>
struct Vec;

template <typename T>
struct Vec<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p, bool ok) { v = ok ? *p : T(0.0f); }
  __device__ __forceinline__ void zero() { v = T(0.0f); }
  __device__ __forceinline__ void get(float (&f)[1]) const { f[0] = (float)v; }
  static __device__ __forceinline__ void store(float* p, const float* f) { *p = *f; }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) { *p = __float2bfloat16_rn(*f); }
};

// A lane's share of a head's row of `cols` values: vectors l, l + G, ...
template <typename T, int V, int G, int NV>
struct Frag {
  Vec<T, V> v[NV];
  __device__ __forceinline__ void load(const T* row, int l, int cols, bool ok) {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j].load(row + (j * G + l) * V, ok && (j * G + l) * V < cols);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int j = 0; j < NV; ++j) v[j].zero();
  }
  __device__ __forceinline__ float dot(const float (&with)[NV * V]) const {
    float t = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V];
      v[j].get(f);
#pragma unroll
      for (int i = 0; i < V; ++i) t = fmaf(f[i], with[j * V + i], t);
    }
    return t;
  }
  __device__ __forceinline__ void add_to(float (&acc)[NV * V], float by) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V];
      v[j].get(f);
#pragma unroll
      for (int i = 0; i < V; ++i) acc[j * V + i] = fmaf(by, f[i], acc[j * V + i]);
    }
  }
  __device__ __forceinline__ void values(float (&to)[NV * V], float by) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[V];
      v[j].get(f);
#pragma unroll
      for (int i = 0; i < V; ++i) to[j * V + i] = f[i] * by;
    }
  }
};

template <typename T, int V, int G, int NV>
__device__ __forceinline__ void store_share(T* row, int l, int cols, const float (&x)[NV * V], float by) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if ((j * G + l) * V >= cols) break;
    float f[V];
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = x[j * V + i] * by;
    Vec<T, V>::store(row + (j * G + l) * V, f);
  }
}

template <int V, int G, int NV>
__device__ __forceinline__ void store_part(float* row, int l, int cols, const float (&x)[NV * V]) {
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = (j * G + l) * V + i;
      if (c < cols) row[c] = x[j * V + i];
    }
}

// The sum of each of U values over the G lanes of a head; every lane gets it.
template <int G, int U>
__device__ __forceinline__ void head_sum(float (&t)[U]) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
    for (int u = 0; u < U; ++u) t[u] += __shfl_xor_sync(0xffffffffu, t[u], o);
}

#define EQMP_NEG_INF __int_as_float(0xff800000)

// ---------------------------------------------------------------- forward
// The general kernels: rows whose heads begin anywhere (bf16), and long heads of
// odd sizes, value by value.  Bound by the latency of one batch after the other:
// 100,000 atoms, 8 heads of 32 + 128 fp32 values, 2237 us forward with vectors of
// 16 bytes, which the rings of attn_ring.cuh have taken over since.
// One warp per piece of a row and 32 / G heads; G lanes hold a head's query and
// its sum in registers, and the edges' keys and values pass once, U edges at a
// time, with the running maximum and sum of a softmax.
template <typename T, int V, int G, int KN, int VN, int U>
__global__ void __launch_bounds__(32 * kAttnWarps) k_attn_fwd(AttnArgs a) {
  const Rows rows{a.off, a.N, a.E, a.block, a.blocks};
  const Piece t = find_piece(rows, blockIdx.x * kAttnWarps + (threadIdx.x >> 5));
  if (t.row < 0) return;
  const int lane = threadIdx.x & 31, l = lane % G, h = blockIdx.y * (32 / G) + lane / G;
  const bool mine = h < a.H;
  const T* k = static_cast<const T*>(a.k) + (long long)h * a.D;
  const T* v = static_cast<const T*>(a.v) + (long long)h * a.Dv;
  float q[KN * V], acc[VN * V], m = EQMP_NEG_INF, z = 0.0f;
  {
    Frag<T, V, G, KN> f;
    f.load(static_cast<const T*>(a.q) + t.row * a.q_ld + (long long)h * a.D, l, a.D, mine);
    f.values(q, a.scale);
  }
#pragma unroll
  for (int i = 0; i < VN * V; ++i) acc[i] = 0.0f;
  for (int e = t.e0; e < t.e1; e += 32) {
    const int my_src = e + lane < t.e1 ? __ldg(a.src + e + lane) : -1;
    const int n = min(32, t.e1 - e);
    for (int b = 0; b < n; b += U) {
      Frag<T, V, G, KN> kf[U];
      Frag<T, V, G, VN> vf[U];
      float s[U], bias[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = __shfl_sync(0xffffffffu, my_src, b + u);
        const bool ok = mine && (unsigned)j < (unsigned)a.Ns;
        kf[u].load(k + j * a.k_ld, l, a.D, ok);
        vf[u].load(v + j * a.v_ld, l, a.Dv, ok);
        bias[u] = b + u >= n ? EQMP_NEG_INF : a.bias && mine ? __ldg(a.bias + (long long)(e + b + u) * a.H + h) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] = kf[u].dot(q);
      head_sum<G, U>(s);
      float top = m;
      bool left_out = false;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u] = bias[u] == EQMP_NEG_INF ? EQMP_NEG_INF : s[u] + bias[u];
        left_out |= s[u] == EQMP_NEG_INF;
        top = fmaxf(top, s[u]);
      }
      if (__any_sync(0xffffffffu, left_out))
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (s[u] == EQMP_NEG_INF) vf[u].zero();  // a weight of 0 would keep a NaN
      const float base = top == EQMP_NEG_INF ? 0.0f : top, keep = __expf(m - base);
      m = top;
      z *= keep;
#pragma unroll
      for (int i = 0; i < VN * V; ++i) acc[i] *= keep;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float p = __expf(s[u] - base);
        z += p;
        vf[u].add_to(acc, p);
      }
    }
  }
  if (!mine) return;
  if (t.slot >= 0) {
    float* to = a.part + ((long long)t.slot * a.H + h) * (a.Dv + 2);
    if (l == 0) to[0] = m, to[1] = z;
    store_part<V, G, VN>(to + 2, l, a.Dv, acc);
    return;
  }
  const long long at = (long long)t.row * a.H + h;
  if (a.stats && l == 0) {
    a.stats[2 * at] = z == 0.0f ? 0.0f : m;
    a.stats[2 * at + 1] = z;
  }
  if (a.out) store_share<T, V, G, VN>(static_cast<T*>(a.out) + at * a.Dv, l, a.Dv, acc, z == 0.0f ? 0.0f : 1.0f / z);
}

// ---------------------------------------------------------------- backward
// sum_e ds k from pdk = sum_e p dp k and pk = sum_e p k.  For the only edge of a row ds is 0, and 0 k is formed, so that a
// NaN, or an infinity in dp, is kept.
__device__ __forceinline__ float query_sum(bool alone, float delta, float pdk, float pk) {
  return fmaf(alone ? delta - delta : -delta, pk, alone ? 0.0f : pdk);
}

// The receivers' pass: p and dp of each edge from one reading of its key and
// value, and dq without a second one:
//   dq = scale (sum_e p dp k  -  delta sum_e p k)
template <typename T, int V, int G, int KN, int VN, int U>
__global__ void __launch_bounds__(32 * kAttnWarps) k_attn_bwd_recv(AttnArgs a) {
  const Rows rows{a.off, a.N, a.E, a.block, a.blocks};
  const Piece t = find_piece(rows, blockIdx.x * kAttnWarps + (threadIdx.x >> 5));
  if (t.row < 0) return;
  const int lane = threadIdx.x & 31, l = lane % G, h = blockIdx.y * (32 / G) + lane / G;
  const bool mine = h < a.H;
  const T* k = static_cast<const T*>(a.k) + (long long)h * a.D;
  const T* v = static_cast<const T*>(a.v) + (long long)h * a.Dv;
  const long long at = (long long)t.row * a.H + h;
  float q[KN * V], g[VN * V], pdk[KN * V], pk[KN * V], delta = 0.0f, dps = 0.0f;
  int live = 0;
  {
    Frag<T, V, G, KN> f;
    f.load(static_cast<const T*>(a.q) + t.row * a.q_ld + (long long)h * a.D, l, a.D, mine);
    f.values(q, a.scale);
    Frag<T, V, G, VN> fg;
    fg.load(static_cast<const T*>(a.g) + t.row * a.g_ld + (long long)h * a.Dv, l, a.Dv, mine);
    fg.values(g, 1.0f);
  }
  const float m = mine ? a.stats[2 * at] : 0.0f, z = mine ? a.stats[2 * at + 1] : 0.0f, rz = 1.0f / z;
#pragma unroll
  for (int i = 0; i < KN * V; ++i) pdk[i] = pk[i] = 0.0f;
  for (int e = t.e0; e < t.e1; e += 32) {
    const int my_src = e + lane < t.e1 ? __ldg(a.src + e + lane) : -1;
    const int n = min(32, t.e1 - e);
    for (int b = 0; b < n; b += U) {
      Frag<T, V, G, KN> kf[U];
      Frag<T, V, G, VN> vf[U];
      float s[2 * U], bias[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = __shfl_sync(0xffffffffu, my_src, b + u);
        const bool ok = mine && (unsigned)j < (unsigned)a.Ns;
        kf[u].load(k + j * a.k_ld, l, a.D, ok);
        vf[u].load(v + j * a.v_ld, l, a.Dv, ok);
        bias[u] = b + u >= n ? EQMP_NEG_INF : a.bias && mine ? __ldg(a.bias + (long long)(e + b + u) * a.H + h) : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u] = kf[u].dot(q);
        s[U + u] = vf[u].dot(g);
      }
      head_sum<G, 2 * U>(s);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        s[u] = bias[u] == EQMP_NEG_INF ? EQMP_NEG_INF : s[u] + bias[u];
        const bool left_out = s[u] == EQMP_NEG_INF || z == 0.0f;
        if (__any_sync(0xffffffffu, left_out) && left_out) kf[u].zero();  // a weight of 0 would keep a NaN
        const float p = left_out ? 0.0f : __expf(s[u] - m) * rz, dp = left_out ? 0.0f : s[U + u];
        if (a.pd && l == 0 && mine && b + u < n)
          a.pd[(long long)(e + b + u) * a.H + h] = make_float2(left_out ? -1.0f : p, dp);
        delta = fmaf(p, dp, delta);
        dps += dp;
        live += !left_out;
        kf[u].add_to(pdk, p * dp);
        kf[u].add_to(pk, p);
      }
    }
  }
  if (!mine) return;
  const bool alone = live == 1;  // the row's only edge: its weight is 1, whatever its score
  if (t.slot >= 0) {
    float* to = a.part + ((long long)t.slot * a.H + h) * (2 * a.D + 3);
    if (l == 0) to[0] = delta, to[1] = dps, to[2] = live;
    store_part<V, G, KN>(to + 3, l, a.D, pdk);
    store_part<V, G, KN>(to + 3 + a.D, l, a.D, pk);
    return;
  }
  if (alone) delta = dps;
  if (a.delta && l == 0) a.delta[at] = delta;
  if (a.gq) {
#pragma unroll
    for (int i = 0; i < KN * V; ++i) pdk[i] = query_sum(alone, delta, pdk[i], pk[i]);
    store_share<T, V, G, KN>(static_cast<T*>(a.gq) + at * a.D, l, a.D, pdk, a.scale);
  }
}

// The receiver of an edge for the senders' pass.  Edges before the first row or behind the last (lists of fixed length, a
// range of receivers) have none, whatever dst holds: the receivers' pass has not written their p and dp.
struct Receivers {
  const int* dst;
  unsigned first, count;  // the edges of the rows
  __device__ __forceinline__ explicit Receivers(const AttnArgs& a) : dst(a.dst), first(0), count(0) {
    if (a.N == 0) return;
    const int lo = clamped(__ldg(a.off), a.E), hi = clamped(__ldg(a.off + a.N), a.E);
    first = lo, count = max(hi - lo, 0);
  }
  __device__ __forceinline__ int of(int edge) const { return (unsigned)edge - first < count ? __ldg(dst + edge) : -1; }
};

// The senders' pass: each sender's dk and dv from the p and dp of its edges and
// the rows of their receivers, in the order of the sender view.
template <typename T, int V, int G, int KN, int VN, int U>
__global__ void __launch_bounds__(32 * kAttnWarps) k_attn_bwd_send(AttnArgs a) {
  const Rows rows{a.send_off, a.Ns, a.E_send, a.block, a.blocks};
  const Piece t = find_piece(rows, blockIdx.x * kAttnWarps + (threadIdx.x >> 5));
  if (t.row < 0) return;
  const int lane = threadIdx.x & 31, l = lane % G, h = blockIdx.y * (32 / G) + lane / G;
  const bool mine = h < a.H;
  const T* q = static_cast<const T*>(a.q) + (long long)h * a.D;
  const T* g = static_cast<const T*>(a.g) + (long long)h * a.Dv;
  float gk[KN * V], gv[VN * V];
#pragma unroll
  for (int i = 0; i < KN * V; ++i) gk[i] = 0.0f;
#pragma unroll
  for (int i = 0; i < VN * V; ++i) gv[i] = 0.0f;
  const Receivers receivers(a);
  for (int c = t.e0; c < t.e1; c += 32) {
    const int my_edge = c + lane < t.e1 ? __ldg(a.send_edges + c + lane) : -1;
    const int my_dst = receivers.of(my_edge);
    const int n = min(32, t.e1 - c);
    for (int b = 0; b < n; b += U) {
      Frag<T, V, G, KN> qf[U];
      Frag<T, V, G, VN> gf[U];
      float2 pd[U];
      float delta[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int edge = __shfl_sync(0xffffffffu, my_edge, b + u), i = __shfl_sync(0xffffffffu, my_dst, b + u);
        const bool ok = mine && (unsigned)i < (unsigned)a.N;
        qf[u].load(q + i * a.q_ld, l, a.D, ok);
        gf[u].load(g + i * a.g_ld, l, a.Dv, ok);
        pd[u] = ok ? a.pd[(long long)edge * a.H + h] : make_float2(-1.0f, 0.0f);
        delta[u] = ok ? a.delta[(long long)i * a.H + h] : 0.0f;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool left_out = pd[u].x < 0.0f;
        if (__any_sync(0xffffffffu, left_out) && left_out) {
          qf[u].zero();
          gf[u].zero();
        }
        const float p = left_out ? 0.0f : pd[u].x, ds = left_out ? 0.0f : p * (pd[u].y - delta[u]);
        qf[u].add_to(gk, ds);
        gf[u].add_to(gv, p);
      }
    }
  }
  if (!mine) return;
  if (t.slot >= 0) {
    float* to = a.part + ((long long)t.slot * a.H + h) * (a.D + a.Dv);
    store_part<V, G, KN>(to, l, a.D, gk);
    store_part<V, G, VN>(to + a.D, l, a.Dv, gv);
    return;
  }
  const long long at = (long long)t.row * a.H + h;
  if (a.gk) store_share<T, V, G, KN>(static_cast<T*>(a.gk) + at * a.D, l, a.D, gk, a.scale);
  if (a.gv) store_share<T, V, G, VN>(static_cast<T*>(a.gv) + at * a.Dv, l, a.Dv, gv, 1.0f);
}

// ---------------------------------------------------------------- joining
// The parts of long rows.  A CTA looks at kJoinBlocks blocks, a lane each: a row
// is joined where the first block that begins inside it is found.  For each such
// row and head threadIdx.x then goes over the columns, threadIdx.y over the parts.
// (Where no row is long, the search is all of it.  By a warp for each block and
// head it was 6.6 M instructions and 12 us on its own at 60,000 rows.)
enum { kJoinFwd, kJoinRecv, kJoinSend };
constexpr int kJoinX = 32, kJoinY = 8, kJoinBlocks = 16;

template <int MODE, typename T>
__device__ void join_row(const AttnArgs& a, int first, int last, int row, int h, float (&red)[kJoinY][kJoinX]) {
  const int x = threadIdx.x, y = threadIdx.y;
  const int width = MODE == kJoinFwd ? a.Dv + 2 : MODE == kJoinRecv ? 2 * a.D + 3 : a.D + a.Dv;
  // part 0: the row's beginning, in the slot of the block where it lies; then the blocks
  auto part = [&](int i) { return a.part + ((long long)(i ? first + i - 1 : a.blocks + first - 1) * a.H + h) * width; };
  const int parts = last - first + 2;
  const long long at = (long long)row * a.H + h;
  auto over_y = [&](float v, bool max) {  // every thread gets its column's
    __syncthreads();
    red[y][x] = v;
    __syncthreads();
    float t = red[0][x];
#pragma unroll
    for (int i = 1; i < kJoinY; ++i) t = max ? fmaxf(t, red[i][x]) : t + red[i][x];
    return t;
  };
  if constexpr (MODE == kJoinFwd) {
    float m = EQMP_NEG_INF, z = 0.0f;
    for (int i = y; i < parts; i += kJoinY) m = fmaxf(m, part(i)[0]);
    m = over_y(m, true);
    const float base = m == EQMP_NEG_INF ? 0.0f : m;
    for (int i = y; i < parts; i += kJoinY) z += part(i)[1] * __expf(part(i)[0] - base);
    z = over_y(z, false);
    if (a.stats && x == 0 && y == 0) {
      a.stats[2 * at] = z == 0.0f ? 0.0f : m;
      a.stats[2 * at + 1] = z;
    }
    if (!a.out) return;
    for (int col = x; col - x < a.Dv; col += kJoinX) {
      float t = 0.0f;
      if (col < a.Dv)
        for (int i = y; i < parts; i += kJoinY) t = fmaf(part(i)[2 + col], __expf(part(i)[0] - base), t);
      t = over_y(t, false);
      if (y == 0 && col < a.Dv) {
        t = z == 0.0f ? 0.0f : t / z;
        Vec<T, 1>::store(static_cast<T*>(a.out) + at * a.Dv + col, &t);
      }
    }
  } else if constexpr (MODE == kJoinRecv) {
    float delta = 0.0f, dps = 0.0f, live = 0.0f;
    for (int i = y; i < parts; i += kJoinY) delta += part(i)[0], dps += part(i)[1], live += part(i)[2];
    delta = over_y(delta, false);
    dps = over_y(dps, false);
    const bool alone = over_y(live, false) == 1.0f;  // the row's only edge, all others left out
    if (alone) delta = dps;
    if (a.delta && x == 0 && y == 0) a.delta[at] = delta;
    if (!a.gq) return;
    for (int col = x; col - x < a.D; col += kJoinX) {
      float t = 0.0f, s = 0.0f;
      if (col < a.D)
        for (int i = y; i < parts; i += kJoinY) {
          t += part(i)[3 + col];
          s += part(i)[3 + a.D + col];
        }
      t = over_y(t, false);
      s = over_y(s, false);
      t = a.scale * query_sum(alone, delta, t, s);
      if (y == 0 && col < a.D) Vec<T, 1>::store(static_cast<T*>(a.gq) + at * a.D + col, &t);
    }
  } else {
    for (int col = x; col - x < a.D + a.Dv; col += kJoinX) {
      float t = 0.0f;
      if (col < a.D + a.Dv)
        for (int i = y; i < parts; i += kJoinY) t += part(i)[col];
      t = over_y(t, false);
      if (y || col >= a.D + a.Dv) continue;
      if (col < a.D) {
        t *= a.scale;
        if (a.gk) Vec<T, 1>::store(static_cast<T*>(a.gk) + at * a.D + col, &t);
      } else if (a.gv) {
        Vec<T, 1>::store(static_cast<T*>(a.gv) + at * a.Dv + col - a.D, &t);
      }
    }
  }
}

// The blocks of CTA x of the join, for the heads y, y + ny, ...
template <int MODE, typename T>
__device__ __forceinline__ void join_blocks(const AttnArgs& a, int x, int y, int ny) {
  __shared__ float red[kJoinY][kJoinX];
  __shared__ int range[kJoinBlocks][3];
  const Rows rows = MODE == kJoinSend ? Rows{a.send_off, a.Ns, a.E_send, a.block, a.blocks}
                                      : Rows{a.off, a.N, a.E, a.block, a.blocks};
  if (threadIdx.y == 0 && threadIdx.x < kJoinBlocks) {
    const int c = x * kJoinBlocks + threadIdx.x, at = c * rows.block;
    int first = -1, last = -1, row = -1, past = rows.n;  // off[row] <= at < off[past], in words
    if (c < rows.blocks) {
      while (past - row > 1) {
        const int mid = row + (past - row) / 2;
        if (__ldg(rows.off + mid) <= at)
          row = mid;
        else
          past = mid;
      }
      if (row >= 0) {
        const int e0 = clamped(__ldg(rows.off + row), rows.E), e1 = clamped(__ldg(rows.off + row + 1), rows.E);
        if (is_long(rows, e0, e1) && e0 < at && at < e1 && e0 / rows.block == c - 1) first = c, last = (e1 - 1) / rows.block;
      }
    }
    range[threadIdx.x][0] = first, range[threadIdx.x][1] = last, range[threadIdx.x][2] = row;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");  // until the kernel that writes the parts is done
  __syncthreads();
  for (int i = 0; i < kJoinBlocks; ++i) {
    if (range[i][0] < 0) continue;
    for (int h = y; h < a.H; h += ny) join_row<MODE, T>(a, range[i][0], range[i][1], range[i][2], h, red);
  }
}

template <int MODE, typename T>
__global__ void __launch_bounds__(kJoinX * kJoinY) k_attn_join(const __grid_constant__ AttnArgs a) {
  join_blocks<MODE, T>(a, blockIdx.x, blockIdx.y, gridDim.y);
}

// dbias = ds, from the p and dp of the receivers' pass: a warp for 32 edges and all their heads.  It goes by the rows and
// not by the sender view, which need not list an edge whose sender is none, nor one that lies outside every row: those
// are written too, the latter as 0.  Bound by the latency of its loads: 10,000 atoms of 48 edges, 8 heads, the whole
// backward pass 449 us with eight items on their way together, 459 with each load behind the last store (442 where the
// senders' pass wrote what its view lists, which left edges out).
constexpr int kFinishEdges = 32 * kJoinY;  // of a CTA

// The row that holds the lane's edge (-1: none): dst where it is right, else searched for between the rows of the warp's
// first and last edge.
__device__ __forceinline__ int row_of_lane(const AttnArgs& a, int first, int e, int last) {
  auto holds = [&](int row) { return (unsigned)row < (unsigned)a.N && __ldg(a.off + row) <= e && e < __ldg(a.off + row + 1); };
  int row = a.dst ? __ldg(a.dst + e) : -1;
  if (__all_sync(0xffffffffu, holds(row))) return row;
  const Rows rows{a.off, a.N, a.E, 0, 0};
  row = row_of_edge(rows, first);
  int past = row_of_edge(rows, last) + 1;  // off[row] <= e < off[past], in words
  while (past - row > 1) {
    const int mid = row + (past - row) / 2;
    if (__ldg(a.off + mid) <= e)
      row = mid;
    else
      past = mid;
  }
  return holds(row) ? row : -1;
}

__device__ __forceinline__ void bias_of_edges(const AttnArgs& a, int x) {
  const int lane = threadIdx.x, e0 = (x * kJoinY + threadIdx.y) * 32, n = min(32, a.E - e0);
  const int row = n > 0 ? row_of_lane(a, e0, e0 + min(lane, n - 1), e0 + n - 1) : -1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long first = (long long)e0 * a.H;
  const int items = n * a.H, step_t = 32 / a.H, step_h = 32 % a.H;
  int t = lane / a.H, h = lane % a.H;  // of the lane's item: the edge and the head
  constexpr int AHEAD = 8;             // items on their way together
  for (int i = lane; i - lane < items; i += 32 * AHEAD) {
    float2 pd[AHEAD];
    float delta[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int r = __shfl_sync(0xffffffffu, row, t & 31);
      const bool in = i + 32 * k < items && r >= 0;
      pd[k] = in ? a.pd[first + i + 32 * k] : make_float2(-1.0f, 0.0f);
      delta[k] = in ? a.delta[(long long)r * a.H + h] : 0.0f;
      t += step_t;
      h += step_h;
      if (h >= a.H) h -= a.H, ++t;
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (i + 32 * k < items) a.gbias[first + i + 32 * k] = pd[k].x < 0.0f ? 0.0f : pd[k].x * (pd[k].y - delta[k]);
  }
}

// The end of the backward pass: the long rows of the senders, `joins` CTAs of the first, and dbias.  One launch for both:
// 1001 atoms with a hub 40 us a call, 43 with two.
template <typename T>
__global__ void __launch_bounds__(kJoinX * kJoinY) k_attn_finish(const __grid_constant__ AttnArgs a, int joins, int ny) {
  if ((int)blockIdx.x < joins)
    join_blocks<kJoinSend, T>(a, blockIdx.x / ny, blockIdx.x % ny, ny);
  else
    bias_of_edges(a, blockIdx.x - joins);
}

}  // namespace eqmp
