// The attention kernels for rows whose heads all begin on 16, 8 or 4 bytes
// (VB; sm_103a).
//
// A warp takes 32 / G heads of a few neighbouring rows and walks over their
// edges, U at a time.  The edges' rows come through a ring in shared memory by
// asynchronous copies, STAGES - 1 batches ahead and across the ends of rows, so
// that neither the indices nor the rows are waited for; a lane copies just the
// bytes that it will read itself.  Places of a batch behind its row's end are
// filled with zeros.
//
// The gather binds.  100,000 atoms, 19 edges each, 8 heads of 32 + 128 fp32 values
// (9.8 GB of rows an edge list through L2): atoms in the order of their cells 630
// us forward (15 TB/s), 724 and 715 the two passes backward (the latter with the
// bias's gradient); in no order 1110 us, by DRAM (a third of the rows hits L2).
// 10,000 atoms, 48 edges each, 8 heads of 32 + 256 bf16 values: 193, 231 and 218 us,
// with 48 to 56 % of the issue slots at 9 warps an SM, which is what shared memory
// has room for.
#pragma once

#include "attn.cuh"

namespace eqmp {

// Of a CTA: with one, as many rings fit an SM as there is shared memory for (10,000
// atoms, bf16, values of 256: forward 205 us, with two 239, with four 253).
constexpr int kRingWarps = 1;

template <int N>
__device__ __forceinline__ void copy_row(uint32_t to, const void* from, int bytes) {  // N bytes, or 0 for zeros
  if constexpr (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(bytes) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(to), "l"(from), "n"(N), "r"(bytes) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_async(uint32_t to, const void* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(N) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ float4 lds128(uint32_t at) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float2 lds64(uint32_t at) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ float lds32(uint32_t at) {
  float v;
  asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
  return v;
}

// VB bytes of a row, and their values as pairs (a single fp32 value with a zero).
template <int VB>
struct RawOf;
template <>
struct RawOf<16> {
  using type = float4;
  static __device__ __forceinline__ float4 lds(uint32_t at) { return lds128(at); }
};
template <>
struct RawOf<8> {
  using type = float2;
  static __device__ __forceinline__ float2 lds(uint32_t at) { return lds64(at); }
};
template <>
struct RawOf<4> {
  using type = float;
  static __device__ __forceinline__ float lds(uint32_t at) { return lds32(at); }
};

template <typename T, int VB>
struct RowVec {
  using Raw = typename RawOf<VB>::type;
  static constexpr int EL = VB / sizeof(T), PAIRS = (EL + 1) / 2;
};

__device__ __forceinline__ float word_of(const float4& v, int i) { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
__device__ __forceinline__ float word_of(const float2& v, int i) { return i == 0 ? v.x : v.y; }
__device__ __forceinline__ float word_of(const float& v, int) { return v; }

template <typename T, int VB>
__device__ __forceinline__ void pairs_of(const typename RowVec<T, VB>::Raw& v, float2 (&f)[RowVec<T, VB>::PAIRS]) {
#pragma unroll
  for (int i = 0; i < RowVec<T, VB>::PAIRS; ++i) {
    if constexpr (sizeof(T) == 2) {
      const uint32_t b = __float_as_uint(word_of(v, i));
      f[i] = make_float2(__uint_as_float(b << 16), __uint_as_float(b & 0xffff0000u));
    } else {
      f[i] = make_float2(word_of(v, 2 * i), VB == 4 ? 0.0f : word_of(v, 2 * i + 1));
    }
  }
}

// What a worker does: n rows from `row` on; lane i < n holds the edges and the
// slot of the i-th (see Piece).
struct Work {
  int row, n;
  int e0, e1, slot;
};

__device__ __forceinline__ Work find_work(const Rows& r, int w, int rows_each) {
  const int lane = threadIdx.x & 31;
  Work t{0, 0, 0, 0, -1};
  if (w < r.blocks) {
    const Piece p = find_piece(r, w);
    if (p.row < 0) return t;
    return Work{p.row, 1, p.e0, p.e1, p.slot};
  }
  const long long first = (long long)(w - r.blocks) * rows_each;
  if (first >= r.n) return t;
  t.row = (int)first;
  t.n = min(rows_each, r.n - t.row);
  if (lane < t.n) {
    t.e0 = clamped(__ldg(r.off + t.row + lane), r.E);
    t.e1 = max(t.e0, clamped(__ldg(r.off + t.row + lane + 1), r.E));
    if (is_long(r, t.e0, t.e1)) {
      t.slot = r.blocks + t.e0 / r.block;
      t.e1 = min(t.e1, (t.e0 / r.block + 1) * r.block);
    }
  }
  return t;
}

// The batches of a worker's edges in order: its rows' edges U at a time.
struct Walk {
  int i, e, end;  // the row, the batch's first edge, the row's end
  __device__ __forceinline__ void start(const Work& w) {
    i = -1;
    e = end = 0;
    next_row(w);
  }
  __device__ __forceinline__ void next_row(const Work& w) {
    while (e >= end && ++i < w.n) {
      e = __shfl_sync(0xffffffffu, w.e0, i);
      end = __shfl_sync(0xffffffffu, w.e1, i);
    }
  }
  __device__ __forceinline__ bool over(const Work& w) const { return i >= w.n; }
};

// Values of consecutive places of an index list, a lane each, loaded 32 places
// ahead; a jump in the list loads anew.
struct Ahead {
  int c, now, next;
  __device__ __forceinline__ int load(const int* list, int at, int n) const {
    return at < n ? __ldg(list + at) : -1;
  }
  __device__ __forceinline__ void start(const int* list, int e, int n) {
    const int lane = threadIdx.x & 31;
    c = e;
    now = load(list, e + lane, n);
    next = load(list, e + 32 + lane, n);
  }
  __device__ __forceinline__ void to(const int* list, int e, int n) {
    if (e - c < 32) return;
    if (e - c >= 64) {
      start(list, e, n);
      return;
    }
    c += 32;
    now = next;
    next = load(list, c + 32 + (threadIdx.x & 31), n);
  }
  // lane t gets the value of place e + t; e is at most 31 behind c
  __device__ __forceinline__ int from(int e) const {
    const int at = e - c + (threadIdx.x & 31);
    const int a = __shfl_sync(0xffffffffu, now, at & 31), b = __shfl_sync(0xffffffffu, next, at & 31);
    return at < 32 ? a : b;
  }
};

// The sums over the G lanes of a head of NV values (a power of two up to G):
// lane l gets that of value l % NV.
template <int G, int NV>
__device__ __forceinline__ float scatter_sum(float (&v)[NV], int l) {
#pragma unroll
  for (int half = NV / 2; half > 0; half /= 2) {
    const bool upper = l & half;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = upper ? v[i] : v[i + half], keep = upper ? v[i + half] : v[i];
      v[i] = keep + __shfl_xor_sync(0xffffffffu, send, half);
    }
  }
#pragma unroll
  for (int o = NV; o < G; o *= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
  return v[0];
}

// The shape of a ring: U edges a batch, each of KN + VN vectors a lane, and per
// batch a few bytes for every edge and head.
// Two stages of 5 to 10 KB leave room for 10 to 20 warps on an SM.  Measured, forward:
// 100,000 atoms in the order of their cells, fp32, 8 heads of 32 + 128: 2 edges and 2
// stages 630 us, 2 and 3 697, 4 and 2 727, 4 and 3 1049; 10,000 atoms of 48 edges, bf16,
// 8 heads of 32 + 256: 4 and 2 191, 2 and 2 203, 2 and 3 229.
template <int VB, int G, int KN, int VN, int U_, int SMALL>
struct RingShape {
  static constexpr int VECS = KN + VN;
  static constexpr int U = U_;
  static constexpr int HEADS = 32 / G;
  static constexpr int VEC = 32 * VB;  // a vector of every lane
  static constexpr int SMALL_AT = U * VECS * VEC;
  static constexpr int BATCH = SMALL_AT + (U * HEADS * SMALL + 31) / 32 * 32;
  static constexpr int STAGES = 2;
  static constexpr int WARP = STAGES * BATCH;
  static constexpr int CTA = kRingWarps * WARP;
};

template <typename T, int VB, int G, int NV>
__device__ __forceinline__ void load_row(const T* row, int l, int cols, bool ok, typename RowVec<T, VB>::Raw (&v)[NV]) {
  using Raw = typename RowVec<T, VB>::Raw;
  constexpr int EL = RowVec<T, VB>::EL;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    v[j] = ok && (j * G + l) * EL < cols ? __ldg(reinterpret_cast<const Raw*>(row + (j * G + l) * EL)) : Raw{};
}

template <typename T, int VB, int NV>
__device__ __forceinline__ void unpack(const typename RowVec<T, VB>::Raw (&v)[NV], float by, float2 (&f)[NV * RowVec<T, VB>::PAIRS]) {
  constexpr int P = RowVec<T, VB>::PAIRS;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float2 p[P];
    pairs_of<T, VB>(v[j], p);
#pragma unroll
    for (int i = 0; i < P; ++i) f[j * P + i] = make_float2(p[i].x * by, p[i].y * by);
  }
}

// sum += by * the lane's vectors at `at`.
template <typename T, int VB, int NV>
__device__ __forceinline__ void add_row(uint32_t at, float by, float2 (&sum)[NV * RowVec<T, VB>::PAIRS]) {
  constexpr int P = RowVec<T, VB>::PAIRS;
  const float2 b = make_float2(by, by);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float2 p[P];
    pairs_of<T, VB>(RawOf<VB>::lds(at + j * 32 * VB), p);
#pragma unroll
    for (int i = 0; i < P; ++i) sum[j * P + i] = __ffma2_rn(b, p[i], sum[j * P + i]);
  }
}

template <typename T, int VB, int NV>
__device__ __forceinline__ float dot_row(uint32_t at, const float2 (&with)[NV * RowVec<T, VB>::PAIRS]) {
  constexpr int P = RowVec<T, VB>::PAIRS;
  float2 t = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    float2 p[P];
    pairs_of<T, VB>(RawOf<VB>::lds(at + j * 32 * VB), p);
#pragma unroll
    for (int i = 0; i < P; ++i) t = __ffma2_rn(p[i], with[j * P + i], t);
  }
  return t.x + t.y;
}

template <typename T, int VB, int G, int NV>
__device__ __forceinline__ void store_row(T* row, int l, int cols, const float2 (&x)[NV * RowVec<T, VB>::PAIRS], float by) {
  constexpr int P = RowVec<T, VB>::PAIRS, EL = RowVec<T, VB>::EL;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if ((j * G + l) * EL >= cols) break;
    T* const to = row + (j * G + l) * EL;
    float f[2 * P];
#pragma unroll
    for (int i = 0; i < P; ++i) f[2 * i] = x[j * P + i].x * by, f[2 * i + 1] = x[j * P + i].y * by;
    if constexpr (sizeof(T) == 4 && VB == 16) {
      *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
    } else if constexpr (sizeof(T) == 4 && VB == 8) {
      *reinterpret_cast<float2*>(to) = make_float2(f[0], f[1]);
    } else if constexpr (sizeof(T) == 4) {
      *to = f[0];
    } else {
      __nv_bfloat162 b[P];
#pragma unroll
      for (int i = 0; i < P; ++i) b[i] = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      *reinterpret_cast<typename RowVec<T, VB>::Raw*>(to) = *reinterpret_cast<const typename RowVec<T, VB>::Raw*>(b);
    }
  }
}

template <typename T, int VB, int G, int NV>
__device__ __forceinline__ void store_row_part(float* row, int l, int cols, const float2 (&x)[NV * RowVec<T, VB>::PAIRS]) {
  constexpr int P = RowVec<T, VB>::PAIRS, EL = RowVec<T, VB>::EL;
#pragma unroll
  for (int j = 0; j < NV; ++j)
#pragma unroll
    for (int i = 0; i < EL; ++i) {
      const int c = (j * G + l) * EL + i;
      if (c < cols) row[c] = i % 2 ? x[j * P + i / 2].y : x[j * P + i / 2].x;
    }
}

// The lane's vectors of a node's head: where they lie, and which of them the
// lane has.  Rows lie `pitch` bytes apart, below 2^32.
template <typename T, int VB, int G, int NV>
struct Lanes {
  const char* base;
  uint32_t pitch;
  bool has[NV];
  __device__ __forceinline__ Lanes(const void* p, long long ld, int h, int cols, int l, bool mine)
      : base(static_cast<const char*>(p) + (long long)h * cols * (int)sizeof(T) + l * VB), pitch((uint32_t)(ld * sizeof(T))) {
#pragma unroll
    for (int i = 0; i < NV; ++i) has[i] = mine && (i * G + l) * VB < cols * (int)sizeof(T);
  }
  __device__ __forceinline__ void copy(uint32_t to, uint32_t node, int bytes) const {
    const char* from = base + (unsigned long long)node * pitch;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (has[i]) copy_row<VB>(to + i * 32 * VB, from + i * G * VB, bytes);
  }
  // Zeros where no copy will write.
  __device__ __forceinline__ void clear(uint32_t at) const {
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (!has[i])
#pragma unroll
        for (int b = 0; b < VB; b += 4) asm volatile("st.shared.f32 [%0], %1;" ::"r"(at + i * 32 * VB + b), "f"(0.0f) : "memory");
  }
};

template <typename Shape, typename A, typename B>
__device__ __forceinline__ void clear_ring(const A& a, const B& b, int a_vecs, uint32_t at_lane) {
#pragma unroll 1
  for (int i = 0; i < Shape::STAGES * Shape::U; ++i) {
    const uint32_t at = at_lane + i / Shape::U * Shape::BATCH + i % Shape::U * Shape::VECS * Shape::VEC;
    a.clear(at);
    b.clear(at + a_vecs * Shape::VEC);
  }
}

// Keys, values and biases of the receivers' passes, into the stages in turn.
template <typename T, int VB, int G, int KN, int VN, int U_>
struct Feed {
  using Shape = RingShape<VB, G, KN, VN, U_, 4>;
  const Lanes<T, VB, G, KN> k;
  const Lanes<T, VB, G, VN> v;
  const float* const bias;  // of edge l and the lane's head; NULL: none for this lane
  const int l;
  uint32_t to, to_bias;  // where the next batch goes
  int stage;
  Walk put;
  Ahead src;

  __device__ __forceinline__ Feed(const AttnArgs& a, const Work& w, uint32_t ring, int lane, int l, int hh, int h, bool mine)
      : k(a.k, a.k_ld, h, a.D, l, mine), v(a.v, a.v_ld, h, a.Dv, l, mine),
        bias(a.bias && mine && l < Shape::U ? a.bias + (long long)l * a.H + h : nullptr), l(l), to(ring + lane * VB),
        to_bias(ring + Shape::SMALL_AT + (hh * Shape::U + l) * 4), stage(0) {
    clear_ring<Shape>(k, v, KN, to);
    put.start(w);
    src.start(a.src, put.e, a.E);
#pragma unroll
    for (int i = 0; i < Shape::STAGES - 1; ++i) batch(a, w);
  }
  __device__ __forceinline__ void batch(const AttnArgs& a, const Work& w) {
    if (!put.over(w)) {
      src.to(a.src, put.e, a.E);
      int node = src.from(put.e);
      const int n = put.end - put.e;
      const bool ok = (unsigned)node < (unsigned)a.Ns;  // a sender that is none reads as zeros
      const unsigned there = __ballot_sync(0xffffffffu, ok) & (n < Shape::U ? (1u << n) - 1 : 0xffffffffu);
      node = ok ? node : 0;
#pragma unroll
      for (int u = 0; u < Shape::U; ++u) {
        const int j = __shfl_sync(0xffffffffu, node, u), bytes = (there >> u & 1) * VB;
        k.copy(to + u * Shape::VECS * Shape::VEC, j, bytes);
        v.copy(to + (u * Shape::VECS + KN) * Shape::VEC, j, bytes);
      }
      if (bias && l < n) copy_async<4>(to_bias, bias + (long long)put.e * a.H);
      put.e += Shape::U;
      put.next_row(w);
    }
    copy_commit();
    const bool wrap = ++stage == Shape::STAGES;
    if (wrap) stage = 0;
    const uint32_t step = wrap ? (uint32_t)(-(Shape::STAGES - 1) * Shape::BATCH) : (uint32_t)Shape::BATCH;
    to += step;
    to_bias += step;
  }
};

// Place u of a batch is left out, by a ballot of the lanes' own places.
__device__ __forceinline__ bool is_out(unsigned out, int lane, int l, int u) { return out >> (lane - l + u) & 1; }

// ---------------------------------------------------------------- forward
// How far a score may lie above m before the sums are scaled, and what the weights are multiplied by, so that they stay
// below 1 (e^8 2^-12 = 0.73) and the sums within the range of the values'.  A power of two rounds nothing.
constexpr float kAhead = 8.0f, kDown = 0x1p-12f;

template <typename T, int VB, int G, int KN, int VN, int U>
__global__ void __launch_bounds__(32 * kRingWarps) k_attn_fwd_ring(const __grid_constant__ AttnArgs a) {
  using Shape = RingShape<VB, G, KN, VN, U, 4>;
  constexpr int P = RowVec<T, VB>::PAIRS, KP = KN * P, VP = VN * P;
  extern __shared__ __align__(128) uint8_t space[];
  const Rows rows{a.off, a.N, a.E, a.block, a.blocks};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % G, hh = lane / G;
  const Work w = find_work(rows, blockIdx.x * kRingWarps + warp, a.rows_each);
  if (w.n == 0) return;
  const int h = blockIdx.y * (32 / G) + hh;
  const bool mine = h < a.H;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(space) + warp * Shape::WARP;
  Feed<T, VB, G, KN, VN, U> feed(a, w, ring, lane, l, hh, h, mine);
  typename RowVec<T, VB>::Raw q_next[KN];
  auto load_q = [&](int i) {
    load_row<T, VB, G, KN>(static_cast<const T*>(a.q) + (w.row + i) * a.q_ld + (long long)h * a.D, l, a.D, mine && i < w.n, q_next);
  };
  load_q(0);
  const uint32_t at0 = ring + lane * VB, bias0 = ring + Shape::SMALL_AT + (hh * U + l % U) * 4;
  uint32_t stage_at = 0;
#pragma unroll 1
  for (int i = 0; i < w.n; ++i) {
    const int e0 = __shfl_sync(0xffffffffu, w.e0, i), e1 = __shfl_sync(0xffffffffu, w.e1, i);
    float2 q[KP], acc[VP];
    unpack<T, VB, KN>(q_next, a.scale, q);
    load_q(i + 1);
#pragma unroll
    for (int x = 0; x < VP; ++x) acc[x] = make_float2(0.0f, 0.0f);
    // Weights are taken relative to m, a score of the row; only a score that is kAhead above it moves it, so that hardly a
    // batch has to find its largest score and scale the sums.  z: of the edges of the lane's place in a batch, as largest.
    float m = EQMP_NEG_INF, largest = EQMP_NEG_INF, z = 0.0f;
#pragma unroll 1
    for (int e = e0; e < e1; e += U) {
      copy_wait<Shape::STAGES - 2>();
      __syncwarp();
      feed.batch(a, w);
      const uint32_t at = at0 + stage_at;
      float s[U];
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] = dot_row<T, VB, KN>(at + u * Shape::VECS * Shape::VEC, q);
      float score = scatter_sum<G, U>(s, l);  // of edge e + l % U
      const bool in = mine && e + l % U < e1;
      if (a.bias) {
        const float bias = lds32(bias0 + stage_at);
        score = bias == EQMP_NEG_INF ? EQMP_NEG_INF : score + bias;
      }
      if (!in) score = EQMP_NEG_INF;
      largest = fmaxf(largest, score);
      if (__any_sync(0xffffffffu, score > m + kAhead)) {
        float top = score;
#pragma unroll
        for (int o = 1; o < U; o *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        top = fmaxf(top, m);
        const float keep = top == EQMP_NEG_INF ? 1.0f : __expf(m - top);
        z *= keep;
#pragma unroll
        for (int x = 0; x < VP; ++x) acc[x] = __fmul2_rn(acc[x], make_float2(keep, keep));
        m = top;
      }
      const float base = m == EQMP_NEG_INF ? 0.0f : m;
      const float p = __expf(score - base) * kDown;
      z += p;
      const unsigned out = __ballot_sync(0xffffffffu, in && score == EQMP_NEG_INF);
      if (out) {  // left out: a weight of 0 would keep a NaN
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
          const float pu = __shfl_sync(0xffffffffu, p, lane - l + u);
          if (!is_out(out, lane, l, u)) add_row<T, VB, VN>(at + (u * Shape::VECS + KN) * Shape::VEC, pu, acc);
        }
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) add_row<T, VB, VN>(at + (u * Shape::VECS + KN) * Shape::VEC, __shfl_sync(0xffffffffu, p, lane - l + u), acc);
      }
      stage_at = stage_at == (Shape::STAGES - 1) * Shape::BATCH ? 0 : stage_at + Shape::BATCH;
    }
#pragma unroll
    for (int o = 1; o < U; o *= 2) {
      z += __shfl_xor_sync(0xffffffffu, z, o);
      largest = fmaxf(largest, __shfl_xor_sync(0xffffffffu, largest, o));
    }
    const float from_m = largest == EQMP_NEG_INF ? 1.0f : __expf(m - largest) * (1.0f / kDown);  // sums relative to the largest score
    const int slot = __shfl_sync(0xffffffffu, w.slot, i);
    if (!mine) continue;
    if (slot >= 0) {
      float* to = a.part + ((long long)slot * a.H + h) * (a.Dv + 2);
      if (l == 0) to[0] = largest, to[1] = z * from_m;
#pragma unroll
      for (int x = 0; x < VP; ++x) acc[x] = __fmul2_rn(acc[x], make_float2(from_m, from_m));
      store_row_part<T, VB, G, VN>(to + 2, l, a.Dv, acc);
      continue;
    }
    const long long to = (long long)(w.row + i) * a.H + h;
    if (a.stats && l == 0) {
      a.stats[2 * to] = z == 0.0f ? 0.0f : largest;
      a.stats[2 * to + 1] = z * from_m;
    }
    if (a.out) store_row<T, VB, G, VN>(static_cast<T*>(a.out) + to * a.Dv, l, a.Dv, acc, z == 0.0f ? 0.0f : 1.0f / z);
  }
  copy_wait<0>();
}

// ---------------------------------------------------------------- backward
// fp32 rows of up to five vectors a lane: registers for 18 warps an SM (96, and 16 bytes
// a thread spilled: 724 us where the compiler's own choice of 126 takes 758; a bound of 20
// takes 757).  0 leaves it to the compiler: bf16 rows of 1 + 4 vectors at a bound of 1
// took 249 us for 235.
template <typename T, int VB, int KN, int VN>
constexpr int kRecvWarps = sizeof(T) == 4 && VB == 16 && KN + VN <= 5 ? 18 : 0;

template <typename T, int VB, int G, int KN, int VN, int U>
__global__ void __launch_bounds__(32 * kRingWarps, (kRecvWarps<T, VB, KN, VN>)) k_attn_recv_ring(const __grid_constant__ AttnArgs a) {
  using Shape = RingShape<VB, G, KN, VN, U, 4>;
  constexpr int P = RowVec<T, VB>::PAIRS, KP = KN * P, VP = VN * P;
  extern __shared__ __align__(128) uint8_t space[];
  const Rows rows{a.off, a.N, a.E, a.block, a.blocks};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % G, hh = lane / G;
  const Work w = find_work(rows, blockIdx.x * kRingWarps + warp, a.rows_each);
  if (w.n == 0) return;
  const int h = blockIdx.y * (32 / G) + hh;
  const bool mine = h < a.H;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(space) + warp * Shape::WARP;
  Feed<T, VB, G, KN, VN, U> feed(a, w, ring, lane, l, hh, h, mine);
  typename RowVec<T, VB>::Raw q_next[KN], g_next[VN];
  float2 st_next;
  auto load_next = [&](int i) {
    const bool ok = mine && i < w.n;
    load_row<T, VB, G, KN>(static_cast<const T*>(a.q) + (w.row + i) * a.q_ld + (long long)h * a.D, l, a.D, ok, q_next);
    load_row<T, VB, G, VN>(static_cast<const T*>(a.g) + (w.row + i) * a.g_ld + (long long)h * a.Dv, l, a.Dv, ok, g_next);
    const float* st = a.stats + 2 * ((long long)(w.row + i) * a.H + h);
    st_next = ok ? make_float2(__ldg(st), __ldg(st + 1)) : make_float2(0.0f, 0.0f);
  };
  load_next(0);
  const uint32_t at0 = ring + lane * VB, bias0 = ring + Shape::SMALL_AT + (hh * U + l % U) * 4;
  uint32_t stage_at = 0;
#pragma unroll 1
  for (int i = 0; i < w.n; ++i) {
    const int e0 = __shfl_sync(0xffffffffu, w.e0, i), e1 = __shfl_sync(0xffffffffu, w.e1, i);
    float2 q[KP], g[VP], pdk[KP], pk[KP];
    unpack<T, VB, KN>(q_next, a.scale, q);
    unpack<T, VB, VN>(g_next, 1.0f, g);
    const float m = st_next.x, z = st_next.y, rz = 1.0f / z;
    load_next(i + 1);
#pragma unroll
    for (int x = 0; x < KP; ++x) pdk[x] = pk[x] = make_float2(0.0f, 0.0f);
    float delta = 0.0f, dps = 0.0f, live = 0.0f;
#pragma unroll 1
    for (int e = e0; e < e1; e += U) {
      copy_wait<Shape::STAGES - 2>();
      __syncwarp();
      feed.batch(a, w);
      const uint32_t at = at0 + stage_at;
      float score, dp;  // of edge e + l % U
      if constexpr (2 * U <= G) {
        float s[2 * U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          s[u] = dot_row<T, VB, KN>(at + u * Shape::VECS * Shape::VEC, q);
          s[U + u] = dot_row<T, VB, VN>(at + (u * Shape::VECS + KN) * Shape::VEC, g);
        }
        const float one = scatter_sum<G, 2 * U>(s, l), other = __shfl_xor_sync(0xffffffffu, one, U);
        score = l & U ? other : one;
        dp = l & U ? one : other;
      } else {
        float s[U], d[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          s[u] = dot_row<T, VB, KN>(at + u * Shape::VECS * Shape::VEC, q);
          d[u] = dot_row<T, VB, VN>(at + (u * Shape::VECS + KN) * Shape::VEC, g);
        }
        score = scatter_sum<G, U>(s, l);
        dp = scatter_sum<G, U>(d, l);
      }
      const bool in = mine && e + l % U < e1;
      if (a.bias) {
        const float bias = lds32(bias0 + stage_at);
        score = bias == EQMP_NEG_INF ? EQMP_NEG_INF : score + bias;
      }
      const bool left_out = score == EQMP_NEG_INF || z == 0.0f;
      const float p = left_out || !in ? 0.0f : __expf(score - m) * rz;
      dp = left_out || !in ? 0.0f : dp;
      if (a.pd && l < U && in) a.pd[(long long)(e + l) * a.H + h] = make_float2(left_out ? -1.0f : p, dp);
      const float pdp = p * dp;
      delta += pdp;
      dps += dp;
      live += left_out || !in ? 0.0f : 1.0f;
      const unsigned out = __ballot_sync(0xffffffffu, in && left_out);  // left out: a weight of 0 would keep a NaN
      auto add = [&](int u) {
        const float pu = __shfl_sync(0xffffffffu, p, lane - l + u), pdpu = __shfl_sync(0xffffffffu, pdp, lane - l + u);
        if (out && is_out(out, lane, l, u)) return;
#pragma unroll
        for (int j = 0; j < KN; ++j) {
          float2 x[P];
          pairs_of<T, VB>(RawOf<VB>::lds(at + (u * Shape::VECS + j) * Shape::VEC), x);
#pragma unroll
          for (int y = 0; y < P; ++y) {
            pk[j * P + y] = __ffma2_rn(make_float2(pu, pu), x[y], pk[j * P + y]);
            pdk[j * P + y] = __ffma2_rn(make_float2(pdpu, pdpu), x[y], pdk[j * P + y]);
          }
        }
      };
      if (out) {
#pragma unroll 1
        for (int u = 0; u < U; ++u) add(u);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) add(u);
      }
      stage_at = stage_at == (Shape::STAGES - 1) * Shape::BATCH ? 0 : stage_at + Shape::BATCH;
    }
#pragma unroll
    for (int o = 1; o < U; o *= 2) {
      delta += __shfl_xor_sync(0xffffffffu, delta, o);
      dps += __shfl_xor_sync(0xffffffffu, dps, o);
      live += __shfl_xor_sync(0xffffffffu, live, o);
    }
    const int slot = __shfl_sync(0xffffffffu, w.slot, i);
    if (!mine) continue;
    if (slot >= 0) {
      float* to = a.part + ((long long)slot * a.H + h) * (2 * a.D + 3);
      if (l == 0) to[0] = delta, to[1] = dps, to[2] = live;
      store_row_part<T, VB, G, KN>(to + 3, l, a.D, pdk);
      store_row_part<T, VB, G, KN>(to + 3 + a.D, l, a.D, pk);
      continue;
    }
    const bool alone = live == 1.0f;  // the row's only edge: its weight is 1, whatever its score
    if (alone) delta = dps;
    const long long to = (long long)(w.row + i) * a.H + h;
    if (l == 0) a.delta[to] = delta;
    if (a.gq) {
#pragma unroll
      for (int x = 0; x < KP; ++x) pdk[x] = make_float2(query_sum(alone, delta, pdk[x].x, pk[x].x), query_sum(alone, delta, pdk[x].y, pk[x].y));
      store_row<T, VB, G, KN>(static_cast<T*>(a.gq) + to * a.D, l, a.D, pdk, a.scale);
    }
  }
  copy_wait<0>();
}

template <typename T, int VB, int G, int KN, int VN, int U>
__global__ void __launch_bounds__(32 * kRingWarps) k_attn_send_ring(const __grid_constant__ AttnArgs a) {
  using Shape = RingShape<VB, G, KN, VN, U, 12>;  // p and dp, delta
  constexpr int P = RowVec<T, VB>::PAIRS, KP = KN * P, VP = VN * P, HEADS = 32 / G;
  constexpr int DELTA_AT = Shape::SMALL_AT + U * HEADS * 8;
  extern __shared__ __align__(128) uint8_t space[];
  const Rows rows{a.send_off, a.Ns, a.E_send, a.block, a.blocks};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, l = lane % G, hh = lane / G;
  const Work w = find_work(rows, blockIdx.x * kRingWarps + warp, a.rows_each);
  if (w.n == 0) return;
  const int h = blockIdx.y * HEADS + hh;
  const bool mine = h < a.H;
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(space) + warp * Shape::WARP, at0 = ring + lane * VB;
  const uint32_t item = hh * U + l % U;  // of the small values: the lane's own edge
  const Lanes<T, VB, G, KN> q(a.q, a.q_ld, h, a.D, l, mine);
  const Lanes<T, VB, G, VN> g(a.g, a.g_ld, h, a.Dv, l, mine);
  clear_ring<Shape>(q, g, KN, at0);

  Walk put;
  put.start(w);
  // a place's edge is loaded 64 places ahead, its receiver 32
  Ahead edges;
  const Receivers receivers(a);
  int later, dst_now, dst_next;
  auto start = [&] {
    edges.start(a.send_edges, put.e, a.E_send);
    later = edges.load(a.send_edges, put.e + 64 + lane, a.E_send);
    dst_now = receivers.of(edges.now);
    dst_next = receivers.of(edges.next);
  };
  start();
  uint32_t put_at = 0;
  auto copy_batch = [&] {
    if (!put.over(w)) {
      if (put.e - edges.c >= 64) {
        start();
      } else if (put.e - edges.c >= 32) {
        edges.c += 32;
        edges.now = edges.next;
        edges.next = later;
        later = edges.load(a.send_edges, edges.c + 64 + lane, a.E_send);
        dst_now = dst_next;
        dst_next = receivers.of(edges.next);
      }
      const int at = put.e - edges.c + lane, my_edge = edges.from(put.e), n = put.end - put.e;
      const int d0 = __shfl_sync(0xffffffffu, dst_now, at & 31), d1 = __shfl_sync(0xffffffffu, dst_next, at & 31);
      const int my_dst = at < 32 ? d0 : d1;
      const bool ok = lane < n && (unsigned)my_dst < (unsigned)a.N;
      const unsigned there = __ballot_sync(0xffffffffu, ok);
      const int node = ok ? my_dst : 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = __shfl_sync(0xffffffffu, node, u), bytes = (there >> u & 1) * VB;
        q.copy(at0 + put_at + u * Shape::VECS * Shape::VEC, i, bytes);
        g.copy(at0 + put_at + (u * Shape::VECS + KN) * Shape::VEC, i, bytes);
      }
      // lane l < U of a head: the small values of edge l; p = -1 where there is no such edge, or no receiver
      const int e = __shfl_sync(0xffffffffu, my_edge, l % U), i = __shfl_sync(0xffffffffu, node, l % U);
      if (l < U) {
        const uint32_t small = ring + put_at;
        if (mine && (there >> l & 1)) {
          copy_async<8>(small + Shape::SMALL_AT + item * 8, a.pd + (long long)e * a.H + h);
          copy_async<4>(small + DELTA_AT + item * 4, a.delta + (long long)i * a.H + h);
        } else {
          asm volatile("st.shared.v2.f32 [%0], {%1, %1};" ::"r"(small + Shape::SMALL_AT + item * 8), "f"(-1.0f) : "memory");
        }
      }
      put.e += U;
      put.next_row(w);
    }
    copy_commit();
    put_at = put_at == (Shape::STAGES - 1) * Shape::BATCH ? 0 : put_at + Shape::BATCH;
  };
#pragma unroll
  for (int i = 0; i < Shape::STAGES - 1; ++i) copy_batch();

  uint32_t stage_at = 0;
#pragma unroll 1
  for (int i = 0; i < w.n; ++i) {
    const int e0 = __shfl_sync(0xffffffffu, w.e0, i), e1 = __shfl_sync(0xffffffffu, w.e1, i);
    float2 gk[KP], gv[VP];
#pragma unroll
    for (int x = 0; x < KP; ++x) gk[x] = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int x = 0; x < VP; ++x) gv[x] = make_float2(0.0f, 0.0f);
#pragma unroll 1
    for (int c = e0; c < e1; c += U) {
      copy_wait<Shape::STAGES - 2>();
      __syncwarp();
      copy_batch();
      const uint32_t at = at0 + stage_at, small = ring + stage_at;
      const float2 pd = lds64(small + Shape::SMALL_AT + item * 8);
      const bool left_out = pd.x < 0.0f;
      const float p = left_out ? 0.0f : pd.x, ds = left_out ? 0.0f : p * (pd.y - lds32(small + DELTA_AT + item * 4));
      const unsigned out = __ballot_sync(0xffffffffu, mine && left_out && c + l % U < e1);  // a weight of 0 would keep a NaN
      auto add = [&](int u) {
        const float pu = __shfl_sync(0xffffffffu, p, lane - l + u), dsu = __shfl_sync(0xffffffffu, ds, lane - l + u);
        if (out && is_out(out, lane, l, u)) return;
        add_row<T, VB, KN>(at + u * Shape::VECS * Shape::VEC, dsu, gk);
        add_row<T, VB, VN>(at + (u * Shape::VECS + KN) * Shape::VEC, pu, gv);
      };
      if (out) {
#pragma unroll 1
        for (int u = 0; u < U; ++u) add(u);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) add(u);
      }
      stage_at = stage_at == (Shape::STAGES - 1) * Shape::BATCH ? 0 : stage_at + Shape::BATCH;
    }
    const int slot = __shfl_sync(0xffffffffu, w.slot, i);
    if (!mine) continue;
    if (slot >= 0) {
      float* to = a.part + ((long long)slot * a.H + h) * (a.D + a.Dv);
      store_row_part<T, VB, G, KN>(to, l, a.D, gk);
      store_row_part<T, VB, G, VN>(to + a.D, l, a.Dv, gv);
      continue;
    }
    const long long to = (long long)(w.row + i) * a.H + h;
    if (a.gk) store_row<T, VB, G, KN>(static_cast<T*>(a.gk) + to * a.D, l, a.D, gk, a.scale);
    if (a.gv) store_row<T, VB, G, VN>(static_cast<T*>(a.gv) + to * a.Dv, l, a.Dv, gv, 1.0f);
  }
  copy_wait<0>();
}

}  // namespace eqmp
