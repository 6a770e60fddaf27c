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
// SHIFT: rows that begin anywhere.  The rows of a group are a multiple of 8
// apart, so all of them begin the same number of values, s < V, behind a
// 16-byte boundary; the lanes take the vectors from that boundary on, columns
// -s, V - s, ..., and only a row's first and last vector are partial: what the
// first holds of the row before is masked, the copy of the last ends with the
// row, and both are stored value by value.
//
// The values move from and to HBM once.  What stands against that rate is the
// issue of instructions and the latency of a row's chain (load, sum, square
// sum, store) with 16 resident warps an SM: at 8 bytes a bf16 value may cost
// 43 lane instructions at full issue, and about half of that keeps pace.  Hence
// the arithmetic is on pairs (fma.rn.f32x2), sums of several values are
// scattered over the lanes as they are formed, rows to come are copied
// asynchronously, and a lane holds 16 values or more where it can, so that what is done
// once a row is shared by more of them.  Tried and not kept: two or four rows
// of a group at once in registers (10,000 x 128 x 16 bf16 backward 71 us against
// 55 then: spills), weights in shared memory instead of registers (49 against
// 42), more resident warps by a lower register bound (backward 20 to 130 %
// slower, forward the same).
#pragma once

#include <type_traits>

#include "common.cuh"
#include "launch.h"
#include "norm.cuh"

namespace eqmp {

struct RowShape {
  int lanes;   // G
  int active;  // lanes that hold values
  int groups;  // rows of a CTA at a time
  int run;     // forward: rounds of a CTA over neighbouring rows; 0: CTAs take turns
  int apart;   // kShiftApart: the inputs that lie otherwise than the outputs
};
enum : int { kApartX = 1, kApartG = 2, kApartR = 4 };
// Where rows begin: on 16 bytes; anywhere, in all arrays alike; anywhere, with
// some fp32 inputs copied value by value.
enum : int { kOn16 = 0, kShift = 1, kShiftApart = 2 };

constexpr int kRowThreads = 128;     // of a CTA, where a group is smaller
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
  __device__ __forceinline__ void load_part(const float* p, int n) {  // the first n < 4 values
    v = make_float4(p[0], n > 1 ? p[1] : 0.0f, n > 2 ? p[2] : 0.0f, 0.0f);
  }
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
  __device__ __forceinline__ void load_part(const __nv_bfloat16* p, int n) {  // the first n < 8 values
    const uint16_t* h = reinterpret_cast<const uint16_t*>(p);
    auto pair = [&](int i) { return (i < n ? (uint32_t)h[i] : 0u) | (i + 1 < n ? (uint32_t)h[i + 1] << 16 : 0u); };
    v = make_uint4(pair(0), pair(2), pair(4), pair(6));
  }
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
  __device__ __forceinline__ void load_part(const T* p, int) { v = *p; }
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

// ---------------------------------------------------------------- feed
// The vectors of the rows to come.  A lane copies its own vectors of the next
// DEPTH - 1 rows into shared memory asynchronously (cp.async; 0 is filled in
// for what lies outside of a row) and reads nothing but its own copies, so no
// barrier is needed, and what is on the way costs no registers.  Single bf16
// values are too small for such copies; they wait in registers, one row ahead.
template <typename T, int V, int NV, int STREAMS, int WORDS>
struct Feed {
  static constexpr int B = sizeof(T) * V;  // bytes of a vector
  static constexpr bool RING = B >= 4;
  static constexpr int ROW = STREAMS * NV * B + WORDS * 4;  // bytes of a lane and row
  static constexpr int DEPTH = !RING ? 2 : WORDS ? (ROW <= 48 ? 4 : ROW <= 80 ? 3 : 2) : ROW <= 32 ? 4 : 2;
  static constexpr int BYTES = RING ? DEPTH * ROW : 0;  // of shared memory, a lane
  uint32_t ring, at;  // the ring; the place in it that is loaded next
  uint32_t step;      // bytes between a lane's vectors
  Pack<T, V> reg[RING ? 1 : STREAMS * NV];
  float word[RING ? 1 : WORDS ? WORDS : 1];

  __device__ __forceinline__ explicit Feed(uint8_t* smem) : at(0) {
    step = blockDim.x * B;
    ring = RING ? smem_u32(smem) : 0;
  }
  __device__ __forceinline__ uint32_t row_bytes() const { return blockDim.x * ROW; }
  // `bytes` of vector j (0: none); the rest of the vector is 0.
  __device__ __forceinline__ void load(int stream, int j, const T* p, int bytes) {
    if constexpr (RING) {
      const uint32_t to = ring + at + (stream * NV + j) * step + threadIdx.x * B;
      if constexpr (B == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(p), "r"(bytes) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(p), "r"(bytes) : "memory");
    } else {
      if (bytes)
        reg[RING ? 0 : stream * NV + j].load(p);
      else
        reg[RING ? 0 : stream * NV + j].zero();
    }
  }
  // Values lo..n-1 of vector j, each by itself; the rest is 0.
  __device__ __forceinline__ void load_values(int stream, int j, const T* p, int lo, int n) {
    if constexpr (sizeof(T) == 4 && V > 1) {
      const uint32_t to = ring + at + (stream * NV + j) * step + threadIdx.x * B;
#pragma unroll
      for (int i = 0; i < V; ++i)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to + 4 * i), "l"(p + i), "r"(i >= lo && i < n ? 4 : 0)
                     : "memory");
    }
  }
  __device__ __forceinline__ void load_word(int k, const float* p, bool ok) {
    if constexpr (RING) {
      const uint32_t to = ring + at + STREAMS * NV * step + (k * blockDim.x + threadIdx.x) * 4;
      asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(to), "l"(p), "r"(ok ? 4 : 0) : "memory");
    } else {
      word[RING ? 0 : k] = ok ? *p : 0.0f;
    }
  }
  // After a row's loads: they are on the way.
  __device__ __forceinline__ void loaded() {
    if constexpr (RING) {
      asm volatile("cp.async.commit_group;" ::: "memory");
      at += row_bytes();
      if (at == DEPTH * row_bytes()) at = 0;
    }
  }
  // Waits for the oldest row and returns its place, for get().  The place that
  // the next load() fills is the one before it, read a round ago.
  __device__ __forceinline__ uint32_t wait() {
    if constexpr (RING) {
      asm volatile("cp.async.wait_group %0;" ::"n"(DEPTH - 2) : "memory");
      const uint32_t old = at + row_bytes();
      return ring + (old == DEPTH * row_bytes() ? 0 : old);
    }
    return 0;
  }
  // Waits for all copies, those that only fill in zeros included.
  __device__ __forceinline__ void drain() const {
    if constexpr (RING) asm volatile("cp.async.wait_all;" ::: "memory");
  }
  __device__ __forceinline__ void get(uint32_t place, int stream, float2 (&p)[NV * V / 2]) const {
    Pack<T, V> v[NV];
    if constexpr (RING) {
      const uint32_t from = place + stream * NV * step + threadIdx.x * B;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if constexpr (B == 16) {
          uint32_t a, b, c, d;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(a), "=r"(b), "=r"(c), "=r"(d)
                       : "r"(from + j * step));
          if constexpr (V == 4)
            v[j].v = make_float4(__uint_as_float(a), __uint_as_float(b), __uint_as_float(c), __uint_as_float(d));
          else
            v[j].v = make_uint4(a, b, c, d);
        } else {
          float f;
          asm volatile("ld.shared.f32 %0, [%1];" : "=f"(f) : "r"(from + j * step));
          v[j].v = f;
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) v[j] = reg[RING ? 0 : stream * NV + j];
    }
    get_pairs<T, V, NV>(v, p);
  }
  __device__ __forceinline__ float get_word(uint32_t place, int k) const {
    if constexpr (RING) {
      float f;
      asm volatile("ld.shared.f32 %0, [%1];"
                   : "=f"(f)
                   : "r"(place + STREAMS * NV * step + (k * blockDim.x + threadIdx.x) * 4));
      return f;
    } else {
      return word[RING ? 0 : k];
    }
  }
};

// ---------------------------------------------------------------- slots
// What a lane knows of its columns.  Values i = 0..V-1 of a vector fall into
// GROUPS of one degree: all of them (L = 0, or V = 1), the first and the other
// three of each four (K a multiple of 4: degrees begin at l^2 = 0 or 1 mod 4),
// or each by itself.
template <int L, int V, int NV, int SHIFT>
struct Slots {
  static constexpr int SHIFTED = SHIFT;
  static constexpr int K = (L + 1) * (L + 1);
  static constexpr bool FOURS = L > 0 && V > 1 && K % 4 == 0;
  static constexpr int GROUPS = L == 0 || V == 1 ? 1 : FOURS ? V / 2 : V;
  static constexpr int PAIRS = V > 1 ? V / 2 : 1;  // pairs of a vector
  using Col = std::conditional_t<(SHIFT > 0), int, uint32_t>;
  Col col[NV];  // of a vector's first value; SHIFT: below 0 in front of the row
  bool has[NV];
  int cols;
  int lane;         // within the group
  int cls[GROUPS];  // degree
  uint2 zero[PAIRS];  // all bits where a value is of degree 0, else none

  // `row`: the first row of the group.
  __device__ __forceinline__ Slots(const RowShape& sh, int cols_, int row) : cols(cols_) {
    lane = threadIdx.x % sh.lanes;
    const int shift = SHIFT ? (int)((uint32_t)row * (uint32_t)cols % V) : 0;  // V divides 2^32
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      col[j] = (lane + j * sh.active) * V - shift;
      has[j] = lane < sh.active && (int)col[j] < cols;
    }
    if constexpr (L == 0) {
      cls[0] = 0;
    } else {
#pragma unroll
      for (int g = 0; g < GROUPS; ++g) {
        const int k = ((int)col[0] + K + (FOURS ? g / 2 * 4 + g % 2 : g)) % K;
        int l = 0;
#pragma unroll
        for (int m = 1; m <= L; ++m) l += k >= m * m;
        cls[g] = l;
      }
    }
    float f[GROUPS];
    float2 first[PAIRS];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) f[g] = cls[g] == 0 ? 1.0f : 0.0f;
    spread(f, first);
#pragma unroll
    for (int s = 0; s < PAIRS; ++s) zero[s] = make_uint2(first[s].x != 0.0f ? ~0u : 0u, first[s].y != 0.0f ? ~0u : 0u);
  }
  // Whether value i of vector j is one of the row's.
  __device__ __forceinline__ bool valid(int j, int i) const {
    return has[j] && (!SHIFT || ((int)col[j] + i >= 0 && (int)col[j] + i < cols));
  }
  __device__ __forceinline__ bool whole(int j) const { return has[j] && (!SHIFT || ((int)col[j] >= 0 && (int)col[j] + V <= cols)); }
  // How many of the values of vector j, from its first, do not lie behind the row.
  __device__ __forceinline__ int count(int j) const { return !has[j] ? 0 : SHIFT && cols - (int)col[j] < V ? cols - (int)col[j] : V; }
  // How many values of vector 0 lie in front of the row.
  __device__ __forceinline__ int front() const { return SHIFT && (int)col[0] < 0 ? -(int)col[0] : 0; }
  // What the first vector holds of the row before is taken out.
  __device__ __forceinline__ void mask_front(float2 (&p)[NV * V / 2]) const {
    if constexpr (SHIFT) {
      if (col[0] < 0) {
#pragma unroll
        for (int i = 0; i < V - 1; ++i) {
          float& t = i & 1 ? p[i / 2].y : p[i / 2].x;
          t = col[0] + i < 0 ? 0.0f : t;
        }
      }
    }
  }
  // Values that are not the row's become 0.
  __device__ __forceinline__ void clear_outside(float2 (&p)[NV * V / 2]) const {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int n = count(j), lo = j ? 0 : front();
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = j * V + i;
        float& t = e & 1 ? p[e / 2].y : p[e / 2].x;
        t = i < n && i >= lo ? t : 0.0f;
      }
    }
  }
  // Whether pair s of a vector may hold a degree 0 (with FOURS its first value only).
  __device__ __forceinline__ static constexpr bool may0(int s) { return !FOURS || s % 2 == 0; }
  // The degree 0 of pair s (with L = 0 all of it), 0 in place of what is of another degree.  By selection: a product
  // with 0 would carry a NaN or an infinity from one degree into another.
  __device__ __forceinline__ float2 only0(int s, float2 v) const {
    if (L == 0) return v;
    return make_float2(__uint_as_float(__float_as_uint(v.x) & zero[s].x),
                       FOURS ? 0.0f : __uint_as_float(__float_as_uint(v.y) & zero[s].y));
  }
  // The degree 0 of vector j, or 0 where it has none: a vector has one at most.
  __device__ __forceinline__ float degree0(const float2* p) const {
    uint32_t t = 0;
#pragma unroll
    for (int s = 0; s < PAIRS; ++s) {
      if (!may0(s)) continue;
      t |= __float_as_uint(p[s].x) & zero[s].x;
      if (!FOURS) t |= __float_as_uint(p[s].y) & zero[s].y;
    }
    return __uint_as_float(t);
  }
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
  // The sums of the pairs put to their degrees.
  __device__ __forceinline__ void by_degree(const float2 (&p)[PAIRS], float* out) const {
    if constexpr (L == 0) {
      float2 t = p[0];
#pragma unroll
      for (int s = 1; s < PAIRS; ++s) t = __fadd2_rn(t, p[s]);
      out[0] = t.x + t.y;
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
        out[l] = t;
      }
    }
  }
};

// Stores the values lo..n-1 of a vector, where either lo is 0 or n is V: in at
// most three pieces, since the vector begins on 16 bytes.
__device__ __forceinline__ void put_part(float* p, const float2* f, int lo, int n) {
  if (lo == 0) {
    if (n & 2) *reinterpret_cast<float2*>(p) = f[0];
    if (n & 1) p[n & 2] = n & 2 ? f[1].x : f[0].x;
  } else {
    if (lo <= 2) *reinterpret_cast<float2*>(p + 2) = f[1];
    if (lo & 1) p[lo] = lo == 1 ? f[0].y : f[1].y;
  }
}
__device__ __forceinline__ void put_part(__nv_bfloat16* p, const float2* f, int lo, int n) {
  const uint32_t w0 = pack_bf16x2(f[0].x, f[0].y), w1 = pack_bf16x2(f[1].x, f[1].y);
  const uint32_t w2 = pack_bf16x2(f[2].x, f[2].y), w3 = pack_bf16x2(f[3].x, f[3].y);
  if (lo == 0) {
    const uint32_t a = n & 4 ? w2 : w0, b = n & 4 ? w3 : w1;
    if (n & 4) *reinterpret_cast<uint2*>(p) = make_uint2(w0, w1);
    if (n & 2) *reinterpret_cast<uint32_t*>(p + (n & 4)) = a;
    if (n & 1) reinterpret_cast<uint16_t*>(p)[n & 6] = (uint16_t)(n & 2 ? b : a);
  } else {
    const int m = 8 - lo;  // values
    const uint32_t a = m & 4 ? w1 : w3, b = m & 4 ? w0 : w2;
    if (m & 4) *reinterpret_cast<uint2*>(p + 4) = make_uint2(w2, w3);
    if (m & 2) *reinterpret_cast<uint32_t*>(p + (lo + (m & 1))) = a;
    if (m & 1) reinterpret_cast<uint16_t*>(p)[lo] = (uint16_t)((m & 2 ? b : a) >> 16);
  }
}

// Stores the values of a row that the lane has.
template <typename T, int V, int NV, typename S>
__device__ __forceinline__ void put_pairs(T* row, const S& at, const float2 (&p)[NV * V / 2]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!at.has[j]) continue;
    if constexpr (V == 1) {
      store1(row + at.col[j], j & 1 ? p[j / 2].y : p[j / 2].x);
    } else {
      if (!S::SHIFTED || at.whole(j))
        Pack<T, V>::store(row + at.col[j], p + j * (V / 2));
      else
        put_part(row + at.col[j], p + j * (V / 2), j ? 0 : at.front(), at.count(j));
    }
  }
}

// ---------------------------------------------------------------- dropout
// Which of a lane's values the dropout keeps.  DIRECT (a draw per element,
// V > 1): each lane draws for its own vectors.  Else the group forms the keep
// bits of its rows' units together, eight a byte, in shared memory, and each
// value looks its unit up: a channel's draw is made once, not once per vector
// that has a part of it.  The bits are formed for as many rows at a time as
// the lanes have blocks for (a batch), so that no warp of a group draws for
// the others while they wait; the caller waits until they are visible.
constexpr int kKeepBytes = kMaxRowThreads * 16 / 8 + kRowThreads;  // a bit a value, a byte each row begun, one more

template <typename S, int V, int NV, bool DIRECT>
struct Keeps {
  static constexpr bool L = S::K > 1;  // a draw for a channel of K values
  PhiloxBlock blocks[DIRECT ? NV : 1];
  uint32_t unit[DIRECT ? 1 : NV];       // of a vector's first value
  int left[V == 1 || DIRECT ? 1 : NV];  // how many of the vector's values it has
  uint8_t* bits;                        // of this row group, two halves taken in turn
  int bytes;                            // of a row
  int batch, my_row, my_byte;           // rows of a batch; the place that this lane forms
  int half, at_row;                     // the current row's half and place in the batch
  __device__ __forceinline__ Keeps(const Dropper& d, const S& at, const RowShape& sh, int cols, uint8_t* smem) {
    if (!d.on) return;
    if constexpr (DIRECT) {
#pragma unroll
      for (int j = 0; j < NV; ++j) blocks[j] = d.of_block(at.col[j] >> 3);
    } else {
      const uint32_t group = L ? (uint32_t)at.K : (uint32_t)d.group;
      bytes = ((uint32_t)cols / group + 7) / 8;
      batch = bytes < sh.lanes ? sh.lanes / bytes : 1;
      my_row = bytes < sh.lanes ? at.lane / bytes : 0;
      my_byte = at.lane - my_row * bytes;
      bits = smem + (threadIdx.x / sh.lanes) * bytes * batch;
      half = at_row = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        unit[j] = at.has[j] && (int)at.col[j] > 0 ? (uint32_t)at.col[j] / group : 0;
        if (V > 1) left[V > 1 ? j : 0] = (int)((unit[j] + 1) * group) - (int)at.col[j];
      }
    }
  }
  // The bits of a batch of rows, `stride` apart from `row` on, into half `to`.
  __device__ __forceinline__ void form(const Dropper& d, const RowShape& sh, int row, int stride, int to) {
    if constexpr (!DIRECT) {
      if (my_row < batch)
        for (int y = my_byte; y < bytes; y += sh.lanes)
          bits[to * kKeepBytes + my_row * bytes + y] = (uint8_t)d.keep_bits(d.block(row + my_row * stride, y));
      if (sh.lanes <= 32) __syncwarp();
    }
  }
  // Before a row's barrier, with its bits wanted behind it.
  __device__ __forceinline__ void form_now(const Dropper& d, const RowShape& sh, int row, int stride) {
    if constexpr (!DIRECT) {
      if (at_row == 0) form(d, sh, row, stride, half);
    }
  }
  // Before a row's barrier, with the next row's bits wanted in front of that one's.
  __device__ __forceinline__ void form_next(const Dropper& d, const RowShape& sh, int row, int stride) {
    if constexpr (!DIRECT) {
      if (at_row + 1 == batch) form(d, sh, row + stride, stride, half ^ 1);
    }
  }
  __device__ __forceinline__ void next_row() {
    if constexpr (!DIRECT) {
      if (++at_row == batch) {
        at_row = 0;
        half ^= 1;
      }
    }
  }
  __device__ __forceinline__ bool kept(uint32_t n) const {
    return bits[half * kKeepBytes + at_row * bytes + (n >> 3)] >> (n & 7) & 1;
  }
  // The values p of the current row, `row`, with the dropout applied.
  __device__ __forceinline__ void apply(const Dropper& d, const S& at, int row, float2 (&p)[NV * V / 2]) const {
    if constexpr (DIRECT) {
      const PhiloxRow pr = d.of_row(row);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float2* f = p + j * (V / 2);
        const uint4 w = d.block(pr, blocks[j]);
        const bool upper = V == 4 && (at.col[j] & 4);
        const uint32_t words[4] = {upper ? w.z : w.x, upper ? w.w : w.y, w.z, w.w};
#pragma unroll
        for (int s = 0; s < V / 2; ++s) {
          f[s] = __fmul2_rn(f[s], both(d.scale));
          f[s].x = words[s] << 16 > d.bound ? f[s].x : 0.0f;
          f[s].y = words[s] > d.bound ? f[s].y : 0.0f;
        }
      }
    } else if constexpr (V == 1) {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float& f = j & 1 ? p[j / 2].y : p[j / 2].x;
        f = kept(unit[j]) ? f * d.scale : 0.0f;
      }
    } else {
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        float2* f = p + j * (V / 2);
#pragma unroll
        for (int s = 0; s < V / 2; ++s) f[s] = __fmul2_rn(f[s], both(d.scale));
        if (S::SHIFTED && !L && d.group == 1) {  // V bits from some place on (of two bytes)
          const uint8_t* b = bits + half * kKeepBytes + at_row * bytes + (unit[j] >> 3);
          uint32_t keep = (b[0] | (uint32_t)b[1] << 8) >> (unit[j] & 7);
          if ((int)at.col[j] < 0) keep <<= -(int)at.col[j];
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float& t = i & 1 ? f[i / 2].y : f[i / 2].x;
            t = keep >> i & 1 ? t : 0.0f;
          }
        } else if (!L && d.group < V) {  // each value's unit by itself
#pragma unroll
          for (int i = 0; i < V; ++i) {
            float& t = i & 1 ? f[i / 2].y : f[i / 2].x;
            t = at.valid(j, i) && kept((at.col[j] + i) / (uint32_t)d.group) ? t : 0.0f;
          }
        } else {  // two units at most
          const int n = left[j];
          const bool k0 = kept(unit[j]);
          bool k1 = k0;
          if ((!L || at.K % V) && n < V && at.has[j]) k1 = kept(unit[j] + 1);
#pragma unroll
          for (int s = 0; s < V / 2; ++s) {
            f[s].x = ((L && at.K % V == 0) || 2 * s < n ? k0 : k1) ? f[s].x : 0.0f;
            f[s].y = ((L && at.K % V == 0) || 2 * s + 1 < n ? k0 : k1) ? f[s].y : 0.0f;
          }
        }
      }
    }
  }
};

// ---------------------------------------------------------------- sums
// Sums N values over the lanes of each group, in a fixed order; fetch(n) then
// gives every lane value n.  Within a warp the values are halved as the lanes
// are (each lane passes on the half that it does not keep), so that N values
// take about as many shuffles as N + log2 G, and fetch() is one more.  The
// warps of a larger group exchange their sums through red, where the rows of
// missing warps up to a multiple of four stay zero.  Up to two values lie as
// [n][warp] and fetch() adds a row, four warps a load; more lie as [warp][n],
// each lane adds a column of them, and fetch() is a shuffle again.  Two halves
// are taken in turn, so that one barrier of the group per sum is enough.  A
// group has at least as many lanes as N rounded up to a power of two.
constexpr int pow2_above(int n) { return n <= 1 ? 1 : 2 * pow2_above((n + 1) / 2); }
constexpr int kRedWarps = kMaxRowThreads / 32 + 4;  // of all groups of a CTA, each rounded up to four

template <int N>
struct GroupSum {
  static constexpr int P = pow2_above(N);
  static constexpr bool ROWS = N <= 2;
  static_assert(P <= 8, "more values than lanes of the smallest group");
  static constexpr int kRed = 2 * P * kRedWarps;  // floats of red, 16-byte aligned
  int lanes, warps4;  // of the group: lanes, warps rounded up to four
  float* red;
  int sums, mine;  // in red: the group's sums, and this warp's place in them
  int base, each;  // value n is at lane base + n each
  float val;
  __device__ __forceinline__ GroupSum(int lanes_, float* red_) : lanes(lanes_), red(red_), val(0.0f) {
    const int warps = lanes >> 5, group = threadIdx.x / lanes, warp = threadIdx.x / 32 - group * warps;
    warps4 = (warps + 3) & ~3;
    sums = group * P * warps4;
    mine = ROWS ? warp : warp * P;
    base = lanes < 32 ? (int)(threadIdx.x & 31) / lanes * lanes : 0;
    each = lanes > 32 ? 1 : lanes / P;
    if (lanes > 32) {
      for (int i = threadIdx.x; i < kRed; i += blockDim.x) red[i] = 0.0f;
      __syncthreads();
    }
  }
  __device__ __forceinline__ float fetch(int n) const {
    if (!ROWS || lanes <= 32) return __shfl_sync(0xffffffffu, val, base + n * each);
    const float4* at = reinterpret_cast<const float4*>(red + sums + n * warps4);
    float4 t = at[0];
    float v = (t.x + t.y) + (t.z + t.w);
    for (int k = 1; k < warps4 / 4; ++k) {
      t = at[k];
      v += (t.x + t.y) + (t.z + t.w);
    }
    return v;
  }
  __device__ __forceinline__ void operator()(const float (&v)[N]) {
    int o = (lanes < 32 ? lanes : 32) >> 1;
    float x[P];
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = i < N ? v[i] : 0.0f;
#pragma unroll
    for (int n = P / 2; n > 0; n >>= 1) {
      const bool up = threadIdx.x & o;
#pragma unroll
      for (int i = 0; i < n; ++i) {
        const float send = up ? x[i] : x[i + n], keep = up ? x[i + n] : x[i];
        x[i] = keep + __shfl_xor_sync(0xffffffffu, send, o);
      }
      o >>= 1;
    }
    for (; o > 0; o >>= 1) x[0] += __shfl_xor_sync(0xffffffffu, x[0], o);
    val = x[0];
    if (lanes <= 32) return;
    sums += sums < kRed / 2 ? kRed / 2 : -kRed / 2;
    const int lane = threadIdx.x & 31, n = lane / (32 / P);
    if (lane % (32 / P) == 0) red[sums + mine + (ROWS ? n * warps4 : n)] = val;
    named_barrier(1 + threadIdx.x / lanes, lanes);
    if (!ROWS) {
      val = red[sums + lane];  // four rows of eight values, or eight of four (the last four are another group's or zero)
      if (P == 4) val = lane < 4 * P ? val : 0.0f;
      for (int i = lane + 4 * P; i < warps4 * P; i += 4 * P) val += lane < 4 * P ? red[sums + i] : 0.0f;
#pragma unroll
      for (int d = P; d < 4 * P; d <<= 1) val += __shfl_xor_sync(0xffffffffu, val, d);
    }
  }
};

// Vector j of one input of a row.
template <typename F, typename S, typename T>
__device__ __forceinline__ void load_vector(F& feed, int stream, int j, const T* row, const S& at, bool live, bool apart) {
  constexpr int V = F::B / (int)sizeof(T);
  if constexpr (S::SHIFTED) {
    const int n = live ? at.count(j) : 0;
    if (S::SHIFTED == kShiftApart && apart)
      feed.load_values(stream, j, row + at.col[j], j ? 0 : at.front(), n);
    else
      feed.load(stream, j, row + at.col[j], n * (int)sizeof(T));
  } else {
    feed.load(stream, j, row + at.col[j], at.has[j] && live ? V * (int)sizeof(T) : 0);
  }
}

// What stands in front of the norm, and behind it in the backward pass.
enum : int {
  kPlain = 0,   // nothing
  kMixed = 1,   // a residual sum, dropout by units, several results
  kDirect = 2,  // as kMixed, with dropout by element drawn lane by lane (V > 1, L = 0)
};

// The values of a parameter [cols] at a lane's columns, in vectors of 16 bytes
// (L = 0, rows on 16 bytes, the parameter too); `otherwise` outside the row.
template <int V, int NV, typename S>
__device__ __forceinline__ void load_columns(const S& at, const float* from, float otherwise, float2 (&w)[NV * V / 2]) {
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < V; i += 4) {
      float4 t = make_float4(otherwise, otherwise, otherwise, otherwise);
      if (at.has[j]) t = *reinterpret_cast<const float4*>(from + at.col[j] + i);
      w[(j * V + i) / 2] = make_float2(t.x, t.y);
      w[(j * V + i) / 2 + 1] = make_float2(t.z, t.w);
    }
  }
}

// The weights of a lane's values.
template <int L, int V, int NV, typename S>
__device__ __forceinline__ void load_weights(const S& at, const NormArgs& a, float2 (&w)[NV * V / 2]) {
  if constexpr (L == 0 && V > 1 && S::SHIFTED == kOn16) {
    if (a.w && reinterpret_cast<uintptr_t>(a.w) % 16 == 0) {
      load_columns<V, NV>(at, a.w, 1.0f, w);
      return;
    }
  }
  if constexpr (L > 0 && V > 1 && S::K % V == 0) {  // a vector lies in one channel
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float t[S::GROUPS];
#pragma unroll
      for (int g = 0; g < S::GROUPS; ++g)
        t[g] = at.has[j] && a.w ? a.w[at.cls[g] * a.C + (int)at.col[j] / S::K] : 1.0f;
      float2 p[S::PAIRS];
      S::spread(t, p);
#pragma unroll
      for (int k = 0; k < S::PAIRS; ++k) w[j * S::PAIRS + k] = p[k];
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int c = ((int)at.col[j] + i) / S::K;
      int l = 0;
      if constexpr (L > 0) l = at.cls[S::GROUPS == 1 ? 0 : S::FOURS ? i / 4 * 2 + (i % 4 > 0) : i];
      const float t = at.valid(j, i) && a.w ? a.w[l * a.C + c] : 1.0f;
      const int e = j * V + i;
      (e & 1 ? w[e / 2].y : w[e / 2].x) = t;
    }
  }
}

// ---------------------------------------------------------------- forward
// One pass: each value is loaded once, kept in registers through the mean and
// the centred squares (two sums, so that a large mean costs no digits), and
// stored once.  GPU time on one GB300, share of the measured copy rate:
//   1,909,372 x 64 bf16                          77.2 us  96 %   (bound by HBM)
//   100,000 x 64 x 16 fp32, residual, dropout     237 us 102 %   (bound by HBM)
//   10,000 x 1024 bf16, residual, dropout        16.9 us  72 %   (about 5 us to fill and to empty the device, the
//       rest at the copy rate: 15.9 us for 9000 rows, 20.7 for 13,000, without a step where a round begins; 40,000
//       rows 56.4 us, 86 %)
//   16,516 x 131 fp32 out of rows of 189          7.3 us  35 %   (instructions, 63 a value: x is copied value by value)
//   20,000 x 64 x 25 bf16                        53.0 us  36 %   (instructions, 45 a value: eight degrees a vector)
template <typename T, int L, int V, int NV, int SHIFT, int MODE>
__global__ void __launch_bounds__(kMaxRowThreads) k_norm_rows(NormArgs a, RowShape sh) {
  using S = Slots<L, V, NV, SHIFT>;
  using F = Feed<T, V, NV, MODE ? 2 : 1, 0>;
  constexpr int P = NV * V / 2, PV = S::PAIRS, NS = L + 1;
  constexpr bool EACH = L == 0 || V == 1;  // a bias per value; else one per vector, which has at most one degree 0
  __shared__ __align__(16) float red1[GroupSum<1>::kRed], red2[GroupSum<NS>::kRed];
  __shared__ uint8_t bits[MODE == kMixed ? 2 * kKeepBytes + 1 : 1];
  extern __shared__ __align__(128) uint8_t ring[];
  const int stride = sh.run ? sh.groups : gridDim.x * sh.groups;
  const int begin = blockIdx.x * (sh.run ? sh.run : 1) * sh.groups;
  const int end = sh.run ? min(a.rows, begin + sh.run * sh.groups) : a.rows;
  int row = begin + threadIdx.x / sh.lanes;
  const S at(sh, a.cols, row);
  F feed(ring);
  const T* x = static_cast<const T*>(a.x) + row * a.x_ld;
  const T* r = static_cast<const T*>(a.r) + row * a.r_ld;
  int ahead = row;  // the row that is loaded next
  auto load_row = [&]() {
    const bool live = ahead < end;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_vector(feed, 0, j, x, at, live, sh.apart & kApartX);
      if (MODE && a.r) load_vector(feed, 1, j, r, at, live, sh.apart & kApartR);
    }
    feed.loaded();
    ahead += stride;
    x += stride * a.x_ld;
    if (MODE) r += stride * a.r_ld;
  };
#pragma unroll 1
  for (int d = 0; d < F::DEPTH - 1; ++d) load_row();
  GroupSum<1> sum1(sh.lanes, red1);
  GroupSum<NS> sum2(sh.lanes, red2);
  const Dropper drop(a.drop);
  Keeps<S, V, NV, MODE == kDirect> keeps(drop, at, sh, a.cols, bits);
  // 32 values a lane: w and b wait in shared memory, one copy for all groups
  // (each of one warp, all with the same columns)
  constexpr bool SHARED = NV * V == 32;
  constexpr int PR = SHARED ? 2 : P;  // pairs in registers
  float4* shared_wb = reinterpret_cast<float4*>(ring + blockDim.x * F::BYTES);
  float2 w[PR], b[EACH ? PR : NV];
  bool all = true;  // whether the lane's values are all of the row
  if constexpr (SHARED) {
    for (int i = threadIdx.x; i < 32 * NV * V; i += blockDim.x) {
      const int lane = i / 4 % 32, v4 = i / 128, col = (lane + v4 / (V / 4) * sh.active) * V + v4 % (V / 4) * 4 + i % 4;
      const bool in = lane < sh.active && col < a.cols;
      reinterpret_cast<float*>(shared_wb)[i] = in && a.w ? a.w[col] : 1.0f;
      reinterpret_cast<float*>(shared_wb + 32 * NV * V / 4)[i] = in && a.b ? a.b[col] : 0.0f;
    }
    __syncthreads();
  } else {
    load_weights<L, V, NV, S>(at, a, w);
  }
  bool biased = SHARED;
  if constexpr (L == 0 && V > 1 && SHIFT == kOn16 && !SHARED) {
    biased = a.b && reinterpret_cast<uintptr_t>(a.b) % 16 == 0;
    if (biased) load_columns<V, NV>(at, a.b, 0.0f, b);
  }
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    all = all && at.whole(j);
    if (biased) continue;
    if constexpr (EACH) {
#pragma unroll
      for (int i = 0; i < V; ++i) {
        const int e = j * V + i, c = ((int)at.col[j] + i) / S::K;
        (e & 1 ? b[e / 2 % PR].y : b[e / 2 % PR].x) = at.valid(j, i) && a.b && at.cls[0] == 0 ? a.b[c] : 0.0f;
      }
    } else {
      const int c = ((int)at.col[j] + V - 1) / S::K;  // the channel that begins in the vector, if one does
      b[j] = both(at.has[j] && a.b && c * S::K >= (int)at.col[j] && c < a.C ? a.b[c] : 0.0f);
    }
  }
  const float inv = 1.0f / (float)a.C;
  float scale[S::GROUPS];
#pragma unroll
  for (int g = 0; g < S::GROUPS; ++g) scale[g] = inv / (float)(2 * at.cls[g] + 1);
  all = __all_sync(0xffffffffu, all);
  if (MODE == kMixed && drop.on) {
    keeps.form(drop, sh, row, stride, 0);
    __syncthreads();
  }
  // the same number of rounds for every group of the CTA
  for (int base = begin; base < end; base += stride, row += stride) {
    float2 v[P], acc[PV];
    const uint32_t place = feed.wait();
    feed.get(place, 0, v);
    at.mask_front(v);
    if constexpr (MODE != kPlain) {
      if (drop.on) keeps.apply(drop, at, row, v);
      if (a.r) {
        float2 f[P];
        feed.get(place, 1, f);
        at.mask_front(f);
#pragma unroll
        for (int p = 0; p < P; ++p) v[p] = __fadd2_rn(v[p], f[p]);
      }
    }
    load_row();
    if (MODE == kMixed && drop.on) keeps.form_next(drop, sh, row, stride);
    const bool live = row < end;
    const long long out = (long long)row * a.cols;
    if (MODE && a.s && live) put_pairs<T, V, NV>(static_cast<T*>(a.s) + out, at, v);
    // the mean of degree 0
    float part[1] = {0.0f};
#pragma unroll
    for (int s = 0; s < PV; ++s) {
      if (!S::may0(s)) continue;
      float2 t = v[s];
#pragma unroll
      for (int p = s + PV; p < P; p += PV) t = __fadd2_rn(t, v[p]);
      t = at.only0(s, t);
      part[0] += t.x + t.y;
    }
    sum1(part);
    const float mean = sum1.fetch(0) * inv;
    // centred; what lies outside the row stays 0
    float2 mu[PV];
#pragma unroll
    for (int s = 0; s < PV; ++s) mu[s] = at.only0(s, both(-mean));
#pragma unroll
    for (int p = 0; p < P; ++p)
      if (S::may0(p % PV)) v[p] = __fadd2_rn(mu[p % PV], v[p]);
    if (!all) at.clear_outside(v);
#pragma unroll
    for (int s = 0; s < PV; ++s) {
      acc[s] = __fmul2_rn(v[s], v[s]);
#pragma unroll
      for (int p = s + PV; p < P; p += PV) acc[s] = __ffma2_rn(v[p], v[p], acc[s]);
    }
    float sq[NS];
    at.by_degree(acc, sq);
    sum2(sq);
    float q[S::GROUPS];  // the approximate root is within 2 units in the last place
#pragma unroll
    for (int g = 0; g < S::GROUPS; ++g) q[g] = rsqrtf(sum2.fetch(at.cls[g]) * scale[g] + a.eps);
    if (a.stats) {
      float* st = a.stats + (long long)row * (L + 2);
      const int l = at.lane < L ? at.lane : L;
      const float ql = L ? rsqrtf(sum2.fetch(l) * (inv / (float)(2 * l + 1)) + a.eps) : q[0];
      if (live && at.lane <= L) st[1 + l] = ql;
      if (live && at.lane == 0) st[0] = mean;
    }
    if (MODE == kMixed && drop.on) keeps.next_row();
    if (!live || !a.y) continue;
    float2 qs[PV];
    S::spread(q, qs);
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const float2 h = __fmul2_rn(v[p], qs[p % PV]);
      if constexpr (SHARED) {
        if (p % 2 == 0) {
          const float4 wv = shared_wb[p / 2 * 32 + at.lane], bv = shared_wb[32 * NV * V / 4 + p / 2 * 32 + at.lane];
          w[0] = make_float2(wv.x, wv.y);
          w[1] = make_float2(wv.z, wv.w);
          b[0] = make_float2(bv.x, bv.y);
          b[1] = make_float2(bv.z, bv.w);
        }
      }
      if (EACH)
        v[p] = __ffma2_rn(h, w[p % PR], b[EACH ? p % PR : 0]);
      else if (S::may0(p % PV))
        v[p] = __ffma2_rn(h, w[p % PR], at.only0(p % PV, b[EACH ? 0 : p / PV]));
      else
        v[p] = __fmul2_rn(h, w[p % PR]);
    }
    put_pairs<T, V, NV>(static_cast<T*>(a.y) + out, at, v);
  }
  feed.drain();  // the zeros of the rows behind the last one
}

// ---------------------------------------------------------------- backward
// Words of a row's statistics that a lane copies.  A group has at least 8
// lanes where L > 0, and the L + 2 <= 8 words go to the first of each warp.
constexpr int stat_words(int L) { return L == 0 ? 2 : 1; }

// One pass over g and s (and dL/ds): the row's sums of a and a h, then dL/ds
// and dL/dx from the registers, while each lane adds g h and g of its columns
// over all the rows of its group.  At the end the groups of a CTA are added in
// their order through shared memory, the orders of a degree with them, and
// the CTA's (L+2) C sums go to its part of the workspace; a second kernel,
// launched while this one runs, adds the parts (4 to 6 us of the times below
// were this tail before it had one barrier and one load latency; about 3 now).
// CTAs are persistent: with many short ones the tails cost more than the order
// of DRAM gains (45 against 60 us and more at 10,000 x 128 x 16).
//   477,664 x 128 bf16                            59.1 us  93 %   (HBM, then the tail)
//   20,000 x 32 x 49 fp32                         61.8 us  90 %   (HBM, barriers of a row's warps)
//   10,000 x 128 x 16 bf16, residual, dropout     35.6 us  85 %   (instructions, 38 a value)
//   16,516 x 509 fp32, residual, dropout          32.2 us  77 %   (instructions, 73 a value: partial vectors, keep bits)
//   40,000 x 768 bf16                             47.1 us  58 %   (a quarter of the places empty, two warps' barrier a row)
//   20,000 x 64 x 25 bf16                         67.1 us  42 %   (instructions, 49 a value: eight degrees a vector, spills)
template <typename T, int L, int V, int NV, int SHIFT, int MODE>
__global__ void __launch_bounds__(kMaxRowThreads) k_norm_bwd_rows(NormArgs a, RowShape sh) {
  using S = Slots<L, V, NV, SHIFT>;
  using F = Feed<T, V, NV, MODE ? 3 : 2, stat_words(L)>;
  constexpr int P = NV * V / 2, PV = S::PAIRS, NS = L + 2;
  constexpr bool EACH = L == 0 || V == 1;  // db per value; else per vector, which has at most one degree 0
  constexpr int DB = EACH ? P : (NV + 1) / 2;  // pairs: of two values, or of two vectors
  __shared__ __align__(16) float red[GroupSum<NS>::kRed];
  __shared__ uint8_t bits[MODE == kMixed ? 2 * kKeepBytes + 1 : 1];
  extern __shared__ __align__(128) uint8_t ring[];  // at the end the column sums: [cols] g h, [C] g
  const int stride = gridDim.x * sh.groups;
  int row = blockIdx.x * sh.groups + threadIdx.x / sh.lanes;
  const S at(sh, a.cols, row);
  F feed(ring);
  const T* x = static_cast<const T*>(a.x) + row * a.x_ld;
  const T* g = static_cast<const T*>(a.g) + row * a.g_ld;
  const T* r = static_cast<const T*>(a.r) + row * a.r_ld;
  const float* st = a.stats + (long long)row * (L + 2);
  int ahead = row;  // the row that is loaded next
  auto load_row = [&]() {
    const bool live = ahead < a.rows;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      load_vector(feed, 0, j, x, at, live, sh.apart & kApartX);
      load_vector(feed, 1, j, g, at, live, sh.apart & kApartG);
      if (MODE && a.r) load_vector(feed, 2, j, r, at, live, sh.apart & kApartR);
    }
    if constexpr (L == 0) {
      feed.load_word(0, st, live);
      feed.load_word(1, st + 1, live);
    } else {  // one word a lane, passed on by shuffles
      feed.load_word(0, st + min((int)(threadIdx.x & 7), L + 1), live);
    }
    feed.loaded();
    ahead += stride;
    x += stride * a.x_ld;
    g += stride * a.g_ld;
    if (MODE) r += stride * a.r_ld;
    st += (long long)stride * (L + 2);
  };
#pragma unroll 1
  for (int d = 0; d < F::DEPTH - 1; ++d) load_row();
  GroupSum<NS> sum(sh.lanes, red);
  const Dropper drop(a.drop);
  Keeps<S, V, NV, MODE == kDirect> keeps(drop, at, sh, a.cols, bits);
  float2 w[P], dw[P], db[DB];
  load_weights<L, V, NV, S>(at, a, w);
#pragma unroll
  for (int p = 0; p < P; ++p) dw[p] = both(0.0f);
#pragma unroll
  for (int p = 0; p < DB; ++p) db[p] = both(0.0f);
  const float inv = 1.0f / (float)a.C;
  float scale[S::GROUPS];
#pragma unroll
  for (int k = 0; k < S::GROUPS; ++k) scale[k] = -inv / (float)(2 * at.cls[k] + 1);
  const int first_lane = sh.lanes < 32 ? (int)(threadIdx.x & 31) / sh.lanes * sh.lanes : 0;  // of the group, in the warp
  for (int base = blockIdx.x * sh.groups; base < a.rows; base += stride, row += stride) {
    const bool live = row < a.rows;
    float2 h[P], av[P], cr[MODE ? P : 1], qs[PV];
    float q[S::GROUPS];
    const uint32_t place = feed.wait();
    feed.get(place, 0, h);
    feed.get(place, 1, av);
    at.mask_front(h);
    at.mask_front(av);
    if constexpr (MODE != kPlain && !F::RING) {
      if (a.r) feed.get(place, 2, cr);
    }
    float2 mu;
    if constexpr (L == 0) {
      mu = both(-feed.get_word(place, 0));
      q[0] = feed.get_word(place, 1);
    } else {
      const float word = feed.get_word(place, 0);
      mu = both(-__shfl_sync(0xffffffffu, word, first_lane));
#pragma unroll
      for (int k = 0; k < S::GROUPS; ++k) q[k] = __shfl_sync(0xffffffffu, word, first_lane + 1 + at.cls[k]);
    }
    load_row();
    if (MODE == kMixed && drop.on) keeps.form_now(drop, sh, row, stride);
    S::spread(q, qs);
    float2 sa[PV], sah[PV], mus[PV];
#pragma unroll
    for (int s = 0; s < PV; ++s) {
      sa[s] = sah[s] = both(0.0f);
      mus[s] = at.only0(s, mu);
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int s = p % PV;
      if (S::may0(s)) h[p] = __fadd2_rn(h[p], mus[s]);
      h[p] = __fmul2_rn(h[p], qs[s]);
      dw[p] = __ffma2_rn(av[p], h[p], dw[p]);
      if (EACH) db[EACH ? p : 0] = __fadd2_rn(db[EACH ? p : 0], av[p]);
      if (!EACH && s == 0) {
        float& t = p / PV & 1 ? db[EACH ? 0 : p / PV / 2].y : db[EACH ? 0 : p / PV / 2].x;
        t += at.degree0(av + p);
      }
      av[p] = __fmul2_rn(av[p], w[p]);
      if (S::may0(s)) sa[s] = __fadd2_rn(sa[s], av[p]);
      sah[s] = __ffma2_rn(av[p], h[p], sah[s]);
    }
    float tot[NS];
    tot[0] = 0.0f;
#pragma unroll
    for (int s = 0; s < PV; ++s) {
      if (!S::may0(s)) continue;
      sa[s] = at.only0(s, sa[s]);
      tot[0] += sa[s].x + sa[s].y;
    }
    at.by_degree(sah, tot + 1);
    sum(tot);
    // r = q a - (q mean(a h)) h - q mean(a) for degree 0
    const float m0 = sum.fetch(0) * -inv;
    float c[S::GROUPS];
#pragma unroll
    for (int k = 0; k < S::GROUPS; ++k) c[k] = sum.fetch(1 + at.cls[k]) * scale[k] * q[k];
    float2 cs[PV];
    S::spread(c, cs);
#pragma unroll
    for (int s = 0; s < PV; ++s) {
      if (!S::may0(s)) continue;
      sa[s] = at.only0(s, __fmul2_rn(qs[s], both(m0)));
    }
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const int s = p % PV;
      const float2 t = S::may0(s) ? __ffma2_rn(av[p], qs[s], sa[s]) : __fmul2_rn(av[p], qs[s]);
      av[p] = __ffma2_rn(h[p], cs[s], t);
    }
    const long long out = (long long)row * a.cols;
    if constexpr (MODE != kPlain) {
      if (a.r) {
        if constexpr (F::RING) feed.get(place, 2, cr);
#pragma unroll
        for (int p = 0; p < P; ++p) av[p] = __fadd2_rn(av[p], cr[p]);
      }
      if (a.gr && live) put_pairs<T, V, NV>(static_cast<T*>(a.gr) + out, at, av);
      if (a.gx) {
        if (drop.on) keeps.apply(drop, at, row, av);
        if (live) put_pairs<T, V, NV>(static_cast<T*>(a.gx) + out, at, av);
      }
      if (MODE == kMixed && drop.on) keeps.next_row();
    } else {
      T* dst = static_cast<T*>(a.gx ? a.gx : a.gr);
      if (dst && live) put_pairs<T, V, NV>(dst + out, at, av);
    }
  }
  // the sums' kernel may be launched; it waits until this one is done
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  feed.drain();  // the zeros of the rows behind the last one; the ring's memory takes the column sums
  if (!a.gw && !a.gb) return;
  __syncthreads();
  // The CTA's sums.  The groups of a warp are added by shuffles (SHIFT: their
  // lanes have different columns); then each warp (or group) puts its columns
  // into a row of its own, [C][K padded to an odd number] g h and [C] g, and
  // the rows are added.
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (!SHIFT && o >= sh.lanes) {
#pragma unroll
      for (int p = 0; p < P; ++p) {
        dw[p].x += __shfl_xor_sync(0xffffffffu, dw[p].x, o);
        dw[p].y += __shfl_xor_sync(0xffffffffu, dw[p].y, o);
      }
#pragma unroll
      for (int p = 0; p < DB; ++p) {
        db[p].x += __shfl_xor_sync(0xffffffffu, db[p].x, o);
        db[p].y += __shfl_xor_sync(0xffffffffu, db[p].y, o);
      }
    }
  }
  constexpr int KP = S::K | 1;
  float* sums = reinterpret_cast<float*>(ring);
  const int unit = !SHIFT && sh.lanes <= 32 ? 32 : sh.lanes;  // threads that add together
  const int units = blockDim.x / unit, width = (KP + 1) * a.C;
  if ((int)(threadIdx.x % unit) < sh.lanes) {
    float* mine = sums + threadIdx.x / unit * width;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      if (!at.has[j]) continue;
#pragma unroll
      for (int i = 0; i < V; ++i) {
        if (!at.valid(j, i)) continue;
        const int e = j * V + i, col = (int)at.col[j] + i;
        const int c = (S::K % V == 0 ? (int)at.col[j] : col) / S::K;  // its place: c KP + col - c K
        mine[col + c * (KP - S::K)] = e & 1 ? dw[e / 2].y : dw[e / 2].x;
        if (EACH && col == c * S::K) mine[KP * a.C + c] = e & 1 ? db[EACH ? e / 2 : 0].y : db[EACH ? e / 2 : 0].x;
      }
      if (!EACH) {
        const int c = ((int)at.col[j] + V - 1) / S::K;  // the channel that begins in the vector, if one does
        if (c * S::K >= (int)at.col[j] && c < a.C) mine[KP * a.C + c] = j & 1 ? db[EACH ? 0 : j / 2].y : db[EACH ? 0 : j / 2].x;
      }
    }
  }
  __syncthreads();
  float* to_w = a.gw;
  float* to_b = a.gb;
  if (a.parts > 1) {
    to_w = a.part + (long long)blockIdx.x * (L + 2) * a.C;
    to_b = to_w + (L + 1) * a.C;
  }
  for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
    float t[L + 2];
#pragma unroll
    for (int l = 0; l < L + 2; ++l) t[l] = 0.0f;
    for (int u = 0; u < units; ++u) {
      const float* from = sums + u * width;
#pragma unroll
      for (int l = 0; l <= L; ++l)
#pragma unroll
        for (int k = l * l; k < (l + 1) * (l + 1); ++k) t[l] += from[c * KP + k];
      t[L + 1] += from[KP * a.C + c];
    }
#pragma unroll
    for (int l = 0; l <= L; ++l)
      if (to_w) to_w[l * a.C + c] = t[l];
    if (to_b) to_b[c] = t[L + 1];
  }
}

// ---------------------------------------------------------------- launch
// Lanes for a row of cols values in vectors of V, NV per lane, at least
// min_lanes (a power of two), and the groups of a CTA: as many as fill it, or
// fewer where the rows would leave some SMs without a CTA.  Not so if one CTA
// is to do it all (`single` rounds of it at most): a backward pass of one CTA
// needs no second launch for the weight sums, which costs more than the rounds.
inline RowShape row_shape(int cols, int K, int V, int NV, int min_lanes, int rows, int sms, int single) {
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
  sh.run = sh.apart = 0;
  if (rows <= single * sh.groups) return sh;
  const int whole = sh.lanes < 32 ? 32 / sh.lanes : 1;  // groups of a warp
  while (sh.groups / 2 >= whole && (long long)sms * (sh.groups / 2) >= rows) sh.groups /= 2;
  return sh;
}

// dw and db from the parts (norm.cu).
eqmp_status launch_norm_bwd_sum(const NormArgs& a, int L, cudaStream_t st);

// CTAs of a persistent launch: what the device holds at a time, at most one
// per tile of rows.
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

constexpr int kSingle = 4;                 // rounds
constexpr int kMaxRingBytes = 220 * 1024;  // of dynamic shared memory, a CTA
constexpr long long kRunBytes = 128 * 1024;

template <typename T, int L, int V, int NV, int SHIFT, bool BACKWARD, int MODE>
static eqmp_status launch_mode(NormArgs a, RowShape sh, const DeviceInfo& dev, cudaStream_t st) {
  static int cache[64][33];
  static unsigned long long attr_done = 0;
  const int threads = sh.lanes * sh.groups;
  const long long tiles = ((long long)a.rows + sh.groups - 1) / sh.groups;
  if constexpr (!BACKWARD) {
    auto kern = k_norm_rows<T, L, V, NV, SHIFT, MODE>;
    const size_t smem = (size_t)threads * Feed<T, V, NV, MODE ? 2 : 1, 0>::BYTES + (NV * V == 32 ? 2 * 32 * 32 * 4 : 0);
    if (ensure_smem_attr(kern, kMaxRingBytes, &attr_done) != cudaSuccess) return EQMP_ERR_CUDA;
    int grid = resident_grid(kern, threads, smem, dev, tiles, cache);
    if (grid < 1) return EQMP_ERR_CUDA;
    // Much work: CTAs in order, each over a run of about 128 KB, so that what
    // is on the way stays a narrow window of DRAM (persistent CTAs drift
    // apart: 100,000 x 64 x 16 fp32 with residual 281 us, in runs 238).
    // Else persistent CTAs in turns, which share out little work evenly.
    const long long bytes = (long long)sh.groups * a.cols * (long long)sizeof(T) * (2 + (a.r != nullptr) + (a.s != nullptr));
    const int run = bytes < kRunBytes ? (int)(kRunBytes / bytes) : 1;
    if (tiles / run >= 4ll * grid && (!SHIFT || sh.groups % 8 == 0)) {
      sh.run = run;
      grid = (int)((tiles + run - 1) / run);
    }
    if (SHIFT && !sh.run && grid < tiles) grid = grid / 8 * 8;  // a group's rows are a multiple of 8 apart
    if (grid < 1) return EQMP_ERR_UNSUPPORTED;
    kern<<<grid, threads, smem, st>>>(a, sh);
    return cuda_status(cudaGetLastError());
  } else {
    auto kern = k_norm_bwd_rows<T, L, V, NV, SHIFT, MODE>;
    if (ensure_smem_attr(kern, kMaxRingBytes, &attr_done) != cudaSuccess) return EQMP_ERR_CUDA;
    const size_t feed = (size_t)threads * Feed<T, V, NV, MODE ? 3 : 2, stat_words(L)>::BYTES;
    constexpr int KP = ((L + 1) * (L + 1)) | 1;  // the CTA's column sums, one row for each warp or group
    const size_t sums = sizeof(float) * (size_t)(KP + 1) * a.C * (!SHIFT && sh.lanes <= 32 ? threads / 32 : sh.groups);
    const size_t smem = feed > sums ? feed : sums;
    int grid = resident_grid(kern, threads, smem, dev, tiles, cache);
    if (grid < 1) return EQMP_ERR_CUDA;
    if (tiles <= kSingle && (!SHIFT || sh.groups % 8 == 0)) grid = 1;
    if (grid > kMaxParts) grid = kMaxParts;
    if (SHIFT && grid < tiles && grid > 1) grid = grid / 8 * 8;  // a group's rows are a multiple of 8 apart
    if (grid < 1) return EQMP_ERR_UNSUPPORTED;
    a.parts = grid;
    kern<<<grid, threads, smem, st>>>(a, sh);
    if (cudaGetLastError() != cudaSuccess) return EQMP_ERR_CUDA;
    if ((!a.gw && !a.gb) || grid == 1) return EQMP_OK;
    return launch_norm_bwd_sum(a, L, st);
  }
}

template <typename T, int L, int V, int NV, int SHIFT, bool BACKWARD>
static eqmp_status launch_rows(const NormArgs& a, const RowShape& sh, const DeviceInfo& dev, cudaStream_t st) {
  if (!a.r && !a.drop.threshold && !(BACKWARD ? a.gr && a.gx : a.s != nullptr))
    return launch_mode<T, L, V, NV, SHIFT, BACKWARD, kPlain>(a, sh, dev, st);
  if constexpr (L == 0 && V > 1 && SHIFT == kOn16) {
    if (a.drop.threshold && a.drop.group == 1) return launch_mode<T, L, V, NV, SHIFT, BACKWARD, kDirect>(a, sh, dev, st);
  }
  return launch_mode<T, L, V, NV, SHIFT, BACKWARD, kMixed>(a, sh, dev, st);
}

// 16 values a lane share the sums' shuffles and barriers over more values; 8
// leave more lanes to work on a row, which is faster where the rows are few,
// and fit the registers of the lanes that handle single values and of the
// backward pass of rows that begin anywhere.  The forward layer norm also
// takes 12 (fp32) or 24 where those leave fewer places of a group empty (24 at
// 768 columns: one warp, every lane full, for two of which a quarter idles) or
// as many and fewer warps (1536 columns: 24.0 us for 20,000 bf16 rows, 29.7
// with 16),
// and bf16 32 where one warp then does for two (769 to 1024 columns).  The
// norms by degree and the backward passes do not weigh empty places: 40,000 x
// 768 bf16 backward fills 48 of 64 lanes, 100,000 x 8 x 49 39 % of its places.
template <typename T, int L, int V, int SHIFT, bool BACKWARD>
static eqmp_status launch_rows_v(const NormArgs& a, int apart, const DeviceInfo& dev, cudaStream_t st, bool* done) {
  constexpr int K = (L + 1) * (L + 1), N8 = 8 / V, N16 = 16 / V;
  constexpr int least = pow2_above(BACKWARD ? L + 2 : L + 1);  // what GroupSum needs
  const int cols = SHIFT ? a.cols + 2 * (V - 1) : a.cols;      // a first and a last vector in part
  const int single = BACKWARD ? kSingle : 0;
  auto shape = [&](int NV) {
    RowShape sh = row_shape(cols, K, V, NV, least, a.rows, dev.sms, single);
    sh.apart = apart;
    return sh;
  };
  const RowShape s8 = shape(N8), s16 = shape(N16);
  const bool few = (long long)a.rows * s8.lanes <= (long long)dev.sms * kMaxRowThreads;
  *done = s16.lanes <= kMaxRowThreads;
  if (!*done) return EQMP_OK;
  if (s8.lanes <= kMaxRowThreads && (V == 1 || few || (SHIFT != kOn16 && BACKWARD)))
    return launch_rows<T, L, V, N8, SHIFT, BACKWARD>(a, s8, dev, st);
  if constexpr (L == 0 && V > 1 && !BACKWARD) {
    const RowShape s24 = shape(24 / V);
    if constexpr (V == 8 && SHIFT == kOn16) {
      const RowShape s32 = shape(4);
      if (s32.lanes == 32 && s24.lanes > 32) return launch_rows<T, L, V, 4, SHIFT, BACKWARD>(a, s32, dev, st);
    }
    const int places = s16.lanes * 16;
    if constexpr (V == 4) {
      const RowShape s12 = shape(3);
      if (s12.lanes <= kMaxRowThreads && s12.lanes * 12 < places && s12.lanes * 12 <= s24.lanes * 24)
        return launch_rows<T, L, V, 3, SHIFT, BACKWARD>(a, s12, dev, st);
    }
    if (s24.lanes * 24 < places || (s24.lanes * 24 == places && s16.lanes > 32))
      return launch_rows<T, L, V, 24 / V, SHIFT, BACKWARD>(a, s24, dev, st);
  }
  return launch_rows<T, L, V, N16, SHIFT, BACKWARD>(a, s16, dev, st);
}

inline bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// Whether the rows of an array begin where packed rows of `cols` elements do,
// counted from a 16-byte boundary.
inline bool lies_packed(const void* p, long long ld, long long cols, int bytes) {
  return on16(p) && ld >= cols && (ld - cols) * bytes % 16 == 0;
}

// Runs the pass if the row fits; *done says whether it did.  Vectors of 16
// bytes where the outputs begin on 16 bytes and the inputs lie as they do;
// fp32 inputs that lie otherwise are copied value by value into the vectors'
// places.  Else, and where rows would be mostly first and last vector, lanes
// handle single values.
template <typename T, int L, bool BACKWARD>
static eqmp_status launch_rows_l(const NormArgs& a, const DeviceInfo& dev, cudaStream_t st, bool* done) {
  constexpr int B = sizeof(T), V = 16 / B;
  const bool outputs = on16(a.s) && on16(a.y) && on16(a.gr) && on16(a.gx);
  const bool whole = a.cols * (long long)B % 16 == 0;  // vectors
  auto apart = [&](const void* p, long long ld, int bit) {
    if (!p || (whole && on16(p) && ld * B % 16 == 0) || (!whole && lies_packed(p, ld, a.cols, B))) return 0;
    return bit;
  };
  const int which = apart(a.x, a.x_ld, kApartX) | apart(a.g, a.g_ld, kApartG) | apart(a.r, a.r_ld, kApartR);
  if (outputs && whole && !which) return launch_rows_v<T, L, V, kOn16, BACKWARD>(a, 0, dev, st, done);
  if constexpr ((L + 1) * (L + 1) * B % 16 != 0) {
    if (outputs && a.cols >= 4 * V && !which) return launch_rows_v<T, L, V, kShift, BACKWARD>(a, 0, dev, st, done);
  }
  if constexpr (L == 0 && B == 4) {  // features are packed
    if (outputs && a.cols >= 4 * V) return launch_rows_v<T, L, V, kShiftApart, BACKWARD>(a, which, dev, st, done);
  }
  return launch_rows_v<T, L, 1, kOn16, BACKWARD>(a, 0, dev, st, done);
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
