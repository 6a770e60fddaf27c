// Host-side checks of arguments that entry points share: alignment, strides and
// whether the memory of two arguments meets.
#pragma once

#include <stdint.h>

namespace eqmp {

inline bool aligned(const void* p, int bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

// One strided matrix: rows of `cols` elements, `ld` elements apart.
struct Plane {
  const void* p;
  long long ld;
};

// The memory of an argument; NULL and empty ones meet nothing.
struct Span {
  uintptr_t begin, end;
};

inline Span span(const void* p, long long bytes) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(p);
  return Span{at, p && bytes > 0 ? at + (uintptr_t)bytes : at};
}

inline Span span(const Plane& a, long long rows, long long cols, int bytes) {
  return span(a.p, rows > 0 ? ((rows - 1) * a.ld + cols) * bytes : 0);
}

inline bool meet(const Span& a, const Span& b) {
  return a.begin < a.end && b.begin < b.end && a.begin < b.end && b.begin < a.end;
}

// Outputs apart from the inputs and from one another.
template <int I, int O>
bool outputs_apart(const Span (&in)[I], const Span (&out)[O]) {
  for (int o = 0; o < O; ++o) {
    for (int i = 0; i < I; ++i)
      if (meet(in[i], out[o])) return false;
    for (int q = 0; q < o; ++q)
      if (meet(out[q], out[o])) return false;
  }
  return true;
}

// A row stride of up to 2^31 elements, so that 2^30 rows stay in 64 bits.
inline bool stride_ok(long long ld) { return ld >= 0 && ld <= 1ll << 31; }

// Inputs: aligned, strides that address forward.  Outputs (packed): aligned.
inline bool planes_ok(const Plane* in, int n_in, void* const* outs, int n_out, int bytes) {
  for (int i = 0; i < n_in; ++i)
    if (in[i].p && (!aligned(in[i].p, bytes) || !stride_ok(in[i].ld))) return false;
  for (int o = 0; o < n_out; ++o)
    if (!aligned(outs[o], bytes)) return false;
  return true;
}

}  // namespace eqmp
