// Entry points of the head norm with its rotation: argument checks and dispatch.
// Contracts are in include/eqmp.h, the formulas in head_norm.cuh.
#include "head_norm.cuh"

#include <math.h>

#include "host_args.h"
#include "launch.h"

namespace eqmp {

constexpr int kMaxHeadDim = 256, kMaxHeads = 65536;
constexpr int kHeadCtas = 3;  // on each SM, in the backward pass: each leaves a part of dw

static eqmp_status check(int64_t N, int32_t Hq, int32_t Hk, int32_t D, eqmp_dtype dtype, const float* pos, const float* freq,
                         int32_t axes) {
  if (N < 0 || Hq < 1 || Hk < 0 || D < 1 || (dtype != EQMP_F32 && dtype != EQMP_BF16)) return EQMP_ERR_INVALID_ARG;
  if (axes < 0 || axes > 3 || (axes > 0 && (D % 2 || (N > 0 && (!pos || !freq)))) || !aligned(pos, 4) || !aligned(freq, 4))
    return EQMP_ERR_INVALID_ARG;
  return N > 1ll << 30 || Hq > kMaxHeads || Hk > kMaxHeads || D > kMaxHeadDim ? EQMP_ERR_UNSUPPORTED : EQMP_OK;
}

static int64_t head_workspace(int64_t N, int32_t D) {
  const int64_t ctas = (N + kHeadWarps - 1) / kHeadWarps, most = 152 * kHeadCtas;
  return (ctas < most ? ctas : most) * 2 * D * 4;
}

template <typename T, int V, int G, int NV>
static eqmp_status launch(HeadNormArgs a, bool backward, cudaStream_t st) {
  // Rows of a step: four of up to 64 values, else two (their angles lie in shared memory); backward one where a lane
  // has 8 values of x and of g, so that three CTAs fit an SM.  100,000 x 16 heads of 32, backward: fp32 four rows 117
  // us, two 121; 50,000 x 8 of 128 two 119, four 124; bf16 one row 113 us, two 129 (two CTAs).
  constexpr int U = G * NV * V <= 64 ? 4 : 2, U_BWD = NV * V >= 8 ? 1 : U;
  const int most = backward ? U_BWD : U, share = a.N / (152 * 64);
  a.each = share < 1 ? 1 : share < most ? share : most;
  a.shift = 0;
  while (a.shift < 5 && 1 << a.shift < a.D / 2) ++a.shift;
  const long long ctas = ((long long)a.N + kHeadWarps * a.each - 1) / (kHeadWarps * a.each);
  if (!backward) {
    DeviceInfo dev;
    const eqmp_status s = device_info(&dev);
    if (s != EQMP_OK) return s;
    const long long most = (long long)dev.sms * 8;
    k_head_norm<T, V, G, NV, U><<<(unsigned)(ctas < most ? ctas : most), 32 * kHeadWarps, 0, st>>>(a);
    return cuda_status(cudaGetLastError());
  }
  const int parts = (int)(ctas < 152 * kHeadCtas ? ctas : 152 * kHeadCtas);
  k_head_norm_bwd<T, V, G, NV, U_BWD><<<parts, 32 * kHeadWarps, 0, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return EQMP_ERR_CUDA;
  if (!a.part) return EQMP_OK;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((2 * a.D + kHeadSumX - 1) / kHeadSumX));
  cfg.blockDim = dim3(kHeadSumX, kHeadSumY);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, k_head_norm_sum, a, parts));
}

template <typename T, int V>
static eqmp_status dispatch(const HeadNormArgs& a, bool backward, cudaStream_t st) {
  const int vectors = (a.D + V - 1) / V;
  if (vectors <= 1) return launch<T, V, 1, 1>(a, backward, st);
  if (vectors <= 2) return launch<T, V, 2, 1>(a, backward, st);
  if (vectors <= 4) return launch<T, V, 4, 1>(a, backward, st);
  if (vectors <= 8) return launch<T, V, 8, 1>(a, backward, st);
  if (vectors <= 16) return launch<T, V, 16, 1>(a, backward, st);
  if (vectors <= 32) return launch<T, V, 32, 1>(a, backward, st);
  if constexpr (V <= 4)
    if (vectors <= 64) return launch<T, V, 32, 2>(a, backward, st);
  if constexpr (V == 2) return launch<T, V, 32, 4>(a, backward, st);
  return EQMP_ERR_UNSUPPORTED;
}

static eqmp_status run(const HeadNormArgs& a, eqmp_dtype dtype, bool vectors, bool backward, cudaStream_t st) {
  if (dtype == EQMP_BF16) return vectors ? dispatch<__nv_bfloat16, 8>(a, backward, st) : dispatch<__nv_bfloat16, 2>(a, backward, st);
  return vectors ? dispatch<float, 4>(a, backward, st) : dispatch<float, 2>(a, backward, st);
}

static bool on16(const void* p, long long ld, int bytes) { return aligned(p, 16) && ld * bytes % 16 == 0; }

}  // namespace eqmp

using namespace eqmp;

extern "C" {

eqmp_status eqmp_head_norm(const void* q, int64_t q_ld, int32_t Hq, const void* k, int64_t k_ld, int32_t Hk, eqmp_dtype dtype,
                           int64_t N, int32_t D, const float* wq, const float* wk, float eps, const float* pos,
                           const float* freq, int32_t axes, void* out_q, void* out_k, float* rstd, eqmp_stream_t stream) {
  const eqmp_status cs = check(N, Hq, Hk, D, dtype, pos, freq, axes);
  if (cs != EQMP_OK) return cs;
  if (!(eps >= 0.0f) || isinf(eps)) return EQMP_ERR_INVALID_ARG;
  if (N == 0 || (!out_q && !out_k && !rstd)) return EQMP_OK;
  const int bytes = dtype == EQMP_BF16 ? 2 : 4;
  const Plane in[] = {{q, q_ld}, {k, k_ld}};
  void* const outs[] = {out_q, out_k};
  if (!q || (Hk > 0 && !k) || !planes_ok(in, 2, outs, 2, bytes) || !aligned(wq, 4) || !aligned(wk, 4) || !aligned(rstd, 4))
    return EQMP_ERR_INVALID_ARG;
  const int64_t cq = (int64_t)Hq * D, ck = (int64_t)Hk * D;
  const Span reads[] = {span(in[0], N, cq, bytes), span(in[1], Hk ? N : 0, ck, bytes), span(wq, D * 4), span(wk, D * 4),
                        span(pos, axes * N * 4), span(freq, axes * (D / 2) * 4)};
  const Span writes[] = {span(out_q, N * cq * bytes), span(out_k, N * ck * bytes), span(rstd, N * (Hq + Hk) * 4)};
  if (!outputs_apart(reads, writes)) return EQMP_ERR_INVALID_ARG;
  HeadNormArgs a{};
  a.q = q, a.q_ld = q_ld, a.k = k, a.k_ld = k_ld, a.wq = wq, a.wk = wk, a.eps = eps;
  a.pos = pos, a.freq = freq, a.axes = axes, a.oq = out_q, a.ok = out_k, a.rstd = rstd;
  a.N = (int)N, a.Hq = Hq, a.Hk = Hk, a.D = D;
  const bool vectors = on16(q, q_ld, bytes) && (!Hk || on16(k, k_ld, bytes)) && aligned(out_q, 16) && aligned(out_k, 16) &&
                       D * bytes % 16 == 0;
  return run(a, dtype, vectors, false, reinterpret_cast<cudaStream_t>(stream));
}

int64_t eqmp_head_norm_backward_workspace_size(int64_t N, int32_t D) {
  return check(N, 1, 0, D, EQMP_F32, nullptr, nullptr, 0) == EQMP_OK ? head_workspace(N, D) : -1;
}

eqmp_status eqmp_head_norm_backward(const void* grad_yq, int64_t grad_yq_ld, const void* grad_yk, int64_t grad_yk_ld,
                                    const void* q, int64_t q_ld, int32_t Hq, const void* k, int64_t k_ld, int32_t Hk,
                                    eqmp_dtype dtype, int64_t N, int32_t D, const float* wq, const float* wk,
                                    const float* rstd, const float* pos, const float* freq, int32_t axes, void* grad_q,
                                    void* grad_k, float* grad_wq, float* grad_wk, float* grad_pos, void* workspace,
                                    int64_t workspace_bytes, eqmp_stream_t stream) {
  const eqmp_status cs = check(N, Hq, Hk, D, dtype, pos, freq, axes);
  if (cs != EQMP_OK) return cs;
  if (grad_pos && !axes) return EQMP_ERR_INVALID_ARG;
  if (!grad_q && !grad_k && !grad_wq && !grad_wk && !grad_pos) return EQMP_OK;
  const int bytes = dtype == EQMP_BF16 ? 2 : 4;
  const Plane in[] = {{q, q_ld}, {k, k_ld}, {grad_yq, grad_yq_ld}, {grad_yk, grad_yk_ld}};
  void* const outs[] = {grad_q, grad_k};
  for (const float* p : {wq, wk, rstd, (const float*)grad_wq, (const float*)grad_wk, (const float*)grad_pos})
    if (!aligned(p, 4)) return EQMP_ERR_INVALID_ARG;
  if (!planes_ok(in, 4, outs, 2, bytes)) return EQMP_ERR_INVALID_ARG;
  if (N > 0 && (!q || !grad_yq || !rstd || (Hk > 0 && (!k || !grad_yk)))) return EQMP_ERR_INVALID_ARG;
  const int64_t ws = grad_wq || grad_wk ? head_workspace(N, D) : 0;
  if (ws > 0 && (!workspace || !aligned(workspace, 16) || workspace_bytes < ws)) return EQMP_ERR_INVALID_ARG;
  const int64_t cq = (int64_t)Hq * D, ck = (int64_t)Hk * D, nk = Hk ? N : 0;
  const Span reads[] = {span(in[0], N, cq, bytes), span(in[1], nk, ck, bytes), span(in[2], N, cq, bytes), span(in[3], nk, ck, bytes),
                        span(wq, D * 4), span(wk, D * 4), span(rstd, N * (Hq + Hk) * 4), span(pos, axes * N * 4),
                        span(freq, axes * (D / 2) * 4)};
  const Span writes[] = {span(grad_q, N * cq * bytes), span(grad_k, N * ck * bytes), span(grad_wq, D * 4), span(grad_wk, D * 4),
                         span(grad_pos, axes * N * 4), span(workspace, ws)};
  if (!outputs_apart(reads, writes)) return EQMP_ERR_INVALID_ARG;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (N == 0) {  // no node: the sums are zero
    if (grad_wq && cudaMemsetAsync(grad_wq, 0, (size_t)D * 4, st) != cudaSuccess) return EQMP_ERR_CUDA;
    if (grad_wk && cudaMemsetAsync(grad_wk, 0, (size_t)D * 4, st) != cudaSuccess) return EQMP_ERR_CUDA;
    return EQMP_OK;
  }
  HeadNormArgs a{};
  a.q = q, a.q_ld = q_ld, a.k = k, a.k_ld = k_ld, a.gq = grad_yq, a.gq_ld = grad_yq_ld, a.gk = grad_yk, a.gk_ld = grad_yk_ld;
  a.wq = wq, a.wk = wk, a.rstd = const_cast<float*>(rstd), a.pos = pos, a.freq = freq, a.axes = axes;
  a.oq = grad_q, a.ok = grad_k, a.gwq = grad_wq, a.gwk = grad_wk, a.gpos = grad_pos;
  a.part = ws > 0 ? static_cast<float*>(workspace) : nullptr;
  a.N = (int)N, a.Hq = Hq, a.Hk = Hk, a.D = D;
  const bool vectors = on16(q, q_ld, bytes) && on16(grad_yq, grad_yq_ld, bytes) && aligned(grad_q, 16) && aligned(grad_k, 16) &&
                       (!Hk || (on16(k, k_ld, bytes) && on16(grad_yk, grad_yk_ld, bytes))) && D * bytes % 16 == 0;
  return run(a, dtype, vectors, true, st);
}

}  // extern "C"
