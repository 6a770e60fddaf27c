// Which form of the attention kernels a call gets, and their launches.
#pragma once

#include "attn.cuh"
#include "attn_ring.cuh"
#include "launch.h"

namespace eqmp {

enum { kAttnFwd, kAttnRecv, kAttnSend };

// A form: vectors of VB bytes (0: the general kernels, value by value), G lanes a
// head, up to KN vectors of a key and VN of a value a lane; rows of a warp.
struct AttnForm {
  int VB, G, KN, VN;
  int rows_each;
};

// One launcher for each pass and type (attn_*.cu).
#define EQMP_ATTN_LAUNCHER(name) eqmp_status name(const AttnArgs& a, const AttnForm& f, cudaStream_t st)
EQMP_ATTN_LAUNCHER(launch_attn_fwd_f32);
EQMP_ATTN_LAUNCHER(launch_attn_fwd_bf16);
EQMP_ATTN_LAUNCHER(launch_attn_recv_f32);
EQMP_ATTN_LAUNCHER(launch_attn_recv_bf16);
EQMP_ATTN_LAUNCHER(launch_attn_send_f32);
EQMP_ATTN_LAUNCHER(launch_attn_send_bf16);

// A kernel that waits for the one before it by itself (griddepcontrol.wait).
template <typename Kernel, typename... Args>
eqmp_status launch_behind(Kernel kernel, dim3 grid, cudaStream_t st, const Args&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kJoinX, kJoinY);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// The end of the backward pass: the senders' long rows, cut into `blocks` blocks, and dbias.
template <typename T>
eqmp_status launch_attn_finish(const AttnArgs& a, int blocks, cudaStream_t st) {
  const int ny = a.H < 16 ? a.H : 16, joins = (blocks + kJoinBlocks - 1) / kJoinBlocks * ny;
  const int ctas = joins + (a.gbias ? (int)(((long long)a.E + kFinishEdges - 1) / kFinishEdges) : 0);
  return ctas ? launch_behind(k_attn_finish<T>, dim3((unsigned)ctas), st, a, joins, ny) : EQMP_OK;
}

// The parts of long rows: the kernel is over at once where there are none.
template <int PASS, typename T>
eqmp_status launch_attn_join(const AttnArgs& a, cudaStream_t st) {
  if (cudaGetLastError() != cudaSuccess) return EQMP_ERR_CUDA;
  if constexpr (PASS == kAttnSend) {
    return launch_attn_finish<T>(a, a.blocks, st);
  } else {
    if (!a.blocks) return EQMP_OK;
    const dim3 grid((unsigned)((a.blocks + kJoinBlocks - 1) / kJoinBlocks), (unsigned)(a.H < 16 ? a.H : 16));
    return launch_behind(k_attn_join<PASS == kAttnFwd ? kJoinFwd : kJoinRecv, T>, grid, st, a);
  }
}

template <int PASS, typename T, int V, int G, int KN, int VN>
eqmp_status launch_attn_form(const AttnArgs& a, cudaStream_t st) {
  constexpr int VALUES = VN * V, U = VALUES <= 16 ? 4 : VALUES <= 32 ? 2 : 1;
  const int rows = PASS == kAttnSend ? a.Ns : a.N;
  const dim3 grid((unsigned)((rows + a.blocks + kAttnWarps - 1) / kAttnWarps), (unsigned)((a.H * G + 31) / 32));
  if constexpr (PASS == kAttnFwd)
    k_attn_fwd<T, V, G, KN, VN, U><<<grid, 32 * kAttnWarps, 0, st>>>(a);
  else if constexpr (PASS == kAttnRecv)
    k_attn_bwd_recv<T, V, G, KN, VN, U><<<grid, 32 * kAttnWarps, 0, st>>>(a);
  else
    k_attn_bwd_send<T, V, G, KN, VN, U><<<grid, 32 * kAttnWarps, 0, st>>>(a);
  return launch_attn_join<PASS, T>(a, st);
}

template <int PASS, typename T, int VB, int G, int KN, int VN>
eqmp_status launch_attn_ring(const AttnArgs& a, cudaStream_t st) {
  constexpr int U = KN + VN <= 4 || (sizeof(T) == 2 && KN + VN <= 5) || VB < 16 ? 4 : 2;
  constexpr int SMEM = RingShape<VB, G, KN, VN, U, PASS == kAttnSend ? 12 : 4>::CTA;
  const long long rows = PASS == kAttnSend ? a.Ns : a.N, workers = a.blocks + (rows + a.rows_each - 1) / a.rows_each;
  const dim3 grid((unsigned)((workers + kRingWarps - 1) / kRingWarps), (unsigned)((a.H * G + 31) / 32));
  static unsigned long long done = 0;
  auto run = [&](auto kernel) {
    if (ensure_smem_attr(kernel, SMEM, &done) != cudaSuccess) return EQMP_ERR_CUDA;
    kernel<<<grid, 32 * kRingWarps, SMEM, st>>>(a);
    return launch_attn_join<PASS, T>(a, st);
  };
  if constexpr (PASS == kAttnFwd)
    return run(k_attn_fwd_ring<T, VB, G, KN, VN, U>);
  else if constexpr (PASS == kAttnRecv)
    return run(k_attn_recv_ring<T, VB, G, KN, VN, U>);
  else
    return run(k_attn_send_ring<T, VB, G, KN, VN, U>);
}

template <int PASS, typename T, int VB, int G>
eqmp_status launch_attn_lanes(const AttnArgs& a, const AttnForm& f, cudaStream_t st) {
  if constexpr (VB == 16) {
    if (f.KN <= 1 && f.VN <= 1) return launch_attn_ring<PASS, T, VB, G, 1, 1>(a, st);
  }
  if (f.KN <= 1 && f.VN <= 2) return launch_attn_ring<PASS, T, VB, G, 1, 2>(a, st);
  if (f.KN <= 1 && f.VN <= 4) return launch_attn_ring<PASS, T, VB, G, 1, 4>(a, st);
  if (f.VN <= 4) return launch_attn_ring<PASS, T, VB, G, 2, 4>(a, st);
  return launch_attn_ring<PASS, T, VB, G, 2, 8>(a, st);
}

// Short heads on 8 or 4 bytes: eight lanes each.
template <int PASS, typename T, int VB>
eqmp_status launch_attn_few(const AttnArgs& a, const AttnForm& f, cudaStream_t st) {
  if (f.KN <= 1 && f.VN <= 2) return launch_attn_ring<PASS, T, VB, 8, 1, 2>(a, st);
  return launch_attn_ring<PASS, T, VB, 8, 2, 8>(a, st);
}

template <int PASS, typename T>
eqmp_status launch_attn(AttnArgs a, const AttnForm& f, cudaStream_t st) {
  a.rows_each = f.rows_each;
  if (f.VB == 16) {
    if (f.G == 8) return launch_attn_lanes<PASS, T, 16, 8>(a, f, st);
    if (f.G == 16) return launch_attn_lanes<PASS, T, 16, 16>(a, f, st);
    return launch_attn_lanes<PASS, T, 16, 32>(a, f, st);
  }
  if (f.VB == 8) return f.G == 8 ? launch_attn_few<PASS, T, 8>(a, f, st) : launch_attn_lanes<PASS, T, 8, 16>(a, f, st);
  if (f.VB == 4) return f.G == 8 ? launch_attn_few<PASS, T, 4>(a, f, st) : launch_attn_lanes<PASS, T, 4, 32>(a, f, st);
  if (f.G == 8) return launch_attn_form<PASS, T, 1, 8, 4, 16>(a, st);
  if (f.KN <= 2 && f.VN <= 8) return launch_attn_form<PASS, T, 1, 32, 2, 8>(a, st);
  return launch_attn_form<PASS, T, 1, 32, 8, 32>(a, st);
}

}  // namespace eqmp
