#include "attn_launch.cuh"

namespace eqmp {
EQMP_ATTN_LAUNCHER(launch_attn_recv_bf16) { return launch_attn<kAttnRecv, __nv_bfloat16>(a, f, st); }
}  // namespace eqmp
