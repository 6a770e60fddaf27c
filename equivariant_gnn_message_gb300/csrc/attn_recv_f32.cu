#include "attn_launch.cuh"

namespace eqmp {
EQMP_ATTN_LAUNCHER(launch_attn_recv_f32) { return launch_attn<kAttnRecv, float>(a, f, st); }
}  // namespace eqmp
