#include "attn_launch.cuh"

namespace eqmp {
EQMP_ATTN_LAUNCHER(launch_attn_send_f32) { return launch_attn<kAttnSend, float>(a, f, st); }
}  // namespace eqmp
