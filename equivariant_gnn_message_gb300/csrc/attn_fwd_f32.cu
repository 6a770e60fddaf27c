#include "attn_launch.cuh"

namespace eqmp {
EQMP_ATTN_LAUNCHER(launch_attn_fwd_f32) { return launch_attn<kAttnFwd, float>(a, f, st); }
}  // namespace eqmp
