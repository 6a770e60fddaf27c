#include "attn_launch.cuh"

namespace eqmp {
EQMP_ATTN_LAUNCHER(launch_attn_fwd_bf16) { return launch_attn<kAttnFwd, __nv_bfloat16>(a, f, st); }
}  // namespace eqmp
