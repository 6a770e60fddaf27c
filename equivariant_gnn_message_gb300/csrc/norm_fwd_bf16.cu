// Forward norms, bf16 storage.
#include "norm_rows.cuh"

namespace eqmp {

eqmp_status launch_norm_rows_bf16(const NormArgs& a, int L, const DeviceInfo& dev, cudaStream_t st, bool* done) {
  return launch_rows_t<__nv_bfloat16, false>(a, L, dev, st, done);
}

}  // namespace eqmp
