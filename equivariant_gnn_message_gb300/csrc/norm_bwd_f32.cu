// Backward of the norms, f32 storage.
#include "norm_rows.cuh"

namespace eqmp {

eqmp_status launch_norm_bwd_rows_f32(const NormArgs& a, int L, const DeviceInfo& dev, cudaStream_t st, bool* done) {
  return launch_rows_t<float, true>(a, L, dev, st, done);
}

}  // namespace eqmp
