// Forward norms, f32 storage.
#include "norm_rows.cuh"

namespace eqmp {

eqmp_status launch_norm_rows_f32(const NormArgs& a, int L, const DeviceInfo& dev, cudaStream_t st, bool* done) {
  return launch_rows_t<float, false>(a, L, dev, st, done);
}

}  // namespace eqmp
