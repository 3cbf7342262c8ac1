// Attention with a sliding window: the kernels for the q8_0 pool.
#include "qmm_kv_window.cuh"

namespace qmm {
namespace window {
cudaError_t launch_q8(const Launch& a, bool decode, cudaStream_t s) {
    return decode ? launch_one<QMM_KV_Q8_0, 128, true>(a, s) : launch_one<QMM_KV_Q8_0, 128, false>(a, s);
}
}  // namespace window
}  // namespace qmm
