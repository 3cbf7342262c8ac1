// Attention with a sliding window: the kernel for the q8_0 pool.
#include "qmm_kv_window.cuh"

namespace qmm {
namespace window {
cudaError_t launch_q8(const Launch& a, cudaStream_t s) { return launch_one<QMM_KV_Q8_0, 128>(a, s); }
}  // namespace window
}  // namespace qmm
