// Attention with a sliding window: the kernels for prompts over the fp16 pools.
#include "qmm_kv_window.cuh"

namespace qmm {
namespace window {
cudaError_t launch_f16_prompts(const Launch& a, int head_dim, cudaStream_t s) {
    return head_dim == 64    ? launch_one<QMM_KV_F16, 64, false>(a, s)
           : head_dim == 128 ? launch_one<QMM_KV_F16, 128, false>(a, s)
                             : launch_one<QMM_KV_F16, 256, false>(a, s);
}
}  // namespace window
}  // namespace qmm
