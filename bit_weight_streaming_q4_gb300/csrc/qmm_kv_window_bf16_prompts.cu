// Attention with a sliding window: the kernels for prompts over the bf16 pools.
#include "qmm_kv_window.cuh"

namespace qmm {
namespace window {
cudaError_t launch_bf16_prompts(const Launch& a, int head_dim, cudaStream_t s) {
    return head_dim == 64    ? launch_one<QMM_KV_BF16, 64, false>(a, s)
           : head_dim == 128 ? launch_one<QMM_KV_BF16, 128, false>(a, s)
                             : launch_one<QMM_KV_BF16, 256, false>(a, s);
}
}  // namespace window
}  // namespace qmm
