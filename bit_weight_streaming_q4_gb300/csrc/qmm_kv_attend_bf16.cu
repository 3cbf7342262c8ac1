// The attention split kernel's instances for QMM_KV_BF16 pools (a translation unit of their own: they
// compile in parallel).
#include "qmm_kv_attend_tc.cuh"

namespace qmm {
namespace kv {

cudaError_t launch_attend_bf16(const AttendLaunch& a, cudaStream_t s) {
    return a.head_dim == 64    ? launch_attend_dim<QMM_KV_BF16, 64>(a, s)
           : a.head_dim == 128 ? launch_attend_tc<QMM_KV_BF16>(a, s)
                               : launch_attend_dim<QMM_KV_BF16, 256>(a, s);
}

}  // namespace kv
}  // namespace qmm
