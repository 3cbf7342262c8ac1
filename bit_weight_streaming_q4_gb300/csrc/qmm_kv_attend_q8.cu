// The attention split kernel's instances for QMM_KV_Q8_0 pools (a translation unit of their own: they
// compile in parallel).
#include "qmm_kv_attend_tc.cuh"

namespace qmm {
namespace kv {

cudaError_t launch_attend_q8(const AttendLaunch& a, cudaStream_t s) {
    return launch_attend_tc<QMM_KV_Q8_0>(a, s);
}

}  // namespace kv
}  // namespace qmm
