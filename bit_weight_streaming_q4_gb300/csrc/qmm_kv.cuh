// Shared by the paged-cache kernels: geometry of the pool's records, argument checks of the C
// entries, and the small device helpers they have in common.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "qmm_ptx.cuh"
#include "qmm_serve.h"

namespace qmm {
namespace kv {

constexpr int kQ8Rec = 17408;   // bytes of a q8_0 record (64 tokens, one KV head)
constexpr int kQ8Half = 8704;   // its K part, and its V part
constexpr int kMaxAgents = 960;      // (the table of sequences shares an SM's memory with the tiles)
constexpr int kMaxShared = 227 * 1024;  // dynamic shared memory of a block
constexpr int kMaxGroupQ = 4096;  // queries of one sequence per KV head in a call
constexpr int kErrTimeout = 1, kErrPage = 2, kErrRange = 4;

// The 16-byte piece key of a q8_0 K row: piece p of token t's row is stored at p ^ key(t).
__host__ __device__ constexpr int q8_key(int t) { return 2 * (t & 3) + ((t >> 2) & 1); }

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Bytes of one (page, KV head) record.
inline int64_t record_bytes(const qmm_kv_dims& d) {
    return d.format == QMM_KV_Q8_0 ? kQ8Rec : int64_t{4} * d.page_tokens * d.head_dim;
}

// The dims of every cache call.  Products are bounded so that slot and item numbers fit 31 bits.
inline qmm_status check_dims(const qmm_kv_dims* d) {
    if (!d || d->heads < 1 || d->kv_heads < 1 || d->heads % d->kv_heads != 0 || d->agents < 1 || d->max_pages < 1 ||
        d->pool_pages < 1 || d->pool_pages > INT32_MAX || d->max_agent_rows < 1)
        return QMM_ERR_INVALID_ARG;
    const int hd = d->head_dim, t = d->page_tokens;
    if (d->format == QMM_KV_Q8_0) {
        if (hd != 128 || t != 64) return QMM_ERR_UNSUPPORTED_SHAPE;
    } else if (d->format == QMM_KV_F16 || d->format == QMM_KV_BF16) {
        if ((hd != 64 && hd != 128 && hd != 256) || (t != 16 && t != 32 && t != 64 && t != 128 && t != 256))
            return QMM_ERR_UNSUPPORTED_SHAPE;
    } else {
        return QMM_ERR_INVALID_ARG;
    }
    if (d->agents > kMaxAgents || d->kv_heads > 65535) return QMM_ERR_UNSUPPORTED_SHAPE;
    if (int64_t{d->max_pages} * t > (int64_t{1} << 30)) return QMM_ERR_UNSUPPORTED_SHAPE;
    return QMM_OK;
}

// The current device, which has to be an sm_103 one, and its number of SMs (looked up once per device).
inline qmm_status check_gpu(int* dev, int* sms) {
    static std::atomic<int> known[64];  // SMs + 1; 1: not an sm_103 device; 0: not looked up
    if (cudaGetDevice(dev) != cudaSuccess) return QMM_ERR_NO_DEVICE;
    int k = *dev >= 0 && *dev < 64 ? known[*dev].load(std::memory_order_relaxed) : 0;
    if (k == 0) {
        int major = 0, minor = 0, n = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, *dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, *dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, *dev) != cudaSuccess)
            return QMM_ERR_NO_DEVICE;
        k = major == 10 && minor == 3 ? n + 1 : 1;
        if (*dev >= 0 && *dev < 64) known[*dev].store(k, std::memory_order_relaxed);
    }
    *sms = k - 1;
    return k > 1 ? QMM_OK : QMM_ERR_NO_DEVICE;
}

// A kernel's attributes, set once per device.
class Once {
    std::atomic<uint64_t> done{0};

public:
    // all the dynamic shared memory that a block without static shared memory, or with `fixed` bytes
    // of it, can have
    template <typename K>
    cudaError_t allow_shared(K kernel, int dev, int fixed = 0, bool big_cluster = false) {
        const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t{1} << dev : 0;
        if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxShared - fixed);
        if (e == cudaSuccess && big_cluster) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
    // clusters of up to 16 blocks
    template <typename K>
    cudaError_t allow_cluster(K kernel, int dev) {
        const uint64_t bit = dev >= 0 && dev < 64 ? uint64_t{1} << dev : 0;
        if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
        return e;
    }
};

// Exclusive prefix of `v` over the block's threads (blockDim.x a multiple of 32, at most 1024)
// and the block's total.  `tmp`: 33 ints of shared memory; every thread takes part, and the
// call ends with the block synchronised.
__device__ __forceinline__ int block_exclusive(int v, int* tmp, int* total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    int s = v;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, s, k);
        if (lane >= k) s += o;
    }
    if (lane == 31) tmp[warp] = s;
    __syncthreads();
    if (warp == 0) {
        const int mine = lane < warps ? tmp[lane] : 0;
        int w = mine;
#pragma unroll
        for (int k = 1; k < 32; k <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, w, k);
            if (lane >= k) w += o;
        }
        if (lane < warps) tmp[lane] = w - mine;
        if (lane == 31) tmp[32] = w;
    }
    __syncthreads();
    const int r = tmp[warp] + s - v;
    *total = tmp[32];
    __syncthreads();
    return r;
}

}  // namespace kv
}  // namespace qmm
