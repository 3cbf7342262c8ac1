// Log probabilities of given tokens, entropy and top alternatives over rows of logits.
//
// One cluster of blocks per row, the row cut evenly among them; a block takes its slice in rounds
// of kRound elements held in registers, so every logit is read from memory once.  With running
// maximum M, per thread and then merged:
//   Z = sum e^(x - M),  U = sum e^(x - M) (x - M);   lse = M + ln Z,  entropy = ln Z - U / Z.
// Alternatives: elements are ordered by (value, lower column first) as 64-bit keys, all distinct.
// The k-th largest of the threads' maxima bounds the k-th largest element from below, and at
// most k threads hold elements above it: so at most k * kPer elements pass the bound, whatever the
// data (a first, coarser bound from the maxima of 32 groups of threads makes it about
// k in practice).  They and the block's list so far are ranked by counting, and the cluster's
// lists in the same way at the end.
#include <cooperative_groups.h>

#include "qmm_kv.cuh"

namespace cg = cooperative_groups;

namespace qmm {
namespace logprobs {

constexpr int kThreads = 512;
constexpr int kPer = 32;                  // elements per thread and round
constexpr int kRound = kThreads * kPer;
constexpr int kMaxTop = 32;
constexpr int kCand = 64 * kPer;          // candidates of a round
constexpr int kMaxRanks = 8;

struct Params {
    const void* logits;
    const int32_t* tokens;
    float* lse;
    float* entropy;
    float* logprob;
    int32_t* top_index;
    float* top_logprob;
    int64_t n, stride, slice;  // columns, row stride, columns per block
    int32_t given, top;
    int32_t vec;  // rows can be read 16 bytes at a time
};

__device__ __forceinline__ uint64_t key_of(float v, uint32_t column) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (static_cast<uint64_t>((u & 0x80000000u) ? ~u : (u | 0x80000000u)) << 32) | (0xFFFFFFFFu - column);
}
__device__ __forceinline__ float value_of(uint64_t k) {
    const uint32_t o = static_cast<uint32_t>(k >> 32);
    return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// The merge of (M, Z, U) pairs: everything relative to the larger maximum.
struct Sums {
    float m, z, u;
};
__device__ __forceinline__ Sums merge(const Sums& a, const Sums& b) {
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return {m, 0.f, 0.f};
    // (a part without finite elements has z = u = 0; any finite distance will do)
    const float da = fmaxf(a.m - m, -1e30f), db = fmaxf(b.m - m, -1e30f);
    const float ea = ex2(da * kLog2e), eb = ex2(db * kLog2e);
    return {m, a.z * ea + b.z * eb, (a.z > 0.f ? (a.u + a.z * da) * ea : 0.f) + (b.z > 0.f ? (b.u + b.z * db) * eb : 0.f)};
}
__device__ __forceinline__ Sums shfl_xor(const Sums& s, int k) {
    return {__shfl_xor_sync(0xffffffffu, s.m, k), __shfl_xor_sync(0xffffffffu, s.z, k), __shfl_xor_sync(0xffffffffu, s.u, k)};
}

struct Shared {
    uint64_t group[32];          // maxima of 16 threads each
    uint64_t first[kThreads];    // the threads' maxima that pass the coarse bound
    uint64_t cand[kCand + kMaxTop];
    uint64_t list[kMaxTop];      // the slice's best so far, best first
    uint64_t all[kMaxRanks * kMaxTop];
    uint64_t bound;
    Sums part[kThreads / 32];
    Sums total;
    int odd;                     // the slice has a NaN or +infinity
    int n_first, n_cand;
};

template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_kernel(const Params p) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    cg::cluster_group cl = cg::this_cluster();
    const int ranks = cl.num_blocks(), rank = cl.block_rank();
    const int64_t row = blockIdx.x / ranks;
    const T* x = static_cast<const T*>(p.logits) + row * p.stride;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t c0 = min(p.n, rank * p.slice), c1 = min(p.n, c0 + p.slice);
    if (tid == 0) sh.odd = 0;
    if (tid < kMaxTop) sh.list[tid] = 0;  // below every key of an element
    __syncthreads();

    constexpr int W = 16 / sizeof(T);  // elements of a 16-byte load
    Sums s = {-INFINITY, 0.f, 0.f};
    bool odd = false;
    for (int64_t r0 = c0; r0 < c1; r0 += kRound) {
        // element i of a thread: r0 + (i / W * kThreads + tid) * W + i % W
        float v[kPer];
        float top = -INFINITY;
        auto column = [&](int i) { return r0 + (static_cast<int64_t>(i / W) * kThreads + tid) * W + i % W; };
#pragma unroll
        for (int i = 0; i < kPer; i += W) {
            const int64_t c = column(i);
            if (p.vec && c + W <= c1) {
                alignas(16) T t[W];
                *reinterpret_cast<uint4*>(t) = __ldcs(reinterpret_cast<const uint4*>(x + c));
#pragma unroll
                for (int k = 0; k < W; ++k) v[i + k] = as_f32(t[k]);
            } else {
#pragma unroll
                for (int k = 0; k < W; ++k) v[i + k] = c + k < c1 ? as_f32(x[c + k]) : -INFINITY;
            }
        }
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            odd |= !(v[i] < INFINITY);  // NaN or +infinity
            top = fmaxf(top, v[i]);
        }
        if (top > -INFINITY) {
            Sums t = {top, 0.f, 0.f};
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                const float d = fmaxf(v[i] - top, -1e30f), e = ex2(d * kLog2e);
                t.z += e;
                t.u = fmaf(e, d, t.u);
            }
            s = merge(s, t);
        }
        if (p.top > 0) {
            const int k = p.top;
            // the thread's largest key (its lowest column among equals); columns past the end have none
            uint64_t best = 0;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (v[i] == top && best == 0 && column(i) < c1) best = key_of(v[i], static_cast<uint32_t>(column(i)));
            // ---- the coarse bound: the k-th largest of 32 groups' maxima, or the list's k-th
            uint64_t gm = best;
#pragma unroll
            for (int b = 1; b < 16; b <<= 1) gm = max64(gm, __shfl_xor_sync(0xffffffffu, gm, b));
            if ((lane & 15) == 0) sh.group[tid >> 4] = gm;
            if (tid == 0) sh.n_first = sh.n_cand = 0;
            __syncthreads();
            if (warp == 0) {
                const uint64_t mine = sh.group[lane];
                int rank_of = 0;
                for (int j = 0; j < 32; ++j) {
                    const uint64_t o = sh.group[j];
                    rank_of += o > mine || (o == mine && j < lane);
                }
                if (rank_of == k - 1) sh.bound = max64(mine, sh.list[k - 1]);
            }
            __syncthreads();
            uint64_t bound = sh.bound;
            // ---- the threads whose maximum passes; if they are many, the k-th largest maximum
            const bool in = best != 0 && best >= bound;
            if (in) sh.first[atomicAdd(&sh.n_first, 1)] = best;
            __syncthreads();
            const int nf = sh.n_first;
            if (nf > kCand / kPer) {
                for (int i = tid; i < nf; i += kThreads) {
                    const uint64_t mine = sh.first[i];
                    int rank_of = 0;
                    for (int j = 0; j < nf; ++j) rank_of += sh.first[j] > mine;
                    if (rank_of == k - 1) sh.bound = max64(mine, sh.bound);
                }
                __syncthreads();
                bound = sh.bound;
            }
            // ---- the elements that pass, and the list so far, ranked by counting
            if (best != 0 && best >= bound) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    const int64_t c = column(i);
                    if (c < c1) {
                        const uint64_t q = key_of(v[i], static_cast<uint32_t>(c));
                        if (q >= bound) sh.cand[atomicAdd(&sh.n_cand, 1)] = q;
                    }
                }
            }
            __syncthreads();
            const int fresh = sh.n_cand;
            if (fresh > 0) {
                if (tid < k) sh.cand[fresh + tid] = sh.list[tid];
                __syncthreads();
                for (int i = tid; i < fresh + k; i += kThreads) {
                    const uint64_t mine = sh.cand[i];
                    int rank_of = 0;
                    for (int j = 0; j < fresh + k; ++j) rank_of += sh.cand[j] > mine;
                    if (mine != 0 && rank_of < k) sh.list[rank_of] = mine;
                }
            }
            __syncthreads();
        }
    }

    // ---- the block's sums, in a fixed order
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) s = merge(s, shfl_xor(s, k));
    if (lane == 0) sh.part[warp] = s;
    if (odd) sh.odd = 1;
    __syncthreads();
    if (tid == 0) {
        Sums t = sh.part[0];
        for (int w = 1; w < kThreads / 32; ++w) t = merge(t, sh.part[w]);
        sh.total = t;
    }
    cl.sync();
    if (rank == 0) {
        // every thread merges the cluster's sums; the lists are ranked as before
        Sums t = sh.total;
        bool bad = sh.odd != 0;
        for (int r = 1; r < ranks; ++r) {
            const Shared* o = cl.map_shared_rank(&sh, r);
            t = merge(t, o->total);
            bad |= o->odd != 0;
        }
        const float nan = __int_as_float(0x7FFFFFFF);
        const float lz = logf(t.z);
        const bool none = t.m == -INFINITY;
        auto lp = [&](float v) { return bad ? nan : none || v == -INFINITY ? -INFINITY : (v - t.m) - lz; };
        if (tid == 0) {
            if (p.lse) p.lse[row] = bad ? nan : none ? -INFINITY : t.m + lz;
            if (p.entropy) p.entropy[row] = bad ? nan : none ? 0.f : fmaxf(lz - t.u / t.z, 0.f);
        }
        for (int i = tid; i < p.given; i += kThreads) {
            const int64_t tok = p.tokens[row * p.given + i];
            p.logprob[row * p.given + i] = tok >= 0 && tok < p.n ? lp(as_f32(x[tok])) : nan;
        }
        const int total = ranks * p.top;
        if (bad) {
            for (int i = tid; i < p.top; i += kThreads) {
                p.top_index[row * p.top + i] = -1;
                p.top_logprob[row * p.top + i] = nan;
            }
        } else if (p.top > 0) {
            for (int i = tid; i < total; i += kThreads)
                sh.all[i] = cl.map_shared_rank(&sh, i / p.top)->list[i % p.top];
            __syncthreads();
            for (int i = tid; i < total; i += kThreads) {
                const uint64_t mine = sh.all[i];
                int rank_of = 0;
                for (int j = 0; j < total; ++j) rank_of += sh.all[j] > mine;
                if (mine != 0 && rank_of < p.top) {
                    const int64_t at = row * p.top + rank_of;
                    p.top_index[at] = static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(mine));
                    p.top_logprob[at] = lp(value_of(mine));
                }
            }
        }
    }
    cl.sync();  // no block leaves while its shared memory is read
}

template <typename T>
cudaError_t launch(const Params& p, int64_t m, int ranks, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(m * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Shared);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, logprobs_kernel<T>, p);
}

}  // namespace logprobs
}  // namespace qmm

extern "C" qmm_status qmm_logprobs(const void* logits, int32_t type, int64_t m, int64_t n, int64_t stride,
                                   const int32_t* tokens, int32_t given, int32_t top, float* lse, float* entropy,
                                   float* logprob, int32_t* top_index, float* top_logprob, void* stream) {
    using namespace qmm::logprobs;
    if (type < QMM_TYPE_F32 || type > QMM_TYPE_BF16 || m < 0 || n < 1 || n > INT32_MAX || stride < n || given < 0 || top < 0 ||
        top > kMaxTop || top > n || (given > 0 && (!tokens || !logprob)) || (top > 0 && (!top_index || !top_logprob)))
        return QMM_ERR_INVALID_ARG;
    if (m == 0) return QMM_OK;
    if (!logits || m > INT32_MAX / kMaxRanks) return QMM_ERR_INVALID_ARG;
    const int size = type == QMM_TYPE_F32 ? 4 : 2;
    using qmm::kv::aligned;
    if (!aligned(logits, size) || !aligned(tokens, 4) || !aligned(lse, 4) || !aligned(entropy, 4) || !aligned(logprob, 4) ||
        !aligned(top_index, 4) || !aligned(top_logprob, 4))
        return QMM_ERR_MISALIGNED;
    int dev = 0, sms = 0;
    const qmm_status st = qmm::kv::check_gpu(&dev, &sms);
    if (st != QMM_OK) return st;
    // blocks per row, by the number of columns alone (so that a row's bits do not depend on the
    // other rows of the call): up to 8, the portable limit, of 8 elements a thread or more
    int ranks = 1;
    while (ranks < kMaxRanks && n > int64_t{ranks} * kThreads * 8) ranks *= 2;
    Params p = {};
    p.logits = logits;
    p.tokens = tokens;
    p.lse = lse;
    p.entropy = entropy;
    p.logprob = logprob;
    p.top_index = top_index;
    p.top_logprob = top_logprob;
    p.n = n;
    p.stride = stride;
    p.slice = ((n + ranks - 1) / ranks + 7) / 8 * 8;
    p.given = given;
    p.top = top;
    p.vec = aligned(logits, 16) && stride * size % 16 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = type == QMM_TYPE_F32   ? launch<float>(p, m, ranks, s)
                          : type == QMM_TYPE_F16 ? launch<__half>(p, m, ranks, s)
                                                 : launch<__nv_bfloat16>(p, m, ranks, s);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}
