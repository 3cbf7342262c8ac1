// Log probabilities of given tokens, entropy and top alternatives over rows of logits.
//
// A row is cut into segments of kSeg columns; a block holds a segment in registers (every logit is
// read from memory once), reduces it and takes the next, and the blocks of a cluster share the
// row's segments.  Per segment, with its maximum M:
//   Z = sum e^(x - M),  U = sum e^(x - M) (x - M);   lse = M + ln Z,  entropy = ln Z - U / Z,
// and the segments' sums are merged in their order at the end, so a row's bits do not depend on
// how many blocks it was given.
// Alternatives, ordered by (value, lower column first): the k-th largest of the maxima of 32
// groups of threads bounds the segment's k-th largest element from below; the elements at or
// above it (about k of them) and the block's list so far are ranked by counting.  Where ties let
// more than kCand elements pass, elements are compared as 64-bit keys of value and column, all
// distinct: at most k threads have an element above the k-th largest of the threads' maxima, so
// at most k * kPer pass, whatever the data.
// What bounds it: the logits' bytes.  %LP%
#include <cooperative_groups.h>

#include "qmm_kv.cuh"

namespace cg = cooperative_groups;

namespace qmm {
namespace logprobs {

constexpr int kThreads = 256;
constexpr int kPer = 40;                  // elements per thread and segment
constexpr int kSeg = kThreads * kPer;
constexpr int kMaxTop = 32;
constexpr int kCand = kMaxTop * kPer;     // candidates of a segment
constexpr int kMaxRanks = 16;
constexpr int kSums = 64;                 // segments whose sums a block keeps apart (see the kernel)

struct Params {
    const void* logits;
    const int32_t* tokens;
    float* lse;
    float* entropy;
    float* logprob;
    int32_t* top_index;
    float* top_logprob;
    int64_t n, stride;  // columns, row stride
    int32_t segs;       // segments per row
    int32_t fold;       // segments per kept sum
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
    if (m == -INFINITY) return {m, a.z + b.z, 0.f};  // (0, or a NaN's)
    // (a part without finite elements has z = u = 0; any finite distance will do)
    const float da = fmaxf(a.m - m, -1e30f), db = fmaxf(b.m - m, -1e30f);
    const float ea = ex2(da * kLog2e), eb = ex2(db * kLog2e);
    return {m, a.z * ea + b.z * eb, (a.z > 0.f ? (a.u + a.z * da) * ea : 0.f) + (b.z > 0.f ? (b.u + b.z * db) * eb : 0.f)};
}
__device__ __forceinline__ Sums shfl_xor(const Sums& s, int k) {
    return {__shfl_xor_sync(0xffffffffu, s.m, k), __shfl_xor_sync(0xffffffffu, s.z, k), __shfl_xor_sync(0xffffffffu, s.u, k)};
}

struct Shared {
    float group[2][32];          // maxima of 8 threads each; two, for alternate segments
    uint64_t first[kThreads];    // the threads' largest keys that pass the bound
    uint64_t cand[kCand + kMaxTop];
    uint64_t list[kMaxTop];      // the block's best so far, best first; 0: none
    uint64_t all[kMaxRanks * kMaxTop];
    uint64_t bound;
    Sums part[2][kThreads / 32];
    Sums sums[kSums];            // of the block's segments, in order
    int n_first, n_cand[2];
};

// The k-th largest of 32 lanes' values (every lane returns it).
__device__ __forceinline__ float kth_of_warp(float v, int k) {
    int above = 0, equal = 0;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const float o = __shfl_sync(0xffffffffu, v, j);
        above += o > v;
        equal += o == v && j < static_cast<int>(threadIdx.x & 31);
    }
    const uint32_t who = __ballot_sync(0xffffffffu, above + equal == k - 1);
    return __shfl_sync(0xffffffffu, v, __ffs(who) - 1);
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) logprobs_kernel(const Params p) {
    extern __shared__ __align__(16) uint8_t raw[];
    Shared& sh = *reinterpret_cast<Shared*>(raw);
    cg::cluster_group cl = cg::this_cluster();
    const int ranks = cl.num_blocks(), rank = cl.block_rank();
    const int64_t row = blockIdx.x / ranks;
    const T* x = static_cast<const T*>(p.logits) + row * p.stride;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // kept sums are dealt out whole: rank r has those of units u0 .. u1 - 1, `fold` segments each
    const int units = (p.segs + p.fold - 1) / p.fold;
    const int u0 = units * rank / ranks, u1 = units * (rank + 1) / ranks;
    const int s0 = min(p.segs, u0 * p.fold), s1 = min(p.segs, u1 * p.fold);
    if (tid < kMaxTop) sh.list[tid] = 0;  // below every key of an element
    if (tid < 2) sh.n_cand[tid] = 0;

    constexpr int W = 16 / sizeof(T);  // elements of a 16-byte load
    const int k = p.top;
    Sums fold = {-INFINITY, 0.f, 0.f};
    for (int seg = s0; seg < s1; ++seg) {
        const int odd = (seg - s0) & 1;
        const int base = seg * kSeg, cols = static_cast<int>(min(static_cast<int64_t>(kSeg), p.n - base));
        // element i of a thread: column base + (i / W * kThreads + tid) * W + i % W
        auto column = [&](int i) { return (i / W * kThreads + tid) * W + i % W; };
        float v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i += W) {
            const int c = column(i);
            if (p.vec && c + W <= cols) {
                alignas(16) T t[W];
                *reinterpret_cast<uint4*>(t) = __ldcs(reinterpret_cast<const uint4*>(x + base + c));
#pragma unroll
                for (int j = 0; j < W; ++j) v[i + j] = as_f32(t[j]);
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) v[i + j] = c + j < cols ? as_f32(x[base + c + j]) : -INFINITY;
            }
        }
        float top = -INFINITY;
#pragma unroll
        for (int i = 0; i < kPer; ++i) top = fmaxf(top, v[i]);
        if (k > 0) {
            float gm = top;
#pragma unroll
            for (int b = 1; b < 8; b <<= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, b));
            if ((lane & 7) == 0) sh.group[odd][tid >> 3] = gm;
        }
        // a NaN, and a +infinity through its difference with itself, ends up in z
        const float ref = top == -INFINITY ? 0.f : top;
        Sums s = {top, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float d = v[i] - ref, e = ex2(d * kLog2e);
            s.z += e;
            s.u = fmaf(e, fmaxf(d, -1e30f), s.u);
        }
#pragma unroll
        for (int b = 16; b >= 1; b >>= 1) s = merge(s, shfl_xor(s, b));
        if (lane == 0) sh.part[odd][warp] = s;
        __syncthreads();  // (also: the last segment's list is complete)
        if (tid == 0) {
            Sums t = sh.part[odd][0];
#pragma unroll
            for (int w = 1; w < kThreads / 32; ++w) t = merge(t, sh.part[odd][w]);
            const int in = seg - u0 * p.fold;
            fold = in % p.fold == 0 ? t : merge(fold, t);
            sh.sums[in / p.fold] = fold;
        }
        if (k > 0) {
            // ---- the bound.  An element equal to the list's last lies in a higher column and loses;
            // -infinity is left to the end
            const float group = kth_of_warp(sh.group[odd][lane], k);
            const uint64_t last = sh.list[k - 1];
            const float worst = last ? value_of(last) : -INFINITY;
            const bool strict = group <= worst;
            const float bound = strict ? worst : group;
            if (strict ? top > bound : top >= bound) {
#pragma unroll
                for (int i = 0; i < kPer; ++i) {
                    if (strict ? v[i] > bound : v[i] >= bound) {
                        const int at = atomicAdd(&sh.n_cand[odd], 1);
                        if (at < kCand) sh.cand[at] = key_of(v[i], static_cast<uint32_t>(base + column(i)));
                    }
                }
            }
            __syncthreads();
            int fresh = sh.n_cand[odd];
            if (fresh > kCand) {
                // ---- ties: the same by keys, with the threads' largest keys as the groups
                uint64_t best = 0;
#pragma unroll
                for (int i = 0; i < kPer; ++i)
                    if (best == 0 && v[i] == top && top > -INFINITY) best = key_of(v[i], static_cast<uint32_t>(base + column(i)));
                if (tid == 0) {
                    sh.n_first = 0;
                    sh.bound = last + 1;
                }
                __syncthreads();
                if (best > last) sh.first[atomicAdd(&sh.n_first, 1)] = best;
                __syncthreads();
                const int nf = sh.n_first;
                if (tid < nf) {
                    const uint64_t mine = sh.first[tid];
                    int rank_of = 0;
                    for (int j = 0; j < nf; ++j) rank_of += sh.first[j] > mine;
                    if (rank_of == k - 1) sh.bound = mine;
                }
                if (tid == 0) sh.n_cand[odd] = 0;
                __syncthreads();
                const uint64_t from = sh.bound;
                if (best >= from) {
#pragma unroll
                    for (int i = 0; i < kPer; ++i) {
                        const uint64_t q = key_of(v[i], static_cast<uint32_t>(base + column(i)));
                        if (v[i] > -INFINITY && q >= from) sh.cand[atomicAdd(&sh.n_cand[odd], 1)] = q;
                    }
                }
                __syncthreads();
                fresh = sh.n_cand[odd];
            }
            if (tid == 0) sh.n_cand[odd ^ 1] = 0;
            if (fresh > 0) {
                // ---- the candidates and the list so far, ranked by counting
                if (tid < k) sh.cand[fresh + tid] = sh.list[tid];
                __syncthreads();
                for (int i = tid; i < fresh + k; i += kThreads) {
                    const uint64_t mine = sh.cand[i];
                    int rank_of = 0;
#pragma unroll 8
                    for (int j = 0; j < fresh + k; ++j) rank_of += sh.cand[j] > mine;
                    if (mine != 0 && rank_of < k) sh.list[rank_of] = mine;
                }
            }
        }
    }
    cl.sync();
    if (rank == 0) {
        // ---- the row's sums, in the segments' order
        if (warp == 0) {
            Sums t = {-INFINITY, 0.f, 0.f};
            for (int r = 0; r < ranks; ++r) {
                const Sums* o = cl.map_shared_rank(sh.sums, r);
                const int n = units * (r + 1) / ranks - units * r / ranks;
                for (int i = 0; i < n; ++i) t = merge(t, o[i]);
            }
            if (lane == 0) sh.part[0][0] = t;
        } else if (k > 0) {
            for (int i = tid - 32; i < ranks * k; i += kThreads - 32) sh.all[i] = cl.map_shared_rank(&sh, i / k)->list[i % k];
        }
        __syncthreads();
        const Sums t = sh.part[0][0];
        const bool bad = t.z != t.z;
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
        if (k > 0) {
            int32_t* index = p.top_index + row * k;
            float* out = p.top_logprob + row * k;
            // how many there are (fewer than k only if the rest of the row is -infinity)
            const int total = ranks * k;
            if (tid == 0) sh.n_first = 0;
            __syncthreads();
            for (int i = tid; i < total; i += kThreads) {
                const uint64_t mine = sh.all[i];
                if (mine == 0) continue;
                int rank_of = 0;
#pragma unroll 8
                for (int j = 0; j < total; ++j) rank_of += sh.all[j] > mine;
                if (rank_of < k) {
                    sh.list[rank_of] = mine;
                    atomicAdd(&sh.n_first, 1);
                }
            }
            __syncthreads();
            const int found = sh.n_first;
            if (tid < k && (bad || tid < found)) {
                index[tid] = bad ? -1 : static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(sh.list[tid]));
                out[tid] = bad ? nan : lp(value_of(sh.list[tid]));
            } else if (!bad && tid == k - 1) {
                // the lowest columns that are not in the list
                int c = 0;
                for (int i = found; i < k; ++c) {
                    bool in = false;
                    for (int j = 0; j < found; ++j) in |= 0xFFFFFFFFu - static_cast<uint32_t>(sh.list[j]) == static_cast<uint32_t>(c);
                    if (in) continue;
                    index[i] = c;
                    out[i++] = -INFINITY;
                }
            }
        }
    }
    cl.sync();  // no block leaves while its shared memory is read
}

template <typename T>
cudaError_t launch(const Params& p, int64_t m, int ranks, cudaStream_t s) {
    cudaError_t e = cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(Shared));
    if (e == cudaSuccess && ranks > 8) e = cudaFuncSetAttribute(logprobs_kernel<T>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
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
    if (type < QMM_TYPE_F32 || type > QMM_TYPE_BF16 || m < 0 || n < 1 || n > (1 << 30) || stride < n || given < 0 || top < 0 ||
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
    // blocks per row: the fewest that give every SM six, up to one per segment and the largest
    // cluster (the row's bits do not depend on it)
    const int32_t segs = static_cast<int32_t>((n + kSeg - 1) / kSeg);
    int ranks = 1;
    while (ranks < kMaxRanks && ranks < segs && m * ranks < 6 * sms) ranks *= 2;
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
    p.segs = segs;
    p.fold = (segs + kSums - 1) / kSums;  // by the number of columns alone
    p.given = given;
    p.top = top;
    p.vec = aligned(logits, 16) && stride * size % 16 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = type == QMM_TYPE_F32   ? launch<float>(p, m, ranks, s)
                          : type == QMM_TYPE_F16 ? launch<__half>(p, m, ranks, s)
                                                 : launch<__nv_bfloat16>(p, m, ranks, s);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}
