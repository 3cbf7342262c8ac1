// Log probabilities of given tokens, entropy and top alternatives over rows of logits.
//
// A row is cut into segments of kSeg columns; a block holds a segment in registers (every logit is
// read from memory once), reduces it and takes the next, and the blocks of a cluster share the
// row's segments.  Per segment, with its maximum M:
//   Z = sum e^(x - M),  U = sum e^(x - M) (x - M);   lse = M + ln Z,  entropy = ln Z - U / Z,
// and the segments' sums are merged in their order at the end, so a row's bits do not depend on
// how many blocks it was given.
// Alternatives, ordered by (value, lower column first): the k-th largest of the maxima of 32
// groups of threads bounds the segment's k-th largest element from below, and with it the row's;
// elements at or above the highest such bound so far (about k of the first segment, fewer of each
// later one) are collected and ranked by counting at the end.  Where ties let more than kCand
// elements pass, what is held is ranked at once and the segment is read again and compared as 64-bit
// keys of value and column, all distinct: at most k threads have an element above the k-th
// largest of the threads' largest keys, so at most k * kPer pass, whatever the data.
// What bounds it: at hundreds of rows the logits' bytes (524 x 151,936 fp32: 53 us without
// alternatives, 5.9 TB/s; 68 us with 5, whose bound and collection lengthen every segment's
// chain of barriers); at a few rows that chain and the cluster's two barriers, about 9 us.  Four
// blocks of 256 threads per SM, 40 elements a thread: 512 threads, or 32 or 24 elements, took
// 4 to 40 % longer, three blocks 20 %.  (Four leave 64 registers, of which it spills 44 bytes.)
#include <cooperative_groups.h>

#include "qmm_kv.cuh"

namespace cg = cooperative_groups;

namespace qmm {
namespace logprobs {

constexpr int kThreads = 256;
constexpr int kPer = 40;                  // elements per thread and segment
constexpr int kSeg = kThreads * kPer;
constexpr int kMaxTop = 32;
constexpr int kPerSm = 4;                 // blocks that an SM holds (registers and shared memory)
constexpr int kCand = kMaxTop * (kPer + 1);  // candidates a block holds
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

// A float's bits in an order that integers compare (-0 counts as +0).
__device__ __forceinline__ uint32_t order_of(float v) {
    const uint32_t u = __float_as_uint(v + 0.0f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float from_order(uint32_t o) { return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o); }

__device__ __forceinline__ uint64_t key_of(float v, uint32_t column) {
    return (static_cast<uint64_t>(order_of(v)) << 32) | (0xFFFFFFFFu - column);
}
__device__ __forceinline__ float value_of(uint64_t k) { return from_order(static_cast<uint32_t>(k >> 32)); }
__device__ __forceinline__ uint64_t max64(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
constexpr float kLeast = -3.402823466e38f;  // the least finite value
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
    uint64_t bar;
    alignas(16) float group[2][32];  // maxima of 8 threads each; two, for alternate segments
    uint64_t first[kThreads];    // the threads' largest keys that pass the bound
    uint64_t cand[kCand];        // (at the end, in the cluster's first block: the lists' entries)
    uint64_t list[kMaxTop];      // the block's best, best first; 0, below every element's key: none
    uint64_t best[kMaxTop];
    uint64_t bound;
    float2 part[2][kThreads / 32];
    Sums total;
    Sums sums[kSums];            // of the block's segments, in order
    float raise[2];              // bounds found by one warp for the segments after
    alignas(16) float most[kThreads];  // the threads' largest candidates
    uint32_t least;
    int n_first, n_all, n_cand;
};

// The k-th largest of 32 values in shared memory, `mine` being the lane's: the least of those with
// fewer than k above them.
__device__ __forceinline__ float kth_of_32(const float* all, float mine, int k) {
    int above = 0;
#pragma unroll
    for (int j = 0; j < 32; j += 4) {
        const float4 o = *reinterpret_cast<const float4*>(all + j);
        above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
    }
    return from_order(__reduce_min_sync(0xffffffffu, above < k ? order_of(mine) : 0xFFFFFFFFu));
}

// Ranks cand[0 .. n) by counting and leaves the best k, in order, in `list` (0 past the last) and at
// the front of cand; returns their number.  Only values that are not below the floor can be among them.
// The whole block takes part.
__device__ __noinline__ int rank_candidates(Shared& sh, int n, int k, float floor) {
    const int tid = threadIdx.x;
    if (tid < kMaxTop) sh.list[tid] = 0;
    if (tid == 0) {
        sh.n_first = 0;
        sh.least = 0xFFFFFFFFu;
    }
    if (n > kThreads) {
        // many (600 at 31 alternatives of 151,936 columns): the k-th largest of the threads' largest is a floor
        // that few more than k pass.  (200 rows: 50 us; 84 with all ranked against all.)
        float top = -INFINITY;
        for (int i = tid; i < n; i += kThreads) top = fmaxf(top, value_of(sh.cand[i]));
        sh.most[tid] = top;
        __syncthreads();
        int above = 0;
#pragma unroll 8
        for (int j = 0; j < kThreads; j += 4) {
            const float4 o = *reinterpret_cast<const float4*>(sh.most + j);
            above += (o.x > top) + (o.y > top) + (o.z > top) + (o.w > top);
        }
        const uint32_t least = __reduce_min_sync(0xffffffffu, above < k ? order_of(top) : 0xFFFFFFFFu);
        if ((tid & 31) == 0) atomicMin(&sh.least, least);
        __syncthreads();
        floor = fmaxf(floor, from_order(sh.least));
    }
    __syncthreads();
    const uint64_t* from = sh.cand;
    if (n > 64) {
        for (int i = tid; i < n; i += kThreads)
            if (value_of(sh.cand[i]) >= floor) {
                const int at = atomicAdd(&sh.n_first, 1);
                if (at < kThreads) sh.first[at] = sh.cand[i];
            }
        __syncthreads();
        if (sh.n_first <= kThreads) {
            from = sh.first;
            n = sh.n_first;
        }
    }
    for (int i = tid; i < n; i += kThreads) {
        const uint64_t mine = from[i];
        int rank_of = 0;
#pragma unroll 8
        for (int j = 0; j < n; ++j) rank_of += from[j] > mine;
        if (rank_of < k) sh.list[rank_of] = mine;
    }
    __syncthreads();
    const int left = min(n, k);
    if (tid < left) sh.cand[tid] = sh.list[tid];
    __syncthreads();
    return left;
}

// A segment (cols columns from x, the first of them column `base`) let too many elements pass:
// ties.  The `before` candidates held when it began are cut to the best k, and the segment is read
// again and compared by keys: at most k threads have an element above the k-th largest of the
// threads' largest keys.  Returns the candidates then held, the best k.
template <typename T>
__device__ __noinline__ int redo_by_keys(Shared& sh, const T* x, int base, int cols, int before, int k, float floor) {
    const int tid = threadIdx.x;
    before = rank_candidates(sh, before, k, floor);
    const uint64_t last = sh.list[k - 1];  // 0 unless there are k
    uint64_t best = 0;
#pragma unroll 4
    for (int c = tid; c < cols; c += kThreads) {
        const float v = as_f32(x[c]);
        if (v >= kLeast) best = max64(best, key_of(v, static_cast<uint32_t>(base + c)));
    }
    if (tid == 0) {
        sh.n_first = 0;
        sh.bound = last + 1;
        sh.n_cand = before;
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
    __syncthreads();
    const uint64_t least = sh.bound;
    if (best >= least)
        for (int c = tid; c < cols; c += kThreads) {
            const float v = as_f32(x[c]);
            const uint64_t q = key_of(v, static_cast<uint32_t>(base + c));
            if (v >= kLeast && q >= least) sh.cand[atomicAdd(&sh.n_cand, 1)] = q;
        }
    __syncthreads();
    const int left = rank_candidates(sh, sh.n_cand, k, floor);
    if (tid == 0) sh.n_cand = left;
    __syncthreads();
    return left;
}

template <typename T>
__global__ void __launch_bounds__(kThreads, kPerSm) logprobs_kernel(const Params p) {
    extern __shared__ __align__(16) uint8_t raw[];
    T* buffer = reinterpret_cast<T*>(raw);  // [kSeg]
    Shared& sh = *reinterpret_cast<Shared*>(raw + kSeg * sizeof(T));
    cg::cluster_group cl = cg::this_cluster();
    const int ranks = cl.num_blocks(), rank = cl.block_rank();
    const int64_t row = blockIdx.x / ranks;
    const T* x = static_cast<const T*>(p.logits) + row * p.stride;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // kept sums are dealt out whole: rank r has those of units u0 .. u1 - 1, `fold` segments each
    const int units = (p.segs + p.fold - 1) / p.fold;
    const int u0 = units * rank / ranks, u1 = units * (rank + 1) / ranks;
    const int s0 = min(p.segs, u0 * p.fold), s1 = min(p.segs, u1 * p.fold);
    if (tid == 0) sh.n_cand = 0;
    if (tid < 2) sh.raise[tid] = kLeast;

    constexpr int W = 16 / sizeof(T);  // elements of a 16-byte load
    const int k = p.top;
    Sums fold = {-INFINITY, 0.f, 0.f};
    float bound = kLeast;  // elements below it are not collected (they are not among the k largest, or -infinity)
    float floor = kLeast;  // a value that the k-th largest element so far is not below
    int held = 0;          // candidates so far

    // a segment whose bytes are whole 16-byte pieces comes by a bulk copy into shared memory, asked for
    // as soon as the one before it is in registers
    auto in_bulk = [&](int seg) { return p.vec && (min(static_cast<int64_t>(kSeg), p.n - seg * kSeg) * sizeof(T)) % 16 == 0; };
    auto fetch = [&](int seg) {
        if (!in_bulk(seg)) return;
        const uint32_t bytes = static_cast<uint32_t>(min(static_cast<int64_t>(kSeg), p.n - seg * kSeg) * sizeof(T));
        fence_proxy_async_smem();  // the buffer's reads, before the copy
        mbar_arrive_expect_tx(&sh.bar, bytes);
        bulk_g2s(buffer, x + seg * kSeg, bytes, &sh.bar, l2_policy_evict_first());
    };
    uint32_t phase = 0;
    bool late = false;  // a copy did not arrive in time: the row becomes NaN
    volatile int never = 0;
    if (tid == 0) {
        mbar_init(&sh.bar, 1);
        fence_mbar_init();
        if (s0 < s1) fetch(s0);
    }
    __syncthreads();

    for (int seg = s0; seg < s1; ++seg) {
        const int odd = (seg - s0) & 1;
        const int base = seg * kSeg, cols = static_cast<int>(min(static_cast<int64_t>(kSeg), p.n - base));
        // element i of a thread: column base + (i / W * kThreads + tid) * W + i % W
        auto column = [&](int i) { return (i / W * kThreads + tid) * W + i % W; };
        const bool bulk = !late && in_bulk(seg);
        if (bulk) late |= !mbar_wait_bounded(&sh.bar, phase, &never);
        phase ^= bulk;
        float v[kPer];
#pragma unroll
        for (int i = 0; i < kPer; i += W) {
            const int c = column(i);
            if (bulk) {
                alignas(16) T t[W];
                *reinterpret_cast<uint4*>(t) = *reinterpret_cast<const uint4*>(buffer + c);
#pragma unroll
                for (int j = 0; j < W; ++j) v[i + j] = c < cols ? as_f32(t[j]) : -INFINITY;
            } else if (p.vec && c + W <= cols) {
                alignas(16) T t[W];
                *reinterpret_cast<uint4*>(t) = __ldcs(reinterpret_cast<const uint4*>(x + base + c));
#pragma unroll
                for (int j = 0; j < W; ++j) v[i + j] = as_f32(t[j]);
            } else {
#pragma unroll
                for (int j = 0; j < W; ++j) v[i + j] = c + j < cols ? as_f32(x[base + c + j]) : -INFINITY;
            }
        }
        float top8[kPer / 8], top = -INFINITY;  // the thread's maxima
#pragma unroll
        for (int i = 0; i < kPer; i += 8) {
            float a = v[i];
#pragma unroll
            for (int j = 1; j < 8; ++j) a = fmaxf(a, v[i + j]);
            top8[i / 8] = a;
            top = fmaxf(top, a);
        }
        float gm = top;
#pragma unroll
        for (int b = 1; b < 8; b <<= 1) gm = fmaxf(gm, __shfl_xor_sync(0xffffffffu, gm, b));
        if ((lane & 7) == 0) sh.group[odd][tid >> 3] = gm;
        late = __syncthreads_or(late);  // (also: the buffer is read)
        if (tid == 0 && seg + 1 < s1 && !late) fetch(seg + 1);
        const float group = sh.group[odd][lane];
        if (k > 0) {
            const float b = sh.raise[odd ^ 1];
            bound = fmaxf(bound, b);
            floor = fmaxf(floor, b);
        }
        const float m = from_order(__reduce_max_sync(0xffffffffu, order_of(group)));
        // a NaN, and a +infinity through its difference with itself, ends up in z
        const float ref = m == -INFINITY ? 0.f : m;
        float z = late ? __int_as_float(0x7FFFFFFF) : 0.f, u = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const float d = v[i] - ref, e = ex2(d * kLog2e);
            z += e;
            u = fmaf(e, fmaxf(d, -1e30f), u);
        }
#pragma unroll
        for (int b = 16; b >= 1; b >>= 1) {
            z += __shfl_xor_sync(0xffffffffu, z, b);
            u += __shfl_xor_sync(0xffffffffu, u, b);
        }
        if (lane == 0) sh.part[odd][warp] = make_float2(z, u);
        if (k > 0 && m >= bound) {
            if (seg == s0 || warp == (seg & 7)) {  // one warp in turn, for the segments after
                const float b = kth_of_32(sh.group[odd], group, k);
                if (seg == s0) bound = floor = fmaxf(bound, b);
                else if (lane == 0) sh.raise[odd] = b;
            }
            // (a warp whose lanes hold none skips the elements; one atomic per lane that holds some)
            if (__any_sync(0xffffffffu, top >= bound)) {
                int mine = 0;
#pragma unroll
                for (int i = 0; i < kPer; i += 8)
                    if (__any_sync(0xffffffffu, top8[i / 8] >= bound)) {
#pragma unroll
                        for (int j = i; j < i + 8; ++j) mine += v[j] >= bound;
                    }
                int at = mine ? atomicAdd(&sh.n_cand, mine) : 0;
#pragma unroll
                for (int i = 0; i < kPer; i += 8)
                    if (__any_sync(0xffffffffu, top8[i / 8] >= bound)) {
#pragma unroll
                        for (int j = i; j < i + 8; ++j)
                            if (v[j] >= bound) {
                                if (at < kCand) sh.cand[at] = key_of(v[j], static_cast<uint32_t>(base + column(j)));
                                ++at;
                            }
                    }
            }
        }
        __syncthreads();
        if (tid == kThreads - 1) {
            float2 s = sh.part[odd][0];
#pragma unroll
            for (int w = 1; w < kThreads / 32; ++w) {
                s.x += sh.part[odd][w].x;
                s.y += sh.part[odd][w].y;
            }
            const int in = seg - u0 * p.fold;
            fold = in % p.fold == 0 ? Sums{m, s.x, s.y} : merge(fold, Sums{m, s.x, s.y});
            sh.sums[in / p.fold] = fold;
        }
        if (k > 0) {
            const int now = sh.n_cand;
            if (now <= kCand) {
                held = now;
            } else {
                held = redo_by_keys(sh, x + base, base, cols, held, k, floor);
                if (held == k) {
                    // a later element equal to the k-th best lies in a higher column and loses
                    const float w = value_of(sh.list[k - 1]);
                    floor = fmaxf(floor, w);
                    bound = fmaxf(bound, nextafterf(w, INFINITY));
                }
            }
        }
    }
    if (k > 0) {
        __syncthreads();
        rank_candidates(sh, held, k, floor);
    }
    if (late && tid == 0) mbar_wait_bounded(&sh.bar, phase ^ 1, &never);  // let the copy land before the block exits
    cl.sync();
    if (rank == 0) {
        // ---- the row's sums, as a tree over the units (a fixed one); of the lists, what is not below
        // another list's last
        if (warp == 0) {
            Sums t = {-INFINITY, 0.f, 0.f};
            for (int i = lane; i < units; i += 32) {
                int r = static_cast<int>(static_cast<int64_t>(i) * ranks / units);  // the rank that has unit i
                while (units * (r + 1) / ranks <= i) ++r;
                t = merge(t, cl.map_shared_rank(sh.sums, r)[i - units * r / ranks]);
            }
#pragma unroll
            for (int b = 16; b >= 1; b >>= 1) t = merge(t, shfl_xor(t, b));
            if (lane == 0) sh.total = t;
        } else if (warp == 1 && k > 0) {
            uint64_t bound = lane < ranks ? cl.map_shared_rank(&sh, lane)->list[k - 1] : 0;
#pragma unroll
            for (int b = 16; b >= 1; b >>= 1) bound = max64(bound, __shfl_xor_sync(0xffffffffu, bound, b));
            if (lane == 0) {
                sh.bound = bound;
                sh.n_first = sh.n_all = 0;
            }
        }
        __syncthreads();
        for (int i = tid; i < ranks * k; i += kThreads) {
            const uint64_t mine = cl.map_shared_rank(&sh, i / k)->list[i % k];
            if (mine != 0 && mine >= sh.bound) sh.cand[atomicAdd(&sh.n_all, 1)] = mine;
        }
        __syncthreads();
        const Sums t = sh.total;
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
            const int total = sh.n_all;
            for (int i = tid; i < total; i += kThreads) {
                const uint64_t mine = sh.cand[i];
                int rank_of = 0;
#pragma unroll 8
                for (int j = 0; j < total; ++j) rank_of += sh.cand[j] > mine;
                if (rank_of < k) {
                    sh.best[rank_of] = mine;
                    atomicAdd(&sh.n_first, 1);
                }
            }
            __syncthreads();
            const int found = sh.n_first;
            if (tid < k && (bad || tid < found)) {
                index[tid] = bad ? -1 : static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(sh.best[tid]));
                out[tid] = bad ? nan : lp(value_of(sh.best[tid]));
            } else if (!bad && tid == k - 1) {
                // the lowest columns that are not in the list
                int c = 0;
                for (int i = found; i < k; ++c) {
                    bool in = false;
                    for (int j = 0; j < found; ++j) in |= 0xFFFFFFFFu - static_cast<uint32_t>(sh.best[j]) == static_cast<uint32_t>(c);
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
constexpr int shared_bytes() { return kSeg * static_cast<int>(sizeof(T)) + static_cast<int>(sizeof(Shared)); }

static_assert(kPerSm * (shared_bytes<float>() + 1024) <= 228 * 1024, "the blocks' shared memory");

template <typename T>
cudaError_t launch(const Params& p, int64_t m, int ranks, int dev, cudaStream_t s) {
    static kv::Once once;
    const cudaError_t e = once.allow_shared(logprobs_kernel<T>, dev, 0, true);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(m * ranks));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = shared_bytes<T>();
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
    // blocks per row: what makes the fewest waves of the shortest blocks, in segments' times, a block's
    // start and end counting as two (the row's bits do not depend on it)
    const int32_t segs = static_cast<int32_t>((n + kSeg - 1) / kSeg);
    int ranks = 1;
    int64_t least = INT64_MAX;
    for (int r = 1; r <= kMaxRanks && (r == 1 || r < 2 * segs); r *= 2) {
        const int64_t cost = (m * r + kPerSm * sms - 1) / (kPerSm * sms) * ((segs + r - 1) / r + 2);
        if (cost < least) {
            least = cost;
            ranks = r;
        }
    }
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
    const cudaError_t e = type == QMM_TYPE_F32   ? launch<float>(p, m, ranks, dev, s)
                          : type == QMM_TYPE_F16 ? launch<__half>(p, m, ranks, dev, s)
                                                 : launch<__nv_bfloat16>(p, m, ranks, dev, s);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}
