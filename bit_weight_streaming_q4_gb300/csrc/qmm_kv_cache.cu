// The paged cache's contents: appending new tokens' K and V, and eviction by accumulated
// attention weight.
#include <cooperative_groups.h>

#include "qmm_kv.cuh"

namespace cg = cooperative_groups;

namespace qmm {
namespace kv {

// ------------------------------------------------------------------------------ append
// One block per 32 slots of a sequence (aligned in slot numbers, so that a q8_0 group lies in
// one page) and KV head; a warp per token, lanes over the head dimension.  The rows' bytes bound
// it (read once, written once): 8,191 fp32 rows of 8 heads into fp16 take 20 us, 5.0 TB/s (23 with 64
// slots a block, 21 with 128); a decode step's few rows cost a launch and one chain of loads, 4 us.
// A q8_0 record keeps V dim-major: the block collects its tokens' V quants in shared memory and
// writes each dim's 32 bytes at once where all 32 slots are new.
constexpr int kAppendThreads = 256;

struct AppendParams {
    uint8_t* pool;
    const int32_t* table;
    const int32_t* agent_rows;
    const int32_t* cache_len;
    const void* src[2];  // K, V
    int64_t stride[2];   // elements per row
    float* weight;
    int32_t* pos;
    const int32_t* row_pos;
    int* err;
    int64_t rec_bytes;
    int32_t rows, agents, kv_heads, max_pages, pool_pages, page_tokens, cap;
    int32_t vec;  // rows can be read 4 elements at a time
};

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// E elements from src, aligned to 4 elements if `vec` (E a multiple of 4) or 2 (E = 2).
template <typename T, int E>
__device__ __forceinline__ void load_row(const T* src, int vec, float (&v)[E]) {
    constexpr int W = E < 4 ? E : 4;
    if (vec) {
#pragma unroll
        for (int i = 0; i < E; i += W) {
            alignas(sizeof(T) * W) T t[W];
            if constexpr (sizeof(T) * W == 16) *reinterpret_cast<uint4*>(t) = *reinterpret_cast<const uint4*>(src + i);
            else if constexpr (sizeof(T) * W == 8) *reinterpret_cast<uint2*>(t) = *reinterpret_cast<const uint2*>(src + i);
            else *reinterpret_cast<uint32_t*>(t) = *reinterpret_cast<const uint32_t*>(src + i);
#pragma unroll
            for (int k = 0; k < W; ++k) v[i + k] = to_f32(t[k]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = to_f32(src[i]);
    }
}

template <int FMT>
__device__ __forceinline__ uint16_t to_16(float v) {
    if constexpr (FMT == QMM_KV_BF16) return __bfloat16_as_ushort(__float2bfloat16_rn(v));
    else return __half_as_ushort(__float2half_rn(v));
}

// q8_0 of a 32-dim block held by 8 lanes, 4 dims each: the block's scale (all lanes) and the
// lane's four quants.  All in fp32, rounded as the header says.
__device__ __forceinline__ __half quantise(const float (&v)[4], uint32_t& q) {
    float big = 0.f;
    bool fine = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        big = fmaxf(big, fabsf(v[i]));
        fine &= fabsf(v[i]) <= 3.4028235e38f;  // false for NaN and infinities
    }
#pragma unroll
    for (int k = 1; k < 8; k <<= 1) {
        big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, k));
        fine &= __shfl_xor_sync(0xffffffffu, fine ? 1 : 0, k) != 0;
    }
    if (!fine) {
        q = 0;
        return __ushort_as_half(0x7FFFu);
    }
    const __half d = __float2half_rn(fminf(__fdiv_rn(big, 127.f), 65504.f));
    const float df = __half2float(d);
    const float inv = df == 0.f ? 0.f : __frcp_rn(df);
    q = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float r = fminf(fmaxf(rintf(__fmul_rn(v[i], inv)), -127.f), 127.f);
        q |= (static_cast<uint32_t>(static_cast<int>(r)) & 0xFFu) << (8 * i);
    }
    return d;
}

template <int FMT, int D, typename T>
__global__ void __launch_bounds__(kAppendThreads) kv_append_kernel(const AppendParams p) {
    constexpr bool q8 = FMT == QMM_KV_Q8_0;
    constexpr int E = D / 32;
    __shared__ int tmp[33], mine[5];
    // [dim][slot of the group], a word further every four dims: a warp's lanes, four dims apart, then store to
    // 32 different banks
    __shared__ __align__(16) uint8_t vq[q8 ? 128 * 32 + 32 * 4 : 16];
    auto vq_at = [](int d) { return d * 32 + (d >> 2) * 4; };
    __shared__ __half vs[q8 ? 4 * 32 : 8];                    // [block][slot]
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = blockIdx.y;
    // this block's sequence and group of slots
    if (tid == 0) mine[0] = -1;
    __syncthreads();
    // (where agent_rows falls anywhere, sequences could share rows, and be more than the grid holds: none is taken)
    int before = 0;
    bool falls = false;
    for (int a0 = 0; a0 < p.agents; a0 += kAppendThreads) {
        const int a = a0 + tid;
        int n = 0, r0 = 0, nr = 0, len = 0;
        if (a < p.agents) {
            r0 = p.agent_rows[a];
            const int r1 = p.agent_rows[a + 1];
            falls |= r1 < r0;
            nr = r0 >= 0 && r1 >= r0 ? r1 - r0 : -1;
            len = p.cache_len[a];
            const bool ok = nr >= 0 && nr <= p.rows - r0 && len >= 0 && len <= p.cap && nr <= p.cap - len;
            if (!ok && blockIdx.x == 0 && g == 0) atomicOr(p.err, kErrRange);
            if (ok && nr > 0) n = (len + nr - 1) / 32 - len / 32 + 1;
        }
        int sum;
        const int at = before + block_exclusive(n, tmp, &sum);
        const int i = static_cast<int>(blockIdx.x) - at;
        if (i >= 0 && i < n) {
            mine[0] = a;
            mine[1] = (len / 32 + i) * 32;  // the group's first slot
            mine[2] = len;
            mine[3] = len + nr;
            mine[4] = r0;
        }
        before += sum;
    }
    if (__syncthreads_or(falls)) return;
    const int a = mine[0];
    if (a < 0) return;
    const int base = mine[1], lo = max(mine[2], base), hi = min(mine[3], base + 32), row0 = mine[4] - mine[2];

    // a warp's tokens, some at once: their loads are in flight together
    // (one at a time 21 us in the case above, four 23: registers leave too few blocks)
    constexpr int kWarps = kAppendThreads / 32, kBatch = 2;
    for (int t0 = lo + warp; t0 < hi; t0 += kWarps * kBatch) {
        float kv[kBatch][2][E];
        int pages[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int t = t0 + k * kWarps;
            if (t >= hi) continue;
            pages[k] = p.table[static_cast<int64_t>(a) * p.max_pages + t / p.page_tokens];
#pragma unroll
            for (int i = 0; i < 2; ++i)
                load_row<T, E>(static_cast<const T*>(p.src[i]) + (row0 + t) * p.stride[i] + g * D + lane * E, p.vec, kv[k][i]);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int t = t0 + k * kWarps;
            if (t >= hi) continue;
            const int pg = pages[k];
            const bool in = pg >= 0 && pg < p.pool_pages;
            if (!in && lane == 0) atomicOr(p.err, kErrPage);
            const int slot = t % p.page_tokens;
            uint8_t* rec = p.pool + (static_cast<int64_t>(in ? pg : 0) * p.kv_heads + g) * p.rec_bytes;
            if constexpr (q8) {
                uint32_t q;
                const __half dk = quantise(kv[k][0], q);
                if (in) {
                    *reinterpret_cast<uint32_t*>(rec + slot * 128 + 16 * ((lane >> 2) ^ q8_key(slot)) + 4 * (lane & 3)) = q;
                    if ((lane & 7) == 0) *reinterpret_cast<__half*>(rec + 8192 + slot * 8 + (lane >> 3) * 2) = dk;
                }
                const __half dv = quantise(kv[k][1], q);
#pragma unroll
                for (int i = 0; i < 4; ++i) vq[vq_at(4 * lane + i) + t - base] = static_cast<uint8_t>(q >> (8 * i));
                if ((lane & 7) == 0) vs[(lane >> 3) * 32 + t - base] = dv;
            } else if (in) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    uint16_t* dst = reinterpret_cast<uint16_t*>(rec) + (i * p.page_tokens + slot) * D + lane * E;
                    alignas(16) uint16_t w[E];
#pragma unroll
                    for (int e = 0; e < E; ++e) w[e] = to_16<FMT>(kv[k][i][e]);
                    if constexpr (E == 2) *reinterpret_cast<uint32_t*>(dst) = *reinterpret_cast<uint32_t*>(w);
                    else if constexpr (E == 4) *reinterpret_cast<uint2*>(dst) = *reinterpret_cast<uint2*>(w);
                    else *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<uint4*>(w);
                }
            }
        }
    }
    if (tid < hi - lo && (p.weight || p.pos)) {  // the slots' arrays, side by side
        const int t = lo + tid, pg = p.table[static_cast<int64_t>(a) * p.max_pages + t / p.page_tokens];
        if (pg >= 0 && pg < p.pool_pages) {
            const int64_t at = (static_cast<int64_t>(a) * p.kv_heads + g) * p.cap + t;
            if (p.weight) p.weight[at] = 0.f;
            if (p.pos && p.row_pos) p.pos[at] = p.row_pos[row0 + t];
        }
    }
    if constexpr (q8) {
        __syncthreads();
        const int pg = p.table[static_cast<int64_t>(a) * p.max_pages + base / 64];  // one page holds the group
        if (pg < 0 || pg >= p.pool_pages) return;
        uint8_t* rec = p.pool + (static_cast<int64_t>(pg) * p.kv_heads + g) * p.rec_bytes;
        const int at = base % 64;
        if (hi - lo == 32) {
            const int d = tid >> 1, part = tid & 1;
            const uint32_t* w = reinterpret_cast<const uint32_t*>(vq + vq_at(d) + 16 * part);
            *reinterpret_cast<uint4*>(rec + 8704 + d * 64 + at + 16 * part) = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
            const int first = lo - base, last = hi - base;
            for (int i = tid; i < 128 * 8; i += kAppendThreads) {  // four slots of a dim
                const int d = i >> 3, t0 = 4 * (i & 7);
                uint8_t* to = rec + 8704 + d * 64 + at + t0;
                const uint8_t* from = vq + vq_at(d) + t0;
                if (t0 >= first && t0 + 4 <= last) {
                    *reinterpret_cast<uint32_t*>(to) = *reinterpret_cast<const uint32_t*>(from);
                } else {
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        if (t0 + t >= first && t0 + t < last) to[t] = from[t];
                }
            }
        }
        for (int i = tid; i < 4 * (hi - lo); i += kAppendThreads) {
            const int b = i & 3, t = lo - base + (i >> 2);
            *reinterpret_cast<__half*>(rec + 16896 + (b * 64 + at + t) * 2) = vs[b * 32 + t];
        }
    }
}

template <int FMT, int D>
cudaError_t launch_append(const AppendParams& p, int32_t type, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(p.rows / 32 + 2 * (p.agents < p.rows ? p.agents : p.rows)),
                    static_cast<unsigned>(p.kv_heads));
    if (type == QMM_TYPE_F32) kv_append_kernel<FMT, D, float><<<grid, kAppendThreads, 0, s>>>(p);
    else if (type == QMM_TYPE_F16) kv_append_kernel<FMT, D, __half><<<grid, kAppendThreads, 0, s>>>(p);
    else kv_append_kernel<FMT, D, __nv_bfloat16><<<grid, kAppendThreads, 0, s>>>(p);
    return cudaGetLastError();
}

template <int FMT>
cudaError_t launch_append_dim(const AppendParams& p, int32_t dim, int32_t type, cudaStream_t s) {
    return dim == 64 ? launch_append<FMT, 64>(p, type, s) : dim == 128 ? launch_append<FMT, 128>(p, type, s) : launch_append<FMT, 256>(p, type, s);
}

// ------------------------------------------------------------------------------ evict
// Two kernels.  The first has a block, or a cluster of blocks with an even share of the slots
// each, per (sequence, KV head).  The keep-th largest
// key is found by a radix select from the top, 13 bits a pass (11 in clusters): count the digit of the keys that
// still match, add the blocks' counts through distributed shared memory, pick a digit; once at
// most kFew keys match they are ranked by counting.  Then each warp walks its run
// of slots: ties at the threshold are kept from the lowest slot on, kept slots below the budget
// stay, and the freed ones and the kept ones past the budget go to two lists in slot order
// (places by prefix sums over the warps).  The second kernel, a whole grid, moves the i-th of
// the one list to the i-th of the other.  The weights and positions are read once (keys stay in
// shared memory while they fit), and each moved token is read and written once; with the order
// of slots given up, nothing else has to move.
// What bounds it: 4 x 23,003 fp16 tokens cut to 11,500 take 58 us, 34 of them the moves (188 MB, 5.5
// TB/s) and the rest the select's chain of barriers on few SMs.  A q8_0 record keeps V
// dim-major, so moving half of a page's tokens touches all of its sectors: the destinations are
// read and written whole, and 8 ragged caches (60 MB of moved tokens, 218 MB of sectors) take 37 us.
constexpr int kEvictThreads = 1024;
constexpr int kMoveThreads = 256;
// Bits of a pass: 13 take fewer passes and collide less than 11, but in a cluster every block reads
// every block's counts (8 x 32 KB took 20 us of 131,071 keys in eight blocks).
template <bool multi>
constexpr int kDigit = multi ? 11 : 13;
constexpr int kBins = 1 << 13;
constexpr int kKeyCap = 24576;  // keys a block holds in shared memory
constexpr int kFew = 256;       // keys that are ranked by counting
constexpr int kSelectStatic = 4096;  // more than the selecting kernel's static shared memory

struct EvictParams {
    uint8_t* pool;
    const int32_t* table;
    const int32_t* cache_len;
    const int32_t* keep;
    const int32_t* protect_from;
    const float* weight;
    const int32_t* pos;
    float* weight_out;
    int32_t* pos_out;
    int32_t* len_out;
    int32_t* moved;  // [sequence][KV head]
    int2* lists;     // [sequence][KV head][2][half]: freed slots, and those that move into them: slot
                     // number, and page * page_tokens + place in the page (-1: a page outside the pool)
    int* err;
    int64_t rec_bytes, half;
    int32_t sink, kv_heads, max_pages, pool_pages, page_tokens, page_shift, cap, head_dim, key_cap;
    int32_t vec;     // weight, pos and their outputs are 16-byte aligned
    int32_t slices;  // blocks of the second kernel per (sequence, KV head)
};

// Keys in the order of eviction's preference: protected tokens above every weight, then the
// weights (-0 as +0), NaN below every other.
__device__ __forceinline__ uint32_t evict_key(float w, int32_t pos, int32_t sink, int32_t from) {
    if (pos < sink || pos >= from) return 0xFFFFFFFFu;
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <bool multi>
__global__ void __launch_bounds__(kEvictThreads) kv_evict_select(const EvictParams p) {
    extern __shared__ __align__(16) int hist[];  // [kBins], then the keys, [key_cap]
    uint32_t* keys = reinterpret_cast<uint32_t*>(hist + kBins);
    __shared__ uint32_t few[kFew];
    __shared__ __align__(16) uint32_t all_few[kFew];
    __shared__ int tmp[33], pick[3], counts[3], n_few;
    __shared__ int4 warp_counts[kEvictThreads / 32];
    griddep_launch_dependents();  // the moving kernel waits for this grid's end
    cg::cluster_group cl = cg::this_cluster();
    const int ranks = cl.num_blocks(), rank = cl.block_rank();
    const int ag = blockIdx.x / ranks, a = ag / p.kv_heads, g = ag % p.kv_heads;
    const int tid = threadIdx.x;
    const int len = p.cache_len[a], want = p.keep[a];
    const bool ok = len >= 0 && len <= p.cap;
    const int n = ok ? len : 0, budget = want >= 0 && want < n ? want : n;
    if (rank == 0 && tid == 0) {
        p.moved[ag] = 0;
        if (g == 0) {
            p.len_out[a] = ok ? budget : len;
            if (!ok) atomicOr(p.err, kErrRange);
        }
    }
    const int64_t base = static_cast<int64_t>(ag) * p.cap;
    const int per = ((n + ranks - 1) / ranks + 31) / 32 * 32, s0 = min(n, rank * per), s1 = min(n, s0 + per);
    if (budget == n) {  // nothing to evict (the whole cluster agrees)
        for (int t = s0 + tid; t < s1; t += kEvictThreads) {
            p.weight_out[base + t] = p.weight[base + t];
            p.pos_out[base + t] = p.pos[base + t];
        }
        return;
    }
    if (budget == 0) return;  // everything goes
    const int from = p.protect_from ? p.protect_from[a] : INT32_MAX;
    const bool cached = per <= p.key_cap;
    auto make = [&](int t) { return evict_key(p.weight[base + t], p.pos[base + t], p.sink, from); };
    auto key = [&](int t) { return cached ? keys[t - s0] : make(t); };
    // The arrays' slots below the budget go out as they are; the second kernel overwrites the freed
    // ones.  (In place, nothing is written.)
    const bool copy = p.weight_out != p.weight || p.pos_out != p.pos;
    auto put = [&](int t, float w, int32_t q) {
        if (t >= budget) return;
        p.weight_out[base + t] = w;
        p.pos_out[base + t] = q;
    };
    if (cached) {
        int t = s0 + 4 * tid;
        if (p.vec)  // four slots by 16-byte loads, four such in flight
            for (; t + 12 * kEvictThreads + 3 < s1; t += 16 * kEvictThreads) {
                float4 w[4];
                int4 q[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[i] = *reinterpret_cast<const float4*>(p.weight + base + t + 4 * i * kEvictThreads);
                    q[i] = *reinterpret_cast<const int4*>(p.pos + base + t + 4 * i * kEvictThreads);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int at = t + 4 * i * kEvictThreads;
                    if (copy && at + 3 < budget) {
                        *reinterpret_cast<float4*>(p.weight_out + base + at) = w[i];
                        *reinterpret_cast<int4*>(p.pos_out + base + at) = q[i];
                    } else if (copy) {
                        put(at, w[i].x, q[i].x), put(at + 1, w[i].y, q[i].y), put(at + 2, w[i].z, q[i].z);
                    }
                    *reinterpret_cast<uint4*>(keys + t - s0 + 4 * i * kEvictThreads) =
                        make_uint4(evict_key(w[i].x, q[i].x, p.sink, from), evict_key(w[i].y, q[i].y, p.sink, from),
                                   evict_key(w[i].z, q[i].z, p.sink, from), evict_key(w[i].w, q[i].w, p.sink, from));
                }
            }
        for (; t < s1; t += 4 * kEvictThreads) {
            float w[4];
            int q[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                w[i] = t + i < s1 ? p.weight[base + t + i] : 0.f;
                q[i] = t + i < s1 ? p.pos[base + t + i] : 0;
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (t + i < s1) {
                    if (copy) put(t + i, w[i], q[i]);
                    keys[t - s0 + i] = evict_key(w[i], q[i], p.sink, from);
                }
        }
    } else if (copy) {
        for (int t = s0 + tid; t < min(s1, budget); t += kEvictThreads) put(t, p.weight[base + t], p.pos[base + t]);
    }

    // ---- the threshold: the key of which `need` are kept, everything above it being kept too
    uint32_t thr = 0, mask = 0;
    int need = budget, match = n, shift = 32;
#pragma unroll 1
    while (match > kFew && shift > 0) {
        const int bits = shift > kDigit<multi> ? kDigit<multi> : shift, bins = 1 << bits;
        shift -= bits;
        for (int i = tid; i < 1 << kDigit<multi>; i += kEvictThreads) hist[i] = 0;
        __syncthreads();
#pragma unroll 4
        for (int t = s0 + tid; t < s1; t += kEvictThreads) {
            const uint32_t k = key(t);
            // (protected keys are many and equal: one addition per warp)
            const uint32_t top = __ballot_sync(__activemask(), k == 0xFFFFFFFFu);
            if (k == 0xFFFFFFFFu) {
                if (mask == thr && (tid & 31) == __ffs(top) - 1) atomicAdd(&hist[bins - 1], __popc(top));
            } else if ((k & mask) == thr) {
                atomicAdd(&hist[(k >> shift) & (bins - 1)], 1);
            }
        }
        cl.sync();
        // the thread's bins, from the highest down
        constexpr int B = (1 << kDigit<multi>) / kEvictThreads;
        const int first = (1 << kDigit<multi>) - B - B * tid;
        int c[B] = {}, mine = 0;
        for (int r = 0; r < ranks; ++r) {
            const int2* v = reinterpret_cast<const int2*>(cl.map_shared_rank(hist, r) + first);
#pragma unroll
            for (int i = 0; i < B / 2; ++i) {
                const int2 x = v[B / 2 - 1 - i];
                c[2 * i] += x.y, c[2 * i + 1] += x.x;
            }
        }
#pragma unroll
        for (int i = 0; i < B; ++i) mine += c[i];
        int total;
        int above = block_exclusive(mine, tmp, &total);
        if (above < need && above + mine >= need) {  // one thread of the block's
#pragma unroll
            for (int i = 0; i < B; ++i) {
                if (above < need && above + c[i] >= need) {
                    pick[0] = first + B - 1 - i;
                    pick[1] = need - above;
                    pick[2] = c[i];
                }
                above += c[i];
            }
        }
        cl.sync();  // (also: every block has read the counts before they are cleared)
        thr |= static_cast<uint32_t>(pick[0]) << shift;
        mask |= static_cast<uint32_t>(bins - 1) << shift;
        need = pick[1];
        match = pick[2];
    }
    if (shift > 0) {
        // few keys match: every block ranks all of them
        if (tid == 0) n_few = 0;
        __syncthreads();
        for (int t = s0 + tid; t < s1; t += kEvictThreads) {
            const uint32_t k = key(t);
            if ((k & mask) == thr) few[atomicAdd(&n_few, 1)] = k;
        }
        cl.sync();
        for (int r = 0, at = 0; r < ranks; ++r) {
            const int c = *cl.map_shared_rank(&n_few, r);
            const uint32_t* from_few = cl.map_shared_rank(few, r);
            for (int i = tid; i < c; i += kEvictThreads) all_few[at + i] = from_few[i];
            at += c;
        }
        __syncthreads();
        if (tid < match) {
            const uint32_t mine = all_few[tid];
            int above = 0, same = 0, i = 0;
#pragma unroll 4
            for (; i + 4 <= match; i += 4) {
                const uint4 o = *reinterpret_cast<const uint4*>(all_few + i);
                above += (o.x > mine) + (o.y > mine) + (o.z > mine) + (o.w > mine);
                same += (o.x == mine) + (o.y == mine) + (o.z == mine) + (o.w == mine);
            }
            for (; i < match; ++i) {
                above += all_few[i] > mine;
                same += all_few[i] == mine;
            }
            if (above < need && above + same >= need) {  // (equal keys write equal values)
                pick[0] = static_cast<int>(mine);
                pick[1] = need - above;
            }
        }
        cl.sync();
        thr = static_cast<uint32_t>(pick[0]);
        need = pick[1];
    }

    // ---- the warp's run of slots, counted: above and at the threshold, below and past the budget
    const int warp = tid >> 5, lane = tid & 31;
    const int run = (per / 32 + kEvictThreads / 32 - 1) / (kEvictThreads / 32) * 32;
    const int t0 = min(s1, s0 + warp * run), t1 = min(s1, t0 + run);
    int4 n4 = make_int4(0, 0, 0, 0);
#pragma unroll 4
    for (int t = t0 + lane; t < t1; t += 32) {
        const uint32_t k = key(t);
        if (t < budget) n4.x += k > thr, n4.y += k == thr;
        else n4.z += k > thr, n4.w += k == thr;
    }
    n4.x = __reduce_add_sync(0xffffffffu, n4.x), n4.y = __reduce_add_sync(0xffffffffu, n4.y);
    n4.z = __reduce_add_sync(0xffffffffu, n4.z), n4.w = __reduce_add_sync(0xffffffffu, n4.w);
    if (lane == 0) warp_counts[warp] = n4;
    __syncthreads();
    // ties before the warp's run: those of the block's earlier warps, and of earlier blocks
    const int4 w4 = warp_counts[lane];
    const int block_ties = __reduce_add_sync(0xffffffffu, w4.y + w4.w);
    if (tid == 0) counts[0] = block_ties;
    cl.sync();
    int tie_block = 0;
    for (int r = 0; r < rank; ++r) tie_block += cl.map_shared_rank(counts, r)[0];
    // (lane l: what warp l keeps on either side of the budget)
    int tie_lane = w4.y + w4.w;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, tie_lane, k);
        if (lane >= k) tie_lane += o;
    }
    tie_lane += tie_block - w4.y - w4.w;
    const int a0 = min(s1, s0 + lane * run), a1 = min(s1, a0 + run);  // warp l's run
    const int below = max(0, min(a1, budget) - a0);
    const int kept_below = w4.x + min(w4.y, max(0, need - tie_lane));
    const int kept_past = w4.z + min(w4.w, max(0, need - tie_lane - w4.y));
    int hole_lane = below - kept_below, move_lane = kept_past;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, hole_lane, k), q = __shfl_up_sync(0xffffffffu, move_lane, k);
        if (lane >= k) hole_lane += o, move_lane += q;
    }
    if (tid == 31) {
        counts[1] = hole_lane;
        counts[2] = move_lane;
    }
    int tie = __shfl_sync(0xffffffffu, tie_lane, warp);
    int hole = __shfl_sync(0xffffffffu, hole_lane - (below - kept_below), warp);
    int move = __shfl_sync(0xffffffffu, move_lane - kept_past, warp);
    cl.sync();
    int total = 0;
    for (int r = 0; r < ranks; ++r) {
        const int* c = cl.map_shared_rank(counts, r);
        if (r < rank) {
            hole += c[1];
            move += c[2];
        }
        total += c[2];
    }
    if (rank == 0 && tid == 0) p.moved[ag] = total;

    // ---- the lists
    int2* to = p.lists + static_cast<int64_t>(ag) * 2 * p.half;
    int2* src = to + p.half;
    const int32_t* table = p.table + static_cast<int64_t>(a) * p.max_pages;
    const uint32_t before = (1u << lane) - 1;
    // the pages of the warp's run, a lane each, if they are at most 32
    const int page0 = t0 >> p.page_shift;
    const bool held = ((t1 - 1) >> p.page_shift) - page0 < 32;
    int pages = -1;
    if (held && ((page0 + lane) << p.page_shift) < t1) pages = table[page0 + lane];
#pragma unroll 4
    for (int t = t0 + lane; t - lane < t1; t += 32) {
        const bool in = t < t1;
        const uint32_t k = in ? key(t) : 0u;
        const uint32_t equal = __ballot_sync(0xffffffffu, in && k == thr);
        const bool kept = in && (k > thr || (k == thr && tie + __popc(equal & before) < need));
        const bool free = in && !kept && t < budget, late = kept && t >= budget;
        const uint32_t frees = __ballot_sync(0xffffffffu, free), lates = __ballot_sync(0xffffffffu, late);
        int pg = __shfl_sync(0xffffffffu, pages, ((t >> p.page_shift) - page0) & 31);
        if (free || late) {
            if (!held) pg = table[t >> p.page_shift];
            int place = -1;
            if (pg >= 0 && pg < p.pool_pages) place = pg * p.page_tokens + (t & (p.page_tokens - 1));
            else atomicOr(p.err, kErrPage);
            if (free) to[hole + __popc(frees & before)] = make_int2(t, place);
            else src[move + __popc(lates & before)] = make_int2(t, place);
        }
        tie += __popc(equal);
        hole += __popc(frees);
        move += __popc(lates);
    }
    cl.sync();  // no block leaves while its counts are read
}

template <bool q8>
__global__ void __launch_bounds__(kMoveThreads) kv_evict_move(const EvictParams p) {
    const int ag = blockIdx.x / p.slices, g = ag % p.kv_heads, lane = threadIdx.x & 31;
    const int64_t base = static_cast<int64_t>(ag) * p.cap;
    const int2* to = p.lists + static_cast<int64_t>(ag) * 2 * p.half;
    const int2* from = to + p.half;
    const int first = (blockIdx.x % p.slices) * kMoveThreads + threadIdx.x, step = p.slices * kMoveThreads;
    griddep_wait();  // the lists are written
    const int moved = p.moved[ag];
    // source slots >= budget > destination slots: nothing read here is written here
    for (int i = first; i < moved; i += step) {
        const int2 src = from[i], dst = to[i];
        if (src.y < 0 || dst.y < 0) continue;  // (K and V stay: so do the slots' numbers)
        p.weight_out[base + dst.x] = p.weight[base + src.x];
        p.pos_out[base + dst.x] = p.pos[base + src.x];
    }
    if constexpr (q8) {
        // a warp moves 32 tokens, a lane each, one fifth at a time: K with the scales, or 32 dims of V.
        // Sources and destinations both rise with the lane, so V's strided bytes share their sectors.
        const int work = (moved + 31) / 32 * 5;
        for (int w = first >> 5; w < work; w += step >> 5) {
            const int i = w / 5 * 32 + lane, part = w % 5;
            const int src = i < moved ? from[i].y : -1, dst = i < moved ? to[i].y : -1;
            if (src < 0 || dst < 0) continue;
            const uint8_t* a = p.pool + (static_cast<int64_t>(src >> 6) * p.kv_heads + g) * kQ8Rec;
            uint8_t* b = p.pool + (static_cast<int64_t>(dst >> 6) * p.kv_heads + g) * kQ8Rec;
            const int ss = src & 63, ds = dst & 63;
            if (part == 4) {
                uint4 row[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) row[c] = *reinterpret_cast<const uint4*>(a + ss * 128 + 16 * (c ^ q8_key(ss)));
                const uint2 ks = *reinterpret_cast<const uint2*>(a + 8192 + ss * 8);
                uint16_t vs[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) vs[c] = *reinterpret_cast<const uint16_t*>(a + 16896 + (c * 64 + ss) * 2);
#pragma unroll
                for (int c = 0; c < 8; ++c) *reinterpret_cast<uint4*>(b + ds * 128 + 16 * (c ^ q8_key(ds))) = row[c];
                *reinterpret_cast<uint2*>(b + 8192 + ds * 8) = ks;
#pragma unroll
                for (int c = 0; c < 4; ++c) *reinterpret_cast<uint16_t*>(b + 16896 + (c * 64 + ds) * 2) = vs[c];
            } else {
                a += 8704 + 32 * part * 64 + ss;
                b += 8704 + 32 * part * 64 + ds;
                uint8_t v[32];
#pragma unroll
                for (int k = 0; k < 32; ++k) v[k] = a[k * 64];
#pragma unroll
                for (int k = 0; k < 32; ++k) b[k * 64] = v[k];
            }
        }
    } else {
        // 16-byte pieces of the tokens' K and V rows, consecutive pieces by consecutive threads, four
        // of a thread's in flight
        const int row = p.head_dim * 2, shift = p.head_dim == 64 ? 4 : p.head_dim == 128 ? 5 : 6;
        const int64_t work = static_cast<int64_t>(moved) << shift;
        const int c = first & ((1 << shift) - 1), half = c >> (shift - 1), off = (c & ((1 << (shift - 1)) - 1)) * 16;
        auto address = [&](int t) {
            const int64_t pg = t >> p.page_shift;
            return p.pool + (pg * p.kv_heads + g) * p.rec_bytes + (half * p.page_tokens + (t & (p.page_tokens - 1))) * row + off;
        };
        // (step is a multiple of the pieces per token: a thread's pieces are the same part of each)
        for (int64_t i0 = first; i0 < work; i0 += 4 * static_cast<int64_t>(step)) {
            int src[4], dst[4];
            uint4 v[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int64_t i = i0 + k * static_cast<int64_t>(step);
                src[k] = i < work ? from[i >> shift].y : -1;
                dst[k] = i < work ? to[i >> shift].y : -1;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (src[k] >= 0) v[k] = __ldcs(reinterpret_cast<const uint4*>(address(src[k])));
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (src[k] >= 0 && dst[k] >= 0) *reinterpret_cast<uint4*>(address(dst[k])) = v[k];
        }
    }
}

namespace {

int64_t list_half(const qmm_kv_dims& d) { return int64_t{d.max_pages} * d.page_tokens / 2 + 1; }

}  // namespace
}  // namespace kv
}  // namespace qmm

extern "C" {

qmm_status qmm_kv_append(const qmm_kv_dims* dims, void* pool, const int32_t* page_table,
                         const int32_t* agent_rows, const int32_t* cache_len, const void* k, int64_t k_stride,
                         const void* v, int64_t v_stride, int32_t type, int64_t rows, float* weight, int32_t* pos,
                         const int32_t* row_pos, int* err_word, void* stream) {
    using namespace qmm::kv;
    qmm_status st = check_dims(dims);
    if (st != QMM_OK) return st;
    if (rows < 0 || type < QMM_TYPE_F32 || type > QMM_TYPE_BF16) return QMM_ERR_INVALID_ARG;
    if (rows == 0) return QMM_OK;
    const int64_t width = int64_t{dims->kv_heads} * dims->head_dim;
    if (!pool || !page_table || !agent_rows || !cache_len || !k || !v || !err_word || k_stride < width || v_stride < width)
        return QMM_ERR_INVALID_ARG;
    if (rows > (1 << 24)) return QMM_ERR_UNSUPPORTED_SHAPE;
    const int size = type == QMM_TYPE_F32 ? 4 : 2;
    if (!aligned(pool, 16) || !aligned(page_table, 4) || !aligned(agent_rows, 4) || !aligned(cache_len, 4) || !aligned(k, size) ||
        !aligned(v, size) || !aligned(weight, 4) || !aligned(pos, 4) || !aligned(row_pos, 4) || !aligned(err_word, 4))
        return QMM_ERR_MISALIGNED;
    int dev = 0, sms = 0;
    st = check_gpu(&dev, &sms);
    if (st != QMM_OK) return st;
    AppendParams p = {};
    p.pool = static_cast<uint8_t*>(pool);
    p.table = page_table;
    p.agent_rows = agent_rows;
    p.cache_len = cache_len;
    p.src[0] = k;
    p.src[1] = v;
    p.stride[0] = k_stride;
    p.stride[1] = v_stride;
    p.weight = weight;
    p.pos = pos;
    p.row_pos = row_pos;
    p.err = err_word;
    p.rec_bytes = record_bytes(*dims);
    p.rows = static_cast<int32_t>(rows);
    p.agents = dims->agents;
    p.kv_heads = dims->kv_heads;
    p.max_pages = dims->max_pages;
    p.pool_pages = static_cast<int32_t>(dims->pool_pages);
    p.page_tokens = dims->page_tokens;
    p.cap = dims->max_pages * dims->page_tokens;
    p.vec = aligned(k, 16) && aligned(v, 16) && k_stride * size % 16 == 0 && v_stride * size % 16 == 0;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = dims->format == QMM_KV_Q8_0  ? launch_append<QMM_KV_Q8_0, 128>(p, type, s)
                          : dims->format == QMM_KV_F16 ? launch_append_dim<QMM_KV_F16>(p, dims->head_dim, type, s)
                                                       : launch_append_dim<QMM_KV_BF16>(p, dims->head_dim, type, s);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

qmm_status qmm_kv_evict_workspace_bytes(const qmm_kv_dims* dims, int64_t* bytes) {
    if (!bytes) return QMM_ERR_INVALID_ARG;
    const qmm_status st = qmm::kv::check_dims(dims);
    if (st != QMM_OK) return st;
    const int64_t groups = int64_t{dims->agents} * dims->kv_heads;
    *bytes = (groups * 4 + 15) / 16 * 16 + groups * 2 * qmm::kv::list_half(*dims) * 8;
    return QMM_OK;
}

qmm_status qmm_kv_evict(const qmm_kv_dims* dims, void* pool, const int32_t* page_table, const int32_t* cache_len,
                        const int32_t* keep, int32_t sink, const int32_t* protect_from, const float* weight,
                        const int32_t* pos, float* weight_out, int32_t* pos_out, int32_t* len_out, void* workspace,
                        int64_t workspace_bytes, int* err_word, void* stream) {
    using namespace qmm::kv;
    int64_t need = 0;
    qmm_status st = qmm_kv_evict_workspace_bytes(dims, &need);
    if (st != QMM_OK) return st;
    if (!pool || !page_table || !cache_len || !keep || !weight || !pos || !weight_out || !pos_out || !len_out ||
        len_out == cache_len || !workspace || !err_word)
        return QMM_ERR_INVALID_ARG;
    if (!aligned(pool, 16) || !aligned(workspace, 16) || !aligned(page_table, 4) || !aligned(cache_len, 4) || !aligned(keep, 4) ||
        !aligned(protect_from, 4) || !aligned(weight, 4) || !aligned(pos, 4) || !aligned(weight_out, 4) || !aligned(pos_out, 4) ||
        !aligned(len_out, 4) || !aligned(err_word, 4))
        return QMM_ERR_MISALIGNED;
    if (workspace_bytes < need) return QMM_ERR_SCRATCH_TOO_SMALL;
    int dev = 0, sms = 0;
    st = check_gpu(&dev, &sms);
    if (st != QMM_OK) return st;
    EvictParams p = {};
    p.pool = static_cast<uint8_t*>(pool);
    p.table = page_table;
    p.cache_len = cache_len;
    p.keep = keep;
    p.protect_from = protect_from;
    p.weight = weight;
    p.pos = pos;
    p.weight_out = weight_out;
    p.pos_out = pos_out;
    p.len_out = len_out;
    const int64_t groups = int64_t{dims->agents} * dims->kv_heads;
    p.moved = static_cast<int32_t*>(workspace);
    p.lists = reinterpret_cast<int2*>(static_cast<uint8_t*>(workspace) + (groups * 4 + 15) / 16 * 16);
    p.err = err_word;
    p.rec_bytes = record_bytes(*dims);
    p.half = list_half(*dims);
    p.sink = sink;
    p.kv_heads = dims->kv_heads;
    p.max_pages = dims->max_pages;
    p.pool_pages = static_cast<int32_t>(dims->pool_pages);
    p.page_tokens = dims->page_tokens;
    p.cap = dims->max_pages * dims->page_tokens;
    p.head_dim = dims->head_dim;
    while ((1 << p.page_shift) < dims->page_tokens) ++p.page_shift;
    // blocks per cluster, up to 8 (the portable limit): as many as the longest sequence's keys need,
    // and up to one per 8,192 slots while every block has an SM to itself (4 x 8 groups of 23,040
    // slots: 66 us with one block each, 58 with four; with eight, which take two waves, 96)
    int ranks = 1;
    while (ranks < 8 && (p.cap > ranks * kKeyCap || (p.cap > ranks * 8192 && groups * ranks * 2 <= sms))) ranks *= 2;
    const int64_t per = ((p.cap + ranks - 1) / ranks + 31) / 32 * 32;
    p.vec = aligned(weight, 16) && aligned(pos, 16) && aligned(weight_out, 16) && aligned(pos_out, 16);
    p.key_cap = static_cast<int32_t>(per < kKeyCap ? per : kKeyCap);
    // the moves: eight blocks per SM over all groups, no more than the most pieces a group can move
    const int64_t pieces = dims->format == QMM_KV_Q8_0 ? (p.half + 31) / 32 * 5 * 32 : p.half * dims->head_dim / 4;
    int64_t slices = (int64_t{sms} * 8 + groups - 1) / groups;
    if (slices > (pieces + kMoveThreads - 1) / kMoveThreads) slices = (pieces + kMoveThreads - 1) / kMoveThreads;
    p.slices = static_cast<int32_t>(slices);
    if (groups * ranks > INT32_MAX || groups * slices > INT32_MAX || dims->pool_pages * dims->page_tokens > INT32_MAX)
        return QMM_ERR_UNSUPPORTED_SHAPE;
    const auto select = ranks > 1 ? kv_evict_select<true> : kv_evict_select<false>;
    static_assert((kBins + kKeyCap) * 4 <= kMaxShared - kSelectStatic);
    static Once once[2];
    cudaError_t e = once[ranks > 1].allow_shared(select, dev, kSelectStatic);
    if (e == cudaSuccess) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(groups * ranks));
        cfg.blockDim = dim3(kEvictThreads);
        cfg.dynamicSmemBytes = static_cast<size_t>(kBins + p.key_cap) * 4;
        cfg.stream = static_cast<cudaStream_t>(stream);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = static_cast<unsigned>(ranks);
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        e = cudaLaunchKernelEx(&cfg, select, p);
        if (e == cudaSuccess) {
            cfg.gridDim = dim3(static_cast<unsigned>(groups * slices));
            cfg.blockDim = dim3(kMoveThreads);
            cfg.dynamicSmemBytes = 0;
            attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
            attr[0].val.programmaticStreamSerializationAllowed = 1;
            e = dims->format == QMM_KV_Q8_0 ? cudaLaunchKernelEx(&cfg, kv_evict_move<true>, p) : cudaLaunchKernelEx(&cfg, kv_evict_move<false>, p);
        }
    }
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

}  // extern "C"
