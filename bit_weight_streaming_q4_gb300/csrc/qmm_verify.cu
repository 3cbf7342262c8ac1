// Verification of drafted tokens against the target's probabilities.
//
// Which drafts are taken, and which token a uniform number picks out of 151,936, must not depend on the
// rounding or the order of a sum.  So a column's weight 2^((x - M) log2(e) / T) is formed as a whole number of
// 2^-44 (weight() below: pairs of fp32, good to 2^-38), and weights are added as 64-bit integers.
//  1. verify_stats: a block per segment of kSeg columns of a target or draft row: its largest
//     logit M_s (with the lowest column), and Z_s = sum of the weights relative to M_s.
//  2. verify_choose: a cluster per sequence.  Every block joins the segments of the sequence's rows
//     (Z = sum Z_s 2^(M_s - M), in integers), judges the drafts, u W_q(x) Z_p < W_p(x) Z_q, and so knows the row to draw
//     from; it reads its share of that row (and of the draft's) again, now from L2, and adds up what is left of p;
//     the blocks exchange their sums, and the one in whose share the number falls looks for the column.
// What bounds it: the logits' bytes in the first kernel, latencies in the second.
#include <cooperative_groups.h>

#include "qmm_decode.h"
#include "qmm_kv.cuh"

namespace cg = cooperative_groups;

namespace qmm {
namespace verify {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPer = 32;                 // columns per thread and segment
constexpr int kSeg = kThreads * kPer;
constexpr int kSteps = kPer / 4;         // a thread's columns are kSteps runs of 4
constexpr int kChoose = 512;             // threads of the second kernel ..
constexpr int kChooseWarps = kChoose / 32;
constexpr int kMaxRanks = 16;            // .. and blocks per sequence
constexpr int kStep = 4 * kChoose;       // columns that one of its blocks takes at a time
constexpr int kSpan = 4;                 // steps whose loads are on their way at once
constexpr int kKept = 32;                // rows of a sequence whose joined numbers are kept for the choice
constexpr int kMaxColumns = 1 << 19;
constexpr int kMaxSegs = kMaxColumns / kSeg;
constexpr int kMaxSteps = kMaxColumns / kStep / 8 + 1;  // of a block (8 blocks a sequence at least)
constexpr int kShift = 44;               // weights count 2^-44

struct alignas(16) Stat {
    uint64_t z;    // sum of the segment's weights relative to m
    float m;       // largest logit, -infinity if there is no other
    int32_t best;  // its lowest column, -1: a NaN or +infinity is among the logits
};

struct Params {
    const void* logits;
    const void* draft;
    const int32_t* agent_rows;
    const int32_t* tokens;
    const float* temperature;
    const float* accept_u;
    const float* sample_u;
    int32_t* accepted;
    int32_t* token;
    float* prob;
    Stat* stats;  // [2][rows][segs]: target rows, draft rows
    int* err;
    int64_t stride, draft_stride;
    int32_t rows, n, segs, agents;
    int32_t vec, draft_vec;  // rows can be read four columns at a time
    int32_t ranks;           // blocks per sequence of the second kernel, 8 or 16
};

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// A pair of fp32 numbers, value hi + lo.
struct Two {
    float hi, lo;
};
__device__ __forceinline__ Two two_of(double v) {
    const float hi = static_cast<float>(v);
    return {hi, static_cast<float>(v - hi)};
}

// log2(e) / T; 0 (no scale) where the sequence is greedy.
__device__ __forceinline__ Two scale_of(const Params& p, int a) {
    const float t = p.temperature ? p.temperature[a] : 1.f;
    if (!(t >= 7.888609e-31f)) return {0.f, 0.f};  // 2^-100
    return two_of(1.4426950408889634074 / static_cast<double>(fminf(t, 1.2676506e30f)));
}

// 2^(i / 64) for i = 0 .. 63, as 2^44ths and as a pair.
struct Table {
    uint64_t fix[64];
    Two two[64];
};
__device__ __forceinline__ void fill(Table& t) {
    if (threadIdx.x < 64) {
        const double v = exp2(threadIdx.x / 64.0);
        t.fix[threadIdx.x] = static_cast<uint64_t>(__double2ll_rn(v * 17592186044416.0));
        t.two[threadIdx.x] = two_of(v);
    }
}

__device__ __forceinline__ int whole(float v) { return __float_as_int(v + 12582912.f) - 0x4B400000; }  // nearest, |v| < 2^22

// 2^((x - m) scale) = w 2^(-44 - k), x <= m, m finite; false where it is below 2^least.  The exponent is a pair: x - m
// without error, times the scale's pair; its 64ths come from the table and 2^r of what is left, |r| <= 2^-7, from its
// series: r ln 2 as a pair, the terms from the square on in fp32 (together at most 2^-16: their roundings are below 2^-38).
__device__ __forceinline__ bool power(float x, float m, Two scale, const Table& t, float least, int64_t& w, int& k) {
    const float s = x - m, b = s - x;
    const float e = (x - (s - b)) - (m + b);
    const float ph = s * scale.hi;
    if (!(ph >= least)) return false;  // (and x = -infinity)
    const float pl = fmaf(s, scale.hi, -ph) + fmaf(s, scale.lo, e * scale.hi);
    const int n = whole(ph * 64.f);
    // (what is left is 0 or a step of ph at least, and pl half a step at most: the sum of the two is exact as a pair)
    const float rest = fmaf(static_cast<float>(n), -0.015625f, ph), rh = rest + pl, rl = pl - (rh - rest);
    constexpr float kHi = 0.693147182464599609375f, kLo = -1.9046542999577680e-9f;  // ln 2
    const float uh = rh * kHi, ul = fmaf(rh, kHi, -uh) + fmaf(rh, kLo, rl * kHi);
    const float q = uh * uh * fmaf(uh, fmaf(uh, fmaf(uh, 1.f / 120, 1.f / 24), 1.f / 6), 0.5f);
    const float vh = uh + q, vl = ul + (q - (vh - uh));  // (|q| < |uh|)
    const Two f = t.two[n & 63];
    const float wh = f.hi * vh, wl = fmaf(f.hi, vh, -wh) + fmaf(f.hi, vl, f.lo * vh);
    const int h = whole(wh * 16777216.f);  // 2^24ths
    const int l = whole((fmaf(static_cast<float>(h), -5.9604644775390625e-8f, wh) + wl) * 17592186044416.f);
    w = static_cast<int64_t>(t.fix[n & 63]) + (static_cast<int64_t>(h) << (kShift - 24)) + l;
    k = -(n >> 6);
    return true;
}
// The same in 2^-44ths, nearest.
__device__ __forceinline__ uint64_t weight(float x, float m, Two scale, const Table& t) {
    int64_t w;
    int k;  // 0 .. 46
    if (!power(x, m, scale, t, -46.f, w, k)) return 0;
    return k > 0 ? (static_cast<uint64_t>(w) + (uint64_t{1} << (k - 1))) >> k : static_cast<uint64_t>(w);
}
// The same with all its bits, for one column.
__device__ __forceinline__ double weight_of(float x, float m, Two scale, const Table& t) {
    int64_t w;
    int k;
    if (!power(x, m, scale, t, -1000.f, w, k)) return 0.0;
    return static_cast<double>(w) * __hiloint2double((1023 - k) << 20, 0);
}

// z w / 2^44, z <= 2^57, w <= 2^44 (or both up to 2^57 and 2^49)
__device__ __forceinline__ uint64_t scaled(uint64_t z, uint64_t w) { return __umul64hi(z << 6, w << 14); }

// Run i of the thread's columns: four from segment column (i * kThreads + tid) * 4.  Columns past the row's end give -infinity.
template <typename T>
__device__ __forceinline__ void load4(const T* row, bool vec, int col, int n, float (&x)[4]) {
    if (vec && col + 4 <= n) {
        if constexpr (sizeof(T) == 4) {
            const float4 v = *reinterpret_cast<const float4*>(row + col);
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
            T v[4];
            *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(row + col);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = as_f32(v[j]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = col + j < n ? as_f32(row[col + j]) : -INFINITY;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 3) verify_stats(const Params p) {
    __shared__ Table table;
    __shared__ Two scale_sm;
    __shared__ float max_sm[kWarps];
    __shared__ int best_sm[kWarps];
    __shared__ uint64_t sum_sm[kWarps];
    __shared__ int first_sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_launch_dependents();
    const int seg = blockIdx.x, row = blockIdx.y;
    const bool draft = blockIdx.z == 1;
    const T* base = draft ? static_cast<const T*>(p.draft) + row * p.draft_stride : static_cast<const T*>(p.logits) + row * p.stride;
    const bool vec = draft ? p.draft_vec : p.vec;
    float x[kSteps][4];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) load4<T>(base, vec, seg * kSeg + (i * kThreads + tid) * 4, p.n, x[i]);
    if (tid == 0) first_sm = 1;
    __syncthreads();
    // the row's sequence (where agent_rows falls there may be several: nobody asks for what comes of it)
    for (int a = tid; a < p.agents; a += kThreads) {
        const int r0 = p.agent_rows[a];
        if (r0 <= row && row < p.agent_rows[a + 1] && !(draft && r0 == row)) {
            scale_sm = scale_of(p, a);
            first_sm = 0;
        }
    }
    fill(table);
    // ---- the largest, its lowest column, and whether something is no number
    float m = -INFINITY;
    bool odd = false;
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            m = fmaxf(m, x[i][j]);
            odd |= !(x[i][j] < INFINITY);
        }
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    if (lane == 0) max_sm[warp] = m;
    odd = __syncthreads_or(odd);
    if (first_sm) return;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, max_sm[w]);
    const Two scale = scale_sm;
    int best = INT32_MAX;
    uint64_t sum = 0;
#pragma unroll
    for (int i = kSteps - 1; i >= 0; --i)
#pragma unroll
        for (int j = 3; j >= 0; --j)
            if (x[i][j] == m) best = seg * kSeg + (i * kThreads + tid) * 4 + j;
    if (scale.hi != 0.f && m > -INFINITY && !odd) {
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) sum += weight(x[i][j], m, scale, table);
    }
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) {
        best = min(best, __shfl_xor_sync(0xffffffffu, best, k));
        sum += __shfl_xor_sync(0xffffffffu, sum, k);
    }
    if (lane == 0) best_sm[warp] = best, sum_sm[warp] = sum;
    __syncthreads();
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < kWarps; ++w) best = min(best, best_sm[w]), sum += sum_sm[w];
        Stat st;
        st.z = sum;
        st.m = m;
        st.best = odd ? -1 : best;
        p.stats[(static_cast<int64_t>(draft) * p.rows + row) * p.segs + seg] = st;
    }
}

// A row's segments joined, by a warp: every lane returns it.
struct Joined {
    float m;       // largest logit
    int32_t best;  // its lowest column
    bool odd;      // no distribution: a NaN or +infinity
    uint64_t z;    // sum of the weights relative to m
};
__device__ __forceinline__ Joined join(const Params& p, bool draft, int row, Two scale, const Table& t) {
    const int lane = threadIdx.x & 31;
    const Stat* st = p.stats + (static_cast<int64_t>(draft) * p.rows + row) * p.segs;
    Joined r = {-INFINITY, INT32_MAX, false, 0};
    constexpr int kMost = kMaxSegs / 32;
    Stat v[kMost];
#pragma unroll
    for (int i = 0; i < kMost; ++i) {
        v[i] = {0, -INFINITY, INT32_MAX};
        if (lane + 32 * i < p.segs) v[i] = st[lane + 32 * i];
        r.odd |= v[i].best < 0;
        if (v[i].m > r.m || (v[i].m == r.m && v[i].best < r.best)) r.m = v[i].m, r.best = v[i].best;
    }
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) {
        const float m = __shfl_xor_sync(0xffffffffu, r.m, k);
        const int best = __shfl_xor_sync(0xffffffffu, r.best, k);
        if (m > r.m || (m == r.m && best < r.best)) r.m = m, r.best = best;
    }
    r.odd = __any_sync(0xffffffffu, r.odd);
    if (!r.odd && r.m > -INFINITY) {
#pragma unroll
        for (int i = 0; i < kMost; ++i)
            if (v[i].z) r.z += scaled(v[i].z, weight(v[i].m, r.m, scale, t));
    }
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) r.z += __shfl_xor_sync(0xffffffffu, r.z, k);
    return r;
}

enum { kPlain = 0, kLess = 1, kWithout = 2 };  // draw from p, from max(p - q, 0), from p without a column

struct Choice {
    int row;       // to draw from, of logits
    int how;
    int column;    // kWithout: the refused draft
    int taken;
    Joined p, q;   // of that row, and of the draft row behind it
};

template <typename T>
__global__ void __launch_bounds__(kChoose) verify_choose(const Params p) {
    __shared__ Table table;
    __shared__ Choice choice;
    __shared__ Joined kept[2][kKept];          // target rows, draft rows
    __shared__ int refused;                    // lowest refused draft
    __shared__ uint64_t share[kMaxRanks];      // the blocks' sums (each block's own copy)
    __shared__ uint64_t part[kMaxSteps * kChooseWarps];
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), ranks = p.ranks, a = blockIdx.x / ranks;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bool falls = false;
    for (int i = tid; i < p.agents; i += kChoose) falls |= p.agent_rows[i + 1] < p.agent_rows[i];
    fill(table);
    const int r0 = p.agent_rows[a], r1 = p.agent_rows[a + 1];
    const Two scale = scale_of(p, a);
    const float sample = p.sample_u[a];
    if (tid == 0) refused = INT32_MAX;
    falls = __syncthreads_or(falls);
    griddep_wait();  // the first kernel's numbers are there
    const bool bad = falls || r0 < 0 || r1 > p.rows;
    if (bad && tid == 0 && rank == 0) atomicOr(p.err, kv::kErrRange);
    if (bad || r1 <= r0) {
        if (tid == 0 && rank == 0) p.accepted[a] = 0, p.token[a] = -1;
        return;  // (the whole cluster)
    }
    const bool greedy = scale.hi == 0.f;
    const T* logits = static_cast<const T*>(p.logits);
    const T* drafts = static_cast<const T*>(p.draft);
    // ---- the drafts: a warp each
    for (int r = r0 + 1 + warp; r < r1; r += kChooseWarps) {
        const int x = p.tokens[r];
        const bool in = x >= 0 && x < p.n;
        // (what the joins do not need is asked for before them)
        const float xp = in ? as_f32(logits[(r - 1) * p.stride + x]) : 0.f, xq = in && drafts ? as_f32(drafts[r * p.draft_stride + x]) : 0.f;
        const float u = p.accept_u[r];
        const Joined tp = join(p, false, r - 1, scale, table);
        Joined tq = tp;
        if (drafts && !greedy) tq = join(p, true, r, scale, table);
        if (lane == 0 && r - r0 <= kKept) kept[0][r - r0 - 1] = tp, kept[1][r - r0 - 1] = tq;
        bool yes = false;
        float prob = 0.f;
        if (tp.odd) {
            prob = __int_as_float(0x7FFFFFFF);
        } else if (greedy) {
            yes = in && tp.m > -INFINITY && tp.best == x;
            prob = yes ? 1.f : 0.f;
        } else {
            double wq = 1, zq = 1;
            const bool none = drafts && (tq.odd || tq.m == -INFINITY);
            if (drafts && in && !none) {
                wq = weight_of(xq, tq.m, scale, table);
                zq = static_cast<double>(tq.z);
            }
            if (none) {
                prob = __int_as_float(0x7FFFFFFF);
            } else if (in && tp.m > -INFINITY) {
                const double wp = weight_of(xp, tp.m, scale, table), zp = static_cast<double>(tp.z);
                yes = static_cast<double>(u) * (wq * zp) < wp * zq;
                prob = wp * zq >= wq * zp ? (wp > 0 ? 1.f : 0.f) : static_cast<float>(wp * zq / (wq * zp));
            }
        }
        if (lane == 0) {
            if (p.prob && rank == 0) p.prob[r] = prob;
            if (!yes) atomicMin(&refused, r);
        }
    }
    if (p.prob && rank == 0 && tid == 0) p.prob[r0] = 0.f;
    __syncthreads();
    // ---- what the next token is drawn from
    if (warp == 0) {
        Choice c;
        const int no = refused;
        c.row = no == INT32_MAX ? r1 - 1 : no - 1;
        c.taken = c.row - r0;
        c.how = kPlain;
        c.column = -1;
        const bool have = no != INT32_MAX && no - r0 <= kKept;
        c.p = have ? kept[0][no - r0 - 1] : join(p, false, c.row, scale, table);
        c.q = c.p;
        if (no != INT32_MAX && !greedy) {
            if (drafts) {
                c.q = have ? kept[1][no - r0 - 1] : join(p, true, no, scale, table);
                if (!c.q.odd && c.q.m > -INFINITY) c.how = kLess;
            } else {
                c.column = p.tokens[no];
                c.how = kWithout;
            }
        }
        if (lane == 0) choice = c;
    }
    __syncthreads();
    const Choice c = choice;
    const bool nothing = c.p.odd || c.p.m == -INFINITY;
    if (greedy || nothing) {
        if (rank == 0 && tid == 0) p.accepted[a] = c.taken, p.token[a] = nothing ? -1 : c.p.best;
        return;
    }
    // The columns' shares of 2^60: weight times 2^60 / Z, p's and q's alike.
    const uint64_t fp = __double2ull_rn(4.0 * 1152921504606846976.0 * (17592186044416.0 / static_cast<double>(c.p.z)));
    const uint64_t fq = __double2ull_rn(4.0 * 1152921504606846976.0 * (17592186044416.0 / static_cast<double>(c.q.z)));
    const T* prow = logits + c.row * p.stride;
    const T* qrow = drafts ? drafts + (c.row + 1) * p.draft_stride : nullptr;
    int how = c.how;
    auto left = [&](float x, float y, int col) -> uint64_t {
        uint64_t w = weight(x, c.p.m, scale, table);
        if (how == kLess) {
            w = __umul64hi(w << 18, fp);
            const uint64_t v = __umul64hi(weight(y, c.q.m, scale, table) << 18, fq);
            w = w > v ? w - v : 0;
        } else if (how == kWithout && col == c.column) {
            w = 0;
        }
        return w;
    };
    // this block's columns: neighbouring steps; a thread has four neighbouring columns of each
    const int steps = (p.n + kStep - 1) / kStep, per = (steps + ranks - 1) / ranks;
    const int step0 = min(steps, rank * per), step1 = min(steps, step0 + per);
    uint64_t total = 0, before = 0, mine = 0;
    for (;;) {
        for (int s0 = step0; s0 < step1; s0 += kSpan) {
            float x[kSpan][4], y[kSpan][4];
#pragma unroll
            for (int i = 0; i < kSpan; ++i) {
                const int col = s0 + i < step1 ? (s0 + i) * kStep + 4 * tid : p.n;
                load4<T>(prow, p.vec, col, p.n, x[i]);
                if (how == kLess) load4<T>(qrow, p.draft_vec, col, p.n, y[i]);
            }
#pragma unroll
            for (int i = 0; i < kSpan; ++i) {
                if (s0 + i >= step1) break;
                uint64_t sum = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) sum += left(x[i][j], how == kLess ? y[i][j] : 0.f, (s0 + i) * kStep + 4 * tid + j);
#pragma unroll
                for (int k = 16; k >= 1; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
                if (lane == 0) part[(s0 + i - step0) * kChooseWarps + warp] = sum;
            }
        }
        __syncthreads();
        if (warp == 0) {
            uint64_t sum = 0;
            for (int i = lane; i < (step1 - step0) * kChooseWarps; i += 32) sum += part[i];
#pragma unroll
            for (int k = 16; k >= 1; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
            if (lane < ranks) *cluster.map_shared_rank(&share[rank], lane) = sum;
        }
        cluster.sync();
        total = before = 0;
        for (int i = 0; i < ranks; ++i) {
            if (i < rank) before += share[i];
            total += share[i];
        }
        mine = share[rank];
        if (total || how == kPlain) break;
        how = kPlain;  // (p and q alike but for their roundings)
        cluster.sync();
    }
    // ---- the lowest column whose running sum passes u * total  (nobody writes to another block any more)
    const double u = fmin(fmax(static_cast<double>(sample), 0.0), 1.0);
    uint64_t target = __double2ull_rd(u * static_cast<double>(total));
    if (target >= total) target = total - 1;
    if (warp > 0 || target < before || target >= before + mine) return;
    // the part in which it falls: part[step][warp] is in the columns' order; a lane takes neighbouring ones
    const uint64_t rest = target - before;
    const int parts = (step1 - step0) * kChooseWarps, each = (parts + 31) / 32;
    uint64_t sum = 0;
    for (int i = lane * each; i < min(parts, (lane + 1) * each); ++i) sum += part[i];
    uint64_t up = sum;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, up, k);
        if (lane >= k) up += o;
    }
    int hit = -1;
    uint64_t low = up - sum;
    if (rest >= low && rest < up) {
        hit = lane * each;
        while (rest >= low + part[hit]) low += part[hit++];
    }
    const int who = __ffs(__ballot_sync(0xffffffffu, hit >= 0)) - 1;  // (the parts' sums reach past rest: one lane has it)
    hit = __shfl_sync(0xffffffffu, hit, who);
    low = __shfl_sync(0xffffffffu, low, who);
    // its 128 columns once more
    const int col = (step0 + hit / kChooseWarps) * kStep + (hit % kChooseWarps) * 128 + 4 * lane;
    float x[4], y[4] = {};
    load4<T>(prow, p.vec, col, p.n, x);
    if (how == kLess) load4<T>(qrow, p.draft_vec, col, p.n, y);
    uint64_t w[4];
    sum = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) sum += w[j] = left(x[j], y[j], col + j);
    up = sum;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
        const uint64_t o = __shfl_up_sync(0xffffffffu, up, k);
        if (lane >= k) up += o;
    }
    low += up - sum;
    if (rest >= low && rest < low + sum) {
        int j = 0;
        while (rest >= low + w[j]) low += w[j++];
        p.accepted[a] = c.taken, p.token[a] = col + j;
    }
}

template <typename T>
cudaError_t launch(const Params& p, int dev, cudaStream_t s) {
    static kv::Once once;
    const cudaError_t o = once.allow_cluster(verify_choose<T>, dev);
    if (o != cudaSuccess) return o;
    if (p.rows > 0) {
        verify_stats<T><<<dim3(p.segs, p.rows, p.draft ? 2 : 1), kThreads, 0, s>>>(p);
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(p.agents) * p.ranks);
    cfg.blockDim = dim3(kChoose);
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(p.ranks);
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, verify_choose<T>, p);
}

int64_t segments(int64_t n) { return (n + kSeg - 1) / kSeg; }

}  // namespace verify
}  // namespace qmm

extern "C" {

qmm_status qmm_verify_workspace_bytes(int64_t rows, int64_t n, int64_t* bytes) {
    using namespace qmm::verify;
    if (!bytes || rows < 0 || n < 1) return QMM_ERR_INVALID_ARG;
    if (n > kMaxColumns || rows > 65535) return QMM_ERR_UNSUPPORTED_SHAPE;
    *bytes = 2 * rows * segments(n) * static_cast<int64_t>(sizeof(Stat));
    return QMM_OK;
}

qmm_status qmm_verify(const void* logits, int32_t type, int64_t stride, int64_t n, const void* draft_logits,
                      int64_t draft_stride, const int32_t* agent_rows, int32_t agents, int64_t rows,
                      const int32_t* tokens, const float* temperature, const float* accept_u, const float* sample_u,
                      int32_t* accepted, int32_t* token, float* prob, void* workspace, int64_t workspace_bytes,
                      int* err_word, void* stream) {
    using namespace qmm::verify;
    using qmm::kv::aligned;
    if (type < QMM_TYPE_F32 || type > QMM_TYPE_BF16 || agents < 1 || rows < 0 || n < 1 || stride < n || (draft_logits && draft_stride < n))
        return QMM_ERR_INVALID_ARG;
    int64_t need = 0;
    qmm_status st = qmm_verify_workspace_bytes(rows, n, &need);
    if (st != QMM_OK) return st;
    if (agents > 65535) return QMM_ERR_UNSUPPORTED_SHAPE;
    if (!agent_rows || !sample_u || !accepted || !token || !err_word || (rows > 0 && (!logits || !tokens || !accept_u || !workspace)))
        return QMM_ERR_INVALID_ARG;
    const int size = type == QMM_TYPE_F32 ? 4 : 2;
    if (!aligned(logits, size) || !aligned(draft_logits, size) || !aligned(agent_rows, 4) || !aligned(tokens, 4) || !aligned(temperature, 4) ||
        !aligned(accept_u, 4) || !aligned(sample_u, 4) || !aligned(accepted, 4) || !aligned(token, 4) || !aligned(prob, 4) ||
        !aligned(workspace, 16) || !aligned(err_word, 4))
        return QMM_ERR_MISALIGNED;
    if (workspace_bytes < need) return QMM_ERR_SCRATCH_TOO_SMALL;
    int dev = 0, sms = 0;
    st = qmm::kv::check_gpu(&dev, &sms);
    if (st != QMM_OK) return st;
    Params p = {};
    p.logits = logits, p.draft = draft_logits, p.agent_rows = agent_rows, p.tokens = tokens, p.temperature = temperature;
    p.accept_u = accept_u, p.sample_u = sample_u, p.accepted = accepted, p.token = token, p.prob = prob;
    p.stats = static_cast<Stat*>(workspace), p.err = err_word;
    p.stride = stride, p.draft_stride = draft_stride;
    p.rows = static_cast<int32_t>(rows), p.n = static_cast<int32_t>(n), p.segs = static_cast<int32_t>(segments(n)), p.agents = agents;
    p.vec = aligned(logits, 4 * size) && stride % 4 == 0;
    p.draft_vec = aligned(draft_logits, 4 * size) && draft_stride % 4 == 0;
    // blocks per sequence: 16 where that leaves no SM with two, and there are columns for them
    p.ranks = int64_t{agents} * kMaxRanks <= sms && n > 8 * kStep ? kMaxRanks : 8;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = type == QMM_TYPE_F32   ? launch<float>(p, dev, s)
                          : type == QMM_TYPE_F16 ? launch<__half>(p, dev, s)
                                                 : launch<__nv_bfloat16>(p, dev, s);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

}  // extern "C"
