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
// What bounds it: instructions in the first kernel, some 60 for a weight (its power of two as a pair of fp32 from a table
// of 64 and a series, the pair's 46 bits made an integer), so that 8 sequences of 8 rows of 151,936 fp32 logits with a draft
// model's, 73 MB, take 70 us where the bytes alone would take 11; latencies in the second, about 15 us whatever the size (the
// rows' numbers, the joins, the row's share again, an exchange in the cluster, the search).  4 x 3 rows: 34 us; 33 x 5 rows of
// 32,001 bf16 logits without a draft model: 33 us.  64-bit floating point and conversions of integers run at 1/64 and 1/8 of
// fp32's rate here: with powers in fp64 4 x 3 rows took 76 us.
#include <cooperative_groups.h>

#include <utility>

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

// 2^(i / 64) for i = 0 .. 63, as 2^44ths and as a pair.  (Rounded from 60 digits; formed on the device, whose 64-bit
// floating point is slow, they took some microseconds a block.)
struct alignas(16) Power {
    uint64_t fix;
    Two two;
};
__device__ const Power kPowers[64] = {
    {17592186044416ull, {0x1.0000000000000p+0f, 0x0.0p+0f}}, {17783752390528ull, {0x1.02c9a40000000p+0f, -0x1.887fa00000000p-28f}},
    {17977404757381ull, {0x1.059b0e0000000p+0f, -0x1.9d4f520000000p-25f}}, {18173165860252ull, {0x1.0874520000000p+0f, -0x1.e2990e0000000p-26f}},
    {18371058661769ull, {0x1.0b55860000000p+0f, 0x1.9f31220000000p-25f}}, {18571106374610ull, {0x1.0e3ec40000000p+0f, -0x1.a585cc0000000p-25f}},
    {18773332464219ull, {0x1.11301e0000000p+0f, -0x1.fdb4960000000p-25f}}, {18977760651566ull, {0x1.1429aa0000000p+0f, 0x1.d525bc0000000p-25f}},
    {19184414915921ull, {0x1.172b840000000p+0f, -0x1.c157420000000p-27f}}, {19393319497675ull, {0x1.1a35be0000000p+0f, 0x1.6df96e0000000p-25f}},
    {19604498901178ull, {0x1.1d48740000000p+0f, -0x1.d2e8ca0000000p-25f}}, {19817977897613ull, {0x1.2063b80000000p+0f, 0x1.0c519a0000000p-25f}},
    {20033781527906ull, {0x1.2387a60000000p+0f, 0x1.ceac480000000p-25f}}, {20251935105661ull, {0x1.26b4560000000p+0f, 0x1.789f380000000p-26f}},
    {20472464220127ull, {0x1.29e9e00000000p+0f, -0x1.5c04240000000p-25f}}, {20695394739203ull, {0x1.2d285a0000000p+0f, 0x1.b900c20000000p-26f}},
    {20920752812471ull, {0x1.306fe00000000p+0f, 0x1.4636e20000000p-25f}}, {21148564874263ull, {0x1.33c08c0000000p+0f, -0x1.b37d200000000p-25f}},
    {21378857646762ull, {0x1.371a740000000p+0f, -0x1.18aac60000000p-25f}}, {21611658143136ull, {0x1.3a7db40000000p+0f, -0x1.634c020000000p-25f}},
    {21846993670708ull, {0x1.3dea640000000p+0f, 0x1.8246840000000p-25f}}, {22084891834158ull, {0x1.4160a20000000p+0f, 0x1.f72e2a0000000p-28f}},
    {22325380538761ull, {0x1.44e0860000000p+0f, 0x1.8624b40000000p-30f}}, {22568487993661ull, {0x1.486a2c0000000p+0f, -0x1.47d8660000000p-25f}},
    {22814242715178ull, {0x1.4bfdae0000000p+0f, -0x1.593abc0000000p-25f}}, {23062673530157ull, {0x1.4f9b280000000p+0f, -0x1.2c5a6c0000000p-25f}},
    {23313809579344ull, {0x1.5342b60000000p+0f, -0x1.2c56100000000p-25f}}, {23567680320808ull, {0x1.56f4740000000p+0f, -0x1.295b040000000p-25f}},
    {23824315533396ull, {0x1.5ab07e0000000p+0f, -0x1.5bd5ec0000000p-27f}}, {24083745320225ull, {0x1.5e76f20000000p+0f, -0x1.4a5bd60000000p-25f}},
    {24346000112214ull, {0x1.6247ec0000000p+0f, -0x1.f8b5500000000p-25f}}, {24611110671650ull, {0x1.6623880000000p+0f, 0x1.2a91120000000p-27f}},
    {24879108095804ull, {0x1.6a09e60000000p+0f, 0x1.9fcef40000000p-26f}}, {25150023820570ull, {0x1.6dfb240000000p+0f, -0x1.cd72e80000000p-27f}},
    {25423889624159ull, {0x1.71f75e0000000p+0f, 0x1.1d8bee0000000p-25f}}, {25700737630824ull, {0x1.75feb60000000p+0f, -0x1.37b3060000000p-25f}},
    {25980600314626ull, {0x1.7a11480000000p+0f, -0x1.829fd00000000p-25f}}, {26263510503246ull, {0x1.7e2f340000000p+0f, -0x1.2616340000000p-25f}},
    {26549501381838ull, {0x1.82589a0000000p+0f, -0x1.accc7c0000000p-26f}}, {26838606496915ull, {0x1.868d9a0000000p+0f, -0x1.2edb440000000p-26f}},
    {27130859760289ull, {0x1.8ace540000000p+0f, 0x1.15506e0000000p-27f}}, {27426295453047ull, {0x1.8f1aea0000000p+0f, -0x1.baa2320000000p-26f}},
    {27724948229574ull, {0x1.93737c0000000p+0f, -0x1.e647440000000p-25f}}, {28026853121614ull, {0x1.97d82a0000000p+0f, -0x1.0d8d840000000p-31f}},
    {28332045542385ull, {0x1.9c49180000000p+0f, 0x1.51f8480000000p-27f}}, {28640561290725ull, {0x1.a0c6680000000p+0f, -0x1.2886a60000000p-26f}},
    {28952436555301ull, {0x1.a5503c0000000p+0f, -0x1.b83b540000000p-25f}}, {29267707918846ull, {0x1.a9e6b60000000p+0f, -0x1.50c0480000000p-25f}},
    {29586412362452ull, {0x1.ae89fa0000000p+0f, -0x1.a94b140000000p-26f}}, {29908587269910ull, {0x1.b33a2c0000000p+0f, -0x1.ec3a820000000p-26f}},
    {30234270432094ull, {0x1.b7f7700000000p+0f, -0x1.a094380000000p-25f}}, {30563500051394ull, {0x1.bcc1ea0000000p+0f, -0x1.f687c60000000p-25f}},
    {30896314746195ull, {0x1.c199be0000000p+0f, -0x1.3d56b20000000p-27f}}, {31232753555409ull, {0x1.c67f120000000p+0f, 0x1.cafa2a0000000p-25f}},
    {31572855943056ull, {0x1.cb720e0000000p+0f, -0x1.8837cc0000000p-27f}}, {31916661802889ull, {0x1.d072d40000000p+0f, 0x1.40f1300000000p-25f}},
    {32264211463077ull, {0x1.d5818e0000000p+0f, -0x1.822dbc0000000p-27f}}, {32615545690931ull, {0x1.da9e600000000p+0f, 0x1.ed99420000000p-27f}},
    {32970705697691ull, {0x1.dfc9740000000p+0f, -0x1.908c940000000p-25f}}, {33329733143360ull, {0x1.e502ee0000000p+0f, 0x1.e2cffe0000000p-26f}},
    {33692670141585ull, {0x1.ea4afa0000000p+0f, 0x1.52486c0000000p-27f}}, {34059559264602ull, {0x1.efa1be0000000p+0f, 0x1.cc2b440000000p-25f}},
    {34430443548229ull, {0x1.f507660000000p+0f, -0x1.246eb00000000p-26f}}, {34805366496913ull, {0x1.fa7c180000000p+0f, 0x1.9e90d80000000p-28f}},
};
struct Table {
    Power at[64];
};
__device__ __forceinline__ void fill(Table& t) {
    if (threadIdx.x < 64) reinterpret_cast<uint4*>(t.at)[threadIdx.x] = reinterpret_cast<const uint4*>(kPowers)[threadIdx.x];
}

// v + kRound, |v| < 2^22, is rounded to a whole number, which is in its low bits (and less kRound again, as a float).
constexpr float kRound = 12582912.f;  // 3 * 2^22
__device__ __forceinline__ int low_bits(float sum) { return __float_as_int(sum) - 0x4B400000; }

// 2^((x - m) scale) = w 2^(-44 - k), x <= m, m finite; false where it is below 2^least.  The exponent is a pair: x - m
// without error, times the scale's pair; its 64ths come from the table and 2^r of what is left, |r| <= 2^-7, from its
// series: r ln 2 as a pair, the terms from the square on in fp32 (together at most 2^-16: their roundings are below 2^-38).
__device__ __forceinline__ bool power(float x, float m, Two scale, const Table& t, float least, int64_t& w, int& k) {
    const float s = x - m, b = s - x;
    const float e = (x - (s - b)) - (m + b);
    const float ph = s * scale.hi;
    if (!(ph >= least)) return false;  // (and x = -infinity)
    const float pl = fmaf(s, scale.hi, -ph) + fmaf(s, scale.lo, e * scale.hi);
    const float near = fmaf(ph, 64.f, kRound);
    const int n = low_bits(near);
    // (what is left is 0 or a step of ph at least, and pl half a step at most: the sum of the two is exact as a pair)
    const float rest = fmaf(near - kRound, -0.015625f, ph), rh = rest + pl, rl = pl - (rh - rest);
    constexpr float kHi = 0.693147182464599609375f, kLo = -1.9046542999577680e-9f;  // ln 2
    const float uh = rh * kHi, ul = fmaf(rh, kHi, -uh) + fmaf(rh, kLo, rl * kHi);
    const float q = uh * uh * fmaf(uh, fmaf(uh, fmaf(uh, 1.f / 120, 1.f / 24), 1.f / 6), 0.5f);
    const float vh = uh + q, vl = ul + (q - (vh - uh));  // (|q| < |uh|)
    const Power power = t.at[n & 63];
    const Two f = power.two;
    const float wh = f.hi * vh, wl = fmaf(f.hi, vh, -wh) + fmaf(f.hi, vl, f.lo * vh);
    const float high = fmaf(wh, 16777216.f, kRound);  // 2^24ths
    const int l = low_bits(fmaf(fmaf(high - kRound, -5.9604644775390625e-8f, wh) + wl, 17592186044416.f, kRound));
    w = static_cast<int64_t>(power.fix) + (static_cast<int64_t>(low_bits(high)) << (kShift - 24)) + l;
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
    __shared__ int counts_sm;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    griddep_launch_dependents();
    const int seg = blockIdx.x, row = blockIdx.y;
    const bool draft = blockIdx.z == 1;
    const T* base = draft ? static_cast<const T*>(p.draft) + row * p.draft_stride : static_cast<const T*>(p.logits) + row * p.stride;
    const bool vec = draft ? p.draft_vec : p.vec;
    if (tid == 0) counts_sm = 0;
    __syncthreads();
    // the row's sequence (where agent_rows falls there may be several: nobody asks for what comes of it)
    auto find = [&] {
        for (int a = tid; a < p.agents; a += kThreads) {
            const int r0 = p.agent_rows[a];
            if (r0 <= row && row < p.agent_rows[a + 1] && !(draft && r0 == row)) {
                const Two scale = scale_of(p, a);
                scale_sm = scale;
                counts_sm = !draft || scale.hi != 0.f;
            }
        }
    };
    // A draft row that does not count (a sequence's first, a greedy one's, one of no sequence) is not read: it may not be there.
    // A target row is, so it is asked for before its sequence is known.
    if (draft) {
        find();
        __syncthreads();
        if (!counts_sm) return;
    }
    float x[kSteps][4];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) load4<T>(base, vec, seg * kSeg + (i * kThreads + tid) * 4, p.n, x[i]);
    if (!draft) find();
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
    if (!counts_sm) return;
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
    __shared__ Two scale_sm;
    __shared__ uint64_t share_of[2];           // 2^106 / Z, of p and q
    __shared__ Joined kept[2][kKept];          // target rows, draft rows
    __shared__ int refused;                    // lowest refused draft
    __shared__ uint64_t share[kMaxRanks];      // the blocks' sums (each block's own copy)
    __shared__ uint64_t part[kMaxSteps * kChooseWarps];
    cg::cluster_group cluster = cg::this_cluster();
    // (the other blocks' shared memory is there once they have started: said here, waited for behind the drafts)
    cg::cluster_group::arrival_token started = cluster.barrier_arrive();
    const int rank = static_cast<int>(cluster.block_rank()), ranks = p.ranks, a = blockIdx.x / ranks;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    bool falls = false;
    for (int i = tid; i < p.agents; i += kChoose) falls |= p.agent_rows[i + 1] < p.agent_rows[i];
    fill(table);
    const int r0 = p.agent_rows[a], r1 = p.agent_rows[a + 1];
    const float sample = p.sample_u[a];
    if (tid == 0) refused = INT32_MAX, scale_sm = scale_of(p, a);  // (64-bit arithmetic by one thread: it is slow)
    falls = __syncthreads_or(falls);
    griddep_wait();  // the first kernel's numbers are there
    const bool bad = falls || r0 < 0 || r1 > p.rows;
    if (bad && tid == 0 && rank == 0) atomicOr(p.err, kv::kErrRange);
    if (bad || r1 <= r0) {
        cluster.barrier_wait(std::move(started));
        if (tid == 0 && rank == 0) p.accepted[a] = 0, p.token[a] = -1;
        return;  // (the whole cluster)
    }
    const Two scale = scale_sm;
    const bool greedy = scale.hi == 0.f;
    const T* logits = static_cast<const T*>(p.logits);
    const T* drafts = static_cast<const T*>(p.draft);
    // ---- the drafts: a warp each
    for (int r = r0 + 1 + warp; r < r1; r += kChooseWarps) {
        const int x = p.tokens[r];
        const bool in = x >= 0 && x < p.n;
        // (what the joins do not need is asked for before them)
        const float xp = in ? as_f32(logits[(r - 1) * p.stride + x]) : 0.f, xq = in && drafts && !greedy ? as_f32(drafts[r * p.draft_stride + x]) : 0.f;
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
                if (p.prob && rank == 0) prob = wp * zq >= wq * zp ? (wp > 0 ? 1.f : 0.f) : static_cast<float>(wp * zq / (wq * zp));
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
        if (lane < 2) {  // the columns' shares of 2^60: weight times 2^60 / Z, p's and q's alike
            const Joined& of = lane ? c.q : c.p;
            if (of.z) share_of[lane] = __double2ull_rn(4.0 * 1152921504606846976.0 * (17592186044416.0 / static_cast<double>(of.z)));
        }
        if (lane == 0) choice = c;
    }
    __syncthreads();
    cluster.barrier_wait(std::move(started));
    const Choice c = choice;
    const bool nothing = c.p.odd || c.p.m == -INFINITY;
    if (greedy || nothing) {
        if (rank == 0 && tid == 0) p.accepted[a] = c.taken, p.token[a] = nothing ? -1 : c.p.best;
        return;
    }
    const uint64_t fp = share_of[0], fq = share_of[1];
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
    if (warp > 0) return;
    const double u = fmin(fmax(static_cast<double>(sample), 0.0), 1.0);
    uint64_t target = __double2ull_rd(u * static_cast<double>(total));
    if (target >= total) target = total - 1;
    if (target < before || target >= before + mine) return;
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
    // (without rows there is no first kernel, and what is read before the wait may come from the caller's kernel before)
    cfg.numAttrs = p.rows > 0 ? 2 : 1;
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
