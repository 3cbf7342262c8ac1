// Attention of new tokens over the paged cache: the joining kernel and the C entries.
//
// The split kernel (qmm_kv_attend.cuh) leaves, per chunk and query, M_c, l_c and o_c.  A row's
// result is out = sum_c w_c o_c / sum_c w_c l_c with w_c = 2^(M_c - max M), its lse the logarithm
// of that denominator (and max M), and a token's weight the sum over queries of 2^(x_t - M) / l.
#include <cudaTypedefs.h>

#include "qmm_kv_attend.cuh"

namespace qmm {
namespace kv {

constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;

// Reference and denominator of one query over its chunks, by the whole block: every thread returns
// them.  Up to 32 chunks every warp does alone; more are taken in a fixed order (thread
// c % kJoinThreads, a butterfly, the warps in turn), so the value depends on the query alone.
__device__ __forceinline__ float2 join_ml(const AttendParams& p, int64_t slot0, int n, float* tmp) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const float2* ml = reinterpret_cast<const float2*>(p.ml) + slot0;
    float m = kNoMax;
    if (n <= 32) {
        float2 v = make_float2(kNoMax, 0.f);
        if (lane < n) v = ml[static_cast<int64_t>(lane) * p.qp];
        m = v.x;
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
        float l = v.y * exp2f(v.x - (m == kNoMax ? 0.f : m));
#pragma unroll
        for (int k = 16; k >= 1; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
        return make_float2(m, l);
    }
#pragma unroll 4
    for (int c = tid; c < n; c += kJoinThreads) m = fmaxf(m, ml[static_cast<int64_t>(c) * p.qp].x);
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
    if (lane == 0) tmp[warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) m = fmaxf(m, tmp[w]);
    const float ref = m == kNoMax ? 0.f : m;
    float l = 0.f;
#pragma unroll 4
    for (int c = tid; c < n; c += kJoinThreads) {
        const float2 v = ml[static_cast<int64_t>(c) * p.qp];
        l = fmaf(v.y, exp2f(v.x - ref), l);
    }
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) l += __shfl_xor_sync(0xffffffffu, l, k);
    if (lane == 0) tmp[kJoinWarps + warp] = l;
    __syncthreads();
    l = 0.f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) l += tmp[kJoinWarps + w];
    return make_float2(m, l);
}

// sum_c 2^(M_c - ref) o_c over the chunks of one query, E consecutive dims a lane: chunks dealt to the warps in
// turn, the warps' sums in order.  Thread i < 32 E returns dim i of the warps' common range.
template <int E>
__device__ __forceinline__ float join_sum(const AttendParams& p, int64_t slot0, int n, float ref, const float* o0, int d, float* jsm) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    float acc[E];
#pragma unroll
    for (int i = 0; i < E; ++i) acc[i] = 0.f;
#pragma unroll(E == 1 ? 8 : 4)
    for (int c = warp; c < n; c += kJoinWarps) {
        const int64_t s = slot0 + static_cast<int64_t>(c) * p.qp;
        const float w = exp2f(p.ml[2 * s] - ref);
        const float* o = o0 + s * d + lane * E;
        float v[E];
        if constexpr (E == 1) v[0] = *o;
        else if constexpr (E == 2) *reinterpret_cast<float2*>(v) = *reinterpret_cast<const float2*>(o);
        else {
#pragma unroll
            for (int i = 0; i < E; i += 4) *reinterpret_cast<float4*>(v + i) = *reinterpret_cast<const float4*>(o + i);
        }
        // (a chunk that the row does not see has w = 0 and o = 0)
#pragma unroll
        for (int i = 0; i < E; ++i) acc[i] = fmaf(v[i], w, acc[i]);
    }
#pragma unroll
    for (int i = 0; i < E; ++i) jsm[(warp * 32 + lane) * E + i] = acc[i];
    __syncthreads();
    float v = 0.f;
    if (tid < 32 * E) {
#pragma unroll
        for (int w = 0; w < kJoinWarps; ++w) v += jsm[w * 32 * E + tid];
    }
    return v;
}

// What an output element is that came out as NaN though its denominator is a number: V is not finite at some slot
// t < n (a probability's second part times an infinity is NaN, if it is 0).  Every probability is positive: infinity
// if all that is not finite is infinity of one sign.  (A slow loop, for a result that is no number either way; as a
// function of its own it costs other calls nothing.)
__device__ __noinline__ float sum_of_infinities(const AttendParams& p, int format, int d, int a, int g, int n, int dim) {
    float sum = 0.f;
    for (int t = 0; t < n; ++t) {
        const int pg = p.table[static_cast<int64_t>(a) * p.max_pages + (t >> p.page_shift)], s = t & (p.page_tokens - 1);
        if (pg < 0 || pg >= p.pool_pages) continue;
        const int64_t rec = static_cast<int64_t>(pg) * p.kv_heads + g;
        float v;
        if (format == QMM_KV_Q8_0) {
            const uint8_t* r = p.pool + rec * kQ8Rec + kQ8Half;
            v = static_cast<float>(static_cast<int8_t>(r[dim * 64 + s])) *
                __half2float(*reinterpret_cast<const __half*>(r + 8192 + ((dim >> 5) * 64 + s) * 2));
        } else {
            const uint16_t w = reinterpret_cast<const uint16_t*>(p.pool)[((rec * 2 + 1) * p.page_tokens + s) * d + dim];
            v = format == QMM_KV_BF16 ? __uint_as_float(static_cast<uint32_t>(w) << 16) : __half2float(__ushort_as_half(w));
        }
        if (!isfinite(v)) sum += v;
        if (sum != sum) break;
    }
    return sum == 0.f ? __int_as_float(0x7FFFFFFF) : sum;  // (all finite: sums that left fp32)
}

// The first weight_blocks blocks: T slots a thread of one (sequence, KV head) each, taken in turn by
// however many blocks there are.  They are the long ones, so they start first and the others fill
// in beside them.  The others: one (row, head) each, or 32 dims of one where that makes few blocks (a
// sequence of 118,000 tokens, D = 256, 3 rows of 2 heads: 1,842 chunks a query).  The bits are the same.
// (Six blocks an SM leave 40 registers: <256, 1> spills 96 bytes, the other instances none to 28.)
template <int D, int T>
__global__ void __launch_bounds__(kJoinThreads, 6) attend_join(const AttendParams p, int weight_blocks, int slices) {
    extern __shared__ __align__(16) float jsm[];  // (read by float4)
    const int tid = threadIdx.x;
    griddep_wait();  // the split kernel has finished and its partials are visible
    if (static_cast<int>(blockIdx.x) >= weight_blocks) {
        const int block = (blockIdx.x - weight_blocks) / slices, slice = (blockIdx.x - weight_blocks) % slices;
        __shared__ int found;
        __shared__ float tmp[2 * kJoinWarps];
        const int h = block % p.heads, r = block / p.heads;
        if (tid == 0) found = -1;
        __syncthreads();
        for (int a = tid; a < p.agents; a += kJoinThreads) {
            const int4 i = p.info[a];
            if (r >= i.y && r - i.y < i.z) found = i.x < 0 ? -2 : a;  // at most one sequence holds the row
        }
        __syncthreads();
        const int a = found, g = h / p.group;
        const int width = slices == 1 ? D : 32;  // dims of the block
        float m = kNoMax, l = 0.f, v = 0.f;
        if (a == -1 && tid == 0 && h == 0 && slice == 0) atomicOr(p.err, kErrRange);
        if (a >= 0) {
            const int n = (min(p.row_len[r], p.info[a].x) + p.chunk - 1) / p.chunk;  // (the partials that there are)
            const int q = (r - p.info[a].y) * p.group + h % p.group;
            const int64_t slot0 = static_cast<int64_t>(a * p.kv_heads + g) * p.chunks * p.qp + q;
            const float2 t = join_ml(p, slot0, n, tmp);
            m = t.x;
            l = t.y;
            const float ref = m == kNoMax ? 0.f : m;
            v = slices == 1 ? join_sum<D / 32>(p, slot0, n, ref, p.o, D, jsm) : join_sum<1>(p, slot0, n, ref, p.o + 32 * slice, D, jsm);
        }
        // Nothing seen: no maximum, and no denominator either.  (A NaN is no maximum, but it is in l: a row whose
        // scores are all NaN comes here with M = -infinity and l = NaN, and divides by it.)
        const bool none = m == kNoMax && l == 0.f;
        if (tid < width) {
            v = none ? 0.f : v / l;
            if (v != v && l == l) v = sum_of_infinities(p, p.format, D, a, g, min(p.row_len[r], p.info[a].x), slice * 32 + tid);
            const int64_t at = static_cast<int64_t>(block) * D + slice * 32 + tid;
            if (p.out_type == QMM_TYPE_F32) static_cast<float*>(p.out)[at] = v;
            else if (p.out_type == QMM_TYPE_F16) static_cast<__half*>(p.out)[at] = __float2half_rn(v);
            else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(v);
        }
        if (tid == 0 && slice == 0 && p.lse) p.lse[block] = none ? kNoMax : (m + log2f(l)) * 0.6931471805599453f;
        return;
    }

    // ---- weights: tokens by thread, queries in order
    float* ref = jsm;           // [qp] M
    float* inv = jsm + p.qp;    // [qp] 1 / l
    constexpr int kSlots = T * kJoinThreads;
    const int per = (p.cap + kSlots - 1) / kSlots;
    const int64_t all = static_cast<int64_t>(p.agents) * p.kv_heads * per;
    for (int64_t b = blockIdx.x; b < all; b += weight_blocks) {
        const int ag = static_cast<int>(b / per), t0 = static_cast<int>(b % per) * kSlots;
        const int4 info = p.info[ag / p.kv_heads];
        if (t0 >= info.x) continue;  // past the sequence's longest row, or a refused sequence (-1)
        const int nq = info.z * p.group;
        __syncthreads();
        // several threads per query, chunks dealt out among them (consecutive queries lie side by side)
        const int per_q = nq <= 8 ? 32 : nq <= 32 ? 8 : nq <= 64 ? 4 : 1;
        for (int q0 = 0; q0 < nq; q0 += kJoinThreads / per_q) {
            const int q = q0 + tid / per_q, part = tid % per_q;
            const int n = q < nq ? (min(p.row_len[info.y + q / p.group], info.x) + p.chunk - 1) / p.chunk : 0;
            const float2* ml = reinterpret_cast<const float2*>(p.ml) + static_cast<int64_t>(ag) * p.chunks * p.qp + q;
            float m = kNoMax, l = 0.f;
#pragma unroll 4
            for (int c = part; c < n; c += per_q) {
                const float2 v = ml[static_cast<int64_t>(c) * p.qp];
                if (v.x > m) l *= exp2f(m - v.x), m = v.x;
                // (without a maximum v.y is 0, or the NaN of a chunk whose scores are all NaN)
                l = v.x > kNoMax ? fmaf(v.y, exp2f(v.x - m), l) : l + v.y;
            }
            for (int k = per_q >> 1; k >= 1; k >>= 1) {
                const float mo = __shfl_xor_sync(0xffffffffu, m, k), lo = __shfl_xor_sync(0xffffffffu, l, k);
                const float mn = fmaxf(m, mo), r = mn == kNoMax ? 0.f : mn;
                l = l * exp2f(m - r) + lo * exp2f(mo - r);
                m = mn;
            }
            if (part == 0 && q < nq) {
                // A query whose denominator is NaN: every score that it sees has to give NaN, and a slot that it does not
                // see (-infinity) nothing.  2^(x + 3.4e38) is infinity for the ones and 0 for the others; times 0.
                const bool nan = l != l;
                ref[q] = nan ? -3.402823466e38f : m == kNoMax ? 0.f : m;
                inv[q] = nan || m == kNoMax ? 0.f : 1.f / l;
            }
        }
        __syncthreads();
        const int64_t base = static_cast<int64_t>(ag) * p.cap, plane = static_cast<int64_t>(p.chunks) * p.chunk;
        const float4* x0 = reinterpret_cast<const float4*>(p.scores) + ag * (p.qp >> 2) * plane;
        // (Blocks beside each other hide the latency better than a thread's own loads: 8 x 16,000 bf16 at 8 rows, whole
        // calls: 169 us by six blocks an SM, 174 by five with the loop unrolled twice, 184 with the next four prefetched.)
        // T tokens a thread at once: their loads are in flight together and share
        // the queries' numbers.  (A token past info.x takes the last one's scores and stores nothing.)
        const float4* x[T];
        float sum[T];
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const int t = t0 + tid + i * kJoinThreads;
            x[i] = x0 + (t < info.x ? t : info.x - 1);
            sum[i] = 0.f;
        }
#pragma unroll(T == 1 ? 4 : 1)
        for (int q = 0; q < (nq & ~3); q += 4) {
            const float4 r = *reinterpret_cast<const float4*>(ref + q), w = *reinterpret_cast<const float4*>(inv + q);
            float4 v[T];
#pragma unroll
            for (int i = 0; i < T; ++i) v[i] = __ldcs(x[i] + (q >> 2) * plane);
#pragma unroll
            for (int i = 0; i < T; ++i) {
                sum[i] = fmaf(ex2(v[i].x - r.x), w.x, sum[i]);
                sum[i] = fmaf(ex2(v[i].y - r.y), w.y, sum[i]);
                sum[i] = fmaf(ex2(v[i].z - r.z), w.z, sum[i]);
                sum[i] = fmaf(ex2(v[i].w - r.w), w.w, sum[i]);
            }
        }
        if (nq & 3) {
            const int q = nq & ~3;
            float4 v[T];
            if ((nq & 3) == 3) {
#pragma unroll
                for (int i = 0; i < T; ++i) v[i] = __ldcs(x[i] + (q >> 2) * plane);
            } else {  // (two a token)
                const float2* x2 = reinterpret_cast<const float2*>(x0 + (q >> 2) * plane);
#pragma unroll
                for (int i = 0; i < T; ++i) {
                    const float2 u = __ldcs(x2 + (x[i] - x0));
                    v[i] = make_float4(u.x, u.y, 0.f, 0.f);
                }
            }
#pragma unroll
            for (int i = 0; i < T; ++i) {
                sum[i] = fmaf(ex2(v[i].x - ref[q]), inv[q], sum[i]);
                if ((nq & 3) > 1) sum[i] = fmaf(ex2(v[i].y - ref[q + 1]), inv[q + 1], sum[i]);
                if ((nq & 3) > 2) sum[i] = fmaf(ex2(v[i].z - ref[q + 2]), inv[q + 2], sum[i]);
            }
        }
#pragma unroll
        for (int i = 0; i < T; ++i) {
            const int t = t0 + tid + i * kJoinThreads;
            if (t < info.x) p.weight_out[base + t] = p.weight_in ? p.weight_in[base + t] + sum[i] : sum[i];
        }
    }
}

namespace {

// Tokens per chunk, by the dims alone (so that a row's bits are those of any other call, and on any GB300, for which
// the grid is a number here): of 1024 ..
// a tile, with pages that one warp can hold (32), the one whose rounds of a GB300's grid (608
// blocks at head dimension 64, 152 at 128, 304 at 256) take the least when all sequences are full, an item being
// its tiles and kItem tiles' time for its start and end (an estimate: the pipeline's fill, and the partial).  At head dimension 64, 61 ragged sequences: 104 us at 1,024, 92 at 512, 93 at 256.  At 128,
// calls with weights at 1,024 and 2,048: 109 and 112 us for a sequence of 131,071 (fp16), 184 and 189 for
// 8 x 16,000 at 8 rows (bf16), 108 and 115 for 4 x 23,000 (q8_0).
int32_t chunk_of(const qmm_kv_dims& d) {
    constexpr double kItem = 1.5;
    const int64_t cap = int64_t{d.max_pages} * d.page_tokens, blocks = d.head_dim == 64 ? 608 : d.head_dim == 128 ? 152 : 304;
    const int32_t tile = d.head_dim == 128 ? kTcTile : kTile;
    int32_t best = tile;
    double least = 0;
    for (int32_t c = tile; c <= 1024 && (c == tile || c <= 32 * d.page_tokens); c *= 2) {
        const int64_t items = (cap + c - 1) / c * d.agents * d.kv_heads;
        const double time = static_cast<double>((items + blocks - 1) / blocks) * (c / tile + kItem);
        if (c == tile || time <= least) {
            best = c;
            least = time;
        }
    }
    return best;
}

struct Layout {
    int64_t info, ml, o, scores, bytes;
    int32_t chunk, chunks, qp;
};

qmm_status layout(const qmm_kv_dims& d, bool weights, Layout* out) {
    const int64_t group = d.heads / d.kv_heads;
    const int64_t q = int64_t{d.max_agent_rows} * group;
    if (q > kMaxGroupQ) return QMM_ERR_UNSUPPORTED_SHAPE;
    Layout l = {};
    l.chunk = chunk_of(d);
    l.chunks = static_cast<int32_t>((int64_t{d.max_pages} * d.page_tokens + l.chunk - 1) / l.chunk);
    l.qp = static_cast<int32_t>((q + 7) / 8 * 8);
    const int64_t groups = int64_t{d.agents} * d.kv_heads;
    // item numbers, and slots of partials, in 31 bits
    if (groups * l.chunks > INT32_MAX / l.qp || groups > INT32_MAX / 8) return QMM_ERR_UNSUPPORTED_SHAPE;
    auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
    int64_t at = up(int64_t{d.agents} * 16);
    l.ml = at;
    at = up(at + groups * l.chunks * l.qp * 8);
    l.o = at;
    at = up(at + groups * l.chunks * l.qp * d.head_dim * 4);
    l.scores = at;
    if (weights) at = up(at + groups * l.chunks * l.chunk * l.qp * 4);
    l.bytes = at;
    *out = l;
    return QMM_OK;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            return nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }();
    return fn;
}

// The pool as rows of head_dim 16-bit elements: boxes of 64 elements (128 bytes, swizzled) x the
// rows of a tile that lie in one page.
qmm_status make_map(const qmm_kv_dims& d, const void* pool, CUtensorMap* map) {
    const int64_t rows = d.pool_pages * d.kv_heads * 2 * d.page_tokens;
    if (rows > INT32_MAX) return QMM_ERR_UNSUPPORTED_SHAPE;
    const PFN_cuTensorMapEncodeTiled_v12000 enc = encode_fn();
    if (!enc) return QMM_ERR_CUDA;
    const int tile = d.head_dim == 128 ? kTcTile : kTile;
    const cuuint64_t size[2] = {static_cast<cuuint64_t>(d.head_dim), static_cast<cuuint64_t>(rows)};
    const cuuint64_t stride[1] = {static_cast<cuuint64_t>(d.head_dim) * 2};
    const cuuint32_t box[2] = {64, static_cast<cuuint32_t>(tile < d.page_tokens ? tile : d.page_tokens)};
    const cuuint32_t one[2] = {1, 1};
    const CUresult r = enc(map, d.format == QMM_KV_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2,
                           const_cast<void*>(pool), size, stride, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? QMM_OK : QMM_ERR_CUDA;
}

template <int D>
cudaError_t launch_join(const AttendParams& p, int sms, cudaStream_t s) {
    const int slices = int64_t{p.rows} * p.heads * (D / 32) <= 4 * sms ? D / 32 : 1;
    const int out_blocks = p.rows * p.heads * slices;
    // slots a thread of the weights' part: four share a block's start; one where that leaves few blocks
    // with many queries, whose time is the latency of their loads (a call of 3 x 20,619 tokens, one KV head, 48
    // queries: 26 us by one, 36 by four; 85,205 tokens and 4 queries: 19 and 18)
    int64_t weight_blocks = 0;
    bool narrow = false;
    if (p.weight_out) {
        const int64_t groups = int64_t{p.agents} * p.kv_heads;
        weight_blocks = groups * ((p.cap + 4 * kJoinThreads - 1) / (4 * kJoinThreads));
        narrow = weight_blocks < 2 * sms && p.qp > 8;
        if (narrow) weight_blocks = groups * ((p.cap + kJoinThreads - 1) / kJoinThreads);
        if (weight_blocks > sms * 8) weight_blocks = sms * 8;
    }
    const int words = kJoinWarps * D > 2 * p.qp ? kJoinWarps * D : 2 * p.qp;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(out_blocks + weight_blocks));
    cfg.blockDim = dim3(kJoinThreads);
    cfg.dynamicSmemBytes = static_cast<size_t>(words) * 4;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, narrow ? attend_join<D, 1> : attend_join<D, 4>, p, static_cast<int>(weight_blocks), slices);
}

}  // namespace
}  // namespace kv
}  // namespace qmm

extern "C" {

qmm_status qmm_kv_attend_workspace_bytes(const qmm_kv_dims* dims, int32_t weights, int64_t* bytes) {
    if (!bytes) return QMM_ERR_INVALID_ARG;
    const qmm_status st = qmm::kv::check_dims(dims);
    if (st != QMM_OK) return st;
    qmm::kv::Layout l;
    const qmm_status sl = qmm::kv::layout(*dims, weights != 0, &l);
    if (sl == QMM_OK) *bytes = l.bytes;
    return sl;
}

qmm_status qmm_kv_attend(const qmm_kv_dims* dims, const void* pool, const int32_t* page_table,
                         const int32_t* agent_rows, const int32_t* row_len, const void* q, int64_t q_stride,
                         int64_t rows, float scale, void* out, int32_t out_type, float* lse, const float* weight_in,
                         float* weight_out, void* workspace, int64_t workspace_bytes, int* err_word, void* stream) {
    using namespace qmm::kv;
    qmm_status st = check_dims(dims);
    if (st != QMM_OK) return st;
    if (rows < 0 || (weight_in && !weight_out) || out_type < QMM_TYPE_F32 || out_type > QMM_TYPE_BF16)
        return QMM_ERR_INVALID_ARG;
    if (rows == 0) return QMM_OK;
    if (!pool || !page_table || !agent_rows || !row_len || !q || !out || !workspace || !err_word ||
        q_stride < int64_t{dims->heads} * dims->head_dim)
        return QMM_ERR_INVALID_ARG;
    if (rows > (1 << 24) / dims->heads) return QMM_ERR_UNSUPPORTED_SHAPE;
    Layout l;
    st = layout(*dims, weight_out != nullptr, &l);
    if (st != QMM_OK) return st;
    if (!aligned(pool, 16) || !aligned(q, 16) || q_stride % 8 != 0 || !aligned(out, 16) || !aligned(workspace, 16) ||
        !aligned(page_table, 4) || !aligned(agent_rows, 4) || !aligned(row_len, 4) || !aligned(lse, 4) || !aligned(weight_in, 4) ||
        !aligned(weight_out, 4) || !aligned(err_word, 4))
        return QMM_ERR_MISALIGNED;
    if (workspace_bytes < l.bytes) return QMM_ERR_SCRATCH_TOO_SMALL;
    AttendLaunch a = {};
    st = check_gpu(&a.device, &a.sms);
    if (st != QMM_OK) return st;
    if (dims->format != QMM_KV_Q8_0) {
        st = make_map(*dims, pool, &a.map);
        if (st != QMM_OK) return st;
    }
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    AttendParams& p = a.p;
    p.pool = static_cast<const uint8_t*>(pool);
    p.table = page_table;
    p.agent_rows = agent_rows;
    p.row_len = row_len;
    p.q = static_cast<const uint16_t*>(q);
    p.weight_in = weight_in;
    p.weight_out = weight_out;
    p.out = out;
    p.lse = lse;
    p.info = reinterpret_cast<int4*>(ws + l.info);
    p.ml = reinterpret_cast<float*>(ws + l.ml);
    p.o = reinterpret_cast<float*>(ws + l.o);
    p.scores = weight_out ? reinterpret_cast<float*>(ws + l.scores) : nullptr;
    p.err = err_word;
    p.q_stride = q_stride;
    p.max_pages = dims->max_pages;
    p.pool_pages = static_cast<int32_t>(dims->pool_pages);
    p.page_tokens = dims->page_tokens;
    while ((1 << p.page_shift) < dims->page_tokens) ++p.page_shift;
    p.heads = dims->heads;
    p.kv_heads = dims->kv_heads;
    p.group = dims->heads / dims->kv_heads;
    p.agents = dims->agents;
    p.rows = static_cast<int32_t>(rows);
    p.max_agent_rows = dims->max_agent_rows;
    p.chunk = l.chunk;
    p.chunks = l.chunks;
    p.qp = l.qp;
    p.cap = dims->max_pages * dims->page_tokens;
    p.out_type = out_type;
    p.format = dims->format;
    p.c2 = scale * 1.4426950408889634f;
    a.head_dim = dims->head_dim;
    a.max_q = dims->max_agent_rows * p.group;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    cudaError_t e = dims->format == QMM_KV_Q8_0  ? launch_attend_q8(a, s)
                    : dims->format == QMM_KV_F16 ? launch_attend_f16(a, s)
                                                 : launch_attend_bf16(a, s);
    if (e == cudaSuccess)
        e = dims->head_dim == 64    ? launch_join<64>(p, a.sms, s)
            : dims->head_dim == 128 ? launch_join<128>(p, a.sms, s)
                                    : launch_join<256>(p, a.sms, s);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

}  // extern "C"
