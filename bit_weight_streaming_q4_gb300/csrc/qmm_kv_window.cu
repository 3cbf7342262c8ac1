// Attention with a sliding window over the paged cache: the joining kernel and the C entries.
//
// Where tokens are cut into chunks the kernel (qmm_kv_window.cuh) leaves, per row, head and chunk that the row
// sees, M_c, l_c and o_c: out = sum_c w_c o_c / sum_c w_c l_c with w_c = 2^(M_c - max M).
#include <cudaTypedefs.h>

#include "qmm_kv_window.cuh"

namespace qmm {
namespace window {

// A warp per (row, head), chunks in order.
template <int D>
__global__ void __launch_bounds__(256) window_join(const Params p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    bool falls = false;
    for (int i = threadIdx.x; i < p.agents; i += blockDim.x) falls |= p.agent_rows[i + 1] < p.agent_rows[i];
    falls = __syncthreads_or(falls);
    griddep_wait();  // the chunks' parts are there
    if (id >= static_cast<int64_t>(p.rows) * p.heads) return;
    const int r = static_cast<int>(id / p.heads);
    int a = 0, hi = p.agents;
    while (hi - a > 1) {
        const int mid = (a + hi) >> 1;
        if (p.agent_rows[mid] <= r) a = mid;
        else hi = mid;
    }
    int n = 0;
    if (!falls && r >= p.agent_rows[a] && r < p.agent_rows[a + 1] && sequence_ok(p, a)) n = chunks_of(p, length_of(p, r)).count();
    const float2* ml = reinterpret_cast<const float2*>(p.ml) + id * p.slots;
    const float* o = p.o + id * p.slots * D + lane * E;
    float top = -INFINITY, l = 0.f, v[E];
#pragma unroll
    for (int i = 0; i < E; ++i) v[i] = 0.f;
    for (int c = lane; c < n; c += 32)
        if (ml[c].y != 0.f) top = fmaxf(top, ml[c].x);
#pragma unroll
    for (int k = 16; k >= 1; k >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, k));
#pragma unroll 4
    for (int c = 0; c < n; ++c) {
        const float2 x = ml[c];
        const float w = x.y == 0.f ? 0.f : ex2(x.x - top);  // (a chunk with nothing to see has y = 0 and o = 0)
        l = fmaf(x.y, w, l);
        float u[E];
#pragma unroll
        for (int i = 0; i < E; i += 2) *reinterpret_cast<float2*>(u + i) = *reinterpret_cast<const float2*>(o + static_cast<int64_t>(c) * D + i);
#pragma unroll
        for (int i = 0; i < E; ++i) v[i] = fmaf(u[i], w, v[i]);
    }
    const bool none = l == 0.f;
    const float inv = none ? 0.f : 1.f / l;
#pragma unroll
    for (int i = 0; i < E; ++i) {
        const float y = none ? 0.f : v[i] * inv;
        const int64_t at = id * D + lane * E + i;
        if (p.out_type == QMM_TYPE_F32) static_cast<float*>(p.out)[at] = y;
        else if (p.out_type == QMM_TYPE_F16) static_cast<__half*>(p.out)[at] = __float2half_rn(y);
        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
    }
    if (lane == 0 && p.lse) p.lse[id] = none ? -INFINITY : (top + log2f(l)) * 0.6931471805599453f;
}

qmm_status check(const qmm_kv_dims* d, int64_t max_rows, int32_t window, int32_t sinks) {
    const qmm_status st = check_dims(d);
    if (st != QMM_OK) return st;
    if (max_rows < 0 || window < 1 || sinks < 0) return QMM_ERR_INVALID_ARG;
    if (max_rows > (1 << 24) / d->heads || d->max_agent_rows > (1 << 24) / (d->heads / d->kv_heads)) return QMM_ERR_UNSUPPORTED_SHAPE;
    return QMM_OK;
}

// How a plan's calls are laid out, by its dims alone (so that a row's bits are those of any other call).  Tokens are cut
// into the chunks whose rounds of items take least time by this estimate, or not at all: 4 sequences of 23,000 with a window
// of 4,096 at q8_0, 3 rows each, take 45 us in chunks of 1,408, 93 as 32 whole windows.
struct Layout {
    int32_t decode, qt, chunk, slots;
    int64_t o, bytes;
};
Layout layout(const qmm_kv_dims& d, int64_t max_rows, int32_t window, int32_t sinks) {
    constexpr int64_t kSms = 152;   // of a GB300
    constexpr double kItem = 7;     // an item's start and end, in the time of a tile of tokens: 15,000 and 2,200 clocks (2 to 20 choose alike there)
    constexpr double kJoin = 3;     // the second kernel
    const int64_t cap = int64_t{d.max_pages} * d.page_tokens, q = int64_t{d.max_agent_rows} * (d.heads / d.kv_heads);
    const int64_t tile = 128;
    Layout l = {};
    l.decode = q <= 128;
    l.qt = d.head_dim == 256 || l.decode ? 128 : 256;
    const int64_t items = d.agents * int64_t{d.kv_heads} * ((q + l.qt - 1) / l.qt);
    int64_t span = int64_t{window} + sinks + d.max_agent_rows;  // tokens that an item may see
    if (span > cap) span = cap;
    auto time = [&](int64_t n, int64_t tokens) { return static_cast<double>((n + kSms - 1) / kSms) * (static_cast<double>((tokens + tile - 1) / tile) + kItem); };
    double least = time(items, span);
    for (int64_t c = 256; c <= 8192 && c < span; c += c < 4096 ? 128 : 1024) {
        const double t = time(items * ((span + c - 1) / c + 1), c) + kJoin;  // (chunks are at fixed places: one more)
        const int64_t slots = ((sinks < cap ? sinks : cap) + c - 1) / c + ((cap + c - 1) / c < (window + c - 1) / c + 1 ? (cap + c - 1) / c : (window + c - 1) / c + 1);
        if (t >= least || max_rows * d.heads * slots > (int64_t{1} << 31) / (4 * d.head_dim)) continue;  // (2 GB of parts at most)
        least = t;
        l.chunk = static_cast<int32_t>(c);
        l.slots = static_cast<int32_t>(slots);
    }
    if (l.chunk) {
        auto up = [](int64_t x) { return (x + 255) / 256 * 256; };
        const int64_t parts = max_rows * d.heads * l.slots;
        l.o = up(parts * 8);
        l.bytes = l.o + up(parts * d.head_dim * 4);
    }
    return l;
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
    const int tile = 64;
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
cudaError_t launch_join(const Params& p, cudaStream_t s) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((int64_t{p.rows} * p.heads + 7) / 8));
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, window_join<D>, p);
}

}  // namespace window
}  // namespace qmm

extern "C" {

qmm_status qmm_kv_window_workspace_bytes(const qmm_kv_dims* dims, int64_t max_rows, int32_t window, int32_t sinks,
                                         int64_t* bytes) {
    if (!bytes) return QMM_ERR_INVALID_ARG;
    const qmm_status st = qmm::window::check(dims, max_rows, window, sinks);
    if (st == QMM_OK) *bytes = qmm::window::layout(*dims, max_rows, window, sinks).bytes;
    return st;
}

qmm_status qmm_kv_attend_window(const qmm_kv_dims* dims, const void* pool, const int32_t* page_table,
                                const int32_t* agent_rows, const int32_t* row_len, const void* q, int64_t q_stride,
                                int64_t rows, int64_t max_rows, float scale, int32_t window, int32_t sinks, void* out,
                                int32_t out_type, float* lse, void* workspace, int64_t workspace_bytes, int* err_word,
                                void* stream) {
    using namespace qmm::window;
    qmm_status st = check(dims, max_rows, window, sinks);
    if (st != QMM_OK) return st;
    if (rows < 0 || rows > max_rows || out_type < QMM_TYPE_F32 || out_type > QMM_TYPE_BF16) return QMM_ERR_INVALID_ARG;
    if (rows == 0) return QMM_OK;
    const Layout l = layout(*dims, max_rows, window, sinks);
    const int64_t need = l.bytes;
    if (!pool || !page_table || !agent_rows || !row_len || !q || !out || !err_word || (need > 0 && !workspace) ||
        q_stride < int64_t{dims->heads} * dims->head_dim)
        return QMM_ERR_INVALID_ARG;
    if (!aligned(pool, 16) || !aligned(q, 16) || q_stride % 8 != 0 || !aligned(out, 16) || !aligned(workspace, 16) ||
        !aligned(page_table, 4) || !aligned(agent_rows, 4) || !aligned(row_len, 4) || !aligned(lse, 4) || !aligned(err_word, 4))
        return QMM_ERR_MISALIGNED;
    if (workspace_bytes < need) return QMM_ERR_SCRATCH_TOO_SMALL;
    Launch a = {};
    int sms = 0;
    st = check_gpu(&a.device, &sms);
    if (st != QMM_OK) return st;
    if (dims->format != QMM_KV_Q8_0) {
        st = make_map(*dims, pool, &a.map);
        if (st != QMM_OK) return st;
    }
    Params& p = a.p;
    p.pool = static_cast<const uint8_t*>(pool), p.table = page_table, p.agent_rows = agent_rows, p.row_len = row_len;
    p.q = static_cast<const uint16_t*>(q), p.out = out, p.lse = lse, p.err = err_word, p.q_stride = q_stride;
    p.max_pages = dims->max_pages, p.pool_pages = static_cast<int32_t>(dims->pool_pages), p.page_tokens = dims->page_tokens;
    while ((1 << p.page_shift) < dims->page_tokens) ++p.page_shift;
    p.heads = dims->heads, p.kv_heads = dims->kv_heads, p.group = dims->heads / dims->kv_heads, p.agents = dims->agents;
    p.rows = static_cast<int32_t>(rows), p.max_agent_rows = dims->max_agent_rows, p.cap = dims->max_pages * dims->page_tokens;
    p.window = window < p.cap ? window : p.cap, p.sinks = sinks < p.cap ? sinks : p.cap;
    p.out_type = out_type, p.head_dim = dims->head_dim;
    p.chunk = l.chunk, p.slots = l.slots;
    p.ml = static_cast<float*>(workspace);
    p.o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + l.o);
    // (fp32's smallest number for a scale of 0: it leaves every finite score within 2^-21 of 0, and -infinity, which marks what a row
    // does not see, as it is)
    p.flip = scale < 0.f ? 0x80008000u : 0u;
    p.c2 = fabsf(scale) * 1.4426950408889634f;
    if (p.c2 == 0.f) p.c2 = 1.40129846e-45f;
    // blocks: one per SM, as far as there can be items
    int64_t most = (rows * p.group + l.qt - 1) / l.qt + (dims->agents < rows ? dims->agents : rows);
    most *= int64_t{dims->kv_heads} * (l.chunk ? l.slots + dims->max_agent_rows / l.chunk + 1 : 1);
    a.grid = static_cast<int>(most < sms ? most : sms);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const bool decode = l.decode && dims->head_dim != 256;  // (256: one stream, the same either way)
    const int hd = dims->head_dim;
    cudaError_t e = dims->format == QMM_KV_Q8_0  ? launch_q8(a, decode, s)
                    : dims->format == QMM_KV_F16 ? (decode ? launch_f16_decode(a, hd, s) : launch_f16_prompts(a, hd, s))
                                                 : (decode ? launch_bf16_decode(a, hd, s) : launch_bf16_prompts(a, hd, s));
    if (e == cudaSuccess && l.chunk)
        e = dims->head_dim == 64 ? launch_join<64>(p, s) : dims->head_dim == 128 ? launch_join<128>(p, s) : launch_join<256>(p, s);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

}  // extern "C"
