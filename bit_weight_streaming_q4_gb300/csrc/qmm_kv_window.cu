// Attention with a sliding window and visible first tokens over the paged cache: the C entries and a
// simple kernel, a warp per (row, head) with one pass over the row's tokens.
//   out = sum_t 2^(x_t - M) v_t / l,   l = sum_t 2^(x_t - M),   M = max_t x_t,   x_t = scale log2(e) q . k_t,
// t < n with t >= n - window or t < sinks.
#include "qmm_decode.h"
#include "qmm_kv.cuh"

namespace qmm {
namespace window {

using namespace qmm::kv;

struct Params {
    const uint8_t* pool;
    const int32_t* table;
    const int32_t* agent_rows;
    const int32_t* row_len;
    const uint16_t* q;
    void* out;
    float* lse;
    int* err;
    int64_t q_stride;
    int32_t max_pages, pool_pages, page_shift, page_tokens, heads, kv_heads, group, agents, rows, max_agent_rows, cap;
    int32_t window, sinks, out_type, format, head_dim;
    float c2;
};

__device__ __forceinline__ float as_f32(uint16_t w, bool bf) {
    return bf ? __uint_as_float(static_cast<uint32_t>(w) << 16) : __half2float(__ushort_as_half(w));
}

template <int D>
__global__ void __launch_bounds__(256) attend_window_simple(const Params p) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t id = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
    bool falls = false;
    for (int i = threadIdx.x; i < p.agents; i += blockDim.x) falls |= p.agent_rows[i + 1] < p.agent_rows[i];
    falls = __syncthreads_or(falls);
    if (id >= static_cast<int64_t>(p.rows) * p.heads) return;
    const int r = static_cast<int>(id / p.heads), h = static_cast<int>(id % p.heads), g = h / p.group;
    int a = 0, hi = p.agents;
    while (hi - a > 1) {
        const int mid = (a + hi) >> 1;
        if (p.agent_rows[mid] <= r) a = mid;
        else hi = mid;
    }
    const int r0 = p.agent_rows[a], r1 = p.agent_rows[a + 1];
    int n = p.row_len[r];
    if (falls || r < r0 || r >= r1 || r0 < 0 || r1 > p.rows || r1 - r0 > p.max_agent_rows || n < 0 || n > p.cap) {
        if (lane == 0) atomicOr(p.err, kErrRange);
        n = 0;
    }
    float q[E], o[E], m = -INFINITY, l = 0.f;
    for (int i = 0; i < E; ++i) {
        q[i] = as_f32(p.q[r * p.q_stride + h * D + lane * E + i], p.format == QMM_KV_BF16);
        o[i] = 0.f;
    }
    const int from = max(0, n - p.window);
    for (int t = min(p.sinks, n) > 0 ? 0 : from; t < n; t = t + 1 == p.sinks ? max(t + 1, from) : t + 1) {
        if (t < from && t >= p.sinks) t = from;
        const int pg = p.table[static_cast<int64_t>(a) * p.max_pages + (t >> p.page_shift)], s = t & (p.page_tokens - 1);
        if (pg < 0 || pg >= p.pool_pages) {
            if (lane == 0) atomicOr(p.err, kErrPage);
            continue;
        }
        const int64_t rec = static_cast<int64_t>(pg) * p.kv_heads + g;
        float x = 0.f, v[E];
        for (int i = 0; i < E; ++i) {
            const int d = lane * E + i;
            float k;
            if (p.format == QMM_KV_Q8_0) {
                const uint8_t* b = p.pool + rec * kQ8Rec;
                k = static_cast<float>(static_cast<int8_t>(b[s * 128 + 16 * ((d >> 4) ^ q8_key(s & 7)) + (d & 15)])) *
                    __half2float(*reinterpret_cast<const __half*>(b + 8192 + (s * 4 + (d >> 5)) * 2));
                v[i] = static_cast<float>(static_cast<int8_t>(b[kQ8Half + d * 64 + s])) *
                       __half2float(*reinterpret_cast<const __half*>(b + kQ8Half + 8192 + ((d >> 5) * 64 + s) * 2));
            } else {
                const uint16_t* b = reinterpret_cast<const uint16_t*>(p.pool) + (rec * 2 * p.page_tokens + s) * D + d;
                k = as_f32(b[0], p.format == QMM_KV_BF16);
                v[i] = as_f32(b[static_cast<int64_t>(p.page_tokens) * D], p.format == QMM_KV_BF16);
            }
            x = fmaf(q[i], k, x);
        }
        for (int k = 16; k >= 1; k >>= 1) x += __shfl_xor_sync(0xffffffffu, x, k);
        x *= p.c2;
        const float mn = fmaxf(m, x), ref = mn == -INFINITY ? 0.f : mn;
        const float scale = exp2f(m - ref), w = exp2f(x - ref);
        l = l * scale + w;
        for (int i = 0; i < E; ++i) o[i] = o[i] * scale + w * v[i];
        m = mn;
    }
    const bool none = m == -INFINITY && l == 0.f;
    for (int i = 0; i < E; ++i) {
        const float y = none ? 0.f : o[i] / l;
        const int64_t at = id * D + lane * E + i;
        if (p.out_type == QMM_TYPE_F32) static_cast<float*>(p.out)[at] = y;
        else if (p.out_type == QMM_TYPE_F16) static_cast<__half*>(p.out)[at] = __float2half_rn(y);
        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(y);
    }
    if (lane == 0 && p.lse) p.lse[id] = none ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

qmm_status check(const qmm_kv_dims* d, int64_t max_rows, int32_t window, int32_t sinks) {
    const qmm_status st = check_dims(d);
    if (st != QMM_OK) return st;
    if (max_rows < 0 || window < 1 || sinks < 0) return QMM_ERR_INVALID_ARG;
    if (max_rows > (1 << 24) / d->heads || d->max_agent_rows > (1 << 24) / (d->heads / d->kv_heads)) return QMM_ERR_UNSUPPORTED_SHAPE;
    return QMM_OK;
}

}  // namespace window
}  // namespace qmm

extern "C" {

qmm_status qmm_kv_window_workspace_bytes(const qmm_kv_dims* dims, int64_t max_rows, int32_t window, int32_t sinks,
                                         int64_t* bytes) {
    if (!bytes) return QMM_ERR_INVALID_ARG;
    const qmm_status st = qmm::window::check(dims, max_rows, window, sinks);
    if (st == QMM_OK) *bytes = 0;
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
    int64_t need = 0;
    st = qmm_kv_window_workspace_bytes(dims, max_rows, window, sinks, &need);
    if (st != QMM_OK) return st;
    if (!pool || !page_table || !agent_rows || !row_len || !q || !out || !err_word || (need > 0 && !workspace) ||
        q_stride < int64_t{dims->heads} * dims->head_dim)
        return QMM_ERR_INVALID_ARG;
    if (!aligned(pool, 16) || !aligned(q, 16) || q_stride % 8 != 0 || !aligned(out, 16) || !aligned(workspace, 16) ||
        !aligned(page_table, 4) || !aligned(agent_rows, 4) || !aligned(row_len, 4) || !aligned(lse, 4) || !aligned(err_word, 4))
        return QMM_ERR_MISALIGNED;
    if (workspace_bytes < need) return QMM_ERR_SCRATCH_TOO_SMALL;
    int dev = 0, sms = 0;
    st = check_gpu(&dev, &sms);
    if (st != QMM_OK) return st;
    Params p = {};
    p.pool = static_cast<const uint8_t*>(pool), p.table = page_table, p.agent_rows = agent_rows, p.row_len = row_len;
    p.q = static_cast<const uint16_t*>(q), p.out = out, p.lse = lse, p.err = err_word, p.q_stride = q_stride;
    p.max_pages = dims->max_pages, p.pool_pages = static_cast<int32_t>(dims->pool_pages), p.page_tokens = dims->page_tokens;
    while ((1 << p.page_shift) < dims->page_tokens) ++p.page_shift;
    p.heads = dims->heads, p.kv_heads = dims->kv_heads, p.group = dims->heads / dims->kv_heads, p.agents = dims->agents;
    p.rows = static_cast<int32_t>(rows), p.max_agent_rows = dims->max_agent_rows, p.cap = dims->max_pages * dims->page_tokens;
    p.window = window, p.sinks = sinks, p.out_type = out_type, p.format = dims->format, p.head_dim = dims->head_dim;
    p.c2 = scale * 1.4426950408889634f;
    const unsigned grid = static_cast<unsigned>((rows * dims->heads + 7) / 8);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dims->head_dim == 64) attend_window_simple<64><<<grid, 256, 0, s>>>(p);
    else if (dims->head_dim == 128) attend_window_simple<128><<<grid, 256, 0, s>>>(p);
    else attend_window_simple<256><<<grid, 256, 0, s>>>(p);
    return cudaGetLastError() == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}

}  // extern "C"
