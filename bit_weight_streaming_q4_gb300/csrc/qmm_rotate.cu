// Norms of queries and keys with the position rotation, in one pass over the qkv matmul's output.
//
// D / 16 lanes take a head, a lane two pieces of 8 neighbouring dims each: those of the first and of the second half that
// turn together (or, interleaved, any two), so that a rotation stays in a lane and a head's sum of squares takes
// log2(D / 16) shuffles.  (A warp a head, with shuffles for both, took 115 us for the case below.)  Cosine and sine of a
// row's rot_dim / 2 angles are formed once per block, for all of its heads.  An angle is pos * f turns, f = inv_freq / 2 pi as
// a 64-bit fraction of a turn: the product modulo 2^64 drops whole turns exactly, for any position, in integers
// (64-bit floating point runs at 1/64 of fp32's rate here; one multiplication per angle is left of it).
// What bounds it: the bytes.  8,191 rows of 48 + 8 heads of 128 with norms, fp32 to fp16, 352 MB: 64 us, 5.5 TB/s, 0.83 of a
// plain copy's rate.  2,345 rows of 16 + 2 heads of 256, bf16, 64 dims of them turned by three axes, 43 MB: 20 us, of which
// the bytes are 6.5; the rest is a block's chain (angles, a barrier, three rounds of heads).  12 rows: 4.4 us, a launch.
#include "qmm_decode.h"
#include "qmm_kv.cuh"

namespace qmm {
namespace rotate {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

struct Params {
    const void* q;
    const void* k;
    const float* q_weight;
    const float* k_weight;
    const int32_t* pos;
    const float* inv_freq;
    const int32_t* axis;
    void* q_out;
    void* k_out;
    int64_t q_stride, k_stride, q_out_stride, k_out_stride, rows;
    int32_t heads, kv_heads, half, axes, interleaved;  // half: rot_dim / 2
    int32_t q_type, k_type;
    int32_t vec;    // inputs can be read, and outputs written, 16 bytes at a time
    int32_t weight_vec;  // .. and the weights
    int32_t parts;  // blocks that share a row's heads
    float eps;
};

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

// Eight neighbouring elements.
template <typename T>
__device__ __forceinline__ void load8(const T* p, bool vec, float (&x)[8]) {
    if (vec) {
        constexpr int N = 8 * sizeof(T) / 16;
        uint4 w[N];
#pragma unroll
        for (int i = 0; i < N; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
        T v[8];
        memcpy(v, w, sizeof(v));
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = as_f32(v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = as_f32(p[i]);
    }
}

__device__ __forceinline__ void to(float& d, float v) { d = v; }
__device__ __forceinline__ void to(__half& d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void to(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

template <typename T>
__device__ __forceinline__ void store8(T* p, bool vec, const float (&x)[8]) {
    T v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) to(v[i], x[i]);
    if (vec) {
        constexpr int N = 8 * sizeof(T) / 16;
        uint4 w[N];
        memcpy(w, v, sizeof(v));
#pragma unroll
        for (int i = 0; i < N; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = v[i];
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const Params p) {
    constexpr int L = D / 16;             // lanes of a head
    constexpr int kHeads = 32 / L;        // heads that a warp takes at a time
    __shared__ float2 turn[D / 2];        // cos, sin
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, i = lane % L;
    const int64_t row = blockIdx.x / p.parts;
    const int part = static_cast<int>(blockIdx.x % p.parts);
    const int all = p.heads + p.kv_heads, eighth = p.half / 8;
    // the lane's pieces: dims a0 .. a0 + 7 and b0 .. b0 + 7
    const bool turns = p.interleaved ? false : i < eighth;
    const int a0 = 8 * (turns ? i : p.interleaved ? 2 * i : 2 * eighth + 2 * (i - eighth)), b0 = turns ? a0 + p.half : a0 + 8;
    const int first = (part * kWarps + warp) * kHeads + lane / L, step = p.parts * kWarps * kHeads;
    auto source = [&](int h) {
        const bool is_q = h < p.heads;
        const int64_t at = is_q ? row * p.q_stride + static_cast<int64_t>(h) * D : row * p.k_stride + static_cast<int64_t>(h - p.heads) * D;
        return static_cast<const T*>(is_q ? p.q : p.k) + at;
    };
    float xa[8], xb[8];
    auto fetch = [&](int h) {
        if (h >= all) return;
        const T* src = source(h);
        load8(src + a0, p.vec, xa);
        load8(src + b0, p.vec, xb);
    };
    fetch(first);  // (on its way while the angles are formed)
    for (int f = tid; f < p.half; f += kThreads) {
        const int ax = p.axis ? p.axis[f] : 0;
        const int32_t at = p.pos[static_cast<int64_t>(ax >= 0 && ax < p.axes ? ax : 0) * p.rows + row];
        const double per = static_cast<double>(p.inv_freq[f]) * 0.15915494309189535;  // 1 / 2 pi: turns per position
        const double part_of_turn = per - floor(per);
        const uint64_t u = static_cast<uint64_t>(part_of_turn * 18446744073709551616.0) * static_cast<uint64_t>(static_cast<int64_t>(at));
        // the nearest of the turns, as half turns in -1 .. 1
        float c, s;
        sincospif(static_cast<float>(static_cast<int32_t>(u >> 32)) * 4.656612873077393e-10f, &s, &c);
        if (!isfinite(per)) c = s = __int_as_float(0x7FFFFFFF);
        turn[f] = make_float2(c, s);
    }
    __syncthreads();
    // the angles of the lane's pairs: dims (a0 + j, b0 + j), or interleaved (a0 + 2 j, a0 + 2 j + 1), then those of b0
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int f = p.interleaved ? (j < 4 ? a0 / 2 + j : b0 / 2 + j - 4) : a0 + j;
        const float2 t = (p.interleaved ? f < p.half : turns) ? turn[f] : make_float2(1.f, 0.f);
        c[j] = t.x, s[j] = t.y;
    }
    for (int h0 = first - lane / L; h0 < all; h0 += step) {  // (the same for the warp: its lanes meet in shuffles)
        const int h = h0 + lane / L;
        const bool is_q = h < p.heads;
        float ya[8], yb[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) ya[j] = xa[j], yb[j] = xb[j];
        fetch(h + step);
        const float* weight = is_q ? p.q_weight : p.k_weight;
        float sum = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fmaf(ya[j], ya[j], fmaf(yb[j], yb[j], sum));
#pragma unroll
        for (int k = L / 2; k >= 1; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
        if (h >= all) continue;
        if (weight) {
            const float r = rsqrtf(sum * (1.f / D) + p.eps);
            float wa[8], wb[8];
            load8(weight + a0, p.weight_vec, wa);
            load8(weight + b0, p.weight_vec, wb);
#pragma unroll
            for (int j = 0; j < 8; ++j) ya[j] = ya[j] * r * wa[j], yb[j] = yb[j] * r * wb[j];
        }
        if (p.interleaved) {
            const bool turns_a = a0 < 2 * p.half, turns_b = b0 < 2 * p.half;  // (of 16 dims that turn, both do)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float u = ya[2 * j], v = ya[2 * j + 1], x = yb[2 * j], y = yb[2 * j + 1];
                if (turns_a) ya[2 * j] = u * c[j] - v * s[j], ya[2 * j + 1] = u * s[j] + v * c[j];
                if (turns_b) yb[2 * j] = x * c[j + 4] - y * s[j + 4], yb[2 * j + 1] = x * s[j + 4] + y * c[j + 4];
            }
        } else if (turns) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const float u = ya[j], v = yb[j];
                ya[j] = u * c[j] - v * s[j], yb[j] = u * s[j] + v * c[j];
            }
        }
        void* base = is_q ? p.q_out : p.k_out;
        const int64_t at = is_q ? row * p.q_out_stride + static_cast<int64_t>(h) * D : row * p.k_out_stride + static_cast<int64_t>(h - p.heads) * D;
        const int type = is_q ? p.q_type : p.k_type;
        auto store = [&](auto* out) {
            store8(out + at + a0, p.vec, ya);
            store8(out + at + b0, p.vec, yb);
        };
        if (type == QMM_TYPE_F32) store(static_cast<float*>(base));
        else if (type == QMM_TYPE_F16) store(static_cast<__half*>(base));
        else store(static_cast<__nv_bfloat16*>(base));
    }
}

template <typename T>
cudaError_t launch(const Params& p, int dim, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(p.rows * p.parts);
    if (dim == 64) rotate_kernel<T, 64><<<grid, kThreads, 0, s>>>(p);
    else if (dim == 128) rotate_kernel<T, 128><<<grid, kThreads, 0, s>>>(p);
    else rotate_kernel<T, 256><<<grid, kThreads, 0, s>>>(p);
    return cudaGetLastError();
}

}  // namespace rotate
}  // namespace qmm

extern "C" qmm_status qmm_rotate(const qmm_rotate_dims* d, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                                 int64_t rows, const float* q_weight, const float* k_weight, const int32_t* pos,
                                 const float* inv_freq, const int32_t* axis, void* q_out, int64_t q_out_stride,
                                 void* k_out, int64_t k_out_stride, void* stream) {
    using namespace qmm::rotate;
    using qmm::kv::aligned;
    if (!d || d->heads < 0 || d->kv_heads < 0 || d->heads + int64_t{d->kv_heads} < 1 || rows < 0 || !(d->eps >= 0.f))
        return QMM_ERR_INVALID_ARG;
    for (const int32_t t : {d->in_type, d->q_type, d->k_type})
        if (t < QMM_TYPE_F32 || t > QMM_TYPE_BF16) return QMM_ERR_INVALID_ARG;
    const int64_t qn = int64_t{d->heads} * d->head_dim, kn = int64_t{d->kv_heads} * d->head_dim;
    if (d->head_dim != 64 && d->head_dim != 128 && d->head_dim != 256) return QMM_ERR_UNSUPPORTED_SHAPE;
    if (d->rot_dim < 0 || d->rot_dim > d->head_dim || d->rot_dim % 16 != 0 || d->axes < 1 || d->axes > 4) return QMM_ERR_UNSUPPORTED_SHAPE;
    if (d->heads > 65536 || d->kv_heads > 65536) return QMM_ERR_UNSUPPORTED_SHAPE;
    if (rows == 0) return QMM_OK;
    if ((d->heads && (!q || !q_out || q_stride < qn || q_out_stride < qn)) ||
        (d->kv_heads && (!k || !k_out || k_stride < kn || k_out_stride < kn)) || (d->rot_dim && (!pos || !inv_freq)))
        return QMM_ERR_INVALID_ARG;
    // in place: only element for element
    if ((d->heads && q_out == q && (d->q_type != d->in_type || q_out_stride != q_stride)) ||
        (d->kv_heads && k_out == k && (d->k_type != d->in_type || k_out_stride != k_stride)))
        return QMM_ERR_INVALID_ARG;
    auto size = [](int32_t t) { return t == QMM_TYPE_F32 ? 4 : 2; };
    const int in = size(d->in_type);
    if ((d->heads && (!aligned(q, in) || !aligned(q_out, size(d->q_type)))) || (d->kv_heads && (!aligned(k, in) || !aligned(k_out, size(d->k_type)))) ||
        !aligned(q_weight, 4) || !aligned(k_weight, 4) || !aligned(pos, 4) || !aligned(inv_freq, 4) || !aligned(axis, 4))
        return QMM_ERR_MISALIGNED;
    int dev = 0, sms = 0;
    const qmm_status st = qmm::kv::check_gpu(&dev, &sms);
    if (st != QMM_OK) return st;
    Params p = {};
    p.q = q, p.k = k, p.q_weight = q_weight, p.k_weight = k_weight, p.pos = pos, p.inv_freq = inv_freq, p.axis = axis;
    p.q_out = q_out, p.k_out = k_out;
    p.q_stride = q_stride, p.k_stride = k_stride, p.q_out_stride = q_out_stride, p.k_out_stride = k_out_stride, p.rows = rows;
    p.heads = d->heads, p.kv_heads = d->kv_heads, p.half = d->rot_dim / 2, p.axes = d->axes, p.interleaved = d->interleaved != 0;
    p.q_type = d->q_type, p.k_type = d->k_type, p.eps = d->eps;
    auto whole = [&](const void* a, int64_t stride, int32_t type) { return aligned(a, 16) && stride * size(type) % 16 == 0; };
    p.vec = (!d->heads || (whole(q, q_stride, d->in_type) && whole(q_out, q_out_stride, d->q_type))) &&
            (!d->kv_heads || (whole(k, k_stride, d->in_type) && whole(k_out, k_out_stride, d->k_type)));
    p.weight_vec = aligned(q_weight, 16) && aligned(k_weight, 16);
    // a block per row, or more of them where that leaves SMs without one, down to a round of heads per warp
    const int all = d->heads + d->kv_heads, round = kWarps * 32 / (d->head_dim / 16), most = (all + round - 1) / round;
    p.parts = 1;
    while (p.parts < most && rows * p.parts < 4 * sms) ++p.parts;
    if (rows > INT32_MAX / p.parts) return QMM_ERR_UNSUPPORTED_SHAPE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = d->in_type == QMM_TYPE_F32   ? launch<float>(p, d->head_dim, s)
                          : d->in_type == QMM_TYPE_F16 ? launch<__half>(p, d->head_dim, s)
                                                       : launch<__nv_bfloat16>(p, d->head_dim, s);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}
