// Norms of queries and keys with the position rotation, in one pass over the qkv matmul's output.
//
// A warp takes a head: a lane holds D / 32 neighbouring dims, the sum of squares is a butterfly, and a
// dim's partner of the rotation is in the same lane (interleaved pairs) or in another one (halves),
// from which a shuffle brings it.  Cosine and sine of a row's rot_dim / 2 angles are formed once per block, for all
// of its heads.  An angle is pos * f turns, f = inv_freq / 2 pi as a 64-bit fraction of a turn: the
// product modulo 2^64 drops whole turns exactly, for any position, in integers (64-bit floating point
// runs at 1/64 of fp32's rate here; one multiplication per angle is left of it).
#include "qmm_decode.h"
#include "qmm_kv.cuh"

namespace qmm {
namespace rotate {

constexpr int kThreads = 256;
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
    int32_t vec;    // inputs can be read, and outputs written, by a lane's dims at once
    int32_t parts;  // blocks that share a row's heads
    float eps;
};

__device__ __forceinline__ float as_f32(float v) { return v; }
__device__ __forceinline__ float as_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ float as_f32(__nv_bfloat16 v) { return __bfloat162float(v); }

template <typename T, int E>
struct alignas(sizeof(T) * E <= 16 ? sizeof(T) * E : 16) Pack {
    T v[E];
};

template <typename T, int E>
__device__ __forceinline__ void load(const T* p, bool vec, float (&x)[E]) {
    if (vec) {
        const Pack<T, E> w = *reinterpret_cast<const Pack<T, E>*>(p);
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = as_f32(w.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) x[i] = as_f32(p[i]);
    }
}

__device__ __forceinline__ void to(float& d, float v) { d = v; }
__device__ __forceinline__ void to(__half& d, float v) { d = __float2half_rn(v); }
__device__ __forceinline__ void to(__nv_bfloat16& d, float v) { d = __float2bfloat16_rn(v); }

template <typename T, int E>
__device__ __forceinline__ void store(T* p, bool vec, const float (&x)[E]) {
    Pack<T, E> w;
#pragma unroll
    for (int i = 0; i < E; ++i) to(w.v[i], x[i]);
    if (vec) {
        *reinterpret_cast<Pack<T, E>*>(p) = w;
    } else {
#pragma unroll
        for (int i = 0; i < E; ++i) p[i] = w.v[i];
    }
}

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) rotate_kernel(const Params p) {
    constexpr int E = D / 32;
    __shared__ float2 turn[D / 2];  // cos, sin
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t row = blockIdx.x / p.parts;
    const int part = static_cast<int>(blockIdx.x % p.parts);
    const int all = p.heads + p.kv_heads;
    auto source = [&](int h) {
        const bool is_q = h < p.heads;
        const int64_t at = is_q ? row * p.q_stride + static_cast<int64_t>(h) * D : row * p.k_stride + static_cast<int64_t>(h - p.heads) * D;
        return static_cast<const T*>(is_q ? p.q : p.k) + at + lane * E;
    };
    const int first = part * kWarps + warp, step = p.parts * kWarps;
    float x[E];
    if (first < all) load<T, E>(source(first), p.vec, x);  // (on its way while the angles are formed)
    if (tid < p.half) {
        const int ax = p.axis ? p.axis[tid] : 0;
        const int32_t at = p.pos[static_cast<int64_t>(ax >= 0 && ax < p.axes ? ax : 0) * p.rows + row];
        const double f = static_cast<double>(p.inv_freq[tid]) * 0.15915494309189535;  // 1 / 2 pi: turns per position
        const double part_of_turn = f - floor(f);
        const uint64_t u = static_cast<uint64_t>(part_of_turn * 18446744073709551616.0) * static_cast<uint64_t>(static_cast<int64_t>(at));
        // the nearest of the turns, as half turns in -1 .. 1
        float c, s;
        sincospif(static_cast<float>(static_cast<int32_t>(u >> 32)) * 4.656612873077393e-10f, &s, &c);
        if (!isfinite(f)) c = s = __int_as_float(0x7FFFFFFF);
        turn[tid] = make_float2(c, s);
    }
    __syncthreads();
    for (int h = first; h < all; h += step) {
        const bool is_q = h < p.heads;
        float y[E];
#pragma unroll
        for (int i = 0; i < E; ++i) y[i] = x[i];
        if (h + step < all) load<T, E>(source(h + step), p.vec, x);
        const float* weight = is_q ? p.q_weight : p.k_weight;
        if (weight) {
            float sum = 0.f;
#pragma unroll
            for (int i = 0; i < E; ++i) sum = fmaf(y[i], y[i], sum);
#pragma unroll
            for (int k = 16; k >= 1; k >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, k);
            const float r = rsqrtf(sum * (1.f / D) + p.eps);
#pragma unroll
            for (int i = 0; i < E; ++i) y[i] = y[i] * r * weight[lane * E + i];
        }
        const int d0 = lane * E;
        float out[E];
        if (p.interleaved) {
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                out[i] = y[i], out[i + 1] = y[i + 1];
                if (d0 + i < 2 * p.half) {
                    const float2 t = turn[(d0 + i) >> 1];
                    out[i] = y[i] * t.x - y[i + 1] * t.y;
                    out[i + 1] = y[i] * t.y + y[i + 1] * t.x;
                }
            }
        } else {
            // (half is a multiple of 8, and so of E: a lane's dims are all of the first half, of the second, or neither)
            const bool low = d0 < p.half, in = d0 < 2 * p.half;
            const int other = in ? lane + (low ? p.half : -p.half) / E : lane;
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float z = __shfl_sync(0xffffffffu, y[i], other);
                out[i] = y[i];
                if (in) {
                    const float2 t = turn[low ? d0 + i : d0 + i - p.half];
                    out[i] = y[i] * t.x + (low ? -z : z) * t.y;
                }
            }
        }
        void* base = is_q ? p.q_out : p.k_out;
        const int64_t at = (is_q ? row * p.q_out_stride + static_cast<int64_t>(h) * D : row * p.k_out_stride + static_cast<int64_t>(h - p.heads) * D) + d0;
        const int type = is_q ? p.q_type : p.k_type;
        if (type == QMM_TYPE_F32) store<float, E>(static_cast<float*>(base) + at, p.vec, out);
        else if (type == QMM_TYPE_F16) store<__half, E>(static_cast<__half*>(base) + at, p.vec, out);
        else store<__nv_bfloat16, E>(static_cast<__nv_bfloat16*>(base) + at, p.vec, out);
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
    // a block per row, or more of them where that leaves SMs without one, down to a head per warp
    const int all = d->heads + d->kv_heads, most = (all + kWarps - 1) / kWarps;
    p.parts = 1;
    while (p.parts < most && rows * p.parts < 2 * sms) ++p.parts;
    if (rows > INT32_MAX / p.parts) return QMM_ERR_UNSUPPORTED_SHAPE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const cudaError_t e = d->in_type == QMM_TYPE_F32   ? launch<float>(p, d->head_dim, s)
                          : d->in_type == QMM_TYPE_F16 ? launch<__half>(p, d->head_dim, s)
                                                       : launch<__nv_bfloat16>(p, d->head_dim, s);
    return e == cudaSuccess ? QMM_OK : QMM_ERR_CUDA;
}
