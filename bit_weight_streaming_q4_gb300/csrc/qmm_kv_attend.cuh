// Attention of new tokens over the paged cache: the split kernel.
//
// For query (row r of sequence a, head h of KV head g's group) and x_t = scale log2(e) q . k_t:
//   out = sum_t 2^(x_t - M) v_t / l,   l = sum_t 2^(x_t - M),   M = max_t x_t,   t < row_len[r].
// A sequence's slots are cut into chunks of p.chunk tokens at fixed places, so what a row
// gets never depends on the other rows of the call.  Each (sequence, chunk, KV head, tile of
// 8 NT queries) is an item, and each warp of the persistent grid takes items on its own: it
// streams the item's K and V tiles through a private ring of three half tiles (one K or V
// part each), keeps a running maximum, denominator and output per query in registers, and
// writes them as the item's partial.  Nothing is shared between warps but the table of
// sequences, so no barrier stands in the loop, and the ring runs on across items: the next
// item's first tiles are in flight while the last one is summed.
//
// Both products run on mma.sync m16n8k16 with tokens (S^T = K Q^T) and then dims
// (O^T = V^T P^T) as the 16 rows and queries as the 8 columns: one new token of a group of
// up to 8 heads fills one column tile, where queries as rows would pad them to 16.  S^T's
// accumulators become P^T's operands by an 8x8 transpose in registers (movmatrix).
// p enters the second product as two 16-bit parts (hi = round(p), lo = round(p - hi)),
// which keeps fp32's accuracy for the price of a second product; the kernel has the room,
// since the cache's bytes bound it.  p carries a factor 2^kShift (the
// denominator too), so that small probabilities stay clear of fp16's subnormals.
//
// 16-bit pools: a tile is 8 KB (64, 32 or 16 tokens), loaded by 2-D bulk tensor copies with
// the 128-byte swizzle, which makes the ldmatrix reads conflict-free.  q8_0 pools: a tile is
// one record; the K quants are exact in fp16, each 32-dim block's partial sum gets its scale
// in fp32.  V's scale depends on token and block and so goes into P: a token's exponent
// e_t = max over blocks of its scales' exponents joins the softmax's reference
// (y_t = x_t + e_t, M = max y_t), p^ = 2^(y_t - M) <= 1 is split, and p^ times the
// normalised scale (scale 2^-e_t) is formed error-free in half2 (product, its error by fma).
// No scale of the format can then overflow or vanish.
#pragma once

#include <cuda.h>

#include "qmm_kv.cuh"

namespace qmm {
namespace kv {

constexpr int kWarps = 8;
constexpr int kSlots = 3;            // half tiles in flight per warp
constexpr float kShift = 13.f;       // p's power of two: p^ <= 2^13, times a scale < 4 <= 2^15
constexpr float kNoMax = -INFINITY;

struct AttendParams {
    const uint8_t* pool;
    const int32_t* table;       // [agents][max_pages]
    const int32_t* agent_rows;  // [agents + 1]
    const int32_t* row_len;     // [rows]
    const uint16_t* q;          // [rows][heads][D]
    const float* weight_in;     // [agents][kv_heads][cap] or null
    float* weight_out;
    void* out;
    float* lse;                 // [rows][heads] or null
    float* ml;                  // [sequence][KV head][chunk][qp][2]: M and l
    float* o;                   // [sequence][KV head][chunk][qp][D]
    float* scores;              // [sequence][KV head][chunks * chunk][qp], x_t; null without weights
    int4* info;                 // [agents]: longest row (-1: refused), first row, rows, 0
    int* err;
    int64_t q_stride;
    int32_t max_pages, pool_pages, page_shift, page_tokens;
    int32_t heads, kv_heads, group, agents, rows;
    int32_t max_agent_rows;
    int32_t chunk, chunks;      // tokens per chunk, chunks per (sequence, KV head)
    int32_t qp;                 // queries per (sequence, KV head) in the workspace, a multiple of 8
    int32_t cap;                // slots per sequence: max_pages * page_tokens
    int32_t out_type;
    float c2;                   // scale * log2(e)
};

template <int FMT, int D>
struct Geo {
    static constexpr bool q8 = FMT == QMM_KV_Q8_0;
    static constexpr int TT = q8 ? 64 : 4096 / D;         // tokens per tile
    static constexpr int HB = q8 ? kQ8Half : TT * D * 2;  // bytes of a half tile
    static constexpr int JB = TT >= 32 ? 2 : 1;           // blocks of 16 tokens per softmax step
    static constexpr int SUB = TT / (16 * JB);            // softmax steps per tile
    static constexpr int MT = D / 16;
    static constexpr int max_nt = D == 256 ? 2 : 3;       // column tiles whose state fits the registers
};

// Dynamic shared memory: the rings (1024-byte aligned), the barriers, the table of sequences.
template <int FMT, int D>
constexpr int attend_smem(int agents) {
    return 1024 + kWarps * kSlots * Geo<FMT, D>::HB + kWarps * kSlots * 8 + 160 + (agents + 1) * 16;
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t a) {
    uint32_t d;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
template <bool BF>
__device__ __forceinline__ void mma16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if constexpr (BF)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
            "{%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        mma_m16n8k16(d, a0, a1, a2, a3, b0, b1);
}
// (hi, lo) 16-bit pairs of two fp32 values: value = hi + lo to 22 (bf16: 16) bits.
template <bool BF>
__device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    if constexpr (BF) {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
        const float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xFFFF0000u);
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(rb), "f"(ra));
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        hi = as_u32(h);
        lo = as_u32(__floats2half2_rn(a - __low2float(h), b - __high2float(h)));
    }
}
// Bytes 0, 1 (sel 0x4140) or 2, 3 (sel 0x4342) of four int8 already XORed with 0x80, as
// fp16x2, exact: the biased byte goes into the mantissa of 1024, and 1024 + 128 comes off.
__device__ __forceinline__ uint32_t i8_to_h2(uint32_t biased, uint32_t sel) {
    return as_u32(__hadd2(as_h2(prmt(biased, 0x64646464u, sel)), as_h2(0xE480E480u)));
}
__device__ __forceinline__ void tma_load_2d_hint(void* smem_dst, const void* tmap, int32_t c0, int32_t c1, uint64_t* bar,
                                                 uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(kWarps * 32, 1)
    attend_partial(const __grid_constant__ CUtensorMap map, const __grid_constant__ AttendParams p) {
    using G = Geo<FMT, D>;
    constexpr bool BF = FMT == QMM_KV_BF16;
    constexpr int TT = G::TT, JB = G::JB, SUB = G::SUB, MT = G::MT, QT = 8 * NT;
    extern __shared__ uint8_t sm_raw[];
    griddep_launch_dependents();  // the joining kernel waits for this grid's end before it reads
    uint8_t* sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
    uint64_t* bars = reinterpret_cast<uint64_t*>(sm + kWarps * kSlots * G::HB);
    int* tmp = reinterpret_cast<int*>(bars + kWarps * kSlots);  // 33 ints; [36]: abort flag
    int4* seq = reinterpret_cast<int4*>(tmp + 40);  // [agents + 1]: first item, longest row, shortest row, first row
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, t4 = lane & 3;
    volatile int* abort_flag = tmp + 36;

    // ---- the table of sequences: every CTA forms the same one
    if (tid < kWarps * kSlots) mbar_init(bars + tid, 1);
    if (tid == 0) {
        *abort_flag = 0;
        fence_mbar_init();
    }
    for (int a = tid; a <= p.agents; a += kWarps * 32) {
        const int r0 = p.agent_rows[a], r1 = a < p.agents ? p.agent_rows[a + 1] : r0;
        const bool ok = r0 >= 0 && r1 >= r0 && r1 <= p.rows && r1 - r0 <= p.max_agent_rows;
        seq[a] = make_int4(ok ? 0 : -1, 0, INT32_MAX, r0);
    }
    __syncthreads();
    for (int r = tid; r < p.rows; r += kWarps * 32) {
        int lo = 0, hi = p.agents;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (seq[mid].w <= r) lo = mid;
            else hi = mid;
        }
        if (r < seq[lo].w || r >= seq[lo + 1].w) continue;  // a row of no sequence
        const int len = p.row_len[r];
        if (len < 0 || len > p.cap) atomicExch(&seq[lo].x, -1);
        else {
            atomicMax(&seq[lo].y, len);
            atomicMin(&seq[lo].z, len);
        }
    }
    __syncthreads();
    int total = 0;
    for (int a0 = 0; a0 < p.agents; a0 += kWarps * 32) {
        const int a = a0 + tid;
        int n = 0;
        if (a < p.agents) {
            const int4 s = seq[a];
            const int nr = seq[a + 1].w - s.w;
            if (s.x >= 0 && nr > 0)
                n = (s.y + p.chunk - 1) / p.chunk * p.kv_heads * ((nr * p.group + QT - 1) / QT);
            if (blockIdx.x == 0) {
                p.info[a] = make_int4(s.x < 0 ? -1 : s.y, s.w, nr, 0);
                if (s.x < 0) atomicOr(p.err, kErrRange);
            }
        }
        int sum;
        const int at = block_exclusive(n, tmp, &sum);
        if (a < p.agents) seq[a].x = total + at;
        total += sum;
    }
    __syncthreads();

    // ---- this warp's items: w, w + stride, ...
    const int stride = gridDim.x * kWarps;
    uint8_t* ring = sm + warp * kSlots * G::HB;
    uint64_t* bar = bars + warp * kSlots;
    const uint64_t policy = l2_policy_evict_first();

    struct Item {
        int a, g, tile, tok0, end;
    };
    auto decode = [&](int item) {
        int lo = 0, hi = p.agents;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (seq[mid].x <= item) lo = mid;
            else hi = mid;
        }
        const int4 s = seq[lo];
        const int tiles = ((seq[lo + 1].w - s.w) * p.group + QT - 1) / QT;
        int rest = item - s.x;
        Item it;
        it.a = lo;
        it.tile = rest % tiles;
        rest /= tiles;
        it.g = rest % p.kv_heads;
        it.tok0 = rest / p.kv_heads * p.chunk;
        it.end = min(it.tok0 + p.chunk, s.y);
        return it;
    };
    // lane l: the item's l-th page (an item spans at most 32), -1 if the table points outside
    // the pool
    auto load_pages = [&](const Item& it) {
        const int first = it.tok0 >> p.page_shift;
        int pg = 0;
        if (((first + lane) << p.page_shift) < it.end) {
            pg = p.table[static_cast<int64_t>(it.a) * p.max_pages + first + lane];
            if (pg < 0 || pg >= p.pool_pages) {
                atomicOr(p.err, kErrPage);
                pg = -1;
            }
        }
        return pg;
    };
    // the producer's place: the item whose tiles are being requested, and the one after it,
    // whose pages are already known by then
    Item pi = {}, ni = {};
    int ppages = 0, npages = 0, ptok = 0, phalf = 0, pslot = 0, nitem = warp * gridDim.x + blockIdx.x;
    uint32_t bad = 0;  // bit s: the half tile in slot s has a page outside the pool
    int issued = 0, taken = 0;
    if (nitem < total) {
        ni = decode(nitem);
        npages = load_pages(ni);
    }
    auto issue = [&]() {
        if (ptok >= pi.end) {
            if (nitem >= total) return;
            pi = ni;
            ppages = npages;
            ptok = pi.tok0;
            phalf = 0;
            nitem += stride;
            if (nitem < total) {
                ni = decode(nitem);
                npages = load_pages(ni);
            }
        }
        uint8_t* dst = ring + pslot * G::HB;
        uint64_t* b = bar + pslot;
        const int first = pi.tok0 >> p.page_shift;
        if (lane == 0) fence_proxy_async_smem();  // the slot's generic accesses, before the copy
        if constexpr (G::q8) {
            const int pg = __shfl_sync(0xffffffffu, ppages, (ptok >> 6) - first);
            bad = pg < 0 ? bad | (1u << pslot) : bad & ~(1u << pslot);
            if (lane == 0) {
                if (pg < 0) mbar_arrive(b);
                else {
                    mbar_arrive_expect_tx(b, kQ8Half);
                    bulk_g2s(dst, p.pool + (static_cast<int64_t>(pg) * p.kv_heads + pi.g) * kQ8Rec + phalf * kQ8Half, kQ8Half,
                             b, policy);
                }
            }
        } else {
            // pieces of min(TT, page_tokens) tokens, those with tokens before the item's end
            const int br = min(TT, p.page_tokens);
            int pg[TT / 16];
            uint32_t bytes = 0;
            bool miss = false;
#pragma unroll
            for (int k = 0; k < TT / 16; ++k) {
                const int tok = ptok + k * br;
                const bool in = k * br < TT && tok < pi.end;
                const int x = __shfl_sync(0xffffffffu, ppages, in ? (tok >> p.page_shift) - first : 0);
                pg[k] = in ? x : -1;
                if (in && x < 0) miss = true;
                if (pg[k] >= 0) bytes += br * D * 2;
            }
            bad = miss ? bad | (1u << pslot) : bad & ~(1u << pslot);
            if (lane == 0) {
                if (bytes == 0) mbar_arrive(b);
                else mbar_arrive_expect_tx(b, bytes);
#pragma unroll
                for (int k = 0; k < TT / 16; ++k) {
                    if (pg[k] < 0) continue;
                    const int y = ((pg[k] * p.kv_heads + pi.g) * 2 + phalf) * p.page_tokens + ((ptok + k * br) & (p.page_tokens - 1));
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tma_load_2d_hint(dst + x * TT * 128 + k * br * 128, &map, 64 * x, y, b, policy);
                }
            }
        }
        ++issued;
        pslot = pslot == kSlots - 1 ? 0 : pslot + 1;
        phalf ^= 1;
        if (phalf == 0) ptok += TT;
    };
    for (int i = 0; i < kSlots; ++i) issue();

    bool live = true;
    int slot = 0, phase = 0;  // the consumer's slot and its barrier's phase
    auto await = [&]() {
        const bool ok = mbar_wait_bounded(bar + slot, phase, abort_flag);
        if (!__all_sync(0xffffffffu, ok)) live = false;
    };
    auto advance = [&]() {  // the slot is read: refill it
        __syncwarp();
        ++taken;
        if (++slot == kSlots) {
            slot = 0;
            phase ^= 1;
        }
        issue();
    };

    for (int item = warp * gridDim.x + blockIdx.x; item < total && live; item += stride) {
        const Item it = decode(item);
        const int r0 = seq[it.a].w, nq = (seq[it.a + 1].w - r0) * p.group, q0 = it.tile * QT;
        const int minlen = seq[it.a].z;
        const int nnt = min(NT, (nq - q0 + 7) >> 3);

        // Q^T's B fragments; k-slots of a q8_0 block are permuted so that a thread's eight dims
        // are contiguous (slots 2t, 2t+1, 2t+8, 2t+9 of step k2: dims 8t + 4 k2 + 0 .. 3)
        uint32_t qb[NT][MT][2];
        int qlen[NT][2], qlen_t[NT];  // tokens seen by the queries of the accumulators' columns, and of g8
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int qa = q0 + 8 * nt + g8;
            const uint16_t* row = nullptr;
            qlen_t[nt] = 0;
            if (qa < nq) {
                const int r = r0 + qa / p.group;
                qlen_t[nt] = p.row_len[r];
                row = p.q + r * p.q_stride + static_cast<int64_t>(it.g * p.group + qa % p.group) * D;
            }
#pragma unroll
            for (int e = 0; e < 2; ++e) qlen[nt][e] = __shfl_sync(0xffffffffu, qlen_t[nt], (2 * t4 + e) << 2);
            if constexpr (G::q8) {
#pragma unroll
                for (int blk = 0; blk < 4; ++blk) {
                    const uint4 v = row ? *reinterpret_cast<const uint4*>(row + 32 * blk + 8 * t4) : make_uint4(0, 0, 0, 0);
                    qb[nt][2 * blk][0] = v.x;
                    qb[nt][2 * blk][1] = v.y;
                    qb[nt][2 * blk + 1][0] = v.z;
                    qb[nt][2 * blk + 1][1] = v.w;
                }
            } else {
#pragma unroll
                for (int ks = 0; ks < MT; ++ks)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        qb[nt][ks][e] = row ? *reinterpret_cast<const uint32_t*>(row + 16 * ks + 2 * t4 + 8 * e) : 0u;
            }
        }

        float mx[NT][2], l[NT][2], o[MT][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mx[nt][0] = mx[nt][1] = kNoMax;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[mt][nt][c] = 0.f;
        }
        float* srow = p.scores ? p.scores + (static_cast<int64_t>(it.a * p.kv_heads + it.g) * p.chunks * p.chunk) * p.qp : nullptr;

        for (int tb = it.tok0; tb < it.end && live; tb += TT) {
            await();
            const uint8_t* kt = ring + slot * G::HB;
            const int vslot = slot == kSlots - 1 ? 0 : slot + 1;
            uint8_t* vt = ring + vslot * G::HB;
            const bool miss = (bad >> slot) & 1;
            if constexpr (G::q8) {  // V's scales join the softmax
                const bool ok = mbar_wait_bounded(bar + vslot, vslot == 0 ? phase ^ 1 : phase, abort_flag);
                if (!__all_sync(0xffffffffu, ok)) live = false;
            }
            if (!live) break;
            const bool edge = miss || tb + TT > minlen;  // some query does not see some token of the tile
#pragma unroll
            for (int sub = 0; sub < SUB; ++sub) {
                // ---- scores: s[jj][nt][c], c0/c1: token A, queries 2t4, 2t4 + 1; c2/c3: token B
                float s[JB][NT][4];
                int ta[JB], tB[JB];  // the thread's tokens within the tile
                uint32_t dv[JB][4][2], dinv[JB][2];  // q8_0: V scales of tokens 16 t4 + 4 j + 0 .. 3 by block
                float ea[JB], eb[JB];                // q8_0: exponents of tokens A and B
#pragma unroll
                for (int jj = 0; jj < JB; ++jj) {
                    const int j = sub * JB + jj;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[jj][nt][c] = 0.f;
                    if constexpr (G::q8) {
                        // row g8 of block j is token 16 (g8 / 2) + 4 j + g8 % 2, row g8 + 8 two on: the
                        // thread's P^T slots are then tokens 16 t4 + 4 j + 0 .. 3, contiguous in V
                        ta[jj] = 16 * (g8 >> 1) + 4 * j + (g8 & 1);
                        tB[jj] = ta[jj] + 2;
                        const int key = 2 * (g8 & 1) + (j & 1);
                        const uint2 sca = *reinterpret_cast<const uint2*>(kt + 8192 + ta[jj] * 8);
                        const uint2 scb = *reinterpret_cast<const uint2*>(kt + 8192 + tB[jj] * 8);
#pragma unroll
                        for (int blk = 0; blk < 4; ++blk) {
                            const uint8_t* ka = kt + ta[jj] * 128 + 16 * ((2 * blk + (t4 >> 1)) ^ key) + 8 * (t4 & 1);
                            const uint8_t* kb = kt + tB[jj] * 128 + 16 * ((2 * blk + (t4 >> 1)) ^ (key + 4)) + 8 * (t4 & 1);
                            uint2 va = *reinterpret_cast<const uint2*>(ka), vb = *reinterpret_cast<const uint2*>(kb);
                            va.x ^= 0x80808080u, va.y ^= 0x80808080u, vb.x ^= 0x80808080u, vb.y ^= 0x80808080u;
                            const __half2 pa = as_h2(blk < 2 ? sca.x : sca.y), pb = as_h2(blk < 2 ? scb.x : scb.y);
                            const float fa = (blk & 1) ? __high2float(pa) : __low2float(pa);
                            const float fb = (blk & 1) ? __high2float(pb) : __low2float(pb);
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                if (nt < nnt) {
                                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma_m16n8k16(d, i8_to_h2(va.x, 0x4140u), i8_to_h2(vb.x, 0x4140u), i8_to_h2(va.x, 0x4342u),
                                                 i8_to_h2(vb.x, 0x4342u), qb[nt][2 * blk][0], qb[nt][2 * blk][1]);
                                    mma_m16n8k16(d, i8_to_h2(va.y, 0x4140u), i8_to_h2(vb.y, 0x4140u), i8_to_h2(va.y, 0x4342u),
                                                 i8_to_h2(vb.y, 0x4342u), qb[nt][2 * blk + 1][0], qb[nt][2 * blk + 1][1]);
                                    s[jj][nt][0] = fmaf(d[0], fa, s[jj][nt][0]);
                                    s[jj][nt][1] = fmaf(d[1], fa, s[jj][nt][1]);
                                    s[jj][nt][2] = fmaf(d[2], fb, s[jj][nt][2]);
                                    s[jj][nt][3] = fmaf(d[3], fb, s[jj][nt][3]);
                                }
                        }
                        // the tokens' exponents (of the largest scale, in -14 .. 14) and normalised scales
                        uint32_t top0 = 0, top1 = 0;
#pragma unroll
                        for (int blk = 0; blk < 4; ++blk) {
                            const uint2 w = *reinterpret_cast<const uint2*>(vt + 8192 + (blk * 64 + 16 * t4 + 4 * j) * 2);
                            dv[jj][blk][0] = w.x;
                            dv[jj][blk][1] = w.y;
                            top0 = as_u32(__hmax2(as_h2(top0), as_h2(w.x & 0x7FFF7FFFu)));
                            top1 = as_u32(__hmax2(as_h2(top1), as_h2(w.y & 0x7FFF7FFFu)));
                        }
                        const __half2 least = as_h2(0x04000400u), most = as_h2(0x74007400u);
                        top0 = as_u32(__hmin2(__hmax2(as_h2(top0 & 0x7C007C00u), least), most));
                        top1 = as_u32(__hmin2(__hmax2(as_h2(top1 & 0x7C007C00u), least), most));
                        dinv[jj][0] = 0x78007800u - top0;  // 2^-e
                        dinv[jj][1] = 0x78007800u - top1;
                        const int sh = 16 * (g8 & 1) + 10;
                        ea[jj] = static_cast<float>(static_cast<int>((__shfl_sync(0xffffffffu, top0, g8 >> 1) >> sh) & 31u) - 15);
                        eb[jj] = static_cast<float>(static_cast<int>((__shfl_sync(0xffffffffu, top1, g8 >> 1) >> sh) & 31u) - 15);
                    } else {
                        ta[jj] = 16 * j + g8;
                        tB[jj] = ta[jj] + 8;
                        const uint32_t base = smem_u32(kt) + (16 * j + (lane & 15)) * 128;
#pragma unroll
                        for (int ks = 0; ks < MT; ++ks) {
                            const int ch = 2 * ks + (lane >> 4);
                            uint32_t a[4];
                            ldmatrix_x4(a, base + (ch >> 3) * (TT * 128) + (((ch & 7) ^ (lane & 7)) << 4));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                if (nt < nnt) mma16<BF>(s[jj][nt], a[0], a[1], a[2], a[3], qb[nt][ks][0], qb[nt][ks][1]);
                        }
                    }
                }
                // ---- base-2 scores, masks, the weights' copy, the step's maxima
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    if (nt >= nnt) continue;
                    float step[2] = {kNoMax, kNoMax};
#pragma unroll
                    for (int jj = 0; jj < JB; ++jj) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) s[jj][nt][c] *= p.c2;
                        if (edge) {
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                if (miss || tb + ta[jj] >= qlen[nt][e]) s[jj][nt][e] = kNoMax;
                                if (miss || tb + tB[jj] >= qlen[nt][e]) s[jj][nt][2 + e] = kNoMax;
                            }
                        }
                        if (srow && q0 + 8 * nt < p.qp) {
                            float* at = srow + static_cast<int64_t>(tb) * p.qp + q0 + 8 * nt + 2 * t4;
                            *reinterpret_cast<float2*>(at + ta[jj] * p.qp) = make_float2(s[jj][nt][0], s[jj][nt][1]);
                            *reinterpret_cast<float2*>(at + tB[jj] * p.qp) = make_float2(s[jj][nt][2], s[jj][nt][3]);
                        }
                        if constexpr (G::q8) {
                            s[jj][nt][0] += ea[jj];
                            s[jj][nt][1] += ea[jj];
                            s[jj][nt][2] += eb[jj];
                            s[jj][nt][3] += eb[jj];
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) step[e] = fmaxf(step[e], fmaxf(s[jj][nt][e], s[jj][nt][2 + e]));
                    }
                    float alpha[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = step[e];
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        m = fmaxf(m, mx[nt][e]);
                        // (nothing seen so far: any finite reference gives 2^-inf = 0)
                        const float ref = m == kNoMax ? 0.f : m;
                        alpha[e] = mx[nt][e] == m ? 1.f : ex2(mx[nt][e] - ref);
                        mx[nt][e] = m;
                        float sum = 0.f;
#pragma unroll
                        for (int jj = 0; jj < JB; ++jj) {
                            const float pa = ex2(s[jj][nt][e] - ref + kShift), pb = ex2(s[jj][nt][2 + e] - ref + kShift);
                            s[jj][nt][e] = pa;
                            s[jj][nt][2 + e] = pb;
                            if constexpr (G::q8)
                                sum += pa * __int_as_float((127 - static_cast<int>(ea[jj])) << 23) +
                                       pb * __int_as_float((127 - static_cast<int>(eb[jj])) << 23);
                            else
                                sum += pa + pb;
                        }
                        l[nt][e] = fmaf(l[nt][e], alpha[e], sum);
                    }
                    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                            for (int c = 0; c < 4; ++c) o[mt][nt][c] *= alpha[c & 1];
                    }
                }
                if (sub == SUB - 1) {
                    advance();  // K is read
                    if constexpr (!G::q8) {
                        if (SUB == 1) await();
                    }
                } else if constexpr (!G::q8) {
                    // V's first use in a tile of two steps; its slot follows K's
                    const bool ok = mbar_wait_bounded(bar + vslot, vslot == 0 ? phase ^ 1 : phase, abort_flag);
                    if (!__all_sync(0xffffffffu, ok)) live = false;
                }
                if (!live) break;

                if constexpr (!G::q8) {
                    if (edge) {
                        // Rows of V that some query does not see.  Past the sequence's end (and in
                        // tiles with a missing page) they hold anything and become zero.  A row that
                        // some queries see is looked at: if it holds a NaN or infinity, its
                        // contribution is added query by query, and zero takes its place.
                        const int lo = 16 * JB * sub, hi = lo + 16 * JB;
                        const int first = miss ? lo : max(lo, minlen - tb), last = miss ? lo : it.end - tb;
                        for (int t = first; t < hi; ++t) {
                            // lane's share of the row: D / 32 elements from dim lane * D / 32
                            constexpr int E = D / 64;  // 32-bit words
                            uint32_t* w = reinterpret_cast<uint32_t*>(vt + ((lane * E) >> 5) * (TT * 128) + t * 128 +
                                                                      (((((lane * E) & 31) >> 2) ^ (t & 7)) << 4) + ((lane * E) & 3) * 4);
                            bool odd = t >= last;
                            if (!odd) {
                                bool here = false;
                                constexpr uint32_t ex = BF ? 0x7F80u : 0x7C00u;
#pragma unroll
                                for (int i = 0; i < E; ++i)
                                    here |= (w[i] & ex) == ex || ((w[i] >> 16) & ex) == ex;
                                odd = __any_sync(0xffffffffu, here);
                                if (odd) {
                                    const int src = ((t & 7) << 2) | t4;
#pragma unroll
                                    for (int jj = 0; jj < JB; ++jj) {
                                        if ((t - lo) >> 4 != jj) continue;
                                        const bool up = t & 8;
#pragma unroll
                                        for (int nt = 0; nt < NT; ++nt) {
                                            if (nt >= nnt) continue;
                                            float pt[2];
#pragma unroll
                                            for (int e = 0; e < 2; ++e) {
                                                const float x = __shfl_sync(0xffffffffu, s[jj][nt][e], src);
                                                const float y = __shfl_sync(0xffffffffu, s[jj][nt][2 + e], src);
                                                pt[e] = up ? y : x;
                                            }
#pragma unroll
                                            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                                for (int c = 0; c < 4; ++c) {
                                                    const int d = 16 * mt + g8 + 8 * (c >> 1);
                                                    const uint16_t u = *reinterpret_cast<const uint16_t*>(
                                                        vt + (d >> 6) * (TT * 128) + t * 128 + ((((d & 63) >> 3) ^ (t & 7)) << 4) + (d & 7) * 2);
                                                    const float v = BF ? __uint_as_float(static_cast<uint32_t>(u) << 16)
                                                                       : __half2float(__ushort_as_half(u));
                                                    if (tb + t < qlen[nt][c & 1]) o[mt][nt][c] = fmaf(pt[c & 1], v, o[mt][nt][c]);
                                                }
                                        }
                                    }
                                }
                            }
                            __syncwarp();
                            if (odd)
#pragma unroll
                                for (int i = 0; i < E; ++i) w[i] = 0u;
                        }
                        __syncwarp();
                    }
                }

                // ---- P^T as B fragments (hi, lo), and O^T += V^T P^T
                if constexpr (G::q8) {
                    uint32_t bh[JB][NT][2], bl[JB][NT][2];
#pragma unroll
                    for (int jj = 0; jj < JB; ++jj)
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            if (nt < nnt) {
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    uint32_t hi, lo;
                                    split2<false>(s[jj][nt][2 * h], s[jj][nt][2 * h + 1], hi, lo);
                                    bh[jj][nt][h] = movmatrix_trans(hi);
                                    bl[jj][nt][h] = movmatrix_trans(lo);
                                }
                            }
#pragma unroll
                    for (int blk = 0; blk < 4; ++blk) {
                        uint2 w[2][2];  // V quants of the step's tokens: [m16 tile][row g8, g8 + 8]
#pragma unroll
                        for (int mt = 0; mt < 2; ++mt)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                w[mt][h] = *reinterpret_cast<const uint2*>(vt + (32 * blk + 16 * mt + 8 * h + g8) * 64 + 16 * t4 + 8 * sub);
                                w[mt][h].x ^= 0x80808080u;
                                w[mt][h].y ^= 0x80808080u;
                            }
#pragma unroll
                        for (int jj = 0; jj < JB; ++jj) {
                            const __half2 d0 = __hmul2(as_h2(dv[jj][blk][0]), as_h2(dinv[jj][0]));
                            const __half2 d1 = __hmul2(as_h2(dv[jj][blk][1]), as_h2(dinv[jj][1]));
                            uint32_t a[2][4];
#pragma unroll
                            for (int mt = 0; mt < 2; ++mt) {
                                const uint32_t w0 = jj ? w[mt][0].y : w[mt][0].x, w1 = jj ? w[mt][1].y : w[mt][1].x;
                                a[mt][0] = i8_to_h2(w0, 0x4140u);
                                a[mt][1] = i8_to_h2(w1, 0x4140u);
                                a[mt][2] = i8_to_h2(w0, 0x4342u);
                                a[mt][3] = i8_to_h2(w1, 0x4342u);
                            }
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                if (nt < nnt) {
                                    // (hi + lo) * scale = ph + pl: the product's rounding error comes back by fma
                                    __half2 ph0 = __hmul2(as_h2(bh[jj][nt][0]), d0), ph1 = __hmul2(as_h2(bh[jj][nt][1]), d1);
                                    __half2 pl0 = __hfma2(as_h2(bl[jj][nt][0]), d0, __hfma2(as_h2(bh[jj][nt][0]), d0, __hneg2(ph0)));
                                    __half2 pl1 = __hfma2(as_h2(bl[jj][nt][1]), d1, __hfma2(as_h2(bh[jj][nt][1]), d1, __hneg2(ph1)));
                                    uint32_t uh0 = as_u32(ph0), uh1 = as_u32(ph1), ul0 = as_u32(pl0), ul1 = as_u32(pl1);
                                    if (edge) {  // a scale that is NaN or infinite has no effect on rows that do not see it
                                        const int t = tb + 16 * t4 + 4 * (sub * JB + jj), n = miss ? 0 : qlen_t[nt];
                                        const uint32_t m0 = (t < n ? 0xFFFFu : 0u) | (t + 1 < n ? 0xFFFF0000u : 0u);
                                        const uint32_t m1 = (t + 2 < n ? 0xFFFFu : 0u) | (t + 3 < n ? 0xFFFF0000u : 0u);
                                        uh0 &= m0, ul0 &= m0, uh1 &= m1, ul1 &= m1;
                                    }
#pragma unroll
                                    for (int mt = 0; mt < 2; ++mt) {
                                        mma_m16n8k16(o[2 * blk + mt][nt], a[mt][0], a[mt][1], a[mt][2], a[mt][3], uh0, uh1);
                                        mma_m16n8k16(o[2 * blk + mt][nt], a[mt][0], a[mt][1], a[mt][2], a[mt][3], ul0, ul1);
                                    }
                                }
                        }
                    }
                } else {
#pragma unroll
                    for (int jj = 0; jj < JB; ++jj) {
                        const int j = sub * JB + jj;
                        uint32_t bh[NT][2], bl[NT][2];
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
                            if (nt < nnt) {
#pragma unroll
                                for (int h = 0; h < 2; ++h) {
                                    uint32_t hi, lo;
                                    split2<BF>(s[jj][nt][2 * h], s[jj][nt][2 * h + 1], hi, lo);
                                    bh[nt][h] = movmatrix_trans(hi);
                                    bl[nt][h] = movmatrix_trans(lo);
                                }
                            }
                        const int t = 16 * j + (lane & 7) + ((lane >> 4) << 3);
                        const uint32_t base = smem_u32(vt) + t * 128;
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            const int ch = 2 * mt + ((lane >> 3) & 1);
                            uint32_t a[4];
                            ldmatrix_x4_trans(a, base + (ch >> 3) * (TT * 128) + (((ch & 7) ^ (lane & 7)) << 4));
#pragma unroll
                            for (int nt = 0; nt < NT; ++nt)
                                if (nt < nnt) {
                                    mma16<BF>(o[mt][nt], a[0], a[1], a[2], a[3], bh[nt][0], bh[nt][1]);
                                    mma16<BF>(o[mt][nt], a[0], a[1], a[2], a[3], bl[nt][0], bl[nt][1]);
                                }
                        }
                    }
                }
            }
            if (!live) break;
            advance();  // V is read
        }
        if (!live) break;

        // ---- the item's partial
        const int64_t slot0 = (static_cast<int64_t>(it.a * p.kv_heads + it.g) * p.chunks + it.tok0 / p.chunk) * p.qp + q0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int qi = 8 * nt + 2 * t4 + e;
                float sum = l[nt][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                if (q0 + qi >= nq) continue;
                float* po = p.o + (slot0 + qi) * D;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    po[16 * mt + g8] = o[mt][nt][e];
                    po[16 * mt + g8 + 8] = o[mt][nt][2 + e];
                }
                if (g8 == 0) *reinterpret_cast<float2*>(p.ml + (slot0 + qi) * 2) = make_float2(mx[nt][e], sum);
            }
    }
    if (!live) {
        if (lane == 0) {
            *abort_flag = 1;
            atomicOr(p.err, kErrTimeout);
            // let every copy still in flight land before the CTA exits
            volatile int go_on = 0;
            for (; taken < issued; ++taken) {
                mbar_wait_bounded(bar + slot, phase, &go_on);
                if (++slot == kSlots) {
                    slot = 0;
                    phase ^= 1;
                }
            }
        }
        __syncwarp();
    }
}

// Launches the split kernel of a format (defined once per format).
struct AttendLaunch {
    AttendParams p;
    CUtensorMap map;
    int32_t head_dim;
    int32_t max_q;  // most queries of one sequence per KV head
    int32_t sms;
};
cudaError_t launch_attend_q8(const AttendLaunch& a, cudaStream_t s);
cudaError_t launch_attend_f16(const AttendLaunch& a, cudaStream_t s);
cudaError_t launch_attend_bf16(const AttendLaunch& a, cudaStream_t s);

template <int FMT, int D, int NT>
cudaError_t launch_attend_one(const AttendLaunch& a, cudaStream_t s) {
    const int bytes = attend_smem<FMT, D>(a.p.agents);
    cudaError_t e = cudaFuncSetAttribute(attend_partial<FMT, D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) return e;
    attend_partial<FMT, D, NT><<<a.sms, kWarps * 32, bytes, s>>>(a.map, a.p);
    return cudaGetLastError();
}

// One column tile of queries, or the most that the registers hold.  (With 8 queries or fewer the
// wide form would carry the registers of empty column tiles.)
template <int FMT, int D>
cudaError_t launch_attend_dim(const AttendLaunch& a, cudaStream_t s) {
    return a.max_q <= 8 ? launch_attend_one<FMT, D, 1>(a, s) : launch_attend_one<FMT, D, Geo<FMT, D>::max_nt>(a, s);
}

}  // namespace kv
}  // namespace qmm
