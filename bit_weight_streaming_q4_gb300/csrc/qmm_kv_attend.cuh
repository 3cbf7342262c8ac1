// Attention of new tokens over the paged cache: what the split kernels share, and the one for head
// dimensions 64 and 256.
//
// For query (row r of sequence a, head h of KV head g's group) and x_t = scale log2(e) q . k_t:
//   out = sum_t 2^(x_t - M) v_t / l,   l = sum_t 2^(x_t - M),   M = max_t x_t,   t < row_len[r].
// A sequence's slots are cut into chunks of p.chunk tokens at fixed places, so what a row
// gets never depends on the other rows of the call.  Each (sequence, chunk, KV head, tile of
// queries) is an item; the blocks of a persistent grid take items in turn and write M, l and the
// unnormalised output as the item's partial, which the joining kernel adds up.  All queries of a
// tile share each K and V tile on chip, so the cache is read once for as many queries as a tile has.
//
// This kernel (16-bit pools).  A block's four warps work on tiles of 64 tokens: each forms the scores
// of 16 tokens for all queries, the maxima meet in shared memory, the probabilities go there as the
// second product's operand, and each warp then sums over all 64 tokens for a quarter of the dims.
// So a thread holds the outputs of D / 4 dims only, and up to four blocks fit an SM: their barriers
// (two a tile) and loads overlap.  K and V parts stream through a ring of half tiles by 2-D bulk
// tensor copies with the 128-byte swizzle, which makes the ldmatrix reads conflict-free; the ring
// runs on across items.  (A first version gave every warp a ring and whole outputs of its own,
// without barriers: 61 ragged bf16 sequences at D = 64 took 118 us, 90 now.)
//
// Both products run on mma.sync m16n8k16 with tokens (S^T = K Q^T) and then dims
// (O^T = V^T P^T) as the 16 rows and queries as the 8 columns: one new token of a group of
// up to 8 heads fills one column tile, where queries as rows would pad them to 16.  S^T's
// accumulators become P^T's operands by an 8x8 transpose in registers (movmatrix).
// p enters the second product as two 16-bit parts (hi = round(p), lo = round(p - hi)), which keeps
// fp32's accuracy for the price of a second product.  It carries a factor 2^kShift (the denominator
// too), so that small probabilities stay clear of fp16's subnormals.
//
// What bounds it: at D = 64 the chain of barriers and waits of a 16 KB tile, not the bytes (61 ragged
// sequences, 250 MB: 63 us, 4.0 TB/s, and 27 for the join and the weights).  An M = 128 tensor core
// product would be half empty at D = 64, and D = 256 leaves it no room for two tiles.
#pragma once

#include <cuda.h>

#include "qmm_kv.cuh"

namespace qmm {
namespace kv {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kTile = 64;            // tokens per tile
constexpr int kTcTile = 128;         // tokens per tile of the tensor core kernel (head dimension 128)
constexpr float kShift = 13.f;       // p's power of two at head dimensions 64 and 256; off again in the partials
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
    float* ml;                  // [sequence][KV head][chunk][qp][2]: a reference M and l = sum 2^(x - M)
    float* o;                   // [sequence][KV head][chunk][qp][D]: sum 2^(x - M) v
    float* scores;              // [sequence][KV head][qp / 4][chunks * chunk][4] x_t, or null without weights;
                                // [..][2] in the last four if the sequence has at most two queries there
    int4* info;                 // [agents]: longest row (-1: refused), first row, rows, 0
    int* err;
    int64_t q_stride;
    int32_t max_pages, pool_pages, page_shift, page_tokens;
    int32_t heads, kv_heads, group, agents, rows;
    int32_t max_agent_rows;
    int32_t chunk, chunks;      // tokens per chunk, chunks per (sequence, KV head)
    int32_t qp;                 // queries per (sequence, KV head) in the workspace, a multiple of 8
    int32_t cap;                // slots per sequence: max_pages * page_tokens
    int32_t out_type, format;
    float c2;                   // scale * log2(e)
};

template <int FMT, int D, int NT>
struct Geo {
    static constexpr int QT = 8 * NT;             // queries of a tile
    static constexpr int HB = kTile * D * 2;      // bytes of a half tile (K or V)
    static constexpr int slots = 3;               // half tiles in flight
    static constexpr int KS = D / 16;
    static constexpr int MW = D / 64;             // m16 tiles of dims per warp
    static constexpr int PS = kTile + 8;          // halves per row of P, and bytes per row of Q: the padding
    static constexpr int QS = 2 * D + 16;         // keeps ldmatrix free of bank conflicts
    // blocks per SM that the registers are limited for (D = 256: the ring alone takes 96 KB)
    static constexpr int blocks = D == 256 ? 2 : 4;
    // dynamic shared memory, after aligning to 1024: ring, Q, P (hi, lo), maxima, lengths, barriers
    static constexpr int off_q = slots * HB;
    static constexpr int off_p = off_q + QT * QS;
    static constexpr int off_red = off_p + 2 * QT * PS * 2;
    static constexpr int off_len = off_red + QT * 16;
    static constexpr int off_bar = (off_len + QT * 4 + 15) / 16 * 16;
    static constexpr int off_misc = off_bar + slots * 8 + 8;  // tmp[33], abort, miss[slots], odd[2][2]
    static constexpr int off_seq = (off_misc + 48 * 4 + 15) / 16 * 16;
    static constexpr int smem(int agents) { return 1024 + off_seq + (agents + 1) * 16; }
};

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

// The table of sequences, in shared memory: every block forms the same one.  seq[a] = (first item,
// longest row, shortest row, first row), one more entry at the end; returns the number of items.
// Block 0 also writes it out for the joining kernel.  tmp: 33 ints.  The whole block takes part.
// Where agent_rows falls anywhere, every sequence is refused: the search below needs it sorted, and so does
// the joining kernel, which takes a row's length as checked if its sequence is not refused.
__device__ __forceinline__ int form_table(const AttendParams& p, int4* seq, int* tmp, int qt) {
    const int tid = threadIdx.x, n_threads = blockDim.x;
    bool falls = false;
    for (int a = tid; a <= p.agents; a += n_threads) {
        const int r0 = p.agent_rows[a], r1 = a < p.agents ? p.agent_rows[a + 1] : r0;
        const bool ok = r0 >= 0 && r1 >= r0 && r1 <= p.rows && r1 - r0 <= p.max_agent_rows;
        seq[a] = make_int4(ok ? 0 : -1, 0, INT32_MAX, r0);
        falls |= r1 < r0;
    }
    if (__syncthreads_or(falls))
        for (int a = tid; a <= p.agents; a += n_threads) seq[a].x = -1;
    for (int r = tid; r < p.rows; r += n_threads) {
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
    for (int a0 = 0; a0 < p.agents; a0 += n_threads) {
        const int a = a0 + tid;
        int n = 0;
        if (a < p.agents) {
            const int4 s = seq[a];
            const int nr = seq[a + 1].w - s.w;
            if (s.x >= 0 && nr > 0) n = (s.y + p.chunk - 1) / p.chunk * p.kv_heads * ((nr * p.group + qt - 1) / qt);
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
    return total;
}

// Item `item` of the table: chunk tok0 .. end - 1 of sequence a for KV head g and its tile-th tile of
// qt queries.  Tiles of the same chunk, and KV heads of the same pages, follow one another.
struct Item {
    int a, g, tile, tok0, end;
};
__device__ __forceinline__ Item decode_item(const AttendParams& p, const int4* seq, int item, int qt) {
    int lo = 0, hi = p.agents;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq[mid].x <= item) lo = mid;
        else hi = mid;
    }
    const int4 s = seq[lo];
    const int tiles = ((seq[lo + 1].w - s.w) * p.group + qt - 1) / qt;
    int rest = item - s.x;
    Item it;
    it.a = lo;
    it.tile = rest % tiles;
    rest /= tiles;
    it.g = rest % p.kv_heads;
    it.tok0 = rest / p.kv_heads * p.chunk;
    it.end = min(it.tok0 + p.chunk, s.y);
    return it;
}

// Lane l: the item's l-th page (an item spans at most 32), -1 if the table points outside the pool.
__device__ __forceinline__ int load_item_pages(const AttendParams& p, const Item& it) {
    const int first = it.tok0 >> p.page_shift, lane = threadIdx.x & 31;
    int pg = 0;
    if (((first + lane) << p.page_shift) < it.end) {
        pg = p.table[static_cast<int64_t>(it.a) * p.max_pages + first + lane];
        if (pg < 0 || pg >= p.pool_pages) {
            atomicOr(p.err, kErrPage);
            pg = -1;
        }
    }
    return pg;
}

template <int FMT, int D, int NT>
__global__ void __launch_bounds__(kThreads, (Geo<FMT, D, NT>::blocks))
    attend_partial(const __grid_constant__ CUtensorMap map, const __grid_constant__ AttendParams p) {
    using G = Geo<FMT, D, NT>;
    constexpr bool BF = FMT == QMM_KV_BF16;
    constexpr int QT = G::QT, MW = G::MW, PS = G::PS, QS = G::QS;
    extern __shared__ uint8_t sm_raw[];
    griddep_launch_dependents();  // the joining kernel waits for this grid's end before it reads
    uint8_t* sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
    uint16_t* Ph = reinterpret_cast<uint16_t*>(sm + G::off_p);  // [QT][PS]
    uint16_t* Pl = Ph + QT * PS;
    float* red = reinterpret_cast<float*>(sm + G::off_red);          // [QT][4 warps]
    int* qlen_sm = reinterpret_cast<int*>(sm + G::off_len);          // [QT]
    uint64_t* bar = reinterpret_cast<uint64_t*>(sm + G::off_bar);
    int* tmp = reinterpret_cast<int*>(sm + G::off_misc);
    volatile int* abort_flag = tmp + 33;
    volatile int* miss_sm = tmp + 34;                                // [slots]: a page of the half tile is outside the pool
    uint32_t* odd_sm = reinterpret_cast<uint32_t*>(tmp + 40);        // [2][2]: rows of V to be taken query by query
    int4* seq = reinterpret_cast<int4*>(sm + G::off_seq);  // [agents + 1]: first item, longest row, shortest row, first row
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g8 = lane >> 2, t4 = lane & 3;

    // ---- the table of sequences: every block forms the same one
    if (tid == 0) {
        for (int i = 0; i < G::slots; ++i) mbar_init(bar + i, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (tid < 4) odd_sm[tid] = 0;
    const int total = form_table(p, seq, tmp, QT);

    auto decode = [&](int item) { return decode_item(p, seq, item, QT); };

    // ---- the producer (warp 0): the item whose half tiles are being requested, and the one after
    // it, whose pages are already on their way.  Lane l holds an item's l-th page (an item spans
    // at most 32), -1 if the table points outside the pool.
    Item pi = {}, ni = {};
    int ppages = 0, npages = 0, ptok = 0, phalf = 0, pslot = 0, nitem = blockIdx.x, issued = 0;
    auto load_pages = [&](const Item& it) { return load_item_pages(p, it); };
    auto issue = [&]() {
        if (ptok >= pi.end) {
            if (nitem >= total) return;
            pi = ni;
            ppages = npages;
            ptok = pi.tok0;
            phalf = 0;
            nitem += gridDim.x;
            if (nitem < total) {
                ni = decode(nitem);
                npages = load_pages(ni);
            }
        }
        uint8_t* dst = sm + pslot * G::HB;
        uint64_t* b = bar + pslot;
        const int first = pi.tok0 >> p.page_shift;
        // pieces of min(64, page_tokens) tokens, those with tokens before the item's end
        const int br = min(kTile, p.page_tokens);
        int pg[kTile / 16];
        uint32_t bytes = 0;
        bool miss = false;
#pragma unroll
        for (int k = 0; k < kTile / 16; ++k) {
            const int tok = ptok + k * br;
            const bool in = k * br < kTile && tok < pi.end;
            const int x = __shfl_sync(0xffffffffu, ppages, in ? (tok >> p.page_shift) - first : 0);
            pg[k] = in ? x : -1;
            miss |= in && x < 0;
            if (pg[k] >= 0) bytes += br * D * 2;
        }
        if (lane == 0) {
            miss_sm[pslot] = miss;
            if (bytes == 0) mbar_arrive(b);
            else mbar_arrive_expect_tx(b, bytes);
            const uint64_t policy = l2_policy_evict_first();
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k) {
                if (pg[k] < 0) continue;
                const int y = ((pg[k] * p.kv_heads + pi.g) * 2 + phalf) * p.page_tokens + ((ptok + k * br) & (p.page_tokens - 1));
#pragma unroll
                for (int x = 0; x < D / 64; ++x)
                    tma_load_2d_hint(dst + x * kTile * 128 + k * br * 128, &map, 64 * x, y, b, policy);
            }
        }
        ++issued;
        pslot = pslot == G::slots - 1 ? 0 : pslot + 1;
        phalf ^= 1;
        if (phalf == 0) ptok += kTile;
    };
    if (warp == 0) {
        if (nitem < total) {
            ni = decode(nitem);
            npages = load_pages(ni);
        }
        for (int i = 0; i < G::slots; ++i) issue();
    }

    bool live = true;
    int slot = 0, phase = 0;  // of the next half tile to be read, and its barrier's phase
    int freed = 0;            // half tiles read that have not been refilled
    int taken = 0;
    uint32_t parity = 0;      // of the tile: which pair of odd_sm it uses
    auto next = [&]() {
        if (++slot == G::slots) {
            slot = 0;
            phase ^= 1;
        }
        ++taken;
    };

    for (int item = blockIdx.x; item < total && live; item += gridDim.x) {
        const Item it = decode(item);
        const int r0 = seq[it.a].w, nq = (seq[it.a + 1].w - r0) * p.group, q0 = it.tile * QT;
        const int minlen = seq[it.a].z;
        const int nnt = min(NT, (nq - q0 + 7) >> 3);
        __syncthreads();  // the previous item's queries, lengths and sums are read
        for (int i = tid; i < QT * (D / 8); i += kThreads) {
            const int qi = i / (D / 8), c = i % (D / 8), qa = q0 + qi;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (qa < nq)
                v = *reinterpret_cast<const uint4*>(p.q + (r0 + qa / p.group) * p.q_stride +
                                                    static_cast<int64_t>(it.g * p.group + qa % p.group) * D + 8 * c);
            *reinterpret_cast<uint4*>(sm + G::off_q + qi * QS + 16 * c) = v;
        }
        if (tid < QT) qlen_sm[tid] = q0 + tid < nq ? p.row_len[r0 + (q0 + tid) / p.group] : 0;
        __syncthreads();

        float mx[NT][2], l[NT][2], o[MW][NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            mx[nt][0] = mx[nt][1] = kNoMax;
            l[nt][0] = l[nt][1] = 0.f;
#pragma unroll
            for (int mt = 0; mt < MW; ++mt)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[mt][nt][c] = 0.f;
        }
        // scores, for the weights: four queries of consecutive tokens side by side
        const int64_t plane = static_cast<int64_t>(p.chunks) * p.chunk * 4;
        float* sbase = p.scores ? p.scores + static_cast<int64_t>(it.a * p.kv_heads + it.g) * (p.qp >> 2) * plane : nullptr;

        for (int tb = it.tok0; tb < it.end; tb += kTile) {
            const uint8_t* kt = sm + slot * G::HB;
            bool ok = mbar_wait_bounded(bar + slot, phase, abort_flag);
            const bool miss = miss_sm[slot] != 0;
            const bool edge = miss || tb + kTile > minlen;  // some query does not see some token of the tile
            next();
            uint8_t* vt = sm + slot * G::HB;

            // ---- scores of tokens 16 warp + g8 (c0, c1) and + 8 (c2, c3), queries 8 nt + 2 t4 + {0, 1}
            const int ta = 16 * warp + g8;
            float s[NT][4];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) s[nt][c] = 0.f;
            const uint32_t base = smem_u32(kt) + (16 * warp + (lane & 15)) * 128;
            const uint32_t qbase = smem_u32(sm + G::off_q) + (lane & 7) * QS + (lane >> 3) * 16;
#pragma unroll
            for (int ks = 0; ks < G::KS; ks += 2) {
                uint32_t a[2][4];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int ch = 2 * (ks + e) + (lane >> 4);
                    ldmatrix_x4(a[e], base + (ch >> 3) * (kTile * 128) + (((ch & 7) ^ (lane & 7)) << 4));
                }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    if (nt < nnt) {
                        uint32_t q[4];
                        ldmatrix_x4(q, qbase + nt * 8 * QS + ks * 32);
                        mma16<BF>(s[nt], a[0][0], a[0][1], a[0][2], a[0][3], q[0], q[1]);
                        mma16<BF>(s[nt], a[1][0], a[1][1], a[1][2], a[1][3], q[2], q[3]);
                    }
            }
            ok &= mbar_wait_bounded(bar + slot, phase, abort_flag);  // V
            next();
            // ---- base-2 scores, masks, the weights' copy, the warp's maxima
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if (nt < nnt) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) s[nt][c] *= p.c2;
                    if (edge) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int n = miss ? 0 : qlen_sm[8 * nt + 2 * t4 + e];
                            if (tb + ta >= n) s[nt][e] = kNoMax;
                            if (tb + ta + 8 >= n) s[nt][2 + e] = kNoMax;
                        }
                    }
                    const int qi = q0 + 8 * nt + 2 * t4;
                    if (sbase && qi < nq) {
                        const int n = nq - (qi & ~3) > 2 ? 4 : 2;
                        float* at = sbase + (qi >> 2) * plane + (tb + ta) * n + (qi & (n - 1));
                        *reinterpret_cast<float2*>(at) = make_float2(s[nt][0], s[nt][1]);
                        *reinterpret_cast<float2*>(at + 8 * n) = make_float2(s[nt][2], s[nt][3]);
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float m = fmaxf(s[nt][e], s[nt][2 + e]);
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 4));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 8));
                        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
                        if (g8 == 0) red[(8 * nt + 2 * t4 + e) * 4 + warp] = m;
                    }
                }
            // every warp is past this tile's K and the last tile's V and P; one decision for all
            if (__syncthreads_or(!ok)) {
                live = false;
                break;
            }
            if (warp == 0) {
                if (lane == 0) fence_proxy_async_smem();  // the slots' generic accesses, before the copies
                for (freed += 1; freed > 0; --freed) issue();
            }
            freed = 1;  // this tile's V, at the next tile's barrier
            if (tid < 2) odd_sm[2 * (parity ^ 1) + tid] = 0;

            // ---- new maxima, rescaling, probabilities to shared memory
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                if (nt < nnt) {
                    float alpha[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const float4 r = *reinterpret_cast<const float4*>(red + (8 * nt + 2 * t4 + e) * 4);
                        const float m = fmaxf(fmaxf(fmaxf(r.x, r.y), fmaxf(r.z, r.w)), mx[nt][e]);
                        // (nothing seen so far: any finite reference gives 2^-inf = 0)
                        const float ref = m == kNoMax ? 0.f : m;
                        alpha[e] = mx[nt][e] == m ? 1.f : ex2(mx[nt][e] - ref);
                        mx[nt][e] = m;
                        const float pa = ex2(s[nt][e] - ref + kShift), pb = ex2(s[nt][2 + e] - ref + kShift);
                        s[nt][e] = pa;
                        s[nt][2 + e] = pb;
                        float sum = pa + pb;
                        l[nt][e] = fmaf(l[nt][e], alpha[e], sum);
                    }
                    if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
                        for (int mt = 0; mt < MW; ++mt)
#pragma unroll
                            for (int c = 0; c < 4; ++c) o[mt][nt][c] *= alpha[c & 1];
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        uint32_t hi, lo;
                        split2<BF>(s[nt][2 * h], s[nt][2 * h + 1], hi, lo);
                        const int at = (8 * nt + g8) * PS + 16 * warp + 8 * h + 2 * t4;
                        *reinterpret_cast<uint32_t*>(Ph + at) = movmatrix_trans(hi);
                        *reinterpret_cast<uint32_t*>(Pl + at) = movmatrix_trans(lo);
                    }
                }
            if (edge) {
                // The warp's rows of V that some query does not see.  Past the sequence's end (and
                // in tiles with a missing page) they hold anything and become zero.  One that
                // some queries see and that holds a NaN or infinity is marked.
                const int last = miss ? 0 : it.end - tb;
                for (int t = max(16 * warp, miss ? 0 : minlen - tb); t < 16 * warp + 16; ++t) {
                    uint32_t* w = reinterpret_cast<uint32_t*>(vt + ((lane * MW) >> 5) * (kTile * 128) + t * 128 +
                                                              (((((lane * MW) & 31) >> 2) ^ (t & 7)) << 4) + ((lane * MW) & 3) * 4);
                    if (t >= last) {
#pragma unroll
                        for (int i = 0; i < MW; ++i) w[i] = 0u;
                    } else {
                        bool here = false;
                        constexpr uint32_t ex = BF ? 0x7F80u : 0x7C00u;
#pragma unroll
                        for (int i = 0; i < MW; ++i) here |= (w[i] & ex) == ex || ((w[i] >> 16) & ex) == ex;
                        if (__any_sync(0xffffffffu, here) && lane == 0) atomicOr(odd_sm + 2 * parity + (t >> 5), 1u << (t & 31));
                    }
                }
            }
            __syncthreads();  // P is complete
            if (edge && (odd_sm[2 * parity] | odd_sm[2 * parity + 1])) {
                // marked rows: added query by query, to those that see them; then zero in the product
#pragma unroll 1
                for (int t = 0; t < kTile; ++t) {
                    if (!((odd_sm[2 * parity + (t >> 5)] >> (t & 31)) & 1)) continue;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c) {
                            const int q = 8 * nt + 2 * t4 + (c & 1);
                            if (nt >= nnt || tb + t >= qlen_sm[q]) continue;
                            const uint32_t h = Ph[q * PS + t], u = Pl[q * PS + t];
                            const float pt = BF ? __uint_as_float(h << 16) + __uint_as_float(u << 16)
                                                : __half2float(__ushort_as_half(h)) + __half2float(__ushort_as_half(u));
#pragma unroll
                            for (int mt = 0; mt < MW; ++mt) {
                                const int d = 16 * (warp * MW + mt) + g8 + 8 * (c >> 1);
                                const uint32_t v = *reinterpret_cast<const uint16_t*>(
                                    vt + (d >> 6) * (kTile * 128) + t * 128 + ((((d & 63) >> 3) ^ (t & 7)) << 4) + (d & 7) * 2);
                                o[mt][nt][c] = fmaf(pt, BF ? __uint_as_float(v << 16) : __half2float(__ushort_as_half(v)), o[mt][nt][c]);
                            }
                        }
                }
                __syncthreads();
                for (int t = warp; t < kTile; t += kWarps)
                    if ((odd_sm[2 * parity + (t >> 5)] >> (t & 31)) & 1)
                        for (int i = lane; i < D / 2; i += 32)
                            *reinterpret_cast<uint32_t*>(vt + (i >> 5) * (kTile * 128) + t * 128 + (i & 31) * 4) = 0u;
                __syncthreads();
            }

            // ---- O^T += V^T P^T for dims D / 4 * warp ..
            const uint32_t pbase = smem_u32(Ph) + ((lane & 7) * PS + (lane >> 3) * 8) * 2;
            const uint32_t vbase = smem_u32(vt) + ((lane & 7) + ((lane >> 4) << 3)) * 128;
#pragma unroll
            for (int ks = 0; ks < 4; ks += 2) {
                uint32_t a[2][MW][4];
#pragma unroll
                for (int e = 0; e < 2; ++e)
#pragma unroll
                    for (int mt = 0; mt < MW; ++mt) {
                        const int ch = 2 * (warp * MW + mt) + ((lane >> 3) & 1);
                        ldmatrix_x4_trans(a[e][mt], vbase + (ch >> 3) * (kTile * 128) + (ks + e) * 16 * 128 +
                                                        (((ch & 7) ^ (lane & 7)) << 4));
                    }
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    if (nt < nnt) {
                        uint32_t bh[4], bl[4];
                        ldmatrix_x4(bh, pbase + (nt * 8 * PS + ks * 16) * 2);
                        ldmatrix_x4(bl, pbase + (QT * PS + nt * 8 * PS + ks * 16) * 2);
#pragma unroll
                        for (int e = 0; e < 2; ++e)
#pragma unroll
                            for (int mt = 0; mt < MW; ++mt) {
                                mma16<BF>(o[mt][nt], a[e][mt][0], a[e][mt][1], a[e][mt][2], a[e][mt][3], bh[2 * e], bh[2 * e + 1]);
                                mma16<BF>(o[mt][nt], a[e][mt][0], a[e][mt][1], a[e][mt][2], a[e][mt][3], bl[2 * e], bl[2 * e + 1]);
                            }
                    }
            }
            parity ^= 1;
        }
        if (!live) break;

        // ---- the item's partial (the shift comes off the sums: taken off M, it could be lost to a large M's spacing)
        constexpr float kUnshift = 1.f / (1 << static_cast<int>(kShift));
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                float sum = l[nt][e];
                sum += __shfl_xor_sync(0xffffffffu, sum, 4);
                sum += __shfl_xor_sync(0xffffffffu, sum, 8);
                sum += __shfl_xor_sync(0xffffffffu, sum, 16);
                l[nt][e] = sum;
            }
        __syncthreads();  // (the maxima in `red` are read)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
                if (g8 == 0) red[(8 * nt + 2 * t4 + e) * 4 + warp] = l[nt][e];
        __syncthreads();
        const int64_t slot0 = (static_cast<int64_t>(it.a * p.kv_heads + it.g) * p.chunks + it.tok0 / p.chunk) * p.qp + q0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int qi = 8 * nt + 2 * t4 + e;
                if (q0 + qi >= nq) continue;
                float* po = p.o + (slot0 + qi) * D + 16 * warp * MW;
#pragma unroll
                for (int mt = 0; mt < MW; ++mt) {
                    po[16 * mt + g8] = o[mt][nt][e] * kUnshift;
                    po[16 * mt + g8 + 8] = o[mt][nt][2 + e] * kUnshift;
                }
                if (warp == 0 && g8 == 0) {
                    const float4 r = *reinterpret_cast<const float4*>(red + qi * 4);
                    *reinterpret_cast<float2*>(p.ml + (slot0 + qi) * 2) = make_float2(mx[nt][e], ((r.x + r.y) + (r.z + r.w)) * kUnshift);
                }
            }
    }
    if (!live && warp == 0 && lane == 0) {
        *abort_flag = 1;
        atomicOr(p.err, kErrTimeout);
        // let every copy still in flight land before the block exits
        volatile int go_on = 0;
        for (; taken < issued; next()) mbar_wait_bounded(bar + slot, phase, &go_on);
    }
}

// Launches the split kernel of a format (defined once per format).
struct AttendLaunch {
    AttendParams p;
    CUtensorMap map;
    int32_t head_dim;
    int32_t max_q;  // most queries of one sequence per KV head
    int32_t device, sms;
};
cudaError_t launch_attend_q8(const AttendLaunch& a, cudaStream_t s);
cudaError_t launch_attend_f16(const AttendLaunch& a, cudaStream_t s);
cudaError_t launch_attend_bf16(const AttendLaunch& a, cudaStream_t s);

template <int FMT, int D, int NT>
cudaError_t launch_attend_one(const AttendLaunch& a, cudaStream_t s) {
    static_assert(Geo<FMT, D, NT>::smem(kMaxAgents) <= kMaxShared);
    const int bytes = Geo<FMT, D, NT>::smem(a.p.agents);
    static Once once;
    const cudaError_t e = once.allow_shared(attend_partial<FMT, D, NT>, a.device);
    if (e != cudaSuccess) return e;
    // blocks per SM: what the registers were limited for, or what shared memory holds
    int per_sm = (228 * 1024) / (bytes + 1024);
    if (per_sm > Geo<FMT, D, NT>::blocks) per_sm = Geo<FMT, D, NT>::blocks;
    attend_partial<FMT, D, NT><<<a.sms * per_sm, kThreads, bytes, s>>>(a.map, a.p);
    return cudaGetLastError();
}

// Column tiles of 8 queries that an item takes.  D = 64: the fewest items per chunk, and of 3 and 4 column
// tiles the fewer where the items are as many (5 x 24,000 tokens, 4 KV heads: 18 queries 61 us by 3 and 85 by
// 2; 30: 77 by 4, 107 by 3; 48: 110 by 3, 131 by 4, 154 by 6, whose registers leave three blocks an SM;
// 64: 135 by 4, 153 by 3).  D = 256: 2, the most of which two blocks fit an SM (18 queries 212 us, 235 by 3;
// 30: 215, 292 by 4; 48: 283, 408 by 3).
template <int FMT, int D>
cudaError_t launch_attend_dim(const AttendLaunch& a, cudaStream_t s) {
    if (a.max_q <= 8) return launch_attend_one<FMT, D, 1>(a, s);
    if (D == 256 || a.max_q <= 16) return launch_attend_one<FMT, D, 2>(a, s);
    return (a.max_q + 31) / 32 < (a.max_q + 23) / 24 ? launch_attend_one<FMT, D, D == 256 ? 2 : 4>(a, s)
                                                     : launch_attend_one<FMT, D, D == 256 ? 2 : 3>(a, s);
}

}  // namespace kv
}  // namespace qmm
