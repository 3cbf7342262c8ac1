// Attention with a sliding window over the paged cache: the kernel on the 5th-generation tensor cores.
//
// For query (row r of sequence a, head h of KV head g's group) and x_t = scale log2(e) q . k_t:
//   out = sum_t 2^(x_t - M) v_t / l,   l = sum_t 2^(x_t - M),   M = max_t x_t
// over the slots t < n with t >= n - window or t < sinks, n = row_len[r].
// The queries of a sequence and a KV head (rows times heads of the group) lie side by side, 128 of them a tile:
//   S[query][token] = Q K^T     M = 128 queries, N = the tokens of a tile, K = the dims
//   O[query][dim]  += P V       M = 128 queries, N = the dims, K = the tokens
// with S and O in tensor memory.  A softmax thread owns a query: its scores, maximum and sum need no exchange.
// P goes back over S as the second product's A operand, in 16 bits.
// An item is a block's work: a sequence, a KV head and
//   prompts (more than 128 queries a sequence): two tiles of queries, which share each K and V tile;
//   decode steps: one tile of queries, whose tokens' tiles are dealt to two streams by their parity; each stream's
//     softmax weighs both outputs at the end, for half of the dims.
// Either way two streams take turns on the tensor cores (one at head dimension 256, for which tensor memory has no more
// room): one's products run while the other's scores become probabilities.  Tiles have 64 tokens, and scores two buffers:
// the next tile's are there when the softmax is done with one.
// The tiles of an item are those that some of its rows sees: the first ones (sinks), and the window's.  Where few
// items would leave SMs idle, tokens are cut into chunks at fixed places of a sequence, an item each, whose unnormalised
// outputs a second kernel joins.  All choices are made by the plan's dims, so a row's bits do not depend on its company.
//   warp 0      forms the items' records; asks for K tiles (q8_0: as they are stored); it or another one asks for V tiles
//   warps 1, 3  one thread each issues a stream's products
//   warp 2      16-bit pools: zeroes the rows of V that must not count, where some are
//   warps 4 ..  softmax, four a stream
//   q8_0: four more convert K (half a token a thread) and V (a dim a thread) to two fp16 parts whose sum is quant
//               times scale
// A query's reference is its first tile's maximum and moves only when a score passes it by more than 2^kSlack (past kFine: when
// one passes it); each query decides for itself.
//
// What bounds it (times as a loop of calls, window of 4,096 and 48 query heads over 8 unless given):
//   prompts, fp16, 2,048 rows at the end of 23,000 tokens, 206 GFLOP: 217 us, 950 TFLOP/s, 0.49 of a library matmul's rate.
//     A score product of 64 columns takes the tensor cores as long as one of 128 (it reads as much of Q): 1,520 clocks of
//     products per tile and two streams, of the 1,770 that a tile takes; the rest are the items' starts and ends, of which
//     384 items on 152 blocks make 2.53 rounds.
//   decode steps, q8_0, 4 x 23,000 tokens, 3 rows, 35 MB: 45 us (one slot of converted V: 55).  The conversion's chain, 600
//     clocks for a tile's K and 1,150 for its V with the waits for their slots.  Both are two fp16 parts; one for V
//     would halve its products but lose 2^-11 of V.
//   decode steps, bf16, 61 ragged sequences to 4,099, 32 heads over 8 of 64, window 1,024, 113 MB: 47 us, 2.4 TB/s.  A tile's
//     chain of roles (2,100 clocks a stream) and an item's start and end (6,000 of its 24,000 clocks, 16,000 for the first).
//   prompts, q8_0, 4 x 524 rows, window 1,024: 138 us; bf16, 3 x 777 rows, 8 heads over 2 of 256, no window: 52 us.  The
//     first: conversion, and warps that wait for instructions (code that does not run, in the softmax's loop or in other roles,
//     cost it up to 5 %).
// Measured and not taken, for the fp16 prompt: tiles of 128 tokens with one product of 128 columns, whose halves two
// threads take (242 us: one buffer of scores); those threads with a vote on the reference (255 to 263); streams that take
// strict turns (255); 64 scores of a thread kept across the two passes (386: registers spill); V tiles asked for by a warp
// of its own (230).
#pragma once

#include <cuda.h>

#include "qmm_decode.h"
#include "qmm_kv.cuh"

namespace qmm {
namespace window {

using namespace qmm::kv;

constexpr float kShift = 9.f;       // p's power of two ..
constexpr float kSlack = 6.f;       // .. and how far a score may pass its reference: p <= 2^15
constexpr int kTile = 64;           // tokens of a tile
// From 2^22 on fp32's spacing swallows the two, and the product of a score and the scale is off by more than an exponent can
// be (16 from 2^28 on: p would leave 16 bits).  A reference past it is kept as the score that it is, which comes off before the
// scale: the largest one's exponent is 0, and p <= 1.  Below, an exponent is the unrounded product less the reference, which is
// off by 1/8 at most.
constexpr float kFine = 4194304.f;

struct Params {
    const uint8_t* pool;
    const int32_t* table;
    const int32_t* agent_rows;
    const int32_t* row_len;
    const uint16_t* q;
    void* out;
    float* lse;
    float* ml;  // [rows][heads][slots][2]: reference and sum
    float* o;   // [rows][heads][slots][D]
    int* err;
    int64_t q_stride;
    int32_t max_pages, pool_pages, page_shift, page_tokens, heads, kv_heads, group, agents, rows, max_agent_rows, cap;
    int32_t window, sinks, out_type, head_dim;
    int32_t chunk;   // tokens per chunk, a multiple of 128; 0: one item has all of a query's tokens and writes its output
    int32_t slots;   // partials per (row, head)
    uint32_t flip;   // sign bits that a negative scale puts on the queries
    float c2;        // |scale| log2(e), positive
};

struct Launch {
    Params p;
    CUtensorMap map;
    int device, grid;
};

// DEC: decode steps, one tile of queries an item and its tokens dealt to two streams; otherwise prompts.
template <int FMT, int D, bool DEC>
struct Geo {
    static constexpr bool q8 = FMT == QMM_KV_Q8_0;
    static constexpr int streams = D == 256 ? 1 : 2;
    static constexpr int part = kTile * D * 2;                   // bytes of a tile's K or V in 16 bits
    static constexpr int tile = q8 ? 2 * part : part;            // q8_0: high and low parts
    static constexpr int k_slots = D == 64 ? 8 : D == 128 && !q8 ? 4 : 2, v_slots = q8 && !DEC ? 1 : k_slots;
    // Barriers that say that a tile's K or V is there: more of them than slots, since a stream of a decode step waits only for
    // tiles of its own, at most three apart.  Then a barrier's phase before the one waited for is over for sure: V's come
    // in order, and the last own tile's K was asked for after the K of k_told tiles before had been used.
    static constexpr int k_told = k_slots <= 4 ? 8 : 16, v_told = v_slots <= 4 ? 4 : 8;
    static constexpr int raw_slots = q8 ? 2 : 0;                 // pages on their way, K and V
    static constexpr int q_tile = 128 * D * 2;
    static constexpr int soft_warps = 4 * streams, conv_warps = q8 ? 4 : 0;
    // The warp that asks for V tiles: one of its own, in decode steps for which it takes four more (which asks faster: 61
    // ragged sequences at head dimension 64 took 59 us, 71 with one warp for K and V); a prompt's softmax wants their
    // registers (2,048 rows: 216 us, 230 with them).
    static constexpr int more_warps = !q8 && streams == 2 && DEC ? 4 : 0;
    static constexpr int v_warp = q8 ? 2 : streams == 1 ? 3 : DEC ? 4 + soft_warps : 0;
    static constexpr int threads = 32 * (4 + soft_warps + conv_warps + more_warps);
    // tensor memory: S (two buffers a stream), P over it, and O
    static constexpr int col_o = 256;
    // shared memory, after aligning to 1024
    static constexpr int off_v = k_slots * tile;
    static constexpr int off_q = off_v + v_slots * tile;
    static constexpr int off_raw = off_q + (DEC ? 1 : streams) * q_tile;  // K's pages, then V's
    static constexpr int off_ml = off_raw + 2 * raw_slots * kQ8Half;  // [2][128] reference and sum of the streams
    static constexpr int off_item = off_ml + 256 * 8;            // [2] of Record
    static constexpr int off_dv = off_item + 2 * 64;             // q8_0: V's scales, zero where a token must not count: [4][64] fp16
    static constexpr int off_bar = off_dv + (q8 ? 512 : 0);
    static constexpr int bars = k_told + k_slots + 2 * v_slots + v_told + 4 * raw_slots + 2 + 4 + 4 + 2 + 2 + 2 + 2 + 4;
    // tmp[33], abort, tmem, accumulate[2], miss[8] (of V tiles), odd[8][2], miss[16] (of all tiles), raw[2][2]
    static constexpr int off_misc = (off_bar + bars * 8 + 15) / 16 * 16;
    static constexpr int off_seq = (off_misc + 81 * 4 + 15) / 16 * 16;
    static constexpr int smem(int agents) { return 1024 + off_seq + (agents + 1) * 16; }
};

// What the roles need to know of an item.
struct alignas(16) Record {
    int a, g, q0, nq, r0;          // sequence, KV head, first query, the sequence's queries, its first row
    int a0, na, b0, nt;            // tiles a0 .. a0 + na - 1, then b0 ..; nt in all
    int lo, hi, minlen, maxlo;     // first slot of a window, longest and shortest row, the last window's first slot
    int sink_end, chunk, pad;      // first slots that are visible to the longest row
};
__device__ __forceinline__ int tile_at(const Record& it, int i) { return i < it.na ? it.a0 + i : it.b0 + i - it.na; }

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t lead) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// A product from descriptors by their low words (the address is in it) and the high ones.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t a_hi, uint32_t b, uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %6, 0;\n\tmov.b64 a, {%1, %2};\n\tmov.b64 b, {%3, %4};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %5, p;\n\t}" ::"r"(d),
        "r"(a), "r"(a_hi), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t b_hi, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %5, 0;\n\tmov.b64 b, {%2, %3};\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %4, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(b_hi), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void tma_load_hint(void* smem_dst, const void* tmap, int32_t c0, int32_t c1, uint64_t* bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3}], [%4], %5;" ::"r"(smem_u32(smem_dst)),
        "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(c1), "r"(smem_u32(bar)), "l"(policy)
        : "memory");
}
__device__ __forceinline__ uint64_t l2_policy_evict_last() {
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

#define QMM_R32(v, c)                                                                                                   \
    c((v)[0]), c((v)[1]), c((v)[2]), c((v)[3]), c((v)[4]), c((v)[5]), c((v)[6]), c((v)[7]), c((v)[8]), c((v)[9]),         \
        c((v)[10]), c((v)[11]), c((v)[12]), c((v)[13]), c((v)[14]), c((v)[15]), c((v)[16]), c((v)[17]), c((v)[18]),       \
        c((v)[19]), c((v)[20]), c((v)[21]), c((v)[22]), c((v)[23]), c((v)[24]), c((v)[25]), c((v)[26]), c((v)[27]),       \
        c((v)[28]), c((v)[29]), c((v)[30]), c((v)[31])
// 32 consecutive columns of the thread's tensor memory lane (to be waited for with tc_wait_ld).
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float* v) {
#define QMM_OUT(x) "=f"(x)
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : QMM_R32(v, QMM_OUT)
        : "r"(taddr)
        : "memory");
#undef QMM_OUT
}
#undef QMM_R32
__device__ __forceinline__ uint32_t tmem_ld1(uint32_t taddr) {
    uint32_t v;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr) : "memory");
    return v;
}

// Two fp32 numbers at once.
__device__ __forceinline__ uint64_t pair(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void unpair(uint64_t r, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(r)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 32 bytes at once, at any 16-byte boundary.
__device__ __forceinline__ void store32(void* p, bool whole, const uint32_t* w) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]),
                     "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        static_cast<uint4*>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

template <bool BF>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    uint32_t d;
    if constexpr (BF) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(b), "f"(a));
    return d;
}
__device__ __forceinline__ float wide(uint32_t w, bool bf) {
    return bf ? __uint_as_float(w << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(w)));
}
// Bytes 0, 1 (sel 0x4140) or 2, 3 (sel 0x4342) of four int8 already XORed with 0x80, as fp16x2, exact.
__device__ __forceinline__ __half2 i8_to_h2(uint32_t biased, uint32_t sel) {
    return __hadd2(as_h2(prmt(biased, 0x64646464u, sel)), as_h2(0xE480E480u));
}

// Whether sequence a can be attended to.
__device__ __forceinline__ bool sequence_ok(const Params& p, int a) {
    const int r0 = p.agent_rows[a], r1 = p.agent_rows[a + 1];
    return r0 >= 0 && r1 >= r0 && r1 <= p.rows && r1 - r0 <= p.max_agent_rows;
}
// A row's length, 0 if it is out of range.
__device__ __forceinline__ int length_of(const Params& p, int r) {
    const int n = p.row_len[r];
    return n < 0 || n > p.cap ? 0 : n;
}
// Chunks of a row, in its order: those of the first slots, then those of its window that are not among them.
struct Chunks {
    int first, from, end;  // 0 .. first - 1 and from .. end - 1
    __device__ int count() const { return first + max(0, end - from); }
};
__device__ __forceinline__ Chunks chunks_of(const Params& p, int n) {
    Chunks c;
    c.first = (min(p.sinks, n) + p.chunk - 1) / p.chunk;
    c.from = max(c.first, max(0, n - p.window) / p.chunk);
    c.end = (n + p.chunk - 1) / p.chunk;
    return c;
}

// The table of sequences, the same in every block, one more entry at the end; returns the number of items.  With chunks
// seq[a] = (first item, chunks of the first slots, the window's first chunk, first row).  Without, entries are (first
// item, rows, sequence, first row); where blocks have several items, longer sequences come first, and in decode steps
// blocks take items there and back (following()), so that the last round has the shortest: 61 ragged sequences of up to
// 4,099 tokens, 488 items, take 47 us, 57 in the order of the call.  (The ranks are counted, a thread a sequence, up to as
// many as the block has threads.)
// tmp: 33 ints.  qt: queries of an item.  Without chunks also writes the rows that no item has.
__device__ __forceinline__ int form_table(const Params& p, int4* seq, int* tmp, int qt) {
    const int tid = threadIdx.x, n_threads = blockDim.x;
    bool falls = false, gaps = false;
    for (int a = tid; a <= p.agents; a += n_threads) {
        const int r0 = p.agent_rows[a], r1 = a < p.agents ? p.agent_rows[a + 1] : r0;
        const bool ok = a == p.agents || sequence_ok(p, a);
        seq[a] = make_int4(ok ? 0 : -1, 0, INT32_MAX, r0);
        falls |= r1 < r0;
        gaps |= !ok || (a == 0 && r0 > 0) || (a == p.agents && r0 < p.rows);
    }
    falls = __syncthreads_or(falls);
    gaps = __syncthreads_or(gaps || falls);
    if (falls)
        for (int a = tid; a <= p.agents; a += n_threads) seq[a].x = -1;
    if (gaps && blockIdx.x == 0 && tid == 0) atomicOr(p.err, kErrRange);
    auto find = [&](int r) {
        int lo = 0, hi = p.agents;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (seq[mid].w <= r) lo = mid;
            else hi = mid;
        }
        return r < seq[lo].w || r >= seq[lo + 1].w ? -1 : lo;
    };
    __syncthreads();
    if (p.chunk) {
        if (!falls)
            for (int r = tid; r < p.rows; r += n_threads) {
                const int a = find(r), n = length_of(p, r);
                if (n != p.row_len[r] && blockIdx.x == 0) atomicOr(p.err, kErrRange);  // (its sequence may have no item to say so)
                if (a < 0 || n == 0) continue;
                atomicMax(&seq[a].y, n);
                atomicMin(&seq[a].z, max(0, n - p.window));
            }
    } else if (gaps) {
        for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
            const int a = falls ? -1 : find(r);
            if (a >= 0 && seq[a].x >= 0) continue;
            const int size = p.out_type == QMM_TYPE_F32 ? 4 : 2, d = p.head_dim;
            uint32_t* o = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(p.out) + static_cast<int64_t>(r) * p.heads * d * size);
            for (int i = tid; i < p.heads * d * size / 4; i += n_threads) o[i] = 0;
            if (p.lse)
                for (int h = tid; h < p.heads; h += n_threads) p.lse[static_cast<int64_t>(r) * p.heads + h] = -INFINITY;
        }
    }
    __syncthreads();
    int total = 0;
    for (int a0 = 0; a0 < p.agents; a0 += n_threads) {
        const int a = a0 + tid;
        int n = 0, first = 0, from = 0;
        if (a < p.agents) {
            const int4 s = seq[a];
            const int nr = seq[a + 1].w - s.w;
            if (s.x >= 0 && nr > 0) {
                int chunks = 1;
                if (p.chunk) {
                    first = (min(p.sinks, s.y) + p.chunk - 1) / p.chunk;
                    from = max(first, s.z / p.chunk);
                    chunks = s.y ? first + max(0, (s.y + p.chunk - 1) / p.chunk - from) : 0;
                }
                n = chunks * p.kv_heads * ((nr * p.group + qt - 1) / qt);
            }
        }
        int sum;
        const int at = block_exclusive(n, tmp, &sum);
        if (a < p.agents) {
            if (p.chunk) seq[a].x = total + at, seq[a].y = first, seq[a].z = from;
            else seq[a].x = total + at, seq[a].y = n, seq[a].z = a;
        }
        total += sum;
    }
    if (tid == 0) seq[p.agents].x = total;
    __syncthreads();
    if (p.chunk) return total;
    const bool order = total > static_cast<int>(gridDim.x) && p.agents <= n_threads;
    auto rows_of = [&](int a) { return seq[a + 1].w - seq[a].w; };
    if (order) {
        int4 mine = make_int4(0, 0, tid, 0);
        int at = 0;
        if (tid < p.agents) {
            mine = seq[tid];
            const int nr = rows_of(tid), n = mine.y ? length_of(p, mine.w + nr - 1) : 0;  // (the last row is the longest, as a rule)
            mine.x = min(n, p.window + p.sinks);
            mine.y = nr;
        }
        __syncthreads();
        if (tid < p.agents) seq[tid].x = mine.x;
        __syncthreads();
        int rank = 0;
        if (tid < p.agents) {
            for (int b = 0; b < p.agents; ++b) {
                const int2 s = *reinterpret_cast<const int2*>(seq + b);  // (its tokens, its items)
                const bool before = s.x > mine.x || (s.x == mine.x && b < tid);
                rank += before;
                at += before ? s.y : 0;
            }
        }
        __syncthreads();
        if (tid < p.agents) seq[rank] = make_int4(at, mine.y, tid, mine.w);
    } else {
        for (int a = tid; a < p.agents; a += n_threads) seq[a].y = rows_of(a);
    }
    __syncthreads();
    return total;
}

// The record of an item, by a warp.
__device__ __forceinline__ Record record_of(const Params& p, const int4* seq, int item, int qt) {
    const int lane = threadIdx.x & 31;
    int lo = 0, hi = p.agents;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (seq[mid].x <= item) lo = mid;
        else hi = mid;
    }
    const int4 s = seq[lo];
    Record it;
    it.a = p.chunk ? lo : s.z;
    it.r0 = s.w;
    it.nq = (p.chunk ? seq[lo + 1].w - s.w : s.y) * p.group;
    const int tiles = (it.nq + qt - 1) / qt;
    int rest = item - s.x;
    it.q0 = rest % tiles * qt;
    rest /= tiles;
    it.g = rest % p.kv_heads;
    rest /= p.kv_heads;
    it.chunk = p.chunk ? (rest < s.y ? rest : s.z + rest - s.y) : 0;
    it.pad = 0;
    // the item's rows
    const int ra = it.r0 + it.q0 / p.group, rb = it.r0 + (min(it.q0 + qt, it.nq) - 1) / p.group;
    int maxlen = 0, minlen = INT32_MAX, minlo = INT32_MAX, maxlo = 0;
    bool bad = false;
    for (int r = ra + lane; r <= rb; r += 32) {
        const int n = length_of(p, r);
        bad |= n != p.row_len[r];
        maxlen = max(maxlen, n);
        minlen = min(minlen, n);
        if (n > 0) {
            minlo = min(minlo, max(0, n - p.window));
            maxlo = max(maxlo, max(0, n - p.window));
        }
    }
    if (bad) atomicOr(p.err, kErrRange);
    it.hi = __reduce_max_sync(0xffffffffu, maxlen);
    it.minlen = __reduce_min_sync(0xffffffffu, minlen);
    it.lo = __reduce_min_sync(0xffffffffu, minlo);
    it.maxlo = __reduce_max_sync(0xffffffffu, maxlo);
    it.sink_end = min(p.sinks, it.hi);
    const int c0 = p.chunk ? it.chunk * (p.chunk / kTile) : 0, c1 = p.chunk ? c0 + p.chunk / kTile : INT32_MAX;
    const int end = min((it.hi + kTile - 1) / kTile, c1);
    it.a0 = c0;
    it.na = max(0, min((it.sink_end + kTile - 1) / kTile, end) - c0);
    it.b0 = max(it.lo / kTile, c0 + it.na);
    it.nt = it.hi ? it.na + max(0, end - it.b0) : 0;
    return it;
}

// Marked tokens of a tile, whose V is not finite, added to the outputs of the queries that see them: p as the products
// take it, V from memory.  (Rare; a function of its own costs the loop around it no registers.)
template <int FMT, int D>
__device__ __noinline__ void add_odd(const Params& p, int a, int g, int t0, const uint32_t* odd, uint32_t ocol, uint32_t pcol, int len,
                                     int from, int first, bool fresh) {
    constexpr bool BF = FMT == QMM_KV_BF16;
#pragma unroll 1
    for (int c = 0; c < D; c += 8) {
        uint32_t o[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) o[j] = fresh ? 0u : tmem_ld1(ocol + c + j);
        tc_wait_ld();
#pragma unroll 1
        for (int j = 0; j < kTile; ++j) {
            if (!((odd[j & 1] >> (j >> 1)) & 1)) continue;
            const uint32_t both = tmem_ld1(pcol + j / 2);
            tc_wait_ld();
            const float pr = wide(j & 1 ? both >> 16 : both & 0xFFFFu, BF);
            const int tok = t0 + j, sl = tok & (p.page_tokens - 1);
            const bool sees = tok < len && (tok >= from || tok < first);
            const int pg = p.table[static_cast<int64_t>(a) * p.max_pages + (tok >> p.page_shift)];  // (checked: it is not missing)
            const int64_t rec = static_cast<int64_t>(pg) * p.kv_heads + g;
#pragma unroll
            for (int d = 0; d < 8; ++d) {
                float y;
                if constexpr (FMT == QMM_KV_Q8_0) {
                    const uint8_t* b = p.pool + rec * kQ8Rec + kQ8Half;
                    y = static_cast<float>(static_cast<int8_t>(b[(c + d) * 64 + sl])) *
                        __half2float(*reinterpret_cast<const __half*>(b + 8192 + (((c + d) >> 5) * 64 + sl) * 2));
                    const float hi = __half2float(__float2half_rn(y));  // (the two parts that the products take)
                    y = hi + __half2float(__float2half_rn(y - hi));
                } else {
                    y = wide(reinterpret_cast<const uint16_t*>(p.pool)[((rec * 2 + 1) * p.page_tokens + sl) * D + c + d], BF);
                }
                if (sees) o[d] = __float_as_uint(fmaf(pr, y, __uint_as_float(o[d])));
            }
        }
        tmem_st8(ocol + c, o);
    }
    tc_wait_st();
}

template <int FMT, int D, bool DEC>
__global__ void __launch_bounds__(Geo<FMT, D, DEC>::threads, 1)
    attend_window_tc(const __grid_constant__ CUtensorMap map, const __grid_constant__ Params p) {
    using G = Geo<FMT, D, DEC>;
    constexpr bool BF = FMT == QMM_KV_BF16;
    constexpr int NS = G::streams;
    extern __shared__ uint8_t sm_raw[];
    griddep_launch_dependents();  // the joining kernel waits for this grid's end before it reads
    uint8_t* sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
    float2* ml_sm = reinterpret_cast<float2*>(sm + G::off_ml);
    Record* item_sm = reinterpret_cast<Record*>(sm + G::off_item);
    uint64_t* kfull = reinterpret_cast<uint64_t*>(sm + G::off_bar);
    uint64_t *kempty = kfull + G::k_told, *vfull = kempty + G::k_slots, *vempty = vfull + G::v_slots, *vready = vempty + G::v_slots;
    uint64_t *rfull = vready + G::v_told, *rempty = rfull + 2 * G::raw_slots;  // (K's, then V's)
    uint64_t *qfull = rempty + 2 * G::raw_slots, *sfull = qfull + 2, *pfull = sfull + 4, *odone = pfull + 4, *ofin = odone + 2;
    uint64_t *ifull = ofin + 2, *iempty = ifull + 2, *mfree = iempty + 2, *mfull = mfree + 1, *drained = mfull + 1;
    int* tmp = reinterpret_cast<int*>(sm + G::off_misc);
    volatile int* abort_flag = tmp + 33;
    uint32_t* tmem_sm = reinterpret_cast<uint32_t*>(tmp + 34);
    volatile int* accum_sm = tmp + 35;                                          // [2] O holds something before the first product
    volatile int* miss_sm = tmp + 37;                                           // [8] a V tile's pieces that are outside the pool
    volatile uint32_t* odd_sm = reinterpret_cast<uint32_t*>(tmp + 45);          // [8][2] tokens that are taken query by query: even ones, odd ones
    volatile int* kmiss_sm = tmp + 61;                                          // [16] miss of the last 16 tiles (more than are under way)
    volatile int* raw_sm = tmp + 77;                                            // q8_0, [2][2]: a page's number, -1 not needed, -2 outside the pool
    int4* seq = reinterpret_cast<int4*>(sm + G::off_seq);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int qt = NS == 2 && !DEC ? 256 : 128;

    if (tid == 0) {
        const int users = NS == 2 && !DEC ? 2 : 1;  // streams that see a tile
        for (int i = 0; i < G::k_told; ++i) mbar_init(kfull + i, G::q8 ? 4 : 1);
        for (int i = 0; i < G::v_told; ++i) mbar_init(vready + i, G::q8 ? 4 : 1);
        for (int i = 0; i < G::k_slots; ++i) mbar_init(kempty + i, users);
        for (int i = 0; i < G::v_slots; ++i) mbar_init(vfull + i, 1), mbar_init(vempty + i, users);
        for (int i = 0; i < 2; ++i) {
            mbar_init(qfull + i, 4);
            mbar_init(odone + i, 1);
            mbar_init(ofin + i, 1);
            mbar_init(ifull + i, 1);
            mbar_init(iempty + i, (G::v_warp != 0) + NS + (G::q8 ? G::conv_warps : 1) + G::soft_warps);
        }
        for (int i = 0; i < 4; ++i) mbar_init(sfull + i, 1), mbar_init(pfull + i, 4);
        for (int i = 0; i < 2 * G::raw_slots; ++i) mbar_init(rfull + i, 1), mbar_init(rempty + i, 4);
        mbar_init(mfree, G::soft_warps);
        mbar_init(mfull, G::soft_warps);
        mbar_init(drained, 1);
        mbar_init(drained + 1, 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc(tmem_sm, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    const int total = form_table(p, seq, tmp, qt);
    tc_fence_after();
    const uint32_t tmem = *tmem_sm;

    // A wait of one of the roles, with one answer for the warp.  Once one has run out, everything ends.
    bool live = true;
    auto await = [&](uint64_t* b, uint32_t parity) {
        if (live && !mbar_wait_bounded(b, parity, abort_flag)) {
            live = false;
            *abort_flag = 1;
        }
        live = __all_sync(0xffffffffu, live);
    };
    int k = 0;  // items so far
    // the block's next item, k being the items up to this one: there and back in the table's order; in turns for chunks and
    // prompts, whose items differ less (4 x 524 rows of q8_0: 2 % more there and back)
    auto following = [&](int item) { return p.chunk || !DEC ? item + static_cast<int>(gridDim.x) : 2 * k * static_cast<int>(gridDim.x) - 1 - item; };
    // the next item's record
    auto next_record = [&]() -> Record {
        await(ifull + (k & 1), (k >> 1) & 1);
        const Record it = item_sm[k & 1];
        __syncwarp();
        if (lane == 0) mbar_arrive(iempty + (k & 1));
        ++k;
        return it;
    };
    // whether some row does not see some token of a tile
    auto edge = [&](const Record& it, int t0) { return !(t0 + kTile <= it.minlen && (t0 >= it.maxlo || t0 + kTile <= p.sinks)); };
    // a token that no row of the item sees
    auto gone = [&](const Record& it, int t) { return t >= it.hi || (t < it.lo && t >= it.sink_end); };
    const int piece_rows = min(kTile, p.page_tokens), piece_shift = 31 - __clz(piece_rows);
    // lane i: the page of piece i of a tile, -1 if nobody needs it, -2 if it is outside the pool: an error if some row sees it,
    // which the row's softmax finds (between windows that lie apart entries may hold anything)
    auto page_of = [&](const Record& it, int t0) {
        int pg = -1;
        const int t = t0 + lane * piece_rows;
        if (lane * piece_rows < kTile && t < it.hi && (t + piece_rows > it.lo || t < it.sink_end)) {
            pg = p.table[static_cast<int64_t>(it.a) * p.max_pages + (t >> p.page_shift)];
            if (pg < 0 || pg >= p.pool_pages) pg = -2;
        }
        return pg;
    };

    // Registers go where the scores are (the shares add up to what the block was launched with, or less:
    // 256 * 200 + 128 * 104 = 384 * 168, with four more warps 256 * 200 + 256 * 56 = 512 * 128; q8_0 256 * 168 + 256 * 80 <= 512 * 128).
    if (warp < 4 || (G::more_warps && warp >= 4 + G::soft_warps)) {
    if constexpr (NS == 2) setmaxnreg_dec<G::q8 ? 80 : G::more_warps ? 56 : 104>();
    if (warp == 0 || warp == G::v_warp) {
        // ---------------------------------------------------------------- records, and K tiles; V tiles
        constexpr int kSlots = G::q8 ? G::raw_slots : G::k_slots;
        static_assert(G::q8 || G::k_slots == G::v_slots);
        const bool does_k = warp == 0, does_v = warp == G::v_warp;
        // the barrier that says that tile t's K (h = 0) or V is there
        auto told = [&](int h, int t) { return G::q8 ? rfull + h * kSlots + t % kSlots : h ? vfull + t % kSlots : kfull + t % G::k_told; };
        // (a prompt's tiles are read by other blocks as well)
        const uint64_t policy = DEC ? l2_policy_evict_first() : l2_policy_evict_last();
        auto ask = [&](int h, int g, int t0, int mine, int t) {  // `mine`: pages, lanes by piece
            const uint32_t there = __ballot_sync(0xffffffffu, mine >= 0);
            const int miss = static_cast<int>(__ballot_sync(0xffffffffu, mine == -2));
            const int s = t % kSlots, round = t / kSlots;
            if (round > 0) await((G::q8 ? rempty + h * kSlots : h ? vempty : kempty) + s, (round - 1) & 1);
            if (!live) return;
            uint64_t* bar = told(h, t);
            if (lane == 0) {
                if constexpr (G::q8) raw_sm[2 * h + s] = mine;
                else if (h) miss_sm[s] = miss;
                else kmiss_sm[t & 15] = miss;
                if (!there) mbar_arrive(bar);
                else mbar_arrive_expect_tx(bar, G::q8 ? kQ8Half : __popc(there) * piece_rows * D * 2);
            }
            __syncwarp();
            if (mine >= 0) {
                fence_proxy_async_smem();  // the slot's generic accesses, before the copies
                if constexpr (G::q8) {
                    bulk_g2s(sm + G::off_raw + (h * kSlots + s) * kQ8Half, p.pool + (static_cast<int64_t>(mine) * p.kv_heads + g) * kQ8Rec + h * kQ8Half,
                             kQ8Half, bar, policy);
                } else {
                    const int y = ((mine * p.kv_heads + g) * 2 + h) * p.page_tokens + ((t0 + lane * piece_rows) & (p.page_tokens - 1));
#pragma unroll
                    for (int x = 0; x < D / 64; ++x)
                        tma_load_hint(sm + (h ? G::off_v : 0) + s * G::tile + x * kTile * 128 + lane * piece_rows * 128, &map, 64 * x, y, bar, policy);
                }
            }
            __syncwarp();
        };
        // (a warp that asks for both: V a tile behind K, whose slots come free first, but not behind an item without tiles,
        // since the record after that takes the place of one that waits for this V)
        int t = 0, v_page = -1, v_t0 = 0, v_g = 0;
        bool behind = false;
        auto ask_behind = [&] {
            if (behind && live) ask(1, v_g, v_t0, v_page, t - 1);
            behind = false;
        };
        for (int item = blockIdx.x; item < total && live; item = following(item)) {
            Record it;
            if (!does_k) {
                it = next_record();
            } else {
                it = record_of(p, seq, item, qt);
                if (k > 1) await(iempty + (k & 1), ((k >> 1) - 1) & 1);
                if (!live) break;
                if (lane == 0) {
                    item_sm[k & 1] = it;
                    mbar_arrive(ifull + (k & 1));
                }
                ++k;
            }
            if (does_k && does_v && it.nt == 0) ask_behind();
            int next = it.nt > 0 ? page_of(it, tile_at(it, 0) * kTile) : -1;
            for (int i = 0; i < it.nt && live; ++i, ++t) {
                const int t0 = tile_at(it, i) * kTile, mine = next;
                if (i + 1 < it.nt) next = page_of(it, tile_at(it, i + 1) * kTile);
                if (does_k && does_v) {
                    ask_behind();
                    ask(0, it.g, t0, mine, t);
                    v_page = mine, v_t0 = t0, v_g = it.g;
                    behind = true;
                } else {
                    ask(does_v, it.g, t0, mine, t);
                }
            }
        }
        ask_behind();
        if (!live && lane == 0) {
            // let every copy still in flight land before the block exits: the last of each slot
            volatile int go_on = 0;
            for (int h = does_k ? 0 : 1; h <= (does_v ? 1 : 0); ++h)
                for (int i = max(0, t - kSlots - 1); i <= t; ++i)
                    mbar_wait_bounded(told(h, i), (i / (!G::q8 && !h ? G::k_told : kSlots)) & 1, &go_on, 100000000ull);
        }
    } else if (warp == 1 || (warp == 3 && NS == 2)) {
        // ---------------------------------------------------------------- a stream's products
        // One thread: its waits cost 60 clocks where a warp's with a vote take 100, and tcgen05.commit speaks for the products
        // of its thread.  It is bound by its own instructions (some 4 clocks each), so both streams have one.
        constexpr uint32_t kType = BF ? (1u << 7) | (1u << 10) : 0u;
        constexpr uint32_t kIdescS = idesc_f16_f32(128, kTile) | kType;
        constexpr uint32_t kIdescO = idesc_f16_f32(128, D) | kType | (G::q8 ? 0u : 1u << 16);  // (16-bit pools: V by dims)
        constexpr uint32_t kHi = static_cast<uint32_t>(uint64_t{1024 >> 4} | uint64_t{1} << 14 | uint64_t{2} << 29);  // of every descriptor here
        const int s = warp == 3;
        if (elect_one()) {
            auto wait = [&](uint64_t* b, uint32_t parity) {
                if (!mbar_try_wait(b, parity) && !(live && mbar_wait_bounded(b, parity, abort_flag))) {
                    live = false;
                    *abort_flag = 1;
                }
            };
            const uint32_t qd = static_cast<uint32_t>(smem_desc_sw128(smem_u32(sm + G::off_q + (DEC ? 0 : s * G::q_tile))));
            const uint32_t kd = static_cast<uint32_t>(smem_desc_sw128(smem_u32(sm)));
            const uint32_t vd = static_cast<uint32_t>(G::q8 ? smem_desc_sw128(smem_u32(sm + G::off_v)) : desc_mn(smem_u32(sm + G::off_v), kTile * 128));
            const uint32_t col = tmem + s * 2 * kTile, o = tmem + G::col_o + s * D;
            uint64_t *sf = sfull + 2 * s, *pf = pfull + 2 * s;
            const bool shares = NS == 2 && !DEC;  // both streams see every tile
            int t = 0, n = 0, m = 0;  // tiles so far; of this stream: scores asked for, and P V
            int pend = -1;            // the tile whose P V is still to come
            uint32_t acc = 0;
            // Products of one thread run in the order in which they are asked for: S may go over a P whose product has been.
            auto product_pv = [&] {
                const int vs = pend % G::v_slots;
                const uint32_t b0 = vd + (vs * G::tile >> 4);
                wait(vready + pend % G::v_told, (pend / G::v_told) & 1);
                const int x = m & 1;
                wait(pf + x, (m >> 1) & 1);
                if (!live) return;
                tc_fence_after();
                if (!acc) acc = accum_sm[s] != 0;
#pragma unroll
                for (int part = 0; part < (G::q8 ? 2 : 1); ++part)
#pragma unroll
                    for (int ks = 0; ks < kTile / 16; ++ks) {
                        mma_ts(o, col + x * kTile + 8 * ks, b0 + ((G::q8 ? part * G::part + ks * 32 : ks * 2048) >> 4), kHi, kIdescO, acc);
                        acc = 1;
                    }
                tc_commit(vempty + vs);
                tc_commit(odone + s);
                ++m;
                pend = -1;
            };
            auto product_s = [&] {
                const int ksl = t % G::k_slots, x = n & 1;
                const uint32_t bk = kd + (ksl * G::tile >> 4);
#pragma unroll
                for (int part = 0; part < (G::q8 ? 2 : 1); ++part)
#pragma unroll
                    for (int ks = 0; ks < D / 16; ++ks)
                        mma_ss(col + x * kTile, qd + (((ks >> 2) * (128 * 128) + (ks & 3) * 32) >> 4), kHi,
                               bk + ((part * G::part + (ks >> 2) * (kTile * 128) + (ks & 3) * 32) >> 4), kHi, kIdescS, part + ks > 0);
                tc_commit(sf + x);
                tc_commit(kempty + ksl);
                ++n;
            };
            int both = 0;  // items of this stream's so far
            for (int item = blockIdx.x; item < total && live; ++k, item = following(item)) {
                wait(ifull + (k & 1), (k >> 1) & 1);
                if (!live) break;
                const Record it = item_sm[k & 1];
                mbar_arrive(iempty + (k & 1));
                const int nt = it.nt;
                if (shares && s == 1 && it.nq - it.q0 <= 128) {  // no queries for this stream: the slots go back without it
                    for (int i = 0; i < nt && live; ++i, ++t) {
                        wait(kfull + t % G::k_told, (t / G::k_told) & 1);
                        wait(vready + t % G::v_told, (t / G::v_told) & 1);
                        if (!live) break;
                        mbar_arrive(kempty + t % G::k_slots);
                        mbar_arrive(vempty + t % G::v_slots);
                    }
                    continue;
                }
                // (decode steps: the first stream's queries are the second's as well)
                wait(qfull + (DEC ? 0 : s), (DEC ? k : both) & 1);
                ++both;
                bool begun = false;
                for (int i = 0; i < nt && live; ++i, ++t) {
                    if (NS == 2 && DEC && (tile_at(it, i) & 1) != s) continue;
                    wait(kfull + t % G::k_told, (t / G::k_told) & 1);
                    if (!live) break;
                    tc_fence_after();
                    product_s();
                    if (pend >= 0) product_pv();
                    if (!begun) acc = 0;
                    pend = t;
                    begun = true;
                }
                if (pend >= 0 && live) product_pv();
                if (begun && live) tc_commit(ofin + s);
            }
            // every product issued has finished before the tensor memory is released
            tc_commit(drained + s);
            volatile int go_on = 0;
            mbar_wait_bounded(drained + s, 0, &go_on, 10000000000ull);
        }
        __syncwarp();
    } else if (warp == 2 && !G::q8) {
        // ---------------------------------------------------------------- V's rows that must not count
        // Slots that nobody sees hold anything (and so do those of missing pages): zero.  One that some rows see
        // and whose V is not finite is marked, to be added query by query, and zero in the product.
        int t = 0;
        for (int item = blockIdx.x; item < total && live; item = following(item)) {
            const Record it = next_record();
            for (int i = 0; i < it.nt && live; ++i, ++t) {
                const int t0 = tile_at(it, i) * kTile, vs = t % G::v_slots;
                await(vfull + vs, (t / G::v_slots) & 1);
                if (!live) break;
                const int miss = miss_sm[vs];
                if (miss != 0 || edge(it, t0)) {
                    uint8_t* vt = sm + G::off_v + vs * G::tile;
#pragma unroll 1
                    for (int j = 0; j < 2; ++j) {
                        const int row = 2 * lane + j, tok = t0 + row;
                        bool zero = gone(it, tok) || ((miss >> (row >> piece_shift)) & 1), odd = false;
                        if (!zero && !(tok < it.minlen && (tok >= it.maxlo || tok < p.sinks))) {
                            constexpr uint32_t ex = BF ? 0x7F80u : 0x7C00u;
                            auto bad = [&](uint32_t w) { return (w & ex) == ex || ((w >> 16) & ex) == ex; };
#pragma unroll 1
                            for (int x = 0; x < D / 64; ++x)
#pragma unroll
                                for (int c = 0; c < 8; ++c) {
                                    const uint4 v = *reinterpret_cast<const uint4*>(vt + x * kTile * 128 + row * 128 + 16 * ((c + lane) & 7));
                                    odd |= bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w);
                                }
                        }
                        if (zero || odd) {
#pragma unroll 1
                            for (int x = 0; x < D / 64; ++x)
#pragma unroll
                                for (int c = 0; c < 8; ++c)
                                    *reinterpret_cast<uint4*>(vt + x * kTile * 128 + row * 128 + 16 * ((c + lane) & 7)) = make_uint4(0, 0, 0, 0);
                        }
                        const uint32_t word = __ballot_sync(0xffffffffu, odd);
                        if (lane == 0) odd_sm[t % G::v_told * 2 + j] = word;
                    }
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(vready + t % G::v_told);
            }
        }
    }
    } else if (warp < 4 + G::soft_warps) {
        if constexpr (NS == 2) setmaxnreg_inc<G::q8 ? 168 : 200>();
        // ---------------------------------------------------------------- softmax: a query per thread
        const int s = (warp - 4) >> 2, me = tid & 127;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * (warp & 3)) << 16);
        const uint32_t ocol = lanes + G::col_o + s * D;
        int tiles = 0;  // all tiles so far
        int n = 0;      // the stream's
        int merges = 0, fins = 0;
        for (int item = blockIdx.x; item < total; item = following(item)) {
            // (the record stays until the item's end, where what the loop has no registers for is read again)
            await(ifull + (k & 1), (k >> 1) & 1);
            if (NS == 2 && DEC && merges > 0) await(mfree, (merges - 1) & 1);  // (the last item's outputs are read)
            if (!live) break;
            // (read as it is needed: the scores take most registers)
            const volatile Record& it = item_sm[k & 1];
            const int nt = it.nt, minlen = it.minlen, maxlo = it.maxlo;
            auto edge_at = [&](int t) { return !(t + kTile <= minlen && (t >= maxlo || t + kTile <= p.sinks)); };
            auto release = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(iempty + (k & 1));
                ++k;
            };
            const int c0 = it.q0 + (NS == 2 && !DEC ? 128 * s : 0), q = c0 + me;
            if (NS == 2 && !DEC && s == 1 && c0 >= it.nq) {  // the item has one tile of queries
                tiles += nt;
                release();
                continue;
            }
            const bool idle = c0 + 32 * (warp & 3) >= it.nq;  // no query of the warp's
            const bool valid = q < it.nq;
            const int row = it.r0 + (valid ? q / p.group : 0), head = it.g * p.group + (valid ? q % p.group : 0);
            const int len = valid ? length_of(p, row) : 0, from = max(0, len - p.window), first = min(p.sinks, len);
            const int nq = it.nq;
            if (s == 0 || !DEC) {  // the queries, swizzled as the copies do: D / 8 lanes a row
                constexpr int L = D / 8 < 32 ? D / 8 : 32, R = 32 / L;  // lanes of a row, rows at once
                const int c = lane % L;
                uint8_t* dst = sm + G::off_q + s * G::q_tile + (c >> 3) * (128 * 128);
                const int64_t src = row * p.q_stride + static_cast<int64_t>(head) * D;
                constexpr int kMost = G::q8 ? 8 : 16, kLoads = 32 / R < kMost ? 32 / R : kMost;  // (on their way at once)
#pragma unroll 1
                for (int i0 = 0; i0 < 32; i0 += kLoads * R) {
                    uint4 v[kLoads];
#pragma unroll
                    for (int j = 0; j < kLoads; ++j) {
                        const int i = i0 + j * R + lane / L;
                        const int64_t o = __shfl_sync(0xffffffffu, src, i);
                        v[j] = c0 + 32 * (warp & 3) + i < nq ? *reinterpret_cast<const uint4*>(p.q + o + 8 * c) : make_uint4(0, 0, 0, 0);
                    }
#pragma unroll
                    for (int j = 0; j < kLoads; ++j) {
                        const int row = 32 * (warp & 3) + i0 + j * R + lane / L;
                        v[j].x ^= p.flip, v[j].y ^= p.flip, v[j].z ^= p.flip, v[j].w ^= p.flip;
                        *reinterpret_cast<uint4*>(dst + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = v[j];
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(qfull + s);
            }
            // Sum, reference and slack, what is added to the scaled scores.  A reference past kFine: ref is the score that it is,
            // shift 0, and lim stays -infinity, so that each tile goes the way of one that moves its reference, where ref comes off
            // the scores (others do not pay for the case: 217 us for the 2,048-row prompt either way, 229 with a test in each tile).
            float l = 0.f, lim = -INFINITY, shift = 0.f, ref = 0.f;
            auto level = [&] { return ref != 0.f ? ref * p.c2 : -shift; };  // what the exponents are relative to
            bool fresh = true;                           // O holds nothing yet
            const int na = it.na;
            int tile = na ? it.a0 : it.b0;
            for (int i = 0; i < nt; ++i, ++tile, ++tiles) {
                if (i == na && i) tile = it.b0;
                const int t0 = tile * kTile;
                if (NS == 2 && DEC && (tile & 1) != s) continue;
                const int x = 2 * s + (n & 1);
                const uint32_t scol = lanes + x * kTile;  // S, and P over it
                await(sfull + x, (n >> 1) & 1);
                const bool some = edge_at(t0);
                const int vi = tiles % G::v_told;
                if (some) await(vready + vi, (tiles / G::v_told) & 1);  // (which tokens' V is not finite)
                if (!live) break;
                float v[kTile], top = -INFINITY, m = -INFINITY;  // scores, the largest, and the same times the scale
                const int miss = kmiss_sm[tiles & 15];
                if (!idle) {
                    tc_fence_after();
#pragma unroll
                    for (int i = 0; i < kTile; i += 32) tmem_ld32(scol + i, v + i);
                    tc_wait_ld();
                    if (some || miss) {
                        // the tokens that the row sees, as bits; a missing piece is 16 tokens at least
                        auto below = [](int j) { return j <= 0 ? 0u : j >= 32 ? ~0u : (1u << j) - 1; };
                        uint32_t lost = 0;  // .. and those among them whose page is missing
#pragma unroll
                        for (int i = 0; i < kTile; i += 32) {
                            const int t = t0 + i;
                            uint32_t sees = below(len - t) & (~below(from - t) | below(first - t));
                            const uint32_t all = sees;
                            if ((miss >> (i >> piece_shift)) & 1) sees &= 0xFFFF0000u;
                            if ((miss >> ((i + 16) >> piece_shift)) & 1) sees &= 0xFFFFu;
                            lost |= sees ^ all;
#pragma unroll
                            for (int j = 0; j < 32; ++j)
                                if (!(sees & (1u << j))) v[i + j] = -INFINITY;
                        }
                        if (lost) atomicOr(p.err, kErrPage);
                    }
                    float m8[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) m8[j] = -INFINITY;
#pragma unroll
                    for (int j = 0; j < kTile; j += 16)
#pragma unroll
                        for (int i = 0; i < 8; ++i) m8[i] = fmaxf(m8[i], fmaxf(v[j + i], v[j + i + 8]));
                    // (a NaN is no maximum)
                    top = fmaxf(fmaxf(fmaxf(m8[0], m8[1]), fmaxf(m8[2], m8[3])), fmaxf(fmaxf(m8[4], m8[5]), fmaxf(m8[6], m8[7])));
                    m = top * p.c2;
                }
                if (__any_sync(0xffffffffu, m > lim)) {
                    const bool passed = ref != 0.f ? top > ref : m > lim;
                    float alpha = 1.f;
                    if (passed) {
                        const bool fine = fabsf(m) < kFine, had = lim > -INFINITY || ref != 0.f;
                        alpha = had ? ex2(level() - (fine ? m - kShift : m)) : 0.f;
                        shift = fine ? kShift - m : 0.f;
                        ref = fine ? 0.f : top;
                        lim = fine ? m + kSlack : -INFINITY;
                        l *= alpha;
                    }
                    if (__any_sync(0xffffffffu, ref != 0.f)) {
                        const uint64_t r2 = pair(-ref, -ref);
#pragma unroll
                        for (int j = 0; j < kTile; j += 2) unpair(add2(pair(v[j], v[j + 1]), r2), v[j], v[j + 1]);
                    }
                    if (!fresh) {
                        // (the last product may be under way; the one before was over before these scores were asked for)
                        await(odone + s, (n - 1) & 1);
                        if (!live) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {  // (rare, and the scores hold most registers)
                            uint32_t o[16];
                            tmem_ld16(ocol + c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
                            tmem_st16(ocol + c, o);
                        }
                    }
                }
                // tokens whose V is not finite
                uint32_t odd = 0;
                if (some) {
#pragma unroll
                    for (int j = 0; j < 2; ++j) odd |= odd_sm[vi * 2 + j];
                }
                if (fresh && me == 0) accum_sm[s] = odd != 0;
                if (!idle) {
                    uint64_t sum[2] = {0, 0};  // pairs of fp32
                    const uint64_t c2 = pair(p.c2, p.c2), off = pair(shift, shift);
#pragma unroll
                    for (int i = 0; i < kTile; i += 32) {
                        const int c = 32 - i;  // (the upper scores first)
                        const float* u = v + c;
                        uint32_t w[16];
#pragma unroll
                        for (int g = 0; g < 32; g += 8) {
                            float e[8];
#pragma unroll
                            for (int j = 0; j < 8; j += 2) unpair(fma2(pair(u[g + j], u[g + j + 1]), c2, off), e[j], e[j + 1]);
#pragma unroll
                            for (int j = 0; j < 8; ++j) e[j] = ex2(e[j]);
#pragma unroll
                            for (int j = 0; j < 8; j += 2) {
                                sum[(j >> 1) & 1] = add2(sum[(j >> 1) & 1], pair(e[j], e[j + 1]));
                                // (one rounding to 16 bits, 2^-11 or bf16's 2^-8 of a probability, as V's own elements have: a second part
                                // would double the second product, half of the tensor cores' time in prompts; the sum is of fp32)
                                w[(g + j) / 2] = pack2<BF>(e[j], e[j + 1]);
                            }
                        }
                        tmem_st16(scol + c / 2, w);
                    }
                    float s0, s1;
                    unpair(add2(sum[0], sum[1]), s0, s1);
                    l += s0 + s1;
                    tc_wait_st();
                }
                if (odd) {  // to those that see them
                    if (!fresh) await(odone + s, (n - 1) & 1);
                    if (!live) break;
                    tc_fence_before();
                    tc_fence_after();
                    add_odd<FMT, D>(p, it.a, it.g, t0, const_cast<const uint32_t*>(odd_sm) + vi * 2, ocol, scol, len, from, first, fresh);
                }
                fresh = false;
                ++n;
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(pfull + x);
            }
            // (the item's last product; odone may be two phases behind here)
            if (!fresh) await(ofin + s, fins++ & 1);
            if (!live) break;
            tc_fence_after();

            // ---- what became of the item
            float base = level();
            float w0 = 1.f, w1 = 0.f;  // the streams' weights
            const bool merge = NS == 2 && DEC;
            if (merge) {  // the streams' softmaxes have the same lanes of tensor memory: each takes half of both's dims
                ml_sm[128 * s + me] = make_float2(base, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(mfull);
                await(mfull, merges++ & 1);
                tc_fence_after();
                const float2 a = ml_sm[me], b = ml_sm[128 + me];
                // (a sum of 0: nothing seen, and nothing of its outputs counts)
                const float top = a.y == 0.f ? b.x : b.y == 0.f ? a.x : fmaxf(a.x, b.x);
                w0 = a.y == 0.f ? 0.f : ex2(a.x - top);
                w1 = b.y == 0.f ? 0.f : ex2(b.x - top);
                l = a.y * w0 + b.y * w1;
                base = top;
            }
            auto outputs_read = [&] {
                tc_fence_before();
                __syncwarp();
                if (merge && lane == 0) mbar_arrive(mfree);
            };
            if (idle || !live) {
                outputs_read();
                release();
                continue;
            }
            const int query = it.q0 + (NS == 2 && !DEC ? 128 * s : 0) + me, item_chunk = it.chunk;
            bool write = query < it.nq;
            const int row2 = it.r0 + (write ? query / p.group : 0), head2 = it.g * p.group + (write ? query % p.group : 0);
            const int len2 = write ? length_of(p, row2) : 0;
            const int64_t at = static_cast<int64_t>(row2) * p.heads + head2;
            release();
            int slot = 0;
            if (p.chunk && write) {
                const Chunks c = chunks_of(p, len2);
                slot = item_chunk < c.first ? item_chunk : c.first + item_chunk - c.from;
                write = item_chunk < c.first || (item_chunk >= c.from && item_chunk < c.end);
            }
            const bool none = l == 0.f;
            const float inv = none ? 0.f : p.chunk ? w0 : w0 / l, inv1 = none ? 0.f : p.chunk ? w1 : w1 / l;
            const int from_d = merge ? s * (D / 2) : 0, to_d = from_d + (merge ? D / 2 : D);
            if (write && from_d == 0) {
                if (p.chunk) *reinterpret_cast<float2*>(p.ml + (at * p.slots + slot) * 2) = make_float2(base, l);
                else if (p.lse) p.lse[at] = none ? -INFINITY : (base + log2f(l)) * 0.6931471805599453f;
            }
            const bool wide32 = p.chunk || p.out_type == QMM_TYPE_F32;
            uint8_t* dst = p.chunk ? reinterpret_cast<uint8_t*>(p.o + (at * p.slots + slot) * D) : static_cast<uint8_t*>(p.out) + at * D * (wide32 ? 4 : 2);
            const bool whole = (reinterpret_cast<uintptr_t>(dst) & 31) == 0;
            // 16 dims of both streams at a time, or 32 of the one
#pragma unroll 1
            for (int c = from_d; c < to_d; c += merge ? 16 : 32) {
                uint32_t w[2][16];
                const uint32_t first_col = lanes + G::col_o + (merge ? 0 : s * D) + c;
                if (merge || !fresh) {
                    tmem_ld16(first_col, w[0]);
                    tmem_ld16(first_col + (merge ? D : 16), w[1]);
                }
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    float o = inv == 0.f ? 0.f : __uint_as_float(w[0][j]) * inv, other = __uint_as_float(w[1][j]);
                    if (merge) o += inv1 == 0.f ? 0.f : other * inv1;
                    else other = inv == 0.f ? 0.f : other * inv;
                    w[0][j] = __float_as_uint(o);
                    w[1][j] = __float_as_uint(other);
                }
                if (write) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        if (merge && i) continue;
                        if (wide32) {
                            store32(dst + 4 * (c + 16 * i), whole, w[i]);
                            store32(dst + 4 * (c + 16 * i) + 32, whole, w[i] + 8);
                        } else {
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                const float a = __uint_as_float(w[i][2 * j]), b = __uint_as_float(w[i][2 * j + 1]);
                                w[i][j] = p.out_type == QMM_TYPE_F16 ? pack2<false>(a, b) : pack2<true>(a, b);
                            }
                            store32(dst + 2 * (c + 16 * i), whole, w[i]);
                        }
                    }
                }
                __syncwarp();
            }
            outputs_read();
        }
        if (!live && lane == 0) atomicOr(p.err, kErrTimeout);
    } else if constexpr (G::q8) {
        setmaxnreg_dec<80>();
        // ---------------------------------------------------------------- q8_0 to fp16; a tile is a page
        // K goes a tile ahead: V of a tile may wait for a product that comes after the next tile's scores.
        const int me = tid & 127, slot = me & 63, half = me >> 6, key = q8_key(slot & 7);
        // (the order in which a thread takes its four pieces of 16 tokens of V, c ^ x by lane, keeps both the reads, 64
        // bytes apart, and the swizzled writes free of bank conflicts)
        const int w4 = warp & 3, turn = (0x78 >> (2 * ((lane >> 1) & 3))) & 3;  // 0, 2, 3, 1
        uint8_t* dv = sm + G::off_dv + w4 * 128;
        auto convert_k = [&](int t) {  // half a token's dims per thread
            const int ks = t % G::k_slots, rs = t % G::raw_slots;
            await(rfull + rs, (t / G::raw_slots) & 1);
            if (!live) return;
            const int pg = raw_sm[rs];
            uint4 row[4];
            uint32_t sc = 0;
            if (pg >= 0) {
                const uint8_t* b = sm + G::off_raw + rs * kQ8Half;
#pragma unroll
                for (int c = 0; c < 4; ++c) row[c] = *reinterpret_cast<const uint4*>(b + slot * 128 + 16 * ((4 * half + c) ^ key));
                sc = *reinterpret_cast<const uint32_t*>(b + 8192 + slot * 8 + 4 * half);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(rempty + rs);
            if (t >= G::k_slots) await(kempty + ks, (t / G::k_slots - 1) & 1);
            if (!live) return;
            if (me == 0) kmiss_sm[t & 15] = pg == -2;
            if (pg >= 0) {
                uint8_t* dst = sm + ks * G::tile + half * (kTile * 128) + slot * 128;
#pragma unroll
                for (int c = 0; c < 8; ++c) {  // eight dims: one 16-byte piece of each part
                    const uint32_t u0 = ((c & 1) ? row[c >> 1].z : row[c >> 1].x) ^ 0x80808080u;
                    const uint32_t u1 = ((c & 1) ? row[c >> 1].w : row[c >> 1].y) ^ 0x80808080u;
                    const __half2 d = __half2half2(c >> 2 ? __high2half(as_h2(sc)) : __low2half(as_h2(sc)));
                    const __half2 z[4] = {i8_to_h2(u0, 0x4140u), i8_to_h2(u0, 0x4342u), i8_to_h2(u1, 0x4140u), i8_to_h2(u1, 0x4342u)};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const __half2 x = __hmul2(z[j], d);
                        hi[j] = as_u32(x);
                        lo[j] = as_u32(__hfma2(z[j], d, __hneg2(x)));
                    }
                    const int at = (c ^ (slot & 7)) << 4;
                    *reinterpret_cast<uint4*>(dst + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(dst + G::part + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(kfull + t % G::k_told);
        };
        auto convert_v = [&](const Record& it, int t0, int t) {  // a dim per thread
            const int vs = t % G::v_slots, rs = t % G::raw_slots;
            await(rfull + G::raw_slots + rs, (t / G::raw_slots) & 1);
            if (t >= G::v_slots) await(vempty + vs, (t / G::v_slots - 1) & 1);
            if (!live) return;
            const int pg = raw_sm[2 + rs];
            const uint8_t* b = sm + G::off_raw + (G::raw_slots + rs) * kQ8Half;
            const uint8_t* scales = b + 8192 + w4 * 128;
            if (pg < 0 || edge(it, t0)) {
                // Scales of 0 for tokens that must not count, as warp 2 zeroes rows of 16-bit pools (what is not finite
                // is a scale, or too large for fp16).  A warp's dims are one block of scales.
                uint32_t mine = 0;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int tok = t0 + 2 * lane + j;
                    const bool none = pg < 0 || gone(it, tok);
                    bool odd = false;
                    if (!none && !(tok < it.minlen && (tok >= it.maxlo || tok < p.sinks))) {
#pragma unroll
                        for (int c = 0; c < 4; ++c) odd |= (*reinterpret_cast<const uint16_t*>(b + 8192 + c * 128 + 4 * lane + 2 * j) & 0x7FFFu) >= (24u << 10);  // 512
                    }
                    const uint32_t who = __ballot_sync(0xffffffffu, odd);
                    if (w4 == 0 && lane == 0) odd_sm[t % G::v_told * 2 + j] = who;
                    if (!none && !odd) mine |= static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(scales + 4 * lane + 2 * j)) << (16 * j);
                }
                *reinterpret_cast<uint32_t*>(dv + 4 * lane) = mine;
                __syncwarp();
                scales = dv;
            }
            uint8_t* dst = sm + G::off_v + vs * G::tile + me * 128;
            // (not unrolled: 4 x 524 rows take 138 us, 143 with four times the code beside the softmax's)
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                const int cc = c ^ turn;  // 16 tokens
                uint4 u = make_uint4(0, 0, 0, 0);
                if (pg >= 0) u = *reinterpret_cast<const uint4*>(b + me * 64 + 16 * cc);
#pragma unroll
                for (int j = 0; j < 2; ++j) {  // eight of them: a 16-byte piece of each part
                    const uint4 d = *reinterpret_cast<const uint4*>(scales + 32 * cc + 16 * j);
                    const uint32_t u0 = (j ? u.z : u.x) ^ 0x80808080u, u1 = (j ? u.w : u.y) ^ 0x80808080u;
                    const __half2 z[4] = {i8_to_h2(u0, 0x4140u), i8_to_h2(u0, 0x4342u), i8_to_h2(u1, 0x4140u), i8_to_h2(u1, 0x4342u)};
                    const __half2 e[4] = {as_h2(d.x), as_h2(d.y), as_h2(d.z), as_h2(d.w)};
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        const __half2 x = __hmul2(z[n], e[n]);
                        hi[n] = as_u32(x);
                        lo[n] = as_u32(__hfma2(z[n], e[n], __hneg2(x)));
                    }
                    const int at = ((2 * cc + j) ^ (me & 7)) << 4;
                    *reinterpret_cast<uint4*>(dst + at) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                    *reinterpret_cast<uint4*>(dst + G::part + at) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(vready + t % G::v_told);
                mbar_arrive(rempty + G::raw_slots + rs);
            }
        };
        Record ahead, it;  // K's item and V's
        ahead.nt = it.nt = 0;
        int item = blockIdx.x, tk = 0, tv = 0, left = 0, i = 0;
        for (;;) {
            if (left == 0 && item < total) {
                ahead = next_record();
                item = following(item);
                left = live ? ahead.nt : 0;
            }
            const bool also = left > 0;  // a tile's K before the V of the one before it
            if (also) {
                convert_k(tk++);
                --left;
            }
            if (!live) break;
            if (tv + also < tk) {  // (without a K too: the record after an item without tiles takes the place of one that waits for this V)
                convert_v(it, tile_at(it, i) * kTile, tv++);
                ++i;
            } else if (!also && item >= total) {
                break;
            }
            if (i == it.nt) {
                it = ahead;
                i = 0;
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

template <int FMT, int D, bool DEC>
cudaError_t launch_one(const Launch& a, cudaStream_t s) {
    using G = Geo<FMT, D, DEC>;
    static_assert(G::smem(kMaxAgents) <= kMaxShared);
    static Once once;
    // (the registers that the roles deal out are those of the launch: fewer would leave a role waiting)
    static const int regs = [] {
        cudaFuncAttributes f = {};
        return cudaFuncGetAttributes(&f, attend_window_tc<FMT, D, DEC>) == cudaSuccess ? f.numRegs : 0;
    }();
    if (G::streams == 2 && regs < (G::threads == 512 ? 128 : 168)) return cudaErrorLaunchOutOfResources;
    const cudaError_t e = once.allow_shared(attend_window_tc<FMT, D, DEC>, a.device);
    if (e != cudaSuccess) return e;
    attend_window_tc<FMT, D, DEC><<<a.grid, G::threads, G::smem(a.p.agents), s>>>(a.map, a.p);
    return cudaGetLastError();
}

cudaError_t launch_q8(const Launch& a, bool decode, cudaStream_t s);
cudaError_t launch_f16_prompts(const Launch& a, int head_dim, cudaStream_t s);
cudaError_t launch_f16_decode(const Launch& a, int head_dim, cudaStream_t s);
cudaError_t launch_bf16_prompts(const Launch& a, int head_dim, cudaStream_t s);
cudaError_t launch_bf16_decode(const Launch& a, int head_dim, cudaStream_t s);

}  // namespace window
}  // namespace qmm
