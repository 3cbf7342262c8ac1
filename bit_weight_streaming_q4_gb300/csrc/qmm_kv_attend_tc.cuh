// Attention of new tokens over the paged cache: the split kernel for head dimension 128, on the
// 5th-generation tensor cores.
//
// The mathematics, the items and the partials are those of qmm_kv_attend.cuh.  A block (one per SM,
// persistent) works on tiles of 128 tokens:
//   S^T[token][query] = K Q^T      M = 128 tokens, N = 16, 32 or 48 queries, K = the dims
//   O^T[dim][query]  += V^T P^T    M = 128 dims, K = the tokens
// with the accumulators in tensor memory, so a thread of the softmax warps owns a token's row of
// scores and needs no exchange to form its probabilities, and the outputs cost no registers.
//   warps 0, 3  ask for K tiles and V tiles (bulk copies into two rings; one warp for both would hold K
//               back while V's slots are in use)
//   warp 1      issues the products: S of tile t + 1 goes before O of tile t, so that it overlaps
//               the softmax
//   warp 2      brings the next item: its numbers and its queries
//   warps 4 ..  softmax, two or three groups of four, a share of the queries each: scores from
//               tensor memory, probabilities into shared memory as the second product's B operand,
//               in two 16-bit parts
//   last four   q8_0 only: K and V quants to fp16 in tensor memory, as A operands (or eight, four for each)
// 16-bit pools: the swizzled tiles are A operands as they come, K by rows and V transposed
// (M-contiguous).  q8_0: K's quants are exact in fp16, one accumulator per 32-dim block takes its
// scale in fp32.  V's scale depends on token and block: the exponent of a token's largest scale (-7 at least)
// is its e_t and joins the softmax's reference (y_t = x_t + e_t, M = max y_t), so that
// p^ = 2^(y_t - M) <= 1 whatever the scales, and V's element, quant times normalised scale
// (scale 2^(8 - e_t), below 2^9: the product is at most 65,504), is split into two fp16 parts without error
// (product, its error by fma); three of the four products of parts count.  That holds while none of the
// token's scales other than 0 has an exponent more than 22 below the largest's, which takes one of 512 or more;
// what the product lacks of other tokens is added one by one in fp32.
//
// A query's reference is its first tile's maximum and moves only when a score passes it by more than
// 2^kSlack (a vote per tile; then the group forms the tile's maxima and rescales what it
// holds).  Each query decides for itself, so its bits depend on nothing but its own tokens.
//
// What it measured (this kernel alone, without weights; in brackets the call, whose join comes after):
// fp16, one sequence of 131,071, 1 row: 80 us (87), 6.7 TB/s, the bytes.  bf16, 8 x 16,000, 8 rows
// (48 queries a head): 93 us (107), 5.6 TB/s.  q8_0, 4 x 23,000, 3 rows (18 queries): 81 us (87), 2.5 TB/s.
// The second is bound by the chain from a tile's scores to its probabilities, some 3,500 clocks a tile
// in a softmax group (by clock readings in a copy of the kernel); q8_0 by the conversion of V as well:
// without three quarters of it, 66 us for 85.  With weights the scores' way through L2 costs 10 to 33 us.
// Not kept, this kernel's time against its time then: groups that take whole tiles in turn, with
// outputs of their own (q8_0 125 us for 90, bf16 144 for 110: each thread then does all queries); four
// groups of 8 queries at q8_0 (97 for 90); registers dealt out anew between the roles (85 for 81).
// On mma.sync with the outputs in registers the three cases took 86, 300 and 113 us.  (qmm_attn_decode's
// kernel does the q8_0 case in 52 us, with p rounded to 16 bits once and without the weights.)
#pragma once

#include "qmm_kv_attend.cuh"

namespace qmm {
namespace kv {

constexpr float kTcShift = 9.f;   // p's power of two ..
constexpr float kSlack = 6.f;     // .. and how far a score may pass its reference: p <= 2^15
constexpr float kFine = 4194304.f;  // 2^22: references below it hold sums with the two (fp32 is spaced by 1/4 at most
                                    // there); a larger one stands alone, without shift and slack: p <= 1 (q8_0, whose
                                    // exponent in -7 .. 15 a large score may round away: 2^15)
constexpr int kVShift = 8;        // q8_0: V's power of two, off again where the outputs are read
constexpr float kLowScale = 2048.f;  // p's low part is kept times this (its products have columns of their
                                     // own), so that p keeps 22 bits down to 2^-23 of the reference's, and 2^-45 of
                                     // it below

// Q: queries of a tile, of N columns.
template <int FMT, int N, int Q>
struct TcGeo {
    static constexpr bool q8 = FMT == QMM_KV_Q8_0;
    static constexpr int groups = N == 48 ? 3 : 2;                 // softmax groups of four warps
    static constexpr int W = Q / groups, B = W % 8 ? W : 8;        // queries of a group, and of a read of tensor memory
    // q8_0, few queries: K and V converted by warps of their own, waits asked for at once and references read
    // early.  4 x 23,000 tokens with weights: 1 row 84 -> 82 us, 3 rows 98 -> 94 (83 and 94 now).  At 32 and 48 queries,
    // whose threads have too few registers for it, 5 rows would go from 108 to 125 and 8 from 136 to 158 (109 and 139 now).
    static constexpr bool eager = q8 && Q <= 24;
    static constexpr int converters = !q8 ? 0 : eager ? 2 : 1;     // groups of four warps
    static constexpr int threads = 128 * (1 + groups + converters);
    static constexpr int half = q8 ? 2 * kQ8Half : kTcTile * 256;  // bytes of a tile's K or V
    static constexpr int k_slots = q8 ? 4 : 2, v_slots = q8 ? 4 : 3;  // (K's are free again once S is formed)
    static constexpr int p_bufs = N == 48 ? 1 : 2;                 // (no room for two beside three V tiles: bf16 8 x 16,000: this kernel 101 us with V's third, 106 with P's second)
    static constexpr int opnd = N * 256;                           // bytes of a B operand: N rows of 128 16-bit values
    // tensor memory columns: scores (one set per 32-dim block of a q8_0 pool), outputs (2 N: those of P's
    // high and of its low parts; of 16-bit pools two sets, items in turn), and the A operands
    static constexpr int o_bufs = q8 ? 1 : 2;
    static constexpr int col_s = 0, col_o = q8 ? 4 * N : 64, col_k = 288, col_vh = 352, col_vl = 416;
    static constexpr int cols = q8 ? 512 : 256;
    // shared memory, after aligning to 1024
    static constexpr int off_v = k_slots * half;
    static constexpr int off_q = (off_v + v_slots * half + 1023) / 1024 * 1024;  // two
    static constexpr int off_p = off_q + 2 * opnd;                              // p_bufs, each 2 N / 32 blocks of [token][32 queries]: high parts, then low ones
    static constexpr int off_dv = off_p + p_bufs * 2 * opnd;                             // q8_0: normalised V scales [2][4][128] fp16
    static constexpr int off_len = off_dv + (q8 ? 2 * 4 * kTcTile * 2 : 0);         // [2][N] tokens that a query sees
    static constexpr int off_lim = off_len + 2 * N * 4;                         // [N] reference + slack
    static constexpr int off_sub = off_lim + N * 4;                             // [N] what comes off the scores: reference - kTcShift
    static constexpr int off_alpha = off_sub + N * 4;                           // [N]
    static constexpr int off_red = off_alpha + N * 4;                           // [group][4 warps][W]
    static constexpr int off_odd = off_red + 4 * N * 4;                         // [4] tokens to be taken query by query
    static constexpr int off_bar = off_odd + 16;
    static constexpr int bars = 2 * k_slots + 2 * v_slots + 4 + 6 + 4 + 2;
    static constexpr int off_item = (off_bar + bars * 8 + 15) / 16 * 16;        // [2] of ItemRec
    static constexpr int off_misc = off_item + 2 * 32;                          // tmp[33], abort, accumulate[2], tmem, miss[v_slots], dead and missed by group, wide by group
    static constexpr int off_seq = (off_misc + 52 * 4 + 15) / 16 * 16;
    static constexpr int smem(int agents) { return 1024 + off_seq + (agents + 1) * 16; }
};

// Shared-memory descriptor of an M-contiguous operand in the 128-byte swizzle: atoms of 64 elements
// (128 bytes) x 8 rows; `lead` bytes to the next 64 elements, 1024 to the next 8 rows.
__device__ __forceinline__ uint64_t smem_desc_sw128_mn(uint32_t saddr, uint32_t lead) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}
// The same of one in the 64-byte swizzle: atoms of 32 elements (64 bytes) x 8 rows, 512 to the next 8 rows.
__device__ __forceinline__ uint64_t smem_desc_sw64_mn(uint32_t saddr, uint32_t lead) {
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(lead >> 4) << 16) |
           (static_cast<uint64_t>(512 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(4) << 61);
}
// V's scales of a q8_0 token, their signs off: the largest (NaN does not count); its biased exponent, which comes off
// the scales (that of 2^-7 at least: its inverse times 2^kVShift is then one fp16 number, and smaller scales
// need no more room; infinity as 65,504); and whether some scale other than 0 is then below what fp16 holds
// exactly, its own exponent (counted from 1) being more than 22 below.  A token whose largest is below kWide never is.
constexpr uint32_t kWide = 24u << 10;  // 512
__device__ __forceinline__ uint32_t largest_scale(const uint32_t (&w)[4]) {
    uint32_t top = 0;
#pragma unroll
    for (int b = 0; b < 4; ++b) top = w[b] > 0x7C00u ? top : max(top, w[b]);
    return top;
}
__device__ __forceinline__ int scale_exponent(uint32_t top) { return min(max(static_cast<int>(top >> 10), 8), 30); }
__device__ __forceinline__ __half scale_inverse(int exponent) { return __ushort_as_half(static_cast<uint16_t>((30 + kVShift - exponent) << 10)); }
__device__ __forceinline__ bool scales_far_apart(const uint32_t (&w)[4]) {
    const int top = scale_exponent(largest_scale(w));
    bool apart = false;
#pragma unroll
    for (int b = 0; b < 4; ++b) apart |= w[b] != 0 && max(static_cast<int>(w[b] >> 10), 1) + 22 < top;
    return apart;
}
// Byte of (token, column) of P: 64-byte rows by token, in blocks of 32 columns.
__device__ __forceinline__ int p_byte(int token, int col) {
    return (col >> 5) * (kTcTile * 64) + token * 64 + ((((col >> 3) & 3) ^ ((token >> 1) & 3)) << 4) + (col & 7) * 2;
}

// 8 consecutive columns of the thread's tensor memory lane (to be waited for with tc_wait_ld).
__device__ __forceinline__ void tmem_load8(uint32_t taddr, float* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_load4(uint32_t taddr, float* v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                 : "r"(taddr)
                 : "memory");
}
__device__ __forceinline__ void tmem_store8(uint32_t taddr, const float* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "f"(v[0]),
                 "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_store4(uint32_t taddr, const float* v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
                 : "memory");
}
template <int B>
__device__ __forceinline__ void tmem_load_n(uint32_t taddr, float (&v)[B]) {
    static_assert(B == 4 || B == 8 || B == 12);
    if constexpr (B == 4) tmem_load4(taddr, v);
    else tmem_load8(taddr, v);
    if constexpr (B == 12) tmem_load4(taddr + 8, v + 8);
}
template <int B>
__device__ __forceinline__ void tmem_store_n(uint32_t taddr, const float (&v)[B]) {
    if constexpr (B == 4) tmem_store4(taddr, v);
    else tmem_store8(taddr, v);
    if constexpr (B == 12) tmem_store4(taddr + 8, v + 8);
}

// Whether a wait would be over now.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// One lane of a converged warp.  (The products' operands stay in uniform registers inside its branch; by
// `lane == 0` an issue took 49 clocks and by a predicate on the instruction 68, against the 40 that the
// smallest product itself takes.)
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// (hi, lo) 16-bit pairs of two fp32 values: value = hi + lo / kLowScale.
template <bool BF>
__device__ __forceinline__ void split2_scaled(float a, float b, uint32_t& hi, uint32_t& lo) {
    if constexpr (BF) {
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(b), "f"(a));
        const float ra = a - __uint_as_float(hi << 16), rb = b - __uint_as_float(hi & 0xFFFF0000u);
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(rb * kLowScale), "f"(ra * kLowScale));
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        hi = as_u32(h);
        lo = as_u32(__floats2half2_rn((a - __low2float(h)) * kLowScale, (b - __high2float(h)) * kLowScale));
    }
}

// v[c] of W <= 32 columns reduced over the warp's lanes by f: lane c returns column c's.  At each
// step a lane keeps half of its columns and hands the other half to its partner.
template <int W, typename F>
__device__ __forceinline__ float reduce_columns(const float (&v)[W], float none, F f) {
    float u[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) u[i] = i < W ? v[i < W ? i : 0] : none;
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int h = 16; h >= 1; h >>= 1) {
        const bool up = lane & h;
#pragma unroll
        for (int i = 0; i < h; ++i) {
            if (i >= W) continue;  // (columns that nobody has)
            const float mine = up ? u[i + h] : u[i], other = up ? u[i] : u[i + h];
            u[i] = f(mine, __shfl_xor_sync(0xffffffffu, other, h));
        }
    }
    return u[0];
}

// What the roles need to know of an item, formed once by the warps that bring its queries.
struct alignas(16) ItemRec {
    int a, g, tok0, end;
    int q0, nq, minlen, r0;  // first query, queries of the sequence and KV head, the sequence's shortest row and first row
};

// (512: at most 128 registers, so that with 384 threads a block of the joining kernel, 40 registers by 256
// threads, fits beside and has begun when the partials are there; without room it cost 2 us a call.  Spilled at
// that: 4, 24 and 28 bytes by the 16-bit tiles of 24, 32 and 48 queries, 8 and 28 by q8_0's of 24 and 48.)
template <int FMT, int N, int Q>
__global__ void __launch_bounds__((TcGeo<FMT, N, Q>::threads > 512 ? TcGeo<FMT, N, Q>::threads : 512), 1)
    attend_partial_tc(const __grid_constant__ CUtensorMap map, const __grid_constant__ AttendParams p) {
    using G = TcGeo<FMT, N, Q>;
    constexpr bool BF = FMT == QMM_KV_BF16;
    constexpr int D = 128;
    extern __shared__ uint8_t sm_raw[];
    griddep_launch_dependents();  // the joining kernel waits for this grid's end before it reads
    uint8_t* sm = sm_raw + ((1024u - (smem_u32(sm_raw) & 1023u)) & 1023u);
    int* qlen_sm = reinterpret_cast<int*>(sm + G::off_len);
    float* lim_sm = reinterpret_cast<float*>(sm + G::off_lim);
    float* sub_sm = reinterpret_cast<float*>(sm + G::off_sub);
    float* alpha_sm = reinterpret_cast<float*>(sm + G::off_alpha);
    float* red_sm = reinterpret_cast<float*>(sm + G::off_red);
    ItemRec* item_sm = reinterpret_cast<ItemRec*>(sm + G::off_item);
    volatile uint32_t* odd_sm = reinterpret_cast<uint32_t*>(sm + G::off_odd);
    uint64_t* kfull = reinterpret_cast<uint64_t*>(sm + G::off_bar);
    uint64_t* kempty = kfull + G::k_slots;
    uint64_t* vfull = kempty + G::k_slots;
    uint64_t* vempty = vfull + G::v_slots;
    uint64_t *qfull = vempty + G::v_slots, *qempty = qfull + 2;                          // two each
    uint64_t *sfull = qempty + 2, *sempty = sfull + 1, *pfull = sfull + 2, *odone = sfull + 4;  // (pfull and odone: two each)
    uint64_t *akfull = sfull + 6, *akfree = sfull + 7, *avfull = sfull + 8, *avfree = sfull + 9, *drained = sfull + 10,
             *oddread = sfull + 11;
    int* tmp = reinterpret_cast<int*>(sm + G::off_misc);
    volatile int* abort_flag = tmp + 33;
    volatile int* accum_sm = tmp + 34;  // [2]: the outputs hold something that P's product adds to
    uint32_t* tmem_sm = reinterpret_cast<uint32_t*>(tmp + 36);
    volatile int* vmiss = tmp + 37;     // [v_slots <= 4]: a page of the tile is outside the pool
    int4* seq = reinterpret_cast<int4*>(sm + G::off_seq);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (tid == 0) {
        for (int i = 0; i < G::k_slots; ++i) {
            mbar_init(kfull + i, 1);
            mbar_init(kempty + i, G::q8 ? 4 + 4 * G::groups : 1);
        }
        for (int i = 0; i < G::v_slots; ++i) {
            mbar_init(vfull + i, 1);
            mbar_init(vempty + i, G::q8 ? 4 + 4 * G::groups : 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(qfull + i, 1);
            mbar_init(qempty + i, 1 + 4 * G::groups + 4 * G::converters);
        }
        mbar_init(sfull, 1);
        mbar_init(sempty, 4 * G::groups);
        for (int i = 0; i < 2; ++i) {
            mbar_init(pfull + i, 4 * G::groups);
            mbar_init(odone + i, 1);
        }
        mbar_init(akfull, 4);
        mbar_init(akfree, 1);
        mbar_init(avfull, 4);
        mbar_init(avfree, 1);
        mbar_init(drained, 1);
        mbar_init(oddread, 4 * G::groups);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (tid < 4) odd_sm[tid] = 0;
    if (tid < 9) tmp[41 + tid] = tid < 6 ? -(tid & 1) : -1;
    if (warp == 1) {
        tmem_alloc(tmem_sm, G::cols);
        tmem_relinquish();
    }
    tc_fence_before();
    const int total = form_table(p, seq, tmp, Q);
    tc_fence_after();
    const uint32_t tmem = *tmem_sm;

    // A wait of one of the roles.  Once one has run out, everything that follows runs dry.
    bool live = true;
    auto await = [&](uint64_t* b, uint32_t parity) {
        if (live && !mbar_wait_bounded(b, parity, abort_flag)) {
            live = false;
            *abort_flag = 1;
        }
        __syncwarp();
    };
    // the same, with one answer for the warp
    auto await_warp = [&](uint64_t* b, uint32_t parity) {
        await(b, parity);
        live = __all_sync(0xffffffffu, live);
    };

    if (warp == 0 || warp == 3) {
        // ---------------------------------------------------------------- producers
        const int h = warp == 3;  // 0: K, 1: V
        const int slots = h ? G::v_slots : G::k_slots;
        uint64_t* full = h ? vfull : kfull;
        uint64_t* empty = h ? vempty : kempty;
        uint8_t* ring = sm + (h ? G::off_v : 0);
        const uint64_t policy = l2_policy_evict_first();
        int nitem = blockIdx.x, t = 0;
        Item ni = {};
        int npages = 0;
        if (nitem < total) {
            ni = decode_item(p, seq, nitem, Q);
            npages = load_item_pages(p, ni);
        }
        while (nitem < total && live) {
            const Item it = ni;
            const int pages = npages, first = it.tok0 >> p.page_shift;
            nitem += gridDim.x;
            if (nitem < total) {
                ni = decode_item(p, seq, nitem, Q);
                npages = load_item_pages(p, ni);
            }
            for (int tb = it.tok0; tb < it.end && live; tb += kTcTile, ++t) {
                // pieces of at most a page, those with tokens before the item's end
                constexpr int kPieces = G::q8 ? 2 : kTcTile / 16;
                const int br = min(kTcTile, p.page_tokens);
                int pg[kPieces];
                int n_pieces = 0;
                bool miss = false;
#pragma unroll
                for (int k = 0; k < kPieces; ++k) {
                    const int tok = tb + k * br;
                    const bool in = k * br < kTcTile && tok < it.end;
                    const int x = __shfl_sync(0xffffffffu, pages, in ? (tok >> p.page_shift) - first : 0);
                    pg[k] = in ? x : -1;
                    miss |= in && x < 0;
                    n_pieces += pg[k] >= 0;
                }
                const int s = t % slots, round = t / slots;
                if (round > 0) await_warp(empty + s, (round - 1) & 1);
                if (!live) break;
                if (lane == 0) {
                    fence_proxy_async_smem();  // the slot's generic accesses, before the copies
                    if (h) vmiss[s] = miss;
                    uint8_t* dst = ring + s * G::half;
                    if (n_pieces == 0) mbar_arrive(full + s);
                    else mbar_arrive_expect_tx(full + s, n_pieces * (G::q8 ? kQ8Half : br * D * 2));
#pragma unroll
                    for (int k = 0; k < kPieces; ++k) {
                        if (pg[k] < 0) continue;
                        if constexpr (G::q8) {
                            bulk_g2s(dst + k * kQ8Half, p.pool + (static_cast<int64_t>(pg[k]) * p.kv_heads + it.g) * kQ8Rec + h * kQ8Half, kQ8Half,
                                     full + s, policy);
                        } else {
                            const int y = ((pg[k] * p.kv_heads + it.g) * 2 + h) * p.page_tokens + ((tb + k * br) & (p.page_tokens - 1));
#pragma unroll
                            for (int x = 0; x < D / 64; ++x)
                                tma_load_2d_hint(dst + x * kTcTile * 128 + k * br * 128, &map, 64 * x, y, full + s, policy);
                        }
                    }
                }
                __syncwarp();
            }
        }
        if (!live && lane == 0) {
            // let every copy still in flight land before the block exits: the last of each slot
            volatile int go_on = 0;
            for (int i = max(0, t - slots); i < t; ++i) mbar_wait_bounded(full + i % slots, (i / slots) & 1, &go_on, 100000000ull);
        }
    } else if (warp == 1) {
        // ---------------------------------------------------------------- products
        constexpr uint32_t kType = BF ? (1u << 7) | (1u << 10) : 0u;
        constexpr uint32_t kIdescS = idesc_f16_f32(128, N) | kType;
        // (both parts of P at once: 2 N columns; B is N-contiguous and, of 16-bit pools, A M-contiguous)
        constexpr uint32_t kIdescO = idesc_f16_f32(128, 2 * N) | kType | 1u << 16 | (G::q8 ? 0u : 1u << 15);
        constexpr uint32_t kIdescL = idesc_f16_f32(128, N) | kType | 1u << 16;
        int t = 0, k = 0;  // tiles and items so far
        const uint64_t bp = smem_desc_sw64_mn(smem_u32(sm + G::off_p), kTcTile * 64);
        auto product_o = [&](int i, int item_no) {
            await_warp(pfull + i % G::p_bufs, (i / G::p_bufs) & 1);
            const int vs = i % G::v_slots;
            if constexpr (G::q8) await_warp(avfull, i & 1);
            else await_warp(vfull + vs, (i / G::v_slots) & 1);
            if (!live) return;
            tc_fence_after();
            const uint64_t av = smem_desc_sw128_mn(smem_u32(sm + G::off_v) + vs * G::half, kTcTile * 128);
            const uint32_t acc = accum_sm[i % G::p_bufs] != 0;
            const uint32_t o = tmem + G::col_o + item_no % G::o_bufs * (2 * N);
            const uint64_t bi = bp + i % G::p_bufs * (2 * G::opnd >> 4);
            if (elect_one()) {
#pragma unroll
                for (int ks = 0; ks < 8; ++ks) {
                    const uint64_t b = bi + (ks * 1024 >> 4);
                    if constexpr (G::q8) {
                        tc_mma_f16_ts(o, tmem + G::col_vh + 8 * ks, b, kIdescO, ks ? 1 : acc);
                        tc_mma_f16_ts(o, tmem + G::col_vl + 8 * ks, b, kIdescL, 1);  // (by the high parts only)
                    } else {
                        tc_mma_f16_ss(o, av + ks * (2048 >> 4), b, kIdescO, ks ? 1 : acc);
                    }
                }
                tc_commit(odone + i % G::p_bufs);
                tc_commit(G::q8 ? avfree : vempty + vs);
            }
            __syncwarp();
        };
        for (int item = blockIdx.x; item < total && live; item += gridDim.x, ++k) {
            await_warp(qfull + (k & 1), (k >> 1) & 1);
            const int tok0 = item_sm[k & 1].tok0, end = item_sm[k & 1].end;
            const uint64_t bq = smem_desc_sw128(smem_u32(sm + G::off_q) + (k & 1) * G::opnd);
            for (int tb = tok0; tb < end && live; tb += kTcTile, ++t) {
                const int s = t % G::k_slots;
                if constexpr (G::q8) await_warp(akfull, t & 1);
                else await_warp(kfull + s, (t / G::k_slots) & 1);
                if (t > 0) await_warp(sempty, (t - 1) & 1);
                if (!live) break;
                tc_fence_after();
                const uint64_t ak = smem_desc_sw128(smem_u32(sm) + s * G::half);
                const bool last = tb + kTcTile >= end;
                if (elect_one()) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks) {
                        const uint64_t b = bq + (((ks >> 2) * (N * 128) + (ks & 3) * 32) >> 4);
                        if constexpr (G::q8)
                            tc_mma_f16_ts(tmem + G::col_s + (ks >> 1) * N, tmem + G::col_k + 8 * ks, b, kIdescS, ks & 1);
                        else
                            tc_mma_f16_ss(tmem + G::col_s, ak + (((ks >> 2) * (kTcTile * 128) + (ks & 3) * 32) >> 4), b, kIdescS, ks > 0);
                    }
                    tc_commit(sfull);
                    tc_commit(G::q8 ? akfree : kempty + s);
                    if (last) tc_commit(qempty + (k & 1));
                }
                __syncwarp();
                if (t > 0) product_o(t - 1, tb == tok0 ? k - 1 : k);
            }
        }
        if (t > 0 && live) product_o(t - 1, k - 1);
        // every product issued has finished before the tensor memory is released
        if (elect_one()) tc_commit(drained);
        volatile int go_on = 0;
        mbar_wait_bounded(drained, 0, &go_on, 10000000000ull);
        __syncwarp();
    } else if (warp == 2) {
        // ---------------------------------------------------------------- the next item: numbers and queries, half a warp per row
        int k = 0;
        for (int item = blockIdx.x; item < total && live; item += gridDim.x, ++k) {
            const Item it = decode_item(p, seq, item, Q);
            const int r0 = seq[it.a].w, nq = (seq[it.a + 1].w - r0) * p.group, q0 = it.tile * Q;
            const int buf = k & 1, c = lane & 15;
            if (k > 1) await_warp(qempty + buf, ((k >> 1) - 1) & 1);
            if (!live) break;
            if (lane == 0) {
                ItemRec rec = {it.a, it.g, it.tok0, it.end, q0, nq, seq[it.a].z, r0};
                item_sm[buf] = rec;
            }
            uint8_t* dst = sm + G::off_q + buf * G::opnd + (c >> 3) * (N * 128);
            for (int i0 = 0; i0 < N; i0 += 16) {
                // eight rows' 16-byte pieces on their way at once, then stored, swizzled as the copies do
                uint4 v[8];
                int len[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int qa = q0 + i0 + 2 * j + (lane >> 4);
                    v[j] = make_uint4(0, 0, 0, 0);
                    len[j] = 0;
                    if (qa < nq) {
                        const int r = r0 + qa / p.group, h = qa % p.group;
                        v[j] = *reinterpret_cast<const uint4*>(p.q + r * p.q_stride + static_cast<int64_t>(it.g * p.group + h) * D + 8 * c);
                        len[j] = p.row_len[r];
                    }
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const int qi = i0 + 2 * j + (lane >> 4);
                    *reinterpret_cast<uint4*>(dst + qi * 128 + (((c & 7) ^ (qi & 7)) << 4)) = v[j];
                    if (c == 0) qlen_sm[buf * N + qi] = len[j];
                }
            }
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(qfull + buf);
        }
    } else if (warp < 4 + 4 * G::groups) {
        // ---------------------------------------------------------------- softmax: a token per thread, then a dim
        constexpr int W = G::W, B = G::B;
        const int grp = (warp - 4) >> 2, me = (tid - 128) & 127, w4 = warp & 3;
        const uint32_t bar_id = 1 + grp;       // the group's barrier
        const int c0 = grp * W;                // the group's first query of the tile
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * w4) << 16);
        float* lim = lim_sm + c0;
        float* sub = sub_sm + c0;
        float* alpha = alpha_sm + c0;
        float* red = red_sm + grp * 4 * W;     // [4][W]
        volatile int* dead = tmp + 41 + 2 * grp;    // some thread's wait ran out
        volatile int* missed = dead + 1;            // the last tile with a missing page
        volatile int* wide_sm = tmp + 47 + grp;     // q8_0: the last tile with a token whose scales may lie far apart
        int t = 0, k = 0;
        uint32_t odds = 0;                     // tiles with marked tokens so far
        auto last_product = [&] { await(odone + (t - 1) % G::p_bufs, ((t - 1) / G::p_bufs) & 1); };  // of tile t - 1
        // The outputs of an item as its partial, a dim per thread.  With two sets of them that waits until the
        // next item's first probabilities are out, so that the tensor cores have work meanwhile.
        float* po = nullptr;                   // where they go, or null
        int left = 0;                          // queries from c0 on
        auto drain = [&](uint32_t cols) {
            constexpr float kBack = G::q8 ? 1.f / (1 << kVShift) : 1.f;
            tc_fence_after();
#pragma unroll
            for (int c = 0; c < W; c += B) {
                float v[2][B];
                tmem_load_n<B>(cols + c, v[0]);
                tmem_load_n<B>(cols + N + c, v[1]);
                tc_wait_ld();
#pragma unroll
                for (int i = 0; i < B; ++i)
                    if (c + i < left) po[(c + i) * D] = fmaf(v[1][i], kBack / kLowScale, v[0][i] * kBack);
            }
            po = nullptr;
        };
        // (what ends the loops is voted on, so that the warps always meet at the same barriers)
        for (int item = blockIdx.x; item < total; item += gridDim.x, ++k) {
            await(qfull + (k & 1), (k >> 1) & 1);
            const ItemRec it = item_sm[k & 1];
            const int* qlen = qlen_sm + (k & 1) * N + c0;
            const int q0 = it.q0 + c0;
            const uint32_t ocol = lanes + G::col_o + k % G::o_bufs * (2 * N) + c0;  // the item's outputs
            float l[W];
#pragma unroll
            for (int q = 0; q < W; ++q) l[q] = 0.f;
            if (me < W) {
                lim[me] = kNoMax;
                sub[me] = -kTcShift;
            }
            named_bar_sync(bar_id, 128);
            const int64_t plane = static_cast<int64_t>(p.chunks) * p.chunk * 4;
            float* sbase = p.scores ? p.scores + (static_cast<int64_t>(it.a * p.kv_heads + it.g) * (p.qp >> 2) + (q0 >> 2)) * plane : nullptr;
            const int mine = it.nq - q0;  // queries from c0 on

            bool stop = false;
            for (int tb = it.tok0; tb < it.end; tb += kTcTile, ++t) {
                const int tok = tb + me;
                const int vs = t % G::v_slots;
                uint8_t* vt = sm + G::off_v + vs * G::half;
                const int ksl = t % G::k_slots;
                bool ready = false, p_free = t < G::p_bufs;  // P's buffer is read
                if constexpr (G::eager) {
                    // (those that are over already, which they mostly are: one after the other each costs some 100 clocks)
                    ready = mbar_test(vfull + vs, (t / G::v_slots) & 1) & mbar_test(sfull, t & 1) &
                            mbar_test(kfull + ksl, (t / G::k_slots) & 1);
                    p_free = p_free || mbar_test(odone + t % G::p_bufs, (t / G::p_bufs - 1) & 1);
                    ready = __all_sync(0xffffffffu, ready);
                    p_free = __all_sync(0xffffffffu, p_free);
                }
                if (!ready) {
                    if constexpr (G::q8) await(kfull + ksl, (t / G::k_slots) & 1);
                    await(vfull + vs, (t / G::v_slots) & 1);
                    await(sfull, t & 1);
                }
                tc_fence_after();
                // ---- base-2 scores, masked; a query's first tile, or one that passes its reference by more
                // than the slack, takes the long way
                float x[W], e = 0.f;
                float4 limit[W / 4];
                bool miss, wide = false;  // (q8_0: the token's V scales may lie far apart)
                auto limits = [&] {
#pragma unroll
                    for (int q = 0; q < W; q += 4) limit[q / 4] = *reinterpret_cast<const float4*>(lim + q);
                };
                if constexpr (G::q8) {
                    float f[4];
#pragma unroll
                    for (int c = 0; c < W; c += B) {
                        float v[4][B];
#pragma unroll
                        for (int b = 0; b < 4; ++b) tmem_load_n<B>(lanes + G::col_s + b * N + c0 + c, v[b]);
                        if (c == 0) {
                            // the token's K scales and the exponent of its largest V scale
                            const uint2 sc = *reinterpret_cast<const uint2*>(sm + ksl * G::half + (me >> 6) * kQ8Half + 8192 + (me & 63) * 8);
                            uint32_t w[4];
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                w[b] = *reinterpret_cast<const uint16_t*>(vt + (me >> 6) * kQ8Half + 8192 + (b * 64 + (me & 63)) * 2) & 0x7FFFu;
                            miss = vmiss[vs] != 0;  // a page of the tile is outside the pool
                            if constexpr (G::eager) limits();
                            f[0] = __low2float(as_h2(sc.x)) * p.c2, f[1] = __high2float(as_h2(sc.x)) * p.c2;
                            f[2] = __low2float(as_h2(sc.y)) * p.c2, f[3] = __high2float(as_h2(sc.y)) * p.c2;
                            const uint32_t top = largest_scale(w);
                            wide = top >= kWide;
                            e = static_cast<float>(scale_exponent(top) - 15);
                        }
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < B; ++i)
                            x[c + i] = fmaf(v[3][i], f[3], fmaf(v[2][i], f[2], fmaf(v[1][i], f[1], v[0][i] * f[0])));
                    }
                } else {
                    float v[W / B][B];
#pragma unroll
                    for (int c = 0; c < W / B; ++c) tmem_load_n<B>(lanes + G::col_s + c0 + B * c, v[c]);
                    miss = vmiss[vs] != 0;
                    tc_wait_ld();
#pragma unroll
                    for (int q = 0; q < W; ++q) x[q] = v[q / B][q % B] * p.c2;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(sempty);
                    if constexpr (G::q8) mbar_arrive(kempty + ksl);
                }
                if (miss || tb + kTcTile > it.minlen) {  // some query does not see some token of the tile
#pragma unroll
                    for (int q = 0; q < W; ++q)
                        if (miss || tok >= qlen[q]) x[q] = kNoMax;
                }
                if (sbase) {
                    float* at = sbase + static_cast<int64_t>(tok) * 4;
#pragma unroll
                    for (int q = 0; q < W; q += 4) {
                        if (q + 2 < mine) *reinterpret_cast<float4*>(at + (q >> 2) * plane) = make_float4(x[q], x[q + 1], x[q + 2], x[q + 3]);
                        else if (q < mine) *reinterpret_cast<float2*>(at + (q >> 2) * plane - 2 * tok) = make_float2(x[q], x[q + 1]);
                    }
                }
                bool over = !live || miss || wide;
                if constexpr (!G::eager) limits();
#pragma unroll
                for (int q = 0; q < W; q += 4) {
                    const float4 m = limit[q / 4];
                    if constexpr (G::q8) over |= x[q] + e > m.x || x[q + 1] + e > m.y || x[q + 2] + e > m.z || x[q + 3] + e > m.w;
                    else over |= x[q] > m.x || x[q + 1] > m.y || x[q + 2] > m.z || x[q + 3] > m.w;
                }
                bool moved = false;  // some reference moves
                float4 base[W / 4];  // the references, as P takes them
                auto bases = [&] {
#pragma unroll
                    for (int q = 0; q < W; q += 4) base[q / 4] = *reinterpret_cast<const float4*>(sub + q);
                };
                if constexpr (G::eager) bases();
                if (!live) *dead = 1;
                if (miss) *missed = t;
                if (G::q8 && wide) *wide_sm = t;
                bool some_wide = false;
                if (bar_or(bar_id, 128, over)) {
                    if (*dead) {
                        stop = true;
                        po = nullptr;
                        break;
                    }
                    miss = *missed == t;
                    some_wide = G::q8 && *wide_sm == t;
                    // (a NaN is no maximum: fmaxf passes it over)
                    float y[W];
#pragma unroll
                    for (int q = 0; q < W; ++q) y[q] = G::q8 ? x[q] + e : x[q];
                    const float r = reduce_columns<W>(y, kNoMax, [](float a, float b) { return fmaxf(a, b); });
                    if (lane < W) red[w4 * W + lane] = r;
                    named_bar_sync(bar_id, 128);
                    if (me < W) {
                        float m = fmaxf(fmaxf(red[me], red[W + me]), fmaxf(red[2 * W + me], red[3 * W + me]));
                        if (fabsf(m) < 1e6f) m = ceilf(m * 16.f) * 0.0625f;  // (sums with the constants are then exact)
                        const bool passed = m > lim[me];
                        const bool fine = fabsf(m) < kFine;
                        const float base = fine ? m - kTcShift : m;
                        // (what was formed with the old reference, by the difference of what was taken off; 0 the first time)
                        alpha[me] = !passed ? 1.f : lim[me] == kNoMax ? 0.f : ex2(sub[me] - base);
                        if (passed) {
                            lim[me] = fine ? m + kSlack : m;
                            sub[me] = base;
                        }
                    }
                    named_bar_sync(bar_id, 128);
#pragma unroll
                    for (int q = 0; q < W; ++q) {
                        const float a = alpha[q];
                        l[q] *= a;
                        moved |= a != 1.f;
                    }
                    if constexpr (G::eager) bases();
                }
                const bool edge = miss || some_wide || tb + kTcTile > it.minlen;
                const bool fresh = tb == it.tok0;  // the outputs hold nothing yet
                if (!p_free) await(odone + t % G::p_bufs, (t / G::p_bufs - 1) & 1);
                if (moved && !fresh) {
                    last_product();  // (only a new reference or a marked token needs its outputs)
                    tc_fence_after();
#pragma unroll
                    for (int c = 0; c < W; c += B) {
                        float v[2][B];
                        tmem_load_n<B>(ocol + c, v[0]);
                        tmem_load_n<B>(ocol + N + c, v[1]);
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < B; ++i) v[0][i] *= alpha[c + i], v[1][i] *= alpha[c + i];
                        tmem_store_n<B>(ocol + c, v[0]);
                        tmem_store_n<B>(ocol + N + c, v[1]);
                    }
                    tc_wait_st();
                }
                // ---- probabilities, as the token's rows of the B operand (queries contiguous, swizzled): 16-byte
                // stores; with tokens contiguous they were 2-byte ones, 32 of a q8_0 thread's
                const float inv = G::q8 ? __int_as_float((127 - static_cast<int>(e)) << 23) : 1.f;  // 2^-e
                uint8_t* pt = sm + G::off_p + t % G::p_bufs * (2 * G::opnd);
                if constexpr (!G::eager) bases();
#pragma unroll
                for (int q = 0; q < W; q += 4) {
                    const float4 m = base[q / 4];
                    x[q] -= m.x, x[q + 1] -= m.y, x[q + 2] -= m.z, x[q + 3] -= m.w;
                    // (e after the reference is off: a large score's spacing could swallow it)
                    if constexpr (G::q8) x[q] += e, x[q + 1] += e, x[q + 2] += e, x[q + 3] += e;
                    x[q] = ex2(x[q]), x[q + 1] = ex2(x[q + 1]), x[q + 2] = ex2(x[q + 2]), x[q + 3] = ex2(x[q + 3]);
                }
#pragma unroll
                for (int q = 0; q < W; q += B == 8 ? 8 : 4) {
                    constexpr int S = B == 8 ? 4 : 2;  // (12 columns begin in the middle of 16 bytes)
                    uint32_t hi[S], lo[S];
#pragma unroll
                    for (int i = 0; i < 2 * S; ++i) l[q + i] = G::q8 ? fmaf(x[q + i], inv, l[q + i]) : l[q + i] + x[q + i];
#pragma unroll
                    for (int i = 0; i < S; ++i) split2_scaled<BF>(x[q + 2 * i], x[q + 2 * i + 1], hi[i], lo[i]);
                    uint8_t *ph = pt + p_byte(me, c0 + q), *pl = pt + p_byte(me, N + c0 + q);
                    if constexpr (S == 4) {
                        *reinterpret_cast<uint4*>(ph) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
                        *reinterpret_cast<uint4*>(pl) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
                    } else {
                        *reinterpret_cast<uint2*>(ph) = make_uint2(hi[0], hi[1]);
                        *reinterpret_cast<uint2*>(pl) = make_uint2(lo[0], lo[1]);
                    }
                }
                bool holds = !fresh;
                if (edge) {
                    // Tokens that some query does not see.  Past the sequence's end (and in tiles with a
                    // missing page) V holds anything and becomes zero (q8_0: its scales do, in the
                    // converting warps).  One that some queries see and whose V (q8_0: a scale) is
                    // not finite is added query by query, to those that see it, and is zero in the
                    // product.  So is, to all, what the product lacks of a q8_0 token whose scales lie far
                    // apart.  (All groups come to the same answers.)
                    const bool gone = miss || tok >= it.end;
                    bool odd = false;
                    auto piece = [&](int c) { return reinterpret_cast<uint4*>(vt + (c >> 3) * (kTcTile * 128) + me * 128 + (((c & 7) ^ (me & 7)) << 4)); };
                    if (!gone && (G::q8 || tok >= it.minlen)) {
                        if constexpr (G::q8) {
                            uint32_t w[4];
#pragma unroll
                            for (int b = 0; b < 4; ++b)
                                w[b] = *reinterpret_cast<const uint16_t*>(vt + (me >> 6) * kQ8Half + 8192 + (b * 64 + (me & 63)) * 2) & 0x7FFFu;
                            odd = scales_far_apart(w);
#pragma unroll
                            for (int b = 0; b < 4; ++b) odd |= tok >= it.minlen && w[b] >= 0x7C00u;
                        } else {
                            constexpr uint32_t ex = BF ? 0x7F80u : 0x7C00u;
                            auto bad = [&](uint32_t w) { return (w & ex) == ex || ((w >> 16) & ex) == ex; };
                            for (int c = 0; c < 16; ++c) {
                                const uint4 v = *piece(c);
                                odd |= bad(v.x) || bad(v.y) || bad(v.z) || bad(v.w);
                            }
                        }
                    }
                    const bool any = bar_or(bar_id, 128, odd);  // (also: P is written)
                    if (any) {
                        const uint32_t who = __ballot_sync(0xffffffffu, odd);
                        if (lane == 0) odd_sm[w4] = who;  // (all groups write the same)
                        named_bar_sync(bar_id, 128);
                        if (holds) {
                            last_product();
                            tc_fence_after();
                        }
                        constexpr int S = 4;  // (few registers: this is rare, and the loop around it has none to spare)
#pragma unroll 1
                        for (int c = 0; c < W; c += S) {
                            float v[S];
                            if (holds) {
                                tmem_load_n<S>(ocol + c, v);
                                tc_wait_ld();
                            } else {
#pragma unroll
                                for (int i = 0; i < S; ++i) v[i] = 0.f;
                            }
#pragma unroll 1
                            for (int j = 0; j < kTcTile; ++j) {
                                if (!((odd_sm[j >> 5] >> (j & 31)) & 1)) continue;
                                float y;  // V of token j, dim me (q8_0: by its normalised scale)
                                if constexpr (G::q8) {
                                    const uint8_t* rec = vt + (j >> 6) * kQ8Half;
                                    const __half d = *reinterpret_cast<const __half*>(rec + 8192 + ((me >> 5) * 64 + (j & 63)) * 2);
                                    uint32_t w[4];
                                    bool zeroed = false;  // (not finite: the converting warps took zeros)
#pragma unroll
                                    for (int b = 0; b < 4; ++b) {
                                        w[b] = *reinterpret_cast<const uint16_t*>(rec + 8192 + (b * 64 + (j & 63)) * 2) & 0x7FFFu;
                                        zeroed |= tb + j >= it.minlen && w[b] >= 0x7C00u;
                                    }
                                    const int ej = scale_exponent(largest_scale(w));
                                    const float quant = static_cast<float>(static_cast<int8_t>(rec[me * 64 + (j & 63)]));
                                    y = quant * (__half2float(d) * __int_as_float((142 + kVShift - ej) << 23));
                                    if (!zeroed) {  // scales far apart: what the product lacks
                                        const __half n = __hmul(d, scale_inverse(ej)), z = __float2half_rn(quant), hi = __hmul(z, n);
                                        // (an infinite one is in it already)
                                        y = isfinite(y) ? y - (__half2float(hi) + __half2float(__hfma(z, n, __hneg(hi)))) : 0.f;
                                    }
                                } else {
                                    const uint32_t u = *reinterpret_cast<const uint16_t*>(
                                        vt + (me >> 6) * (kTcTile * 128) + j * 128 + ((((me & 63) >> 3) ^ (j & 7)) << 4) + (me & 7) * 2);
                                    y = BF ? __uint_as_float(u << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(u)));
                                }
#pragma unroll
                                for (int i = 0; i < S; ++i) {
                                    const int q = c + i;
                                    const uint32_t h = *reinterpret_cast<const uint16_t*>(pt + p_byte(j, c0 + q));
                                    const uint32_t u = *reinterpret_cast<const uint16_t*>(pt + p_byte(j, N + c0 + q));
                                    const float ph = BF ? __uint_as_float(h << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(h)));
                                    const float pl = BF ? __uint_as_float(u << 16) : __half2float(__ushort_as_half(static_cast<uint16_t>(u)));
                                    const float pr = fmaf(pl, 1.f / kLowScale, ph);
                                    if (tb + j < qlen[q]) v[i] = fmaf(pr, y, v[i]);
                                }
                            }
                            tmem_store_n<S>(ocol + c, v);
                            if (!holds) {
                                const float zero[S] = {};
                                tmem_store_n<S>(ocol + N + c, zero);
                            }
                        }
                        tc_wait_st();
                        holds = true;
                        __syncwarp();
                        if (lane == 0) mbar_arrive(oddread);
                        await(oddread, odds++ & 1);  // V's rows are read by every group
                    }
                    if constexpr (!G::q8) {
                        if (grp == 0 && (gone || odd))
                            for (int c = 0; c < 16; ++c) *piece(c) = make_uint4(0, 0, 0, 0);
                    }
                }
                if (me == 0 && grp == 0) accum_sm[t % G::p_bufs] = holds;
                fence_proxy_async_smem();  // P and V, before the tensor cores read them
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(pfull + t % G::p_bufs);
                    if constexpr (G::q8) mbar_arrive(vempty + vs);
                }
                if (G::o_bufs == 2 && po) {  // the last item's outputs (with one buffer of P its products are waited for above)
                    if (G::p_bufs == 2) last_product();
                    drain(lanes + G::col_o + (k - 1) % 2 * (2 * N) + c0);
                }
            }
            if (stop) break;

            // ---- the item's partial
            const int64_t slot0 = (static_cast<int64_t>(it.a * p.kv_heads + it.g) * p.chunks + it.tok0 / p.chunk) * p.qp + q0;
            po = p.o + slot0 * D + me;
            left = it.nq - q0;
            if (G::o_bufs == 1) {
                last_product();
                drain(ocol);
            }
            tc_fence_before();
            const float r = reduce_columns<W>(l, 0.f, [](float a, float b) { return a + b; });
            if (lane < W) red[w4 * W + lane] = r;
            named_bar_sync(bar_id, 128);
            if (me < W && q0 + me < it.nq) {
                const float m = lim[me] == kNoMax ? kNoMax : sub[me];  // (as it was taken off, so that parts meet exactly)
                const float s = (red[me] + red[W + me]) + (red[2 * W + me] + red[3 * W + me]);
                *reinterpret_cast<float2*>(p.ml + (slot0 + me) * 2) = make_float2(m, s);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(qempty + (k & 1));
            named_bar_sync(bar_id, 128);  // (the sums and references are read)
        }
        if (po) {
            last_product();
            if (__all_sync(0xffffffffu, live)) drain(lanes + G::col_o + (k - 1) % 2 * (2 * N) + c0);
        }
        if (!live && me == 0) atomicOr(p.err, kErrTimeout);
    } else if (G::q8) {
        // ---------------------------------------------------------------- q8_0 to fp16: a token per thread, then a dim
        constexpr uint32_t kBar = 4;
        const int me = tid & 127, w4 = warp & 3;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(32 * w4) << 16);
        __half* dv = reinterpret_cast<__half*>(sm + G::off_dv);  // [2][4][128]
        const int slot = me & 63, key = q8_key(slot & 7);
        // K of tile i: a token per thread
        auto convert_k = [&](int i) {
            const int ks = i % G::k_slots;
            await_warp(kfull + ks, (i / G::k_slots) & 1);
            if (i > 0) await_warp(akfree, (i - 1) & 1);
            tc_fence_after();
            const uint8_t* kt = sm + ks * G::half + (me >> 6) * kQ8Half + slot * 128;
            uint4 row[8];  // (loaded before the first store to tensor memory, which the compiler may not load past)
#pragma unroll
            for (int c = 0; c < 8; ++c) row[c] = *reinterpret_cast<const uint4*>(kt + 16 * (c ^ key));
#pragma unroll
            for (int c = 0; c < 8; c += 2) {
                uint32_t out[16];
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint4 w = row[c + j];
                    const uint32_t u[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
#pragma unroll
                    for (int n = 0; n < 4; ++n) {
                        out[8 * j + 2 * n] = i8_to_h2(u[n], 0x4140u);
                        out[8 * j + 2 * n + 1] = i8_to_h2(u[n], 0x4342u);
                    }
                }
                tmem_st16(lanes + G::col_k + 8 * c, out);
            }
            tc_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(akfull);
                mbar_arrive(kempty + ks);
            }
        };
        int t = 0, k = 0;
        bool go = true;
        if (G::converters == 2 && warp < G::threads / 32 - 4) {  // K only
            for (int item = blockIdx.x; item < total && live; item += gridDim.x, ++k) {
                await_warp(qfull + (k & 1), (k >> 1) & 1);
                const int tok0 = item_sm[k & 1].tok0, end = item_sm[k & 1].end;
                __syncwarp();
                if (lane == 0) mbar_arrive(qempty + (k & 1));
                for (int tb = tok0; tb < end && live; tb += kTcTile, ++t) convert_k(t);
            }
            go = false;
        }
        for (int item = blockIdx.x; item < total && go; item += gridDim.x, ++k) {
            await(qfull + (k & 1), (k >> 1) & 1);
            const ItemRec it = item_sm[k & 1];
            if (G::converters == 1 && k == 0) convert_k(0);
            for (int tb = it.tok0; tb < it.end; tb += kTcTile, ++t) {
                // the next tile's K goes first: it is free to, while V waits for the last products
                if (G::converters == 1 && (tb + kTcTile < it.end || item + gridDim.x < total)) convert_k(t + 1);
                const int vs = t % G::v_slots;
                await(vfull + vs, (t / G::v_slots) & 1);
                const uint8_t* vt = sm + G::off_v + vs * G::half;
                // ---- V: normalised scales by token, then elements by dim
                const int tok = tb + me;
                const uint8_t* sc = vt + (me >> 6) * kQ8Half + 8192 + slot * 2;
                uint32_t d[4], w[4];
                bool odd = false;
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                    d[b] = *reinterpret_cast<const uint16_t*>(sc + b * 128);
                    w[b] = d[b] & 0x7FFFu;
                    odd |= (d[b] & 0x7C00u) == 0x7C00u;
                }
                const __half inv = scale_inverse(scale_exponent(largest_scale(w)));
                const bool none = vmiss[vs] != 0 || tok >= it.end || (odd && tok >= it.minlen);
                __half* dt = dv + (t & 1) * 4 * kTcTile;
#pragma unroll
                for (int b = 0; b < 4; ++b)
                    dt[b * kTcTile + me] = none ? __ushort_as_half(0) : __hmul(__ushort_as_half(static_cast<uint16_t>(d[b])), inv);
                uint4 row[8];
#pragma unroll
                for (int c = 0; c < 8; ++c) row[c] = *reinterpret_cast<const uint4*>(vt + (c >> 2) * kQ8Half + me * 64 + 16 * (c & 3));
                if (t > 0) await(avfree, (t - 1) & 1);
                if (bar_or(kBar, 128, !live)) {  // (also: the scales are written)
                    go = false;
                    break;
                }
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < 8; ++c) {  // 16 tokens
                    const uint4 w = row[c];
                    const uint4 s0 = *reinterpret_cast<const uint4*>(dt + w4 * kTcTile + 16 * c);
                    const uint4 s1 = *reinterpret_cast<const uint4*>(dt + w4 * kTcTile + 16 * c + 8);
                    const uint32_t u[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
                    const uint32_t s[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
                    uint32_t hi[8], lo[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const __half2 v = as_h2(i8_to_h2(u[i >> 1], (i & 1) ? 0x4342u : 0x4140u));
                        const __half2 h = __hmul2(v, as_h2(s[i]));
                        hi[i] = as_u32(h);
                        lo[i] = as_u32(__hfma2(v, as_h2(s[i]), __hneg2(h)));
                    }
                    tmem_st8(lanes + G::col_vh + 8 * c, hi);
                    tmem_st8(lanes + G::col_vl + 8 * c, lo);
                }
                tc_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(avfull);
                    mbar_arrive(vempty + vs);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(qempty + (k & 1));
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, G::cols);
}

template <int FMT, int N, int Q>
cudaError_t launch_attend_tc_one(const AttendLaunch& a, cudaStream_t s) {
    using G = TcGeo<FMT, N, Q>;
    static_assert(G::smem(kMaxAgents) <= kMaxShared);
    static Once once;
    const cudaError_t e = once.allow_shared(attend_partial_tc<FMT, N, Q>, a.device);
    if (e != cudaSuccess) return e;
    attend_partial_tc<FMT, N, Q><<<a.sms, G::threads, G::smem(a.p.agents), s>>>(a.map, a.p);
    return cudaGetLastError();
}

// The fewest queries a tile that take all of a sequence's, up to 48.
template <int FMT>
cudaError_t launch_attend_tc(const AttendLaunch& a, cudaStream_t s) {
    return a.max_q <= 16   ? launch_attend_tc_one<FMT, 16, 16>(a, s)
           : a.max_q <= 24 ? launch_attend_tc_one<FMT, 32, 24>(a, s)
           : a.max_q <= 32 ? launch_attend_tc_one<FMT, 32, 32>(a, s)
                           : launch_attend_tc_one<FMT, 48, 48>(a, s);
}

}  // namespace kv
}  // namespace qmm
