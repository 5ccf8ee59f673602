// attn.cu -- causal attention over packed sequences with grouped heads, forward and
// gradient: the attention core between the q|k|v and o projections.
//
// Sequence s owns the rows [seq_start[s], seq_start[s+1]) of q, k and v.  For a query
// row i of head h and the keys j <= i of its sequence (key head g = h / (heads / kv_heads)):
//   S = scale q_i . k_j,  lse_i = log sum_j exp S,  P = exp(S - lse_i),  o_i = sum_j P v_j
// and with the upstream gradient do:
//   delta_i = do_i . o_i,  dP = do_i . v_j,  dS = P (dP - delta_i)
//   dq_i = scale sum_j dS k_j,  dk_j = scale sum_{h in g, i} dS q_i,  dv_j = sum P do_i
#include <cmath>

#include "overlap.cuh"
#include "quant.cuh"

namespace pact {
namespace attn {

struct Params {
    const pact_bf16 *q, *k, *v, *o_in, *dout;
    int64_t ldq, ldk, ldv, ldo, lddo;
    pact_bf16 *o, *dq, *dk, *dv;
    int64_t lddq, lddk, lddv;
    float *lse;                 // [heads x M]
    float *delta, *lse2;        // [heads x M] scratch of the gradient: delta and lse log2(e)
    const int32_t *seq_start;
    int nseq, heads, kv_heads, M;
    float scale;
};

// ---------------------------------------------------------------- tiles and work items
constexpr int TILE = 128;          // queries and keys per tile (the MMA's M; its N for scores)
constexpr int BOX_BYTES = TILE * 128;   // a 64-column box of a tile, 128-byte swizzled rows
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.69314718055994531f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 2^x of a pair by the special-function units, which take 8 cycles a warp and value ...
__device__ __forceinline__ uint64_t ex2_pair(uint64_t x) {
    float a, b;
    f2_unpack(x, a, b);
    return f2_pack(ex2(a), ex2(b));
}
// ... and by the FP32 units: x = n + f with n the nearest whole number (adding 1.5 2^23
// rounds it into the low bits), 2^f by the polynomial of degree 4 with the least relative
// error on [-1/2, 1/2] (Remez exchange: 2.6e-6, under the BF16 rounding of a probability by
// a factor of 700), n added to the exponent.  Below -126 it gives about 2^-126.  A NaN would
// come out as a finite number (the maximum drops it, and n added to its bits would do the
// same); with NANS the maximum keeps it and 2^n enters as a factor.  dk and dv need that.  dq does
// not: P is NaN there only where the row's lse is, whose o and so delta are NaN too, and dS =
// P (dP - delta) with them (at 4 x 2048 tokens with heads of 64 NANS would cost dq 10 us of 349).
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
template <bool NANS>
__device__ __forceinline__ uint64_t ex2_fma(uint64_t x) {
    float a, b;
    f2_unpack(x, a, b);
    x = NANS ? f2_pack(max_nan(a, -126.0f), max_nan(b, -126.0f)) : f2_pack(fmaxf(a, -126.0f), fmaxf(b, -126.0f));
    const uint64_t magic = f2_pack(12582912.0f, 12582912.0f), minus = f2_pack(-12582912.0f, -12582912.0f);
    const uint64_t t = f2_add(x, magic), n = f2_add(t, minus);
    const uint64_t f = f2_fma(n, f2_pack(-1.0f, -1.0f), x);
    uint64_t y = f2_fma(f, f2_pack(0.00957010201f, 0.00957010201f), f2_pack(0.0559178603f, 0.0559178603f));
    y = f2_fma(f, y, f2_pack(0.240247448f, 0.240247448f));
    y = f2_fma(f, y, f2_pack(0.693121815f, 0.693121815f));
    y = f2_fma(f, y, f2_pack(0.999999261f, 0.999999261f));
    const uint64_t base = NANS ? f2_pack(1.0f, 1.0f) : y;
    const uint32_t lo = (uint32_t)base + ((uint32_t)t << 23), hi = (uint32_t)(base >> 32) + ((uint32_t)(t >> 32) << 23);
    const uint64_t scaled = (uint64_t)hi << 32 | lo;
    return NANS ? f2_mul(y, scaled) : scaled;
}
// Of EX2_PERIOD pairs, this many go to the FP32 units.  Gradients over 4 x 2048 tokens, cold L2, 24 and 8
// heads of 128: 390 us with none, 384 so, 388 with half of dq's, 396 with half of dk and dv's; 32
// and 8 heads of 64: 355, 349, 365, 367.  The forward gains nothing (heads of 128, 114 us with none,
// one or two, 120 with three).
constexpr int EX2_PERIOD = 8, EX2_BY_FMA_DQ = 2, EX2_BY_FMA_DKV = 1;

// 128 columns of a lane.
__device__ __forceinline__ void tmem_ld_row(uint32_t taddr, uint32_t (&r)[128]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        tmem_ld_32x32b_x32(taddr + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(r + 32 * i));
    tmem_ld_wait();
}
// Scores of a diagonal block: keys after the query become -infinity, in place, by a loop of
// its own (one block of many takes it, and the code of the others stays short).
__device__ __forceinline__ void mask_diagonal(uint32_t taddr, int row) {
#pragma unroll 1
    for (int i = 0; i < 128; i += 32) {
        if (!__any_sync(0xffffffffu, i + 31 > row)) continue;
        uint32_t a[32];
        tmem_ld_32x32b_x32(taddr + i, a);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 32; ++e)
            if (i + e > row) a[e] = 0xFF800000u;
        tmem_st_32x32b_x32(taddr + i, a);
    }
    tmem_st_wait();
}

__device__ __forceinline__ void tmem_st_32x32b_x8(uint32_t taddr, const uint32_t *v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
                 "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
                 : "memory");
}

// D (+)= A(tmem) . B(smem)^T, BF16 x BF16 -> FP32, K = 16: the rows of A are tensor-memory
// lanes, eight 32-bit columns hold its 16 BF16 values.
__device__ __forceinline__ void mma_bf16_ts(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate));
}

// One lane of a converged warp.  The MMA warps run as that one thread: the compiler knows
// such a branch to be uniform, and the operands of the MMAs cost few instructions.  Beside
// busy softmax warps a 128 x 128 x 16 MMA issues every 66 cycles this way, and only every 93
// with a lane predicate on each instruction (64 is the tensor core's rate).
__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(one));
    return one != 0;
}

// The K-major descriptor of 16 contraction columns (step s) of a [128 x D] tile, and the
// MN-major one of 16 contraction rows (the tile as the second operand of a product over
// its rows).
__device__ __forceinline__ uint64_t desc_cols(uint32_t tile, int s) {
    return smem_desc(tile + (s >> 2) * BOX_BYTES + (s & 3) * 32, 16, 1024, SW_128);
}
__device__ __forceinline__ uint64_t desc_rows(uint32_t tile, int s) {
    return smem_desc(tile + s * 2048, BOX_BYTES, 1024, SW_128);
}

// tmem (+)= X . Y^T over D columns of two [128 x D] tiles.
template <int D>
__device__ __forceinline__ void mma_cols(uint32_t tmem, uint32_t x, uint32_t y) {
    constexpr uint32_t idesc = idesc_bf16(TILE, TILE, false, false);
#pragma unroll
    for (int s = 0; s < D / 16; ++s) mma_bf16(tmem, desc_cols(x, s), desc_cols(y, s), idesc, s > 0);
}
// tmem (+)= A . Y: A [128 x 128] BF16 in tensor memory, Y a [128 x D] tile; steps [S0, S1) of 16
// contraction rows.
template <int D, int S0 = 0, int S1 = TILE / 16>
__device__ __forceinline__ void mma_rows(uint32_t tmem, uint32_t a, uint32_t y, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16(TILE, D, false, true);
#pragma unroll
    for (int s = S0; s < S1; ++s) mma_bf16_ts(tmem, a + 8 * s, desc_rows(y, s), idesc, accumulate || s > 0);
}

// A [128 x D] tile by TMA: column `x` of the map, rows from `row`.
template <int D>
__device__ __forceinline__ void load_tile(uint8_t *dst, const CUtensorMap *map, uint64_t *bar, int x, int row) {
#pragma unroll
    for (int b = 0; b < D / 64; ++b) tma_load_2d(dst + b * BOX_BYTES, map, bar, x + 64 * b, row);
}
// Zero the tile's rows from `row` on (a warp): rows of other sequences, which a product over
// the tile's rows would multiply by a zero probability; 0 times infinity or NaN is not zero.
template <int D>
__device__ __forceinline__ void clear_rows(uint8_t *tile, int row, int lane) {
    const uint32_t base = smem_u32(tile);
#pragma unroll 4
    for (int i = row * 128 + lane * 16; i < BOX_BYTES; i += 512)
#pragma unroll
        for (int b = 0; b < D / 64; ++b)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(base + b * BOX_BYTES + i), "r"(0) : "memory");
    fence_proxy_async_smem();
    __syncwarp();
}

// N accumulator columns (from `taddr`) of a warp's 32 lanes, each times its lane's f, as BF16 to the rows of
// dst (leading dimension ld, first column already added), rows from `rows` on left out.  A lane holds
// a row, so the values pass through 4 KiB of shared memory (16-byte chunk c of row r at
// c ^ (r % 8)): stores of whole 128-byte lines, four rows an instruction.
// Stored straight from the lanes, 32 rows an instruction, a tile took 4.4 us; this way 1.
template <int N>
__device__ __forceinline__ void store_rows(uint32_t taddr, float f, uint8_t *slab, pact_bf16 *dst, int64_t ld,
                                           int rows, int lane) {
    constexpr int C = N < 64 ? N : 64, CH = C / 8;   // columns at a time, their 16-byte chunks
    const uint32_t base = smem_u32(slab);
#pragma unroll
    for (int i = 0; i < N; i += C) {
#pragma unroll
        for (int k = 0; k < C; k += 32) {
            uint32_t a[32];
            tmem_ld_32x32b_x32(taddr + i + k, a);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
                uint32_t w[4];
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    w[q] = pack_bf16x2(__uint_as_float(a[e + 2 * q]) * f, __uint_as_float(a[e + 2 * q + 1]) * f);
                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                 base + lane * 128 + ((((k + e) >> 3) ^ (lane & 7)) << 4)),
                             "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                             : "memory");
            }
        }
        __syncwarp();
#pragma unroll
        for (int r0 = 0; r0 < 32; r0 += 32 / CH) {
            const int r = r0 + lane / CH, c = lane % CH;
            uint4 w;
            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                         : "r"(base + r * 128 + ((c ^ (r & 7)) << 4))
                         : "memory");
            if (r < rows) *reinterpret_cast<uint4 *>(dst + r * ld + i + 8 * c) = w;
        }
        __syncwarp();
    }
}

// The order of work.  Each sequence is cut into tiles of 1 << shift rows, and a tile's work grows with its
// place in the sequence (query tiles: later queries see more keys) or with the tiles behind it (key
// tiles).  Long work goes first, or a long sequence at the wrong end of a ragged batch keeps a
// few SMs busy when the others are done (8061 tokens in eight sequences of 1 to 2900, 12 and 2
// heads of 128, cold L2: forward 82 us in the order of the batch, 68 sorted, gradients 224 and
// 210).  Sorted are up to 32 sequences, one to a lane; more come in the order of the batch
// and pay that difference where they are as uneven.  Query tiles are sorted by their place over all
// sequences; key tiles one sequence after the other, the longest first, because all of a
// sequence's key tiles read its queries and output gradients, which then stay in L2 (gradients
// over 4 x 2048 tokens: 3% faster than sorted by place).
struct Tiles {
    int shift;    // 128 or 256 rows
    int pairs;    // pairs of units per tile (below)
    int slots;    // at least as many as there are tiles: each sequence rounds up by less than one
};

// The k-th tile in that order (a warp's lanes search together): sequence rows [b, b + len), tile x of it;
// false: there are no more.  BACK: the last tiles are the longest work, else the first.
template <bool BACK>
__device__ __forceinline__ bool find_tile(const Params &p, const Tiles &ts, int k, int lane, int *b, int *len, int *x) {
    auto start = [&](int i) { return min(max(p.seq_start[i], 0), p.M); };
    auto tiles = [&](int n) { return (n >> ts.shift) + ((n & ((1 << ts.shift) - 1)) != 0); };
    if (p.nseq <= 32) {
        int s = 0, n = 0;   // a sequence per lane
        if (lane < p.nseq) {
            s = start(lane);
            n = max(start(lane + 1) - s, 0);
        }
        const int count = tiles(n);
        int src, place;
        if (BACK) {
            // By place in the sequence: sum max(0, count - level) tiles lie at `level` or behind it; the k-th
            // is on the highest level whose sum exceeds k.
            auto sum = [&](int level) { return __reduce_add_sync(0xffffffffu, max(0, count - level)); };
            if (k >= sum(0)) return false;
            int lo = 0, hi = __reduce_max_sync(0xffffffffu, count);
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (sum(mid) > k) lo = mid;
                else hi = mid;
            }
            place = lo;
            const int nth = k - sum(lo + 1);   // of the sequences that reach this level
            const uint32_t reach = __ballot_sync(0xffffffffu, count > lo);
            src = __ffs(__ballot_sync(0xffffffffu, count > lo && __popc(reach & ((1u << lane) - 1)) == nth)) - 1;
        } else {
            // Longest sequence first; `before` counts the tiles of the longer ones.
            int before = 0;
            for (int i = 0; i < p.nseq; ++i) {
                const int other = __shfl_sync(0xffffffffu, count, i);
                if (other > count || (other == count && i < lane)) before += other;
            }
            const uint32_t mine = __ballot_sync(0xffffffffu, k >= before && k < before + count);
            if (mine == 0) return false;
            src = __ffs(mine) - 1;
            place = k - __shfl_sync(0xffffffffu, before, src);
        }
        *b = __shfl_sync(0xffffffffu, s, src);
        *len = __shfl_sync(0xffffffffu, n, src);
        *x = place;
        return true;
    }
    // Many sequences: the sequences one behind the other, sequence s in the slots from (start >> shift) + s on
    // (rounding up takes less than one more), found by a search of seq_start.
    const int slot = BACK ? ts.slots - 1 - k : k;
    auto first = [&](int i) { return (start(i) >> ts.shift) + i; };
    int lo = 0, n = p.nseq;
    while (n > 1) {
        const int step = (n + 31) / 32, i = lane * step;
        const uint32_t mask = __ballot_sync(0xffffffffu, i < n && first(lo + i) <= slot);
        const int j = mask ? 31 - __clz(mask) : 0;
        lo += j * step;
        n = min(step, n - j * step);
    }
    *b = start(lo);
    *len = max(start(lo + 1) - *b, 0);
    *x = slot - first(lo);
    return *x >= 0 && *x < tiles(*len);
}

// A unit is a 128-query tile of one query head.  A pair of units shares a key head: two heads of one tile,
// or, for an odd number of heads a group, any two that follow one another in a tile of 256 rows
// (one head a group: its two halves).  Work item `it`: the pairs of a tile side by side, their key
// heads within them.  Query tiles t0, t1 of heads h0, h1; t1 = t0 where there is no second.
struct __align__(16) Pair {
    int b, len, g, t0, t1, h0, h1;
    bool any, two;
};
__device__ __forceinline__ Pair find_pair(const Params &p, const Tiles &ts, int it, int lane) {
    Pair w;
    const int per = ts.pairs * p.kv_heads, k = it / per, pair = (it - k * per) / p.kv_heads, group = p.heads / p.kv_heads;
    w.g = it % p.kv_heads;
    w.b = w.len = 0;
    int x = 0;
    w.any = find_tile<true>(p, ts, k, lane, &w.b, &w.len, &x);
    x <<= ts.shift - 7;   // in tiles of 128
    const int tiles = (w.len + TILE - 1) / TILE, u = 2 * pair, hh = u % group, next = hh + 1 == group;
    w.t0 = x + u / group;
    w.h0 = w.g * group + hh;
    w.any = w.any && w.t0 < tiles;
    w.two = w.any && w.t0 + next < tiles;
    w.t1 = w.two ? w.t0 + next : w.t0;
    w.h1 = w.g * group + (next ? 0 : hh + 1);
    return w;
}

// The n-th pair the TMA warp planned, from two slots of shared memory in turn (a warp); `read` learns that
// it has been read.  any = false: no more.
__device__ __forceinline__ Pair planned_pair(const Pair *plan, uint64_t *planned, uint64_t *read, int n, int lane) {
    Pair w;
    if (!warp_all(mbar_wait(&planned[n & 1], (n >> 1) & 1))) {
        w.any = false;
        return w;
    }
    w = plan[n & 1];
    __syncwarp();
    if (lane == 0) mbar_arrive(&read[n & 1]);
    return w;
}

// Dynamic scheduling: a grid has a CTA for every work item, and a running CTA that runs out of work cancels
// the launch of the next pending one and takes over its item (clusterlaunchcontrol).  The
// items differ by a factor of 16 in length; handed out in turn they left the slowest SM
// with 58 blocks of 43 on average.
__device__ __forceinline__ void request_item(uint4 *response, uint64_t *bar) {
    mbar_arrive_expect_tx(bar, 16);
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
                     smem_u32(response)),
                 "r"(smem_u32(bar))
                 : "memory");
}
// The cancelled CTA's number, or -1 where none was left.
__device__ __forceinline__ int answered_item(const uint4 *response) {
    uint32_t x = 0, got;
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b128 r;\n\t"
        "ld.shared.b128 r, [%2];\n\t"
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, r;\n\t"
        "selp.u32 %1, 1, 0, p;\n\t"
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%0, _, _, _}, r;\n\t}"
        : "+r"(x), "=r"(got)
        : "r"(smem_u32(response))
        : "memory");
    return got ? (int)x : -1;
}

constexpr int SPLIT_THREADS = 384;   // three warpgroups; registers are moved to the first two
__device__ __forceinline__ void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 216;"); }
__device__ __forceinline__ void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 72;"); }
static_assert(2 * 128 * 216 + 128 * 72 <= SPLIT_THREADS * 168, "more registers than the block is launched with");

// ------------------------------------------------------------------------- forward
// A CTA computes pairs of units that share a key head; K and V tiles are loaded once for both, and the
// tensor core runs one unit's products while the other's softmax runs:
//   warps 0-3, 4-7   softmax of unit 0, 1: a thread owns a query row (a tensor-memory lane),
//                    so maximum and sum need no exchange.  P overwrites the scores as BF16 and
//                    is the next product's operand from tensor memory; the product starts on
//                    its first 64 keys while the rest is computed.
//   warp 8           the plan, and TMA: the two Q tiles, then K and V tiles through a ring
//   warp 9           the MMAs, in the order  P0 V(j), S0(j+1), P1 V(j), S1(j+1)
// The running maximum and sum are those of the online softmax (Milakov and Gimelshein, 2018).  The
// accumulator is rescaled only when a row's maximum grew by more than 2^8 since the last time
// (any factor cancels in O / l; FP32 has the room), which is rare after the first block; this, and
// exponentials on the FP32 units in the gradients, are published for attention on this
// generation of GPUs.  S(j+1) is issued behind P V(j), so a unit that sees its scores ready
// also knows its accumulator at rest.  The CTA is persistent: the next pair's Q, K and scores
// come under the last pair's output.
// Rounding: P to BF16, as the MMA takes it (by at most 2^-8 of a probability); the row sums add the FP32 values.
// 4 x 2048 tokens, 24 and 8 heads of 128: 118 to 122 us, some 860 TFLOP/s of the 103 GFLOP under the
// diagonal (52% of the measured BF16 rate); 32 and 8 heads of 64: 131 us, 524 TFLOP/s.  At D = 128 a block of a
// pair takes 3000 cycles for 2048 of MMAs: a unit's softmax takes 1500 (1024 of them the
// special-function units'), and with two units in tensor memory it is not wholly under the other's
// products.  Those blocks, 45 an SM, are 71% of the cycles that an SM is active (the tensor pipe is
// active in 48%); the rest is what comes once a pair: its first loads and scores, the mask of the diagonal
// block, the output.  It has not been taken apart.  Tried without gain: sixteen softmax warps, two threads a row that
// exchange their maxima (3% slower), and with them a share of the exponentials on the FP32 units (more so).
namespace fwd {
constexpr int STAGES = 4;
template <int D>
struct Layout {
    static constexpr int TILE_BYTES = D / 64 * BOX_BYTES;
    static constexpr int SMEM = 1024 + (2 + STAGES) * TILE_BYTES + 8 * 4096 + 512;   // ... a slab per softmax warp
};

template <int D>
__global__ void __launch_bounds__(SPLIT_THREADS, 1)
k_attn_fwd(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
           const __grid_constant__ CUtensorMap tmV, const Params p, const Tiles ts) {
    constexpr int TILE_BYTES = Layout<D>::TILE_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *ring = smem + 2 * TILE_BYTES, *slabs = ring + STAGES * TILE_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(slabs + 8 * 4096);
    uint64_t *full = bars, *empty = bars + STAGES, *q_full = bars + 2 * STAGES, *q_empty = q_full + 1, *tail = q_full + 2;
    uint64_t *s_full = tail + 1, *o_full = s_full + 2, *p_ready = o_full + 2, *o_empty = p_ready + 4;
    uint64_t *read = o_empty + 2, *planned = read + 2, *answered = planned + 2;
    Pair *plan = reinterpret_cast<Pair *>(answered + 1 + ((answered + 1 - bars) & 1));   // two; 16-byte aligned
    uint4 *response = reinterpret_cast<uint4 *>(plan + 2);
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(response + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (uint64_t *b = bars; b < p_ready; ++b) mbar_init(b, 1);
        for (uint64_t *b = p_ready; b < read; ++b) mbar_init(b, 4);       // four warps each
        for (uint64_t *b = read; b < planned; ++b) mbar_init(b, 9);       // the MMA warp and the softmax warps
        for (uint64_t *b = planned; b <= answered; ++b) mbar_init(b, 1);
        fence_barrier_init();
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // all 512 columns are the block's, so they start at 0: S0, S1 (128 each), then O0, O1 (D each)
    constexpr uint32_t tmem = 0;
    pdl_wait();

    if (warp >= 8) {
        regs_down();
        if (warp == 8) {
            uint32_t stage = 0, phase = 0;
            int issued = 0, done = 0, tails = 0;   // ring loads, work items, last V tiles
            bool ok = true;
            int asked = 0;
            auto ask = [&] {
                if (lane == 0) request_item(response, answered);
                ++asked;
            };
            auto answer = [&] {
                if (!(ok = warp_all(mbar_wait(answered, (asked - 1) & 1)))) return -1;
                const int it = answered_item(response);
                fence_proxy_async_smem();   // the next answer is written by the async proxy
                __syncwarp();
                return it;
            };
            for (int it = blockIdx.x; ok;) {
                Pair w;
                w.any = false;
                while (it >= 0 && ok && !(w = find_pair(p, ts, it, lane)).any) {   // slots without work
                    ask();
                    it = answer();
                }
                if (!ok || !(ok = warp_all(mbar_wait(&read[done & 1], ((done >> 1) & 1) ^ 1)))) break;
                if (lane == 0) {
                    plan[done & 1] = w;
                    mbar_arrive(&planned[done & 1]);
                }
                if (!w.any || !(ok = warp_all(mbar_wait(q_empty, (done & 1) ^ 1)))) break;
                ++done;
                if (lane == 0) {
                    mbar_arrive_expect_tx(q_full, (w.two ? 2 : 1) * TILE_BYTES);
                    load_tile<D>(smem, &tmQ, q_full, w.h0 * D, w.b + w.t0 * TILE);
                    if (w.two) load_tile<D>(smem + TILE_BYTES, &tmQ, q_full, w.h1 * D, w.b + w.t1 * TILE);
                }
                // the next item is asked for two blocks before the last loads: early enough for its plan to
                // wait for the other warps, late enough for the items to go where there is room
                const int loads = 2 * (w.t1 + 1), ask_at = max(0, loads - 4);
                for (int i = 0; i < loads && ok; ++i) {   // K(0), V(0), K(1), ...
                    if (i == ask_at) ask();
                    if (!(ok = warp_all(mbar_wait(&empty[stage], phase ^ 1)))) break;
                    const int row = w.b + (i >> 1) * TILE, rows = w.len - (i >> 1) * TILE;
                    uint8_t *dst = ring + stage * TILE_BYTES;
                    if ((i & 1) && rows < TILE) {   // the sequence's last V tile
                        if (lane == 0) {
                            mbar_arrive_expect_tx(tail, TILE_BYTES);
                            load_tile<D>(dst, &tmV, tail, w.g * D, row);
                        }
                        if (!(ok = warp_all(mbar_wait(tail, tails++ & 1)))) break;
                        clear_rows<D>(dst, rows, lane);
                        if (lane == 0) mbar_arrive(&full[stage]);
                    } else if (lane == 0) {
                        mbar_arrive_expect_tx(&full[stage], TILE_BYTES);
                        load_tile<D>(dst, i & 1 ? &tmV : &tmK, &full[stage], w.g * D, row);
                    }
                    ++issued;
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (ok) it = answer();
            }
            // every copy and answer lands before the CTA may leave
            if (asked) mbar_wait(answered, (asked - 1) & 1);
            if (done) mbar_wait(q_full, (done - 1) & 1);
            for (int s = 0; s < STAGES && s < issued; ++s) mbar_wait(&full[s], ((issued - 1 - s) / STAGES) & 1);
        } else if (warp == 9) {
            const uint32_t q0 = smem_u32(smem), q1 = q0 + TILE_BYTES, r0 = smem_u32(ring);
            const uint32_t S0 = tmem, S1 = tmem + TILE, O0 = tmem + 2 * TILE, O1 = O0 + D;
            bool ok = true;
            int done = 0, done1 = 0, load = 0, c0 = 0, c1 = 0;   // items, items with a second unit, ring loads, blocks
            while (ok) {
                const Pair w = planned_pair(plan, planned, read, done, lane);
                if (!w.any) break;
                const int t0 = w.t0, t1 = w.t1, blocks = t1 + 1;
                const bool two = w.two;
                if (elect_one()) {
                    ok = mbar_wait(q_full, done & 1) && mbar_wait(&full[load % STAGES], (load / STAGES) & 1);
                    tc_fence_after();
                    if (ok) {
                        const uint32_t k = r0 + load % STAGES * TILE_BYTES;
                        mma_cols<D>(S0, q0, k);
                        tc_commit(&s_full[0]);
                        if (two) {
                            mma_cols<D>(S1, q1, k);
                            tc_commit(&s_full[1]);
                        }
                        tc_commit(&empty[load % STAGES]);
                        if (blocks == 1) tc_commit(q_empty);
                    }
                    for (int j = 0; j < blocks && ok; ++j) {
                        const int vi = load + 2 * j + 1, ki = vi + 1, vs = vi % STAGES, ks = ki % STAGES;
                        const bool more0 = j < t0, more1 = two && j < t1;   // another block after this one
                        if (!(ok = mbar_wait(&full[vs], (vi / STAGES) & 1))) break;
                        if (j <= t0) {
                            // the unit's last output has left its accumulator
                            if (j == 0 && !(ok = mbar_wait(&o_empty[0], (done & 1) ^ 1))) break;
                            if (!(ok = mbar_wait(&p_ready[0], (c0 + j) & 1))) break;
                            tc_fence_after();
                            mma_rows<D, 0, 4>(O0, S0, r0 + vs * TILE_BYTES, j > 0);
                            if (!(ok = mbar_wait(&p_ready[1], (c0 + j) & 1))) break;
                            tc_fence_after();
                            mma_rows<D, 4, 8>(O0, S0, r0 + vs * TILE_BYTES, true);
                            if (!more0) tc_commit(&o_full[0]);
                        }
                        if (more0 || more1) {
                            if (!(ok = mbar_wait(&full[ks], (ki / STAGES) & 1))) break;
                            tc_fence_after();
                        }
                        if (more0) {
                            mma_cols<D>(S0, q0, r0 + ks * TILE_BYTES);
                            tc_commit(&s_full[0]);
                        }
                        if (two) {
                            if (j == 0 && !(ok = mbar_wait(&o_empty[1], (done1 & 1) ^ 1))) break;
                            if (!(ok = mbar_wait(&p_ready[2], (c1 + j) & 1))) break;
                            tc_fence_after();
                            mma_rows<D, 0, 4>(O1, S1, r0 + vs * TILE_BYTES, j > 0);
                            if (!(ok = mbar_wait(&p_ready[3], (c1 + j) & 1))) break;
                            tc_fence_after();
                            mma_rows<D, 4, 8>(O1, S1, r0 + vs * TILE_BYTES, true);
                            if (!more1) tc_commit(&o_full[1]);
                        }
                        tc_commit(&empty[vs]);
                        if (more1) {
                            mma_cols<D>(S1, q1, r0 + ks * TILE_BYTES);
                            tc_commit(&s_full[1]);
                        }
                        if (more0 || more1) {
                            tc_commit(&empty[ks]);
                            if (j + 2 == blocks) tc_commit(q_empty);   // the last scores are issued
                        }
                    }
                }
                ok = warp_all(ok);
                ++done;
                done1 += two;
                load += 2 * blocks;
                c0 += t0 + 1;
                if (two) c1 += t1 + 1;
            }
        }
    } else {
        regs_up();
        const int u = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // this warp's 32 tensor-memory lanes
        const uint32_t S = tmem + u * TILE + lanes, O = tmem + 2 * TILE + u * D + lanes;
        const float c = p.scale * LOG2E;
        bool ok = true;
        int done = 0, seen = 0;   // work items and blocks of this unit
        for (int n = 0; ok; ++n) {
            const Pair w = planned_pair(plan, planned, read, n, lane);
            if (!w.any) break;
            if (u && !w.two) continue;
            const int t = u ? w.t1 : w.t0;
            float m = -INFINITY, l = 0.0f;   // reference of the exponentials (times c), row sum
            for (int j = 0; j <= t && ok; ++j, ++seen) {
                if (!(ok = warp_all(mbar_wait(&s_full[u], seen & 1)))) break;
                tc_fence_after();
                if (j == t) mask_diagonal(S, row);
                uint32_t r[128];
                tmem_ld_row(S, r);
                float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int e = 0; e < 128; e += 2)
                    mx[(e >> 1) & 3] = max3(mx[(e >> 1) & 3], __uint_as_float(r[e]), __uint_as_float(r[e + 1]));
                const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
                if (j == 0) {
                    m = top;
                } else {
                    const bool grew = top > m + 8.0f;
                    if (__any_sync(0xffffffffu, grew)) {
                        const float f = grew ? ex2(m - top) : 1.0f;
                        if (grew) m = top;
                        l *= f;
#pragma unroll 1
                        for (int i = 0; i < D / 16; ++i) {
                            uint32_t a[16];
                            tmem_ld_32x32b_x16(O + 16 * i, a);
                            tmem_ld_wait();
#pragma unroll
                            for (int e = 0; e < 16; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * f);
                            tmem_st_32x32b_x16(O + 16 * i, a);
                        }
                    }
                }
                const uint64_t c2 = f2_pack(c, c), m2 = f2_pack(-m, -m);
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 2; ++i) {   // keys 0-63, 64-127: the first product starts on the first half
                    uint32_t w[32];
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const uint64_t x = f2_fma((uint64_t)r[64 * i + 2 * e + 1] << 32 | r[64 * i + 2 * e], c2, m2);
                        const uint64_t y = ex2_pair(x);
                        sum[e & 1] = f2_add(sum[e & 1], y);
                        float y0, y1;
                        f2_unpack(y, y0, y1);
                        w[e] = pack_bf16x2(y0, y1);
                    }
                    tmem_st_32x32b_x32(S + 32 * i, w);
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&p_ready[2 * u + i]);
                }
                float s0, s1;
                f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
                l += s0 + s1;
            }
            if (!ok || !(ok = warp_all(mbar_wait(&o_full[u], done & 1)))) break;
            ++done;
            tc_fence_after();
            const int q0 = t * TILE + (warp & 3) * 32, h = u ? w.h1 : w.h0;   // the warp's first query
            store_rows<D>(O, 1.0f / l, slabs + warp * 4096, p.o + (int64_t)(w.b + q0) * p.ldo + (int64_t)h * D, p.ldo,
                          w.len - q0, lane);
            tc_fence_before();
            if (lane == 0) mbar_arrive(&o_empty[u]);
            if (q0 + lane < w.len) p.lse[(int64_t)h * p.M + w.b + q0 + lane] = fmaf(m, LN2, logf(l));
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 9) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}
}  // namespace fwd

// ------------------------------------------------------------------ gradient of q
// The same pairs of units as the forward, sharing K and V.  A unit keeps one 128-column
// region of tensor memory that holds S, then dP (once S is in registers), then dS as
// BF16, the operand of dQ += dS K; so two units and their accumulators fill the 512
// columns.  The exponentials of one unit run under the other's products:
//   S0 S1 | dP0 dP1 | dQ0 S0(j+1) dQ1 S1(j+1) | ...
// dq has a kernel of its own, with S and dP formed a second time for dk and dv (7 products
// instead of 5): summing dq over key tiles from one kernel takes atomics in FP32, whose
// order would change the result from call to call, and a pass to clear and round it.
// This kernel also leaves delta and lse log2(e) for the other one, which is launched while this one
// runs, loads its first tiles and waits with those two alone (some 2 us a call).
// Rounding: dS to BF16, as the MMA takes it; P, dP and the sums stay FP32.
// 4 x 2048 tokens, 24 and 8 heads of 128, alone with a cold L2: 190 us (three products, 155 GFLOP: 49% of the
// measured BF16 rate).  A block of a pair takes 4700 cycles for 48 MMAs of 64; the tensor core waits for
// dS, 1400 cycles after dP.  The blocks are 71% of an SM's active cycles; the rest is what a CTA does once
// (set-up, first tiles, delta, output), five CTAs an SM one after the other.  P beside dP exceeds the 104
// registers a thread: 52 bytes are spilled and 68 read back a block at D = 128, 32 and 48 at D = 64.
// Tried without gain: persistent CTAs (V's memory is needed to pass the output on), MMA waits
// moved ahead, dO for delta from its tile.
// The gradient kernels' softmax needs no exchange between the columns of a row (lse is known), so
// four warpgroups do it: four warps a scheduler hide one another's latencies, where two left
// the schedulers idle two cycles in three.
constexpr int GRAD_WARPS = 16, GRAD_THREADS = 32 * GRAD_WARPS + 128;
__device__ __forceinline__ void grad_regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 104;"); }
__device__ __forceinline__ void grad_regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 64;"); }
static_assert(512 * 104 + 128 * 64 <= GRAD_THREADS * 96, "more registers than the block is launched with");

// tmem (+)= A . Y over steps [S0, S1) of 16 contraction rows: the BF16 values of a step (8 columns)
// lie over the first half of the 16 FP32 columns they were computed from.
template <int D, int S0, int S1>
__device__ __forceinline__ void mma_spread(uint32_t tmem, uint32_t a, uint32_t y, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16(TILE, D, false, true);
#pragma unroll
    for (int s = S0; s < S1; ++s) mma_bf16_ts(tmem, a + 16 * s, desc_rows(y, s), idesc, accumulate || s > 0);
}
__device__ __forceinline__ uint32_t pack_pair(uint64_t v) {
    float x, y;
    f2_unpack(v, x, y);
    return pack_bf16x2(x, y);
}

namespace dq {
template <int D>
struct Layout {
    static constexpr int TILE_BYTES = D / 64 * BOX_BYTES;
    static constexpr int DELTA = 7 * TILE_BYTES;                // Q0 Q1 dO0 dO1, K twice, V
    static constexpr int BARS = DELTA + 2 * TILE * 4;           // delta of both units
    static constexpr int SMEM = 1024 + BARS + 256;
};

template <int D>
__global__ void __launch_bounds__(GRAD_THREADS, 1)
k_attn_dq(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
          const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params p,
          const Tiles ts) {
    constexpr int TB = Layout<D>::TILE_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *sk = smem + 4 * TB, *sv = smem + 6 * TB;
    float *s_delta = reinterpret_cast<float *>(smem + Layout<D>::DELTA);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Layout<D>::BARS);
    uint64_t *q_full = bars, *tail = bars + 1, *v_full = bars + 2, *v_empty = bars + 3, *k_full = bars + 4,
             *k_empty = bars + 6, *s_full = bars + 8, *dp_full = bars + 10, *dq_full = bars + 12,
             *s_read = bars + 14, *ds_ready = bars + 16;   // ds_ready: [unit][keys 0-63, 64-127]
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 20);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 20; ++i) mbar_init(&bars[i], i >= 14 ? GRAD_WARPS / 2 : 1);
        fence_barrier_init();
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmG);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    pdl_wait();
    // The next kernel may take up its CTAs as this one's leave: what it reads before it waits for this one
    // was complete here.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    const Pair w = find_pair(p, ts, blockIdx.x, lane);
    if (!w.any) return;   // block-uniform, before tensor memory is allocated
    const int b = w.b, len = w.len, g = w.g, t0 = w.t0, t1 = w.t1, h0 = w.h0, h1 = w.h1;
    const bool two = w.two;
    const int blocks = t1 + 1;

    if (warp == GRAD_WARPS + 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // all 512 columns, from 0: two regions of 128, then dQ0, dQ1 (D each)
    constexpr uint32_t tmem = 0;

    if (warp >= GRAD_WARPS) {
        grad_regs_down();
        if (warp == GRAD_WARPS) {
            if (lane == 0) {
                mbar_arrive_expect_tx(q_full, (two ? 4 : 2) * TB);
                load_tile<D>(smem, &tmQ, q_full, h0 * D, b + t0 * TILE);
                load_tile<D>(smem + 2 * TB, &tmG, q_full, h0 * D, b + t0 * TILE);
                if (two) {
                    load_tile<D>(smem + TB, &tmQ, q_full, h1 * D, b + t1 * TILE);
                    load_tile<D>(smem + 3 * TB, &tmG, q_full, h1 * D, b + t1 * TILE);
                }
            }
            bool ok = true;
            int nk = 0, nv = 0;
            for (int j = 0; j < blocks; ++j) {
                const int row = b + j * TILE, rows = len - j * TILE;
                uint8_t *dst = sk + (j & 1) * TB;
                if (!(ok = warp_all(mbar_wait(&k_empty[j & 1], ((j >> 1) & 1) ^ 1)))) break;
                const bool partial = rows < TILE;   // the sequence's last K tile
                uint64_t *kb = partial ? tail : &k_full[j & 1];
                if (lane == 0) {
                    mbar_arrive_expect_tx(kb, TB);
                    load_tile<D>(dst, &tmK, kb, g * D, row);
                }
                const bool v_free = warp_all(mbar_wait(v_empty, (j & 1) ^ 1));
                if (v_free && lane == 0) {
                    mbar_arrive_expect_tx(v_full, TB);
                    load_tile<D>(sv, &tmV, v_full, g * D, row);
                }
                nv += v_free;
                if (partial) {
                    if (!(ok = warp_all(mbar_wait(tail, 0)))) break;
                    clear_rows<D>(dst, rows, lane);
                    if (lane == 0) mbar_arrive(&k_full[j & 1]);
                }
                ++nk;
                ok = v_free;
                if (!ok) break;
            }
            // every copy lands before the CTA may leave
            mbar_wait(q_full, 0);
            if (nk > 0) mbar_wait(&k_full[(nk - 1) & 1], ((nk - 1) >> 1) & 1);
            if (nk > 1) mbar_wait(&k_full[nk & 1], ((nk - 2) >> 1) & 1);
            if (nv > 0) mbar_wait(v_full, (nv - 1) & 1);
        } else if (warp == GRAD_WARPS + 1 && elect_one()) {
            const uint32_t base = smem_u32(smem), k0 = smem_u32(sk), v0 = smem_u32(sv);
            bool ok = mbar_wait(q_full, 0) && mbar_wait(&k_full[0], 0);
            tc_fence_after();
            if (ok) {
                mma_cols<D>(tmem, base, k0);
                tc_commit(&s_full[0]);
                if (two) {
                    mma_cols<D>(tmem + TILE, base + TB, k0);
                    tc_commit(&s_full[1]);
                }
            }
            for (int j = 0; j < blocks && ok; ++j) {
                if (!(ok = mbar_wait(v_full, j & 1))) break;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (u ? !two : j > t0) continue;
                    if (!(ok = mbar_wait(&s_read[u], j & 1))) break;
                    tc_fence_after();
                    mma_cols<D>(tmem + u * TILE, base + (2 + u) * TB, v0);
                    tc_commit(&dp_full[u]);
                }
                if (!ok) break;
                tc_commit(v_empty);
                const uint32_t kj = k0 + (j & 1) * TB, kn = k0 + ((j + 1) & 1) * TB;
                bool next = false;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    if (u ? !two : j > t0) continue;
                    if (!(ok = mbar_wait(&ds_ready[2 * u], j & 1))) break;
                    tc_fence_after();
                    mma_spread<D, 0, 4>(tmem + 2 * TILE + u * D, tmem + u * TILE, kj, j > 0);
                    if (!(ok = mbar_wait(&ds_ready[2 * u + 1], j & 1))) break;
                    tc_fence_after();
                    mma_spread<D, 4, 8>(tmem + 2 * TILE + u * D, tmem + u * TILE, kj, true);
                    if (j == (u ? t1 : t0)) {
                        tc_commit(&dq_full[u]);
                        continue;
                    }
                    if (!next) {
                        if (!(ok = mbar_wait(&k_full[(j + 1) & 1], ((j + 1) >> 1) & 1))) break;
                        tc_fence_after();
                        next = true;
                    }
                    mma_cols<D>(tmem + u * TILE, base + u * TB, kn);
                    tc_commit(&s_full[u]);
                }
                if (ok) tc_commit(&k_empty[j & 1]);
            }
        }
    } else {
        grad_regs_up();
        const int u = warp >> 3, half = (warp >> 2) & 1, row = threadIdx.x & 127;
        const int t = u ? t1 : t0, h = u ? h1 : h0, last = u && !two ? -1 : t;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;
        // this warp's lanes; its columns are 32 half .. + 31 of both 64-key halves of a block
        const uint32_t X = tmem + u * TILE + half * 32 + lanes;
        const int q0 = t * TILE + (warp & 3) * 32;                // the warp's first query
        float delta = 0.0f, lse2 = 0.0f;
        if (last >= 0) {
            const int64_t stat = (int64_t)h * p.M + b + q0 + lane;
            if (q0 + lane < len) lse2 = p.lse[stat] * LOG2E;
            // delta of 16 of the 32 rows (the other half's warp sums the rest), D / 8 lanes a row:
            // whole rows of o and do at a time
            constexpr int L = D / 8, R = 32 / L, N = 16 / R;   // lanes a row, rows a load, loads
            const pact_bf16 *po = p.o_in + (int64_t)h * D + (lane % L) * 8, *pd = p.dout + (int64_t)h * D + (lane % L) * 8;
            uint4 x[N], y[N];
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int r = half * 16 + i * R + lane / L;
                const int64_t at = b + q0 + r;
                x[i] = y[i] = make_uint4(0, 0, 0, 0);
                if (q0 + r < len) {
                    x[i] = *reinterpret_cast<const uint4 *>(po + at * p.ldo);
                    y[i] = *reinterpret_cast<const uint4 *>(pd + at * p.lddo);
                }
            }
            float *sd = s_delta + u * TILE + (warp & 3) * 32;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                float u8[8], v8[8], s = 0.0f;
                unpack8_bf16(x[i], u8);
                unpack8_bf16(y[i], v8);
#pragma unroll
                for (int e = 0; e < 8; ++e) s = fmaf(u8[e], v8[e], s);
#pragma unroll
                for (int o = L / 2; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
                if (lane % L == 0) sd[half * 16 + i * R + lane / L] = s;
            }
            asm volatile("bar.sync %0, 256;" ::"r"(1 + u) : "memory");   // the unit's eight warps
            delta = sd[lane];
            if (half == 0 && q0 + lane < len) {
                p.delta[stat] = delta;
                p.lse2[stat] = lse2;
            }
        }
        const float c = p.scale * LOG2E;
        const uint64_t c2 = f2_pack(c, c), m2 = f2_pack(-lse2, -lse2), d2 = f2_pack(-delta, -delta);
        bool ok = true;
        for (int j = 0; j <= last && ok; ++j) {
            if (!(ok = warp_all(mbar_wait(&s_full[u], j & 1)))) break;
            tc_fence_after();
            uint32_t r[64];
            tmem_ld_32x32b_x32(X, *reinterpret_cast<uint32_t(*)[32]>(r));
            tmem_ld_32x32b_x32(X + 64, *reinterpret_cast<uint32_t(*)[32]>(r + 32));
            tmem_ld_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&s_read[u]);
            uint64_t pr[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const uint64_t x = f2_fma((uint64_t)r[2 * e + 1] << 32 | r[2 * e], c2, m2);
                pr[e] = e % EX2_PERIOD < EX2_BY_FMA_DQ ? ex2_fma<false>(x) : ex2_pair(x);
            }
            if (!(ok = warp_all(mbar_wait(&dp_full[u], j & 1)))) break;
            tc_fence_after();
            const int n = row - half * 32;
#pragma unroll
            for (int i = 0; i < 4; ++i) {   // 16 columns at a time: the registers hold no more
                const int c0 = 64 * (i >> 1) + 16 * (i & 1);
                uint32_t a[16], w[8];
                tmem_ld_32x32b_x16(X + c0, a);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    pr[8 * i + e] = f2_mul(pr[8 * i + e], f2_add((uint64_t)a[2 * e + 1] << 32 | a[2 * e], d2));
                if (j == t) {   // the diagonal block: keys after the query
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float x, y;
                        f2_unpack(pr[8 * i + e], x, y);
                        pr[8 * i + e] = f2_pack(c0 + 2 * e > n ? 0.0f : x, c0 + 2 * e + 1 > n ? 0.0f : y);
                    }
                }
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = pack_pair(pr[8 * i + e]);
                tmem_st_32x32b_x8(X + c0, w);
                if (i & 1) {
                    tmem_st_wait();
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ds_ready[2 * u + (i >> 1)]);
                }
            }
        }
        ok = last >= 0 && ok && warp_all(mbar_wait(&dq_full[u], 0));
        if (ok) {
            tc_fence_after();
            // half of the columns each; the unit's Q and dO tiles are no longer read and pass the
            // output on
            const int col = half * (D / 2);
            store_rows<D / 2>(tmem + 2 * TILE + u * D + col + lanes, p.scale, smem + (u + 2 * half) * TB + (warp & 3) * 4096,
                              p.dq + (int64_t)(b + q0) * p.lddq + (int64_t)h * D + col, p.lddq, len - q0, lane);
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == GRAD_WARPS + 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}
}  // namespace dq

// ------------------------------------------------------------- gradients of k and v
// A CTA owns a tile of 128 keys of one key head and runs over the query tiles at and
// after it, of every query head of the group: the group's sum stays in tensor memory.
// Everything is transposed (rows are keys), so P^T and dS^T come out of the softmax warps
// as the left operands, in tensor memory, of dV += P^T dO and dK += dS^T Q, and dO and Q
// serve as both operands of their two products from one copy in shared memory.
// 512 columns: S^T | dP^T | dV | dK; P^T and dS^T lie over S^T and dP^T.  Order of the MMAs:
//   dV(n) S(n+1) | dK(n) dP(n+1): the exponentials of n+1 run under the second pair.
// Four warpgroups share the columns: warps 4 w .. 4 w + 3 take queries 16 w .. 16 w + 15 of both halves of a tile.
// Rounding: P and dS to BF16, as the MMA takes them.
// 4 x 2048 tokens, 24 and 8 heads of 128, alone with a cold L2: 186 us (four products, 206 GFLOP: 67% of the
// measured BF16 rate); with dq's kernel 380 to 400 a call.  The units are 80% of an SM's active cycles.  A
// unit takes 2530 cycles for 2048 of MMAs: P (1220, of them 900 the special-function units') and dV, S(n+1)
// behind it follow one another, as D = 128 leaves no tensor memory for a second S.  A second S at D = 64
// and a third Q slot changed nothing (P and dS then follow one another without a gap, in the same time).
namespace dkv {
template <int D>
struct Layout {
    static constexpr int TILE_BYTES = D / 64 * BOX_BYTES;
    static constexpr int STATS = 6 * TILE_BYTES;               // K, V, Q twice, dO twice
    static constexpr int BARS = STATS + 2 * 2 * TILE * 4;      // lse2 and delta of two units
    static constexpr int SMEM = 1024 + BARS + 256;
};

// Pairs of a masked tile: columns before `first` or from `end` on become zero.
__device__ __forceinline__ void clear_edge(uint64_t (&v)[8], int first, int end) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        float x, y;
        f2_unpack(v[e], x, y);
        if (2 * e < first || 2 * e >= end) x = 0.0f;
        if (2 * e + 1 < first || 2 * e + 1 >= end) y = 0.0f;
        v[e] = f2_pack(x, y);
    }
}

// The group's query heads over a cluster of `ns` CTAs: each left its FP32 sums (dv, dk: [128 x D],
// 16-byte chunk c of row r at c ^ (r % 8)) in its own shared memory at `part`; CTA `rank` adds its
// share of the rows over the CTAs in order and stores them.
template <int D>
__device__ __forceinline__ void join(const Params &p, uint32_t part, int ns, int rank, int b, int len, int t, int g) {
    constexpr int CH = D / 8;   // 8 columns a thread
    const int rows = TILE / ns;
    for (int i = threadIdx.x; i < 2 * rows * CH; i += GRAD_THREADS) {
        const int c = i % CH, r = rank * rows + i / CH % rows, kj = t * TILE + r;
        const bool is_k = i / (CH * rows) != 0;
        if (kj >= len) continue;
        float v[8] = {};
        for (int q = 0; q < ns; ++q) {
            const uint32_t base = mapa_shared(part + ((is_k ? TILE : 0) + r) * D * 4, q);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                float x[4];
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
                             : "r"(base + (((2 * c + h) ^ (r & 7)) << 4))
                             : "memory");
#pragma unroll
                for (int e = 0; e < 4; ++e) v[4 * h + e] += x[e];
            }
        }
        const float f = is_k ? p.scale : 1.0f;
        pact_bf16 *dst = (is_k ? p.dk + (int64_t)(b + kj) * p.lddk : p.dv + (int64_t)(b + kj) * p.lddv) + (int64_t)g * D + 8 * c;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(v[0] * f, v[1] * f), pack_bf16x2(v[2] * f, v[3] * f),
                                                     pack_bf16x2(v[4] * f, v[5] * f), pack_bf16x2(v[6] * f, v[7] * f));
    }
}
// N accumulator columns of a lane to columns col .. of its row of `part`.
template <int D, int N>
__device__ __forceinline__ void leave(uint32_t taddr, uint32_t part, int row, int col) {
#pragma unroll
    for (int i = 0; i < N; i += 16) {
        uint32_t a[16];
        tmem_ld_32x32b_x16(taddr + i, a);
        tmem_ld_wait();
#pragma unroll
        for (int e = 0; e < 16; e += 4)
            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                             part + row * D * 4 + ((((col + i + e) >> 2) ^ (row & 7)) << 4)),
                         "r"(a[e]), "r"(a[e + 1]), "r"(a[e + 2]), "r"(a[e + 3])
                         : "memory");
    }
}

template <int D>
__global__ void __launch_bounds__(GRAD_THREADS, 1)
k_attn_dkv(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmG,
           const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Params p,
           const Tiles ts, const int ns) {
    constexpr int TB = Layout<D>::TILE_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *sq = smem + 2 * TB, *sg = smem + 4 * TB;
    float *stats = reinterpret_cast<float *>(smem + Layout<D>::STATS);   // [unit & 1][-lse2, -delta][128]
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem + Layout<D>::BARS);
    uint64_t *kv_full = bars, *tail = bars + 1, *q_full = bars + 2, *q_empty = bars + 4, *g_full = bars + 6,
             *g_empty = bars + 8, *s_full = bars + 10, *dp_full = bars + 11, *done = bars + 12,
             *p_ready = bars + 13, *ds_ready = bars + 15;   // queries 0-63 of a tile, 64-127
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 17);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 17; ++i) mbar_init(&bars[i], i >= 13 ? GRAD_WARPS : i == 2 || i == 3 ? 2 : 1);
        fence_barrier_init();
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmG);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    const int rank = blockIdx.x % ns, cluster = blockIdx.x / ns;   // the cluster's CTAs take every ns-th head
    const int g = cluster % p.kv_heads, group = p.heads / p.kv_heads;
    int b, len, t;
    if (!find_tile<false>(p, ts, cluster / p.kv_heads, lane, &b, &len, &t)) {   // cluster-uniform, before tensor memory is allocated
        pdl_wait();   // nor may this kernel end before the one ahead of it
        return;
    }
    const int tiles = (len + TILE - 1) / TILE;
    const int heads = (group - rank + ns - 1) / ns;
    const int units = (tiles - t) * heads;   // unit n: query tile t + n / heads, head rank + n % heads ns of the group

    if (warp == GRAD_WARPS + 1) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    constexpr uint32_t tmem = 0;   // all 512 columns
    const uint32_t S = tmem, dP = tmem + TILE, dV = tmem + 2 * TILE, dK = dV + D;

    if (warp >= GRAD_WARPS) {
        grad_regs_down();
        if (warp == GRAD_WARPS) {
            if (lane == 0) {
                mbar_arrive_expect_tx(kv_full, 2 * TB);
                load_tile<D>(smem, &tmK, kv_full, g * D, b + t * TILE);
                load_tile<D>(smem + TB, &tmV, kv_full, g * D, b + t * TILE);
            }
            int n = 0, tails = 0, i = t, hh = 0;
            for (; n < units; ++n) {
                const int s = n & 1, par = ((n >> 1) & 1) ^ 1, h = g * group + rank + hh * ns, row = b + i * TILE;
                const int rows = len - i * TILE;
                uint8_t *dq_ = sq + s * TB, *dg = sg + s * TB;
                const bool partial = rows < TILE;   // the sequence's last query tile
                uint64_t *qb = partial ? tail : &q_full[s], *gb = partial ? tail : &g_full[s];
                // (the unit's two slots were last read two units ago; dO's is free first)
                if (!warp_all(mbar_wait(&g_empty[s], par)) || !warp_all(mbar_wait(&q_empty[s], par))) break;
                if (lane == 0) {
                    mbar_arrive_expect_tx(qb, partial ? 2 * TB : TB);
                    load_tile<D>(dq_, &tmQ, qb, h * D, row);
                    if (!partial) mbar_arrive_expect_tx(gb, TB);
                    load_tile<D>(dg, &tmG, gb, h * D, row);
                }
                if (n == 0) pdl_wait();   // delta and lse2 are the gradient of q's; all else was there before it
                float *st = stats + s * 2 * TILE;
#pragma unroll
                for (int e = lane; e < TILE; e += 32) {
                    const int64_t at = (int64_t)h * p.M + row + e;
                    st[e] = e < rows ? -p.lse2[at] : 0.0f;
                    st[TILE + e] = e < rows ? -p.delta[at] : 0.0f;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&q_full[s]);
                if (partial) {
                    if (!warp_all(mbar_wait(tail, tails & 1))) break;
                    ++tails;
                    clear_rows<D>(dq_, rows, lane);
                    clear_rows<D>(dg, rows, lane);
                    if (lane == 0) {
                        mbar_arrive(&q_full[s]);
                        mbar_arrive(&g_full[s]);
                    }
                }
                if (++hh == heads) { hh = 0; ++i; }
            }
            // every copy lands before the CTA may leave
            mbar_wait(kv_full, 0);
            for (int k = 1; k <= 2 && k <= n; ++k) {
                mbar_wait(&q_full[(n - k) & 1], ((n - k) >> 1) & 1);
                mbar_wait(&g_full[(n - k) & 1], ((n - k) >> 1) & 1);
            }
        } else if (warp == GRAD_WARPS + 1 && elect_one()) {
            const uint32_t k0 = smem_u32(smem), v0 = k0 + TB, q0 = smem_u32(sq), g0 = smem_u32(sg);
            bool ok = mbar_wait(kv_full, 0) && mbar_wait(&q_full[0], 0);
            tc_fence_after();
            if (ok) {
                mma_cols<D>(S, k0, q0);
                tc_commit(s_full);
                ok = mbar_wait(&g_full[0], 0);
                tc_fence_after();
            }
            if (ok) {
                mma_cols<D>(dP, v0, g0);
                tc_commit(dp_full);
            }
            for (int n = 0; n < units && ok; ++n) {
                const int s = n & 1, s1 = s ^ 1, par1 = ((n + 1) >> 1) & 1;
                const bool more = n + 1 < units;
                if (!(ok = mbar_wait(&p_ready[0], n & 1))) break;
                tc_fence_after();
                mma_spread<D, 0, 4>(dV, S, g0 + s * TB, n > 0);
                if (!(ok = mbar_wait(&p_ready[1], n & 1))) break;
                tc_fence_after();
                mma_spread<D, 4, 8>(dV, S, g0 + s * TB, true);
                tc_commit(&g_empty[s]);
                if (more) {
                    if (!(ok = mbar_wait(&q_full[s1], par1))) break;
                    tc_fence_after();
                    mma_cols<D>(S, k0, q0 + s1 * TB);
                    tc_commit(s_full);
                }
                if (!(ok = mbar_wait(&ds_ready[0], n & 1))) break;
                tc_fence_after();
                mma_spread<D, 0, 4>(dK, dP, q0 + s * TB, n > 0);
                if (!(ok = mbar_wait(&ds_ready[1], n & 1))) break;
                tc_fence_after();
                mma_spread<D, 4, 8>(dK, dP, q0 + s * TB, true);
                tc_commit(&q_empty[s]);
                if (more) {
                    if (!(ok = mbar_wait(&g_full[s1], par1))) break;
                    tc_fence_after();
                    mma_cols<D>(dP, v0, g0 + s1 * TB);
                    tc_commit(dp_full);
                }
            }
            tc_commit(done);
        }
    } else {
        grad_regs_up();
        const int quarter = warp >> 2, row = threadIdx.x & 127;
        // this warp's lanes; its columns are 16 quarter .. + 15 of both halves of a tile, so that the
        // first half of P, dS is ready early and the products start on it
        const uint32_t off = ((uint32_t)(warp & 3) << 21) + quarter * 16;
        const uint64_t c2 = f2_pack(p.scale * LOG2E, p.scale * LOG2E);
        bool ok = true;
        int i = t, hh = 0;
        for (int n = 0; n < units; ++n) {
            const float *st = stats + (n & 1) * 2 * TILE + quarter * 16;
            // a masked pair: the query is before the key, or behind the sequence
            const int first = i == t ? row - quarter * 16 : 0, end = len - i * TILE - quarter * 16;
            const bool edge = i == t || end < 80;
            if (!(ok = warp_all(mbar_wait(&q_full[n & 1], (n >> 1) & 1)))) break;   // the statistics
            if (!(ok = warp_all(mbar_wait(s_full, n & 1)))) break;
            tc_fence_after();
            uint32_t r[2][16];
            uint64_t pr[2][8];
            tmem_ld_32x32b_x16(S + off, r[0]);
            tmem_ld_32x32b_x16(S + off + 64, r[1]);
            tmem_ld_wait();
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const ulonglong2 ls = *reinterpret_cast<const ulonglong2 *>(st + 64 * hf + 2 * e);
#pragma unroll
                    for (int k = e; k < e + 2; ++k) {
                        const uint64_t x = f2_fma((uint64_t)r[hf][2 * k + 1] << 32 | r[hf][2 * k], c2, k == e ? ls.x : ls.y);
                        pr[hf][k] = k % EX2_PERIOD < EX2_BY_FMA_DKV ? ex2_fma<true>(x) : ex2_pair(x);
                    }
                }
                if (edge) clear_edge(pr[hf], first - 64 * hf, end - 64 * hf);
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = pack_pair(pr[hf][e]);
                tmem_st_32x32b_x8(S + off + 64 * hf, w);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_ready[hf]);
            }
            if (!(ok = warp_all(mbar_wait(dp_full, n & 1)))) break;
            tc_fence_after();
            tmem_ld_32x32b_x16(dP + off, r[0]);
            tmem_ld_32x32b_x16(dP + off + 64, r[1]);
            tmem_ld_wait();
#pragma unroll
            for (int hf = 0; hf < 2; ++hf) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    const ulonglong2 dl = *reinterpret_cast<const ulonglong2 *>(st + TILE + 64 * hf + 2 * e);
                    pr[hf][e] = f2_mul(pr[hf][e], f2_add((uint64_t)r[hf][2 * e + 1] << 32 | r[hf][2 * e], dl.x));
                    pr[hf][e + 1] = f2_mul(pr[hf][e + 1], f2_add((uint64_t)r[hf][2 * e + 3] << 32 | r[hf][2 * e + 2], dl.y));
                }
                if (edge) clear_edge(pr[hf], first - 64 * hf, end - 64 * hf);   // 0 times what is not finite
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = pack_pair(pr[hf][e]);
                tmem_st_32x32b_x8(dP + off + 64 * hf, w);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ds_ready[hf]);
            }
            if (++hh == heads) { hh = 0; ++i; }
        }
        ok = ok && warp_all(mbar_wait(done, 0));
        if (ok) {
            tc_fence_after();
            // dv by the first two warpgroups, dk by the others, half of the columns each
            const int k0 = t * TILE + (warp & 3) * 32, c0 = (quarter & 1) * (D / 2);   // the warp's first key
            const uint32_t acc = (quarter < 2 ? dV : dK) + ((uint32_t)(warp & 3) << 21) + c0;
            if (ns > 1) {
                leave<D, D / 2>(acc, smem_u32(sq) + (quarter < 2 ? 0 : TILE * D * 4), row, c0);
            } else {
                const int64_t at = b + k0, col = (int64_t)g * D + c0;
                uint8_t *slab = sq + warp * 4096;   // the query tiles are no longer read
                if (quarter < 2) store_rows<D / 2>(acc, 1.0f, slab, p.dv + at * p.lddv + col, p.lddv, len - k0, lane);
                else store_rows<D / 2>(acc, p.scale, slab, p.dk + at * p.lddk + col, p.lddk, len - k0, lane);
            }
        }
        tc_fence_before();
    }
    __syncthreads();
    if (ns > 1) {
        __syncwarp();
        cluster_sync();
        join<D>(p, smem_u32(sq), ns, rank, b, len, t, g);
        __syncwarp();
        cluster_sync();   // no CTA leaves while another reads its sums
    }
    if (warp == GRAD_WARPS + 1) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}
}  // namespace dkv

static pact_status check(const pact_attention_t *a, const char *what) {
    PACT_CHECK(a && a->q && a->k && a->v && a->seq_start, PACT_ERR_INVALID_ARG, "%s: NULL argument", what);
    PACT_CHECK(a->head_dim == 64 || a->head_dim == 128, PACT_ERR_SHAPE, "%s: head_dim must be 64 or 128 (got %d)",
               what, a->head_dim);
    PACT_CHECK(a->heads >= 1 && a->kv_heads >= 1 && a->heads <= 32768 && a->heads % a->kv_heads == 0, PACT_ERR_SHAPE,
               "%s: heads must be a multiple of kv_heads, at most 32768 (got %d, %d)", what, a->heads, a->kv_heads);
    PACT_CHECK(a->M >= 1 && a->M <= (1 << 30) && a->nseq >= 1 && a->nseq <= (1 << 20), PACT_ERR_SHAPE,
               "%s: M in [1, 2^30] and nseq in [1, 2^20] (got %lld, %d)", what, (long long)a->M, a->nseq);
    PACT_CHECK((a->M / TILE + 1) * a->heads <= 0x7FFFFFFF, PACT_ERR_SHAPE, "%s: too many tiles", what);
    PACT_CHECK(std::isfinite(a->scale) && a->scale > 0, PACT_ERR_INVALID_ARG, "%s: scale must be positive and finite",
               what);
    const int64_t nq = (int64_t)a->heads * a->head_dim, nk = (int64_t)a->kv_heads * a->head_dim;
    PACT_CHECK(a->ldq >= nq && a->ldk >= nk && a->ldv >= nk, PACT_ERR_SHAPE, "%s: leading dimensions too small", what);
    PACT_CHECK(aligned16(a->q) && aligned16(a->k) && aligned16(a->v) && a->ldq % 8 == 0 && a->ldk % 8 == 0 &&
                   a->ldv % 8 == 0 && ((uintptr_t)a->seq_start & 3) == 0,
               PACT_ERR_ALIGN, "%s: q, k, v need 16-byte aligned rows, seq_start 4-byte alignment", what);
    return PACT_OK;
}

static bool row_ok(const void *p, int64_t ld, int64_t cols) { return aligned16(p) && ld % 8 == 0 && ld >= cols; }

static Params base(const pact_attention_t *a) {
    Params p = {};
    p.q = a->q; p.k = a->k; p.v = a->v;
    p.ldq = a->ldq; p.ldk = a->ldk; p.ldv = a->ldv;
    p.seq_start = a->seq_start;
    p.nseq = a->nseq; p.heads = a->heads; p.kv_heads = a->kv_heads; p.M = (int)a->M;
    p.scale = a->scale;
    return p;
}

// Raise a kernel's shared-memory limit, once per device.
template <typename K>
static pact_status allow_smem(K kernel, int bytes, std::atomic<uint64_t> &done, const char *what) {
    const int d = current_device();
    if (d >= 0 && d < 64 && (done.load(std::memory_order_acquire) >> d & 1)) return PACT_OK;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    PACT_CHECK(e == cudaSuccess, PACT_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    if (d >= 0 && d < 64) done.fetch_or(1ull << d, std::memory_order_release);
    return PACT_OK;
}

// The map of a [M x cols] BF16 matrix in boxes of 128 rows x 64 columns.
static pact_status map_rows(CUtensorMap *m, const pact_bf16 *base, int64_t cols, int64_t M, int64_t ld,
                            const char *what) {
    return lmma::map_bf16(m, base, cols, M, ld, 64, TILE, what);
}

// Tiles for pairs of units: an odd group pairs over two tiles.
static Tiles pair_tiles(const Params &p) {
    const int group = p.heads / p.kv_heads, shift = group % 2 ? 8 : 7;
    return {shift, group % 2 ? group : group / 2, (p.M >> shift) + p.nseq};
}

template <int D>
static pact_status run_fwd(const Params &p, cudaStream_t st) {
    const char *what = "pact_attention_fwd";
    static std::atomic<uint64_t> done{0};
    pact_status s = allow_smem(fwd::k_attn_fwd<D>, fwd::Layout<D>::SMEM, done, what);
    CUtensorMap q, k, v;
    if (s == PACT_OK) s = map_rows(&q, p.q, (int64_t)p.heads * D, p.M, p.ldq, what);
    if (s == PACT_OK) s = map_rows(&k, p.k, (int64_t)p.kv_heads * D, p.M, p.ldk, what);
    if (s == PACT_OK) s = map_rows(&v, p.v, (int64_t)p.kv_heads * D, p.M, p.ldv, what);
    if (s != PACT_OK) return s;
    const Tiles ts = pair_tiles(p);
    const int64_t grid = (int64_t)ts.slots * ts.pairs * p.kv_heads;
    PACT_CHECK(grid <= 0x7FFFFFFF, PACT_ERR_SHAPE, "%s: too many tiles", what);
    return launch_dep(fwd::k_attn_fwd<D>, dim3((unsigned)grid), dim3(SPLIT_THREADS), fwd::Layout<D>::SMEM, st, what, q,
                      k, v, p, ts);
}

template <int D>
static pact_status run_bwd(const Params &p, cudaStream_t st) {
    const char *what = "pact_attention_bwd";
    static std::atomic<uint64_t> done_q{0}, done_kv{0};
    pact_status s = allow_smem(dq::k_attn_dq<D>, dq::Layout<D>::SMEM, done_q, what);
    if (s == PACT_OK) s = allow_smem(dkv::k_attn_dkv<D>, dkv::Layout<D>::SMEM, done_kv, what);
    CUtensorMap q, g, k, v;
    const int64_t nq = (int64_t)p.heads * D, nk = (int64_t)p.kv_heads * D;
    if (s == PACT_OK) s = map_rows(&q, p.q, nq, p.M, p.ldq, what);
    if (s == PACT_OK) s = map_rows(&g, p.dout, nq, p.M, p.lddo, what);
    if (s == PACT_OK) s = map_rows(&k, p.k, nk, p.M, p.ldk, what);
    if (s == PACT_OK) s = map_rows(&v, p.v, nk, p.M, p.ldv, what);
    if (s != PACT_OK) return s;
    const Tiles pairs = pair_tiles(p), tiles = {7, 1, (p.M >> 7) + p.nseq};
    const int64_t grid_q = (int64_t)pairs.slots * pairs.pairs * p.kv_heads, grid_kv = (int64_t)tiles.slots * p.kv_heads;
    PACT_CHECK(grid_q <= 0x7FFFFFFF && grid_kv <= 0x7FFFFFFF, PACT_ERR_SHAPE, "%s: too many tiles", what);
    s = launch_dep(dq::k_attn_dq<D>, dim3((unsigned)grid_q), dim3(GRAD_THREADS), dq::Layout<D>::SMEM, st, what, q, g,
                   k, v, p, pairs);
    if (s != PACT_OK) return s;
    // A key tile's CTA runs over all later query tiles of the group's heads.  Where there are fewer key
    // tiles than SMs, the heads are spread over a cluster of CTAs that add their sums at the end,
    // for some 5 us.  Gradients (cold L2) over 2048 tokens, 12 and 2 heads of 128 (32 tiles): 202 us with one CTA
    // a tile, 142 with two, 124 with four; 1999 tokens, 32 and 8 heads of 64 (128 tiles): 118, 101, 132; 8192
    // tokens, 24 and 8 heads of 128 (512 tiles): 380, 492 with two.  The rule sees tiles, not the lengths
    // that make them: four sequences of 512, 32 and 8 heads of 64 (128 tiles again, but short): 62, 69, 91.
    const int group = p.heads / p.kv_heads;
    int ns = 1;
    while (2 * ns <= group && ns < 8 && ns * (int64_t)(p.M / TILE + 1) * p.kv_heads < sm_count()) ns *= 2;
    PACT_CHECK(grid_kv * ns <= 0x7FFFFFFF, PACT_ERR_SHAPE, "%s: too many tiles", what);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(grid_kv * ns));
    cfg.blockDim = dim3(GRAD_THREADS);
    cfg.dynamicSmemBytes = dkv::Layout<D>::SMEM;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ns;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, dkv::k_attn_dkv<D>, q, g, k, v, p, tiles, ns);
    PACT_CHECK(e == cudaSuccess, PACT_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
    return launch_status(what);
}

}  // namespace attn
}  // namespace pact

extern "C" {

pact_status pact_attention_fwd(const pact_attention_t *a, pact_bf16 *o, int64_t ldo, float *lse,
                               pact_stream_t stream) {
    using namespace pact;
    pact_status s = attn::check(a, "pact_attention_fwd");
    if (s != PACT_OK) return s;
    const int64_t nq = (int64_t)a->heads * a->head_dim;
    PACT_CHECK(o && lse, PACT_ERR_INVALID_ARG, "pact_attention_fwd: NULL output");
    PACT_CHECK(attn::row_ok(o, ldo, nq) && aligned16(lse), PACT_ERR_ALIGN,
               "pact_attention_fwd: o needs 16-byte aligned rows of at least %lld elements, lse 16-byte alignment",
               (long long)nq);
    const int64_t nk = (int64_t)a->kv_heads * a->head_dim;
    const int64_t M = a->M;
    const Rows all[] = {matrix(o, ldo, nq, M),         memory(lse, 4 * M * a->heads),  matrix(a->q, a->ldq, nq, M),
                        matrix(a->k, a->ldk, nk, M),   matrix(a->v, a->ldv, nk, M),    memory(a->seq_start, 4 * (a->nseq + 1))};
    PACT_CHECK(!overlap_any(all, 2, 6), PACT_ERR_INVALID_ARG,
               "pact_attention_fwd: o or lse overlaps the other, q, k, v or seq_start");
    attn::Params p = attn::base(a);
    p.o = o; p.ldo = ldo; p.lse = lse;
    return a->head_dim == 64 ? attn::run_fwd<64>(p, (cudaStream_t)stream) : attn::run_fwd<128>(p, (cudaStream_t)stream);
}

size_t pact_attention_bwd_workspace_bytes(int64_t M, int heads) {
    return M < 1 || heads < 1 ? 0 : 2 * (((size_t)M * heads + 3) & ~size_t(3)) * sizeof(float);
}

pact_status pact_attention_bwd(const pact_attention_t *a, const pact_attention_grad_t *g, void *workspace,
                               size_t ws_bytes, pact_stream_t stream) {
    using namespace pact;
    const char *what = "pact_attention_bwd";
    pact_status s = attn::check(a, what);
    if (s != PACT_OK) return s;
    PACT_CHECK(g && g->o && g->lse && g->dout && g->dq && g->dk && g->dv && workspace, PACT_ERR_INVALID_ARG,
               "%s: NULL argument", what);
    PACT_CHECK(ws_bytes >= pact_attention_bwd_workspace_bytes(a->M, a->heads), PACT_ERR_INVALID_ARG,
               "%s: workspace too small", what);
    const int64_t nq = (int64_t)a->heads * a->head_dim, nk = (int64_t)a->kv_heads * a->head_dim;
    PACT_CHECK(attn::row_ok(g->o, g->ldo, nq) && attn::row_ok(g->dout, g->lddout, nq) &&
                   attn::row_ok(g->dq, g->lddq, nq) && attn::row_ok(g->dk, g->lddk, nk) &&
                   attn::row_ok(g->dv, g->lddv, nk) && aligned16(g->lse) && aligned16(workspace),
               PACT_ERR_ALIGN, "%s: rows must be 16-byte aligned with leading dimensions at least their width", what);
    const int64_t M = a->M;
    const Rows all[] = {matrix(g->dq, g->lddq, nq, M),
                        matrix(g->dk, g->lddk, nk, M),
                        matrix(g->dv, g->lddv, nk, M),
                        memory(workspace, (int64_t)pact_attention_bwd_workspace_bytes(M, a->heads)),
                        matrix(a->q, a->ldq, nq, M),
                        matrix(a->k, a->ldk, nk, M),
                        matrix(a->v, a->ldv, nk, M),
                        matrix(g->o, g->ldo, nq, M),
                        matrix(g->dout, g->lddout, nq, M),
                        memory(g->lse, 4 * M * a->heads),
                        memory(a->seq_start, 4 * (a->nseq + 1))};
    PACT_CHECK(!overlap_any(all, 4, 11), PACT_ERR_INVALID_ARG,
               "%s: dq, dk, dv or the workspace overlap one another or an input", what);
    attn::Params p = attn::base(a);
    p.o_in = g->o; p.ldo = g->ldo; p.dout = g->dout; p.lddo = g->lddout;
    p.lse = const_cast<float *>(g->lse);
    p.delta = static_cast<float *>(workspace);
    p.dq = g->dq; p.lddq = g->lddq; p.dk = g->dk; p.lddk = g->lddk; p.dv = g->dv; p.lddv = g->lddv;
    p.lse2 = p.delta + (((size_t)a->M * a->heads + 3) & ~size_t(3));
    return a->head_dim == 64 ? attn::run_bwd<64>(p, (cudaStream_t)stream) : attn::run_bwd<128>(p, (cudaStream_t)stream);
}

}  // extern "C"
