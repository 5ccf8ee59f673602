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

#include "quant.cuh"

namespace pact {
namespace attn {

struct Params {
    const pact_bf16 *q, *k, *v, *o_in, *dout;
    int64_t ldq, ldk, ldv, ldo, lddo;
    pact_bf16 *o, *dq, *dk, *dv;
    int64_t lddq, lddk, lddv;
    float *lse, *delta;         // [heads x M]
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

// D (+)= A(tmem) . B(smem)^T, BF16 x BF16 -> FP32, K = 16: the rows of A are tensor-memory
// lanes, eight 32-bit columns hold its 16 BF16 values.  Lane 0 of a converged warp issues.
__device__ __forceinline__ void mma_bf16_ts_w(uint32_t d, uint32_t a, uint64_t bdesc, uint32_t idesc,
                                              uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t.reg .b32 l;\n\t"
        "mov.u32 l, %%laneid;\n\t"
        "setp.eq.u32 q, l, 0;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(bdesc), "r"(idesc), "r"(accumulate));
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
    for (int s = 0; s < D / 16; ++s) mma_bf16_w(tmem, desc_cols(x, s), desc_cols(y, s), idesc, s > 0);
}
// tmem (+)= A . Y: A [128 x 128] BF16 in tensor memory, Y a [128 x D] tile.
template <int D>
__device__ __forceinline__ void mma_rows(uint32_t tmem, uint32_t a, uint32_t y, bool accumulate) {
    constexpr uint32_t idesc = idesc_bf16(TILE, D, false, true);
#pragma unroll
    for (int s = 0; s < TILE / 16; ++s) mma_bf16_ts_w(tmem, a + 8 * s, desc_rows(y, s), idesc, accumulate || s > 0);
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
#pragma unroll
    for (int b = 0; b < D / 64; ++b)
        for (int i = row * 8 + lane; i < TILE * 8; i += 32)
            *reinterpret_cast<uint4 *>(tile + b * BOX_BYTES + i * 16) = make_uint4(0, 0, 0, 0);
    fence_proxy_async_smem();
    __syncwarp();
}

// Sequence s gets the work slots [slot0(s), slot0(s + 1)), at least as many as it has
// work items of `per` rows (each of `group` units): floor(start group / per) rounds away less
// than one item, and the extra slots cover the partial tile and the odd unit.  So the
// grid depends on M and nseq alone, and a slot finds its sequence by searching
// seq_start, without a prefix sum over the sequences.
struct Slots {
    int64_t group, per;
    int extra;
    __host__ __device__ int64_t first(int64_t start, int64_t s) const { return start * group / per + s * extra; }
};

// The sequence of work slot `slot`: rows [b, b + len) and the slot's number inside it;
// len = 0 where the slot lies before the first.  A warp's lanes search together.
__device__ __forceinline__ void find_slot(const Params &p, const Slots &sl, int64_t slot, int lane, int *b, int *len,
                                          int *item) {
    auto start = [&](int i) { return min(max(p.seq_start[i], 0), p.M); };
    int lo = 0, n = p.nseq;
    while (n > 1) {
        const int step = (n + 31) / 32, i = lane * step;
        const bool before = i < n && sl.first(start(lo + i), lo + i) <= slot;
        const uint32_t mask = __ballot_sync(0xffffffffu, before);
        const int k = mask ? 31 - __clz(mask) : 0;
        lo += k * step;
        n = min(step, n - k * step);
    }
    *b = start(lo);
    *len = max(start(lo + 1) - *b, 0);
    const int64_t it = slot - sl.first(*b, lo);
    *item = it < 0 || it > 0x7FFFFFFF ? 0x7FFFFFFF : (int)it;
}

// ------------------------------------------------------------------------- forward
// A CTA computes two units that share a key head: a unit is a 128-query tile of one query
// head, and the units of a sequence run tile-major over the group's heads, so a pair is
// two heads of one tile, or the last head of a tile and the first of the next (one head
// per group: two tiles).  K and V tiles are loaded once for both.  Two tiles in flight let the
// tensor core run one unit's products while the other's softmax runs:
//   warps 0-3, 4-7   softmax of unit 0, 1: a thread owns a query row (a tensor-memory lane),
//                    so maximum and sum need no exchange.  P overwrites the scores as BF16 and
//                    is the next product's operand from tensor memory.
//   warp 8           TMA: the two Q tiles, then K and V tiles through a ring
//   warp 9           the MMAs, in the order  P0 V(j), S0(j+1), P1 V(j), S1(j+1)
// The accumulator is rescaled only when a row's maximum grew by more than 2^8 since the
// last time (any factor cancels in O / l; FP32 has the room), which is rare after the
// first block.  S(j+1) is issued behind P V(j), so a unit that sees its scores ready
// also knows its accumulator at rest.
namespace fwd {
constexpr int THREADS = 320;
constexpr int STAGES = 4;
template <int D>
struct Layout {
    static constexpr int TILE_BYTES = D / 64 * BOX_BYTES;
    static constexpr int SMEM = 1024 + (2 + STAGES) * TILE_BYTES + 256;
};

template <int D>
__global__ void __launch_bounds__(THREADS, 1)
k_attn_fwd(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
           const __grid_constant__ CUtensorMap tmV, const Params p, const Slots sl) {
    constexpr int TILE_BYTES = Layout<D>::TILE_BYTES;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t *ring = smem + 2 * TILE_BYTES;
    uint64_t *bars = reinterpret_cast<uint64_t *>(ring + STAGES * TILE_BYTES);
    uint64_t *full = bars, *empty = bars + STAGES, *q_full = bars + 2 * STAGES, *tail = q_full + 1;
    uint64_t *s_full = tail + 1, *p_ready = s_full + 2, *o_full = p_ready + 2;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(o_full + 2);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        mbar_init(q_full, 1);
        mbar_init(tail, 1);
        for (int u = 0; u < 2; ++u) {
            mbar_init(&s_full[u], 1);
            mbar_init(&p_ready[u], 4);
            mbar_init(&o_full[u], 1);
        }
        fence_barrier_init();
        prefetch_tensormap(&tmQ);
        prefetch_tensormap(&tmK);
        prefetch_tensormap(&tmV);
    }
    pdl_wait();
    const int g = blockIdx.x % p.kv_heads, group = p.heads / p.kv_heads;
    int b, len, item;
    find_slot(p, sl, gridDim.x / p.kv_heads - 1 - blockIdx.x / p.kv_heads, lane, &b, &len, &item);
    const int64_t units = (int64_t)((len + TILE - 1) / TILE) * group, u0 = 2 * (int64_t)item;
    if (u0 >= units) return;   // block-uniform, before tensor memory is allocated
    const bool two = u0 + 1 < units;
    const int t0 = (int)(u0 / group), h0 = g * group + (int)(u0 % group);
    const int t1 = two ? (int)((u0 + 1) / group) : t0, h1 = g * group + (int)((u0 + 1) % group);
    const int blocks = t1 + 1;

    if (warp == 9) {
        tmem_alloc(tmem_slot, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;   // S0, S1: 128 columns each, then O0, O1: D columns each

    if (warp == 8) {
        if (lane == 0) {
            mbar_arrive_expect_tx(q_full, (two ? 2 : 1) * TILE_BYTES);
            load_tile<D>(smem, &tmQ, q_full, h0 * D, b + t0 * TILE);
            if (two) load_tile<D>(smem + TILE_BYTES, &tmQ, q_full, h1 * D, b + t1 * TILE);
        }
        uint32_t stage = 0, phase = 0;
        bool ok = true;
        int issued = 0;
        for (int i = 0; i < 2 * blocks && ok; ++i) {   // K(0), V(0), K(1), ...
            if (!(ok = warp_all(mbar_wait(&empty[stage], phase ^ 1)))) break;
            const int row = b + (i >> 1) * TILE, rows = len - (i >> 1) * TILE;
            uint8_t *dst = ring + stage * TILE_BYTES;
            if ((i & 1) && rows < TILE) {   // the sequence's last V tile
                if (lane == 0) {
                    mbar_arrive_expect_tx(tail, TILE_BYTES);
                    load_tile<D>(dst, &tmV, tail, g * D, row);
                }
                if (!(ok = warp_all(mbar_wait(tail, 0)))) break;
                clear_rows<D>(dst, rows, lane);
                if (lane == 0) mbar_arrive(&full[stage]);
            } else if (lane == 0) {
                mbar_arrive_expect_tx(&full[stage], TILE_BYTES);
                load_tile<D>(dst, i & 1 ? &tmV : &tmK, &full[stage], g * D, row);
            }
            ++issued;
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
        // every copy lands before the CTA may leave
        mbar_wait(q_full, 0);
        for (int s = 0; s < STAGES && s < issued; ++s) mbar_wait(&full[s], ((issued - 1 - s) / STAGES) & 1);
    } else if (warp == 9) {
        const uint32_t q0 = smem_u32(smem), q1 = q0 + TILE_BYTES, r0 = smem_u32(ring);
        const uint32_t S0 = tmem, S1 = tmem + TILE, O0 = tmem + 2 * TILE, O1 = O0 + D;
        bool ok = warp_all(mbar_wait(q_full, 0)) && warp_all(mbar_wait(&full[0], 0));
        tc_fence_after();
        if (ok) {
            mma_cols<D>(S0, q0, r0);
            tc_commit_w(&s_full[0]);
            if (two) {
                mma_cols<D>(S1, q1, r0);
                tc_commit_w(&s_full[1]);
            }
            tc_commit_w(&empty[0]);
        }
        for (int j = 0; j < blocks && ok; ++j) {
            const int vi = 2 * j + 1, ki = vi + 1, vs = vi % STAGES, ks = ki % STAGES;
            const bool more0 = j < t0, more1 = two && j < t1;   // another block after this one
            if (!(ok = warp_all(mbar_wait(&full[vs], (vi / STAGES) & 1)))) break;
            if (j <= t0) {
                if (!(ok = warp_all(mbar_wait(&p_ready[0], j & 1)))) break;
                tc_fence_after();
                mma_rows<D>(O0, S0, r0 + vs * TILE_BYTES, j > 0);
                if (!more0) tc_commit_w(&o_full[0]);
            }
            if (more0 || more1) {
                if (!(ok = warp_all(mbar_wait(&full[ks], (ki / STAGES) & 1)))) break;
                tc_fence_after();
            }
            if (more0) {
                mma_cols<D>(S0, q0, r0 + ks * TILE_BYTES);
                tc_commit_w(&s_full[0]);
            }
            if (two) {
                if (!(ok = warp_all(mbar_wait(&p_ready[1], j & 1)))) break;
                tc_fence_after();
                mma_rows<D>(O1, S1, r0 + vs * TILE_BYTES, j > 0);
                if (!more1) tc_commit_w(&o_full[1]);
            }
            tc_commit_w(&empty[vs]);
            if (more1) {
                mma_cols<D>(S1, q1, r0 + ks * TILE_BYTES);
                tc_commit_w(&s_full[1]);
            }
            if (more0 || more1) tc_commit_w(&empty[ks]);
        }
        __syncwarp();
    } else {
        const int u = warp >> 2, row = threadIdx.x & 127, t = u ? t1 : t0;
        const int last = u && !two ? -1 : t;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;   // this warp's 32 tensor-memory lanes
        const uint32_t S = tmem + u * TILE + lanes, O = tmem + 2 * TILE + u * D + lanes;
        const float c = p.scale * LOG2E;
        float m = -INFINITY, l = 0.0f;   // reference of the exponentials (times c), row sum
        bool ok = true;
        for (int j = 0; j <= last && ok; ++j) {
            if (!(ok = warp_all(mbar_wait(&s_full[u], j & 1)))) break;
            tc_fence_after();
            uint32_t r[4][32];
#pragma unroll
            for (int i = 0; i < 4; ++i) tmem_ld_32x32b_x32(S + 32 * i, r[i]);
            tmem_ld_wait();
            if (j == t) {   // the diagonal block: keys after the query
#pragma unroll
                for (int i = 0; i < 128; ++i)
                    if (i > row) r[i >> 5][i & 31] = 0xFF800000u;
            }
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int i = 0; i < 128; ++i) mx[i & 3] = fmaxf(mx[i & 3], __uint_as_float(r[i >> 5][i & 31]));
            const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c;
            if (j == 0) {
                m = top;
            } else {
                const bool grew = top > m + 8.0f;
                if (__any_sync(0xffffffffu, grew)) {
                    const float f = grew ? ex2(m - top) : 1.0f;
                    if (grew) m = top;
                    l *= f;
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        uint32_t a[32];
                        tmem_ld_32x32b_x32(O + 32 * i, a);
                        tmem_ld_wait();
#pragma unroll
                        for (int e = 0; e < 32; ++e) a[e] = __float_as_uint(__uint_as_float(a[e]) * f);
                        tmem_st_32x32b_x32(O + 32 * i, a);
                    }
                }
            }
            float sum[4] = {};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const float x = ex2(fmaf(__uint_as_float(r[i][2 * e]), c, -m));
                    const float y = ex2(fmaf(__uint_as_float(r[i][2 * e + 1]), c, -m));
                    sum[2 * (e & 1)] += x;
                    sum[2 * (e & 1) + 1] += y;
                    w[e] = pack_bf16x2(x, y);
                }
                tmem_st_32x32b_x16(S + 16 * i, w);
            }
            l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&p_ready[u]);
        }
        ok = last >= 0 && ok && warp_all(mbar_wait(&o_full[u], 0));
        if (ok) {
            tc_fence_after();
            const int qi = t * TILE + row, h = u ? h1 : h0;
            const bool live = qi < len;
            const float inv = 1.0f / l;
            pact_bf16 *dst = p.o + (int64_t)(b + qi) * p.ldo + (int64_t)h * D;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                uint32_t a[32];
                tmem_ld_32x32b_x32(O + 32 * i, a);
                tmem_ld_wait();
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    uint4 w;
                    w.x = pack_bf16x2(__uint_as_float(a[e]) * inv, __uint_as_float(a[e + 1]) * inv);
                    w.y = pack_bf16x2(__uint_as_float(a[e + 2]) * inv, __uint_as_float(a[e + 3]) * inv);
                    w.z = pack_bf16x2(__uint_as_float(a[e + 4]) * inv, __uint_as_float(a[e + 5]) * inv);
                    w.w = pack_bf16x2(__uint_as_float(a[e + 6]) * inv, __uint_as_float(a[e + 7]) * inv);
                    if (live) *reinterpret_cast<uint4 *>(dst + 32 * i + e) = w;
                }
            }
            if (live) p.lse[(int64_t)h * p.M + b + qi] = fmaf(m, LN2, logf(l));
        }
        tc_fence_before();
    }
    __syncthreads();
    if (warp == 9) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}
}  // namespace fwd

// Rows [*b, *e) of the sequence that holds `row`; false for a row of none.
__device__ __forceinline__ bool find_sequence(const Params &p, int row, int *b, int *e) {
    int lo = 0, hi = p.nseq;    // last sequence with start <= row
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.seq_start[mid] <= row) lo = mid;
        else hi = mid;
    }
    *b = max(p.seq_start[lo], 0);
    *e = min(p.seq_start[lo + 1], p.M);
    return row >= *b && row < *e;
}

template <int V>
__device__ __forceinline__ void load_row(const pact_bf16 *p, float (&x)[V]) {
    const uint32_t *w = reinterpret_cast<const uint32_t *>(p);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
        const uint32_t u = w[i];
        x[2 * i] = bf16lo(u);
        x[2 * i + 1] = bf16hi(u);
    }
}
template <int V>
__device__ __forceinline__ void store_row(pact_bf16 *p, const float (&x)[V]) {
    uint32_t *w = reinterpret_cast<uint32_t *>(p);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(x[2 * i], x[2 * i + 1]);
}
template <int V>
__device__ __forceinline__ float dot_warp(const float (&a)[V], const float (&b)[V]) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < V; ++i) s += a[i] * b[i];
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    return s;
}

// dq and delta: one warp per (row, query head).
template <int D>
__global__ void k_attn_dq(const Params p) {
    constexpr int V = D / 32;
    pdl_wait();
    const int row = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, h = blockIdx.y, lane = threadIdx.x & 31;
    int b, e;
    if (row >= p.M || !find_sequence(p, row, &b, &e)) return;
    const int g = h / (p.heads / p.kv_heads), c = lane * V;
    float q[V], k[V], v[V], d[V], o[V], acc[V] = {};
    load_row(p.q + row * p.ldq + h * D + c, q);
    load_row(p.dout + row * p.lddo + h * D + c, d);
    load_row(p.o_in + row * p.ldo + h * D + c, o);
    const float delta = dot_warp(d, o), lse = p.lse[(int64_t)h * p.M + row];
    if (lane == 0) p.delta[(int64_t)h * p.M + row] = delta;
    for (int j = b; j <= row; ++j) {
        load_row(p.k + j * p.ldk + g * D + c, k);
        load_row(p.v + j * p.ldv + g * D + c, v);
        const float ds = expf(dot_warp(q, k) * p.scale - lse) * (dot_warp(d, v) - delta) * p.scale;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] += ds * k[i];
    }
    store_row(p.dq + row * p.lddq + h * D + c, acc);
}

// dk and dv: one warp per (row, key head), over the group's query heads and later rows.
template <int D>
__global__ void k_attn_dkv(const Params p) {
    constexpr int V = D / 32;
    pdl_wait();
    const int row = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, g = blockIdx.y, lane = threadIdx.x & 31;
    int b, e;
    if (row >= p.M || !find_sequence(p, row, &b, &e)) return;
    const int group = p.heads / p.kv_heads, c = lane * V;
    float q[V], k[V], v[V], d[V], ak[V] = {}, av[V] = {};
    load_row(p.k + row * p.ldk + g * D + c, k);
    load_row(p.v + row * p.ldv + g * D + c, v);
    for (int h = g * group; h < (g + 1) * group; ++h) {
        for (int i = row; i < e; ++i) {
            load_row(p.q + i * p.ldq + h * D + c, q);
            load_row(p.dout + i * p.lddo + h * D + c, d);
            const float w = expf(dot_warp(q, k) * p.scale - p.lse[(int64_t)h * p.M + i]);
            const float ds = w * (dot_warp(d, v) - p.delta[(int64_t)h * p.M + i]) * p.scale;
#pragma unroll
            for (int t = 0; t < V; ++t) {
                ak[t] += ds * q[t];
                av[t] += w * d[t];
            }
        }
    }
    store_row(p.dk + row * p.lddk + g * D + c, ak);
    store_row(p.dv + row * p.lddv + g * D + c, av);
}

static pact_status check(const pact_attention_t *a, const char *what) {
    PACT_CHECK(a && a->q && a->k && a->v && a->seq_start, PACT_ERR_INVALID_ARG, "%s: NULL argument", what);
    PACT_CHECK(a->head_dim == 64 || a->head_dim == 128, PACT_ERR_SHAPE, "%s: head_dim must be 64 or 128 (got %d)",
               what, a->head_dim);
    PACT_CHECK(a->heads >= 1 && a->kv_heads >= 1 && a->heads <= 32768 && a->heads % a->kv_heads == 0, PACT_ERR_SHAPE,
               "%s: heads must be a multiple of kv_heads, at most 32768 (got %d, %d)", what, a->heads, a->kv_heads);
    PACT_CHECK(a->M >= 1 && a->M <= (1 << 30) && a->nseq >= 1 && a->nseq <= (1 << 20), PACT_ERR_SHAPE,
               "%s: M in [1, 2^30] and nseq in [1, 2^20] (got %lld, %d)", what, (long long)a->M, a->nseq);
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
    // pairs of units: ceil(tiles group / 2) a sequence, at most len group / 256 + 127 group / 256 + 1/2
    const int group = p.heads / p.kv_heads;
    const Slots sl = {group, 2 * TILE, group / 2 + 2};
    const int64_t grid = sl.first(p.M, p.nseq) * p.kv_heads;
    PACT_CHECK(grid <= 0x7FFFFFFF, PACT_ERR_SHAPE, "%s: too many tiles", what);
    return launch_dep(fwd::k_attn_fwd<D>, dim3((unsigned)grid), dim3(fwd::THREADS), fwd::Layout<D>::SMEM, st, what, q,
                      k, v, p, sl);
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
    attn::Params p = attn::base(a);
    p.o = o; p.ldo = ldo; p.lse = lse;
    return a->head_dim == 64 ? attn::run_fwd<64>(p, (cudaStream_t)stream) : attn::run_fwd<128>(p, (cudaStream_t)stream);
}

size_t pact_attention_bwd_workspace_bytes(int64_t M, int heads) {
    return M < 1 || heads < 1 ? 0 : (size_t)M * heads * sizeof(float);
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
    attn::Params p = attn::base(a);
    p.o_in = g->o; p.ldo = g->ldo; p.dout = g->dout; p.lddo = g->lddout;
    p.lse = const_cast<float *>(g->lse);
    p.delta = static_cast<float *>(workspace);
    p.dq = g->dq; p.lddq = g->lddq; p.dk = g->dk; p.lddk = g->lddk; p.dv = g->dv; p.lddv = g->lddv;
    const bool small = a->head_dim == 64;
    const dim3 grid_q((p.M + 7) / 8, p.heads), grid_k((p.M + 7) / 8, p.kv_heads);
    s = launch_dep(small ? attn::k_attn_dq<64> : attn::k_attn_dq<128>, grid_q, dim3(256), 0, (cudaStream_t)stream,
                   what, p);
    if (s != PACT_OK) return s;
    return launch_dep(small ? attn::k_attn_dkv<64> : attn::k_attn_dkv<128>, grid_k, dim3(256), 0,
                      (cudaStream_t)stream, what, p);
}

}  // extern "C"
