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

// One warp per (row, query head); a lane holds D / 32 neighbouring columns.
template <int D>
__global__ void k_attn_fwd(const Params p) {
    constexpr int V = D / 32;
    pdl_wait();
    const int row = blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32, h = blockIdx.y, lane = threadIdx.x & 31;
    int b, e;
    if (row >= p.M || !find_sequence(p, row, &b, &e)) return;
    const int g = h / (p.heads / p.kv_heads), c = lane * V;
    float q[V], k[V], v[V], acc[V] = {};
    load_row(p.q + row * p.ldq + h * D + c, q);
    float m = -INFINITY, l = 0.0f;
    for (int j = b; j <= row; ++j) {
        load_row(p.k + j * p.ldk + g * D + c, k);
        load_row(p.v + j * p.ldv + g * D + c, v);
        const float s = dot_warp(q, k) * p.scale, mn = fmaxf(m, s), f = expf(m - mn), w = expf(s - mn);
        l = l * f + w;
        m = mn;
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = acc[i] * f + w * v[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] /= l;
    store_row(p.o + row * p.ldo + h * D + c, acc);
    if (lane == 0) p.lse[(int64_t)h * p.M + row] = m + logf(l);
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
    PACT_CHECK(std::isfinite(a->scale), PACT_ERR_INVALID_ARG, "%s: scale must be finite", what);
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
    return launch_dep(a->head_dim == 64 ? attn::k_attn_fwd<64> : attn::k_attn_fwd<128>,
                      dim3((p.M + 7) / 8, p.heads), dim3(256), 0, (cudaStream_t)stream, "pact_attention_fwd", p);
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
