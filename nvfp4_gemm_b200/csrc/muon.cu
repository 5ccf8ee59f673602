// muon.cu -- the adapters' update by an orthogonalised momentum (the Muon optimiser's
// Newton-Schulz products), for many skinny matrices in one call.
//
// With gradient g, momentum m and weight W of a matrix with r = min(rows, cols) <= 64:
//   m' = mu m + g;  u = g + mu m' (Nesterov) or m';  X0 = u / (|u|_F + eps)
//   five times  A = X X^T,  X <- a X + (b A + c A^2) X     (on the side of the r rows)
//   W' = (1 - lr wd) W - lr sqrt(max(1, rows / cols)) X
// Every product is a polynomial of the r x r Gram matrix S0 = X0 X0^T, so the whole
// iteration is X = P u with P = Q4 Q3 Q2 Q1 Q0 / (|u|_F + eps), Q_k = a I + b S_k + c S_k^2,
// S_{k+1} = Q_k S_k Q_k (all of them commute): u is read once for S0 and once for P u,
// instead of ten times.  Adapter gradients are close to low rank, and P is up to
// a^5 = 485 on the weak directions while the strong ones cancel to about 1; S0, the
// products and P u are therefore kept in FP64 (an FP32 Gram matrix loses the directions
// below 3e-4 of the strongest).
//
//   k_muon_gram   a slab of the long side per CTA: m' is written, the slab's part of
//                 u u^T goes to scratch
//   k_muon_poly   one CTA per matrix: S0 from the parts in a fixed order, then P
//   k_muon_apply  a slab per CTA again: u from g and m', W' and its BF16 copy
#include <algorithm>
#include <cmath>

#include "quant.cuh"

namespace pact {
namespace muon {

constexpr int THREADS = 256;
constexpr int WARPS = THREADS / 32;
constexpr int BATCH = 128;     // matrices per launch: their descriptors are kernel parameters
constexpr int STEPS = 5;
constexpr double NS_A = 3.4445, NS_B = -4.7750, NS_C = 2.0315, EPS = 1e-7;

// NB blocks of 8 cover r; a slab holds about 16384 elements.
__host__ __device__ constexpr int slab_len(int nb) { return nb == 2 ? 1024 : nb == 4 ? 512 : 256; }
__host__ __device__ constexpr int pitch(int nb) { return slab_len(nb) + 4; }   // rows 4 banks apart
__host__ __device__ constexpr int tri(int nb) { return nb * (nb + 1) / 2; }
__host__ __device__ constexpr int mat_pitch(int nb) { return 8 * nb + 4; }
__host__ __device__ constexpr int mat_size(int nb) { return 8 * nb * mat_pitch(nb); }
__host__ __device__ constexpr size_t stage_smem(int nb) { return sizeof(float) * 8 * nb * pitch(nb); }
__host__ __device__ constexpr size_t apply_smem(int nb) { return stage_smem(nb) + sizeof(double) * 64 * nb * nb; }
__host__ __device__ constexpr size_t poly_smem(int nb) { return sizeof(double) * 5 * mat_size(nb); }

struct Matrix {
    const void *grad;
    const float *m;
    float *m_out;
    const float *w;
    float *w_out;
    pact_bf16 *w16;
    double *parts;     // per matrix: [slabs x tri x 64], then P [8 NB x 8 NB]
    int32_t slab0;     // first slab of the launch
    int32_t mat0;      // first matrix of the launch
    int32_t len;       // long side
    int32_t slabs;     // per matrix
    int16_t r;
    int16_t tall;      // stored [len x r], else [r x len]
    int16_t vec;       // 4 where every row starts 16-byte aligned and r, len allow it, else 1
};

struct Params {
    Matrix mat[BATCH];   // each of one or more matrices of one shape
    int n, grad_fp32, nesterov;
    float mu;
    double keep, lr;   // 1 - lr wd, lr
};

__device__ __forceinline__ void dmma(double (&c)[2], double a, double b) {
    asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
                 : "+d"(c[0]), "+d"(c[1])
                 : "d"(a), "d"(b));
}

// The entry that holds slab (BY_SLAB) or matrix number `i` of the launch, its pointers moved to the
// matrix; *slab: the slab's number inside the matrix.
template <int NB, bool BY_SLAB>
__device__ __forceinline__ Matrix find_matrix(const Params &p, int i, int *slab) {
    int lo = 0, hi = p.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if ((BY_SLAB ? p.mat[mid].slab0 : p.mat[mid].mat0) <= i) lo = mid;
        else hi = mid;
    }
    Matrix a = p.mat[lo];
    const int j = BY_SLAB ? (i - a.slab0) / a.slabs : i - a.mat0;
    *slab = BY_SLAB ? i - a.slab0 - j * a.slabs : 0;
    const int64_t off = (int64_t)j * a.r * a.len;
    a.grad = static_cast<const uint8_t *>(a.grad) + off * (p.grad_fp32 ? 4 : 2);
    a.m += off;
    a.m_out += off;
    a.w += off;
    a.w_out += off;
    if (a.w16) a.w16 += off;
    a.parts += (int64_t)j * (a.slabs * tri(NB) * 64 + 64 * NB * NB);
    return a;
}

// f(element offset, row of the short side, position in the slab) for every VEC-th element of a slab
// [k0, k0 + n) of the long side, in memory order (coalesced in both orientations).
template <int VEC, typename F>
__device__ __forceinline__ void for_slab(const Matrix &a, int k0, int n, F f) {
    if (a.tall) {
        const int total = n * a.r;
        for (int t = threadIdx.x * VEC; t < total; t += THREADS * VEC)
            f((int64_t)k0 * a.r + t, t % a.r, t / a.r);
    } else {
        const int per = n / VEC;
        for (int t = threadIdx.x; t < a.r * per; t += THREADS) {
            const int i = t / per, k = (t - i * per) * VEC;
            f((int64_t)i * a.len + k0 + k, i, k);
        }
    }
}

__device__ __forceinline__ float load_grad(const Params &p, const Matrix &a, int64_t e) {
    return p.grad_fp32 ? static_cast<const float *>(a.grad)[e]
                       : __uint_as_float((uint32_t) static_cast<const pact_bf16 *>(a.grad)[e] << 16);
}
__device__ __forceinline__ float4 load_grad4(const Params &p, const Matrix &a, int64_t e) {
    if (p.grad_fp32) return *reinterpret_cast<const float4 *>(static_cast<const float *>(a.grad) + e);
    const uint2 w = *reinterpret_cast<const uint2 *>(static_cast<const pact_bf16 *>(a.grad) + e);
    return make_float4(bf16lo(w.x), bf16hi(w.x), bf16lo(w.y), bf16hi(w.y));
}

// u of a slab into shared memory as [short side x position]; FIRST also forms and writes m'.
template <bool FIRST>
__device__ __forceinline__ void stage_u(const Params &p, const Matrix &a, int k0, int n, float *us, int ld) {
    const float mu = p.mu;
    auto one = [&](float g, float m, float *mo) {
        if (FIRST) *mo = m = fmaf(mu, m, g);
        return p.nesterov ? fmaf(mu, m, g) : m;
    };
    const float *m_in = FIRST ? a.m : a.m_out;
    if (a.vec == 4) {
        for_slab<4>(a, k0, n, [&](int64_t e, int i, int k) {
            const float4 g = load_grad4(p, a, e), m = *reinterpret_cast<const float4 *>(m_in + e);
            float4 mo;
            const float u0 = one(g.x, m.x, &mo.x), u1 = one(g.y, m.y, &mo.y), u2 = one(g.z, m.z, &mo.z),
                        u3 = one(g.w, m.w, &mo.w);
            if (FIRST) *reinterpret_cast<float4 *>(a.m_out + e) = mo;
            if (a.tall) {
                us[i * ld + k] = u0;
                us[(i + 1) * ld + k] = u1;
                us[(i + 2) * ld + k] = u2;
                us[(i + 3) * ld + k] = u3;
            } else {
                *reinterpret_cast<float4 *>(us + i * ld + k) = make_float4(u0, u1, u2, u3);
            }
        });
    } else {
        for_slab<1>(a, k0, n, [&](int64_t e, int i, int k) {
            float mo;
            us[i * ld + k] = one(load_grad(p, a, e), m_in[e], &mo);
            if (FIRST) a.m_out[e] = mo;
        });
    }
}

template <int NB>
__global__ void __launch_bounds__(THREADS) k_muon_gram(const __grid_constant__ Params p) {
    constexpr int L = slab_len(NB), LD = pitch(NB), T = tri(NB);
    extern __shared__ __align__(16) float us[];
    pdl_wait();
    int slab;
    const Matrix a = find_matrix<NB, true>(p, blockIdx.x, &slab);
    const int k0 = slab * L, n = min(L, a.len - k0);
    const int n4 = (n + 3) & ~3;
    // rows past r and positions past the end count as zero
    for (int t = threadIdx.x; t < 8 * NB * L; t += THREADS) {
        const int i = t / L, k = t - i * L;
        if (i >= a.r || (k >= n && k < n4)) us[i * LD + k] = 0.0f;
    }
    stage_u<true>(p, a, k0, n, us, LD);
    __syncthreads();
    // u u^T by FP64 tensor instructions: the fragments of both operands of an 8 x 8
    // block of a symmetric product are the same registers (row lane / 4, position lane % 4)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double acc[T][2] = {};
    for (int k = warp * 4; k < n4; k += WARPS * 4) {
        double f[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) f[b] = (double)us[(8 * b + (lane >> 2)) * LD + k + (lane & 3)];
        int t = 0;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int c = b; c < NB; ++c) dmma(acc[t++], f[b], f[c]);
    }
    __syncthreads();
    // sum the warps' parts in order
    double *sum = reinterpret_cast<double *>(us);
    for (int t = 0; t < T; ++t) {
#pragma unroll
        for (int u = 0; u < T; ++u)
            if (u == t) {
                sum[warp * 64 + lane * 2] = acc[u][0];
                sum[warp * 64 + lane * 2 + 1] = acc[u][1];
            }
        __syncthreads();
        if (threadIdx.x < 64) {
            double s = 0.0;
            for (int w = 0; w < WARPS; ++w) s += sum[w * 64 + threadIdx.x];
            a.parts[((int64_t)slab * T + t) * 64 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}

// out = x y for matrices in shared memory, an 8 x 8 block per warp; with eye, out = f(x y) of
// Q = a I + b x + c x y.
template <int NB, bool EYE = false>
__device__ __forceinline__ void product(double *out, const double *x, const double *y, int first, int step) {
    constexpr int LD = mat_pitch(NB);
    const int lane = threadIdx.x & 31;
    for (int blk = first; blk < NB * NB; blk += step) {
        const int bi = blk / NB * 8, bj = blk % NB * 8;
        double c[2] = {};
#pragma unroll
        for (int k = 0; k < 8 * NB; k += 4)
            dmma(c, x[(bi + (lane >> 2)) * LD + k + (lane & 3)], y[(k + (lane & 3)) * LD + bj + (lane >> 2)]);
        const int i = bi + (lane >> 2), j = bj + 2 * (lane & 3);
#pragma unroll
        for (int e = 0; e < 2; ++e)
            out[i * LD + j + e] = EYE ? NS_B * x[i * LD + j + e] + NS_C * c[e] + (i == j + e ? NS_A : 0.0) : c[e];
    }
}

template <int NB>
__global__ void __launch_bounds__(THREADS) k_muon_poly(const __grid_constant__ Params p) {
    constexpr int N = 8 * NB, LD = mat_pitch(NB), T = tri(NB), SZ = mat_size(NB);
    extern __shared__ __align__(16) double sm[];
    __shared__ double gain;
    double *S = sm, *Q = sm + SZ, *QS = sm + 2 * SZ, *P = sm + 3 * SZ, *P2 = sm + 4 * SZ;
    pdl_wait();
    int unused;
    const Matrix a = find_matrix<NB, false>(p, blockIdx.x, &unused);
    const int slabs = a.slabs;
    for (int t = threadIdx.x; t < T * 64; t += THREADS) {
        double s = 0.0;
#pragma unroll 4
        for (int i = 0; i < slabs; ++i) s += a.parts[((int64_t)i * T) * 64 + t];
        int b = 0, c = t >> 6;   // block (b, c), c >= b, of the upper triangle
        while (c >= NB - b) c -= NB - b++;
        c += b;
        const int l = (t & 63) >> 1, i = 8 * b + (l >> 2), j = 8 * c + 2 * (l & 3) + (t & 1);
        S[i * LD + j] = s;
        if (c > b) S[j * LD + i] = s;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        double tr = 0.0;
        for (int i = 0; i < a.r; ++i) tr += S[i * LD + i];
        gain = 1.0 / (sqrt(tr) + EPS);
    }
    __syncthreads();
    const double g2 = gain * gain;
    for (int t = threadIdx.x; t < N * N; t += THREADS) {
        const int i = t / N, j = t % N;
        S[i * LD + j] *= g2;
        P[i * LD + j] = i == j ? gain : 0.0;
    }
    __syncthreads();
    const int warp = threadIdx.x >> 5;
#pragma unroll 1
    for (int it = 0; it < STEPS; ++it) {
        product<NB, true>(Q, S, S, warp, WARPS);
        __syncthreads();
        // P <- Q P beside QS = Q S, on one half of the warps each
        if (warp < WARPS / 2) product<NB>(P2, Q, P, warp, WARPS / 2);
        else product<NB>(QS, Q, S, warp - WARPS / 2, WARPS / 2);
        __syncthreads();
        if (it + 1 < STEPS) product<NB>(S, QS, Q, warp, WARPS);
        __syncthreads();
        double *t = P;
        P = P2;
        P2 = t;
    }
    double *out = a.parts + (int64_t)slabs * T * 64;
    for (int t = threadIdx.x; t < N * N; t += THREADS) out[t] = P[t / N * LD + t % N];
}

template <int NB>
__global__ void __launch_bounds__(THREADS) k_muon_apply(const __grid_constant__ Params p) {
    constexpr int L = slab_len(NB), LD = pitch(NB), N = 8 * NB, POS = L / THREADS;
    extern __shared__ __align__(16) float us[];
    double *P = reinterpret_cast<double *>(us + 8 * NB * LD);
    pdl_wait();
    int slab;
    const Matrix a = find_matrix<NB, true>(p, blockIdx.x, &slab);
    const int k0 = slab * L, n = min(L, a.len - k0);
    const double *src = a.parts + (int64_t)a.slabs * tri(NB) * 64;
    for (int t = threadIdx.x; t < N * N; t += THREADS) P[t] = src[t];
    for (int t = threadIdx.x; t < 8 * NB * L; t += THREADS) {
        const int i = t / L, k = t - i * L;
        if (i >= a.r || k >= n) us[i * LD + k] = 0.0f;
    }
    stage_u<false>(p, a, k0, n, us, LD);
    __syncthreads();
    // X = P u: a thread owns POS positions, THREADS apart, and overwrites its columns of u
    {
        double u[N][POS];
#pragma unroll
        for (int j = 0; j < N; ++j)
#pragma unroll
            for (int q = 0; q < POS; ++q) u[j][q] = (double)us[j * LD + threadIdx.x + q * THREADS];
        for (int i = 0; i < a.r; ++i) {
            double x[POS] = {};
#pragma unroll
            for (int j = 0; j < N; ++j)
#pragma unroll
                for (int q = 0; q < POS; ++q) x[q] = fma(P[i * N + j], u[j][q], x[q]);
#pragma unroll
            for (int q = 0; q < POS; ++q) us[i * LD + threadIdx.x + q * THREADS] = (float)x[q];
        }
    }
    __syncthreads();
    const double step = p.lr * (a.tall ? sqrt((double)a.len / a.r) : 1.0), keep = p.keep;
    if (a.vec == 4) {
        for_slab<4>(a, k0, n, [&](int64_t e, int i, int k) {
            const float4 w = *reinterpret_cast<const float4 *>(a.w + e);
            const int s = a.tall ? LD : 1;
            const float *x = us + i * LD + k;
            const float4 o = make_float4((float)(keep * w.x - step * x[0]), (float)(keep * w.y - step * x[s]),
                                         (float)(keep * w.z - step * x[2 * s]), (float)(keep * w.w - step * x[3 * s]));
            *reinterpret_cast<float4 *>(a.w_out + e) = o;
            if (a.w16)
                *reinterpret_cast<uint2 *>(a.w16 + e) = make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
        });
    } else {
        for_slab<1>(a, k0, n, [&](int64_t e, int i, int k) {
            const float o = (float)(keep * a.w[e] - step * us[i * LD + k]);
            a.w_out[e] = o;
            if (a.w16) a.w16[e] = __bfloat16_as_ushort(__float2bfloat16_rn(o));
        });
    }
}

static int blocks_of(int r) { return r <= 16 ? 2 : r <= 32 ? 4 : r <= 48 ? 6 : 8; }

template <int NB>
static pact_status launch(const Params &p, int matrices, int slabs, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};   // devices whose shared-memory limits are set
    const int d = current_device();
    if (d < 0 || d >= 64 || !(done.load(std::memory_order_acquire) >> d & 1)) {
        cudaError_t e = cudaFuncSetAttribute(k_muon_gram<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)stage_smem(NB));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k_muon_poly<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)poly_smem(NB));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k_muon_apply<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)apply_smem(NB));
        PACT_CHECK(e == cudaSuccess, PACT_ERR_CUDA, "pact_muon_step: %s", cudaGetErrorString(e));
        if (d >= 0 && d < 64) done.fetch_or(1ull << d, std::memory_order_release);
    }
    const char *what = "pact_muon_step";
    pact_status s = launch_dep(k_muon_gram<NB>, dim3(slabs), dim3(THREADS), stage_smem(NB), st, what, p);
    if (s == PACT_OK) s = launch_dep(k_muon_poly<NB>, dim3(matrices), dim3(THREADS), poly_smem(NB), st, what, p);
    if (s == PACT_OK) s = launch_dep(k_muon_apply<NB>, dim3(slabs), dim3(THREADS), apply_smem(NB), st, what, p);
    return s;
}

static pact_status check(const pact_muon_matrix_t *mats, int n, const char *what) {
    PACT_CHECK(mats && n >= 1, PACT_ERR_INVALID_ARG, "%s: no matrices", what);
    for (int i = 0; i < n; ++i) {
        const pact_muon_matrix_t &m = mats[i];
        PACT_CHECK(m.grad && m.momentum && m.momentum_out && m.weight && m.weight_out, PACT_ERR_INVALID_ARG,
                   "%s: entry %d: NULL pointer", what, i);
        PACT_CHECK(m.count >= 1 && m.count <= (1 << 20), PACT_ERR_SHAPE, "%s: entry %d: count in [1, 2^20]", what, i);
        PACT_CHECK(m.rows >= 1 && m.cols >= 1 && (m.rows <= 64 || m.cols <= 64) && m.rows <= (1 << 24) &&
                       m.cols <= (1 << 24),
                   PACT_ERR_SHAPE, "%s: entry %d: the shorter side is at most 64, the longer at most 2^24 (got %lld x %lld)",
                   what, i, (long long)m.rows, (long long)m.cols);
        PACT_CHECK((((uintptr_t)m.momentum | (uintptr_t)m.momentum_out | (uintptr_t)m.weight | (uintptr_t)m.weight_out) &
                    3) == 0 && (((uintptr_t)m.grad | (uintptr_t)m.weight_bf16) & 1) == 0,
                   PACT_ERR_ALIGN, "%s: entry %d: pointers must be aligned to their elements", what, i);
    }
    return PACT_OK;
}

}  // namespace muon
}  // namespace pact

extern "C" {

size_t pact_muon_workspace_bytes(const pact_muon_matrix_t *mats, int n) {
    using namespace pact::muon;
    if (!mats || n < 1) return 0;
    int r = 1;
    for (int i = 0; i < n; ++i) {
        const int64_t s = mats[i].rows < mats[i].cols ? mats[i].rows : mats[i].cols;
        if (s < 1 || s > 64 || mats[i].count < 1) return 0;
        if (s > r) r = (int)s;
    }
    const int nb = blocks_of(r);
    size_t d = 0;
    for (int i = 0; i < n; ++i) {
        const int64_t len = mats[i].rows < mats[i].cols ? mats[i].cols : mats[i].rows;
        d += (size_t)mats[i].count * ((size_t)((len + slab_len(nb) - 1) / slab_len(nb)) * tri(nb) * 64 + 64 * nb * nb);
    }
    return d * sizeof(double);
}

pact_status pact_muon_step(const pact_muon_matrix_t *mats, int n, int grad_fp32, double lr, double momentum,
                           double weight_decay, int nesterov, void *workspace, size_t ws_bytes,
                           pact_stream_t stream) {
    using namespace pact;
    using muon::blocks_of, muon::slab_len, muon::tri, muon::BATCH;
    const char *what = "pact_muon_step";
    pact_status s = muon::check(mats, n, what);
    if (s != PACT_OK) return s;
    PACT_CHECK(std::isfinite(lr) && std::isfinite(momentum) && std::isfinite(weight_decay), PACT_ERR_INVALID_ARG,
               "%s: lr, momentum and weight_decay must be finite", what);
    PACT_CHECK(workspace && ws_bytes >= pact_muon_workspace_bytes(mats, n), PACT_ERR_INVALID_ARG,
               "%s: workspace too small", what);
    PACT_CHECK(aligned16(workspace), PACT_ERR_ALIGN, "%s: workspace must be 16-byte aligned", what);
    int rmax = 1;
    for (int i = 0; i < n; ++i) rmax = std::max(rmax, (int)std::min(mats[i].rows, mats[i].cols));
    const int nb = blocks_of(rmax), L = slab_len(nb);
    double *ws = static_cast<double *>(workspace);
    muon::Params p;
    p.grad_fp32 = grad_fp32 != 0;
    p.nesterov = nesterov != 0;
    p.mu = (float)momentum;
    p.lr = lr;
    p.keep = 1.0 - lr * weight_decay;
    for (int first = 0; first < n; first += BATCH) {
        p.n = std::min(BATCH, n - first);
        int64_t slabs = 0, matrices = 0;
        for (int i = 0; i < p.n; ++i) {
            const pact_muon_matrix_t &m = mats[first + i];
            muon::Matrix &a = p.mat[i];
            a.grad = m.grad; a.m = m.momentum; a.m_out = m.momentum_out; a.w = m.weight; a.w_out = m.weight_out;
            a.w16 = m.weight_bf16;
            a.tall = m.rows > m.cols;
            a.r = (int16_t)(a.tall ? m.cols : m.rows);
            a.len = (int32_t)(a.tall ? m.rows : m.cols);
            const bool al = aligned16(m.grad) && aligned16(m.momentum) && aligned16(m.momentum_out) &&
                            aligned16(m.weight) && aligned16(m.weight_out) && aligned16(m.weight_bf16);
            a.vec = al && m.cols % 4 == 0 ? 4 : 1;
            a.slabs = (a.len + L - 1) / L;
            a.slab0 = (int32_t)slabs;
            a.mat0 = (int32_t)matrices;
            a.parts = ws;
            slabs += a.slabs * m.count;
            matrices += m.count;
            PACT_CHECK(slabs <= 0x7FFFFFFF, PACT_ERR_SHAPE, "%s: too many elements", what);
            ws += (size_t)m.count * ((size_t)a.slabs * tri(nb) * 64 + 64 * nb * nb);
        }
        const cudaStream_t st = (cudaStream_t)stream;
        s = nb == 2 ? muon::launch<2>(p, (int)matrices, (int)slabs, st) : nb == 4 ? muon::launch<4>(p, (int)matrices, (int)slabs, st)
            : nb == 6 ? muon::launch<6>(p, (int)matrices, (int)slabs, st) : muon::launch<8>(p, (int)matrices, (int)slabs, st);
        if (s != PACT_OK) return s;
    }
    return PACT_OK;
}

}  // extern "C"
