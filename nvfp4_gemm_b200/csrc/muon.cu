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
// A matrix that fits the shared memory of a cluster of CTAs takes one kernel and one pass over
// memory (k_muon_fused): u stays in shared memory between its Gram matrix and P u.  Its phases
// (load, Gram matrix, P, P u, store) follow one another in a CTA and overlap only between the two
// CTAs of an SM: the 392 adapter matrices of 28 layers (rank 16, 406 MB) take 126 us, 3.2 TB/s or
// 49% of the measured copy rate, the 14 of one layer 18.  Tried: whole float4s of u through shared memory
// (4% slower), clusters of sixteen with three or four CTAs an SM (10 to 30% slower), a later CTA's g and m
// asked into L2 ahead of it (3% faster, not worth its code).  Larger ones take three kernels.
// The largest rank of a call sets the block size of all its matrices, and beyond 48 all of them take
// the three kernels: one matrix of 64 x 64 beside those 392 makes 1374 us of 132 (cold L2).  One that
// needs more shared memory than two CTAs have room for on an SM leaves one an SM to every matrix of its
// launch: one of 16 x 14000 beside them, 198 us.  The 14 matrices of one layer at rank 48: 129 us, at
// rank 64: 159 (rank 16: 28).  The three kernels:
//   k_muon_gram   a slab of the long side per CTA: m' is written, the slab's part of
//                 u u^T goes to scratch
//   k_muon_poly   one CTA per matrix: S0 from the parts in a fixed order, then P
//   k_muon_apply  a slab per CTA again: u from g and m', W' and its BF16 copy
#include <algorithm>
#include <cmath>

#include "overlap.cuh"
#include "quant.cuh"

namespace pact {
namespace muon {

constexpr int THREADS = 512;
constexpr int WARPS = THREADS / 32;
constexpr int BATCH = 128;     // matrices per launch: their descriptors are kernel parameters
constexpr int STEPS = 5;
constexpr double NS_A = 3.4445, NS_B = -4.7750, NS_C = 2.0315, EPS = 1e-7;

// NB blocks of 8 cover r; a slab holds about 16384 elements.
__host__ __device__ constexpr int slab_len(int nb) { return nb == 2 ? 1024 : nb == 4 ? 512 : 256; }
__host__ __device__ constexpr int pitch(int nb) { return slab_len(nb) + 8; }   // rows 8 banks apart
__host__ __device__ constexpr int tri(int nb) { return nb * (nb + 1) / 2; }
__host__ __device__ constexpr int mat_pitch(int nb) { return 8 * nb + 4; }
__host__ __device__ constexpr int mat_size(int nb) { return 8 * nb * mat_pitch(nb); }
__host__ __device__ constexpr size_t stage_smem(int nb) { return sizeof(float) * 8 * nb * pitch(nb); }
__host__ __device__ constexpr size_t gram_smem(int nb) { return stage_smem(nb) + sizeof(double) * WARPS * 64; }
__host__ __device__ constexpr size_t apply_smem(int nb) { return stage_smem(nb) + sizeof(double) * mat_size(nb); }
__host__ __device__ constexpr size_t poly_smem(int nb) { return sizeof(double) * 5 * mat_size(nb); }
// The fused kernel: slab, the CTA's part of the Gram matrix, the five matrices (first the warps' exchange).
__host__ __device__ constexpr size_t fused_smem(int nb, int len) {
    return sizeof(float) * 8 * nb * ((len + 31) / 32 * 32 + 8) + sizeof(double) * tri(nb) * 64 + poly_smem(nb);
}
constexpr size_t FUSED_FIRST = 110 * 1024;   // two CTAs an SM
constexpr size_t FUSED_MOST = 226 * 1024;
constexpr int FUSED_NB = 6;                  // beyond, the FP64 matrices leave no room for a slab
constexpr int CLUSTER = 8;
static_assert(WARPS * 64 <= 5 * mat_size(2), "the warps exchange their sums where the matrices come to lie");

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
    int32_t slab;      // fused: positions per CTA
    int16_t ctas;      // fused: CTAs per matrix, a power of two up to CLUSTER
    int16_t r;
    int16_t tall;      // stored [len x r], else [r x len]
    int16_t vec;       // 4 where every row starts 16-byte aligned and r, len allow it, else 1
};

struct Params {
    Matrix mat[BATCH];   // each of one or more matrices of one shape
    int n, grad_fp32, nesterov;
    int cluster;         // fused: CTAs per cluster; slab0 counts CTAs, mat0 is not used
    float mu;
    double keep, lr;   // 1 - lr wd, lr
};

__device__ __forceinline__ void dmma(double (&c)[2], double a, double b) {
    asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
                 : "+d"(c[0]), "+d"(c[1])
                 : "d"(a), "d"(b));
}

// Move an entry's pointers to its matrix j.
__device__ __forceinline__ void to_matrix(const Params &p, Matrix &a, int j) {
    const int64_t off = (int64_t)j * a.r * a.len;
    a.grad = static_cast<const uint8_t *>(a.grad) + off * (p.grad_fp32 ? 4 : 2);
    a.m += off;
    a.m_out += off;
    a.w += off;
    a.w_out += off;
    if (a.w16) a.w16 += off;
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
    to_matrix(p, a, j);
    a.parts += (int64_t)j * (a.slabs * tri(NB) * 64 + 64 * NB * NB);
    return a;
}

// A thread's VEC-element pieces of a slab [k0, k0 + n) of the long side, in memory order (coalesced in
// both orientations): piece t = threadIdx.x + i THREADS, kept as (fast, slow) without divisions.
template <int VEC>
struct Walk {
    int fast, slow, per, dfast, dslow, left;
    int64_t base, row;   // element of piece (0, 0); elements from one slow index to the next
    bool tall;
    __device__ __forceinline__ Walk(const Matrix &a, int k0, int n) {
        tall = a.tall;
        per = (tall ? a.r : n) / VEC;
        const int total = per * (tall ? n : a.r), t = threadIdx.x;
        base = tall ? (int64_t)k0 * a.r : k0;
        row = tall ? a.r : a.len;
        slow = per ? t / per : 0;
        fast = t - slow * per;
        dslow = per ? THREADS / per : 0;
        dfast = THREADS - dslow * per;
        left = total - t;
    }
    __device__ __forceinline__ bool more() const { return left > 0; }
    __device__ __forceinline__ int64_t element() const { return base + slow * row + fast * VEC; }
    __device__ __forceinline__ int at(int ld) const { return tall ? fast * VEC * ld + slow : slow * ld + fast * VEC; }
    __device__ __forceinline__ void next() {
        left -= THREADS;
        slow += dslow;
        fast += dfast;
        if (fast >= per) {
            fast -= per;
            ++slow;
        }
    }
};

template <int VEC>
struct Piece {
    float v[VEC];
};
template <int VEC>
__device__ __forceinline__ Piece<VEC> load_f32(const float *p) {
    Piece<VEC> x;
    if constexpr (VEC == 4) {
        const float4 f = *reinterpret_cast<const float4 *>(p);
        x.v[0] = f.x; x.v[1] = f.y; x.v[2] = f.z; x.v[3] = f.w;
    } else {
        x.v[0] = *p;
    }
    return x;
}
template <int VEC>
__device__ __forceinline__ Piece<VEC> load_grad(const Params &p, const Matrix &a, int64_t e) {
    if (p.grad_fp32) return load_f32<VEC>(static_cast<const float *>(a.grad) + e);
    const pact_bf16 *g = static_cast<const pact_bf16 *>(a.grad) + e;
    Piece<VEC> x;
    if constexpr (VEC == 4) {
        const uint2 w = *reinterpret_cast<const uint2 *>(g);
        x.v[0] = bf16lo(w.x); x.v[1] = bf16hi(w.x); x.v[2] = bf16lo(w.y); x.v[3] = bf16hi(w.y);
    } else {
        x.v[0] = __uint_as_float((uint32_t)*g << 16);
    }
    return x;
}

// u of a slab into shared memory as [short side x position]; FIRST also forms and writes m'.  Four pieces
// are loaded before any is stored: the output may be the input, which the compiler must assume.
template <bool FIRST, int VEC>
__device__ __forceinline__ void stage_vec(const Params &p, const Matrix &a, int k0, int n, float *us, int ld) {
    constexpr int U = 4;
    const float mu = p.mu;
    const float *m_in = FIRST ? a.m : a.m_out;
    Walk<VEC> w(a, k0, n);
    while (w.more()) {
        Piece<VEC> g[U], m[U];
        int64_t e[U];
        int at[U], have = 0;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (!w.more()) continue;
            e[i] = w.element();
            at[i] = w.at(ld);
            g[i] = load_grad<VEC>(p, a, e[i]);
            m[i] = load_f32<VEC>(m_in + e[i]);
            if (FIRST && VEC == 4) asm volatile("prefetch.global.L2 [%0];" ::"l"(a.w + e[i]));
            have = i + 1;
            w.next();
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i >= have) continue;
#pragma unroll
            for (int c = 0; c < VEC; ++c) {
                if (FIRST) m[i].v[c] = fmaf(mu, m[i].v[c], g[i].v[c]);
                us[at[i] + (a.tall ? c * ld : c)] = p.nesterov ? fmaf(mu, m[i].v[c], g[i].v[c]) : m[i].v[c];
            }
            if (FIRST) {
                if constexpr (VEC == 4)
                    *reinterpret_cast<float4 *>(a.m_out + e[i]) = make_float4(m[i].v[0], m[i].v[1], m[i].v[2], m[i].v[3]);
                else a.m_out[e[i]] = m[i].v[0];
            }
        }
    }
}
template <bool FIRST>
__device__ __forceinline__ void stage_u(const Params &p, const Matrix &a, int k0, int n, float *us, int ld) {
    if (a.vec == 4) stage_vec<FIRST, 4>(p, a, k0, n, us, ld);
    else stage_vec<FIRST, 1>(p, a, k0, n, us, ld);
}
// Zero the rows past r and the positions from n to n8 of [8 NB x n8].
template <int NB>
__device__ __forceinline__ void clear_rest(const Matrix &a, int n, int n8, float *us, int ld) {
    for (int i = 0; i < 8 * NB; ++i)
        for (int k = (i < a.r ? n : 0) + threadIdx.x; k < n8; k += THREADS) us[i * ld + k] = 0.0f;
}

// W' = keep W - step X for a slab whose X lies in shared memory.
template <int VEC>
__device__ __forceinline__ void update_vec(const Params &p, const Matrix &a, int k0, int n, const float *us, int ld) {
    constexpr int U = 4;
    const double step = p.lr * (a.tall ? sqrt((double)a.len / a.r) : 1.0), keep = p.keep;
    Walk<VEC> w(a, k0, n);
    while (w.more()) {
        Piece<VEC> x[U];
        int64_t e[U];
        int at[U], have = 0;
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (!w.more()) continue;
            e[i] = w.element();
            at[i] = w.at(ld);
            x[i] = load_f32<VEC>(a.w + e[i]);
            have = i + 1;
            w.next();
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (i >= have) continue;
            float o[VEC];
#pragma unroll
            for (int c = 0; c < VEC; ++c)   // in FP64, rounded once
                o[c] = (float)(keep * x[i].v[c] - step * us[at[i] + (a.tall ? c * ld : c)]);
            if constexpr (VEC == 4) {
                *reinterpret_cast<float4 *>(a.w_out + e[i]) = make_float4(o[0], o[1], o[2], o[3]);
                if (a.w16)
                    *reinterpret_cast<uint2 *>(a.w16 + e[i]) = make_uint2(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]));
            } else {
                a.w_out[e[i]] = o[0];
                if (a.w16) a.w16[e[i]] = __bfloat16_as_ushort(__float2bfloat16_rn(o[0]));
            }
        }
    }
}
__device__ __forceinline__ void update_w(const Params &p, const Matrix &a, int k0, int n, const float *us, int ld) {
    if (a.vec == 4) update_vec<4>(p, a, k0, n, us, ld);
    else update_vec<1>(p, a, k0, n, us, ld);
}

// The slab's part of u u^T, summed over the warps in order: the upper 8 x 8 blocks, as the lanes of the
// FP64 tensor instruction hold them, to out[tri x 64].  The fragments of both operands of a block of a
// symmetric product are the same registers (row lane / 4, position lane % 4).
template <int NB, int B0, int B1>   // block rows [B0, B1) of the triangle
__device__ __forceinline__ void gram_rows(const float *us, int ld, int n8, double *sum, double *out) {
    constexpr int T0 = tri(NB) - tri(NB - B0), T = tri(NB) - tri(NB - B1) - T0;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    double acc[T][2] = {};
    for (int k = warp * 8; k < n8; k += WARPS * 8) {
#pragma unroll
        for (int h = 0; h < 8; h += 4) {
            double f[NB];
#pragma unroll
            for (int b = B0; b < NB; ++b) f[b] = (double)us[(8 * b + (lane >> 2)) * ld + k + h + (lane & 3)];
            int t = 0;
#pragma unroll
            for (int b = B0; b < B1; ++b)
#pragma unroll
                for (int c = b; c < NB; ++c) dmma(acc[t++], f[b], f[c]);
        }
    }
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
            out[(T0 + t) * 64 + threadIdx.x] = s;
        }
        __syncthreads();
    }
}
template <int NB>
__device__ __forceinline__ void gram(const float *us, int ld, int n8, double *sum, double *out) {
    if constexpr (NB <= 6) {
        gram_rows<NB, 0, NB>(us, ld, n8, sum, out);
    } else {   // the 36 blocks of r = 64 exceed the registers: 21 and 15
        gram_rows<NB, 0, 3>(us, ld, n8, sum, out);
        gram_rows<NB, 3, NB>(us, ld, n8, sum, out);
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
    const int n8 = (n + 7) & ~7;
    clear_rest<NB>(a, n, n8, us, LD);
    stage_u<true>(p, a, k0, n, us, LD);
    __syncthreads();
    gram<NB>(us, LD, n8, reinterpret_cast<double *>(us + 8 * NB * LD), a.parts + (int64_t)slab * T * 64);
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

// S0 and then P from the Gram matrix's blocks (read by `part`: block entry -> its sum), in five matrices
// of shared memory at sm; returns P.
template <int NB, typename F>
__device__ __forceinline__ double *polynomial(const Matrix &a, double *sm, F part) {
    constexpr int N = 8 * NB, LD = mat_pitch(NB), T = tri(NB), SZ = mat_size(NB);
    __shared__ double gain;
    double *S = sm, *Q = sm + SZ, *QS = sm + 2 * SZ, *P = sm + 3 * SZ, *P2 = sm + 4 * SZ;
    for (int t = threadIdx.x; t < T * 64; t += THREADS) {
        const double s = part(t);
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
    return P;
}

// X = P u in place: a warp takes eight positions, its FP64 fragments of u, and every block row of P.
template <int NB>
__device__ __forceinline__ void apply(float *us, int ld, int n8, const double *P) {
    constexpr int LD = mat_pitch(NB);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int k = warp * 8; k < n8; k += WARPS * 8) {
        double f[2 * NB];   // row 4 s + lane % 4, position lane / 4
#pragma unroll
        for (int s = 0; s < 2 * NB; ++s) f[s] = (double)us[(4 * s + (lane & 3)) * ld + k + (lane >> 2)];
        __syncwarp();
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            double c[2] = {};
#pragma unroll
            for (int s = 0; s < 2 * NB; ++s) dmma(c, P[(8 * b + (lane >> 2)) * LD + 4 * s + (lane & 3)], f[s]);
            *reinterpret_cast<float2 *>(us + (8 * b + (lane >> 2)) * ld + k + 2 * (lane & 3)) =
                make_float2((float)c[0], (float)c[1]);
        }
    }
}

template <int NB>
__global__ void __launch_bounds__(THREADS) k_muon_poly(const __grid_constant__ Params p) {
    constexpr int LD = mat_pitch(NB), T = tri(NB);
    extern __shared__ __align__(16) double sm[];
    pdl_wait();
    int unused;
    const Matrix a = find_matrix<NB, false>(p, blockIdx.x, &unused);
    const double *P = polynomial<NB>(a, sm, [&](int t) {
        double s = 0.0;
#pragma unroll 4
        for (int i = 0; i < a.slabs; ++i) s += a.parts[(int64_t)i * T * 64 + t];
        return s;
    });
    double *out = a.parts + (int64_t)a.slabs * T * 64;
    for (int t = threadIdx.x; t < 64 * NB * NB; t += THREADS) out[t] = P[t / (8 * NB) * LD + t % (8 * NB)];
}

template <int NB>
__global__ void __launch_bounds__(THREADS) k_muon_apply(const __grid_constant__ Params p) {
    constexpr int L = slab_len(NB), LD = pitch(NB), N = 8 * NB;
    extern __shared__ __align__(16) float us[];
    double *P = reinterpret_cast<double *>(us + 8 * NB * LD);
    pdl_wait();
    int slab;
    const Matrix a = find_matrix<NB, true>(p, blockIdx.x, &slab);
    const int k0 = slab * L, n = min(L, a.len - k0), n8 = (n + 7) & ~7;
    const double *src = a.parts + (int64_t)a.slabs * tri(NB) * 64;
    for (int t = threadIdx.x; t < N * N; t += THREADS) P[t / N * mat_pitch(NB) + t % N] = src[t];
    clear_rest<NB>(a, n, n8, us, LD);
    stage_u<false>(p, a, k0, n, us, LD);
    __syncthreads();
    apply<NB>(us, LD, n8, P);
    __syncthreads();
    update_w(p, a, k0, n, us, LD);
}

// One pass: `ctas` CTAs of a cluster hold a matrix's u in shared memory, add their parts of the Gram
// matrix in order through distributed shared memory, and each forms P (the same bits) for its
// own slab.
template <int NB>
__global__ void __launch_bounds__(THREADS, NB == 2 ? 2 : 1) k_muon_fused(const __grid_constant__ Params p) {
    constexpr int T = tri(NB);
    extern __shared__ __align__(16) float us[];
    pdl_wait();
    int lo = 0, hi = p.n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (p.mat[mid].slab0 <= (int)blockIdx.x) lo = mid;
        else hi = mid;
    }
    Matrix a = p.mat[lo];
    const int cta = blockIdx.x - a.slab0, j = cta / a.ctas, rank = cta % a.ctas;
    const bool idle = j >= a.slabs;   // slabs: here the entry's matrices; its last cluster may not be full
    to_matrix(p, a, idle ? 0 : j);
    const int ld = (a.slab + 31) / 32 * 32 + 8, k0 = rank * a.slab, n = idle ? 0 : max(0, min(a.slab, a.len - k0));
    const int n8 = (n + 7) & ~7;
    double *part = reinterpret_cast<double *>(us + 8 * NB * ld), *sm = part + T * 64;
    clear_rest<NB>(a, n, n8, us, ld);
    stage_u<true>(p, a, k0, n, us, ld);
    __syncthreads();
    gram<NB>(us, ld, n8, sm, part);
    if (a.ctas > 1) cluster_sync();
    const uint32_t mine = smem_u32(part), first = cluster_ctarank() / a.ctas * a.ctas;
    const double *P = polynomial<NB>(a, sm, [&](int t) {
        if (a.ctas == 1) return part[t];
        double v[CLUSTER], s = 0.0;
#pragma unroll
        for (int q = 0; q < CLUSTER; ++q) {
            v[q] = 0.0;
            if (q < a.ctas)
                asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v[q]) : "r"(mapa_shared(mine + 8 * t, first + q)) : "memory");
        }
#pragma unroll
        for (int q = 0; q < CLUSTER; ++q)
            if (q < a.ctas) s += v[q];
        return s;
    });
    // (every part has been read once a CTA arrives here: polynomial() ends with a barrier)
    if (a.ctas > 1) asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    apply<NB>(us, ld, n8, P);
    __syncthreads();
    update_w(p, a, k0, n, us, ld);
    __syncwarp();
    if (a.ctas > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");   // no CTA leaves before its part was read
}

// CTAs per matrix of the fused kernel; 0 where the matrix does not fit a cluster.
static int fused_ctas(const pact_muon_matrix_t &m, int nb) {
    const int64_t len = std::max(m.rows, m.cols);
    for (int c = 1; c <= CLUSTER; c *= 2) {
        const int64_t slab = (len + c - 1) / c + 3;
        if (slab < (1 << 20) && fused_smem(nb, (int)slab) <= (c < CLUSTER ? std::max(FUSED_FIRST, fused_smem(nb, 256)) : FUSED_MOST))
            return c;
    }
    return 0;
}

static int blocks_of(int r) { return r <= 16 ? 2 : r <= 32 ? 4 : r <= 48 ? 6 : 8; }

// Run `kernel` with clusters of `cluster` CTAs.
static pact_status launch_clusters(void (*kernel)(Params), int grid, int cluster, size_t smem, cudaStream_t st,
                                   const char *what, const Params &p) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, p);
    PACT_CHECK(e == cudaSuccess, PACT_ERR_CUDA, "%s: launch failed: %s", what, cudaGetErrorString(e));
    return launch_status(what);
}

template <int NB>
static pact_status launch_fused(const Params &p, int grid, size_t smem, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};   // devices whose shared-memory limit is set
    const int d = current_device();
    if (d < 0 || d >= 64 || !(done.load(std::memory_order_acquire) >> d & 1)) {
        const cudaError_t e = cudaFuncSetAttribute(k_muon_fused<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)FUSED_MOST);
        PACT_CHECK(e == cudaSuccess, PACT_ERR_CUDA, "pact_muon_step: %s", cudaGetErrorString(e));
        if (d >= 0 && d < 64) done.fetch_or(1ull << d, std::memory_order_release);
    }
    return launch_clusters(k_muon_fused<NB>, grid, p.cluster, smem, st, "pact_muon_step", p);
}

template <int NB>
static pact_status launch(const Params &p, int matrices, int slabs, cudaStream_t st) {
    static std::atomic<uint64_t> done{0};   // devices whose shared-memory limits are set
    const int d = current_device();
    if (d < 0 || d >= 64 || !(done.load(std::memory_order_acquire) >> d & 1)) {
        cudaError_t e = cudaFuncSetAttribute(k_muon_gram<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)gram_smem(NB));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k_muon_poly<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)poly_smem(NB));
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(k_muon_apply<NB>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     (int)apply_smem(NB));
        PACT_CHECK(e == cudaSuccess, PACT_ERR_CUDA, "pact_muon_step: %s", cudaGetErrorString(e));
        if (d >= 0 && d < 64) done.fetch_or(1ull << d, std::memory_order_release);
    }
    const char *what = "pact_muon_step";
    pact_status s = launch_dep(k_muon_gram<NB>, dim3(slabs), dim3(THREADS), gram_smem(NB), st, what, p);
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
    // A matrix given twice would be updated by two CTAs at once, and what is read must not change under the
    // call: a gradient, for one, is read again after the momentum is written where a matrix takes three
    // kernels.  Only a momentum or weight that is its own output may be both.
    Ranges all(6 * (int64_t)n + 1);
    for (int i = 0; i < n; ++i) {
        const pact_muon_matrix_t &m = mats[i];
        const int64_t size = m.count * m.rows * m.cols;
        all.add(m.momentum_out, 4 * size, true);
        all.add(m.weight_out, 4 * size, true);
        all.add(m.weight_bf16, 2 * size, true);
        all.add(m.grad, (grad_fp32 ? 4 : 2) * size, false);
        if (m.momentum != m.momentum_out) all.add(m.momentum, 4 * size, false);
        if (m.weight != m.weight_out) all.add(m.weight, 4 * size, false);
    }
    all.add(workspace, (int64_t)pact_muon_workspace_bytes(mats, n), true);
    PACT_CHECK(all.disjoint(), PACT_ERR_INVALID_ARG,
               "%s: an output or the workspace overlaps another output (a matrix given twice?) or an input", what);
    int rmax = 1;
    for (int i = 0; i < n; ++i) rmax = std::max(rmax, (int)std::min(mats[i].rows, mats[i].cols));
    const int nb = blocks_of(rmax);
    const cudaStream_t st = (cudaStream_t)stream;
    muon::Params p;
    p.grad_fp32 = grad_fp32 != 0;
    p.nesterov = nesterov != 0;
    p.mu = (float)momentum;
    p.lr = lr;
    p.keep = 1.0 - lr * weight_decay;
    auto describe = [&](const pact_muon_matrix_t &m) {
        muon::Matrix a = {};
        a.grad = m.grad; a.m = m.momentum; a.m_out = m.momentum_out; a.w = m.weight; a.w_out = m.weight_out;
        a.w16 = m.weight_bf16;
        a.tall = m.rows > m.cols;
        a.r = (int16_t)(a.tall ? m.cols : m.rows);
        a.len = (int32_t)(a.tall ? m.rows : m.cols);
        const bool al = aligned16(m.grad) && aligned16(m.momentum) && aligned16(m.momentum_out) && aligned16(m.weight) &&
                        aligned16(m.weight_out) && aligned16(m.weight_bf16);
        a.vec = al && m.cols % 4 == 0 ? 4 : 1;
        return a;
    };
    // The matrices that fit a cluster's shared memory: as few CTAs each as leave two CTAs room on an SM
    // (or, in clusters of eight, as fit at all), more while the SMs are not all busy.
    int64_t fused = 0;
    for (int first = 0; first < n && nb <= muon::FUSED_NB; first += BATCH) {
        p.n = 0;
        for (int i = first; i < std::min(n, first + BATCH); ++i)
            if (muon::fused_ctas(mats[i], nb)) p.mat[p.n++] = describe(mats[i]);
        if (p.n == 0) continue;
        fused += p.n;
        int64_t ctas = 0;
        for (int k = 0, i = first; i < std::min(n, first + BATCH); ++i)
            if (int c = muon::fused_ctas(mats[i], nb)) {
                p.mat[k].slabs = (int32_t)mats[i].count;
                p.mat[k++].ctas = (int16_t)c;
                ctas += c * mats[i].count;
            }
        p.cluster = 1;
        while (ctas < sm_count()) {
            int64_t more = 0;
            for (int k = 0; k < p.n; ++k)
                if (p.mat[k].ctas < muon::CLUSTER && p.mat[k].len > 64 * p.mat[k].ctas) {
                    more += (int64_t)p.mat[k].ctas * p.mat[k].slabs;
                    p.mat[k].ctas *= 2;
                }
            ctas += more;
            if (more == 0) break;
        }
        int64_t grid = 0;
        size_t smem = 0;
        for (int k = 0; k < p.n; ++k) p.cluster = std::max(p.cluster, (int)p.mat[k].ctas);
        for (int k = 0; k < p.n; ++k) {
            muon::Matrix &a = p.mat[k];
            a.slab = ((a.len + a.ctas - 1) / a.ctas + 3) & ~3;
            a.slab0 = (int32_t)grid;
            smem = std::max(smem, muon::fused_smem(nb, a.slab));
            grid += ((int64_t)a.slabs * a.ctas + p.cluster - 1) / p.cluster * p.cluster;
            PACT_CHECK(grid <= 0x7FFFFFFF, PACT_ERR_SHAPE, "%s: too many elements", what);
        }
        s = nb == 2 ? muon::launch_fused<2>(p, (int)grid, smem, st) : nb == 4 ? muon::launch_fused<4>(p, (int)grid, smem, st)
                                                                            : muon::launch_fused<6>(p, (int)grid, smem, st);
        if (s != PACT_OK) return s;
    }
    if (fused == n) return PACT_OK;
    const int L = slab_len(nb);
    double *ws = static_cast<double *>(workspace);
    for (int i = 0; i < n;) {
        p.n = 0;
        int64_t slabs = 0, matrices = 0;
        for (; i < n && p.n < BATCH; ++i) {
            const pact_muon_matrix_t &m = mats[i];
            if (nb <= muon::FUSED_NB && muon::fused_ctas(m, nb)) continue;
            muon::Matrix &a = p.mat[p.n++] = describe(m);
            a.slabs = (a.len + L - 1) / L;
            a.slab0 = (int32_t)slabs;
            a.mat0 = (int32_t)matrices;
            a.parts = ws;
            slabs += a.slabs * m.count;
            matrices += m.count;
            PACT_CHECK(slabs <= 0x7FFFFFFF, PACT_ERR_SHAPE, "%s: too many elements", what);
            ws += (size_t)m.count * ((size_t)a.slabs * tri(nb) * 64 + 64 * nb * nb);
        }
        if (p.n == 0) break;
        s = nb == 2   ? muon::launch<2>(p, (int)matrices, (int)slabs, st)
            : nb == 4 ? muon::launch<4>(p, (int)matrices, (int)slabs, st)
            : nb == 6 ? muon::launch<6>(p, (int)matrices, (int)slabs, st)
                      : muon::launch<8>(p, (int)matrices, (int)slabs, st);
        if (s != PACT_OK) return s;
    }
    return PACT_OK;
}

}  // extern "C"
