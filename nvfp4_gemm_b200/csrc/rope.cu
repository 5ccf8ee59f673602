// rope.cu -- rotation of query and key heads by position, and its gradient (the
// rotation by the opposite angle).
//
// For a row at position p and the pair (a, b) = (x[i], x[i + D/2]) of a head:
//   y[i] = a c - b s,  y[i + D/2] = b c + a s,  c, s = cos, sin(p * inv_freq[i]).
// Bound by HBM: 2 bytes in and 2 out per element, 3 FLOPs.  The angles of a row are
// shared by its heads, so a CTA computes the cosines and sines of its rows once into
// shared memory, and each thread keeps those of its eight pairs in registers while it
// streams heads past them.  8192 rows, 32 heads of 128: 26.2 us with a cold L2, 134 MB at
// 5.1 TB/s (78% of the measured copy rate); 31.8 us with the angles read from shared memory
// for every head.
#include "overlap.cuh"
#include "quant.cuh"

namespace pact {
namespace rope {

constexpr int THREADS = 256;
constexpr int MAX_HALF = 64;    // D / 2 at most
constexpr int CHUNK = 8;        // pairs per thread: 16-byte loads of both halves

// Turns per position, inv_freq / (2 pi), by value: the caller's array is host memory.
struct Turns {
    double per_pos[MAX_HALF];
};

struct Params {
    const pact_bf16 *x;
    pact_bf16 *y;
    const int32_t *pos;
    int64_t ldx, ldy, M;
    int heads, half, inverse;
};

// R consecutive rows per CTA.
template <int R>
__global__ void __launch_bounds__(THREADS) k_rope(const Params p, const Turns turns) {
    __shared__ __align__(16) float2 cs[R][MAX_HALF];
    __shared__ int live[R];
    pdl_wait();
    const int64_t row0 = (int64_t)blockIdx.x * R;
    const int half = p.half, chunks = half / CHUNK;
    // The angle is reduced to a fraction of a turn in FP64: at position 131072 an FP32
    // angle would be off by 8e-3 radians.  sincospif of the reduced angle is then good
    // to FP32.
    for (int t = threadIdx.x; t < R * half; t += THREADS) {
        const int r = t / half, i = t - r * half;
        const int64_t row = row0 + r;
        const int pos = row < p.M ? p.pos[row] : -1;
        if (i == 0) live[r] = pos >= 0;
        const double turn = (double)pos * turns.per_pos[i];
        float s, c;
        sincospif((float)(2.0 * (turn - rint(turn))), &s, &c);
        cs[r][i] = make_float2(c, p.inverse ? -s : s);
    }
    __syncthreads();
    // A thread keeps the angles of one chunk of one row and takes every `step`-th head.  U heads are loaded
    // before any is stored: y may be x, which the compiler must assume.
    constexpr int U = 2;
    const int c = threadIdx.x % chunks, r = threadIdx.x / chunks % R, step = THREADS / (R * chunks);
    if (!live[r]) return;   // rows behind the last sequence stay as they are
    float2 v[8];
#pragma unroll
    for (int j = 0; j < 8; j += 2)
        *reinterpret_cast<float4 *>(&v[j]) = *reinterpret_cast<const float4 *>(&cs[r][c * CHUNK + j]);
    const pact_bf16 *x = p.x + (row0 + r) * p.ldx + c * CHUNK;
    pact_bf16 *y = p.y + (row0 + r) * p.ldy + c * CHUNK;
    for (int h = threadIdx.x / (R * chunks); h < p.heads; h += U * step) {
        uint4 aw[U], bw[U];
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (h + k * step >= p.heads) break;
            aw[k] = *reinterpret_cast<const uint4 *>(x + (h + k * step) * 2 * half);
            bw[k] = *reinterpret_cast<const uint4 *>(x + (h + k * step) * 2 * half + half);
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
            if (h + k * step >= p.heads) break;
            float a[8], b[8], ya[8], yb[8];
            unpack8_bf16(aw[k], a);
            unpack8_bf16(bw[k], b);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                ya[j] = a[j] * v[j].x - b[j] * v[j].y;
                yb[j] = b[j] * v[j].x + a[j] * v[j].y;
            }
            pact_bf16 *dst = y + (h + k * step) * 2 * half;
            *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(ya[0], ya[1]), pack_bf16x2(ya[2], ya[3]),
                                                         pack_bf16x2(ya[4], ya[5]), pack_bf16x2(ya[6], ya[7]));
            *reinterpret_cast<uint4 *>(dst + half) = make_uint4(pack_bf16x2(yb[0], yb[1]), pack_bf16x2(yb[2], yb[3]),
                                                                pack_bf16x2(yb[4], yb[5]), pack_bf16x2(yb[6], yb[7]));
        }
    }
}

}  // namespace rope
}  // namespace pact

extern "C" pact_status pact_rope(const pact_bf16 *x, int64_t ldx, int64_t M, int heads, int head_dim,
                                 const int32_t *positions, const double *inv_freq, int inverse, pact_bf16 *y,
                                 int64_t ldy, pact_stream_t stream) {
    using namespace pact;
    PACT_CHECK(x && y && positions && inv_freq, PACT_ERR_INVALID_ARG, "pact_rope: NULL argument");
    PACT_CHECK(head_dim == 64 || head_dim == 128, PACT_ERR_SHAPE, "pact_rope: head_dim must be 64 or 128 (got %d)",
               head_dim);
    PACT_CHECK(M >= 1 && M <= 0x7FFFFF00 && heads >= 1 && heads <= 65536, PACT_ERR_SHAPE,
               "pact_rope: M in [1, 2^31 - 256] and heads in [1, 65536] (got %lld, %d)", (long long)M, heads);
    const int64_t cols = (int64_t)heads * head_dim;
    PACT_CHECK(ldx >= cols && ldy >= cols, PACT_ERR_SHAPE, "pact_rope: leading dimensions below heads * head_dim");
    PACT_CHECK(aligned16(x) && aligned16(y) && ldx % 8 == 0 && ldy % 8 == 0 && ((uintptr_t)positions & 3) == 0,
               PACT_ERR_ALIGN, "pact_rope: 16-byte aligned rows and 4-byte aligned positions needed");
    const Rows out = matrix(y, ldy, cols, M);
    PACT_CHECK((x == y && (ldx == ldy || M == 1)) || !overlap(out, matrix(x, ldx, cols, M)), PACT_ERR_INVALID_ARG,
               "pact_rope: y overlaps x but is not x itself with its stride");
    PACT_CHECK(!overlap(out, memory(positions, 4 * M)), PACT_ERR_INVALID_ARG, "pact_rope: y overlaps positions");
    rope::Turns turns = {};
    for (int i = 0; i < head_dim / 2; ++i) turns.per_pos[i] = inv_freq[i] * 0.15915494309189533577;   // 1 / (2 pi)
    const rope::Params p = {x, y, positions, ldx, ldy, M, heads, head_dim / 2, inverse != 0};
    // Four rows to a CTA once that still gives every SM a CTA (2047 rows, 14 heads of 128: 6.3 us, 8.5 with
    // one); one row where rows are few.
    if (M >= 4 * (int64_t)sm_count())
        return launch_dep(rope::k_rope<4>, dim3((unsigned)((M + 3) / 4)), dim3(rope::THREADS), 0,
                          (cudaStream_t)stream, "pact_rope", p, turns);
    return launch_dep(rope::k_rope<1>, dim3((unsigned)M), dim3(rope::THREADS), 0, (cudaStream_t)stream, "pact_rope",
                      p, turns);
}
