// kda_gdr_prep.hip -- what the chunked gated delta rule needs of a chunk before any state
// is known: X = (I + N diag(beta))^-1 and the tokens' decays (kda_gdr.hpp), all chunks at once.
//
// One workgroup has one chunk of one value head, wavefront w its token tile w.  K K^T goes from
// global memory straight into the matrix cores (exact bf16 inputs).  Decays come from
// differences of the prefix sums in 64 bits: a strong decay early in the chunk would otherwise
// take digits from the weak ones behind it (as powers of two, which is what the hardware
// exponential takes).  X: the four diagonal 16 x 16 blocks by forward substitution in
// registers, one a wavefront, then X_mn = -X_mm sum_j M_mj X_jn block by block in fp32 on the
// fp32 matrix cores, m = 1, 2, 3, the blocks of one m on different wavefronts.
// Bound by the length of that chain of dependent steps, two thirds of the time spent waiting:
// 65,536 tokens of 16 heads, dk = 128, bf16: 160 us for 0.5 GB (3.1 TB/s; a copy takes 90 us).
#include "kda_gdr.hpp"
#include "kda_launch.hpp"

namespace kda {
namespace gdr {

namespace {

// Rows 4 B .. 4 B + 3 of the forward substitution: lane (g, r) holds rows 4 g + i of column
// r of X and of M (a diagonal block).  Group B finishes its rows, then the groups below
// take them off theirs.
template <int B>
__device__ __forceinline__ void solve_rows(f32x4& x, const f32x4& m, int lane, int g) {
    f32x4 y = x;
    y[1] -= row_lane<4 * B>(m[1]) * y[0];
    y[2] -= row_lane<4 * B>(m[2]) * y[0] + row_lane<4 * B + 1>(m[2]) * y[1];
    y[3] -= row_lane<4 * B>(m[3]) * y[0] + row_lane<4 * B + 1>(m[3]) * y[1] + row_lane<4 * B + 2>(m[3]) * y[2];
    if (g == B) x = y;
    if constexpr (B < 3) {
        const float b0 = row_to_all<B>(x[0], lane), b1 = row_to_all<B>(x[1], lane), b2 = row_to_all<B>(x[2], lane),
                    b3 = row_to_all<B>(x[3], lane);
        f32x4 z;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            z[i] = x[i] - (row_lane<4 * B>(m[i]) * b0 + row_lane<4 * B + 1>(m[i]) * b1 + row_lane<4 * B + 2>(m[i]) * b2 +
                           row_lane<4 * B + 3>(m[i]) * b3);
        if (g > B) x = z;
    }
}

// 16 x 16 fp32 tiles in LDS: M's below the diagonal, X's on and below it.
constexpr int LD = 20;
constexpr int TILE = 16 * LD;
__device__ __forceinline__ int m_tile(int m, int n) { return (m * (m - 1) / 2 + n) * TILE; }
__device__ __forceinline__ int x_tile(int m, int n) { return (6 + m * (m + 1) / 2 + n) * TILE; }

template <typename E, int DK>
__global__ void __launch_bounds__(256)
prep_kernel(Args a, const E* __restrict__ k, const float* __restrict__ gate, const float* __restrict__ beta,
            char* __restrict__ ws) {
    typedef Arith<E> A;
    constexpr int KB = DK / 32;
    __shared__ alignas(16) float tiles[16 * TILE];
    __shared__ alignas(16) double Gs[C];   // prefix sums, in powers of two
    __shared__ alignas(16) float Bs[C];
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = (int)(blockIdx.x / (unsigned)a.Hv), h = (int)(blockIdx.x % (unsigned)a.Hv);
    const Chunk ch = chunk_at(a, slot, lane);
    if (ch.n < 0) return;   // the same for the whole workgroup
    const int hk = h / (a.Hv / a.Hk);
    const int64_t ld = (int64_t)a.Hk * DK;
    const E* kc = k + ch.row0 * ld + hk * DK + 8 * g;
    char* out = ws + (int64_t)blockIdx.x * PREP_BYTES;
    const f32x4 zero = {0, 0, 0, 0};

    const int64_t at = (ch.row0 + (lane < ch.valid ? lane : 0)) * a.Hv + h;
    const float gt0 = gate[at], bt0 = beta[at];
    auto row = [&](int m) { return (int64_t)(16 * m + r < ch.valid ? 16 * m + r : ch.valid - 1) * ld; };
    typename A::Ex kw[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) kw[b] = A::ld_row(kc + row(w) + 32 * b);
    if (w == 0) {   // past the chunk's end g = 0 and beta = 0: tokens that change nothing
        const float gt = gt0 < -120.0f ? -120.0f : gt0;   // e^-120 is zero in fp32 already; keeps -inf out of the differences
        double G = lane < ch.valid ? (double)gt * 1.4426950408889634074 : 0.0;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const double up = __shfl_up(G, m);
            if (lane >= m) G += up;
        }
        const float bt = lane < ch.valid ? bt0 : 0.0f;
        Gs[lane] = G;
        Bs[lane] = bt;
        const double end = __shfl(G, 63);
        const float om = __builtin_amdgcn_exp2f((float)(end - G));
        float* f = reinterpret_cast<float*>(out + X_BYTES);
        f[lane] = __builtin_amdgcn_exp2f((float)G);
        f[C + lane] = om * bt;
        f[2 * C + lane] = om;
        f[3 * C + lane] = bt;
        reinterpret_cast<double*>(f + 4 * C)[lane] = G;
    }
    f32x4 nn[MT];   // K K^T: rows tokens of w, columns of n
#pragma unroll
    for (int n = 0; n < MT; ++n) {
        nn[n] = zero;
        if (n <= w) {
#pragma unroll
            for (int b = 0; b < KB; ++b) nn[n] = A::mma(kw[b], A::ld_row(kc + row(n) + 32 * b), nn[n]);
        }
    }
    __syncthreads();
    f32x4 md = zero;
    double Gw[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) Gw[i] = Gs[16 * w + 4 * g + i];
#pragma unroll
    for (int n = 0; n < MT; ++n) {
        if (n <= w) {
            const double Gn = Gs[16 * n + r];
            f32x4 m4;
            const float bs = Bs[16 * n + r];
#pragma unroll
            for (int i = 0; i < 4; ++i) {   // M of token 16 w + 4 g + i on token 16 n + r
                const bool in = 16 * n + r < 16 * w + 4 * g + i;
                const float d = __builtin_amdgcn_exp2f(in ? (float)(Gw[i] - Gn) : 0.0f);
                m4[i] = in ? d * nn[n][i] * bs : 0.0f;
            }
            if (n == w) {
                md = m4;
            } else {
#pragma unroll
                for (int i = 0; i < 4; ++i) tiles[m_tile(w, n) + (4 * g + i) * LD + r] = m4[i];
            }
        }
    }
    // the diagonal block of X
    f32x4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = 4 * g + i == r ? 1.0f : 0.0f;
    solve_rows<0>(x, md, lane, g);
    solve_rows<1>(x, md, lane, g);
    solve_rows<2>(x, md, lane, g);
    solve_rows<3>(x, md, lane, g);
#pragma unroll
    for (int i = 0; i < 4; ++i) tiles[x_tile(w, w) + (4 * g + i) * LD + r] = x[i];
    lds_barrier();
    // the blocks below it, row of blocks by row of blocks
    for (int m = 1; m < MT; ++m) {
        if (w < m) {
            f32x4 y = zero;
            for (int j = w; j < m; ++j) {
                const f32x4 mm = *reinterpret_cast<const f32x4*>(&tiles[m_tile(m, j) + r * LD + 4 * g]);
#pragma unroll
                for (int i = 0; i < 4; ++i) y = mfma_k4(mm[i], tiles[x_tile(j, w) + (4 * g + i) * LD + r], y);
            }
            const f32x4 xm = *reinterpret_cast<const f32x4*>(&tiles[x_tile(m, m) + r * LD + 4 * g]);
            f32x4 z = zero;
#pragma unroll
            for (int i = 0; i < 4; ++i) z = mfma_k4(xm[i], y[i], z);
#pragma unroll
            for (int i = 0; i < 4; ++i) tiles[x_tile(m, w) + (4 * g + i) * LD + r] = -z[i];
        }
        lds_barrier();
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        if (b <= w / 2) {
            const f32x4 lo = *reinterpret_cast<const f32x4*>(&tiles[x_tile(w, 2 * b) + r * LD + 4 * g]);
            const f32x4 hi = 2 * b + 1 <= w ? *reinterpret_cast<const f32x4*>(&tiles[x_tile(w, 2 * b + 1) + r * LD + 4 * g]) : zero;
            st_rec(out, lower_block(w, b), lane, lo, hi);
        }
    }
}

template <typename E, int DK>
hipError_t prep_t(const Args& a, const void* k, const float* g, const float* beta, char* ws, hipStream_t stream) {
    const dim3 grid((unsigned)(places_of(a.nseq, a.T, a.cu != nullptr, C) * a.Hv));
    hipLaunchKernelGGL((prep_kernel<E, DK>), grid, dim3(256), 0, stream, a, (const E*)k, g, beta, ws);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_prep(bool f32, int dk, const Args& a, const void* k, const float* g, const float* beta, char* ws,
                       hipStream_t stream) {
#define KDA_GP(E, D) return prep_t<E, D>(a, k, g, beta, ws, stream)
    if (f32) {
        switch (dk) {
            case 32: KDA_GP(float, 32);
            case 64: KDA_GP(float, 64);
            case 128: KDA_GP(float, 128);
        }
    } else {
        switch (dk) {
            case 32: KDA_GP(bf16, 32);
            case 64: KDA_GP(bf16, 64);
            case 128: KDA_GP(bf16, 128);
        }
    }
#undef KDA_GP
    return hipErrorInvalidValue;
}

}  // namespace gdr
}  // namespace kda
