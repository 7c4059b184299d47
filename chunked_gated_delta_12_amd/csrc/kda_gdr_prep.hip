// kda_gdr_prep.hip -- what the chunked gated delta rule needs of a chunk before any state
// is known: X = (I + N diag(beta))^-1 and P (kda_gdr.hpp), all chunks at once.
//
// One workgroup has one chunk of one value head, wavefront w its token tile w.  Operands
// of the two products Q K^T and K K^T go from global memory straight into the matrix
// cores (exact bf16 inputs), P as K Q^T so that its result sits in the lanes as the
// fragment that the chain reads.  Decays come from differences of the prefix sums in 64
// bits: a strong decay early in the chunk would otherwise take digits from the weak ones
// behind it.  X: the four diagonal 16 x 16 blocks by forward substitution in registers,
// one a wavefront, then X_mn = -X_mm sum_j M_mj X_jn block by block in fp32 on the fp32
// matrix cores, m = 1, 2, 3, the blocks of one m on different wavefronts.
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

constexpr int LD = 68;   // row length of the fp32 tiles in LDS

template <typename E, int DK, bool BWD>
__global__ void __launch_bounds__(256)
prep_kernel(Args a, const E* __restrict__ q, const E* __restrict__ k, const float* __restrict__ gate,
            const float* __restrict__ beta, char* __restrict__ ws) {
    typedef Arith<E> A;
    constexpr int KB = DK / 32;
    __shared__ alignas(16) float Ms[C * LD];
    __shared__ alignas(16) float Xs[C * LD];
    __shared__ double Gs[C];
    __shared__ float Bs[C];
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int slot = (int)(blockIdx.x / (unsigned)a.Hv), h = (int)(blockIdx.x % (unsigned)a.Hv);
    const Chunk ch = chunk_at(a, slot, lane);
    if (ch.n < 0) return;   // the same for the whole workgroup
    const int hk = h / (a.Hv / a.Hk);
    const int64_t ld = (int64_t)a.Hk * DK;
    const E* kc = k + ch.row0 * ld + hk * DK + 8 * g;
    const E* qc = q + ch.row0 * ld + hk * DK + 8 * g;
    char* out = ws + (int64_t)blockIdx.x * prep_bytes(BWD);

    if (w == 0) {   // prefix sums; past the chunk's end g = 0 and beta = 0: tokens that change nothing
        const int64_t at = (ch.row0 + (lane < ch.valid ? lane : 0)) * a.Hv + h;
        float gt = gate[at];
        const float bt = beta[at];
        gt = gt < -120.0f ? -120.0f : gt;   // e^-120 is zero in fp32 already; keeps -inf out of the differences
        double G = lane < ch.valid ? (double)gt : 0.0;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) {
            const double up = __shfl_up(G, m);
            if (lane >= m) G += up;
        }
        Gs[lane] = G;
        Bs[lane] = lane < ch.valid ? bt : 0.0f;
        const double end = __shfl(G, 63);
        float* gm = reinterpret_cast<float*>(out + prep_bytes(BWD) - 2 * C * 4);
        if (BWD) reinterpret_cast<double*>(out + 4 * TRI_BYTES)[lane] = G;
        gm[lane] = expf((float)G);
        gm[C + lane] = expf((float)(end - G));
    }
    auto row = [&](int m) { return (int64_t)(16 * m + r < ch.valid ? 16 * m + r : ch.valid - 1) * ld; };
    typename A::Ex kw[KB], qw[KB];
#pragma unroll
    for (int b = 0; b < KB; ++b) {
        kw[b] = A::ld_row(kc + row(w) + 32 * b);
        qw[b] = A::ld_row(qc + row(w) + 32 * b);
    }
    const f32x4 zero = {0, 0, 0, 0};
    f32x4 nn[MT], pp[MT], pt[MT];
#pragma unroll
    for (int n = 0; n < MT; ++n) {
        nn[n] = pp[n] = pt[n] = zero;
        if (n <= w) {
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                const typename A::Ex kn = A::ld_row(kc + row(n) + 32 * b);
                nn[n] = A::mma(kw[b], kn, nn[n]);   // rows tokens of w, columns tokens of n
                pp[n] = A::mma(kn, qw[b], pp[n]);   // rows keys of n, columns queries of w
            }
        }
        if (BWD && n >= w) {
#pragma unroll
            for (int b = 0; b < KB; ++b)
                pt[n] = A::mma(A::ld_row(qc + row(n) + 32 * b), kw[b], pt[n]);   // rows queries of n, columns keys of w
        }
    }
    __syncthreads();
    f32x4 md = zero;
#pragma unroll
    for (int n = 0; n < MT; ++n) {
        if (n <= w) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * w + 4 * g + i, s = 16 * n + r;
                const bool in = s < t;
                const float d = expf(in ? (float)(Gs[t] - Gs[s]) : 0.0f);
                const float m = in ? d * nn[n][i] * Bs[s] : 0.0f;
                Ms[t * LD + s] = m;
                if (n == w) md[i] = m;
                const int t2 = 16 * w + r, s2 = 16 * n + 4 * g + i;
                const bool in2 = s2 <= t2;
                const float d2 = expf(in2 ? (float)(Gs[t2] - Gs[s2]) : 0.0f);
                pp[n][i] = in2 && t2 < ch.valid ? a.scale * d2 * pp[n][i] : 0.0f;
            }
        }
        if (BWD && n >= w) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = 16 * n + 4 * g + i, s = 16 * w + r;
                const bool in = s <= t;
                const float d = expf(in ? (float)(Gs[t] - Gs[s]) : 0.0f);
                pt[n][i] = in && t < ch.valid ? a.scale * d * pt[n][i] : 0.0f;
            }
        }
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        if (b <= w / 2) A::st_sp(out + TRI_BYTES, lower_block(w, b), lane, A::split(pp[2 * b], pp[2 * b + 1]));
        if (BWD && b >= w / 2) A::st_sp(out + 3 * TRI_BYTES, upper_block(w, b), lane, A::split(pt[2 * b], pt[2 * b + 1]));
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
    for (int i = 0; i < 4; ++i) Xs[(16 * w + 4 * g + i) * LD + 16 * w + r] = x[i];
    __syncthreads();
    // the blocks below it, row of blocks by row of blocks
    for (int m = 1; m < MT; ++m) {
        if (w < m) {
            f32x4 y = zero;
            for (int j = w; j < m; ++j) {
                const f32x4 mm = *reinterpret_cast<const f32x4*>(&Ms[(16 * m + r) * LD + 16 * j + 4 * g]);
#pragma unroll
                for (int i = 0; i < 4; ++i) y = mfma_k4(mm[i], Xs[(16 * j + 4 * g + i) * LD + 16 * w + r], y);
            }
            const f32x4 xm = *reinterpret_cast<const f32x4*>(&Xs[(16 * m + r) * LD + 16 * m + 4 * g]);
            f32x4 z = zero;
#pragma unroll
            for (int i = 0; i < 4; ++i) z = mfma_k4(xm[i], y[i], z);
#pragma unroll
            for (int i = 0; i < 4; ++i) Xs[(16 * m + 4 * g + i) * LD + 16 * w + r] = -z[i];
        }
        __syncthreads();
    }
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        if (b <= w / 2) {
            const float* p = &Xs[(16 * w + r) * LD + 32 * b + 4 * g];
            const f32x4 lo = *reinterpret_cast<const f32x4*>(p);
            const f32x4 hi = 2 * b + 1 <= w ? *reinterpret_cast<const f32x4*>(p + 16) : zero;
            A::st_sp(out, lower_block(w, b), lane, A::split(lo, hi));
        }
        if (BWD && b >= w / 2) {
            f32x4 lo = zero, hi;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (2 * b >= w) lo[i] = Xs[(32 * b + 4 * g + i) * LD + 16 * w + r];
                hi[i] = Xs[(32 * b + 16 + 4 * g + i) * LD + 16 * w + r];
            }
            A::st_sp(out + 2 * TRI_BYTES, upper_block(w, b), lane, A::split(lo, hi));
        }
    }
}

template <typename E, int DK>
hipError_t prep_t(bool bwd, const Args& a, int64_t slots, const void* q, const void* k, const float* g, const float* beta,
                  char* ws, hipStream_t stream) {
    const dim3 grid((unsigned)(slots * a.Hv));
    if (bwd)
        hipLaunchKernelGGL((prep_kernel<E, DK, true>), grid, dim3(256), 0, stream, a, (const E*)q, (const E*)k, g, beta, ws);
    else
        hipLaunchKernelGGL((prep_kernel<E, DK, false>), grid, dim3(256), 0, stream, a, (const E*)q, (const E*)k, g, beta, ws);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_prep(bool f32, int dk, bool bwd, const Args& a, const void* q, const void* k, const float* g,
                       const float* beta, char* ws, hipStream_t stream) {
    const int64_t slots = slots_of(a.nseq, a.T, a.cu != nullptr);
#define KDA_GP(E, D) return prep_t<E, D>(bwd, a, slots, q, k, g, beta, ws, stream)
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
