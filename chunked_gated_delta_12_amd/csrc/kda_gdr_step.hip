// kda_gdr_step.hip -- the gated delta rule with one decay a head, token by token, from
// and to a state in a pool (decode: one token a request; a few proposed tokens).
//
// With gam = e^g and the state read once for both products,
//     a = S^T k,  b = S^T q,  c = k.q
//     e = v - gam a,   o = scale (gam b + beta c e),   S <- gam S + k (beta e)^T
// so a call reads and writes each state once, whatever the number of tokens: an HBM
// stream of 8 dk dv bytes a head.  Columns of S are independent: one wavefront owns 32 of
// them, a lane dk/8 rows by 4 columns, so the state stays in registers over the tokens,
// the sums over rows are in the lane and then over 8 lanes, and no wavefront waits for another.
// 32 columns make 128-byte rows and, at one request of 32 heads, 128 wavefronts.
// Measured, 128 x 128: 256 requests of 16 heads, one token, 115 us with the call (541 MB, 4.7 TB/s;
// the kernel alone 85 us, part of the states being in the last-level cache); 32 requests of 16 heads, up to
// six tokens, 17 us; one request of 32 heads 4.1 us, its call 9 us of host time.
#include "kda_device.hpp"
#include "kda_launch.hpp"

namespace kda {

namespace {

// The sum over the eight lanes that hold one column group: lanes 8, 16 and 32 apart.
__device__ __forceinline__ float row_groups_sum(float x) {
    x += __shfl_xor(x, 8);
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

template <int N>
__device__ __forceinline__ void ld_row(const float* p, float* out) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(p + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) out[i + j] = a[j];
    }
}
template <int N>
__device__ __forceinline__ void ld_row(const bf16* p, float* out) {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
        const bf16x4 a = *reinterpret_cast<const bf16x4*>(p + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) out[i + j] = (float)a[j];
    }
}
__device__ __forceinline__ void st_quad(float* p, const float* x) { *reinterpret_cast<f32x4*>(p) = f32x4{x[0], x[1], x[2], x[3]}; }
__device__ __forceinline__ void st_quad(bf16* p, const float* x) {
    *reinterpret_cast<bf16x4*>(p) = bf16x4{(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]};
}

template <typename E, int DK>
__global__ void __launch_bounds__(64)
gdr_step_kernel(int T, int Hk, int Hv, int dv, int nslot, float scale, const E* __restrict__ q, const E* __restrict__ k,
                const E* __restrict__ v, const float* __restrict__ g, const float* __restrict__ beta, float* S,
                const int* __restrict__ slots, const int* __restrict__ ntok, E* __restrict__ o) {
    constexpr int R = DK / 8;   // rows a lane
    const int lane = threadIdx.x, cg = lane & 7, rg = lane >> 3;
    const int nslab = dv / 32;
    const int slab = (int)(blockIdx.x % (unsigned)nslab);
    const int64_t bh = blockIdx.x / (unsigned)nslab;
    const int h = (int)(bh % Hv);
    const int b = (int)(bh / Hv);
    int n = T;
    if (ntok) {
        n = ntok[b];
        n = n < T ? n : T;
    }
    const int slot = slots ? slots[b] : b;
    if (n <= 0 || slot < 0 || slot >= nslot) return;   // a padded row: nothing of it is touched
    const int col = 32 * slab + 4 * cg;
    float* Sp = S + ((int64_t)slot * Hv + h) * DK * dv + (int64_t)rg * R * dv + col;
    f32x4 s[R];
#pragma unroll
    for (int i = 0; i < R; ++i) s[i] = *reinterpret_cast<const f32x4*>(Sp + (int64_t)i * dv);
    if (slots) {   // of the rows with tokens that name one slot, the first has it; the others are padding
        int twice = 0;
        for (int i = lane; i < b; i += 64)
            if (slots[i] == slot) twice |= !ntok || ntok[i] > 0;
        if (__ballot(twice)) return;
    }
    const int hk = h / (Hv / Hk);
    const int64_t tok0 = (int64_t)b * T;
    for (int t = 0; t < n; ++t) {
        const int64_t tok = tok0 + t;
        float kr[R], qr[R], vr[4];
        ld_row<R>(k + (tok * Hk + hk) * DK + rg * R, kr);
        ld_row<R>(q + (tok * Hk + hk) * DK + rg * R, qr);
        ld_row<4>(v + (tok * Hv + h) * dv + col, vr);
        const float gam = expf(g[tok * Hv + h]), bt = beta[tok * Hv + h];
        float a[4] = {0, 0, 0, 0}, bq[4] = {0, 0, 0, 0}, c = 0.0f;
#pragma unroll
        for (int i = 0; i < R; ++i) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                a[j] += s[i][j] * kr[i];
                bq[j] += s[i][j] * qr[i];
            }
            c += kr[i] * qr[i];
        }
        c = row_groups_sum(c);
        float u[4], ov[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = row_groups_sum(a[j]);
            bq[j] = row_groups_sum(bq[j]);
            u[j] = bt * (vr[j] - gam * a[j]);
            ov[j] = scale * (gam * bq[j] + c * u[j]);
        }
#pragma unroll
        for (int i = 0; i < R; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) s[i][j] = gam * s[i][j] + kr[i] * u[j];
        if (rg == 0) st_quad(o + (tok * Hv + h) * dv + col, ov);
    }
#pragma unroll
    for (int i = 0; i < R; ++i) *reinterpret_cast<f32x4*>(Sp + (int64_t)i * dv) = s[i];
}

template <typename E, int DK>
hipError_t step_t(int B, int T, int Hk, int Hv, int dv, int nslot, float scale, const void* q, const void* k, const void* v,
                  const float* g, const float* beta, float* S, const int* slots, const int* ntok, void* o, hipStream_t stream) {
    const unsigned grid = (unsigned)((int64_t)B * Hv * (dv / 32));
    hipLaunchKernelGGL((gdr_step_kernel<E, DK>), dim3(grid), dim3(64), 0, stream, T, Hk, Hv, dv, nslot, scale, (const E*)q,
                       (const E*)k, (const E*)v, g, beta, S, slots, ntok, (E*)o);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gdr_step(bool f32, int B, int T, int Hk, int Hv, int dk, int dv, int nslot, float scale, const void* q,
                           const void* k, const void* v, const float* g, const float* beta, float* S, const int* slots,
                           const int* ntok, void* o, hipStream_t stream) {
#define KDA_GS(E, D) return step_t<E, D>(B, T, Hk, Hv, dv, nslot, scale, q, k, v, g, beta, S, slots, ntok, o, stream)
    if (f32) {
        switch (dk) {
            case 32: KDA_GS(float, 32);
            case 64: KDA_GS(float, 64);
            case 128: KDA_GS(float, 128);
        }
    } else {
        switch (dk) {
            case 32: KDA_GS(bf16, 32);
            case 64: KDA_GS(bf16, 64);
            case 128: KDA_GS(bf16, 128);
        }
    }
#undef KDA_GS
    return hipErrorInvalidValue;
}

}  // namespace kda
