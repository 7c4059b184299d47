// kda_scan_step.hip -- the selective scan token by token, from and to states in a pool
// (decode: one token a request; a few proposed tokens).  kda_scan.hpp has the formulas.
//
// A call reads and writes each state once, whatever the number of tokens: an HBM stream of
// 8 D N bytes a request.  Four lanes a channel, so that a wavefront's states are one run of
// 16 N floats, and four tokens at a time, as in the walk over whole sequences.
// Measured, 2,048 channels of 16 states, bf16: 256 requests 17.5 us (71 MB, 4.1 TB/s; the states of 34 MB are partly in
// the last-level cache), one request 10.5 us, its call's host time; 4,096 requests of 256 channels 50 us, half of it the search for duplicates.
#include "kda_scan.hpp"

namespace kda {
namespace scan {

struct StepArgs {
    int T, D, G, nslot;
    bool softplus;
    const void *x, *dt, *b, *c, *z;
    const float *A, *skip, *bias;
    float* S;
    const int *slots, *ntok;
    void* y;
};

// NS values as they are stored.
template <typename E, int NS>
struct StateVec {
    static constexpr int V = NS < 4 ? NS : 4;
    typedef E T __attribute__((__vector_size__(V * sizeof(E))));
    T v[NS / V];
    __device__ __forceinline__ void load(const E* p) {
#pragma unroll
        for (int i = 0; i < NS / V; ++i) v[i] = *reinterpret_cast<const T*>(p + V * i);
    }
    __device__ __forceinline__ float at(int i) const { return (float)v[i / V][i % V]; }
};

template <typename E, int NS>
__global__ void __launch_bounds__(BLOCK) scan_step(StepArgs a) {
    constexpr int N = 4 * NS;
    const int per = (a.D / a.G + BLOCK_CH - 1) / BLOCK_CH, nblk = a.G * per;
    const int blk = (int)(blockIdx.x % (unsigned)nblk), r = (int)(blockIdx.x / (unsigned)nblk);
    const int grp = blk / per, Dg = a.D / a.G;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, q = lane & 3;
    const int in_group = (blk % per) * BLOCK_CH + wave * WAVE_CH + (lane >> 2);
    int n = a.T;
    if (a.ntok) {
        n = a.ntok[r];
        n = n < a.T ? n : a.T;
    }
    const int slot = a.slots ? a.slots[r] : r;
    if (n <= 0 || slot < 0 || slot >= a.nslot) return;   // a padded row: nothing of it is touched
    const bool real = in_group < Dg;
    const int ch = grp * Dg + (real ? in_group : Dg - 1);
    float* Sp = a.S + ((int64_t)slot * a.D + ch) * N + q * NS;
    const int64_t row = (int64_t)r * a.T, ld = (int64_t)a.G * N;
    const E *b = (const E*)a.b + row * ld + grp * N + q * NS, *c = (const E*)a.c + row * ld + grp * N + q * NS;
    // everything that the first tokens take is asked for before the search for an earlier row of the slot
    float h[NS], A2[NS];
    ld_states<NS>(Sp, h);
    ld_states<NS>(a.A + (int64_t)ch * N + q * NS, A2);
    const float bias = a.bias ? a.bias[ch] : 0.0f, skip = a.skip ? a.skip[ch] : 0.0f;
    E xr, dr, zr;
    auto fetch = [&](int t0) {
        const int64_t off = (row + (t0 + q < n ? t0 + q : n - 1)) * a.D + ch;
        xr = ((const E*)a.x)[off];
        dr = ((const E*)a.dt)[off];
        if (a.z) zr = ((const E*)a.z)[off];
    };
    StateVec<E, NS> nb, nc;
    fetch(0);
    nb.load(b);
    nc.load(c);
    if (a.slots) {   // of the rows with tokens that name one slot, the first has it; the others are padding
        if (earlier_row(a.slots, a.ntok, r, slot, lane)) return;
    }
#pragma unroll
    for (int i = 0; i < NS; ++i) A2[i] *= LOG2E;
    for (int t0 = 0; t0 < n; t0 += 4) {
        const float xv = (float)xr, zv = a.z ? (float)zr : 0.0f;
        float d = (float)dr + bias;
        if (t0 + 4 < n) fetch(t0 + 4);
        if (a.softplus) d = softplus(d);
        const float u = d * xv;
        float yj[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        each_of_quad([&](auto J) {
            constexpr int j = decltype(J)::value;
            if (t0 + j >= n) return;
            const StateVec<E, NS> bv = nb, cv = nc;
            if (t0 + j + 1 < n) {   // the next token's
                nb.load(b + (t0 + j + 1) * ld);
                nc.load(c + (t0 + j + 1) * ld);
            }
            const float dj = quad_lane<j>(d), uj = quad_lane<j>(u);
            float s = 0.0f;
#pragma unroll
            for (int i = 0; i < NS; ++i) {
                h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(dj * A2[i]), h[i], uj * bv.at(i));
                s = i ? __builtin_fmaf(cv.at(i), h[i], s) : cv.at(i) * h[i];
            }
            yj[j] = s;
        });
        float yv = quad_sums(yj, q);
        if (a.skip) yv = __builtin_fmaf(skip, xv, yv);
        if (a.z) yv *= zv * gate_sigmoid<E>(zv);
        if (t0 + q < n && real) ((E*)a.y)[(row + t0 + q) * a.D + ch] = from_f<E>(yv);
    }
    if (real) st_states<NS>(Sp, h);
}

template <typename E, int NS>
static hipError_t step_t(int B, const StepArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((scan_step<E, NS>), dim3((unsigned)((int64_t)B * blocks_of(a.D, a.G))), dim3(BLOCK), 0, stream, a);
    return hipGetLastError();
}

}  // namespace scan

int64_t scan_step_workgroups(int B, int D, int G) { return (int64_t)B * scan::blocks_of(D, G); }

hipError_t launch_scan_step(bool f32, int B, int T, int D, int N, int G, int nslot, bool softplus, const void* x, const void* dt,
                            const float* A, const void* b, const void* c, const float* skip, const void* z, const float* bias,
                            float* S, const int* slots, const int* ntok, void* y, hipStream_t stream) {
    const scan::StepArgs a{T, D, G, nslot, softplus, x, dt, b, c, z, A, skip, bias, S, slots, ntok, y};
#define KDA_SS(N) return f32 ? scan::step_t<float, N / 4>(B, a, stream) : scan::step_t<bf16, N / 4>(B, a, stream)
    switch (N) {
        case 8: KDA_SS(8);
        case 16: KDA_SS(16);
        case 32: KDA_SS(32);
        case 64: KDA_SS(64);
    }
#undef KDA_SS
    return hipErrorInvalidValue;
}

}  // namespace kda
