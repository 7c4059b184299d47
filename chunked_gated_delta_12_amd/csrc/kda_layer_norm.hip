// kda_layer_norm.hip -- the layer norm with its residual sum, and their backward pass.
//
// Per row of D channels, x, w and b optional:
//     r = x + y,   u = (r - mean(r)) rho,   rho = 1 / sqrt(mean((r - mean(r))^2) + eps),   h = u w + b
// and, with t = dh w:
//     dy = dx = dr + rho (t - mean(t) - u mean(t u)),   dw = sum dh u,   db = sum dh   (over rows)
// Everything is formed in fp32 and rounded once; the squares are of r less its mean, so a row far
// from zero keeps its digits; the backward pass rebuilds r from the inputs.  Both are bound by HBM: a row stays in
// registers, each operand is read once and each result written once, and the next row is asked for before
// this one's sums meet.
// Measured, bf16, all parts: forwards 65,536 rows of 2,048 channels 212 to 217 us (1.07 GB, 5 TB/s, a large copy's rate), backwards
// 16,384 rows of 2,048 75 us (336 MB, 4.5 TB/s), of 2,056 100, 4,096 of 8,192 93 (one workgroup a compute unit, whose three sums a
// row little overlaps); 7 rows of 1,000 in fp32 11 us, the call's host time.
#include "kda_launch.hpp"
#include "kda_rows.hpp"

namespace kda {

namespace {

// Lanes a row: a power of two within two wavefronts; beyond, whole wavefronts, up to eight any number, then an even one.
// Beside powers of two throughout, bf16, all parts, 2^25 values forwards and backwards: 1,536 channels 49 and 91 us, now 47 and 78;
// 2,560 50 and 102, now 47 and 93; 5,120 67 and 122, now 52 and 106; 6,144 61 and 110, now 47 and 101.
int ln_lanes(int D) {
    if (D <= 1024) return lanes_of(D);
    const int waves = (D + 511) / 512;
    return 64 * (waves <= 8 ? waves : (waves + 1) / 2 * 2);
}
constexpr int ln_block(int L) { return L > 128 ? L : 256; }

struct LnArgs {
    int64_t rows;
    int D;
    float eps;
    const void *y, *x, *dr, *dh;
    const float *w, *b;
    void *r, *h, *dy;
    float* part;   // [2][workgroup][D]: dw, db
    bool want_w, want_b;
};

// v less its row's mean, and rho.  The mean is rounded, so what is left of it is summed with the squares
// and taken off too: a row of equal values comes out as zeros, one far from zero keeps its digits.
template <int L>
__device__ __forceinline__ float centred(V8& v, bool on, float D, float eps, float* lds, int& turn) {
    float s[2] = {0.0f, 0.0f};
#pragma unroll
    for (int e = 0; e < 8; ++e) s[0] += on ? v.f[e] : 0.0f;
    float first[1] = {s[0]};
    row_sum<L>(first, lds, turn);
    const float mean = first[0] / D;
    s[0] = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        v.f[e] = on ? v.f[e] - mean : 0.0f;
        s[0] += v.f[e];
        s[1] += v.f[e] * v.f[e];
    }
    row_sum<L>(s, lds, turn);
    const float rest = s[0] / D, var = s[1] / D - rest * rest;
#pragma unroll
    for (int e = 0; e < 8; ++e) v.f[e] = on ? v.f[e] - rest : 0.0f;
    return 1.0f / sqrtf((var < 0.0f ? 0.0f : var) + eps);
}

template <typename E, int L>
__global__ void __launch_bounds__(ln_block(L)) ln_fwd_kernel(LnArgs a) {
    __shared__ float lds[64];
    constexpr int G = ln_block(L) / L;   // rows at a time
    const int lane = threadIdx.x % L, grp = threadIdx.x / L;
    const bool on = lane < a.D / 8;
    int turn = 0;
    V8 w, b;
    if (on) {
        if (a.w) w = ld8(a.w + 8 * lane);
        if (a.b) b = ld8(a.b + 8 * lane);
    }
    Raw<E> ry{}, rx{};
    auto fetch = [&](int64_t row) {
        if (row < a.rows && on) {
            const int64_t at = row * a.D + 8 * lane;
            ld_raw((const E*)a.y + at, ry);
            if (a.x) ld_raw((const E*)a.x + at, rx);
        }
    };
    fetch((int64_t)blockIdx.x * G + grp);
    for (int64_t base = (int64_t)blockIdx.x * G; base < a.rows; base += (int64_t)gridDim.x * G) {
        const int64_t row = base + grp, at = row * a.D + 8 * lane;
        const bool in = row < a.rows;
        V8 v = to_f8(ry);
        const V8 vx = to_f8(rx);
        fetch(row + (int64_t)gridDim.x * G);
        if (a.x)
#pragma unroll
            for (int e = 0; e < 8; ++e) v.f[e] += vx.f[e];
        if (a.r && in && on) st8((E*)a.r + at, v);
        const float rho = centred<L>(v, on, (float)a.D, a.eps, lds, turn);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v.f[e] *= rho;
            if (a.w) v.f[e] *= w.f[e];
            if (a.b) v.f[e] += b.f[e];
        }
        if (in && on) st8((E*)a.h + at, v);
    }
}

template <typename E, int L>
__global__ void __launch_bounds__(ln_block(L)) ln_bwd_kernel(LnArgs a) {
    __shared__ float lds[64];
    constexpr int G = ln_block(L) / L;
    constexpr int GW = L < 64 ? ln_block(L) / 64 : G;   // parts that meet in LDS: groups in one wavefront sum by lane exchange
    __shared__ float acc[GW > 1 ? GW * L * 8 : 1];
    const int lane = threadIdx.x % L, grp = threadIdx.x / L;
    const bool on = lane < a.D / 8;
    const float inv = 1.0f / (float)a.D;
    int turn = 0;
    V8 w, aw{}, ab{};
    if (on && a.w) w = ld8(a.w + 8 * lane);
    Raw<E> ry, rx, rh, rd;
    auto fetch = [&](int64_t row) {
        ry = rx = rh = rd = Raw<E>{};
        if (row < a.rows && on) {
            const int64_t at = row * a.D + 8 * lane;
            ld_raw((const E*)a.y + at, ry);
            ld_raw((const E*)a.dh + at, rh);
            if (a.x) ld_raw((const E*)a.x + at, rx);
            if (a.dr) ld_raw((const E*)a.dr + at, rd);
        }
    };
    // from 896 lanes a row on the registers do not hold a second row in fp32
    constexpr bool AHEAD = L < 896 || sizeof(E) == 2;
    if (AHEAD) fetch((int64_t)blockIdx.x * G + grp);
    for (int64_t base = (int64_t)blockIdx.x * G; base < a.rows; base += (int64_t)gridDim.x * G) {
        const int64_t row = base + grp;
        if (!AHEAD) fetch(row);
        const bool in = row < a.rows;
        V8 v = to_f8(ry), t = to_f8(rh);
        const V8 vx = to_f8(rx), vd = to_f8(rd);
        if (AHEAD) fetch(row + (int64_t)gridDim.x * G);
#pragma unroll
        for (int e = 0; e < 8; ++e) v.f[e] += vx.f[e];
        float rho = centred<L>(v, on, (float)a.D, a.eps, lds, turn);
        rho = in ? rho : 0.0f;   // eps may be 0: lanes without a row add nothing to the weights' sums
        float k[2] = {0.0f, 0.0f};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v.f[e] *= rho;
            aw.f[e] += t.f[e] * v.f[e];
            ab.f[e] += t.f[e];
            if (a.w) t.f[e] = on ? t.f[e] * w.f[e] : 0.0f;
            k[0] += t.f[e];
            k[1] += t.f[e] * v.f[e];
        }
        row_sum<L>(k, lds, turn);
#pragma unroll
        for (int e = 0; e < 8; ++e) t.f[e] = vd.f[e] + rho * (t.f[e] - k[0] * inv - v.f[e] * (k[1] * inv));
        if (in && on) st8((E*)a.dy + row * a.D + 8 * lane, t);
    }
    // the workgroup's rows, always in the same order
    for (int p = 0; p < 2; ++p) {
        if (!(p ? a.want_b : a.want_w)) continue;
        V8 s = p ? ab : aw;
        if constexpr (G > 1) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
#pragma unroll
                for (int m = L; m < 64; m <<= 1) s.f[e] += __shfl_xor(s.f[e], m);
            const int gw = L < 64 ? (int)threadIdx.x / 64 : grp;
            __syncthreads();
            if (L >= 64 || (int)(threadIdx.x & 63) < L)
#pragma unroll
                for (int e = 0; e < 8; ++e) acc[(gw * 8 + e) * L + lane] = s.f[e];
            __syncthreads();
            if (grp == 0)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float u = 0.0f;
                    for (int gg = 0; gg < GW; ++gg) u += acc[(gg * 8 + e) * L + lane];
                    s.f[e] = u;
                }
        }
        if (grp == 0 && on) st8(a.part + ((int64_t)p * gridDim.x + blockIdx.x) * a.D + 8 * lane, s);
    }
}

// Workgroups of the backward pass: as many as are resident at once, each one a row of parts.  The registers leave four
// wavefronts a SIMD, 256 compute units have four SIMDs, and a workgroup of five has two on one of them (13,107 rows of 2,560:
// two workgroups a compute unit 93 us, three 110, 819 for all of them, which is a round and a part, 140).
int ln_bwd_blocks(int64_t rows, int D) {
    const int L = ln_lanes(D), G = ln_block(L) / L;
    const int64_t want = (rows + G - 1) / G;
    const int waves = ln_block(L) / 64;
    const int64_t cap = 256 * (waves <= 4 ? 16 / waves : 4 / ((waves + 3) / 4));
    return (int)(want < cap ? want : cap);
}

template <typename E, int L>
hipError_t ln_fwd_t(const LnArgs& a, hipStream_t stream) {
    constexpr int G = ln_block(L) / L;
    const int64_t want = (a.rows + G - 1) / G;
    hipLaunchKernelGGL((ln_fwd_kernel<E, L>), dim3((unsigned)(want < 2048 ? want : 2048)), dim3(ln_block(L)), 0, stream, a);
    return hipGetLastError();
}

template <typename E, int L>
hipError_t ln_bwd_t(const LnArgs& a, float* dw, float* db, hipStream_t stream) {
    const int nblk = ln_bwd_blocks(a.rows, a.D);
    hipLaunchKernelGGL((ln_bwd_kernel<E, L>), dim3((unsigned)nblk), dim3(ln_block(L)), 0, stream, a);
    if (dw || db)
        launch_part_sums(PartSums{{a.part, a.part + (int64_t)nblk * a.D, nullptr}, {dw, db, nullptr}, {a.D, a.D, 0}, nblk}, stream);
    return hipGetLastError();
}

#define KDA_LN_SIZES(CALL)       \
    switch (ln_lanes(D)) {       \
        case 1: CALL(1);         \
        case 2: CALL(2);         \
        case 4: CALL(4);         \
        case 8: CALL(8);         \
        case 16: CALL(16);       \
        case 32: CALL(32);       \
        case 64: CALL(64);       \
        case 128: CALL(128);     \
        case 192: CALL(192);     \
        case 256: CALL(256);     \
        case 320: CALL(320);     \
        case 384: CALL(384);     \
        case 448: CALL(448);     \
        case 512: CALL(512);     \
        case 640: CALL(640);     \
        case 768: CALL(768);     \
        case 896: CALL(896);     \
        case 1024: CALL(1024);   \
    }

}  // namespace

size_t layer_norm_bwd_workspace_bytes(int64_t rows, int D) { return (size_t)ln_bwd_blocks(rows, D) * 2 * D * sizeof(float); }

hipError_t launch_layer_norm_fwd(bool f32, int64_t rows, int D, float eps, const void* y, const void* x, const float* w, const float* b,
                                 void* r, void* h, hipStream_t stream) {
    LnArgs a{};
    a.rows = rows, a.D = D, a.eps = eps, a.y = y, a.x = x, a.w = w, a.b = b, a.r = r, a.h = h;
#define KDA_LF(L) return f32 ? ln_fwd_t<float, L>(a, stream) : ln_fwd_t<bf16, L>(a, stream)
    KDA_LN_SIZES(KDA_LF)
#undef KDA_LF
    return hipErrorInvalidValue;
}

hipError_t launch_layer_norm_bwd(bool f32, int64_t rows, int D, float eps, const void* y, const void* x, const float* w, const void* dr,
                                 const void* dh, void* dy, float* dw, float* db, float* part, hipStream_t stream) {
    LnArgs a{};
    a.rows = rows, a.D = D, a.eps = eps, a.y = y, a.x = x, a.dr = dr, a.dh = dh, a.w = w, a.dy = dy, a.part = part;
    a.want_w = dw != nullptr, a.want_b = db != nullptr;
#define KDA_LB(L) return f32 ? ln_bwd_t<float, L>(a, dw, db, stream) : ln_bwd_t<bf16, L>(a, dw, db, stream)
    KDA_LN_SIZES(KDA_LB)
#undef KDA_LB
    return hipErrorInvalidValue;
}

}  // namespace kda
