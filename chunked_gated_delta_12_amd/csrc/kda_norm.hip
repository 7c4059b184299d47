// kda_norm.hip -- the norms around a block fused with its gate, residual scale and
// residual sum, and their backward pass.
//
// Per row of D channels, every part but y optional:
//     n = y rho_y w_post,   rho_y = 1 / sqrt(mean(y^2) + eps)     norm after the block
//     a = n act(z) s                                              gate, residual scale
//     r = x + a                                                   residual stream
//     h = r rho_r w_pre                                           norm before the next block
// and, with t = dh w_pre, c = dn w_post:
//     dr' = dr + rho_r t - r rho_r^3 mean(t r)      dx = dr'
//     dz = dr' s n act'(z),  dn = dr' s act(z),  dy = rho_y c - y rho_y^3 mean(c y)
//     dw_pre = sum dh r rho_r,  ds = sum dr' n act(z),  dw_post = sum dn y rho_y   (over rows)
// Everything is formed in fp32 and rounded once; h takes r before its rounding, and
// the backward pass rebuilds n, a and r from the inputs, so that the forward saves
// nothing.  Both passes are bound by HBM: a row stays in registers between its loads
// and its stores, each operand is read once and each result written once.
//
// A row belongs to L lanes (a power of two: the fewest that hold it, 8 channels
// each), so short rows share a wavefront and reduce by lane
// exchange alone, and rows above 512 channels span wavefronts and reduce through LDS.
// Workgroups walk over the rows with the weights in registers.
// Measured: forwards 1,048,576 rows of 128 channels in bf16 with y, w_post and z 160 us (805 MB, 5.0
// TB/s); backwards 16,384 rows of 2,048 channels in bf16, all parts, 120 us (537 MB, 4.5 TB/s), but
// 8,192 of 4,096 211 us and 4,096 of 8,192 182 us, where a row is eight and sixteen wavefronts', and
// 16,384 of 2,056, nearly half of the lanes idle, 356 us (all 537 MB); small calls are bound by their host time, 11 us forwards and 16 us backwards.
#include "kda_launch.hpp"
#include "kda_rows.hpp"

namespace kda {

namespace {

constexpr int NV = 1;   // vectors of 8 channels a lane

template <typename E, int L>
__global__ void __launch_bounds__(block_of(L))
norm_fwd_kernel(int64_t rows, int D, float eps, bool silu, const E* __restrict__ y, const E* x, const E* __restrict__ z,
                const float* __restrict__ w_post, const float* __restrict__ s, const float* __restrict__ w_pre,
                E* r, E* __restrict__ h) {
    __shared__ float lds[64];
    constexpr int G = block_of(L) / L;   // rows at a time
    const int lane = threadIdx.x % L, grp = threadIdx.x / L;
    const int nvec = D / 8;
    const float inv = 1.0f / (float)D;
    int turn = 0;
    bool on[NV];
    V8 wp[NV], sc[NV], wn[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = lane + i * L;
        on[i] = j < nvec;
        if (on[i]) {
            if (w_post) wp[i] = ld8(w_post + 8 * j);
            if (s) sc[i] = ld8(s + 8 * j);
            if (w_pre) wn[i] = ld8(w_pre + 8 * j);
        }
    }
    for (int64_t base = (int64_t)blockIdx.x * G; base < rows; base += (int64_t)gridDim.x * G) {
        const int64_t row = base + grp;
        const bool in = row < rows;
        V8 vy[NV], vx[NV], vz[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            vy[i] = V8{};
            vx[i] = V8{};
            vz[i] = V8{};
            const int64_t at = row * D + 8 * (lane + i * L);
            if (in && on[i]) {
                vy[i] = ld8(y + at);
                if (x) vx[i] = ld8(x + at);
                if (z) vz[i] = ld8(z + at);
            }
        }
        float rho = 1.0f;
        if (w_post) {
            float q[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) q[0] += vy[i].f[e] * vy[i].f[e];
            row_sum<L>(q, lds, turn);
            rho = 1.0f / sqrtf(q[0] * inv + eps);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float a = vy[i].f[e];
                if (w_post) a = a * rho * wp[i].f[e];
                if (z) {
                    const float sg = sigmoid<E>(vz[i].f[e]);
                    a *= silu ? vz[i].f[e] * sg : sg;
                }
                if (s) a *= sc[i].f[e];
                vx[i].f[e] += a;
                if (!on[i]) vx[i].f[e] = 0.0f;
            }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in && on[i]) st8(r + row * D + 8 * (lane + i * L), vx[i]);
        if (w_pre) {
            float q[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) q[0] += vx[i].f[e] * vx[i].f[e];
            row_sum<L>(q, lds, turn);
            const float rr = 1.0f / sqrtf(q[0] * inv + eps);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
#pragma unroll
                for (int e = 0; e < 8; ++e) vx[i].f[e] *= rr * wn[i].f[e];
                if (in && on[i]) st8(h + row * D + 8 * (lane + i * L), vx[i]);
            }
        }
    }
}

// Backward.  part: one row of sums a workgroup for each weight, [workgroup][3][D]
// (dw_post, ds, dw_pre), or NULL when no weight is given.
template <typename E, int L>
__global__ void __launch_bounds__(block_of(L))
norm_bwd_kernel(int64_t rows, int D, float eps, bool silu, const E* __restrict__ y, const E* __restrict__ x,
                const E* __restrict__ z, const float* __restrict__ w_post, const float* __restrict__ s,
                const float* __restrict__ w_pre, const E* __restrict__ dr, const E* __restrict__ dh,
                E* __restrict__ dy, E* __restrict__ dx, E* __restrict__ dz, float* __restrict__ part) {
    __shared__ float lds[64];
    constexpr int G = block_of(L) / L;
    // Groups of lanes that share a wavefront sum by lane exchange, then GW parts through LDS.
    constexpr int GW = L < 64 ? block_of(L) / 64 : G;
    __shared__ float acc_lds[GW > 1 ? GW * L * NV * 8 : 1];
    // 1,024 lanes a row leave 128 registers a lane, too few for three weights' sums beside a row:
    // the sums of w_pre are in LDS there, every lane at entries of its own
    constexpr bool PRE_LDS = L == 1024;
    __shared__ float pre_lds[PRE_LDS ? L * NV * 8 : 1];
    const int lane = threadIdx.x % L, grp = threadIdx.x / L;
    const int nvec = D / 8;
    const float inv = 1.0f / (float)D;
    int turn = 0;
    bool on[NV];
    V8 wp[NV], sc[NV], wn[NV], a_post[NV], a_s[NV], a_pre[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int j = lane + i * L;
        on[i] = j < nvec;
        a_post[i] = a_s[i] = a_pre[i] = V8{};
        if constexpr (PRE_LDS)
#pragma unroll
            for (int e = 0; e < 8; ++e) pre_lds[(i * 8 + e) * L + lane] = 0.0f;
        if (on[i]) {
            if (w_post) wp[i] = ld8(w_post + 8 * j);
            if (s) sc[i] = ld8(s + 8 * j);
            if (w_pre) wn[i] = ld8(w_pre + 8 * j);
        }
    }
    // A row's operands are asked for one row ahead (8 x 2,048 rows of 2,048 channels in bf16, all
    // parts: 185 -> 126 us); at 1,024 lanes a row the registers do not hold a second one.
    constexpr bool AHEAD = L < 1024;
    Raw<E> ry[NV], rx[NV], rz[NV], rd[NV], rh[NV];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            ry[i] = rx[i] = rz[i] = rd[i] = rh[i] = Raw<E>{};
            const int64_t at = row * D + 8 * (lane + i * L);
            if (row < rows && on[i]) {
                ld_raw(y + at, ry[i]);
                if (x) ld_raw(x + at, rx[i]);
                if (z) ld_raw(z + at, rz[i]);
                if (dr) ld_raw(dr + at, rd[i]);
                if (dh) ld_raw(dh + at, rh[i]);
            }
        }
    };
    if (AHEAD) fetch((int64_t)blockIdx.x * G + grp);
    for (int64_t base = (int64_t)blockIdx.x * G; base < rows; base += (int64_t)gridDim.x * G) {
        const int64_t row = base + grp;
        const bool in = G == 1 || row < rows;
        if (!AHEAD) fetch(row);
        V8 vy[NV], vx[NV], vz[NV], vd[NV], vh[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            vy[i] = to_f8(ry[i]);
            vx[i] = to_f8(rx[i]);
            vz[i] = to_f8(rz[i]);
            vd[i] = to_f8(rd[i]);
            vh[i] = to_f8(rh[i]);
        }
        if (AHEAD) fetch(row + (int64_t)gridDim.x * G);
        float rho = 1.0f;
        if (w_post) {
            float q[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) q[0] += vy[i].f[e] * vy[i].f[e];
            row_sum<L>(q, lds, turn);
            rho = in ? 1.0f / sqrtf(q[0] * inv + eps) : 0.0f;   // eps may be 0: lanes without a row add nothing to the weights' sums
        }
        if (dh) {
            // r from its parts, then the norm's backward into dr'
            float q[2] = {0.0f, 0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float a = vy[i].f[e];
                    if (w_post) a = a * rho * wp[i].f[e];
                    if (z) {
                        const float sg = sigmoid<E>(vz[i].f[e]);
                        a *= silu ? vz[i].f[e] * sg : sg;
                    }
                    if (s) a *= sc[i].f[e];
                    vx[i].f[e] += a;
                    if (!on[i]) vx[i].f[e] = 0.0f;
                    q[0] += vx[i].f[e] * vx[i].f[e];
                    q[1] += on[i] ? vh[i].f[e] * wn[i].f[e] * vx[i].f[e] : 0.0f;
                }
            row_sum<L>(q, lds, turn);
            const float rr = in ? 1.0f / sqrtf(q[0] * inv + eps) : 0.0f;
            const float k = rr * (rr * (q[1] * inv));   // times r rr: rr^3 alone would leave fp32's range from |r| of 1e13 and 1e-13 on
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = vx[i].f[e] * rr;
                    vd[i].f[e] += rr * vh[i].f[e] * wn[i].f[e] - u * k;
                    if constexpr (PRE_LDS) pre_lds[(i * 8 + e) * L + lane] += vh[i].f[e] * u;
                    else a_pre[i].f[e] += vh[i].f[e] * u;
                }
        }
        if (dx)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in && on[i]) st8(dx + row * D + 8 * (lane + i * L), vd[i]);
        // through the residual scale and the gate: vd becomes dn, vz dz
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float n = vy[i].f[e];
                if (w_post) n = n * rho * wp[i].f[e];
                float al = 1.0f, slope = 0.0f;
                if (z) {
                    const float zz = vz[i].f[e], sg = sigmoid<E>(zz);
                    al = silu ? zz * sg : sg;
                    slope = silu ? sg * (1.0f + zz * (1.0f - sg)) : sg * (1.0f - sg);
                }
                if (s) {
                    a_s[i].f[e] += vd[i].f[e] * n * al;
                    vd[i].f[e] *= sc[i].f[e];
                }
                if (z) {
                    vz[i].f[e] = vd[i].f[e] * n * slope;
                    vd[i].f[e] *= al;
                }
            }
        if (dz)
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in && on[i]) st8(dz + row * D + 8 * (lane + i * L), vz[i]);
        if (w_post) {
            float q[1] = {0.0f};
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) q[0] += on[i] ? vd[i].f[e] * wp[i].f[e] * vy[i].f[e] : 0.0f;
            row_sum<L>(q, lds, turn);
            const float k = rho * (rho * (q[0] * inv));
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const float u = vy[i].f[e] * rho;
                    a_post[i].f[e] += vd[i].f[e] * u;
                    vd[i].f[e] = rho * vd[i].f[e] * wp[i].f[e] - u * k;
                }
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (in && on[i]) st8(dy + row * D + 8 * (lane + i * L), vd[i]);
    }
    if (!part) return;
    // the workgroup's rows, always in the same order (20,001 rows of 64 fp32 channels: 11.5 us, with all
    // groups through LDS 12.6)
    float* out = part + (int64_t)blockIdx.x * 3 * D;
    if constexpr (PRE_LDS)
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int e = 0; e < 8; ++e) a_pre[i].f[e] = pre_lds[(i * 8 + e) * L + lane];
    for (int k = 0; k < 3; ++k) {
        if (!(k == 0 ? w_post : k == 1 ? s : w_pre)) continue;
        V8 a[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) a[i] = k == 0 ? a_post[i] : k == 1 ? a_s[i] : a_pre[i];
        if constexpr (G > 1) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < 8; ++e)
#pragma unroll
                    for (int m = L; m < 64; m <<= 1) a[i].f[e] += __shfl_xor(a[i].f[e], m);
            const int gw = L < 64 ? (int)threadIdx.x / 64 : grp;
            __syncthreads();
            if (L >= 64 || (int)(threadIdx.x & 63) < L)
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) acc_lds[((gw * NV + i) * 8 + e) * L + lane] = a[i].f[e];
            __syncthreads();
            if (grp == 0) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        float t = 0.0f;
                        for (int gg = 0; gg < GW; ++gg) t += acc_lds[((gg * NV + i) * 8 + e) * L + lane];
                        a[i].f[e] = t;
                    }
            }
        }
        if (grp == 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (on[i]) st8(out + (int64_t)k * D + 8 * (lane + i * L), a[i]);
        }
    }
}

// Sums the workgroups' rows: 64 columns and 16 row strides a workgroup.
__global__ void __launch_bounds__(1024)
norm_weights_kernel(int nrow, int D, const float* __restrict__ part, float* __restrict__ dw_post, float* __restrict__ ds,
                    float* __restrict__ dw_pre) {
    __shared__ float lds[16][64];
    float* out = blockIdx.y == 0 ? dw_post : blockIdx.y == 1 ? ds : dw_pre;
    if (!out) return;
    const int c = blockIdx.x * 64 + (threadIdx.x & 63), k = threadIdx.x >> 6;
    float t = 0.0f;
    if (c < D) {
        const float* p = part + (int64_t)blockIdx.y * D + c;
        const int64_t ld = 3 * (int64_t)D;
        float u[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        int i = k;
        for (; i + 7 * 16 < nrow; i += 8 * 16)   // eight loads in flight
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] += p[(i + 16 * j) * ld];
        for (; i < nrow; i += 16) u[0] += p[i * ld];
        t = ((u[0] + u[1]) + (u[2] + u[3])) + ((u[4] + u[5]) + (u[6] + u[7]));
    }
    lds[k][threadIdx.x & 63] = t;
    __syncthreads();
    if (k == 0 && c < D) {
        t = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += lds[i][threadIdx.x];
        out[c] = t;
    }
}

constexpr int kMaxBlocks = 2048;

}  // namespace

int norm_bwd_blocks(int64_t rows, int D) {
    const int L = lanes_of(D), G = block_of(L) / L;
    const int64_t want = (rows + G - 1) / G;
    // a workgroup's row of sums costs what a row of a gradient does: as many workgroups as are
    // resident at once (three wavefronts a SIMD), and no more
    const int64_t cap = 3 * 1024 / (block_of(L) / 64 > 4 ? block_of(L) / 64 : 4);
    return (int)(want < cap ? want : cap);
}

size_t norm_bwd_workspace_bytes(int64_t rows, int D) { return (size_t)norm_bwd_blocks(rows, D) * 3 * D * sizeof(float); }

template <typename E, int L>
static hipError_t norm_fwd_t(int64_t rows, int D, float eps, bool silu, const void* y, const void* x, const void* z,
                             const float* w_post, const float* s, const float* w_pre, void* r, void* h, hipStream_t stream) {
    constexpr int G = block_of(L) / L;
    const int64_t want = (rows + G - 1) / G;
    hipLaunchKernelGGL((norm_fwd_kernel<E, L>), dim3((unsigned)(want < kMaxBlocks ? want : kMaxBlocks)), dim3(block_of(L)), 0,
                       stream, rows, D, eps, silu, (const E*)y, (const E*)x, (const E*)z, w_post, s, w_pre, (E*)r, (E*)h);
    return hipGetLastError();
}

template <typename E, int L>
static hipError_t norm_bwd_t(int64_t rows, int D, float eps, bool silu, const void* y, const void* x, const void* z,
                             const float* w_post, const float* s, const float* w_pre, const void* dr, const void* dh, void* dy,
                             void* dx, void* dz, float* dw_post, float* ds, float* dw_pre, float* part, hipStream_t stream) {
    const int nblk = norm_bwd_blocks(rows, D);
    const bool weights = dw_post || ds || dw_pre;
    hipLaunchKernelGGL((norm_bwd_kernel<E, L>), dim3((unsigned)nblk), dim3(block_of(L)), 0, stream, rows, D, eps, silu,
                       (const E*)y, (const E*)x, (const E*)z, w_post, s, w_pre, (const E*)dr, (const E*)dh, (E*)dy, (E*)dx,
                       (E*)dz, weights ? part : nullptr);
    if (weights)
        hipLaunchKernelGGL(norm_weights_kernel, dim3((unsigned)((D + 63) / 64), 3), dim3(1024), 0, stream, nblk, D, part,
                           dw_post, ds, dw_pre);
    return hipGetLastError();
}

#define KDA_NORM_SIZES(CALL)                    \
    switch (lanes_of(D)) {                      \
        case 1: CALL(1);                        \
        case 2: CALL(2);                        \
        case 4: CALL(4);                        \
        case 8: CALL(8);                        \
        case 16: CALL(16);                      \
        case 32: CALL(32);                      \
        case 64: CALL(64);                      \
        case 128: CALL(128);                    \
        case 256: CALL(256);                    \
        case 512: CALL(512);                    \
        case 1024: CALL(1024);                  \
    }

hipError_t launch_norm_fwd(bool f32, int64_t rows, int D, float eps, bool silu, const void* y, const void* x, const void* z,
                           const float* w_post, const float* s, const float* w_pre, void* r, void* h, hipStream_t stream) {
#define KDA_NF(L)                                                                                                    \
    return f32 ? norm_fwd_t<float, L>(rows, D, eps, silu, y, x, z, w_post, s, w_pre, r, h, stream)                \
               : norm_fwd_t<bf16, L>(rows, D, eps, silu, y, x, z, w_post, s, w_pre, r, h, stream)
    KDA_NORM_SIZES(KDA_NF)
#undef KDA_NF
    return hipErrorInvalidValue;
}

hipError_t launch_norm_bwd(bool f32, int64_t rows, int D, float eps, bool silu, const void* y, const void* x, const void* z,
                           const float* w_post, const float* s, const float* w_pre, const void* dr, const void* dh, void* dy,
                           void* dx, void* dz, float* dw_post, float* ds, float* dw_pre, float* part, hipStream_t stream) {
#define KDA_NB(L)                                                                                                    \
    return f32 ? norm_bwd_t<float, L>(rows, D, eps, silu, y, x, z, w_post, s, w_pre, dr, dh, dy, dx, dz, dw_post, \
                                         ds, dw_pre, part, stream)                                                   \
               : norm_bwd_t<bf16, L>(rows, D, eps, silu, y, x, z, w_post, s, w_pre, dr, dh, dy, dx, dz, dw_post,  \
                                        ds, dw_pre, part, stream)
    KDA_NORM_SIZES(KDA_NB)
#undef KDA_NB
    return hipErrorInvalidValue;
}

}  // namespace kda
