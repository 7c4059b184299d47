// kda_rows.hpp -- building blocks of the kernels that work on rows of channels (the norms, the
// short convolution): eight channels a lane, sums over a row's lanes, sums over rows of parts.
#pragma once

#include "kda_device.hpp"

namespace kda {

namespace {

struct V8 {
    float f[8];
};

__device__ __forceinline__ V8 ld8(const float* p) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
    return V8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
}
__device__ __forceinline__ V8 ld8(const bf16* p) {
    const bf16x8 a = *reinterpret_cast<const bf16x8*>(p);
    V8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v.f[i] = (float)a[i];
    return v;
}
// Eight channels as they are stored, on their way.
template <typename E> struct Raw;
template <> struct Raw<float> { f32x4 a, b; };
template <> struct Raw<bf16> { bf16x8 a; };
__device__ __forceinline__ void ld_raw(const float* p, Raw<float>& x) {
    x.a = *reinterpret_cast<const f32x4*>(p);
    x.b = *reinterpret_cast<const f32x4*>(p + 4);
}
__device__ __forceinline__ void ld_raw(const bf16* p, Raw<bf16>& x) { x.a = *reinterpret_cast<const bf16x8*>(p); }
__device__ __forceinline__ V8 to_f8(const Raw<float>& x) {
    return V8{{x.a[0], x.a[1], x.a[2], x.a[3], x.b[0], x.b[1], x.b[2], x.b[3]}};
}
__device__ __forceinline__ V8 to_f8(const Raw<bf16>& x) {
    V8 v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v.f[i] = (float)x.a[i];
    return v;
}
__device__ __forceinline__ void st8(float* p, const V8& v) {
    *reinterpret_cast<f32x4*>(p) = f32x4{v.f[0], v.f[1], v.f[2], v.f[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{v.f[4], v.f[5], v.f[6], v.f[7]};
}
__device__ __forceinline__ void st8(bf16* p, const V8& v) {
    bf16x8 a;
#pragma unroll
    for (int i = 0; i < 8; ++i) a[i] = (bf16)v.f[i];
    *reinterpret_cast<bf16x8*>(p) = a;
}

// sigmoid(z): in fp32 storage from the library exponential and a true division
// (a unit or two in the last place); in bf16 storage from the hardware exponential and reciprocal,
// whose error of a few 2^-23 |z| is far below the rounding of what is stored in bf16.  Weights' gradients are fp32: there it is a
// term's, of sums over all rows whose own roundings are as large (convolution, 32,768 rows by 2,048 channels, against 64 bits: dw off by
// 1.83e-7 and dbias by 1.86e-7 of their root mean square; with a sigmoid of a few 2^-24 1.84e-7 and 1.84e-7, in 2% more time).
template <typename E> __device__ __forceinline__ float sigmoid(float z);
template <> __device__ __forceinline__ float sigmoid<float>(float z) { return 1.0f / (1.0f + expf(-z)); }
template <> __device__ __forceinline__ float sigmoid<bf16>(float z) { return out_sigmoid(z); }

// Sums of K values over the L lanes of a row, in a fixed order.  Rows that span
// wavefronts exchange through one of two LDS areas in turn, so one barrier each is
// enough: an area is written again only after the barrier of the other's sum.
template <int L, int K>
__device__ __forceinline__ void row_sum(float (&v)[K], float* lds, int& turn) {
#pragma unroll
    for (int m = 1; m < (L < 64 ? L : 64); m <<= 1)
#pragma unroll
        for (int k = 0; k < K; ++k) v[k] += __shfl_xor(v[k], m);
    if constexpr (L > 64) {
        constexpr int W = L / 64;
        const int wave = threadIdx.x >> 6, first = wave / W * W;
        float* area = lds + turn * 32;
        turn ^= 1;
        if ((threadIdx.x & 63) == 0) {
#pragma unroll
            for (int k = 0; k < K; ++k) area[wave * 2 + k] = v[k];
        }
        lds_barrier();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float s = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) s += area[(first + w) * 2 + k];
            v[k] = s;
        }
    }
}

constexpr int block_of(int L) { return L > 256 ? L : 256; }

// Lanes a row: the fewest (a power of two) that hold it.
inline int lanes_of(int D) {
    int L = 1;
    while (L * 8 < D) L <<= 1;
    return L;
}

// Columns of up to three tables of parts, [rows][width] each, summed over their rows in a fixed
// order: 64 columns and 16 row strides a workgroup.
struct PartSums {
    const float* from[3];
    float* to[3];       // NULL: not asked for
    int64_t width[3], rows;
};
__device__ __forceinline__ void part_sums(const PartSums& s, int64_t blk) {   // 1,024 threads
    __shared__ float lds[16][64];
    int k = 0;
    for (; k < 2 && blk >= (s.width[k] + 63) / 64; ++k) blk -= (s.width[k] + 63) / 64;
    if (!s.to[k]) return;
    const int64_t c = blk * 64 + (threadIdx.x & 63), width = s.width[k];
    const int first = threadIdx.x >> 6;
    float t = 0.0f;
    if (c < width) {
        const float* p = s.from[k] + c;
        float u[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        int64_t i = first;
        for (; i + 7 * 16 < s.rows; i += 8 * 16)   // eight loads in flight
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] += p[(i + 16 * j) * width];
        for (; i < s.rows; i += 16) u[0] += p[i * width];
        t = ((u[0] + u[1]) + (u[2] + u[3])) + ((u[4] + u[5]) + (u[6] + u[7]));
    }
    lds[first][threadIdx.x & 63] = t;
    __syncthreads();
    if (first == 0 && c < width) {
        t = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; ++i) t += lds[i][threadIdx.x];
        s.to[k][c] = t;
    }
}
inline int64_t part_sums_blocks(const PartSums& s) {
    int64_t blocks = 0;
    for (int k = 0; k < 3; ++k) blocks += (s.width[k] + 63) / 64;
    return blocks;
}
template <int = 0>   // a template: files without a call have no copy of it
__global__ void __launch_bounds__(1024) part_sums_kernel(PartSums s) { part_sums(s, blockIdx.x); }
inline void launch_part_sums(const PartSums& s, hipStream_t stream) {
    hipLaunchKernelGGL(part_sums_kernel<>, dim3((unsigned)part_sums_blocks(s)), dim3(1024), 0, stream, s);
}

}  // namespace

}  // namespace kda
