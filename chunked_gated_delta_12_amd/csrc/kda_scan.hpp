// kda_scan.hpp -- what the kernels of the selective scan share.
//
// Per sequence and channel d (its group is d / (D / G)), with N states h_n from a start state:
//     delta_t = softplus(dt_t + bias)                        (or dt_t + bias)
//     h_n    <- exp(delta_t A_n) h_n + delta_t x_t b_t,n
//     y_t     = (sum_n c_t,n h_n + skip x_t) silu(z_t)
// A, the states and all arithmetic are fp32; x, dt, z, b, c, y are stored in the dtype.
//
// Lanes: four neighbouring lanes (a quad) hold one channel, N/4 states each, so a wavefront
// has 16 channels.  What belongs to a (token, channel) alone -- the step size, the gate, the
// loads and stores -- is done for four tokens at a time, one a lane, and handed round the quad
// by DPP, and so are the sums over states: with one channel a lane these would cost as much
// registers and loads for four times fewer wavefronts.
//
// Sequences are cut into pieces of `piece` tokens where there are too few channels to fill the
// device: a piece's map is (sum of delta, end state from nothing), its decay being
// exp(A sum delta) whatever its length.  The pieces of sequence n start at slot
// first(n) = its first row / piece + n (n * ceil(T / piece) for sequences of T tokens each),
// which leaves room for each sequence's last, part piece.
#pragma once

#include "kda_device.hpp"
#include "kda_launch.hpp"

namespace kda {
namespace scan {

constexpr float LOG2E = 1.4426950408889634f;
constexpr int BLOCK = 256, WAVE_CH = 16, BLOCK_CH = 64;   // threads a workgroup; channels a wavefront and a workgroup
constexpr int TILE = 32;                                  // tokens whose b and c are staged at a time

struct Seqs {
    int nseq, T, piece;
    const int* cu;
};

// What a slot has: the sequence, its rows [row0, row0 + len), the piece's number and how many there are.
struct Place {
    int seq, k, pieces, len;
    int64_t row0, first;
};

__device__ __forceinline__ int held(int v, int lo, int hi) { return v < lo ? lo : v > hi ? hi : v; }

// False where the slot has no piece.  Offsets out of order or range are held to both.
__device__ __forceinline__ bool place_of(const Seqs& s, int64_t slot, Place& p) {
    if (!s.cu) {
        const int pieces = (s.T + s.piece - 1) / s.piece;
        p.seq = (int)(slot / pieces);
        p.k = (int)(slot - (int64_t)p.seq * pieces);
        p.pieces = pieces;
        p.len = s.T;
        p.row0 = (int64_t)p.seq * s.T;
        p.first = (int64_t)p.seq * pieces;
        return true;
    }
    int lo = 0, hi = s.nseq - 1;   // the last sequence whose first slot is not behind this one
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (held(s.cu[mid], 0, s.T) / s.piece + (int64_t)mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    const int r0 = held(s.cu[lo], 0, s.T), r1 = held(s.cu[lo + 1], r0, s.T);
    p.seq = lo;
    p.row0 = r0;
    p.len = r1 - r0;
    p.first = r0 / s.piece + (int64_t)lo;
    p.pieces = p.len > s.piece ? (p.len - 1) / s.piece + 1 : 1;   // a sequence without tokens has one, empty
    const int64_t k = slot - p.first;
    p.k = (int)k;
    return k >= 0 && k < p.pieces;
}

// e^v to an ulp or two: the product's rounding is put back.
__device__ __forceinline__ float exp_full(float v) {
    const float t = v * LOG2E;
    const float r = __builtin_fmaf(v, LOG2E, -t) + v * 1.9259629911266175e-8f;   // log2(e) - LOG2E
    const float e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e, r * 0.6931471805599453f, e);
}

// softplus(v) = max(v, 0) + log(1 + e^-|v|), with log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3,
// from atanh's series: relative error below 2^-22 for every v, also where e is small and a
// logarithm of the rounded 1 + e would lose it.  The series' terms left out start at s^16 / 17 = 1.4e-9.
__device__ __forceinline__ float softplus(float v) {
    const float a = __builtin_fabsf(v);
    // e^-a is 0 in fp32 from 104 on; holding the argument keeps exp_full's correction finite at infinity
    const float e = a < 104.0f ? exp_full(-a) : a != a ? a : 0.0f;
    const float s = e * __builtin_amdgcn_rcpf(2.0f + e), q = s * s;
    float p = 1.0f / 15.0f;
    p = __builtin_fmaf(p, q, 1.0f / 13.0f);
    p = __builtin_fmaf(p, q, 1.0f / 11.0f);
    p = __builtin_fmaf(p, q, 1.0f / 9.0f);
    p = __builtin_fmaf(p, q, 1.0f / 7.0f);
    p = __builtin_fmaf(p, q, 1.0f / 5.0f);
    p = __builtin_fmaf(p, q, 1.0f / 3.0f);
    p = __builtin_fmaf(p, q, 1.0f);
    return __builtin_fmaf(2.0f * s, p, v > 0.0f ? v : 0.0f);
}

// sigmoid(v) to a few ulp; exactly 0 and 1 in the tails.
__device__ __forceinline__ float sigmoid(float v) {
    const float a = __builtin_fabsf(v);
    const float e = a < 104.0f ? exp_full(-a) : a != a ? a : 0.0f;
    const float d = 1.0f + e, r = __builtin_amdgcn_rcpf(d);
    const float i = __builtin_fmaf(r, __builtin_fmaf(-d, r, 1.0f), r);   // one step: 1 / (1 + e)
    return v < 0.0f ? e * i : i;
}

// ---------------------------------------------------------------- quads
template <int CTRL>
__device__ __forceinline__ float quad_perm(float v) {
    return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <int J>
__device__ __forceinline__ float quad_lane(float v) { return quad_perm<J * 0x55>(v); }
__device__ __forceinline__ float quad_xor1(float v) { return quad_perm<0xb1>(v); }
__device__ __forceinline__ float quad_xor2(float v) { return quad_perm<0x4e>(v); }
__device__ __forceinline__ float quad_sum(float v) {
    v += quad_xor1(v);
    return v + quad_xor2(v);
}
// Lane j of the quad gets the sum of v[j] over the quad.
__device__ __forceinline__ float quad_sums(const float* v, int q) {
    const bool b0 = q & 1, b1 = q & 2;
    const float r01 = (b0 ? v[1] : v[0]) + quad_xor1(b0 ? v[0] : v[1]);
    const float r23 = (b0 ? v[3] : v[2]) + quad_xor1(b0 ? v[2] : v[3]);
    return (b1 ? r23 : r01) + quad_xor2(b1 ? r01 : r23);
}

// ---------------------------------------------------------------- memory
// A value `bytes` behind a base that all lanes share: the base stays in scalar registers, and a
// lane's part is 32 bits (a tile of tokens is at most TILE * 2^20 channels * 4 bytes).
template <typename E>
__device__ __forceinline__ E ld_off(const E* base, uint32_t bytes) {
    return *reinterpret_cast<const E*>(reinterpret_cast<const char*>(base) + bytes);
}
template <typename E>
__device__ __forceinline__ void st_off(E* base, uint32_t bytes, float v) {
    *reinterpret_cast<E*>(reinterpret_cast<char*>(base) + bytes) = from_f<E>(v);
}

template <int NS>
__device__ __forceinline__ void ld_states(const float* p, float* out) {
    if constexpr (NS % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NS; i += 4) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(p + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) out[i + j] = a[j];
        }
    } else {
        const f32x2 a = *reinterpret_cast<const f32x2*>(p);
        out[0] = a[0];
        out[1] = a[1];
    }
}
template <int NS>
__device__ __forceinline__ void st_states(float* p, const float* x) {
    if constexpr (NS % 4 == 0) {
#pragma unroll
        for (int i = 0; i < NS; i += 4) *reinterpret_cast<f32x4*>(p + i) = f32x4{x[i], x[i + 1], x[i + 2], x[i + 3]};
    } else {
        *reinterpret_cast<f32x2*>(p) = f32x2{x[0], x[1]};
    }
}

// Four neighbouring values as they are stored, and as fp32.
template <typename E> struct Four;
template <> struct Four<float> { typedef f32x4 T; };
template <> struct Four<bf16> { typedef bf16x4 T; };
template <typename E>
__device__ __forceinline__ f32x4 to_f4(typename Four<E>::T v) { return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]}; }

// b and c of a tile of tokens on their way from memory to LDS, fp32 there: [2][TILE][N].
// Every token's row is the same for all channels of a group, so the workgroup converts it once.
// Rows behind the last token are zero, whatever follows them in memory.
template <typename E, int N>
struct Rows {
    static constexpr int VECS = 2 * TILE * N / 4, PER = (VECS + BLOCK - 1) / BLOCK;
    typename Four<E>::T v[PER];

    __device__ __forceinline__ static int token_of(int i) { return i % (VECS / 2) / (N / 4); }

    __device__ __forceinline__ void fetch(const E* b, const E* c, int64_t row, int64_t ld, int t0, int n) {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int i = p * BLOCK + (int)threadIdx.x;
            v[p] = typename Four<E>::T{};
            if (VECS % BLOCK && i >= VECS) continue;
            const int t = t0 + token_of(i);
            if (t < n) v[p] = *reinterpret_cast<const typename Four<E>::T*>((i < VECS / 2 ? b : c) + (row + t) * ld + i % (N / 4) * 4);
        }
    }
    __device__ __forceinline__ void store(float* lds) const {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int i = p * BLOCK + (int)threadIdx.x;
            if (VECS % BLOCK && i >= VECS) continue;
            *reinterpret_cast<f32x4*>(lds + 4 * i) = to_f4<E>(v[p]);
        }
    }
};

// ---------------------------------------------------------------- sizes
// Workgroups of 64 channels: none straddles two groups of channels.
__host__ __device__ __forceinline__ int blocks_of(int D, int G) { return G * ((D / G + BLOCK_CH - 1) / BLOCK_CH); }

// Slots of the pieces of all sequences.
inline int64_t slots_of(int nseq, int T, int piece, bool packed) {
    return packed ? (int64_t)T / piece + nseq : (int64_t)nseq * (((int64_t)T + piece - 1) / piece);
}

}  // namespace scan
}  // namespace kda
