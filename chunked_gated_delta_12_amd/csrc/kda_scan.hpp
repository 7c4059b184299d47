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
// which leaves room for each sequence's last, part piece.  A slot is a place in a launch alone: of maps a sequence
// has one less than pieces, floor((length - 1) / piece), which is no more than the multiples of a piece that it spans, so the first
// row / piece is their place in the workspace, and sequences that are not cut take none of it.
#pragma once

#include <type_traits>

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
    int64_t row0, map0;   // map0: the place of the sequence's first map
};

// A value that all lanes share, in a scalar register: what was loaded may have come through vector ones.
__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ int64_t uniform64(int64_t v) {
    return (int64_t)(((uint64_t)(uint32_t)uniform((int)(v >> 32)) << 32) | (uint32_t)uniform((int)v));
}

// Zeros in the rows of no sequence, those before the first and behind the last, of a tensor of D values a row: workgroup blk of
// the REST_BLOCKS that a launch has for that behind its others.
constexpr int REST_BLOCKS = 64;
template <typename E>
__device__ __forceinline__ void clear_rest(const Seqs& s, E* p, int D, int64_t blk) {
    const int lo = held(s.cu[0], 0, s.T), hi = held(s.cu[s.nseq], lo, s.T);
    const int64_t words = D / (int)(16 / sizeof(E));   // 16 bytes each; D is a multiple of 8
    const int64_t first = lo * words, gap = (hi - lo) * words, n = s.T * words - gap;
    for (int64_t i = blk * blockDim.x + threadIdx.x; i < n; i += (int64_t)REST_BLOCKS * blockDim.x)
        ((f32x4*)p)[i < first ? i : gap + i] = f32x4{};
}

// False where the slot has no piece.  Offsets out of order or range are held to both.
__device__ __forceinline__ bool place_of(const Seqs& s, int64_t slot, Place& p) {
    if (!s.cu) {
        const int pieces = (s.T - 1) / s.piece + 1;
        p.seq = uniform((int)(slot / pieces));
        p.k = (int)(slot - (int64_t)p.seq * pieces);
        p.pieces = pieces;
        p.len = s.T;
        p.row0 = (int64_t)p.seq * s.T;
        p.map0 = (int64_t)p.seq * (pieces - 1);
        return true;
    }
    // The last sequence whose first slot is not behind this one: 64 candidates at a time, so that 4,096 sequences take
    // two loads one after the other.
    const int lane = (int)threadIdx.x & 63;
    int lo = 0, n = s.nseq;   // it is one of lo .. lo + n - 1
    while (n > 1) {
        const int by = (n + 63) / 64, i = lane * by;
        const bool behind = i < n && held(s.cu[lo + i], 0, s.T) / s.piece + (int64_t)(lo + i) > slot;
        const uint64_t before = __ballot(i < n && !behind);
        // offsets that rise leave one run of candidates before; the first is taken where there is none
        const int k = before ? 63 - __builtin_clzll(before) : 0;
        lo = uniform(lo + k * by);
        n = uniform(n - k * by < by ? n - k * by : by);
    }
    const int r0 = uniform(held(s.cu[lo], 0, s.T)), r1 = uniform(held(s.cu[lo + 1], r0, s.T));
    p.seq = lo;
    p.row0 = r0;
    p.len = r1 - r0;
    p.map0 = r0 / s.piece;
    p.pieces = p.len > s.piece ? (p.len - 1) / s.piece + 1 : 1;   // a sequence without tokens has one, empty
    const int64_t k = slot - p.map0 - lo;
    p.k = (int)k;
    return k >= 0 && k < p.pieces;
}

// e^-|v|, without a branch: the hardware's power of two of the rounded product t = -|v| log2(e), and what that rounding left,
// -|v| - t ln 2, put back (of ln 2's own rounding 2.8e-9 |v| of the result stays).  0 below 2^-126; NaN stays; the hold to
// [-1, 1] is for infinities, whose difference is none.  In bf16 storage too: a step size goes on to states and gradients that are
// fp32, and without the correction up to 1.2 x 2^-24 |v| of it would be lost, v being dt + bias, for three instructions of a
// token's hundred or so.
__device__ __forceinline__ float exp_minus(float v) {
    const float a = __builtin_fabsf(v), t = a * -LOG2E, e = __builtin_amdgcn_exp2f(t);
    return __builtin_fmaf(e, __builtin_amdgcn_fmed3f(__builtin_fmaf(t, -0.6931471805599453f, -a), -1.0f, 1.0f), e);
}

// softplus(v) = max(v, 0) + log(1 + e^-|v|), with log(1 + e) = 2 atanh(s), s = e / (2 + e) <= 1/3: from e, a relative
// error of a few 2^-24 for every v, also where e is small and a logarithm of the rounded 1 + e would
// lose it.  atanh(s) / s is interpolated in s^2 on [0, 1/9] at Chebyshev's points, off by at most 4e-9 (here twice that).
__device__ __forceinline__ float softplus_of(float v, float e) {   // e = e^-|v|
    const float s = e * __builtin_amdgcn_rcpf(2.0f + e), q = s * s;
    float p = 2 * 1.4078889183e-01f;
    p = __builtin_fmaf(p, q, 2 * 1.3982578873e-01f);
    p = __builtin_fmaf(p, q, 2 * 2.0012297615e-01f);
    p = __builtin_fmaf(p, q, 2 * 3.3333160821e-01f);
    p = __builtin_fmaf(p, q, 2.0f);
    float m;
    asm("v_max_f32 %0, 0, %1" : "=v"(m) : "v"(v));   // the compiler's is two instructions; NaN comes through p
    return __builtin_fmaf(s, p, m);
}

__device__ __forceinline__ float softplus(float v) { return softplus_of(v, exp_minus(v)); }
// softplus(v) and its slope sigmoid(v), from one exponential.
__device__ __forceinline__ float softplus(float v, float& slope) {
    const float e = exp_minus(v), i = __builtin_amdgcn_rcpf(1.0f + e);
    slope = v < 0.0f ? e * i : i;
    return softplus_of(v, e);
}

// sigmoid(v) = 1 / (1 + e^-v) to a few ulp, the exponential as above; the power of two is held finite, so below e^-87 comes
// e^-87 or 0.
__device__ __forceinline__ float sigmoid(float v) {
    const float t = __builtin_fminf(v * -LOG2E, 126.0f), e = __builtin_amdgcn_exp2f(t);
    const float rest = __builtin_amdgcn_fmed3f(__builtin_fmaf(t, -0.6931471805599453f, -v), -1.0f, 1.0f);
    return __builtin_amdgcn_rcpf(1.0f + __builtin_fmaf(e, rest, e));
}
// The gate of an output that is stored in E: in bf16 from the hardware exponential and reciprocal, whose error of a few 2^-24 |v| is
// far below that rounding.  The backward pass takes sigmoid, since dA, dskip, ddt_bias and dS0 are fp32.
template <typename E> __device__ __forceinline__ float gate_sigmoid(float v);
template <> __device__ __forceinline__ float gate_sigmoid<float>(float v) { return sigmoid(v); }
template <> __device__ __forceinline__ float gate_sigmoid<bf16>(float v) { return out_sigmoid(v); }

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
// f for the quad's four lanes, the lane's number a constant.
template <typename F>
__device__ __forceinline__ void each_of_quad(F f) {
    f(std::integral_constant<int, 0>{}), f(std::integral_constant<int, 1>{}), f(std::integral_constant<int, 2>{}), f(std::integral_constant<int, 3>{});
}
// out[i] = lane J's v times x[i].  The products follow the exchange directly, so that it becomes a
// modifier of theirs: a multiplication takes a neighbour's operand, a fused one does not.
template <int J, int NS>
__device__ __forceinline__ void quad_times(float v, const float* x, float* out) {
    const float w = quad_lane<J>(v);
#pragma unroll
    for (int i = 0; i < NS; ++i) out[i] = w * x[i];
}
// s += sum over j of lane j's v times x[j].  The compiler takes the exchange into a multiplication but not into
// a fused one; the two wait states are those between a write of v and its exchange, wherever that write stands.
__device__ __forceinline__ void quad_fma(float& s, float v, const float (&x)[4]) {
    asm("s_nop 1\n\t"
        "v_fmac_f32_dpp %0, %1, %2 quad_perm:[0,0,0,0] row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %3 quad_perm:[1,1,1,1] row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %4 quad_perm:[2,2,2,2] row_mask:0xf bank_mask:0xf\n\t"
        "v_fmac_f32_dpp %0, %1, %5 quad_perm:[3,3,3,3] row_mask:0xf bank_mask:0xf"
        : "+v"(s)
        : "v"(v), "v"(x[0]), "v"(x[1]), "v"(x[2]), "v"(x[3]));
}
// Lane j of the quad gets the sum of v[j] over the quad.
__device__ __forceinline__ float quad_sums(const float* v, int q) {
    const bool b0 = q & 1, b1 = q & 2;
    const float r01 = (b0 ? v[1] : v[0]) + quad_xor1(b0 ? v[0] : v[1]);
    const float r23 = (b0 ? v[3] : v[2]) + quad_xor1(b0 ? v[2] : v[3]);
    return (b1 ? r23 : r01) + quad_xor2(b1 ? r01 : r23);
}

// ---------------------------------------------------------------- memory
// Rows of a tile of tokens through a buffer resource that ends behind the last one: the base is in
// scalar registers, a lane's part 32 bits and the same for every tile, and what lies behind is
// read as zero and not written.  NOWHERE keeps a lane without a channel out.
constexpr uint32_t NOWHERE = 0x80000000u;   // a tile has less than half of that, so what is added to it does not wrap
template <typename E>
__device__ __forceinline__ Rsrc rows_rsrc(const void* p, int64_t row, int64_t ld, int tokens) {
    // at most TILE tokens of 2^20 channels of 4 bytes
    return make_rsrc((const E*)p + row * ld, (uint32_t)tokens * (uint32_t)ld * (uint32_t)sizeof(E));
}
// A value on its way, 32 bits wide: two of bf16 would be packed into one register and taken apart again.
template <typename E> __device__ __forceinline__ uint32_t ld_one(Rsrc r, uint32_t off);
template <> __device__ __forceinline__ uint32_t ld_one<float>(Rsrc r, uint32_t off) { return __builtin_amdgcn_raw_buffer_load_b32(r, (int)off, 0, 0); }
template <> __device__ __forceinline__ uint32_t ld_one<bf16>(Rsrc r, uint32_t off) {
    return (uint32_t)(unsigned short)__builtin_amdgcn_raw_buffer_load_b16(r, (int)off, 0, 0);
}
template <typename E>
__device__ __forceinline__ float value(uint32_t raw) { return __builtin_bit_cast(float, sizeof(E) == 2 ? raw << 16 : raw); }
template <typename E> __device__ __forceinline__ void st_one(Rsrc r, uint32_t off, float v);
template <> __device__ __forceinline__ void st_one<float>(Rsrc r, uint32_t off, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), r, (int)off, 0, 0);
}
template <> __device__ __forceinline__ void st_one<bf16>(Rsrc r, uint32_t off, float v) {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(unsigned short, (bf16)v), r, (int)off, 0, 0);
}

// ---------------------------------------------------------------- vectors of states
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

// v <- exp(A2 sum_j) v + local_j along `count` pieces, the first where local and sums point, the others in steps of `by`, the loads of
// eight at a time in flight: a chain of dependent loads takes half a microsecond a piece.
template <int NS>
__device__ __forceinline__ void along_pieces(float (&v)[NS], const float (&A2)[NS], const float* local, const float* sums, int by, int count,
                                             int64_t states, int D) {
    constexpr int AT_ONCE = NS <= 4 ? 8 : NS == 8 ? 4 : 2;
    for (int k = 0; k < count; k += AT_ONCE) {
        float l[AT_ONCE][NS], s[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const int64_t j = (int64_t)by * (k + u < count ? k + u : count - 1);
            ld_states<NS>(local + j * states, l[u]);
            s[u] = sums[j * D];
        }
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u)
            if (k + u < count)
#pragma unroll
                for (int i = 0; i < NS; ++i) v[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(s[u] * A2[i]), v[i], l[u][i]);
    }
}

// Four neighbouring values as they are stored as fp32.
template <typename E>
__device__ __forceinline__ f32x4 to_f4(typename Four<E>::T v) { return f32x4{(float)v[0], (float)v[1], (float)v[2], (float)v[3]}; }

// b and c of T tokens on their way from memory to LDS, fp32 there.  Every token's row is the same
// for all channels of a group, so the workgroup converts it once.  Rows behind the last token are zero.
// A wavefront's vectors are all of b or all of c, each filled up to whole wavefronts.
template <typename E, int N, int T>
struct Rows {
    static constexpr int VECS = T * N / 4, HALF = (VECS + 63) / 64 * 64, PER = (2 * HALF + BLOCK - 1) / BLOCK;
    typename Four<E>::T v[PER];

    // b, c: at the group's first state of the first token; ld: elements a token
    __device__ __forceinline__ void fetch(const E* b, const E* c, int64_t ld, int tokens) {
        const int wave = uniform((int)threadIdx.x >> 6);
        const uint32_t bytes = ((uint32_t)(tokens - 1) * (uint32_t)ld + N) * (uint32_t)sizeof(E);
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int first = p * BLOCK + wave * 64;
            if (first >= 2 * HALF) break;
            const int i = (p * BLOCK + (int)threadIdx.x) % HALF;   // tokens from T on are behind the end
            v[p] = BufQuad<E>::ld(make_rsrc(first < HALF ? b : c, bytes),
                                  ((uint32_t)(i / (N / 4)) * (uint32_t)ld + i % (N / 4) * 4) * (uint32_t)sizeof(E), 0);
        }
    }
    // f(of c?, token, first of four states, the four)
    template <typename F>
    __device__ __forceinline__ void each(F f) const {
#pragma unroll
        for (int p = 0; p < PER; ++p) {
            const int at = p * BLOCK + (int)threadIdx.x, i = at % HALF;
            if (at < 2 * HALF && i < VECS) f(at >= HALF, i / (N / 4), i % (N / 4) * 4, to_f4<E>(v[p]));
        }
    }
    // [2][T][N]
    __device__ __forceinline__ void store(float* lds) const {
        each([&](bool of_c, int t, int n, f32x4 x) { *reinterpret_cast<f32x4*>(lds + ((of_c ? T : 0) + t) * N + n) = x; });
    }
};

// ---------------------------------------------------------------- sizes
// Workgroups of 64 channels: none straddles two groups of channels.
__host__ __device__ __forceinline__ int blocks_of(int D, int G) { return G * ((D / G + BLOCK_CH - 1) / BLOCK_CH); }

// Tokens a piece where sequences are cut: as many pieces of all rows as make 2,048 workgroups, of two tiles at the least, and at most
// 256 a sequence of T tokens, each of which puts its start together from all before it; whole tiles, no more than T has.
inline int cut_piece(int nseq, int T, int D, int G, bool packed) {
    const int64_t blocks = blocks_of(D, G), rows = packed ? T : (int64_t)nseq * T;
    const int64_t most = 2048 / blocks > 1 ? 2048 / blocks : 1, whole = ((int64_t)T + TILE - 1) / TILE * TILE;
    int64_t len = rows / most;
    if (len < 2 * TILE) len = 2 * TILE;
    if (len < ((int64_t)T + 255) / 256) len = ((int64_t)T + 255) / 256;
    len = (len + TILE - 1) / TILE * TILE;
    return (int)(len < whole ? len : whole);
}

// Slots of the pieces of all sequences.
inline int64_t slots_of(int nseq, int T, int piece, bool packed) {
    return packed ? (int64_t)T / piece + nseq : (int64_t)nseq * (((int64_t)T + piece - 1) / piece);
}

// Maps of all sequences.
inline int64_t maps_of(int nseq, int T, int piece, bool packed) {
    return packed ? (int64_t)T / piece : (int64_t)nseq * (((int64_t)T + piece - 1) / piece - 1);
}

}  // namespace scan
}  // namespace kda
