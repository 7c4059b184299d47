// kda_scan_bwd.hip -- the backward pass of the selective scan (kda_scan.hpp has the forward's
// formulas and how lanes and pieces are laid out).
//
// With dy' = dy silu(z), a_t,n = exp(delta_t A_n), and from the last token to the first, mu
// starting as the last state's gradient:
//     lam_n  = c_t,n dy'_t + mu_n                       gradient of h_t
//     dc_t,n = dy'_t h_t,n,   db_t,n = u_t lam_n        summed over a group's channels, u = delta x
//     w_n    = lam_n a_t,n h_t-1,n
//     ddelta = x_t sum_n lam_n b_t,n + sum_n A_n w_n    dx_t = delta_t sum_n lam_n b_t,n + skip dy'_t
//     dA_n  += delta_t w_n                              mu_n = a_t,n lam_n
// and ddt = ddelta softplus'(dt + bias), dz = dy (sum_n c h + skip x) silu'(z).
//
// Three launches.  Maps: every piece forwards from nothing, leaving the state before each 16
// tokens but the first, the piece's end state, and its part of the state's gradient before it (which needs the running product of
// the decays only, so it is formed in the same sweep).  Gradients: every piece backwards, 16 tokens at a time; a
// state's 16 decays and states stay in registers between the sweep forwards and the one back.  Sums: what
// several workgroups have parts of, always in the same order.
//
// What bounds it: vector instructions, eight a token, channel and state in the maps and twenty in the gradients, of which
// four are the sums over channels for db and dc: every lane's values of 16 tokens meet over the wavefront's 16 channels,
// halved at each exchange.  The gradients' registers are the other bound: 16 tokens' three sums over states, decays and states
// are 80 a lane, so the per-state values wait in LDS and the loop over states holds one (as one unrolled
// piece of code the compiler spills), b and c are read four tokens at a time, and bf16 at 16 states fits 168 registers, three
// wavefronts a SIMD; with two, 1,022 us where it took 900.  The sums over channels on the fp32 matrix instructions (a product with one
// column a token) came to 1,435 us of a call of 1,225 for dc alone, 1,626 for both: their 32 cycles each add to the vector
// instructions' time.
// Measured, 8 x 4,096 tokens by 2,048 channels, 16 states, bf16, every part: 1,228 us (maps 324, gradients 890 and sums 32 under the profiler;
// 0.94 GB in and out, and 0.8 GB through the workspace); four packed sequences of 4,096 tokens by 512 channels in fp32 70 us.  At 64 states
// a workgroup's LDS, 141,312 bytes, leaves one a compute unit, one wavefront a SIMD, where the registers (201 and 205) would hold two.
#include "kda_rows.hpp"
#include "kda_scan.hpp"

namespace kda {
namespace scan {

constexpr int CH = 16;         // tokens at a time
constexpr int BPAD = CH + 4;   // floats a state's row of b or c in LDS: four lanes' rows start in different banks

struct BwdArgs {
    Seqs seqs;
    int D, G;
    bool softplus;
    const void *x, *dt, *b, *c, *z, *dy;
    const float *A, *skip, *bias, *S0, *dS_T;
    void *dx, *ddt, *dz;
    float* dS0;
    // workspace.  Of each piece with one behind it: end state [map][D][N]; of each with one before it: gradient before it [map][D][N],
    // sum of delta [map][D].  Of each 16 tokens of a piece but its first: state before them [chunk][D][N], sum of delta
    // before them within the piece [chunk][D]; chunk 0 is zeros, which is what a piece's first 16 tokens have.
    float *local, *grad, *sums, *start, *before;
    // parts: dA [part][D][N], dskip and dbias [part][D], db and dc [workgroup of channels][row][2][N]
    float *pA, *pskip, *pbias, *pbc;
    int64_t rows, slots, parts;
};

// The chunk before a sequence's second 16 tokens, by the rule of its maps' places.
__device__ __forceinline__ int64_t first_chunk(const Seqs& s, const Place& p) {
    return s.cu ? p.row0 / CH : (int64_t)p.seq * ((s.T + CH - 1) / CH - 1);
}

// BACK: sequences may be cut, and the gradient before a piece is asked for (the first piece's goes unused).
template <typename E, int NS, bool SOFTPLUS, bool BACK>
__global__ void __launch_bounds__(BLOCK) scan_bwd_map(BwdArgs a) {
    constexpr int N = 4 * NS, GROUPS = TILE / 4;
    __shared__ float rows[2][2 * TILE * N];
    const int per = (a.D / a.G + BLOCK_CH - 1) / BLOCK_CH, nblk = a.G * per;
    const int blk = (int)(blockIdx.x % (unsigned)nblk);
    const int64_t slot = blockIdx.x / (unsigned)nblk;
    const int grp = blk / per, Dg = a.D / a.G;
    const int lane = threadIdx.x & 63, q = lane & 3;
    const int in_group = (blk % per) * BLOCK_CH + (int)(threadIdx.x >> 6) * WAVE_CH + (lane >> 2);
    const bool real = in_group < Dg;
    const int ch = grp * Dg + (real ? in_group : Dg - 1);
    const int64_t at_state = (int64_t)ch * N + q * NS, states = (int64_t)a.D * N;
    if (slot == 0 && real) {
        const float zero[NS] = {};
        st_states<NS>(a.start + at_state, zero);
        if (q == 0) a.before[ch] = 0.0f;
    }
    Place pl;
    if (!place_of(a.seqs, slot, pl)) return;
    const int t_first = pl.k * a.seqs.piece;
    const int n = uniform(pl.len - t_first < a.seqs.piece ? pl.len - t_first : a.seqs.piece);
    const int64_t row = uniform64(pl.row0 + t_first);
    const int64_t ld = (int64_t)a.G * N;
    const bool gated = a.z != nullptr;
    uint32_t own[GROUPS];
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) own[g] = real ? ((uint32_t)(4 * g + q) * (uint32_t)a.D + ch) * (uint32_t)sizeof(E) : NOWHERE;
    const float bias = a.bias ? a.bias[ch] : 0.0f;
    float* start = a.start + (first_chunk(a.seqs, pl) + t_first / CH) * states + at_state;
    float* before = a.before + (first_chunk(a.seqs, pl) + t_first / CH) * a.D + ch;

    Rows<E, N, TILE> next;
    uint32_t nx[GROUPS], nt[GROUPS], nz[GROUPS], nd[GROUPS];
    auto tokens_at = [&](int t0) { return uniform(n - t0 < 0 ? 0 : n - t0 < TILE ? n - t0 : TILE); };
    auto fetch_rows = [&](int t0) {
        const int64_t at = (row + t0) * ld + grp * N;
        next.fetch((const E*)a.b + at, (const E*)a.c + at, ld, tokens_at(t0));
    };
    // a lane's own tokens are asked for a tile ahead, each as soon as the one in its place is used
    Rsrc rx, rt, rd, rz;
    auto at_tile = [&](int t0) {
        const int tokens = tokens_at(t0);
        rx = rows_rsrc<E>(a.x, row + t0, a.D, tokens), rt = rows_rsrc<E>(a.dt, row + t0, a.D, tokens);
        if (BACK) rd = rows_rsrc<E>(a.dy, row + t0, a.D, tokens), rz = rows_rsrc<E>(a.z, gated ? row + t0 : 0, a.D, gated ? tokens : 0);
    };
    auto fetch = [&](int g) {
        nx[g] = ld_one<E>(rx, own[g]);
        nt[g] = ld_one<E>(rt, own[g]);
        if (BACK) {
            nd[g] = ld_one<E>(rd, own[g]);
            nz[g] = ld_one<E>(rz, own[g]);
        }
    };
    if (n > 0) {
        fetch_rows(0);
        at_tile(0);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) fetch(g);
    }
    float A2[NS], h[NS], m[NS], P[NS];
    ld_states<NS>(a.A + at_state, A2);
#pragma unroll
    for (int i = 0; i < NS; ++i) A2[i] *= LOG2E, h[i] = m[i] = 0.0f, P[i] = 1.0f;
    if (pl.k == 0 && a.S0) ld_states<NS>(a.S0 + (int64_t)pl.seq * states + at_state, h);
    float sum = 0.0f;
    for (int t0 = 0, buf = 0; t0 < n; t0 += TILE, buf ^= 1) {
        next.store(rows[buf]);
        lds_barrier();
        if (t0 + TILE < n) fetch_rows(t0 + TILE);
        const float* bl = rows[buf] + q * NS;
        const float* cl = bl + TILE * N;
        const int left = n - t0 - q;
        at_tile(t0 + TILE);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            if (g % (CH / 4) == 0) {
                if (t0 + 4 * g >= n) break;
                const int chunk = (t0 + 4 * g) / CH;
                const float s = quad_sum(sum);
                if (real && chunk > 0) {
                    st_states<NS>(start + chunk * states, h);
                    if (q == 0) before[(int64_t)chunk * a.D] = s;
                }
            }
            const float xv = value<E>(nx[g]), raw = value<E>(nt[g]) + bias, dyv = BACK ? value<E>(nd[g]) : 0.0f, zv = BACK ? value<E>(nz[g]) : 0.0f;
            fetch(g);
            float d = SOFTPLUS ? softplus(raw) : raw;
            d = 4 * g < left ? d : 0.0f;   // a step of nothing behind the last token: x and dy are zero there
            const float u = d * xv, v = dyv * (gated ? zv * sigmoid(zv) : 1.0f);
            sum += d;
            each_of_quad([&](auto J) {
                constexpr int j = decltype(J)::value;
                float bv[NS], cv[NS], e[NS];
                ld_states<NS>(bl + (4 * g + j) * N, bv);
                if (BACK) ld_states<NS>(cl + (4 * g + j) * N, cv);
                quad_times<j, NS>(d, A2, e);
                quad_times<j, NS>(u, bv, bv);
                if (BACK) quad_times<j, NS>(v, cv, cv);
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    e[i] = __builtin_amdgcn_exp2f(e[i]);
                    h[i] = __builtin_fmaf(e[i], h[i], bv[i]);
                    if (BACK) {
                        P[i] *= e[i];
                        m[i] = __builtin_fmaf(P[i], cv[i], m[i]);
                    }
                }
            });
            // a group at a time: drawn together, a tile's operands do not fit the registers and its exchanges lie too far from
            // the products that take them
#pragma unroll
            for (int i = 0; i < NS; ++i) asm volatile("" : : "v"(h[i]), "v"(m[i]));
        }
    }
    sum = quad_sum(sum);
    if (BACK && real && pl.pieces > 1) {   // what the other pieces of the sequence ask for
        const int64_t map = pl.map0 + pl.k;
        if (pl.k < pl.pieces - 1) st_states<NS>(a.local + map * states + at_state, h);
        if (pl.k > 0) {
            st_states<NS>(a.grad + (map - 1) * states + at_state, m);
            if (q == 0) a.sums[(map - 1) * a.D + ch] = sum;
        }
    }
}

// ---------------------------------------------------------------- sums over a wavefront's channels
typedef unsigned u32x2 __attribute__((__vector_size__(8)));

__device__ __forceinline__ float sum_of(u32x2 r) {
    const unsigned a = r[0], b = r[1];   // a bit cast of r[1] itself takes r[0]
    return __builtin_bit_cast(float, a) + __builtin_bit_cast(float, b);
}

// The sum over the 16 channels (lane bits 5 to 2) of a value a token, each lane left with token
// (lane >> 2)'s of its quad place.  Every step halves the values: a lane keeps one of a pair and sends
// the other.
__device__ __forceinline__ float channel_sums(float (&v)[CH], int lane) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
        v[i] = sum_of(__builtin_amdgcn_permlane32_swap(__builtin_bit_cast(unsigned, v[i]), __builtin_bit_cast(unsigned, v[i + 8]), false, false));
#pragma unroll
    for (int i = 0; i < 4; ++i)
        v[i] = sum_of(__builtin_amdgcn_permlane16_swap(__builtin_bit_cast(unsigned, v[i]), __builtin_bit_cast(unsigned, v[i + 4]), false, false));
    const bool b3 = lane & 8, b2 = lane & 4;
#pragma unroll
    for (int i = 0; i < 2; ++i)   // row_ror:8, the lane with bit 3 turned
        v[i] = (b3 ? v[i + 2] : v[i]) + quad_perm<0x128>(b3 ? v[i] : v[i + 2]);
    // bit 2 turned: row_shr:4 for all, then row_shl:4 over it in the banks of four lanes where the bit is 0
    const int send = __builtin_bit_cast(int, b2 ? v[0] : v[1]);
    const int down = __builtin_amdgcn_update_dpp(0, send, 0x114, 0xf, 0xf, false);
    return (b2 ? v[1] : v[0]) + __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(down, send, 0x104, 0xf, 0x5, false));
}

// Token T of 16's value, which lane T % 4 of the quad holds in v[T / 4].
template <int T>
__device__ __forceinline__ float token(const float* v) { return quad_lane<T % 4>(v[T / 4]); }

// Which channel and states thread `me` of the workgroup of channels blk has.
struct Mine {
    int q, ch;
    bool real;
    int64_t at_state;
};
template <int NS>
__device__ __forceinline__ Mine mine_of(const BwdArgs& a, int blk, int me) {
    const int Dg = a.D / a.G, per = (Dg + BLOCK_CH - 1) / BLOCK_CH, in_group = blk % per * BLOCK_CH + (me >> 2);
    Mine m;
    m.q = me & 3;
    m.real = in_group < Dg;
    m.ch = blk / per * Dg + (m.real ? in_group : Dg - 1);
    m.at_state = (int64_t)m.ch * 4 * NS + m.q * NS;
    return m;
}

// MANY: a workgroup has several slots.  Where it has one, as in every call but one of very many short sequences, the loop would cost:
// 8 x 4,096 tokens by 2,048 channels 1,232 us without, 1,252 with it; 2,048 x 16 tokens by 1,024 channels 607 and 660.
template <typename E, int NS, bool MANY>
__global__ void __launch_bounds__(BLOCK) __attribute__((amdgpu_waves_per_eu(NS <= 4 && sizeof(E) == 2 ? 3 : NS <= 8 ? 2 : 1))) scan_bwd_grad(BwdArgs a) {
    constexpr int N = 4 * NS, GROUPS = CH / 4, WAVES = BLOCK / 64;
    __shared__ float bc[2][N * BPAD];
    __shared__ float part[WAVES][CH][2][N];
    // A lane's states, one word each, in turn in registers: 16 tokens' work on one fill those.
    __shared__ float sA[NS][BLOCK], smu[NS][BLOCK], sdA[NS][BLOCK], sh0[NS][BLOCK], sh[NS][BLOCK];
    // what the outputs need of a lane's own tokens beside, while the registers are the states'
    __shared__ float aside[3][GROUPS][BLOCK];
    __shared__ float chan[4][BLOCK];   // a channel's bias and skip, and its parts of their gradients
    const int nblk = blocks_of(a.D, a.G);
    const int blk = (int)(blockIdx.x % (unsigned)nblk);
    const int64_t part0 = blockIdx.x / (unsigned)nblk;
    const int grp = blk / (nblk / a.G);
    const int64_t states = (int64_t)a.D * N, ld = (int64_t)a.G * N;
    const bool gated = a.z != nullptr;
    int me = threadIdx.x;
    {
        const Mine m = mine_of<NS>(a, blk, me);
        float A2[NS];
        ld_states<NS>(a.A + m.at_state, A2);
#pragma unroll
        for (int i = 0; i < NS; ++i) sA[i][me] = A2[i] * LOG2E, sdA[i][me] = 0.0f;
        chan[0][me] = a.bias ? a.bias[m.ch] : 0.0f;
        chan[1][me] = a.skip ? a.skip[m.ch] : 0.0f;
        chan[2][me] = chan[3][me] = 0.0f;
    }
    int64_t slot = part0;
    do {
        // hides the thread's number: what follows from it would stay in registers from before the loop to behind it, and in bf16
        // up to 16 states there are none to spare
        asm volatile("" : "+v"(me));
        const Mine m = mine_of<NS>(a, blk, me);
        const int q = m.q, ch = m.ch;
        const bool real = m.real;
        const int64_t at_state = m.at_state;
        const int wave = uniform(me >> 6), lane = me & 63;
        const uint32_t own = real ? ((uint32_t)q * (uint32_t)a.D + ch) * (uint32_t)sizeof(E) : NOWHERE, four = 4 * (uint32_t)a.D * (uint32_t)sizeof(E);
        Place pl;
        if (!place_of(a.seqs, slot, pl)) continue;
        const int t_first = pl.k * a.seqs.piece;
        const int n = uniform(pl.len - t_first < a.seqs.piece ? pl.len - t_first : a.seqs.piece);
        const int64_t row = uniform64(pl.row0 + t_first);
        const int64_t chunk0 = first_chunk(a.seqs, pl) + t_first / CH;
        {
            float A2[NS], mu[NS], h0[NS];
#pragma unroll
            for (int i = 0; i < NS; ++i) A2[i] = sA[i][me], mu[i] = h0[i] = 0.0f;
            if (a.dS_T) ld_states<NS>(a.dS_T + (int64_t)pl.seq * states + at_state, mu);
            // what the pieces behind make of it, and the state that the pieces before leave
            const int64_t last = pl.map0 + pl.pieces - 2;
            along_pieces<NS>(mu, A2, a.grad + last * states + at_state, a.sums + last * a.D + ch, -1, pl.pieces - 1 - pl.k, states, a.D);
            if (pl.k > 0) {
                ld_states<NS>(a.local + pl.map0 * states + at_state, h0);
                along_pieces<NS>(h0, A2, a.local + (pl.map0 + 1) * states + at_state, a.sums + pl.map0 * a.D + ch, 1, pl.k - 1, states, a.D);
            }
#pragma unroll
            for (int i = 0; i < NS; ++i) smu[i][me] = mu[i], sh0[i][me] = h0[i];
        }

        // a chunk's operands are asked for one chunk ahead
        Rows<E, N, CH> next;
        uint32_t nx[GROUPS], nt[GROUPS], nz[GROUPS], nd[GROUPS];
        float nh[NS], ns = 0.0f;
        auto fetch = [&](int chunk) {
            const int tokens = n - CH * chunk < CH ? n - CH * chunk : CH;
            const int64_t from = row + CH * chunk, at = from * ld + grp * N;
            next.fetch((const E*)a.b + at, (const E*)a.c + at, ld, tokens);
            const Rsrc rx = rows_rsrc<E>(a.x, from, a.D, tokens), rt = rows_rsrc<E>(a.dt, from, a.D, tokens),
                       rd = rows_rsrc<E>(a.dy, from, a.D, tokens);
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                nx[g] = ld_one<E>(rx, own + g * four);
                nt[g] = ld_one<E>(rt, own + g * four);
                nd[g] = ld_one<E>(rd, own + g * four);
            }
            if (gated) {
                const Rsrc rz = rows_rsrc<E>(a.z, from, a.D, tokens);
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) nz[g] = ld_one<E>(rz, own + g * four);
            }
            const float* from_S0 = a.S0 + (int64_t)pl.seq * states;
            const int64_t at_chunk = chunk > 0 ? chunk0 + chunk : 0;
            ld_states<NS>((chunk == 0 && pl.k == 0 && a.S0 ? from_S0 : a.start + at_chunk * states) + (uint32_t)at_state, nh);
            ns = a.before[at_chunk * a.D + (uint32_t)ch];
        };
        const int chunks = (n + CH - 1) / CH;
        if (chunks > 0) fetch(chunks - 1);
        for (int k = chunks - 1; k >= 0; --k) {
            float dv[GROUPS], uv[GROUPS], vy[GROUPS];
            next.each([&](bool of_c, int t, int n0, f32x4 x) {
#pragma unroll
                for (int j = 0; j < 4; ++j) bc[of_c ? 1 : 0][(n0 + j) * BPAD + t] = x[j];
            });
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                dv[g] = value<E>(nt[g]) + chan[0][me];
                uv[g] = aside[2][g][me] = value<E>(nx[g]);
                vy[g] = value<E>(nd[g]);
            }
            if (a.softplus) {
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    float slope;
                    dv[g] = softplus(dv[g], slope);
                    aside[0][g][me] = slope;
                }
            } else {
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) aside[0][g][me] = 1.0f;
            }
            if (gated)
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) {
                    const float zv = value<E>(nz[g]), sg = sigmoid(zv);
                    aside[1][g][me] = vy[g] * (sg * (1.0f + zv * (1.0f - sg)));
                    vy[g] *= zv * sg;
                }
            // a step of nothing behind the last token, where x and dy are zero, and of lanes without a channel, which read zeros: their
            // bias alone could make states of any size, and zero times infinity would reach the sums over channels
            const int left = real ? n - CH * k - q : 0;
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                if (4 * g >= left) dv[g] = aside[0][g][me] = 0.0f;
                uv[g] *= dv[g];
            }
#pragma unroll
            for (int i = 0; i < NS; ++i)
                sh[i][me] = pl.k > 0 ? __builtin_fmaf(__builtin_amdgcn_exp2f(ns * sA[i][me]), sh0[i][me], nh[i]) : nh[i];
            lds_barrier();
            if (k > 0) fetch(k - 1);

            float s1[CH], s2[CH], sy[CH];
#pragma unroll
            for (int t = 0; t < CH; ++t) s1[t] = s2[t] = sy[t] = 0.0f;
#pragma unroll 1
            for (int i = 0; i < NS; ++i) {
                // Operands are handed round the quad as modifiers of multiplications, which have to follow one another closely for
                // that; the empty statements keep the compiler from drawing the tokens together.
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) asm volatile("" : "+v"(dv[g]), "+v"(uv[g]), "+v"(vy[g]));
                float e[CH], hp[CH], v[CH];
                const float *bi = bc[0] + (q * NS + i) * BPAD, *ci = bc[1] + (q * NS + i) * BPAD;
                float h = sh[i][me];
                const float A2i = sA[i][me], Ai = A2i * (1.0f / LOG2E);
                each_of_quad([&](auto Gr) {
                    constexpr int t0 = 4 * decltype(Gr)::value;
                    float bv[4], cv[4];
                    ld_states<4>(bi + t0, bv);
                    ld_states<4>(ci + t0, cv);
                    each_of_quad([&](auto J) {
                        constexpr int j = decltype(J)::value, t = t0 + j;
                        hp[t] = h;
                        e[t] = __builtin_amdgcn_exp2f(token<t>(dv) * A2i);
                        h = __builtin_fmaf(e[t], h, token<t>(uv) * bv[j]);
                        sy[t] = __builtin_fmaf(cv[j], h, sy[t]);
                        v[t] = token<t>(vy) * h;   // zero of lanes without a channel: no dy, and the last channel's state kept
                    });
                    asm volatile("" : : "v"(v[t0]), "v"(v[t0 + 1]), "v"(v[t0 + 2]), "v"(v[t0 + 3]), "v"(sy[t0 + 3]) : "memory");
                });
                const int t_mine = lane >> 2;
                part[wave][t_mine][1][q * NS + i] = channel_sums(v, lane);
#pragma unroll
                for (int g = 0; g < GROUPS; ++g) asm volatile("" : "+v"(dv[g]), "+v"(uv[g]), "+v"(vy[g]) : : "memory");
                float m = smu[i][me], s = 0.0f;
                each_of_quad([&](auto Gr) {
                    constexpr int t0 = CH - 4 - 4 * decltype(Gr)::value;
                    float bv[4], cv[4];
                    ld_states<4>(bi + t0, bv);
                    ld_states<4>(ci + t0, cv);
                    float w[4];
                    each_of_quad([&](auto J) {
                        constexpr int j = 3 - decltype(J)::value, t = t0 + j;
                        const float lam = token<t>(vy) * cv[j] + m;
                        v[t] = token<t>(uv) * lam;
                        m = e[t] * lam;
                        w[j] = m * hp[t];   // lam a_t h_t-1
                        s1[t] = __builtin_fmaf(lam, bv[j], s1[t]);
                        s2[t] = __builtin_fmaf(Ai, w[j], s2[t]);
                    });
                    quad_fma(s, dv[t0 / 4], w);
                    asm volatile("" : : "v"(v[t0]), "v"(v[t0 + 1]), "v"(v[t0 + 2]), "v"(v[t0 + 3]), "v"(s) : "memory");
                });
                smu[i][me] = m;
                sdA[i][me] += s;
                part[wave][t_mine][0][q * NS + i] = channel_sums(v, lane);
            }
            const int64_t from = row + CH * k;
            const int tokens = n - CH * k < CH ? n - CH * k : CH;
            const Rsrc wx = rows_rsrc<E>(a.dx, from, a.D, tokens), wt = rows_rsrc<E>(a.ddt, from, a.D, tokens);
            const float skip = chan[1][me];
            float dskip = chan[3][me], dbias = chan[2][me];
#pragma unroll
            for (int g = 0; g < GROUPS; ++g) {
                const float lb = quad_sums(s1 + 4 * g, q), lw = quad_sums(s2 + 4 * g, q);
                const float xv = aside[2][g][me], ddt = __builtin_fmaf(xv, lb, lw) * aside[0][g][me];
                st_one<E>(wx, own + g * four, __builtin_fmaf(skip, vy[g], dv[g] * lb));
                st_one<E>(wt, own + g * four, ddt);
                dskip = __builtin_fmaf(vy[g], xv, dskip);
                dbias += ddt;   // zero where there is no token
            }
            if (gated) {
                const Rsrc wz = rows_rsrc<E>(a.dz, from, a.D, tokens);
#pragma unroll
                for (int g = 0; g < GROUPS; ++g)
                    st_one<E>(wz, own + g * four, aside[1][g][me] * __builtin_fmaf(skip, aside[2][g][me], quad_sums(sy + 4 * g, q)));
            }
            chan[3][me] = dskip;
            chan[2][me] = dbias;
            lds_barrier();
            // the workgroup's part of db and dc
            float* to = a.pbc + ((int64_t)blk * a.rows + row + CH * k) * 2 * N;
            for (int i = me; i < CH * 2 * N; i += BLOCK) {
                if (CH * k + i / (2 * N) >= n) break;
                float s = 0.0f;
#pragma unroll
                for (int w = 0; w < WAVES; ++w) s += (&part[w][0][0][0])[i];
                to[i] = s;
            }
        }
        if (pl.k == 0 && a.dS0 && real) {
            float mu[NS];
#pragma unroll
            for (int i = 0; i < NS; ++i) mu[i] = smu[i][me];
            st_states<NS>(a.dS0 + (int64_t)pl.seq * states + at_state, mu);
        }
    } while (MANY && (slot += a.parts) < a.slots);
    asm volatile("" : "+v"(me));
    const Mine m = mine_of<NS>(a, blk, me);
    const float dskip = quad_sum(chan[3][me]), dbias = quad_sum(chan[2][me]);
    float dA[NS];
#pragma unroll
    for (int i = 0; i < NS; ++i) dA[i] = sdA[i][me];
    if (m.real) {
        st_states<NS>(a.pA + part0 * states + m.at_state, dA);
        if (m.q == 0) {
            a.pskip[part0 * a.D + m.ch] = dskip;
            a.pbias[part0 * a.D + m.ch] = dbias;
        }
    }
}

// What several workgroups have parts of: the first workgroups sum those of dA, dskip and ddt_bias, the others those
// of db and dc, and the last clear all gradients' rows of no sequence.
template <typename E>
__global__ void __launch_bounds__(1024)
scan_bwd_sums(PartSums params, int64_t nparams, Seqs s, int64_t rows, int G, int N, int per, const float* __restrict__ part,
              E* __restrict__ db, E* __restrict__ dc, E* dx, E* ddt, E* dz, int D) {
    if ((int64_t)blockIdx.x < nparams) {
        part_sums(params, blockIdx.x);
        return;
    }
    const int64_t blk = blockIdx.x - nparams, nblk = gridDim.x - nparams - (s.cu ? REST_BLOCKS : 0);
    if (blk >= nblk) {
        E* const rest[] = {dx, ddt, dz};
        for (E* p : rest)
            if (p) clear_rest(s, p, D, blk - nblk);
        clear_rest(s, db, G * N, blk - nblk);
        clear_rest(s, dc, G * N, blk - nblk);
        return;
    }
    const int64_t each = 2 * (int64_t)G * N, total = rows * each;
    int64_t lo = 0, hi = rows;
    if (s.cu) {
        lo = held(s.cu[0], 0, s.T);
        hi = held(s.cu[s.nseq], 0, s.T);
    }
    for (int64_t i = blk * 1024 + threadIdx.x; i < total; i += nblk * 1024) {
        const int64_t row = i / each;
        const int r = (int)(i - row * each), g = r / (2 * N), j = r - g * 2 * N;
        if (row < lo || row >= hi) continue;
        const float* p = part + ((int64_t)g * per * rows + row) * 2 * N + j;
        const int64_t ld = rows * 2 * N;
        float u[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        int k = 0;
        for (; k + 8 <= per; k += 8)   // eight loads in flight
#pragma unroll
            for (int e = 0; e < 8; ++e) u[e] += p[(k + e) * ld];
        for (; k < per; ++k) u[0] += p[k * ld];
        const float t = ((u[0] + u[1]) + (u[2] + u[3])) + ((u[4] + u[5]) + (u[6] + u[7]));
        (j < N ? db : dc)[(row * G + g) * N + (j < N ? j : j - N)] = from_f<E>(t);
    }
}

// Tokens a piece: cut_piece, always by workgroups, since the maps run in any case (8 x 4,096 tokens by
// 2,048 channels: 256 workgroups 2,857 us, 512 1,499, 1,024 1,351, 2,048 1,272, 4,096 1,261).
struct BwdPlan {
    int piece;
    int64_t rows, slots, parts;
    int64_t local, grad, sums, start, before, pA, pskip, pbias, pbc, floats;
};
static BwdPlan plan_of(int nseq, int T, int D, int N, int G, bool packed) {
    BwdPlan p;
    p.piece = cut_piece(nseq, T, D, G, packed);
    p.rows = packed ? T : (int64_t)nseq * T;
    p.slots = slots_of(nseq, T, p.piece, packed);
    const int64_t maps = maps_of(nseq, T, p.piece, packed), chunks = maps_of(nseq, T, CH, packed);
    // Of dA, dskip and ddt_bias a workgroup has the part of one slot, unless there are more than four times the slots that the rows
    // make pieces (and more than fill the device): many short sequences, whose parts would be most of the workspace.
    const int64_t fill = 2048 / blocks_of(D, G), four = 4 * (p.rows / p.piece), most = fill > four ? fill : four;
    p.parts = p.slots < most ? p.slots : most > 1 ? most : 1;
    int64_t at = 0;
    auto take = [&](int64_t n) {
        const int64_t r = at;
        at += (n + 3) / 4 * 4;
        return r;
    };
    const int64_t states = (int64_t)D * N;
    p.local = take(maps * states);
    p.grad = take(maps * states);
    p.pA = take(p.parts * states);
    p.start = take((1 + chunks) * states);
    p.pbc = take((int64_t)blocks_of(D, G) * p.rows * 2 * N);
    p.sums = take(maps * D);
    p.pskip = take(p.parts * D);
    p.pbias = take(p.parts * D);
    p.before = take((1 + chunks) * D);
    p.floats = at;
    return p;
}

template <typename E, int NS>
static hipError_t bwd_t(const BwdArgs& a, const BwdPlan& p, void* db, void* dc, float* dA, float* dskip, float* dbias, hipStream_t stream) {
    constexpr int N = 4 * NS;
    const int blocks = blocks_of(a.D, a.G);
    const unsigned grid = (unsigned)(p.slots * blocks);
    auto map = p.piece < a.seqs.T ? (a.softplus ? scan_bwd_map<E, NS, true, true> : scan_bwd_map<E, NS, false, true>)
                                  : (a.softplus ? scan_bwd_map<E, NS, true, false> : scan_bwd_map<E, NS, false, false>);
    hipLaunchKernelGGL(map, dim3(grid), dim3(BLOCK), 0, stream, a);
    auto grad = p.parts < p.slots ? scan_bwd_grad<E, NS, true> : scan_bwd_grad<E, NS, false>;
    hipLaunchKernelGGL(grad, dim3((unsigned)(p.parts * blocks)), dim3(BLOCK), 0, stream, a);
    const PartSums params{{a.pA, a.pskip, a.pbias}, {dA, dskip, dbias}, {(int64_t)a.D * N, a.D, a.D}, p.parts};
    const int64_t nparams = part_sums_blocks(params), want = (p.rows * 2 * a.G * N + 1023) / 1024;
    hipLaunchKernelGGL(scan_bwd_sums<E>, dim3((unsigned)(nparams + (want < 2048 ? want : 2048) + (a.seqs.cu ? REST_BLOCKS : 0))), dim3(1024), 0, stream, params, nparams, a.seqs,
                       p.rows, a.G, N, blocks / a.G, a.pbc, (E*)db, (E*)dc, (E*)a.dx, (E*)a.ddt, (E*)a.dz, a.D);
    return hipGetLastError();
}

}  // namespace scan

int64_t scan_bwd_workgroups(int nseq, int T, int D, int G, bool packed) {
    return scan::slots_of(nseq, T, scan::cut_piece(nseq, T, D, G, packed), packed) * scan::blocks_of(D, G);
}

size_t scan_bwd_workspace_bytes(int nseq, int T, int D, int N, int G, bool packed) {
    return (size_t)scan::plan_of(nseq, T, D, N, G, packed).floats * sizeof(float);
}

hipError_t launch_scan_bwd(const ScanCall& c, const void* dy, const float* dS_T, void* dx, void* ddt, float* dA, void* db, void* dc,
                           float* dskip, void* dz, float* dbias, float* dS0, void* workspace, hipStream_t stream) {
    const scan::BwdPlan p = scan::plan_of(c.nseq, c.T, c.D, c.N, c.G, c.cu != nullptr);
    float* w = (float*)workspace;
    const scan::BwdArgs a{{c.nseq, c.T, p.piece, c.cu}, c.D, c.G, c.softplus, c.x, c.dt, c.b, c.c, c.z, dy, c.A, c.skip, c.bias, c.S0, dS_T,
                          dx, ddt, dz, dS0, w + p.local, w + p.grad, w + p.sums, w + p.start, w + p.before, w + p.pA, w + p.pskip,
                          w + p.pbias, w + p.pbc, p.rows, p.slots, p.parts};
#define KDA_SB(N)                                                                                          \
    return c.f32 ? scan::bwd_t<float, N / 4>(a, p, db, dc, dA, dskip, dbias, stream)                       \
                 : scan::bwd_t<bf16, N / 4>(a, p, db, dc, dA, dskip, dbias, stream)
    switch (c.N) {
        case 8: KDA_SB(8);
        case 16: KDA_SB(16);
        case 32: KDA_SB(32);
        case 64: KDA_SB(64);
    }
#undef KDA_SB
    return hipErrorInvalidValue;
}

}  // namespace kda
