// kda_scan_fwd.hip -- the selective scan over whole sequences (kda_scan.hpp has the formulas
// and how lanes and pieces are laid out).
//
// What bounds it: vector instructions.  A token, channel and state takes two products, an exponential (two
// instructions' time), two fused products for y and the state: six of them forwards, five in a map, against
// half a byte of HBM in the walk and a quarter in a map (16 states, bf16).  So operands that a quad shares are handed round inside the products (kda_scan.hpp), b and c
// are converted once a workgroup, a lane's own tokens are asked for a tile ahead through buffer resources that
// take no vector address, and each as soon as its predecessor is used, which keeps a wavefront below 100 registers (16
// states: five wavefronts a SIMD).  Counters: 90% of the vector issue slots taken, 65% of those the six and five.
// Measured, bf16, 16 states, gate, skip and softplus: 65,536 tokens by 2,048 channels 886 us (43% in the maps; 1.2
// TB/s, 2.4e12 states a second), 32 x 4,096 by 4,096 uncut 1.97 ms (4.4e12); ten packed prompts of 1 to 8,192 tokens 237 us.
// Before: addresses in vector registers, operands exchanged by instructions of their own, a whole tile's tokens held
// while the next ones came: 1,376, 413.
//
// Two launches: the maps of every piece but a sequence's last, and the walk that forms y, each
// piece first putting its start state together from the maps before it (a chain of one
// exponential a piece, at most 256).  Where nothing is cut only the walk runs.
#include "kda_scan.hpp"

namespace kda {
namespace scan {

struct FwdArgs {
    Seqs seqs;
    int D, G;
    const void *x, *dt, *b, *c, *z;
    const float *A, *skip, *bias, *S0;
    void* y;
    unsigned walks;   // workgroups with a piece; those behind them clear y's rows of no sequence
    float *S_T, *local, *keep, *sums;   // maps: end state from nothing [map][D][N], sum of delta [map][D]; S0 of cut sequences [..][D][N]
};

// Places for the S0 of cut sequences: one a sequence, or by its first row, whichever is fewer (kept_of).
__device__ __forceinline__ bool kept_by_row(const Seqs& s) { return s.cu && s.nseq > s.T / s.piece; }

template <typename E, int NS, bool SOFTPLUS, bool MAP, bool GATED>
__global__ void __launch_bounds__(BLOCK) scan_walk(FwdArgs a) {
    constexpr int N = 4 * NS, GROUPS = TILE / 4;
    __shared__ float rows[2][2 * TILE * N];
    const int per = (a.D / a.G + BLOCK_CH - 1) / BLOCK_CH, nblk = a.G * per;
    const int blk = (int)(blockIdx.x % (unsigned)nblk);
    const int64_t slot = blockIdx.x / (unsigned)nblk;
    if (!MAP && blockIdx.x >= a.walks) {
        clear_rest(a.seqs, (E*)a.y, a.D, blockIdx.x - a.walks);
        return;
    }
    Place pl;
    if (!place_of(a.seqs, slot, pl)) return;
    if (MAP && pl.k == pl.pieces - 1) return;
    const int grp = blk / per, Dg = a.D / a.G;
    const int lane = threadIdx.x & 63, q = lane & 3;
    const int in_group = (blk % per) * BLOCK_CH + (int)(threadIdx.x >> 6) * WAVE_CH + (lane >> 2);
    const bool real = in_group < Dg;
    const int ch = grp * Dg + (real ? in_group : Dg - 1);   // lanes without a channel repeat the last one's states and store nothing
    const int t_first = pl.k * a.seqs.piece;
    const int n = uniform(pl.len - t_first < a.seqs.piece ? pl.len - t_first : a.seqs.piece);
    const int64_t row = uniform64(pl.row0 + t_first);
    const int64_t ld = (int64_t)a.G * N;
    uint32_t own[GROUPS];   // a lane's own tokens of a tile: every fourth
#pragma unroll
    for (int g = 0; g < GROUPS; ++g) own[g] = real ? ((uint32_t)(4 * g + q) * (uint32_t)a.D + ch) * (uint32_t)sizeof(E) : NOWHERE;
    const float bias = a.bias ? a.bias[ch] : 0.0f, skip = a.skip ? a.skip[ch] : 0.0f;
    const int64_t at_state = (int64_t)ch * N + q * NS, states = (int64_t)a.D * N;

    Rows<E, N, TILE> next;
    uint32_t nx[GROUPS], nt[GROUPS], nz[GROUPS];
    auto tokens_at = [&](int t0) { return uniform(n - t0 < 0 ? 0 : n - t0 < TILE ? n - t0 : TILE); };   // a median of three is a vector instruction
    auto fetch_rows = [&](int t0) {
        const int64_t at = (row + t0) * ld + grp * N;
        next.fetch((const E*)a.b + at, (const E*)a.c + at, ld, tokens_at(t0));
    };
    if (n > 0) {
        fetch_rows(0);
        const Rsrc rx = rows_rsrc<E>(a.x, row, a.D, tokens_at(0)), rt = rows_rsrc<E>(a.dt, row, a.D, tokens_at(0));
        Rsrc rz;
        if (GATED) rz = rows_rsrc<E>(a.z, row, a.D, tokens_at(0));
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            nx[g] = ld_one<E>(rx, own[g]);
            nt[g] = ld_one<E>(rt, own[g]);
            if (GATED) nz[g] = ld_one<E>(rz, own[g]);
        }
    }

    float A2[NS], h[NS];
    ld_states<NS>(a.A + at_state, A2);
#pragma unroll
    for (int i = 0; i < NS; ++i) A2[i] *= LOG2E, h[i] = 0.0f;
    float* local = a.local + at_state;
    if (pl.k == 0) {
        // S_T may overwrite S0 during the walk, so the maps keep a copy for the first piece
        float* kept = a.keep + (kept_by_row(a.seqs) ? pl.map0 : pl.seq) * states + at_state;
        const float* from = !MAP && pl.pieces > 1 ? kept : a.S0 + (int64_t)pl.seq * states + at_state;
        if (a.S0) ld_states<NS>(from, h);
        if (MAP && a.S0 && real) st_states<NS>(kept, h);
    } else if (!MAP) {
        ld_states<NS>(local + pl.map0 * states, h);   // the first piece's map starts from S0
        along_pieces<NS>(h, A2, local + (pl.map0 + 1) * states, a.sums + (pl.map0 + 1) * a.D + ch, 1, pl.k - 1, states, a.D);
    }
    float sum = 0.0f;
    for (int t0 = 0, buf = 0; t0 < n; t0 += TILE, buf ^= 1) {
        next.store(rows[buf]);
        lds_barrier();   // one a tile: a buffer is written again only after the barrier of the other's tile
        if (t0 + TILE < n) fetch_rows(t0 + TILE);
        const float* bl = rows[buf] + q * NS;
        const float* cl = bl + TILE * N;
        // a lane's own tokens are asked for a tile ahead, each as soon as the one in its place is used
        const int ahead = tokens_at(t0 + TILE), left = n - t0 - q;
        const Rsrc rx = rows_rsrc<E>(a.x, row + t0 + TILE, a.D, ahead), rt = rows_rsrc<E>(a.dt, row + t0 + TILE, a.D, ahead);
        Rsrc rz, ry;
        if (GATED) rz = rows_rsrc<E>(a.z, row + t0 + TILE, a.D, ahead);
        if (!MAP) ry = rows_rsrc<E>(a.y, row + t0, a.D, tokens_at(t0));
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            if (g % 4 == 0 && t0 + 4 * g >= n) break;
            const float xv = value<E>(nx[g]), raw = value<E>(nt[g]) + bias, zv = GATED ? value<E>(nz[g]) : 0.0f;
            nx[g] = ld_one<E>(rx, own[g]);
            nt[g] = ld_one<E>(rt, own[g]);
            if (GATED) nz[g] = ld_one<E>(rz, own[g]);
            float d = SOFTPLUS ? softplus(raw) : raw;
            d = 4 * g < left ? d : 0.0f;   // a step of nothing behind the last token: x is zero there
            const float u = d * xv, gate = GATED ? zv * gate_sigmoid<E>(zv) : 1.0f;
            if (MAP) sum += d;
            float yj[4];
            each_of_quad([&](auto J) {
                constexpr int j = decltype(J)::value;
                float bv[NS], cv[NS], e[NS];
                ld_states<NS>(bl + (4 * g + j) * N, bv);
                if (!MAP) ld_states<NS>(cl + (4 * g + j) * N, cv);
                quad_times<j, NS>(d, A2, e);
                quad_times<j, NS>(u, bv, bv);
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(e[i]), h[i], bv[i]);
                    if (!MAP) s = i ? __builtin_fmaf(cv[i], h[i], s) : cv[i] * h[i];
                }
                yj[j] = s;
            });
            if (MAP) {
                // a group at a time, as the walk's stores have it: drawn together, a tile's exchanges lie too far from the
                // products that take them
#pragma unroll
                for (int i = 0; i < NS; ++i) asm volatile("" : : "v"(h[i]));
            } else {
                const float yv = __builtin_fmaf(skip, xv, quad_sums(yj, q));
                st_one<E>(ry, own[g], GATED ? yv * gate : yv);
            }
        }
    }
    if (MAP) {
        sum = quad_sum(sum);
        if (real) {
            st_states<NS>(local + (pl.map0 + pl.k) * states, h);
            if (q == 0) a.sums[(pl.map0 + pl.k) * a.D + ch] = sum;
        }
    } else if (a.S_T && pl.k == pl.pieces - 1 && real) {
        st_states<NS>(a.S_T + (int64_t)pl.seq * states + at_state, h);
    }
}

// Tokens a piece.  A cut call forms every state twice, but 256 workgroups are one wavefront a SIMD, whose
// instructions wait for each other.  Measured, sequences of 4,096 tokens by 2,048 channels of 16 states, when the call below took 896: at 256
// workgroups whole 544 us, cut 514; at 512 whole 697, cut 907 (now 600 and 829).  A packed call's lengths are not known here, so it is
// cut however many sequences it has.  Pieces are as many as give 2,048 workgroups, eight a
// compute unit (65,536 tokens, in the course of the work: 512 workgroups 1,259 us, 1,024 951, 2,048 896, 4,096 916), of 64 tokens at the least
// (2 x 1,000 tokens by 256 channels of 32 states: 32 tokens 29.7 us, 64 30.9, 128 43.8; the backward pass of four
// sequences by 512 channels, which has the same rule: 90.7, 81.8, 107.7).
static int fwd_piece(int nseq, int T, int D, int G, bool packed) {
    if (!packed && (int64_t)nseq * blocks_of(D, G) >= 512) return (int)(((int64_t)T + TILE - 1) / TILE * TILE);
    return cut_piece(nseq, T, D, G, packed);
}

static int64_t kept_of(int nseq, int T, int piece, bool packed) { return packed && nseq > T / piece ? T / piece : nseq; }

template <typename E, int NS, bool SOFTPLUS>
static hipError_t fwd_t(const FwdArgs& a, bool cut, bool zero_rest, hipStream_t stream) {
    const unsigned grid = a.walks + (zero_rest ? REST_BLOCKS : 0);
    if (cut) hipLaunchKernelGGL((scan_walk<E, NS, SOFTPLUS, true, false>), dim3(a.walks), dim3(BLOCK), 0, stream, a);
    if (a.z) hipLaunchKernelGGL((scan_walk<E, NS, SOFTPLUS, false, true>), dim3(grid), dim3(BLOCK), 0, stream, a);
    else hipLaunchKernelGGL((scan_walk<E, NS, SOFTPLUS, false, false>), dim3(grid), dim3(BLOCK), 0, stream, a);
    return hipGetLastError();
}

}  // namespace scan

int64_t scan_fwd_workgroups(int nseq, int T, int D, int G, bool packed) {
    return scan::slots_of(nseq, T, scan::fwd_piece(nseq, T, D, G, packed), packed) * scan::blocks_of(D, G) + (packed ? scan::REST_BLOCKS : 0);
}

size_t scan_fwd_workspace_bytes(int nseq, int T, int D, int N, int G, bool packed) {
    const int piece = scan::fwd_piece(nseq, T, D, G, packed);
    if (piece >= T) return 0;
    return (size_t)(scan::maps_of(nseq, T, piece, packed) + scan::kept_of(nseq, T, piece, packed)) * D * (N + 1) * sizeof(float);
}

hipError_t launch_scan_fwd(const ScanCall& c, bool zero_rest, void* y, float* S_T, void* workspace, hipStream_t stream) {
    const bool packed = c.cu != nullptr;
    const int piece = scan::fwd_piece(c.nseq, c.T, c.D, c.G, packed);
    const int64_t slots = scan::slots_of(c.nseq, c.T, piece, packed);
    const int64_t maps = scan::maps_of(c.nseq, c.T, piece, packed), kept = scan::kept_of(c.nseq, c.T, piece, packed), states = (int64_t)c.D * c.N;
    float* local = (float*)workspace;
    const scan::FwdArgs a{{c.nseq, c.T, piece, c.cu}, c.D, c.G, c.x, c.dt, c.b, c.c, c.z, c.A, c.skip, c.bias, c.S0,
                          y, (unsigned)(slots * scan::blocks_of(c.D, c.G)), S_T, local, local ? local + maps * states : nullptr,
                          local ? local + (maps + kept) * states : nullptr};
    const bool cut = piece < c.T;
#define KDA_SF(N)                                                                                                          \
    return c.f32 ? c.softplus ? scan::fwd_t<float, N / 4, true>(a, cut, zero_rest && packed, stream) : scan::fwd_t<float, N / 4, false>(a, cut, zero_rest && packed, stream) \
                 : c.softplus ? scan::fwd_t<bf16, N / 4, true>(a, cut, zero_rest && packed, stream) : scan::fwd_t<bf16, N / 4, false>(a, cut, zero_rest && packed, stream)
    switch (c.N) {
        case 8: KDA_SF(8);
        case 16: KDA_SF(16);
        case 32: KDA_SF(32);
        case 64: KDA_SF(64);
    }
#undef KDA_SF
    return hipErrorInvalidValue;
}

}  // namespace kda
