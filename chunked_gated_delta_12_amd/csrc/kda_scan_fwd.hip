// kda_scan_fwd.hip -- the selective scan over whole sequences (kda_scan.hpp has the formulas
// and how lanes and pieces are laid out).
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
    bool softplus;
    const void *x, *dt, *b, *c, *z;
    const float *A, *skip, *bias, *S0;
    void* y;
    float *S_T, *local, *sums;   // maps: end state from nothing [slot][D][N], sum of delta [slot][D]
};

template <typename E, int NS, bool MAP>
__global__ void __launch_bounds__(BLOCK) scan_walk(FwdArgs a) {
    constexpr int N = 4 * NS, GROUPS = TILE / 4;
    __shared__ float rows[2][2 * TILE * N];
    const int per = (a.D / a.G + BLOCK_CH - 1) / BLOCK_CH, nblk = a.G * per;
    const int blk = (int)(blockIdx.x % (unsigned)nblk);
    const int64_t slot = blockIdx.x / (unsigned)nblk;
    Place pl;
    if (!place_of(a.seqs, slot, pl)) return;
    if (MAP && pl.k == pl.pieces - 1) return;
    const int grp = blk / per, Dg = a.D / a.G;
    const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, q = lane & 3;
    const int in_group = (blk % per) * BLOCK_CH + wave * WAVE_CH + (lane >> 2);
    const bool real = in_group < Dg;
    const int ch = grp * Dg + (real ? in_group : Dg - 1);   // lanes without a channel repeat the last and store nothing
    const int t_first = pl.k * a.seqs.piece;
    const int n = pl.len - t_first < a.seqs.piece ? pl.len - t_first : a.seqs.piece;
    const int64_t row = pl.row0 + t_first;
    const bool gated = a.z != nullptr;
    const uint32_t own = (uint32_t)ch * sizeof(E), ld_x = (uint32_t)a.D * sizeof(E);
    const int64_t ld = (int64_t)a.G * N;
    const E *b = (const E*)a.b + grp * N, *c = (const E*)a.c + grp * N;
    const float bias = a.bias ? a.bias[ch] : 0.0f, skip = a.skip ? a.skip[ch] : 0.0f;
    const int64_t at_state = (int64_t)ch * N + q * NS, states = (int64_t)a.D * N;

    Rows<E, N> next;
    E nx[GROUPS], nt[GROUPS], nz[GROUPS];
    auto fetch = [&](int t0) {
        next.fetch(b, c, row, ld, t0, n);
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            const int t = 4 * g + q, last = n - 1 - t0;
            const uint32_t off = own + (uint32_t)(t < last ? t : last) * ld_x;
            const int64_t base = (row + t0) * a.D;
            nx[g] = ld_off((const E*)a.x + base, off);
            nt[g] = ld_off((const E*)a.dt + base, off);
            if (!MAP && gated) nz[g] = ld_off((const E*)a.z + base, off);
        }
    };
    if (n > 0) fetch(0);

    float A2[NS], h[NS];
    ld_states<NS>(a.A + at_state, A2);
#pragma unroll
    for (int i = 0; i < NS; ++i) A2[i] *= LOG2E, h[i] = 0.0f;
    float* local = a.local + at_state;
    if (pl.k == 0) {
        // the last piece has no map: its place keeps S0, which S_T may overwrite during the walk
        const float* from = !MAP && pl.pieces > 1 ? local + (pl.first + pl.pieces - 1) * states
                                                  : a.S0 + (int64_t)pl.seq * states + at_state;
        if (a.S0) ld_states<NS>(from, h);
        if (MAP && a.S0 && real) st_states<NS>(local + (pl.first + pl.pieces - 1) * states, h);
    } else if (!MAP) {
        for (int j = 0; j < pl.k; ++j) {
            float l[NS];
            ld_states<NS>(local + (pl.first + j) * states, l);
            const float s = a.sums[(pl.first + j) * a.D + ch];
#pragma unroll
            for (int i = 0; i < NS; ++i) h[i] = j ? __builtin_fmaf(__builtin_amdgcn_exp2f(s * A2[i]), h[i], l[i]) : l[i];
        }
    }
    float sum = 0.0f;
    for (int t0 = 0, buf = 0; t0 < n; t0 += TILE, buf ^= 1) {
        next.store(rows[buf]);
        E cx[GROUPS], ct[GROUPS], cz[GROUPS];
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) cx[g] = nx[g], ct[g] = nt[g], cz[g] = nz[g];
        lds_barrier();   // one a tile: a buffer is written again only after the barrier of the other's tile
        if (t0 + TILE < n) fetch(t0 + TILE);
        const float* bl = rows[buf] + q * NS;
        const float* cl = bl + TILE * N;
#pragma unroll
        for (int g = 0; g < GROUPS; ++g) {
            if (t0 + 4 * g >= n) break;
            const int t = t0 + 4 * g + q;
            const float xv = (float)cx[g];
            float d = (float)ct[g] + bias;
            if (a.softplus) d = softplus(d);
            float u = d * xv;
            if (t >= n) d = u = 0.0f;   // a step of nothing
            sum += d;
            float dj[4] = {quad_lane<0>(d), quad_lane<1>(d), quad_lane<2>(d), quad_lane<3>(d)};
            float uj[4] = {quad_lane<0>(u), quad_lane<1>(u), quad_lane<2>(u), quad_lane<3>(u)};
            float yj[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                float bv[NS], cv[NS];
                ld_states<NS>(bl + (4 * g + j) * N, bv);
                if (!MAP) ld_states<NS>(cl + (4 * g + j) * N, cv);
                float s = 0.0f;
#pragma unroll
                for (int i = 0; i < NS; ++i) {
                    h[i] = __builtin_fmaf(__builtin_amdgcn_exp2f(dj[j] * A2[i]), h[i], uj[j] * bv[i]);
                    if (!MAP) s = i ? __builtin_fmaf(cv[i], h[i], s) : cv[i] * h[i];
                }
                yj[j] = s;
            }
            if (!MAP) {
                float yv = quad_sums(yj, q);
                if (a.skip) yv = __builtin_fmaf(skip, xv, yv);
                if (gated) {
                    const float zv = (float)cz[g];
                    yv *= zv * sigmoid(zv);
                }
                if (t < n && real) st_off((E*)a.y + (row + t0) * a.D, own + (uint32_t)(4 * g + q) * ld_x, yv);
            }
        }
    }
    if (MAP) {
        sum = quad_sum(sum);
        if (real) {
            st_states<NS>(local + slot * states, h);
            if (q == 0) a.sums[slot * a.D + ch] = sum;
        }
    } else if (a.S_T && pl.k == pl.pieces - 1 && real) {
        st_states<NS>(a.S_T + (int64_t)pl.seq * states + at_state, h);
    }
}

// Tokens a piece.
static int fwd_piece(int nseq, int T, int D, int G, bool packed) {
    const int64_t blocks = blocks_of(D, G), rows = packed ? T : (int64_t)nseq * T;
    const int64_t whole = ((int64_t)T + TILE - 1) / TILE * TILE;
    if (!packed && nseq * blocks >= 256) return (int)whole;
    const int64_t pieces = 512 / blocks > 1 ? 512 / blocks : 1;
    int64_t len = rows / pieces;
    if (len < 2 * TILE) len = 2 * TILE;
    if (len < T / 256) len = T / 256;
    len = (len + TILE - 1) / TILE * TILE;
    return (int)(len < whole ? len : whole);
}

template <typename E, int NS>
static hipError_t fwd_t(const FwdArgs& a, int64_t slots, bool cut, hipStream_t stream) {
    const unsigned grid = (unsigned)(slots * blocks_of(a.D, a.G));
    if (cut) hipLaunchKernelGGL((scan_walk<E, NS, true>), dim3(grid), dim3(BLOCK), 0, stream, a);
    hipLaunchKernelGGL((scan_walk<E, NS, false>), dim3(grid), dim3(BLOCK), 0, stream, a);
    return hipGetLastError();
}

}  // namespace scan

int64_t scan_fwd_workgroups(int nseq, int T, int D, int G, bool packed) {
    return scan::slots_of(nseq, T, scan::fwd_piece(nseq, T, D, G, packed), packed) * scan::blocks_of(D, G);
}

size_t scan_fwd_workspace_bytes(int nseq, int T, int D, int N, int G, bool packed) {
    const int piece = scan::fwd_piece(nseq, T, D, G, packed);
    if (piece >= T) return 0;
    return (size_t)scan::slots_of(nseq, T, piece, packed) * D * (N + 1) * sizeof(float);
}

hipError_t launch_scan_fwd(const ScanCall& c, void* y, float* S_T, void* workspace, hipStream_t stream) {
    const bool packed = c.cu != nullptr;
    const int piece = scan::fwd_piece(c.nseq, c.T, c.D, c.G, packed);
    const int64_t slots = scan::slots_of(c.nseq, c.T, piece, packed);
    float* local = (float*)workspace;
    const scan::FwdArgs a{{c.nseq, c.T, piece, c.cu}, c.D, c.G, c.softplus, c.x, c.dt, c.b, c.c, c.z, c.A, c.skip, c.bias, c.S0,
                          y, S_T, local, local ? local + slots * c.D * c.N : nullptr};
    const bool cut = piece < c.T;
#define KDA_SF(N) return c.f32 ? scan::fwd_t<float, N / 4>(a, slots, cut, stream) : scan::fwd_t<bf16, N / 4>(a, slots, cut, stream)
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
