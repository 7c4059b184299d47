// kda_gdr_grad.hip -- the chunked gated delta rule's gradients of q, k, g and beta inside a
// chunk, from its start state S, the gradient dS at its end, e and Z (kda_gdr.hpp), all
// chunks at once.  With X_ts = do_t.e_s and W_ts = Z_t.e_s,
//     a'_ts = scale D_ts X_ts (q_t.k_s) (s <= t),   b'_ts = -D_ts W_ts (k_t.k_s) (s < t)
//     dq = scale gam (dO S^T) + (scale D X beta_s) K
//     dk = om beta (E dS^T) - gam (Z S^T) + (scale D X beta_s)^T Q + (M + M^T) K,  M = -D W beta_s
//     dbeta_s = sum_t (a' + b')_ts + om_s k_s.(E dS^T)_s
//     dG_t  = sum_s beta_s (a' + b')_ts - beta_t sum_u (a' + b')_ut
//             + gam_t (scale q_t.(dO S^T)_t - k_t.(Z S^T)_t) - om_t beta_t k_t.(E dS^T)_t
//     dG_end += sum_t om_t beta_t k_t.(E dS^T)_t + gam_end <S, dS>,   dg_t = sum_{u >= t} dG_u
// A unit is one value head of one chunk (of up to GB 32-column blocks at a time).  A workgroup
// goes through the value heads of a key head, so that the gradients of the shared q and k
// are summed in registers, and then on to its next chunk.  Each of its eight wavefronts has
// one tile of 16 channels (at dk < 128 two or four share one and split the tokens): its
// rows of S and dS go from memory into registers as operands, all of a unit's at once, and
// results are [channel][token], four channels of one token a lane, which is how they are
// stored, how the tokens' factors apply and what the dot products with q and k need.  e, Z
// and dO, which every wavefront needs, lie in LDS.  The ten tiles of X and W on and below the
// diagonal go to the wavefronts in turn and reach the others through LDS as the operands of the
// last products, read there as rows of queries and, transposed, as rows of keys.
// Memory bounds it: 192 KB of states and rows a unit at dk = dv = 128.  The next unit's loads
// are issued before this unit's last part, as many as fit the registers.  Measured at 8 x 4,096 tokens,
// 16 heads, dk = dv = 128: 650-690 us, 2.3 GB, 3.4 TB/s.
#include <type_traits>

#include "kda_gdr.hpp"
#include "kda_launch.hpp"

namespace kda {
namespace gdr {

namespace {

constexpr int GTHR = 512;

template <typename E, int DK>
struct GradLay {
    static constexpr int KB = DK / 32, ST = DK / 16, EXB = Arith<E>::EXB;
    static constexpr int SPLIT = 8 / ST, TT = MT / SPLIT;     // wavefronts a channel tile, token tiles of each
    static constexpr int GB = sizeof(E) == 2 ? 4 : 1;         // 32-column blocks of a unit in LDS at once
    static constexpr int QK = MT * KB * EXB;
    static constexpr int SPB = Arith<E>::SPB, TB = TRI * SPB;
    static constexpr int E_AT = 0, Z_AT = MT * SPB, O_AT = 2 * MT * SPB, BLK = O_AT + MT * EXB;   // one column block
    static constexpr int BUF = GB * BLK;
    static_assert(2 * TB <= BUF, "the exchanged tiles lie over the column blocks");
    static constexpr int PQK = QK / 16, NQK = (PQK + GTHR - 1) / GTHR;
    static constexpr int PO = MT * EXB / 16, NO = (GB * PO + GTHR - 1) / GTHR;   // pieces of do in a block; a thread's in all
};

__device__ __forceinline__ float over_groups(float x) {
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

template <typename E, int DK>
__global__ void __launch_bounds__(GTHR, 2)
grad_kernel(Args a, int items, const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ dout,
            const char* __restrict__ prep, const char* __restrict__ recs, E* __restrict__ dq, E* __restrict__ dk, float* __restrict__ dg, float* __restrict__ dbeta) {
    typedef Arith<E> A;
    typedef GradLay<E, DK> L;
    typedef typename A::Sp Sp;
    typedef typename A::Ex Ex;
    constexpr int KB = L::KB, ST = L::ST, TT = L::TT, GB = L::GB;
    __shared__ alignas(16) char kl[L::QK];
    __shared__ alignas(16) char ql[L::QK];
    __shared__ alignas(16) char lds[L::BUF];
    __shared__ double Gs[C];
    __shared__ alignas(16) float csum[10][16];
    __shared__ float gam[C], om[C], bts[C], part[3][ST][C], rsum[10][16], dots[8];
    int tid, lane, g, r;
    // Addresses are formed anew from the thread's number in every unit: kept over the loop they
    // would not fit in the registers beside the operands in flight.
    auto anew = [&]() {
        tid = threadIdx.x;
        asm volatile("" : "+v"(tid));
        lane = tid & 63;
        g = lane >> 4;
        r = lane & 15;
    };
    anew();
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ct = w % ST, m0 = w / ST * TT;   // this wavefront's channel tile and first token tile
    const int rep = a.Hv / a.Hk, nb = a.dv / 32, ngrp = (nb + GB - 1) / GB;
    const int64_t ldk = (int64_t)a.Hk * DK, ldv = (int64_t)a.Hv * a.dv;
    const f32x4 zero = {0, 0, 0, 0};
    char* const xch = lds;   // scale D X beta_s and M, [t][s], once a unit's column blocks have been read

    // A unit: group `grp` of value head vh of an item, the item's chunk in ch.
    struct Unit3 {
        int item, vh, grp, valid;
        int64_t row0;
    };
    auto first = [&](int item) {   // the first item from here on that has a chunk
        Unit3 u{item, 0, 0, 0, 0};
        for (; u.item < items; u.item += (int)gridDim.x) {
            const Chunk ch = chunk_at(a, u.item / a.Hk, lane);
            u.valid = ch.valid;
            u.row0 = ch.row0;
            if (ch.n >= 0) break;
        }
        return u;
    };
    auto next = [&](const Unit3& u) {
        if (u.grp + 1 < ngrp) return Unit3{u.item, u.vh, u.grp + 1, u.valid, u.row0};
        if (u.vh + 1 < rep) return Unit3{u.item, u.vh + 1, 0, u.valid, u.row0};
        return first(u.item + (int)gridDim.x);
    };

    const uint32_t sbytes = (uint32_t)state_bytes(DK, a.dv), ebytes = (uint32_t)rows_bytes(a.dv), rbytes = 2 * (sbytes + ebytes);
    Rec sf[GB], df[GB];
    u32x4 se[GB], sz[GB], so[L::NO], sk[L::NQK], sq[L::NQK];
    float fac[3] = {0, 0, 0};
    double facG = 0.0;
    auto rec_of = [&](const Unit3& u) { return (int64_t)(u.item / a.Hk) * a.Hv + u.item % a.Hk * rep + u.vh; };
    // The states' blocks lo .. hi of a unit; past the last block an offset beyond the record:
    // zeros, which add nothing.
    auto load_states = [&](const Unit3& u, auto lo, auto hi) {
        const Rsrc rs = make_rsrc(recs + rec_of(u) * rbytes, rbytes);
        const int b0 = u.grp * GB;
#pragma unroll
        for (int b = decltype(lo)::value; b < decltype(hi)::value; ++b) {
            const uint32_t at = b0 + b < nb ? (uint32_t)((ct * nb + b0 + b) * WSB) + rec_at(lane, 0) : 0x80000000u;
            sf[b] = ld_rec(rs, at);
            df[b] = ld_rec(rs, at + sbytes);
        }
    };
    typedef std::integral_constant<int, 0> B0;
    typedef std::integral_constant<int, sizeof(E) == 2 ? 1 : 0> BH;   // how many are asked for a unit ahead: what the registers hold
    typedef std::integral_constant<int, GB> BN;
    auto load = [&](const Unit3& u) {
        const int hk = u.item % a.Hk, h = hk * rep + u.vh, b0 = u.grp * GB;
        const Rsrc rs = make_rsrc(recs + rec_of(u) * rbytes, rbytes);
#pragma unroll
        for (int b = 0; b < GB; ++b) {   // 512 pieces of e and of Z a block: one a thread
            const uint32_t at = b0 + b < nb ? 2 * sbytes + (uint32_t)(((tid >> 7) * nb + b0 + b) * WSB + (tid & 127) * 16) : 0x80000000u;
            se[b] = buf_ld128(rs, at);
            sz[b] = buf_ld128(rs, at + ebytes);
        }
        const Rsrc ro = make_rsrc(dout + u.row0 * ldv + (int64_t)h * a.dv, (uint32_t)((u.valid - 1) * ldv + a.dv) * (uint32_t)sizeof(E));
#pragma unroll
        for (int j = 0; j < L::NO; ++j) {   // accumulator slots of a row; rows past the end are zero
            const int p = tid + j * GTHR, b = p / L::PO, x = p % L::PO, l = x & 63;
            const int m = sizeof(E) == 2 ? x >> 6 : x >> 7, half = sizeof(E) == 2 ? 0 : (x >> 6) & 1;
            const uint32_t at = b < GB && b0 + b < nb ? (uint32_t)((16 * m + (l & 15)) * ldv + 32 * (b0 + b) + 4 * (l >> 4) + 16 * half) * (uint32_t)sizeof(E) : 0x80000000u;
            if constexpr (sizeof(E) == 2) {
                const f32x2 lo = buf_ld_f2(ro, at, 0), hi = buf_ld_f2(ro, at + 32, 0);
                so[j] = __builtin_bit_cast(u32x4, f32x4{lo[0], lo[1], hi[0], hi[1]});
            } else {
                so[j] = buf_ld128(ro, at);
            }
        }
        load_states(u, B0{}, BH{});
    };

    // K, Q and the tokens' factors, for the second half of a unit
    auto load_kq = [&](const Unit3& u) {
        const int hk = u.item % a.Hk;
        const uint32_t kbytes = (uint32_t)((u.valid - 1) * ldk + DK) * (uint32_t)sizeof(E);
        const Rsrc rk = make_rsrc(k + u.row0 * ldk + (int64_t)hk * DK, kbytes), rq = make_rsrc(q + u.row0 * ldk + (int64_t)hk * DK, kbytes);
#pragma unroll
        for (int j = 0; j < L::NQK; ++j) {
            const int p = tid + j * GTHR, l = p & 63, blk = sizeof(E) == 2 ? p >> 6 : p >> 7, half = sizeof(E) == 2 ? 0 : (p >> 6) & 1;
            const uint32_t at = p < L::PQK ? (uint32_t)((16 * (blk / KB) + (l & 15)) * ldk + 32 * (blk % KB) + 8 * (l >> 4) + 4 * half) * (uint32_t)sizeof(E) : 0x80000000u;
            sk[j] = buf_ld128(rk, at);
            sq[j] = buf_ld128(rq, at);
        }
        if (tid < C) {
            const float* f = reinterpret_cast<const float*>(prep + rec_of(u) * PREP_BYTES + X_BYTES);
            fac[0] = f[tid];
            fac[1] = f[2 * C + tid];
            fac[2] = f[3 * C + tid];
            facG = reinterpret_cast<const double*>(f + 4 * C)[tid];
        }
    };

    // The tiles of X and W, queries m and keys n <= m, as [s][t]: one a wavefront, the last two on
    // wavefronts 0 and 1.
    auto tile_of = [&](int j, int& m, int& n) {
        const int t = 8 * j + w;
        m = t >= 6 ? 3 : t >= 3 ? 2 : t >= 1 ? 1 : 0;
        n = t - m * (m + 1) / 2;
        return t < 10;
    };
    Unit3 u = first((int)blockIdx.x);
    if (u.item >= items) return;
    load(u);
    f32x4 aq[TT], ak[TT], dos[TT], zs[TT], eds[TT], x[2], mm[2];
    float dot = 0.0f;   // <S, dS>
#pragma unroll
    for (int t = 0; t < TT; ++t) aq[t] = ak[t] = dos[t] = zs[t] = eds[t] = zero;
#pragma unroll
    for (int j = 0; j < 2; ++j) x[j] = mm[j] = zero;
    for (;;) {
        const int hk = u.item % a.Hk, h = hk * rep + u.vh;
        anew();
        lds_barrier();   // the unit before is done with LDS
#pragma unroll
        for (int b = 0; b < GB; ++b) {
            put_piece<E>(lds + b * L::BLK + L::E_AT, tid, se[b]);
            put_piece<E>(lds + b * L::BLK + L::Z_AT, tid, sz[b]);
        }
#pragma unroll
        for (int j = 0; j < L::NO; ++j) {
            const int p = tid + j * GTHR;
            if (GB * L::PO % GTHR == 0 || p < GB * L::PO) *reinterpret_cast<u32x4*>(lds + (p / L::PO) * L::BLK + L::O_AT + (p % L::PO) * 16) = so[j];
        }
        lds_barrier();
        anew();
        load_states(u, BH{}, BN{});   // into the registers that e and Z have left
#pragma unroll
        for (int b = 0; b < GB; ++b) {
            const char* buf = lds + b * L::BLK;
            if (b == GB / 2) load_kq(u);   // into the registers that the first states have left
            if (L::SPLIT == 1 || m0 == 0)
#pragma unroll
                for (int i = 0; i < 4; ++i) dot += sf[b].a[i] * df[b].a[i] + sf[b].b[i] * df[b].b[i];
            asm volatile("" : "+v"(dot));   // here, while the states' registers are needed anyway
            {
                const Sp s = A::split(sf[b].a, sf[b].b);
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    dos[t] = A::mma(s, A::ld_ex(buf + L::O_AT, m0 + t, swz(lane)), dos[t]);
                    zs[t] = A::mma(s, A::ld_sp(buf + L::Z_AT, m0 + t, lane), zs[t]);
                }
            }
            {
                const Sp d = A::split(df[b].a, df[b].b);
#pragma unroll
                for (int t = 0; t < TT; ++t) eds[t] = A::mma(d, A::ld_sp(buf + L::E_AT, m0 + t, lane), eds[t]);
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                int m, n;
                if (!tile_of(j, m, n)) continue;
                const Sp e = A::ld_sp(buf + L::E_AT, n, lane);
                x[j] = A::mma(e, A::ld_ex(buf + L::O_AT, m, swz(lane)), x[j]);
                mm[j] = A::mma(e, A::ld_sp(buf + L::Z_AT, m, lane), mm[j]);
            }
        }
        const Unit3 nu = next(u);
        const bool more = nu.item < items, whole = u.grp + 1 == ngrp;
        if (tid < C) {
            gam[tid] = fac[0];
            om[tid] = fac[1];
            bts[tid] = fac[2];
            Gs[tid] = facG;
        }
        if (u.vh == 0 && u.grp == 0) {
#pragma unroll
            for (int j = 0; j < L::NQK; ++j) {
                const int p = tid + j * GTHR, to = ((p & ~63) + swz(p & 63)) * 16;
                if (L::PQK % GTHR == 0 || p < L::PQK) {
                    *reinterpret_cast<u32x4*>(kl + to) = sk[j];
                    *reinterpret_cast<u32x4*>(ql + to) = sq[j];
                }
            }
        }
        anew();
        if (more) load(nu);
        if (whole) {
            lds_barrier();   // K and Q are there
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                int m, n;
                if (!tile_of(j, m, n)) continue;
                f32x4 qk = zero, kk = zero, xv, mv;
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    const Ex kn = A::ld_ex(kl, n * KB + b, lane);
                    qk = A::mma(kn, A::ld_ex(ql, m * KB + b, lane), qk);
                    kk = A::mma(kn, A::ld_ex(kl, m * KB + b, lane), kk);
                }
                float row = 0.0f;   // the query's sum of beta_s (a' + b')
                f32x4 col;          // a' + b' of four keys
                const int tq = 16 * m + r;
#pragma unroll
                for (int l = 0; l < 4; ++l) {
                    const int ts = 16 * n + 4 * g + l;
                    const bool in = ts <= tq;
                    const float d = __builtin_amdgcn_exp2f(in ? (float)(Gs[tq] - Gs[ts]) : 0.0f), b = bts[ts];
                    xv[l] = in ? a.scale * d * x[j][l] : 0.0f;
                    mv[l] = ts < tq ? -d * mm[j][l] : 0.0f;
                    col[l] = xv[l] * qk[l] + mv[l] * kk[l];
                    row += b * col[l];
                    xv[l] *= b;
                    mv[l] *= b;
                }
                A::put_half(xch, lower_block(m, n / 2), lane, n & 1, xv);
                A::put_half(xch + L::TB, lower_block(m, n / 2), lane, n & 1, mv);
                row = over_groups(row);
#pragma unroll
                for (int s = 1; s < 16; s <<= 1)
#pragma unroll
                    for (int l = 0; l < 4; ++l) col[l] += __shfl_xor(col[l], s);
                const int t = m * (m + 1) / 2 + n;
                if (g == 0) rsum[t][r] = row;
                if (r == 0) *reinterpret_cast<f32x4*>(&csum[t][4 * g]) = col;
                x[j] = mm[j] = zero;
            }
            if (w < 4) A::put_half(xch + (w & 1) * L::TB, w < 2 ? lower_block(0, 0) : lower_block(2, 1), lane, 1, zero);   // beyond the diagonal
            // the states' parts, and their products with q and k over this channel tile
#pragma unroll
            for (int t = 0; t < TT; ++t) {
                const int tok = 16 * (m0 + t) + r;
                const float gt = gam[tok], ob = om[tok] * bts[tok];
                const Ex qv = A::ld_ex(ql, (m0 + t) * KB + ct / 2, lane), kv = A::ld_ex(kl, (m0 + t) * KB + ct / 2, lane);
                float qs = 0.0f, kz = 0.0f, ke = 0.0f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float qi = ct & 1 ? A::at(qv, 4 + i) : A::at(qv, i), ki = ct & 1 ? A::at(kv, 4 + i) : A::at(kv, i);
                    qs += qi * dos[t][i];
                    kz += ki * zs[t][i];
                    ke += ki * eds[t][i];
                    aq[t][i] += a.scale * gt * dos[t][i];
                    ak[t][i] += ob * eds[t][i] - gt * zs[t][i];
                }
                qs = over_groups(qs);
                kz = over_groups(kz);
                ke = over_groups(ke);
                if (g == 0) {
                    part[0][ct][tok] = qs;
                    part[1][ct][tok] = kz;
                    part[2][ct][tok] = ke;
                }
                dos[t] = zs[t] = eds[t] = zero;
            }
#pragma unroll
            for (int s = 1; s < 64; s <<= 1) dot += __shfl_xor(dot, s);
            if (lane == 0) dots[w] = dot;
            dot = 0.0f;
            lds_barrier();
            anew();
            // Tokens' block by block from the transposed K and Q.  bf16: both blocks' operands at once, token tiles
            // outside; fp32, where an operand is eight registers, one block after the other (the sums' order is the same).
            if constexpr (sizeof(E) == 2) {
                Ex kt[2], qt[2];
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    kt[tb] = A::template ld_ex_t<KB>(kl, ct / 2, ct & 1, tb, g, r);
                    qt[tb] = A::template ld_ex_t<KB>(ql, ct / 2, ct & 1, tb, g, r);
                }
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const int m = m0 + t;
#pragma unroll
                    for (int tb = 0; tb < 2; ++tb) {
                        if (tb <= m / 2) {
                            aq[t] = A::mma(kt[tb], A::ld_sp(xch, lower_block(m, tb), lane), aq[t]);
                            ak[t] = A::mma(kt[tb], A::ld_sp(xch + L::TB, lower_block(m, tb), lane), ak[t]);
                        }
                        if (tb >= m / 2) {
                            ak[t] = A::mma(qt[tb], A::ld_tri_t(xch, m, tb, g, r), ak[t]);
                            ak[t] = A::mma(kt[tb], A::ld_tri_t(xch + L::TB, m, tb, g, r), ak[t]);
                        }
                    }
                }
            } else {
                auto block = [&](int tb, const Ex& kt, const Ex& qt) {
#pragma unroll
                    for (int t = 0; t < TT; ++t) {
                        const int m = m0 + t;
                        if (tb <= m / 2) {
                            aq[t] = A::mma(kt, A::ld_sp(xch, lower_block(m, tb), lane), aq[t]);
                            ak[t] = A::mma(kt, A::ld_sp(xch + L::TB, lower_block(m, tb), lane), ak[t]);
                        }
                        if (tb >= m / 2) {
                            ak[t] = A::mma(qt, A::ld_tri_t(xch, m, tb, g, r), ak[t]);
                            ak[t] = A::mma(kt, A::ld_tri_t(xch + L::TB, m, tb, g, r), ak[t]);
                        }
                    }
                };
#pragma unroll
                for (int tb = 0; tb < 2; ++tb)
                    block(tb, A::template ld_ex_t<KB>(kl, ct / 2, ct & 1, tb, g, r), A::template ld_ex_t<KB>(ql, ct / 2, ct & 1, tb, g, r));
            }
            if (w == 0) {   // g's and beta's: lane is the token
                float qs = 0.0f, kz = 0.0f, ke = 0.0f, ab = 0.0f, ac = 0.0f, sd = 0.0f;
#pragma unroll
                for (int j = 0; j < ST; ++j) {
                    qs += part[0][j][lane];
                    kz += part[1][j][lane];
                    ke += part[2][j][lane];
                }
#pragma unroll
                for (int o = 0; o < MT; ++o) {   // row sums over the keys' tiles, column sums over the queries'
                    if (o <= g) ab += rsum[g * (g + 1) / 2 + o][r];
                    if (o >= g) ac += csum[o * (o + 1) / 2 + g][r];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) sd += dots[j];
                const float b = bts[lane], o = om[lane], obk = o * b * ke;
                double v = (double)ab - (double)(b * ac) + (double)(gam[lane] * (a.scale * qs - kz)) - (double)obk;
                double e = (double)obk;
#pragma unroll
                for (int s = 32; s >= 1; s >>= 1) e += __shfl_xor(e, s);
                if (lane == 63) v += e + (double)(gam[C - 1] * sd);   // the chunk's end decays into every om, and the state
#pragma unroll
                for (int s = 1; s < 64; s <<= 1) {
                    const double dn = __shfl_down(v, s);
                    if (lane + s < 64) v += dn;
                }
                if (lane < u.valid) {
                    dg[(u.row0 + lane) * a.Hv + h] = (float)v;
                    dbeta[(u.row0 + lane) * a.Hv + h] = ac + o * ke;
                }
            }
            if (u.vh + 1 == rep) {
#pragma unroll
                for (int t = 0; t < TT; ++t) {
                    const int tok = 16 * (m0 + t) + r;
                    const int64_t at = (u.row0 + tok) * ldk + hk * DK + 32 * (ct / 2) + 8 * g + 4 * (ct & 1);
                    if (tok < u.valid) {
                        A::st4(dq + at, aq[t]);
                        A::st4(dk + at, ak[t]);
                    }
                    aq[t] = ak[t] = zero;
                }
            }
        }
        if (!more) return;
        u = nu;
    }
}

template <typename E, int DK>
hipError_t grad_t(const Args& a, const void* q, const void* k, const void* dout, const char* prep,
                  const char* recs, void* dq, void* dk, float* dg,
                  float* dbeta, hipStream_t stream) {
    const int items = (int)(places_of(a.nseq, a.T, a.cu != nullptr, C) * a.Hk);
    const int grid = items < 256 ? items : 256;   // one resident workgroup a compute unit
    hipLaunchKernelGGL((grad_kernel<E, DK>), dim3((unsigned)grid), dim3(GTHR), 0, stream, a, items, (const E*)q, (const E*)k,
                       (const E*)dout, prep, recs, (E*)dq, (E*)dk, dg, dbeta);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grad(bool f32, int dk_, const Args& a, const void* q, const void* k, const void* dout,
                       const char* prep, const char* recs, void* dq,
                       void* dk, float* dg, float* dbeta, hipStream_t stream) {
#define KDA_GG(E, D) return grad_t<E, D>(a, q, k, dout, prep, recs, dq, dk, dg, dbeta, stream)
    if (f32) {
        switch (dk_) {
            case 32: KDA_GG(float, 32);
            case 64: KDA_GG(float, 64);
            case 128: KDA_GG(float, 128);
        }
    } else {
        switch (dk_) {
            case 32: KDA_GG(bf16, 32);
            case 64: KDA_GG(bf16, 64);
            case 128: KDA_GG(bf16, 128);
        }
    }
#undef KDA_GG
    return hipErrorInvalidValue;
}

}  // namespace gdr
}  // namespace kda
