// kda_gdr_chain.hip -- the chunked gated delta rule's walk over a sequence's chunks: the
// states forwards (with the outputs, saving each chunk's start state for the backward
// pass, or forming a piece's affine map), and the states' gradients backwards.
// Mathematics, precision and layouts: kda_gdr.hpp.
//
// Columns of the state (dv) are independent.  A workgroup of NW wavefronts has one head of
// one piece of a sequence and 16 NW NC columns, a wavefront NC tiles of 16: its slice of the state
// stays in fp32 accumulators for the whole walk, and every product of a chunk takes its
// result straight from the one before it (an accumulator tile is a B operand; read as an A
// operand it is its transpose), so the wavefronts share nothing but the chunk's operands.
// Those lie in LDS as fragment blocks: bf16 double-buffered, the next chunk's loads in
// flight in registers under this chunk's products, one barrier a chunk.  Loads go through
// buffer resources that end with the chunk's last token, so a part chunk reads zeros.
//   forwards:   e = X (V - gam (K S));  S <- gam_end S + K^T (om beta e)
//               O^T = scale gam (S^T Q^T) + e^T P^T
//   backwards:  Z = X^T (om beta (K dS) + P^T dO)
//               dS <- gam_end dS + Q^T (scale gam dO) - K^T (gam Z)
// K^T, Q^T and X^T are read from the same blocks as K, Q and X with the transposing LDS read.
// P is formed here, its tiles spread over the wavefronts: read from memory it would be a fifth
// of the chunk's bytes.  A chunk's outputs are stored at the start of the next one: behind the
// loads they would be waited for at the loop's end.
//
// What bounds a walk is one chunk after another: by count, at 128 x 128, the products of the two
// wavefronts of a SIMD take 3 us (221 matrix instructions each), their splits 1.5 and the workgroup's LDS
// reads 2.2, and they overlap little.  Measured at 65,536 tokens of 16 heads, 128 x 128, bf16, in 16 pieces: the walk
// with outputs 450-530 us (its memory accesses alone 277), the maps, two column tiles a wavefront,
// 480-560 us (230).  With operands in two parts they took 340-373 and 335-367, at a
// twentieth of the precision (kda_gdr.hpp).
#include "kda_gdr.hpp"
#include "kda_launch.hpp"

namespace kda {
namespace gdr {

namespace {

enum Mode { FWD, SAVE, MAP, BACK, BMAP };

// LDS of one buffer: K, Q, the chunk's record (X and the factors) and the value rows; P once.
template <typename E, int DK, int NW, int MODE, int NC>
struct Lay {
    static constexpr int KB = DK / 32, NTHR = 64 * NW, SLAB = 16 * NC * NW;
    static constexpr bool BWD = MODE >= BACK;                      // rows of dO instead of V
    static constexpr bool HAS_Q = MODE == FWD || BWD, HAS_P = HAS_Q;
    static constexpr int QK = MT * KB * Arith<E>::EXB;
    // a row of values: 32 bytes more than its columns, so that the rows of a transposing read
    // spread over the banks
    static constexpr int VLD = SLAB + 32 / (int)sizeof(E), VROW = SLAB * (int)sizeof(E) / 16, VB = C * VLD * (int)sizeof(E);
    static constexpr int TB = TRI * Arith<E>::SPB;   // bytes of X, and of P
    static constexpr int Q_AT = QK, X_AT = Q_AT + (HAS_Q ? QK : 0), F_AT = X_AT + TB, V_AT = F_AT + F_BYTES,
                         BYTES = V_AT + VB, PB = HAS_P ? TB : 0;
    static constexpr int BUFS = 2 * BYTES + PB <= 160 * 1024 ? 2 : 1, ALL = BUFS * BYTES + PB;
    // 16-byte pieces, and how many of them a thread moves
    static constexpr int PQK = QK / 16, PX = X_BYTES / 16, PXP = PREP_BYTES / 16, PV = C * VROW;
    static constexpr int NQK = (PQK + NTHR - 1) / NTHR, NXP = (PXP + NTHR - 1) / NTHR, NV = (PV + NTHR - 1) / NTHR;
    // bf16 rows leave through LDS, in the buffer that the chunk is done with
    static constexpr bool ROWS = (MODE == FWD || MODE == BACK) && sizeof(E) == 2 && BUFS == 2;
};

__device__ __forceinline__ f32x4 ld4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

// One chunk's operands on their way from global memory to LDS.
template <typename E, int DK, int NW, int MODE, int NC>
struct Stage {
    typedef Lay<E, DK, NW, MODE, NC> L;
    u32x4 k[L::NQK], q[L::NQK], x[L::NXP], v[L::NV];
    uint32_t kq_off[L::NQK], v_off[L::NV];   // byte offsets in a chunk's rows, the same for every chunk

    __device__ __forceinline__ void init(int64_t ldk, int64_t ldv, int ncol) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int j = 0; j < L::NQK; ++j) {
            const int u = tid + j * L::NTHR, l = u & 63;
            const int blk = sizeof(E) == 2 ? u >> 6 : u >> 7, half = sizeof(E) == 2 ? 0 : (u >> 6) & 1;
            const int row = 16 * (blk / L::KB) + (l & 15), ch = 32 * (blk % L::KB) + 8 * (l >> 4) + 4 * half;
            kq_off[j] = u < L::PQK ? (uint32_t)(row * ldk + ch) * (uint32_t)sizeof(E) : 0xffffffffu;
        }
        constexpr int EPP = 16 / (int)sizeof(E);
#pragma unroll
        for (int j = 0; j < L::NV; ++j) {
            const int u = tid + j * L::NTHR, row = u / L::VROW, col = (u % L::VROW) * EPP;
            v_off[j] = u < L::PV && col < ncol ? (uint32_t)(row * ldv + col) * (uint32_t)sizeof(E) : 0xffffffffu;
        }
    }

    __device__ __forceinline__ void load_k(Rsrc kr) {
#pragma unroll
        for (int j = 0; j < L::NQK; ++j) k[j] = buf_ld128(kr, kq_off[j]);
    }
    __device__ __forceinline__ void load_q(Rsrc qr) {
        if constexpr (L::HAS_Q)
#pragma unroll
            for (int j = 0; j < L::NQK; ++j) q[j] = buf_ld128(qr, kq_off[j]);
    }
    __device__ __forceinline__ void load_x(Rsrc xr) {
#pragma unroll
        for (int j = 0; j < L::NXP; ++j) x[j] = buf_ld128(xr, (uint32_t)(threadIdx.x + j * L::NTHR) * 16);
    }
    __device__ __forceinline__ void load_v(Rsrc vr) {
#pragma unroll
        for (int j = 0; j < L::NV; ++j) v[j] = buf_ld128(vr, v_off[j]);
    }

    __device__ __forceinline__ void store(char* buf) const {
        const int tid = threadIdx.x;
#pragma unroll
        for (int j = 0; j < L::NQK; ++j) {
            const int u = tid + j * L::NTHR;
            if (L::PQK % L::NTHR == 0 || u < L::PQK) {
                const int at = ((u & ~63) + swz(u & 63)) * 16;
                *reinterpret_cast<u32x4*>(buf + at) = k[j];
                if constexpr (L::HAS_Q) *reinterpret_cast<u32x4*>(buf + L::Q_AT + at) = q[j];
            }
        }
#pragma unroll
        for (int j = 0; j < L::NXP; ++j) {
            const int u = tid + j * L::NTHR;
            if (u < L::PX) put_piece<E>(buf + L::X_AT, u, x[j]);
            else if (u < L::PXP) *reinterpret_cast<u32x4*>(buf + L::F_AT + (u - L::PX) * 16) = x[j];
        }
#pragma unroll
        for (int j = 0; j < L::NV; ++j) {
            const int u = tid + j * L::NTHR;
            if (L::PV % L::NTHR == 0 || u < L::PV)
                *reinterpret_cast<u32x4*>(buf + L::V_AT + (u / L::VROW) * L::VLD * (int)sizeof(E) + (u % L::VROW) * 16) = v[j];
        }
    }
};

struct Ptrs {
    const void *q, *k, *v;      // v: do where the walk is backwards
    const float* init;          // [nseq] states (or their gradients) or NULL
    const float* starts;        // those of the pieces of cut sequences, [piece place][Hv][dk][dv]
    const char* prep;
    void* out;                  // o; dv where the walk is backwards
    float* last;                // S_T or dS0, or NULL
    char* recs;                 // SAVE, BACK: the chunks' records
    float* maps;                // MAP: [piece place][Hv][dk][dv + dk]; BMAP: [..][dk][dv]
    bool all;
    int places;
};

// One walk by workgroup `block` of those that the walk has.
// NC: column tiles a wavefront.
template <typename E, int DK, int NW, int MODE, int NC>
__device__ __forceinline__ void walk(const Args& a, const Segs& sg, const Ptrs& io, unsigned block, char* lds) {
    typedef Arith<E> A;
    static_assert(NC == 1 || MODE == MAP, "the other walks' wavefronts have one column tile");
    typedef Lay<E, DK, NW, MODE, NC> L;
    constexpr int KB = L::KB, ST = DK / 16;
    constexpr bool BWD = L::BWD;
    char* const pl = lds + L::BUFS * L::BYTES;   // P
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int ncols = MODE == MAP ? a.dv + DK : a.dv;
    const int nslab = (ncols + L::SLAB - 1) / L::SLAB;
    // Workgroups (the first of a walk at a multiple of eight) go to the eight XCDs in turn: those of one key head's value heads and slabs,
    // which read the same K and Q, are eight apart and share one XCD's L2.
    const unsigned inner = (unsigned)(a.Hv / a.Hk * nslab), grp = block / (8 * inner), in8 = block % (8 * inner);
    const unsigned outer = grp * 8 + in8 % 8, sub = in8 / 8;
    int place = (int)(outer / (unsigned)a.Hk);
    const int hk = (int)(outer % (unsigned)a.Hk);
    const int h = hk * (a.Hv / a.Hk) + (int)(sub / (unsigned)nslab), slab = (int)(sub % (unsigned)nslab);
    if (place >= io.places) return;
    if ((MODE == MAP || MODE == BMAP) && sg.apart) place += a.nseq;   // a launch over the pieces alone
    const Piece pc = piece_at(a, sg, place, lane);
    if (pc.n < 0) return;
    // maps: forwards of every piece but the last one (all where both directions are joined),
    // backwards of every one but the first
    if (MODE == MAP && (pc.cnt < 2 || (!io.all && pc.i + 1 == pc.cnt))) return;
    if (MODE == BMAP && pc.i == 0) return;
    const int nch = pc.c1 - pc.c0;
    const int64_t ldk = (int64_t)a.Hk * DK, ldv = (int64_t)a.Hv * a.dv;
    const int c0 = slab * L::SLAB, col0 = c0 + w * 16 * NC;   // the slab's and the wavefront's first column
    bool on[NC], isM[NC];                                     // its tiles; those of the map's linear part have no values
#pragma unroll
    for (int j = 0; j < NC; ++j) {
        on[j] = col0 + 16 * j < ncols;
        isM[j] = MODE == MAP && col0 + 16 * j >= a.dv;
    }
    const bool act = on[0];
    const E* kp = (const E*)io.k + pc.s.row0 * ldk + (int64_t)hk * DK;
    const E* qp = (const E*)io.q + pc.s.row0 * ldk + (int64_t)hk * DK;
    const E* vp = (const E*)io.v + pc.s.row0 * ldv + (int64_t)h * a.dv + c0;

    // the state at the piece's start (backwards: the gradient at its end)
    f32x4 S[NC][ST];
    {
        const float* from = nullptr;
        if (MODE != MAP && MODE != BMAP) {
            if (pc.cnt > 1) from = io.starts + ((int64_t)pc.at * a.Hv + h) * DK * a.dv;
            else if (io.init) from = io.init + ((int64_t)pc.n * a.Hv + h) * DK * a.dv;
        }
#pragma unroll
        for (int j = 0; j < NC; ++j)
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = 32 * (t / 2) + 8 * g + 4 * (t & 1) + i, col = col0 + 16 * j + r;
                    S[j][t][i] = from && on[j] ? from[(int64_t)row * a.dv + col] : isM[j] && col == a.dv + row ? 1.0f : 0.0f;
                }
    }

    // The start state has arrived before the loop: otherwise the loop would wait for its loads
    // anew in every iteration, and so for the chunk that it has just asked for.
#pragma unroll
    for (int j = 0; j < NC; ++j)
#pragma unroll
        for (int t = 0; t < ST; ++t) asm volatile("" : "+v"(S[j][t]));
    Stage<E, DK, NW, MODE, NC> st;
    st.init(ldk, ldv, a.dv - c0);
    struct Res { Rsrc k, q, v, x; };
    auto res_of = [&](int c) {
        const int left = pc.s.len - c * C;
        const int valid = left < C ? left : C;
        const int64_t row = (int64_t)c * C;
        // rows past the chunk's last token read as zero; the head's offset is in the base
        const int vc = a.dv - c0 < L::SLAB ? a.dv - c0 : L::SLAB;   // none in a slab of the linear part alone
        return Res{make_rsrc(kp + row * ldk, (uint32_t)((valid - 1) * ldk + DK) * (uint32_t)sizeof(E)),
                   make_rsrc(qp + row * ldk, (uint32_t)((valid - 1) * ldk + DK) * (uint32_t)sizeof(E)),
                   make_rsrc(vp + row * ldv, vc > 0 ? (uint32_t)((valid - 1) * ldv + vc) * (uint32_t)sizeof(E) : 0u),
                   make_rsrc(io.prep + (((int64_t)pc.slot + c) * a.Hv + h) * PREP_BYTES, PREP_BYTES)};
    };
    auto chunk_of = [&](int it) { return BWD ? pc.c1 - 1 - it : pc.c0 + it; };
    // A chunk's finished rows are stored one chunk later: from LDS, 16 bytes a thread in whole
    // rows of the slab (`from`: that chunk's buffer), or from the registers.
    typename A::Q4 fin[MT];
    auto flush = [&](int c, const char* from) {
        const int left = pc.s.len - c * C, valid = left < C ? left : C;
        const Rsrc orr = make_rsrc((E*)io.out + (pc.s.row0 + (int64_t)c * C) * ldv, (uint32_t)(valid * ldv) * (uint32_t)sizeof(E));
        if constexpr (L::ROWS) {
#pragma unroll
            for (int j = 0; j < L::NV; ++j) {
                const int u = (int)threadIdx.x + j * L::NTHR, row = u / L::VROW, col = c0 + (u % L::VROW) * 8;
                const u32x4 x = *reinterpret_cast<const u32x4*>(from + L::V_AT + row * L::VLD * 2 + (u % L::VROW) * 16);
                __builtin_amdgcn_raw_buffer_store_b128(
                    x, orr, col < a.dv ? (int)((row * ldv + (int64_t)h * a.dv + col) * 2) : (int)0x80000000u, 0, 0);
            }
        } else {
#pragma unroll
            for (int m = 0; m < MT; ++m)
                buf_st_quad(fin[m], orr, act ? (uint32_t)((16 * m + r) * ldv + (int64_t)h * a.dv + col0 + 4 * g) * (uint32_t)sizeof(E) : 0x80000000u);
        }
    };
    // the row of a finished token: 4 g .. of this wavefront's columns of token 16 m + r
    auto done = [&](const char* buf, int m, f32x4 x) {
        if constexpr (L::ROWS)
            *reinterpret_cast<typename A::Q4*>(const_cast<char*>(buf) + L::V_AT + ((16 * m + r) * L::VLD + w * 16 + 4 * g) * 2) = A::q4(x);
        else
            fin[m] = A::q4(x);
    };
    if (L::HAS_P) {   // the halves of P's blocks above the diagonal, which stay zero
        const f32x4 none = {0, 0, 0, 0};
        if (w == 0) A::put_half(pl, BWD ? upper_block(1, 0) : lower_block(0, 0), lane, BWD ? 0 : 1, none);
        if (w == 1) A::put_half(pl, BWD ? upper_block(3, 1) : lower_block(2, 1), lane, BWD ? 0 : 1, none);
    }
    if (nch > 0) {
        const Res rs = res_of(chunk_of(0));
        st.load_k(rs.k);
        st.load_q(rs.q);
        st.load_x(rs.x);
        st.load_v(rs.v);
        st.store(lds);
    }
    lds_barrier();
    // where this wavefront's columns are in a record; past its end where it has none
    const uint32_t w_off = act ? (uint32_t)(col0 / 32 * WSB) + rec_at(lane, (col0 >> 4) & 1) : 0x80000000u;
    const typename A::Ex pk0 = pick_half<E>(0, g, r), pk1 = pick_half<E>(1, g, r);
    for (int it = 0; it < nch; ++it) {
        const char* buf = lds + (L::BUFS == 2 ? (it & 1) * L::BYTES : 0);
        const int c = chunk_of(it);
        if ((MODE == FWD || MODE == BACK) && it > 0) flush(chunk_of(it - 1), lds + (L::BUFS == 2 ? ((it - 1) & 1) * L::BYTES : 0));
        const Res rs = res_of(chunk_of(it + 1 < nch ? it + 1 : it));   // the last chunk again rather than a branch
        st.load_k(rs.k);
        {
            const float *gam = reinterpret_cast<const float*>(buf + L::F_AT), *ob = gam + C;
            const f32x4 zero = {0, 0, 0, 0};
            const char* vl = buf + L::V_AT;
            if constexpr (L::HAS_P) {
                // P's ten tiles on the wavefronts in turn: of queries m and keys n, [s][t] (backwards
                // [t][s]), so that a lane has a quarter fragment
                const float* bt = gam + 3 * C;
                const double* G = reinterpret_cast<const double*>(gam + 4 * C);
                for (int i = w; i < 10; i += NW) {
                    const int m = i >= 6 ? 3 : i >= 3 ? 2 : i >= 1 ? 1 : 0, n = i - m * (m + 1) / 2;
                    f32x4 p = zero;
#pragma unroll
                    for (int b = 0; b < KB; ++b) {
                        const typename A::Ex kf = A::ld_ex(buf, n * KB + b, lane), qf = A::ld_ex(buf + L::Q_AT, m * KB + b, lane);
                        p = BWD ? A::mma(qf, kf, p) : A::mma(kf, qf, p);
                    }
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int t = BWD ? 16 * m + 4 * g + j : 16 * m + r, s = BWD ? 16 * n + r : 16 * n + 4 * g + j;
                        const float d = __builtin_amdgcn_exp2f(s <= t ? (float)(G[t] - G[s]) : 0.0f);
                        p[j] = s <= t ? a.scale * d * bt[s] * p[j] : 0.0f;
                    }
                    A::put_half(pl, BWD ? upper_block(n, m >> 1) : lower_block(m, n >> 1), lane, BWD ? m & 1 : n & 1, p);
                }
                if (BWD) lds_barrier();
            }
            typename A::Sp sb[NC][KB];
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int b = 0; b < KB; ++b) sb[j][b] = A::split(S[j][2 * b], S[j][2 * b + 1]);
            const int64_t rec = ((int64_t)pc.slot + c) * a.Hv + h;
            if constexpr (MODE == SAVE || MODE == BACK) {
                const Rsrc to = make_rsrc(io.recs + rec * rec_bytes(DK, a.dv) + (BWD ? state_bytes(DK, a.dv) : 0), (uint32_t)state_bytes(DK, a.dv));
#pragma unroll
                for (int b = 0; b < KB; ++b)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) A::put_t(to, w_off + (uint32_t)((2 * b + hh) * (a.dv / 32) * WSB), sb[0][b], hh ? pk1 : pk0);
            }
            f32x4 y[NC][MT], dov[MT];
            typename A::Ex dob[2];
            if constexpr (BWD) {
#pragma unroll
                for (int m = 0; m < MT; ++m) dov[m] = A::ld_col(vl, L::VLD, m, w * 16, g, r);
#pragma unroll
                for (int b = 0; b < 2; ++b) dob[b] = A::cols(dov[2 * b], dov[2 * b + 1]);
            }
            st.load_q(rs.q);
            __builtin_amdgcn_sched_barrier(0x1 | 0x2 | 0x4 | 0x8 | 0x100 | 0x200);
            // V - gam (K S), or om beta (K dS) + P^T dO
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int m = 0; m < MT; ++m) y[j][m] = zero;
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                typename A::Ex kf[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) kf[m] = A::ld_ex(buf, m * KB + b, lane);
#pragma unroll
                for (int j = 0; j < NC; ++j) A::mma_n(kf, sb[j][b], y[j]);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                if constexpr (BWD) {
                    y[0][m] *= ld4(ob + 16 * m + 4 * g);
                } else {
                    const f32x4 gm = ld4(gam + 16 * m + 4 * g);
#pragma unroll
                    for (int j = 0; j < NC; ++j) {
                        f32x4 vv = A::ld_col(vl, L::VLD, m, (w * NC + j) * 16, g, r);
                        if (isM[j]) vv = zero;
                        y[j][m] = vv - gm * y[j][m];
                    }
                }
            }
            if constexpr (BWD) {
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int m = 0; m <= 2 * b + 1; ++m) y[0][m] = A::mma(A::ld_sp(pl, upper_block(m, b), lane), dob[b], y[0][m]);
            }
            st.load_v(rs.v);
            __builtin_amdgcn_sched_barrier(0x1 | 0x2 | 0x4 | 0x8 | 0x100 | 0x200);
            // e = X y, or Z = X^T y
            typename A::Sp yb[NC][2];
#pragma unroll
            for (int j = 0; j < NC; ++j) {
#pragma unroll
                for (int b = 0; b < 2; ++b) yb[j][b] = A::split(y[j][2 * b], y[j][2 * b + 1]);
#pragma unroll
                for (int m = 0; m < MT; ++m) y[j][m] = zero;
            }
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int m = BWD ? 0 : 2 * b; m < (BWD ? 2 * b + 2 : MT); ++m) {
                    const typename A::Sp xf = BWD ? A::ld_tri_t(buf + L::X_AT, m, b, g, r) : A::ld_sp(buf + L::X_AT, lower_block(m, b), lane);
#pragma unroll
                    for (int j = 0; j < NC; ++j) y[j][m] = A::mma(xf, yb[j][b], y[j][m]);
                }
            typename A::Sp eb[2], wb[NC][2], db[2];
            if constexpr (MODE != MAP && MODE != BMAP) {
#pragma unroll
                for (int b = 0; b < 2; ++b) eb[b] = A::split(y[0][2 * b], y[0][2 * b + 1]);
            }
            if constexpr (MODE == SAVE || MODE == BACK) {
                const Rsrc to = make_rsrc(io.recs + rec * rec_bytes(DK, a.dv) + 2 * state_bytes(DK, a.dv) + (BWD ? rows_bytes(a.dv) : 0),
                                          (uint32_t)rows_bytes(a.dv));
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const f32x4 z = A::put_t(to, w_off + (uint32_t)((2 * b + hh) * (a.dv / 32) * WSB), eb[b], hh ? pk1 : pk0);
                        if constexpr (MODE == BACK) done(buf, 2 * b + hh, z);
                    }
            }
            // om beta e, or -gam Z and scale gam dO, for the state
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const f32x4 f4 = ld4((BWD ? gam : ob) + 16 * m + 4 * g);
                if constexpr (BWD) {
                    y[0][m] *= -f4;
                    dov[m] *= f4 * a.scale;
                } else {
#pragma unroll
                    for (int j = 0; j < NC; ++j) y[j][m] *= f4;
                }
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
#pragma unroll
                for (int j = 0; j < NC; ++j) wb[j][b] = A::split(y[j][2 * b], y[j][2 * b + 1]);
                if constexpr (BWD) db[b] = A::split(dov[2 * b], dov[2 * b + 1]);
            }
            st.load_x(rs.x);
            __builtin_amdgcn_sched_barrier(0x1 | 0x2 | 0x4 | 0x8 | 0x100 | 0x200);
            const float ge = gam[C - 1];
#pragma unroll
            for (int j = 0; j < NC; ++j)
#pragma unroll
                for (int t = 0; t < ST; ++t) S[j][t] *= ge;
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                typename A::Ex kt[ST];
                if constexpr (BWD) {
#pragma unroll
                    for (int t = 0; t < ST; ++t) kt[t] = A::template ld_ex_t<KB>(buf + L::Q_AT, t / 2, t & 1, tb, g, r);
                    A::mma_n(kt, db[tb], S[0]);
                }
#pragma unroll
                for (int t = 0; t < ST; ++t) kt[t] = A::template ld_ex_t<KB>(buf, t / 2, t & 1, tb, g, r);
#pragma unroll
                for (int j = 0; j < NC; ++j) A::mma_n(kt, wb[j][tb], S[j]);
            }
            if constexpr (MODE == FWD) {
                // O^T: lane (g, r) has columns 4 g.. of token r
                f32x4 ot[MT];
#pragma unroll
                for (int m = 0; m < MT; ++m) ot[m] = zero;
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    typename A::Ex qf[MT];
#pragma unroll
                    for (int m = 0; m < MT; ++m) qf[m] = A::ld_ex(buf + L::Q_AT, m * KB + b, lane);
                    A::mma_n(sb[0][b], qf, ot);
                }
#pragma unroll
                for (int m = 0; m < MT; ++m) ot[m] *= a.scale * gam[16 * m + r];
                lds_barrier();   // every tile of P is there
#pragma unroll
                for (int b = 0; b < 2; ++b)
#pragma unroll
                    for (int m = 2 * b; m < MT; ++m) ot[m] = A::mma(eb[b], A::ld_sp(pl, lower_block(m, b), lane), ot[m]);
#pragma unroll
                for (int m = 0; m < MT; ++m) done(buf, m, ot[m]);
            }
        }
        if constexpr (L::BUFS == 1) lds_barrier();
        st.store(lds + (L::BUFS == 2 ? ((it + 1) & 1) * L::BYTES : 0));
        lds_barrier();
    }
    if ((MODE == FWD || MODE == BACK) && nch > 0) flush(chunk_of(nch - 1), lds + (L::BUFS == 2 ? ((nch - 1) & 1) * L::BYTES : 0));
    // the state behind the piece
    float* to = nullptr;
    int64_t ld = a.dv;
    if (MODE == MAP || MODE == BMAP) {
        ld = ncols;
        to = io.maps + ((int64_t)pc.at * a.Hv + h) * DK * ld;
    } else if (io.last && (BWD ? pc.i == 0 : pc.i + 1 == pc.cnt)) {
        to = io.last + ((int64_t)pc.n * a.Hv + h) * DK * ld;
    }
#pragma unroll
    for (int j = 0; j < NC; ++j)
        if (to && on[j])
#pragma unroll
            for (int t = 0; t < ST; ++t)
#pragma unroll
                for (int i = 0; i < 4; ++i) to[(32 * (t / 2) + 8 * g + 4 * (t & 1) + i) * ld + col0 + 16 * j + r] = S[j][t][i];
}

template <typename E, int DK, int NW, int MODE, int NC>
__global__ void __launch_bounds__(64 * NW, NW / 4)
chain_kernel(Args a, Segs sg, Ptrs io) {
    __shared__ alignas(16) char lds[Lay<E, DK, NW, MODE, NC>::ALL];
    walk<E, DK, NW, MODE, NC>(a, sg, io, blockIdx.x, lds);
}

// Two walks in one launch, the longer one's workgroups first: the backward pass walks each way
// once, neither needs the other, and each alone leaves compute units idle where there are
// fewer than 256 workgroups (8 sequences of 4,096 tokens, 16 heads of 128 x 128 in bf16: 880-900 us together in
// workgroups of eight wavefronts; the whole call 1,660 us, in workgroups of four 1,700).
template <typename E, int DK, int NW, int BACKWARDS, int FORWARDS>
__global__ void __launch_bounds__(64 * NW, NW / 4)
pair_kernel(Args a, Segs sg, Ptrs back, Ptrs forth, unsigned nback) {
    constexpr int B = Lay<E, DK, NW, BACKWARDS, 1>::ALL, F = Lay<E, DK, NW, FORWARDS, 1>::ALL;
    __shared__ alignas(16) char lds[B > F ? B : F];
    if (blockIdx.x < nback) walk<E, DK, NW, BACKWARDS, 1>(a, sg, back, blockIdx.x, lds);
    else walk<E, DK, NW, FORWARDS, 1>(a, sg, forth, blockIdx.x - nback, lds);
}

// Joins the maps of a cut sequence's pieces: forwards X_0 = S0, X_{i+1} = M_i X_i + N_i, backwards
// X_last = dS_T, X_{i-1} = M_i^T X_i + N'_i, every X_i written to `starts`.  A workgroup has one
// head and 16 columns, a wavefront one tile of rows; X goes from step to step through LDS as
// fragments, the next step's M and N are in flight meanwhile.  On the fp32 matrix cores whatever the
// storage: M and X come as fp32 values, and nothing is split on the way.  Bound by a step's way through L2:
// 2.6 us; 16 pieces of 16 heads, 128 x 128: 42 us, with 32 columns a workgroup 70.
template <int DK, bool BWD>
__device__ __forceinline__ void join(const Args& a, const Segs& sg, const float* __restrict__ init, const float* __restrict__ maps,
                                     const float* __restrict__ nmaps, float* __restrict__ starts, char (&lds)[2][DK / 32 * WSB]) {
    typedef Arith<float> A;
    constexpr int KB = DK / 32, ST = DK / 16;
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nslab = a.dv / 16;
    const int slab = (int)(blockIdx.x % (unsigned)nslab), h = (int)(blockIdx.x / (unsigned)nslab % (unsigned)a.Hv);
    int n = (int)(blockIdx.x / (unsigned)nslab / (unsigned)a.Hv);
    if (sg.apart) {   // the cut sequence whose first piece is at place 2 n
        const Unit u = cut_unit_at(a, sg, 2 * n, lane);
        if (u.n < 0 || u.i != 0) return;
        n = u.n;
    }
    const int nch = (int)(((int64_t)seq_of(a, n).len + C - 1) / C);
    if (!is_cut(a, sg, nch, lane)) return;
    const int p0 = __builtin_amdgcn_readfirstlane(first_piece(a, sg, n)), cnt = (nch + sg.seg - 1) / sg.seg;
    const int col = 16 * slab + r;
    const bool on = w < ST;
    const int t = on ? w : 0;   // wavefronts past the rows work on the first tile and store nothing
    const int64_t mld = a.dv + DK, nld = BWD ? a.dv : mld;
    f32x4 X, N, M[KB][2];
    const int row0 = 32 * (t / 2) + 8 * g + 4 * (t & 1);                          // this lane's first row as a result
    const int rowa = 32 * (t / 2) + 8 * (r >> 2) + 4 * (t & 1) + (r & 3);         // and its row as an operand
    auto place = [&](int s) { return p0 + (BWD ? cnt - 1 - s : s); };
    auto fetch = [&](int s) {
        const float* m = maps + ((int64_t)place(s) * a.Hv + h) * DK * mld + a.dv;
        const float* nn = nmaps + ((int64_t)place(s) * a.Hv + h) * DK * nld;
#pragma unroll
        for (int b = 0; b < KB; ++b)
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                if constexpr (BWD) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) M[b][q][i] = m[(int64_t)(32 * b + 8 * g + 4 * q + i) * mld + rowa];
                } else {
                    M[b][q] = ld4(m + rowa * mld + 32 * b + 8 * g + 4 * q);
                }
            }
#pragma unroll
        for (int i = 0; i < 4; ++i) N[i] = nn[(int64_t)(row0 + i) * nld + col];
    };
    fetch(0);
#pragma unroll
    for (int i = 0; i < 4; ++i) X[i] = init ? init[(((int64_t)n * a.Hv + h) * DK + row0 + i) * a.dv + col] : 0.0f;
    for (int s = 0; s < cnt; ++s) {
        float* to = starts + ((int64_t)place(s) * a.Hv + h) * DK * a.dv + col;
        char* buf = lds[s & 1];
        if (on) {
#pragma unroll
            for (int i = 0; i < 4; ++i) to[(int64_t)(row0 + i) * a.dv] = X[i];
            A::put_half(buf, t / 2, lane, t & 1, X);
        }
        if (s + 1 == cnt) break;
        typename A::Sp mf[KB];
        X = N;
#pragma unroll
        for (int b = 0; b < KB; ++b) mf[b] = A::split(M[b][0], M[b][1]);
        fetch(s + 2 < cnt ? s + 1 : s);
        lds_barrier();
#pragma unroll
        for (int b = 0; b < KB; ++b) X = A::mma(mf[b], A::ld_sp(buf, b, lane), X);
    }
}

// The backward pass joins both ways in one launch (blockIdx.y).
template <int DK>
__global__ void __launch_bounds__(512)
join_kernel(Args a, Segs sg, const float* init, const float* maps, float* starts, const float* dinit, const float* nmaps,
            float* dstarts) {
    __shared__ alignas(16) char lds[2][DK / 32 * WSB];
    if (blockIdx.y == 0) join<DK, false>(a, sg, init, maps, maps, starts, lds);
    else join<DK, true>(a, sg, dinit, maps, nmaps, dstarts, lds);
}

// Workgroups of a walk over `cols` columns: a multiple of eight.
int64_t groups_of(const Args& a, int places, int cols, int slab) {
    return ((int64_t)places * a.Hk + 7) / 8 * 8 * (a.Hv / a.Hk) * ((cols + slab - 1) / slab);
}

// Places of a launch: the maps' is over the pieces alone.
int places_for(const Args& a, const Segs& sg, bool maps) {
    return (int)(maps ? pieces_of(a.nseq, a.T, a.cu != nullptr, sg) : walk_places(a.nseq, a.T, a.cu != nullptr, sg));
}

// Whether sequences are cut, and pieces times heads to expect.  The lengths of packed sequences
// are not known here: as if all were equal.
bool cut_of(const Args& a, const Segs& sg) {
    return sg.seg && places_of(a.nseq, a.T, a.cu != nullptr, C) / a.nseq > sg.over;
}
int64_t walks_of(const Args& a, const Segs& sg) {
    return (cut_of(a, sg) ? places_of(a.nseq, a.T, a.cu != nullptr, seg_unit(sg)) : a.nseq) * a.Hv;
}
// Wavefronts a workgroup: eight share one set of operands over 128 columns; four where a
// head has no more columns, or where workgroups of eight would leave half the chip empty.
// `slabs` of 64 columns a head.
bool wide(const Args& a, const Segs& sg, int slabs) { return walks_of(a, sg) * slabs > 256; }

template <typename E, int DK, int NW, int MODE, int NC>
hipError_t one_t(const Args& a, const Segs& sg, const Ptrs& io, int cols, hipStream_t stream) {
    hipLaunchKernelGGL((chain_kernel<E, DK, NW, MODE, NC>), dim3((unsigned)groups_of(a, io.places, cols, 16 * NC * NW)), dim3(64 * NW), 0,
                       stream, a, sg, io);
    return hipGetLastError();
}

template <typename E, int DK, int MODE>
hipError_t one_d(const Args& a, const Segs& sg, Ptrs io, hipStream_t stream) {
    const int cols = MODE == MAP ? a.dv + DK : a.dv;
    io.places = places_for(a, sg, MODE == MAP);
    if constexpr (sizeof(E) == 2) {
        // Two column tiles a wavefront read every operand once for both, in 8 us a chunk against 4.4:
        // where workgroups of 128 columns would take a second round (65,536 tokens of 16 heads, the
        // whole call: 1,165 us against 1,220; ten packed sequences with 128 workgroups of 256 columns: 411 against 340).
        if constexpr (MODE == MAP)
            if (cols > 128 && cut_of(a, sg) && walks_of(a, sg) * ((cols + 127) / 128) > 256)
                return one_t<E, DK, 8, MODE, 2>(a, sg, io, cols, stream);
        if (cols > 64 && wide(a, sg, (cols + 63) / 64)) return one_t<E, DK, 8, MODE, 1>(a, sg, io, cols, stream);
    }
    return one_t<E, DK, 4, MODE, 1>(a, sg, io, cols, stream);
}

template <typename E, int DK, int NW, int BACKWARDS, int FORWARDS>
hipError_t pair_t(const Args& a, const Segs& sg, const Ptrs& back, const Ptrs& forth, int fcols, hipStream_t stream) {
    const int64_t nback = groups_of(a, back.places, a.dv, 16 * NW), nforth = groups_of(a, back.places, fcols, 16 * NW);
    hipLaunchKernelGGL((pair_kernel<E, DK, NW, BACKWARDS, FORWARDS>), dim3((unsigned)(nback + nforth)), dim3(64 * NW), 0, stream, a,
                       sg, back, forth, (unsigned)nback);
    return hipGetLastError();
}

template <typename E, int DK, int BACKWARDS, int FORWARDS>
hipError_t pair_d(const Args& a, const Segs& sg, Ptrs back, Ptrs forth, hipStream_t stream) {
    const int fcols = FORWARDS == MAP ? a.dv + DK : a.dv;
    back.places = forth.places = places_for(a, sg, BACKWARDS == BMAP);
    if constexpr (sizeof(E) == 2)
        if (a.dv > 64 && wide(a, sg, (a.dv + 63) / 64 + (fcols + 63) / 64))
            return pair_t<E, DK, 8, BACKWARDS, FORWARDS>(a, sg, back, forth, fcols, stream);
    return pair_t<E, DK, 4, BACKWARDS, FORWARDS>(a, sg, back, forth, fcols, stream);
}

template <typename E, int DK>
hipError_t fwd_d(const Args& a, const Segs& sg, const Ptrs& io, hipStream_t stream) {
    return one_d<E, DK, FWD>(a, sg, io, stream);
}
template <typename E, int DK>
hipError_t map_d(const Args& a, const Segs& sg, const Ptrs& io, hipStream_t stream) {
    return one_d<E, DK, MAP>(a, sg, io, stream);
}
template <typename E, int DK>
hipError_t grads_d(bool maps, const Args& a, const Segs& sg, const Ptrs& back, const Ptrs& forth, hipStream_t stream) {
    return maps ? pair_d<E, DK, BMAP, MAP>(a, sg, back, forth, stream) : pair_d<E, DK, BACK, SAVE>(a, sg, back, forth, stream);
}

template <int DK>
hipError_t join_d(const Args& a, const Segs& sg, const float* init, const float* maps, float* starts, const float* dinit,
                  const float* nmaps, float* dstarts, hipStream_t stream) {
    const dim3 grid((unsigned)(joins_of(a.nseq, a.T, sg) * a.Hv * (a.dv / 16)), nmaps ? 2 : 1);
    hipLaunchKernelGGL((join_kernel<DK>), grid, dim3(512), 0, stream, a, sg, init, maps, starts, dinit, nmaps, dstarts);
    return hipGetLastError();
}

#define KDA_GDR_TYPES(F, ...)                                \
    if (f32) {                                               \
        switch (dk) {                                        \
            case 32: return F<float, 32>(__VA_ARGS__);       \
            case 64: return F<float, 64>(__VA_ARGS__);       \
            case 128: return F<float, 128>(__VA_ARGS__);     \
        }                                                    \
    } else {                                                 \
        switch (dk) {                                        \
            case 32: return F<bf16, 32>(__VA_ARGS__);        \
            case 64: return F<bf16, 64>(__VA_ARGS__);        \
            case 128: return F<bf16, 128>(__VA_ARGS__);      \
        }                                                    \
    }                                                        \
    return hipErrorInvalidValue

}  // namespace

hipError_t launch_fwd_chain(bool f32, int dk, const Args& a, const Segs& sg, const void* q, const void* k, const void* v,
                            const float* S0, const float* starts, const char* prep, void* o, float* S_T, hipStream_t stream) {
    const Ptrs io{q, k, v, S0, starts, prep, o, S_T, nullptr, nullptr, false, 0};
    KDA_GDR_TYPES(fwd_d, a, sg, io, stream);
}

hipError_t launch_maps(bool f32, int dk, const Args& a, const Segs& sg, const void* k, const void* v, const char* prep,
                       float* maps, hipStream_t stream) {
    const Ptrs io{k, k, v, nullptr, nullptr, prep, nullptr, nullptr, nullptr, maps, false, 0};
    KDA_GDR_TYPES(map_d, a, sg, io, stream);
}

hipError_t launch_bwd_maps(bool f32, int dk, const Args& a, const Segs& sg, const void* q, const void* k, const void* v,
                           const void* dout, const char* prep, float* maps, float* nmaps, hipStream_t stream) {
    const Ptrs back{q, k, dout, nullptr, nullptr, prep, nullptr, nullptr, nullptr, nmaps, false, 0};
    const Ptrs forth{k, k, v, nullptr, nullptr, prep, nullptr, nullptr, nullptr, maps, true, 0};
    KDA_GDR_TYPES(grads_d, true, a, sg, back, forth, stream);
}

hipError_t launch_bwd_chains(bool f32, int dk, const Args& a, const Segs& sg, const void* q, const void* k, const void* v,
                             const void* dout, const float* S0, const float* starts, const float* dS_T, const float* dstarts,
                             const char* prep, void* dv, float* dS0, char* recs, hipStream_t stream) {
    const Ptrs back{q, k, dout, dS_T, dstarts, prep, dv, dS0, recs, nullptr, false, 0};
    const Ptrs forth{k, k, v, S0, starts, prep, nullptr, nullptr, recs, nullptr, false, 0};
    KDA_GDR_TYPES(grads_d, false, a, sg, back, forth, stream);
}

hipError_t launch_join(int dk, const Args& a, const Segs& sg, const float* init, const float* maps, float* starts,
                       const float* dinit, const float* nmaps, float* dstarts, hipStream_t stream) {
    switch (dk) {
        case 32: return join_d<32>(a, sg, init, maps, starts, dinit, nmaps, dstarts, stream);
        case 64: return join_d<64>(a, sg, init, maps, starts, dinit, nmaps, dstarts, stream);
        case 128: return join_d<128>(a, sg, init, maps, starts, dinit, nmaps, dstarts, stream);
    }
    return hipErrorInvalidValue;
}

}  // namespace gdr
}  // namespace kda
