// kda_gdr_chain.hip -- the chunked gated delta rule's walk over a sequence's chunks: the
// states forwards (with the outputs, or saving each chunk's start state for the backward
// pass), and the states' gradients backwards.  Mathematics, precision and layouts: kda_gdr.hpp.
//
// Columns of the state (dv) are independent.  A workgroup of four wavefronts has one head
// of one sequence and 64 NTL columns, a wavefront 16 NTL of them: its slice of the state
// stays in fp32 accumulators for the whole walk, and every product of a chunk takes its
// result straight from the one before it (an accumulator tile is a B operand; read as an A
// operand it is its transpose), so the wavefronts share nothing but the chunk's operands.
// Those lie in LDS as fragment blocks: bf16 double-buffered, the next chunk's loads in
// flight in registers under this chunk's products, one barrier a chunk.
//   forwards:   Y = V - gam (K S);  e = X Y;  O^T = scale gam (S^T Q^T) + U^T P^T, U = beta e;
//               S <- gam_end S + K^T (om U)
//   backwards:  dU = om (K dS) + P^T dO;  Z = X^T (beta dU);
//               dS <- gam_end dS + Q^T (scale gam dO) - K^T (gam Z)
// K^T and Q^T are read from the same blocks as K and Q with the transposing LDS read.
#include "kda_gdr.hpp"
#include "kda_launch.hpp"

namespace kda {
namespace gdr {

namespace {

constexpr int NW = 4;                 // wavefronts a workgroup
constexpr int NTHR = 64 * NW;

enum Mode { FWD, SAVE, BACK };

// LDS of one buffer, and the 16-byte pieces a thread loads of each part.
template <typename E, int DK, int NTL, int MODE>
struct Lay {
    static constexpr int KB = DK / 32;
    static constexpr int SLAB = 16 * NTL * NW;
    static constexpr int QK = MT * KB * Arith<E>::EXB;         // K or Q
    static constexpr bool HAS_Q = MODE != SAVE, HAS_P = MODE != SAVE;
    static constexpr int Q_AT = QK, X_AT = Q_AT + (HAS_Q ? QK : 0), P_AT = X_AT + TRI_BYTES,
                         V_AT = P_AT + (HAS_P ? TRI_BYTES : 0), VB = C * SLAB * (int)sizeof(E), F_AT = V_AT + VB,
                         BYTES = F_AT + 3 * C * 4;
    static constexpr int BUFS = 2 * BYTES <= 160 * 1024 ? 2 : 1;
    static constexpr int NQK = QK / (16 * NTHR) ? QK / (16 * NTHR) : 1, NTRI = TRI_BYTES / (16 * NTHR),
                         NV = VB / (16 * NTHR) ? VB / (16 * NTHR) : 1;
};

// One chunk's operands on their way from global memory to LDS.
template <typename E, int DK, int NTL, int MODE>
struct Stage {
    typedef Lay<E, DK, NTL, MODE> L;
    u32x4 k[L::NQK], q[L::NQK], x[L::NTRI], p[L::NTRI], v[L::NV];
    float f;

    // piece u of a K or Q block set: row and channel it starts at
    static __device__ __forceinline__ void place(int u, int& row, int& ch) {
        const int lane = u & 63, g = lane >> 4, r = lane & 15;
        int blk, half = 0;
        if constexpr (sizeof(E) == 2) {
            blk = u >> 6;
        } else {
            blk = u >> 7;
            half = (u >> 6) & 1;
        }
        row = 16 * (blk / L::KB) + r;
        ch = 32 * (blk % L::KB) + 8 * g + 4 * half;
    }

    // kq: rows of the key head; vv: rows of the value head from the slab's first column, ncol
    // of them; pre: the chunk's X (or its transpose); preP: P (or its transpose); gm: gam, om
    __device__ __forceinline__ void load(const E* kk, const E* qq, int64_t ldk, const E* vv, int64_t ldv, int ncol,
                                         const float* bt, int ldb, const char* pre, const char* preP, const float* gm,
                                         int valid) {
        const int tid = threadIdx.x;
#pragma unroll
        for (int j = 0; j < L::NQK; ++j) {
            int row, ch;
            place((tid + j * NTHR) % (L::QK / 16), row, ch);
            row = row < valid ? row : valid - 1;
            k[j] = *reinterpret_cast<const u32x4*>(kk + row * ldk + ch);
            if constexpr (L::HAS_Q) q[j] = *reinterpret_cast<const u32x4*>(qq + row * ldk + ch);
        }
#pragma unroll
        for (int j = 0; j < L::NTRI; ++j) {
            x[j] = *reinterpret_cast<const u32x4*>(pre + (tid + j * NTHR) * 16);
            if constexpr (L::HAS_P) p[j] = *reinterpret_cast<const u32x4*>(preP + (tid + j * NTHR) * 16);
        }
        constexpr int EPP = 16 / (int)sizeof(E), PPR = L::SLAB / EPP;   // elements a piece, pieces a row
#pragma unroll
        for (int j = 0; j < L::NV; ++j) {
            const int u = (tid + j * NTHR) % (C * PPR);
            int row = u / PPR, col = (u % PPR) * EPP;
            col = col < ncol ? col : 0;   // columns past the head's end are not used
            const bool in = row < valid;
            row = in ? row : valid - 1;
            v[j] = *reinterpret_cast<const u32x4*>(vv + row * ldv + col);
            if (MODE == BACK && !in) v[j] = u32x4{0, 0, 0, 0};   // no gradient past the end
        }
        f = 0.0f;
        if (tid < 2 * C) f = gm[tid];
        else if (tid < 3 * C && tid - 2 * C < valid) f = bt[(int64_t)(tid - 2 * C) * ldb];
    }

    __device__ __forceinline__ void store(char* buf) const {
        const int tid = threadIdx.x;
#pragma unroll
        for (int j = 0; j < L::NQK; ++j) {
            const int u = tid + j * NTHR;
            if (L::QK / 16 >= NTHR || u < L::QK / 16) {
                *reinterpret_cast<u32x4*>(buf + u * 16) = k[j];
                if constexpr (L::HAS_Q) *reinterpret_cast<u32x4*>(buf + L::Q_AT + u * 16) = q[j];
            }
        }
#pragma unroll
        for (int j = 0; j < L::NTRI; ++j) {
            *reinterpret_cast<u32x4*>(buf + L::X_AT + (tid + j * NTHR) * 16) = x[j];
            if constexpr (L::HAS_P) *reinterpret_cast<u32x4*>(buf + L::P_AT + (tid + j * NTHR) * 16) = p[j];
        }
#pragma unroll
        for (int j = 0; j < L::NV; ++j) *reinterpret_cast<u32x4*>(buf + L::V_AT + (tid + j * NTHR) * 16) = v[j];
        if (tid < 3 * C) reinterpret_cast<float*>(buf + L::F_AT)[tid] = f;
    }
};

__device__ __forceinline__ f32x4 ld4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

// Forwards.  SAVE writes no output but, per chunk, the start state and e as the gradient
// kernel's operands.  S0 and S_T may be NULL.
template <typename E, int DK, int NTL, int MODE>
__global__ void __launch_bounds__(NTHR, 1)
chain_kernel(Args a, const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ v,
             const float* __restrict__ beta, const float* S0, const char* __restrict__ prep, int64_t prep_stride,
             E* __restrict__ o, float* S_T, char* __restrict__ ws_s, char* __restrict__ ws_e) {
    typedef Arith<E> A;
    typedef Lay<E, DK, NTL, MODE> L;
    constexpr int KB = L::KB, ST = DK / 16;
    __shared__ alignas(16) char lds[L::BUFS * L::BYTES];
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nslab = (a.dv + L::SLAB - 1) / L::SLAB;
    const int slab = (int)(blockIdx.x % (unsigned)nslab);
    const int h = (int)(blockIdx.x / (unsigned)nslab % (unsigned)a.Hv);
    const int n = (int)(blockIdx.x / (unsigned)nslab / (unsigned)a.Hv);
    const Seq sq = seq_of(a, n);
    const int nch = (sq.len + C - 1) / C;
    const int hk = h / (a.Hv / a.Hk);
    const int64_t ldk = (int64_t)a.Hk * DK, ldv = (int64_t)a.Hv * a.dv;
    const int c0 = slab * L::SLAB, col0 = c0 + w * 16 * NTL;   // the slab's and the wavefront's first column
    const bool act = col0 < a.dv;
    const E* kp = k + sq.row0 * ldk + (int64_t)hk * DK;
    const E* qp = q + sq.row0 * ldk + (int64_t)hk * DK;
    const E* vp = v + sq.row0 * ldv + (int64_t)h * a.dv + c0;
    const float* bp = beta + sq.row0 * a.Hv + h;
    const int64_t sbase = ((int64_t)n * a.Hv + h) * DK * a.dv;

    f32x4 S[NTL][ST];
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int j = 0; j < NTL; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                S[j][t][i] = S0 && act ? S0[sbase + (int64_t)(32 * (t / 2) + 8 * g + 4 * (t & 1) + i) * a.dv + col0 + 16 * j + r] : 0.0f;

    Stage<E, DK, NTL, MODE> st;
    auto load = [&](int c) {
        const int left = sq.len - c * C;
        const char* pre = prep + (((int64_t)sq.slot + c) * a.Hv + h) * prep_stride;
        st.load(kp + (int64_t)c * C * ldk, qp + (int64_t)c * C * ldk, ldk, vp + (int64_t)c * C * ldv, ldv, a.dv - c0,
                bp + (int64_t)c * C * a.Hv, a.Hv, pre, pre + TRI_BYTES,
                reinterpret_cast<const float*>(pre + prep_stride - 2 * C * 4), left < C ? left : C);
    };
    if (nch > 0) {
        load(0);
        st.store(lds);
    }
    lds_barrier();
    for (int c = 0; c < nch; ++c) {
        const char* buf = lds + (L::BUFS == 2 ? (c & 1) * L::BYTES : 0);
        load(c + 1 < nch ? c + 1 : c);   // the last chunk again rather than a branch
        if (act) {
            const float* gam = reinterpret_cast<const float*>(buf + L::F_AT);
            const float *om = gam + C, *bt = gam + 2 * C;
            const f32x4 zero = {0, 0, 0, 0};
            typename A::Sp sb[NTL][KB];
#pragma unroll
            for (int j = 0; j < NTL; ++j)
#pragma unroll
                for (int b = 0; b < KB; ++b) sb[j][b] = A::split(S[j][2 * b], S[j][2 * b + 1]);
            if constexpr (MODE == SAVE) {
                char* to = ws_s + (((int64_t)sq.slot + c) * a.Hv + h) * state_bytes(DK, a.dv);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const typename A::Ex pk = pick_half<E>(hh, g, r);
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int j = 0; j < NTL; ++j) {
                            const int ct = col0 / 16 + j;
                            A::put_t(to + ((int64_t)(2 * b + hh) * (a.dv / 32) + ct / 2) * SPB, lane, ct & 1, sb[j][b], pk);
                        }
                }
            }
            // Y = V - gam (K S)
            f32x4 y[NTL][MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int j = 0; j < NTL; ++j) y[j][m] = zero;
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    const typename A::Ex kf = A::ld_ex(buf, m * KB + b, lane);
#pragma unroll
                    for (int j = 0; j < NTL; ++j) y[j][m] = A::mma(kf, sb[j][b], y[j][m]);
                }
                const f32x4 gm = ld4(gam + 16 * m + 4 * g);
#pragma unroll
                for (int j = 0; j < NTL; ++j) {
                    const f32x4 vv = A::ld_col(buf + L::V_AT, L::SLAB, m, w * 16 * NTL + 16 * j, g, r);
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[j][m][i] = vv[i] - gm[i] * y[j][m][i];
                }
            }
            // e = X Y; U = beta e, and om U for the state
            typename A::Sp yb[NTL][2], ub[NTL][2], wb[NTL][2];
#pragma unroll
            for (int j = 0; j < NTL; ++j)
#pragma unroll
                for (int b = 0; b < 2; ++b) yb[j][b] = A::split(y[j][2 * b], y[j][2 * b + 1]);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int j = 0; j < NTL; ++j) y[j][m] = zero;
#pragma unroll
                for (int b = 0; b <= m / 2; ++b) {
                    const typename A::Sp xf = A::ld_sp(buf + L::X_AT, lower_block(m, b), lane);
#pragma unroll
                    for (int j = 0; j < NTL; ++j) y[j][m] = A::mma(xf, yb[j][b], y[j][m]);
                }
            }
            if constexpr (MODE == SAVE) {
                char* to = ws_e + (((int64_t)sq.slot + c) * a.Hv + h) * rows_bytes(a.dv);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const typename A::Ex pk = pick_half<E>(hh, g, r);
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int j = 0; j < NTL; ++j) {
                            const int ct = col0 / 16 + j;
                            A::put_t(to + ((int64_t)(2 * b + hh) * (a.dv / 32) + ct / 2) * SPB, lane, ct & 1,
                                     A::split(y[j][2 * b], y[j][2 * b + 1]), pk);
                        }
                }
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const f32x4 b4 = ld4(bt + 16 * m + 4 * g);
#pragma unroll
                for (int j = 0; j < NTL; ++j) y[j][m] *= b4;
            }
            if constexpr (MODE == FWD) {
#pragma unroll
                for (int j = 0; j < NTL; ++j)
#pragma unroll
                    for (int b = 0; b < 2; ++b) ub[j][b] = A::split(y[j][2 * b], y[j][2 * b + 1]);
            }
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const f32x4 o4 = ld4(om + 16 * m + 4 * g);
#pragma unroll
                for (int j = 0; j < NTL; ++j) y[j][m] *= o4;
            }
#pragma unroll
            for (int j = 0; j < NTL; ++j)
#pragma unroll
                for (int b = 0; b < 2; ++b) wb[j][b] = A::split(y[j][2 * b], y[j][2 * b + 1]);
            // S <- gam_end S + K^T (om U)
            const float ge = gam[C - 1];
#pragma unroll
            for (int t = 0; t < ST; ++t) {
#pragma unroll
                for (int j = 0; j < NTL; ++j) S[j][t] *= ge;
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    const typename A::Ex kt = A::template ld_ex_t<KB>(buf, t / 2, t & 1, tb, g, r);
#pragma unroll
                    for (int j = 0; j < NTL; ++j) S[j][t] = A::mma(kt, wb[j][tb], S[j][t]);
                }
            }
            if constexpr (MODE == FWD) {
                // O^T = scale gam (S^T Q^T) + U^T P^T: lane (g, r) has columns 4 g.. of token r
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    f32x4 ot[NTL];
#pragma unroll
                    for (int j = 0; j < NTL; ++j) ot[j] = zero;
#pragma unroll
                    for (int b = 0; b < KB; ++b) {
                        const typename A::Ex qf = A::ld_ex(buf + L::Q_AT, m * KB + b, lane);
#pragma unroll
                        for (int j = 0; j < NTL; ++j) ot[j] = A::mma(sb[j][b], qf, ot[j]);
                    }
                    const float gs = a.scale * gam[16 * m + r];
#pragma unroll
                    for (int j = 0; j < NTL; ++j) ot[j] *= gs;
#pragma unroll
                    for (int b = 0; b <= m / 2; ++b) {
                        const typename A::Sp pf = A::ld_sp(buf + L::P_AT, lower_block(m, b), lane);
#pragma unroll
                        for (int j = 0; j < NTL; ++j) ot[j] = A::mma(ub[j][b], pf, ot[j]);
                    }
                    const int64_t tok = (int64_t)c * C + 16 * m + r;
                    if (tok < sq.len)
#pragma unroll
                        for (int j = 0; j < NTL; ++j)
                            A::st4(o + (sq.row0 + tok) * ldv + (int64_t)h * a.dv + col0 + 16 * j + 4 * g, ot[j]);
                }
            }
        }
        if constexpr (L::BUFS == 1) lds_barrier();
        st.store(lds + (L::BUFS == 2 ? ((c + 1) & 1) * L::BYTES : 0));
        lds_barrier();
    }
    if (S_T && act)
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int j = 0; j < NTL; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    S_T[sbase + (int64_t)(32 * (t / 2) + 8 * g + 4 * (t & 1) + i) * a.dv + col0 + 16 * j + r] = S[j][t][i];
}

// Backwards: per chunk, the states' gradient at its end and Z, as the gradient kernel's
// operands, and dV = Z; after the first chunk dS0.  dS_T and dS0 may be NULL.
template <typename E, int DK, int NTL>
__global__ void __launch_bounds__(NTHR, 1)
back_kernel(Args a, const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ dout,
            const float* __restrict__ beta, const float* dS_T, const char* __restrict__ prep, int64_t prep_stride,
            E* __restrict__ dv, float* dS0, char* __restrict__ ws_d, char* __restrict__ ws_z) {
    typedef Arith<E> A;
    typedef Lay<E, DK, NTL, BACK> L;
    constexpr int KB = L::KB, ST = DK / 16;
    __shared__ alignas(16) char lds[L::BUFS * L::BYTES];
    const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int nslab = (a.dv + L::SLAB - 1) / L::SLAB;
    const int slab = (int)(blockIdx.x % (unsigned)nslab);
    const int h = (int)(blockIdx.x / (unsigned)nslab % (unsigned)a.Hv);
    const int n = (int)(blockIdx.x / (unsigned)nslab / (unsigned)a.Hv);
    const Seq sq = seq_of(a, n);
    const int nch = (sq.len + C - 1) / C;
    const int hk = h / (a.Hv / a.Hk);
    const int64_t ldk = (int64_t)a.Hk * DK, ldv = (int64_t)a.Hv * a.dv;
    const int c0 = slab * L::SLAB, col0 = c0 + w * 16 * NTL;
    const bool act = col0 < a.dv;
    const E* kp = k + sq.row0 * ldk + (int64_t)hk * DK;
    const E* qp = q + sq.row0 * ldk + (int64_t)hk * DK;
    const E* dp = dout + sq.row0 * ldv + (int64_t)h * a.dv + c0;
    const float* bp = beta + sq.row0 * a.Hv + h;
    const int64_t sbase = ((int64_t)n * a.Hv + h) * DK * a.dv;

    f32x4 S[NTL][ST];
#pragma unroll
    for (int t = 0; t < ST; ++t)
#pragma unroll
        for (int j = 0; j < NTL; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                S[j][t][i] = dS_T && act ? dS_T[sbase + (int64_t)(32 * (t / 2) + 8 * g + 4 * (t & 1) + i) * a.dv + col0 + 16 * j + r] : 0.0f;

    Stage<E, DK, NTL, BACK> st;
    auto load = [&](int c) {
        const int left = sq.len - c * C;
        const char* pre = prep + (((int64_t)sq.slot + c) * a.Hv + h) * prep_stride;
        st.load(kp + (int64_t)c * C * ldk, qp + (int64_t)c * C * ldk, ldk, dp + (int64_t)c * C * ldv, ldv, a.dv - c0,
                bp + (int64_t)c * C * a.Hv, a.Hv, pre + 2 * TRI_BYTES, pre + 3 * TRI_BYTES,
                reinterpret_cast<const float*>(pre + prep_stride - 2 * C * 4), left < C ? left : C);
    };
    if (nch > 0) {
        load(nch - 1);
        st.store(lds);
    }
    lds_barrier();
    for (int it = 0; it < nch; ++it) {
        const int c = nch - 1 - it;
        const char* buf = lds + (L::BUFS == 2 ? (it & 1) * L::BYTES : 0);
        load(c > 0 ? c - 1 : 0);
        if (act) {
            const float* gam = reinterpret_cast<const float*>(buf + L::F_AT);
            const float *om = gam + C, *bt = gam + 2 * C;
            const f32x4 zero = {0, 0, 0, 0};
            typename A::Sp sb[NTL][KB];
#pragma unroll
            for (int j = 0; j < NTL; ++j)
#pragma unroll
                for (int b = 0; b < KB; ++b) sb[j][b] = A::split(S[j][2 * b], S[j][2 * b + 1]);
            {
                char* to = ws_d + (((int64_t)sq.slot + c) * a.Hv + h) * state_bytes(DK, a.dv);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const typename A::Ex pk = pick_half<E>(hh, g, r);
#pragma unroll
                    for (int b = 0; b < KB; ++b)
#pragma unroll
                        for (int j = 0; j < NTL; ++j) {
                            const int ct = col0 / 16 + j;
                            A::put_t(to + ((int64_t)(2 * b + hh) * (a.dv / 32) + ct / 2) * SPB, lane, ct & 1, sb[j][b], pk);
                        }
                }
            }
            // dO of this wavefront's columns
            f32x4 dov[NTL][MT];
            typename A::Ex dob[NTL][2];
#pragma unroll
            for (int j = 0; j < NTL; ++j) {
#pragma unroll
                for (int m = 0; m < MT; ++m) dov[j][m] = A::ld_col(buf + L::V_AT, L::SLAB, m, w * 16 * NTL + 16 * j, g, r);
#pragma unroll
                for (int b = 0; b < 2; ++b) dob[j][b] = A::cols(dov[j][2 * b], dov[j][2 * b + 1]);
            }
            // beta dU = beta (om (K dS) + P^T dO)
            f32x4 y[NTL][MT];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int j = 0; j < NTL; ++j) y[j][m] = zero;
#pragma unroll
                for (int b = 0; b < KB; ++b) {
                    const typename A::Ex kf = A::ld_ex(buf, m * KB + b, lane);
#pragma unroll
                    for (int j = 0; j < NTL; ++j) y[j][m] = A::mma(kf, sb[j][b], y[j][m]);
                }
                const f32x4 o4 = ld4(om + 16 * m + 4 * g), b4 = ld4(bt + 16 * m + 4 * g);
#pragma unroll
                for (int j = 0; j < NTL; ++j) y[j][m] *= o4;
#pragma unroll
                for (int b = m / 2; b < 2; ++b) {
                    const typename A::Sp pf = A::ld_sp(buf + L::P_AT, upper_block(m, b), lane);
#pragma unroll
                    for (int j = 0; j < NTL; ++j) y[j][m] = A::mma(pf, dob[j][b], y[j][m]);
                }
#pragma unroll
                for (int j = 0; j < NTL; ++j) y[j][m] *= b4;
            }
            // Z = X^T (beta dU)
            typename A::Sp yb[NTL][2];
#pragma unroll
            for (int j = 0; j < NTL; ++j)
#pragma unroll
                for (int b = 0; b < 2; ++b) yb[j][b] = A::split(y[j][2 * b], y[j][2 * b + 1]);
#pragma unroll
            for (int m = 0; m < MT; ++m) {
#pragma unroll
                for (int j = 0; j < NTL; ++j) y[j][m] = zero;
#pragma unroll
                for (int b = m / 2; b < 2; ++b) {
                    const typename A::Sp xf = A::ld_sp(buf + L::X_AT, upper_block(m, b), lane);
#pragma unroll
                    for (int j = 0; j < NTL; ++j) y[j][m] = A::mma(xf, yb[j][b], y[j][m]);
                }
            }
            {
                char* to = ws_z + (((int64_t)sq.slot + c) * a.Hv + h) * rows_bytes(a.dv);
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const typename A::Ex pk = pick_half<E>(hh, g, r);
#pragma unroll
                    for (int b = 0; b < 2; ++b)
#pragma unroll
                        for (int j = 0; j < NTL; ++j) {
                            const int ct = col0 / 16 + j;
                            const f32x4 z = A::put_t(to + ((int64_t)(2 * b + hh) * (a.dv / 32) + ct / 2) * SPB, lane, ct & 1,
                                                     A::split(y[j][2 * b], y[j][2 * b + 1]), pk);
                            const int64_t tok = (int64_t)c * C + 32 * b + 16 * hh + r;
                            if (tok < sq.len) A::st4(dv + (sq.row0 + tok) * ldv + (int64_t)h * a.dv + 16 * ct + 4 * g, z);
                        }
                }
            }
            // dS <- gam_end dS + Q^T (scale gam dO) - K^T (gam Z)
            typename A::Sp zb[NTL][2], db[NTL][2];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const f32x4 gm = ld4(gam + 16 * m + 4 * g);
#pragma unroll
                for (int j = 0; j < NTL; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        y[j][m][i] *= -gm[i];
                        dov[j][m][i] *= a.scale * gm[i];
                    }
            }
#pragma unroll
            for (int j = 0; j < NTL; ++j)
#pragma unroll
                for (int b = 0; b < 2; ++b) {
                    zb[j][b] = A::split(y[j][2 * b], y[j][2 * b + 1]);
                    db[j][b] = A::split(dov[j][2 * b], dov[j][2 * b + 1]);
                }
            const float ge = gam[C - 1];
#pragma unroll
            for (int t = 0; t < ST; ++t) {
#pragma unroll
                for (int j = 0; j < NTL; ++j) S[j][t] *= ge;
#pragma unroll
                for (int tb = 0; tb < 2; ++tb) {
                    const typename A::Ex kt = A::template ld_ex_t<KB>(buf, t / 2, t & 1, tb, g, r);
                    const typename A::Ex qt = A::template ld_ex_t<KB>(buf + L::Q_AT, t / 2, t & 1, tb, g, r);
#pragma unroll
                    for (int j = 0; j < NTL; ++j) {
                        S[j][t] = A::mma(qt, db[j][tb], S[j][t]);
                        S[j][t] = A::mma(kt, zb[j][tb], S[j][t]);
                    }
                }
            }
        }
        if constexpr (L::BUFS == 1) lds_barrier();
        st.store(lds + (L::BUFS == 2 ? ((it + 1) & 1) * L::BYTES : 0));
        lds_barrier();
    }
    if (dS0 && act)
#pragma unroll
        for (int t = 0; t < ST; ++t)
#pragma unroll
            for (int j = 0; j < NTL; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dS0[sbase + (int64_t)(32 * (t / 2) + 8 * g + 4 * (t & 1) + i) * a.dv + col0 + 16 * j + r] = S[j][t][i];
}

template <int NTL>
unsigned chain_grid(const Args& a) {
    const int slab = 16 * NTL * NW;
    return (unsigned)((int64_t)a.nseq * a.Hv * ((a.dv + slab - 1) / slab));
}

// Two column tiles a wavefront share each operand fragment's LDS read, one leaves twice the
// workgroups: two where the workgroups then still fill the chip.
bool wide(bool f32, const Args& a) { return !f32 && (int64_t)a.nseq * a.Hv * ((a.dv + 127) / 128) >= 256 && a.dv % 128 == 0; }

template <typename E, int DK, int NTL>
hipError_t fwd_t(bool save, const Args& a, const void* q, const void* k, const void* v, const float* beta, const float* S0,
                 const char* prep, int64_t stride, void* o, float* S_T, char* ws_s, char* ws_e, hipStream_t stream) {
    const dim3 grid(chain_grid<NTL>(a));
    if (save)
        hipLaunchKernelGGL((chain_kernel<E, DK, NTL, SAVE>), grid, dim3(NTHR), 0, stream, a, (const E*)q, (const E*)k,
                           (const E*)v, beta, S0, prep, stride, (E*)o, S_T, ws_s, ws_e);
    else
        hipLaunchKernelGGL((chain_kernel<E, DK, NTL, FWD>), grid, dim3(NTHR), 0, stream, a, (const E*)q, (const E*)k,
                           (const E*)v, beta, S0, prep, stride, (E*)o, S_T, ws_s, ws_e);
    return hipGetLastError();
}

template <typename E, int DK, int NTL>
hipError_t back_t(const Args& a, const void* q, const void* k, const void* dout, const float* beta, const float* dS_T,
                  const char* prep, int64_t stride, void* dv, float* dS0, char* ws_d, char* ws_z, hipStream_t stream) {
    hipLaunchKernelGGL((back_kernel<E, DK, NTL>), dim3(chain_grid<NTL>(a)), dim3(NTHR), 0, stream, a, (const E*)q, (const E*)k,
                       (const E*)dout, beta, dS_T, prep, stride, (E*)dv, dS0, ws_d, ws_z);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_chain(bool f32, int dk, bool save, const Args& a, const void* q, const void* k, const void* v,
                        const float* beta, const float* S0, const char* prep, int64_t stride, void* o, float* S_T,
                        char* ws_s, char* ws_e, hipStream_t stream) {
#define KDA_GC(E, D, N) return fwd_t<E, D, N>(save, a, q, k, v, beta, S0, prep, stride, o, S_T, ws_s, ws_e, stream)
    if (f32) {
        switch (dk) {
            case 32: KDA_GC(float, 32, 1);
            case 64: KDA_GC(float, 64, 1);
            case 128: KDA_GC(float, 128, 1);
        }
    } else if (wide(f32, a)) {
        switch (dk) {
            case 32: KDA_GC(bf16, 32, 2);
            case 64: KDA_GC(bf16, 64, 2);
            case 128: KDA_GC(bf16, 128, 2);
        }
    } else {
        switch (dk) {
            case 32: KDA_GC(bf16, 32, 1);
            case 64: KDA_GC(bf16, 64, 1);
            case 128: KDA_GC(bf16, 128, 1);
        }
    }
#undef KDA_GC
    return hipErrorInvalidValue;
}

hipError_t launch_back(bool f32, int dk, const Args& a, const void* q, const void* k, const void* dout, const float* beta,
                       const float* dS_T, const char* prep, int64_t stride, void* dv, float* dS0, char* ws_d, char* ws_z,
                       hipStream_t stream) {
#define KDA_GB(E, D, N) return back_t<E, D, N>(a, q, k, dout, beta, dS_T, prep, stride, dv, dS0, ws_d, ws_z, stream)
    if (f32) {
        switch (dk) {
            case 32: KDA_GB(float, 32, 1);
            case 64: KDA_GB(float, 64, 1);
            case 128: KDA_GB(float, 128, 1);
        }
    } else if (wide(f32, a)) {
        switch (dk) {
            case 32: KDA_GB(bf16, 32, 2);
            case 64: KDA_GB(bf16, 64, 2);
            case 128: KDA_GB(bf16, 128, 2);
        }
    } else {
        switch (dk) {
            case 32: KDA_GB(bf16, 32, 1);
            case 64: KDA_GB(bf16, 64, 1);
            case 128: KDA_GB(bf16, 128, 1);
        }
    }
#undef KDA_GB
    return hipErrorInvalidValue;
}

}  // namespace gdr
}  // namespace kda
