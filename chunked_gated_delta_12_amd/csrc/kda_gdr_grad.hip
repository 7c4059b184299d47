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
// One workgroup has one chunk of one key head and goes through its value heads, so the
// gradients of the shared q and k are summed in registers; wavefront w has token tile w, as
// columns: results are [channel][token], four channels of one token a lane, which is how
// they are stored, how the tokens' factors apply and what the dot products with q and k
// need.  It forms the rows of its tokens (s <= t) and their columns (t >= s), five of the
// four-by-four tiles for every wavefront.  dv is walked in blocks of 32 columns, the next
// block's operands in flight in registers.
#include "kda_gdr.hpp"
#include "kda_launch.hpp"

namespace kda {
namespace gdr {

namespace {

template <typename E, int DK>
struct GradLay {
    static constexpr int KB = DK / 32, ST = DK / 16, EXB = Arith<E>::EXB;
    static constexpr int QK = MT * KB * EXB;
    static constexpr int S_AT = 0, D_AT = ST * SPB, E_AT = 2 * ST * SPB, Z_AT = E_AT + MT * SPB, O_AT = Z_AT + MT * SPB,
                         STEP = O_AT + MT * EXB;
    static constexpr int FIX = 2 * QK + 4 * C * 4 + 2 * C * 8 + 16;   // K, Q, the tokens' values
    static constexpr int BUFS = FIX + 2 * STEP <= 160 * 1024 ? 2 : 1;
    static constexpr int NS = ST * SPB / 4096 ? ST * SPB / 4096 : 1;   // 16-byte pieces a thread of S and of dS
    static constexpr int NE = MT * SPB / 4096;                          // of e and of Z
    static constexpr int NO = MT * EXB / 4096;                          // of do
};

__device__ __forceinline__ float over_groups(float x) {
    x += __shfl_xor(x, 16);
    x += __shfl_xor(x, 32);
    return x;
}

template <typename E, int DK>
__global__ void __launch_bounds__(256, 1)
grad_kernel(Args a, const E* __restrict__ q, const E* __restrict__ k, const E* __restrict__ dout,
            const char* __restrict__ prep, const char* __restrict__ ws_s,
            const char* __restrict__ ws_e, const char* __restrict__ ws_d, const char* __restrict__ ws_z,
            E* __restrict__ dq, E* __restrict__ dk, float* __restrict__ dg, float* __restrict__ dbeta) {
    typedef Arith<E> A;
    typedef GradLay<E, DK> L;
    typedef typename A::Sp Sp;
    typedef typename A::Ex Ex;
    constexpr int KB = L::KB, ST = L::ST;
    __shared__ alignas(16) char kl[L::QK];
    __shared__ alignas(16) char ql[L::QK];
    __shared__ alignas(16) char lds[L::BUFS * L::STEP];
    __shared__ double Gs[C], dGs[C];
    __shared__ float gam[C], om[C], bts[C], kes[C], dots[4];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, r = lane & 15;
    const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int slot = (int)(blockIdx.x / (unsigned)a.Hk), hk = (int)(blockIdx.x % (unsigned)a.Hk);
    const Chunk ch = chunk_at(a, slot, lane);
    if (ch.n < 0) return;
    const int rep = a.Hv / a.Hk, nb = a.dv / 32;
    const int64_t ldk = (int64_t)a.Hk * DK, ldv = (int64_t)a.Hv * a.dv;
    const f32x4 zero = {0, 0, 0, 0};
    const int tok = 16 * w + r;   // this lane's token

    // K and Q as fragment blocks
    const E* kc = k + ch.row0 * ldk + hk * DK;
    const E* qc = q + ch.row0 * ldk + hk * DK;
#pragma unroll
    for (int j = 0; j < L::QK / 16; j += 256) {
        const int u = j + tid;
        const int l = u & 63, blk = sizeof(E) == 2 ? u >> 6 : u >> 7, half = sizeof(E) == 2 ? 0 : (u >> 6) & 1;
        int row = 16 * (blk / KB) + (l & 15);
        row = row < ch.valid ? row : ch.valid - 1;
        const int64_t at = row * ldk + 32 * (blk % KB) + 8 * (l >> 4) + 4 * half;
        const int to = ((u & ~63) + swz(l)) * 16;
        *reinterpret_cast<u32x4*>(kl + to) = *reinterpret_cast<const u32x4*>(kc + at);
        *reinterpret_cast<u32x4*>(ql + to) = *reinterpret_cast<const u32x4*>(qc + at);
    }

    // one 32-column block of one value head's operands
    u32x4 ss[L::NS], sd[L::NS], se[L::NE], sz[L::NE], so[L::NO];
    const E* dc = dout + ch.row0 * ldv;
    auto load = [&](int vh, int b) {
        const int64_t rec = (int64_t)slot * a.Hv + hk * rep + vh;
        const char* ps = ws_s + rec * state_bytes(DK, a.dv) + b * SPB;
        const char* pd = ws_d + rec * state_bytes(DK, a.dv) + b * SPB;
        const char* pe = ws_e + rec * rows_bytes(a.dv) + b * SPB;
        const char* pz = ws_z + rec * rows_bytes(a.dv) + b * SPB;
#pragma unroll
        for (int j = 0; j < L::NS; ++j) {   // 128 pieces a block
            const int u = tid + 256 * j;
            const int64_t at = (int64_t)(u >> 7) * nb * SPB + (u & 127) * 16;
            ss[j] = *reinterpret_cast<const u32x4*>(ps + at);
            sd[j] = *reinterpret_cast<const u32x4*>(pd + at);
        }
#pragma unroll
        for (int j = 0; j < L::NE; ++j) {
            const int u = tid + 256 * j;
            const int64_t at = (int64_t)(u >> 7) * nb * SPB + (u & 127) * 16;
            se[j] = *reinterpret_cast<const u32x4*>(pe + at);
            sz[j] = *reinterpret_cast<const u32x4*>(pz + at);
        }
#pragma unroll
        for (int j = 0; j < L::NO; ++j) {
            const int u = tid + 256 * j, l = u & 63;
            const int m = sizeof(E) == 2 ? u >> 6 : u >> 7;
            const int row = 16 * m + (l & 15);
            const E* p = dc + (int64_t)(row < ch.valid ? row : ch.valid - 1) * ldv + (int64_t)(hk * rep + vh) * a.dv + 32 * b + 4 * (l >> 4);
            if constexpr (sizeof(E) == 2) so[j] = __builtin_bit_cast(u32x4, A::ld_row_acc((const bf16*)p));
            else so[j] = *reinterpret_cast<const u32x4*>(p + 16 * ((u >> 6) & 1));
            if (row >= ch.valid) so[j] = u32x4{0, 0, 0, 0};
        }
    };
    auto store = [&](char* buf) {
#pragma unroll
        for (int j = 0; j < L::NS; ++j) {
            *reinterpret_cast<u32x4*>(buf + L::S_AT + (tid + 256 * j) * 16) = ss[j];
            *reinterpret_cast<u32x4*>(buf + L::D_AT + (tid + 256 * j) * 16) = sd[j];
        }
#pragma unroll
        for (int j = 0; j < L::NE; ++j) {
            *reinterpret_cast<u32x4*>(buf + L::E_AT + (tid + 256 * j) * 16) = se[j];
            *reinterpret_cast<u32x4*>(buf + L::Z_AT + (tid + 256 * j) * 16) = sz[j];
        }
#pragma unroll
        for (int j = 0; j < L::NO; ++j) *reinterpret_cast<u32x4*>(buf + L::O_AT + (tid + 256 * j) * 16) = so[j];
    };
    load(0, 0);
    store(lds);
    lds_barrier();

    f32x4 aq[ST], ak[ST];
#pragma unroll
    for (int t = 0; t < ST; ++t) aq[t] = ak[t] = zero;
    int step = 0;
    for (int vh = 0; vh < rep; ++vh) {
        const int64_t rec = (int64_t)slot * a.Hv + hk * rep + vh;
        const int h = hk * rep + vh;
        if (tid < C) {
            const float* f = reinterpret_cast<const float*>(prep + rec * PREP_BYTES + TRI_BYTES);
            gam[tid] = f[tid];
            om[tid] = f[2 * C + tid];
            bts[tid] = f[3 * C + tid];
            Gs[tid] = reinterpret_cast<const double*>(f + 4 * C)[tid];
        }
        f32x4 dos[ST], zs[ST], eds[ST], xl[MT], wl[MT], xu[MT], wu[MT];
        float dot = 0.0f;   // <S, dS>
#pragma unroll
        for (int t = 0; t < ST; ++t) dos[t] = zs[t] = eds[t] = zero;
#pragma unroll
        for (int n = 0; n < MT; ++n) xl[n] = wl[n] = xu[n] = wu[n] = zero;
        for (int b = 0; b < nb; ++b, ++step) {
            const char* buf = lds + (L::BUFS == 2 ? (step & 1) * L::STEP : 0);
            {
                const int nv = b + 1 < nb ? vh : vh + 1 < rep ? vh + 1 : vh;
                load(nv, b + 1 < nb ? b + 1 : vh + 1 < rep ? 0 : b);
            }
            const Ex ow = A::ld_ex(buf + L::O_AT, w, swz(lane));
            const Sp zw = A::ld_rec(buf + L::Z_AT, w, lane), ew = A::ld_rec(buf + L::E_AT, w, lane);
#pragma unroll
            for (int t = 0; t < ST; ++t) {
                const Sp sf = A::ld_rec(buf + L::S_AT, t, lane), df = A::ld_rec(buf + L::D_AT, t, lane);
                dos[t] = A::mma(sf, ow, dos[t]);
                zs[t] = A::mma(sf, zw, zs[t]);
                eds[t] = A::mma(df, ew, eds[t]);
                if (t % 4 == w) dot += A::dot(sf, df);
            }
#pragma unroll
            for (int n = 0; n < MT; ++n) {
                const Sp en = A::ld_rec(buf + L::E_AT, n, lane);
                if (n <= w) {
                    xl[n] = A::mma(en, ow, xl[n]);
                    wl[n] = A::mma(en, zw, wl[n]);
                }
                if (n >= w) {
                    xu[n] = A::mma(A::ld_ex(buf + L::O_AT, n, swz(lane)), ew, xu[n]);
                    wu[n] = A::mma(A::ld_rec(buf + L::Z_AT, n, lane), ew, wu[n]);
                }
            }
            if constexpr (L::BUFS == 1) lds_barrier();
            store(lds + (L::BUFS == 2 ? ((step + 1) & 1) * L::STEP : 0));
            lds_barrier();
        }
        // inside the chunk
        const float gt = gam[tok], bt = bts[tok], ob = om[tok] * bt;
        const double Gt = Gs[tok];
        float dGp = 0.0f, dGm = 0.0f, db = 0.0f;   // rows' and columns' sums; the latter without beta
        Ex qw[KB], kw[KB];
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            qw[b] = A::ld_ex(ql, w * KB + b, lane);
            kw[b] = A::ld_ex(kl, w * KB + b, lane);
        }
#pragma unroll
        for (int n = 0; n < MT; ++n) {
            f32x4 x = zero, m = zero, x2 = zero, m2 = zero;
            // q.k and k.k: of this wavefront's rows as [s][t], of its columns as [t][s]
            f32x4 qkl = zero, kkl = zero, qku = zero, kku = zero;
#pragma unroll
            for (int b = 0; b < KB; ++b) {
                const Ex kn = A::ld_ex(kl, n * KB + b, lane);
                if (n <= w) {
                    qkl = A::mma(kn, qw[b], qkl);
                    kkl = A::mma(kn, kw[b], kkl);
                }
                if (n >= w) {
                    qku = A::mma(A::ld_ex(ql, n * KB + b, lane), kw[b], qku);
                    kku = A::mma(kn, kw[b], kku);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int o = 16 * n + 4 * g + i;
                if (n <= w) {   // [s = o][t = tok]
                    const bool in = o <= tok;
                    const float d = in ? __builtin_amdgcn_exp2f((float)(Gt - Gs[o])) * bts[o] : 0.0f;
                    x[i] = in ? a.scale * d * xl[n][i] : 0.0f;
                    m[i] = o < tok ? -d * wl[n][i] : 0.0f;
                    dGp += x[i] * qkl[i] + m[i] * kkl[i];
                }
                if (n >= w) {   // [t = o][s = tok]
                    const bool in = tok <= o;
                    const float d = in ? __builtin_amdgcn_exp2f((float)(Gs[o] - Gt)) : 0.0f;
                    x2[i] = in ? a.scale * d * xu[n][i] : 0.0f;
                    m2[i] = tok < o ? -d * wu[n][i] : 0.0f;
                    dGm += x2[i] * qku[i] + m2[i] * kku[i];
                    x2[i] *= bt;
                    m2[i] *= bt;
                }
            }
            xl[n] = x;
            wl[n] = m;
            xu[n] = x2;
            wu[n] = m2;
        }
        Sp xlf[2], wlf[2], xuf[2], wuf[2];
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            xlf[b] = A::split(xl[2 * b], xl[2 * b + 1]);
            wlf[b] = A::split(wl[2 * b], wl[2 * b + 1]);
            xuf[b] = A::split(xu[2 * b], xu[2 * b + 1]);
            wuf[b] = A::split(wu[2 * b], wu[2 * b + 1]);
        }
        float qs = 0.0f, kz = 0.0f, ke = 0.0f;   // q.(dO S^T), k.(Z S^T), k.(E dS^T) of the token
#pragma unroll
        for (int t = 0; t < ST; ++t) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float qv = A::at(qw[t / 2], 4 * (t & 1) + i), kv = A::at(kw[t / 2], 4 * (t & 1) + i);
                qs += qv * dos[t][i];
                kz += kv * zs[t][i];
                ke += kv * eds[t][i];
                aq[t][i] += a.scale * gt * dos[t][i];
                ak[t][i] += ob * eds[t][i] - gt * zs[t][i];
            }
#pragma unroll
            for (int tb = 0; tb < 2; ++tb) {
                const Ex kt = A::template ld_ex_t<KB>(kl, t / 2, t & 1, tb, g, r);
                if (tb <= w / 2) {
                    aq[t] = A::mma(kt, xlf[tb], aq[t]);
                    ak[t] = A::mma(kt, wlf[tb], ak[t]);
                }
                if (tb >= w / 2) {
                    const Ex qt = A::template ld_ex_t<KB>(ql, t / 2, t & 1, tb, g, r);
                    ak[t] = A::mma(qt, xuf[tb], ak[t]);
                    ak[t] = A::mma(kt, wuf[tb], ak[t]);
                }
            }
        }
        qs = over_groups(qs);
        kz = over_groups(kz);
        ke = over_groups(ke);
        dGp = over_groups(dGp);
        dGm = over_groups(dGm);
        db = dGm + om[tok] * ke;
#pragma unroll
        for (int m = 1; m < 64; m <<= 1) dot += __shfl_xor(dot, m);
        if (lane == 0) dots[w] = dot;
        double d = (double)dGp - (double)(bt * dGm) + (double)(gt * (a.scale * qs - kz)) - (double)(ob * ke);
        if (g == 0) {
            dGs[tok] = d;
            kes[tok] = ob * ke;   // the chunk's end decays into every om
            if (tok < ch.valid) dbeta[(ch.row0 + tok) * a.Hv + h] = db;
        }
        lds_barrier();
        if (w == 0) {
            double x = dGs[lane];
            double e = (double)kes[lane];
#pragma unroll
            for (int m = 32; m >= 1; m >>= 1) e += __shfl_xor(e, m);
            if (lane == 63) x += e + (double)(gam[C - 1] * ((dots[0] + dots[1]) + (dots[2] + dots[3])));
#pragma unroll
            for (int m = 1; m < 64; m <<= 1) {
                const double dn = __shfl_down(x, m);
                if (lane + m < 64) x += dn;
            }
            if (lane < ch.valid) dg[(ch.row0 + lane) * a.Hv + h] = (float)x;
        }
        lds_barrier();
    }
    if (tok < ch.valid) {
        E* pq = dq + (ch.row0 + tok) * ldk + hk * DK + 8 * g;
        E* pk = dk + (ch.row0 + tok) * ldk + hk * DK + 8 * g;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
            A::st4(pq + 32 * b, aq[2 * b]);
            A::st4(pq + 32 * b + 4, aq[2 * b + 1]);
            A::st4(pk + 32 * b, ak[2 * b]);
            A::st4(pk + 32 * b + 4, ak[2 * b + 1]);
        }
    }
}

template <typename E, int DK>
hipError_t grad_t(const Args& a, const void* q, const void* k, const void* dout, const char* prep,
                  const char* ws_s, const char* ws_e, const char* ws_d, const char* ws_z, void* dq, void* dk, float* dg,
                  float* dbeta, hipStream_t stream) {
    const int64_t slots = places_of(a.nseq, a.T, a.cu != nullptr, C);
    hipLaunchKernelGGL((grad_kernel<E, DK>), dim3((unsigned)(slots * a.Hk)), dim3(256), 0, stream, a, (const E*)q, (const E*)k,
                       (const E*)dout, prep, ws_s, ws_e, ws_d, ws_z, (E*)dq, (E*)dk, dg, dbeta);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grad(bool f32, int dk_, const Args& a, const void* q, const void* k, const void* dout,
                       const char* prep, const char* ws_s, const char* ws_e, const char* ws_d, const char* ws_z, void* dq,
                       void* dk, float* dg, float* dbeta, hipStream_t stream) {
#define KDA_GG(E, D) return grad_t<E, D>(a, q, k, dout, prep, ws_s, ws_e, ws_d, ws_z, dq, dk, dg, dbeta, stream)
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
