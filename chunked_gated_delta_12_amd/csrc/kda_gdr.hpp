// kda_gdr.hpp -- building blocks of the chunked gated delta rule with one decay a head.
//
// A chunk is 64 tokens.  With S the state at its start, G_t the sum of g over its tokens
// up to t, gam = e^G, om_t = e^(G_end - G_t) and D_ts = e^(G_t - G_s):
//     N_ts = D_ts k_t.k_s (s < t),   X = (I + N diag(beta))^-1,   e = X (V - gam (K S))
//     P_ts = scale D_ts q_t.k_s beta_s (s <= t),   O = scale gam (Q S) + P e
//     S'   = gam_end S + K^T (om beta e)
// and backwards, dS' being the gradient at the chunk's end:
//     Z = X^T (P^T dO + om beta (K dS')) = dV
//     dS = gam_end dS' + scale Q^T (gam dO) - K^T (gam Z)
// No factor exceeds one for g <= 0, so the decay needs no bound.
//
// Precision: q, k, v and do enter the bf16 matrix cores as they are.  Every other
// operand (X, P, S, e, Z, ...) is an fp32 value split into three bf16 parts, x = hi + mid + lo:
// each takes 8 bits and a sign of what the one before left, so 2^-27 |x| at most is left over, and a product is the
// sum of the parts' products down to 2^-18 of it: three matrix instructions against an exact
// operand, six against a split one (what is left out is below 2^-26).  That is fp32's own
// precision at 3/16 and 6/16 of the time of its matrix instructions.  Two parts (two and three
// instructions) left the state 4e-6 and the gradients of g and beta up to 1e-5 off, where fp32
// products give 2e-7 and 5e-7; one rounding to bf16 leaves 3e-3.
// In fp32 storage all of it runs on the fp32 matrix cores.
//
// Operands live in LDS and in the workspace as fragment blocks of 16 rows by 32 columns
// of the contraction: lane (g, r) = 16 g + r holds row r and its eight slots of group g
// contiguously, so reads are 16 bytes a lane without bank conflicts.  In the workspace values are
// fp32, and are split on their way into LDS or registers.  Two slot maps:
//   natural:      slot s of group g is column 8 g + s           (rows of q, k: channels)
//   accumulator:  slot s < 4 is column 4 g + s, s >= 4 is 16 + 4 g + (s - 4), which is what
//                 two accumulator tiles hold in place           (tokens, and dv columns)
// A state's accumulator tile t = 2 b + h holds in row 4 g + i channel 32 b + 8 g + 4 h + i:
// with that, pairs of its tiles are B operands of the natural map.
#pragma once

#include "kda_device.hpp"

namespace kda {
namespace gdr {

constexpr int C = 64;                   // tokens a chunk
constexpr int MT = 4;                   // 16-token tiles a chunk
constexpr int WSB = 2048;               // bytes of a fragment block of fp32 values in the workspace
constexpr int TRI = 6;                  // blocks of a triangular 64 x 64 operand that are not zero

typedef short s16x4 __attribute__((__vector_size__(8)));
typedef uint32_t u32x4 __attribute__((__vector_size__(16)));

// Blocks (m, kb) of a lower triangular operand: kb <= m / 2; of an upper one: kb >= m / 2.
__host__ __device__ constexpr int lower_block(int m, int kb) { return m < 2 ? m : 2 + 2 * (m - 2) + kb; }
__host__ __device__ constexpr int upper_block(int m, int kb) { return m < 2 ? 2 * m + kb : 4 + (m - 2); }

// What a call works on.  Sequences either all have T tokens (cu NULL; rows are [nseq][T])
// or are packed into T rows, sequence n from cu[n] to cu[n + 1].
struct Args {
    int nseq, T, Hk, Hv, dv;
    const int* cu;
    float scale;
};

// Units of `unit` tokens have places in the workspace: those of sequence n from place_of(n) on.
// Packed, floor(first row / unit) + n leaves room for a part unit a sequence.
__device__ __forceinline__ int place_of(const Args& a, int n, int64_t unit) {
    if (!a.cu) return (int)((int64_t)n * ((a.T + unit - 1) / unit));
    int lo = a.cu[n];
    lo = lo < 0 ? 0 : lo > a.T ? a.T : lo;
    return (int)(lo / unit) + n;
}
__host__ __device__ inline int64_t places_of(int nseq, int T, bool packed, int64_t unit) {
    return packed ? (int64_t)T / unit + nseq : (int64_t)nseq * (((int64_t)T + unit - 1) / unit);
}

// A sequence's rows (n the same for the wavefront).  Offsets are held to [0, T] and to their
// order, so that none reads or writes past the tensors.
struct Seq {
    int64_t row0;
    int len;
};
__device__ __forceinline__ Seq seq_of(const Args& a, int n) {
    if (!a.cu) return Seq{(int64_t)n * a.T, a.T};
    int lo = __builtin_amdgcn_readfirstlane(a.cu[n]), hi = __builtin_amdgcn_readfirstlane(a.cu[n + 1]);
    lo = lo < 0 ? 0 : lo > a.T ? a.T : lo;
    hi = hi < lo ? lo : hi > a.T ? a.T : hi;
    return Seq{lo, hi - lo};
}

// The sequence whose places hold `place`, and which of its units it is; n < 0: none.
struct Unit {
    int n, i;
};
__device__ __forceinline__ Unit unit_at(const Args& a, int place, int64_t unit, int lane) {
    int n;
    if (!a.cu) {
        n = (int)(place / ((a.T + unit - 1) / unit));
    } else {
        // Places rise with the sequence: the last that starts at or before this one, 64 evenly spaced
        // sequences a step (two steps for 4,096; counting them all was most of a short sequence's time).
        // With offsets out of order any of them, but one of the call's.
        int first = 0, cnt = a.nseq;
        for (;;) {
            const int step = (cnt + 63) / 64, at = lane * step;
            const int k = __popcll(__ballot(at < cnt && place_of(a, first + at, unit) <= place));
            if (k == 0) return Unit{-1, 0};
            first += (k - 1) * step;
            cnt -= (k - 1) * step;
            if (step == 1) break;
            cnt = cnt < step ? cnt : step;
        }
        n = first;
    }
    if (n < 0) return Unit{-1, 0};
    return Unit{n, place - __builtin_amdgcn_readfirstlane(place_of(a, n, unit))};
}

// The chunk at a place of 64-token units; n < 0: none is there.
struct Chunk {
    int n, c, valid;
    int64_t row0;
};
__device__ __forceinline__ Chunk chunk_at(const Args& a, int place, int lane) {
    const Unit u = unit_at(a, place, C, lane);
    if (u.n < 0 || u.i < 0) return Chunk{-1, 0, 0, 0};
    const Seq s = seq_of(a, u.n);
    if ((int64_t)u.i * C >= s.len) return Chunk{-1, 0, 0, 0};
    const int left = s.len - u.i * C;
    return Chunk{u.n, u.i, left < C ? left : C, s.row0 + (int64_t)u.i * C};
}

// Segments: where a sequence has more than `over` chunks, those of more than `seg` are walked in
// pieces of `seg` chunks, joined by their affine maps; others in one piece.  seg = 0: none is cut.
//
// A piece's map and start state are at its place.  Few sequences have the places of units of seg_unit
// tokens, cut or not.  Many packed ones (`apart`: more than whole units fit the rows) would
// leave nearly all of those empty, so the pieces of cut ones have places of their own: those of a
// sequence that starts at row lo from 2 floor(lo / unit) on.  A cut sequence is longer than a unit, len / unit = l > 1,
// so that 2 floor(l) >= ceil(l): its pieces end before those of the next one begin, and
// before 2 floor(rows / unit).
struct Segs {
    int seg, over;
    bool apart;
};
__host__ __device__ inline int64_t seg_unit(const Segs& g) { return g.seg ? (int64_t)g.seg * C : (int64_t)1 << 40; }
// Places of pieces (where sequences are cut at all), and of walks: apart, one a sequence goes before the pieces'.
__host__ __device__ inline int64_t pieces_of(int nseq, int T, bool packed, const Segs& g) {
    return g.apart ? 2 * (T / seg_unit(g)) : places_of(nseq, T, packed, seg_unit(g));
}
// Sequences that a join has workgroups for: apart, of those that start in the same unit one at most is cut.
__host__ __device__ inline int64_t joins_of(int nseq, int T, const Segs& g) { return g.apart ? T / seg_unit(g) : nseq; }
__host__ __device__ inline int64_t walk_places(int nseq, int T, bool packed, const Segs& g) {
    return pieces_of(nseq, T, packed, g) + (g.apart ? nseq : 0);
}

// Whether a sequence of nch chunks is cut: the same in every kernel of a call.
__device__ __forceinline__ bool is_cut(const Args& a, const Segs& g, int nch, int lane) {
    if (!g.seg || nch <= g.seg) return false;
    if (nch > g.over || !a.cu) return nch > g.over;
    for (int n0 = 0; n0 < a.nseq; n0 += 64) {   // is there a longer one?
        bool more = false;
        if (n0 + lane < a.nseq) {
            int lo = a.cu[n0 + lane], hi = a.cu[n0 + lane + 1];
            lo = lo < 0 ? 0 : lo > a.T ? a.T : lo;
            hi = hi < lo ? lo : hi > a.T ? a.T : hi;
            more = ((int64_t)(hi - lo) + C - 1) / C > g.over;
        }
        if (__ballot(more)) return true;
    }
    return false;
}

// The first place of a cut sequence's pieces.
__device__ __forceinline__ int first_piece(const Args& a, const Segs& sg, int n) {
    if (!sg.apart) return place_of(a, n, seg_unit(sg));
    int lo = a.cu[n];
    lo = lo < 0 ? 0 : lo > a.T ? a.T : lo;
    return 2 * (lo / (sg.seg * C));
}

// Apart: the cut sequence whose pieces hold place `at`, the last one that begins there or before, and
// which of its pieces; n < 0: none.
__device__ __forceinline__ Unit cut_unit_at(const Args& a, const Segs& sg, int at, int lane) {
    int n = -1;
    bool any = false;   // is any sequence long enough for the cut?
    for (int n0 = 0; n0 < a.nseq; n0 += 64) {
        bool cut = false, longer = false, behind = false;
        if (n0 + lane < a.nseq) {
            int lo = a.cu[n0 + lane], hi = a.cu[n0 + lane + 1];
            lo = lo < 0 ? 0 : lo > a.T ? a.T : lo;
            hi = hi < lo ? lo : hi > a.T ? a.T : hi;
            const int nch = (int)(((int64_t)(hi - lo) + C - 1) / C);
            longer = nch > sg.over;
            behind = 2 * (lo / (sg.seg * C)) > at;
            cut = nch > sg.seg && !behind;
        }
        any |= __ballot(longer) != 0;
        const uint64_t m = __ballot(cut);
        if (m) n = n0 + 63 - __builtin_clzll(m);
        if (any && __ballot(behind)) break;
    }
    if (!any || n < 0) return Unit{-1, 0};
    return Unit{n, at - __builtin_amdgcn_readfirstlane(first_piece(a, sg, n))};
}

// The piece at a place of walk_places: chunks [c0, c1) of sequence n, piece i of cnt.
struct Piece {
    int n, i, cnt, c0, c1;
    int at;         // its place among the pieces, where it is one of several
    int slot;       // the sequence's first place among the chunks
    Seq s;
};
__device__ __forceinline__ Piece piece_at(const Args& a, const Segs& sg, int place, int lane) {
    const bool whole = !sg.seg || (sg.apart && place < a.nseq);   // a place for a sequence that is not cut
    const int at = sg.apart ? place - a.nseq : place;
    const Unit u = whole ? Unit{place, 0} : sg.apart ? cut_unit_at(a, sg, at, lane) : unit_at(a, place, seg_unit(sg), lane);
    Piece p{-1, 0, 0, 0, 0, 0, 0, Seq{0, 0}};
    if (u.n < 0 || u.i < 0) return p;
    p.s = seq_of(a, u.n);
    const int nch = (int)(((int64_t)p.s.len + C - 1) / C);
    const bool cut = is_cut(a, sg, nch, lane);
    p.cnt = cut ? (nch + sg.seg - 1) / sg.seg : 1;
    if (u.i >= p.cnt || (sg.apart && cut == whole)) return p;
    p.n = u.n;
    p.at = at;
    p.i = u.i;
    p.c0 = p.cnt > 1 ? u.i * sg.seg : 0;
    p.c1 = p.cnt > 1 && u.i + 1 < p.cnt ? p.c0 + sg.seg : nch;
    p.slot = __builtin_amdgcn_readfirstlane(place_of(a, u.n, C));
    return p;
}

// ---------------------------------------------------------------- operands
// Where lane (g, r)'s 16 bytes of a natural block of q or k lie in LDS: row r of group g at
// r ^ 4 g, so that the transposed reads, which take a row of every group, spread over the banks.
__device__ __forceinline__ u32x4 buf_ld128(Rsrc s, uint32_t off) {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(s, (int)off, 0, 0));
}

__device__ __forceinline__ int swz(int lane) { return lane ^ ((lane >> 4) << 2); }

template <typename E> struct Arith;

template <> struct Arith<bf16> {
    typedef bf16x8 Ex;                        // an operand that is exact in bf16
    struct Sp { bf16x8 hi, mid, lo; };        // an fp32 operand in three parts
    static constexpr int EXB = 1024;          // bytes of an exact block
    static constexpr int SPB = 3 * EXB;       // bytes of a split one: three planes
    // One part of two values, and what is left of them: five instructions, a packed
    // conversion, its values back as floats, two differences (exact).
    static __device__ __forceinline__ uint32_t part2(float& a, float& b) {
        uint32_t p = __builtin_bit_cast(uint32_t, bf16x2{(bf16)a, (bf16)b});
        asm("" : "+v"(p));   // one conversion for both values, not another one for each of the parts
        a -= __builtin_bit_cast(float, p << 16);
        b -= __builtin_bit_cast(float, p & 0xffff0000u);
        return p;
    }
    static __device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& mid, uint32_t& lo) {
        hi = part2(a, b);
        mid = part2(a, b);
        lo = __builtin_bit_cast(uint32_t, bf16x2{(bf16)a, (bf16)b});
    }
    static __device__ __forceinline__ Sp split(f32x4 a, f32x4 b) {
        u32x4 h, m, l;
        uint32_t x, y, z;
        split2(a[0], a[1], x, y, z); h[0] = x; m[0] = y; l[0] = z;
        split2(a[2], a[3], x, y, z); h[1] = x; m[1] = y; l[1] = z;
        split2(b[0], b[1], x, y, z); h[2] = x; m[2] = y; l[2] = z;
        split2(b[2], b[3], x, y, z); h[3] = x; m[3] = y; l[3] = z;
        return Sp{__builtin_bit_cast(bf16x8, h), __builtin_bit_cast(bf16x8, m), __builtin_bit_cast(bf16x8, l)};
    }
    static __device__ __forceinline__ f32x4 mma(Ex a, Ex b, f32x4 c) { return mfma_k32(a, b, c); }
    static __device__ __forceinline__ f32x4 mma(Ex a, const Sp& b, f32x4 c) {
        return mfma_k32(a, b.hi, mfma_k32(a, b.mid, mfma_k32(a, b.lo, c)));
    }
    static __device__ __forceinline__ f32x4 mma(const Sp& a, Ex b, f32x4 c) {
        return mfma_k32(a.hi, b, mfma_k32(a.mid, b, mfma_k32(a.lo, b, c)));
    }
    static __device__ __forceinline__ f32x4 mma(const Sp& a, const Sp& b, f32x4 c) {   // the small products first
        c = mfma_k32(a.mid, b.mid, mfma_k32(a.hi, b.lo, mfma_k32(a.lo, b.hi, c)));
        return mfma_k32(a.hi, b.hi, mfma_k32(a.hi, b.mid, mfma_k32(a.mid, b.hi, c)));
    }
    // The same for N accumulators: one part's product of each before the next, so that no
    // instruction waits for the one before it.
    template <int N>
    static __device__ __forceinline__ void mma_n(const Ex (&a)[N], const Sp& b, f32x4 (&c)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = mfma_k32(a[i], b.lo, c[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = mfma_k32(a[i], b.mid, c[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = mfma_k32(a[i], b.hi, c[i]);
    }
    template <int N>
    static __device__ __forceinline__ void mma_n(const Sp& a, const Ex (&b)[N], f32x4 (&c)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = mfma_k32(a.lo, b[i], c[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = mfma_k32(a.mid, b[i], c[i]);
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = mfma_k32(a.hi, b[i], c[i]);
    }
    static __device__ __forceinline__ Ex ld_ex(const char* base, int blk, int lane) {
        return *reinterpret_cast<const bf16x8*>(base + blk * EXB + swz(lane) * 16);
    }
    static __device__ __forceinline__ Sp ld_sp(const char* base, int blk, int lane) {
        const char* p = base + blk * SPB + lane * 16;
        return Sp{*reinterpret_cast<const bf16x8*>(p), *reinterpret_cast<const bf16x8*>(p + 1024),
                  *reinterpret_cast<const bf16x8*>(p + 2048)};
    }
    // Eight natural slots of a row in global memory.
    static __device__ __forceinline__ Ex ld_row(const bf16* p) { return *reinterpret_cast<const bf16x8*>(p); }
    // Four rows by 16 columns read transposed: lane r of a group of 16 gives the address of
    // row r >> 2, columns 4 (r & 3).., and receives column r of the four rows.
    static __device__ __forceinline__ bf16x4 ld_tr(const char* p) {
        typedef __attribute__((address_space(3))) s16x4* L;
        return __builtin_bit_cast(bf16x4, __builtin_amdgcn_ds_read_tr16_b64_v4i16((L)(__attribute__((address_space(3))) void*)p));
    }
    // Rows of a natural-map block set [token tile][kb], transposed: channel tile 2 kb + h as
    // rows, the 32 tokens of block tb as accumulator slots.
    template <int KB>
    static __device__ __forceinline__ Ex ld_ex_t(const char* base, int kb, int h, int tb, int g, int r) {
        const int at = swz((r & 3) * 16 + 4 * g + (r >> 2)) * 16 + h * 8;
        return cat8(ld_tr(base + ((2 * tb) * KB + kb) * EXB + at), ld_tr(base + ((2 * tb + 1) * KB + kb) * EXB + at));
    }
    // Row tile n of the transpose of a lower triangular split operand, columns of block tb.
    static __device__ __forceinline__ Sp ld_tri_t(const char* base, int n, int tb, int g, int r) {
        const int at = ((r & 3) * 16 + 4 * g + (r >> 2)) * 16 + (n & 1) * 8;
        const char *a = base + lower_block(2 * tb, n / 2) * SPB + at, *b = base + lower_block(2 * tb + 1, n / 2) * SPB + at;
        return Sp{cat8(ld_tr(a), ld_tr(b)), cat8(ld_tr(a + 1024), ld_tr(b + 1024)), cat8(ld_tr(a + 2048), ld_tr(b + 2048))};
    }
    // Tokens 16 m + 4 g + i of column col + r of a row-major tile with `ld` columns.
    static __device__ __forceinline__ f32x4 ld_col(const char* base, int ld, int m, int col, int g, int r) {
        const bf16x4 x = ld_tr(base + ((16 * m + 4 * g + (r >> 2)) * ld + col + 4 * (r & 3)) * 2);
        return f32x4{(float)x[0], (float)x[1], (float)x[2], (float)x[3]};
    }
    static __device__ __forceinline__ Ex cols(f32x4 a, f32x4 b) {
        return Ex{(bf16)a[0], (bf16)a[1], (bf16)a[2], (bf16)a[3], (bf16)b[0], (bf16)b[1], (bf16)b[2], (bf16)b[3]};
    }
    // Column n = r of the 32 x 16 matrix that picks slot `s` of group `grp`.
    static __device__ __forceinline__ Ex pick(int s, bool here) {
        Ex x;
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = (bf16)(here && i == s ? 1.0f : 0.0f);
        return x;
    }
    // a's rows, transposed through the product with a picking matrix (exact, and so is the sum
    // of the parts), as half a block of accumulator slots at byte `blk` of the record; returns the values.
    static __device__ __forceinline__ f32x4 put_t(Rsrc rec, uint32_t blk, const Sp& a, Ex j) {
        const f32x4 x = mma(a, j, f32x4{0, 0, 0, 0});
        buf_st_quad(x, rec, blk);
        return x;
    }
    static __device__ __forceinline__ float at(Ex x, int i) { return (float)x[i]; }
    typedef bf16x4 Q4;
    static __device__ __forceinline__ Q4 q4(f32x4 x) { return Q4{(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]}; }
    // One accumulator tile as half a split block.
    static __device__ __forceinline__ void put_half(char* base, int blk, int lane, int half, f32x4 x) {
        char* p = base + blk * SPB + lane * 16 + half * 8;
        typedef uint32_t u32x2 __attribute__((__vector_size__(8)));
        uint32_t h[2], m[2], l[2];
        split2(x[0], x[1], h[0], m[0], l[0]);
        split2(x[2], x[3], h[1], m[1], l[1]);
        *reinterpret_cast<u32x2*>(p) = u32x2{h[0], h[1]};
        *reinterpret_cast<u32x2*>(p + 1024) = u32x2{m[0], m[1]};
        *reinterpret_cast<u32x2*>(p + 2048) = u32x2{l[0], l[1]};
    }
    static __device__ __forceinline__ void st4(bf16* p, f32x4 x) {
        *reinterpret_cast<bf16x4*>(p) = bf16x4{(bf16)x[0], (bf16)x[1], (bf16)x[2], (bf16)x[3]};
    }
};

template <> struct Arith<float> {
    struct Ex { f32x4 a, b; };
    typedef Ex Sp;
    static constexpr int EXB = WSB, SPB = WSB;
    static __device__ __forceinline__ Sp split(f32x4 a, f32x4 b) { return Sp{a, b}; }
    static __device__ __forceinline__ f32x4 mma(const Ex& x, const Ex& y, f32x4 c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c = mfma_k4(x.a[i], y.a[i], c);
#pragma unroll
        for (int i = 0; i < 4; ++i) c = mfma_k4(x.b[i], y.b[i], c);
        return c;
    }
    template <int N>
    static __device__ __forceinline__ void mma_n(const Ex (&a)[N], const Ex& b, f32x4 (&c)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = mma(a[i], b, c[i]);
    }
    template <int N>
    static __device__ __forceinline__ void mma_n(const Ex& a, const Ex (&b)[N], f32x4 (&c)[N]) {
#pragma unroll
        for (int i = 0; i < N; ++i) c[i] = mma(a, b[i], c[i]);
    }
    // a block is two planes of 16 bytes a lane: slots 0..3 and 4..7
    static __device__ __forceinline__ Ex ld_ex(const char* base, int blk, int lane) { return ld_sp(base, blk, swz(lane)); }
    static __device__ __forceinline__ Sp ld_sp(const char* base, int blk, int lane) {
        const char* p = base + blk * SPB + lane * 16;
        return Ex{*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 1024)};
    }
    static __device__ __forceinline__ Ex ld_row(const float* p) {
        return Ex{*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4)};
    }
    template <int KB>
    static __device__ __forceinline__ Ex ld_ex_t(const char* base, int kb, int h, int tb, int g, int r) {
        Ex x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = h * 1024 + swz((r >> 2) * 16 + 4 * g + i) * 16 + (r & 3) * 4;
            x.a[i] = *reinterpret_cast<const float*>(base + ((2 * tb) * KB + kb) * SPB + at);
            x.b[i] = *reinterpret_cast<const float*>(base + ((2 * tb + 1) * KB + kb) * SPB + at);
        }
        return x;
    }
    static __device__ __forceinline__ Sp ld_tri_t(const char* base, int n, int tb, int g, int r) {
        Sp x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int at = (n & 1) * 1024 + ((r >> 2) * 16 + 4 * g + i) * 16 + (r & 3) * 4;
            x.a[i] = *reinterpret_cast<const float*>(base + lower_block(2 * tb, n / 2) * SPB + at);
            x.b[i] = *reinterpret_cast<const float*>(base + lower_block(2 * tb + 1, n / 2) * SPB + at);
        }
        return x;
    }
    static __device__ __forceinline__ f32x4 ld_col(const char* base, int ld, int m, int col, int g, int r) {
        const float* p = reinterpret_cast<const float*>(base) + (16 * m + 4 * g) * ld + col + r;
        return f32x4{p[0], p[ld], p[2 * ld], p[3 * ld]};
    }
    static __device__ __forceinline__ Ex cols(f32x4 a, f32x4 b) { return Ex{a, b}; }
    static __device__ __forceinline__ Ex pick(int s, bool here) {
        Ex x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x.a[i] = here && i == s ? 1.0f : 0.0f;
            x.b[i] = here && 4 + i == s ? 1.0f : 0.0f;
        }
        return x;
    }
    static __device__ __forceinline__ f32x4 put_t(Rsrc rec, uint32_t blk, const Sp& a, const Ex& j) {
        const f32x4 x = mma(a, j, f32x4{0, 0, 0, 0});
        buf_st_quad(x, rec, blk);
        return x;
    }
    static __device__ __forceinline__ float at(const Ex& x, int i) { return i < 4 ? x.a[i & 3] : x.b[i & 3]; }
    typedef f32x4 Q4;
    static __device__ __forceinline__ Q4 q4(f32x4 x) { return x; }
    static __device__ __forceinline__ void put_half(char* base, int blk, int lane, int half, f32x4 x) {
        *reinterpret_cast<f32x4*>(base + blk * SPB + half * 1024 + lane * 16) = x;
    }
    static __device__ __forceinline__ void st4(float* p, f32x4 x) { *reinterpret_cast<f32x4*>(p) = x; }
};

// The picking matrix of put_t for half h of a block: slot 4 h + (r & 3) of group r >> 2.  In
// an accumulator-map block of tokens that is token 16 h + r; in a natural-map block of
// channels it is the channel that row r of accumulator tile h holds.
template <typename E>
__device__ __forceinline__ typename Arith<E>::Ex pick_half(int h, int g, int r) {
    return Arith<E>::pick(4 * h + (r & 3), (r >> 2) == g);
}

// ---------------------------------------------------------------- workspace
// A fragment block there: two planes of 16 bytes a lane, slots 0..3 and 4..7.
__device__ __forceinline__ uint32_t rec_at(int lane, int half) { return (uint32_t)(half * 1024 + lane * 16); }
struct Rec { f32x4 a, b; };
__device__ __forceinline__ Rec ld_rec(Rsrc rec, uint32_t at) {
    typedef BufQuad<float> Q;
    return Rec{Q::ld(rec, at, 0), Q::ld(rec, at + 1024, 0)};
}
__device__ __forceinline__ void st_rec(char* base, int blk, int lane, f32x4 a, f32x4 b) {
    char* p = base + blk * WSB + lane * 16;
    *reinterpret_cast<f32x4*>(p) = a;
    *reinterpret_cast<f32x4*>(p + 1024) = b;
}
// 16-byte piece u of consecutive blocks of the workspace, as it lies in LDS.
template <typename E>
__device__ __forceinline__ void put_piece(char* base, int u, u32x4 x) {
    Arith<E>::put_half(base, u >> 7, u & 63, (u >> 6) & 1, __builtin_bit_cast(f32x4, x));
}

// A chunk of one head: X, then per token gam, om beta, om, beta, and G log2(e) in 64 bits.
constexpr int X_BYTES = TRI * WSB, F_BYTES = 4 * C * 4 + C * 8, PREP_BYTES = X_BYTES + F_BYTES;
// The map of a piece of one head, [dk][dv + dk] fp32: N, then M.
__host__ __device__ constexpr int64_t map_bytes(int dk, int dv) { return (int64_t)dk * (dv + dk) * 4; }
// The backward pass's records of a chunk of one head: a state (dk / 16 by dv / 32 blocks,
// rows channels in the order of the accumulator tiles) and a 64 x dv operand (4 by dv / 32 blocks, rows tokens).
__host__ __device__ constexpr int64_t state_bytes(int dk, int dv) { return (int64_t)(dk / 16) * (dv / 32) * WSB; }
__host__ __device__ constexpr int64_t rows_bytes(int dv) { return (int64_t)MT * (dv / 32) * WSB; }
// One behind the other: the start state, the end's gradient, e, Z.
__host__ __device__ constexpr int64_t rec_bytes(int dk, int dv) { return 2 * (state_bytes(dk, dv) + rows_bytes(dv)); }

}  // namespace gdr
}  // namespace kda
