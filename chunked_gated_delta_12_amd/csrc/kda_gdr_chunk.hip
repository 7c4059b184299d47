// kda_gdr_chunk.hip -- the launches of the chunked gated delta rule with one decay a head and
// the layout of its workspace.
//   forward:   prep (X and the decays of every chunk) -> [maps -> join] -> chain (states, outputs)
//   backward:  prep -> [maps both ways -> joins] -> chains both ways, saving the states and
//              their gradients -> grad
// The steps in brackets run where sequences are cut into pieces that are walked side by side.
#include "kda_gdr.hpp"
#include "kda_launch.hpp"

namespace kda {
namespace gdr {

hipError_t launch_prep(bool f32, int dk, const Args& a, const void* k, const float* g, const float* beta, char* ws,
                       hipStream_t stream);
hipError_t launch_fwd_chain(bool f32, int dk, const Args& a, const Segs& sg, const void* q, const void* k, const void* v,
                            const float* S0, const float* starts, const char* prep, void* o, float* S_T, hipStream_t stream);
hipError_t launch_maps(bool f32, int dk, const Args& a, const Segs& sg, const void* k, const void* v, const char* prep,
                       float* maps, hipStream_t stream);
hipError_t launch_bwd_maps(bool f32, int dk, const Args& a, const Segs& sg, const void* q, const void* k, const void* v,
                           const void* dout, const char* prep, float* maps, float* nmaps, hipStream_t stream);
hipError_t launch_bwd_chains(bool f32, int dk, const Args& a, const Segs& sg, const void* q, const void* k, const void* v,
                             const void* dout, const float* S0, const float* starts, const float* dS_T, const float* dstarts,
                             const char* prep, void* dv, float* dS0, char* recs, hipStream_t stream);
hipError_t launch_join(int dk, const Args& a, const Segs& sg, const float* init, const float* maps, float* starts,
                       const float* dinit, const float* nmaps, float* dstarts, hipStream_t stream);
hipError_t launch_grad(bool f32, int dk_, const Args& a, const void* q, const void* k, const void* dout,
                       const char* prep, const char* recs, void* dq, void* dk, float* dg, float* dbeta, hipStream_t stream);

namespace {

// Cutting a sequence costs a second walk of it (the maps, over dv + dk columns) and the join of
// its pieces, so it pays where its own walk would outlast the others' by much.  With a chunk
// taking about 6.8 us in a walk and 4.4 us in a map, and a piece 2.6 us in the join (bf16,
// 128 x 128), L chunks in pieces of s take 11.2 s + 2.6 L / s us: least at s^2 = 0.23 L, and flat
// around it.  `seg` is from s^2 = 0.31 L, but at least the even share
// of the call's work over the 256 compute units, half a workgroup set aside for the part piece that
// each sequence ends with.  Uncut the walk takes 6.8 L us: longer than the pieces from about
// L = 1.7 seg + 3 on, which is `over`; once any sequence is longer than that the maps run
// anyway, and all longer than a piece are cut.  0.23 and 0.31 were measured over both passes and types,
// 32 x 64 to 128 x 256, one to eight heads, 2,000 to 30,000 tokens: prefill in bf16 of 8,492 tokens, 4 heads of
// 128 x 256, 164 and 147 us, of 2 x 1,000 tokens, 4 heads of 64 x 64, 49 and 53; fp32 forwards
// 4,096 tokens, one head of 128 x 128, 140 and 151; the others within 10% either way.
Segs segs_of(int nseq, int T, int Hv, int dv, bool packed) {
    const int64_t heads = (int64_t)Hv * ((dv + 127) / 128), work = places_of(nseq, T, packed, C) * heads;
    const int64_t longest = ((int64_t)T + C - 1) / C;   // that a sequence can be
    int64_t share = 256 - nseq * heads / 2;
    if (share < 64) share = 64;
    int64_t seg = 2;
    while (100 * seg * seg < 31 * longest) ++seg;
    if (seg < (work + share - 1) / share) seg = (work + share - 1) / share;
    const int64_t over = (17 * seg + 30) / 10;
    if (longest <= over) return Segs{0, 0, false};
    return Segs{(int)seg, (int)over, packed && nseq > T / (seg * C)};
}

// The parts of a workspace, in order; each a multiple of 16 bytes.
struct Plan {
    Segs sg;
    int64_t prep, recs, maps, nmaps, starts, dstarts, bytes;
};
Plan plan_of(bool bwd, int nseq, int T, int Hv, int dk, int dv, bool packed) {
    Plan p{};
    p.sg = segs_of(nseq, T, Hv, dv, packed);
    const int64_t n = places_of(nseq, T, packed, C) * Hv;
    const int64_t m = p.sg.seg ? pieces_of(nseq, T, packed, p.sg) * Hv : 0;
    int64_t at = 0;
    auto take = [&](int64_t& x, int64_t bytes) {
        x = at;
        at += bytes;
    };
    take(p.prep, n * (int64_t)PREP_BYTES);
    if (bwd) take(p.recs, n * rec_bytes(dk, dv));
    take(p.maps, m * map_bytes(dk, dv));
    take(p.starts, m * dk * dv * 4);
    if (bwd) {
        take(p.nmaps, m * dk * dv * 4);
        take(p.dstarts, m * dk * dv * 4);
    }
    p.bytes = at;
    return p;
}

// Zeros in the rows of no sequence, those before the first and behind the last: words of one
// tensor (blockIdx.y), 16 bytes a lane where rows are whole pieces of it.
struct Clear {
    void* p[GDR_CLEAR_MAX];
    int64_t row[GDR_CLEAR_MAX];   // bytes
};
template <typename W>
__device__ __forceinline__ void clear_words(W* p, int64_t lo, int64_t hi, int64_t end) {
    const int64_t step = (int64_t)gridDim.x * blockDim.x;
    const int64_t n = lo + (end - hi);
    for (int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += step) p[i < lo ? i : hi + (i - lo)] = W{};
}
__global__ void __launch_bounds__(256) clear_kernel(int nseq, int T, const int* __restrict__ cu, Clear c) {
    int lo = cu[0], hi = cu[nseq];
    lo = lo < 0 ? 0 : lo > T ? T : lo;
    hi = hi < lo ? lo : hi > T ? T : hi;
    void* const p = c.p[blockIdx.y];
    const int64_t row = c.row[blockIdx.y];
    if (row % 16 == 0) clear_words((u32x4*)p, lo * (row / 16), hi * (row / 16), T * (row / 16));
    else clear_words((uint32_t*)p, lo * (row / 4), hi * (row / 4), T * (row / 4));
}

Args args_of(const GdrCall& c) { return Args{c.nseq, c.T, c.Hk, c.Hv, c.dv, c.cu, c.scale}; }

}  // namespace
}  // namespace gdr

size_t gdr_fwd_workspace_bytes(int nseq, int T, int Hv, int dk, int dv, bool packed) {
    return (size_t)gdr::plan_of(false, nseq, T, Hv, dk, dv, packed).bytes;
}

size_t gdr_bwd_workspace_bytes(int nseq, int T, int Hv, int dk, int dv, bool packed) {
    return (size_t)gdr::plan_of(true, nseq, T, Hv, dk, dv, packed).bytes;
}

#define KDA_DO(CALL)                         \
    do {                                     \
        const hipError_t e_ = (CALL);        \
        if (e_ != hipSuccess) return e_;     \
    } while (0)

hipError_t launch_gdr_fwd(const GdrCall& c, void* o, float* S_T, void* workspace, hipStream_t stream) {
    const gdr::Args a = gdr::args_of(c);
    const gdr::Plan p = gdr::plan_of(false, c.nseq, c.T, c.Hv, c.dk, c.dv, c.cu != nullptr);
    char* ws = (char*)workspace;
    float *maps = (float*)(ws + p.maps), *starts = (float*)(ws + p.starts);
    KDA_DO(gdr::launch_prep(c.f32, c.dk, a, c.k, c.g, c.beta, ws + p.prep, stream));
    if (p.sg.seg) {
        KDA_DO(gdr::launch_maps(c.f32, c.dk, a, p.sg, c.k, c.v, ws + p.prep, maps, stream));
        KDA_DO(gdr::launch_join(c.dk, a, p.sg, c.S0, maps, starts, nullptr, nullptr, nullptr, stream));
    }
    return gdr::launch_fwd_chain(c.f32, c.dk, a, p.sg, c.q, c.k, c.v, c.S0, starts, ws + p.prep, o, S_T, stream);
}

hipError_t launch_gdr_bwd(const GdrCall& c, const void* dout, const float* dS_T, void* dq, void* dk, void* dv, float* dg,
                          float* dbeta, float* dS0, void* workspace, hipStream_t stream) {
    const gdr::Args a = gdr::args_of(c);
    const gdr::Plan p = gdr::plan_of(true, c.nseq, c.T, c.Hv, c.dk, c.dv, c.cu != nullptr);
    char* ws = (char*)workspace;
    float *maps = (float*)(ws + p.maps), *nmaps = (float*)(ws + p.nmaps);
    float *starts = (float*)(ws + p.starts), *dstarts = (float*)(ws + p.dstarts);
    KDA_DO(gdr::launch_prep(c.f32, c.dk, a, c.k, c.g, c.beta, ws + p.prep, stream));
    if (p.sg.seg) {
        KDA_DO(gdr::launch_bwd_maps(c.f32, c.dk, a, p.sg, c.q, c.k, c.v, dout, ws + p.prep, maps, nmaps, stream));
        KDA_DO(gdr::launch_join(c.dk, a, p.sg, c.S0, maps, starts, dS_T, nmaps, dstarts, stream));
    }
    KDA_DO(gdr::launch_bwd_chains(c.f32, c.dk, a, p.sg, c.q, c.k, c.v, dout, c.S0, starts, dS_T, dstarts, ws + p.prep, dv, dS0,
                                  ws + p.recs, stream));
    return gdr::launch_grad(c.f32, c.dk, a, c.q, c.k, dout, ws + p.prep, ws + p.recs, dq, dk, dg, dbeta, stream);
}

hipError_t launch_gdr_clear(int nseq, int T, const int* cu, int n, void* const* tensors, const size_t* row_bytes,
                            hipStream_t stream) {
    gdr::Clear c{};
    for (int i = 0; i < n; ++i) {
        c.p[i] = tensors[i];
        c.row[i] = (int64_t)row_bytes[i];
    }
    hipLaunchKernelGGL(gdr::clear_kernel, dim3(128, (unsigned)n), dim3(256), 0, stream, nseq, T, cu, c);
    return hipGetLastError();
}

}  // namespace kda
