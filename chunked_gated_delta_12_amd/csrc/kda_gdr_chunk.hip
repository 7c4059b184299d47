// kda_gdr_chunk.hip -- the launches of the chunked gated delta rule with one decay a head and
// the layout of its workspace.
//   forward:   prep (X, P of every chunk) -> chain (states, outputs)
//   backward:  prep (with transposes) -> chain (states saved) -> chain backwards -> grad
#include "kda_gdr.hpp"
#include "kda_launch.hpp"

namespace kda {
namespace gdr {

hipError_t launch_prep(bool f32, int dk, bool bwd, const Args& a, const void* q, const void* k, const float* g,
                       const float* beta, char* ws, hipStream_t stream);
hipError_t launch_chain(bool f32, int dk, bool save, const Args& a, const void* q, const void* k, const void* v,
                        const float* beta, const float* S0, const char* prep, int64_t stride, void* o, float* S_T,
                        char* ws_s, char* ws_e, hipStream_t stream);
hipError_t launch_back(bool f32, int dk, const Args& a, const void* q, const void* k, const void* dout, const float* beta,
                       const float* dS_T, const char* prep, int64_t stride, void* dv, float* dS0, char* ws_d, char* ws_z,
                       hipStream_t stream);
hipError_t launch_grad(bool f32, int dk_, const Args& a, const void* q, const void* k, const float* beta, const void* dout,
                       const char* prep, const char* ws_s, const char* ws_e, const char* ws_d, const char* ws_z, void* dq,
                       void* dk, float* dg, float* dbeta, hipStream_t stream);

}  // namespace gdr

size_t gdr_fwd_workspace_bytes(int nseq, int T, int Hv, int dk, int dv, bool packed) {
    (void)dk;
    (void)dv;
    return (size_t)(gdr::slots_of(nseq, T, packed) * Hv * gdr::prep_bytes(false));
}

size_t gdr_bwd_workspace_bytes(int nseq, int T, int Hv, int dk, int dv, bool packed) {
    return (size_t)(gdr::slots_of(nseq, T, packed) * Hv *
                    (gdr::prep_bytes(true) + 2 * gdr::state_bytes(dk, dv) + 2 * gdr::rows_bytes(dv)));
}

static gdr::Args args_of(const GdrCall& c) { return gdr::Args{c.nseq, c.T, c.Hk, c.Hv, c.dv, c.cu, c.scale}; }

hipError_t launch_gdr_fwd(const GdrCall& c, void* o, float* S_T, void* workspace, hipStream_t stream) {
    const gdr::Args a = args_of(c);
    char* ws = (char*)workspace;
    hipError_t e = gdr::launch_prep(c.f32, c.dk, false, a, c.q, c.k, c.g, c.beta, ws, stream);
    if (e != hipSuccess) return e;
    return gdr::launch_chain(c.f32, c.dk, false, a, c.q, c.k, c.v, c.beta, c.S0, ws, gdr::prep_bytes(false), o, S_T, nullptr,
                             nullptr, stream);
}

hipError_t launch_gdr_bwd(const GdrCall& c, const void* dout, const float* dS_T, void* dq, void* dk, void* dv, float* dg,
                          float* dbeta, float* dS0, void* workspace, hipStream_t stream) {
    const gdr::Args a = args_of(c);
    const int64_t n = gdr::slots_of(c.nseq, c.T, c.cu != nullptr) * c.Hv;
    const int64_t pb = gdr::prep_bytes(true);
    char* prep = (char*)workspace;
    char* ws_s = prep + n * pb;
    char* ws_d = ws_s + n * gdr::state_bytes(c.dk, c.dv);
    char* ws_e = ws_d + n * gdr::state_bytes(c.dk, c.dv);
    char* ws_z = ws_e + n * gdr::rows_bytes(c.dv);
    hipError_t e = gdr::launch_prep(c.f32, c.dk, true, a, c.q, c.k, c.g, c.beta, prep, stream);
    if (e != hipSuccess) return e;
    e = gdr::launch_chain(c.f32, c.dk, true, a, c.q, c.k, c.v, c.beta, c.S0, prep, pb, nullptr, nullptr, ws_s, ws_e, stream);
    if (e != hipSuccess) return e;
    e = gdr::launch_back(c.f32, c.dk, a, c.q, c.k, dout, c.beta, dS_T, prep, pb, dv, dS0, ws_d, ws_z, stream);
    if (e != hipSuccess) return e;
    return gdr::launch_grad(c.f32, c.dk, a, c.q, c.k, c.beta, dout, prep, ws_s, ws_e, ws_d, ws_z, dq, dk, dg, dbeta, stream);
}

}  // namespace kda
