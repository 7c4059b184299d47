// kda_api.cpp -- the C ABI of libkda (declared in include/kda.h).
//
// Every entry point validates all of its arguments on the host first (sizes,
// dtype, NULL pointers, 16-byte alignment, overlaps, workspace size) and only
// then touches HIP, so a rejected call enqueues nothing.  Problems are
// reported as kda_status codes plus a thread-local message.
#include <hip/hip_runtime.h>

#include <stdarg.h>
#include <stdint.h>
#include <stdio.h>

#include <mutex>

#include "kda.h"
#include "kda_launch.hpp"

// Device scratch of kda_chunk_fwd_noalloc: the workspace of a segmented
// prefill (segment maps, segment start states, every chunk's T') for callers
// that cannot allocate.  Each device holds its own copy from the first call on
// it until the process ends.  In host code `scratch` names a host-side
// stand-in, never the device memory: kernels and copies get the per-device
// address that hipGetSymbolAddress returns (scratch_on_current_device).
static __device__ __align__(256) unsigned char scratch[KDA_NOALLOC_SCRATCH_BYTES];

namespace {

// Device addresses of `scratch`, one per device, resolved once per device.
constexpr int kMaxDevices = 64;
std::mutex g_scratch_mu;
void* g_scratch_ptr[kMaxDevices] = {};

thread_local char g_last_error[512] = "";

int fail(int status, const char* fmt, ...) {
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(g_last_error, sizeof(g_last_error), fmt, ap);
    va_end(ap);
    return status;
}

int ok() {
    g_last_error[0] = '\0';
    return KDA_OK;
}

bool supported_d(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

struct Range {
    const char* name;
    uintptr_t lo, hi;   // [lo, hi); empty when the pointer is NULL
};

Range rng(const char* name, const void* p, size_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Range{name, a, p ? a + bytes : a};
}

bool overlap(const Range& a, const Range& b) {
    if (a.lo == a.hi || b.lo == b.hi) return false;
    return a.lo < b.hi && b.lo < a.hi;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Product of sizes must stay far inside int64 for the kernels' index math.
bool sizes_fit(int64_t a, int64_t b, int64_t c, int64_t d) {
    const double x = (double)a * (double)b * (double)c * (double)d;
    return x < 4.0e18;
}

// The size limits every entry point and size query applies (after check_common).
int check_sizes(int B, int T, int H, int dk) {
    if (T < 1) return fail(KDA_ERR_SHAPE, "T=%d must be >= 1", T);
    if (!sizes_fit(B, T, H, dk)) return fail(KDA_ERR_SHAPE, "B*T*H*d too large");
    // a chunk of one fp32 [B, T, H, d] tensor, 16*H*d*4 bytes, is addressed with
    // 32-bit offsets
    if ((int64_t)H * dk * KDA_CHUNK * 4 >= (1LL << 32))
        return fail(KDA_ERR_SHAPE, "H*d=%lld too large (64*H*d must stay below 2^32)", (long long)H * dk);
    return KDA_OK;
}

int check_common(int dtype, int B, int H, int dk, int dv) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return fail(KDA_ERR_DTYPE, "unknown dtype %d", dtype);
    if (B < 1 || H < 1) return fail(KDA_ERR_SHAPE, "B=%d H=%d must be >= 1", B, H);
    if (!supported_d(dk) || dk != dv)
        return fail(KDA_ERR_SHAPE, "dk=%d dv=%d: need dk == dv in {16, 32, 64, 128}", dk, dv);
    return KDA_OK;
}

// Alignment of every pointer that is not NULL, and no output over an input or another output.
int check_ranges(const Range* in, int nin, const Range* out, int nout) {
    for (int i = 0; i < nin + nout; ++i) {
        const Range& r = i < nin ? in[i] : out[i - nin];
        if (r.lo & 15u) return fail(KDA_ERR_ALIGN, "%s is not 16-byte aligned", r.name);
    }
    for (int o = 0; o < nout; ++o) {
        for (int i = 0; i < nin; ++i)
            if (overlap(out[o], in[i])) return fail(KDA_ERR_ALIAS, "%s overlaps %s", out[o].name, in[i].name);
        for (int p = 0; p < o; ++p)
            if (overlap(out[o], out[p])) return fail(KDA_ERR_ALIAS, "%s overlaps %s", out[o].name, out[p].name);
    }
    return KDA_OK;
}

// Sizes of the gated delta rule with one decay a head: `a` sequences or rows of T tokens.
int check_gdr(int dtype, int a, int T, int Hk, int Hv, int dk, int dv, float scale) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return fail(KDA_ERR_DTYPE, "unknown dtype %d", dtype);
    if (a < 1 || T < 1 || Hk < 1) return fail(KDA_ERR_SHAPE, "sequences=%d T=%d Hk=%d must be >= 1", a, T, Hk);
    if (Hv < Hk || Hv % Hk) return fail(KDA_ERR_SHAPE, "Hv=%d must be a multiple of Hk=%d", Hv, Hk);
    if (dk != 32 && dk != 64 && dk != 128) return fail(KDA_ERR_SHAPE, "dk=%d not in {32, 64, 128}", dk);
    if (dv < 32 || dv > 256 || dv % 32) return fail(KDA_ERR_SHAPE, "dv=%d must be a multiple of 32 from 32 to 256", dv);
    if (!(scale - scale == 0.0f)) return fail(KDA_ERR_SHAPE, "scale must be finite");
    if (!sizes_fit(a, T, Hv, 256)) return fail(KDA_ERR_SHAPE, "sequences*T*Hv too large");
    return KDA_OK;
}

}  // namespace

extern "C" {

const char* kda_status_string(int status) {
    switch (status) {
        case KDA_OK: return "ok";
        case KDA_ERR_NULL: return "a required pointer is NULL";
        case KDA_ERR_SHAPE: return "unsupported or inconsistent sizes";
        case KDA_ERR_DTYPE: return "unknown dtype";
        case KDA_ERR_ALIGN: return "pointer not 16-byte aligned";
        case KDA_ERR_WORKSPACE: return "workspace missing or too small";
        case KDA_ERR_ALIAS: return "output overlaps an input";
        case KDA_ERR_HIP: return "HIP runtime error";
    }
    return "unknown status";
}

const char* kda_last_error(void) { return g_last_error; }

int kda_abi_version(void) { return KDA_ABI_VERSION; }

int kda_chunk_fwd_auto_segments(int B, int T, int H, int dk, int dv) {
    if (B < 1 || T < 1 || H < 1 || !supported_d(dk) || dk != dv) return 0;
    if (check_sizes(B, T, H, dk) != KDA_OK) return 0;
    // The map and output passes run one workgroup per compute unit: aim for one
    // resident round of 256 workgroups (every head of a run of segments at once;
    // at least two segments below 512 sequences, where the single-segment kernel,
    // two workgroups per compute unit, would leave the chip half empty), keeping
    // every segment at least 16 chunks long.
    const int64_t bh = (int64_t)B * H;
    const int64_t nchunks = ((int64_t)T + KDA_CHUNK - 1) / KDA_CHUNK;
    if (bh >= 512) return 1;
    int64_t want = (256 + bh - 1) / bh;
    if (want < 2) want = 2;
    int64_t cap = nchunks / 16;
    if (cap < 1) cap = 1;
    if (want > cap) want = cap;
    return (int)kda::plan_segments(T, (int)want).nseg;
}

int kda_chunk_fwd_workspace_size(int B, int T, int H, int dk, int dv, int segments, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_NULL, "bytes is NULL");
    int st = check_common(KDA_BF16, B, H, dk, dv);
    if (st) return st;
    if ((st = check_sizes(B, T, H, dk))) return st;
    const int nchunks = (int)(((int64_t)T + KDA_CHUNK - 1) / KDA_CHUNK);
    if (segments < 0 || segments > nchunks)
        return fail(KDA_ERR_SHAPE, "segments=%d outside [0, %d]", segments, nchunks);
    const int req = segments ? segments : kda_chunk_fwd_auto_segments(B, T, H, dk, dv);
    const kda::SegPlan p = kda::plan_segments(T, req);
    *bytes = kda::chunk_workspace_bytes(B, H, dk, dv, p.nseg, p.nchunks);
    return ok();
}

// The address of `scratch` on the calling thread's current device (resolved
// with that device current on its first use there).
static int scratch_on_current_device(void** out) {
    int dev = -1;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "hipGetDevice failed: %s", hipGetErrorString(e));
    if (dev < 0 || dev >= kMaxDevices) return fail(KDA_ERR_HIP, "device %d outside [0, %d)", dev, kMaxDevices);
    std::lock_guard<std::mutex> lock(g_scratch_mu);
    if (!g_scratch_ptr[dev]) {
        void* p = nullptr;
        e = hipGetSymbolAddress(&p, HIP_SYMBOL(scratch));
        if (e != hipSuccess || !p)
            return fail(KDA_ERR_HIP, "hipGetSymbolAddress(scratch) failed on device %d: %s", dev,
                        hipGetErrorString(e));
        g_scratch_ptr[dev] = p;
    }
    *out = g_scratch_ptr[dev];
    return KDA_OK;
}

// kda_chunk_fwd, kda_chunk_fwd_gated, kda_chunk_fwd_unbounded and
// kda_chunk_fwd_noalloc; z (the output gate's pre-activation) is NULL but for
// the gated call.  noalloc: the workspace is the current device's static
// scratch instead of the caller's (workspace is then NULL and workspace_bytes 0).
static int chunk_fwd_impl(int dtype, int B, int T, int H, int dk, int dv, int segments, const void* q,
                          const void* k, const void* v, const float* theta, const float* beta,
                          const float* S0, const void* z, void* o, float* S_T, void* workspace,
                          size_t workspace_bytes, void* stream, bool unbounded = false,
                          bool noalloc = false) {
    int st = check_common(dtype, B, H, dk, dv);
    if (st) return st;
    if ((st = check_sizes(B, T, H, dk))) return st;
    const int nchunks = (int)(((int64_t)T + KDA_CHUNK - 1) / KDA_CHUNK);
    if (segments < 0 || segments > nchunks)
        return fail(KDA_ERR_SHAPE, "segments=%d outside [0, %d]", segments, nchunks);
    if (!q || !k || !v || !theta || !beta || !o)
        return fail(KDA_ERR_NULL, "q, k, v, theta, beta and o must be non-NULL");
    const void* all[] = {q, k, v, theta, beta, S0, o, S_T, workspace, z};
    const char* names[] = {"q", "k", "v", "theta", "beta", "S0", "o", "S_T", "workspace", "z"};
    for (int i = 0; i < 10; ++i)
        if (all[i] && !aligned16(all[i])) return fail(KDA_ERR_ALIGN, "%s is not 16-byte aligned", names[i]);

    const int req = segments ? segments : kda_chunk_fwd_auto_segments(B, T, H, dk, dv);
    const kda::SegPlan plan = kda::plan_segments(T, req);
    const size_t need = kda::chunk_workspace_bytes(B, H, dk, dv, plan.nseg, plan.nchunks);
    if (noalloc) {
        if (need > (size_t)KDA_NOALLOC_SCRATCH_BYTES)
            return fail(KDA_ERR_WORKSPACE,
                        "%d segments need %zu bytes of scratch, more than the static %zu; pass fewer "
                        "segments (1 needs none) or call kda_chunk_fwd with a workspace",
                        plan.nseg, need, (size_t)KDA_NOALLOC_SCRATCH_BYTES);
    } else if (need > 0 && (!workspace || workspace_bytes < need)) {
        return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu%s", need,
                    workspace_bytes, workspace ? "" : " (NULL)");
    }

    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    const size_t tok = (size_t)B * T * H;
    const size_t st_bytes = (size_t)B * H * dk * dv * 4;
    const Range in[] = {rng("q", q, tok * dk * es), rng("k", k, tok * dk * es), rng("v", v, tok * dv * es),
                        rng("theta", theta, tok * dk * 4), rng("beta", beta, tok * 4),
                        rng("S0", S0, S0 ? st_bytes : 0), rng("z", z, z ? tok * dv * es : 0)};
    const Range r_o = rng("o", o, tok * dv * es);
    const Range r_st = rng("S_T", S_T, S_T ? st_bytes : 0);
    const Range r_ws = rng("workspace", workspace, need);
    for (const Range& x : in) {
        if (overlap(r_o, x)) return fail(KDA_ERR_ALIAS, "o overlaps %s", x.name);
        if (overlap(r_ws, x)) return fail(KDA_ERR_ALIAS, "workspace overlaps %s", x.name);
        if (overlap(r_st, x) && !(x.name[0] == 'S' && (const void*)S0 == (const void*)S_T))
            return fail(KDA_ERR_ALIAS, "S_T overlaps %s (only S_T == S0 is allowed)", x.name);
    }
    if (overlap(r_o, r_st)) return fail(KDA_ERR_ALIAS, "o overlaps S_T");
    if (overlap(r_o, r_ws)) return fail(KDA_ERR_ALIAS, "o overlaps workspace");
    if (overlap(r_st, r_ws)) return fail(KDA_ERR_ALIAS, "S_T overlaps workspace");

    if (noalloc && need > 0) {   // every argument check is done: now the first HIP call
        st = scratch_on_current_device(&workspace);
        if (st) return st;
    }
    hipError_t e = kda::launch_chunk_fwd(dtype == KDA_F32, B, T, H, dk, plan, q, k, v, theta, beta, S0,
                                         z, o, S_T, need ? workspace : nullptr,
                                         reinterpret_cast<hipStream_t>(stream), unbounded);
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

int kda_chunk_fwd(int dtype, int B, int T, int H, int dk, int dv, int segments, const void* q,
                  const void* k, const void* v, const float* theta, const float* beta,
                  const float* S0, void* o, float* S_T, void* workspace, size_t workspace_bytes,
                  void* stream) {
    return chunk_fwd_impl(dtype, B, T, H, dk, dv, segments, q, k, v, theta, beta, S0, nullptr, o, S_T,
                          workspace, workspace_bytes, stream);
}

int kda_chunk_fwd_noalloc(int dtype, int B, int T, int H, int dk, int dv, int segments, const void* q,
                          const void* k, const void* v, const float* theta, const float* beta,
                          const float* S0, void* o, float* S_T, void* stream) {
    return chunk_fwd_impl(dtype, B, T, H, dk, dv, segments, q, k, v, theta, beta, S0, nullptr, o, S_T,
                          nullptr, 0, stream, false, true);
}

int kda_chunk_fwd_gated(int dtype, int B, int T, int H, int dk, int dv, int segments, const void* q,
                        const void* k, const void* v, const float* theta, const float* beta,
                        const float* S0, const void* z, void* o, float* S_T, void* workspace,
                        size_t workspace_bytes, void* stream) {
    if (!z) return fail(KDA_ERR_NULL, "z must be non-NULL");
    return chunk_fwd_impl(dtype, B, T, H, dk, dv, segments, q, k, v, theta, beta, S0, z, o, S_T,
                          workspace, workspace_bytes, stream);
}

int kda_chunk_fwd_unbounded(int dtype, int B, int T, int H, int dk, int dv, const void* q, const void* k,
                            const void* v, const float* theta, const float* beta, const float* S0,
                            void* o, float* S_T, void* stream) {
    return chunk_fwd_impl(dtype, B, T, H, dk, dv, 1, q, k, v, theta, beta, S0, nullptr, o, S_T, nullptr, 0,
                          stream, true);
}

int kda_chunk_bwd_workspace_size(int B, int T, int H, int dk, int dv, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_NULL, "bytes is NULL");
    int st = check_common(KDA_BF16, B, H, dk, dv);
    if (st) return st;
    if ((st = check_sizes(B, T, H, dk))) return st;
    *bytes = kda::chunk_bwd_workspace_bytes(B, T, H, dk);
    return ok();
}

int kda_chunk_bwd(int dtype, int B, int T, int H, int dk, int dv, const void* q, const void* k,
                  const void* v, const float* theta, const float* beta, const float* S0, const void* dout,
                  const float* dS_T, float* dq, float* dkk, float* dvv, float* dtheta, float* dbeta,
                  float* dS0, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_common(dtype, B, H, dk, dv);
    if (st) return st;
    if ((st = check_sizes(B, T, H, dk))) return st;
    if (!q || !k || !v || !theta || !beta || !dout || !dq || !dkk || !dvv || !dtheta || !dbeta)
        return fail(KDA_ERR_NULL, "q, k, v, theta, beta, do and every gradient but dS0 must be non-NULL");
    const void* all[] = {q, k, v, theta, beta, S0, dout, dS_T, dq, dkk, dvv, dtheta, dbeta, dS0, workspace};
    const char* names[] = {"q", "k", "v", "theta", "beta", "S0", "do", "dS_T", "dq", "dk", "dv",
                           "dtheta", "dbeta", "dS0", "workspace"};
    for (int i = 0; i < 15; ++i)
        if (all[i] && !aligned16(all[i])) return fail(KDA_ERR_ALIGN, "%s is not 16-byte aligned", names[i]);
    const size_t need = kda::chunk_bwd_workspace_bytes(B, T, H, dk);
    if (!workspace || workspace_bytes < need)
        return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu%s", need, workspace_bytes,
                    workspace ? "" : " (NULL)");
    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    const size_t tok = (size_t)B * T * H;
    const size_t st_bytes = (size_t)B * H * dk * dv * 4;
    const Range in[] = {rng("q", q, tok * dk * es), rng("k", k, tok * dk * es), rng("v", v, tok * dv * es),
                        rng("theta", theta, tok * dk * 4), rng("beta", beta, tok * 4),
                        rng("S0", S0, S0 ? st_bytes : 0), rng("do", dout, tok * dv * es),
                        rng("dS_T", dS_T, dS_T ? st_bytes : 0)};
    const Range out[] = {rng("dq", dq, tok * dk * 4), rng("dk", dkk, tok * dk * 4), rng("dv", dvv, tok * dv * 4),
                         rng("dtheta", dtheta, tok * dk * 4), rng("dbeta", dbeta, tok * 4),
                         rng("dS0", dS0, dS0 ? st_bytes : 0), rng("workspace", workspace, need)};
    for (const Range& o : out) {
        for (const Range& x : in)
            if (overlap(o, x)) return fail(KDA_ERR_ALIAS, "%s overlaps %s", o.name, x.name);
        for (const Range& o2 : out)
            if (&o2 != &o && overlap(o, o2)) return fail(KDA_ERR_ALIAS, "%s overlaps %s", o.name, o2.name);
    }
    hipError_t e = kda::launch_chunk_bwd(dtype == KDA_F32, B, T, H, dk, q, k, v, theta, beta, S0, dout, dS_T,
                                         dq, dkk, dvv, dtheta, dbeta, dS0, workspace,
                                         reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

// kda_decode_step and kda_decode_step_gated; z is NULL for the former.
static int decode_step_impl(int dtype, int B, int H, int dk, int dv, const void* q, const void* k,
                            const void* v, const float* theta, const float* beta, float* S,
                            const void* z, void* o, void* stream) {
    int st = check_common(dtype, B, H, dk, dv);
    if (st) return st;
    if (!sizes_fit(B, H, dk, dv) || (int64_t)B * H > 0x7fffffffLL)
        return fail(KDA_ERR_SHAPE, "B*H too large");
    if (!q || !k || !v || !theta || !beta || !S || !o)
        return fail(KDA_ERR_NULL, "q, k, v, theta, beta, S and o must be non-NULL");
    const void* all[] = {q, k, v, theta, beta, S, o, z};
    const char* names[] = {"q", "k", "v", "theta", "beta", "S", "o", "z"};
    for (int i = 0; i < 8; ++i)
        if (all[i] && !aligned16(all[i])) return fail(KDA_ERR_ALIGN, "%s is not 16-byte aligned", names[i]);
    const size_t es = dtype == KDA_BF16 ? 2 : 4;
    const size_t bh = (size_t)B * H;
    const Range in[] = {rng("q", q, bh * dk * es), rng("k", k, bh * dk * es), rng("v", v, bh * dv * es),
                        rng("theta", theta, bh * dk * 4), rng("beta", beta, bh * 4),
                        rng("z", z, z ? bh * dv * es : 0)};
    const Range r_s = rng("S", S, bh * dk * dv * 4);
    const Range r_o = rng("o", o, bh * dv * es);
    for (const Range& x : in) {
        if (overlap(r_o, x)) return fail(KDA_ERR_ALIAS, "o overlaps %s", x.name);
        if (overlap(r_s, x)) return fail(KDA_ERR_ALIAS, "S overlaps %s", x.name);
    }
    if (overlap(r_o, r_s)) return fail(KDA_ERR_ALIAS, "o overlaps S");

    hipError_t e = kda::launch_decode(dtype == KDA_F32, B, H, dk, q, k, v, theta, beta, S, z, o,
                                      reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

int kda_decode_step(int dtype, int B, int H, int dk, int dv, const void* q, const void* k,
                    const void* v, const float* theta, const float* beta, float* S, void* o,
                    void* stream) {
    return decode_step_impl(dtype, B, H, dk, dv, q, k, v, theta, beta, S, nullptr, o, stream);
}

int kda_decode_step_gated(int dtype, int B, int H, int dk, int dv, const void* q, const void* k,
                          const void* v, const float* theta, const float* beta, float* S,
                          const void* z, void* o, void* stream) {
    if (!z) return fail(KDA_ERR_NULL, "z must be non-NULL");
    return decode_step_impl(dtype, B, H, dk, dv, q, k, v, theta, beta, S, z, o, stream);
}

int kda_gate(int B, int T, int H, int dk, const float* theta, float* g, float* g_cum, void* stream) {
    if (B < 1 || T < 1 || H < 1) return fail(KDA_ERR_SHAPE, "B=%d T=%d H=%d must be >= 1", B, T, H);
    if (!supported_d(dk)) return fail(KDA_ERR_SHAPE, "dk=%d not in {16, 32, 64, 128}", dk);
    if (int st = check_sizes(B, T, H, dk)) return st;
    if (!theta) return fail(KDA_ERR_NULL, "theta is NULL");
    if (!g && !g_cum) return fail(KDA_ERR_NULL, "both g and g_cum are NULL");
    const void* all[] = {theta, g, g_cum};
    const char* names[] = {"theta", "g", "g_cum"};
    for (int i = 0; i < 3; ++i)
        if (all[i] && !aligned16(all[i])) return fail(KDA_ERR_ALIGN, "%s is not 16-byte aligned", names[i]);
    const size_t n = (size_t)B * T * H * dk * 4;
    const Range rt = rng("theta", theta, n), rg_ = rng("g", g, g ? n : 0), rc = rng("g_cum", g_cum, g_cum ? n : 0);
    if (overlap(rg_, rt) || overlap(rc, rt)) return fail(KDA_ERR_ALIAS, "g or g_cum overlaps theta");
    if (overlap(rg_, rc)) return fail(KDA_ERR_ALIAS, "g overlaps g_cum");

    hipError_t e = kda::launch_gate(B, T, H, dk, theta, g, g_cum, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

// ---------------------------------------------------------------- one decay a head
int kda_gdr_step(int dtype, int B, int T, int Hk, int Hv, int dk, int dv, int nslot, float scale, const void* q,
                 const void* k, const void* v, const float* g, const float* beta, float* S, const int* slots,
                 const int* ntok, void* o, void* stream) {
    int st = check_gdr(dtype, B, T, Hk, Hv, dk, dv, scale);
    if (st) return st;
    if (nslot < 1 || (!slots && nslot < B))
        return fail(KDA_ERR_SHAPE, "nslot=%d states for B=%d rows%s", nslot, B, slots ? "" : " without slots");
    if (!sizes_fit(nslot, Hv, dk, dv) || (int64_t)B * Hv * (dv / 32) >= 1LL << 26)   // workgroups of 64 threads
        return fail(KDA_ERR_SHAPE, "B*Hv or nslot*Hv too large");
    if (!q || !k || !v || !g || !beta || !S || !o)
        return fail(KDA_ERR_NULL, "q, k, v, g, beta, S and o must be non-NULL");
    const size_t es = dtype == KDA_BF16 ? 2 : 4, tok = (size_t)B * T;
    const Range in[] = {rng("q", q, tok * Hk * dk * es), rng("k", k, tok * Hk * dk * es), rng("v", v, tok * Hv * dv * es),
                        rng("g", g, tok * Hv * 4), rng("beta", beta, tok * Hv * 4), rng("slots", slots, (size_t)B * 4),
                        rng("ntok", ntok, (size_t)B * 4)};
    const Range out[] = {rng("S", S, (size_t)nslot * Hv * dk * dv * 4), rng("o", o, tok * Hv * dv * es)};
    if ((st = check_ranges(in, 7, out, 2))) return st;
    hipError_t e = kda::launch_gdr_step(dtype == KDA_F32, B, T, Hk, Hv, dk, dv, nslot, scale, q, k, v, g, beta, S, slots,
                                        ntok, o, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

static int check_gdr_chunk(int dtype, int nseq, int T, int Hk, int Hv, int dk, int dv, float scale, bool packed) {
    int st = check_gdr(dtype, nseq, T, Hk, Hv, dk, dv, scale);
    if (st) return st;
    // A launch has at most 2^32 threads.  The preparation has 256 a chunk and head.  Two walks
    // together have eight a column, up to 2^11 a sequence and head, and as many again for each of
    // the pieces, of which there are 512 heads' at most (two for each of 256 compute units); a join has up to 2^14
    // for each head of a sequence that may be cut, 256 at most.
    const int64_t slots = packed ? (int64_t)T / 64 + nseq : (int64_t)nseq * (((int64_t)T + 63) / 64);
    if (slots >= (1LL << 24) / Hv || (int64_t)nseq * Hv >= 1LL << 20)
        return fail(KDA_ERR_SHAPE, "sequences*chunks*Hv too large");
    // a chunk of one tensor, 64*H*d*4 bytes at most, is addressed with 32-bit offsets
    if ((int64_t)Hk * dk >= (1LL << 23) || (int64_t)Hv * dv >= (1LL << 23))
        return fail(KDA_ERR_SHAPE, "Hk*dk=%lld or Hv*dv=%lld too large (256*H*d must stay below 2^31)", (long long)Hk * dk,
                    (long long)Hv * dv);
    return KDA_OK;
}

static int gdr_workspace_size(bool bwd, int nseq, int T, int Hv, int dk, int dv, int packed, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_NULL, "bytes is NULL");
    int st = check_gdr_chunk(KDA_BF16, nseq, T, 1, Hv, dk, dv, 1.0f, packed != 0);
    if (st) return st;
    *bytes = bwd ? kda::gdr_bwd_workspace_bytes(nseq, T, Hv, dk, dv, packed != 0)
                 : kda::gdr_fwd_workspace_bytes(nseq, T, Hv, dk, dv, packed != 0);
    return ok();
}

int kda_gdr_chunk_fwd_workspace_size(int nseq, int T, int Hv, int dk, int dv, int packed, size_t* bytes) {
    return gdr_workspace_size(false, nseq, T, Hv, dk, dv, packed, bytes);
}

int kda_gdr_chunk_bwd_workspace_size(int nseq, int T, int Hv, int dk, int dv, int packed, size_t* bytes) {
    return gdr_workspace_size(true, nseq, T, Hv, dk, dv, packed, bytes);
}

int kda_gdr_chunk_fwd(int dtype, int nseq, int T, int Hk, int Hv, int dk, int dv, float scale, const int* cu_seqlens,
                      const void* q, const void* k, const void* v, const float* g, const float* beta, const float* S0,
                      void* o, float* S_T, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_gdr_chunk(dtype, nseq, T, Hk, Hv, dk, dv, scale, cu_seqlens != nullptr);
    if (st) return st;
    if (!q || !k || !v || !g || !beta || !o) return fail(KDA_ERR_NULL, "q, k, v, g, beta and o must be non-NULL");
    const size_t need = kda::gdr_fwd_workspace_bytes(nseq, T, Hv, dk, dv, cu_seqlens != nullptr);
    if (!workspace || workspace_bytes < need)
        return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu%s", need, workspace_bytes,
                    workspace ? "" : " (NULL)");
    const size_t es = dtype == KDA_BF16 ? 2 : 4, tok = cu_seqlens ? (size_t)T : (size_t)nseq * T;
    const size_t sb = (size_t)nseq * Hv * dk * dv * 4;
    const Range in[] = {rng("q", q, tok * Hk * dk * es), rng("k", k, tok * Hk * dk * es), rng("v", v, tok * Hv * dv * es),
                        rng("g", g, tok * Hv * 4), rng("beta", beta, tok * Hv * 4),
                        rng("cu_seqlens", cu_seqlens, ((size_t)nseq + 1) * 4), rng("S0", S0 == S_T ? nullptr : S0, sb)};
    const Range out[] = {rng("o", o, tok * Hv * dv * es), rng("S_T", S_T, sb), rng("workspace", workspace, need)};
    if ((st = check_ranges(in, 7, out, 3))) return st;
    const kda::GdrCall c{dtype == KDA_F32, nseq, T, Hk, Hv, dk, dv, cu_seqlens, scale, q, k, v, g, beta, S0};
    hipError_t e = kda::launch_gdr_fwd(c, o, S_T, workspace, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

int kda_gdr_chunk_bwd(int dtype, int nseq, int T, int Hk, int Hv, int dk, int dv, float scale, const int* cu_seqlens,
                      const void* q, const void* k, const void* v, const float* g, const float* beta, const float* S0,
                      const void* dout, const float* dS_T, void* dq, void* dkk, void* dvv, float* dg, float* dbeta,
                      float* dS0, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_gdr_chunk(dtype, nseq, T, Hk, Hv, dk, dv, scale, cu_seqlens != nullptr);
    if (st) return st;
    if (!q || !k || !v || !g || !beta || !dout || !dq || !dkk || !dvv || !dg || !dbeta)
        return fail(KDA_ERR_NULL, "q, k, v, g, beta, do and every gradient but dS0 must be non-NULL");
    const size_t need = kda::gdr_bwd_workspace_bytes(nseq, T, Hv, dk, dv, cu_seqlens != nullptr);
    if (!workspace || workspace_bytes < need)
        return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu%s", need, workspace_bytes,
                    workspace ? "" : " (NULL)");
    const size_t es = dtype == KDA_BF16 ? 2 : 4, tok = cu_seqlens ? (size_t)T : (size_t)nseq * T;
    const size_t sb = (size_t)nseq * Hv * dk * dv * 4, nq = tok * Hk * dk * es, nv = tok * Hv * dv * es, ng = tok * Hv * 4;
    const Range in[] = {rng("q", q, nq), rng("k", k, nq), rng("v", v, nv), rng("g", g, ng), rng("beta", beta, ng),
                        rng("cu_seqlens", cu_seqlens, ((size_t)nseq + 1) * 4), rng("S0", S0, sb), rng("do", dout, nv),
                        rng("dS_T", dS_T, sb)};
    const Range out[] = {rng("dq", dq, nq), rng("dk", dkk, nq), rng("dv", dvv, nv), rng("dg", dg, ng),
                         rng("dbeta", dbeta, ng), rng("dS0", dS0, sb), rng("workspace", workspace, need)};
    if ((st = check_ranges(in, 9, out, 7))) return st;
    const kda::GdrCall c{dtype == KDA_F32, nseq, T, Hk, Hv, dk, dv, cu_seqlens, scale, q, k, v, g, beta, S0};
    hipError_t e = kda::launch_gdr_bwd(c, dout, dS_T, dq, dkk, dvv, dg, dbeta, dS0, workspace,
                                       reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

int kda_gdr_clear_rows(int nseq, int T, const int* cu_seqlens, int n, void* const* tensors, const size_t* row_bytes,
                       void* stream) {
    if (nseq < 1 || T < 1) return fail(KDA_ERR_SHAPE, "sequences=%d T=%d must be >= 1", nseq, T);
    if (n < 1 || n > kda::GDR_CLEAR_MAX) return fail(KDA_ERR_SHAPE, "n=%d tensors outside [1, %d]", n, kda::GDR_CLEAR_MAX);
    if (!cu_seqlens || !tensors || !row_bytes) return fail(KDA_ERR_NULL, "cu_seqlens, tensors and row_bytes must be non-NULL");
    Range out[kda::GDR_CLEAR_MAX];
    for (int i = 0; i < n; ++i) {
        if (!tensors[i]) return fail(KDA_ERR_NULL, "tensor %d is NULL", i);
        if (row_bytes[i] < 4 || row_bytes[i] % 4 || row_bytes[i] >= (size_t)1 << 31)
            return fail(KDA_ERR_SHAPE, "rows of %zu bytes: must be a multiple of 4 below 2^31", row_bytes[i]);
        out[i] = rng("tensor", tensors[i], (size_t)T * row_bytes[i]);
    }
    const Range in[] = {rng("cu_seqlens", cu_seqlens, ((size_t)nseq + 1) * 4)};
    if (int st = check_ranges(in, 1, out, n)) return st;
    hipError_t e = kda::launch_gdr_clear(nseq, T, cu_seqlens, n, tensors, row_bytes, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

// ---------------------------------------------------------------- block norm
static int check_norm(int dtype, int act, long long rows, int D, float eps) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return fail(KDA_ERR_DTYPE, "unknown dtype %d", dtype);
    if (act != KDA_ACT_SIGMOID && act != KDA_ACT_SILU) return fail(KDA_ERR_SHAPE, "unknown act %d", act);
    if (rows < 1 || rows > (1LL << 40)) return fail(KDA_ERR_SHAPE, "rows=%lld outside [1, 2^40]", rows);
    if (D < 8 || D > 8192 || D % 8) return fail(KDA_ERR_SHAPE, "D=%d must be a multiple of 8 from 8 to 8192", D);
    if (!(eps >= 0.0f) || eps > 1.0f) return fail(KDA_ERR_SHAPE, "eps=%g outside [0, 1]", (double)eps);
    return KDA_OK;
}

int kda_block_norm_fwd(int dtype, int act, long long rows, int D, float eps, const void* y, const void* x, const void* z,
                       const float* w_post, const float* s, const float* w_pre, void* r, void* h, void* stream) {
    int st = check_norm(dtype, act, rows, D, eps);
    if (st) return st;
    if (!y || !r) return fail(KDA_ERR_NULL, "y and r must be non-NULL");
    if (!w_pre != !h) return fail(KDA_ERR_NULL, "h and w_pre go together: both or neither may be NULL");
    const size_t n = (size_t)rows * D * (dtype == KDA_BF16 ? 2 : 4), w = (size_t)D * 4;
    // r may be x itself: the residual stream updated in place
    const Range in[] = {rng("y", y, n), rng("z", z, n), rng("w_post", w_post, w), rng("s", s, w), rng("w_pre", w_pre, w),
                        rng("x", x == r ? nullptr : x, n)};
    const Range out[] = {rng("r", r, n), rng("h", h, n)};
    if ((st = check_ranges(in, 6, out, 2))) return st;
    hipError_t e = kda::launch_norm_fwd(dtype == KDA_F32, rows, D, eps, act == KDA_ACT_SILU, y, x, z, w_post, s, w_pre, r,
                                        h, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

int kda_block_norm_bwd_workspace_size(long long rows, int D, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_NULL, "bytes is NULL");
    int st = check_norm(KDA_BF16, KDA_ACT_SIGMOID, rows, D, 0.0f);
    if (st) return st;
    *bytes = kda::norm_bwd_workspace_bytes(rows, D);
    return ok();
}

int kda_block_norm_bwd(int dtype, int act, long long rows, int D, float eps, const void* y, const void* x, const void* z,
                       const float* w_post, const float* s, const float* w_pre, const void* dr, const void* dh, void* dy,
                       void* dx, void* dz, float* dw_post, float* ds, float* dw_pre, void* workspace,
                       size_t workspace_bytes, void* stream) {
    int st = check_norm(dtype, act, rows, D, eps);
    if (st) return st;
    if (!y || !dy || (!dr && !dh)) return fail(KDA_ERR_NULL, "y, dy and one of dr and dh must be non-NULL");
    if (!w_pre != !dh) return fail(KDA_ERR_NULL, "dh and w_pre go together: both or neither may be NULL");
    if ((dx && !x) || (dz && !z) || (dw_post && !w_post) || (ds && !s) || (dw_pre && !w_pre))
        return fail(KDA_ERR_NULL, "a gradient is asked for of an input that is NULL");
    const size_t n = (size_t)rows * D * (dtype == KDA_BF16 ? 2 : 4), w = (size_t)D * 4;
    const size_t need = dw_post || ds || dw_pre ? kda::norm_bwd_workspace_bytes(rows, D) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu%s", need, workspace_bytes,
                    workspace ? "" : " (NULL)");
    const Range in[] = {rng("y", y, n), rng("x", x, n), rng("z", z, n), rng("w_post", w_post, w), rng("s", s, w),
                        rng("w_pre", w_pre, w), rng("dr", dr, n), rng("dh", dh, n)};
    const Range out[] = {rng("dy", dy, n), rng("dx", dx, n), rng("dz", dz, n), rng("dw_post", dw_post, w), rng("ds", ds, w),
                         rng("dw_pre", dw_pre, w), rng("workspace", need ? workspace : nullptr, need)};
    if ((st = check_ranges(in, 8, out, 7))) return st;
    hipError_t e = kda::launch_norm_bwd(dtype == KDA_F32, rows, D, eps, act == KDA_ACT_SILU, y, x, z, w_post, s, w_pre, dr,
                                        dh, dy, dx, dz, dw_post, ds, dw_pre, (float*)workspace,
                                        reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

// ---------------------------------------------------------------- selective scan
static int check_scan(int dtype, int a, int T, int D, int N, int G, int softplus) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return fail(KDA_ERR_DTYPE, "unknown dtype %d", dtype);
    if (a < 1 || T < 1) return fail(KDA_ERR_SHAPE, "sequences=%d T=%d must be >= 1", a, T);
    if (T > 1 << 30) return fail(KDA_ERR_SHAPE, "T=%d above 2^30", T);
    if (G < 1 || D < 8 || D > 1 << 20 || D % G || D / G % 8)
        return fail(KDA_ERR_SHAPE, "D=%d, G=%d: D must be at most 2^20 and D / G a multiple of 8", D, G);
    if (N != 8 && N != 16 && N != 32 && N != 64) return fail(KDA_ERR_SHAPE, "N=%d not in {8, 16, 32, 64}", N);
    if (softplus != 0 && softplus != 1) return fail(KDA_ERR_SHAPE, "softplus=%d must be 0 or 1", softplus);
    if (!sizes_fit(a, T, D, N)) return fail(KDA_ERR_SHAPE, "sequences*T*D*N too large");
    return KDA_OK;
}

// A launch has at most 2^32 threads, 256 a workgroup.
static int check_workgroups(int64_t n) {
    if (n >= 1LL << 24) return fail(KDA_ERR_SHAPE, "sequences, T and D need %lld workgroups: 2^24 is too many", (long long)n);
    return KDA_OK;
}

static int scan_workspace_size(bool bwd, int nseq, int T, int D, int N, int G, int packed, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_NULL, "bytes is NULL");
    int st = check_scan(KDA_BF16, nseq, T, D, N, G, 1);
    if (st) return st;
    if ((st = check_workgroups(bwd ? kda::scan_bwd_workgroups(nseq, T, D, G, packed != 0)
                                   : kda::scan_fwd_workgroups(nseq, T, D, G, packed != 0))))
        return st;
    *bytes = bwd ? kda::scan_bwd_workspace_bytes(nseq, T, D, N, G, packed != 0)
                 : kda::scan_fwd_workspace_bytes(nseq, T, D, N, G, packed != 0);
    return ok();
}

int kda_sel_scan_fwd_workspace_size(int nseq, int T, int D, int N, int G, int packed, size_t* bytes) {
    return scan_workspace_size(false, nseq, T, D, N, G, packed, bytes);
}

int kda_sel_scan_bwd_workspace_size(int nseq, int T, int D, int N, int G, int packed, size_t* bytes) {
    return scan_workspace_size(true, nseq, T, D, N, G, packed, bytes);
}

int kda_sel_scan_fwd(int dtype, int nseq, int T, int D, int N, int G, int softplus, const int* cu_seqlens, int zero_rest,
                     const void* x, const void* dt, const float* A, const void* b, const void* c, const float* skip, const void* z,
                     const float* dt_bias, const float* S0, void* y, float* S_T, void* workspace, size_t workspace_bytes,
                     void* stream) {
    int st = check_scan(dtype, nseq, T, D, N, G, softplus);
    if (st) return st;
    const bool packed = cu_seqlens != nullptr;
    if ((st = check_workgroups(kda::scan_fwd_workgroups(nseq, T, D, G, packed)))) return st;
    if (zero_rest != 0 && zero_rest != 1) return fail(KDA_ERR_SHAPE, "zero_rest=%d not in {0, 1}", zero_rest);
    if (!x || !dt || !A || !b || !c || !y) return fail(KDA_ERR_NULL, "x, dt, A, b, c and y must be non-NULL");
    const size_t need = kda::scan_fwd_workspace_bytes(nseq, T, D, N, G, packed);
    if (need && (!workspace || workspace_bytes < need))
        return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu%s", need, workspace_bytes,
                    workspace ? "" : " (NULL)");
    const size_t es = dtype == KDA_BF16 ? 2 : 4, tok = packed ? (size_t)T : (size_t)nseq * T;
    const size_t nx = tok * D * es, nb = tok * G * N * es, nd = (size_t)D * 4, ns = (size_t)nseq * D * N * 4;
    const Range in[] = {rng("x", x, nx), rng("dt", dt, nx), rng("A", A, nd * N), rng("b", b, nb), rng("c", c, nb),
                        rng("skip", skip, nd), rng("z", z, nx), rng("dt_bias", dt_bias, nd),
                        rng("cu_seqlens", cu_seqlens, ((size_t)nseq + 1) * 4), rng("S0", S0 == S_T ? nullptr : S0, ns)};
    const Range out[] = {rng("y", y, nx), rng("S_T", S_T, ns), rng("workspace", need ? workspace : nullptr, need)};
    if ((st = check_ranges(in, 10, out, 3))) return st;
    const kda::ScanCall call{dtype == KDA_F32, nseq, T, D, N, G, softplus != 0, cu_seqlens, x, dt, b, c, z, A, skip, dt_bias, S0};
    hipError_t e = kda::launch_scan_fwd(call, zero_rest != 0, y, S_T, need ? workspace : nullptr, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

int kda_sel_scan_bwd(int dtype, int nseq, int T, int D, int N, int G, int softplus, const int* cu_seqlens, const void* x,
                     const void* dt, const float* A, const void* b, const void* c, const float* skip, const void* z,
                     const float* dt_bias, const float* S0, const void* dy, const float* dS_T, void* dx, void* ddt, float* dA,
                     void* db, void* dc, float* dskip, void* dz, float* ddt_bias, float* dS0, void* workspace,
                     size_t workspace_bytes, void* stream) {
    int st = check_scan(dtype, nseq, T, D, N, G, softplus);
    if (st) return st;
    const bool packed = cu_seqlens != nullptr;
    if ((st = check_workgroups(kda::scan_bwd_workgroups(nseq, T, D, G, packed)))) return st;
    if (!x || !dt || !A || !b || !c || !dy || !dx || !ddt || !dA || !db || !dc)
        return fail(KDA_ERR_NULL, "x, dt, A, b, c, dy, dx, ddt, dA, db and dc must be non-NULL");
    if (!z != !dz || (dskip && !skip) || (ddt_bias && !dt_bias))
        return fail(KDA_ERR_NULL, "z and dz go together, and dskip and ddt_bias need skip and dt_bias");
    const size_t need = kda::scan_bwd_workspace_bytes(nseq, T, D, N, G, packed);
    if (!workspace || workspace_bytes < need)
        return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu%s", need, workspace_bytes,
                    workspace ? "" : " (NULL)");
    const size_t es = dtype == KDA_BF16 ? 2 : 4, tok = packed ? (size_t)T : (size_t)nseq * T;
    const size_t nx = tok * D * es, nb = tok * G * N * es, nd = (size_t)D * 4, ns = (size_t)nseq * D * N * 4;
    const Range in[] = {rng("x", x, nx), rng("dt", dt, nx), rng("A", A, nd * N), rng("b", b, nb), rng("c", c, nb),
                        rng("skip", skip, nd), rng("z", z, nx), rng("dt_bias", dt_bias, nd),
                        rng("cu_seqlens", cu_seqlens, ((size_t)nseq + 1) * 4), rng("S0", S0, ns), rng("dy", dy, nx),
                        rng("dS_T", dS_T, ns)};
    const Range out[] = {rng("dx", dx, nx), rng("ddt", ddt, nx), rng("dA", dA, nd * N), rng("db", db, nb), rng("dc", dc, nb),
                         rng("dskip", dskip, nd), rng("dz", dz, nx), rng("ddt_bias", ddt_bias, nd), rng("dS0", dS0, ns),
                         rng("workspace", workspace, need)};
    if ((st = check_ranges(in, 12, out, 10))) return st;
    const kda::ScanCall call{dtype == KDA_F32, nseq, T, D, N, G, softplus != 0, cu_seqlens, x, dt, b, c, z, A, skip, dt_bias, S0};
    hipError_t e = kda::launch_scan_bwd(call, dy, dS_T, dx, ddt, dA, db, dc, dskip, dz, ddt_bias, dS0, workspace,
                                        reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

int kda_sel_scan_step(int dtype, int B, int T, int D, int N, int G, int nslot, int softplus, const void* x, const void* dt,
                      const float* A, const void* b, const void* c, const float* skip, const void* z, const float* dt_bias,
                      float* S, const int* slots, const int* ntok, void* y, void* stream) {
    int st = check_scan(dtype, B, T, D, N, G, softplus);
    if (st) return st;
    if (nslot < 1 || (!slots && nslot < B))
        return fail(KDA_ERR_SHAPE, "nslot=%d states for B=%d rows%s", nslot, B, slots ? "" : " without slots");
    if (!sizes_fit(nslot, D, N, 1)) return fail(KDA_ERR_SHAPE, "nslot*D*N too large");
    if ((st = check_workgroups(kda::scan_step_workgroups(B, D, G)))) return st;
    if (!x || !dt || !A || !b || !c || !S || !y) return fail(KDA_ERR_NULL, "x, dt, A, b, c, S and y must be non-NULL");
    const size_t es = dtype == KDA_BF16 ? 2 : 4, tok = (size_t)B * T;
    const size_t nx = tok * D * es, nb = tok * G * N * es, nd = (size_t)D * 4;
    const Range in[] = {rng("x", x, nx), rng("dt", dt, nx), rng("A", A, nd * N), rng("b", b, nb), rng("c", c, nb),
                        rng("skip", skip, nd), rng("z", z, nx), rng("dt_bias", dt_bias, nd), rng("slots", slots, (size_t)B * 4),
                        rng("ntok", ntok, (size_t)B * 4)};
    const Range out[] = {rng("S", S, (size_t)nslot * nd * N), rng("y", y, nx)};
    if ((st = check_ranges(in, 10, out, 2))) return st;
    hipError_t e = kda::launch_scan_step(dtype == KDA_F32, B, T, D, N, G, nslot, softplus != 0, x, dt, A, b, c, skip, z, dt_bias,
                                         S, slots, ntok, y, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

// ---------------------------------------------------------------- short convolution
static int check_conv(int dtype, int act, int a, int T, int D, int W) {
    if (dtype != KDA_BF16 && dtype != KDA_F32) return fail(KDA_ERR_DTYPE, "unknown dtype %d", dtype);
    if (act != KDA_CONV_LINEAR && act != KDA_CONV_SILU) return fail(KDA_ERR_SHAPE, "unknown act %d", act);
    if (a < 1 || T < 1) return fail(KDA_ERR_SHAPE, "sequences=%d T=%d must be >= 1", a, T);
    if (T > 1 << 30) return fail(KDA_ERR_SHAPE, "T=%d above 2^30", T);
    if (D < 8 || D > 1 << 20 || D % 8) return fail(KDA_ERR_SHAPE, "D=%d must be a multiple of 8 from 8 to 2^20", D);
    if (W < 2 || W > 4) return fail(KDA_ERR_SHAPE, "W=%d not in {2, 3, 4}", W);
    // a launch has at most 2^32 threads: one for eight channels of eight rows at the least, filled up to whole
    // wavefronts, and one for eight channels of each sequence's state
    if (((int64_t)a * T / 8 + 2 * (int64_t)a + 1) >= (1LL << 30) / (D / 8)) return fail(KDA_ERR_SHAPE, "sequences*T*D too large");
    return KDA_OK;
}

int kda_short_conv_fwd(int dtype, int act, int nseq, int T, int D, int W, const int* cu_seqlens, int zero_rest, const void* x,
                       const float* w, const float* bias, const void* S0, void* y, void* S_T, void* stream) {
    int st = check_conv(dtype, act, cu_seqlens ? 1 : nseq, T, D, W);
    if (st) return st;
    if (cu_seqlens && (st = check_conv(dtype, act, nseq, 1, D, W))) return st;
    if (zero_rest != 0 && zero_rest != 1) return fail(KDA_ERR_SHAPE, "zero_rest=%d not in {0, 1}", zero_rest);
    if (!x || !w || !y) return fail(KDA_ERR_NULL, "x, w and y must be non-NULL");
    const size_t es = dtype == KDA_BF16 ? 2 : 4, tok = cu_seqlens ? (size_t)T : (size_t)nseq * T;
    const size_t nx = tok * D * es, ns = (size_t)nseq * (W - 1) * D * es;
    const Range in[] = {rng("x", x, nx), rng("w", w, (size_t)D * W * 4), rng("bias", bias, (size_t)D * 4),
                        rng("cu_seqlens", cu_seqlens, ((size_t)nseq + 1) * 4), rng("S0", S0 == S_T ? nullptr : S0, ns)};
    const Range out[] = {rng("y", y, nx), rng("S_T", S_T, ns)};
    if ((st = check_ranges(in, 5, out, 2))) return st;
    const kda::ConvCall call{dtype == KDA_F32, nseq, T, D, W, act == KDA_CONV_SILU, cu_seqlens, x, S0, w, bias};
    hipError_t e = kda::launch_conv_fwd(call, zero_rest != 0, y, S_T, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

int kda_short_conv_bwd_workspace_size(long long rows, int D, int W, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_NULL, "bytes is NULL");
    if (rows < 1 || rows > 1LL << 40) return fail(KDA_ERR_SHAPE, "rows=%lld outside [1, 2^40]", rows);
    int st = check_conv(KDA_BF16, KDA_CONV_LINEAR, 1, 1, D, W);
    if (st) return st;
    *bytes = kda::conv_bwd_workspace_bytes(rows, D, W);
    return ok();
}

int kda_short_conv_bwd(int dtype, int act, int nseq, int T, int D, int W, const int* cu_seqlens, const void* x, const float* w,
                       const float* bias, const void* S0, const void* dy, const void* dS_T, void* dx, float* dw, float* dbias,
                       void* dS0, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_conv(dtype, act, cu_seqlens ? 1 : nseq, T, D, W);
    if (st) return st;
    if (cu_seqlens && (st = check_conv(dtype, act, nseq, 1, D, W))) return st;
    if (!x || !w || !dy || !dx || !dw) return fail(KDA_ERR_NULL, "x, w, dy, dx and dw must be non-NULL");
    if (dbias && !bias) return fail(KDA_ERR_NULL, "dbias needs bias");
    const size_t es = dtype == KDA_BF16 ? 2 : 4, tok = cu_seqlens ? (size_t)T : (size_t)nseq * T;
    const size_t nx = tok * D * es, ns = (size_t)nseq * (W - 1) * D * es, nw = (size_t)D * W * 4, nb = (size_t)D * 4;
    const size_t need = kda::conv_bwd_workspace_bytes((int64_t)tok, D, W);
    if (!workspace || workspace_bytes < need)
        return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu%s", need, workspace_bytes,
                    workspace ? "" : " (NULL)");
    const Range in[] = {rng("x", x, nx), rng("w", w, nw), rng("bias", bias, nb),
                        rng("cu_seqlens", cu_seqlens, ((size_t)nseq + 1) * 4), rng("S0", S0, ns), rng("dy", dy, nx),
                        rng("dS_T", dS_T, ns)};
    const Range out[] = {rng("dx", dx, nx), rng("dw", dw, nw), rng("dbias", dbias, nb), rng("dS0", dS0, ns),
                         rng("workspace", workspace, need)};
    if ((st = check_ranges(in, 7, out, 5))) return st;
    const kda::ConvCall call{dtype == KDA_F32, nseq, T, D, W, act == KDA_CONV_SILU, cu_seqlens, x, S0, w, bias};
    hipError_t e = kda::launch_conv_bwd(call, dy, dS_T, dx, dw, dbias, dS0, (float*)workspace, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

int kda_short_conv_step(int dtype, int act, int B, int T, int D, int W, int nslot, const void* x, const float* w,
                        const float* bias, void* S, const int* slots, const int* ntok, void* y, void* stream) {
    int st = check_conv(dtype, act, B, T, D, W);
    if (st) return st;
    if (nslot < 1 || (!slots && nslot < B))
        return fail(KDA_ERR_SHAPE, "nslot=%d states for B=%d rows%s", nslot, B, slots ? "" : " without slots");
    if ((int64_t)B * ((D / 8 + 63) / 64) >= 1LL << 26) return fail(KDA_ERR_SHAPE, "B*D too large");   // workgroups of 64 threads
    if (!x || !w || !S || !y) return fail(KDA_ERR_NULL, "x, w, S and y must be non-NULL");
    const size_t es = dtype == KDA_BF16 ? 2 : 4, nx = (size_t)B * T * D * es;
    const Range in[] = {rng("x", x, nx), rng("w", w, (size_t)D * W * 4), rng("bias", bias, (size_t)D * 4),
                        rng("slots", slots, (size_t)B * 4), rng("ntok", ntok, (size_t)B * 4)};
    const Range out[] = {rng("S", S, (size_t)nslot * (W - 1) * D * es), rng("y", y, nx)};
    if ((st = check_ranges(in, 5, out, 2))) return st;
    const kda::ConvCall call{dtype == KDA_F32, B, T, D, W, act == KDA_CONV_SILU, nullptr, x, nullptr, w, bias};
    hipError_t e = kda::launch_conv_step(call, B, nslot, S, slots, ntok, y, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

// ---------------------------------------------------------------- layer norm
int kda_layer_norm_fwd(int dtype, long long rows, int D, float eps, const void* y, const void* x, const float* w, const float* b,
                       void* r, void* h, void* stream) {
    int st = check_norm(dtype, KDA_ACT_SIGMOID, rows, D, eps);
    if (st) return st;
    if (!y || !h) return fail(KDA_ERR_NULL, "y and h must be non-NULL");
    if (!x != !r) return fail(KDA_ERR_NULL, "r and x go together: both or neither may be NULL");
    const size_t n = (size_t)rows * D * (dtype == KDA_BF16 ? 2 : 4), nw = (size_t)D * 4;
    // r may be x itself: the residual stream updated in place
    const Range in[] = {rng("y", y, n), rng("x", x == r ? nullptr : x, n), rng("w", w, nw), rng("b", b, nw)};
    const Range out[] = {rng("r", r, n), rng("h", h, n)};
    if ((st = check_ranges(in, 4, out, 2))) return st;
    hipError_t e = kda::launch_layer_norm_fwd(dtype == KDA_F32, rows, D, eps, y, x, w, b, r, h, reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

int kda_layer_norm_bwd_workspace_size(long long rows, int D, size_t* bytes) {
    if (!bytes) return fail(KDA_ERR_NULL, "bytes is NULL");
    int st = check_norm(KDA_BF16, KDA_ACT_SIGMOID, rows, D, 0.0f);
    if (st) return st;
    *bytes = kda::layer_norm_bwd_workspace_bytes(rows, D);
    return ok();
}

int kda_layer_norm_bwd(int dtype, long long rows, int D, float eps, const void* y, const void* x, const float* w, const void* dr,
                       const void* dh, void* dy, float* dw, float* db, void* workspace, size_t workspace_bytes, void* stream) {
    int st = check_norm(dtype, KDA_ACT_SIGMOID, rows, D, eps);
    if (st) return st;
    if (!y || !dh || !dy) return fail(KDA_ERR_NULL, "y, dh and dy must be non-NULL");
    if (dr && !x) return fail(KDA_ERR_NULL, "dr without x: the norm alone has no residual stream");
    const size_t n = (size_t)rows * D * (dtype == KDA_BF16 ? 2 : 4), nw = (size_t)D * 4;
    const size_t need = dw || db ? kda::layer_norm_bwd_workspace_bytes(rows, D) : 0;
    if (need && (!workspace || workspace_bytes < need))
        return fail(KDA_ERR_WORKSPACE, "workspace of %zu bytes needed, got %zu%s", need, workspace_bytes,
                    workspace ? "" : " (NULL)");
    const Range in[] = {rng("y", y, n), rng("x", x, n), rng("w", w, nw), rng("dr", dr, n), rng("dh", dh, n)};
    const Range out[] = {rng("dy", dy, n), rng("dw", dw, nw), rng("db", db, nw), rng("workspace", need ? workspace : nullptr, need)};
    if ((st = check_ranges(in, 5, out, 4))) return st;
    hipError_t e = kda::launch_layer_norm_bwd(dtype == KDA_F32, rows, D, eps, y, x, w, dr, dh, dy, dw, db, (float*)workspace,
                                              reinterpret_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(KDA_ERR_HIP, "launch failed: %s", hipGetErrorString(e));
    return ok();
}

}  // extern "C"
