// kda_conv.hip -- the short causal convolution of every channel with itself, forwards,
// backwards, and token by token from and to a pool of states.
//
// Per channel, with W taps, x_-1 .. x_-(W-1) the state (the last inputs, oldest first) or zero:
//     p_t = bias + sum_j w_j x_{t-W+1+j},   y_t = p_t  or  p_t sigmoid(p_t)
// and, with dp_t = dy_t act'(p_t), zero behind the last token:
//     dx_s = sum_j w_j dp_{s+W-1-j} (+ the last state's gradient),  dw_j = sum_t dp_t x_{t-W+1+j},  dbias = sum_t dp_t
// All arithmetic is fp32, rounded once.  Both passes are bound by HBM: a lane owns eight channels and
// a run of rows, whose last W inputs stay in registers; a run reads W - 1 rows of its neighbour's.
// Measured, bf16, 4 taps, silu: forwards 65,536 rows of 6,144 channels 316 us (1.61 GB, 5.1 TB/s, a large copy's rate);
// backwards 32,768 rows of 2,048 channels in six packed sequences 99 us (403 MB, 4.1 TB/s; 5 us of it the sums'
// launch), where the taps, their sums, the inputs and the waiting gradients are 242 registers and a SIMD
// has two wavefronts; in fp32 266, one wavefront, and 215 us (805 MB, 3.7 TB/s).  Four channels a lane (119), two (114 to 120), rows without branches in the middle of
// a run (114 beside 110) and other lengths of runs gained nothing there.
#include "kda_launch.hpp"
#include "kda_rows.hpp"

namespace kda {

namespace {

struct ConvArgs {
    int nseq, T, D, run;   // run: rows a lane
    int64_t rows;
    bool silu, zero_rest;   // zero_rest: zeros in y's rows of no sequence (in dx's always)
    const int* cu;
    const void *x, *S0, *dy, *dS_T;
    const float *w, *bias;
    void *y, *S_T, *dx, *dS0;
    float *pw, *pb;   // parts of dw [workgroup row][D * W] and of dbias [workgroup row][D]
};

// The rows of a sequence; offsets out of order or range are held to both.
struct Span {
    int n;
    int64_t lo, hi;
};
__device__ __forceinline__ Span span_at(const ConvArgs& a, int n) {
    if (!a.cu) return Span{n, (int64_t)n * a.T, (int64_t)(n + 1) * a.T};
    const int lo = held(a.cu[n], 0, a.T);
    return Span{n, lo, held(a.cu[n + 1], lo, a.T)};
}
// The last sequence that starts at or before the row, or the first.
__device__ __forceinline__ Span span_of(const ConvArgs& a, int64_t row) {
    if (!a.cu) return span_at(a, (int)(row / a.T));
    int lo = 0, hi = a.nseq - 1;
    while (lo < hi) {
        const int mid = lo + (hi - lo + 1) / 2;
        if (a.cu[mid] <= row) lo = mid;
        else hi = mid - 1;
    }
    return span_at(a, lo);
}

template <typename E>
__device__ __forceinline__ V8 ld_row(const void* p, int64_t row, int D, int vec) { return ld8((const E*)p + row * D + 8 * vec); }

// Input `back` places before the sequence's row: from the tensor, the state or nothing.
template <typename E, int W>
__device__ __forceinline__ V8 input_at(const ConvArgs& a, const Span& s, int64_t row, int vec) {
    if (row >= s.lo) return ld_row<E>(a.x, row, a.D, vec);
    if (a.S0) return ld_row<E>(a.S0, (int64_t)s.n * (W - 1) + (W - 1) + (row - s.lo), a.D, vec);
    return V8{};
}

template <int W>
struct Taps {
    V8 w[W], bias;
    __device__ __forceinline__ void load(const ConvArgs& a, int vec) {
#pragma unroll
        for (int i = 0; i < 2 * W; ++i) {   // a channel's taps lie side by side
            const f32x4 v = *reinterpret_cast<const f32x4*>(a.w + (int64_t)8 * vec * W + 4 * i);
#pragma unroll
            for (int k = 0; k < 4; ++k) w[(4 * i + k) % W].f[(4 * i + k) / W] = v[k];
        }
        bias = a.bias ? ld8(a.bias + 8 * vec) : V8{};
    }
    // win[k]: the input k places back
    __device__ __forceinline__ V8 apply(const V8 (&win)[W]) const {
        V8 p = bias;
#pragma unroll
        for (int j = 0; j < W; ++j)
#pragma unroll
            for (int e = 0; e < 8; ++e) p.f[e] = __builtin_fmaf(w[j].f[e], win[W - 1 - j].f[e], p.f[e]);
        return p;
    }
};

template <int W>
__device__ __forceinline__ void shift(V8 (&win)[W]) {
#pragma unroll
    for (int k = W - 1; k > 0; --k) win[k] = win[k - 1];
}

// The last W - 1 inputs of sequence n, its state's among them where it is short.
template <typename E, int W>
__device__ __forceinline__ void last_state(const ConvArgs& a, int n, int vec) {
    const Span s = span_at(a, n);
    V8 v[W - 1];
#pragma unroll
    for (int i = 0; i < W - 1; ++i) v[i] = input_at<E, W>(a, s, s.hi - (W - 1) + i, vec);
#pragma unroll
    for (int i = 0; i < W - 1; ++i) st8((E*)a.S_T + ((int64_t)n * (W - 1) + i) * a.D + 8 * vec, v[i]);
}

template <typename E, int W>
__global__ void __launch_bounds__(256) conv_state_kernel(ConvArgs a) {
    const int nvec = a.D / 8;
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < (int64_t)a.nseq * nvec) last_state<E, W>(a, (int)(i / nvec), (int)(i % nvec));
}

template <typename E, int W>
__global__ void __launch_bounds__(256) conv_fwd_kernel(ConvArgs a) {
    constexpr int AHEAD = 8;   // rows asked for at a time
    const int nvec = a.D / 8;
    const int64_t runs = (a.rows + a.run - 1) / a.run;
    int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (id >= runs * nvec) {   // behind the runs: the last states
        id -= runs * nvec;
        if (a.S_T && id < (int64_t)a.nseq * nvec) last_state<E, W>(a, (int)(id / nvec), (int)(id % nvec));
        return;
    }
    const int vec = (int)(id % nvec);
    const int64_t r0 = id / nvec * a.run, r1 = r0 + a.run < a.rows ? r0 + a.run : a.rows;
    Raw<E> ahead[AHEAD];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) ld_raw((const E*)a.x + (row + i < r1 ? row + i : r1 - 1) * a.D + 8 * vec, ahead[i]);
    };
    fetch(r0);
    Taps<W> taps;
    taps.load(a, vec);
    Span s = span_of(a, r0);
    V8 win[W];
#pragma unroll
    for (int k = 0; k < W; ++k) win[k] = V8{};
    if (r0 > s.lo && r0 < s.hi)   // at a sequence's first row the loop does it
#pragma unroll
        for (int k = 1; k < W; ++k) win[k - 1] = input_at<E, W>(a, s, r0 - k, vec);
    for (int64_t base = r0; base < r1; base += AHEAD) {
        Raw<E> now[AHEAD];
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) now[i] = ahead[i];
        if (base + AHEAD < r1) fetch(base + AHEAD);
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int64_t row = base + i;
            if (row >= r1) break;
            while (row >= s.hi && s.n + 1 < a.nseq) s = span_at(a, s.n + 1);   // the next sequence with rows
            if (row == s.lo)
#pragma unroll
                for (int k = 1; k < W; ++k) win[k - 1] = input_at<E, W>(a, s, row - k, vec);
            shift<W>(win);
            win[0] = to_f8(now[i]);
            if (row < s.lo || row >= s.hi) {   // a row of no sequence
                if (a.zero_rest) st8((E*)a.y + row * a.D + 8 * vec, V8{});
                continue;
            }
            V8 p = taps.apply(win);
            if (a.silu)
#pragma unroll
                for (int e = 0; e < 8; ++e) p.f[e] *= sigmoid<E>(p.f[e]);
            st8((E*)a.y + row * a.D + 8 * vec, p);
        }
    }
}

// act'(p) dy
template <typename E>
__device__ __forceinline__ V8 through_act(bool silu, const V8& p, const V8& dy) {
    V8 d = dy;
    if (silu)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float sg = sigmoid<E>(p.f[e]);
            d.f[e] *= sg * (1.0f + p.f[e] * (1.0f - sg));
        }
    return d;
}

// VB lanes side by side hold eight channels each, 256 / VB runs of rows a workgroup.
template <typename E, int W>
__global__ void __launch_bounds__(256) conv_bwd_kernel(ConvArgs a, int VB, int state_blocks) {
    constexpr int AHEAD = 2;
    __shared__ float lds[8 * 256];
    const int nvec = a.D / 8, nvb = (nvec + VB - 1) / VB;
    if ((int)blockIdx.x < state_blocks) {   // the start states' gradients
        const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
        if (i >= (int64_t)a.nseq * nvec) return;
        const int n = (int)(i / nvec), vec = (int)(i % nvec);
        const Span s = span_at(a, n);
        Taps<W> taps;
        taps.load(a, vec);
        const int64_t len = s.hi - s.lo;
        V8 g[W - 1], win[W];
#pragma unroll
        for (int k = 0; k < W - 1; ++k) {
            g[k] = V8{};
            if (k >= len && a.dS_T) g[k] = ld_row<E>(a.dS_T, (int64_t)n * (W - 1) + k - len, a.D, vec);
        }
#pragma unroll
        for (int k = 1; k < W; ++k) win[k - 1] = input_at<E, W>(a, s, s.lo - k, vec);
#pragma unroll
        for (int j = 0; j < W - 1; ++j) {
            if (j >= len) break;
            shift<W>(win);
            win[0] = ld_row<E>(a.x, s.lo + j, a.D, vec);
            const V8 d = through_act<E>(a.silu, taps.apply(win), ld_row<E>(a.dy, s.lo + j, a.D, vec));
#pragma unroll
            for (int k = j; k < W - 1; ++k)   // state k meets tap k - j at token j
#pragma unroll
                for (int e = 0; e < 8; ++e) g[k].f[e] = __builtin_fmaf(taps.w[k - j].f[e], d.f[e], g[k].f[e]);
        }
#pragma unroll
        for (int k = 0; k < W - 1; ++k) st8((E*)a.dS0 + ((int64_t)n * (W - 1) + k) * a.D + 8 * vec, g[k]);
        return;
    }
    const int64_t blk = (int64_t)blockIdx.x - state_blocks;
    const int lane = (int)threadIdx.x % VB, sub = (int)threadIdx.x / VB, runs = 256 / VB;
    const int vec = (int)(blk % nvb) * VB + lane;
    const int64_t r0 = (blk / nvb * runs + sub) * a.run, r1 = r0 + a.run < a.rows ? r0 + a.run : a.rows;
    const bool on = vec < nvec && r0 < a.rows;
    V8 dw[W], db{};
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j] = V8{};
    if (on) {
        Taps<W> taps;
        taps.load(a, vec);
        Span s = span_of(a, r0);
        V8 win[W], out[W];   // out[k]: what row t - k has of its gradient
#pragma unroll
        for (int k = 0; k < W; ++k) win[k] = out[k] = V8{};
        if (r0 > s.lo && r0 < s.hi)   // at a sequence's first row the loop does it
#pragma unroll
            for (int k = 1; k < W; ++k) win[k - 1] = input_at<E, W>(a, s, r0 - k, vec);
        const int64_t last = r1 + W - 1 < a.rows ? r1 + W - 1 : a.rows;
        // rows are asked for AHEAD at a time, one batch ahead of their use
        Raw<E> nx[AHEAD], nd[AHEAD];
        auto fetch = [&](int64_t t) {
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int64_t at = (t + i < last ? t + i : last - 1) * a.D + 8 * vec;
                ld_raw((const E*)a.x + at, nx[i]);
                ld_raw((const E*)a.dy + at, nd[i]);
            }
        };
        // The rows that wait at the end of a sequence have all that comes, but the last state's gradient.
        auto flush = [&](int64_t t) {
#pragma unroll
            for (int k = W - 1; k > 0; --k) {
                const int64_t row = t - k;
                if (row < s.lo || row < r0 || row >= r1 || t > s.hi) continue;
                V8 g = out[k - 1];
                if (a.dS_T) {
                    const V8 d = ld_row<E>(a.dS_T, (int64_t)s.n * (W - 1) + (W - 1) - k, a.D, vec);
#pragma unroll
                    for (int e = 0; e < 8; ++e) g.f[e] += d.f[e];
                }
                st8((E*)a.dx + row * a.D + 8 * vec, g);
            }
        };
        fetch(r0);
        for (int64_t t0 = r0; t0 < last; t0 += AHEAD) {
            Raw<E> cx[AHEAD], cd[AHEAD];
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) cx[i] = nx[i], cd[i] = nd[i];
            if (t0 + AHEAD < last) fetch(t0 + AHEAD);
#pragma unroll
            for (int i = 0; i < AHEAD; ++i) {
                const int64_t t = t0 + i;
                if (t >= last) break;
                if (t >= s.hi) {
                    flush(t);
                    while (t >= s.hi && s.n + 1 < a.nseq) s = span_at(a, s.n + 1);
                }
                if (t == s.lo) {
#pragma unroll
                    for (int k = 0; k < W; ++k) out[k] = V8{};
#pragma unroll
                    for (int k = 1; k < W; ++k) win[k - 1] = input_at<E, W>(a, s, t - k, vec);
                }
                if (t < s.lo || t >= s.hi) {   // a row of no sequence
                    if (t < r1) st8((E*)a.dx + t * a.D + 8 * vec, V8{});
                    continue;
                }
                shift<W>(win);
                win[0] = to_f8(cx[i]);
                const V8 d = through_act<E>(a.silu, taps.apply(win), to_f8(cd[i]));
                if (t < r1)
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j].f[e] = __builtin_fmaf(d.f[e], win[W - 1 - j].f[e], dw[j].f[e]);
                        db.f[e] += d.f[e];
                    }
                shift<W>(out);
                out[0] = V8{};
#pragma unroll
                for (int k = 0; k < W; ++k)
#pragma unroll
                    for (int e = 0; e < 8; ++e) out[k].f[e] = __builtin_fmaf(taps.w[W - 1 - k].f[e], d.f[e], out[k].f[e]);
                const int64_t row = t - (W - 1);
                if (row >= s.lo && row >= r0) st8((E*)a.dx + row * a.D + 8 * vec, out[W - 1]);
            }
        }
        if (last >= s.hi) flush(last);
    }
    // the workgroup's runs, halved step by step in a fixed order
    float* pw = a.pw + blk / nvb * a.D * W + (int64_t)8 * vec * W;
#pragma unroll
    for (int j = 0; j <= W; ++j) {
        V8 v = j < W ? dw[j < W ? j : 0] : db;
        for (int half = runs / 2; half > 0; half /= 2) {
            __syncthreads();
            if (sub >= half && sub < 2 * half)
#pragma unroll
                for (int e = 0; e < 8; ++e) lds[e * 256 + threadIdx.x] = v.f[e];
            __syncthreads();
            if (sub < half)
#pragma unroll
                for (int e = 0; e < 8; ++e) v.f[e] += lds[e * 256 + threadIdx.x + half * VB];
        }
        if (sub == 0 && vec < nvec)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                if (j < W) pw[e * W + j] = v.f[e];
                else a.pb[blk / nvb * a.D + 8 * vec + e] = v.f[e];
            }
    }
}

struct ConvStepArgs {
    ConvArgs c;   // x, w, bias, y, silu, D
    int T, nslot;
    void* S;
    const int *slots, *ntok;
};

template <typename E, int W>
__global__ void __launch_bounds__(64) conv_step_kernel(ConvStepArgs a) {
    const int D = a.c.D, nvec = D / 8, nvb = (nvec + 63) / 64;
    const int r = (int)(blockIdx.x / (unsigned)nvb), vec = (int)(blockIdx.x % (unsigned)nvb) * 64 + (int)threadIdx.x;
    int n = a.T;
    if (a.ntok) {
        n = a.ntok[r];
        n = n < a.T ? n : a.T;
    }
    const int slot = a.slots ? a.slots[r] : r;
    if (n <= 0 || slot < 0 || slot >= a.nslot) return;   // a padded row: nothing of it is touched
    if (a.slots) {   // of the rows with tokens that name one slot, the first has it; the others are padding
        if (earlier_row(a.slots, a.ntok, r, slot, (int)threadIdx.x)) return;
    }
    if (vec >= nvec) return;
    E* Sp = (E*)a.S + (int64_t)slot * (W - 1) * D + 8 * vec;
    V8 win[W];
#pragma unroll
    for (int k = 1; k < W; ++k) win[k - 1] = ld8(Sp + (int64_t)(W - 1 - k) * D);
    Taps<W> taps;
    taps.load(a.c, vec);
    for (int t = 0; t < n; ++t) {
        const int64_t at = ((int64_t)r * a.T + t) * D + 8 * vec;
        shift<W>(win);
        win[0] = ld8((const E*)a.c.x + at);
        V8 p = taps.apply(win);
        if (a.c.silu)
#pragma unroll
            for (int e = 0; e < 8; ++e) p.f[e] *= sigmoid<E>(p.f[e]);
        st8((E*)a.c.y + at, p);
    }
#pragma unroll
    for (int k = 1; k < W; ++k) st8(Sp + (int64_t)(W - 1 - k) * D, win[k - 1]);
}

// Rows a lane: long runs read little of their neighbours' (3 rows in 32), short ones fill the device: 2^18 lanes
// are 16 wavefronts a compute unit.
int fwd_run(int64_t rows, int D) {
    int run = 32;
    while (run > 8 && (rows + run - 1) / run * (D / 8) < 1 << 18) run /= 2;
    return run;
}

struct BwdRuns {
    int run, VB;
    int64_t parts, blocks;   // rows of parts; workgroups
};
BwdRuns bwd_runs(int64_t rows, int D) {
    const int nvec = D / 8;
    BwdRuns r;
    r.VB = 1;
    while (r.VB < nvec && r.VB < 64) r.VB *= 2;
    r.run = 64;
    while (r.run > 8 && (rows + r.run - 1) / r.run * nvec < 1 << 17) r.run /= 2;
    const int64_t per = (int64_t)r.run * (256 / r.VB);
    r.parts = (rows + per - 1) / per;
    r.blocks = r.parts * ((nvec + r.VB - 1) / r.VB);
    return r;
}

template <typename E, int W>
hipError_t conv_fwd_t(ConvArgs a, hipStream_t stream) {
    const int64_t nvec = a.D / 8, states = (a.nseq * nvec + 255) / 256;
    const bool apart = a.S_T && a.S_T == a.S0;   // in place: only after the rows have read it
    const int64_t lanes = (a.rows + a.run - 1) / a.run * nvec + (a.S_T && !apart ? a.nseq * nvec : 0);
    ConvArgs f = a;
    if (apart) f.S_T = nullptr;
    hipLaunchKernelGGL((conv_fwd_kernel<E, W>), dim3((unsigned)((lanes + 255) / 256)), dim3(256), 0, stream, f);
    if (apart) hipLaunchKernelGGL((conv_state_kernel<E, W>), dim3((unsigned)states), dim3(256), 0, stream, a);
    return hipGetLastError();
}

template <typename E, int W>
hipError_t conv_bwd_t(ConvArgs a, float* dw, float* dbias, hipStream_t stream) {
    const BwdRuns r = bwd_runs(a.rows, a.D);
    const int64_t states = a.dS0 ? ((int64_t)a.nseq * (a.D / 8) + 255) / 256 : 0;
    hipLaunchKernelGGL((conv_bwd_kernel<E, W>), dim3((unsigned)(states + r.blocks)), dim3(256), 0, stream, a, r.VB, (int)states);
    launch_part_sums(PartSums{{a.pw, a.pb, nullptr}, {dw, dbias, nullptr}, {(int64_t)a.D * W, a.D, 0}, r.parts}, stream);
    return hipGetLastError();
}

template <typename E, int W>
hipError_t conv_step_t(int B, const ConvStepArgs& a, hipStream_t stream) {
    hipLaunchKernelGGL((conv_step_kernel<E, W>), dim3((unsigned)((int64_t)B * ((a.c.D / 8 + 63) / 64))), dim3(64), 0, stream, a);
    return hipGetLastError();
}

ConvArgs args_of(const ConvCall& c) {
    ConvArgs a{};
    a.nseq = c.nseq, a.T = c.T, a.D = c.D, a.silu = c.silu, a.cu = c.cu;
    a.rows = c.cu ? c.T : (int64_t)c.nseq * c.T;
    a.x = c.x, a.S0 = c.S0, a.w = c.w, a.bias = c.bias;
    return a;
}

#define KDA_CONV_TAPS(W, CALL) \
    switch (W) {               \
        case 2: CALL(2);       \
        case 3: CALL(3);       \
        case 4: CALL(4);       \
    }

}  // namespace

hipError_t launch_conv_fwd(const ConvCall& c, bool zero_rest, void* y, void* S_T, hipStream_t stream) {
    ConvArgs a = args_of(c);
    a.run = fwd_run(a.rows, a.D);
    a.zero_rest = zero_rest, a.y = y, a.S_T = S_T;
#define KDA_CF(W) return c.f32 ? conv_fwd_t<float, W>(a, stream) : conv_fwd_t<bf16, W>(a, stream)
    KDA_CONV_TAPS(c.W, KDA_CF)
#undef KDA_CF
    return hipErrorInvalidValue;
}

size_t conv_bwd_workspace_bytes(int64_t rows, int D, int W) { return (size_t)bwd_runs(rows, D).parts * D * (W + 1) * sizeof(float); }

hipError_t launch_conv_bwd(const ConvCall& c, const void* dy, const void* dS_T, void* dx, float* dw, float* dbias, void* dS0, float* part,
                           hipStream_t stream) {
    ConvArgs a = args_of(c);
    const BwdRuns r = bwd_runs(a.rows, a.D);
    a.run = r.run;
    a.dy = dy, a.dS_T = dS_T, a.dx = dx, a.dS0 = dS0;
    a.pw = part, a.pb = part + r.parts * a.D * c.W;
#define KDA_CB(W) return c.f32 ? conv_bwd_t<float, W>(a, dw, dbias, stream) : conv_bwd_t<bf16, W>(a, dw, dbias, stream)
    KDA_CONV_TAPS(c.W, KDA_CB)
#undef KDA_CB
    return hipErrorInvalidValue;
}

hipError_t launch_conv_step(const ConvCall& c, int B, int nslot, void* S, const int* slots, const int* ntok, void* y, hipStream_t stream) {
    ConvStepArgs a{args_of(c), c.T, nslot, S, slots, ntok};
    a.c.y = y;
#define KDA_CS(W) return c.f32 ? conv_step_t<float, W>(B, a, stream) : conv_step_t<bf16, W>(B, a, stream)
    KDA_CONV_TAPS(c.W, KDA_CS)
#undef KDA_CS
    return hipErrorInvalidValue;
}

}  // namespace kda
