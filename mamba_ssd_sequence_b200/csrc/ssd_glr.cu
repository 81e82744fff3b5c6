// Gated linear recurrence h_t = a_t h_{t-1} + f_t x_t per channel (ssd.h,
// ssd_glr_fwd / ssd_glr_bwd / ssd_glr_step).
//
// One thread per channel of a batch, walking the tokens in order (forward) or
// in chunks from the last to the first with h recomputed from the saved
// states (backward).
#include <cuda_bf16.h>
#include <math.h>

#include "ssd_internal.h"
#include "ssd_view.h"

namespace ssd {
namespace {

constexpr int kThreads = 64;
constexpr int kChunk = SSD_GLR_CHUNK;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

struct GlrArgs {
    ssd_view x, gate, out, dy, dx, dgate;
    const float *A_log, *dt_bias, *h0, *dh_out;
    const int *lengths;
    float *h_out, *states, *dh0, *partA, *partb;
    int B, H, N, d, flags;
};

// One token's gate: la = log a, f the value factor, s = dt, sg = d dt / d gate.
struct Gate {
    float la, a, f, s, sg;
};

__device__ __forceinline__ Gate gate_of(float g, float rate, float bias, int flags) {
    Gate o;
    o.s = 0.0f;
    o.sg = 1.0f;
    if (flags & SSD_GLR_LOG_DECAY) {
        o.la = g;
    } else {
        const float p = g + bias;
        const float u = expf(-fabsf(p));
        o.s = fmaxf(p, 0.0f) + log1pf(u);
        o.sg = (p >= 0.0f ? 1.0f : u) / (1.0f + u);
        o.la = -rate * o.s;
    }
    o.a = expf(o.la);
    o.f = (flags & SSD_VALUE_DT) ? o.s : (flags & SSD_GLR_COMPLEMENT) ? -expm1f(o.la) : 1.0f;
    return o;
}

__device__ __forceinline__ int length_of(const int *lengths, int b, int N) {
    return lengths ? min(max(lengths[b], 0), N) : N;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) glr_fwd_kernel(GlrArgs g) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long C = (long long)g.H * g.d;
    if (i >= g.B * C) return;
    const int b = (int)(i / C), c = (int)(i % C), h = c / g.d, j = c % g.d;
    const T *x = static_cast<const T *>(g.x.ptr) + b * g.x.stride_b + h * g.x.stride_h + j;
    const T *gt = static_cast<const T *>(g.gate.ptr) + b * g.gate.stride_b + h * g.gate.stride_h + j;
    T *out = static_cast<T *>(g.out.ptr) + b * g.out.stride_b + h * g.out.stride_h + j;
    const float rate = g.A_log ? expf(g.A_log[c]) : 1.0f, bias = g.dt_bias ? g.dt_bias[c] : 0.0f;
    const int len = length_of(g.lengths, b, g.N), nc = (g.N + kChunk - 1) / kChunk;
    float hs = g.h0 ? g.h0[i] : 0.0f;
    for (int t = 0; t < g.N; ++t) {
        if (g.states && t % kChunk == 0)
            g.states[((long long)(b * g.H + h) * nc + t / kChunk) * g.d + j] = hs;
        float y = 0.0f;
        if (t < len) {
            const Gate o = gate_of(to_f32(gt[t * g.gate.stride_n]), rate, bias, g.flags);
            hs = fmaf(o.a, hs, o.f * to_f32(x[t * g.x.stride_n]));
            y = hs;
        }
        out[t * g.out.stride_n] = from_f32<T>(y);
    }
    if (g.h_out) g.h_out[i] = hs;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) glr_bwd_kernel(GlrArgs g) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long C = (long long)g.H * g.d;
    if (i >= g.B * C) return;
    const int b = (int)(i / C), c = (int)(i % C), h = c / g.d, j = c % g.d;
    const T *x = static_cast<const T *>(g.x.ptr) + b * g.x.stride_b + h * g.x.stride_h + j;
    const T *gt = static_cast<const T *>(g.gate.ptr) + b * g.gate.stride_b + h * g.gate.stride_h + j;
    const T *dy = static_cast<const T *>(g.dy.ptr) + b * g.dy.stride_b + h * g.dy.stride_h + j;
    T *dx = static_cast<T *>(g.dx.ptr) + b * g.dx.stride_b + h * g.dx.stride_h + j;
    T *dg = static_cast<T *>(g.dgate.ptr) + b * g.dgate.stride_b + h * g.dgate.stride_h + j;
    const float rate = g.A_log ? expf(g.A_log[c]) : 1.0f, bias = g.dt_bias ? g.dt_bias[c] : 0.0f;
    const int len = length_of(g.lengths, b, g.N), nc = (g.N + kChunk - 1) / kChunk;
    float lam = g.dh_out ? g.dh_out[i] : 0.0f;  // a_{t+1} l_{t+1}, the adjoint of the state after token t
    float sumA = 0.0f, sumb = 0.0f;
    for (int k = nc - 1; k >= 0; --k) {
        const int t0 = k * kChunk;
        float before[kChunk];
        float hs = g.states[((long long)(b * g.H + h) * nc + k) * g.d + j];
        for (int e = 0; e < kChunk; ++e) {
            before[e] = hs;
            const int t = t0 + e;
            if (t < len) {
                const Gate o = gate_of(to_f32(gt[t * g.gate.stride_n]), rate, bias, g.flags);
                hs = fmaf(o.a, hs, o.f * to_f32(x[t * g.x.stride_n]));
            }
        }
        for (int e = kChunk - 1; e >= 0; --e) {
            const int t = t0 + e;
            if (t >= g.N) continue;
            float gx = 0.0f, gg = 0.0f;
            if (t < len) {
                const Gate o = gate_of(to_f32(gt[t * g.gate.stride_n]), rate, bias, g.flags);
                const float xv = to_f32(x[t * g.x.stride_n]);
                const float l = lam + to_f32(dy[t * g.dy.stride_n]);
                gx = o.f * l;
                lam = o.a * l;
                float dla = lam * before[e];
                if (g.flags & SSD_GLR_COMPLEMENT) dla = fmaf(-lam, xv, dla);
                if (g.flags & SSD_GLR_LOG_DECAY) {
                    gg = dla;
                } else {
                    float ds = -rate * dla;
                    if (g.flags & SSD_VALUE_DT) ds = fmaf(l, xv, ds);
                    gg = ds * o.sg;
                    // a = 0 below: log a may be -infinity there, the product is 0
                    sumA = fmaf(dla, fmaxf(o.la, -200.0f), sumA);
                    sumb += gg;
                }
            }
            dx[t * g.dx.stride_n] = from_f32<T>(gx);
            dg[t * g.dgate.stride_n] = from_f32<T>(gg);
        }
    }
    if (g.dh0) g.dh0[i] = lam;
    if (g.partA) g.partA[i] = sumA;
    if (g.partb) g.partb[i] = sumb;
}

// dA_log and ddt_bias: sums over the batch, in order.
__global__ void __launch_bounds__(kThreads)
glr_param_kernel(const float *partA, const float *partb, int B, long long C, float *dA, float *db) {
    const long long c = (long long)blockIdx.x * kThreads + threadIdx.x;
    if (c >= C) return;
    float sa = 0.0f, sb = 0.0f;
    for (int b = 0; b < B; ++b) {
        sa += partA[b * C + c];
        sb += partb[b * C + c];
    }
    if (dA) dA[c] = sa;
    if (db) db[c] = sb;
}

int check_flags(int flags) {
    if (flags & ~(SSD_VALUE_DT | SSD_GLR_LOG_DECAY | SSD_GLR_COMPLEMENT)) return SSD_ERR_FLAGS;
    if ((flags & SSD_VALUE_DT) && flags != SSD_VALUE_DT) return SSD_ERR_FLAGS;
    return SSD_OK;
}

int check_glr(int B, int H, int N, int d, int dtype, int flags, const void *const *f32, int nf32) {
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (!sizes_ok(B, H, N, d)) return SSD_ERR_SHAPE;
    if (check_flags(flags) != SSD_OK) return SSD_ERR_FLAGS;
    for (int i = 0; i < nf32; ++i)
        if (misaligned(f32[i], 4)) return SSD_ERR_ALIGN;
    return SSD_OK;
}

unsigned blocks_for(long long n) { return (unsigned)((n + kThreads - 1) / kThreads); }

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_glr_fwd(const ssd_view *x, const ssd_view *gate, const float *A_log, const float *dt_bias,
                const float *h0, const int *lengths, int B, int H, int N, int d_h, int dtype, int flags,
                const ssd_view *out, float *h_out, float *states, void *stream) {
    if (!x || !gate || !out) return SSD_ERR_NULL;
    const void *f32[] = {A_log, dt_bias, h0, lengths, h_out, states};
    int rc = check_glr(B, H, N, d_h, dtype, flags, f32, 6);
    if (rc != SSD_OK) return rc;
    const size_t e = elem_size(dtype);
    if ((rc = check_view(x, B, H, N, d_h, e, false)) || (rc = check_view(gate, B, H, N, d_h, e, false)) ||
        (rc = check_view(out, B, H, N, d_h, e, true)))
        return rc;
    GlrArgs g{};
    g.x = *x;
    g.gate = *gate;
    g.out = *out;
    const bool log = flags & SSD_GLR_LOG_DECAY;
    g.A_log = log ? nullptr : A_log;
    g.dt_bias = log ? nullptr : dt_bias;
    g.h0 = h0;
    g.lengths = lengths;
    g.h_out = h_out;
    g.states = states;
    g.B = B, g.H = H, g.N = N, g.d = d_h, g.flags = flags;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = blocks_for((long long)B * H * d_h);
    if (dtype == SSD_F32)
        glr_fwd_kernel<float><<<grid, kThreads, 0, s>>>(g);
    else
        glr_fwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(g);
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

size_t ssd_glr_bwd_workspace_bytes(int B, int H, int N, int d_h, int dtype, int flags) {
    if (check_glr(B, H, N, d_h, dtype, flags, nullptr, 0) != SSD_OK) return 0;
    return align_up((size_t)B * H * d_h * 2 * sizeof(float), 256);
}

int ssd_glr_bwd(const ssd_view *dy, const ssd_view *x, const ssd_view *gate, const float *A_log,
                const float *dt_bias, const float *states, const int *lengths, const float *dh_out,
                int B, int H, int N, int d_h, int dtype, int flags, const ssd_view *dx,
                const ssd_view *dgate, float *dA_log, float *ddt_bias, float *dh0, void *workspace,
                size_t workspace_bytes, void *stream) {
    if (!dy || !x || !gate || !states || !dx || !dgate) return SSD_ERR_NULL;
    const void *f32[] = {A_log, dt_bias, states, lengths, dh_out, dA_log, ddt_bias, dh0};
    int rc = check_glr(B, H, N, d_h, dtype, flags, f32, 8);
    if (rc != SSD_OK) return rc;
    const bool log = flags & SSD_GLR_LOG_DECAY;
    if (log && (dA_log || ddt_bias)) return SSD_ERR_FLAGS;
    const size_t e = elem_size(dtype);
    if ((rc = check_view(dy, B, H, N, d_h, e, false)) || (rc = check_view(x, B, H, N, d_h, e, false)) ||
        (rc = check_view(gate, B, H, N, d_h, e, false)) || (rc = check_view(dx, B, H, N, d_h, e, true)) ||
        (rc = check_view(dgate, B, H, N, d_h, e, true)))
        return rc;
    if (!workspace || workspace_bytes < ssd_glr_bwd_workspace_bytes(B, H, N, d_h, dtype, flags))
        return SSD_ERR_WORKSPACE;
    if (misaligned(workspace, 256)) return SSD_ERR_ALIGN;
    GlrArgs g{};
    g.dy = *dy;
    g.x = *x;
    g.gate = *gate;
    g.dx = *dx;
    g.dgate = *dgate;
    g.A_log = log ? nullptr : A_log;
    g.dt_bias = log ? nullptr : dt_bias;
    g.lengths = lengths;
    g.dh_out = dh_out;
    g.states = const_cast<float *>(states);
    g.dh0 = dh0;
    const long long C = (long long)H * d_h;
    const bool params = dA_log || ddt_bias;
    if (params) {
        g.partA = static_cast<float *>(workspace);
        g.partb = g.partA + B * C;
    }
    g.B = B, g.H = H, g.N = N, g.d = d_h, g.flags = flags;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = blocks_for(B * C);
    if (dtype == SSD_F32)
        glr_bwd_kernel<float><<<grid, kThreads, 0, s>>>(g);
    else
        glr_bwd_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(g);
    if (params) glr_param_kernel<<<blocks_for(C), kThreads, 0, s>>>(g.partA, g.partb, B, C, dA_log, ddt_bias);
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

int ssd_glr_step(const ssd_view *x, const ssd_view *gate, const float *A_log, const float *dt_bias, int B,
                 int H, int d_h, int dtype, int flags, float *h, const ssd_view *out, void *stream) {
    if (!h) return SSD_ERR_NULL;
    return ssd_glr_fwd(x, gate, A_log, dt_bias, h, nullptr, B, H, 1, d_h, dtype, flags, out, h, nullptr, stream);
}

}  // extern "C"
