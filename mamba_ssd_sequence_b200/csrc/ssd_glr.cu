// Gated linear recurrence: entry points (ssd.h, ssd_glr_fwd / ssd_glr_bwd /
// ssd_glr_step), the cut of a call into clusters, and the decode step.
#include <initializer_list>

#include "ssd_glr.cuh"

namespace ssd {
namespace glr {

Cut cut_of(int B, int H, int N, int d, int dtype) {
    const int nt = dtype == SSD_F32 ? Threads<float>::n : Threads<__nv_bfloat16>::n;
    const long long BH = (long long)B * H;
    auto tok = [&](int cb) { return nt / (cb / 2) * kSeg; };
    auto blocks = [&](int cb) { return BH * ((d + cb - 1) / cb); };
    Cut p;
    p.cb = d <= 16 ? 16 : d <= 32 || (d + 63) / 64 * 2 > (d + 31) / 32 ? 32 : 64;
    // narrower blocks where even clusters of 8 would leave SMs idle
    while (p.cb > 16 && blocks(p.cb) * 8 < 222 && N > tok(p.cb)) p.cb /= 2;
    p.nblk = (d + p.cb - 1) / p.cb;
    p.blocks = blocks(p.cb);
    // Clusters that fill the SMs with two blocks each and all run at once: 256
    // blocks do in any cluster size (36 channel blocks of 21707 tokens: 41 us in
    // clusters of 7, 50 of 8; 84 of 2047: 17 us of 3, 21 of 4); else the power of two
    // that comes to 222 blocks, one and a half an SM (32 channel blocks of 65536
    // tokens: 240 us in clusters of 8, 292 of 4, 869 alone).
    const auto useful = [&](int c) { return (long long)(c - 1) * tok(p.cb) < N; };
    for (p.cluster = kMaxCluster; p.cluster > 1; --p.cluster)
        if (useful(p.cluster) && p.blocks * p.cluster >= 230 && p.blocks * p.cluster <= 256) return p;
    while (p.cluster < kMaxCluster && p.blocks * p.cluster < 222 && useful(p.cluster + 1)) p.cluster *= 2;
    return p;
}

namespace {

constexpr int kThreads = 128;

// One token of one channel (both halves of the pairwise forms take it).
template <typename T, int kMode>
__device__ __forceinline__ float step(float g, float bias, float nrate2, float x, float h) {
    const Gate o = gate_of<T, kMode>(both(g), both(bias), both(nrate2));
    float2 w;
    const float a = exact_decay(o.l, &w).x;  // steps follow one another: as exact as a segment's product
    return fmaf(a, h, value_of<kMode>(o, both(x)).x);
}

template <typename T>
__global__ void __launch_bounds__(kThreads) glr_step_kernel(const Args g, int mode) {
    const long long i = (long long)blockIdx.x * kThreads + threadIdx.x;
    const long long C = (long long)g.H * g.d;
    if (i >= g.B * C) return;
    const int b = (int)(i / C), c = (int)(i % C), h = c / g.d, j = c % g.d;
    const float xv = to_f32(static_cast<const T *>(g.x.ptr)[b * g.x.stride_b + h * g.x.stride_h + j]);
    const float gv = to_f32(static_cast<const T *>(g.gate.ptr)[b * g.gate.stride_b + h * g.gate.stride_h + j]);
    const float h0 = g.h0[i];
    const float nrate2 = -1.4426950408889634f * (g.A_log ? expf(g.A_log[c]) : 1.0f), bias = g.dt_bias ? g.dt_bias[c] : 0.0f;
    float y;
    switch (mode) {
    case kDtNone: y = step<T, kDtNone>(gv, bias, nrate2, xv, h0); break;
    case kDtDt: y = step<T, kDtDt>(gv, bias, nrate2, xv, h0); break;
    case kDtComplement: y = step<T, kDtComplement>(gv, bias, nrate2, xv, h0); break;
    case kLogNone: y = step<T, kLogNone>(gv, bias, nrate2, xv, h0); break;
    default: y = step<T, kLogComplement>(gv, bias, nrate2, xv, h0); break;
    }
    g.h_out[i] = y;
    store_one(static_cast<T *>(g.out.ptr) + b * g.out.stride_b + h * g.out.stride_h + j, y);
}

unsigned blocks_for(long long n) { return (unsigned)((n + kThreads - 1) / kThreads); }

int mode_of(int flags) {
    if (flags & SSD_GLR_LOG_DECAY) return flags & SSD_GLR_COMPLEMENT ? kLogComplement : kLogNone;
    return flags & SSD_VALUE_DT ? kDtDt : flags & SSD_GLR_COMPLEMENT ? kDtComplement : kDtNone;
}

// How the views allow their elements to be moved (Args::aligned): by 16 bytes, by
// two elements, or one by one.
int alignment_of(std::initializer_list<const ssd_view *> views, int d, size_t esize) {
    uintptr_t all = (uintptr_t)d * esize;
    for (const ssd_view *v : views)
        all |= reinterpret_cast<uintptr_t>(v->ptr) |
               (uintptr_t)((v->stride_b | v->stride_h | v->stride_n) * (long long)esize);
    return all % 16 == 0 ? 2 : all % (2 * esize) == 0 ? 1 : 0;
}

int check_flags(int flags) {
    if (flags & ~(SSD_VALUE_DT | SSD_GLR_LOG_DECAY | SSD_GLR_COMPLEMENT)) return SSD_ERR_FLAGS;
    if ((flags & SSD_VALUE_DT) && flags != SSD_VALUE_DT) return SSD_ERR_FLAGS;
    return SSD_OK;
}

// What the failure tests ask for (ssd_debug_glr_fwd).
bool late_ok(int late_block, long long late_ns, long long wait_ns) {
    return late_block >= -1 && late_block < kMaxCluster && late_ns >= 0 && late_ns <= kWaitNs && wait_ns >= 0 &&
           wait_ns <= kWaitNs;
}
LateArgs late_args(const Args &g, int late_block, long long late_ns, long long wait_ns) {
    return {g, wait_ns ? wait_ns : kWaitNs, late_ns, late_block};
}

int check_glr(int B, int H, int N, int d, int dtype, int flags, const void *const *f32, int nf32) {
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (!sizes_ok(B, H, N, d) || (long long)B * H * d >= (1ll << 31) - 65536) return SSD_ERR_SHAPE;
    if (check_flags(flags) != SSD_OK) return SSD_ERR_FLAGS;
    for (int i = 0; i < nf32; ++i)
        if (misaligned(f32[i], 4)) return SSD_ERR_ALIGN;
    return SSD_OK;
}

}  // namespace
}  // namespace glr
}  // namespace ssd

using namespace ssd;
using namespace ssd::glr;

extern "C" {

int ssd_debug_glr_fwd(const ssd_view *x, const ssd_view *gate, const float *A_log, const float *dt_bias,
                      const float *h0, const int *lengths, int B, int H, int N, int d_h, int dtype, int flags,
                      const ssd_view *out, float *h_out, float *states, void *stream, int late_block,
                      long long late_ns, long long wait_ns) {
    if (!x || !gate || !out) return SSD_ERR_NULL;
    const void *f32[] = {A_log, dt_bias, h0, lengths, h_out, states};
    int rc = check_glr(B, H, N, d_h, dtype, flags, f32, 6);
    if (rc != SSD_OK) return rc;
    const size_t e = elem_size(dtype);
    if ((rc = check_view(x, B, H, N, d_h, e, false)) || (rc = check_view(gate, B, H, N, d_h, e, false)) ||
        (rc = check_view(out, B, H, N, d_h, e, true)))
        return rc;
    if (!late_ok(late_block, late_ns, wait_ns)) return SSD_ERR_SHAPE;
    Args g{};
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
    g.B = B, g.H = H, g.N = N, g.d = d_h;
    g.aligned = alignment_of({x, gate, out}, d_h, e);
    const Cut p = cut_of(B, H, N, d_h, dtype);
    g.nblk = p.nblk;
    const LateArgs late = late_args(g, late_block, late_ns, wait_ns);
    return launch_fwd(g, late_block < 0 ? nullptr : &late, p, dtype, mode_of(flags), static_cast<cudaStream_t>(stream));
}

int ssd_glr_fwd(const ssd_view *x, const ssd_view *gate, const float *A_log, const float *dt_bias,
                const float *h0, const int *lengths, int B, int H, int N, int d_h, int dtype, int flags,
                const ssd_view *out, float *h_out, float *states, void *stream) {
    return ssd_debug_glr_fwd(x, gate, A_log, dt_bias, h0, lengths, B, H, N, d_h, dtype, flags, out, h_out, states, stream,
                             -1, 0, 0);
}

size_t ssd_glr_bwd_workspace_bytes(int B, int H, int N, int d_h, int dtype, int flags) {
    if (check_glr(B, H, N, d_h, dtype, flags, nullptr, 0) != SSD_OK) return 0;
    const Cut p = cut_of(B, H, N, d_h, dtype);
    return align_up((size_t)B * p.cluster * H * d_h * 2 * sizeof(float), 256);
}

int ssd_debug_glr_bwd(const ssd_view *dy, const ssd_view *x, const ssd_view *gate, const float *A_log,
                      const float *dt_bias, const float *states, const int *lengths, const float *dh_out,
                      int B, int H, int N, int d_h, int dtype, int flags, const ssd_view *dx,
                      const ssd_view *dgate, float *dA_log, float *ddt_bias, float *dh0, void *workspace,
                      size_t workspace_bytes, void *stream, int late_block, long long late_ns,
                      long long wait_ns) {
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
    if (!late_ok(late_block, late_ns, wait_ns)) return SSD_ERR_SHAPE;
    Args g{};
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
    if (params) g.part = static_cast<float *>(workspace);
    g.B = B, g.H = H, g.N = N, g.d = d_h;
    g.aligned = alignment_of({dy, x, gate, dx, dgate}, d_h, e);
    const Cut p = cut_of(B, H, N, d_h, dtype);
    g.nblk = p.nblk;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const LateArgs late = late_args(g, late_block, late_ns, wait_ns);
    rc = launch_bwd(g, late_block < 0 ? nullptr : &late, p, dtype, mode_of(flags), s);
    if (rc != SSD_OK || !params) return rc;
    return sum_parts(g.part, (unsigned)(B * p.cluster), 2 * C, (int)C, dA_log, ddt_bias, s);
}

int ssd_glr_bwd(const ssd_view *dy, const ssd_view *x, const ssd_view *gate, const float *A_log,
                const float *dt_bias, const float *states, const int *lengths, const float *dh_out,
                int B, int H, int N, int d_h, int dtype, int flags, const ssd_view *dx,
                const ssd_view *dgate, float *dA_log, float *ddt_bias, float *dh0, void *workspace,
                size_t workspace_bytes, void *stream) {
    return ssd_debug_glr_bwd(dy, x, gate, A_log, dt_bias, states, lengths, dh_out, B, H, N, d_h, dtype, flags, dx, dgate,
                             dA_log, ddt_bias, dh0, workspace, workspace_bytes, stream, -1, 0, 0);
}

int ssd_glr_step(const ssd_view *x, const ssd_view *gate, const float *A_log, const float *dt_bias, int B,
                 int H, int d_h, int dtype, int flags, float *h, const ssd_view *out, void *stream) {
    if (!x || !gate || !h || !out) return SSD_ERR_NULL;
    const void *f32[] = {A_log, dt_bias, h};
    int rc = check_glr(B, H, 1, d_h, dtype, flags, f32, 3);
    if (rc != SSD_OK) return rc;
    const size_t e = elem_size(dtype);
    if ((rc = check_view(x, B, H, 1, d_h, e, false)) || (rc = check_view(gate, B, H, 1, d_h, e, false)) ||
        (rc = check_view(out, B, H, 1, d_h, e, true)))
        return rc;
    Args g{};
    g.x = *x;
    g.gate = *gate;
    g.out = *out;
    const bool log = flags & SSD_GLR_LOG_DECAY;
    g.A_log = log ? nullptr : A_log;
    g.dt_bias = log ? nullptr : dt_bias;
    g.h0 = h;
    g.h_out = h;
    g.B = B, g.H = H, g.N = 1, g.d = d_h;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned grid = blocks_for((long long)B * H * d_h);
    if (dtype == SSD_F32)
        glr_step_kernel<float><<<grid, kThreads, 0, s>>>(g, mode_of(flags));
    else
        glr_step_kernel<__nv_bfloat16><<<grid, kThreads, 0, s>>>(g, mode_of(flags));
    return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // extern "C"
