// Norms before and after a block (ssd.h): the residual add with its scale and
// a root-mean-square norm, the gated root-mean-square norm behind the
// operator, and their gradients.
//
// A block walks the rows (a token, or a token's group of channels) of one
// slab; a thread always meets the same channels, so the gradients of the
// per-channel parameters are summed by one thread each over the slab's rows,
// and then over the slabs in order.
#include <cuda_bf16.h>
#include <math.h>

#include "ssd_internal.h"
#include "ssd_view.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Sum over the block, the same in every thread.
__device__ __forceinline__ float block_sum(float v) {
    __shared__ float red[kThreads / 32];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (threadIdx.x % 32 == 0) red[threadIdx.x / 32] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) s += red[i];
    return s;
}

struct AddNormArgs {
    ssd_rows x, res, r, out, dy, dres, dr, dx;
    const float *scale, *w;
    float *rstd, *part;
    int M, C;
    float eps;
};

template <typename T>
__device__ __forceinline__ T *row_of(const ssd_rows &v, long long m) {
    return v.ptr ? static_cast<T *>(v.ptr) + m * v.stride : nullptr;
}

template <typename T, typename R>
__global__ void __launch_bounds__(kThreads) add_norm_kernel(AddNormArgs g) {
    for (long long m = blockIdx.x; m < g.M; m += gridDim.x) {
        const T *x = row_of<const T>(g.x, m);
        const R *res = row_of<const R>(g.res, m);
        R *r = row_of<R>(g.r, m);
        T *out = row_of<T>(g.out, m);
        // the product and the sum are rounded one after the other, as two operations on the stream are
        auto stream_value = [&](int c) {
            float v = to_f32(x[c]);
            if (g.scale) v = __fmul_rn(g.scale[c], v);
            if (res) v = __fadd_rn(to_f32(res[c]), v);
            return from_f32<R>(v);
        };
        float ss = 0.0f;
        for (int c = threadIdx.x; c < g.C; c += kThreads) {
            const float v = to_f32(stream_value(c));
            ss = fmaf(v, v, ss);
        }
        const float rs = rsqrtf(block_sum(ss) / g.C + g.eps);
        for (int c = threadIdx.x; c < g.C; c += kThreads) {
            const R v = stream_value(c);
            if (r) r[c] = v;
            out[c] = from_f32<T>(to_f32(v) * rs * (g.w ? g.w[c] : 1.0f));
        }
        if (g.rstd && threadIdx.x == 0) g.rstd[m] = rs;
    }
}

template <typename T, typename R>
__global__ void __launch_bounds__(kThreads) add_norm_bwd_kernel(AddNormArgs g) {
    float *pw = g.part ? g.part + (long long)blockIdx.x * 2 * g.C : nullptr, *ps = pw ? pw + g.C : nullptr;
    if (pw)
        for (int c = threadIdx.x; c < g.C; c += kThreads) pw[c] = ps[c] = 0.0f;
    for (long long m = blockIdx.x; m < g.M; m += gridDim.x) {
        const R *r = row_of<const R>(g.r, m);
        const T *dy = row_of<const T>(g.dy, m);
        const T *x = row_of<const T>(g.x, m);
        const R *dres = row_of<const R>(g.dres, m);
        R *dr = row_of<R>(g.dr, m);
        T *dx = row_of<T>(g.dx, m);
        const float rs = g.rstd[m];
        float dot = 0.0f;
        for (int c = threadIdx.x; c < g.C; c += kThreads)
            dot = fmaf(to_f32(dy[c]) * (g.w ? g.w[c] : 1.0f), to_f32(r[c]) * rs, dot);
        dot = block_sum(dot) / g.C;
        for (int c = threadIdx.x; c < g.C; c += kThreads) {
            const float d = to_f32(dy[c]), xhat = to_f32(r[c]) * rs;
            float v = rs * fmaf(-xhat, dot, d * (g.w ? g.w[c] : 1.0f));
            if (dres) v += to_f32(dres[c]);
            if (pw) {
                pw[c] = fmaf(d, xhat, pw[c]);
                if (x) ps[c] = fmaf(v, to_f32(x[c]), ps[c]);
            }
            dr[c] = from_f32<R>(v);
            if (dx) dx[c] = from_f32<T>(g.scale ? v * g.scale[c] : v);
        }
    }
}

// Sums of the slabs' partial rows, in order.
__global__ void __launch_bounds__(kThreads) sum_parts_kernel(const float *part, int slabs, long long stride, int C,
                                                            float *out) {
    const int c = blockIdx.x * kThreads + threadIdx.x;
    if (c >= C) return;
    float s = 0.0f;
    for (int i = 0; i < slabs; ++i) s += part[i * stride + c];
    out[c] = s;
}

struct GatedNormArgs {
    ssd_view x, z, out, dy, dx, dz;
    const float *w;
    float *rstd, *part;
    int B, H, N, d, groups, after;
    float eps;
};

__device__ __forceinline__ long long offset_of(const ssd_view &v, int b, int n, int c, int d) {
    return b * v.stride_b + n * v.stride_n + (c / d) * v.stride_h + c % d;
}

template <typename T, bool kBackward>
__global__ void __launch_bounds__(kThreads) gated_norm_kernel(GatedNormArgs g) {
    const int C = g.H * g.d, L = C / g.groups;
    const long long tokens = (long long)g.B * g.N;
    const int c0 = blockIdx.y * L;
    float *pw = kBackward && g.part ? g.part + (long long)blockIdx.x * C + c0 : nullptr;
    if (pw)
        for (int c = threadIdx.x; c < L; c += kThreads) pw[c] = 0.0f;
    for (long long m = blockIdx.x; m < tokens; m += gridDim.x) {
        const int b = (int)(m / g.N), n = (int)(m % g.N);
        auto at = [&](const ssd_view &v, int c) { return static_cast<T *>(v.ptr) + offset_of(v, b, n, c0 + c, g.d); };
        auto gate = [&](int c, float *sig) {
            const float z = to_f32(*at(g.z, c));
            *sig = 1.0f / (1.0f + expf(-z));
            return z;
        };
        float *rstd = g.rstd ? g.rstd + m * g.groups + blockIdx.y : nullptr;
        if (!kBackward) {
            float ss = 0.0f;
            for (int c = threadIdx.x; c < L; c += kThreads) {
                float u = to_f32(*at(g.x, c)), sig;
                if (g.z.ptr && !g.after) u *= gate(c, &sig) * sig;
                ss = fmaf(u, u, ss);
            }
            const float rs = rsqrtf(block_sum(ss) / L + g.eps);
            for (int c = threadIdx.x; c < L; c += kThreads) {
                float u = to_f32(*at(g.x, c)) * rs, sig;
                if (g.z.ptr) u *= gate(c, &sig) * sig;
                *at(g.out, c) = from_f32<T>(g.w ? u * g.w[c0 + c] : u);
            }
            if (rstd && threadIdx.x == 0) *rstd = rs;
        } else {
            const float rs = *rstd;
            float dot = 0.0f;
            for (int c = threadIdx.x; c < L; c += kThreads) {
                const float dy = to_f32(*at(g.dy, c)), x = to_f32(*at(g.x, c));
                float sig = 0.0f, s = 1.0f;
                if (g.z.ptr) s = gate(c, &sig) * sig;
                // xhat (.) g is the same product in both orders of gate and norm
                dot = fmaf(dy * s * (g.w ? g.w[c0 + c] : 1.0f), x * rs, dot);
            }
            dot = block_sum(dot) / L;
            for (int c = threadIdx.x; c < L; c += kThreads) {
                const float dy = to_f32(*at(g.dy, c)), x = to_f32(*at(g.x, c)), w = g.w ? g.w[c0 + c] : 1.0f;
                float sig = 0.0f, s = 1.0f, z = 0.0f;
                if (g.z.ptr) {
                    z = gate(c, &sig);
                    s = z * sig;
                }
                float dx, ds;
                if (g.after) {
                    dx = rs * fmaf(-x * rs, dot, dy * s * w);
                    ds = dy * x * rs * w;
                } else {
                    const float du = rs * fmaf(-x * s * rs, dot, dy * w);
                    dx = du * s;
                    ds = du * x;
                }
                if (pw) pw[c] = fmaf(dy * s, x * rs, pw[c]);
                *at(g.dx, c) = from_f32<T>(dx);
                if (g.z.ptr) *at(g.dz, c) = from_f32<T>(ds * sig * (1.0f + z * (1.0f - sig)));
            }
        }
    }
}

unsigned slabs_for(long long rows) { return (unsigned)(rows < 592 ? rows : 592); }

bool eps_ok(float eps) { return eps > 0.0f && eps < 1e30f; }

int check_add(int M, int C, int dtype, int res_dtype) {
    if ((dtype != SSD_F32 && dtype != SSD_BF16) || (res_dtype != dtype && res_dtype != SSD_F32)) return SSD_ERR_DTYPE;
    return sizes_ok(1, 1, M, C) ? SSD_OK : SSD_ERR_SHAPE;
}

int check_gated(int B, int H, int N, int d, int dtype, int groups) {
    if (dtype != SSD_F32 && dtype != SSD_BF16) return SSD_ERR_DTYPE;
    if (!sizes_ok(B, H, N, d) || groups < 1 || groups > 65535 || ((long long)H * d) % groups) return SSD_ERR_SHAPE;
    return SSD_OK;
}

int launched() { return cudaGetLastError() == cudaSuccess ? SSD_OK : SSD_ERR_CUDA; }

}  // namespace
}  // namespace ssd

using namespace ssd;

extern "C" {

int ssd_add_norm(const ssd_rows *x, const ssd_rows *residual, const float *scale, const float *w, int M,
                 int C, int dtype, int res_dtype, const ssd_norm_params *p, const ssd_rows *r,
                 const ssd_rows *out, float *rstd, void *stream) {
    if (!x || !out || !p) return SSD_ERR_NULL;
    if (!r && (residual || scale || dtype != res_dtype)) return SSD_ERR_NULL;
    int rc = check_add(M, C, dtype, res_dtype);
    if (rc != SSD_OK) return rc;
    if (!eps_ok(p->eps)) return SSD_ERR_SHAPE;
    const size_t e = elem_size(dtype), er = elem_size(res_dtype);
    if ((rc = check_rows(x, M, C, e, false)) || (rc = check_rows(out, M, C, e, true)) ||
        (residual && (rc = check_rows(residual, M, C, er, false))) || (r && (rc = check_rows(r, M, C, er, true))))
        return rc;
    if (misaligned(scale, 4) || misaligned(w, 4) || misaligned(rstd, 4)) return SSD_ERR_ALIGN;
    AddNormArgs g{};
    g.x = *x;
    if (residual) g.res = *residual;
    if (r) g.r = *r;
    g.out = *out;
    g.scale = scale, g.w = w, g.rstd = rstd, g.M = M, g.C = C, g.eps = p->eps;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SSD_F32)
        add_norm_kernel<float, float><<<slabs_for(M), kThreads, 0, s>>>(g);
    else if (res_dtype == SSD_F32)
        add_norm_kernel<__nv_bfloat16, float><<<slabs_for(M), kThreads, 0, s>>>(g);
    else
        add_norm_kernel<__nv_bfloat16, __nv_bfloat16><<<slabs_for(M), kThreads, 0, s>>>(g);
    return launched();
}

size_t ssd_add_norm_bwd_workspace_bytes(int M, int C) {
    if (!sizes_ok(1, 1, M, C)) return 0;
    return align_up((size_t)slabs_for(M) * 2 * C * sizeof(float), 256);
}

int ssd_add_norm_bwd(const ssd_rows *dy, const ssd_rows *r, const float *rstd, const float *w,
                     const ssd_rows *x, const float *scale, const ssd_rows *dres, int M, int C, int dtype,
                     int res_dtype, const ssd_rows *dr, const ssd_rows *dx, float *dw, float *dscale,
                     void *workspace, size_t workspace_bytes, void *stream) {
    if (!dy || !r || !rstd || !dr || (dscale && !x)) return SSD_ERR_NULL;
    int rc = check_add(M, C, dtype, res_dtype);
    if (rc != SSD_OK) return rc;
    const size_t e = elem_size(dtype), er = elem_size(res_dtype);
    if ((rc = check_rows(dy, M, C, e, false)) || (rc = check_rows(r, M, C, er, false)) ||
        (rc = check_rows(dr, M, C, er, true)) || (dscale && (rc = check_rows(x, M, C, e, false))) ||
        (dres && (rc = check_rows(dres, M, C, er, false))) || (dx && (rc = check_rows(dx, M, C, e, true))))
        return rc;
    const void *f32[] = {rstd, w, scale, dw, dscale};
    for (const void *q : f32)
        if (misaligned(q, 4)) return SSD_ERR_ALIGN;
    if (!workspace || workspace_bytes < ssd_add_norm_bwd_workspace_bytes(M, C)) return SSD_ERR_WORKSPACE;
    if (misaligned(workspace, 256)) return SSD_ERR_ALIGN;
    AddNormArgs g{};
    g.dy = *dy;
    g.r = *r;
    g.dr = *dr;
    if (dscale) g.x = *x;
    if (dres) g.dres = *dres;
    if (dx) g.dx = *dx;
    g.scale = scale, g.w = w, g.rstd = const_cast<float *>(rstd), g.M = M, g.C = C;
    if (dw || dscale) g.part = static_cast<float *>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    const unsigned slabs = slabs_for(M);
    if (dtype == SSD_F32)
        add_norm_bwd_kernel<float, float><<<slabs, kThreads, 0, s>>>(g);
    else if (res_dtype == SSD_F32)
        add_norm_bwd_kernel<__nv_bfloat16, float><<<slabs, kThreads, 0, s>>>(g);
    else
        add_norm_bwd_kernel<__nv_bfloat16, __nv_bfloat16><<<slabs, kThreads, 0, s>>>(g);
    const unsigned cb = (unsigned)((C + kThreads - 1) / kThreads);
    if (dw) sum_parts_kernel<<<cb, kThreads, 0, s>>>(g.part, (int)slabs, 2ll * C, C, dw);
    if (dscale) sum_parts_kernel<<<cb, kThreads, 0, s>>>(g.part + C, (int)slabs, 2ll * C, C, dscale);
    return launched();
}

int ssd_gated_norm(const ssd_view *x, const ssd_view *z, const float *w, int B, int H, int N, int d_h,
                   int dtype, const ssd_norm_params *p, const ssd_view *out, float *rstd, void *stream) {
    if (!x || !out || !p) return SSD_ERR_NULL;
    int rc = check_gated(B, H, N, d_h, dtype, p->groups);
    if (rc != SSD_OK) return rc;
    if (p->flags & ~SSD_NORM_GATE_AFTER) return SSD_ERR_FLAGS;
    if (!eps_ok(p->eps)) return SSD_ERR_SHAPE;
    const size_t e = elem_size(dtype);
    if ((rc = check_view(x, B, H, N, d_h, e, false)) || (z && (rc = check_view(z, B, H, N, d_h, e, false))) ||
        (rc = check_view(out, B, H, N, d_h, e, true)))
        return rc;
    if (misaligned(w, 4) || misaligned(rstd, 4)) return SSD_ERR_ALIGN;
    GatedNormArgs g{};
    g.x = *x;
    if (z) g.z = *z;
    g.out = *out;
    g.w = w, g.rstd = rstd, g.B = B, g.H = H, g.N = N, g.d = d_h, g.groups = p->groups;
    g.after = p->flags & SSD_NORM_GATE_AFTER, g.eps = p->eps;
    const dim3 grid(slabs_for((long long)B * N), p->groups);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SSD_F32)
        gated_norm_kernel<float, false><<<grid, kThreads, 0, s>>>(g);
    else
        gated_norm_kernel<__nv_bfloat16, false><<<grid, kThreads, 0, s>>>(g);
    return launched();
}

size_t ssd_gated_norm_bwd_workspace_bytes(int B, int H, int N, int d_h, int groups) {
    if (check_gated(B, H, N, d_h, SSD_F32, groups) != SSD_OK) return 0;
    return align_up((size_t)slabs_for((long long)B * N) * H * d_h * sizeof(float), 256);
}

int ssd_gated_norm_bwd(const ssd_view *dy, const ssd_view *x, const ssd_view *z, const float *w,
                       const float *rstd, int B, int H, int N, int d_h, int dtype,
                       const ssd_norm_params *p, const ssd_view *dx, const ssd_view *dz, float *dw,
                       void *workspace, size_t workspace_bytes, void *stream) {
    if (!dy || !x || !rstd || !dx || !p || !z != !dz) return SSD_ERR_NULL;
    int rc = check_gated(B, H, N, d_h, dtype, p->groups);
    if (rc != SSD_OK) return rc;
    if (p->flags & ~SSD_NORM_GATE_AFTER) return SSD_ERR_FLAGS;
    const size_t e = elem_size(dtype);
    if ((rc = check_view(dy, B, H, N, d_h, e, false)) || (rc = check_view(x, B, H, N, d_h, e, false)) ||
        (z && (rc = check_view(z, B, H, N, d_h, e, false))) || (rc = check_view(dx, B, H, N, d_h, e, true)) ||
        (dz && (rc = check_view(dz, B, H, N, d_h, e, true))))
        return rc;
    if (misaligned(w, 4) || misaligned(rstd, 4) || misaligned(dw, 4)) return SSD_ERR_ALIGN;
    if (!workspace || workspace_bytes < ssd_gated_norm_bwd_workspace_bytes(B, H, N, d_h, p->groups))
        return SSD_ERR_WORKSPACE;
    if (misaligned(workspace, 256)) return SSD_ERR_ALIGN;
    GatedNormArgs g{};
    g.dy = *dy;
    g.x = *x;
    if (z) g.z = *z;
    g.dx = *dx;
    if (dz) g.dz = *dz;
    g.w = w, g.rstd = const_cast<float *>(rstd), g.B = B, g.H = H, g.N = N, g.d = d_h, g.groups = p->groups;
    g.after = p->flags & SSD_NORM_GATE_AFTER;
    if (dw) g.part = static_cast<float *>(workspace);
    const unsigned slabs = slabs_for((long long)B * N);
    const dim3 grid(slabs, p->groups);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SSD_F32)
        gated_norm_kernel<float, true><<<grid, kThreads, 0, s>>>(g);
    else
        gated_norm_kernel<__nv_bfloat16, true><<<grid, kThreads, 0, s>>>(g);
    const int C = H * d_h;
    if (dw) sum_parts_kernel<<<(C + kThreads - 1) / kThreads, kThreads, 0, s>>>(g.part, (int)slabs, C, C, dw);
    return launched();
}

}  // extern "C"
