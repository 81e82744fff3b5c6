// Norms before and after a block (ssd.h): the residual add with its scale and
// a root-mean-square norm, the gated root-mean-square norm behind the
// operator, and their gradients.
//
// A row (a token, or a token's group of channels) stays in the registers of
// `tpr` threads, kNv vectors of kVec channels each, from its one load to its
// one store.  A thread meets the same channels in every row, so the gradients
// of per-channel parameters are sums in registers, joined over a block's rows
// in shared memory and over the blocks by a second kernel, in a fixed order.
//
// Floor: HBM.  Measured in bf16: residual norm of 65536 x 2048 on an fp32 stream 248 us
// (6.5 TB/s, HBM-bound), its gradients 399 us (6.1 TB/s); gated norm of the
// same rows 147 us (5.5 TB/s), bounded by issue slots (71 % active, 27 instructions a
// channel); its gradients 312 us (4.3 TB/s), bounded by latency: four warps a scheduler
// and about 40 instructions a channel keep 54 % of the issue slots active.
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>

#include "ptx.cuh"
#include "ssd_internal.h"
#include "ssd_math.cuh"
#include "ssd_view.h"

namespace ssd {
namespace {

constexpr int kThreads = 256;  // of a block, unless a row takes more

// ------------------------------------------------------------ vectors of a row
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// 16 bytes of a type
template <typename T>
constexpr int kVecOf = 16 / (int)sizeof(T);

// The words of a vector as it is stored.
template <typename T, int kVec>
__device__ __forceinline__ void pack(const float (&v)[kVec], uint32_t (&w)[kVec * sizeof(T) / 4]) {
#pragma unroll
    for (int i = 0; i < kVec * (int)sizeof(T) / 4; ++i) {
        if constexpr (sizeof(T) == 4) {
            w[i] = __float_as_uint(v[i]);
        } else {
            const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t *>(&b);
        }
    }
}
template <int kWords>
__device__ __forceinline__ void store16(void *p, const uint32_t (&w)[kWords]) {
#pragma unroll
    for (int i = 0; i < kWords / 4; ++i)
        static_cast<uint4 *>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

// kVec channels of a row as they were loaded: the next row's are fetched before
// the present one is reduced, and take few registers until then.  Where rows,
// views and parameters are not all 16-byte aligned, each vector goes by the widest
// loads that its own address allows, and channel by channel at a row's end
// (`left` channels remain, the rest reads 0); a thread holds the same channels
// either way, so the sums have the same bits.
template <typename T, int kVec, bool kAligned>
struct Raw {
    static constexpr int n = kVec * (int)sizeof(T) / 16;
    uint32_t w[4 * n];
    __device__ __forceinline__ void load16(const void *p) {
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const uint4 q = static_cast<const uint4 *>(p)[i];
            w[4 * i] = q.x, w[4 * i + 1] = q.y, w[4 * i + 2] = q.z, w[4 * i + 3] = q.w;
        }
    }
    __device__ __forceinline__ void set(int e, T v) {  // element e, from the first on
        if constexpr (sizeof(T) == 4) {
            w[e] = __float_as_uint(v);
        } else {
            const uint32_t bits = __bfloat16_as_ushort(v);
            w[e / 2] = e % 2 ? w[e / 2] | bits << 16 : bits;
        }
    }
    __device__ __forceinline__ void load(const T *p, int left) {
        if constexpr (kAligned) {
            load16(p);
        } else {
            const uintptr_t at = reinterpret_cast<uintptr_t>(p);
            if (left >= kVec && at % 16 == 0) {
                load16(p);
            } else if (left >= kVec && at % 8 == 0) {
#pragma unroll
                for (int i = 0; i < 2 * n; ++i) {
                    const uint2 q = reinterpret_cast<const uint2 *>(p)[i];
                    w[2 * i] = q.x, w[2 * i + 1] = q.y;
                }
            } else if (left >= kVec && at % 4 == 0) {
#pragma unroll
                for (int i = 0; i < 4 * n; ++i) w[i] = reinterpret_cast<const uint32_t *>(p)[i];
            } else {
#pragma unroll
                for (int e = 0; e < kVec; ++e) set(e, e < left ? p[e] : T(0.0f));
            }
        }
    }
    // the same across heads of d channels, `hop` apart
    __device__ __forceinline__ void load_heads(const T *p, long long hop, int j, int d, int left) {
        if (j + kVec <= d) {
            load(p, left);
            return;
        }
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            set(e, e < left ? *p : T(0.0f));
            ++p;
            if (++j == d) j = 0, p += hop;
        }
    }
    __device__ __forceinline__ void get(float (&v)[kVec]) const {
#pragma unroll
        for (int k = 0; k < 4 * n; ++k) {
            if constexpr (sizeof(T) == 4) {
                v[k] = __uint_as_float(w[k]);
            } else {
                v[2 * k] = __uint_as_float(w[k] << 16);
                v[2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
            }
        }
    }
};
template <typename T, int kVec, bool kAligned>
__device__ __forceinline__ void get_pairs(const Raw<T, kVec, kAligned> &r, float2 (&v)[kVec / 2]) {
    float f[kVec];
    r.get(f);
#pragma unroll
    for (int e = 0; e < kVec / 2; ++e) v[e] = make_float2(f[2 * e], f[2 * e + 1]);
}
template <bool kAligned, typename T, int kVec>
__device__ __forceinline__ void store(T *p, int left, const float (&v)[kVec]) {
    constexpr int kWords = kVec * (int)sizeof(T) / 4;
    uint32_t w[kWords];
    pack<T>(v, w);
    if constexpr (kAligned) {
        store16(p, w);
    } else {
        const uintptr_t at = reinterpret_cast<uintptr_t>(p);
        if (left >= kVec && at % 16 == 0) {
            store16(p, w);
        } else if (left >= kVec && at % 4 == 0) {
#pragma unroll
            for (int i = 0; i < kWords; ++i) reinterpret_cast<uint32_t *>(p)[i] = w[i];
        } else {
#pragma unroll
            for (int e = 0; e < kVec; ++e)
                if (e < left) p[e] = from_f32<T>(v[e]);
        }
    }
}
// A thread's channels of a per-channel parameter.
template <bool kAligned, int kVec>
__device__ __forceinline__ void load_param(const float *p, int c, int left, float otherwise, float (&v)[kVec]) {
#pragma unroll
    for (int e = 0; e < kVec; ++e) v[e] = otherwise;
    if (p && left > 0) {
        Raw<float, kVec, kAligned> q;
        q.load(p + c, left);
        q.get(v);
    }
}

// Sum over a row's `tpr` threads (a power of two), the same bits in each.
// Rows of more than a warp meet in `red` ([2][32], by the parity of `turn`, so
// that one barrier a row is enough); every thread of the block calls this.
__device__ __forceinline__ float row_sum(float v, int tpr, float (*red)[32], int turn) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        if (o < tpr) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (tpr <= 32) return v;
    float *r = red[turn & 1];
    const int warp = threadIdx.x / 32, per_row = tpr / 32, first = warp / per_row * per_row;
    if (threadIdx.x % 32 == 0) r[warp] = v;
    __syncthreads();
    float s = r[first];
    for (int i = 1; i < per_row; ++i) s += r[first + i];
    return s;
}

// Joins the block's rows' sums of a per-channel gradient and writes them to
// the block's place.  `acc` is [kNv][kVec] of each thread; the rows that share
// channels are `rows` threads' worth of tpr apart by `step`.
template <int kNv, int kVec>
__device__ __forceinline__ void write_part(const float (&acc)[kNv][kVec], float *sh, int slot, int slots, int lane,
                                           int tpr, int same, int L, float *part) {
    // slots s, s + same, s + 2 same, ... hold the same channels
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kNv; ++i)
#pragma unroll
        for (int e = 0; e < kVec; ++e) sh[(i * kVec + e) * blockDim.x + threadIdx.x] = acc[i][e];
    __syncthreads();
    if (slot < same) {
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            const int c = (lane + i * tpr) * kVec;
            if (c < L) {
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    const float *p = sh + (i * kVec + e) * blockDim.x + threadIdx.x;
                    float s = p[0];
                    for (int k = same; k < slots; k += same) s += p[k * tpr];
                    if (c + e < L) part[c + e] = s;
                }
            }
        }
    }
}

template <typename T>
__device__ __forceinline__ T *row_of(const ssd_rows &v, long long m) {
    return v.ptr ? static_cast<T *>(v.ptr) + m * v.stride : nullptr;
}

// ------------------------------------------------------- residual add and norm
struct AddNormArgs {
    ssd_rows x, res, r, out, dy, dres, dr, dx;
    const float *scale, *w;
    float *rstd, *part;
    int M, C, tpr, want_scale;
    float eps;
};

template <typename T, typename R, bool kAligned, int kNv, int kMax>
__global__ void __launch_bounds__(kMax, kMax == kThreads ? (sizeof(T) == 2 ? 3 : 2) : 1) add_norm_kernel(const AddNormArgs g) {
    constexpr int kVec = kVecOf<T>;
    constexpr bool kAhead = kMax == kThreads;  // registers for the next row too
    __shared__ float red[2][32];
    const int tpr = g.tpr, lane = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr;
    const long long step = (long long)gridDim.x * slots;
    const bool has_res = g.res.ptr;
    const float inv_row = 1.0f / g.C;
    auto at = [&](int i) { return (lane + i * tpr) * kVec; };
    Raw<T, kVec, kAligned> x[kNv];
    Raw<R, kVec, kAligned> res[kNv];
    auto fetch = [&](long long m) {
        if (m >= g.M) return;
#pragma unroll
        for (int i = 0; i < kNv; ++i)
            if (at(i) < g.C) {
                x[i].load(row_of<const T>(g.x, m) + at(i), g.C - at(i));
                if (has_res) res[i].load(row_of<const R>(g.res, m) + at(i), g.C - at(i));
            }
    };
    long long m = (long long)blockIdx.x * slots + slot;
    if (kAhead) fetch(m);
    int turn = 0;
    for (long long m0 = (long long)blockIdx.x * slots; m0 < g.M; m0 += step, m += step, ++turn) {
        const bool on = m < g.M;
        if (!kAhead) fetch(m);
        float v[kNv][kVec], ss = 0.0f;
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if (on && at(i) < g.C) {
                x[i].get(v[i]);
                // the product and the sum are rounded one after the other, as
                // two operations on the stream are
                if (g.scale) {
                    float sc[kVec];
                    load_param<kAligned>(g.scale, at(i), g.C - at(i), 1.0f, sc);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) v[i][e] = __fmul_rn(sc[e], v[i][e]);
                }
                if (has_res) {
                    float q[kVec];
                    res[i].get(q);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) v[i][e] = __fadd_rn(q[e], v[i][e]);
                }
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    v[i][e] = to_f32(from_f32<R>(v[i][e]));
                    ss = fmaf(v[i][e], v[i][e], ss);
                }
            }
        }
        if (kAhead) fetch(m + step);
        const float rs = rsqrtf(row_sum(ss, tpr, red, turn) * inv_row + g.eps);
        if (!on) continue;
        R *r = row_of<R>(g.r, m);
        T *out = row_of<T>(g.out, m);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if (at(i) < g.C) {
                if (r) store<kAligned>(r + at(i), g.C - at(i), v[i]);
                float w[kVec];
                load_param<kAligned>(g.w, at(i), g.C - at(i), 1.0f, w);
#pragma unroll
                for (int e = 0; e < kVec; ++e) v[i][e] = v[i][e] * rs * w[e];
                store<kAligned>(out + at(i), g.C - at(i), v[i]);
            }
        }
        if (g.rstd && lane == 0) g.rstd[m] = rs;
    }
}

template <typename T, typename R, bool kAligned, int kNv, int kMax>
__global__ void __launch_bounds__(kMax, kMax == kThreads ? (sizeof(T) == 2 && kNv == 1 ? 3 : 2) : 1) add_norm_bwd_kernel(const AddNormArgs g) {
    constexpr int kVec = kVecOf<T>;
    constexpr bool kAhead = kMax == kThreads;  // registers for the next row too
    extern __shared__ float sh[];
    __shared__ float red[2][32];
    const int tpr = g.tpr, lane = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr;
    const long long step = (long long)gridDim.x * slots;
    const bool has_res = g.dres.ptr, has_x = g.x.ptr;
    const float inv_row = 1.0f / g.C;
    auto at = [&](int i) { return (lane + i * tpr) * kVec; };
    Raw<R, kVec, kAligned> r[kNv], dres[kNv];
    Raw<T, kVec, kAligned> dy[kNv], x[kNv];
    float rs = 0.0f;
    auto fetch = [&](long long m) {  // what the reduction needs; the rest follows before it
        if (m >= g.M) return;
        rs = g.rstd[m];
#pragma unroll
        for (int i = 0; i < kNv; ++i)
            if (at(i) < g.C) {
                r[i].load(row_of<const R>(g.r, m) + at(i), g.C - at(i));
                dy[i].load(row_of<const T>(g.dy, m) + at(i), g.C - at(i));
            }
    };
    auto fetch_rest = [&](long long m) {
        if (m >= g.M) return;
#pragma unroll
        for (int i = 0; i < kNv; ++i)
            if (at(i) < g.C) {
                if (has_res) dres[i].load(row_of<const R>(g.dres, m) + at(i), g.C - at(i));
                if (has_x) x[i].load(row_of<const T>(g.x, m) + at(i), g.C - at(i));
            }
    };
    long long m = (long long)blockIdx.x * slots + slot;
    if (kAhead) fetch(m);
    float dw[kNv][kVec] = {}, dsc[kNv][kVec] = {};
    int turn = 0;
    for (long long m0 = (long long)blockIdx.x * slots; m0 < g.M; m0 += step, m += step, ++turn) {
        const bool on = m < g.M;
        if (!kAhead) fetch(m);
        fetch_rest(m);
        const float rsm = rs;
        float xh[kNv][kVec], gy[kNv][kVec], dot = 0.0f;
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if (on && at(i) < g.C) {
                r[i].get(xh[i]);
                dy[i].get(gy[i]);
                float w[kVec];
                load_param<kAligned>(g.w, at(i), g.C - at(i), 1.0f, w);
#pragma unroll
                for (int e = 0; e < kVec; ++e) {
                    xh[i][e] *= rsm;
                    dw[i][e] = fmaf(gy[i][e], xh[i][e], dw[i][e]);
                    gy[i][e] *= w[e];
                    dot = fmaf(gy[i][e], xh[i][e], dot);
                }
            }
        }
        if (kAhead) fetch(m + step);
        dot = row_sum(dot, tpr, red, turn) * inv_row;
        if (!on) continue;
        R *dr = row_of<R>(g.dr, m);
        T *dx = row_of<T>(g.dx, m);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if (at(i) < g.C) {
                float q[kVec];
#pragma unroll
                for (int e = 0; e < kVec; ++e) gy[i][e] = rsm * fmaf(-xh[i][e], dot, gy[i][e]);
                if (has_res) {
                    dres[i].get(q);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) gy[i][e] += q[e];
                }
                store<kAligned>(dr + at(i), g.C - at(i), gy[i]);
                if (has_x) {
                    x[i].get(q);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) dsc[i][e] = fmaf(gy[i][e], q[e], dsc[i][e]);
                }
                if (dx) {
                    load_param<kAligned>(g.scale, at(i), g.C - at(i), 1.0f, q);
#pragma unroll
                    for (int e = 0; e < kVec; ++e) q[e] *= gy[i][e];
                    store<kAligned>(dx + at(i), g.C - at(i), q);
                }
            }
        }
    }
    if (g.part) {
        float *part = g.part + (long long)blockIdx.x * 2 * g.C;
        write_part<kNv, kVec>(dw, sh, slot, slots, lane, tpr, 1, g.C, part);
        if (g.want_scale) write_part<kNv, kVec>(dsc, sh, slot, slots, lane, tpr, 1, g.C, part + g.C);
    }
}

// Sums of the blocks' partial rows, in a fixed order: 32 channels and 32
// interleaved ranges of rows a block, so that all of a thread's few loads are in
// flight at once.  blockIdx.y selects the parameter.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float *part, int rows, long long stride, int C, float *out0,
                                                         float *out1) {
    __shared__ float red[32][33];
    const int lane = threadIdx.x % 32, k = threadIdx.x / 32, c = blockIdx.x * 32 + lane;
    float *out = blockIdx.y ? out1 : out0;
    part += (long long)blockIdx.y * C;
    float s = 0.0f;
    ptx::pdl_wait();
    if (c < C && out) {
#pragma unroll 8
        for (int i = k; i < rows; i += 32) s += part[i * stride + c];
    }
    red[k][lane] = s;
    __syncthreads();
    s = red[lane][k];  // channel blockIdx.x * 32 + k
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0 && blockIdx.x * 32 + k < C && out) out[blockIdx.x * 32 + k] = s;
}

// ------------------------------------------------------------------ gated norm
struct GatedNormArgs {
    ssd_view x, z, out, dy, dx, dz;
    const float *w;
    float *rstd, *part;
    int B, H, N, d, groups, gpb, L, tpr, after;
    float eps;
};

// SiLU's sigmoid.  For fp32 the library's exponential; for bf16 the hardware's,
// whose argument is rounded (|z| 2^-24 relative), far below the result's rounding.
template <typename T>
__device__ __forceinline__ float sigmoid(float z) {
    const float e = sizeof(T) == 4 ? expf(-z) : ptx::ex2_approx(z * -1.4426950408889634f);
    return ptx::rcp_approx(1.0f + e);
}

// A thread's place in one view, walked by a fixed number of tokens at a time: no
// division, and one addition a view.
template <typename T>
struct Walk {
    T *p;
    long long hop, wrap;  // of a step, and when it passes the end of a batch
    __device__ __forceinline__ Walk(const ssd_view &v, int b, int n, int h, int j, int step_b, int step_n, int N)
        : p(static_cast<T *>(v.ptr) + b * v.stride_b + n * v.stride_n + h * v.stride_h + j),
          hop(step_b * v.stride_b + step_n * v.stride_n), wrap(v.stride_b - N * v.stride_n) {}
    __device__ __forceinline__ void advance(bool wraps) { p += wraps ? hop + wrap : hop; }
};

enum GateKind { kNoGate = 0, kGateBefore = 1, kGateAfter = 2 };

// A vector of a token's channels from place j of a head on, in any of the
// views.  Unaligned vectors may run into the next head, `hop` behind this one.
template <typename T, int kVec, bool kAligned>
__device__ __forceinline__ void load_heads(Raw<T, kVec, kAligned> &q, const T *p, long long hop, int j, int d, int left) {
    if constexpr (kAligned)
        q.load16(p);
    else
        q.load_heads(p, hop, j, d, left);
}
template <bool kAligned, typename T, int kVec>
__device__ __forceinline__ void store_heads(T *p, long long hop, int j, int d, int left, const float (&v)[kVec]) {
    if (kAligned || j + kVec <= d) {
        store<kAligned>(p, left, v);
    } else {
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
            if (e < left) *p = from_f32<T>(v[e]);
            ++p;
            if (++j == d) j = 0, p += hop;
        }
    }
}

// A thread's own vectors of the rows to come, in shared memory: a ring of kDepth
// rows of kPer 16-byte pieces a thread, filled by asynchronous copies that take
// no registers and that only the thread itself waits for.  (Gated norm of 65536 x
// 2048, when it was added: 164 us, 196 with one row ahead in registers.  The residual norm moves
// more per channel, and is faster with registers: 248 us, 323 with a ring.)
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}
template <int kPer>
struct Ring {
    static constexpr int kDepth = kPer <= 8 ? 3 : 2;
    static constexpr size_t bytes(int threads) { return (size_t)kDepth * kPer * threads * 16; }
    const unsigned char *own;
    uint32_t at, piece, put, get;  // own's shared address; bytes between pieces, and of the rows' places
    __device__ __forceinline__ explicit Ring(void *smem)
        : own(static_cast<unsigned char *>(smem) + threadIdx.x * 16), at(ptx::smem_u32(own)), piece(blockDim.x * 16),
          put(0), get(0) {}
    __device__ __forceinline__ void next(uint32_t &row) const {
        row += kPer * piece;
        if (row == kDepth * kPer * piece) row = 0;
    }
    // piece `first` on of the row being put: one vector
    template <typename T, int kVec>
    __device__ __forceinline__ void copy(int first, const T *p) const {
#pragma unroll
        for (int i = 0; i < Raw<T, kVec, true>::n; ++i)
            copy16(at + put + (first + i) * piece, reinterpret_cast<const uint4 *>(p) + i);
    }
    __device__ __forceinline__ void put_done() {
        copies_commit();
        next(put);
    }
    __device__ __forceinline__ void get_wait() const { copies_wait<kDepth - 1>(); }
    template <typename T, int kVec>
    __device__ __forceinline__ void load(int first, Raw<T, kVec, true> &r) const {
#pragma unroll
        for (int i = 0; i < Raw<T, kVec, true>::n; ++i) {
            const uint4 q = *reinterpret_cast<const uint4 *>(own + get + (first + i) * piece);
            r.w[4 * i] = q.x, r.w[4 * i + 1] = q.y, r.w[4 * i + 2] = q.z, r.w[4 * i + 3] = q.w;
        }
    }
    __device__ __forceinline__ void get_done() { next(get); }
};

// Rows of at most kThreads threads are fetched ahead through a ring.
template <bool kAligned, int kMax>
constexpr bool kRings = kAligned && kMax <= kThreads;

// SiLU's sigmoid of a pair.
template <typename T>
__device__ __forceinline__ float2 sigmoid2(float2 z) {
    return make_float2(sigmoid<T>(z.x), sigmoid<T>(z.y));
}

template <typename T, bool kAligned, int kGate, int kNv, int kMax>
__global__ void __launch_bounds__(kMax, kMax == kThreads ? (sizeof(T) == 2 ? 3 : 2) : 1)
gated_norm_kernel(const GatedNormArgs g) {
    constexpr int kVec = kVecOf<T>, kPairs = kVec / 2;
    constexpr bool kRing = kRings<kAligned, kMax>, has_z = kGate != kNoGate, after = kGate == kGateAfter;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float red[2][32];
    const int tpr = g.tpr, lane = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr / g.gpb;
    const int group = blockIdx.y * g.gpb + slot % g.gpb, c0 = group * g.L;
    const long long tokens = (long long)g.B * g.N, step = (long long)gridDim.x * slots;
    const float inv_row = 1.0f / g.L;
    int h[kNv], j[kNv], left[kNv];
#pragma unroll
    for (int i = 0; i < kNv; ++i) {
        const int cl = (lane + i * tpr) * kVec;
        h[i] = (c0 + cl) / g.d, j[i] = (c0 + cl) % g.d, left[i] = g.L - cl;
    }
    // vector i of a view is this far behind vector 0
    auto off = [&](const ssd_view &v, int i) { return i ? (h[i] - h[0]) * v.stride_h + (j[i] - j[0]) : 0ll; };
    Ring<2 * kNv> ring(smem);
    const int step_b = (int)(step / g.N), step_n = (int)(step % g.N);
    long long m0 = (long long)blockIdx.x * slots, m = m0 + slot / g.gpb;
    const int b = (int)(m / g.N);
    unsigned n = (unsigned)(m - (long long)b * g.N), n_next = n;
    Walk<const T> x(g.x, b, n, h[0], j[0], step_b, step_n, g.N), z(g.z, b, n, h[0], j[0], step_b, step_n, g.N);
    Walk<T> out(g.out, b, n, h[0], j[0], step_b, step_n, g.N);
    long long ahead = m;
    auto fetch = [&]() {  // the next row to come
        if constexpr (kRing) {
            if (ahead < tokens) {
#pragma unroll
                for (int i = 0; i < kNv; ++i)
                    if (left[i] > 0) {
                        ring.template copy<T, kVec>(i, x.p + off(g.x, i));
                        if (has_z) ring.template copy<T, kVec>(kNv + i, z.p + off(g.z, i));
                    }
            }
            ring.put_done();
            ahead += step;
            const bool w = next_token(n_next, step_n, g.N);
            x.advance(w);
            if (has_z) z.advance(w);
        }
    };
#pragma unroll
    for (int k = 0; k + 1 < ring.kDepth; ++k) fetch();
    int turn = 0;
    for (; m0 < tokens; m0 += step, m += step, ++turn) {
        const bool on = m < tokens;
        fetch();
        if (kRing) ring.get_wait();
        float2 v[kNv][kPairs], ss = both(0.0f);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if (on && left[i] > 0) {
                Raw<T, kVec, kAligned> xr, zr;
                if constexpr (kRing) {
                    ring.load(i, xr);
                    if (has_z) ring.load(kNv + i, zr);
                } else {
                    load_heads(xr, x.p + off(g.x, i), g.x.stride_h - g.d, j[i], g.d, left[i]);
                    if (has_z) load_heads(zr, z.p + off(g.z, i), g.z.stride_h - g.d, j[i], g.d, left[i]);
                }
                float2 zv[kPairs];
                get_pairs(xr, v[i]);
                if (has_z) get_pairs(zr, zv);
#pragma unroll
                for (int e = 0; e < kPairs; ++e) {
                    if (after) ss = fma2(v[i][e], v[i][e], ss);
                    if (has_z) v[i][e] = mul2(v[i][e], mul2(zv[e], sigmoid2<T>(zv[e])));
                    if (!after) ss = fma2(v[i][e], v[i][e], ss);
                }
            }
        }
        ring.get_done();
        const float rs = rsqrtf(row_sum(ss.x + ss.y, tpr, red, turn) * inv_row + g.eps);
        if (on) {
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                if (left[i] > 0) {
                    float w[kVec];
                    load_param<kAligned>(g.w, c0 + g.L - left[i], left[i], 1.0f, w);
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) {
                        const float2 y = mul2(mul2(v[i][e], both(rs)), make_float2(w[2 * e], w[2 * e + 1]));
                        w[2 * e] = y.x, w[2 * e + 1] = y.y;
                    }
                    store_heads<kAligned>(out.p + off(g.out, i), g.out.stride_h - g.d, j[i], g.d, left[i], w);
                }
            }
            if (g.rstd && lane == 0) g.rstd[m * g.groups + group] = rs;
        }
        const bool w = next_token(n, step_n, g.N);
        out.advance(w);
        if (!kRing) {
            x.advance(w);
            if (has_z) z.advance(w);
        }
    }
}

template <typename T, bool kAligned, int kGate, int kNv, int kMax>
__global__ void __launch_bounds__(kMax, kMax == kThreads ? 2 : 1) gated_norm_bwd_kernel(const GatedNormArgs g) {
    constexpr int kVec = kVecOf<T>, kPairs = kVec / 2;
    constexpr bool kRing = kRings<kAligned, kMax>, has_z = kGate != kNoGate, after = kGate == kGateAfter;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float red[2][32];
    const int tpr = g.tpr, lane = threadIdx.x % tpr, slot = threadIdx.x / tpr, slots = blockDim.x / tpr / g.gpb;
    const int group = blockIdx.y * g.gpb + slot % g.gpb, c0 = group * g.L;
    const long long tokens = (long long)g.B * g.N, step = (long long)gridDim.x * slots;
    const float inv_row = 1.0f / g.L;
    int h[kNv], j[kNv], left[kNv];
    float dw[kNv][kVec] = {};
#pragma unroll
    for (int i = 0; i < kNv; ++i) {
        const int cl = (lane + i * tpr) * kVec;
        h[i] = (c0 + cl) / g.d, j[i] = (c0 + cl) % g.d, left[i] = g.L - cl;
    }
    auto off = [&](const ssd_view &v, int i) { return i ? (h[i] - h[0]) * v.stride_h + (j[i] - j[0]) : 0ll; };
    Ring<3 * kNv> ring(smem);
    const int step_b = (int)(step / g.N), step_n = (int)(step % g.N);
    long long m0 = (long long)blockIdx.x * slots, m = m0 + slot / g.gpb;
    const int b = (int)(m / g.N);
    unsigned n = (unsigned)(m - (long long)b * g.N), n_next = n;
    Walk<const T> x(g.x, b, n, h[0], j[0], step_b, step_n, g.N), z(g.z, b, n, h[0], j[0], step_b, step_n, g.N),
        dy(g.dy, b, n, h[0], j[0], step_b, step_n, g.N);
    Walk<T> dx(g.dx, b, n, h[0], j[0], step_b, step_n, g.N), dz(g.dz, b, n, h[0], j[0], step_b, step_n, g.N);
    long long ahead = m;
    auto fetch = [&]() {  // the next row to come
        if constexpr (kRing) {
            if (ahead < tokens) {
#pragma unroll
                for (int i = 0; i < kNv; ++i)
                    if (left[i] > 0) {
                        ring.template copy<T, kVec>(i, x.p + off(g.x, i));
                        ring.template copy<T, kVec>(kNv + i, dy.p + off(g.dy, i));
                        if (has_z) ring.template copy<T, kVec>(2 * kNv + i, z.p + off(g.z, i));
                    }
            }
            ring.put_done();
            ahead += step;
            const bool w = next_token(n_next, step_n, g.N);
            x.advance(w), dy.advance(w);
            if (has_z) z.advance(w);
        }
    };
#pragma unroll
    for (int k = 0; k + 1 < ring.kDepth; ++k) fetch();
    float rs_next = m < tokens ? g.rstd[m * g.groups + group] : 0.0f;
    int turn = 0;
    for (; m0 < tokens; m0 += step, m += step, ++turn) {
        const bool on = m < tokens;
        const float rs = rs_next;
        if (m + step < tokens) rs_next = g.rstd[(m + step) * g.groups + group];
        fetch();
        if (kRing) ring.get_wait();
        auto take = [&](int i, float2 (&xv)[kPairs], float2 (&yv)[kPairs]) {
            Raw<T, kVec, kAligned> xr, yr;
            if constexpr (kRing) {
                ring.load(i, xr);
                ring.load(kNv + i, yr);
            } else {
                load_heads(xr, x.p + off(g.x, i), g.x.stride_h - g.d, j[i], g.d, left[i]);
                load_heads(yr, dy.p + off(g.dy, i), g.dy.stride_h - g.d, j[i], g.d, left[i]);
            }
            get_pairs(xr, xv);
            get_pairs(yr, yv);
        };
        // SiLU(z) and its slope are kept over the reduction; x and dy too for one
        // vector, with more they are read again from where they lie (65536 x 2048: 322 us
        // when that was done, 458 with spills)
        constexpr bool kHold = kNv == 1;
        float2 hx[kPairs], hy[kPairs], sl[kNv][kPairs], sp[kNv][kPairs], dot2 = both(0.0f);
#pragma unroll
        for (int i = 0; i < kNv; ++i) {
            if (on && left[i] > 0) {
                float2 xv[kPairs], yv[kPairs], zv[kPairs];
                take(i, xv, yv);
                if (kHold) {
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) hx[e] = xv[e], hy[e] = yv[e];
                }
                if (has_z) {
                    Raw<T, kVec, kAligned> zr;
                    if constexpr (kRing)
                        ring.load(2 * kNv + i, zr);
                    else
                        load_heads(zr, z.p + off(g.z, i), g.z.stride_h - g.d, j[i], g.d, left[i]);
                    get_pairs(zr, zv);
                }
                float w[kVec];
                load_param<kAligned>(g.w, c0 + g.L - left[i], left[i], 1.0f, w);
#pragma unroll
                for (int e = 0; e < kPairs; ++e) {
                    float2 t = mul2(yv[e], mul2(xv[e], both(rs)));  // dy xhat, but for the gate
                    if (has_z) {
                        const float2 sig = sigmoid2<T>(zv[e]);
                        sl[i][e] = mul2(zv[e], sig);
                        // SiLU' = sig (1 + z (1 - sig)) = sig + SiLU (1 - sig)
                        sp[i][e] = fma2(sl[i][e], add2(both(1.0f), neg2(sig)), sig);
                        t = mul2(t, sl[i][e]);
                    }
                    dw[i][2 * e] += t.x, dw[i][2 * e + 1] += t.y;
                    dot2 = fma2(t, make_float2(w[2 * e], w[2 * e + 1]), dot2);
                }
            }
        }
        const float dot = row_sum(dot2.x + dot2.y, tpr, red, turn) * inv_row;
        if (on) {
            const float2 rs2 = both(rs), c = both(-rs * dot);
#pragma unroll
            for (int i = 0; i < kNv; ++i) {
                if (left[i] > 0) {
                    float2 xv[kPairs], yv[kPairs];
                    if (!kHold) take(i, xv, yv);
                    float w[kVec], vx[kVec], vz[kVec];
                    load_param<kAligned>(g.w, c0 + g.L - left[i], left[i], 1.0f, w);
#pragma unroll
                    for (int e = 0; e < kPairs; ++e) {
                        const float2 x1 = kHold ? hx[e] : xv[e], gw = mul2(kHold ? hy[e] : yv[e], make_float2(w[2 * e], w[2 * e + 1]));
                        float2 a, s;
                        if (!has_z) {
                            a = mul2(rs2, fma2(x1, c, gw));
                        } else if (after) {
                            a = mul2(rs2, fma2(x1, c, mul2(gw, sl[i][e])));
                            s = mul2(mul2(gw, mul2(x1, rs2)), sp[i][e]);
                        } else {
                            const float2 du = mul2(rs2, fma2(mul2(x1, sl[i][e]), c, gw));
                            a = mul2(du, sl[i][e]);
                            s = mul2(mul2(du, x1), sp[i][e]);
                        }
                        vx[2 * e] = a.x, vx[2 * e + 1] = a.y;
                        if (has_z) vz[2 * e] = s.x, vz[2 * e + 1] = s.y;
                    }
                    store_heads<kAligned>(dx.p + off(g.dx, i), g.dx.stride_h - g.d, j[i], g.d, left[i], vx);
                    if (has_z) store_heads<kAligned>(dz.p + off(g.dz, i), g.dz.stride_h - g.d, j[i], g.d, left[i], vz);
                }
            }
        }
        ring.get_done();
        const bool w = next_token(n, step_n, g.N);
        dx.advance(w);
        if (has_z) dz.advance(w);
        if (!kRing) {
            x.advance(w), dy.advance(w);
            if (has_z) z.advance(w);
        }
    }
    if (g.part) {
        copies_wait<0>();
        write_part<kNv, kVec>(dw, reinterpret_cast<float *>(smem), slot, slots * g.gpb, lane, tpr, g.gpb, g.L,
                              g.part + (long long)blockIdx.x * g.H * g.d + c0);
    }
}

// ------------------------------------------------------------------- wide rows
// Rows that no block holds in registers: a block walks a row twice, and its
// partial sums of the parameter gradients are in memory (one thread a channel).
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


template <typename T, typename R>
__global__ void __launch_bounds__(kThreads) add_norm_wide_kernel(AddNormArgs g) {
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
__global__ void __launch_bounds__(kThreads) add_norm_bwd_wide_kernel(AddNormArgs g) {
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

__device__ __forceinline__ long long offset_of(const ssd_view &v, int b, int n, int c, int d) {
    return b * v.stride_b + n * v.stride_n + (c / d) * v.stride_h + c % d;
}

template <typename T, bool kBackward>
__global__ void __launch_bounds__(kThreads) gated_norm_wide_kernel(GatedNormArgs g) {
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


// ------------------------------------------------------------------ the launch
// How rows of L channels are given to threads: vectors of 16 bytes, `nv` of them
// a thread, `tpr` threads a row, gpb groups a block side by side; nv = 0: a wide
// row.  A thread holds up to 16 values of a row (and backward as many sums), and
// the next row's as loaded.
struct Cut {
    int nv, tpr, threads, gpb;
    unsigned blocks;
};

constexpr int kSMs = 148;
constexpr size_t kMaxSmem = 104 * 1024;  // the largest ring: 96 KB
constexpr unsigned kMaxParts = 4 * kSMs;  // blocks of a backward pass: bounds its workspace

Cut cut_rows(int L, long long rows, int groups, size_t esize, bool backward, bool gated) {
    Cut c{};
    const int vec = (int)(16 / esize), n = (L + vec - 1) / vec, most = backward ? 512 : 1024;
    // the residual norm's gradients in bf16: one vector and three blocks an SM while a
    // row is at most a block (8192 x 1024: 27 us, 30 with two vectors and two blocks;
    // 65536 x 2048 on an fp32 stream: 399 us, 423)
    const bool light = backward && !gated && esize == 2 && n <= 256;
    c.nv = n <= 32 || light ? 1 : esize == 4 ? 4 : 2;
    c.tpr = 1;
    while (c.tpr * c.nv < n) c.tpr *= 2;
    c.gpb = 1;
    // rows that need a barrier wait for fewer others in a smaller block (gated norm of 65536 x
    // 2048, one row ahead: 203 us in blocks of 256, 196 of 128); a gradient's partial sums want large ones
    c.threads = !backward && c.tpr > 32 ? kThreads / 2 : kThreads;
    if (c.tpr > most) {
        c.nv = 0;
        c.blocks = (unsigned)(rows < 2 * kSMs ? rows : 2 * kSMs);
        return c;
    }
    if (c.tpr > c.threads) c.threads = c.tpr;
    // few rows: smaller blocks reach more SMs
    while (c.threads > 32 && c.threads > c.tpr && rows * groups * c.tpr < (long long)c.threads * kSMs) c.threads /= 2;
    while (c.gpb * 2 * c.tpr <= c.threads && groups % (c.gpb * 2) == 0) c.gpb *= 2;
    const long long slots = c.threads / c.tpr / c.gpb, want = (rows + slots - 1) / slots;
    // as many blocks as run at once
    const int per_sm = light ? 3 : backward || esize == 4 ? 2 : 3;
    long long most_blocks = (long long)per_sm * kSMs * kThreads / c.threads;
    if (backward && most_blocks > kMaxParts) most_blocks = kMaxParts;
    const unsigned gy = (unsigned)(groups / c.gpb);
    // a long forward pass in more blocks than run at once, of ten rows a slot: the SMs
    // stay evenly loaded to the end (residual norm of 65536 x 2048 on an fp32 stream: 290
    // us in 888 blocks, 247 in 6553; the gated norm of the same rows 143 and 147)
    if (!backward && want / 10 > most_blocks) most_blocks = want / 10;
    most_blocks = (most_blocks + gy - 1) / gy;
    c.blocks = (unsigned)(want < most_blocks ? want : most_blocks);
    return c;
}

// Dispatch on alignment, vectors a thread and the largest block.
#define SSD_NORM_DISPATCH(NVBIG, BIG, RUN)                             \
    do {                                                               \
        if (c.nv == 1) {                                               \
            if (aligned) { RUN(true, 1, kThreads); } else { RUN(false, 1, kThreads); } \
        } else if (c.threads <= kThreads) {                            \
            if (aligned) { RUN(true, NVBIG, kThreads); } else { RUN(false, NVBIG, kThreads); } \
        } else {                                                       \
            if (aligned) { RUN(true, NVBIG, BIG); } else { RUN(false, NVBIG, BIG); } \
        }                                                              \
    } while (0)

// Launches a kernel with `smem` bytes of dynamic shared memory, whose limit
// (48 KB with the static part, unless raised) is
// set once per CUDA context (the driver never reuses a context's ID).
template <auto kernel, typename A>
void launch(dim3 grid, const Cut &c, size_t smem, cudaStream_t s, const A &g) {
    static std::atomic<unsigned long long> set_in{0};
    unsigned long long id = 0;
    if (smem > 40 * 1024 && (!current_context_id(&id) || set_in.load(std::memory_order_relaxed) != id + 1)) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kMaxSmem) != cudaSuccess)
            return;  // the caller reads the error
        if (id) set_in.store(id + 1, std::memory_order_relaxed);
    }
    kernel<<<grid, c.threads, smem, s>>>(g);
}
size_t larger(size_t a, size_t b) { return a > b ? a : b; }
size_t part_bytes(const Cut &c, int vec) { return (size_t)c.threads * c.nv * vec * sizeof(float); }

template <typename T, typename R>
void run_add(const AddNormArgs &g, const Cut &c, bool aligned, cudaStream_t s) {
    if (c.nv == 0) {
        add_norm_wide_kernel<T, R><<<c.blocks, kThreads, 0, s>>>(g);
        return;
    }
#define RUN(AL, NV, MX) launch<add_norm_kernel<T, R, AL, NV, MX>>(dim3(c.blocks), c, 0, s, g)
    SSD_NORM_DISPATCH((sizeof(T) == 4 ? 4 : 2), 1024, RUN);
#undef RUN
}

template <typename T, typename R>
void run_add_bwd(const AddNormArgs &g, const Cut &c, bool aligned, cudaStream_t s) {
    if (c.nv == 0) {
        add_norm_bwd_wide_kernel<T, R><<<c.blocks, kThreads, 0, s>>>(g);
        return;
    }
    const size_t pb = g.part ? part_bytes(c, kVecOf<T>) : 0;
#define RUN(AL, NV, MX) launch<add_norm_bwd_kernel<T, R, AL, NV, MX>>(dim3(c.blocks), c, pb, s, g)
    SSD_NORM_DISPATCH((sizeof(T) == 4 ? 4 : 2), 512, RUN);
#undef RUN
}

template <typename T>
void run_gated(const GatedNormArgs &g, const Cut &c, bool aligned, cudaStream_t s) {
    if (c.nv == 0) {
        gated_norm_wide_kernel<T, false><<<dim3(c.blocks, g.groups), kThreads, 0, s>>>(g);
        return;
    }
    const dim3 grid(c.blocks, g.groups / c.gpb);
#define RUN(AL, NV, MX)                                                                         \
    {                                                                                           \
        const size_t rb = kRings<AL, MX> ? Ring<2 * NV>::bytes(c.threads) : 0;                  \
        if (!g.z.ptr) launch<gated_norm_kernel<T, AL, kNoGate, NV, MX>>(grid, c, rb, s, g);      \
        else if (g.after) launch<gated_norm_kernel<T, AL, kGateAfter, NV, MX>>(grid, c, rb, s, g); \
        else launch<gated_norm_kernel<T, AL, kGateBefore, NV, MX>>(grid, c, rb, s, g);           \
    }
    SSD_NORM_DISPATCH((sizeof(T) == 4 ? 4 : 2), 1024, RUN);
#undef RUN
}

template <typename T>
void run_gated_bwd(const GatedNormArgs &g, const Cut &c, bool aligned, cudaStream_t s) {
    if (c.nv == 0) {
        gated_norm_wide_kernel<T, true><<<dim3(c.blocks, g.groups), kThreads, 0, s>>>(g);
        return;
    }
    const dim3 grid(c.blocks, g.groups / c.gpb);
    const size_t pb = g.part ? part_bytes(c, kVecOf<T>) : 0;
#define RUN(AL, NV, MX)                                                                             \
    {                                                                                               \
        const size_t sm = larger(kRings<AL, MX> ? Ring<3 * NV>::bytes(c.threads) : 0, pb);            \
        if (!g.z.ptr) launch<gated_norm_bwd_kernel<T, AL, kNoGate, NV, MX>>(grid, c, sm, s, g);      \
        else if (g.after) launch<gated_norm_bwd_kernel<T, AL, kGateAfter, NV, MX>>(grid, c, sm, s, g); \
        else launch<gated_norm_bwd_kernel<T, AL, kGateBefore, NV, MX>>(grid, c, sm, s, g);           \
    }
    SSD_NORM_DISPATCH((sizeof(T) == 4 ? 4 : 2), 512, RUN);
#undef RUN
}

bool rows16(const ssd_rows &v, size_t esize) {
    return !misaligned(v.ptr, 16) && v.stride * (long long)esize % 16 == 0;
}
bool view16(const ssd_view &v, size_t esize) {
    return !misaligned(v.ptr, 16) && ((v.stride_b | v.stride_h | v.stride_n) * (long long)esize) % 16 == 0;
}

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

// The second step of the parameter gradients; starts while the first drains.
int sum_parts(const float *part, unsigned rows, long long stride, int C, float *out0, float *out1, cudaStream_t s) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)((C + 31) / 32), out1 ? 2 : 1);
    c.blockDim = dim3(1024);
    c.stream = s;
    c.attrs = pdl;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, sum_parts_kernel, part, (int)rows, stride, C, out0, out1) == cudaSuccess
               ? SSD_OK : SSD_ERR_CUDA;
}

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
    const bool aligned = rows16(g.x, e) && rows16(g.out, e) && rows16(g.res, er) && rows16(g.r, er) &&
                         !misaligned(scale, 16) && !misaligned(w, 16) && (C * e) % 16 == 0;
    const Cut c = cut_rows(C, M, 1, e, false, false);
    g.tpr = c.tpr;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SSD_F32)
        run_add<float, float>(g, c, aligned, s);
    else if (res_dtype == SSD_F32)
        run_add<__nv_bfloat16, float>(g, c, aligned, s);
    else
        run_add<__nv_bfloat16, __nv_bfloat16>(g, c, aligned, s);
    return launched();
}

size_t ssd_add_norm_bwd_workspace_bytes(int M, int C) {
    if (!sizes_ok(1, 1, M, C)) return 0;
    return align_up((size_t)(M < (int)kMaxParts ? M : kMaxParts) * 2 * C * sizeof(float), 256);
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
    g.want_scale = dscale != nullptr;
    const bool aligned = rows16(g.dy, e) && rows16(g.r, er) && rows16(g.dr, er) && rows16(g.x, e) && rows16(g.dres, er) &&
                         rows16(g.dx, e) && !misaligned(scale, 16) && !misaligned(w, 16) && (C * e) % 16 == 0;
    const Cut c = cut_rows(C, M, 1, e, true, false);
    g.tpr = c.tpr;
    if (dtype == SSD_F32)
        run_add_bwd<float, float>(g, c, aligned, s);
    else if (res_dtype == SSD_F32)
        run_add_bwd<__nv_bfloat16, float>(g, c, aligned, s);
    else
        run_add_bwd<__nv_bfloat16, __nv_bfloat16>(g, c, aligned, s);
    rc = launched();
    if (rc != SSD_OK || !g.part) return rc;
    return sum_parts(g.part, c.blocks, 2ll * C, C, dw, dscale, s);
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
    g.L = H * d_h / p->groups;
    // a vector lies in one head and one group
    const bool aligned = view16(g.x, e) && view16(g.z, e) && view16(g.out, e) && !misaligned(w, 16) &&
                         (d_h * e) % 16 == 0 && (g.L * e) % 16 == 0;
    const Cut c = cut_rows(g.L, (long long)B * N, g.groups, e, false, true);
    g.tpr = c.tpr, g.gpb = c.gpb;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SSD_F32)
        run_gated<float>(g, c, aligned, s);
    else
        run_gated<__nv_bfloat16>(g, c, aligned, s);
    return launched();
}

size_t ssd_gated_norm_bwd_workspace_bytes(int B, int H, int N, int d_h, int groups) {
    if (check_gated(B, H, N, d_h, SSD_F32, groups) != SSD_OK) return 0;
    const long long rows = (long long)B * N;
    return align_up((size_t)(rows < kMaxParts ? rows : kMaxParts) * H * d_h * sizeof(float), 256);
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
    g.L = H * d_h / p->groups;
    const bool aligned = view16(g.dy, e) && view16(g.x, e) && view16(g.z, e) && view16(g.dx, e) && view16(g.dz, e) &&
                         !misaligned(w, 16) && (d_h * e) % 16 == 0 && (g.L * e) % 16 == 0;
    const Cut c = cut_rows(g.L, (long long)B * N, g.groups, e, true, true);
    g.tpr = c.tpr, g.gpb = c.gpb;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (dtype == SSD_F32)
        run_gated_bwd<float>(g, c, aligned, s);
    else
        run_gated_bwd<__nv_bfloat16>(g, c, aligned, s);
    rc = launched();
    if (rc != SSD_OK || !dw) return rc;
    return sum_parts(g.part, c.blocks, (long long)H * d_h, H * d_h, dw, nullptr, s);
}

}  // extern "C"
