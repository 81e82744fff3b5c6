// Device parts shared by the kernels of the gated linear recurrence
// (ssd_glr_fwd.cu, ssd_glr_bwd.cu, ssd_glr.cu).
//
// A tile is kTok tokens of kCb channels.  A thread holds two neighbouring
// channels of a segment of SSD_GLR_CHUNK consecutive tokens, so a warp reads
// whole rows of the tile; the segments of a block follow one another in time,
// and so do the blocks of a cluster.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <type_traits>

#include "ptx.cuh"
#include "ssd_internal.h"
#include "ssd_math.cuh"
#include "ssd_view.h"

namespace ssd {
namespace glr {

constexpr int kSeg = SSD_GLR_CHUNK;  // tokens per thread and per saved state
constexpr int kMaxCluster = 8;

struct Args {
    ssd_view x, gate, out, dy, dx, dgate;
    const float *A_log, *dt_bias, *h0, *dh_out;
    const int *lengths;
    float *h_out, *states, *dh0, *part;
    int B, H, N, d, nblk;
    int aligned;  // all views: 2 by 16 bytes, 1 by two elements, 0 by one
};

// The failure tests' kernels: one block of each cluster starts late, and a wait has a
// limit of its own.  Kernels and arguments apart from the others', since the delay takes
// registers (padded gradients 34.2 us, 33.0 without) and longer arguments a launch's time
// (a decode step 4.0 us, 3.65 without).
constexpr long long kWaitNs = 1000000000;  // the usual limit
struct LateArgs : Args {
    long long wait_ns, late_ns;
    int late;
};
template <bool kLate>
using ArgsOf = std::conditional_t<kLate, LateArgs, Args>;
template <bool kLate>
__device__ __forceinline__ long long wait_limit(const ArgsOf<kLate> &g) {
    if constexpr (kLate)
        return g.wait_ns;
    else
        return kWaitNs;
}
template <bool kLate>
__device__ __forceinline__ void start_late(const ArgsOf<kLate> &g, int rank) {
    if constexpr (kLate) {
        if (rank == g.late) ptx::sleep_for((uint64_t)g.late_ns);
    }
}

// Gate kinds and value factors, as template arguments.
enum Mode { kDtNone = 0, kDtDt = 1, kDtComplement = 2, kLogNone = 3, kLogComplement = 4 };
template <int kMode>
struct ModeOf {
    static constexpr bool log = kMode >= kLogNone;
    static constexpr bool dt = kMode == kDtDt;
    static constexpr bool complement = kMode == kDtComplement || kMode == kLogComplement;
};

// Block size: 16 KB of each activation per tile in both types.
template <typename T>
struct Threads;
template <>
struct Threads<float> { static constexpr int n = 128; };
template <>
struct Threads<__nv_bfloat16> { static constexpr int n = 256; };

template <typename T, int kCb>
struct Tile {
    static constexpr int nt = Threads<T>::n;
    static constexpr int lanes = kCb / 2;            // threads per row
    static constexpr int segs = nt / lanes;          // segments per tile
    static constexpr int per_warp = 32 / lanes;      // segments per warp
    static constexpr int warps = nt / 32;
    static constexpr int tok = segs * kSeg;
    static constexpr int row = kCb * (int)sizeof(T);  // bytes
    // a warp's segments start in different banks
    static constexpr int seg = kSeg * row + (per_warp > 1 ? row : 0);
    static constexpr int bytes = segs * seg;          // one activation
};

__device__ __forceinline__ float2 load_pair(const float *p) { return *reinterpret_cast<const float2 *>(p); }
__device__ __forceinline__ float2 load_pair(const __nv_bfloat16 *p) {
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ void store_pair(float *p, float2 v) { *reinterpret_cast<float2 *>(p) = v; }
__device__ __forceinline__ void store_pair(__nv_bfloat16 *p, float2 v) {
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(v.x, v.y);
}
// Two fp32 values in the places of a thread's own x and gate of a token, once
// it has read those: registers are scarcer than shared memory here.
__device__ __forceinline__ void keep_pair(float *x, float *, float2 v) { store_pair(x, v); }
__device__ __forceinline__ float2 kept_pair(const float *x, const float *) { return load_pair(x); }
__device__ __forceinline__ void keep_pair(__nv_bfloat16 *x, __nv_bfloat16 *gate, float2 v) {
    *reinterpret_cast<float *>(x) = v.x;
    *reinterpret_cast<float *>(gate) = v.y;
}
__device__ __forceinline__ float2 kept_pair(const __nv_bfloat16 *x, const __nv_bfloat16 *gate) {
    return make_float2(*reinterpret_cast<const float *>(x), *reinterpret_cast<const float *>(gate));
}
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void store_one(float *p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16 *p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ float minus_infinity() { return __uint_as_float(0xFF800000u); }

// q of exp(s) = 1 + s q(s) for |s| < 1/2 (1 - exp(-t) = t q(-t): coefficients from
// mamba_ssd_sequence_b200/gen_decay_poly.py, relative error 2.1e-7).
__device__ __forceinline__ float2 decay_poly(float2 s) {
    float2 p = both(1.398218563e-03f);
    p = fma2(p, s, both(8.408029564e-03f));
    p = fma2(p, s, both(4.166579247e-02f));
    p = fma2(p, s, both(1.666596532e-01f));
    p = fma2(p, s, both(5.000000000e-01f));
    return fma2(p, s, both(1.000000119e+00f));
}
// The larger one; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 ex2(float2 x) { return make_float2(ptx::ex2_approx(x.x), ptx::ex2_approx(x.y)); }

// a = 2^l.  The hardware exponential is off by 1.4e-7 at most, but by -2e-8 on
// the mean (measured over l in [-0.5, 0]), which adds up over the many tokens
// that a slow decay spans.  So a segment's product of decays is evaluated
// from the sum of its l, near 1 by the polynomial (segment_decay), and the
// hardware's error acts within a segment only.
__device__ __forceinline__ float2 exact_decay(float2 l, float2 *one_minus) {
    const float2 la = mul2(l, both(0.6931471806f)), q = decay_poly(la), e = ex2(l);
    const float2 c = fma2(la, q, both(1.0f)), w = mul2(la, q);
    const bool sx = fabsf(la.x) < 0.5f, sy = fabsf(la.y) < 0.5f;
    *one_minus = make_float2(sx ? -w.x : 1.0f - e.x, sy ? -w.y : 1.0f - e.y);
    return make_float2(sx ? c.x : e.x, sy ? c.y : e.y);
}

// dt = softplus(p) = max(p, 0) + log1p(u), u = exp(-|p|), with the polynomial
// of softplus_fast (ssd_math.cuh).  u is the hardware's base-2 exponential of m log2(e),
// m = -|p|, whose argument is rounded: |p| 2^-24 of u and of a small dt (8e-7 at dt =
// 1e-6).  For bf16 activations that is far below the 2^-9 |p| which the gate's own type
// leaves open.  For fp32 ones u is corrected by what the rounding left of m: with e2
// the rounded argument, u (1 + (m - e2 ln 2)), which leaves 0.05 |p| 2^-24 (ln 2 in
// fp32 is off by 2.8e-9 relative).  m is kept finite for that; 2^-288 is 0 as well.
// 134M elements of 32 heads forward in fp32: 277 us, 272 without, 293 with expf().
template <typename T>
__device__ __forceinline__ float2 softplus2(float2 p, float2 *u_out) {
    float2 u;
    if constexpr (sizeof(T) == 4) {
        const float2 m = make_float2(max_nan(-fabsf(p.x), -200.0f), max_nan(-fabsf(p.y), -200.0f));
        const float2 e2 = mul2(m, both(1.4426950408889634f)), e = ex2(e2);
        u = fma2(e, fma2(e2, both(-0.6931471806f), m), e);
    } else {
        const float2 p2 = mul2(p, both(1.4426950408889634f));
        u = ex2(make_float2(-fabsf(p2.x), -fabsf(p2.y)));
    }
    float2 q = both(5.126102362e-03f);
    q = fma2(q, u, both(-2.907406539e-02f));
    q = fma2(q, u, both(7.751608640e-02f));
    q = fma2(q, u, both(-1.360224783e-01f));
    q = fma2(q, u, both(1.907688081e-01f));
    q = fma2(q, u, both(-2.483539879e-01f));
    q = fma2(q, u, both(3.331812024e-01f));
    q = fma2(q, u, both(-4.999944568e-01f));
    q = fma2(q, u, both(9.999999404e-01f));
    *u_out = u;
    return fma2(u, q, make_float2(fmaxf(p.x, 0.0f), fmaxf(p.y, 0.0f)));
}

// One token of two channels.
struct Gate {
    float2 l;      // log2 a
    float2 a, f;   // the decay, the factor of x (f = 1 is not used)
    float2 p, u;   // softplus gates: gate + bias, exp(-|p|)
};

// nrate2 = -exp(A_log) log2(e).  l is -infinity where a decay is 0 by an infinite
// gate.  a is the hardware's exponential in both types: the rounding of l makes it off
// by |log a| 2^-24 relative, which is at most 0.37 2^-24 of the state that it multiplies.
template <typename T, int kMode>
__device__ __forceinline__ Gate gate_of(float2 g, float2 bias, float2 nrate2) {
    using M = ModeOf<kMode>;
    Gate o;
    if (M::log) {
        o.l = mul2(g, both(1.4426950408889634f));
    } else {
        o.p = add2(g, bias);
        o.f = softplus2<T>(o.p, &o.u);
        o.l = mul2(nrate2, o.f);
    }
    if (M::complement)
        o.a = exact_decay(o.l, &o.f);
    else
        o.a = ex2(o.l);
    return o;
}
// f x
template <int kMode>
__device__ __forceinline__ float2 value_of(const Gate &o, float2 x) {
    return kMode == kDtNone || kMode == kLogNone ? x : mul2(o.f, x);
}
// d dt / d p = sigmoid(p)
__device__ __forceinline__ float2 slope_of(const Gate &o) {
    const float2 v = add2(both(1.0f), o.u);
    return mul2(make_float2(o.p.x >= 0.0f ? 1.0f : o.u.x, o.p.y >= 0.0f ? 1.0f : o.u.y),
                make_float2(ptx::rcp_approx(v.x), ptx::rcp_approx(v.y)));
}
// the map of a segment from the sum of its log2 a
__device__ __forceinline__ float2 segment_decay(float2 sum) {
    float2 w;
    return exact_decay(sum, &w);
}

__device__ __forceinline__ int length_of(const int *lengths, int b, int N) {
    return lengths ? min(max(lengths[b], 0), N) : N;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void *src, bool valid) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(valid ? 4 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int n>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(n) : "memory");
}
// Writes 16 bytes to a block of the cluster and counts them at its mbarrier:
// the reader needs no fence, and the writer's other stores are not waited for.
__device__ __forceinline__ void st_async_f4(uint32_t cluster_addr, uint32_t cluster_bar, float4 v) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%2, %3, %4, %5}, [%1];" ::"r"(
                     cluster_addr),
                 "r"(cluster_bar), "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w)
                 : "memory");
}

// fetch_tile() of views that are not 16-byte aligned; a call, so that its registers
// are not taken from the others.
template <typename T, int kCb>
__device__ __noinline__ void fetch_unaligned(unsigned char *dst, const T *base, long long stride_n, long long t0, int len,
                                             int c0, int d, int aligned) {
    using Tl = Tile<T, kCb>;
    if (sizeof(T) == 4 || aligned == 1) {
        constexpr int vec = 4 / sizeof(T), cpr = kCb / vec, per_thread = Tl::tok * cpr / Tl::nt, step = Tl::nt / cpr;
        const int col = (threadIdx.x % cpr) * vec, row0 = threadIdx.x / cpr;
        const bool cv = c0 + col < d;
        const uint32_t s = ptx::smem_u32(dst) + col * (int)sizeof(T);
#pragma unroll 8
        for (int i = 0; i < per_thread; ++i) {
            const int row = row0 + i * step;
            const bool v = cv && t0 + row < len;
            cp_async4(s + row / kSeg * Tl::seg + row % kSeg * Tl::row, v ? base + (t0 + row) * stride_n + c0 + col : base, v);
        }
    } else {
        constexpr int per_thread = Tl::tok * kCb / Tl::nt, step = Tl::nt / kCb, batch = 16;
        static_assert(per_thread % batch == 0, "");
        const int col = threadIdx.x % kCb, row0 = threadIdx.x / kCb;
        const bool cv = c0 + col < d;
        T *out = reinterpret_cast<T *>(dst) + col;
#pragma unroll 1
        for (int i0 = 0; i0 < per_thread; i0 += batch) {
            T v[batch];
#pragma unroll
            for (int i = 0; i < batch; ++i) {
                const long long t = t0 + row0 + (i0 + i) * step;
                v[i] = cv && t < len ? base[t * stride_n + c0 + col] : T(0.0f);
            }
#pragma unroll
            for (int i = 0; i < batch; ++i) {
                const int row = row0 + (i0 + i) * step;
                out[(row / kSeg * Tl::seg + row % kSeg * Tl::row) / (int)sizeof(T)] = v[i];
            }
        }
    }
}

// Fetches a tile of one activation (base: its token 0, channel 0; tokens from
// t0, channels from c0) into shared memory.  Places at or behind token `len`
// or channel `d` receive 0.  Aligned views go through asynchronous copies of 16
// bytes, others of 4; where those would not be aligned either (bf16 at odd
// elements), through registers.
template <typename T, int kCb>
__device__ __forceinline__ void fetch_tile(unsigned char *dst, const T *base, long long stride_n, long long t0, int len,
                                           int c0, int d, int aligned) {
    using Tl = Tile<T, kCb>;
    if (aligned == 2) {
        constexpr int vec = 16 / sizeof(T), cpr = kCb / vec, per_thread = Tl::tok * cpr / Tl::nt, step = Tl::nt / cpr;
        constexpr int pad = Tl::seg - kSeg * Tl::row;
        static_assert(step % kSeg == 0 || pad == 0, "the thread's rows are evenly spaced in shared memory");
        const int col = (threadIdx.x % cpr) * vec, row0 = threadIdx.x / cpr;
        const bool cv = c0 + col < d;
        uint32_t s = ptx::smem_u32(dst) + col * (int)sizeof(T) + row0 * Tl::row + row0 / kSeg * pad;
        const T *p = cv ? base + (t0 + row0) * stride_n + c0 + col : base;
        const long long hop = cv ? step * stride_n : 0;
        if (t0 + Tl::tok <= len) {
#pragma unroll
            for (int i = 0; i < per_thread; ++i, p += hop) cp_async16(s + i * (step * Tl::row + step / kSeg * pad), p, cv);
        } else {
#pragma unroll
            for (int i = 0; i < per_thread; ++i, p += hop) {
                const bool v = cv && t0 + row0 + i * step < len;
                cp_async16(s + i * (step * Tl::row + step / kSeg * pad), v ? p : base, v);
            }
        }
    } else {
        fetch_unaligned<T, kCb>(dst, base, stride_n, t0, len, c0, d, aligned);
    }
}

// The 16-token column pair of this thread in a fetched tile.
template <typename T, int kCb>
__device__ __forceinline__ T *own_column(unsigned char *tile) {
    using Tl = Tile<T, kCb>;
    return reinterpret_cast<T *>(tile + (threadIdx.x / Tl::lanes) * Tl::seg) + 2 * (threadIdx.x % Tl::lanes);
}

// Softplus gates of tokens that do not count become -infinity (a = 1, dt = 0);
// a log-decay of 0, which the fetch left there, means the same.  A thread
// touches only what it reads itself.
template <typename T, int kCb>
__device__ __forceinline__ void close_gates(T *col, int valid) {
    for (int k = max(valid, 0); k < kSeg; ++k)
        store_pair(col + k * kCb, make_float2(minus_infinity(), minus_infinity()));
}

// The map h_in -> A h_in + h of two channels over a span of tokens, as {A0, A1,
// h0, h1}.  then(p, q): p's span, and q's after it in the direction of the scan.
__device__ __forceinline__ float4 make_map(float2 A, float2 h) { return make_float4(A.x, A.y, h.x, h.y); }
__device__ __forceinline__ float2 apply(float4 m, float2 h) {
    return fma2(make_float2(m.x, m.y), h, make_float2(m.z, m.w));
}
__device__ __forceinline__ float4 then(float4 p, float4 q) {
    return make_map(mul2(make_float2(p.x, p.y), make_float2(q.x, q.y)), apply(q, make_float2(p.z, p.w)));
}
__device__ __forceinline__ float4 identity_map() { return make_float4(1.0f, 1.0f, 0.0f, 0.0f); }
template <bool kUp>
__device__ __forceinline__ float4 shift(float4 m, int n) {
    float4 r;
    if (kUp) {
        r.x = __shfl_up_sync(0xffffffffu, m.x, n), r.y = __shfl_up_sync(0xffffffffu, m.y, n);
        r.z = __shfl_up_sync(0xffffffffu, m.z, n), r.w = __shfl_up_sync(0xffffffffu, m.w, n);
    } else {
        r.x = __shfl_down_sync(0xffffffffu, m.x, n), r.y = __shfl_down_sync(0xffffffffu, m.y, n);
        r.z = __shfl_down_sync(0xffffffffu, m.z, n), r.w = __shfl_down_sync(0xffffffffu, m.w, n);
    }
    return r;
}

// What the threads of a block, and the blocks of a cluster, tell one another:
// the maps of the block's warps, and those of the cluster's tiles for two
// rounds, each with an mbarrier that counts the tiles' bytes.  A block sends
// round r + 2 after it has every tile of round r + 1, whose block had then read
// round r: two rounds' places are enough.
template <int kLanes, int kWarps>
struct Maps {
    float4 warp[kWarps][kLanes];
    float4 tile[2][kMaxCluster][kLanes];
    uint64_t bar[2];
};
template <typename T, int kCb>
using MapsOf = Maps<Tile<T, kCb>::lanes, Tile<T, kCb>::warps>;

// Before the first round; ends with a barrier of the cluster, since peers may
// send as soon as they have passed it.
template <typename M>
__device__ __forceinline__ void init_maps(M *m, int cluster) {
    if (cluster == 1) return;
    if (threadIdx.x == 0) {
        const uint32_t bytes = (uint32_t)cluster * sizeof(m->tile[0][0]);
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(&m->bar[i], 1);
            ptx::mbar_arrive_expect_tx(&m->bar[i], bytes);
        }
        ptx::fence_mbar_init();
    }
    ptx::cluster_sync_all();
}

// The state (or, kForward false, the adjoint) that enters this thread's
// segment, given the segment's own map and the carry that enters the round's
// first tile (the last one, backwards); the carry is advanced over the whole
// round.  Every thread of the cluster takes part.
//
// A wait that runs out (never expected: the blocks of a cluster run together)
// makes the thread's carry NaN from this round on.  Such a thread neither waits
// nor sends nor announces bytes again: its round's phase is left as it is, and no
// peer can complete a phase with bytes of another round, or have a map overwritten
// that it has not read, since nothing is sent of round r + 2 unless all of r + 1
// has arrived.  Peers that wait for what is not sent run out in their turn.
template <typename T, int kCb, bool kForward>
__device__ __forceinline__ float2 enter_segment(float4 own, float2 &carry, MapsOf<T, kCb> *maps, int round, int rank,
                                                int cluster, long long wait_ns, bool &lost) {
    using Tl = Tile<T, kCb>;
    const int lane = threadIdx.x % Tl::lanes, warp = threadIdx.x / 32, in_warp = (threadIdx.x % 32) / Tl::lanes;
    // the maps of the segments before this one in its warp, and up to it
    float4 before = identity_map(), upto = own;
    if (Tl::per_warp > 1) {
#pragma unroll
        for (int n = 1; n < Tl::per_warp; n *= 2) {
            const float4 o = shift<kForward>(upto, n * Tl::lanes);
            if (kForward ? in_warp >= n : in_warp + n < Tl::per_warp) upto = then(o, upto);
        }
        const float4 o = shift<kForward>(upto, Tl::lanes);
        if (kForward ? in_warp > 0 : in_warp + 1 < Tl::per_warp) before = o;
    }
    if (in_warp == (kForward ? Tl::per_warp - 1 : 0)) maps->warp[warp][lane] = upto;
    __syncthreads();
    if (cluster == 1) {  // every thread joins the tile's map for itself
        float4 base = identity_map(), all = identity_map();
#pragma unroll
        for (int i = 0; i < Tl::warps; ++i) {
            const int w = kForward ? i : Tl::warps - 1 - i;
            const float4 m = maps->warp[w][lane];
            if (w == warp) base = all;
            all = i == 0 ? m : then(all, m);
        }
        const float2 h = apply(base, carry);
        carry = apply(all, carry);
        return Tl::per_warp > 1 ? apply(before, h) : h;
    }
    // the threads of the tile's last segment join and send the tile's map
    const int two = round & 1;
    if (warp == (kForward ? Tl::warps - 1 : 0) && in_warp == (kForward ? Tl::per_warp - 1 : 0) && !lost) {
        float4 all = maps->warp[kForward ? 0 : Tl::warps - 1][lane];
#pragma unroll
        for (int i = 1; i < Tl::warps - 1; ++i) all = then(all, maps->warp[kForward ? i : Tl::warps - 1 - i][lane]);
        all = then(all, upto);
        const uint32_t at = ptx::smem_u32(&maps->tile[two][rank][lane]), bar = ptx::smem_u32(&maps->bar[two]);
        for (int r = 0; r < cluster; ++r) st_async_f4(ptx::mapa_shared(at, r), ptx::mapa_shared(bar, r), all);
    }
    if (!lost) lost = !ptx::mbar_wait_cluster(&maps->bar[two], (round >> 1) & 1, (uint64_t)wait_ns);
    if (lost) carry = both(__uint_as_float(0x7FC00000u));
    // every thread waits for this phase itself; the next one's bytes are announced here
    if (threadIdx.x == 0 && !lost)
        ptx::mbar_arrive_expect_tx(&maps->bar[two], (uint32_t)cluster * sizeof(maps->tile[0][0]));
    float2 h = carry;
    for (int i = 0; i < cluster; ++i) {
        const int r = kForward ? i : cluster - 1 - i;
        if (r == rank) h = carry;
        carry = apply(maps->tile[two][r][lane], carry);
    }
    if (kForward) {
        for (int w = 0; w < warp; ++w) h = apply(maps->warp[w][lane], h);
    } else {
        for (int w = Tl::warps - 1; w > warp; --w) h = apply(maps->warp[w][lane], h);
    }
    return Tl::per_warp > 1 ? apply(before, h) : h;
}

// The end of a block: no block leaves while a peer may still write to its shared memory.  All
// is sent by then, and a thread that has waited for every round has received all;
// one that gave up stays for a millisecond more, for maps that are on their way.
__device__ __forceinline__ void leave_cluster(int cluster, bool lost) {
    if (cluster == 1) return;
    __syncwarp();  // the barrier is for whole warps, whose threads gave up each for itself
    ptx::cluster_sync_all();
    if (lost) ptx::sleep_for(1000000);
}

// How a call is cut up: blocks of cb channels, and `cluster` blocks that share
// a channel block's sequence, tile by tile.
struct Cut {
    int cb, cluster, nblk;
    long long blocks;
};
Cut cut_of(int B, int H, int N, int d, int dtype);

// `late`: the failure tests' kernel, or NULL (the others are then those of Args).
int launch_fwd(const Args &g, const LateArgs *late, const Cut &p, int dtype, int mode, cudaStream_t s);
int launch_bwd(const Args &g, const LateArgs *late, const Cut &p, int dtype, int mode, cudaStream_t s);

// Launches a kernel in clusters.  Its shared memory limit is set once per CUDA
// context (the driver never reuses a context's ID).
template <auto kernel, typename A>
int launch_cluster(const A &g, const Cut &p, int threads, size_t smem, cudaStream_t s) {
    static std::atomic<unsigned long long> set_in{0};
    unsigned long long id = 0;
    if (!current_context_id(&id) || set_in.load(std::memory_order_relaxed) != id + 1) {
        if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
            return SSD_ERR_CUDA;
        if (id) set_in.store(id + 1, std::memory_order_relaxed);
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)p.cluster;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)(p.blocks * p.cluster));
    c.blockDim = dim3((unsigned)threads);
    c.dynamicSmemBytes = smem;
    c.stream = s;
    c.attrs = attr;
    c.numAttrs = 1;
    return cudaLaunchKernelEx(&c, kernel, g) == cudaSuccess ? SSD_OK : SSD_ERR_CUDA;
}

}  // namespace glr
}  // namespace ssd
