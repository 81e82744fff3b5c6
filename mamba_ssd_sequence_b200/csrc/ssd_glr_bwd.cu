// Gradients of the gated linear recurrence.
//
// The tiles, threads and rounds of the forward pass, walked from the last
// round to the first: the adjoint l_t = dy_t + a_{t+1} l_{t+1} is the same kind
// of scan in the other direction.  The states that the forward pass saved, one
// per thread segment, restart h without a second scan, so a round reads x, the
// gate and dy once and writes dx and dgate once.
//
// A thread reduces its 16 tokens to three numbers each before the maps of the
// adjoint are joined: two in registers, one in the place of x and the gate in
// shared memory.  The second walk, which has l, is a handful of products.
//
// Floor: HBM, 10 bytes an element in bf16, 20 in fp32, and the states (0.25).
// Measured in bf16 with softplus gates: 134M elements in 303 us (1024 heads of 2048
// tokens; 4.5 TB/s), 16.8M in 62 us (16 heads of 16384, clusters of 8; 2.8 TB/s).
// What bounds it: the arithmetic (without the gates' 253 and 54 us), and in
// clusters the rounds' exchange (56 us without it).  Evaluating the softplus again
// in the second walk took 417 and 78 us.
#include "ssd_glr.cuh"

namespace ssd {
namespace glr {
namespace {

constexpr int kStages = 2;

// a and 1 - a of a decay a <= 1 in one number: 1 - a where that is below 1/2, else
// -a; so each keeps its own relative precision.
__device__ __forceinline__ float pack_decay(float a, float w) { return w < 0.5f ? w : -a; }
__device__ __forceinline__ void unpack_decay(float c, float &a, float &w) {
    const bool is_a = __float_as_int(c) < 0;  // -0 too
    a = is_a ? -c : 1.0f - c;
    w = is_a ? 1.0f + c : c;
}

template <typename T, int kCb>
constexpr size_t smem_bytes() {
    using Tl = Tile<T, kCb>;
    return (size_t)kStages * 3 * Tl::bytes + sizeof(MapsOf<T, kCb>);
}

template <typename T, int kCb, int kMode, bool kLate = false>
__global__ void __launch_bounds__(Threads<T>::n, 2) glr_bwd_kernel(const ArgsOf<kLate> g) {
    using Tl = Tile<T, kCb>;
    using M = ModeOf<kMode>;
    extern __shared__ __align__(128) unsigned char sm[];
    auto *maps = reinterpret_cast<MapsOf<T, kCb> *>(sm + kStages * 3 * Tl::bytes);

    uint32_t cluster;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cluster));
    const int rank = (int)ptx::cluster_ctarank();
    const long long blk = blockIdx.x / cluster;
    const int c0 = (int)(blk % g.nblk) * kCb;
    const int h = (int)((blk / g.nblk) % g.H), b = (int)(blk / g.nblk / g.H);
    const int lane = threadIdx.x % Tl::lanes, seg = threadIdx.x / Tl::lanes, c = c0 + 2 * lane;
    const bool on0 = c < g.d, on1 = c + 1 < g.d;
    const int len = length_of(g.lengths, b, g.N);

    const T *x = static_cast<const T *>(g.x.ptr) + b * g.x.stride_b + h * g.x.stride_h;
    const T *gate = static_cast<const T *>(g.gate.ptr) + b * g.gate.stride_b + h * g.gate.stride_h;
    const T *dy = static_cast<const T *>(g.dy.ptr) + b * g.dy.stride_b + h * g.dy.stride_h;
    const long long round_tok = (long long)cluster * Tl::tok;
    const int rounds = (int)((len + round_tok - 1) / round_tok);
    const long long chunks = (g.N + kSeg - 1) / kSeg;
    const float *states = g.states + ((long long)(b * g.H + h) * chunks) * g.d + c;
    auto first_token = [&](int i) { return (rounds - 1 - i) * round_tok + (long long)rank * Tl::tok; };
    auto fetch = [&](int i) {
        if (i < rounds) {
            unsigned char *st = sm + (i % kStages) * 3 * Tl::bytes;
            const long long t0 = first_token(i);
            fetch_tile<T, kCb>(st, x, g.x.stride_n, t0, len, c0, g.d, g.aligned);
            fetch_tile<T, kCb>(st + Tl::bytes, gate, g.gate.stride_n, t0, len, c0, g.d, g.aligned);
            fetch_tile<T, kCb>(st + 2 * Tl::bytes, dy, g.dy.stride_n, t0, len, c0, g.d, g.aligned);
        }
        cp_async_commit();
    };
    auto state_at = [&](int i) {
        const long long t0 = first_token(i) + seg * kSeg;
        float2 v = make_float2(0.0f, 0.0f);
        if (i < rounds && t0 < len) {
            if (on0) v.x = states[t0 / kSeg * g.d];
            if (on1) v.y = states[t0 / kSeg * g.d + 1];
        }
        return v;
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(i);
    float2 next_state = state_at(0);

    constexpr float log2e = 1.4426950408889634f;
    float2 nrate2 = both(-log2e), bias = make_float2(0.0f, 0.0f), carry = make_float2(0.0f, 0.0f);
    const long long pc = (long long)h * g.d + c, bc = (long long)b * g.H * g.d + pc;
    if (!M::log) {
        if (g.A_log) nrate2 = make_float2(on0 ? -log2e * expf(g.A_log[pc]) : 0.0f, on1 ? -log2e * expf(g.A_log[pc + 1]) : 0.0f);
        if (g.dt_bias) bias = make_float2(on0 ? g.dt_bias[pc] : 0.0f, on1 ? g.dt_bias[pc + 1] : 0.0f);
    }
    if (g.dh_out) carry = make_float2(on0 ? g.dh_out[bc] : 0.0f, on1 ? g.dh_out[bc + 1] : 0.0f);

    T *dx = static_cast<T *>(g.dx.ptr) + b * g.dx.stride_b + h * g.dx.stride_h + c;
    T *dgate = static_cast<T *>(g.dgate.ptr) + b * g.dgate.stride_b + h * g.dgate.stride_h + c;
    auto store = [&](T *o, float2 v) {
        if (g.aligned) {
            if (on0) store_pair(o, v);
        } else {
            if (on0) store_one(o, v.x);
            if (on1) store_one(o + 1, v.y);
        }
    };
    float2 sumA = make_float2(0.0f, 0.0f), sumb = make_float2(0.0f, 0.0f);
    const float2 nrate = mul2(nrate2, both(0.6931471806f));

    bool lost = false;
    init_maps(maps, (int)cluster);
    start_late<kLate>(g, rank);
    for (int i = 0; i < rounds; ++i) {
        cp_async_wait<kStages - 2>();
        __syncthreads();  // this round has arrived for every thread, and the one before it is consumed
        fetch(i + kStages - 1);
        unsigned char *st = sm + (i % kStages) * 3 * Tl::bytes;
        T *xc = own_column<T, kCb>(st);
        T *gc = own_column<T, kCb>(st + Tl::bytes);
        const T *yc = own_column<T, kCb>(st + 2 * Tl::bytes);
        const long long t0 = first_token(i) + seg * kSeg;
        const int valid = (int)max(0ll, min((long long)kSeg, len - t0));
        if (!M::log && valid < kSeg) close_gates<T, kCb>(gc, valid);
        float2 hs = next_state;
        next_state = state_at(i + 1);
        // With q = a h_{t-1} (a (h_{t-1} - x) for f = 1 - a), d log a = l q.  All
        // that the second walk needs but l goes into three numbers a token:
        //   c   a, or for f = dt that, or for f = 1 - a one of 1 - a and -a
        //   r   dgate / l
        //   z   softplus gates: d A_log's term / l; log-decays: f = 1 - a
        float2 c[kSeg], r[kSeg], sum = both(0.0f), decay = both(1.0f), first = both(0.0f);  // l behind -> a_0 l_0
#pragma unroll
        for (int k = 0; k < kSeg; ++k) {
            const float2 xv = load_pair(xc + k * kCb), yv = load_pair(yc + k * kCb);
            const Gate o = gate_of<T, kMode>(load_pair(gc + k * kCb), bias, nrate2);
            const float2 q = mul2(o.a, M::complement ? add2(hs, neg2(xv)) : hs);
            hs = fma2(o.a, hs, value_of<kMode>(o, xv));
            sum = add2(sum, o.l);
            decay = mul2(decay, o.a);
            first = fma2(decay, yv, first);
            c[k] = M::dt ? o.f : o.a;
            if (M::log) {
                r[k] = q;
                if (M::complement) keep_pair(xc + k * kCb, gc + k * kCb, o.f);
            } else {
                if (M::complement) c[k] = make_float2(pack_decay(o.a.x, o.f.x), pack_decay(o.a.y, o.f.y));
                r[k] = mul2(slope_of(o), M::dt ? fma2(nrate, q, xv) : mul2(nrate, q));
                // the logarithm is kept finite, so that its product with a = 0 is 0
                keep_pair(xc + k * kCb, gc + k * kCb,
                          mul2(q, make_float2(fmaxf(o.l.x, -3.0e38f), fmaxf(o.l.y, -3.0e38f))));
            }
        }
        const float4 own = make_map(segment_decay(sum), first);
        float2 lc = enter_segment<T, kCb, false>(own, carry, maps, i, rank, (int)cluster, wait_limit<kLate>(g), lost);
        if (M::dt) {  // a is evaluated again: kept from above it would take the registers back
#pragma unroll
            for (int k = 0; k < kSeg; ++k) asm volatile("" : "+f"(c[k].x), "+f"(c[k].y));
        }
        float2 segA = both(0.0f), segb = both(0.0f);
        // token k: the gradients of x and the gate
        auto token = [&](int k, float2 *vx, float2 *vg) {
            const float2 l = add2(lc, load_pair(yc + k * kCb));
            const float2 z = M::log && !M::complement ? both(1.0f) : kept_pair(xc + k * kCb, gc + k * kCb);
            *vx = l;
            *vg = mul2(l, r[k]);
            float2 a = c[k];
            if (M::dt) {
                a = ex2(mul2(nrate2, c[k]));
                *vx = mul2(c[k], l);
            }
            if (M::complement && !M::log) {
                float2 f;
                unpack_decay(c[k].x, a.x, f.x);
                unpack_decay(c[k].y, a.y, f.y);
                *vx = mul2(f, l);
            }
            if (M::complement && M::log) *vx = mul2(z, l);
            lc = mul2(a, l);
            if (!M::log) {
                segA = fma2(l, z, segA);
                segb = add2(segb, *vg);
            }
        };
        if (g.aligned && valid == kSeg) {
            T *ox = dx + (t0 + kSeg - 1) * g.dx.stride_n, *og = dgate + (t0 + kSeg - 1) * g.dgate.stride_n;
#pragma unroll
            for (int k = kSeg - 1; k >= 0; --k, ox -= g.dx.stride_n, og -= g.dgate.stride_n) {
                float2 vx, vg;
                token(k, &vx, &vg);
                if (on0) {
                    store_pair(ox, vx);
                    store_pair(og, vg);
                }
            }
        } else {
#pragma unroll
            for (int k = kSeg - 1; k >= 0; --k) {
                float2 vx, vg;
                token(k, &vx, &vg);
                if (k >= valid) vx = vg = both(0.0f);
                if (t0 + k < g.N) {
                    store(dx + (t0 + k) * g.dx.stride_n, vx);
                    store(dgate + (t0 + k) * g.dgate.stride_n, vg);
                }
            }
        }
        sumA = make_float2(sumA.x + segA.x, sumA.y + segA.y);
        sumb = make_float2(sumb.x + segb.x, sumb.y + segb.y);
    }
    cp_async_wait<0>();

    // whole rounds behind the length
    for (long long t = rounds * round_tok + (long long)rank * Tl::tok + seg * kSeg; t < g.N; t += round_tok)
        for (int k = 0; k < kSeg && t + k < g.N; ++k) {
            store(dx + (t + k) * g.dx.stride_n, make_float2(0.0f, 0.0f));
            store(dgate + (t + k) * g.dgate.stride_n, make_float2(0.0f, 0.0f));
        }
    if (g.dh0 && rank == 0 && seg == 0) {
        if (on0) g.dh0[bc] = carry.x;
        if (on1) g.dh0[bc + 1] = carry.y;
    }
    // the block's sums of dA_log and ddt_bias, segment by segment
    if (!M::log && g.part) {
        __syncthreads();
        float4 *sums = reinterpret_cast<float4 *>(sm);
        constexpr float ln2 = 0.6931471806f;  // the terms are in units of log2 a
        sums[threadIdx.x] = make_float4(ln2 * sumA.x, sumb.x, ln2 * sumA.y, sumb.y);
        __syncthreads();
        if (seg == 0) {
            float4 v = sums[lane];
            for (int k = 1; k < Tl::segs; ++k) {
                const float4 o = sums[k * Tl::lanes + lane];
                v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
            }
            const long long C = (long long)g.H * g.d;
            float *part = g.part + ((long long)b * cluster + rank) * 2 * C + pc;
            if (on0) part[0] = v.x, part[C] = v.y;
            if (on1) part[1] = v.z, part[C + 1] = v.w;
        }
    }
    leave_cluster((int)cluster, lost);
}

template <typename T, int kCb>
int launch_mode(const Args &g, const LateArgs *late, const Cut &p, int mode, cudaStream_t s) {
    constexpr size_t sm = smem_bytes<T, kCb>();
    constexpr int nt = Threads<T>::n;
    if (late) {
        if constexpr (kCb == 16) {
            if (mode == kDtNone) return launch_cluster<glr_bwd_kernel<T, kCb, kDtNone, true>>(*late, p, nt, sm, s);
        }
        return SSD_ERR_UNSUPPORTED;
    }
    switch (mode) {
    case kDtNone: return launch_cluster<glr_bwd_kernel<T, kCb, kDtNone>>(g, p, nt, sm, s);
    case kDtDt: return launch_cluster<glr_bwd_kernel<T, kCb, kDtDt>>(g, p, nt, sm, s);
    case kDtComplement: return launch_cluster<glr_bwd_kernel<T, kCb, kDtComplement>>(g, p, nt, sm, s);
    case kLogNone: return launch_cluster<glr_bwd_kernel<T, kCb, kLogNone>>(g, p, nt, sm, s);
    default: return launch_cluster<glr_bwd_kernel<T, kCb, kLogComplement>>(g, p, nt, sm, s);
    }
}

template <typename T>
int launch_cb(const Args &g, const LateArgs *late, const Cut &p, int mode, cudaStream_t s) {
    return p.cb == 64 ? launch_mode<T, 64>(g, late, p, mode, s)
                      : p.cb == 32 ? launch_mode<T, 32>(g, late, p, mode, s) : launch_mode<T, 16>(g, late, p, mode, s);
}

}  // namespace

int launch_bwd(const Args &g, const LateArgs *late, const Cut &p, int dtype, int mode, cudaStream_t s) {
    return dtype == SSD_F32 ? launch_cb<float>(g, late, p, mode, s) : launch_cb<__nv_bfloat16>(g, late, p, mode, s);
}

}  // namespace glr
}  // namespace ssd
