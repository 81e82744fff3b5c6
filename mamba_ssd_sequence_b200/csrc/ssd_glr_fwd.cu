// Forward pass of the gated linear recurrence h_t = a_t h_{t-1} + f_t x_t.
//
// A cluster takes one block of channels through its sequence in rounds of
// cluster x tile tokens.  In a round each thread evaluates the gates of its
// 16-token segment once, keeps a and f x in registers (x itself is read again
// where f = 1), and reduces them to the segment's map h_in -> A h_in + h; the
// maps are joined over the segments of a warp (shuffles), the warps of a block
// (shared memory) and the blocks of the cluster (distributed shared memory),
// which gives each segment its h_in; a second walk then gives h.  So x and the
// gate are read and h is written once, whatever the number of channels, and the
// result does not depend on timing.
//
// Floor: HBM, 6 bytes an element in bf16, 12 in fp32.  Measured in bf16: 134M elements
// in 159 us with a given log-decay, 32 heads of 65536 tokens (clusters of 8;
// 5.1 TB/s), and in 162 us with softplus gates, 1024 heads of 2048 (5.0 TB/s);
// 235 us with softplus gates and 32 heads.  What bounds it: the gates'
// arithmetic (25 to 40 instructions an element; without it 148 and 136 us) and, in
// clusters, the rounds' exchange (without it 142 us, 204 with softplus gates) with 256
// blocks on 148 SMs.  Tried and slower: 8 tokens a thread (the work per
// tile outweighs the higher occupancy: 310 us), blocks of 128 threads, clusters of
// 16, narrower channel blocks, three stages.
#include "ssd_glr.cuh"

namespace ssd {
namespace glr {
namespace {

constexpr int kStages = 2;

template <typename T, int kCb>
constexpr size_t smem_bytes() {
    using Tl = Tile<T, kCb>;
    return (size_t)kStages * 2 * Tl::bytes + sizeof(MapsOf<T, kCb>);
}

template <typename T, int kCb, int kMode, bool kLate = false>
__global__ void __launch_bounds__(Threads<T>::n, 2) glr_fwd_kernel(const ArgsOf<kLate> g) {
    using Tl = Tile<T, kCb>;
    using M = ModeOf<kMode>;
    constexpr bool kPlain = kMode == kDtNone || kMode == kLogNone;  // f x is x
    extern __shared__ __align__(128) unsigned char sm[];
    auto *maps = reinterpret_cast<MapsOf<T, kCb> *>(sm + kStages * 2 * Tl::bytes);

    uint32_t cluster;
    asm("mov.u32 %0, %%cluster_nctaid.x;" : "=r"(cluster));
    const int rank = (int)ptx::cluster_ctarank();
    const long long blk = blockIdx.x / cluster;
    const int c0 = (int)(blk % g.nblk) * kCb;
    const int h = (int)((blk / g.nblk) % g.H), b = (int)(blk / g.nblk / g.H);
    const int seg = threadIdx.x / Tl::lanes, c = c0 + 2 * (threadIdx.x % Tl::lanes);
    const bool on0 = c < g.d, on1 = c + 1 < g.d;
    const int len = length_of(g.lengths, b, g.N);

    const T *x = static_cast<const T *>(g.x.ptr) + b * g.x.stride_b + h * g.x.stride_h;
    const T *gate = static_cast<const T *>(g.gate.ptr) + b * g.gate.stride_b + h * g.gate.stride_h;
    const long long round_tok = (long long)cluster * Tl::tok;
    const int rounds = (int)((len + round_tok - 1) / round_tok);
    auto fetch = [&](int r) {
        if (r < rounds) {
            unsigned char *st = sm + (r % kStages) * 2 * Tl::bytes;
            const long long t0 = r * round_tok + (long long)rank * Tl::tok;
            fetch_tile<T, kCb>(st, x, g.x.stride_n, t0, len, c0, g.d, g.aligned);
            fetch_tile<T, kCb>(st + Tl::bytes, gate, g.gate.stride_n, t0, len, c0, g.d, g.aligned);
        }
        cp_async_commit();
    };
#pragma unroll
    for (int r = 0; r < kStages - 1; ++r) fetch(r);

    constexpr float log2e = 1.4426950408889634f;
    float2 nrate2 = both(-log2e), bias = make_float2(0.0f, 0.0f), carry = make_float2(0.0f, 0.0f);
    const long long pc = (long long)h * g.d + c, bc = (long long)b * g.H * g.d + pc;
    if (!M::log) {
        if (g.A_log) nrate2 = make_float2(on0 ? -log2e * expf(g.A_log[pc]) : 0.0f, on1 ? -log2e * expf(g.A_log[pc + 1]) : 0.0f);
        if (g.dt_bias) bias = make_float2(on0 ? g.dt_bias[pc] : 0.0f, on1 ? g.dt_bias[pc + 1] : 0.0f);
    }
    if (g.h0) carry = make_float2(on0 ? g.h0[bc] : 0.0f, on1 ? g.h0[bc + 1] : 0.0f);

    T *out = static_cast<T *>(g.out.ptr) + b * g.out.stride_b + h * g.out.stride_h + c;
    const long long chunks = (g.N + kSeg - 1) / kSeg;
    float *states = g.states ? g.states + ((long long)(b * g.H + h) * chunks) * g.d + c : nullptr;
    auto store = [&](long long t, float2 v) {
        T *o = out + t * g.out.stride_n;
        if (g.aligned) {
            if (on0) store_pair(o, v);
        } else {
            if (on0) store_one(o, v.x);
            if (on1) store_one(o + 1, v.y);
        }
    };
    auto save = [&](long long chunk, float2 v) {
        if (on0) states[chunk * g.d] = v.x;
        if (on1) states[chunk * g.d + 1] = v.y;
    };

    bool lost = false;
    init_maps(maps, (int)cluster);
    start_late<kLate>(g, rank);
    for (int r = 0; r < rounds; ++r) {
        cp_async_wait<kStages - 2>();
        __syncthreads();  // round r has arrived for every thread, and round r - 1 is consumed
        fetch(r + kStages - 1);
        unsigned char *st = sm + (r % kStages) * 2 * Tl::bytes;
        const T *xc = own_column<T, kCb>(st);
        T *gc = own_column<T, kCb>(st + Tl::bytes);
        const long long t0 = r * round_tok + (long long)rank * Tl::tok + seg * kSeg;
        const int valid = (int)max(0ll, min((long long)kSeg, len - t0));
        if (!M::log && valid < kSeg) close_gates<T, kCb>(gc, valid);
        float2 a[kSeg], u[kPlain ? 1 : kSeg], sum = both(0.0f), end = both(0.0f);
#pragma unroll
        for (int k = 0; k < kSeg; ++k) {
            const float2 xv = load_pair(xc + k * kCb);
            const Gate o = gate_of<T, kMode>(load_pair(gc + k * kCb), bias, nrate2);
            const float2 fx = value_of<kMode>(o, xv);
            a[k] = o.a;
            sum = add2(sum, o.l);
            end = fma2(o.a, end, fx);
            if (!kPlain) u[k] = fx;
        }
        auto value = [&](int k) { return kPlain ? load_pair(xc + k * kCb) : u[kPlain ? 0 : k]; };
        const float4 own = make_map(segment_decay(sum), end);
        float2 hs = enter_segment<T, kCb, true>(own, carry, maps, r, rank, (int)cluster, wait_limit<kLate>(g), lost);
        if (states && t0 < g.N) save(t0 / kSeg, hs);
        if (g.aligned && valid == kSeg) {
            if (on0) {
                T *o = out + t0 * g.out.stride_n;
#pragma unroll
                for (int k = 0; k < kSeg; ++k, o += g.out.stride_n) {
                    hs = fma2(a[k], hs, value(k));
                    store_pair(o, hs);
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < kSeg; ++k) {
                hs = fma2(a[k], hs, value(k));
                if (t0 + k < g.N) store(t0 + k, k < valid ? hs : both(0.0f));
            }
        }
    }
    cp_async_wait<0>();

    // whole rounds behind the length
    for (long long t = rounds * round_tok + (long long)rank * Tl::tok + seg * kSeg; t < g.N; t += round_tok) {
        if (states) save(t / kSeg, carry);
        for (int k = 0; k < kSeg && t + k < g.N; ++k) store(t + k, make_float2(0.0f, 0.0f));
    }
    if (g.h_out && rank == 0 && seg == 0) {
        if (on0) g.h_out[bc] = carry.x;
        if (on1) g.h_out[bc + 1] = carry.y;
    }
    leave_cluster((int)cluster, lost);
}

template <typename T, int kCb>
int launch_mode(const Args &g, const LateArgs *late, const Cut &p, int mode, cudaStream_t s) {
    constexpr size_t sm = smem_bytes<T, kCb>();
    constexpr int nt = Threads<T>::n;
    if (late) {
        if constexpr (kCb == 16) {
            if (mode == kDtNone) return launch_cluster<glr_fwd_kernel<T, kCb, kDtNone, true>>(*late, p, nt, sm, s);
        }
        return SSD_ERR_UNSUPPORTED;
    }
    switch (mode) {
    case kDtNone: return launch_cluster<glr_fwd_kernel<T, kCb, kDtNone>>(g, p, nt, sm, s);
    case kDtDt: return launch_cluster<glr_fwd_kernel<T, kCb, kDtDt>>(g, p, nt, sm, s);
    case kDtComplement: return launch_cluster<glr_fwd_kernel<T, kCb, kDtComplement>>(g, p, nt, sm, s);
    case kLogNone: return launch_cluster<glr_fwd_kernel<T, kCb, kLogNone>>(g, p, nt, sm, s);
    default: return launch_cluster<glr_fwd_kernel<T, kCb, kLogComplement>>(g, p, nt, sm, s);
    }
}

template <typename T>
int launch_cb(const Args &g, const LateArgs *late, const Cut &p, int mode, cudaStream_t s) {
    return p.cb == 64 ? launch_mode<T, 64>(g, late, p, mode, s)
                      : p.cb == 32 ? launch_mode<T, 32>(g, late, p, mode, s) : launch_mode<T, 16>(g, late, p, mode, s);
}

}  // namespace

int launch_fwd(const Args &g, const LateArgs *late, const Cut &p, int dtype, int mode, cudaStream_t s) {
    return dtype == SSD_F32 ? launch_cb<float>(g, late, p, mode, s) : launch_cb<__nv_bfloat16>(g, late, p, mode, s);
}

}  // namespace glr
}  // namespace ssd
