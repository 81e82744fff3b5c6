// Strided activations of the recurrence and the norms: host-side checks, and the
// walk over a batch's tokens.
#pragma once

#include <stdint.h>

#include "ssd.h"

namespace ssd {

inline bool misaligned(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

// Sizes for which every offset fits 64 bits, every index of a token or channel
// 32 (rounded up to a tile too; the gated norm's steps are larger, see next_token)
// and every grid its limits.
inline bool sizes_ok(long long B, long long H, long long N, long long d) {
    constexpr long long most = (1ll << 31) - 65536;
    return B >= 1 && H >= 1 && N >= 1 && d >= 1 && B * H < most && H * d < most && N < most &&
           B * H * N < (1ll << 40) / d;
}

// Checks a view of [B, H, N, d].  An output's elements must be distinct: with
// the dimensions longer than one sorted by stride, each stride is at least the
// extent of all that lie inside it.
inline int check_view(const ssd_view *v, int B, int H, int N, int d, size_t esize, bool output) {
    if (!v || !v->ptr) return SSD_ERR_NULL;
    if (v->stride_b < 0 || v->stride_h < 0 || v->stride_n < 0) return SSD_ERR_SHAPE;
    if (misaligned(v->ptr, esize)) return SSD_ERR_ALIGN;
    if (output) {
        long long st[3], n[3];
        int k = 0;
        const long long all_st[3] = {v->stride_b, v->stride_h, v->stride_n}, all_n[3] = {B, H, N};
        for (int i = 0; i < 3; ++i)
            if (all_n[i] > 1) {
                int j = k++;
                for (; j > 0 && st[j - 1] > all_st[i]; --j) {
                    st[j] = st[j - 1];
                    n[j] = n[j - 1];
                }
                st[j] = all_st[i];
                n[j] = all_n[i];
            }
        long long extent = d;
        for (int i = 0; i < k; ++i) {
            if (st[i] < extent) return SSD_ERR_SHAPE;
            extent += (n[i] - 1) * st[i];
        }
    }
    return SSD_OK;
}

inline int check_rows(const ssd_rows *v, int M, int C, size_t esize, bool output) {
    if (!v || !v->ptr) return SSD_ERR_NULL;
    if (v->stride < 0 || (output && M > 1 && v->stride < C)) return SSD_ERR_SHAPE;
    return misaligned(v->ptr, esize) ? SSD_ERR_ALIGN : SSD_OK;
}

// Moves token n of a batch of N on by step tokens (n, step < N); true where that
// passes the batch's end, and n is then a token of the next one.  Unsigned, since
// n + step may pass 2^31 (a step is up to a tenth of all tokens), never 2^32.
#ifdef __CUDACC__
__host__ __device__
#endif
inline bool next_token(unsigned &n, unsigned step, unsigned N) {
    n += step;
    const bool passes = n >= N;
    if (passes) n -= N;
    return passes;
}

inline size_t elem_size(int dtype) { return dtype == SSD_F32 ? 4 : 2; }

}  // namespace ssd
