// ssm_device.h -- what the selective scan's kernels share (gfx950).
#pragma once

#include "rows_device.h"
#include "ssm_internal.h"

namespace ssm {

using namespace rows;

// A long sequence is cut into segments that are scanned at once: a first launch finds what each
// segment leaves of a zero state (L_j) and the sum of its steps (D_j, 64 bits, rounded once), and
// a segment's entering state is the fold h <- e^(D_j A) h + L_j over those before it; the
// backward's entering gradient the same over those behind it.  `slot`: of the first one folded, `step`: 1 or -1.
template <int NS>
__device__ __forceinline__ void fold_segments(const Args& p, int slot, int step, int count, int ch, int n0,
                                              const float (&A2)[NS], float (&h)[NS]) {
#pragma unroll 4
    for (int j = 0; j < count; ++j, slot += step) {
        const float d = p.sum_d[(int64_t)slot * p.C + ch];
        const float* l = p.sum_h + ((int64_t)slot * p.C + ch) * p.S + n0;
#pragma unroll
        for (int s = 0; s < NS; ++s) h[s] = fmaf(exp2_f(d * A2[s]), h[s], l[s]);
    }
}

// How the 16 tokens by CH channels of a block, and its b and c, are dealt to NT threads for
// loading: thread tid has channel tid % CH and every STEP-th token from tid / CH on, LT of them,
// and HB values each of b and c.  Rows are addressed from one pointer per wave (the block's
// first token, STEP tokens apart) and one offset per lane and tensor.
template <typename InT, int CH, int NT, int S>
struct Deal {
    static constexpr int TB = kBlock, STEP = NT / CH, LT = TB / STEP, HB = TB * S / NT;
    static_assert(LT * STEP == TB && HB * NT == TB * S, "a block is dealt out evenly");
    int lc, lt, lch;
    bool lon;
    __device__ __forceinline__ Deal(int tid, int cb, int C) : lc(tid % CH), lt(tid / CH) {
        lon = cb * CH + lc < C;
        lch = lon ? cb * CH + lc : C - 1;      // whole blocks are loaded without a condition: an address that exists
    }
    __device__ __forceinline__ uint32_t off(int64_t ld) const { return (uint32_t)(lt * (int)ld + lch) * (uint32_t)sizeof(InT); }
    static __device__ __forceinline__ uint32_t off_b(int tid, int64_t ld) {
        return (uint32_t)(tid / S * (int)ld + tid % S) * (uint32_t)sizeof(InT);
    }
    // rows of this thread's channel from token t0 of a sequence on, `end` the first one that is not read
    __device__ __forceinline__ void rows(const InT* base, int64_t ld, uint32_t off, int t0, int end, bool full,
                                         InT (&r)[LT]) const {
        const InT* p = base + t0 * ld;
#pragma unroll
        for (int i = 0; i < LT; ++i, p += STEP * ld)
            r[i] = full || (lon && t0 + lt + i * STEP < end) ? ldo<InT>(p, off) : InT(0);
    }
    static __device__ __forceinline__ void mat(const InT* base, int64_t ld, uint32_t off, int tid, int t0, int end, bool full,
                                               InT (&r)[HB]) {
        const InT* p = base + t0 * ld;
#pragma unroll
        for (int i = 0; i < HB; ++i, p += (NT / S) * ld)
            r[i] = full || t0 + (tid + i * NT) / S < end ? ldo<InT>(p, off) : InT(0);
    }
};

}  // namespace ssm
