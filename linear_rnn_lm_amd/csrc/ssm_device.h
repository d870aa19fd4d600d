// ssm_device.h -- what the selective scan's kernels share (gfx950).
#pragma once

#include "rows_device.h"
#include "ssm_internal.h"

namespace ssm {

using namespace rows;

// A long sequence is cut into segments that are scanned at once: a first launch finds what each
// segment leaves of a zero state (L_j) and the sum of its steps (D_j, of sums of up to four in 64 bits, rounded once), and
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

// What the k-th workgroup of a channel block works on; false: nothing.  Packed sequences go by length,
// the longest first, so that none starts when the others are nearly done (17 sequences, 8193 tokens,
// 2048 channels of 64 states: 300 us in their order, 256 by length).
__device__ __forceinline__ bool segment_of(const Args& p, const Seqs& seqs, int k, int& n, int& piece) {
    return p.cu && p.N > 1 && p.N <= 64 ? by_length(seqs, k, p.seg, n, piece) : slot_piece(seqs, k, p.seg, n, piece);
}

// Where a segment ends: its start and length together may pass 2^31, where the sequence does not end.
__device__ __forceinline__ int segment_end(int t_begin, int seg, int len) {
    return (int)min((uint32_t)t_begin + (uint32_t)seg, (uint32_t)len);
}

// Token rows through buffer resources, so that a ragged end needs no branch: loads behind a
// sequence's (segment's) end return 0 and stores there are dropped; lanes whose channel does not
// exist have kNowhere for an offset.
constexpr uint32_t kNowhere = 0x80000000u;     // beyond any resource
template <typename T>
__device__ __forceinline__ T bload(wkv7::Rsrc r, uint32_t off) {
    if constexpr (sizeof(T) == 2) return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
    else return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}
__device__ __forceinline__ void bstore(uint16_t, wkv7::Rsrc r, uint32_t off, float v) {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v), r, off, 0, 0);
}
__device__ __forceinline__ void bstore(float, wkv7::Rsrc r, uint32_t off, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, off, 0, 0);
}

// A walk over rows of `width` bytes, `row` bytes apart, block by block.
struct Stream {
    const char* p;
    uint32_t row, width;
    // the resource of the present block's first `rows` rows (0: none)
    __device__ __forceinline__ wkv7::Rsrc rsrc(int rows) const {
        return wkv7::make_rsrc(p, rows > 0 ? (uint32_t)(rows - 1) * row + width : 0u);
    }
    __device__ __forceinline__ void next() { p += kBlock * row; }
    __device__ __forceinline__ void back() { p -= kBlock * row; }
};
// From row t0 on; no rows at all without a base.
template <typename T>
__device__ __forceinline__ Stream stream(const T* base, int64_t ld, int width, int t0) {
    return {reinterpret_cast<const char*>(base + t0 * ld), (uint32_t)ld * (uint32_t)sizeof(T), (uint32_t)width * (uint32_t)sizeof(T)};
}
// Rows of the block at t0 that exist, below `end`.
__device__ __forceinline__ int block_rows(int t0, int end) { return max(0, min(kBlock, end - t0)); }

// LDS matrices hold a block's 16 tokens side by side, a channel or a state to a row of kPitch
// floats: four tokens to an access, and 16 rows' accesses spread over all banks.
constexpr int kPitch = 20;

// How the 16 tokens by CH channels of a block, and its b and c, are dealt to NT threads for
// loading: thread tid has channel tid % CH and the LT tokens from LT (tid / CH) on, and MB of the
// 2 x 16 x S values of b and c.
template <typename InT, int CH, int NT, int S>
struct Deal {
    static constexpr int TB = kBlock, LT = TB * CH / NT, MB = 2 * TB * S / NT;
    static_assert(LT * NT == TB * CH && MB * NT == 2 * TB * S, "a block is dealt out evenly");
    int lc, lt, lch;
    bool lon;
    __device__ __forceinline__ Deal(int tid, int cb, int C) : lc(tid % CH), lt(tid / CH * LT) {
        lon = cb * CH + lc < C;
        lch = lon ? cb * CH + lc : C - 1;
    }
    // offset of this thread's i-th value of a block's rows
    __device__ __forceinline__ uint32_t off(int64_t ld) const {
        return lon ? (uint32_t)(lt * (int)ld + lch) * (uint32_t)sizeof(InT) : kNowhere;
    }
    static __device__ __forceinline__ uint32_t row(int64_t ld, int i) { return (uint32_t)(i * (int)ld) * (uint32_t)sizeof(InT); }
    __device__ __forceinline__ void rows(const Stream& s, int n, int64_t ld, uint32_t off, InT (&v)[LT]) const {
        const wkv7::Rsrc r = s.rsrc(n);
#pragma unroll
        for (int i = 0; i < LT; ++i) v[i] = bload<InT>(r, off + row(ld, i));
    }
};
// b's and c's: value tid + i NT of b's 16 x S, then c's.  A wave's values are all of one of them.
template <typename InT, int NT, int S>
struct Mats {
    static constexpr int TB = kBlock, MB = 2 * TB * S / NT, H = MB > 1 ? MB / 2 : 1;
    Stream b, c;             // MB 1: b alone, which is c for the upper half of the threads
    uint32_t ob, oc;
    int at;                  // where the first value lies in an LDS matrix
    __device__ __forceinline__ Mats(const InT* bp, int64_t b_ld, const InT* cp, int64_t c_ld, int tid, int t0) {
        if constexpr (MB == 1) {
            const bool upper = uniform(tid >= TB * S);
            tid %= TB * S;
            b = c = stream(upper ? cp : bp, upper ? c_ld : b_ld, S, t0);
            b_ld = upper ? c_ld : b_ld;
            at = upper ? S * kPitch : 0;
        } else {
            b = stream(bp, b_ld, S, t0);
            c = stream(cp, c_ld, S, t0);
            at = 0;
        }
        ob = (uint32_t)(tid / S * (int)b_ld + tid % S) * (uint32_t)sizeof(InT);
        oc = (uint32_t)(tid / S * (int)c_ld + tid % S) * (uint32_t)sizeof(InT);
        at += tid % S * kPitch + tid / S;
    }
    __device__ __forceinline__ void load(int n, int64_t b_ld, int64_t c_ld, InT (&r)[MB]) const {
        const wkv7::Rsrc rb = b.rsrc(n), rc = c.rsrc(n);
#pragma unroll
        for (int i = 0; i < H; ++i) {
            r[i] = bload<InT>(rb, ob + (uint32_t)(i * (NT / S) * (int)b_ld) * (uint32_t)sizeof(InT));
            if constexpr (MB > 1) r[H + i] = bload<InT>(rc, oc + (uint32_t)(i * (NT / S) * (int)c_ld) * (uint32_t)sizeof(InT));
        }
    }
    // into s_bc: (2, S, kPitch)
    __device__ __forceinline__ void put(float* s_bc, const InT (&r)[MB]) const {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            s_bc[at + i * (NT / S)] = widen(r[i]);
            if constexpr (MB > 1) s_bc[S * kPitch + at + i * (NT / S)] = widen(r[H + i]);
        }
    }
    __device__ __forceinline__ void next() {
        b.next();
        c.next();
    }
    __device__ __forceinline__ void back() {
        b.back();
        c.back();
    }
};

// LT neighbouring floats of LDS.
template <int LT>
__device__ __forceinline__ void put_lds(float* p, const float (&v)[LT]) {
    if constexpr (LT == 4) *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
    else if constexpr (LT == 2) *reinterpret_cast<float2*>(p) = make_float2(v[0], v[1]);
    else *p = v[0];
}
template <int LT>
__device__ __forceinline__ void get_lds(const float* p, float (&v)[LT]) {
    if constexpr (LT == 4) {
        const f32x4 x = *reinterpret_cast<const f32x4*>(p);
        v[0] = x[0], v[1] = x[1], v[2] = x[2], v[3] = x[3];
    } else if constexpr (LT == 2) {
        const float2 x = *reinterpret_cast<const float2*>(p);
        v[0] = x.x, v[1] = x.y;
    } else {
        v[0] = *p;
    }
}
// softplus(v), or v, and its slope.  Both are formed: a branch here would keep the scan's instructions from
// being mixed with these.
__device__ __forceinline__ float step_of(bool soft, float v, float& slope) {
    float sl, sp = softplus(v, sl);
    asm volatile("" : "+v"(sp));
    slope = soft ? sl : 1.f;
    return soft ? sp : v;
}
__device__ __forceinline__ float step_of(bool soft, float v) {
    float slope;
    return step_of(soft, v, slope);
}
__device__ __forceinline__ f32x4 lds4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }

}  // namespace ssm
