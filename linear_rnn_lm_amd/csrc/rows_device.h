// rows_device.h -- device-side building blocks of the selective scan, the short
// convolution and the block norm (gfx950): token values, activations, lane sums, and where
// the sequences of a call lie.
#pragma once

#include <float.h>

#include "wkv7_device.h"

namespace rows {

using wkv7::f32x4;
using wkv7::lds_barrier;

// One value of a token tensor.  widen() is apart from the load, so that a load ahead of its
// use does not wait where it is issued.
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
template <typename T>
__device__ __forceinline__ float ld(const T* p) { return widen(*p); }
__device__ __forceinline__ void st(float* p, float v) { *p = v; }
__device__ __forceinline__ void st(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_f(float x) { return __builtin_amdgcn_exp2f(x); }
// e^-v is 2^t, t = -log2(e) v rounded, times e^r, r = -v - t ln 2 what the rounding took (and log2(e)'s own; one
// fma, exact up to |v| E / 20, E = 2^-24).  Without it the relative error is |v| E; with it 1 + r, for r < 2^-16 where
// 2^t is neither 0 nor infinity, leaves 3 E of the exponential's last place and these roundings.  Beyond, where r is large or no
// number, the clamp keeps 0 and infinity as they are; a NaN comes through 2^t.
__device__ __forceinline__ float exp_rest(float minus_v, float t) { return fmaf(t, -kLn2, minus_v); }

// 1 / (1 + e^-v), good to 8 E: e^-v may overflow to infinity, its reciprocal is then 0, as it should be.
__device__ __forceinline__ float sigmoid(float v) {
    const float t = -kLog2e * v, m = __builtin_amdgcn_fmed3f(1.f + exp_rest(-v, t), 0.5f, 2.f);
    return __builtin_amdgcn_rcpf(fmaf(exp2_f(t), m, 1.f));
}
// The same for an output of type T, or its gradient, which it scales.  One that is rounded to bf16 (half a step: 2^-8)
// goes without the correction: |v| E, below 2^-17 wherever the result is not 0, and in the terms of sums that stay in fp32 less
// than 6 E of a gate's size, |v| e^-|v| being below 0.4 (convolution of 12289 packed tokens of 2048 channels 24.5 us, with it
// 25.2; training B4 T4096 C4096 1406, with it and the step's slope by itself 1420).
template <typename T>
__device__ __forceinline__ float sigmoid_for(float v) {
    if constexpr (sizeof(T) == 2) return __builtin_amdgcn_rcpf(1.f + exp2_f(-kLog2e * v));
    else return sigmoid(v);
}
// max(v, 0) + log(1 + e), e = e^-|v|, good to 8 E.  With w = 1 + e rounded and r = e - (w - 1) what the rounding
// took, log(1 + e) = log(w) + r / w up to r^2; r is at most half a last place of w, so r in place of r / w costs
// at most E of the result.  For e below half a last place of 1 that leaves e itself.
// `slope`: 1 / (1 + e^-v), from the same e, where it is used.
__device__ __forceinline__ float softplus(float v, float& slope) {
    const float a = __builtin_fabsf(v), t = -kLog2e * a, e0 = exp2_f(t);
    const float e = fmaf(e0, __builtin_amdgcn_fmed3f(exp_rest(-a, t), -1.f, 1.f), e0), w = 1.f + e, r = e - (w - 1.f);
    slope = (v > 0.f ? 1.f : e) * __builtin_amdgcn_rcpf(w);
    return __builtin_fmaxf(v, 0.f) + fmaf(kLn2, __builtin_amdgcn_logf(w), r);
}
__device__ __forceinline__ float softplus(float v) {
    float slope;
    return softplus(v, slope);
}

// log2(e) A, the lowest number in place of -infinity: a step of 0 (of a token behind the end of a sequence too) times it is
// 0, so that it passes the state on, and any other step clears the state.
__device__ __forceinline__ float rate_of(float A) {
    const float a = kLog2e * A;
    return a < -FLT_MAX ? -FLT_MAX : a;                    // a NaN stays
}

// A value that is the same for the whole wave, in scalar registers.
__device__ __forceinline__ int64_t uniform(int64_t x) {
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)x), hi = __builtin_amdgcn_readfirstlane((uint32_t)(x >> 32));
    return (int64_t)((uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, false));
}

// Sums over the four lanes l, l + 16, l + 32, l + 48 of four values: lane (g, r), g = l / 16,
// gets the sum of value row_of(g).  A swap and an add sum two values at once, each half of the
// lanes keeping one.
__device__ __forceinline__ int row_of(int g) { return ((g & 1) << 1) | (g >> 1); }
__device__ __forceinline__ float rows_sum4(float y0, float y1, float y2, float y3) {
    auto pair32 = [](float a, float b) {
        const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
        return __uint_as_float(h[0]) + __uint_as_float(h[1]);
    };
    const float p = pair32(y0, y1), q = pair32(y2, y3);
    const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(p), __float_as_uint(q), false, false);
    return __uint_as_float(h[0]) + __uint_as_float(h[1]);
}

// Where the sequences lie, and how they are cut into pieces of `len` tokens.  Dense: sequence
// n is row n of (B, T), its pieces are slots n per + i.  Packed: sequence n is the tokens cu[n] ..
// cu[n + 1] - 1, its piece i is slot cu[n] / len + n + i: strictly increasing over
// sequences and pieces, at most T / len + N - 1, so no table is needed.  The offsets come from
// device memory: they are clamped to 0 .. T and to non-decreasing pairs, so that no value of
// theirs leads outside the tensors.
struct Seqs {
    const int* cu;   // NULL: dense
    int N, T;
};

__device__ __forceinline__ void seq_span(const Seqs& s, int n, int64_t& tok0, int& len) {
    if (s.cu) {
        const int a = min(max(s.cu[n], 0), s.T), b = min(max(s.cu[n + 1], a), s.T);
        tok0 = a;
        len = b - a;
    } else {
        tok0 = (int64_t)n * s.T;
        len = s.T;
    }
}
__device__ __forceinline__ int pieces_dense(int T, int len) { return (T - 1) / len + 1; }
__device__ __forceinline__ int first_slot(const Seqs& s, int n, int64_t tok0, int len) {
    return s.cu ? (int)tok0 / len + n : n * pieces_dense(s.T, len);
}

// The piece of a slot: its sequence n and its index i there; false if the slot is no
// sequence's.  The first piece of an empty sequence exists.
__device__ __forceinline__ bool slot_piece(const Seqs& s, int slot, int len, int& n, int& i) {
    if (!s.cu) {
        const int per = pieces_dense(s.T, len);
        n = slot / per;
        i = slot % per;
        return true;
    }
    // the last sequence whose first slot is at or before this one
    int lo = 0, hi = s.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (min(max(s.cu[mid], 0), s.T) / len + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    int64_t t0;
    int L;
    seq_span(s, lo, t0, L);
    n = lo;
    i = slot - first_slot(s, lo, t0, len);
    return i == 0 || (i > 0 && (int64_t)i * len < L);
}

// Zeroes the rows of a token tensor that no packed sequence covers; by `count` threads, this one is number i.
template <typename U>
__device__ __forceinline__ void zero_span(void* base, int64_t from, int64_t to, int64_t i, int64_t count) {
    U* p = static_cast<U*>(base);
    for (int64_t u = from / sizeof(U) + i; u < to / (int64_t)sizeof(U); u += count) p[u] = U{};
}
constexpr int kZeroBlocks = 128;   // workgroups of 256 that do so, behind those of a launch
__device__ __forceinline__ void zero_outside(const Seqs& s, void* base, int64_t row_bytes, int64_t i) {
    const int a = min(max(s.cu[0], 0), s.T), b = min(max(s.cu[s.N], a), s.T);
    constexpr int64_t count = kZeroBlocks * 256;
    const int64_t any = reinterpret_cast<intptr_t>(base) | row_bytes;
    const int64_t from[2] = {0, b * row_bytes}, to[2] = {a * row_bytes, s.T * row_bytes};
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        if (any % 16 == 0) zero_span<uint4>(base, from[k], to[k], i, count);
        else if (any % 4 == 0) zero_span<uint32_t>(base, from[k], to[k], i, count);
        else zero_span<uint16_t>(base, from[k], to[k], i, count);
    }
}

// Piece k of N <= 64 packed sequences, counted from the longest sequence to the shortest: a sequence to a
// lane, each adds up the pieces before its own.  False if there are fewer.
__device__ __forceinline__ bool by_length(const Seqs& s, int k, int piece_len, int& n, int& i) {
    const int lane = threadIdx.x & 63;
    int64_t tok0;
    int len = -1;
    if (lane < s.N) seq_span(s, lane, tok0, len);
    const int mine = lane < s.N ? max(1, pieces_dense(len, piece_len)) : 0;
    int before = 0;
    for (int j = 0; j < s.N; ++j) {
        const int l = __builtin_amdgcn_readlane(len, j), c = __builtin_amdgcn_readlane(mine, j);
        before += l > len || (l == len && j < lane) ? c : 0;
    }
    n = __ffsll(__ballot(before <= k && k < before + mine)) - 1;
    if (n < 0) {
        n = i = 0;
        return false;
    }
    i = k - __builtin_amdgcn_readlane(before, n);
    return true;
}

}  // namespace rows
