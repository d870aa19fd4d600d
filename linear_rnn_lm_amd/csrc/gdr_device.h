// gdr_device.h -- device-side building blocks of the gated delta rule (gfx950).
//
// Per value head with state S (V x K, rows i paired with v and o, columns j
// paired with q and k), token t with log decay g_t and write strength b_t:
//     S <- e^g S;   u = b (v - S k);   S <- S + u k^T;   o = scale S q.
//
// Chunked form, 64 tokens to a chunk.  With G_t the sum of the chunk's log
// decays up to t, Lam[t][s] = e^(G_t - G_s) for s <= t, S0 the state entering:
//     A = strict_lower(b_t Lam K K^T),   T = (I + A)^-1,   M = lower(Lam Q K^T)
//     R = V - e^G K S0^T,                U = T (b R)
//     O = scale (e^G Q S0^T + M U),      S1 = e^(G_C) S0 + U^T (e^(G_C - G) K)
// Every factor is a ratio of a later to an earlier decay, at most 1, so no
// decay is too small; the sums G are held in 64 bits, because the differences
// of two of them are small next to the sums themselves.
//
// Matrix products run on v_mfma_f32_16x16x32_bf16.  An fp32 value x is held as
// up to three bf16 planes, x = p0 + p1 + p2 (each the rounding of what is left;
// three hold 24 bits), and a product of X and Y sums the plane products p_i q_j
// with i + j < ORD.  bf16 inputs are exact in one plane, so a product of
// an input and a state costs three instructions, not six.
//
// Index order.  A 64-long index is dealt to 16-wide tiles as
//     idx(tile, m) = 32 (tile / 2) + 8 (m / 4) + 4 (tile % 2) + m % 4.
// An accumulator tile holds rows m = 4g + q (lane (g, r), register q), so lane g of
// the tile pair (2c, 2c + 1) holds the eight consecutive indices 32c + 8g ..
// + 7: exactly the eight contraction indices that lane g feeds to a 32-deep
// product.  A result is therefore the next product's operand without leaving
// its registers, and the other operand is read from row-major memory in
// 16-byte pieces (rows) or by the LDS transpose (columns).
//
// LDS matrices are row-major bf16 planes of U 16-byte units per row; unit u of
// row t lies in slot u ^ swz(t), which spreads both kinds of reads over the banks.
#pragma once

#include "wkv7_device.h"

namespace gdr {

using wkv7::bf16x2;
using wkv7::bf16x4;
using wkv7::bf16x8;
using wkv7::f32x4;
using wkv7::lds_barrier;
using wkv7::zero4;

constexpr int C = 64;  // chunk length

// Gates of one chunk of one head, written by the prepare kernel: e^G, e^(G_C -
// G), b (the last two 0 for tokens past the sequence's end), then G log2(e) as a
// whole number n and a rest f in +-1/2, so that e^(G_t - G_s) = 2^(n_t - n_s)
// 2^(f_t - f_s) is good to fp32 however large the sums are.
constexpr int kGateFloats = 320;
constexpr int kGateEG = 0, kGateToEnd = 64, kGateBeta = 128, kGateN = 192, kGateF = 256;

// A write strength of 0 is taken as 2^-60: the token's u then holds b times
// the error v - S k it would have written, which no fp32 sum notices, and the
// gradient of b, (dL/du . u) / b, needs no case of its own.
constexpr float kBetaMin = 8.673617379884035e-19f;

// A log decay below -200 counts as -200: e^-200 is 0 in fp32, and -inf would
// make differences of sums undefined.
constexpr float kMinLogDecay = -200.f;

__device__ __forceinline__ int idx(int tile, int m) {
    return 32 * (tile >> 1) + 8 * (m >> 2) + 4 * (tile & 1) + (m & 3);
}

template <int NP>
struct PF {
    bf16x8 p[NP];
};

// Two fp32 values to NP bf16 planes.
template <int NP>
__device__ __forceinline__ void planes2(wkv7::f32x2 v, bf16x2 (&o)[NP]) {
#pragma unroll
    for (int i = 0; i < NP; ++i) {
        o[i] = __builtin_convertvector(v, bf16x2);
        if (i + 1 < NP) v = v - __builtin_convertvector(o[i], wkv7::f32x2);
    }
}

// Fragment of an accumulator tile pair (see the index order above).
template <int NP>
__device__ __forceinline__ PF<NP> pf_acc(f32x4 a0, f32x4 a1) {
    bf16x2 x[4][NP];
    planes2<NP>(wkv7::f32x2{a0[0], a0[1]}, x[0]);
    planes2<NP>(wkv7::f32x2{a0[2], a0[3]}, x[1]);
    planes2<NP>(wkv7::f32x2{a1[0], a1[1]}, x[2]);
    planes2<NP>(wkv7::f32x2{a1[2], a1[3]}, x[3]);
    PF<NP> f;
#pragma unroll
    for (int i = 0; i < NP; ++i)
        f.p[i] = bf16x8{x[0][i][0], x[0][i][1], x[1][i][0], x[1][i][1], x[2][i][0], x[2][i][1], x[3][i][0], x[3][i][1]};
    return f;
}

// acc += X Y^T over one 32-deep step: plane products with i + j < ORD, the
// smaller ones first.
template <int ORD, int NX, int NY>
__device__ __forceinline__ f32x4 pmma(f32x4 acc, const PF<NX>& x, const PF<NY>& y) {
#pragma unroll
    for (int s = ORD - 1; s >= 0; --s)
#pragma unroll
        for (int i = 0; i < NX; ++i)
            if (s - i >= 0 && s - i < NY) acc = wkv7::mfma_bf16(x.p[i], y.p[s - i], acc);
    return acc;
}

// Slot permutation of a row with U units (8 or 16).
template <int U>
__device__ __forceinline__ int swz(int row) {
    return ((row & 3) | ((row >> 1) & 12)) & (U - 1);
}

// Rows: lane (g, r) gets X[row][32 ks + 8g .. + 7], `row` its own choice.
template <int U, int NP>
__device__ __forceinline__ PF<NP> frag_row(const char* X, int plane, int row, int ks, int lane) {
    const char* p = X + (row * U + ((4 * ks + (lane >> 4)) ^ swz<U>(row))) * 16;
    PF<NP> f;
#pragma unroll
    for (int i = 0; i < NP; ++i) f.p[i] = *reinterpret_cast<const bf16x8*>(p + i * plane);
    return f;
}

// Columns: lane (g, r) gets X[32 ks + 8g + e][idx(tile, r)], e = 0..7, with the
// LDS transpose read: within each group of 16 lanes, lane 4i + e receives
// element e of the 8-byte reads of lanes i, i + 4, i + 8, i + 12.
template <int U, int NP>
__device__ __forceinline__ PF<NP> frag_col(const char* X, int plane, int tile, int ks, int lane) {
    const int row = 32 * ks + 8 * (lane >> 4) + ((lane & 15) >> 2);
    const int unit = 4 * (tile >> 1) + (lane & 3), half = 8 * (tile & 1);
    const char* p0 = X + (row * U + (unit ^ swz<U>(row))) * 16 + half;
    const char* p1 = X + ((row + 4) * U + (unit ^ swz<U>(row + 4))) * 16 + half;
    PF<NP> f;
#pragma unroll
    for (int i = 0; i < NP; ++i)
        f.p[i] = wkv7::cat8(
            wkv7::as_bf16x4(__builtin_amdgcn_ds_read_tr16_b64_v4i16((wkv7::lds_i16x4*)(p0 + i * plane))),
            wkv7::as_bf16x4(__builtin_amdgcn_ds_read_tr16_b64_v4i16((wkv7::lds_i16x4*)(p1 + i * plane))));
    return f;
}

// T and M are lower triangular: only their three lower 32 x 32 blocks exist, in
// the order (0, 0), (1, 0), (1, 1), each with rows of four units, unit u of row t
// in slot u ^ (t / 8).  Rows and columns as above (ks <= tile / 2, ks >= tile / 2).
constexpr int kTriBytes = 3 * 32 * 64;   // one plane
__device__ __forceinline__ int tri_block(int br, int bc) { return (br + bc) * 2048; }
template <int NP>
__device__ __forceinline__ PF<NP> tri_row(const char* X, int tile, int ks, int lane) {
    const int row = idx(tile & 1, lane & 15);
    const char* p = X + tri_block(tile >> 1, ks) + (row * 4 + ((lane >> 4) ^ (row >> 3))) * 16;
    PF<NP> f;
#pragma unroll
    for (int i = 0; i < NP; ++i) f.p[i] = *reinterpret_cast<const bf16x8*>(p + i * kTriBytes);
    return f;
}
template <int NP>
__device__ __forceinline__ PF<NP> tri_col(const char* X, int tile, int ks, int lane) {
    const int row = 8 * (lane >> 4) + ((lane & 15) >> 2);
    const char* p = X + tri_block(ks, tile >> 1) + (row * 4 + ((lane & 3) ^ (lane >> 4))) * 16 + 8 * (tile & 1);
    PF<NP> f;
#pragma unroll
    for (int i = 0; i < NP; ++i)
        f.p[i] = wkv7::cat8(
            wkv7::as_bf16x4(__builtin_amdgcn_ds_read_tr16_b64_v4i16((wkv7::lds_i16x4*)(p + i * kTriBytes))),
            wkv7::as_bf16x4(__builtin_amdgcn_ds_read_tr16_b64_v4i16((wkv7::lds_i16x4*)(p + 256 + i * kTriBytes))));
    return f;
}

// Eight consecutive values of a row into the planes of an LDS matrix.
template <int U, int NP>
__device__ __forceinline__ void put8(char* X, int plane, int row, int unit, const PF<NP>& f) {
    char* p = X + (row * U + (unit ^ swz<U>(row))) * 16;
#pragma unroll
    for (int i = 0; i < NP; ++i) *reinterpret_cast<bf16x8*>(p + i * plane) = f.p[i];
}

// One value of a token tensor.  widen() is apart from the load, so that a load
// ahead of its use does not wait where it is issued.
__device__ __forceinline__ float widen(float x) { return x; }
__device__ __forceinline__ float widen(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
template <typename T>
__device__ __forceinline__ float ld(const T* p) { return widen(*p); }
__device__ __forceinline__ void st(float* p, float v) { *p = v; }
__device__ __forceinline__ void st(uint16_t* p, float v) { *p = __builtin_bit_cast(uint16_t, (__bf16)v); }

// e^x for a 64-bit x, good to fp32: the whole part of x log2(e) is taken off in 64 bits.
__device__ __forceinline__ float exp_d(double x) {
    const double y = x * 1.4426950408889634074;
    const double n = __builtin_rint(y);
    return __builtin_ldexpf(__builtin_amdgcn_exp2f((float)(y - n)), (int)n);
}
// e^(G_t - G_s) from two tokens' whole and remaining parts.  The parts' differences are
// exact to 2^-25; their sum y is rounded by 2^-24 |y|, which 2^y has where it is small.
__device__ __forceinline__ float decay(float nt, float ft, float ns, float fs) {
    return __builtin_amdgcn_exp2f((nt - ns) + (ft - fs));
}

// Where the sequences lie.  Dense: sequence n is row n of (B, T), its chunks
// are slots n NC .. .  Packed: cu[n] .. cu[n + 1] are the tokens of sequence n,
// chunk c of it is slot cu[n] / 64 + n + c: strictly increasing over sequences
// and chunks, at most T / 64 + N - 1, so no table is needed.  The offsets come
// from device memory: they are clamped to 0 .. T and to non-decreasing
// pairs, so that no value of theirs leads outside the tensors.
struct Seqs {
    const int* cu;   // NULL: dense
    int N, T, NC;    // sequences; tokens per row; chunk slots per row (dense) or in all (packed)
};

__device__ __forceinline__ void seq_span(const Seqs& s, int n, int64_t& tok0, int& len, int& slot0) {
    if (s.cu) {
        const int a = min(max(s.cu[n], 0), s.T), b = min(max(s.cu[n + 1], a), s.T);
        tok0 = a;
        len = b - a;
        slot0 = a / C + n;
    } else {
        tok0 = (int64_t)n * s.T;
        len = s.T;
        slot0 = n * s.NC;
    }
}

// The chunk of a slot: its first token and how many of its tokens exist;
// false if the slot belongs to no sequence.
__device__ __forceinline__ bool slot_chunk(const Seqs& s, int slot, int& n, int64_t& tok, int& len) {
    if (!s.cu) {
        n = slot / s.NC;
        const int c = slot % s.NC;
        tok = (int64_t)n * s.T + c * C;
        len = min(C, s.T - c * C);
        return true;
    }
    // the last sequence whose first slot is at or before this one
    int lo = 0, hi = s.N - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (min(max(s.cu[mid], 0), s.T) / C + mid <= slot) lo = mid;
        else hi = mid - 1;
    }
    int64_t t0;
    int l, s0;
    seq_span(s, lo, t0, l, s0);
    const int c = slot - s0;
    n = lo;
    if (c < 0 || c * C >= l) return false;
    tok = t0 + c * C;
    len = min(C, l - c * C);
    return true;
}

// One wave copies 1 KiB of LDS (64 units, lane l the l-th) from per-lane addresses.
__device__ __forceinline__ void dma16(const void* src, char* lds) {
    __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                     (__attribute__((address_space(3))) void*)lds, 16, 0, 0);
}

}  // namespace gdr
