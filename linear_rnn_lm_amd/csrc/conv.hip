// conv.hip -- the short causal convolution, forward, backward and step (gfx950).
//
// Bound by HBM: a thread holds VEC neighbouring channels (16 bytes) and their filters in
// registers and walks a run of tokens with the last W - 1 inputs in a window, so x is read
// once (and W - 1 tokens again per run), four tokens being loaded ahead.  The backward, with four channels to a
// thread, forms s again from x, walks W - 1 tokens past its run for the gradients that reach back into it,
// and sums the filters' gradients over its run; one row of sums per run, then one pass over
// those.  Where C is no multiple of VEC the last thread of a row has the row's last VEC channels, some of
// them its neighbour's too, which both work out alike; loads and stores need a value's own alignment only.
// Few channels or tokens go by single channels.
//
// B8 T4096 C4096 bf16: forward 95 us (5.7 TB/s), backward 191 us (4.2 TB/s), its sums 7 us.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "abi_checks.h"
#include "column_sums.h"
#include "conv.h"
#include "rows_device.h"

namespace conv {
namespace {

using namespace rows;
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(2)));   // at any value's address
typedef unsigned int u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

constexpr int kAhead = 8;       // tokens loaded at once; runs are multiples of it
constexpr int kAheadFwd = 4;    // forward (B8 T4096 C4096: 95 us, with 8 101)
constexpr int NT = 256;

struct Args {
    const void *x, *w, *bias, *h0, *dy, *dhT;
    void *y, *hT, *dx, *dh0;
    float* part;
    int64_t x_ld;
    const int* cu;
    int silu, B, T, C, N, run, runs;   // tokens of a run, run slots
    int zero;                          // rows outside the sequences are zeroed
    bool wbf16;   // filters in bf16
    uint32_t zero_from;                // the workgroups from this one on zero rows outside the sequences
};

struct StepArgs {
    const void *x, *w, *bias, *state;
    void *state_out, *y;
    int64_t x_ld;
    const int* slots;
    int silu, B, T, C, P;
    bool wbf16;   // filters in bf16
};

// VEC values as stored.
template <typename T, int VEC>
struct __attribute__((aligned(sizeof(T) * VEC))) Raw {
    T v[VEC];
    __device__ __forceinline__ void load(const T* p) {
        if constexpr (VEC * sizeof(T) == 16) *reinterpret_cast<u32x4*>(v) = *reinterpret_cast<const u32x4_any*>(p);
        else if constexpr (VEC * sizeof(T) == 8) *reinterpret_cast<u32x2*>(v) = *reinterpret_cast<const u32x2_any*>(p);
        else v[0] = *p;
    }
    __device__ __forceinline__ void store(T* p) const {
        if constexpr (VEC * sizeof(T) == 16) *reinterpret_cast<u32x4_any*>(p) = *reinterpret_cast<const u32x4*>(v);
        else if constexpr (VEC * sizeof(T) == 8) *reinterpret_cast<u32x2_any*>(p) = *reinterpret_cast<const u32x2*>(v);
        else *p = v[0];
    }
    // without the first `skip`
    __device__ __forceinline__ void store(T* p, int skip) const {
        if (skip == 0) {
            store(p);
        } else {
#pragma unroll
            for (int e = 1; e < VEC; ++e)
                if (e >= skip) p[e] = v[e];
        }
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = T(0);
    }
};
template <typename T, int VEC>
__device__ __forceinline__ void store_as(T* p, const float (&f)[VEC], int skip = 0) {
    Raw<T, VEC> r;
#pragma unroll
    for (int e = 0; e < VEC; ++e) st(&r.v[e], f[e]);
    r.store(p, skip);
}

// N values of either type; four at a time where N is a multiple of four.
template <int N>
__device__ __forceinline__ void load_values(const void* base, bool bf16, int64_t at, float (&v)[N]) {
    if constexpr (N % 4 == 0) {
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            if (bf16) {
                const u32x2 u = *reinterpret_cast<const u32x2_any*>(static_cast<const uint16_t*>(base) + at + i);
                v[i] = __uint_as_float(u[0] << 16), v[i + 1] = __uint_as_float(u[0] & 0xffff0000u);
                v[i + 2] = __uint_as_float(u[1] << 16), v[i + 3] = __uint_as_float(u[1] & 0xffff0000u);
            } else {
                const u32x4 u = *reinterpret_cast<const u32x4_any*>(static_cast<const float*>(base) + at + i);
#pragma unroll
                for (int k = 0; k < 4; ++k) v[i + k] = __uint_as_float(u[k]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
            v[i] = bf16 ? widen(static_cast<const uint16_t*>(base)[at + i]) : static_cast<const float*>(base)[at + i];
    }
}
// The filters (C, W) and biases of channels c .. c + VEC - 1.
template <int W, int VEC>
__device__ __forceinline__ void load_filters(const void* w, const void* bias, bool bf16, int c, float (&f)[W][VEC],
                                             float (&b)[VEC]) {
    float all[VEC * W];
    load_values<VEC * W>(w, bf16, (int64_t)c * W, all);
#pragma unroll
    for (int e = 0; e < VEC; ++e)
#pragma unroll
        for (int j = 0; j < W; ++j) f[j][e] = all[e * W + j];
    if (bias) {
        load_values<VEC>(bias, bf16, c, b);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) b[e] = 0.f;
    }
}

// The W - 1 inputs before token t of a sequence (its state before its first token).
template <typename T, int W, int VEC>
__device__ __forceinline__ void load_window(const T* x, int64_t x_ld, const T* h0, int C, int t, Raw<T, VEC> (&win)[W - 1]) {
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
        const int q = t - (W - 1) + j;
        if (q >= 0) win[j].load(x + q * x_ld);
        else if (h0) win[j].load(h0 + (int64_t)(q + W - 1) * C);
        else win[j].clear();
    }
}

template <typename T, int W, int VEC>
__global__ __launch_bounds__(NT) void fwd_kernel(Args p) {
    if (blockIdx.x >= p.zero_from) {
        zero_outside(Seqs{p.cu, p.N, p.T}, p.y, (int64_t)p.C * sizeof(T), (int64_t)(blockIdx.x - p.zero_from) * NT + threadIdx.x);
        return;
    }
    const int CV = (p.C + VEC - 1) / VEC;
    const int64_t id = (int64_t)blockIdx.x * NT + threadIdx.x;
    const int slot = (int)(id / CV), c = min((int)(id % CV) * VEC, p.C - VEC);
    const Seqs seqs{p.cu, p.N, p.T};
    int n, piece, len;
    if (slot >= p.runs || !slot_piece(seqs, slot, p.run, n, piece)) return;
    int64_t tok0;
    seq_span(seqs, n, tok0, len);
    const int t_begin = piece * p.run, t_end = min(len, t_begin + p.run);
    const T* x = static_cast<const T*>(p.x) + tok0 * p.x_ld + c;
    const T* h0 = p.h0 ? static_cast<const T*>(p.h0) + (int64_t)n * (W - 1) * p.C + c : nullptr;
    T* y = static_cast<T*>(p.y) + tok0 * p.C + c;
    float f[W][VEC], b[VEC];
    load_filters<W, VEC>(p.w, p.bias, p.wbf16, c, f, b);
    Raw<T, VEC> win[W - 1], next[kAheadFwd];
    load_window<T, W, VEC>(x, p.x_ld, h0, p.C, t_begin, win);
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < kAheadFwd; ++i)
            if (t0 + i < t_end) next[i].load(x + (t0 + i) * p.x_ld);
    };
    fetch(t_begin);
    for (int t0 = t_begin; t0 < t_end; t0 += kAheadFwd) {
        Raw<T, VEC> cur[kAheadFwd];
#pragma unroll
        for (int i = 0; i < kAheadFwd; ++i) cur[i] = next[i];
        fetch(t0 + kAheadFwd);
#pragma unroll
        for (int i = 0; i < kAheadFwd; ++i) {
            if (t0 + i >= t_end) break;
            float s[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s[e] = b[e];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) s[e] = fmaf(f[j][e], widen(win[j].v[e]), s[e]);
                s[e] = fmaf(f[W - 1][e], widen(cur[i].v[e]), s[e]);
                if (p.silu) s[e] *= sigmoid_for<T>(s[e]);
            }
            store_as(y + (int64_t)(t0 + i) * p.C, s);
#pragma unroll
            for (int j = 0; j < W - 2; ++j) win[j] = win[j + 1];
            win[W - 2] = cur[i];
        }
    }
    if (p.hT && t_end == len) {
        T* hT = static_cast<T*>(p.hT) + (int64_t)n * (W - 1) * p.C + c;
#pragma unroll
        for (int j = 0; j < W - 1; ++j) win[j].store(hT + (int64_t)j * p.C);
    }
}

// Token t gives ds_t (0 past the sequence's end); with it dx of token t - W + 1 is complete:
// dx_q = sum_j w_j ds_(q + W - 1 - j), and for q before the first token that is dh0.
template <typename T, int W, int VEC>
__global__ __launch_bounds__(NT) void bwd_kernel(Args p) {
    if (blockIdx.x >= p.zero_from) {
        zero_outside(Seqs{p.cu, p.N, p.T}, p.dx, (int64_t)p.C * sizeof(T), (int64_t)(blockIdx.x - p.zero_from) * NT + threadIdx.x);
        return;
    }
    const int CV = (p.C + VEC - 1) / VEC;
    const int64_t id = (int64_t)blockIdx.x * NT + threadIdx.x;
    const int slot = (int)(id / CV), c = min((int)(id % CV) * VEC, p.C - VEC);
    if (slot >= p.runs) return;
    const Seqs seqs{p.cu, p.N, p.T};
    float dw[W][VEC], db[VEC];
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
        db[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
    }
    int n, piece, len;
    if (slot_piece(seqs, slot, p.run, n, piece)) {
        int64_t tok0;
        seq_span(seqs, n, tok0, len);
        const int t_begin = piece * p.run, t_end = min(len, t_begin + p.run);
        const T* x = static_cast<const T*>(p.x) + tok0 * p.x_ld + c;
        const T* dy = static_cast<const T*>(p.dy) + tok0 * p.C + c;
        T* dx = static_cast<T*>(p.dx) + tok0 * p.C + c;
        const int64_t state = (int64_t)n * (W - 1) * p.C + c;
        const T* h0 = p.h0 ? static_cast<const T*>(p.h0) + state : nullptr;
        const T* dhT = p.dhT ? static_cast<const T*>(p.dhT) + state : nullptr;
        T* dh0 = p.dh0 ? static_cast<T*>(p.dh0) + state : nullptr;
        float f[W][VEC], b[VEC], win[W - 1][VEC], ds[W - 1][VEC];     // x of the W - 1 tokens before, ds[j] of token t - 1 - j
        load_filters<W, VEC>(p.w, p.bias, p.wbf16, c, f, b);
        {
            Raw<T, VEC> raw[W - 1];
            load_window<T, W, VEC>(x, p.x_ld, h0, p.C, t_begin, raw);
#pragma unroll
            for (int j = 0; j < W - 1; ++j)
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    win[j][e] = widen(raw[j].v[e]);
                    ds[j][e] = 0.f;
                }
        }
        Raw<T, VEC> nx[kAhead], ny[kAhead];
        const int t_stop = t_end + W - 1;                  // the last tokens' dx need what lies behind
        auto fetch = [&](int t0) {
            const int end = min(t_stop, len);
#pragma unroll
            for (int i = 0; i < kAhead; ++i)
                if (t0 + i < end) {
                    nx[i].load(x + (t0 + i) * p.x_ld);
                    ny[i].load(dy + (int64_t)(t0 + i) * p.C);
                }
        };
        // One token of x and dy; behind the sequence (not real) its ds is 0 whatever the window holds, and its sums
        // count if it lies in this run.
        auto token = [&](const Raw<T, VEC>& rx, const Raw<T, VEC>& ry, bool real, bool mine, float (&g)[VEC]) {
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float xe = widen(rx.v[e]);
                float s = b[e], d = widen(ry.v[e]);
#pragma unroll
                for (int j = 0; j < W - 1; ++j) s = fmaf(f[j][e], win[j][e], s);
                s = fmaf(f[W - 1][e], xe, s);
                if (p.silu) {
                    const float sg = sigmoid(s);
                    d *= fmaf(s * sg, 1.f - sg, sg);
                }
                if (!real) d = 0.f;
                if (mine) {
#pragma unroll
                    for (int j = 0; j < W - 1; ++j) dw[j][e] = fmaf(d, win[j][e], dw[j][e]);
                    dw[W - 1][e] = fmaf(d, xe, dw[W - 1][e]);
                    db[e] += d;
                }
                g[e] = f[0][e] * d;
#pragma unroll
                for (int j = 1; j < W; ++j) g[e] = fmaf(f[j][e], ds[j - 1][e], g[e]);
#pragma unroll
                for (int j = W - 2; j > 0; --j) ds[j][e] = ds[j - 1][e];
                ds[0][e] = d;
#pragma unroll
                for (int j = 0; j < W - 2; ++j) win[j][e] = win[j + 1][e];
                win[W - 2][e] = xe;
            }
        };
        fetch(t_begin);
        for (int t0 = t_begin; t0 < t_stop; t0 += kAhead) {
            Raw<T, VEC> cx[kAhead], cy[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                cx[i] = nx[i];
                cy[i] = ny[i];
            }
            fetch(t0 + kAhead);
            float g[VEC];
            if (t0 > t_begin && t0 + kAhead <= t_end) {    // whole blocks, all but the first
#pragma unroll
                for (int i = 0; i < kAhead; ++i) {
                    token(cx[i], cy[i], true, true, g);
                    store_as(dx + (int64_t)(t0 + i - (W - 1)) * p.C, g);
                }
                continue;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int t = t0 + i, q = t - (W - 1);
                if (t >= t_stop) break;
                if (t >= len) {
                    cx[i].clear();
                    cy[i].clear();
                }
                token(cx[i], cy[i], t < len, t < t_end, g);
                if (q < t_begin && !(piece == 0 && dh0)) continue;
                if (dhT && q >= len - (W - 1)) {
                    Raw<T, VEC> last;
                    last.load(dhT + (int64_t)(q - len + W - 1) * p.C);
#pragma unroll
                    for (int e = 0; e < VEC; ++e) g[e] += widen(last.v[e]);
                }
                if (q >= 0) store_as(dx + (int64_t)q * p.C, g);
                else store_as(dh0 + (int64_t)(q + W - 1) * p.C, g);
            }
        }
    }
    float* part = p.part + (int64_t)slot * (W + 1) * p.C;    // [channel][filter], then the biases
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
#pragma unroll
        for (int j = 0; j < W; ++j) part[(int64_t)(c + e) * W + j] = dw[j][e];
        part[(int64_t)W * p.C + c + e] = db[e];
    }
}

// Batch row r works on state slots[r]; rows of the same slot are done by the first of them,
// in batch order, so no two workgroups share a state.
template <typename T, int W, int VEC>
__global__ __launch_bounds__(NT) void step_kernel(StepArgs p, int nsub) {
    const int sub = blockIdx.x % nsub, r = blockIdx.x / nsub, c0 = (sub * NT + threadIdx.x) * VEC, c = min(c0, p.C - VEC);
    const bool on = c0 < p.C;
    const int twice = c0 - c;    // channels that a neighbour has too; it alone writes them, for their states may change in place
    T* y = static_cast<T*>(p.y) + c;
    int slot = r, end = r + 1;                             // rows r .. end - 1 are looked through
    if (p.slots) {
        slot = p.slots[r];
        if (slot < 0 || slot >= p.P) {
            Raw<T, VEC> zero;
            zero.clear();
            for (int t = 0; t < p.T && on; ++t) zero.store(y + ((int64_t)r * p.T + t) * p.C, twice);
            return;
        }
        bool before = false, after = false;                // whether other rows have this slot; every wave for itself
        for (int e = threadIdx.x & 63; e < p.B; e += 64) {
            const bool same = p.slots[e] == slot;
            before |= same && e < r;
            after |= same && e > r;
        }
        if (__ballot(before)) return;
        if (__ballot(after)) end = p.B;
    }
    if (!on) return;
    const T* x = static_cast<const T*>(p.x) + c;
    const int64_t at = (int64_t)slot * (W - 1) * p.C + c;
    Raw<T, VEC> win[W - 1];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j].load(static_cast<const T*>(p.state) + at + (int64_t)j * p.C);
    float f[W][VEC], b[VEC];
    load_filters<W, VEC>(p.w, p.bias, p.wbf16, c, f, b);
    for (int row = r; row < end; ++row) {
        if (row != r && p.slots[row] != slot) continue;
        for (int t = 0; t < p.T; ++t) {
            const int64_t tok = (int64_t)row * p.T + t;
            Raw<T, VEC> cur;
            cur.load(x + tok * p.x_ld);
            float s[VEC];
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                s[e] = b[e];
#pragma unroll
                for (int j = 0; j < W - 1; ++j) s[e] = fmaf(f[j][e], widen(win[j].v[e]), s[e]);
                s[e] = fmaf(f[W - 1][e], widen(cur.v[e]), s[e]);
                if (p.silu) s[e] *= sigmoid_for<T>(s[e]);
            }
            store_as(y + tok * p.C, s, twice);
#pragma unroll
            for (int j = 0; j < W - 2; ++j) win[j] = win[j + 1];
            win[W - 2] = cur;
        }
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j) win[j].store(static_cast<T*>(p.state_out) + at + (int64_t)j * p.C, twice);
}

enum { kFwd, kBwd };

template <typename T, int W, int VEC>
hipError_t run(const Args& a, int what, hipStream_t s) {
    constexpr int BV = VEC > 4 ? 4 : VEC;      // the backward by four channels: its sums and windows are many registers
    const int BW = what == kFwd ? VEC : BV;
    const int64_t threads = (int64_t)a.runs * ((a.C + BW - 1) / BW);
    Args b = a;
    b.zero_from = (uint32_t)((threads + NT - 1) / NT);
    const dim3 grid(b.zero_from + (a.cu && a.zero ? kZeroBlocks : 0));
    if (what == kFwd) hipLaunchKernelGGL((fwd_kernel<T, W, VEC>), grid, dim3(NT), 0, s, b);
    else hipLaunchKernelGGL((bwd_kernel<T, W, BV>), grid, dim3(NT), 0, s, b);
    return hipGetLastError();
}
template <typename T, int W, int VEC>
hipError_t run(const StepArgs& a, int, hipStream_t s) {
    // by four channels too: half the loads to a thread before its first product (4096 channels of bf16: 4 rows 4.0 -> 2.5
    // us, 256 rows 8.7 -> 6.8)
    constexpr int BV = VEC > 4 ? 4 : VEC;
    const int nsub = (a.C + BV * NT - 1) / (BV * NT);
    hipLaunchKernelGGL((step_kernel<T, W, BV>), dim3((uint32_t)a.B * nsub), dim3(NT), 0, s, a, nsub);
    return hipGetLastError();
}
template <typename T, int VEC, typename A>
hipError_t pick_w(const A& a, int W, int what, hipStream_t s) {
    switch (W) {
        case 2: return run<T, 2, VEC>(a, what, s);
        case 3: return run<T, 3, VEC>(a, what, s);
        default: return run<T, 4, VEC>(a, what, s);
    }
}
// Vectors, or one channel to a thread: many short loads beat few long ones until the vectors alone fill the
// chip.  1001 channels of bf16, forward: of 2000 tokens (16 thousand threads in runs of 16) 7.9 us by
// vectors, 4.9 by single channels, of 4000 8.5 and 7.2, of 8000 9.3 and 10.8; gradient: of 2000 15.8 and
// 11.5, of 4000 19.1 and 16.2, of 8000 (125 thousand threads) 25.1 and 25.2.
bool by_vectors(const Args& a, int what, bool bf16) {
    const int vec = bf16 && what == kFwd ? 8 : 4;
    return a.C >= (bf16 ? 8 : 4) && (int64_t)a.B * a.T / 16 * ((a.C + vec - 1) / vec) >= (what == kFwd ? 49152 : 131072);
}
bool by_vectors(const StepArgs& a, int, bool bf16) { return a.C >= (bf16 ? 8 : 4); }

template <typename A>
hipError_t launch(const A& a, int W, bool bf16, int what, hipStream_t s) {
    const bool vec = by_vectors(a, what, bf16);
    if (bf16) return vec ? pick_w<uint16_t, 8>(a, W, what, s) : pick_w<uint16_t, 1>(a, W, what, s);
    return vec ? pick_w<float, 4>(a, W, what, s) : pick_w<float, 1>(a, W, what, s);
}

// Tokens of a run: as many as still leave 2^16 threads of 16 bytes each, 16 to 128 (12289 tokens of 2048
// channels, packed: runs of 32 28 us, of 16 31).
int run_of(int64_t tokens, int C) {
    const int64_t threads = tokens * ((C + 7) / 8);
    int run = 16;
    while (run < 128 && threads / (2 * run) >= 65536) run *= 2;
    return run;
}
int64_t runs_of(int B, int T, int N, bool packed, int run) {
    return packed ? T / run + (int64_t)N : (int64_t)B * ((T - 1) / run + 1);
}

bool is_dtype(int d) { return d == WKV7_F32 || d == WKV7_BF16; }
int esz(int d) { return d == WKV7_BF16 ? 2 : 4; }

wkv7_status check_shape(int B, int T, int C, int W, int N, bool packed) {
    if (B < 1 || T < 1 || C < 1 || W < 2 || W > 4 || (packed && (B != 1 || N < 1))) return WKV7_ERR_SHAPE;
    if (C > (1 << 20) || (int64_t)B * T > (int64_t(1) << 40) / C || (int64_t)B * T > INT32_MAX - 1024)
        return WKV7_ERR_SHAPE;                             // 32-bit positions, past the end too
    // a launch takes fewer than 2^32 threads: one for each run and channel at most
    if (runs_of(B, T, N, packed, run_of((int64_t)B * T, C)) > (int64_t(1) << 30) / C) return WKV7_ERR_SHAPE;
    return WKV7_OK;
}
int64_t span(int64_t rows, int64_t ld, int64_t C, int e) { return ((rows - 1) * ld + C) * e; }

}  // namespace
}  // namespace conv

extern "C" {

wkv7_status conv_fwd(int B, int T, int C, int W, wkv7_dtype x_dtype, wkv7_dtype w_dtype, const void* x, int64_t x_ld,
                     const void* weight, const void* bias, int silu, const int32_t* cu_seqlens, int N, int zero_outside,
                     const void* h0, void* y, void* hT, void* stream) {
    using namespace conv;
    if (!is_dtype(x_dtype) || !is_dtype(w_dtype)) return WKV7_ERR_DTYPE;
    const bool packed = cu_seqlens != nullptr;
    wkv7_status st = check_shape(B, T, C, W, N, packed);
    if (st != WKV7_OK) return st;
    const int e = esz(x_dtype), we = esz(w_dtype);
    const int64_t tokens = (int64_t)B * T, sb = (int64_t)(packed ? N : B) * (W - 1) * C * e;
    if (x_ld < C || x_ld > (int64_t(1) << 40) / tokens) return WKV7_ERR_SHAPE;
    const abi::Buf bufs[] = {{x, span(tokens, x_ld, C, e), true, false, e}, {weight, (int64_t)C * W * we, true, false, we},
                             {bias, (int64_t)C * we, false, false, we},
                             {cu_seqlens, (N + 1) * 4LL, false, false, 4}, {h0, sb, false, false, e},
                             {y, tokens * C * e, true, true, e}, {hT, sb, false, true, e}};
    st = abi::check(bufs);
    if (st != WKV7_OK) return st;
    Args a = {};
    a.x = x; a.w = weight; a.bias = bias; a.h0 = h0; a.y = y; a.hT = hT; a.x_ld = x_ld; a.cu = cu_seqlens;
    a.silu = silu; a.B = B; a.T = T; a.C = C; a.N = packed ? N : B; a.wbf16 = w_dtype == WKV7_BF16;
    a.zero = zero_outside;
    a.run = run_of(tokens, C);
    a.runs = (int)runs_of(B, T, N, packed, a.run);
    return launch(a, W, x_dtype == WKV7_BF16, kFwd, static_cast<hipStream_t>(stream)) == hipSuccess ? WKV7_OK
                                                                                                         : WKV7_ERR_HIP;
}

size_t conv_bwd_workspace_bytes(int B, int T, int C, int W, int N, int packed) {
    if (conv::check_shape(B, T, C, W, N, packed != 0) != WKV7_OK) return 0;
    return (size_t)conv::runs_of(B, T, N, packed != 0, conv::run_of((int64_t)B * T, C)) * (W + 1) * C * 4;
}

wkv7_status conv_bwd(int B, int T, int C, int W, wkv7_dtype x_dtype, wkv7_dtype w_dtype, const void* dy,
                     const void* dhT, const void* x, int64_t x_ld, const void* weight, const void* bias, int silu,
                     const int32_t* cu_seqlens, int N, int zero_outside, const void* h0, void* dx, float* dweight, float* dbias, void* dh0,
                     void* workspace, size_t workspace_bytes, void* stream) {
    using namespace conv;
    if (!is_dtype(x_dtype) || !is_dtype(w_dtype)) return WKV7_ERR_DTYPE;
    const bool packed = cu_seqlens != nullptr;
    wkv7_status st = check_shape(B, T, C, W, N, packed);
    if (st != WKV7_OK) return st;
    const int e = esz(x_dtype), we = esz(w_dtype);
    const int64_t tokens = (int64_t)B * T, nb = tokens * C * e, sb = (int64_t)(packed ? N : B) * (W - 1) * C * e;
    if (x_ld < C || x_ld > (int64_t(1) << 40) / tokens) return WKV7_ERR_SHAPE;
    const int64_t need = (int64_t)conv_bwd_workspace_bytes(B, T, C, W, N, packed);
    const abi::Buf bufs[] = {{dy, nb, true, false, e}, {dhT, sb, false, false, e},
                             {x, span(tokens, x_ld, C, e), true, false, e}, {weight, (int64_t)C * W * we, true, false, we},
                             {bias, (int64_t)C * we, false, false, we}, {cu_seqlens, (N + 1) * 4LL, false, false, 4},
                             {h0, sb, false, false, e}, {dx, nb, true, true, e}, {dweight, (int64_t)C * W * 4, true, true, 4},
                             {dbias, (int64_t)C * 4, false, true, 4}, {dh0, sb, false, true, e},
                             {workspace, need, false, true, 16}};
    st = abi::check(bufs);
    if (st != WKV7_OK) return st;
    if (!workspace || workspace_bytes < (size_t)need) return WKV7_ERR_WORKSPACE;
    Args a = {};
    a.x = x; a.w = weight; a.bias = bias; a.h0 = h0; a.dy = dy; a.dhT = dhT; a.dx = dx; a.dh0 = dh0; a.x_ld = x_ld;
    a.cu = cu_seqlens; a.silu = silu; a.B = B; a.T = T; a.C = C; a.N = packed ? N : B; a.wbf16 = w_dtype == WKV7_BF16;
    a.zero = zero_outside;
    a.run = run_of(tokens, C);
    a.runs = (int)runs_of(B, T, N, packed, a.run);
    a.part = static_cast<float*>(workspace);
    hipStream_t hs = static_cast<hipStream_t>(stream);
    hipError_t err = launch(a, W, x_dtype == WKV7_BF16, kBwd, hs);
    if (err == hipSuccess)
        err = sums::launch_column_sums(a.part, a.runs, (int64_t)(W + 1) * C, dweight, (int64_t)W * C, dbias, C, nullptr, hs);
    return err == hipSuccess ? WKV7_OK : WKV7_ERR_HIP;
}

wkv7_status conv_step(int B, int T, int C, int W, wkv7_dtype x_dtype, wkv7_dtype w_dtype, const void* x, int64_t x_ld,
                      const void* weight, const void* bias, int silu, const int32_t* slots, int P, const void* state,
                      void* state_out, void* y, void* stream) {
    using namespace conv;
    if (!is_dtype(x_dtype) || !is_dtype(w_dtype)) return WKV7_ERR_DTYPE;
    if (B < 1 || T < 1 || C < 1 || W < 2 || W > 4 || P < 1 || (!slots && P < B)) return WKV7_ERR_SHAPE;
    if (C > (1 << 20) || B > (int64_t(1) << 31) / (C + NT) || (int64_t)B * T > (int64_t(1) << 40) / C || P > (int64_t(1) << 38) / C)
        return WKV7_ERR_SHAPE;
    const int e = esz(x_dtype), we = esz(w_dtype);
    const int64_t tokens = (int64_t)B * T, sb = (int64_t)P * (W - 1) * C * e;
    if (x_ld < C || x_ld > (int64_t(1) << 40) / tokens) return WKV7_ERR_SHAPE;
    const abi::Buf bufs[] = {{x, span(tokens, x_ld, C, e), true, false, e}, {weight, (int64_t)C * W * we, true, false, we},
                             {bias, (int64_t)C * we, false, false, we}, {slots, B * 4LL, false, false, 4},
                             {state, sb, true, false, e}, {state_out, sb, true, true, e},
                             {y, tokens * C * e, true, true, e}};
    wkv7_status st = abi::check(bufs, state == state_out ? state : nullptr);
    if (st != WKV7_OK) return st;
    StepArgs a = {};
    a.x = x; a.w = weight; a.bias = bias; a.state = state; a.state_out = state_out; a.y = y; a.x_ld = x_ld;
    a.slots = slots; a.silu = silu; a.B = B; a.T = T; a.C = C; a.P = P; a.wbf16 = w_dtype == WKV7_BF16;
    return launch(a, W, x_dtype == WKV7_BF16, 0, static_cast<hipStream_t>(stream)) == hipSuccess ? WKV7_OK
                                                                                                      : WKV7_ERR_HIP;
}

}  // extern "C"
