// gdr_scan.hip -- the state of the gated delta rule, and its gradient, carried
// from chunk to chunk (gfx950).
//
// The chunks of a head are a chain, so what counts is how long one chunk takes.
// A state wave holds 16 rows i of S (or of its gradient) for all K columns in
// its accumulators, as K / 16 tiles of S^T, and shares nothing with the other
// state waves: every product of the chain has the form (operand from LDS) x
// (that wave's registers).  What the chain does not wait for is done by a
// helper wave beside each state wave, one chunk behind (forward: o and the
// stores for the backward) or one chunk ahead (backward: the parts of dU and of the state
// gradient that come from dout alone); the two pass fp32 tiles through LDS, in
// accumulator order.  Memory waves copy the next chunks' K, T and gates into LDS.  One
// barrier per chunk.
#include "gdr_device.h"
#include "gdr_internal.h"
#include "wkv7_internal.h"

namespace gdr {
namespace {

using wkv7::make_rsrc;
using wkv7::Rsrc;

constexpr int NP = kPlanes;
constexpr int kLds = 160 * 1024;

// LDS plan.  One chunk's K rows, T planes and gates (e^G, e^(G_C - G), b); the backward
// also stages Q rows, one chunk further ahead; then the tiles that state and
// helper waves pass on, double-buffered by chunk parity.
template <int NX, int K, int NCW, bool BWD>
struct Plan {
    static constexpr int XB = C * K * 2;                  // one plane of K or Q rows
    static constexpr int Kr = 0, T = Kr + NX * XB, G = T + NP * kTriBytes, bytes = G + 1024;
    static constexpr int QB = BWD ? NX * XB : 0;
    static constexpr int ST = K / 16 * 1024, UT = 4 * 1024;   // state tiles, token tiles of one wave
    static constexpr int pass = 2 * NCW * (ST + UT);
    static constexpr int NBUF = 3 * bytes + 2 * QB + pass <= kLds ? 3 : 2 * bytes + 2 * QB + pass <= kLds ? 2 : 1;
    static constexpr int NQ = NBUF > 1 ? 2 : 1;
    static constexpr int Q0 = NBUF * bytes, P0 = Q0 + NQ * QB, total = P0 + pass;
    static_assert(total <= kLds, "scan LDS");
};

// A raw value of a token tensor by byte offset; 0 past the resource's end.
__device__ __forceinline__ uint16_t bload(const uint16_t*, Rsrc r, int off) {
    return __builtin_amdgcn_raw_buffer_load_b16(r, off, 0, 0);
}
__device__ __forceinline__ float bload(const float*, Rsrc r, int off) {
    return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(r, off, 0, 0));
}
__device__ __forceinline__ void bput(uint16_t*, Rsrc r, int off, float v) {
    __builtin_amdgcn_raw_buffer_store_b16(__builtin_bit_cast(uint16_t, (__bf16)v), r, off, 0, 0);
}
__device__ __forceinline__ void bput(float*, Rsrc r, int off, float v) {
    __builtin_amdgcn_raw_buffer_store_b32(__float_as_uint(v), r, off, 0, 0);
}

// Rows of K or Q of one chunk into LDS, 1 KiB pieces dealt to the memory waves.
template <int NX, int K, int NMW>
__device__ __forceinline__ void stage_rows(const Planes& x, char* buf, int64_t row0, int64_t stride, int len, int mw,
                                           int lane) {
    constexpr int U = K / 8, RPP = 64 / U;                // units per row, rows per piece
    const uint16_t* src = x.p + row0;
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
        for (int u = 0; u < C / RPP / NMW; ++u) {
            const int pc = u * NMW + mw, row = pc * RPP + lane / U;
            dma16(src + i * x.plane + min(row, len - 1) * stride + 8 * ((lane % U) ^ swz<U>(row)),
                  buf + i * C * K * 2 + pc * 1024);
        }
}

// The sequence, head and 16-row slice of a workgroup.
struct Where {
    int n, h, hk, sub, len, slot0, nc;
    int64_t tok0;
    __device__ __forceinline__ Where(const Args& p, int nsub) {
        sub = blockIdx.x % nsub;
        const int nh = blockIdx.x / nsub;
        h = nh % p.H;
        n = nh / p.H;
        hk = h / (p.H / p.Hk);
        seq_span(Seqs{p.cu, p.N, p.T, p.NC}, n, tok0, len, slot0);
        nc = (len + C - 1) / C;
    }
    __device__ __forceinline__ int64_t block(const Args& p, int c) const { return (int64_t)(slot0 + c) * p.H + h; }
};

// Byte offsets of a lane's 16 values of a chunk: tokens in accumulator order, one column.
template <typename InT>
__device__ __forceinline__ void token_offsets(int (&off)[16], const Args& p, int i, int g4) {
#pragma unroll
    for (int e = 0; e < 16; ++e)
        off[e] = (int)(((int64_t)idx(e >> 2, 4 * g4 + (e & 3)) * p.H * p.V + i) * (int64_t)sizeof(InT));
}
// Chunk c of a (tokens, H, V) tensor, ending with the sequence.
template <typename T>
__device__ __forceinline__ Rsrc chunk_rsrc(T* x, const Args& p, const Where& w, int c) {
    const int64_t stride = (int64_t)p.H * p.V;
    const bool on = x && c >= 0 && c < w.nc;
    const int rows = on ? min(C, w.len - c * C) : 0;
    return make_rsrc(on ? x + (w.tok0 + (int64_t)c * C) * stride + (int64_t)w.h * p.V : nullptr,
                     on ? (uint32_t)(((rows - 1) * stride + p.V) * (int64_t)sizeof(T)) : 0u);
}

template <int KT>
__device__ __forceinline__ void load_state(f32x4 (&s)[KT], const float* src, int64_t off) {
#pragma unroll
    for (int t = 0; t < KT; ++t)
        s[t] = src ? *reinterpret_cast<const f32x4*>(src + off + 32 * (t >> 1) + 4 * (t & 1)) : zero4();
}
template <int KT>
__device__ __forceinline__ void store_state(float* dst, int64_t off, const f32x4 (&s)[KT]) {
#pragma unroll
    for (int t = 0; t < KT; ++t) *reinterpret_cast<f32x4*>(dst + off + 32 * (t >> 1) + 4 * (t & 1)) = s[t];
}
// Token tiles of one column i to row i of a (V, 64) block.
__device__ __forceinline__ void store_tokens(float* dst, int i, int g4, const f32x4 (&u)[4]) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
        *reinterpret_cast<f32x4*>(dst + (int64_t)i * C + 32 * (t >> 1) + 8 * g4 + 4 * (t & 1)) = u[t];
}

template <int N>
__device__ __forceinline__ void pass_put(char* p, int lane, const f32x4 (&x)[N]) {
#pragma unroll
    for (int t = 0; t < N; ++t) *reinterpret_cast<f32x4*>(p + t * 1024 + lane * 16) = x[t];
}
template <int N>
__device__ __forceinline__ void pass_get(const char* p, int lane, f32x4 (&x)[N]) {
#pragma unroll
    for (int t = 0; t < N; ++t) x[t] = *reinterpret_cast<const f32x4*>(p + t * 1024 + lane * 16);
}

// Memory waves.  Buffers hold NBUF - 1 chunks ahead of the one in use (none ahead, and two
// barriers per chunk, where a single buffer is all that fits).
template <int NX, int K, int NCW, int NMW, bool BWD>
__device__ __forceinline__ void memory_wave(const Args& p, const Where& w, char* smem, int mw, int lane) {
    using L = Plan<NX, K, NCW, BWD>;
    const int64_t stride = (int64_t)p.Hk * K;
    auto chunk_of = [&](int it) { return BWD ? w.nc - 1 - it : it; };
    auto rows_of = [&](int c) { return (w.tok0 + (int64_t)c * C) * stride + (int64_t)w.hk * K; };
    auto fetch = [&](int it) {
        const int c = chunk_of(it), len = min(C, w.len - c * C);
        char* buf = smem + (it % L::NBUF) * L::bytes;
        const int64_t block = w.block(p, c);
        stage_rows<NX, K, NMW>(p.kp, buf + L::Kr, rows_of(c), stride, len, mw, lane);
        const char* ops = p.ops + block * kOpsBytes;
#pragma unroll
        for (int u = 0; u < NP * kTriBytes / 1024 / NMW; ++u)
            dma16(ops + (u * NMW + mw) * 1024 + 16 * lane, buf + L::T + (u * NMW + mw) * 1024);
        if (mw == 0) dma16(reinterpret_cast<const char*>(p.gates + block * kGateFloats) + 16 * lane, buf + L::G);
    };
    auto fetch_q = [&](int it) {
        if constexpr (BWD) {
            if (it >= w.nc) return;                       // an empty sequence has no chunk 0
            const int c = chunk_of(it);
            stage_rows<NX, K, NMW>(p.qp, smem + L::Q0 + (it % L::NQ) * L::QB, rows_of(c), stride, min(C, w.len - c * C),
                                   mw, lane);
        }
    };
    auto landed = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };
    constexpr int ahead = L::NBUF - 1;
    if constexpr (L::NBUF == 1) {
        // forward: chunk it's buffer; backward: Q of chunk it + 1 beside K of chunk it
        fetch_q(0);
        landed();
        lds_barrier();
        if constexpr (BWD) lds_barrier();                 // the helper's first chunk
        for (int it = 0; it < w.nc; ++it) {
            fetch(it);
            fetch_q(it + 1);
            landed();
            lds_barrier();
            lds_barrier();                                // its readers are done
        }
        return;
    }
    for (int it = 0; it < min(ahead, w.nc); ++it) fetch(it);
    fetch_q(0);
    fetch_q(1);
    landed();
    lds_barrier();
    if constexpr (BWD) lds_barrier();                     // the helper's first chunk
    for (int it = 0; it < w.nc; ++it) {
        fetch_q(it + 2);                                  // first: the helper reads it in the next iteration
        if (it + ahead < w.nc) fetch(it + ahead);
        if constexpr (ahead == 1) {
            landed();
        } else {
            // chunk it + 1 was fetched in the iteration before: only this iteration's chunk may be
            // in flight (loads land in order)
            constexpr int n = NX * C * K * 2 / 1024 / NMW + NP * kTriBytes / 1024 / NMW;
            if (it + ahead < w.nc) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
            else landed();
        }
        lds_barrier();
    }
}

// v -> o, the states entering the chunks and U (ckpt), hT.
template <typename InT, int NX, int K, int NCW, int NMW>
__global__ __launch_bounds__(64 * (2 * NCW + NMW)) void fwd_kernel(Args p, int nsub) {
    using L = Plan<NX, K, NCW, false>;
    constexpr int U = K / 8, KS = K / 32, KT = K / 16;
    // o leaves in in_dtype: for bf16 two planes (2^-17) in its own products lose nothing
    // beside its rounding; the state's products keep all three
    constexpr int NO = sizeof(InT) == 2 ? 2 : NP;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g4 = lane >> 4, r16 = lane & 15;
    const Where w(p, nsub);
    if (wave >= 2 * NCW) {
        memory_wave<NX, K, NCW, NMW, false>(p, w, smem, wave - 2 * NCW, lane);
        return;
    }
    const int cw = wave % NCW, i = 16 * (w.sub * NCW + cw) + r16;     // this lane's state row
    auto pass = [&](int it) { return smem + L::P0 + ((it & 1) * NCW + cw) * (L::ST + L::UT); };
    const int64_t soff = (((int64_t)w.n * p.H + w.h) * p.V + i) * K + 8 * g4;

    if (wave < NCW) {
        // ---- state wave
        f32x4 s[KT];                                      // s[2c + hh][q] = S[i][32c + 8g + 4hh + q]
        load_state(s, p.h0, soff);
        const InT* v = static_cast<const InT*>(p.v);
        int off[16];
        token_offsets<InT>(off, p, i, g4);
        InT xn[16];
        auto load_v = [&](int c) {
            const Rsrc r = chunk_rsrc(v, p, w, c);
#pragma unroll
            for (int e = 0; e < 16; ++e) xn[e] = bload(v, r, off[e]);
        };
        load_v(0);
        lds_barrier();
        for (int it = 0; it < w.nc; ++it) {
            if constexpr (L::NBUF == 1) lds_barrier();
            const char* buf = smem + (it % L::NBUF) * L::bytes;
            const float* gates = reinterpret_cast<const float*>(buf + L::G);
            auto gate = [&](int which, int t) { return *reinterpret_cast<const f32x4*>(gates + which + idx(t, 4 * g4)); };
            f32x4 xa[4];
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) xa[t][q] = widen(xn[4 * t + q]);
            load_v(it + 1);
            pass_put(pass(it), lane, s);
            // a = K S^T;  R = V - e^G a;  U = T (b R)
            f32x4 a[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) a[t] = zero4();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const PF<NP> sf = pf_acc<NP>(s[2 * ks], s[2 * ks + 1]);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    a[t] = pmma<NP>(a[t], frag_row<U, NX>(buf + L::Kr, L::XB, idx(t, r16), ks, lane), sf);
            }
            f32x4 u[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) a[t] = gate(kGateBeta, t) * (xa[t] - gate(kGateEG, t) * a[t]);
            const PF<NP> rf[2] = {pf_acc<NP>(a[0], a[1]), pf_acc<NP>(a[2], a[3])};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u[t] = zero4();
#pragma unroll
                for (int ks = 0; ks <= (t >> 1); ++ks) u[t] = pmma<NP>(u[t], tri_row<NP>(buf + L::T, t, ks, lane), rf[ks]);
            }
            pass_put(pass(it) + L::ST, lane, u);
            // S1^T = e^(G_C) S0^T + K^T (e^(G_C - G) U)
#pragma unroll
            for (int t = 0; t < 4; ++t) u[t] = gate(kGateToEnd, t) * u[t];
            const float eGC = gates[kGateEG + C - 1];
            const PF<NP> ue[2] = {pf_acc<NP>(u[0], u[1]), pf_acc<NP>(u[2], u[3])};
#pragma unroll
            for (int t = 0; t < KT; ++t) s[t] = eGC * s[t];
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int t = 0; t < KT; ++t)
                    s[t] = pmma<NP>(s[t], frag_col<U, NX>(buf + L::Kr, L::XB, t, ks, lane), ue[ks]);
            lds_barrier();
        }
        if (p.hT) store_state(p.hT, soff, s);
        return;
    }

    // ---- helper wave: chunk it - 1 in iteration it
    const int64_t stride = (int64_t)p.Hk * K;
    InT* o = static_cast<InT*>(p.o);
    int off[16];
    token_offsets<InT>(off, p, i, g4);
    PF<NX> qf[4][KS];
    PF<NO> mf[6];                                         // tiles 0, 1 (step 0), 2, 3 (steps 0, 1)
    f32x4 eg[4];
    auto load = [&](int c) {
        if (c >= w.nc || !o) return;
        const int len = min(C, w.len - c * C);
        const uint16_t* q = p.qp.p + (w.tok0 + (int64_t)c * C) * stride + (int64_t)w.hk * K + 8 * g4;
        const int64_t block = w.block(p, c);
        const char* m = p.ops + block * kOpsBytes + NP * kTriBytes + 16 * lane;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int j = 0; j < NX; ++j)
                    qf[t][ks].p[j] = *reinterpret_cast<const bf16x8*>(q + j * p.qp.plane +
                                                                     min(idx(t, r16), len - 1) * stride + 32 * ks);
            eg[t] = *reinterpret_cast<const f32x4*>(p.gates + block * kGateFloats + kGateEG + idx(t, 4 * g4));
        }
#pragma unroll
        for (int f = 0; f < 6; ++f)
#pragma unroll
            for (int j = 0; j < NO; ++j) mf[f].p[j] = *reinterpret_cast<const bf16x8*>(m + j * kTriBytes + f * 1024);
    };
    load(0);
    lds_barrier();
    for (int it = 0; it <= w.nc; ++it) {
        if constexpr (L::NBUF == 1) {
            if (it < w.nc) lds_barrier();
        }
        if (it > 0) {
            const int c = it - 1;
            f32x4 s[KT], u[4];
            pass_get(pass(c), lane, s);
            pass_get(pass(c) + L::ST, lane, u);
            if (p.ckpt) {
                float* ck = p.ckpt + w.block(p, c) * (int64_t)p.V * (K + C);
                store_state(ck, (int64_t)i * K + 8 * g4, s);
                store_tokens(ck + (int64_t)p.V * K, i, g4, u);
            }
            if (o) {
                // O = scale (e^G Q S0^T + M U)
                f32x4 b[4];
#pragma unroll
                for (int t = 0; t < 4; ++t) b[t] = zero4();
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    const PF<NO> sf = pf_acc<NO>(s[2 * ks], s[2 * ks + 1]);
#pragma unroll
                    for (int t = 0; t < 4; ++t) b[t] = pmma<NO>(b[t], qf[t][ks], sf);
                }
                const PF<NO> uf[2] = {pf_acc<NO>(u[0], u[1]), pf_acc<NO>(u[2], u[3])};
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    b[t] = eg[t] * b[t];
#pragma unroll
                    for (int ks = 0; ks <= (t >> 1); ++ks) b[t] = pmma<NO>(b[t], mf[t < 2 ? t : 2 * t - 2 + ks], uf[ks]);
                }
                load(it);
                const Rsrc r = chunk_rsrc(o, p, w, c);
#pragma unroll
                for (int e = 0; e < 16; ++e) bput(o, r, off[e], p.scale * b[e >> 2][e & 3]);
            }
        }
        if (it < w.nc) lds_barrier();
    }
}

// dout -> dv, the state gradients at the chunks' ends (dend), Z, dh0.
//   dU = scale M^T DO + e^(G_C - G) K G1^T      (G1: gradient at the chunk's end)
//   Z  = T^T dU,   dv = b Z
//   G0 = e^(G_C) G1 + scale DO^T e^G Q - (b Z)^T e^G K
template <typename InT, int NX, int K, int NCW, int NMW>
__global__ __launch_bounds__(64 * (2 * NCW + NMW)) void bwd_kernel(Args p, int nsub) {
    using L = Plan<NX, K, NCW, true>;
    constexpr int U = K / 8, KS = K / 32, KT = K / 16;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g4 = lane >> 4, r16 = lane & 15;
    const Where w(p, nsub);
    if (wave >= 2 * NCW) {
        memory_wave<NX, K, NCW, NMW, true>(p, w, smem, wave - 2 * NCW, lane);
        return;
    }
    const int cw = wave % NCW, i = 16 * (w.sub * NCW + cw) + r16;
    auto chunk_of = [&](int it) { return w.nc - 1 - it; };
    auto pass = [&](int it) { return smem + L::P0 + ((it & 1) * NCW + cw) * (L::ST + L::UT); };
    const int64_t soff = (((int64_t)w.n * p.H + w.h) * p.V + i) * K + 8 * g4;
    int off[16];
    token_offsets<InT>(off, p, i, g4);

    if (wave < NCW) {
        // ---- state wave
        f32x4 s[KT];
        load_state(s, p.dhT, soff);
        InT* dv = static_cast<InT*>(p.dv);
        lds_barrier();
        lds_barrier();
        for (int it = 0; it < w.nc; ++it) {
            if constexpr (L::NBUF == 1) lds_barrier();
            const int c = chunk_of(it);
            const int64_t block = w.block(p, c);
            const char* buf = smem + (it % L::NBUF) * L::bytes;
            const float* gates = reinterpret_cast<const float*>(buf + L::G);
            auto gate = [&](int which, int t) { return *reinterpret_cast<const f32x4*>(gates + which + idx(t, 4 * g4)); };
            store_state(p.dend + block * (int64_t)p.V * K, (int64_t)i * K + 8 * g4, s);
            f32x4 a[4], z[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) a[t] = zero4();
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) {
                const PF<NP> sf = pf_acc<NP>(s[2 * ks], s[2 * ks + 1]);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    a[t] = pmma<NP>(a[t], frag_row<U, NX>(buf + L::Kr, L::XB, idx(t, r16), ks, lane), sf);
            }
            f32x4 d[4];
            pass_get(pass(it) + L::ST, lane, d);
#pragma unroll
            for (int t = 0; t < 4; ++t) a[t] = gate(kGateToEnd, t) * a[t] + d[t];
            const PF<NP> uf[2] = {pf_acc<NP>(a[0], a[1]), pf_acc<NP>(a[2], a[3])};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                z[t] = zero4();
#pragma unroll
                for (int ks = (t >> 1); ks < 2; ++ks) z[t] = pmma<NP>(z[t], tri_col<NP>(buf + L::T, t, ks, lane), uf[ks]);
            }
            store_tokens(p.z + block * (int64_t)C * p.V, i, g4, z);
            f32x4 g[KT];
            pass_get(pass(it), lane, g);
            const float eGC = gates[kGateEG + C - 1];
#pragma unroll
            for (int t = 0; t < KT; ++t) s[t] = eGC * s[t] + g[t];
            const Rsrc r = chunk_rsrc(dv, p, w, c);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                z[t] = gate(kGateBeta, t) * z[t];
#pragma unroll
                for (int q = 0; q < 4; ++q) bput(dv, r, off[4 * t + q], z[t][q]);
                z[t] = -gate(kGateEG, t) * z[t];
            }
            const PF<NP> zf[2] = {pf_acc<NP>(z[0], z[1]), pf_acc<NP>(z[2], z[3])};
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int t = 0; t < KT; ++t)
                    s[t] = pmma<NP>(s[t], frag_col<U, NX>(buf + L::Kr, L::XB, t, ks, lane), zf[ks]);
            lds_barrier();
        }
        if (p.dh0) store_state(p.dh0, soff, s);
        return;
    }

    // ---- helper wave: chunk it + 1 in iteration it
    const InT* dout = static_cast<const InT*>(p.dout);
    InT xn[16];
    PF<NP> mf[6];                                         // tiles 0, 1 (steps 0, 1), 2, 3 (step 1)
    f32x4 eg[4];
    auto load = [&](int it) {
        const int c = chunk_of(it);
        const Rsrc r = chunk_rsrc(dout, p, w, c);
#pragma unroll
        for (int e = 0; e < 16; ++e) xn[e] = bload(dout, r, off[e]);
        if (c < 0) return;
        const int64_t block = w.block(p, c);
        const char* m = p.ops + block * kOpsBytes + NP * kTriBytes + 16 * lane;
#pragma unroll
        for (int t = 0; t < 4; ++t)
            eg[t] = *reinterpret_cast<const f32x4*>(p.gates + block * kGateFloats + kGateEG + idx(t, 4 * g4));
#pragma unroll
        for (int f = 0; f < 6; ++f)
#pragma unroll
            for (int j = 0; j < NP; ++j) mf[f].p[j] = *reinterpret_cast<const bf16x8*>(m + j * kTriBytes + f * 1024);
    };
    auto work = [&](int it) {
        const char* q = smem + L::Q0 + (it % L::NQ) * L::QB;
        f32x4 x[4], d[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) x[t][e] = p.scale * widen(xn[4 * t + e]);
        // scale M^T DO: DO is exact in one plane for bf16 inputs, the scale is applied after
        f32x4 y[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int e = 0; e < 4; ++e) y[t][e] = widen(xn[4 * t + e]);
        const PF<NX> df[2] = {pf_acc<NX>(y[0], y[1]), pf_acc<NX>(y[2], y[3])};
#pragma unroll
        for (int t = 0; t < 4; ++t) {
            d[t] = zero4();
#pragma unroll
            for (int ks = (t >> 1); ks < 2; ++ks) d[t] = pmma<NP>(d[t], mf[t < 2 ? 2 * t + ks : t + 2], df[ks]);
            d[t] = p.scale * d[t];
            x[t] = eg[t] * x[t];
        }
        load(it + 1);
        pass_put(pass(it) + L::ST, lane, d);
        // Q^T (scale e^G DO)
        const PF<NP> xf[2] = {pf_acc<NP>(x[0], x[1]), pf_acc<NP>(x[2], x[3])};
        f32x4 g[KT];
#pragma unroll
        for (int t = 0; t < KT; ++t) {
            g[t] = zero4();
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) g[t] = pmma<NP>(g[t], frag_col<U, NX>(q, L::XB, t, ks, lane), xf[ks]);
        }
        pass_put(pass(it), lane, g);
    };
    load(0);
    lds_barrier();
    if (w.nc > 0) work(0);
    lds_barrier();
    for (int it = 0; it < w.nc; ++it) {
        if constexpr (L::NBUF == 1) lds_barrier();
        if (it + 1 < w.nc) work(it + 1);
        lds_barrier();
    }
}

template <typename InT, int NX, int K, int NCW, int NMW, bool BWD>
hipError_t launch_typed(const Args& a, hipStream_t s) {
    constexpr int lds = Plan<NX, K, NCW, BWD>::total;
    auto kern = [] {
        if constexpr (BWD) return bwd_kernel<InT, NX, K, NCW, NMW>;
        else return fwd_kernel<InT, NX, K, NCW, NMW>;
    }();
    static wkv7::PerDeviceOnce once;
    const hipError_t e = wkv7::set_smem_once(once, kern, lds);
    if (e != hipSuccess) return e;
    const int nsub = a.V / (16 * NCW);
    hipLaunchKernelGGL(kern, dim3((uint32_t)a.N * a.H * nsub), dim3(64 * (2 * NCW + NMW)), lds, s, a, nsub);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_fwd_scan(const Args& a, bool bf16, hipStream_t s) {
    if (bf16)
        return a.K == 64 ? launch_typed<uint16_t, 1, 64, 2, 2, false>(a, s) : launch_typed<uint16_t, 1, 128, 2, 2, false>(a, s);
    return a.K == 64 ? launch_typed<float, 3, 64, 1, 2, false>(a, s) : launch_typed<float, 3, 128, 1, 2, false>(a, s);
}
hipError_t launch_bwd_scan(const Args& a, bool bf16, hipStream_t s) {
    if (bf16)
        return a.K == 64 ? launch_typed<uint16_t, 1, 64, 2, 2, true>(a, s) : launch_typed<uint16_t, 1, 128, 2, 2, true>(a, s);
    return a.K == 64 ? launch_typed<float, 3, 64, 1, 2, true>(a, s) : launch_typed<float, 3, 128, 1, 2, true>(a, s);
}

}  // namespace gdr
