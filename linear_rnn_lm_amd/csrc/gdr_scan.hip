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
// accumulator order.  One wave copies the next chunks' K and gates into LDS, another
// splits their T into planes there; in the forward, two more form M.  One barrier
// per chunk.
#include "gdr_device.h"
#include "gdr_internal.h"
#include "wkv7_internal.h"

namespace gdr {
namespace {

using wkv7::make_rsrc;
using wkv7::Rsrc;

constexpr int NP = kPlanes;
constexpr int kLds = 160 * 1024;

// LDS plan.  One chunk's K rows, T planes and gates; the backward also stages Q
// rows, one chunk further ahead; the forward keeps M^T (NO planes) from one chunk
// to the next; then the tiles that state and helper waves pass on, all of
// these double-buffered by chunk parity.
template <int NX, int K, int NCW, bool BWD>
struct Plan {
    // o leaves in in_dtype: for bf16 two planes (2^-17) in its own products lose nothing
    // beside its rounding; the products of the state keep all three
    static constexpr int NO = NX == 1 ? 2 : NP;
    static constexpr int XB = C * K * 2;                  // one plane of K or Q rows
    static constexpr int Kr = 0, T = Kr + NX * XB, G = T + NP * kTriBytes, bytes = G + kGateFloats * 4;
    static constexpr int QB = BWD ? NX * XB : 0, MB = BWD ? 0 : NO * kTriBytes;
    static constexpr int ST = K / 16 * 1024, UT = 4 * 1024;   // state tiles, token tiles of one wave
    static constexpr int pass = 2 * NCW * (ST + UT), rest = 2 * QB + 2 * MB + pass;
    static constexpr int NBUF = 3 * bytes + rest <= kLds ? 3 : 2 * bytes + rest <= kLds ? 2 : 1;
    static constexpr int NQ = NBUF > 1 ? 2 : 1;
    static constexpr int Q0 = NBUF * bytes, M0 = Q0 + NQ * QB, P0 = M0 + 2 * MB, total = P0 + pass;
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

// Rows of K or Q of one chunk into LDS, in 1 KiB pieces.
template <int NX, int K>
__device__ __forceinline__ void stage_rows(const Planes& x, char* buf, int64_t row0, int64_t stride, int len, int lane) {
    constexpr int U = K / 8, RPP = 64 / U;                // units per row, rows per piece
    const uint16_t* src = x.p + row0;
#pragma unroll
    for (int i = 0; i < NX; ++i)
#pragma unroll
        for (int pc = 0; pc < C / RPP; ++pc) {
            const int row = pc * RPP + lane / U;
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

// A gate's values for a lane's tokens, per tile.
__device__ __forceinline__ void read_gate(f32x4 (&x)[4], const float* gate, int g4) {
#pragma unroll
    for (int t = 0; t < 4; ++t) x[t] = *reinterpret_cast<const f32x4*>(gate + idx(t, 4 * g4));
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

// The two memory waves.  They work NBUF - 1 chunks ahead of the one in use (none
// ahead, and two barriers per chunk, where a single buffer is all that fits).
template <int NX, int K, int NCW, bool BWD>
__device__ __forceinline__ void memory_wave(const Args& p, const Where& w, char* smem, int mw, int lane) {
    using L = Plan<NX, K, NCW, BWD>;
    constexpr int ahead = L::NBUF - 1;
    const int64_t stride = (int64_t)p.Hk * K;
    auto chunk_of = [&](int it) { return BWD ? w.nc - 1 - it : it; };
    auto rows_of = [&](int c) { return (w.tok0 + (int64_t)c * C) * stride + (int64_t)w.hk * K; };
    auto buf = [&](int it) { return smem + (it % L::NBUF) * L::bytes; };
    auto tri = [&](int it) { return p.tri + w.block(p, chunk_of(it)) * p.tri_stride; };
    auto landed = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };

    if (mw == 1) {
        // T: fp32 pieces of eight values, one chunk ahead in registers, into planes
        f32x4 x[6][2];
        auto load = [&](int it) {
            if (it >= w.nc) return;
            const float* src = tri(it) + 8 * lane;
#pragma unroll
            for (int j = 0; j < 6; ++j) {
                x[j][0] = *reinterpret_cast<const f32x4*>(src + 512 * j);
                x[j][1] = *reinterpret_cast<const f32x4*>(src + 512 * j + 4);
            }
        };
        auto put = [&](int it) {
            if (it >= w.nc) return;
#pragma unroll
            for (int j = 0; j < 6; ++j) {
                const int e = 64 * j + lane, blk = e >> 7, row = (e >> 2) & 31, u = e & 3;
                const PF<NP> f = pf_acc<NP>(x[j][0], x[j][1]);
                char* dst = buf(it) + L::T + blk * 2048 + (row * 4 + (u ^ (row >> 3))) * 16;
#pragma unroll
                for (int i = 0; i < NP; ++i) *reinterpret_cast<bf16x8*>(dst + i * kTriBytes) = f.p[i];
            }
            load(it + 1);
        };
        load(0);
        if constexpr (L::NBUF == 1) {
            lds_barrier();
            if constexpr (BWD) lds_barrier();
            for (int it = 0; it < w.nc; ++it) {
                put(it);
                lds_barrier();
                lds_barrier();
            }
        } else {
            for (int it = 0; it < ahead; ++it) put(it);
            lds_barrier();
            if constexpr (BWD) lds_barrier();
            for (int it = 0; it < w.nc; ++it) {
                put(it + ahead);
                lds_barrier();
            }
        }
        return;
    }

    auto fetch = [&](int it) {
        if (it >= w.nc) return;
        const int c = chunk_of(it);
        stage_rows<NX, K>(p.kp, buf(it) + L::Kr, rows_of(c), stride, min(C, w.len - c * C), lane);
        const char* gates = reinterpret_cast<const char*>(tri(it) + kTriFloats) + 16 * lane;
        dma16(gates, buf(it) + L::G);
        if (lane < kGateFloats / 4 - 64) dma16(gates + 1024, buf(it) + L::G + 1024);
    };
    auto fetch_q = [&](int it) {
        if constexpr (BWD) {
            if (it >= w.nc) return;                       // an empty sequence has no chunk 0
            const int c = chunk_of(it);
            stage_rows<NX, K>(p.qp, smem + L::Q0 + (it % L::NQ) * L::QB, rows_of(c), stride, min(C, w.len - c * C), lane);
        }
    };
    if constexpr (L::NBUF == 1) {
        // backward: Q of chunk it + 1 beside K of chunk it
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
    for (int it = 0; it < ahead; ++it) fetch(it);
    fetch_q(0);
    fetch_q(1);
    landed();
    lds_barrier();
    if constexpr (BWD) lds_barrier();                     // the helper's first chunk
    for (int it = 0; it < w.nc; ++it) {
        fetch_q(it + 2);                                  // first: the helper reads it in the next iteration
        fetch(it + ahead);
        // chunk it + 1 was fetched in the iteration before where ahead is 2: only this iteration's
        // chunk may be in flight (loads land in order)
        constexpr int n = NX * C * K * 2 / 1024 + 2;
        if (ahead == 2 && it + ahead < w.nc) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
        else landed();
        lds_barrier();
    }
}

// ---------------------------------------------------------------------------
// The products of the chain, with every LDS operand read a step ahead of its
// use: an MFMA that waits for its own operand loses about 120 cycles, eight
// times its length.  fence() keeps the compiler from moving the reads back to
// their uses; interleave() deals VALU work out between MFMAs, which run 16 cycles each.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }
template <int N, int VALU>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);     // one MFMA
        __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);  // then VALU
    }
}

template <int U, int NX, int KS>
__device__ __forceinline__ void read_rows(PF<NX> (&f)[KS][4], const char* X, int XB, int lane) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int t = 0; t < 4; ++t) f[ks][t] = frag_row<U, NX>(X, XB, idx(t, lane & 15), ks, lane);
}
template <int U, int NX, int KT>
__device__ __forceinline__ void read_cols(PF<NX> (&f)[2][KT], const char* X, int XB, int lane) {
#pragma unroll
    for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int t = 0; t < KT; ++t) f[ks][t] = frag_col<U, NX>(X, XB, t, ks, lane);
}
// Fragments of a lower triangular matrix's rows, or of its columns (TR), tile and step as numbered by tri_at.
template <bool TR>
__device__ __forceinline__ constexpr int tri_at(int t, int ks) {
    return TR ? (t < 2 ? 2 * t + ks : t + 2) : (t < 2 ? t : 2 * t - 2 + ks);
}
template <bool TR>
__device__ __forceinline__ void read_tri(PF<NP> (&f)[6], const char* X, int lane) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
            if (TR ? ks >= (t >> 1) : ks <= (t >> 1)) {
                if constexpr (TR) f[tri_at<TR>(t, ks)] = tri_col<NP>(X, t, ks, lane);
                else f[tri_at<TR>(t, ks)] = tri_row<NP>(X, t, ks, lane);
            }
}

// a[t] = X S^T over all K columns, S split on the way
template <int NX, int KS, int KT>
__device__ __forceinline__ void rows_times_state(f32x4 (&a)[4], const PF<NX> (&f)[KS][4], const f32x4 (&s)[KT]) {
#pragma unroll
    for (int t = 0; t < 4; ++t) a[t] = zero4();
    PF<NP> sf = pf_acc<NP>(s[0], s[1]);
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
        fence();
#pragma unroll
        for (int o = NP - 1; o >= 0; --o)
#pragma unroll
            for (int i = 0; i < NX; ++i)
                if (o - i >= 0)
#pragma unroll
                    for (int t = 0; t < 4; ++t) a[t] = wkv7::mfma_bf16(f[ks][t].p[i], sf.p[o - i], a[t]);
        if (ks + 1 < KS) {
            sf = pf_acc<NP>(s[2 * ks + 2], s[2 * ks + 3]);
            interleave<4 * (NX == 1 ? 3 : 6), 4>();
        }
    }
    fence();
}
// u[t] = (triangular) r
template <bool TR>
__device__ __forceinline__ void tri_times(f32x4 (&u)[4], const PF<NP> (&f)[6], const PF<NP> (&r)[2]) {
#pragma unroll
    for (int t = 0; t < 4; ++t) u[t] = zero4();
#pragma unroll
    for (int o = NP - 1; o >= 0; --o)
#pragma unroll
        for (int i = 0; i <= o; ++i)
#pragma unroll
            for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    if (TR ? ks >= (t >> 1) : ks <= (t >> 1))
                        u[t] = wkv7::mfma_bf16(f[tri_at<TR>(t, ks)].p[i], r[ks].p[o - i], u[t]);
}
// s[t] += X^T r
template <int NX, int KT>
__device__ __forceinline__ void add_cols_times(f32x4 (&s)[KT], const PF<NX> (&f)[2][KT], const PF<NP> (&r)[2]) {
#pragma unroll
    for (int o = NP - 1; o >= 0; --o)
#pragma unroll
        for (int i = 0; i < NX; ++i)
            if (o - i >= 0)
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
#pragma unroll
                    for (int t = 0; t < KT; ++t) s[t] = wkv7::mfma_bf16(f[ks][t].p[i], r[ks].p[o - i], s[t]);
}

// One token row of a chunk of q or k from memory, as operand fragments (a token past the end repeats the last one).
template <int NX, int KS>
__device__ __forceinline__ void load_row(PF<NX> (&f)[KS], const Planes& x, const Args& p, const Where& w, int c, int t,
                                         int g4) {
    const uint16_t* row = x.p + ((w.tok0 + (int64_t)c * C + min(t, w.len - c * C - 1)) * p.Hk + w.hk) * (KS * 32) + 8 * g4;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int j = 0; j < NX; ++j) f[ks].p[j] = *reinterpret_cast<const bf16x8*>(row + j * x.plane + 32 * ks);
}

// The two M waves of the forward: M^T = (Lam Q K^T)^T of chunk it in iteration it, in six
// pieces of one tile of s by 32 tokens t (rows s of eight consecutive t per lane), as
// planes in LDS for the helpers and in fp32 for the backward.  Wave 0 takes pieces
// (0, 0), (1, 0), (0, 1), wave 1 pieces (1, 1), (2, 1), (3, 1) of (tile, 32 tokens).
template <int NX, int K, int NCW, int MW>
__device__ __forceinline__ void m_wave(const Args& p, const Where& w, char* smem, int lane) {
    using L = Plan<NX, K, NCW, false>;
    constexpr int U = K / 8, KS = K / 32, NO = L::NO, T0 = MW == 0 ? 0 : 2;
    const int g4 = lane >> 4, r16 = lane & 15;
    const bool want = p.o || p.ckpt;
    PF<NX> qf[4 - T0][KS];
    auto load = [&](int c) {
        if (c >= w.nc || !want) return;
#pragma unroll
        for (int t = T0; t < 4; ++t) load_row<NX, KS>(qf[t - T0], p.qp, p, w, c, idx(t, r16), g4);
    };
    load(0);
    lds_barrier();
    for (int it = 0; it < w.nc; ++it) {
        if constexpr (L::NBUF == 1) lds_barrier();
        if (want) {
            const char* buf = smem + (it % L::NBUF) * L::bytes;
            const float* gates = reinterpret_cast<const float*>(buf + L::G);
            char* m = smem + L::M0 + (it & 1) * L::MB;
            f32x4 x[3][2];
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                const int ts = MW == 0 ? j & 1 : j + 1, ks = MW == 0 ? j >> 1 : 1;
                x[j][0] = x[j][1] = zero4();
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const PF<NX> kf = frag_row<U, NX>(buf + L::Kr, L::XB, idx(ts, r16), k, lane);
                    x[j][0] = pmma<NP>(x[j][0], qf[2 * ks - T0][k], kf);
                    x[j][1] = pmma<NP>(x[j][1], qf[2 * ks + 1 - T0][k], kf);
                }
            }
            load(it + 1);
#pragma unroll
            for (int j = 0; j < 3; ++j) {
                const int ts = MW == 0 ? j & 1 : j + 1, ks = MW == 0 ? j >> 1 : 1, s = idx(ts, r16);
                const float ns = gates[kGateN + s], fs = gates[kGateF + s];
#pragma unroll
                for (int hh = 0; hh < 2; ++hh) {
                    const int t0 = 32 * ks + 8 * g4 + 4 * hh;
                    const f32x4 nt = *reinterpret_cast<const f32x4*>(gates + kGateN + t0);
                    const f32x4 ft = *reinterpret_cast<const f32x4*>(gates + kGateF + t0);
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        x[j][hh][q] = s <= t0 + q ? x[j][hh][q] * decay(nt[q], ft[q], ns, fs) : 0.f;
                }
                const PF<NO> mf = pf_acc<NO>(x[j][0], x[j][1]);
                const int row = idx(ts & 1, r16);
                char* dst = m + tri_block(ts >> 1, ks) + (row * 4 + (g4 ^ (row >> 3))) * 16;
#pragma unroll
                for (int o = 0; o < NO; ++o) *reinterpret_cast<bf16x8*>(dst + o * kTriBytes) = mf.p[o];
                if (p.ckpt && w.sub == 0) {
                    float* mt = p.ckpt + w.block(p, it) * p.ckpt_stride + (int64_t)p.V * (K + C) +
                                (64 * tri_at<true>(ts, ks) + lane) * 8;
                    *reinterpret_cast<f32x4*>(mt) = x[j][0];
                    *reinterpret_cast<f32x4*>(mt + 4) = x[j][1];
                }
            }
        }
        lds_barrier();
    }
}

// v -> o, hT and what the backward needs (ckpt).
template <typename InT, int NX, int K, int NCW>
__global__ __launch_bounds__(64 * (2 * NCW + 4)) void fwd_kernel(Args p, int nsub) {
    using L = Plan<NX, K, NCW, false>;
    constexpr int U = K / 8, KS = K / 32, KT = K / 16, NO = L::NO;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g4 = lane >> 4, r16 = lane & 15;
    const Where w(p, nsub);
    if (wave >= 2 * NCW) {
        if (wave < 2 * NCW + 2) memory_wave<NX, K, NCW, false>(p, w, smem, wave - 2 * NCW, lane);
        else if (wave == 2 * NCW + 2) m_wave<NX, K, NCW, 0>(p, w, smem, lane);
        else m_wave<NX, K, NCW, 1>(p, w, smem, lane);
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
            f32x4 bt[4], eg[4], te[4], a[4], u[4];
            PF<NX> kf[KS][4];
            read_rows<U, NX, KS>(kf, buf + L::Kr, L::XB, lane);
            read_gate(bt, gates + kGateBeta, g4);
            read_gate(eg, gates + kGateEG, g4);
            const float eGC = gates[kGateEG + C - 1];
            fence();
            // a = K S^T;  R = V - e^G a;  U = T (b R)
            pass_put(pass(it), lane, s);
            rows_times_state<NX, KS, KT>(a, kf, s);
            PF<NP> tf[6];
            read_tri<false>(tf, buf + L::T, lane);
            read_gate(te, gates + kGateToEnd, g4);
            fence();
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) a[t][q] = bt[t][q] * (widen(xn[4 * t + q]) - eg[t][q] * a[t][q]);
            load_v(it + 1);
            const PF<NP> rf[2] = {pf_acc<NP>(a[0], a[1]), pf_acc<NP>(a[2], a[3])};
            fence();
            tri_times<false>(u, tf, rf);
            fence();
            PF<NX> kc[2][KT];
            read_cols<U, NX, KT>(kc, buf + L::Kr, L::XB, lane);
            fence();
            // S1^T = e^(G_C) S0^T + K^T (e^(G_C - G) U)
#pragma unroll
            for (int t = 0; t < KT; ++t) s[t] = eGC * s[t];
            pass_put(pass(it) + L::ST, lane, u);
#pragma unroll
            for (int t = 0; t < 4; ++t) u[t] = te[t] * u[t];
            const PF<NP> ue[2] = {pf_acc<NP>(u[0], u[1]), pf_acc<NP>(u[2], u[3])};
            fence();
            add_cols_times<NX, KT>(s, kc, ue);
            lds_barrier();
        }
        if (p.hT) store_state(p.hT, soff, s);
        return;
    }

    // ---- helper wave: chunk it - 1 in iteration it
    InT* o = static_cast<InT*>(p.o);
    int off[16];
    token_offsets<InT>(off, p, i, g4);
    PF<NX> qf[4][KS];
    f32x4 eg[4];
    auto load = [&](int c) {
        if (c >= w.nc || !o) return;
#pragma unroll
        for (int t = 0; t < 4; ++t) load_row<NX, KS>(qf[t], p.qp, p, w, c, idx(t, r16), g4);
        read_gate(eg, p.tri + w.block(p, c) * p.tri_stride + kTriFloats + kGateEG, g4);
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
                float* ck = p.ckpt + w.block(p, c) * p.ckpt_stride;
                store_state(ck, (int64_t)i * K + 8 * g4, s);
                store_tokens(ck + (int64_t)p.V * K, i, g4, u);
            }
            if (o) {
                // O = scale (e^G Q S0^T + M U)
                const char* m = smem + L::M0 + (c & 1) * L::MB;
                PF<NO> mf[6];
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int ks = 0; ks <= (t >> 1); ++ks) mf[tri_at<false>(t, ks)] = tri_col<NO>(m, t, ks, lane);
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
                for (int t = 0; t < 4; ++t) b[t] = eg[t] * b[t];
                load(it);
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int ks = 0; ks <= (t >> 1); ++ks) b[t] = pmma<NO>(b[t], mf[tri_at<false>(t, ks)], uf[ks]);
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
template <typename InT, int NX, int K, int NCW>
__global__ __launch_bounds__(64 * (2 * NCW + 2)) void bwd_kernel(Args p, int nsub) {
    using L = Plan<NX, K, NCW, true>;
    constexpr int U = K / 8, KS = K / 32, KT = K / 16;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g4 = lane >> 4, r16 = lane & 15;
    const Where w(p, nsub);
    if (wave >= 2 * NCW) {
        memory_wave<NX, K, NCW, true>(p, w, smem, wave - 2 * NCW, lane);
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
            f32x4 bt[4], eg[4], te[4], a[4], z[4];
            PF<NX> kf[KS][4];
            read_rows<U, NX, KS>(kf, buf + L::Kr, L::XB, lane);
            read_gate(te, gates + kGateToEnd, g4);
            pass_get(pass(it) + L::ST, lane, z);          // scale M^T DO
            fence();
            store_state(p.dend + block * (int64_t)p.V * K, (int64_t)i * K + 8 * g4, s);
            rows_times_state<NX, KS, KT>(a, kf, s);
            PF<NP> tf[6];
            read_tri<true>(tf, buf + L::T, lane);
            fence();
#pragma unroll
            for (int t = 0; t < 4; ++t) a[t] = te[t] * a[t] + z[t];
            const PF<NP> uf[2] = {pf_acc<NP>(a[0], a[1]), pf_acc<NP>(a[2], a[3])};
            fence();
            tri_times<true>(z, tf, uf);
            read_gate(bt, gates + kGateBeta, g4);
            read_gate(eg, gates + kGateEG, g4);
            const float eGC = gates[kGateEG + C - 1];
            fence();
            PF<NX> kc[2][KT];
            read_cols<U, NX, KT>(kc, buf + L::Kr, L::XB, lane);
            f32x4 g[KT];
            pass_get(pass(it), lane, g);
            store_tokens(p.z + block * (int64_t)C * p.V, i, g4, z);
            const Rsrc r = chunk_rsrc(dv, p, w, c);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                z[t] = bt[t] * z[t];
#pragma unroll
                for (int q = 0; q < 4; ++q) bput(dv, r, off[4 * t + q], z[t][q]);
                z[t] = -eg[t] * z[t];
            }
            const PF<NP> zf[2] = {pf_acc<NP>(z[0], z[1]), pf_acc<NP>(z[2], z[3])};
#pragma unroll
            for (int t = 0; t < KT; ++t) s[t] = eGC * s[t] + g[t];
            fence();
            add_cols_times<NX, KT>(s, kc, zf);
            lds_barrier();
        }
        if (p.dh0) store_state(p.dh0, soff, s);
        return;
    }

    // ---- helper wave: chunk it + 1 in iteration it
    const InT* dout = static_cast<const InT*>(p.dout);
    InT xn[16];
    f32x4 mt[6][2];                                       // M^T: tiles 0, 1 (steps 0, 1), 2, 3 (step 1)
    f32x4 eg[4];
    auto load = [&](int it) {
        const int c = chunk_of(it);
        const Rsrc r = chunk_rsrc(dout, p, w, c);
#pragma unroll
        for (int e = 0; e < 16; ++e) xn[e] = bload(dout, r, off[e]);
        if (c < 0) return;
        const float* m = p.ckpt + w.block(p, c) * p.ckpt_stride + (int64_t)p.V * (K + C);
        read_gate(eg, m + 2 * kTriFloats + kGateEG, g4);
#pragma unroll
        for (int f = 0; f < 6; ++f) {
            mt[f][0] = *reinterpret_cast<const f32x4*>(m + (64 * f + lane) * 8);
            mt[f][1] = *reinterpret_cast<const f32x4*>(m + (64 * f + lane) * 8 + 4);
        }
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
            for (int ks = (t >> 1); ks < 2; ++ks) {
                const f32x4 (&m)[2] = mt[tri_at<true>(t, ks)];
                d[t] = pmma<NP>(d[t], pf_acc<NP>(m[0], m[1]), df[ks]);
            }
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

template <typename InT, int NX, int K, int NCW, bool BWD>
hipError_t launch_typed(const Args& a, hipStream_t s) {
    constexpr int lds = Plan<NX, K, NCW, BWD>::total;
    auto kern = [] {
        if constexpr (BWD) return bwd_kernel<InT, NX, K, NCW>;
        else return fwd_kernel<InT, NX, K, NCW>;
    }();
    static wkv7::PerDeviceOnce once;
    const hipError_t e = wkv7::set_smem_once(once, kern, lds);
    if (e != hipSuccess) return e;
    const int nsub = a.V / (16 * NCW);
    hipLaunchKernelGGL(kern, dim3((uint32_t)a.N * a.H * nsub), dim3(64 * (2 * NCW + (BWD ? 2 : 4))), lds, s, a, nsub);
    return hipGetLastError();
}

template <bool BWD>
hipError_t launch_scan(const Args& a, bool bf16, hipStream_t s) {
    if (bf16) return a.K == 64 ? launch_typed<uint16_t, 1, 64, 2, BWD>(a, s) : launch_typed<uint16_t, 1, 128, 2, BWD>(a, s);
    return a.K == 64 ? launch_typed<float, 3, 64, 1, BWD>(a, s) : launch_typed<float, 3, 128, 1, BWD>(a, s);
}

}  // namespace

hipError_t launch_fwd_scan(const Args& a, bool bf16, hipStream_t s) { return launch_scan<false>(a, bf16, s); }
hipError_t launch_bwd_scan(const Args& a, bool bf16, hipStream_t s) { return launch_scan<true>(a, bf16, s); }

}  // namespace gdr
