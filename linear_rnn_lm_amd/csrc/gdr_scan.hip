// gdr_scan.hip -- the state of the gated delta rule, and its gradient, carried
// from chunk to chunk (gfx950).
//
// The chunks of a head are a chain, so what counts is how long one chunk takes.
// A state wave holds 16 rows i of S (or of its gradient) for all K columns in
// its accumulators, as K / 16 tiles of S^T, and shares nothing with the other
// state waves: every product of the chain has the form (operand from LDS) x
// (that wave's registers).  What the chain does not wait for is done by other
// waves: in the forward four output waves, one tile of 16 tokens each, one chunk
// behind (M, o, the stores for the backward); in the backward a helper beside
// each state wave, one chunk ahead (the parts of dU and of the state gradient
// that come from dout alone).  They pass fp32 tiles through LDS, in accumulator
// order.  Of two memory waves one copies the next chunks' K, v and gates into
// LDS, the other splits their T into planes there.  One barrier per chunk.
//
// What bounds it.  With few heads the chain: one chunk of 64 tokens takes 4700 cycles at K = V =
// 128 (B1 T32768 H32: 1.15 ms a call, 0.14 of them preparation, 512 chunks; the state wave's MFMAs
// and the VALU work between them, measured alone, took seven eighths of that) and about 3.0 us forward, 2.5
// backward at K = V = 64 with two slices (B12 T1024 H6: 48 and 40 us for 16 chunks).  With heads
// enough HBM: at B8 T4096 H32 64 x 64 the training forward moves 1.51 GB (S, U, M and T to and fro)
// in 383 to 411 us, the backward scan 1.51 GB in 376 to 383, 3.7 to 4.0 TB/s.
//
// Memory instructions are issued one wave at a time on a compute unit, 16 and more
// cycles each, and a wave that issues one waits its turn; so token columns
// go through LDS in 16-byte pieces, and the state waves of the forward issue none.
#include "gdr_device.h"
#include "gdr_internal.h"
#include "wkv7_internal.h"

namespace gdr {
namespace {

constexpr int NP = kPlanes;
constexpr int kLds = 160 * 1024;

// LDS plan.  Of one chunk: K rows, T planes and gates, and in the forward the
// workgroup's columns of v.  The backward stages Q rows and dout's columns one chunk
// further ahead.  Then the tiles that waves pass on, double-buffered by chunk parity.
template <typename InT, int NX, int K, int NCW, bool BWD>
struct Plan {
    static constexpr int XB = C * K * 2;                  // one plane of K or Q rows
    static constexpr int RB = NCW * 16 * (int)sizeof(InT), VB = C * RB;   // a token's columns, a chunk's
    static constexpr int Kr = 0, T = Kr + NX * XB, G = T + NP * kTriBytes, V = G + kGateFloats * 4;
    static constexpr int bytes = V + (BWD ? 0 : VB);
    static constexpr int QB = BWD ? NX * XB + VB : 0;
    // what one wave passes on: state tiles (fp32, or all planes of the forward's S for bf16 inputs), token tiles
    static constexpr int ST = BWD || NX > 1 ? K / 16 * 1024 : NP * K / 32 * 1024, UT = 4 * 1024;
    static constexpr int pass = 2 * NCW * (ST + UT), OB = BWD ? 0 : 4 * 16 * RB, rest = 2 * QB + pass + OB;
    static constexpr int NBUF = 3 * bytes + rest <= kLds ? 3 : 2 * bytes + rest <= kLds ? 2 : 1;
    static constexpr int NQ = NBUF > 1 ? 2 : 1;
    static constexpr int Q0 = NBUF * bytes, P0 = Q0 + NQ * QB, O0 = P0 + pass, total = O0 + OB;
    static_assert(total <= kLds, "scan LDS");
};

// A row block of 16 token columns per wave, staged in LDS with RB bytes per token: the wave's
// column in accumulator order (tokens idx(t, 4g + q)), tiles t0 and t0 + 1.
template <int RB>
__device__ __forceinline__ void column_tiles(f32x4 (&x)[4], const char* buf, int cw, int lane, uint16_t, int t0) {
    const char* p = buf + (8 * (lane >> 4) + ((lane & 15) >> 2)) * RB + 32 * cw + 8 * (lane & 3);
#pragma unroll
    for (int t = t0; t < t0 + 2; ++t) {
        const wkv7::i16x4 v = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
            (wkv7::lds_i16x4*)(p + (32 * (t >> 1) + 4 * (t & 1)) * RB));
#pragma unroll
        for (int q = 0; q < 4; ++q) x[t][q] = widen((uint16_t)v[q]);
    }
}
template <int RB>
__device__ __forceinline__ void column_tiles(f32x4 (&x)[4], const char* buf, int cw, int lane, float, int t0) {
    const char* p = buf + 64 * cw + 4 * (lane & 15);
#pragma unroll
    for (int t = t0; t < t0 + 2; ++t)
#pragma unroll
        for (int q = 0; q < 4; ++q) x[t][q] = *reinterpret_cast<const float*>(p + idx(t, 4 * (lane >> 4) + q) * RB);
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

// The packed sequence that is the r-th longest of N <= 64 (r from 0): one sequence per lane, each counts those before it.
__device__ __forceinline__ int longest(const Seqs& s, int r) {
    const int lane = threadIdx.x & 63;
    int64_t tok0;
    int len = -1, slot0;
    if (lane < s.N) seq_span(s, lane, tok0, len, slot0);
    int before = 0;
    for (int k = 0; k < s.N; ++k) {
        const int l = __builtin_amdgcn_readlane(len, k);
        before += l > len || (l == len && k < lane);
    }
    return __ffsll(__ballot(lane < s.N && before == r)) - 1;
}

// The sequence, head and 16-row slice of a workgroup.
struct Where {
    int n, h, hk, sub, len, slot0, nc;
    int64_t tok0;
    __device__ __forceinline__ Where(const Args& p, int nsub) {
        // Workgroups go to the eight XCDs in turn; those that read the same q and k (the slices of the
        // heads of a key head) are put on one, so that its L2 serves all but the first of them.
        const uint32_t group = nsub * (p.H / p.Hk), round = 8 * group, whole = gridDim.x / round * round;
        uint32_t id = blockIdx.x;
        if (id < whole) id = id / round * round + id % 8 * group + id % round / 8;
        sub = id % nsub;
        const int nh = id / nsub;
        h = nh % p.H;
        n = nh / p.H;
        hk = h / (p.H / p.Hk);
        const Seqs seqs{p.cu, p.N, p.T, p.NC};
        // long ones first, so that none starts when the others are done (training of 9 packed sequences, 8200 tokens,
        // 16 heads of 128, 576 workgroups: 513 -> 488 us, 485 -> 468, 506 -> 472 by the lengths); of many workgroups per
        // unit the last is a small part, and the search costs as much (1536 of 12 sequences, forward: 255 -> 247,
        // 265 -> 249, 262 -> 245; 1152 of 9: 229 -> 220, 217 -> 221, 215 -> 216; 2048 of 16: 330 -> 328, 323 -> 325,
        // 321 -> 329; 2944 of 23: 354 -> 363, 360 -> 361, 356 -> 361).  1024: four per unit.
        if (p.cu && p.N > 1 && p.N <= 64 && gridDim.x <= 1024) n = longest(seqs, n);
        seq_span(seqs, n, tok0, len, slot0);
        nc = (len + C - 1) / C;
    }
    __device__ __forceinline__ int64_t block(const Args& p, int c) const { return (int64_t)(slot0 + c) * p.H + h; }
};

// The workgroup's columns of a chunk of a (tokens, H, V) tensor into LDS.
template <typename InT, int RB>
__device__ __forceinline__ void stage_columns(const InT* x, char* buf, const Args& p, const Where& w, int c, int lane) {
    constexpr int UPR = RB / 16, EPU = 16 / (int)sizeof(InT);
    const int len = min(C, w.len - c * C);
    const InT* src = x + ((w.tok0 + (int64_t)c * C) * p.H + w.h) * p.V + w.sub * (RB / (int)sizeof(InT));
#pragma unroll
    for (int pc = 0; pc < C * UPR / 64; ++pc) {
        const int e = pc * 64 + lane;
        dma16(src + (int64_t)min(e / UPR, len - 1) * p.H * p.V + (e % UPR) * EPU, buf + pc * 1024);
    }
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

// A gate's values for a lane's tokens, per tile; of the tile pair t0 only.
__device__ __forceinline__ void read_gate2(f32x4 (&x)[4], const float* gate, int g4, int t0) {
    x[t0] = *reinterpret_cast<const f32x4*>(gate + idx(t0, 4 * g4));
    x[t0 + 1] = *reinterpret_cast<const f32x4*>(gate + idx(t0 + 1, 4 * g4));
}
__device__ __forceinline__ void read_gate(f32x4 (&x)[4], const float* gate, int g4) {
#pragma unroll
    for (int t = 0; t < 4; ++t) x[t] = *reinterpret_cast<const f32x4*>(gate + idx(t, 4 * g4));
}

template <int N>
__device__ __forceinline__ void pass_put(char* p, int lane, const f32x4 (&x)[N]) {
#pragma unroll
    for (int t = 0; t < N; ++t) *reinterpret_cast<f32x4*>(p + t * 1024 + lane * 16) = x[t];
}
// tiles t, t + 1 only
__device__ __forceinline__ void pass_put2(char* p, int lane, const f32x4 (&x)[4], int t) {
    *reinterpret_cast<f32x4*>(p + t * 1024 + lane * 16) = x[t];
    *reinterpret_cast<f32x4*>(p + (t + 1) * 1024 + lane * 16) = x[t + 1];
}
__device__ __forceinline__ void pass_get2(const char* p, int lane, f32x4 (&x)[4], int t) {
    x[t] = *reinterpret_cast<const f32x4*>(p + t * 1024 + lane * 16);
    x[t + 1] = *reinterpret_cast<const f32x4*>(p + (t + 1) * 1024 + lane * 16);
}
template <int N>
__device__ __forceinline__ void pass_get(const char* p, int lane, f32x4 (&x)[N]) {
#pragma unroll
    for (int t = 0; t < N; ++t) x[t] = *reinterpret_cast<const f32x4*>(p + t * 1024 + lane * 16);
}

// The two memory waves.  They work NBUF - 1 chunks ahead of the one in use (none
// ahead, and two barriers per chunk, where a single buffer is all that fits).
template <typename InT, int NX, int K, int NCW, bool BWD>
__device__ __forceinline__ void memory_wave(const Args& p, const Where& w, char* smem, int mw, int lane) {
    using L = Plan<InT, NX, K, NCW, BWD>;
    constexpr int ahead = L::NBUF - 1;
    const int64_t stride = (int64_t)p.Hk * K;
    auto chunk_of = [&](int it) { return BWD ? w.nc - 1 - it : it; };
    auto rows_of = [&](int c) { return (w.tok0 + (int64_t)c * C) * stride + (int64_t)w.hk * K; };
    auto buf = [&](int it) { return smem + (it % L::NBUF) * L::bytes; };
    auto tri = [&](int it) { return p.tri + w.block(p, chunk_of(it)) * p.tri_stride; };
    auto landed = [] { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); };

    if (mw == 1) {
        // T: fp32 pieces of eight values, two chunks ahead in two register sets, into planes
        auto load = [&](f32x4 (&x)[6][2], int it) {
            if (it >= w.nc) return;
            const float* src = tri(it) + 8 * lane;
#pragma unroll
            for (int j = 0; j < 6; ++j) {
                x[j][0] = *reinterpret_cast<const f32x4*>(src + 512 * j);
                x[j][1] = *reinterpret_cast<const f32x4*>(src + 512 * j + 4);
            }
        };
        auto put = [&](f32x4 (&x)[6][2], int it) {
            if (it >= w.nc) return;
#pragma unroll
            for (int j = 0; j < 6; ++j) {
                const int e = 64 * j + lane, blk = e >> 7, row = (e >> 2) & 31, u = e & 3;
                const PF<NP> f = pf_acc<NP>(x[j][0], x[j][1]);
                char* dst = buf(it) + L::T + blk * 2048 + (row * 4 + (u ^ (row >> 3))) * 16;
#pragma unroll
                for (int i = 0; i < NP; ++i) *reinterpret_cast<bf16x8*>(dst + i * kTriBytes) = f.p[i];
            }
            load(x, it + 2);
        };
        f32x4 even[6][2], odd[6][2];                      // chunks of even and odd number
        load(even, 0);
        load(odd, 1);
        if constexpr (ahead > 0) put(even, 0);
        if constexpr (ahead > 1) put(odd, 1);
        lds_barrier();
        if constexpr (BWD) lds_barrier();
        for (int it = 0; it < w.nc; it += 2) {
            if constexpr (ahead == 1) put(odd, it + ahead);
            else put(even, it + ahead);
            lds_barrier();
            if constexpr (L::NBUF == 1) lds_barrier();
            if (it + 1 == w.nc) break;
            if constexpr (ahead == 1) put(even, it + 1 + ahead);
            else put(odd, it + 1 + ahead);
            lds_barrier();
            if constexpr (L::NBUF == 1) lds_barrier();
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
        if constexpr (!BWD) stage_columns<InT, L::RB>(static_cast<const InT*>(p.v), buf(it) + L::V, p, w, c, lane);
    };
    auto fetch_q = [&](int it) {
        if constexpr (BWD) {
            if (it >= w.nc) return;                       // an empty sequence has no chunk 0
            const int c = chunk_of(it);
            char* q = smem + L::Q0 + (it % L::NQ) * L::QB;
            stage_rows<NX, K>(p.qp, q, rows_of(c), stride, min(C, w.len - c * C), lane);
            stage_columns<InT, L::RB>(static_cast<const InT*>(p.dout), q + NX * L::XB, p, w, c, lane);
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
        constexpr int n = NX * C * K * 2 / 1024 + 2 + (BWD ? 0 : L::VB / 1024);
        if (ahead == 2 && it + ahead < w.nc) asm volatile("s_waitcnt vmcnt(%0)" ::"n"(n) : "memory");
        else landed();
        lds_barrier();
    }
}

// ---------------------------------------------------------------------------
// The products of the chain.  One wave has a SIMD's matrix unit nearly to itself, and its
// MFMAs (16 cycles each) and its VALU work (splitting values into planes, gates) take
// about as long; so a chunk is cut into regions, each with the MFMAs of one step
// and the VALU work of the next, dealt out between them by interleave().  LDS operands
// are read a region ahead; fence() keeps the compiler from moving them back to their uses.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }
template <int N, int VALU>
__device__ __forceinline__ void interleave() {
#pragma unroll
    for (int i = 0; i < N; ++i) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);     // one MFMA
        __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);  // then VALU
    }
    fence();
}
// plane products of an input (NX planes) and a derived value
template <int NX>
constexpr int products() { return NX == 1 ? NP : NP * (NP + 1) / 2; }

template <int U, int NX, int KS>
__device__ __forceinline__ void read_rows(PF<NX> (&f)[KS][4], const char* X, int XB, int lane) {
#pragma unroll
    for (int ks = 0; ks < KS; ++ks)
#pragma unroll
        for (int t = 0; t < 4; ++t) f[ks][t] = frag_row<U, NX>(X, XB, idx(t, lane & 15), ks, lane);
}
template <int U, int NX, int KT>
__device__ __forceinline__ void read_cols(PF<NX> (&f)[KT], const char* X, int XB, int ks, int lane) {
#pragma unroll
    for (int t = 0; t < KT; ++t) f[t] = frag_col<U, NX>(X, XB, t, ks, lane);
}
// Fragments of a lower triangular matrix's rows, or of its columns (TR), tile and step as numbered by tri_at.
template <bool TR>
__device__ __forceinline__ constexpr int tri_at(int t, int ks) {
    return TR ? (t < 2 ? 2 * t + ks : t + 2) : (t < 2 ? t : 2 * t - 2 + ks);
}
template <bool TR>
__device__ __forceinline__ void read_tri(PF<NP> (&f)[6], const char* X, int ks, int lane) {
#pragma unroll
    for (int t = 0; t < 4; ++t)
        if (TR ? ks >= (t >> 1) : ks <= (t >> 1)) {
            if constexpr (TR) f[tri_at<TR>(t, ks)] = tri_col<NP>(X, t, ks, lane);
            else f[tri_at<TR>(t, ks)] = tri_row<NP>(X, t, ks, lane);
        }
}

// a[t] += X S^T over 32 columns, tiles T0 .. T0 + N - 1
template <int NX, int T0, int N>
__device__ __forceinline__ void rows_step(f32x4 (&a)[4], const PF<NX> (&f)[4], const PF<NP>& sf) {
#pragma unroll
    for (int o = NP - 1; o >= 0; --o)
#pragma unroll
        for (int i = 0; i < NX; ++i)
            if (o - i >= 0)
#pragma unroll
                for (int t = T0; t < T0 + N; ++t) a[t] = wkv7::mfma_bf16(f[t].p[i], sf.p[o - i], a[t]);
}
// a = X S^T over all columns but the last 32 (whose planes it returns), S split on the way; the
// planes go to `pass` if given
template <int NX, int KS, int KT>
__device__ __forceinline__ PF<NP> rows_times_state(f32x4 (&a)[4], const PF<NX> (&f)[KS][4], const f32x4 (&s)[KT],
                                                   char* pass) {
    PF<NP> sf = pf_acc<NP>(s[0], s[1]);
    auto hand = [&](int ks) {
        if (pass) {
#pragma unroll
            for (int i = 0; i < NP; ++i) *reinterpret_cast<bf16x8*>(pass + (NP * ks + i) * 1024) = sf.p[i];
        }
    };
    hand(0);
#pragma unroll
    for (int t = 0; t < 4; ++t) a[t] = zero4();
#pragma unroll
    for (int ks = 0; ks + 1 < KS; ++ks) {
        fence();
        rows_step<NX, 0, 4>(a, f[ks], sf);
        sf = pf_acc<NP>(s[2 * ks + 2], s[2 * ks + 3]);
        interleave<4 * products<NX>(), 4>();
        hand(ks + 1);
    }
    fence();
    return sf;
}
// u[t] += (triangular) r over 32 tokens
template <bool TR>
__device__ __forceinline__ void tri_step(f32x4 (&u)[4], const PF<NP> (&f)[6], int ks, const PF<NP>& r) {
#pragma unroll
    for (int o = NP - 1; o >= 0; --o)
#pragma unroll
        for (int i = 0; i <= o; ++i)
#pragma unroll
            for (int t = 0; t < 4; ++t)
                if (TR ? ks >= (t >> 1) : ks <= (t >> 1))
                    u[t] = wkv7::mfma_bf16(f[tri_at<TR>(t, ks)].p[i], r.p[o - i], u[t]);
}
// s[t] += X^T r over 32 tokens
template <int NX, int KT>
__device__ __forceinline__ void cols_step(f32x4 (&s)[KT], const PF<NX> (&f)[KT], const PF<NP>& r) {
#pragma unroll
    for (int o = NP - 1; o >= 0; --o)
#pragma unroll
        for (int i = 0; i < NX; ++i)
            if (o - i >= 0)
#pragma unroll
                for (int t = 0; t < KT; ++t) s[t] = wkv7::mfma_bf16(f[t].p[i], r.p[o - i], s[t]);
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

// An output wave of the forward: tokens of tile TT.  In iteration it it finishes chunk it - 1,
//     O = scale (e^G Q S0^T + M U),
// and forms its rows of M = Lam Q K^T of chunk it, as operand fragments that stay in its
// registers.  For the backward it stores its share of U, and its rows of M as
// fragments of M^T, which takes the product a second time, the other way round.
template <typename InT, int NX, int K, int NCW, int TT>
__device__ __forceinline__ void output_wave(const Args& p, const Where& w, char* smem, int lane) {
    using L = Plan<InT, NX, K, NCW, false>;
    constexpr int U = K / 8, KS = K / 32, KT = K / 16, MS = TT / 2 + 1;   // 32-token steps of M's rows
    const int g4 = lane >> 4, r16 = lane & 15, t = idx(TT, r16);
    InT* o = static_cast<InT*>(p.o);
    const bool want = o || p.ckpt;
    char* stage = smem + L::O0 + TT * 16 * L::RB;
    PF<NX> qn[KS], qf[KS];
    PF<NP> mf[MS];
    f32x4 eg = zero4();
    auto load = [&](int c) {
        if (c < w.nc && want) load_row<NX, KS>(qn, p.qp, p, w, c, t, g4);
    };
    load(0);
    lds_barrier();
    for (int it = 0; it <= w.nc; ++it) {
        if constexpr (L::NBUF == 1) {
            if (it < w.nc) lds_barrier();
        }
        if (it > 0 && want) {
            const int c = it - 1;
            const char* pass = smem + L::P0 + (c & 1) * NCW * (L::ST + L::UT);
            float* ck = p.ckpt ? p.ckpt + w.block(p, c) * p.ckpt_stride : nullptr;
            constexpr int TWO = NCW < 2 ? 1 : 2;          // slices at a time
#pragma unroll
            for (int c0 = 0; c0 < NCW; c0 += TWO) {
                // S arrives in planes for bf16 inputs, as fp32 tiles otherwise
                f32x4 s[TWO][NX == 1 ? 1 : KT], u[TWO][4];
                PF<NP> sf[TWO][KS];
#pragma unroll
                for (int cs = 0; cs < TWO; ++cs) {
                    const char* ps = pass + (c0 + cs) * (L::ST + L::UT);
                    if constexpr (NX == 1) {
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                            for (int j = 0; j < NP; ++j)
                                sf[cs][ks].p[j] = *reinterpret_cast<const bf16x8*>(ps + (NP * ks + j) * 1024 + 16 * lane);
                    } else {
                        pass_get(ps, lane, s[cs]);
                    }
                    pass_get(ps + L::ST, lane, u[cs]);
                }
                fence();
#pragma unroll
                for (int cs = 0; cs < TWO; ++cs) {
                    f32x4 b = zero4();
#pragma unroll
                    for (int ks = 0; ks < KS; ++ks) {
                        if constexpr (NX > 1) sf[cs][ks] = pf_acc<NP>(s[cs][2 * ks], s[cs][2 * ks + 1]);
                        b = pmma<NP>(b, qf[ks], sf[cs][ks]);
                    }
                    b = eg * b;
#pragma unroll
                    for (int ks = 0; ks < MS; ++ks) b = pmma<NP>(b, mf[ks], pf_acc<NP>(u[cs][2 * ks], u[cs][2 * ks + 1]));
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        st(reinterpret_cast<InT*>(stage + (4 * g4 + q) * L::RB) + 16 * (c0 + cs) + r16, p.scale * b[q]);
                }
                if (ck) {
#pragma unroll
                    for (int cs = 0; cs < TWO; ++cs) {
                        const int i = 16 * (w.sub * NCW + c0 + cs) + r16;
#pragma unroll
                        for (int ks = 0; ks < KS; ++ks)
                            if (NX > 1 && ((c0 + cs) * KS + ks) % 4 == TT) {
                                float* d = ck + (int64_t)i * K + 8 * g4 + 32 * ks;
                                *reinterpret_cast<f32x4*>(d) = s[cs][NX > 1 ? 2 * ks : 0];
                                *reinterpret_cast<f32x4*>(d + 4) = s[cs][NX > 1 ? 2 * ks + 1 : 0];
                            }
#pragma unroll
                        for (int ks = 0; ks < 2; ++ks)
                            if (((c0 + cs) * 2 + ks) % 4 == 3 - TT) {
                                float* d = ck + (int64_t)p.V * K + (int64_t)i * C + 8 * g4 + 32 * ks;
                                *reinterpret_cast<f32x4*>(d) = u[cs][2 * ks];
                                *reinterpret_cast<f32x4*>(d + 4) = u[cs][2 * ks + 1];
                            }
                    }
                }
            }
            if (o) {
                constexpr int UPR = L::RB / 16, EPU = 16 / (int)sizeof(InT);
                wkv7::wave_lds_sync();
#pragma unroll
                for (int j = 0; j < (16 * UPR + 63) / 64; ++j) {
                    const int e = 64 * j + lane, tt = c * C + idx(TT, e / UPR);
                    if (16 * UPR < 64 && e >= 16 * UPR) continue;
                    const f32x4 v = *reinterpret_cast<const f32x4*>(stage + 16 * e);
                    if (tt < w.len)
                        *reinterpret_cast<f32x4*>(o + ((w.tok0 + tt) * p.H + w.h) * p.V + w.sub * NCW * 16 + (e % UPR) * EPU) = v;
                }
            }
        }
        if (it < w.nc) {
            if (want) {
                const char* buf = smem + (it % L::NBUF) * L::bytes;
                const float* gates = reinterpret_cast<const float*>(buf + L::G);
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) qf[ks] = qn[ks];
                load(it + 1);
                eg = *reinterpret_cast<const f32x4*>(gates + kGateEG + idx(TT, 4 * g4));
                const float nt = gates[kGateN + t], ft = gates[kGateF + t];
                PF<NX> kf[2 * MS][KS];
                for (int k = 0; k < KS; ++k) {
#pragma unroll
                    for (int ts = 0; ts < 2 * MS; ++ts)
                        if (NX == 1) kf[ts][k] = frag_row<U, NX>(buf + L::Kr, L::XB, idx(ts, r16), k, lane);
                }
                fence();
                // three planes of them would not fit the registers: those are read at their use
                auto kfrag = [&](int ts, int k) {
                    if constexpr (NX == 1) return kf[ts][k];
                    else return frag_row<U, NX>(buf + L::Kr, L::XB, idx(ts, r16), k, lane);
                };
                f32x4 x[2 * MS];                          // rows s of tile ts, column t
#pragma unroll
                for (int ts = 0; ts < 2 * MS; ++ts) {
                    x[ts] = zero4();
#pragma unroll
                    for (int k = 0; k < KS; ++k) x[ts] = pmma<NP>(x[ts], kfrag(ts, k), qf[k]);
                }
#pragma unroll
                for (int ts = 0; ts < 2 * MS; ++ts) {
                    const int s0 = 32 * (ts >> 1) + 8 * g4 + 4 * (ts & 1);
                    const f32x4 ns = *reinterpret_cast<const f32x4*>(gates + kGateN + s0);
                    const f32x4 fs = *reinterpret_cast<const f32x4*>(gates + kGateF + s0);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        x[ts][q] *= decay(nt, ft, ns[q], fs[q]);
                        if (ts / 2 == TT / 2 && s0 + q > t) x[ts][q] = 0.f;   // other tiles lie below the diagonal
                    }
                }
#pragma unroll
                for (int m = 0; m < MS; ++m) mf[m] = pf_acc<NP>(x[2 * m], x[2 * m + 1]);
                if (p.ckpt && w.sub == 0) {
                    // piece (tile ts of s, 32 tokens): this wave's half of each lane's eight tokens
                    float* mt = p.ckpt + w.block(p, it) * p.ckpt_stride + (int64_t)p.V * (K + C) + 4 * (TT & 1);
                    const f32x4 nq = *reinterpret_cast<const f32x4*>(gates + kGateN + idx(TT, 4 * g4));
                    const f32x4 fq = *reinterpret_cast<const f32x4*>(gates + kGateF + idx(TT, 4 * g4));
#pragma unroll
                    for (int ts = 0; ts < 2 * MS; ++ts) {
                        f32x4 y = zero4();                // rows t, column s
                        const int s = idx(ts, r16);
#pragma unroll
                        for (int k = 0; k < KS; ++k) y = pmma<NP>(y, qf[k], kfrag(ts, k));
                        const float ns = gates[kGateN + s], fs = gates[kGateF + s];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            y[q] *= decay(nq[q], fq[q], ns, fs);
                            if (ts / 2 == TT / 2 && s > idx(TT, 4 * g4) + q) y[q] = 0.f;
                        }
                        *reinterpret_cast<f32x4*>(mt + (64 * tri_at<true>(ts, TT / 2) + lane) * 8) = y;
                    }
                }
            }
            lds_barrier();
        }
    }
}

// v -> o, hT and what the backward needs (ckpt).
template <typename InT, int NX, int K, int NCW>
__global__ __launch_bounds__(64 * (NCW + 6)) void fwd_kernel(Args p, int nsub) {
    using L = Plan<InT, NX, K, NCW, false>;
    constexpr int U = K / 8, KS = K / 32, KT = K / 16;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g4 = lane >> 4, r16 = lane & 15;
    const Where w(p, nsub);
    // Waves are dealt to the four SIMDs in turn: with two state waves, those share theirs with the memory
    // waves, and the heavier output waves (more rows of M) with the lighter ones.
    switch (wave - NCW) {
        case 0: output_wave<InT, NX, K, NCW, 3>(p, w, smem, lane); return;
        case 1: output_wave<InT, NX, K, NCW, 2>(p, w, smem, lane); return;
        case 2: memory_wave<InT, NX, K, NCW, false>(p, w, smem, 1, lane); return;
        case 3: memory_wave<InT, NX, K, NCW, false>(p, w, smem, 0, lane); return;
        case 4: output_wave<InT, NX, K, NCW, 0>(p, w, smem, lane); return;
        case 5: output_wave<InT, NX, K, NCW, 1>(p, w, smem, lane); return;
        default: break;
    }
    const int i = 16 * (w.sub * NCW + wave) + r16;        // this lane's state row
    auto pass = [&](int it) { return smem + L::P0 + ((it & 1) * NCW + wave) * (L::ST + L::UT); };
    const int64_t soff = (((int64_t)w.n * p.H + w.h) * p.V + i) * K + 8 * g4;
    f32x4 s[KT];                                          // s[2c + hh][q] = S[i][32c + 8g + 4hh + q]
    load_state(s, p.h0, soff);
    __builtin_amdgcn_s_setprio(3);                        // the chain goes first on its SIMD
    lds_barrier();
    for (int it = 0; it < w.nc; ++it) {
        if constexpr (L::NBUF == 1) lds_barrier();
        const char* buf = smem + (it % L::NBUF) * L::bytes;
        const float* gates = reinterpret_cast<const float*>(buf + L::G);
        f32x4 bt[4], eg[4], te[4], a[4], u[4], v[4];
        PF<NX> kf[KS][4];
        read_rows<U, NX, KS>(kf, buf + L::Kr, L::XB, lane);
        const float eGC = gates[kGateEG + C - 1];
        fence();
        // a = K S^T
        char* hand = nullptr;
        if constexpr (NX == 1) {
            hand = pass(it) + 16 * lane;
            if (p.ckpt) store_state(p.ckpt + w.block(p, it) * p.ckpt_stride, (int64_t)i * K + 8 * g4, s);
        } else {
            pass_put(pass(it), lane, s);
        }
        const PF<NP> sl = rows_times_state<NX, KS, KT>(a, kf, s, hand);
        column_tiles<L::RB>(v, buf + L::V, wave, lane, InT(), 0);
        read_gate2(bt, gates + kGateBeta, g4, 0);
        read_gate2(eg, gates + kGateEG, g4, 0);
        PF<NP> tf[6];
        read_tri<false>(tf, buf + L::T, 0, lane);
        fence();
        rows_step<NX, 0, 2>(a, kf[KS - 1], sl);
        fence();
        // the last of a; b R = b (V - e^G a) of the first 32 tokens
        rows_step<NX, 2, 2>(a, kf[KS - 1], sl);
#pragma unroll
        for (int t = 0; t < 2; ++t) a[t] = bt[t] * (v[t] - eg[t] * a[t]);
        const PF<NP> r0 = pf_acc<NP>(a[0], a[1]);
        interleave<2 * products<NX>(), 12>();
        // U = T (b R): what the first 32 tokens add; b R of the others; e^(G_C) S
        column_tiles<L::RB>(v, buf + L::V, wave, lane, InT(), 2);
        read_gate2(bt, gates + kGateBeta, g4, 2);
        read_gate2(eg, gates + kGateEG, g4, 2);
        fence();
#pragma unroll
        for (int t = 0; t < 4; ++t) u[t] = zero4();
        tri_step<false>(u, tf, 0, r0);
#pragma unroll
        for (int t = 2; t < 4; ++t) a[t] = bt[t] * (v[t] - eg[t] * a[t]);
        const PF<NP> r1 = pf_acc<NP>(a[2], a[3]);
#pragma unroll
        for (int t = 0; t < KT; ++t) s[t] = eGC * s[t];
        interleave<24, 4>();
        // the rest of U; e^(G_C - G) U of the first 32 tokens
        PF<NX> kc[KT], kd[KT];
        read_tri<false>(tf, buf + L::T, 1, lane);
        read_gate(te, gates + kGateToEnd, g4);
        read_cols<U, NX, KT>(kc, buf + L::Kr, L::XB, 0, lane);
        fence();
        tri_step<false>(u, tf, 1, r1);
        pass_put2(pass(it) + L::ST, lane, u, 0);
        const PF<NP> e0 = pf_acc<NP>(te[0] * u[0], te[1] * u[1]);
        interleave<12, 4>();
        // S1^T = e^(G_C) S0^T + K^T (e^(G_C - G) U)
        read_cols<U, NX, KT>(kd, buf + L::Kr, L::XB, 1, lane);
        fence();
        cols_step<NX, KT>(s, kc, e0);
        pass_put2(pass(it) + L::ST, lane, u, 2);
        const PF<NP> e1 = pf_acc<NP>(te[2] * u[2], te[3] * u[3]);
        interleave<KT * products<NX>(), 3>();
        cols_step<NX, KT>(s, kd, e1);
        lds_barrier();
    }
    if (p.hT) store_state(p.hT, soff, s);
}

// dout -> dv, the state gradients at the chunks' ends (dend), Z, dh0.
//   dU = scale M^T DO + e^(G_C - G) K G1^T      (G1: gradient at the chunk's end)
//   Z  = T^T dU,   dv = b Z
//   G0 = e^(G_C) G1 + scale DO^T e^G Q - (b Z)^T e^G K
template <typename InT, int NX, int K, int NCW>
__global__ __launch_bounds__(64 * (2 * NCW + 2)) void bwd_kernel(Args p, int nsub) {
    using L = Plan<InT, NX, K, NCW, true>;
    constexpr int U = K / 8, KS = K / 32, KT = K / 16;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g4 = lane >> 4, r16 = lane & 15;
    const Where w(p, nsub);
    if (wave >= 2 * NCW) {
        memory_wave<InT, NX, K, NCW, true>(p, w, smem, wave - 2 * NCW, lane);
        return;
    }
    const int cw = wave % NCW, i = 16 * (w.sub * NCW + cw) + r16;
    auto chunk_of = [&](int it) { return w.nc - 1 - it; };
    auto pass = [&](int it) { return smem + L::P0 + ((it & 1) * NCW + cw) * (L::ST + L::UT); };
    const int64_t soff = (((int64_t)w.n * p.H + w.h) * p.V + i) * K + 8 * g4;

    if (wave < NCW) {
        // ---- state wave
        f32x4 s[KT];
        load_state(s, p.dhT, soff);
        __builtin_amdgcn_s_setprio(3);                    // the chain goes first on its SIMD
        InT* dv = static_cast<InT*>(p.dv);
        const int lane0 = lane, i0 = i;
        lds_barrier();
        lds_barrier();
        for (int it = 0; it < w.nc; ++it) {
            // opaque in every chunk, or the LDS addresses, all functions of these, stay in registers
            int lane = lane0, i = i0;
            asm volatile("" : "+v"(lane), "+v"(i));
            const int g4 = lane >> 4, r16 = lane & 15;
            if constexpr (L::NBUF == 1) lds_barrier();
            const int c = chunk_of(it);
            const int64_t block = w.block(p, c);
            const char* buf = smem + (it % L::NBUF) * L::bytes;
            const float* gates = reinterpret_cast<const float*>(buf + L::G);
            f32x4 bt[4], eg[4], te[4], a[4], d[4], z[4], g[KT];
            PF<NX> kf[KS][4];
            read_rows<U, NX, KS>(kf, buf + L::Kr, L::XB, lane);
            const float eGC = gates[kGateEG + C - 1];
            fence();
            // a = K G1^T
            store_state(p.dend + block * (int64_t)p.V * K, (int64_t)i * K + 8 * g4, s);
            const PF<NP> sl = rows_times_state<NX, KS, KT>(a, kf, s, nullptr);
            read_gate2(te, gates + kGateToEnd, g4, 2);
            pass_get2(pass(it) + L::ST, lane, d, 2);      // scale M^T DO
            PF<NP> tf[6];
            read_tri<true>(tf, buf + L::T, 1, lane);
            fence();
            rows_step<NX, 2, 2>(a, kf[KS - 1], sl);
            fence();
            // the last of a; dU = e^(G_C - G) a + scale M^T DO of the last 32 tokens
            rows_step<NX, 0, 2>(a, kf[KS - 1], sl);
            const PF<NP> u1 = pf_acc<NP>(te[2] * a[2] + d[2], te[3] * a[3] + d[3]);
            interleave<2 * products<NX>(), 10>();
            // Z = T^T dU: what the last 32 tokens add; dU of the others; e^(G_C) G1 and dout's part
            read_gate2(te, gates + kGateToEnd, g4, 0);
            pass_get2(pass(it) + L::ST, lane, d, 0);
            pass_get(pass(it), lane, g);
            fence();
#pragma unroll
            for (int t = 0; t < 4; ++t) z[t] = zero4();
            tri_step<true>(z, tf, 1, u1);
            const PF<NP> u0 = pf_acc<NP>(te[0] * a[0] + d[0], te[1] * a[1] + d[1]);
#pragma unroll
            for (int t = 0; t < KT; ++t) s[t] = eGC * s[t] + g[t];
            interleave<24, 4>();
            // the rest of Z; dv = b Z and -e^G dv of the last 32 tokens
            read_tri<true>(tf, buf + L::T, 0, lane);
            read_gate2(bt, gates + kGateBeta, g4, 2);
            read_gate2(eg, gates + kGateEG, g4, 2);
            PF<NX> kc[KT], kd[KT];
            read_cols<U, NX, KT>(kd, buf + L::Kr, L::XB, 1, lane);
            fence();
            // dv: through the tiles just read, whose next writer comes after the barrier, to 16-byte pieces
            char* stage = pass(it) + L::ST;
            constexpr int SB = 16 * (int)sizeof(InT);     // a token's 16 columns
            f32x4 e[4];
            auto finish = [&](int t) {
                const f32x4 x = bt[t] * z[t];
#pragma unroll
                for (int q = 0; q < 4; ++q) st(reinterpret_cast<InT*>(stage + idx(t, 4 * g4 + q) * SB) + r16, x[q]);
                e[t] = -eg[t] * x;
            };
            tri_step<true>(z, tf, 0, u0);
            finish(2);
            finish(3);
            const PF<NP> z1 = pf_acc<NP>(e[2], e[3]);
            interleave<12, 6>();
            // G0^T = e^(G_C) G1^T + ... - K^T (e^G dv)
            read_gate2(bt, gates + kGateBeta, g4, 0);
            read_gate2(eg, gates + kGateEG, g4, 0);
            read_cols<U, NX, KT>(kc, buf + L::Kr, L::XB, 0, lane);
            fence();
            cols_step<NX, KT>(s, kd, z1);
            finish(0);
            finish(1);
            const PF<NP> z0 = pf_acc<NP>(e[0], e[1]);
            interleave<KT * products<NX>(), 4>();
            cols_step<NX, KT>(s, kc, z0);
            store_tokens(p.z + block * (int64_t)C * p.V, i, g4, z);
            wkv7::wave_lds_sync();
#pragma unroll
            for (int j = 0; j < C * SB / 1024; ++j) {
                const int n = 64 * j + lane, tt = c * C + n / (SB / 16);
                const f32x4 x = *reinterpret_cast<const f32x4*>(stage + 16 * n);
                if (tt < w.len)
                    *reinterpret_cast<f32x4*>(dv + ((w.tok0 + tt) * p.H + w.h) * p.V + 16 * (w.sub * NCW + cw) +
                                              (n % (SB / 16)) * (16 / (int)sizeof(InT))) = x;
            }
            lds_barrier();
        }
        if (p.dh0) store_state(p.dh0, soff, s);
        return;
    }

    // ---- helper wave: chunk it + 1 in iteration it
    f32x4 mt[6][2];                                       // M^T: tiles 0, 1 (steps 0, 1), 2, 3 (step 1)
    f32x4 eg[4];
    auto load = [&](int it) {
        const int c = chunk_of(it);
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
        const int c = chunk_of(it);
        // two workgroups of the gradient kernel add to dg where K = 128
        if (K == 128 && w.sub == 0 && cw == 0 && c * C + lane < w.len) p.dg[(w.tok0 + c * C + lane) * p.H + w.h] = 0.f;
        f32x4 x[4], y[4], d[4];
        column_tiles<L::RB>(y, q + NX * L::XB, cw, lane, InT(), 0);
        column_tiles<L::RB>(y, q + NX * L::XB, cw, lane, InT(), 2);
        if (w.len - c * C < C) {                          // tokens past the end repeat the last one there
#pragma unroll
            for (int t = 0; t < 4; ++t)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (c * C + idx(t, 4 * g4 + e) >= w.len) y[t][e] = 0.f;
        }
        // scale M^T DO: DO is exact in one plane for bf16 inputs, the scale is applied after
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
            x[t] = p.scale * eg[t] * y[t];
        }
        load(it + 1);
        PF<NX> qc[KT];
        read_cols<U, NX, KT>(qc, q, L::XB, 0, lane);
        pass_put(pass(it) + L::ST, lane, d);
        // Q^T (scale e^G DO)
        const PF<NP> xf[2] = {pf_acc<NP>(x[0], x[1]), pf_acc<NP>(x[2], x[3])};
        f32x4 g[KT];
#pragma unroll
        for (int t = 0; t < KT; ++t) g[t] = zero4();
        cols_step<NX, KT>(g, qc, xf[0]);
        read_cols<U, NX, KT>(qc, q, L::XB, 1, lane);
        cols_step<NX, KT>(g, qc, xf[1]);
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
    constexpr int lds = Plan<InT, NX, K, NCW, BWD>::total;
    auto kern = [] {
        if constexpr (BWD) return bwd_kernel<InT, NX, K, NCW>;
        else return fwd_kernel<InT, NX, K, NCW>;
    }();
    static wkv7::PerDeviceOnce once;
    const hipError_t e = wkv7::set_smem_once(once, kern, lds);
    if (e != hipSuccess) return e;
    const int nsub = a.V / (16 * NCW);
    hipLaunchKernelGGL(kern, dim3((uint32_t)a.N * a.H * nsub), dim3(64 * (BWD ? 2 * NCW + 2 : NCW + 6)), lds, s, a, nsub);
    return hipGetLastError();
}

template <bool BWD>
hipError_t launch_scan(const Args& a, bool bf16, hipStream_t s) {
    int n_cu = 0;
    const hipError_t e = wkv7::device_cus(&n_cu);
    if (e != hipSuccess) return e;
    // 16 rows to a workgroup where that leaves none waiting for a compute unit: a unit's issue slots are
    // what bounds a chunk, and with one slice they serve one chain (forward calls of 64 chunks at K = 128, one
    // slice and two: 256 slices 163 and 178 us, 512 slices 311 and 210).  At K = 64 four slices to a workgroup
    // share one copy of K and T in LDS once that leaves every unit one (32 chunks; one, two and four: 256 slices
    // 73, 86, 115 us; 512: 129, 99, 127; 1024: 258, 199, 174; 2048: 548, 405, 347).  Three planes of fp32 inputs
    // leave LDS for one slice.
    const int64_t slices = (int64_t)a.N * a.H * (a.V / 16);
    if (bf16) {
        if (a.K == 128)
            return slices <= n_cu ? launch_typed<uint16_t, 1, 128, 1, BWD>(a, s)
                                  : launch_typed<uint16_t, 1, 128, 2, BWD>(a, s);
        if (slices <= n_cu) return launch_typed<uint16_t, 1, 64, 1, BWD>(a, s);
        return slices >= 4 * n_cu ? launch_typed<uint16_t, 1, 64, 4, BWD>(a, s)
                                  : launch_typed<uint16_t, 1, 64, 2, BWD>(a, s);
    }
    return a.K == 64 ? launch_typed<float, 3, 64, 1, BWD>(a, s) : launch_typed<float, 3, 128, 1, BWD>(a, s);
}

}  // namespace

hipError_t launch_fwd_scan(const Args& a, bool bf16, hipStream_t s) { return launch_scan<false>(a, bf16, s); }
hipError_t launch_bwd_scan(const Args& a, bool bf16, hipStream_t s) { return launch_scan<true>(a, bf16, s); }

}  // namespace gdr
