// gdr_scan.hip -- the state of the gated delta rule, and its gradient, carried
// from chunk to chunk (gfx950).
//
// One compute wave holds 16 rows i of S (or of the state's gradient) for all K
// columns in its accumulators, as K / 16 tiles of S^T, and shares nothing
// with other waves: every product of a chunk has the form (operand from LDS)
// x (that wave's registers), so a chunk needs one barrier, for the staging only.
// Memory waves copy the next chunk's K, Q, T, M and gates into the other LDS
// buffer while the compute waves work.
#include "gdr_device.h"
#include "gdr_internal.h"
#include "wkv7_internal.h"

namespace gdr {
namespace {

constexpr int NP = kPlanes;

// LDS buffer of one chunk.
template <int NX, int K>
struct Buf {
    static constexpr int XB = C * K * 2;                  // one plane of K or Q rows
    static constexpr int Kr = 0, Qr = Kr + NX * XB, T = Qr + NX * XB, M = T + NP * kTriBytes;
    static constexpr int G = M + NP * kTriBytes;          // e^G, e^(G_C - G), b, unused
    static constexpr int bytes = G + 1024;
    static constexpr int NBUF = 2 * bytes <= 160 * 1024 ? 2 : 1;
};

// The memory waves' copy of one chunk: 1 KiB pieces dealt to the waves in turn.
template <int NX, int K, int NMW>
__device__ __forceinline__ void stage(const Args& p, char* buf, int64_t tok, int len, int64_t block, int hk, int mw,
                                      int lane) {
    using B = Buf<NX, K>;
    constexpr int U = K / 8, RPP = 64 / U;                // units per row, rows per piece
    const int64_t stride = (int64_t)p.Hk * K;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
        const Planes x = m ? p.qp : p.kp;
        const uint16_t* src = x.p + tok * stride + (int64_t)hk * K;
#pragma unroll
        for (int i = 0; i < NX; ++i)
#pragma unroll
            for (int u = 0; u < C / RPP / NMW; ++u) {
                const int pc = u * NMW + mw, row = pc * RPP + lane / U, slot = lane % U;
                dma16(src + i * x.plane + min(row, len - 1) * stride + 8 * (slot ^ swz<U>(row)),
                      buf + (m ? B::Qr : B::Kr) + i * B::XB + pc * 1024);
            }
    }
    const char* ops = p.ops + block * kOpsBytes;          // as the LDS holds it
#pragma unroll
    for (int u = 0; u < kOpsBytes / 1024 / NMW; ++u)
        dma16(ops + (u * NMW + mw) * 1024 + 16 * lane, buf + B::T + (u * NMW + mw) * 1024);
    if (mw == 0) dma16(reinterpret_cast<const char*>(p.gates + block * kGateFloats) + 16 * lane, buf + B::G);
}

// BWD = false: v -> o, states entering the chunks and U (ckpt), hT.
// BWD = true : dout -> dv, the state gradients at the chunks' ends (dend), Z, dh0.
//   dU = scale M^T DO + e^(G_C - G) K G1^T      (G1: gradient at the chunk's end)
//   Z  = T^T dU,   dv = b Z
//   G0 = e^(G_C) G1 + scale DO^T e^G Q - (b Z)^T e^G K
template <typename InT, int NX, int K, int NCW, int NMW, bool BWD>
__global__ __launch_bounds__(64 * (NCW + NMW)) void scan_kernel(Args p, int nsub) {
    using B = Buf<NX, K>;
    constexpr int U = K / 8, KS = K / 32, KT = K / 16;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g4 = lane >> 4, r16 = lane & 15;
    const int sub = blockIdx.x % nsub, nh = blockIdx.x / nsub, h = nh % p.H, n = nh / p.H;
    const int hk = h / (p.H / p.Hk);
    const Seqs seqs{p.cu, p.N, p.T, p.NC};
    int64_t tok0;
    int len, slot0;
    seq_span(seqs, n, tok0, len, slot0);
    const int nc = (len + C - 1) / C;
    auto chunk_of = [&](int it) { return BWD ? nc - 1 - it : it; };
    auto block_of = [&](int c) { return (int64_t)(slot0 + c) * p.H + h; };

    if (wave >= NCW) {
        const int mw = wave - NCW;
        auto fetch = [&](int it) {
            const int c = chunk_of(it);
            stage<NX, K, NMW>(p, smem + (it % B::NBUF) * B::bytes, tok0 + (int64_t)c * C, min(C, len - c * C), block_of(c),
                              hk, mw, lane);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        };
        if (nc > 0) fetch(0);
        lds_barrier();
        for (int it = 0; it < nc; ++it) {
            if constexpr (B::NBUF == 1) lds_barrier();    // the buffer's readers are done
            if (it + 1 < nc) fetch(it + 1);
            lds_barrier();
        }
        return;
    }

    const int i0 = 16 * (sub * NCW + wave), i = i0 + r16;   // this lane's state row
    const int64_t soff = (((int64_t)n * p.H + h) * p.V + i) * K + 8 * g4;
    const float* s0 = BWD ? p.dhT : p.h0;
    // s[2c + hh][q] = S[i][32c + 8g + 4hh + q]
    f32x4 s[KT];
#pragma unroll
    for (int t = 0; t < KT; ++t)
        s[t] = s0 ? *reinterpret_cast<const f32x4*>(s0 + soff + 32 * (t >> 1) + 4 * (t & 1)) : zero4();

    const InT* x = static_cast<const InT*>(BWD ? p.dout : p.v);
    InT* y = static_cast<InT*>(BWD ? p.dv : p.o);
    const int64_t xstride = (int64_t)p.H * p.V, xoff = tok0 * xstride + (int64_t)h * p.V + i;
    // column i of a chunk's v or dout rows, in accumulator order, as stored; rows past the
    // end repeat the last one and are cleared at their use
    auto load_x = [&](InT (&r)[16], int it) {
        const int c = chunk_of(min(it, nc - 1));
#pragma unroll
        for (int e = 0; e < 16; ++e)
            r[e] = x[xoff + min(c * C + idx(e >> 2, 4 * g4 + (e & 3)), len - 1) * xstride];
    };
    InT xr[16];
    if (nc > 0) load_x(xr, 0);
    lds_barrier();
    for (int it = 0; it < nc; ++it) {
        const int c = chunk_of(it);
        const int64_t block = block_of(c);
        const char* buf = smem + (it % B::NBUF) * B::bytes;
        const float* gates = reinterpret_cast<const float*>(buf + B::G);
        InT xn[16];
        load_x(xn, it + 1);
        // the state entering the chunk, or the gradient at its end
        float* keep = BWD ? p.dend : p.ckpt;
        const int64_t kblock = BWD ? (int64_t)p.V * K : (int64_t)p.V * (K + C);
        if (keep) {
#pragma unroll
            for (int t = 0; t < KT; ++t)
                *reinterpret_cast<f32x4*>(keep + block * kblock + (int64_t)i * K + 8 * g4 + 32 * (t >> 1) + 4 * (t & 1)) = s[t];
        }
        // gates of this lane's tokens, per tile
        auto gate = [&](int which, int t) { return *reinterpret_cast<const f32x4*>(gates + which + idx(t, 4 * g4)); };
        f32x4 xa[4];
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) xa[t][q] = c * C + idx(t, 4 * g4 + q) < len ? widen(xr[4 * t + q]) : 0.f;
        const float eGC = gates[kGateEG + C - 1];

        f32x4 a[4], b[4];
#pragma unroll
        for (int t = 0; t < 4; ++t) a[t] = b[t] = zero4();
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            const PF<NP> sf = pf_acc<NP>(s[2 * ks], s[2 * ks + 1]);
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                a[t] = pmma<NP>(a[t], frag_row<U, NX>(buf + B::Kr, B::XB, idx(t, r16), ks, lane), sf);
                if constexpr (!BWD)
                    b[t] = pmma<NP>(b[t], frag_row<U, NX>(buf + B::Qr, B::XB, idx(t, r16), ks, lane), sf);
            }
        }
        if constexpr (!BWD) {
            // a = K S^T, b = Q S^T;  R = V - e^G a;  U = T (beta R)
            f32x4 R[4], u[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) R[t] = gate(kGateBeta, t) * (xa[t] - gate(kGateEG, t) * a[t]);
            const PF<NP> rf[2] = {pf_acc<NP>(R[0], R[1]), pf_acc<NP>(R[2], R[3])};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                u[t] = zero4();
#pragma unroll
                for (int ks = 0; ks <= (t >> 1); ++ks)
                    u[t] = pmma<NP>(u[t], tri_row<NP>(buf + B::T, t, ks, lane), rf[ks]);
            }
            if (keep) {
                float* ku = keep + block * kblock + (int64_t)p.V * K + i;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int q = 0; q < 4; ++q) ku[(int64_t)idx(t, 4 * g4 + q) * p.V] = u[t][q];
            }
            const PF<NP> uf[2] = {pf_acc<NP>(u[0], u[1]), pf_acc<NP>(u[2], u[3])};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                f32x4 o = gate(kGateEG, t) * b[t];
#pragma unroll
                for (int ks = 0; ks <= (t >> 1); ++ks)
                    o = pmma<NP>(o, tri_row<NP>(buf + B::M, t, ks, lane), uf[ks]);
                if (y) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const int tt = c * C + idx(t, 4 * g4 + q);
                        if (tt < len) st(y + xoff + tt * xstride, p.scale * o[q]);
                    }
                }
            }
            // S1^T = e^(G_C) S0^T + K^T (e^(G_C - G) U)
#pragma unroll
            for (int t = 0; t < 4; ++t) u[t] = gate(kGateToEnd, t) * u[t];
            const PF<NP> ue[2] = {pf_acc<NP>(u[0], u[1]), pf_acc<NP>(u[2], u[3])};
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                s[t] = eGC * s[t];
#pragma unroll
                for (int ks = 0; ks < 2; ++ks)
                    s[t] = pmma<NP>(s[t], frag_col<U, NX>(buf + B::Kr, B::XB, t, ks, lane), ue[ks]);
            }
        } else {
            // a = K G1^T;  dU = e^(G_C - G) a + scale M^T DO;  Z = T^T dU
            f32x4 du[4], z[4];
            const PF<NX> df[2] = {pf_acc<NX>(xa[0], xa[1]), pf_acc<NX>(xa[2], xa[3])};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                f32x4 m = zero4();
#pragma unroll
                for (int ks = (t >> 1); ks < 2; ++ks)
                    m = pmma<NP>(m, tri_col<NP>(buf + B::M, t, ks, lane), df[ks]);
                du[t] = gate(kGateToEnd, t) * a[t] + p.scale * m;
            }
            const PF<NP> uf[2] = {pf_acc<NP>(du[0], du[1]), pf_acc<NP>(du[2], du[3])};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                z[t] = zero4();
#pragma unroll
                for (int ks = (t >> 1); ks < 2; ++ks)
                    z[t] = pmma<NP>(z[t], tri_col<NP>(buf + B::T, t, ks, lane), uf[ks]);
            }
            float* kz = p.z + block * (int64_t)C * p.V + i;
            f32x4 zg[4], xg[4];
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                const f32x4 dr = gate(kGateBeta, t) * z[t];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int tl = idx(t, 4 * g4 + q), tt = c * C + tl;
                    kz[(int64_t)tl * p.V] = z[t][q];
                    if (tt < len) st(y + xoff + tt * xstride, dr[q]);
                }
                zg[t] = -gate(kGateEG, t) * dr;
                xg[t] = p.scale * gate(kGateEG, t) * xa[t];
            }
            const PF<NP> zf[2] = {pf_acc<NP>(zg[0], zg[1]), pf_acc<NP>(zg[2], zg[3])};
            const PF<NP> xf[2] = {pf_acc<NP>(xg[0], xg[1]), pf_acc<NP>(xg[2], xg[3])};
#pragma unroll
            for (int t = 0; t < KT; ++t) {
                s[t] = eGC * s[t];
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    s[t] = pmma<NP>(s[t], frag_col<U, NX>(buf + B::Kr, B::XB, t, ks, lane), zf[ks]);
                    s[t] = pmma<NP>(s[t], frag_col<U, NX>(buf + B::Qr, B::XB, t, ks, lane), xf[ks]);
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) xr[e] = xn[e];
        if constexpr (B::NBUF == 1) lds_barrier();
        lds_barrier();
    }
    float* sT = BWD ? p.dh0 : p.hT;
    if (sT) {
#pragma unroll
        for (int t = 0; t < KT; ++t) *reinterpret_cast<f32x4*>(sT + soff + 32 * (t >> 1) + 4 * (t & 1)) = s[t];
    }
}

template <typename InT, int NX, int K, int NCW, int NMW, bool BWD>
hipError_t launch_typed(const Args& a, hipStream_t s) {
    constexpr int lds = Buf<NX, K>::NBUF * Buf<NX, K>::bytes;
    static_assert(lds <= 160 * 1024, "scan LDS");
    auto kern = scan_kernel<InT, NX, K, NCW, NMW, BWD>;
    static wkv7::PerDeviceOnce once;
    const hipError_t e = wkv7::set_smem_once(once, kern, lds);
    if (e != hipSuccess) return e;
    const int nsub = a.V / (16 * NCW);
    hipLaunchKernelGGL(kern, dim3((uint32_t)a.N * a.H * nsub), dim3(64 * (NCW + NMW)), lds, s, a, nsub);
    return hipGetLastError();
}

template <bool BWD>
hipError_t launch_scan(const Args& a, bool bf16, hipStream_t s) {
    if (bf16)
        return a.K == 64 ? launch_typed<uint16_t, 1, 64, 4, 4, BWD>(a, s) : launch_typed<uint16_t, 1, 128, 4, 4, BWD>(a, s);
    return a.K == 64 ? launch_typed<float, 3, 64, 4, 4, BWD>(a, s) : launch_typed<float, 3, 128, 4, 4, BWD>(a, s);
}

}  // namespace

hipError_t launch_fwd_scan(const Args& a, bool bf16, hipStream_t s) { return launch_scan<false>(a, bf16, s); }
hipError_t launch_bwd_scan(const Args& a, bool bf16, hipStream_t s) { return launch_scan<true>(a, bf16, s); }

}  // namespace gdr
