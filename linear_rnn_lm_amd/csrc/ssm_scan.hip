// ssm_scan.hip -- the selective scan over whole sequences, forward (gfx950).
//
// Per channel and state h <- e^(delta A) h + delta x b, y = sum c h: the decay differs
// per channel, state and token, so the scan has no matrix form; it is bound by vector
// instructions (an exponential, which takes four issue slots, and four more per state
// and token).  A wave works on 16 channels (lane % 16) and 4 NS states, NS to a lane
// (lane / 16), which stay in registers from the first token to the last; WN waves share
// the channels of one block, WC of them lie beside each other.  16 tokens at a time: all
// threads load x, dt, z, b, c (the next block's while this one is worked on), put delta,
// delta x, b and c into LDS as fp32, the waves scan, and the threads that loaded z
// finish y.
#include "rows_device.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

using namespace rows;

template <typename InT, int NS, int WN, int WC>
__global__ __launch_bounds__(64 * WN * WC) void fwd_kernel(Args p, int blocks) {
    constexpr int S = 4 * NS * WN, CH = 16 * WC, NT = 64 * WN * WC, TB = kBlock;
    constexpr int LT = TB * CH / NT;             // tokens of its channel that a thread loads
    constexpr int BC = (2 * TB * S + NT - 1) / NT;
    __shared__ float2 s_du[2][TB][CH];           // delta, delta x
    __shared__ float s_bc[2][2][TB][S];
    __shared__ float s_y[WN][TB][CH];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wn = wave % WN, wc = wave / WN;
    const int cb = blockIdx.x % blocks, slot = blockIdx.x / blocks;
    const Seqs seqs{p.cu, p.N, p.T};
    int n, piece, len;
    if (!slot_piece(seqs, slot, p.seg, n, piece)) return;
    int64_t tok0;
    seq_span(seqs, n, tok0, len);
    const int t_begin = piece * p.seg, t_end = min(len, t_begin + p.seg);

    // scanning: channel and first state of this lane
    const int cl = wc * 16 + (lane & 15), g = lane >> 4, ch = cb * CH + cl, n0 = (wn * 4 + g) * NS;
    const bool on = ch < p.C;
    float A2[NS], h[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        A2[s] = on ? kLog2e * p.A[(int64_t)ch * S + n0 + s] : 0.f;
        h[s] = on && p.h0 ? p.h0[((int64_t)n * p.C + ch) * S + n0 + s] : 0.f;
    }
    // loading: channel and first token of this thread
    const int lc = tid % CH, lt = tid / CH, lch = cb * CH + lc;
    const bool lon = lch < p.C;
    const InT* x = static_cast<const InT*>(p.x) + tok0 * p.x_ld + lch;
    const InT* dt = static_cast<const InT*>(p.dt) + tok0 * p.dt_ld + lch;
    const InT* z = p.z ? static_cast<const InT*>(p.z) + tok0 * p.z_ld + lch : nullptr;
    InT* y = p.y ? static_cast<InT*>(p.y) + tok0 * p.C + lch : nullptr;
    const int64_t go = (int64_t)(cb * CH / (p.C / p.G)) * S;
    const InT* b = static_cast<const InT*>(p.b) + tok0 * p.b_ld + go;
    const InT* c = static_cast<const InT*>(p.c) + tok0 * p.c_ld + go;
    const float bias = lon && p.dt_bias ? p.dt_bias[lch] : 0.f, Dv = lon && p.D ? p.D[lch] : 0.f;

    InT rx[LT], rd[LT], rz[LT], rbc[BC];
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const int t = t0 + lt + i * (NT / CH);
            const bool ok = lon && t < t_end;
            rx[i] = ok ? x[t * p.x_ld] : InT(0);
            rd[i] = ok ? dt[t * p.dt_ld] : InT(0);
            rz[i] = ok && z ? z[t * p.z_ld] : InT(0);
        }
#pragma unroll
        for (int i = 0; i < BC; ++i) {
            const int e = tid + i * NT, t = t0 + e / S % TB;
            rbc[i] = e < 2 * TB * S && t < t_end ? (e < TB * S ? b + t * p.b_ld : c + t * p.c_ld)[e % S] : InT(0);
        }
    };
    int64_t ck = ((int64_t)(first_slot(seqs, n, tok0, TB) + t_begin / TB) * p.C + ch) * S + n0;
    int buf = 0;
    if (t_begin < t_end) fetch(t_begin);
    for (int t0 = t_begin; t0 < t_end; t0 += TB, buf ^= 1) {
        float xv[LT], zv[LT];
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const int t = lt + i * (NT / CH);
            xv[i] = widen(rx[i]);
            const float v = widen(rd[i]) + bias;
            const float d = t0 + t < t_end ? (p.softplus ? softplus(v) : v) : 0.f;   // no token: the state stays
            s_du[buf][t][lc] = make_float2(d, d * xv[i]);
            zv[i] = widen(rz[i]);
        }
#pragma unroll
        for (int i = 0; i < BC; ++i) {
            const int e = tid + i * NT;
            if (e < 2 * TB * S) (&s_bc[buf][0][0][0])[e] = widen(rbc[i]);
        }
        lds_barrier();
        if (t0 + TB < t_end) fetch(t0 + TB);
        if (p.ckpt && on) {
#pragma unroll
            for (int s = 0; s < NS; ++s) p.ckpt[ck + s] = h[s];
        }
        ck += (int64_t)p.C * S;
#pragma unroll
        for (int t4 = 0; t4 < TB; t4 += 4) {
            float yt[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 du = s_du[buf][t4 + i][cl];
                const float* bt = &s_bc[buf][0][t4 + i][n0];
                const float* ct = &s_bc[buf][1][t4 + i][n0];
                yt[i] = 0.f;
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    h[s] = fmaf(exp2_f(du.x * A2[s]), h[s], du.y * bt[s]);
                    yt[i] = fmaf(ct[s], h[s], yt[i]);
                }
            }
            s_y[wn][t4 + row_of(g)][cl] = rows_sum4(yt[0], yt[1], yt[2], yt[3]);
        }
        lds_barrier();
        if (y && lon) {
#pragma unroll
            for (int i = 0; i < LT; ++i) {
                const int t = lt + i * (NT / CH);
                if (t0 + t >= t_end) continue;
                float v = Dv * xv[i];
#pragma unroll
                for (int w = 0; w < WN; ++w) v += s_y[w][t][lc];
                st(y + (int64_t)(t0 + t) * p.C, p.z ? v * zv[i] * sigmoid(zv[i]) : v);
            }
        }
    }
    if (p.hT && on && t_end == len) {
#pragma unroll
        for (int s = 0; s < NS; ++s) p.hT[((int64_t)n * p.C + ch) * S + n0 + s] = h[s];
    }
}

template <typename InT, int NS, int WN, int WC>
hipError_t run(const Args& a, hipStream_t s) {
    const int blocks = (a.C + 16 * WC - 1) / (16 * WC);
    hipLaunchKernelGGL((fwd_kernel<InT, NS, WN, WC>), dim3((uint32_t)blocks * a.segs), dim3(64 * WN * WC), 0, s, a,
                       blocks);
    return hipGetLastError();
}

template <typename InT>
hipError_t pick(const Args& a, hipStream_t s) {
    switch (a.S) {
        case 16: return run<InT, 4, 1, 4>(a, s);
        case 32: return run<InT, 4, 2, 4>(a, s);
        default: return run<InT, 4, 4, 2>(a, s);
    }
}

}  // namespace

hipError_t launch_fwd(const Args& a, bool bf16, hipStream_t s) {
    return bf16 ? pick<uint16_t>(a, s) : pick<float>(a, s);
}

}  // namespace ssm
