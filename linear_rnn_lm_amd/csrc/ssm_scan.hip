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
#include "ssm_device.h"

namespace ssm {
namespace {

template <typename InT, int NS, int WN, int WC>
__global__ __launch_bounds__(64 * WN * WC) void fwd_kernel(Args p, int blocks) {
    constexpr int S = 4 * NS * WN, CH = 16 * WC, NT = 64 * WN * WC, TB = kBlock;
    using D_ = Deal<InT, CH, NT, S>;
    constexpr int LT = D_::LT, HB = D_::HB, STEP = D_::STEP;
    __shared__ float2 s_du[2][TB][CH];           // delta, delta x
    __shared__ float s_b[2][TB][S], s_c[2][TB][S];
    __shared__ float s_y[WN][TB][CH];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), wn = wave % WN, wc = wave / WN;
    const int cb = blockIdx.x % blocks, slot = blockIdx.x / blocks;
    const Seqs seqs{p.cu, p.N, p.T};
    int n, piece, len;
    if (!slot_piece(seqs, slot, p.seg, n, piece)) return;
    int64_t tok0;
    seq_span(seqs, n, tok0, len);
    n = uniform(n), piece = uniform(piece), len = uniform(len), tok0 = uniform(tok0);
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
    if (p.split && on) fold_segments<NS>(p, slot - piece, 1, piece, ch, n0, A2, h);
    // loading
    const D_ deal(tid, cb, p.C);
    const InT* x = static_cast<const InT*>(p.x) + tok0 * p.x_ld;
    const InT* dt = static_cast<const InT*>(p.dt) + tok0 * p.dt_ld;
    const InT* z = p.z ? static_cast<const InT*>(p.z) + tok0 * p.z_ld : nullptr;
    InT* y = p.y ? static_cast<InT*>(p.y) + tok0 * p.C : nullptr;
    const int64_t go = (int64_t)(cb * CH / (p.C / p.G)) * S;
    const InT* b = static_cast<const InT*>(p.b) + tok0 * p.b_ld + go;
    const InT* c = static_cast<const InT*>(p.c) + tok0 * p.c_ld + go;
    const uint32_t ox = deal.off(p.x_ld), od = deal.off(p.dt_ld), oz = deal.off(p.z_ld), oy = deal.off(p.C);
    const uint32_t ob = D_::off_b(tid, p.b_ld), oc = D_::off_b(tid, p.c_ld);
    const float bias = p.dt_bias ? p.dt_bias[deal.lch] : 0.f, Dv = p.D ? p.D[deal.lch] : 0.f;
    const bool wide = (cb + 1) * CH <= p.C;

    InT rx[LT], rd[LT], rz[LT], rb[HB], rc[HB];
    auto fetch = [&](int t0) {
        const bool full = wide && t0 + TB <= t_end;
        deal.rows(x, p.x_ld, ox, t0, t_end, full, rx);
        deal.rows(dt, p.dt_ld, od, t0, t_end, full, rd);
        if (z) deal.rows(z, p.z_ld, oz, t0, t_end, full, rz);
        D_::mat(b, p.b_ld, ob, tid, t0, t_end, full, rb);
        D_::mat(c, p.c_ld, oc, tid, t0, t_end, full, rc);
    };
    float* ck = p.ckpt ? p.ckpt + (int64_t)(first_slot(seqs, n, tok0, TB) + t_begin / TB) * p.C * S : nullptr;
    const uint32_t ock = (uint32_t)(ch * S + n0) * 4u;
    int buf = 0;
    if (t_begin < t_end) fetch(t_begin);
    for (int t0 = t_begin; t0 < t_end; t0 += TB, buf ^= 1) {
        const bool full = t0 + TB <= t_end;
        float xv[LT], zv[LT];
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const int t = deal.lt + i * STEP;
            xv[i] = widen(rx[i]);
            const float v = widen(rd[i]) + bias;
            float d = p.softplus ? softplus(v) : v;
            if (!full) d = t0 + t < t_end ? d : 0.f;       // no token: the state stays
            s_du[buf][t][deal.lc] = make_float2(d, d * xv[i]);
            if (z) zv[i] = widen(rz[i]);
        }
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            (&s_b[buf][0][0])[tid + i * NT] = widen(rb[i]);
            (&s_c[buf][0][0])[tid + i * NT] = widen(rc[i]);
        }
        lds_barrier();
        if (t0 + TB < t_end) fetch(t0 + TB);
        if (ck) {
            if (on) {
#pragma unroll
                for (int s = 0; s < NS; ++s) *pto<float>(ck, ock + 4 * s) = h[s];
            }
            ck += (int64_t)p.C * S;
        }
#pragma unroll
        for (int t4 = 0; t4 < TB; t4 += 4) {
            float yt[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 du = s_du[buf][t4 + i][cl];
                const float* bt = &s_b[buf][t4 + i][n0];
                const float* ct = &s_c[buf][t4 + i][n0];
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
        if (y) {
            InT* yb = y + (int64_t)t0 * p.C;
#pragma unroll
            for (int i = 0; i < LT; ++i, yb += (int64_t)STEP * p.C) {
                const int t = deal.lt + i * STEP;
                float v = Dv * xv[i];
#pragma unroll
                for (int w = 0; w < WN; ++w) v += s_y[w][t][deal.lc];
                if (z) v *= zv[i] * sigmoid(zv[i]);
                if (deal.lon && (full || t0 + t < t_end)) st(pto<InT>(yb, oy), v);
            }
        }
    }
    if (p.hT && on && t_end == len) {
#pragma unroll
        for (int s = 0; s < NS; ++s) p.hT[((int64_t)n * p.C + ch) * S + n0 + s] = h[s];
    }
}

// What a segment leaves of a zero state, forward (h <- a h + delta x b) or, for the backward,
// in reverse (g <- a (g + c dy)), and the sum of its steps.  Five sixths of the forward's
// instructions, without its outputs.
template <typename InT, int NS, int WN, int WC, bool BWD>
__global__ __launch_bounds__(64 * WN * WC) void segment_kernel(Args p, int blocks) {
    constexpr int S = 4 * NS * WN, CH = 16 * WC, NT = 64 * WN * WC, TB = kBlock;
    using D_ = Deal<InT, CH, NT, S>;
    constexpr int LT = D_::LT, HB = D_::HB, STEP = D_::STEP;
    __shared__ float2 s_du[2][TB][CH];           // delta, and delta x or dy
    __shared__ float s_b[2][TB][S];              // b or c
    __shared__ double s_d[NT];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), wn = wave % WN, wc = wave / WN;
    const int cb = blockIdx.x % blocks, slot = blockIdx.x / blocks;
    const Seqs seqs{p.cu, p.N, p.T};
    int n, piece, len;
    if (!slot_piece(seqs, slot, p.seg, n, piece)) return;
    int64_t tok0;
    seq_span(seqs, n, tok0, len);
    n = uniform(n), piece = uniform(piece), len = uniform(len), tok0 = uniform(tok0);
    const int t_begin = piece * p.seg, t_end = min(len, t_begin + p.seg);
    if (BWD ? t_begin == 0 : t_end == len) return;         // nothing lies behind it
    const int cl = wc * 16 + (lane & 15), g = lane >> 4, ch = cb * CH + cl, n0 = (wn * 4 + g) * NS;
    const bool on = ch < p.C;
    float A2[NS], h[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        A2[s] = on ? kLog2e * p.A[(int64_t)ch * S + n0 + s] : 0.f;
        h[s] = 0.f;
    }
    const D_ deal(tid, cb, p.C);
    const int64_t u_ld = BWD ? p.C : p.x_ld, b_ld = BWD ? p.c_ld : p.b_ld;
    const InT* dt = static_cast<const InT*>(p.dt) + tok0 * p.dt_ld;
    const InT* u = static_cast<const InT*>(BWD ? p.dy : p.x) + tok0 * u_ld;
    const InT* z = BWD && p.z ? static_cast<const InT*>(p.z) + tok0 * p.z_ld : nullptr;
    const InT* b = static_cast<const InT*>(BWD ? p.c : p.b) + tok0 * b_ld + (int64_t)(cb * CH / (p.C / p.G)) * S;
    const uint32_t ou = deal.off(u_ld), od = deal.off(p.dt_ld), oz = deal.off(p.z_ld), ob = D_::off_b(tid, b_ld);
    const float bias = p.dt_bias ? p.dt_bias[deal.lch] : 0.f;
    const bool wide = (cb + 1) * CH <= p.C;
    double total = 0.;

    InT ru[LT], rd[LT], rz[LT], rb[HB];
    auto fetch = [&](int t0) {
        const bool full = wide && t0 + TB <= t_end;
        deal.rows(u, u_ld, ou, t0, t_end, full, ru);
        deal.rows(dt, p.dt_ld, od, t0, t_end, full, rd);
        if (z) deal.rows(z, p.z_ld, oz, t0, t_end, full, rz);
        D_::mat(b, b_ld, ob, tid, t0, t_end, full, rb);
    };
    const int n_blocks = (t_end - t_begin + TB - 1) / TB;
    int buf = 0;
    fetch(BWD ? t_begin + (n_blocks - 1) * TB : t_begin);
    for (int k = 0; k < n_blocks; ++k, buf ^= 1) {
        const int t0 = t_begin + (BWD ? n_blocks - 1 - k : k) * TB;
        const bool full = t0 + TB <= t_end;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const int t = deal.lt + i * STEP;
            const float v = widen(rd[i]) + bias;
            float d = p.softplus ? softplus(v) : v, uv = widen(ru[i]);
            if (!full) d = t0 + t < t_end ? d : 0.f;
            if (z) {
                const float zv = widen(rz[i]);
                uv *= zv * sigmoid(zv);
            }
            s_du[buf][t][deal.lc] = make_float2(d, BWD ? uv : d * uv);
            sum += d;
        }
        total += (double)sum;
#pragma unroll
        for (int i = 0; i < HB; ++i) (&s_b[buf][0][0])[tid + i * NT] = widen(rb[i]);
        lds_barrier();
        if (k + 1 < n_blocks) fetch(BWD ? t0 - TB : t0 + TB);
#pragma unroll
        for (int i = 0; i < TB; ++i) {
            const int t = BWD ? TB - 1 - i : i;
            const float2 du = s_du[buf][t][cl];
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const float a = exp2_f(du.x * A2[s]), bt = s_b[buf][t][n0 + s];
                h[s] = BWD ? a * fmaf(du.y, bt, h[s]) : fmaf(a, h[s], du.y * bt);
            }
        }
    }
    if (on) {
#pragma unroll
        for (int s = 0; s < NS; ++s) p.sum_h[((int64_t)slot * p.C + ch) * S + n0 + s] = h[s];
    }
    s_d[tid] = total;                                      // NT / CH threads hold sums of one channel
    lds_barrier();
    if (tid < CH && deal.lon) {
#pragma unroll
        for (int i = 1; i < NT / CH; ++i) total += s_d[i * CH + tid];
        p.sum_d[(int64_t)slot * p.C + deal.lch] = (float)total;
    }
}

template <typename InT, int NS, int WN, int WC>
hipError_t run(const Args& a, hipStream_t s) {
    const int blocks = (a.C + 16 * WC - 1) / (16 * WC);
    hipLaunchKernelGGL((fwd_kernel<InT, NS, WN, WC>), dim3((uint32_t)blocks * a.segs), dim3(64 * WN * WC), 0, s, a,
                       blocks);
    return hipGetLastError();
}

template <typename InT, int NS, int WN, int WC>
hipError_t run_segments(const Args& a, bool bwd, hipStream_t s) {
    const int blocks = (a.C + 16 * WC - 1) / (16 * WC);
    const dim3 grid((uint32_t)blocks * a.segs), threads(64 * WN * WC);
    if (bwd) hipLaunchKernelGGL((segment_kernel<InT, NS, WN, WC, true>), grid, threads, 0, s, a, blocks);
    else hipLaunchKernelGGL((segment_kernel<InT, NS, WN, WC, false>), grid, threads, 0, s, a, blocks);
    return hipGetLastError();
}

template <typename InT>
hipError_t pick_segments(const Args& a, bool bwd, hipStream_t s) {
    switch (a.S) {
        case 16: return run_segments<InT, 4, 1, 4>(a, bwd, s);
        case 32: return run_segments<InT, 4, 2, 4>(a, bwd, s);
        default: return run_segments<InT, 4, 4, 2>(a, bwd, s);
    }
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

hipError_t launch_segments(const Args& a, bool bf16, bool bwd, hipStream_t s) {
    return bf16 ? pick_segments<uint16_t>(a, bwd, s) : pick_segments<float>(a, bwd, s);
}

hipError_t launch_fwd(const Args& a, bool bf16, hipStream_t s) {
    return bf16 ? pick<uint16_t>(a, s) : pick<float>(a, s);
}

}  // namespace ssm
