// ssm_scan.hip -- the selective scan over whole sequences, forward (gfx950).
//
// Per channel and state h <- e^(delta A) h + delta x b, y = sum c h: the decay differs
// per channel, state and token, so the scan has no matrix form; it is bound by vector
// instructions (an exponential, which takes two issue slots, and four more per state
// and token).  A wave works on 16 channels (lane % 16) and 4 NS states, NS to a lane
// (lane / 16), which stay in registers from the first token to the last; WN waves share
// the channels of one block, WC of them lie beside each other.  16 tokens at a time: all
// threads load x, dt, z, b, c, put delta, delta x, b and c into LDS as fp32, the waves scan,
// and the threads that loaded z finish y.
//
// B4 T4096 C4096 S16 bf16, two states to a lane: 353 us, the vector units busy for 75 % of it; B1 T16384 in 16
// segments: 190 us for their sums and 270, 95 and 92 %; 17 packed sequences, T8193 C2048 S64: 230 us, 93 %.  Four states of
// 16 to a lane take all 128 registers of four waves per SIMD: two to five of them are in scratch (20 bytes in bf16 with z) while the
// loop over blocks runs, none within it.
#include "ssm_device.h"

namespace ssm {
namespace {

// What a lane reads of LDS for GT tokens: delta, delta x (or dy), and NS states' b and c.  Read
// whole, ahead of its use: left alone the compiler waits for LDS once every two tokens.
template <int NS, int GT, bool C>
struct Group {
    f32x4 d[GT / 4], u[GT / 4], b[NS][GT / 4], c[C ? NS : 1][GT / 4];
    __device__ __forceinline__ void read(const float* s_d, const float* s_u, const float* s_b, const float* s_c, int t) {
#pragma unroll
        for (int k = 0; k < GT / 4; ++k) {
            d[k] = lds4(s_d + t + 4 * k);
            u[k] = lds4(s_u + t + 4 * k);
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                b[s][k] = lds4(s_b + s * kPitch + t + 4 * k);
                if (C) c[s][k] = lds4(s_c + s * kPitch + t + 4 * k);
            }
        }
    }
};

// Blocks ahead: a block takes a wave alone on its unit about 2600 cycles with 4 states to a lane, 1500
// with 2, a load up to 2000.
template <int NS>
struct Ahead {
    static constexpr int value = NS == 2 ? 2 : 1;
    static constexpr bool groups = NS == 2;        // operands in LDS read a group ahead
    static constexpr int waves = NS == 2 ? 1 : 4;  // per SIMD: where other waves hide what is not read ahead
};

template <typename InT, int NS, int WN, int WC, bool HZ>
__global__ __launch_bounds__(64 * WN * WC, Ahead<NS>::waves) void fwd_kernel(Args p, int blocks) {
    constexpr int S = 4 * NS * WN, CH = 16 * WC, NT = 64 * WN * WC, TB = kBlock, GT = 16 / NS;
    using D_ = Deal<InT, CH, NT, S>;
    constexpr int LT = D_::LT;
    __shared__ __attribute__((aligned(16))) float s_d[2][CH][kPitch], s_u[2][CH][kPitch], s_bc[2][2][S][kPitch];
    __shared__ __attribute__((aligned(16))) float s_y[2][WN][CH][kPitch];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), wn = wave % WN, wc = wave / WN;
    const int cb = blockIdx.x % blocks;
    const Seqs seqs{p.cu, p.N, p.T};
    int n, piece, len;
    if (!segment_of(p, seqs, blockIdx.x / blocks, n, piece)) return;
    int64_t tok0;
    seq_span(seqs, n, tok0, len);
    n = uniform(n), piece = uniform(piece), len = uniform(len), tok0 = uniform(tok0);
    const int t_begin = piece * p.seg, t_end = segment_end(t_begin, p.seg, len);

    // scanning: channel and first state of this lane
    const int cl = wc * 16 + (lane & 15), g = lane >> 4, ch = cb * CH + cl, n0 = (wn * 4 + g) * NS;
    const bool on = ch < p.C;
    float A2[NS], h[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        A2[s] = on ? rate_of(p.A[(int64_t)ch * S + n0 + s]) : 0.f;
        h[s] = on && p.h0 ? p.h0[((int64_t)n * p.C + ch) * S + n0 + s] : 0.f;
    }
    if (p.split && on) fold_segments<NS>(p, first_slot(seqs, n, tok0, p.seg), 1, piece, ch, n0, A2, h);
    // loading and storing
    const D_ deal(tid, cb, p.C);
    const int64_t go = (int64_t)(cb * CH / (p.C / p.G)) * S;
    Stream sx = stream(static_cast<const InT*>(p.x) + tok0 * p.x_ld, p.x_ld, p.C, t_begin);
    Stream sd = stream(static_cast<const InT*>(p.dt) + tok0 * p.dt_ld, p.dt_ld, p.C, t_begin);
    Stream sz = stream(HZ ? static_cast<const InT*>(p.z) + tok0 * p.z_ld : nullptr, p.z_ld, p.C, t_begin);
    Stream sy = stream(static_cast<const InT*>(p.y) + tok0 * p.C, p.C, p.C, t_begin - TB);   // of the block being finished
    Mats<InT, NT, S> mats(static_cast<const InT*>(p.b) + tok0 * p.b_ld + go, p.b_ld,
                          static_cast<const InT*>(p.c) + tok0 * p.c_ld + go, p.c_ld, tid, t_begin);
    const uint32_t ox = deal.off(p.x_ld), od = deal.off(p.dt_ld), oz = deal.off(p.z_ld), oy = deal.off(p.C);
    const float bias = p.dt_bias ? p.dt_bias[deal.lch] : 0.f, Dv = p.D ? p.D[deal.lch] : 0.f;
    float* ck = p.ckpt + (int64_t)(first_slot(seqs, n, tok0, TB) + t_begin / TB) * p.C * S;
    const uint32_t ck_bytes = p.ckpt ? (uint32_t)p.C * S * 4u : 0u;
    const uint32_t ock = on ? (uint32_t)(ch * S + n0) * 4u : kNowhere;
    const int out_rows = p.y ? TB : 0;

    constexpr int PF = Ahead<NS>::value;         // blocks that are on their way from memory
    InT rx[PF][LT], rd[PF][LT], rz[PF][LT], rm[PF][D_::MB];
    int t_fetch = t_begin;
    auto fetch = [&](int j) {
        const int rows = block_rows(t_fetch, t_end);
        deal.rows(sx, rows, p.x_ld, ox, rx[j]);
        deal.rows(sd, rows, p.dt_ld, od, rd[j]);
        if (HZ) deal.rows(sz, rows, p.z_ld, oz, rz[j]);
        mats.load(rows, p.b_ld, p.c_ld, rm[j]);
        t_fetch += TB;
        sx.next(), sd.next(), sz.next(), mats.next();
    };
    float xs[3][LT], zs[3][LT];                  // x and z of the blocks being finished, scanned, prepared
    auto prepare = [&](int t0, int j, int buf, float (&xv)[LT], float (&zv)[LT]) {
        float d[LT], u[LT];
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            xv[i] = widen(rx[j][i]);
            zv[i] = HZ ? widen(rz[j][i]) : 0.f;
            const float v = step_of(p.softplus, widen(rd[j][i]) + bias);
            d[i] = t0 + deal.lt + i < t_end ? v : 0.f;               // no token: the state stays
            u[i] = d[i] * xv[i];
        }
        put_lds<LT>(&s_d[buf][deal.lc][deal.lt], d);
        put_lds<LT>(&s_u[buf][deal.lc][deal.lt], u);
        mats.put(&s_bc[buf][0][0][0], rm[j]);
    };
    auto finish = [&](int rows, int buf, const float (&xv)[LT], const float (&zv)[LT]) {
        const wkv7::Rsrc r = sy.rsrc(rows);
        sy.next();
        float v[LT];
#pragma unroll
        for (int i = 0; i < LT; ++i) v[i] = Dv * xv[i];
#pragma unroll
        for (int w = 0; w < WN; ++w) {
            float part[LT];
            get_lds<LT>(&s_y[buf][w][deal.lc][deal.lt], part);
#pragma unroll
            for (int i = 0; i < LT; ++i) v[i] += part[i];
        }
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            if (HZ) v[i] *= zv[i] * sigmoid_for<InT>(zv[i]);
            bstore(InT(0), r, oy + D_::row(p.C, i), v[i]);
        }
    };
    // One barrier per block of 16 tokens: in one go the next block is prepared, this one scanned and
    // the one before it finished, so that their waits hide each other.
    auto block = [&](int t0, int j, int buf) {
        lds_barrier();
        Group<NS, GT, true> grp[2];
        const float *pd = s_d[buf][cl], *pu = s_u[buf][cl], *pb = s_bc[buf][0][n0], *pc = s_bc[buf][1][n0];
        grp[0].read(pd, pu, pb, pc, 0);
        prepare(t0 + TB, j, buf ^ 1, xs[2], zs[2]);
        fetch(j);
        finish(t0 > t_begin ? out_rows : 0, buf ^ 1, xs[0], zs[0]);
        const wkv7::Rsrc rk = wkv7::make_rsrc(ck, ck_bytes);
        if constexpr (NS == 4) wkv7::bstore4(f32x4{h[0], h[1], h[2], h[3]}, rk, ock, 0);
        else wkv7::bstore2(make_float2(h[0], h[1]), rk, ock, 0);
        ck += (int64_t)p.C * S;
#pragma unroll
        for (int k = 0; k < TB / GT; ++k) {
            const Group<NS, GT, true>& q = grp[k & 1];
            if (!Ahead<NS>::groups && k > 0) grp[k & 1].read(pd, pu, pb, pc, k * GT);
            if (Ahead<NS>::groups && k + 1 < TB / GT) {
                grp[(k + 1) & 1].read(pd, pu, pb, pc, (k + 1) * GT);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int t4 = 0; t4 < GT; t4 += 4) {
                float yt[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    yt[i] = 0.f;
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        h[s] = fmaf(exp2_f(q.d[t4 / 4][i] * A2[s]), h[s], q.u[t4 / 4][i] * q.b[s][t4 / 4][i]);
                        yt[i] = fmaf(q.c[s][t4 / 4][i], h[s], yt[i]);
                    }
                }
                s_y[buf][wn][cl][k * GT + t4 + row_of(g)] = rows_sum4(yt[0], yt[1], yt[2], yt[3]);
            }
        }
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            xs[0][i] = xs[1][i], xs[1][i] = xs[2][i];
            zs[0][i] = zs[1][i], zs[1][i] = zs[2][i];
        }
    };
    fetch(PF - 1);
#pragma unroll
    for (int j = 0; j < PF - 1; ++j) fetch(j);
    prepare(t_begin, PF - 1, 0, xs[1], zs[1]);
    fetch(PF - 1);
#pragma unroll
    for (int i = 0; i < LT; ++i) xs[0][i] = zs[0][i] = 0.f;
    int last = 0;
    constexpr int U = PF > 1 ? PF : 2;
    for (int t0 = t_begin; t0 < t_end; t0 += U * TB) {
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (t0 + j * TB < t_end) {
                block(t0 + j * TB, j % PF, j & 1);
                last = j & 1;
            }
    }
    lds_barrier();
    finish(t_begin < t_end && p.y ? (t_end - 1 - t_begin) % TB + 1 : 0, last, xs[0], zs[0]);
    if (p.hT && on && t_end == len) {
#pragma unroll
        for (int s = 0; s < NS; ++s) p.hT[((int64_t)n * p.C + ch) * S + n0 + s] = h[s];
    }
}

// What a segment leaves of a zero state, forward (h <- a h + delta x b) or, for the backward,
// in reverse (g <- a (g + c dy)), and the sum of its steps, a thread's neighbouring tokens (up to four) in
// 32 bits, those sums in 64.  Five sixths of the forward's
// instructions, without its outputs.
template <typename InT, int NS, int WN, int WC, bool BWD, bool HZ>
__global__ __launch_bounds__(64 * WN * WC) void segment_kernel(Args p, int blocks) {
    constexpr int S = 4 * NS * WN, CH = 16 * WC, NT = 64 * WN * WC, TB = kBlock, GT = 16 / NS;
    using D_ = Deal<InT, CH, NT, S>;
    constexpr int LT = D_::LT, MB = (TB * S + NT - 1) / NT;
    __shared__ __attribute__((aligned(16))) float s_d[2][CH][kPitch], s_u[2][CH][kPitch];   // delta, and delta x or dy
    __shared__ __attribute__((aligned(16))) float s_b[2][S][kPitch];                        // b or c
    __shared__ double s_sum[NT];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), wn = wave % WN, wc = wave / WN;
    const int cb = blockIdx.x % blocks;
    const Seqs seqs{p.cu, p.N, p.T};
    int n, piece, len;
    if (!segment_of(p, seqs, blockIdx.x / blocks, n, piece)) return;
    int64_t tok0;
    seq_span(seqs, n, tok0, len);
    n = uniform(n), piece = uniform(piece), len = uniform(len), tok0 = uniform(tok0);
    const int t_begin = piece * p.seg, t_end = segment_end(t_begin, p.seg, len);
    const int cl = wc * 16 + (lane & 15), g = lane >> 4, ch = cb * CH + cl, n0 = (wn * 4 + g) * NS;
    const bool on = ch < p.C;
    if (!BWD && p.h0_copy && piece == 0 && on) {
        const int64_t at = ((int64_t)n * p.C + ch) * S + n0;
#pragma unroll
        for (int s = 0; s < NS; ++s) p.h0_copy[at + s] = p.h0[at + s];
    }
    if (BWD ? t_begin == 0 : t_end == len) return;         // nothing lies behind it
    float A2[NS], h[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        A2[s] = on ? rate_of(p.A[(int64_t)ch * S + n0 + s]) : 0.f;
        h[s] = 0.f;
    }
    const D_ deal(tid, cb, p.C);
    const int64_t u_ld = BWD ? p.C : p.x_ld, b_ld = BWD ? p.c_ld : p.b_ld;
    const float bias = p.dt_bias ? p.dt_bias[deal.lch] : 0.f;
    const int n_blocks = (t_end - t_begin + TB - 1) / TB;
    int t0 = BWD ? t_begin + (n_blocks - 1) * TB : t_begin;
    Stream su = stream(static_cast<const InT*>(BWD ? p.dy : p.x) + tok0 * u_ld, u_ld, p.C, t0);
    Stream sd = stream(static_cast<const InT*>(p.dt) + tok0 * p.dt_ld, p.dt_ld, p.C, t0);
    Stream sz = stream(HZ ? static_cast<const InT*>(p.z) + tok0 * p.z_ld : nullptr, p.z_ld, p.C, t0);
    Stream sb = stream(static_cast<const InT*>(BWD ? p.c : p.b) + tok0 * b_ld + (int64_t)(cb * CH / (p.C / p.G)) * S, b_ld, S, t0);
    const uint32_t ou = deal.off(u_ld), od = deal.off(p.dt_ld), oz = deal.off(p.z_ld);
    const uint32_t ob = (uint32_t)(tid / S * (int)b_ld + tid % S) * (uint32_t)sizeof(InT);
    double total = 0.;
    int blocks_left = n_blocks;

    constexpr int PF = Ahead<NS>::value;
    InT ru[PF][LT], rd[PF][LT], rz[PF][LT], rb[PF][MB];
    int t_fetch = t0;
    auto fetch = [&](int j) {
        const int rows = block_rows(t_fetch, t_end);
        deal.rows(su, rows, u_ld, ou, ru[j]);
        deal.rows(sd, rows, p.dt_ld, od, rd[j]);
        if (HZ) deal.rows(sz, rows, p.z_ld, oz, rz[j]);
        const wkv7::Rsrc r = sb.rsrc(rows);
#pragma unroll
        for (int i = 0; i < MB; ++i) rb[j][i] = bload<InT>(r, ob + (uint32_t)(i * (NT / S) * (int)b_ld) * (uint32_t)sizeof(InT));
        // backward no further than to the first block, which is then read again and not used
        if (!BWD || --blocks_left > 0) {
            t_fetch += BWD ? -TB : TB;
            for (Stream* s : {&su, &sd, &sz, &sb}) BWD ? s->back() : s->next();
        }
    };
    auto prepare = [&](int t0, int j, int buf) {
        float sum = 0.f, d[LT], u[LT];
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const float v = step_of(p.softplus, widen(rd[j][i]) + bias);
            d[i] = t0 >= t_begin && t0 + deal.lt + i < t_end ? v : 0.f;
            u[i] = widen(ru[j][i]);
            if (HZ) {
                const float zv = widen(rz[j][i]);
                u[i] *= zv * sigmoid_for<InT>(zv);
            }
            if (!BWD) u[i] *= d[i];
            sum += d[i];
        }
        total += (double)sum;
        put_lds<LT>(&s_d[buf][deal.lc][deal.lt], d);
        put_lds<LT>(&s_u[buf][deal.lc][deal.lt], u);
#pragma unroll
        for (int i = 0; i < MB; ++i)
            if (MB * NT == TB * S || tid < TB * S) s_b[buf][tid % S][tid / S + i * (NT / S)] = widen(rb[j][i]);
    };
    // as in the forward: the next block is prepared while this one is scanned
    constexpr int step = BWD ? -TB : TB;
    auto block = [&](int t0, int j, int buf) {
        lds_barrier();
        Group<NS, GT, false> grp[2];
        const float *pd = s_d[buf][cl], *pu = s_u[buf][cl], *pb = s_b[buf][n0];
        grp[0].read(pd, pu, pb, nullptr, BWD ? TB - GT : 0);
        prepare(t0 + step, j, buf ^ 1);
        fetch(j);
#pragma unroll
        for (int k = 0; k < TB / GT; ++k) {
            const Group<NS, GT, false>& q = grp[k & 1];
            if (!Ahead<NS>::groups && k > 0) grp[k & 1].read(pd, pu, pb, nullptr, BWD ? TB - (k + 1) * GT : k * GT);
            if (Ahead<NS>::groups && k + 1 < TB / GT) {
                grp[(k + 1) & 1].read(pd, pu, pb, nullptr, BWD ? TB - (k + 2) * GT : (k + 1) * GT);
                __builtin_amdgcn_sched_barrier(0);
            }
#pragma unroll
            for (int i = 0; i < GT; ++i) {
                const int t = BWD ? GT - 1 - i : i;
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const float a = exp2_f(q.d[t / 4][t % 4] * A2[s]), u = q.u[t / 4][t % 4], bt = q.b[s][t / 4][t % 4];
                    h[s] = BWD ? a * fmaf(u, bt, h[s]) : fmaf(a, h[s], u * bt);
                }
            }
        }
    };
    fetch(PF - 1);
#pragma unroll
    for (int j = 0; j < PF - 1; ++j) fetch(j);
    prepare(t0, PF - 1, 0);
    fetch(PF - 1);
    constexpr int U = PF > 1 ? PF : 2;
    for (int k = 0; k < n_blocks; k += U, t0 += U * step) {
#pragma unroll
        for (int j = 0; j < U; ++j)
            if (k + j < n_blocks) block(t0 + j * step, j % PF, j & 1);
    }
    const int slot = first_slot(seqs, n, tok0, p.seg) + piece;
    if (on) {
#pragma unroll
        for (int s = 0; s < NS; ++s) p.sum_h[((int64_t)slot * p.C + ch) * S + n0 + s] = h[s];
    }
    s_sum[tid] = total;                                    // NT / CH threads hold sums of one channel
    lds_barrier();
    if (tid < CH && deal.lon) {
#pragma unroll
        for (int i = 1; i < NT / CH; ++i) total += s_sum[i * CH + tid];
        p.sum_d[(int64_t)slot * p.C + deal.lch] = (float)total;
    }
}

__global__ __launch_bounds__(256) void zero_kernel(Args p, int64_t row_bytes) {
    zero_outside(Seqs{p.cu, p.N, p.T}, p.y, row_bytes, (int64_t)blockIdx.x * 256 + threadIdx.x);
}

enum What { kFwd, kSums, kSumsBack };

template <typename InT, int NS, int WN, int WC>
hipError_t run(const Args& a, What what, hipStream_t s) {
    const int blocks = (a.C + 16 * WC - 1) / (16 * WC);
    const dim3 grid((uint32_t)blocks * a.segs), threads(64 * WN * WC);
    if (what == kFwd && a.z) hipLaunchKernelGGL((fwd_kernel<InT, NS, WN, WC, true>), grid, threads, 0, s, a, blocks);
    else if (what == kFwd) hipLaunchKernelGGL((fwd_kernel<InT, NS, WN, WC, false>), grid, threads, 0, s, a, blocks);
    else if (what == kSums) hipLaunchKernelGGL((segment_kernel<InT, NS, WN, WC, false, false>), grid, threads, 0, s, a, blocks);
    else if (a.z) hipLaunchKernelGGL((segment_kernel<InT, NS, WN, WC, true, true>), grid, threads, 0, s, a, blocks);
    else hipLaunchKernelGGL((segment_kernel<InT, NS, WN, WC, true, false>), grid, threads, 0, s, a, blocks);
    return hipGetLastError();
}

template <typename InT>
hipError_t pick(const Args& a, What what, hipStream_t s) {
    switch (a.S) {
        case 16: return (what == kFwd ? a.halves : a.halves_sums) ? run<InT, 2, 2, 4>(a, what, s) : run<InT, 4, 1, 4>(a, what, s);
        case 32: return run<InT, 4, 2, 4>(a, what, s);
        default: return run<InT, 4, 4, 2>(a, what, s);
    }
}
hipError_t launch(const Args& a, bool bf16, What what, hipStream_t s) {
    return bf16 ? pick<uint16_t>(a, what, s) : pick<float>(a, what, s);
}

}  // namespace

hipError_t launch_segments(const Args& a, bool bf16, bool bwd, hipStream_t s) { return launch(a, bf16, bwd ? kSumsBack : kSums, s); }
hipError_t launch_fwd(const Args& a, bool bf16, hipStream_t s) {
    const hipError_t e = launch(a, bf16, kFwd, s);
    if (e != hipSuccess || !a.zero) return e;
    hipLaunchKernelGGL(zero_kernel, dim3(kZeroBlocks), dim3(256), 0, s, a, (int64_t)a.C * (bf16 ? 2 : 4));
    return hipGetLastError();
}

}  // namespace ssm
