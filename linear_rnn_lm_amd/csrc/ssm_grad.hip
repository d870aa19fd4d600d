// ssm_grad.hip -- the selective scan's backward (gfx950).
//
// With g_t the gradient of the state after token t (a_t = e^(delta A)):
//     g_t = c_t dy_t + a_(t+1) g_(t+1),    p_t = g_t a_t h_(t-1)
//     db_t = sum_channels g_t delta x,     dc_t = sum_channels dy_t h_t
//     du_t = sum_s g_t b_t,                ddelta_t = x du_t + sum_s p_t A
//     dA = sum_t p_t delta,                dx_t = delta du_t + D dy_t
// where dy is the output's gradient times z sigmoid(z).  16 tokens at a time, last block
// first: from the block's checkpoint the states are formed again, a_t and a_t h_(t-1)
// staying in registers (128 of them), then the block is walked backwards.  Lanes as in the
// forward (16 channels by 4 groups of 4 states); sums over states are swaps of lane rows.
// Sums over a wave's 16 channels go through LDS, two tokens at a time, and come back with four
// channels to a lane, so that most of the adding is done without exchanges.
// Sums over workgroups (db, dc: one part per 64 channels, 32 with 64 states; dA, dD, ddt_bias: one per
// segment) go through memory and a second launch, in a fixed order.
//
// Bound by vector instructions, 85 per wave and token: B4 T4096 C4096
// S16 bf16 815 us, the vector units busy for 81 % of it at two waves per SIMD (all that 128 registers of a and
// a h_(t-1) leave); the sums of db and dc 24 us (5.5 TB/s).
#include "column_sums.h"
#include "ssm_device.h"

namespace ssm {
namespace {

// Orders a wave's LDS accesses for the compiler; the LDS itself serves a wave's in order.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <typename InT, int WN, int WC, bool HZ>
__global__ __launch_bounds__(64 * WN * WC, 2) void bwd_kernel(Args p, int blocks) {
    constexpr int NS = 4, S = 4 * NS * WN, CH = 16 * WC, NT = 64 * WN * WC, TB = kBlock;
    using D_ = Deal<InT, CH, NT, S>;
    constexpr int LT = D_::LT;
    static_assert(CH == chans(S), "one part of db and dc per workgroup");
    typedef float Rows[CH][kPitch];
    __shared__ __attribute__((aligned(16))) Rows s_d, s_u, s_dy, s_x, s_ds, s_zf;   // delta, delta x, dy, x, delta's slope, dz / y
    __shared__ __attribute__((aligned(16))) float s_bc[2][S][kPitch];
    __shared__ __attribute__((aligned(16))) Rows s_y[WN], s_gb[WN], s_pa[WN];
    __shared__ __attribute__((aligned(16))) float s_v[WN * WC][2][2][4 * NS][kPitch];   // two tokens' terms of db and dc
    __shared__ float s_g[WC][TB][2][S];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), wn = wave % WN, wc = wave / WN;
    const int cb = blockIdx.x % blocks, slot = blockIdx.x / blocks;
    const Seqs seqs{p.cu, p.N, p.T};
    const int r16 = lane & 15, g4 = lane >> 4, cl = wc * 16 + r16, ch = cb * CH + cl, n0 = (wn * 4 + g4) * NS;
    const bool on = ch < p.C;
    const D_ deal(tid, cb, p.C);
    float A2[NS], dA[NS], gr[NS], dD = 0.f, dbias = 0.f;
    int n, piece, len = 0;
    int64_t tok0 = 0;
    const bool used = segment_of(p, seqs, slot, n, piece);
    if (used) seq_span(seqs, n, tok0, len);
    n = uniform(n), piece = uniform(piece), len = uniform(len), tok0 = uniform(tok0);
    const int t_begin = used ? piece * p.seg : 0, t_end = used ? segment_end(t_begin, p.seg, len) : 0;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        A2[s] = on ? rate_of(p.A[(int64_t)ch * S + n0 + s]) : 0.f;
        dA[s] = 0.f;
        gr[s] = used && on && p.dhT ? p.dhT[((int64_t)n * p.C + ch) * S + n0 + s] : 0.f;
    }
    if (p.split && used && on) {                           // the segments behind this one, last first
        const int behind = len > t_end ? (len - 1) / p.seg - piece : 0;
        fold_segments<NS>(p, first_slot(seqs, n, tok0, p.seg) + piece + behind, -1, behind, ch, n0, A2, gr);
    }
    int n_blocks = t_begin < t_end ? (t_end - 1 - t_begin) / TB + 1 : 0;
    const int t_last = t_begin + (n_blocks - 1) * TB, t_from = n_blocks ? t_last : t_begin;
    const int64_t go = (int64_t)(cb * CH / (p.C / p.G)) * S;
    Stream sx = stream(static_cast<const InT*>(p.x) + tok0 * p.x_ld, p.x_ld, p.C, t_from);
    Stream sd = stream(static_cast<const InT*>(p.dt) + tok0 * p.dt_ld, p.dt_ld, p.C, t_from);
    Stream sz = stream(HZ ? static_cast<const InT*>(p.z) + tok0 * p.z_ld : nullptr, p.z_ld, p.C, t_from);
    Stream sy = stream(static_cast<const InT*>(p.dy) + tok0 * p.C, p.C, p.C, t_from);
    Mats<InT, NT, S> mats(static_cast<const InT*>(p.b) + tok0 * p.b_ld + go, p.b_ld,
                          static_cast<const InT*>(p.c) + tok0 * p.c_ld + go, p.c_ld, tid, t_from);
    const uint32_t ox = deal.off(p.x_ld), od = deal.off(p.dt_ld), oz = deal.off(p.z_ld), oy = deal.off(p.C);
    const float bias = p.dt_bias ? p.dt_bias[deal.lch] : 0.f, Dv = p.D ? p.D[deal.lch] : 0.f;
    float* part_bc = p.part_bc + ((int64_t)cb * p.B * p.T + tok0) * 2 * S;
    const float* ck = p.ckpt + (int64_t)((used ? first_slot(seqs, n, tok0, TB) : 0) + t_from / TB) * p.C * S;
    const uint32_t ock = on ? (uint32_t)(ch * S + n0) * 4u : kNowhere;

    InT rx[LT], rd[LT], rz[LT], ry[LT], rm[D_::MB];
    float hn[NS];
    int t_fetch = t_from;
    auto fetch = [&] {                                     // the block before the first one is not loaded: its first one again
        const int rows = block_rows(t_fetch, t_end);
        deal.rows(sx, rows, p.x_ld, ox, rx);
        deal.rows(sd, rows, p.dt_ld, od, rd);
        if (HZ) deal.rows(sz, rows, p.z_ld, oz, rz);
        deal.rows(sy, rows, p.C, oy, ry);
        mats.load(rows, p.b_ld, p.c_ld, rm);
        const wkv7::Rsrc r = wkv7::make_rsrc(ck, n_blocks > 0 ? (uint32_t)p.C * S * 4u : 0u);
#pragma unroll
        for (int s = 0; s < NS; ++s) hn[s] = bload<float>(r, ock + 4 * s);
        if (--n_blocks > 0) {
            sx.back(), sd.back(), sz.back(), sy.back(), mats.back();
            ck -= (int64_t)p.C * S;
            t_fetch -= TB;
        }
    };
    fetch();
    for (int t0 = t_last; t0 >= t_begin; t0 -= TB) {
        float h[NS], dAb[NS];
        {
            float d[LT], u[LT], xv[LT], sl[LT], dyv[LT], zf[LT];
#pragma unroll
            for (int i = 0; i < LT; ++i) {
                xv[i] = widen(rx[i]);
                const float v = widen(rd[i]) + bias, yv = widen(ry[i]), st = step_of(p.softplus, v, sl[i]);
                d[i] = deal.lon && t0 + deal.lt + i < t_end ? st : 0.f;
                u[i] = d[i] * xv[i];
                dyv[i] = yv;
                if (HZ) {
                    const float zv = widen(rz[i]), sg = sigmoid_for<InT>(zv), zs = zv * sg;
                    dyv[i] = yv * zs;
                    zf[i] = yv * fmaf(zs, 1.f - sg, sg);
                }
            }
            put_lds<LT>(&s_d[deal.lc][deal.lt], d);
            put_lds<LT>(&s_u[deal.lc][deal.lt], u);
            put_lds<LT>(&s_dy[deal.lc][deal.lt], dyv);
            put_lds<LT>(&s_x[deal.lc][deal.lt], xv);
            put_lds<LT>(&s_ds[deal.lc][deal.lt], sl);
            if (HZ) put_lds<LT>(&s_zf[deal.lc][deal.lt], zf);
            mats.put(&s_bc[0][0][0], rm);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            h[s] = hn[s];
            dAb[s] = 0.f;
        }
        lds_barrier();

        // forward over the block; four tokens' operands are read ahead of their use
        float a[TB][NS], ah[TB][NS];
        {
            f32x4 d[2], u[2], b[2][NS];
            auto read = [&](int k) {
                d[k & 1] = lds4(&s_d[cl][4 * k]);
                u[k & 1] = lds4(&s_u[cl][4 * k]);
#pragma unroll
                for (int s = 0; s < NS; ++s) b[k & 1][s] = lds4(&s_bc[0][n0 + s][4 * k]);
            };
            read(0);
#pragma unroll
            for (int k = 0; k < TB / 4; ++k) {
                if (k + 1 < TB / 4) read(k + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 4 * k + i;
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        a[t][s] = exp2_f(d[k & 1][i] * A2[s]);
                        ah[t][s] = a[t][s] * h[s];
                        h[s] = fmaf(u[k & 1][i], b[k & 1][s][i], ah[t][s]);
                    }
                }
            }
        }
        // and back.  Two tokens' terms of db and dc go to LDS, channels side by side, and come back four channels
        // to a lane; they are added up after the next two tokens, when they have long arrived.
        f32x4 d, u, dyq, b[NS], c[NS], v[4];
        auto read = [&](int k) {
            d = lds4(&s_d[cl][4 * k]);
            u = lds4(&s_u[cl][4 * k]);
            dyq = lds4(&s_dy[cl][4 * k]);
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                b[s] = lds4(&s_bc[0][n0 + s][4 * k]);
                c[s] = lds4(&s_bc[1][n0 + s][4 * k]);
            }
        };
        auto add_up = [&](int t) {                         // tokens t, t + 1: v[j] is db, dc of t, then of t + 1
            float sum[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) sum[j] = (v[j][0] + v[j][1]) + (v[j][2] + v[j][3]);
            (&s_g[wc][t][0][0])[(row_of(g4) >> 1) * 2 * S + (row_of(g4) & 1) * S + 16 * wn + r16] =
                rows_sum4(sum[0], sum[1], sum[2], sum[3]);
        };
        read(TB / 4 - 1);
#pragma unroll
        for (int k = TB / 4 - 1; k >= 0; --k) {
            if (k == 0) fetch();                           // most of a and ah is done with: their registers hold it
            float gb[4], pa[4], yt[4];
#pragma unroll
            for (int i2 = 2; i2 >= 0; i2 -= 2) {
#pragma unroll
                for (int i = i2 + 1; i >= i2; --i) {
                    const int t = 4 * k + i;
                    gb[i] = pa[i] = yt[i] = 0.f;
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        const float bt = b[s][i], ct = c[s][i], ht = fmaf(u[i], bt, ah[t][s]);
                        gr[s] = fmaf(ct, dyq[i], gr[s]);
                        yt[i] = fmaf(ct, ht, yt[i]);
                        gb[i] = fmaf(gr[s], bt, gb[i]);
                        const float q = gr[s] * ah[t][s];
                        pa[i] = fmaf(q, A2[s], pa[i]);
                        dAb[s] = fmaf(q, d[i], dAb[s]);
                        s_v[wave][i - i2][0][4 * g4 + s][r16] = gr[s] * u[i];
                        s_v[wave][i - i2][1][4 * g4 + s][r16] = dyq[i] * ht;
                        gr[s] *= a[t][s];
                    }
                }
                if (4 * k + i2 + 2 < TB) add_up(4 * k + i2 + 2);
                wave_order();
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] = lds4(&s_v[wave][j >> 1][j & 1][r16][4 * g4]);
                if (i2 == 0 && k > 0) read(k - 1);
                wave_order();
            }
            s_gb[wn][cl][4 * k + row_of(g4)] = rows_sum4(gb[0], gb[1], gb[2], gb[3]);
            s_pa[wn][cl][4 * k + row_of(g4)] = rows_sum4(pa[0], pa[1], pa[2], pa[3]);
            if (HZ) s_y[wn][cl][4 * k + row_of(g4)] = rows_sum4(yt[0], yt[1], yt[2], yt[3]);
        }
        add_up(0);
#pragma unroll
        for (int s = 0; s < NS; ++s) dA[s] += dAb[s];
        lds_barrier();
        // What is read here a thread wrote itself, or waves wrote before this barrier and write again after the next
        // one; so the next block's values may go to LDS without another.
        const int64_t at = (tok0 + t0) * p.C;
        const uint32_t bytes = (uint32_t)(min(TB, t_end - t0) * p.C) * (uint32_t)sizeof(InT);
        const wkv7::Rsrc r_dx = wkv7::make_rsrc(static_cast<InT*>(p.dx) + at, bytes);
        const wkv7::Rsrc r_ddt = wkv7::make_rsrc(static_cast<InT*>(p.ddt) + at, bytes);
        const wkv7::Rsrc r_dz = wkv7::make_rsrc(static_cast<InT*>(p.dz) + at, bytes);
        {
            float d1[LT], xv[LT], sl[LT], dyv[LT], zf[LT], gb[LT], pa[LT], yr[LT], part[LT];
            get_lds<LT>(&s_d[deal.lc][deal.lt], d1);
            get_lds<LT>(&s_x[deal.lc][deal.lt], xv);
            get_lds<LT>(&s_ds[deal.lc][deal.lt], sl);
            get_lds<LT>(&s_dy[deal.lc][deal.lt], dyv);
            if (HZ) get_lds<LT>(&s_zf[deal.lc][deal.lt], zf);
            get_lds<LT>(&s_gb[0][deal.lc][deal.lt], gb);
            get_lds<LT>(&s_pa[0][deal.lc][deal.lt], pa);
            if (HZ) get_lds<LT>(&s_y[0][deal.lc][deal.lt], yr);
#pragma unroll
            for (int w = 1; w < WN; ++w) {
                get_lds<LT>(&s_gb[w][deal.lc][deal.lt], part);
#pragma unroll
                for (int i = 0; i < LT; ++i) gb[i] += part[i];
                get_lds<LT>(&s_pa[w][deal.lc][deal.lt], part);
#pragma unroll
                for (int i = 0; i < LT; ++i) pa[i] += part[i];
                if (HZ) {
                    get_lds<LT>(&s_y[w][deal.lc][deal.lt], part);
#pragma unroll
                    for (int i = 0; i < LT; ++i) yr[i] += part[i];
                }
            }
#pragma unroll
            for (int i = 0; i < LT; ++i) {                 // tokens and channels that do not exist have dy = x = 0
                const uint32_t o = oy + D_::row(p.C, i);
                const float dd = fmaf(xv[i], gb[i], kLn2 * pa[i]) * sl[i];
                bstore(InT(0), r_dx, o, fmaf(d1[i], gb[i], Dv * dyv[i]));
                bstore(InT(0), r_ddt, o, dd);
                if (HZ) bstore(InT(0), r_dz, o, fmaf(Dv, xv[i], yr[i]) * zf[i]);
                dD = fmaf(dyv[i], xv[i], dD);
                dbias += deal.lon && t0 + deal.lt + i < t_end ? dd : 0.f;
            }
        }
        // part_bc: [token][db, dc][state]
        const wkv7::Rsrc r_bc = wkv7::make_rsrc(part_bc + (int64_t)t0 * 2 * S, (uint32_t)min(TB, t_end - t0) * 2 * S * 4);
#pragma unroll
        for (int i = 0; i < D_::MB; ++i) {
            float sum = 0.f;
#pragma unroll
            for (int w = 0; w < WC; ++w) sum += (&s_g[w][0][0][0])[tid + i * NT];
            wkv7::bstore(sum, r_bc, (tid + i * NT) * 4, 0);
        }
    }
    if (used && p.dh0 && on && piece == 0) {
#pragma unroll
        for (int s = 0; s < NS; ++s) p.dh0[((int64_t)n * p.C + ch) * S + n0 + s] = gr[s];
    }
    float* part = p.part + (int64_t)slot * p.C * (S + 2);  // (C, S) of dA, then dD's and ddt_bias' (C)
    if (on) {
#pragma unroll
        for (int s = 0; s < NS; ++s) part[(int64_t)ch * S + n0 + s] = dA[s];
    }
    lds_barrier();
    float* s_sum = &s_g[0][0][0][0];                       // NT / CH threads hold sums of one channel
    static_assert(2 * NT <= WC * TB * 2 * S, "two sums for each thread fit");
    s_sum[tid] = dD;
    s_sum[NT + tid] = dbias;
    lds_barrier();
    if (tid < CH && deal.lon) {
        float sum_D = 0.f, sum_bias = 0.f;
#pragma unroll
        for (int i = 0; i < NT / CH; ++i) {
            sum_D += s_sum[i * CH + tid];
            sum_bias += s_sum[NT + i * CH + tid];
        }
        part[(int64_t)p.C * S + deal.lch] = sum_D;
        part[(int64_t)p.C * (S + 1) + deal.lch] = sum_bias;
    }
}

// db and dc of every token in a sequence: sums over the channel blocks of a group, four neighbours to a
// thread.  Bound by HBM: the parts are the most that the gradient kernel writes.
template <typename InT>
__global__ __launch_bounds__(256) void bc_kernel(ReduceArgs p, int blocks, uint32_t zero_from) {
    if (blockIdx.x >= zero_from) {                         // rows outside the sequences
        const Seqs seqs{p.cu, p.N, p.T};
        const int64_t at = (int64_t)(blockIdx.x - zero_from) * 256 + threadIdx.x, row = (int64_t)p.C * sizeof(InT);
        zero_outside(seqs, p.dx, row, at);
        zero_outside(seqs, p.ddt, row, at);
        if (p.dz) zero_outside(seqs, p.dz, row, at);
        zero_outside(seqs, p.db, (int64_t)p.G * p.S * sizeof(InT), at);
        zero_outside(seqs, p.dc, (int64_t)p.G * p.S * sizeof(InT), at);
        return;
    }
    const int64_t tokens = (int64_t)p.B * p.T, all = tokens * p.G * (p.S / 2);
    const int per = p.G > 1 ? blocks / p.G : blocks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)zero_from * 256) {
        const int e = (int)(i % (p.S / 2)) * 4, g = (int)(i / (p.S / 2) % p.G);
        const int64_t t = i / (p.S / 2) / p.G;
        if (p.cu && (t < p.cu[0] || t >= p.cu[p.N])) continue;
        const float* src = p.part_bc + ((int64_t)g * per * tokens + t) * 2 * p.S + e;
        f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int k = 0; k < per; ++k) s += *reinterpret_cast<const f32x4*>(src + (int64_t)k * tokens * 2 * p.S);
        InT* out = static_cast<InT*>(e < p.S ? p.db : p.dc) + (t * p.G + g) * p.S + e % p.S;
#pragma unroll
        for (int q = 0; q < 4; ++q) st(out + q, s[q]);
    }
}

template <typename InT, int WN, int WC>
hipError_t run(const Args& a, hipStream_t s) {
    const int blocks = (a.C + 16 * WC - 1) / (16 * WC);
    const dim3 grid((uint32_t)blocks * a.segs), threads(64 * WN * WC);
    if (a.z) hipLaunchKernelGGL((bwd_kernel<InT, WN, WC, true>), grid, threads, 0, s, a, blocks);
    else hipLaunchKernelGGL((bwd_kernel<InT, WN, WC, false>), grid, threads, 0, s, a, blocks);
    return hipGetLastError();
}

template <typename InT>
hipError_t pick(const Args& a, hipStream_t s) {
    switch (a.S) {
        case 16: return run<InT, 1, 4>(a, s);
        case 32: return run<InT, 2, 4>(a, s);
        default: return run<InT, 4, 2>(a, s);
    }
}

}  // namespace

hipError_t launch_bwd(const Args& a, bool bf16, hipStream_t s) {
    return bf16 ? pick<uint16_t>(a, s) : pick<float>(a, s);
}

hipError_t launch_reduce(const ReduceArgs& a, bool bf16, hipStream_t s) {
    const int64_t CS = (int64_t)a.C * a.S;
    const hipError_t e = sums::launch_column_sums(a.part, a.segs, CS + 2 * a.C, a.dA, CS, a.dD, a.C, a.ddt_bias, s);
    if (e != hipSuccess) return e;
    const int blocks = (a.C + chans(a.S) - 1) / chans(a.S);
    const int64_t n = (int64_t)a.B * a.T * a.G * (a.S / 2);
    const uint32_t main = (uint32_t)((n + 255) / 256 < 1 << 20 ? (n + 255) / 256 : 1 << 20);     // fewer than 2^32 threads
    const dim3 grid(main + (a.zero ? kZeroBlocks : 0));
    if (bf16) hipLaunchKernelGGL(bc_kernel<uint16_t>, grid, dim3(256), 0, s, a, blocks, main);
    else hipLaunchKernelGGL(bc_kernel<float>, grid, dim3(256), 0, s, a, blocks, main);
    return hipGetLastError();
}

}  // namespace ssm
