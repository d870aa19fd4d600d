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
#include "ssm_device.h"

namespace ssm {
namespace {

// Orders a wave's LDS accesses for the compiler; the LDS itself serves a wave's in order.
__device__ __forceinline__ void wave_order() {
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

template <typename InT, int WN, int WC>
__global__ __launch_bounds__(64 * WN * WC, 2) void bwd_kernel(Args p, int blocks) {
    constexpr int NS = 4, S = 4 * NS * WN, CH = 16 * WC, NT = 64 * WN * WC, TB = kBlock;
    using D_ = Deal<InT, CH, NT, S>;
    constexpr int LT = D_::LT, HB = D_::HB, STEP = D_::STEP;
    constexpr int VP = 20;                       // a row of s_v: 16 channels, padded against bank conflicts
    static_assert(CH == chans(S), "one part of db and dc per workgroup");
    __shared__ float2 s_du[TB][CH];              // delta, delta x
    __shared__ float s_dy[TB][CH], s_b[TB][S], s_c[TB][S];
    __shared__ float s_x[TB][CH], s_ds[TB][CH], s_zf[TB][CH];     // x, delta's slope, dz / y
    __shared__ float s_y[WN][TB][CH], s_gb[WN][TB][CH], s_pa[WN][TB][CH];
    __shared__ float s_v[WN * WC][2][2][16][VP];
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
    const bool used = slot_piece(seqs, slot, p.seg, n, piece);
    if (used) seq_span(seqs, n, tok0, len);
    n = uniform(n), piece = uniform(piece), len = uniform(len), tok0 = uniform(tok0);
    const int t_begin = used ? piece * p.seg : 0, t_end = used ? min(len, t_begin + p.seg) : 0;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        A2[s] = on ? kLog2e * p.A[(int64_t)ch * S + n0 + s] : 0.f;
        dA[s] = 0.f;
        gr[s] = used && on && p.dhT ? p.dhT[((int64_t)n * p.C + ch) * S + n0 + s] : 0.f;
    }
    if (p.split && used && on) {                           // the segments behind this one, last first
        const int behind = len > t_end ? (len - 1) / p.seg - piece : 0;
        fold_segments<NS>(p, slot + behind, -1, behind, ch, n0, A2, gr);
    }
    const InT* x = static_cast<const InT*>(p.x) + tok0 * p.x_ld;
    const InT* dt = static_cast<const InT*>(p.dt) + tok0 * p.dt_ld;
    const InT* z = p.z ? static_cast<const InT*>(p.z) + tok0 * p.z_ld : nullptr;
    const InT* dy = static_cast<const InT*>(p.dy) + tok0 * p.C;
    const int64_t go = (int64_t)(cb * CH / (p.C / p.G)) * S;
    const InT* b = static_cast<const InT*>(p.b) + tok0 * p.b_ld + go;
    const InT* c = static_cast<const InT*>(p.c) + tok0 * p.c_ld + go;
    const uint32_t ox = deal.off(p.x_ld), od = deal.off(p.dt_ld), oz = deal.off(p.z_ld), oy = deal.off(p.C);
    const uint32_t ob = D_::off_b(tid, p.b_ld), oc = D_::off_b(tid, p.c_ld);
    const float bias = p.dt_bias ? p.dt_bias[deal.lch] : 0.f, Dv = p.D ? p.D[deal.lch] : 0.f;
    float* part_bc = p.part_bc + ((int64_t)cb * p.B * p.T + tok0) * 2 * S;
    const bool wide = (cb + 1) * CH <= p.C;

    InT rx[LT], rd[LT], rz[LT], ry[LT], rb[HB], rc[HB];
    float hn[NS];
    const float* ck = p.ckpt + (int64_t)(used ? first_slot(seqs, n, tok0, TB) : 0) * p.C * S;
    const uint32_t ock = (uint32_t)((on ? ch : p.C - 1) * S + n0) * 4u;
    auto fetch = [&](int t0) {
        const bool full = wide && t0 + TB <= t_end;
        deal.rows(x, p.x_ld, ox, t0, t_end, full, rx);
        deal.rows(dt, p.dt_ld, od, t0, t_end, full, rd);
        if (z) deal.rows(z, p.z_ld, oz, t0, t_end, full, rz);
        deal.rows(dy, p.C, oy, t0, t_end, full, ry);
        D_::mat(b, p.b_ld, ob, tid, t0, t_end, full, rb);
        D_::mat(c, p.c_ld, oc, tid, t0, t_end, full, rc);
        const float* q = ck + (int64_t)(t0 / TB) * p.C * S;
#pragma unroll
        for (int s = 0; s < NS; ++s) hn[s] = ldo<float>(q, ock + 4 * s);
    };
    const int t_last = t_begin < t_end ? t_begin + (t_end - 1 - t_begin) / TB * TB : t_begin - TB;
    if (t_last >= t_begin) fetch(t_last);
    for (int t0 = t_last; t0 >= t_begin; t0 -= TB) {
        const bool full = wide && t0 + TB <= t_end;
        float h[NS], dAb[NS];
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const int t = deal.lt + i * STEP;
            const float xv = widen(rx[i]), v = widen(rd[i]) + bias, yv = widen(ry[i]);
            float d = p.softplus ? softplus(v) : v;
            if (!full) d = deal.lon && t0 + t < t_end ? d : 0.f;
            s_du[t][deal.lc] = make_float2(d, d * xv);
            s_x[t][deal.lc] = xv;
            s_ds[t][deal.lc] = p.softplus ? sigmoid(v) : 1.f;
            if (z) {
                const float zv = widen(rz[i]), sg = sigmoid(zv), zs = zv * sg;
                s_dy[t][deal.lc] = yv * zs;
                s_zf[t][deal.lc] = yv * fmaf(zs, 1.f - sg, sg);
            } else {
                s_dy[t][deal.lc] = yv;
            }
        }
#pragma unroll
        for (int i = 0; i < HB; ++i) {
            (&s_b[0][0])[tid + i * NT] = widen(rb[i]);
            (&s_c[0][0])[tid + i * NT] = widen(rc[i]);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            h[s] = on ? hn[s] : 0.f;
            dAb[s] = 0.f;
        }
        lds_barrier();
        if (t0 > t_begin) fetch(t0 - TB);

        float a[TB][NS], ah[TB][NS];
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            const float2 du = s_du[t][cl];
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                a[t][s] = exp2_f(du.x * A2[s]);
                ah[t][s] = a[t][s] * h[s];
                h[s] = fmaf(du.y, s_b[t][n0 + s], ah[t][s]);
            }
        }
#pragma unroll
        for (int t4 = TB - 4; t4 >= 0; t4 -= 4) {
            float gb[4], pa[4], yt[4];
#pragma unroll
            for (int i2 = 2; i2 >= 0; i2 -= 2) {
#pragma unroll
                for (int i = i2 + 1; i >= i2; --i) {
                    const int t = t4 + i;
                    const float2 du = s_du[t][cl];
                    const float dyt = s_dy[t][cl];
                    gb[i] = pa[i] = yt[i] = 0.f;
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        const float bt = s_b[t][n0 + s], ct = s_c[t][n0 + s], ht = fmaf(du.y, bt, ah[t][s]);
                        gr[s] = fmaf(ct, dyt, gr[s]);
                        yt[i] = fmaf(ct, ht, yt[i]);
                        gb[i] = fmaf(gr[s], bt, gb[i]);
                        const float q = gr[s] * ah[t][s];
                        pa[i] = fmaf(q, A2[s], pa[i]);
                        dAb[s] = fmaf(q, du.x, dAb[s]);
                        s_v[wave][i - i2][0][4 * g4 + s][r16] = gr[s] * du.y;
                        s_v[wave][i - i2][1][4 * g4 + s][r16] = dyt * ht;
                        gr[s] *= a[t][s];
                    }
                }
                wave_order();
                float sum[4];                              // two tokens' db, dc; four channels here, the rest by rows
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const f32x4 v = *reinterpret_cast<const f32x4*>(&s_v[wave][i >> 1][i & 1][r16][4 * g4]);
                    sum[i] = (v[0] + v[1]) + (v[2] + v[3]);
                }
                wave_order();
                (&s_g[wc][t4 + i2][0][0])[(row_of(g4) >> 1) * 2 * S + (row_of(g4) & 1) * S + 16 * wn + r16] =
                    rows_sum4(sum[0], sum[1], sum[2], sum[3]);
            }
            s_gb[wn][t4 + row_of(g4)][cl] = rows_sum4(gb[0], gb[1], gb[2], gb[3]);
            s_pa[wn][t4 + row_of(g4)][cl] = rows_sum4(pa[0], pa[1], pa[2], pa[3]);
            if (z) s_y[wn][t4 + row_of(g4)][cl] = rows_sum4(yt[0], yt[1], yt[2], yt[3]);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) dA[s] += dAb[s];
        lds_barrier();
        const int64_t o = (tok0 + t0) * p.C;
        InT* dx = static_cast<InT*>(p.dx) + o;
        InT* ddt = static_cast<InT*>(p.ddt) + o;
        InT* dz = static_cast<InT*>(p.dz) + o;
#pragma unroll
        for (int i = 0; i < LT; ++i, dx += (int64_t)STEP * p.C, ddt += (int64_t)STEP * p.C, dz += (int64_t)STEP * p.C) {
            const int t = deal.lt + i * STEP;
            const float xv = s_x[t][deal.lc], dyt = s_dy[t][deal.lc];
            float gb = 0.f, pa = 0.f, yr = Dv * xv;
#pragma unroll
            for (int w = 0; w < WN; ++w) {
                gb += s_gb[w][t][deal.lc];
                pa += s_pa[w][t][deal.lc];
                if (z) yr += s_y[w][t][deal.lc];
            }
            const float dd = fmaf(xv, gb, kLn2 * pa) * s_ds[t][deal.lc];
            if (full || (deal.lon && t0 + t < t_end)) {
                st(pto<InT>(dx, oy), fmaf(s_du[t][deal.lc].x, gb, Dv * dyt));
                st(pto<InT>(ddt, oy), dd);
                if (z) st(pto<InT>(dz, oy), yr * s_zf[t][deal.lc]);
                dD = fmaf(dyt, xv, dD);
                dbias += dd;
            }
        }
#pragma unroll
        for (int i = 0; i < 2 * HB; ++i) {                 // part_bc: [token][db, dc][state]
            const int e = tid + i * NT;
            if (t0 + e / (2 * S) >= t_end) continue;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < WC; ++w) v += (&s_g[w][0][0][0])[e];
            part_bc[(int64_t)t0 * 2 * S + e] = v;
        }
        lds_barrier();                                     // the next block overwrites what this one's end reads
    }
    if (used && p.dh0 && on && piece == 0) {
#pragma unroll
        for (int s = 0; s < NS; ++s) p.dh0[((int64_t)n * p.C + ch) * S + n0 + s] = gr[s];
    }
    if (on) {
#pragma unroll
        for (int s = 0; s < NS; ++s) p.part_A[((int64_t)slot * p.C + ch) * S + n0 + s] = dA[s];
    }
    lds_barrier();
    float* s_d = &s_gb[0][0][0];                           // NT / CH threads hold sums of one channel
    s_d[tid] = dD;
    s_d[NT + tid] = dbias;
    lds_barrier();
    if (tid < CH && deal.lon) {
        float u = 0.f, v = 0.f;
#pragma unroll
        for (int i = 0; i < NT / CH; ++i) {
            u += s_d[i * CH + tid];
            v += s_d[NT + i * CH + tid];
        }
        p.part_D[(int64_t)slot * p.C + deal.lch] = u;
        p.part_bias[(int64_t)slot * p.C + deal.lch] = v;
    }
}

// Column sums of `rows` rows of n values.
__global__ __launch_bounds__(256) void sum_kernel(const float* part, int rows, int64_t n, float* out) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n) return;
    float s = 0.f;
    for (int r = 0; r < rows; ++r) s += part[r * n + i];
    out[i] = s;
}

// db and dc of every token in a sequence: sums over the channel blocks of a group.
template <typename InT>
__global__ __launch_bounds__(256) void bc_kernel(ReduceArgs p, int blocks) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, tokens = (int64_t)p.B * p.T;
    if (i >= tokens * p.G * 2 * p.S) return;
    const int e = (int)(i % (2 * p.S)), g = (int)(i / (2 * p.S) % p.G);
    const int64_t t = i / (2 * p.S) / p.G;
    if (p.cu && (t < p.cu[0] || t >= p.cu[p.N])) return;
    const int per = p.G > 1 ? blocks / p.G : blocks;
    float s = 0.f;
    for (int k = 0; k < per; ++k) s += p.part_bc[((int64_t)(g * per + k) * tokens + t) * 2 * p.S + e];
    InT* out = static_cast<InT*>(e < p.S ? p.db : p.dc);
    st(out + (t * p.G + g) * p.S + e % p.S, s);
}

template <typename InT, int WN, int WC>
hipError_t run(const Args& a, hipStream_t s) {
    const int blocks = (a.C + 16 * WC - 1) / (16 * WC);
    hipLaunchKernelGGL((bwd_kernel<InT, WN, WC>), dim3((uint32_t)blocks * a.segs), dim3(64 * WN * WC), 0, s, a, blocks);
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

void sum(const float* part, int rows, int64_t n, float* out, hipStream_t s) {
    if (out) hipLaunchKernelGGL(sum_kernel, dim3((uint32_t)((n + 255) / 256)), dim3(256), 0, s, part, rows, n, out);
}

}  // namespace

hipError_t launch_bwd(const Args& a, bool bf16, hipStream_t s) {
    return bf16 ? pick<uint16_t>(a, s) : pick<float>(a, s);
}

hipError_t launch_reduce(const ReduceArgs& a, bool bf16, hipStream_t s) {
    sum(a.part_A, a.segs, (int64_t)a.C * a.S, a.dA, s);
    sum(a.part_D, a.segs, a.C, a.dD, s);
    sum(a.part_bias, a.segs, a.C, a.ddt_bias, s);
    const int blocks = (a.C + chans(a.S) - 1) / chans(a.S);
    const int64_t n = (int64_t)a.B * a.T * a.G * 2 * a.S;
    const dim3 grid((uint32_t)((n + 255) / 256));
    if (bf16) hipLaunchKernelGGL(bc_kernel<uint16_t>, grid, dim3(256), 0, s, a, blocks);
    else hipLaunchKernelGGL(bc_kernel<float>, grid, dim3(256), 0, s, a, blocks);
    return hipGetLastError();
}

}  // namespace ssm
