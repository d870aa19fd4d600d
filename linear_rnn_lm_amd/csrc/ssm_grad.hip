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
// forward (16 channels by 4 groups of 4 states); sums over states are swaps of lane rows,
// sums over a wave's 16 channels exchanges within them, two tokens' eight values at a time.
// Sums over workgroups (db, dc: one part per 64 channels, 32 with 64 states; dA, dD, ddt_bias: one per
// segment) go through memory and a second launch, in a fixed order.
#include "rows_device.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

using namespace rows;

// Sums over the 16 lanes of a row of 16 values: lane r gets the sum of value r.  Each step
// exchanges the half of the values that the other lane keeps.
__device__ __forceinline__ float row_scatter16(const float (&v)[16], int lane) {
    const bool b8 = lane & 8, b4 = lane & 4, b2 = lane & 2, b1 = lane & 1;
    float p[8], q[4], r[2];
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] = (b8 ? v[i + 8] : v[i]) + dpp<0x128>(b8 ? v[i] : v[i + 8]);   // row_ror:8
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = (b4 ? p[i + 4] : p[i]) + dpp<0x141>(b4 ? p[i] : p[i + 4]);   // half mirror
#pragma unroll
    for (int i = 0; i < 2; ++i) r[i] = (b2 ? q[i + 2] : q[i]) + dpp<0x4E>(b2 ? q[i] : q[i + 2]);    // quad 2,3,0,1
    return (b1 ? r[1] : r[0]) + dpp<0xB1>(b1 ? r[0] : r[1]);                                        // quad 1,0,3,2
}

template <typename InT, int WN, int WC>
__global__ __launch_bounds__(64 * WN * WC) void bwd_kernel(Args p, int blocks) {
    constexpr int NS = 4, S = 4 * NS * WN, CH = 16 * WC, NT = 64 * WN * WC, TB = kBlock;
    constexpr int LT = TB * CH / NT, BC = (2 * TB * S + NT - 1) / NT;
    static_assert(CH == chans(S), "one part of db and dc per workgroup");
    __shared__ float2 s_du[TB][CH];              // delta, delta x
    __shared__ float s_dy[TB][CH], s_bc[2][TB][S];
    __shared__ float s_y[WN][TB][CH], s_gb[WN][TB][CH], s_pa[WN][TB][CH];
    __shared__ float s_g[WC][TB][2][S];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, wn = wave % WN, wc = wave / WN;
    const int cb = blockIdx.x % blocks, slot = blockIdx.x / blocks;
    const Seqs seqs{p.cu, p.N, p.T};
    const int cl = wc * 16 + (lane & 15), g4 = lane >> 4, ch = cb * CH + cl, n0 = (wn * 4 + g4) * NS;
    const bool on = ch < p.C;
    const int lc = tid % CH, lt = tid / CH, lch = cb * CH + lc;
    const bool lon = lch < p.C;
    float A[NS], dA[NS], gr[NS], dD = 0.f, dbias = 0.f;
    int n, piece, len = 0;
    int64_t tok0 = 0;
    const bool used = slot_piece(seqs, slot, p.seg, n, piece);
    if (used) seq_span(seqs, n, tok0, len);
    const int t_begin = used ? piece * p.seg : 0, t_end = used ? min(len, t_begin + p.seg) : 0;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
        A[s] = on ? p.A[(int64_t)ch * S + n0 + s] : 0.f;
        dA[s] = 0.f;
        gr[s] = used && on && p.dhT ? p.dhT[((int64_t)n * p.C + ch) * S + n0 + s] : 0.f;
    }
    const InT* x = static_cast<const InT*>(p.x) + tok0 * p.x_ld + lch;
    const InT* dt = static_cast<const InT*>(p.dt) + tok0 * p.dt_ld + lch;
    const InT* z = p.z ? static_cast<const InT*>(p.z) + tok0 * p.z_ld + lch : nullptr;
    const InT* dy = static_cast<const InT*>(p.dy) + tok0 * p.C + lch;
    InT* dx = static_cast<InT*>(p.dx) + tok0 * p.C + lch;
    InT* ddt = static_cast<InT*>(p.ddt) + tok0 * p.C + lch;
    InT* dz = p.z ? static_cast<InT*>(p.dz) + tok0 * p.C + lch : nullptr;
    const int64_t go = (int64_t)(cb * CH / (p.C / p.G)) * S;
    const InT* b = static_cast<const InT*>(p.b) + tok0 * p.b_ld + go;
    const InT* c = static_cast<const InT*>(p.c) + tok0 * p.c_ld + go;
    const float bias = lon && p.dt_bias ? p.dt_bias[lch] : 0.f, Dv = lon && p.D ? p.D[lch] : 0.f;
    float* part_bc = p.part_bc + ((int64_t)cb * p.B * p.T + tok0) * 2 * S;

    InT rx[LT], rd[LT], rz[LT], ry[LT], rbc[BC];
    float hn[NS];
    const int64_t ck = ((int64_t)(used ? first_slot(seqs, n, tok0, TB) : 0) * p.C + ch) * S + n0;
    auto fetch = [&](int t0) {
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const int t = t0 + lt + i * (NT / CH);
            const bool ok = lon && t < t_end;
            rx[i] = ok ? x[t * p.x_ld] : InT(0);
            rd[i] = ok ? dt[t * p.dt_ld] : InT(0);
            rz[i] = ok && z ? z[t * p.z_ld] : InT(0);
            ry[i] = ok ? dy[(int64_t)t * p.C] : InT(0);
        }
#pragma unroll
        for (int i = 0; i < BC; ++i) {
            const int e = tid + i * NT, t = t0 + e / S % TB;
            rbc[i] = e < 2 * TB * S && t < t_end ? (e < TB * S ? b + t * p.b_ld : c + t * p.c_ld)[e % S] : InT(0);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) hn[s] = on ? p.ckpt[ck + (int64_t)(t0 / TB) * p.C * S + s] : 0.f;
    };
    const int t_last = t_begin < t_end ? t_begin + (t_end - 1 - t_begin) / TB * TB : t_begin - TB;
    if (t_last >= t_begin) fetch(t_last);
    for (int t0 = t_last; t0 >= t_begin; t0 -= TB) {
        float xv[LT], dv[LT], vv[LT], zv[LT], sz[LT], yv[LT], h[NS];
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const int t = lt + i * (NT / CH);
            xv[i] = widen(rx[i]);
            vv[i] = widen(rd[i]) + bias;
            dv[i] = t0 + t < t_end ? (p.softplus ? softplus(vv[i]) : vv[i]) : 0.f;
            zv[i] = widen(rz[i]);
            sz[i] = p.z ? sigmoid(zv[i]) : 1.f;
            yv[i] = widen(ry[i]);
            s_du[t][lc] = make_float2(dv[i], dv[i] * xv[i]);
            s_dy[t][lc] = p.z ? yv[i] * zv[i] * sz[i] : yv[i];
        }
#pragma unroll
        for (int i = 0; i < BC; ++i) {
            const int e = tid + i * NT;
            if (e < 2 * TB * S) (&s_bc[0][0][0])[e] = widen(rbc[i]);
        }
#pragma unroll
        for (int s = 0; s < NS; ++s) h[s] = hn[s];
        lds_barrier();
        if (t0 > t_begin) fetch(t0 - TB);

        float a[TB][NS], ah[TB][NS];
#pragma unroll
        for (int t4 = 0; t4 < TB; t4 += 4) {
            float yt[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = t4 + i;
                const float2 du = s_du[t][cl];
                yt[i] = 0.f;
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    a[t][s] = exp2_f(du.x * (kLog2e * A[s]));
                    ah[t][s] = a[t][s] * h[s];
                    h[s] = fmaf(du.y, s_bc[0][t][n0 + s], ah[t][s]);
                    yt[i] = fmaf(s_bc[1][t][n0 + s], h[s], yt[i]);
                }
            }
            if (p.z) s_y[wn][t4 + row_of(g4)][cl] = rows_sum4(yt[0], yt[1], yt[2], yt[3]);
        }
#pragma unroll
        for (int t4 = TB - 4; t4 >= 0; t4 -= 4) {
            float gb[4], pa[4], v[2][16];
#pragma unroll
            for (int i = 3; i >= 0; --i) {
                const int t = t4 + i;
                const float2 du = s_du[t][cl];
                const float dyt = s_dy[t][cl];
                gb[i] = pa[i] = 0.f;
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const float bt = s_bc[0][t][n0 + s], ct = s_bc[1][t][n0 + s];
                    gr[s] = fmaf(ct, dyt, gr[s]);
                    gb[i] = fmaf(gr[s], bt, gb[i]);
                    const float q = gr[s] * ah[t][s];
                    pa[i] = fmaf(q, A[s], pa[i]);
                    dA[s] = fmaf(q, du.x, dA[s]);
                    v[i >> 1][(i & 1) * 8 + s] = gr[s] * du.y;
                    v[i >> 1][(i & 1) * 8 + 4 + s] = dyt * fmaf(du.y, bt, ah[t][s]);
                    gr[s] *= a[t][s];
                }
            }
            s_gb[wn][t4 + row_of(g4)][cl] = rows_sum4(gb[0], gb[1], gb[2], gb[3]);
            s_pa[wn][t4 + row_of(g4)][cl] = rows_sum4(pa[0], pa[1], pa[2], pa[3]);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                s_g[wc][t4 + 2 * i + ((lane >> 3) & 1)][(lane >> 2) & 1][n0 + (lane & 3)] = row_scatter16(v[i], lane);
        }
        lds_barrier();
#pragma unroll
        for (int i = 0; i < LT; ++i) {
            const int t = lt + i * (NT / CH);
            if (!lon || t0 + t >= t_end) continue;
            float gb = 0.f, pa = 0.f, yr = Dv * xv[i];
#pragma unroll
            for (int w = 0; w < WN; ++w) {
                gb += s_gb[w][t][lc];
                pa += s_pa[w][t][lc];
                if (p.z) yr += s_y[w][t][lc];
            }
            const int64_t o = (int64_t)(t0 + t) * p.C;
            const float dyt = p.z ? yv[i] * zv[i] * sz[i] : yv[i];
            const float dd = fmaf(xv[i], gb, pa) * (p.softplus ? sigmoid(vv[i]) : 1.f);
            st(dx + o, fmaf(dv[i], gb, Dv * dyt));
            st(ddt + o, dd);
            if (p.z) st(dz + o, yv[i] * yr * sz[i] * fmaf(zv[i], 1.f - sz[i], 1.f));
            dD = fmaf(dyt, xv[i], dD);
            dbias += dd;
        }
#pragma unroll
        for (int i = 0; i < BC; ++i) {                     // part_bc: [token][db, dc][state]
            const int e = tid + i * NT, t = t0 + e / (2 * S);
            if (e >= 2 * TB * S || t >= t_end) continue;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < WC; ++w) v += (&s_g[w][0][0][0])[e];
            part_bc[(int64_t)t0 * 2 * S + e] = v;
        }
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
    if (tid < CH && lon) {
        float u = 0.f, v = 0.f;
#pragma unroll
        for (int i = 0; i < NT / CH; ++i) {
            u += s_d[i * CH + tid];
            v += s_d[NT + i * CH + tid];
        }
        p.part_D[(int64_t)slot * p.C + lch] = u;
        p.part_bias[(int64_t)slot * p.C + lch] = v;
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
