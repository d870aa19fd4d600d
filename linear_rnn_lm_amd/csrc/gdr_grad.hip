// gdr_grad.hip -- input gradients of the gated delta rule, all chunks at once
// (gfx950).  From the state S entering a chunk, its written rows U (both left by
// the forward), the gradient G1 at its end and Z = dL/dU's solved form (both
// left by the backward scan), with Lam[t][s] = e^(G_t - G_s):
//
//     P  = lower(scale Lam DO U^T)          N = -b_t strict_lower(Lam Z U^T)
//     dQ = scale e^G DO S + P K
//     dK = [N K - b e^G Z S]  +  [P^T Q + N^T K + e^(G_C - G) U G1]
//     db_t = (Z_t . U_t) / b_t
//     dG_t = q_t . dQ_t + k_t . (first part of dK)_t - k_t . (second part)_t
//     dG_C += sum_t k_t . e^(G_C - G_t) (U G1)_t + e^(G_C) <S, G1>
//     dg_t = sum_{t' >= t} dG_t'
//
// (the decays enter every product as a row or column factor, so their gradients
// are row sums of terms that are there anyway).  q and k of one key head serve
// H / Hk value heads: one workgroup does all of them in turn, so the sums over
// the heads stay in registers and in one order.
#include "gdr_device.h"
#include "gdr_internal.h"
#include "wkv7_internal.h"

namespace gdr {
namespace {

constexpr int NP = kPlanes;
constexpr int NT = 512;

template <int NX>
struct Lds {
    static constexpr int MB = kMatBytes;                  // one plane of a 64 x 64 matrix
    static constexpr int U = 0, Z = U + NP * MB;          // then P, N
    static constexpr int P = U, N = Z;
    static constexpr int S = Z + NP * MB, G = S + NP * MB;
    static constexpr int DO = G + NP * MB;
    static constexpr int after = DO + NX * MB;
    static constexpr bool apart = NX == 1;                // K, Q beside S, G or in their place
    static constexpr int Kr = apart ? after : S, Qr = Kr + NX * MB;
    static constexpr int small = apart ? Qr + NX * MB : after;
    static constexpr int bytes = small + 7 * 64 * 4 + 2 * 128 * 4;
};

// Eight consecutive fp32 values.
struct F8 {
    f32x4 a, b;
};
__device__ __forceinline__ F8 load8(const float* p) {
    return F8{*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 4)};
}
__device__ __forceinline__ void store8(float* p, const F8& v) {
    *reinterpret_cast<f32x4*>(p) = v.a;
    *reinterpret_cast<f32x4*>(p + 4) = v.b;
}
__device__ __forceinline__ void store8(uint16_t* p, const F8& v) {
    const PF<1> f = pf_acc<1>(v.a, v.b);
    *reinterpret_cast<bf16x8*>(p) = f.p[0];
}
// Eight values of an LDS matrix's row, summed over the planes.
template <int NX>
__device__ __forceinline__ F8 get8(const char* X, int row, int unit) {
    const char* p = X + (row * 8 + (unit ^ swz<8>(row))) * 16;
    F8 v{zero4(), zero4()};
#pragma unroll
    for (int i = NX - 1; i >= 0; --i) {
        const bf16x8 x = *reinterpret_cast<const bf16x8*>(p + i * kMatBytes);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            v.a[e] += (float)x[e];
            v.b[e] += (float)x[e + 4];
        }
    }
    return v;
}
__device__ __forceinline__ float dot4(f32x4 a, f32x4 b) {
    return fmaf(a[0], b[0], fmaf(a[1], b[1], fmaf(a[2], b[2], a[3] * b[3])));
}

template <typename InT, int NX, int K>
__global__ __launch_bounds__(NT) void grad_kernel(Args p) {
    using L = Lds<NX>;
    constexpr int KJ = K / 64;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    float* Gn = reinterpret_cast<float*>(smem + L::small);
    float* Gf = Gn + 64;
    float* eG = Gf + 64;
    float* toEnd = eG + 64;
    float* beta = toEnd + 64;
    float* dbeta = beta + 64;
    float* red = dbeta + 64;             // 8 floats used
    float* dGp = red + 64;               // [2][64]
    float* ep = dGp + 128;               // [2][64]
    const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int g4 = lane >> 4, r16 = lane & 15;
    const int slot = blockIdx.x / p.Hk, hk = blockIdx.x % p.Hk, rep = p.H / p.Hk;
    const Seqs seqs{p.cu, p.N, p.T, p.NC};
    int n, len;
    int64_t tok;
    if (!slot_chunk(seqs, slot, n, tok, len)) return;

    const int c = wave & 1, tt = wave >> 1;          // index pair 32c .. + 31, token tile tt
    const int t = idx(tt, r16);                      // this lane's token (as a column of an accumulator)
    const int row8 = tid >> 3, u8 = tid & 7;         // staging: row and unit of a 64 x 64 matrix
    const int V = p.V;

    F8 gq[KJ], gk[KJ];
#pragma unroll
    for (int j = 0; j < KJ; ++j) gq[j] = gk[j] = F8{zero4(), zero4()};

    for (int hr = 0; hr < rep; ++hr) {
        const int h = hk * rep + hr;
        const int64_t block = (int64_t)slot * p.H + h;
        const float* S = p.ckpt + block * p.ckpt_stride;
        const float* Um = S + (int64_t)V * K;
        const float* G1 = p.dend + block * (int64_t)V * K;
        const float* Zm = p.z + block * (int64_t)C * V;
        const float* gates = p.tri + block * p.tri_stride + kTriFloats;
        __syncthreads();
        if (tid < 64) {
            Gn[tid] = gates[kGateN + tid];
            Gf[tid] = gates[kGateF + tid];
            eG[tid] = gates[kGateEG + tid];
            toEnd[tid] = gates[kGateToEnd + tid];
            beta[tid] = gates[kGateBeta + tid];
        }
        if (tid < 128) dGp[tid] = ep[tid] = 0.f;
        float sg = 0.f;

#pragma unroll
        for (int js = 0; js < KJ; ++js) {
            auto put_kq = [&] {
                const int64_t rowk = (tok + min(row8, len - 1)) * p.Hk + hk;
#pragma unroll
                for (int i = 0; i < NX; ++i) {
                    const int64_t o = i * p.kp.plane + rowk * K + 64 * js + 8 * u8;
                    const PF<1> fk{{*reinterpret_cast<const bf16x8*>(p.kp.p + o)}};
                    const PF<1> fq{{*reinterpret_cast<const bf16x8*>(p.qp.p + o)}};
                    put8<8, 1>(smem + L::Kr + i * kMatBytes, 0, row8, u8, fk);
                    put8<8, 1>(smem + L::Qr + i * kMatBytes, 0, row8, u8, fq);
                }
            };
            f32x4 dos[2], zs[2], ug[2], pa[2], na[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) dos[hh] = zs[hh] = ug[hh] = pa[hh] = na[hh] = zero4();
            for (int is = 0; is < V / 64; ++is) {
                const F8 u = load8(Um + (64 * is + row8) * C + 8 * u8);      // rows i, columns t
                const F8 z = load8(Zm + (64 * is + row8) * C + 8 * u8);
                const F8 s = load8(S + (int64_t)(64 * is + row8) * K + 64 * js + 8 * u8);
                const F8 g = load8(G1 + (int64_t)(64 * is + row8) * K + 64 * js + 8 * u8);
                PF<NX> d;
                if constexpr (NX == 1) {
                    d.p[0] = bf16x8{};
                    if (row8 < len)
                        d.p[0] = *reinterpret_cast<const bf16x8*>(static_cast<const uint16_t*>(p.dout) +
                                                                  ((tok + row8) * p.H + h) * V + 64 * is + 8 * u8);
                } else {
                    F8 x{zero4(), zero4()};
                    if (row8 < len)
                        x = load8(static_cast<const float*>(p.dout) + ((tok + row8) * p.H + h) * V + 64 * is + 8 * u8);
                    d = pf_acc<NX>(x.a, x.b);
                }
                sg += dot4(s.a, g.a) + dot4(s.b, g.b);
                __syncthreads();                          // the readers of the last slices are done
                put8<8, NP>(smem + L::U, kMatBytes, row8, u8, pf_acc<NP>(u.a, u.b));
                put8<8, NP>(smem + L::Z, kMatBytes, row8, u8, pf_acc<NP>(z.a, z.b));
                put8<8, NP>(smem + L::S, kMatBytes, row8, u8, pf_acc<NP>(s.a, s.b));
                put8<8, NP>(smem + L::G, kMatBytes, row8, u8, pf_acc<NP>(g.a, g.b));
                put8<8, NX>(smem + L::DO, kMatBytes, row8, u8, d);
                if (L::apart && is == 0) put_kq();
                __syncthreads();
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const PF<NX> df = frag_row<8, NX>(smem + L::DO, kMatBytes, t, ks, lane);
                    const PF<NP> zf = frag_col<8, NP>(smem + L::Z, kMatBytes, tt, ks, lane);
                    const PF<NP> uf = frag_col<8, NP>(smem + L::U, kMatBytes, tt, ks, lane);
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const PF<NP> sf = frag_col<8, NP>(smem + L::S, kMatBytes, 2 * c + hh, ks, lane);
                        const PF<NP> gf = frag_col<8, NP>(smem + L::G, kMatBytes, 2 * c + hh, ks, lane);
                        dos[hh] = pmma<NP>(dos[hh], sf, df);
                        zs[hh] = pmma<NP>(zs[hh], sf, zf);
                        ug[hh] = pmma<NP>(ug[hh], gf, uf);
                        if (c <= (tt >> 1)) {
                            const PF<NP> us = frag_col<8, NP>(smem + L::U, kMatBytes, 2 * c + hh, ks, lane);
                            pa[hh] = pmma<NP>(pa[hh], us, df);
                            na[hh] = pmma<NP>(na[hh], us, zf);
                        }
                    }
                }
            }
            const float bt = beta[t], egt = eG[t], tet = toEnd[t], nt = Gn[t], ft = Gf[t];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int s = 32 * c + 8 * g4 + 4 * hh + q;
                    const float lam = s <= t ? decay(nt, ft, Gn[s], Gf[s]) : 0.f;
                    if (s == t) dbeta[t] = t < len ? na[hh][q] / bt : 0.f;
                    pa[hh][q] = s <= t ? p.scale * lam * pa[hh][q] : 0.f;
                    na[hh][q] = s < t ? -bt * lam * na[hh][q] : 0.f;
                }
            __syncthreads();
            put8<8, NP>(smem + L::P, kMatBytes, t, 4 * c + g4, pf_acc<NP>(pa[0], pa[1]));
            put8<8, NP>(smem + L::N, kMatBytes, t, 4 * c + g4, pf_acc<NP>(na[0], na[1]));
            if (!L::apart) put_kq();
            __syncthreads();
            f32x4 pk[2], nk[2], pq[2];
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) pk[hh] = nk[hh] = pq[hh] = zero4();
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                if (ks <= (tt >> 1)) {
                    const PF<NP> pr = frag_row<8, NP>(smem + L::P, kMatBytes, t, ks, lane);
                    const PF<NP> nr = frag_row<8, NP>(smem + L::N, kMatBytes, t, ks, lane);
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        const PF<NX> kf = frag_col<8, NX>(smem + L::Kr, kMatBytes, 2 * c + hh, ks, lane);
                        pk[hh] = pmma<NP>(pk[hh], kf, pr);
                        nk[hh] = pmma<NP>(nk[hh], kf, nr);
                    }
                }
                if (ks >= (tt >> 1)) {
                    const PF<NP> pc = frag_col<8, NP>(smem + L::P, kMatBytes, tt, ks, lane);
                    const PF<NP> nc = frag_col<8, NP>(smem + L::N, kMatBytes, tt, ks, lane);
#pragma unroll
                    for (int hh = 0; hh < 2; ++hh) {
                        pq[hh] = pmma<NP>(pq[hh], frag_col<8, NX>(smem + L::Qr, kMatBytes, 2 * c + hh, ks, lane), pc);
                        pq[hh] = pmma<NP>(pq[hh], frag_col<8, NX>(smem + L::Kr, kMatBytes, 2 * c + hh, ks, lane), nc);
                    }
                }
            }
            const F8 kv = get8<NX>(smem + L::Kr, t, 4 * c + g4), qv = get8<NX>(smem + L::Qr, t, 4 * c + g4);
            float dG = 0.f, e = 0.f;
#pragma unroll
            for (int hh = 0; hh < 2; ++hh) {
                const f32x4 k4 = hh ? kv.b : kv.a, q4 = hh ? qv.b : qv.a;
                const f32x4 dq = p.scale * egt * dos[hh] + pk[hh];
                const f32x4 plus = nk[hh] - egt * bt * zs[hh];
                const f32x4 end = tet * ug[hh];
                const f32x4 minus = pq[hh] + end;
                dG += dot4(q4, dq) + dot4(k4, plus - minus);
                e += dot4(k4, end);
                if (hh) {
                    gq[js].b += dq;
                    gk[js].b += plus + minus;
                } else {
                    gq[js].a += dq;
                    gk[js].a += plus + minus;
                }
            }
            dG += __shfl_xor(dG, 16);
            e += __shfl_xor(e, 16);
            dG += __shfl_xor(dG, 32);
            e += __shfl_xor(e, 32);
            if (g4 == 0) {                                // one lane per (c, t)
                dGp[c * 64 + t] += dG;
                ep[c * 64 + t] += e;
            }
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) sg += __shfl_xor(sg, d);
        if (lane == 0) red[wave] = sg;
        __syncthreads();
        if (wave == 0) {
            double x = (double)dGp[lane] + dGp[64 + lane];
            float e = ep[lane] + ep[64 + lane];
#pragma unroll
            for (int d = 32; d; d >>= 1) e += __shfl_xor(e, d);
            if (lane == 63) {
                float sgs = 0.f;
#pragma unroll
                for (int i = 0; i < NT / 64; ++i) sgs += red[i];
                x += (double)e + (double)eG[63] * sgs;
            }
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const double o = __shfl_down(x, d);
                if (lane + d < 64) x += o;
            }
            if (lane < len) {
                p.dg[(tok + lane) * p.H + h] = (float)x;
                p.dbeta[(tok + lane) * p.H + h] = dbeta[lane];
            }
        }
    }
    if (t < len) {
#pragma unroll
        for (int js = 0; js < KJ; ++js) {
            const int64_t o = ((tok + t) * p.Hk + hk) * K + 64 * js + 32 * c + 8 * g4;
            store8(static_cast<InT*>(p.dq) + o, gq[js]);
            store8(static_cast<InT*>(p.dk) + o, gk[js]);
        }
    }
}

template <typename InT, int NX, int K>
hipError_t launch_typed(const Args& a, hipStream_t s) {
    static_assert(Lds<NX>::bytes <= 160 * 1024, "gradient LDS");
    auto kern = grad_kernel<InT, NX, K>;
    static wkv7::PerDeviceOnce once;
    const hipError_t e = wkv7::set_smem_once(once, kern, Lds<NX>::bytes);
    if (e != hipSuccess) return e;
    hipLaunchKernelGGL(kern, dim3((uint32_t)a.slots * a.Hk), dim3(NT), Lds<NX>::bytes, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_grad(const Args& a, bool bf16, hipStream_t s) {
    if (bf16) return a.K == 64 ? launch_typed<uint16_t, 1, 64>(a, s) : launch_typed<uint16_t, 1, 128>(a, s);
    return a.K == 64 ? launch_typed<float, 3, 64>(a, s) : launch_typed<float, 3, 128>(a, s);
}

}  // namespace gdr
