// gdr_grad.hip -- input gradients of the gated delta rule, all chunks at once
// (gfx950).  From the state S entering a chunk, its written rows U (both left by
// the forward), the gradient G1 at its end and Z = dL/dU's solved form (both
// left by the backward scan), with Lam[t][s] = e^(G_t - G_s):
//
//     P  = lower(scale Lam DO U^T)          N = -b_t strict_lower(Lam Z U^T)
//     dQ = scale e^G DO S + P K
//     dK = [N K - b e^G Z S]  +  [P^T Q + N^T K + e^(G_C - G) U G1]
//     db_t = (Z_t . U_t) / b_t
//     dg_j = sum_{s < j <= t} W[t][s] + sum_{t >= j} a_t + sum_{s < j} e_s + e^(G_C) <S, G1>
//       W[t][s] = P[t][s] q_t . k_s + N[t][s] k_t . k_s,   e_s = k_s . e^(G_C - G_s) (U G1)_s
//       a_t = q_t . scale e^G (dO S)_t - k_t . b e^G (Z S)_t
//
// Each term of dg_j is one that the decay of token j enters, once, as a factor.  (Suffix
// sums of q.dQ and k.dK would need no W, but undecayed terms, the diagonal of P and the end
// terms of later tokens, come and go in them: with log decays of -5 dg was off by 6e-5 to 1e-4
// of itself, with -10 by 1e-2, with -20 it had no digit left.)  The sum over s < j is a
// prefix along a lane's eight s and the lanes that hold a row, the sum over t >= j one over
// the lanes of a tile.  q and k of one key head serve H / Hk value heads: one workgroup does
// all of them in turn, so the sums over the heads stay in registers and in one order.
//
// It reads S, U, G1, Z, q, k and dout and writes dq and dk: 1.83 GB at B8 T4096 H32 64 x 64,
// 360 us at the rate of a large copy; it takes 490 to 510 (the splitting into planes
// and the products overlap the loads of the other workgroup on the unit, not wholly).
// K = 128 takes a workgroup for either half of the columns: with one for both, 8200 packed
// tokens of 8 key and 16 value heads made 2.1 rounds of the chip's 512 and 232 us, with
// 4.3 rounds of half the work 207 (213 since dg has W).
#include "gdr_device.h"
#include "gdr_internal.h"
#include "wkv7_internal.h"

namespace gdr {
namespace {

constexpr int NP = kPlanes;
constexpr int NT = 512;

// LDS plan.  The rows i of U, Z (V x 64 each), S and G1 are taken 32 at a time, which
// keeps a workgroup at half a compute unit's LDS for bf16 inputs, so that the loads,
// the splitting and the products of two workgroups overlap.  P and N take
// the place of U, Z, S, G1 once those are used up.
template <int NX>
struct Lds {
    static constexpr int MB = kMatBytes, HB = kMatBytes / 2;   // one plane of 64 x 64, of 32 x 64
    static constexpr int U = 0, Z = U + NP * HB, S = Z + NP * HB, G = S + NP * HB;
    static constexpr int P = 0, N = P + NP * MB;
    static constexpr int DO = G + NP * HB, Kr = DO + NX * MB, Qr = Kr + NX * MB;
    static constexpr int small = Qr + NX * MB;
    static constexpr int bytes = small + 8 * 64 * 4 + 2 * 128 * 4 + 256 * 4;
    static_assert(N + NP * MB <= DO, "P and N in place of U, Z, S, G1");
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
template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, false));
}
// Eight sums over the 16 lanes of a row: lane r gets that of x[r / 2].  Each step halves the
// values and the lanes that a value is spread over.
__device__ __forceinline__ float row_sums8(const float (&x)[8], int r) {
    float y[4], z[2];
#pragma unroll
    for (int i = 0; i < 4; ++i)                           // row_mirror
        y[i] = (r & 8 ? x[4 + i] : x[i]) + dpp<0x140>(r & 8 ? x[i] : x[4 + i]);
#pragma unroll
    for (int i = 0; i < 2; ++i)                           // row_half_mirror
        z[i] = (r & 4 ? y[2 + i] : y[i]) + dpp<0x141>(r & 4 ? y[i] : y[2 + i]);
    const float w = (r & 2 ? z[1] : z[0]) + dpp<0x4E>(r & 2 ? z[0] : z[1]);   // quad_perm 2,3,0,1
    return w + dpp<0xB1>(w);                              // quad_perm 1,0,3,2
}

// ONE: one value head to a key head, so nothing is summed over heads.
template <typename InT, int NX, int K, bool ONE>
__global__ __launch_bounds__(NT, NX == 1 ? 4 : 2) void grad_kernel(Args p) {
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
    float* rest = red + 64;              // row sums of W over s < 32
    float* ap = rest + 64;               // [2][64]
    float* ep = ap + 128;                // [2][64]
    float* wp = ep + 128;                // [tile of t][s]
    const int tid0 = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid0 >> 6);
    // K = 128: two workgroups, one for either half js of the columns, eight apart in the launch's order, so
    // that they are on one XCD and share U and Z in its L2
    const int js = KJ == 1 ? 0 : blockIdx.x / 8 % KJ, work = KJ == 1 ? blockIdx.x : blockIdx.x / (8 * KJ) * 8 + blockIdx.x % 8;
    const int slot = work / p.Hk, hk = work % p.Hk, rep = ONE ? 1 : p.H / p.Hk;
    if (slot >= p.slots) return;
    const Seqs seqs{p.cu, p.N, p.T, p.NC};
    int n, len;
    int64_t tok;
    if (!slot_chunk(seqs, slot, n, tok, len)) return;

    // A wave takes one tile tt of 16 tokens (its lanes' columns) and 32 of a slice's 64
    // columns j (its accumulators' rows).
    const int c = wave & 1, tt = wave >> 1;
    const int V = p.V;

    F8 gq{zero4(), zero4()}, gk{zero4(), zero4()};
    for (int hr = 0; hr < rep; ++hr) {
        // The thread's number is made opaque in every round, or the loops' many LDS
        // addresses, all functions of it, are kept in registers that are not there.
        int tid = tid0;
        asm volatile("" : "+v"(tid));
        const int lane = tid & 63, g4 = lane >> 4, r16 = lane & 15, t = idx(tt, r16);
        // staging: the first half of the threads moves U and Z, the second S and G1, one row of
        // 32 and unit of eight values each; of 64 x 64 matrices every thread moves one unit
        const bool second = wave >= 4;
        const int row8 = (tid & 255) >> 3, u8 = tid & 7, row64 = tid >> 3;
        auto store = [&](const F8& q, const F8& k) {
            if (t < len) {
                const int64_t o = ((tok + t) * p.Hk + hk) * K + 64 * js + 32 * c + 8 * g4;
                store8(static_cast<InT*>(p.dq) + o, q);
                store8(static_cast<InT*>(p.dk) + o, k);
            }
        };
        const int h = hk * rep + hr;
        const int64_t block = (int64_t)slot * p.H + h;
        const float* ck = p.ckpt + block * p.ckpt_stride;           // S (V x K), U (V x 64)
        const float* gates = p.tri + block * p.tri_stride + kTriFloats;
        float sg = 0.f;
        {
            // this thread's two of the four matrices, and how far apart their rows are
            const float* src0 = second ? ck + (int64_t)row8 * K + 64 * js + 8 * u8
                                       : ck + (int64_t)V * K + row8 * C + 8 * u8;
            const float* src1 = second ? p.dend + block * (int64_t)V * K + (int64_t)row8 * K + 64 * js + 8 * u8
                                       : p.z + block * (int64_t)C * V + row8 * C + 8 * u8;
            const int step = second ? K : C;
            F8 x0 = load8(src0), x1 = load8(src1);    // the next 32 rows, on their way (ONE; else no registers are left)
            PF<NX> kx, qx;
            const int64_t rowk = ((tok + min(row64, len - 1)) * p.Hk + hk) * K + 64 * js + 8 * u8;
#pragma unroll
            for (int i = 0; i < NX; ++i) {
                kx.p[i] = *reinterpret_cast<const bf16x8*>(p.kp.p + i * p.kp.plane + rowk);
                qx.p[i] = *reinterpret_cast<const bf16x8*>(p.qp.p + i * p.qp.plane + rowk);
            }
            float gate = 0.f;
            if (tid < kGateFloats) gate = gates[tid];
            f32x4 dos[2], zs[2], ug[2], pa[2], na[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) dos[j] = zs[j] = ug[j] = pa[j] = na[j] = zero4();
            for (int i0 = 0; i0 < V; i0 += 32) {
                PF<NX> d;
                if (i0 % 64 == 0) {                   // 64 columns of dout, for two rounds
                    const int64_t o = ((tok + min(row64, len - 1)) * p.H + h) * V + i0 + 8 * u8;
                    if constexpr (NX == 1) {
                        d.p[0] = *reinterpret_cast<const bf16x8*>(static_cast<const uint16_t*>(p.dout) + o);
                        if (row64 >= len) d.p[0] = bf16x8{};
                    } else {
                        F8 x = load8(static_cast<const float*>(p.dout) + o);
                        if (row64 >= len) x = F8{zero4(), zero4()};
                        d = pf_acc<NX>(x.a, x.b);
                    }
                }
                if (!ONE && i0 > 0) {
                    x0 = load8(src0 + (int64_t)i0 * step);
                    x1 = load8(src1 + (int64_t)i0 * step);
                }
                if (second) sg += dot4(x0.a, x1.a) + dot4(x0.b, x1.b);
                __syncthreads();                      // the readers of what lay here are done
                put8<8, NP>(smem + (second ? L::S : L::U), L::HB, row8, u8, pf_acc<NP>(x0.a, x0.b));
                put8<8, NP>(smem + (second ? L::G : L::Z), L::HB, row8, u8, pf_acc<NP>(x1.a, x1.b));
                if (i0 % 64 == 0) put8<8, NX>(smem + L::DO, L::MB, row64, u8, d);
                if (i0 == 0) {
                    put8<8, NX>(smem + L::Kr, L::MB, row64, u8, kx);
                    put8<8, NX>(smem + L::Qr, L::MB, row64, u8, qx);
                    if (tid < kGateFloats) {          // in the order e^G, e^(G_C - G), b, n, f
                        float* to = tid < 64 ? eG : tid < 128 ? toEnd - 64 : tid < 192 ? beta - 128 : tid < 256 ? Gn - 192 : Gf - 256;
                        to[tid] = gate;
                    }
                }
                if (ONE && i0 + 32 < V) {
                    x0 = load8(src0 + (int64_t)(i0 + 32) * step);
                    x1 = load8(src1 + (int64_t)(i0 + 32) * step);
                }
                __syncthreads();
                const PF<NX> df = frag_row<8, NX>(smem + L::DO, L::MB, t, (i0 >> 5) & 1, lane);
                const PF<NP> zf = frag_col<8, NP>(smem + L::Z, L::HB, tt, 0, lane);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const PF<NP> sf = frag_col<8, NP>(smem + L::S, L::HB, 2 * c + j, 0, lane);
                    dos[j] = pmma<NP>(dos[j], sf, df);
                    zs[j] = pmma<NP>(zs[j], sf, zf);
                }
                if (c <= (tt >> 1)) {                 // tokens s of 32 c .. + 31 at or before t
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const PF<NP> us = frag_col<8, NP>(smem + L::U, L::HB, 2 * c + j, 0, lane);
                        pa[j] = pmma<NP>(pa[j], us, df);
                        na[j] = pmma<NP>(na[j], us, zf);
                    }
                }
                const PF<NP> uf = frag_col<8, NP>(smem + L::U, L::HB, tt, 0, lane);
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    ug[j] = pmma<NP>(ug[j], frag_col<8, NP>(smem + L::G, L::HB, 2 * c + j, 0, lane), uf);
            }
            const float bt = beta[t], egt = eG[t], tet = toEnd[t], nt = Gn[t], ft = Gf[t];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int s0 = 32 * c + 8 * g4 + 4 * j;
                const f32x4 ns = *reinterpret_cast<const f32x4*>(Gn + s0), fs = *reinterpret_cast<const f32x4*>(Gf + s0);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int s = s0 + q;
                    const float lam = s <= t ? decay(nt, ft, ns[q], fs[q]) : 0.f;
                    if (s == t) dbeta[t] = t < len ? na[j][q] / bt : 0.f;
                    pa[j][q] = s <= t ? p.scale * lam * pa[j][q] : 0.f;
                    na[j][q] = s < t ? -bt * lam * na[j][q] : 0.f;
                }
            }
            if (c <= (tt >> 1)) {                     // W, and for every s its sums over t > s of sum_{s' <= s} W[t][s']
                f32x4 qk[2], kk[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) qk[j] = kk[j] = zero4();
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    const PF<NX> qt = frag_row<8, NX>(smem + L::Qr, L::MB, t, ks, lane);
                    const PF<NX> kt = frag_row<8, NX>(smem + L::Kr, L::MB, t, ks, lane);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const PF<NX> kf = frag_row<8, NX>(smem + L::Kr, L::MB, idx(2 * c + j, r16), ks, lane);
                        qk[j] = pmma<NX>(qk[j], kf, qt);
                        kk[j] = pmma<NX>(kk[j], kf, kt);
                    }
                }
                const int s0 = 32 * c + 8 * g4;
                float x[8], sum = 0.f;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const int j = e / 4, q = e % 4;
                    if (s0 + e < t) sum += pa[j][q] * qk[j][q] + na[j][q] * kk[j][q];
                    x[e] = sum;
                }
                const float by16 = __shfl_xor(sum, 16), pair = sum + by16, by32 = __shfl_xor(pair, 32);
                const float before = (g4 & 1 ? by16 : 0.f) + (g4 & 2 ? by32 : 0.f);
                if (c == 0 && g4 == 0) rest[t] = pair + by32;
#pragma unroll
                for (int e = 0; e < 8; ++e) x[e] = s0 + e < t ? x[e] + before : 0.f;
                const float w = row_sums8(x, r16);
                if (!(r16 & 1)) wp[64 * tt + s0 + (r16 >> 1)] = w;
            }
            __syncthreads();
            put8<8, NP>(smem + L::P, L::MB, t, 4 * c + g4, pf_acc<NP>(pa[0], pa[1]));
            put8<8, NP>(smem + L::N, L::MB, t, 4 * c + g4, pf_acc<NP>(na[0], na[1]));
            __syncthreads();
            const F8 kv = get8<NX>(smem + L::Kr, t, 4 * c + g4), qv = get8<NX>(smem + L::Qr, t, 4 * c + g4);
            float a = 0.f, e = 0.f;
            f32x4 dk[2];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const f32x4 k4 = j ? kv.b : kv.a, q4 = j ? qv.b : qv.a, zt = egt * bt * zs[j], end = tet * ug[j];
                dos[j] = p.scale * egt * dos[j];      // then + P K
                a += dot4(q4, dos[j]) - dot4(k4, zt);
                e += dot4(k4, end);
                dk[j] = end - zt;                     // then + P^T Q + N^T K + N K
            }
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                if (ks <= (tt >> 1)) {
                    const PF<NP> pr = frag_row<8, NP>(smem + L::P, L::MB, t, ks, lane);
                    const PF<NP> nr = frag_row<8, NP>(smem + L::N, L::MB, t, ks, lane);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const PF<NX> kf = frag_col<8, NX>(smem + L::Kr, L::MB, 2 * c + j, ks, lane);
                        dos[j] = pmma<NP>(dos[j], kf, pr);
                        dk[j] = pmma<NP>(dk[j], kf, nr);
                    }
                }
                if (ks >= (tt >> 1)) {
                    const PF<NP> pc = frag_col<8, NP>(smem + L::P, L::MB, tt, ks, lane);
                    const PF<NP> nc = frag_col<8, NP>(smem + L::N, L::MB, tt, ks, lane);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        dk[j] = pmma<NP>(dk[j], frag_col<8, NX>(smem + L::Qr, L::MB, 2 * c + j, ks, lane), pc);
                        dk[j] = pmma<NP>(dk[j], frag_col<8, NX>(smem + L::Kr, L::MB, 2 * c + j, ks, lane), nc);
                    }
                }
            }
            if constexpr (ONE) {
                store(F8{dos[0], dos[1]}, F8{dk[0], dk[1]});
            } else {
                gq.a += dos[0];
                gq.b += dos[1];
                gk.a += dk[0];
                gk.b += dk[1];
                if (hr == rep - 1) store(gq, gk);
            }
            a += __shfl_xor(a, 16);
            e += __shfl_xor(e, 16);
            a += __shfl_xor(a, 32);
            e += __shfl_xor(e, 32);
            if (g4 == 0) {                            // one lane per (c, t)
                ap[c * 64 + t] = a;
                ep[c * 64 + t] = e;
            }
        }
#pragma unroll
        for (int d = 32; d; d >>= 1) sg += __shfl_xor(sg, d);
        if (lane == 0) red[wave] = sg;
        __syncthreads();
        if (wave == 0) {
            // token `lane`: a_t and, where s < 32 lies left of what wp holds for it, whole rows of those s, from
            // itself on; e_s before itself; <S, G1>; W's sums
            float a = ap[lane] + ap[64 + lane], r = lane > 32 ? rest[lane] : 0.f;
            float e = lane > 0 ? ep[lane - 1] + ep[63 + lane] : 0.f, x = 0.f;
#pragma unroll
            for (int i = 0; i < NT / 64; ++i) x += red[i];
            x *= eG[63];
            if (lane > 0) {
                if (lane <= 32) x += wp[lane - 1] + wp[64 + lane - 1];   // tiles of t below 32 have no s from 32 on
                x += wp[128 + lane - 1] + wp[192 + lane - 1];
            }
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const float ad = __shfl_down(a, d), rd = __shfl_down(r, d), eu = __shfl_up(e, d);
                a += lane + d < 64 ? ad : 0.f;
                r += lane + d < 64 ? rd : 0.f;
                e += lane >= d ? eu : 0.f;
            }
            x += a + e + (lane > 32 ? r : 0.f);
            if (lane < len) {
                float* dg = p.dg + (tok + lane) * p.H + h;
                // two halves, added to the zero that the scan left: the order makes no difference to a sum of two
                if (KJ > 1) unsafeAtomicAdd(dg, x);
                else *dg = x;
                if (js == 0) p.dbeta[(tok + lane) * p.H + h] = dbeta[lane];
            }
        }
        if (!ONE) __syncthreads();                    // wave 0 reads what the next round overwrites
    }
}

template <typename InT, int NX, int K, bool ONE>
hipError_t launch_typed(const Args& a, hipStream_t s) {
    static_assert(Lds<NX>::bytes <= 160 * 1024, "gradient LDS");
    auto kern = grad_kernel<InT, NX, K, ONE>;
    static wkv7::PerDeviceOnce once;
    const hipError_t e = wkv7::set_smem_once(once, kern, Lds<NX>::bytes);
    if (e != hipSuccess) return e;
    const uint32_t n = (uint32_t)a.slots * a.Hk;
    hipLaunchKernelGGL(kern, dim3(K == 64 ? n : (n + 7) / 8 * 16), dim3(NT), Lds<NX>::bytes, s, a);
    return hipGetLastError();
}

template <bool ONE>
hipError_t launch_k(const Args& a, bool bf16, hipStream_t s) {
    if (bf16) return a.K == 64 ? launch_typed<uint16_t, 1, 64, ONE>(a, s) : launch_typed<uint16_t, 1, 128, ONE>(a, s);
    return a.K == 64 ? launch_typed<float, 3, 64, ONE>(a, s) : launch_typed<float, 3, 128, ONE>(a, s);
}

}  // namespace

hipError_t launch_grad(const Args& a, bool bf16, hipStream_t s) {
    return a.H == a.Hk ? launch_k<true>(a, bf16, s) : launch_k<false>(a, bf16, s);
}

}  // namespace gdr
