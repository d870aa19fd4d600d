// rnorm.hip -- the fused end of a block, forward and backward (gfx950):
//     r = res + scale act(gate) (norm1(o) weight + bias),   h = norm2(r) weight2 + bias2
//
// Bound by HBM: a row's o, gate and res are read once and stay in registers for both norms.
// A row belongs to a team of L lanes (part of a wave, a wave or a workgroup), NV vectors of
// VEC values per lane; a team walks rows with the sums for the five weights' gradients in
// registers, in the forward with its weights too; the backward has those in LDS, and the next
// row's values on their way while it works on one.  A part of norm1 is 8 to 64
// neighbouring lanes of one vector, so its sums are exchanges within a wave.  The backward
// forms r again from what the forward read (res costs what r would), unrounded.
//
// 32768 rows of 2048 channels, 32 parts, fp32 o, the rest bf16: forward 150 us (5.4 TB/s), backward
// 280 us (4.8 TB/s).  Rows of more than 4096 channels are the exception: a lane of 1024 has half the
// registers, the backward spills some and takes three times what its bytes take.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "abi_checks.h"
#include "column_sums.h"
#include "rnorm.h"
#include "rows_device.h"
#include "wkv7_internal.h"

namespace resnorm {
namespace {

using namespace rows;
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
using wkv7::bf16x8;

struct Args {
    const void *o, *gate, *res, *weight, *bias, *scale, *weight2, *bias2, *dr, *dh;
    void *r, *h, *do_, *dgate, *dres;
    float *stats, *part;
    int64_t rows, gate_ld;
    float eps, eps2;
    int C, G, lanes;           // lanes of a part of norm1 (parts of a whole row: 0)
    int norm, norm2, act;
    bool obf, iobf, rbf, wbf;  // which types are bf16
};

// VEC values of either type; the type is the same for a whole launch.
template <int VEC>
__device__ __forceinline__ void load(const void* base, int64_t at, bool bf, float (&v)[VEC]) {
    if (bf) {
        const uint16_t* p = static_cast<const uint16_t*>(base) + at;
        if constexpr (VEC == 8) {
            const u32x4 u = *reinterpret_cast<const u32x4*>(p);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[2 * e] = __uint_as_float(u[e] << 16);
                v[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
            }
        } else {
            v[0] = ld(p);
        }
    } else {
        const float* p = static_cast<const float*>(base) + at;
        if constexpr (VEC == 8) {
            const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                v[e] = a[e];
                v[4 + e] = b[e];
            }
        } else {
            v[0] = *p;
        }
    }
}
template <int VEC>
__device__ __forceinline__ void store(void* base, int64_t at, bool bf, const float (&v)[VEC]) {
    if (bf) {
        uint16_t* p = static_cast<uint16_t*>(base) + at;
        if constexpr (VEC == 8) {
            bf16x8 o;
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = (__bf16)v[e];
            *reinterpret_cast<bf16x8*>(p) = o;
        } else {
            st(p, v[0]);
        }
    } else {
        float* p = static_cast<float*>(base) + at;
        if constexpr (VEC == 8) {
            *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
            *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
        } else {
            *p = v[0];
        }
    }
}

// Sum over groups of `lanes` (8, 16, 32 or 64) neighbouring lanes, in every lane: each step adds
// the same two numbers in both lanes of a pair.
__device__ __forceinline__ float lane_sum(float x, int lanes) {
    x += dpp<0xB1>(x);                                     // quad 1,0,3,2
    x += dpp<0x4E>(x);                                     // quad 2,3,0,1
    x += dpp<0x141>(x);                                    // half row mirror
    if (lanes >= 16) x += dpp<0x140>(x);                   // row mirror
    if (lanes >= 32) {
        const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(h[0]) + __uint_as_float(h[1]);
    }
    if (lanes >= 64) {
        const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(h[0]) + __uint_as_float(h[1]);
    }
    return x;
}

template <int L>
constexpr int threads() { return L >= 128 ? L : 256; }

// Sum over a team.  Workgroup-wide teams go through LDS, four buffers in turn: a buffer is
// written again only after three other sums, so after barriers that every wave's reads precede.
template <int L>
struct TeamSum {
    float (*red)[16];
    int turn = 0;
    __device__ __forceinline__ explicit TeamSum(float (*r)[16]) : red(r) {}
    __device__ __forceinline__ float operator()(float x) {
        x = lane_sum(x, L < 64 ? L : 64);
        if constexpr (L > 64) {
            turn = (turn + 1) & 3;
            if ((threadIdx.x & 63) == 0) red[turn][threadIdx.x >> 6] = x;
            lds_barrier();
            x = 0.f;
#pragma unroll
            for (int i = 0; i < L / 64; ++i) x += red[turn][i];
        }
        return x;
    }
};

// Sums of s[i] over norm1's parts, in every lane of a part; a whole row's is one number.
template <int L, int NV>
__device__ __forceinline__ void part_sums(float (&s)[NV], int lanes, TeamSum<L>& team) {
    if (lanes) {
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = lane_sum(s[i], lanes);
    } else {
        float x = s[0];
#pragma unroll
        for (int i = 1; i < NV; ++i) x += s[i];
        x = team(x);
#pragma unroll
        for (int i = 0; i < NV; ++i) s[i] = x;
    }
}

__device__ __forceinline__ float act_of(int act, float g) {
    const float s = sigmoid(g);
    return act == RN_SILU ? g * s : s;
}
__device__ __forceinline__ float slope_of(int act, float g) {
    const float s = sigmoid(g);
    return act == RN_SILU ? s * fmaf(g, 1.f - s, 1.f) : s * (1.f - s);
}

template <int VEC>
__device__ __forceinline__ void load_w(const Args& p, const void* w, int c, float dflt, float (&v)[VEC]) {
    if (w) {
        load<VEC>(w, c, p.wbf, v);
    } else {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = dflt;
    }
}

template <int VEC, int L, int NV>
__global__ __launch_bounds__(threads<L>()) void fwd_kernel(Args p, int64_t step) {
    __shared__ float red[4][16];
    const int lane = threadIdx.x % L;
    int64_t row = ((int64_t)blockIdx.x * threads<L>() + threadIdx.x) / L;
    TeamSum<L> team(red);
    int c[NV];
    bool on[NV];
    float w1[NV][VEC], b1[NV][VEC], sc[NV][VEC], w2[NV][VEC], b2[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        c[i] = (i * L + lane) * VEC;
        on[i] = c[i] < p.C;
        if (!on[i]) continue;
        load_w<VEC>(p, p.weight, c[i], 1.f, w1[i]);
        load_w<VEC>(p, p.bias, c[i], 0.f, b1[i]);
        load_w<VEC>(p, p.scale, c[i], 1.f, sc[i]);
        load_w<VEC>(p, p.weight2, c[i], 1.f, w2[i]);
        load_w<VEC>(p, p.bias2, c[i], 0.f, b2[i]);
    }
    const float inv1 = 1.f / (float)(p.C / p.G), inv2 = 1.f / (float)p.C;
    for (; row < p.rows; row += step) {
        const int64_t at = row * p.C;
        float v[NV][VEC], a[NV][VEC], r[NV][VEC], m[NV], q[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            m[i] = q[i] = 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                v[i][e] = r[i][e] = 0.f;
                a[i][e] = 1.f;
            }
            if (!on[i]) continue;
            load<VEC>(p.o, at + c[i], p.obf, v[i]);
            if (p.gate) load<VEC>(p.gate, row * p.gate_ld + c[i], p.iobf, a[i]);
            if (p.res) load<VEC>(p.res, at + c[i], p.rbf, r[i]);
        }
        if (p.norm == RN_LAYER) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) m[i] += v[i][e];
            part_sums<L, NV>(m, p.lanes, team);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            m[i] *= inv1;
            if (on[i])
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    v[i][e] -= m[i];
                    q[i] = fmaf(v[i][e], v[i][e], q[i]);
                }
        }
        part_sums<L, NV>(q, p.lanes, team);
        float m2 = 0.f, q2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            q[i] = 1.f / sqrtf(fmaf(q[i], inv1, p.eps));
            if (!on[i]) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                float u = fmaf(v[i][e] * q[i], w1[i][e], b1[i][e]);
                if (p.gate) u *= act_of(p.act, a[i][e]);
                r[i][e] = fmaf(sc[i][e], u, r[i][e]);
                m2 += r[i][e];
            }
            store<VEC>(p.r, at + c[i], p.rbf, r[i]);
            if (p.stats) {
                // one lane of each part writes its statistics
                float* s = p.stats + row * (2 * p.G + 2);
                const int part = p.lanes ? c[i] / (8 * p.lanes) : 0;
                if (p.lanes ? lane % p.lanes == 0 : i == 0 && lane == 0) {
                    s[part] = m[i];
                    s[p.G + part] = q[i];
                }
            }
        }
        if (p.norm2 == RN_NONE) continue;
        m2 = p.norm2 == RN_LAYER ? team(m2) * inv2 : 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (on[i])
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    r[i][e] -= m2;
                    q2 = fmaf(r[i][e], r[i][e], q2);
                }
        q2 = 1.f / sqrtf(fmaf(team(q2), inv2, p.eps2));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!on[i]) continue;
#pragma unroll
            for (int e = 0; e < VEC; ++e) r[i][e] = fmaf(r[i][e] * q2, w2[i][e], b2[i][e]);
            store<VEC>(p.h, at + c[i], p.iobf, r[i]);
        }
        if (p.stats && lane == 0) {
            p.stats[row * (2 * p.G + 2) + 2 * p.G] = m2;
            p.stats[row * (2 * p.G + 2) + 2 * p.G + 1] = q2;
        }
    }
}

// With oh, rh the normalised o and r, a = act(gate), u = oh weight + bias:
//     dr' = dr + rstd2 (e2 - mean(e2) - rh mean(e2 rh)),  e2 = dh weight2       (= dres)
//     du = dr' scale a,  dgate = dr' scale u act'(gate),  e1 = du weight
//     do = rstd1 (e1 - mean(e1) - oh mean(e1 oh))                              (means over a part)
// and over the rows dweight = sum du oh, dbias = sum du, dscale = sum dr' a u, dweight2 = sum dh
// rh, dbias2 = sum dh; a root-mean-square norm has no mean(e).
// VEC values as stored, of either type, widened at their use, so that the next row's loads do not
// wait where they are issued.
template <int VEC>
struct Raw {
    u32x4 v[VEC == 8 ? 2 : 1];
    __device__ __forceinline__ void load(const void* base, int64_t at, bool bf) {
        if constexpr (VEC == 8) {
            const char* p = static_cast<const char*>(base) + at * (bf ? 2 : 4);
            v[0] = reinterpret_cast<const u32x4*>(p)[0];
            if (!bf) v[1] = reinterpret_cast<const u32x4*>(p)[1];
        } else {
            v[0][0] = bf ? (uint32_t)static_cast<const uint16_t*>(base)[at] << 16 : static_cast<const uint32_t*>(base)[at];
        }
    }
    __device__ __forceinline__ void widen(bool bf, float (&o)[VEC]) const {
        if constexpr (VEC == 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
                o[e] = __uint_as_float(bf ? e % 2 ? v[0][e / 2] & 0xffff0000u : v[0][e / 2] << 16 : v[e / 4][e % 4]);
        } else {
            o[0] = __uint_as_float(v[0][0]);
        }
    }
};

// A row's weights lie in LDS as fp32 (weight, bias, scale, weight2), vectors of 8 in two planes of four so
// that neighbouring lanes' accesses are neighbours: they would be 32 registers for each vector.
template <int VEC>
__device__ __forceinline__ void lds_w(const float* s_w, int C, int k, int c, float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        const f32x4 a = *reinterpret_cast<const f32x4*>(s_w + k * C + c / 2);
        const f32x4 b = *reinterpret_cast<const f32x4*>(s_w + k * C + C / 2 + c / 2);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
    } else {
        v[0] = s_w[k * C + c];
    }
}

template <int VEC, int L, int NV>
__global__ __launch_bounds__(threads<L>(), NV * VEC > 8 ? 1 : L > 512 ? 4 : 2) void bwd_kernel(Args p, int64_t step) {
    __shared__ float red[4][16];
    extern __shared__ __attribute__((aligned(16))) float s_mem[];     // the weights; in the end the teams' sums
    const int lane = threadIdx.x % L;
    TeamSum<L> team(red);
    for (int q = threadIdx.x; q < p.C; q += threads<L>()) {
        const int to = VEC == 8 ? (q % 8 / 4) * (p.C / 2) + q / 8 * 4 + q % 4 : q;
        const void* w[4] = {p.weight, p.bias, p.scale, p.weight2};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float v[1];
            load_w<1>(p, w[k], q, k == 1 ? 0.f : 1.f, v);
            s_mem[k * p.C + to] = v[0];
        }
    }
    __syncthreads();
    int c[NV];
    bool on[NV];
    float acc[5][NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        c[i] = (i * L + lane) * VEC;
        on[i] = c[i] < p.C;
#pragma unroll
        for (int e = 0; e < VEC; ++e)
#pragma unroll
            for (int k = 0; k < 5; ++k) acc[k][i][e] = 0.f;
    }
    const float inv1 = 1.f / (float)(p.C / p.G), inv2 = 1.f / (float)p.C;
    constexpr bool AHEAD = NV == 1 && L <= 512; // the next row on its way while this one is worked on
    Raw<VEC> ro[NV], rg[NV], rr[NV], rd[NV], ry[NV];
    float nm[NV], nrs[NV], nm2 = 0.f, nrs2 = 0.f;
    auto fetch = [&](int64_t row) {
        const int64_t at = row * p.C;
        const float* stat = p.stats + row * (2 * p.G + 2);
        nm2 = stat[2 * p.G], nrs2 = stat[2 * p.G + 1];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!on[i]) continue;
            const int part = p.lanes ? c[i] / (8 * p.lanes) : 0;
            nm[i] = stat[part], nrs[i] = stat[p.G + part];
            ro[i].load(p.o, at + c[i], p.obf);
            if (p.gate) rg[i].load(p.gate, row * p.gate_ld + c[i], p.iobf);
            if (p.dr) rd[i].load(p.dr, at + c[i], p.rbf);
            if (p.dh) ry[i].load(p.dh, at + c[i], p.iobf);
            if (p.dh && p.res) rr[i].load(p.res, at + c[i], p.rbf);
        }
    };
    int64_t row = ((int64_t)blockIdx.x * threads<L>() + threadIdx.x) / L;
    if (AHEAD && row < p.rows) fetch(row);
    for (; row < p.rows; row += step) {
        const int64_t at = row * p.C;
        if (!AHEAD) fetch(row);
        float oh[NV][VEC], g[NV][VEC], d[NV][VEC], y[NV][VEC], r[NV][VEC], rs[NV], w1[VEC], b1[VEC], sc[VEC], w2[VEC];
        const float m2 = nm2, rs2 = nrs2;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            rs[i] = 0.f;
#pragma unroll
            for (int e = 0; e < VEC; ++e) oh[i][e] = g[i][e] = d[i][e] = y[i][e] = r[i][e] = 0.f;
            if (!on[i]) continue;
            rs[i] = nrs[i];
            ro[i].widen(p.obf, oh[i]);
            if (p.gate) rg[i].widen(p.iobf, g[i]);
            if (p.dr) rd[i].widen(p.rbf, d[i]);
            if (p.dh) ry[i].widen(p.iobf, y[i]);
            if (p.dh && p.res) rr[i].widen(p.rbf, r[i]);
#pragma unroll
            for (int e = 0; e < VEC; ++e) oh[i][e] = (oh[i][e] - nm[i]) * rs[i];
        }
        if (AHEAD && row + step < p.rows) fetch(row + step);
        if (p.dh) {
            float s1 = 0.f, s2 = 0.f;
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!on[i]) continue;
                lds_w<VEC>(s_mem, p.C, 0, c[i], w1);
                lds_w<VEC>(s_mem, p.C, 1, c[i], b1);
                lds_w<VEC>(s_mem, p.C, 2, c[i], sc);
                lds_w<VEC>(s_mem, p.C, 3, c[i], w2);
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    float u = fmaf(oh[i][e], w1[e], b1[e]);
                    if (p.gate) u *= act_of(p.act, g[i][e]);
                    const float rh = (fmaf(sc[e], u, r[i][e]) - m2) * rs2;
                    acc[3][i][e] = fmaf(y[i][e], rh, acc[3][i][e]);
                    acc[4][i][e] += y[i][e];
                    y[i][e] *= w2[e];
                    s1 += y[i][e];
                    s2 = fmaf(y[i][e], rh, s2);
                    r[i][e] = rh;
                }
            }
            s1 = p.norm2 == RN_LAYER ? team(s1) * inv2 : 0.f;
            s2 = team(s2) * inv2;
#pragma unroll
            for (int i = 0; i < NV; ++i)
#pragma unroll
                for (int e = 0; e < VEC; ++e) d[i][e] = fmaf(rs2, y[i][e] - s1 - r[i][e] * s2, d[i][e]);
        }
        float t1[NV], t2[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            t1[i] = t2[i] = 0.f;
            if (!on[i]) continue;
            if (p.dres) store<VEC>(p.dres, at + c[i], p.rbf, d[i]);
            lds_w<VEC>(s_mem, p.C, 0, c[i], w1);
            lds_w<VEC>(s_mem, p.C, 1, c[i], b1);
            lds_w<VEC>(s_mem, p.C, 2, c[i], sc);
#pragma unroll
            for (int e = 0; e < VEC; ++e) {
                const float u = fmaf(oh[i][e], w1[e], b1[e]), ds = d[i][e] * sc[e];
                float du = ds, s = u;
                if (p.gate) {
                    const float a = act_of(p.act, g[i][e]);
                    du *= a;
                    s *= a;
                    g[i][e] = ds * u * slope_of(p.act, g[i][e]);
                }
                acc[2][i][e] = fmaf(d[i][e], s, acc[2][i][e]);
                acc[0][i][e] = fmaf(du, oh[i][e], acc[0][i][e]);
                acc[1][i][e] += du;
                d[i][e] = du * w1[e];
                t1[i] += d[i][e];
                t2[i] = fmaf(d[i][e], oh[i][e], t2[i]);
            }
            if (p.gate) store<VEC>(p.dgate, at + c[i], p.iobf, g[i]);
        }
        if (!p.do_) continue;
        if (p.norm == RN_LAYER) part_sums<L, NV>(t1, p.lanes, team);
        part_sums<L, NV>(t2, p.lanes, team);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!on[i]) continue;
            const float u1 = p.norm == RN_LAYER ? t1[i] * inv1 : 0.f, u2 = t2[i] * inv1;
#pragma unroll
            for (int e = 0; e < VEC; ++e) d[i][e] = rs[i] * (d[i][e] - u1 - oh[i][e] * u2);
            store<VEC>(p.do_, at + c[i], p.obf, d[i]);
        }
    }
    if (!p.part) return;
    constexpr int TEAMS = threads<L>() / L;
    const int mine = threadIdx.x / L;
#pragma unroll
    for (int k = 0; k < 5; ++k) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (on[i])
#pragma unroll
                for (int e = 0; e < VEC; ++e) s_mem[mine * p.C + c[i] + e] = acc[k][i][e];
        __syncthreads();
        for (int q = threadIdx.x; q < p.C; q += threads<L>()) {
            float s = 0.f;
            for (int j = 0; j < TEAMS; ++j) s += s_mem[j * p.C + q];
            p.part[((int64_t)blockIdx.x * 5 + k) * p.C + q] = s;
        }
    }
}

// Lanes per team and vectors per lane for C channels: a 16-byte vector per lane and as many lanes as that
// takes (4096 channels by 256 lanes of two vectors instead: forward of 4 rows 5.1 us against 4.0, of 16384 229
// against 157, gradient 397 against 216; 1024 channels by a wave: 41 against 31, 102 against 68).  C that is no
// multiple of 8 goes by single values.
struct Plan {
    int vec, L, NV;
};
Plan plan_of(int C) {
    if (C % 8 == 0) {
        const int u = C / 8;
        if (u <= 16) return {8, 16, 1};
        if (u <= 32) return {8, 32, 1};
        if (u <= 64) return {8, 64, 1};
        if (u <= 128) return {8, 128, 1};
        if (u <= 256) return {8, 256, 1};
        if (u <= 512) return {8, 512, 1};
        return {8, 1024, 1};
    }
    if (C <= 256) return {1, 64, 4};
    if (C <= 1024) return {1, 64, 16};
    if (C <= 4096) return {1, 256, 16};
    return {1, 512, 16};
}
int team_threads(int L) { return L >= 128 ? L : 256; }

// Workgroups of the backward, each of which leaves one row of sums: as many as are resident at once (two waves per
// SIMD, of 1024 threads four), two rows to a team at least.
int parts_of(int64_t rows, int C) {
    const Plan pl = plan_of(C);
    const int64_t per = 2 * (team_threads(pl.L) / pl.L), n = (rows + per - 1) / per;
    const int most = pl.L >= 512 ? 256 : 131072 / team_threads(pl.L);   // of 256 CUs
    return (int)(n < most ? n : most);
}

template <int VEC, int L, int NV>
hipError_t run(const Args& a, bool bwd, hipStream_t s) {
    constexpr int nt = threads<L>(), teams = nt / L;
    int64_t grid;
    if (bwd) {
        grid = parts_of(a.rows, a.C);
    } else {
        int n_cu = 0;
        const hipError_t e = wkv7::device_cus(&n_cu);
        if (e != hipSuccess) return e;
        const int64_t most = (int64_t)n_cu * 8, need = (a.rows + teams - 1) / teams;
        grid = need < most ? need : most;
    }
    if (bwd) {
        const int rows_of = teams > 4 ? teams : 4;             // the weights' four rows, or the teams' sums
        static wkv7::PerDeviceOnce once;
        if (4 * VEC * L * NV * 4 > 65536 - 1024) {             // beyond what a launch may have unasked
            const hipError_t e = wkv7::set_smem_once(once, bwd_kernel<VEC, L, NV>, 4 * VEC * L * NV * 4);
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL((bwd_kernel<VEC, L, NV>), dim3((uint32_t)grid), dim3(nt), rows_of * a.C * 4, s, a, grid * teams);
    } else {
        hipLaunchKernelGGL((fwd_kernel<VEC, L, NV>), dim3((uint32_t)grid), dim3(nt), 0, s, a, grid * teams);
    }
    return hipGetLastError();
}

hipError_t launch(const Args& a, bool bwd, hipStream_t s) {
    const Plan pl = plan_of(a.C);
    if (pl.vec == 8) {
        switch (pl.L * pl.NV) {
            case 16: return run<8, 16, 1>(a, bwd, s);
            case 32: return run<8, 32, 1>(a, bwd, s);
            case 64: return run<8, 64, 1>(a, bwd, s);
            case 128: return run<8, 128, 1>(a, bwd, s);
            case 256: return run<8, 256, 1>(a, bwd, s);
            case 512: return run<8, 512, 1>(a, bwd, s);
            default: return run<8, 1024, 1>(a, bwd, s);
        }
    }
    if (pl.L == 64) return pl.NV == 4 ? run<1, 64, 4>(a, bwd, s) : run<1, 64, 16>(a, bwd, s);
    return pl.L == 256 ? run<1, 256, 16>(a, bwd, s) : run<1, 512, 16>(a, bwd, s);
}

bool is_dtype(int d) { return d == WKV7_F32 || d == WKV7_BF16; }
int64_t esz(int d) { return d == WKV7_BF16 ? 2 : 4; }

wkv7_status check_shape(int64_t rows, int C, int groups) {
    if (rows < 1 || C < 1 || C > 8192 || groups < 1 || C % groups || rows > (int64_t(1) << 40) / C) return WKV7_ERR_SHAPE;
    const int D = C / groups;
    if (groups > 1 && D != 64 && D != 128 && D != 256 && D != 512) return WKV7_ERR_SHAPE;
    return WKV7_OK;
}
wkv7_status check_kinds(int norm, int norm2, int act, int od, int iod, int rd, int wd) {
    if (!is_dtype(od) || !is_dtype(iod) || !is_dtype(rd) || !is_dtype(wd)) return WKV7_ERR_DTYPE;
    if ((od != iod && od != WKV7_F32) || (rd != iod && rd != WKV7_F32)) return WKV7_ERR_DTYPE;
    if (norm != RN_LAYER && norm != RN_RMS) return WKV7_ERR_ARG;
    if (norm2 != RN_NONE && norm2 != RN_LAYER && norm2 != RN_RMS) return WKV7_ERR_ARG;
    return act == RN_ONE || act == RN_SILU || act == RN_SIGMOID ? WKV7_OK : WKV7_ERR_ARG;
}

}  // namespace
}  // namespace resnorm

extern "C" {

wkv7_status rn_fwd(int64_t rows, int C, int groups, rn_norm norm, rn_norm norm2, rn_act act, wkv7_dtype o_dtype,
                   wkv7_dtype io_dtype, wkv7_dtype r_dtype, wkv7_dtype w_dtype, float eps, float eps2, const void* o,
                   const void* gate, int64_t gate_ld, const void* res, const void* weight, const void* bias,
                   const void* scale, const void* weight2, const void* bias2, void* r, void* h, float* stats,
                   void* stream) {
    using namespace resnorm;
    wkv7_status s = check_kinds(norm, norm2, act, o_dtype, io_dtype, r_dtype, w_dtype);
    if (s == WKV7_OK) s = check_shape(rows, C, groups);
    if (s != WKV7_OK) return s;
    if (!res && r_dtype != io_dtype) return WKV7_ERR_DTYPE;
    if ((gate != nullptr) != (act != RN_ONE) || (h != nullptr) != (norm2 != RN_NONE)) return WKV7_ERR_ARG;
    if (gate && (gate_ld < C || gate_ld > (int64_t(1) << 40) / rows)) return WKV7_ERR_SHAPE;
    const bool vec = C % 8 == 0;
    if (vec && gate && gate_ld % 8) return WKV7_ERR_ALIGN;
    const int64_t n = rows * C, ob = esz(o_dtype), ib = esz(io_dtype), rb = esz(r_dtype), wb = esz(w_dtype);
    const int oa = vec ? 16 : (int)ob, ia = vec ? 16 : (int)ib, ra = vec ? 16 : (int)rb, wa = vec ? 16 : (int)wb;
    const abi::Buf bufs[] = {{o, n * ob, true, false, oa}, {gate, ((rows - 1) * gate_ld + C) * ib, false, false, ia},
                             {res, n * rb, false, false, ra}, {weight, C * wb, false, false, wa},
                             {bias, C * wb, false, false, wa}, {scale, C * wb, false, false, wa},
                             {weight2, C * wb, false, false, wa}, {bias2, C * wb, false, false, wa},
                             {r, n * rb, true, true, ra}, {h, n * ib, false, true, ia},
                             {stats, rows * (2LL * groups + 2) * 4, false, true, 4}};
    s = abi::check(bufs);
    if (s != WKV7_OK) return s;
    Args a = {};
    a.o = o; a.gate = gate; a.res = res; a.weight = weight; a.bias = bias; a.scale = scale; a.weight2 = weight2;
    a.bias2 = bias2; a.r = r; a.h = h; a.stats = stats; a.rows = rows; a.gate_ld = gate_ld; a.eps = eps; a.eps2 = eps2;
    a.C = C; a.G = groups; a.lanes = groups > 1 ? C / groups / 8 : 0; a.norm = norm; a.norm2 = norm2; a.act = act;
    a.obf = o_dtype == WKV7_BF16; a.iobf = io_dtype == WKV7_BF16; a.rbf = r_dtype == WKV7_BF16;
    a.wbf = w_dtype == WKV7_BF16;
    return launch(a, false, static_cast<hipStream_t>(stream)) == hipSuccess ? WKV7_OK : WKV7_ERR_HIP;
}

size_t rn_bwd_workspace_bytes(int64_t rows, int C, int groups) {
    if (resnorm::check_shape(rows, C, groups) != WKV7_OK) return 0;
    return (size_t)resnorm::parts_of(rows, C) * C * 5 * 4;
}

wkv7_status rn_bwd(int64_t rows, int C, int groups, rn_norm norm, rn_norm norm2, rn_act act, wkv7_dtype o_dtype,
                   wkv7_dtype io_dtype, wkv7_dtype r_dtype, wkv7_dtype w_dtype, const void* dr, const void* dh,
                   const void* o, const void* gate, int64_t gate_ld, const void* res, const float* stats,
                   const void* weight, const void* bias, const void* scale, const void* weight2, void* do_, void* dgate,
                   void* dres, float* dw, void* workspace, size_t workspace_bytes, void* stream) {
    using namespace resnorm;
    wkv7_status s = check_kinds(norm, norm2, act, o_dtype, io_dtype, r_dtype, w_dtype);
    if (s == WKV7_OK) s = check_shape(rows, C, groups);
    if (s != WKV7_OK) return s;
    if (!res && r_dtype != io_dtype) return WKV7_ERR_DTYPE;
    if ((gate != nullptr) != (act != RN_ONE) || (gate != nullptr) != (dgate != nullptr)) return WKV7_ERR_ARG;
    if ((!dr && !dh) || (dh && norm2 == RN_NONE) || (dres && !res)) return WKV7_ERR_ARG;
    if (gate && (gate_ld < C || gate_ld > (int64_t(1) << 40) / rows)) return WKV7_ERR_SHAPE;
    const bool vec = C % 8 == 0;
    if (vec && gate && gate_ld % 8) return WKV7_ERR_ALIGN;
    const int64_t n = rows * C, ob = esz(o_dtype), ib = esz(io_dtype), rb = esz(r_dtype), wb = esz(w_dtype);
    const int oa = vec ? 16 : (int)ob, ia = vec ? 16 : (int)ib, ra = vec ? 16 : (int)rb, wa = vec ? 16 : (int)wb;
    const int64_t need = dw ? (int64_t)rn_bwd_workspace_bytes(rows, C, groups) : 0;
    const abi::Buf bufs[] = {{dr, n * rb, false, false, ra}, {dh, n * ib, false, false, ia}, {o, n * ob, true, false, oa},
                             {gate, ((rows - 1) * gate_ld + C) * ib, false, false, ia}, {res, n * rb, false, false, ra},
                             {stats, rows * (2LL * groups + 2) * 4, true, false, 4}, {weight, C * wb, false, false, wa},
                             {bias, C * wb, false, false, wa}, {scale, C * wb, false, false, wa},
                             {weight2, C * wb, false, false, wa}, {do_, n * ob, false, true, oa},
                             {dgate, n * ib, false, true, ia}, {dres, n * rb, false, true, ra},
                             {dw, 5LL * C * 4, false, true, 4}, {workspace, need, false, true, 16}};
    s = abi::check(bufs);
    if (s != WKV7_OK) return s;
    if (need && (!workspace || workspace_bytes < (size_t)need)) return WKV7_ERR_WORKSPACE;
    Args a = {};
    a.dr = dr; a.dh = dh; a.o = o; a.gate = gate; a.res = res; a.stats = const_cast<float*>(stats); a.weight = weight;
    a.bias = bias; a.scale = scale; a.weight2 = weight2; a.do_ = do_; a.dgate = dgate; a.dres = dres;
    a.part = dw ? static_cast<float*>(workspace) : nullptr; a.rows = rows; a.gate_ld = gate_ld;
    a.C = C; a.G = groups; a.lanes = groups > 1 ? C / groups / 8 : 0; a.norm = norm; a.norm2 = norm2; a.act = act;
    a.obf = o_dtype == WKV7_BF16; a.iobf = io_dtype == WKV7_BF16; a.rbf = r_dtype == WKV7_BF16;
    a.wbf = w_dtype == WKV7_BF16;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    hipError_t e = launch(a, true, hs);
    if (e == hipSuccess && dw)
        e = sums::launch_column_sums(a.part, parts_of(rows, C), 5LL * C, dw, 5LL * C, nullptr, 0, nullptr, hs);
    return e == hipSuccess ? WKV7_OK : WKV7_ERR_HIP;
}

}  // extern "C"
