// rnorm.hip -- the fused end of a block, forward and backward (gfx950):
//     r = res + scale act(gate) (norm1(o) weight + bias),   h = norm2(r) weight2 + bias2
//
// Bound by HBM: a row's o, gate and res are read once and stay in registers for both norms.
// A row belongs to a team of L lanes (part of a wave, a wave or a workgroup), eight neighbouring
// values to a lane; a team walks rows with the sums for the five weights' gradients in
// registers, in the forward with its weights too; the backward has those in LDS, and the next
// row's values on their way while it works on one.  A part of norm1 is 8 to 64
// neighbouring lanes, so its sums are exchanges within a wave.  The backward
// forms r again from what the forward read (res costs what r would), unrounded.
//
// 32768 rows of 2048 channels, 32 parts, fp32 o, the rest bf16: forward 165 us (4.9 TB/s), backward
// 267 us (5.0 TB/s).  Rows of more than 4096 channels are the exception: a lane of 1024 has half the
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

// A lane's eight neighbouring values c .. c + 7 of a row.  Where C is no multiple of 8 (RAGGED) the last
// lane's are the row's last eight: its first `twice` belong to the lane before it too, which counts them in
// sums over the row; everything else both lanes do alike.  Loads and stores need no more alignment than a
// value's own.  Fewer than 8 channels go one by one.
struct Cols {
    int c, twice, n;             // n: values that exist
    bool on;
    __device__ __forceinline__ Cols(int lane, int C) : c(lane * 8), twice(0), n(8), on(lane * 8 < C) {}
};
template <bool RAGGED>
__device__ __forceinline__ Cols cols_of(int lane, int C) {
    Cols k(lane, C);
    if (RAGGED && k.on) {
        k.n = min(8, C);
        k.c = min(k.c, C - k.n);
        k.twice = lane * 8 - k.c;
    }
    return k;
}
// Whether value e counts in sums over the row.
template <bool RAGGED>
__device__ __forceinline__ bool counts(const Cols& k, int e) { return !RAGGED || (e >= k.twice && e < k.n); }

typedef unsigned int u32x4_any __attribute__((ext_vector_type(4), aligned(2)));

// Eight values as stored, of either type (the same for a whole launch), widened at their use, so that loads
// ahead of it do not wait where they are issued.
struct Raw {
    u32x4 v[2];
    template <bool RAGGED>
    __device__ __forceinline__ void load(const void* base, int64_t at, bool bf, const Cols& k) {
        const char* p = static_cast<const char*>(base) + at * (bf ? 2 : 4);
        if (!RAGGED || k.n == 8) {
            v[0] = reinterpret_cast<const u32x4_any*>(p)[0];
            if (!bf) v[1] = reinterpret_cast<const u32x4_any*>(p)[1];
        } else {
            uint32_t x[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
                x[e] = e >= k.n ? 0u : bf ? reinterpret_cast<const uint16_t*>(p)[e] : reinterpret_cast<const uint32_t*>(p)[e];
            v[0] = bf ? u32x4{x[0] | x[1] << 16, x[2] | x[3] << 16, x[4] | x[5] << 16, x[6] | x[7] << 16}
                      : u32x4{x[0], x[1], x[2], x[3]};
            v[1] = u32x4{x[4], x[5], x[6], x[7]};
        }
    }
    __device__ __forceinline__ void widen(bool bf, float (&o)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e)
            o[e] = __uint_as_float(bf ? e % 2 ? v[0][e / 2] & 0xffff0000u : v[0][e / 2] << 16 : v[e / 4][e % 4]);
    }
};
template <bool RAGGED>
__device__ __forceinline__ void load(const void* base, int64_t at, bool bf, const Cols& k, float (&v)[8]) {
    Raw r;
    r.load<RAGGED>(base, at, bf, k);
    r.widen(bf, v);
}
template <bool RAGGED>
__device__ __forceinline__ void store(void* base, int64_t at, bool bf, const Cols& k, const float (&v)[8]) {
    char* p = static_cast<char*>(base) + at * (bf ? 2 : 4);
    if (RAGGED && k.n < 8) {
#pragma unroll
        for (int e = 0; e < 7; ++e) {
            if (e >= k.n) continue;
            if (bf) st(reinterpret_cast<uint16_t*>(p) + e, v[e]);
            else reinterpret_cast<float*>(p)[e] = v[e];
        }
    } else if (bf) {
        bf16x8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (__bf16)v[e];
        *reinterpret_cast<u32x4_any*>(p) = __builtin_bit_cast(u32x4, o);
    } else {
        u32x4 a, b;
#pragma unroll
        for (int e = 0; e < 4; ++e) a[e] = __float_as_uint(v[e]), b[e] = __float_as_uint(v[4 + e]);
        reinterpret_cast<u32x4_any*>(p)[0] = a;
        reinterpret_cast<u32x4_any*>(p)[1] = b;
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

// Sum over a part of norm1, in every lane of it: `lanes` neighbours, or the row.
template <int L>
__device__ __forceinline__ float part_sum(float x, int lanes, TeamSum<L>& team) { return lanes ? lane_sum(x, lanes) : team(x); }

__device__ __forceinline__ float act_of(int act, float g) {
    const float s = sigmoid(g);
    return act == RN_SILU ? g * s : s;
}
__device__ __forceinline__ float slope_of(int act, float g) {
    const float s = sigmoid(g);
    return act == RN_SILU ? s * fmaf(g, 1.f - s, 1.f) : s * (1.f - s);
}

template <bool RAGGED>
__device__ __forceinline__ void load_w(const Args& p, const void* w, const Cols& k, float dflt, float (&v)[8]) {
    if (w) {
        load<RAGGED>(w, k.c, p.wbf, k, v);
    } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = dflt;
    }
}

template <int L, bool RAGGED>
__global__ __launch_bounds__(threads<L>()) void fwd_kernel(Args p, int64_t step) {
    __shared__ float red[4][16];
    const int lane = threadIdx.x % L;
    int64_t row = ((int64_t)blockIdx.x * threads<L>() + threadIdx.x) / L;
    TeamSum<L> team(red);
    const Cols k = cols_of<RAGGED>(lane, p.C);
    const int part = p.lanes ? lane / p.lanes : 0;
    float w1[8], b1[8], sc[8], w2[8], b2[8];
    if (k.on) {
        load_w<RAGGED>(p, p.weight, k, 1.f, w1);
        load_w<RAGGED>(p, p.bias, k, 0.f, b1);
        load_w<RAGGED>(p, p.scale, k, 1.f, sc);
        load_w<RAGGED>(p, p.weight2, k, 1.f, w2);
        load_w<RAGGED>(p, p.bias2, k, 0.f, b2);
    }
    const float inv1 = 1.f / (float)(p.C / p.G), inv2 = 1.f / (float)p.C;
    for (; row < p.rows; row += step) {
        const int64_t at = row * p.C + k.c;
        float v[8], a[8], r[8], m = 0.f, q = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            v[e] = r[e] = 0.f;
            a[e] = 1.f;
        }
        if (k.on) {
            load<RAGGED>(p.o, at, p.obf, k, v);
            if (p.gate) load<RAGGED>(p.gate, row * p.gate_ld + k.c, p.iobf, k, a);
            if (p.res) load<RAGGED>(p.res, at, p.rbf, k, r);
        }
        if (p.norm == RN_LAYER) {
#pragma unroll
            for (int e = 0; e < 8; ++e) m += counts<RAGGED>(k, e) ? v[e] : 0.f;
            m = part_sum<L>(m, p.lanes, team) * inv1;
        }
        if (k.on)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                v[e] -= m;
                const float d = counts<RAGGED>(k, e) ? v[e] : 0.f;
                q = fmaf(d, d, q);
            }
        q = 1.f / sqrtf(fmaf(part_sum<L>(q, p.lanes, team), inv1, p.eps));
        float m2 = 0.f, q2 = 0.f;
        if (k.on) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                float u = fmaf(v[e] * q, w1[e], b1[e]);
                if (p.gate) u *= act_of(p.act, a[e]);
                r[e] = fmaf(sc[e], u, r[e]);
                m2 += counts<RAGGED>(k, e) ? r[e] : 0.f;
            }
            store<RAGGED>(p.r, at, p.rbf, k, r);
            if (p.stats && (p.lanes ? lane % p.lanes : lane) == 0) {    // one lane of each part
                float* s = p.stats + row * (2 * p.G + 2);
                s[part] = m;
                s[p.G + part] = q;
            }
        }
        if (p.norm2 == RN_NONE) continue;
        m2 = p.norm2 == RN_LAYER ? team(m2) * inv2 : 0.f;
        if (k.on)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                r[e] -= m2;
                const float d = counts<RAGGED>(k, e) ? r[e] : 0.f;
                q2 = fmaf(d, d, q2);
            }
        q2 = 1.f / sqrtf(fmaf(team(q2), inv2, p.eps2));
        if (k.on) {
#pragma unroll
            for (int e = 0; e < 8; ++e) r[e] = fmaf(r[e] * q2, w2[e], b2[e]);
            store<RAGGED>(p.h, at, p.iobf, k, r);
        }
        if (p.stats && lane == 0) {
            p.stats[row * (2 * p.G + 2) + 2 * p.G] = m2;
            p.stats[row * (2 * p.G + 2) + 2 * p.G + 1] = q2;
        }
    }
}

// The weights in LDS as fp32 (weight, bias, scale, weight2): a lane's eight in two planes of four, so that
// neighbouring lanes' accesses are neighbours.  In registers they would be 32 of them.
template <int L>
__device__ __forceinline__ float* lds_at(float* s_w, int k, int lane) { return s_w + k * 8 * L + lane * 4; }
template <int L>
__device__ __forceinline__ void lds_w(float* s_w, int k, int lane, float (&v)[8]) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(lds_at<L>(s_w, k, lane));
    const f32x4 b = *reinterpret_cast<const f32x4*>(lds_at<L>(s_w, k, lane) + 4 * L);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = a[e], v[4 + e] = b[e];
}
// Floats of LDS: the weights, or in the end the teams' sums.
template <int L>
constexpr int lds_floats(int C) { return 4 * 8 * L > threads<L>() / L * C ? 4 * 8 * L : threads<L>() / L * C; }

// With oh, rh the normalised o and r, a = act(gate), u = oh weight + bias:
//     dr' = dr + rstd2 (e2 - mean(e2) - rh mean(e2 rh)),  e2 = dh weight2       (= dres)
//     du = dr' scale a,  dgate = dr' scale u act'(gate),  e1 = du weight
//     do = rstd1 (e1 - mean(e1) - oh mean(e1 oh))                              (means over a part)
// and over the rows dweight = sum du oh, dbias = sum du, dscale = sum dr' a u, dweight2 = sum dh
// rh, dbias2 = sum dh; a root-mean-square norm has no mean(e).
template <int L, bool RAGGED>
__global__ __launch_bounds__(threads<L>(), L > 512 ? 4 : 2) void bwd_kernel(Args p, int64_t step) {
    __shared__ float red[4][16];
    extern __shared__ __attribute__((aligned(16))) float s_mem[];
    const int lane = threadIdx.x % L;
    TeamSum<L> team(red);
    const Cols k = cols_of<RAGGED>(lane, p.C);
    const int part = p.lanes ? lane / p.lanes : 0;
    if (threadIdx.x < L && k.on) {
        const void* w[4] = {p.weight, p.bias, p.scale, p.weight2};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float v[8];
            load_w<RAGGED>(p, w[j], k, j == 1 ? 0.f : 1.f, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) lds_at<L>(s_mem, j, lane)[e / 4 * 4 * L + e % 4] = v[e];
        }
    }
    __syncthreads();
    float acc[5][8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
#pragma unroll
        for (int j = 0; j < 5; ++j) acc[j][e] = 0.f;
    const float inv1 = 1.f / (float)(p.C / p.G), inv2 = 1.f / (float)p.C;
    constexpr bool AHEAD = L <= 512;           // the next row on its way while this one is worked on
    Raw ro, rg, rr, rd, ry;
    float nm = 0.f, nrs = 0.f, nm2 = 0.f, nrs2 = 0.f;
    auto fetch = [&](int64_t row) {
        const int64_t at = row * p.C + k.c;
        const float* stat = p.stats + row * (2 * p.G + 2);
        nm2 = stat[2 * p.G], nrs2 = stat[2 * p.G + 1];
        if (!k.on) return;
        nm = stat[part], nrs = stat[p.G + part];
        ro.load<RAGGED>(p.o, at, p.obf, k);
        if (p.gate) rg.load<RAGGED>(p.gate, row * p.gate_ld + k.c, p.iobf, k);
        if (p.dr) rd.load<RAGGED>(p.dr, at, p.rbf, k);
        if (p.dh) ry.load<RAGGED>(p.dh, at, p.iobf, k);
        if (p.dh && p.res) rr.load<RAGGED>(p.res, at, p.rbf, k);
    };
    int64_t row = ((int64_t)blockIdx.x * threads<L>() + threadIdx.x) / L;
    if (AHEAD && row < p.rows) fetch(row);
    for (; row < p.rows; row += step) {
        const int64_t at = row * p.C + k.c;
        if (!AHEAD) fetch(row);
        float oh[8], g[8], d[8], y[8], r[8], rs = 0.f, w1[8], b1[8], sc[8], w2[8];
        const float m2 = nm2, rs2 = nrs2;
#pragma unroll
        for (int e = 0; e < 8; ++e) oh[e] = g[e] = d[e] = y[e] = r[e] = 0.f;
        if (k.on) {
            rs = nrs;
            ro.widen(p.obf, oh);
            if (p.gate) rg.widen(p.iobf, g);
            if (p.dr) rd.widen(p.rbf, d);
            if (p.dh) ry.widen(p.iobf, y);
            if (p.dh && p.res) rr.widen(p.rbf, r);
#pragma unroll
            for (int e = 0; e < 8; ++e) oh[e] = (oh[e] - nm) * rs;
        }
        if (AHEAD && row + step < p.rows) fetch(row + step);
        if (p.dh) {
            float s1 = 0.f, s2 = 0.f;
            if (k.on) {
                lds_w<L>(s_mem, 0, lane, w1);
                lds_w<L>(s_mem, 1, lane, b1);
                lds_w<L>(s_mem, 2, lane, sc);
                lds_w<L>(s_mem, 3, lane, w2);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    float u = fmaf(oh[e], w1[e], b1[e]);
                    if (p.gate) u *= act_of(p.act, g[e]);
                    const float rh = (fmaf(sc[e], u, r[e]) - m2) * rs2;
                    acc[3][e] = fmaf(y[e], rh, acc[3][e]);
                    acc[4][e] += y[e];
                    y[e] *= w2[e];
                    const float yc = counts<RAGGED>(k, e) ? y[e] : 0.f;
                    s1 += yc;
                    s2 = fmaf(yc, rh, s2);
                    r[e] = rh;
                }
            }
            s1 = p.norm2 == RN_LAYER ? team(s1) * inv2 : 0.f;
            s2 = team(s2) * inv2;
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = fmaf(rs2, y[e] - s1 - r[e] * s2, d[e]);
        }
        float t1 = 0.f, t2 = 0.f;
        if (k.on) {
            if (p.dres) store<RAGGED>(p.dres, at, p.rbf, k, d);
            lds_w<L>(s_mem, 0, lane, w1);
            lds_w<L>(s_mem, 1, lane, b1);
            lds_w<L>(s_mem, 2, lane, sc);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float u = fmaf(oh[e], w1[e], b1[e]), ds = d[e] * sc[e];
                float du = ds, s = u;
                if (p.gate) {
                    const float a = act_of(p.act, g[e]);
                    du *= a;
                    s *= a;
                    g[e] = ds * u * slope_of(p.act, g[e]);
                }
                acc[2][e] = fmaf(d[e], s, acc[2][e]);
                acc[0][e] = fmaf(du, oh[e], acc[0][e]);
                acc[1][e] += du;
                d[e] = du * w1[e];
                const float dc = counts<RAGGED>(k, e) ? d[e] : 0.f;
                t1 += dc;
                t2 = fmaf(dc, oh[e], t2);
            }
            if (p.gate) store<RAGGED>(p.dgate, at, p.iobf, k, g);
        }
        if (!p.do_) continue;
        t1 = p.norm == RN_LAYER ? part_sum<L>(t1, p.lanes, team) * inv1 : 0.f;
        t2 = part_sum<L>(t2, p.lanes, team) * inv1;
        if (k.on) {
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e] = rs * (d[e] - t1 - oh[e] * t2);
            store<RAGGED>(p.do_, at, p.obf, k, d);
        }
    }
    if (!p.part) return;
    constexpr int TEAMS = threads<L>() / L;
    const int mine = threadIdx.x / L;
#pragma unroll
    for (int j = 0; j < 5; ++j) {
        __syncthreads();
        if (k.on)
#pragma unroll
            for (int e = 0; e < 8; ++e)
                if (!RAGGED || e < k.n) s_mem[mine * p.C + k.c + e] = acc[j][e];
        __syncthreads();
        for (int q = threadIdx.x; q < p.C; q += threads<L>()) {
            float s = 0.f;
            for (int t = 0; t < TEAMS; ++t) s += s_mem[t * p.C + q];
            p.part[((int64_t)blockIdx.x * 5 + j) * p.C + q] = s;
        }
    }
}

// Lanes of a team for C channels, eight to a lane (4096 channels by 256 lanes of sixteen instead: forward of 4
// rows 5.1 us against 4.0, of 16384 229 against 157, gradient 397 against 216; 1024 channels by a wave: 41
// against 31, 102 against 68).
int lanes_of(int C) {
    int L = 16;
    while (8 * L < C) L *= 2;
    return L;
}
int team_threads(int L) { return L >= 128 ? L : 256; }

// Workgroups of the backward, each of which leaves one row of sums: as many as are resident at once (two waves per
// SIMD, of 1024 threads four), two rows to a team at least.
int parts_of(int64_t rows, int C) {
    const int L = lanes_of(C);
    const int64_t per = 2 * (team_threads(L) / L), n = (rows + per - 1) / per;
    const int most = L >= 512 ? 256 : 131072 / team_threads(L);        // of 256 CUs
    return (int)(n < most ? n : most);
}

template <int L, bool RAGGED>
hipError_t run(const Args& a, bool bwd, hipStream_t s) {
    constexpr int nt = threads<L>(), teams = nt / L, most_lds = lds_floats<L>(8 * L) * 4;
    if (bwd) {
        const int64_t grid = parts_of(a.rows, a.C);
        static wkv7::PerDeviceOnce once;
        if (most_lds > 65536 - 1024) {                         // beyond what a launch may have unasked
            const hipError_t e = wkv7::set_smem_once(once, bwd_kernel<L, RAGGED>, most_lds);
            if (e != hipSuccess) return e;
        }
        hipLaunchKernelGGL((bwd_kernel<L, RAGGED>), dim3((uint32_t)grid), dim3(nt), lds_floats<L>(a.C) * 4, s, a, grid * teams);
    } else {
        int n_cu = 0;
        const hipError_t e = wkv7::device_cus(&n_cu);
        if (e != hipSuccess) return e;
        const int64_t most = (int64_t)n_cu * 8, need = (a.rows + teams - 1) / teams, grid = need < most ? need : most;
        hipLaunchKernelGGL((fwd_kernel<L, RAGGED>), dim3((uint32_t)grid), dim3(nt), 0, s, a, grid * teams);
    }
    return hipGetLastError();
}
template <int L>
hipError_t run(const Args& a, bool bwd, hipStream_t s) { return a.C % 8 ? run<L, true>(a, bwd, s) : run<L, false>(a, bwd, s); }

hipError_t launch(const Args& a, bool bwd, hipStream_t s) {
    switch (lanes_of(a.C)) {
        case 16: return run<16>(a, bwd, s);
        case 32: return run<32>(a, bwd, s);
        case 64: return run<64>(a, bwd, s);
        case 128: return run<128>(a, bwd, s);
        case 256: return run<256>(a, bwd, s);
        case 512: return run<512>(a, bwd, s);
        default: return run<1024>(a, bwd, s);
    }
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
    if (vec && gate && gate_ld * esz(io_dtype) % 16) return WKV7_ERR_ALIGN;
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
    if (vec && gate && gate_ld * esz(io_dtype) % 16) return WKV7_ERR_ALIGN;
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
