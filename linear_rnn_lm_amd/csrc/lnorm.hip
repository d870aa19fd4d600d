// lnorm.hip -- layer norm over the parts of a row, forward and backward (gfx950).
//
// Bound by HBM: x is read once and kept in registers for the mean, the centred
// variance and the output (32768 x 2048 in 32 parts, bf16: 48 us, 5.6 TB/s); the backward
// reads x and dy once (the same: 84 us, 4.8 TB/s).  Small calls are bound by the launch
// (256 x 4096: 4.6 us on the GPU, 11 us a call).  A part of D
// channels belongs to a team of L lanes (part of a wave, a wave, or a
// workgroup), NV vectors of VEC values per lane.  A team keeps one group index and walks
// rows, so its weight and bias stay in registers, and in the backward so
// do its sums for dweight and dbias.  Neighbouring teams hold neighbouring
// groups of the same row, so a workgroup's accesses stay contiguous.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "abi_checks.h"
#include "lnorm.h"
#include "wkv7_device.h"
#include "wkv7_internal.h"

namespace lnorm {
namespace {

using wkv7::bf16x8;
using wkv7::f32x4;
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));

struct Args {
    const void *x, *dy, *weight, *bias;
    void *y, *dx;
    float *mean, *rstd;
    float* part;         // backward: (2, parts, C) sums over rows, or NULL
    float eps;
    int64_t rows;
    int C, G, D, teams;  // teams: a multiple of G
    int parts;           // row count of `part`
    bool combine;        // backward: a workgroup adds up its teams of one group
    bool wbf16;
};

// VEC values as stored, widened only at their use, so that the next row's loads
// do not wait where they are issued.
template <typename T, int VEC>
struct Raw {
    typename std::conditional<VEC == 8, typename std::conditional<sizeof(T) == 2, u32x4, f32x4>::type, T>::type v[VEC == 8 ? sizeof(T) / 2 : 1];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (size_t i = 0; i < sizeof(v) / sizeof(v[0]); ++i) v[i] = reinterpret_cast<const std::remove_reference_t<decltype(v[0])>*>(p)[i];
    }
    __device__ __forceinline__ void widen(float (&o)[VEC]) const {
        if constexpr (VEC == 8 && sizeof(T) == 2) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                o[2 * e] = __uint_as_float(v[0][e] << 16);
                o[2 * e + 1] = __uint_as_float(v[0][e] & 0xffff0000u);
            }
        } else if constexpr (VEC == 8) {
#pragma unroll
            for (int e = 0; e < 8; ++e) o[e] = v[e / 4][e % 4];
        } else if constexpr (sizeof(T) == 2) {
            o[0] = __uint_as_float((uint32_t)v[0] << 16);
        } else {
            o[0] = v[0];
        }
    }
};
template <int VEC, typename T>
__device__ __forceinline__ void loadv(const T* p, float (&v)[VEC]) {
    Raw<T, VEC> r;
    r.load(p);
    r.widen(v);
}
template <int VEC>
__device__ __forceinline__ void storev(float* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        *reinterpret_cast<f32x4*>(p) = f32x4{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4*>(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
    } else {
        *p = v[0];
    }
}
template <int VEC>
__device__ __forceinline__ void storev(uint16_t* p, const float (&v)[VEC]) {
    if constexpr (VEC == 8) {
        bf16x8 o;
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = (__bf16)v[e];
        *reinterpret_cast<bf16x8*>(p) = o;
    } else {
        *p = __builtin_bit_cast(uint16_t, (__bf16)v[0]);
    }
}

// Sum over teams of L <= 64 neighbouring lanes, in every lane: quad permutes,
// mirrors within a DPP row, then row and half swaps.  Each step adds the same
// two numbers in both lanes of a pair, so all lanes of a team agree.
template <int L>
__device__ __forceinline__ float wave_sum(float x) {
    x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0xB1, 0xf, 0xf, false));
    x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x4E, 0xf, 0xf, false));
    x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x141, 0xf, 0xf, false));
    if constexpr (L >= 16) x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x140, 0xf, 0xf, false));
    if constexpr (L >= 32) {
        const auto h = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(h[0]) + __uint_as_float(h[1]);
    }
    if constexpr (L >= 64) {
        const auto h = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
        x = __uint_as_float(h[0]) + __uint_as_float(h[1]);
    }
    return x;
}

// Sum over a team.  Workgroup-wide teams go through LDS; `red` has one float per
// wave and is alternated by the caller, so one barrier per sum is enough.
template <int L>
__device__ __forceinline__ float team_sum(float x, float* red) {
    x = wave_sum<(L < 64 ? L : 64)>(x);
    if constexpr (L > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = x;
        wkv7::lds_barrier();
        x = 0.f;
#pragma unroll
        for (int i = 0; i < L / 64; ++i) x += red[i];
    }
    return x;
}

template <int L>
constexpr int threads() { return L > 256 ? L : 256; }

template <int VEC, int L, int NV>
struct Team {
    int64_t row, step;
    int g, lane;
    bool on;
    __device__ __forceinline__ Team(const Args& p) {
        const int64_t id = ((int64_t)blockIdx.x * threads<L>() + threadIdx.x) / L;
        on = id < p.teams;
        g = (int)(id % p.G);
        row = id / p.G;
        step = p.teams / p.G;
        lane = threadIdx.x % L;
    }
    __device__ __forceinline__ int d(int i) const { return (i * L + lane) * VEC; }
};

template <int VEC>
__device__ __forceinline__ void load_w(const Args& p, const void* w, int c, float dflt, float (&v)[VEC]) {
    if (!w) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) v[e] = dflt;
    } else if (p.wbf16) {
        loadv<VEC>(static_cast<const uint16_t*>(w) + c, v);
    } else {
        loadv<VEC>(static_cast<const float*>(w) + c, v);
    }
}

template <typename InT, typename OutT, int VEC, int L, int NV>
__global__ __launch_bounds__(threads<L>()) void fwd_kernel(Args p) {
    __shared__ float red[2][16];
    const Team<VEC, L, NV> t(p);
    if (!t.on) return;                        // whole workgroups only where L > 64
    const InT* x = static_cast<const InT*>(p.x) + (int64_t)t.g * p.D;
    OutT* y = static_cast<OutT*>(p.y) + (int64_t)t.g * p.D;
    const float inv = 1.f / (float)p.D;
    float w[NV][VEC], b[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (t.d(i) < p.D) {
            load_w<VEC>(p, p.weight, t.g * p.D + t.d(i), 1.f, w[i]);
            load_w<VEC>(p, p.bias, t.g * p.D + t.d(i), 0.f, b[i]);
        }
    Raw<InT, VEC> next[NV];
    auto fetch = [&](int64_t row) {
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t.d(i) < p.D) next[i].load(x + row * p.C + t.d(i));
    };
    if (t.row < p.rows) fetch(t.row);
    for (int64_t row = t.row; row < p.rows; row += t.step) {
        float v[NV][VEC], s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) next[i].widen(v[i]);
        if (row + t.step < p.rows) fetch(row + t.step);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t.d(i) < p.D) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) s += v[i][e];
            }
        const float mean = team_sum<L>(s, red[0]) * inv;
        s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t.d(i) < p.D) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) {
                    v[i][e] -= mean;
                    s = fmaf(v[i][e], v[i][e], s);
                }
            }
        const float rstd = 1.f / sqrtf(team_sum<L>(s, red[1]) * inv + p.eps);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t.d(i) < p.D) {
#pragma unroll
                for (int e = 0; e < VEC; ++e) v[i][e] = fmaf(v[i][e] * rstd, w[i][e], b[i][e]);
                storev<VEC>(y + row * p.C + t.d(i), v[i]);
            }
        if (p.mean && t.lane == 0) {
            p.mean[row * p.G + t.g] = mean;
            p.rstd[row * p.G + t.g] = rstd;
        }
    }
}

// With xh = (x - mean) rstd and e = dy weight:
//     dx = rstd (e - mean(e) - xh mean(e xh)),  dweight = sum dy xh,  dbias = sum dy
template <typename InT, typename OutT, int VEC, int L, int NV>
__global__ __launch_bounds__(threads<L>()) void bwd_kernel(Args p) {
    __shared__ float red[4][16];
    const Team<VEC, L, NV> t(p);
    const int64_t c0 = (int64_t)t.g * p.D;
    const InT* x = static_cast<const InT*>(p.x) + c0;
    const OutT* dy = static_cast<const OutT*>(p.dy) + c0;
    InT* dx = static_cast<InT*>(p.dx) + c0;
    const float inv = 1.f / (float)p.D;
    float w[NV][VEC], dw[NV][VEC], db[NV][VEC];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int e = 0; e < VEC; ++e) w[i][e] = dw[i][e] = db[i][e] = 0.f;
        if (t.on && t.d(i) < p.D) load_w<VEC>(p, p.weight, t.g * p.D + t.d(i), 1.f, w[i]);
    }
    Raw<InT, VEC> nx[NV];
    Raw<OutT, VEC> ny[NV];
    float nmean = 0.f, nrstd = 0.f;
    auto fetch = [&](int64_t row) {
        nmean = p.mean[row * p.G + t.g];
        nrstd = p.rstd[row * p.G + t.g];
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t.d(i) < p.D) {
                nx[i].load(x + row * p.C + t.d(i));
                ny[i].load(dy + row * p.C + t.d(i));
            }
    };
    if (t.on && t.row < p.rows) fetch(t.row);
    int flip = 0;
    for (int64_t row = t.on ? t.row : p.rows; row < p.rows; row += t.step, flip ^= 2) {
        const float mean = nmean, rstd = nrstd;
        float xh[NV][VEC], e[NV][VEC], s1 = 0.f, s2 = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            nx[i].widen(xh[i]);
            ny[i].widen(e[i]);
        }
        if (row + t.step < p.rows) fetch(row + t.step);
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t.d(i) < p.D) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) {
                    xh[i][k] = (xh[i][k] - mean) * rstd;
                    dw[i][k] = fmaf(e[i][k], xh[i][k], dw[i][k]);
                    db[i][k] += e[i][k];
                    e[i][k] *= w[i][k];
                    s1 += e[i][k];
                    s2 = fmaf(e[i][k], xh[i][k], s2);
                }
            }
        if (!p.dx) continue;
        s1 = team_sum<L>(s1, red[flip]) * inv;
        s2 = team_sum<L>(s2, red[flip + 1]) * inv;
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t.d(i) < p.D) {
#pragma unroll
                for (int k = 0; k < VEC; ++k) e[i][k] = rstd * (e[i][k] - s1 - xh[i][k] * s2);
                storev<VEC>(dx + row * p.C + t.d(i), e[i]);
            }
    }
    if (!p.part) return;
    if constexpr (L <= 64) {
        if (p.combine) {          // the workgroup holds whole rows of teams: one row of sums
            constexpr int S = threads<L>() / L;
            __shared__ float sum[threads<L>() * NV * VEC];
            const int team = threadIdx.x / L, W = p.G * p.D;
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                __syncthreads();
#pragma unroll
                for (int i = 0; i < NV; ++i)
                    if (t.d(i) < p.D)
#pragma unroll
                        for (int k = 0; k < VEC; ++k) sum[team * p.D + t.d(i) + k] = m ? db[i][k] : dw[i][k];
                __syncthreads();
                for (int c = threadIdx.x; c < W; c += threads<L>()) {
                    float s = 0.f;
                    for (int j = 0; j < S / p.G; ++j) s += sum[j * W + c];
                    p.part[((int64_t)m * p.parts + blockIdx.x) * p.C + c] = s;
                }
            }
            return;
        }
    }
    if (!t.on) return;
    float* pw = p.part + t.row * p.C + c0;
    float* pb = pw + (int64_t)p.parts * p.C;
#pragma unroll
    for (int i = 0; i < NV; ++i)
        if (t.d(i) < p.D) {
            storev<VEC>(pw + t.d(i), dw[i]);
            storev<VEC>(pb + t.d(i), db[i]);
        }
}

// Column sums of the (parts, C) sums, 3 to 5 us (a launch and one round trip): 32 columns by 32 rows of threads, four rows each in flight.
__global__ __launch_bounds__(1024) void reduce_kernel(const float* part, int parts, int C, float* dweight, float* dbias) {
    __shared__ float red[32][33];
    const int cl = threadIdx.x & 31, c = blockIdx.x * 32 + cl, r0 = threadIdx.x >> 5;
    const float* src = part + (blockIdx.y ? (int64_t)parts * C : 0) + min(c, C - 1);
    float s[4] = {0.f, 0.f, 0.f, 0.f};
    for (int r = r0; r < parts; r += 128) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const float x = src[(int64_t)min(r + 32 * u, parts - 1) * C];
            s[u] += r + 32 * u < parts ? x : 0.f;
        }
    }
    red[r0][cl] = (s[0] + s[1]) + (s[2] + s[3]);
    __syncthreads();
    // the wave of rows 2c, 2c + 1 adds up columns 2c, 2c + 1
    float x = wave_sum<32>(red[threadIdx.x & 31][r0]);
    if ((threadIdx.x & 31) == 0 && blockIdx.x * 32 + r0 < C) (blockIdx.y ? dbias : dweight)[blockIdx.x * 32 + r0] = x;
}

// Lanes per team and vectors per lane for D channels: the fewest lanes that hold a part in
// four 16-byte vectors each, so that a workgroup keeps many rows in flight and a sum takes
// few exchanges; D that is no multiple of 8 goes by single values.
struct Plan {
    int vec, L, NV;
};
Plan plan_of(int D) {
    if (D % 8 == 0) {
        const int u = D / 8;
        for (int L : {8, 16, 32, 64, 256})
            for (int nv : {1, 2, 3, 4})
                if (L * nv >= u) return {8, L, nv};
        return {8, 1024, 2};
    }
    if (D <= 256) return {1, 64, 4};
    if (D <= 1024) return {1, 256, 4};
    if (D <= 4096) return {1, 256, 16};
    return {1, 1024, 16};
}

// Teams of a launch: a multiple of G, at most what the chip holds at once (32 waves per
// unit; 16 or 64 changed nothing from 12288 x 384 to 65536 x 768).
int teams_of(int64_t rows, int G, int L, int n_cu, int waves_per_cu) {
    const int64_t most = (int64_t)n_cu * waves_per_cu * 64 / L;
    int64_t r = most / G;
    if (r < 1) r = 1;
    if (r > rows) r = rows;
    return (int)(r * G);
}

// How the backward's rows are shared out.  Where a workgroup of 256 holds the teams of one or
// more whole rows (combine), each workgroup leaves one row of sums; otherwise each team
// leaves its own.  At least two (eight) rows to a team, so that the sums stay small beside
// x, dy and dx; from 256 workgroups on at least eight, and at most 512 of them: the sums
// are written and read again, and more rows in flight no longer help (gradients of 65536
// x 768: 53 us, with 1024 of them 60, with 256 53; 32768 x 2048 in 32 parts: 84, 86, 119;
// 4096 x 2048: 22 with 256, 24 with 512).  Without combining: 65536 x 768 92 us,
// 12288 x 384 20 instead of 14; part counts that do not divide 256 / L go that way (forward and
// gradients of 32768 x 768 in 12 parts 54 us, in 8 parts 47; 12288 x 384 in 6 parts 30, in one 29).
// 256 units of 16 waves bound the teams then: the chip's own, since the workspace is asked
// for without a device.
struct Share {
    bool combine;
    int parts;
};
Share bwd_share(int64_t rows, int D, int G) {
    const Plan pl = plan_of(D);
    const int S = 256 / pl.L;
    if (pl.L <= 64 && S % G == 0) {
        const int64_t per = S / G, few = (rows + 2 * per - 1) / (2 * per), good = rows / (8 * per);
        const int64_t most = good < 256 ? 256 : good < 512 ? good : 512;
        return {true, (int)(few < most ? few : most)};
    }
    const int64_t most = (int64_t)256 * 16 * 64 / pl.L / G + 1, few = (rows + 7) / 8;
    return {false, (int)(few < most ? few : most)};
}

template <typename InT, typename OutT, int VEC, int L, int NV>
hipError_t run(Args a, bool bwd, hipStream_t s) {
    constexpr int nt = threads<L>();
    int n_cu = 0;
    const hipError_t e = wkv7::device_cus(&n_cu);
    if (e != hipSuccess) return e;
    a.teams = !bwd ? teams_of(a.rows, a.G, L, n_cu, 32) : a.combine ? a.parts * (nt / L) : a.parts * a.G;
    const dim3 grid((uint32_t)(((int64_t)a.teams * L + nt - 1) / nt));
    if (bwd) hipLaunchKernelGGL((bwd_kernel<InT, OutT, VEC, L, NV>), grid, dim3(nt), 0, s, a);
    else hipLaunchKernelGGL((fwd_kernel<InT, OutT, VEC, L, NV>), grid, dim3(nt), 0, s, a);
    return hipGetLastError();
}

template <typename InT, typename OutT, int VEC, int L>
hipError_t pick_nv(const Args& a, int nv, bool bwd, hipStream_t s) {
    switch (nv) {
        case 1: return run<InT, OutT, VEC, L, 1>(a, bwd, s);
        case 2: return run<InT, OutT, VEC, L, 2>(a, bwd, s);
        case 3: return run<InT, OutT, VEC, L, 3>(a, bwd, s);
        default: return run<InT, OutT, VEC, L, 4>(a, bwd, s);
    }
}

template <typename InT, typename OutT>
hipError_t pick(const Args& a, bool bwd, hipStream_t s) {
    const Plan pl = plan_of(a.D);
    if (pl.vec == 8) {
        switch (pl.L) {
            case 8: return pick_nv<InT, OutT, 8, 8>(a, pl.NV, bwd, s);
            case 16: return pick_nv<InT, OutT, 8, 16>(a, pl.NV, bwd, s);
            case 32: return pick_nv<InT, OutT, 8, 32>(a, pl.NV, bwd, s);
            case 64: return pick_nv<InT, OutT, 8, 64>(a, pl.NV, bwd, s);
            case 256: return pick_nv<InT, OutT, 8, 256>(a, pl.NV, bwd, s);
            default: return run<InT, OutT, 8, 1024, 2>(a, bwd, s);
        }
    }
    if (pl.L == 64) return run<InT, OutT, 1, 64, 4>(a, bwd, s);
    if (pl.L == 1024) return run<InT, OutT, 1, 1024, 16>(a, bwd, s);
    return pl.NV == 4 ? run<InT, OutT, 1, 256, 4>(a, bwd, s) : run<InT, OutT, 1, 256, 16>(a, bwd, s);
}

hipError_t launch(const Args& a, wkv7_dtype xd, wkv7_dtype yd, bool bwd, hipStream_t s) {
    if (xd == WKV7_BF16) return pick<uint16_t, uint16_t>(a, bwd, s);
    return yd == WKV7_BF16 ? pick<float, uint16_t>(a, bwd, s) : pick<float, float>(a, bwd, s);
}

bool is_dtype(int d) { return d == WKV7_F32 || d == WKV7_BF16; }

wkv7_status check_shape(int64_t rows, int C, int groups, int xd, int yd, int wd) {
    if (!is_dtype(xd) || !is_dtype(yd) || !is_dtype(wd) || (xd == WKV7_BF16 && yd != WKV7_BF16)) return WKV7_ERR_DTYPE;
    if (rows < 1 || C < 1 || groups < 1 || C % groups || C / groups > 16384) return WKV7_ERR_SHAPE;
    if (C > (1 << 26) || groups > (1 << 20)) return WKV7_ERR_SHAPE;   // a launch takes fewer than 2^32 threads
    if (rows > (int64_t(1) << 40) / C) return WKV7_ERR_SHAPE;
    return WKV7_OK;
}

int64_t esz(wkv7_dtype d) { return d == WKV7_BF16 ? 2 : 4; }
int align_of(int D, wkv7_dtype d) { return D % 8 == 0 ? 16 : (int)esz(d); }   // rows by vectors, or value by value

}  // namespace
}  // namespace lnorm

extern "C" {

wkv7_status ln_fwd(int64_t rows, int C, int groups, wkv7_dtype x_dtype, wkv7_dtype y_dtype, wkv7_dtype w_dtype,
                   const void* x, const void* weight, const void* bias, float eps, void* y, float* mean, float* rstd,
                   void* stream) {
    wkv7_status st = lnorm::check_shape(rows, C, groups, x_dtype, y_dtype, w_dtype);
    if (st != WKV7_OK) return st;
    if ((mean == nullptr) != (rstd == nullptr)) return WKV7_ERR_ARG;
    const int64_t n = rows * C, wb = C * lnorm::esz(w_dtype), sb = rows * groups * 4;
    const int D = C / groups, xa = lnorm::align_of(D, x_dtype), ya = lnorm::align_of(D, y_dtype), wa = lnorm::align_of(D, w_dtype);
    const abi::Buf bufs[] = {{x, n * lnorm::esz(x_dtype), true, false, xa}, {weight, wb, false, false, wa},
                             {bias, wb, false, false, wa}, {y, n * lnorm::esz(y_dtype), true, true, ya},
                             {mean, sb, false, true, 4}, {rstd, sb, false, true, 4}};
    st = abi::check(bufs);
    if (st != WKV7_OK) return st;
    lnorm::Args a = {};
    a.x = x; a.weight = weight; a.bias = bias; a.y = y; a.mean = mean; a.rstd = rstd; a.eps = eps;
    a.rows = rows; a.C = C; a.G = groups; a.D = C / groups; a.wbf16 = w_dtype == WKV7_BF16;
    return lnorm::launch(a, x_dtype, y_dtype, false, static_cast<hipStream_t>(stream)) == hipSuccess ? WKV7_OK
                                                                                                      : WKV7_ERR_HIP;
}

size_t ln_bwd_workspace_bytes(int64_t rows, int C, int groups) {
    if (lnorm::check_shape(rows, C, groups, WKV7_F32, WKV7_F32, WKV7_F32) != WKV7_OK) return 0;
    return (size_t)lnorm::bwd_share(rows, C / groups, groups).parts * C * 2 * 4;
}

wkv7_status ln_bwd(int64_t rows, int C, int groups, wkv7_dtype x_dtype, wkv7_dtype y_dtype, wkv7_dtype w_dtype,
                   const void* dy, const void* x, const void* weight, const float* mean, const float* rstd, void* dx,
                   float* dweight, float* dbias, void* workspace, size_t workspace_bytes, void* stream) {
    wkv7_status st = lnorm::check_shape(rows, C, groups, x_dtype, y_dtype, w_dtype);
    if (st != WKV7_OK) return st;
    if ((dweight == nullptr) != (dbias == nullptr) || (!dx && !dweight)) return WKV7_ERR_ARG;
    const int64_t n = rows * C, sb = rows * groups * 4;
    const int64_t need = dweight ? (int64_t)ln_bwd_workspace_bytes(rows, C, groups) : 0;
    const int D = C / groups, xa = lnorm::align_of(D, x_dtype), ya = lnorm::align_of(D, y_dtype), wa = lnorm::align_of(D, w_dtype);
    const abi::Buf bufs[] = {{dy, n * lnorm::esz(y_dtype), true, false, ya}, {x, n * lnorm::esz(x_dtype), true, false, xa},
                             {weight, C * lnorm::esz(w_dtype), false, false, wa}, {mean, sb, true, false, 4},
                             {rstd, sb, true, false, 4}, {dx, n * lnorm::esz(x_dtype), false, true, xa},
                             {dweight, C * 4LL, false, true, 4}, {dbias, C * 4LL, false, true, 4},
                             {workspace, need, false, true, 16}};
    st = abi::check(bufs);
    if (st != WKV7_OK) return st;
    if (need && (!workspace || workspace_bytes < (size_t)need)) return WKV7_ERR_WORKSPACE;
    lnorm::Args a = {};
    a.x = x; a.dy = dy; a.weight = weight; a.dx = dx; a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd); a.rows = rows; a.C = C; a.G = groups; a.D = C / groups;
    a.wbf16 = w_dtype == WKV7_BF16;
    const lnorm::Share share = lnorm::bwd_share(rows, a.D, groups);
    a.parts = share.parts; a.combine = share.combine;
    a.part = dweight ? static_cast<float*>(workspace) : nullptr;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    hipError_t e = lnorm::launch(a, x_dtype, y_dtype, true, hs);
    if (e == hipSuccess && dweight) {
        hipLaunchKernelGGL(lnorm::reduce_kernel, dim3((uint32_t)((C + 31) / 32), 2), dim3(1024), 0, hs, a.part, a.parts, C,
                           dweight, dbias);
        e = hipGetLastError();
    }
    return e == hipSuccess ? WKV7_OK : WKV7_ERR_HIP;
}

}  // extern "C"
