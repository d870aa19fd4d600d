// gdr_prepare.hip -- per-chunk operands of the gated delta rule (gfx950): what the
// chain of states needs of a chunk of 64 tokens of one head apart from the state.
//
//     T = (I + A)^-1,  A = strict_lower(b_t Lam K K^T)
//
// with the chunk's gates (see gdr_device.h).  All chunks of all heads run at
// once, one workgroup of four waves each.
#include "gdr_device.h"
#include "gdr_internal.h"
#include "wkv7_internal.h"

namespace gdr {
namespace {

constexpr int LDA = 68;  // row stride (floats) of the fp32 64 x 64 matrices

// fp32 q (y = 0) and k (y = 1) to three bf16 planes (24 bits).
__global__ __launch_bounds__(256) void split_kernel(const float* q, const float* k, uint16_t* qp, uint16_t* kp, int64_t n) {
    const float* x = blockIdx.y ? k : q;
    uint16_t* o = blockIdx.y ? kp : qp;
    const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;   // n is a multiple of 64
    if (i >= n) return;
    const f32x4 v = *reinterpret_cast<const f32x4*>(x + i);
    bf16x2 a[3], b[3];
    planes2<3>(wkv7::f32x2{v[0], v[1]}, a);
    planes2<3>(wkv7::f32x2{v[2], v[3]}, b);
#pragma unroll
    for (int p = 0; p < 3; ++p)
        *reinterpret_cast<bf16x4*>(o + p * n + i) = bf16x4{a[p][0], a[p][1], b[p][0], b[p][1]};
}

// Rows outside every sequence; one workgroup in x per share of them, y = tensor.
__global__ __launch_bounds__(256) void zero_outside_kernel(ZeroArgs p) {
    const int64_t a = min(max(p.cu[0], 0), p.T), b = min(max(p.cu[p.N], (int)a), p.T), w = p.words[blockIdx.y];
    const int64_t n = (a + (p.T - b)) * w, head = a * w, skip = (b - a) * w;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256)
        p.p[blockIdx.y][i < head ? i : i + skip] = 0u;
}

// Operand rows straight from memory: lane (g, r) gets X[row][32 ks + 8g .. + 7].
template <int NX>
__device__ __forceinline__ PF<NX> frag_mem(const Planes& x, int64_t row, int stride, int ks, int lane) {
    PF<NX> f;
#pragma unroll
    for (int i = 0; i < NX; ++i)
        f.p[i] = *reinterpret_cast<const bf16x8*>(x.p + i * x.plane + row * stride + 32 * ks + 8 * (lane >> 4));
    return f;
}

// T = (I + A)^-1 for the strictly lower 64 x 64 matrix A, held transposed (At[s][t] =
// A[t][s]).  Diagonal 16 x 16 blocks by forward substitution (one wave each, one
// column per lane), then [[X, 0], [Z, Y]]^-1 = [[X', 0], [-Y' Z X', Y']] for blocks of
// 16 and of 32 with fp32 MFMA products: stable for any A, unlike a series in
// powers of A.  Z (16 x 16) = sign X Y over kn; XT: X is given transposed.
template <bool XT>
__device__ __forceinline__ void block_product(const float* X, const float* Y, float* Z, int kn, float sign, int lane) {
    const int r = lane & 15, g = lane >> 4;
    f32x4 acc = zero4();
    for (int k0 = 0; k0 < kn; k0 += 4)
        acc = wkv7::mfma_f32(XT ? X[(k0 + g) * LDA + r] : X[r * LDA + k0 + g], Y[(k0 + g) * LDA + r], acc);
#pragma unroll
    for (int q = 0; q < 4; ++q) Z[(4 * g + q) * LDA + r] = sign * acc[q];
}

template <int NX, int K>
__global__ __launch_bounds__(256, 4) void prepare_kernel(Args p) {
    __shared__ __attribute__((aligned(16))) float At[C * LDA];
    __shared__ __attribute__((aligned(16))) float Ts[C * LDA];
    __shared__ float nf[2][C], bs[C];
    const int tid = threadIdx.x, lane = tid & 63, w = tid >> 6;
    const int g4 = lane >> 4, r16 = lane & 15;
    const int slot = blockIdx.x / p.H, h = blockIdx.x % p.H;
    const Seqs seqs{p.cu, p.N, p.T, p.NC};
    int n, len;
    int64_t tok;
    if (!slot_chunk(seqs, slot, n, tok, len)) return;
    const int hk = h / (p.H / p.Hk);
    const int64_t block = (int64_t)slot * p.H + h;

    // row tile w of K K^T (lower 32 x 32 blocks), rows straight from memory
    constexpr int KS = K / 32;
    const int stride = p.Hk * K;
    Planes kp = p.kp;
    kp.p += tok * stride + hk * K;
    auto row = [&](int t) { return min(t, len - 1); };   // tokens past the end: masked below
    PF<NX> ka[KS], kb[4][KS];
    const int ra = row(idx(w, r16));
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) ka[ks] = frag_mem<NX>(kp, ra, stride, ks, lane);
    if constexpr (NX == 1) {                             // all rows at once: one wait for memory
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
            if (nt < 2 || w >= 2) {
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) kb[nt][ks] = frag_mem<NX>(kp, row(idx(nt, r16)), stride, ks, lane);
            }
        __builtin_amdgcn_sched_barrier(0);
    }

    if (w == 3) {
        float g = 0.f, b = 0.f;
        if (lane < len) {
            g = p.g[(tok + lane) * p.H + h];
            b = p.beta[(tok + lane) * p.H + h];
            g = g < kMinLogDecay ? kMinLogDecay : g;
            b = fabsf(b) < kBetaMin ? kBetaMin : b;
        }
        double G = g;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const double o = __shfl_up(G, d);
            if (lane >= d) G += o;
        }
        const double Gc = __shfl(G, 63);
        const double y = G * 1.4426950408889634074, n2 = __builtin_rint(y);
        nf[0][lane] = (float)n2;
        nf[1][lane] = (float)(y - n2);
        bs[lane] = b;
        float* gt = p.tri + block * p.tri_stride + kTriFloats;
        gt[kGateEG + lane] = exp_d(G);
        gt[kGateToEnd + lane] = lane < len ? exp_d(Gc - G) : 0.f;
        gt[kGateBeta + lane] = b;
        gt[kGateN + lane] = (float)n2;
        gt[kGateF + lane] = (float)(y - n2);
    } else if (w < 2) {
        // the zero 16 x 16 blocks of T's diagonal 32 x 32 blocks
        *reinterpret_cast<f32x4*>(Ts + (32 * w + (lane >> 2)) * LDA + 32 * w + 16 + 4 * (lane & 3)) = zero4();
    }
    f32x4 kk[4];
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        kk[nt] = zero4();
        if (nt >= 2 && w < 2) continue;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            if constexpr (NX > 1) kb[nt][ks] = frag_mem<NX>(kp, row(idx(nt, r16)), stride, ks, lane);
            kk[nt] = pmma<NX>(kk[nt], ka[ks], kb[nt][ks]);
        }
    }
    __syncthreads();
    const int t0 = idx(w, 4 * g4);
    const f32x4 nt4 = *reinterpret_cast<const f32x4*>(&nf[0][t0]), ft4 = *reinterpret_cast<const f32x4*>(&nf[1][t0]);
    const f32x4 b4 = *reinterpret_cast<const f32x4*>(&bs[t0]);
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        if (nt >= 2 && w < 2) continue;
        const int s = idx(nt, r16);
        f32x4 a;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            a[q] = s < t0 + q && t0 + q < len ? b4[q] * decay(nt4[q], ft4[q], nf[0][s], nf[1][s]) * kk[nt][q] : 0.f;
        *reinterpret_cast<f32x4*>(At + s * LDA + t0) = a;
    }
    __syncthreads();

    if (lane < 16) {
        const int o = 16 * w;
        float x[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) x[t] = t == lane ? 1.f : 0.f;
        // once x[s] is final every later row takes A[t][s] x[s]; column s of A is read in
        // 16-byte pieces, five columns ahead of their use
#pragma unroll
        for (int s0 = 0; s0 < 15; s0 += 5) {
            f32x4 col[5][4];
#pragma unroll
            for (int s = s0; s < s0 + 5; ++s)
#pragma unroll
                for (int c = (s + 1) / 4; c < 4; ++c)
                    col[s - s0][c] = *reinterpret_cast<const f32x4*>(At + (o + s) * LDA + o + 4 * c);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = s0; s < s0 + 5; ++s)
#pragma unroll
                for (int t = s + 1; t < 16; ++t) x[t] = fmaf(-col[s - s0][t / 4][t % 4], x[s], x[t]);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int t = 0; t < 16; ++t) Ts[(o + t) * LDA + o + lane] = x[t];
    }
    __syncthreads();
    // blocks of 16: the scratch products lie in At's part for t < s, which is unused
    if (w < 2) {
        const int o = 32 * w;
        float* scr = At + (o + 16) * LDA + o;
        block_product<true>(At + o * LDA + o + 16, Ts + o * LDA + o, scr, 16, 1.f, lane);
        wkv7::wave_lds_sync();
        block_product<false>(Ts + (o + 16) * LDA + o + 16, scr, Ts + (o + 16) * LDA + o, 16, -1.f, lane);
    }
    __syncthreads();
    // blocks of 32: wave (mr, mc) forms one 16 x 16 tile of each product
    const int mr = 16 * (w >> 1), mc = 16 * (w & 1);
    block_product<true>(At + 32 + mr, Ts + mc, At + (32 + mr) * LDA + mc, 32, 1.f, lane);
    __syncthreads();
    block_product<false>(Ts + (32 + mr) * LDA + 32, At + 32 * LDA + mc, Ts + (32 + mr) * LDA + mc, 32, -1.f, lane);
    __syncthreads();

    // the three lower 32 x 32 blocks, in pieces of eight values: block, row, eight columns
    float* out = p.tri + block * p.tri_stride;
    for (int e = tid; e < 768; e += 256) {
        const int blk = e >> 8, row = (e >> 3) & 31, u = e & 7;
        *reinterpret_cast<f32x4*>(out + 4 * e) =
            *reinterpret_cast<const f32x4*>(Ts + ((blk ? 32 : 0) + row) * LDA + (blk == 2 ? 32 : 0) + 4 * u);
    }
}

template <int NX>
hipError_t launch_k(const Args& a, hipStream_t s) {
    const dim3 grid((uint32_t)a.slots * a.H);
    if (a.K == 64) hipLaunchKernelGGL((prepare_kernel<NX, 64>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((prepare_kernel<NX, 128>), grid, dim3(256), 0, s, a);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_zero_outside(const ZeroArgs& a, hipStream_t s) {
    hipLaunchKernelGGL(zero_outside_kernel, dim3(64, (uint32_t)a.n), dim3(256), 0, s, a);
    return hipGetLastError();
}

hipError_t launch_split(const float* q, const float* k, uint16_t* qp, uint16_t* kp, int64_t n, hipStream_t s) {
    hipLaunchKernelGGL(split_kernel, dim3((uint32_t)((n / 4 + 255) / 256), 2), dim3(256), 0, s, q, k, qp, kp, n);
    return hipGetLastError();
}

hipError_t launch_prepare(const Args& a, bool bf16, hipStream_t s) {
    return bf16 ? launch_k<1>(a, s) : launch_k<3>(a, s);
}

}  // namespace gdr
