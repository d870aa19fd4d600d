// gdr_prepare.hip -- per-chunk operands of the gated delta rule (gfx950): what the
// chain of states needs of a chunk of 64 tokens of one head apart from the state.
//
//     T = (I + A)^-1,  A = strict_lower(b_t Lam K K^T)
//
// with the chunk's gates (see gdr_device.h).  All chunks of all heads run at
// once, one workgroup of four waves each.  The data moved would take 83 us at B8
// T4096 H32 K64 (16384 chunks of heads; 420 MB by the counters, g and beta once per XCD), the
// kernel takes 122 to 129: each workgroup is a row
// of dependent steps (loads, products, substitution, two levels of block products), so
// what counts is how many of them a unit holds.  Seven fit 18 KB of LDS and 72 registers
// each; four, with A and T apart and five columns of A ahead, took 171 us, and eight, which
// have to spill, 144 where seven took 129.  At K = 128 (B1 T32768 H32, 355 MB) 147 us.
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

// T = (I + A)^-1 for the strictly lower 64 x 64 matrix A.  Diagonal 16 x 16 blocks by
// forward substitution (one column per lane), then [[X, 0], [Z, Y]]^-1 =
// [[X', 0], [-Y' Z X', Y']] for blocks of 16 and of 32 with fp32 MFMA products: stable
// for any A, unlike a series in powers of A.  One LDS matrix holds both: A transposed in
// its upper half, T in its lower (a diagonal block of T replaces A's once that is used
// up).  18 KB to a workgroup instead of 35 lets more of them overlap their waits.
// A 16 x 16 tile of X Y over kn; XT: X is given transposed.
template <bool XT>
__device__ __forceinline__ f32x4 block_product(const float* X, const float* Y, int kn, int lane) {
    const int r = lane & 15, g = lane >> 4;
    f32x4 acc = zero4();
    for (int k0 = 0; k0 < kn; k0 += 4)
        acc = wkv7::mfma_f32(XT ? X[(k0 + g) * LDA + r] : X[r * LDA + k0 + g], Y[(k0 + g) * LDA + r], acc);
    return acc;
}
__device__ __forceinline__ void put_tile(float* Z, f32x4 x, int lane) {
#pragma unroll
    for (int q = 0; q < 4; ++q) Z[(4 * (lane >> 4) + q) * LDA + (lane & 15)] = x[q];
}

template <int NX, int K>
__global__ __launch_bounds__(256, NX == 1 ? 7 : 4) void prepare_kernel(Args p) {
    __shared__ __attribute__((aligned(16))) float X[C * LDA];   // X[s][t] = A[t][s] for s < t; X[t][s] = T[t][s]
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
    // 64 columns of the rows at a time (32 of three planes): all of them at once, one wait for memory
    constexpr int KB = NX == 1 ? 2 : 1;
    // tile i here is tile w ^ i of the matrix: the first is this wave's own rows as well
    PF<NX> kb[4][KB];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int ks = 0; ks < KB; ++ks) {
#pragma unroll
            for (int nt = 0; nt < 4; ++nt)
                if (nt < 2 || w >= 2) kb[nt][ks] = frag_mem<NX>(kp, row(idx(w ^ nt, r16)), stride, k0 + ks, lane);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    fetch(0);

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
    }
    f32x4 kk[4] = {zero4(), zero4(), zero4(), zero4()};
#pragma unroll
    for (int k0 = 0; k0 < KS; k0 += KB) {
        if (k0 > 0) fetch(k0);
#pragma unroll
        for (int nt = 0; nt < 4; ++nt)
            if (nt < 2 || w >= 2) {
#pragma unroll
                for (int ks = 0; ks < KB; ++ks) kk[nt] = pmma<NX>(kk[nt], kb[0][ks], kb[nt][ks]);
            }
    }
    __syncthreads();
    const int t0 = idx(w, 4 * g4);
    const f32x4 nt4 = *reinterpret_cast<const f32x4*>(&nf[0][t0]), ft4 = *reinterpret_cast<const f32x4*>(&nf[1][t0]);
    const f32x4 b4 = *reinterpret_cast<const f32x4*>(&bs[t0]);
#pragma unroll
    for (int nt = 0; nt < 4; ++nt) {
        if (nt >= 2 && w < 2) continue;
        const int s = idx(w ^ nt, r16);
        f32x4 a;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            a[q] = s < t0 + q && t0 + q < len ? b4[q] * decay(nt4[q], ft4[q], nf[0][s], nf[1][s]) * kk[nt][q] : 0.f;
        *reinterpret_cast<f32x4*>(X + s * LDA + t0) = a;
    }
    __syncthreads();

    // all four diagonal blocks on one wave, 16 lanes each; which one varies, so that each SIMD gets its share
    if (w == (int)(blockIdx.x * 0x9E3779B1u >> 30)) {
        const int o = 16 * g4;
        float x[16];
#pragma unroll
        for (int t = 0; t < 16; ++t) x[t] = t == r16 ? 1.f : 0.f;
        // once x[s] is final every later row takes A[t][s] x[s]; the columns of A are read three
        // at a time, in 16-byte pieces, and then used (more of them ahead cost a workgroup per unit)
#pragma unroll
        for (int s0 = 0; s0 < 15; s0 += 3) {
            f32x4 col[3][4];
#pragma unroll
            for (int s = s0; s < s0 + 3; ++s)
#pragma unroll
                for (int c = (s + 1) / 4; c < 4; ++c)
                    col[s - s0][c] = *reinterpret_cast<const f32x4*>(X + (o + s) * LDA + o + 4 * c);
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int s = s0; s < s0 + 3; ++s)
#pragma unroll
                for (int t = s + 1; t < 16; ++t) x[t] = fmaf(-col[s - s0][t / 4][t % 4], x[s], x[t]);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int t = 0; t < 16; ++t) X[(o + t) * LDA + o + r16] = x[t];
    }
    __syncthreads();
    // blocks of 16, Z X' in its result's place; A's block then becomes T's zero block
    if (w < 2) {
        float* d = X + 32 * w * (LDA + 1);
        put_tile(d + 16 * LDA, block_product<true>(d + 16, d, 16, lane), lane);
        wkv7::wave_lds_sync();
        const f32x4 z = block_product<false>(d + 16 * LDA + 16, d + 16 * LDA, 16, lane);
        wkv7::wave_lds_sync();
        put_tile(d + 16 * LDA, -z, lane);
        put_tile(d + 16, zero4(), lane);
    }
    __syncthreads();
    // blocks of 32: wave (mr, mc) forms one 16 x 16 tile of each product
    const int mr = 16 * (w >> 1), mc = 16 * (w & 1);
    float* d = X + (32 + mr) * LDA + mc;
    put_tile(d, block_product<true>(X + 32 + mr, X + mc, 32, lane), lane);
    __syncthreads();
    const f32x4 z = block_product<false>(X + (32 + mr) * LDA + 32, X + 32 * LDA + mc, 32, lane);
    __syncthreads();
    put_tile(d, -z, lane);
    __syncthreads();

    // the three lower 32 x 32 blocks, in pieces of eight values: block, row, eight columns
    float* out = p.tri + block * p.tri_stride;
    for (int e = tid; e < 768; e += 256) {
        const int blk = e >> 8, row = (e >> 3) & 31, u = e & 7;
        *reinterpret_cast<f32x4*>(out + 4 * e) =
            *reinterpret_cast<const f32x4*>(X + ((blk ? 32 : 0) + row) * LDA + (blk == 2 ? 32 : 0) + 4 * u);
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
