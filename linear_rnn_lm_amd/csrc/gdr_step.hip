// gdr_step.hip -- the gated delta rule token by token (gfx950): one or a few new
// tokens per sequence, states in a pool.
//
// A thread holds RT consecutive rows of four columns of the state; the K / 4
// threads of a row share a half wave or a DPP row, so the row sums S k and S q
// need no LDS.  The state is read once and written once: bound by HBM (256 rows of
// 64 heads of 64 x 64: 537 MB in 84 us, 6.4 TB/s; 100 us where slots say which state is
// whose, since those loads wait for the slot).
#include "gdr_device.h"
#include "gdr_internal.h"
#include "wkv7_internal.h"

namespace gdr {
namespace {

constexpr int NT = 256;

__device__ __forceinline__ float row_allsum16(float x) {
    x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0xB1, 0xf, 0xf, false));   // quad_perm 1,0,3,2
    x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x4E, 0xf, 0xf, false));   // quad_perm 2,3,0,1
    x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x141, 0xf, 0xf, false));  // row_half_mirror
    x += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), 0x140, 0xf, 0xf, false));  // row_mirror
    return x;
}
template <int K>
__device__ __forceinline__ float rowsum(float x) {
    return K == 64 ? row_allsum16(x) : wkv7::half_sum32(x);
}

__device__ __forceinline__ f32x4 load4(const float* p) { return *reinterpret_cast<const f32x4*>(p); }
__device__ __forceinline__ f32x4 load4(const uint16_t* p) {
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                 __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u)};
}

// Slots.  Batch row b works on state slots[b] (b itself without slots); a
// slot outside 0 .. P - 1 has no state: o is 0 and nothing is written.  Rows of
// the same slot are consecutive tokens of one sequence, in batch order:
// the first of them does the work of all, so no two workgroups share a state.
template <typename InT, int K, int RT>
__global__ __launch_bounds__(NT) void step_kernel(StepArgs p, int nsub) {
    constexpr int LPR = K / 4;                       // lanes per row
    const int tid = threadIdx.x;
    const int sub = blockIdx.x % nsub, bh = blockIdx.x / nsub, h = bh % p.H, b = bh / p.H;
    const int hk = h / (p.H / p.Hk);
    const int c0 = 4 * (tid % LPR), r0 = sub * (NT / LPR * RT) + RT * (tid / LPR);
    const InT* q = static_cast<const InT*>(p.q);
    const InT* k = static_cast<const InT*>(p.k);
    const InT* v = static_cast<const InT*>(p.v);
    InT* o = static_cast<InT*>(p.o);

    int slot = b, end = b + 1;                             // rows b .. end - 1 are looked through
    if (p.slots) {
        slot = p.slots[b];
        if (slot < 0 || slot >= p.P) {
            for (int t = 0; t < p.T; ++t)
                if (tid % LPR == 0)
                    for (int i = 0; i < RT; ++i) st(o + (((int64_t)b * p.T + t) * p.H + h) * p.V + r0 + i, 0.f);
            return;
        }
    }
    const int64_t soff = (((int64_t)slot * p.H + h) * p.V + r0) * K + c0;
    f32x4 s[RT];
#pragma unroll
    for (int i = 0; i < RT; ++i)
        s[i] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p.state + soff + i * K));
    if (p.slots) {                                         // while the state is on its way; every wave for itself
        bool before = false, after = false;                // whether other rows have this slot
#pragma unroll 4
        for (int e = tid & 63; e < p.B; e += 64) {
            const bool same = p.slots[e] == slot;
            before |= same && e < b;
            after |= same && e > b;
        }
        if (__ballot(before)) return;
        if (__ballot(after)) end = p.B;
    }
    for (int row = b; row < end; ++row) {
        if (row != b && p.slots[row] != slot) continue;
        for (int t = 0; t < p.T; ++t) {
            const int64_t tok = (int64_t)row * p.T + t;
            const f32x4 q4 = load4(q + (tok * p.Hk + hk) * K + c0), k4 = load4(k + (tok * p.Hk + hk) * K + c0);
            const float g = p.g[tok * p.H + h], beta = p.beta[tok * p.H + h];
            const float a = exp_d(g < kMinLogDecay ? kMinLogDecay : g);
            float vr[RT], or_[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) vr[i] = ld(v + (tok * p.H + h) * p.V + r0 + i);
#pragma unroll
            for (int i = 0; i < RT; ++i) {
                f32x4 x = a * s[i];
                const float kv = rowsum<K>(fmaf(x[0], k4[0], fmaf(x[1], k4[1], fmaf(x[2], k4[2], x[3] * k4[3]))));
                const float u = beta * (vr[i] - kv);
#pragma unroll
                for (int c = 0; c < 4; ++c) x[c] = fmaf(u, k4[c], x[c]);
                s[i] = x;
                or_[i] = p.scale *
                         rowsum<K>(fmaf(x[0], q4[0], fmaf(x[1], q4[1], fmaf(x[2], q4[2], x[3] * q4[3]))));
            }
            if (tid % LPR == 0) {
#pragma unroll
                for (int i = 0; i < RT; ++i) st(o + (tok * p.H + h) * p.V + r0 + i, or_[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
        __builtin_nontemporal_store(s[i], reinterpret_cast<f32x4*>(p.state_out + soff + i * K));
}

template <typename InT, int K>
hipError_t launch_typed(const StepArgs& a, hipStream_t s) {
    constexpr int RT = 4, rows = NT / (K / 4) * RT;
    const int nsub = a.V / rows;
    hipLaunchKernelGGL((step_kernel<InT, K, RT>), dim3((uint32_t)a.B * a.H * nsub), dim3(NT), 0, s, a, nsub);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_step(const StepArgs& a, bool bf16, hipStream_t s) {
    if (bf16) return a.K == 64 ? launch_typed<uint16_t, 64>(a, s) : launch_typed<uint16_t, 128>(a, s);
    return a.K == 64 ? launch_typed<float, 64>(a, s) : launch_typed<float, 128>(a, s);
}

}  // namespace gdr
