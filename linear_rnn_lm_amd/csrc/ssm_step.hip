// ssm_step.hip -- the selective scan token by token (gfx950): one or a few new tokens per
// sequence, states in a pool.
//
// A lane holds four states of a channel (16 bytes), the S / 4 lanes of a channel are
// neighbours, so the state goes in and out in whole lines, once, and y is a sum within a row
// of 16 lanes.  Bound by HBM with many rows (256 rows of 4096 channels, 16 states, all of them
// new to the caches: 32 us, 4.4 TB/s), by the launch and two round trips with few (3 us).
#include "rows_device.h"
#include "ssm_internal.h"

namespace ssm {
namespace {

using namespace rows;
constexpr int NT = 256;

template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
    x += dpp<0xB1>(x);                         // quad 1,0,3,2
    x += dpp<0x4E>(x);                         // quad 2,3,0,1
    if (LANES >= 8) x += dpp<0x141>(x);        // half row mirror
    if (LANES >= 16) x += dpp<0x140>(x);       // row mirror
    return x;
}
// Four neighbouring values; `four`: at a multiple of four.
__device__ __forceinline__ f32x4 load4(const float* p, bool four) {
    return four ? *reinterpret_cast<const f32x4*>(p) : f32x4{p[0], p[1], p[2], p[3]};
}
__device__ __forceinline__ f32x4 load4(const uint16_t* p, bool four) {
    if (!four) return f32x4{ld(p), ld(p + 1), ld(p + 2), ld(p + 3)};
    const uint2 u = *reinterpret_cast<const uint2*>(p);
    return f32x4{__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u), __uint_as_float(u.y << 16),
                 __uint_as_float(u.y & 0xffff0000u)};
}

// Batch row r works on state slots[r] (state r without slots); a slot outside 0 .. P - 1 has
// no state: y is 0 and nothing is read.  Rows of the same slot are consecutive tokens of one
// sequence, in batch order: the first of them does the work of all, so no two workgroups
// share a state.  A wave has K times the channels that its lanes hold at once.
template <typename InT, int S, int K>
__global__ __launch_bounds__(NT) void step_kernel(StepArgs p, int nsub) {
    constexpr int LPC = S / 4, CW = 64 / LPC;              // lanes per channel, channels that a wave's lanes hold at once
    const int tid = threadIdx.x, lane = tid & 63, sub = blockIdx.x % nsub, r = blockIdx.x / nsub;
    const int ch0 = (sub * (NT / 64) + (tid >> 6)) * CW * K, n0 = 4 * (lane % LPC);    // of one group: CW K divides 64
    int ch[K];
    bool on[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        ch[k] = ch0 + k * CW + lane / LPC;
        on[k] = ch[k] < p.C;
    }
    const bool first = lane % LPC == 0;
    InT* y = static_cast<InT*>(p.y);
    int slot = r, end = r + 1;                             // rows r .. end - 1 are looked through
    if (p.slots) {
        slot = p.slots[r];
        if (slot < 0 || slot >= p.P) {
            for (int t = 0; t < p.T; ++t)
#pragma unroll
                for (int k = 0; k < K; ++k)
                    if (on[k] && first) st(y + ((int64_t)r * p.T + t) * p.C + ch[k], 0.f);
            return;
        }
    }
    const int64_t at = (int64_t)slot * p.C * S + n0;
    f32x4 h[K], A2[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        h[k] = A2[k] = f32x4{0.f, 0.f, 0.f, 0.f};
        if (on[k]) h[k] = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p.state + at + (int64_t)ch[k] * S));
    }
    if (p.slots) {                                         // while the state is on its way; every wave for itself
        bool before = false, after = false;                // whether other rows have this slot
#pragma unroll 4
        for (int e = lane; e < p.B; e += 64) {
            const bool same = p.slots[e] == slot;
            before |= same && e < r;
            after |= same && e > r;
        }
        if (__ballot(before)) return;
        if (__ballot(after)) end = p.B;
    }
    float bias[K], Dv[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        if (on[k]) A2[k] = *reinterpret_cast<const f32x4*>(p.A + (int64_t)ch[k] * S + n0);
#pragma unroll
        for (int i = 0; i < 4; ++i) A2[k][i] = rate_of(A2[k][i]);
        bias[k] = on[k] && p.dt_bias ? p.dt_bias[ch[k]] : 0.f;
        Dv[k] = on[k] && p.D ? p.D[ch[k]] : 0.f;
    }
    const int64_t go = (int64_t)(ch0 < p.C ? ch0 / (p.C / p.G) : 0) * S + n0;
    for (int row = r; row < end; ++row) {
        if (row != r && p.slots[row] != slot) continue;
        for (int t = 0; t < p.T; ++t) {
            const int64_t tok = (int64_t)row * p.T + t;
            float x[K], v[K], z[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                x[k] = v[k] = z[k] = 0.f;
                if (!on[k]) continue;
                x[k] = ld(static_cast<const InT*>(p.x) + tok * p.x_ld + ch[k]);
                v[k] = ld(static_cast<const InT*>(p.dt) + tok * p.dt_ld + ch[k]) + bias[k];
                if (p.z) z[k] = ld(static_cast<const InT*>(p.z) + tok * p.z_ld + ch[k]);
            }
            const f32x4 b = load4(static_cast<const InT*>(p.b) + tok * p.b_ld + go, p.bc_four);
            const f32x4 c = load4(static_cast<const InT*>(p.c) + tok * p.c_ld + go, p.bc_four);
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const float d = p.softplus ? softplus(v[k]) : v[k], u = d * x[k];
                float s = 0.f;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    h[k][i] = fmaf(exp2_f(d * A2[k][i]), h[k][i], u * b[i]);
                    s = fmaf(c[i], h[k][i], s);
                }
                s = fmaf(Dv[k], x[k], lanes_sum<LPC>(s));
                if (on[k] && first) st(y + tok * p.C + ch[k], p.z ? s * z[k] * sigmoid_for<InT>(z[k]) : s);
            }
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
        if (on[k]) __builtin_nontemporal_store(h[k], reinterpret_cast<f32x4*>(p.state_out + at + (int64_t)ch[k] * S));
}

template <typename InT, int S, int K>
hipError_t run(const StepArgs& a, hipStream_t s) {
    constexpr int CH = NT / (S / 4) * K;
    const int nsub = (a.C + CH - 1) / CH;
    hipLaunchKernelGGL((step_kernel<InT, S, K>), dim3((uint32_t)a.B * nsub), dim3(NT), 0, s, a, nsub);
    return hipGetLastError();
}
// Four times the channels per wave, so four loads of states at once, where that still leaves two workgroups
// per CU (4096 channels of 16 states: 64 rows 11.4 -> 8.9 us, 256 39 -> 32, but 16 rows 4.6 -> 5.6).
template <typename InT, int S>
hipError_t pick_k(const StepArgs& a, hipStream_t s) {
    constexpr int CH = NT / (S / 4);
    return (int64_t)a.B * ((a.C + CH - 1) / CH) >= 2048 ? run<InT, S, 4>(a, s) : run<InT, S, 1>(a, s);
}
template <typename InT>
hipError_t pick(const StepArgs& a, hipStream_t s) {
    switch (a.S) {
        case 16: return pick_k<InT, 16>(a, s);
        case 32: return pick_k<InT, 32>(a, s);
        default: return pick_k<InT, 64>(a, s);
    }
}

}  // namespace

hipError_t launch_step(const StepArgs& a, bool bf16, hipStream_t s) {
    return bf16 ? pick<uint16_t>(a, s) : pick<float>(a, s);
}

}  // namespace ssm
