// ssm_step.hip -- the selective scan token by token (gfx950): one or a few new tokens per
// sequence, states in a pool.
//
// A lane holds four states of a channel (16 bytes), the S / 4 lanes of a channel are
// neighbours, so the state goes in and out in whole lines, once, and y is a sum within a row
// of 16 lanes.  Bound by HBM.
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
__device__ __forceinline__ f32x4 load4(const float* p) { return f32x4{p[0], p[1], p[2], p[3]}; }
__device__ __forceinline__ f32x4 load4(const uint16_t* p) { return f32x4{ld(p), ld(p + 1), ld(p + 2), ld(p + 3)}; }

// Batch row r works on state slots[r] (state r without slots); a slot outside 0 .. P - 1 has
// no state: y is 0 and nothing is read.  Rows of the same slot are consecutive tokens of one
// sequence, in batch order: the first of them does the work of all, so no two workgroups
// share a state.
template <typename InT, int S>
__global__ __launch_bounds__(NT) void step_kernel(StepArgs p, int nsub) {
    constexpr int LPC = S / 4;                             // lanes per channel
    const int tid = threadIdx.x, sub = blockIdx.x % nsub, r = blockIdx.x / nsub;
    const int ch = sub * (NT / LPC) + tid / LPC, n0 = 4 * (tid % LPC);
    const bool on = ch < p.C, first = on && tid % LPC == 0;
    InT* y = static_cast<InT*>(p.y) + ch;
    int slot = r, end = r + 1;                             // rows r .. end - 1 are looked through
    if (p.slots) {
        slot = p.slots[r];
        if (slot < 0 || slot >= p.P) {
            for (int t = 0; t < p.T && first; ++t) st(y + ((int64_t)r * p.T + t) * p.C, 0.f);
            return;
        }
    }
    const int64_t at = ((int64_t)slot * p.C + ch) * S + n0;
    f32x4 h = {0.f, 0.f, 0.f, 0.f}, A2 = h;
    if (on) h = __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(p.state + at));
    if (p.slots) {                                         // while the state is on its way; every wave for itself
        bool before = false, after = false;                // whether other rows have this slot
#pragma unroll 4
        for (int e = tid & 63; e < p.B; e += 64) {
            const bool same = p.slots[e] == slot;
            before |= same && e < r;
            after |= same && e > r;
        }
        if (__ballot(before)) return;
        if (__ballot(after)) end = p.B;
    }
    if (on) A2 = kLog2e * *reinterpret_cast<const f32x4*>(p.A + (int64_t)ch * S + n0);
    const float bias = on && p.dt_bias ? p.dt_bias[ch] : 0.f, Dv = on && p.D ? p.D[ch] : 0.f;
    const int64_t go = (int64_t)(on ? ch / (p.C / p.G) : 0) * S + n0;
    for (int row = r; row < end; ++row) {
        if (row != r && p.slots[row] != slot) continue;
        for (int t = 0; t < p.T; ++t) {
            const int64_t tok = (int64_t)row * p.T + t;
            float x = 0.f, v = 0.f, z = 0.f;
            if (on) {
                x = ld(static_cast<const InT*>(p.x) + tok * p.x_ld + ch);
                v = ld(static_cast<const InT*>(p.dt) + tok * p.dt_ld + ch) + bias;
                if (p.z) z = ld(static_cast<const InT*>(p.z) + tok * p.z_ld + ch);
            }
            const f32x4 b = load4(static_cast<const InT*>(p.b) + tok * p.b_ld + go);
            const f32x4 c = load4(static_cast<const InT*>(p.c) + tok * p.c_ld + go);
            const float d = p.softplus ? softplus(v) : v, u = d * x;
            float s = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                h[i] = fmaf(exp2_f(d * A2[i]), h[i], u * b[i]);
                s = fmaf(c[i], h[i], s);
            }
            s = fmaf(Dv, x, lanes_sum<LPC>(s));
            if (first) st(y + tok * p.C, p.z ? s * z * sigmoid(z) : s);
        }
    }
    if (on) __builtin_nontemporal_store(h, reinterpret_cast<f32x4*>(p.state_out + at));
}

template <typename InT, int S>
hipError_t run(const StepArgs& a, hipStream_t s) {
    constexpr int CH = NT / (S / 4);
    const int nsub = (a.C + CH - 1) / CH;
    hipLaunchKernelGGL((step_kernel<InT, S>), dim3((uint32_t)a.B * nsub), dim3(NT), 0, s, a, nsub);
    return hipGetLastError();
}
template <typename InT>
hipError_t pick(const StepArgs& a, hipStream_t s) {
    switch (a.S) {
        case 16: return run<InT, 16>(a, s);
        case 32: return run<InT, 32>(a, s);
        default: return run<InT, 64>(a, s);
    }
}

}  // namespace

hipError_t launch_step(const StepArgs& a, bool bf16, hipStream_t s) {
    return bf16 ? pick<uint16_t>(a, s) : pick<float>(a, s);
}

}  // namespace ssm
