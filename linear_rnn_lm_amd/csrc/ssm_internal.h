// ssm_internal.h -- launchers of the selective scan, shared between its translation units.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace ssm {

constexpr int kBlock = 16;      // tokens that are worked on together; a checkpoint lies before each
constexpr int chans(int S) { return S == 64 ? 32 : 64; }   // channels of a workgroup, with S states each

struct Args {
    const void *x, *dt, *b, *c, *z, *dy;
    int64_t x_ld, dt_ld, b_ld, c_ld, z_ld;
    const float *A, *D, *dt_bias, *h0, *dhT;
    void *y, *dx, *ddt, *dz;
    float *ckpt, *hT, *dh0;
    float *part, *part_bc;   // backward: sums per segment ((C, S) of dA, (C) of dD and of ddt_bias); per channel block and token
    float *sum_h, *sum_d;    // per segment slot: what it leaves of a zero state (backward: of a zero gradient), (C, S);
                             // the sum of its steps, (C)
    float* h0_copy;          // where the segments' sums put a copy of h0, or NULL
    const int* cu;
    int softplus, B, T, C, S, G, N;
    int seg, segs;   // tokens of a segment (a multiple of kBlock) and segment slots
    bool split;      // whether a sequence may have more than one segment
    bool zero;       // rows of y outside the sequences are zeroed
    bool halves, halves_sums;   // S = 16, forward and segments' sums: two states to a lane
};

struct StepArgs {
    const void *x, *dt, *b, *c, *z;
    int64_t x_ld, dt_ld, b_ld, c_ld, z_ld;
    const float *A, *D, *dt_bias, *state;
    float* state_out;
    void* y;
    const int* slots;
    int softplus, B, T, C, S, G, P;
    bool bc_four;    // b and c lie at multiples of four values
};

// Sums of the backward's parts.
struct ReduceArgs {
    const float *part, *part_bc;
    float *dA, *dD, *ddt_bias;
    void *db, *dc;
    const int* cu;
    int B, T, C, S, G, N, segs;
    bool zero;       // rows of these and of db, dc outside the sequences are zeroed
    void *dx, *ddt, *dz;
};

// With several segments to a sequence (split): their sums first, then all segments at once.
hipError_t launch_segments(const Args& a, bool bf16, bool backward, hipStream_t s);
hipError_t launch_fwd(const Args& a, bool bf16, hipStream_t s);      // y's rows outside the sequences too
hipError_t launch_bwd(const Args& a, bool bf16, hipStream_t s);
hipError_t launch_reduce(const ReduceArgs& a, bool bf16, hipStream_t s);
hipError_t launch_step(const StepArgs& a, bool bf16, hipStream_t s);

}  // namespace ssm
