// gdr_internal.h -- host-side launchers of the gated delta rule, shared between
// its translation units.  Not part of the public ABI (include/gdr.h is).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace gdr {

// A token operand as bf16 planes: the tensor itself for bf16 inputs, three
// planes of a workspace copy for fp32 inputs.
struct Planes {
    const uint16_t* p;
    int64_t plane;   // elements from one plane to the next
};

struct Args {
    const void *q, *k, *v, *dout;       // token inputs, in_dtype
    const float *g, *beta;              // (tokens, H)
    const float *h0, *dhT;              // (N, H, V, K) or NULL
    const int* cu;                      // packed offsets or NULL
    void *o, *dq, *dk, *dv;             // token outputs, in_dtype
    float *dg, *dbeta;                  // (tokens, H)
    float *hT, *dh0;                    // (N, H, V, K) or NULL
    // Per (slot, head), `stride` floats apart: what the forward leaves for the backward
    // (state entering the chunk V x K, u V x 64, M^T), or NULL; then T and the gates,
    // in the same blocks or, without them, in the workspace.
    float* ckpt;
    int64_t ckpt_stride;
    float* tri;
    int64_t tri_stride;
    Planes qp, kp;                      // set by the launcher
    float *dend, *z;                    // backward: (slots, H, V, K), (slots, H, V, 64)
    float scale;
    int B, T, Hk, H, K, V, N, NC, slots;
};

// bf16 planes of a derived value, and of an input, by input type.
constexpr int kPlanes = 3;
// T and M^T of one chunk of one head: three 32 x 32 blocks in fp32.
constexpr int kTriFloats = 3 * 32 * 32;
// Bytes of one plane of a row-major 64 x 64 matrix.
constexpr int kMatBytes = 64 * 64 * 2;

struct StepArgs {
    const void *q, *k, *v;
    const float *g, *beta;
    const int* slots;
    const float* state;
    float* state_out;
    void* o;
    float scale;
    int B, T, Hk, H, K, V, P;
};

struct ZeroArgs {
    uint32_t* p[8];
    int64_t words[8];   // 32-bit words per token row
    const int* cu;
    int T, N, n;
};

hipError_t launch_zero_outside(const ZeroArgs& a, hipStream_t s);
hipError_t launch_split(const float* q, const float* k, uint16_t* qp, uint16_t* kp, int64_t n, hipStream_t s);
hipError_t launch_prepare(const Args& a, bool bf16, hipStream_t s);
hipError_t launch_fwd_scan(const Args& a, bool bf16, hipStream_t s);
hipError_t launch_bwd_scan(const Args& a, bool bf16, hipStream_t s);
hipError_t launch_grad(const Args& a, bool bf16, hipStream_t s);
hipError_t launch_step(const StepArgs& a, bool bf16, hipStream_t s);

}  // namespace gdr
