// gdr_api.hip -- the C ABI of the gated delta rule (declared in include/gdr.h):
// argument checks on the host, then kernel launches on the caller's stream.
#include <stdint.h>

#include "abi_checks.h"
#include "gdr.h"
#include "gdr_internal.h"

namespace {

using abi::Buf;

constexpr int kChunk = 64;
constexpr int kGateFloats = 320;   // per chunk and head, as the kernels lay them out

struct Shape {
    int64_t slots, tokens, q_elems, v_elems, gate_elems, state_elems, ckpt_elems;
    int64_t ckpt_stride, tri_stride, tri_bytes, split_bytes, dend_bytes, z_bytes;
    int N;
    bool bf16;
    int64_t e() const { return bf16 ? 2 : 4; }
};

int64_t slots_of(int B, int T, int N, bool packed) {
    return packed ? T / kChunk + (int64_t)N : (int64_t)B * ((T + (int64_t)kChunk - 1) / kChunk);
}

wkv7_status heads_ok(int B, int T, int Hk, int H, int K, int V) {
    if (B < 1 || T < 1 || Hk < 1 || H < 1 || H % Hk || (K != 64 && K != 128) || (V != 64 && V != 128))
        return WKV7_ERR_SHAPE;
    return WKV7_OK;
}

wkv7_status shape(int B, int T, int Hk, int H, int K, int V, int dt, int N, bool packed, Shape* s) {
    if (dt != WKV7_F32 && dt != WKV7_BF16) return WKV7_ERR_DTYPE;
    if (heads_ok(B, T, Hk, H, K, V) != WKV7_OK) return WKV7_ERR_SHAPE;
    if (packed && (B != 1 || N < 1)) return WKV7_ERR_SHAPE;
    s->bf16 = dt == WKV7_BF16;
    s->N = packed ? N : B;
    s->slots = slots_of(B, T, N, packed);
    s->tokens = (int64_t)B * T;
    // a launch takes fewer than 2^32 threads: at most 2 x 512 for each chunk and head (and 15 workgroups more), 8 x
    // 448 for each sequence and head
    if (s->slots > ((1 << 22) - 16) / H || s->N > (1 << 20) / H) return WKV7_ERR_SHAPE;
    if (s->tokens > (int64_t(1) << 40) / ((int64_t)H * 128)) return WKV7_ERR_SHAPE;
    if ((int64_t)kChunk * H * V * 4 > INT32_MAX) return WKV7_ERR_SHAPE;   // 32-bit offsets inside a chunk
    s->q_elems = s->tokens * Hk * K;
    s->v_elems = s->tokens * H * V;
    s->gate_elems = s->tokens * H;
    s->state_elems = (int64_t)s->N * H * V * K;
    s->tri_stride = gdr::kTriFloats + kGateFloats;
    s->ckpt_stride = (int64_t)(K + kChunk) * V + gdr::kTriFloats + s->tri_stride;
    s->ckpt_elems = s->slots * H * s->ckpt_stride;
    s->tri_bytes = s->slots * H * s->tri_stride * 4;
    s->split_bytes = s->bf16 ? 0 : 2 * 3 * s->q_elems * 2;
    s->dend_bytes = s->slots * H * (int64_t)V * K * 4;
    s->z_bytes = s->slots * H * (int64_t)V * kChunk * 4;
    return WKV7_OK;
}

// T and gates of a forward without checkpoints (with them they lie there), planes of fp32 inputs;
// the backward's state gradients and Z, and those planes.  Never 0, so that a size of 0 is always
// one of invalid shapes, and a NULL workspace always an error.
constexpr int64_t kMinWorkspace = 256;
int64_t fwd_ws(const Shape& s, bool ckpt) {
    const int64_t n = (ckpt ? 0 : s.tri_bytes) + s.split_bytes;
    return n < kMinWorkspace ? kMinWorkspace : n;
}
int64_t bwd_ws(const Shape& s) { return s.dend_bytes + s.z_bytes + s.split_bytes; }

wkv7_status status_of(hipError_t e) { return e == hipSuccess ? WKV7_OK : WKV7_ERR_HIP; }

// Arguments shared by both directions.  `planes`: where the planes of fp32 q and k go.
gdr::Args args_of(int B, int T, int Hk, int H, int K, int V, const Shape& s, const void* q, const void* k,
                  const void* v, const float* g, const float* beta, const int32_t* cu, float scale, char* planes) {
    gdr::Args a = {};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.cu = cu; a.scale = scale;
    a.B = B; a.T = T; a.Hk = Hk; a.H = H; a.K = K; a.V = V; a.N = s.N;
    a.slots = (int)s.slots;
    a.NC = cu ? (int)s.slots : (T + kChunk - 1) / kChunk;
    a.ckpt_stride = s.ckpt_stride;
    if (s.bf16) {
        a.qp = {static_cast<const uint16_t*>(q), 0};
        a.kp = {static_cast<const uint16_t*>(k), 0};
    } else {
        uint16_t* p = reinterpret_cast<uint16_t*>(planes);
        a.qp = {p, s.q_elems};
        a.kp = {p + 3 * s.q_elems, s.q_elems};
    }
    return a;
}

// T and gates behind the rest of each checkpoint block.
void tri_in_ckpt(gdr::Args* a) {
    a->tri = a->ckpt + (int64_t)(a->K + kChunk) * a->V + gdr::kTriFloats;
    a->tri_stride = a->ckpt_stride;
}

hipError_t split(const gdr::Args& a, const Shape& s, hipStream_t st) {
    if (s.bf16) return hipSuccess;
    return gdr::launch_split(static_cast<const float*>(a.q), static_cast<const float*>(a.k),
                             const_cast<uint16_t*>(a.qp.p), const_cast<uint16_t*>(a.kp.p), s.q_elems, st);
}

}  // namespace

extern "C" {

int64_t gdr_slots(int B, int T, int N, int packed) {
    if (B < 1 || T < 1 || (packed && (N < 1 || B != 1))) return 0;
    return slots_of(B, T, N, packed != 0);
}

size_t gdr_ckpt_bytes(int B, int T, int Hk, int H, int K, int V, int N, int packed) {
    Shape s;
    return shape(B, T, Hk, H, K, V, WKV7_BF16, N, packed != 0, &s) == WKV7_OK ? (size_t)s.ckpt_elems * 4 : 0;
}

size_t gdr_fwd_workspace_bytes(int B, int T, int Hk, int H, int K, int V, wkv7_dtype in_dtype, int N, int packed) {
    Shape s;
    return shape(B, T, Hk, H, K, V, in_dtype, N, packed != 0, &s) == WKV7_OK ? (size_t)fwd_ws(s, false) : 0;
}

size_t gdr_fwd_train_workspace_bytes(int B, int T, int Hk, int H, int K, int V, wkv7_dtype in_dtype, int N, int packed) {
    Shape s;
    return shape(B, T, Hk, H, K, V, in_dtype, N, packed != 0, &s) == WKV7_OK ? (size_t)fwd_ws(s, true) : 0;
}

size_t gdr_bwd_workspace_bytes(int B, int T, int Hk, int H, int K, int V, wkv7_dtype in_dtype, int N, int packed) {
    Shape s;
    return shape(B, T, Hk, H, K, V, in_dtype, N, packed != 0, &s) == WKV7_OK ? (size_t)bwd_ws(s) : 0;
}

wkv7_status gdr_fwd(int B, int T, int Hk, int H, int K, int V, wkv7_dtype in_dtype, const void* q, const void* k,
                    const void* v, const float* g, const float* beta, const int32_t* cu_seqlens, int N, float scale,
                    const float* h0, void* o, float* ckpt, float* hT, void* workspace, size_t workspace_bytes,
                    void* stream) {
    Shape s;
    wkv7_status st = shape(B, T, Hk, H, K, V, in_dtype, N, cu_seqlens != nullptr, &s);
    if (st != WKV7_OK) return st;
    const Buf bufs[] = {{q, s.q_elems * s.e(), true, false, 16}, {k, s.q_elems * s.e(), true, false, 16},
                        {v, s.v_elems * s.e(), true, false, 16}, {g, s.gate_elems * 4, true, false, 4},
                        {beta, s.gate_elems * 4, true, false, 4}, {cu_seqlens, (s.N + 1) * 4LL, false, false, 4},
                        {h0, s.state_elems * 4, false, false, 16}, {o, s.v_elems * s.e(), false, true, 16},
                        {ckpt, s.ckpt_elems * 4, false, true, 16}, {hT, s.state_elems * 4, false, true, 16},
                        {workspace, fwd_ws(s, ckpt != nullptr), false, true, 16}};
    if (!o && !ckpt && !hT) return WKV7_ERR_ARG;
    st = abi::check(bufs, h0 == hT ? h0 : nullptr);
    if (st != WKV7_OK) return st;
    if (!workspace || workspace_bytes < (size_t)fwd_ws(s, ckpt != nullptr)) return WKV7_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    gdr::Args a = args_of(B, T, Hk, H, K, V, s, q, k, v, g, beta, cu_seqlens, scale, ws + (ckpt ? 0 : s.tri_bytes));
    a.h0 = h0; a.o = o; a.ckpt = ckpt; a.hT = hT;
    if (ckpt) {
        tri_in_ckpt(&a);
    } else {
        a.tri = reinterpret_cast<float*>(ws);
        a.tri_stride = s.tri_stride;
    }
    hipStream_t hs = static_cast<hipStream_t>(stream);
    hipError_t e = split(a, s, hs);
    if (e == hipSuccess) e = gdr::launch_prepare(a, s.bf16, hs);
    if (e == hipSuccess) e = gdr::launch_fwd_scan(a, s.bf16, hs);
    return status_of(e);
}

wkv7_status gdr_bwd(int B, int T, int Hk, int H, int K, int V, wkv7_dtype in_dtype, const void* dout,
                    const float* dhT, const void* q, const void* k, const void* v, const float* g, const float* beta,
                    const int32_t* cu_seqlens, int N, float scale, const float* ckpt, void* dq, void* dk, void* dv,
                    float* dg, float* dbeta, float* dh0, void* workspace, size_t workspace_bytes, void* stream) {
    Shape s;
    wkv7_status st = shape(B, T, Hk, H, K, V, in_dtype, N, cu_seqlens != nullptr, &s);
    if (st != WKV7_OK) return st;
    const int64_t qb = s.q_elems * s.e(), vb = s.v_elems * s.e(), gb = s.gate_elems * 4, sb = s.state_elems * 4;
    const Buf bufs[] = {{dout, vb, true, false, 16}, {dhT, sb, false, false, 16}, {q, qb, true, false, 16},
                        {k, qb, true, false, 16}, {v, vb, true, false, 16}, {g, gb, true, false, 4},
                        {beta, gb, true, false, 4}, {cu_seqlens, (s.N + 1) * 4LL, false, false, 4},
                        {ckpt, s.ckpt_elems * 4, true, false, 16}, {dq, qb, true, true, 16}, {dk, qb, true, true, 16},
                        {dv, vb, true, true, 16}, {dg, gb, true, true, 4}, {dbeta, gb, true, true, 4},
                        {dh0, sb, false, true, 16}, {workspace, bwd_ws(s), false, true, 16}};
    st = abi::check(bufs);
    if (st != WKV7_OK) return st;
    if (!workspace || workspace_bytes < (size_t)bwd_ws(s)) return WKV7_ERR_WORKSPACE;
    char* ws = static_cast<char*>(workspace);
    gdr::Args a = args_of(B, T, Hk, H, K, V, s, q, k, v, g, beta, cu_seqlens, scale, ws + s.dend_bytes + s.z_bytes);
    a.dout = dout; a.dhT = dhT; a.ckpt = const_cast<float*>(ckpt);
    a.dend = reinterpret_cast<float*>(ws);
    a.z = reinterpret_cast<float*>(ws + s.dend_bytes);
    tri_in_ckpt(&a);
    a.dq = dq; a.dk = dk; a.dv = dv; a.dg = dg; a.dbeta = dbeta; a.dh0 = dh0;
    hipStream_t hs = static_cast<hipStream_t>(stream);
    hipError_t e = split(a, s, hs);
    if (e == hipSuccess) e = gdr::launch_bwd_scan(a, s.bf16, hs);
    if (e == hipSuccess) e = gdr::launch_grad(a, s.bf16, hs);
    return status_of(e);
}

wkv7_status gdr_zero_outside(int T, int N, const int32_t* cu_seqlens, int n, void* const* ptrs,
                             const int64_t* row_bytes, void* stream) {
    if (T < 1 || N < 1) return WKV7_ERR_SHAPE;
    if (!cu_seqlens || !ptrs || !row_bytes || n < 1 || n > 8) return WKV7_ERR_ARG;
    gdr::ZeroArgs a = {};
    a.cu = cu_seqlens; a.T = T; a.N = N; a.n = n;
    for (int i = 0; i < n; ++i) {
        if (!ptrs[i]) return WKV7_ERR_ARG;
        if (row_bytes[i] < 4 || row_bytes[i] % 4) return WKV7_ERR_SHAPE;
        if (reinterpret_cast<uintptr_t>(ptrs[i]) & 3u) return WKV7_ERR_ALIGN;
        a.p[i] = static_cast<uint32_t*>(ptrs[i]);
        a.words[i] = row_bytes[i] / 4;
    }
    return status_of(gdr::launch_zero_outside(a, static_cast<hipStream_t>(stream)));
}

wkv7_status gdr_step(int B, int T, int Hk, int H, int K, int V, wkv7_dtype in_dtype, const void* q, const void* k,
                     const void* v, const float* g, const float* beta, const int32_t* slots, int P, float scale,
                     const float* state, float* state_out, void* o, void* stream) {
    if (in_dtype != WKV7_F32 && in_dtype != WKV7_BF16) return WKV7_ERR_DTYPE;
    wkv7_status st = heads_ok(B, T, Hk, H, K, V);
    if (st != WKV7_OK) return st;
    if (P < 1 || (!slots && P < B)) return WKV7_ERR_SHAPE;
    if (B > ((1 << 22) - 1) / H) return WKV7_ERR_SHAPE;           // at most 4 x 256 threads for each row and head
    const int64_t tokens = (int64_t)B * T, lim = (int64_t(1) << 40) / ((int64_t)H * 128);
    if (tokens > lim || (int64_t)P * 128 > lim) return WKV7_ERR_SHAPE;
    const int64_t e = in_dtype == WKV7_BF16 ? 2 : 4, qb = tokens * Hk * K * e, vb = tokens * H * V * e;
    const int64_t gb = tokens * H * 4, sb = (int64_t)P * H * V * K * 4;
    const Buf bufs[] = {{q, qb, true, false, 16}, {k, qb, true, false, 16}, {v, vb, true, false, 16},
                        {g, gb, true, false, 4}, {beta, gb, true, false, 4}, {slots, B * 4LL, false, false, 4},
                        {state, sb, true, false, 16}, {state_out, sb, true, true, 16}, {o, vb, true, true, 16}};
    st = abi::check(bufs, state == state_out ? state : nullptr);
    if (st != WKV7_OK) return st;
    gdr::StepArgs a = {};
    a.q = q; a.k = k; a.v = v; a.g = g; a.beta = beta; a.slots = slots; a.state = state; a.state_out = state_out;
    a.o = o; a.scale = scale; a.B = B; a.T = T; a.Hk = Hk; a.H = H; a.K = K; a.V = V; a.P = P;
    return status_of(gdr::launch_step(a, in_dtype == WKV7_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
