// ssm_api.hip -- the C ABI of the selective scan (declared in include/ssm.h): argument
// checks on the host, then kernel launches on the caller's stream.
#include <stdint.h>

#include "abi_checks.h"
#include "ssm.h"
#include "ssm_internal.h"

namespace {

using abi::Buf;

struct Shape {
    int64_t tokens, slots, state, ckpt;   // checkpoint slots; values of the states and of the checkpoints
    int64_t part_bc;                      // values of the backward's parts per channel block and token
    int N, seg[2], segs[2];               // forward, backward
    bool split[2], halves, halves_sums[2];
    int64_t per_seg;                      // values of (C, S) and two (C)
    int e;
};

constexpr int64_t kMax = int64_t(1) << 40;
constexpr int64_t kMaxTokens = INT32_MAX - 1024;   // the kernels' 32-bit positions go a few blocks past the end

int64_t slots_of(int B, int T, int N, bool packed, int len) {
    return packed ? T / len + (int64_t)N : (int64_t)B * ((T - 1) / len + 1);
}

wkv7_status dims_ok(int B, int T, int C, int S, int G) {
    if (B < 1 || T < 1 || C < 1 || G < 1 || (S != 16 && S != 32 && S != 64)) return WKV7_ERR_SHAPE;
    if (C % G || (G > 1 && C / G % 64) || C > (1 << 20)) return WKV7_ERR_SHAPE;
    if ((int64_t)B * T > kMax / C || (int64_t)B * T > kMaxTokens) return WKV7_ERR_SHAPE;
    return WKV7_OK;
}

// How many waves a launch has without segments, a wave for 16 channels and 16 of their states
// (packed: in all sequences together, if they are even).
int64_t waves_of(int N, int C, int S) { return (int64_t)N * ((C + 15) / 16) * (S / 16); }

// Tokens of a segment: a sequence is cut into n, at most 128, of 64 tokens at least.  Up to one and a half waves per SIMD
// many short segments, which fill the last round of workgroups evenly; beyond, the segments' sums cost more than the idle
// waves, but for a backward (two waves per SIMD at once) with a little more than one round.  us with n = 1, 2, 4, 8, 16, 32, 64:
//     forward  64 waves of T 8192 845 662 338 176 98 81 77, 256 of 4096 420 340 176 139 127 - -, of 8192 - - - 266 237 232 247,
//              1280 of 4096 622 625 562 518 536, 1792 of 2048 319 376 367 376 394
//     backward 128 of 4096 - - - 205 158 158 174, 576 of 1024 305 287 228 189 180, 1024 of 4096 1245 1112 1047 1055 1067,
//              1280 of 4096 1698 1608 1337 1308 1330, 1792 of 2048 866 976 934 933 969, 2560 of 2048 1368 1277 1288 1313 1370,
//              3584 of 1024 854 878 905 950 1038
// Packed sequences are of lengths that the host does not know: pieces of T are what counts, and twice as many, but
// where the sequences are enough to fill half the chip (backward: the chip) only one of more than T / 4 is cut.  n = 4, 16, 32, 64:
//     backward of 5 sequences, T 8193, 64 waves each 650 293 177 178; of 17, 128 waves each 364 316 310 317, forward 127 197 140 137;
//     of 17, 512 waves each (forward 1, 4, 8: 241 235 330) 904 988 1057 1140
// Where even segments of 64 leave a wave for three quarters of the SIMDs at most they are of 32 (999 tokens of 320 channels, 32 states,
// 6 sequences, forward and backward 27.7 + 50.6 -> 22.4 + 38.8; but 8 x 1024 of 256 channels 32.1 + 56.9 -> 37.5 + 65.5).
int segment_of(int N, int T, int C, int S, bool packed, bool halves, bool back) {
    const int64_t waves = waves_of(N, C, S), each = waves_of(1, C, S);
    int64_t n = 1;
    if (packed) n = waves > (back ? 4096 : 2048) ? 4 : 8192 / each > 8 ? 8192 / each : 8;
    else if (!halves && waves <= 1536) n = 4096 / waves > 8 ? 4096 / waves : 8;
    else if (back && waves > 2048 && waves <= 3 * 1024) n = 2;
    if (n > 128) n = 128;
    int64_t seg = n > 1 ? (T + n - 1) / n : T;
    const int64_t least = T > 64 && (packed ? each : waves) * ((T + 63) / 64) <= 768 ? 32 : 64;
    if (seg < least) seg = least;
    if (seg > T) seg = T;
    return (int)((seg + ssm::kBlock - 1) / ssm::kBlock * ssm::kBlock);
}

wkv7_status shape(int B, int T, int C, int S, int G, int N, bool packed, Shape* s) {
    if (dims_ok(B, T, C, S, G) != WKV7_OK || (packed && (B != 1 || N < 1))) return WKV7_ERR_SHAPE;
    s->N = packed ? N : B;
    s->tokens = (int64_t)B * T;
    s->slots = slots_of(B, T, N, packed, ssm::kBlock);
    const int64_t blocks = (C + ssm::chans(S) - 1) / ssm::chans(S);
    // Forward with two states to a lane instead of segments: twice the waves for a twelfth more instructions, in workgroups
    // of eight of which a CU holds one, so where they are nearly as many as the CUs (4096 channels, T 4096, against segments:
    // 4 sequences, 1024 waves without halves, 363 us to 433, but 3, 768 waves, 353 to 340; 1152 waves of T 1024 180 to 156).
    const int64_t waves = waves_of(s->N, C, S);
    s->halves = S == 16 && !packed && waves > 832 && waves <= 1024;
    for (int back = 0; back < 2; ++back) {
        s->seg[back] = segment_of(s->N, T, C, S, packed, !back && s->halves, back);
        s->split[back] = s->seg[back] < T;
        // the segments' sums alike, up to three waves per SIMD (backward of 10 x 2048 tokens of 4096 channels, 2560 waves: 1348
        // -> 1280 us, of 12 x 2048 of 3500, 2628: 1527 -> 1466; but forward of 8 x 512 of 1024, 3584 waves: 42.8 -> 46.2, of
        // 12 x 1024 of 768, 4032: 84 -> 88)
        s->halves_sums[back] = S == 16 && !packed && waves * ((T - 1) / s->seg[back]) <= 3 * 1024;
        const int64_t segs = slots_of(B, T, N, packed, s->seg[back]);
        // a launch takes fewer than 2^32 threads: at most 512 for each segment and channel block
        if (segs > ((1 << 23) - 1) / blocks) return WKV7_ERR_SHAPE;
        s->segs[back] = (int)segs;
    }
    if (s->slots > INT32_MAX) return WKV7_ERR_SHAPE;
    s->per_seg = (int64_t)C * (S + 2);
    s->state = (int64_t)s->N * C * S;
    s->ckpt = s->slots * C * S;
    if (s->slots > kMax / (C * S) || s->N > kMax / (C * S)) return WKV7_ERR_SHAPE;
    s->part_bc = blocks * s->tokens * 2 * S;
    return WKV7_OK;
}

// What the segments leave, and h0's copy; behind the parts of the backward.  Never 0, so that a size of 0 is
// always one of invalid shapes, and a NULL workspace always an error.
int64_t fwd_ws(const Shape& s) { return s.split[0] ? (s.segs[0] * s.per_seg + s.state) * 4 : 256; }
int64_t bwd_ws(const Shape& s) { return (s.part_bc + s.segs[1] * s.per_seg * (s.split[1] ? 2 : 1)) * 4; }
int64_t span(int64_t rows, int64_t ld, int64_t n, int e) { return ((rows - 1) * ld + n) * e; }
constexpr int64_t kMaxLd = 1 << 24;   // over sequences: 16 rows are addressed with 32-bit byte offsets; the step has 64 bits
bool lds_ok(int64_t tokens, int C, int GS, int64_t x, int64_t dt, int64_t b, int64_t c, const void* z, int64_t z_ld, int64_t max_ld) {
    const int64_t most = kMax / tokens < max_ld ? kMax / tokens : max_ld;
    return x >= C && dt >= C && b >= GS && c >= GS && (!z || z_ld >= C) && x <= most && dt <= most && b <= most && c <= most &&
           (!z || z_ld <= most);
}
wkv7_status status_of(hipError_t e) { return e == hipSuccess ? WKV7_OK : WKV7_ERR_HIP; }

}  // namespace

extern "C" {

int64_t ssm_slots(int B, int T, int N, int packed) {
    if (B < 1 || T < 1 || (packed && (N < 1 || B != 1))) return 0;
    return slots_of(B, T, N, packed != 0, ssm::kBlock);
}

size_t ssm_ckpt_bytes(int B, int T, int C, int S, int G, int N, int packed) {
    Shape s;
    return shape(B, T, C, S, G, N, packed != 0, &s) == WKV7_OK ? (size_t)s.ckpt * 4 : 0;
}
size_t ssm_fwd_workspace_bytes(int B, int T, int C, int S, int G, int N, int packed) {
    Shape s;
    return shape(B, T, C, S, G, N, packed != 0, &s) == WKV7_OK ? (size_t)fwd_ws(s) : 0;
}
size_t ssm_bwd_workspace_bytes(int B, int T, int C, int S, int G, int N, int packed) {
    Shape s;
    return shape(B, T, C, S, G, N, packed != 0, &s) == WKV7_OK ? (size_t)bwd_ws(s) : 0;
}

wkv7_status ssm_fwd(int B, int T, int C, int S, int G, wkv7_dtype in_dtype, const void* x, int64_t x_ld, const void* dt,
                    int64_t dt_ld, const float* A, const void* b, int64_t b_ld, const void* c, int64_t c_ld,
                    const float* D, const void* z, int64_t z_ld, const float* dt_bias, int softplus,
                    const int32_t* cu_seqlens, int N, int zero_outside, const float* h0, void* y, float* ckpt, float* hT, void* workspace,
                    size_t workspace_bytes, void* stream) {
    if (in_dtype != WKV7_F32 && in_dtype != WKV7_BF16) return WKV7_ERR_DTYPE;
    Shape s;
    wkv7_status st = shape(B, T, C, S, G, N, cu_seqlens != nullptr, &s);
    if (st != WKV7_OK) return st;
    if (!lds_ok(s.tokens, C, G * S, x_ld, dt_ld, b_ld, c_ld, z, z_ld, kMaxLd)) return WKV7_ERR_SHAPE;
    const int e = in_dtype == WKV7_BF16 ? 2 : 4;
    const int64_t need = fwd_ws(s), n = s.tokens;
    const Buf bufs[] = {{x, span(n, x_ld, C, e), true, false, e}, {dt, span(n, dt_ld, C, e), true, false, e},
                        {A, (int64_t)C * S * 4, true, false, 16}, {b, span(n, b_ld, G * S, e), true, false, e},
                        {c, span(n, c_ld, G * S, e), true, false, e}, {D, C * 4LL, false, false, 4},
                        {z, span(n, z_ld, C, e), false, false, e}, {dt_bias, C * 4LL, false, false, 4},
                        {cu_seqlens, (s.N + 1) * 4LL, false, false, 4}, {h0, s.state * 4, false, false, 16},
                        {y, n * C * e, false, true, e}, {ckpt, s.ckpt * 4, false, true, 16},
                        {hT, s.state * 4, false, true, 16}, {workspace, need, false, true, 16}};
    if (!y && !ckpt && !hT) return WKV7_ERR_ARG;
    st = abi::check(bufs, h0 == hT ? h0 : nullptr);
    if (st != WKV7_OK) return st;
    if (!workspace || workspace_bytes < (size_t)need) return WKV7_ERR_WORKSPACE;
    ssm::Args a = {};
    a.x = x; a.dt = dt; a.b = b; a.c = c; a.z = z; a.x_ld = x_ld; a.dt_ld = dt_ld; a.b_ld = b_ld; a.c_ld = c_ld;
    a.z_ld = z_ld; a.A = A; a.D = D; a.dt_bias = dt_bias; a.h0 = h0; a.y = y; a.ckpt = ckpt; a.hT = hT; a.cu = cu_seqlens;
    a.softplus = softplus; a.B = B; a.T = T; a.C = C; a.S = S; a.G = G; a.N = s.N; a.seg = s.seg[0]; a.segs = s.segs[0];
    a.split = s.split[0];
    a.zero = cu_seqlens && y && zero_outside;
    // h0 in place: every segment starts from h0, the last one writes hT, so they read a copy
    if (a.split && h0 && h0 == hT) a.h0_copy = static_cast<float*>(workspace);
    a.sum_h = static_cast<float*>(workspace) + s.state;
    a.sum_d = a.sum_h + (int64_t)s.segs[0] * C * S;
    a.halves = s.halves; a.halves_sums = s.halves_sums[0];
    hipStream_t hs = static_cast<hipStream_t>(stream);
    hipError_t err = a.split ? ssm::launch_segments(a, in_dtype == WKV7_BF16, false, hs) : hipSuccess;
    if (a.h0_copy) a.h0 = a.h0_copy;
    if (err == hipSuccess) err = ssm::launch_fwd(a, in_dtype == WKV7_BF16, hs);
    return status_of(err);
}

wkv7_status ssm_bwd(int B, int T, int C, int S, int G, wkv7_dtype in_dtype, const void* dy, const float* dhT,
                    const void* x, int64_t x_ld, const void* dt, int64_t dt_ld, const float* A, const void* b,
                    int64_t b_ld, const void* c, int64_t c_ld, const float* D, const void* z, int64_t z_ld,
                    const float* dt_bias, int softplus, const int32_t* cu_seqlens, int N, int zero_outside, const float* ckpt, void* dx,
                    void* ddt, float* dA, void* db, void* dc, float* dD, void* dz, float* ddt_bias, float* dh0,
                    void* workspace, size_t workspace_bytes, void* stream) {
    if (in_dtype != WKV7_F32 && in_dtype != WKV7_BF16) return WKV7_ERR_DTYPE;
    Shape s;
    wkv7_status st = shape(B, T, C, S, G, N, cu_seqlens != nullptr, &s);
    if (st != WKV7_OK) return st;
    if (!lds_ok(s.tokens, C, G * S, x_ld, dt_ld, b_ld, c_ld, z, z_ld, kMaxLd)) return WKV7_ERR_SHAPE;
    if ((D != nullptr) != (dD != nullptr) || (z != nullptr) != (dz != nullptr)) return WKV7_ERR_ARG;
    const int e = in_dtype == WKV7_BF16 ? 2 : 4;
    const int64_t n = s.tokens, rows = n * C * e, brows = n * G * S * e, sb = s.state * 4;
    const Buf bufs[] = {{dy, rows, true, false, e}, {dhT, sb, false, false, 16}, {x, span(n, x_ld, C, e), true, false, e},
                        {dt, span(n, dt_ld, C, e), true, false, e}, {A, (int64_t)C * S * 4, true, false, 16},
                        {b, span(n, b_ld, G * S, e), true, false, e}, {c, span(n, c_ld, G * S, e), true, false, e},
                        {D, C * 4LL, false, false, 4}, {z, span(n, z_ld, C, e), false, false, e},
                        {dt_bias, C * 4LL, false, false, 4}, {cu_seqlens, (s.N + 1) * 4LL, false, false, 4},
                        {ckpt, s.ckpt * 4, true, false, 16}, {dx, rows, true, true, e}, {ddt, rows, true, true, e},
                        {dA, (int64_t)C * S * 4, true, true, 4}, {db, brows, true, true, e}, {dc, brows, true, true, e},
                        {dD, C * 4LL, false, true, 4}, {dz, rows, false, true, e}, {ddt_bias, C * 4LL, false, true, 4},
                        {dh0, sb, false, true, 16}, {workspace, bwd_ws(s), false, true, 16}};
    st = abi::check(bufs);
    if (st != WKV7_OK) return st;
    if (!workspace || workspace_bytes < (size_t)bwd_ws(s)) return WKV7_ERR_WORKSPACE;
    ssm::Args a = {};
    a.x = x; a.dt = dt; a.b = b; a.c = c; a.z = z; a.x_ld = x_ld; a.dt_ld = dt_ld; a.b_ld = b_ld; a.c_ld = c_ld;
    a.z_ld = z_ld; a.A = A; a.D = D; a.dt_bias = dt_bias; a.dy = dy; a.dhT = dhT; a.ckpt = const_cast<float*>(ckpt);
    a.dx = dx; a.ddt = ddt; a.dz = dz; a.dh0 = dh0; a.cu = cu_seqlens;
    a.softplus = softplus; a.B = B; a.T = T; a.C = C; a.S = S; a.G = G; a.N = s.N; a.seg = s.seg[1]; a.segs = s.segs[1];
    float* ws = static_cast<float*>(workspace);
    a.part_bc = ws;
    a.part = ws + s.part_bc;
    a.split = s.split[1]; a.halves_sums = s.halves_sums[1];
    a.sum_h = a.part + s.segs[1] * s.per_seg;
    a.sum_d = a.sum_h + (int64_t)s.segs[1] * C * S;
    ssm::ReduceArgs r = {};
    r.part = a.part; r.part_bc = a.part_bc;
    r.dA = dA; r.dD = dD; r.ddt_bias = ddt_bias; r.db = db; r.dc = dc; r.cu = cu_seqlens;
    r.zero = cu_seqlens && zero_outside;
    r.dx = dx; r.ddt = ddt; r.dz = dz;
    r.B = B; r.T = T; r.C = C; r.S = S; r.G = G; r.N = s.N; r.segs = s.segs[1];
    hipStream_t hs = static_cast<hipStream_t>(stream);
    hipError_t err = a.split ? ssm::launch_segments(a, in_dtype == WKV7_BF16, true, hs) : hipSuccess;
    if (err == hipSuccess) err = ssm::launch_bwd(a, in_dtype == WKV7_BF16, hs);
    if (err == hipSuccess) err = ssm::launch_reduce(r, in_dtype == WKV7_BF16, hs);
    return status_of(err);
}

wkv7_status ssm_step(int B, int T, int C, int S, int G, wkv7_dtype in_dtype, const void* x, int64_t x_ld, const void* dt,
                     int64_t dt_ld, const float* A, const void* b, int64_t b_ld, const void* c, int64_t c_ld,
                     const float* D, const void* z, int64_t z_ld, const float* dt_bias, int softplus,
                     const int32_t* slots, int P, const float* state, float* state_out, void* y, void* stream) {
    if (in_dtype != WKV7_F32 && in_dtype != WKV7_BF16) return WKV7_ERR_DTYPE;
    wkv7_status st = dims_ok(B, T, C, S, G);
    if (st != WKV7_OK) return st;
    if (P < 1 || (!slots && P < B) || P > kMax / ((int64_t)C * S)) return WKV7_ERR_SHAPE;
    if (B > (1 << 24) / ((C + 15) / 16 + 1)) return WKV7_ERR_SHAPE;   // a launch takes fewer than 2^32 threads
    const int64_t n = (int64_t)B * T, sb = (int64_t)P * C * S * 4;
    if (!lds_ok(n, C, G * S, x_ld, dt_ld, b_ld, c_ld, z, z_ld, kMax)) return WKV7_ERR_SHAPE;
    const int e = in_dtype == WKV7_BF16 ? 2 : 4;
    const Buf bufs[] = {{x, span(n, x_ld, C, e), true, false, e}, {dt, span(n, dt_ld, C, e), true, false, e},
                        {A, (int64_t)C * S * 4, true, false, 16}, {b, span(n, b_ld, G * S, e), true, false, e},
                        {c, span(n, c_ld, G * S, e), true, false, e}, {D, C * 4LL, false, false, 4},
                        {z, span(n, z_ld, C, e), false, false, e}, {dt_bias, C * 4LL, false, false, 4},
                        {slots, B * 4LL, false, false, 4}, {state, sb, true, false, 16}, {state_out, sb, true, true, 16},
                        {y, n * C * e, true, true, e}};
    st = abi::check(bufs, state == state_out ? state : nullptr);
    if (st != WKV7_OK) return st;
    ssm::StepArgs a = {};
    a.x = x; a.dt = dt; a.b = b; a.c = c; a.z = z; a.x_ld = x_ld; a.dt_ld = dt_ld; a.b_ld = b_ld; a.c_ld = c_ld;
    a.z_ld = z_ld; a.A = A; a.D = D; a.dt_bias = dt_bias; a.state = state; a.state_out = state_out; a.y = y;
    a.slots = slots; a.softplus = softplus; a.B = B; a.T = T; a.C = C; a.S = S; a.G = G; a.P = P;
    a.bc_four = (reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c)) % (4 * e) == 0 && (b_ld | c_ld) % 4 == 0;
    return status_of(ssm::launch_step(a, in_dtype == WKV7_BF16, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
