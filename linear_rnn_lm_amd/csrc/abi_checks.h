// abi_checks.h -- host-side argument checks of the entry points beside the recurrence's
// (gated delta rule, layer norm, selective scan, short convolution, block norm): NULL,
// alignment and aliasing, before any launch.
#pragma once

#include <stdint.h>

#include "wkv7.h"

namespace abi {

struct Buf {
    const void* p;
    int64_t bytes;
    bool required, output;
    int align;
};

inline bool overlap(const Buf& a, const Buf& b) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return a.p && b.p && a.bytes > 0 && b.bytes > 0 && x < y + (uintptr_t)b.bytes && y < x + (uintptr_t)a.bytes;
}

// `same`: one pointer that may be given both as an input and as an output (an
// update in place); everything else that overlaps an output is refused.
template <int N>
wkv7_status check(const Buf (&b)[N], const void* same = nullptr) {
    for (const Buf& x : b)
        if (x.required && !x.p) return WKV7_ERR_ARG;
    for (const Buf& x : b)
        if (x.p && (reinterpret_cast<uintptr_t>(x.p) & (uintptr_t)(x.align - 1))) return WKV7_ERR_ALIGN;
    for (int i = 0; i < N; ++i)
        for (int j = 0; j < N; ++j) {
            if (i == j || !b[i].output || (b[j].output && j < i)) continue;
            if (same && b[i].p == same && b[j].p == same) continue;
            if (overlap(b[i], b[j])) return WKV7_ERR_ALIAS;
        }
    return WKV7_OK;
}

}  // namespace abi
