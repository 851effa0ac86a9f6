// q4_checks.cuh -- argument checks shared by the translation units of the C ABI (host only).
#pragma once

#include "q4_common.cuh"

namespace q4 {

inline bool valid_group(int32_t g) { return g == 32 || g == 64 || g == 128; }

// Byte ranges [lo, hi) of the arrays of a call, for the check that no output overlaps
// an input or another output (the kernels read inputs while other CTAs store results).
struct Span {
    uintptr_t lo, hi;
};
inline Span span(const void *p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, p == nullptr ? a : a + static_cast<uintptr_t>(bytes)};
}
inline bool overlap(Span a, Span b) { return a.lo < b.hi && b.lo < a.hi; }
inline bool overlaps_any(Span out, const Span *in, int n) {
    for (int i = 0; i < n; ++i)
        if (overlap(out, in[i])) return true;
    return false;
}
// The packed-weight arrays of an N x K matrix of group g (zeros may be null).
inline int weight_spans(const void *codes, const void *scales, const void *zeros, int64_t N, int64_t K, int32_t g,
                        Span *out) {
    const int64_t nb = K / g;
    out[0] = span(codes, N * (K / 2));
    out[1] = span(scales, N * nb * 2);
    out[2] = span(zeros, N * ((nb + 1) / 2));
    return 3;
}

// Scalar checks shared by the packed-weight entry points.
inline int check_shape(int64_t M, int64_t N, int64_t K, int32_t group) {
    if (M < 0 || N < 0 || K < 1 || !valid_group(group) || K % group != 0) return Q4_ERR_INVALID_ARG;
    if (N > 0x7fffffffLL || K > 0x7fffffffLL) return Q4_ERR_UNSUPPORTED;
    return Q4_OK;
}

// Per-call options of an entry point that accepts the flags in `allowed`.
inline int options_from(const q4_run_options_t *o, uint32_t allowed, CallOptions &out) {
    out = CallOptions{};   // built-in defaults, whatever the process-wide settings are
    if (o == nullptr) return Q4_OK;
    if (o->reserved != 0 || (o->flags & ~allowed) != 0) return Q4_ERR_INVALID_ARG;
    out.overlap = (o->flags & Q4_RUN_OVERLAPPED) != 0;
    out.exact_x = (o->flags & Q4_RUN_EXACT_X) != 0;
    if (o->flags & Q4_RUN_WAIT_TIMEOUT) out.wait_ns = o->wait_timeout_ns;
    return Q4_OK;
}

}  // namespace q4
