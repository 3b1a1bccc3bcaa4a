// checks.h -- argument checks shared by the C-ABI translation units of the
// training operators (layer norm, the norm backward passes, the softmax with a
// relative position bias).  Host code only, no CUDA call.
#pragma once
#include <cstdint>

namespace rmsnorm {

// A buffer an entry point was given: address (0 = absent) and size in bytes.
struct Span {
    uintptr_t p;
    uint64_t n;
};

inline Span span(const void* p, uint64_t n) { return {reinterpret_cast<uintptr_t>(p), n}; }

inline bool overlaps(const Span& a, const Span& b) {
    return a.p && b.p && a.n && b.n && a.p < b.p + b.n && b.p < a.p + a.n;
}

// True if `out` overlaps any of the `n` spans, an exact alias of one of the
// first `same` spans (same address) excepted: an elementwise operator may
// write its result over an input of the same layout.
inline bool clashes(const Span& out, const Span* s, int n, int same) {
    for (int i = 0; i < n; ++i)
        if (overlaps(out, s[i]) && !(i < same && out.p == s[i].p)) return true;
    return false;
}

inline bool aligned(const void* p, uintptr_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Widest vector (16 bytes down to one element of sz bytes) that the addresses
// in `bits` (ORed together) and a row pitch allow.
inline int widest_vector(uintptr_t bits, int64_t pitch, int sz) {
    for (int v = 16; v > sz; v >>= 1)
        if (bits % v == 0 && pitch % v == 0) return v;
    return sz;
}

inline int64_t div_up(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace rmsnorm
