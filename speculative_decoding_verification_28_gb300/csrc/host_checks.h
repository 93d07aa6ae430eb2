// host_checks.h -- what the entry points check about their arguments on the
// host (internal).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "specverify.h"

namespace spec {

inline bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
inline int launched(cudaError_t e) { return e == cudaSuccess ? SPEC_OK : SPEC_ECUDA; }

// A large tensor of a call, in bytes (null: none).
struct Span {
    uintptr_t at, n;
};
// n elements of e bytes from element `first` of p; sizes past what memory can
// hold are cut to that, so that nothing wraps
inline Span span(const void *p, double first, double n, int e)
{
    const double top = 1e18;
    const double f = first * e, x = n * e;
    return Span{p ? reinterpret_cast<uintptr_t>(p) + (uintptr_t)(f < top ? f : top) : 0,
                p ? (uintptr_t)(x < top ? x : top) : 0};
}
inline bool overlap(const Span &a, const Span &b) { return a.n && b.n && a.at < b.at + b.n && b.at < a.at + a.n; }

inline bool int_arrays_ok(const void *a, const void *b, const void *c, const void *d, const void *e)
{
    return aligned(a, 4) && aligned(b, 4) && aligned(c, 4) && aligned(d, 4) && aligned(e, 4);
}

// Waits of attention calls: clocks until the next one gives up (about 2 s, or
// what spec_attend_starve_next said for the thread's next call), and whether
// that is a test's.
struct Waits {
    long long clocks;
    int starve;
};
Waits next_waits();

}  // namespace spec
