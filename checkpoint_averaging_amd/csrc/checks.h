// Argument checks shared by the C entry points (host code, no launches).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dlmerge.h"

namespace dlk {

struct Span {
    uintptr_t lo, hi;                // [lo, hi)
    bool overlaps(const Span& o) const { return lo < o.hi && o.lo < hi; }
    bool same(const Span& o) const { return lo == o.lo && hi == o.hi; }
};

inline Span span_of(const void* p, int64_t bytes) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    return Span{a, a + static_cast<uintptr_t>(bytes)};
}

// A HIP error left pending on this thread by earlier work (a failed call, or
// an asynchronous fault the runtime has reported) is the caller's to see:
// the library neither launches over it nor clears it.  "Not ready" from an
// event or stream query is a status, not a failure: it is consumed so that
// the launch status read after this call's own launch is that launch's.
inline bool hip_error_pending() {
    const hipError_t e = hipPeekAtLastError();
    if (e == hipErrorNotReady) {
        (void)hipGetLastError();
        return false;
    }
    return e != hipSuccess;
}

// The span must lie inside one device allocation known to the HIP runtime.
// A host pointer or a span running past its allocation is rejected here
// instead of faulting the GPU.  Every call reaches this check before its
// launch, so a pending HIP error is reported here as DL_E_HIP, before the
// runtime is asked anything.  `allocation`, if given, receives the allocation.
inline int check_device_span(const void* p, int64_t bytes, Span* allocation = nullptr) {
    if (p == nullptr) return DL_E_INVAL;
    if (hip_error_pending()) return DL_E_HIP;
    hipDeviceptr_t base = nullptr;
    size_t size = 0;
    if (hipMemGetAddressRange(&base, &size, const_cast<void*>(p)) != hipSuccess) {
        (void)hipGetLastError();     // do not leave the failure as a sticky error
        return DL_E_INVAL;
    }
    const uintptr_t b = reinterpret_cast<uintptr_t>(base);
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    if (a < b || bytes < 0 || static_cast<uint64_t>(bytes) > size - (a - b)) return DL_E_INVAL;
    if (allocation != nullptr) *allocation = Span{b, b + size};
    return DL_OK;
}

inline bool aligned_to(const void* p, uintptr_t n) {
    return (reinterpret_cast<uintptr_t>(p) % n) == 0;
}

}  // namespace dlk
