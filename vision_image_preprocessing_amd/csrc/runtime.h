// runtime.h -- host-side launch plumbing shared by the library's entry
// points: descriptor-table uploads, launch timing events, the dispatch
// counter and HIP error reporting.
#pragma once

#include <hip/hip_runtime.h>

#include <atomic>
#include <cstdint>
#include <initializer_list>

#include "internal.h"

namespace mimo {

extern std::atomic<int64_t> g_dispatches;     // kernel launches made so far
extern thread_local hipEvent_t g_launch_start;  // caller's events, or null
extern thread_local hipEvent_t g_launch_stop;

// Records the caller's timing events around one kernel launch.
template <typename Launch>
hipError_t timed_launch(hipStream_t s, Launch &&launch) {
    hipError_t e = hipSuccess;
    if (g_launch_start && (e = hipEventRecord(g_launch_start, s)) != hipSuccess) return e;
    launch();
    if ((e = hipGetLastError()) != hipSuccess) return e;
    if (g_launch_stop && (e = hipEventRecord(g_launch_stop, s)) != hipSuccess) return e;
    return hipSuccess;
}

// Copies a host table to device memory on `stream` through a pinned
// staging ring (asynchronous; the host buffer may be reused at once).
hipError_t upload_table(const void *table, size_t bytes, void *dst, hipStream_t stream);

// Records a HIP failure as the thread's last error; returns MIMO_E_HIP.
int hip_error(hipError_t e, const char *what);

inline int check_ptr_align(const void *p, uintptr_t align) {
    return (reinterpret_cast<uintptr_t>(p) & (align - 1)) == 0;
}

// Whether two arrays, of so many bytes each, share one.
inline bool arrays_meet(const void *a, int64_t a_bytes, const void *b, int64_t b_bytes) {
    const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
    return a_bytes > 0 && b_bytes > 0 && p < q + uintptr_t(b_bytes) && q < p + uintptr_t(a_bytes);
}

// A dense array of a call's arguments, or none (null).
struct Span {
    const void *p;
    int64_t bytes;
};
// Whether one that is written shares bytes with another that is, or with one
// that is read, without beginning where that begins (some may be the same
// array; who may is for the caller to say).
inline bool overlap_in_part(std::initializer_list<Span> written, std::initializer_list<Span> read) {
    for (const Span *w = written.begin(); w != written.end(); ++w) {
        if (!w->p) continue;
        for (const Span *o = written.begin(); o != w; ++o)
            if (o->p && o->p != w->p && arrays_meet(o->p, o->bytes, w->p, w->bytes)) return true;
        for (const Span &r : read)
            if (r.p && r.p != w->p && arrays_meet(r.p, r.bytes, w->p, w->bytes)) return true;
    }
    return false;
}
// Whether `space` shares bytes with one of the others.
inline bool overlaps_any(const Span &space, std::initializer_list<Span> others) {
    for (const Span &o : others)
        if (o.p && arrays_meet(o.p, o.bytes, space.p, space.bytes)) return true;
    return false;
}

}  // namespace mimo
