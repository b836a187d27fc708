// Host helpers shared by the C ABI's translation units (defined in kda_api.cpp): errors,
// descriptor checks, the KDA_CHECK=1 device checks, launch timing records and the cached
// per-stream workspace.
#pragma once
#include <hip/hip_runtime.h>

#include "../../include/kda.h"
#include "kda_launch.hpp"

namespace kda_host {

// Sets the thread's last error and returns st.
kda_status_t fail(kda_status_t st, const char *fmt, ...);
kda_status_t hip_fail(hipError_t e, const char *what);

struct Span {
    uintptr_t lo = 0, hi = 0;  // [lo, hi) in bytes; empty when lo == hi
};
size_t elem_size(int32_t dt);
Span span_of(const kda_tensor_t *t);
bool overlaps(const Span &a, const Span &b);
bool same_view(const kda_tensor_t *a, const kda_tensor_t *b);
int64_t numel(const kda_tensor_t *t);
kda_status_t check_basic(const kda_tensor_t *t, const char *name, bool allow_null);

bool env_on(const char *name);

// The KDA_CHECK=1 device checks, before anything else of the call is enqueued: cu_seqlens
// (when given: cu[0] == 0, non-decreasing, cu[N] == T_tot), the values of g (when given:
// within [g.lo, g.hi], NaN refused) and decode's slot indices (when given: no two requests
// name the same slot in [0, P)).  Zeroes three flags, runs the checks, reads the flags back
// and synchronises the stream; returns KDA_ERR_SHAPE, KDA_ERR_RANGE or KDA_ERR_ALIAS.
struct DeviceChecks {
    const int32_t *cu = nullptr;
    int64_t N = 0, Ttot = 0;
    bool check_g = false;
    kda::CheckG g{};
    const int32_t *slots = nullptr;
    int64_t R = 0, P = 0;
};
// flags: device memory for the three flags, or NULL for the library's own buffer (allocated on
// a device's first check).
kda_status_t run_device_checks(const DeviceChecks &c, hipStream_t st, int32_t *flags);

size_t align256(size_t x);
int device_cus();

// Launch timing (kda_profile_*): brackets launch() with events on st when profiling is on.
bool prof_on();
hipError_t prof_begin(hipStream_t st, hipEvent_t &a, hipEvent_t &b);
hipError_t prof_end(const char *name, hipStream_t st, hipEvent_t a, hipEvent_t b);
template <typename F>
hipError_t timed(const char *name, hipStream_t st, F &&launch)
{
    if (!prof_on()) return launch();
    hipEvent_t a, b;
    hipError_t e = prof_begin(st, a, b);
    if (e != hipSuccess) return e;
    if ((e = launch()) != hipSuccess) return e;
    return prof_end(name, st, a, b);
}

// Calls run(workspace, arg) with the library's workspace of the current device and `stream`,
// grown to `bytes` first; the cache stays locked until run has enqueued its kernels.
kda_status_t with_cached_ws(size_t bytes, void *stream, kda_status_t (*run)(void *ws, void *arg), void *arg);

}  // namespace kda_host
