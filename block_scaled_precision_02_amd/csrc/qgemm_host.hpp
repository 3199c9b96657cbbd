// qgemm_host.hpp -- what the C entry points share on the host: the error text,
// the device check, the launch hook (defined in qgemm_api.cpp).
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/qgemm.h"

namespace qgemm {

constexpr int64_t LD_LIMIT = (int64_t)1 << 31;

inline bool aligned(const void *p, unsigned a) { return ((uintptr_t)p & (a - 1)) == 0; }

// Set the calling thread's error text and return st.
qgemm_status fail(qgemm_status st, const char *fmt, ...) __attribute__((format(printf, 2, 3), visibility("hidden")));

// gfx950 or a failure.
qgemm_status check_device() __attribute__((visibility("hidden")));

// The launch error that a test asked for, or 0.
int injected_launch_error() __attribute__((visibility("hidden")));

#define TRY(x)                                  \
    do {                                        \
        qgemm_status st_ = (x);                 \
        if (st_ != QGEMM_OK)                    \
            return st_;                         \
    } while (0)

// Every launch goes through here: the kernel launch (f), or the injected
// launch error, which leaves the output and everything else untouched.
template <class F>
qgemm_status launch(F &&f)
{
    if (const int e = injected_launch_error())
        return fail(QGEMM_ERR_HIP, "kernel launch: injected error %d", e);
    const hipError_t e = f();
    if (e != hipSuccess)
        return fail(QGEMM_ERR_HIP, "kernel launch: %s", hipGetErrorString(e));
    return QGEMM_OK;
}

}  // namespace qgemm
