// Host-side helpers shared by the entry points' sources: status and detail text, plan options, launch records.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <mutex>
#include <vector>

#include "retention.h"

// Launch records: a caller-owned object (ret_options_t.timer); the library keeps none of its own.
struct ret_timer {
    struct Rec {
        const char* name;
        hipEvent_t start, stop;
    };
    std::mutex mu;
    std::vector<Rec> recs;
};

namespace ret {

// Sets the calling thread's detail text (ret_last_error) and returns st.
ret_status_t fail(ret_status_t st, const char* fmt, ...) __attribute__((format(printf, 2, 3)));

// The plan options with the library's defaults filled in (ret_options_t documents each field).
struct Opts {
    int segments = 0, target_wgs = 0, prerotate = -1, onchip = 1, variant = 0;
    int step_cw = 0, step_wr = 0, step_pairs = 0, bwd_direct = 1, step_cache = 0;
    long long chain_spin = 0;
    ret_timer_t* timer = nullptr;
};
Opts resolve(const ret_options_t* o);

struct LaunchTimer {
    hipEvent_t start = nullptr, stop = nullptr;
    hipStream_t stream;
    const char* name;
    ret_timer_t* t;
    LaunchTimer(const char* n, hipStream_t s, const Opts& op) : stream(s), name(n), t(op.timer) {
        if (t && hipEventCreate(&start) == hipSuccess && hipEventCreate(&stop) == hipSuccess)
            (void)hipEventRecord(start, stream);
        else
            t = nullptr;
    }
    void done() {
        if (!t) return;
        (void)hipEventRecord(stop, stream);
        std::lock_guard<std::mutex> lk(t->mu);
        t->recs.push_back({name, start, stop});
    }
};

ret_status_t launch_status(const char* what);

// Whether a launch runs whole: one of 2^32 work-items or more along x runs short without an error, and y and z have their
// own limit.
inline bool grid_fits(unsigned long long x, unsigned long long y, unsigned long long z, int threads) {
    return x * (unsigned)threads < 1ull << 32 && y <= 65535 && z <= 65535;
}

inline bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte (null ranges share none).
inline bool overlaps(const void* a, size_t na, const void* b, size_t nb) {
    if (!a || !b || na == 0 || nb == 0) return false;
    const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
    return x < y + nb && y < x + na;
}

// One buffer of a call. over (written ones): bit j set where it may take the place of the j-th read buffer, that is have
// its start and size. align: 16 bytes, or an element's where kernels access it one element at a time.
struct Buf {
    const char* name;
    const void* p;
    size_t bytes;
    unsigned over = 0, align = 16;
};

// Every written buffer apart from every other buffer of the call, but for the places it may take; all aligned.
template <int NW, int NR>
ret_status_t check_apart(const Buf (&w)[NW], const Buf (&r)[NR]) {
    for (int i = 0; i < NW; ++i) {
        for (int j = i + 1; j < NW; ++j)
            if (overlaps(w[i].p, w[i].bytes, w[j].p, w[j].bytes))
                return fail(RET_ERR_INVALID_ARG, "%s overlaps %s", w[i].name, w[j].name);
        for (int j = 0; j < NR; ++j)
            if (overlaps(w[i].p, w[i].bytes, r[j].p, r[j].bytes) &&
                !((w[i].over >> j & 1) && w[i].p == r[j].p && w[i].bytes == r[j].bytes))
                return fail(RET_ERR_INVALID_ARG, "%s overlaps %s", w[i].name, r[j].name);
    }
    for (const Buf& b : w)
        if ((uintptr_t)b.p % b.align) return fail(RET_ERR_INVALID_ARG, "%s must be %u-byte aligned", b.name, b.align);
    for (const Buf& b : r)
        if ((uintptr_t)b.p % b.align) return fail(RET_ERR_INVALID_ARG, "%s must be %u-byte aligned", b.name, b.align);
    return RET_OK;
}

}  // namespace ret
