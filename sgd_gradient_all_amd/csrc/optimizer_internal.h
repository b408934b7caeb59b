// optimizer_internal.h -- what the optimizers' handles share: spans of flat
// buffers, the registry of live handles, and the device memory of a handle.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <mutex>
#include <vector>

#include "../../include/ddl.h"
#include "hip_call.h"

namespace ddl {

struct Span {
    uint64_t at, count;
};
// A workgroup's part of a span.
struct Chunk {
    uint64_t at;
    uint32_t count;
    uint32_t owner;  // index of the span
};
struct Replicas {
    float *w[DDL_MAX_RANKS];
    int count;
};
constexpr size_t kMaxGrid = 1u << 30;
constexpr uint64_t kMaxElements = 1ull << 40;

inline bool disjoint(std::vector<Span> s) {
    for (const Span &x : s)
        if (x.at > kMaxElements || x.count > kMaxElements)
            return false;
    // empty spans overlap nothing, and between two others would part them
    s.erase(std::remove_if(s.begin(), s.end(), [](const Span &x) { return !x.count; }), s.end());
    std::sort(s.begin(), s.end(), [](const Span &a, const Span &b) { return a.at < b.at; });
    for (size_t i = 1; i < s.size(); ++i)
        if (s[i - 1].at + s[i - 1].count > s[i].at)
            return false;
    return true;
}

// Chunks of up to `size` elements; all but a span's first start at a multiple
// of 8 elements, where 16-byte accesses start for every element type.
inline void cut_chunks(const Span &s, uint32_t size, std::vector<Chunk> &out,
                       uint32_t owner = 0) {
    uint64_t at = s.at, end = s.at + s.count;
    if (at % 8 && at < end) {
        const uint64_t n = std::min<uint64_t>(8 - at % 8, end - at);
        out.push_back({at, (uint32_t)n, owner});
        at += n;
    }
    for (; at < end; at += size)
        out.push_back({at, (uint32_t)std::min<uint64_t>(size, end - at), owner});
}

inline bool float_type(int t) { return t == DDL_F32 || t == DDL_F16 || t == DDL_BF16; }
inline bool aligned_to(const void *p, int t) {
    return (uintptr_t)p % (t == DDL_F32 ? 4 : 2) == 0;
}

inline int take_replicas(float *const *weights, int n, Replicas &r) {
    if (!weights)
        return DDL_E_NULL;
    r.count = n;
    for (int i = 0; i < n; ++i) {
        if (!weights[i])
            return DDL_E_NULL;
        if (!aligned_to(weights[i], DDL_F32))
            return DDL_E_ALIGN;
        r.w[i] = weights[i];
    }
    return DDL_OK;
}

// Handles that a create call returned and no destroy call has freed, so that
// another value is an error code and not a use of freed memory.  hold_handle
// keeps the registry locked: calls on handles are enqueued one at a time.
void register_handle(const void *h);
bool unregister_handle(const void *h);
bool hold_handle(const void *h, std::unique_lock<std::mutex> &lk);

// The device that a handle's memory is on: the one of its first step.
struct Handle {
    int device = -1;

    template <class F>
    int bind(hipStream_t stream, F &&make) {
        int now, rc = hip_result(hipGetDevice(&now));
        if (rc)
            return rc;
        if (device >= 0)
            return now == device ? DDL_OK : DDL_E_DEVICE;
        rc = not_capturing(stream);
        rc = rc ? rc : make();
        if (!rc)
            device = now;
        return rc;
    }
    // the memory has to be there before a capture
    static int not_capturing(hipStream_t stream) {
        hipStreamCaptureStatus st = hipStreamCaptureStatusNone;
        const int rc = hip_result(hipStreamIsCapturing(stream, &st));
        return rc ? rc : st == hipStreamCaptureStatusNone ? DDL_OK : DDL_E_UNBOUND;
    }
    // hipFree waits for the device's work
    template <class... P>
    void release(P *...p) {
        if (device < 0)
            return;
        int now = device;
        (void)hipGetDevice(&now);
        if (now != device)
            (void)hipSetDevice(device);
        ((void)hipFree((void *)p), ...);
        if (now != device)
            (void)hipSetDevice(now);
    }
};

template <class V>
int upload(const std::vector<V> &v, V **d) {
    int rc = device_memory(d, std::max<size_t>(v.size(), 1));
    if (rc)
        return rc;
    rc = hip_result(hipMemcpy(*d, v.data(), v.size() * sizeof(V), hipMemcpyHostToDevice));
    if (rc) {
        (void)hipFree(*d);
        *d = nullptr;
    }
    return rc;
}

}  // namespace ddl
