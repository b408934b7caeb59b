// operators_host_driver.cpp -- the operators' host code on a fake HIP runtime.
//
// The host code of the operators (no GPU code) is linked against a fake HIP
// runtime: device memory is host memory, launches are counted and run nothing.
//
// With arguments: the names of the kernels that a call launches, one a line.
//   linear OP M N K          (OP 0, 1, 2: forward, dgrad, wgrad)
//   muon ROWS COLS [ROWS COLS ..]
//
// Without: the optimizers' handles where memory runs out.  Every allocation that a create or a first call makes, of the host or of the
// device, is refused once: the call has to return DDL_E_NOMEM, launch nothing,
// leave no device memory (a first call), no host memory (a create) and no
// error of the runtime behind, and succeed when it is made again.
// Prints "ok N refusals".
#include <hip/hip_runtime_api.h>

#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <new>
#include <string>
#include <vector>

#include "../include/ddl.h"

static long g_host_left = -1, g_device_left = -1;  // until one is refused; < 0: none
static long g_host_live = 0, g_device_live = 0, g_launches = 0;
static hipError_t g_last = hipSuccess;
static bool g_print = false;

// the kernels by the address that launches name; never destroyed
static std::map<const void *, std::string> &kernels() {
    static auto *m = new std::map<const void *, std::string>;
    return *m;
}

static bool refuse(long &left) { return left >= 0 && left-- == 0; }

void *operator new(size_t n) {
    if (refuse(g_host_left))
        throw std::bad_alloc();
    void *p = std::malloc(n ? n : 1);
    if (!p)
        throw std::bad_alloc();
    ++g_host_live;
    return p;
}
// (sorts ask this way for room that they can do without)
void *operator new(size_t n, const std::nothrow_t &) noexcept {
    ++g_host_live;
    return std::malloc(n ? n : 1);
}
void operator delete(void *p) noexcept {
    if (p)
        --g_host_live;
    std::free(p);
}
void operator delete(void *p, size_t) noexcept { operator delete(p); }
void operator delete(void *p, const std::nothrow_t &) noexcept { operator delete(p); }

extern "C" {
hipError_t hipMalloc(void **p, size_t n) {
    *p = nullptr;
    if (refuse(g_device_left))
        return g_last = hipErrorOutOfMemory;
    *p = std::malloc(n ? n : 1);
    ++g_device_live;
    return hipSuccess;
}
hipError_t hipFree(void *p) {
    g_device_live -= p != nullptr;
    std::free(p);
    return hipSuccess;
}
hipError_t hipMemcpy(void *d, const void *s, size_t n, hipMemcpyKind) {
    if (n)
        std::memcpy(d, s, n);
    return hipSuccess;
}
hipError_t hipGetDevice(int *d) {
    *d = 0;
    return hipSuccess;
}
hipError_t hipSetDevice(int) { return hipSuccess; }
hipError_t hipStreamIsCapturing(hipStream_t, hipStreamCaptureStatus *st) {
    *st = hipStreamCaptureStatusNone;
    return hipSuccess;
}
hipError_t hipGetLastError(void) {
    const hipError_t e = g_last;
    g_last = hipSuccess;
    return e;
}
hipError_t hipFuncSetAttribute(const void *, hipFuncAttribute, int) { return hipSuccess; }
hipError_t hipLaunchKernel(const void *f, dim3, dim3, void **, size_t, hipStream_t) {
    ++g_launches;
    if (g_print)
        std::printf("%s\n", kernels()[f].c_str());
    return hipSuccess;
}
// what the compiler's start-up code asks for
void **__hipRegisterFatBinary(const void *) {
    static void *handle;
    return &handle;
}
void __hipUnregisterFatBinary(void **) {}
void __hipRegisterFunction(void **, const void *f, char *, const char *name, unsigned, void *,
                           void *, void *, void *, int *) {
    kernels()[f] = name;
}
void __hipRegisterVar(void **, void *, char *, char *, int, size_t, int, int) {}
hipError_t __hipPopCallConfiguration(dim3 *, dim3 *, size_t *, hipStream_t *) {
    return hipSuccess;
}
}

static void fail(const char *what, long i, int rc) {
    std::printf("FAILED: %s, refusal %ld: returned %d, launches %ld, live %ld on the device and "
                "%ld on the host, error left %d\n",
                what, i, rc, g_launches, g_device_live, g_host_live, (int)g_last);
    std::exit(1);
}

static long g_refusals = 0;

// Refuses the 1st, 2nd, .. allocation of `call` until it makes no more.
template <class Make, class Call, class End>
static void each_refusal(const char *what, long &left, Make make, Call call, End end,
                         bool device_empty) {
    for (long i = 0;; ++i) {
        make();
        const long host = g_host_live, device = g_device_live;
        g_launches = 0;
        left = i;
        int rc = call();
        const bool refused = left < 0;
        left = -1;
        if (refused) {
            ++g_refusals;
            if (rc != DDL_E_NOMEM || g_launches || g_last != hipSuccess || g_host_live != host
                || (device_empty && g_device_live != device))
                fail(what, i, rc);
            rc = call();
        }
        if (rc)
            fail(what, i, rc);
        end();
        if (g_device_live)
            fail(what, i, rc);
        if (!refused)
            return;
    }
}

// The kernels of one linear product over dense binary16 arrays, never touched.
static int linear(int op, size_t m, size_t n, size_t k) {
    void *p = (void *)(uintptr_t)4096;
    const size_t all = (size_t)1 << 40;
    if (op == DDL_LINEAR_FORWARD) {
        ddl_linear_args a = {};
        a.m = m, a.n = n, a.k = k, a.dtype = DDL_F16;
        a.x = a.w = a.y = p;
        a.ldx = a.ldw = k, a.ldy = n;
        return ddl_linear(&a, p, all, nullptr);
    }
    if (op == DDL_LINEAR_DGRAD) {
        ddl_dgrad_args a = {};
        a.m = m, a.n = n, a.k = k, a.dtype = DDL_F16;
        a.dz = a.w = a.dx = p;
        a.lddz = n, a.ldw = a.lddx = k;
        return ddl_linear_dgrad(&a, p, all, nullptr);
    }
    ddl_wgrad_args a = {};
    a.m = m, a.n = n, a.k = k, a.dtype = DDL_F16, a.out_dtype = DDL_F32;
    a.dz = a.x = a.dw = a.db = p;
    a.lddz = n, a.ldx = a.lddw = k;
    return ddl_linear_wgrad(&a, p, all, nullptr);
}

static int muon(int count, char **sides) {
    std::vector<ddl_muon_matrix> mats;
    size_t at = 0;
    for (int i = 0; i + 1 < count; i += 2) {
        mats.push_back({at, std::strtoull(sides[i], nullptr, 10),
                        std::strtoull(sides[i + 1], nullptr, 10), 1.0});
        at += mats.back().rows * mats.back().cols;
    }
    ddl_muon h = nullptr;
    int rc = ddl_muon_create(&h, mats.data(), (int)mats.size());
    float some = 0.0f, *w[] = {&some};
    rc = rc ? rc
            : ddl_muon_step(h, &some, DDL_F32, &some, w, 1, nullptr, 0, 0.1, 0.9, 1, 0.0, nullptr);
    return rc ? rc : ddl_muon_destroy(h);
}

int main(int argc, char **argv) {
    if (argc > 1) {
        g_print = true;
        auto number = [&](int i) { return std::strtoull(argv[i], nullptr, 10); };
        return std::string(argv[1]) == "linear"
                   ? linear((int)number(2), number(3), number(4), number(5))
                   : muon(argc - 2, argv + 2);
    }
    // two short matrices and a long one, whose sums are cut into parts
    const ddl_muon_matrix mats[] = {{0, 40, 48, 1.0}, {1920, 48, 40, 1.0}, {3840, 40, 20000, 1.0}};
    const size_t offs[] = {3, 5000}, counts[] = {4097, 11};
    static float some[4];
    float *w[] = {some, some + 1};
    ddl_muon muon = nullptr;
    ddl_adamw adam = nullptr;
    auto make_muon = [&]() { return ddl_muon_create(&muon, mats, 3); };
    auto make_adam = [&]() { return ddl_adamw_create(&adam, offs, counts, 2); };
    auto end_muon = [&]() { ddl_muon_destroy(muon); };
    auto end_adam = [&]() { ddl_adamw_destroy(adam); };
    auto nothing = []() {};
    for (long *left : {&g_host_left, &g_device_left}) {
        each_refusal("muon create", *left, nothing, make_muon, end_muon, true);
        each_refusal("adamw create", *left, nothing, make_adam, end_adam, true);
        each_refusal("muon step", *left, make_muon, [&]() {
            return ddl_muon_step(muon, some, DDL_F32, some, w, 2, nullptr, 0, 0.1, 0.9, 1, 0.0,
                                 nullptr);
        }, end_muon, true);
        each_refusal("orthogonalise, 16 bits", *left, make_muon, [&]() {
            return ddl_muon_orthogonalise(muon, some, some, DDL_BF16, nullptr);
        }, end_muon, true);
        // a first call for the pairs' memory, which stays where the second
        // type's is refused
        each_refusal("orthogonalise, 32 bits", *left, make_muon, [&]() {
            return ddl_muon_orthogonalise(muon, some, some, DDL_F32, nullptr);
        }, end_muon, false);
        each_refusal("adamw step", *left, make_adam, [&]() {
            return ddl_adamw_step(adam, some, DDL_F16, some, some, w, 2, nullptr, 0, 0.1, 0.9,
                                  0.99, 1e-8, 0.0, 1, nullptr);
        }, end_adam, true);
    }
    std::printf("ok %ld refusals\n", g_refusals);
    return 0;
}
