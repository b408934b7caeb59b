// hip_call.h -- HIP calls of the operators, each reported by its own result.
// hipGetLastError after a launch would also report what an earlier call of the
// program left behind, and the operator would stop half way for it.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/ddl.h"

namespace ddl {

// DDL_OK, or `code` for a failed call, which leaves nothing behind for the
// next reader of hipGetLastError.
inline int hip_result(hipError_t e, int code = DDL_E_HIP) {
    if (e == hipSuccess)
        return DDL_OK;
    (void)hipGetLastError();
    return code;
}

template <class P>
struct Given {
    using type = P;
};
template <class... P>
int launch(void (*kernel)(P...), dim3 grid, dim3 block, size_t lds, hipStream_t stream,
           typename Given<P>::type... args) {
    void *pointers[] = {(void *)&args...};
    return hip_result(
        hipLaunchKernel((const void *)kernel, grid, block, pointers, lds, stream));
}

// Dynamic LDS over 64 KB has to be allowed for.
template <class... P>
int allow_lds(void (*kernel)(P...), int bytes) {
    if (bytes <= 65536)
        return DDL_OK;
    return hip_result(hipFuncSetAttribute((const void *)kernel,
                                          hipFuncAttributeMaxDynamicSharedMemorySize, bytes));
}

template <class V>
int device_memory(V **d, size_t count) {
    void *p = nullptr;
    const int rc = hip_result(hipMalloc(&p, count * sizeof(V)), DDL_E_NOMEM);
    *d = rc ? nullptr : (V *)p;
    return rc;
}

}  // namespace ddl
