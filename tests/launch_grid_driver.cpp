// launch_grid_driver.cpp -- the cross entropy's launches on the fake HIP runtime of
// operators_host_driver.cpp, each with its grid:
//
//   OP M N K DTYPE OUT WOFF   as training_ends_host_driver.cpp's ce; w starts WOFF
//                             bytes past a 16-byte boundary
// Prints "<kernel> <workgroups>" a line.
#define main operators_main
#define hipLaunchKernel silent_launch
#include "operators_host_driver.cpp"
#undef hipLaunchKernel
#undef main

extern "C" hipError_t hipLaunchKernel(const void *f, dim3 grid, dim3, void **, size_t,
                                      hipStream_t) {
    std::printf("%s %u\n", kernels()[f].c_str(), grid.x);
    return hipSuccess;
}

int main(int argc, char **argv) {
    if (argc != 8)
        return 2;
    auto number = [&](int i) { return (size_t)std::strtoull(argv[i], nullptr, 10); };
    char *p = (char *)(uintptr_t)4096;
    const size_t all = (size_t)1 << 45;
    ddl_ce_grad_args a = {};
    ddl_ce_args &l = a.layer;
    l.m = number(2), l.n = number(3), l.k = number(4), l.dtype = (int)number(5);
    l.x = p, l.w = p + number(7), l.ldx = l.ldw = l.k;
    l.target = (const long long *)p;
    l.loss = l.lse = (float *)p;
    if (number(1) == DDL_CE_FORWARD)
        return ddl_cross_entropy(&l, p, all, nullptr);
    a.scale = 1.0;
    a.dx = a.dw = a.db = p, a.lddx = a.lddw = l.k, a.dw_dtype = (int)number(6);
    return ddl_cross_entropy_grad(&a, p, all, nullptr);
}
