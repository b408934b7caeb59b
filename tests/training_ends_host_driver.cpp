// training_ends_host_driver.cpp -- the cross entropy's and AdamW8's host code on the
// fake HIP runtime of operators_host_driver.cpp.
//
//   ce OP M N K DTYPE OUT   the kernels that a call launches, one a line (OP 0: the
//                           loss, 1: the gradient; OUT: dw's type)
// Without arguments: AdamW8's handles where memory runs out, as the optimizers'
// there.  Prints "ok N refusals".
#define main operators_main
#include "operators_host_driver.cpp"
#undef main

static int ce(int op, size_t m, size_t n, size_t k, int dtype, int out) {
    void *p = (void *)(uintptr_t)4096;
    const size_t all = (size_t)1 << 45;
    ddl_ce_grad_args a = {};
    ddl_ce_args &l = a.layer;
    l.m = m, l.n = n, l.k = k, l.dtype = dtype;
    l.x = l.w = p, l.ldx = l.ldw = k;
    l.target = (const long long *)p;
    l.loss = l.lse = (float *)p;
    if (op == DDL_CE_FORWARD)
        return ddl_cross_entropy(&l, p, all, nullptr);
    a.scale = 1.0;
    a.dx = a.dw = a.db = p, a.lddx = a.lddw = k, a.dw_dtype = out;
    return ddl_cross_entropy_grad(&a, p, all, nullptr);
}

int main(int argc, char **argv) {
    if (argc > 1) {
        g_print = true;
        auto number = [&](int i) { return std::strtoull(argv[i], nullptr, 10); };
        return ce((int)number(2), number(3), number(4), number(5), (int)number(6),
                  (int)number(7));
    }
    const size_t offs[] = {3, 9000}, counts[] = {4097, 11};
    static float some[4];
    static signed char m[4];
    static unsigned char v[4];
    float *w[] = {some, some + 1};
    ddl_adamw8 h = nullptr;
    auto make = [&]() { return ddl_adamw8_create(&h, offs, counts, 2); };
    auto end = [&]() { ddl_adamw8_destroy(h); };
    auto nothing = []() {};
    for (long *left : {&g_host_left, &g_device_left}) {
        each_refusal("adamw8 create", *left, nothing, make, end, true);
        each_refusal("adamw8 step", *left, make, [&]() {
            return ddl_adamw8_step(h, some, DDL_F16, m, v, some, some, w, 2, nullptr, 0, 0.1, 0.9,
                                   0.99, 1e-8, 0.0, 1, nullptr);
        }, end, true);
        each_refusal("adamw8 values", *left, make, [&]() {
            return ddl_adamw8_values(h, m, v, some, some, some, some, nullptr);
        }, end, true);
    }
    std::printf("ok %ld refusals\n", g_refusals);
    return 0;
}
