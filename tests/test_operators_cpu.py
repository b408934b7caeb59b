"""The linear layer and the optimizers without a GPU: sizes, refusals, handles."""
import ctypes
import glob
import os
import re
import subprocess

import pytest
import torch

import sgd_gradient_all_amd as ddl
import test_gpu_operators as gpu_tests
from sgd_gradient_all_amd import _operators as ops

E_NULL, E_ARG, E_BUCKETS, E_ALIGN, E_SCRATCH = -1, -2, -3, -4, -10
# an address that is only checked, never used: every call below is refused
SOME = 1 << 20


def lib():
    return ops._lib()


def forward_args(**kw):
    a = ops.ddl_linear_args()
    a.m, a.n, a.k, a.dtype, a.act = 4, 8, 16, ddl.DDL_F16, 0
    a.x, a.ldx, a.w, a.ldw, a.y, a.ldy = SOME, 16, SOME, 16, SOME, 8
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=ddl.DDL_F32), E_ARG), (dict(dtype=7), E_ARG), (dict(act=5), E_ARG),
    (dict(act=-1), E_ARG), (dict(n=(1 << 22) + 1), E_ARG), (dict(m=(1 << 30) + 1), E_ARG),
    (dict(ldx=15), E_ARG), (dict(ldw=15), E_ARG), (dict(ldy=7), E_ARG),
    (dict(residual=SOME, ldr=7), E_ARG), (dict(z=SOME, ldz=7), E_ARG),
    (dict(x=None), E_NULL), (dict(w=None), E_NULL), (dict(y=None), E_NULL),
    (dict(x=SOME + 1), E_ALIGN), (dict(bias=SOME + 1), E_ALIGN), (dict(y=SOME + 1), E_ALIGN),
])
def test_linear_refusals(kw, code):
    assert lib().ddl_linear(ctypes.byref(forward_args(**kw)), None, 0, None) == code


def test_null_arguments():
    assert lib().ddl_linear(None, None, 0, None) == E_NULL
    assert lib().ddl_linear_dgrad(None, None, 0, None) == E_NULL
    assert lib().ddl_linear_wgrad(None, None, 0, None) == E_NULL
    assert lib().ddl_linear_workspace(0, 1, 1, 1, None) == E_NULL


def test_dgrad_refusals():
    def call(**kw):
        a = ops.ddl_dgrad_args()
        a.m, a.n, a.k, a.dtype, a.act = 4, 8, 16, ddl.DDL_BF16, 0
        a.dz, a.lddz, a.w, a.ldw, a.dx, a.lddx = SOME, 8, SOME, 16, SOME, 16
        for k, v in kw.items():
            setattr(a, k, v)
        return lib().ddl_linear_dgrad(ctypes.byref(a), None, 0, None)
    assert call(act=1) == E_NULL  # an activation without z_prev
    assert call(z_prev=SOME, ldz_prev=16) == E_NULL  # without dz_prev
    assert call(z_prev=SOME, ldz_prev=15, dz_prev=SOME, lddz_prev=16) == E_ARG
    assert call(lddx=15) == E_ARG
    assert call(dx=SOME + 1) == E_ALIGN


def test_wgrad_refusals():
    def call(**kw):
        a = ops.ddl_wgrad_args()
        a.m, a.n, a.k, a.dtype, a.out_dtype = 4096, 8, 16, ddl.DDL_BF16, ddl.DDL_F32
        a.dz, a.lddz, a.x, a.ldx, a.dw, a.lddw = SOME, 8, SOME, 16, SOME, 16
        ws, size = kw.pop("workspace", (SOME, 1 << 30))
        for k, v in kw.items():
            setattr(a, k, v)
        return lib().ddl_linear_wgrad(ctypes.byref(a), ws, size, None)
    assert call(out_dtype=ddl.DDL_F16) == E_ARG  # neither f32 nor the operands' type
    assert call(accumulate=2) == E_ARG
    assert call(dw=None) == E_NULL
    assert call(dw=SOME + 2) == E_ALIGN  # f32 wants 4
    assert call(workspace=(None, 0)) == E_NULL
    assert call(workspace=(SOME, 1)) == E_SCRATCH
    assert call(workspace=(SOME + 8, 1 << 30)) == E_ALIGN


def test_empty_outputs_need_nothing():
    assert lib().ddl_linear(ctypes.byref(forward_args(m=0, x=None, y=None)), None, 0, None) == 0
    assert lib().ddl_linear(ctypes.byref(forward_args(n=0, w=None, y=None)), None, 0, None) == 0


def test_workspace_sizes():
    assert ddl.linear_workspace("forward", 8192, 16384, 4096) == 0  # the card is full as it is
    assert ddl.linear_workspace("forward", 0, 16, 16) == 0
    assert ddl.linear_workspace("wgrad", 4096, 4096, 4096) >= 4096 * 4  # db's partial sums
    # parts of a sum are cut only where they cost less than 64 outputs' worth
    one = ddl.linear_workspace("forward", 1, 4096, 4096)
    assert 0 <= one <= 64 * 4096 * 4 + 256
    with pytest.raises(ValueError):
        ddl.linear_workspace("backward", 1, 1, 1)
    with pytest.raises(ValueError):
        ddl.linear_workspace("forward", -1, 1, 1)
    with pytest.raises(ddl.DDLError) as e:
        ddl.linear_workspace("forward", 1, 1 << 23, 1)
    assert e.value.code == E_ARG


def test_python_refuses_cpu_tensors_and_shapes():
    x, w, y = torch.zeros(2, 3).half(), torch.zeros(4, 3).half(), torch.zeros(2, 4).half()
    with pytest.raises(ValueError, match="GPU tensor"):
        ddl.linear(x, w, y)
    with pytest.raises(ValueError, match="shape"):
        ddl.linear(x[0], w, y)
    with pytest.raises(ValueError, match="GPU tensor"):
        ddl.linear_dgrad(y, w, x)
    with pytest.raises(ValueError, match="GPU tensor"):
        ddl.linear_wgrad(y, x, w)
    with pytest.raises(ValueError, match="activation"):
        ops._act("tanh")
    a = ddl.AdamW([(0, 4)])
    v = torch.zeros(4)
    with pytest.raises(ValueError, match="GPU tensor"):
        a.step(v, v, v, [v], lr=1.0)
    m = ddl.Muon([(0, 2, 2, 1.0)])
    with pytest.raises(ValueError, match="GPU tensor"):
        m.orthogonalise(v, v)
    with pytest.raises(ValueError, match="GPU tensor"):
        m.step(v, v, [v], lr=1.0)


def test_handles():
    a = ddl.AdamW([(5, 7), (12, 0), (20, 3)])
    assert a.need == 23
    h = a.handle
    a.destroy()
    a.destroy()  # twice is once
    assert lib().ddl_adamw_destroy(h) == E_ARG  # not a live handle
    assert lib().ddl_adamw_destroy(None) == E_NULL
    m = ddl.Muon([(0, 3, 5, 1.0), (15, 5, 3, 2.0), (30, 0, 4, 1.0)])
    assert m.need == 30
    h = m.handle
    m.destroy()
    assert lib().ddl_muon_destroy(h) == E_ARG
    assert lib().ddl_muon_orthogonalise(h, SOME, SOME, 0, None) == E_ARG
    for spans in ([(0, 8), (7, 2)], [(0, 1 << 41)], [(4, 2), (4, 2)]):
        with pytest.raises(ddl.DDLError) as e:
            ddl.AdamW(spans)
        assert e.value.code == E_BUCKETS
    with pytest.raises(ddl.DDLError) as e:
        ddl.Muon([(0, 4, 4, 1.0), (15, 2, 2, 1.0)])
    assert e.value.code == E_BUCKETS
    for bad in ((0, 1 << 17, 2, 1.0), (0, 2, 2, float("nan")), (0, 2, 2, float("inf"))):
        with pytest.raises(ddl.DDLError) as e:
            ddl.Muon([bad])
        assert e.value.code == E_ARG
    with pytest.raises(ValueError):
        ddl.Muon([(0, -1, 2, 1.0)])
    with pytest.raises(ValueError):
        ddl.AdamW([(-1, 2)])
    ddl.AdamW([]).destroy()
    ddl.Muon([]).destroy()


def adamw_call(h, **kw):
    d = dict(grad=SOME, type=0, m=SOME, v=SOME, w=[SOME], copy=None, copy_type=0, lr=1e-3,
             b1=0.9, b2=0.99, eps=1e-8, wd=0.0, step=1)
    d.update(kw)
    w = (ctypes.c_void_p * max(1, len(d["w"])))(*d["w"])
    return lib().ddl_adamw_step(h, d["grad"], d["type"], d["m"], d["v"], w, len(d["w"]),
                                d["copy"], d["copy_type"], d["lr"], d["b1"], d["b2"], d["eps"],
                                d["wd"], d["step"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), E_ARG), (dict(step=0), E_ARG), (dict(b1=1.0), E_ARG), (dict(b2=-0.1), E_ARG),
    (dict(eps=-1.0), E_ARG), (dict(lr=float("nan")), E_ARG), (dict(wd=float("inf")), E_ARG),
    (dict(w=[]), E_ARG), (dict(copy=SOME, copy_type=0), E_ARG), (dict(grad=None), E_NULL),
    (dict(m=None), E_NULL), (dict(w=[SOME, None]), E_NULL), (dict(m=SOME + 2), E_ALIGN),
    (dict(w=[SOME + 1]), E_ALIGN), (dict(copy=SOME + 1, copy_type=1), E_ALIGN),
])
def test_adamw_refusals(kw, code):
    a = ddl.AdamW([(0, 4)])
    assert adamw_call(a.handle, **kw) == code


def test_nothing_to_step_is_no_work():
    assert adamw_call(ddl.AdamW([]).handle, grad=None, m=None, v=None, w=[SOME]) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(type=3), E_ARG), (dict(lr=float("nan")), E_ARG), (dict(nesterov=2), E_ARG),
    (dict(mu=float("inf")), E_ARG), (dict(w=[]), E_ARG), (dict(grad=None), E_NULL),
    (dict(momentum=None), E_NULL), (dict(grad=SOME + 1), E_ALIGN),
    (dict(copy=SOME, copy_type=0), E_ARG),
])
def test_muon_refusals(kw, code):
    h = ddl.Muon([(0, 2, 2, 1.0)])
    d = dict(grad=SOME, type=0, momentum=SOME, w=[SOME], copy=None, copy_type=0, lr=1e-3, mu=0.9,
             nesterov=1)
    d.update(kw)
    w = (ctypes.c_void_p * max(1, len(d["w"])))(*d["w"])
    assert lib().ddl_muon_step(h.handle, d["grad"], d["type"], d["momentum"], w, len(d["w"]),
                               d["copy"], d["copy_type"], d["lr"], d["mu"], d["nesterov"], 0.0,
                               None) == code


def test_exchange_still_refuses_bfloat16():
    with pytest.raises(ddl.DDLError):
        ddl.Plan(2, 16, ddl.DDL_BF16)


@pytest.mark.parametrize("spans", [[(0, 10), (5, 0), (6, 3)], [(0, 10), (0, 0), (0, 1)],
                                   [(4, 0), (4, 4), (6, 0), (7, 0), (7, 1)]])
def test_empty_spans_hide_no_overlap(spans):
    with pytest.raises(ddl.DDLError) as e:
        ddl.AdamW(spans)
    assert e.value.code == E_BUCKETS


def test_empty_spans_overlap_nothing():
    a = ddl.AdamW([(0, 10), (5, 0), (10, 3), (13, 0), (12, 0)])
    assert a.need == 13


def test_assembly_declares_m0():
    """Inline assembly that writes m0 names it among its clobbers."""
    csrc = os.path.join(os.path.dirname(ddl.__file__), "csrc")
    found = 0
    for path in glob.glob(os.path.join(csrc, "*")):
        with open(path) as f:
            text = f.read()
        for asm in re.findall(r"\basm\b[^;]*;", text):
            if re.search(r"s_mov_b32 m0", asm):
                found += 1
                assert re.search(r':[^:]*"m0"[^:]*$', asm), f"{path}: {asm}"
    assert found == 2


class OnDevice:
    """A tensor's shape and place, without memory: every call below is refused
    before it would use it."""

    def __init__(self, index, *shape, dtype=torch.float16):
        self.index, self.shape, self.dtype = index, shape, dtype
        self.device = f"cuda:{index}"

    def get_device(self):
        return self.index

    def stride(self, i=None):
        s = [1]
        for n in self.shape[:0:-1]:
            s.insert(0, s[0] * n)
        return tuple(s) if i is None else s[i]

    def numel(self):
        return int(torch.Size(self.shape).numel())

    def is_contiguous(self):
        return True

    def element_size(self):
        return self.dtype.itemsize

    def data_ptr(self):
        return None  # refused below the binding too


@pytest.mark.parametrize("index,current", [(1, 0), (0, 1)])
def test_arrays_of_another_device_are_refused(index, current, monkeypatch):
    """Kernels are launched on the current device; arrays of another one would
    be used from there without its streams' order."""
    monkeypatch.setattr(ops, "_current_device", lambda: current, raising=False)
    h = lambda *s: OnDevice(index, *s)  # noqa: E731
    f = lambda *s: OnDevice(index, *s, dtype=torch.float32)  # noqa: E731
    adam, muon = ddl.AdamW([(0, 4)]), ddl.Muon([(0, 2, 2, 1.0)])
    for call in (lambda: ddl.linear(h(2, 8), h(4, 8), h(2, 4)),
                 lambda: ddl.linear_dgrad(h(2, 4), h(4, 8), h(2, 8)),
                 lambda: ddl.linear_wgrad(h(2, 4), h(2, 8), f(4, 8)),
                 lambda: adam.step(f(4), f(4), f(4), [f(4)], lr=1.0),
                 lambda: muon.orthogonalise(f(4), f(4)),
                 lambda: muon.step(f(4), f(4), [f(4)], lr=1.0)):
        with pytest.raises(ValueError, match="current"):
            call()


@pytest.fixture(scope="module")
def host_driver(tmp_path_factory):
    """The operators' host code on a fake runtime (operators_host_driver.cpp)."""
    tmp = tmp_path_factory.mktemp("operators_host")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    hipcc = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
    csrc, objects = os.path.join(root, "sgd_gradient_all_amd", "csrc"), []
    for name in ("adamw_kernels.hip", "linear_kernels.hip", "muon_kernels.hip"):
        objects.append(str(tmp / (name + ".o")))
        subprocess.run([hipcc, "--offload-arch=gfx950", "--offload-host-only", "-O1", "-std=c++17",
                        "-fPIC", "-c", os.path.join(csrc, name), "-o", objects[-1]], check=True)
    exe = str(tmp / "operators_host")
    # the kernels' code, which is not built here, is the one name left open
    subprocess.run(["g++", "-std=c++17", "-O1", "-D__HIP_PLATFORM_AMD__", "-I/opt/rocm/include",
                    os.path.join(root, "tests", "operators_host_driver.cpp"),
                    os.path.join(csrc, "optimizer.cpp"), *objects, "-o", exe,
                    "-Wl,--unresolved-symbols=ignore-in-object-files"], check=True)

    def run(*args):
        out = subprocess.run([exe, *map(str, args)], capture_output=True, text=True, timeout=60)
        assert out.returncode == 0, out.stdout + out.stderr
        return out.stdout
    return run


def test_handles_where_memory_runs_out(host_driver):
    """Every allocation of the optimizers' host code is refused once."""
    out = host_driver()
    assert re.fullmatch(r"ok \d\d+ refusals\n", out), out


def side_of(name):
    """The side of a product kernel's tile, from its mangled name."""
    return int(re.search(r"Core.*?Li(\d+)ELi(\d+)E", name).group(1))


@pytest.mark.parametrize("op,order", [(0, "mnk"), (1, "mkn"), (2, "nkm")])
def test_large_linear_cases_take_their_tiles(op, order, host_driver):
    """The GPU tests' sizes reach the tiles and the parts of sums that they name."""
    for side, parts, *sizes in gpu_tests.LARGE:
        size = dict(zip(order, sizes))
        names = host_driver("linear", op, size["m"], size["n"], size["k"]).split()
        product, *rest = [x for x in names if "column" not in x]
        assert "linear_kernel" in product and side_of(product) == side
        assert len(rest) == (parts > 1) and all("linear_join" in x for x in rest)
        # the last of the tile's flags: whether rows go through registers
        staged = re.search(r"Lb\dELb\dELb(\d)E", product).group(1) == "1"
        assert staged == (sizes[0] % 8 != 0)


@pytest.mark.parametrize("side,shapes", gpu_tests.MUON_LARGE + [
    (64, [(64, 64)] * 300), (64, [(16, 4096)] * 300), (64, [(300, 900)] * 100),
    (64, [(4096, 16)] * 300), (64, [(4096, 1024)]), (128, [(400, 1600)] * 100),
    (128, [(512, 512)] * 100), (128, [(1024, 1024)] * 26), (256, [(4096, 4096)] * 3)])
def test_muon_takes_the_tile_that_its_matrices_fill(side, shapes, host_driver):
    """Padding is not counted as work: many small matrices keep small tiles."""
    assert gpu_tests.muon_tile(shapes) == side
    names = host_driver("muon", *[n for s in shapes for n in s]).split()
    products = [x for x in names if "product_kernel" in x]
    assert len(products) == 15 and {side_of(x) for x in products} == {side}


@pytest.mark.parametrize("m,slices", [(0, 1), (1, 1), (1000, 1), (1024, 2), (2048, 4),
                                      (1 << 20, 32)])
def test_bias_gradients_of_many_rows_take_several_workgroups(m, slices, host_driver):
    names = host_driver("linear", 2, m, 1000, 64).split()
    assert sum("column_join" in x for x in names) == (slices > 1)
    # workspace: the slices' sums, next to the parts of the product
    alone = ddl.linear_workspace("dgrad", 1000, m, 64)  # the same product without db
    assert ddl.linear_workspace("wgrad", m, 1000, 64) - alone == (slices > 1) * slices * 1000 * 4
